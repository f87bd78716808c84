"""Sampling, rotary positions and the cache's forks and moves: the refusals that are
found on the host (CPU only: no kernel is launched), and the frequencies."""
import ctypes
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_80_gb300 as sd
from tests import decode_reference as ref

P = ctypes.c_void_p
fake = P(0x1000)
other = P(0x2000)


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_80_gb300 import build

    build.build()
    return sd.load_library()


def test_error_bit():
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "specdec_step.h")).read()
    assert re.search(rf"#define\s+SPECDEC_DEV_ERR_SAMPLE\s+{sd.DEV_ERR_SAMPLE}u\b", text)


def test_sample_refusals(lib):
    def call(x=fake, out=fake, dtype=1, B=2, n=1, V=100, u=fake, tokens=fake):
        return lib.spec_sample(x, out, dtype, B, n, V, None, None, None, None, None, u, tokens, None, None)

    assert call(dtype=2) == 1 and call(B=-1) == 1 and call(n=-1) == 1 and call(V=0) == 1 and call(x=None) == 1
    assert call(u=None) == 1 and call(tokens=None) == 1 and call(out=None, u=None, tokens=None) == 1
    assert call(x=P(0x1001)) == 1 and call(out=P(0x1001)) == 1 and call(dtype=0, x=P(0x1002)) == 1
    assert call(V=(1 << 18) + 1) == 2 and call(n=65) == 2 and call(B=65537) == 2
    assert call(B=0, x=None) == 0


def test_rotary_refusals(lib):
    def call(q=fake, k=fake, dtype=1, T=5, Hq=8, H=2, D=64, qs=(512, 64), ks=(128, 64), pos=fake, turns=fake, R=64, pairs=0, factor=1.0,
             qo=fake, qos=None, ko=fake, kos=None):
        return lib.spec_rotary(q, k, dtype, T, Hq, H, D, *qs, *ks, pos, turns, R, pairs, factor, qo, *(qos or qs), ko, *(kos or ks), None)

    assert call(dtype=7) == 1 and call(T=-1) == 1 and call(Hq=-1) == 1 and call(Hq=0, H=0) == 1 and call(D=0) == 1
    assert call(R=0) == 1 and call(R=63) == 1 and call(R=66) == 1 and call(pairs=2) == 1
    assert call(factor=0.0) == 1 and call(factor=float("nan")) == 1 and call(factor=float("inf")) == 1 and call(factor=-1.0) == 1
    assert call(q=None) == 1 and call(ko=None) == 1 and call(pos=None) == 1 and call(turns=None) == 1 and call(turns=P(0x1004)) == 1
    assert call(q=P(0x1001)) == 1 and call(qs=(-512, 64)) == 1
    assert call(qos=(1024, 64)) == 1                      # in place with other strides
    assert call(qo=other, qos=(32, 64)) == 1 and call(qo=other, qos=(512, 32)) == 1   # rows of an output that overlap
    assert call(qo=other, qos=(64, 64)) == 1 and call(qo=other, qos=(500, 64)) == 1 and call(qs=(64, 64)) == 1   # tokens over heads
    assert call(qs=(64, 319)) == 1                        # heads over tokens
    assert call(D=2000, R=64) == 2 and call(Hq=70000) == 2
    assert call(T=0, q=None) == 0


def test_fork_refusals(lib):
    def call(n=(2, 4), bs=16, width=8, blocks=100, table=fake, kv=fake, held=fake, parent=fake, shares=fake, ring=fake, table_out=other,
             kv_out=other, held_out=other, copies=fake, count=fake, ws=fake, ws_bytes=1 << 30, acc=None):
        return lib.kv_fork(*n, bs, width, blocks, table, kv, acc, held, parent, None, shares, ring, fake, table_out, kv_out, held_out, shares,
                           fake, copies, count, ws, ws_bytes, None, None)

    assert call(n=(-1, 4)) == 1 and call(n=(2, -1)) == 1 and call(width=0) == 1 and call(blocks=0) == 1
    assert call(table=None) == 1 and call(parent=None) == 1 and call(shares=None) == 1 and call(ring=None) == 1 and call(count=None) == 1
    assert call(copies=None) == 1 and call(held_out=None) == 1
    assert call(table_out=fake) == 1 and call(kv_out=fake) == 1 and call(held_out=fake) == 1 and call(acc=other) == 1  # its own inputs
    assert call(bs=20) == 2 and call(n=(65537, 1)) == 2 and call(n=(1, 65537)) == 2 and call(blocks=1 << 27) == 2 and call(width=1 << 27) == 2
    need = sd.page_workspace_bytes(100)
    assert call(ws=None) == 3 and call(ws_bytes=need - 1) == 3 and call(ws=P(0x1008)) == 3


def test_compact_refusals(lib):
    def call(B=2, width=8, blocks=100, table=fake, held=fake, renamed=fake, copies=fake, ring=fake, ws=fake, ws_bytes=1 << 30):
        return lib.kv_compact(B, width, blocks, table, held, fake, ring, fake, fake, fake, ring, fake, renamed, copies, fake, ws, ws_bytes,
                              None, None)

    assert call(B=-1) == 1 and call(width=0) == 1 and call(blocks=0) == 1 and call(table=None) == 1 and call(held=None) == 1
    assert call(renamed=None) == 1 and call(copies=None) == 1 and call(ring=None) == 1
    assert call(B=65537) == 2 and call(blocks=(1 << 27) + 1) == 2
    assert call(ws=None) == 3 and call(ws_bytes=sd.page_workspace_bytes(100) - 1) == 3


def test_copy_refusals(lib):
    def call(copies=fake, count=fake, cap=4, layers=1, caches=(0x1000,) * 4, blocks=100, bs=16, H=8, D=64):
        c = (P * 4)(*caches) if caches is not None else None
        return lib.kv_copy(copies, count, cap, layers, c, blocks, bs, H, D, None)

    assert call(cap=-1) == 1 and call(layers=-1) == 1 and call(blocks=0) == 1 and call(H=0) == 1
    assert call(copies=None) == 1 and call(count=None) == 1 and call(caches=None) == 1
    assert call(caches=(0x1000, 0, 0x1000, 0x1000)) == 1 and call(caches=(0x1008, 0x1000, 0x1000, 0x1000)) == 1
    assert call(caches=(0x1000, 0x1000, 0x1002, 0x1000)) == 1
    assert call(bs=8) == 2 and call(D=96) == 2 and call(blocks=1 << 28) == 2
    assert call(cap=0, copies=None) == 0 and call(layers=0, caches=None) == 0


def test_binding_rejects_wrong_tensors_on_the_host():
    i32 = torch.int32
    z = lambda *s, dtype=i32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    x = torch.zeros(2, 3, 100)
    with pytest.raises(ValueError):
        sd.spec_sample(x)  # neither tokens nor rows
    with pytest.raises(ValueError):
        sd.spec_sample(x[0], out=x[0])
    with pytest.raises(ValueError):
        sd.spec_sample(x, out=x, tokens=z(2, 3))
    with pytest.raises(ValueError):
        sd.spec_sample(x, uniform=torch.zeros(2, 2))
    with pytest.raises(TypeError):
        sd.spec_sample(x, uniform=torch.zeros(2, 3), top_k=z(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        sd.spec_sample(x, out=torch.zeros(2, 3, 99))
    with pytest.raises(ValueError):
        sd.spec_sample(x, out=x)  # not on a GPU
    q = torch.zeros(5, 4, 64)
    turns = z(32, dtype=torch.int64)
    with pytest.raises(ValueError):
        sd.spec_rotary(None, None, z(5), turns)
    with pytest.raises(ValueError):
        sd.spec_rotary(q, None, z(5), turns, layout="quarter")
    with pytest.raises(TypeError):
        sd.spec_rotary(q, q.half(), z(5), turns)
    with pytest.raises(ValueError):
        sd.spec_rotary(q, q[:4], z(5), turns)
    with pytest.raises(ValueError):
        sd.spec_rotary(q.transpose(1, 2), None, z(5), turns)
    with pytest.raises(ValueError):
        sd.spec_rotary(q, None, z(4), turns)
    with pytest.raises(TypeError):
        sd.spec_rotary(q, None, z(5), z(32))
    with pytest.raises(ValueError):
        sd.spec_rotary(q, None, z(5), z(33, dtype=torch.int64))
    with pytest.raises(ValueError):
        sd.spec_rotary(q, None, z(5), turns, k_out=q)
    with pytest.raises(ValueError):
        sd.spec_rotary(q, None, z(5), turns)  # not on a GPU
    with pytest.raises(ValueError):
        sd.kv_fork(z(4, 8), z(5), z(4), z(4), z(20), z(20), z(2), 16)
    with pytest.raises(ValueError):
        sd.kv_fork(z(4, 8), z(4), z(4), z(6), z(19), z(20), z(2), 16)
    with pytest.raises(TypeError):
        sd.kv_fork(z(4, 8), z(4), z(4), z(6, dtype=torch.int64), z(20), z(20), z(2), 16)
    with pytest.raises(ValueError):
        sd.kv_compact(z(4, 8), z(4), z(19), z(20), z(2))
    cache = torch.zeros(3, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        sd.kv_layers([])
    with pytest.raises(ValueError):
        sd.kv_layers([(cache, cache, torch.zeros(3, 2), torch.zeros(3, 2))])  # not on a GPU
    with pytest.raises(ValueError):
        sd.kv_layers([(cache, cache, torch.zeros(3, 2), torch.zeros(3, 1))])


def test_frequencies():
    freq, factor = sd.rotary_frequencies(8, base=10000.0)
    assert factor == 1.0 and freq == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15)
    assert sd.rotary_frequencies(8, scaling=dict(type="linear", factor=4))[0] == pytest.approx([f / 4 for f in freq], rel=1e-15)
    ntk = sd.rotary_frequencies(8, scaling=dict(type="ntk", factor=4))[0]
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(freq[-1] / 4, rel=1e-12)  # the slowest pair is scaled by the factor
    yarn, factor = sd.rotary_frequencies(128, scaling=dict(type="yarn", factor=16, original=8192))
    plain = sd.rotary_frequencies(128)[0]
    assert factor == pytest.approx(0.1 * math.log(16) + 1) and yarn[0] == plain[0] and yarn[-1] == pytest.approx(plain[-1] / 16)
    assert all(a <= b * (1 + 1e-12) for a, b in zip(yarn, plain)) and all(a >= b / 16 * (1 - 1e-12) for a, b in zip(yarn, plain))
    bands, _ = sd.rotary_frequencies(128, scaling=dict(type="bands", factor=8, original=8192))
    for f, g in zip(plain, bands):
        turns = 8192 * f / (2 * math.pi)
        assert g == pytest.approx(f if turns >= 4 else f / 8 if turns <= 1 else (f * (turns - 1) + f / 8 * (4 - turns)) / 3)


@pytest.mark.parametrize("bad", [dict(type="linear"), dict(type="cubic", factor=2), dict(type="linear", factor=0.5),
                                 dict(type="yarn", factor=4), dict(type="bands", factor=4, original=100, low=4, high=4),
                                 dict(type="linear", factor=2, original=7), dict(type="yarn", factor=4, original=10, fast=1, slow=2)])
def test_frequencies_refuse(bad):
    with pytest.raises(ValueError):
        sd.rotary_frequencies(64, scaling=bad)
    with pytest.raises(ValueError):
        sd.rotary_frequencies(63)
    with pytest.raises(ValueError):
        sd.rotary_frequencies(64, base=1.0)


def test_turns_are_the_frequencies_in_64_bits():
    turns, _ = sd.rotary_turns(128, base=500000.0, device="cpu")
    freq, _ = sd.rotary_frequencies(128, base=500000.0)
    got = [(int(t) & (2 ** 64 - 1)) / 2.0 ** 64 * 2 * math.pi for t in turns]
    assert got == pytest.approx(freq, rel=1e-12)


def test_plain_sampling_by_hand():
    row = [0.0, math.log(2), math.log(4), math.log(2)]  # weights 1, 2, 4, 2; order 2, 1, 3, 0
    assert ref.sample_row(row, u=0.0) == ({0, 1, 2, 3}, 2)
    assert ref.sample_row(row, k=2, u=0.9) == ({1, 2}, 1)
    assert ref.sample_row(row, p=0.6, u=0.99)[0] == {2, 1}
    assert ref.sample_row(row, m=0.45)[0] == {1, 2, 3}
    assert ref.sample_row(row, T=0.0, u=0.3) == ({2}, 2)
    assert ref.sample_row([-math.inf, math.nan], u=0.3) == (set(), -1)


def test_plain_fork_by_hand():
    table = np.array([[3, 5, -1], [7, -1, -1]])
    # 20 tokens in blocks 3 and 5 go on three times, request 1 ends
    f = ref.fork(table, [20, 9], None, [2, 1], [0, 0, 0], None, [0] * 10, np.array([0, 1, 2, 4, -1, -1, -1, -1, -1, -1]), [0, 4], 16)
    assert f["copies"] == [(5, 0), (5, 1)] and f["block_table"].tolist() == [[3, 0, -1], [3, 1, -1], [3, 5, -1]]
    assert f["shares"][3] == 2 and f["shares"][5] == 0 and f["ring_state"].tolist() == [2, 3] and f["ring"][4] == 7 and not f["bad"]
