"""The operators around the verify step: the header, the exports and the
refusals that are found on the host (CPU only: no kernel is launched), and the
plain implementations that the GPU tests compare with."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import speculative_decoding_verification_80_gb300 as sd
from speculative_decoding_verification_80_gb300 import step
from tests import step_reference as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "specdec_step.h")
P = ctypes.c_void_p
fake = P(0x1000)


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_80_gb300 import build

    build.build()
    return sd.load_library()


def _text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_exports_and_constants(lib):
    names = re.findall(r"specdec_status_t\s+(\w+)\(", _text())
    assert sorted(names) == sorted(step.STEP_EXPORTS)
    for name in names:
        assert hasattr(lib, name)
    text = open(HEADER).read()
    for name, value in (("SPECDEC_DEV_ERR_BLOCKS", sd.DEV_ERR_BLOCKS), ("SPECDEC_DEV_ERR_PENALTY", sd.DEV_ERR_PENALTY)):
        assert re.search(rf"#define\s+{name}\s+{value}u\b", text)
    assert sd.ATTENTION_WORKSPACE_BYTES == 64 << 20
    assert "#define SPECDEC_ATTENTION_WORKSPACE_BYTES (64u << 20)" in text


def test_block_step_refusals(lib):
    def call(B=4, bs=16, width=8, blocks=100, kv=fake, cap=10, slots=fake, ring=fake):
        return lib.kv_block_step(B, bs, width, blocks, kv, None, fake, fake, fake, ring, fake, fake, fake, fake, fake, fake,
                                 slots, fake, cap, None, None)

    assert call(B=-1) == 1 and call(width=0) == 1 and call(blocks=0) == 1 and call(cap=-1) == 1
    assert call(kv=None) == 1 and call(ring=None) == 1 and call(slots=None) == 1
    assert call(bs=24) == 2 and call(bs=256) == 2 and call(B=65537) == 2
    assert call(blocks=1 << 28) == 2      # slots past 32 bits
    assert call(width=1 << 28) == 2
    assert call(B=0, kv=None) == 0


def test_append_refusals(lib):
    def call(k=fake, dtype=1, T=5, H=8, D=128, ts=1024, hs=128, blocks=100, bs=16, cache=fake, slots=fake):
        return lib.kv_append(k, fake, dtype, T, H, D, ts, hs, 1024, 128, slots, blocks, bs, cache, fake, fake, fake, None)

    assert call(dtype=5) == 1 and call(T=-1) == 1 and call(H=0) == 1 and call(k=None) == 1 and call(slots=None) == 1
    assert call(cache=None) == 1
    assert call(D=96) == 2 and call(bs=8) == 2 and call(blocks=1 << 28) == 2
    assert call(k=P(0x1008)) == 1         # 16-byte alignment
    assert call(ts=1020) == 1 and call(hs=4) == 1 and call(ts=-1024) == 1
    assert call(T=0, k=None) == 0


def test_attention_refusals(lib):
    def call(q=fake, stride=8192, T=5, Hq=64, H=8, D=128, B=2, table=fake, width=8, blocks=100, bs=16, scale=0.0, out=fake,
             ws=fake, ws_bytes=64 << 20):
        return lib.spec_attention(q, stride, T, Hq, H, D, B, fake, fake, table, width, blocks, bs, fake, fake, fake, fake,
                                  scale, out, ws, ws_bytes, None)

    assert call(T=-1) == 1 and call(B=-1) == 1 and call(Hq=0) == 1 and call(Hq=12) == 1 and call(width=0) == 1
    assert call(q=None) == 1 and call(table=None) == 1 and call(out=None) == 1
    assert call(stride=8190) == 1 and call(stride=4096) == 1 and call(q=P(0x1002)) == 1
    assert call(scale=-1.0) == 1 and call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(D=80) == 2 and call(bs=48) == 2 and call(blocks=1 << 28) == 2
    assert call(ws=None) == 3 and call(ws_bytes=1 << 20) == 3 and call(ws=P(0x1004)) == 3
    assert call(T=0, q=None) == 0 and call(B=0, q=None) == 0


def test_process_logits_refusals(lib):
    def call(x=fake, out=fake, dtype=1, B=2, n=1, V=100, S=4, hist=fake, drafts=fake, bias=None, ids=None, nb=0, mask=None,
             mc=0, mr=None):
        return lib.spec_process_logits(x, out, dtype, B, n, V, hist, S, fake, fake, drafts, None, None, None, None, bias, ids,
                                       fake, nb, mask, mc, mr, None, None)

    assert call(dtype=3) == 1 and call(B=-1) == 1 and call(V=0) == 1 and call(x=None) == 1 and call(out=None) == 1
    assert call(hist=None) == 1 and call(drafts=None) == 1 and call(S=-1) == 1
    assert call(bias=fake, nb=3) == 1 and call(nb=-1) == 1
    assert call(mask=fake, mc=2) == 1 and call(mr=fake) == 1
    assert call(x=P(0x1001)) == 1
    assert call(V=1 << 20) == 2 and call(n=65) == 2 and call(B=65537) == 2
    assert call(B=0, x=None) == 0


def test_binding_rejects_wrong_tensors_on_the_host():
    i32 = torch.int32
    z = lambda *s, dtype=i32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError):
        sd.kv_block_step(z(4, 8), z(5), z(4), z(4), z(20), z(2), 16, 10)
    with pytest.raises(TypeError):
        sd.kv_block_step(z(4, 8), z(4), z(4), z(4, dtype=torch.int64), z(20), z(2), 16, 10)
    with pytest.raises(ValueError):
        sd.kv_block_step(z(4, 8), z(4), z(4), z(4), z(20), z(3), 16, 10)
    cache = torch.zeros(3, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.zeros(3, 2)
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        sd.kv_append(k, k, z(5), cache.float(), cache, scale, scale)
    with pytest.raises(ValueError):
        sd.kv_append(k[:, :, :32], k[:, :, :32], z(5), cache, cache, scale, scale)
    with pytest.raises(ValueError):
        sd.kv_append(k, k, z(4), cache, cache, scale, scale)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        sd.spec_attention(q.float(), z(3), z(2), z(2, 4), cache, cache, scale, scale)
    with pytest.raises(ValueError):
        sd.spec_attention(q, z(2), z(2), z(2, 4), cache, cache, scale, scale)
    with pytest.raises(ValueError):
        sd.spec_attention(q, z(3), z(2), z(2, 4), cache, cache, scale, scale, scale=0.0)
    x = torch.zeros(2, 3, 100)
    with pytest.raises(ValueError):
        sd.spec_process_logits(x)  # rows after the first need the drafts
    with pytest.raises(ValueError):
        sd.spec_process_logits(x[:, :1], mask=z(2, 3), mask_rows=z(2, 1))
    with pytest.raises(ValueError):
        sd.spec_process_logits(x[:, :1], history=z(2, 8))
    with pytest.raises(ValueError):
        sd.spec_process_logits(x[:, :1].contiguous(), z(2, 8), z(2), z(2))  # not on a GPU


def test_plain_codes_agree_with_torch():
    x = torch.cat([torch.randn(4000, generator=torch.Generator().manual_seed(1)) * 10 ** s for s in (-3, -1, 0, 1, 2)])
    x = torch.cat([x.clamp(-448, 448), torch.tensor(ref.VALUES[:127], dtype=torch.float32),
                   torch.tensor((ref.VALUES[:126] + ref.VALUES[1:127]) / 2, dtype=torch.float32)])
    got = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (ref.to_e4m3(x.numpy()) == got).all()
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).float().numpy(), ref.VALUES, equal_nan=True)


def test_plain_scale_is_the_least_power_of_two():
    for amax in (1e-30, 2.0 ** -9, 1.0, 1.75, 447.9, 448.0, 448.1, 1e20):
        s = ref.pow2_scale(amax)
        assert amax <= 448 * s and amax > 448 * s / 2


def test_step_refuses_what_its_counters_cannot_hold(lib):
    # a history of 2^29 ids: a token's count keeps 29 bits
    def logits(S):
        return lib.spec_process_logits(fake, fake, 1, 2, 0, 100, fake, S, fake, fake, None, None, None, None, None, None, None,
                                       None, 0, None, 0, None, None, None)

    assert logits(1 << 29) == 2
    # tiles of positions times heads and groups of rows: their cost keeps 31 bits
    def attention(T, width):
        return lib.spec_attention(fake, 8192, T, 64, 8, 128, 1, fake, fake, fake, width, 100, 16, fake, fake, fake, fake, 0.0,
                                  fake, fake, 64 << 20, None)

    assert attention(1 << 20, 1 << 26) == 2


def test_attention_refuses_positions_past_32_bits(lib):
    def attention(T, width):
        return lib.spec_attention(fake, 8, T, 1, 1, 64, 1, fake, fake, fake, width, 100, 16, fake, fake, fake, fake, 0.0, fake,
                                  fake, 64 << 20, None)

    # (the token stride is refused where the sizes are not)
    assert attention(16, (1 << 27) - 1) == 2 and attention(1 << 20, (1 << 27) - 1000) == 2
    assert attention(15, (1 << 27) - 1) == 1


def test_attention_refuses_a_scale_whose_product_with_log2_e_overflows(lib):
    def attention(scale, stride=8):
        return lib.spec_attention(fake, stride, 5, 1, 1, 64, 1, fake, fake, fake, 8, 100, 16, fake, fake, fake, fake, scale, fake,
                                  None, 64 << 20, None)

    # (without a workspace the call goes no further)
    assert attention(2.9e38, 64) == 1 and attention(2.37e38, 64) == 1 and attention(2.3e38, 64) == 3
