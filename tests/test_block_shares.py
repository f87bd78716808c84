"""kv_block_step beside shared blocks: requests that would write or give back a block
that others hold are refused, others are served as ever."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_80_gb300 as sd
from tests import step_reference as ref

P = ctypes.c_void_p
fake = P(0x1000)


def plain(c, bs, capacity, shares):
    """What the step leaves: the requests that must not be served are given a length and an ask that change
    nothing, and everything else is the step without shares."""
    new, held = c["new"].copy(), c["held"]
    refused = []
    for b in range(len(held)):
        tokens = int(c["kv_len"][b]) + max(int(c["accepted"][b]), -1) + 1
        want = max(int(new[b]), 0)
        kept = tokens if new[b] >= 0 else 0
        first = kept // bs if want else -(-kept // bs)
        if any(shares[c["table"][b, j]] > 0 for j in range(first, int(held[b]))):
            refused.append(b)
    order = [b for b in range(len(held)) if b not in refused]
    sub = ref.block_step(c["table"][order], c["kv_len"][order], held[order], new[order], c["ring"], c["state"], bs, capacity,
                         c["accepted"][order])
    out = dict(ring=sub["ring"], ring_state=sub["ring_state"], slot_map=sub["slot_map"], positions=sub["positions"], bad=sub["bad"] or bool(refused))
    kv, h, cu, cub, at = [], [], [0], [0], {b: i for i, b in enumerate(order)}
    table = c["table"].copy()
    for b in range(len(held)):
        if b in at:
            i = at[b]
            kv.append(sub["kv_len"][i])
            h.append(sub["held"][i])
            cu.append(sub["cu_tokens"][i + 1])
            cub.append(sub["cu_blocks"][i + 1])
            table[b] = sub["table"][i]
        else:
            kv.append(int(c["kv_len"][b]) + max(int(c["accepted"][b]), -1) + 1)
            h.append(int(held[b]))
            cu.append(cu[-1])
            cub.append(cub[-1])
    out.update(kv_len=kv, held=h, cu_tokens=cu, cu_blocks=cub, table=table, refused=refused)
    return out


def _case(rng, B, W, bs, spare, most, some=0.3):
    """Requests whose first blocks may be others' too; ends, waits and new tokens."""
    held = rng.integers(0, W + 1, B)
    N = int(held.sum()) + spare
    ids = list(rng.permutation(N))
    table, shares = np.full((B, W), -1, dtype=np.int32), np.zeros(N, dtype=np.int64)
    for b in range(B):
        c = 0
        if b and rng.random() < some:
            q = int(rng.integers(0, b))
            c = int(rng.integers(0, min(held[b], held[q]) + 1))
            table[b, :c] = table[q, :c]
            shares[table[b, :c]] += 1
        for j in range(c, held[b]):
            table[b, j] = ids.pop()
    head = int(rng.integers(0, N))
    ring = np.full(N, -1, dtype=np.int32)
    ring[(head + np.arange(len(ids))) % N] = ids
    tokens = np.array([rng.integers(0, h * bs + 1) for h in held])
    accepted = np.minimum(rng.integers(-1, 4, B), tokens - 1)
    i32 = lambda x: np.asarray(x, dtype=np.int32)  # noqa: E731
    new = np.where(rng.random(B) < 0.3, -1, rng.integers(0, most + 1, B))
    return dict(table=table, held=i32(held), kv_len=i32(tokens - np.maximum(accepted, -1) - 1), accepted=i32(accepted), new=i32(new), ring=ring,
                state=i32([head, len(ids)])), i32(shares)


def test_refusals():
    from speculative_decoding_verification_80_gb300 import build

    build.build()
    lib = sd.load_library()

    def call(B=4, bs=16, width=8, blocks=100, kv=fake, cap=10, ring=fake):
        return lib.kv_block_step_shared(B, bs, width, blocks, kv, None, fake, fake, fake, ring, fake, fake, fake, fake, fake, fake, fake, fake, fake,
                                        cap, None, None)

    assert call(B=-1) == 1 and call(width=0) == 1 and call(cap=-1) == 1 and call(kv=None) == 1 and call(ring=None) == 1
    assert call(bs=24) == 2 and call(B=65537) == 2 and call(blocks=1 << 28) == 2
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    for shares in (z(19), z(20, dtype=torch.int64), z(20)):  # (the last is not on a GPU, as the others)
        with pytest.raises((ValueError, TypeError)):
            sd.kv_block_step(z(4, 8), z(4), z(4), z(4), z(20), z(2), 16, 10, shares=shares)


def _check(c, shares, bs, capacity, alias):
    want = plain(c, bs, capacity, shares)
    dev = lambda x: torch.as_tensor(np.ascontiguousarray(x)).cuda()  # noqa: E731
    table, ring, kv, held, state = (dev(c[k]) for k in ("table", "ring", "kv_len", "held", "state"))
    B, out = len(c["held"]), None
    if alias:
        e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        out = sd.BlockStep(kv, held, state, e(B + 1), e(B + 1), e(capacity), e(capacity))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    step = sd.kv_block_step(table, kv, held, dev(c["new"]), ring, state, bs, capacity, accepted_len=dev(c["accepted"]), out=out, error_word=err,
                            shares=dev(shares))
    torch.cuda.synchronize()
    for name in ("kv_len", "held", "ring_state", "cu_tokens", "cu_blocks", "slot_map", "positions"):
        assert getattr(step, name).tolist() == list(want[name]), name
    got = table.cpu().numpy()
    for b in range(B):
        assert (got[b, :want["held"][b]] == want["table"][b, :want["held"][b]]).all()
    h, n = want["ring_state"]
    at = (h + np.arange(n)) % len(c["ring"])
    free = ring.cpu().numpy()[at]
    assert (free == want["ring"][at]).all()
    named = {int(x) for b in range(B) for x in got[b, :want["held"][b]]}
    assert not named & {int(x) for x in free} and len(set(free.tolist())) == len(free)  # no block is both held and free
    assert err.item() == (sd.DEV_ERR_BLOCKS if want["bad"] else 0)
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("B,W,bs,most", [(1, 1, 16, 3), (2, 3, 16, 20), (9, 5, 32, 8), (40, 70, 16, 300), (700, 4, 64, 5), (2100, 9, 16, 40)])
def test_steps_beside_shared_blocks(B, W, bs, most, alias):
    rng = np.random.default_rng(B * 3 + W)
    for some in (0.0, 0.5):
        c, shares = _case(rng, B, W, bs, spare=B * (most // bs + 2), most=most, some=some)
        want = _check(c, shares, bs, B * most, alias)
        assert some == 0.5 or not want["refused"]
        assert some == 0.0 or B < 9 or want["refused"]


@pytest.mark.gpu
def test_an_end_of_a_shared_request_gives_nothing_back():
    """Two requests share two blocks: neither may end here, both go on in blocks of their own."""
    c = dict(table=np.array([[1, 2, 3], [1, 2, 4]], dtype=np.int32), held=np.array([3, 3], dtype=np.int32),
             kv_len=np.array([40, 33], dtype=np.int32), accepted=np.array([-1, -1], dtype=np.int32), new=np.array([-1, 20], dtype=np.int32),
             ring=np.array([0, 5, -1, -1, -1, -1], dtype=np.int32), state=np.array([0, 2], dtype=np.int32))
    shares = np.array([0, 1, 1, 0, 0, 0], dtype=np.int32)
    want = _check(c, shares, 16, 40, False)
    # (request 1's 53 tokens are 4 blocks, for which a row of 3 has no room either)
    assert want["refused"] == [0] and want["held"] == [3, 3] and want["kv_len"] == [40, 33] and want["ring_state"] == [0, 2]
    wide = dict(c, table=np.concatenate([c["table"], np.full((2, 1), -1, dtype=np.int32)], 1))
    want = _check(wide, shares, 16, 40, False)
    assert want["refused"] == [0] and want["held"] == [3, 4] and want["kv_len"] == [40, 33] and want["ring_state"] == [1, 1]
    # a request that is cut back into a shared block does not write it
    c["kv_len"][1], c["new"][:] = 20, [0, 5]
    want = _check(c, shares, 16, 40, True)
    assert want["refused"] == [1] and want["cu_tokens"] == [0, 0, 0]


@pytest.mark.gpu
def test_a_step_after_a_fork_serves_all():
    """kv_fork leaves no request that the next step refuses; ends go through kv_fork."""
    rng = np.random.default_rng(5)
    N, bs, W = 400, 16, 12
    i32 = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
    held = rng.integers(1, 8, 6)
    table, used = np.full((6, W), -1), 0
    for b in range(6):
        table[b, :held[b]] = np.arange(used, used + held[b])
        used += held[b]
    ring, state = i32(list(range(used, N)) + [-1] * used), i32([0, N - used])
    tokens = [int(rng.integers((h - 1) * bs + 1, h * bs + 1)) for h in held]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = sd.kv_fork(i32(table), i32(tokens), i32(held), i32(np.arange(24) % 6), i32(np.zeros(N)), ring, state, bs, error_word=err)
    step = sd.kv_block_step(f.block_table, f.kv_len, f.held, i32(np.full(24, 5)), ring, f.ring_state, bs, 24 * 5, error_word=err, shares=f.shares)
    torch.cuda.synchronize()
    assert err.item() == 0 and step.cu_tokens[-1].item() == 24 * 5
    # one of them ends here: refused; by a fork: its own blocks alone go back
    ends = np.full(24, 0)
    ends[3] = -1
    again = sd.kv_block_step(f.block_table, step.kv_len, step.held, i32(ends), ring, step.ring_state, bs, 8,
                             accepted_len=i32(np.full(24, 4)), error_word=err, shares=f.shares)
    torch.cuda.synchronize()
    assert err.item() == sd.DEV_ERR_BLOCKS and again.held.tolist() == step.held.tolist() and again.ring_state.tolist() == step.ring_state.tolist()
