"""GPU tests of calls of sampling, rotary positions, forks and compaction that are
allowed and easily forgotten: workspaces that several pools share, kept logits to
the bit, the largest temperatures, far strides."""
import numpy as np
import pytest
import torch

from tests import test_gpu_decode_ops as ops

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_80_gb300")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sd.load_library()


@pytest.mark.parametrize("order", [("compact", "fork"), ("fork", "compact"), ("compact", "compact"), ("fork", "fork")])
@pytest.mark.parametrize("sizes", [(100, 200), (200, 100), (33, 5000), (5000, 64, 4999, 33, 5000)])
def test_one_workspace_for_pools_of_several_sizes(sizes, order):
    rng = np.random.default_rng(sum(sizes) + len(order[0]))
    ws = sd.new_page_workspace(max(sizes))
    for i in range(2 * len(sizes)):
        N, what = sizes[i % len(sizes)], order[i % 2]
        W = 4
        c = ops._pool(rng, max(1, N // 8), W, 16, spare=0)
        spare = N - len(c["ring"])
        assert spare > 0
        c["ring"] = np.concatenate([np.full(spare, -1), c["ring"]])
        c["shares"] = np.concatenate([c["shares"], np.zeros(spare, dtype=np.int64)])
        # the new ids are free, and so are those that were
        free = set(range(N)) - {int(x) for p, h in enumerate(c["held"]) for x in c["table"][p, :h]}
        c["ring"] = np.array(sorted(free) + [-1] * (N - len(free)))
        c["state"] = np.array([0, len(free)])
        if what == "fork":
            P = len(c["held"])
            want = ops._check_fork(c, rng.integers(-1, P, P + 3), 16, ws=ws)
            ops._consistent(want, None, 16)
        else:
            assert not ops._check_compact(c, ws=ws)["bad"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [999, 5003, 70001])
def test_kept_logits_keep_their_bits(V, dtype):
    """-0 stays -0, whichever way a row goes: zeros that fill a bin, beside NaN, infinities and finite logits."""
    rng = np.random.default_rng(V)
    zeros = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    high = zeros.copy()
    high[rng.integers(0, V, 40)] = 5000.0 + 32 * rng.integers(0, 9, 40)
    nan = np.where(rng.random(V) < 0.1, np.nan, zeros)
    some = np.where(rng.random(V) < 0.2, zeros, rng.normal(0, 1, V))
    tiny = np.where(rng.random(V) < 0.5, zeros, rng.normal(0, 1e-8, V))
    none = np.where(rng.random(V) < 0.5, zeros, -np.inf)
    word = torch.int16 if dtype is torch.bfloat16 else torch.int32
    for name, row in dict(zeros=zeros, high=high, nan=nan, some=some, tiny=tiny, none=none).items():
        x = ops.dev(np.tile(row, (4, 1)).astype(np.float32), dtype).view(4, 1, V)
        kw = dict(T=[1.0, 5000.0, 1.0, 0.0], k=[0, 0, V // 2, 0], p=[1.0, 0.9, 1.0, 1.0], u=rng.random((4, 1)).astype(np.float32))
        before = x.clone()
        for in_place in (False, True):
            _, out = ops._sample(x, in_place=in_place, **kw)
            kept = out > -np.inf
            assert int(kept.sum()) > 0
            assert torch.equal(out.view(word)[kept], before.view(word)[kept]), (name, in_place)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [2, 300, 5003, 70001])
def test_sample_borders_among_the_types_lowest_value(V, dtype):
    """Rows that are masked whole by the type's lowest value, or whose last ids are: all of them are ids as others."""
    rng = np.random.default_rng(V)
    x = torch.full((4, 1, V), torch.finfo(dtype).min, dtype=dtype, device="cuda")
    x[2, 0, ::2] = -float("inf")
    x[3, 0, :V // 2] = float(x[0, 0, 0]) / 2
    u = rng.random((4, 1)).astype(np.float32)
    for kw in (dict(), dict(p=np.full(4, 0.3)), dict(p=np.full(4, 0.71), m=np.full(4, 0.5)), dict(k=np.full(4, max(2, V - 1)), p=np.full(4, 0.9)),
               dict(p=np.full(4, 0.0))):
        ops._sample(x, u=u, **kw)
        ops._sample(x, T=np.full(4, 1e4), u=u, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [2.0 ** 63, 2.0 ** 64, 3e25, 1e34, 1e36, 1e38, 3e38])
def test_sample_at_the_largest_temperatures(T, dtype):
    """Logits as far apart as temperatures are high, up to the type's ends."""
    rng = np.random.default_rng(int(np.log2(T)))
    for V in (501, 20011):
        top = min(3.38e38, 4 * T)
        x = ops.dev(rng.uniform(-top, top, (6, 1, V)).astype(np.float32), dtype)
        x[1, 0, ::2] = -float("inf")
        x[2, 0, 1:] = torch.finfo(dtype).min
        u = rng.random((6, 1)).astype(np.float32)
        ops._sample(x, T=np.full(6, T), u=u)
        ops._sample(x, T=np.full(6, T), p=np.full(6, 0.7), u=u)
        ops._sample(x, T=np.full(6, T), k=np.full(6, V // 3), m=np.full(6, 0.02), u=u)
        ops._sample(x, T=np.full(6, T), k=np.full(6, V - 7), p=np.full(6, 0.9), m=np.full(6, 0.3), u=u)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotary_of_heads_far_apart(dtype):
    """Keys of a cache in the order of heads, tokens, values, whose heads lie more than 2^29 values apart; and tokens as far apart."""
    far, D = (1 << 29) + 64, 64
    size = 2 * far
    if torch.cuda.mem_get_info()[0] < 3 * size * torch.finfo(dtype).bits // 8:
        pytest.skip("needs some GB")
    turns, _ = sd.rotary_turns(D)
    pos = torch.arange(7, 10, dtype=torch.int32, device="cuda")
    big = torch.zeros(size, dtype=dtype, device="cuda")
    for shape, strides in (((3, 2, D), (D, far, 1)), ((2, 3, D), (far, D, 1)), ((1, 2, D), (far, far, 1))):
        x = torch.randn(shape, device="cuda").to(dtype)
        want, _ = sd.spec_rotary(x.clone(), None, pos[:shape[0]], turns)
        view = big.as_strided(shape, strides)
        view.copy_(x)
        got, _ = sd.spec_rotary(view, None, pos[:shape[0]], turns)
        assert torch.equal(got, want)
        view.zero_()
        _, out = sd.spec_rotary(None, x, pos[:shape[0]], turns, k_out=view)
        assert torch.equal(out, want)
        view.zero_()
    assert int(big.count_nonzero()) == 0  # and nothing else was written


def test_rotary_strides_of_one_token_or_head_do_not_matter():
    import ctypes

    lib, turns = sd.load_library(), sd.rotary_turns(64)[0]
    pos = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    x = torch.randn(1, 4, 64, device="cuda")
    want, _ = sd.spec_rotary(x.clone(), None, pos, turns)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    y = x.clone()
    none = (None, 0, 0)
    torch.cuda.synchronize()
    assert lib.spec_rotary(p(y), None, 0, 1, 4, 0, 64, 0, 64, 0, 0, p(pos), p(turns), 64, 0, 1.0, p(y), 256, 64, *none, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    y = x.view(4, 1, 64).clone()  # four tokens of one head
    pos = torch.full((4,), 5, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert lib.spec_rotary(p(y), None, 0, 4, 1, 0, 64, 64, 64, 0, 0, p(pos), p(turns), 64, 0, 1.0, p(y), 64, 3, *none, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(y.view(1, 4, 64), want)


def test_large_forks_and_compactions_in_a_graph():
    """As many blocks as take a grid of CTAs, captured and replayed."""
    rng = np.random.default_rng(17)
    c = ops._pool(rng, 900, 60, 16, spare=20000)
    N, B = len(c["ring"]), 1500
    parent = ops.i32(rng.integers(-1, 900, B))
    args = [ops.i32(c[n]) for n in ("table", "kv", "held")]
    shares, ring, state = (ops.i32(c[n]) for n in ("shares", "ring", "state"))
    ws = sd.new_page_workspace(N)
    first_ring = ring.clone()
    fork = sd.kv_fork(*args, parent, shares, ring, state, 16, workspace=ws)
    packed = sd.kv_compact(fork.block_table, fork.held, fork.shares, ring, fork.ring_state, workspace=ws)
    after = ring.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fork2 = sd.kv_fork(*args, parent, shares, ring, state, 16, workspace=ws)
        packed2 = sd.kv_compact(fork2.block_table, fork2.held, fork2.shares, ring, fork2.ring_state, workspace=ws)
    n, moves, free = int(fork.count), int(packed.count), int(packed.ring_state[1])
    assert n > 0 and moves > 0
    for _ in range(2):
        ring.copy_(first_ring)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ring, after) and torch.equal(fork.copies[:n], fork2.copies[:n]) and torch.equal(packed.copies[:moves], packed2.copies[:moves])
        for name in ("block_table", "kv_len", "held", "shares", "ring_state", "count"):
            assert torch.equal(getattr(fork, name), getattr(fork2, name)), name
        for name in ("block_table", "shares", "renamed", "ring_state", "count"):
            assert torch.equal(getattr(packed, name), getattr(packed2, name)), name
        assert torch.equal(packed.free_ring[:free], packed2.free_ring[:free])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_rows_past_32_bits(dtype):
    """More than 2^31 logits, cut in place: the last rows as they are alone."""
    V, R = 262144, 65
    B = (1 << 31) // (R * V) + 2
    if torch.cuda.mem_get_info()[0] < 2 * B * R * V * torch.finfo(dtype).bits // 8:
        pytest.skip("needs some GB")
    x = torch.empty(B, R, V, dtype=dtype, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    u, p = torch.rand(B, R, device="cuda"), torch.full((B,), 0.8, device="cuda")
    last = x[B - 1:].clone()
    k = torch.full((B,), 50, dtype=torch.int32, device="cuda")
    tokens = sd.spec_sample(x, top_k=k, top_p=p, uniform=u, out=x)
    alone = torch.empty_like(last)
    want = sd.spec_sample(last, top_k=k[:1], top_p=p[:1], uniform=u[B - 1:].contiguous(), out=alone)
    torch.cuda.synchronize()
    assert torch.equal(tokens[B - 1:], want) and torch.equal(x[B - 1], alone[0])
    assert int((x[0] > -float("inf")).sum(1).max()) <= 50 and int((x[B - 1] > -float("inf")).sum(1).min()) > 0
