"""GPU tests of sampling, rotary positions and the cache's forks and moves against
plain implementations (tests/decode_reference.py), at the sizes, masks and strides
where they can go wrong."""
import math

import numpy as np
import pytest
import torch

from tests import decode_reference as ref
from tests.parity import wait_gpu

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_80_gb300")
E4M3 = torch.float8_e4m3fn
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sd.load_library()


def dev(x, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(x):
    return dev(np.asarray(x, dtype=np.int32))


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------- spec_sample

def _sample(x, T=None, k=None, p=None, m=None, u=None, n=None, rows=True, in_place=False, bits=0):
    """Runs the kernel on x [B, rows, V] (a GPU tensor) and compares with the plain rows."""
    B, R, V = x.shape
    f32 = lambda v: None if v is None else dev(np.asarray(v, dtype=np.float32))  # noqa: E731
    before = x.clone()
    out = None if not rows else (x if in_place else torch.full_like(x, 7.0))
    untouched = before if in_place else torch.full_like(x, 7.0)
    err = err_word()
    tokens = sd.spec_sample(x, f32(T), None if k is None else i32(k), f32(p), f32(m), f32(u), None if n is None else i32(n), out=out,
                            error_word=err)
    wait_gpu()
    assert err.item() == bits
    host = before.float().cpu().numpy()
    got = None if out is None else out.float().cpu().numpy()
    per = lambda v, b, default: default if v is None else v[b]  # noqa: E731
    for b in range(B):
        for j in range(R):
            if n is not None and j > min(max(n[b], 0), R - 1):
                if tokens is not None:
                    assert tokens[b, j].item() == -1
                if got is not None:
                    assert torch.equal(out[b, j], untouched[b, j])
                continue
            kept, token = ref.sample_row(host[b, j], per(T, b, 1.0), per(k, b, 0), per(p, b, 1.0), per(m, b, 0.0), None if u is None else u[b][j])
            if tokens is not None:
                assert tokens[b, j].item() == token, (b, j)
            if got is not None:
                want = np.full(V, -INF, dtype=np.float32)
                ids = np.fromiter(kept, dtype=np.int64, count=len(kept))
                want[ids] = host[b, j, ids]
                same = got[b, j] == want
                assert same.all(), (b, j, len(kept), np.flatnonzero(~same)[:5])
    return tokens, out


def _rows(rng, B, R, V, dtype, spread=3.0, peaks=20, lift=10.0):
    x = rng.normal(0, spread, (B, R, V))
    at = rng.integers(0, V, (B, R, min(peaks, V)))
    np.put_along_axis(x, at, np.take_along_axis(x, at, 2) + lift * rng.random(at.shape), 2)
    return dev(x.astype(np.float32), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 255, 1000, 4097, 32003, 50001, 128256, 262144])
def test_sample_sizes(V, dtype):
    rng = np.random.default_rng(V)
    B, R = (6, 3) if V < 60000 else (3, 2)
    x = _rows(rng, B, R, V, dtype)
    _sample(x, T=0.4 + rng.random(B), k=rng.choice([0, 1, 3, 40, 1000], B), p=rng.choice([1.0, 0.9, 0.5], B), m=rng.choice([0.0, 0.05], B),
            u=rng.random((B, R)).astype(np.float32), n=rng.integers(0, R, B))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("what", ["none", "T", "k", "p", "m", "kp", "km", "pm", "kpm"])
def test_sample_each_cut_and_together(what, dtype):
    rng = np.random.default_rng(len(what) + 10)
    B, R, V = 12, 2, 20011
    x = _rows(rng, B, R, V, dtype, lift=6.0)
    kw = {}
    if "T" in what:
        kw["T"] = rng.choice([0.0, 1e-6, 0.01, 0.3, 1.0, 3.0, 50.0, 1e4, 3e38], B)
    if "k" in what:
        kw["k"] = rng.choice([-3, 0, 1, 2, 17, 500, V - 1, V, V + 5], B)
    if "p" in what:
        kw["p"] = rng.choice([0.0, 1e-6, 0.3, 0.95, 0.99999, 1.0, 2.0], B)
    if "m" in what:
        kw["m"] = rng.choice([0.0, 1e-7, 0.01, 0.3, 1.0], B)
    u = np.concatenate([[[0.0, 1 - 2.0 ** -24]], rng.random((B - 1, R))]).astype(np.float32)
    _sample(x, u=u, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_flat_and_tied_rows(dtype):
    rng = np.random.default_rng(3)
    V = 5003
    rows = [np.zeros(V), np.full(V, -7.25), rng.integers(-3, 4, V).astype(float), np.round(rng.normal(0, 2, V) * 4) / 4,
            np.where(np.arange(V) % 2 == 0, 0.0, -0.0), rng.normal(0, 1e-3, V), rng.normal(0, 1e-20, V), rng.normal(1000, 1.0, V),
            rng.normal(-30000, 5000.0, V), np.where(rng.random(V) < 0.999, 0.0, 30.0)]
    for j, row in enumerate(rows):
        x = dev(np.tile(row, (8, 1)).astype(np.float32), dtype).view(8, 1, V)
        _sample(x, T=[1.0, 0.5, 0.02, 1.0, 1.0, 7.0, 1.0, 1.0], k=[0, 0, 0, 700, 5, 0, 3000, 2], p=[1.0, 0.5, 0.9, 1.0, 0.25, 0.999, 0.7, 0.5],
                m=[0, 0, 0, 0.2, 0, 0.9, 0, 1.0], u=rng.random((8, 1)).astype(np.float32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_masks_infinities_and_nan(dtype):
    rng = np.random.default_rng(8)
    V, lowest = 3001, torch.finfo(dtype).min
    x = rng.normal(0, 2, (10, V)).astype(np.float32)
    x[0] = -INF                                   # nothing left: -1, and the bit
    x[1, :] = -INF
    x[1, 2999] = -5.0                             # one id
    x[2, ::2] = -INF
    x[3, ::3] = math.nan
    x[4] = lowest                                 # the type's lowest value is a value
    x[5, ::2] = lowest
    x[6, [7, 100, 2000]] = INF                    # infinite ones are equal
    x[7] = math.nan
    x[8, 1:] = -INF
    x[9, 5] = INF
    x[9, 6:] = -INF
    t = dev(x, dtype).view(10, 1, V)
    u = rng.random((10, 1)).astype(np.float32)
    _sample(t, u=u, bits=sd.DEV_ERR_SAMPLE)
    _sample(t, T=np.full(10, 0.7), k=[0, 5, 40, 1000, 7, 1600, 2, 1, 3, 1], p=np.full(10, 0.9), u=u, bits=sd.DEV_ERR_SAMPLE)
    _sample(t, m=np.full(10, 0.1), u=u, bits=sd.DEV_ERR_SAMPLE)
    _sample(t, T=np.zeros(10), u=u, bits=sd.DEV_ERR_SAMPLE)


def _special_rows(V, rng):
    lowest = -3.3895e38
    few = np.full(V, -INF)
    few[rng.integers(0, V, 30)] = rng.normal(0, 2, 30)
    return {
        "equal": np.zeros(V), "equal and low": np.full(V, -9000.0), "two values": np.where(np.arange(V) % 3 == 0, 1.0, 0.5),
        "whole numbers": rng.integers(-4, 5, V).astype(float), "far": rng.normal(9000, 3, V), "around zero": rng.normal(0, 1e-7, V),
        "tiny": rng.normal(0, 1e-30, V), "some tiny": np.where(rng.random(V) < 0.3, rng.normal(0, 1e-8, V), rng.normal(0, 1, V)),
        "lowest value masks": np.where(rng.random(V) < 0.9, lowest, rng.normal(0, 2, V)), "few left": few,
        "few left by lowest values": np.where(np.isinf(few), lowest, few), "infinite": np.where(np.arange(V) % 5000 == 7, INF, 0.0),
        "nan": np.where(rng.random(V) < 0.1, math.nan, rng.normal(0, 2, V)), "one high": np.where(np.arange(V) == V - 1, 50.0, rng.normal(0, 2, V)),
        "negative": -np.abs(rng.normal(20, 5, V)), "down to minus 5000": -5000 * rng.random(V), "high": rng.normal(3900, 100, V),
        "nothing": np.full(V, -INF)}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [3001, 70001])
def test_sample_special_rows(V, dtype):
    """Rows that the usual way's bins do not tell apart, in one part and (70001) in several."""
    rng = np.random.default_rng(V + 1)
    asks = [dict(), dict(k=[100], p=[0.9]), dict(p=[0.97]), dict(k=[20000], m=[0.3]), dict(m=[0.05]), dict(T=[100.0], k=[2500], p=[0.5]),
            dict(T=[2e-4], p=[0.8])]
    for name, row in _special_rows(V, rng).items():
        x = dev(row.astype(np.float32), dtype).view(1, 1, V)
        for ask in asks:
            try:
                _sample(x, u=rng.random((1, 1)).astype(np.float32), bits=sd.DEV_ERR_SAMPLE if name == "nothing" else 0, **ask)
            except AssertionError as e:
                raise AssertionError(f"{name}, {ask}") from e


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [1, 3, 9, 30, 70, 160])
def test_sample_row_in_parts(B, dtype):
    """As many CTAs a row as there is room for, in place and from any element on."""
    V = 66003
    rng = np.random.default_rng(B)
    x = _rows(rng, B, 1, V, dtype, lift=8.0)
    kw = dict(T=0.5 + rng.random(B), k=rng.choice([0, 1, 30, 3000], B), p=rng.choice([1.0, 0.9], B), m=rng.choice([0.0, 0.1], B),
              u=rng.random((B, 1)).astype(np.float32))
    a, _ = _sample(x.clone(), **kw)
    b, _ = _sample(x.clone(), in_place=True, **kw)
    c, _ = _sample(torch.empty(x.numel() + 5, dtype=dtype, device="cuda")[5:].view_as(x).copy_(x), **kw)
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [200, 70001])
def test_sample_border_among_the_lowest(V, dtype):
    """Top-k's border at logits of -4096 and below, beside masked ones."""
    rng = np.random.default_rng(V)
    x = np.full((2, 1, V), -INF)
    for b in range(2):
        at = rng.permutation(V)[:45]
        x[b, 0, at[:40]] = -5000.0 - 64 * rng.integers(0, 9, 40)
        x[b, 0, at[40:]] = rng.normal(0, 1, 5)
    x = dev(x.astype(np.float32), dtype)
    for k in (3, 20, 45, 46, 100):
        for T in (1.0, 1000.0):
            _sample(x, T=np.full(2, T), k=np.full(2, k), u=rng.random((2, 1)).astype(np.float32))
            _sample(x, T=np.full(2, T), k=np.full(2, k), p=np.full(2, 0.9), u=rng.random((2, 1)).astype(np.float32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("k", [0, 700, 4096, 4097, 9000])
def test_sample_draws_among_equal_ids(k, dtype):
    """Tokens of rows with a few hundred values, whose ids' order decides, for lists with and without ids."""
    rng = np.random.default_rng(k)
    B, V = 12, 20001
    x = dev((rng.integers(0, 400, (B, 1, V)) / 64).astype(np.float32), dtype)
    kw = dict(T=0.5 + rng.random(B), k=np.full(B, k), u=rng.random((B, 1)).astype(np.float32))
    _sample(x, rows=False, **kw)
    _sample(x, **kw)
    _sample(x, p=np.full(B, 0.7), **kw)


@pytest.mark.parametrize("B,V", [(1, 262144), (3, 128256), (40, 128256), (20, 200003)])
def test_sample_fp32_borders_in_full_bins(B, V):
    """Flat rows away from 0, some thousand ids in each bin where borders lie."""
    rng = np.random.default_rng(V + B)
    x = dev(rng.normal(6, 2.5, (B, 1, V)).astype(np.float32), torch.float32)
    u = rng.random((B, 1)).astype(np.float32)
    T = 1.5 + rng.random(B)
    _sample(x, T=T, u=u)
    _sample(x, T=T, p=np.full(B, 0.8), u=u)
    _sample(x, T=T, k=np.full(B, V // 3), m=np.full(B, 0.02), u=u)
    _sample(x, T=T, k=np.full(B, 6000), p=np.full(B, 0.7), m=np.full(B, 0.05), u=u)
    _sample(-x, T=T, p=np.full(B, 0.6), m=np.full(B, 0.1), u=u)
    _sample(torch.round(8 * x) / 8, T=T, p=np.full(B, 0.6), u=u)  # (and many of each value)


@pytest.mark.parametrize("B", [1, 40])
def test_sample_fp32_parts_with_and_without_room(B):
    """More ids that min-p keeps than some parts of a row can list, none in the others."""
    rng = np.random.default_rng(B)
    V = 262144
    x = rng.normal(-20, 1, (B, 1, V))
    x[:, :, :65536] = 1 + 7 * rng.random((B, 1, 65536))
    x = dev(x.astype(np.float32), torch.float32)
    u = rng.random((B, 1)).astype(np.float32)
    _sample(x, T=np.full(B, 2.0), m=np.full(B, 0.02), u=u)
    _sample(x, T=np.full(B, 2.0), m=np.full(B, 0.6), u=u)
    _sample(x, T=np.full(B, 2.0), k=np.full(B, 8000), m=np.full(B, 0.7), u=u)
    _sample(x, T=np.full(B, 2.0), k=np.full(B, 40000), p=np.full(B, 0.8), m=np.full(B, 0.1), u=u)


def test_sample_reports_bad_values():
    rng = np.random.default_rng(4)
    x = _rows(rng, 6, 2, 999, torch.float32)
    u = rng.random((6, 2)).astype(np.float32)
    _sample(x, T=[-1.0, math.nan, 1e-7, INF, 1.0, 0.0], u=u, bits=sd.DEV_ERR_TEMPERATURE)
    _sample(x, p=[-0.1, math.nan, 0.5, 0.5, 0.5, 0.5], u=u, bits=sd.DEV_ERR_SAMPLE)
    _sample(x, m=[-0.1, math.nan, 1.5, 0.1, 0.1, 0.1], u=u, bits=sd.DEV_ERR_SAMPLE)
    bad = u.copy()
    bad[0, 0], bad[1, 1], bad[2, 0], bad[3, 0] = 1.0, -0.5, math.nan, 7.0
    _sample(x, u=bad, bits=sd.DEV_ERR_SAMPLE)
    _sample(x, u=u, n=[0, 1, 2, -1, 1, 0], bits=sd.DEV_ERR_DRAFT_LEN)


@pytest.mark.parametrize("V", [4096, 4099])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_in_place_and_unaligned(V, dtype):
    rng = np.random.default_rng(V)
    x = _rows(rng, 5, 3, V, dtype)
    kw = dict(T=np.full(5, 0.8), k=[50, 0, 3, 7, 1], p=np.full(5, 0.9), u=rng.random((5, 3)).astype(np.float32), n=[2, 1, 0, 2, 2])
    a, _ = _sample(x.clone(), **kw)
    b, _ = _sample(x.clone(), in_place=True, **kw)
    assert torch.equal(a, b)
    # a batch that starts at any element, into memory with another start
    for off in (1, 3):
        src = torch.empty(x.numel() + off, dtype=dtype, device="cuda")[off:].view_as(x).copy_(x)
        _sample(src, **kw)


def test_sample_tokens_alone_and_rows_alone():
    rng = np.random.default_rng(6)
    x = _rows(rng, 4, 2, 9001, torch.bfloat16)
    _sample(x, p=np.full(4, 0.8), u=rng.random((4, 2)).astype(np.float32), rows=False)
    tokens, _ = _sample(x, p=np.full(4, 0.8))
    assert tokens is None


def test_sample_follows_the_shares():
    """Tokens of evenly spread random numbers: each id as often as its share says."""
    w = np.array([0.4, 0.05, 0.3, 0.25])
    n = 4096
    x = dev(np.tile(np.log(w), (64, n // 64, 1)).astype(np.float32))
    u = ((torch.arange(n, device="cuda") + 0.5) / n).view(64, n // 64)
    got = torch.bincount(sd.spec_sample(x, uniform=u).flatten().long(), minlength=4).cpu().numpy()
    assert np.abs(got - n * w).max() <= 1  # the borders fall between two of the numbers


@pytest.mark.parametrize("B,V", [(5, 32003), (2, 128256), (30, 70001)])
def test_sample_in_a_graph_and_on_another_stream(B, V):
    rng = np.random.default_rng(9)
    x = _rows(rng, B, 1, V, torch.bfloat16)
    u = dev(rng.random((B, 1)).astype(np.float32))
    p = torch.full((B,), 0.9, device="cuda")
    out, tokens = torch.zeros_like(x), torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sd.spec_sample(x, top_p=p, uniform=u, out=out, tokens=tokens, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    out2, tokens2 = torch.zeros_like(x), torch.zeros_like(tokens)
    with torch.cuda.graph(g):
        sd.spec_sample(x, top_p=p, uniform=u, out=out2, tokens=tokens2)
    for seed in range(3):
        y = _rows(np.random.default_rng(seed), B, 1, V, torch.bfloat16)
        if seed:
            x.copy_(y)
            sd.spec_sample(x, top_p=p, uniform=u, out=out, tokens=tokens)
        g.replay()
        wait_gpu()
        assert torch.equal(out, out2) and torch.equal(tokens, tokens2)


def test_sample_then_verify_keeps_to_the_cut_rows():
    """Drafts drawn from cut rows, verified against cut target rows: every token made may be drawn."""
    rng = np.random.default_rng(12)
    B, n, V = 16, 3, 2000
    draft, target = (_rows(rng, B, r, V, torch.float32, lift=6.0) for r in (n, n + 1))
    p = torch.full((B,), 0.7, device="cuda")
    T = torch.full((B,), 0.9, device="cuda")
    x = sd.spec_sample(draft, temperature=T, top_p=p, uniform=dev(rng.random((B, n)).astype(np.float32)), out=draft)
    sd.spec_sample(target, temperature=T, top_p=p, out=target)
    length = torch.full((B,), n, dtype=torch.int32, device="cuda")
    acc, out = sd.spec_verify(target, draft, x, length, T, seed=5)
    wait_gpu()
    for b in range(B):
        for j in range(int(acc[b]) + 1):
            assert target[b, j, int(out[b, j])] > -INF


# -------------------------------------------------------------- spec_rotary

def _rotary(T, Hq, H, D, R, layout, dtype, in_place, scaling=None, far=200000, views=True, seed=0):
    rng = np.random.default_rng(seed + T + D + R)
    fused = torch.randn(T, Hq + 2 * H, D, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)
    q, k = fused[:, :Hq], fused[:, Hq:Hq + H]
    if not views:
        q, k = q.contiguous(), k.contiguous()
    pos = rng.integers(0, far, T).astype(np.int32)
    pos[rng.random(T) < 0.1] = -1
    freq, factor = sd.rotary_frequencies(R, scaling=scaling)
    turns, f2 = sd.rotary_turns(R, scaling=scaling)
    assert factor == f2
    q0, k0 = q.double().cpu().numpy(), k.double().cpu().numpy()
    outs = (None, None) if in_place else (torch.full((T, Hq, D), 5.0, dtype=dtype, device="cuda"), torch.full((T, H, D), 5.0, dtype=dtype, device="cuda"))
    rest = fused[:, Hq + H:].clone()
    a, b = sd.spec_rotary(q, k, i32(pos), turns, layout=layout, factor=factor, q_out=outs[0], k_out=outs[1])
    wait_gpu()
    assert torch.equal(rest, fused[:, Hq + H:])
    # one rounding of the result, half a step of the type; before it products and their
    # sum in 32 bits, and sine and cosine to 2^-21 of |a| + |b|
    half = torch.finfo(dtype).eps / 2
    for got, x0 in ((a, q0), (b, k0)):
        before = x0 if in_place else np.full(x0.shape, 5.0)
        want = ref.rotate(x0, pos, freq, layout == "pairs", factor, before)
        size = ref.rotate(np.abs(x0), np.where(pos < 0, -1, 0), [0.0] * len(freq), layout == "pairs", 1.0, np.abs(before))
        other = np.roll(np.abs(x0), 1, 2) + np.roll(np.abs(x0), -1, 2) if layout == "pairs" else np.roll(np.abs(x0), R // 2, 2) + np.roll(np.abs(x0), -(R // 2), 2)
        limit = half * np.abs(want) + (2.0 ** -21 * factor * (size + other + np.abs(x0).max(2, keepdims=True)) if dtype == torch.float32
                                       else 2.0 ** -20 * factor * (size + other + np.abs(x0).max(2, keepdims=True)))
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= limit).all(), float((err - limit).max())
        skipped = pos < 0
        assert np.array_equal(got.double().cpu().numpy()[skipped], before[skipped])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,Hq,H,D,R", [(1, 32, 8, 64, 64), (7, 8, 2, 128, 128), (33, 12, 3, 128, 64), (5, 4, 1, 96, 40), (3, 2, 2, 80, 36),
                                        (9, 3, 1, 18, 6), (2, 1, 1, 2, 2), (700, 4, 1, 128, 128)])
def test_rotary(T, Hq, H, D, R, layout, dtype, in_place):
    _rotary(T, Hq, H, D, R, layout, dtype, in_place)


@pytest.mark.parametrize("scaling", [dict(type="linear", factor=4), dict(type="ntk", factor=8), dict(type="yarn", factor=16, original=8192),
                                     dict(type="bands", factor=8, original=8192)])
def test_rotary_scaled_and_far(scaling):
    _rotary(60, 4, 2, 128, 128, "half", torch.float32, False, scaling=scaling, far=2 ** 31 - 1)


def test_rotary_many_tokens_in_groups():
    T, Hq, H, D = 20000, 2, 1, 64
    x = torch.randn(T, Hq + H, D, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    turns, _ = sd.rotary_turns(D)
    a, b = sd.spec_rotary(x[:, :Hq], x[:, Hq:], pos, turns, q_out=torch.empty(T, Hq, D, device="cuda"), k_out=torch.empty(T, H, D, device="cuda"))
    for t in (0, 1, 7, 8, 1215, 12345, T - 1):
        c, d = sd.spec_rotary(x[t:t + 1, :Hq].clone(), x[t:t + 1, Hq:].clone(), pos[t:t + 1], turns)
        assert torch.equal(a[t:t + 1], c) and torch.equal(b[t:t + 1], d)


def test_rotary_of_one_side_and_of_nothing():
    turns, _ = sd.rotary_turns(32)
    x = torch.randn(4, 3, 64, device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    want, _ = sd.spec_rotary(x.clone(), x.clone(), pos, turns)
    q, none = sd.spec_rotary(x.clone(), None, pos, turns)
    none2, k = sd.spec_rotary(None, x.clone(), pos, turns)
    assert none is None and none2 is None and torch.equal(q, want) and torch.equal(k, want)
    e, _ = sd.spec_rotary(x[:0], None, pos[:0], turns)
    assert e.shape == (0, 3, 64)


def test_rotary_products_depend_on_the_distance_alone():
    """q at p and k at p - 5: the same product at any p."""
    turns, _ = sd.rotary_turns(64)
    q, k = (torch.randn(1, 1, 64, device="cuda").expand(50, 1, 64).contiguous() for _ in range(2))
    pos = torch.linspace(10, 1e9, 50, device="cuda").to(torch.int32)
    a, _ = sd.spec_rotary(q.clone(), None, pos, turns)
    b, _ = sd.spec_rotary(k.clone(), None, pos - 5, turns)
    dots = (a.double() * b.double()).sum((1, 2))
    size = float((q[0].double().abs() * k[0].double().abs()).sum())
    assert float((dots - dots[0]).abs().max()) <= 64 * 2.0 ** -21 * max(size, 1.0)


# ---------------------------------------------------- kv_fork and kv_compact

def _pool(rng, P, W, bs, spare, shared=0.5):
    """Old requests with some common beginnings; every block is held or in the ring."""
    held = rng.integers(0, W + 1, P)
    N = int(held.sum()) + spare
    ids = list(rng.permutation(N))
    table = np.full((P, W), -1, dtype=np.int32)
    shares = np.zeros(N, dtype=np.int64)
    for p in range(P):
        c = 0
        if p and rng.random() < shared:
            q = int(rng.integers(0, p))
            c = int(rng.integers(0, min(held[p], held[q]) + 1))
            table[p, :c] = table[q, :c]
            shares[table[p, :c]] += 1
        for j in range(c, held[p]):
            table[p, j] = ids.pop()
    head = int(rng.integers(0, N))
    ring = np.full(N, -1, dtype=np.int32)
    ring[(head + np.arange(len(ids))) % N] = ids
    kv = np.array([rng.integers(max(0, (h - 1) * bs), h * bs + 1) for h in held])
    return dict(table=table, held=held, kv=kv, shares=shares, ring=ring, state=np.array([head, len(ids)]))


def _check_fork(c, parent, bs, keep=None, accepted=None, ws=None, alias=False):
    kv = c["kv"] if accepted is None else c["kv"] - (np.maximum(accepted, -1) + 1)
    want = ref.fork(c["table"], kv, accepted, c["held"], parent, keep, c["shares"], c["ring"], c["state"], bs)
    ring, shares, state = i32(c["ring"]), i32(c["shares"]), i32(c["state"])
    err, out = err_word(), None
    B, W, N = len(parent), c["table"].shape[1], len(c["ring"])
    if alias:
        e = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
        out = sd.Fork(e(B, W), e(B), e(B), shares, state, e(B, 2), e(1))
    ws = sd.new_page_workspace(N) if ws is None else ws
    f = sd.kv_fork(i32(c["table"]), i32(kv), i32(c["held"]), i32(parent), shares, ring, state, bs,
                   accepted_len=None if accepted is None else i32(accepted), keep=None if keep is None else i32(keep), out=out, workspace=ws,
                   error_word=err)
    wait_gpu()
    for name in ("block_table", "kv_len", "held", "shares", "ring_state"):
        assert np.array_equal(getattr(f, name).cpu().numpy(), want[name]), name
    assert f.count.item() == len(want["copies"])
    assert [tuple(x) for x in f.copies[:f.count.item()].tolist()] == want["copies"]
    assert np.array_equal(ring.cpu().numpy(), want["ring"])
    assert err.item() == (sd.DEV_ERR_BLOCKS if want["bad"] else 0)
    assert int(ws.view(torch.int32)[:4 * N].abs().sum()) == 0  # the counts are zero again
    return want


def _consistent(want, parent, bs):
    """Every block is free once or held by shares + 1 requests, and what a request writes next is its own."""
    N = len(want["ring"])
    head, n = want["ring_state"]
    free = [int(want["ring"][(head + i) % N]) for i in range(n)]
    holders = np.zeros(N, dtype=int)
    for row, h in zip(want["block_table"], want["held"]):
        for x in row[:h]:
            holders[x] += 1
    assert sorted(free) == sorted(np.flatnonzero(holders == 0)) and len(set(free)) == n
    assert ((holders > 0) <= (want["shares"] == holders - 1)).all()
    for row, h, t in zip(want["block_table"], want["held"], want["kv_len"]):
        if t % bs:
            assert holders[row[h - 1]] == 1


@pytest.mark.parametrize("P,B,W,bs", [(1, 1, 1, 16), (1, 8, 5, 16), (7, 7, 9, 32), (20, 50, 6, 64), (64, 3, 40, 16), (300, 1500, 3, 128),
                                      (1100, 2100, 2, 16), (5, 0, 4, 16), (4, 6, 2500, 16)])
def test_fork(P, B, W, bs):
    rng = np.random.default_rng(P * 7 + B)
    c = _pool(rng, P, W, bs, spare=B + 3)
    parent = rng.integers(-1, P, B)
    want = _check_fork(c, parent, bs, alias=B % 2 == 1)
    assert not want["bad"]
    _consistent(want, parent, bs)
    keep = rng.integers(-2, W * bs + 5, B)
    _consistent(_check_fork(c, parent, bs, keep=keep), parent, bs)
    accepted = np.minimum(rng.integers(-1, 6, P), c["kv"] - 1)
    _consistent(_check_fork(c, parent, bs, keep=keep, accepted=accepted), parent, bs)


def test_fork_of_one_parent_copies_for_all_but_the_last():
    c = dict(table=np.array([[2, 0, 4, -1]]), held=[3], kv=np.array([40]), shares=np.zeros(9, dtype=int),
             ring=np.array([1, 3, 5, 6, 7, 8, -1, -1, -1]), state=np.array([0, 6]))
    want = _check_fork(c, np.zeros(4, dtype=int), 16)
    assert want["copies"] == [(4, 1), (4, 3), (4, 5)] and want["block_table"][3].tolist() == [2, 0, 4, -1] and want["shares"][2] == 3
    # a request that stays beside them, with a block more, keeps it
    c["kv"] = np.array([48])
    want = _check_fork(c, np.zeros(4, dtype=int), 16, keep=np.array([40, 48, 33, 32]))
    assert want["copies"] == [(4, 1), (4, 3)] and want["shares"][4] == 0


def test_fork_without_enough_blocks_serves_in_order():
    for spare in (0, 1, 5):
        rng = np.random.default_rng(spare)
        c = _pool(rng, 6, 5, 16, spare=spare, shared=0.0)
        want = _check_fork(c, np.arange(30) % 6, 16)
        assert want["bad"] and len(want["copies"]) == spare
        _consistent(want, None, 16)


def test_fork_that_ends_everything_gives_all_blocks_back():
    rng = np.random.default_rng(2)
    c = _pool(rng, 40, 30, 16, spare=5)
    want = _check_fork(c, np.full(3, -1), 16)
    assert want["ring_state"][1] == len(c["ring"])
    _consistent(want, None, 16)


def test_fork_keeps_blocks_that_others_hold():
    """A block with a holder outside of the tables neither goes back nor is written."""
    c = dict(table=np.array([[1, 2]]), held=[2], kv=np.array([20]), shares=np.array([0, 1, 1, 0]), ring=np.array([0, 3, -1, -1]),
             state=np.array([0, 2]))
    want = _check_fork(c, np.array([0]), 16)
    assert want["copies"] == [(2, 0)] and want["shares"].tolist() == [0, 1, 0, 0]
    want = _check_fork(c, np.array([-1]), 16)
    assert want["ring_state"].tolist() == [0, 2] and want["shares"].tolist() == [0, 0, 0, 0]


def test_fork_reports_bad_values():
    rng = np.random.default_rng(3)
    for what in range(6):
        c = _pool(rng, 9, 6, 16, spare=40)
        parent = rng.integers(-1, 9, 14)
        if what == 0:
            parent[3], parent[5] = 9, -2
        elif what == 1:
            c["held"][4] = 7
        elif what == 2:
            c["held"][2] = -1
        elif what == 3:
            c["kv"][:] = 6 * 16 + 1
        elif what == 4:
            c["table"][1, 0], c["table"][2, :] = 1 << 30, -5
            c["held"][1:3] = 6
        else:
            c["state"][:] = [-4, 1 << 30]
        assert _check_fork(c, parent, 16)["bad"]


def test_fork_reports_a_bad_block_of_the_ring():
    c = dict(table=np.array([[2, 0]]), held=[2], kv=np.array([20]), shares=np.zeros(5, dtype=int), ring=np.array([1, 5, -7, 3, 4]),
             state=np.array([1, 2]))
    want = _check_fork(c, np.zeros(3, dtype=int), 16)
    assert want["bad"] and want["copies"] == [(0, 5), (0, -7)]
    layers = _layers(2, 5, 1, 16, 64)
    _check_copy(layers, want["copies"] + [(0, 4)], 3, 3)  # (passes the two over)


def test_forks_one_after_another_on_one_workspace():
    rng = np.random.default_rng(21)
    c = _pool(rng, 12, 8, 16, spare=200)
    ws = sd.new_page_workspace(len(c["ring"]))
    for i in range(6):
        P = len(c["held"])
        want = _check_fork(c, rng.integers(-1, P, 12), 16, ws=ws, keep=rng.integers(1, 130, 12))
        _consistent(want, None, 16)
        c = dict(table=want["block_table"], held=want["held"], kv=want["kv_len"], shares=want["shares"], ring=want["ring"], state=want["ring_state"])


def _check_compact(c, alias=False, ws=None):
    want = ref.compact(c["table"], c["held"], c["shares"], c["ring"], c["state"])
    table, shares, ring, state = i32(c["table"]), i32(c["shares"]), i32(c["ring"]), i32(c["state"])
    N, out, err = len(c["ring"]), None, err_word()
    if alias:
        e = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
        out = sd.Compaction(table, shares, ring, state, e(N), e(N // 2, 2), e(1))
    ws = sd.new_page_workspace(N) if ws is None else ws
    f = sd.kv_compact(table, i32(c["held"]), shares, ring, state, out=out, workspace=ws, error_word=err)
    wait_gpu()
    for name in ("block_table", "shares", "renamed"):
        assert np.array_equal(getattr(f, name).cpu().numpy(), want[name]), name
    assert f.ring_state.tolist() == [0, len(want["free"])] and f.free_ring[:len(want["free"])].tolist() == want["free"]
    assert f.count.item() == len(want["copies"]) and [tuple(x) for x in f.copies[:f.count.item()].tolist()] == want["copies"]
    assert err.item() == (sd.DEV_ERR_BLOCKS if want["bad"] else 0)
    assert int(ws.view(torch.int32)[:4 * N + (N + 31) // 32].abs().sum()) == 0
    return want


@pytest.mark.parametrize("P,W,spare", [(4, 2, 0), (1, 1, 1), (3, 4, 20), (10, 3, 0), (40, 30, 700), (200, 9, 1), (0, 3, 17), (500, 300, 60000)])
@pytest.mark.parametrize("alias", [False, True])
def test_compact(P, W, spare, alias):
    rng = np.random.default_rng(P + spare)
    c = _pool(rng, P, W, 16, spare=spare)
    assert not _check_compact(c, alias)["bad"]


def test_compact_of_one_block():
    c = dict(table=np.array([[0]]), held=np.array([1]), shares=np.array([0]), ring=np.array([-1]), state=np.array([0, 0]))
    _check_compact(c)
    _check_compact(c, alias=True)


def test_compact_keeps_blocks_that_no_table_names():
    c = dict(table=np.array([[6]]), held=np.array([1]), shares=np.array([0, 0, 0, 0, 4, 0, 1, 0]), ring=np.array([2, 0, 7, 3, -1, -1, -1, -1]),
             state=np.array([0, 4]))
    want = _check_compact(c)  # 1, 4, 5 and 6 are in use
    assert want["copies"] == [(4, 0), (5, 2), (6, 3)] and want["shares"].tolist() == [4, 0, 0, 1, 0, 0, 0, 0]


def test_compact_reports_bad_values():
    rng = np.random.default_rng(5)
    for what in range(5):
        c = _pool(rng, 9, 6, 16, spare=40)
        if what == 0:
            c["held"][4] = 7
        elif what == 1:
            c["held"][2] = -1
        elif what == 2:
            c["table"][:, 0] = 1 << 30
            c["held"][:] = np.maximum(c["held"], 1)
        elif what == 3:
            c["ring"][:] = np.where(np.arange(len(c["ring"])) % 3 == 0, -7, c["ring"])
            c["table"][:] = np.where(c["table"] < 0, 0, c["table"])
        else:
            c["state"][:] = [1 << 20, 5]
        assert _check_compact(c, alias=what % 2 == 0)["bad"] or what == 3


# ------------------------------------------------------------------ kv_copy

def _layers(L, N, H, bs, D, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(L):
        k, v = (torch.randint(0, 256, (N, H, bs, D), generator=g, device="cuda", dtype=torch.uint8).view(E4M3) for _ in range(2))
        out.append((k, v, torch.rand(N, H, generator=g, device="cuda"), torch.rand(N, H, generator=g, device="cuda")))
    return out


def _check_copy(layers, pairs, count, capacity):
    N = layers[0][0].shape[0]
    codes = np.full((capacity, 2), -1, dtype=np.int32)
    codes[:len(pairs)] = pairs
    want = [[(x.view(torch.uint8) if x.dtype == E4M3 else x).clone() for x in layer] for layer in layers]
    for a, b in pairs[:max(0, min(count, capacity))]:
        if 0 <= a < N and 0 <= b < N:
            for layer in want:
                for x in layer:
                    x[b] = x[a]
    sd.kv_copy(i32(codes), i32([count]), layers)
    wait_gpu()
    for layer, w in zip(layers, want):
        for x, y in zip(layer, w):
            assert torch.equal(x.view(torch.uint8) if x.dtype == E4M3 else x, y)


@pytest.mark.parametrize("L,N,H,bs,D", [(1, 2, 1, 16, 64), (3, 40, 8, 16, 64), (2, 33, 3, 128, 128), (70, 12, 2, 16, 64), (1, 300, 5, 32, 128)])
def test_copy(L, N, H, bs, D):
    rng = np.random.default_rng(N)
    ids = rng.permutation(N)
    half = N // 2
    pairs = list(zip(ids[:half].tolist(), ids[half:2 * half].tolist()))
    layers = _layers(L, N, H, bs, D)
    _check_copy(layers, pairs, half, half)
    _check_copy(layers, pairs, half // 2, half + 3)


def test_copy_bounds():
    layers = _layers(2, 20, 2, 16, 64)
    _check_copy(layers, [(1, 2), (-1, 3), (4, 20), (1 << 30, 5), (6, 6), (7, 8)], 6, 6)
    _check_copy(layers, [(1, 2), (3, 4)], 0, 2)
    _check_copy(layers, [(1, 2), (3, 4)], -5, 2)
    _check_copy(layers, [(9, 10), (11, 12)], 1000, 2)  # no more than there is room for
    _check_copy(layers, [(1, 15), (1, 16), (1, 17)], 3, 3)  # one block to several


def test_copy_past_32_bits():
    """A cache of more than 2^32 bytes, its last blocks."""
    N, H, bs, D = 40000, 8, 128, 128
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GB")
    k = torch.zeros(N, H, bs, D, dtype=torch.uint8, device="cuda").view(E4M3)
    ks = torch.zeros(N, H, device="cuda")
    v = torch.zeros(N, H, bs, D, dtype=torch.uint8, device="cuda").view(E4M3)
    k.view(torch.uint8)[7] = 3
    v.view(torch.uint8)[N - 1] = 5
    ks[N - 1] = 2.0
    sd.kv_copy(i32([[7, N - 2], [N - 1, 9]]), i32([2]), [(k, v, ks, ks.clone())])
    wait_gpu()
    assert bool((k.view(torch.uint8)[N - 2] == 3).all()) and bool((v.view(torch.uint8)[9] == 5).all()) and bool((ks[9] == 2).all())
    assert int(k.view(torch.uint8)[N - 3].sum()) == 0 and int(v.view(torch.uint8)[10].sum()) == 0


def test_pages_in_a_graph_and_on_another_stream():
    rng = np.random.default_rng(31)
    c = _pool(rng, 10, 8, 16, spare=60)
    N = len(c["ring"])
    layers = sd.kv_layers(_layers(3, N, 2, 16, 64))
    parent = i32(rng.integers(0, 10, 20))
    args = [i32(c[n]) for n in ("table", "kv", "held")], [i32(c[n]) for n in ("shares", "ring", "state")]
    ws = sd.new_page_workspace(N)
    run = lambda **kw: sd.kv_fork(*args[0], parent, *args[1], 16, workspace=ws, **kw)  # noqa: E731
    first = run()
    ring = args[1][1].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = run(stream=s)
        sd.kv_copy(second.copies, second.count, layers, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    before = [x.clone() for layer in layers.tensors for x in layer]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        third = run()
        sd.kv_copy(third.copies, third.count, layers)
        packed = sd.kv_compact(third.block_table, third.held, third.shares, args[1][1], third.ring_state, workspace=ws)
    results = []
    for _ in range(2):
        g.replay()
        wait_gpu()
        results.append([x.clone() for x in packed[:2]])
        for x, y in zip(first, third):
            n = first.count.item()
            assert torch.equal(x[:n], y[:n]) if x.shape == (20, 2) else torch.equal(x, y)
        assert torch.equal(args[1][1], ring)
    assert all(torch.equal(x, y) for x, y in zip(*results))
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(before, [x for layer in layers.tensors for x in layer]))
