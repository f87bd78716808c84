"""GPU tests of the operators around the verify step against plain
implementations in 64 bits (tests/step_reference.py), at the sizes, masks and
strides where they can go wrong."""
import math

import numpy as np
import pytest
import torch

from tests import step_reference as ref
from tests.parity import wait_gpu

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_80_gb300")
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sd.load_library()


def dev(x, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ kv_block_step

def _block_case(rng, B, bs, width, spare, most_new, ends=0.1, bad=False):
    held = rng.integers(0, width + 1, B)
    N = int(held.sum()) + spare
    ids = rng.permutation(N)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    head = int(rng.integers(0, N))
    ring = np.full(N, -1, dtype=np.int32)
    ring[(head + np.arange(spare)) % N] = ids[at:]
    kv = np.array([rng.integers(0, h * bs + 1) for h in held])
    acc = np.array([rng.integers(-1, min(7, h * bs - k - 1) + 1) if h * bs > k else -1 for h, k in zip(held, kv)])
    new = rng.integers(0, most_new + 1, B)
    new[rng.random(B) < ends] = -1
    if bad:
        kv[::5] += 1000 * bs
        acc[1::7] = -9
        held = held.copy()
        held[2::11] = width + 3
    i32 = lambda x: np.asarray(x, dtype=np.int32)  # noqa: E731
    return dict(table=table, kv_len=i32(kv), held=i32(held), new=i32(new), ring=ring, state=i32([head, spare]), accepted=i32(acc))


def _check_blocks(c, bs, capacity, alias=False, use_accepted=True):
    want = ref.block_step(c["table"], c["kv_len"], c["held"], c["new"], c["ring"], c["state"], bs, capacity,
                          c["accepted"] if use_accepted else None)
    table, ring, kv, held, state = (dev(c[k]) for k in ("table", "ring", "kv_len", "held", "state"))
    out = None
    B = len(c["held"])
    if alias:
        e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        out = sd.BlockStep(kv, held, state, e(B + 1), e(B + 1), e(capacity), e(capacity))
    err = err_word()
    step = sd.kv_block_step(table, kv, held, dev(c["new"]), ring, state, bs, capacity,
                            accepted_len=dev(c["accepted"]) if use_accepted else None, out=out, error_word=err)
    wait_gpu()
    for name in ("kv_len", "held", "ring_state", "cu_tokens", "cu_blocks", "slot_map", "positions"):
        assert getattr(step, name).tolist() == list(want[name]), name
    got = table.cpu().numpy()
    for b in range(B):
        assert (got[b, :want["held"][b]] == want["table"][b, :want["held"][b]]).all()
    # the free part of the ring, and every block in exactly one place
    N = len(c["ring"])
    h, n = want["ring_state"]
    at = (h + np.arange(n)) % N
    assert (ring.cpu().numpy()[at] == want["ring"][at]).all()
    assert err.item() == (sd.DEV_ERR_BLOCKS if want["bad"] else 0)
    return want, ring.cpu().numpy()[at], got


@pytest.mark.parametrize("B,bs,width,most_new", [(1, 16, 1, 1), (1, 16, 40, 300), (7, 32, 5, 8), (64, 16, 20, 8), (1000, 64, 3, 3),
                                                 (1025, 16, 6, 9), (2100, 128, 4, 70)])
@pytest.mark.parametrize("alias", [False, True])
def test_block_step(B, bs, width, most_new, alias):
    rng = np.random.default_rng(B * 31 + bs)
    c = _block_case(rng, B, bs, width, spare=B * (most_new // bs + 2), most_new=most_new)
    want, free, table = _check_blocks(c, bs, capacity=B * most_new, alias=alias)
    owned = [int(x) for b in range(B) for x in table[b, :want["held"][b]]]
    assert sorted(owned + [int(x) for x in free]) == list(range(len(c["ring"])))  # nothing lost, nothing twice


def test_block_step_large_capacity_uses_many_ctas():
    rng = np.random.default_rng(5)
    c = _block_case(rng, 40, 16, 60, spare=1000, most_new=700)
    c["held"] = np.minimum(c["held"], 10).astype(np.int32)
    c["kv_len"] = np.minimum(c["kv_len"], c["held"] * 16 - np.where(c["held"] > 0, 1, 0)).astype(np.int32)
    c["accepted"][:] = -1
    _check_blocks(c, 16, capacity=40 * 700)
    _check_blocks(c, 16, capacity=40 * 700, alias=True, use_accepted=False)


def test_block_step_without_enough_blocks_serves_in_order():
    rng = np.random.default_rng(7)
    for spare in (0, 1, 5, 30):
        c = _block_case(rng, 50, 16, 30, spare=spare, most_new=60)
        want, _, _ = _check_blocks(c, 16, capacity=3000)
        assert want["bad"] or spare >= 5


def test_block_step_cuts_at_the_capacity_and_clamps_bad_lengths():
    rng = np.random.default_rng(11)
    c = _block_case(rng, 30, 16, 8, spare=60, most_new=20)
    _check_blocks(c, 16, capacity=57)
    _check_blocks(c, 16, capacity=0)
    c = _block_case(rng, 60, 16, 8, spare=100, most_new=20, bad=True)
    c["table"] = np.maximum(c["table"], 0)
    _check_blocks(c, 16, capacity=1200)
    c = _block_case(rng, 9, 16, 4, spare=20, most_new=9)
    c["state"] = np.array([len(c["ring"]) + 5, 7], dtype=np.int32)
    _check_blocks(c, 16, capacity=81)


def test_block_step_idle_ended_and_empty_requests():
    c = dict(table=np.arange(12, dtype=np.int32).reshape(4, 3), kv_len=np.array([40, 0, 17, 48], dtype=np.int32),
             held=np.array([3, 3, 3, 3], dtype=np.int32), new=np.array([0, 0, -1, 0], dtype=np.int32),
             ring=np.full(12, -1, dtype=np.int32), state=np.array([4, 0], dtype=np.int32),
             accepted=np.array([-1, -1, 3, -1], dtype=np.int32))
    want, free, _ = _check_blocks(c, 16, capacity=4)
    assert want["held"] == [3, 0, 0, 3] and sorted(free.tolist()) == [3, 4, 5, 6, 7, 8]


# ---------------------------------------------------------------- kv_append

def _cache(rng, N, H, bs, D, zero=0.1):
    codes = rng.integers(0, 256, (N, H, bs, D), dtype=np.uint8)
    codes[(codes & 127) == 127] = 0
    scale = np.exp2(rng.integers(-12, 3, (N, H))).astype(np.float32)
    scale[rng.random((N, H)) < zero] = 0
    return codes, scale


def _run_append(k, v, slots, caches):
    t = [dev(x) if x.dtype != np.uint8 else dev(x).view(E4M3) for x in caches]
    sd.kv_append(k, v, dev(slots.astype(np.int32)), t[0], t[1], t[2], t[3])
    wait_gpu()
    return [x.view(torch.uint8).cpu().numpy() if x.dtype == E4M3 else x.cpu().numpy() for x in t]


def _check_append(k, v, slots, kc, vc, ks, vs):
    got = _run_append(k, v, slots, (kc, vc, ks, vs))
    for x, c, s, gc, gs in ((k, kc, ks, got[0], got[2]), (v, vc, vs, got[1], got[3])):
        wc, ws = ref.append(x.double().cpu().numpy(), slots, c, s)
        assert (gs == ws).all()
        # a NaN has one magnitude; the sign of a NaN or a zero says nothing
        a, b = ref.VALUES[gc], ref.VALUES[wc]
        assert np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,H,bs", [(64, 8, 16), (128, 2, 32), (128, 1, 64), (64, 3, 128), (128, 8, 16)])
def test_append_runs_at_every_offset(D, H, bs, dtype):
    rng = np.random.default_rng(D + bs)
    N = 40
    kc, ks = _cache(rng, N, H, bs, D)
    vc, vs = _cache(rng, N, H, bs, D)
    blocks = list(rng.permutation(N))
    slots = []
    while blocks:  # requests of one to four blocks, part-filled at both ends
        n = min(len(blocks), int(rng.integers(1, 5)))
        own = [blocks.pop() for _ in range(n)]
        first, last = int(rng.integers(0, bs)), int(rng.integers(1, bs + 1))
        ps = [(i, o) for i in range(n) for o in range(bs)][first:(n - 1) * bs + max(last, first + 1)]
        slots += [own[i] * bs + o for i, o in ps]
    slots = np.array(slots)
    g = torch.Generator(device="cuda").manual_seed(bs)
    x = torch.randn(len(slots), 3 * H, D, generator=g, device="cuda") * torch.exp2(
        torch.randint(-20, 10, (len(slots), 3 * H, 1), generator=g, device="cuda").float())
    x = x.to(dtype)
    _check_append(x[:, H:2 * H], x[:, 2 * H:], slots, kc, vc, ks, vs)  # strided as in a fused projection


def test_append_one_token_and_none():
    rng = np.random.default_rng(3)
    kc, ks = _cache(rng, 4, 2, 16, 128)
    vc, vs = _cache(rng, 4, 2, 16, 128)
    k = torch.randn(1, 2, 128, device="cuda")
    for s in (0, 17, 47, 63):
        _check_append(k, k * 3, np.array([s]), kc, vc, ks, vs)
    _check_append(k, k, np.array([-1]), kc, vc, ks, vs)
    _check_append(k, k, np.array([64]), kc, vc, ks, vs)  # past the cache: skipped
    got = _run_append(k[:0], k[:0], np.zeros(0), (kc, vc, ks, vs))
    assert (got[0] == kc).all() and (got[2] == ks).all()


def test_append_zeros_infinities_nan_and_range_ends():
    rng = np.random.default_rng(4)
    kc, ks = _cache(rng, 8, 1, 16, 64)
    vc, vs = _cache(rng, 8, 1, 16, 64)
    k = torch.zeros(16, 1, 64, device="cuda")
    k[1] = 5.0
    k[2, 0, 3] = float("inf")
    k[2, 0, 4] = -float("inf")
    k[2, 0, 5] = float("nan")
    k[2, 0, 6] = 1.5
    k[3] = 3e38
    k[4] = 1e-38
    k[5] = 1e-42
    k[6] = 448.0
    k[7] = 448.1
    slots = np.array([0, 17, 32, 48, 64, 80, 96, 112] + [-1] * 8)
    _check_append(k, -k, slots, kc, vc, ks, vs)
    # a block of zeros (scale 0) takes the scale of what is added to it
    kc[1] = 0
    ks[1] = 0
    _check_append(k, k, slots, kc, vc, ks, vs)


def test_append_rounds_another_writers_scale_up_to_a_power_of_two():
    rng = np.random.default_rng(6)
    kc, ks = _cache(rng, 2, 1, 16, 64, zero=0)
    ks[:] = 0.3
    k = torch.full((1, 1, 64), 0.01, device="cuda")
    got = _run_append(k, k, np.array([5]), (kc, kc, ks, ks))
    assert got[2][0, 0] == 0.5
    old, new = ref.VALUES[kc[0, 0, :5]] * np.float64(np.float32(0.3)), ref.VALUES[got[0][0, 0, :5]] * 0.5
    # half a step of the type: 2^-4 of the value, and half of the least step at the new scale
    assert (np.abs(old - new) <= np.abs(old) / 16 + 0.5 * 2.0 ** -10).all()
    assert (got[0][0, 0, 6:] == kc[0, 0, 6:]).all() and (got[0][1] == kc[1]).all()


def test_append_many_tokens_in_one_call():
    # long prompts: windows of several tokens per CTA, runs across windows
    rng = np.random.default_rng(8)
    H, bs, D = 8, 32, 64
    lens = [1500, 1, 700, 33, 31]
    N = sum(-(-n // bs) for n in lens) + 3
    kc, ks = _cache(rng, N, H, bs, D)
    vc, vs = _cache(rng, N, H, bs, D)
    free = list(rng.permutation(N))
    slots = []
    for n in lens:
        for i in range(0, n, bs):
            first = free.pop() * bs
            slots += range(first, first + min(bs, n - i))
    slots = np.array(slots)
    k = torch.randn(len(slots), H, D, device="cuda").to(torch.bfloat16)
    _check_append(k, k.flip(0), slots, kc, vc, ks, vs)


# ------------------------------------------------------------ spec_attention

def _attn_case(rng, new, kv, Hq, H, D, bs, extra_rows=0, pow2=False, stale=True):
    B = len(new)
    L = np.array(new) + np.array(kv)
    held = -(-L // bs)
    N = int(held.sum()) + 2
    codes = [rng.integers(0, 256, (N, H, bs, D), dtype=np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 127) == 127] ^= 1
    # rows of about unit size
    scales = [(rng.uniform(0.5, 1.5, (N, H)) / 100).astype(np.float32) for _ in range(2)]
    if pow2:
        scales = [np.exp2(np.round(np.log2(s))).astype(np.float32) for s in scales]
    ids = list(rng.permutation(N))
    width = max(1, int(held.max()) if B else 1) + 1
    table = np.full((B, width), -1, dtype=np.int32)
    for b in range(B):
        for i in range(held[b]):
            table[b, i] = ids.pop()
        if stale and L[b] % bs and held[b]:  # what lies past a request's last token is no number
            for c in codes:
                c[table[b, held[b] - 1], :, L[b] % bs:] = 0x7F
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1]) + extra_rows
    q = rng.standard_normal((T, Hq, D)) * 1.5
    return dict(q=torch.tensor(q).to(torch.bfloat16), cu=cu, kv=np.array(kv, dtype=np.int32), table=table, codes=codes, scales=scales)


def _attn_gpu(c, q=None, **kw):
    q = c["q"].cuda() if q is None else q
    out = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
    kc, vc = (dev(x).view(E4M3) for x in c["codes"])
    args = [dev(c["cu"]), dev(c["kv"]), dev(c["table"]), kc, vc, dev(c["scales"][0]), dev(c["scales"][1])]
    if "stream" in kw:
        kw["stream"].wait_stream(torch.cuda.current_stream())
    sd.spec_attention(q, *args, out=out, **kw)
    wait_gpu()
    return out


def _check_attn(c, out, scale=None, q=None):
    """Tolerance: the output is rounded to bf16 (2^-9 of it); probabilities have
    8 significant bits relative to themselves (2^-9 of each, so of the sum of
    p |v|), and their sum, in 32 bits, none of that; scores are sums of D exact
    products in 32 bits (2^-24 a step, at most D steps of the sum of |q k|, and
    an error of the score is one of the probability, twice for the quotient).
    Each is doubled for what follows in 32 bits."""
    q = c["q"] if q is None else q
    D = q.shape[2]
    s = 1 / math.sqrt(D) if scale is None else scale
    want, mag, big = ref.attention(q.double().cpu().numpy(), c["cu"], c["kv"], c["table"], c["codes"][0], c["codes"][1],
                                   c["scales"][0], c["scales"][1], s)
    got = out.double().cpu().numpy()
    none = np.isnan(want).all(axis=2)
    lo, hi = max(0, int(c["cu"][0])), min(q.shape[0], int(c["cu"][-1]))
    outside = np.ones(q.shape[0], dtype=bool)
    outside[lo:hi] = False
    assert (got[outside] == 77.0).all()
    want[outside] = got[outside]
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 4 * D * 2.0 ** -24 * big[:, :, None]) * mag + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3], none.sum())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,H", [(8, 1), (8, 8), (12, 2)])
def test_attention_lengths(D, bs, Hq, H):
    # one token on an empty cache, lengths around blocks and tiles, requests without new tokens
    new = [1, 1, 2, 1, 5, 0, 8, 3, 1, 2, 1]
    kv = [0, 1, 13, 15, 16, 50, 120, 126, 127, 254, 300]
    c = _attn_case(np.random.default_rng(D + bs + Hq), new, kv, Hq, H, D, bs)
    _check_attn(c, _attn_gpu(c))


@pytest.mark.parametrize("Hq,H,D,bs", [(64, 8, 128, 32), (32, 8, 64, 16), (1, 1, 128, 16), (16, 1, 128, 64), (40, 2, 64, 128),
                                       (6, 6, 64, 16), (128, 1, 128, 32), (33, 3, 128, 16), (129, 1, 64, 16)])
def test_attention_head_layouts(Hq, H, D, bs):
    c = _attn_case(np.random.default_rng(Hq), [5, 1, 9], [700, 250, 33], Hq, H, D, bs, pow2=True)
    _check_attn(c, _attn_gpu(c))


@pytest.mark.parametrize("new,kv", [([65], [1000]), ([130, 70], [0, 511]), ([300], [5])])
def test_attention_many_query_tokens(new, kv):
    # long drafts and prompts: more rows than one tile holds, the diagonal across tiles
    c = _attn_case(np.random.default_rng(sum(new)), new, kv, 8, 2, 128, 32)
    _check_attn(c, _attn_gpu(c))


def test_attention_one_long_request_split_over_the_gpu():
    c = _attn_case(np.random.default_rng(1), [2], [20000], 8, 1, 128, 64)
    _check_attn(c, _attn_gpu(c))
    c = _attn_case(np.random.default_rng(2), [1], [9999], 16, 2, 64, 16)
    _check_attn(c, _attn_gpu(c))


def test_attention_many_requests_of_mixed_lengths():
    rng = np.random.default_rng(9)
    new = rng.integers(0, 5, 200).tolist()
    kv = (rng.integers(0, 20, 200) ** 2).tolist()
    c = _attn_case(rng, new, kv, 8, 2, 64, 16, extra_rows=3)
    _check_attn(c, _attn_gpu(c))


@pytest.mark.parametrize("D,bs,H", [(128, 16, 4), (64, 32, 4), (128, 64, 8)])
def test_attention_many_tiles_a_cta_and_rows_of_every_count(D, bs, H):
    # some twenty tiles a CTA, in segments of 8 to 64 rows next to one another
    rng = np.random.default_rng(D + H)
    B = 160 // H
    new = [1 + (3 * b) % 8 for b in range(B)]
    kv = rng.integers(1200, 3000, B).tolist()
    kv[3], kv[7], kv[11] = 0, 100, 130
    c = _attn_case(rng, new, kv, 8 * H, H, D, bs)
    out = _attn_gpu(c)
    _check_attn(c, out)
    ws = sd.new_attention_workspace()
    for _ in range(20):
        assert torch.equal(_attn_gpu(c, workspace=ws), out)


def test_attention_a_sink_and_a_long_faint_tail():
    # one position far above 4000 others: the others' weights are below 2^-14 of its, together not
    D, bs = 128, 16
    rng = np.random.default_rng(12)
    c = _attn_case(rng, [1], [4095], 8, 1, D, bs)
    q = np.zeros((1, 8, D))
    q[:, :, 0] = 8.0
    c["q"] = torch.tensor(q).to(torch.bfloat16)
    c["scales"][0][:] = 1.0
    c["codes"][0][:] = 0
    c["codes"][0][..., 0] = 0
    first = c["table"][0, 0]
    c["codes"][0][first, 0, 3, 0] = ref.to_e4m3(14.0)  # score 8 * 14 / sqrt(128) = 9.9
    _check_attn(c, _attn_gpu(c))


def test_attention_scales_far_apart_and_zero_blocks():
    rng = np.random.default_rng(13)
    c = _attn_case(rng, [3, 2], [500, 200], 8, 2, 64, 16)
    c["scales"][1][:] = np.exp2(rng.integers(-30, 20, c["scales"][1].shape))
    c["scales"][0][::3] = 0.0
    c["scales"][1][::4] = 0.0
    _check_attn(c, _attn_gpu(c))
    c["scales"][1][:] = 0.0
    assert (_attn_gpu(c).float()[:5] == 0).all()


def test_attention_not_a_number_stays_in_its_place():
    rng = np.random.default_rng(14)
    c = _attn_case(rng, [4, 3], [100, 300], 8, 2, 128, 16)
    base = _attn_gpu(c).float()
    # the third new token's value of request 0 has a NaN: queries before it do not see it
    p = 102
    blk = c["table"][0, p // 16]
    c["codes"][1][blk, 0, p % 16, 5] = 0x7F
    got = _attn_gpu(c).float()
    seen = torch.isnan(got)
    assert seen[2:4, :4, 5].all() and seen.sum() == 8
    assert torch.equal(got[~seen], base[~seen])
    # a key of the last new token: only the last query's scores
    c["codes"][1][blk, 0, p % 16, 5] = 0
    c["codes"][0][c["table"][0, 103 // 16], 1, 103 % 16, 0] = 0xFF
    got = _attn_gpu(c).float()
    assert torch.isnan(got[3, 4:]).all() and not torch.isnan(got[:3]).any() and not torch.isnan(got[4:]).any()
    # a query row of no numbers spoils itself alone
    c["codes"][0][c["table"][0, 103 // 16], 1, 103 % 16, 0] = 0
    ok = _attn_gpu(c).float()
    c["q"][1, 2, 7] = float("nan")
    c["q"][5, 3, 7] = float("inf")
    got = _attn_gpu(c).float()
    rows = torch.zeros(7, 8, dtype=torch.bool, device="cuda")
    rows[1, 2] = rows[5, 3] = True
    assert torch.isnan(got[rows]).all() and torch.equal(got[~rows], ok[~rows])


def test_attention_bad_blocks_and_short_tables():
    rng = np.random.default_rng(15)
    c = _attn_case(rng, [2, 2, 1], [60, 90, 40], 8, 2, 64, 16)
    c["table"][0, 1] = -1
    c["table"][1, 3] = 1 << 30
    _check_attn(c, _attn_gpu(c))
    c = _attn_case(rng, [2, 2], [60, 90], 8, 2, 64, 16)
    c["table"] = np.ascontiguousarray(c["table"][:, :3])  # both need more
    _check_attn(c, _attn_gpu(c))
    c["kv"][1] = -2  # the first query of request 1 has nothing to attend to, the second neither
    _check_attn(c, _attn_gpu(c))
    assert (_attn_gpu(c)[2:4] == 0).all()
    c["kv"][1] = -1  # its second query sees one position
    _check_attn(c, _attn_gpu(c))


def test_attention_strided_queries_scale_stream_and_default_workspace():
    rng = np.random.default_rng(16)
    c = _attn_case(rng, [2, 3], [100, 77], 8, 2, 64, 16)
    qkv = torch.zeros(5, 12, 64, dtype=torch.bfloat16, device="cuda")
    qkv[:, 2:10] = c["q"].cuda()
    ws = sd.new_attention_workspace()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = _attn_gpu(c, q=qkv[:, 2:10], scale=0.3, workspace=ws, stream=s)
    s.synchronize()
    _check_attn(c, out, scale=0.3)
    again = _attn_gpu(c, scale=0.3, workspace=ws)
    assert torch.equal(out, again)  # same sums in the same order, whatever ran before


def test_attention_same_bits_every_time():
    c = _attn_case(np.random.default_rng(17), [3, 1, 8], [5000, 9000, 200], 16, 2, 128, 32)
    ws = sd.new_attention_workspace()
    first = _attn_gpu(c, workspace=ws)
    for _ in range(5):
        assert torch.equal(_attn_gpu(c, workspace=ws), first)


def test_attention_in_a_cuda_graph():
    c = _attn_case(np.random.default_rng(18), [2, 2], [300, 40], 8, 2, 128, 16)
    want = _attn_gpu(c)
    q, cu, kv, table = c["q"].cuda(), dev(c["cu"]), dev(c["kv"]), dev(c["table"])
    kc, vc = (dev(x).view(E4M3) for x in c["codes"])
    ks, vs = dev(c["scales"][0]), dev(c["scales"][1])
    out, ws = torch.zeros_like(q), sd.new_attention_workspace()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sd.spec_attention(q, cu, kv, table, kc, vc, ks, vs, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        wait_gpu()
        assert torch.equal(out, want)


# -------------------------------------------------------- spec_process_logits

def _logit_case(rng, B, n, V, S, masks=3, biases=6, ragged=True):
    i32 = lambda x: np.asarray(x, dtype=np.int32)  # noqa: E731
    hl = rng.integers(0, S + 1, B)
    off = np.concatenate([[0], np.cumsum(rng.integers(0, biases + 1, B))])
    few = max(1, min(V, 40))
    c = dict(history=i32(rng.integers(0, few, (B, S))), history_len=i32(hl), prompt_len=i32([rng.integers(0, h + 1) for h in hl]),
             draft_tokens=i32(rng.integers(0, few, (B, n))), draft_len=i32(rng.integers(0, n + 1, B) if ragged else [n] * B),
             repetition=rng.uniform(0.5, 2.0, B).astype(np.float32), presence=rng.uniform(-1, 1, B).astype(np.float32),
             frequency=rng.uniform(-0.5, 0.5, B).astype(np.float32), bias_offsets=i32(off),
             bias_ids=i32(rng.integers(0, V, max(1, off[-1]))), bias_values=rng.normal(0, 5, max(1, off[-1])).astype(np.float32))
    if masks:
        c["mask"] = rng.integers(-2**31, 2**31, (masks, (V + 31) // 32)).astype(np.int32)
        c["mask_rows"] = i32(rng.integers(-1, masks, (B, n + 1)))
    return c


def _run_logits(x, c, in_place=False, err=None):
    out = x.clone() if in_place else torch.full_like(x, 77.0)
    sd.spec_process_logits(out if in_place else x, out=out, error_word=err, **{k: dev(v) for k, v in c.items()})
    wait_gpu()
    return out


def _check_logits(x, c, got, untouched, n_of=None):
    """Tolerance: at most six operations in 32 bits on the magnitudes that meet
    in a value (2^-24 each, doubled), then one rounding to the type (2^-9 of a
    bf16 value, doubled where the 32-bit result sits on the other side of a tie)."""
    want, mag = ref.process_logits(x.double().cpu().numpy(), **c)
    B, rows, V = x.shape
    n = c.get("draft_len", np.full(B, rows - 1))
    got = got.double().cpu().numpy()
    for b in range(B):
        past = got[b, n[b] + 1:]
        assert (past == (untouched if np.isscalar(untouched) else untouched[b, n[b] + 1:])).all()
        w, g, m = want[b, :n[b] + 1], got[b, :n[b] + 1], mag[b, :n[b] + 1]
        inf = np.isinf(w)
        assert (g[inf] == w[inf]).all() and np.isfinite(g[~inf]).all()
        tol = 12 * 2.0 ** -24 * m + (2.0 ** -8 * np.abs(w) if x.dtype == torch.bfloat16 else 0)
        assert (np.abs(g[~inf] - w[~inf]) <= tol[~inf]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,n,V,S", [(1, 0, 1, 1), (1, 0, 7, 5), (3, 2, 33, 40), (4, 3, 1024, 300), (2, 7, 4097, 50), (5, 1, 4104, 1),
                                     (2, 4, 32003, 3000), (1, 12, 5000, 20)])
def test_process_logits(B, n, V, S, dtype):
    rng = np.random.default_rng(V + n)
    c = _logit_case(rng, B, n, V, S)
    x = torch.tensor(rng.normal(0, 3, (B, n + 1, V))).to(dtype).cuda()
    _check_logits(x, c, _run_logits(x, c), 77.0)
    _check_logits(x, c, _run_logits(x, c, in_place=True), x.double().cpu().numpy())


@pytest.mark.parametrize("keys", [(), ("history",), ("bias",), ("mask",), ("penalties",), ("history", "penalties")])
def test_process_logits_parts_alone(keys):
    rng = np.random.default_rng(len(keys))
    full = _logit_case(rng, 3, 2, 2048, 64)
    c = {k: full[k] for k in ("draft_tokens", "draft_len")}
    names = {"history": ("history", "history_len", "prompt_len"), "bias": ("bias_offsets", "bias_ids", "bias_values"),
             "mask": ("mask", "mask_rows"), "penalties": ("repetition", "presence", "frequency")}
    for k in keys:
        c.update({n: full[n] for n in names[k]})
    x = torch.tensor(rng.normal(0, 3, (3, 3, 2048))).to(torch.bfloat16).cuda()
    _check_logits(x, c, _run_logits(x, c), 77.0)


def test_process_logits_empty_masks_infinities_and_nan():
    rng = np.random.default_rng(21)
    B, n, V = 2, 1, 1000
    c = _logit_case(rng, B, n, V, 30, masks=2, ragged=False)
    c["mask"][0] = 0                      # nothing allowed
    c["mask_rows"][:] = [[0, 1], [-1, 0]]
    x = torch.tensor(rng.normal(0, 3, (B, n + 1, V))).cuda()
    x[:, :, 5] = float("-inf")
    x[1, 0, 6] = float("nan")
    x[0, :, 7] = float("nan")
    x = x.float()
    got = _run_logits(x, c)
    assert (got[0, 0] == float("-inf")).all() and (got[1, 1] == float("-inf")).all()
    assert (got[:, :, 5] == float("-inf")).all() and torch.isnan(got[1, 0, 6])
    allowed = (int(c["mask"][1, 0]) >> 7) & 1
    assert torch.isnan(got[0, 1, 7]) if allowed else got[0, 1, 7] == float("-inf")


def test_process_logits_out_of_range_ids_and_bad_penalties():
    rng = np.random.default_rng(22)
    c = _logit_case(rng, 4, 2, 500, 40)
    c["history"][:, ::3] = -1
    c["history"][:, 1::7] = 500
    c["draft_tokens"][0] = [-5, 900]
    c["bias_ids"][::2] = 700
    x = torch.tensor(rng.normal(0, 3, (4, 3, 500))).float().cuda()
    err = err_word()
    _check_logits(x, c, _run_logits(x, c, err=err), 77.0)
    assert err.item() == 0
    c["repetition"][:] = [0.0, -1.0, float("nan"), float("inf")]
    c["presence"][1] = float("inf")
    c["frequency"][2] = float("nan")
    got = _run_logits(x, c, err=err)
    assert err.item() == sd.DEV_ERR_PENALTY
    c["repetition"][:] = 1.0
    c["presence"][1] = c["frequency"][2] = 0.0
    _check_logits(x, c, got, 77.0)
    err.zero_()
    c["history_len"][0], c["draft_len"][1], c["prompt_len"][2] = 99, 7, 50
    got = _run_logits(x, c, err=err)
    assert err.item() == sd.DEV_ERR_PENALTY
    c["history_len"][0], c["draft_len"][1], c["prompt_len"][2] = 40, 2, c["history_len"][2]
    _check_logits(x, c, got, 77.0)


def test_process_logits_many_biases_and_long_history():
    # more biases of one CTA's entries than its list holds; one token made 5000 times
    rng = np.random.default_rng(23)
    c = _logit_case(rng, 2, 1, 2500, 5000, ragged=False)
    c["history"][0] = 11
    c["history_len"][0], c["prompt_len"][0] = 5000, 0
    k = 900
    c["bias_offsets"] = np.array([0, k, 2 * k], dtype=np.int32)
    c["bias_ids"] = rng.integers(0, 300, 2 * k).astype(np.int32)
    c["bias_values"] = rng.normal(0, 1, 2 * k).astype(np.float32)
    x = torch.tensor(rng.normal(0, 3, (2, 2, 2500))).float().cuda()
    got = _run_logits(x, c)
    want, mag = ref.process_logits(x.double().cpu().numpy(), **c)
    # sums of up to a dozen biases in 32 bits
    m = mag + 40.0
    ok = ~np.isinf(want)
    assert (np.abs(got.double().cpu().numpy()[ok] - want[ok]) <= 32 * 2.0 ** -24 * m[ok]).all()
    assert (got.cpu().numpy()[~ok] == -np.inf).all()
    # the order of a token's biases is the list's: the same bits every time
    assert torch.equal(got, _run_logits(x, c))


def test_process_logits_feeds_the_verify_step():
    # a grammar that allows one token a row: greedy verification accepts exactly the drafts that follow it
    B, n, V = 6, 3, 5000
    rng = np.random.default_rng(24)
    path = rng.integers(0, V, (B, n + 1))
    mask = np.zeros((B * (n + 1), (V + 31) // 32), dtype=np.uint32)
    for i, v in enumerate(path.ravel()):
        mask[i, v // 32] = np.uint32(1) << np.uint32(v % 32)
    drafts = path[:, :n].copy()
    wrong = np.array([0, 1, 2, 3, 3, 1])
    for b in range(B):
        if wrong[b] < n:
            drafts[b, wrong[b]] = (drafts[b, wrong[b]] + 1) % V
    x = torch.randn(B, n + 1, V, device="cuda").to(torch.bfloat16)
    d = dev(drafts.astype(np.int32))
    L = torch.full((B,), n, dtype=torch.int32, device="cuda")
    sd.spec_process_logits(x, draft_tokens=d, mask=dev(mask.view(np.int32)), mask_rows=dev(np.arange(B * (n + 1), dtype=np.int32).reshape(B, n + 1)))
    acc, out = sd.spec_verify(x, None, d, L, torch.zeros(B, device="cuda"))
    wait_gpu()
    assert acc.tolist() == wrong.tolist()
    for b in range(B):
        assert out[b, :wrong[b] + 1].tolist() == path[b, :wrong[b] + 1].tolist()


# ------------------------------------------- where the kernels' parts meet

@pytest.mark.parametrize("B,capacity", [(8192, 20000), (8193, 20000), (3000, 3)])
@pytest.mark.parametrize("alias", [False, True])
def test_block_step_many_requests(B, capacity, alias):
    rng = np.random.default_rng(B)
    c = _block_case(rng, B, 16, 3, spare=B // 2, most_new=5)
    _check_blocks(c, 16, capacity, alias=alias)


def test_block_step_positions_at_any_alignment():
    rng = np.random.default_rng(2)
    for capacity in (1, 2, 3, 5, 31, 33):
        c = _block_case(rng, 9, 16, 4, spare=30, most_new=4)
        _check_blocks(c, 16, capacity)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_append_long_runs_with_infinities_and_nan(D, dtype):
    # whole blocks of 128: a team's runs, and the longest a block can have
    rng = np.random.default_rng(D)
    H, bs, N = 3, 128, 7
    kc, ks = _cache(rng, N, H, bs, D)
    vc, vs = _cache(rng, N, H, bs, D)
    slots = np.concatenate([np.arange(2 * bs, 3 * bs), np.arange(5 * bs + 1, 6 * bs), np.arange(60), 3 * bs + np.arange(90, 128)])
    x = torch.randn(len(slots), 2 * H, D, generator=torch.Generator(device="cuda").manual_seed(D), device="cuda").to(dtype)
    x[17, 0, 5] = float("inf")
    x[150, 1, 9] = -float("inf")
    x[150, 1, 10] = float("nan")
    x[270, 4, 0] = float("nan")
    _check_append(x[:, :H], x[:, H:], slots, kc, vc, ks, vs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("a,b,w", [(0, 0, 1), (1, 1, 2), (3, 3, 3), (1, 2, 0), (5, 0, 1)])
def test_process_logits_at_any_alignment(a, b, w, dtype):
    # logits, out and masks that start a, b and w elements past 16 bytes; rows of an odd length
    rng = np.random.default_rng(10 * a + b)
    B, n, V = 3, 2, 9001
    c = _logit_case(rng, B, n, V, 200)
    x = torch.tensor(rng.normal(0, 3, (B, n + 1, V))).to(dtype).cuda()
    at = lambda t, k: torch.cat([t.new_full((k,), 9), t.flatten(), t.new_full((3,), 9)])[k:k + t.numel()].view(t.shape)  # noqa: E731
    args = {k: dev(v) for k, v in c.items()}
    args["mask"] = at(args["mask"], w)
    src, out = at(x, a), at(torch.full_like(x, 77.0), b)
    assert src.data_ptr() % 16 == a * x.element_size() % 16 and out.data_ptr() % 16 == b * x.element_size() % 16
    sd.spec_process_logits(src, out=out, **args)
    wait_gpu()
    _check_logits(x, c, out, 77.0)
    sd.spec_process_logits(src, **args)
    wait_gpu()
    _check_logits(x, c, src, x.double().cpu().numpy())
    # nothing around the tensors has changed
    for t, k in ((src, a), (out, b)):
        whole = t.as_strided((k + t.numel() + 3,), (1,), 0)
        assert (whole[:k] == 9).all() and (whole[-3:] == 9).all()


@pytest.mark.parametrize("in_place", [False, True])
def test_process_logits_many_items_and_the_most_rows(in_place):
    # more items than two for each SM, requests with 1 to 65 rows, some rows without a mask
    rng = np.random.default_rng(31)
    for B, n, V in ((700, 1, 700), (40, 64, 600), (160, 3, 17000)):
        c = _logit_case(rng, B, n, V, 60, biases=4)
        x = torch.tensor(rng.normal(0, 3, (B, n + 1, V))).to(torch.bfloat16).cuda()
        _check_logits(x, c, _run_logits(x, c, in_place=in_place), x.double().cpu().numpy() if in_place else 77.0)


def test_process_logits_more_biases_than_an_item_lists():
    rng = np.random.default_rng(32)
    B, n, V = 4, 1, 300
    c = _logit_case(rng, B, n, V, 30, biases=900)
    x = torch.tensor(rng.normal(0, 3, (B, n + 1, V))).to(torch.float32).cuda()
    # (its biases meet in one value: as many additions as there are)
    want, mag = ref.process_logits(x.double().cpu().numpy(), **c)
    got = _run_logits(x, c).double().cpu().numpy()
    most = int(np.diff(c["bias_offsets"]).max())
    for b in range(B):
        rows = c["draft_len"][b] + 1
        w, g, m = want[b, :rows], got[b, :rows], mag[b, :rows]
        inf = np.isinf(w)
        assert (g[inf] == w[inf]).all()
        assert (np.abs(g[~inf] - w[~inf]) <= (12 + most) * 2.0 ** -24 * m[~inf]).all()


@pytest.mark.parametrize("new,kv,Hq,H,D", [
    ([14], [300], 64, 8, 128), ([13], [249], 64, 8, 128), ([22], [300], 64, 8, 64), ([28], [300], 32, 8, 64),
    ([6, 6, 8], [16, 3231, 260], 8, 1, 64)])
def test_attention_items_that_begin_at_the_end_of_a_part(new, kv, Hq, H, D):
    # two CTAs of an item's have no tile of it; the workspace is ready for the next call all the same
    c = _attn_case(np.random.default_rng(len(new) + new[0]), new, kv, Hq, H, D, 16)
    ws = sd.new_attention_workspace()
    for _ in range(2):
        _check_attn(c, _attn_gpu(c, workspace=ws))
        assert not ws[:64 * 1024].any()
    other = _attn_case(np.random.default_rng(5), [2], [20000], 8, 1, 128, 64)
    _check_attn(other, _attn_gpu(other, workspace=ws))


@pytest.mark.parametrize("D", [64, 128])
def test_attention_many_short_items_a_cta(D):
    # items of 8 to 64 rows and one to three tiles next to one another, several whole ones a CTA: what the output
    # warps keep of one must not meet the next
    rng = np.random.default_rng(100 + D)
    B, H = 170, 6
    new = rng.integers(1, 9, B).tolist()
    kv = rng.integers(0, 260, B).tolist()
    c = _attn_case(rng, new, kv, 8 * H, H, D, 16)
    ws = sd.new_attention_workspace()
    base = _attn_gpu(c, workspace=ws)
    _check_attn(c, base)
    for _ in range(20):
        assert torch.equal(_attn_gpu(c, workspace=ws), base)
    # values of new tokens that are no numbers, in a dimension of every (request, head)
    want = torch.zeros(base.shape, dtype=torch.bool)
    for b in range(B):
        for h in range(H):
            i, d = int(rng.integers(0, new[b])), int(rng.integers(0, D))
            p = kv[b] + i
            c["codes"][1][c["table"][b, p // 16], h, p % 16, d] = 0x7F
            want[int(c["cu"][b]) + i:int(c["cu"][b + 1]), 8 * h:8 * h + 8, d] = True
    want = want.cuda()
    for _ in range(20):
        got = _attn_gpu(c, workspace=ws)
        assert torch.equal(torch.isnan(got), want)
        assert torch.equal(got[~want], base[~want])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bad", [3, 1 << 30, -2, -2**31])
def test_process_logits_reports_masks_that_are_not_there(bad, in_place):
    rng = np.random.default_rng(33)
    B, n, V = 3, 2, 700
    c = _logit_case(rng, B, n, V, 20, ragged=False)
    c["mask_rows"][:] = rng.integers(-1, 3, (B, n + 1))
    c["draft_len"][2] = 1
    x = torch.tensor(rng.normal(0, 3, (B, n + 1, V))).float().cuda()
    untouched = x.double().cpu().numpy() if in_place else 77.0
    err = err_word()
    # a row that is not there may name anything
    c["mask_rows"][2, 2] = bad
    _check_logits(x, c, _run_logits(x, c, in_place=in_place, err=err), untouched)
    assert err.item() == 0
    c["mask_rows"][1, 2] = bad
    got = _run_logits(x, c, in_place=in_place, err=err)
    assert err.item() == sd.DEV_ERR_PENALTY
    c["mask_rows"][1, 2] = -1  # as a row without a mask
    _check_logits(x, c, got, untouched)


@pytest.mark.parametrize("capacity", [0, 5, 5000])
@pytest.mark.parametrize("alias", [False, True])
def test_block_step_without_requests_leaves_its_outputs(capacity, alias):
    e = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    ring, state = torch.arange(7, dtype=torch.int32, device="cuda"), dev(np.array([5, 4], dtype=np.int32))
    fill = lambda n: torch.full((n,), 99, dtype=torch.int32, device="cuda")  # noqa: E731
    out = sd.BlockStep(e(0), e(0), state if alias else fill(2), fill(1), fill(1), fill(capacity), fill(capacity))
    err = err_word()
    step = sd.kv_block_step(e(0, 3), e(0), e(0), e(0), ring, state, 16, capacity, out=out, error_word=err)
    wait_gpu()
    assert step.ring_state.tolist() == [5, 4] and step.cu_tokens.tolist() == [0] and step.cu_blocks.tolist() == [0]
    assert (step.slot_map == -1).all() and (step.positions == -1).all()
    assert ring.tolist() == list(range(7)) and state.tolist() == [5, 4] and err.item() == 0
    # outputs of its own; in a graph; and the ring's state is looked at as ever
    junk = [torch.full((4 + 2 * capacity,), 99, dtype=torch.int32, device="cuda") for _ in range(3)]
    del junk
    step = sd.kv_block_step(e(0, 3), e(0), e(0), e(0), ring, state, 16, capacity)
    wait_gpu()
    assert step.ring_state.tolist() == [5, 4] and step.cu_tokens.tolist() == [0] and (step.slot_map == -1).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sd.kv_block_step(e(0, 3), e(0), e(0), e(0), ring, state, 16, capacity, out=out, error_word=err)
    for t in out:
        if t is not state:
            t.fill_(99)
    state[1] = 9
    g.replay()
    wait_gpu()
    assert out.ring_state.tolist() == [5, 7] and (out.positions == -1).all() and err.item() == sd.DEV_ERR_BLOCKS


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,n", [(64, 1), (128, 5), (128, 16)])
def test_append_infinities_among_zeros_are_the_largest_number(D, n, dtype):
    # scale 0: the codes are still numbers (448 times 0 is 0; a NaN would spoil every query that sees it)
    kc = np.full((4, 1, 16, D), 0x11, dtype=np.uint8)
    zero, two = np.zeros((4, 1), dtype=np.float32), np.full((4, 1), 2.0, dtype=np.float32)
    x = torch.zeros(n, 1, D, device="cuda").to(dtype)
    x[0, 0, 1], x[n - 1, 0, 2], x[n - 1, 0, 7] = float("inf"), -float("inf"), float("nan")
    want = np.zeros((n, D))
    want[0, 1], want[n - 1, 2], want[n - 1, 7] = 448, -448, np.nan
    # into an empty block, behind a block's older tokens of scale 0, and behind some of scale 2
    for first, scale, after in ((16, two, 0.0), (32 + 16 - n, zero, 0.0), (48 + 16 - n, two, 0.0 if n == 16 else 2.0)):
        slots = np.arange(first, first + n)
        got = _run_append(x, -x, slots, (kc, kc, scale, scale))
        for codes, scales, sign in ((got[0], got[2], 1), (got[1], got[3], -1)):
            b, o = first // 16, first % 16
            assert np.array_equal(ref.VALUES[codes[b, 0, o:o + n]], sign * want, equal_nan=True)
            assert (codes[b, 0, :o] == 0x11).all() and scales[b, 0] == after


def test_attention_reports_requests_that_decrease_or_leave_the_tokens():
    rng = np.random.default_rng(40)
    c = _attn_case(rng, [2, 2, 0], [60, 90, 10], 8, 2, 64, 16)
    ws = sd.new_attention_workspace()
    want = _attn_gpu(c, workspace=ws)
    assert sd.get_error(ws) == 0
    for cu in ([0, 2, 9, 4], [-3, 2, 4, 1], [0, 2, 4, -1], [0, 2, 5, 5]):
        c["cu"] = np.array(cu, dtype=np.int32)
        assert torch.equal(_attn_gpu(c, workspace=ws), want)
        assert sd.get_error(ws) == sd.DEV_ERR_SEGMENT
    c["cu"] = np.array([0, 2, 4, 4], dtype=np.int32)
    assert torch.equal(_attn_gpu(c, workspace=ws), want)
    assert sd.get_error(ws) == 0


def test_attention_requests_that_overlap_past_its_count():
    # 64 tokens that every second of 4096 requests claims: 10^10 units in all
    B, T, H, D, bs, width = 4096, 64, 64, 64, 128, 8192
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T] * (B // 2) + [0], **i32)
    kv = torch.full((B,), width * bs - T, **i32)
    table = torch.zeros(B, width, **i32)
    cache = torch.zeros(1, H, bs, D, dtype=torch.uint8, device="cuda").view(E4M3)
    scale = torch.ones(1, H, device="cuda")
    q = torch.randn(T, H, D, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 77.0)
    ws = sd.new_attention_workspace()
    sd.spec_attention(q, cu, kv, table, cache, cache, scale, scale, out=out, workspace=ws)
    wait_gpu()
    assert (out == 77.0).all() and sd.get_error(ws) == sd.DEV_ERR_SEGMENT and not ws.any()
    c = _attn_case(np.random.default_rng(41), [3, 5], [400, 77], 16, 2, 64, 16)
    _check_attn(c, _attn_gpu(c, workspace=ws))


@pytest.mark.parametrize("D", [64, 128])
def test_attention_lengths_far_past_the_table(D):
    # all tokens attend to what the table's row holds, however long the request is said to be
    c = _attn_case(np.random.default_rng(42), [3, 5, 2], [400, 77, 250], 16, 2, D, 16)
    c["table"] = np.maximum(c["table"][:, :4], 0)
    c["codes"] = [np.where((x & 0x7F) == 0x7F, 0, x).astype(np.uint8) for x in c["codes"]]
    c["kv"][:] = 1000
    want = _attn_gpu(c)
    _check_attn(c, want)
    for far in (2**31 - 1, 2**31 - 3, 1 << 30):
        c["kv"][:] = far
        assert torch.equal(_attn_gpu(c), want)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_queries_far_below_their_rows_largest(D):
    # the largest of a row meets keys of 0, so the scores are those of the rest: 2^-16 to 2^-9 of it
    rng = np.random.default_rng(D)
    c = _attn_case(rng, [1], [1], 8, 1, D, 16, stale=False)
    u = np.exp2(-8.0) * np.array([2.34375, 1.25, 1.2578125, 0.6171875, 0.31, 0.155, 0.08, 0.04])[:, None] * np.ones((8, D))
    u[3:] *= rng.uniform(1, 2, (5, D))
    signs = np.where(rng.random(D) < 0.5, -1.0, 1.0)
    q = u * signs
    q[:, 0] = 225.0
    c["q"] = torch.tensor(q[None]).to(torch.bfloat16)
    block = c["table"][0, 0]
    for p in (0, 1):  # two positions with opposite keys and values
        key = np.where(signs * (1 - 2 * p) > 0, ref.to_e4m3(448.0), ref.to_e4m3(-448.0))
        key[0] = 0
        c["codes"][0][block, 0, p] = key
        c["codes"][1][block, 0, p] = ref.to_e4m3(1.0 - 2 * p)
    c["scales"][0][:] = c["scales"][1][:] = 1.0
    qs = c["q"].double().numpy()
    for r in range(8):
        # every row's scores are +-0.5; a query's values are off by 2^-14 at most, which the softmax's quotient
        # takes twice; the rest as in _check_attn
        s = 0.5 / (448 * np.abs(qs[0, r, 1:]).sum())
        want, mag, _ = ref.attention(qs, c["cu"], c["kv"], c["table"], c["codes"][0], c["codes"][1], c["scales"][0],
                                     c["scales"][1], s)
        got = _attn_gpu(c, scale=s).double().cpu().numpy()
        off = 2.0 ** -14 * 448 * (D - 1) * s
        tol = 2.0 ** -8 * np.abs(want[0, r]) + (2.0 ** -8 + 2 * off) * mag[0, r]
        assert (np.abs(got[0, r] - want[0, r]) <= tol).all(), (r, got[0, r, 0], want[0, r, 0], tol[0])


def test_strides_of_a_single_token_or_head_do_not_matter():
    rng = np.random.default_rng(43)
    buf = torch.randn(8 * 64, device="cuda").to(torch.bfloat16)
    kc, ks = _cache(rng, 4, 8, 16, 64)
    _check_append(buf.as_strided((1, 8, 64), (7, 64, 1)), buf.as_strided((1, 8, 64), (1, 64, 1)), np.array([21]), kc, kc, ks, ks)
    kc, ks = _cache(rng, 4, 1, 16, 64)
    slots = np.arange(20, 28)
    _check_append(buf.as_strided((8, 1, 64), (64, 3, 1)), buf.as_strided((8, 1, 64), (64, 0, 1)), slots, kc, kc, ks, ks)
    c = _attn_case(rng, [8], [30], 1, 1, 64, 16)
    c["q"] = buf.view(8, 1, 64).cpu()
    out = _attn_gpu(c)
    assert torch.equal(_attn_gpu(c, q=buf.as_strided((8, 1, 64), (64, 5, 1))), out)
    c = _attn_case(rng, [1], [30], 8, 1, 64, 16)
    c["q"] = buf.view(1, 8, 64).cpu()
    out = _attn_gpu(c)
    assert torch.equal(_attn_gpu(c, q=buf.as_strided((1, 8, 64), (3, 64, 1))), out)


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int32, torch.float64])
def test_attention_workspaces_of_any_type(dtype):
    c = _attn_case(np.random.default_rng(44), [3], [400], 16, 2, 64, 16)
    ws = torch.zeros(sd.ATTENTION_WORKSPACE_BYTES // torch.empty(0, dtype=dtype).element_size(), dtype=dtype, device="cuda")
    _check_attn(c, _attn_gpu(c, workspace=ws))
    with pytest.raises(sd.SpecDecError, match="WORKSPACE"):
        _attn_gpu(c, workspace=ws[:-1])
