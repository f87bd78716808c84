"""More operators of a decode step: what is measured, with a plain form of each.

Four operators, a case's ``"op"`` names the one it calls:

* ``sample``: tokens drawn with temperature, top-k, top-p and min-p from given random numbers, and the rows cut to
  what may be drawn, as ``spec_verify`` reads them;
* ``rotary``: rotary positions of the new tokens' queries and keys;
* ``fork``: requests that go on from others' tokens over a paged cache: shared, copied and freed blocks;
* ``compact``: a cache's blocks moved to its lowest ids.

``own`` selects the framework's calls; otherwise ``run`` is the plain form.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
FAR = 131072  # the context that scaled rotary positions were trained on is a part of this


def listed():
    return [
        # one draft step of a single user: a token and its row for the verify call
        dict(name="sample_draft_one", op="sample", B=1, n=0, V=128256, dtype="bf16", draw=True, rows=True, flat=0.0, masked=0.0),
        # the target's rows of the draft-target batch, cut before they are verified
        dict(name="sample_verify_64", op="sample", B=64, n=4, V=128256, dtype="bf16", draw=False, rows=True, flat=0.2, masked=0.5),
        # plain sampling of a large batch: tokens only, an odd vocabulary, fp32 rows
        dict(name="sample_tokens_f32_300", op="sample", B=300, n=0, V=50001, dtype="f32", draw=True, rows=False, flat=0.2, masked=0.0),
        # ragged verify batch: up to eight rows of each request
        dict(name="sample_ragged_128", op="sample", B=128, n=7, V=152064, dtype="bf16", draw=True, rows=True, flat=0.1, masked=0.1),
        # one user, one token, the small draft model's heads
        dict(name="rotary_one", op="rotary", T=1, Hq=32, H=8, D=64, part=64, layout="pairs", dtype="bf16", scaling="none"),
        # MTP verify in fp32, half of the head turned
        dict(name="rotary_mtp_512", op="rotary", T=512, Hq=32, H=8, D=128, part=64, layout="half", dtype="f32", scaling="linear"),
        # prompts of some thousand tokens each, contexts past those of the training
        dict(name="rotary_prompts", op="rotary", T=50000, Hq=32, H=8, D=128, part=128, layout="half", dtype="bf16", scaling="yarn"),
        # eight continuations of one prompt
        dict(name="fork_samples_one", op="fork", P=1, n=8, beams=False, kept=1900, back=0.0, bs=16, H=8, D=64, layers=16),
        # beam search: 64 groups of four choose their parents anew
        dict(name="fork_beams_64", op="fork", P=64, n=4, beams=True, kept=300, back=0.0, bs=32, H=8, D=128, layers=4),
        # four samples of each of 128 long prompts, some of them from an earlier token
        dict(name="fork_samples_128", op="fork", P=128, n=4, beams=False, kept=700, back=0.3, bs=64, H=4, D=128, layers=4),
        # a small cache after some requests have ended
        dict(name="compact_small", op="compact", B=24, kept=600, used=0.6, bs=16, H=8, D=64, layers=4),
        # a large one, half empty
        dict(name="compact_half", op="compact", B=200, kept=1200, used=0.5, bs=16, H=8, D=128, layers=2),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "rotary", "fork", "compact"])
    if op == "sample":
        n = rng.randint(0, 7)
        V = rng.choice([1024, 32003, 50001, 128256, 129280, 152064])
        B = _log(rng, 1, max(1, min(512, int(1.0e8 / ((n + 1) * V)))))
        mode = rng.choice([(True, True), (True, False), (False, True)])
        return dict(op=op, B=B, n=n, V=V, dtype=rng.choice(["bf16", "bf16", "f32"]), draw=mode[0], rows=mode[1],
                    flat=rng.choice([0.0, 0.2, 0.5]), masked=rng.choice([0.0, 0.1, 0.5]))
    if op == "rotary":
        Hq, H, D = rng.choice([(32, 8, 64), (64, 8, 128), (32, 8, 128), (8, 8, 128), (12, 2, 128), (8, 1, 64)])
        return dict(op=op, T=_log(rng, 1, 13000), Hq=Hq, H=H, D=D, part=rng.choice([D, D, D // 2, 40]),
                    layout=rng.choice(["half", "pairs"]), dtype=rng.choice(["bf16", "f32"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]))
    H, D = rng.choice([(8, 64), (8, 128), (1, 128), (4, 128)])
    bs, layers = rng.choice([16, 32, 64, 128]), _log(rng, 1, 16)
    most = 600e6 / (2 * H * D * layers)  # tokens that the layers' caches may hold
    if op == "fork":
        n, beams = rng.randint(2, 8), rng.random() < 0.5
        kept = _log(rng, 1, 2000)
        P = _log(rng, 1, max(1, min(128, int(most / ((n if beams else 1) * (kept + bs) + 2 * n * bs)))))
        return dict(op=op, P=P, n=n, beams=beams, kept=kept, back=rng.choice([0.0, 0.3]), bs=bs, H=H, D=D, layers=layers)
    kept, used = _log(rng, 1, 2000), rng.choice([0.3, 0.5, 0.9, 1.0])
    B = _log(rng, 1, max(1, min(300, int(most * used / (kept + bs)))))
    return dict(op=op, B=B, kept=kept, used=used, bs=bs, H=H, D=D, layers=layers)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def _spread(lo, hi, B):
    """B whole numbers from hi down to lo: the lengths that a case's requests have in some order."""
    return [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]


def prepare(case, seed):
    s = {"op": case["op"]}
    {"sample": _prepare_sample, "rotary": _prepare_rotary, "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](case, seed, s)
    return s


def _prepare_sample(case, seed, s):
    g = _gen(seed)
    B, n, V = case["B"], case["n"], case["V"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    rand = lambda *shape: torch.rand(*shape, generator=g, device=DEV)  # noqa: E731
    # a model's row: most of the vocabulary near its mean, some candidates far above it; flat rows have none
    x = torch.empty(B, n + 1, V, dtype=dt, device=DEV).normal_(0.0, 2.5, generator=g)
    many = min(64, V)
    ids = ((torch.arange(many, device=DEV) + 0.999 * rand(B, n + 1, many)) * (V / many)).long().clamp(max=V - 1)  # one in each part
    lift = (9.0 + 9.0 * rand(B, n + 1, 1)) * rand(B, n + 1, many).square()
    lift = torch.where(rand(B, n + 1, 1) < case["flat"], 0.0, lift).to(dt)
    x.scatter_(2, ids, x.gather(2, ids) + lift)
    # grammars leave a part of the vocabulary
    for b in range(B):
        if case["masked"] and float(np.random.default_rng([seed, b]).random()) < case["masked"]:
            x[b].masked_fill_(rand(1, V) < 0.6, -math.inf)
    s["logits"] = x
    pick = lambda values: torch.tensor(values, device=DEV)[(rand(B) * len(values)).long().clamp(max=len(values) - 1)]  # noqa: E731
    T = 0.3 + rand(B)
    s["temperature"] = torch.where(rand(B) < 0.1, 0.0, T)
    s["top_k"] = pick([0, 0, 1, 20, 50, 200, 5000]).to(torch.int32)
    s["top_p"] = torch.where(rand(B) < 0.3, 1.0, 0.75 + 0.245 * rand(B))
    s["min_p"] = torch.where(rand(B) < 0.6, 0.0, 0.15 * rand(B))
    s["draft_len"] = ((n + 1) // 2 + (rand(B) * (n + 1 - (n + 1) // 2)).to(torch.int32)).clamp(max=n).to(torch.int32)
    s["uniform"] = rand(B, n + 1) if case["draw"] else None
    s["tokens"] = torch.zeros(B, n + 1, dtype=torch.int32, device=DEV) if case["draw"] else None
    s["out"] = torch.zeros(B, n + 1, V, dtype=dt, device=DEV) if case["rows"] else None


def _scaling(case):
    """How the frequencies are scaled for contexts longer than the training's."""
    return {"none": None, "linear": dict(type="linear", factor=4.0), "ntk": dict(type="ntk", factor=8.0),
            "yarn": dict(type="yarn", factor=16.0, original=FAR // 16, fast=32.0, slow=1.0),
            "bands": dict(type="bands", factor=8.0, original=FAR // 16, low=1.0, high=4.0)}[case["scaling"]]


def _frequencies(R, base, scaling):
    """Angle a position of each pair, in 64 bits, and the factor of the result."""
    i = np.arange(R // 2, dtype=np.float64)
    f = base ** (-2.0 * i / R)
    if scaling is None:
        return f, 1.0
    by = scaling["factor"]
    if scaling["type"] == "linear":
        return f / by, 1.0
    if scaling["type"] == "ntk":
        return (base * by ** (R / (R - 2.0))) ** (-2.0 * i / R), 1.0
    length = scaling["original"]
    if scaling["type"] == "yarn":
        at = lambda turns: R * math.log(length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(scaling["fast"])), 0), min(math.ceil(at(scaling["slow"])), R - 1)
        ramp = np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        return f * (1.0 - ramp) + f / by * ramp, 0.1 * math.log(by) + 1.0
    turns = length * f / (2.0 * math.pi)
    smooth = np.clip((turns - scaling["low"]) / (scaling["high"] - scaling["low"]), 0.0, 1.0)
    return f * smooth + f / by * (1.0 - smooth), 1.0


def _prepare_rotary(case, seed, s):
    g = _gen(seed)
    T, Hq, H, D = case["T"], case["Hq"], case["H"], case["D"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    qkv = torch.randn(T, Hq + 2 * H, D, generator=g, device=DEV).to(dt)  # a fused projection's rows
    s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + H]
    s["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device=DEV)
    s["k_out"] = torch.zeros(T, H, D, dtype=dt, device=DEV)
    # runs of tokens from a position each; a few places of the batch hold no token
    run = 1 + T // 40
    first = (torch.rand((T + run - 1) // run, generator=g, device=DEV) * (FAR - run)).to(torch.int32)
    p = first.repeat_interleave(run)[:T] + (torch.arange(T, device=DEV) % run).to(torch.int32)
    s["positions"] = torch.where(torch.rand(T, generator=g, device=DEV) < (0.02 if T > 8 else 0.0), -1, p).to(torch.int32)
    s["layout"] = case["layout"]
    f, factor = _frequencies(case["part"], 10000.0, _scaling(case))
    if own:
        import speculative_decoding_verification_80_gb300 as sd

        s["turns"], s["factor"] = sd.rotary_turns(case["part"], base=10000.0, scaling=_scaling(case), device=DEV)
    else:
        s["freq"], s["factor"] = torch.as_tensor(f).to(DEV), factor


def _caches(s, case, N, g):
    """The layers' caches, parts of four tensors: codes of unit normal rows, and scales."""
    L, H, D, bs = case["layers"], case["H"], case["D"], case["bs"]
    k, v = (torch.stack([(128.0 * torch.randn(N, H, bs, D, generator=g, device=DEV, dtype=torch.bfloat16)).to(E4M3) for _ in range(L)]) for _ in range(2))
    ks, vs = (torch.exp2(torch.floor(-9.0 + 2.0 * torch.rand(L, N, H, generator=g, device=DEV))) for _ in range(2))
    s["caches"] = {"k": k, "v": v, "k_scale": ks, "v_scale": vs}
    s["layers"] = [(k[i], v[i], ks[i], vs[i]) for i in range(L)]
    s["block_size"] = bs


def _new_workspace(s, N):
    if own:
        import speculative_decoding_verification_80_gb300 as sd

        s["workspace"] = sd.new_page_workspace(N, device=DEV)
        s["handle"] = sd.kv_layers(s["layers"])


def _fork_shape(case):
    """Lengths of the old requests, their blocks' number without shared ones, and the new requests' number."""
    P, n, kept, bs = case["P"], case["n"], case["kept"], case["bs"]
    if case["beams"]:
        # beams of one group share the prompt's full blocks
        lens = [L for L in _spread(max(1, kept // 2), kept, P) for _ in range(n)]
        shared = [(L // 2) // bs for L in lens]
        used = sum((L + bs - 1) // bs - (c if i % n else 0) for i, (L, c) in enumerate(zip(lens, shared)))
        return lens, shared, used, P * n
    lens = _spread(max(1, kept // 2), kept, P)
    return lens, [0] * P, sum((L + bs - 1) // bs for L in lens), P * n


def _prepare_fork(case, seed, s):
    rng = np.random.default_rng(seed)
    n, bs = case["n"], case["bs"]
    lens, shared, used, B = _fork_shape(case)
    P = len(lens)
    N = used + 2 * B + 3
    W = (case["kept"] + 8 * bs) // bs
    ids, at = rng.permutation(N), 0
    table, held, shares = np.full((P, W), -1), np.zeros(P, dtype=np.int64), np.zeros(N, dtype=np.int64)
    for p in range(P):
        need, c = (lens[p] + bs - 1) // bs, shared[p] if case["beams"] and p % n else 0
        held[p] = need
        if c:
            table[p, :c] = table[p - p % n, :c]
            shares[table[p, :c]] += 1
        table[p, c:need] = ids[at:at + need - c]
        at += need - c
    head = int(rng.integers(0, N))
    ring = np.full(N, -1)
    ring[(head + np.arange(N - at)) % N] = ids[at:]
    accepted = np.minimum(rng.integers(-1, 8, P), np.asarray(lens) - 1)
    if case["beams"]:
        parent = np.arange(B) // n * n + rng.integers(0, n, B)
        parent[rng.random(B) < 0.05] = -1
    else:
        parent = np.arange(B) // n
    keep = None
    if case["back"]:
        keep = np.asarray(lens)[np.maximum(parent, 0)]
        keep = np.where(rng.random(B) < case["back"], keep - rng.integers(0, 3 * bs, B), keep).clip(min=0)
    for name, v in (("block_table", table), ("held", held), ("shares", shares), ("free_ring", ring), ("ring_state", [head, N - at]),
                    ("kv_len", np.asarray(lens) - accepted - 1), ("accepted_len", accepted), ("parent", parent)):
        s[name] = _i32(v)
    s["keep"] = None if keep is None else _i32(keep)
    _caches(s, case, N, _gen(seed))
    _new_workspace(s, N)


def _compact_shape(case):
    lens = _spread(max(1, case["kept"] // 4), case["kept"], case["B"])
    used = sum((L + case["bs"] - 1) // case["bs"] for L in lens)
    return lens, used, max(used, int(used / case["used"]))


def _prepare_compact(case, seed, s):
    rng = np.random.default_rng(seed)
    bs, B = case["bs"], case["B"]
    lens, used, N = _compact_shape(case)
    W = (case["kept"] + 8 * bs) // bs
    ids, at = rng.permutation(N), 0
    table, held, shares = np.full((B, W), -1), np.zeros(B, dtype=np.int64), np.zeros(N, dtype=np.int64)
    for b in range(B):
        need = (lens[b] + bs - 1) // bs
        # every eighth request goes on from the one before it
        c = min(need, held[b - 1]) // 2 if b % 8 == 7 else 0
        held[b] = need
        if c:
            table[b, :c] = table[b - 1, :c]
            shares[table[b, :c]] += 1
        table[b, c:need] = ids[at:at + need - c]
        at += need - c
    head = int(rng.integers(0, N))
    ring = np.full(N, -1)
    ring[(head + np.arange(N - at)) % N] = ids[at:]
    for name, v in (("block_table", table), ("held", held), ("shares", shares), ("free_ring", ring), ("ring_state", [head, N - at])):
        s[name] = _i32(v)
    _caches(s, case, N, _gen(seed))
    _new_workspace(s, N)


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if own:
        import speculative_decoding_verification_80_gb300 as sd

        if op == "sample":
            tokens = sd.spec_sample(s["logits"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                                    uniform=s["uniform"], draft_len=s["draft_len"], out=s["out"], tokens=s["tokens"])
            return {k: v for k, v in (("tokens", tokens), ("out", s["out"])) if v is not None}
        if op == "rotary":
            sd.spec_rotary(s["q"], s["k"], s["positions"], s["turns"], layout=s["layout"], factor=s["factor"], q_out=s["q_out"], k_out=s["k_out"])
            return [s["q_out"], s["k_out"]]
        if op == "fork":
            f = sd.kv_fork(s["block_table"], s["kv_len"], s["held"], s["parent"], s["shares"], s["free_ring"], s["ring_state"], s["block_size"],
                           accepted_len=s["accepted_len"], keep=s["keep"], workspace=s["workspace"])
            sd.kv_copy(f.copies, f.count, s["handle"])
            return {"table": f.block_table, "held": f.held, "kv_len": f.kv_len, "shares": f.shares, "ring": s["free_ring"],
                    "ring_state": f.ring_state, "count": f.count, "caches": s["caches"]}
        c = sd.kv_compact(s["block_table"], s["held"], s["shares"], s["free_ring"], s["ring_state"], workspace=s["workspace"])
        sd.kv_copy(c.copies, c.count, s["handle"])
        return {"table": c.block_table, "shares": c.shares, "ring_state": c.ring_state, "renamed": c.renamed, "count": c.count, "caches": s["caches"]}
    return {"sample": _plain_sample, "rotary": _plain_rotary, "fork": _plain_fork, "compact": _plain_compact}[op](s)


def _plain_sample(s):
    B, rows, V = s["logits"].shape
    step = max(1, (1 << 26) // (rows * V))
    for b in range(0, B, step):
        _plain_sample_part(s, slice(b, min(B, b + step)))
    return {k: s[k] for k in ("tokens", "out") if s[k] is not None}


def _plain_sample_part(s, part):
    x = s["logits"][part]
    B, rows, V = x.shape
    per = lambda name: s[name][part].double()[:, None, None]  # noqa: E731
    there = torch.arange(rows, device=DEV)[None] <= s["draft_len"][part][:, None]
    # sums and their borders in 64 bits
    vals, ids = torch.sort(x.float(), dim=2, descending=True, stable=True)
    T = per("temperature")
    w = torch.exp((vals.double() - vals[..., :1].double()) / torch.where(T > 0, T, 1.0))
    rank = torch.arange(V, device=DEV)
    k = s["top_k"][part].long()[:, None, None]
    k = torch.where(T > 0, torch.where(k > 0, k, V), 1)
    w = torch.where(rank < k, w, 0.0)
    run_sum = torch.cumsum(w, 2)
    before = torch.nn.functional.pad(run_sum, (1, 0))[..., :-1]
    p = per("top_p")
    kept = (rank < k) & ((before < p * run_sum[..., -1:]) | (p >= 1.0)) & (w >= per("min_p")) & (vals > -math.inf)
    del before
    if s["tokens"] is not None:
        run_sum = torch.cumsum(torch.where(kept, w, 0.0), 2)
        at = (run_sum > s["uniform"][part].double()[..., None] * run_sum[..., -1:]).to(torch.int8).argmax(2, keepdim=True)
        s["tokens"][part] = torch.where(there, ids.gather(2, at)[..., 0], -1).to(torch.int32)
    del run_sum, w
    if s["out"] is not None:
        may = torch.zeros(B, rows, V, dtype=torch.bool, device=DEV).scatter(2, ids, kept)
        s["out"][part] = torch.where(there[..., None], torch.where(may, x, -math.inf), s["out"][part])


def _plain_rotary(s):
    R = 2 * s["freq"].numel()
    p = s["positions"]
    angle = p.double()[:, None] * s["freq"]
    cos, sin = ((s["factor"] * f(angle)).float()[:, None] for f in (torch.cos, torch.sin))
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = x.float()
        if s["layout"] == "half":
            a, b = y[..., :R // 2], y[..., R // 2:R]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], 2)
        else:
            a, b = y[..., :R:2], y[..., 1:R:2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], 3).flatten(2)
        y = torch.cat([turned, y[..., R:]], 2).to(x.dtype)
        out.copy_(torch.where((p >= 0)[:, None, None], y, out))
    return [s["q_out"], s["k_out"]]


def _plain_copy(s, src, dst, live):
    """cache[dst] = cache[src] for the pairs that live; the others repeat the first (a block onto itself without any)."""
    src, dst = (torch.where(live, v, torch.where(live[:1], v[:1], 0)) for v in (src, dst))
    for layer in s["layers"]:
        for x in layer:
            x = x.view(torch.uint8) if x.dtype == E4M3 else x
            x[dst] = x[src]


def _count(N, ids, live):
    """How often each of N ids is there."""
    return torch.zeros(N + 1, dtype=torch.int64, device=DEV).scatter_add(0, torch.where(live, ids, N).reshape(-1), torch.ones_like(ids).reshape(-1))[:N]


def _plain_fork(s):
    bs, table, ring = s["block_size"], s["block_table"].long(), s["free_ring"]
    P, W = table.shape
    N = ring.numel()
    parent = s["parent"].long()
    B = parent.numel()
    p = parent.clamp(min=0)
    tokens = (s["kv_len"].long() + s["accepted_len"].long() + 1)[p]
    if s["keep"] is not None:
        tokens = torch.minimum(tokens, s["keep"].long())
    tokens = torch.where(parent < 0, 0, tokens)
    need, full = (tokens + bs - 1) // bs, tokens // bs
    j = torch.arange(W, device=DEV)[None]
    rows = table[p]
    old, new = _count(N, table, j < s["held"].long()[:, None]), _count(N, rows, j < need[:, None])
    holders = s["shares"].long() + 1 - old + new
    part = need > full
    last = rows.gather(1, full.clamp(max=W - 1)[:, None])[:, 0]
    at = torch.where(part, last, N)
    parts = _count(N, last, part)
    b = torch.arange(B, device=DEV)
    latest = torch.full((N + 1,), -1, dtype=torch.int64, device=DEV).scatter_reduce(0, at, b, "amax")[:N]
    # all but the last of those that write a block take one of their own, unless another holds it whole
    safe = last.clamp(min=0)
    ask = part & ~((parts[safe] == holders[safe]) & (latest[safe] == b))
    number = torch.cumsum(ask.long(), 0) - ask.long()
    head, free = s["ring_state"].long()[0], s["ring_state"].long()[1]
    got = ask & (number < free)
    refused = ask & ~got
    fresh = ring.long()[(head + number) % N]
    held = torch.where(refused, full, need)
    rows = torch.where((j == full[:, None]) & got[:, None], fresh[:, None], rows)
    after = torch.where(parts == holders, holders.clamp(max=1), holders - parts)
    seen = old > 0
    gone = seen & (holders <= 0)
    place = torch.cumsum(gone.long(), 0) - 1
    padded = torch.cat([ring, ring.new_zeros(1)]).scatter(0, torch.where(gone, (head + free + place) % N, N), torch.arange(N, device=DEV).to(torch.int32))
    ring.copy_(padded[:N])
    taken = got.sum()
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    _plain_copy(s, *(torch.full((B + 1,), -1, dtype=torch.int64, device=DEV).scatter(0, torch.where(got, number, B), v)[:B] for v in (last, fresh)),
                torch.arange(B, device=DEV) < taken)
    return {"table": i32(torch.where(j < held[:, None], rows, -1)), "held": i32(held), "kv_len": i32(torch.where(refused, full * bs, tokens)),
            "shares": i32(torch.where(seen, (after - 1).clamp(min=0), s["shares"].long())), "ring": ring,
            "ring_state": i32(torch.stack([(head + taken) % N, free - taken + gone.sum()])), "count": i32(taken).view(1), "caches": s["caches"]}


def _plain_compact(s):
    table, ring, shares = s["block_table"].long(), s["free_ring"].long(), s["shares"].long()
    N = ring.numel()
    head, free = s["ring_state"].long()[0], s["ring_state"].long()[1]
    i = torch.arange(N, device=DEV)
    is_free = torch.zeros(N + 1, dtype=torch.bool, device=DEV).scatter(0, torch.where(i < free, ring[(head + i) % N], N), True)[:N]
    n = N - free
    hole, moves = is_free & (i < n), ~is_free & (i >= n)
    count = moves.sum()
    to = torch.full((N + 1,), -1, dtype=torch.int64, device=DEV).scatter(0, torch.where(hole, torch.cumsum(hole.long(), 0) - 1, N), i)[:N]
    src = torch.full((N + 1,), -1, dtype=torch.int64, device=DEV).scatter(0, torch.where(moves, torch.cumsum(moves.long(), 0) - 1, N), i)[:N]
    renamed = torch.where(moves, to[(torch.cumsum(moves.long(), 0) - 1).clamp(min=0)], torch.where(is_free, -1, i))
    j = torch.arange(table.shape[1], device=DEV)[None]
    fresh = torch.where(j < s["held"].long()[:, None], renamed[table.clamp(min=0)], -1)
    shares_out = torch.zeros(N + 1, dtype=torch.int64, device=DEV).scatter(0, torch.where(renamed >= 0, renamed, N), shares)[:N]
    live = i[:N // 2 + 1] < count
    _plain_copy(s, src[:N // 2 + 1], to[:N // 2 + 1], live)
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"table": i32(fresh), "shares": i32(shares_out), "ring_state": i32(torch.stack([torch.zeros_like(free), free])),
            "renamed": i32(renamed), "count": i32(count).view(1), "caches": s["caches"]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "sample":
        elt = 2 if case["dtype"] == "bf16" else 4
        rows = case["B"] * (1 + ((case["n"] + 1) // 2 + case["n"]) / 2)  # drafts are between half of n and n
        return {"bytes": rows * (case["V"] * elt * (2 if case["rows"] else 1) + (8.0 if case["draw"] else 0.0)) + 16.0 * case["B"], "flops": 0.0}
    if op == "rotary":
        elt = 2 if case["dtype"] == "bf16" else 4
        values = case["T"] * (case["Hq"] + case["H"])
        return {"bytes": values * case["D"] * 2.0 * elt + 4.0 * case["T"], "flops": 3.0 * values * case["part"]}
    bs, layers = case["bs"], case["layers"]
    block = layers * (2.0 * case["H"] * bs * case["D"] + 8.0 * case["H"])
    if op == "fork":
        lens, _, _, B = _fork_shape(case)
        # the tables in and out; every new request but the last of a parent's copies its part-filled block
        n = case["n"]
        mean = sum((L + bs - 1) // bs for L in lens) / len(lens)
        copies = B * (1.0 - (1.0 - (1.0 - 1.0 / n) ** n if case["beams"] else 1.0 / n)) * (1.0 - 1.0 / bs)
        return {"bytes": 4.0 * mean * (len(lens) + 2 * B) + 2.0 * block * copies, "flops": 0.0}
    lens, used, N = _compact_shape(case)
    moves = used / N * (N - used)
    return {"bytes": 8.0 * used + 12.0 * N + 2.0 * block * moves, "flops": 0.0}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "fork":
        return _exact_moves(s, _exact_fork(s), ("table", "held", "kv_len", "shares", "ring", "ring_state", "count"))
    if op == "compact":
        return _exact_moves(s, _exact_compact(s), ("table", "shares", "ring_state", "renamed", "count"))
    if op == "rotary":
        return _exact_rotary(case, s)
    if s["out"] is None:
        return None
    out = {"out": _exact_rows(s)}
    return {"tokens": None, **out} if case["draw"] else out


def _exact_rotary(case, s):
    R, D = case["part"], case["D"]
    f, factor = _frequencies(R, 10000.0, _scaling(case))
    pair = torch.arange(R, device=DEV)
    first = (pair < R // 2) if case["layout"] == "half" else (pair % 2 == 0)
    which = pair % (R // 2) if case["layout"] == "half" else pair // 2
    other = torch.where(first, pair + (R // 2 if case["layout"] == "half" else 1), pair - (R // 2 if case["layout"] == "half" else 1))
    turn = torch.as_tensor(f).to(DEV)[which]
    results = []
    for x, before in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        out = before.double()
        for t0 in range(0, case["T"], 4096):
            y = x[t0:t0 + 4096].double()
            p = s["positions"][t0:t0 + 4096].double()
            a = (p[:, None] * turn)[:, None]
            y[..., :R] = factor * (y[..., :R] * torch.cos(a) + torch.where(first, -1.0, 1.0) * y[..., other] * torch.sin(a))
            out[t0:t0 + 4096] = torch.where((p >= 0)[:, None, None], y, out[t0:t0 + 4096])
        results.append(out)
    return results


def _exact_rows(s):
    """Row by row: what may be drawn, by going through the ids in order."""
    B, rows, V = s["logits"].shape
    out = s["out"].double()
    K, P, M, T, N = (s[k].tolist() for k in ("top_k", "top_p", "min_p", "temperature", "draft_len"))
    for b in range(B):
        for j in range(N[b] + 1):
            l = s["logits"][b, j].double()
            if T[b] == 0.0:
                top = torch.arange(V, device=DEV) == (l == l.max()).to(torch.int8).argmax()
                out[b, j] = torch.where(top, l, -math.inf)
                continue
            order = torch.argsort(l, descending=True, stable=True)
            if 0 < K[b] < V:
                order = order[:K[b]]
            share = torch.softmax(l[order] / T[b], 0)
            if P[b] < 1.0:
                enough = torch.cumsum(share, 0) >= P[b]
                share = share[:int(enough.to(torch.int8).argmax()) + 1 if bool(enough[-1]) else V]
            order = order[:share.numel()][share >= M[b] * share[0]]
            row = torch.full_like(l, -math.inf)
            row[order] = l[order]
            out[b, j] = row
    return out


def _exact_moves(s, pairs, whole):
    """What the caches hold after the copies, one by one; the whole numbers have no such value."""
    out = {name: x.double() for name, x in s["caches"].items()}
    for src, dst in pairs:
        for x in out.values():
            x[:, dst] = x[:, src]
    return {**{name: None for name in whole}, "caches": out}


def _exact_fork(s):
    """The copies (from, to), request by request."""
    bs, table, held = s["block_size"], s["block_table"].tolist(), s["held"].tolist()
    kv, acc, keep = s["kv_len"].tolist(), s["accepted_len"].tolist(), None if s["keep"] is None else s["keep"].tolist()
    ring, (head, free) = s["free_ring"].tolist(), s["ring_state"].tolist()
    holders = [n + 1 for n in s["shares"].tolist()]
    for row, h in zip(table, held):
        for x in row[:h]:
            holders[x] -= 1
    writers = []
    for b, p in enumerate(s["parent"].tolist()):
        if p < 0:
            continue
        n = kv[p] + acc[p] + 1 if keep is None else min(keep[b], kv[p] + acc[p] + 1)
        for x in table[p][:-(-n // bs)]:
            holders[x] += 1
        if n % bs:
            writers.append(table[p][n // bs])
    pairs = []
    for x in writers:
        if holders[x] > 1:
            holders[x] -= 1
            if len(pairs) < free:
                pairs.append((x, ring[(head + len(pairs)) % len(ring)]))
    return pairs


def _exact_compact(s):
    ring, (head, free) = s["free_ring"].tolist(), s["ring_state"].tolist()
    N = len(ring)
    empty = {ring[(head + i) % N] for i in range(free)}
    return list(zip((i for i in range(N - free, N) if i not in empty), sorted(i for i in empty if i < N - free)))
