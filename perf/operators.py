"""The operators of a decode step around the verify: what is measured, with a plain form of each.

Four operators, a case's ``"op"`` names the one it calls:

* ``logits``: penalties, biases and grammar masks on the rows that ``spec_verify`` reads;
* ``blocks``: block tables and slot maps from request lengths;
* ``append``: keys and values of new tokens into the cache held in 8 bits;
* ``attention``: attention of the new tokens over that cache.

``own`` selects the framework's calls; otherwise ``run`` is the plain form.
"""
import math

import torch

own = False

DEV = "cuda"
WORKSPACE_BYTES = 64 << 20  # scratch that a serving program allocates once, zero-filled
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one draft step of a single user: the penalties of a short conversation, no grammar
        dict(name="logits_draft_one", op="logits", B=1, n=0, V=128256, dtype="bf16", S=640, bias=0, masked=0.0),
        # verify rows of the draft-target batch, biases on every request, a grammar on half of them
        dict(name="logits_verify_64", op="logits", B=64, n=4, V=128256, dtype="bf16", S=2048, bias=24, masked=0.5),
        # ragged verify batch with long histories, few grammars
        dict(name="logits_ragged_256", op="logits", B=256, n=7, V=152064, dtype="bf16", S=8192, bias=5, masked=0.1),
        # one decode step of the ragged batch: a few tokens each, a few blocks change hands
        dict(name="blocks_decode_1024", op="blocks", B=1024, new=8, kept=4096, bs=16),
        # admission of long prompts: every block is new
        dict(name="blocks_prompts_512", op="blocks", B=512, new=2000, kept=0, bs=16),
        # one user, one token, the small draft model's heads
        dict(name="append_one", op="append", B=1, new=1, kept=900, H=8, D=64, bs=16, dtype="bf16"),
        # MTP verify: two tokens for each of 256 requests, fp32 keys from a rotary step in fp32
        dict(name="append_mtp_256", op="append", B=256, new=2, kept=2048, H=8, D=128, bs=32, dtype="f32"),
        # prompts of some thousand tokens each
        dict(name="append_prompts", op="append", B=16, new=5000, kept=40, H=8, D=128, bs=64, dtype="bf16"),
        # one user's draft step over a short context, the small draft model's heads
        dict(name="attention_draft_one", op="attention", B=1, new=1, kept=700, Hq=32, H=8, D=64, bs=16),
        # verify rows of the draft-target batch
        dict(name="attention_verify_64", op="attention", B=64, new=5, kept=8000, Hq=64, H=8, D=128, bs=32),
        # one user with a very long context, two query tokens
        dict(name="attention_long_one", op="attention", B=1, new=2, kept=131000, Hq=64, H=8, D=128, bs=64),
        # ragged verify batch, up to eight query tokens each, small blocks
        dict(name="attention_ragged_256", op="attention", B=256, new=8, kept=4000, Hq=32, H=8, D=128, bs=16),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logits", "blocks", "append", "attention", "attention"])
    if op == "logits":
        n = rng.randint(0, 7)
        V = rng.choice([1024, 32003, 50001, 128256, 129280, 152064])
        B = _log(rng, 1, max(1, min(256, int(3.0e8 / ((n + 1) * V)))))
        return dict(op=op, B=B, n=n, V=V, dtype=rng.choice(["bf16", "bf16", "f32"]), S=_log(rng, 1, 8192),
                    bias=rng.choice([0, 3, 24, 200]), masked=rng.choice([0.0, 0.1, 0.5, 1.0]))
    if op == "blocks":
        B = _log(rng, 1, 1024)
        new = _log(rng, 1, min(2000, 1000000 // B))
        return dict(op=op, B=B, new=new, kept=rng.choice([0, _log(rng, 1, 4096)]), bs=rng.choice([16, 32, 64, 128]))
    if op == "append":
        B = _log(rng, 1, 256)
        H, D = rng.choice([(8, 64), (8, 128), (1, 128), (4, 128)])
        return dict(op=op, B=B, new=_log(rng, 1, min(5000, 80000 // B)), kept=rng.choice([0, _log(rng, 1, 2048)]), H=H, D=D,
                    bs=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "f32"]))
    Hq, H, D = rng.choice([(32, 8, 64), (64, 8, 128), (32, 8, 128), (8, 8, 128), (12, 2, 128), (8, 1, 64)])
    kept = _log(rng, 1, 131000)
    B = _log(rng, 1, max(1, min(256, 500000 // (kept + 8))))
    return dict(op=op, B=B, new=_log(rng, 1, 8), kept=kept, Hq=Hq, H=H, D=D, bs=rng.choice([16, 32, 64, 128]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randint(lo, hi, shape, g):
    """int32 in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV).to(torch.int32)


def _spread(lo, hi, B):
    """B whole numbers from hi down to lo: the lengths that a case's requests have in some order."""
    return [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]


def _kept_of(case):
    return _spread(case["kept"] // 8, case["kept"], case["B"])


def _new_of(case):
    return _spread(max(1, case["new"] // 4), case["new"], case["B"])


def _lengths(case, g):
    """Tokens kept in the cache and new tokens of each request, in an order of their own."""
    kept, new = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (_kept_of(case), _new_of(case)))
    return tuple(v[torch.randperm(case["B"], generator=g, device=DEV)] for v in (kept, new))


def _blocks_of(case, extra=0):
    """Blocks that hold the case's tokens, however the lengths fall: a part-filled one for each request."""
    return (sum(_kept_of(case)) + sum(_new_of(case)) + extra * case["B"]) // case["bs"] + case["B"]


def _prefix(x):
    """[0, x_0, x_0 + x_1, ...] in int32."""
    return torch.cat([torch.zeros(1, dtype=torch.int64, device=x.device), torch.cumsum(x.long(), 0)]).to(torch.int32)


def _paged(lengths, bs, width, blocks, g):
    """A block table [B, width] over shuffled blocks of `blocks` that holds `lengths` tokens each."""
    held = (lengths.long() + bs - 1) // bs
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    j = torch.arange(width, device=DEV)[None]
    at = _prefix(held).long()[:-1, None] + j
    return torch.where(j < held[:, None], perm[at.clamp(max=blocks - 1)], -1).to(torch.int32).contiguous(), perm


def _slots(table, kept, new, bs):
    """Slot of each new token, packed by request."""
    cu = _prefix(new).long()
    t = torch.arange(int(cu[-1]), device=DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    p = kept.long()[b] + t - cu[b]
    return (table.long()[b, p // bs] * bs + p % bs).to(torch.int32)


def _filled_cache(blocks, H, bs, D, g):
    """Codes and scales of a cache whose blocks hold unit normal rows, some heads louder than others."""
    x = torch.randn(blocks, H, bs, D, generator=g, device=DEV) * (0.5 + torch.arange(H, device=DEV).view(1, H, 1, 1) / H)
    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / 448.0)))
    return (x / scale[:, :, None, None]).to(E4M3), scale


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op}
    if op == "logits":
        B, n, V, S = case["B"], case["n"], case["V"], case["S"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["logits"] = torch.empty(B, n + 1, V, dtype=dt, device=DEV).normal_(0.0, 3.0, generator=g)
        s["out"] = torch.zeros(B, n + 1, V, dtype=dt, device=DEV)
        # token ids repeat as text does: squares of uniform numbers, so low ids come often
        ids = lambda *shape: (torch.rand(*shape, generator=g, device=DEV).square() * V).to(torch.int32).clamp(max=V - 1)  # noqa: E731
        s["history"] = ids(B, S)
        s["history_len"] = _randint(S // 2, S, (B,), g)
        s["prompt_len"] = (s["history_len"].float() * torch.rand(B, generator=g, device=DEV)).to(torch.int32)
        s["draft_tokens"] = ids(B, n)
        s["draft_len"] = _randint((n + 1) // 2, n, (B,), g)
        s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device=DEV)
        s["presence"] = torch.rand(B, generator=g, device=DEV)
        s["frequency"] = 0.2 * torch.rand(B, generator=g, device=DEV)
        count = _randint(case["bias"] // 2, case["bias"], (B,), g)
        s["bias_offsets"] = _prefix(count)
        s["bias_ids"] = ids(max(1, B * case["bias"]))
        s["bias_values"] = torch.randn(max(1, B * case["bias"]), generator=g, device=DEV) * 5.0
        # grammars: a handful of states allow few tokens, others most of them
        masks = 64
        words = (V + 31) // 32
        few = torch.rand(masks, 1, generator=g, device=DEV) < 0.5
        m = _randint(-2**31, 2**31 - 1, (masks, words), g)
        s["mask"] = torch.where(few, m & _randint(-2**31, 2**31 - 1, (masks, words), g) & _randint(-2**31, 2**31 - 1, (masks, words), g), m)
        s["mask_rows"] = torch.where(torch.rand(B, 1, generator=g, device=DEV) < case["masked"], _randint(0, masks - 1, (B, n + 1), g), -1).to(torch.int32)
        return s
    bs = case["bs"]
    kept, new = _lengths(case, g)
    if op == "blocks":
        # the last step appended up to eight tokens, of which the accepted ones and one more stay
        B = case["B"]
        accepted = torch.minimum(_randint(-1, 7, (B,), g), kept - 1).to(torch.int32)
        s["kv_len"] = (kept - accepted - 1).to(torch.int32)
        s["accepted_len"] = accepted
        s["new_tokens"] = torch.where(torch.rand(B, generator=g, device=DEV) < 0.02, -1, new).to(torch.int32)
        appended = torch.maximum(kept, s["kv_len"] + 8 * (kept > 0))
        s["held"] = ((appended.long() + bs - 1) // bs).to(torch.int32)
        width = (case["kept"] + 8 + case["new"] + bs - 1) // bs
        used, blocks = s["held"].long().sum(), 2 * _blocks_of(case, 8) + B
        s["block_table"], perm = _paged(appended, bs, width, blocks, g)
        # the free blocks are what the tables do not name, and wrap around the ring's end
        head = blocks - blocks // 5
        i = torch.arange(blocks, device=DEV)
        s["free_ring"] = torch.where(i < blocks - used, perm[(used + i) % blocks], -1).to(torch.int32).roll(head)
        s["ring_state"] = torch.stack([torch.full_like(used, head), blocks - used]).to(torch.int32)
        s["block_size"] = bs
        s["capacity"] = sum(_new_of(case))
        return s
    H, D = case["H"], case["D"]
    blocks, T = _blocks_of(case), sum(_new_of(case))
    table, _ = _paged(kept + new, bs, (case["kept"] + case["new"] + bs - 1) // bs, blocks, g)
    s["k_cache"], s["k_scale"] = _filled_cache(blocks, H, bs, D, g)
    s["v_cache"], s["v_scale"] = _filled_cache(blocks, H, bs, D, g)
    if op == "append":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        qkv = torch.randn(T, 3 * H, D, generator=g, device=DEV).to(dt)  # a fused projection's rows
        s["k"], s["v"] = qkv[:, H:2 * H], qkv[:, 2 * H:]
        s["slot_map"] = _slots(table, kept, new, bs)
        return s
    s["kv_len"], s["block_table"] = kept, table
    s["cu_tokens"] = _prefix(new)
    s["q"] = (2.0 * torch.randn(T, case["Hq"], D, generator=g, device=DEV)).to(torch.bfloat16)
    s["out"] = torch.zeros(T, case["Hq"], D, dtype=torch.bfloat16, device=DEV)
    s["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)
    s["most_new"], s["most_kv"] = case["new"], case["kept"] + case["new"]
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if own:
        import speculative_decoding_verification_80_gb300 as sd

        if op == "logits":
            return sd.spec_process_logits(s["logits"], s["history"], s["prompt_len"], s["history_len"], draft_tokens=s["draft_tokens"],
                                          draft_len=s["draft_len"], repetition=s["repetition"], presence=s["presence"],
                                          frequency=s["frequency"], bias_offsets=s["bias_offsets"], bias_ids=s["bias_ids"],
                                          bias_values=s["bias_values"], mask=s["mask"], mask_rows=s["mask_rows"], out=s["out"])
        if op == "blocks":
            step = sd.kv_block_step(s["block_table"], s["kv_len"], s["held"], s["new_tokens"], s["free_ring"], s["ring_state"],
                                    s["block_size"], s["capacity"], accepted_len=s["accepted_len"])
            return {"table": s["block_table"], "ring": s["free_ring"], "kv_len": step.kv_len, "held": step.held, "ring_state": step.ring_state,
                    "cu_tokens": step.cu_tokens, "slot_map": step.slot_map, "positions": step.positions}
        if op == "append":
            sd.kv_append(s["k"], s["v"], s["slot_map"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
            return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]
        return sd.spec_attention(s["q"], s["cu_tokens"], s["kv_len"], s["block_table"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                 out=s["out"], workspace=s["workspace"])
    return {"logits": _plain_logits, "blocks": _plain_blocks, "append": _plain_append, "attention": _plain_attention}[op](s)


def _plain_logits(s):
    x = s["logits"]
    B, rows, V = x.shape
    S = s["history"].shape[1]
    at = torch.arange(S, device=DEV)[None]
    zeros = torch.zeros(B, V, device=DEV)
    hist = s["history"].long()
    prompt = zeros.scatter_add(1, hist, (at < s["prompt_len"][:, None]).float()) > 0
    made = ((at >= s["prompt_len"][:, None]) & (at < s["history_len"][:, None])).float()
    count = zeros.scatter_add(1, hist, made)[:, None].repeat(1, rows, 1)
    # row j counts the drafts before it
    drafts = torch.zeros(B, rows, V, device=DEV)
    n = rows - 1
    if n:
        one = (torch.arange(n, device=DEV)[None] < s["draft_len"][:, None]).float()
        drafts[:, 1:].scatter_add_(2, s["draft_tokens"].long()[:, :, None], one[:, :, None])
        count = count + torch.cumsum(drafts, 1)
    per = lambda v: v[:, None, None]  # noqa: E731
    y = x.float()
    seen = prompt[:, None] | (count > 0)
    y = torch.where(seen, torch.where(y > 0, y / per(s["repetition"]), y * per(s["repetition"])), y)
    y = y - per(s["frequency"]) * count
    y = torch.where(count > 0, y - per(s["presence"]), y)
    k = torch.arange(s["bias_ids"].numel(), device=DEV)
    owner = (torch.searchsorted(s["bias_offsets"].long(), k, right=True) - 1).clamp(max=B - 1)
    inside = k < s["bias_offsets"][-1]
    bias = zeros.view(-1).scatter_add(0, owner * V + s["bias_ids"].long(), s["bias_values"] * inside).view(B, V)
    y = y + bias[:, None]
    words = s["mask"][s["mask_rows"].long().clamp(min=0)]  # [B, rows, words]
    v = torch.arange(V, device=DEV)
    allowed = (words[:, :, v // 32] >> (v % 32).to(torch.int32)) & 1
    y = torch.where((allowed == 0) & (s["mask_rows"] >= 0)[:, :, None], -math.inf, y)
    there = (torch.arange(rows, device=DEV)[None] <= s["draft_len"][:, None])[:, :, None]
    s["out"].copy_(torch.where(there, y.to(x.dtype), s["out"]))
    return s["out"]


def _plain_blocks(s):
    bs, table, ring = s["block_size"], s["block_table"], s["free_ring"]
    B, width = table.shape
    N = ring.numel()
    new, held = s["new_tokens"].long(), s["held"].long()
    kept = torch.where(new < 0, 0, s["kv_len"].long() + s["accepted_len"].long() + 1)
    want = new.clamp(min=0)
    need = (kept + want + bs - 1) // bs
    grow = torch.where(need <= width, (need - held).clamp(min=0), 0)
    head, free = s["ring_state"].long()[0], s["ring_state"].long()[1]
    granted = (need <= width) & ((grow == 0) | (torch.cumsum(grow, 0) <= free))
    taken = torch.where(granted, grow, 0)
    given = torch.where(granted, (held - need).clamp(min=0), 0)
    held_out = held + taken - given
    before = torch.cumsum(taken, 0) - taken
    j = torch.arange(width, device=DEV)[None]
    fresh = (j >= held[:, None]) & (j < held_out[:, None])
    gone = (j >= held_out[:, None]) & (j < held[:, None])
    from_ring = ring.long()[(head + before[:, None] + j - held[:, None]) % N]
    back = torch.cumsum(given, 0) - given
    to_ring = (head + free + back[:, None] + j - held_out[:, None]) % N
    padded = torch.cat([ring, ring.new_zeros(1)]).scatter(0, torch.where(gone, to_ring, N).view(-1), table.view(-1))
    ring.copy_(padded[:N])
    table.copy_(torch.where(fresh, from_ring, table.long()).to(torch.int32))
    tokens = torch.where(granted, want, 0)
    cu = _prefix(tokens)
    t = torch.arange(s["capacity"], device=DEV)
    b = (torch.searchsorted(cu.long(), t, right=True) - 1).clamp(max=B - 1)
    p = kept[b] + t - cu.long()[b]
    live = t < cu[-1]
    block = table.long()[b, torch.where(live, p // bs, 0)]
    return {"table": table, "ring": ring, "kv_len": kept.to(torch.int32), "held": held_out.to(torch.int32),
            "ring_state": torch.stack([(head + taken.sum()) % N, free - taken.sum() + given.sum()]).to(torch.int32),
            "cu_tokens": cu, "slot_map": torch.where(live, block * bs + p % bs, -1).to(torch.int32),
            "positions": torch.where(live, p, -1).to(torch.int32)}


def _pow2_scale(amax):
    """The least power of two that brings `amax` within the type's 448; 0 of 0."""
    f, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), torch.where(f <= 0.875, e - 9, e - 8)), 0.0)


def _plain_append_one(x, slot, cache, scale):
    blocks, H, bs, D = cache.shape
    x = x.float()
    block, off = slot.long() // bs, slot.long() % bs
    # the first new offset of each block, and the largest new magnitude of each block and head
    first = torch.full((blocks,), bs, dtype=torch.int64, device=DEV).scatter_reduce(0, block, off, "amin")
    amax = torch.zeros(blocks, H, device=DEV).scatter_reduce(0, block[:, None].expand(-1, H), x.abs().amax(2), "amax")
    fresh = _pow2_scale(amax)
    now = torch.where((first == bs)[:, None], scale, torch.where((first == 0)[:, None], fresh, torch.maximum(scale, fresh)))
    older = torch.arange(bs, device=DEV)[None] < first[:, None]
    change = (older & (first < bs)[:, None])[:, None] & (now > scale)[:, :, None]
    ratio = torch.where(now > 0, scale / now, 1.0)
    values = cache.float()
    values = torch.where(change[..., None], (values * ratio[:, :, None, None]).to(E4M3).float(), values)
    own_scale = now[block]
    codes = torch.where(own_scale[..., None] > 0, x / own_scale[..., None], 0.0).clamp(-448.0, 448.0).to(E4M3).float()
    flat = values.permute(0, 2, 1, 3).reshape(blocks * bs, H, D).index_copy(0, slot.long(), codes)
    cache.copy_(flat.view(blocks, bs, H, D).permute(0, 2, 1, 3).to(E4M3))
    scale.copy_(now)


def _plain_append(s):
    _plain_append_one(s["k"], s["slot_map"], s["k_cache"], s["k_scale"])
    _plain_append_one(s["v"], s["slot_map"], s["v_cache"], s["v_scale"])
    return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _rows(cache, scale, table, L):
    """The first L tokens of each request in 32 bits: [B, H, L, D]."""
    _, H, bs, D = cache.shape
    B = table.shape[0]
    blocks = table.long()[:, :(L + bs - 1) // bs].clamp(min=0)
    x = cache.view(torch.uint8)[blocks].view(E4M3).float() * scale[blocks][:, :, :, None, None]
    return x.transpose(1, 2).reshape(B, H, -1, D)[:, :, :L]


def _plain_attention(s):
    q, cu = s["q"], s["cu_tokens"].long()
    T, Hq, D = q.shape
    B, H, L, Q = cu.numel() - 1, s["k_cache"].shape[1], s["most_kv"], s["most_new"]
    G = Hq // H
    i = torch.arange(Q, device=DEV)[None]
    there = i < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(there, cu[:-1, None] + i, 0)
    x = q.float()[at].view(B, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
    k = _rows(s["k_cache"], s["k_scale"], s["block_table"], L)
    scores = torch.matmul(x, k.transpose(2, 3)).view(B, H, Q, G, L) * (1.0 / math.sqrt(D))
    del k
    t = torch.arange(L, device=DEV)
    seen = t[None, None] <= s["kv_len"].long()[:, None, None] + i[..., None]  # [B, Q, L]
    scores = scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    scores -= scores.amax(4, keepdim=True)
    p = scores.exp_()
    p /= p.sum(4, keepdim=True)
    v = _rows(s["v_cache"], s["v_scale"], s["block_table"], L)
    v = torch.where((t[None] < (s["kv_len"].long() + (cu[1:] - cu[:-1]))[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p.view(B, H, Q * G, L), v).view(B, H, Q, G, D).permute(0, 2, 1, 3, 4).reshape(B, Q, Hq, D)
    b = torch.searchsorted(cu, torch.arange(T, device=DEV), right=True) - 1
    s["out"].copy_(o[b, torch.arange(T, device=DEV) - cu[b]])
    return s["out"]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "logits":
        elt = 2 if case["dtype"] == "bf16" else 4
        rows = case["B"] * (1 + 0.75 * case["n"])  # drafts are between n/2 and n
        mask = case["masked"] * min(64, rows) * (case["V"] / 8)
        return {"bytes": rows * case["V"] * 2 * elt + case["B"] * (3 * case["S"] + 8 * case["bias"]) + mask, "flops": 0.0}
    B = case["B"]
    kept, new = _kept_of(case), _new_of(case)
    if op == "blocks":
        # new slots and positions, the table entries and ring places that are read or written, the requests' numbers
        return {"bytes": 8.0 * sum(new) + 8.0 * sum(new) / case["bs"] + 32.0 * B, "flops": 0.0}
    H, D = case["H"], case["D"]
    if op == "append":
        elt = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": sum(new) * (2.0 * H * D * (elt + 1) + 4.0 + 16.0 * H / case["bs"]), "flops": 0.0}
    Hq = case["Hq"]
    tokens = sum(kept) + sum(new)
    # a token attends to what is kept and, on average, half of the new ones; long and short meet in any order
    pairs = (sum(kept) + 0.5 * sum(new)) * sum(new) / B
    return {"bytes": 2.0 * tokens * H * (D + 4.0 / case["bs"]) + 4.0 * sum(new) * Hq * D, "flops": 4.0 * pairs * Hq * D}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "blocks":
        return None  # whole numbers
    if op == "append":
        out = []
        for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
            out.append(_exact_append(x.double(), s["slot_map"].long(), cache.double(), scale.double()))
        return [out[0][0], out[1][0], out[0][1], out[1][1]]
    if op == "logits":
        return _exact_logits(case, s)
    return _exact_attention(case, s)


def _exact_append(x, slot, cache, scale):
    blocks, H, bs, D = cache.shape
    block = slot // bs
    touched = torch.zeros(blocks, dtype=torch.bool, device=DEV)
    touched[block] = True
    is_new = torch.zeros(blocks * bs, dtype=torch.bool, device=DEV)
    is_new[slot] = True
    is_new = is_new.view(blocks, bs)
    # tokens before the first new one of their block stay
    stays = (torch.cumsum(is_new.long(), 1) == 0) & touched[:, None]
    rows = torch.zeros(blocks * bs, H, D, dtype=torch.float64, device=DEV)
    rows[slot] = x
    rows = rows.view(blocks, bs, H, D).transpose(1, 2)
    big = rows.abs().amax(dim=(2, 3))
    # the least power of two s with big <= 448 s
    s_new = torch.exp2(torch.ceil(torch.log2(big.clamp(min=1e-300) / 448.0)))
    s_new = torch.where(s_new * 448.0 < big, s_new * 2, s_new)
    s_new = torch.where(s_new * 224.0 >= big, s_new / 2, s_new)
    s_new = torch.where(big > 0, s_new, 0.0)
    after = torch.where(stays.any(1)[:, None], torch.maximum(scale, s_new), s_new)
    after = torch.where(touched[:, None], after, scale)
    div = after.clamp(min=1e-300)[:, :, None, None]
    moved = torch.where((after > scale)[:, :, None, None], _to_e4m3(cache * scale[:, :, None, None] / div), cache)
    codes = torch.where(is_new[:, None, :, None], _to_e4m3(rows / div), torch.where(stays[:, None, :, None], moved, cache))
    return codes, after


def _to_e4m3(x):
    """Nearest value of the 8-bit type, ties to even, saturating, in 64 bits."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e + 1) <= x.abs(), e + 1, e)
    step = torch.exp2(e.clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_logits(case, s):
    B, rows, V = s["logits"].shape
    out = s["out"].double()
    off = s["bias_offsets"].tolist()
    P, S, N = s["prompt_len"].tolist(), s["history_len"].tolist(), s["draft_len"].tolist()
    mr = s["mask_rows"].tolist()
    bits = torch.arange(32, dtype=torch.int32, device=DEV)
    for b in range(B):
        rep, pres, freq = (s[k][b].double() for k in ("repetition", "presence", "frequency"))
        h = s["history"][b, :S[b]].long()
        prompt = torch.bincount(h[:P[b]], minlength=V)
        bias = torch.zeros(V, dtype=torch.float64, device=DEV)
        bias.index_put_((s["bias_ids"][off[b]:off[b + 1]].long(),), s["bias_values"][off[b]:off[b + 1]].double(), accumulate=True)
        for j in range(N[b] + 1):
            count = torch.bincount(torch.cat([h[P[b]:], s["draft_tokens"][b, :j].long()]), minlength=V)
            y = s["logits"][b, j].double()
            seen = (prompt + count) > 0
            y = torch.where(seen & (y > 0), y / rep, torch.where(seen, y * rep, y))
            y = y - freq * count - pres * (count > 0) + bias
            if mr[b][j] >= 0:
                allow = ((s["mask"][mr[b][j]][:, None] >> bits) & 1).view(-1)[:V]
                y = torch.where(allow > 0, y, -math.inf)
            out[b, j] = y
    return out


def _exact_attention(case, s):
    D, H, Hq, bs = case["D"], case["H"], case["Hq"], case["bs"]
    G = Hq // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    cu, kept = s["cu_tokens"].tolist(), s["kv_len"].tolist()
    for b in range(case["B"]):
        n = cu[b + 1] - cu[b]
        L = kept[b] + n
        blocks = s["block_table"][b, :(L + bs - 1) // bs].long()
        k, v = ((c.view(torch.uint8)[blocks].view(E4M3).double() * sc[blocks].double()[:, :, None, None]).transpose(0, 1).reshape(H, -1, D)[:, :L]
                for c, sc in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
        x = s["q"][cu[b]:cu[b + 1]].double().view(n, H, G, D).permute(1, 0, 2, 3).reshape(H, n * G, D)
        w = torch.matmul(x, k.transpose(1, 2)).view(H, n, G, L) / math.sqrt(D)
        late = torch.arange(L, device=DEV)[None] > kept[b] + torch.arange(n, device=DEV)[:, None]
        w = torch.softmax(w.masked_fill(late[None, :, None], -math.inf), dim=3)
        o = torch.matmul(w.view(H, n * G, L), v).view(H, n, G, D)
        out[cu[b]:cu[b + 1]] = o.permute(1, 0, 2, 3).reshape(n, Hq, D)
    return out
