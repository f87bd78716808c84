"""Sampling, rotary positions, forks and compaction together, as
examples/decode_step.py runs them with the other operators."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _decoder(**kw):
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.Decoder(**{**dict(V=1000, hidden=128, Hq=8, H=2, D=64, max_len=200), **kw})


def _prompts(B, n=37):
    return torch.randint(0, 1000, (B, n), generator=torch.Generator(device="cuda").manual_seed(B), device="cuda", dtype=torch.int32)


def _blocks(d):
    """Every block is free once, or held by shares + 1 requests."""
    held, (head, count) = d.state.held.tolist(), d.state.ring_state.tolist()
    N = d.ring.numel()
    free = [int(d.ring[(head + i) % N]) for i in range(count)]
    owned = torch.cat([d.table[b, :held[b]] for b in range(d.B)]).cpu()
    times = torch.bincount(owned.long(), minlength=N)
    assert sorted(free + sorted(set(owned.tolist()))) == list(range(N))
    assert torch.equal(times[times > 0] - 1, d.shares.cpu()[times > 0].long()) and int(d.shares.cpu()[times == 0].sum()) == 0


@pytest.mark.parametrize("rotary", [False, True])
@pytest.mark.parametrize("B,drafts", [(1, 3), (6, 2), (5, 0)])
def test_one_id_left_is_the_greedy_loop(B, drafts, rotary):
    runs = []
    for kw in (dict(), dict(temperature=0.7, top_k=1), dict(temperature=0.7, top_p=1e-6), dict(temperature=1.3, top_k=1, min_p=1.0)):
        d = _decoder(B=B, drafts=drafts, rotary=rotary, **kw)
        d.prompt(_prompts(B))
        for _ in range(8):
            d.step()
        torch.cuda.synchronize()
        assert int(d.error) == 0
        runs.append((d.history_len.clone(), d.history.clone()))
    for length, history in runs[1:]:
        assert torch.equal(length, runs[0][0]) and torch.equal(history, runs[0][1])


def test_drawn_tokens_vary_and_repeat_by_the_seed():
    out = []
    for seed in (0, 0, 3):
        d = _decoder(B=4, drafts=3, rotary=True, temperature=1.0, top_k=50, top_p=0.95)
        d.random.manual_seed(seed)
        d.prompt(_prompts(4))
        for _ in range(6):
            d.step()
        torch.cuda.synchronize()
        assert int(d.error) == 0
        _blocks(d)
        out.append(d.history.clone())
    assert torch.equal(out[0], out[1]) and not torch.equal(out[0], out[2])


@pytest.mark.parametrize("block_size,drafts", [(16, 3), (64, 1)])
def test_forks_go_on_as_their_parents_do(block_size, drafts):
    """Greedy: a child makes what its parent would have made, whoever else writes beside it."""
    plain = _decoder(B=6, drafts=drafts, rotary=True, block_size=block_size)
    plain.prompt(_prompts(6))
    forked = _decoder(B=6, drafts=drafts, rotary=True, block_size=block_size)
    forked.prompt(_prompts(6))
    for _ in range(3):
        plain.step()
        forked.step()
    parent = torch.tensor([0, 0, 3, 3, 3, 5], dtype=torch.int32, device="cuda")
    forked.fork(parent)
    _blocks(forked)
    assert (int(forked.shares.sum()) > 0) == (block_size <= 37)  # a prompt of 37 fills blocks of 16, none of 64
    for i in range(6):
        plain.step()
        forked.step()
        if i == 2:
            forked.fork(torch.arange(6, dtype=torch.int32, device="cuda"))  # everyone goes on from itself
            _blocks(forked)
    torch.cuda.synchronize()
    assert int(forked.error) == 0
    want, got = plain.history[parent.long()], forked.history
    assert torch.equal(plain.history_len[parent.long()], forked.history_len)
    for b in range(6):
        n = int(forked.history_len[b])
        assert torch.equal(want[b, :n], got[b, :n])
    _blocks(forked)


def test_compaction_changes_no_token():
    runs = []
    for compact in (False, True):
        d = _decoder(B=5, drafts=2, rotary=True, temperature=0.9, top_p=0.9)
        d.prompt(_prompts(5))
        for i in range(8):
            if i == 2:
                d.fork(torch.tensor([4, 4, 2, 2, 0], dtype=torch.int32, device="cuda"))
            if compact and i in (1, 3, 6):
                d.compact()
                _blocks(d)
                held = d.state.held.tolist()
                named = {int(x) for b in range(5) for x in d.table[b, :held[b]]}
                assert named == set(range(len(named)))
            d.step()
        torch.cuda.synchronize()
        assert int(d.error) == 0
        _blocks(d)
        runs.append((d.history_len.clone(), d.history.clone()))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
