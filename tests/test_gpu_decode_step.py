"""The operators of a decode step together, as examples/decode_step.py runs them."""
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
    return m.Decoder(**kw)


def _run(B, drafts, steps, block_size, max_len=200):
    g = torch.Generator(device="cuda").manual_seed(B)
    allowed = torch.rand(B, 1000, generator=g, device="cuda") < 0.3
    d = _decoder(B=B, drafts=drafts, V=1000, hidden=128, Hq=8, H=2, D=64, block_size=block_size, max_len=max_len, allowed=allowed)
    d.prompt(torch.randint(0, 1000, (B, 37), generator=g, device="cuda", dtype=torch.int32))
    lens, accepted = [d.history_len.tolist()], []
    for _ in range(steps):
        d.step()
        lens.append(d.history_len.tolist())
        accepted.append(d.accepted.tolist())
    torch.cuda.synchronize()
    return d, allowed.cpu(), lens, accepted


@pytest.mark.parametrize("B,drafts,block_size", [(1, 4, 16), (5, 3, 32), (33, 1, 16), (3, 0, 64)])
def test_decode_loop(B, drafts, block_size):
    steps = 12
    d, allowed, lens, accepted = _run(B, drafts, steps, block_size)
    assert int(d.error) == 0
    for i in range(steps):
        assert all(0 <= a <= drafts for a in accepted[i])
        assert [x - y for x, y in zip(lens[i + 1], lens[i])] == [a + 1 for a in accepted[i]]
    history = d.history.cpu()
    for b in range(B):
        made = history[b, 37:lens[-1][b]].long()
        assert bool(allowed[b][made].all())  # the grammar holds for every token made
    # what the cache keeps before the coming step is all but the last step's rejected drafts
    kept = (d.state.kv_len + d.accepted + 1).tolist()
    assert kept == [n - 1 for n in lens[-1]]  # the last token made has not been fed yet
    # no block is lost or held twice
    held, head, count = d.state.held.tolist(), *d.state.ring_state.tolist()
    N = d.ring.numel()
    free = [int(d.ring[(head + i) % N]) for i in range(count)]
    owned = [int(x) for b in range(B) for x in d.table[b, :held[b]]]
    assert sorted(free + owned) == list(range(N))


def test_decode_loop_is_the_same_every_time():
    a, _, lens_a, _ = _run(4, 3, 10, 16)
    b, _, lens_b, _ = _run(4, 3, 10, 16)
    assert lens_a == lens_b and torch.equal(a.history, b.history)
