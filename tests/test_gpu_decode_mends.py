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
