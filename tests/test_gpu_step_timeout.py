"""The failure path of spec_process_logits on the GPU, without a fault: a build of
the step's operators in which the first CTA never hands on its second item
(SPECDEC_TEST_WAIT_RUNS_OUT, with short waits).  The CTA's roles give up in turn,
the call reports SPECDEC_DEV_ERR_TIMEOUT, every other CTA's rows are right, and
nothing outside the call's rows is touched."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from tests.parity import wait_gpu
from tests.test_gpu_step import _check_logits, _logit_case, dev, err_word

pytestmark = pytest.mark.gpu

sd = pytest.importorskip("speculative_decoding_verification_80_gb300")
PKG = os.path.dirname(sd.__file__)
ROOT = os.path.dirname(PKG)


@pytest.fixture(scope="module")
def stall_lib(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sd.load_library()
    out = str(tmp_path_factory.mktemp("stall") / "libstep_stall.so")
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-shared", "-Xcompiler",
                    "-fPIC", f"-I{os.path.join(ROOT, 'include')}", f"-I{os.path.join(PKG, 'csrc')}",
                    "-DSPECDEC_TEST_WAIT_RUNS_OUT", "-DSPECDEC_STEP_WAIT_LOOKS=(1u<<14)",
                    os.path.join(PKG, "csrc", "step_api.cu"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    from speculative_decoding_verification_80_gb300 import step

    step.declare(lib)
    return lib


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("masks", [0, 3])
def test_a_wait_that_runs_out_ends_the_call(stall_lib, in_place, masks):
    rng = np.random.default_rng(7 + masks)
    B, n, V = 160, 3, 17000
    c = _logit_case(rng, B, n, V, 60, masks=masks)
    x = torch.tensor(rng.normal(0, 3, (B, n + 1, V))).to(torch.bfloat16).cuda()
    # the rows lie between others that the call must not touch
    pad = 4 * V
    buf = torch.full((x.numel() + 2 * pad,), 77.0, dtype=torch.bfloat16, device="cuda")
    out = buf[pad:pad + x.numel()].view(x.shape)
    if in_place:
        out.copy_(x)
    err = err_word()
    P = ctypes.c_void_p
    d = {k: dev(v) for k, v in c.items()}
    p = lambda k: P(d[k].data_ptr()) if k in d else None  # noqa: E731
    st = stall_lib.spec_process_logits(
        P((out if in_place else x).data_ptr()), P(out.data_ptr()), sd.BF16, B, n, V, p("history"), c["history"].shape[1],
        p("prompt_len"), p("history_len"), p("draft_tokens"), p("draft_len"), p("repetition"), p("presence"), p("frequency"),
        p("bias_offsets"), p("bias_ids"), p("bias_values"), len(c["bias_ids"]), p("mask"), masks, p("mask_rows"),
        P(err.data_ptr()), P(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    wait_gpu(timeout_s=60.0)
    assert err.item() == sd.DEV_ERR_TIMEOUT
    assert (buf[:pad] == 77).all() and (buf[-pad:] == 77).all()
    # the first CTA's items from its second on may hold anything in their own rows; all else is right
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    share, chunks = 8192, 3
    assert B * chunks > 2 * sms
    want = sd.spec_process_logits(x, out=torch.full_like(x, 77.0) if not in_place else x.clone(), **d)
    wait_gpu()
    for i in range(1, B * chunks // sms + 1):
        item = i * sms + (7 * i) % sms
        if item < B * chunks:
            b, v0 = item // chunks, item % chunks * share
            rows = int(c["draft_len"][b]) + 1
            out[b, :rows, v0:v0 + share] = want[b, :rows, v0:v0 + share]
    untouched = x.double().cpu().numpy() if in_place else 77.0
    _check_logits(x, c, out, untouched)
    _check_logits(x, c, want, untouched)  # the library's own call, on the same context
