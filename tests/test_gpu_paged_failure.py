"""Failure detection of paged attention's kernel for chunks of prompts, without a GPU fault: its
bounded waits run out when one internal signal is withheld (test hook), every warp leaves through
the abort path, the device status word reports it, and the next call is right."""
import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged_attn import make, run

pytestmark = pytest.mark.gpu


# one half of a block and two; fewer tiles than the stages of its rings and more; sequences of the narrow
# kernel beside it; a window
@pytest.mark.parametrize("lens,nq,kw", [([1400], [1300], {}), ([640, 7], [640, 1], {}), ([2000, 800], [30, 400], {}),
                                        ([900, 500], [500, 300], dict(window=100, sinks=3))])
def test_waits_that_run_out(spin_gpu, lens, nq, kw):
    q, cache, table, cu = make(lens, nq, 32, 8, 64, seed=sum(nq))
    want = run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16, **kw)
    torch.cuda.synchronize()
    assert spin_gpu.device_status(reset=True) == 0
    try:
        spin_gpu.test_stall_tensor_core_waits(True)
        run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16, **kw)
        torch.cuda.synchronize()  # returns: every wait is bounded
    finally:
        spin_gpu.test_stall_tensor_core_waits(False)
    assert spin_gpu.device_status(reset=True) != 0
    assert spin_gpu.device_status() == 0
    again = run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16, **kw)
    torch.cuda.synchronize()
    assert torch.equal(again, want) and spin_gpu.device_status() == 0


@pytest.mark.parametrize("lens,nq,wide", [([100] * 280 + [700], [1] * 280 + [20], False),
                                          ([100] * 900 + [700, 300], [1] * 900 + [64, 65], False),
                                          ([100] * 280 + [700], [1] * 280 + [300], True),
                                          ([90] * 20, [17] * 20, True), ([90] * 20, [16] * 20, False)])
def test_few_wide_rows_stay_with_the_narrow_kernel(spin_gpu, lens, nq, wide):
    """A call of many tokens whose chunks are too small to fill the GPU in blocks of 256 rows: the kernel
    for chunks leaves them alone, which the hook shows (it has no wait that could run out)."""
    q, cache, table, cu = make(lens, nq, 32, 8, 32, seed=len(lens))
    spin_gpu.device_status(reset=True)
    try:
        spin_gpu.test_stall_tensor_core_waits(True)
        got = run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
    finally:
        spin_gpu.test_stall_tensor_core_waits(False)
    assert (spin_gpu.device_status(reset=True) != 0) == wide
    if wide:
        got = run(spin_gpu, q, cache, table, lens, cu, out_dtype=torch.bfloat16)
    ref.check_attention(got, ref.attention(q, cache, table, lens, cu), "bf16")
