"""Attention over the INT4 KV cache in pages where numbers leave the usual range: NaN queries,
scales and zeros that are not finite and are seen by some rows of a tile only, scales far apart,
large scores, long sequences. Against the binary64 statement."""
import math

import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged_attn import make, run

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

# (lens, nq, hq, hkv): one warp writes the row; warps of a block join it; blocks join it; several
# tokens; the kernel for chunks of prompts, in the first half of a block and in the second
SHAPES = {"short": ([50, 40], [1, 1], 8, 2), "joined in a block": ([460], [1], 8, 2),
          "joined by blocks": ([40000, 300], [1, 1], 8, 2), "drafts": ([3000, 70], [4, 2], 64, 8),
          "chunk": ([900, 333], [500, 300], 32, 8), "chunk, one head": ([1700], [1700], 8, 8)}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_nan_queries_give_nan(spin_gpu, shape, dtype):
    """A NaN (or an infinite) query row is not hidden behind a 0, and no other row knows of it."""
    lens, nq, hq, hkv = SHAPES[shape]
    q, cache, table, cu = make(lens, nq, hq, hkv, 64, seed=1)
    tokens = q.shape[0]
    bad = sorted({0, tokens // 3, tokens - 1})
    for t in bad:
        q[t] = math.nan
    inf = tokens // 2 if tokens > 4 else None
    if inf is not None:
        q[inf, :, 5] = math.inf
    q[bad[0], 1] = 0.5  # a head of the same token that is fine
    got = run(spin_gpu, q, cache, table, lens, cu, out_dtype=dtype)
    want = ref.attention(torch.nan_to_num(q, 1.0, 1.0, 1.0), cache, table, lens, cu)
    for t in bad:
        whole = torch.ones(hq, dtype=torch.bool, device="cuda")
        whole[1] = t != bad[0]
        assert torch.isnan(got[t, whole]).all(), t
    assert torch.isfinite(got[bad[0], 1]).all()
    rows = [t for t in range(tokens) if t not in bad[1:] and t != inf]
    if inf is not None:
        assert not torch.isfinite(got[inf]).any()
    fine = torch.zeros(tokens, hq, dtype=torch.bool)
    fine[rows] = True
    fine[bad[0]] = False
    fine[bad[0], 1] = True
    got = torch.where(fine[..., None].cuda(), got, want[0].to(got.dtype).cuda())
    what = "" if dtype == F32 else "prefill" if shape.startswith("chunk") else "bf16"
    ref.check_attention(got, want, what)
