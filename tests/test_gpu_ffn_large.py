"""GPU: checkpoints of tensors past what one launch holds (2^32 threads of 8
values).  About 100 GB of device memory."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_gmm_amd as gmm
import test_gpu_ffn as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.slow
def test_checkpoint_past_one_launch():
    K = 1 << 15
    M = (1 << 20) + 3                        # M K = 2^35 + 3 K: the last rows are past 2^32 threads
    if torch.cuda.mem_get_info()[0] < 115e9:
        pytest.skip("needs 115 GB of free device memory")
    rows = [0, (1 << 19) - 1, 1 << 19, (1 << 20) - 1, 1 << 20, M - 1]
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    vals = T.normal(5, (len(rows), K))
    for i, r in enumerate(rows):
        x[r] = vals[i].to(DEV)
    q, s = gmm.gmm_quantize_mx8(x)
    _, c, want = T.mx8_64(T.f64(vals))
    for i, r in enumerate(rows):
        assert np.array_equal(T.raw(s[r]), c[i]), r
    x.fill_(float("nan"))
    gmm.gmm_dequantize_mx8(q, s, out=x)
    for i, r in enumerate(rows):
        assert np.array_equal(T.f64(x[r]), want[i]), r
        x[r] = 0
    for lo in range(0, M, 1 << 17):          # every other row: zeros
        assert (x[lo:lo + (1 << 17)] == 0).all(), lo
