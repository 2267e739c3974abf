"""grouped_mxfp4_gemm with as many rows as a call takes, all of one expert: the
count of its row tiles adds a tile's rows less one to 2^31 - 1, which 32 bits with a
sign do not hold."""
import numpy as np
import pytest
import torch

import fp4_quantized_gemm_amd as F
from tests.test_gpu_mxfp4 import cu, operands, say

pytestmark = pytest.mark.gpu


def test_one_expert_with_all_rows(dev):
    say("mxfp4 2^31 - 1 rows")
    rng = np.random.default_rng(31)
    P, N, K, M_src = 2 ** 31 - 1, 16, 128, 5
    ac, asc, wc, wsc = (cu(a) for a in operands(rng, M_src, 2, N, K))
    rows = torch.arange(P, dtype=torch.int32, device="cuda").remainder_(M_src)
    # the second expert of two: the first one's tiles are none
    y = F.grouped_mxfp4_gemm(ac, asc, rows, wc, wsc, cu(np.array([0, 0, P], np.int32)))
    few = F.grouped_mxfp4_gemm(ac, asc, None, wc, wsc, cu(np.array([0, 0, M_src], np.int32)))
    step = 1 << 24                                       # (what torch's indexing takes at once)
    for i in range(0, P, step):
        assert torch.equal(y[i:i + step], few[rows[i:i + step].long()]), i
