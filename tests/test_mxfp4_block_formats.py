"""Weights of the MXFP4 block, on the CPU: those of another format are refused
before any call is made."""
import pytest

import fp4_quantized_gemm_amd as F
from fp4_quantized_gemm_amd import pipeline
from tests.test_abi_train import there
from tests.test_mxfp4_block_arguments import forward, made, mx  # noqa: F401
from tests.test_train_arguments import E, F32, H, I, T, TK, calls, weights  # noqa: F401


@pytest.mark.parametrize("first,down", [
    (weights(E, 2 * I, H), weights(E, H, I)), (mx(E, 2 * I, H), weights(E, H, I)),
    (weights(E, 2 * I, H), mx(E, H, I)), (None, None), (mx(E, 2 * I, H), None),
    (there(E, 2 * I, H), there(E, H, I)),
])
def test_serving_takes_mxfp4_weights_only(made, first, down):  # noqa: F811
    """Both of the other format fit together, and would be found out only by
    the first product, after the routing."""
    with pytest.raises(F.NvfpError):
        pipeline.moe_forward_mxfp4(there(T, H), there(T, E, dtype=F32), TK, first, down)
    assert not made
    forward(False)
    assert made
