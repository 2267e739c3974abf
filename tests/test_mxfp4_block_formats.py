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


@pytest.mark.parametrize("keep", [False, True])
def test_calls_of_a_step_that_keeps_y2(made, monkeypatch, keep):  # noqa: F811
    """y2's gradient is taken before any weight gradient is added to, and d_topk_w
    and the logits' gradient are formed from its result."""
    exact, seen = there(T, TK, dtype=F32), []
    monkeypatch.setattr(pipeline, "moe_unpermute_combine_backward",
                        lambda *a: made.append(("combine_backward", {})) or (None, exact))
    route = pipeline.moe_permute_backward
    monkeypatch.setattr(pipeline, "moe_permute_backward", lambda *a, **kw: seen.append(a[2]) or route(*a, **kw))
    args = (there(T, H), there(T, E, dtype=F32), TK, mx(E, 2 * I, H), mx(E, H, I))
    st = pipeline.moe_train_forward(*args, keep_y2=keep)[1]
    assert (st.y2 is not None) == keep
    made.clear()
    g = pipeline.moe_train_backward(st, there(T, H), want_d_logits=True)
    names = [n for n, _ in made]
    assert ("combine_backward" in names) == keep and (g["d_topk_w"] is exact) == keep
    assert (seen[0] is exact) == keep
    if keep:
        assert names.index("combine_backward") < names.index("grouped_wgrad")
    made.clear()
    with pytest.raises(F.NvfpError):
        pipeline.moe_train_backward(st, there(T, 2 * H)[:, :H])
    assert not made
