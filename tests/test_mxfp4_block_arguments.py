"""Arguments of the MXFP4 block, on the CPU: operands that do not fit together
are refused before any call is made."""
import pytest
import torch

import fp4_quantized_gemm_amd as F
from fp4_quantized_gemm_amd import pipeline
from tests.test_abi_train import there
from tests.test_train_arguments import E, F32, H, I, T, TK, U8, calls, state, weights  # noqa: F401

BF16 = torch.bfloat16


def mx(e, n, k, transposed=True, **kw):
    t = (there(e, k, n // 2, dtype=U8), there(e, k, n // 32, dtype=U8)) if transposed else (None, None)
    w = pipeline.MxWeights(there(e, n, k // 2, dtype=U8), there(e, n, k // 32, dtype=U8), *t)
    for name, v in kw.items():
        setattr(w, name, v)
    return w


def forward(train, x=None, logits=None, bias=None, w_first=None, w_down=None):
    f = pipeline.moe_train_forward if train else pipeline.moe_forward_mxfp4
    return f(there(T, H) if x is None else x, there(T, E, dtype=F32) if logits is None else logits, TK,
             w_first or mx(E, 2 * I, H), w_down or mx(E, H, I), bias)


@pytest.fixture
def made(calls, monkeypatch):                            # noqa: F811
    P = T * TK
    for name, result in (("mxfp4_quantize", (there(P, 64, dtype=U8), there(P, 4, dtype=U8))),
                         ("grouped_mxfp4_gemm", there(P, 2 * I)), ("grouped_mxfp4_gemm_swiglu", there(P, I)),
                         ("moe_permute_backward", (there(T, E, dtype=F32), there(E, dtype=F32)))):
        def call(*a, _r=result, _n=name, **kw):
            calls.append((_n, kw))
            return _r
        monkeypatch.setattr(pipeline, name, call)
    return calls


@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("kw", [
    dict(x=there(T, H, dtype=F32)), dict(x=there(T + 1, H)), dict(x=there(T, H + 128)), dict(x=None, logits=there(T, E)),
    dict(logits=there(T, E + 1, dtype=F32)), dict(bias=there(E + 1, dtype=F32)), dict(bias=there(E)),
    dict(w_first=mx(E + 1, 2 * I, H)), dict(w_first=mx(E, 2 * I, 2 * H)), dict(w_first=mx(E, 4 * I, H)),
    dict(w_first=mx(E, 2 * I, H, scales=there(E, 2 * I, H // 16, dtype=U8))),
    dict(w_down=mx(E, H, 2 * I)), dict(w_down=mx(E, H // 2, I)), dict(w_down=mx(E, H, I, codes=there(E, H, I // 2))),
    dict(w_down=weights(E, H, I)), dict(w_first=weights(E, 2 * I, H)),
])
def test_what_does_not_fit_is_refused(made, train, kw):
    with pytest.raises(F.NvfpError):
        forward(train, **kw)
    assert not made


@pytest.mark.parametrize("kw", [
    dict(w_first=mx(E, 2 * I, H, transposed=False)), dict(w_down=mx(E, H, I, transposed=False)),
    dict(w_down=mx(E, H, I, t_codes=there(E, H, I // 2, dtype=U8))),
    dict(w_first=mx(E, 2 * I, H, t_scales=there(E, H, I // 32, dtype=U8))),
])
def test_training_needs_the_transposes(made, kw):
    with pytest.raises(F.NvfpError):
        forward(True, **kw)
    assert not made


def test_calls_of_a_forward_and_a_step(made):
    forward(False, w_first=mx(E, 2 * I, H, transposed=False))
    assert [c[0] for c in made] == ["moe_permute", "mxfp4_quantize", "grouped_mxfp4_gemm_swiglu", "mxfp4_quantize",
                                    "grouped_mxfp4_gemm", "moe_unpermute_combine"]
    made.clear()
    _, st = forward(True, bias=there(E, dtype=F32))
    assert st.has_bias
    g = pipeline.moe_train_backward(st, there(T, H), want_d_logits=True)
    assert "d_bias" in g and made[-1] == ("moe_permute_backward", dict(want_bias=True))
    assert not any(n.startswith("grouped_w4a16") for n, _ in made)


def test_gradient_of_the_logits_on_request(made):
    g = pipeline.moe_train_backward(state(), there(T, H))
    assert "d_logits" not in g and not any(n == "moe_permute_backward" for n, _ in made)
    g = pipeline.moe_train_backward(state(), there(T, H), want_d_logits=True)
    assert "d_logits" in g and "d_bias" not in g


def test_gradients_to_add_to_fit(made):
    st = forward(True)[1]
    made.clear()
    for kw in (dict(dw_first=there(E, 2 * I, H)), dict(dw_first=there(E, H, 2 * I, dtype=F32)),
               dict(dw_down=there(E, H, H, dtype=F32)), dict(dw_dtype=torch.float16)):
        with pytest.raises(F.NvfpError):
            pipeline.moe_train_backward(st, there(T, H), **kw)
    assert not made
    pipeline.moe_train_backward(st, there(T, H), dw_first=there(E, 2 * I, H, dtype=F32),
                                dw_down=there(E, H, I, dtype=F32))


def test_training_refuses_strided_rows_at_once(made):
    """The products would take them, the weight gradients after them not: then
    the first gradient would have been added to."""
    wide = there(T, 2 * H)[:, :H]
    with pytest.raises(F.NvfpError):
        forward(True, x=wide)
    assert not made
    forward(False, x=wide)
    st = forward(True)[1]
    made.clear()
    for bad in (wide, there(T, H, dtype=F32)):
        with pytest.raises(F.NvfpError):
            pipeline.moe_train_backward(st, bad, dw_first=there(E, 2 * I, H, dtype=F32))
    assert not made


def test_prepared_weights_are_stacked():
    for w in (there(4, 128), there(2, 4, 128, dtype=F32), torch.zeros(2, 4, 128, dtype=BF16), None):
        with pytest.raises(F.NvfpError):
            pipeline.prepare_mxfp4_weights(w)
