"""Arguments of pipeline.moe_train_forward and moe_train_backward, on the CPU:
what does not fit together is refused before any call is made, so a refused
backward pass has added nothing to the gradients it was given.  The library's
calls are recorded instead of made."""
import pytest
import torch

import fp4_quantized_gemm_amd as F
from fp4_quantized_gemm_amd import pipeline
from tests.test_abi_train import OnDevice, there

T, H, E, TK, I = 6, 384, 4, 2, 128
F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


def weights(e, n, k):
    return pipeline.QuantWeights(None, None, there(e, dtype=F32), None,
                                 there(e, 2, n // 16, k // 64, 16, 32, dtype=U8),
                                 there(e, 2, n // 16, k // 64, 16, 4, dtype=U8))


def state(**kw):
    P = T * TK
    s = dict(x=there(T, H, dtype=U8), x_scales=there(T, H // 32, dtype=U8),
             y1=there(P, 2 * I, dtype=U8), y1_scales=there(P, 2 * I // 32, dtype=U8),
             topk_ids=there(T, TK, dtype=I32), topk_w=there(T, TK, dtype=F32),
             offsets=there(E + 1, dtype=I32), perm_token=there(P, dtype=I32),
             inv_perm=there(T, TK, dtype=I32), w_first=weights(E, 2 * I, H),
             w_down=weights(E, H, I))
    return pipeline.TrainState(**{**s, **kw})


@pytest.fixture
def calls(monkeypatch):
    """(name, keyword arguments) of every call, none made."""
    made = []
    P = T * TK

    def stub(name, result):
        def call(*a, **kw):
            made.append((name, kw))
            return result(*a, **kw) if callable(result) else result
        monkeypatch.setattr(pipeline, name, call)

    stub("moe_permute", (there(T, TK, dtype=I32), there(T, TK, dtype=F32), there(E + 1, dtype=I32),
                         there(P, dtype=I32), there(T, TK, dtype=I32)))
    stub("grouped_w4a16_gemm", there(P, 2 * I))
    stub("mxfp8_checkpoint", dict(codes=there(P, 2 * I, dtype=U8),
                                  scales=there(P, 2 * I // 32, dtype=U8), h=there(P, I)))
    stub("moe_unpermute_combine", there(T, H))
    stub("grouped_w4a16_dgrad", there(P, I))
    stub("moe_swiglu_backward", (there(P, 2 * I), there(P, I), there(T, TK, dtype=F32)))
    stub("grouped_wgrad", lambda *a, **kw: kw.get("out"))
    return made


@pytest.mark.parametrize("kw", [
    dict(dw_first=there(E, 2 * I, H)),                               # bf16 cannot be added to
    dict(dw_first=there(E, H, 2 * I, dtype=F32)),
    dict(dw_first=there(E, 2 * I, 2 * H, dtype=F32)[:, :, ::2]),
    dict(dw_first=torch.zeros(E, 2 * I, H)),                         # a host tensor
    dict(dw_first=there(E, 2 * I, H, dtype=F32), dw_down=there(E, I, H, dtype=F32)),
    dict(dw_dtype=torch.float16),                                    # of dw_first, which is not given
])
def test_a_refused_backward_has_added_nothing(calls, kw):
    kw.setdefault("dw_down", there(E, H, I, dtype=F32))
    with pytest.raises(F.NvfpError):
        pipeline.moe_train_backward(state(), there(T, H), **kw)
    assert not calls


def test_the_larger_weight_gradient_comes_first(calls, monkeypatch):
    """Limits that only grouped_wgrad knows (4 GiB operands, 2^30 elements of
    dw) are passed by the down projection's whenever they are by the first's."""
    first = there(E, 2 * I, H, dtype=F32)

    def refuse(*a, **kw):
        if kw["out"] is first:
            raise F.NvfpError("dy or x exceeds 4 GiB")
        calls.append(("grouped_wgrad", kw))
    monkeypatch.setattr(pipeline, "grouped_wgrad", refuse)
    with pytest.raises(F.NvfpError, match="4 GiB"):
        pipeline.moe_train_backward(state(), there(T, H), dw_first=first,
                                    dw_down=there(E, H, I, dtype=F32))
    assert "grouped_wgrad" not in [c[0] for c in calls]


@pytest.mark.parametrize("d_out", [there(T - 1, H), there(T + 1, H), there(T * H), there(T, 2 * H)])
def test_backward_refuses_d_out_of_other_tokens(calls, d_out):
    """Its rows are gathered by token: too few would be read as the last one."""
    with pytest.raises(F.NvfpError, match="d_out"):
        pipeline.moe_train_backward(state(), d_out)
    assert not calls


def test_backward_runs(calls):
    first, down = there(E, 2 * I, H, dtype=F32), there(E, H, I, dtype=F32)
    g = pipeline.moe_train_backward(state(), there(T, H), dw_first=first, dw_down=down,
                                    dw_dtype=None)
    assert g["dw_first"] is first and g["dw_down"] is down
    assert all(c[1]["accumulate"] for c in calls if c[0] == "grouped_wgrad")
    for dt in (F32, BF16):
        del calls[:]
        pipeline.moe_train_backward(state(), there(T, H), dw_dtype=dt)
        assert [c[1]["dtype"] for c in calls if c[0] == "grouped_wgrad"] == [dt, dt]


def forward(x=None, logits=None, topk=TK, w_first=None, w_down=None, **kw):
    return pipeline.moe_train_forward(
        there(T, H) if x is None else x, there(T, E, dtype=F32) if logits is None else logits, topk,
        w_first or weights(E, 2 * I, H), w_down or weights(E, H, I), **kw)


@pytest.mark.parametrize("kw,name", [
    (dict(x=there(T - 1, H)), "logits"), (dict(x=there(T + 1, H)), "logits"),
    (dict(x=torch.zeros(T, H, dtype=BF16)), "x"), (dict(x=there(T, H, dtype=F32)), "x"),
    (dict(logits=there(T, E - 1, dtype=F32)), "w_first"),            # offsets of E - 1 experts
    (dict(logits=there(T, E + 1, dtype=F32)), "w_first"),
    (dict(x=there(T, 2 * H)), "w_first"),                            # weights read past their end
    (dict(w_first=weights(E + 1, 2 * I, H)), "w_first"),
    (dict(w_down=weights(E + 1, H, I)), "w_down"), (dict(w_down=weights(E, H, 2 * I)), "w_down"),
    (dict(w_down=weights(E, 2 * H, I)), "w_down"), (dict(w_first=weights(E, I, H)), "w_down"),
    (dict(bias=there(E - 1, dtype=F32)), "bias"), (dict(bias=there(E)), "bias"),
    (dict(bias=torch.zeros(E)), "bias"),
])
def test_forward_refuses_what_does_not_fit(calls, kw, name):
    """The products take their sizes from one operand and index the others
    with them on the device."""
    with pytest.raises(F.NvfpError, match=name):
        forward(**kw)
    assert not calls


def test_forward_runs(calls):
    out, st = forward(bias=there(E, dtype=F32))
    assert out.shape == (T, H) and st.w_down.g.shape == (E,)
    forward(bias=there(1, E, dtype=F32), checkpoint="bf16")
    assert [c[0] for c in calls].count("grouped_w4a16_gemm") == 4


@pytest.fixture
def current(monkeypatch):
    """Which device is current, as torch.cuda.device sets it."""
    stack = ["cuda:0"]

    class Device:
        def __init__(self, dev):
            self.dev = str(dev)

        def __enter__(self):
            stack.append(self.dev)

        def __exit__(self, *exc):
            stack.pop()
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(OnDevice, "device", property(lambda t: torch.device("cuda", 1)),
                        raising=False)
    return stack


def test_a_step_runs_with_its_tensors_device_current(calls, current, monkeypatch):
    """Some of the calls launch on the current device's default stream: all run
    where the tensors are, and the device that was current is so again."""
    where = []
    for name in ["moe_permute", "grouped_w4a16_gemm", "mxfp8_checkpoint", "moe_unpermute_combine",
                 "grouped_w4a16_dgrad", "moe_swiglu_backward", "grouped_wgrad"]:
        def call(*a, _f=getattr(pipeline, name), **kw):
            where.append(current[-1])
            return _f(*a, **kw)
        monkeypatch.setattr(pipeline, name, call)
    forward()
    pipeline.moe_train_backward(state(), there(T, H))
    assert len(where) == 12 and set(where) == {"cuda:1"} and current == ["cuda:0"]
    with pytest.raises(F.NvfpError):
        forward(x=there(T - 1, H))
    assert current == ["cuda:0"]


@pytest.mark.parametrize("bad", [None, 3.0, [[1.0]]])
def test_what_is_no_tensor_is_refused_like_the_rest(calls, bad):
    with pytest.raises(F.NvfpError, match="d_out"):
        pipeline.moe_train_backward(state(), bad)
    with pytest.raises(F.NvfpError, match="x must"):
        pipeline.moe_train_forward(bad, there(T, E, dtype=F32), TK, weights(E, 2 * I, H),
                                   weights(E, H, I))
    with pytest.raises(F.NvfpError, match="logits must"):
        pipeline.moe_train_forward(there(T, H), bad, TK, weights(E, 2 * I, H), weights(E, H, I))
    assert not calls
