"""What the expert-layer calls and their tensor helpers refuse before they touch a device."""
from types import SimpleNamespace

import pytest
import torch

import lossless_entropy_coded_exponent_b200 as dfx
from lossless_entropy_coded_exponent_b200 import build as dfx_build


def weight(*shape, block_rows=128):
    """An Fp8 of shape [.., rows, cols]."""
    *lead, rows, cols = shape
    up = lambda n, to: -(-n // to) * to  # noqa: E731
    return dfx.Fp8(torch.zeros(*lead, rows, up(cols, 16), dtype=torch.uint8),
                   torch.zeros(*lead, -(-rows // block_rows), up(-(-cols // 128), 16), dtype=torch.uint8), cols, block_rows)


LAYER = dict(x=torch.zeros(10, 200), logits=torch.zeros(10, 4), w_in=weight(4, 96, 200), w_out=weight(4, 200, 48), topk=2)


def test_a_sound_layer_is_only_stopped_by_the_missing_device():
    with pytest.raises(ValueError, match="CUDA device"):
        dfx.experts_fp8(**LAYER)
    with pytest.raises(ValueError, match="CUDA device"):  # one matrix for one expert
        dfx.experts_fp8(**{**LAYER, "logits": torch.zeros(10, 1), "w_in": weight(96, 200), "w_out": weight(200, 48), "topk": 1})


@pytest.mark.parametrize("changes", [
    dict(logits=torch.zeros(9, 4)),            # fewer tokens than x: rows of the result would be missing
    dict(logits=torch.zeros(11, 4)),           # more: rows that x does not have
    dict(logits=torch.zeros(4)),
    dict(x=torch.zeros(1, 10, 200)),
    dict(x=torch.zeros(10, 199)),
    dict(logits=torch.zeros(10, 5)),           # an expert without a matrix
    dict(logits=torch.zeros(10, 3)),
    dict(w_in=weight(4, 98, 200)),             # gates and values of other widths than w_out's
    dict(w_out=weight(4, 200, 47)),
    dict(w_out=weight(4, 199, 48)),
    dict(w_out=weight(3, 200, 48)),
    dict(w_in=weight(96, 200)),
    dict(w_in=weight(2, 2, 96, 200)),
    dict(w_in=weight(4, 96, 200, block_rows=1)),
])
def test_layers_whose_parts_do_not_fit_are_refused(changes):
    with pytest.raises(ValueError, match="experts_fp8: (x|w_in)"):
        dfx.experts_fp8(**{**LAYER, **changes})


class Elsewhere(torch.Tensor):
    """Only claims its device."""
    is_cuda, device = True, torch.device("cuda", 0)


def elsewhere(t):
    if isinstance(t, dfx.Fp8):
        return t._replace(values=elsewhere(t.values), scales=elsewhere(t.scales))
    return t.as_subclass(Elsewhere)


@pytest.mark.parametrize("helper,args", [
    ("route", (torch.zeros(4, 8), 2)),
    ("quantize_fp8", (torch.zeros(4, 8),)),
    ("gemm_fp8", (weight(4, 128, block_rows=1), weight(4, 128))),
    ("combine", (torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))),
    ("experts_fp8", tuple(LAYER.values())),
])
def test_a_stream_of_another_device_is_refused(helper, args, monkeypatch):
    """Its kernels would get addresses of a device that is not theirs."""
    monkeypatch.setattr(dfx, "dfx_plan", lambda n: pytest.fail("the call went on"))
    args = [a if isinstance(a, int) else elsewhere(a) for a in args]
    with pytest.raises(ValueError, match="a stream of cuda:1"):
        getattr(dfx, helper)(*args, stream=SimpleNamespace(device=torch.device("cuda", 1)))


@pytest.mark.parametrize("changes", [
    dict(bias=torch.zeros(4)),
    dict(logits=LAYER["logits"]),
    dict(w_in=elsewhere(LAYER["w_in"])._replace(scales=LAYER["w_in"].scales)),
    dict(w_out=elsewhere(LAYER["w_out"])._replace(values=LAYER["w_out"].values)),
])
@pytest.mark.parametrize("stream", [None, SimpleNamespace(device=torch.device("cuda", 0))])
def test_a_layer_on_several_devices_is_refused(changes, stream):
    layer = {k: v if isinstance(v, int) else elsewhere(v) for k, v in LAYER.items()}
    with pytest.raises(ValueError, match="different devices"):
        dfx.experts_fp8(**{**layer, **changes}, stream=stream)


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes a plan and pointers that are not the device's")
def test_sums_too_long_for_the_waits_are_refused():
    """The warps that wait for a sum over K give up after some 0.35 s, and 128 columns take some 0.4 us."""
    from test_experts_cpu import CUDA, GEMM, TOO_LARGE, call

    dfx_build.build()
    for cols, code in ((1 << 25, CUDA), ((1 << 25) + 1, TOO_LARGE), (1 << 30, TOO_LARGE)):
        ld, blocks = -(-cols // 16) * 16, -(-cols // 512) * 4
        assert call("dfx_gemm_fp8", GEMM, cols=cols, ld_x=ld, ld_w=ld, ld_sx=blocks, ld_sw=blocks) == code
