"""Every tensor of an NVF4 or expert-layer call must be on the current GPU, as for
the FP8 calls: a host tensor and one of another GPU are refused before the library
is called.  Stand-ins for tensors, no GPU."""

import pytest
import torch

from test_fp8_devices_host import F8, F16, F32, I32, Called, Stand, dg  # noqa: F401

U8 = torch.uint8


def nvf4(rows, k, *lead):
    return (Stand(U8, *lead, rows, k // 2), Stand(F8, *lead, -(-rows // 128), -(-k // 64), 32, 16),
            Stand(F32, *lead, rows))


def calls():
    """name -> (function's name, its arguments by position, by keyword); tuples hold tensors."""
    a, b, w = nvf4(4, 256), nvf4(128, 256), nvf4(128, 256, 3)
    x, d = Stand(F16, 4, 256), Stand(F16, 4, 128)
    ids, wt = Stand(I32, 4, 2), Stand(F32, 4, 2)
    f8 = (Stand(F8, 3, 128, 256), Stand(F32, 3, 1, 2)), (Stand(F8, 3, 256, 128), Stand(F32, 3, 2, 1))
    bias = dict(bias_up=Stand(F16, 3, 128), bias_down=Stand(F16, 3, 256))
    return {
        "quantize": ("quantize_nvf4", [x], dict(out=a)),
        "given": ("quantize_nvf4", [x], dict(out=a[:2] + (None,), row_scales=a[2])),
        "dispatch": ("moe_dispatch_nvf4", [x, Stand(I32, 8), 2, *nvf4(8, 256)], {}),
        "dequantize": ("dequantize_nvf4", [*a, x], {}),
        "gemm": ("gemm_nvf4", [*a, *b, d], dict(bias=Stand(F16, 128), epilogue="bias")),
        "grouped": ("gemm_nvf4_grouped", [*a, *w, Stand(I32, 4), d],
                    dict(bias=Stand(F16, 3, 128), epilogue="bias")),
        "layer_nvf4": ("moe_layer", [x, ids, wt, w, nvf4(256, 128, 3), Stand(F16, 4, 256)], bias),
        "layer_fp8": ("moe_layer", [x, ids, wt, *f8, Stand(F16, 4, 256)], bias),
    }


def places(pos, kw):
    """Where the call's tensors are: (list or dict, key, place in a tuple or None)."""
    for where, items in ((0, enumerate(pos)), (1, kw.items())):
        for key, v in items:
            for i, t in enumerate(v if isinstance(v, tuple) else (v,)):
                if isinstance(t, Stand):
                    yield where, key, i if isinstance(v, tuple) else None


def moved(pos, kw, at, device):
    out = [list(pos), dict(kw)]
    where, key, i = at
    v = out[where][key]
    old = v if i is None else v[i]
    new = Stand(old.dtype, *old.shape, device=device)
    out[where][key] = new if i is None else v[:i] + (new,) + v[i + 1:]
    return out


@pytest.mark.parametrize("gpus,device", [(2, -1), (2, 1), (1, -1)])
@pytest.mark.parametrize("which", sorted(calls()))
def test_each_tensor_is_on_the_current_gpu(dg, monkeypatch, which, gpus, device):  # noqa: F811
    monkeypatch.setattr(dg, "_gpus", gpus)
    name, pos, kw = calls()[which]
    with pytest.raises(Called):
        getattr(dg, name)(*pos, **kw)
    n = 0
    for at in places(pos, kw):
        p, k = moved(pos, kw, at, device)
        with pytest.raises(ValueError, match="GPU"):
            getattr(dg, name)(*p, **k)
        n += 1
    assert n >= 4


@pytest.mark.parametrize("which", sorted(calls()))
def test_the_tensors_gpu_is_the_current_one(dg, monkeypatch, which):  # noqa: F811
    name, pos, kw = calls()[which]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        getattr(dg, name)(*pos, **kw)


def test_shapes_are_checked(dg):  # noqa: F811
    a, b, x = nvf4(4, 256), nvf4(128, 256), Stand(F16, 4, 256)
    w = nvf4(128, 256, 3)
    for name, args in (
            ("gemm_nvf4", (*a, *nvf4(128, 192), Stand(F16, 4, 128))),
            ("gemm_nvf4", (*a, *b, Stand(F16, 4, 120))),
            ("gemm_nvf4", (*a, *w, Stand(F16, 4, 128))),
            ("gemm_nvf4", (a[0], nvf4(130, 256)[1], a[2], *b, Stand(F16, 4, 128))),
            ("gemm_nvf4_grouped", (*a, *w, Stand(I32, 3), Stand(F16, 4, 128))),
            ("dequantize_nvf4", (*a, Stand(F16, 4, 254))),
            ("quantize_nvf4", (Stand(F16, 2, 2, 2, 16),)),
            ("moe_layer", (x, Stand(I32, 4, 2), None, w, nvf4(256, 120, 3), x)),
            ("moe_layer", (x, Stand(I32, 3, 2), None, w, nvf4(256, 128, 3), x)),
            ("moe_layer", (x, Stand(I32, 4, 2), None, w, nvf4(248, 128, 3), x)),
            ("moe_layer", (x, Stand(I32, 4, 2), None, w, nvf4(256, 128, 2), x))):
        with pytest.raises(ValueError):
            getattr(dg, name)(*args)
    with pytest.raises(ValueError, match="activation"):
        dg.moe_layer(x, Stand(I32, 4, 2), None, w, nvf4(256, 128, 3), x, activation="relu")
