"""Every tensor of an FP8 or expert-routing call must be on the current GPU: a
host tensor, one of another GPU, and a call for a GPU that is not the current one
are refused before the library is called.  Stand-ins for tensors, no GPU."""

import pytest
import torch

F8, F16, F32, I32 = torch.float8_e4m3fn, torch.float16, torch.float32, torch.int32


class Stand:
    """A tensor's shape, type and device without its memory."""

    def __init__(self, dtype, *shape, device=0):
        self.t = torch.empty(shape, dtype=dtype, device="meta")
        self.dtype, self.shape, self.on = dtype, self.t.shape, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    @property
    def is_cuda(self):
        return self.on >= 0

    @property
    def device(self):
        return torch.device("cuda", self.on) if self.on >= 0 else torch.device("cpu")

    def get_device(self):
        return self.on

    def data_ptr(self):
        return 0x10000


class Called(Exception):
    pass


class Library:
    def __getattr__(self, name):
        def call(*args):
            raise Called(name)
        return call


@pytest.fixture
def dg(monkeypatch):
    import precision_matmul_dg_gb300 as m
    m._fp()
    monkeypatch.setattr(m, "lib", Library)
    monkeypatch.setattr(m, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(m, "_gpus", 2, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return m


def calls():
    """name -> (function's name, its tensors by position, its tensors by keyword, the rest)."""
    a, sa = Stand(F8, 4, 256), Stand(F32, 4, 2)
    b, sb = Stand(F8, 128, 256), Stand(F32, 1, 2)
    w, ws = Stand(F8, 3, 128, 256), Stand(F32, 3, 1, 2)
    off, ids = Stand(I32, 4), Stand(I32, 4, 2)
    x, d, rows = Stand(F16, 4, 256), Stand(F16, 4, 128), Stand(I32, 8)
    q, qs, y = Stand(F8, 8, 256), Stand(F32, 8, 2), Stand(F16, 8, 256)
    wt = Stand(F32, 4, 2)
    return {
        "quantize": ("quantize_fp8", [x], dict(out=(a, sa)), {}),
        "gemm": ("gemm_fp8", [a, sa, b, sb, d], dict(bias=Stand(F16, 128)), dict(epilogue="bias")),
        "grouped": ("gemm_fp8_grouped", [a, sa, w, ws, off, d], dict(bias=Stand(F16, 3, 128)),
                    dict(epilogue="bias")),
        "wgrad": ("gemm_fp8_grouped_wgrad", [a, sa, b, Stand(F32, 128, 2), off,
                                             Stand(F32, 3, 4, 128)], {}, {}),
        "sort": ("moe_sort", [ids, 3], dict(out=(off, rows, Stand(I32, 4, 2))), {}),
        "dispatch": ("moe_dispatch", [x, rows, 2, y], {}, {}),
        "dispatch_fp8": ("moe_dispatch_fp8", [x, rows, 2, q, qs], {}, {}),
        "combine": ("moe_combine", [y, ids, x], dict(weights=wt), {}),
        "backward": ("moe_combine_backward", [x, y, ids, rows, wt, Stand(F16, 8, 256),
                                              Stand(F32, 4, 2)], {}, {}),
    }


def moved(pos, kw, k, device):
    """The k-th tensor of the call on another device; None past the last."""
    flat = list(pos) + [t for v in kw.values() for t in (v if isinstance(v, tuple) else (v,))]
    at = [i for i, t in enumerate(flat) if isinstance(t, Stand)]
    if k >= len(at):
        return None
    old = flat[at[k]]
    flat[at[k]] = Stand(old.dtype, *old.shape, device=device)
    pos, rest, out = flat[:len(pos)], flat[len(pos):], {}
    for name, v in kw.items():
        n = len(v) if isinstance(v, tuple) else 1
        out[name], rest = tuple(rest[:n]) if isinstance(v, tuple) else rest[0], rest[n:]
    return pos, out


@pytest.mark.parametrize("device", [-1, 1])
@pytest.mark.parametrize("which", sorted(calls()))
def test_each_tensor_is_on_the_current_gpu(dg, which, device):
    name, pos, kw, rest = calls()[which]
    with pytest.raises(Called):
        getattr(dg, name)(*pos, **kw, **rest)
    k = 0
    while (m := moved(pos, kw, k, device)) is not None:
        with pytest.raises(ValueError):
            getattr(dg, name)(*m[0], **m[1], **rest)
        k += 1
    assert k >= 4 or which in ("quantize", "dispatch")


@pytest.mark.parametrize("which", sorted(calls()))
def test_the_tensors_gpu_is_the_current_one(dg, monkeypatch, which):
    name, pos, kw, rest = calls()[which]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        getattr(dg, name)(*pos, **kw, **rest)


def test_optional_tensors_may_be_missing(dg):
    for name, args in (("moe_combine", (Stand(F16, 8, 256), Stand(I32, 4, 2), Stand(F16, 4, 256))),
                       ("moe_combine_backward", (Stand(F16, 4, 256), None, Stand(I32, 4, 2),
                                                 Stand(I32, 8), None, Stand(F16, 8, 256)))):
        with pytest.raises(Called):
            getattr(dg, name)(*args)


@pytest.mark.parametrize("gpus", [0, 1])
@pytest.mark.parametrize("which", sorted(calls()))
def test_host_tensors(dg, monkeypatch, which, gpus):
    # refused one by one with one GPU, where no device is compared, and all
    # together with none, without asking for one
    name, pos, kw, rest = calls()[which]

    def none():
        raise RuntimeError("no GPU")
    monkeypatch.setattr(dg, "_gpus", gpus)
    monkeypatch.setattr(torch.cuda, "current_device", none)

    def host(v):
        if isinstance(v, tuple):
            return tuple(map(host, v))
        return Stand(v.dtype, *v.shape, device=-1) if isinstance(v, Stand) else v
    with pytest.raises(ValueError, match="on the GPU"):
        getattr(dg, name)(*map(host, pos), **{k: host(v) for k, v in kw.items()}, **rest)
    k = 0
    while gpus == 1 and (m := moved(pos, kw, k, -1)) is not None:
        with pytest.raises(ValueError, match="on the GPU"):
            getattr(dg, name)(*m[0], **m[1], **rest)
        k += 1
