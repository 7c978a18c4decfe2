"""The example's mixture-of-experts layer in FP8, forward and backward, against
64-bit arithmetic on unquantized values: what differs is the quantization
(at most 2^-4 of each value, errors of many values added in quadrature)."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import fp8_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    spec = importlib.util.spec_from_file_location(
        "fp8_experts", os.path.join(ROOT, "examples", "fp8_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def inputs(tokens, experts, top_k, n, k, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, k, generator=g).bfloat16()
    W = (torch.randn(experts, n, k, generator=g) / k ** 0.5).bfloat16()
    ids = torch.stack([torch.randperm(experts, generator=g)[:top_k] for _ in range(tokens)]).int()
    ids[0] = -1
    if tokens > 3:
        ids[3, 0] = experts
    w = torch.softmax(torch.randn(tokens, top_k, generator=g), 1)
    return x, W, ids, w


def rel(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


# A code's error is uniform within half a step, at most 2^-4 of its value: in
# the root mean square at most 2^-4 / sqrt(3).  A product's two operands add
# theirs in quadrature; a chain of two products through GELU, whose slope is at
# most 1.13, adds the second's to 1.13 times the first's.  (BF16 roundings, 2^-9,
# are below 2% of that.)
ONE = 1.02 * 2.0 ** -4 * (2 / 3) ** 0.5
TWO = ONE * (1 + 1.13 ** 2) ** 0.5


@pytest.mark.parametrize("tokens", [5, 200])
def test_forward(layer, tokens):
    experts, top_k, hidden, width = 6, 2, 384, 256
    x, W_up, ids, w = inputs(tokens, experts, top_k, hidden, width, 1)
    W_down = (torch.randn(experts, width, hidden, generator=torch.Generator().manual_seed(2)) /
              hidden ** 0.5).bfloat16()
    y = layer.forward(x.cuda(), ids.cuda(), w.cuda(), layer.quantize_weights(W_up.cuda()),
                      layer.quantize_weights(W_down.cuda()))
    want = np.zeros((tokens, width))
    for t in range(tokens):
        for j in range(top_k):
            e = int(ids[t, j])
            if 0 <= e < experts:
                h = ref.gelu(W_up[e].double().numpy() @ x[t].double().numpy())
                want[t] += float(w[t, j]) * (W_down[e].double().numpy() @ h)
    got = y.double().cpu().numpy()
    assert (got[0] == 0.0).all()
    assert rel(got, want) < TWO


def test_training_step(layer):
    tokens, experts, top_k, n, k = 300, 5, 2, 256, 384
    x, W, ids, w = inputs(tokens, experts, top_k, n, k, 3)
    dy = (1e-3 * torch.randn(tokens, n, generator=torch.Generator().manual_seed(4))).bfloat16()
    y, dx, dW, dw = layer.training_step(x.cuda(), ids.cuda(), w.cuda(), W.cuda(), dy.cuda())
    x64, W64, w64, dy64 = (v.double().requires_grad_(v is not dy) for v in (x, W, w, dy))
    keep = (ids >= 0) & (ids < experts)
    rows = torch.einsum("tjnk,tk->tjn", W64[ids.clamp(0, experts - 1).long()], x64)
    want = (rows * (w64 * keep)[..., None]).sum(1)
    (want * dy64).sum().backward()
    for got, wanted, bound in ((y, want, ONE), (dx, x64.grad, ONE), (dW, W64.grad, ONE),
                               (dw, w64.grad, ONE)):
        assert rel(got.double().cpu().numpy(), wanted.detach().numpy()) < bound
    assert (dx[0] == 0).all() and (dw[0] == 0).all()


def test_forward_in_a_graph(layer):
    # the whole layer under CUDA-graph capture, replayed on new values
    x, W, ids, w = (v.cuda() for v in inputs(64, 8, 2, 256, 256, 5))
    up, down = layer.quantize_weights(W), layer.quantize_weights(W.transpose(1, 2).contiguous())
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer.forward(x, ids, w, up, down)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = layer.forward(x, ids, w, up, down)
    x2, _, ids2, w2 = inputs(64, 8, 2, 256, 256, 6)
    for a, b in ((x, x2), (ids, ids2), (w, w2)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, layer.forward(x, ids, w, up, down))
