"""An expert layer on NVF4 weights by both ways: many tokens through the sort, the
quantizing gather, the grouped products and the way back, each step against the
oracle on what the step before it gave; a few through the layer kernels; and the
example's program for both."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import fp8_ref, nvf4_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    spec = importlib.util.spec_from_file_location(
        "nvf4_experts", os.path.join(ROOT, "examples", "nvf4_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def inputs(tokens, experts, top_k, width, hidden, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, width, generator=g).bfloat16()
    up = (torch.randn(experts, hidden, width, generator=g) / width ** 0.5).bfloat16()
    down = (torch.randn(experts, width, hidden, generator=g) / hidden ** 0.5).bfloat16()
    ids = torch.stack([torch.randperm(experts, generator=g)[:top_k] for _ in range(tokens)]).int()
    ids[0] = -1
    if tokens > 3:
        ids[3, 0] = experts
    w = torch.softmax(torch.randn(tokens, top_k, generator=g), 1)
    return x, up, down, ids, w


def values(q, e):
    rows, width = q[0].shape[1:]
    codes = ref.unpack(q[0][e].cpu().numpy(), 2 * width)
    t = q[1][e].view(torch.uint8).cpu().numpy()
    groups = -(-2 * width // 16)
    r = np.arange(rows)
    s = np.stack([t[r // 128, g // 4, r % 32, 4 * (r % 128 // 32) + g % 4] for g in range(groups)], 1)
    return ref.values(codes, s, q[2][e].cpu().numpy())


def outside(got, want, err, dtype="bf16"):
    return ~(np.abs(got.double().cpu().numpy() - want) <= fp8_ref.rounded_bound(want, err, dtype))


def test_steps_of_a_prompt(layer):
    dg = layer.dg
    tokens, experts, top_k, width, hidden = 90, 5, 2, 256, 320
    x, up, down, ids, w = inputs(tokens, experts, top_k, width, hidden, 1)
    qu, qd = layer.quantize_weights(up.cuda()), layer.quantize_weights(down.cuda())
    offsets, row_slot, slot_row = dg.moe_sort(ids.cuda(), experts, align=128)
    rows = row_slot.shape[0]
    a = dg.moe_dispatch_nvf4(x.cuda(), row_slot, top_k, *dg.nvf4_buffers(rows, width))
    slots = row_slot.cpu().numpy()
    xs = fp8_ref.dispatch(x.double().numpy(), slots, top_k)
    codes, scales, r = ref.quantize(xs)
    assert np.array_equal(a[0].cpu().numpy(), ref.pack(codes))
    assert np.array_equal(a[1].view(torch.uint8).cpu().numpy(), ref.tiles(scales))
    h = torch.zeros(rows, hidden, dtype=torch.bfloat16, device="cuda")
    dg.gemm_nvf4_grouped(*a, *qu, offsets, h, epilogue="gelu")
    b = dg.quantize_nvf4(h)
    hq = ref.quantize(h.double().cpu().numpy())
    assert np.array_equal(b[0].cpu().numpy(), ref.pack(hq[0]))
    y = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    dg.gemm_nvf4_grouped(*b, *qd, offsets, y)
    d = dg.moe_combine(y, slot_row, torch.empty(tokens, width, dtype=torch.bfloat16, device="cuda"),
                       weights=w.cuda())
    dg.check_status()
    av, hv, ends = ref.values(codes, scales, r), ref.values(*hq), offsets.tolist()
    for e in range(experts):
        at = slice(ends[e], ends[e + 1])
        assert not outside(h[at], *ref.product(av[at], values(qu, e), use_gelu=True)).any()
        assert not outside(y[at], *ref.product(hv[at], values(qd, e))).any()
    want, mags = fp8_ref.combine(y.double().cpu().numpy(), slot_row.cpu().numpy(), w.numpy())
    assert not outside(d, want, mags * (top_k + 1) * 2.0 ** -23).any()


# A code's error is at most half of E2M1's widest step, 1 of 6, and uniform within
# it: in the root mean square 1 / (6 * 3^0.5) = 0.096 of the block's largest value
# (17/16 of that with its scale's rounding), which for 16 normal values is on
# average 2.1 of their deviation: 0.22 in all.  The chain has two products, each
# with one quantized operand, and GELU, whose slope is at most 1.13, between them.
# (The weights are the same on both sides.)
TWO = 0.22 * (1 + 1.13 ** 2) ** 0.5


@pytest.mark.parametrize("tokens", [6, 16])
def test_both_ways(layer, tokens):
    experts, top_k, width, hidden = 6, 2, 256, 384
    x, up, down, ids, w = inputs(tokens, experts, top_k, width, hidden, 2)
    qu, qd = layer.quantize_weights(up.cuda()), layer.quantize_weights(down.cuda())
    few = layer.decode(x.cuda(), ids.cuda(), w.cuda(), qu, qd).double().cpu().numpy()
    y, err = ref.layer(x.double().numpy(), ids.numpy(), w.numpy(),
                       np.stack([values(qu, e) for e in range(experts)]),
                       np.stack([values(qd, e) for e in range(experts)]))
    assert (np.abs(few - y) <= fp8_ref.rounded_bound(y, err, "bf16")).all()
    many = layer.prompt(x.cuda(), ids.cuda(), w.cuda(), qu, qd).double().cpu().numpy()
    assert (many[0] == 0).all() and (few[0] == 0).all()
    assert np.linalg.norm(many - y) / np.linalg.norm(y) < TWO
    fu, fd = layer.quantize_weights(up.cuda(), "fp8"), layer.quantize_weights(down.cuda(), "fp8")
    f8 = layer.decode(x.cuda(), ids.cuda(), w.cuda(), fu, fd).double().cpu().numpy()
    u, v = [np.stack([fp8_ref.values(q[0][e].view(torch.uint8).cpu().numpy(), q[1][e].cpu().numpy(), 128)
                      for e in range(experts)]) for q in (fu, fd)]
    y, err = ref.layer(x.double().numpy(), ids.numpy(), w.numpy(), u, v)
    assert (np.abs(f8 - y) <= fp8_ref.rounded_bound(y, err, "bf16")).all()


def test_prompt_in_a_graph(layer):
    x, up, down, ids, w = (v.cuda() for v in inputs(64, 8, 2, 256, 256, 3))
    qu, qd = layer.quantize_weights(up), layer.quantize_weights(down)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        layer.prompt(x, ids, w, qu, qd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = layer.prompt(x, ids, w, qu, qd)
    x2, _, _, ids2, w2 = inputs(64, 8, 2, 256, 256, 4)
    for a, b in ((x, x2), (ids, ids2), (w, w2)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, layer.prompt(x, ids, w, qu, qd))
