"""A mixture-of-experts layer in 8-bit floating point on libdg.

    python examples/fp8_experts.py [--tokens 4096] [--experts 64] [--top-k 8]
                                   [--width 2048] [--hidden 4096]

forward(): tokens sorted by expert and quantized on the way, the experts' two
products (the first with GELU), and the way back with the routing weights.
training_step(): forward and backward of one linear layer per expert: the
gradients of the tokens, the weights and the routing weights.  The program
runs both, compares them with plain FP32 torch and prints times.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import precision_matmul_dg_gb300 as dg  # noqa: E402


def quantize_weights(W, form="rows"):
    """W [experts, N, K] as FP8 with 128 x 128 blocks: codes [experts, N, K] and
    scales, or ("transposed") those of each expert's transpose."""
    parts = [dg.quantize_fp8(w, form=form, block_rows=128) for w in W]
    return torch.stack([p[0].view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn), \
        torch.stack([p[1] for p in parts])


def forward(x, ids, weights, up, down):
    """x [tokens, width] -> [tokens, width]; ids, weights [tokens, top_k]; up and
    down: (codes, scales) of quantize_weights ([experts, hidden, width] and
    [experts, width, hidden])."""
    experts, hidden = up[0].shape[:2]
    tokens, width = x.shape
    top_k = ids.shape[1]
    offsets, row_slot, slot_row = dg.moe_sort(ids, experts)
    rows = row_slot.shape[0]
    codes = torch.empty(rows, width, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty(rows, -(-width // 128), device=x.device)
    dg.moe_dispatch_fp8(x, row_slot, top_k, codes, scales)
    # rows past the last segment (dropped choices) are not written by the product
    h = torch.zeros(rows, hidden, dtype=x.dtype, device=x.device)
    dg.gemm_fp8_grouped(codes, scales, *up, offsets, h, epilogue="gelu")
    y = torch.zeros(rows, width, dtype=x.dtype, device=x.device)
    dg.gemm_fp8_grouped(*dg.quantize_fp8(h), *down, offsets, y)
    return dg.moe_combine(y, slot_row, torch.empty_like(x), weights=weights)


def training_step(x, ids, weights, W, dy):
    """y = sum over j of weights[t, j] * W[ids[t, j]] x[t], and the gradients of
    sum(y * dy): returns y, dx, dW (float32), dweights."""
    experts, n, k = W.shape
    top_k = ids.shape[1]

    def empty(*shape, dtype=x.dtype):
        return torch.empty(shape, dtype=dtype, device=x.device)
    offsets, row_slot, slot_row = dg.moe_sort(ids, experts, align=128)
    rows = row_slot.shape[0]
    xs = dg.moe_dispatch(x, row_slot, top_k, empty(rows, k))
    codes, scales, codes_t, scales_t = dg.quantize_fp8(xs, form="both")
    ys = torch.zeros(rows, n, dtype=x.dtype, device=x.device)
    dg.gemm_fp8_grouped(codes, scales, *quantize_weights(W), offsets, ys)
    y = dg.moe_combine(ys, slot_row, empty(x.shape[0], n), weights=weights)

    dys, dweights = dg.moe_combine_backward(dy, ys, slot_row, row_slot, weights, empty(rows, n),
                                            empty(*ids.shape, dtype=torch.float32))
    g, gs, g_t, gs_t = dg.quantize_fp8(dys, form="both")
    dxs = torch.zeros(rows, k, dtype=x.dtype, device=x.device)
    dg.gemm_fp8_grouped(g, gs, *quantize_weights(W, "transposed"), offsets, dxs)
    dx = dg.moe_combine(dxs, slot_row, empty(*x.shape))
    dW = dg.gemm_fp8_grouped_wgrad(g_t, gs_t, codes_t, scales_t, offsets,
                                   empty(experts, n, k, dtype=torch.float32))
    return y, dx, dW, dweights


def routing(tokens, experts, top_k, seed=0):
    """Each token's experts and softmax weights from random scores."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    score, ids = torch.randn(tokens, experts, generator=g, device="cuda").topk(top_k, dim=1)
    return ids.to(torch.int32).contiguous(), torch.softmax(score, 1).contiguous()


def plain_forward(x, ids, weights, up, down):
    """forward() in FP32 torch on unquantized weights, expert by expert."""
    y = torch.zeros(x.shape, device=x.device)
    for e in range(up.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = torch.nn.functional.gelu(x[t].float() @ up[e].float().t())
        y.index_add_(0, t, weights[t, j][:, None] * (h @ down[e].float().t()))
    return y


def time_us(f, reps=20):
    f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    for _ in range(reps):
        f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / reps * 1e3


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("experts", 64), ("top-k", 8), ("width", 2048),
                        ("hidden", 4096)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=g, device="cuda")).bfloat16()
    x = normal(a.tokens, a.width)
    W_up = normal(a.experts, a.hidden, a.width, std=a.width ** -0.5)
    W_down = normal(a.experts, a.width, a.hidden, std=a.hidden ** -0.5)
    ids, weights = routing(a.tokens, a.experts, a.top_k)
    up, down = quantize_weights(W_up), quantize_weights(W_down)
    y = forward(x, ids, weights, up, down).float()
    want = plain_forward(x, ids, weights, W_up, W_down)
    print("forward: relative difference from FP32 %.3f, %.0f us" % (
        (y - want).norm() / want.norm(), time_us(lambda: forward(x, ids, weights, up, down))))
    dy = normal(a.tokens, a.hidden, std=1e-3)
    _, dx, dW, dweights = training_step(x, ids, weights, W_up, dy)
    print("training step: |dx| %.4g, |dW| %.4g, |dweights| %.4g, %.0f us" % (
        dx.float().norm(), dW.norm(), dweights.norm(),
        time_us(lambda: training_step(x, ids, weights, W_up, dy), 3)))
    dg.check_status()


if __name__ == "__main__":
    main()
