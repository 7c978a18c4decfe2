"""A mixture-of-experts layer with 4-bit or 8-bit weights on libdg, for serving.

    python examples/nvf4_experts.py [--experts 64] [--top-k 8] [--width 2048]
                                    [--hidden 4096] [--prompt 4096] [--batch 8]

prompt(): many tokens, activations in 4 bits too: sorted by expert and quantized
on the way, the experts' two products (the first with GELU), and the way back
with the routing weights.  decode(): a few tokens, activations in 16 bits, the
whole layer in three kernels, on the same weights or on 8-bit ones.  The program
runs both, compares them with plain FP32 torch and prints times.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import precision_matmul_dg_gb300 as dg  # noqa: E402


def quantize_weights(W, form="nvf4"):
    """W [experts, N, K] as NVF4 (codes, scales, row scales) in one call, or as FP8
    with 128 x 128 blocks (codes, scales)."""
    if form == "nvf4":
        return dg.quantize_nvf4(W)
    parts = [dg.quantize_fp8(w, block_rows=128) for w in W]
    return torch.stack([p[0].view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn), \
        torch.stack([p[1] for p in parts])


def prompt(x, ids, weights, up, down):
    """x [tokens, width] -> [tokens, width]; ids, weights [tokens, top_k]; up and
    down: NVF4 stacks [experts, hidden, width] and [experts, width, hidden]."""
    experts, hidden = up[0].shape[:2]
    tokens, width = x.shape
    offsets, row_slot, slot_row = dg.moe_sort(ids, experts, align=128)
    rows = row_slot.shape[0]
    a = dg.moe_dispatch_nvf4(x, row_slot, ids.shape[1],
                             *dg.nvf4_buffers(rows, width, device=x.device))
    # rows past the last segment (dropped choices) are not written by the product
    h = torch.zeros(rows, hidden, dtype=x.dtype, device=x.device)
    dg.gemm_nvf4_grouped(*a, *up, offsets, h, epilogue="gelu")
    y = torch.zeros(rows, width, dtype=x.dtype, device=x.device)
    dg.gemm_nvf4_grouped(*dg.quantize_nvf4(h), *down, offsets, y)
    return dg.moe_combine(y, slot_row, torch.empty_like(x), weights=weights)


def decode(x, ids, weights, up, down):
    """The same for a few tokens; up and down NVF4 or FP8."""
    return dg.moe_layer(x, ids, weights, up, down, torch.empty_like(x))


def routing(tokens, experts, top_k, seed=0):
    """Each token's experts and softmax weights from random scores."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    score, ids = torch.randn(tokens, experts, generator=g, device="cuda").topk(top_k, dim=1)
    return ids.to(torch.int32).contiguous(), torch.softmax(score, 1).contiguous()


def plain(x, ids, weights, up, down):
    """The layer in FP32 torch on unquantized weights, expert by expert."""
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
    for name, value in (("experts", 64), ("top-k", 8), ("width", 2048), ("hidden", 4096),
                        ("prompt", 4096), ("batch", 8)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=g, device="cuda")).bfloat16()
    W_up = normal(a.experts, a.hidden, a.width, std=a.width ** -0.5)
    W_down = normal(a.experts, a.width, a.hidden, std=a.hidden ** -0.5)
    nvf4, fp8 = [[quantize_weights(W, form) for W in (W_up, W_down)] for form in ("nvf4", "fp8")]
    for name, f, tokens, of in (("prompt, NVF4", prompt, a.prompt, nvf4),
                                ("decode, NVF4", decode, a.batch, nvf4),
                                ("decode, FP8", decode, a.batch, fp8)):
        x = normal(tokens, a.width)
        ids, weights = routing(tokens, a.experts, a.top_k)
        y = f(x, ids, weights, *of).float()
        want = plain(x, ids, weights, W_up, W_down)
        print("%s: %d tokens, relative difference from FP32 %.3f, %.0f us" % (
            name, tokens, (y - want).norm() / want.norm(), time_us(lambda: f(x, ids, weights, *of))))
    dg.check_status()


if __name__ == "__main__":
    main()
