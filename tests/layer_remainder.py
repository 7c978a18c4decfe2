"""An expert layer whose results are differences of hidden values that agree in their first
11 bits, so that they show what the second FP16 value of h (include/dg.h: 22 bits) holds.

x[t] = (a size, nine small powers of two in an order of t's own); W1's row i takes the size 1, 2
or 4 times (by i's group of 32) and some of the small ones; W2's row n is hidden value n less
another of its group.  h = 64 to 1024 and multiples of 2^-9 behind it: exact in FP32, and in two
FP16 values, where one is off by up to 2^-5 to 2^-2.  Numpy only.
"""

import numpy as np

SMALL = 9


class Layer:
    """x [tokens, width], ids [tokens, 1], codes' values up and down (also what they stand
    for: all scales are 1), the hidden values' partners, and the 64-bit result."""

    def __init__(self, tokens=7, count=2, hidden=1152, gated=False, seed=0):
        rng = np.random.default_rng(seed)
        self.gated, self.hidden = gated, hidden
        width = 16
        # (gated: h = silu(32) * value, where silu(32) is 32 to 13 digits)
        unit = 1 / 32 if gated else 1.0
        self.x = np.zeros((tokens, width))
        self.x[:, 0] = 64.0 * unit * 2.0 ** rng.integers(0, 3, tokens)
        for t in range(tokens):
            self.x[t, 1:1 + SMALL] = unit * 2.0 ** -(1.0 + rng.permutation(SMALL))
        self.x[:, 15] = 32.0
        self.ids = (np.arange(tokens) % 6 == 5).astype(np.int32)[:, None] % count
        value = np.zeros((count, hidden, width))
        value[..., 0] = 2.0 ** (np.arange(hidden) // 32 % 3)
        value[..., 1:1 + SMALL] = rng.integers(0, 2, (count, hidden, SMALL))
        gate = np.zeros_like(value)
        gate[..., 15] = 1.0
        self.up = np.concatenate([gate, value], 1) if gated else value
        n = np.arange(hidden)
        self.partner = n // 32 * 32 + (n % 32 * 5 + 7) % 32
        self.down = np.zeros((count, hidden, hidden))
        self.down[:, n, n], self.down[:, n, self.partner] = 1.0, -1.0

    def h(self, t):
        """The hidden values of token t in 64 bits (GELU and SiLU of 32 and more are their
        arguments)."""
        v = self.up[self.ids[t, 0], -self.hidden:] @ self.x[t]
        return 32.0 * v if self.gated else v

    def held(self, mistake=None):
        """h [tokens, hidden] as the kernels hold it, or with a mistake: "bits" (the second
        value lost), "slot" (another token's second values), "power" (the second values with
        the power of the group before)."""
        hi, rest, power = [], [], []
        for t in range(len(self.x)):
            g = self.h(t).reshape(-1, 32)
            f = 2.0 ** (14 - np.floor(np.log2(np.abs(g).max(1, keepdims=True))))
            a = (g * f).astype(np.float16).astype(np.float64)
            b = (g * f - a).astype(np.float16).astype(np.float64)
            hi.append(a), rest.append(b), power.append(1 / f)
        hi, rest, power = np.array(hi), np.array(rest), np.array(power)
        if mistake == "bits":
            rest = 0 * rest
        elif mistake == "slot":
            rest = np.roll(rest, 1, 0)
        of_rest = np.roll(power, 1, 1) if mistake == "power" else power
        return (hi * power + rest * of_rest).reshape(len(self.x), -1)

    def results(self, held):
        return held - held[:, self.partner]
