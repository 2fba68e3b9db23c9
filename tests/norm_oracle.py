"""Plain implementation (64 bits, CPU) of the root-mean-square norm, and how far fp32 arithmetic may be from it."""
import torch

# fp32 sums of up to 32768 squares: a thread adds at most 64 of them one by one, 10 steps join the threads, so the sum is
# off by at most 74 * 2^-24 of itself (all terms are positive) and 1 / sqrt of it by half of that; rsqrt by 2 units, the
# mean, eps, gain (two) and product by one rounding each: (37 + 4 + 5) * 2^-24 < 2^-18.
REL = 2.0 ** -18


def stream(x, residual):
    """s as it is stored: one rounding of the exact sum (fp32 holds the sum of two bf16 up to a rounding that does not
    change the second; the sum of bf16 and fp32 is rounded once)."""
    return x if residual is None else (x.float() + residual.float()).to(residual.dtype)


def norm(s, weight, eps, offset=0.0):
    s = s.double()
    y = s / (s.square().mean(-1, keepdim=True) + eps).sqrt()
    return y if weight is None else y * (weight.double() + offset)
