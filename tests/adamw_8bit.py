"""The 8-bit moments of the AdamW step in plain torch operations on the CPU,
one rounding an operation as the formula's: what the kernel has to store, code
for code."""
import numpy as np
import torch

NEAREST_BETA = 0.95
STEP, ELEMENT, HALF = 0x9E3779B9, 0x85EBCA6B, 0x80000000


def phases(t, first):
    """The phase of each of a block's 256 elements at step t, of 2^20; first:
    whether of the first moment."""
    i = torch.arange(256, dtype=torch.int64)
    return ((t * STEP % 2 ** 32 + i * ELEMENT + (HALF if first else 0)) % 2 ** 32 >> 12).to(torch.int32)


def either_code(y, phase):
    """One of the two e4m3 values around y, by phase / 2^20 of their spacing."""
    lift = torch.where(y.abs() < 2.0 ** -6, 2.0 ** -6, 0.0)
    z = ((y.abs() + lift).view(torch.int32) + phase) & ~0xFFFFF
    return torch.copysign(z.view(torch.float32) - lift, y)


def store(x, t, beta, first):
    """(codes as fp32 values, scales) of x [blocks, 256] after step t."""
    s = x.abs().amax(1, keepdim=True) * torch.tensor(1 / 448, dtype=torch.float32)
    y = torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0).clamp(-448, 448)
    if beta > NEAREST_BETA:
        y = either_code(y, phases(t, first))
    if not first:
        y = torch.where((x > 0) & (s > 0), y.clamp_min(2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn).float(), s


def moments(m, r, g, b1, b2):
    """The moments' new values (m, root) from the stored ones, fp32 [blocks, 256].
    The root is taken in 64 bits and rounded: torch's own in 32 is off by a
    unit in the last place on some processors."""
    f = lambda x: torch.tensor(np.float32(x))  # noqa: E731
    return m * f(b1) + g * f(1 - b1), (r * r * f(b2) + g * g * f(1 - b2)).double().sqrt().float()
