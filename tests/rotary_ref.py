"""Rotary positions in float64 for the tests: every pair of channels as a complex number, turned by its angle."""
import numpy as np
import torch


def angles(rotary, positions):
    """[T, pairs] in float64, reduced within a turn: positions [axes, T] (int), the product formed in extended precision."""
    pairs = rotary.rot_dim // 2
    freq = np.array(rotary.freq[:pairs], dtype=np.longdouble)
    axis = np.array(rotary.axis[:pairs])
    pos = positions.cpu().numpy().astype(np.longdouble)[axis].T  # [T, pairs]
    a = pos * freq
    turn = 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))
    return torch.from_numpy((a - np.rint(a / turn) * turn).astype(np.float64))


def split(x, rotary):
    """The two channels of every pair of x [..., d]: a, b [..., pairs]."""
    r = rotary.rot_dim
    return (x[..., 0:r:2], x[..., 1:r:2]) if rotary.adjacent else (x[..., :r // 2], x[..., r // 2:r])


def turned(x, rotary, positions, inverse=False):
    """x [T, heads, d] turned, in float64."""
    x = x.detach().double().cpu()
    t = angles(rotary, positions)[:, None] * (-1 if inverse else 1)
    a, b = split(x, rotary)
    z = torch.complex(a, b) * torch.polar(torch.ones_like(t), t)
    y = x.clone()
    ya, yb = split(y, rotary)
    ya.copy_(z.real)
    yb.copy_(z.imag)
    return y


def size(x, rotary):
    """|a| + |b| of every value's pair (0 past rot_dim): what an error of the sine and cosine is multiplied by."""
    x = x.detach().double().cpu().abs()
    s = torch.zeros_like(x)
    a, b = split(x, rotary)
    sa, sb = split(s, rotary)
    sa.copy_(a + b)
    sb.copy_(a + b)
    return s


def places(lens, new):
    """[1, sum(new)]: the places of every sequence's new tokens."""
    return torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)] or [torch.zeros(0, dtype=torch.int64)])[None]
