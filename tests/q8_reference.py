"""The 8-bit cache's number format and layer in 64 bits, from its definition in include/unstep.h
(nothing here is shared with the library)."""
from __future__ import annotations

import torch

from causal_video_diffusion_b200 import binding

BLOCK, E_MIN = 32, -111


def make_cache(shape, cap, max_pos_t, **kw) -> binding.LayerCacheQ8:
    return binding.LayerCacheQ8(shape.B, shape.H, shape.D, shape.Hg, shape.Wg, shape.d_t,
                                shape.d_h, shape.d_w, cap_frames=cap, max_pos_t=max_pos_t,
                                theta=shape.theta, **kw)


def exponents(x: torch.Tensor) -> torch.Tensor:
    """E of every 32-channel block of x (fp64, finite): smallest integer >= -111 with
    a <= 448 * 2^E."""
    a = x.unflatten(-1, (-1, BLOCK)).abs().amax(-1)
    m, e = torch.frexp(a / 448)                   # a / 448 = m 2^e, 1/2 <= m < 1: 2^(e-1) <= . < 2^e
    E = torch.where(m == 0.5, e - 1, e)
    return torch.where(a == 0, torch.full_like(E, E_MIN), E.clamp(min=E_MIN))


def step_of(x: torch.Tensor, E: torch.Tensor) -> torch.Tensor:
    """Spacing of the stored numbers around x under its block's exponent E."""
    s = torch.exp2(E.double()).repeat_interleave(BLOCK, -1)
    t = (x.abs() / s).clamp(min=2.0 ** -6)
    m, e = torch.frexp(t)
    return torch.exp2((e - 1).double() - 3) * s


def stored(x: torch.Tensor) -> torch.Tensor:
    """Values an 8-bit cache keeps of x (fp64, finite, below the top scale)."""
    step = step_of(x, exponents(x))
    return torch.round(x / step) * step


def values(codes: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """Codes under their scale bytes, in fp64 (byte 255: NaN)."""
    b = scale.view(torch.uint8).double()
    s = torch.where(b == 255, torch.full_like(b, float("nan")), torch.exp2(b - 127))
    return codes.double() * s.repeat_interleave(BLOCK, -1)


def angles(shape, first: int, frames: int, device) -> torch.Tensor:
    """[tokens][D/2] rotation angles of `frames` frames from `first` on."""
    def axis(pos, d):
        j = torch.arange(d // 2, dtype=torch.float64, device=device)
        return pos.double()[:, None] * torch.pow(torch.tensor(shape.theta, dtype=torch.float64,
                                                              device=device), -2 * j / max(d, 1))

    n = torch.arange(frames * shape.Tf, device=device)
    tok = n % shape.Tf
    return torch.cat([axis(first + n // shape.Tf, shape.d_t), axis(tok // shape.Wg, shape.d_h),
                      axis(tok % shape.Wg, shape.d_w)], 1)


def rotate(x: torch.Tensor, ang: torch.Tensor) -> torch.Tensor:
    """x [B][L][H][D] rotated, fp64."""
    a, b = x.double()[..., 0::2], x.double()[..., 1::2]
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def ring_rows(shape, cap: int, first: int, frames: int, device) -> torch.Tensor:
    f = torch.arange(first, first + frames, device=device) % cap
    return (f[:, None] * shape.Tf + torch.arange(shape.Tf, device=device)).reshape(-1)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
    """(out, bound) of attention in fp64: q [B][L][H][D], k and v [B][H][keys][D].

    The bound is the kernel's rounding, element by element, with A the attention of |v|:
    probabilities rounded to bf16 (2^-8 A), the exponentials (1e-4, once in P and once in the
    sum), fp32 accumulation of the scores (ds, in the exponent of P and of the sum) and of PV and
    the sum (one 2^-24 per term, at most 2^-11 A for 2^13 tiles' worth of adds), and the output's
    own rounding (2^-8 |out|)."""
    D, keys = q.shape[-1], k.shape[2]
    s = (q.double().transpose(1, 2) @ k.transpose(-1, -2)) / D ** 0.5
    top = (q.double().transpose(1, 2).abs() @ k.abs().transpose(-1, -2)).amax(-1, keepdim=True)
    ds = (D + 8) * 2.0 ** -24 * top / D ** 0.5
    p = torch.softmax(s, -1)
    out, A = p @ v, p @ v.abs()
    rel = 2.0 ** -8 + 2e-4 + 2 * ds + min(keys, 2 ** 13) * 2.0 ** -24
    bound = rel * A + 2.0 ** -8 * (1 + rel) * out.abs() + 1e-30
    return out.transpose(1, 2), bound.transpose(1, 2)
