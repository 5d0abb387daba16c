"""Refusals of the norm calls through the C ABI, without a GPU (nothing is launched)."""
import ctypes

import pytest

from causal_video_diffusion_b200 import binding as B

P = 0x100000


@pytest.fixture(scope="module")
def L():
    from causal_video_diffusion_b200 import build
    build.build()
    return B.lib()


def norm(**kw):
    n = B.unstep_norm_t()
    n.kind, n.eps, n.param_type = B.UNSTEP_NORM_LAYER, 1e-6, B.UNSTEP_F32
    for k, v in kw.items():
        setattr(n, k, v)
    return n


def modulate(L, x=P, x_type=0, ldx=64, y=2 * P, ldy=64, rows=4, C=64, per=2, n=None):
    return L.unstep_norm_modulate(x, x_type, ldx, y, ldy, rows, C, per,
                                  ctypes.byref(n if n is not None else norm()), None)


def gated(L, x=P, x_type=0, ldx=64, y=2 * P, ldy=64, gate=None, gate_type=0, gs=0, s=1.0,
          post=None, nxt=True, xo=3 * P, ldxo=64, h=4 * P, ldh=64, rows=4, C=64, per=2):
    n = norm() if nxt is True else nxt
    return L.unstep_gate_residual_norm(
        x, x_type, ldx, y, ldy, gate, gate_type, gs, s, None if post is None else ctypes.byref(post),
        None if n is None else ctypes.byref(n), xo, ldxo, h, ldh, rows, C, per, None)


ARG, SHAPE, ALIGN, UNSUP = (B.UNSTEP_ERR_ARG, B.UNSTEP_ERR_SHAPE, B.UNSTEP_ERR_ALIGN,
                            B.UNSTEP_ERR_UNSUPPORTED)
BOTH = [(dict(x=None), ARG), (dict(y=None), ARG), (dict(x_type=2), ARG), (dict(x=P + 8), ALIGN),
        (dict(y=P + 2), ALIGN), (dict(ldx=60), SHAPE), (dict(ldx=56), SHAPE), (dict(ldy=56), SHAPE),
        (dict(rows=-1), SHAPE), (dict(C=0), SHAPE), (dict(C=12), SHAPE), (dict(per=0), SHAPE),
        (dict(C=16392, ldx=16392, ldy=16392, ldxo=16392, ldh=16392), UNSUP)]
NORMS = [(dict(kind=2), ARG), (dict(kind=-1), ARG), (dict(eps=-1e-6), ARG),
         (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(param_type=7), ARG),
         (dict(weight=P + 4), ALIGN), (dict(bias=P + 8), ALIGN), (dict(scale=P + 4), ALIGN),
         (dict(shift=P + 2), ALIGN), (dict(scale=P, mod_stride=-64), SHAPE),
         (dict(shift=P, mod_stride=68), SHAPE)]


def test_norm_modulate_refusals(L):
    for kw, want in BOTH:
        kw = {k: v for k, v in kw.items() if k not in ("ldxo", "ldh")}
        assert modulate(L, **kw) == want, kw
    for kw, want in NORMS:
        assert modulate(L, n=norm(**kw)) == want, kw
    assert L.unstep_norm_modulate(P, 0, 64, P, 64, 4, 64, 2, None, None) == ARG
    assert modulate(L, y=P, x_type=1) == ARG                      # fp32 rows cannot be overwritten
    assert modulate(L, y=P, ldy=128) == ARG
    assert modulate(L, rows=0, x=None, y=None) == B.UNSTEP_OK
    assert modulate(L, rows=0, n=norm(kind=9)) == ARG


def test_gate_residual_norm_refusals(L):
    for kw, want in BOTH:
        assert gated(L, **kw) == want, kw
    for kw, want in NORMS:
        assert gated(L, nxt=norm(**kw)) == want, kw
        assert gated(L, post=norm(**kw)) == want, kw
    for kw, want in [(dict(xo=None), ARG), (dict(xo=3 * P + 4), ALIGN), (dict(h=4 * P + 8), ALIGN),
                     (dict(gate=P + 4), ALIGN), (dict(gate=P, gs=4), SHAPE),
                     (dict(gate=P, gs=-8), SHAPE), (dict(gate_type=3), ARG),
                     (dict(s=float("nan")), ARG), (dict(s=float("inf")), ARG),
                     (dict(ldxo=56), SHAPE), (dict(ldh=56), SHAPE),
                     (dict(h=None), ARG), (dict(nxt=None), ARG), (dict(xo=P, ldxo=128), ARG),
                     (dict(h=P), ARG), (dict(h=2 * P), ARG), (dict(h=3 * P), ARG),
                     (dict(xo=2 * P), ARG)]:
        assert gated(L, **kw) == want, kw
    assert gated(L, rows=0, x=None, y=None, xo=None) == B.UNSTEP_OK
