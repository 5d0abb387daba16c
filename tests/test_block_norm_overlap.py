"""Outputs of the norm calls that lie across an input, a parameter or each other, through the C ABI:
refused before a launch; what shares no byte is not."""
import random

import pytest
import torch

from causal_video_diffusion_b200 import binding as B
from tests.test_block_norm import ARG, L, P, gated, modulate, norm  # noqa: F401 (L: a fixture)

# a call that passes its checks is launched: only where that cannot reach a device
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on made-up addresses")
C, ROWS = 64, 4


def test_shifted_rows_are_refused(L):  # noqa: F811
    row = 2 * C
    for d in (row, -row, 16, -16, 3 * row, -3 * row, 4 * row - 16, -(4 * row - 16)):
        assert modulate(L, y=P + d) == ARG, d
        assert gated(L, xo=P + d, h=8 * P) == ARG, d                 # over x
        assert gated(L, xo=2 * P + d, h=8 * P) == ARG, d             # over y
        assert gated(L, h=P + d) == ARG and gated(L, h=2 * P + d) == ARG and gated(L, h=3 * P + d) == ARG
    # fp32 rows are twice as long
    assert modulate(L, x_type=1, y=P + 4 * C * ROWS - 16) == ARG
    assert gated(L, x_type=1, xo=P + 4 * C * ROWS - 16, h=8 * P) == ARG
    assert gated(L, x_type=1, h=P + 4 * C * ROWS - 16) == ARG
    # rows that meet only behind the first of both: strides 2 C and 3 C, 6 C apart
    assert modulate(L, y=P + 2 * C, ldx=2 * C, ldy=3 * C) == ARG
    assert modulate(L, y=P + 4 * C * 2 - 16, ldx=2 * C, ldy=3 * C, rows=3) == ARG


def test_outputs_over_parameters_are_refused(L):  # noqa: F811
    last = 2 * P + 2 * C * ROWS - 16                                   # within y's last row
    for field in ("weight", "bias", "scale", "shift"):
        for at in (2 * P, last, 2 * P - 4 * C + 16):
            assert modulate(L, n=norm(**{field: at, "mod_stride": C})) == ARG, (field, at)
            at += P                                                    # x_out, then h
            assert gated(L, nxt=norm(**{field: at, "mod_stride": C})) == ARG, (field, at)
            assert gated(L, post=norm(**{field: at + P, "mod_stride": C})) == ARG, (field, at)
    # the second group's row alone
    assert modulate(L, n=norm(scale=2 * P - 4 * 1024, mod_stride=1024)) == ARG
    assert gated(L, gate=3 * P - 2 * 1024, gs=1024) == ARG
    assert gated(L, gate=4 * P, gs=0) == ARG


@no_device
def test_what_shares_no_byte_is_not_refused(L):  # noqa: F811
    gone = B.UNSTEP_ERR_CUDA
    assert modulate(L, y=P) == gone                                    # x itself
    assert modulate(L, y=P + 2 * C * ROWS) == gone and modulate(L, y=P - 2 * C * ROWS) == gone
    for d in (2 * C, 4 * C, -2 * C, 16 * C):                           # column blocks of a wider tensor
        assert modulate(L, ldx=3 * C, ldy=3 * C, y=P + d) == gone
    assert modulate(L, ldx=2 * C, ldy=4 * C, y=P + 2 * C) == gone      # between rows, other strides
    assert gated(L, xo=P) == gone
    assert gated(L, ldx=4 * C, ldy=4 * C, ldxo=4 * C, ldh=4 * C, y=P + 2 * C, xo=P + 4 * C,
                 h=P + 6 * C) == gone
    assert modulate(L, n=norm(scale=2 * P - 4 * 1024 - 4 * C, mod_stride=1024)) == gone
    # one group (rows_per_group above the rows): what would be the second's row is not there
    assert modulate(L, n=norm(scale=2 * P - 4 * 1024, mod_stride=1024), per=4) == gone


@no_device
def test_against_the_bytes_themselves(L):  # noqa: F811
    rng = random.Random(11)
    seen = set()
    for _ in range(3000):
        rows = rng.randint(1, 7)
        lds = [8 * rng.randint(1, 12) for _ in range(2)]
        if rng.random() < 0.4:
            lds[1] = lds[0]
        c = 8 * rng.randint(1, min(lds) // 8)
        x_type = rng.randint(0, 1)
        w = (4 if x_type else 2, 2)
        d = 16 * rng.randint(-60, 60)
        span = [set() for _ in range(2)]
        for i, at in enumerate((0, d)):
            for r in range(rows):
                span[i].update(range(at + r * lds[i] * w[i], at + (r * lds[i] + c) * w[i]))
        got = modulate(L, x_type=x_type, ldx=lds[0], ldy=lds[1], y=P + d, rows=rows, C=c, per=rows)
        whole = d == 0 and not x_type and lds[0] == lds[1]
        want = ARG if span[0] & span[1] and not whole else B.UNSTEP_ERR_CUDA
        assert got == want, (rows, lds, c, x_type, d)
        seen.add((want, lds[0] == lds[1]))
    assert len(seen) == 4
