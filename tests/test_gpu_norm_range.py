"""gdn_group_norm over the whole range of x, and in calls of more groups than one launch takes.

Tolerances as in test_gpu_group_norm: 40 x 2^-24 of |n w| (plus the mean's share, centred); rows are
scaled by powers of two where their squares leave the fp32 range, which rounds nothing."""

import pytest

from tests.gpu_helpers import announce
from tests.test_gpu_group_norm import check, formula, make, run

pytestmark = pytest.mark.gpu


# (centred, a group of one is x - x)
@pytest.mark.parametrize("size,centered", [(s, c) for s in (1, 7, 100, 128, 512, 2048, 2049, 10001) for c in (False, True)
                                           if s > 1 or not c])
@pytest.mark.parametrize("power", [-120, -80, -64, 60, 63, 100, 124])
def test_rows_of_any_magnitude(size, centered, power):
    """Values around 2^power: eps is 0, so n is of size 1 throughout."""
    announce(f"norm: 2^{power}, size {size}, centered {centered}")
    o = dict(groups=3, size=size, silu=False, eps=0.0, centered=centered, bias=True)
    x, gate, w, b, y = make(o, 4, seed=size)
    x.copy_(x.sign() * x.abs().clamp(0.05, 4.0))
    x[1:] *= 2.0 ** power  # (row 0 beside them, of size 1)
    run(o, x, gate, w, b, y)
    check(o, x, gate, w, b, y)


@pytest.mark.parametrize("size", [100, 512, 2500])
def test_epsilon_beside_large_and_small_rows(size):
    """eps counts where it is not small beside the mean square, and only there."""
    announce(f"norm: eps, size {size}")
    for eps, power in ((1e-5, 70), (1e-5, -60), (1e-30, -50), (1e-37, -62), (1e20, 35), (1e-5, -90)):
        for centered in (False, True):
            o = dict(groups=2, size=size, silu=False, eps=eps, centered=centered)
            x, gate, w, b, y = make(o, 3, seed=size)
            x *= 2.0 ** power
            run(o, x, gate, w, b, y)
            check(o, x, gate, w, b, y)


@pytest.mark.parametrize("size", [100, 2500])
def test_groups_of_zeros(size):
    """0 / sqrt(0 + eps): 0, and NaN for eps 0. Their neighbours are as without them."""
    import torch

    announce(f"norm: zero groups, size {size}")
    for eps in (0.0, 1e-6, 1e-40):
        for centered in (False, True):
            o = dict(groups=2, size=size, silu=False, eps=eps, centered=centered)
            x, gate, w, b, y = make(o, 5, seed=1)
            x[2, size:] = 0.0
            run(o, x, gate, w, b, y)
            assert (torch.isnan(y[2, size:]) if eps == 0 else y[2, size:] == 0).all()
            y[2, size:] = 0.0
            want, scale = formula(o, x, gate, w, b)
            want[2, size:] = 0.0
            scale[2, size:] = 0.0
            assert ((y.double() - want).abs() <= 40 * 2.0 ** -24 * scale + 1e-38).all()


@pytest.mark.parametrize("size", [128, 2500])
def test_gate_first_of_large_products(size):
    announce(f"norm: gate first, size {size}")
    o = dict(groups=2, size=size, silu=False, eps=1e-5, first=True, gate="f32")
    x, gate, w, b, y = make(o, 3, seed=2)
    x *= 2.0 ** 70
    run(o, x, gate, w, b, y)
    check(o, x, gate, w, b, y)


@pytest.mark.parametrize("groups,size,rows,pad", [(3, 2, (1 << 23) // 3 + 5, 3), (1, 1, (1 << 23) + 3, 1), (4096, 2, 2050, 7),
                                                  ((1 << 23) + 1, 1, 2, 0), (1 << 23, 2, 2, 5)])
def test_more_groups_than_a_launch_takes(groups, size, rows, pad):
    """A call of more than 2^23 groups goes in pieces of rows; so does a row of as many by itself."""
    announce(f"norm: {rows} x {groups} groups of {size}")
    o = dict(groups=groups, size=size, gate="bf16", y="f32")
    t = make(o, rows, seed=3, pad=pad)
    t[4].fill_(7.0)
    run(o, *t)
    for a in range(0, rows, 1 << 21):
        part = slice(a, min(rows, a + (1 << 21)))
        check(o, t[0][part], t[1][part], t[2], None, t[4][part])
