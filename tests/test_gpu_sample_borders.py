"""gdn_sample where the random number falls next to a border: rows made for it."""

import math

import numpy as np
import pytest

from tests.gpu_helpers import announce
from tests.test_gpu_sample import run

pytestmark = pytest.mark.gpu

F = np.float32


def nearest_below(w):
    """The largest fp32 x <= 0 with e^x <= w."""
    x = F(min(math.log(w), 0.0))
    while math.exp(float(x)) > w:
        x = np.nextafter(x, F(-np.inf))
    return x


def balanced_rows(first, short):
    """1026 logits: 512 of `first`; a second and third tile with one 0 whose weights sum to those of the first tile less `short`
    units of 2^-51, so that u = 1/2 falls between them."""
    w = math.exp(float(first))
    x = np.full(1026, first, F)
    x[512] = 0.0
    left = 3 * w - 1 - short * 2.0 ** -51  # what four tokens have to weigh: half of it, then as much as there is each time
    for i, share in ((1022, 0.5), (1023, 1.0), (1024, 1.0), (1025, 1.0)):
        x[i] = nearest_below(left * share)
        left -= math.exp(float(x[i]))
    return x


def test_a_number_at_the_end_of_a_tile_of_equal_tokens():
    """A first tile that weighs 2^60 units of its own, and u times the sum within a few hundred units of its end: a token is
    written all the same, the tile's last or the next tile's first (either is right this near to the border)."""
    import torch

    announce("sample: u at the end of a heavy tile")
    rows = np.stack([balanced_rows(F(-0.00197 * (1 + i / 64)), s) for i in range(16) for s in range(-2048, 2049, 128)])
    got, chance = run(torch.from_numpy(rows).cuda(), np.full(len(rows), 0.5, F))
    w = np.exp(rows.astype(np.float64))
    assert np.isin(got, [511, 512]).all(), f"{np.count_nonzero(got == -7)} of {len(rows)} rows not answered"
    want = w[np.arange(len(rows)), got] / w.sum(1)
    assert (np.abs(chance - want) <= 2.0 ** -23 * want).all()
