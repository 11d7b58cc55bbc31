"""gdn_sample where the random number falls next to a border: rows made for it."""

import math

import numpy as np
import pytest

from tests.gpu_helpers import announce
from tests.sample_ref import sample
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


# A weight is e^(x / T) to 2^-51 of the largest, rounded to a multiple of 2^-51 in small vocabularies: half a unit more. Of two
# tokens, with one rounding of their sum and one of u times it, a border is met within 2 x 1.5 x 2^-51 + 2 x 2^-52 = 2^-49 of the sum.
NEAR = 2.0 ** -49


def all_fp32(lo, hi):
    """Every fp32 number in (lo, hi], both negative."""
    a, b = (int(F(v).view(np.uint32)) for v in (hi, lo))
    return np.arange(a, b, dtype=np.uint32).view(F)


@pytest.mark.parametrize("use", ["plain", "min_p", "top_p"])
def test_numbers_nearer_to_a_border_than_40_bits(use):
    """Two tokens, x and 0, the first one's share of the weight within 2^-43 of u, but not within 2^-48."""
    import torch

    announce(f"sample: u within 2^-43 of a border, {use}")
    x = np.concatenate([all_fp32(-0.5, -0.25), all_fp32(-1.0, -0.75)])
    w = np.exp(x.astype(np.float64))
    share = w / (1 + w)  # (to 2^-52)
    u = np.rint(share * 2.0 ** 24) * 2.0 ** -24
    off = np.abs(share - u)
    rows = np.flatnonzero((off < 2.0 ** -43) & (off > 2 * NEAR))
    assert len(rows) > 40
    logits = np.stack([x[rows], np.zeros(len(rows), F)], 1)
    # (a filter that takes nothing away, for the other path)
    kw = {"plain": {}, "min_p": {"least": np.full(len(rows), 1e-30, F)}, "top_p": {"p": np.full(len(rows), 0.9999999, F)}}[use]
    got, chance = run(torch.from_numpy(logits).cuda(), u[rows].astype(F), **kw)
    want = (u[rows] >= share[rows]).astype(int)
    assert (got == want).all(), f"{np.count_nonzero(got != want)} of {len(rows)}"
    for r in range(0, len(rows), 10):
        assert sample(logits[r], float(u[rows][r]))[0] == want[r]


def test_weights_next_to_min_p():
    """Two tokens, the second one's weight within 2^-42 of min_p: it stays if it is as large."""
    import torch

    announce("sample: weights within 2^-42 of min_p")
    x = np.concatenate([all_fp32(-0.5, -0.25), all_fp32(-1.0, -0.75)])
    w = np.exp(x.astype(np.float64))
    least = w.astype(F)
    off = np.abs(w - least.astype(np.float64))
    rows = np.flatnonzero((off < 2.0 ** -42) & (off > NEAR))
    assert len(rows) > 40
    logits = np.stack([np.zeros(len(rows), F), x[rows]], 1)
    got, _ = run(torch.from_numpy(logits).cuda(), np.full(len(rows), 0.9999, F), least=least[rows])
    want = (w[rows] >= least[rows]).astype(int)
    assert (got == want).all(), f"{np.count_nonzero(got != want)} of {len(rows)}"
