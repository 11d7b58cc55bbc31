"""Linear attention whose terms cancel: the products keep what fp32 keeps, whatever type the outputs have.

Tolerance, in the sum of the terms' magnitudes M. A score is one exact product of two bf16 values times the scale: one
rounding, 2^-24. A state's element times a bf16 value, or a score times one, goes into the sum exactly, in up to 6 matrix
instructions; each joins its products and the sum so far in up to 4 steps that may cut instead of round, 2^-23 each. The sum
with the state is multiplied by the scale once more, and added to, 2 x 2^-24. All in all 24 x 2^-23 + 3 x 2^-24 = 51 x 2^-24. bf16
outputs add half a step of the value, 2^-8 of it."""

import numpy as np
import pytest

from tests.gpu_helpers import announce, bits_of
from tests.test_gpu_linear import BF16, F32, Case

pytestmark = pytest.mark.gpu
OFF = 51 * 2.0 ** -24


def near(got, want, magnitude, out):
    got = got.double().cpu().numpy()
    off = np.abs(got - want) - OFF * magnitude
    if out == BF16:
        off -= 2.0 ** -8 * (np.abs(want) + OFF * magnitude)
    assert np.isfinite(got).all() and (off <= 0).all(), f"{(off > 0).mean():.3f} of the outputs off, by up to " \
                                                        f"{(np.abs(got - want) / magnitude).max() * 2 ** 24:.0f} x 2^-24 of the terms"


def opposites(rng):
    """8-bit mantissas a, b and all pairs x, y with |a x - b y| in 1 .. 4 of about 2^15 (eight at least), over 128."""
    m = np.arange(128, 256)
    while True:
        a, b = rng.integers(128, 256, 2)
        diff = np.abs(a * m[:, None] - b * m[None, :])
        pairs = np.argwhere((diff >= 1) & (diff <= 4)) + 128
        if len(pairs) >= 8:
            return (a / 128, b / 128), pairs / 128


def case(lens, out, seed, form=0):
    import torch

    c = Case(lens, Hk=2, Hv=4, d=64, dtype=BF16, out=out, seed=seed, form=form, g=torch.zeros(sum(lens), 4))
    c.x.zero_()
    return c


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("mma", [0, 1, 2])
def test_two_tokens_that_cancel(out, mma):
    """Of every pair of tokens the second sees the first and itself, with opposite values: a score times a value each, the sum 2^-13
    and less of either."""
    import torch

    announce(f"linear prefill: cancelling tokens -> {out}, policy {mma}")
    c = case([64], out, 1)
    c.dims.mma = mma
    c.state.zero_()
    r = np.random.default_rng(2)
    q, k, v = np.zeros((64, 2, 64)), np.zeros((64, 2, 64)), np.zeros((64, 4, 64))
    for p in range(32):
        for h in range(2):
            keys, pairs = opposites(r)
            x = pairs[r.integers(0, len(pairs), (2, 64))]
            k[2 * p, h, p], k[2 * p + 1, h, p] = keys
            q[2 * p + 1, h, p] = r.integers(128, 256) / 128 * 2.0 ** r.integers(-3, 4)
            v[2 * p, 2 * h:2 * h + 2], v[2 * p + 1, 2 * h:2 * h + 2] = x[..., 0], -x[..., 1]
    for t, x in ((c.q, q), (c.k, k), (c.v, v)):
        t.copy_(torch.from_numpy(x.reshape(64, -1)).to(torch.bfloat16).cuda())
        assert (t.double().cpu().numpy() == x.reshape(64, -1)).all()
    c.prefill()
    torch.cuda.synchronize()
    q, k = np.repeat(q, 2, 1), np.repeat(k, 2, 1)
    scores = np.einsum("ihd,jhd->hij", q, k) * np.tril(np.ones((64, 64))) * float(np.float32(c.scale))
    want = np.einsum("hij,jhv->ihv", scores, v)
    magnitude = np.einsum("hij,jhv->ihv", np.abs(scores), np.abs(v))
    live = np.arange(1, 64, 2)
    assert (np.abs(want[live]) < 2.0 ** -11 * magnitude[live]).all()
    near(c.o[live], want[live], magnitude[live], out)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("lens,form", [([64, 30], 1), ([700, 5], 2)])
def test_columns_of_the_state_that_cancel(out, lens, form):
    """Tokens that only read: q has two entries, whose columns of the state cancel to 2^-12 and less; the state keeps its bits."""
    import torch

    announce(f"linear prefill: cancelling columns of the state -> {out}, {lens}")
    c = case(lens, out, 3, form)
    r = np.random.default_rng(4)
    T = sum(lens)
    q = np.zeros((T, 2, 64))
    a, b = r.integers(128, 256, (2, 32)) / 128
    for t in range(T):
        q[t, :, 2 * (t % 32)], q[t, :, 2 * (t % 32) + 1] = a[t % 32], -b[t % 32]
    S = r.standard_normal((len(lens), 4, 64, 64)).astype(np.float32)
    S[..., 1::2] = (S[..., ::2] * (a / b) * (1 + 2.0 ** -12 * r.random((len(lens), 4, 64, 32)))).astype(np.float32)
    c.q.copy_(torch.from_numpy(q.reshape(T, -1)).to(torch.bfloat16).cuda())
    c.state[c.slot] = torch.from_numpy(S).cuda()
    before = bits_of(c.state)
    c.prefill()
    torch.cuda.synchronize()
    assert (bits_of(c.state) == before).all()
    seq = np.repeat(np.arange(len(lens)), lens)
    q, S, scale = np.repeat(q, 2, 1), S.astype(np.float64), float(np.float32(c.scale))
    want = np.concatenate([scale * np.einsum("hvk,thk->thv", S[i], q[seq == i]) for i in range(len(lens))])
    magnitude = np.concatenate([scale * np.einsum("hvk,thk->thv", np.abs(S[i]), np.abs(q[seq == i])) for i in range(len(lens))])
    near(c.o, want, magnitude, out)
