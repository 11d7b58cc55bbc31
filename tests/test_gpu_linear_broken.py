"""Infinities and NaN inside sequences cut into several tiles: what comes before them, other heads and other sequences
keep their bits."""

import pytest

from tests.gpu_helpers import announce, bits_of
from tests.test_gpu_linear import BF16, F32, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,out", [(BF16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("what", ["q", "k", "v", "g"])
@pytest.mark.parametrize("token", [30, 127, 128, 401, 699])
def test_what_a_broken_value_leaves_alone(dtype, out, what, token):
    """A sequence of 700 tokens in tiles of 128, with one broken value in its first, a middle or its last tile."""
    import numpy as np
    import torch

    for bad in (float("nan"), float("inf"), -float("inf")):
        if what == "g" and bad == bad:
            continue  # (minus infinity is a decay like others, plus infinity none)
        announce(f"linear prefill {what}[{token} of 700] = {bad} {dtype}->{out}")
        clean, c = (Case([90, 700, 40], Hk=2, Hv=4, d=64, dtype=dtype, out=out, seed=4, form=2) for _ in range(2))
        row, head, hit = 90 + token, 1, {"q": [0, 1], "k": [0, 1], "v": [1], "g": [1]}[what]
        if what == "g":
            c.g[row, head] = bad
        elif what == "v":
            c.v[row, head * 64 + 5] = bad
        else:
            getattr(c, what)[row, 5] = bad
        clean.prefill()
        c.prefill()
        torch.cuda.synchronize()
        a, b = bits_of(c.o), bits_of(clean.o)
        others = [h for h in range(4) if h not in hit]
        assert (a[:row] == b[:row]).all() and (a[790:] == b[790:]).all() and (a[:, others] == b[:, others]).all()
        sa, sb = bits_of(c.state), bits_of(clean.state)
        assert (sa[c.slot[[0, 2]]] == sb[c.slot[[0, 2]]]).all() and (sa[:, others] == sb[:, others]).all()
        o, S = c.o.float().cpu().numpy(), c.state[c.slot[1]].cpu().numpy()
        if what == "q":
            assert not np.isfinite(o[row, hit]).any()
            assert (a[row + 1:] == b[row + 1:]).all() and (sa == sb).all()
        elif what == "k":  # (the state's column 5; every later output reads it)
            assert not np.isfinite(o[row:790, hit]).any() and not np.isfinite(S[hit, :, 5]).any()
        elif what == "v":
            rest = [x for x in range(64) if x != 5]
            assert not np.isfinite(o[row:790, head, 5]).any() and not np.isfinite(S[head, 5]).any()
            assert (a[:, head][:, rest] == b[:, head][:, rest]).all() and (sa[c.slot[1], head][rest] == sb[c.slot[1], head][rest]).all()
        else:
            assert not np.isfinite(o[row:790, head]).any() and not np.isfinite(S[head]).any()
