"""gdn_sample in calls of so many tokens that a wave takes several tiles of a row, as batches of a server's vocabulary do (tiles of 512
tokens; a row's workgroups of 8 waves are as many as make about 768 in the call, but no more than the row has work for)."""

import numpy as np
import pytest

from tests.gpu_helpers import announce
from tests.test_gpu_sample import check, logits, numbers, run

pytestmark = pytest.mark.gpu
INF = float("inf")


def tiles_a_wave(rows, vocab):
    tiles = -(-vocab // 512)
    groups = min(-(-768 // rows), -(-tiles // 8))
    return -(-tiles // (8 * groups))


def batch(rows, vocab, dtype, seed):
    """Rows of all kinds: banned tokens, one token left, none, infinities, NaN, all equal, nearly equal."""
    x = logits(rows, vocab, dtype, seed=seed).clone()
    r = np.random.default_rng(seed)
    x[1, ::2] = -INF
    x[2] = -INF
    x[3] = -INF
    x[3, vocab - 1] = 0.5
    x[4, vocab // 2] = INF
    x[5, 3::vocab // 7] = INF
    x[6, ::3] = float("nan")
    x[7] = 1.5
    x[8, vocab // 2:] = 9.0
    x[9, :vocab // 2] = 9.0
    x[10] = -3e38
    x[10, [5, vocab - 2]] = 0.0
    u = r.random(rows).astype(np.float32)
    u[:2], u[8:10] = [0.0, 1 - 2.0 ** -24], [0.75, 0.25]
    return x, u


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(70, 50001), (800, 9001), (200, 20480)])
@pytest.mark.parametrize("use", ["", "t", "m", "k", "p", "tkpm"])
def test_several_tiles_a_wave(dtype, rows, vocab, use):
    announce(f"sample {rows} x {vocab} {dtype}, filters '{use}'")
    assert tiles_a_wave(rows, vocab) > 1 and vocab == 20480 or -(-vocab // 512) % 8 != 0
    x, u = batch(rows, vocab, dtype, vocab + 1)
    n = numbers(rows, vocab)
    n["t"][11:13], n["k"][13], n["p"][14] = 0.0, 0, 1.0
    got = check(x, u, t=n["t"] if "t" in use else None, k=n["k"] if "k" in use else None, p=n["p"] if "p" in use else None,
                least=n["least"] if "m" in use else None)
    assert got[2] == -1 and got[3] == vocab - 1 and got[4] == vocab // 2


@pytest.mark.parametrize("rows,vocab,dtype", [(1024, 131072, "bf16"), (900, 100003, "f32")])
def test_a_workgroup_a_row(rows, vocab, dtype):
    """Temperature alone, one workgroup a row, against 64 bits on the GPU."""
    import torch

    announce(f"sample {rows} x {vocab} {dtype}, temperature alone")
    assert tiles_a_wave(rows, vocab) >= 16
    x = torch.cat([logits(64, vocab, dtype, seed=40 + i, std=2.5) for i in range((rows + 63) // 64)])[:rows].contiguous()
    x[3::8] = torch.where(torch.arange(vocab, device="cuda") % 97 == 5, x[3::8].float(), -INF).to(x.dtype)
    x[49::50] = -INF
    n = numbers(rows, 41)
    got, chance = run(x, n["u"], t=n["t"])
    u, t = (torch.from_numpy(n[k]).double().cuda()[:, None] for k in ("u", "t"))
    for a in range(0, rows, 64):
        b = min(a + 64, rows)
        y = x[a:b].double()
        some = y.amax(1) > -INF
        w = torch.exp((y - y.amax(1, keepdim=True).clamp(min=-1e300)) / t[a:b])
        sums = w.cumsum(1)
        whole = sums[:, -1:].clamp(min=1e-300)
        # a border lies off by half a unit, 2^-46, of the largest weight a token and as much again where tiles are rounded, and by
        # 2^-38 of the sum for the exponentials
        near = ((w > 0).sum(1) * 2.0 ** -45 * w.amax(1) / whole[:, 0] + 2.0 ** -38)[some]
        assert ((sums / whole - u[a:b]).abs().amin(1)[some] > near).all(), "choose another seed"
        token = (sums > u[a:b] * whole).int().argmax(1)
        prob = (w.gather(1, token[:, None]) / whole)[:, 0]
        want = torch.where(some, token, -1).cpu().numpy()
        assert (got[a:b] == want).all(), f"rows {a} .. {b}"
        prob = torch.where(some, prob, 0.0).cpu().numpy()
        assert (np.abs(chance[a:b] - prob) <= 2.0 ** -23 * prob).all()
