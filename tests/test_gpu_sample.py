"""gdn_sample against its definition in 64 bits (tests/sample_ref.py): tokens equal, probabilities within 2^-23.

A random number that falls nearer to a border of its distribution than the weights' whole multiples allow (sample_ref.border)
would prove nothing; the fixed seeds have none (asserted)."""

import numpy as np
import pytest

from tests.gpu_helpers import announce
from tests.sample_ref import border, sample

pytestmark = pytest.mark.gpu


def run(x, u, t=None, k=None, p=None, least=None, prob=True, **kw):
    import torch

    import gated_delta_rule_conv_amd as gdn

    rows, vocab = x.shape
    dev = lambda a, kind: None if a is None else torch.as_tensor(a, dtype=kind).cuda()  # noqa: E731
    tokens = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    chance = torch.full((rows,), -7.0, device="cuda") if prob else None
    gdn.sample(x, dev(u, torch.float32), tokens, gdn.sample_workspace(rows, vocab), temperature=dev(t, torch.float32),
               top_k=dev(k, torch.int32), top_p=dev(p, torch.float32), min_p=dev(least, torch.float32), prob=chance, **kw)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), None if chance is None else chance.cpu().numpy()


def check(x, u, t=None, k=None, p=None, least=None):
    got, chance = run(x, u, t, k, p, least)
    h = x.float().cpu().numpy()
    f32 = lambda a, i, off: off if a is None else float(np.float32(a[i]))  # noqa: E731
    for r in range(h.shape[0]):
        kw = dict(t=f32(t, r, 1.0), k=0 if k is None else int(k[r]), p=f32(p, r, 1.0), least=f32(least, r, 0.0))
        v = float(np.float32(u[r]))
        want, prob = sample(h[r], v, **kw)
        if v > 0 and v < 1:
            assert border(h[r], v, **kw) > 1, f"row {r}: choose another seed"
        assert got[r] == want, f"row {r}: {got[r]}, not {want} ({kw}, u {u[r]})"
        assert abs(chance[r] - prob) <= 2.0 ** -23 * prob, f"row {r}"
    return got


def logits(rows, vocab, dtype="f32", seed=0, std=2.5, stride=None):
    import torch

    g = torch.Generator().manual_seed(seed)
    x = (std * torch.randn((rows, stride or vocab), generator=g)).to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
    return x.cuda()[:, :vocab]


def numbers(rows, seed=1):
    r = np.random.default_rng(seed)
    return dict(u=r.random(rows).astype(np.float32), t=(0.4 + r.random(rows)).astype(np.float32), k=r.integers(1, 60, rows),
                p=(0.5 + 0.5 * r.random(rows)).astype(np.float32), least=(0.2 * r.random(rows)).astype(np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 63, 64, 1000, 1023, 4096, 4097, 8192, 8193, 50001, 131072])
def test_every_filter_alone_and_together(dtype, vocab):
    announce(f"sample vocab {vocab} {dtype}")
    rows = 9
    x, n = logits(rows, vocab, dtype, seed=vocab), numbers(rows, vocab)
    for use in ("", "t", "tk", "tp", "tm", "kp", "tkpm"):
        check(x, n["u"], t=n["t"] if "t" in use else None, k=n["k"] if "k" in use else None, p=n["p"] if "p" in use else None,
              least=n["least"] if "m" in use else None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_values_everywhere(dtype):
    """Ties go to the lowest index: rows of one value, of two, of few; the filters' borders inside the ties."""
    import torch

    announce(f"sample ties {dtype}")
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    for vocab in (5, 1000, 70001):
        x = torch.zeros(8, vocab, dtype=kind, device="cuda")
        x[1:3] = 3.5
        x[2, ::2] = 4.5
        x[3, ::3] = -0.0
        x[4] = torch.arange(vocab, device="cuda").remainder(5).to(kind)
        x[5] = -torch.arange(vocab, device="cuda").remainder(7).to(kind)
        x[6, vocab // 2:] = 9.0
        n = numbers(8, vocab + 1)
        check(x, n["u"])
        check(x, n["u"], k=[1, 2, vocab // 2, vocab - 1, 3, vocab // 3, vocab // 4 + 1, vocab])
        check(x, n["u"], p=[0.5, 0.25, 0.999, 0.1, 0.75, 0.3, 0.01, 0.5], t=n["t"])
        check(x, n["u"], p=n["p"], k=n["k"] * 7 + 1, t=n["t"], least=[1.0, 0.5, 1.0, 0.0, 0.3, 0.1, 2.0, 0.9])


def test_masks_infinities_and_nan():
    import torch

    announce("sample: banned tokens, infinities, NaN")
    inf, vocab = float("inf"), 9001
    x = logits(12, vocab, seed=5)
    x[0] = -inf
    x[1] = float("nan")
    x[2, :] = -inf
    x[2, 77] = -3e38
    x[3, ::2] = -inf
    x[4, 17] = inf
    x[5, 100:200:7] = inf
    x[6, ::3] = float("nan")
    x[7] = 3e38
    x[7, 5] = -3e38
    x[8] = -3e38
    x[9, 8000:] = -inf
    x[9, :7999] = -inf
    x[10] = torch.finfo(torch.float32).min
    x[10, 9000] = 0.0
    n = numbers(12, 6)
    for kw in (dict(), dict(t=n["t"]), dict(k=n["k"]), dict(p=n["p"]), dict(t=n["t"], k=n["k"], p=n["p"], least=n["least"])):
        got = check(x, n["u"], **kw)
        assert got[0] == -1 and got[1] == -1 and got[2] == 77 and got[4] == 17 and got[9] == 7999


def test_numbers_at_their_ends():
    """u of 0 and just under 1 and outside; temperatures of 0, below, tiny, infinite; p and min_p outside their range; k of
    1, vocab and beyond."""
    announce("sample: ends of the ranges")
    inf, nan = float("inf"), float("nan")
    x = logits(10, 5000, seed=8)
    u = np.array([0.0, 1 - 2.0 ** -24, 1.0, 7.0, -3.0, nan, 0.5, 0.25, 0.9, 0.1], np.float32)
    check(x, u)
    check(x, u, k=[1, 5000, 5001, 2 ** 31 - 1, 0, -5, 2, 3, 4, 4999], p=[1.0, 2.0, nan, inf, 0.0, -1.0, 1e-30, 0.3, 0.99999994, 0.5])
    u[:] = 0.37
    check(x, u, t=[0.0, -1.0, nan, 1e-30, 1e-3, inf, 1e30, 100.0, 1e-45, 0.05])
    check(x, u, least=[1.0, 1.5, inf, nan, 0.0, -1.0, 1e-30, 0.3, 0.999, 1e-6])


def test_flat_and_steep_rows():
    """Whole vocabularies inside a filter's first bin, and weights below every multiple."""
    import torch

    announce("sample: flat and steep rows")
    g = torch.Generator().manual_seed(3)
    x = torch.empty(6, 40000)
    x[0] = 1 + 1e-6 * torch.rand(40000, generator=g)
    x[1] = 100 + torch.rand(40000, generator=g)
    x[2] = 1e-38 * torch.randn(40000, generator=g)
    x[3] = 200 * torch.randn(40000, generator=g)
    x[4] = -torch.arange(40000).float() / 1000
    x[5] = 1e30 * torch.randn(40000, generator=g)
    n = numbers(6, 11)
    for kw in (dict(), dict(p=n["p"]), dict(k=[1, 100, 20000, 30000, 39999, 5], p=n["p"]), dict(k=[39999] * 6, p=[0.999] * 6, t=n["t"])):
        check(x.cuda(), n["u"], **kw)


def test_parts_of_a_row_that_weigh_nothing():
    """Long runs of tokens whose weight rounds to 0, before, between and after the others: not even u = 0 gives one of them."""
    import torch

    announce("sample: runs without weight")
    inf, vocab = float("inf"), 9000
    x = torch.full((8, vocab), -1000.0)
    x[0:4, [3000, 3001, 7000]] = 0.0
    x[4:6, 5000:] = inf
    x[6, 8999] = 0.0
    x[7, 0] = 0.0
    u = np.array([0.0, 1e-20, 0.5, 1 - 2.0 ** -24, 0.0, 1 - 2.0 ** -24, 0.0, 1 - 2.0 ** -24], np.float32)
    for kw in (dict(), dict(least=[1e-30] * 8), dict(p=[0.9] * 8), dict(k=[8999] * 8)):
        got, chance = run(x.cuda(), u, **kw)
        stay = 3600 if "p" in kw else 4000  # of the infinities
        assert got.tolist() == [3000, 3000, 3001, 7000, 5000, 4999 + stay, 8999, 0]
        assert np.allclose(chance, [1 / 3] * 4 + [1 / stay] * 2 + [1.0] * 2, rtol=2.0 ** -22, atol=0)


def test_rows_strides_and_neighbours():
    """Rows of a wider tensor at odd addresses; a row's token does not depend on the others."""
    announce("sample: strides, rows alone")
    x = logits(33, 3001, "bf16", seed=9, stride=3010)[:, :]
    n = numbers(33, 12)
    kw = dict(t=n["t"], k=n["k"], p=n["p"], least=n["least"])
    got = check(x, n["u"], **kw)
    for r in (0, 7, 32):
        alone, _ = run(x[r:r + 1], n["u"][r:r + 1], n["t"][r:r + 1], n["k"][r:r + 1], n["p"][r:r + 1], n["least"][r:r + 1], prob=False)
        assert alone[0] == got[r]


def test_offsets_past_32_bits():
    """The last row of logits begins beyond 2^32 bytes (and 2^31 elements)."""
    import torch

    announce("sample: rows beyond 2^32 bytes")
    rows, stride = 3, (1 << 30) + 8
    base = torch.empty(2 * stride + 1000, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((rows, 1000), (stride, 1))
    x.copy_(logits(rows, 1000, "bf16", seed=10))
    check(x, numbers(rows, 13)["u"], k=[5, 50, 500])


def test_the_largest_vocabulary():
    announce("sample: 2^20 tokens")
    x, n = logits(2, 1 << 20, seed=30, std=1.0), numbers(2, 31)
    check(x, n["u"], t=n["t"], k=[0, 5000], p=n["p"])
    check(x, n["u"])


def test_the_frequencies_are_the_probabilities():
    """4000 numbers spread evenly over [0, 1): a token's count is 4000 times its probability to within one."""
    import torch

    announce("sample: frequencies")
    one = logits(1, 50, seed=2)
    x = one.expand(4000, 50).contiguous()
    u = ((np.arange(4000) + 0.5) / 4000).astype(np.float32)
    got, _ = run(x, u, t=np.full(4000, 0.8, np.float32))
    w = torch.softmax(one.double().cpu()[0] / float(np.float32(0.8)), 0).numpy()
    assert (np.abs(np.bincount(got, minlength=50) - 4000 * w) <= 1.001).all()


def test_captured_twice_with_one_workspace():
    """Two graphs that share a workspace and an eager call between them, replayed in turn."""
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce("sample in two graphs")
    a, b = logits(5, 20000, seed=20), logits(5, 20000, "bf16", seed=21)
    n = numbers(5, 14)
    u, p = torch.tensor(n["u"]).cuda(), torch.tensor(n["p"]).cuda()
    want = [run(t, n["u"], p=n["p"])[0] for t in (a, b)]
    work, out = gdn.sample_workspace(5, 20000), torch.empty(2, 5, dtype=torch.int32, device="cuda")
    graphs = []
    for i, t in enumerate((a, b)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gdn.sample(t, u, out[i], work, top_p=p)
        graphs.append(graph)
    for _ in range(4):
        out.fill_(-9)
        for i in (0, 1):
            graphs[i].replay()
        gdn.sample(a, u, torch.empty(5, dtype=torch.int32, device="cuda"), work)
        torch.cuda.synchronize()
        assert (out.cpu().numpy() == np.stack(want)).all()
