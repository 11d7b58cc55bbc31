"""gdn_tree_verify with nodes that are not finite, or whose products are not: their descendants'
results are NaN, and every other node keeps the bits it has in the same call without them."""

import numpy as np
import pytest

from gen.inputs import LayerShape, _store
from tests.gpu_helpers import TOL_F32, announce, bits_of
from tests.test_gpu_tree import accept, check_o, device, make_case, make_dims, oracle_tree, verify

pytestmark = pytest.mark.gpu

# one shape a form of the kernel: 16, 32 and 64 nodes, heads after each other and side by side, fp32 products (fp32
# input) and pairs of halves (bf16 input)
FORMS = [(1, 2, 32, "f32", 16), (2, 4, 32, "bf16", 31), (1, 3, 64, "f32", 64), (1, 2, 128, "bf16", 16), (1, 2, 128, "f32", 30),
         (2, 4, 128, "bf16", 64), (1, 2, 64, "bf16", 50), (2, 2, 32, "bf16", 64), (1, 3, 128, "f32", 64)]


def descendants(c, tree, node):
    """The node (a number inside its tree) and those below it."""
    a, hit = int(c["cu"][tree]), {node}
    for t in range(node + 1, c["lens"][tree]):
        if int(c["parents"][a + t]) in hit:
            hit.add(t)
    return hit


def token_conv(c):
    """The conv hands each token on as it is (width 2), so a token is seen by itself and below only
    through the rule."""
    w = np.zeros((c["shape"].channels, 2))
    w[:, 1] = 1.0
    c["conv_w"] = _store(w, c["shape"].in_dtype)


def rig(hk, hv, d, dtype, n, seed=11, kind="tree", **kw):
    sh = LayerShape(hk, hv, d, conv_width=2, in_dtype=dtype)
    c = make_case(sh, [5, n], kind, seed=seed)
    token_conv(c)
    return c, device(c, make_dims(sh, **kw))


def same_but(c, tree, hit, clean, got, heads=None):
    """Every row but the hit nodes' (of the given heads) has the clean run's bits."""
    import torch

    a = int(c["cu"][tree])
    for name, x, y in (("o", clean["o"], got["o"]), ("u", clean["rec"][1], got["rec"][1])):
        for t in range(len(c["parents"])):
            for j in range(x.shape[1]):
                if t - a in hit and (heads is None or j in heads):
                    continue
                assert torch.equal(x[t, j], y[t, j]), (name, t, j)


@pytest.mark.parametrize("hk,hv,d,dtype,n", FORMS)
@pytest.mark.parametrize("what,bad", [("g", float("nan")), ("g", float("inf")), ("beta", float("nan")), ("beta", float("inf"))])
def test_a_broken_gate_reaches_only_its_descendants(hk, hv, d, dtype, n, what, bad):
    """One v-head's gate of one node, in the tree's first block of 16 and in its last."""
    import torch

    announce(f"tree: {what} = {bad}, hk={hk} hv={hv} d={d} {dtype} {n} nodes")
    c, e = rig(hk, hv, d, dtype, n)
    verify(e)
    for node in sorted({1, n - 9}):
        for head in (0, hv - 1):
            f = device(c, e["dims"])
            f[what][5 + node, head] = bad
            verify(f)
            torch.cuda.synchronize()
            hit = descendants(c, 1, node)
            same_but(c, 1, hit, e, f, heads={head})
            for t in hit:
                assert torch.isnan(f["o"][5 + t, head]).all() and torch.isnan(f["rec"][1][5 + t, head]).all(), (node, t)
            ok = max(t for t in range(n) if t not in hit)
            g = device(c, e["dims"])
            accept(dict(f), [3, ok])
            accept(dict(g, rec=e["rec"]), [3, ok])
            torch.cuda.synchronize()
            np.testing.assert_array_equal(bits_of(f["pool"].state), bits_of(g["pool"].state))


@pytest.mark.parametrize("hk,hv,d,dtype,n", FORMS)
def test_a_wholly_broken_token(hk, hv, d, dtype, n):
    """NaN in x, g and beta of two nodes, as a broken hidden state gives."""
    import torch

    announce(f"tree: broken token, hk={hk} hv={hv} d={d} {dtype} {n} nodes")
    c, e = rig(hk, hv, d, dtype, n)
    verify(e)
    f = device(c, e["dims"])
    hit = set()
    for node in (2, n - 3):
        for k in ("x", "g", "beta"):
            f[k][5 + node] = float("nan")
        hit |= descendants(c, 1, node)
    verify(f)
    torch.cuda.synchronize()
    same_but(c, 1, hit, e, f)
    for t in hit:
        assert torch.isnan(f["o"][5 + t]).all()


def test_a_state_row_that_is_not_finite_stays_alone():
    """One NaN (infinity) in one row of the slot's state: that row's results of every node, no other."""
    import torch

    announce("tree: state rows not finite")
    c, e = rig(1, 2, 64, "f32", 40)
    verify(e)
    for bad in (float("nan"), float("inf")):
        f = device(c, e["dims"])
        f["pool"].state[c["slots"][1], 1, 21, 5] = bad
        verify(f)
        torch.cuda.synchronize()
        rows = [r for r in range(64) if r != 21]
        assert torch.equal(f["o"][:, 0], e["o"][:, 0]) and torch.equal(f["o"][:, 1, rows], e["o"][:, 1, rows])
        assert torch.equal(f["o"][:5], e["o"][:5]) and not torch.isfinite(f["o"][5:, 1, 21]).any()


@pytest.mark.parametrize("hk,hv,d,dtype,n", FORMS)
@pytest.mark.parametrize("what", ["k", "q"])
def test_a_zero_row_without_epsilon(hk, hv, d, dtype, n, what):
    """l2_eps = 0 and a key (query) of zeros: 0 / 0, in its own node and, for a key, below it."""
    import torch

    announce(f"tree: zero {what}, l2_eps 0, hk={hk} hv={hv} d={d} {dtype} {n} nodes")
    c, e = rig(hk, hv, d, dtype, n, l2_eps=0.0)
    verify(e)
    for node in (1, n - 4):
        f = device(c, e["dims"])
        first = hk * d if what == "k" else 0
        f["x"][5 + node, first:first + d] = 0.0  # (k-head 0: v-heads 0 .. hv / hk - 1)
        verify(f)
        torch.cuda.synchronize()
        hit = descendants(c, 1, node) if what == "k" else {node}
        heads = set(range(hv // hk))
        a = 5
        for t in range(n):
            for j in range(hv):
                if t in hit and j in heads:
                    assert torch.isnan(f["o"][a + t, j]).all(), (node, t, j)
                else:
                    assert torch.equal(f["o"][a + t, j], e["o"][a + t, j]), (node, t, j)


@pytest.mark.parametrize("hk,hv,d,dtype,n", FORMS)
def test_an_unnormalised_key_beyond_the_square_root(hk, hv, d, dtype, n):
    """qk_l2norm_off, one leaf with q of 1e20 (1e-25) and beta = 0: o = e^G S q, finite, to the usual gate."""
    import torch

    announce(f"tree: q of 1e20 and 1e-25, no norm, hk={hk} hv={hv} d={d} {dtype}")
    c, _ = rig(hk, hv, d, dtype, 12, kind="star")
    for size in (1e20, 1e-25):
        r = np.random.default_rng(3)
        x = r.standard_normal((len(c["parents"]), c["shape"].channels)) * d ** -0.5
        x[:, :hk * d] *= size
        x[:, hk * d:2 * hk * d] *= 1e-3 if size > 1 else size
        c["x"] = _store(x, dtype)
        c["beta"][:] = 0.0
        dims = make_dims(c["shape"], qk_l2norm=False)
        o, _, _ = oracle_tree(c, dict(qk_l2norm=False))
        e = device(c, dims)
        verify(e)
        torch.cuda.synchronize()
        check_o(c, e["o"], o, TOL_F32)
@pytest.mark.parametrize("hk,hv,d,dtype,n", FORMS)
def test_keys_whose_square_overflows(hk, hv, d, dtype, n):
    """qk_l2norm_off and one finite key of 1e20s, whose |k|^2 is above the largest fp32 number: its
    descendants' products overflow, nobody else's do."""
    import torch

    announce(f"tree: k of 1e20, no norm, hk={hk} hv={hv} d={d} {dtype} {n} nodes")
    c, e = rig(hk, hv, d, dtype, n, qk_l2norm=False)
    e["x"].mul_(d ** -0.5)
    verify(e)
    for node in (1, n - 4):
        f = device(c, e["dims"])
        f["x"].mul_(d ** -0.5)
        f["x"][5 + node, hk * d:hk * d + d] = 1e20
        verify(f)
        torch.cuda.synchronize()
        same_but(c, 1, descendants(c, 1, node), e, f, heads=set(range(hv // hk)))


@pytest.mark.parametrize("hk,hv,d,dtype,n", FORMS)
def test_a_path_that_diverges_reaches_only_itself(hk, hv, d, dtype, n):
    """qk_l2norm_off and keys of |k|^2 = 1e6 on one chain: (I - beta k k^T) expands its state until it
    overflows. Every second node is on the chain; the others are children of the slot or of each other."""
    import torch

    announce(f"tree: diverging chain, hk={hk} hv={hv} d={d} {dtype} {n} nodes")
    c, _ = rig(hk, hv, d, dtype, n)
    for t in range(n):
        c["parents"][5 + t] = t - 2 if t % 2 else (-1 if t % 4 == 0 else t - 2)
    odd = [5 + t for t in range(1, n, 2)]
    dims = make_dims(c["shape"], qk_l2norm=False)
    runs = []
    for size in (d ** -0.5, 1e3 * d ** -0.5):
        e = device(c, dims)
        e["x"].mul_(d ** -0.5)
        e["x"][odd, hk * d:2 * hk * d] = size
        e["beta"][odd] = 1.0
        e["g"][odd] = -1e-3
        verify(e)
        runs.append(e)
    torch.cuda.synchronize()
    if n > 32:
        assert not torch.isfinite(runs[1]["o"][odd]).all()  # (it did diverge)
    same_but(c, 1, set(range(1, n, 2)), *runs)


@pytest.mark.parametrize("hk,hv,d,dtype,n", FORMS)
def test_values_next_to_the_largest_number(hk, hv, d, dtype, n):
    """v of 3e38 along a chain of equal keys: u overflows below it, not beside it."""
    import torch

    announce(f"tree: v of 3e38, hk={hk} hv={hv} d={d} {dtype} {n} nodes")
    c, _ = rig(hk, hv, d, dtype, n)
    for t in range(n):
        c["parents"][5 + t] = t - 2 if t % 2 else (-1 if t % 4 == 0 else t - 2)
    odd = [5 + t for t in range(1, n, 2)]
    runs = []
    for sign in (0.0, 1.0):
        e = device(c, make_dims(c["shape"]))
        e["x"][odd, hk * d:2 * hk * d] = 1.0
        # signs that add up in u: v, -v, v ..
        for i, t in enumerate(odd):
            e["x"][t, 2 * hk * d:] = 3e38 * sign * (-1) ** i
        e["beta"][odd] = 1.0
        e["g"][odd] = 0.0
        verify(e)
        runs.append(e)
    torch.cuda.synchronize()
    same_but(c, 1, set(range(1, n, 2)), *runs)
