"""gdn_tree_follow against the walk written out on the host."""

import numpy as np
import pytest

from tests.gpu_helpers import announce

pytestmark = pytest.mark.gpu


def walk(cu, parents, drafted, sampled, pending, most):
    acc, nxt, paths = [], [], []
    for i, want in enumerate(pending):
        n = min(cu[i + 1] - cu[i], most)
        up = [p if -1 <= p < j else -1 for j, p in enumerate(parents[cu[i]:cu[i] + n])]
        at, path = -1, []
        while True:
            fit = [j for j in range(n) if up[j] == at and drafted[cu[i] + j] == want and want >= 0]
            if not fit:
                break
            at = fit[0]
            path.append(at)
            want = sampled[cu[i] + at]
        acc.append(at)
        nxt.append(want)
        paths.append(path + [-1] * (most - len(path)))
    return np.array(acc), np.array(nxt), np.array(paths)


def run(cu, parents, drafted, sampled, pending, most, path=True, in_place=False):
    import torch

    import gated_delta_rule_conv_amd as gdn

    dev = lambda a: None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    pend, m = dev(pending), len(pending)
    acc = torch.full((m,), -5, dtype=torch.int32, device="cuda")
    nxt = pend if in_place else torch.full((m,), -5, dtype=torch.int32, device="cuda")
    nodes = torch.full((m, most), -5, dtype=torch.int32, device="cuda") if path else None
    gdn.tree_follow(dev(drafted), dev(sampled), pend, dev(parents), dev(cu), most, acc, nxt, path=nodes)
    torch.cuda.synchronize()
    return acc.cpu().numpy(), nxt.cpu().numpy(), None if nodes is None else nodes.cpu().numpy()


def trees(m, most, seed, chain=False, tokens=3):
    """Few different tokens, so that paths are long and siblings often equal."""
    r = np.random.default_rng(seed)
    lens = r.integers(0, most + 1, m)
    cu = np.concatenate([[0], np.cumsum(lens)])
    parents = np.concatenate([[j - 1 if chain else int(r.integers(-1, j)) for j in range(n)] for n in lens] + [[]]).astype(int)
    T = cu[-1]
    return cu, parents, r.integers(0, tokens, T), r.integers(0, tokens, T), r.integers(0, tokens, m)


@pytest.mark.parametrize("m,most", [(1, 1), (1, 4), (3, 5), (64, 16), (513, 64), (7, 64)])
@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("tokens", [1, 2, 5])
def test_paths(m, most, chain, tokens):
    announce(f"follow {m} x {most} chain={chain} tokens={tokens}")
    t = trees(m, most, m * 100 + most, chain, tokens)
    want = walk(*t, most)
    for kw in (dict(), dict(path=False), dict(in_place=True)):
        got = run(*t, most, **kw)
        for a, b in zip(got, want):
            assert a is None or (a == b).all()
    if chain:
        got = run(t[0], None, *t[2:], most)
        assert all((a == b).all() for a, b in zip(got, want))


def test_odd_trees():
    """Parents that are none count as the slot; negative tokens are never followed; trees longer than max_nodes are cut; no nodes at all."""
    announce("follow: odd trees")
    cu, parents = [0, 6, 6, 8], [-9, 5, 0, 3, 1, 2, -1, 0]
    drafted, sampled, pending = [4, 4, 5, 5, 5, 6, -1, 2], [5, 5, 6, 6, -1, 7, 2, 9], [4, 8, -1]
    want = walk(cu, parents, drafted, sampled, pending, 8)
    got = run(cu, parents, drafted, sampled, pending, 8)
    assert all((a == b).all() for a, b in zip(got, want))
    assert got[0].tolist()[1:] == [-1, -1] and got[1].tolist()[1:] == [8, -1]
    want = walk(cu, parents, drafted, sampled, pending, 2)
    got = run(cu, parents, drafted, sampled, pending, 2)
    assert all((a == b).all() for a, b in zip(got, want))
    none = run([0, 0, 0], [], [], [], [3, 4], 4)
    assert none[0].tolist() == [-1, -1] and none[1].tolist() == [3, 4] and (none[2] == -1).all()
