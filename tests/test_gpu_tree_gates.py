"""gdn_tree_verify and gdn_tree_accept behind strongly forgetting tokens, against the fp64 oracle.

Decays between two nodes are exponentials of sums of g between them. Verification forms those sums
without cancellation, so its gate is the usual one, 1e-5 of the largest element of a (slot, v-head) block. The
record holds the path sums G in fp32: a difference of two is off by half a step of each, at most 2^-18 while |G| <= 128
(and beyond that the sum starts again), so a decay is off by 2 x 2^-18 = 7.6e-6 of itself, which acceptance adds to its gate."""

import numpy as np
import pytest

from gen.inputs import LayerShape
from tests.gpu_helpers import TOL_F32, announce, normwise_err
from tests.test_gpu_tree import accept, check_o, device, make_case, make_dims, oracle_tree, verify

pytestmark = pytest.mark.gpu

TOL_ACCEPT = TOL_F32 + 2.0 ** -17
STRONG = [-20.0, -50.0, -100.0, -127.0, -129.0, -200.0, -1e3, -1e5, -1e9, -3e38]


def run(c, tol_o=TOL_F32, **kw):
    import torch

    sh = c["shape"]
    o, S, cs = oracle_tree(c, {})
    e = device(c, make_dims(sh, **kw))
    verify(e)
    torch.cuda.synchronize()
    check_o(c, e["o"], o, tol_o)
    for last in ([n - 1 for n in c["lens"]], [n // 2 for n in c["lens"]], [n // 3 + 1 for n in c["lens"]]):
        f = device(c, e["dims"])
        accept(dict(f, rec=e["rec"]), last)
        torch.cuda.synchronize()
        got = f["pool"].state.cpu().numpy()
        for i, slot in enumerate(c["slots"]):
            for j in range(sh.num_v_heads):
                assert normwise_err(got[slot, j], S[c["cu"][i] + last[i]][j]) <= TOL_ACCEPT, (last, i, j)
    return e


@pytest.mark.parametrize("strong", STRONG)
@pytest.mark.parametrize("hk,hv,d,dtype,n,kind", [(1, 2, 32, "f32", 64, "chain"), (1, 2, 128, "bf16", 16, "chain"),
                                                   (2, 2, 64, "f32", 40, "tree"), (1, 1, 128, "bf16", 48, "two")])
def test_mild_tokens_after_a_strong_one(hk, hv, d, dtype, n, kind, strong):
    announce(f"tree: one g = {strong}, {kind} of {n}, d={d} {dtype}")
    sh = LayerShape(hk, hv, d, in_dtype=dtype)
    c = make_case(sh, [n, 9], kind, seed=5, slow=0.02)
    c["g"][3] = strong
    c["g"][n + 2, 0] = strong
    run(c)


@pytest.mark.parametrize("hk,hv,d,dtype,n", [(1, 2, 32, "f32", 64), (1, 2, 128, "bf16", 16), (1, 2, 64, "bf16", 32)])
def test_strong_tokens_again_and_again(hk, hv, d, dtype, n):
    """Every fourth token strong, a different strength each time; and every token strong."""
    announce(f"tree: many strong gates, d={d} {dtype} {n} nodes")
    sh = LayerShape(hk, hv, d, in_dtype=dtype)
    for every in (4, 1):
        c = make_case(sh, [n, 7], "chain", seed=9, slow=0.05)
        for i, t in enumerate(range(2, len(c["g"]), every)):
            c["g"][t] = STRONG[(3 * i) % len(STRONG)]
        run(c)


def test_no_token_writes_after_a_strong_one():
    """beta = 0 behind a gate of -70 and one of -20: all that is left is e^-90 of the state, to the gate."""
    announce("tree: nothing but decay")
    sh = LayerShape(1, 2, 32, in_dtype="f32")
    c = make_case(sh, [12, 5], "chain", seed=2, slow=0.01)
    c["beta"][:] = 0.0
    c["g"][1], c["g"][4] = -60.0, -20.0
    run(c)


def test_the_record_of_ordinary_gates_is_the_path_sum():
    """Sums of g down to -128 are recorded as they are, rounded once from a sum kept in two halves."""
    import torch

    announce("tree: record of G")
    sh = LayerShape(1, 2, 32, in_dtype="f32")
    c = make_case(sh, [64, 30], "chain", seed=4)
    e = device(c, make_dims(sh))
    verify(e)
    torch.cuda.synchronize()
    g = c["g"].astype(np.float64)
    want = np.concatenate([np.cumsum(g[:64], 0), np.cumsum(g[64:], 0)])
    got = e["rec"][2].cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= 2.0 ** -24 * 1.001 * np.abs(want)).all()


@pytest.mark.parametrize("first", [-1e9, -150.0])
def test_many_equal_steps_after_a_restart(first):
    """A sum that starts again, falls to -100 at once and then by 0.01 sixty times: each entry is rounded once, not
    once a node on its path."""
    announce(f"tree: g = {first}, -100, then -0.01 sixty times")
    sh = LayerShape(1, 2, 32, in_dtype="f32")
    c = make_case(sh, [64, 9], "chain", seed=14)
    c["g"][:] = -0.01
    c["g"][1], c["g"][2] = first, -100.0
    run(c)
