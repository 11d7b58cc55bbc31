"""gdn_tree_verify and gdn_tree_accept against the fp64 oracle, one decode step per tree node
from its parent's state.

Tolerances: an output element is a sum of at most d = 128 products with the state and N = 64 with
other nodes, each accumulated in fp32 from factors rounded in fp32 (2^-24 a rounding), after a
128-term norm; independent roundings give about sqrt(3 * 192) * 2^-24 = 1.5e-6 of the largest terms, and
seven times that is the gate of the fp32 paths, 1e-5 of the largest element of a (slot, v-head)
block. bf16 outputs add half a step, 2^-8 of the value. Conv states and untouched rows: bits.
"""

import numpy as np
import pytest

from gen.inputs import LayerShape, _store
from oracle import decode_layer, storage_to_f64
from tests.gpu_helpers import TOL_F32, announce, bits_of, normwise_err, to_dev

pytestmark = pytest.mark.gpu

SENTINEL = 12345.0


def make_parents(rng, n, kind):
    if kind == "chain":
        return np.arange(n) - 1
    if kind == "star":
        return np.full(n, -1)
    if kind == "two":  # two interleaved chains
        return np.maximum(np.arange(n) - 2, -1)
    return np.array([rng.integers(-1, t) if t else -1 for t in range(n)])


def make_case(shape, lens, kind="tree", seed=0, slow=1.0, bias=False, stride_pad=0):
    r = np.random.default_rng([77, seed])
    C, K, d, Hk, Hv = shape.channels, shape.conv_width, shape.head_dim, shape.num_k_heads, shape.num_v_heads
    m, T = len(lens), int(sum(lens))
    pool = m + 2
    c = dict(shape=shape, lens=list(lens), cu=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    c["parents"] = np.concatenate([make_parents(r, n, kind) for n in lens] or [np.zeros(0)]).astype(np.int32)
    c["x"] = _store(r.standard_normal((T, C)), shape.in_dtype)
    c["pad"] = stride_pad
    c["conv_w"] = _store(r.uniform(-0.5, 0.5, (C, K)), shape.in_dtype)
    c["conv_b"] = _store(r.uniform(-0.5, 0.5, (C,)), shape.in_dtype) if bias else None
    c["g"] = (-np.logaddexp(0.0, r.standard_normal((T, Hv))) * slow).astype(np.float32)
    c["beta"] = (1.0 / (1.0 + np.exp(-r.standard_normal((T, Hv))))).astype(np.float32)
    c["S"] = (r.standard_normal((pool, Hv, d, d)) * 0.05).astype(np.float32)
    c["cs"] = _store(r.standard_normal((pool, K - 1, C)), shape.in_dtype)
    c["slots"] = r.permutation(pool)[:m]
    return c


def oracle_tree(c, kw):
    """Per node: o, the state after it, and the conv state after it (bits)."""
    sh = c["shape"]
    T = len(c["parents"])
    o, S, cs = np.zeros((T, sh.num_v_heads, sh.head_dim)), [None] * T, [None] * T
    for i, slot in enumerate(c["slots"]):
        a = int(c["cu"][i])
        for t in range(c["lens"][i]):
            p = int(c["parents"][a + t])
            S0, cs0 = (c["S"][slot], c["cs"][slot]) if p < 0 else (S[a + p], cs[a + p])
            r = decode_layer(c["x"][a + t:a + t + 1], c["conv_w"], cs0[None], np.asarray(S0)[None],
                             c["g"][a + t:a + t + 1], c["beta"][a + t:a + t + 1], sh.num_k_heads, sh.num_v_heads,
                             sh.head_dim, conv_b=c["conv_b"], in_dtype=sh.in_dtype, **kw)
            o[a + t], S[a + t] = r["o"][0], r["S"][0]
            cs[a + t] = np.concatenate([cs0[1:], c["x"][a + t:a + t + 1]])
    return o, S, cs


def device(c, dims):
    import torch

    import gated_delta_rule_conv_amd as gdn

    sh = c["shape"]
    T, C = c["x"].shape
    e = dict(dims=dims, T=T, m=len(c["lens"]), mx=max([1, *c["lens"]]))
    wide = torch.zeros((T, C + c["pad"]), dtype=torch.bfloat16 if sh.in_dtype == "bf16" else torch.float32, device="cuda")
    wide[:, :C] = to_dev(c["x"], sh.in_dtype)
    e["x"] = wide[:, :C]
    e["w"], e["b"] = to_dev(c["conv_w"], sh.in_dtype), to_dev(c["conv_b"], sh.in_dtype)
    e["g"], e["beta"] = to_dev(c["g"], "f32"), to_dev(c["beta"], "f32")
    e["parents"] = torch.tensor(c["parents"], dtype=torch.int32, device="cuda")
    e["cu"] = torch.tensor(c["cu"], dtype=torch.int32, device="cuda")
    e["pool"] = gdn.SlotPool(dims, len(c["S"]), state=to_dev(c["S"], "f32"), conv_state=to_dev(c["cs"], sh.in_dtype))
    e["sp"], e["cp"] = e["pool"].pointers(torch.tensor(c["slots"], dtype=torch.int32, device="cuda"))
    e["o"] = torch.full((T, sh.num_v_heads, sh.head_dim), SENTINEL, device="cuda",
                        dtype=torch.bfloat16 if dims.out_dtype == gdn.GDN_BF16 else torch.float32)
    e["rec"] = tuple(t.fill_(SENTINEL) for t in gdn.tree_record(dims, T))
    return e


def verify(e, record=True, **kw):
    import gated_delta_rule_conv_amd as gdn

    e = dict(e, **kw)
    gdn.tree_verify(e["dims"], e["x"], e["w"], e["b"], e["g"], e["beta"], e["o"], e["parents"], e["cu"], e["mx"], e["sp"],
                    e["cp"], record=e["rec"] if record else None, stream=e.get("stream"))


def accept(e, accepted, **kw):
    import torch

    import gated_delta_rule_conv_amd as gdn

    e = dict(e, **kw)
    if not torch.is_tensor(accepted):
        accepted = torch.tensor(accepted, dtype=torch.int32, device="cuda")
    gdn.tree_accept(e["dims"], e["x"], e["rec"], e["parents"], e["cu"], e["mx"], accepted, e["sp"], e["cp"],
                    stream=e.get("stream"))


def make_dims(sh, **kw):
    import gated_delta_rule_conv_amd as gdn

    return gdn.make_dims(sh.num_k_heads, sh.num_v_heads, sh.head_dim, conv_width=sh.conv_width,
                         in_dtype=gdn.GDN_BF16 if sh.in_dtype == "bf16" else gdn.GDN_F32, **kw)


def check_o(c, got, want, tol, extra=0.0):
    got = got.float().cpu().numpy().astype(np.float64)
    for i in range(len(c["lens"])):
        a, b = c["cu"][i], c["cu"][i + 1]
        for j in range(want.shape[1] if b > a else 0):
            w = want[a:b, j]
            off = np.abs(got[a:b, j] - w) - extra * np.abs(w)
            assert off.max() <= tol * np.abs(w).max(), (i, j, off.max(), np.abs(w).max())


CASES = [
    # hk, hv, d, dtype, K, lens, kind, options
    (1, 1, 32, "f32", 4, [1], "tree", {}),
    (2, 2, 32, "f32", 2, [16, 0, 15, 1], "tree", {}),
    (1, 3, 32, "bf16", 3, [17, 31, 32], "tree", dict(bias=True, silu=True)),
    (2, 4, 64, "f32", 4, [33, 5], "chain", dict(pad=12)),
    (2, 2, 64, "bf16", 4, [64, 48, 49], "tree", dict(out="bf16")),
    (1, 2, 128, "bf16", 4, [64, 64], "chain", dict(slow=0.01)),
    (2, 4, 128, "bf16", 4, [16, 7, 0, 12, 1], "tree", dict(pad=64, scale=0.37)),
    (1, 2, 128, "f32", 4, [40, 64], "two", dict(slow=0.01, silu=True)),
    (3, 6, 128, "bf16", 2, [20, 32], "star", dict(bias=True)),
    (1, 4, 128, "f32", 3, [9], "tree", dict(norm=False)),
]


@pytest.mark.parametrize("hk,hv,d,dtype,K,lens,kind,opt", CASES)
def test_verify_then_accept_against_the_oracle(hk, hv, d, dtype, K, lens, kind, opt):
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce(f"tree {kind} {lens} hk={hk} hv={hv} d={d} {dtype} K={K} {opt}")
    sh = LayerShape(hk, hv, d, conv_width=K, in_dtype=dtype)
    c = make_case(sh, lens, kind, seed=d + sum(lens), slow=opt.get("slow", 1.0), bias=opt.get("bias", False),
                  stride_pad=opt.get("pad", 0))
    norm = opt.get("norm", True)
    if not norm:  # |k|^2 near 1, as a caller of this option has it
        c["x"] = _store(storage_to_f64(c["x"], dtype) / np.sqrt(d), dtype)
        c["cs"] = _store(storage_to_f64(c["cs"], dtype) / np.sqrt(d), dtype)
    dims = make_dims(sh, activation=gdn.GDN_ACT_SILU if opt.get("silu") else gdn.GDN_ACT_NONE, scale=opt.get("scale", 1.0),
                     out_dtype=gdn.GDN_BF16 if opt.get("out") == "bf16" else gdn.GDN_F32, qk_l2norm=norm)
    o, S, cs = oracle_tree(c, dict(activation="silu" if opt.get("silu") else "none", scale=opt.get("scale", 1.0),
                                   qk_l2norm=norm))
    e = device(c, dims)
    S0, cs0 = bits_of(e["pool"].state), bits_of(e["pool"].conv_state)
    verify(e)
    torch.cuda.synchronize()
    check_o(c, e["o"], o, TOL_F32, 2.0 ** -8 if opt.get("out") == "bf16" else 0.0)
    np.testing.assert_array_equal(bits_of(e["pool"].state), S0)
    np.testing.assert_array_equal(bits_of(e["pool"].conv_state), cs0)
    # without the record: the same bits
    o1 = bits_of(e["o"])
    e["o"].fill_(SENTINEL)
    verify(e, record=False)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits_of(e["o"]), o1)

    r = np.random.default_rng(5)
    for take in ("last", "random", "none"):
        last = [n - 1 if take == "last" else int(r.integers(-1, n)) if take == "random" and n else -1 for n in lens]
        f = device(c, dims)
        accept(dict(f, rec=e["rec"]), last)
        torch.cuda.synchronize()
        got, gcs = f["pool"].state.cpu().numpy(), bits_of(f["pool"].conv_state)
        moved = set()
        for i, slot in enumerate(c["slots"]):
            if last[i] < 0:
                continue
            moved.add(slot)
            t = c["cu"][i] + last[i]
            for j in range(hv):
                assert normwise_err(got[slot, j], S[t][j]) <= TOL_F32, (take, i, j)
            want = cs[t].view(np.int16) if dtype == "bf16" else cs[t].view(np.int32)
            np.testing.assert_array_equal(gcs[slot], want)
        still = [s for s in range(len(c["S"])) if s not in moved]
        np.testing.assert_array_equal(bits_of(f["pool"].state)[still], S0[still])
        np.testing.assert_array_equal(gcs[still], cs0[still])


def _rig(lens, kind="tree", seed=3, shape=None, **kw):
    sh = shape or LayerShape(2, 4, 128, in_dtype="bf16")
    c = make_case(sh, lens, kind, seed=seed)
    return c, device(c, make_dims(sh, **kw))


def test_a_slot_alone_gives_the_bits_it_gives_in_a_batch():
    """... and whatever max_nodes the call names."""
    import torch

    announce("tree: batch invariance")
    c, e = _rig([13, 16, 40, 1, 0, 29])
    verify(e)
    accept(e, [5, -1, 39, 0, -1, 7])
    torch.cuda.synchronize()
    whole, rec, S = bits_of(e["o"]), [bits_of(t) for t in e["rec"]], bits_of(e["pool"].state)
    for i in (0, 2, 5):
        for mx in (c["lens"][i], 64):
            f = device(c, e["dims"])
            a, b = int(c["cu"][i]), int(c["cu"][i + 1])
            one = dict(x=f["x"][a:b], g=f["g"][a:b], beta=f["beta"][a:b], o=f["o"][a:b], parents=f["parents"][a:b],
                       rec=tuple(t[a:b] for t in f["rec"]), cu=torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
                       sp=f["sp"][i:i + 1], cp=f["cp"][i:i + 1], mx=mx)
            verify(f, **one)
            accept(f, [[5, -1, 39, 0, -1, 7][i]], **one)
            torch.cuda.synchronize()
            np.testing.assert_array_equal(bits_of(f["o"])[a:b], whole[a:b])
            for t, want in zip(f["rec"], rec):
                np.testing.assert_array_equal(bits_of(t)[a:b], want[a:b])
            slot = c["slots"][i]
            np.testing.assert_array_equal(bits_of(f["pool"].state)[slot], S[slot])


@pytest.mark.parametrize("hk,hv,d,dtype,m,top", [
    (32, 64, 32, "bf16", 9, 16),
    (16, 48, 32, "f32", 12, 40),   # groups of three: a pair and one alone
    (32, 32, 64, "bf16", 9, 30),   # one v-head a k-head
    (16, 32, 64, "f32", 17, 64),
    (16, 32, 128, "bf16", 17, 16),
    (16, 48, 128, "bf16", 9, 32),
    (8, 24, 128, "bf16", 17, 64),  # larger trees, a pair and one alone
    (8, 16, 128, "f32", 33, 50),
])
def test_large_batches_give_the_bits_of_single_slots(hk, hv, d, dtype, m, top):
    """From m * hk * ceil(hv / hk / 2) = 256 on a workgroup takes two v-heads of a k-head (below, as
    in every one-slot call here, one): the same bits for every slot."""
    import torch

    announce(f"tree: batch of {m}, hk={hk} hv={hv} d={d} {dtype} up to {top} nodes")
    r = np.random.default_rng(d + m)
    lens = [top] + [int(v) for v in r.integers(0, top + 1, m - 1)]
    assert m * hk * ((hv // hk + 1) // 2) >= 256
    c, e = _rig(lens, seed=m, shape=LayerShape(hk, hv, d, in_dtype=dtype))
    last = [int(r.integers(-1, n)) if n else -1 for n in lens]
    verify(e)
    accept(e, last)
    torch.cuda.synchronize()
    f = device(c, e["dims"])
    for i in range(m):
        a, b = int(c["cu"][i]), int(c["cu"][i + 1])
        if a == b:
            continue
        one = dict(x=f["x"][a:b], g=f["g"][a:b], beta=f["beta"][a:b], o=f["o"][a:b], parents=f["parents"][a:b],
                   rec=tuple(t[a:b] for t in f["rec"]), cu=torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
                   sp=f["sp"][i:i + 1], cp=f["cp"][i:i + 1], mx=b - a)
        verify(f, **one)
        accept(f, [last[i]], **one)
    torch.cuda.synchronize()
    assert torch.equal(e["o"], f["o"])
    for x, y in zip(e["rec"], f["rec"]):
        assert torch.equal(x, y)
    assert torch.equal(e["pool"].state, f["pool"].state)
    assert torch.equal(e["pool"].conv_state, f["pool"].conv_state)


def test_no_parents_is_a_chain():
    import torch

    announce("tree: parents None")
    c, e = _rig([30, 4, 17], "chain")
    verify(e)
    accept(e, [29, 2, -1])
    f = device(c, e["dims"])
    verify(f, parents=None)
    accept(f, [29, 2, -1], parents=None)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits_of(e["o"]), bits_of(f["o"]))
    np.testing.assert_array_equal(bits_of(e["pool"].state), bits_of(f["pool"].state))
    np.testing.assert_array_equal(bits_of(e["pool"].conv_state), bits_of(f["pool"].conv_state))


def test_inactive_slots_and_rows_outside_the_trees_stay():
    """A 0 in either pointer array, rows past max_nodes, rows no tree owns, and cu_nodes entries
    outside the packed rows: nothing of theirs is written."""
    import torch

    announce("tree: inactive slots, clipped trees")
    c, e = _rig([10, 20, 12, 18])
    whole = device(c, e["dims"])
    verify(whole)
    e["sp"][1] = 0
    e["cp"][3] = 0
    S0, cs0 = bits_of(e["pool"].state), bits_of(e["pool"].conv_state)
    verify(e, mx=11)
    torch.cuda.synchronize()
    o, want = e["o"].cpu(), whole["o"].cpu()
    assert torch.equal(o[:10], want[:10]) and torch.equal(o[30:41], want[30:41])
    assert (o[10:30] == SENTINEL).all() and (o[41:] == SENTINEL).all()
    for t in e["rec"]:
        assert (t[10:30] == SENTINEL).all() and (t[41:] == SENTINEL).all()
    accept(e, [9, 3, 11, 2], mx=11)  # slot 2's tree holds 11 nodes in this call: number 11 is not one
    torch.cuda.synchronize()
    moved = c["slots"][0]
    keep = [s for s in range(len(c["S"])) if s != moved]
    np.testing.assert_array_equal(bits_of(e["pool"].state)[keep], S0[keep])
    np.testing.assert_array_equal(bits_of(e["pool"].conv_state)[keep], cs0[keep])
    assert not np.array_equal(bits_of(e["pool"].state)[moved], S0[moved])
    f = device(c, e["dims"])
    bad = torch.tensor([-5, 10, 100, 90, 4], dtype=torch.int32, device="cuda")
    verify(f, cu=bad, mx=64)
    torch.cuda.synchronize()
    assert (f["o"][:10] == SENTINEL).all()  # slot 0 begins before the rows, 2 and 3 past or backwards


def test_parents_outside_their_tree_read_as_roots():
    import torch

    announce("tree: odd parents")
    c, e = _rig([20, 9])
    p = c["parents"].copy()
    p[3], p[7], p[25] = -9, 7, 1 << 30
    q = p.copy()
    q[[3, 7, 25]] = -1
    f = device(c, e["dims"])
    for x, par in ((e, p), (f, q)):
        par = torch.tensor(par, device="cuda")
        verify(x, parents=par)
        accept(x, [7, 5], parents=par)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits_of(e["o"]), bits_of(f["o"]))
    np.testing.assert_array_equal(bits_of(e["pool"].state), bits_of(f["pool"].state))
    np.testing.assert_array_equal(bits_of(e["pool"].conv_state), bits_of(f["pool"].conv_state))


@pytest.mark.parametrize("where", ["k", "q", "v", "all"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_broken_token_reaches_only_its_descendants(where, bad):
    import torch

    announce(f"tree: {bad} in {where} of one node")
    sh = LayerShape(1, 2, 64, conv_width=2, in_dtype="f32")
    c = make_case(sh, [24, 40], "tree", seed=11)
    e = device(c, make_dims(sh))
    verify(e)
    f = device(c, e["dims"])
    node = 24 + 5
    col = {"k": slice(64, 65), "q": slice(3, 4), "v": slice(128 + 64 + 9, 128 + 64 + 10), "all": slice(0, 256)}[where]
    f["x"][node, col] = bad
    verify(f)
    torch.cuda.synchronize()
    hit = set()
    for t in range(40):  # the token is seen by itself, its children (conv) and their descendants
        p = int(c["parents"][24 + t])
        if t == 5 or p in hit:
            hit.add(t)
    for t in range(64):
        o, clean = f["o"][t], e["o"][t]
        if t < 24 or t - 24 not in hit:
            assert torch.equal(o, clean), t
        elif where == "v":
            others = [r for r in range(64) if r != 9]
            assert torch.equal(o[0], clean[0]) and torch.equal(o[1][others], clean[1][others])
            assert torch.isnan(o[1][9]), t
        elif where != "q":
            assert torch.isnan(o).all(), t
    if where == "q":
        assert torch.isnan(f["o"][node]).all()
    # a path around the broken node is accepted as if it were not there
    ok = max(t for t in range(40) if t not in hit)
    accept(e, [3, ok])
    accept(f, [3, ok])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits_of(e["pool"].state), bits_of(f["pool"].state))


def test_graph_replays_match_eager_calls():
    """verify + accept captured once: every replay moves the slots as the eager calls do."""
    import torch

    announce("tree: graph replay")
    c, e = _rig([16, 9, 31])
    last = torch.tensor([3, -1, 12], dtype=torch.int32, device="cuda")
    want = []
    for _ in range(3):
        verify(e)
        accept(e, last)
        torch.cuda.synchronize()
        want.append([bits_of(t) for t in (e["o"], e["pool"].state, e["pool"].conv_state)])
    f = device(c, e["dims"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        verify(f)
        accept(f, last)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert float(torch.ones(1 << 16, device="cuda").sum().item()) == float(1 << 16)
        for t, b in zip((f["o"], f["pool"].state, f["pool"].conv_state), want[i]):
            np.testing.assert_array_equal(bits_of(t), b)


def test_two_streams_at_once():
    import torch

    announce("tree: two streams")
    c, e = _rig([33, 20], seed=8)
    c2, e2 = _rig([16, 48, 3], seed=9)
    verify(e)
    verify(e2)
    accept(e, [30, 2])
    accept(e2, [4, 40, 0])
    torch.cuda.synchronize()
    f, f2 = device(c, e["dims"]), device(c2, e2["dims"])
    torch.cuda.synchronize()
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        verify(f)
        accept(f, torch.tensor([30, 2], dtype=torch.int32, device="cuda"))
    verify(f2, stream=s2)
    with torch.cuda.stream(s2):
        accept(f2, torch.tensor([4, 40, 0], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for a, b in ((e, f), (e2, f2)):
        np.testing.assert_array_equal(bits_of(a["o"]), bits_of(b["o"]))
        np.testing.assert_array_equal(bits_of(a["pool"].state), bits_of(b["pool"].state))


def test_rows_beyond_32_bit_offsets():
    """x rows 2^28 elements apart: element offsets pass 2^32."""
    import torch

    announce("tree: far rows")
    sh = LayerShape(1, 1, 32, in_dtype="bf16")
    c = make_case(sh, [18, 2], seed=4)
    e = device(c, make_dims(sh))
    verify(e)
    accept(e, [17, 1])
    f = device(c, e["dims"])
    far = torch.empty((20 << 28) + 128, dtype=torch.bfloat16, device="cuda")
    x = far.as_strided((20, sh.channels), (1 << 28, 1))
    x.copy_(f["x"])
    verify(f, x=x)
    accept(f, [17, 1], x=x)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits_of(e["o"]), bits_of(f["o"]))
    np.testing.assert_array_equal(bits_of(e["pool"].conv_state), bits_of(f["pool"].conv_state))


def test_two_slots_may_verify_on_one_state():
    import torch

    announce("tree: shared state")
    c, e = _rig([8, 8])
    e["sp"][1], e["cp"][1] = e["sp"][0], e["cp"][0]
    for k in ("x", "g", "beta", "parents"):
        e[k][8:] = e[k][:8]
    verify(e)
    torch.cuda.synchronize()
    o = bits_of(e["o"])
    np.testing.assert_array_equal(o[:8], o[8:])


@pytest.mark.parametrize("d,dtype", [(32, "f32"), (128, "bf16")])
@pytest.mark.parametrize("kind", ["same", "two", "signs"])
def test_drafts_that_repeat_their_keys(d, dtype, kind):
    """Chains and trees whose keys are one direction, two in turn, or one with changing signs, next to no decay
    and write strengths of 1: the triangular system at its fullest (every entry below the diagonal near
    +-1 or 0). The rule is stable there (I + the lower part of a Gram matrix has an inverse of norm at most
    2), so the usual gate holds."""
    import torch

    announce(f"tree: repeated keys {kind} d={d}")
    sh = LayerShape(1, 2, d, conv_width=2, in_dtype=dtype)
    c = make_case(sh, [64, 50], "chain" if kind != "two" else "tree", seed=6)
    r = np.random.default_rng(3)
    x = storage_to_f64(c["x"], dtype)
    two = r.standard_normal((2, d))
    for t in range(len(x)):
        x[t, d:2 * d] = two[0] if kind == "same" else two[t % 2] if kind == "two" else two[0] * r.choice([-1, 1])
    c["x"] = _store(x, dtype)
    w = np.zeros((sh.channels, 2))
    w[:, 1] = 1.0  # the conv hands the token on
    c["conv_w"] = _store(w, dtype)
    c["g"][:] = -1e-4
    c["beta"][:] = 1.0
    dims = make_dims(sh)
    o, S, cs = oracle_tree(c, {})
    e = device(c, dims)
    verify(e)
    last = [63, 49]
    accept(e, last)
    torch.cuda.synchronize()
    check_o(c, e["o"], o, TOL_F32)
    got = e["pool"].state.cpu().numpy()
    for i, slot in enumerate(c["slots"]):
        for j in range(2):
            assert normwise_err(got[slot, j], S[c["cu"][i] + last[i]][j]) <= TOL_F32


def test_as_many_slots_as_a_call_takes():
    """65535 slots of one node each, on one state: equal rows for equal tokens."""
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce("tree: 65535 slots")
    sh = LayerShape(1, 1, 32, in_dtype="bf16")
    c = make_case(sh, [1], seed=2)
    e = device(c, make_dims(sh))
    verify(e)
    m = 65535
    many = {k: e[k].expand(m, *e[k].shape[1:]).contiguous() for k in ("x", "g", "beta", "o", "parents", "sp", "cp")}
    many["cu"] = torch.arange(m + 1, dtype=torch.int32, device="cuda")
    rec = gdn.tree_record(e["dims"], m)
    verify(dict(e, rec=rec), **many)
    torch.cuda.synchronize()
    assert torch.equal(many["o"], e["o"].expand_as(many["o"]))
    for a, b in zip(rec, e["rec"]):
        assert torch.equal(a, b.expand_as(a))
