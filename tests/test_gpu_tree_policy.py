"""gdn_tree_verify's precision policies (gdn_dims.mma): fp32 products keep a row's small values
beside large ones, fp16 pairs keep a value to 2^-37 of its row's norm."""

import numpy as np
import pytest

from gen.inputs import LayerShape, _store
from oracle import storage_to_f64
from tests.gpu_helpers import TOL_F32, announce, normwise_err
from tests.test_gpu_tree import accept, check_o, device, make_case, make_dims, oracle_tree, verify

pytestmark = pytest.mark.gpu


def wide_case(hk, hv, d, dtype, n, seed=8):
    """Every q and k has one value 1e8 times the rest, where the state has zeros; nothing is written
    (beta = 0), so o = e^G S q is a sum of the small values' products alone."""
    sh = LayerShape(hk, hv, d, conv_width=2, in_dtype=dtype)
    c = make_case(sh, [n, 3], "tree", seed=seed)
    x = storage_to_f64(c["x"], dtype)
    for h in range(2 * hk):
        x[:, h * d + 7] = 1e8
    c["x"] = _store(x, dtype)
    w = np.zeros((sh.channels, 2))
    w[:, 1] = 1.0
    c["conv_w"] = _store(w, dtype)
    c["S"][..., 7] = 0.0
    c["beta"][:] = 0.0
    return c


@pytest.mark.parametrize("hk,hv,d,dtype,n", [(1, 2, 32, "f32", 12), (1, 2, 64, "f32", 60), (2, 4, 128, "f32", 16),
                                             (1, 2, 128, "f32", 64), (1, 2, 128, "bf16", 30), (1, 1, 128, "bf16", 64)])
def test_fp32_products_keep_small_values_beside_large_ones(hk, hv, d, dtype, n):
    """fp32 accuracy is relative to the sum of the products' magnitudes: the usual gate."""
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce(f"tree: wide rows, fp32 products, hk={hk} hv={hv} d={d} {dtype} {n} nodes")
    c = wide_case(hk, hv, d, dtype, n)
    o, _, _ = oracle_tree(c, {})
    for mma in ([gdn.GDN_MMA_AUTO] if dtype == "f32" else []) + [gdn.GDN_MMA_FP32]:
        e = device(c, make_dims(c["shape"], mma=mma))
        verify(e)
        torch.cuda.synchronize()
        check_o(c, e["o"], o, TOL_F32)


@pytest.mark.parametrize("hk,hv,d,dtype,lens,kind", [
    (1, 3, 32, "bf16", [17, 31, 0, 32], "tree"), (2, 4, 64, "f32", [33, 5], "chain"), (2, 2, 64, "bf16", [64, 48], "tree"),
    (1, 2, 128, "bf16", [16, 7, 1], "tree"), (1, 3, 128, "f32", [40, 64], "two"), (3, 6, 128, "f32", [20, 32], "star")])
def test_both_policies_against_the_oracle(hk, hv, d, dtype, lens, kind):
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce(f"tree: policies, hk={hk} hv={hv} d={d} {dtype} {lens}")
    sh = LayerShape(hk, hv, d, in_dtype=dtype)
    c = make_case(sh, lens, kind, seed=12, slow=0.3)
    o, S, _ = oracle_tree(c, {})
    outs = []
    for mma in (gdn.GDN_MMA_FP32, gdn.GDN_MMA_BF16X3, gdn.GDN_MMA_AUTO):
        e = device(c, make_dims(sh, mma=mma))
        verify(e)
        last = [n - 1 for n in lens]
        accept(e, last)
        torch.cuda.synchronize()
        check_o(c, e["o"], o, TOL_F32)
        outs.append(e["o"])
        got = e["pool"].state.cpu().numpy()
        for i, slot in enumerate(c["slots"]):
            for j in range(hv if lens[i] else 0):
                assert normwise_err(got[slot, j], S[c["cu"][i] + last[i]][j]) <= TOL_F32
    # the automatic policy is the input type's
    assert torch.equal(outs[2], outs[0] if dtype == "f32" else outs[1])


@pytest.mark.parametrize("d,m,top", [(32, 24, 40), (128, 40, 16), (128, 40, 60)])
def test_fp32_products_give_a_slot_its_bits_in_any_batch(d, m, top):
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce(f"tree: fp32 products, batch of {m}, d={d}")
    sh = LayerShape(8, 24, d, in_dtype="f32")
    r = np.random.default_rng(m)
    lens = [top] + [int(v) for v in r.integers(1, top + 1, m - 1)]
    c = make_case(sh, lens, seed=m)
    e = device(c, make_dims(sh, mma=gdn.GDN_MMA_FP32))
    verify(e)
    f = device(c, e["dims"])
    for i in (0, 1, m - 1):
        a, b = int(c["cu"][i]), int(c["cu"][i + 1])
        verify(f, x=f["x"][a:b], g=f["g"][a:b], beta=f["beta"][a:b], o=f["o"][a:b], parents=f["parents"][a:b],
               rec=tuple(t[a:b] for t in f["rec"]), cu=torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
               sp=f["sp"][i:i + 1], cp=f["cp"][i:i + 1], mx=b - a)
        torch.cuda.synchronize()
        assert torch.equal(e["o"][a:b], f["o"][a:b])
        for s, t in zip(e["rec"], f["rec"]):
            assert torch.equal(s[a:b], t[a:b])
