"""The slot operators run as a serving loop runs them: a stored prefix into slots, drafts
verified, their outputs normed, the accepted paths taken, a plain decode step, and the slots stored
again -- against the fp64 oracle fed the accepted tokens one by one from the stored (quantised)
states.

Tolerances: as the parts' own tests: 1e-5 of a block's largest element for o and the states (fp32 paths),
and for the normed output 2^-8 of the value (its bf16 rounding) and 1e-5 of the group's root mean square,
times the weight and the gate, for o's own error."""

import numpy as np
import pytest

from gen import DECODE_M16_POOL64, make_decode_pool, make_decode_step
from gen.inputs import LayerShape, _store
from oracle import decode_layer, storage_to_f64
from tests.gpu_helpers import TOL_F32, announce, bits_of, normwise_err, storage_of, to_dev

pytestmark = pytest.mark.gpu


def test_restore_verify_norm_accept_decode_store():
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce("speculative run: 3 slots from 2 snapshots, 3 rounds")
    sh = LayerShape(2, 4, 128, in_dtype="bf16")
    dims = gdn.make_dims(2, 4, 128, in_dtype=gdn.GDN_BF16)
    nd = gdn.make_norm_dims(4, 128)
    base = make_decode_pool(DECODE_M16_POOL64, pool=6, shape=sh)
    pool = gdn.SlotPool(dims, 6, state=to_dev(base["S"], "f32"), conv_state=to_dev(base["conv_state"], "bf16"))
    w = to_dev(base["conv_w"], "bf16")
    store = gdn.packed_slots(dims, 4, gdn.GDN_PACK_INT8)

    def idx(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    pool.pack_slots(idx([5, 3]), store, gdn.GDN_PACK_INT8)
    slots = [0, 1, 4]
    pool.unpack_slots(store, idx([0, 1, 0]), idx(slots), gdn.GDN_PACK_INT8)
    torch.cuda.synchronize()
    S = [pool.state[s].cpu().numpy().astype(np.float64) for s in slots]
    cs = [storage_of(pool.conv_state[s], "bf16") for s in slots]
    step_of_row = np.abs(base["S"][[5, 3, 5]]).max(-1, keepdims=True) / 254
    assert (np.abs(np.stack(S) - base["S"][[5, 3, 5]]) <= step_of_row * 1.0001).all()
    sp, cp = pool.pointers(idx(slots))
    r = np.random.default_rng(21)
    kw = dict(in_dtype="bf16")

    for turn in range(3):
        lens = [int(v) for v in r.integers(1, 20, 3)]
        T = sum(lens)
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        par = np.concatenate([[int(r.integers(-1, t)) if t else -1 for t in range(n)] for n in lens]).astype(np.int32)
        x = _store(r.standard_normal((T, sh.channels)), "bf16")
        z = _store(r.standard_normal((T, 512)), "bf16")
        nw = _store(1 + 0.1 * r.standard_normal(128), "bf16")
        g = (-np.logaddexp(0, r.standard_normal((T, 4))) * 0.2).astype(np.float32)
        beta = (1 / (1 + np.exp(-r.standard_normal((T, 4))))).astype(np.float32)
        dx, dpar, dcu = to_dev(x, "bf16"), torch.tensor(par, device="cuda"), torch.tensor(cu, device="cuda")
        o = torch.empty((T, 4, 128), device="cuda")
        y = torch.empty((T, 512), dtype=torch.bfloat16, device="cuda")
        rec = gdn.tree_record(dims, T)
        gdn.tree_verify(dims, dx, w, None, to_dev(g, "f32"), to_dev(beta, "f32"), o, dpar, dcu, max(lens), sp, cp, record=rec)
        gdn.group_norm(nd, o, to_dev(nw, "bf16"), y, gate=to_dev(z, "bf16"))
        last = [int(r.integers(-1, n)) for n in lens]
        gdn.tree_accept(dims, dx, rec, dpar, dcu, max(lens), idx(last), sp, cp)
        torch.cuda.synchronize()
        got = y.float().cpu().numpy().reshape(T, 4, 128).astype(np.float64)
        for i, n in enumerate(lens):
            after = {-1: (S[i], cs[i])}
            for t in range(n):
                a = cu[i] + t
                S0, c0 = after[int(par[a])]
                res = decode_layer(x[a:a + 1], base["conv_w"], c0[None], S0[None], g[a:a + 1], beta[a:a + 1], 2, 4, 128, **kw)
                after[t] = (res["S"][0], np.concatenate([c0[1:], x[a:a + 1]]))
                for j in range(4):
                    ref = res["o"][0, j]
                    assert normwise_err(o[a, j].cpu().numpy(), ref) <= 3 * TOL_F32  # (one token's o, not a block's)
                    zz = storage_to_f64(z[a, 128 * j:128 * j + 128], "bf16")
                    f = storage_to_f64(nw, "bf16") * zz / (1 + np.exp(-zz))
                    rs = 1 / np.sqrt((ref ** 2).mean() + 1e-6)
                    room = 3 * TOL_F32 * np.abs(ref).max() * rs * 2 * np.abs(f)
                    assert (np.abs(got[a, j] - ref * rs * f) <= room + (np.abs(ref * rs * f) + room) * 2.0 ** -8).all()
            S[i], cs[i] = after[last[i]]
        for i, s in enumerate(slots):
            for j in range(4):
                assert normwise_err(pool.state[s, j].cpu().numpy(), S[i][j]) <= 2 * TOL_F32 * (turn + 1)
            np.testing.assert_array_equal(storage_of(pool.conv_state[s], "bf16"), cs[i])
        # the token after the accepted ones, drawn by the model itself: an ordinary decode step
        st = make_decode_step(DECODE_M16_POOL64, turn, 3, shape=sh)
        o1 = torch.empty((3, 4, 128), device="cuda")
        gdn.decode_fused(dims, to_dev(st["x"], "bf16"), w, None, to_dev(st["g"], "f32"), to_dev(st["beta"], "f32"), o1, sp, cp)
        torch.cuda.synchronize()
        ref = decode_layer(st["x"], base["conv_w"], np.stack(cs), np.stack(S), st["g"], st["beta"], 2, 4, 128, **kw)
        for i in range(3):
            for j in range(4):
                assert normwise_err(o1[i, j].cpu().numpy(), ref["o"][i, j]) <= 3 * TOL_F32 * (turn + 1)
            S[i], cs[i] = ref["S"][i], np.concatenate([cs[i][1:], st["x"][i:i + 1]])

    # store them again, beside the first two, and bring one back elsewhere
    pool.pack_slots(idx(slots), store, gdn.GDN_PACK_INT8)
    pool.unpack_slots(store, idx([2]), idx([2]), gdn.GDN_PACK_INT8)
    torch.cuda.synchronize()
    room = np.abs(S[2]).max(-1, keepdims=True) / 254 + 12 * TOL_F32 * np.abs(S[2]).max()
    assert (np.abs(pool.state[2].cpu().numpy() - S[2]) <= room).all()
    np.testing.assert_array_equal(bits_of(pool.conv_state[2]), bits_of(pool.conv_state[4]))
