"""8-bit slot snapshots: codes, scales and read-back values against the documented arithmetic.

The arithmetic is elementwise fp32 with one rounding an operation, so int8 codes, scales and the
values read back are compared bit for bit with the same operations in NumPy; e4m3 codes with
torch's conversion on the CPU."""

import numpy as np
import pytest

from tests.gpu_helpers import announce, bits_of

pytestmark = pytest.mark.gpu

TOP = {"int8": np.float32(127.0), "e4m3": np.float32(448.0)}
SHAPES = [(1, 1, 32, "f32", 4), (2, 6, 64, "f32", 3), (16, 32, 128, "bf16", 4), (3, 3, 128, "bf16", 2), (1, 5, 32, "bf16", 4)]


def rig(hk, hv, d, dtype, K, slots, seed=0):
    import torch

    import gated_delta_rule_conv_amd as gdn

    dims = gdn.make_dims(hk, hv, d, conv_width=K, in_dtype=gdn.GDN_BF16 if dtype == "bf16" else gdn.GDN_F32)
    g = torch.Generator().manual_seed(seed)
    state = torch.randn((slots, hv, d, d), generator=g) * torch.exp(torch.randn((slots, hv, d, 1), generator=g) * 3)
    pool = gdn.SlotPool(dims, slots, state=state.cuda())
    pool.conv_state.copy_(torch.randn(pool.conv_state.shape, generator=g).cuda())
    return dims, pool


def fmt_of(name):
    import gated_delta_rule_conv_amd as gdn

    return gdn.GDN_PACK_INT8 if name == "int8" else gdn.GDN_PACK_E4M3


def reference(S, name):
    """codes (as bytes), scales and read-back values of states S [..., d] (float32)."""
    import torch

    a = np.abs(S).max(-1, keepdims=True)
    finite = np.isfinite(S).all(-1, keepdims=True)
    live = finite & (a >= np.float32(2.0 ** -100))
    with np.errstate(all="ignore"):
        t = np.where(live, S * (TOP[name] * (np.float32(1) / np.where(live, a, np.float32(1)))), np.float32(0)).astype(np.float32)
    scale = np.where(live, a / TOP[name], np.where(finite, np.float32(0), np.float32(np.nan))).astype(np.float32)
    if name == "int8":
        q = np.rint(t).astype(np.int8)
        codes, vals = q.view(np.uint8), q.astype(np.float32)
    else:
        q = torch.from_numpy(np.ascontiguousarray(t)).to(torch.float8_e4m3fn)
        vals, codes = q.float().numpy(), q.view(torch.uint8).numpy()
        codes = np.where(live, codes, 0).astype(np.uint8)
    return codes, scale[..., 0], (vals * scale).astype(np.float32)


def idx(v):
    import torch

    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("name", ["int8", "e4m3"])
@pytest.mark.parametrize("hk,hv,d,dtype,K", SHAPES)
def test_pack_and_unpack_are_the_documented_arithmetic(hk, hv, d, dtype, K, name):
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce(f"snapshot {name} hk={hk} hv={hv} d={d} {dtype} K={K}")
    dims, pool = rig(hk, hv, d, dtype, K, 7)
    # special rows: zeros, tiny, the largest, one value alone, ties, infinity, NaN
    s = pool.state
    s[2, 0, 0] = 0
    s[2, 0, 1] = s[2, 0, 1].sign() * 2.0 ** -101
    s[2, 0, 2, :] = 2.0 ** -100
    s[2, 0, 3, 0] = 3.4e38
    s[2, 0, 4] = 0
    s[2, 0, 4, d - 1] = -7.0
    s[2, 0, 5, :] = torch.arange(d, device="cuda") + 0.5
    s[2, 0, 5, 0] = 127.0
    s[2, 0, 6, 5] = float("inf")
    s[2, 0, 7, d - 1] = float("nan")
    s[2, 0, 8, 3] = -float("inf")
    s[2, 0, 9] = 1e-44
    before = bits_of(s), bits_of(pool.conv_state)
    store = gdn.packed_slots(dims, 5, fmt_of(name))
    store.fill_(0xAB)
    slots = [2, 6, 0]
    pool.pack_slots(idx(slots), store, fmt_of(name))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits_of(s), before[0])
    codes, scale, vals = reference(s.cpu().numpy(), name)
    n, rows = hv * d * d, hv * d
    blocks = store.cpu().numpy()
    for i, slot in enumerate(slots):
        np.testing.assert_array_equal(blocks[i, :n], codes[slot].reshape(-1))
        np.testing.assert_array_equal(blocks[i, n:n + 4 * rows].view(np.uint32) & 0x7FFFFFFF,
                                      scale[slot].reshape(-1).view(np.uint32) & 0x7FFFFFFF)
        np.testing.assert_array_equal(blocks[i, n + 4 * rows:],
                                      pool.conv_state[slot].contiguous().view(torch.uint8).cpu().numpy().reshape(-1))
    assert (blocks[3:] == 0xAB).all()

    # read back: block 0 into two slots, block 2 into one; index -1 skips
    pool.unpack_slots(store, idx([0, 2, 0, 1]), idx([4, 1, 5, -1]), fmt_of(name))
    torch.cuda.synchronize()
    got, conv = s.cpu().numpy(), bits_of(pool.conv_state)
    for slot, src in ((4, 2), (1, 0), (5, 2)):
        np.testing.assert_array_equal(got[slot], vals[src])  # (NaN equals NaN here)
        np.testing.assert_array_equal(conv[slot], before[1][src])
    rest = [0, 2, 3, 6]
    np.testing.assert_array_equal(bits_of(s)[rest], before[0][rest])
    np.testing.assert_array_equal(conv[rest], before[1][rest])


@pytest.mark.parametrize("name", ["int8", "e4m3"])
def test_error_of_a_round_trip(name):
    """int8: half a step of the row's scale, a / 254; e4m3: 2^-4 of the value (its half step), or
    half a subnormal step, 2^-10 of the scale. Both with fp32 roundings of 4 x 2^-24 besides."""
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce(f"snapshot round trip {name}")
    dims, pool = rig(2, 4, 128, "bf16", 4, 2)
    s0 = pool.state[0].double().cpu()
    store = gdn.packed_slots(dims, 1, fmt_of(name))
    pool.pack_slots(idx([0]), store, fmt_of(name))
    pool.unpack_slots(store, idx([0]), idx([1]), fmt_of(name))
    torch.cuda.synchronize()
    off = (pool.state[1].double().cpu() - s0).abs()
    a = s0.abs().amax(-1, keepdim=True)
    bound = a / 254 if name == "int8" else torch.maximum(s0.abs() / 16, a / 448 * 2.0 ** -10)
    assert (off <= bound + a * 2.0 ** -22).all()


def test_without_conv_states_their_part_stays():
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce("snapshot: state only, inactive entries")
    dims, pool = rig(2, 2, 64, "bf16", 4, 3)
    fmt = gdn.GDN_PACK_INT8
    store = gdn.packed_slots(dims, 2, fmt)
    store.fill_(7)
    n = 2 * 64 * 64 + 2 * 64 * 4
    pool.pack_slots(idx([0, 9]), store, fmt, conv_state=False)  # slot 9 is outside the pool: skipped
    torch.cuda.synchronize()
    assert (store[0, n:] == 7).all() and (store[1] == 7).all() and not (store[0, :n] == 7).all()
    conv = bits_of(pool.conv_state)
    pool.unpack_slots(store, idx([0]), idx([2]), fmt, conv_state=False)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits_of(pool.conv_state), conv)
    # any 0 pointer skips the whole entry
    sp, cp = pool.pointers(idx([0, 1]))
    cp[1] = 0
    store.fill_(7)
    bp = store.data_ptr() + torch.arange(2, device="cuda") * store.shape[1]
    gdn.slot_pack(dims, fmt, sp, cp, bp)
    torch.cuda.synchronize()
    assert (store[1] == 7).all()


def test_many_blocks_and_a_replayed_graph():
    """More slots than XCDs x workgroups in one call, captured; replays follow the states."""
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce("snapshot: 300 slots, graph")
    dims, pool = rig(1, 2, 32, "f32", 4, 300)
    fmt = gdn.GDN_PACK_E4M3
    store = gdn.packed_slots(dims, 300, fmt)
    sp, cp = pool.pointers(idx(list(range(300))))
    bp = store.data_ptr() + torch.arange(300, device="cuda") * store.shape[1]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.slot_pack(dims, fmt, sp, cp, bp)
        gdn.slot_unpack(dims, fmt, bp, sp, cp)
    for _ in range(3):
        pool.state.mul_(1.7)
        _, _, vals = reference(pool.state.cpu().numpy(), "e4m3")
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(pool.state.cpu().numpy(), vals)
