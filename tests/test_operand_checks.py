"""The tensor helpers hand addresses to the kernels, so they refuse operands of another type, size, layout or
device first (no GPU: operands are host tensors, or stand in for tensors of a GPU, and the launch is watched)."""

import pytest
import torch

import gated_delta_rule_conv_amd as gdn
from gated_delta_rule_conv_amd import _lib

BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


class OnGpu:
    """A host tensor that says it is on a GPU's device."""

    def __init__(self, t, index=0):
        self._t, self._index = t, index

    def __getattr__(self, name):
        return getattr(self._t, name)

    def __getitem__(self, i):
        return OnGpu(self._t[i], self._index)

    def get_device(self):
        return self._index

    @property
    def device(self):
        return torch.device("cuda", self._index)

    @property
    def is_cuda(self):
        return True


@pytest.fixture
def launches(monkeypatch):
    seen = []
    monkeypatch.setattr(_lib, "_launch", lambda name, *a: seen.append(name))
    return seen


def wrong_forms(t, rows_may_be_apart=False):
    """t in another type, one value short, and with gaps."""
    other = {BF16: F32, F32: BF16, I32: I64, I64: I32, torch.uint8: I32}[t.dtype]
    yield "type", t.to(other)
    yield "short", t.reshape(-1)[:-1].clone() if t.dim() == 1 else t[..., :-1].clone()
    yield "gaps", torch.stack([t, t], -1)[..., 0]


def refused_one_at_a_time(operands, call, launches):
    """call(operands) launches once; with any one operand in a wrong form, or on the host, or on another GPU, not."""
    gpu = {k: None if t is None else OnGpu(t) for k, t in operands.items()}
    launches.clear()
    call(gpu)
    assert len(launches) == 1
    for name, t in operands.items():
        if t is None:
            continue
        forms = [(what, OnGpu(w)) for what, w in wrong_forms(t)] + [("host", t), ("elsewhere", OnGpu(t, 1))]
        for what, w in forms:
            with pytest.raises(ValueError):
                call(dict(gpu, **{name: w}))
            assert len(launches) == 1, (name, what)


def tree_operands(dtype=BF16, out=F32, bias=True):
    hk, hv, d, width, rows, m = 2, 4, 32, 3, 5, 2
    ch = (2 * hk + hv) * d
    return dict(x=torch.zeros(rows, ch, dtype=dtype), conv_w=torch.zeros(ch, width, dtype=dtype),
                conv_b=torch.zeros(ch, dtype=dtype) if bias else None, g=torch.zeros(rows, hv), beta=torch.zeros(rows, hv),
                o=torch.zeros(rows, hv, d, dtype=out), parents=torch.zeros(rows, dtype=I32), cu=torch.zeros(m + 1, dtype=I32),
                accepted=torch.zeros(m, dtype=I32), sp=torch.zeros(m, dtype=I64), cp=torch.zeros(m, dtype=I64),
                k=torch.zeros(rows, hk, d), u=torch.zeros(rows, hv, d), gamma=torch.zeros(rows, hv))


def tree_dims(dtype, out):
    kinds = {BF16: gdn.GDN_BF16, F32: gdn.GDN_F32}
    return gdn.make_dims(2, 4, 32, conv_width=3, in_dtype=kinds[dtype], out_dtype=kinds[out])


@pytest.mark.parametrize("dtype,out,bias", [(BF16, F32, True), (F32, BF16, False)])
def test_tree_verify_operands(dtype, out, bias, launches):
    t = tree_operands(dtype, out, bias)
    del t["accepted"]
    d = tree_dims(dtype, out)
    refused_one_at_a_time(t, lambda a: gdn.tree_verify(d, a["x"], a["conv_w"], a["conv_b"], a["g"], a["beta"], a["o"],
                                                       a["parents"], a["cu"], 8, a["sp"], a["cp"],
                                                       record=(a["k"], a["u"], a["gamma"])), launches)


def test_tree_accept_operands(launches):
    t = tree_operands()
    for k in ("conv_w", "conv_b", "g", "beta", "o"):
        del t[k]
    d = tree_dims(BF16, F32)
    refused_one_at_a_time(t, lambda a: gdn.tree_accept(d, a["x"], (a["k"], a["u"], a["gamma"]), a["parents"], a["cu"], 8,
                                                       a["accepted"], a["sp"], a["cp"]), launches)


def test_tree_calls_that_are_fine(launches):
    """x rows apart, no parents, no record, one node, none."""
    d = tree_dims(BF16, F32)
    t = tree_operands()
    g = {k: OnGpu(v) for k, v in t.items()}
    wide = OnGpu(torch.zeros(5, t["x"].shape[1] + 8, dtype=BF16)[:, :t["x"].shape[1]])
    gdn.tree_verify(d, wide, g["conv_w"], None, g["g"], g["beta"], g["o"], None, g["cu"], 8, g["sp"], g["cp"])
    for n in (1, 0):
        c = {k: OnGpu(t[k][:n]) for k in ("x", "g", "beta", "o", "parents", "k", "u", "gamma")}
        rec = (c["k"], c["u"], c["gamma"])
        gdn.tree_verify(d, c["x"], g["conv_w"], g["conv_b"], c["g"], c["beta"], c["o"], c["parents"], g["cu"], 8, g["sp"], g["cp"],
                        record=rec)
        gdn.tree_accept(d, c["x"], rec, None, g["cu"], 8, g["accepted"], g["sp"], g["cp"])
    assert len(launches) == 5


def test_the_wrong_operand_is_named():
    """(state_ptrs gives the number of slots: a short one is told by cu_nodes)"""
    t = tree_operands()
    d = tree_dims(BF16, F32)

    def call(**kw):
        a = dict(t, **kw)
        gdn.tree_verify(d, a["x"], a["conv_w"], a["conv_b"], a["g"], a["beta"], a["o"], a["parents"], a["cu"], 8, a["sp"],
                        a["cp"], record=(a["k"], a["u"], a["gamma"]))

    for name, said in dict(t, x="x must", conv_w="conv_w", conv_b="conv_b", g="g must", beta="beta", o="o must",
                           parents="parents", cu="cu_nodes", sp="state_ptrs|cu_nodes", cp="conv_state_ptrs", k="k of the record",
                           u="u of the record", gamma="gamma of the record").items():
        if name == "accepted":
            continue
        for what, w in wrong_forms(t[name]):
            with pytest.raises(ValueError, match=said):
                call(**{name: w})
    with pytest.raises(ValueError, match="on the GPU"):
        call()


@pytest.mark.parametrize("fn", [gdn.slot_pack, gdn.slot_unpack])
def test_snapshot_operands(fn, launches):
    """Pointer arrays of another type or length, with gaps or on another device."""
    d = gdn.make_dims(1, 2, 32)
    order = ("state", "conv", "packed") if fn is gdn.slot_pack else ("packed", "state", "conv")

    def call(a):
        fn(d, gdn.GDN_PACK_INT8, *(a[k] for k in order))

    # (the state pointers give the number of slots)
    t = {k: torch.zeros(3, dtype=I64) for k in ("state", "conv", "packed")}
    refused_one_at_a_time(t, call, launches)
    refused_one_at_a_time(dict(t, conv=None), call, launches)


def test_snapshot_store_operands(launches, monkeypatch):
    """pack_slots and unpack_slots: a store of another size, type or layout, on the host or on another GPU; more slots
    than rows; indices of another type, length or device."""
    made = []
    monkeypatch.setattr(_lib, "gdn_slot_pointers", lambda *a: made.append(a))
    d = gdn.make_dims(1, 2, 32)
    size = gdn.gdn_slot_packed_size(d, gdn.GDN_PACK_INT8)
    pool = gdn.SlotPool(d, 4, device="cpu")
    pool.state, pool.conv_state = OnGpu(pool.state), OnGpu(pool.conv_state)
    monkeypatch.setattr(gdn.SlotPool, "pointers", lambda self, idx: (OnGpu(torch.zeros(idx.numel(), dtype=I64)),) * 2)
    good = OnGpu(torch.zeros(2, size, dtype=torch.uint8))
    idx = OnGpu(torch.zeros(2, dtype=I32))
    bad = [good._t, OnGpu(good._t, 1), OnGpu(good._t[:, :-16].contiguous()), OnGpu(good._t[:, ::2]), OnGpu(good._t.to(I32)),
           OnGpu(torch.zeros(2 * size, dtype=torch.uint8)), OnGpu(torch.zeros(2, size + 16, dtype=torch.uint8)[:, :size])]
    for store in bad:
        with pytest.raises(ValueError):
            pool.pack_slots(idx, store, gdn.GDN_PACK_INT8)
        with pytest.raises(ValueError):
            pool.unpack_slots(store, idx, idx, gdn.GDN_PACK_INT8)
    with pytest.raises(ValueError):
        pool.pack_slots(OnGpu(torch.zeros(3, dtype=I32)), good, gdn.GDN_PACK_INT8)
    for other in (OnGpu(torch.zeros(2, dtype=I64)), torch.zeros(2, dtype=I32), OnGpu(idx._t, 1), OnGpu(torch.zeros(3, dtype=I32)),
                  OnGpu(torch.zeros(4, dtype=I32)[::2])):
        with pytest.raises(ValueError):
            pool.unpack_slots(good, other, idx, gdn.GDN_PACK_INT8)
    assert not made and not launches


def test_addresses_may_be_unsigned(launches):
    d = gdn.make_dims(1, 2, 32)
    p = OnGpu(torch.zeros(3, dtype=torch.uint64))
    gdn.slot_pack(d, gdn.GDN_PACK_INT8, p, OnGpu(torch.zeros(3, dtype=I64)), p)
    assert len(launches) == 1


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("x,gate,param,y", [(F32, BF16, BF16, BF16), (BF16, F32, F32, F32)])
def test_group_norm_operands(x, gate, param, y, shared, launches):
    kinds = {BF16: gdn.GDN_BF16, F32: gdn.GDN_F32}
    d = gdn.make_norm_dims(3, 8, in_dtype=kinds[x], gate_dtype=kinds[gate], param_dtype=kinds[param], out_dtype=kinds[y],
                           shared_params=shared)
    per = 8 if shared else 24
    t = dict(x=torch.zeros(5, 24, dtype=x), gate=torch.zeros(5, 24, dtype=gate), weight=torch.zeros(per, dtype=param),
             bias=torch.zeros(per, dtype=param), y=torch.zeros(5, 24, dtype=y))
    refused_one_at_a_time(t, lambda a: gdn.group_norm(d, a["x"], a["weight"], a["y"], gate=a["gate"], bias=a["bias"]), launches)


def test_a_bf16_o_needs_dims_that_say_so(launches):
    """make_norm_dims() expects fp32 x by default: a bf16 o of the layer is not read as fp32."""
    o, y = OnGpu(torch.zeros(5, 4, 32, dtype=BF16)), OnGpu(torch.zeros(5, 128, dtype=BF16))
    with pytest.raises(ValueError, match="x must be"):
        gdn.group_norm(gdn.make_norm_dims(4, 32), o, None, y)
    gdn.group_norm(gdn.make_norm_dims(4, 32, in_dtype=gdn.GDN_BF16), o, None, y)
    assert len(launches) == 1


def test_group_norm_layouts(launches):
    """Rows apart, three axes, axes of length 1 whatever stride they carry, no rows."""
    d = gdn.make_norm_dims(4, 32, gate_dtype=gdn.GDN_F32, out_dtype=gdn.GDN_F32)
    one = gdn.make_norm_dims(1, 32, out_dtype=gdn.GDN_F32)
    ones = gdn.make_norm_dims(4, 1, out_dtype=gdn.GDN_F32, shared_params=False)
    wide = torch.zeros(5, 160)
    fine = [(d, wide[:, :128], wide[:, 32:]), (d, torch.zeros(5, 4, 32), wide[:, :128].view(5, 4, 32)),
            (d, torch.zeros(0, 128), torch.zeros(0, 4, 32)), (d, wide[1:2, 3:131], torch.zeros(1, 4, 32)),
            (one, torch.zeros(5, 4, 32)[:, 2:3], torch.zeros(5, 32)), (one, torch.zeros(5, 32, 4).transpose(1, 2)[:, :1].contiguous(),
                                                                       torch.zeros(5, 1, 32)),
            (ones, torch.zeros(5, 4).as_strided((5, 4, 1), (4, 1, 7)), torch.zeros(5, 4))]
    for dims, x, y in fine:
        gdn.group_norm(dims, OnGpu(x), None, OnGpu(y))
    assert len(launches) == len(fine)
    for bad in (torch.zeros(5, 256)[:, ::2], torch.zeros(5, 8, 32)[:, ::2], torch.zeros(128, 5).t(), torch.zeros(640),
                torch.zeros(5, 2, 2, 32), torch.zeros(4, 160), torch.zeros(5, 4, 64)[..., :32]):
        with pytest.raises(ValueError):
            gdn.group_norm(d, OnGpu(bad), None, OnGpu(torch.zeros(5, 128)))
    assert len(launches) == len(fine)


def test_a_pool_on_another_gpu_than_the_current_one(monkeypatch):
    """pack_slots and unpack_slots: the pointer arrays are built on the pool's device, as the blocks are moved."""
    current, where = [0], []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, current[0] = current[0], self.device

        def __exit__(self, *a):
            current[0] = self.before

    class Lib:
        def __getattr__(self, name):
            return lambda *a: where.append((name, current[0], a[-1])) or 0

    size = gdn.gdn_slot_packed_size(gdn.make_dims(1, 2, 32), gdn.GDN_PACK_INT8)
    monkeypatch.setattr(_lib, "_LIB", Lib())
    monkeypatch.setattr(_lib, "gdn_slot_packed_size", lambda *a: size)
    monkeypatch.setattr(_lib, "_current_device", lambda: current[0])
    monkeypatch.setattr(_lib, "_device_guard", Guard)
    monkeypatch.setattr(_lib, "_raw_stream", lambda device: 1000 + device)
    empty, arange = torch.empty, torch.arange
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: OnGpu(empty(*a, **k), device.index))
    monkeypatch.setattr(torch, "arange", lambda *a, device=None, **k: OnGpu(arange(*a, **k), device.index))
    pool = gdn.SlotPool(gdn.make_dims(1, 2, 32), 4, device="cpu")
    pool.state, pool.conv_state = OnGpu(pool.state, 1), OnGpu(pool.conv_state, 1)
    idx, store = OnGpu(torch.zeros(2, dtype=I32), 1), OnGpu(torch.zeros(2, size, dtype=torch.uint8), 1)
    pool.pack_slots(idx, store, gdn.GDN_PACK_INT8)
    pool.unpack_slots(store, idx, idx, gdn.GDN_PACK_INT8)
    assert [w[0] for w in where] == (["gdn_slot_pointers"] * 3 + ["gdn_slot_pack"]) + (["gdn_slot_pointers"] * 3 + ["gdn_slot_unpack"])
    assert all(w[1:] == (1, 1001) for w in where) and current == [0]
