"""Host-side refusals of the tree, snapshot and norm entry points (no GPU): each call below
fails a host check, so nothing is launched and the fake addresses are never dereferenced."""

import ctypes

import pytest

import gated_delta_rule_conv_amd as gdn
from gated_delta_rule_conv_amd import _lib

FAKE = 0x7F0000000000


def dims(**kw):
    return gdn.make_dims(**dict(dict(num_k_heads=16, num_v_heads=32, head_dim=128), **kw))


def status(fn, *args):
    with pytest.raises(gdn.GDNError) as e:
        fn(*args)
    return e.value.status


VERIFY = dict(x=FAKE, x_stride=8192, conv_w=FAKE, conv_b=None, g=FAKE, beta=FAKE, o=FAKE, parents=FAKE, cu_nodes=FAKE,
              m=4, total_nodes=20, max_nodes=8, state_ptrs=FAKE, conv_state_ptrs=FAKE, k_rec=None, u_rec=None,
              gamma_rec=None, stream=0)
ACCEPT = dict(x=FAKE, x_stride=8192, k_rec=FAKE, u_rec=FAKE, gamma_rec=FAKE, parents=FAKE, cu_nodes=FAKE,
              accepted=FAKE, m=4, total_nodes=20, max_nodes=8, state_ptrs=FAKE, conv_state_ptrs=FAKE, stream=0)

SHARED = [
    (dict(m=-1), _lib.GDN_ERR_SHAPE),
    (dict(total_nodes=-1), _lib.GDN_ERR_SHAPE),
    (dict(m=0), _lib.GDN_ERR_SHAPE),
    (dict(m=65536), _lib.GDN_ERR_SHAPE),
    (dict(max_nodes=0), _lib.GDN_ERR_SHAPE),
    (dict(max_nodes=65), _lib.GDN_ERR_UNSUPPORTED),
    (dict(x=None), _lib.GDN_ERR_NULL),
    (dict(cu_nodes=None), _lib.GDN_ERR_NULL),
    (dict(state_ptrs=None), _lib.GDN_ERR_NULL),
    (dict(conv_state_ptrs=None), _lib.GDN_ERR_NULL),
    (dict(x=FAKE + 8), _lib.GDN_ERR_ALIGN),
    (dict(x_stride=8193), _lib.GDN_ERR_ALIGN),
    (dict(x_stride=4096), _lib.GDN_ERR_SHAPE),
    (dict(x_stride=-8192), _lib.GDN_ERR_SHAPE),
]


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(conv_w=None), _lib.GDN_ERR_NULL),
    (dict(g=None), _lib.GDN_ERR_NULL),
    (dict(beta=None), _lib.GDN_ERR_NULL),
    (dict(o=None), _lib.GDN_ERR_NULL),
    (dict(k_rec=FAKE), _lib.GDN_ERR_NULL),
    (dict(k_rec=FAKE, u_rec=FAKE), _lib.GDN_ERR_NULL),
    (dict(k_rec=FAKE + 4, u_rec=FAKE, gamma_rec=FAKE), _lib.GDN_ERR_ALIGN),
    (dict(k_rec=FAKE, u_rec=FAKE + 4, gamma_rec=FAKE), _lib.GDN_ERR_ALIGN),
    (dict(conv_w=FAKE + 2), _lib.GDN_ERR_ALIGN),
    (dict(conv_b=FAKE + 2), _lib.GDN_ERR_ALIGN),
])
def test_verify_refusals(kw, want):
    assert status(gdn.gdn_tree_verify, dims(), *dict(VERIFY, **kw).values()) == want


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(k_rec=None), _lib.GDN_ERR_NULL),
    (dict(u_rec=None), _lib.GDN_ERR_NULL),
    (dict(gamma_rec=None), _lib.GDN_ERR_NULL),
    (dict(accepted=None), _lib.GDN_ERR_NULL),
    (dict(k_rec=FAKE + 4), _lib.GDN_ERR_ALIGN),
    (dict(u_rec=FAKE + 4), _lib.GDN_ERR_ALIGN),
])
def test_accept_refusals(kw, want):
    assert status(gdn.gdn_tree_accept, dims(), *dict(ACCEPT, **kw).values()) == want


@pytest.mark.parametrize("kw,want", [
    (dict(head_dim=96), _lib.GDN_ERR_UNSUPPORTED),
    (dict(conv_width=5), _lib.GDN_ERR_UNSUPPORTED),
    (dict(in_dtype=7), _lib.GDN_ERR_DTYPE),
    (dict(num_k_heads=3), _lib.GDN_ERR_SHAPE),
])
def test_bad_dims_rejected_by_the_slot_operators(kw, want):
    d = dims(**kw)
    assert status(gdn.gdn_tree_verify, d, *VERIFY.values()) == want
    assert status(gdn.gdn_tree_accept, d, *ACCEPT.values()) == want
    assert status(gdn.gdn_slot_packed_size, d, 0) == want
    assert status(gdn.gdn_slot_pack, d, 0, FAKE, FAKE, FAKE, 2, 0) == want
    assert status(gdn.gdn_slot_unpack, d, 0, FAKE, FAKE, FAKE, 2, 0) == want


def test_empty_calls_are_fine():
    gdn.gdn_tree_verify(dims(), *dict(VERIFY, m=0, total_nodes=0, x=None, max_nodes=0).values())
    gdn.gdn_tree_verify(dims(), *dict(VERIFY, total_nodes=0).values())
    gdn.gdn_tree_accept(dims(), *dict(ACCEPT, total_nodes=0).values())
    gdn.gdn_slot_pack(dims(), 0, None, None, None, 0, 0)
    gdn.gdn_slot_unpack(dims(), 1, None, None, None, 0, 0)
    gdn.gdn_group_norm(gdn.make_norm_dims(4, 32), None, 128, None, 0, None, None, None, 128, 0, 0)


@pytest.mark.parametrize("fn", ["gdn_slot_pack", "gdn_slot_unpack"])
def test_pack_refusals(fn):
    f, ptrs = getattr(gdn, fn), {"gdn_slot_pack": ("state", "conv", "packed"), "gdn_slot_unpack": ("packed", "state", "conv")}[fn]

    def call(fmt=0, n=2, **null):
        return status(f, dims(), fmt, *[None if p in null else FAKE for p in ptrs], n, 0)

    assert call(fmt=2) == _lib.GDN_ERR_DTYPE
    assert call(fmt=-1) == _lib.GDN_ERR_DTYPE
    assert call(n=-1) == _lib.GDN_ERR_SHAPE
    assert call(n=65536) == _lib.GDN_ERR_SHAPE
    assert call(state=1) == _lib.GDN_ERR_NULL
    assert call(packed=1) == _lib.GDN_ERR_NULL


def test_packed_size():
    """codes, scales, conv state: 32 x 128 x 128 + 32 x 128 x 4 + 3 x 8192 x 2 bytes."""
    assert gdn.gdn_slot_packed_size(dims(), gdn.GDN_PACK_INT8) == 32 * 128 * 128 + 32 * 128 * 4 + 3 * 8192 * 2
    d = dims(num_k_heads=2, num_v_heads=6, head_dim=32, conv_width=2, in_dtype=gdn.GDN_F32)
    assert gdn.gdn_slot_packed_size(d, gdn.GDN_PACK_E4M3) == 6 * 32 * 32 + 6 * 32 * 4 + 320 * 4
    assert _lib.lib().gdn_slot_packed_size(ctypes.byref(d), 0, None) == _lib.GDN_ERR_NULL


NORM = dict(x=FAKE, x_stride=4096, gate=FAKE, gate_stride=4096, weight=FAKE, bias=None, y=FAKE, y_stride=4096, rows=8,
            stream=0)


@pytest.mark.parametrize("fields,kw,want", [
    ({}, dict(x=None), _lib.GDN_ERR_NULL),
    ({}, dict(y=None), _lib.GDN_ERR_NULL),
    (dict(gate_first=1), dict(gate=None), _lib.GDN_ERR_NULL),
    ({}, dict(rows=-1), _lib.GDN_ERR_SHAPE),
    ({}, dict(x_stride=4095), _lib.GDN_ERR_SHAPE),
    ({}, dict(gate_stride=4095), _lib.GDN_ERR_SHAPE),
    ({}, dict(y_stride=4095), _lib.GDN_ERR_SHAPE),
    ({}, dict(x_stride=-4096), _lib.GDN_ERR_SHAPE),
    ({}, dict(x=FAKE + 2), _lib.GDN_ERR_ALIGN),
    ({}, dict(gate=FAKE + 1), _lib.GDN_ERR_ALIGN),
    ({}, dict(weight=FAKE + 1), _lib.GDN_ERR_ALIGN),
    ({}, dict(bias=FAKE + 1), _lib.GDN_ERR_ALIGN),
    ({}, dict(y=FAKE + 1), _lib.GDN_ERR_ALIGN),
    (dict(struct_size=4), {}, _lib.GDN_ERR_SHAPE),
    (dict(groups=0), {}, _lib.GDN_ERR_SHAPE),
    (dict(group_size=0), {}, _lib.GDN_ERR_SHAPE),
    (dict(groups=1 << 20, group_size=1 << 20), {}, _lib.GDN_ERR_SHAPE),
    (dict(in_dtype=2), {}, _lib.GDN_ERR_DTYPE),
    (dict(gate_dtype=2), {}, _lib.GDN_ERR_DTYPE),
    (dict(param_dtype=-1), {}, _lib.GDN_ERR_DTYPE),
    (dict(out_dtype=2), {}, _lib.GDN_ERR_DTYPE),
    (dict(activation=2), {}, _lib.GDN_ERR_DTYPE),
    (dict(centered=2), {}, _lib.GDN_ERR_DTYPE),
    (dict(gate_first=2), {}, _lib.GDN_ERR_DTYPE),
    (dict(shared_params=2), {}, _lib.GDN_ERR_DTYPE),
    (dict(eps=-1.0), {}, _lib.GDN_ERR_SHAPE),
    (dict(eps=float("nan")), {}, _lib.GDN_ERR_SHAPE),
    (dict(eps=float("inf")), {}, _lib.GDN_ERR_SHAPE),
])
def test_norm_refusals(fields, kw, want):
    d = gdn.make_norm_dims(32, 128)
    for k, v in fields.items():
        setattr(d, k, v)
    assert status(gdn.gdn_group_norm, d, *dict(NORM, **kw).values()) == want


def test_null_dims():
    lib = _lib.lib()
    assert lib.gdn_group_norm(None, FAKE, 8, None, 0, None, None, FAKE, 8, 1, None) == _lib.GDN_ERR_NULL
    assert lib.gdn_slot_pack(None, 0, FAKE, None, FAKE, 1, None) == _lib.GDN_ERR_NULL
    assert lib.gdn_tree_accept(None, *ACCEPT.values()) == _lib.GDN_ERR_NULL
    assert ctypes.sizeof(_lib.gdn_norm_dims) == 12 * 4


def test_host_tensors_are_refused_before_any_launch():
    import torch

    t = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        gdn.group_norm(gdn.make_norm_dims(4, 32), t, None, t.clone(), gate=None)
    d = gdn.make_dims(1, 1, 32)
    p = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError):
        gdn.slot_pack(d, gdn.GDN_PACK_INT8, p, None, p)
