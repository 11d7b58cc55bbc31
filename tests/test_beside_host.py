"""Refusals of the linear attention, block norm, sampling and follow entry points (no GPU): each call below fails a host
check, so nothing is launched and the fake addresses are never read; and what the tensor helpers refuse."""

import ctypes

import pytest
import torch

import gated_delta_rule_conv_amd as gdn
from gated_delta_rule_conv_amd import _lib
from tests.test_operand_checks import BF16, F32, I32, I64, OnGpu, launches, refused_one_at_a_time  # noqa: F401

FAKE = 0x7F0000000000
NULL, SHAPE, DTYPE, ALIGN, WORK, UNSUP = (_lib.GDN_ERR_NULL, _lib.GDN_ERR_SHAPE, _lib.GDN_ERR_DTYPE, _lib.GDN_ERR_ALIGN,
                                          _lib.GDN_ERR_WORKSPACE, _lib.GDN_ERR_UNSUPPORTED)


def refused(fn, base, kw, want):
    with pytest.raises(gdn.GDNError) as e:
        fn(**dict(base, **kw))
    assert e.value.status == want and gdn.gdn_last_error().startswith(fn.__name__)


def linear(**kw):
    return gdn.make_linear_dims(**dict(dict(num_k_heads=16, num_v_heads=32, head_dim=128), **kw))


BOTH = [
    (dict(dims=gdn.make_dims(16, 32, 128)), UNSUP),
    (dict(dims=linear(head_dim=96)), UNSUP),
    (dict(dims=linear(num_v_heads=33)), SHAPE),
    (dict(dims=linear(scale=0.0)), SHAPE),
    (dict(dims=linear(in_dtype=2)), DTYPE),
    (dict(dims=linear(out_dtype=7)), DTYPE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(g=None), NULL), (dict(o=None), NULL),
    (dict(state_ptrs=None), NULL),
    (dict(q=FAKE + 8), ALIGN), (dict(k=FAKE + 2), ALIGN), (dict(v=FAKE + 4), ALIGN),
    (dict(q_stride=8196), ALIGN), (dict(k_stride=8193), ALIGN), (dict(v_stride=8196), ALIGN),
    (dict(q_stride=2040), SHAPE), (dict(k_stride=0), SHAPE), (dict(v_stride=4088), SHAPE), (dict(v_stride=-8192), SHAPE),
    (dict(g_stride=31), SHAPE), (dict(g_stride=-32), SHAPE),
]
PREFILL = dict(dims=linear(), q=FAKE, q_stride=8192, k=FAKE, k_stride=8192, v=FAKE, v_stride=8192, g=FAKE, g_stride=32, o=FAKE,
               cu_seqlens=FAKE, num_seqs=2, total_tokens=5000, state_ptrs=FAKE, workspace=FAKE, workspace_bytes=1 << 40, stream=0)
DECODE = dict(dims=linear(), q=FAKE, q_stride=8192, k=FAKE, k_stride=8192, v=FAKE, v_stride=8192, g=FAKE, g_stride=32, o=FAKE,
              state_ptrs=FAKE, m=4, stream=0)


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(num_seqs=-1), SHAPE), (dict(total_tokens=-1), SHAPE), (dict(num_seqs=0), SHAPE), (dict(cu_seqlens=None), NULL),
    (dict(workspace=FAKE + 128), ALIGN), (dict(q_stride=1 << 23), UNSUP), (dict(k_stride=1 << 23), UNSUP),
    (dict(v_stride=1 << 23), UNSUP), (dict(g_stride=1 << 22), UNSUP),
])
def test_linear_prefill_refusals(kw, want):
    refused(gdn.gdn_linear_prefill, PREFILL, kw, want)


@pytest.mark.parametrize("kw,want", BOTH + [(dict(m=-1), SHAPE), (dict(m=65536), SHAPE)])
def test_linear_decode_refusals(kw, want):
    refused(gdn.gdn_linear_decode, DECODE, kw, want)


def test_linear_prefill_workspace():
    need = gdn.gdn_linear_workspace_size(PREFILL["dims"], 2, 5000)
    if need:
        refused(gdn.gdn_linear_prefill, PREFILL, dict(workspace=None), WORK)
        refused(gdn.gdn_linear_prefill, PREFILL, dict(workspace_bytes=need - 1), WORK)


def test_linear_calls_with_nothing_to_do():
    gdn.gdn_linear_prefill(**dict(PREFILL, total_tokens=0, q=None, workspace=None))
    gdn.gdn_linear_prefill(**dict(PREFILL, num_seqs=0, total_tokens=0, cu_seqlens=None))
    gdn.gdn_linear_decode(**dict(DECODE, m=0, q=None))


def test_linear_workspace_covers_every_smaller_call():
    for form in (0, 1, 2):
        for heads in ((1, 1), (2, 4), (16, 32)):
            d = linear(num_k_heads=heads[0], num_v_heads=heads[1], prefill_form=form)
            most = gdn.gdn_linear_workspace_size(d, 70, 9000)
            for n in (0, 1, 2, 64, 65, 70):
                for t in (0, 1, 63, 64, 511, 512, 513, 4096, 9000):
                    assert gdn.gdn_linear_workspace_size(d, n, t) <= most
    with pytest.raises(gdn.GDNError):
        gdn.gdn_linear_workspace_size(gdn.make_dims(2, 4, 64), 1, 64)
    with pytest.raises(gdn.GDNError):
        gdn.gdn_linear_workspace_size(linear(), -1, 64)


def block(**kw):
    return gdn.make_block_norm_dims(**dict(dict(width=1024, post_norm=True), **kw))


BLOCK = dict(dims=block(), x=FAKE, x_stride=1024, residual=FAKE, residual_stride=1024, gate=FAKE, gate_stride=1024,
             post_weight=FAKE, post_bias=FAKE, pre_weight=FAKE, pre_bias=FAKE, residual_out=FAKE, residual_out_stride=1024,
             y=FAKE, y_stride=1024, rows=3, stream=0)


def sized(d, n):
    d.struct_size = n
    return d


@pytest.mark.parametrize("kw,want", [
    (dict(dims=sized(block(), 44)), SHAPE),
    (dict(dims=block(width=0)), SHAPE), (dict(dims=block(width=-4)), SHAPE), (dict(dims=block(width=32769)), UNSUP),
    (dict(dims=block(in_dtype=2)), DTYPE), (dict(dims=block(residual_dtype=-1)), DTYPE), (dict(dims=block(gate_dtype=3)), DTYPE),
    (dict(dims=block(param_dtype=2)), DTYPE), (dict(dims=block(out_dtype=2)), DTYPE), (dict(dims=block(activation=3)), DTYPE),
    (dict(dims=block(eps=-1.0)), SHAPE), (dict(dims=block(eps=float("nan"))), SHAPE), (dict(dims=block(scale=float("inf"))), SHAPE),
    (dict(dims=block(scale=float("nan"))), SHAPE), (dict(dims=block(post_norm=False)), SHAPE),
    (dict(x=None), NULL), (dict(y=None, residual_out=None, pre_weight=None, pre_bias=None), NULL), (dict(y=None), NULL),
    (dict(rows=-1), SHAPE), (dict(x_stride=1000), SHAPE), (dict(x_stride=0), SHAPE), (dict(residual_stride=0), SHAPE),
    (dict(gate_stride=1), SHAPE), (dict(gate_stride=-1024), SHAPE), (dict(residual_out_stride=1023), SHAPE), (dict(y_stride=8), SHAPE),
    (dict(residual_out_stride=2048), SHAPE),
    (dict(x=FAKE + 1), ALIGN), (dict(residual=FAKE + 1), ALIGN), (dict(gate=FAKE + 1), ALIGN), (dict(y=FAKE + 1), ALIGN),
    (dict(residual_out=FAKE + 1), ALIGN), (dict(post_weight=FAKE + 1), ALIGN), (dict(pre_bias=FAKE + 1), ALIGN),
])
def test_block_norm_refusals(kw, want):
    refused(gdn.gdn_block_norm, BLOCK, kw, want)


def test_block_norm_switches():
    for name in ("post_norm", "centered"):
        d = block()
        setattr(d, name, 2)
        refused(gdn.gdn_block_norm, BLOCK, dict(dims=d), DTYPE)
    gdn.gdn_block_norm(**dict(BLOCK, rows=0, x=None))


def test_the_sigmoid_is_the_block_norms_alone():
    d = gdn.make_dims(16, 32, 128, activation=gdn.GDN_ACT_SIGMOID)
    with pytest.raises(gdn.GDNError) as e:
        gdn.gdn_prefill_workspace_size(d, 1, 1)
    assert e.value.status == DTYPE


SAMPLE = dict(logits=FAKE, stride=1000, dtype=0, rows=4, vocab=1000, temperature=None, top_k=None, top_p=None, min_p=None, uniform=FAKE,
              tokens=FAKE, prob=None, workspace=FAKE, workspace_bytes=1 << 40, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=(1 << 20) + 1, stride=1 << 25), SHAPE), (dict(dtype=2), DTYPE),
    (dict(logits=None), NULL), (dict(uniform=None), NULL), (dict(tokens=None), NULL), (dict(stride=999), SHAPE), (dict(stride=-1000), SHAPE),
    (dict(logits=FAKE + 2), ALIGN), (dict(dtype=1, logits=FAKE + 1), ALIGN), (dict(workspace=FAKE + 16), ALIGN),
])
def test_sample_refusals(kw, want):
    refused(gdn.gdn_sample, SAMPLE, kw, want)


def test_sample_workspace():
    need = gdn.gdn_sample_workspace_size(4, 1000)
    if need:
        refused(gdn.gdn_sample, SAMPLE, dict(workspace_bytes=need - 1), WORK)
        refused(gdn.gdn_sample, SAMPLE, dict(workspace=None), WORK)
    for r in (0, 1, 3, 4):
        for v in (1, 64, 999, 1000):
            assert gdn.gdn_sample_workspace_size(r, v) <= need
    gdn.gdn_sample(**dict(SAMPLE, rows=0, logits=None))
    out = ctypes.c_size_t()
    for args, want in (((4, 1000, None), NULL), ((-1, 5, ctypes.byref(out)), SHAPE), ((1, 0, ctypes.byref(out)), SHAPE)):
        assert _lib.lib().gdn_sample_workspace_size(*args) == want


FOLLOW = dict(drafted=FAKE, sampled=FAKE, pending=FAKE, parents=None, cu_nodes=FAKE, m=4, total_nodes=20, max_nodes=8, accepted=FAKE,
              next=FAKE, path=None, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), SHAPE), (dict(total_nodes=-1), SHAPE), (dict(m=0), SHAPE), (dict(max_nodes=0), SHAPE), (dict(max_nodes=65), UNSUP),
    (dict(drafted=None), NULL), (dict(sampled=None), NULL), (dict(pending=None), NULL), (dict(cu_nodes=None), NULL),
    (dict(accepted=None), NULL), (dict(next=None), NULL),
])
def test_follow_refusals(kw, want):
    refused(gdn.gdn_tree_follow, FOLLOW, kw, want)


# ------------------------------------------------------------------ the tensor helpers


@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("fixed", [False, True])
def test_linear_operands(dtype, out, fixed, launches):  # noqa: F811
    kinds = {BF16: gdn.GDN_BF16, F32: gdn.GDN_F32}
    d = gdn.make_linear_dims(2, 4, 32, in_dtype=kinds[dtype], out_dtype=kinds[out])
    t = dict(q=torch.zeros(5, 64, dtype=dtype), k=torch.zeros(5, 2, 32, dtype=dtype), v=torch.zeros(5, 128, dtype=dtype),
             g=torch.zeros(4) if fixed else torch.zeros(5, 4), o=torch.zeros(5, 4, 32, dtype=out), sp=torch.zeros(5, dtype=I64))
    refused_one_at_a_time(t, lambda a: gdn.linear_decode(d, a["q"], a["k"], a["v"], a["g"], a["o"], a["sp"]), launches)
    t.update(sp=torch.zeros(2, dtype=I64), cu=torch.zeros(3, dtype=I32))
    work = OnGpu(torch.zeros(1024, dtype=torch.uint8))
    refused_one_at_a_time(t, lambda a: gdn.linear_prefill(d, a["q"], a["k"], a["v"], a["g"], a["o"], a["cu"], a["sp"], work), launches)


def test_overlapping_rows_are_told(launches):  # noqa: F811
    d = gdn.make_linear_dims(1, 2, 32, in_dtype=gdn.GDN_F32)
    t = {k: OnGpu(v) for k, v in dict(q=torch.zeros(3, 32), k=torch.zeros(3, 32), v=torch.zeros(3, 64), o=torch.zeros(3, 2, 32),
                                      sp=torch.zeros(3, dtype=I64)).items()}
    with pytest.raises(ValueError):
        gdn.linear_decode(d, t["q"], t["k"], t["v"], OnGpu(torch.zeros(1, 2).expand(3, 2)), t["o"], t["sp"])
    b = gdn.make_block_norm_dims(32)
    x, y = OnGpu(torch.zeros(3, 32, dtype=BF16)), OnGpu(torch.zeros(3, 32, dtype=BF16))
    with pytest.raises(ValueError):
        gdn.block_norm(b, x, x, y, gate=OnGpu(torch.zeros(1, 32, dtype=BF16).expand(3, 32)))
    assert launches == []


@pytest.mark.parametrize("vector", [False, True])
def test_block_norm_operands(vector, launches):  # noqa: F811
    d = gdn.make_block_norm_dims(32, in_dtype=gdn.GDN_F32, residual_dtype=gdn.GDN_F32, gate_dtype=gdn.GDN_BF16, out_dtype=gdn.GDN_BF16,
                                 post_norm=True)
    t = dict(x=torch.zeros(3, 32), r=torch.zeros(3, 32), y=torch.zeros(3, 32, dtype=BF16), h=torch.zeros(3, 32),
             gate=torch.zeros(32, dtype=BF16) if vector else torch.zeros(3, 32, dtype=BF16), a=torch.zeros(32, dtype=BF16),
             b=torch.zeros(32, dtype=BF16), c=torch.zeros(32, dtype=BF16), e=torch.zeros(32, dtype=BF16))
    refused_one_at_a_time(t, lambda a: gdn.block_norm(d, a["x"], a["r"], a["y"], residual_out=a["h"], gate=a["gate"], post_weight=a["a"],
                                                      post_bias=a["b"], pre_weight=a["c"], pre_bias=a["e"]), launches)


def test_sample_operands(launches):  # noqa: F811
    t = dict(u=torch.zeros(3), tokens=torch.zeros(3, dtype=I32), t=torch.zeros(3), k=torch.zeros(3, dtype=I32), p=torch.zeros(3),
             m=torch.zeros(3), prob=torch.zeros(3))
    x, work = OnGpu(torch.zeros(3, 50)), OnGpu(torch.zeros(256, dtype=torch.uint8))
    refused_one_at_a_time(t, lambda a: gdn.sample(x, a["u"], a["tokens"], work, temperature=a["t"], top_k=a["k"], top_p=a["p"], min_p=a["m"],
                                                  prob=a["prob"]), launches)
    for bad in (torch.zeros(3, 50, dtype=torch.float16), torch.zeros(150), torch.zeros(50, 3).t()):
        with pytest.raises(ValueError):
            gdn.sample(OnGpu(bad), OnGpu(t["u"]), OnGpu(t["tokens"]), work)


def test_follow_operands(launches):  # noqa: F811
    t = dict(drafted=torch.zeros(6, dtype=I32), sampled=torch.zeros(6, dtype=I32), pending=torch.zeros(2, dtype=I32),
             parents=torch.zeros(6, dtype=I32), cu=torch.zeros(3, dtype=I32), acc=torch.zeros(2, dtype=I32), nxt=torch.zeros(2, dtype=I32),
             path=torch.zeros(2, 4, dtype=I32))
    refused_one_at_a_time(t, lambda a: gdn.tree_follow(a["drafted"], a["sampled"], a["pending"], a["parents"], a["cu"], 4, a["acc"],
                                                       a["nxt"], path=a["path"]), launches)
