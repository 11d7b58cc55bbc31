"""gdn_group_norm against its formula in 64 bits.

Tolerance, fp32 results: the mean of squares of n values accumulated in fp32 in a tree (at most
about 12 levels after 32 serial terms): 44 x 2^-24 of the sum at the very worst, half of it after the root; the
factors, gate and parameters add about 12 roundings: under 40 x 2^-24 = 2.4e-6 of |n w act(z)| + |b act(z)|,
plus, centred, 44 x 2^-24 of mean|x| rs |w act(z)| for the mean. silu(z) itself is good to 4 x 2^-24 plus the
rounding of its exponent, |z| 2^-24. bf16 results add half a step, 2^-8 of the value."""

import numpy as np
import pytest

from tests.gpu_helpers import announce, bits_of

pytestmark = pytest.mark.gpu


def act(t):
    import torch

    return t / (1 + torch.exp(-t))


def formula(o, x, gate, w, b):
    import torch

    rows, G, D = x.shape[0], o["groups"], o["size"]
    x = x.double().reshape(rows, G, D)
    f = act if o.get("silu", True) else lambda t: t
    z = None if gate is None else gate.double().reshape(rows, G, D)
    zf = None if z is None else f(z)
    if o.get("first"):
        x = x * zf
    mean = x.mean(-1, keepdim=True) if o.get("centered") else torch.zeros_like(x[..., :1])
    rs = 1 / torch.sqrt((x - mean).pow(2).mean(-1, keepdim=True) + o.get("eps", 1e-5))
    w = torch.ones(1, D, dtype=torch.float64, device=x.device) if w is None else w.double().reshape(-1, D)
    b = torch.zeros(1, D, dtype=torch.float64, device=x.device) if b is None else b.double().reshape(-1, D)
    n = (x - mean) * rs
    y = n * w + b
    # what the fp32 error is a share of
    size = n.abs() * w.abs() + b.abs() + (x.abs().mean(-1, keepdim=True) * rs * w.abs() if o.get("centered") else 0)
    if z is None:
        size = size * (1 + y.abs()) if o.get("silu", True) else size
        y = f(y)
    elif not o.get("first"):
        size = size * zf.abs() * (1 + z.abs() / 8)
        y = y * zf
    else:
        size = size * (1 + z.abs().amax(-1, keepdim=True) / 8)
    return y.reshape(rows, -1), size.reshape(rows, -1)


def make(o, rows, seed=0, pad=0, offset=0):
    import torch

    g = torch.Generator().manual_seed(seed)
    kinds = {"f32": torch.float32, "bf16": torch.bfloat16}
    width = o["groups"] * o["size"]
    per = o["size"] if o.get("shared", True) else width

    def rows_of(kind, mean=0.0):
        t = torch.empty(rows * (width + pad) + offset, dtype=kinds[kind], device="cuda")
        v = t[offset:].as_strided((rows, width), (width + pad, 1))
        v.copy_(torch.randn((rows, width), generator=g) + mean)
        return v

    x = rows_of(o.get("x", "f32"), 0.5)
    gate = rows_of(o["gate"]) if o.get("gate") else None
    w = None if o.get("no_w") else (1 + 0.2 * torch.randn(per, generator=g)).to(kinds[o.get("param", "f32")]).cuda()
    b = (0.2 * torch.randn(per, generator=g)).to(kinds[o.get("param", "f32")]).cuda() if o.get("bias") else None
    y = rows_of(o.get("y", "f32"))
    return x, gate, w, b, y


def run(o, x, gate, w, b, y, **kw):
    import gated_delta_rule_conv_amd as gdn

    k = {"f32": gdn.GDN_F32, "bf16": gdn.GDN_BF16}
    d = gdn.make_norm_dims(o["groups"], o["size"], in_dtype=k[o.get("x", "f32")], gate_dtype=k[o.get("gate") or "f32"],
                           param_dtype=k[o.get("param", "f32")], out_dtype=k[o.get("y", "f32")],
                           activation=gdn.GDN_ACT_SILU if o.get("silu", True) else gdn.GDN_ACT_NONE,
                           centered=o.get("centered", False), gate_first=o.get("first", False),
                           shared_params=o.get("shared", True), eps=o.get("eps", 1e-5))
    gdn.group_norm(d, x, w, y, gate=gate, bias=b, **kw)


def check(o, x, gate, w, b, y):
    want, size = formula(o, x, gate, w, b)
    off = (y.double() - want).abs()
    tol = 40 * 2.0 ** -24 * size + 1e-38
    if o.get("y") == "bf16":
        tol = tol * (1 + 2.0 ** -8) + want.abs() * 2.0 ** -8 + 2.0 ** -134
    worst = (off / tol).max().item()
    assert worst <= 1.0, worst


SIZES = [1, 2, 3, 4, 5, 8, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 200, 256, 257, 510, 512, 514, 1000, 1024, 1025, 2047,
         2048, 2049, 2500, 8192, 10001]


@pytest.mark.parametrize("size", SIZES)
def test_sizes(size):
    """Every lane layout and group tail, odd strides and addresses."""
    announce(f"norm size {size}")
    for n, o in enumerate([dict(gate="bf16"), dict(x="bf16", gate="f32", centered=True, bias=True, param="bf16", y="bf16"),
                           dict(x="bf16", y="f32", centered=True, shared=False, bias=True), dict(gate="f32", first=True, y="bf16")]):
        for rows, groups, pad, offset in ((1, 1, 0, 0), (3, 5, 0, 0), (7, 2, 3, 1)):
            o = dict(o, groups=groups, size=size)
            t = make(o, rows, seed=size + n, pad=pad, offset=offset)
            run(o, *t)
            check(o, *t)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [None, "f32", "bf16"])
@pytest.mark.parametrize("param", ["f32", "bf16"])
def test_types(x, y, gate, param):
    announce(f"norm types {x} {y} {gate} {param}")
    for silu in (False, True):
        for first in (False, True) if gate else (False,):
            for shared in (False, True):
                o = dict(groups=6, size=128, x=x, y=y, gate=gate, param=param, silu=silu, first=first, shared=shared,
                         bias=shared, centered=not shared)
                t = make(o, 37, seed=3)
                run(o, *t)
                check(o, *t)


def test_neither_weight_nor_bias():
    announce("norm: no parameters")
    o = dict(groups=4, size=64, no_w=True, gate="bf16", y="bf16", x="bf16")
    t = make(o, 9)
    run(o, *t)
    check(o, *t)


def test_special_rows():
    """Zero rows with eps 0 and not; a NaN or an infinity stays in its group; large and small values."""
    import torch

    announce("norm: special rows")
    o = dict(groups=3, size=100, silu=False, eps=1e-6)
    x, gate, w, b, y = make(o, 6)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 100:200] *= 1e15
    x[3, 205] = float("inf")
    x[4] *= 1e-12
    run(o, x, gate, w, b, y)
    assert (y[0] == 0).all()
    assert torch.isnan(y[1, :100]).all() and torch.isfinite(y[1, 100:]).all()
    assert torch.isnan(y[3, 205]) and torch.isfinite(y[3, :200]).all()
    rest = [2, 4, 5]
    check(o, x[rest], None, w, b, y[rest])


def test_rows_alone_and_in_a_batch_give_the_same_bits():
    announce("norm: row invariance")
    import torch

    o = dict(groups=32, size=128, gate="bf16", y="bf16", param="bf16")
    x, gate, w, b, y = make(o, 700)
    run(o, x, gate, w, b, y)
    y2 = torch.empty_like(y)
    for r in (0, 13, 699):
        run(o, x[r:r + 1], gate[r:r + 1], w, b, y2[r:r + 1])
        np.testing.assert_array_equal(bits_of(y2[r]), bits_of(y[r]))


def test_rows_beyond_32_bit_offsets_and_neighbours_untouched():
    """Rows 2^27 values apart (offsets past 2^32 values); what lies between them keeps its bits."""
    import torch

    announce("norm: far rows")
    o = dict(groups=2, size=65, x="bf16", y="bf16", gate="bf16")
    step = 1 << 27
    far = [torch.empty(40 * step, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    x, gate, w, b, y = make(o, 40)
    xf, yf = (t.as_strided((40, 130), (step, 1)) for t in far)
    xf.copy_(x)
    around = far[1].as_strided((40, 136), (step, 1))
    around.fill_(3.0)
    run(o, xf, gate, w, b, yf)
    run(o, x, gate, w, b, y)
    np.testing.assert_array_equal(bits_of(yf), bits_of(y))
    assert (around[:, 130:] == 3.0).all()


def test_three_axes_streams_and_graph():
    import torch

    announce("norm: [T, heads, d] views, another stream, graph")
    o = dict(groups=8, size=64, gate="bf16", y="bf16")
    x, gate, w, b, y = make(o, 50)
    run(o, x, gate, w, b, y)
    want = bits_of(y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2 = torch.zeros_like(y)
    torch.cuda.synchronize()
    run(o, x.reshape(50, 8, 64), gate.reshape(50, 8, 64), w, b, y2.view(50, 8, 64), stream=s)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits_of(y2), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(o, x, gate, w, b, y2)
    for _ in range(3):
        y2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(bits_of(y2), want)
