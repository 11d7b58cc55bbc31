"""gdn_block_norm against its formula in 64 bits.

Tolerance of a norm's result: the mean of squares of n values in fp32 is a tree of at most 32 serial terms a lane and 10 levels,
42 x 2^-24 of it, half of that after the root; its own factors and roundings add 10: 31 x 2^-24 of |n w|, plus, centered,
42 x 2^-24 of mean|x| rs |w| for the mean. h adds the gate (sigmoid and silu: 4 x 2^-24, and the rounding of the exponent,
|z| 2^-24 of a factor 1 / (1 + e^-z) whose relative slope is below 1), the scale and the sum: 40 (1 + |z| / 16) x 2^-24 of
|scale gate a| + 2^-24 |r|. An error of h passes the second norm times its weight and rs, and once more through the
root (its relative error averaged): twice the row's largest error ratio covers that. bf16 results add half a step, 2^-8."""

import numpy as np
import pytest

from tests.gpu_helpers import announce, bits_of

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24


def act(kind, z):
    import torch

    soft = 1 / (1 + torch.exp(-z))
    return {"none": z, "sigmoid": soft, "silu": z * soft}[kind]


def norm(x, w, b, centered, eps):
    """The norm in 64 bits and its error in fp32 (without x's own)."""
    mean = x.mean(-1, keepdim=True) if centered else 0 * x[:, :1]
    rs = 1 / ((x - mean).pow(2).mean(-1, keepdim=True) + eps).sqrt()
    w = 1.0 if w is None else w.double()
    b = 0.0 if b is None else b.double()
    n = (x - mean) * rs * w
    off = 31 * STEP * n.abs() + (42 * STEP * x.abs().mean(-1, keepdim=True) * rs if centered else 0) * (w if isinstance(w, float) else w.abs())
    y = n + b
    return y, off + STEP * y.abs(), rs * (w if isinstance(w, float) else w.abs())


def formula(o, t):
    x = t["x"].double()
    eps, centered = o.get("eps", 1e-5), o.get("centered", False)
    a, off = x, 0 * x
    if o.get("post"):
        a, off, _ = norm(x, t["post_w"], t["post_b"], centered, eps)
    if t["gate"] is not None:
        z = t["gate"].double()
        f = act(o.get("act", "none"), z)
        off = off * f.abs() + 9 * (1 + z.abs()) * STEP * (a * f).abs()
        a = a * f
    s = o.get("scale", 1.0)
    r = t["r"].double() if t["r"] is not None else 0 * x
    h = r + s * a
    off = abs(s) * off + 2 * STEP * (s * a).abs() + STEP * h.abs()
    y, off_y, slope = norm(h, t["pre_w"], t["pre_b"], centered, eps)
    through = slope * (off + 2 * off.pow(2).mean(-1, keepdim=True).sqrt() * ((h / h.pow(2).mean(-1, keepdim=True).add(1e-300).sqrt()).abs() + 1))
    return h, off, y, off_y + through


def make(o, rows, width, seed=0, pad=0, offset=0):
    import torch

    g = torch.Generator().manual_seed(seed)
    kinds = {"f32": torch.float32, "bf16": torch.bfloat16}

    def rows_of(kind, fill=None):
        t = torch.empty(rows * (width + pad) + offset, dtype=kinds[kind], device="cuda")
        v = t[offset:].as_strided((rows, width), (width + pad, 1))
        t.fill_(5.0)
        if fill is not None:
            v.copy_(fill)
        return v

    rand = lambda: torch.randn((rows, width), generator=g)  # noqa: E731
    param = kinds[o.get("param", "bf16")]
    vec = lambda m, s: (m + s * torch.randn(width, generator=g)).to(param).cuda()  # noqa: E731
    t = {"x": rows_of(o.get("x", "bf16"), rand() + 0.3), "r": rows_of(o.get("r", "bf16"), 3 * rand()) if o.get("residual", True) else None}
    t["gate"] = None
    if o.get("gate"):
        t["gate"] = torch.randn(width, generator=g).to(kinds[o["gate"]]).cuda() if o.get("vector") else rows_of(o["gate"], rand())
    t["post_w"] = vec(1, 0.2) if o.get("post") and not o.get("no_w") else None
    t["post_b"] = vec(0, 0.2) if o.get("post") and o.get("bias") else None
    t["pre_w"] = None if o.get("no_w") else vec(1, 0.2)
    t["pre_b"] = vec(0, 0.2) if o.get("bias") else None
    t["h"], t["y"] = rows_of(o.get("r", "bf16")), rows_of(o.get("y", "bf16"))
    return t


def dims_of(o, width):
    import gated_delta_rule_conv_amd as gdn

    k = {"f32": gdn.GDN_F32, "bf16": gdn.GDN_BF16}
    acts = {"none": gdn.GDN_ACT_NONE, "silu": gdn.GDN_ACT_SILU, "sigmoid": gdn.GDN_ACT_SIGMOID}
    return gdn.make_block_norm_dims(width, in_dtype=k[o.get("x", "bf16")], residual_dtype=k[o.get("r", "bf16")],
                                    gate_dtype=k[o.get("gate") or "bf16"], param_dtype=k[o.get("param", "bf16")],
                                    out_dtype=k[o.get("y", "bf16")], activation=acts[o.get("act", "none")],
                                    post_norm=bool(o.get("post")), centered=o.get("centered", False), scale=o.get("scale", 1.0),
                                    eps=o.get("eps", 1e-5))


def call(o, t, h="h", y="y", **kw):
    import gated_delta_rule_conv_amd as gdn

    d = dims_of(o, t["x"].shape[1])
    gdn.block_norm(d, t["x"], t["r"], t[y] if y else None, residual_out=t[h] if h else None, gate=t["gate"], post_weight=t["post_w"],
                   post_bias=t["post_b"], pre_weight=t["pre_w"] if y else None, pre_bias=t["pre_b"] if y else None, **kw)


def near(got, want, off):
    import torch

    half = 2.0 ** -8 * (want.abs() + off) if got.dtype == torch.bfloat16 else 0
    over = (got.double() - want).abs() - off - half
    assert torch.isfinite(got).all() and float(over.max()) <= 0, f"{float(over.max())} over"


def check(o, rows, width, **kw):
    t = make(o, rows, width, **kw)
    h, off_h, y, off_y = formula(o, t)
    call(o, t)
    near(t["h"], h, off_h)
    near(t["y"], y, off_y)
    return t


OPTIONS = [
    {},
    {"post": True, "scale": 0.5},
    {"post": True, "gate": "bf16", "act": "sigmoid", "r": "f32"},
    {"gate": "f32", "act": "silu", "x": "f32", "y": "f32", "param": "f32", "centered": True, "bias": True, "post": True, "r": "f32"},
    {"gate": "bf16", "vector": True, "centered": True, "residual": False, "y": "f32"},
    {"no_w": True, "x": "f32", "r": "f32", "y": "f32", "scale": -1.5},
]


@pytest.mark.parametrize("o", OPTIONS, ids=lambda o: "-".join(f"{k}={v}" for k, v in o.items()) or "plain")
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (5, 512), (5, 513), (9, 1024), (3, 1031), (4, 2048), (3, 4096), (2, 4099), (2, 8192),
                                        (2, 10000), (1, 16384), (1, 32768), (1, 32765), (5, 520), (2, 7001), (2, 12001)])
def test_formula(o, rows, width):
    announce(f"block norm {rows} x {width} {o}")
    check(o, rows, width, seed=width)


@pytest.mark.parametrize("o", OPTIONS[1:4], ids=["post", "sigmoid", "centered"])
@pytest.mark.parametrize("pad,offset", [(1, 1), (3, 2), (8, 0)])
def test_strides_and_offsets(o, pad, offset):
    """Rows of any stride and alignment; what lies between them stays."""
    announce(f"block norm stride +{pad} offset {offset} {o}")
    t = check(o, 6, 777, pad=pad, offset=offset, seed=3)
    for name in ("h", "y"):
        whole = t[name].as_strided((6, 777 + pad), (777 + pad, 1), t[name].storage_offset())[:5, 777:]
        assert (whole.float() == 5).all()


def test_in_place_and_in_part():
    """h on top of the residual; h alone; y alone: the same bits."""
    import torch

    announce("block norm in place, and one output alone")
    o = {"post": True, "gate": "bf16", "act": "silu"}
    for width in (300, 3000):
        t = make(o, 11, width, seed=1)
        call(o, t)
        h, y = bits_of(t["h"]), bits_of(t["y"])
        t["h"].fill_(0.0)
        t["y"].fill_(0.0)
        call(o, t, y=None)
        assert (bits_of(t["h"]) == h).all()
        call(o, t, h=None)
        assert (bits_of(t["y"]) == y).all()
        t["y"].fill_(0.0)
        call(o, t, h="r")
        torch.cuda.synchronize()
        assert (bits_of(t["r"]) == h).all() and (bits_of(t["y"]) == y).all()


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e18, 1e30])
@pytest.mark.parametrize("width", [100, 4096, 20000])
@pytest.mark.parametrize("centered", [False, True])
def test_any_finite_size(size, width, centered):
    """Values whose squares leave fp32, and a stream far larger or smaller than the block."""
    import torch

    announce(f"block norm of values near {size}, width {width}, centered {centered}")
    o = {"post": True, "x": "f32", "r": "f32", "y": "f32", "param": "f32", "eps": 0.0, "centered": centered}
    t = make(o, 3, width, seed=2)
    t["x"].mul_(size)
    t["r"].mul_(size)
    h, off_h, y, off_y = formula(o, t)
    call(o, t)
    near(t["h"], h, off_h)
    near(t["y"], y, off_y)
    assert torch.isfinite(t["y"]).all()


def test_no_row_touches_another():
    """A row of NaN and one of infinities leave the others' bits alone."""
    announce("block norm with broken rows")
    o = {"post": True, "gate": "bf16"}
    for width in (200, 1500, 5000):
        a, b = make(o, 9, width, seed=5), make(o, 9, width, seed=5)
        b["x"][3, width // 2] = float("nan")
        b["r"][6] = float("inf")
        call(o, a)
        call(o, b)
        for name in ("h", "y"):
            x, y = bits_of(a[name]), bits_of(b[name])
            rest = [i for i in range(9) if i not in (3, 6)]
            assert (x[rest] == y[rest]).all()
        assert not np.isfinite(b["y"][3].float().cpu().numpy()).any()


def test_captured_and_on_another_stream():
    import torch

    announce("block norm in a graph and on another stream")
    o = {"post": True, "gate": "bf16", "act": "sigmoid"}
    t = make(o, 64, 2048, seed=6)
    call(o, t)
    torch.cuda.synchronize()
    h, y = bits_of(t["h"]), bits_of(t["y"])
    s = torch.cuda.Stream()
    for name in ("h", "y"):
        t[name].fill_(0.0)
    torch.cuda.synchronize()
    call(o, t, stream=s)
    s.synchronize()
    assert (bits_of(t["h"]) == h).all() and (bits_of(t["y"]) == y).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o, t)
    for _ in range(3):
        t["h"].fill_(0.0)
        t["y"].fill_(0.0)
        graph.replay()
        torch.cuda.synchronize()
        assert (bits_of(t["h"]) == h).all() and (bits_of(t["y"]) == y).all()


def test_no_rows():
    announce("block norm of no rows")
    call({}, make({}, 0, 64))


def test_more_rows_than_a_launch_holds():
    """2^21 + 5 rows go in two launches: every row as in calls of fewer rows, in place and with one gate for all."""
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce("block norm of 2^21 + 5 rows")
    rows, width = (1 << 21) + 5, 3
    g = torch.Generator().manual_seed(1)
    x, r = (torch.randn(rows, width, generator=g).cuda() for _ in range(2))
    gate, w = torch.randn(width, generator=g).cuda(), torch.randn(width, generator=g).cuda()
    f32 = dict(in_dtype=gdn.GDN_F32, residual_dtype=gdn.GDN_F32, gate_dtype=gdn.GDN_F32, param_dtype=gdn.GDN_F32, out_dtype=gdn.GDN_F32)
    dims = gdn.make_block_norm_dims(width, post_norm=True, scale=0.5, **f32)

    def run(a, b):
        h, y = r[a:b].clone(), torch.full((b - a, width), 7.0, device="cuda")
        gdn.block_norm(dims, x[a:b], h, y, residual_out=h, gate=gate, pre_weight=w)
        return h, y

    whole = run(0, rows)
    parts = [run(a, min(a + (1 << 20), rows)) for a in range(0, rows, 1 << 20)]
    torch.cuda.synchronize()
    for i in (0, 1):
        assert torch.equal(whole[i], torch.cat([p[i] for p in parts]))
    a = x.double() / torch.sqrt((x.double() ** 2).mean(1, keepdim=True) + 1e-6)
    assert float((whole[0] - (r.double() + 0.5 * gate.double() * a)).abs().max()) < 1e-5
