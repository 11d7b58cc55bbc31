"""gdn_linear_prefill and gdn_linear_decode against their recurrence in 64 bits (tests/linear_ref.py, where the
tolerances come from; a bf16 output adds half a step, 2^-8 of the value)."""

import numpy as np
import pytest

from tests.gpu_helpers import announce, bits_of
from tests.linear_ref import bound, packed

pytestmark = pytest.mark.gpu

BF16, F32 = "bf16", "f32"


class Case:
    """q, k, v as columns of one tensor, g, a pool of slots in a shuffled order, on the GPU and in 64 bits."""

    def __init__(self, lens, Hk=2, Hv=4, d=64, dtype=BF16, out=F32, fixed=False, seed=0, decay=0.2, pad=8, form=0, mma=0, g=None):
        import torch

        import gated_delta_rule_conv_amd as gdn

        kinds = {BF16: torch.bfloat16, F32: torch.float32}
        own = {BF16: gdn.GDN_BF16, F32: gdn.GDN_F32}
        self.lens, self.Hk, self.Hv, self.d, self.out = lens, Hk, Hv, d, out
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        T, n = int(self.cu[-1]), len(lens)
        r = torch.Generator().manual_seed(seed)
        wide = (2 * Hk + Hv) * d
        x = torch.randn((T, wide + pad), generator=r).to(kinds[dtype])
        self.x = x.cuda()
        self.split()
        gg = -decay * torch.nn.functional.softplus(2 * torch.randn((1 if fixed else T, Hv), generator=r)) if g is None else g
        self.g = (gg[0] if fixed else gg).float().contiguous().cuda()
        self.state = (0.5 * torch.randn((n + 2, Hv, d, d), generator=r)).cuda()
        self.slot = torch.randperm(n + 2, generator=r)[:n]
        self.o = torch.full((T, Hv, d), 7.0, dtype=kinds[out], device="cuda")
        self.scale = 0.37
        self.dims = gdn.make_linear_dims(Hk, Hv, d, in_dtype=own[dtype], out_dtype=own[out], scale=self.scale, mma=mma,
                                         prefill_form=form)
        self.ptrs = (self.state.data_ptr() + self.slot * (Hv * d * d * 4)).cuda()
        self.cu_dev = torch.tensor(self.cu, dtype=torch.int32, device="cuda")
        self.work = gdn.linear_workspace(self.dims, n, T)

    def split(self):
        a, b = self.Hk * self.d, 2 * self.Hk * self.d
        self.q, self.k, self.v = self.x[:, :a], self.x[:, a:b], self.x[:, b:b + self.Hv * self.d]

    def exact(self):
        T = self.x.shape[0]
        f = lambda t, h: t.double().cpu().numpy().reshape(T, h, self.d)  # noqa: E731
        g = np.broadcast_to(self.g.double().cpu().numpy(), (T, self.Hv))
        return (f(self.q, self.Hk), f(self.k, self.Hk), f(self.v, self.Hv), g, self.state.double().cpu().numpy()[self.slot.numpy()],
                self.scale, self.cu)

    def prefill(self, **kw):
        import gated_delta_rule_conv_amd as gdn

        gdn.linear_prefill(self.dims, self.q, self.k, self.v, self.g, self.o, self.cu_dev, self.ptrs, self.work, **kw)

    def decode(self, **kw):
        import gated_delta_rule_conv_amd as gdn

        gdn.linear_decode(self.dims, self.q, self.k, self.v, self.g, self.o, self.ptrs, **kw)


def near(got, want, tol, out):
    """|got - want| <= tol, plus half a step for bf16."""
    got = got.double().cpu().numpy()
    off = np.abs(got - want) - tol - (np.abs(want) + tol) * (2.0 ** -8 if out == BF16 else 0.0)
    assert np.isfinite(got).all()
    assert (off <= 0).all(), f"off by {np.abs(got - want).max()}, {off.max()} over"


def check(c, call):
    import torch

    args = c.exact()
    before = bits_of(c.state)
    call()
    torch.cuda.synchronize()
    (o, S), (to, tS) = packed(*args), bound(*args)
    near(c.o, o, to, c.out)
    near(c.state[c.slot], S, tS, F32)
    idle = [i for i in range(len(c.state)) if i not in c.slot.tolist()]
    assert (bits_of(c.state)[idle] == before[idle]).all()


@pytest.mark.parametrize("dtype,out", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("fixed", [False, True])
def test_prefill_of_ragged_prompts(dtype, out, d, fixed):
    announce(f"linear prefill ragged d={d} {dtype}->{out} fixed={fixed}")
    c = Case([1, 17, 0, 64, 65, 300, 2, 128, 63], d=d, dtype=dtype, out=out, fixed=fixed, seed=d)
    check(c, c.prefill)


@pytest.mark.parametrize("lens", [[1], [2], [63], [64], [65], [127], [129], [700], [1, 1, 1], [0, 5, 0], [513, 511, 1025]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_lengths(lens, dtype):
    announce(f"linear prefill lengths {lens} {dtype}")
    c = Case(lens, Hk=1, Hv=2, d=64, dtype=dtype, seed=3)
    check(c, c.prefill)


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 5), (3, 3), (2, 8), (16, 32)])
@pytest.mark.parametrize("form", [0, 1, 2])
def test_prefill_head_layouts_and_forms(Hk, Hv, form):
    announce(f"linear prefill heads {Hk}/{Hv} form {form}")
    c = Case([150, 30, 600] if Hv < 16 else [40, 530], Hk=Hk, Hv=Hv, d=128 if Hv >= 5 else 64, seed=Hv, form=form)
    check(c, c.prefill)


@pytest.mark.parametrize("decay", [0.0, 1e-3, 3.0, 40.0])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_decays_from_none_to_all(decay, dtype):
    announce(f"linear prefill decay {decay} {dtype}")
    c = Case([200, 77], Hk=1, Hv=2, d=128, dtype=dtype, seed=5, decay=decay)
    check(c, c.prefill)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decays_that_keep_nothing(dtype):
    """g of minus infinity starts the state anew at its token, and mild tokens behind a strong one keep their digits."""
    import torch

    announce(f"linear prefill resets {dtype}")
    r = torch.Generator().manual_seed(8)
    g = -0.02 * torch.rand((150, 2), generator=r)
    g[0, 0], g[40, 0], g[41, 0], g[64, 0], g[128, 0] = -float("inf"), -float("inf"), -1e9, -float("inf"), -300.0
    g[20, 1], g[70, 1], g[100, 1] = -90.0, -120.0, -float("inf")
    c = Case([100, 50], Hk=1, Hv=2, d=64, dtype=dtype, seed=9, g=g)
    check(c, c.prefill)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_token_before_a_broken_one_is_touched(dtype):
    """Infinities and NaN in q, k, v and g reach no earlier token and no other sequence or head."""
    import torch

    for what in ("q", "k", "v", "g"):
        for bad in (float("nan"), float("inf")):
            announce(f"linear prefill {what} = {bad} {dtype}")
            clean, c = (Case([90, 100], Hk=2, Hv=4, d=64, dtype=dtype, seed=4) for _ in range(2))
            t, row, head = 30, 30 + 90, 1  # token 30 of the second sequence
            if what == "g":
                c.g[row, head] = bad if bad != bad else -bad
                if bad == bad:
                    clean.g[row, head] = -bad  # (minus infinity is a value like others)
            elif what == "v":
                c.v[row, head * 64 + 5] = bad
            else:
                getattr(c, what)[row, 0 * 64 + 5] = bad
            args = clean.exact()
            (o_exact, _), (o_bound, _) = packed(*args), bound(*args)
            clean.prefill()
            c.prefill()
            torch.cuda.synchronize()
            hit = {"q": [0, 1], "k": [0, 1], "v": [head], "g": [head]}[what]
            a, b = bits_of(c.o), bits_of(clean.o)
            others = [h for h in range(4) if h not in hit]
            assert (a[:, others] == b[:, others]).all()
            # (the chunk that holds a broken value is taken token by token: rounding may differ there)
            near(c.o[:row], o_exact[:row], o_bound[:row], F32)
            assert (a[:90] == b[:90]).all()
            o = c.o.float().cpu().numpy()
            if what == "q":
                assert not np.isfinite(o[row][hit]).any() and np.isfinite(o[row + 1:]).all()
                assert torch.isfinite(c.state).all()
            elif what == "k":
                assert not np.isfinite(o[row:, hit]).any()
            elif what == "v":
                assert not np.isfinite(o[row:, head, 5]).any()
                rest = [x for x in range(64) if x != 5]
                assert np.isfinite(o[row:, head][:, rest]).all()


def test_rows_and_slots_that_are_not_the_calls():
    """Rows behind the last sequence, inactive slots' rows and states stay as they were."""
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce("linear prefill: rows behind the last sequence, inactive slots")
    c = Case([70, 20, 40, 25], seed=6)
    c.cu_dev = torch.tensor([0, 70, 90, 130], dtype=torch.int32, device="cuda")  # (25 rows belong to nobody)
    ptrs = c.ptrs[:3].clone()
    ptrs[1] = 0
    before = bits_of(c.state)
    gdn.linear_prefill(c.dims, c.q, c.k, c.v, c.g, c.o, c.cu_dev, ptrs, c.work)
    torch.cuda.synchronize()
    o = c.o.float().cpu().numpy()
    assert (o[130:] == 7).all() and (o[70:90] == 7).all() and (o[:70] != 7).any() and (o[90:130] != 7).any()
    for i in (1, 3):
        assert (bits_of(c.state)[c.slot[i]] == before[c.slot[i]]).all()
    d = Case([1] * 5, seed=7)
    before = bits_of(d.state)
    d.ptrs[2] = 0
    d.decode()
    torch.cuda.synchronize()
    assert (d.o[2].float().cpu() == 7).all() and (bits_of(d.state)[d.slot[2]] == before[d.slot[2]]).all()


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 32), (BF16, 64)])
@pytest.mark.parametrize("form", [1, 2])
def test_a_sequence_has_the_same_bits_alone_and_packed(dtype, d, form):
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce(f"linear prefill packed = solo {dtype} d={d} form {form}")
    lens = [5, 600, 64, 129, 1, 320, 321]
    c = Case(lens, d=d, dtype=dtype, seed=2, form=form)
    first = c.state.clone()
    c.prefill()
    whole, end = bits_of(c.o), bits_of(c.state)
    for i, n in enumerate(lens):
        a, b = int(c.cu[i]), int(c.cu[i + 1])
        c.state.copy_(first)
        o = torch.empty_like(c.o[a:b])
        gdn.linear_prefill(c.dims, c.q[a:b], c.k[a:b], c.v[a:b], c.g[a:b], o, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                           c.ptrs[i:i + 1], gdn.linear_workspace(c.dims, 1, n))
        assert (bits_of(o) == whole[a:b]).all()
        assert (bits_of(c.state)[c.slot[i]] == end[c.slot[i]]).all()


def test_many_short_sequences():
    announce("linear prefill of 1100 short sequences")
    r = np.random.default_rng(0)
    c = Case([int(x) for x in r.integers(0, 7, 1100)], Hk=1, Hv=1, d=32, seed=1)
    check(c, c.prefill)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("many", [False, True])
def test_longer_tiles_in_larger_calls(dtype, many):
    """Calls whose tokens make the tiles of a long sequence longer, with few sequences and with more than 64."""
    announce(f"linear prefill of 9000 tokens {dtype} {many}")
    r = np.random.default_rng(4)
    short = [int(x) for x in r.integers(0, 60, 70)] if many else [257]
    c = Case(short[:-1] + [5000, 0, 321, 9000 - 5321 - sum(short[:-1])] + short[-1:], Hk=8, Hv=40, d=32, dtype=dtype, seed=17)
    check(c, c.prefill)


@pytest.mark.parametrize("dtype,out", [(BF16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("m,Hk,Hv", [(1, 2, 4), (7, 1, 3), (40, 16, 32)])
def test_decode(dtype, out, d, m, Hk, Hv):
    announce(f"linear decode m={m} {Hk}/{Hv} d={d} {dtype}->{out}")
    c = Case([1] * m, Hk=Hk, Hv=Hv, d=d, dtype=dtype, out=out, seed=m, fixed=m == 7)
    check(c, c.decode)


def test_decode_bits_do_not_depend_on_the_batch():
    import torch

    announce("linear decode batch = single")
    a, b = (Case([1] * 40, Hk=16, Hv=32, d=128, seed=3) for _ in range(2))
    a.decode()
    import gated_delta_rule_conv_amd as gdn

    for i in range(0, 40, 7):
        gdn.linear_decode(b.dims, b.q[i:i + 1], b.k[i:i + 1], b.v[i:i + 1], b.g[i:i + 1], b.o[i:i + 1], b.ptrs[i:i + 1])
        torch.cuda.synchronize()
        assert (bits_of(a.o[i]) == bits_of(b.o[i])).all()
        assert (bits_of(a.state[a.slot[i]]) == bits_of(b.state[b.slot[i]])).all()


def test_prefill_then_decode_is_a_longer_prefill():
    """Tokens 0 .. 99 as a prompt, 100 .. 119 one by one, against all at once in 64 bits."""
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce("linear prefill then decode")
    c = Case([120], Hk=2, Hv=4, d=64, seed=12)
    args = c.exact()
    cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    gdn.linear_prefill(c.dims, c.q[:100], c.k[:100], c.v[:100], c.g[:100], c.o[:100], cu, c.ptrs, c.work)
    for t in range(100, 120):
        gdn.linear_decode(c.dims, c.q[t:t + 1], c.k[t:t + 1], c.v[t:t + 1], c.g[t:t + 1], c.o[t:t + 1], c.ptrs)
    torch.cuda.synchronize()
    (o, S), (to, tS) = packed(*args), bound(*args)
    near(c.o, o, to, F32)  # (20 steps of decode add 2 roundings each: within the bound's doubling)
    near(c.state[c.slot], S, tS, F32)


def test_long_memory_over_many_chunks():
    """3000 tokens that forget next to nothing, against 64 bits on the GPU: within 1e-6 of the result's norm, the roundings of 200
    sums of random signs and 47 chunks (sqrt(200 + 47 + 128) 2^-24 = 1.2e-6 if all were as large as the last)."""
    import torch

    announce("linear prefill, 3000 tokens, slow decay")
    for dtype in (BF16, F32):
        c = Case([3000], Hk=1, Hv=2, d=128, dtype=dtype, seed=13, decay=2e-4)
        q, k, v = (t.double().view(3000, h, 128) for t, h in ((c.q, 1), (c.k, 1), (c.v, 2)))
        S, o, g = c.state[c.slot[0]].double(), torch.empty(3000, 2, 128, dtype=torch.float64, device="cuda"), c.g.double().exp()
        for t in range(3000):
            S = g[t][:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            o[t] = c.scale * (S * q[t][:, None, :]).sum(-1)
        c.prefill()
        torch.cuda.synchronize()
        assert float((c.o.double() - o).norm() / o.norm()) < 1.2e-6
        assert float((c.state[c.slot[0]].double() - S).norm() / S.norm()) < 1.2e-6


def test_captured_calls_replay():
    """A prefill and a decode captured once each, replayed with eager work between, equal the eager calls bit for bit."""
    import torch

    announce("linear prefill and decode in graphs")
    for lens in ([5, 600, 64], [1] * 6):
        c, e = (Case(lens, d=64, seed=14) for _ in range(2))
        calls = ("prefill", "decode") if len(lens) == 6 else ("prefill",)
        for name in calls:
            start = c.state.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                getattr(c, name)()
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                getattr(c, name)()
            c.state.copy_(start)
            e.state.copy_(start)
            for _ in range(4):
                c.o.fill_(3.0)
                graph.replay()
                getattr(e, name)()
                torch.cuda.synchronize()
                assert (bits_of(c.o) == bits_of(e.o)).all() and (bits_of(c.state) == bits_of(e.state)).all()


def test_two_streams_at_once():
    """Two calls on two streams, each with its own workspace."""
    import torch

    announce("linear prefill on two streams")
    a, b = Case([900, 40], seed=15), Case([700, 300], seed=16)
    ea, eb = Case([900, 40], seed=15), Case([700, 300], seed=16)
    ea.prefill()
    eb.prefill()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    a.prefill(stream=s)
    b.prefill(stream=t)
    torch.cuda.synchronize()
    for x, y in ((a, ea), (b, eb)):
        assert (bits_of(x.o) == bits_of(y.o)).all() and (bits_of(x.state) == bits_of(y.state)).all()
