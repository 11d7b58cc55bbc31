"""The operators of a hybrid model's serving loop run together as a program calls them: prompts through a linear attention layer,
its output norm and block norms, sampled tokens fed back step by step, slots copied and snapshotted between; and a
speculative step of a delta-rule layer whose drafts are sampled, followed and accepted on the GPU.

All in fp32, against 64 bits. An error of 1e-6 in a layer's output moves a border of a row's distribution by less than 1e-5 of
its sum here (logits of a few units), so tokens are compared where the random number is further than 1e-4 from every border
(asserted), and probabilities to 1e-4."""

import numpy as np
import pytest

from tests.gpu_helpers import announce, normwise_err
from tests.linear_ref import recurrence
from tests.sample_ref import distribution, sample

pytestmark = pytest.mark.gpu

HK, HV, D, VOCAB = 2, 4, 32, 211
W = HV * D


def away(x, u, **kw):
    ids, w = distribution(x, **kw)
    return np.abs(np.cumsum(w) / w.sum() - u).min() > 1e-4


def norm(x, w, eps=1e-6):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


class Model:
    """One linear attention layer between an embedding and its transpose; decays and the gate from the stream too."""

    def __init__(self, seed):
        r = np.random.default_rng(seed)
        f = lambda *s, std=1.0: (std * r.standard_normal(s)).astype(np.float32)  # noqa: E731
        self.embed, self.qkv = f(VOCAB, W), f(W, (2 * HK + HV) * D, std=W ** -0.5)
        self.gates, self.z, self.out = f(W, HV, std=W ** -0.5), f(W, W, std=W ** -0.5), f(W, W, std=W ** -0.5)
        self.pre, self.head, self.post, self.last = (1 + f(n, std=0.1) for n in (W, D, W, W))
        self.ls = f(W, std=0.5)
        self.scale, self.alpha = 0.3, 0.7

    def exact(self, tokens, S):
        """Logits [T, VOCAB] of one sequence's tokens after state S, and the new state, in 64 bits."""
        m = {k: v.astype(np.float64) for k, v in vars(self).items() if isinstance(v, np.ndarray)}
        r = m["embed"][tokens]
        y = norm(r, m["pre"])
        q, k, v = np.split(y @ m["qkv"], [HK * D, 2 * HK * D], axis=1)
        g = -np.logaddexp(0, y @ m["gates"]) * 0.1
        T = len(tokens)
        o, S = recurrence(q.reshape(T, HK, D), k.reshape(T, HK, D), v.reshape(T, HV, D), g, S, self.scale)
        z = y @ m["z"]
        o = (norm(o, m["head"]).reshape(T, W) * (z / (1 + np.exp(-z)))) @ m["out"]
        h = r + self.alpha * m["ls"] * norm(o, m["post"])
        return norm(h, m["last"]) @ m["embed"].T * 0.2, S


class OnGpu:
    def __init__(self, m, slots):
        import torch

        import gated_delta_rule_conv_amd as gdn

        self.m, self.gdn, self.torch = m, gdn, torch
        self.t = {k: torch.from_numpy(v).cuda() for k, v in vars(m).items() if isinstance(v, np.ndarray)}
        f32 = dict(in_dtype=gdn.GDN_F32, residual_dtype=gdn.GDN_F32, gate_dtype=gdn.GDN_F32, param_dtype=gdn.GDN_F32, out_dtype=gdn.GDN_F32)
        self.dims = gdn.make_linear_dims(HK, HV, D, in_dtype=gdn.GDN_F32, scale=m.scale)
        self.first, self.second = gdn.make_block_norm_dims(W, **f32), gdn.make_block_norm_dims(W, post_norm=True, scale=m.alpha, **f32)
        self.heads = gdn.make_norm_dims(HV, D, in_dtype=gdn.GDN_F32, gate_dtype=gdn.GDN_F32, param_dtype=gdn.GDN_F32, out_dtype=gdn.GDN_F32)
        self.pool = gdn.SlotPool(self.dims, slots)

    def logits(self, tokens, ptrs, cu=None):
        t, torch, gdn = self.t, self.torch, self.gdn
        r = t["embed"][tokens.long()]
        y, o, n = torch.empty_like(r), torch.empty(len(r), HV, D, device="cuda"), torch.empty_like(r)
        gdn.block_norm(self.first, r, None, y, pre_weight=t["pre"])
        x = y @ t["qkv"]
        q, k, v = x[:, :HK * D], x[:, HK * D:2 * HK * D], x[:, 2 * HK * D:]
        g = -torch.nn.functional.softplus(y @ t["gates"]) * 0.1
        if cu is None:
            gdn.linear_decode(self.dims, q, k, v, g, o, ptrs)
        else:
            gdn.linear_prefill(self.dims, q, k, v, g, o, cu, ptrs, gdn.linear_workspace(self.dims, len(ptrs), len(r)))
        gdn.group_norm(self.heads, o, t["head"], n, gate=y @ t["z"])
        gdn.block_norm(self.second, n @ t["out"], r, y, residual_out=r, gate=t["ls"], post_weight=t["post"], pre_weight=t["last"])
        return y @ t["embed"].t().contiguous() * 0.2


def test_prompts_then_sampled_tokens():
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce("hybrid run: prompts, 6 sampled steps, slots copied and stored between")
    m = Model(3)
    gpu = OnGpu(m, 8)
    r = np.random.default_rng(5)
    prompts = [r.integers(0, VOCAB, n) for n in (70, 3, 131)]
    S = [np.zeros((HV, D, D)) for _ in prompts]
    slots = torch.tensor([6, 1, 4], dtype=torch.int32, device="cuda")
    ptrs, _ = gpu.pool.pointers(slots)
    cu = torch.tensor(np.concatenate([[0], np.cumsum([len(p) for p in prompts])]), dtype=torch.int32, device="cuda")
    x = gpu.logits(torch.from_numpy(np.concatenate(prompts)).cuda(), ptrs, cu)[(cu[1:] - 1).long()].contiguous()
    kw = dict(t=0.9, k=40, p=0.95, least=0.02)
    par = {n: torch.full((3,), v, device="cuda") for n, v in (("temperature", 0.9), ("top_p", 0.95), ("min_p", 0.02))}
    par["top_k"] = torch.full((3,), 40, dtype=torch.int32, device="cuda")
    kw = {a: float(np.float32(b)) for a, b in kw.items()}
    kw["k"] = 40
    tokens, prob, work = (torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(3, device="cuda"), gdn.sample_workspace(3, VOCAB))
    want = list(prompts)
    for step in range(6):
        u = r.random(3).astype(np.float32)
        gdn.sample(x, torch.from_numpy(u).cuda(), tokens, work, prob=prob, **par)
        torch.cuda.synchronize()
        new = []
        for i in range(3):
            ref, S[i] = m.exact(want[i], S[i])
            got = x[i].double().cpu().numpy()
            assert normwise_err(got, ref[-1]) < 1e-5
            assert away(ref[-1], float(u[i]), **kw), "choose another seed"
            token, p = sample(ref[-1], float(u[i]), **kw)
            assert int(tokens[i]) == token and abs(float(prob[i]) - p) < 1e-4
            new.append([token])
        want = new
        if step == 2:  # the slots move to others, by way of the store for one
            to = torch.tensor([0, 5, 7], dtype=torch.int32, device="cuda")
            gpu.pool.copy_slots(slots, to, conv_state=False)
            gpu.pool.state[slots.long()] = float("nan")
            slots = to
            ptrs, _ = gpu.pool.pointers(slots)
        x = gpu.logits(tokens, ptrs)
    for i in range(3):
        _, S[i] = m.exact(want[i], S[i])
        assert normwise_err(gpu.pool.state[int(slots[i])].cpu().numpy(), S[i]) < 1e-5
    store = gdn.packed_slots(gpu.dims, 3, gdn.GDN_PACK_INT8)
    gpu.pool.pack_slots(slots, store, gdn.GDN_PACK_INT8, conv_state=False)
    before = gpu.pool.state[slots.long()].clone()
    gpu.pool.unpack_slots(store, torch.arange(3, dtype=torch.int32, device="cuda"), slots, gdn.GDN_PACK_INT8, conv_state=False)
    after = gpu.pool.state[slots.long()]
    assert ((after - before).abs() <= before.abs().amax(-1, keepdim=True) / 254 * 1.0001).all()


def test_sampled_drafts_are_what_decoding_gives():
    """Drafted trees verified, every node's token sampled, the path followed and accepted, against the same tokens decoded one
    by one with the path's random numbers."""
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce("speculative step with sampling and following")
    r = np.random.default_rng(11)
    f = lambda *s, std=1.0: torch.from_numpy((std * r.standard_normal(s)).astype(np.float32)).cuda()  # noqa: E731
    C, m = (2 * HK + HV) * D, 5
    dims = gdn.make_dims(HK, HV, D, in_dtype=gdn.GDN_F32)
    heads = gdn.make_norm_dims(HV, D, in_dtype=gdn.GDN_F32, param_dtype=gdn.GDN_F32, out_dtype=gdn.GDN_F32)
    embed, conv_w, nw, head = f(VOCAB, C), f(C, 4, std=0.4), 1 + f(D, std=0.1), f(W, VOCAB, std=W ** -0.5)
    gate, beta = -0.3 * torch.rand(VOCAB, HV, device="cuda"), torch.rand(VOCAB, HV, device="cuda")

    def new_pool():
        return gdn.SlotPool(dims, m, state=state0.clone(), conv_state=conv0.clone())

    state0, conv0 = f(m, HV, D, D, std=0.3), f(m, 3, C)
    idx = torch.arange(m, dtype=torch.int32, device="cuda")
    t = torch.full((1,), 0.8, device="cuda")

    def token_of(o, u):
        n = torch.empty(len(o), W, device="cuda")
        gdn.group_norm(heads, o, nw, n)
        out = torch.empty(len(o), dtype=torch.int32, device="cuda")
        gdn.sample(n @ head, u, out, gdn.sample_workspace(len(o), VOCAB), temperature=t.expand(len(o)).contiguous())
        return out

    depth, pending = 7, torch.from_numpy(r.integers(0, VOCAB, m)).int().cuda()
    u = torch.from_numpy(r.random((depth, m)).astype(np.float32)).cuda()
    plain, want = new_pool(), [pending]
    sp, cp = plain.pointers(idx)
    states, convs = [plain.state.clone()], [plain.conv_state.clone()]
    for d in range(depth):
        at, o = want[-1].long(), torch.empty(m, HV, D, device="cuda")
        gdn.decode_fused(dims, embed[at], conv_w, None, gate[at], beta[at], o, sp, cp)
        want.append(token_of(o, u[d]))
        states.append(plain.state.clone())
        convs.append(plain.conv_state.clone())
    truth = torch.stack(want).cpu().numpy()  # [depth + 1, m]: pending, then what decoding gives
    # trees: i right tokens in a row for slot i + 1, wrong siblings before and beside them, wrong tails
    drafted, parents, level, cu = [], [], [], [0]
    keep = [1, 2, 4, 7, 0]
    for i in range(m):
        at, n = -1, 0
        for d in range(depth):
            right = int(truth[d, i])
            wrong = (right + 1 + d) % VOCAB
            kids = [wrong, right, right, wrong] if d < keep[i] else [wrong, wrong]
            base = n
            for token in kids:
                drafted.append(token)
                parents.append(at)
                level.append(d)
                n += 1
            at = base + 1 if d < keep[i] else base
        cu.append(len(drafted))
    T = len(drafted)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    drafted, parents, cu = dev(drafted), dev(parents), dev(cu)
    seq = torch.repeat_interleave(torch.arange(m, device="cuda"), (cu[1:] - cu[:-1]).long())
    pool, rec = new_pool(), gdn.tree_record(dims, T)
    sp, cp = pool.pointers(idx)
    at, o = drafted.long(), torch.empty(T, HV, D, device="cuda")
    acc, nxt, path = dev([9] * m), pending.clone(), torch.empty(m, 32, dtype=torch.int32, device="cuda")
    gdn.tree_verify(dims, embed[at], conv_w, None, gate[at], beta[at], o, parents, cu, 32, sp, cp, record=rec)
    said = token_of(o, u[torch.tensor(level, device="cuda"), seq])
    gdn.tree_follow(drafted, said, nxt, parents, cu, 32, acc, nxt, path=path)
    gdn.tree_accept(dims, embed[at], rec, parents, cu, 32, acc, sp, cp)
    torch.cuda.synchronize()
    for i in range(m):
        steps = int((path[i] >= 0).sum())
        assert steps == keep[i] and int(nxt[i]) == truth[steps, i]
        assert drafted[int(cu[i]) + path[i][:steps].long()].tolist() == truth[:steps, i].tolist()
        assert int(acc[i]) == (int(path[i][steps - 1]) if steps else -1)
        assert normwise_err(pool.state[i].cpu().numpy(), states[steps][i].cpu().numpy()) < 1e-5
        assert torch.equal(pool.conv_state[i], convs[steps][i])


def test_one_step_on_another_stream_and_in_a_graph():
    """Norm, decode, output norm, norm, sampling and following with every operand fixed: on the current stream, on a stream that
    is given, and captured and replayed with eager work between; the same bits each time."""
    import torch

    import gated_delta_rule_conv_amd as gdn

    announce("hybrid step: streams and graphs")
    m, g = 5, torch.Generator().manual_seed(6)
    rand = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    gpu, r, g_t = OnGpu(Model(9), m), rand(m, W), -torch.rand(m, HV, generator=g).cuda()
    qkv, head, logits, u = rand(m, (2 * HK + HV) * D), rand(m, W), rand(m, 5000), torch.rand(m, generator=g).cuda()
    start = rand(m, HV, D, D)
    ptrs, _ = gpu.pool.pointers(torch.arange(m, dtype=torch.int32, device="cuda"))
    p = torch.full((m,), 0.9, device="cuda")
    drafted = torch.randint(0, 3, (4 * m,), dtype=torch.int32, generator=g).cuda()
    sampled = torch.randint(0, 3, (4 * m,), dtype=torch.int32, generator=g).cuda()
    cu = (4 * torch.arange(m + 1, dtype=torch.int32)).cuda()
    out = dict(h=torch.empty(m, W, device="cuda"), y=torch.empty(m, W, device="cuda"), o=torch.empty(m, HV, D, device="cuda"),
               n=torch.empty(m, W, device="cuda"), y2=torch.empty(m, W, device="cuda"),
               **{k: torch.empty(m, dtype=torch.int32, device="cuda") for k in ("tokens", "acc", "next")})
    work, pending = gdn.sample_workspace(m, 5000), torch.zeros(m, dtype=torch.int32, device="cuda")

    def step(stream=None):
        gdn.block_norm(gpu.first, head, r, out["y"], residual_out=out["h"], pre_weight=gpu.t["pre"], stream=stream)
        gdn.linear_decode(gpu.dims, qkv[:, :HK * D], qkv[:, HK * D:2 * HK * D], qkv[:, 2 * HK * D:], g_t, out["o"], ptrs, stream=stream)
        gdn.group_norm(gpu.heads, out["o"], gpu.t["head"], out["n"], gate=out["y"], stream=stream)
        gdn.block_norm(gpu.second, out["n"], out["h"], out["y2"], gate=gpu.t["ls"], post_weight=gpu.t["post"], stream=stream)
        gdn.sample(logits, u, out["tokens"], work, top_p=p, stream=stream)
        gdn.tree_follow(drafted, sampled, pending, None, cu, 4, out["acc"], out["next"], stream=stream)

    def clear():
        gpu.pool.state.copy_(start)
        for t in out.values():
            t.fill_(7)

    def bits():
        torch.cuda.synchronize()
        return [t.cpu().numpy().tobytes() for t in (*out.values(), gpu.pool.state)]

    clear()
    step()
    want = bits()
    side = torch.cuda.Stream()
    clear()
    side.wait_stream(torch.cuda.current_stream())
    step(side)  # (not the current stream)
    assert bits() == want
    graph = torch.cuda.CUDAGraph()
    clear()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        clear()
        graph.replay()
        assert bits() == want
        clear()
        step()
        assert bits() == want
