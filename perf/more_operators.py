"""The operators beside the layer core in a hybrid model's serving step, as measured cases.

  prefill  linear attention with a decay for each head over packed prompts, slots of state
           in place
  decode   the same for one token of every slot
  block    the norm after a block, its gate and scale, the residual sum and the norm before
           the next block
  sample   one token a row of logits from a given random number: temperature, top-k, top-p,
           min-p
  follow   the path of a drafted tree that the sampled tokens take

With ``own`` false, run() computes them in elementary torch operations; with ``own`` true
it calls the library.
"""

import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
TORCH = {BF16: torch.bfloat16, F32: torch.float32}
SIZE = {BF16: 2, F32: 4, "none": 0}
DEVICE = "cuda"
CHUNK = 64  # tokens the plain form of prefill takes together

# ------------------------------------------------------------------------------ cases


def _heads(hk, hv, d, dtype, out=F32, fixed=False):
    """fixed: one decay a head for all tokens; else one for every token."""
    return {"hk": hk, "hv": hv, "d": d, "dtype": dtype, "out": out, "fixed": fixed}


def _sampler(rows, vocab, dtype, temperature=True, top_k=True, top_p=True, min_p=True, spread=2.5):
    return {"rows": rows, "vocab": vocab, "dtype": dtype, "temperature": temperature, "top_k": top_k, "top_p": top_p,
            "min_p": min_p, "spread": spread}


def listed():
    return [
        # one short prompt through a small fp32 layer: the smallest prefill
        {"name": "prefill_f32_37", "op": "prefill", **_heads(2, 4, 64, F32, fixed=True), "lengths": "37"},
        # one prompt of 4096 tokens, 16 k-heads and 32 v-heads, decays given by the tokens, bf16 outputs
        {"name": "prefill_4096_bf16", "op": "prefill", **_heads(16, 32, 128, BF16, BF16), "lengths": "4096"},
        # the ragged pack of prompts, one decay a head
        {"name": "prefill_ragged_15717", "op": "prefill", **_heads(16, 32, 128, BF16, fixed=True),
         "lengths": "1 17 64 300 1000 2048 4095 8192"},
        # one stream's next token
        {"name": "decode_1", "op": "decode", **_heads(16, 32, 128, BF16, BF16), "m": 1},
        # a full batch's next tokens
        {"name": "decode_64", "op": "decode", **_heads(16, 32, 128, BF16, fixed=True), "m": 64},
        # between two blocks in a decode step of 64 slots: both norms, a gate a channel, bf16 stream
        {"name": "block_64", "op": "block", "rows": 64, "width": 4096, "x": BF16, "residual": BF16, "gate": BF16, "y": BF16,
         "param": BF16, "vector_gate": True, "act": "none", "post": True, "centered": False, "scale": 1.0},
        # between two blocks in the ragged prefill: gated by the tokens, fp32 stream, scaled residual
        {"name": "block_15717", "op": "block", "rows": 15717, "width": 4096, "x": BF16, "residual": F32, "gate": BF16,
         "y": BF16, "param": BF16, "vector_gate": False, "act": "sigmoid", "post": True, "centered": False, "scale": 0.5},
        # one stream's token: latency
        {"name": "sample_1", "op": "sample", **_sampler(1, 131072, BF16)},
        # a batch, every filter, fp32 logits of an odd vocabulary
        {"name": "sample_64_f32", "op": "sample", **_sampler(64, 99991, F32)},
        # every node of 64 drafted trees of 16, temperature alone
        {"name": "sample_1024_plain", "op": "sample", **_sampler(1024, 131072, BF16, top_k=False, top_p=False, min_p=False)},
        # one stream with a chain of 4 drafts
        {"name": "follow_1_chain4", "op": "follow", "m": 1, "nodes": 4, "chain": True},
        # a batch of the largest trees
        {"name": "follow_512_tree64", "op": "follow", "m": 512, "nodes": 64, "chain": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "block", "sample", "sample", "follow"])
    if op == "block":
        width = _log(rng, 64, 16384)
        gate = rng.choice([F32, BF16, BF16, "none"])
        return {"op": op, "rows": _log(rng, 1, max(1, min(20000, 15717 * 4096 // width))), "width": width,
                "x": rng.choice([F32, BF16, BF16]), "residual": rng.choice([F32, BF16]), "gate": gate, "y": rng.choice([F32, BF16, BF16]),
                "param": rng.choice([F32, BF16]), "vector_gate": rng.random() < 0.5,
                "act": rng.choice(["none", "silu", "sigmoid"]), "post": rng.random() < 0.7, "centered": rng.random() < 0.3,
                "scale": rng.choice([1.0, 0.5, 0.22])}
    if op == "sample":
        vocab = _log(rng, 40, 260000)
        return {"op": op, **_sampler(_log(rng, 1, max(1, min(1024, 60000000 // vocab))), vocab, rng.choice([F32, BF16]), rng.random() < 0.8,
                                     rng.random() < 0.5, rng.random() < 0.6, rng.random() < 0.4, rng.choice([0.3, 1.0, 2.5, 6.0]))}
    if op == "follow":
        return {"op": op, "m": _log(rng, 1, 512), "nodes": _log(rng, 1, 64), "chain": rng.random() < 0.3}
    hk = _log(rng, 1, 16)
    d = rng.choice([32, 64, 128, 128])
    c = _heads(hk, hk * rng.choice([1, 2, 2, 3, 4]), d, rng.choice([BF16, BF16, F32]), rng.choice([F32, BF16]), rng.random() < 0.5)
    if op == "decode":
        return {"op": op, **c, "m": _log(rng, 1, max(1, min(300, 64 * 32 * 128 * 128 // (c["hv"] * d * d))))}
    tokens = _log(rng, 1, max(1, min(15717, 15717 * 32 * 128 // (c["hv"] * d * (1 if c["dtype"] == BF16 else 2)))))
    n = min(tokens, _log(rng, 1, 48))
    cuts = [0] + sorted(rng.randint(0, tokens) for _ in range(n - 1)) + [tokens]
    return {"op": op, **c, "lengths": " ".join(str(b - a) for a, b in zip(cuts, cuts[1:]))}


# ----------------------------------------------------------------------------- inputs


def _normal(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32) * std).to(dtype)


def _uniform(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _prepare_heads(c, gen, rows, slots):
    """q, k and v as columns of one projection's rows; a pool of slots in a shuffled order."""
    hk, hv, d, dt = c["hk"], c["hv"], c["d"], TORCH[c["dtype"]]
    x = _normal(gen, rows, (2 * hk + hv) * d + 64, dtype=dt)
    c["q"], c["k"], c["v"] = x[:, :hk * d], x[:, hk * d:2 * hk * d], x[:, 2 * hk * d:(2 * hk + hv) * d]
    if c["fixed"]:  # from half a token's memory to that of thousands
        c["g"] = -torch.exp2(-12.0 * torch.arange(hv, device=DEVICE, dtype=torch.float32) / max(1, hv - 1))
    else:
        c["g"] = -0.2 * torch.nn.functional.softplus(_normal(gen, rows, hv, std=2.0))
    c["scale"] = d ** -0.5
    c["state"] = _normal(gen, slots + 3, hv, d, d, std=0.05)
    c["slot"] = torch.randperm(slots + 3, generator=gen, device=DEVICE)[:slots]
    c["state_ptrs"] = c["state"].data_ptr() + c["slot"] * (hv * d * d * 4)
    c["o"] = torch.empty(rows, hv, d, dtype=TORCH[c["out"]], device=DEVICE)


def _prepare_block(c, gen):
    rows, width = c["rows"], c["width"]
    c["x_t"] = _normal(gen, rows, width, dtype=TORCH[c["x"]])
    c["r_t"] = _normal(gen, rows, width, std=3.0, dtype=TORCH[c["residual"]])
    c["z_t"] = None
    if c["gate"] != "none":
        c["z_t"] = _normal(gen, width if c["vector_gate"] else rows * width, dtype=TORCH[c["gate"]])
        c["z_t"] = c["z_t"] if c["vector_gate"] else c["z_t"].view(rows, width)
    c["post_w"] = (1.0 + 0.1 * _normal(gen, width)).to(TORCH[c["param"]]) if c["post"] else None
    c["pre_w"] = (1.0 + 0.1 * _normal(gen, width)).to(TORCH[c["param"]])
    c["h_t"] = torch.empty_like(c["r_t"])
    c["y_t"] = torch.empty(rows, width, dtype=TORCH[c["y"]], device=DEVICE)


def _prepare_sample(c, gen):
    rows, vocab = c["rows"], c["vocab"]
    # one row in eight from a grammar that bans most of its tokens, every fiftieth with all of them banned
    c["logits"] = _normal(gen, rows, vocab, std=c["spread"], dtype=TORCH[c["dtype"]])
    row = torch.arange(rows, device=DEVICE)
    for first in range(3, rows, 8):
        c["logits"][first].masked_fill_(_uniform(gen, vocab) < 0.99, -math.inf)
    c["logits"][49::50] = -math.inf
    c["u"] = _uniform(gen, rows)
    u = _uniform(gen, 4, rows)
    c["t"] = torch.where(row % 7 == 5, 0.0, 0.5 + u[0]) if c["temperature"] else None  # (0: the likeliest)
    c["k"] = torch.where(row % 5 == 4, 0, (10 * (100 ** u[1])).int()).int() if c["top_k"] else None  # (0: all)
    c["p"] = 0.6 + 0.4 * u[2] if c["top_p"] else None
    c["min"] = 0.1 * u[3] if c["min_p"] else None
    c["tokens"] = torch.empty(rows, dtype=torch.int32, device=DEVICE)
    c["prob"] = torch.empty(rows, dtype=torch.float32, device=DEVICE)


def _sizes(c):
    """Trees of between nodes / 2 and nodes nodes, the first slot's the largest."""
    return [c["nodes"] - i * 5 % (c["nodes"] // 2 + 1) for i in range(c["m"])]


def _prepare_follow(c, gen):
    lens = torch.tensor(_sizes(c), device=DEVICE)
    c["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEVICE), lens.cumsum(0)]).to(torch.int32)
    total = c["total"] = int(c["cu"][-1])
    seq = torch.searchsorted(c["cu"][1:].contiguous(), torch.arange(total, device=DEVICE, dtype=torch.int32), right=True)
    local = torch.arange(total, device=DEVICE) - c["cu"][seq]
    if c["chain"]:
        parents = local - 1
    else:  # any earlier node, the slot itself for the first
        parents = torch.minimum((_uniform(gen, total) * local).floor().long(), local - 1)
    c["parents"] = parents.to(torch.int32)
    c["pending"] = (_uniform(gen, c["m"]) * 100000).to(torch.int32)
    c["sampled"] = (_uniform(gen, total) * 100000).to(torch.int32)
    # three drafts in four are what the model then says
    above = torch.where(parents < 0, c["pending"][seq], c["sampled"][(c["cu"][seq] + parents).clamp(min=0)])
    c["drafted"] = torch.where(_uniform(gen, total) < 0.75, above, (_uniform(gen, total) * 100000).to(torch.int32)).to(torch.int32)
    c["accepted"] = torch.empty(c["m"], dtype=torch.int32, device=DEVICE)
    c["next"] = torch.empty(c["m"], dtype=torch.int32, device=DEVICE)
    c["path"] = torch.empty(c["m"], c["nodes"], dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    if c["op"] == "prefill":
        lens = [int(x) for x in c["lengths"].split()]
        _prepare_heads(c, gen, sum(lens), len(lens))
        c["cu"] = torch.tensor([0] + lens, device=DEVICE).cumsum(0).to(torch.int32)
    elif c["op"] == "decode":
        _prepare_heads(c, gen, c["m"], c["m"])
    else:
        {"block": _prepare_block, "sample": _prepare_sample, "follow": _prepare_follow}[c["op"]](c, gen)
    return c


# ------------------------------------------------------------------------- plain forms


def _prefill(c):
    """Chunks of every sequence's tokens: scores inside a chunk, what a chunk adds to the state, and the state
    before a chunk as the decayed sum of what the chunks before it added."""
    hk, hv, d, cu = c["hk"], c["hv"], c["d"], c["cu"].long()
    rows, n = c["q"].shape[0], cu.numel() - 1
    chunks = (cu[1:] - cu[:-1] + CHUNK - 1) // CHUNK
    first = torch.cat([torch.zeros_like(chunks[:1]), chunks.cumsum(0)])  # a sequence's first chunk
    most = rows // CHUNK + n
    chunk = torch.arange(most, device=cu.device)
    seq = torch.searchsorted(first[1:].contiguous(), chunk, right=True).clamp(max=n - 1)
    at = cu[seq, None] + (chunk - first[seq])[:, None] * CHUNK + torch.arange(CHUNK, device=cu.device)
    there = (at < cu[seq + 1][:, None]) & (chunk < first[-1])[:, None]
    at = at.clamp(max=rows - 1)

    def heads(x, h):  # [chunks, hv, CHUNK, d]
        x = torch.where(there[..., None], x.float()[at], 0.0).view(most, CHUNK, h, d)
        return x.transpose(1, 2).repeat_interleave(hv // h, 1)

    q, k, v = heads(c["q"], hk), heads(c["k"], hk), heads(c["v"], hv)
    g = c["g"].double().expand(rows, hv)[at]
    g = torch.where(there[..., None], g, 0.0).cumsum(1).transpose(1, 2)  # [chunks, hv, CHUNK]
    lower = torch.ones(CHUNK, CHUNK, device=cu.device).tril() > 0
    decay = torch.exp(torch.where(lower, g[..., :, None] - g[..., None, :], -math.inf)).float()
    o = (q @ k.transpose(-1, -2).contiguous() * decay) @ v
    added = (v * torch.exp(g[..., -1:] - g).float()[..., None]).transpose(-1, -2).contiguous() @ k
    # [hv, chunks + 1]: the sum of g before each chunk
    before = torch.cat([torch.zeros(hv, 1, dtype=torch.float64, device=cu.device), g[..., -1].t().cumsum(1)], 1)
    earlier = (seq[None, :] == seq[:, None]) & (chunk[None, :] < chunk[:, None])
    carry = torch.exp(torch.where(earlier, before[:, :-1, None] - before[:, None, 1:], -math.inf)).float()
    added = added.transpose(0, 1).reshape(hv, most, d * d)
    start = c["state"][c["slot"]]  # [n, hv, d, d]
    kept = torch.exp(before[:, :-1] - before[:, first[seq]]).float()
    state = (carry @ added).view(hv, most, d, d).transpose(0, 1) + kept.t()[..., None, None] * start[seq]
    o = o + torch.exp(g).float()[..., None] * (q @ state.transpose(-1, -2).contiguous())
    mine = (seq[None, :] == torch.arange(n, device=cu.device)[:, None]) & (chunk < first[-1])
    tail = torch.exp(torch.where(mine, before[:, first[1:], None] - before[:, None, 1:], -math.inf)).float()
    end = (tail @ added).view(hv, n, d, d).transpose(0, 1)
    end = end + torch.exp(before[:, first[1:]] - before[:, first[:-1]]).float().t()[..., None, None] * start
    c["state"][c["slot"]] = end
    token = torch.arange(rows, device=cu.device)
    of = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    place = token - cu[of]
    o = o[first[of] + place // CHUNK, :, place % CHUNK]
    return {"o": (o * c["scale"]).to(TORCH[c["out"]]), "state": c["state"]}


def _decode(c):
    hk, hv, d, m = c["hk"], c["hv"], c["d"], c["m"]
    q, k = (x.float().view(m, hk, d).repeat_interleave(hv // hk, 1) for x in (c["q"], c["k"]))
    v = c["v"].float().view(m, hv, d)
    g = torch.exp(c["g"].expand(m, hv))[..., None, None]
    s = c["state"][c["slot"]] * g + v[..., :, None] * k[..., None, :]
    o = (s * q[..., None, :]).sum(-1) * c["scale"]
    c["state"][c["slot"]] = s
    return {"o": o.to(TORCH[c["out"]]), "state": c["state"]}


def _normed(x, w, centered):
    if centered:
        x = x - x.mean(-1, keepdim=True)
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5) * w.float()


def _block(c):
    a = c["x_t"].float()
    if c["post"]:
        a = _normed(a, c["post_w"], c["centered"])
    if c["z_t"] is not None:
        z = c["z_t"].float()
        if c["act"] == "sigmoid":
            z = torch.sigmoid(z)
        elif c["act"] == "silu":
            z = z * torch.sigmoid(z)
        a = a * z
    h = c["r_t"].float() + c["scale"] * a
    return {"h": h.to(c["h_t"].dtype), "y": _normed(h, c["pre_w"], c["centered"]).to(c["y_t"].dtype)}


def _sample(c):
    """Weights e^((x - largest) / temperature) in 64 bits; kept: the first k of the order by value (the lower index first among
    equals), of those the shortest beginning that holds the share p of their weight, of those the weights from min_p up. The
    token is the first, by index, with which the kept weight passes u times its sum; with it its share of the sum."""
    x = c["logits"].float() + 0.0
    rows, vocab = x.shape
    x = torch.where(torch.isnan(x), -math.inf, x)
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    top = x[:, :1].double()
    t = c["t"].double()[:, None] if c["t"] is not None else torch.ones_like(top)
    w = torch.exp((x.double() - top) / torch.where(t > 0, t, 1.0))
    w = torch.where(t > 0, w, 0.0)
    w = torch.where(torch.isnan(w), 0.0, w)
    w[:, 0] = 1.0
    place = torch.arange(vocab, device=x.device)
    if c["k"] is not None:
        k = c["k"].long()[:, None]
        w = torch.where((place < k) | (k <= 0), w, 0.0)
    if c["p"] is not None:
        p = c["p"].double()[:, None]
        before = w.cumsum(1) - w
        w = torch.where((before < p * w.sum(1, keepdim=True)) | (place == 0) | (p >= 1), w, 0.0)
    if c["min"] is not None:
        w = torch.where(w >= c["min"].double()[:, None].clamp(max=1.0), w, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, w)
    sums = w.cumsum(1)
    hit = sums > c["u"].double()[:, None] * sums[:, -1:]
    token = hit.int().argmax(1)
    some = top[:, 0] > -math.inf
    prob = w.gather(1, token[:, None])[:, 0] / sums[:, -1]
    return {"tokens": torch.where(some, token, -1).int(), "prob": torch.where(some, prob, 0.0).float()}


def _follow(c):
    cu, n, m = c["cu"].long(), c["nodes"], c["m"]
    node = torch.arange(n, device=cu.device)
    rows = cu[:-1, None] + node
    there = rows < cu[1:, None]
    rows = rows.clamp(max=c["total"] - 1)
    up = torch.where(there, c["parents"].long()[rows], -1)
    drafted, sampled = c["drafted"].long()[rows], c["sampled"].long()[rows]
    wanted = torch.where(up < 0, c["pending"].long()[:, None], sampled.gather(1, up.clamp(min=0)))
    good = there & (drafted == wanted) & (drafted >= 0)
    same = (up[:, :, None] == up[:, None, :]) & good[:, None, :] & (node[None, :] < node[:, None])
    good = good & ~same.any(-1)  # the first of equal siblings

    def climb(good, up):
        over = up.clamp(min=0)
        return good & ((up < 0) | good.gather(1, over)), torch.where(up < 0, up, up.gather(1, over))

    good, up = climb(*climb(*climb(*climb(*climb(*climb(good, up))))))
    last = torch.where(good, node, -1).amax(1)
    follows = torch.where(last < 0, c["pending"].long(), sampled.gather(1, last.clamp(min=0)[:, None])[:, 0])
    path = torch.where(good, node, n).sort(1)[0]
    return {"accepted": last.int(), "next": follows.int(), "path": torch.where(path < n, path, -1).int()}


# -------------------------------------------------------------------- the library's calls


def _own(c):
    import gated_delta_rule_conv_amd as gdn

    kinds = {BF16: gdn.GDN_BF16, F32: gdn.GDN_F32, "none": gdn.GDN_F32}
    if c["op"] in ("prefill", "decode"):
        if "dims" not in c:
            c["dims"] = gdn.make_linear_dims(c["hk"], c["hv"], c["d"], in_dtype=kinds[c["dtype"]], out_dtype=kinds[c["out"]],
                                             scale=c["scale"])
            if c["op"] == "prefill":
                c["work"] = gdn.linear_workspace(c["dims"], c["slot"].numel(), c["q"].shape[0])
        if c["op"] == "prefill":
            gdn.linear_prefill(c["dims"], c["q"], c["k"], c["v"], c["g"], c["o"], c["cu"], c["state_ptrs"], c["work"])
        else:
            gdn.linear_decode(c["dims"], c["q"], c["k"], c["v"], c["g"], c["o"], c["state_ptrs"])
        return {"o": c["o"], "state": c["state"]}
    if c["op"] == "block":
        if "dims" not in c:
            acts = {"none": gdn.GDN_ACT_NONE, "silu": gdn.GDN_ACT_SILU, "sigmoid": gdn.GDN_ACT_SIGMOID}
            c["dims"] = gdn.make_block_norm_dims(
                c["width"], in_dtype=kinds[c["x"]], residual_dtype=kinds[c["residual"]], gate_dtype=kinds[c["gate"]],
                param_dtype=kinds[c["param"]], out_dtype=kinds[c["y"]], activation=acts[c["act"]], post_norm=c["post"],
                centered=c["centered"], scale=c["scale"], eps=1e-5)
        gdn.block_norm(c["dims"], c["x_t"], c["r_t"], c["y_t"], residual_out=c["h_t"], gate=c["z_t"], post_weight=c["post_w"],
                       pre_weight=c["pre_w"])
        return {"h": c["h_t"], "y": c["y_t"]}
    if c["op"] == "sample":
        if "work" not in c:
            c["work"] = gdn.sample_workspace(c["rows"], c["vocab"])
        gdn.sample(c["logits"], c["u"], c["tokens"], c["work"], temperature=c["t"], top_k=c["k"], top_p=c["p"], min_p=c["min"],
                   prob=c["prob"])
        return {"tokens": c["tokens"], "prob": c["prob"]}
    gdn.tree_follow(c["drafted"], c["sampled"], c["pending"], c["parents"], c["cu"], c["nodes"], c["accepted"], c["next"],
                    path=c["path"])
    return {"accepted": c["accepted"], "next": c["next"], "path": c["path"]}


def run(state):
    if own:
        return _own(state)
    return {"prefill": _prefill, "decode": _decode, "block": _block, "sample": _sample, "follow": _follow}[state["op"]](state)


# -------------------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "block":
        n = c["rows"] * c["width"]
        gate = SIZE[c["gate"]] * (c["width"] if c["vector_gate"] else n)
        return {"bytes": n * (SIZE[c["x"]] + 2 * SIZE[c["residual"]] + SIZE[c["y"]]) + gate, "flops": 15 * n}
    if c["op"] == "sample":
        return {"bytes": c["rows"] * (c["vocab"] * SIZE[c["dtype"]] + 28), "flops": 10 * c["rows"] * c["vocab"]}
    if c["op"] == "follow":
        total = sum(_sizes(c))
        return {"bytes": 12 * total + 4 * c["m"] * (4 + c["nodes"]), "flops": 2 * total}
    hk, hv, d = c["hk"], c["hv"], c["d"]
    lens = [1] * c["m"] if c["op"] == "decode" else [int(x) for x in c["lengths"].split()]
    rows, state = sum(lens), 4 * hv * d * d
    moved = 2 * state * sum(x > 0 for x in lens) + rows * ((2 * hk + hv) * d * SIZE[c["dtype"]] + hv * d * SIZE[c["out"]])
    moved += 4 * hv * (1 if c["fixed"] else rows)
    # S q and v k^T for every token: no form takes less
    return {"bytes": moved, "flops": rows * hv * 4 * d * d}


# ------------------------------------------------------------------------------- exact


def _np(t):
    return t.detach().double().cpu().numpy()


def _exact_linear(c):
    """Token by token, all sequences side by side, in 64 bits."""
    hk, hv, d = c["hk"], c["hv"], c["d"]
    rows, n = c["q"].shape[0], c["slot"].numel()
    cu = torch.arange(n + 1, device=DEVICE) if c["op"] == "decode" else c["cu"].long()
    lens = cu[1:] - cu[:-1]
    s = c["state"][c["slot"]].double()
    o = torch.zeros(rows, hv, d, dtype=torch.float64, device=DEVICE)
    for t in range(int(lens.max())):
        live = (lens > t).nonzero()[:, 0]
        at = cu[live] + t
        q, k = (x[at].double().view(-1, hk, 1, d).expand(-1, hk, hv // hk, d).reshape(-1, hv, d) for x in (c["q"], c["k"]))
        f = (c["g"] if c["fixed"] else c["g"][at]).double().exp()
        now = s[live] * f.reshape(-1, hv, 1, 1) + torch.einsum("shv,shk->shvk", c["v"][at].double().view(-1, hv, d), k)
        s[live] = now
        o[at] = (now * q[:, :, None, :]).sum(-1) * c["scale"]
    state = c["state"].double()
    state[c["slot"]] = s
    return {"o": _np(o), "state": _np(state)}


def _exact_block(c):
    def norm(t, w):
        t = t - t.mean(1, keepdim=True) if c["centered"] else t
        return t * torch.rsqrt(t.pow(2).mean(1, keepdim=True) + 1e-5) * w.double()

    a = c["x_t"].double()
    a = norm(a, c["post_w"]) if c["post"] else a
    if c["z_t"] is not None:
        z = c["z_t"].double()
        soft = 1 / (1 + torch.exp(-z))
        a = a * {"none": z, "sigmoid": soft, "silu": z * soft}[c["act"]]
    h = c["r_t"].double() + c["scale"] * a
    return {"h": _np(h), "y": _np(norm(h, c["pre_w"]))}


def _exact_sample(c):
    x, u = c["logits"].float().cpu().numpy().astype(np.float64), c["u"].double().tolist()
    given = [None if c[n] is None else c[n].double().tolist() for n in ("t", "k", "p", "min")]
    out, prob = [], []
    for r in range(c["rows"]):
        t, k, p, least = (g[r] if g else off for g, off in zip(given, (1.0, 0, 1.0, 0.0)))
        row = x[r]
        top = row.max()
        if top == -np.inf:
            out.append(-1)
            prob.append(0.0)
            continue
        if t <= 0:
            out.append(int(np.flatnonzero(row == top)[0]))
            prob.append(1.0)
            continue
        ids = np.lexsort((np.arange(row.size), -row))
        ids = ids[:int(k)] if k > 0 else ids
        w = np.exp((row[ids] - top) / t)
        if p < 1:
            share = np.concatenate([[0.0], np.cumsum(w)])
            w = w[:max(1, int(np.searchsorted(share[:-1], p * share[-1])))]
        ids = ids[:w.size][w >= min(least, 1.0)]
        ids = np.sort(ids)
        share = np.cumsum(np.exp((row[ids] - top) / t))
        at = np.searchsorted(share, u[r] * share[-1], side="right")
        out.append(int(ids[at]))
        prob.append(np.exp((row[ids[at]] - top) / t) / share[-1])
    return {"tokens": np.array(out, dtype=np.int32), "prob": np.array(prob)}


def _exact_follow(c):
    cu, up, drafted, sampled = (c[n].tolist() for n in ("cu", "parents", "drafted", "sampled"))
    accepted, follows, paths = [], [], []
    for i, want in enumerate(c["pending"].tolist()):
        at, path = -1, []
        while True:
            child = [j for j in range(cu[i + 1] - cu[i]) if up[cu[i] + j] == at and drafted[cu[i] + j] == want]
            if not child:
                break
            at = child[0]
            path.append(at)
            want = sampled[cu[i] + at]
        accepted.append(at)
        follows.append(want)
        paths.append(path + [-1] * (c["nodes"] - len(path)))
    return {"accepted": np.array(accepted, np.int32), "next": np.array(follows, np.int32), "path": np.array(paths, np.int32)}


def exact(case, seed):
    if case["op"] == "sample" and case["rows"] * case["vocab"] > 60000000:
        return None
    c = prepare(case, seed)
    return {"prefill": _exact_linear, "decode": _exact_linear, "block": _exact_block, "sample": _exact_sample,
            "follow": _exact_follow}[c["op"]](c)
