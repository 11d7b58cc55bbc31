"""The operators of a serving loop around the layer core, as measured cases.

  verify  a tree of drafted tokens per slot answered against the slot's state and conv
          state, which stay as they are
  accept  the slots moved along the accepted root paths
  pack    slots written into 8-bit snapshots
  unpack  8-bit snapshots read back into slots
  norm    the norm of every head of every token, times the activated gate

With ``own`` false, run() computes them in elementary torch operations; with ``own`` true
it calls the library.
"""

import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
TORCH = {BF16: torch.bfloat16, F32: torch.float32}
TOP = {"int8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -100  # rows below this magnitude are packed as zeros

# ------------------------------------------------------------------------------ cases


def _layer(hk, hv, d, dtype, width=4, silu=False, bias=False, out=F32):
    return {"hk": hk, "hv": hv, "d": d, "dtype": dtype, "width": width, "silu": silu, "bias": bias, "out": out}


BIG = _layer(16, 32, 128, BF16)


def listed():
    return [
        # one stream, a chain of 4 tokens from a one-head drafter: the smallest step, where latency counts
        {"name": "verify_m1_chain4", "op": "verify", **BIG, "m": 1, "nodes": 4, "chain": True},
        # a full batch with the usual small trees
        {"name": "verify_m64_tree16", "op": "verify", **BIG, "m": 64, "nodes": 16, "chain": False},
        # odd sizes, fp32, a smaller layer with conv bias and activation
        {"name": "verify_f32_m7_tree37", "op": "verify", **_layer(2, 6, 64, F32, 3, True, True), "m": 7, "nodes": 37,
         "chain": False},
        # a full batch with the largest trees, bf16 outputs
        {"name": "verify_m64_tree64_bf16", "op": "verify", **dict(BIG, out=BF16), "m": 64, "nodes": 64,
         "chain": False},
        # the step after verify_m64_tree16
        {"name": "accept_m64_tree16", "op": "accept", **BIG, "m": 64, "nodes": 16, "chain": False},
        # few streams of a small fp32 layer, long accepted chains
        {"name": "accept_f32_m5_chain33", "op": "accept", **_layer(2, 2, 32, F32), "m": 5, "nodes": 33, "chain": True},
        # a batch of finished prefixes written to the snapshot store
        {"name": "pack_int8_64", "op": "pack", **BIG, "n": 64, "format": "int8"},
        # a few slots of a small fp32 layer
        {"name": "pack_e4m3_f32_3", "op": "pack", **_layer(2, 6, 64, F32, 3), "n": 3, "format": "e4m3"},
        # 64 streams started from stored prefixes, several of them from the same one
        {"name": "unpack_int8_64", "op": "unpack", **BIG, "n": 64, "format": "int8"},
        # one stream restored
        {"name": "unpack_e4m3_1", "op": "unpack", **BIG, "n": 1, "format": "e4m3"},
        # the output norm of a decode step of 64 slots: fp32 o, bf16 gate and result
        {"name": "norm_decode_64", "op": "norm", "rows": 64, "groups": 32, "size": 128, "x": F32, "gate": BF16, "y": BF16,
         "param": BF16, "centered": False, "gate_first": False, "bias": False, "shared": True},
        # the output norm of the ragged prefill of 15717 tokens
        {"name": "norm_prefill_15717", "op": "norm", "rows": 15717, "groups": 32, "size": 128, "x": F32, "gate": BF16,
         "y": BF16, "param": BF16, "centered": False, "gate_first": False, "bias": False, "shared": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["verify", "verify", "accept", "pack", "unpack", "norm"])
    if op == "norm":
        size, groups = _log(rng, 8, 2048), _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, min(20000, (15717 * 4096) // (size * groups))))
        gate = rng.choice([F32, BF16, BF16, "none"])
        return {"op": op, "rows": rows, "groups": groups, "size": size, "x": rng.choice([F32, BF16]), "gate": gate,
                "y": rng.choice([F32, BF16]), "param": rng.choice([F32, BF16]), "centered": rng.random() < 0.4,
                "gate_first": gate != "none" and rng.random() < 0.3, "bias": rng.random() < 0.4,
                "shared": rng.random() < 0.5}
    hk = _log(rng, 1, 16)
    d, dtype = rng.choice([32, 64, 128, 128]), rng.choice([BF16, BF16, F32])
    c = _layer(hk, hk * rng.choice([1, 2, 2, 3, 4]), d, dtype, rng.choice([2, 3, 4, 4]), rng.random() < 0.5,
               rng.random() < 0.3, rng.choice([F32, BF16]))
    if op in ("pack", "unpack"):
        n = _log(rng, 1, max(1, min(200, 64 * 32 * 128 * 128 // (c["hv"] * d * d))))
        return {"op": op, **c, "n": n, "format": rng.choice(["int8", "int8", "e4m3"])}
    nodes = _log(rng, 1, 64)
    m = _log(rng, 1, max(1, min(128, 64 * 64 * 32 * 128 * 128 // (max(nodes, 32) * c["hv"] * d * d))))
    return {"op": op, **c, "m": m, "nodes": nodes, "chain": rng.random() < 0.3}


# ----------------------------------------------------------------------------- inputs


def _pointers(t, idx):
    """Addresses of t[idx[i]]."""
    return t.data_ptr() + idx.to(torch.int64) * (t[0].numel() * t.element_size())


def _sizes(c):
    """Bytes of a snapshot's codes, scales and conv state, in this order in a block."""
    hv, d = c["hv"], c["d"]
    return hv * d * d, hv * d * 4, (c["width"] - 1) * (2 * c["hk"] + hv) * d * (2 if c["dtype"] == BF16 else 4)


def _lengths(c):
    """Trees of between nodes / 2 and nodes nodes, the first slot's the largest."""
    return [c["nodes"] - i * 5 % (c["nodes"] // 2 + 1) for i in range(c["m"])]


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev, dtype=torch.float32) * std).to(dtype)

    def uniform(*shape, dtype=torch.float32):
        return (torch.rand(shape, generator=gen, device=dev, dtype=torch.float32) - 0.5).to(dtype)

    if c["op"] == "norm":
        width = c["groups"] * c["size"]
        per = c["size"] if c["shared"] else width
        c["x_t"] = normal(c["rows"], width, dtype=TORCH[c["x"]]) * 0.3
        c["gate_t"] = None if c["gate"] == "none" else normal(c["rows"], width, dtype=TORCH[c["gate"]])
        c["w_t"] = (1.0 + 0.1 * normal(per)).to(TORCH[c["param"]])
        c["b_t"] = normal(per, std=0.1, dtype=TORCH[c["param"]]) if c["bias"] else None
        c["y_t"] = torch.empty(c["rows"], width, dtype=TORCH[c["y"]], device=dev)
        return c

    hk, hv, d, width = c["hk"], c["hv"], c["d"], c["width"]
    ch, dt = (2 * hk + hv) * d, TORCH[c["dtype"]]
    slots = c.get("m") or c["n"]
    pool = slots + 3
    c["state"] = normal(pool, hv, d, d, std=0.05)
    c["conv_state"] = normal(pool, width - 1, ch, dtype=dt)
    c["slot"] = torch.randperm(pool, generator=gen, device=dev)[:slots]
    c["state_ptrs"] = _pointers(c["state"], c["slot"])
    c["conv_ptrs"] = _pointers(c["conv_state"], c["slot"])
    if c["op"] in ("pack", "unpack"):
        codes, scales, conv = _sizes(c)
        # a snapshot store; when read back, every fourth slot starts from the first block
        c["blocks"] = torch.zeros(slots, codes + scales + conv, dtype=torch.uint8, device=dev)
        c["block"] = torch.arange(slots, device=dev)
        if c["op"] == "unpack":
            c["block"][::4] = 0
            if c["format"] == "int8":
                raw = torch.randint(-127, 128, (slots, codes), generator=gen, device=dev).to(torch.int8).view(torch.uint8)
            else:
                raw = (torch.rand((slots, codes), generator=gen, device=dev) * 896 - 448).to(torch.float8_e4m3fn).view(torch.uint8)
            c["blocks"][:, :codes] = raw
            c["blocks"][:, codes:codes + scales] = (torch.rand((slots, scales // 4), generator=gen, device=dev) * 1e-3).view(torch.uint8)
            c["blocks"][:, codes + scales:] = normal(slots, (width - 1) * ch, dtype=dt).view(torch.uint8)
        c["block_ptrs"] = _pointers(c["blocks"], c["block"])
        return c

    lens = torch.tensor(_lengths(c), device=dev)
    c["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), lens.cumsum(0)]).to(torch.int32)
    total = c["total"] = int(c["cu"][-1])
    seq = torch.searchsorted(c["cu"][1:].contiguous(), torch.arange(total, device=dev, dtype=torch.int32), right=True)
    local = torch.arange(total, device=dev) - c["cu"][seq]
    if c["chain"]:
        parents = local - 1
    else:  # any earlier node, or the slot itself (about one in local + 1)
        parents = (torch.rand(total, generator=gen, device=dev) * (local + 1)).floor().long() - 1
        parents = torch.minimum(parents, local - 1)
    c["parents"] = parents.to(torch.int32)
    # the conv inputs lie in rows of a wider projection output
    c["x_t"] = normal(total, ch + 64, dtype=dt)[:, :ch]
    if c["op"] == "verify":
        c["conv_w"] = uniform(ch, width, dtype=dt)
        c["conv_b"] = uniform(ch, dtype=dt) if c["bias"] else None
        c["g"] = -torch.nn.functional.softplus(normal(total, hv))
        c["beta"] = torch.sigmoid(normal(total, hv))
        c["o_t"] = torch.empty(total, hv, d, dtype=TORCH[c["out"]], device=dev)
        c["record"] = (torch.empty(total, hk, d, device=dev), torch.empty(total, hv, d, device=dev),
                       torch.empty(total, hv, device=dev))
        return c
    k = normal(total, hk, d)
    # gamma falls along every path: a node at path depth n has the sum of n decays; any falling
    # sequence over the node numbers is one, since parents come before their children
    fall = torch.nn.functional.softplus(normal(total, hv)).cumsum(0)
    start = torch.cat([torch.zeros(1, hv, device=dev), fall])[c["cu"][:-1].long()]
    c["record"] = (k / k.norm(dim=-1, keepdim=True), normal(total, hv, d, std=0.3), -0.2 * (fall - start[seq]))
    # the last accepted node: any of the tree, or none
    u = torch.rand(slots, generator=gen, device=dev)
    c["accepted"] = ((u * (lens + 1)).floor().long() - 1).clamp(max=c["nodes"] - 1).to(torch.int32)
    return c


# ------------------------------------------------------------------------- plain forms


def _padded(c):
    """Row numbers [m, N] of the packed nodes, which of them exist, and the parents."""
    cu = c["cu"].long()
    rows = cu[:-1, None] + torch.arange(c["nodes"], device=cu.device)
    exists = rows < cu[1:, None]
    rows = rows.clamp(max=c["total"] - 1)
    parents = torch.where(exists, c["parents"].long()[rows], -1)
    return rows, exists, parents


def _paths(parents):
    """[m, N, N] 1.0 where node j lies on the root path of node i (i itself among it): the
    powers of I + (one-hot parents), doubled until they hold 64 levels."""
    n = parents.shape[1]
    r = torch.eye(n, device=parents.device) + (parents[:, :, None] == torch.arange(n, device=parents.device)).float()
    r = (r @ r).clamp(max=1.0)
    r = (r @ r).clamp(max=1.0)
    r = (r @ r).clamp(max=1.0)
    r = (r @ r).clamp(max=1.0)
    r = (r @ r).clamp(max=1.0)
    return (r @ r).clamp(max=1.0)


def _window(c, parents):
    """For node i the rows of [conv state, nodes] that precede it, newest first: [m, K-1, N]."""
    k1 = c["width"] - 1
    m = parents.shape[0]
    state = torch.arange(-1, k1 - 1, device=parents.device).expand(m, k1)
    up = torch.cat([state, torch.where(parents >= 0, parents + k1, k1 - 1)], 1)
    one = up[:, k1:]
    two = up.gather(1, one.clamp(min=0))
    three = up.gather(1, two.clamp(min=0))
    return torch.stack([one, two, three][:k1], 1)


def _verify(c):
    hk, hv, d, width = c["hk"], c["hv"], c["d"], c["width"]
    rows, exists, parents = _padded(c)
    m, n = rows.shape
    x = c["x_t"][rows].float()
    z = torch.cat([c["conv_state"][c["slot"]].float(), x], 1)
    w = c["conv_w"].float()
    back = _window(c, parents)
    take = torch.arange(m, device=x.device)[:, None, None]
    y = x * w[:, width - 1]
    y = y + (z[take, back] * w.t()[:width - 1].flip(0)[None, :, None, :]).sum(1)
    if c["conv_b"] is not None:
        y = y + c["conv_b"].float()
    if c["silu"]:
        y = y * torch.sigmoid(y)
    q = y[..., :hk * d].reshape(m, n, hk, d)
    k = y[..., hk * d:2 * hk * d].reshape(m, n, hk, d)
    v = y[..., 2 * hk * d:].reshape(m, n, hv, d).transpose(1, 2)
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    kh = k.transpose(1, 2).repeat_interleave(hv // hk, 1)  # [m, hv, n, d]
    qh = q.transpose(1, 2).repeat_interleave(hv // hk, 1)
    path = _paths(parents)
    gamma = path @ c["g"][rows]  # [m, n, hv]
    gh = gamma.transpose(1, 2)
    beta = c["beta"][rows].transpose(1, 2)[..., None]
    decay = torch.exp(torch.where(path[:, None] > 0, gh[..., :, None] - gh[..., None, :], -math.inf))
    strict = 1.0 - torch.eye(n, device=x.device)
    s = c["state"][c["slot"]].transpose(-1, -2)
    u = beta * (v - torch.exp(gh)[..., None] * (kh @ s))
    # (I + A)^-1 = (I - A)(I + A^2)(I + A^4) .. with A^64 = 0
    a = -beta * strict * decay * (kh @ kh.transpose(-1, -2))
    u = u + a @ u
    a = a @ a
    u = u + a @ u
    a = a @ a
    u = u + a @ u
    a = a @ a
    u = u + a @ u
    a = a @ a
    u = u + a @ u
    a = a @ a
    u = u + a @ u
    o = torch.exp(gh)[..., None] * (qh @ s) + (decay * (qh @ kh.transpose(-1, -2))) @ u
    seq = torch.searchsorted(c["cu"][1:].contiguous(), torch.arange(c["total"], device=x.device, dtype=torch.int32), right=True)
    local = torch.arange(c["total"], device=x.device) - c["cu"].long()[seq]
    return {"o": o[seq, :, local].to(TORCH[c["out"]]), "k": k[seq, local], "u": u[seq, :, local], "gamma": gamma[seq, local]}


def _accept(c):
    hk, hv, width = c["hk"], c["hv"], c["width"]
    rows, exists, parents = _padded(c)
    last = c["accepted"].long()
    m = rows.shape[0]
    take = torch.arange(m, device=rows.device)
    kept = _paths(parents)[take, last.clamp(min=0)] * (last >= 0)[:, None]  # [m, n]
    k, u, gamma = c["record"]
    gr = gamma[rows].transpose(1, 2)  # [m, hv, n]
    end = torch.where(last[:, None] >= 0, gr[take, :, last.clamp(min=0)], 0.0)
    f = torch.exp(torch.where(kept[:, None] > 0, end[..., None] - gr, -math.inf))
    kh = k[rows].transpose(1, 2).repeat_interleave(hv // hk, 1)
    uh = u[rows].transpose(1, 2) * f[..., None]
    s = c["state"][c["slot"]] * torch.exp(end)[..., None, None] + uh.transpose(-1, -2).contiguous() @ kh
    z = torch.cat([c["conv_state"][c["slot"]], c["x_t"][rows]], 1)
    k1 = width - 1
    back = _window(c, parents)[take, :, last.clamp(min=0)]  # rows before the node, newest first
    new = torch.cat([(last + k1)[:, None], back[:, :k1 - 1]], 1).flip(1)
    new = torch.where((last >= 0)[:, None], new, torch.arange(k1, device=rows.device))
    c["state"][c["slot"]] = s
    c["conv_state"][c["slot"]] = z[take[:, None], new]
    return {"state": c["state"], "conv_state": c["conv_state"]}


def _block_views(c):
    codes, scales, _ = _sizes(c)
    b, hv, d = c["blocks"], c["hv"], c["d"]
    kind = torch.int8 if c["format"] == "int8" else torch.float8_e4m3fn
    return {"codes": b[:, :codes].view(kind).view(-1, hv, d, d), "scales": b[:, codes:codes + scales].view(torch.float32).view(-1, hv, d),
            "conv_state": b[:, codes + scales:].view(TORCH[c["dtype"]]).view(len(b), c["width"] - 1, -1)}


def _pack(c):
    out = _block_views(c)
    s = c["state"][c["slot"]]
    top = s.abs().amax(-1, keepdim=True)
    live = top >= TINY
    code = torch.where(live, s * (TOP[c["format"]] / torch.where(live, top, 1.0)), 0.0)
    out["codes"].copy_((code.round() if c["format"] == "int8" else code).to(out["codes"].dtype))
    out["scales"].copy_(torch.where(live, top / TOP[c["format"]], 0.0)[..., 0])
    out["conv_state"].copy_(c["conv_state"][c["slot"]])
    return out


def _unpack(c):
    b = _block_views(c)
    c["state"][c["slot"]] = b["codes"][c["block"]].float() * b["scales"][c["block"]][..., None]
    c["conv_state"][c["slot"]] = b["conv_state"][c["block"]]
    return {"state": c["state"], "conv_state": c["conv_state"]}


def _norm(c):
    rows, groups, size = c["rows"], c["groups"], c["size"]
    x = c["x_t"].float().view(rows, groups, size)
    gate = None
    if c["gate_t"] is not None:
        z = c["gate_t"].float().view(rows, groups, size)
        gate = z * torch.sigmoid(z)
    if gate is not None and c["gate_first"]:
        x = x * gate
    if c["centered"]:
        x = x - x.mean(-1, keepdim=True)
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    n = n * c["w_t"].float().view(-1, size)
    if c["b_t"] is not None:
        n = n + c["b_t"].float().view(-1, size)
    if gate is None:
        n = n * torch.sigmoid(n)
    elif not c["gate_first"]:
        n = n * gate
    return {"y": n.reshape(rows, groups * size).to(c["y_t"].dtype)}


# -------------------------------------------------------------------- the library's calls


def _own(c):
    import gated_delta_rule_conv_amd as gdn

    kinds = {BF16: gdn.GDN_BF16, F32: gdn.GDN_F32}
    if c["op"] == "norm":
        if "dims" not in c:
            c["dims"] = gdn.make_norm_dims(
                c["groups"], c["size"], in_dtype=kinds[c["x"]], gate_dtype=kinds.get(c["gate"], gdn.GDN_F32),
                param_dtype=kinds[c["param"]], out_dtype=kinds[c["y"]], activation=gdn.GDN_ACT_SILU, centered=c["centered"],
                gate_first=c["gate_first"], shared_params=c["shared"], eps=1e-5)
        gdn.group_norm(c["dims"], c["x_t"], c["w_t"], c["y_t"], gate=c["gate_t"], bias=c["b_t"])
        return {"y": c["y_t"]}
    if "dims" not in c:
        c["dims"] = gdn.make_dims(c["hk"], c["hv"], c["d"], conv_width=c["width"], in_dtype=kinds[c["dtype"]],
                                  activation=gdn.GDN_ACT_SILU if c["silu"] else gdn.GDN_ACT_NONE, out_dtype=kinds[c["out"]])
    if c["op"] == "verify":
        gdn.tree_verify(c["dims"], c["x_t"], c["conv_w"], c["conv_b"], c["g"], c["beta"], c["o_t"], c["parents"], c["cu"],
                        c["nodes"], c["state_ptrs"], c["conv_ptrs"], record=c["record"])
        return {"o": c["o_t"], "k": c["record"][0], "u": c["record"][1], "gamma": c["record"][2]}
    if c["op"] == "accept":
        gdn.tree_accept(c["dims"], c["x_t"], c["record"], c["parents"], c["cu"], c["nodes"], c["accepted"], c["state_ptrs"],
                        c["conv_ptrs"])
        return {"state": c["state"], "conv_state": c["conv_state"]}
    form = gdn.GDN_PACK_INT8 if c["format"] == "int8" else gdn.GDN_PACK_E4M3
    if c["op"] == "pack":
        gdn.slot_pack(c["dims"], form, c["state_ptrs"], c["conv_ptrs"], c["block_ptrs"])
        return _block_views(c)
    gdn.slot_unpack(c["dims"], form, c["block_ptrs"], c["state_ptrs"], c["conv_ptrs"])
    return {"state": c["state"], "conv_state": c["conv_state"]}


def run(state):
    if own:
        return _own(state)
    return {"verify": _verify, "accept": _accept, "pack": _pack, "unpack": _unpack, "norm": _norm}[state["op"]](state)


# -------------------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["groups"] * c["size"]
        size = {BF16: 2, F32: 4, "none": 0}
        return {"bytes": n * (size[c["x"]] + size[c["gate"]] + size[c["y"]]), "flops": 10 * n}
    hk, hv, d = c["hk"], c["hv"], c["d"]
    esz, osz = (2 if c["dtype"] == BF16 else 4), (2 if c["out"] == BF16 else 4)
    ch = (2 * hk + hv) * d
    state, conv = 4 * hv * d * d, (c["width"] - 1) * ch * esz
    if c["op"] in ("pack", "unpack"):
        packed = hv * d * d + 4 * hv * d
        # unpack: three slots in four read a block of their own
        blocks = c["n"] if c["op"] == "pack" else c["n"] - (c["n"] + 3) // 4 + 1
        return {"bytes": c["n"] * (state + conv) + blocks * (packed + conv), "flops": 3 * c["n"] * hv * d * d}
    m, lens = c["m"], _lengths(c)
    if c["op"] == "verify":
        total, pairs = sum(lens), sum(n * n for n in lens)
        moved = m * (state + conv) + total * (ch * esz + 8 * hv + 4 + hv * d * osz + 4 * (hk * d + hv * d + hv))
        # S k and S q; k k^T and q k^T of the pairs of nodes; the two products of the pairs with u
        flops = 4 * total * hv * d * d + pairs * (2 * hk * d + 2 * hv * d) + 2 * total * ch * c["width"]
        return {"bytes": moved, "flops": flops}
    # the path of a random node: half the nodes of a chain, about their logarithm in these trees
    path = sum(n / 2 if c["chain"] else math.log(n + 1) for n in lens)
    return {"bytes": m * 2 * (state + conv) + path * 4 * (hk * d + hv * d + hv), "flops": 2 * path * hv * d * d}


# ------------------------------------------------------------------------------- exact


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _exact_verify(c):
    """Every node's own state from its parent's, node by node, slot by slot, in 64 bits."""
    hk, hv, d, width, dev = c["hk"], c["hv"], c["d"], c["width"], c["x_t"].device
    cu, par = c["cu"].tolist(), c["parents"].tolist()
    o = torch.zeros(c["total"], hv, d, dtype=torch.float64, device=dev)
    ks, us, gs = torch.zeros(c["total"], hk, d, dtype=torch.float64, device=dev), o.clone(), o[..., 0].clone()
    w = c["conv_w"].double()
    for i, slot in enumerate(c["slot"].tolist()):
        states, sums = [], []
        hist = list(c["conv_state"][slot].double().unbind(0))
        hists = []
        for n in range(cu[i + 1] - cu[i]):
            t = cu[i] + n
            p = par[t]
            before, rows, gsum = (c["state"][slot].double(), hist, 0.0) if p < 0 else (states[p], hists[p], sums[p])
            z = rows[-(width - 1):] + [c["x_t"][t].double()]
            y = (torch.stack(z, 1) * w).sum(1)
            if c["conv_b"] is not None:
                y = y + c["conv_b"].double()
            if c["silu"]:
                y = y / (1 + torch.exp(-y))
            q, k, v = y[:hk * d].view(hk, d), y[hk * d:2 * hk * d].view(hk, d), y[2 * hk * d:].view(hv, d)
            q = q / (q.pow(2).sum(1, keepdim=True) + 1e-6).sqrt()
            k = k / (k.pow(2).sum(1, keepdim=True) + 1e-6).sqrt()
            q2, k2 = q.repeat_interleave(hv // hk, 0), k.repeat_interleave(hv // hk, 0)
            s = before * c["g"][t].double().exp()[:, None, None]
            u = c["beta"][t].double()[:, None] * (v - (s * k2[:, None, :]).sum(-1))
            s = s + u[:, :, None] * k2[:, None, :]
            states.append(s)
            hists.append(z[1:])
            sums.append(gsum + c["g"][t].double())
            o[t], ks[t], us[t], gs[t] = (s * q2[:, None, :]).sum(-1), k, u, sums[-1]
    return {"o": _np(o), "k": _np(ks), "u": _np(us), "gamma": _np(gs)}


def _exact_accept(c):
    state, conv = c["state"].double(), c["conv_state"].double()
    k, u, gamma = (t.double() for t in c["record"])
    cu, par, last = c["cu"].tolist(), c["parents"].tolist(), c["accepted"].tolist()
    rep = c["hv"] // c["hk"]
    for i, slot in enumerate(c["slot"].tolist()):
        path, n = [], last[i]
        while n >= 0:
            path.insert(0, cu[i] + n)
            n = par[cu[i] + n]
        s, g = state[slot].clone(), torch.zeros(c["hv"], dtype=torch.float64, device=state.device)
        rows = list(conv[slot].clone().unbind(0))
        for t in path:
            s = s * (gamma[t] - g).exp()[:, None, None] + u[t][:, :, None] * k[t].repeat_interleave(rep, 0)[:, None, :]
            g = gamma[t]
            rows.append(c["x_t"][t].double())
        state[slot] = s
        conv[slot] = torch.stack(rows[-(c["width"] - 1):])
    return {"state": _np(state), "conv_state": _np(conv)}


def _exact_pack(c):
    s = c["state"].double()[c["slot"]]
    return {"codes": None, "scales": _np(s.abs().amax(-1) / TOP[c["format"]]), "conv_state": _np(c["conv_state"][c["slot"]])}


def _exact_unpack(c):
    codes, scales, _ = _sizes(c)
    raw = c["blocks"].cpu().numpy()[c["block"].cpu().numpy()]
    hv, d = c["hv"], c["d"]
    byte = raw[:, :codes].astype(np.int64)
    if c["format"] == "int8":
        value = np.where(byte > 127, byte - 256, byte).astype(np.float64)
    else:  # 1 sign, 4 exponent (bias 7), 3 mantissa bits
        e, f = (byte >> 3) & 15, byte & 7
        value = np.where(byte > 127, -1.0, 1.0) * np.where(e > 0, (1 + f / 8.0) * 2.0 ** (e - 7), f / 8.0 * 2.0 ** -6)
    scale = np.ascontiguousarray(raw[:, codes:codes + scales]).view(np.float32).astype(np.float64)
    state = _np(c["state"])
    state[c["slot"].cpu().numpy()] = value.reshape(-1, hv, d, d) * scale.reshape(-1, hv, d, 1)
    tail = np.ascontiguousarray(raw[:, codes + scales:])
    rows = tail.view(np.float32) if c["dtype"] == F32 else (tail.view(np.uint16).astype(np.uint32) << 16).view(np.float32)
    conv = _np(c["conv_state"])
    conv[c["slot"].cpu().numpy()] = rows.astype(np.float64).reshape(len(raw), c["width"] - 1, -1)
    return {"state": state, "conv_state": conv}


def _exact_norm(c):
    shape = (c["rows"], c["groups"], c["size"])
    x = c["x_t"].double().view(shape)
    act = lambda t: t / (1 + torch.exp(-t))  # noqa: E731
    z = None if c["gate_t"] is None else act(c["gate_t"].double().view(shape))
    if z is not None and c["gate_first"]:
        x = x * z
    mean = x.mean(-1, keepdim=True) if c["centered"] else torch.zeros_like(x[..., :1])
    y = (x - mean) * torch.rsqrt((x - mean).pow(2).mean(-1, keepdim=True) + 1e-5) * c["w_t"].double().view(-1, c["size"])
    if c["b_t"] is not None:
        y = y + c["b_t"].double().view(-1, c["size"])
    y = act(y) if z is None else y if c["gate_first"] else y * z
    return {"y": _np(y.reshape(c["rows"], -1))}


def exact(case, seed):
    c = prepare(case, seed)
    return {"verify": _exact_verify, "accept": _exact_accept, "pack": _exact_pack, "unpack": _exact_unpack,
            "norm": _exact_norm}[c["op"]](c)
