"""Tensor-level helpers over the C ABI (argument marshalling only).

``SlotPool`` is the caller-owned slot pool: one device allocation of equal-sized
fp32 recurrent-state blocks and one of conv-state blocks, addressed per call through
device arrays of 64-bit block addresses that gdn_slot_pointers builds on the device.
(The "qLLM" page, section "What this is", keeps the linear-attention layers' recurrent
and conv state in such a pool of slots; aprender #5279, "Phase plan", phase P5, puts
the slot index on the launch grid and hands the kernels one address per slot.)

``conv_update``, ``prefill``, ``decode``, ``decode_fused``, ``tree_verify``, ``tree_accept``,
``slot_pack``, ``slot_unpack``, ``group_norm``, ``linear_prefill``, ``linear_decode``, ``block_norm``, ``sample`` and
``tree_follow`` derive pointers, strides and views from torch tensors and call the library; all arithmetic happens in
the HIP kernels. From ``tree_verify`` on they check the type, size, layout and device of every operand first
(ValueError): the kernels see addresses alone.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import GDN_BF16, GDN_F32, gdn_dims


def channels(dims: gdn_dims) -> int:
    return dims.head_dim * (2 * dims.num_k_heads + dims.num_v_heads)


def torch_in_dtype(dims: gdn_dims) -> torch.dtype:
    return torch.bfloat16 if dims.in_dtype == GDN_BF16 else torch.float32


class SlotPool:
    """pool_slots fixed-size slots: state [Hv, d, d] fp32 and conv state [K-1, C] in_dtype."""

    def __init__(self, dims: gdn_dims, pool_slots: int, device="cuda", state=None, conv_state=None):
        self.dims = dims
        self.pool_slots = pool_slots
        d, Hv, K, C = dims.head_dim, dims.num_v_heads, dims.conv_width, channels(dims)
        self.state = state if state is not None else torch.zeros(
            (pool_slots, Hv, d, d), dtype=torch.float32, device=device)
        self.conv_state = conv_state if conv_state is not None else torch.zeros(
            (pool_slots, K - 1, C), dtype=torch_in_dtype(dims), device=device)
        assert self.state.is_contiguous() and self.conv_state.is_contiguous()
        assert tuple(self.state.shape) == (pool_slots, Hv, d, d)
        assert tuple(self.conv_state.shape) == (pool_slots, K - 1, C)

    @property
    def state_slot_bytes(self) -> int:
        return self.state[0].numel() * 4

    @property
    def conv_slot_bytes(self) -> int:
        return self.conv_state[0].numel() * self.conv_state.element_size()

    def pointers(self, slot_idx: torch.Tensor):
        """Device u64 pointer arrays (state, conv state) for int32 slot indices on the
        device; indices outside the pool give 0 (inactive slot)."""
        assert slot_idx.dtype == torch.int32 and slot_idx.is_cuda
        m = slot_idx.numel()
        sp = torch.empty(m, dtype=torch.int64, device=slot_idx.device)
        cp = torch.empty(m, dtype=torch.int64, device=slot_idx.device)
        _lib.gdn_slot_pointers(self.state.data_ptr(), self.state_slot_bytes, self.pool_slots, slot_idx, m, sp)
        _lib.gdn_slot_pointers(self.conv_state.data_ptr(), self.conv_slot_bytes, self.pool_slots, slot_idx, m, cp)
        return sp, cp


    def copy_slots(self, src_idx: torch.Tensor, dst_idx: torch.Tensor, state: bool = True,
                   conv_state: bool = True, stream=None) -> None:
        """Snapshot / fork: slot dst_idx[i] takes the state and conv state of slot src_idx[i]
        (int32 device index tensors of equal length; destinations distinct from each other
        and from every source)."""
        assert src_idx.numel() == dst_idx.numel()
        n = src_idx.numel()
        ss, sc = self.pointers(src_idx)
        ds, dc = self.pointers(dst_idx)
        _lib.gdn_slot_copy(self.dims, ss if state else None, ds if state else None, sc if conv_state else None,
                           dc if conv_state else None, n, stream)


    def pack_slots(self, slot_idx: torch.Tensor, packed: torch.Tensor, fmt: int, conv_state: bool = True) -> None:
        """8-bit snapshots: slot slot_idx[i] into row i of packed (from packed_slots())."""
        if slot_idx.numel() > packed.shape[0]:
            raise ValueError(f"pack_slots: {slot_idx.numel()} slots for {packed.shape[0]} rows of packed")
        blocks = self._blocks(packed, slot_idx)
        sp, cp = self.pointers(slot_idx)
        slot_pack(self.dims, fmt, sp, cp if conv_state else None, blocks)

    def unpack_slots(self, packed: torch.Tensor, block_idx: torch.Tensor, slot_idx: torch.Tensor, fmt: int,
                     conv_state: bool = True) -> None:
        """Slot slot_idx[i] filled from row block_idx[i] of packed (int32 device index tensors, slots
        distinct; one block may fill several slots). An index outside its pool skips the entry."""
        blocks = self._blocks(packed, slot_idx, block_idx)
        sp, cp = self.pointers(slot_idx)
        slot_unpack(self.dims, fmt, blocks, sp, cp if conv_state else None)

    def _blocks(self, packed: torch.Tensor, slot_idx: torch.Tensor, block_idx=None) -> torch.Tensor:
        """Device addresses of packed's rows block_idx (default: 0, 1, ..), 0 outside it."""
        n, at, size = slot_idx.numel(), self.state.get_device(), \
            _lib.gdn_slot_packed_size(self.dims, _lib.GDN_PACK_INT8)  # (both formats')
        _at("packed slots", "packed", packed, torch.uint8, packed.shape[0] * size, at)
        if packed.dim() != 2:
            raise ValueError(f"packed slots: packed must be rows of {size} bytes (got shape {tuple(packed.shape)})")
        if block_idx is None:
            block_idx = torch.arange(n, dtype=torch.int32, device=slot_idx.device)
        _at("packed slots", "the slots' indices", slot_idx, _I32, n, at)
        _at("packed slots", "the blocks' indices", block_idx, _I32, n, at)
        out = torch.empty(n, dtype=torch.int64, device=slot_idx.device)
        _lib.gdn_slot_pointers(packed.data_ptr(), packed.shape[1], packed.shape[0], block_idx, n, out)
        return out


def packed_slots(dims: gdn_dims, n: int, fmt: int, device="cuda") -> torch.Tensor:
    """Room for n 8-bit snapshots: uint8 [n, gdn_slot_packed_size]."""
    return torch.zeros((n, _lib.gdn_slot_packed_size(dims, fmt)), dtype=torch.uint8, device=device)


def qkv_views(dims: gdn_dims, y: torch.Tensor):
    """q, k, v views of the conv output y [T, C] (channels [q | k | v])."""
    hk = dims.num_k_heads * dims.head_dim
    return y[:, :hk], y[:, hk:2 * hk], y[:, 2 * hk:]


def conv_update(dims: gdn_dims, x: torch.Tensor, y: torch.Tensor, conv_w: torch.Tensor, conv_b,
                conv_state_ptrs: torch.Tensor, cu_seqlens=None, stream=None) -> None:
    n = conv_state_ptrs.numel()
    _lib.gdn_conv_update(dims, x, x.stride(0), y, y.stride(0), conv_w, conv_b, cu_seqlens, conv_state_ptrs, n,
                         x.shape[0], stream)


def prefill(dims: gdn_dims, y: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, o: torch.Tensor,
            cu_seqlens: torch.Tensor, state_ptrs: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    q, k, v = qkv_views(dims, y)
    _lib.gdn_prefill_chunked(dims, q, q.stride(0), k, k.stride(0), v, v.stride(0), g, beta, o, cu_seqlens,
                             state_ptrs.numel(), y.shape[0], state_ptrs, workspace,
                             workspace.numel() * workspace.element_size(), stream)


def prefill_fused(dims: gdn_dims, x: torch.Tensor, conv_w: torch.Tensor, conv_b, g: torch.Tensor, beta: torch.Tensor,
                  o: torch.Tensor, cu_seqlens: torch.Tensor, state_ptrs: torch.Tensor, conv_state_ptrs: torch.Tensor,
                  workspace: torch.Tensor, stream=None) -> None:
    """conv_update (prefill mode) + prefill in one call; workspace from prefill_fused_workspace()."""
    _lib.gdn_prefill_fused(dims, x, x.stride(0), conv_w, conv_b, g, beta, o, cu_seqlens, state_ptrs.numel(),
                           x.shape[0], state_ptrs, conv_state_ptrs, workspace,
                           workspace.numel() * workspace.element_size(), stream)


def prefill_fused_static(dims: gdn_dims, x: torch.Tensor, conv_w: torch.Tensor, conv_b, g: torch.Tensor,
                         beta: torch.Tensor, o: torch.Tensor, cu_seqlens: torch.Tensor, state_ptrs: torch.Tensor,
                         conv_state_ptrs: torch.Tensor, stream=None) -> None:
    """prefill_fused with the library's own 64 MiB device workspace: nothing allocated."""
    _lib.gdn_prefill_fused_static(dims, x, x.stride(0), conv_w, conv_b, g, beta, o, cu_seqlens, state_ptrs.numel(),
                                  x.shape[0], state_ptrs, conv_state_ptrs, stream)


def decode(dims: gdn_dims, y: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, o: torch.Tensor,
           state_ptrs: torch.Tensor, stream=None) -> None:
    q, k, v = qkv_views(dims, y)
    _lib.gdn_decode_batched(dims, q, q.stride(0), k, k.stride(0), v, v.stride(0), g, beta, o, state_ptrs,
                            state_ptrs.numel(), stream)


def decode_fused(dims: gdn_dims, x: torch.Tensor, conv_w: torch.Tensor, conv_b, g: torch.Tensor, beta: torch.Tensor,
                 o: torch.Tensor, state_ptrs: torch.Tensor, conv_state_ptrs: torch.Tensor,
                 conv_state_out_ptrs=None, stream=None) -> None:
    """conv_update (decode mode) + decode in one launch. The new conv states go to
    conv_state_out_ptrs (other buffers, the faster form) or, when None, in place."""
    _lib.gdn_decode_fused(dims, x, x.stride(0), conv_w, conv_b, g, beta, o, state_ptrs, conv_state_ptrs,
                          conv_state_out_ptrs, state_ptrs.numel(), stream)


def tree_record(dims: gdn_dims, total_nodes: int, device="cuda"):
    """What tree_verify leaves for tree_accept: fp32 (k [T, Hk, d], u [T, Hv, d], gamma [T, Hv])."""
    Hk, Hv, d = dims.num_k_heads, dims.num_v_heads, dims.head_dim
    return (torch.empty((total_nodes, Hk, d), dtype=torch.float32, device=device),
            torch.empty((total_nodes, Hv, d), dtype=torch.float32, device=device),
            torch.empty((total_nodes, Hv), dtype=torch.float32, device=device))


_F32, _I32, _I64 = torch.float32, torch.int32, torch.int64
_DTYPES = {GDN_F32: torch.float32, GDN_BF16: torch.bfloat16}
_KINDS = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}


def _at(fn: str, name: str, t: torch.Tensor, dtype, n: int, device: int) -> int:
    """The address of t, which must be n contiguous values of dtype (addresses: of int64 or uint64) on the device:
    the kernels see no more of it."""
    if (t.dtype is dtype or (dtype is _I64 and t.dtype is torch.uint64)) and t.numel() == n and t.is_contiguous() \
            and t.get_device() == device:
        return t.data_ptr()
    raise ValueError(f"{fn}: {name} must be {n} contiguous values of {dtype} on the device of the first operand (got "
                     f"{t.numel()} of {t.dtype}, shape {tuple(t.shape)}, strides {t.stride()}, device {t.device})")


def _check_rows(fn: str, dims, x: torch.Tensor, wide: int):
    dtype = _DTYPES.get(dims.in_dtype)
    if x.dtype is not dtype or x.dim() != 2 or x.shape[1] != wide or x.stride(1) != 1:
        raise ValueError(f"{fn}: x must be rows of {wide} adjacent values of {dtype} (got {x.dtype}, shape "
                         f"{tuple(x.shape)}, strides {x.stride()})")
    return dtype


def _record_at(fn: str, record, rows: int, Hk: int, Hv: int, d: int, device: int):
    k, u, gamma = record
    return (_at(fn, "k of the record", k, _F32, rows * Hk * d, device), _at(fn, "u of the record", u, _F32, rows * Hv * d, device),
            _at(fn, "gamma of the record", gamma, _F32, rows * Hv, device))


def tree_verify(dims: gdn_dims, x: torch.Tensor, conv_w: torch.Tensor, conv_b, g: torch.Tensor, beta: torch.Tensor,
                o: torch.Tensor, parents, cu_nodes: torch.Tensor, max_nodes: int, state_ptrs: torch.Tensor,
                conv_state_ptrs: torch.Tensor, record=None, stream=None) -> None:
    """The drafted trees of m slots answered against their states, which stay as they are;
    parents None: chains. record (from tree_record()) is needed to accept nodes afterwards."""
    fn, Hk, Hv, d = "tree_verify", dims.num_k_heads, dims.num_v_heads, dims.head_dim
    rows, m, at = x.shape[0], state_ptrs.numel(), x.get_device()
    wide, gates = (2 * Hk + Hv) * d, rows * Hv
    dtype = _check_rows(fn, dims, x, wide)
    k, u, gamma = _record_at(fn, record, rows, Hk, Hv, d, at) if record is not None else (None, None, None)
    _lib._launch(
        "gdn_tree_verify", _lib._LIB.gdn_tree_verify, stream, x, ctypes.byref(dims), x.data_ptr(), x.stride(0), _at(fn, "conv_w", conv_w, dtype, wide * dims.conv_width, at),
        None if conv_b is None else _at(fn, "conv_b", conv_b, dtype, wide, at), _at(fn, "g", g, _F32, gates, at),
        _at(fn, "beta", beta, _F32, gates, at), _at(fn, "o", o, _DTYPES.get(dims.out_dtype), gates * d, at),
        None if parents is None else _at(fn, "parents", parents, _I32, rows, at),
        _at(fn, "cu_nodes", cu_nodes, _I32, m + 1, at), m, rows, max_nodes,
        _at(fn, "state_ptrs", state_ptrs, _I64, m, at), _at(fn, "conv_state_ptrs", conv_state_ptrs, _I64, m, at), k, u, gamma)


def tree_accept(dims: gdn_dims, x: torch.Tensor, record, parents, cu_nodes: torch.Tensor, max_nodes: int,
                accepted: torch.Tensor, state_ptrs: torch.Tensor, conv_state_ptrs: torch.Tensor, stream=None) -> None:
    """Slot i's state and conv state moved along the root path of node accepted[i] (-1: none)."""
    fn, Hk, Hv, d = "tree_accept", dims.num_k_heads, dims.num_v_heads, dims.head_dim
    rows, m, at = x.shape[0], state_ptrs.numel(), x.get_device()
    _check_rows(fn, dims, x, (2 * Hk + Hv) * d)
    k, u, gamma = _record_at(fn, record, rows, Hk, Hv, d, at)
    _lib._launch(
        "gdn_tree_accept", _lib._LIB.gdn_tree_accept, stream, x, ctypes.byref(dims), x.data_ptr(), x.stride(0), k, u, gamma, None if parents is None else _at(fn, "parents", parents, _I32, rows, at),
        _at(fn, "cu_nodes", cu_nodes, _I32, m + 1, at), _at(fn, "accepted", accepted, _I32, m, at), m, rows, max_nodes,
        _at(fn, "state_ptrs", state_ptrs, _I64, m, at), _at(fn, "conv_state_ptrs", conv_state_ptrs, _I64, m, at))


def _block_operands(fn: str, state_ptrs: torch.Tensor, conv_state_ptrs, packed_ptrs: torch.Tensor):
    n, at = state_ptrs.numel(), state_ptrs.get_device()
    return (_at(fn, "state_ptrs", state_ptrs, _I64, n, at),
            None if conv_state_ptrs is None else _at(fn, "conv_state_ptrs", conv_state_ptrs, _I64, n, at),
            _at(fn, "packed_ptrs", packed_ptrs, _I64, n, at), n)


def slot_pack(dims: gdn_dims, fmt: int, state_ptrs: torch.Tensor, conv_state_ptrs, packed_ptrs: torch.Tensor,
              stream=None) -> None:
    sp, cp, bp, n = _block_operands("slot_pack", state_ptrs, conv_state_ptrs, packed_ptrs)
    _lib._launch("gdn_slot_pack", _lib._LIB.gdn_slot_pack, stream, state_ptrs, ctypes.byref(dims), fmt, sp, cp, bp, n)


def slot_unpack(dims: gdn_dims, fmt: int, packed_ptrs: torch.Tensor, state_ptrs: torch.Tensor, conv_state_ptrs,
                stream=None) -> None:
    sp, cp, bp, n = _block_operands("slot_unpack", state_ptrs, conv_state_ptrs, packed_ptrs)
    _lib._launch("gdn_slot_unpack", _lib._LIB.gdn_slot_unpack, stream, state_ptrs, ctypes.byref(dims), fmt, bp, sp, cp, n)


def group_norm(dims, x: torch.Tensor, weight, y: torch.Tensor, gate=None, bias=None, stream=None) -> None:
    """y = the norm of every group of every row of x, times weight, plus bias, gated (dims from
    make_norm_dims(), the types of x, gate, weight, bias and y among them). Rows are the first axis; the other
    axes of x, gate and y are contiguous. weight and bias: [group_size], or with their own for every group
    [groups * group_size]."""
    rows, size, at = x.shape[0], dims.group_size, x.get_device()
    n = rows * dims.groups * size
    per, param = size if dims.shared_params else dims.groups * size, _DTYPES.get(dims.param_dtype)
    _lib._launch(
        "gdn_group_norm", _lib._LIB.gdn_group_norm, stream, x, ctypes.byref(dims), x.data_ptr(),
        _row_stride("x", x, _DTYPES.get(dims.in_dtype), rows, n, at), None if gate is None else gate.data_ptr(),
        0 if gate is None else _row_stride("gate", gate, _DTYPES.get(dims.gate_dtype), rows, n, at),
        None if weight is None else _at("group_norm", "weight", weight, param, per, at),
        None if bias is None else _at("group_norm", "bias", bias, param, per, at), y.data_ptr(),
        _row_stride("y", y, _DTYPES.get(dims.out_dtype), rows, n, at), rows)


def _row_stride(name: str, t: torch.Tensor, dtype, rows: int, n: int, device: int, fn: str = "group_norm") -> int:
    """Row stride of t, which holds n values in `rows` contiguous rows, [rows, width] or [rows, a, b] (an axis of
    length 1 has no stride to speak of)."""
    s, shape = t.stride(), t.shape
    if t.dtype is dtype and t.get_device() == device and t.numel() == n and shape[0] == rows and (
            len(s) == 2 and (s[1] == 1 or shape[1] == 1)
            or len(s) == 3 and (s[2] == 1 or shape[2] == 1) and (s[1] == shape[2] or shape[1] == 1) or n == 0):
        return s[0]
    raise ValueError(f"{fn}: {name} must be {rows} rows of {n // rows if rows else 0} adjacent values of {dtype}, [rows, "
                     f"width] or [rows, a, b], on the device of x (got {t.dtype}, shape {tuple(shape)}, strides {s}, "
                     f"device {t.device})")


def _linear_operands(fn: str, dims: gdn_dims, q, k, v, g, o, state_ptrs):
    """q, k, v and g with their strides, and o's and the pointers' addresses."""
    rows, at, dtype = q.shape[0], q.get_device(), _DTYPES.get(dims.in_dtype)
    wide, values = rows * dims.num_k_heads * dims.head_dim, rows * dims.num_v_heads * dims.head_dim
    if g.dim() == 1:
        gp, gs = _at(fn, "g", g, _F32, dims.num_v_heads, at), 0
    else:
        gp, gs = g.data_ptr(), _row_stride("g", g, _F32, rows, rows * dims.num_v_heads, at, fn)
        if gs < dims.num_v_heads and rows > 1:  # (a stride of 0 would be read as one row of decays for all tokens)
            raise ValueError(f"{fn}: the rows of g overlap (strides {g.stride()}); one row of decays for all tokens is given as "
                             f"[{dims.num_v_heads}]")
        gs = max(gs, dims.num_v_heads)
    return (q.data_ptr(), _row_stride("q", q, dtype, rows, wide, at, fn), k.data_ptr(), _row_stride("k", k, dtype, rows, wide, at, fn),
            v.data_ptr(), _row_stride("v", v, dtype, rows, values, at, fn), gp, gs,
            _at(fn, "o", o, _DTYPES.get(dims.out_dtype), values, at), _at(fn, "state_ptrs", state_ptrs, _I64, state_ptrs.numel(), at))


def linear_prefill(dims: gdn_dims, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, o: torch.Tensor,
                   cu_seqlens: torch.Tensor, state_ptrs: torch.Tensor, workspace, stream=None) -> None:
    """Linear attention with a decay for each head over packed prompts, the slots' states in place (dims from
    make_linear_dims(), workspace from linear_workspace()). q, k: [T, Hk * d] or [T, Hk, d], v likewise, rows
    of a wider tensor allowed; g: fp32 [T, Hv], or [Hv] for one decay a head."""
    fn, n, rows = "linear_prefill", state_ptrs.numel(), q.shape[0]
    qp, qs, kp, ks, vp, vs, gp, gs, op, sp = _linear_operands(fn, dims, q, k, v, g, o, state_ptrs)
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _lib._launch("gdn_linear_prefill", _lib._LIB.gdn_linear_prefill, stream, q, ctypes.byref(dims), qp, qs, kp, ks, vp, vs, gp, gs, op,
                 _at(fn, "cu_seqlens", cu_seqlens, _I32, n + 1, q.get_device()), n, rows, sp,
                 None if workspace is None else _at(fn, "workspace", workspace, workspace.dtype, workspace.numel(), q.get_device()), size)


def linear_decode(dims: gdn_dims, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, o: torch.Tensor,
                  state_ptrs: torch.Tensor, stream=None) -> None:
    """linear_prefill for one token of each of m slots: row i of q, k, v, g and o is slot i's."""
    fn, m = "linear_decode", state_ptrs.numel()
    qp, qs, kp, ks, vp, vs, gp, gs, op, sp = _linear_operands(fn, dims, q, k, v, g, o, state_ptrs)
    if q.shape[0] != m:
        raise ValueError(f"{fn}: {q.shape[0]} rows for {m} slots")
    _lib._launch("gdn_linear_decode", _lib._LIB.gdn_linear_decode, stream, q, ctypes.byref(dims), qp, qs, kp, ks, vp, vs, gp, gs, op, sp, m)


def block_norm(dims, x: torch.Tensor, residual, y, residual_out=None, gate=None, post_weight=None, post_bias=None,
               pre_weight=None, pre_bias=None, stream=None) -> None:
    """h = residual + scale act(gate) a with a = x or its norm, and y the norm of h (dims from make_block_norm_dims(), all
    operands' types among them). h goes to residual_out (may be residual itself; None: not stored); y None: no
    second norm; residual None: 0. x, residual, residual_out, y: [rows, width]; gate: the same, or [width] for all rows; weights and
    biases [width]."""
    fn, rows, width, at = "block_norm", x.shape[0], dims.width, x.get_device()
    n, stream_t, param = rows * width, _DTYPES.get(dims.residual_dtype), _DTYPES.get(dims.param_dtype)

    def of(name, t, dtype):
        return (None, 0) if t is None else (t.data_ptr(), _row_stride(name, t, dtype, rows, n, at, fn))

    def vector(name, t):
        return None if t is None else _at(fn, name, t, param, width, at)

    gate_t = _DTYPES.get(dims.gate_dtype)
    one = gate is not None and gate.dim() == 1
    gp, gs = (_at(fn, "gate", gate, gate_t, width, at), 0) if one else of("gate", gate, gate_t)
    if not one and gate is not None and gs < width and rows > 1:
        raise ValueError(f"{fn}: the rows of gate overlap (strides {gate.stride()}); one row for all is given as [{width}]")
    if gate is not None and not one:
        gs = max(gs, width)
    _lib._launch("gdn_block_norm", _lib._LIB.gdn_block_norm, stream, x, ctypes.byref(dims), *of("x", x, _DTYPES.get(dims.in_dtype)),
                 *of("residual", residual, stream_t), gp, gs, vector("post_weight", post_weight), vector("post_bias", post_bias),
                 vector("pre_weight", pre_weight), vector("pre_bias", pre_bias), *of("residual_out", residual_out, stream_t),
                 *of("y", y, _DTYPES.get(dims.out_dtype)), rows)


def sample(logits: torch.Tensor, uniform: torch.Tensor, tokens: torch.Tensor, workspace, temperature=None, top_k=None,
           top_p=None, min_p=None, prob=None, stream=None) -> None:
    """tokens[r] (int32) drawn from row r of logits [rows, vocab] by the random number uniform[r] in [0, 1): softmax at
    temperature[r] (0: the likeliest token), cut by top_k[r] (int32), top_p[r] and min_p[r]; prob[r]: its
    probability there. fp32 where not said; None leaves a filter out. workspace from sample_workspace()."""
    fn, at = "sample", logits.get_device()
    if logits.dim() != 2 or logits.dtype not in _KINDS:
        raise ValueError(f"{fn}: logits must be fp32 or bf16 [rows, vocab] (got {logits.dtype}, shape {tuple(logits.shape)})")
    rows, vocab = logits.shape

    def of(name, t, dtype=_F32):
        return None if t is None else _at(fn, name, t, dtype, rows, at)

    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _lib._launch("gdn_sample", _lib._LIB.gdn_sample, stream, logits, logits.data_ptr(),
                 _row_stride("logits", logits, logits.dtype, rows, rows * vocab, at, fn), _KINDS[logits.dtype], rows, vocab,
                 of("temperature", temperature), of("top_k", top_k, _I32), of("top_p", top_p), of("min_p", min_p),
                 _at(fn, "uniform", uniform, _F32, rows, at), _at(fn, "tokens", tokens, _I32, rows, at), of("prob", prob),
                 None if workspace is None else _at(fn, "workspace", workspace, workspace.dtype, workspace.numel(), at), size)


def tree_follow(drafted: torch.Tensor, sampled: torch.Tensor, pending: torch.Tensor, parents, cu_nodes: torch.Tensor,
                max_nodes: int, accepted: torch.Tensor, next: torch.Tensor, path=None, stream=None) -> None:
    """The path that the sampled tokens take through each slot's drafted tree: its last node in accepted (tree_accept's
    operand), the token after it in next (may be pending itself), its nodes in path [m, max_nodes]. All int32."""
    fn, m, rows, at = "tree_follow", pending.numel(), drafted.numel(), pending.get_device()
    _lib._launch("gdn_tree_follow", _lib._LIB.gdn_tree_follow, stream, pending, _at(fn, "drafted", drafted, _I32, rows, at),
                 _at(fn, "sampled", sampled, _I32, rows, at), _at(fn, "pending", pending, _I32, m, at),
                 None if parents is None else _at(fn, "parents", parents, _I32, rows, at), _at(fn, "cu_nodes", cu_nodes, _I32, m + 1, at),
                 m, rows, max_nodes, _at(fn, "accepted", accepted, _I32, m, at), _at(fn, "next", next, _I32, m, at),
                 None if path is None else _at(fn, "path", path, _I32, m * max_nodes, at))


def linear_workspace(dims: gdn_dims, num_seqs: int, total_tokens: int, device="cuda") -> torch.Tensor:
    nbytes = _lib.gdn_linear_workspace_size(dims, num_seqs, total_tokens)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def sample_workspace(rows: int, vocab: int, device="cuda") -> torch.Tensor:
    nbytes = _lib.gdn_sample_workspace_size(rows, vocab)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def prefill_workspace(dims: gdn_dims, num_seqs: int, total_tokens: int, device="cuda") -> torch.Tensor:
    nbytes = _lib.gdn_prefill_workspace_size(dims, num_seqs, total_tokens)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def prefill_fused_workspace(dims: gdn_dims, num_seqs: int, total_tokens: int, device="cuda") -> torch.Tensor:
    nbytes = _lib.gdn_prefill_fused_workspace_size(dims, num_seqs, total_tokens)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


__all__ = ["SlotPool", "block_norm", "channels", "conv_update", "decode", "decode_fused", "group_norm", "linear_decode",
           "linear_prefill", "linear_workspace", "packed_slots", "prefill", "prefill_fused", "prefill_fused_static",
           "prefill_fused_workspace", "prefill_workspace", "qkv_views", "sample", "sample_workspace", "slot_pack",
           "slot_unpack", "torch_in_dtype", "tree_accept", "tree_follow", "tree_record", "tree_verify",
           "GDN_F32", "GDN_BF16"]
