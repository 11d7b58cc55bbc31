"""Tensor-level helpers over the C ABI (argument marshalling only).

``SlotPool`` is the caller-owned slot pool: one device allocation of equal-sized
fp32 recurrent-state blocks and one of conv-state blocks, addressed per call through
device arrays of 64-bit block addresses that gdn_slot_pointers builds on the device.
(The "qLLM" page, section "What this is", keeps the linear-attention layers' recurrent
and conv state in such a pool of slots; aprender #5279, "Phase plan", phase P5, puts
the slot index on the launch grid and hands the kernels one address per slot.)

``conv_update``, ``prefill``, ``decode``, ``decode_fused``, ``tree_verify``, ``tree_accept``,
``slot_pack``, ``slot_unpack`` and ``group_norm`` derive pointers, strides and views from torch
tensors and call the library; all arithmetic happens in the HIP kernels.
"""

from __future__ import annotations

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
        assert slot_idx.numel() <= packed.shape[0]
        sp, cp = self.pointers(slot_idx)
        slot_pack(self.dims, fmt, sp, cp if conv_state else None, self._blocks(packed, slot_idx))

    def unpack_slots(self, packed: torch.Tensor, block_idx: torch.Tensor, slot_idx: torch.Tensor, fmt: int,
                     conv_state: bool = True) -> None:
        """Slot slot_idx[i] filled from row block_idx[i] of packed (int32 device index tensors, slots
        distinct; one block may fill several slots). An index outside its pool skips the entry."""
        assert block_idx.numel() == slot_idx.numel()
        sp, cp = self.pointers(slot_idx)
        slot_unpack(self.dims, fmt, self._blocks(packed, slot_idx, block_idx), sp, cp if conv_state else None)

    def _blocks(self, packed: torch.Tensor, slot_idx: torch.Tensor, block_idx=None) -> torch.Tensor:
        """Device addresses of packed's rows block_idx (default: 0, 1, ..), 0 outside it."""
        n = slot_idx.numel()
        assert packed.dtype == torch.uint8 and packed.dim() == 2 and packed.is_contiguous()
        assert packed.shape[1] == _lib.gdn_slot_packed_size(self.dims, _lib.GDN_PACK_INT8)  # (both formats')
        if block_idx is None:
            block_idx = torch.arange(n, dtype=torch.int32, device=slot_idx.device)
        assert block_idx.dtype == torch.int32 and block_idx.is_cuda
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


def _check_tree(dims, x, parents, cu_nodes, state_ptrs, conv_state_ptrs) -> None:
    m = state_ptrs.numel()
    assert x.shape[1] == channels(dims) and x.stride(1) == 1 and x.dtype == torch_in_dtype(dims)
    assert cu_nodes.dtype == torch.int32 and cu_nodes.is_cuda and cu_nodes.numel() == m + 1
    assert conv_state_ptrs.numel() == m
    assert parents is None or (parents.dtype == torch.int32 and parents.is_cuda and parents.numel() == x.shape[0])


def _check_record(dims, record, rows: int):
    k, u, gamma = record
    Hk, Hv, d = dims.num_k_heads, dims.num_v_heads, dims.head_dim
    assert k.numel() == rows * Hk * d and u.numel() == rows * Hv * d and gamma.numel() == rows * Hv
    return record


def tree_verify(dims: gdn_dims, x: torch.Tensor, conv_w: torch.Tensor, conv_b, g: torch.Tensor, beta: torch.Tensor,
                o: torch.Tensor, parents, cu_nodes: torch.Tensor, max_nodes: int, state_ptrs: torch.Tensor,
                conv_state_ptrs: torch.Tensor, record=None, stream=None) -> None:
    """The drafted trees of m slots answered against their states, which stay as they are;
    parents None: chains. record (from tree_record()) is needed to accept nodes afterwards."""
    _check_tree(dims, x, parents, cu_nodes, state_ptrs, conv_state_ptrs)
    rows = x.shape[0]
    gates = rows * dims.num_v_heads
    assert g.numel() == gates and beta.numel() == gates and o.numel() == gates * dims.head_dim and o.is_contiguous()
    k, u, gamma = _check_record(dims, record, rows) if record is not None else (None, None, None)
    _lib.gdn_tree_verify(dims, x, x.stride(0), conv_w, conv_b, g, beta, o, parents, cu_nodes, state_ptrs.numel(),
                         x.shape[0], max_nodes, state_ptrs, conv_state_ptrs, k, u, gamma, stream)


def tree_accept(dims: gdn_dims, x: torch.Tensor, record, parents, cu_nodes: torch.Tensor, max_nodes: int,
                accepted: torch.Tensor, state_ptrs: torch.Tensor, conv_state_ptrs: torch.Tensor, stream=None) -> None:
    """Slot i's state and conv state moved along the root path of node accepted[i] (-1: none)."""
    _check_tree(dims, x, parents, cu_nodes, state_ptrs, conv_state_ptrs)
    assert accepted.dtype == torch.int32 and accepted.is_cuda and accepted.numel() == state_ptrs.numel()
    k, u, gamma = _check_record(dims, record, x.shape[0])
    _lib.gdn_tree_accept(dims, x, x.stride(0), k, u, gamma, parents, cu_nodes, accepted, state_ptrs.numel(),
                         x.shape[0], max_nodes, state_ptrs, conv_state_ptrs, stream)


def slot_pack(dims: gdn_dims, fmt: int, state_ptrs: torch.Tensor, conv_state_ptrs, packed_ptrs: torch.Tensor,
              stream=None) -> None:
    _lib.gdn_slot_pack(dims, fmt, state_ptrs, conv_state_ptrs, packed_ptrs, state_ptrs.numel(), stream)


def slot_unpack(dims: gdn_dims, fmt: int, packed_ptrs: torch.Tensor, state_ptrs: torch.Tensor, conv_state_ptrs,
                stream=None) -> None:
    _lib.gdn_slot_unpack(dims, fmt, packed_ptrs, state_ptrs, conv_state_ptrs, state_ptrs.numel(), stream)


def group_norm(dims, x: torch.Tensor, weight, y: torch.Tensor, gate=None, bias=None, stream=None) -> None:
    """y = the norm of every group of every row of x, times weight, plus bias, gated (dims from
    make_norm_dims()). Rows are the first axis; the other axes of x, gate and y are contiguous."""
    rows = x.shape[0]
    n = rows * dims.groups * dims.group_size
    _lib.gdn_group_norm(dims, x, _row_stride(x, rows, n), gate, 0 if gate is None else _row_stride(gate, rows, n),
                        weight, bias, y, _row_stride(y, rows, n), rows, stream)


def _row_stride(t: torch.Tensor, rows: int, n: int) -> int:
    """Row stride of t, which holds n values in `rows` contiguous rows, [rows, width] or [rows, a, b]."""
    s, shape = t.stride(), t.shape
    assert s[-1] == 1 and shape[0] == rows and t.numel() == n and (len(s) == 2 or (len(s) == 3 and s[1] == shape[2]))
    return s[0]


def prefill_workspace(dims: gdn_dims, num_seqs: int, total_tokens: int, device="cuda") -> torch.Tensor:
    nbytes = _lib.gdn_prefill_workspace_size(dims, num_seqs, total_tokens)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def prefill_fused_workspace(dims: gdn_dims, num_seqs: int, total_tokens: int, device="cuda") -> torch.Tensor:
    nbytes = _lib.gdn_prefill_fused_workspace_size(dims, num_seqs, total_tokens)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


__all__ = ["SlotPool", "channels", "conv_update", "decode", "decode_fused", "group_norm", "packed_slots", "prefill",
           "prefill_fused", "prefill_fused_static", "prefill_fused_workspace", "prefill_workspace", "qkv_views",
           "slot_pack", "slot_unpack", "torch_in_dtype", "tree_accept", "tree_record", "tree_verify",
           "GDN_F32", "GDN_BF16"]
