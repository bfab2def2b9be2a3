"""Python binding of libsconv: torch tensors in, one C-ABI call out.

Each function only checks what the C ABI cannot see (tensor dtype, device,
dimensionality), turns tensors into pointers, element strides and the
current HIP stream, and calls the library.  All computation happens in the
HIP kernels; there is no CPU path.  Argument names follow the source pages.
"""
from __future__ import annotations

import ctypes
from typing import List, Optional, Sequence

import torch

from . import _lib

_DT = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}


def _dtype(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"element type must be float32 or bfloat16, got {t.dtype}")
    return _DT[t.dtype]


def _act(activation) -> int:
    if activation in (None, False, "none"):
        return _lib.ACT_NONE
    if activation in (True, "silu", "swish"):
        return _lib.ACT_SILU
    raise ValueError(f"unknown activation {activation!r}")


def _dev(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libsconv tensors must live on the GPU")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _vec(t: torch.Tensor, dtype: torch.dtype, name: str, min_len: int = 0):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous 1-D tensor")
    if t.numel() < min_len:
        raise ValueError(f"{name} has {t.numel()} entries, needs {min_len}")


def _stream(t: torch.Tensor):
    return torch.cuda.current_stream(t.device).cuda_stream


def sconv_init() -> None:
    """Load the library's GPU code on the current device (before a first
    call that is captured into a graph)."""
    _lib.check(_lib.load().sconv_init(), "sconv_init")


def sconv_seq_metadata(query_start_loc: torch.Tensor, num_reqs: int, num_actual_tokens: int,
                       seq_idx_out: torch.Tensor, query_start_out: torch.Tensor,
                       num_padded_tokens: Optional[int] = None) -> None:
    """Fill the static per-token seq_idx / query_start buffers in one launch."""
    if num_padded_tokens is None:
        num_padded_tokens = num_actual_tokens
    _dev(query_start_loc, seq_idx_out, query_start_out)
    _vec(query_start_loc, torch.int32, "query_start_loc", num_reqs + 1 if num_actual_tokens else 0)
    _vec(seq_idx_out, torch.int32, "seq_idx_out")
    _vec(query_start_out, torch.int32, "query_start_out")
    rc = _lib.load().sconv_seq_metadata(
        _ptr(query_start_loc), int(num_reqs), int(num_actual_tokens), int(num_padded_tokens),
        _ptr(seq_idx_out), seq_idx_out.numel(), _ptr(query_start_out), query_start_out.numel(),
        _stream(seq_idx_out))
    _lib.check(rc, "sconv_seq_metadata")


def _fused_checks(x, weight, cache, positions, block_table, slot_mapping, off_s, ws,
                  block_size, out):
    T = x.shape[0]
    if x.dim() != 2 or weight.dim() != 2 or cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("x [T, C], weight [C, W], cache [nb, H, N, D], block_table [R, M]")
    if block_table.shape[1] > 1 and block_table.stride(1) != 1:
        # the C ABI takes a row stride only: entries of a row are contiguous
        raise ValueError("block_table needs contiguous entries within a row")
    _dev(x, weight, cache, positions, block_table, slot_mapping, out)
    dt = _dtype(x)
    if weight.dtype != x.dtype or cache.dtype != x.dtype or out.dtype != x.dtype:
        raise TypeError("x, weight, cache and out must share one element type")
    if x.stride(1) != 1 or out.stride(1) != 1:
        raise ValueError("x and out need contiguous channels")
    if cache.stride(3) != 1:
        raise ValueError("cache D-dim must be contiguous")
    nb, H, N, D = cache.shape
    if N != block_size:
        raise ValueError(f"block_size {block_size} != cache block dim {N}")
    if x.shape[1] != H * ws or weight.shape[0] != H * ws or out.shape != x.shape:
        raise ValueError("x / weight / out channel dim must be H*ws")
    if block_table.dtype != torch.int32:
        raise TypeError("block_table must be int32")
    _vec(positions, torch.int64, "positions", T)
    _vec(slot_mapping, torch.int64, "slot_mapping", T)
    return dt


def _table_rows(block_table: torch.Tensor, num_reqs: int):
    # With the request offsets the launch may read any row below num_reqs.
    if block_table.shape[0] < num_reqs:
        raise ValueError(f"block_table has {block_table.shape[0]} rows, needs num_reqs="
                         f"{num_reqs}")


def sconv_fused_insert_conv(x: torch.Tensor, weight: torch.Tensor, cache: torch.Tensor,
                            positions: torch.Tensor, block_table: torch.Tensor,
                            seq_idx: torch.Tensor, slot_mapping: torch.Tensor,
                            query_start: torch.Tensor, off_s: int, ws: int, block_size: int,
                            activation: Optional[str] = None, use_residual: bool = True,
                            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Single-launch insert + depthwise causal conv1d over the paged cache.

    x [T, H*ws], weight [H*ws, W], cache [num_blocks, H, N, D] (modified),
    positions int64 [T], block_table int32 [num_reqs, max_blocks],
    seq_idx / query_start int32 [T], slot_mapping int64 [T] (-1 = PAD).
    Returns ``out`` (new [T, H*ws] tensor unless given; PAD rows untouched).
    """
    if out is None:
        out = torch.empty_like(x)
    if x.shape[0] == 0:
        return out
    dt = _fused_checks(x, weight, cache, positions, block_table, slot_mapping, off_s, ws,
                       block_size, out)
    T = x.shape[0]
    _dev(seq_idx, query_start)
    _vec(seq_idx, torch.int32, "seq_idx", T)
    _vec(query_start, torch.int32, "query_start", T)
    nb, H, N, D = cache.shape
    rc = _lib.load().sconv_fused_insert_conv(
        _ptr(x), x.stride(0), _ptr(weight), weight.stride(0), weight.stride(1),
        _ptr(cache), nb, H, N, D, cache.stride(0), cache.stride(1), cache.stride(2),
        _ptr(positions), _ptr(block_table), block_table.stride(0), block_table.shape[1],
        _ptr(seq_idx), _ptr(slot_mapping), _ptr(query_start), _ptr(out), out.stride(0),
        T, int(off_s), int(ws), weight.shape[1], dt, _act(activation), int(bool(use_residual)),
        _stream(x))
    _lib.check(rc, "sconv_fused_insert_conv")
    return out


def sconv_fused_insert_conv_qsl(x: torch.Tensor, weight: torch.Tensor, cache: torch.Tensor,
                                positions: torch.Tensor, block_table: torch.Tensor,
                                query_start_loc: torch.Tensor, num_reqs: int,
                                slot_mapping: torch.Tensor, off_s: int, ws: int,
                                block_size: int, activation: Optional[str] = None,
                                use_residual: bool = True,
                                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """sconv_seq_metadata + sconv_fused_insert_conv in one launch: rows find
    their request in query_start_loc [num_reqs + 1] inside the kernel."""
    if out is None:
        out = torch.empty_like(x)
    if x.shape[0] == 0:
        return out
    dt = _fused_checks(x, weight, cache, positions, block_table, slot_mapping, off_s, ws,
                       block_size, out)
    T = x.shape[0]
    _dev(query_start_loc)
    _vec(query_start_loc, torch.int32, "query_start_loc", num_reqs + 1)
    _table_rows(block_table, num_reqs)
    nb, H, N, D = cache.shape
    rc = _lib.load().sconv_fused_insert_conv_qsl(
        _ptr(x), x.stride(0), _ptr(weight), weight.stride(0), weight.stride(1),
        _ptr(cache), nb, H, N, D, cache.stride(0), cache.stride(1), cache.stride(2),
        _ptr(positions), _ptr(block_table), block_table.stride(0), block_table.shape[1],
        _ptr(query_start_loc), int(num_reqs), _ptr(slot_mapping), _ptr(out), out.stride(0),
        T, int(off_s), int(ws), weight.shape[1], dt, _act(activation), int(bool(use_residual)),
        _stream(x))
    _lib.check(rc, "sconv_fused_insert_conv_qsl")
    return out


def sconv_fused_insert_conv_streams(xs: Sequence[torch.Tensor], weights: Sequence[torch.Tensor],
                                    cache: torch.Tensor, positions: torch.Tensor,
                                    block_table: torch.Tensor, slot_mapping: torch.Tensor,
                                    off_s: Sequence[int], ws: Sequence[int], block_size: int,
                                    activation=None, use_residual=True,
                                    seq_idx: Optional[torch.Tensor] = None,
                                    query_start: Optional[torch.Tensor] = None,
                                    query_start_loc: Optional[torch.Tensor] = None,
                                    num_reqs: Optional[int] = None,
                                    outs: Optional[Sequence[torch.Tensor]] = None
                                    ) -> List[torch.Tensor]:
    """The insert + conv of up to four streams of one layer in one launch.

    Stream s has x ``xs[s]`` [T, H*ws[s]], weight ``weights[s]`` [H*ws[s], W]
    and cache columns [off_s[s], off_s[s] + ws[s]) of every head.
    ``activation`` and ``use_residual`` are one value for all streams or a
    sequence with one per stream.  Rows find their request either from
    ``seq_idx`` / ``query_start`` or, inside the launch, from
    ``query_start_loc`` with ``num_reqs``.  Returns the outputs.
    """
    if outs is None:
        outs = [torch.empty_like(x) for x in xs]
    args = _streams_args(xs, weights, cache, positions, block_table, slot_mapping, off_s, ws,
                         block_size, activation, use_residual, seq_idx, query_start,
                         query_start_loc, num_reqs, outs)
    if args is None:
        return list(outs)
    rc = _lib.load().sconv_fused_insert_conv_streams(*args, _stream(xs[0]))
    _lib.check(rc, "sconv_fused_insert_conv_streams")
    return list(outs)


def sconv_fused_plan(xs: Sequence[torch.Tensor], weights: Sequence[torch.Tensor],
                     cache: torch.Tensor, positions: torch.Tensor, block_table: torch.Tensor,
                     slot_mapping: torch.Tensor, off_s: Sequence[int], ws: Sequence[int],
                     block_size: int, activation=None, use_residual=True,
                     seq_idx: Optional[torch.Tensor] = None,
                     query_start: Optional[torch.Tensor] = None,
                     query_start_loc: Optional[torch.Tensor] = None,
                     num_reqs: Optional[int] = None,
                     outs: Optional[Sequence[torch.Tensor]] = None,
                     gather: Optional[tuple] = None) -> dict:
    """The launch sconv_fused_insert_conv_streams (or, with ``gather`` =
    (src, abs_positions, real_count_gpu, out, d_conv),
    sconv_fused_insert_conv_gather) would make for these arguments, as a
    dict of the plan's fields; nothing is launched."""
    if outs is None:
        outs = [torch.empty_like(x) for x in xs]
    plan = _lib.FusedPlan()
    args = _streams_args(xs, weights, cache, positions, block_table, slot_mapping, off_s, ws,
                         block_size, activation, use_residual, seq_idx, query_start,
                         query_start_loc, num_reqs, outs)
    g = None if gather is None else _window_gather(*gather)[0]
    if args is not None:
        rc = _lib.load().sconv_fused_plan(*args, None if g is None else ctypes.byref(g),
                                          ctypes.byref(plan))
        _lib.check(rc, "sconv_fused_plan")
    return {name: getattr(plan, name) for name, _ in _lib.FusedPlan._fields_}


def _streams_args(xs, weights, cache, positions, block_table, slot_mapping, off_s, ws,
                  block_size, activation, use_residual, seq_idx, query_start, query_start_loc,
                  num_reqs, outs):
    """Checked C arguments of the multi-stream entry points (without the
    stream), or None when there is nothing to launch."""
    n = len(xs)
    if not (len(weights) == len(off_s) == len(ws) == n):
        raise ValueError("xs, weights, off_s and ws need one entry per stream")
    acts = list(activation) if isinstance(activation, (list, tuple)) else [activation] * n
    ress = list(use_residual) if isinstance(use_residual, (list, tuple)) else [use_residual] * n
    if len(acts) != n or len(ress) != n or len(outs) != n:
        raise ValueError("activation, use_residual and outs need one entry per stream")
    T = xs[0].shape[0] if n else 0
    if n == 0 or T == 0:
        return None
    if any(x.shape[0] != T for x in xs):
        raise ValueError("every stream needs the same rows T")
    dt = None
    for x, w, o, a, b in zip(xs, weights, outs, off_s, ws):
        dt = _fused_checks(x, w, cache, positions, block_table, slot_mapping, a, b, block_size, o)
    if any(w.shape[1] != weights[0].shape[1] for w in weights):
        raise ValueError("every stream needs the same filter width W")
    if any(x.dtype != xs[0].dtype for x in xs):
        raise TypeError("every stream needs the same element type")
    if query_start_loc is not None:
        if seq_idx is not None or query_start is not None or num_reqs is None:
            raise ValueError("give query_start_loc with num_reqs, or seq_idx and query_start")
        _dev(query_start_loc)
        _vec(query_start_loc, torch.int32, "query_start_loc", num_reqs + 1)
        _table_rows(block_table, num_reqs)
    else:
        if seq_idx is None or query_start is None:
            raise ValueError("give query_start_loc with num_reqs, or seq_idx and query_start")
        _dev(seq_idx, query_start)
        _vec(seq_idx, torch.int32, "seq_idx", T)
        _vec(query_start, torch.int32, "query_start", T)
    arr = (_lib.StreamT * n)()
    for i, (x, w, o) in enumerate(zip(xs, weights, outs)):
        arr[i] = _lib.StreamT(_ptr(x), x.stride(0), _ptr(w), w.stride(0), w.stride(1), _ptr(o),
                              o.stride(0), int(off_s[i]), int(ws[i]), _act(acts[i]),
                              int(bool(ress[i])))
    nb, H, N, D = cache.shape
    return (arr, n, _ptr(cache), nb, H, N, D, cache.stride(0), cache.stride(1), cache.stride(2),
            _ptr(positions), _ptr(block_table), block_table.stride(0), block_table.shape[1],
            _ptr(seq_idx), _ptr(query_start), _ptr(query_start_loc),
            int(num_reqs) if num_reqs is not None else 0, _ptr(slot_mapping), T,
            weights[0].shape[1], dt)


def causal_conv1d_varlen_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                             conv_states: torch.Tensor, query_start_loc: torch.Tensor,
                             cache_indices: Optional[torch.Tensor],
                             has_initial_state: Optional[torch.Tensor], silu_activation: bool,
                             pad_slot_id: int = -1, out: Optional[torch.Tensor] = None
                             ) -> torch.Tensor:
    """Varlen causal conv1d over channel-major x [dim, total_T].

    conv_states [num_slots, dim, W-1] is updated in place.  With ``out`` None
    the result overwrites x (in place, as the source op does) and x is
    returned.
    """
    if out is None:
        out = x
    if x.dim() != 2 or weight.dim() != 2 or conv_states.dim() != 3:
        raise ValueError("x [dim, total_T], weight [dim, W], conv_states [slots, dim, W-1]")
    dim, total_T = x.shape
    W = weight.shape[1]
    batch = query_start_loc.numel() - 1
    _dev(x, weight, bias, conv_states, query_start_loc, cache_indices, has_initial_state, out)
    dt = _dtype(x)
    for t in (weight, conv_states, out) + ((bias,) if bias is not None else ()):
        if t.dtype != x.dtype:
            raise TypeError("x, weight, bias, conv_states and out must share one element type")
    if weight.shape[0] != dim or conv_states.shape[1] != dim or conv_states.shape[2] != W - 1:
        raise ValueError("weight / conv_states shapes do not match x")
    if out.shape != x.shape:
        raise ValueError("out must have x's shape")
    if bias is not None:
        _vec(bias, x.dtype, "bias", dim)
    _vec(query_start_loc, torch.int32, "query_start_loc")
    if cache_indices is not None:
        _vec(cache_indices, torch.int32, "cache_indices", batch)
    hi = None
    if has_initial_state is not None:
        hi = has_initial_state
        if hi.dtype == torch.bool:
            hi = hi.view(torch.uint8)
        _vec(hi, torch.uint8, "has_initial_state", batch)
    rc = _lib.load().causal_conv1d_varlen_fwd(
        _ptr(x), x.stride(0), x.stride(1), _ptr(weight), weight.stride(0), weight.stride(1),
        _ptr(bias), _ptr(conv_states), conv_states.shape[0], conv_states.stride(0),
        conv_states.stride(1), conv_states.stride(2), _ptr(query_start_loc), batch,
        _ptr(cache_indices), _ptr(hi), _ptr(out), out.stride(0), out.stride(1), dim, total_T,
        W, dt, _lib.ACT_SILU if silu_activation else _lib.ACT_NONE, int(pad_slot_id), _stream(x))
    _lib.check(rc, "causal_conv1d_varlen_fwd")
    return out


def causal_conv1d_update(x: torch.Tensor, conv_state: torch.Tensor, weight: torch.Tensor,
                         bias: Optional[torch.Tensor], silu_activation: bool,
                         cache_seqlens: Optional[torch.Tensor] = None,
                         conv_state_indices: Optional[torch.Tensor] = None,
                         pad_slot_id: int = -1, out: Optional[torch.Tensor] = None
                         ) -> torch.Tensor:
    """One decode step: x [batch, dim]; conv_state [num_slots, dim, W-1]
    updated in place.  With ``out`` None the result overwrites x."""
    if out is None:
        out = x
    if x.dim() != 2 or weight.dim() != 2 or conv_state.dim() != 3:
        raise ValueError("x [batch, dim], weight [dim, W], conv_state [slots, dim, W-1]")
    batch, dim = x.shape
    W = weight.shape[1]
    _dev(x, conv_state, weight, bias, conv_state_indices, out)
    dt = _dtype(x)
    for t in (weight, conv_state, out) + ((bias,) if bias is not None else ()):
        if t.dtype != x.dtype:
            raise TypeError("x, weight, bias, conv_state and out must share one element type")
    if x.stride(1) != 1 or out.stride(1) != 1:
        raise ValueError("x and out need contiguous channels")
    if weight.shape[0] != dim or conv_state.shape[1] != dim or conv_state.shape[2] != W - 1:
        raise ValueError("weight / conv_state shapes do not match x")
    if bias is not None:
        _vec(bias, x.dtype, "bias", dim)
    if conv_state_indices is not None:
        _vec(conv_state_indices, torch.int32, "conv_state_indices", batch)
    if cache_seqlens is not None:
        _dev(cache_seqlens)
        _vec(cache_seqlens, torch.int32, "cache_seqlens", batch)
    rc = _lib.load().causal_conv1d_update(
        _ptr(x), x.stride(0), _ptr(conv_state), conv_state.shape[0], conv_state.stride(0),
        conv_state.stride(1), conv_state.stride(2), _ptr(weight), weight.stride(0),
        weight.stride(1), _ptr(bias), _ptr(cache_seqlens), _ptr(conv_state_indices), _ptr(out),
        out.stride(0), batch, dim, W, dt, _lib.ACT_SILU if silu_activation else _lib.ACT_NONE,
        int(pad_slot_id), _stream(x))
    _lib.check(rc, "causal_conv1d_update")
    return out


def causal_conv1d_update_tokens(x: torch.Tensor, conv_state: torch.Tensor, weight: torch.Tensor,
                                bias: Optional[torch.Tensor], silu_activation: bool,
                                cache_seqlens: Optional[torch.Tensor] = None,
                                conv_state_indices: Optional[torch.Tensor] = None,
                                pad_slot_id: int = -1, out: Optional[torch.Tensor] = None
                                ) -> torch.Tensor:
    """seqlen decode tokens per row: x [batch, dim, seqlen] (any strides);
    conv_state [num_slots, dim, state_len] (W-1 <= state_len <= 8) updated in
    place, a ring indexed by position when ``cache_seqlens`` (int32 [batch])
    is given.  With ``out`` None the result overwrites x."""
    if out is None:
        out = x
    if x.dim() != 3 or weight.dim() != 2 or conv_state.dim() != 3 or out.shape != x.shape:
        raise ValueError("x and out [batch, dim, seqlen], weight [dim, W], "
                         "conv_state [slots, dim, state_len]")
    batch, dim, seqlen = x.shape
    W = weight.shape[1]
    _dev(x, conv_state, weight, bias, conv_state_indices, cache_seqlens, out)
    dt = _dtype(x)
    for t in (weight, conv_state, out) + ((bias,) if bias is not None else ()):
        if t.dtype != x.dtype:
            raise TypeError("x, weight, bias, conv_state and out must share one element type")
    if weight.shape[0] != dim or conv_state.shape[1] != dim:
        raise ValueError("weight / conv_state shapes do not match x")
    if bias is not None:
        _vec(bias, x.dtype, "bias", dim)
    if conv_state_indices is not None:
        _vec(conv_state_indices, torch.int32, "conv_state_indices", batch)
    if cache_seqlens is not None:
        _vec(cache_seqlens, torch.int32, "cache_seqlens", batch)
    rc = _lib.load().causal_conv1d_update_tokens(
        _ptr(x), x.stride(0), x.stride(1), x.stride(2), seqlen, _ptr(conv_state),
        conv_state.shape[0], conv_state.shape[2], conv_state.stride(0), conv_state.stride(1),
        conv_state.stride(2), _ptr(weight), weight.stride(0), weight.stride(1), _ptr(bias),
        _ptr(cache_seqlens), _ptr(conv_state_indices), _ptr(out), out.stride(0), out.stride(1),
        out.stride(2), batch, dim, W, dt, _lib.ACT_SILU if silu_activation else _lib.ACT_NONE,
        int(pad_slot_id), _stream(x))
    _lib.check(rc, "causal_conv1d_update_tokens")
    return out


def gather_intermediate_conv_window(src: torch.Tensor, abs_positions: torch.Tensor,
                                    real_count_gpu: torch.Tensor, out: torch.Tensor,
                                    d_conv: int) -> None:
    """Gather length-d_conv windows of src[0] ending before abs_positions
    into out [max_count, conv_dim, d_conv] for the first real_count slots
    (count read on the device)."""
    g, dt = _window_gather(src, abs_positions, real_count_gpu, out, d_conv)
    rc = _lib.load().gather_intermediate_conv_window(
        g.src, g.seq_len, g.conv_dim, g.src_stride_s, g.src_stride_c, g.abs_positions,
        g.real_count, g.max_count, g.out, g.out_slot_stride, g.d_conv, dt, _stream(src))
    _lib.check(rc, "gather_intermediate_conv_window")


def _window_gather(src, abs_positions, real_count_gpu, out, d_conv):
    """Checked sconv_window_gather_t of a window gather, and its dtype code."""
    if src.dim() != 3 or out.dim() != 3:
        raise ValueError("src [batch, seq_len, conv_dim], out [max_count, conv_dim, d_conv]")
    _dev(src, abs_positions, real_count_gpu, out)
    dt = _dtype(src)
    if out.dtype != src.dtype:
        raise TypeError("src and out must share one element type")
    max_count, conv_dim, dc = out.shape
    if dc != d_conv or conv_dim != src.shape[2]:
        raise ValueError("out must be [max_count, conv_dim, d_conv]")
    if out.stride(2) != 1 or out.stride(1) != d_conv:
        raise ValueError("out slots must be dense (conv_dim, d_conv)")
    _vec(abs_positions, torch.int32, "abs_positions", max_count)
    _vec(real_count_gpu, torch.int32, "real_count_gpu", 1)
    g = _lib.WindowGather(_ptr(src), src.shape[1], conv_dim, src.stride(1), src.stride(2),
                          _ptr(abs_positions), _ptr(real_count_gpu), max_count, _ptr(out),
                          out.stride(0), d_conv)
    return g, dt


def sconv_fused_insert_conv_gather(xs: Sequence[torch.Tensor], weights: Sequence[torch.Tensor],
                                   cache: torch.Tensor, positions: torch.Tensor,
                                   block_table: torch.Tensor, slot_mapping: torch.Tensor,
                                   off_s: Sequence[int], ws: Sequence[int], block_size: int,
                                   gather_src: torch.Tensor, abs_positions: torch.Tensor,
                                   real_count_gpu: torch.Tensor, gather_out: torch.Tensor,
                                   d_conv: int, activation=None, use_residual=True,
                                   seq_idx: Optional[torch.Tensor] = None,
                                   query_start: Optional[torch.Tensor] = None,
                                   query_start_loc: Optional[torch.Tensor] = None,
                                   num_reqs: Optional[int] = None,
                                   outs: Optional[Sequence[torch.Tensor]] = None
                                   ) -> List[torch.Tensor]:
    """sconv_fused_insert_conv_streams and gather_intermediate_conv_window
    (gather_src, abs_positions, real_count_gpu, gather_out, d_conv) in one
    launch.  Returns the conv outputs; gather_out is written in place."""
    if outs is None:
        outs = [torch.empty_like(x) for x in xs]
    g, gdt = _window_gather(gather_src, abs_positions, real_count_gpu, gather_out, d_conv)
    args = _streams_args(xs, weights, cache, positions, block_table, slot_mapping, off_s, ws,
                         block_size, activation, use_residual, seq_idx, query_start,
                         query_start_loc, num_reqs, outs)
    if args is None:  # no rows: the gather alone
        gather_intermediate_conv_window(gather_src, abs_positions, real_count_gpu, gather_out,
                                        d_conv)
        return list(outs)
    if gdt != args[-1]:
        raise TypeError("the gather and the conv must share one element type")
    rc = _lib.load().sconv_fused_insert_conv_gather(*args, ctypes.byref(g), _stream(xs[0]))
    _lib.check(rc, "sconv_fused_insert_conv_gather")
    return list(outs)


def gather_intermediate_ssm_state(states: torch.Tensor, chunk_indices: torch.Tensor,
                                  real_count_gpu: torch.Tensor, out: torch.Tensor) -> None:
    """Copy states[chunk_indices[i]] into out[i] for the first real_count
    slots (count read on the device).  states [num_chunks, *state_shape],
    out [max_count, *state_shape]; each row must be dense."""
    _dev(states, chunk_indices, real_count_gpu, out)
    dt = _dtype(states)
    if out.dtype != states.dtype:
        raise TypeError("states and out must share one element type")
    if states.shape[1:] != out.shape[1:]:
        raise ValueError("states and out rows must have one shape")
    flat = 1
    for d in states.shape[1:]:
        flat *= d
    for t, name in ((states, "states"), (out, "out")):
        if t.dim() > 1 and not t[0].is_contiguous():
            raise ValueError(f"{name} rows must be dense")
    max_count = out.shape[0]
    _vec(chunk_indices, torch.int64, "chunk_indices", max_count)
    _vec(real_count_gpu, torch.int32, "real_count_gpu", 1)
    rc = _lib.load().gather_intermediate_ssm_state(
        _ptr(states), states.shape[0], flat, states.stride(0) if states.dim() > 1 else 1,
        _ptr(chunk_indices), _ptr(real_count_gpu), max_count, _ptr(out),
        out.stride(0) if out.dim() > 1 else 1, dt, _stream(states))
    _lib.check(rc, "gather_intermediate_ssm_state")


# ---------------------------------------------------------------- the layer around the conv

# The host's share of a small call is most of its time (a decode step's kernel
# takes 3 us): these helpers ask each tensor for little, and once.
_getters = [getattr(torch._C, n, None)
            for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice")]
_functions = {}


def _current_stream(index: int) -> int:
    if _getters[0] is not None:
        return _getters[0](index)
    return torch.cuda.current_stream(index).cuda_stream


def _current_device() -> int:
    return _getters[1]() if _getters[1] is not None else torch.cuda.current_device()


def _one_device(first: torch.Tensor, *ts):
    """Every tensor on the first one's GPU."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("libsconv tensors must live on the GPU")
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {first.device} and {t.device} in one call")


def _call(name: str, on: torch.Tensor, *args):
    """One library call on the current stream of `on`'s device."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(_lib.load(), name)
    index = on.get_device()
    if _current_device() == index:
        rc = fn(*args, _current_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _current_stream(index))
    if rc:
        _lib.check(rc, name)


def _floats(name: str, *args) -> int:
    """What a host query of the library writes to its last argument."""
    n = ctypes.c_int64()
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(_lib.load(), name)
    rc = fn(*args, ctypes.byref(n))
    if rc:
        _lib.check(rc, name)
    return n.value


def _same_type(x: torch.Tensor, what: str, *ts) -> int:
    dtype = x.dtype
    for t in ts:
        if t is not None and t.dtype != dtype:
            raise TypeError(f"{what} must share one element type")
    return _dtype(x)


def _dense(t: torch.Tensor, dtype: torch.dtype, name: str, min_len: int = 0):
    """t is a contiguous 1-D tensor of a type, of min_len entries at least."""
    if t.dtype != dtype or t.dim() != 1 or not t.is_contiguous() or t.numel() < min_len:
        _vec(t, dtype, name, min_len)


def _planes(shape, *ts):
    """[ptr, stride_c, stride_t] of each [dim, total_T] tensor."""
    args = []
    for t in ts:
        if t.shape != shape:
            raise ValueError("the [dim, total_T] tensors of a call must have one shape")
        args.append(t.data_ptr())
        args += t.stride()
    return args


def _packing(query_start_loc, cache_indices, has_initial_state):
    """(batch, has_initial_state as uint8) after checks."""
    batch = query_start_loc.numel() - 1
    _dense(query_start_loc, torch.int32, "query_start_loc", 1)
    if cache_indices is not None:
        _dense(cache_indices, torch.int32, "cache_indices", batch)
    hi = has_initial_state
    if hi is not None:
        if hi.dtype == torch.bool:
            hi = hi.view(torch.uint8)
        _dense(hi, torch.uint8, "has_initial_state", batch)
    return batch, hi


def _pool(t: Optional[torch.Tensor], dim: int, name: str):
    """(ptr, slots, slot stride) of an fp32 [num_slots, dim] state pool."""
    if t is None:
        return None, 0, 0
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != dim:
        raise ValueError(f"{name} must be [num_slots, dim]")
    stride = t.stride()
    if dim > 1 and stride[1] != 1:
        raise ValueError(f"{name} needs contiguous channels")
    return t.data_ptr(), shape[0], stride[0]


def _rows(shape, *ts):
    """[ptr, row stride] of each [rows, dim] tensor (None: NULL, 0)."""
    args = []
    wide = shape[1] > 1
    for t in ts:
        if t is None:
            args += (None, 0)
            continue
        stride = t.stride()
        if t.shape != shape or (wide and stride[1] != 1):
            raise ValueError("the [rows, dim] tensors of a call need one shape and contiguous "
                             "channels")
        args += (t.data_ptr(), stride[0])
    return args


def _checkpoint_rows(t: torch.Tensor, dim: int) -> int:
    if t.dtype != torch.float32 or t.dim() != 2 or t.shape[1] != dim or not t.is_contiguous():
        raise ValueError("checkpoints must be a dense float32 [rows, dim] tensor")
    return t.shape[0]


def gated_linear_recurrence_checkpoints(x: torch.Tensor, query_start_loc: torch.Tensor
                                        ) -> torch.Tensor:
    """The buffer in which gated_linear_recurrence_varlen_fwd leaves what its
    backward call needs, for inputs like x [dim, total_T]."""
    if x.dim() != 2:
        raise ValueError("x [dim, total_T]")
    rows = _floats("gated_linear_recurrence_checkpoint_rows", x.shape[1],
                   query_start_loc.numel() - 1)
    return torch.empty(rows, x.shape[0], dtype=torch.float32, device=x.device)


def _recurrence_workspace(total_T: int, batch: int, dim: int, backward: bool, x: torch.Tensor):
    """(tensor or None, floats) of workspace for one packed call."""
    fwd = ctypes.c_int64()
    bwd = _floats("gated_linear_recurrence_workspace", total_T, batch, dim, ctypes.byref(fwd))
    n = bwd if backward else fwd.value
    return (torch.empty(n, dtype=torch.float32, device=x.device) if n else None), n


def gated_linear_recurrence_varlen_fwd(x: torch.Tensor, gate_a: torch.Tensor,
                                       gate_x: torch.Tensor, decay: torch.Tensor,
                                       states: Optional[torch.Tensor],
                                       query_start_loc: torch.Tensor,
                                       cache_indices: Optional[torch.Tensor] = None,
                                       has_initial_state: Optional[torch.Tensor] = None,
                                       decay_scale: float = 8.0, pad_slot_id: int = -1,
                                       out: Optional[torch.Tensor] = None,
                                       checkpoints: Optional[torch.Tensor] = None
                                       ) -> torch.Tensor:
    """h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_x) x over packed
    sequences, a = exp(-decay_scale softplus(decay) sigmoid(gate_a)).

    x, gate_a, gate_x [dim, total_T] (any strides), decay float32 [dim].
    states float32 [num_slots, dim] is updated in place (None: start at zero,
    keep nothing).  ``checkpoints`` (gated_linear_recurrence_checkpoints) is
    filled for the backward call.  With ``out`` None a new tensor is returned,
    whose rows outside the sequences (or in skipped ones) are undefined.
    """
    if x.dim() != 2 or decay.dim() != 1:
        raise ValueError("x, gate_a, gate_x [dim, total_T], decay [dim]")
    if out is None:
        out = torch.empty_like(x)
    dim, total_T = x.shape
    _one_device(x, gate_a, gate_x, decay, states, query_start_loc, cache_indices,
                has_initial_state, out, checkpoints)
    dt = _same_type(x, "x, the gates and out", gate_a, gate_x, out)
    batch, hi = _packing(query_start_loc, cache_indices, has_initial_state)
    _dense(decay, torch.float32, "decay", dim)
    pool, slots, slot_stride = _pool(states, dim, "states")
    rows = _checkpoint_rows(checkpoints, dim) if checkpoints is not None else 0
    pl = _planes(x.shape, x, gate_a, gate_x, out)
    ws, n = (_recurrence_workspace(total_T, batch, dim, False, x) if pl[1] == 1
             else (None, 0))  # only rows of tokens use one
    _call("gated_linear_recurrence_varlen_fwd", x, *pl[:9], decay.data_ptr(), decay_scale, pool,
          slots, slot_stride, query_start_loc.data_ptr(), batch, _ptr(cache_indices), _ptr(hi),
          *pl[9:], _ptr(checkpoints), rows, _ptr(ws), n, dim, total_T, dt, int(pad_slot_id))
    return out


def gated_linear_recurrence_varlen_bwd(dout: torch.Tensor, x: torch.Tensor, gate_a: torch.Tensor,
                                       gate_x: torch.Tensor, decay: torch.Tensor,
                                       checkpoints: torch.Tensor, query_start_loc: torch.Tensor,
                                       cache_indices: Optional[torch.Tensor] = None,
                                       has_initial_state: Optional[torch.Tensor] = None,
                                       decay_scale: float = 8.0, pad_slot_id: int = -1,
                                       dfinal_states: Optional[torch.Tensor] = None,
                                       dinitial_states: Optional[torch.Tensor] = None,
                                       dx: Optional[torch.Tensor] = None,
                                       dgate_a: Optional[torch.Tensor] = None,
                                       dgate_x: Optional[torch.Tensor] = None):
    """Gradients of gated_linear_recurrence_varlen_fwd: (dx, dgate_a, dgate_x,
    ddecay).  ``checkpoints`` is what the forward call left; the other inputs
    are the forward's.  dfinal_states / dinitial_states float32 [num_slots,
    dim]: gradient of each sequence's last state (read) and of its initial
    state (written).  Gradients made here are undefined at tokens outside the
    sequences (or in skipped ones)."""
    if x.dim() != 2 or decay.dim() != 1:
        raise ValueError("dout, x, gate_a, gate_x [dim, total_T], decay [dim]")
    dim, total_T = x.shape
    dx = torch.empty_like(x) if dx is None else dx
    dgate_a = torch.empty_like(gate_a) if dgate_a is None else dgate_a
    dgate_x = torch.empty_like(gate_x) if dgate_x is None else dgate_x
    _one_device(x, dout, gate_a, gate_x, decay, checkpoints, query_start_loc, cache_indices,
                has_initial_state, dfinal_states, dinitial_states, dx, dgate_a, dgate_x)
    dt = _same_type(x, "dout, x, the gates and their gradients", dout, gate_a, gate_x, dx, dgate_a,
                    dgate_x)
    batch, hi = _packing(query_start_loc, cache_indices, has_initial_state)
    _dense(decay, torch.float32, "decay", dim)
    dfinal, slots, df_stride = _pool(dfinal_states, dim, "dfinal_states")
    dinitial, di_slots, di_stride = _pool(dinitial_states, dim, "dinitial_states")
    if slots and di_slots and slots != di_slots:
        raise ValueError("dfinal_states and dinitial_states must have one shape")
    rows = _checkpoint_rows(checkpoints, dim)
    pl = _planes(x.shape, dout, x, gate_a, gate_x, dx, dgate_a, dgate_x)
    ddecay = torch.empty(dim, dtype=torch.float32, device=x.device)
    ws, n = _recurrence_workspace(total_T, batch, dim, True, x)
    _call("gated_linear_recurrence_varlen_bwd", x, *pl[:12], decay.data_ptr(), decay_scale,
          checkpoints.data_ptr(), rows, query_start_loc.data_ptr(), batch, _ptr(cache_indices),
          _ptr(hi), slots or di_slots, dfinal, df_stride, dinitial, di_stride, *pl[12:],
          ddecay.data_ptr(), _ptr(ws), n, dim, total_T, dt, int(pad_slot_id))
    return dx, dgate_a, dgate_x, ddecay


def gated_linear_recurrence_update(x: torch.Tensor, gate_a: torch.Tensor, gate_x: torch.Tensor,
                                   decay: torch.Tensor, states: torch.Tensor,
                                   state_indices: Optional[torch.Tensor] = None,
                                   decay_scale: float = 8.0, pad_slot_id: int = -1,
                                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode token per row: x, gate_a, gate_x [batch, dim]; states
    float32 [num_slots, dim] updated in place.  With ``out`` None a new tensor
    is returned, whose skipped rows are undefined."""
    if x.dim() != 2 or decay.dim() != 1:
        raise ValueError("x, gate_a, gate_x [batch, dim], decay [dim]")
    if out is None:
        out = torch.empty_like(x)
    batch, dim = x.shape
    _one_device(x, gate_a, gate_x, decay, states, state_indices, out)
    dt = _same_type(x, "x, the gates and out", gate_a, gate_x, out)
    rows = _rows(x.shape, x, gate_a, gate_x, out)
    _dense(decay, torch.float32, "decay", dim)
    pool, slots, slot_stride = _pool(states, dim, "states")
    if state_indices is not None:
        _dense(state_indices, torch.int32, "state_indices", batch)
    _call("gated_linear_recurrence_update", x, *rows[:6], decay.data_ptr(), decay_scale, pool,
          slots, slot_stride, _ptr(state_indices), *rows[6:], batch, dim, dt, int(pad_slot_id))
    return out


def causal_conv1d_varlen_bwd(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                             bias: Optional[torch.Tensor], initial_states: Optional[torch.Tensor],
                             query_start_loc: torch.Tensor,
                             cache_indices: Optional[torch.Tensor],
                             has_initial_state: Optional[torch.Tensor], silu_activation: bool,
                             pad_slot_id: int = -1,
                             dfinal_states: Optional[torch.Tensor] = None,
                             dinitial_states: Optional[torch.Tensor] = None,
                             dx: Optional[torch.Tensor] = None):
    """Gradients of causal_conv1d_varlen_fwd: (dx, dweight float32 [dim, W],
    dbias float32 [dim] or None).  dout, x [dim, total_T] (x as it was before
    the forward call, which may run in place); initial_states [num_slots, dim,
    W-1]: the state pool before the forward call.  dfinal_states /
    dinitial_states, same shape: gradient of the state that the forward left
    (read) and of the initial state (written).  A dx made here is undefined at
    tokens outside the sequences (or in skipped ones)."""
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("dout, x [dim, total_T], weight [dim, W]")
    dim, total_T = x.shape
    W = weight.shape[1]
    dx = torch.empty_like(x) if dx is None else dx
    pools = (initial_states, dfinal_states, dinitial_states)
    _one_device(x, dout, weight, bias, query_start_loc, cache_indices, has_initial_state, dx,
                *pools)
    dt = _same_type(x, "dout, x, weight, bias, the states and dx", dout, weight, bias, dx, *pools)
    if weight.shape[0] != dim:
        raise ValueError("weight must be [dim, W]")
    if bias is not None:
        _dense(bias, x.dtype, "bias", dim)
    batch, hi = _packing(query_start_loc, cache_indices, has_initial_state)
    slots, pool_args = 0, []
    for t in pools:
        if t is None:
            pool_args.append((None, 0, 0, 0))
            continue
        shape = t.shape
        if len(shape) != 3 or shape[1] != dim or shape[2] != W - 1:
            raise ValueError("states and their gradients must be [num_slots, dim, W-1]")
        if slots and shape[0] != slots:
            raise ValueError("states and their gradients must have one number of slots")
        slots = shape[0]
        pool_args.append((t.data_ptr(), *t.stride()))
    pl = _planes(x.shape, dout, x, dx)
    dweight = torch.empty(dim, W, dtype=torch.float32, device=x.device)
    dbias = torch.empty(dim, dtype=torch.float32, device=x.device) if bias is not None else None
    n = _floats("causal_conv1d_varlen_bwd_workspace", total_T, batch, dim, W)
    ws = torch.empty(n, dtype=torch.float32, device=x.device)
    _call("causal_conv1d_varlen_bwd", x, *pl[:6], weight.data_ptr(), weight.stride(0),
          weight.stride(1), _ptr(bias), *pool_args[0], slots, query_start_loc.data_ptr(), batch,
          _ptr(cache_indices), _ptr(hi), *pool_args[1], *pool_args[2], *pl[6:],
          dweight.data_ptr(), _ptr(dbias), ws.data_ptr(), n, dim, total_T, W, dt,
          _lib.ACT_SILU if silu_activation else _lib.ACT_NONE, int(pad_slot_id))
    return dx, dweight, dbias


def _norm(x, weight, eps, residual, residual_out, out, scales, group_size, out_dt):
    if x.dim() != 2 or weight.dim() != 1:
        raise ValueError("x [rows, dim], weight [dim]")
    rows, dim = x.shape
    if residual is not None and residual_out is None:
        residual_out = residual
    _one_device(x, weight, residual, residual_out, out, scales)
    dt = _same_type(x, "x, weight, residual and residual_out", weight, residual, residual_out)
    _dense(weight, x.dtype, "weight", dim)
    a = _rows(x.shape, x, residual, residual_out, out)
    _call("rms_norm_fwd", x, *a[:4], weight.data_ptr(), eps, *a[4:], _ptr(scales),
          scales.stride(0) if scales is not None else 0, group_size, rows, dim, dt,
          dt if out_dt is None else out_dt)


def rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: Optional[torch.Tensor] = None,
                 residual_out: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """s / sqrt(mean(s^2) + eps) * weight over rows, s = x + residual.

    x, residual [rows, dim], weight [dim].  The sum goes to ``residual_out``,
    or back to residual if that is None (in place, as a layer's stream does).
    """
    if out is None:
        out = torch.empty_like(x)
    if out.dtype != x.dtype:
        raise TypeError("x and out must share one element type")
    _norm(x, weight, eps, residual, residual_out, out, None, 0, None)
    return out


def rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, group_size: int = 0,
                   residual: Optional[torch.Tensor] = None,
                   residual_out: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """rms_norm_fwd with an 8-bit output: (codes float8_e4m3fn [rows, dim],
    scales float32 [rows, dim / group_size]).  group_size 32, 64, 128 or 256
    channels share a scale; 0: a whole row does ([rows, 1])."""
    if x.dim() != 2:
        raise ValueError("x [rows, dim]")
    rows, dim = x.shape
    if group_size < 0 or (group_size and dim % group_size):
        raise ValueError(f"group_size {group_size} does not divide dim {dim}")
    n = dim // group_size if group_size else 1
    if out is None:
        out = torch.empty(rows, dim, dtype=torch.float8_e4m3fn, device=x.device)
    if scales is None:
        scales = torch.empty(rows, n, dtype=torch.float32, device=x.device)
    if out.dtype != torch.float8_e4m3fn or scales.dtype != torch.float32:
        raise TypeError("codes are float8_e4m3fn, scales float32")
    if scales.shape != (rows, n) or (n > 1 and scales.stride(1) != 1):
        raise ValueError("scales must be [rows, groups] with contiguous groups")
    _norm(x, weight, eps, residual, residual_out, out, scales, int(group_size), _lib.E4M3)
    return out, scales


def rms_norm_bwd(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 dresidual: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None):
    """Gradients of rms_norm_fwd at the rows x that it normalised (its
    residual_out, or its x): (dx, dweight float32 [dim]).  ``dresidual``, the
    gradient that reaches residual_out from elsewhere, is added to dx, which
    is then the gradient of x and of residual."""
    if x.dim() != 2 or weight.dim() != 1:
        raise ValueError("dout, x [rows, dim], weight [dim]")
    rows, dim = x.shape
    dx = torch.empty_like(x) if dx is None else dx
    _one_device(x, dout, weight, dresidual, dx)
    dt = _same_type(x, "dout, x, weight, dresidual and dx", dout, weight, dresidual, dx)
    _dense(weight, x.dtype, "weight", dim)
    a = _rows(x.shape, dout, x, dresidual, dx)
    n = _floats("rms_norm_bwd_workspace", rows, dim)
    dweight = torch.empty(dim, dtype=torch.float32, device=x.device)
    ws = torch.empty(n, dtype=torch.float32, device=x.device)
    _call("rms_norm_bwd", x, *a[:4], weight.data_ptr(), eps, *a[4:], dweight.data_ptr(),
          ws.data_ptr(), n, rows, dim, dt)
    return dx, dweight


# ---------------------------------------------------------------- gated delta rule

def _heads(shape, what: str, *ts):
    """[ptr, stride_t, stride_h] of each [tokens, heads, channels] tensor."""
    args = []
    wide = shape[2] > 1
    for t in ts:
        stride = t.stride()
        if t.shape != shape or (wide and stride[2] != 1):
            raise ValueError(f"{what} must be {list(shape)} with contiguous channels")
        args += (t.data_ptr(), stride[0], stride[1])
    return args


def _delta(q, k, v, g, beta):
    """(pointers and strides of the inputs, sizes, types) after checks."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k [tokens, key_heads, K], v [tokens, value_heads, V]")
    tokens, key_heads, K = q.shape
    _, value_heads, V = v.shape
    dt = _same_type(q, "q, k, v and out", k, v)
    if g.dtype != beta.dtype or g.dtype not in (torch.float32, q.dtype):
        raise TypeError("g and beta must both be float32 or of the inputs' type")
    if g.shape != (tokens, value_heads) or beta.shape != g.shape or v.shape[0] != tokens:
        raise ValueError("g and beta must be [tokens, value_heads], as v is")
    args = _heads(q.shape, "q and k", q, k) + _heads(v.shape, "v", v)
    for t in (g, beta):
        args += (t.data_ptr(), *t.stride())
    return args, (key_heads, value_heads, K, V, dt, _DT[g.dtype])


def _matrix_pool(t: Optional[torch.Tensor], heads: int, K: int, V: int, name: str):
    """(ptr, slots, slot stride) of an fp32 [num_slots, heads, K, V] state pool."""
    if t is None:
        return None, 0, 0
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.dim() != 4 or t.shape[1:] != (heads, K, V):
        raise ValueError(f"{name} must be [num_slots, value_heads, K, V]")
    stride = t.stride()
    if stride[1:] != (K * V, V, 1) and t.shape[0] and not t[0].is_contiguous():
        raise ValueError(f"{name} needs dense slots")
    return t.data_ptr(), t.shape[0], stride[0]


def _sixteens(n: int) -> int:
    return -(-n // 16) * 16


def _delta_marks(t: Optional[torch.Tensor], heads: int, K: int, V: int):
    if t is None:
        return 0
    if t.dtype != torch.float32 or t.dim() != 4 or not t.is_contiguous() \
            or t.shape[1:] != (heads, _sixteens(K), _sixteens(V)):
        raise ValueError("checkpoints must be what gated_delta_rule_checkpoints makes")
    return t.shape[0]


def _delta_workspace(tokens: int, batch: int, sizes, backward: bool, x: torch.Tensor):
    """(tensor, floats) of workspace for one packed call."""
    fwd = ctypes.c_int64()
    bwd = _floats("gated_delta_rule_workspace", tokens, batch, *sizes[1:5], ctypes.byref(fwd))
    n = bwd if backward else fwd.value
    return torch.empty(n, dtype=torch.float32, device=x.device), n


def _delta_scale(scale: Optional[float], K: int) -> float:
    return (K ** -0.5 if K else 1.0) if scale is None else float(scale)


def gated_delta_rule_checkpoints(k: torch.Tensor, v: torch.Tensor, query_start_loc: torch.Tensor
                                 ) -> torch.Tensor:
    """The buffer in which gated_delta_rule_varlen_fwd leaves what its backward
    call needs, for inputs like k [total_T, key_heads, K] and v [total_T,
    value_heads, V]."""
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError("k [total_T, key_heads, K], v [total_T, value_heads, V]")
    rows = _floats("gated_delta_rule_checkpoint_rows", v.shape[0], query_start_loc.numel() - 1,
                   _dtype(v))
    return torch.empty(rows, v.shape[1], _sixteens(k.shape[2]), _sixteens(v.shape[2]),
                       dtype=torch.float32, device=v.device)


def gated_delta_rule_varlen_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                g: torch.Tensor, beta: torch.Tensor,
                                states: Optional[torch.Tensor], query_start_loc: torch.Tensor,
                                cache_indices: Optional[torch.Tensor] = None,
                                has_initial_state: Optional[torch.Tensor] = None,
                                scale: Optional[float] = None, pad_slot_id: int = -1,
                                out: Optional[torch.Tensor] = None,
                                checkpoints: Optional[torch.Tensor] = None) -> torch.Tensor:
    """S' = exp(g) S, u = beta (v - S'^T k), S = S' + k u^T, out = scale S^T q
    over packed sequences, a K x V state for each value head.

    q, k [total_T, key_heads, K], v [total_T, value_heads, V], g, beta
    [total_T, value_heads] (float32 or the inputs' type); key head kh serves
    value_heads / key_heads value heads.  states float32 [num_slots,
    value_heads, K, V] is updated in place (None: start at zero, keep nothing).
    scale: None is K ** -0.5.  ``checkpoints`` (gated_delta_rule_checkpoints)
    is filled for the backward call.  With ``out`` None a new tensor is
    returned, whose rows outside the sequences (or in skipped ones) are
    undefined."""
    _one_device(q, k, v, g, beta, states, query_start_loc, cache_indices, has_initial_state, out,
                checkpoints)
    args, sizes = _delta(q, k, v, g, beta)
    _, heads, K, V, _, _ = sizes
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    _same_type(v, "q, k, v and out", out)
    batch, hi = _packing(query_start_loc, cache_indices, has_initial_state)
    pool = _matrix_pool(states, heads, K, V, "states")
    rows = _delta_marks(checkpoints, heads, K, V)
    tokens = v.shape[0]
    ws, n = _delta_workspace(tokens, batch, sizes, False, v)
    _call("gated_delta_rule_varlen_fwd", v, *args, _delta_scale(scale, K), *pool,
          query_start_loc.data_ptr(), batch, _ptr(cache_indices), _ptr(hi),
          *_heads(v.shape, "out", out), _ptr(checkpoints), rows, ws.data_ptr(), n, tokens, *sizes,
          int(pad_slot_id))
    return out


def gated_delta_rule_varlen_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                                v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                                checkpoints: torch.Tensor, query_start_loc: torch.Tensor,
                                cache_indices: Optional[torch.Tensor] = None,
                                has_initial_state: Optional[torch.Tensor] = None,
                                scale: Optional[float] = None, pad_slot_id: int = -1,
                                dfinal_states: Optional[torch.Tensor] = None,
                                dinitial_states: Optional[torch.Tensor] = None,
                                dq: Optional[torch.Tensor] = None,
                                dk: Optional[torch.Tensor] = None,
                                dv: Optional[torch.Tensor] = None):
    """Gradients of gated_delta_rule_varlen_fwd: (dq, dk, dv, dg, dbeta), dq
    and dk summed over the value heads of a key head.  ``checkpoints`` is what
    the forward call left; the other inputs are the forward's.  dfinal_states /
    dinitial_states float32 [num_slots, value_heads, K, V]: gradient of each
    sequence's last state (read) and of its initial state (written).  Gradients
    made here are undefined at tokens outside the sequences (or in skipped
    ones)."""
    _one_device(v, dout, q, k, g, beta, checkpoints, query_start_loc, cache_indices,
                has_initial_state, dfinal_states, dinitial_states, dq, dk, dv)
    args, sizes = _delta(q, k, v, g, beta)
    _, heads, K, V, _, _ = sizes
    new = lambda t: torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
    dq = new(q) if dq is None else dq
    dk = new(k) if dk is None else dk
    dv = new(v) if dv is None else dv
    dg, dbeta = new(g), new(beta)
    _same_type(v, "q, k, v, dout and their gradients", dout, dq, dk, dv)
    batch, hi = _packing(query_start_loc, cache_indices, has_initial_state)
    dfinal, slots, df_stride = _matrix_pool(dfinal_states, heads, K, V, "dfinal_states")
    dinitial, di_slots, di_stride = _matrix_pool(dinitial_states, heads, K, V, "dinitial_states")
    if slots and di_slots and slots != di_slots:
        raise ValueError("dfinal_states and dinitial_states must have one shape")
    rows = _delta_marks(checkpoints, heads, K, V)
    tokens = v.shape[0]
    ws, n = _delta_workspace(tokens, batch, sizes, True, v)
    _call("gated_delta_rule_varlen_bwd", v, *_heads(v.shape, "dout", dout), *args,
          _delta_scale(scale, K), checkpoints.data_ptr(), rows, query_start_loc.data_ptr(), batch,
          _ptr(cache_indices), _ptr(hi), slots or di_slots, dfinal, df_stride, dinitial, di_stride,
          *_heads(q.shape, "dq and dk", dq, dk), *_heads(v.shape, "dv", dv), dg.data_ptr(),
          *dg.stride(), dbeta.data_ptr(), *dbeta.stride(), ws.data_ptr(), n, tokens, *sizes,
          int(pad_slot_id))
    return dq, dk, dv, dg, dbeta


def gated_delta_rule_update(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                            beta: torch.Tensor, states: torch.Tensor,
                            state_indices: Optional[torch.Tensor] = None,
                            scale: Optional[float] = None, pad_slot_id: int = -1,
                            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode token per row: q, k [batch, key_heads, K], v [batch,
    value_heads, V], g, beta [batch, value_heads]; states float32 [num_slots,
    value_heads, K, V] updated in place.  scale: None is K ** -0.5.  With
    ``out`` None a new tensor is returned, whose skipped rows are undefined."""
    _one_device(q, k, v, g, beta, states, state_indices, out)
    args, sizes = _delta(q, k, v, g, beta)
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    _same_type(v, "q, k, v and out", out)
    pool = _matrix_pool(states, *sizes[1:4], "states")
    batch = v.shape[0]
    if state_indices is not None:
        _dense(state_indices, torch.int32, "state_indices", batch)
    _call("gated_delta_rule_update", v, *args, _delta_scale(scale, sizes[2]), *pool,
          _ptr(state_indices), *_heads(v.shape, "out", out), batch, *sizes, int(pad_slot_id))
    return out


# ---------------------------------------------------------------- layer norm

def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   eps: float = 1e-5, residual: Optional[torch.Tensor] = None,
                   residual_out: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """(s - mean(s)) / sqrt(var(s) + eps) * weight + bias over rows, s = x +
    residual.

    x, residual [rows, dim], weight, bias [dim].  The sum goes to
    ``residual_out``, or back to residual if that is None (in place, as a
    layer's stream does).
    """
    if x.dim() != 2 or weight.dim() != 1:
        raise ValueError("x [rows, dim], weight, bias [dim]")
    rows, dim = x.shape
    if out is None:
        out = torch.empty_like(x)
    if residual is not None and residual_out is None:
        residual_out = residual
    _one_device(x, weight, bias, residual, residual_out, out)
    dt = _same_type(x, "x, weight, bias, residual, residual_out and out", weight, bias, residual,
                    residual_out, out)
    _dense(weight, x.dtype, "weight", dim)
    if bias is not None:
        _dense(bias, x.dtype, "bias", dim)
    a = _rows(x.shape, x, residual, residual_out, out)
    _call("layer_norm_fwd", x, *a[:4], weight.data_ptr(), _ptr(bias), eps, *a[4:], rows, dim, dt)
    return out


def layer_norm_bwd(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5,
                   dresidual: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None):
    """Gradients of layer_norm_fwd at the rows x that it normalised (its
    residual_out, or its x): (dx, dweight float32 [dim], dbias float32 [dim]).
    ``dresidual``, the gradient that reaches residual_out from elsewhere, is
    added to dx, which is then the gradient of x and of residual."""
    if x.dim() != 2 or weight.dim() != 1:
        raise ValueError("dout, x [rows, dim], weight [dim]")
    rows, dim = x.shape
    dx = torch.empty_like(x) if dx is None else dx
    _one_device(x, dout, weight, dresidual, dx)
    dt = _same_type(x, "dout, x, weight, dresidual and dx", dout, weight, dresidual, dx)
    _dense(weight, x.dtype, "weight", dim)
    a = _rows(x.shape, dout, x, dresidual, dx)
    n = _floats("layer_norm_bwd_workspace", rows, dim)
    dweight, dbias = (torch.empty(dim, dtype=torch.float32, device=x.device) for _ in range(2))
    ws = torch.empty(n, dtype=torch.float32, device=x.device)
    _call("layer_norm_bwd", x, *a[:4], weight.data_ptr(), eps, *a[4:], dweight.data_ptr(),
          dbias.data_ptr(), ws.data_ptr(), n, rows, dim, dt)
    return dx, dweight, dbias


# ---------------------------------------------------------------- a step's paged metadata

def sconv_paged_metadata(query_lens: torch.Tensor, context_lens: torch.Tensor,
                         free_blocks: torch.Tensor, block_table: torch.Tensor, block_size: int,
                         query_start_loc: torch.Tensor, seq_idx_out: Optional[torch.Tensor],
                         query_start_out: Optional[torch.Tensor], positions_out: torch.Tensor,
                         slot_mapping_out: torch.Tensor,
                         blocks_used: Optional[torch.Tensor] = None) -> None:
    """Fill a step's static metadata buffers from its requests' lengths.

    query_lens, context_lens int32 [num_reqs]: tokens of this step, and tokens
    before it.  Blocks that a request's row of block_table (int32 [num_reqs,
    max_blocks], updated in place) lacks come from free_blocks (int32), in the
    order of the requests; blocks_used int32 [1] says how many they need.
    query_start_loc int32 [num_reqs + 1], seq_idx_out, query_start_out int32
    and positions_out, slot_mapping_out int64, all of one length (the padded
    token count), are written; seq_idx_out and query_start_out may be None.
    Rows behind the last token have slot -1 and zeros elsewhere; where
    free_blocks or a table's row ends, slots are -1."""
    _one_device(query_lens, context_lens, free_blocks, block_table, query_start_loc, seq_idx_out,
                query_start_out, positions_out, slot_mapping_out, blocks_used)
    reqs, padded = query_lens.numel(), slot_mapping_out.numel()
    _dense(query_lens, torch.int32, "query_lens")
    _dense(context_lens, torch.int32, "context_lens", reqs)
    _dense(free_blocks, torch.int32, "free_blocks")
    _dense(query_start_loc, torch.int32, "query_start_loc", reqs + 1)
    _dense(positions_out, torch.int64, "positions_out", padded)
    _dense(slot_mapping_out, torch.int64, "slot_mapping_out", padded)
    for t, name, n in ((seq_idx_out, "seq_idx_out", padded),
                       (query_start_out, "query_start_out", padded),
                       (blocks_used, "blocks_used", 1)):
        if t is not None:
            _dense(t, torch.int32, name, n)
    if block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise TypeError("block_table must be int32 [num_reqs, max_blocks]")
    max_blocks = block_table.shape[1]
    if max_blocks > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table needs contiguous entries within a row")
    _table_rows(block_table, reqs)
    _call("sconv_paged_metadata", slot_mapping_out, query_lens.data_ptr(), context_lens.data_ptr(),
          reqs, free_blocks.data_ptr(), free_blocks.numel(), block_table.data_ptr(),
          block_table.stride(0), max_blocks, int(block_size), query_start_loc.data_ptr(), padded,
          _ptr(seq_idx_out), _ptr(query_start_out), positions_out.data_ptr(),
          slot_mapping_out.data_ptr(), _ptr(blocks_used))
