"""Torch-tensor front end over the libep C ABI.

Mirrors the Buffer methods of the "DeepEP-Ascend" README ("API Overview":
get_dispatch_layout, dispatch, combine, low_latency_dispatch /
low_latency_combine) and the expert-centric calls asked for in "[Feature
Request] Support Expert-Choice Routing via Native Expert-Centric API"
(Solution 1: dispatch_expert_choice with token_indices [E, C] and weights).
In front of them, the router that makes topk_idx and topk_weights, with its
balance loss and gradients (route, balance_loss, route_backward); and, over
the same topk_idx, low-rank adapters beside a shared projection
(adapter_project and its backward).  Between dispatch and combine, the experts:
their weights in MXFP4 (mx_quantize), the products on the dispatched rows
(expert_product and its backward), and for a few tokens the whole layer in one
call (low_latency_experts).

torch only allocates device memory and supplies the current stream; every
step runs in the HIP kernels of libep.so.  Errors from the library raise
EpError (a ValueError).
"""
from __future__ import annotations

import contextlib
import functools
from dataclasses import dataclass
from typing import List, Optional

import torch

from . import _native as N


# The current stream's handle without a Stream object around it, where torch
# offers it: 0.1 us instead of 1.9 us a call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev: torch.device) -> int:
    if _raw_stream is not None and dev.index is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


_HERE = contextlib.nullcontext()


def _on(dev: torch.device):
    """Makes dev the current device, if it is another one."""
    return _HERE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _same_device(dev: torch.device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other operands on {dev}")


def _out(out: Optional[torch.Tensor], shape, dev: torch.device) -> torch.Tensor:
    """A caller's output tensor, checked before the kernel writes shape[0] rows
    into it, or a new one."""
    if out is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must be {tuple(shape)}, got {tuple(out.shape)}")
    _same_device(dev, out=out)
    return out


@dataclass
class Layout:
    """Result of get_dispatch_layout.  The workspace carries per-chunk tables
    to the dispatch that follows and must not be reused before it."""
    num_tokens_per_rank: torch.Tensor          # [R] int32
    num_tokens_per_rdma_rank: None             # needs a node topology: not produced
    num_tokens_per_expert: torch.Tensor        # [E] int32 (count form)
    is_token_in_rank: torch.Tensor             # [T, R] uint8
    offsets: torch.Tensor                      # [E+1] int32 (prefix-sum form)
    num_invalid: torch.Tensor                  # [1] int32
    topk_idx: torch.Tensor
    num_experts: int
    num_ranks: int
    workspace: torch.Tensor


@dataclass
class Handle:
    """What combine needs from dispatch: the receive row of every (t, k)."""
    slot: torch.Tensor                         # [T, K] int32, -1 = not received
    recv_src: torch.Tensor                     # [rows] int32, source token of each written row
    num_dropped: torch.Tensor                  # [1] int32
    rows: int
    recv_layout: str
    cap: Optional[int]
    recv_count: Optional[torch.Tensor] = None  # [E] int32, rows each expert holds (low latency)
    num_invalid: Optional[torch.Tensor] = None  # [1] int32 (low latency)


@dataclass
class ExpertChoiceHandle:
    tok_off: torch.Tensor                      # [T+1] int32
    tok_ent: torch.Tensor                      # [E*C] int32
    weights: torch.Tensor                      # [E, C] float32
    num_invalid: torch.Tensor                  # [1] int32
    num_tokens: int


def get_dispatch_layout(topk_idx: torch.Tensor, num_experts: int, num_ranks: int = 1) -> Layout:
    _need(topk_idx, "topk_idx", torch.int32, 2)
    T, K = topk_idx.shape
    E, R = int(num_experts), int(num_ranks)
    dev = topk_idx.device
    ws_bytes = N.ep_workspace_bytes(T, K, E, R)
    if ws_bytes == 0:
        raise N.EpError("ep_workspace_bytes", N.EP_ERR_INVALID_ARG)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    tpr = torch.empty(R, dtype=torch.int32, device=dev)
    itr = torch.empty((T, R), dtype=torch.uint8, device=dev)
    ninv = torch.empty(1, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        N.ep_get_dispatch_layout(_ptr(topk_idx), T, K, E, R, _ptr(counts), _ptr(offsets),
                                 _ptr(tpr), _ptr(itr), _ptr(ninv), _ptr(ws), ws_bytes,
                                 _stream(dev))
    return Layout(tpr, None, counts, itr, offsets, ninv, topk_idx, E, R, ws)


def get_dispatch_layout_rounds(topk_idx: torch.Tensor, num_experts: int, round_tokens: int,
                               num_ranks: int = 1) -> List[Layout]:
    """The layouts of rounds of at most `round_tokens` tokens ("DeepSeek-V4
    昇腾 NPU 推理部署实践", custom_params: moe_chunk_max_len), all from one
    call: round r's Layout equals get_dispatch_layout(topk_idx[r*rt:(r+1)*rt])
    and carries its own slice of the shared workspace for that round's
    dispatch."""
    _need(topk_idx, "topk_idx", torch.int32, 2)
    if round_tokens < 1:
        raise ValueError("round_tokens must be >= 1")
    T, K = topk_idx.shape
    E, R = int(num_experts), int(num_ranks)
    dev = topk_idx.device
    ws_bytes = N.ep_workspace_bytes_rounds(T, K, E, R, round_tokens)
    if ws_bytes == 0:
        raise N.EpError("ep_workspace_bytes_rounds", N.EP_ERR_INVALID_ARG)
    rt = min(round_tokens, T)
    nr = (T + rt - 1) // rt if T else 0
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    counts = torch.empty((max(nr, 1), E), dtype=torch.int32, device=dev)
    offsets = torch.empty((max(nr, 1), E + 1), dtype=torch.int32, device=dev)
    tpr = torch.empty((max(nr, 1), R), dtype=torch.int32, device=dev)
    itr = torch.empty((T, R), dtype=torch.uint8, device=dev)
    ninv = torch.empty(max(nr, 1), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        N.ep_get_dispatch_layout_rounds(_ptr(topk_idx), T, K, E, R, round_tokens, _ptr(counts),
                                        _ptr(offsets), _ptr(tpr), _ptr(itr), _ptr(ninv),
                                        _ptr(ws), ws_bytes, _stream(dev))
    stride = N.ep_workspace_bytes(rt, K, E, R) if nr else 0
    out = []
    for r in range(nr):
        t0, t1 = r * rt, min(T, (r + 1) * rt)
        b = N.ep_workspace_bytes(t1 - t0, K, E, R)
        out.append(Layout(tpr[r], None, counts[r], itr[t0:t1], offsets[r], ninv[r:r + 1],
                          topk_idx[t0:t1], E, R, ws[stride * r:stride * r + b]))
    return out


# quant name -> (ep_quant_t, receive dtype, H divisor of a receive row,
# scale shape: H -> (columns or 0 for one per row, dtype), or None)
_QUANT = {
    "bf16": (N.EP_QUANT_BF16, torch.bfloat16, 1, None),
    "fp8_e4m3_g128": (N.EP_QUANT_FP8_E4M3_G128, torch.float8_e4m3fn, 1,
                      lambda H: (H // 128, torch.float32)),
    "fp8_e4m3_token": (N.EP_QUANT_FP8_E4M3_TOKEN, torch.float8_e4m3fn, 1,
                       lambda H: (0, torch.float32)),
    "int8_token": (N.EP_QUANT_INT8_TOKEN, torch.int8, 1, lambda H: (0, torch.float32)),
    "mxfp8_e4m3": (N.EP_QUANT_MXFP8_E4M3, torch.float8_e4m3fn, 1, lambda H: (H // 32, torch.uint8)),
    "mxfp8_e5m2": (N.EP_QUANT_MXFP8_E5M2, torch.float8_e5m2, 1, lambda H: (H // 32, torch.uint8)),
    "mxfp4_e2m1": (N.EP_QUANT_MXFP4_E2M1, torch.uint8, 2, lambda H: (H // 32, torch.uint8)),
}
_QUANT_ALIASES = {"pertoken_fp8_e4m3": "fp8_e4m3_token", "int8": "int8_token",
                  "mx_fp8_e4m3": "mxfp8_e4m3", "mx_fp8_e5m2": "mxfp8_e5m2",
                  "mx_fp4_e2m1": "mxfp4_e2m1"}


def dispatch(x: torch.Tensor, layout: Layout, *, quant: str = "bf16",
             recv_layout: str = "contiguous", cap: Optional[int] = None,
             max_rows: Optional[int] = None):
    """-> (recv_x, recv_scales or None, Handle).

    recv_layout "contiguous": expert blocks back to back, `max_rows` rows
    (default T*K, always enough).  "padded": [E, cap] rows, the low-latency
    form.  quant (names of the DeepEP-Ascend quantisation modes in
    parentheses):
      "bf16"                                 recv bf16 [rows, H], no scales
      "fp8_e4m3_g128"                        e4m3 [rows, H] + fp32 [rows, H/128]
      "fp8_e4m3_token" ("pertoken_fp8_e4m3") e4m3 [rows, H] + fp32 [rows]
      "int8_token" ("int8")                  int8 [rows, H] + fp32 [rows]
      "mxfp8_e4m3" ("mx_fp8_e4m3")           e4m3 [rows, H] + e8m0 codes uint8 [rows, H/32]
      "mxfp8_e5m2" ("mx_fp8_e5m2")           e5m2 [rows, H] + e8m0 codes uint8 [rows, H/32]
      "mxfp4_e2m1" ("mx_fp4_e2m1")           uint8 [rows, H/2], two e2m1 codes per byte
                                             (low nibble first) + e8m0 uint8 [rows, H/32]"""
    _need(x, "x", torch.bfloat16, 2)
    T, H = x.shape
    idx = layout.topk_idx
    if idx.shape[0] != T:
        raise ValueError("x and topk_idx disagree on the number of tokens")
    K, E = idx.shape[1], layout.num_experts
    quant = _QUANT_ALIASES.get(quant, quant)
    if quant not in _QUANT:
        raise ValueError(f"unknown quant mode {quant!r}")
    q, rdt, row_div, scale_shape = _QUANT[quant]
    if recv_layout == "contiguous":
        lay, arg = N.EP_LAYOUT_CONTIGUOUS, (T * K if max_rows is None else int(max_rows))
        rows = arg
    elif recv_layout == "padded":
        if cap is None:
            raise ValueError("padded layout needs cap")
        lay, arg = N.EP_LAYOUT_PADDED, int(cap)
        rows = E * arg
    else:
        raise ValueError(f"unknown receive layout {recv_layout!r}")
    dev = x.device
    _same_device(dev, topk_idx=idx, workspace=layout.workspace)
    recv = torch.empty((rows, H // row_div), dtype=rdt, device=dev)
    scales = None
    if scale_shape is not None:
        ncol, sdt = scale_shape(H)
        scales = torch.empty((rows, ncol) if ncol else (rows,), dtype=sdt, device=dev)
    slot = torch.empty((T, K), dtype=torch.int32, device=dev)
    src = torch.empty(rows, dtype=torch.int32, device=dev)
    nd = torch.empty(1, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        N.ep_dispatch(_ptr(x), T, H, _ptr(idx), K, E, _ptr(layout.offsets), lay, arg, q,
                      _ptr(recv), _ptr(scales), _ptr(slot), _ptr(src), _ptr(nd),
                      _ptr(layout.workspace), layout.workspace.numel(), _stream(dev))
    return recv, scales, Handle(slot, src, nd, rows, recv_layout, cap if lay else None)


def combine(y: torch.Tensor, handle: Handle, topk_weights: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = bf16(sum_k w[t,k] * y[slot[t,k]]), fp32 sums; w = 1 if None."""
    _need(y, "y", torch.bfloat16, 2)
    T, K = handle.slot.shape
    H = y.shape[1]
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, 2)
        if tuple(topk_weights.shape) != (T, K):
            raise ValueError("topk_weights must be [T, K]")
    dev = y.device
    _same_device(dev, slot=handle.slot, topk_weights=topk_weights)
    out = _out(out, (T, H), dev)
    with torch.cuda.device(dev):
        N.ep_combine(_ptr(y), y.shape[0], H, _ptr(handle.slot), _ptr(topk_weights), T, K,
                     _ptr(out), _stream(dev))
    return out


def low_latency_dispatch(x: torch.Tensor, topk_idx: torch.Tensor,
                         num_max_dispatch_tokens_per_rank: int, num_experts: int, *,
                         quant: str = "fp8_e4m3_g128"):
    """The decode-phase call of "DeepEP-Ascend" README, API Overview
    (low_latency_dispatch(x, topk_idx, num_max_dispatch_tokens_per_rank,
    num_experts)): one launch, no layout call, into the capacity-padded buffer
    of num_max_dispatch_tokens_per_rank rows per expert.  Quantised by default
    (e4m3 with one fp32 scale per 128 channels); quant="bf16" turns it off.
    The same slots, codes and scales as get_dispatch_layout + dispatch with
    recv_layout="padded"; built for decode batches (T*K <= 4096, K <= 64),
    beyond which the library reports the request as unsupported and that pair
    is the call to use.
    -> (recv_x [E, cap, H or H/2], recv_scales [E, cap, ...] or None, Handle);
    the shapes are views of the flat receive rows, and handle.recv_count [E]
    holds the rows each expert received (at most cap)."""
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_idx, "topk_idx", torch.int32, 2)
    T, H = x.shape
    if topk_idx.shape[0] != T:
        raise ValueError("x and topk_idx disagree on the number of tokens")
    K = topk_idx.shape[1]
    E, cap = int(num_experts), int(num_max_dispatch_tokens_per_rank)
    quant = _QUANT_ALIASES.get(quant, quant)
    if quant not in _QUANT:
        raise ValueError(f"unknown quant mode {quant!r}")
    q, rdt, row_div, scale_shape = _QUANT[quant]
    if E < 1 or cap < 0:
        raise ValueError("num_experts must be >= 1 and the capacity >= 0")
    rows = E * cap
    dev = x.device
    _same_device(dev, topk_idx=topk_idx)
    recv = torch.empty((rows, H // row_div), dtype=rdt, device=dev)
    scales = None
    if scale_shape is not None:
        ncol, sdt = scale_shape(H)
        scales = torch.empty((rows, ncol) if ncol else (rows,), dtype=sdt, device=dev)
    slot = torch.empty((T, K), dtype=torch.int32, device=dev)
    src = torch.empty(rows, dtype=torch.int32, device=dev)
    cnt = torch.empty(E, dtype=torch.int32, device=dev)
    nd = torch.empty(1, dtype=torch.int32, device=dev)
    ninv = torch.empty(1, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        N.ep_low_latency_dispatch(_ptr(x), T, H, _ptr(topk_idx), K, E, cap, q, _ptr(recv),
                                  _ptr(scales), _ptr(slot), _ptr(src), _ptr(cnt), _ptr(nd),
                                  _ptr(ninv), _stream(dev))
    recv = recv.view(E, cap, *recv.shape[1:])
    if scales is not None:
        scales = scales.view(E, cap, *scales.shape[1:])
    return recv, scales, Handle(slot, src, nd, rows, "padded", cap, cnt, ninv)


def low_latency_combine(y: torch.Tensor, topk_idx: torch.Tensor,
                        topk_weights: Optional[torch.Tensor], handle: Handle,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The decode-phase combine of "DeepEP-Ascend" README, API Overview
    (low_latency_combine(x, topk_idx, topk_weights, handle)): y holds the
    experts' bf16 rows in the receive layout, [E, cap, H] or [E*cap, H];
    out[t] = bf16(sum_k w[t,k] * y[slot[t,k]]) with fp32 sums.  topk_idx
    must be the one the handle came from (its shape is checked; the slots in
    the handle already encode it)."""
    if y.dim() == 3:
        _need(y, "y", torch.bfloat16, 3)
        y = y.view(-1, y.shape[-1])
    _need(topk_idx, "topk_idx", torch.int32, 2)
    if tuple(topk_idx.shape) != tuple(handle.slot.shape):
        raise ValueError("topk_idx does not match the handle")
    return combine(y, handle, topk_weights, out=out)


def dispatch_combine_chunked(x: torch.Tensor, topk_idx: torch.Tensor, num_experts: int, *,
                             chunk: int, topk_weights: Optional[torch.Tensor] = None,
                             expert=None, quant: str = "bf16", num_ranks: int = 1,
                             keep_rounds: bool = False):
    """Long prefill in rounds of at most `chunk` tokens ("DeepSeek-V4 昇腾
    NPU 推理部署实践", custom_params: moe_chunk_max_len bounds the tokens an
    MoE layer handles at once, against running out of memory on long
    sequences).  One call lays out every round (get_dispatch_layout_rounds);
    each round then runs dispatch, `expert` and combine on its own slice of
    tokens, so a receive buffer holds chunk*K rows instead of T*K.  `expert(recv, scales, layout) -> y` maps the received rows to the
    bf16 rows combine reads (default: identity, bf16 only).  Results equal
    the unchunked call: a token's rows and their order do not depend on the
    other tokens of its round.  -> out [T, H], plus the per-round (layout,
    handle) pairs when keep_rounds is set."""
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_idx, "topk_idx", torch.int32, 2)
    if chunk < 1:
        raise ValueError("chunk must be >= 1")
    if expert is None and quant != "bf16":
        raise ValueError("a quantised dispatch needs an expert that returns bf16 rows")
    T = x.shape[0]
    if topk_idx.shape[0] != T:
        raise ValueError("x and topk_idx disagree on the number of tokens")
    out = torch.empty_like(x)
    rounds = []
    for r, L in enumerate(get_dispatch_layout_rounds(topk_idx, num_experts, chunk, num_ranks)):
        t0 = r * min(chunk, T)
        t1 = t0 + L.topk_idx.shape[0]
        recv, scales, h = dispatch(x[t0:t1], L, quant=quant)
        y = recv if expert is None else expert(recv, scales, L)
        combine(y, h, None if topk_weights is None else topk_weights[t0:t1], out=out[t0:t1])
        if keep_rounds:
            rounds.append((L, h))
    return (out, rounds) if keep_rounds else out


def dispatch_expert_choice(x: torch.Tensor, token_indices: torch.Tensor, weights: torch.Tensor):
    """-> (recv_x [E, C, H], ExpertChoiceHandle).  The weights are kept in the
    handle and applied by combine_expert_choice."""
    _need(x, "x", torch.bfloat16, 2)
    _need(token_indices, "token_indices", torch.int32, 2)
    _need(weights, "weights", torch.float32, 2)
    T, H = x.shape
    E, C = token_indices.shape
    if tuple(weights.shape) != (E, C):
        raise ValueError("weights must be [E, C] like token_indices")
    dev = x.device
    _same_device(dev, token_indices=token_indices, weights=weights)
    ws_bytes = N.ep_ec_workspace_bytes(T, E, C)
    if ws_bytes == 0:
        raise N.EpError("ep_ec_workspace_bytes", N.EP_ERR_INVALID_ARG)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    recv = torch.empty((E, C, H), dtype=torch.bfloat16, device=dev)
    off = torch.empty(T + 1, dtype=torch.int32, device=dev)
    ent = torch.empty(E * C, dtype=torch.int32, device=dev)
    ninv = torch.empty(1, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        N.ep_dispatch_expert_choice(_ptr(x), T, H, _ptr(token_indices), E, C, _ptr(recv),
                                    _ptr(off), _ptr(ent), _ptr(ninv), _ptr(ws), ws_bytes,
                                    _stream(dev))
    return recv, ExpertChoiceHandle(off, ent, weights, ninv, T)


def combine_expert_choice(y: torch.Tensor, handle: ExpertChoiceHandle,
                          out: Optional[torch.Tensor] = None) -> torch.Tensor:
    _need(y, "y", torch.bfloat16, 3)
    E, C, H = y.shape
    T = handle.num_tokens
    if tuple(handle.weights.shape) != (E, C):
        raise ValueError(f"y is [{E}, {C}, H] but the handle's weights are "
                         f"{tuple(handle.weights.shape)}")
    dev = y.device
    _same_device(dev, weights=handle.weights, tok_off=handle.tok_off, tok_ent=handle.tok_ent)
    out = _out(out, (T, H), dev)
    with torch.cuda.device(dev):
        N.ep_combine_expert_choice(_ptr(y), _ptr(handle.weights), E, C, H, _ptr(handle.tok_off),
                                   _ptr(handle.tok_ent), T, _ptr(out), _stream(dev))
    return out


# ---------------------------------------------------------------- one rank's share
@dataclass
class RankPack:
    """What the sender packs ("DeepEP-Ascend" README, API Overview: the
    dispatch sends each token to the ranks of its experts): rows grouped by
    destination rank, each token once per rank that holds one of its
    experts, with that rank's local expert ids."""
    num_tokens_per_rank: torch.Tensor          # [R] int32
    rank_offsets: torch.Tensor                 # [R+1] int32: rank r's rows start here
    send_x: torch.Tensor                       # [rows, H] bf16
    send_src: torch.Tensor                     # [rows] int32: source token
    send_idx: torch.Tensor                     # [rows, K] int32: local expert ids, -1 elsewhere
    send_w: torch.Tensor                       # [rows, K] float32: weights, 0 where send_idx is -1
    pack_pos: torch.Tensor                     # [T, R] int32: row of (t, r) or -1
    num_dropped: torch.Tensor                  # [1] int32
    num_ranks: int
    experts_per_rank: int


def pack_by_rank(x: torch.Tensor, topk_idx: torch.Tensor, num_experts: int, num_ranks: int,
                 topk_weights: Optional[torch.Tensor] = None,
                 max_rows: Optional[int] = None) -> RankPack:
    """The sender's rows for R ranks (rank r owns experts [r E/R, (r+1) E/R)):
    rows ordered by rank, then token.  `max_rows` defaults to T * min(K, R),
    always enough; rows beyond it are dropped and counted."""
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_idx, "topk_idx", torch.int32, 2)
    T, H = x.shape
    if topk_idx.shape[0] != T:
        raise ValueError("x and topk_idx disagree on the number of tokens")
    K = topk_idx.shape[1]
    E, R = int(num_experts), int(num_ranks)
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, 2)
        if tuple(topk_weights.shape) != (T, K):
            raise ValueError("topk_weights must be [T, K]")
    dev = x.device
    _same_device(dev, topk_idx=topk_idx, topk_weights=topk_weights)
    rows = T * min(K, R) if max_rows is None else int(max_rows)
    ws_bytes = N.ep_pack_workspace_bytes(T, K, E, R)
    if ws_bytes == 0:
        raise N.EpError("ep_pack_workspace_bytes", N.EP_ERR_INVALID_ARG)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    tpr = torch.empty(R, dtype=torch.int32, device=dev)
    off = torch.empty(R + 1, dtype=torch.int32, device=dev)
    sx = torch.empty((rows, H), dtype=torch.bfloat16, device=dev)
    src = torch.empty(rows, dtype=torch.int32, device=dev)
    sidx = torch.empty((rows, K), dtype=torch.int32, device=dev)
    sw = torch.empty((rows, K), dtype=torch.float32, device=dev)
    pos = torch.empty((T, R), dtype=torch.int32, device=dev)
    nd = torch.empty(1, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        N.ep_pack_by_rank(_ptr(x), T, H, _ptr(topk_idx), _ptr(topk_weights), K, E, R, rows,
                          _ptr(tpr), _ptr(off), _ptr(sx), _ptr(src), _ptr(sidx), _ptr(sw),
                          _ptr(pos), _ptr(nd), _ptr(ws), ws_bytes, _stream(dev))
    return RankPack(tpr, off, sx, src, sidx, sw, pos, nd, R, E // R)


def receive(recv_x: torch.Tensor, recv_idx: torch.Tensor, experts_per_rank: int, *,
            quant: str = "bf16", max_rows: Optional[int] = None):
    """The receiving rank's scatter of the rows it received (the blocks of
    its source ranks, concatenated in rank order) into its local experts:
    the layout and the stable scatter with the received local ids as
    topk_idx, so an expert's rows are in (source rank, source token, k)
    order.  -> (Layout, recv, recv_scales or None, Handle)."""
    layout = get_dispatch_layout(recv_idx, experts_per_rank)
    recv, scales, handle = dispatch(recv_x, layout, quant=quant, max_rows=max_rows)
    return layout, recv, scales, handle


def combine_partial(y: torch.Tensor, handle: Handle, weights: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The receiving rank's combine: per received row, sum_k w * y[slot] in
    fp32, kept in fp32 for the sender (the partial sums of the exchange)."""
    _need(y, "y", torch.bfloat16, 2)
    S, K = handle.slot.shape
    H = y.shape[1]
    if weights is not None:
        _need(weights, "weights", torch.float32, 2)
        if tuple(weights.shape) != (S, K):
            raise ValueError("weights must be [rows, K]")
    dev = y.device
    _same_device(dev, slot=handle.slot, weights=weights)
    if out is None:
        out = torch.empty((S, H), dtype=torch.float32, device=dev)
    else:
        _need(out, "out", torch.float32, 2)
        if tuple(out.shape) != (S, H):
            raise ValueError(f"out must be {(S, H)}, got {tuple(out.shape)}")
        _same_device(dev, out=out)
    with torch.cuda.device(dev):
        N.ep_combine_partial(_ptr(y), y.shape[0], H, _ptr(handle.slot), _ptr(weights), S, K,
                             _ptr(out), _stream(dev))
    return out


def combine_ranks(partial: torch.Tensor, pack: RankPack,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The sender's sum of the partial rows the ranks returned (at the rows
    their tokens had in send_x), in rank order, rounded once to bf16."""
    _need(partial, "partial", torch.float32, 2)
    T, R = pack.pack_pos.shape
    H = partial.shape[1]
    dev = partial.device
    _same_device(dev, pack_pos=pack.pack_pos)
    out = _out(out, (T, H), dev)
    with torch.cuda.device(dev):
        N.ep_combine_ranks(_ptr(partial), partial.shape[0], H, _ptr(pack.pack_pos), T, R,
                           _ptr(out), _stream(dev))
    return out


# ---------------------------------------------------------------- the router
_SCORES = {"softmax": N.EP_SCORE_SOFTMAX, "sigmoid": N.EP_SCORE_SIGMOID}
_LOGIT_DTYPES = {torch.bfloat16: N.EP_DTYPE_BF16, torch.float32: N.EP_DTYPE_F32}


def _logits_dtype(logits: torch.Tensor, score: str) -> int:
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a tensor")
    if logits.dtype not in _LOGIT_DTYPES:
        raise ValueError(f"logits must be torch.bfloat16 or torch.float32, got {logits.dtype}")
    _need(logits, "logits", logits.dtype, 2)
    if score not in _SCORES:
        raise ValueError(f"unknown score {score!r}")
    return _LOGIT_DTYPES[logits.dtype]


@dataclass
class Routing:
    """Result of route, and what route_backward needs of it.  The logits must
    still hold their values when the backward runs."""
    topk_idx: torch.Tensor                     # [T, K] int32, -1 = nothing left to choose
    topk_weights: torch.Tensor                 # [T, K] float32
    num_invalid: torch.Tensor                  # [T] int32: NaN and +inf logits of each token
    logits: torch.Tensor
    score: str
    renormalise: bool
    scale: float


@dataclass
class BalanceLoss:
    """Result of balance_loss, and what its backward needs of it."""
    loss: torch.Tensor                         # [1] float32
    num_tokens_per_expert: torch.Tensor        # [S, E] int32: entries of topk_idx per sequence
    num_invalid: torch.Tensor                  # [2] int32: bad entries of topk_idx, bad logits
    state: torch.Tensor                        # [S*E + 1] float32: what the gradient needs of the loss
    logits: torch.Tensor
    score: str
    seq_offsets: Optional[torch.Tensor]


def route(logits: torch.Tensor, num_topk: int, *, score: str = "softmax",
          bias: Optional[torch.Tensor] = None, renormalise: bool = True,
          scale: float = 1.0) -> Routing:
    """The router in front of dispatch: each token's num_topk experts with the
    largest scores (descending, ties to the lower expert) and their weights.
    logits: bf16 or fp32 [T, E]; a -inf logit masks its expert, a row of them
    is padding (topk_idx -1).  score: "softmax" or "sigmoid"; with "sigmoid" a
    `bias` [E] (fp32) may be added to the scores for the choice alone.  The
    weights are scale times the scores, renormalised over the chosen experts
    (as workloads.router_topk draws them) or as they are.  Tensors carry no
    autograd graph: the gradient is route_backward."""
    dt = _logits_dtype(logits, score)
    T, E = logits.shape
    K = int(num_topk)
    if bias is not None:
        if score != "sigmoid":
            raise ValueError("a selection bias needs sigmoid scores")
        _need(bias, "bias", torch.float32, 1)
        if bias.shape[0] != E:
            raise ValueError("bias must be [E]")
    if K < 1 or K > E:
        raise ValueError(f"num_topk must be in [1, {E}], got {K}")
    dev = logits.device
    _same_device(dev, bias=bias)
    idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    w = torch.empty((T, K), dtype=torch.float32, device=dev)
    ninv = torch.empty(T, dtype=torch.int32, device=dev)
    with _on(dev):
        N.ep_route(_ptr(logits), dt, T, E, K, _SCORES[score], _ptr(bias), int(renormalise),
                   float(scale), _ptr(idx), _ptr(w), _ptr(ninv), _stream(dev))
    return Routing(idx, w, ninv, logits, score, bool(renormalise), float(scale))


def balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, *, score: str = "softmax",
                 coef: float = 1.0, seq_offsets: Optional[torch.Tensor] = None) -> BalanceLoss:
    """The balance loss of a choice of experts, with their counts:
    coef * mean over the sequences of sum_e f_e P_e, where f_e is the share of
    expert e among the sequence's entries of topk_idx, times E, and P_e its
    mean probability.  seq_offsets: int32 [S+1], non-decreasing (default: all
    tokens are one sequence); tokens outside all sequences take no part.  Its
    gradient is balance_loss_backward, or route_backward with balance=."""
    dt = _logits_dtype(logits, score)
    _need(topk_idx, "topk_idx", torch.int32, 2)
    T, E = logits.shape
    if topk_idx.shape[0] != T:
        raise ValueError("logits and topk_idx disagree on the number of tokens")
    K = topk_idx.shape[1]
    S = 1
    if seq_offsets is not None:
        _need(seq_offsets, "seq_offsets", torch.int32, 1)
        S = seq_offsets.shape[0] - 1
        if S < 1:
            raise ValueError("seq_offsets needs at least two entries")
    dev = logits.device
    _same_device(dev, topk_idx=topk_idx, seq_offsets=seq_offsets)
    ws_bytes = N.ep_balance_workspace_bytes(T, E, S)
    if ws_bytes == 0:
        raise N.EpError("ep_balance_workspace_bytes", N.EP_ERR_INVALID_ARG)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    state = torch.empty(S * E + 1, dtype=torch.float32, device=dev)
    counts = torch.empty((S, E), dtype=torch.int32, device=dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    ninv = torch.empty(2, dtype=torch.int32, device=dev)
    with _on(dev):
        N.ep_balance_loss(_ptr(logits), dt, T, E, _ptr(topk_idx), K, _SCORES[score],
                          _ptr(seq_offsets), S, float(coef), _ptr(counts), _ptr(state),
                          _ptr(loss), _ptr(ninv), _ptr(ws), ws_bytes, _stream(dev))
    return BalanceLoss(loss, counts, ninv, state, logits, score, seq_offsets)


def _router_backward(logits, score, d_w, routing, d_loss, balance):
    T, E = logits.shape
    dev = logits.device
    K, renorm, scale, idx = 1, False, 1.0, None
    if d_w is not None:
        _need(d_w, "d_weights", torch.float32, 2)
        idx, renorm, scale = routing.topk_idx, routing.renormalise, routing.scale
        if tuple(d_w.shape) != tuple(idx.shape):
            raise ValueError("d_weights must be [T, K] like the weights")
        K = idx.shape[1]
    slope, seq, S = None, None, 1
    if balance is not None:
        if d_loss is None:
            raise ValueError("the balance loss's gradient needs d_loss")
        _need(d_loss, "d_loss", torch.float32, 1)
        if d_loss.shape[0] != 1:
            raise ValueError("d_loss must be [1]")
        seq = balance.seq_offsets
        S = 1 if seq is None else seq.shape[0] - 1
        slope = _ptr(balance.state)
    _same_device(dev, d_weights=d_w, topk_idx=idx, d_loss=d_loss)
    d_logits = torch.empty_like(logits)
    with _on(dev):
        N.ep_router_backward(_ptr(logits), _LOGIT_DTYPES[logits.dtype], T, E, K, _SCORES[score],
                             int(renorm), scale, _ptr(idx), _ptr(d_w), slope, _ptr(seq), S,
                             _ptr(d_loss), _ptr(d_logits), _stream(dev))
    return d_logits


def route_backward(d_weights: torch.Tensor, routing: Routing, *,
                   balance: Optional[BalanceLoss] = None,
                   d_loss: Optional[torch.Tensor] = None) -> torch.Tensor:
    """d_logits [T, E] (the logits' dtype) from d_weights [T, K] fp32.  With
    `balance` and `d_loss` ([1] fp32, on the GPU) the balance loss's gradient
    is added in the same pass; it must be of the same logits and score."""
    if balance is None and d_loss is not None:
        raise ValueError("d_loss needs balance")
    if balance is not None and (balance.logits.data_ptr() != routing.logits.data_ptr() or
                                balance.logits.shape != routing.logits.shape or
                                balance.logits.dtype != routing.logits.dtype or
                                balance.score != routing.score):
        raise ValueError("balance is of other logits or another score than routing")
    return _router_backward(routing.logits, routing.score, d_weights, routing, d_loss, balance)


def balance_loss_backward(d_loss: torch.Tensor, balance: BalanceLoss) -> torch.Tensor:
    """d_logits [T, E] (the logits' dtype) of the balance loss; zero for tokens
    outside all sequences.  d_loss: [1] fp32, on the GPU."""
    return _router_backward(balance.logits, balance.score, None, None, d_loss, balance)


# ---------------------------------------------------------------- adapters
def _apart(out: torch.Tensor, **inputs):
    """Refuses an output in an input's memory: other blocks still read it."""
    lo = out.data_ptr()
    hi = lo + out.numel() * out.element_size()
    for name, t in inputs.items():
        if t is None or lo == hi:
            continue
        if t.data_ptr() < hi and lo < t.data_ptr() + t.numel() * t.element_size():
            raise ValueError(f"out must not overlap {name}")


_NO_STATE = 256         # bytes of the stub that the ABI asks for where a call leaves no state


@functools.lru_cache(maxsize=256)
def _adapter_bytes(T: int, H: int, O: int, E: int, K: int, r: int):
    """The state's and the two workspaces' bytes, which go by the sizes alone."""
    return (N.ep_adapter_state_bytes(T, H, O, E, K, r),
            N.ep_adapter_workspace_bytes(T, H, O, E, K, r, 0),
            N.ep_adapter_workspace_bytes(T, H, O, E, K, r, 1))


@dataclass
class AdapterHandle:
    """What adapter_project_backward needs from adapter_project.  The operands
    must still hold their values when the backward runs."""
    x: torch.Tensor
    weight: torch.Tensor
    a: torch.Tensor
    b: torch.Tensor
    topk_idx: torch.Tensor
    topk_weights: Optional[torch.Tensor]
    scale: float
    num_invalid: torch.Tensor                  # [1] int32: entries neither -1 nor in [0, E)
    state: Optional[torch.Tensor]              # None after a call of a few tokens, which leaves none


def adapter_project(x: torch.Tensor, weight: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                    topk_idx: torch.Tensor, topk_weights: Optional[torch.Tensor] = None, *,
                    scale: float = 1.0, out: Optional[torch.Tensor] = None):
    """Low-rank adapters beside a shared projection:
    out[t] = bf16(weight x_t + sum_k scale * topk_weights[t,k] * b[e] (a[e] x_t)),
    e = topk_idx[t,k] (-1 = none; weights 1 if None).  One adapter per request:
    topk_idx [T, 1]; low-rank experts beside a shared one: the topk_idx and
    topk_weights of route.  x [T, H], weight [O, H], a [E, r, H], b [E, O, r],
    all bf16; r a multiple of 8 up to 128.  `out` may not overlap an operand.
    -> (out [T, O] bf16, AdapterHandle).  Tensors carry no autograd graph: the
    gradients are adapter_project_backward."""
    _need(x, "x", torch.bfloat16, 2)
    _need(weight, "weight", torch.bfloat16, 2)
    _need(a, "a", torch.bfloat16, 3)
    _need(b, "b", torch.bfloat16, 3)
    _need(topk_idx, "topk_idx", torch.int32, 2)
    T, H = x.shape
    O = weight.shape[0]
    E, r = a.shape[:2]
    if weight.shape[1] != H or a.shape[2] != H:
        raise ValueError("weight and a must have x's H channels")
    if tuple(b.shape) != (E, O, r):
        raise ValueError(f"b must be [E, O, r] = {(E, O, r)}, got {tuple(b.shape)}")
    if topk_idx.shape[0] != T:
        raise ValueError("x and topk_idx disagree on the number of tokens")
    K = topk_idx.shape[1]
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, 2)
        if tuple(topk_weights.shape) != (T, K):
            raise ValueError("topk_weights must be [T, K]")
    dev = x.device
    _same_device(dev, weight=weight, a=a, b=b, topk_idx=topk_idx, topk_weights=topk_weights)
    state_bytes, ws_bytes, _ = _adapter_bytes(T, H, O, E, K, r)
    given = out is not None
    out = _out(out, (T, O), dev)
    if given:
        _apart(out, x=x, weight=weight, a=a, b=b, topk_idx=topk_idx, topk_weights=topk_weights)
    ninv = torch.empty(1, dtype=torch.int32, device=dev)
    # a call of a few tokens leaves nothing for its backward: one allocation for
    # both, and none of it kept
    state = torch.empty(state_bytes, dtype=torch.uint8, device=dev) if state_bytes > _NO_STATE else None
    scratch = torch.empty(ws_bytes + (0 if state is not None else state_bytes), dtype=torch.uint8, device=dev)
    ws = scratch.data_ptr()
    at = ws + ws_bytes if state is None else state.data_ptr()
    with _on(dev):
        N.ep_adapter_project(_ptr(x), T, H, _ptr(weight), O, _ptr(a), _ptr(b), E, r,
                             _ptr(topk_idx), _ptr(topk_weights), K, float(scale), _ptr(out),
                             _ptr(ninv), at, state_bytes, ws, ws_bytes, _stream(dev))
    return out, AdapterHandle(x, weight, a, b, topk_idx, topk_weights, float(scale), ninv, state)


def adapter_project_backward(d_out: torch.Tensor, handle: AdapterHandle):
    """-> (dx [T, H] bf16, da [E, r, H] bf16, db [E, O, r] bf16, d_weights
    [T, K] fp32): the gradients for d_out [T, O] bf16.  The shared weight is
    frozen and has none; adapters that no token names get 0."""
    _need(d_out, "d_out", torch.bfloat16, 2)
    x, weight, a, b, idx = handle.x, handle.weight, handle.a, handle.b, handle.topk_idx
    T, H = x.shape
    O = weight.shape[0]
    E, r = a.shape[:2]
    K = idx.shape[1]
    if tuple(d_out.shape) != (T, O):
        raise ValueError(f"d_out must be {(T, O)}, got {tuple(d_out.shape)}")
    dev = x.device
    _same_device(dev, d_out=d_out)
    state_bytes, _, ws_bytes = _adapter_bytes(T, H, O, E, K, r)
    state = handle.state
    ws = torch.empty(ws_bytes + (0 if state is not None else state_bytes), dtype=torch.uint8, device=dev)
    at = ws.data_ptr() + ws_bytes if state is None else state.data_ptr()
    dx, da, db = torch.empty_like(x), torch.empty_like(a), torch.empty_like(b)
    dw = torch.empty((T, K), dtype=torch.float32, device=dev)
    with _on(dev):
        N.ep_adapter_project_backward(_ptr(d_out), _ptr(x), T, H, _ptr(weight), O, _ptr(a),
                                      _ptr(b), E, r, _ptr(idx), _ptr(handle.topk_weights), K,
                                      handle.scale, at, state_bytes,
                                      _ptr(dx), _ptr(da), _ptr(db), _ptr(dw), _ptr(ws), ws_bytes,
                                      _stream(dev))
    return dx, da, db, dw


# ---------------------------------------------------------------- the experts
_MX_OF = {torch.uint8: "mxfp4_e2m1", torch.float8_e4m3fn: "mxfp8_e4m3", torch.float8_e5m2: "mxfp8_e5m2"}
_ACTIVATIONS = {None: N.EP_ACT_NONE, "swiglu": N.EP_ACT_SWIGLU}


def _sizes(call: str, *sizes: int):
    """The C calls' sizes are 32 bits: a larger one would arrive as what is left of it."""
    if max(sizes) > 0x7FFFFFFF:
        raise N.EpError(call, N.EP_ERR_UNSUPPORTED)


def _mx_mode(quant: str) -> str:
    quant = _QUANT_ALIASES.get(quant, quant)
    if quant not in _MX_OF.values():
        raise ValueError(f"quant must be an MX mode, got {quant!r}")
    return quant


def _need_codes(codes: torch.Tensor, scales: Optional[torch.Tensor], name: str, ndim: int):
    """Checks a microscaled tensor; -> its mode and channels."""
    if not isinstance(codes, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if codes.dtype not in _MX_OF:
        raise ValueError(f"{name} must hold MX codes (uint8, float8_e4m3fn or float8_e5m2), got {codes.dtype}")
    _need(codes, name, codes.dtype, ndim)
    _need(scales, f"{name}'s scales", torch.uint8, ndim)
    quant = _MX_OF[codes.dtype]
    H = codes.shape[-1] * _QUANT[quant][2]
    if H % 32 != 0 or tuple(scales.shape) != (*codes.shape[:-1], H // 32):
        raise ValueError(f"{name} {tuple(codes.shape)} needs one scale per 32 channels, got {tuple(scales.shape)}")
    _same_device(codes.device, **{f"{name}'s scales": scales})
    return quant, H


def mx_quantize(x: torch.Tensor, quant: str = "mxfp4_e2m1"):
    """bf16 [..., H] (weights, activations) -> (codes, e8m0 scales [..., H/32]),
    the ones that dispatch makes of such rows: "mxfp4_e2m1" uint8 [..., H/2],
    "mxfp8_e4m3" and "mxfp8_e5m2" [..., H] of the torch type."""
    quant = _mx_mode(quant)
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a tensor")
    if x.dim() < 1:
        raise ValueError("x must have a last dimension of channels")
    _need(x, "x", torch.bfloat16, x.dim())
    H = x.shape[-1]
    q, dt, div, _ = _QUANT[quant]
    if H < 32 or H % 32 != 0:
        raise ValueError(f"x must have a multiple of 32 channels, got {H}")
    _sizes("ep_mx_quantize", x.numel() // H, H)
    dev = x.device
    codes = torch.empty((*x.shape[:-1], H // div), dtype=dt, device=dev)
    scales = torch.empty((*x.shape[:-1], H // 32), dtype=torch.uint8, device=dev)
    with _on(dev):
        N.ep_mx_quantize(_ptr(x), x.numel() // H, H, q, _ptr(codes), _ptr(scales), _stream(dev))
    return codes, scales


def mx_dequantize(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """bf16 [..., H] of codes and scales as mx_quantize and dispatch make them
    (the mode is told by the codes' type)."""
    if not isinstance(codes, torch.Tensor):
        raise TypeError("codes must be a tensor")
    if codes.dim() < 1:
        raise ValueError("codes must have a last dimension of channels")
    quant, H = _need_codes(codes, scales, "codes", codes.dim())
    if H < 32:
        raise ValueError("codes must have a multiple of 32 channels")
    _sizes("ep_mx_dequantize", scales.numel() * 32 // H, H)
    dev = codes.device
    out = torch.empty((*codes.shape[:-1], H), dtype=torch.bfloat16, device=dev)
    with _on(dev):
        N.ep_mx_dequantize(_ptr(codes), _ptr(scales), out.numel() // H, H, _QUANT[quant][0], _ptr(out),
                           _stream(dev))
    return out


@dataclass
class ExpertHandle:
    """What expert_product_backward needs from expert_product.  The operands must
    still hold their values when the backward runs (without an activation x is not
    looked at)."""
    x: torch.Tensor
    x_scales: Optional[torch.Tensor]
    weight: torch.Tensor
    weight_scales: torch.Tensor
    offsets: Optional[torch.Tensor]
    counts: Optional[torch.Tensor]
    activation: Optional[str]


def _expert_sizes(x, x_scales, weight, weight_scales, offsets, counts, activation):
    """Checks the operands of an expert's product; -> quant, rows, cap, E, O, H."""
    if activation not in _ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a tensor")
    ndim = 3 if offsets is None else 2
    if x.dtype == torch.bfloat16:
        if x_scales is not None:
            raise ValueError("bf16 rows have no scales")
        _need(x, "x", torch.bfloat16, ndim)
        quant, H = "bf16", x.shape[-1]
    else:
        quant, H = _need_codes(x, x_scales, "x", ndim)
    mode, wH = _need_codes(weight, weight_scales, "weight", 3)
    if mode != "mxfp4_e2m1":
        raise ValueError("weight must be in MXFP4 (uint8 codes)")
    E, O = weight.shape[:2]
    if wH != H:
        raise ValueError(f"weight has {wH} channels, the rows {H}")
    if offsets is not None:
        if counts is not None:
            raise ValueError("rows go by offsets or by counts, not by both")
        _need(offsets, "offsets", torch.int32, 1)
        if offsets.shape[0] != E + 1:
            raise ValueError(f"offsets must be [E + 1] = {E + 1}, got {offsets.shape[0]}")
        rows, cap = x.shape[0], 0
    else:
        if x.shape[0] != E:
            raise ValueError(f"padded rows must be [E, cap, ...] of the weight's {E} experts, got {tuple(x.shape)}")
        if counts is not None:
            _need(counts, "counts", torch.int32, 1)
            if counts.shape[0] != E:
                raise ValueError(f"counts must be [E] = {E}, got {counts.shape[0]}")
        cap = x.shape[1]
        rows = E * cap
    _sizes("ep_expert_product", rows, cap, E, O, H)
    _same_device(x.device, x_scales=x_scales, weight=weight, weight_scales=weight_scales, offsets=offsets,
                 counts=counts)
    return quant, rows, cap, E, O, H


def _rows_out(out: Optional[torch.Tensor], shape, dt, dev: torch.device, **inputs) -> torch.Tensor:
    """A caller's output rows, checked, or new ones."""
    if out is None:
        return torch.empty(shape, dtype=dt, device=dev)
    _need(out, "out", dt, len(shape))
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must be {tuple(shape)}, got {tuple(out.shape)}")
    _same_device(dev, out=out)
    _apart(out, **inputs)
    return out


def expert_product(x: torch.Tensor, x_scales: Optional[torch.Tensor], weight: torch.Tensor,
                   weight_scales: torch.Tensor, *, offsets: Optional[torch.Tensor] = None,
                   counts: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                   quant: str = "bf16", out: Optional[torch.Tensor] = None):
    """Every expert's matrix on the expert's rows, between dispatch and combine:
    y[r] = weight[e] x[r], or with activation="swiglu" (weight [E, 2I, H])
    silu(a) * b of its two halves.  weight, weight_scales: MXFP4, [E, O, H/2] and
    [E, O, H/32] (mx_quantize).
    x, x_scales: rows as dispatch makes them, MXFP4 or MXFP8 (quant "mxfp4_e2m1",
    "mxfp8_e4m3", "mxfp8_e5m2"), or bf16 with None.  [rows, ...] with `offsets`
    [E+1] (Layout.offsets), or the padded [E, cap, ...] with `counts` [E]
    (Handle.recv_count; None: every row).  Rows that no expert has are neither
    read nor written.
    quant: "bf16", or an MX mode for the next product's rows.  `out` (bf16 only)
    may not overlap an operand.
    -> (y, y_scales or None, ExpertHandle).  Tensors carry no autograd graph: the
    rows' gradient is expert_product_backward."""
    mode, rows, cap, E, O, H = _expert_sizes(x, x_scales, weight, weight_scales, offsets, counts, activation)
    width = O // 2 if activation else O
    if activation and O % 2 != 0:
        raise ValueError("swiglu needs an even number of weight rows")
    if quant != "bf16":
        quant = _mx_mode(quant)
        if width % 32 != 0:
            raise ValueError(f"quantised rows need a multiple of 32 channels, got {width}")
        if out is not None:
            raise ValueError("out is for bf16 rows")
    q, dt, div, _ = _QUANT[quant]
    dev = x.device
    lead = tuple(x.shape[:-1])
    y = _rows_out(out, (*lead, width // div), dt, dev, x=x, x_scales=x_scales, weight=weight,
                  weight_scales=weight_scales, offsets=offsets, counts=counts)
    scales = None if quant == "bf16" else torch.empty((*lead, width // 32), dtype=torch.uint8, device=dev)
    with _on(dev):
        N.ep_expert_product(_ptr(x), _ptr(x_scales), _QUANT[mode][0], rows, _ptr(weight), _ptr(weight_scales), E, O,
                            H, _ptr(offsets), _ptr(counts), cap, _ACTIVATIONS[activation], q, _ptr(y),
                            _ptr(scales), _stream(dev))
    return y, scales, ExpertHandle(x, x_scales, weight, weight_scales, offsets, counts, activation)


def expert_product_backward(d_y: torch.Tensor, handle: ExpertHandle, *,
                            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dx, bf16 rows like x, for d_y (bf16, like y).  The weight is frozen and has
    no gradient; a quantisation of x or of y passes the gradient on as it is.
    Rows that no expert has are not written."""
    h = handle
    mode, rows, cap, E, O, H = _expert_sizes(h.x, h.x_scales, h.weight, h.weight_scales, h.offsets, h.counts,
                                             h.activation)
    lead = tuple(h.x.shape[:-1])
    _need(d_y, "d_y", torch.bfloat16, len(lead) + 1)
    want = (*lead, O // 2 if h.activation else O)
    if tuple(d_y.shape) != want:
        raise ValueError(f"d_y must be {want}, got {tuple(d_y.shape)}")
    dev = h.x.device
    _same_device(dev, d_y=d_y)
    dx = _rows_out(out, (*lead, H), torch.bfloat16, dev, d_y=d_y, x=h.x, x_scales=h.x_scales, weight=h.weight,
                   weight_scales=h.weight_scales, offsets=h.offsets, counts=h.counts)
    act = _ACTIVATIONS[h.activation]
    ws_bytes = N.ep_expert_workspace_bytes(rows, O, act)
    if ws_bytes == 0:
        raise N.EpError("ep_expert_workspace_bytes", N.EP_ERR_INVALID_ARG)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    with _on(dev):
        N.ep_expert_product_backward(_ptr(d_y), _ptr(h.x), _ptr(h.x_scales), _QUANT[mode][0], rows, _ptr(h.weight),
                                     _ptr(h.weight_scales), E, O, H, _ptr(h.offsets), _ptr(h.counts), cap, act,
                                     _ptr(dx), _ptr(ws), ws_bytes, _stream(dev))
    return dx


@functools.lru_cache(maxsize=256)
def _few_bytes(T: int, K: int, E: int, H: int, I: int) -> int:
    return N.ep_low_latency_experts_workspace_bytes(T, K, E, H, I)


def low_latency_experts(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: Optional[torch.Tensor],
                        up: torch.Tensor, down: torch.Tensor, *, up_scales: Optional[torch.Tensor] = None,
                        down_scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """A whole layer of experts for a decode batch (up to 128 tokens), instead of
    low_latency_dispatch, the experts' products and low_latency_combine, in two
    launches: out[t] = sum_k topk_weights[t,k] * down[e] (silu(a) * b), a and b the
    halves of up[e] x_t, e = topk_idx[t,k] (-1 = none; weights 1 if None).
    x [T, H] bf16; up [E, 2I, H] and down [E, H, I] in bf16, or both in MXFP4
    (mx_quantize: codes, with up_scales and down_scales).  `out` may not overlap an
    operand.  -> (out [T, H] bf16, num_invalid [1] int32: entries neither -1 nor in
    [0, E))."""
    _need(x, "x", torch.bfloat16, 2)
    _need(topk_idx, "topk_idx", torch.int32, 2)
    T, H = x.shape
    if topk_idx.shape[0] != T:
        raise ValueError("x and topk_idx disagree on the number of tokens")
    K = topk_idx.shape[1]
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, 2)
        if tuple(topk_weights.shape) != (T, K):
            raise ValueError("topk_weights must be [T, K]")
    if up_scales is None and down_scales is None:
        _need(up, "up", torch.bfloat16, 3)
        _need(down, "down", torch.bfloat16, 3)
        uH, I = up.shape[2], down.shape[2]
    else:
        if up_scales is None or down_scales is None:
            raise ValueError("up and down are both in bf16 or both in MXFP4")
        (mu, uH), (md, I) = _need_codes(up, up_scales, "up", 3), _need_codes(down, down_scales, "down", 3)
        if mu != "mxfp4_e2m1" or md != "mxfp4_e2m1":
            raise ValueError("up and down must be in MXFP4 (uint8 codes)")
    E = up.shape[0]
    if uH != H or tuple(up.shape[:2]) != (E, 2 * I) or tuple(down.shape[:2]) != (E, H):
        raise ValueError(f"up must be [E, 2I, H] and down [E, H, I] with H = {H}")
    _sizes("ep_low_latency_experts", T, K, E, H, I)
    dev = x.device
    _same_device(dev, topk_idx=topk_idx, topk_weights=topk_weights, up=up, down=down, up_scales=up_scales,
                 down_scales=down_scales)
    out = _rows_out(out, (T, H), torch.bfloat16, dev, x=x, topk_idx=topk_idx, topk_weights=topk_weights, up=up,
                    down=down, up_scales=up_scales, down_scales=down_scales)
    ninv = torch.empty(1, dtype=torch.int32, device=dev)
    ws_bytes = _few_bytes(T, K, E, H, I)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    with _on(dev):
        N.ep_low_latency_experts(_ptr(x), T, H, _ptr(topk_idx), _ptr(topk_weights), K, _ptr(up), _ptr(up_scales),
                                 _ptr(down), _ptr(down_scales), E, I, _ptr(out), _ptr(ninv), _ptr(ws), ws_bytes,
                                 _stream(dev))
    return out, ninv
