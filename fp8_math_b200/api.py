"""Allocating convenience wrappers over the C ABI (torch tensors in and out).

Each helper allocates its output tensors on the input's device with
``torch.empty`` and calls one libbsq entry point through ``fp8_math_b200.bsq``;
all arithmetic runs in the library's CUDA kernels.  Shapes and layouts are
those of include/bsq.h.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import bsq


def sf_bytes(rows: int, nblocks: int) -> int:
    return bsq.bsq_sf_bytes(rows, nblocks)


def _ld(x: torch.Tensor) -> int:
    assert x.dim() == 2 and x.stride(1) == 1, "row-major 2-D tensor expected"
    return x.stride(0)


def amax(x, rht_mask=None, row_index=None, out=None):
    M = x.shape[0] if row_index is None else row_index.shape[0]
    out = torch.empty(1, dtype=torch.float32, device=x.device) if out is None else out
    bsq.bsq_amax(x, M, x.shape[1], _ld(x), rht_mask is not None, rht_mask or 0, row_index, out)
    return out


def quant_nvfp4(x, block_2d=False, four_over_six=False, rht_mask=None, row_index=None, groups=None,
                amax_in=None, out=None):
    """Returns (codes [R, K/2] uint8, sf swizzled uint8, global_scale [1] fp32).
    groups = (row_offsets int32 [G+1], sf_row_offsets int32 [G+1], sf_rows)."""
    K = x.shape[1]
    R = x.shape[0] if row_index is None else row_index.shape[0]
    G, ro, so = 0, None, None
    sf_rows = R
    if groups is not None:
        ro, so, sf_rows = groups
        G = ro.shape[0] - 1
    if out is None:
        codes = torch.empty(R, K // 2, dtype=torch.uint8, device=x.device)
        sf = torch.zeros(sf_bytes(sf_rows, K // 16), dtype=torch.uint8, device=x.device)
        gs = torch.empty(1, dtype=torch.float32, device=x.device)
    else:
        codes, sf, gs = out
    bsq.bsq_quant_nvfp4(x, R, K, _ld(x), block_2d, four_over_six, rht_mask is not None, rht_mask or 0, row_index,
                        G, ro, so, amax_in, gs, codes, sf)
    return codes, sf, gs


def quant_mxfp8(x, colwise=False, sr=False, seed=0, stream_id=0, out=None):
    """Returns (codes, sf swizzled) in the output orientation ([M,K] or [K,M])."""
    M, K = x.shape
    R, Cc = (K, M) if colwise else (M, K)
    if out is None:
        codes = torch.empty(R, Cc, dtype=torch.uint8, device=x.device)
        sf = torch.zeros(sf_bytes(R, Cc // 32), dtype=torch.uint8, device=x.device)
    else:
        codes, sf = out
    bsq.bsq_quant_mxfp8(x, M, K, _ld(x), colwise, bsq.BSQ_SR if sr else bsq.BSQ_RNE, seed, stream_id, codes, sf)
    return codes, sf


def quant_mxfp8_rowcol(x, sr=False, seed=0, stream_id_row=0, stream_id_col=1, out=None):
    """Row-wise and column-wise MXFP8 in one pass.  Returns
    (codes_row [M,K], sf_row, codes_col [K,M], sf_col)."""
    M, K = x.shape
    if out is None:
        cr = torch.empty(M, K, dtype=torch.uint8, device=x.device)
        sr_ = torch.zeros(sf_bytes(M, K // 32), dtype=torch.uint8, device=x.device)
        cc = torch.empty(K, M, dtype=torch.uint8, device=x.device)
        sc = torch.zeros(sf_bytes(K, M // 32), dtype=torch.uint8, device=x.device)
    else:
        cr, sr_, cc, sc = out
    bsq.bsq_quant_mxfp8_rowcol(x, M, K, _ld(x), bsq.BSQ_SR if sr else bsq.BSQ_RNE, seed, stream_id_row,
                               stream_id_col, cr, sr_, cc, sc)
    return cr, sr_, cc, sc


def requant_nvfp4_mxfp8(codes, sf, gs, sr=True, seed=0, stream_id=1, out=None):
    """NVFP4 [R, C] (codes [R, C/2], swizzled sf, gs [1]) -> column-wise MXFP8.
    Returns (codes [C, R], sf swizzled)."""
    R, C = codes.shape[0], codes.shape[1] * 2
    if out is None:
        cc = torch.empty(C, R, dtype=torch.uint8, device=codes.device)
        sc = torch.zeros(sf_bytes(C, R // 32), dtype=torch.uint8, device=codes.device)
    else:
        cc, sc = out
    bsq.bsq_requant_nvfp4_mxfp8(codes, sf, gs, R, C, bsq.BSQ_SR if sr else bsq.BSQ_RNE, seed, stream_id, cc, sc)
    return cc, sc


def quant_nvfp4_sr(x, block_2d=False, rht_mask=None, row_index=None, amax_in=None, seed=0, stream_id=0, out=None):
    """NVFP4 with stochastic rounding of the elements.  Returns (codes
    [R, K/2] uint8, sf swizzled uint8, global_scale [1] fp32)."""
    K = x.shape[1]
    R = x.shape[0] if row_index is None else row_index.shape[0]
    if out is None:
        codes = torch.empty(R, K // 2, dtype=torch.uint8, device=x.device)
        sf = torch.zeros(sf_bytes(R, K // 16), dtype=torch.uint8, device=x.device)
        gs = torch.empty(1, dtype=torch.float32, device=x.device)
    else:
        codes, sf, gs = out
    bsq.bsq_quant_nvfp4_sr(x, R, K, _ld(x), block_2d, rht_mask is not None, rht_mask or 0, row_index, amax_in, gs,
                           seed, stream_id, codes, sf)
    return codes, sf, gs


def quant_mxfp4(x, sr=False, seed=0, stream_id=0, out=None):
    """Row-wise MXFP4.  Returns (codes [M,K/2], sf swizzled)."""
    M, K = x.shape
    if out is None:
        codes = torch.empty(M, K // 2, dtype=torch.uint8, device=x.device)
        sf = torch.zeros(sf_bytes(M, K // 32), dtype=torch.uint8, device=x.device)
    else:
        codes, sf = out
    bsq.bsq_quant_mxfp4(x, M, K, _ld(x), bsq.BSQ_SR if sr else bsq.BSQ_RNE, seed, stream_id, codes, sf)
    return codes, sf


def rht(x, mask, out=None):
    y = torch.empty_like(x) if out is None else out
    bsq.bsq_rht(x, y, x.shape[0], x.shape[1], _ld(x), _ld(y), mask)
    return y


def requant_transpose(codes_row, sf_row, sr=True, seed=0, stream_id=1, out=None):
    M, K = codes_row.shape
    if out is None:
        cc = torch.empty(K, M, dtype=torch.uint8, device=codes_row.device)
        sc = torch.zeros(sf_bytes(K, M // 32), dtype=torch.uint8, device=codes_row.device)
    else:
        cc, sc = out
    bsq.bsq_requant_transpose(codes_row, sf_row, M, K, bsq.BSQ_SR if sr else bsq.BSQ_RNE, seed, stream_id, cc, sc)
    return cc, sc


def _out(M, N, dtype, device):
    """[M, N] output whose row stride is a multiple of 16 bytes (a view of a
    padded buffer when N needs it)."""
    per = 16 // torch.tensor([], dtype=dtype).element_size()
    ld = -(-N // per) * per
    return torch.empty(M, ld, dtype=dtype, device=device)[:, :N]


def gemm(fmt, A, sfA, B, sfB, M, N, K, gsA=None, gsB=None, out_dtype=torch.bfloat16, out=None):
    C_out = _out(M, N, out_dtype, A.device) if out is None else out
    ot = bsq.BSQ_OUT_BF16 if C_out.dtype == torch.bfloat16 else bsq.BSQ_OUT_F32
    bsq.bsq_gemm_blockscaled(fmt, A, sfA, gsA, B, sfB, gsB, M, N, K, C_out, C_out.stride(0), ot)
    return C_out


def grouped_gemm(fmt, row_offsets, sf_row_offsets, A, sfA, B, sfB, M_total, N, K, gsA=None, gsB=None,
                 out_dtype=torch.bfloat16, out=None):
    G = row_offsets.shape[0] - 1
    C_out = _out(M_total, N, out_dtype, A.device) if out is None else out
    ot = bsq.BSQ_OUT_BF16 if C_out.dtype == torch.bfloat16 else bsq.BSQ_OUT_F32
    bsq.bsq_grouped_gemm(fmt, G, row_offsets, sf_row_offsets, M_total, A, sfA, gsA, B, sfB, gsB, N, K, C_out,
                         C_out.stride(0), ot)
    return C_out


def grouped_gemm_nvfp4_out(row_offsets, sf_row_offsets, A, sfA, B, sfB, M_total, N, K, out_gs, sf_rows,
                           gsA=None, gsB=None, four_over_six=True, amax=True, bf16_out=False, out=None):
    """Grouped NVFP4 GEMM with the output quantized to NVFP4 in the epilogue
    (given global scale out_gs [1]).  Returns (codes [M_total, N/2], sf
    swizzled with sf_rows rows, amax [1] or None, C bf16 or None)."""
    G = row_offsets.shape[0] - 1
    if out is None:
        codes = torch.empty(M_total, N // 2, dtype=torch.uint8, device=A.device)
        sf = torch.zeros(sf_bytes(sf_rows, N // 16), dtype=torch.uint8, device=A.device)
        am = torch.empty(1, dtype=torch.float32, device=A.device) if amax else None
        C_out = _out(M_total, N, torch.bfloat16, A.device) if bf16_out else None
    else:
        codes, sf, am, C_out = out
    bsq.bsq_grouped_gemm_nvfp4_out(bsq.BSQ_NVFP4, G, row_offsets, sf_row_offsets, M_total, A, sfA, gsA, B, sfB, gsB,
                                   N, K, out_gs, four_over_six, codes, sf, am, C_out,
                                   C_out.stride(0) if C_out is not None else 0)
    return codes, sf, am, C_out


def quant_s2f6(x, rht_mask=None, out=None):
    """RHT (optional) + block-scaled S2F6.  Returns (codes [M, K] int8, sf [M, K/32] uint8)."""
    M, K = x.shape
    if out is None:
        codes = torch.empty(M, K, dtype=torch.int8, device=x.device)
        sf = torch.empty(M, K // 32, dtype=torch.uint8, device=x.device)
    else:
        codes, sf = out
    bsq.bsq_quant_s2f6(x, M, K, _ld(x), rht_mask is not None, rht_mask or 0, codes, sf)
    return codes, sf


def combine_s2f6(codes, sf, token_offsets, rows, weights, rht_mask, out=None):
    """Per token: weighted sum of its S2F6 rows, inverse RHT, bf16 [T, K]."""
    K = codes.shape[1]
    T = token_offsets.shape[0] - 1
    y = torch.empty(T, K, dtype=torch.bfloat16, device=codes.device) if out is None else out
    bsq.bsq_combine_s2f6(codes, sf, K, token_offsets, rows, weights, T, rht_mask, y, _ld(y))
    return y


def quant_nvfp4_gather(x, row_index, four_over_six=False, rht_mask=None, groups=None, amax_in=None, out=None,
                       workspace=None):
    """bsq_quant_nvfp4 of the rows x[row_index] (same bytes), computed by
    quantizing each source row once.  Returns (codes, sf, global_scale)."""
    T, K = x.shape
    R = row_index.shape[0]
    G, ro, so = 0, None, None
    sf_rows = R
    if groups is not None:
        ro, so, sf_rows = groups
        G = ro.shape[0] - 1
    if out is None:
        codes = torch.empty(R, K // 2, dtype=torch.uint8, device=x.device)
        sf = torch.zeros(sf_bytes(sf_rows, K // 16), dtype=torch.uint8, device=x.device)
        gs = torch.empty(1, dtype=torch.float32, device=x.device)
    else:
        codes, sf, gs = out
    nbytes = bsq.bsq_quant_nvfp4_gather_workspace(T, K)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    bsq.bsq_quant_nvfp4_gather(x, T, K, _ld(x), row_index, R, four_over_six, rht_mask is not None, rht_mask or 0, G,
                               ro, so, amax_in, gs, codes, sf, workspace, workspace.numel())
    return codes, sf, gs


# ---------------------------------------------------------------- mixture-of-experts training step
# The library sees pointers only: types, shapes and devices are checked here,
# with as few calls per tensor as will do (a rollout's calls take microseconds).
def _refuse(fn):
    raise bsq.BsqError(fn, bsq.BSQ_ERR_INVALID)


def _arr(fn, t, dtype, n, dev):
    """t is a contiguous tensor of n elements of this type on device dev (the current one)."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or
            t.get_device() != dev):
        _refuse(fn)


def _mat(fn, t, dtype, rows, cols, dev):
    """t is a row-major [rows, cols] matrix; returns its leading dimension."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != (rows, cols) or t.get_device() != dev:
        _refuse(fn)
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        _refuse(fn)
    return ld if rows > 1 else max(ld, -(-cols // 8) * 8)


class MoeRoute(NamedTuple):
    """Outputs of moe_route (include/bsq.h, bsq_moe_route)."""
    expert_ids: torch.Tensor               # [T, k] int32, -1: empty slot
    weights: torch.Tensor                  # [T, k] fp32
    rows: torch.Tensor                     # [T, k] int32, -1: empty slot
    row_index: torch.Tensor                # [T * k] int32
    row_offsets: torch.Tensor              # [E + 1] int32
    sf_row_offsets: torch.Tensor           # [E + 1] int32
    counts: torch.Tensor                   # [E + 1] int32, the last one the tokens with a slot
    prob_sums: Optional[torch.Tensor]      # [E] fp32, with the balance loss
    loss: Optional[torch.Tensor]           # [1] fp32


def moe_route_workspace(T: int, E: int) -> int:
    return bsq.bsq_moe_route_workspace(T, E)


def moe_route(logits, topk, token_mask=None, renorm=True, balance_coef=None, out=None, workspace=None):
    """Top-k routing of logits [T, E] (fp32 or bf16) -> MoeRoute.  token_mask
    uint8 or bool [T], 0 for padding; balance_coef None for no balance loss.
    The most routed rows is T * topk; a buffer for scale factors of all of
    them needs T * topk + 127 * min(E, T * topk) rows at most (each expert's
    rows pad to 128)."""
    fn = "moe_route"
    dev = torch.cuda.current_device()
    dtype = logits.dtype
    if logits.dim() != 2 or (dtype is not torch.float32 and dtype is not torch.bfloat16) or topk < 1:
        _refuse(fn)
    T, E = logits.shape
    ld = _mat(fn, logits, dtype, T, E, dev)
    with_loss = balance_coef is not None
    if out is None:
        i32 = dict(dtype=torch.int32, device=logits.device)
        f32 = dict(dtype=torch.float32, device=logits.device)
        out = MoeRoute(torch.empty(T, topk, **i32), torch.empty(T, topk, **f32), torch.empty(T, topk, **i32),
                       torch.empty(T * topk, **i32), torch.empty(E + 1, **i32), torch.empty(E + 1, **i32),
                       torch.empty(E + 1, **i32), torch.empty(E, **f32) if with_loss else None,
                       torch.empty(1, **f32) if with_loss else None)
    else:
        out = MoeRoute(*out)
        ids, weights, rows, row_index, row_offsets, sf_row_offsets, counts, prob_sums, loss = out
        n, i32 = T * topk, torch.int32
        _arr(fn, ids, i32, n, dev)
        _arr(fn, weights, torch.float32, n, dev)
        _arr(fn, rows, i32, n, dev)
        _arr(fn, row_index, i32, n, dev)
        _arr(fn, row_offsets, i32, E + 1, dev)
        _arr(fn, sf_row_offsets, i32, E + 1, dev)
        _arr(fn, counts, i32, E + 1, dev)
        if prob_sums is not None:
            _arr(fn, prob_sums, torch.float32, E, dev)
        if loss is not None:
            _arr(fn, loss, torch.float32, 1, dev)
        if (loss is not None) != with_loss:  # a coefficient and a place for the loss come together
            _refuse(fn)
    if token_mask is not None:
        _arr(fn, token_mask, torch.bool if token_mask.dtype is torch.bool else torch.uint8, T, dev)
    if workspace is None:
        workspace = torch.empty(bsq.bsq_moe_route_workspace(T, E), dtype=torch.uint8, device=logits.device)
    nbytes = workspace.numel()
    _arr(fn, workspace, torch.uint8, nbytes, dev)
    bsq.bsq_moe_route(logits, bsq.BSQ_OUT_F32 if dtype is torch.float32 else bsq.BSQ_OUT_BF16, T, E, ld, token_mask,
                      topk, renorm, *out[:8], balance_coef if with_loss else 0.0, out[8], workspace, nbytes)
    return out


def moe_route_bwd(logits, expert_ids, weights, dweights=None, counts=None, dloss=None, balance_coef=None, renorm=True,
                  out=None):
    """Gradient of the logits from the weights' gradient (fp32 [T, k]) and the
    balance loss's (fp32 [1]; it takes the router's counts and balance_coef,
    and is refused without them)."""
    fn = "moe_route_bwd"
    dev = torch.cuda.current_device()
    dtype = logits.dtype
    if logits.dim() != 2 or (dtype is not torch.float32 and dtype is not torch.bfloat16) or expert_ids.dim() != 2:
        _refuse(fn)
    T, E = logits.shape
    k = expert_ids.shape[1]
    n = T * k
    ld = _mat(fn, logits, dtype, T, E, dev)
    _arr(fn, expert_ids, torch.int32, n, dev)
    _arr(fn, weights, torch.float32, n, dev)
    if dweights is not None:
        _arr(fn, dweights, torch.float32, n, dev)
    if counts is not None:
        _arr(fn, counts, torch.int32, E + 1, dev)
    if dloss is not None:
        _arr(fn, dloss, torch.float32, 1, dev)
        if balance_coef is None:
            _refuse(fn)
    if out is None:
        out = torch.empty(T, E, dtype=dtype, device=logits.device)
    ldd = _mat(fn, out, dtype, T, E, dev)
    bsq.bsq_moe_route_bwd(logits, bsq.BSQ_OUT_F32 if dtype is torch.float32 else bsq.BSQ_OUT_BF16, T, E, ld, k, renorm,
                          expert_ids, weights, dweights, counts, 0.0 if balance_coef is None else balance_coef, dloss,
                          out, ldd)
    return out


def moe_combine(y, rows, weights=None, out=None):
    """Per token: the weighted sum of its rows of y [R, H] (bf16), bf16
    [T, H].  rows int32 [T, k] (-1: none), weights fp32 [T, k] or None for 1."""
    fn = "moe_combine"
    dev = torch.cuda.current_device()
    if y.dim() != 2 or rows.dim() != 2:
        _refuse(fn)
    R, H = y.shape
    T, k = rows.shape
    ldy = _mat(fn, y, torch.bfloat16, R, H, dev)
    _arr(fn, rows, torch.int32, T * k, dev)
    if weights is not None:
        _arr(fn, weights, torch.float32, T * k, dev)
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=y.device)
    ldo = _mat(fn, out, torch.bfloat16, T, H, dev)
    bsq.bsq_moe_combine(y, R, H, ldy, rows, weights, T, k, out, ldo)
    return out


def moe_combine_bwd(dout, y, rows, weights, out=None):
    """Gradients of moe_combine: (dy [R, H] bf16, dweights [T, k] fp32).  y is
    the bf16 [R, H], or the MXFP8 pair (codes [R, H], sf) it was kept as.
    Without out, the rows of dy that no token has are zeros."""
    fn = "moe_combine_bwd"
    dev = torch.cuda.current_device()
    codes = sf = None
    if isinstance(y, (tuple, list)):
        codes, sf = y
        y = None
    kept = y if codes is None else codes
    if kept.dim() != 2 or rows.dim() != 2:
        _refuse(fn)
    R, H = kept.shape
    T, k = rows.shape
    ldy = H
    if codes is None:
        ldy = _mat(fn, y, torch.bfloat16, R, H, dev)
    else:
        _arr(fn, codes, torch.uint8, R * H, dev)
        _scales(fn, sf, R, H // 32, dev)
    ldo = _mat(fn, dout, torch.bfloat16, T, H, dev)
    _arr(fn, rows, torch.int32, T * k, dev)
    _arr(fn, weights, torch.float32, T * k, dev)
    if out is None:
        out = (torch.zeros(R, H, dtype=torch.bfloat16, device=dout.device),
               torch.empty(T, k, dtype=torch.float32, device=dout.device))
    dy, dweights = out
    lddy = _mat(fn, dy, torch.bfloat16, R, H, dev)
    _arr(fn, dweights, torch.float32, T * k, dev)
    bsq.bsq_moe_combine_bwd(dout, ldo, y, ldy, codes, sf, R, H, rows, weights, T, k, dy, lddy, dweights)
    return dy, dweights


def _scales(fn, sf, rows, nblocks, dev):
    """sf is a swizzled scale-factor buffer for at least this many rows."""
    if not isinstance(sf, torch.Tensor):
        _refuse(fn)
    _arr(fn, sf, torch.uint8, sf.numel(), dev)
    if sf.numel() < -(-rows // 128) * 128 * (-(-nblocks // 4) * 4):
        _refuse(fn)


def swiglu_ckpt(u, n_rows=None, amax=True, out=None):
    """h = silu(gate) * v of u [M, 2F] = (gate | v) in bf16, and u in MXFP8 for
    the backward pass: (h [M, F] bf16, codes [M, 2F], sf swizzled, amax [1] of
    h or None).  n_rows int32 [1]: only that many rows exist; without out, the
    others are zeros."""
    fn = "swiglu_ckpt"
    dev = torch.cuda.current_device()
    if u.dim() != 2 or u.shape[1] % 2:
        _refuse(fn)
    M, F = u.shape[0], u.shape[1] // 2
    ldu = _mat(fn, u, torch.bfloat16, M, 2 * F, dev)
    if out is None:
        make = torch.empty if n_rows is None else torch.zeros
        out = (make(M, F, dtype=torch.bfloat16, device=u.device),
               make(M, 2 * F, dtype=torch.uint8, device=u.device),
               torch.zeros(sf_bytes(M, F // 16), dtype=torch.uint8, device=u.device),
               torch.empty(1, dtype=torch.float32, device=u.device) if amax else None)
    h, codes, sf, am = out
    ldh = _mat(fn, h, torch.bfloat16, M, F, dev)
    _arr(fn, codes, torch.uint8, M * 2 * F, dev)
    _scales(fn, sf, M, F // 16, dev)
    if am is not None:
        _arr(fn, am, torch.float32, 1, dev)
    if n_rows is not None:
        _arr(fn, n_rows, torch.int32, 1, dev)
    bsq.bsq_swiglu_ckpt(u, M, F, ldu, n_rows, h, ldh, codes, sf, am)
    return h, codes, sf, am


def swiglu_ckpt_bwd(dh, codes, sf, n_rows=None, recompute_h=False, out=None):
    """Gradient of swiglu_ckpt's u from dh [M, F] (bf16) and the checkpoint:
    (du [M, 2F] bf16, h [M, F] bf16 formed again from the checkpoint, or None).
    n_rows as in swiglu_ckpt."""
    fn = "swiglu_ckpt_bwd"
    dev = torch.cuda.current_device()
    if dh.dim() != 2:
        _refuse(fn)
    M, F = dh.shape
    lddh = _mat(fn, dh, torch.bfloat16, M, F, dev)
    _arr(fn, codes, torch.uint8, M * 2 * F, dev)
    _scales(fn, sf, M, F // 16, dev)
    if n_rows is not None:
        _arr(fn, n_rows, torch.int32, 1, dev)
    if out is None:
        make = torch.empty if n_rows is None else torch.zeros
        out = (make(M, 2 * F, dtype=torch.bfloat16, device=dh.device),
               make(M, F, dtype=torch.bfloat16, device=dh.device) if recompute_h else None)
    du, h = out
    lddu = _mat(fn, du, torch.bfloat16, M, 2 * F, dev)
    ldh = _mat(fn, h, torch.bfloat16, M, F, dev) if h is not None else 0
    bsq.bsq_swiglu_ckpt_bwd(dh, lddh, codes, sf, M, F, n_rows, du, lddu, h, ldh)
    return du, h
