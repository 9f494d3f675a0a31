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
def _need(fn, ok):
    """The library sees pointers only: shapes, types and devices are checked here."""
    if not ok:
        raise bsq.BsqError(fn, bsq.BSQ_ERR_INVALID)


def _dev(fn, *tensors):
    """Every tensor given lives on the current CUDA device (where the call is enqueued)."""
    d = torch.cuda.current_device()
    for t in tensors:
        _need(fn, t is None or (t.is_cuda and t.get_device() == d))


def _arr(fn, t, dtype, *shape):
    """t is None or a contiguous tensor of this type and shape."""
    _need(fn, t is None or (t.dtype == dtype and t.shape == shape and t.is_contiguous()))


def _mat(fn, t, dtype, rows, cols):
    """t is a row-major [rows, cols] matrix; returns its leading dimension."""
    _need(fn, t.dtype == dtype and t.shape == (rows, cols) and (cols <= 1 or t.stride(1) == 1))
    return t.stride(0) if rows > 1 else max(t.stride(0), -(-cols // 8) * 8)


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
    _need(fn, logits.dim() == 2 and logits.dtype in (torch.float32, torch.bfloat16))
    T, E = logits.shape
    ld = _mat(fn, logits, logits.dtype, T, E)
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
        _arr(fn, out.expert_ids, torch.int32, T, topk)
        _arr(fn, out.weights, torch.float32, T, topk)
        _arr(fn, out.rows, torch.int32, T, topk)
        _arr(fn, out.row_index, torch.int32, T * topk)
        for t in (out.row_offsets, out.sf_row_offsets, out.counts):
            _arr(fn, t, torch.int32, E + 1)
        _arr(fn, out.prob_sums, torch.float32, E)
        _arr(fn, out.loss, torch.float32, 1)
        _need(fn, with_loss or out.loss is None)
    if token_mask is not None:
        _need(fn, token_mask.dtype in (torch.uint8, torch.bool) and token_mask.shape == (T,) and
              token_mask.is_contiguous())
    if workspace is None:
        workspace = torch.empty(bsq.bsq_moe_route_workspace(T, E), dtype=torch.uint8, device=logits.device)
    _need(fn, workspace.dtype == torch.uint8 and workspace.is_contiguous())
    _dev(fn, logits, token_mask, workspace, *out)
    bsq.bsq_moe_route(logits, bsq.BSQ_OUT_F32 if logits.dtype == torch.float32 else bsq.BSQ_OUT_BF16, T, E, ld,
                      token_mask, topk, renorm, out.expert_ids, out.weights, out.rows, out.row_index, out.row_offsets,
                      out.sf_row_offsets, out.counts, out.prob_sums, balance_coef if with_loss else 0.0, out.loss,
                      workspace, workspace.numel())
    return out


def moe_route_bwd(logits, expert_ids, weights, dweights=None, counts=None, dloss=None, balance_coef=0.0, renorm=True,
                  out=None):
    """Gradient of the logits from the weights' gradient (fp32 [T, k]) and the
    balance loss's (fp32 [1], with the router's counts and its balance_coef)."""
    fn = "moe_route_bwd"
    _need(fn, logits.dim() == 2 and logits.dtype in (torch.float32, torch.bfloat16) and expert_ids.dim() == 2)
    T, E = logits.shape
    k = expert_ids.shape[1]
    ld = _mat(fn, logits, logits.dtype, T, E)
    _arr(fn, expert_ids, torch.int32, T, k)
    _arr(fn, weights, torch.float32, T, k)
    _arr(fn, dweights, torch.float32, T, k)
    _arr(fn, counts, torch.int32, E + 1)
    _need(fn, dloss is None or (dloss.dtype == torch.float32 and dloss.numel() == 1))
    if out is None:
        out = torch.empty(T, E, dtype=logits.dtype, device=logits.device)
    ldd = _mat(fn, out, logits.dtype, T, E)
    _dev(fn, logits, expert_ids, weights, dweights, counts, dloss, out)
    bsq.bsq_moe_route_bwd(logits, bsq.BSQ_OUT_F32 if logits.dtype == torch.float32 else bsq.BSQ_OUT_BF16, T, E, ld, k,
                          renorm, expert_ids, weights, dweights, counts, balance_coef, dloss, out, ldd)
    return out


def moe_combine(y, rows, weights=None, out=None):
    """Per token: the weighted sum of its rows of y [R, H] (bf16), bf16
    [T, H].  rows int32 [T, k] (-1: none), weights fp32 [T, k] or None for 1."""
    fn = "moe_combine"
    _need(fn, y.dim() == 2 and rows.dim() == 2)
    R, H = y.shape
    T, k = rows.shape
    ldy = _mat(fn, y, torch.bfloat16, R, H)
    _arr(fn, rows, torch.int32, T, k)
    _arr(fn, weights, torch.float32, T, k)
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=y.device)
    ldo = _mat(fn, out, torch.bfloat16, T, H)
    _dev(fn, y, rows, weights, out)
    bsq.bsq_moe_combine(y, R, H, ldy, rows, weights, T, k, out, ldo)
    return out


def moe_combine_bwd(dout, y, rows, weights, out=None):
    """Gradients of moe_combine: (dy [R, H] bf16, dweights [T, k] fp32).  y is
    the bf16 [R, H], or the MXFP8 pair (codes [R, H], sf) it was kept as.
    Without out, the rows of dy that no token has are zeros."""
    fn = "moe_combine_bwd"
    codes = sf = None
    if isinstance(y, (tuple, list)):
        codes, sf = y
        y = None
    kept = y if codes is None else codes
    _need(fn, kept.dim() == 2 and rows.dim() == 2)
    R, H = kept.shape
    T, k = rows.shape
    ldy = H
    if codes is None:
        ldy = _mat(fn, y, torch.bfloat16, R, H)
    else:
        _arr(fn, codes, torch.uint8, R, H)
        _need(fn, sf.dtype == torch.uint8 and sf.is_contiguous() and sf.numel() >= sf_bytes(R, H // 32))
    ldo = _mat(fn, dout, torch.bfloat16, T, H)
    _arr(fn, rows, torch.int32, T, k)
    _arr(fn, weights, torch.float32, T, k)
    if out is None:
        out = (torch.zeros(R, H, dtype=torch.bfloat16, device=dout.device),
               torch.empty(T, k, dtype=torch.float32, device=dout.device))
    dy, dweights = out
    lddy = _mat(fn, dy, torch.bfloat16, R, H)
    _arr(fn, dweights, torch.float32, T, k)
    _dev(fn, dout, y, codes, sf, rows, weights, dy, dweights)
    bsq.bsq_moe_combine_bwd(dout, ldo, y, ldy, codes, sf, R, H, rows, weights, T, k, dy, lddy, dweights)
    return dy, dweights


def swiglu_ckpt(u, n_rows=None, amax=True, out=None):
    """h = silu(gate) * v of u [M, 2F] = (gate | v) in bf16, and u in MXFP8 for
    the backward pass: (h [M, F] bf16, codes [M, 2F], sf swizzled, amax [1] of
    h or None).  n_rows int32 [1]: only that many rows exist."""
    fn = "swiglu_ckpt"
    _need(fn, u.dim() == 2 and u.shape[1] % 2 == 0)
    M, F = u.shape[0], u.shape[1] // 2
    ldu = _mat(fn, u, torch.bfloat16, M, 2 * F)
    nb = sf_bytes(M, F // 16)
    if out is None:
        out = (torch.empty(M, F, dtype=torch.bfloat16, device=u.device),
               torch.empty(M, 2 * F, dtype=torch.uint8, device=u.device),
               torch.zeros(nb, dtype=torch.uint8, device=u.device),
               torch.empty(1, dtype=torch.float32, device=u.device) if amax else None)
    h, codes, sf, am = out
    ldh = _mat(fn, h, torch.bfloat16, M, F)
    _arr(fn, codes, torch.uint8, M, 2 * F)
    _need(fn, sf.dtype == torch.uint8 and sf.is_contiguous() and sf.numel() >= nb)
    _arr(fn, am, torch.float32, 1)
    _need(fn, n_rows is None or (n_rows.dtype == torch.int32 and n_rows.numel() == 1))
    _dev(fn, u, n_rows, h, codes, sf, am)
    bsq.bsq_swiglu_ckpt(u, M, F, ldu, n_rows, h, ldh, codes, sf, am)
    return h, codes, sf, am


def swiglu_ckpt_bwd(dh, codes, sf, n_rows=None, recompute_h=False, out=None):
    """Gradient of swiglu_ckpt's u from dh [M, F] (bf16) and the checkpoint:
    (du [M, 2F] bf16, h [M, F] bf16 formed again from the checkpoint, or None)."""
    fn = "swiglu_ckpt_bwd"
    _need(fn, dh.dim() == 2)
    M, F = dh.shape
    lddh = _mat(fn, dh, torch.bfloat16, M, F)
    _arr(fn, codes, torch.uint8, M, 2 * F)
    _need(fn, sf.dtype == torch.uint8 and sf.is_contiguous() and sf.numel() >= sf_bytes(M, F // 16))
    _need(fn, n_rows is None or (n_rows.dtype == torch.int32 and n_rows.numel() == 1))
    if out is None:
        out = (torch.empty(M, 2 * F, dtype=torch.bfloat16, device=dh.device),
               torch.empty(M, F, dtype=torch.bfloat16, device=dh.device) if recompute_h else None)
    du, h = out
    lddu = _mat(fn, du, torch.bfloat16, M, 2 * F)
    ldh = _mat(fn, h, torch.bfloat16, M, F) if h is not None else 0
    _dev(fn, dh, codes, sf, n_rows, du, h)
    bsq.bsq_swiglu_ckpt_bwd(dh, lddh, codes, sf, M, F, n_rows, du, lddu, h, ldh)
    return du, h
