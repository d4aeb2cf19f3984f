"""Torch-tensor front end of ``libmi_moe`` (argument marshalling only).

The functions mirror the pages' Python signatures:

- :func:`grouped_mm_bf16`            -- flashinfer.grouped_mm.grouped_mm_bf16
- :func:`bgmv_moe_gemm2_lora_delta`  -- flashinfer.fused_moe.bgmv_moe_gemm2_lora_delta
- :func:`mm_nvfp4_lora`              -- flashinfer.gemm.mm_nvfp4_lora
- :func:`prepare_nvfp4_lora_adapter` -- flashinfer.gemm.prepare_nvfp4_lora_adapter

Every computation happens in the HIP library; tensors only provide device
memory and the current stream.  Inputs must already live on the GPU.
"""
from __future__ import annotations

import functools

import numpy as np
import torch

from . import _lib
from ._lib import MI_BF16, MI_F16, MI_F32, check

__all__ = [
    "grouped_mm_bf16",
    "grouped_mm_swiglu",
    "bgmv_moe_gemm2_lora_delta",
    "moe_finalize_lora",
    "moe_fc1_lora_delta",
    "moe_route_permutation",
    "moe_permute_rows",
    "route_workspace_bytes",
    "delta_workspace_bytes",
    "finalize_workspace_bytes",
    "fill_w_ptr",
    "mm_nvfp4_lora",
    "grouped_mm_nvfp4",
    "prepare_nvfp4_lora_adapter",
    "PreparedNvFp4LoraAdapter",
    "StaleAdapterError",
    "nvfp4_dequant",
    "fp4_quantize",
    "sf_bytes_needed",
    "fp8_scale_cols",
    "fp8_quantize",
    "add_rmsnorm_fp8",
    "mm_fp8_block",
    "grouped_mm_fp8_block",
    "moe_combine_rows",
    "moe_combine_rows_backward",
    "moe_permute_rows_backward",
    "mm_lora",
    "mm_lora_backward",
    "lora_mm_workspace_bytes",
    "moe_route_topk",
    "moe_balance_loss",
    "moe_route_backward",
    "balance_workspace_bytes",
]

_DT = {torch.bfloat16: MI_BF16, torch.float16: MI_F16, torch.float32: MI_F32}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev: torch.device):
    return torch.cuda.current_stream(dev).cuda_stream


def _need_cuda(name, *tensors):
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name}: all tensors must be on the GPU")


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


# ---------------------------------------------------------------------------
# grouped GEMM
# ---------------------------------------------------------------------------

def grouped_mm_bf16(a: torch.Tensor, b: torch.Tensor, m_indptr: torch.Tensor,
                    out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16, *,
                    backend: str = "auto", tactic: int = -1) -> torch.Tensor:
    """``out[m_indptr[e]:m_indptr[e+1]] = a[...] @ b[e]^T`` for every expert.

    ``a`` bf16 ``(cum_m, k)``, ``b`` bf16 ``(batch, n, k)``, ``m_indptr`` int32
    ``(batch+1,)`` read on the device.  Rows outside
    ``[m_indptr[0], m_indptr[-1])`` of a caller-provided ``out`` are untouched
    (a fresh ``out`` is zero-filled there).  ``backend`` is accepted for
    signature compatibility; there is one program and ``tactic`` must be -1.
    """
    _need(tactic == -1, "grouped_mm_bf16: tactic must be -1 (single program)")
    _need(a.dtype in (torch.bfloat16, torch.float16) and b.dtype == a.dtype,
          "grouped_mm_bf16: a and b must both be bfloat16 or both float16")
    _need(a.dim() == 2 and b.dim() == 3 and b.shape[2] == a.shape[1],
          "grouped_mm_bf16: a must be (cum_m, k) and b (batch_size, n, k)")
    _need(m_indptr.dtype == torch.int32 and m_indptr.shape == (b.shape[0] + 1,),
          "grouped_mm_bf16: m_indptr must be int32 of shape (batch_size + 1,)")
    _need(out_dtype in (torch.bfloat16, torch.float32, torch.float16),
          "grouped_mm_bf16: out_dtype must be bfloat16, float16 or float32")
    _need_cuda("grouped_mm_bf16", a, b, m_indptr, out)
    a, b, m_indptr = a.contiguous(), b.contiguous(), m_indptr.contiguous()
    if out is None:
        out = torch.zeros((a.shape[0], b.shape[1]), dtype=out_dtype, device=a.device)
    _need(out.shape == (a.shape[0], b.shape[1]) and out.dtype == out_dtype and out.is_contiguous(),
          "grouped_mm_bf16: out must be a contiguous (cum_m, n) tensor of out_dtype")
    check(_lib.lib().mi_grouped_mm_bf16(_ptr(a), a.shape[0], a.shape[1], _DT[a.dtype], _ptr(b),
                                        b.shape[0], b.shape[1], _ptr(m_indptr), _ptr(out),
                                        _DT[out_dtype], _stream(a.device)))
    return out


# ---------------------------------------------------------------------------
# FC2 LoRA delta
# ---------------------------------------------------------------------------

def grouped_mm_swiglu(a: torch.Tensor, b: torch.Tensor, m_indptr: torch.Tensor, *,
                      fc1_delta: torch.Tensor | None = None,
                      gemm1_alpha: torch.Tensor | None = None,
                      gemm1_beta: torch.Tensor | None = None,
                      gemm1_clamp_limit: torch.Tensor | None = None,
                      out: torch.Tensor | None = None,
                      out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """FC1 of a routed MoE: ``h = a @ b[e]^T (+ fc1_delta)`` per expert's rows,
    then ``out = g * sigmoid(alpha*g) * (u + beta)`` with ``g`` the clamped gate
    half and ``u`` the clamped up half of ``h`` (plain SwiGLU by default).

    ``a`` bf16/fp16 ``(cum_m, k)``, ``b`` ``(batch, 2I, k)`` (gate rows, then
    up rows), ``fc1_delta`` bf16 ``(cum_m, 2I)``, ``gemm1_*`` fp32 ``(batch,)``.
    Returns ``(cum_m, I)``; rows outside the groups of a caller-provided ``out``
    are untouched (a fresh ``out`` is zero-filled there).
    """
    _need(a.dtype in (torch.bfloat16, torch.float16) and b.dtype == a.dtype,
          "grouped_mm_swiglu: a and b must both be bfloat16 or both float16")
    _need(a.dim() == 2 and b.dim() == 3 and b.shape[2] == a.shape[1] and b.shape[1] % 2 == 0,
          "grouped_mm_swiglu: a must be (cum_m, k) and b (batch_size, 2*I, k)")
    _need(m_indptr.dtype == torch.int32 and m_indptr.shape == (b.shape[0] + 1,),
          "grouped_mm_swiglu: m_indptr must be int32 of shape (batch_size + 1,)")
    _need(out_dtype in (torch.bfloat16, torch.float32, torch.float16),
          "grouped_mm_swiglu: out_dtype must be bfloat16, float16 or float32")
    E, two_i = b.shape[0], b.shape[1]
    for name, t in (("gemm1_alpha", gemm1_alpha), ("gemm1_beta", gemm1_beta),
                    ("gemm1_clamp_limit", gemm1_clamp_limit)):
        _need(t is None or (t.dtype == torch.float32 and t.numel() == E),
              f"grouped_mm_swiglu: {name} must be float32 with one value per expert")
    _need(fc1_delta is None or (fc1_delta.dtype == torch.bfloat16 and
                                fc1_delta.shape == (a.shape[0], two_i)),
          "grouped_mm_swiglu: fc1_delta must be bfloat16 (cum_m, 2*I)")
    _need_cuda("grouped_mm_swiglu", a, b, m_indptr, fc1_delta, gemm1_alpha, gemm1_beta,
               gemm1_clamp_limit, out)
    a, b, m_indptr = a.contiguous(), b.contiguous(), m_indptr.contiguous()
    opt = [None if t is None else t.contiguous()
           for t in (fc1_delta, gemm1_alpha, gemm1_beta, gemm1_clamp_limit)]
    if out is None:
        out = torch.zeros((a.shape[0], two_i // 2), dtype=out_dtype, device=a.device)
    _need(out.shape == (a.shape[0], two_i // 2) and out.dtype == out_dtype and
          out.is_contiguous(),
          "grouped_mm_swiglu: out must be a contiguous (cum_m, I) tensor of out_dtype")
    check(_lib.lib().mi_grouped_mm_swiglu(
        _ptr(a), a.shape[0], a.shape[1], _DT[a.dtype], _ptr(b), E, two_i // 2, _ptr(m_indptr),
        *(_ptr(t) for t in opt), _ptr(out), _DT[out_dtype], _stream(a.device)))
    return out


def fill_w_ptr(bank: torch.Tensor) -> torch.Tensor:
    """Base-pointer table ``[1, E]`` (int64 byte addresses) of a contiguous
    ``[L, E, x, y]`` LoRA bank: entry e addresses adapter 0's ``[x, y]`` block
    of expert e; adapter l is ``lora_stride = E*x*y`` elements further."""
    _need(bank.dim() == 4 and bank.is_contiguous(), "fill_w_ptr: bank must be contiguous [L, E, x, y]")
    L, E, x, y = bank.shape
    step = x * y * bank.element_size()
    return (bank.data_ptr() + torch.arange(E, dtype=torch.int64) * step).reshape(1, E).to(
        bank.device)


def delta_workspace_bytes(num_tokens, top_k, num_experts, num_adapters, rank) -> int:
    return int(_lib.lib().mi_moe_fc2_lora_delta_workspace_size(num_tokens, top_k, num_experts,
                                                               num_adapters, rank))


def finalize_workspace_bytes(num_tokens, top_k, num_experts, num_adapters, rank,
                             hidden_size) -> int:
    """Workspace of the two-pass finalize (the delta's plus an fp32 [T, H] delta)."""
    return int(_lib.lib().mi_moe_fc2_finalize_workspace_size(num_tokens, top_k, num_experts,
                                                             num_adapters, rank, hidden_size))


def bgmv_moe_gemm2_lora_delta(gemm1_activation_output: torch.Tensor,
                              expanded_idx_to_permuted_idx: torch.Tensor, w_ptr_a: torch.Tensor,
                              lora_stride_a: int, w_ptr_b: torch.Tensor, lora_stride_b: int,
                              topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                              lora_ids: torch.Tensor, rank: int, hidden_size: int, *,
                              num_adapters: int, lora_dtype: torch.dtype = torch.bfloat16,
                              scale: float = 1.0, out_dtype: torch.dtype = torch.bfloat16,
                              out: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """FC2 LoRA delta ``[T, H]`` to be added to the MoE output.

    ``num_adapters`` is the number of adapters in the banks (ids at or above
    it are treated as no adapter); the other arguments follow the page.
    """
    return _delta_call(None, gemm1_activation_output, expanded_idx_to_permuted_idx, w_ptr_a,
                       lora_stride_a, w_ptr_b, lora_stride_b, topk_ids, topk_weights, lora_ids,
                       rank, hidden_size, num_adapters, lora_dtype, scale, out_dtype, out,
                       workspace)


def moe_finalize_lora(fc2_out: torch.Tensor, gemm1_activation_output: torch.Tensor,
                      expanded_idx_to_permuted_idx: torch.Tensor, w_ptr_a: torch.Tensor,
                      lora_stride_a: int, w_ptr_b: torch.Tensor, lora_stride_b: int,
                      topk_ids: torch.Tensor, topk_weights: torch.Tensor, lora_ids: torch.Tensor,
                      rank: int, hidden_size: int, *, num_adapters: int,
                      lora_dtype: torch.dtype = torch.bfloat16, scale: float = 1.0,
                      out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None) -> torch.Tensor:
    """MoE output ``[T, H]``: the routing-weighted combine of the FC2 rows
    (``fc2_out``, permuted ``[padded_rows, H]`` in bf16, fp16 or fp32) with
    the FC2 LoRA delta added, in one pass and one rounding.  The other
    arguments are those of :func:`bgmv_moe_gemm2_lora_delta`."""
    _need(isinstance(fc2_out, torch.Tensor) and fc2_out.dim() == 2 and
          fc2_out.shape[1] == hidden_size and
          fc2_out.shape[0] == gemm1_activation_output.shape[0],
          "moe_finalize_lora: fc2_out must be [padded_rows, hidden_size]")
    _need(fc2_out.dtype in _DT, "moe_finalize_lora: fc2_out must be bf16, fp16 or fp32")
    return _delta_call(fc2_out, gemm1_activation_output, expanded_idx_to_permuted_idx, w_ptr_a,
                       lora_stride_a, w_ptr_b, lora_stride_b, topk_ids, topk_weights, lora_ids,
                       rank, hidden_size, num_adapters, lora_dtype, scale, out_dtype, out,
                       workspace)


def _delta_call(fc2, act, perm, w_ptr_a, lora_stride_a, w_ptr_b, lora_stride_b, topk_ids,
                topk_weights, lora_ids, rank, hidden_size, num_adapters, lora_dtype, scale,
                out_dtype, out, workspace):
    _need(act.dim() == 2, "bgmv_moe_gemm2_lora_delta: activation must be [padded_rows, I]")
    _need(topk_ids.dim() == 2 and topk_weights.shape == topk_ids.shape,
          "bgmv_moe_gemm2_lora_delta: topk_ids / topk_weights must be [T, top_k]")
    T, top_k = topk_ids.shape
    _need(perm.numel() == T * top_k and perm.dtype == torch.int32,
          "bgmv_moe_gemm2_lora_delta: expanded_idx_to_permuted_idx must be int32 [T*top_k]")
    _need(topk_ids.dtype == torch.int32 and lora_ids.dtype == torch.int32 and
          topk_weights.dtype == torch.float32,
          "bgmv_moe_gemm2_lora_delta: ids must be int32 and topk_weights float32")
    _need(lora_ids.numel() == T, "bgmv_moe_gemm2_lora_delta: lora_ids must be [T]")
    _need(w_ptr_a.dtype == torch.int64 and w_ptr_b.dtype == torch.int64 and
          w_ptr_a.numel() == w_ptr_b.numel(),
          "bgmv_moe_gemm2_lora_delta: w_ptr_a / w_ptr_b must be int64 [1, num_experts]")
    _need(act.dtype == lora_dtype, "bgmv_moe_gemm2_lora_delta: activation dtype must be lora_dtype")
    _need(lora_dtype in _DT and out_dtype in _DT, "bgmv_moe_gemm2_lora_delta: unsupported dtype")
    _need_cuda("bgmv_moe_gemm2_lora_delta", act, perm, w_ptr_a, w_ptr_b, topk_ids, topk_weights,
               lora_ids, out, workspace, fc2)
    E = w_ptr_a.numel()
    act = act.contiguous()
    perm, topk_ids, topk_weights, lora_ids = (x.contiguous() for x in
                                             (perm, topk_ids, topk_weights, lora_ids))
    w_ptr_a, w_ptr_b = w_ptr_a.contiguous(), w_ptr_b.contiguous()
    if out is None:
        out = torch.empty((T, hidden_size), dtype=out_dtype, device=act.device)
    _need(out.shape == (T, hidden_size) and out.dtype == out_dtype and out.is_contiguous(),
          "bgmv_moe_gemm2_lora_delta: out must be a contiguous [T, H] tensor of out_dtype")
    need = delta_workspace_bytes(T, top_k, E, num_adapters, rank) if fc2 is None else \
        finalize_workspace_bytes(T, top_k, E, num_adapters, rank, hidden_size)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=act.device)
    args = (_ptr(act), act.shape[0], act.shape[1], _ptr(perm), _ptr(w_ptr_a), int(lora_stride_a),
            _ptr(w_ptr_b), int(lora_stride_b), _ptr(topk_ids), _ptr(topk_weights), _ptr(lora_ids),
            T, top_k, E, int(num_adapters), int(rank), int(hidden_size), _DT[lora_dtype],
            float(scale), _DT[out_dtype], _ptr(out), _ptr(workspace), workspace.numel(),
            _stream(act.device))
    if fc2 is None:
        check(_lib.lib().mi_moe_fc2_lora_delta(*args))
    else:
        fc2 = fc2.contiguous()
        check(_lib.lib().mi_moe_fc2_finalize_lora(_ptr(fc2), _DT[fc2.dtype], *args))
    return out


def moe_fc1_lora_delta(act: torch.Tensor, expanded_idx_to_permuted_idx: torch.Tensor,
                       w_ptr_a: torch.Tensor, lora_stride_a: int, w_ptr_b: torch.Tensor,
                       lora_stride_b: int, topk_ids: torch.Tensor, lora_ids: torch.Tensor,
                       rank: int, out_features: int, *, num_adapters: int,
                       lora_dtype: torch.dtype = torch.bfloat16, scale: float = 1.0,
                       out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None) -> torch.Tensor:
    """FC1 (gate/up) LoRA delta ``[padded_rows, out_features]``: row
    ``perm[t*top_k+j]`` is ``scale * B[l, e] @ (A[l, e] @ act[row])`` for
    each routed slot, +0 for a slot without adapter; the ``fc1_delta`` of
    :func:`grouped_mm_swiglu`.  A fresh ``out`` is zero-filled first, so rows
    no slot points at are 0; a caller's ``out`` keeps them."""
    _need(act.dim() == 2 and act.dtype == lora_dtype,
          "moe_fc1_lora_delta: act must be [padded_rows, hidden] of lora_dtype")
    _need(topk_ids.dim() == 2 and topk_ids.dtype == torch.int32 and lora_ids.dtype == torch.int32,
          "moe_fc1_lora_delta: topk_ids must be int32 [T, top_k] and lora_ids int32 [T]")
    T, top_k = topk_ids.shape
    perm = expanded_idx_to_permuted_idx
    _need(perm.numel() == T * top_k and perm.dtype == torch.int32 and lora_ids.numel() == T,
          "moe_fc1_lora_delta: expanded_idx_to_permuted_idx must be int32 [T*top_k]")
    _need(w_ptr_a.dtype == torch.int64 and w_ptr_b.dtype == torch.int64 and
          w_ptr_a.numel() == w_ptr_b.numel(),
          "moe_fc1_lora_delta: w_ptr_a / w_ptr_b must be int64 [1, num_experts]")
    _need(lora_dtype in (torch.bfloat16, torch.float16) and out_dtype in _DT,
          "moe_fc1_lora_delta: unsupported dtype")
    _need_cuda("moe_fc1_lora_delta", act, perm, w_ptr_a, w_ptr_b, topk_ids, lora_ids, out,
               workspace)
    E = w_ptr_a.numel()
    act = act.contiguous()
    perm, topk_ids, lora_ids = perm.contiguous(), topk_ids.contiguous(), lora_ids.contiguous()
    if out is None:
        out = torch.zeros((act.shape[0], out_features), dtype=out_dtype, device=act.device)
    _need(out.shape == (act.shape[0], out_features) and out.dtype == out_dtype and
          out.is_contiguous(), "moe_fc1_lora_delta: out must be a contiguous "
          "[padded_rows, out_features] tensor of out_dtype")
    need = int(_lib.lib().mi_moe_fc1_lora_delta_workspace_size(T, top_k, E, num_adapters, rank))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=act.device)
    check(_lib.lib().mi_moe_fc1_lora_delta(
        _ptr(act), act.shape[0], act.shape[1], _ptr(perm), _ptr(w_ptr_a.contiguous()),
        int(lora_stride_a), _ptr(w_ptr_b.contiguous()), int(lora_stride_b), _ptr(topk_ids),
        _ptr(lora_ids), T, top_k, E, int(num_adapters), int(rank), int(out_features),
        _DT[lora_dtype], float(scale), _DT[out_dtype], _ptr(out), _ptr(workspace),
        workspace.numel(), _stream(act.device)))
    return out


# ---------------------------------------------------------------------------
# routing output -> permutation, permuted rows
# ---------------------------------------------------------------------------

def route_workspace_bytes(num_slots: int, num_experts: int) -> int:
    return int(_lib.lib().mi_moe_route_workspace_size(num_slots, num_experts))


def moe_route_permutation(topk_ids: torch.Tensor, num_experts: int, *,
                          with_inverse: bool = False, workspace: torch.Tensor | None = None):
    """``(m_indptr, expanded_idx_to_permuted_idx[, permuted_idx_to_expanded_idx])``
    from ``topk_ids`` int32 ``[T, top_k]``: the slots sorted stably by expert
    id, ids outside ``[0, num_experts)`` left out (entry -1).  All int32 on
    the device; ``m_indptr`` is ``[num_experts + 1]``."""
    _need(topk_ids.dim() == 2 and topk_ids.dtype == torch.int32,
          "moe_route_permutation: topk_ids must be int32 [num_tokens, top_k]")
    _need_cuda("moe_route_permutation", topk_ids, workspace)
    T, top_k = topk_ids.shape
    dev = topk_ids.device
    topk_ids = topk_ids.contiguous()
    m_indptr = torch.empty(int(num_experts) + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(T * top_k, dtype=torch.int32, device=dev)
    inverse = torch.empty(T * top_k, dtype=torch.int32, device=dev) if with_inverse else None
    need = route_workspace_bytes(T * top_k, num_experts)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    check(_lib.lib().mi_moe_route_permutation(
        _ptr(topk_ids), T, top_k, int(num_experts), _ptr(m_indptr), _ptr(perm), _ptr(inverse),
        _ptr(workspace), workspace.numel(), _stream(dev)))
    return (m_indptr, perm, inverse) if with_inverse else (m_indptr, perm)


def moe_permute_rows(x: torch.Tensor, expanded_idx_to_permuted_idx: torch.Tensor, top_k: int,
                     out_rows: int | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """``out[perm[t*top_k + j]] = x[t]`` for every slot whose row lies in
    ``[0, out_rows)`` (other rows of ``out`` untouched; a fresh ``out`` is
    zero-filled).  ``x`` ``[T, ...]`` of any dtype, rows of a multiple of 16 bytes."""
    _need(x.dim() >= 1, "moe_permute_rows: x must be [num_tokens, ...]")
    perm = expanded_idx_to_permuted_idx
    _need(perm.dtype == torch.int32 and perm.numel() == x.shape[0] * int(top_k),
          "moe_permute_rows: expanded_idx_to_permuted_idx must be int32 [num_tokens*top_k]")
    _need_cuda("moe_permute_rows", x, perm, out)
    x, perm = x.contiguous(), perm.contiguous()
    if out is None:
        rows = perm.numel() if out_rows is None else int(out_rows)
        out = torch.zeros((rows,) + tuple(x.shape[1:]), dtype=x.dtype, device=x.device)
    _need(out.dtype == x.dtype and out.shape[1:] == x.shape[1:] and out.is_contiguous(),
          "moe_permute_rows: out must be contiguous [out_rows, ...] of x's dtype")
    row_bytes = x[0].numel() * x.element_size() if x.shape[0] else 16
    check(_lib.lib().mi_moe_permute_rows(_ptr(x), x.shape[0], row_bytes, _ptr(perm), int(top_k),
                                         _ptr(out), out.shape[0], _stream(x.device)))
    return out


# ---------------------------------------------------------------------------
# NVFP4 + LoRA
# ---------------------------------------------------------------------------

class StaleAdapterError(ValueError):
    """A prepared adapter's alpha or source tensors changed since the fold."""


def _pin(t: torch.Tensor):
    return (t.data_ptr(), t._version, tuple(t.shape), t.device, t.dtype)


class PreparedNvFp4LoraAdapter:
    """A folded LoRA-up weight ``b_folded = bf16(lora_b * lora_scale / alpha)``
    with its device zero-adapter flag and the snapshot pins of its sources."""

    def __init__(self, lora_b, lora_scale, alpha, b_folded, fold_flags):
        self.lora_b = lora_b
        self.lora_scale = lora_scale
        self.alpha = alpha
        self.b_folded = b_folded
        self.fold_flags = fold_flags
        self.refresh_pins()

    def refresh_pins(self):
        self._pins = (_pin(self.lora_b), _pin(self.lora_scale), _pin(self.alpha))

    def check_fresh(self, alpha):
        if alpha is not self.alpha:
            raise StaleAdapterError("mm_nvfp4_lora: the prepared adapter was folded for a different "
                                    "alpha tensor; re-prepare it for this call's alpha")
        if self._pins != (_pin(self.lora_b), _pin(self.lora_scale), _pin(self.alpha)):
            raise StaleAdapterError("mm_nvfp4_lora: lora_b, lora_scale or alpha changed since the "
                                    "adapter was prepared; re-prepare it")


def _fold(lora_b, lora_scale, alpha, b_folded, fold_flags):
    check(_lib.lib().mi_prepare_lora_fold(_ptr(lora_b), lora_b.shape[0], lora_b.shape[1],
                                          _ptr(lora_scale), _ptr(alpha), _ptr(b_folded),
                                          _ptr(fold_flags), _stream(lora_b.device)))


def prepare_nvfp4_lora_adapter(lora_b: torch.Tensor, lora_scale: torch.Tensor,
                               alpha: torch.Tensor, *,
                               out: PreparedNvFp4LoraAdapter | None = None
                               ) -> PreparedNvFp4LoraAdapter:
    """Fold one adapter for the prepared path.

    ``out=None``: lora_scale and alpha are read back to the host once; a zero
    alpha or a ratio that is not finite raises ValueError, otherwise the fold
    kernel runs.  ``out=adapter``: in-place refold with no host read; the
    alpha tensor has to be the one the adapter was prepared with, and lora_b
    keeps its shape and device.
    """
    _need(lora_b.dtype == torch.bfloat16 and lora_b.dim() == 2 and lora_b.is_contiguous(),
          "prepare_nvfp4_lora_adapter: lora_b must be contiguous bf16 [N, r]")
    _need(lora_scale.dtype == torch.float32 and lora_scale.numel() == 1,
          "prepare_nvfp4_lora_adapter: lora_scale must be an fp32 tensor of shape (1,)")
    _need(alpha.dtype == torch.float32 and alpha.numel() >= 1,
          "prepare_nvfp4_lora_adapter: alpha must be an fp32 device tensor")
    _need_cuda("prepare_nvfp4_lora_adapter", lora_b, lora_scale, alpha)
    if out is None:
        host = torch.cat([lora_scale.reshape(1), alpha.reshape(-1)[:1]]).cpu().numpy()
        s, a = np.float32(host[0]), np.float32(host[1])
        _need(a != 0, "prepare_nvfp4_lora_adapter: alpha == 0 is refused (lora_scale / alpha is "
                      "undefined); use the raw path for an alpha == 0 LoRA-only call")
        with np.errstate(all="ignore"):
            _need(np.isfinite(np.float32(s / a)),
                  "prepare_nvfp4_lora_adapter: lora_scale / alpha is not finite")
        b_folded = torch.empty_like(lora_b)
        flags = torch.zeros(1, dtype=torch.int32, device=lora_b.device)
        _fold(lora_b, lora_scale, alpha, b_folded, flags)
        return PreparedNvFp4LoraAdapter(lora_b, lora_scale, alpha, b_folded, flags)
    _need(alpha is out.alpha, "prepare_nvfp4_lora_adapter: alpha must be the tensor the adapter was prepared with")
    _need(lora_b.shape == out.b_folded.shape and lora_b.device == out.b_folded.device,
          "prepare_nvfp4_lora_adapter: lora_b must keep out's [N, r] shape and device")
    _fold(lora_b, lora_scale, alpha, out.b_folded, out.fold_flags)
    out.lora_b, out.lora_scale = lora_b, lora_scale
    out.refresh_pins()
    return out


def sf_bytes_needed(rows: int, k: int) -> int:
    return (-(-rows // 128)) * (-(-(k // 16) // 4)) * 512


def mm_nvfp4_lora(a: torch.Tensor, b: torch.Tensor, a_sf: torch.Tensor, b_sf: torch.Tensor,
                  alpha: torch.Tensor, d: torch.Tensor | None = None,
                  lora_b: torch.Tensor | None = None, lora_scale: torch.Tensor | None = None, *,
                  lora_adapter: PreparedNvFp4LoraAdapter | None = None,
                  bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  out_dtype: torch.dtype = torch.bfloat16, backend: str = "auto",
                  enable_pdl: bool | None = None) -> torch.Tensor:
    """NVFP4 base GEMM with a BF16 LoRA correction (raw or prepared path)."""
    _need(out_dtype == torch.bfloat16, "mm_nvfp4_lora: out_dtype must be torch.bfloat16")
    _need(a.dtype == torch.uint8 and b.dtype == torch.uint8 and a.dim() == 2 and b.dim() == 2,
          "mm_nvfp4_lora: a and b must be uint8 [M, K/2] and [N, K/2]")
    _need(a.shape[1] == b.shape[1], "mm_nvfp4_lora: a and b must have the same K")
    _need(a_sf.dtype == torch.uint8 and b_sf.dtype == torch.uint8,
          "mm_nvfp4_lora: a_sf / b_sf must be uint8")
    _need(alpha.dtype == torch.float32, "mm_nvfp4_lora: alpha must be an fp32 device tensor")
    raw_given = lora_b is not None or lora_scale is not None
    _need(not (lora_adapter is not None and raw_given),
          "mm_nvfp4_lora: pass either lora_b/lora_scale (raw path) or lora_adapter (prepared "
          "path), not both")
    _need_cuda("mm_nvfp4_lora", a, b, a_sf, b_sf, alpha, d, lora_b, lora_scale, bias, out)
    M, N, K = a.shape[0], b.shape[0], 2 * a.shape[1]
    a, b = a.contiguous(), b.contiguous()
    _need(a_sf.is_contiguous() and b_sf.is_contiguous(), "mm_nvfp4_lora: scale buffers must be "
          "contiguous")
    rank = 0
    d_ptr = lb_ptr = ls_ptr = bf_ptr = ff_ptr = None
    if lora_adapter is not None:
        _need(d is not None, "mm_nvfp4_lora: the prepared path requires d")
        lora_adapter.check_fresh(alpha)
        d_ptr, bf_ptr, ff_ptr = _ptr(d), _ptr(lora_adapter.b_folded), _ptr(lora_adapter.fold_flags)
        _need(lora_adapter.b_folded.shape == (N, d.shape[1]),
              "mm_nvfp4_lora: prepared adapter must be [N, r] with r = d.shape[1]")
        rank = d.shape[1]
    elif lora_scale is not None:
        _need(d is not None and lora_b is not None,
              "mm_nvfp4_lora: lora_scale needs d and lora_b (raw path)")
        _need(lora_scale.dtype == torch.float32 and lora_scale.numel() == 1,
              "mm_nvfp4_lora: lora_scale must be a one-element fp32 device tensor")
        _need(lora_b.dtype == torch.bfloat16 and lora_b.is_contiguous() and
              lora_b.shape == (N, d.shape[1]),
              "mm_nvfp4_lora: lora_b must be contiguous bf16 [N, r] (transpose a [r, N] factor)")
        d_ptr, lb_ptr, ls_ptr = _ptr(d), _ptr(lora_b), _ptr(lora_scale)
        rank = d.shape[1]
    if d_ptr is not None:
        _need(d.dtype == torch.bfloat16 and d.is_contiguous() and d.shape[0] == M,
              "mm_nvfp4_lora: d must be contiguous bf16 [M, r]")
    if bias is not None:
        _need(bias.dtype == torch.bfloat16 and bias.numel() == N and bias.is_contiguous(),
              "mm_nvfp4_lora: bias must be contiguous bf16 [N]")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _need(out.shape == (M, N) and out.dtype == torch.bfloat16 and out.is_contiguous(),
          "mm_nvfp4_lora: out must be a contiguous bf16 [M, N] tensor")
    check(_lib.lib().mi_mm_nvfp4_lora(_ptr(a), _ptr(b), _ptr(a_sf), a_sf.numel(), _ptr(b_sf),
                                      b_sf.numel(), _ptr(alpha), M, N, K, d_ptr, rank, lb_ptr,
                                      ls_ptr, bf_ptr, ff_ptr, _ptr(bias), _ptr(out),
                                      _stream(a.device)))
    return out


def grouped_mm_nvfp4(a: torch.Tensor, a_sf: torch.Tensor, b: torch.Tensor, b_sf: torch.Tensor,
                     m_indptr: torch.Tensor, alpha: torch.Tensor,
                     out: torch.Tensor | None = None,
                     out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """``out[m_indptr[e]:m_indptr[e+1]] = alpha[e] * dequant(a[...]) @ dequant(b[e])^T``.

    ``a`` uint8 ``(cum_m, k/2)`` with its 128x4 scales ``a_sf`` over all
    rows; ``b`` uint8 ``(batch, n, k/2)`` with ``b_sf`` holding one 128x4
    scale buffer per expert; ``alpha`` fp32 ``(batch,)``; ``m_indptr`` int32
    ``(batch+1,)`` read on the device.  Rows outside the groups of a
    caller-provided ``out`` are untouched (a fresh ``out`` is zero-filled there).
    """
    _need(a.dtype == torch.uint8 and b.dtype == torch.uint8 and a.dim() == 2 and b.dim() == 3
          and b.shape[2] == a.shape[1],
          "grouped_mm_nvfp4: a must be uint8 (cum_m, k/2) and b uint8 (batch_size, n, k/2)")
    _need(a_sf.dtype == torch.uint8 and b_sf.dtype == torch.uint8,
          "grouped_mm_nvfp4: scale buffers must be uint8")
    _need(m_indptr.dtype == torch.int32 and m_indptr.shape == (b.shape[0] + 1,),
          "grouped_mm_nvfp4: m_indptr must be int32 of shape (batch_size + 1,)")
    _need(alpha.dtype == torch.float32 and alpha.numel() == b.shape[0],
          "grouped_mm_nvfp4: alpha must be float32 with one value per expert")
    _need(out_dtype in (torch.bfloat16, torch.float32),
          "grouped_mm_nvfp4: out_dtype must be bfloat16 or float32")
    _need_cuda("grouped_mm_nvfp4", a, a_sf, b, b_sf, m_indptr, alpha, out)
    cum_m, k = a.shape[0], a.shape[1] * 2
    n = b.shape[1]
    a, b, a_sf, b_sf = a.contiguous(), b.contiguous(), a_sf.contiguous(), b_sf.contiguous()
    m_indptr, alpha = m_indptr.contiguous(), alpha.contiguous()
    if out is None:
        out = torch.zeros((cum_m, n), dtype=out_dtype, device=a.device)
    _need(out.shape == (cum_m, n) and out.dtype == out_dtype and out.is_contiguous(),
          "grouped_mm_nvfp4: out must be a contiguous (cum_m, n) tensor of out_dtype")
    check(_lib.lib().mi_grouped_mm_nvfp4(
        _ptr(a), _ptr(a_sf), a_sf.numel(), cum_m, k, _ptr(b), _ptr(b_sf), b_sf.numel(),
        b.shape[0], n, _ptr(m_indptr), _ptr(alpha), _ptr(out), _DT[out_dtype],
        _stream(a.device)))
    return out


def nvfp4_dequant(codes: torch.Tensor, sf: torch.Tensor, k: int | None = None) -> torch.Tensor:
    """bf16 ``[rows, K]`` dequantisation with the GEMM's own decoder."""
    _need(codes.dtype == torch.uint8 and codes.dim() == 2 and sf.dtype == torch.uint8,
          "nvfp4_dequant: codes [rows, K/2] and sf must be uint8")
    _need_cuda("nvfp4_dequant", codes, sf)
    k = 2 * codes.shape[1] if k is None else k
    out = torch.empty((codes.shape[0], k), dtype=torch.bfloat16, device=codes.device)
    check(_lib.lib().mi_nvfp4_dequant_bf16(_ptr(codes.contiguous()), _ptr(sf), sf.numel(),
                                           codes.shape[0], k, _ptr(out), _stream(codes.device)))
    return out


def fp4_quantize(x: torch.Tensor, global_scale: torch.Tensor, *, codes: torch.Tensor | None = None,
                 sf: torch.Tensor | None = None):
    """NVFP4 quantisation of ``x`` (bf16 / fp16 / fp32, ``[rows, K]`` or a batch
    ``[B, rows, K]`` of matrices) with fp32 global scale(s) ``global_scale``
    (one per matrix).  Returns ``(codes, sf)``: uint8 ``[..., rows, K/2]`` and
    the 128x4 scale buffer(s) (one per matrix, concatenated), the operands
    of :func:`mm_nvfp4_lora` / :func:`grouped_mm_nvfp4`."""
    _need(x.dtype in _DT and x.dim() in (2, 3), "fp4_quantize: x must be a bf16, fp16 or fp32 "
          "[rows, K] or [B, rows, K] tensor")
    _need_cuda("fp4_quantize", x, global_scale, codes, sf)
    batch = 1 if x.dim() == 2 else x.shape[0]
    rows, k = x.shape[-2], x.shape[-1]
    _need(global_scale.dtype == torch.float32 and global_scale.numel() == batch,
          "fp4_quantize: global_scale must be fp32 with one value per matrix")
    x = x.contiguous()
    per = (-(-rows // 128)) * (k // 64) * 512
    if codes is None:
        codes = torch.empty((*x.shape[:-1], k // 2), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty(batch * per, dtype=torch.uint8, device=x.device)
    _need(codes.dtype == torch.uint8 and codes.shape == (*x.shape[:-1], k // 2) and
          codes.is_contiguous(), "fp4_quantize: codes must be contiguous uint8 [..., rows, K/2]")
    _need(sf.dtype == torch.uint8 and sf.is_contiguous(), "fp4_quantize: sf must be contiguous uint8")
    check(_lib.lib().mi_fp4_quantize(_ptr(x), batch, rows, k, _DT[x.dtype],
                                     _ptr(global_scale.contiguous()), _ptr(codes), _ptr(sf),
                                     sf.numel(), _stream(x.device)))
    return codes, sf


# ---------------------------------------------------------------------------
# 8-bit block-scaled operands
# ---------------------------------------------------------------------------

_F8 = torch.float8_e4m3fn


def _one_gpu(name, first, *others):
    """The index of the GPU that all of them (None aside) are on."""
    i = first.get_device()
    for t in others:
        if t is not None and t.get_device() != i:
            _need_cuda(name, first, t)
            raise ValueError(f"{name}: all tensors must be on the same GPU")
    if i < 0:
        _need_cuda(name, first)
    return i


def _launch(i, fn, *args):
    """Enqueue on GPU `i`'s current stream, with `i` the current device for the launch.

    torch's own accessors give the device and the stream's handle without a Stream
    object around it (1.9 us less a call).  They are looked up here: a torch without
    GPU support has none, and its tensors are refused before this."""
    c = torch._C
    if c._cuda_getDevice() == i:
        status = fn(*args, c._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(i):
            status = fn(*args, c._cuda_getCurrentRawStream(i))
    if status:
        check(status)


def fp8_scale_cols(k: int) -> int:
    """Columns of the scale rows of ``k`` values: one per 128, padded to a multiple of 4."""
    return 4 * (-(-k // 512))


def _fp8_out(name, x, codes, scales, codes_shape, scale_shape):
    if codes is None:
        codes = (torch.empty_like(x, dtype=_F8) if x.shape == codes_shape and x.is_contiguous()
                 else torch.empty(codes_shape, dtype=_F8, device=x.device))
    elif not (codes.dtype == _F8 and codes.shape == codes_shape and codes.is_contiguous()):
        raise ValueError(f"{name}: codes must be contiguous float8_e4m3fn of shape "
                         f"{tuple(codes_shape)}")
    if scales is None:
        scales = torch.empty(scale_shape, dtype=torch.float32, device=x.device)
    elif not (scales.dtype == torch.float32 and scales.shape == scale_shape and
              scales.is_contiguous()):
        raise ValueError(f"{name}: scales must be contiguous float32 of shape "
                         f"{tuple(scale_shape)}")
    return codes, scales


def _own_out(name, what, out, shape, dtype):
    """A caller's output tensor."""
    if not (out.shape == shape and out.dtype == dtype and out.is_contiguous()):
        raise ValueError(f"{name}: out must be a contiguous {what} tensor of out_dtype")


def fp8_quantize(x: torch.Tensor, *, block_rows: int = 1, swiglu: bool = False,
                 codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """``(codes, scales)`` of ``x`` (bf16 / fp16 / fp32, ``[rows, K]`` or ``[B, rows, K]``):
    float8_e4m3fn codes of its shape and fp32 scales ``amax / 448`` of every
    block, the operands of :func:`mm_fp8_block` and :func:`grouped_mm_fp8_block`.

    ``block_rows=1``: a scale per row and 128 columns (activations), scales
    ``[..., rows, fp8_scale_cols(K)]``; ``block_rows=128``: one per 128 x 128
    block (weights), ``[..., ceil(rows / 128), fp8_scale_cols(K)]``.  With
    ``swiglu`` (``block_rows=1``) the rows of ``x`` are ``[gate | up]`` of
    ``2K`` columns and ``silu(gate) * up`` is quantised.  K is a multiple of 16.
    """
    _need(x.dtype in _DT and x.dim() in (2, 3), "fp8_quantize: x must be a bf16, fp16 or fp32 "
          "[rows, K] or [B, rows, K] tensor")
    _need(block_rows in (1, 128), "fp8_quantize: block_rows must be 1 or 128")
    gpu = _one_gpu("fp8_quantize", x, codes, scales)
    rows, k = x.shape[-2], x.shape[-1]
    if swiglu:
        _need(k % 2 == 0, "fp8_quantize: swiglu needs rows [gate | up]")
        k //= 2
    lead = x.shape[:-2]
    codes, scales = _fp8_out("fp8_quantize", x, codes, scales, (*lead, rows, k),
                             (*lead, -(-rows // block_rows), fp8_scale_cols(k)))
    x = x.contiguous()
    _launch(gpu, _lib.lib().mi_fp8_quantize, x.data_ptr(), lead[0] if lead else 1, rows, k,
            _DT[x.dtype], block_rows, int(swiglu), codes.data_ptr(), scales.data_ptr())
    return codes, scales


def add_rmsnorm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                    *, eps: float = 1e-6, with_norm: bool = False,
                    codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                    residual_out: torch.Tensor | None = None,
                    norm_out: torch.Tensor | None = None):
    """``h = x + residual``, ``y = h / sqrt(mean(h^2) + eps) * weight`` and the 1 x 128
    quantisation of ``y``: ``(codes, scales, residual_out)``, with ``y`` itself in
    ``x``'s type as a fourth where ``with_norm`` is set or ``norm_out`` is given.

    ``x`` (and ``residual``) ``[T, H]`` bf16, fp16 or fp32; ``weight`` ``[H]`` of
    that type or fp32.  ``residual_out`` is ``h`` rounded once (the norm uses the
    unrounded sum); it may be ``residual`` or ``x`` itself, and is None without a
    residual.
    """
    _need(x.dim() == 2 and x.dtype in _DT, "add_rmsnorm_fp8: x must be [T, H] bf16, fp16 or fp32")
    T, H = x.shape
    _need(weight.shape == (H,) and weight.dtype in (x.dtype, torch.float32),
          "add_rmsnorm_fp8: weight must be [H] of x's type or float32")
    _need(residual is None or (residual.shape == x.shape and residual.dtype == x.dtype),
          "add_rmsnorm_fp8: residual must have x's shape and type")
    _need(residual is not None or residual_out is None,
          "add_rmsnorm_fp8: residual_out needs a residual")
    gpu = _one_gpu("add_rmsnorm_fp8", x, weight, residual, codes, scales, residual_out, norm_out)
    codes, scales = _fp8_out("add_rmsnorm_fp8", x, codes, scales, (T, H), (T, fp8_scale_cols(H)))
    for t in (residual_out, norm_out):
        _need(t is None or (t.shape == x.shape and t.dtype == x.dtype and t.is_contiguous()),
              "add_rmsnorm_fp8: residual_out and norm_out must be contiguous with x's shape "
              "and type")
    x, weight = x.contiguous(), weight.contiguous()
    if residual is not None:
        residual = residual.contiguous()
        if residual_out is None:
            residual_out = torch.empty_like(x)
    if norm_out is None and with_norm:
        norm_out = torch.empty_like(x)
    _launch(gpu, _lib.lib().mi_add_rmsnorm_fp8, x.data_ptr(), _ptr(residual),
            weight.data_ptr(), _DT[x.dtype], _DT[weight.dtype], T, H, float(eps),
            _ptr(residual_out), _ptr(norm_out), codes.data_ptr(), scales.data_ptr())
    return (codes, scales, residual_out) if norm_out is None else \
        (codes, scales, residual_out, norm_out)


def mm_fp8_block(a: torch.Tensor, b: torch.Tensor, a_scale: torch.Tensor, b_scale: torch.Tensor,
                 *, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """``(a * a_scale) @ (b * b_scale)^T`` of e4m3 codes with a scale per block of 128.

    ``a`` float8_e4m3fn ``[M, K]`` with fp32 ``a_scale`` ``[M, fp8_scale_cols(K)]``
    (1 x 128 blocks), ``b`` ``[N, K]`` with ``b_scale`` ``[ceil(N / 128),
    fp8_scale_cols(K)]`` (128 x 128 blocks); N and K multiples of 16, any M.
    One rounding to ``out_dtype`` (bf16, fp16 or fp32).  With float32 the sums are
    fp32 throughout.  For 16-bit outputs the 8-bit matrix instruction adds every 8
    consecutive products in 13 bits below the largest of them: off by at most
    ``7 * 2**-13`` of that product for each 8, 2e-5 of the outputs' rms on normally
    distributed codes, 1e-4 with large outlier columns.  For fp32 sums in a 16-bit
    result ask for float32 and convert.

    The gradient of the rows is the same product: the output's gradient, quantised
    with ``block_rows=1``, times ``b.t()`` with the scales ``b_scale[:, :ceil(K / 128)].t()``
    padded with zeros to ``fp8_scale_cols(N)`` columns.
    """
    _need(a.dtype == _F8 and b.dtype == _F8 and a.dim() == 2 and b.dim() == 2 and
          a.shape[1] == b.shape[1],
          "mm_fp8_block: a and b must be float8_e4m3fn [M, K] and [N, K]")
    (M, K), N = a.shape, b.shape[0]
    cols = fp8_scale_cols(K)
    _need(a_scale.dtype == torch.float32 and a_scale.shape == (M, cols),
          "mm_fp8_block: a_scale must be float32 (M, fp8_scale_cols(K))")
    _need(b_scale.dtype == torch.float32 and b_scale.shape == (-(-N // 128), cols),
          "mm_fp8_block: b_scale must be float32 (ceil(N / 128), fp8_scale_cols(K))")
    _need(out_dtype in _DT, "mm_fp8_block: out_dtype must be bfloat16, float16 or float32")
    gpu = _one_gpu("mm_fp8_block", a, b, a_scale, b_scale, out)
    a, b, a_scale, b_scale = (a.contiguous(), b.contiguous(), a_scale.contiguous(),
                              b_scale.contiguous())
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    else:
        _own_out("mm_fp8_block", "(M, N)", out, (M, N), out_dtype)
    _launch(gpu, _lib.lib().mi_mm_fp8_block, a.data_ptr(), a_scale.data_ptr(), M, K,
            b.data_ptr(), b_scale.data_ptr(), N, out.data_ptr(), _DT[out_dtype])
    return out


def grouped_mm_fp8_block(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor,
                         b_scale: torch.Tensor, m_indptr: torch.Tensor,
                         out: torch.Tensor | None = None,
                         out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """:func:`mm_fp8_block` of every expert's rows ``m_indptr[e] : m_indptr[e+1]`` with ``b[e]``.

    ``a`` ``(cum_m, K)`` and ``a_scale`` ``(cum_m, fp8_scale_cols(K))``, ``b``
    ``(batch, N, K)`` and ``b_scale`` ``(batch, ceil(N / 128), fp8_scale_cols(K))``,
    ``m_indptr`` int32 ``(batch+1,)`` read on the device.  Rows outside the
    groups of a caller-provided ``out`` are untouched (a fresh ``out`` is
    zero-filled there).  The sums have the precision that :func:`mm_fp8_block`
    states: fp32 for float32 outputs, fewer bits for 16-bit ones.  The rows' gradient
    is given there too, with ``b.transpose(1, 2)`` and each expert's scales so.
    """
    _need(a.dtype == _F8 and b.dtype == _F8 and a.dim() == 2 and b.dim() == 3 and
          a.shape[1] == b.shape[2],
          "grouped_mm_fp8_block: a and b must be float8_e4m3fn (cum_m, K) and (batch, N, K)")
    (M, K), (E, N) = a.shape, b.shape[:2]
    cols = fp8_scale_cols(K)
    _need(a_scale.dtype == torch.float32 and a_scale.shape == (M, cols),
          "grouped_mm_fp8_block: a_scale must be float32 (cum_m, fp8_scale_cols(K))")
    _need(b_scale.dtype == torch.float32 and b_scale.shape == (E, -(-N // 128), cols),
          "grouped_mm_fp8_block: b_scale must be float32 (batch, ceil(N / 128), "
          "fp8_scale_cols(K))")
    _need(m_indptr.dtype == torch.int32 and m_indptr.shape == (E + 1,),
          "grouped_mm_fp8_block: m_indptr must be int32 of shape (batch_size + 1,)")
    _need(out_dtype in _DT, "grouped_mm_fp8_block: out_dtype must be bfloat16, float16 or float32")
    gpu = _one_gpu("grouped_mm_fp8_block", a, a_scale, b, b_scale, m_indptr, out)
    a, a_scale, b, b_scale, m_indptr = (a.contiguous(), a_scale.contiguous(), b.contiguous(),
                                        b_scale.contiguous(), m_indptr.contiguous())
    fresh = out is None
    if fresh:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    else:
        _own_out("grouped_mm_fp8_block", "(cum_m, N)", out, (M, N), out_dtype)
    _launch(gpu, _lib.lib().mi_grouped_mm_fp8_block, a.data_ptr(), a_scale.data_ptr(), M, K,
            b.data_ptr(), b_scale.data_ptr(), E, N, m_indptr.data_ptr(), int(fresh),
            out.data_ptr(), _DT[out_dtype])
    return out


# ---------------------------------------------------------------------------
# permuted rows -> token rows, and the gradients
# ---------------------------------------------------------------------------

def _combine(name, rows, perm, weights, T, top_k, out_dtype, out):
    out_dtype = rows.dtype if out_dtype is None else out_dtype
    if not (rows.dim() == 2 and rows.dtype in _DT and out_dtype in _DT):
        raise ValueError(f"{name}: the rows must be [num_rows, H] bf16, fp16 or fp32, and "
                         "out_dtype one of them")
    if not (perm.dtype == torch.int32 and perm.numel() == T * top_k):
        raise ValueError(f"{name}: expanded_idx_to_permuted_idx must be int32 "
                         "[num_tokens*top_k]")
    gpu = _one_gpu(name, rows, perm, weights, out)
    rows, perm = rows.contiguous(), perm.contiguous()
    weights = None if weights is None else weights.contiguous()
    P, H = rows.shape
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=rows.device)
    else:
        _own_out(name, "[T, H]", out, (T, H), out_dtype)
    _launch(gpu, _lib.lib().mi_moe_combine_rows, rows.data_ptr(), _DT[rows.dtype], P, H,
            perm.data_ptr(), _ptr(weights), T, top_k, out.data_ptr(), _DT[out_dtype])
    return out


def moe_combine_rows(rows: torch.Tensor, expanded_idx_to_permuted_idx: torch.Tensor,
                     topk_weights: torch.Tensor, *, out_dtype: torch.dtype | None = None,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """``out[t] = sum_j topk_weights[t, j] * rows[perm[t*top_k + j]]``: ``rows``
    (bf16, fp16 or fp32 ``[num_rows, H]``, permuted order) back in token order
    ``[T, H]``.  Slots whose entry lies outside ``[0, num_rows)`` contribute
    nothing.  fp32 sums in slot order, one rounding to ``out_dtype`` (the
    rows' type by default).  ``topk_weights`` fp32 ``[T, top_k]``.  Slots may share
    a row here; :func:`moe_combine_rows_backward` needs one row a slot."""
    _need(topk_weights.dim() == 2 and topk_weights.dtype == torch.float32 and
          topk_weights.shape[1] >= 1, "moe_combine_rows: topk_weights must be float32 [T, top_k]")
    T, top_k = topk_weights.shape
    return _combine("moe_combine_rows", rows, expanded_idx_to_permuted_idx, topk_weights, T,
                    top_k, out_dtype, out)


def moe_permute_rows_backward(grad_rows: torch.Tensor, expanded_idx_to_permuted_idx: torch.Tensor,
                              top_k: int, *, out_dtype: torch.dtype | None = None,
                              out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of :func:`moe_permute_rows` with respect to ``x``:
    ``out[t] = sum_j grad_rows[perm[t*top_k + j]]`` over the token's slots
    that have a row, fp32 sums, one rounding."""
    top_k = int(top_k)
    n = expanded_idx_to_permuted_idx.numel()
    _need(top_k >= 1 and n % top_k == 0,
          "moe_permute_rows_backward: expanded_idx_to_permuted_idx must hold num_tokens*top_k "
          "entries")
    return _combine("moe_permute_rows_backward", grad_rows, expanded_idx_to_permuted_idx, None,
                    n // top_k, top_k, out_dtype, out)


def moe_combine_rows_backward(grad_out: torch.Tensor, rows: torch.Tensor,
                              expanded_idx_to_permuted_idx: torch.Tensor,
                              topk_weights: torch.Tensor, *,
                              permuted_idx_to_expanded_idx: torch.Tensor | None = None,
                              with_weights: bool = True,
                              grad_rows: torch.Tensor | None = None,
                              grad_weights: torch.Tensor | None = None):
    """``(grad_rows, grad_weights)`` of :func:`moe_combine_rows` for ``grad_out`` ``[T, H]``:
    ``grad_rows[perm[t*top_k + j]] = topk_weights[t, j] * grad_out[t]`` in the rows'
    type and ``grad_weights[t, j] = <rows[perm[t*top_k + j]], grad_out[t]>`` in
    fp32 (0 for a slot without a row; None with ``with_weights=False``, which
    does not read the rows).

    With ``permuted_idx_to_expanded_idx`` (the inverse that
    :func:`moe_route_permutation` returns, one entry per row) the call writes
    every row: the gradient of the slot the inverse names, zeros where that slot
    does not point at the row (it was taken out of the permutation) or there is
    none.  Without it rows no slot points at are zero in a fresh ``grad_rows`` and
    untouched in a caller's.  Each row may be pointed at once: of two slots that
    share a row, ``grad_rows`` has the named slot's gradient, not the sum (without
    the inverse either's, element by element).
    """
    name = "moe_combine_rows_backward"
    _need(rows.dim() == 2 and rows.dtype in _DT,
          "moe_combine_rows_backward: rows must be [num_rows, H] bf16, fp16 or fp32")
    _need(topk_weights.dim() == 2 and topk_weights.dtype == torch.float32 and
          topk_weights.shape[1] >= 1, "moe_combine_rows_backward: topk_weights must be float32 [T, top_k]")
    T, top_k = topk_weights.shape
    P, H = rows.shape
    _need(grad_out.shape == (T, H) and grad_out.dtype in _DT,
          "moe_combine_rows_backward: grad_out must be [T, H] bf16, fp16 or fp32")
    perm, inverse = expanded_idx_to_permuted_idx, permuted_idx_to_expanded_idx
    _need(perm.dtype == torch.int32 and perm.numel() == T * top_k,
          "moe_combine_rows_backward: expanded_idx_to_permuted_idx must be int32 [num_tokens*top_k]")
    _need(inverse is None or (inverse.dtype == torch.int32 and inverse.numel() == P),
          "moe_combine_rows_backward: permuted_idx_to_expanded_idx must be int32 [num_rows]")
    _need(with_weights or grad_weights is None, "moe_combine_rows_backward: grad_weights needs with_weights")
    gpu = _one_gpu(name, rows, grad_out, perm, topk_weights, inverse, grad_rows, grad_weights)
    grad_out, rows, perm, topk_weights = (grad_out.contiguous(), rows.contiguous(),
                                          perm.contiguous(), topk_weights.contiguous())
    inverse = None if inverse is None else inverse.contiguous()
    if grad_rows is None:
        grad_rows = (torch.zeros_like if inverse is None else torch.empty_like)(rows)
    if grad_weights is None and with_weights:
        grad_weights = torch.empty_like(topk_weights)
    _need(grad_rows.shape == rows.shape and grad_rows.dtype == rows.dtype and
          grad_rows.is_contiguous(), "moe_combine_rows_backward: grad_rows must be contiguous like rows")
    _need(grad_weights is None or (grad_weights.shape == topk_weights.shape and
                                   grad_weights.dtype == torch.float32 and
                                   grad_weights.is_contiguous()),
          "moe_combine_rows_backward: grad_weights must be contiguous float32 [T, top_k]")
    _launch(gpu, _lib.lib().mi_moe_combine_rows_backward, grad_out.data_ptr(),
            _DT[grad_out.dtype], rows.data_ptr(), _DT[rows.dtype], P, H, perm.data_ptr(),
            _ptr(inverse), topk_weights.data_ptr(), T, top_k, grad_rows.data_ptr(),
            _ptr(grad_weights))
    return grad_rows, grad_weights


# ---------------------------------------------------------------------------
# a projection with low-rank adapters
# ---------------------------------------------------------------------------

_HALF = (torch.bfloat16, torch.float16)


class _Devices(dict):
    """Device objects by index (making one costs as much as a check)."""

    def __missing__(self, i):
        self[i] = d = torch.device("cuda", i)
        return d


_CUDA = _Devices()


@functools.lru_cache(maxsize=1024)
def _lora_mm_bytes(m, n, k, num_adapters, rank, backward):
    return int(_lib.lib().mi_mm_lora_workspace_size(m, n, k, num_adapters, rank, backward))


def lora_mm_workspace_bytes(m, n, k, num_adapters, rank, *, backward: bool = False) -> int:
    """Workspace of :func:`mm_lora` (or of :func:`mm_lora_backward`) for ``m`` rows or fewer; 0 for
    sizes they refuse."""
    return _lora_mm_bytes(m, n, k, num_adapters, rank, int(backward))


def _lora_operands(name, rows, cols, w, lora_a, lora_b, lora_ids, lora_scale):
    """(M, K, N, L, R) of x (or grad_out, of `cols` columns) and the adapters' operands."""
    if not (rows.dim() == 2 and rows.dtype in _HALF):
        raise ValueError(f"{name}: the rows must be a bfloat16 or float16 matrix")
    if not (w.dim() == 2 and w.dtype == rows.dtype and w.shape[cols] == rows.shape[1]):
        raise ValueError(f"{name}: w must be [N, K] of the rows' type")
    (N, K), M = w.shape, rows.shape[0]
    if not (lora_a.dim() == 3 and lora_a.dtype == rows.dtype and lora_a.shape[2] == K):
        raise ValueError(f"{name}: lora_a must be [L, R, K] of the rows' type")
    L, R = lora_a.shape[:2]
    if not (lora_b.shape == (L, N, R) and lora_b.dtype == rows.dtype):
        raise ValueError(f"{name}: lora_b must be [L, N, R] of the rows' type")
    if not (lora_ids.dtype == torch.int32 and lora_ids.shape == (M,)):
        raise ValueError(f"{name}: lora_ids must be int32 [M]")
    if not (lora_scale is None or (lora_scale.dtype == torch.float32 and
                                   lora_scale.shape == (L,))):
        raise ValueError(f"{name}: lora_scale must be float32 [L]")
    return M, K, N, L, R


def _given(name, what, t, shape, dtype, gpu):
    """A caller's output tensor, or a new one on GPU `gpu`."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=_CUDA[gpu])
    if not (t.shape == shape and t.dtype == dtype and t.is_contiguous()):
        raise ValueError(f"{name}: {what} must be contiguous {dtype} of shape {tuple(shape)}")
    return t


def _workspace(name, workspace, need, gpu):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=_CUDA[gpu])
    if not (workspace.dtype == torch.uint8 and workspace.is_contiguous()):
        raise ValueError(f"{name}: workspace must be a contiguous uint8 tensor")
    return workspace


def mm_lora(x: torch.Tensor, w: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
            lora_ids: torch.Tensor, lora_scale: torch.Tensor | None = None, *,
            bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
            out_dtype: torch.dtype | None = None, with_act: bool = False,
            act: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """``out[t] = x[t] @ w^T + bias + lora_scale[l] * (x[t] @ lora_a[l]^T) @ lora_b[l]^T``
    with ``l = lora_ids[t]``: a projection that many requests share, each with its own
    low-rank adapter.

    ``x`` bf16 or fp16 ``[M, K]``, ``w`` ``[N, K]``, ``lora_a`` ``[L, R, K]``, ``lora_b``
    ``[L, N, R]`` and ``bias`` ``[N]`` of that type; ``lora_ids`` int32 ``[M]`` in any order,
    a row whose id lies outside ``[0, L)`` has the projection alone; ``lora_scale`` fp32
    ``[L]`` (default 1).  K, N and R are multiples of 8, R at most 256, L at most 1024.
    fp32 sums, one rounding to ``out_dtype`` (x's type, the default, or float32).

    With ``with_act`` (or a tensor ``act``) the call returns ``(out, act)``: ``act`` fp32
    ``[M, R]`` is ``x[t] @ lora_a[l]^T``, which :func:`mm_lora_backward` takes.
    """
    name = "mm_lora"
    M, K, N, L, R = _lora_operands(name, x, 1, w, lora_a, lora_b, lora_ids, lora_scale)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    _need(out_dtype in (x.dtype, torch.float32), "mm_lora: out_dtype must be x's type or float32")
    _need(bias is None or (bias.shape == (N,) and bias.dtype == x.dtype),
          "mm_lora: bias must be [N] of x's type")
    gpu = _one_gpu(name, x, w, lora_a, lora_b, lora_ids, lora_scale, bias, out, act, workspace)
    x, w, lora_a, lora_b, lora_ids = (x.contiguous(), w.contiguous(), lora_a.contiguous(),
                                      lora_b.contiguous(), lora_ids.contiguous())
    lora_scale = None if lora_scale is None else lora_scale.contiguous()
    bias = None if bias is None else bias.contiguous()
    out = _given(name, "out", out, (M, N), out_dtype, gpu)
    if with_act or act is not None:
        act = _given(name, "act", act, (M, R), torch.float32, gpu)
    workspace = _workspace(name, workspace, _lora_mm_bytes(M, N, K, L, R, 0), gpu)
    _launch(gpu, _lib.lib().mi_mm_lora, x.data_ptr(), M, K, _DT[x.dtype], w.data_ptr(), N,
            lora_a.data_ptr(), lora_b.data_ptr(), L, R, lora_ids.data_ptr(), _ptr(lora_scale),
            _ptr(bias), out.data_ptr(), _DT[out_dtype], _ptr(act), workspace.data_ptr(),
            workspace.numel())
    return out if act is None else (out, act)


def mm_lora_backward(grad_out: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                     lora_a: torch.Tensor, lora_b: torch.Tensor, lora_ids: torch.Tensor,
                     lora_scale: torch.Tensor | None = None, *, act: torch.Tensor | None = None,
                     with_x: bool = True, with_adapters: bool = True,
                     grad_dtype: torch.dtype | None = None, grad_x: torch.Tensor | None = None,
                     grad_a: torch.Tensor | None = None, grad_b: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None):
    """``(grad_x, grad_a, grad_b)`` of :func:`mm_lora` for ``grad_out`` ``[M, N]`` of x's type;
    ``w``, the bias and the scales are frozen::

        grad_x[t] = grad_out[t] @ w + lora_scale[l] * (grad_out[t] @ lora_b[l]) @ lora_a[l]
        grad_a[l] = lora_scale[l] * sum_t (grad_out[t] @ lora_b[l])^T x[t]     t with id l
        grad_b[l] = lora_scale[l] * sum_t grad_out[t]^T (x[t] @ lora_a[l]^T)

    ``grad_a`` and ``grad_b`` are like the banks, in ``grad_dtype`` (the banks' type, the
    default, or float32), zeros for an adapter without rows.  ``act`` is the forward's;
    without it, it is computed again.  ``with_x=False`` or ``with_adapters=False`` leaves
    those gradients out (None).  Equal inputs give equal bits.
    """
    name = "mm_lora_backward"
    M, K, N, L, R = _lora_operands(name, grad_out, 0, w, lora_a, lora_b, lora_ids, lora_scale)
    _need(x.shape == (M, K) and x.dtype == grad_out.dtype,
          "mm_lora_backward: x must be [M, K] of grad_out's type")
    grad_dtype = x.dtype if grad_dtype is None else grad_dtype
    _need(grad_dtype in (x.dtype, torch.float32),
          "mm_lora_backward: grad_dtype must be the banks' type or float32")
    _need(with_x or with_adapters, "mm_lora_backward: no gradient is asked for")
    _need(with_x or grad_x is None, "mm_lora_backward: grad_x needs with_x")
    _need(with_adapters or (grad_a is None and grad_b is None),
          "mm_lora_backward: grad_a and grad_b need with_adapters")
    _need(act is None or (act.shape == (M, R) and act.dtype == torch.float32),
          "mm_lora_backward: act must be float32 [M, R]")
    gpu = _one_gpu(name, grad_out, x, w, lora_a, lora_b, lora_ids, lora_scale, act, grad_x,
                   grad_a, grad_b, workspace)
    grad_out, x, w, lora_a, lora_b, lora_ids = (
        grad_out.contiguous(), x.contiguous(), w.contiguous(), lora_a.contiguous(),
        lora_b.contiguous(), lora_ids.contiguous())
    lora_scale = None if lora_scale is None else lora_scale.contiguous()
    act = None if act is None else act.contiguous()

    if with_x:
        grad_x = _given(name, "grad_x", grad_x, (M, K), x.dtype, gpu)
    if with_adapters:
        grad_a = _given(name, "grad_a", grad_a, (L, R, K), grad_dtype, gpu)
        grad_b = _given(name, "grad_b", grad_b, (L, N, R), grad_dtype, gpu)
    workspace = _workspace(name, workspace, _lora_mm_bytes(M, N, K, L, R, 1), gpu)
    _launch(gpu, _lib.lib().mi_mm_lora_backward, grad_out.data_ptr(), x.data_ptr(), M, K, _DT[x.dtype],
            w.data_ptr(), N, lora_a.data_ptr(), lora_b.data_ptr(), L, R, lora_ids.data_ptr(),
            _ptr(lora_scale), _ptr(act), _ptr(grad_x), _ptr(grad_a), _ptr(grad_b),
            _DT[grad_dtype], workspace.data_ptr(), workspace.numel())
    return grad_x, grad_a, grad_b


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------

def _router_logits(name, logits, token_mask):
    if not (logits.dim() == 2 and logits.dtype in _DT):
        raise ValueError(f"{name}: logits must be [T, E] bf16, fp16 or fp32")
    if not (token_mask is None or (token_mask.dtype in (torch.bool, torch.uint8) and
                                   token_mask.shape == (logits.shape[0],))):
        raise ValueError(f"{name}: token_mask must be bool or uint8 [T]")


def moe_route_topk(logits: torch.Tensor, top_k: int, *, renormalize: bool = True,
                   token_mask: torch.Tensor | None = None,
                   topk_weights: torch.Tensor | None = None,
                   topk_ids: torch.Tensor | None = None):
    """``(topk_weights, topk_ids)`` of the router's ``logits`` (bf16, fp16 or fp32 ``[T, E]``):
    the ``top_k`` largest of every token in falling order, ties to the lowest expert, and
    their softmax probabilities in fp32, divided by their sum with ``renormalize``.  They
    are the operands of :func:`moe_route_permutation` and :func:`moe_combine_rows`.

    A logit of -inf is never chosen: where a token has fewer than ``top_k`` others, the
    rest has id -1 and weight 0.  NaN is above every number and makes its token's weights
    NaN.  Tokens that ``token_mask`` (bool or uint8 ``[T]``) takes out, padding, have ids -1
    and weights 0.  E is at most 1024, ``top_k`` at most 64.
    """
    name = "moe_route_topk"
    _router_logits(name, logits, token_mask)
    top_k = int(top_k)
    T, E = logits.shape
    gpu = _one_gpu(name, logits, token_mask, topk_weights, topk_ids)
    logits = logits.contiguous()
    token_mask = None if token_mask is None else token_mask.contiguous()
    _need(1 <= top_k <= min(E, 64), "moe_route_topk: top_k must be in [1, min(E, 64)]")
    topk_weights = _given(name, "topk_weights", topk_weights, (T, top_k), torch.float32, gpu)
    topk_ids = _given(name, "topk_ids", topk_ids, (T, top_k), torch.int32, gpu)
    _launch(gpu, _lib.lib().mi_moe_route_topk, logits.data_ptr(), _DT[logits.dtype], T, E, top_k,
            int(renormalize), _ptr(token_mask), topk_weights.data_ptr(), topk_ids.data_ptr())
    return topk_weights, topk_ids


@functools.lru_cache(maxsize=1024)
def _balance_bytes(num_tokens, num_experts):
    return int(_lib.lib().mi_moe_balance_loss_workspace_size(num_tokens, num_experts))


def balance_workspace_bytes(num_tokens, num_experts) -> int:
    """Workspace of :func:`moe_balance_loss`."""
    return _balance_bytes(num_tokens, num_experts)


def moe_balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor, *, coef: float = 1.0,
                     token_mask: torch.Tensor | None = None,
                     given_counts: torch.Tensor | None = None,
                     loss: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                     slopes: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None):
    """``(loss, counts, slopes)`` of a batch's routing: ``counts`` int32 ``[E]`` are the choices
    of every expert in ``topk_ids`` (int32 ``[T, top_k]``, ids outside ``[0, E)`` are none),
    ``loss = coef * E * sum_e f[e] * P[e]`` an fp32 scalar with ``f = counts / sum(counts)``
    and ``P`` the mean of ``softmax(logits)``, and ``slopes`` fp32 ``[E]`` the loss's derivative
    by each token's probabilities, which :func:`moe_route_backward` takes.  Tokens that
    ``token_mask`` takes out count nowhere.  With ``given_counts`` (int32 ``[E]``: counts summed
    over more than these tokens, such as all ranks' or micro-batches') ``f`` is theirs.
    """
    name = "moe_balance_loss"
    _router_logits(name, logits, token_mask)
    T, E = logits.shape
    _need(topk_ids.dtype == torch.int32 and topk_ids.dim() == 2 and topk_ids.shape[0] == T and
          topk_ids.shape[1] >= 1, "moe_balance_loss: topk_ids must be int32 [T, top_k]")
    _need(given_counts is None or (given_counts.dtype == torch.int32 and
                                   given_counts.shape == (E,)),
          "moe_balance_loss: given_counts must be int32 [E]")
    gpu = _one_gpu(name, logits, topk_ids, token_mask, given_counts, loss, counts, slopes,
                   workspace)
    logits, topk_ids = logits.contiguous(), topk_ids.contiguous()
    token_mask = None if token_mask is None else token_mask.contiguous()
    given_counts = None if given_counts is None else given_counts.contiguous()
    loss = _given(name, "loss", loss, (), torch.float32, gpu)
    counts = _given(name, "counts", counts, (E,), torch.int32, gpu)
    slopes = _given(name, "slopes", slopes, (E,), torch.float32, gpu)
    workspace = _workspace(name, workspace, _balance_bytes(T, E), gpu)
    _launch(gpu, _lib.lib().mi_moe_balance_loss, logits.data_ptr(), _DT[logits.dtype], T, E,
            topk_ids.data_ptr(), topk_ids.shape[1], _ptr(token_mask), _ptr(given_counts),
            float(coef), loss.data_ptr(), counts.data_ptr(), slopes.data_ptr(),
            workspace.data_ptr(), workspace.numel())
    return loss, counts, slopes


def moe_route_backward(logits: torch.Tensor, *, topk_ids: torch.Tensor | None = None,
                       topk_weights: torch.Tensor | None = None,
                       grad_weights: torch.Tensor | None = None, renormalize: bool = True,
                       slopes: torch.Tensor | None = None,
                       grad_loss: torch.Tensor | None = None,
                       token_mask: torch.Tensor | None = None,
                       grad_dtype: torch.dtype | None = None,
                       grad_logits: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of ``logits`` through the weights of :func:`moe_route_topk`
    (``grad_weights`` fp32 ``[T, top_k]``, with its ``topk_ids`` and, where they were
    renormalised, its ``topk_weights``), through the loss of :func:`moe_balance_loss` (its
    ``slopes`` with ``grad_loss``, one fp32 value on the GPU), or through both.

    Slots whose id lies outside ``[0, E)`` have no gradient; tokens that ``token_mask`` takes
    out get zeros.  ``grad_logits`` ``[T, E]`` is of ``grad_dtype`` (the logits' type by
    default) and may be ``logits`` itself.
    """
    name = "moe_route_backward"
    _router_logits(name, logits, token_mask)
    T, E = logits.shape
    top_k = 1
    _need(grad_weights is not None or slopes is not None,
          "moe_route_backward: grad_weights or slopes is needed")
    if grad_weights is not None:
        _need(grad_weights.dtype == torch.float32 and grad_weights.dim() == 2 and
              grad_weights.shape[0] == T and grad_weights.shape[1] >= 1,
              "moe_route_backward: grad_weights must be float32 [T, top_k]")
        top_k = grad_weights.shape[1]
        _need(topk_ids is not None and topk_ids.dtype == torch.int32 and
              topk_ids.shape == grad_weights.shape,
              "moe_route_backward: grad_weights needs topk_ids, int32 [T, top_k]")
        _need(not renormalize or (topk_weights is not None and
                                  topk_weights.dtype == torch.float32 and
                                  topk_weights.shape == grad_weights.shape),
              "moe_route_backward: renormalised weights need topk_weights, float32 [T, top_k]")
    _need((slopes is None) == (grad_loss is None),
          "moe_route_backward: slopes and grad_loss are given together")
    _need(slopes is None or (slopes.dtype == torch.float32 and slopes.shape == (E,) and
                             grad_loss.dtype == torch.float32 and grad_loss.numel() == 1),
          "moe_route_backward: slopes must be float32 [E] and grad_loss one float32")
    gpu = _one_gpu(name, logits, topk_ids, topk_weights, grad_weights, slopes, grad_loss,
                   token_mask, grad_logits)
    logits = logits.contiguous()
    topk_ids, topk_weights, grad_weights, slopes, token_mask = (
        None if t is None else t.contiguous()
        for t in (topk_ids, topk_weights, grad_weights, slopes, token_mask))
    if grad_dtype is None:
        grad_dtype = logits.dtype if grad_logits is None else grad_logits.dtype
    _need(grad_dtype in _DT, "moe_route_backward: grad_dtype must be bfloat16, float16 or float32")
    grad_logits = _given(name, "grad_logits", grad_logits, (T, E), grad_dtype, gpu)
    _launch(gpu, _lib.lib().mi_moe_route_backward, logits.data_ptr(), _DT[logits.dtype], T, E,
            _ptr(topk_ids), _ptr(topk_weights), _ptr(grad_weights), top_k, int(renormalize),
            _ptr(slopes), _ptr(grad_loss), _ptr(token_mask), grad_logits.data_ptr(),
            _DT[grad_dtype])
    return grad_logits
