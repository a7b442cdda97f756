"""Products with an epilogue (bias, activation, residual, the next product's
operand), their gradient, and products grouped by expert with the rows' way there
and back.

Operands are the codes and scales that quantize, rmsnorm, swiglu and the calls
here leave; other matrices are 2-D CUDA tensors of torch.bfloat16 (or raw 16-bit
patterns) or torch.float32 whose rows are contiguous.  All tensors of a call are on
one device.  Outputs and workspaces are allocated with torch unless given (through the
dispatcher where a dispatch mode, the profiler or torch's deterministic fill looks).
A `stream` other than the current one becomes the current one for the call.  None of them
records an autograd node, copies to the host or waits: plans are made and read on
the device, and every call can be captured in a CUDA graph.

ValueError for tensors a call does not take, MXError for a status; see include/mx.h.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _binding as _b
from . import _block

ACT_NONE, ACT_RELU, ACT_RELU2, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(6)
FMT_MXFP4, FMT_MXFP8 = _block.FMT_MXFP4, _block.FMT_MXFP8


def _calls():
    return _block._calls or _block._load()


def _f32(dtype):
    """Whether an output is fp32 (else bf16)."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("dtype must be torch.bfloat16 or torch.float32")
    return dtype == torch.float32


class GemmOut(NamedTuple):
    """y: act(z) + residual (None if not wanted); z: bf16, for the gradient (None if not
    wanted); codes, scales: the encoded y (None without fmt)."""
    y: Optional[torch.Tensor]
    z: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


class BiasActGrad(NamedTuple):
    dz: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


class ExpertPlan(NamedTuple):
    """Where the rows of each expert lie (all int32, on the device): offsets [experts + 1],
    multiples of 128; counts [experts]; slot [T, picks], -1 for a dropped choice; source
    [rows], -1 for a row without a token."""
    offsets: torch.Tensor
    counts: torch.Tensor
    slot: torch.Tensor
    source: torch.Tensor


class ExpertRows(NamedTuple):
    """y: bf16 [rows, K] (None if not wanted); codes, scales: the encoded rows (None without fmt)."""
    y: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


class ExpertGrad(NamedTuple):
    """The rows' gradient as ExpertRows has them; dweights: fp32 [T, picks] (None if not wanted)."""
    y: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    dweights: Optional[torch.Tensor]


def gemm_bias_act(Aq, As, Bq, Bs, M: int, N: int, K: int, bias=None, act: int = ACT_NONE, residual=None,
                  dtype=torch.bfloat16, want_y: bool = True, want_z: bool = False, fmt=None,
                  operands: int = FMT_MXFP4, out=None, stream=None) -> GemmOut:
    """z = A B^T + bias, y = act(z) + residual, in one launch: y in dtype (want_y) and / or encoded
    along its rows (fmt) as the next product's operand, z in bf16 (want_z) for bias_act_backward.
    `operands`: the format of A [M, K] and B [N, K].  out (for y) may be the residual itself.
    See mx_gemm_bias_act."""
    if stream is not None:
        with _block._on(stream, Aq):
            return gemm_bias_act(Aq, As, Bq, Bs, M, N, K, bias, act, residual, dtype, want_y, want_z, fmt, operands, out)
    return GemmOut._make(_calls().gemm_bias_act(Aq, As, Bq, Bs, M, N, K, bias, act, residual, _f32(dtype), want_y,
                                                want_z, fmt, operands, out))


def bias_act_backward_workspace_bytes(T: int, N: int) -> int:
    return int(_b.lib().mx_bias_act_backward_workspace_bytes(T, N))


def bias_act_backward(dy, z=None, act: int = ACT_NONE, want_dz: bool = True, want_dbias: bool = True, fmt=None,
                      ws=None, stream=None) -> BiasActGrad:
    """dz = dy * act'(z) in bf16 (want_dz) and / or encoded along its rows (fmt) as the Dgrad's operand,
    and dbias = its sum over all rows in fp32 (want_dbias; of gemm_experts' bias, not by expert).
    See mx_bias_act_backward."""
    if stream is not None:
        with _block._on(stream, dy):
            return bias_act_backward(dy, z, act, want_dz, want_dbias, fmt, ws)
    return BiasActGrad._make(_calls().bias_act_backward(dy, z, act, want_dz, want_dbias, fmt, ws))


def expert_rows(T: int, picks: int, experts: int) -> int:
    return int(_b.lib().mx_expert_rows(T, picks, experts))


def expert_plan_workspace_bytes(T: int, picks: int, experts: int) -> int:
    return int(_b.lib().mx_expert_plan_workspace_bytes(T, picks, experts))


def expert_plan(experts, num_experts: int, ws=None, stream=None) -> ExpertPlan:
    """The plan for experts [T, picks] (int32 or int64), the expert of each token's choices; numbers
    outside 0 .. num_experts - 1 are dropped choices.  See mx_expert_plan."""
    if stream is not None:
        with _block._on(stream, experts):
            return expert_plan(experts, num_experts, ws)
    return ExpertPlan._make(_calls().expert_plan(experts, num_experts, ws))


def expert_dispatch(x, plan: ExpertPlan, fmt=None, want_y: bool = True, stream=None) -> ExpertRows:
    """The rows of x [T, K] in the plan's order, in bf16 (want_y) and / or encoded along the rows (fmt)
    as gemm_experts' operand; other rows are zero.  Its gradient is expert_combine without
    weights.  See mx_expert_dispatch."""
    if stream is not None:
        with _block._on(stream, x):
            return expert_dispatch(x, plan, fmt, want_y)
    return ExpertRows._make(_calls().expert_dispatch(x, *plan, fmt, want_y))


def expert_combine(rows, plan: ExpertPlan, weights=None, residual=None, dtype=None, out=None, stream=None) -> torch.Tensor:
    """residual + the sum over each token's choices of weight * row, [T, K]; in dtype, else the
    residual's, else the rows' type.  out may be the residual itself.  See mx_expert_combine."""
    if stream is not None:
        with _block._on(stream, rows):
            return expert_combine(rows, plan, weights, residual, dtype, out)
    return _calls().expert_combine(rows, *plan, weights, residual, None if dtype is None else _f32(dtype), out)


def expert_combine_backward(dy, rows, plan: ExpertPlan, weights, fmt=None, want_y: bool = True,
                            want_dweights: bool = True, stream=None) -> ExpertGrad:
    """The gradients of expert_combine for its output's dy [T, K]: of the rows, in bf16 (want_y) and / or
    encoded (fmt), and of the weights (rows is read for these alone).  See mx_expert_combine_backward."""
    if stream is not None:
        with _block._on(stream, dy):
            return expert_combine_backward(dy, rows, plan, weights, fmt, want_y, want_dweights)
    return ExpertGrad._make(_calls().expert_combine_backward(dy, rows, *plan, weights, fmt, want_y, want_dweights))


def quantize_experts(w, contract: int = _b.CONTRACT_COLS, operands: int = FMT_MXFP4, rot: int = _b.ROT_NONE,
                     rot_block: int = 32, seed: int = 0, stream=None):
    """(codes, scales) of w [experts, rows, columns] in bf16, each matrix an operand of its own, as
    gemm_experts reads them.  FMT_MXFP8 takes contract=CONTRACT_ROWS (lines are the columns).  One launch
    along the columns where the rows are a multiple of 128, else one an expert.  See mx_quantize_experts."""
    if stream is not None:
        with _block._on(stream, w):
            return quantize_experts(w, contract, operands, rot, rot_block, seed)
    return _calls().quantize_experts(w, contract, operands, rot, rot_block, seed)


def gemm_experts(Aq, As, Bq, Bs, plan: ExpertPlan, N: int, K: int, bias=None, act: int = ACT_NONE,
                 dtype=torch.bfloat16, want_y: bool = True, want_z: bool = False, fmt=None,
                 operands: int = FMT_MXFP4, stream=None) -> GemmOut:
    """z = A B_e^T + bias_e, y = act(z) for the plan's rows of every expert e, [rows, N]; rows without a
    token are zero.  A [rows, K] as expert_dispatch leaves it, B as quantize_experts does, bias
    [experts, N]; outputs as gemm_bias_act's.  See mx_gemm_experts."""
    if stream is not None:
        with _block._on(stream, Aq):
            return gemm_experts(Aq, As, Bq, Bs, plan, N, K, bias, act, dtype, want_y, want_z, fmt, operands)
    return GemmOut._make(_calls().gemm_experts(Aq, As, Bq, Bs, *plan, N, K, bias, act, _f32(dtype), want_y, want_z,
                                               fmt, operands))


def gemm_experts_wgrad(Aq, As, Bq, Bs, plan: ExpertPlan, M: int, N: int, dtype=torch.float32,
                       operands: int = FMT_MXFP4, out=None, stream=None) -> torch.Tensor:
    """[experts, M, N] = A_e B_e^T over each expert's rows, of operands encoded down the plan's rows
    (A with M lines, B with N).  See mx_gemm_experts_wgrad."""
    if stream is not None:
        with _block._on(stream, Aq):
            return gemm_experts_wgrad(Aq, As, Bq, Bs, plan, M, N, dtype, operands, out)
    return _calls().gemm_experts_wgrad(Aq, As, Bq, Bs, *plan, M, N, _f32(dtype), operands, out)


def linear_experts_wgrad_workspace_bytes(operands: int, rows: int, N: int, K: int) -> int:
    return int(_b.lib().mx_linear_experts_wgrad_workspace_bytes(operands, rows, N, K))


def linear_experts_wgrad(dY, X, plan: ExpertPlan, operands: int = FMT_MXFP4, rot: int = _b.ROT_HADAMARD_DET,
                         rot_block: int = 32, rnd: int = _b.ROUND_RNE, seed: int = 0, dtype=torch.float32,
                         ws=None, out=None, stream=None) -> torch.Tensor:
    """dW [experts, N, K] = dY_e^T X_e over each expert's rows, with dY [rows, N], X [rows, K] in bf16 (rows
    without a token zero) encoded first, as linear_wgrad does.  FMT_MXFP8 takes rot=ROT_NONE.
    See mx_linear_experts_wgrad."""
    if stream is not None:
        with _block._on(stream, dY):
            return linear_experts_wgrad(dY, X, plan, operands, rot, rot_block, rnd, seed, dtype, ws, out)
    return _calls().linear_experts_wgrad(dY, X, *plan, operands, rot, rot_block, rnd, seed, _f32(dtype), ws, out)
