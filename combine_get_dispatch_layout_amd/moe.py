"""Thin Python binding of the calls of include/ep_moe.h (router and its balance
loss, products with expert weights, whole expert layer), over torch tensors.

As in ep.py: argument marshalling only, the functions carry the C names, the
work is queued on the current stream of the tensors' device, and outputs are
allocated with torch when none are passed.  ep_gate and ep_balance_loss take
part in autograd (first order, reverse mode); the other calls' outputs have no
gradient.
"""
import ctypes
from dataclasses import dataclass, field
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

from . import ep
from .ep import EP_OK, Handle, _check, lib

EP_SCORE_SOFTMAX, EP_SCORE_SIGMOID = 0, 1
EP_LOGITS_FP32, EP_LOGITS_BF16 = 0, 1
EP_WEIGHT_BF16, EP_WEIGHT_MXFP4, EP_WEIGHT_INT4, EP_WEIGHT_INT8 = 0, 1, 2, 3
EP_ACT_NONE, EP_ACT_SWIGLU = 0, 1
EP_MOE_MAX_TOKENS = 256
EP_BALANCE_MAX_SEQUENCES = 1 << 18

# Every symbol include/ep_moe.h declares.
SYMBOLS = ("ep_gate", "ep_gate_backward", "ep_balance_workspace_size", "ep_balance_loss",
           "ep_balance_loss_backward", "ep_matvec", "ep_expert_matvec", "ep_matmul",
           "ep_matmul_workspace_size", "ep_matmul_split", "ep_expert_matmul", "ep_moe_workspace_size", "ep_moe_layer")


class ep_gate_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("num_experts", "num_topk", "scoring", "renormalize", "num_groups", "topk_groups",
                 "group_top", "group_limit", "logits_type")] + [("scale", ctypes.c_float)]


class ep_balance_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("num_experts", "num_topk", "scoring", "normalize", "logits_type")] + \
               [("coefficient", ctypes.c_float)]


class ep_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("format", "group", "num_experts", "rows", "cols", "reserved")] + \
               [(n, ctypes.c_void_p) for n in ("d_data", "d_scales", "d_zeros")]


_bound = None


def _lib():
    """ep.py's library with this header's signatures set."""
    global _bound
    L = ep._lib
    if L is None or _bound is not L:
        L = lib()
        P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        L.ep_gate.argtypes = [P, P, P, P, I64, P, P, P]
        L.ep_gate_backward.argtypes = [P, P, P, P, I64, P, P]
        L.ep_matvec.argtypes = [P, P, I64, I32, P, P]
        L.ep_expert_matvec.argtypes = [P, P, P, I64, I32, P, P]
        L.ep_balance_workspace_size.argtypes = [P, I64, I64, P]
        L.ep_balance_loss.argtypes = [P, P, P, P, I64, P, I64, P, P, P, P, P, I64, P]
        L.ep_balance_loss_backward.argtypes = [P, P, P, I64, P, I64, P, P, P, P, P]
        L.ep_matmul.argtypes = [P, P, P, I64, I32, P, P]
        L.ep_matmul_workspace_size.argtypes = [P, I64, I32, P]
        L.ep_matmul_split.argtypes = [P, P, P, I64, I32, P, P, I64, P]
        L.ep_expert_matmul.argtypes = [P, P, P, P, I64, I32, P, P]
        L.ep_moe_workspace_size.argtypes = [P, P, P, I64, P]
        L.ep_moe_layer.argtypes = [P, P, P, P, P, P, I64, P, P, I64, P]
        for name in SYMBOLS:
            getattr(L, name).restype = ctypes.c_int
        _bound = L
    return L


def _check_tensor(name, t, dtypes, shape, device):
    """ep._check_tensor, with its tests in an order that costs a good call
    little: these calls take as long on the host as on the GPU."""
    if t is not None and not (t.dtype in dtypes and t.shape == shape and t.device == device):
        ep._check_tensor(name, t, dtypes, shape, device)


def _ptr(t):
    """The address of a contiguous GPU tensor as an int (None for None)."""
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        ep._ptr(t)                  # raises
    return t.data_ptr()


def _call(device, fn, *args):
    """fn(*args, stream) on the device's current stream, with the device
    current.  (By torch's internal names: torch.cuda.current_stream alone takes
    1.9 us of a call's 9.)"""
    index = device.index
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != EP_OK:
        _check(st)


# ---- router ----------------------------------------------------------------


@dataclass(frozen=True)
class GateConfig:
    num_experts: int
    num_topk: int
    scoring: int = EP_SCORE_SOFTMAX
    renormalize: bool = True
    num_groups: int = 0
    topk_groups: int = 0
    group_top: int = 0
    group_limit: bool = False
    scale: float = 1.0
    _c: dict = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        make = lambda kind: ep_gate_config(  # noqa: E731
            self.num_experts, self.num_topk, self.scoring, int(bool(self.renormalize)),
            self.num_groups, self.topk_groups, self.group_top, int(bool(self.group_limit)), kind,
            self.scale)
        object.__setattr__(self, "_c", {torch.float32: make(EP_LOGITS_FP32),
                                        torch.bfloat16: make(EP_LOGITS_BF16)})

    def c(self, dtype):
        return ctypes.byref(self._c[dtype])


def _check_logits(cfg, logits):
    if (logits.dtype not in (torch.float32, torch.bfloat16) or logits.dim() != 2
            or logits.shape[1] != cfg.num_experts):
        raise ValueError("logits must be fp32 or bf16 [N, num_experts]")
    return logits.shape[0], logits.device


def _records(name, logits):
    """Whether autograd records a call on logits.  A tangent (forward mode) is
    refused: it would be lost without a word."""
    if forward_ad._current_level >= 0 and forward_ad.unpack_dual(logits).tangent is not None:
        raise RuntimeError(f"{name} has no forward mode derivative")
    return logits.requires_grad and torch.is_grad_enabled()


class _Gate(torch.autograd.Function):
    """ep_gate with ep_gate_backward as its weights' gradient."""

    @staticmethod
    def forward(ctx, cfg, logits, bias, token_mask, given_idx, given_weights):
        topk_idx, topk_weights = ep_gate(cfg, logits, bias, token_mask, given_idx, given_weights)
        ctx.cfg, ctx.leaf = cfg, logits.is_leaf
        # a given buffer may be filled again before the backward pass
        ctx.save_for_backward(logits, topk_idx if given_idx is None else topk_idx.clone())
        # outputs of their own, in the given memory: the buffers keep no graph
        if given_idx is not None:
            topk_idx = topk_idx.detach()
        if given_weights is not None:
            topk_weights = topk_weights.detach()
        ctx.mark_non_differentiable(topk_idx)
        ctx.set_materialize_grads(False)
        return topk_idx, topk_weights

    @staticmethod
    def backward(ctx, _, grad_weights):
        if grad_weights is None:
            return (None,) * 6
        if torch.is_grad_enabled():     # create_graph: would lose the second order silently
            raise RuntimeError("ep_gate has a first order gradient only")
        # a leaf's gradient accumulates on the stream of its first use, which a
        # captured backward pass must not touch
        if ctx.leaf and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the backward pass of ep_gate into leaf logits must not be captured: "
                               "capture ep_gate_backward")
        logits, topk_idx = ctx.saved_tensors
        grad = ep_gate_backward(ctx.cfg, logits, topk_idx, grad_weights.contiguous())
        return None, grad, None, None, None, None


def ep_gate(cfg: GateConfig, logits: torch.Tensor, bias: Optional[torch.Tensor] = None,
            token_mask: Optional[torch.Tensor] = None, topk_idx: Optional[torch.Tensor] = None,
            topk_weights: Optional[torch.Tensor] = None):
    """Chooses num_topk experts per row of logits [N, E] (fp32 or bf16).  bias
    fp32 [E] acts on the choice only; token_mask bool / uint8 [N]: rows with 0
    get none.  Returns (topk_idx int32 [N,K], topk_weights fp32 [N,K]).  Where
    autograd records and the logits require a gradient, the returned weights
    have one, the choice held fixed (a topk_weights passed in is filled, but it
    is the returned tensor that has the gradient)."""
    if _records("ep_gate", logits):
        return _Gate.apply(cfg, logits, bias, token_mask, topk_idx, topk_weights)
    N, dev = _check_logits(cfg, logits)
    shape = (N, cfg.num_topk)
    if topk_idx is None:
        topk_idx = torch.empty(shape, dtype=torch.int32, device=dev)
    else:
        _check_tensor("topk_idx", topk_idx, (torch.int32,), shape, dev)
    if topk_weights is None:
        topk_weights = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _check_tensor("topk_weights", topk_weights, (torch.float32,), shape, dev)
    _check_tensor("bias", bias, (torch.float32,), (cfg.num_experts,), dev)
    _check_tensor("token_mask", token_mask, (torch.bool, torch.uint8), (N,), dev)
    _call(dev, _lib().ep_gate, cfg.c(logits.dtype), _ptr(logits), _ptr(bias), _ptr(token_mask), N,
          _ptr(topk_idx), _ptr(topk_weights))
    return topk_idx, topk_weights


def ep_gate_backward(cfg: GateConfig, logits: torch.Tensor, topk_idx: torch.Tensor,
                     grad_weights: torch.Tensor, grad_logits: Optional[torch.Tensor] = None):
    """Gradient of ep_gate's weights with respect to the logits, for the given
    choice: grad_logits [N, E] of the logits' type."""
    N, dev = _check_logits(cfg, logits)
    _check_tensor("topk_idx", topk_idx, (torch.int32,), (N, cfg.num_topk), dev)
    _check_tensor("grad_weights", grad_weights, (torch.float32,), (N, cfg.num_topk), dev)
    if grad_logits is None:
        grad_logits = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    else:
        _check_tensor("grad_logits", grad_logits, (logits.dtype,), logits.shape, dev)
    _call(dev, _lib().ep_gate_backward, cfg.c(logits.dtype), _ptr(logits), _ptr(topk_idx),
          _ptr(grad_weights), N, _ptr(grad_logits))
    return grad_logits


# ---- balance loss --------------------------------------------------------------


@dataclass(frozen=True)
class BalanceConfig:
    num_experts: int
    num_topk: int
    scoring: int = EP_SCORE_SOFTMAX
    normalize: bool = True
    coefficient: float = 1.0
    _c: dict = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        make = lambda kind: ep_balance_config(  # noqa: E731
            self.num_experts, self.num_topk, self.scoring, int(bool(self.normalize)), kind,
            self.coefficient)
        object.__setattr__(self, "_c", {torch.float32: make(EP_LOGITS_FP32),
                                        torch.bfloat16: make(EP_LOGITS_BF16)})

    def c(self, dtype):
        return ctypes.byref(self._c[dtype])


class Balance(NamedTuple):
    """What ep_balance_loss returns."""
    loss: torch.Tensor          # fp32 []
    counts: torch.Tensor        # int32 [Q, E]
    seq_tokens: torch.Tensor    # int32 [Q]
    score_sums: torch.Tensor    # fp32 [Q, E]


def ep_balance_workspace_size(cfg: BalanceConfig, num_tokens: int, num_sequences: int = 1) -> int:
    out = ctypes.c_int64()
    _check(_lib().ep_balance_workspace_size(cfg.c(torch.float32), num_tokens, num_sequences,
                                            ctypes.byref(out)))
    return out.value


def _check_sequences(seq_start, device):
    """Number of sequences."""
    if seq_start is None:
        return 1
    if (seq_start.dtype != torch.int32 or seq_start.dim() != 1 or seq_start.numel() < 2
            or seq_start.device != device):
        raise ValueError(f"seq_start must be int32 [sequences + 1] on {device}")
    return seq_start.numel() - 1


class _BalanceLoss(torch.autograd.Function):
    """ep_balance_loss with ep_balance_loss_backward as the loss's gradient."""

    @staticmethod
    def forward(ctx, cfg, logits, topk_idx, token_mask, seq_start, loss, counts, seq_tokens,
                score_sums, workspace):
        out = ep_balance_loss(cfg, logits, topk_idx, token_mask, seq_start, loss, counts, seq_tokens,
                              score_sums, workspace)
        ctx.cfg, ctx.leaf = cfg, logits.is_leaf
        # copies: before the backward pass the caller may fill a given buffer again,
        # or sum the counts over ranks in place, which raises no version
        ctx.save_for_backward(logits, token_mask, seq_start, out.counts.clone(), out.seq_tokens.clone())
        # outputs of their own, in the given memory: the buffers keep no graph
        out = [o if given is None else o.detach()
               for o, given in zip(out, (loss, counts, seq_tokens, score_sums))]
        ctx.mark_non_differentiable(*out[1:])
        ctx.set_materialize_grads(False)
        return tuple(out)

    @staticmethod
    def backward(ctx, grad_loss, *_):
        if grad_loss is None:
            return (None,) * 10
        if torch.is_grad_enabled():     # create_graph: would lose the second order silently
            raise RuntimeError("ep_balance_loss has a first order gradient only")
        # a leaf's gradient accumulates on the stream of its first use, which a
        # captured backward pass must not touch
        if ctx.leaf and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the backward pass of ep_balance_loss into leaf logits must not be "
                               "captured: capture ep_balance_loss_backward")
        logits, token_mask, seq_start, counts, seq_tokens = ctx.saved_tensors
        grad = ep_balance_loss_backward(ctx.cfg, logits, counts, seq_tokens, grad_loss.contiguous(),
                                        token_mask, seq_start)
        return (None, grad) + (None,) * 8


def ep_balance_loss(cfg: BalanceConfig, logits: torch.Tensor, topk_idx: torch.Tensor,
                    token_mask: Optional[torch.Tensor] = None,
                    seq_start: Optional[torch.Tensor] = None, loss: Optional[torch.Tensor] = None,
                    counts: Optional[torch.Tensor] = None, seq_tokens: Optional[torch.Tensor] = None,
                    score_sums: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> Balance:
    """Per-expert counts of the routing topk_idx int32 [N, K] and the balance
    loss of the logits [N, E] (fp32 or bf16).  token_mask bool / uint8 [N]: rows
    with 0 do not count; seq_start int32 [Q+1]: the sequences' bounds (default:
    the batch is one).  Returns Balance(loss [], counts [Q, E], seq_tokens [Q],
    score_sums [Q, E]).  Where autograd records and the logits require a
    gradient, the returned loss has one (a loss passed in is filled, but it is
    the returned tensor that has the gradient).  workspace: uint8, at least
    ep_balance_workspace_size bytes (allocated for this call when not given)."""
    if _records("ep_balance_loss", logits):
        return Balance(*_BalanceLoss.apply(cfg, logits, topk_idx, token_mask, seq_start, loss, counts,
                                           seq_tokens, score_sums, workspace))
    N, dev = _check_logits(cfg, logits)
    Q = _check_sequences(seq_start, dev)
    _check_tensor("topk_idx", topk_idx, (torch.int32,), (N, cfg.num_topk), dev)
    _check_tensor("token_mask", token_mask, (torch.bool, torch.uint8), (N,), dev)

    def output(name, given, dtype, shape):
        if given is None:
            return logits.new_empty(shape, dtype=dtype)
        _check_tensor(name, given, (dtype,), shape, dev)
        return given

    E = cfg.num_experts
    loss = output("loss", loss, torch.float32, ())
    counts = output("counts", counts, torch.int32, (Q, E))
    seq_tokens = output("seq_tokens", seq_tokens, torch.int32, (Q,))
    score_sums = output("score_sums", score_sums, torch.float32, (Q, E))
    if workspace is None:
        workspace = torch.empty(ep_balance_workspace_size(cfg, N, Q), dtype=torch.uint8, device=dev)
    elif workspace.device != dev:
        raise ValueError("workspace must be on the logits' device")
    _call(dev, _lib().ep_balance_loss, cfg.c(logits.dtype), _ptr(logits), _ptr(topk_idx),
          _ptr(token_mask), N, _ptr(seq_start), Q, _ptr(loss), _ptr(counts), _ptr(seq_tokens),
          _ptr(score_sums), _ptr(workspace), workspace.numel() * workspace.element_size())
    return Balance(loss, counts, seq_tokens, score_sums)


def ep_balance_loss_backward(cfg: BalanceConfig, logits: torch.Tensor, counts: torch.Tensor,
                             seq_tokens: torch.Tensor, grad_loss: torch.Tensor,
                             token_mask: Optional[torch.Tensor] = None,
                             seq_start: Optional[torch.Tensor] = None,
                             grad_logits: Optional[torch.Tensor] = None):
    """Gradient of ep_balance_loss's loss with respect to the logits, given its
    counts and seq_tokens (or their sums over ranks): grad_logits [N, E] of the
    logits' type."""
    N, dev = _check_logits(cfg, logits)
    Q = _check_sequences(seq_start, dev)
    _check_tensor("counts", counts, (torch.int32,), (Q, cfg.num_experts), dev)
    _check_tensor("seq_tokens", seq_tokens, (torch.int32,), (Q,), dev)
    _check_tensor("grad_loss", grad_loss, (torch.float32,), (), dev)
    _check_tensor("token_mask", token_mask, (torch.bool, torch.uint8), (N,), dev)
    if grad_logits is None:
        grad_logits = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    else:
        _check_tensor("grad_logits", grad_logits, (logits.dtype,), logits.shape, dev)
    _call(dev, _lib().ep_balance_loss_backward, cfg.c(logits.dtype), _ptr(logits), _ptr(token_mask), N,
          _ptr(seq_start), Q, _ptr(counts), _ptr(seq_tokens), _ptr(grad_loss), _ptr(grad_logits))
    return grad_logits


# ---- products with expert weights --------------------------------------------


class Weights:
    """A stack of weight matrices [E, rows, cols] in one storage format; keeps
    its tensors alive.  data: bf16 [E, rows, cols], or uint8 [E, rows, cols/2]
    (two codes a byte, column 2i in the low nibble) with scales
    [E, rows, cols/group]: uint8 E8M0 (MXFP4) or bf16 (INT4, optionally with
    uint8 zeros), or int8 [E, rows, cols] with fp32 scales [E, rows] (INT8).  A
    missing first dimension stands for one matrix."""

    def __init__(self, format: int, data: torch.Tensor, scales: Optional[torch.Tensor] = None,
                 zeros: Optional[torch.Tensor] = None, group: int = 0):
        if format not in (EP_WEIGHT_BF16, EP_WEIGHT_MXFP4, EP_WEIGHT_INT4, EP_WEIGHT_INT8):
            raise ValueError(f"unknown weight format {format}")
        want = {EP_WEIGHT_BF16: torch.bfloat16, EP_WEIGHT_INT8: torch.int8}.get(format, torch.uint8)
        per = 2 if want == torch.uint8 else 1       # columns of an element
        if data.dtype != want or data.dim() not in (2, 3):
            raise ValueError(f"data must be {want} [E, rows, cols{'/2' if per == 2 else ''}]")
        stack = data if data.dim() == 3 else data[None]
        E, M = stack.shape[:2]
        C = stack.shape[2] * per
        if format == EP_WEIGHT_BF16:
            if scales is not None or zeros is not None or group:
                raise ValueError("bf16 weights have no scales, zeros or group")
        elif format == EP_WEIGHT_INT8:
            if zeros is not None or group:
                raise ValueError("INT8 weights have no zeros or group")
            if scales is None:
                raise ValueError("INT8 weights need scales")
            _check_tensor("scales", scales, (torch.float32,), data.shape[:-1], data.device)
        else:
            group = group or (32 if format == EP_WEIGHT_MXFP4 else 0)
            if group <= 0 or C % group:
                raise ValueError(f"group={group} must divide cols={C}")
            if scales is None:
                raise ValueError("4-bit weights need scales")
            shape = (*data.shape[:-1], C // group)
            _check_tensor("scales", scales,
                          (torch.uint8 if format == EP_WEIGHT_MXFP4 else torch.bfloat16,), shape,
                          data.device)
            if zeros is not None and format != EP_WEIGHT_INT4:
                raise ValueError("only INT4 weights have zeros")
            _check_tensor("zeros", zeros, (torch.uint8,), shape, data.device)
        self.format, self.group = format, group
        self.num_experts, self.rows, self.cols = E, M, C
        self.data, self.scales, self.zeros = data, scales, zeros
        self.device = data.device
        self._c = ep_weights(format, group, E, M, C, 0, _ptr(data), _ptr(scales), _ptr(zeros))
        self._ref = ctypes.byref(self._c)
        self._workspace = {}        # bytes for (rows, activation) of ep_matmul


def _check_product(w, x, y, activation, dtype=torch.bfloat16):
    if activation not in (EP_ACT_NONE, EP_ACT_SWIGLU):
        raise ValueError(f"unknown activation {activation}")
    if activation == EP_ACT_SWIGLU and w.rows % 2:
        raise ValueError("SWIGLU needs an even number of weight rows")
    if x.dtype != dtype or x.dim() != 2 or x.shape[1] != w.cols or x.device != w.device:
        raise ValueError(f"x must be {'bf16' if dtype == torch.bfloat16 else 'int8'} [rows, {w.cols}] "
                         f"on {w.device}")
    shape = (x.shape[0], w.rows // 2 if activation else w.rows)
    if y is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=x.device)
    _check_tensor("y", y, (torch.bfloat16,), shape, x.device)
    return y


def ep_matvec(w: Weights, x: torch.Tensor, y: Optional[torch.Tensor] = None,
              activation: int = EP_ACT_NONE):
    """y = act(x W^T) for a few rows x bf16 [rows, cols] and one matrix."""
    y = _check_product(w, x, y, activation)
    _call(x.device, _lib().ep_matvec, w._ref, _ptr(x), x.shape[0], activation, _ptr(y))
    return y


def ep_expert_matvec(h: Handle, w: Weights, x: torch.Tensor, y: Optional[torch.Tensor] = None,
                     activation: int = EP_ACT_NONE):
    """y[s] = act(W[expert of receive row s] x[s]) for x bf16 [rows, cols] in
    the receive-row order of h's layout.  Rows without a token are not written
    (left unset in a y allocated here)."""
    if h.device != x.device:
        raise ValueError("x must be on the handle's device")
    y = _check_product(w, x, y, activation)
    _call(x.device, _lib().ep_expert_matvec, h.ptr, w._ref, _ptr(x), x.shape[0], activation, _ptr(y))
    return y


def _check_x_scales(x, x_scales):
    """[rows], or the [rows, 1] of a dispatch's recv_scales."""
    if x_scales.dim() == 2:
        _check_tensor("x_scales", x_scales, (torch.float32,), (x.shape[0], 1), x.device)
    else:
        _check_tensor("x_scales", x_scales, (torch.float32,), (x.shape[0],), x.device)


# Sizes that one Weights remembers: a server's batches have any number of rows.
_MAX_SIZES = 256


def ep_matmul_workspace_size(w: Weights, rows: int, activation: int = EP_ACT_NONE) -> int:
    n = w._workspace.get((rows, activation))
    if n is None:
        out = ctypes.c_int64()
        _check(_lib().ep_matmul_workspace_size(w._ref, rows, activation, ctypes.byref(out)))
        if len(w._workspace) >= _MAX_SIZES:
            w._workspace.clear()
        n = w._workspace[rows, activation] = out.value
    return n


def ep_matmul(w: Weights, x: torch.Tensor, x_scales: torch.Tensor, y: Optional[torch.Tensor] = None,
              activation: int = EP_ACT_NONE, workspace: Optional[torch.Tensor] = None):
    """y bf16 = act((x W^T) * x_scales * w's scales) in 8-bit integers, for x
    int8 [rows, cols] with x_scales fp32 [rows] or [rows, 1] and one matrix
    (INT8 weights).  Few rows of many columns are split (ep_matmul_split) in a
    workspace: uint8, at least ep_matmul_workspace_size bytes (allocated for this
    call when not given)."""
    y = _check_product(w, x, y, activation, torch.int8)
    _check_x_scales(x, x_scales)
    need = ep_matmul_workspace_size(w, x.shape[0], activation)
    if need == 0:
        _call(x.device, _lib().ep_matmul, w._ref, _ptr(x), _ptr(x_scales), x.shape[0], activation, _ptr(y))
        return y
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    elif workspace.dtype != torch.uint8 or workspace.device != x.device:
        raise ValueError(f"workspace must be uint8 on {x.device}")
    _call(x.device, _lib().ep_matmul_split, w._ref, _ptr(x), _ptr(x_scales), x.shape[0], activation,
          _ptr(y), _ptr(workspace), workspace.numel())
    return y


def ep_expert_matmul(h: Handle, w: Weights, x: torch.Tensor, x_scales: torch.Tensor,
                     y: Optional[torch.Tensor] = None, activation: int = EP_ACT_NONE):
    """The same for x in the receive-row order of h's layout (an int8
    dispatch's recv_x and recv_scales), each row with its expert's matrix.  Rows
    without a token are not written (left unset in a y allocated here)."""
    if h.device != x.device:
        raise ValueError("x must be on the handle's device")
    y = _check_product(w, x, y, activation, torch.int8)
    _check_x_scales(x, x_scales)
    _call(x.device, _lib().ep_expert_matmul, h.ptr, w._ref, _ptr(x), _ptr(x_scales), x.shape[0],
          activation, _ptr(y))
    return y


def ep_moe_workspace_size(h: Handle, w_up: Weights, w_down: Weights, num_tokens: int) -> int:
    out = ctypes.c_int64()
    _check(_lib().ep_moe_workspace_size(h.ptr, w_up._ref, w_down._ref, num_tokens,
                                        ctypes.byref(out)))
    return out.value


def ep_moe_layer(h: Handle, w_up: Weights, w_down: Weights, x: torch.Tensor,
                 topk_idx: torch.Tensor, topk_weights: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """The whole expert layer of up to EP_MOE_MAX_TOKENS tokens x bf16
    [N, hidden]; returns out bf16 [N, hidden].  workspace: uint8, at least
    ep_moe_workspace_size bytes (allocated for this call when not given)."""
    cfg, dev = h.cfg, x.device
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != cfg.hidden:
        raise ValueError("x must be bf16 [N, hidden]")
    if h.device != dev or w_up.device != dev or w_down.device != dev:
        raise ValueError("the handle, the weights and x must be on one device")
    N = x.shape[0]
    _check_tensor("topk_idx", topk_idx, (torch.int32,), (N, cfg.num_topk), dev)
    _check_tensor("topk_weights", topk_weights, (torch.float32,), (N, cfg.num_topk), dev)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _check_tensor("out", out, (torch.bfloat16,), x.shape, dev)
    if workspace is None:
        workspace = torch.empty(ep_moe_workspace_size(h, w_up, w_down, N), dtype=torch.uint8,
                                device=dev)
    elif workspace.device != dev:
        raise ValueError("workspace must be on x's device")
    _call(dev, _lib().ep_moe_layer, h.ptr, w_up._ref, w_down._ref, _ptr(x), _ptr(topk_idx),
          _ptr(topk_weights), N, _ptr(out), _ptr(workspace),
          workspace.numel() * workspace.element_size())
    return out
