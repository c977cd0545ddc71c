"""Log-probabilities, entropy, top alternatives and 8-bit logits of a classifier head.

All of these work on hidden states e [..., D] (bf16) and a classifier of V rows, with logits
z = e @ c.T + bias and y = z / temperature, and none but ``int8_linear`` writes the [N, V] logits:

* ``linear_logprobs``      y_t - lse at given tokens t and the entropy of each position, with
                           gradients for e, c and the bias; the top alternatives in the same pass.
* ``linear_top_logprobs``  the k most probable tokens with their log-probabilities.
* ``quantize_int8``        rows of 8-bit integers with one scale each.
* ``int8_linear``          the logits themselves, for a classifier of 8-bit integers.

A classifier is a bf16 tensor [V, D], or ``Int8Rows`` (from ``quantize_int8``): its products then run on
8-bit integers, the hidden states being rounded to 8 bits row by row inside the call, and no gradient
flows. ``linear_logprobs``, whose outputs do have gradients, therefore refuses an 8-bit classifier where one is
asked for; the results of the others are never part of a graph. Forward-mode derivatives are refused. As in
``ops``, the compute runs in libcce.so on the current stream, arguments are checked here before a pointer
reaches the library, and there is no CPU path.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import NamedTuple, Optional, Tuple, Union

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import ops
from .ops import _bias_arg, _check, _ptr, _require_cuda

MAX_TOKENS = 32  # given tokens a position
MAX_TOP = 24     # alternatives a position
MIN_TEMPERATURE, MAX_TEMPERATURE = 1e-6, 1e6


class Int8Rows(NamedTuple):
    """Rows of 8-bit integers: row r stands for values[r] * scale[r]."""
    values: torch.Tensor  # int8 [rows, D]
    scale: torch.Tensor   # fp32 [rows]


class Logprobs(NamedTuple):
    logprobs: torch.Tensor                # fp32, in the shape of the tokens
    entropy: torch.Tensor                 # fp32, one a position
    top_logprobs: Optional[torch.Tensor]  # fp32 [..., top_k], or None
    top_ids: Optional[torch.Tensor]       # int64 [..., top_k], or None


class TopLogprobs(NamedTuple):
    logprobs: torch.Tensor  # fp32 [..., k], highest first
    ids: torch.Tensor       # int64 [..., k]


Classifier = Union[torch.Tensor, Int8Rows]


def _refuse(message: str) -> None:
    raise ops.CCEError(1, message)


def _check_classifier(c: Classifier, D: int) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The classifier's rows [V, D] and, for 8-bit ones, their scales."""
    if isinstance(c, Int8Rows):
        rows, scale = c
        if rows.dtype != torch.int8 or rows.dim() != 2:
            _refuse(f"Int8Rows.values must be int8 [V, D], got {rows.dtype} {tuple(rows.shape)}")
        if scale.dtype != torch.float32 or scale.numel() != rows.shape[0]:
            _refuse(f"Int8Rows.scale must be float32 with {rows.shape[0]} entries, got {scale.dtype} "
                    f"{tuple(scale.shape)}")
        if D % 16 != 0:
            _refuse(f"D must be a multiple of 16 for 8-bit operands, got {D}")
    else:
        rows, scale = c, None
        if rows.dim() != 2:
            _refuse(f"c must be 2-D, got {tuple(rows.shape)}")
        if rows.dtype != torch.bfloat16:
            _refuse(f"c must be bfloat16 or Int8Rows, got {rows.dtype}")
    if rows.shape[1] != D:
        _refuse(f"c must be [V, {D}], got {tuple(rows.shape)}")
    return rows, scale


def _no_tangent(name: str, e: torch.Tensor, c: Optional[Classifier] = None,
                bias: Optional[torch.Tensor] = None) -> None:
    """Refuse dual tensors: the outputs would come without a tangent, which torch takes as zero."""
    if getattr(forward_ad, "_current_level", 0) < 0:  # outside forward-mode there are none
        return
    for t in (e, bias) + (c if isinstance(c, Int8Rows) else (c,)):
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError(f"{name} has no forward-mode derivative")


def _flat(e: torch.Tensor) -> torch.Tensor:
    if e.dim() < 1:
        _refuse("e must have a last dimension of size D")
    if e.dtype != torch.bfloat16:
        _refuse(f"e must be bfloat16, got {e.dtype}")
    return e if e.dim() == 2 else e.reshape(-1, e.shape[-1])


def _check_matrix(E: torch.Tensor) -> Tuple[int, int]:
    if E.dim() != 2 or E.dtype != torch.bfloat16:
        _refuse(f"E must be bfloat16 [N, D], got {E.dtype} {tuple(E.shape)}")
    return E.shape


def _check_tokens(tokens: torch.Tensor, N: int) -> int:
    if tokens.dtype != torch.int64 or tokens.dim() != 2 or tokens.shape[0] != N:
        _refuse(f"tokens must be int64 [{N}, K], got {tokens.dtype} {tuple(tokens.shape)}")
    K = tokens.shape[1]
    if not 1 <= K <= MAX_TOKENS:
        _refuse(f"1 to {MAX_TOKENS} tokens a position, got {K}")
    return K


def _check_stats(row_stats: torch.Tensor, N: int) -> None:
    if row_stats.dtype != torch.float32 or row_stats.shape != (2, N) or not row_stats.is_contiguous():
        _refuse(f"row_stats must be contiguous float32 [2, {N}], got {row_stats.dtype} {tuple(row_stats.shape)}")


def _aligned(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """Contiguous, and at an address the kernels' 16-byte loads can start from (a slice of a larger
    buffer may begin anywhere: it is copied then)."""
    if t is None:
        return None
    if not t.is_contiguous():
        t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _check_scalars(top_k: int, V: int, temperature: float) -> None:
    if not MIN_TEMPERATURE <= temperature <= MAX_TEMPERATURE:
        raise ValueError(f"temperature must be in [{MIN_TEMPERATURE}, {MAX_TEMPERATURE}], got {temperature}")
    if not 0 <= top_k <= min(MAX_TOP, V):
        raise ValueError(f"the number of alternatives must be in [0, {min(MAX_TOP, V)}], got {top_k}")


_HERE = contextlib.nullcontext()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle alone, without a Stream object


def _stream(dev: torch.device) -> int:
    return ops._stream(dev) if _raw_stream is None else _raw_stream(dev.index)


def _on(dev: torch.device):
    """The device of a call as the current one (entering the context costs more than looking)."""
    return _HERE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def cce_logprobs(E: torch.Tensor, C: Classifier, tokens: Optional[torch.Tensor], top_k: int = 0,
                 bias: Optional[torch.Tensor] = None, temperature: float = 1.0, ignore_index: int = -100,
                 save_max: bool = False, check: bool = False, save_lse: bool = True,
                 row_stats: Optional[torch.Tensor] = None):
    """Run the forward for E [N, D] and tokens [N, K] (or None). Returns (logprobs [N, K], entropy [N],
    lse [N], tile_max or None, top_logprobs [N, top_k], top_ids [N, top_k]) as device tensors; the first
    three are None without tokens, the last two without alternatives. ``save_max`` keeps what a backward
    that skips units needs; without ``save_lse`` lse is None. ``row_stats``, fp32 [2, N], is filled with what the
    backward forms probabilities from: with lse alone they carry its rounding, which tells at small temperatures."""
    lib = ops.load_library()
    N, D = _check_matrix(E)
    rows, scale = _check_classifier(C, D)
    V = rows.shape[0]
    _check_scalars(top_k, V, temperature)
    K = 0 if tokens is None else _check_tokens(tokens, N)
    if row_stats is not None:
        if not K:
            _refuse("row_stats are formed with given tokens only")
        _check_stats(row_stats, N)
        _require_cuda(E, row_stats)
    dev = _require_cuda(E, rows)
    E, rows = _aligned(E), _aligned(rows)
    if scale is not None:
        _require_cuda(E, scale)
        scale = _aligned(scale)
    if bias is not None:
        bias = _aligned(_bias_arg(bias, V, dev))
    if K:
        _require_cuda(E, tokens)
        tokens = tokens.contiguous()
    p = ctypes.byref(ops.LogprobProblem(N, D, V, ignore_index, K, top_k, temperature, scale is not None, 0))
    ws_bytes = lib.cce_logprobs_workspace_size(p)
    if ws_bytes == 0:
        _refuse(f"bad problem N={N} D={D} V={V} tokens={K} top_k={top_k} ignore_index={ignore_index}")
    logprobs = entropy = lse = tile_max = top_lp = top_ids = None
    lse_bytes = 4 * N if K and not save_lse else 0  # kept behind the workspace then
    ws = torch.empty(ws_bytes + lse_bytes, device=dev, dtype=torch.uint8)
    lse_ptr = ws.data_ptr() + ws_bytes
    if K:
        logprobs = torch.empty(N, K, device=dev, dtype=torch.float32)
        entropy = torch.empty(N, device=dev, dtype=torch.float32)
        if save_lse:
            lse = torch.empty(N, device=dev, dtype=torch.float32)
            lse_ptr = lse.data_ptr()
    if save_max:
        tile_max = torch.empty(max(-(-V // 64) * N, 1), device=dev, dtype=torch.float32)
    if top_k:
        top_lp = torch.empty(N, top_k, device=dev, dtype=torch.float32)
        top_ids = torch.empty(N, top_k, device=dev, dtype=torch.int64)
    with _on(dev):
        _check(lib.cce_logprobs_stats(p, E.data_ptr(), rows.data_ptr(), _ptr(scale), _ptr(bias), _ptr(tokens),
                                      _ptr(logprobs), _ptr(entropy), lse_ptr, _ptr(row_stats), _ptr(tile_max),
                                      _ptr(top_lp), _ptr(top_ids), ws.data_ptr(), ws_bytes, _stream(dev)))
        if check:
            _check(lib.cce_check_device_error(_ptr(ws), _stream(dev)))
    return logprobs, entropy, lse, tile_max, top_lp, top_ids


def cce_logprobs_backward(E: torch.Tensor, C: torch.Tensor, tokens: torch.Tensor, logprobs: torch.Tensor,
                          lse: torch.Tensor, entropy: torch.Tensor, tile_max: Optional[torch.Tensor],
                          grad_logprobs: Optional[torch.Tensor], grad_entropy: Optional[torch.Tensor],
                          filter_eps: float = 0.0, bias: Optional[torch.Tensor] = None, dbias: Optional[bool] = None,
                          temperature: float = 1.0, ignore_index: int = -100, out_fp32: int = ops.OUT_BF16,
                          check: bool = False, row_stats: Optional[torch.Tensor] = None, dbias_fp32: bool = False):
    """Run the backward of ``cce_logprobs``. Returns (dE, dC, filtered_tiles) as device tensors, then
    dbias when it is computed (by default whenever ``bias`` is given), in fp32 with ``dbias_fp32``.
    ``row_stats`` as the forward filled it."""
    lib = ops.load_library()
    N, D = _check_matrix(E)
    if isinstance(C, Int8Rows):
        _refuse("a classifier of 8-bit integers has no gradient")
    rows, _ = _check_classifier(C, D)
    V = rows.shape[0]
    _check_scalars(0, V, temperature)
    K = _check_tokens(tokens, N)
    for name, t, n in (("logprobs", logprobs, N * K), ("lse", lse, N), ("entropy", entropy, N),
                       ("grad_logprobs", grad_logprobs, N * K), ("grad_entropy", grad_entropy, N)):
        if t is not None and (t.dtype != torch.float32 or t.numel() != n):
            _refuse(f"{name} must be float32 with {n} entries, got {t.dtype} {tuple(t.shape)}")
    if row_stats is not None:
        _check_stats(row_stats, N)
    if filter_eps > 0.0:
        need = -(-V // 64) * N
        if tile_max is None or tile_max.dtype != torch.float32 or tile_max.numel() < need:
            _refuse(f"filter_eps > 0 needs tile_max, float32 with at least {need} entries")
    mode = int(out_fp32)
    if mode not in (ops.OUT_BF16, ops.OUT_FP32, ops.OUT_DE_FP32):
        _refuse(f"out_fp32 must be 0, 1 or 2, got {out_fp32!r}")
    dev = _require_cuda(*(t for t in (E, rows, tokens, logprobs, lse, row_stats, entropy, tile_max, grad_logprobs,
                                      grad_entropy) if t is not None))
    E, rows, bias = _aligned(E), _aligned(rows), _aligned(_bias_arg(bias, V, dev))
    tokens, logprobs = tokens.contiguous(), logprobs.contiguous()
    lse, entropy = lse.contiguous(), entropy.contiguous()
    g_lp = None if grad_logprobs is None else grad_logprobs.contiguous()
    g_h = None if grad_entropy is None else grad_entropy.contiguous()
    tile_max = None if tile_max is None else tile_max.contiguous()
    want_dbias = (bias is not None) if dbias is None else bool(dbias)
    p = ctypes.byref(ops.LogprobProblem(N, D, V, ignore_index, K, 0, temperature, 0, 0))
    ws_bytes = lib.cce_logprobs_backward_workspace_size(p, mode)
    if ws_bytes == 0:
        _refuse(f"bad problem: {lib.cce_last_error_message().decode()}")
    de_dtype = torch.float32 if mode in (ops.OUT_FP32, ops.OUT_DE_FP32) else torch.bfloat16
    dc_dtype = torch.float32 if mode == ops.OUT_FP32 else torch.bfloat16
    dE = torch.empty(N, D, device=dev, dtype=de_dtype)
    dC = torch.empty(V, D, device=dev, dtype=dc_dtype)
    db = torch.empty(V, device=dev, dtype=torch.float32 if dbias_fp32 else dc_dtype) if want_dbias else None
    filtered = torch.empty(1, device=dev, dtype=torch.int64)
    ws = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    with _on(dev):
        _check(lib.cce_logprobs_stats_backward(
            p, E.data_ptr(), rows.data_ptr(), _ptr(bias), tokens.data_ptr(), logprobs.data_ptr(), lse.data_ptr(),
            _ptr(row_stats), entropy.data_ptr(), _ptr(tile_max), _ptr(g_lp), _ptr(g_h), float(filter_eps),
            dE.data_ptr(), dC.data_ptr(), _ptr(db), mode, bool(dbias_fp32), filtered.data_ptr(), ws.data_ptr(),
            ws_bytes, _stream(dev)))
        if check:
            _check(lib.cce_check_device_error(_ptr(ws), _stream(dev)))
    return (dE, dC, filtered) + ((db,) if want_dbias else ())


class _LinearLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, E, C, bias, tokens, shape, top_k, temperature, ignore_index, filter_eps):
        stats = torch.empty(2, E.shape[0], device=E.device, dtype=torch.float32)
        logprobs, entropy, lse, tile_max, top_lp, top_ids = cce_logprobs(
            E, C, tokens, top_k, bias, temperature, ignore_index, save_max=filter_eps > 0.0, row_stats=stats)
        logprobs = logprobs.view(shape)  # here, where it adds no node to the graph
        ctx.save_for_backward(E, C, bias, tokens, logprobs, lse, entropy, tile_max, stats)
        ctx.cfg = (temperature, ignore_index, filter_eps)
        ctx.set_materialize_grads(False)
        if top_k:
            ctx.mark_non_differentiable(top_lp, top_ids)
        return logprobs, entropy, top_lp, top_ids

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_logprobs, grad_entropy, _lp, _ids):
        E, C, bias, tokens, logprobs, lse, entropy, tile_max, stats = ctx.saved_tensors
        temperature, ignore_index, filter_eps = ctx.cfg
        want_db = bias is not None and ctx.needs_input_grad[2]
        out = cce_logprobs_backward(E, C, tokens, logprobs, lse, entropy, tile_max, grad_logprobs, grad_entropy,
                                    filter_eps, bias, want_db, temperature, ignore_index, row_stats=stats,
                                    dbias_fp32=want_db and bias.dtype != torch.bfloat16)
        dbias = out[3].to(bias.dtype).reshape(bias.shape) if want_db else None
        return out[0], out[1], dbias, None, None, None, None, None, None


def linear_logprobs(e: torch.Tensor, c: Classifier, tokens: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    temperature: float = 1.0, ignore_index: int = -100, top_k: int = 0, filter_eps: float = 0.0,
                    shift: bool = False) -> Logprobs:
    """Log-probabilities of given tokens under softmax((e @ c.T + bias) / temperature), and its entropy.

    e: [..., D] bf16 hidden states; c: [V, D] bf16 classifier or ``Int8Rows`` (no gradient); bias:
    optional [V]. tokens: int64, one a position in the shape e.shape[:-1], or up to 32 a position in the
    shape [..., K] (a token may be given twice). A token equal to ``ignore_index`` asks for nothing: 0,
    without a gradient; a position where every token does has entropy 0 and gives no gradient, whatever
    its hidden state holds. Other tokens outside [0, V) give NaN
    and no gradient; the entropy of their position is as usual.

    Gradients of both outputs flow to e, c and bias, each in its own type (policy gradients with an
    entropy bonus, preference losses, distillation on a teacher's alternatives). Nothing is left out of
    them by default; ``filter_eps`` > 0 skips units of 128 positions x 64 tokens whose probabilities are
    all below it, as ``linear_cross_entropy`` does, except units that hold a given token.

    top_k: also return the top_k (up to 24) most probable tokens of each position, without gradients,
    as ``linear_top_logprobs`` does. ``shift`` makes e[..., i, :] predict tokens[..., i + 1] (one token a
    position); every output is then one position shorter along the sequence axis.
    """
    _no_tangent("linear_logprobs", e, c, bias)
    lead = e.shape[:-1]
    if tokens.shape == lead:
        many = False
    elif tokens.dim() == e.dim() and tokens.shape[:-1] == lead:
        many = True
    else:
        raise ValueError(f"tokens shape {tuple(tokens.shape)} must equal e.shape[:-1] {tuple(lead)}, "
                         "with or without a last dimension of several tokens")
    if math.isnan(filter_eps):
        raise ValueError("filter_eps is NaN")
    if shift:
        if many or not lead or lead[-1] < 1:
            raise ValueError("shift needs one token a position and a sequence axis of length >= 1")
        tokens = ops.shift_targets(tokens, ignore_index)
    E = _flat(e)
    t = tokens if tokens.dtype == torch.int64 else tokens.to(torch.int64)
    if not many:
        t = t.reshape(-1, 1)
    elif t.dim() != 2:
        t = t.reshape(E.shape[0], t.shape[-1])
    grad = torch.is_grad_enabled() and (e.requires_grad or (bias is not None and bias.requires_grad) or
                                        (isinstance(c, torch.Tensor) and c.requires_grad))
    if not grad:
        logprobs, entropy, _, _, top_lp, top_ids = cce_logprobs(E, c, t, top_k, bias, temperature, ignore_index,
                                                                save_lse=False)
        logprobs = logprobs.view(tokens.shape)
    elif isinstance(c, Int8Rows):
        raise ValueError("a classifier of 8-bit integers has no gradient: call under torch.no_grad(), or detach e and "
                         "bias")
    else:
        logprobs, entropy, top_lp, top_ids = _LinearLogprobs.apply(
            E, c, bias, t, tokens.shape, int(top_k), float(temperature), ignore_index, float(filter_eps))
    if len(lead) != 1:
        entropy = entropy.reshape(lead)
        if top_k:
            top_lp, top_ids = top_lp.reshape(*lead, top_k), top_ids.reshape(*lead, top_k)
    if shift:
        logprobs, entropy = logprobs[..., :-1], entropy[..., :-1]
        if top_k:
            top_lp, top_ids = top_lp[..., :-1, :], top_ids[..., :-1, :]
    return Logprobs(logprobs, entropy, top_lp, top_ids)


def linear_top_logprobs(e: torch.Tensor, c: Classifier, k: int, bias: Optional[torch.Tensor] = None,
                        temperature: float = 1.0) -> TopLogprobs:
    """The k (1 to 24) most probable tokens of each position under softmax((e @ c.T + bias) /
    temperature) and their log-probabilities, highest first, the lower id first among equal ones.

    Alternatives nearer to each other than the rounding of their 32-bit sums are ordered by their logits in
    64 bits, so the ids depend neither on the batch they are computed in nor on how the work was split,
    unless nine or more tokens below one of them are as near to it as that. No gradient flows.
    """
    _no_tangent("linear_top_logprobs", e, c, bias)
    if k < 1:
        raise ValueError(f"k must be at least 1, got {k}")
    out = cce_logprobs(_flat(e), c, None, k, bias, temperature)
    lead = e.shape[:-1]
    if len(lead) == 1:
        return TopLogprobs(out[4], out[5])
    return TopLogprobs(out[4].reshape(*lead, k), out[5].reshape(*lead, k))


def quantize_int8(x: torch.Tensor) -> Int8Rows:
    """Rows of x [rows, D] (bf16) as 8-bit integers with one scale each: scale = max |x| / 127 and
    values = x / scale, rounded to the nearest integer, halves to the even one. D must be a multiple of
    16. A row of zeros gets scale 0; a row that holds an infinity or a NaN gets the scale NaN."""
    _no_tangent("quantize_int8", x)
    lib = ops.load_library()
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        _refuse(f"x must be bfloat16 [rows, D], got {x.dtype} {tuple(x.shape)}")
    if x.shape[1] < 16 or x.shape[1] % 16 != 0:
        _refuse(f"D must be a positive multiple of 16, got {x.shape[1]}")
    dev = _require_cuda(x)
    x = _aligned(x.detach())
    out = Int8Rows(torch.empty(x.shape, device=dev, dtype=torch.int8),
                   torch.empty(x.shape[0], device=dev, dtype=torch.float32))
    with _on(dev):
        _check(lib.cce_quantize_int8(_ptr(x), x.shape[0], x.shape[1], _ptr(out.values), _ptr(out.scale), _stream(dev)))
    return out


def int8_linear(e: torch.Tensor, c: Int8Rows, bias: Optional[torch.Tensor] = None,
                out_dtype: torch.dtype = torch.bfloat16, check: bool = False) -> torch.Tensor:
    """The logits e @ c.T + bias [..., V] of a classifier of 8-bit integers, in bf16 or fp32.

    Each row of e (bf16) is rounded to 8-bit integers with a scale of its own, the sums of integer
    products are exact, and the two scales and the bias are applied in fp32. No gradient flows."""
    _no_tangent("int8_linear", e, c, bias)
    lib = ops.load_library()
    if not isinstance(c, Int8Rows):
        _refuse(f"c must be Int8Rows (see quantize_int8), got {type(c).__name__}")
    if out_dtype not in (torch.bfloat16, torch.float32):
        _refuse(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    E = _flat(e)
    N, D = E.shape
    rows, scale = _check_classifier(c, D)
    V = rows.shape[0]
    dev = _require_cuda(E, rows, scale)
    E, rows, scale, bias = _aligned(E), _aligned(rows), _aligned(scale), _aligned(_bias_arg(bias, V, dev))
    ws_bytes = lib.cce_int8_linear_workspace_size(N, D, V)
    if ws_bytes == 0:
        _refuse(f"bad problem N={N} D={D} V={V}")
    out = torch.empty(N, V, device=dev, dtype=out_dtype)
    ws = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    with _on(dev):
        _check(lib.cce_int8_linear(N, D, V, E.data_ptr(), rows.data_ptr(), scale.data_ptr(), _ptr(bias),
                                   out.data_ptr(), out_dtype == torch.float32, ws.data_ptr(), ws_bytes, _stream(dev)))
        if check:
            _check(lib.cce_check_device_error(_ptr(ws), _stream(dev)))
    return out if e.dim() == 2 else out.reshape(*e.shape[:-1], V)
