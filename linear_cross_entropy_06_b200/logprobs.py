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
flows. As in ``ops``, the compute runs in libcce.so on the current stream, arguments are checked here
before a pointer reaches the library, and there is no CPU path.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import ops
from .ops import _bias_arg, _check, _ptr, _require, _require_cuda, _stream

MAX_TOKENS = 32  # given tokens a position
MAX_TOP = 24     # alternatives a position


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


def _check_classifier(c: Classifier, D: int) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The classifier's rows [V, D] and, for 8-bit ones, their scales."""
    if isinstance(c, Int8Rows):
        values, scale = c
        _require(values.dtype == torch.int8 and values.dim() == 2,
                 f"Int8Rows.values must be int8 [V, D], got {values.dtype} {tuple(values.shape)}")
        _require(scale.dtype == torch.float32 and scale.numel() == values.shape[0],
                 f"Int8Rows.scale must be float32 with {values.shape[0]} entries, got {scale.dtype} {tuple(scale.shape)}")
        _require(D % 16 == 0, f"D must be a multiple of 16 for 8-bit operands, got {D}")
        rows = values
    else:
        _require(c.dim() == 2, f"c must be 2-D, got {tuple(c.shape)}")
        _require(c.dtype == torch.bfloat16, f"c must be bfloat16 or Int8Rows, got {c.dtype}")
        rows, scale = c, None
    _require(rows.shape[1] == D, f"c must be [V, {D}], got {tuple(rows.shape)}")
    return rows, scale


def _flat(e: torch.Tensor) -> torch.Tensor:
    _require(e.dim() >= 1, "e must have a last dimension of size D")
    _require(e.dtype == torch.bfloat16, f"e must be bfloat16, got {e.dtype}")
    return e.reshape(-1, e.shape[-1])


def _aligned(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """Contiguous, and at an address the kernels' 16-byte loads can start from (a slice of a larger
    buffer may begin anywhere: it is copied then)."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _problem(N: int, D: int, V: int, ignore_index: int, tokens: int, top_k: int, temperature: float,
             int8: bool) -> ops.LogprobProblem:
    return ops.LogprobProblem(N, D, V, ignore_index, tokens, top_k, temperature, int(int8), 0)


def _check_scalars(top_k: int, V: int, temperature: float) -> None:
    if not (math.isfinite(temperature) and temperature > 0.0):
        raise ValueError(f"temperature must be finite and > 0, got {temperature}")
    if not 0 <= top_k <= min(MAX_TOP, V):
        raise ValueError(f"the number of alternatives must be in [0, {min(MAX_TOP, V)}], got {top_k}")


def cce_logprobs(E: torch.Tensor, C: Classifier, tokens: Optional[torch.Tensor], top_k: int = 0,
                 bias: Optional[torch.Tensor] = None, temperature: float = 1.0, ignore_index: int = -100,
                 save_max: bool = False, check: bool = False):
    """Run the forward for E [N, D] and tokens [N, K] (or None). Returns (logprobs [N, K], entropy [N],
    lse [N], tile_max or None, top_logprobs [N, top_k], top_ids [N, top_k]) as device tensors; the first
    three are None without tokens, the last two without alternatives. ``save_max`` keeps what a backward
    that skips units needs."""
    lib = ops.load_library()
    _require(E.dim() == 2, f"E must be 2-D, got {tuple(E.shape)}")
    E = _flat(E)
    N, D = E.shape
    rows, scale = _check_classifier(C, D)
    V = rows.shape[0]
    _check_scalars(top_k, V, temperature)
    K = 0
    if tokens is not None:
        _require(tokens.dtype == torch.int64, f"tokens must be int64, got {tokens.dtype}")
        _require(tokens.dim() == 2 and tokens.shape[0] == N, f"tokens must be [{N}, K], got {tuple(tokens.shape)}")
        K = tokens.shape[1]
        _require(1 <= K <= MAX_TOKENS, f"1 to {MAX_TOKENS} tokens a position, got {K}")
    dev = _require_cuda(E, rows, *(t for t in (scale, tokens) if t is not None))
    E, rows, scale, bias = _aligned(E), _aligned(rows), _aligned(scale), _aligned(_bias_arg(bias, V, dev))
    tokens = None if tokens is None else tokens.contiguous()
    p = _problem(N, D, V, ignore_index, K, top_k, temperature, scale is not None)
    ws_bytes = lib.cce_logprobs_workspace_size(ctypes.byref(p))
    _require(ws_bytes > 0, f"bad problem N={N} D={D} V={V} tokens={K} top_k={top_k}")

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, device=dev, dtype=dtype)

    logprobs, entropy, lse = (empty(N, K), empty(N), empty(N)) if K else (None, None, None)
    tile_max = empty(max(-(-V // 64) * N, 1)) if save_max else None
    top_lp, top_ids = (empty(N, top_k), empty(N, top_k, dtype=torch.int64)) if top_k else (None, None)
    ws = empty(ws_bytes, dtype=torch.uint8)
    with torch.cuda.device(dev):
        _check(lib.cce_logprobs(ctypes.byref(p), _ptr(E), _ptr(rows), _ptr(scale), _ptr(bias), _ptr(tokens),
                                _ptr(logprobs), _ptr(entropy), _ptr(lse), _ptr(tile_max), _ptr(top_lp), _ptr(top_ids),
                                _ptr(ws), ws_bytes, _stream(dev)))
        if check:
            _check(lib.cce_check_device_error(_ptr(ws), _stream(dev)))
    return logprobs, entropy, lse, tile_max, top_lp, top_ids


def cce_logprobs_backward(E: torch.Tensor, C: torch.Tensor, tokens: torch.Tensor, lse: torch.Tensor,
                          entropy: torch.Tensor, tile_max: Optional[torch.Tensor],
                          grad_logprobs: Optional[torch.Tensor], grad_entropy: Optional[torch.Tensor],
                          filter_eps: float = 0.0, bias: Optional[torch.Tensor] = None, dbias: Optional[bool] = None,
                          temperature: float = 1.0, ignore_index: int = -100, out_fp32: int = ops.OUT_BF16,
                          check: bool = False):
    """Run the backward of ``cce_logprobs``. Returns (dE, dC, filtered_tiles) as device tensors, then
    dbias when it is computed (by default whenever ``bias`` is given)."""
    lib = ops.load_library()
    _require(E.dim() == 2, f"E must be 2-D, got {tuple(E.shape)}")
    E = _flat(E)
    N, D = E.shape
    _require(isinstance(C, torch.Tensor), "a classifier of 8-bit integers has no gradient")
    rows, _ = _check_classifier(C, D)
    V = rows.shape[0]
    _check_scalars(0, V, temperature)
    _require(tokens.dtype == torch.int64 and tokens.dim() == 2 and tokens.shape[0] == N,
             f"tokens must be int64 [{N}, K], got {tokens.dtype} {tuple(tokens.shape)}")
    K = tokens.shape[1]
    _require(1 <= K <= MAX_TOKENS, f"1 to {MAX_TOKENS} tokens a position, got {K}")
    for name, t, n in (("lse", lse, N), ("entropy", entropy, N), ("grad_logprobs", grad_logprobs, N * K),
                       ("grad_entropy", grad_entropy, N)):
        _require(t is None or (t.dtype == torch.float32 and t.numel() == n), f"{name} must be float32 with {n} entries")
    if filter_eps > 0.0:
        need = -(-V // 64) * N
        _require(tile_max is not None and tile_max.dtype == torch.float32 and tile_max.numel() >= need,
                 f"filter_eps > 0 needs tile_max, float32 with at least {need} entries")
    mode = int(out_fp32)
    _require(mode in (ops.OUT_BF16, ops.OUT_FP32, ops.OUT_DE_FP32), f"out_fp32 must be 0, 1 or 2, got {out_fp32!r}")
    dev = _require_cuda(*(t for t in (E, rows, tokens, lse, entropy, tile_max, grad_logprobs, grad_entropy)
                          if t is not None))
    E, rows, bias = _aligned(E), _aligned(rows), _aligned(_bias_arg(bias, V, dev))
    tokens, lse, entropy = tokens.contiguous(), lse.contiguous(), entropy.contiguous()
    g_lp = None if grad_logprobs is None else grad_logprobs.contiguous()
    g_h = None if grad_entropy is None else grad_entropy.contiguous()
    tile_max = None if tile_max is None else tile_max.contiguous()
    want_dbias = (bias is not None) if dbias is None else bool(dbias)
    p = _problem(N, D, V, ignore_index, K, 0, temperature, False)
    ws_bytes = lib.cce_logprobs_backward_workspace_size(ctypes.byref(p), mode)
    _require(ws_bytes > 0, f"bad problem: {lib.cce_last_error_message().decode()}")
    de_dtype = torch.float32 if mode in (ops.OUT_FP32, ops.OUT_DE_FP32) else torch.bfloat16
    dc_dtype = torch.float32 if mode == ops.OUT_FP32 else torch.bfloat16
    dE = torch.empty(N, D, device=dev, dtype=de_dtype)
    dC = torch.empty(V, D, device=dev, dtype=dc_dtype)
    db = torch.empty(V, device=dev, dtype=dc_dtype) if want_dbias else None
    filtered = torch.empty(1, device=dev, dtype=torch.int64)
    ws = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    with torch.cuda.device(dev):
        _check(lib.cce_logprobs_backward(ctypes.byref(p), _ptr(E), _ptr(rows), _ptr(bias), _ptr(tokens), _ptr(lse),
                                         _ptr(entropy), _ptr(tile_max), _ptr(g_lp), _ptr(g_h), float(filter_eps),
                                         _ptr(dE), _ptr(dC), _ptr(db), mode, _ptr(filtered), _ptr(ws), ws_bytes,
                                         _stream(dev)))
        if check:
            _check(lib.cce_check_device_error(_ptr(ws), _stream(dev)))
    return (dE, dC, filtered) + ((db,) if want_dbias else ())


class _LinearLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, E, C, bias, tokens, top_k, temperature, ignore_index, filter_eps):
        logprobs, entropy, lse, tile_max, top_lp, top_ids = cce_logprobs(
            E, C, tokens, top_k, bias, temperature, ignore_index, save_max=filter_eps > 0.0)
        ctx.save_for_backward(E, C, bias, tokens, lse, entropy, tile_max)
        ctx.cfg = (temperature, ignore_index, filter_eps)
        ctx.set_materialize_grads(False)
        if top_k:
            ctx.mark_non_differentiable(top_lp, top_ids)
        return logprobs, entropy, top_lp, top_ids

    @staticmethod
    def backward(ctx, grad_logprobs, grad_entropy, _lp, _ids):
        E, C, bias, tokens, lse, entropy, tile_max = ctx.saved_tensors
        temperature, ignore_index, filter_eps = ctx.cfg
        want_db = bias is not None and ctx.needs_input_grad[2]
        out = cce_logprobs_backward(E, C, tokens, lse, entropy, tile_max, grad_logprobs, grad_entropy, filter_eps,
                                    bias, want_db, temperature, ignore_index)
        dbias = out[3].to(bias.dtype).reshape(bias.shape) if want_db else None
        return out[0], out[1], dbias, None, None, None, None, None


def linear_logprobs(e: torch.Tensor, c: Classifier, tokens: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    temperature: float = 1.0, ignore_index: int = -100, top_k: int = 0, filter_eps: float = 0.0,
                    shift: bool = False) -> Logprobs:
    """Log-probabilities of given tokens under softmax((e @ c.T + bias) / temperature), and its entropy.

    e: [..., D] bf16 hidden states; c: [V, D] bf16 classifier or ``Int8Rows`` (no gradient); bias:
    optional [V]. tokens: int64, one a position in the shape e.shape[:-1], or up to 32 a position in the
    shape [..., K] (a token may be given twice). A token equal to ``ignore_index`` asks for nothing: 0,
    without a gradient; a position where every token does has entropy 0 and gives no gradient, whatever
    its hidden state holds. Other tokens outside [0, V) give NaN.

    Gradients of both outputs flow to e, c and bias (policy gradients with an entropy bonus, preference
    losses, distillation on a teacher's alternatives). They are exact by default; ``filter_eps`` > 0
    skips units of 128 positions x 64 tokens whose probabilities are all below it, as
    ``linear_cross_entropy`` does, except units that hold a given token.

    top_k: also return the top_k (up to 24) most probable tokens of each position, without gradients,
    as ``linear_top_logprobs`` does. ``shift`` makes e[..., i, :] predict tokens[..., i + 1] (one token a
    position); every output is then one position shorter along the sequence axis.
    """
    lead = e.shape[:-1]
    if tokens.shape == lead:
        many = False
    elif tokens.dim() == e.dim() and tokens.shape[:-1] == lead:
        many = True
    else:
        raise ValueError(f"tokens shape {tuple(tokens.shape)} must equal e.shape[:-1] {tuple(lead)}, "
                         "with or without a last dimension of several tokens")
    if shift:
        if many or not lead or lead[-1] < 1:
            raise ValueError("shift needs one token a position and a sequence axis of length >= 1")
        tokens = ops.shift_targets(tokens, ignore_index)
    E = _flat(e)
    t = tokens.to(torch.int64).reshape(E.shape[0], -1) if E.shape[0] else \
        tokens.to(torch.int64).reshape(0, tokens.shape[-1] if many else 1)
    if isinstance(c, Int8Rows):
        if torch.is_grad_enabled() and (e.requires_grad or (bias is not None and bias.requires_grad)):
            raise ValueError("a classifier of 8-bit integers has no gradient: call under torch.no_grad(), or detach e "
                             "and bias")
        logprobs, entropy, _, _, top_lp, top_ids = cce_logprobs(E, c, t, top_k, bias, temperature, ignore_index)
    else:
        logprobs, entropy, top_lp, top_ids = _LinearLogprobs.apply(E, c, bias, t, int(top_k), float(temperature),
                                                                   ignore_index, float(filter_eps))
    out = Logprobs(logprobs.reshape(tokens.shape), entropy.reshape(lead),
                   None if top_lp is None else top_lp.reshape(*lead, top_k),
                   None if top_ids is None else top_ids.reshape(*lead, top_k))
    if not shift:
        return out
    return Logprobs(out.logprobs[..., :-1], out.entropy[..., :-1],
                    None if top_lp is None else out.top_logprobs[..., :-1, :],
                    None if top_ids is None else out.top_ids[..., :-1, :])


def linear_top_logprobs(e: torch.Tensor, c: Classifier, k: int, bias: Optional[torch.Tensor] = None,
                        temperature: float = 1.0) -> TopLogprobs:
    """The k (1 to 24) most probable tokens of each position under softmax((e @ c.T + bias) /
    temperature) and their log-probabilities, highest first, the lower id first among equal ones.

    Close alternatives are ordered by their logits in 64 bits, so the ids depend neither on the batch
    they are computed in nor on how the work was split. No gradient flows.
    """
    if k < 1:
        raise ValueError(f"k must be at least 1, got {k}")
    with torch.no_grad():
        E = _flat(e)
        out = cce_logprobs(E, c, None, int(k), bias, float(temperature))
    lead = e.shape[:-1]
    return TopLogprobs(out[4].reshape(*lead, k), out[5].reshape(*lead, k))


def quantize_int8(x: torch.Tensor) -> Int8Rows:
    """Rows of x [rows, D] (bf16) as 8-bit integers with one scale each: scale = max |x| / 127 and
    values = x / scale, rounded to the nearest integer, halves to the even one. D must be a multiple of
    16. A row of zeros gets scale 0; a row that holds an infinity or a NaN gets the scale NaN."""
    lib = ops.load_library()
    _require(x.dim() == 2 and x.dtype == torch.bfloat16, f"x must be bfloat16 [rows, D], got {x.dtype} {tuple(x.shape)}")
    _require(x.shape[1] >= 16 and x.shape[1] % 16 == 0, f"D must be a positive multiple of 16, got {x.shape[1]}")
    dev = _require_cuda(x)
    x = _aligned(x.detach())
    out = Int8Rows(torch.empty(x.shape, device=dev, dtype=torch.int8),
                   torch.empty(x.shape[0], device=dev, dtype=torch.float32))
    with torch.cuda.device(dev):
        _check(lib.cce_quantize_int8(_ptr(x), x.shape[0], x.shape[1], _ptr(out.values), _ptr(out.scale), _stream(dev)))
    return out


def int8_linear(e: torch.Tensor, c: Int8Rows, bias: Optional[torch.Tensor] = None,
                out_dtype: torch.dtype = torch.bfloat16, check: bool = False) -> torch.Tensor:
    """The logits e @ c.T + bias [..., V] of a classifier of 8-bit integers, in bf16 or fp32.

    Each row of e (bf16) is rounded to 8-bit integers with a scale of its own, the sums of integer
    products are exact, and the two scales and the bias are applied in fp32. No gradient flows."""
    lib = ops.load_library()
    _require(isinstance(c, Int8Rows), f"c must be Int8Rows (see quantize_int8), got {type(c).__name__}")
    _require(out_dtype in (torch.bfloat16, torch.float32), f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    E = _flat(e).detach()
    N, D = E.shape
    rows, scale = _check_classifier(c, D)
    V = rows.shape[0]
    dev = _require_cuda(E, rows, scale)
    E, rows, scale = _aligned(E), _aligned(rows), _aligned(scale)
    bias = _aligned(_bias_arg(None if bias is None else bias.detach(), V, dev))
    ws_bytes = lib.cce_int8_linear_workspace_size(N, D, V)
    _require(ws_bytes > 0, f"bad problem N={N} D={D} V={V}")
    out = torch.empty(N, V, device=dev, dtype=out_dtype)
    ws = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    with torch.cuda.device(dev):
        _check(lib.cce_int8_linear(N, D, V, _ptr(E), _ptr(rows), _ptr(scale), _ptr(bias), _ptr(out),
                                   int(out_dtype == torch.float32), _ptr(ws), ws_bytes, _stream(dev)))
        if check:
            _check(lib.cce_check_device_error(_ptr(ws), _stream(dev)))
    return out.reshape(*e.shape[:-1], V)
