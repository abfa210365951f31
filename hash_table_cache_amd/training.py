"""Training operators between a table's ``find`` and its ``assign``.

ctypes binding of ``libhkv_train.so`` (the C ABI of ``include/hkv_train.h``,
which states the formulas): every step runs in the HIP library; the functions
here check their arguments, allocate outputs and workspace and pass pointers.
There is no fallback implementation.

Logits are two-dimensional [rows, vocab] tensors of float32, bfloat16 or
float16 whose rows may lie inside wider ones (stride(0) >= vocab, stride(1) ==
1). Labels are int64; a negative one leaves its row out. Work is enqueued on
``stream`` (a ``torch.cuda.Stream`` or a handle; torch's current stream by
default), and what a call allocates belongs to that stream. Gradients are
returned, not recorded: pass one on with ``logits.backward(grad)``. A gradient
written over its logits (``grad_out=logits``) is written behind autograd's back;
what ``orthogonalize`` and ``muon_update`` write in place counts as modified, so that
a backward pass that saved it fails instead of taking the new values.
"""

from __future__ import annotations

import array
import ctypes
import functools
import math
import operator
import pathlib
import struct
from typing import NamedTuple, Optional

import torch

from ._native import HKV_OK, HkvError

LIB_PATH = pathlib.Path(__file__).resolve().parent / "_lib" / "libhkv_train.so"

# Every entry point declared in include/hkv_train.h.
EXPORTS = (
    "hkv_train_workspace_bytes",
    "hkv_token_logprobs",
    "hkv_token_logprobs_backward",
    "hkv_token_stats_workspace_bytes",
    "hkv_token_stats",
    "hkv_token_stats_backward",
    "hkv_preference_loss",
    "hkv_policy_loss",
    "hkv_clip_grad_norm",
    "hkv_orthogonalize_workspace_bytes",
    "hkv_orthogonalize",
    "hkv_muon_update",
    "hkv_train_last_error",
)

KINDS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class TokenStats(NamedTuple):
    logp: torch.Tensor  # [rows] float32
    lse: torch.Tensor  # [rows] float32
    entropy: torch.Tensor  # [rows] float32
    top_logp: torch.Tensor  # [rows, k] float32, falling
    top_ids: torch.Tensor  # [rows, k] int64, -1 past a row's last candidate


class PreferenceLoss(NamedTuple):
    loss: torch.Tensor  # [] float32: the mean over pairs
    losses: torch.Tensor  # [pairs] float32
    rewards: torch.Tensor  # [2 * pairs] float32
    logp: torch.Tensor  # [rows] float32
    grad: Optional[torch.Tensor]  # like logits


class PolicyLoss(NamedTuple):
    loss: torch.Tensor  # [] float32: the weighted sum
    token_loss: torch.Tensor  # [rows] float32
    kl: torch.Tensor  # [rows] float32
    logp: torch.Tensor  # [rows] float32
    grad: Optional[torch.Tensor]  # like logits


def _load() -> ctypes.CDLL:
    if not LIB_PATH.exists():
        raise ImportError(
            f"{LIB_PATH} is missing; build it with `python -m hash_table_cache_amd.build`"
        )
    L = ctypes.CDLL(str(LIB_PATH))
    vp, u64, u32, f32, st = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_float, ctypes.c_int32
    logits = [u64, u64, u32, vp, u64, vp, f32]
    L.hkv_train_workspace_bytes.argtypes = [u64, u64, u64]
    L.hkv_train_workspace_bytes.restype = u64
    L.hkv_token_logprobs.argtypes = [*logits, vp, vp, vp, u64, vp]
    L.hkv_token_logprobs.restype = st
    L.hkv_token_logprobs_backward.argtypes = [*logits, vp, vp, vp, u64, vp]
    L.hkv_token_logprobs_backward.restype = st
    L.hkv_token_stats_workspace_bytes.argtypes = [u64, u64, u32, u32]
    L.hkv_token_stats_workspace_bytes.restype = u64
    L.hkv_token_stats.argtypes = [*logits, u32, vp, vp, vp, vp, vp, vp, u64, vp]
    L.hkv_token_stats.restype = st
    L.hkv_token_stats_backward.argtypes = [*logits, vp, vp, vp, vp, vp, u64, vp]
    L.hkv_token_stats_backward.restype = st
    L.hkv_preference_loss.argtypes = [*logits, u64, vp, vp, f32, f32, f32, vp, vp, vp, vp, vp, u64, vp, u64, vp]
    L.hkv_preference_loss.restype = st
    L.hkv_policy_loss.argtypes = [*logits, vp, vp, vp, vp, f32, f32, f32, f32, vp, vp, vp, vp, vp, u64, vp, u64, vp]
    L.hkv_policy_loss.restype = st
    L.hkv_clip_grad_norm.argtypes = [u64, vp, vp, vp, vp, f32, vp, vp, u64, vp]
    L.hkv_clip_grad_norm.restype = st
    f64 = ctypes.c_double
    L.hkv_orthogonalize_workspace_bytes.argtypes = [u64, vp, vp, vp]
    L.hkv_orthogonalize_workspace_bytes.restype = u64
    L.hkv_orthogonalize.argtypes = [u64, vp, u32, vp, f64, vp, u64, vp]
    L.hkv_orthogonalize.restype = st
    L.hkv_muon_update.argtypes = [u64, vp, f64, u32, f64, u32, vp, f64, vp, u64, vp]
    L.hkv_muon_update.restype = st
    L.hkv_train_last_error.argtypes = []
    L.hkv_train_last_error.restype = ctypes.c_char_p
    return L


_LIB = None


def load() -> ctypes.CDLL:
    """The loaded ``libhkv_train.so`` (loaded on the first call)."""
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def _check(status: int) -> None:
    if status != HKV_OK:
        raise HkvError(status, load().hkv_train_last_error().decode(errors="replace"))


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_stream(device):
    """Handle of torch's current stream: the raw lookup where torch has it (the
    public one builds a Stream object, 2 us of every call)."""
    return _raw_stream(device.index) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream


def _on(stream, device):
    """Context in which a call's tensors are allocated on, and its work goes to,
    the stream that its caller named."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        stream = (torch.cuda.ExternalStream(handle, device=device) if handle
                  else torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


def _logits(x, labels):
    if x.dtype not in KINDS:
        raise TypeError(f"logits: dtype {x.dtype} not in {tuple(KINDS)}")
    if x.dim() != 2:
        raise ValueError(f"logits must have two dimensions, rows and vocab, not {x.dim()}")
    if not x.is_cuda:
        raise ValueError("logits must be on a GPU")
    rows, vocab = x.shape
    if vocab == 0:
        raise ValueError("logits have no columns")
    _vector(labels, torch.int64, rows, "labels", x.device)
    return rows, vocab, _row_stride(x, "logits")


def _row_stride(x, name):
    rows, vocab = x.shape
    s0, s1 = x.stride()
    if vocab > 1 and s1 != 1:
        raise ValueError(f"{name}: the elements of a row must be next to each other (stride(1) is {s1})")
    if rows > 1 and s0 < vocab:
        raise ValueError(f"{name}: rows overlap (stride(0) is {s0}, vocab {vocab})")
    return s0 if rows > 1 else vocab


def _vector(t, dtype, numel, name, device):
    if (t is not None and t.dtype is dtype and t.dim() == 1 and t.numel() == numel and t.is_contiguous()
            and t.get_device() == device.index):
        return t.data_ptr()
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype} is not {dtype}")
    if t.dim() != 1 or t.shape[0] != numel:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, needs [{numel}]")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, logits on {device}")


def _grad(x, grad_out):
    """The tensor that takes the gradient, and its row stride."""
    if grad_out is None:
        grad = torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        return grad, x.shape[1]
    if grad_out.dtype != x.dtype or grad_out.shape != x.shape or grad_out.device != x.device:
        raise ValueError(f"grad_out: {grad_out.dtype} {tuple(grad_out.shape)} on {grad_out.device}, "
                         f"logits are {x.dtype} {tuple(x.shape)} on {x.device}")
    return grad_out, _row_stride(grad_out, "grad_out")


@functools.lru_cache(maxsize=256)
def _workspace_bytes(rows, pairs, tensors):
    return load().hkv_train_workspace_bytes(rows, pairs, tensors)


# Results have memory of their own each, and the workspace goes when the call
# returns: parts of one allocation would cost a call 2 us less, but a kept logp
# would hold all of it, torch.save would write all of it, and autograd would
# take a write into one result for a write into the others.
def _floats(size, device):
    return torch.empty(size, dtype=torch.float32, device=device)


def _scalar(device):
    return torch.empty_strided((), (), dtype=torch.float32, device=device)


def _workspace(size, device):
    return torch.empty(size, dtype=torch.uint8, device=device)


def token_logprobs(logits, labels, *, temperature: float = 1.0, stream=None):
    """(logp, lse), both [rows] float32: the log-probability of each row's
    label under softmax(logits / temperature), and the normaliser. Autograd does
    not follow them: a loss made of logp gives its gradient with respect to logp
    to token_logprobs_backward."""
    if stream is not None:
        with _on(stream, logits.device):
            return token_logprobs(logits, labels, temperature=temperature)
    rows, vocab, stride = _logits(logits, labels)
    dev = logits.device
    logp, lse = _floats(rows, dev), _floats(rows, dev)
    ws, nb = None, 0
    if rows < 64 and vocab * logits.element_size() > 1 << 18:  # few long rows, the only ones that take a workspace
        nb = _workspace_bytes(rows, 0, 0)
        ws = _workspace(nb, dev)
    _check(load().hkv_token_logprobs(rows, vocab, KINDS[logits.dtype], logits.data_ptr(), stride, labels.data_ptr(),
                                     temperature, logp.data_ptr(), lse.data_ptr(), ws if ws is None else ws.data_ptr(),
                                     nb, _current_stream(dev)))
    return logp, lse


def token_logprobs_backward(logits, labels, lse, grad_logp, *, temperature: float = 1.0, grad_out=None, stream=None):
    """The gradient of (grad_logp * logp).sum() with respect to the logits;
    grad_out takes it where given (it may be the logits, or other columns of
    their rows)."""
    if stream is not None:
        with _on(stream, logits.device):
            return token_logprobs_backward(logits, labels, lse, grad_logp, temperature=temperature, grad_out=grad_out)
    rows, vocab, stride = _logits(logits, labels)
    dev = logits.device
    z = _vector(lse, torch.float32, rows, "lse", dev)
    g = _vector(grad_logp, torch.float32, rows, "grad_logp", dev)
    grad_out, gstride = _grad(logits, grad_out)
    _check(load().hkv_token_logprobs_backward(rows, vocab, KINDS[logits.dtype], logits.data_ptr(), stride,
                                              labels.data_ptr(), temperature, z, g, grad_out.data_ptr(), gstride,
                                              _current_stream(dev)))
    return grad_out


@functools.lru_cache(maxsize=256)
def _stats_workspace_bytes(rows, vocab, kind, k):
    return load().hkv_token_stats_workspace_bytes(rows, vocab, kind, k)


def token_stats(logits, labels, k: int = 0, *, temperature: float = 1.0, stream=None) -> TokenStats:
    """token_logprobs with the entropy of each row's distribution and its k
    largest logits (k <= 64), as log-probabilities with their indices, the
    lowest index first among equal ones. Masked logits (-inf) are no
    alternatives: past a row's last candidate, and in rows that are left out,
    top_ids is -1 and top_logp -inf."""
    if stream is not None:
        with _on(stream, logits.device):
            return token_stats(logits, labels, k, temperature=temperature)
    rows, vocab, stride = _logits(logits, labels)
    k = operator.index(k)
    if not 0 <= k <= 64:
        raise ValueError(f"k = {k} is outside 0 .. 64")
    dev, kind = logits.device, KINDS[logits.dtype]
    logp, lse, entropy = _floats(rows, dev), _floats(rows, dev), _floats(rows, dev)
    top_logp = _floats((rows, k), dev)
    top_ids = torch.empty((rows, k), dtype=torch.int64, device=dev)
    nb = _stats_workspace_bytes(rows, vocab, kind, k)
    ws = _workspace(nb, dev) if nb else None
    _check(load().hkv_token_stats(rows, vocab, kind, logits.data_ptr(), stride, labels.data_ptr(), temperature, k,
                                  logp.data_ptr(), lse.data_ptr(), entropy.data_ptr(), top_logp.data_ptr(),
                                  top_ids.data_ptr(), ws if ws is None else ws.data_ptr(), nb, _current_stream(dev)))
    return TokenStats(logp, lse, entropy, top_logp, top_ids)


def token_stats_backward(logits, labels, lse, entropy=None, grad_logp=None, grad_entropy=None, *,
                         temperature: float = 1.0, grad_out=None, stream=None):
    """The gradient of (grad_logp * logp).sum() + (grad_entropy *
    entropy).sum() with respect to the logits. lse and entropy are
    token_stats's; one of the two gradients may be left out, and without
    grad_entropy entropy too. grad_out as in token_logprobs_backward."""
    if stream is not None:
        with _on(stream, logits.device):
            return token_stats_backward(logits, labels, lse, entropy, grad_logp, grad_entropy,
                                        temperature=temperature, grad_out=grad_out)
    rows, vocab, stride = _logits(logits, labels)
    dev = logits.device
    if grad_logp is None and grad_entropy is None:
        raise ValueError("grad_logp or grad_entropy is required")
    z = _vector(lse, torch.float32, rows, "lse", dev)
    g = None if grad_logp is None else _vector(grad_logp, torch.float32, rows, "grad_logp", dev)
    h = ge = None
    if grad_entropy is not None:
        ge = _vector(grad_entropy, torch.float32, rows, "grad_entropy", dev)
        h = _vector(entropy, torch.float32, rows, "entropy", dev)
    grad_out, gstride = _grad(logits, grad_out)
    _check(load().hkv_token_stats_backward(rows, vocab, KINDS[logits.dtype], logits.data_ptr(), stride,
                                           labels.data_ptr(), temperature, z, h, g, ge, grad_out.data_ptr(), gstride,
                                           _current_stream(dev)))
    return grad_out


def preference_loss(logits, labels, cu_seqlens, ref_logp=None, *, beta: float = 0.1, label_smoothing: float = 0.0,
                    temperature: float = 1.0, grad_scale: float = 1.0, with_grad: bool = True, grad_out=None,
                    stream=None) -> PreferenceLoss:
    """Preference loss on pairs of sequences: 2p preferred to 2p + 1, each the
    rows [cu_seqlens[s], cu_seqlens[s + 1]). cu_seqlens: [2 * pairs + 1] int64;
    ref_logp: [rows] float32 log-probabilities of the reference (token_logprobs
    of its logits), 0 where not given. grad is grad_scale times the gradient of
    loss; with_grad=False leaves it out."""
    if stream is not None:
        with _on(stream, logits.device):
            return preference_loss(logits, labels, cu_seqlens, ref_logp, beta=beta, label_smoothing=label_smoothing,
                                   temperature=temperature, grad_scale=grad_scale, with_grad=with_grad,
                                   grad_out=grad_out)
    rows, vocab, stride = _logits(logits, labels)
    dev = logits.device
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] % 2 != 1:
        raise ValueError(f"cu_seqlens has shape {tuple(cu_seqlens.shape)}, needs [2 * pairs + 1]")
    pairs = cu_seqlens.shape[0] // 2
    cu = _vector(cu_seqlens, torch.int64, 2 * pairs + 1, "cu_seqlens", dev)
    ref = None if ref_logp is None else _vector(ref_logp, torch.float32, rows, "ref_logp", dev)
    loss, losses, rewards, logp = _scalar(dev), _floats(pairs, dev), _floats(2 * pairs, dev), _floats(rows, dev)
    nb = _workspace_bytes(rows, pairs, 0)
    ws = _workspace(nb, dev)
    grad, gstride = _grad(logits, grad_out) if with_grad else (None, 0)
    _check(load().hkv_preference_loss(rows, vocab, KINDS[logits.dtype], logits.data_ptr(), stride, labels.data_ptr(),
                                      temperature, pairs, cu, ref, beta, label_smoothing, grad_scale,
                                      loss.data_ptr(), losses.data_ptr(), rewards.data_ptr(), logp.data_ptr(),
                                      None if grad is None else grad.data_ptr(), gstride, ws.data_ptr(), nb,
                                      _current_stream(dev)))
    return PreferenceLoss(loss, losses, rewards, logp, grad)


def policy_loss(logits, labels, old_logp, advantages, weights, ref_logp=None, *, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0, grad_scale: float = 1.0,
                with_grad: bool = True, grad_out=None, stream=None) -> PolicyLoss:
    """Clipped policy loss with a divergence term. old_logp, advantages,
    weights (what each row counts in the sum), ref_logp: [rows] float32; a
    kl_coef needs ref_logp. grad is grad_scale times the gradient of loss;
    with_grad=False leaves it out."""
    if stream is not None:
        with _on(stream, logits.device):
            return policy_loss(logits, labels, old_logp, advantages, weights, ref_logp, clip_low=clip_low,
                               clip_high=clip_high, kl_coef=kl_coef, temperature=temperature, grad_scale=grad_scale,
                               with_grad=with_grad, grad_out=grad_out)
    rows, vocab, stride = _logits(logits, labels)
    dev = logits.device
    old = _vector(old_logp, torch.float32, rows, "old_logp", dev)
    adv = _vector(advantages, torch.float32, rows, "advantages", dev)
    wts = _vector(weights, torch.float32, rows, "weights", dev)
    ref = None if ref_logp is None else _vector(ref_logp, torch.float32, rows, "ref_logp", dev)
    if kl_coef != 0.0 and ref is None:
        raise ValueError("kl_coef needs ref_logp")
    loss, token_loss, kl, logp = _scalar(dev), _floats(rows, dev), _floats(rows, dev), _floats(rows, dev)
    nb = _workspace_bytes(rows, 0, 0)
    ws = _workspace(nb, dev)
    grad, gstride = _grad(logits, grad_out) if with_grad else (None, 0)
    _check(load().hkv_policy_loss(rows, vocab, KINDS[logits.dtype], logits.data_ptr(), stride, labels.data_ptr(),
                                  temperature, old, adv, wts, ref, clip_low, clip_high, kl_coef, grad_scale,
                                  loss.data_ptr(), token_loss.data_ptr(), kl.data_ptr(), logp.data_ptr(),
                                  None if grad is None else grad.data_ptr(), gstride, ws.data_ptr(), nb,
                                  _current_stream(dev)))
    return PolicyLoss(loss, token_loss, kl, logp, grad)


_dtype = operator.attrgetter("dtype")


def _dense(t) -> bool:
    """Whether t's elements fill one stretch of memory, in whatever order of its axes."""
    if t.is_contiguous():
        return True
    want = 1
    for size, step in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n != 1), key=lambda p: p[1]):
        if step != want:
            return False
        want *= size
    return True


def clip_grad_norm(grads, max_norm: float, *, out=None, stream=None):
    """Scales the gradients (a sequence of tensors, of mixed float types) so
    that their global 2-norm is at most max_norm; returns the norm that they
    had ([] float32, on their GPU). out: tensors of the gradients' types and
    sizes that take the result (by default it replaces them). Each tensor has
    to fill one stretch of memory; the order of its axes is free, and out's is
    the same."""
    grads = list(grads)
    if not grads:
        raise ValueError("clip_grad_norm needs at least one tensor")
    if stream is not None:
        with _on(stream, grads[0].device):
            return clip_grad_norm(grads, max_norm, out=out)
    dev, n = grads[0].device, len(grads)
    if dev.type != "cuda":
        raise ValueError("gradients must be on a GPU")
    dtypes = list(map(_dtype, grads))
    try:
        kinds = bytes(map(KINDS.__getitem__, dtypes))
    except KeyError:
        i = next(i for i, d in enumerate(dtypes) if d not in KINDS)
        raise TypeError(f"gradient {i}: dtype {dtypes[i]} not in {tuple(KINDS)}") from None
    in_order = all(map(torch.Tensor.is_contiguous, grads))
    if not in_order:
        for i, g in enumerate(grads):
            if not _dense(g):
                raise ValueError(f"gradient {i} does not fill one stretch of memory (strides {g.stride()})")
    # on which GPU each lies is asked of its address, by the library
    ptrs = array.array("Q", map(torch.Tensor.data_ptr, grads))
    numel = array.array("Q", map(torch.Tensor.numel, grads))
    optrs = None
    if out is not None:
        outs = list(out)
        if len(outs) != n:
            raise ValueError(f"{len(outs)} tensors in out, {n} gradients")
        in_order = in_order and all(map(torch.Tensor.is_contiguous, outs))
        if (list(map(_dtype, outs)) != dtypes or array.array("Q", map(torch.Tensor.numel, outs)) != numel
                or not (in_order or [(o.shape, o.stride()) for o in outs] == [(g.shape, g.stride()) for g in grads])):
            for i, (g, o) in enumerate(zip(grads, outs)):
                if (o.dtype, o.numel()) != (g.dtype, g.numel()) or not (
                        (o.shape, o.stride()) == (g.shape, g.stride()) or (o.is_contiguous() and g.is_contiguous())):
                    raise ValueError(f"out {i}: {o.dtype} {tuple(o.shape)} with strides {o.stride()}, its gradient is "
                                     f"{g.dtype} {tuple(g.shape)} with strides {g.stride()}")
        optrs = array.array("Q", map(torch.Tensor.data_ptr, outs))
    norm = _scalar(dev)
    nb = _workspace_bytes(0, 0, n)
    ws = _workspace(nb, dev)
    _check(load().hkv_clip_grad_norm(n, ptrs.buffer_info()[0], optrs and optrs.buffer_info()[0],
                                     numel.buffer_info()[0], kinds, max_norm, norm.data_ptr(), ws.data_ptr(),
                                     nb, _current_stream(dev)))
    return norm


# Steps of X <- a X + (b A + c A A) X, A = X X^T, that take singular values to
# between 0.68 and 1.13 from anywhere above 0.01 in five.
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


_MUON_MATRIX = struct.Struct("10Q2d")  # hkv_muon_matrix


def _matrix(t, name, i):
    """Type and row stride of one matrix of a list."""
    if t.dtype not in KINDS:
        raise TypeError(f"{name} {i}: dtype {t.dtype} not in {tuple(KINDS)}")
    if t.dim() != 2:
        raise ValueError(f"{name} {i} must have two dimensions, not {t.dim()}")
    rows, cols = t.shape
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        raise ValueError(f"{name} {i}: the elements of a row must be next to each other (stride(1) is {s1})")
    if rows > 1 and s0 < cols:
        raise ValueError(f"{name} {i}: rows overlap (stride(0) is {s0}, {cols} columns)")
    return KINDS[t.dtype], s0 if rows > 1 else cols


_modified = torch.autograd.graph.increment_version  # tensors that were written by address


@functools.lru_cache(maxsize=64)
def _steps(steps, coefficients):
    """a, b, c of every step, for a triple or a sequence of them."""
    steps = operator.index(steps)
    if not 1 <= steps <= 64:
        raise ValueError(f"steps = {steps} is outside 1 .. 64")
    flat = coefficients if isinstance(coefficients[0], tuple) else (coefficients,) * steps
    if len(flat) != steps or any(len(c) != 3 for c in flat):
        raise ValueError(f"coefficients: a triple, or one for each of {steps} steps")
    return array.array("d", [float(v) for c in flat for v in c])


def _coefficients(steps, coefficients):
    return _steps(steps, tuple(tuple(c) if isinstance(c, (list, tuple)) else c for c in coefficients))


@functools.lru_cache(maxsize=64)
def _polar_workspace_bytes(shapes, kinds):
    rows, cols = (array.array("Q", [s[i] for s in shapes]) for i in (0, 1))
    return load().hkv_orthogonalize_workspace_bytes(len(shapes), rows.buffer_info()[0], cols.buffer_info()[0], kinds)


def orthogonalize(matrices, *, steps: int = 5, coefficients=NEWTON_SCHULZ, eps: float = 1e-7, out=None, stream=None):
    """The matrices of a sequence (of mixed types and shapes) drawn towards the
    nearest orthogonal ones by Newton-Schulz steps; returns a list of tensors.
    coefficients: a, b, c, or a sequence of `steps` such triples. out: tensors of
    the matrices' shapes that take the results (they may be the matrices); their
    types decide the precision, float32 and float16 being computed as precisely
    as float32 is, bfloat16 to less than its rounding with the coefficients and up
    to 6 steps (include/hkv_train.h has the exceptions)."""
    matrices = list(matrices)
    if not matrices:
        raise ValueError("orthogonalize needs at least one matrix")
    dev = matrices[0].device
    if dev.type != "cuda":
        raise ValueError("matrices must be on a GPU")
    if stream is not None:
        with _on(stream, dev):
            return orthogonalize(matrices, steps=steps, coefficients=coefficients, eps=eps, out=out)
    c = _coefficients(steps, coefficients)
    if out is None:
        out = [torch.empty(u.shape, dtype=u.dtype, device=dev) for u in matrices]
    else:
        out = list(out)
        if len(out) != len(matrices):
            raise ValueError(f"{len(out)} tensors in out, {len(matrices)} matrices")
    table, shapes, kinds = array.array("Q"), [], bytearray()
    for i, (u, o) in enumerate(zip(matrices, out)):
        kind, stride = _matrix(u, "matrix", i)
        okind, ostride = _matrix(o, "out", i)
        if o.shape != u.shape:
            raise ValueError(f"out {i}: {tuple(o.shape)}, its matrix is {tuple(u.shape)}")
        table.extend((u.data_ptr(), o.data_ptr(), *u.shape, stride, ostride, kind, okind))
        shapes.append(tuple(u.shape))
        kinds.append(okind)
    nb = _polar_workspace_bytes(tuple(shapes), bytes(kinds))
    ws = _workspace(nb, dev)
    _check(load().hkv_orthogonalize(len(matrices), table.buffer_info()[0], steps, c.buffer_info()[0], eps,
                                    ws.data_ptr(), nb, _current_stream(dev)))
    _modified(out)
    return out


def muon_update(weights, grads, momenta, lr, *, momentum: float = 0.95, nesterov: bool = True,
                weight_decay: float = 0.0, scale: Optional[str] = "shape", steps: int = 5,
                coefficients=NEWTON_SCHULZ, eps: float = 1e-7, stream=None) -> None:
    """One step of dense weight matrices, in place, by their orthogonalised
    momentum. weights, grads: sequences of matrices, each of a float type;
    momenta: float32, kept by the caller (zeros at first), in place too. lr: a
    number, or one for each matrix. scale multiplies lr by the matrix's shape:
    "shape" by sqrt(max(1, rows / cols)), "rms" by 0.2 sqrt(max(rows, cols)),
    which gives updates the size of an adaptive optimiser's, None by 1. The weights'
    types decide the precision as out's do in orthogonalize: a program to which
    bfloat16's is not enough keeps its weights in float32."""
    weights, grads, momenta = list(weights), list(grads), list(momenta)
    n = len(weights)
    if not weights:
        raise ValueError("muon_update needs at least one matrix")
    if len(grads) != n or len(momenta) != n:
        raise ValueError(f"{n} weights, {len(grads)} gradients, {len(momenta)} momenta")
    dev = weights[0].device
    if dev.type != "cuda":
        raise ValueError("weights must be on a GPU")
    if stream is not None:
        with _on(stream, dev):
            return muon_update(weights, grads, momenta, lr, momentum=momentum, nesterov=nesterov,
                               weight_decay=weight_decay, scale=scale, steps=steps, coefficients=coefficients, eps=eps)
    if scale not in ("shape", "rms", None):
        raise ValueError(f"scale = {scale!r} is none of 'shape', 'rms', None")
    lrs = [float(v) for v in lr] if isinstance(lr, (list, tuple)) else [float(lr)] * n
    if len(lrs) != n:
        raise ValueError(f"{len(lrs)} learning rates, {n} weights")
    c = _coefficients(steps, coefficients)
    table, shapes, kinds = bytearray(), [], bytearray()
    for i, (w, g, m) in enumerate(zip(weights, grads, momenta)):
        kind, stride = _matrix(w, "weight", i)
        gkind, gstride = _matrix(g, "gradient", i)
        mkind, mstride = _matrix(m, "momentum", i)
        if g.shape != w.shape or m.shape != w.shape:
            raise ValueError(f"matrix {i}: weight {tuple(w.shape)}, gradient {tuple(g.shape)}, momentum {tuple(m.shape)}")
        if mkind:
            raise TypeError(f"momentum {i}: dtype {m.dtype} is not {torch.float32}")
        rows, cols = shape = tuple(w.shape)
        factor = 1.0
        if scale == "shape" and cols:
            factor = math.sqrt(max(1.0, rows / cols))
        elif scale == "rms":
            factor = 0.2 * math.sqrt(max(rows, cols))
        table += _MUON_MATRIX.pack(w.data_ptr(), g.data_ptr(), m.data_ptr(), rows, cols, stride, gstride, mstride, kind,
                                   gkind, lrs[i], factor)
        shapes.append(shape)
        kinds.append(kind)
    nb = _polar_workspace_bytes(tuple(shapes), bytes(kinds))
    ws = _workspace(nb, dev)
    _check(load().hkv_muon_update(n, bytes(table), momentum, bool(nesterov), weight_decay, steps, c.buffer_info()[0],
                                  eps, ws.data_ptr(), nb, _current_stream(dev)))
    _modified(weights + momenta)
