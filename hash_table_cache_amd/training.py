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
written over its logits (``grad_out=logits``) is written behind autograd's back.
"""

from __future__ import annotations

import array
import ctypes
import functools
import operator
import pathlib
from typing import NamedTuple, Optional

import torch

from ._native import HKV_OK, HkvError

LIB_PATH = pathlib.Path(__file__).resolve().parent / "_lib" / "libhkv_train.so"

# Every entry point declared in include/hkv_train.h.
EXPORTS = (
    "hkv_train_workspace_bytes",
    "hkv_token_logprobs",
    "hkv_token_logprobs_backward",
    "hkv_preference_loss",
    "hkv_policy_loss",
    "hkv_clip_grad_norm",
    "hkv_train_last_error",
)

KINDS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


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
    L.hkv_preference_loss.argtypes = [*logits, u64, vp, vp, f32, f32, f32, vp, vp, vp, vp, vp, u64, vp, u64, vp]
    L.hkv_preference_loss.restype = st
    L.hkv_policy_loss.argtypes = [*logits, vp, vp, vp, vp, f32, f32, f32, f32, vp, vp, vp, vp, vp, u64, vp, u64, vp]
    L.hkv_policy_loss.restype = st
    L.hkv_clip_grad_norm.argtypes = [u64, vp, vp, vp, vp, f32, vp, vp, u64, vp]
    L.hkv_clip_grad_norm.restype = st
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
