"""Python binding of the verification of drafts (include/whead_verify.h): argument checks and marshalling only.

A walk drafts gamma tokens, the target gives logits after the last token and after each of them, and these calls say what they are worth:

    said, count = verify(logits, drafts, draft_logits, temperature=T, seed=seed)   # what stays, and the token after it
    cache.compact(start, keep, count)                                              # (kv.py) the others leave the cache
    r = logprobs(logits, said, top=5)                                              # log probabilities, entropy, alternatives

No gradients pass through them: inputs that ask for gradients are refused outside torch.no_grad(), inputs with forward-mode tangents everywhere.
Calls go to the current torch stream. There is no fallback: without the built library, loading raises.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

from . import whead as _wh

BF16, F16, F32 = 0, 1, 2
MAX_TOP = 32
MAX_DRAFTS = 255
MAX_ROWS = 1 << 27

# Every symbol include/whead_verify.h declares.
EXPORTS = ("whead_logprobs", "whead_verify_workspace_bytes", "whead_verify")

_vp, _i32, _i64, _u32, _u64, _f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_double


class LogprobsArgs(ctypes.Structure):
    _fields_ = [("logits", _vp), ("tokens", _vp), ("logprob", _vp), ("entropy", _vp), ("lse", _vp), ("top_tokens", _vp), ("top_logprobs", _vp),
                ("stride_n", _i64), ("stride_t", _i64), ("n", _i64), ("t", _i64), ("V", _i64), ("temperature", _f64), ("dtype", _i32),
                ("top", _i32), ("stream", _vp)]


class VerifyArgs(ctypes.Structure):
    _fields_ = [("target", _vp), ("draft", _vp), ("tokens", _vp), ("drafted", _vp), ("said", _vp), ("count", _vp), ("target_stride_n", _i64),
                ("target_stride_t", _i64), ("draft_stride_n", _i64), ("draft_stride_t", _i64), ("n", _i64), ("V", _i64), ("gamma", _i32),
                ("target_dtype", _i32), ("draft_dtype", _i32), ("step", _u32), ("temperature", _f64), ("draft_temperature", _f64),
                ("seed", _u64), ("workspace", _vp), ("workspace_bytes", _i64), ("stream", _vp)]


class LogProbs(NamedTuple):
    """What logprobs() gives, of the shape of its rows; the alternatives have one dimension more."""
    logprob: Optional[object]       # float32: of the given tokens
    entropy: object                 # float32
    lse: object                     # float32: log of the sum of exp(logits / temperature)
    top_tokens: Optional[object]    # int32, best first
    top_logprobs: Optional[object]  # float32


_lib = None
_torch = _CODES = _raw_stream = _device = _int32 = _float32 = None


def load() -> ctypes.CDLL:
    """The library with these calls declared. Raises if it is not built."""
    global _lib, _torch, _CODES, _raw_stream, _device, _int32, _float32
    if _lib is None:
        import torch
        L = _wh.load()
        L.whead_logprobs.argtypes = [_vp]
        L.whead_logprobs.restype = ctypes.c_int
        L.whead_verify_workspace_bytes.argtypes = [_i64, _i32]
        L.whead_verify_workspace_bytes.restype = _i64
        L.whead_verify.argtypes = [_vp]
        L.whead_verify.restype = ctypes.c_int
        _torch, _int32, _float32 = torch, torch.int32, torch.float32
        _CODES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # a torch without CUDA has neither
        _device = getattr(torch._C, "_cuda_getDevice", None)
        _lib = L
    return _lib


def _logits(x, shape, strides, dims, index, what):
    """The code of a tensor of logits, checked."""
    code = _CODES.get(x.dtype)
    if code is None:
        raise TypeError(f"{what}: {x.dtype} is not supported")
    if _wh.asks_for_gradients(x):
        raise ValueError(f"{what}: no gradients are passed on; call it on detached tensors or, where none has a forward-mode tangent, under torch.no_grad()")
    if len(shape) not in dims or shape[-1] < 1 or strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{what}: {' or '.join(map(str, dims))} dimensions are wanted, the last one the vocabulary and contiguous")
    if not x.is_cuda or x.get_device() != index:
        raise ValueError(f"{what}: a tensor on one CUDA device with the others is wanted")
    return code


def _ints(x, shape, index, what):
    if x.dtype is not _int32 or x.shape != shape or not x.is_contiguous() or x.get_device() != index:
        raise ValueError(f"{what}: a contiguous int32 tensor of shape {tuple(shape)} on the logits' device is wanted")
    return x.data_ptr()


def _call(call, args, index):
    if _device() == index:
        rc = call(ctypes.addressof(args))
    else:
        with _torch.cuda.device(index):
            rc = call(ctypes.addressof(args))
    if rc:
        raise _wh.WheadError(rc, call.__name__)


def logprobs(logits, tokens=None, *, top=0, temperature=1.0) -> LogProbs:
    """Log probabilities of softmax(logits / temperature) for logits (n, V) or (n, t, V), bfloat16, float16 or float32, rows of any stride.

    tokens (int32, contiguous, the shape of the rows): the tokens whose log probabilities are asked for; one outside 0 .. V - 1 has -inf.
    top: how many of the best tokens to give (at most 32), equal logits in the tokens' order; -1 and -inf past the tokens that can be.
    Logits of -inf are tokens that cannot be. A row of nothing else has lse and log probabilities of -inf and entropy 0; a row with NaN or
    +inf gives NaN, and -1 for every alternative."""
    L = _lib or load()
    index, shape, strides = logits.get_device(), logits.shape, logits.stride()
    code = _logits(logits, shape, strides, (2, 3), index, "logits")
    if not 0 <= top <= MAX_TOP:
        raise ValueError(f"0 <= top <= {MAX_TOP} is wanted")
    device, empty, f32 = logits.device, _torch.empty, _float32
    if len(shape) == 2:
        n, V = shape
        t, stride_t, rows = 1, 0, (n,)
    else:
        n, t, V = shape
        stride_t, rows = strides[1], (n, t)
    # addresses first, tensors after: what is not asked for stays None
    logprob = top_tokens = top_logprobs = a0 = a1 = a2 = a3 = None
    if tokens is not None:
        a0 = _ints(tokens, rows, index, "tokens")
        logprob = empty(rows, dtype=f32, device=device)
        a1 = logprob.data_ptr()
    entropy = empty(rows, dtype=f32, device=device)
    lse = empty(rows, dtype=f32, device=device)
    if top:
        wide = (*rows, top)
        top_tokens = empty(wide, dtype=_int32, device=device)
        top_logprobs = empty(wide, dtype=f32, device=device)
        a2, a3 = top_tokens.data_ptr(), top_logprobs.data_ptr()
    _call(L.whead_logprobs, LogprobsArgs(logits.data_ptr(), a0, a1, entropy.data_ptr(), lse.data_ptr(), a2, a3, strides[0], stride_t, n, t, V,
                                         temperature, code, top, _raw_stream(index)), index)
    return LogProbs(logprob, entropy, lse, top_tokens, top_logprobs)


def verify(target, tokens, draft=None, *, temperature=0.0, draft_temperature=None, seed=0, step=0, drafted=None):
    """Which drafts stay, and the token after them: (said (n, gamma + 1), count (n,)), int32.

    target (n, gamma + 1, V): the target's logits, row t after the first t drafts; tokens (n, gamma) int32: the drafts; draft (n, gamma, V): the logits
    that the drafts were drawn from at draft_temperature (default: temperature), or None for drafts that were not drawn (greedy walks,
    tokens found in a text). Logits are bfloat16, float16 or float32, target and draft each of its own, rows of any stride. drafted (n,)
    int32: how many of its drafts an entry has (None: gamma).
    said[i, :count[i]] are the drafts that stay and the token after them, -1 the rest; count[i] is what KvCache.compact keeps of the last
    token and the drafts. temperature 0: drafts stay while they are the target's best token. Above: every token said is distributed as the
    target's own; seed and step number the draws, step .. step + gamma for all entries of a call, however far each has come: these only have to be
    fresh, and may be the walk's seed and t0.
    In a row of target with NaN, +inf or nothing but -inf no draft stays and the token after is -1."""
    L = _lib or load()
    index, shape, strides = target.get_device(), target.shape, target.stride()
    code = _logits(target, shape, strides, (3,), index, "target")
    n, rows, V = shape
    gamma = rows - 1
    if not 0 <= gamma <= MAX_DRAFTS:
        raise ValueError(f"target: (n, gamma + 1, V) with 0 <= gamma <= {MAX_DRAFTS} is wanted")
    token_ptr = _ints(tokens, (n, gamma), index, "tokens")
    drafted_ptr = None if drafted is None else _ints(drafted, (n,), index, "drafted")
    draft_ptr, draft_code, d0, d1 = None, 0, 0, 0
    if draft is not None:
        draft_strides = draft.stride()
        draft_code = _logits(draft, draft.shape, draft_strides, (3,), index, "draft")
        if draft.shape != (n, gamma, V):
            raise ValueError(f"draft: shape {(n, gamma, V)} is wanted")
        draft_ptr, (d0, d1, _) = draft.data_ptr(), draft_strides
    step, seed = int(step), int(seed)  # whole numbers of any type
    if not 0 <= step < 2 ** 32:
        raise ValueError("0 <= step < 2^32 is wanted")
    need = L.whead_verify_workspace_bytes(n, gamma)
    if need < 0:
        raise _wh.WheadError(need, "whead_verify_workspace_bytes")
    device, empty = target.device, _torch.empty
    said = empty((n, rows), dtype=_int32, device=device)
    count = empty((n,), dtype=_int32, device=device)
    workspace = empty((need,), dtype=_torch.uint8, device=device)
    _call(L.whead_verify, VerifyArgs(target.data_ptr(), draft_ptr, token_ptr, drafted_ptr, said.data_ptr(), count.data_ptr(), strides[0], strides[1],
                                     d0, d1, n, V, gamma, code, draft_code, step, temperature,
                                     temperature if draft_temperature is None else draft_temperature, seed & 0xFFFFFFFFFFFFFFFF,
                                     workspace.data_ptr(), need, _raw_stream(index)), index)
    return said, count
