"""Python binding of the verification of drafts (include/whead_verify.h): argument checks and marshalling only.

A walk drafts gamma tokens, the target gives logits after the last token and after each of them, and these calls say what they are worth:

    said, count = verify(logits, drafts, draft_logits, temperature=T, seed=seed)   # what stays, and the token after it
    cache.compact(start, keep, count)                                              # (kv.py) the others leave the cache
    r = logprobs(logits, said, top=5)                                              # log probabilities, entropy, alternatives

No gradients pass through them: inputs that ask for gradients are refused outside torch.no_grad(). Calls go to the current torch
stream. There is no fallback: without the built library, loading raises.
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
_CODES = None


def load() -> ctypes.CDLL:
    """The library with these calls declared. Raises if it is not built."""
    global _lib, _CODES
    if _lib is None:
        import torch
        L = _wh.load()
        L.whead_logprobs.argtypes = [_vp]
        L.whead_logprobs.restype = ctypes.c_int
        L.whead_verify_workspace_bytes.argtypes = [_i64, _i32]
        L.whead_verify_workspace_bytes.restype = _i64
        L.whead_verify.argtypes = [_vp]
        L.whead_verify.restype = ctypes.c_int
        _CODES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}
        _lib = L
    return _lib


def _logits(x, dims, what, device=None):
    """The code of a tensor of logits, checked."""
    import torch
    code = _CODES.get(x.dtype)
    if code is None:
        raise TypeError(f"{what}: {x.dtype} is not supported")
    if x.dim() not in dims or x.shape[-1] < 1 or x.stride(-1) != 1 and x.shape[-1] > 1:
        raise ValueError(f"{what}: {' or '.join(map(str, dims))} dimensions are wanted, the last one the vocabulary and contiguous")
    if not x.is_cuda or (device is not None and x.get_device() != device):
        raise ValueError(f"{what}: a tensor on one CUDA device with the others is wanted")
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what}: no gradients are passed on; call it under torch.no_grad() or on detached tensors")
    return code


def _ints(x, shape, device, what):
    import torch
    if x.dtype is not torch.int32 or x.shape != shape or not x.is_contiguous() or x.get_device() != device:
        raise ValueError(f"{what}: a contiguous int32 tensor of shape {tuple(shape)} on the logits' device is wanted")
    return x.data_ptr()


def _call(call, args, index):
    import torch
    args.stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        rc = call(ctypes.addressof(args))
    else:
        with torch.cuda.device(index):
            rc = call(ctypes.addressof(args))
    if rc:
        raise _wh.WheadError(rc, call.__name__)


def logprobs(logits, tokens=None, *, top=0, temperature=1.0) -> LogProbs:
    """Log probabilities of softmax(logits / temperature) for logits (n, V) or (n, t, V), bfloat16, float16 or float32, rows of any stride.

    tokens (int32, contiguous, the shape of the rows): the tokens whose log probabilities are asked for; one outside 0 .. V - 1 has -inf.
    top: how many of the best tokens to give (at most 32), equal logits in the tokens' order; -1 and -inf past the tokens that can be.
    Logits of -inf are tokens that cannot be. A row of nothing else has lse and log probabilities of -inf and entropy 0; a row with NaN or
    +inf gives NaN, and -1 for every alternative."""
    import torch
    L = load()
    code = _logits(logits, (2, 3), "logits")
    index, device = logits.get_device(), logits.device
    shape, strides = logits.shape, logits.stride()
    rows = shape[:-1]
    n, t = (shape[0], 1) if len(shape) == 2 else (shape[0], shape[1])
    top, temperature = int(top), float(temperature)
    if not 0 <= top <= MAX_TOP:
        raise ValueError(f"0 <= top <= {MAX_TOP} is wanted")
    entropy = torch.empty(rows, dtype=torch.float32, device=device)
    lse = torch.empty(rows, dtype=torch.float32, device=device)
    logprob = top_tokens = top_logprobs = token_ptr = None
    if tokens is not None:
        token_ptr = _ints(tokens, rows, index, "tokens")
        logprob = torch.empty(rows, dtype=torch.float32, device=device)
    if top:
        top_tokens = torch.empty((*rows, top), dtype=torch.int32, device=device)
        top_logprobs = torch.empty((*rows, top), dtype=torch.float32, device=device)
    a = LogprobsArgs(logits.data_ptr(), token_ptr, None if logprob is None else logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(),
                     top_tokens.data_ptr() if top else None, top_logprobs.data_ptr() if top else None, strides[0],
                     strides[1] if len(shape) == 3 else 0, n, t, shape[-1], temperature, code, top)
    _call(L.whead_logprobs, a, index)
    return LogProbs(logprob, entropy, lse, top_tokens, top_logprobs)


def verify(target, tokens, draft=None, *, temperature=0.0, draft_temperature=None, seed=0, step=0, drafted=None):
    """Which drafts stay, and the token after them: (said (n, gamma + 1), count (n,)), int32.

    target (n, gamma + 1, V): the target's logits, row t after the first t drafts; tokens (n, gamma) int32: the drafts; draft (n, gamma, V): the logits
    that the drafts were drawn from at draft_temperature (default: temperature), or None for drafts that were not drawn (greedy walks,
    tokens found in a text). Logits are bfloat16, float16 or float32, target and draft each of its own, rows of any stride. drafted (n,)
    int32: how many of its drafts an entry has (None: gamma).
    said[i, :count[i]] are the drafts that stay and the token after them, -1 the rest; count[i] is what KvCache.compact keeps of the last
    token and the drafts. temperature 0: drafts stay while they are the target's best token. Above: every token said is distributed as the
    target's own; seed and step (the walk's t0) number the draws as they do the walk's, and may be the walk's.
    In a row of target with NaN, +inf or nothing but -inf no draft stays and the token after is -1."""
    import torch
    L = load()
    code = _logits(target, (3,), "target")
    index, device = target.get_device(), target.device
    n, rows, V = target.shape
    gamma = rows - 1
    if not 0 <= gamma <= MAX_DRAFTS:
        raise ValueError(f"target: (n, gamma + 1, V) with 0 <= gamma <= {MAX_DRAFTS} is wanted")
    token_ptr = _ints(tokens, (n, gamma), index, "tokens")
    drafted_ptr = None if drafted is None else _ints(drafted, (n,), index, "drafted")
    temperature, step, seed = float(temperature), int(step), int(seed)
    draft_ptr, draft_code, d0, d1 = None, 0, 0, 0
    if draft is not None:
        draft_code = _logits(draft, (3,), "draft", index)
        if draft.shape != (n, gamma, V):
            raise ValueError(f"draft: shape {(n, gamma, V)} is wanted")
        draft_ptr, (d0, d1, _) = draft.data_ptr(), draft.stride()
    if not 0 <= step < 2 ** 32:
        raise ValueError("0 <= step < 2^32 is wanted")
    need = L.whead_verify_workspace_bytes(n, gamma)
    if need < 0:
        raise _wh.WheadError(need, "whead_verify_workspace_bytes")
    said = torch.empty((n, rows), dtype=torch.int32, device=device)
    count = torch.empty(n, dtype=torch.int32, device=device)
    workspace = torch.empty(need, dtype=torch.uint8, device=device)
    s0, s1, _ = target.stride()
    a = VerifyArgs(target.data_ptr(), draft_ptr, token_ptr, drafted_ptr, said.data_ptr(), count.data_ptr(), s0, s1, d0, d1, n, V, gamma, code,
                   draft_code, step, temperature, temperature if draft_temperature is None else float(draft_temperature), seed & (2 ** 64 - 1),
                   workspace.data_ptr(), need)
    _call(L.whead_verify, a, index)
    return said, count
