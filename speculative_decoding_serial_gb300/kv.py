"""Python binding of the 4-bit paged KV cache (include/whead_kv.h): argument checks and marshalling only.

A serial draft head returns gamma tokens a walk; this cache holds the target's keys and values that verify them:

    cache = KvCache(num_pages, page_size, kv_heads, head_dim, max_seqs, max_pages)
    cache.append(k, v)                      # the last token and the drafts, quantized into pages
    out, lse = cache.attend(q)              # their attention over everything that is cached
    cache.compact(start, keep, count)       # what was accepted stays
    cache.fork(parents)                     # candidates take over one another's sequences

No gradients pass through the cache: inputs that ask for them are refused outside torch.no_grad(), inputs with forward-mode tangents everywhere.
Calls go to the current torch stream. They share the cache's workspace: calls on other streams have to be ordered
after them by events. There is no fallback: without the built library, loading raises.
"""
from __future__ import annotations

import ctypes
import math

from . import whead as _wh

BF16, F16, F32 = 0, 1, 2
MAX_BLOCK = 256
INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1

# Every symbol include/whead_kv.h declares.
EXPORTS = ("whead_kv_page_bytes", "whead_kv_workspace_bytes", "whead_kv_append", "whead_kv_read", "whead_kv_attend",
           "whead_kv_compact", "whead_kv_fork", "whead_kv_status")

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class KvParams(ctypes.Structure):
    _fields_ = [("page_size", _i32), ("kv_heads", _i32), ("head_dim", _i32), ("max_seqs", _i32), ("max_pages", _i32),
                ("num_pages", _i32), ("pool", _vp), ("lens", _vp), ("refs", _vp), ("tables", _vp), ("k_scale", _vp),
                ("v_scale", _vp), ("workspace", _vp), ("workspace_bytes", _i64), ("stream", _vp)]


class KvAttendArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("out", _vp), ("lse", _vp), ("indptr", _vp), ("slots", _vp), ("tree", _vp), ("total", _i64),
                ("q_token_stride", _i64), ("q_head_stride", _i64), ("n", _i32), ("heads", _i32), ("max_q", _i32),
                ("dtype", _i32), ("causal", _i32), ("window", _i32), ("tree_words", _i32), ("scale", ctypes.c_float), ("sinks", _i32)]


_lib = None


def load() -> ctypes.CDLL:
    """The library with the cache's calls declared. Raises if it is not built."""
    global _lib
    if _lib is None:
        L = _wh.load()
        L.whead_kv_page_bytes.argtypes = [_i32, _i32, _i32]
        L.whead_kv_page_bytes.restype = _i64
        L.whead_kv_workspace_bytes.argtypes = [_vp]
        L.whead_kv_workspace_bytes.restype = _i64
        L.whead_kv_append.argtypes = [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _vp, _vp, _i32, _i64]
        L.whead_kv_read.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp]
        L.whead_kv_attend.argtypes = [_vp, _vp]
        L.whead_kv_compact.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32]
        L.whead_kv_fork.argtypes = [_vp, _vp]
        L.whead_kv_status.argtypes = [_vp]
        for name in EXPORTS[2:]:
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def page_bytes(page_size: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of one page of the pool (no device needed)."""
    n = int(load().whead_kv_page_bytes(int(page_size), int(kv_heads), int(head_dim)))
    if n < 0:
        raise _wh.WheadError(n, "whead_kv_page_bytes")
    return n


_CODES = None


def _code(dtype, what, f32=True):
    global _CODES
    if _CODES is None:
        import torch
        _CODES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}
    code = _CODES.get(dtype)
    if code is None or (code == F32 and not f32):
        raise TypeError(f"{what}: {dtype} is not supported")
    return code


class KvCache:
    """A paged KV cache held in 4 bits: e2m1 codes, an e4m3 scale for 16 channels of a token, an fp32 scale a KV head.

    num_pages pages of page_size (16, 32, 64 or 128) tokens, kv_heads heads of head_dim (64, 128 or 256); max_seqs slots
    of at most max_pages pages. k_scale, v_scale: (kv_heads,) float32, the heads' fixed scales (default 1 / 64, which puts
    blocks whose largest value lies between 0.01 and 40 into e4m3's normal range). pool (uint8, (num_pages, kv_heads,
    page_size / 16, 18 * head_dim)) and state (int32, max_seqs + num_pages + max_seqs * max_pages: lens, refs, tables)
    may be the caller's; what is not given is made here, empty. `state.copy_()` of a kept copy takes the cache back to it
    as long as the pages it names have not been written since.
    """

    def __init__(self, num_pages, page_size, kv_heads, head_dim, max_seqs, max_pages, *, k_scale=None, v_scale=None,
                 pool=None, state=None, device="cuda"):
        import torch
        self._torch = torch
        L = load()
        self._lib = L
        num_pages, page_size, kv_heads, head_dim, max_seqs, max_pages = (
            int(x) for x in (num_pages, page_size, kv_heads, head_dim, max_seqs, max_pages))
        each = page_bytes(page_size, kv_heads, head_dim)
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = num_pages, page_size, kv_heads, head_dim
        self.max_seqs, self.max_pages = max_seqs, max_pages
        if pool is not None:
            device = pool.device
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("the cache lives on a CUDA device")
        shape = (num_pages, kv_heads, page_size // 16, 18 * head_dim)
        if pool is None:
            pool = torch.zeros(shape, dtype=torch.uint8, device=self.device)
        if pool.dtype != torch.uint8 or tuple(pool.shape) != shape or not pool.is_contiguous():
            raise ValueError(f"pool: a contiguous uint8 tensor of shape {shape} is wanted")
        words = max_seqs + num_pages + max_seqs * max_pages
        if state is None:
            state = torch.zeros(words, dtype=torch.int32, device=self.device)
            state[max_seqs + num_pages:] = -1
        if state.dtype != torch.int32 or tuple(state.shape) != (words,) or not state.is_contiguous():
            raise ValueError(f"state: a contiguous int32 tensor of {words} words is wanted")
        scales = []
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            s = torch.full((kv_heads,), 1.0 / 64, dtype=torch.float32, device=self.device) if s is None else s
            if s.dtype != torch.float32 or tuple(s.shape) != (kv_heads,) or not s.is_contiguous():
                raise ValueError(f"{name}: a contiguous float32 tensor of {kv_heads} values is wanted")
            scales.append(s)
        self.pool, self.state, (self.k_scale, self.v_scale) = pool, state, scales
        self.lens = state[:max_seqs]
        self.refs = state[max_seqs:max_seqs + num_pages]
        self.tables = state[max_seqs + num_pages:].view(max_seqs, max_pages)
        for t in (pool, state, *scales):
            if t.device != pool.device or not t.is_cuda:
                raise ValueError("pool, state and scales have to be on one CUDA device")
        self.device = pool.device
        p = KvParams(page_size=page_size, kv_heads=kv_heads, head_dim=head_dim, max_seqs=max_seqs, max_pages=max_pages,
                     num_pages=num_pages, pool=pool.data_ptr(), lens=self.lens.data_ptr(), refs=self.refs.data_ptr(),
                     tables=self.tables.data_ptr(), k_scale=scales[0].data_ptr(), v_scale=scales[1].data_ptr())
        self._p, self._ref = p, ctypes.addressof(p)
        with torch.cuda.device(self.device):
            n = int(L.whead_kv_workspace_bytes(self._ref))
        if n < 0:
            raise _wh.WheadError(n, "whead_kv_workspace_bytes")
        # the control words and counters at the workspace's head start at zero; the rest is written before it is read
        self._workspace = torch.empty(n, dtype=torch.uint8, device=self.device)
        self._workspace[:16384].zero_()
        p.workspace, p.workspace_bytes = self._workspace.data_ptr(), n
        assert self.device.index is not None
        self._index = self.device.index
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._device = torch._C._cuda_getDevice
        self._int32 = torch.int32
        self._scale = 1.0 / math.sqrt(head_dim)

    def _call(self, call, *args):
        self._p.stream = self._raw_stream(self._index)
        if self._device() == self._index:
            rc = call(self._ref, *args)
        else:
            with self._torch.cuda.device(self._index):
                rc = call(self._ref, *args)
        if rc:
            raise _wh.WheadError(rc, call.__name__)

    def _ints(self, x, shape, what):
        """The pointer of an int32 tensor of this shape on the cache's device, or None."""
        if x is None:
            return None
        if x.dtype is not self._int32 or x.shape != shape or not x.is_contiguous() or x.get_device() != self._index:
            raise ValueError(f"{what}: a contiguous int32 tensor of shape {shape} on {self.device} is wanted")
        return x.data_ptr()

    @staticmethod
    def _no_grad(what, *tensors):
        if _wh.asks_for_gradients(*tensors):
            raise ValueError(f"{what}: the cache passes no gradients on; call it on detached tensors or, where none has a forward-mode tangent, under torch.no_grad()")

    def _entries(self, indptr, slots):
        """How many entries a call has, and the pointers of its offsets and slots."""
        n = slots.shape[0] if slots is not None else indptr.shape[0] - 1 if indptr is not None else self.max_seqs
        if n < 0 or n > self.max_seqs:
            raise ValueError(f"{n} entries: the cache has {self.max_seqs} slots")
        return n, self._ints(indptr, (n + 1,), "indptr"), self._ints(slots, (n,), "slots")

    def append(self, k, v, indptr=None, slots=None):
        """Appends tokens: k, v (total, kv_heads, head_dim) in bfloat16, float16 or float32, channels contiguous. Entry i's
        are rows indptr[i] .. indptr[i + 1] - 1 (None: an equal share each) and go to slot slots[i] (None: slot i)."""
        n, ip, sl = self._entries(indptr, slots)
        shape = k.shape
        if shape != v.shape or len(shape) != 3 or shape[1] != self.kv_heads or shape[2] != self.head_dim:
            raise ValueError(f"k and v: shape (total, {self.kv_heads}, {self.head_dim}) is wanted")
        if k.dtype is not v.dtype or k.get_device() != self._index or v.get_device() != self._index:
            raise ValueError("k and v: one type, on the cache's device")
        ks, vs = k.stride(), v.stride()
        if ks[2] != 1 or vs[2] != 1:
            raise ValueError("k and v: channels have to be contiguous")
        self._no_grad("k and v", k, v)
        self._call(self._lib.whead_kv_append, k.data_ptr(), v.data_ptr(), _code(k.dtype, "k and v"), ks[0], ks[1], vs[0], vs[1], ip, sl,
                   n, shape[0])

    def read(self, start, count, slots=None, *, dtype=None):
        """The held values of `count` tokens from positions start (int32, one an entry): k, v of (n, count, kv_heads,
        head_dim) in dtype (default bfloat16); zeros past a slot's length."""
        torch = self._torch
        n, _, sl = self._entries(None, slots)
        if slots is None and start.shape[0] != n:
            raise ValueError(f"start: {n} values are wanted")
        dtype = torch.bfloat16 if dtype is None else dtype
        code, count = _code(dtype, "read"), int(count)
        if not 0 <= count <= INT_MAX:
            raise ValueError("read: 0 <= count < 2^31 is wanted")
        shape = (n, count, self.kv_heads, self.head_dim)
        k = torch.empty(shape, dtype=dtype, device=self.device)
        v = torch.empty(shape, dtype=dtype, device=self.device)
        self._call(self._lib.whead_kv_read, self._ints(start, (n,), "start"), sl, n, count, code, k.data_ptr(), v.data_ptr())
        return k, v

    def attend(self, q, indptr=None, slots=None, *, scale=None, causal=True, window=0, sinks=0, tree=None, max_q=None, out=None,
               lse=None):
        """Attention of q (total, heads, head_dim), bfloat16 or float16, over the slots' keys and values: (out, lse).

        Entry i's query tokens are rows indptr[i] .. indptr[i + 1] - 1 (None: an equal share each); they are its slot's
        last tokens, so append them first. A token sees its slot's keys, with causal those up to itself, with a window the
        latest `window` of these and of the slot's first `sinks` (streams that a model has to see the beginning of). tree (int64, (total,) or (total, words)): for each token, the bits of the entry's own
        tokens that it sees, besides everything before them. scale defaults to head_dim ** -0.5. With indptr, max_q says
        how many query tokens an entry has at most (default: total, or as many as tree has bits for); one that has more is
        reported by status() and its rows are not written. A token that sees nothing gets zeros and -inf. out (as q,
        contiguous) and lse (total, heads) float32 may be given."""
        torch = self._torch
        n, ip, sl = self._entries(indptr, slots)
        shape, strides = q.shape, q.stride()
        if len(shape) != 3 or shape[2] != self.head_dim or strides[2] != 1 or q.get_device() != self._index:
            raise ValueError(f"q: shape (total, heads, {self.head_dim}) with contiguous channels on the cache's device is wanted")
        self._no_grad("q", q)
        total, heads = shape[0], shape[1]
        dtype = q.dtype
        code = _code(dtype, "attend", f32=False)
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=self.device)
        elif out.shape != shape or out.dtype is not dtype or not out.is_contiguous() or out.get_device() != self._index:
            raise ValueError("out: a contiguous tensor like q is wanted")
        if lse is None:
            lse = torch.empty((total, heads), dtype=torch.float32, device=self.device)
        elif lse.shape != (total, heads) or lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.get_device() != self._index:
            raise ValueError("lse: a contiguous float32 tensor (total, heads) is wanted")
        words, bits = 0, None
        if tree is not None:
            if tree.dtype is not torch.int64 or tree.dim() not in (1, 2) or tree.shape[0] != total or not tree.is_contiguous() \
                    or tree.get_device() != self._index:
                raise ValueError("tree: a contiguous int64 tensor (total,) or (total, words) is wanted")
            words, bits = 1 if tree.dim() == 1 else tree.shape[1], tree.data_ptr()
        if max_q is None:
            max_q = total // max(n, 1) if indptr is None else min(total, 64 * words) if words else total
        if not (INT_MIN <= window <= INT_MAX and INT_MIN <= max_q <= INT_MAX and INT_MIN <= sinks <= INT_MAX) or (sinks < 0 and not window):
            # ctypes would wrap them; the library refuses what is negative, but looks at sinks with a window alone
            raise ValueError("0 <= window, max_q, sinks < 2^31 is wanted")
        a = KvAttendArgs(q.data_ptr(), out.data_ptr(), lse.data_ptr(), ip, sl, bits, total, strides[0], strides[1], n, heads, max_q, code,
                         bool(causal), window, words, self._scale if scale is None else scale, sinks)
        self._call(self._lib.whead_kv_attend, ctypes.addressof(a))
        return out, lse

    def compact(self, start, keep=None, count=None, slots=None):
        """Of each entry's tokens from start (int32) on, those at start + keep[i, j], j < count[i], move to start + j and the
        slot ends after them. keep (n, width) int32, ascending offsets below MAX_BLOCK; without keep the slots are
        cut at start."""
        n, _, sl = self._entries(None, slots)
        if (keep is None) != (count is None):
            raise ValueError("keep and count go together")
        width = 0
        if keep is not None:
            if keep.dim() != 2 or keep.shape[1] > MAX_BLOCK:
                raise ValueError(f"keep: (n, width) with width <= {MAX_BLOCK} is wanted")
            width = keep.shape[1]
        self._call(self._lib.whead_kv_compact, self._ints(start, (n,), "start"), self._ints(keep, (n, width), "keep"),
                   self._ints(count, (n,), "count"), sl, n, width)

    def fork(self, parents):
        """Slot i takes over what slot parents[i] (int32, max_seqs) held: i leaves it alone, -1 empties it."""
        self._call(self._lib.whead_kv_fork, self._ints(parents, (self.max_seqs,), "parents"))

    def free(self, slots):
        """Empties the given slots (int32)."""
        self.compact(self._torch.zeros_like(slots), slots=slots)

    def status(self, check=False) -> int:
        """Waits for the current stream and returns the first device-side error since the last call (0: none)."""
        self._p.stream = self._raw_stream(self._index)
        with self._torch.cuda.device(self._index):
            code = int(self._lib.whead_kv_status(self._ref))
        if check and code:
            raise _wh.WheadError(code, "whead_kv_status")
        return code
