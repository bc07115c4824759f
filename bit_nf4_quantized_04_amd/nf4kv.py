"""Binding of libnf4kv.so (csrc/kv/nf4kv.h): a paged key/value cache held in 4
bits, the attention that reads it, rotary positions and the bookkeeping of its
pages.

Names follow the C ABI.  Checks of shapes, types and devices, output and
workspace allocation and the call on the current stream are made by the module
_nf4kv (csrc/kv/bind), because a decode step makes a handful of these calls
between kernels of a few microseconds; the C functions themselves are also here
through ctypes (_lib).  With a `stream` the call is made, and what it allocates
is allocated, as under torch.cuda.stream(stream).  Importing this module raises
ImportError when the libraries have not been built.
"""

from __future__ import annotations

import ctypes as C
import os
from typing import NamedTuple

import torch

from .nf4qlora import NF4_ELAUNCH, NF4_OK, NF4Error, nf4_strerror

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnf4kv.so")
if not os.path.exists(LIB_PATH) or not os.path.exists(os.path.join(_HERE, "_nf4kv.so")):
    raise ImportError("libnf4kv.so is not built; run `python -m bit_nf4_quantized_04_amd.build`")
_lib = C.CDLL(LIB_PATH)
from . import _nf4kv  # noqa: E402

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {None: 0, "none": 0, "linear": 1, "base": 2, "parts": 3}
PAGE_SIZES = (16, 32, 64, 128, 256)
HEAD_DIMS = (64, 128, 256)


class nf4_kv_cache(C.Structure):
    _fields_ = [("k_codes", C.c_void_p), ("k_scales", C.c_void_p), ("v_codes", C.c_void_p), ("v_scales", C.c_void_p),
                ("n_pages", C.c_int64), ("n_heads", C.c_int32), ("head_dim", C.c_int32), ("page_size", C.c_int32),
                ("quant_type", C.c_int32)]


class nf4_rope_scaling(C.Structure):
    _fields_ = [("kind", C.c_int32), ("factor", C.c_float), ("low", C.c_float), ("high", C.c_float),
                ("original", C.c_float), ("amplitude", C.c_float)]


_P, _I64, _I32 = C.c_void_p, C.c_int64, C.c_int32
_ROPE = [_P, _I64, _I64, _P, _I64, _I64, _I64, _I32, _I32, _I32, _P, _P, _I64, _I32, _I32, _P]
_ATTENTION = [_P, _P, _I64, _I64, _I32, _P, _P, _P, _I32, _I32, _I32, _I32, C.c_float, _I32, _I32, _P, _I64, _P,
              C.c_size_t, _P]
_SIGS = {
    "nf4_kv_last_hip_error": (C.c_int, []),
    "nf4_rope_table": (C.c_int, [_P, _I64, _I32, C.c_float, C.POINTER(nf4_rope_scaling), _P]),
    "nf4_rope_forward": (C.c_int, _ROPE),
    "nf4_rope_backward": (C.c_int, _ROPE),
    "nf4_kv_plan": (C.c_int, [_P, _P, _P, _I32, _P, _I32, _I32, _P, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "nf4_kv_append": (C.c_int, [_P, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I32,
                                _P, _P, _I64, _I32, _I32, _P]),
    "nf4_kv_read": (C.c_int, [_P, _P, _I64, _P, _P, _P]),
    "nf4_kv_attention_ws_bytes": (C.c_size_t, [_I32] * 8),
    "nf4_kv_attention": (C.c_int, _ATTENTION),
    "nf4_kv_attention_padded": (C.c_int, _ATTENTION),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTS = tuple(_SIGS)


class NF4KVError(NF4Error):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = nf4_strerror(code)
        if code == NF4_ELAUNCH:
            msg = "HIP kernel launch failed (hipError %d)" % _lib.nf4_kv_last_hip_error()
        RuntimeError.__init__(self, "%s: %s" % (where, msg))


_nf4kv.set_error(NF4KVError)


def _check(rc: int, where: str) -> None:
    if rc != NF4_OK:
        raise NF4KVError(rc, where)


def _on(stream, call, *args):
    """The call on the given stream.  (Outputs and workspaces come from that
    stream's part of torch's allocator: memory of the current stream, given back
    when the call returns, could go to other work while the kernels run.)"""
    if stream is None:
        return call(*args)
    with torch.cuda.stream(stream):
        return call(*args)


# ------------------------------------------------------------ rotary positions
def nf4_rope_table(max_pos: int, rot: int, base: float = 10000.0, scaling=None, factor: float = 1.0, low: float = 1.0,
                   high: float = 4.0, original: float = 8192.0, amplitude: float = 1.0, device="cuda", stream=None):
    """fp32 [max_pos, rot]: the cosines, then the sines, of every position's
    rot/2 angles.  scaling: None, "linear", "base" or "parts" (csrc/kv/nf4kv.h)."""
    s = nf4_rope_scaling(ROPE_SCALINGS[scaling], factor, low, high, original, amplitude)

    def make():
        t = torch.empty((max_pos, rot), dtype=torch.float32, device=device)
        if not t.is_cuda or t.device.index != torch.cuda.current_device():
            raise ValueError("device: the current GPU")
        _check(_lib.nf4_rope_table(t.data_ptr(), max_pos, rot, float(base), C.byref(s),
                                   torch.cuda.current_stream().cuda_stream), "nf4_rope_table")
        return t

    return _on(stream, make)


def nf4_rope_forward(x, positions, table, layout: str = "half", out=None, stream=None):
    """x bf16 or fp32 [tokens, heads, head_dim] (any token and head strides: a
    slice of a fused projection will do, or [heads, tokens, head_dim] transposed)
    with its first table.shape[1] elements rotated to int32 `positions`.  out,
    with strides of its own, may be x."""
    return _on(stream, _nf4kv.rope, x, positions, table, ROPE_LAYOUTS[layout], out, False)


def nf4_rope_backward(dy, positions, table, layout: str = "half", out=None, stream=None):
    """The gradient of nf4_rope_forward's input for its output's gradient dy."""
    return _on(stream, _nf4kv.rope, dy, positions, table, ROPE_LAYOUTS[layout], out, True)


# -------------------------------------------------------------------- the cache
class NF4KVCache:
    """Device buffers of a paged 4-bit cache (torch tensors): codes uint8
    [n_pages, n_heads, page_size, head_dim/2], absmax bf16 [..., head_dim/64];
    quant_type "nf4" or "fp4".  Every call reads and checks them anew."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, quant_type: str = "nf4"):
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.quant_type = quant_type
        _nf4kv.cache(self)  # (ValueError for parts that do not fit)

    def c_struct(self) -> nf4_kv_cache:
        """For the C functions: the addresses hold until a part is replaced."""
        return nf4_kv_cache.from_buffer_copy(_nf4kv.cache(self))

    n_pages = property(lambda self: self.k_codes.shape[0])
    n_heads = property(lambda self: self.k_codes.shape[1])
    page_size = property(lambda self: self.k_codes.shape[2])
    head_dim = property(lambda self: 2 * self.k_codes.shape[3])

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k_codes, self.k_scales, self.v_codes, self.v_scales))


def nf4_kv_cache_alloc(n_pages: int, n_heads: int, head_dim: int, page_size: int = 32, quant_type: str = "nf4",
                       device="cuda") -> NF4KVCache:
    """An empty cache (every entry zero)."""
    if head_dim not in HEAD_DIMS or page_size not in PAGE_SIZES:
        raise ValueError("head_dim: 64, 128 or 256; page_size: 16 to 256, a power of 2")
    zero = 0x77 if quant_type == "nf4" else 0
    codes = [torch.full((n_pages, n_heads, page_size, head_dim // 2), zero, dtype=torch.uint8, device=device)
             for _ in range(2)]
    scales = [torch.zeros((n_pages, n_heads, page_size, head_dim // 64), dtype=torch.bfloat16, device=device)
              for _ in range(2)]
    return NF4KVCache(codes[0], scales[0], codes[1], scales[1], quant_type)


class NF4KVPlan(NamedTuple):
    """One step's bookkeeping: what nf4_kv_plan returns (device tensors)."""

    kv_lens: object    # int32 [batch]: lengths with the step's tokens
    cu_new: object     # int32 [batch + 1]: each request's first new token
    slots: object      # int64 [max_tokens]: where each token goes, -1 past the last
    positions: object  # int32 [max_tokens]
    free_state: object  # int32 [2]: {head, count} of the ring of free pages
    refused: object    # int32 [1]


def nf4_kv_plan(kv_lens, new_lens, block_table, free_pages, free_state, page_size: int, max_tokens: int, done=None,
                stream=None) -> NF4KVPlan:
    """Extend int32 block_table [batch, width] (in place) by the pages that
    kv_lens + new_lens need, taken from the ring free_pages whose {head, count}
    is free_state; requests with done != 0 end and give theirs back (to the
    ring, in place).  Requests that do not fit are refused and keep their length;
    the step's tokens are those of the others (cu_new, not new_lens, says where
    each one's are).  No host synchronization; the next step passes the returned
    kv_lens and free_state."""
    return NF4KVPlan(*_on(stream, _nf4kv.plan, kv_lens, new_lens, block_table, free_pages, free_state, page_size,
                          max_tokens, done))


def nf4_kv_append(cache: NF4KVCache, k, v, slots, positions=None, table=None, q=None, layout: str = "half",
                  q_out=None, stream=None):
    """Quantize bf16 k, v [tokens, heads, head_dim] (any token stride) into the
    cache's int64 `slots`, k rotated to `positions` by the rope `table` first
    (None: not rotated).  Returns q [tokens, q_heads, head_dim] rotated, when given."""
    return _on(stream, _nf4kv.append, cache, k, v, slots, positions, table, q, ROPE_LAYOUTS[layout], q_out)


def nf4_kv_read(cache: NF4KVCache, slots, stream=None):
    """The stored keys and values of int64 `slots`, bf16 [tokens, heads,
    head_dim] each (zeros for a slot outside the cache)."""
    return _on(stream, _nf4kv.read, cache, slots)


def nf4_kv_attention_ws_bytes(cache: NF4KVCache, batch: int, q_heads: int, max_q: int, max_len: int, window: int = 0,
                              sinks: int = 0) -> int:
    return int(_lib.nf4_kv_attention_ws_bytes(batch, q_heads, cache.n_heads, cache.head_dim, max_q, max_len, window,
                                              sinks))


def nf4_kv_attention(cache: NF4KVCache, q, cu_q, kv_lens, block_table, max_q: int, max_len=None, scale=None,
                     window: int = 0, sinks: int = 0, out=None, ws=None, stream=None):
    """Causal attention of bf16 q [total_q, q_heads, head_dim] over the cache.
    Request i's queries, rows cu_q[i] to cu_q[i+1], are the last of its
    kv_lens[i] cached tokens, found through int32 block_table [batch, width].
    window > 0: only the last `window` tokens and the first `sinks` are seen.
    max_q and max_len bound every request's queries and length (max_len: by
    default what the table can hold; a tight bound is faster).  scale: 1/sqrt(head_dim) by default.
    Rows that no request has, and queries past max_q, are zeros; in a given out
    they stay as they are."""
    return _on(stream, _nf4kv.attention, cache, q, cu_q, kv_lens, block_table, max_q, max_len, scale, window,
               sinks, out, ws)
