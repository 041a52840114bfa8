"""ctypes binding of libloong_attn.so: argument marshalling only.

Every function named ``loong_*`` calls the C entry point of the same name in
``include/loong_attn.h``; tensors are passed as raw device pointers and every
step of the computation runs in the library's kernels.  The library is loaded
on first use; a missing library raises ``RuntimeError`` (there is no other
implementation to fall back to).
"""
import contextlib
import ctypes
import functools
import math
import os
import sys

import torch

from .inputs import Workload

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libloong_attn.so")
# the same library with device address checks (LOONG_CHECKED)
CHECKED_LIB_PATH = os.path.join(_PKG, "libloong_attn_checked.so")

LOONG_OK = 0
LOONG_ERR_INVALID_ARG = -1
LOONG_ERR_WORKSPACE = -2
LOONG_ERR_UNSUPPORTED = -3
LOONG_ERR_CUDA = -4
LOONG_ERR_DEVICE_TIMEOUT = -5
LOONG_ERR_DEVICE_CHECK = -6
PLACEMENT_CONTIGUOUS, PLACEMENT_ZIGZAG = 0, 1
MODE_STEPWISE, MODE_FUSED, MODE_STEPWISE_COPY, MODE_STEPWISE_COPY_AB = 0, 1, 2, 3
LAYOUT_NATURAL, LAYOUT_RANK_MAJOR = 0, 1

EXPORTS = ("loong_version", "loong_status_string", "loong_last_cuda_error", "loong_attn_check",
           "loong_attn_workspace_size", "loong_ring_schedule", "loong_attn_fwd", "loong_attn_fwd_ranks",
           "loong_attn_bwd",
           "loong_attn_bwd_noalloc", "loong_lse_merge", "loong_headctx_pack", "loong_headctx_pack_n",
           "loong_rel_bias_check", "loong_attn_bias_workspace_size", "loong_attn_bias_fwd", "loong_attn_bias_bwd",
           "loong_qk_norm_rope_fwd", "loong_qk_norm_rope_bwd_workspace_size", "loong_qk_norm_rope_bwd",
           "loong_attn_2d_host_workspace_size", "loong_attn_2d_host", "loong_host_alloc", "loong_host_free",
           "loong_set_timing_events", "loong_get_device_status", "loong_selftest_wait_timeout")
NOALLOC_SCRATCH_BYTES = 32 << 20   # LOONG_NOALLOC_SCRATCH_BYTES


class LoongAttnDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("hp", ctypes.c_int32), ("cp", ctypes.c_int32),
                ("ring_inner", ctypes.c_int32), ("ring_outer", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("placement", ctypes.c_int32), ("mode", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("layout", ctypes.c_int32)]


class LoongRelBias(ctypes.Structure):
    _fields_ = [("num_buckets", ctypes.c_int32), ("num_bounds", ctypes.c_int32),
                ("bounds", ctypes.POINTER(ctypes.c_int32)), ("bucket_of", ctypes.POINTER(ctypes.c_int32)),
                ("table", ctypes.c_void_p)]


class LoongQkOpts(ctypes.Structure):
    _fields_ = [("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("dq_stride", ctypes.c_int64), ("dk_stride", ctypes.c_int64), ("dv_stride", ctypes.c_int64),
                ("pos_begin", ctypes.c_int64), ("rot_base", ctypes.c_double),
                ("inv_freq", ctypes.POINTER(ctypes.c_double)),
                ("eps", ctypes.c_float), ("w_offset", ctypes.c_float), ("rot_scale", ctypes.c_float),
                ("norm", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class LoongError(RuntimeError):
    def __init__(self, fn, status, lib):
        msg = lib.loong_status_string(status).decode()
        if status == LOONG_ERR_CUDA:
            msg += " (" + lib.loong_last_cuda_error().decode() + ")"
        super().__init__(f"{fn} failed: {status} {msg}")
        self.status = status


_lib = None


def lib():
    """Load the library once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m head_context_attention_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        D = ctypes.POINTER(LoongAttnDesc)
        L.loong_version.restype = ctypes.c_int
        L.loong_status_string.restype = ctypes.c_char_p
        L.loong_status_string.argtypes = [ctypes.c_int]
        L.loong_last_cuda_error.restype = ctypes.c_char_p
        L.loong_attn_check.argtypes = [D]
        L.loong_attn_workspace_size.restype = SZ
        L.loong_attn_workspace_size.argtypes = [D, ctypes.c_int]
        L.loong_ring_schedule.argtypes = [I32, I32, ctypes.POINTER(ctypes.c_int32)]
        L.loong_attn_fwd.argtypes = [D, P, P, P, P, P, P, P, SZ, P]
        L.loong_attn_fwd_ranks.argtypes = [D, I32, I32, P, P, P, P, P, P, SZ, P]
        L.loong_attn_bwd.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.loong_attn_bwd_noalloc.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P]
        L.loong_lse_merge.argtypes = [I64, I32, I32, P, P, P, P, ctypes.c_int, P]
        L.loong_headctx_pack.argtypes = [I64, I32, I32, I64, I32, I32, ctypes.c_int, ctypes.c_int,
                                         P, P, P]
        L.loong_headctx_pack_n.argtypes = [I32, I64, I32, I32, I64, ctypes.POINTER(ctypes.c_int32), I32,
                                           ctypes.c_int, ctypes.c_int, ctypes.POINTER(P), ctypes.POINTER(P), P]
        RB, QO = ctypes.POINTER(LoongRelBias), ctypes.POINTER(LoongQkOpts)
        L.loong_rel_bias_check.argtypes = [D, RB]
        L.loong_attn_bias_workspace_size.restype = SZ
        L.loong_attn_bias_workspace_size.argtypes = [D, RB, ctypes.c_int]
        L.loong_attn_bias_fwd.argtypes = [D, RB, P, P, P, P, P, P, P, SZ, P]
        L.loong_attn_bias_bwd.argtypes = [D, RB, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.loong_qk_norm_rope_fwd.argtypes = [D, QO, P, P, P, P, P, P, P, P, P, P]
        L.loong_qk_norm_rope_bwd_workspace_size.restype = SZ
        L.loong_qk_norm_rope_bwd_workspace_size.argtypes = [D, QO]
        L.loong_qk_norm_rope_bwd.argtypes = [D, QO, P, P, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.loong_attn_2d_host_workspace_size.restype = SZ
        L.loong_attn_2d_host_workspace_size.argtypes = [D, ctypes.c_int]
        L.loong_attn_2d_host.argtypes = [D, I32, P, P, P, P, P, P, P, P, P, P, SZ, P, P]
        L.loong_host_alloc.argtypes = [SZ, ctypes.POINTER(ctypes.c_void_p)]
        L.loong_host_free.argtypes = [P]
        L.loong_set_timing_events.argtypes = [P, P]
        L.loong_get_device_status.argtypes = [P]
        L.loong_selftest_wait_timeout.argtypes = [ctypes.c_uint32, P]
        _lib = L
    return _lib


def _check(fn, status):
    if status != LOONG_OK:
        raise LoongError(fn, status, lib())
    return status


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    """A cudaStream_t: of a torch stream, the current one (None), or given as a number."""
    if type(stream) is int:
        return stream
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_raw_stream(index):
    """The current stream of a device as a number (a torch stream object costs 3 us)."""
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def make_desc(w, mode=MODE_FUSED, scale=0.0, layout=LAYOUT_NATURAL):
    """Descriptor for a ``inputs.Workload`` (or anything with the same fields)."""
    return LoongAttnDesc(w.batch, w.seqlen, w.hq, w.hkv, w.head_dim, w.hp, w.cp, w.ring_inner,
                         w.ring_outer, 1 if getattr(w, "causal", True) else 0, w.placement, mode, scale, layout)


# ------------------------------------------------------------------ C entry points
def loong_attn_check(desc):
    return lib().loong_attn_check(ctypes.byref(desc))


def loong_attn_workspace_size(desc, pass_):
    return lib().loong_attn_workspace_size(ctypes.byref(desc), pass_)


def loong_ring_schedule(inner, outer):
    cp = inner * outer
    buf = (ctypes.c_int32 * (cp * cp))()
    _check("loong_ring_schedule", lib().loong_ring_schedule(inner, outer, buf))
    return [[buf[t * cp + c] for c in range(cp)] for t in range(cp)]


def _nbytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


def loong_attn_fwd(desc, q, k, v, o, lse, o_res, ws, stream=None):
    return _check("loong_attn_fwd", lib().loong_attn_fwd(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(o_res), _ptr(ws),
        _nbytes(ws), _stream(stream)))


def loong_attn_fwd_ranks(desc, rank_begin, rank_end, q, k, v, o, lse, ws, stream=None):
    return _check("loong_attn_fwd_ranks", lib().loong_attn_fwd_ranks(
        ctypes.byref(desc), rank_begin, rank_end, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
        _ptr(ws), _nbytes(ws), _stream(stream)))


def loong_attn_bwd(desc, q, k, v, o, o_res, lse, dout, dq, dk, dv, ws, stream=None):
    return _check("loong_attn_bwd", lib().loong_attn_bwd(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(o_res), _ptr(lse), _ptr(dout),
        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), _nbytes(ws), _stream(stream)))


def loong_attn_bwd_noalloc(desc, q, k, v, o, o_res, lse, dout, dq, dk, dv, stream=None):
    return _check("loong_attn_bwd_noalloc", lib().loong_attn_bwd_noalloc(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(o_res), _ptr(lse), _ptr(dout),
        _ptr(dq), _ptr(dk), _ptr(dv), _stream(stream)))


def loong_lse_merge(o_parts, lse_parts, o_out, lse_out, stream=None):
    n, rows, d = o_parts.shape
    out_bf16 = 1 if o_out.dtype == torch.bfloat16 else 0
    return _check("loong_lse_merge", lib().loong_lse_merge(
        rows, d, n, _ptr(o_parts), _ptr(lse_parts), _ptr(o_out), _ptr(lse_out), out_bf16,
        _stream(stream)))


def loong_headctx_pack(x, out, batch, cp, P, s_local, heads, d, direction, gather, stream=None):
    return _check("loong_headctx_pack", lib().loong_headctx_pack(
        batch, cp, P, s_local, heads, d, direction, gather, _ptr(x), _ptr(out), _stream(stream)))


def loong_headctx_pack_n(xs, outs, batch, cp, P, s_local, heads, d, direction, gather, stream=None):
    """loong_headctx_pack over the tensors xs -> outs (up to 4), heads[t] heads each, one launch."""
    n = len(xs)
    hs = (ctypes.c_int32 * n)(*heads)
    ins = (ctypes.c_void_p * n)(*[t.data_ptr() for t in xs])
    ous = (ctypes.c_void_p * n)(*[t.data_ptr() for t in outs])
    return _check("loong_headctx_pack_n", lib().loong_headctx_pack_n(
        n, batch, cp, P, s_local, hs, d, direction, gather, ins, ous, _stream(stream)))


class RelBuckets:
    """Buckets of the distance query - key: distance n lies in interval number
    #{bounds <= n}, interval i belongs to bucket ``bucket_of[i]`` (None: bucket
    i).  Keeps the host arrays that loong_rel_bias points at."""

    def __init__(self, num_buckets, bounds, bucket_of=None):
        bounds = [int(x) for x in bounds]
        if any(not -2 ** 31 <= x < 2 ** 31 for x in bounds):
            raise ValueError("bounds must fit 32 bits")
        self.num_buckets, self.num_bounds = int(num_buckets), len(bounds)
        self._bounds = (ctypes.c_int32 * max(1, len(bounds)))(*bounds)
        self._bucket_of = None
        if bucket_of is not None:
            if len(bucket_of) != len(bounds) + 1:
                raise ValueError("bucket_of needs one bucket for each of the len(bounds) + 1 intervals")
            self._bucket_of = (ctypes.c_int32 * len(bucket_of))(*[int(x) for x in bucket_of])
        p32 = ctypes.POINTER(ctypes.c_int32)
        self._struct = LoongRelBias(self.num_buckets, self.num_bounds, ctypes.cast(self._bounds, p32),
                                    None if self._bucket_of is None else ctypes.cast(self._bucket_of, p32), None)
        self._problems = {}

    @property
    def bounds(self):
        return list(self._bounds)[:self.num_bounds]

    @property
    def bucket_of(self):
        return list(range(self.num_bounds + 1)) if self._bucket_of is None else list(self._bucket_of)

    def struct(self, table=None):
        b = LoongRelBias.from_buffer_copy(self._struct)
        b.keep = self    # it points at this object's arrays
        if table is not None:
            b.table = table.data_ptr()
        return b

    def _problem(self, w, mode, layout):
        """(descriptor, workspace bytes forward, backward), checked; kept for a
        Workload, which cannot change (nor can these buckets)."""
        kept = type(w) is Workload
        if kept:
            p = self._problems.get((w, mode, layout))
            if p is not None:
                return p
        desc, bias = make_desc(w, mode, layout=layout), self.struct()
        _check("loong_rel_bias_check", loong_rel_bias_check(desc, bias))
        p = desc, loong_attn_bias_workspace_size(desc, bias, 0), loong_attn_bias_workspace_size(desc, bias, 1)
        if kept:
            if len(self._problems) >= 64:
                self._problems.clear()
            self._problems[w, mode, layout] = p
        return p


def log_buckets(num_buckets, max_distance, causal=True):
    """Buckets whose width grows with the distance: of a direction's n buckets
    the first e = n // 2 hold the distances 0 .. e - 1 one by one, bucket e + t
    starts at the first distance x with x / e >= (max_distance / e)^(t / (n - e)),
    and the last one has every distance from its start on.  Formed in whole
    numbers.  causal: all num_buckets for distances >= 0; else the first half
    for those and the second half, by |distance|, for negative ones (its first
    bucket stays empty).  Where two buckets would start at one distance the later
    one has it."""
    n = num_buckets if causal else num_buckets // 2
    if num_buckets < 2 or (not causal and num_buckets % 2) or n < 2:
        raise ValueError("need at least 2 buckets for each direction, and an even number of them when not causal")
    e = n // 2
    if max_distance <= e:
        raise ValueError(f"max_distance must be above {e}, the distances with a bucket of their own")
    first = {x: x for x in range(1, e + 1)}    # first distance -> bucket
    x = e
    for t in range(1, n - e):
        while x ** (n - e) * e ** t < max_distance ** t * e ** (n - e):
            # far below the bound: jump near it, then step
            near = int(e * (max_distance / e) ** (t / (n - e))) - 2
            x = max(x + 1, min(near, max_distance))
        first[x] = e + t
    starts = sorted(first)
    bounds, of = list(starts), [0] + [first[s] for s in starts]
    if not causal:
        bounds = [1 - s for s in reversed(starts)] + bounds
        of = [n + first[s] for s in reversed(starts)] + of
    return RelBuckets(num_buckets, bounds, of)


def loong_rel_bias_check(desc, bias):
    return lib().loong_rel_bias_check(ctypes.byref(desc), ctypes.byref(bias))


def loong_attn_bias_workspace_size(desc, bias, pass_):
    return lib().loong_attn_bias_workspace_size(ctypes.byref(desc), ctypes.byref(bias), pass_)


def loong_attn_bias_fwd(desc, bias, q, k, v, o, lse, o_res, ws, stream=None):
    return _check("loong_attn_bias_fwd", lib().loong_attn_bias_fwd(
        ctypes.byref(desc), ctypes.byref(bias), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(o_res), _ptr(ws),
        _nbytes(ws), _stream(stream)))


def loong_attn_bias_bwd(desc, bias, q, k, v, o, o_res, lse, dout, dq, dk, dv, dtable, ws, stream=None):
    return _check("loong_attn_bias_bwd", lib().loong_attn_bias_bwd(
        ctypes.byref(desc), ctypes.byref(bias), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(o_res), _ptr(lse),
        _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dtable), _ptr(ws), _nbytes(ws), _stream(stream)))


def loong_qk_norm_rope_fwd(desc, opts, q, k, v, wq, wk, positions, q_out, k_out, v_out, stream=None):
    return _check("loong_qk_norm_rope_fwd", lib().loong_qk_norm_rope_fwd(
        ctypes.byref(desc), ctypes.byref(opts), _ptr(q), _ptr(k), _ptr(v), _ptr(wq), _ptr(wk), _ptr(positions),
        _ptr(q_out), _ptr(k_out), _ptr(v_out), _stream(stream)))


def loong_qk_norm_rope_bwd_workspace_size(desc, opts):
    return lib().loong_qk_norm_rope_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(opts))


def loong_qk_norm_rope_bwd(desc, opts, q, k, wq, wk, positions, dq_out, dk_out, dv_out, dq, dk, dv, dwq, dwk, ws,
                           stream=None):
    return _check("loong_qk_norm_rope_bwd", lib().loong_qk_norm_rope_bwd(
        ctypes.byref(desc), ctypes.byref(opts), _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(positions), _ptr(dq_out),
        _ptr(dk_out), _ptr(dv_out), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dwq), _ptr(dwk), _ptr(ws), _nbytes(ws),
        _stream(stream)))


def loong_attn_2d_host_workspace_size(desc, pass_):
    return lib().loong_attn_2d_host_workspace_size(ctypes.byref(desc), pass_)


def loong_attn_2d_host(desc, slot, q, k, v, dout, o, lse, dq, dk, dv, ws, stream=None, done_event=None):
    """One 2D-attention pass from host tensors to host tensors (pinned for
    overlap); dout=None runs the forward alone.  done_event: a recorded
    torch.cuda.Event marking the host outputs ready, or None."""
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    ev = None if done_event is None else ctypes.c_void_p(done_event.cuda_event)
    return _check("loong_attn_2d_host", lib().loong_attn_2d_host(
        ctypes.byref(desc), slot, _ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(o), _ptr(lse), _ptr(dq),
        _ptr(dk), _ptr(dv), _ptr(ws), nbytes, _stream(stream), ev))


def loong_host_alloc(nbytes):
    """Pinned, huge-page-backed host memory of ``nbytes`` bytes (an address,
    or None for 0 bytes); release it with loong_host_free."""
    p = ctypes.c_void_p()
    _check("loong_host_alloc", lib().loong_host_alloc(nbytes, ctypes.byref(p)))
    return p.value


def loong_host_free(ptr):
    return _check("loong_host_free", lib().loong_host_free(ptr))


_HOST_BUFFERS = {}


def host_empty(shape, dtype):
    """A CPU tensor over loong_host_alloc memory (pinned, huge pages where the
    kernel offers them), for the host arguments of loong_attn_2d_host.  It
    stays allocated until host_release(t) or the end of the process."""
    n = 1
    for e in shape:
        n *= int(e)
    nbytes = n * torch.empty((), dtype=dtype).element_size()
    if nbytes == 0:
        return torch.empty(shape, dtype=dtype)
    ptr = loong_host_alloc(nbytes)
    raw = (ctypes.c_uint8 * nbytes).from_address(ptr)
    t = torch.frombuffer(raw, dtype=torch.uint8).view(dtype).view(shape)
    _HOST_BUFFERS[t.data_ptr()] = (ptr, raw)
    return t


def host_release(t):
    """Free the memory of a host_empty tensor; the tensor must not be used afterwards."""
    ptr, _ = _HOST_BUFFERS.pop(t.data_ptr())
    loong_host_free(ptr)


def loong_set_timing_events(start=None, stop=None):
    """Record torch.cuda.Event ``start``/``stop`` around the main attention
    kernels of this thread's next fwd/bwd calls (None, None to stop).  torch
    creates an event on its first record(), so record both once before
    passing them."""
    sp = None if start is None else ctypes.c_void_p(start.cuda_event)
    ep = None if stop is None else ctypes.c_void_p(stop.cuda_event)
    return _check("loong_set_timing_events", lib().loong_set_timing_events(sp, ep))


def loong_get_device_status(stream=None):
    return lib().loong_get_device_status(_stream(stream))


def loong_selftest_wait_timeout(limit_us, stream=None):
    return lib().loong_selftest_wait_timeout(limit_us, _stream(stream))


# ------------------------------------------------------------------ conveniences
def workspace(desc, pass_, device="cuda"):
    n = loong_attn_workspace_size(desc, pass_)
    return None if n == 0 else torch.empty(n, dtype=torch.uint8, device=device)


def attn_fwd(w, q, k, v, mode=MODE_FUSED, stream=None, layout=LAYOUT_NATURAL, res=True):
    """Allocate O, LSE (and O's rounding residual) with torch, run
    loong_attn_fwd, return (o, lse, o_res); o_res is None when ``res`` is
    false.  With LAYOUT_RANK_MAJOR, q/k/v (and o) are headctx_pack outputs."""
    desc = make_desc(w, mode, layout=layout)
    _check("loong_attn_check", loong_attn_check(desc))
    o = torch.empty_like(q)
    o_res = torch.empty_like(q) if res else None
    lse = torch.empty((w.batch, w.hq, w.seqlen), dtype=torch.float32, device=q.device)
    loong_attn_fwd(desc, q, k, v, o, lse, o_res, workspace(desc, 0, q.device), stream)
    return o, lse, o_res


def attn_bwd(w, q, k, v, o, lse, do, o_res=None, mode=MODE_FUSED, stream=None, layout=LAYOUT_NATURAL):
    """Allocate dQ/dK/dV with torch, run loong_attn_bwd, return them (in the
    layout of q, k).  ``o_res``: the forward's residual of O (D from O + o_res),
    or None (D from O alone)."""
    desc = make_desc(w, mode, layout=layout)
    _check("loong_attn_check", loong_attn_check(desc))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    loong_attn_bwd(desc, q, k, v, o, o_res, lse, do, dq, dk, dv, workspace(desc, 1, q.device), stream)
    return dq, dk, dv


def headctx_pack(x_nat, cp, P, gather=1, stream=None):
    """Natural [B, S, H, d] -> rank-major [B*cp, P, S/cp, H/P, d]."""
    B, S, H, d = x_nat.shape
    s_local = S // (cp * P)
    out = torch.empty((B * cp, P, S // cp, H // P, d), dtype=x_nat.dtype, device=x_nat.device)
    loong_headctx_pack(x_nat, out, B, cp, P, s_local, H, d, 0, gather, stream)
    return out


def headctx_unpack(y, batch, cp, P, gather=1, stream=None):
    """Rank-major [B*cp, P, S/cp, H/P, d] -> natural [B, S, H, d]."""
    n, P_, sgrp, hp, d = y.shape
    S = cp * sgrp
    out = torch.empty((batch, S, hp * P, d), dtype=y.dtype, device=y.device)
    loong_headctx_pack(y, out, batch, cp, P, sgrp // P, hp * P, d, 1, gather, stream)
    return out


def default_scale(d):
    return 1.0 / math.sqrt(d)


def _same(name, t, shape, dtype, device):
    """The tensor arguments of the calls below: what the C entry cannot see."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on {device}, not {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")


def _contiguous(name, t, shape, dtype, device):
    _same(name, t, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _attn_shape(w, heads, layout):
    if layout == LAYOUT_RANK_MAJOR:
        return (w.batch * w.cp, w.hp, w.seqlen // w.cp, heads // w.hp, w.head_dim)
    return (w.batch, w.seqlen, heads, w.head_dim)


_NOTHING = contextlib.nullcontext()


def _on(device, stream):
    """The calls below run on the tensors' device, on its current stream unless
    one is given, a torch stream or a number: (what to enter, the stream).  What
    a call allocates belongs to that stream.  Nothing to enter where both are
    current already."""
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, not {device}")
    if stream is None and device.index == torch.cuda.current_device():
        return _NOTHING, _current_raw_stream(device.index)
    where = contextlib.ExitStack()
    where.enter_context(torch.cuda.device(device))
    if type(stream) is int:  # 1 is the legacy default stream, as 0 is
        stream = torch.cuda.ExternalStream(0 if stream == 1 else stream, device=device)
    stream = torch.cuda.current_stream(device) if stream is None else stream
    where.enter_context(torch.cuda.stream(stream))
    return where, stream


def _checked_desc(w, layout):
    desc = make_desc(w, MODE_FUSED, layout=layout)
    _check("loong_attn_check", loong_attn_check(desc))
    return desc


_kept_desc = functools.lru_cache(maxsize=256)(_checked_desc)


def _desc_of(w, layout):
    """A checked descriptor for reading only: kept for a Workload, which cannot change."""
    return _kept_desc(w, layout) if type(w) is Workload else _checked_desc(w, layout)


def attn_bias_fwd(w, q, k, v, table, buckets, mode=MODE_FUSED, stream=None, layout=LAYOUT_NATURAL, res=True):
    """attn_fwd with a learned relative position bias: ``table`` bf16
    [num_buckets, hq], ``buckets`` a RelBuckets (log_buckets makes the usual
    ones).  Returns (o, lse, o_res); o_res is None when ``res`` is false."""
    desc, nbytes, _ = buckets._problem(w, mode, layout)
    _contiguous("table", table, (buckets.num_buckets, w.hq), torch.bfloat16, table.device)
    for n, t, h in (("q", q, w.hq), ("k", k, w.hkv), ("v", v, w.hkv)):
        _contiguous(n, t, _attn_shape(w, h, layout), torch.bfloat16, table.device)
    where, stream = _on(table.device, stream)
    with where:
        o = torch.empty_like(q)
        o_res = torch.empty_like(q) if res else None
        lse = torch.empty((w.batch, w.hq, w.seqlen), dtype=torch.float32, device=q.device)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        loong_attn_bias_fwd(desc, buckets.struct(table), q, k, v, o, lse, o_res, ws, stream)
    return o, lse, o_res


def attn_bias_bwd(w, q, k, v, o, lse, do, table, buckets, o_res=None, mode=MODE_FUSED, stream=None,
                  layout=LAYOUT_NATURAL):
    """Gradient of attn_bias_fwd: (dq, dk, dv, dtable), dtable bf16 like the table."""
    desc, _, nbytes = buckets._problem(w, mode, layout)
    _contiguous("table", table, (buckets.num_buckets, w.hq), torch.bfloat16, table.device)
    for n, t, h in (("q", q, w.hq), ("k", k, w.hkv), ("v", v, w.hkv), ("o", o, w.hq), ("do", do, w.hq),
                    ("o_res", o_res, w.hq)):
        if t is not None or n != "o_res":
            _contiguous(n, t, _attn_shape(w, h, layout), torch.bfloat16, table.device)
    _contiguous("lse", lse, (w.batch, w.hq, w.seqlen), torch.float32, table.device)
    where, stream = _on(table.device, stream)
    with where:
        dq, dk, dv, dtable = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(table)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        loong_attn_bias_bwd(desc, buckets.struct(table), q, k, v, o, o_res, lse, do, dq, dk, dv, dtable, ws, stream)
    return dq, dk, dv, dtable


class QkOpts:
    """What qk_norm_rope does to Q and K (loong_qk_opts, without the strides and
    pos_begin, which belong to a call)."""

    def __init__(self, head_dim, eps=1e-6, norm=True, w_offset=0.0, rot_dim=None, base=10000.0, inv_freq=None,
                 interleaved=False, rot_scale=1.0):
        self.rot_dim = head_dim if rot_dim is None else int(rot_dim)
        self.norm = bool(norm)
        self._inv = self._formed = None
        n = max(0, self.rot_dim // 2)
        if inv_freq is not None:
            inv = [float(x) for x in inv_freq]
            if len(inv) != n:
                raise ValueError(f"inv_freq needs {n} values")
            self._inv = self._formed = (ctypes.c_double * max(1, n))(*inv)
        elif sys.float_info.min <= base < math.inf:  # what the library would form from the base, once
            self._formed = (ctypes.c_double * max(1, n))(*[float(base) ** (-2.0 * i / self.rot_dim) for i in range(n)])
        self._structs = {}
        self._fixed = (float(base), float(eps), float(w_offset), float(rot_scale), 1 if norm else 0, self.rot_dim,
                       1 if interleaved else 0)

    def struct(self, x_strides=(0, 0, 0), dx_strides=(0, 0, 0), pos_begin=0, formed=False):
        """loong_qk_opts; formed: with the frequencies of ``base`` spelled out."""
        base, eps, w_offset, rot_scale, norm, rot_dim, inter = self._fixed
        inv = self._formed if formed else self._inv
        inv = None if inv is None else ctypes.cast(inv, ctypes.POINTER(ctypes.c_double))
        return LoongQkOpts(*x_strides, *dx_strides, pos_begin, base, inv, eps, w_offset, rot_scale, norm, rot_dim, inter)

    def _struct_of(self, x_strides, dx_strides=(0, 0, 0), pos_begin=0):
        """struct(...), kept by the strides, of which a program has a few; a
        position of its own, which counts up from call to call, takes a copy (the
        kept one may be in use by another thread's call)."""
        key = (*x_strides, *dx_strides)
        o = self._structs.get(key)
        if o is None:
            if len(self._structs) >= 64:
                self._structs.clear()
            o = self._structs[key] = self.struct(x_strides, dx_strides, formed=True)
        if pos_begin:
            o = LoongQkOpts.from_buffer_copy(o)
            o.pos_begin = pos_begin
        return o


def make_qk_opts(head_dim, **kw):
    return QkOpts(head_dim, **kw)


def _token_strides(names, ts, w, device):
    """Elements from token to token of projections: [B, S, heads, d] views whose
    heads are contiguous and whose sequences follow each other; 0 for None.  An
    expanded view repeats one token's memory: its stride of 0 is not the
    library's 0 (contiguous), and neither it nor one below a token's elements is
    taken."""
    b, s, d = w.batch, w.seqlen, w.head_dim
    out = []
    for name, t, heads in zip(names, ts, (w.hq, w.hkv, w.hkv)):
        if t is None:
            out.append(0)
            continue
        _same(name, t, (b, s, heads, d), torch.bfloat16, device)
        sb, ss, sh, sd = t.stride()
        if s == 1:  # the token's stride is the sequence's
            ss = sb if b > 1 else heads * d
        if sd != 1 or (sh != d and heads > 1) or (b > 1 and sb != s * ss) or ss < heads * d:
            raise ValueError(f"{name} must have contiguous heads and evenly spaced tokens, not strides {t.stride()}")
        out.append(ss)
    return out


def _qk_weights(w, wq, wk, positions, device):
    if wq is not None:
        _contiguous("wq", wq, (w.head_dim,), torch.float32, device)
    if wk is not None:
        _contiguous("wk", wk, (w.head_dim,), torch.float32, device)
    if positions is not None:
        _contiguous("positions", positions, (w.batch, w.seqlen), torch.int64, device)


def qk_norm_rope(w, opts, q, k, v=None, wq=None, wk=None, positions=None, pos_begin=0, layout=LAYOUT_NATURAL,
                 stream=None):
    """RMS norm and position rotation of every query and key head and the
    attention's layout, in one pass: projections [B, S, heads, d] (views of one
    fused projection, or contiguous) -> (q, k, v) as attn_fwd takes them.  ``v``
    is only brought into the layout; None leaves it out."""
    desc = _desc_of(w, layout)
    _qk_weights(w, wq, wk, positions, q.device)
    o = opts._struct_of(_token_strides(("q", "k", "v"), (q, k, v), w, q.device), pos_begin=pos_begin)
    where, stream = _on(q.device, stream)
    with where:
        out = [None if t is None else q.new_empty(_attn_shape(w, h, layout))
               for t, h in ((q, w.hq), (k, w.hkv), (v, w.hkv))]
        loong_qk_norm_rope_fwd(desc, o, q, k, v, wq, wk, positions, *out, stream)
    return tuple(out)


def qk_norm_rope_bwd(w, opts, q, k, dq, dk, dv=None, wq=None, wk=None, positions=None, pos_begin=0,
                     layout=LAYOUT_NATURAL, into=None, stream=None):
    """Gradient of qk_norm_rope: from dq, dk, dv in the attention's layout to
    (dq, dk, dv, dwq, dwk) of the projections and the norm weights (None where
    there is none).  ``into``: the three projection gradients to write, e.g.
    views of one fused gradient (the third None without dv); else they are made
    contiguous."""
    desc = _desc_of(w, layout)
    _qk_weights(w, wq, wk, positions, q.device)
    for n, t, h in (("dq", dq, w.hq), ("dk", dk, w.hkv), ("dv", dv, w.hkv)):
        if t is not None or n != "dv":
            _contiguous(n, t, _attn_shape(w, h, layout), torch.bfloat16, q.device)
    if into is not None and (into[2] is None) != (dv is None):
        raise ValueError("into[2] belongs to dv: give both or neither")
    where, stream = _on(q.device, stream)
    with where:
        if into is None:
            into = [None if t is None else q.new_empty((w.batch, w.seqlen, h, w.head_dim))
                    for t, h in ((dq, w.hq), (dk, w.hkv), (dv, w.hkv))]
        o = opts._struct_of(_token_strides(("q", "k", "v"), (q, k, None), w, q.device),
                            _token_strides(("into[0]", "into[1]", "into[2]"), into, w, q.device), pos_begin)
        dwq = None if wq is None or not opts.norm else torch.empty_like(wq)
        dwk = None if wk is None or not opts.norm else torch.empty_like(wk)
        n = loong_qk_norm_rope_bwd_workspace_size(desc, o)
        ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n and (dwq is not None or dwk is not None) else None
        loong_qk_norm_rope_bwd(desc, o, q, k, wq, wk, positions, dq, dk, dv, *into, dwq, dwk, ws, stream)
    return (*into, dwq, dwk)
