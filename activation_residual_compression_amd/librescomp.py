"""ctypes binding of the librescomp C ABI (``include/librescomp.h``).

Argument marshalling only: every step of the compression path runs in the HIP
kernels of ``librescomp.so``. Functions keep the C names; a non-RC_OK status
raises :class:`RcError`. Tensor arguments may be torch tensors (their
``data_ptr()`` is passed) or raw integer device addresses; the low-rank start
matrices ``q0`` may also be a host numpy array, which ``Plan`` copies to the
device for the plan's set-up. Streams may be a ``torch.cuda.Stream``, a raw
``hipStream_t`` integer, or None for torch's current stream.

The library must be built first (``__graft_entry__.build()`` or
``python -m activation_residual_compression_amd.build``); importing this module
without it raises, so nothing can silently fall back to another implementation.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# LIBRESCOMP_LIB names another build of the library (the CPU sanitizer build
# of the host code); by default the in-tree build is loaded.
LIB_PATH = os.environ.get("LIBRESCOMP_LIB") or os.path.join(_HERE, "lib", "librescomp.so")

RC_OK, RC_ERR_INVALID_ARG, RC_ERR_UNSUPPORTED, RC_ERR_ALIGNMENT, RC_ERR_HIP = 0, 1, 2, 3, 4
RC_ERR_NUMERIC, RC_ERR_NONFINITE = 5, 6
RC_BF16, RC_F32 = 0, 1
RC_Q1, RC_Q2, RC_NM, RC_LOWRANK, RC_BLOCKSEL = 0, 1, 2, 3, 4
RC_MAX_PEERS = 8
RC_LR_BF16_FACTORS = 1  # rc_params_t.flags, RC_LOWRANK only
RC_LR_ONE_STREAM = 2    # rc_params_t.flags, RC_LOWRANK only: no second stream in rc_compress
RC_BS_SCORE_LAST_SENT = 4  # rc_params_t.flags, RC_BLOCKSEL only: score against ahat
RC_CHECK_FINITE = 8        # rc_params_t.flags, any scheme: reject NaN / Inf inputs (syncs)
RC_LR_CHECK_NUMERIC = 16   # rc_params_t.flags, RC_LOWRANK only: report dead pivots (syncs)

SCHEMES = {"q1": RC_Q1, "q2": RC_Q2, "nm": RC_NM, "lr": RC_LOWRANK, "bs": RC_BLOCKSEL}
DTYPES = {"bf16": RC_BF16, "f32": RC_F32}


class rc_shape_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32)]


class rc_params_t(ctypes.Structure):
    _fields_ = [("group", ctypes.c_int32), ("nm_keep", ctypes.c_int32),
                ("nm_block", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("iters", ctypes.c_int32), ("seed", ctypes.c_uint64), ("q0", ctypes.c_void_p),
                ("flags", ctypes.c_uint32),
                ("grid_w", ctypes.c_int32), ("keep_blocks", ctypes.c_int32)]


class rc_state_t(ctypes.Structure):
    _fields_ = [("ahat", ctypes.c_void_p), ("e", ctypes.c_void_p)]


RC_KV_BLOCK, RC_KV_QTILE, RC_KV_MAX_BLOCKS = 64, 128, 8192  # librescomp_kv.h
RC_KV_CAUSAL = 1  # rc_kv_params_t.flags


class rc_kv_shape_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "q_heads", "kv_heads", "head_dim", "pool_blocks",
                                              "seq_blocks")]


class rc_kv_params_t(ctypes.Structure):
    _fields_ = [("max_queries", ctypes.c_int32), ("scale", ctypes.c_float), ("q_tile", ctypes.c_int32),
                ("keep_blocks", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class rc_kv_cache_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale")]


class rc_kv_view_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int), ("batch_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class RcError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, rc_status_string(status)))


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            "librescomp.so is not built (expected at %s); run __graft_entry__.build() "
            "or python -m activation_residual_compression_amd.build" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    st = ctypes.c_int
    lib.rc_plan_create.restype = st
    lib.rc_plan_create.argtypes = [rc_shape_t, ctypes.c_int, ctypes.c_int,
                                   ctypes.POINTER(rc_params_t), ctypes.POINTER(vp)]
    lib.rc_compress.restype = st
    lib.rc_compress.argtypes = [vp, vp, vp, ctypes.POINTER(rc_state_t), vp]
    lib.rc_compress_lowrank_noalloc.restype = st
    lib.rc_compress_lowrank_noalloc.argtypes = [rc_shape_t, ctypes.c_int, ctypes.POINTER(rc_params_t),
                                                vp, vp, ctypes.POINTER(rc_state_t), vp]
    lib.rc_decompress.restype = st
    lib.rc_decompress.argtypes = [vp, vp, vp, vp]
    lib.rc_compress_send.restype = st
    lib.rc_compress_send.argtypes = [vp, vp, vp, vp, ctypes.POINTER(rc_state_t), vp, vp, ctypes.c_int]
    lib.rc_decompress_many.restype = st
    lib.rc_decompress_many.argtypes = [vp, vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.c_int]
    lib.rc_plan_destroy.restype = st
    lib.rc_plan_destroy.argtypes = [vp]
    lib.rc_plan_reset_state.restype = st
    lib.rc_plan_reset_state.argtypes = [vp, vp]
    for f in ("rc_packed_bytes", "rc_tensor_packed_bytes", "rc_workspace_bytes"):
        getattr(lib, f).restype = sz
        getattr(lib, f).argtypes = [vp]
    lib.rc_kv_plan_create.restype = st
    lib.rc_kv_plan_create.argtypes = [rc_kv_shape_t, ctypes.c_int, ctypes.POINTER(rc_kv_params_t),
                                      ctypes.POINTER(vp)]
    cache, view = ctypes.POINTER(rc_kv_cache_t), ctypes.POINTER(rc_kv_view_t)
    lib.rc_kv_store.restype = st
    lib.rc_kv_store.argtypes = [vp, vp, cache, vp, vp, vp, ctypes.c_int, view, view]
    lib.rc_kv_select.restype = st
    lib.rc_kv_select.argtypes = [vp, vp, cache, vp, vp, ctypes.c_int64, ctypes.c_int, view, vp]
    lib.rc_kv_attend.restype = st
    lib.rc_kv_attend.argtypes = [vp, vp, cache, vp, vp, ctypes.c_int64, ctypes.c_int, view, vp, view, vp]
    lib.rc_kv_plan_destroy.restype = st
    lib.rc_kv_plan_destroy.argtypes = [vp]
    lib.rc_kv_workspace_bytes.restype = sz
    lib.rc_kv_workspace_bytes.argtypes = [vp]
    lib.rc_status_string.restype = ctypes.c_char_p
    lib.rc_status_string.argtypes = [ctypes.c_int]
    lib.rcx_lowrank_workspace.restype = ctypes.c_int
    lib.rcx_lowrank_r_probe.restype = ctypes.c_int
    lib.rcx_lowrank_r_probe.argtypes = [vp, ctypes.c_int, vp]
    lib.rcx_lowrank_workspace.argtypes = [vp, ctypes.POINTER(vp), ctypes.c_int]
    lib.rcx_device_to_host.restype = ctypes.c_int
    lib.rcx_device_to_host.argtypes = [vp, vp, sz]
    lib.rcx_hbm_probe.restype = ctypes.c_int
    lib.rcx_hbm_probe.argtypes = [ctypes.c_int, vp, vp, vp, ctypes.c_int64, vp]
    return lib


_lib = _load()
lib = _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if hasattr(x, "ctypes"):  # numpy (host)
        return x.ctypes.data
    raise TypeError("cannot take a device pointer of %r" % type(x))


def _dev_buffer(x, nbytes, what):
    """Device pointer of x, checked when x is a tensor: on a GPU, contiguous and
    at least nbytes long (the kernels would otherwise read or write past it, or
    dereference host memory). Raw integers pass through unchecked."""
    if hasattr(x, "data_ptr") and hasattr(x, "is_cuda"):
        if not x.is_cuda:
            raise ValueError("%s must be a device tensor" % what)
        if not x.is_contiguous():
            raise ValueError("%s must be contiguous" % what)
        have = x.numel() * x.element_size()
        if have < nbytes:
            raise ValueError("%s holds %d bytes, the call needs %d" % (what, have, nbytes))
    return _ptr(x)


def _sized(x, nbytes, what):
    """Pointer of x (device or pinned host), checked for size when x is a tensor."""
    if hasattr(x, "numel") and hasattr(x, "element_size"):
        have = x.numel() * x.element_size()
        if have < nbytes:
            raise ValueError("%s holds %d bytes, the call needs %d" % (what, have, nbytes))
    return _ptr(x)


def _current_stream():
    """torch's current stream of the current device, as a raw hipStream_t."""
    global _current_stream
    import torch
    raw, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
    if raw is not None and device is not None:   # without building a Stream object: 0.2 us instead of 3
        torch.cuda.init()
        _current_stream = lambda: raw(device())  # noqa: E731
    else:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _current_stream()


def _stream(s):
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int, where: str):
    if status != RC_OK:
        raise RcError(status, where)


# ------------------------------------------------------------------ C names
def rc_status_string(status: int) -> str:
    return _lib.rc_status_string(int(status)).decode()


def rc_plan_create(shape, dtype, scheme, params: rc_params_t):
    """shape: rc_shape_t or (batch, rows, cols); dtype/scheme: enum ints or names."""
    if not isinstance(shape, rc_shape_t):
        shape = rc_shape_t(*shape)
    dtype = DTYPES.get(dtype, dtype)
    scheme = SCHEMES.get(scheme, scheme)
    plan = ctypes.c_void_p()
    _check(_lib.rc_plan_create(shape, int(dtype), int(scheme), ctypes.byref(params),
                               ctypes.byref(plan)), "rc_plan_create")
    return plan


def rc_compress(plan, stream, a_t, state: rc_state_t, packed_out):
    _check(_lib.rc_compress(plan, _stream(stream), _ptr(a_t), ctypes.byref(state), _ptr(packed_out)),
           "rc_compress")


RC_NOALLOC_SCRATCH_BYTES = 64 << 20


def rc_compress_lowrank_noalloc(shape, dtype, params: rc_params_t, stream, a_t, state: rc_state_t,
                                packed_out):
    """The plan-free, allocation-free low-rank sender step (librescomp.h)."""
    if not isinstance(shape, rc_shape_t):
        shape = rc_shape_t(*shape)
    _check(_lib.rc_compress_lowrank_noalloc(shape, int(DTYPES.get(dtype, dtype)), ctypes.byref(params),
                                            _stream(stream), _ptr(a_t), ctypes.byref(state),
                                            _ptr(packed_out)), "rc_compress_lowrank_noalloc")


def rc_decompress(plan, stream, packed_in, recon_state):
    _check(_lib.rc_decompress(plan, _stream(stream), _ptr(packed_in), _ptr(recon_state)),
           "rc_decompress")


def rc_compress_send(plan, stream, copy_stream, a_t, state: rc_state_t, packed_out, packed_dst,
                     chunk):
    _check(_lib.rc_compress_send(plan, _stream(stream), _stream(copy_stream), _ptr(a_t),
                                 ctypes.byref(state), _ptr(packed_out), _ptr(packed_dst), int(chunk)),
           "rc_compress_send")


def rc_decompress_many(plan, stream, packed_in, recon_states):
    """packed_in, recon_states: equal-length sequences (one entry per peer)."""
    n = len(packed_in)
    if n != len(recon_states):
        raise ValueError("one recon state per packed stream")
    pk = (ctypes.c_void_p * max(n, 1))(*[_ptr(x) for x in packed_in])
    rs = (ctypes.c_void_p * max(n, 1))(*[_ptr(x) for x in recon_states])
    _check(_lib.rc_decompress_many(plan, _stream(stream), pk, rs, n), "rc_decompress_many")


def rc_plan_reset_state(plan, stream):
    _check(_lib.rc_plan_reset_state(plan, _stream(stream)), "rc_plan_reset_state")


def rc_plan_destroy(plan):
    _check(_lib.rc_plan_destroy(plan), "rc_plan_destroy")


def rc_packed_bytes(plan) -> int:
    return int(_lib.rc_packed_bytes(plan))


def rc_tensor_packed_bytes(plan) -> int:
    return int(_lib.rc_tensor_packed_bytes(plan))


def rc_workspace_bytes(plan) -> int:
    return int(_lib.rc_workspace_bytes(plan))


def make_params(scheme, *, group=0, nm_keep=0, nm_block=0, rank=0, iters=0, seed=0, q0=None,
                flags=0, grid_w=0, keep_blocks=0):
    """rc_params_t for a scheme; q0 (device fp32 [batch][cols][rank], or None to
    draw the start matrices from `seed`) is referenced, not copied, so keep it
    alive until rc_plan_create returns."""
    p = rc_params_t(int(group), int(nm_keep), int(nm_block), int(rank), int(iters), int(seed),
                    _ptr(q0), int(flags), int(grid_w), int(keep_blocks))
    p._q0_ref = q0
    return p


RCX_PROBE_COPY, RCX_PROBE_READ, RCX_PROBE_WRITE, RCX_PROBE_SENDER_MIX, RCX_PROBE_RECEIVER_RMW = range(5)
RCX_R_PROBE_RQ, RCX_R_PROBE_RTP = 0, 1


def rcx_device_to_host(src, nbytes):
    """bytes at device address src, copied synchronously (librescomp_diag.h)."""
    import numpy as np
    out = np.empty(int(nbytes), np.uint8)
    err = _lib.rcx_device_to_host(out.ctypes.data, _ptr(src), int(nbytes))
    if err != 0:
        raise RuntimeError("rcx_device_to_host: hipError %d" % err)
    return out


def rcx_hbm_probe(kind, a, b, c, n, stream=None):
    """Launch one HBM reference kernel (librescomp_diag.h); raises on a HIP error."""
    err = _lib.rcx_hbm_probe(int(kind), _ptr(a), _ptr(b), _ptr(c), int(n), _stream(stream))
    if err != 0:
        raise RuntimeError("rcx_hbm_probe: hipError %d" % err)


# ------------------------------------------------------------------ convenience
class Plan:
    """Owns one rc_plan_t; a thin wrapper over the C calls above."""

    def __init__(self, shape, dtype, scheme, **params):
        self.shape = tuple(shape)
        self.dtype = dtype
        self.scheme = scheme
        q0 = params.get("q0")
        if q0 is not None:
            want = self.shape[0] * self.shape[2] * int(params.get("rank", 0))
            size = q0.numel() if hasattr(q0, "numel") else int(getattr(q0, "size", -1))
            if SCHEMES.get(scheme, scheme) == RC_LOWRANK and size != want:
                # the library reads batch * cols * rank floats through the pointer
                raise ValueError("q0 holds %d floats; [batch][cols][rank] needs %d" % (size, want))
            if hasattr(q0, "data_ptr"):
                if not (q0.is_cuda and q0.is_contiguous()) or str(q0.dtype) != "torch.float32":
                    raise ValueError("q0 must be a contiguous fp32 device tensor")
            else:  # host array: a device copy for the plan's set-up
                import numpy as np
                import torch
                q0 = torch.from_numpy(np.ascontiguousarray(q0, dtype=np.float32)).to("cuda")
                torch.cuda.synchronize()
            params["q0"] = q0
        self._params = make_params(scheme, **params)
        self.handle = rc_plan_create(self.shape, dtype, scheme, self._params)
        self._params._q0_ref = None  # the plan has its own copy of the start matrices
        self.packed_bytes = rc_packed_bytes(self.handle)
        self.tensor_packed_bytes = rc_tensor_packed_bytes(self.handle)
        self.workspace_bytes = rc_workspace_bytes(self.handle)

    def _elems(self):
        return self.shape[0] * self.shape[1] * self.shape[2]

    def _in_bytes(self):
        return self._elems() * (2 if DTYPES.get(self.dtype, self.dtype) == RC_BF16 else 4)

    def _input(self, a_t):
        """a_t checked as _dev_buffer does, and for the plan's dtype (an fp32 tensor
        given to a bf16 plan would otherwise be read as pairs of bf16 values)."""
        if hasattr(a_t, "dtype") and hasattr(a_t, "data_ptr"):
            want = "torch.bfloat16" if DTYPES.get(self.dtype, self.dtype) == RC_BF16 else "torch.float32"
            if str(a_t.dtype) != want:
                raise ValueError("a_t is %s, the plan takes %s" % (a_t.dtype, want))
        return _dev_buffer(a_t, self._in_bytes(), "a_t")

    def compress(self, a_t, ahat, e, packed_out, stream=None):
        a = self._input(a_t)
        st = rc_state_t(_dev_buffer(ahat, 4 * self._elems(), "ahat"),
                        _dev_buffer(e, 4 * self._elems(), "e"))
        rc_compress(self.handle, stream, a, st,
                    _dev_buffer(packed_out, self.packed_bytes, "packed_out"))

    def decompress(self, packed_in, recon_state, stream=None):
        rc_decompress(self.handle, stream, _dev_buffer(packed_in, self.packed_bytes, "packed_in"),
                      _dev_buffer(recon_state, 4 * self._elems(), "recon_state"))

    def compress_send(self, a_t, ahat, e, packed_out, packed_dst, chunk, copy_stream, stream=None):
        a = self._input(a_t)
        st = rc_state_t(_dev_buffer(ahat, 4 * self._elems(), "ahat"),
                        _dev_buffer(e, 4 * self._elems(), "e"))
        rc_compress_send(self.handle, stream, copy_stream, a, st,
                         _dev_buffer(packed_out, self.packed_bytes, "packed_out"),
                         _sized(packed_dst, self.packed_bytes, "packed_dst"), chunk)

    def decompress_many(self, packed_in, recon_states, stream=None):
        rc_decompress_many(self.handle, stream,
                           [_dev_buffer(p, self.packed_bytes, "packed_in") for p in packed_in],
                           [_dev_buffer(r, 4 * self._elems(), "recon_state") for r in recon_states])

    def reset_state(self, stream=None):
        rc_plan_reset_state(self.handle, stream)

    def r_probe(self, pattern, stream=None):
        """Read this low-rank plan's R in the pattern of its R*Q (RCX_R_PROBE_RQ)
        or R^T*P (RCX_R_PROBE_RTP) pass and nothing else (librescomp_diag.h)."""
        err = _lib.rcx_lowrank_r_probe(self.handle, int(pattern), _stream(stream))
        if err != 0:
            raise RuntimeError("rcx_lowrank_r_probe: %d" % err)

    def lowrank_workspace(self):
        """Device pointers (R, P, Pbt, Qt, Q0t, Qtb, gsum, linv) and rows_pad (diagnostics)."""
        arr = (ctypes.c_void_p * 8)()
        rp = _lib.rcx_lowrank_workspace(self.handle, arr, 8)
        if rp < 0:
            raise ValueError("not a low-rank plan")
        return [int(v or 0) for v in arr], rp

    def close(self):
        if self.handle is not None:
            rc_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


# ------------------------------------------------------------------ 8-bit key/value cache
def rc_kv_plan_create(shape, dtype, params: rc_kv_params_t):
    """shape: rc_kv_shape_t or its fields in order; dtype: enum int or name."""
    if not isinstance(shape, rc_kv_shape_t):
        shape = rc_kv_shape_t(*shape)
    plan = ctypes.c_void_p()
    _check(_lib.rc_kv_plan_create(shape, int(DTYPES.get(dtype, dtype)), ctypes.byref(params), ctypes.byref(plan)),
           "rc_kv_plan_create")
    return plan


def rc_kv_store(plan, stream, cache: rc_kv_cache_t, table, start, count, tokens, k: rc_kv_view_t, v: rc_kv_view_t):
    _check(_lib.rc_kv_store(plan, _stream(stream), ctypes.byref(cache), _ptr(table), _ptr(start), _ptr(count),
                            int(tokens), ctypes.byref(k), ctypes.byref(v)), "rc_kv_store")


def rc_kv_select(plan, stream, cache: rc_kv_cache_t, table, kv_len, max_len, queries, q: rc_kv_view_t, blocks):
    _check(_lib.rc_kv_select(plan, _stream(stream), ctypes.byref(cache), _ptr(table), _ptr(kv_len), int(max_len),
                             int(queries), ctypes.byref(q), _ptr(blocks)), "rc_kv_select")


def rc_kv_attend(plan, stream, cache: rc_kv_cache_t, table, kv_len, max_len, queries, q: rc_kv_view_t, blocks,
                 out: rc_kv_view_t, lse):
    _check(_lib.rc_kv_attend(plan, _stream(stream), ctypes.byref(cache), _ptr(table), _ptr(kv_len), int(max_len),
                             int(queries), ctypes.byref(q), _ptr(blocks), ctypes.byref(out), _ptr(lse)),
           "rc_kv_attend")


def rc_kv_plan_destroy(plan):
    _check(_lib.rc_kv_plan_destroy(plan), "rc_kv_plan_destroy")


def rc_kv_workspace_bytes(plan) -> int:
    return int(_lib.rc_kv_workspace_bytes(plan))


class KvCache:
    """The tensors of an 8-bit key/value cache (librescomp_kv.h), the caller's:
    k [pool, heads, D/16, 64, 16] and v [pool, heads, 4, D, 16] of one byte an
    element (float8_e4m3fn, or uint8), k_scale, v_scale and k_mean_scale fp32
    [pool, heads], k_mean int8 [pool, heads, D], all contiguous on the GPU."""

    def __init__(self, k, v, k_scale, v_scale, k_mean, k_mean_scale):
        self.pool_blocks, self.kv_heads, chunks = (int(n) for n in k.shape[:3])
        self.head_dim = 16 * chunks
        row = (self.pool_blocks, self.kv_heads)
        for what, x, shape, types in (
                ("k", k, row + (chunks, RC_KV_BLOCK, 16), ("torch.float8_e4m3fn", "torch.uint8")),
                ("v", v, row + (4, self.head_dim, 16), ("torch.float8_e4m3fn", "torch.uint8")),
                ("k_scale", k_scale, row, ("torch.float32",)), ("v_scale", v_scale, row, ("torch.float32",)),
                ("k_mean", k_mean, row + (self.head_dim,), ("torch.int8",)),
                ("k_mean_scale", k_mean_scale, row, ("torch.float32",))):
            if tuple(x.shape) != shape:
                raise ValueError("%s is %s, a cache of this k has %s" % (what, tuple(x.shape), shape))
            if str(x.dtype) not in types:
                raise ValueError("%s is %s, the cache takes %s" % (what, x.dtype, " or ".join(types)))
        for what, x in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale), ("k_mean", k_mean),
                        ("k_mean_scale", k_mean_scale)):
            _dev_buffer(x, 0, what)
        self.k, self.v, self.k_scale, self.v_scale, self.k_mean, self.k_mean_scale = \
            k, v, k_scale, v_scale, k_mean, k_mean_scale
        self.struct = rc_kv_cache_t(*(x.data_ptr() for x in (k, v, k_scale, v_scale, k_mean, k_mean_scale)))
        self.geometry = (self.pool_blocks, self.kv_heads, self.head_dim)

    @classmethod
    def empty(cls, pool_blocks, kv_heads, head_dim, device="cuda"):
        """A cache that holds nothing (all zero)."""
        import torch
        row = (pool_blocks, kv_heads)

        def zeros(shape, dtype):
            return torch.zeros(shape, dtype=dtype, device=device)
        return cls(zeros(row + (head_dim // 16, RC_KV_BLOCK, 16), torch.uint8).view(torch.float8_e4m3fn),
                   zeros(row + (4, head_dim, 16), torch.uint8).view(torch.float8_e4m3fn),
                   zeros(row, torch.float32) + 1.0, zeros(row, torch.float32) + 1.0,
                   zeros(row + (head_dim,), torch.int8), zeros(row, torch.float32))


class KvPlan:
    """Owns one rc_kv_plan_t; a thin wrapper over the calls above that checks what
    it is given. Tensors are [batch, tokens, heads, head_dim] with contiguous rows
    (any strides between them)."""

    def __init__(self, batch, q_heads, kv_heads, head_dim, pool_blocks, seq_blocks, dtype="bf16", max_queries=1,
                 causal=False, scale=0.0, q_tile=0, keep_blocks=0):
        import torch
        self._codes, self._int32 = {torch.bfloat16: RC_BF16, torch.float32: RC_F32}, torch.int32
        self.batch, self.q_heads, self.kv_heads, self.head_dim = int(batch), int(q_heads), int(kv_heads), int(head_dim)
        self.seq_blocks, self.q_tile, self.keep_blocks = int(seq_blocks), int(q_tile), int(keep_blocks)
        self.geometry = (int(pool_blocks), self.kv_heads, self.head_dim)
        params = rc_kv_params_t(int(max_queries), float(scale), self.q_tile, self.keep_blocks,
                                RC_KV_CAUSAL if causal else 0)
        self.handle = None
        self.dtype = DTYPES.get(dtype, dtype)
        self.handle = rc_kv_plan_create((self.batch, self.q_heads, self.kv_heads, self.head_dim, int(pool_blocks),
                                         self.seq_blocks), self.dtype, params)
        self.workspace_bytes = rc_kv_workspace_bytes(self.handle)

    def _rows(self, x, heads, what, tokens=None, dtype=None):
        """View of x, checked for device, shape and type."""
        if not x.is_cuda:
            raise ValueError("%s must be a device tensor" % what)
        shape = x.shape
        if len(shape) != 4 or shape != (self.batch, shape[1] if tokens is None else tokens, heads, self.head_dim):
            raise ValueError("%s is %s, the call takes (%d, %s, %d, %d)" % (
                what, tuple(shape), self.batch, "tokens" if tokens is None else tokens, heads, self.head_dim))
        code = self._codes.get(x.dtype)
        if code is None or (dtype is not None and code != dtype):
            raise ValueError("%s is %s, the call takes %s" % (what, x.dtype, {
                None: "bfloat16 or float32", RC_BF16: "bfloat16", RC_F32: "float32"}[dtype]))
        b, t, h, d = x.stride()
        if d != 1:
            raise ValueError("%s must have contiguous rows of head_dim" % what)
        return rc_kv_view_t(x.data_ptr(), code, b, t, h)

    def _ints(self, x, n, what):
        if x is None:
            return None
        if x.dtype is not self._int32 or not x.is_cuda or not x.is_contiguous() or x.numel() != n:
            raise ValueError("%s must be a contiguous int32 device tensor of %d values" % (what, n))
        return x.data_ptr()

    def _cache(self, cache):
        if cache.geometry != self.geometry:
            raise ValueError("the cache has (blocks, heads, head_dim) %s, the plan %s" % (cache.geometry, self.geometry))
        return cache.struct

    def store(self, cache, start, k, v, table=None, count=None, stream=None):
        """Quantise k, v [batch, tokens, kv_heads, head_dim] into the cache, from
        position start[b] of each sequence on."""
        tokens = k.shape[1]
        kv, vv = self._rows(k, self.kv_heads, "k"), self._rows(v, self.kv_heads, "v", tokens)
        rc_kv_store(self.handle, stream, self._cache(cache), self._ints(table, self.batch * self.seq_blocks, "table"),
                    self._ints(start, self.batch, "start"), self._ints(count, self.batch, "count"), tokens, kv, vv)

    def _lists(self, blocks, queries):
        tiles = -(-queries // self.q_tile) if self.q_tile else 0
        return self._ints(blocks, self.batch * self.kv_heads * tiles * self.keep_blocks, "blocks")

    def select(self, cache, kv_len, q, blocks, table=None, max_len=0, stream=None):
        """Choose blocks for q [batch, queries, q_heads, head_dim]; writes blocks, int32
        [batch, kv_heads, ceil(queries / q_tile), keep_blocks]."""
        queries = q.shape[1]
        view = self._rows(q, self.q_heads, "q", None, self.dtype)
        rc_kv_select(self.handle, stream, self._cache(cache), self._ints(table, self.batch * self.seq_blocks, "table"),
                     self._ints(kv_len, self.batch, "kv_len"), max_len, queries, view, self._lists(blocks, queries))

    def attend(self, cache, kv_len, q, out, lse=None, table=None, max_len=0, blocks=None, stream=None):
        """Attention of q over the cache (over the chosen blocks, if given); writes out,
        like q, and lse, fp32 [batch, queries, q_heads]. In bf16 the softmax weights have 11
        bits in their product with the values, in fp32 queries and weights have 22."""
        queries = q.shape[1]
        view = self._rows(q, self.q_heads, "q", None, self.dtype)
        to = self._rows(out, self.q_heads, "out", queries, self.dtype)
        if lse is not None:
            if self._codes.get(lse.dtype) != RC_F32 or lse.numel() != self.batch * queries * self.q_heads:
                raise ValueError("lse must hold %d fp32 values" % (self.batch * queries * self.q_heads))
            lse = _dev_buffer(lse, 0, "lse")
        rc_kv_attend(self.handle, stream, self._cache(cache), self._ints(table, self.batch * self.seq_blocks, "table"),
                     self._ints(kv_len, self.batch, "kv_len"), max_len, queries, view, self._lists(blocks, queries), to,
                     lse)

    def close(self):
        if self.handle is not None:
            rc_kv_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
