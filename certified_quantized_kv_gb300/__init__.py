"""Python binding of libkvq: certified quantized-KV decode attention on GB300 (sm_103a).

Argument marshalling only: every step of the path runs in the CUDA kernels of
``libkvq.so`` behind the C ABI declared in ``include/kvq.h``.  Torch supplies device
memory and streams.  Importing this module fails loudly if the library is not built
(``python -c "import __graft_entry__ as g; g.build()"``); there is no fallback.
"""

from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

KVQ_OK = 0
KVQ_ERR_INVALID = 1
KVQ_ERR_OOM = 2
KVQ_ERR_HOST_OOM = 3
KVQ_ERR_CAPACITY = 4
KVQ_ERR_CUDA = 5
KVQ_ERR_TIMEOUT = 6

DEBUG_FORCE_RANK_FAIL = 0x1
DEBUG_FORCE_DENSE = 0x2
DEBUG_SYNC = 0x4
DEBUG_PROFILE = 0x8
DEBUG_BOUNDS = 0x10
DEBUG_FAIL_MIRROR = 0x20

HEAD_DIM = 128
BLOCK = 64
VALUE_GROUP = 32


class KvqError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"kvq status {status}: {msg}")
        self.status = status


class kvq_config(ctypes.Structure):
    _fields_ = [
        ("n_layers", ctypes.c_int), ("batch", ctypes.c_int), ("n_q_heads", ctypes.c_int),
        ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("block_tokens", ctypes.c_int),
        ("value_group", ctypes.c_int), ("max_ctx", ctypes.c_int), ("rank_positions", ctypes.c_int),
        ("l4_head_fraction", ctypes.c_float), ("value_bits", ctypes.c_int),
        ("v_tol", ctypes.c_float), ("resident_blocks", ctypes.c_int),
    ]


class kvq_kernel_stat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int64), ("total_ms", ctypes.c_double)]


class kvq_rope_config(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
        ("scaling", ctypes.c_int), ("base", ctypes.c_double), ("factor", ctypes.c_double),
        ("original_ctx", ctypes.c_int), ("low", ctypes.c_double), ("high", ctypes.c_double),
        ("magnitude", ctypes.c_double),
    ]


class kvq_rope_plan(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("magnitude", ctypes.c_float), ("step", ctypes.c_uint64 * 128)]


CERT_DTYPE = np.dtype([("e_key", "<f4"), ("e_val", "<f4"), ("rank_ok", "<i4"), ("level", "<i4"),
                       ("k_star", "<i4"), ("n_val_promoted", "<i4"), ("promoted_bytes", "<i8")])
assert CERT_DTYPE.itemsize == 32

_lib = None


def load_library() -> ctypes.CDLL:
    """Load libkvq.so from this package directory (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libkvq.so not built at {LIB_PATH}; run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64
    sigs = {
        "kvq_cache_create": [ctypes.POINTER(kvq_config), ctypes.POINTER(vp)],
        "kvq_cache_destroy": [vp],
        "kvq_append": [vp, i32, vp, vp, i32, vp],
        "kvq_decode_attention": [vp, i32, vp, f32, f32, vp, vp, vp, vp],
        "kvq_decode_attention_uncertified": [vp, i32, vp, vp, vp, vp],
        "kvq_set_debug": [vp, i32],
        "kvq_cache_length": [vp, i32, ctypes.POINTER(i32)],
        "kvq_export_tier1": [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp],
        "kvq_export_decode_state": [vp, vp, vp, vp, vp, vp, vp, vp],
        "kvq_profile_read": [vp, ctypes.POINTER(kvq_kernel_stat), i32, ctypes.POINTER(i32), i32],
        "kvq_dense_decode_noalloc": [vp, vp, vp, i32, i32, i32, i32, vp, vp],
        "kvq_dense_attention_workspace": [i32, i32, i32, i32, ctypes.POINTER(ctypes.c_size_t)],
        "kvq_dense_attention": [vp, vp, vp, i32, i32, i32, i32, vp, vp, ctypes.c_size_t, vp],
        "kvq_debug_fill_tier2": [vp, i32, ctypes.c_uint16],
        "kvq_residency_stats": [vp, i32, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64),
                                ctypes.POINTER(i32), i32],
        "kvq_rope_plan_init": [ctypes.POINTER(kvq_rope_config), ctypes.POINTER(kvq_rope_plan)],
        "kvq_rope": [vp, i32, vp, i64, i64, vp, i32, i32, vp, i64, i64, vp],
        "kvq_paged_page_bytes": [i32, ctypes.POINTER(ctypes.c_size_t)],
        "kvq_paged_append": [vp, i32, vp, i64, i64, vp, i64, i64, vp, vp, i32, i32, i32, vp, i32,
                             vp, i64, i64, i32, vp, i64, i64, vp],
        "kvq_paged_gather": [vp, i32, vp, i32, i32, i32, i32, vp, i64, i64, vp, i64, i64, vp],
        "kvq_paged_attention_workspace": [i32, i32, i32, i32, i32, ctypes.POINTER(ctypes.c_size_t)],
        "kvq_paged_attention": [i32, vp, i64, i64, vp, i32, vp, i64, i32, vp, i32, i32, i32, i32, i32, i32, f32,
                                vp, vp, vp, ctypes.c_size_t, vp],
    }
    for name, argt in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = argt
        fn.restype = ctypes.c_int
    lib.kvq_last_error.argtypes = []
    lib.kvq_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int):
    if status != KVQ_OK:
        raise KvqError(status, load_library().kvq_last_error().decode())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, shape=None, nbytes=None):
    """Check a tensor argument before its pointer crosses the C ABI (which sees only the
    address): contiguous, of `dtype`, and of `shape` or `nbytes` when given."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if nbytes is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} must hold at least {nbytes} bytes")


def _stream(stream) -> int | None:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream or None
    return getattr(stream, "cuda_stream", stream) or None


def certificates(raw) -> np.ndarray:
    """View a raw certificate buffer (torch uint8 tensor or bytes) as a structured array."""
    import torch
    if isinstance(raw, torch.Tensor):
        raw = raw.detach().cpu().numpy()
    return np.frombuffer(np.ascontiguousarray(raw).tobytes(), dtype=CERT_DTYPE)


class Cache:
    """A tiered certified KV cache for `n_layers` layers (kvq_cache_create)."""

    def __init__(self, n_layers, batch, n_q_heads, n_kv_heads, max_ctx, rank_positions=1,
                 l4_head_fraction=0.5, head_dim=HEAD_DIM, block_tokens=BLOCK,
                 value_group=VALUE_GROUP, value_bits=4, v_tol=0.0, resident_blocks=0):
        self.lib = load_library()
        self.cfg = kvq_config(n_layers, batch, n_q_heads, n_kv_heads, head_dim, block_tokens,
                              value_group, max_ctx, rank_positions, l4_head_fraction, value_bits,
                              v_tol, resident_blocks)
        self.value_bits = value_bits
        h = ctypes.c_void_p()
        _check(self.lib.kvq_cache_create(ctypes.byref(self.cfg), ctypes.byref(h)))
        self.handle = h
        self.batch, self.n_q_heads, self.n_kv_heads = batch, n_q_heads, n_kv_heads

    def close(self):
        if getattr(self, "handle", None):
            self.lib.kvq_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_debug(self, flags: int):
        _check(self.lib.kvq_set_debug(self.handle, flags))

    def length(self, layer: int) -> int:
        n = ctypes.c_int()
        _check(self.lib.kvq_cache_length(self.handle, layer, ctypes.byref(n)))
        return n.value

    def append(self, layer: int, k, v, stream=None):
        """k, v: contiguous fp16 CUDA tensors [B, Hkv, n, 128]."""
        import torch
        if k.dim() != 4:
            raise ValueError("k must be [batch, n_kv_heads, n_tokens, 128]")
        shape = (self.batch, self.n_kv_heads, k.shape[2], HEAD_DIM)
        _need(k, "k", torch.float16, shape)
        _need(v, "v", torch.float16, shape)
        _check(self.lib.kvq_append(self.handle, layer, _ptr(k), _ptr(v), k.shape[2], _stream(stream)))

    def decode(self, layer: int, q, tau_cov: float, eps: float, out, cert=None, ladder_level=None,
               stream=None):
        """q, out: contiguous fp16 tensors [B, Hq, 128] (device or host); cert: uint8 tensor
        of B*Hq*32 bytes or None; ladder_level: int32 tensor [B] or None.  Pinned host
        tensors are copied in stream order (read the results after a synchronize);
        pageable host tensors make the call wait for its copies."""
        self._check_decode_args(q, out, cert)
        if ladder_level is not None:
            import torch
            _need(ladder_level, "ladder_level", torch.int32, (self.batch,))
        st = _stream(stream) if (q.is_cuda or out.is_cuda) else None
        _check(self.lib.kvq_decode_attention(self.handle, layer, _ptr(q), float(tau_cov), float(eps),
                                             _ptr(out), _ptr(cert), _ptr(ladder_level), st))

    def decode_uncertified(self, layer: int, q, out, cert=None, stream=None):
        """Plain INT8/INT4 decode attention, nothing paged in and no ladder
        (kvq_decode_attention_uncertified); cert receives the unenforced bounds."""
        self._check_decode_args(q, out, cert)
        st = _stream(stream) if (q.is_cuda or out.is_cuda) else None
        _check(self.lib.kvq_decode_attention_uncertified(self.handle, layer, _ptr(q), _ptr(out),
                                                         _ptr(cert), st))

    def _check_decode_args(self, q, out, cert):
        import torch
        shape = (self.batch, self.n_q_heads, HEAD_DIM)
        _need(q, "q", torch.float16, shape)
        _need(out, "out", torch.float16, shape)
        if cert is not None:
            _need(cert, "cert", torch.uint8, nbytes=self.batch * self.n_q_heads * CERT_DTYPE.itemsize)

    def export_tier1(self, layer: int, stream=None) -> dict:
        """Tier-1 contents of `layer` in canonical layout, as CUDA tensors."""
        import torch
        B, H, n = self.batch, self.n_kv_heads, self.length(layer)
        nb = n // BLOCK
        dev = torch.device("cuda")
        out = dict(
            kc=torch.empty(B, H, nb, BLOCK, HEAD_DIM, dtype=torch.int8, device=dev),
            ks=torch.empty(B, H, nb, HEAD_DIM, dtype=torch.float16, device=dev),
            vc=torch.empty(B, H, nb, BLOCK, HEAD_DIM, dtype=torch.uint8, device=dev),
            vs=torch.empty(B, H, nb, BLOCK, HEAD_DIM // VALUE_GROUP, dtype=torch.float16, device=dev),
            vo=torch.empty(B, H, nb, BLOCK, HEAD_DIM // VALUE_GROUP, dtype=torch.float16, device=dev),
            eta=torch.empty(B, H, nb, dtype=torch.float32, device=dev),
            vmin=torch.empty(B, H, HEAD_DIM, dtype=torch.float32, device=dev),
            vmax=torch.empty(B, H, HEAD_DIM, dtype=torch.float32, device=dev),
        )
        o = out
        _check(self.lib.kvq_export_tier1(self.handle, layer, _ptr(o["kc"]), _ptr(o["ks"]), _ptr(o["vc"]),
                                         _ptr(o["vs"]), _ptr(o["vo"]), _ptr(o["eta"]), _ptr(o["vmin"]),
                                         _ptr(o["vmax"]), _stream(stream)))
        return out

    def export_decode_state(self, nb: int, stream=None) -> dict:
        """Selection state of the last certified decode call (nb = its full blocks)."""
        import torch
        B, Hq, H = self.batch, self.n_q_heads, self.n_kv_heads
        dev = torch.device("cuda")
        o = dict(
            sel=torch.zeros(B, Hq, nb, dtype=torch.uint8, device=dev),
            kprom0=torch.zeros(B, H, nb, dtype=torch.uint8, device=dev),
            kprom1=torch.zeros(B, H, nb, dtype=torch.uint8, device=dev),
            vprom1=torch.zeros(B, H, nb, dtype=torch.uint8, device=dev),
            lse8=torch.zeros(B, Hq, nb, dtype=torch.float32, device=dev),
            delta=torch.zeros(B, Hq, nb, dtype=torch.float32, device=dev),
        )
        _check(self.lib.kvq_export_decode_state(self.handle, _ptr(o["sel"]), _ptr(o["kprom0"]),
                                                _ptr(o["kprom1"]), _ptr(o["vprom1"]), _ptr(o["lse8"]),
                                                _ptr(o["delta"]), _stream(stream)))
        return o

    def residency_stats(self, layer: int, reset: bool = False) -> dict:
        """FP16 block bytes of `layer` served from resident HBM copies and read over the
        host link since the last reset, and the slots in use (kvq_residency_stats)."""
        hit, host, used = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int()
        _check(self.lib.kvq_residency_stats(self.handle, layer, ctypes.byref(hit), ctypes.byref(host),
                                            ctypes.byref(used), int(reset)))
        return {"resident_bytes": hit.value, "host_bytes": host.value, "slots_in_use": used.value}

    def debug_fill_tier2(self, layer: int, bits: int):
        """Test aid (kvq_debug_fill_tier2): overwrite `layer`'s tier-2 FP16 originals with
        the binary16 bit pattern `bits`, after the device has finished queued work."""
        _check(self.lib.kvq_debug_fill_tier2(self.handle, layer, int(bits) & 0xFFFF))

    def profile_read(self, reset: bool = True) -> dict:
        arr = (kvq_kernel_stat * 16)()
        n = ctypes.c_int()
        _check(self.lib.kvq_profile_read(self.handle, arr, 16, ctypes.byref(n), int(reset)))
        return {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms) for i in range(n.value)}


def dense_decode_noalloc(q, k, v, out, stream=None):
    """Exact dense FP16 decode attention with no allocation (kvq_dense_decode_noalloc).

    For callers that cannot allocate device memory at call time; q, out: device fp16
    [B, Hq, 128]; k, v: device fp16 [B, Hkv, n_tokens, 128].  Its scratch is a fixed
    8 MiB device array shared by every call, so overlapping calls must be serialised.
    """
    import torch
    if q.dim() != 3 or k.dim() != 4:
        raise ValueError("q must be [batch, n_q_heads, 128] and k, v [batch, n_kv_heads, n_tokens, 128]")
    B, Hq, _ = q.shape
    Hkv, N = k.shape[1], k.shape[2]
    _need(q, "q", torch.float16, (B, Hq, HEAD_DIM))
    _need(k, "k", torch.float16, (B, Hkv, N, HEAD_DIM))
    _need(v, "v", torch.float16, (B, Hkv, N, HEAD_DIM))
    _need(out, "out", torch.float16, (B, Hq, HEAD_DIM))
    dev = q.device
    if any(t.device != dev for t in (k, v, out)):
        raise ValueError("q, k, v and out must be on one CUDA device")
    if dev.type == "cuda":
        with torch.cuda.device(dev):   # the call runs on the tensors' device and its stream
            _check(load_library().kvq_dense_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), B, Hq, Hkv, N,
                                                           _ptr(out), _stream(stream)))
        return
    _check(load_library().kvq_dense_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), B, Hq, Hkv, N,
                                                   _ptr(out), _stream(stream)))


def dense_attention_workspace(batch: int, n_q_heads: int, n_kv_heads: int, n_tokens: int) -> int:
    """Workspace bytes kvq_dense_attention needs for this shape on the current device."""
    n = ctypes.c_size_t(0)
    _check(load_library().kvq_dense_attention_workspace(batch, n_q_heads, n_kv_heads, n_tokens, ctypes.byref(n)))
    return int(n.value)


def dense_attention(q, k, v, out, workspace=None, stream=None):
    """Exact dense FP16 decode attention over K/V in device memory (kvq_dense_attention).

    q, out: device fp16 [B, Hq, 128]; k, v: device fp16 [B, Hkv, n_tokens, 128].
    `workspace` is a device uint8 tensor of at least dense_attention_workspace(...) bytes
    (allocated here when omitted).  Returns `workspace` so a caller can reuse it.
    """
    import torch
    if q.dim() != 3 or k.dim() != 4:
        raise ValueError("q must be [batch, n_q_heads, 128] and k, v [batch, n_kv_heads, n_tokens, 128]")
    B, Hq, _ = q.shape
    Hkv, N = k.shape[1], k.shape[2]
    _need(q, "q", torch.float16, (B, Hq, HEAD_DIM))
    _need(k, "k", torch.float16, (B, Hkv, N, HEAD_DIM))
    _need(v, "v", torch.float16, (B, Hkv, N, HEAD_DIM))
    _need(out, "out", torch.float16, (B, Hq, HEAD_DIM))
    dev = q.device
    if dev.type != "cuda" or any(t.device != dev for t in (k, v, out)):
        raise ValueError("q, k, v and out must be on one CUDA device")
    with torch.cuda.device(dev):
        need = dense_attention_workspace(B, Hq, Hkv, N)
        if workspace is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        _need(workspace, "workspace", torch.uint8, nbytes=need)
        _check(load_library().kvq_dense_attention(_ptr(q), _ptr(k), _ptr(v), B, Hq, Hkv, N, _ptr(out),
                                                  _ptr(workspace), workspace.numel(), _stream(stream)))
    return workspace


# ---- rotary positions and the paged 4-bit cache ----

PAGE = 64   # tokens per page
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3, "yarn": 4}


class RopePlan:
    """Rotary frequencies of a model, for `rope` and `paged_append` (kvq_rope_plan_init).

    layout: "half" pairs elements (i, i + rotary_dim / 2), "interleaved" (2i, 2i + 1).
    scaling: "none", "linear", "ntk", "parts" (frequencies blended by their turns within
    original_ctx, between low and high) or "yarn" (blended over the pair index, cos and sin
    times 0.1 ln(factor) + 1 unless `magnitude` is given); see include/kvq.h.
    """

    def __init__(self, head_dim, rotary_dim=None, layout="half", base=10000.0, scaling="none", factor=1.0,
                 original_ctx=0, low=1.0, high=32.0, magnitude=0.0):
        if layout not in ("half", "interleaved"):
            raise ValueError('layout must be "half" or "interleaved"')
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
        cfg = kvq_rope_config(head_dim, head_dim if rotary_dim is None else rotary_dim, int(layout == "interleaved"),
                              ROPE_SCALINGS[scaling], base, factor, original_ctx, low, high, magnitude)
        self.plan = kvq_rope_plan()
        _check(load_library().kvq_rope_plan_init(ctypes.byref(cfg), ctypes.byref(self.plan)))
        self.address = ctypes.addressof(self.plan)
        self.head_dim = head_dim

    # copies and pickled plans hold a struct of their own, at their own address
    def __getstate__(self):
        return {**self.__dict__, "plan": bytes(self.plan), "address": None}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self.plan = kvq_rope_plan.from_buffer_copy(state["plan"])
        self.address = ctypes.addressof(self.plan)


# The calls below are made once per layer and token, where their host time counts (a decoding
# step of a few microseconds on the device): operands are checked with as few attribute reads
# as that takes, and what they need of torch is looked up once.

_torch = None


def _lookup():
    global _torch, _F16, _BF16, _I32, _raw_stream, _current_device
    import torch
    _F16, _BF16, _I32 = torch.float16, torch.bfloat16, torch.int32
    # the address alone: building a Stream object costs 2.7 us
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch
    return torch


def _rows(t, name, dtype, shape):
    """Address and (token, head) strides of a [tokens, heads, head_dim] operand whose rows
    are contiguous."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    a, b, c = t.stride()
    T, H, D = shape
    if c != 1 and D != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # a dimension of one row has no stride to speak of
    return t.data_ptr(), a if T > 1 else 8, b if H > 1 else 8


def _ints(t, name, n, dev):
    if t.dtype is not _I32 or t.shape != (n,) or t.get_device() != dev or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous torch.int32 tensor of {n} elements on CUDA device {dev}")
    return t.data_ptr()


def _float_code(t, name) -> int:
    dt = t.dtype
    if dt is _F16:
        return 0
    if dt is _BF16:
        return 1
    raise ValueError(f"{name} must be torch.float16 or torch.bfloat16, got {dt}")


def _device_of(t, name) -> int:
    """Index of the CUDA device that a call runs on: the one of its first tensor.  The library
    refuses buffers that are not on it."""
    if _torch is None:
        _lookup()
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _call(dev, stream, fn, *args):
    """Run a library call on device `dev` and `stream` (the device's current one when None)."""
    stream = _raw_stream(dev) if stream is None else getattr(stream, "cuda_stream", stream)
    if dev == _current_device():
        status = fn(*args, stream or None)
    else:
        with _torch.cuda.device(dev):
            status = fn(*args, stream or None)
    if status != KVQ_OK:
        _check(status)


def rope(x, positions, plan, out=None, stream=None):
    """Rotary positions (kvq_rope): x [T, H, head_dim] fp16 or bf16 with contiguous rows (any
    token and head strides, e.g. a slice of a fused projection), positions [T] int32.
    out=None allocates the result; out=x works in place.  Returns out."""
    shape = x.shape
    if len(shape) != 3:
        raise ValueError("x must be [n_tokens, n_heads, head_dim]")
    if out is None:
        if stream is not None:
            raise ValueError("out must be given with a stream")
        out = (_torch or _lookup()).empty(shape, dtype=x.dtype, device=x.device)
    dev = _device_of(x, "x")
    code, dt = _float_code(x, "x"), x.dtype
    T, H, hd = shape
    if hd != plan.head_dim:
        raise ValueError(f"x must have head_dim {plan.head_dim}, got {hd}")
    a = _rows(x, "x", dt, shape)
    b = a if out is x else _rows(out, "out", dt, shape)
    _call(dev, stream, load_library().kvq_rope, plan.address, code, *a, _ints(positions, "positions", T, dev), T, H, *b)
    return out


def paged_page_bytes(head_dim: int = HEAD_DIM) -> int:
    """Bytes of one page of one KV head: a pool of pages is a contiguous CUDA uint8 tensor
    [n_pages, n_kv_heads, paged_page_bytes(head_dim)] (its initial contents do not matter)."""
    n = ctypes.c_size_t(0)
    _check(load_library().kvq_paged_page_bytes(head_dim, ctypes.byref(n)))
    return int(n.value)


_PAGE_BYTES = {64: 5120, 128: 10240}


def _pool(pages, n_kv_heads, head_dim):
    """Address and page count of a pool of pages."""
    nbytes = _PAGE_BYTES.get(head_dim)
    if nbytes is None:
        raise ValueError("head_dim must be 64 or 128")
    shape = pages.shape
    if pages.dtype is not _torch.uint8 or len(shape) != 3 or shape[1] != n_kv_heads or shape[2] != nbytes \
            or not pages.is_contiguous():
        raise ValueError(f"pages must be a contiguous uint8 tensor [n_pages, {n_kv_heads}, {nbytes}]")
    return pages.data_ptr(), shape[0]


def paged_append(pages, k, v, slots, positions=None, plan=None, q=None, q_out=None, stream=None):
    """Write tokens into a pool of pages in 4 bits (kvq_paged_append).

    k, v: [T, n_kv_heads, head_dim] fp16 or bf16 with contiguous rows; slots: int32 [T] (page *
    64 + offset; outside the pool, e.g. -1: skipped; all distinct).  With a RopePlan and
    positions (int32 [T]) keys are rotated on the way, and q [T, n_q_heads, head_dim], when
    given, into q_out (which may be q)."""
    shape = k.shape
    if len(shape) != 3:
        raise ValueError("k must be [n_tokens, n_kv_heads, head_dim]")
    dev = _device_of(k, "k")
    code, dt = _float_code(k, "k"), k.dtype
    T, hkv, hd = shape
    if (plan is None) != (positions is None):
        raise ValueError("plan and positions go together")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    hq, qa, oa = 0, (None, 0, 0), (None, 0, 0)
    if q is not None:
        qs = q.shape
        if len(qs) != 3:
            raise ValueError("q must be [n_tokens, n_q_heads, head_dim]")
        hq = qs[1]
        qa = _rows(q, "q", dt, (T, hq, hd))
        oa = qa if q_out is q else _rows(q_out, "q_out", dt, (T, hq, hd))
    _call(dev, stream, load_library().kvq_paged_append, None if plan is None else plan.address, code,
          *_rows(k, "k", dt, shape), *_rows(v, "v", dt, shape), _ints(slots, "slots", T, dev),
          None if positions is None else _ints(positions, "positions", T, dev), T, hkv, hd, *_pool(pages, hkv, hd),
          *qa, hq, *oa)


def paged_gather(pages, slots, k, v, stream=None):
    """Read tokens back from a pool of pages (kvq_paged_gather): k, v [T, n_kv_heads, head_dim]
    fp16 or bf16 receive what the slots hold (rows of slots outside the pool become 0)."""
    shape = k.shape
    if len(shape) != 3:
        raise ValueError("k must be [n_tokens, n_kv_heads, head_dim]")
    dev = _device_of(pages, "pages")
    code, dt = _float_code(k, "k"), k.dtype
    T, hkv, hd = shape
    _call(dev, stream, load_library().kvq_paged_gather, *_pool(pages, hkv, hd), _ints(slots, "slots", T, dev), T, hkv, hd,
          code, *_rows(k, "k", dt, shape), *_rows(v, "v", dt, shape))


def paged_attention_workspace(batch: int, n_q_tokens: int, n_q_heads: int, n_kv_heads: int,
                              head_dim: int = HEAD_DIM) -> int:
    """Workspace bytes kvq_paged_attention needs for this shape on the current device."""
    n = ctypes.c_size_t(0)
    _check(load_library().kvq_paged_attention_workspace(batch, n_q_tokens, n_q_heads, n_kv_heads, head_dim,
                                                        ctypes.byref(n)))
    return int(n.value)


def paged_attention(q, pages, page_table, seq_lens, out, lse=None, scale=None, window=0, workspace=None, stream=None):
    """Decode attention over a pool of 4-bit pages (kvq_paged_attention).

    q: [B, Hq, head_dim] or [B, n_q_tokens, Hq, head_dim] fp16 or bf16, the last tokens of each
    sequence; page_table: int32 [B, max_pages]; seq_lens: int32 [B], those tokens included (0:
    a padding sequence, whose out is 0); out: like q, contiguous; lse: float32 like q without
    its last dimension, or None; scale: None (or 0) for 1 / sqrt(head_dim).  `workspace` is a
    device uint8 tensor of at least paged_attention_workspace(...) bytes, zeroed once before its
    first use (allocated here when omitted).  Returns `workspace` so a caller can reuse it."""
    shape = q.shape
    if len(shape) not in (3, 4):
        raise ValueError("q must be [batch, n_q_heads, head_dim] or [batch, n_q_tokens, n_q_heads, head_dim]")
    dev = _device_of(q, "q")
    code, st, dt = _float_code(q, "q"), q.stride(), q.dtype
    B, hq, hd = shape[0], shape[-2], shape[-1]
    Q = shape[1] if len(shape) == 4 else 1
    if st[-1] != 1:
        raise ValueError("q: the last dimension must be contiguous")
    qt = st[1] if Q > 1 else st[0] if B > 1 else 8
    if Q > 1 and B > 1 and st[0] != Q * st[1]:
        raise ValueError("q: the query tokens must be evenly spaced in memory")
    pool = pages.shape
    if len(pool) != 3:
        raise ValueError("pages must be [n_pages, n_kv_heads, page bytes]")
    hkv = pool[1]
    pool = _pool(pages, hkv, hd)
    if out.dtype is not dt or out.shape != shape or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's shape and type")
    if lse is not None and (lse.dtype is not _torch.float32 or lse.shape != shape[:-1] or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32, of q's shape without the last dimension")
    ts = page_table.stride()
    if page_table.dtype is not _I32 or len(ts) != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table must be int32 [{B}, max_pages]")
    max_pages = page_table.shape[1]
    if ts[1] != 1 and max_pages > 1:
        raise ValueError("page_table: the last dimension must be contiguous")
    lens = _ints(seq_lens, "seq_lens", B, dev)
    if workspace is None:
        torch = _torch
        with torch.cuda.device(dev):
            workspace = torch.zeros(paged_attention_workspace(B, Q, hq, hkv, hd), dtype=torch.uint8, device=q.device)
            if stream is not None:
                # zeroed on the current stream and used on the other one
                other = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
                other.wait_stream(torch.cuda.current_stream())
                workspace.record_stream(other)
    elif workspace.dtype is not _torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    _call(dev, stream, load_library().kvq_paged_attention, code, q.data_ptr(), qt, st[-2] if hq > 1 else 8, *pool,
          page_table.data_ptr(), ts[0] if B > 1 else max_pages, max_pages, lens, B, Q, hq, hkv, hd, window,
          0.0 if scale is None else float(scale), out.data_ptr(), None if lse is None else lse.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return workspace


def header_functions(header_path: str | None = None) -> list[str]:
    """Names of the functions declared in include/kvq.h."""
    import re
    path = header_path or os.path.join(os.path.dirname(_HERE), "include", "kvq.h")
    text = open(path).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_]+\s*\*?\s*(kvq_[a-z0-9_]+)\s*\(", text, re.M)))
