"""ctypes binding of the C ABI in include/fa_attention.h -- argument marshalling only.

Every step of the computation runs in the CUDA kernels of ``libfa_attention.so``;
this module turns torch tensors into pointers, sizes and the current stream,
and turns status codes into exceptions.  There is no fallback: if the library
is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfa_attention.so")

FA_OK = 0
STATUS = {
    0: "FA_OK",
    1: "FA_ERR_INVALID_ARG",
    2: "FA_ERR_UNSUPPORTED",
    3: "FA_ERR_MISALIGNED",
    4: "FA_ERR_WORKSPACE",
    5: "FA_ERR_CUDA",
    6: "FA_ERR_DEVICE_TIMEOUT",
    7: "FA_ERR_DEVICE_CHECK",
}
FA_FP16, FA_BF16 = 0, 1

# Every symbol the header declares, with (restype, argtypes).
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "fa_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _vp]),
    "fa_fwd_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _i, _vp]),
    "fa_bwd_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fa_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i, _i, _i, _i, _f, _i, _i, _vp]),
    "fa_bwd_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i, _i, _i, _i, _i, _i, _f, _i, _i,
                       _vp]),
    "fa_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _vp]),
    "fa_fwd_rule_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "fa_bwd_rule_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "fa_fwd_rule": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "fa_bwd_rule": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i, _i, _i, _i, _i, _i, _f, _i,
                         _vp]),
    "fa_kv4_append": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _i, _vp]),
    "fa_kv4_read": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _vp]),
    "fa_kv4_attend_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "fa_kv4_attend": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _vp, _i, _f, _vp, _vp, _sz, _i, _i, _i, _f, _vp]),
    "fa_kv4_attend_tree_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "fa_kv4_attend_tree": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _sz, _i, _i, _i, _f, _vp]),
    "fa_kv4_tree_many_rows": (_i, [_i, _i, _i, _i, _i, ctypes.c_longlong, _i]),
    "fa_kv4_keep": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _i, _i, _vp]),
    "fa_kv4_plan": (_i, [_vp, _vp, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _vp]),
    "fa_rotary": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _f, _i, _i, _i, _i, _i, _i, _vp]),
    "fa_rotary_turns": (ctypes.c_uint64, [ctypes.c_double]),
    "fa_kv4_row": (ctypes.c_longlong, [ctypes.POINTER(ctypes.c_int32), _i, _i, _i, ctypes.c_longlong]),
    "fa_host_scratch_size": (_sz, [_i, _i, _i, _i, _i]),
    "fa_host_chunk_plan": (_i, [_i, _i, _i, _i, ctypes.POINTER(ctypes.c_int), _i]),
    "fa_cta_head_group": (_i, [ctypes.c_longlong, _i, _sz, _i, _i]),
    "fa_fwd_host": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _sz, _i, _i, _i, _i, _f, _i, _i, _i, _vp]),
    "fa_fwd_bwd_host": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i, _i, _i, _i, _f, _i, _i, _i,
                             _vp]),
    "fa_check_device_status": (_i, [_vp]),
    "fa_selftest_wait_timeout": (_i, [ctypes.c_uint32, _vp]),
    "fa_selftest_device_check": (_i, [_i, _vp]),
    "fa_last_device_error_bits": (ctypes.c_uint32, []),
    "fa_last_device_error_detail": (None, [_vp]),
    "fa_status_string": (ctypes.c_char_p, [_i]),
    "fa_profile_begin": (_i, [_i]),
    "fa_profile_end": (_i, [_vp, _vp, _i]),
    "fa_version": (ctypes.c_uint32, []),
}


class FaError(RuntimeError):
    def __init__(self, where: str, code: int, detail=None):
        extra = f" (device record {detail})" if detail else ""
        super().__init__(f"{where} failed: {STATUS.get(code, code)}{extra}")
        self.code = code
        self.detail = detail


_lib = None


def open_library(path: str):
    """Open a build of the library at ``path`` and declare its signatures (no caching)."""
    if not os.path.exists(path):
        raise FaError(f"loading {os.path.basename(path)} (not built; run exact_attention_37_gb300.build)", -1)
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load(path: str = LIB_PATH):
    """Load the shared library (once) and declare its signatures.  Raises if it is missing."""
    global _lib
    if _lib is None:
        _lib = open_library(path)
    return _lib


_native = None
_NATIVE_CALLS = ("fa_fwd_rule_workspace_size", "fa_bwd_rule_workspace_size", "fa_fwd_rule", "fa_bwd_rule", "fa_kv4_append",
                 "fa_kv4_read", "fa_kv4_attend_workspace_size", "fa_kv4_attend", "fa_kv4_attend_tree_workspace_size",
                 "fa_kv4_attend_tree", "fa_kv4_keep", "fa_kv4_plan", "fa_rotary")


def native():
    """The binding's native module (csrc/binding.cpp), bound to the loaded library: the same marshalling
    as here for the calls that are made every few microseconds.  Raises if it is missing."""
    global _native
    if _native is None:
        import torch  # noqa: F401  (its libraries are the module's)

        try:
            from . import _native as module
        except ImportError as e:
            raise FaError(f"loading _native.so (not built; run exact_attention_37_gb300.build): {e}", -1) from e
        lib = load()
        module.bind(*[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _NATIVE_CALLS])
        _native = module
    return _native


def _check(where: str, code: int):
    if code != FA_OK:
        raise FaError(where, code)


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.float16:
        return FA_FP16
    if t.dtype == torch.bfloat16:
        return FA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: fp16 or bf16 only")


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _shape(q):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    return tuple(int(x) for x in q.shape)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _check_shapes(q, k, v):
    B, H, Nq, d = _shape(q)
    Bk, Hkv, Nk, dk = _shape(k)
    if tuple(v.shape) != tuple(k.shape) or Bk != B or dk != d:
        raise ValueError("k and v must be [B, H_kv, N_k, d] with q's B and d")
    if Hkv < 1 or H % Hkv:
        raise ValueError("the key/value head count must divide the query head count")
    return B, H, Hkv, Nq, Nk, d


def fa_fwd(q, k, v, o, lse, scale: float, causal: bool, stream=None):
    """O and L into caller-owned ``o`` [B,H,N_q,d] and ``lse`` [B,H,N_q] fp32 (all CUDA, contiguous).

    k, v: [B, H_kv, N_k, d] (H_kv divides H; N_k may differ from N_q)."""
    lib = load()
    B, H, Hkv, Nq, Nk, d = _check_shapes(q, k, v)
    for t in (q, k, v, o, lse):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    code = lib.fa_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, Nq, Nk, d, float(scale),
                         int(bool(causal)), _dtype_code(q), _stream(stream))
    _check("fa_fwd_ex", code)


def fa_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_size(B, H, N, d))


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale: float, causal: bool, stream=None):
    """dQ, dK, dV into caller-owned tensors; ``workspace`` is a CUDA uint8 tensor of at least
    fa_bwd_workspace_size(B, H, N_q, d) bytes."""
    lib = load()
    B, H, Hkv, Nq, Nk, d = _check_shapes(q, k, v)
    for t in (q, k, v, o, dout, lse, dq, dk, dv):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    code = lib.fa_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                         _ptr(workspace), ws_bytes, B, H, Hkv, Nq, Nk, d, float(scale), int(bool(causal)),
                         _dtype_code(q), _stream(stream))
    _check("fa_bwd_ex", code)


def fa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, scale: float, causal: bool, stream=None):
    """fa_bwd with the library's fixed device scratch instead of a caller workspace (no allocation)."""
    lib = load()
    B, H, N, d = _shape(q)
    for t in (q, k, v, o, dout, lse, dq, dk, dv):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    code = lib.fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                              _ptr(dv), B, H, N, d, float(scale), int(bool(causal)), _dtype_code(q), _stream(stream))
    _check("fa_bwd_noalloc", code)


class ScoreRuleStruct(ctypes.Structure):
    """fa_score_rule of the header."""

    _fields_ = [("causal", _i), ("cap", _f), ("slopes", _vp), ("q_doc", _vp), ("k_doc", _vp), ("prefix", _vp)]


@dataclasses.dataclass
class ScoreRule:
    """What happens to a score between Q K^T and the softmax, and which keys a query sees.

    With u = scale q_i.k_j and the query's position p = i + N_k - N_q:
    z = cap tanh(u / cap) (u for cap 0), y = z - slopes[h] |p - j|.  Key j is visible when
    its document id equals the query's and is not negative (with ids), and, under the
    causal mask, j <= p or j < prefix[b].

    slopes: fp32 [H]; q_doc [B, N_q] and k_doc [B, N_k]: int32, both or neither; prefix:
    int32 [B].  All on the inputs' device, contiguous.  A negative id marks padding."""

    causal: bool = False
    cap: float = 0.0
    slopes: object = None
    q_doc: object = None
    k_doc: object = None
    prefix: object = None

    def struct(self, dev: int, B: int, H: int, Nq: int, Nk: int):
        """The C struct after checks of types, shapes and devices."""
        import torch

        slopes, q_doc, k_doc, prefix = self.slopes, self.q_doc, self.k_doc, self.prefix
        if slopes is not None:
            _check_array(slopes, torch.float32, (H,), dev, "slopes")
        if (q_doc is None) != (k_doc is None):
            raise ValueError("q_doc and k_doc go together")
        if q_doc is not None:
            _check_array(q_doc, torch.int32, (B, Nq), dev, "q_doc")
            _check_array(k_doc, torch.int32, (B, Nk), dev, "k_doc")
        if prefix is not None:
            _check_array(prefix, torch.int32, (B,), dev, "prefix")
        return ScoreRuleStruct(1 if self.causal else 0, self.cap, _addr(slopes), _addr(q_doc), _addr(k_doc), _addr(prefix))


def _addr(t):
    return None if t is None else t.data_ptr()


def _check_array(t, dtype, shape, dev: int, name: str):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")


def _device_of(t) -> int:
    """Index of the CUDA device that t is on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    return dev


class _Device:
    """Makes a device (by index) current for a call; does nothing when it is."""

    __slots__ = ("guard",)

    def __init__(self, dev: int):
        import torch

        self.guard = None if torch._C._cuda_getDevice() == dev else torch.cuda.device(dev)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *e):
        if self.guard is not None:
            self.guard.__exit__(*e)


def _raw_stream(stream, dev: int):
    """The stream's handle: the one given, which has to be the device's, or its current one."""
    import torch

    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream must be one of cuda:{dev}")
    return stream.cuda_stream


def _ws_bytes(workspace, dev: int) -> int:
    if workspace is None:
        return 0
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on cuda:{dev}")
    return workspace.numel() * workspace.element_size()


def _rule_sizes(q, k, v):
    """(B, H, H_kv, N_q, N_k, d, dtype code, device index) of a call's inputs, checked."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    B, H, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if v.shape != k.shape or Bk != B or dk != d:
        raise ValueError("k and v must be [B, H_kv, N_k, d] with q's B and d")
    if Hkv < 1 or H % Hkv:
        raise ValueError("the key/value head count must divide the query head count")
    t, dev = q.dtype, _device_of(q)
    if k.dtype is not t or v.dtype is not t or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k and v must have one type and be on one device")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("tensors must be contiguous")
    return B, H, Hkv, Nq, Nk, d, _dtype_code(q), dev


def fa_fwd_rule_workspace_size(B: int, H: int, N_q: int, N_k: int, d: int, docs: bool) -> int:
    return load().fa_fwd_rule_workspace_size(B, H, N_q, N_k, d, 1 if docs else 0)


def fa_bwd_rule_workspace_size(B: int, H: int, N_q: int, N_k: int, d: int, docs: bool) -> int:
    return load().fa_bwd_rule_workspace_size(B, H, N_q, N_k, d, 1 if docs else 0)


def fa_fwd_rule(q, k, v, o, lse, rule: ScoreRule, workspace, scale: float, stream=None):
    """fa_fwd with a score rule; ``workspace``: CUDA uint8 of at least
    fa_fwd_rule_workspace_size(...) bytes (None where that is 0)."""
    import torch

    sizes = _rule_sizes(q, k, v)
    _check_array(o, q.dtype, q.shape, sizes[7], "o")
    _check_array(lse, torch.float32, q.shape[:3], sizes[7], "lse")
    B, H, Hkv, Nq, Nk, d, code, dev = sizes
    r = rule.struct(dev, B, H, Nq, Nk)
    with _Device(dev):
        st = load().fa_fwd_rule(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), ctypes.addressof(r),
                                _addr(workspace), _ws_bytes(workspace, dev), B, H, Hkv, Nq, Nk, d, scale, code,
                                _raw_stream(stream, dev))
    _check("fa_fwd_rule", st)


def fa_bwd_rule(q, k, v, o, dout, lse, dq, dk, dv, rule: ScoreRule, workspace, scale: float, stream=None):
    """fa_bwd with a score rule; ``workspace``: CUDA uint8 of at least
    fa_bwd_rule_workspace_size(...) bytes."""
    import torch

    sizes = _rule_sizes(q, k, v)
    for t, like, what in ((dq, q, "dq"), (dk, k, "dk"), (dv, k, "dv")):
        _check_array(t, q.dtype, like.shape, sizes[7], what)
    B, H, Hkv, Nq, Nk, d, code, dev = sizes
    _check_array(o, q.dtype, q.shape, dev, "o")
    _check_array(dout, q.dtype, q.shape, dev, "dout")
    _check_array(lse, torch.float32, q.shape[:3], dev, "lse")
    r = rule.struct(dev, B, H, Nq, Nk)
    with _Device(dev):
        st = load().fa_bwd_rule(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
                                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ctypes.addressof(r), _addr(workspace),
                                _ws_bytes(workspace, dev), B, H, Hkv, Nq, Nk, d, scale, code, _raw_stream(stream, dev))
    _check("fa_bwd_rule", st)


class KV4CacheStruct(ctypes.Structure):
    """fa_kv4_cache of the header."""

    _fields_ = [("k_codes", _vp), ("k_params", _vp), ("v_codes", _vp), ("v_params", _vp), ("num_pages", _i),
                ("page_size", _i), ("H_kv", _i), ("d", _i), ("dtype", _i)]


KV4_GROUP = 32  # channels that share a scale and a low value


class KV4Cache:
    """Pools of a paged 4-bit key/value cache: codes [pages, H_kv, page_size, d / 2] uint8 and
    params [pages, H_kv, page_size, d / 32, 2] fp16 or bf16 (scale, low), keys and values.
    Channel c of a row stands for T(low + scale * code); byte i holds channel 2 i low."""

    def __init__(self, k_codes, k_params, v_codes, v_params):
        self.pools = (k_codes, k_params, v_codes, v_params)
        self.num_pages, self.H_kv, self.page_size, self.d, self.dtype_code, self.dev = native().kv4_check(*self.pools)

    k_codes = property(lambda self: self.pools[0])
    k_params = property(lambda self: self.pools[1])
    v_codes = property(lambda self: self.pools[2])
    v_params = property(lambda self: self.pools[3])
    dtype = property(lambda self: self.pools[1].dtype)

    @property
    def device(self):
        return self.k_codes.device

    @classmethod
    def empty(cls, num_pages: int, H_kv: int, page_size: int, d: int, dtype, device="cuda"):
        """Uninitialised pools."""
        import torch

        codes = lambda: torch.empty(num_pages, H_kv, page_size, d // 2, dtype=torch.uint8, device=device)  # noqa: E731
        params = lambda: torch.empty(num_pages, H_kv, page_size, d // KV4_GROUP, 2, dtype=dtype, device=device)  # noqa: E731
        return cls(codes(), params(), codes(), params())

    def struct(self):
        return KV4CacheStruct(self.k_codes.data_ptr(), self.k_params.data_ptr(), self.v_codes.data_ptr(),
                              self.v_params.data_ptr(), self.num_pages, self.page_size, self.H_kv, self.d,
                              self.dtype_code)


def _check_table(cache, page_table, B: int, *ints):
    """max_pages of a [B, max_pages] page table, after checks of it and of [B] int arrays."""
    import torch

    i32, dev = torch.int32, cache.dev
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    n = page_table.shape[1]
    _check_array(page_table, i32, (B, n), dev, "page_table")
    for t in ints:
        if t is None:
            raise ValueError("start and lengths must be given")
        _check_array(t, i32, (B,), dev, "start, count and lengths")
    return n


def fa_kv4_append(cache: KV4Cache, k, v, page_table, start, count=None, stream=None):
    """Rows k, v [B, H_kv, N, d] into the cache as tokens start[b] + i, i < count[b]."""
    if k.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    B, _, N, _ = k.shape
    dev, shape = cache.dev, (B, cache.H_kv, N, cache.d)
    _check_array(k, cache.dtype, shape, dev, "k")
    _check_array(v, cache.dtype, shape, dev, "v")
    n = _check_table(cache, page_table, B, start, *(() if count is None else (count,)))
    c = cache.struct()
    with _Device(dev):
        st = load().fa_kv4_append(ctypes.addressof(c), k.data_ptr(), v.data_ptr(), page_table.data_ptr(), n, start.data_ptr(),
                                  _addr(count), B, N, _raw_stream(stream, dev))
    _check("fa_kv4_append", st)


def fa_kv4_read(cache: KV4Cache, page_table, start, lengths, k, v, stream=None):
    """Values of tokens start[b] + i into k, v [B, H_kv, N, d]; zeros from lengths[b] on."""
    if k.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    shape = (k.shape[0], cache.H_kv, k.shape[2], cache.d)
    _check_array(k, cache.dtype, shape, cache.dev, "k")
    _check_array(v, cache.dtype, shape, cache.dev, "v")
    B, _, N, _ = k.shape
    dev = cache.dev
    n = _check_table(cache, page_table, B, start, lengths)
    c = cache.struct()
    with _Device(dev):
        st = load().fa_kv4_read(ctypes.addressof(c), page_table.data_ptr(), n, start.data_ptr(), lengths.data_ptr(),
                                k.data_ptr(), v.data_ptr(), B, N, _raw_stream(stream, dev))
    _check("fa_kv4_read", st)


def fa_kv4_attend_workspace_size(B: int, H: int, H_kv: int, N_q: int, d: int) -> int:
    return load().fa_kv4_attend_workspace_size(B, H, H_kv, N_q, d)


def fa_kv4_attend(q, cache: KV4Cache, page_table, lengths, o, lse, workspace, scale: float, causal: bool = True,
                  cap: float = 0.0, slopes=None, stream=None):
    """q, o [B, H, N_q, d] over the lengths[b] cached tokens of each sequence; ``workspace``:
    CUDA uint8 of at least fa_kv4_attend_workspace_size(...) bytes."""
    import torch

    _check_array(o, cache.dtype, q.shape, cache.dev, "o")
    _check_array(lse, torch.float32, q.shape[:3], cache.dev, "lse")
    if q.dim() != 4 or q.shape[3] != cache.d or cache.H_kv < 1 or q.shape[1] % cache.H_kv:
        raise ValueError("q must be [B, H, N_q, d] with the cache's d, its head count dividing H")
    B, H, N, _ = q.shape
    dev = cache.dev
    _check_array(q, cache.dtype, q.shape, dev, "q")
    if slopes is not None:
        _check_array(slopes, torch.float32, (H,), dev, "slopes")
    n = _check_table(cache, page_table, B, lengths)
    c = cache.struct()
    with _Device(dev):
        st = load().fa_kv4_attend(q.data_ptr(), ctypes.addressof(c), page_table.data_ptr(), n, lengths.data_ptr(),
                                  o.data_ptr(), lse.data_ptr(), 1 if causal else 0, cap, _addr(slopes), _addr(workspace),
                                  _ws_bytes(workspace, dev), B, H, N, scale, _raw_stream(stream, dev))
    _check("fa_kv4_attend", st)


def fa_kv4_attend_tree_workspace_size(B: int, H: int, H_kv: int, N_q: int, d: int) -> int:
    return load().fa_kv4_attend_tree_workspace_size(B, H, H_kv, N_q, d)


def fa_kv4_attend_tree(q, cache: KV4Cache, page_table, lengths, parents, count, o, lse, workspace, scale: float,
                       cap: float = 0.0, slopes=None, stream=None):
    """q, o [B, H, N_q, d]: the last count[b] of each sequence's lengths[b] cached tokens are a tree of drafted tokens
    (parents [B, N_q]); ``workspace``: CUDA uint8 of at least fa_kv4_attend_tree_workspace_size(...) bytes."""
    import torch

    _check_array(o, cache.dtype, q.shape, cache.dev, "o")
    _check_array(lse, torch.float32, q.shape[:3], cache.dev, "lse")
    if q.dim() != 4 or q.shape[3] != cache.d or cache.H_kv < 1 or q.shape[1] % cache.H_kv:
        raise ValueError("q must be [B, H, N_q, d] with the cache's d, its head count dividing H")
    B, H, N, _ = q.shape
    dev = cache.dev
    _check_array(q, cache.dtype, q.shape, dev, "q")
    if parents is None:
        raise ValueError("parents must be given")
    _check_array(parents, torch.int32, (B, N), dev, "parents")
    if slopes is not None:
        _check_array(slopes, torch.float32, (H,), dev, "slopes")
    n = _check_table(cache, page_table, B, lengths, *(() if count is None else (count,)))
    c = cache.struct()
    with _Device(dev):
        st = load().fa_kv4_attend_tree(q.data_ptr(), ctypes.addressof(c), page_table.data_ptr(), n, lengths.data_ptr(),
                                       parents.data_ptr(), _addr(count), o.data_ptr(), lse.data_ptr(), cap, _addr(slopes),
                                       _addr(workspace), _ws_bytes(workspace, dev), B, H, N, scale, _raw_stream(stream, dev))
    _check("fa_kv4_attend_tree", st)


def fa_kv4_tree_many_rows(B: int, H: int, H_kv: int, N_q: int, d: int, room: int, num_sms: int = 0) -> bool:
    """Whether a tree call of these sizes, with a page table for ``room`` tokens a sequence, goes to the kernel for
    many rows (host query; num_sms 0: the current device's)."""
    y = load().fa_kv4_tree_many_rows(B, H, H_kv, N_q, d, room, num_sms)
    if y < 0:
        raise FaError("fa_kv4_tree_many_rows", 1)
    return bool(y)


def fa_kv4_keep(cache: KV4Cache, page_table, start, path, kept, stream=None):
    """Tokens start[b] + path[b, j] become tokens start[b] + j, j < kept[b]; path [B, N] int32."""
    import torch

    if path.dim() != 2:
        raise ValueError("path must be [B, N]")
    B, N = path.shape
    dev = cache.dev
    _check_array(path, torch.int32, (B, N), dev, "path")
    n = _check_table(cache, page_table, B, start, kept)
    c = cache.struct()
    with _Device(dev):
        st = load().fa_kv4_keep(ctypes.addressof(c), page_table.data_ptr(), n, start.data_ptr(), path.data_ptr(),
                                kept.data_ptr(), B, N, _raw_stream(stream, dev))
    _check("fa_kv4_keep", st)


class KV4Pages:
    """What a server keeps of its pages, int32 on one device: table [B, max_pages], the pages of
    each sequence in order (the first held[b] of its row), and a stack of free pages, the first
    free_count[0] of free."""

    def __init__(self, table, held, free, free_count):
        self.arrays = (table, held, free, free_count)
        self.dev = native().kv4_pages_check(*self.arrays)

    table = property(lambda self: self.arrays[0])
    held = property(lambda self: self.arrays[1])
    free = property(lambda self: self.arrays[2])
    free_count = property(lambda self: self.arrays[3])

    @property
    def device(self):
        return self.table.device

    @classmethod
    def empty(cls, B: int, max_pages: int, num_pages: int, device="cuda"):
        """No sequence holds a page: all of 0 .. num_pages - 1 are free."""
        import torch

        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.full((B, max_pages), -1, **i32), torch.zeros(B, **i32),
                   torch.arange(num_pages - 1, -1, -1, **i32), torch.full((1,), num_pages, **i32))


def fa_kv4_plan(pages: KV4Pages, page_size: int, start, count, parents, out_count, lengths, slots, positions, stream=None):
    """Pages for count[b] tokens behind start[b] into ``pages``; out_count, lengths [B] and positions [B, N] int32,
    slots [B, N] int64."""
    import torch

    if slots.dim() != 2:
        raise ValueError("slots must be [B, N]")
    B, max_pages = pages.table.shape
    N, dev = slots.shape[1], pages.dev
    for t, name in ((start, "start"), (count, "count"), (out_count, "out_count"), (lengths, "lengths")):
        if t is None:
            raise ValueError(f"{name} must be given")
        _check_array(t, torch.int32, (B,), dev, name)
    if parents is not None:
        _check_array(parents, torch.int32, (B, N), dev, "parents")
    _check_array(slots, torch.int64, (B, N), dev, "slots")
    _check_array(positions, torch.int32, (B, N), dev, "positions")
    with _Device(dev):
        st = load().fa_kv4_plan(pages.table.data_ptr(), pages.held.data_ptr(), max_pages, pages.free.data_ptr(),
                                pages.free.shape[0], pages.free_count.data_ptr(), page_size, start.data_ptr(), count.data_ptr(),
                                _addr(parents), out_count.data_ptr(), lengths.data_ptr(), slots.data_ptr(),
                                positions.data_ptr(), B, N, _raw_stream(stream, dev))
    _check("fa_kv4_plan", st)


class RotaryRowsStruct(ctypes.Structure):
    """fa_rotary_rows of the header."""

    _fields_ = [("in_", _vp), ("out", _vp), ("in_stride", ctypes.c_longlong * 3), ("out_stride", ctypes.c_longlong * 3)]


def _rotary_rows(x, out, like, dev: int):
    for t in (x, out):
        if (t.dim() != 4 or t.dtype is not like.dtype or t.get_device() != dev or t.shape != x.shape or t.shape[0] != like.shape[0]
                or t.shape[2:] != like.shape[2:] or (t.shape[3] > 1 and t.stride(3) != 1)):
            raise ValueError("q, k and their outputs must be [B, heads, N, d] of one type and device, their channels neighbours")
    c3 = ctypes.c_longlong * 3
    return RotaryRowsStruct(x.data_ptr(), out.data_ptr(), c3(*x.stride()[:3]), c3(*out.stride()[:3]))


def fa_rotary(q, k, positions, freqs, out_q, out_k, interleaved: bool = False, backward: bool = False, amplitude: float = 1.0,
              stream=None):
    """Rows q [B, H, N, d] and k [B, H_kv, N, d] (None: no keys), any strides, turned by their positions
    [B, N] (None: 0 .. N - 1) into out_q and out_k; freqs: float64 [dims / 2]."""
    import torch

    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    dev = _device_of(q)
    B, H, N, d = q.shape
    rq = _rotary_rows(q, out_q, q, dev)
    rk = _rotary_rows(k, out_k, q, dev) if k is not None else None
    if positions is not None:
        _check_array(positions, torch.int32, (B, N), dev, "positions")
    if freqs.dim() != 1:
        raise ValueError("freqs must be [dims / 2]")
    _check_array(freqs, torch.float64, freqs.shape, dev, "freqs")
    with _Device(dev):
        st = load().fa_rotary(ctypes.addressof(rq), ctypes.addressof(rk) if rk is not None else None, _addr(positions),
                              freqs.data_ptr(), 2 * freqs.shape[0], 1 if interleaved else 0, 1 if backward else 0, amplitude, B, H,
                              k.shape[1] if k is not None else 0, N, d, _dtype_code(q), _raw_stream(stream, dev))
    _check("fa_rotary", st)


def fa_rotary_turns(freq: float) -> int:
    """Fraction of a turn, in units of 2^-64, of one position's angle of ``freq`` radians (host query)."""
    return int(load().fa_rotary_turns(freq))


def fa_kv4_row(pages, page_size: int, num_pages: int, pos: int) -> int:
    """Row of the pool, seen as [num_pages, page_size], of token ``pos`` of a sequence whose
    pages are the ints ``pages``, or -1 (host query: the kernels' lookup)."""
    arr = (ctypes.c_int32 * max(1, len(pages)))(*pages)
    return int(load().fa_kv4_row(arr, len(pages), page_size, num_pages, pos))


def fa_host_scratch_size(B: int, H: int, N: int, d: int, backward: bool = True) -> int:
    return int(load().fa_host_scratch_size(B, H, N, d, int(bool(backward))))


def fa_host_chunk_plan(B: int, H: int, N: int, chunks: int = 0) -> list:
    """Heads per chunk of the host-buffer pipeline for these sizes (host query)."""
    plan = (ctypes.c_int * 64)()
    n = load().fa_host_chunk_plan(B, H, N, chunks, plan, 64)
    if n < 0:
        raise FaError("fa_host_chunk_plan", 1)
    return list(plan[:n])


def fa_cta_head_group(nheads: int, nblocks: int, bytes_per_head: int, causal: bool, num_sms: int) -> int:
    """Heads per group of the kernels' CTA order (host query)."""
    g = load().fa_cta_head_group(nheads, nblocks, bytes_per_head, int(bool(causal)), num_sms)
    if g < 0:
        raise FaError("fa_cta_head_group", 1)
    return int(g)


def _host_tensors(*ts):
    for t in ts:
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("host entry points take contiguous CPU tensors (pinned for overlap)")


def fa_fwd_host(q, k, v, o, lse, scratch, scale: float, causal: bool, chunks: int = 0, stream=None):
    """Forward pass on host tensors (q, k, v, o [B,H,N,d]; lse [B,H,N] fp32) through a CUDA
    ``scratch`` (uint8) of at least fa_host_scratch_size(B, H, N, d, False) bytes."""
    lib = load()
    B, H, N, d = _shape(q)
    _host_tensors(q, k, v, o, lse)
    code = lib.fa_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(scratch),
                           scratch.numel() * scratch.element_size(), B, H, N, d, float(scale), int(bool(causal)),
                           _dtype_code(q), int(chunks), _stream(stream))
    _check("fa_fwd_host", code)


def fa_fwd_bwd_host(q, k, v, dout, o, lse, dq, dk, dv, scratch, scale: float, causal: bool, chunks: int = 0,
                    stream=None):
    """Forward and backward pass on host tensors through a CUDA ``scratch`` (uint8) of at
    least fa_host_scratch_size(B, H, N, d, True) bytes; outputs valid after ``stream`` syncs."""
    lib = load()
    B, H, N, d = _shape(q)
    _host_tensors(q, k, v, dout, o, lse, dq, dk, dv)
    code = lib.fa_fwd_bwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(o), _ptr(lse), _ptr(dq), _ptr(dk),
                               _ptr(dv), _ptr(scratch), scratch.numel() * scratch.element_size(), B, H, N, d,
                               float(scale), int(bool(causal)), _dtype_code(q), int(chunks), _stream(stream))
    _check("fa_fwd_bwd_host", code)


def fa_check_device_status(stream=None):
    """Synchronize and raise FaError: FA_ERR_DEVICE_TIMEOUT if a kernel gave up on a wait,
    FA_ERR_DEVICE_CHECK if a cached token had no page (or, in the checked build, a check failed)."""
    lib = load()
    code = lib.fa_check_device_status(_stream(stream))
    if code != FA_OK:
        rec = (ctypes.c_uint32 * 4)()
        lib.fa_last_device_error_detail(rec)
        raise FaError("fa_check_device_status", code, [int(x) for x in rec])


def fa_selftest_wait_timeout(limit_us: int, stream=None):
    """Launch the failure-detection self-test (a wait that gives up after ``limit_us``);
    the next fa_check_device_status reports it."""
    _check("fa_selftest_wait_timeout", load().fa_selftest_wait_timeout(int(limit_us), _stream(stream)))


PROFILE_KINDS = {0: "fwd", 1: "bwd_kv", 2: "bwd_q", 3: "bwd_fused"}


def fa_profile_begin(n: int):
    """Record the time of each of the next ``n`` main-kernel launches of fa_fwd / fa_bwd."""
    _check("fa_profile_begin", load().fa_profile_begin(int(n)))


def fa_profile_end(max_out: int = 65536):
    """Wait for the recorded events; returns [(kind, ms)] in launch order, kind one of
    PROFILE_KINDS' names."""
    ms = (ctypes.c_float * max_out)()
    kind = (ctypes.c_int * max_out)()
    n = load().fa_profile_end(ms, kind, max_out)
    if n < 0:
        raise FaError("fa_profile_end", 5)
    return [(PROFILE_KINDS.get(kind[i], str(kind[i])), float(ms[i])) for i in range(n)]


def fa_status_string(code: int) -> str:
    return load().fa_status_string(int(code)).decode()


def fa_version() -> int:
    return int(load().fa_version())
