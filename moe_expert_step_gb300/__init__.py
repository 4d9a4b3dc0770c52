"""Block-diffusion MoE denoising step for GB300 (sm_103a): Python binding of libmoestep.

Every function here marshals torch tensors into the C ABI declared in
``include/moestep.h`` and calls it; all computation happens in the library's
CUDA kernels.  There is no Python or CPU fallback: if the library is not
built, importing works but every call raises ``MoeStepError``.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

from . import _build

BF16 = 0
F32 = 1
FP8 = 2

ROTARY_PLAIN, ROTARY_LINEAR, ROTARY_ROTATIONS, ROTARY_DIMENSIONS = 0, 1, 2, 3

OK = 0
EINVAL = -1
EWORKSPACE = -2
EALIGN = -3
ECUDA = -4
EDEVICE = -5
EUNSUPPORTED = -6
ETIMEOUT = -7
EDEVINPUT = -8

PROF_KERNELS = ["route", "coreset", "gather", "expert_ffn", "expert_down", "combine", "lm_head", "commit", "other"]

EXPORTS = [
    "moestep_workspace_size", "moestep_workspace_init", "moe_block_route", "moe_route_from_logits", "coreset_select", "moe_block_ffn",
    "lm_head_commit", "lm_commit_from_logits", "block_embed", "block_decode_step", "block_decode_loop",
    "moestep_read_device_error",
    "moestep_error_string", "moestep_last_cuda_error", "moestep_prof_enable", "moestep_prof_read",
    "moestep_set_wait_timeout_ns", "moestep_set_route_fusion", "moestep_route_fusion", "moestep_launch_count",
    "moe_block_route_noalloc",
    "moestep_kv_workspace_size", "kv_cache_write", "kv_cache_read", "block_attention", "block_residual_norm",
    "kv_cache_plan", "rotary_frequencies", "block_rotary", "moestep_delta_workspace_size", "block_delta_rule",
]


class MoeStepError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        # the library's text for the code, once it is loaded (loading it may be what failed)
        text = error_string(code) if _LIB is not None else "library not loaded"
        super().__init__(f"{what}: {text} ({code})")


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("H", "E", "k", "I", "Is", "V", "P", "dtype")]


class Layer(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("Wr", "Wgu", "Wd", "Wsgu", "Wsd", "Sgu", "Sd", "Ssgu", "Ssd")]


class Trace(ctypes.Structure):
    _fields_ = [("n_sel", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("hidden", ctypes.c_void_p),
                ("sel", ctypes.c_void_p), ("x", ctypes.c_void_p), ("h", ctypes.c_void_p)]


class KvDimsC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("Hq", "Hkv", "D", "page", "n_pages", "max_pages", "dtype")]


class KvCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_exp", "v_exp", "table")]
    _holds = None  # of the tensors (kv_cache): type, Hkv, page, D, max_pages


class DeltaDimsC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("Hk", "Hv", "Dk", "Dv", "n_slots", "dtype")]


_LIB = None


def library_path() -> str:
    return _build.LIB


def lib():
    """The loaded libmoestep.so (raises MoeStepError if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(_build.LIB):
            raise MoeStepError(EDEVICE, f"{_build.LIB} is not built (run __graft_entry__.build())")
        L = ctypes.CDLL(_build.LIB)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        D = ctypes.POINTER(Dims)
        ll, KD, KC = ctypes.c_longlong, ctypes.POINTER(KvDimsC), ctypes.POINTER(KvCache)
        f64, DD = ctypes.c_double, ctypes.POINTER(DeltaDimsC)
        sig = {
            "moestep_workspace_size": [D, i, ctypes.POINTER(sz)],
            "moestep_workspace_init": [vp, sz, vp],
            "moe_block_route": [D, i, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_route_from_logits": [D, i, vp, vp, vp, vp, vp, sz, vp],
            "moe_block_route_noalloc": [D, i, vp, vp, vp, vp, vp, vp, vp],
            "coreset_select": [D, i, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_block_ffn": [D, i, vp, ctypes.POINTER(Layer), vp, vp, vp, sz, vp],
            "lm_head_commit": [D, i, vp, vp, f, f, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "lm_commit_from_logits": [D, i, vp, f, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "block_embed": [D, i, vp, vp, vp, vp, i, vp, vp],
            "block_decode_step": [D, i, i, ctypes.POINTER(Layer), vp, vp, f, f, vp, vp, vp, vp, vp, vp, vp, vp,
                                  ctypes.POINTER(Trace), vp, sz, vp],
            "block_decode_loop": [D, i, i, ctypes.POINTER(Layer), vp, vp, vp, i, vp, f, f, i, vp, vp, vp, vp, sz, vp],
            "moestep_read_device_error": [vp, sz, vp, ctypes.POINTER(i)],
            "moestep_error_string": [i],
            "moestep_last_cuda_error": [],
            "moestep_prof_enable": [i],
            "moestep_prof_read": [i, ctypes.POINTER(i), ctypes.POINTER(ctypes.c_double)],
            "moestep_set_wait_timeout_ns": [ctypes.c_ulonglong],
            "moestep_set_route_fusion": [ctypes.c_int],
            "moestep_route_fusion": [],
            "moestep_launch_count": [],
            "moestep_kv_workspace_size": [KD, i, i, ctypes.POINTER(sz)],
            "kv_cache_write": [KD, i, i, vp, vp, ll, vp, KC, vp, sz, vp],
            "kv_cache_read": [KD, i, i, vp, KC, vp, vp, vp, sz, vp],
            "block_attention": [KD, i, i, vp, ll, vp, KC, f, i, i, vp, vp, vp, sz, vp],
            "block_residual_norm": [D, i, vp, i, vp, vp, ll, f, vp, vp, vp, vp, f, vp],
            "kv_cache_plan": [KD, i, i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "rotary_frequencies": [i, f64, i, f64, f64, f64, f64, vp, vp],
            "block_rotary": [KD, i, i, vp, ll, vp, ll, vp, vp, i, i, f, vp, ll, vp, ll, vp],
            "moestep_delta_workspace_size": [DD, i, i, ctypes.POINTER(sz)],
            "block_delta_rule": [DD, i, i, vp, ll, vp, ll, vp, ll, vp, vp, vp, vp, vp, vp, vp, f, f, vp, vp, sz, vp],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = {"moestep_error_string": ctypes.c_char_p,
                          "moestep_launch_count": ctypes.c_longlong}.get(name, ctypes.c_int)
        _LIB = L
    return _LIB


def error_string(code: int) -> str:
    try:
        return lib().moestep_error_string(code).decode()
    except MoeStepError:
        return "library not built"


def _check(rc: int, what: str) -> None:
    if rc != OK:
        if rc == ECUDA:
            what = f"{what} (cudaError {lib().moestep_last_cuda_error()})"
        raise MoeStepError(rc, what)


def _p(t):
    """Raw pointer of a tensor (None -> NULL)."""
    if t is None:
        return None
    return t.data_ptr()


_CURRENT = None  # torch's functions for the current device and the handle of its current stream, once CUDA is up


def _s(stream):
    """cudaStream_t of a torch stream (None: the current one), or of an integer handle."""
    global _CURRENT
    if stream is None:
        if _CURRENT is not None:
            return _CURRENT[1](_CURRENT[0]())
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle alone: no Stream object
        if raw is not None and torch.cuda.is_initialized():
            _CURRENT = torch._C._cuda_getDevice, raw
            return raw(torch._C._cuda_getDevice())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


@dataclass(frozen=True)
class ModelDims:
    H: int
    E: int
    k: int
    I: int
    Is: int
    V: int
    P: int = 32
    dtype: int = BF16

    def c(self) -> Dims:
        return Dims(self.H, self.E, self.k, self.I, self.Is, self.V, self.P, self.dtype)


def layer(Wr, Wgu, Wd, Wsgu=None, Wsd=None, Sgu=None, Sd=None, Ssgu=None, Ssd=None) -> Layer:
    """Device pointers of one layer; the four row-scale tensors only with FP8 expert weights.
    The returned struct holds references to the tensors, so their memory stays allocated for
    as long as the struct is alive."""
    lay = Layer(_p(Wr), _p(Wgu), _p(Wd), _p(Wsgu), _p(Wsd), _p(Sgu), _p(Sd), _p(Ssgu), _p(Ssd))
    lay._tensors = (Wr, Wgu, Wd, Wsgu, Wsd, Sgu, Sd, Ssgu, Ssd)
    return lay


def workspace_size(d: ModelDims, R: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moestep_workspace_size(ctypes.byref(d.c()), R, ctypes.byref(n)), "moestep_workspace_size")
    return n.value


def workspace_init(ws, stream=None) -> None:
    _check(lib().moestep_workspace_init(_p(ws), ws.numel(), _s(stream)), "moestep_workspace_init")


def workspace(d: ModelDims, R: int, device="cuda", stream=None):
    """Allocate (through torch) and initialise a workspace for R requests."""
    import torch
    ws = torch.empty(workspace_size(d, R), dtype=torch.uint8, device=device)
    workspace_init(ws, stream)
    return ws


def moe_block_route(d: ModelDims, x, Wr, idx, mass, gate, ws, logits=None, stream=None) -> None:
    _check(lib().moe_block_route(ctypes.byref(d.c()), x.shape[0], _p(x), _p(Wr), _p(idx), _p(mass), _p(gate),
                                 _p(logits), _p(ws), ws.numel(), _s(stream)), "moe_block_route")


def moe_block_route_noalloc(d: ModelDims, x, Wr, idx, mass, gate, logits=None, stream=None) -> None:
    """The router without a workspace (scratch in a fixed array inside the library); for callers
    that cannot allocate device memory.  Calls that overlap on the GPU race on that array."""
    _check(lib().moe_block_route_noalloc(ctypes.byref(d.c()), x.shape[0], _p(x), _p(Wr), _p(idx), _p(mass),
                                         _p(gate), _p(logits), _s(stream)), "moe_block_route_noalloc")


def moe_route_from_logits(d: ModelDims, logits, idx, mass, gate, ws, stream=None) -> None:
    _check(lib().moe_route_from_logits(ctypes.byref(d.c()), logits.shape[0], _p(logits), _p(idx), _p(mass),
                                       _p(gate), _p(ws), ws.numel(), _s(stream)), "moe_route_from_logits")


def coreset_select(d: ModelDims, R: int, top_p, idx, mass, n_sel, sel, survive, gate_rr, ws, stream=None) -> None:
    _check(lib().coreset_select(ctypes.byref(d.c()), R, _p(top_p), _p(idx), _p(mass), _p(n_sel), _p(sel),
                                _p(survive), _p(gate_rr), _p(ws), ws.numel(), _s(stream)), "coreset_select")


def moe_block_ffn(d: ModelDims, R: int, x, lay: Layer, gate_rr, out, ws, stream=None) -> None:
    _check(lib().moe_block_ffn(ctypes.byref(d.c()), R, _p(x), ctypes.byref(lay), _p(gate_rr), _p(out), _p(ws),
                               ws.numel(), _s(stream)), "moe_block_ffn")


def lm_head_commit(d: ModelDims, R: int, hidden, Wlm, threshold, tokens, masked, choice, conf, accept, n_committed,
                   ws, logit_scale=1.0, logits=None, stream=None) -> None:
    _check(lib().lm_head_commit(ctypes.byref(d.c()), R, _p(hidden), _p(Wlm), float(logit_scale), float(threshold),
                                _p(tokens), _p(masked), _p(choice), _p(conf), _p(accept), _p(n_committed),
                                _p(logits), _p(ws), ws.numel(), _s(stream)), "lm_head_commit")


def lm_commit_from_logits(d: ModelDims, R: int, logits, threshold, tokens, masked, choice, conf, accept, n_committed,
                          ws, stream=None) -> None:
    _check(lib().lm_commit_from_logits(ctypes.byref(d.c()), R, _p(logits), float(threshold), _p(tokens), _p(masked),
                                       _p(choice), _p(conf), _p(accept), _p(n_committed), _p(ws), ws.numel(),
                                       _s(stream)), "lm_commit_from_logits")


def block_embed(d: ModelDims, R: int, tokens, masked, emb, pos, mask_id: int, h, stream=None) -> None:
    _check(lib().block_embed(ctypes.byref(d.c()), R, _p(tokens), _p(masked), _p(emb), _p(pos), int(mask_id), _p(h),
                             _s(stream)), "block_embed")


def block_decode_step(d: ModelDims, R: int, layers, Wlm, top_p, threshold, h_in, tokens, masked, choice, conf,
                      accept, n_committed, ws, h_out=None, logit_scale=1.0, trace_n_sel=None, trace_idx=None,
                      trace_hidden=None, trace_sel=None, trace_x=None, trace_h=None, stream=None) -> None:
    """One denoising round; the optional trace_* tensors receive the per-layer records of
    moestep_trace (trace_x: each layer's MoE input, trace_h: the residual entering it)."""
    arr = (Layer * max(1, len(layers)))(*layers)
    tr = Trace(_p(trace_n_sel), _p(trace_idx), _p(trace_hidden), _p(trace_sel), _p(trace_x), _p(trace_h))
    _check(lib().block_decode_step(ctypes.byref(d.c()), R, len(layers), arr, _p(Wlm), _p(top_p), float(logit_scale),
                                   float(threshold), _p(h_in), _p(h_out), _p(tokens), _p(masked), _p(choice),
                                   _p(conf), _p(accept), _p(n_committed), ctypes.byref(tr), _p(ws), ws.numel(),
                                   _s(stream)), "block_decode_step")


def block_decode_loop(d: ModelDims, R: int, layers, Wlm, emb, pos, mask_id: int, top_p, threshold, tokens, masked,
                      rounds, ws, max_rounds=None, logit_scale=1.0, stream=None) -> None:
    """Every LowConfidence round of the block on the device (CUDA-graph while loop); rounds[0] = rounds run."""
    arr = (Layer * max(1, len(layers)))(*layers)
    mr = d.P if max_rounds is None else int(max_rounds)
    _check(lib().block_decode_loop(ctypes.byref(d.c()), R, len(layers), arr, _p(Wlm), _p(emb), _p(pos), int(mask_id),
                                   _p(top_p), float(logit_scale), float(threshold), mr, _p(tokens), _p(masked),
                                   _p(rounds), _p(ws), ws.numel(), _s(stream)), "block_decode_loop")


# ------------------------------------------------------------------------------ the attention side of a layer


@dataclass(frozen=True)
class KvDims:
    """Shape of a paged key-value cache and of the heads that read it (moestep_kv_dims)."""
    Hq: int
    Hkv: int
    D: int
    page: int
    n_pages: int
    max_pages: int
    dtype: int = BF16

    def __post_init__(self):
        c = KvDimsC(self.Hq, self.Hkv, self.D, self.page, self.n_pages, self.max_pages, self.dtype)
        object.__setattr__(self, "_c", ctypes.byref(c))  # kept: single-token calls are short
        object.__setattr__(self, "_holds", (self.dtype, self.Hkv, self.page, self.D, self.max_pages))

    def __reduce__(self):  # (a reference into a C struct cannot be copied or pickled)
        return KvDims, (self.Hq, self.Hkv, self.D, self.page, self.n_pages, self.max_pages, self.dtype)


def kv_cache(k, v, table, k_exp=None, v_exp=None) -> KvCache:
    """Device pointers of one paged cache: k, v [n_pages, Hkv, page, D] in bf16, fp32 or, for MOESTEP_FP8, E4M3 codes
    (or their bytes), table [R, max_pages] int32, and with MOESTEP_FP8 k_exp, v_exp [n_pages, Hkv, page] uint8.  The
    struct keeps the tensors alive; each call compares them with its dims and R (a pool may have more pages, a table
    more rows than a call names)."""
    import torch
    tensors = (k, v, table, k_exp, v_exp)
    for t in tensors:
        if t is not None and not t.is_contiguous():
            raise MoeStepError(EINVAL, "kv_cache: tensors must be contiguous")
    kind = {torch.bfloat16: BF16, torch.float32: F32, torch.float8_e4m3fn: FP8, torch.uint8: FP8}.get(k.dtype)
    if kind is None or k.dim() != 4 or v.dtype is not k.dtype or v.shape != k.shape:
        raise MoeStepError(EINVAL, "kv_cache: k and v must be [n_pages, Hkv, page, D], bf16, fp32 or E4M3, and alike")
    if table.dim() != 2 or table.dtype is not torch.int32:
        raise MoeStepError(EINVAL, "kv_cache: table must be [R, max_pages] int32")
    for e in (k_exp, v_exp) if kind == FP8 else ():
        if e is None or e.dtype is not torch.uint8 or e.shape != k.shape[:3]:
            raise MoeStepError(EINVAL, "kv_cache: k_exp and v_exp must be [n_pages, Hkv, page] uint8")
    if not all(t is None or t.is_cuda for t in tensors):
        raise MoeStepError(EINVAL, "kv_cache: tensors must be on the GPU")
    c = KvCache(_p(k), _p(v), _p(k_exp), _p(v_exp), _p(table))
    c._tensors = tensors
    c._holds = (kind, *k.shape[1:], table.shape[1])
    c._n_pages, c._rows = k.shape[0], table.shape[0]
    return c


def _fits(cache: KvCache, kd: KvDims, R: int, ws, what: str) -> None:
    """The cache holds what kd and R say (a struct of raw pointers is taken as it is), the workspace is on the GPU."""
    holds = cache._holds
    if holds is not None and (holds != kd._holds or cache._n_pages < kd.n_pages or cache._rows < R):
        raise MoeStepError(EINVAL, f"{what}: the cache does not have the type, the pages or the table of {kd}, R = {R}")
    if not ws.is_cuda:
        raise MoeStepError(EINVAL, f"{what}: ws must be on the GPU")


def kv_workspace_size(kd: KvDims, R: int, n_q: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moestep_kv_workspace_size(kd._c, R, n_q, ctypes.byref(n)), "moestep_kv_workspace_size")
    return n.value


def kv_workspace(kd: KvDims, R: int, n_q: int, device="cuda", stream=None):
    """Allocate (through torch) and initialise a workspace for the cache calls."""
    import torch
    ws = torch.empty(kv_workspace_size(kd, R, n_q), dtype=torch.uint8, device=device)
    workspace_init(ws, stream)
    return ws


_ACT = {}  # torch types of the activations of each dtype and of the integers (torch is imported late)


def _types() -> dict:
    if not _ACT:
        import torch
        _ACT.update({BF16: torch.bfloat16, FP8: torch.bfloat16, F32: torch.float32, "int": torch.int32, "turn": torch.int64,
                     "byte": torch.uint8})
    return _ACT


def _rows(t, heads: int, kd: KvDims, what: str) -> int:
    """Distance between the rows of t [tokens, heads, D], which may be part of a wider row."""
    st, shape = t.stride(), t.shape
    if (len(st) != 3 or st[2] != 1 or (heads > 1 and st[1] != kd.D) or shape[1] != heads or shape[2] != kd.D
            or t.dtype is not _types().get(kd.dtype)):
        raise MoeStepError(EINVAL, f"{what} must be [tokens, {heads}, {kd.D}] in the activations' type, heads dense")
    if not t.is_cuda:
        raise MoeStepError(EINVAL, f"{what} must be on the GPU")
    return st[0] if shape[0] > 1 else heads * kd.D  # (of one row: any)


def _dense(t, shape, dtype, what: str) -> None:
    """t is a contiguous GPU tensor of the shape and type."""
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise MoeStepError(EINVAL, f"{what} must be contiguous, of shape {list(shape)} and type {dtype}")
    if not t.is_cuda:
        raise MoeStepError(EINVAL, f"{what} must be on the GPU")


def kv_cache_write(kd: KvDims, R: int, k, v, pos, cache: KvCache, ws, stream=None) -> None:
    """Store the keys and values k, v [R * n, Hkv, D] (rows may be parts of wider rows) at positions
    pos [R, n] int32; a negative position is not stored."""
    n = pos.shape[1]
    _dense(pos, (R, n), _types()["int"], "kv_cache_write: pos")
    ld = _rows(k, kd.Hkv, kd, "kv_cache_write: k")
    if _rows(v, kd.Hkv, kd, "kv_cache_write: v") != ld or k.shape[0] != R * n or v.shape[0] != R * n:
        raise MoeStepError(EINVAL, "kv_cache_write: k and v must have R * n rows, equally far apart")
    _fits(cache, kd, R, ws, "kv_cache_write")
    _check(lib().kv_cache_write(kd._c, R, n, k.data_ptr(), v.data_ptr(), ld, pos.data_ptr(), cache, ws.data_ptr(),
                                ws.numel(), _s(stream)), "kv_cache_write")


def kv_cache_read(kd: KvDims, R: int, pos, cache: KvCache, k, v, ws, stream=None) -> None:
    """Read the cached vectors at positions pos [R, n] back into k, v [R * n, Hkv, D] (zeros where negative)."""
    n = pos.shape[1]
    _dense(pos, (R, n), _types()["int"], "kv_cache_read: pos")
    act = _types().get(kd.dtype)
    _dense(k, (R * n, kd.Hkv, kd.D), act, "kv_cache_read: k")
    _dense(v, (R * n, kd.Hkv, kd.D), act, "kv_cache_read: v")
    _fits(cache, kd, R, ws, "kv_cache_read")
    _check(lib().kv_cache_read(kd._c, R, n, pos.data_ptr(), cache, k.data_ptr(), v.data_ptr(), ws.data_ptr(),
                               ws.numel(), _s(stream)), "kv_cache_read")


def block_attention(kd: KvDims, R: int, q, kv_len, cache: KvCache, out, ws, scale: float, causal: bool = False,
                    window: int = 0, lse=None, stream=None) -> None:
    """Attention of q [R * n_q, Hq, D] (rows may be parts of wider rows) over the first kv_len [R] cached
    positions of each request, the last n_q of which are the queries' own; see block_attention in moestep.h."""
    T = q.shape[0]
    n_q = T // R if R > 0 else 0
    ld = _rows(q, kd.Hq, kd, "block_attention: q")
    _dense(out, (R * n_q, kd.Hq, kd.D), _types().get(kd.dtype), "block_attention: out")
    _dense(kv_len, (R,), _types()["int"], "block_attention: kv_len")
    if R * n_q != T:
        raise MoeStepError(EINVAL, "block_attention: q must have R * n_q rows")
    if lse is not None:
        _dense(lse, (T, kd.Hq), _types()[F32], "block_attention: lse")
    _fits(cache, kd, R, ws, "block_attention")
    _check(lib().block_attention(kd._c, R, n_q, q.data_ptr(), ld, kv_len.data_ptr(), cache, scale, int(causal),
                                 min(int(window), 0x7fffffff), out.data_ptr(), _p(lse), ws.data_ptr(), ws.numel(), _s(stream)),
           "block_attention")


def block_residual_norm(d: ModelDims, y, h_in, h_out, x, w_pre=None, w_post=None, gate=None, res_scale: float = 1.0,
                        eps: float = 1e-6, stream=None) -> None:
    """h_out = h_in + res_scale * gate * (w_post * y / rms(y)); x = w_pre * h_out / rms(h_out).  y [T, H] fp32 or
    bf16; gate fp32 [H], or [requests, H] with one row for each d.P tokens; see block_residual_norm in moestep.h."""
    T, H = y.shape[0], d.H
    shape, types = (T, H), _types()
    f32, act = types[F32], types.get(d.dtype)
    if y.dtype is not f32 and y.dtype is not types[BF16]:
        raise MoeStepError(EINVAL, "block_residual_norm: y must be bf16 or fp32")
    _dense(y, shape, y.dtype, "block_residual_norm: y")
    _dense(h_in, shape, f32, "block_residual_norm: h_in")
    _dense(h_out, shape, f32, "block_residual_norm: h_out")
    if x is not None:
        _dense(x, shape, act, "block_residual_norm: x")
    for w in (w_pre, w_post):
        if w is not None:
            _dense(w, (H,), act, "block_residual_norm: w_pre, w_post")
    gate_ld = 0
    if gate is not None:
        rows, st = gate.shape, gate.stride()
        if (len(rows) not in (1, 2) or rows[-1] != H or st[-1] != 1 or gate.dtype is not f32 or not gate.is_cuda
                or (len(rows) == 2 and rows[0] * d.P < T)):
            raise MoeStepError(EINVAL, "block_residual_norm: gate must be fp32 on the GPU, [H] or [requests, H]")
        gate_ld = st[0] if len(rows) == 2 and rows[0] > 1 else 0
    _check(lib().block_residual_norm(ctypes.byref(d.c()), T, y.data_ptr(), F32 if y.dtype is f32 else BF16, _p(w_post),
                                     _p(gate), gate_ld, res_scale, h_in.data_ptr(), h_out.data_ptr(), _p(w_pre),
                                     _p(x), eps, _s(stream)), "block_residual_norm")


# ------------------------------------------------------------------------------ pages, positions, the delta rule


def _device() -> int:
    """The current device: launches go to it, so a call's tensors have to be there.  (0 before CUDA is up: none are.)"""
    if _CURRENT is not None:
        return _CURRENT[0]()
    import torch
    return torch.cuda.current_device() if torch.cuda.is_initialized() else 0


def _here(t, shape, dtype, what: str, device: int) -> None:
    """t is contiguous, of the shape and type, on the GPU of that index."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        _dense(t, shape, dtype, what)
        raise MoeStepError(EINVAL, f"{what} must be on the current device")


def kv_cache_plan(kd: KvDims, R: int, kv_len, n_new, ring, head, head_out, table, new_len, pos, ws, slots=None,
                  stream=None) -> None:
    """Give R requests pages and positions for n_new [R] more tokens each (negative: the last -n_new go): pages from
    the ring of free ones [n_pages] with head [2] = (first, count), or back to it; the tables [R, max_pages] are
    extended, pos [R, n] (-1 behind the new tokens), slots [R, n] and new_len [R] are written.  All int32; see
    kv_cache_plan in moestep.h."""
    n, i32, requests, dev = pos.shape[-1], _types()["int"], (R,), _device()
    _here(kv_len, requests, i32, "kv_cache_plan: kv_len", dev)
    _here(n_new, requests, i32, "kv_cache_plan: n_new", dev)
    _here(new_len, requests, i32, "kv_cache_plan: new_len", dev)
    _here(ring, (kd.n_pages,), i32, "kv_cache_plan: ring", dev)
    _here(head, (2,), i32, "kv_cache_plan: head", dev)
    _here(head_out, (2,), i32, "kv_cache_plan: head_out", dev)
    _here(pos, (R, n), i32, "kv_cache_plan: pos", dev)
    rows = table.shape[0]
    _here(table, (rows, kd.max_pages), i32, "kv_cache_plan: table", dev)
    if rows < R:
        raise MoeStepError(EINVAL, "kv_cache_plan: table must have a row a request")
    if slots is not None:
        _here(slots, (R, n), i32, "kv_cache_plan: slots", dev)
    _on_gpu(ws, "kv_cache_plan", dev)
    rc = lib().kv_cache_plan(kd._c, R, n, kv_len.data_ptr(), n_new.data_ptr(), ring.data_ptr(), head.data_ptr(),
                             head_out.data_ptr(), table.data_ptr(), new_len.data_ptr(), pos.data_ptr(), _p(slots),
                             ws.data_ptr(), ws.numel(), _s(stream))
    if rc:
        _check(rc, "kv_cache_plan")


def _on_gpu(ws, what: str, device: int) -> None:
    if ws.get_device() != device or not ws.is_contiguous() or ws.element_size() != 1:
        raise MoeStepError(EINVAL, f"{what}: ws must be bytes on the GPU, the current device")


def rotary_frequencies(rot: int, base: float, scaling: int = ROTARY_PLAIN, factor: float = 1.0, original: float = 1.0,
                       low: float = 1.0, high: float = 2.0, device="cuda", stream=None):
    """Table for block_rotary, [rot / 2] int64 holding the bits of uint64: the fraction of a turn that each pair makes
    a position, times 2^64.  Pairs turn base^(-2 i / rot) radians, or less where that is scaled for a context longer
    than the `original` one (ROTARY_*); see rotary_frequencies in moestep.h."""
    import torch
    if int(rot) != rot or rot <= 0 or rot % 2:
        raise MoeStepError(EINVAL, "rotary_frequencies: rot must be even and positive")
    freq = torch.empty(int(rot) // 2, dtype=torch.int64, device=device)
    if freq.get_device() != _device():
        raise MoeStepError(EINVAL, "rotary_frequencies: device must be the current one")
    _check(lib().rotary_frequencies(int(rot), base, scaling, factor, original, low, high, freq.data_ptr(), _s(stream)),
           "rotary_frequencies")
    return freq


def block_rotary(kd: KvDims, q, k, pos, freq, q_out, k_out, interleaved: bool = False, mscale: float = 1.0,
                 stream=None) -> None:
    """Turn the first 2 * len(freq) of the D elements of q [R * n, Hq, D] and k [R * n, Hkv, D] (either may be None;
    rows may be parts of wider rows) by the positions pos [R, n] (negative: the row is left) into q_out, k_out,
    which may be q and k themselves.  freq: of rotary_frequencies; pairs are halves of the rotated part apart, or
    neighbours where interleaved; see block_rotary in moestep.h."""
    types, dev = _types(), _device()
    if pos.dim() != 2 or freq.dim() != 1 or (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise MoeStepError(EINVAL, "block_rotary: pos must be [R, n], freq [rot / 2]; q and k come with their outputs")
    R, n = shape = pos.shape
    _here(pos, shape, types["int"], "block_rotary: pos", dev)
    _here(freq, freq.shape, types["turn"], "block_rotary: freq", dev)
    act, q_ld, k_ld, qo_ld, ko_ld = types.get(kd.dtype), 0, 0, 0, 0
    qp = kp = qo = ko = None
    if q is not None:
        heads = (R * n, kd.Hq, kd.D)
        qp, q_ld = q.data_ptr(), _head_rows(q, heads, act, "block_rotary: q", dev)
        qo, qo_ld = q_out.data_ptr(), _head_rows(q_out, heads, act, "block_rotary: q_out", dev)
    if k is not None:
        heads = (R * n, kd.Hkv, kd.D)
        kp, k_ld = k.data_ptr(), _head_rows(k, heads, act, "block_rotary: k", dev)
        ko, ko_ld = k_out.data_ptr(), _head_rows(k_out, heads, act, "block_rotary: k_out", dev)
    rc = lib().block_rotary(kd._c, R, n, qp, q_ld, kp, k_ld, pos.data_ptr(), freq.data_ptr(), 2 * freq.shape[0],
                            interleaved, mscale, qo, qo_ld, ko, ko_ld, _s(stream))
    if rc:
        _check(rc, "block_rotary")


@dataclass(frozen=True)
class DeltaDims:
    """Shape of a layer of the gated delta rule and of its pool of states (moestep_delta_dims)."""
    Hk: int
    Hv: int
    Dk: int
    Dv: int
    n_slots: int
    dtype: int = BF16

    def __post_init__(self):
        c = DeltaDimsC(self.Hk, self.Hv, self.Dk, self.Dv, self.n_slots, self.dtype)
        object.__setattr__(self, "_c", ctypes.byref(c))

    def __reduce__(self):
        return DeltaDims, (self.Hk, self.Hv, self.Dk, self.Dv, self.n_slots, self.dtype)


def delta_workspace_size(dd: DeltaDims, R: int, n: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().moestep_delta_workspace_size(dd._c, R, n, ctypes.byref(out)), "moestep_delta_workspace_size")
    return out.value


def delta_workspace(dd: DeltaDims, R: int, n: int, device="cuda", stream=None):
    """Allocate (through torch) and initialise a workspace for block_delta_rule."""
    import torch
    ws = torch.empty(delta_workspace_size(dd, R, n), dtype=torch.uint8, device=device)
    workspace_init(ws, stream)
    return ws


def _head_rows(t, shape, dtype, what: str, device: int) -> int:
    """Distance between the rows of t [tokens, heads, D], which may be part of a wider row."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise MoeStepError(EINVAL, f"{what} must be {list(shape)} in the activations' type, on the GPU, the current device")
    ld, head, one = t.stride()
    if one != 1 or (head != shape[2] and shape[1] > 1):
        raise MoeStepError(EINVAL, f"{what}: heads and their elements must be dense")
    return ld if shape[0] > 1 else shape[1] * shape[2]


def block_delta_rule(dd: DeltaDims, R: int, q, k, v, g, beta, state, out, ws, state_out=None, slot=None, length=None,
                     fresh=None, scale: float = 1.0, qk_eps: float = 0.0, stream=None) -> None:
    """The gated delta rule over the tokens of R requests: q, k [R * n, Hk, Dk] and v [R * n, Hv, Dv] (rows may be
    parts of wider rows), g (logarithm of the decay) and beta [R * n, Hv] fp32, state [n_slots, Hv, Dv, Dk] fp32 with
    the request's slot [R], out [R * n, Hv, Dv].  state_out: where the new states go (state itself, or None: not
    wanted); length [R]: tokens of each; fresh [R] uint8: begin from nothing; see block_delta_rule in moestep.h."""
    T, types, dev = q.shape[0], _types(), _device()
    n = T // R if R > 0 else 0
    if R * n != T:
        raise MoeStepError(EINVAL, "block_delta_rule: q must have R * n rows")
    act = types.get(dd.dtype) if dd.dtype != FP8 else None
    keys, values, gates = (T, dd.Hk, dd.Dk), (T, dd.Hv, dd.Dv), (T, dd.Hv)
    q_ld = _head_rows(q, keys, act, "block_delta_rule: q", dev)
    k_ld = _head_rows(k, keys, act, "block_delta_rule: k", dev)
    v_ld = _head_rows(v, values, act, "block_delta_rule: v", dev)
    f32, pool = types[F32], (dd.n_slots, dd.Hv, dd.Dv, dd.Dk)
    _here(g, gates, f32, "block_delta_rule: g", dev)
    _here(beta, gates, f32, "block_delta_rule: beta", dev)
    _here(state, pool, f32, "block_delta_rule: state", dev)
    _here(out, values, act, "block_delta_rule: out", dev)
    if state_out is not None and state_out is not state:
        _here(state_out, pool, f32, "block_delta_rule: state_out", dev)
    if slot is not None:
        _here(slot, (R,), types["int"], "block_delta_rule: slot", dev)
    if length is not None:
        _here(length, (R,), types["int"], "block_delta_rule: length", dev)
    if fresh is not None:
        _here(fresh, (R,), types["byte"], "block_delta_rule: fresh", dev)
    _on_gpu(ws, "block_delta_rule", dev)
    rc = lib().block_delta_rule(dd._c, R, n, q.data_ptr(), q_ld, k.data_ptr(), k_ld, v.data_ptr(), v_ld, g.data_ptr(),
                                beta.data_ptr(), _p(length), _p(slot), _p(fresh), state.data_ptr(), _p(state_out), scale,
                                qk_eps, out.data_ptr(), ws.data_ptr(), ws.numel(), _s(stream))
    if rc:
        _check(rc, "block_delta_rule")


def read_device_error(ws, stream=None) -> int:
    w = ctypes.c_int(0)
    _check(lib().moestep_read_device_error(_p(ws), ws.numel(), _s(stream), ctypes.byref(w)),
           "moestep_read_device_error")
    return w.value


SEPARATE_HEAD, FUSED_COMBINE_HEAD = 0, 2


def set_route_fusion(mode) -> None:
    """What block_decode_step runs between expert launches: SEPARATE_HEAD (0) the combine /
    router / coreset / gather launches; FUSED_COMBINE_HEAD (2, the default) the combine inside
    the router's launch (bit-identical results)."""
    _check(lib().moestep_set_route_fusion(int(mode)), "moestep_set_route_fusion")


def route_fusion() -> int:
    """The mode last set by set_route_fusion."""
    return int(lib().moestep_route_fusion())


def set_wait_timeout_ns(ns: int) -> None:
    _check(lib().moestep_set_wait_timeout_ns(int(ns)), "moestep_set_wait_timeout_ns")


def prof_enable(kernels=None) -> None:
    """Time the named kernels (None = all, [] = off) with CUDA events on their stream."""
    names = PROF_KERNELS if kernels is None else list(kernels)
    mask = 0
    for n in names:
        mask |= 1 << PROF_KERNELS.index(n)
    _check(lib().moestep_prof_enable(mask), "moestep_prof_enable")


def launch_count() -> int:
    return int(lib().moestep_launch_count())


def prof_read() -> dict:
    """{kernel name: (launches, total ms)} of everything launched while profiling was on."""
    out = {}
    for kid, name in enumerate(PROF_KERNELS):
        n = ctypes.c_int(0)
        ms = ctypes.c_double(0.0)
        _check(lib().moestep_prof_read(kid, ctypes.byref(n), ctypes.byref(ms)), "moestep_prof_read")
        out[name] = (n.value, ms.value)
    return out


def build(quiet: bool = True) -> str:
    global _LIB
    _LIB = None
    return _build.build(quiet=quiet)
