"""ctypes binding of libattn25.so — argument marshalling only.

Every function here has the name of the C entry point it calls (declared in
include/attn25.h) and does no attention work of its own: it checks tensor
metadata, turns torch tensors into device pointers and sizes, and raises
AttnError on a non-zero status.  PyTorch provides device memory and streams.
There is no fallback: if the shared library is missing or fails to load,
importing this module raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# ATTN25_LIBRARY may name the profiling build (libattn25_trace.so) instead.
LIB_PATH = os.environ.get("ATTN25_LIBRARY") or os.path.join(_HERE, "libattn25.so")

MOD_NONE = 0
MOD_CAUSAL = 1
MOD_ALIBI = 2
MOD_SOFTCAP = 3
MOD_SLIDING_WINDOW = 4
MOD_LOCAL_BOOST = 5
MOD_DOCUMENT = 6
# Mask flags ORed onto a kind to compose mods (score transform of the kind,
# AND of the masks).
MASK_CAUSAL = 0x100
MASK_SLIDING_WINDOW = 0x200
MASK_DOCUMENT = 0x400
MASK_BITMAP = 0x800
MASK_VARLEN = 0x1000

ATTN_ERR_TIMEOUT = -6
ATTN_ERR_INDEX = -8


class AttnError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {code} ({attn_strerror(code)})")
        self.code = code


class CModParams(ctypes.Structure):
    _fields_ = [
        ("softcap", ctypes.c_float),
        ("window", ctypes.c_int32),
        ("boost", ctypes.c_float),
        ("boost_radius", ctypes.c_int32),
        ("alibi_slopes", ctypes.c_void_p),
        ("doc_offsets", ctypes.c_void_p),
        ("num_docs", ctypes.c_int32),
        ("bitmap", ctypes.c_void_p),
        ("bitmap_row_words", ctypes.c_int32),
        ("bitmap_heads", ctypes.c_int32),
        ("bitmap_head_stride", ctypes.c_int64),
        ("bitmap_batch_stride", ctypes.c_int64),
        ("q_offsets", ctypes.c_void_p),
        ("k_offsets", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int32),
    ]


class CStrides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("s", ctypes.c_int64)]


class CLayouts(ctypes.Structure):
    _fields_ = [(n, CStrides) for n in ("q", "k", "v", "out", "dout", "dq", "dk", "dv")]


class CBlockMask(ctypes.Structure):
    _fields_ = [
        ("tile_class", ctypes.c_void_p),
        ("kv_count", ctypes.c_void_p),
        ("kv_index", ctypes.c_void_p),
        ("q_count", ctypes.c_void_p),
        ("q_index", ctypes.c_void_p),
        ("fwd_order", ctypes.c_void_p),
        ("bwd_order", ctypes.c_void_p),
        ("B", ctypes.c_int32),
        ("Sq", ctypes.c_int32),
        ("Skv", ctypes.c_int32),
        ("nq_tiles", ctypes.c_int32),
        ("nk_tiles", ctypes.c_int32),
        ("mod_kind", ctypes.c_int32),
    ]


class CCache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_strides", CStrides),
        ("v_strides", CStrides),
        ("page_table", ctypes.c_void_p),
        ("lens", ctypes.c_void_p),
        ("B", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("D", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python tiled_attention_25_b200/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, P, P, P]
    lib.attn_fwd.restype = I
    lib.attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, S, I, I, I, I, I, I, F, I, P, P, P]
    lib.attn_bwd.restype = I
    lib.attn_bwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, P, P]
    lib.attn_bwd_noalloc.restype = I
    lib.attn_bwd_noalloc_max_workspace.argtypes = []
    lib.attn_bwd_noalloc_max_workspace.restype = S
    lib.attn_bwd_workspace_size.argtypes = [I, I, I, I]
    lib.attn_bwd_workspace_size.restype = S
    lib.attn_block_mask_bytes.argtypes = [I, I, I]
    lib.attn_block_mask_bytes.restype = S
    lib.attn_block_mask_bind.argtypes = [P, S, I, I, I, ctypes.POINTER(CBlockMask)]
    lib.attn_block_mask_bind.restype = I
    lib.build_block_mask.argtypes = [I, P, I, I, I, ctypes.POINTER(CBlockMask), P]
    lib.build_block_mask.restype = I
    lib.attn_fwd_strided.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, P, P, P, P]
    lib.attn_fwd_strided.restype = I
    lib.attn_bwd_strided.argtypes = [P, P, P, P, P, P, P, P, P, P, S, I, I, I, I, I, I, F, I, P, P, P, P]
    lib.attn_bwd_strided.restype = I
    lib.attn_bwd_deterministic.argtypes = [P, P, P, P, P, P, P, P, P, P, S, I, I, I, I, I, I, F, I, P, P, P]
    lib.attn_bwd_deterministic.restype = I
    lib.attn_bwd_deterministic_workspace_size.argtypes = [I, I, I, I]
    lib.attn_bwd_deterministic_workspace_size.restype = S
    lib.attn_fwd_fp8.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, P, P]
    lib.attn_fwd_fp8.restype = I
    lib.attn_fp8_rotate_quantize.argtypes = [P, P, P, P, I, I, I, I, P]
    lib.attn_fp8_rotate_quantize.restype = I
    lib.attn_cache_append.argtypes = [P, P, P, P, P, P, I, P, P, P, P]
    lib.attn_cache_append.restype = I
    lib.attn_tree_workspace_size.argtypes = [I, I, I, I]
    lib.attn_tree_workspace_size.restype = S
    lib.attn_tree_fwd.argtypes = [P, P, P, P, P, P, P, S, P, P, I, I, F, I, P, P, P]
    lib.attn_tree_fwd.restype = I
    lib.attn_cache_weights.argtypes = [P, P, P, P, P, P, P, I, I, F, I, P, P, P]
    lib.attn_cache_weights.restype = I
    lib.attn_evict_plan.argtypes = [P, P, P, P, P, P, I, I, I, P]
    lib.attn_evict_plan.restype = I
    lib.attn_cache_compact.argtypes = [P, P, P, I, P, P, P]
    lib.attn_cache_compact.restype = I
    lib.attn_get_status.argtypes = [P]
    lib.attn_get_status.restype = I
    lib.attn_set_wait_limit_ms.argtypes = [ctypes.c_uint32]
    lib.attn_set_wait_limit_ms.restype = None
    lib.attn_set_work_walk.argtypes = [I]
    lib.attn_set_work_walk.restype = I
    lib.attn_check_wait_timeout.argtypes = [P]
    lib.attn_check_wait_timeout.restype = I
    lib.attn_strerror.argtypes = [I]
    lib.attn_strerror.restype = ctypes.c_char_p
    if hasattr(lib, "attn_trace_read"):  # profiling build only
        lib.attn_trace_read.argtypes = [ctypes.POINTER(ctypes.c_ulonglong), I]
        lib.attn_trace_read.restype = I
        lib.attn_trace_reset.argtypes = []
        lib.attn_trace_reset.restype = I
        lib.attn_trace_window.argtypes = [I]
        lib.attn_trace_window.restype = I
    return lib


LIB = _load()

EXPORTED = ("attn_fwd", "attn_bwd", "attn_bwd_workspace_size", "attn_bwd_noalloc",
            "attn_bwd_noalloc_max_workspace", "attn_block_mask_bytes",
            "attn_block_mask_bind", "build_block_mask", "attn_get_status",
            "attn_set_wait_limit_ms", "attn_strerror", "attn_fwd_strided", "attn_bwd_strided",
            "attn_bwd_deterministic", "attn_bwd_deterministic_workspace_size", "attn_check_wait_timeout",
            "attn_fp8_rotate_quantize", "attn_fwd_fp8", "attn_set_work_walk", "attn_cache_append",
            "attn_tree_workspace_size", "attn_tree_fwd", "attn_cache_weights", "attn_evict_plan",
            "attn_cache_compact")


def attn_strerror(code: int) -> str:
    return LIB.attn_strerror(int(code)).decode()


def _check(code: int, what: str):
    if code != 0:
        raise AttnError(code, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


class ModParams:
    """Mod scalars plus the device tensors they point at (kept alive here)."""

    def __init__(self, softcap=50.0, window=1024, boost=1.1, boost_radius=128,
                 alibi_slopes=None, doc_offsets=None, bitmap=None, q_offsets=None, k_offsets=None):
        self.softcap = float(softcap)
        self.window = int(window)
        self.boost = float(boost)
        self.boost_radius = int(boost_radius)
        self.alibi_slopes = alibi_slopes        # device fp32 [Hq] or None
        self.doc_offsets = doc_offsets          # device int32 [B][num_docs+1] or None
        if doc_offsets is not None:
            assert doc_offsets.dtype == torch.int32 and doc_offsets.is_contiguous() and doc_offsets.dim() == 2
        if alibi_slopes is not None:
            assert alibi_slopes.dtype == torch.float32 and alibi_slopes.is_contiguous()
        # device int32 [B or 1][Hq or 1][Sq][row_words] keep bits (bit j & 31 of word j >> 5)
        # device int32 [B][num_seqs + 1] each: the varlen mask's query and key offsets
        self.q_offsets, self.k_offsets = q_offsets, k_offsets
        if (q_offsets is None) != (k_offsets is None):
            raise ValueError("the varlen mask needs both query and key offsets")
        if q_offsets is not None:
            for t in (q_offsets, k_offsets):
                assert t.dtype == torch.int32 and t.is_contiguous() and t.dim() == 2
            assert q_offsets.shape == k_offsets.shape
        self.bitmap = bitmap
        if bitmap is not None:
            assert bitmap.dtype == torch.int32 and bitmap.is_contiguous() and bitmap.dim() == 4

    def c(self) -> CModParams:
        bm = self.bitmap
        if bm is None:
            bm_args = (None, 0, 0, 0, 0)
        else:
            nb, nh, sq, rw = bm.shape
            bm_args = (bm.data_ptr(), rw, nh, 0 if nh == 1 else sq * rw, 0 if nb == 1 else nh * sq * rw)
        return CModParams(self.softcap, self.window, self.boost, self.boost_radius,
                          None if self.alibi_slopes is None else self.alibi_slopes.data_ptr(),
                          None if self.doc_offsets is None else self.doc_offsets.data_ptr(),
                          0 if self.doc_offsets is None else self.doc_offsets.shape[1] - 1, *bm_args,
                          None if self.q_offsets is None else self.q_offsets.data_ptr(),
                          None if self.k_offsets is None else self.k_offsets.data_ptr(),
                          0 if self.q_offsets is None else self.q_offsets.shape[1] - 1)


class BlockMask:
    """A bound block mask: the C struct plus the device buffer that holds it."""

    def __init__(self, buffer: torch.Tensor, c: CBlockMask):
        self.buffer = buffer
        self.c = c

    def view(self, name):
        """The named array as a torch view of the buffer (for inspection and tests)."""
        c = self.c
        B, nq, nk = c.B, c.nq_tiles, c.nk_tiles
        npairs = (nq + 1) // 2
        shapes = {"tile_class": (torch.uint8, (B, nq, nk)), "kv_count": (torch.int32, (B, nq)),
                  "kv_index": (torch.int32, (B, nq, nk)), "q_count": (torch.int32, (B, nk)),
                  "q_index": (torch.int32, (B, nk, nq)), "fwd_order": (torch.int32, (B * npairs,)),
                  "bwd_order": (torch.int32, (B * nk,))}
        dtype, shape = shapes[name]
        off = getattr(c, name) - self.buffer.data_ptr()
        n = 1
        for s in shape:
            n *= s
        size = n * (1 if dtype == torch.uint8 else 4)
        return self.buffer[off:off + size].view(dtype).view(shape)


def _mp(mod_params, mod_kind, B, Hq, Sq):
    """Marshal the mod params; a bitmap tensor must cover every (b, h, row) the
    call reads (the C side cannot see its extent)."""
    if mod_params is None:
        return None
    code = int(mod_kind)
    # offsets arrays: one row per batch row (the C side cannot see their extent)
    if (code & 0xFF) == MOD_DOCUMENT or code & MASK_DOCUMENT:
        t = mod_params.doc_offsets
        if t is None or t.shape[0] < B:
            raise ValueError(f"the document mask needs doc_offsets with {B} rows")
    if code & MASK_VARLEN:
        t = mod_params.q_offsets
        if t is None or t.shape[0] < B:
            raise ValueError(f"the varlen mask needs q_offsets and k_offsets with {B} rows")
    bm = mod_params.bitmap
    if int(mod_kind) & MASK_BITMAP and bm is not None:
        nb, nh, sq, _ = bm.shape
        if nb not in (1, B) or (Hq is not None and nh not in (1, Hq)) or sq < Sq:
            raise ValueError(f"bitmap of shape {tuple(bm.shape)} does not cover B={B}, Hq={Hq}, Sq={Sq}")
    cm = mod_params.c()
    return ctypes.byref(cm), cm


def _dims(q, k, v, out):
    for t in (q, k, v, out):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q, k, v, out must be contiguous CUDA bf16 [B][H][S][D] tensors")
    B, Hq, Sq, D = q.shape
    Bk, Hkv, Skv, Dk = k.shape
    if tuple(v.shape) != (Bk, Hkv, Skv, Dk) or Bk != B or Dk != D or tuple(out.shape) != (B, Hq, Sq, D):
        raise ValueError("inconsistent q/k/v/out shapes")
    return B, Hq, Hkv, Sq, Skv, D


def attn_fwd(q, k, v, out, lse=None, scale=None, mod_kind=MOD_NONE, mod_params=None,
             block_mask=None, stream=None):
    B, Hq, Hkv, Sq, Skv, D = _dims(q, k, v, out)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, Sq) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 [B][Hq][Sq] tensor")
    scale = D ** -0.5 if scale is None else float(scale)
    mp = _mp(mod_params, mod_kind, B, Hq, Sq)
    rc = LIB.attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq, Skv, D,
                      scale, int(mod_kind), None if mp is None else mp[0],
                      None if block_mask is None else ctypes.byref(block_mask.c), _stream(stream))
    _check(rc, "attn_fwd")


def _strides(t, shape, what):
    """Element strides (b, h, s) of a [B][H][S][D] CUDA bf16 view with D contiguous."""
    if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 4 or tuple(t.shape) != tuple(shape) \
            or t.stride(3) != 1:
        raise ValueError(f"{what} must be a CUDA bf16 {tuple(shape)} view with its last dimension contiguous")
    return CStrides(t.stride(0), t.stride(1), t.stride(2))


def _layouts(**views):
    lay = CLayouts()
    for name, (t, shape) in views.items():
        setattr(lay, name, _strides(t, shape, name))
    return lay


def attn_fwd_strided(q, k, v, out, lse=None, scale=None, mod_kind=MOD_NONE, mod_params=None, block_mask=None,
                     stream=None):
    """attn_fwd on [B][H][S][D] views of any strides whose last dimension is
    contiguous (e.g. x.permute(0, 2, 1, 3) of a [B][S][H][D] tensor)."""
    B, Hq, Sq, D = q.shape
    _, Hkv, Skv, _ = k.shape
    lay = _layouts(q=(q, (B, Hq, Sq, D)), k=(k, (B, Hkv, Skv, D)), v=(v, (B, Hkv, Skv, D)),
                   out=(out, (B, Hq, Sq, D)))
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, Sq) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 [B][Hq][Sq] tensor")
    scale = D ** -0.5 if scale is None else float(scale)
    mp = _mp(mod_params, mod_kind, B, Hq, Sq)
    rc = LIB.attn_fwd_strided(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq, Skv, D, scale,
                              int(mod_kind), None if mp is None else mp[0],
                              None if block_mask is None else ctypes.byref(block_mask.c), ctypes.byref(lay),
                              _stream(stream))
    _check(rc, "attn_fwd_strided")


def attn_bwd_strided(q, k, v, out, lse, dout, dq, dk, dv, workspace, scale=None, mod_kind=MOD_NONE,
                     mod_params=None, block_mask=None, stream=None):
    """attn_bwd on strided views (see attn_fwd_strided)."""
    B, Hq, Sq, D = q.shape
    _, Hkv, Skv, _ = k.shape
    qs, ks = (B, Hq, Sq, D), (B, Hkv, Skv, D)
    lay = _layouts(q=(q, qs), k=(k, ks), v=(v, ks), out=(out, qs), dout=(dout, qs), dq=(dq, qs), dk=(dk, ks),
                   dv=(dv, ks))
    scale = D ** -0.5 if scale is None else float(scale)
    mp = _mp(mod_params, mod_kind, B, Hq, Sq)
    rc = LIB.attn_bwd_strided(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                              _ptr(dv), _ptr(workspace), workspace.numel() * workspace.element_size(), B, Hq, Hkv,
                              Sq, Skv, D, scale, int(mod_kind), None if mp is None else mp[0],
                              None if block_mask is None else ctypes.byref(block_mask.c), ctypes.byref(lay),
                              _stream(stream))
    _check(rc, "attn_bwd_strided")


def attn_fp8_rotate_quantize(x, signs, codes, scales, stream=None):
    """x: CUDA bf16 [B][H][S][D]; signs: CUDA int8 [D] of +-1; codes: CUDA uint8
    like x; scales: CUDA fp32 [B][H]."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous() or x.dim() != 4:
        raise ValueError("x must be a contiguous CUDA bf16 [B][H][S][D] tensor")
    B, H, S, D = x.shape
    if signs.dtype != torch.int8 or tuple(signs.shape) != (D,) or not signs.is_contiguous():
        raise ValueError("signs must be a contiguous int8 [D] tensor")
    if codes.dtype != torch.uint8 or tuple(codes.shape) != (B, H, S, D) or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous uint8 tensor shaped like x")
    if scales.dtype != torch.float32 or tuple(scales.shape) != (B, H) or not scales.is_contiguous():
        raise ValueError("scales must be a contiguous fp32 [B][H] tensor")
    _check(LIB.attn_fp8_rotate_quantize(_ptr(x), _ptr(signs), _ptr(codes), _ptr(scales), B, H, S, D,
                                        _stream(stream)), "attn_fp8_rotate_quantize")


def attn_fwd_fp8(q8, k8, q_scales, k_scales, v, out, lse=None, scale=None, mod_kind=MOD_NONE, mod_params=None,
                 block_mask=None, stream=None):
    """The forward with e4m3 Q and K (codes from attn_fp8_rotate_quantize)."""
    for t, name in ((q8, "q8"), (k8, "k8")):
        if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous CUDA uint8 [B][H][S][D] tensor")
    B, Hq, Sq, D = q8.shape
    Bk, Hkv, Skv, Dk = k8.shape
    if (Bk, Dk) != (B, D) or tuple(v.shape) != (B, Hkv, Skv, D) or tuple(out.shape) != (B, Hq, Sq, D):
        raise ValueError("inconsistent q8/k8/v/out shapes")
    for t in (v, out):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("v and out must be contiguous CUDA bf16 tensors")
    if tuple(q_scales.shape) != (B, Hq) or tuple(k_scales.shape) != (B, Hkv):
        raise ValueError("q_scales must be [B][Hq] and k_scales [B][Hkv]")
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, Sq) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 [B][Hq][Sq] tensor")
    scale = D ** -0.5 if scale is None else float(scale)
    mp = _mp(mod_params, mod_kind, B, Hq, Sq)
    rc = LIB.attn_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(q_scales), _ptr(k_scales), _ptr(v), _ptr(out), _ptr(lse),
                          B, Hq, Hkv, Sq, Skv, D, scale, int(mod_kind), None if mp is None else mp[0],
                          None if block_mask is None else ctypes.byref(block_mask.c), _stream(stream))
    _check(rc, "attn_fwd_fp8")


def attn_bwd_deterministic_workspace_size(B, Hq, Sq, D) -> int:
    return int(LIB.attn_bwd_deterministic_workspace_size(B, Hq, Sq, D))


def attn_bwd_deterministic(q, k, v, out, lse, dout, dq, dk, dv, workspace, scale=None, mod_kind=MOD_NONE,
                           mod_params=None, block_mask=None, stream=None):
    """attn_bwd with a bitwise reproducible dQ (see include/attn25.h)."""
    B, Hq, Hkv, Sq, Skv, D = _dims(q, k, v, out)
    for t in (dout, dq):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != (B, Hq, Sq, D) or not t.is_contiguous():
            raise ValueError("dout/dq must be contiguous bf16 like q")
    for t in (dk, dv):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != (B, Hkv, Skv, D) or not t.is_contiguous():
            raise ValueError("dk/dv must be contiguous bf16 like k")
    scale = D ** -0.5 if scale is None else float(scale)
    mp = _mp(mod_params, mod_kind, B, Hq, Sq)
    rc = LIB.attn_bwd_deterministic(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
                                    _ptr(dk), _ptr(dv), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), B, Hq, Hkv, Sq, Skv, D,
                                    scale, int(mod_kind), None if mp is None else mp[0],
                                    None if block_mask is None else ctypes.byref(block_mask.c), _stream(stream))
    _check(rc, "attn_bwd_deterministic")


def attn_bwd_workspace_size(B, Hq, Sq, D) -> int:
    return int(LIB.attn_bwd_workspace_size(B, Hq, Sq, D))


def attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, workspace, scale=None, mod_kind=MOD_NONE,
             mod_params=None, block_mask=None, stream=None):
    B, Hq, Hkv, Sq, Skv, D = _dims(q, k, v, out)
    for t in (dout, dq):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != (B, Hq, Sq, D) or not t.is_contiguous():
            raise ValueError("dout/dq must be contiguous bf16 like q")
    for t in (dk, dv):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != (B, Hkv, Skv, D) or not t.is_contiguous():
            raise ValueError("dk/dv must be contiguous bf16 like k")
    scale = D ** -0.5 if scale is None else float(scale)
    mp = _mp(mod_params, mod_kind, B, Hq, Sq)
    rc = LIB.attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
                      _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel() * workspace.element_size(),
                      B, Hq, Hkv, Sq, Skv, D, scale, int(mod_kind), None if mp is None else mp[0],
                      None if block_mask is None else ctypes.byref(block_mask.c), _stream(stream))
    _check(rc, "attn_bwd")


def attn_bwd_noalloc(q, k, v, out, lse, dout, dq, dk, dv, scale=None, mod_kind=MOD_NONE,
                     mod_params=None, block_mask=None, stream=None):
    """attn_bwd on the library's own fixed workspace (see include/attn25.h)."""
    B, Hq, Hkv, Sq, Skv, D = _dims(q, k, v, out)
    for t in (dout, dq):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != (B, Hq, Sq, D) or not t.is_contiguous():
            raise ValueError("dout/dq must be contiguous bf16 like q")
    for t in (dk, dv):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != (B, Hkv, Skv, D) or not t.is_contiguous():
            raise ValueError("dk/dv must be contiguous bf16 like k")
    scale = D ** -0.5 if scale is None else float(scale)
    mp = _mp(mod_params, mod_kind, B, Hq, Sq)
    rc = LIB.attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
                              _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq, Skv, D, scale, int(mod_kind),
                              None if mp is None else mp[0],
                              None if block_mask is None else ctypes.byref(block_mask.c), _stream(stream))
    _check(rc, "attn_bwd_noalloc")


def attn_bwd_noalloc_max_workspace() -> int:
    return int(LIB.attn_bwd_noalloc_max_workspace())


def attn_block_mask_bytes(B, Sq, Skv) -> int:
    return int(LIB.attn_block_mask_bytes(B, Sq, Skv))


def attn_block_mask_bind(buffer, B, Sq, Skv) -> BlockMask:
    c = CBlockMask()
    rc = LIB.attn_block_mask_bind(_ptr(buffer), buffer.numel() * buffer.element_size(), B, Sq, Skv,
                                  ctypes.byref(c))
    _check(rc, "attn_block_mask_bind")
    return BlockMask(buffer, c)


def build_block_mask(mod_kind, mod_params, B, Sq, Skv, mask: BlockMask, stream=None):
    mp = _mp(mod_params, mod_kind, B, None, Sq)
    rc = LIB.build_block_mask(int(mod_kind), None if mp is None else mp[0], B, Sq, Skv,
                              ctypes.byref(mask.c), _stream(stream))
    _check(rc, "build_block_mask")


class AttnCache:
    """A paged KV cache: the C struct plus the tensors it points at (kept
    alive here).  k, v: CUDA bf16 [pages][Hkv][page_size][D] views with their
    last dimension contiguous; lens: int32 [B]; page_table: int32
    [B][pages of a row], or None for pages b * n, b * n + 1, ... of row b
    (n = pages / B)."""

    def __init__(self, k, v, lens, page_table=None):
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must be [pages][Hkv][page_size][D] pools of one shape")
        if not k.is_cuda:
            raise ValueError("k and v must be CUDA tensors")
        self.device, self._index = k.device, k.get_device()
        P, Hkv, page, D = k.shape
        B = lens.shape[0] if lens.dim() == 1 else 0
        self._own(lens, torch.int32, (B,), "lens")
        if page_table is None:
            if B == 0 or P % B:
                raise ValueError("without a page table the pages must divide evenly among the rows")
            n = P // B
        else:
            n = page_table.shape[-1]
            self._own(page_table, torch.int32, (B, n), "page_table")
        self.k, self.v, self.lens, self.page_table = k, v, lens, page_table
        self.B, self.Hkv, self.D, self.capacity = B, Hkv, D, n * page
        self.slots = torch.Size((B, Hkv, n * page))  # of weights and positions
        self.c = CCache(k.data_ptr(), v.data_ptr(), _strides(k, k.shape, "k"), _strides(v, k.shape, "v"),
                        None if page_table is None else page_table.data_ptr(), lens.data_ptr(), B, Hkv, D, P, page, n)
        self._ref = ctypes.byref(self.c)
        self._own(k, torch.bfloat16, None, "k")
        self._own(v, torch.bfloat16, None, "v")

    def _own(self, t, dtype, shape, what):
        """An argument's type, device and (where given) shape and contiguity;
        its pointer (None stays None)."""
        if t is None:
            return None
        if t.dtype is not dtype or t.get_device() != self._index:
            raise ValueError(f"{what} must be a {dtype} tensor on the cache's CUDA device")
        if shape is not None and (t.shape != shape or not t.is_contiguous()):
            raise ValueError(f"{what} must be a contiguous {tuple(shape)} tensor")
        return t.data_ptr()

    def _views(self, **views):
        """bf16 [B][H][S][D] views (layout member = (tensor or None, shape)):
        their pointers, and their strides where any is not contiguous."""
        lay, ptrs = None, []
        for name, (t, shape) in views.items():
            if t is None:
                ptrs.append(None)
                continue
            if t.dtype is not torch.bfloat16 or t.get_device() != self._index or t.shape != shape:
                raise ValueError(f"{name} must be a bf16 {tuple(shape)} view on the cache's device")
            ptrs.append(t.data_ptr())
            if lay is None and not t.is_contiguous():
                lay = CLayouts()
        if lay is not None:
            for name, (t, shape) in views.items():
                if t is not None:
                    setattr(lay, name, _strides(t, shape, name))
        return ptrs, None if lay is None else ctypes.byref(lay)

    def _call(self, name, fn, stream, *args):
        """The C call with the cache's device current, on `stream` (default:
        that device's current stream)."""
        dev = self._index
        if stream is None:
            raw = torch._C._cuda_getCurrentRawStream(dev)  # current_stream(dev).cuda_stream without a Stream object
        else:
            raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if torch.cuda.current_device() == dev:
            rc = fn(*args, raw)
        else:
            with torch.cuda.device(dev):
                rc = fn(*args, raw)
        if rc != 0:
            raise AttnError(rc, name)


def _softcap(mod_params):
    return None if mod_params is None else ctypes.byref(mod_params.c())


def attn_cache_append(cache: AttnCache, k_new, v_new, lens_out=None, path=None, counts=None, positions=None, seen=None,
                      stream=None):
    """Append (chosen) new K and V rows to the cache (see include/attn25.h).
    k_new, v_new: bf16 [B][Hkv][T][D] views; path: int32 [B][T]; counts,
    seen, lens_out: int32 [B]; positions: int32 [B][Hkv][capacity]."""
    B, T, own, i32 = cache.B, k_new.shape[2], cache._own, torch.int32
    shape = (B, cache.Hkv, T, cache.D)
    (k_ptr, v_ptr), lay = cache._views(k=(k_new, shape), v=(v_new, shape))
    cache._call("attn_cache_append", LIB.attn_cache_append, stream, cache._ref, k_ptr, v_ptr,
                own(lens_out, i32, (B,), "lens_out"), own(path, i32, (B, T), "path"), own(counts, i32, (B,), "counts"), T, lay,
                own(positions, i32, cache.slots, "positions"), own(seen, i32, (B,), "seen"))


def attn_tree_workspace_size(Hq, Hkv, T, D) -> int:
    return int(LIB.attn_tree_workspace_size(Hq, Hkv, T, D))


def attn_tree_fwd(q, k_new, v_new, cache: AttnCache, out, lse, workspace, parents=None, counts=None, scale=None,
                  mod_kind=MOD_NONE, mod_params=None, stream=None):
    """Attention of new tokens (a tree, a chain, a single one) over the cache
    and their own ancestors (see include/attn25.h).  q, out: bf16
    [B][Hq][T][D] views; k_new, v_new: [B][Hkv][T][D] views, or None both;
    lse: fp32 [B][Hq][T] or None; parents: int32 [B][T]; counts: int32 [B]."""
    _, Hq, T, D = q.shape
    B, own = cache.B, cache._own
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    shape, kv_shape = (B, Hq, T, cache.D), (B, cache.Hkv, T, cache.D)
    (q_ptr, k_ptr, v_ptr, o_ptr), lay = cache._views(q=(q, shape), k=(k_new, kv_shape), v=(v_new, kv_shape), out=(out, shape))
    cache._call("attn_tree_fwd", LIB.attn_tree_fwd, stream, q_ptr, k_ptr, v_ptr, cache._ref, o_ptr,
                own(lse, torch.float32, (B, Hq, T), "lse"), own(workspace, torch.uint8, None, "workspace"),
                workspace.numel(), own(parents, torch.int32, (B, T), "parents"),
                own(counts, torch.int32, (B,), "counts"), Hq, T, D ** -0.5 if scale is None else scale,
                mod_kind, _softcap(mod_params), lay)


def attn_cache_weights(q, lse, cache: AttnCache, weights_in, weights_out, path=None, counts=None, scale=None,
                       mod_kind=MOD_NONE, mod_params=None, stream=None):
    """Add the attention weight each cached slot received (see
    include/attn25.h).  q: bf16 [B][Hq][T][D] view; lse: fp32 [B][Hq][T];
    weights_in (or None), weights_out: fp32 [B][Hkv][capacity]; path: int32
    [B][T]; counts: int32 [B]."""
    _, Hq, T, D = q.shape
    B, own, f32 = cache.B, cache._own, torch.float32
    (q_ptr,), lay = cache._views(q=(q, (B, Hq, T, cache.D)))
    cache._call("attn_cache_weights", LIB.attn_cache_weights, stream, q_ptr, own(lse, f32, (B, Hq, T), "lse"), cache._ref,
                own(weights_in, f32, cache.slots, "weights_in"), own(weights_out, f32, cache.slots, "weights_out"),
                own(path, torch.int32, (B, T), "path"), own(counts, torch.int32, (B,), "counts"), Hq, T,
                D ** -0.5 if scale is None else scale, mod_kind, _softcap(mod_params), lay)


def attn_evict_plan(cache: AttnCache, weights, positions, seen, moves, n_moves, budget, first=0, recent=0, stream=None):
    """Plan which slots to evict (see include/attn25.h).  weights: fp32,
    positions: int32, both [B][Hkv][capacity]; seen: int32 [B]; moves: int32
    [B][Hkv][budget][2]; n_moves: int32 [B][Hkv]."""
    B, H, own, i32 = cache.B, cache.Hkv, cache._own, torch.int32
    cache._call("attn_evict_plan", LIB.attn_evict_plan, stream, cache._ref, own(weights, torch.float32, cache.slots, "weights"),
                own(positions, i32, cache.slots, "positions"), own(seen, i32, (B,), "seen"),
                own(moves, i32, (B, H, budget, 2), "moves"), own(n_moves, i32, (B, H), "n_moves"), budget, first, recent)


def attn_cache_compact(cache: AttnCache, moves, n_moves, budget, weights=None, positions=None, stream=None):
    """Carry an eviction's moves out (see include/attn25.h)."""
    B, H, own, i32 = cache.B, cache.Hkv, cache._own, torch.int32
    cache._call("attn_cache_compact", LIB.attn_cache_compact, stream, cache._ref, own(moves, i32, (B, H, budget, 2), "moves"),
                own(n_moves, i32, (B, H), "n_moves"), budget, own(weights, torch.float32, cache.slots, "weights"),
                own(positions, i32, cache.slots, "positions"))


def attn_get_status(stream=None) -> int:
    return int(LIB.attn_get_status(_stream(stream)))


def attn_set_wait_limit_ms(ms: int):
    LIB.attn_set_wait_limit_ms(int(ms))


WALK_STATIC = 0
WALK_CLUSTER_LAUNCH_CONTROL = 1
WALK_DEFAULT = WALK_CLUSTER_LAUNCH_CONTROL


def attn_set_work_walk(walk: int):
    """How the persistent kernels take their work units (see include/attn25.h)."""
    _check(LIB.attn_set_work_walk(int(walk)), "attn_set_work_walk")


def attn_check_wait_timeout(stream=None):
    """Launch the timeout self-check (see include/attn25.h); read the outcome
    with attn_get_status."""
    _check(LIB.attn_check_wait_timeout(_stream(stream)), "attn_check_wait_timeout")


def attn_trace_read(n: int = 256) -> list:
    """Per-role cycle counters of the profiling build (libattn25_trace.so)."""
    buf = (ctypes.c_ulonglong * n)()
    _check(LIB.attn_trace_read(buf, n), "attn_trace_read")
    return list(buf)


def attn_trace_reset():
    _check(LIB.attn_trace_reset(), "attn_trace_reset")


def attn_trace_window(first_step: int):
    """First backward step whose per-role event clocks the profiling build records."""
    _check(LIB.attn_trace_window(first_step), "attn_trace_window")
