"""Python binding of libsq: the C-ABI entry points under the same names.

Argument marshalling only: every step of the compressed-KV path runs in the
CUDA library. PyTorch supplies device memory and streams. A missing or
unloadable libsq raises at import of the first call; there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsq.so")

SQ_OK, SQ_ERR_ARG, SQ_ERR_UNSUPPORTED, SQ_ERR_CUDA = 0, 1, 2, 3
SQ_ERR_NOT_CONVERGED, SQ_ERR_CAPACITY, SQ_ERR_WORKSPACE, SQ_ERR_RECORD = 4, 5, 6, 7
SQ_F32, SQ_F16, SQ_BF16 = 0, 1, 2
SQ_FLAG_CAPACITY, SQ_FLAG_RECORD, SQ_FLAG_SEQLEN, SQ_FLAG_TIMEOUT = 1, 2, 4, 0x80000000
SQ_FLAG_PAGE, SQ_FLAG_ROPE = 8, 16
DTYPE_CODE = {torch.float32: SQ_F32, torch.float16: SQ_F16, torch.bfloat16: SQ_BF16}


class SqError(RuntimeError):
    def __init__(self, status: int, what: str):
        detail = f" [{lib().sq_last_error().decode()}]" if status == SQ_ERR_CUDA else ""
        super().__init__(f"{what}: {sq_status_str(status)} ({status}){detail}")
        self.status = status


class sq_calib_params(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int), ("n_heads", ctypes.c_int), ("avg_bits", ctypes.c_double),
                ("is_key", ctypes.c_int), ("qjl", ctypes.c_int), ("normalize", ctypes.c_int),
                ("d_eff_override", ctypes.c_int), ("max_bits", ctypes.c_int), ("seed", ctypes.c_uint64),
                ("max_sweeps", ctypes.c_int), ("tol", ctypes.c_double), ("rotation", ctypes.c_int),
                ("cumvar", ctypes.c_double), ("codebooks", ctypes.c_int), ("fit_iters", ctypes.c_int)]


class sq_cache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("norm", ctypes.c_void_p), ("rnorm", ctypes.c_void_p),
                ("batch", ctypes.c_int), ("n_heads", ctypes.c_int), ("cap", ctypes.c_int64),
                ("words", ctypes.c_int)]


class sq_kv4_cache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("table", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("table_stride", ctypes.c_int64), ("batch", ctypes.c_int), ("pages_per_row", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("d", ctypes.c_int), ("page_tokens", ctypes.c_int)]


class sq_rope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("n_pos", ctypes.c_int64), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int)]


_lib = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SIGNATURES = {
    "sq_abi_version": (ctypes.c_int, []),
    "sq_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "sq_last_error": (ctypes.c_char_p, []),
    "sq_calib_bytes": (ctypes.c_size_t, [ctypes.c_int]),
    "sq_record_words": (ctypes.c_int, [ctypes.POINTER(sq_calib_params)]),
    "sq_codebook": (ctypes.c_int, [ctypes.c_int, _P, _P, _P]),
    "sq_init": (ctypes.c_int, []),
    "sq_set_option": (ctypes.c_int, [ctypes.c_int, ctypes.c_int]),
    "sq_calibrate_workspace": (ctypes.c_size_t, [ctypes.POINTER(sq_calib_params), ctypes.c_int64]),
    "sq_calibrate": (ctypes.c_int, [ctypes.POINTER(sq_calib_params), _P, ctypes.c_int, ctypes.c_int64,
                                    ctypes.c_int64, ctypes.c_int64, _P, _P, ctypes.c_size_t, _P, _P]),
    "sq_calib_import": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int, _P, _P]),
    "sq_compress_kv": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int64, _P, ctypes.POINTER(sq_cache), ctypes.POINTER(sq_cache),
                                      _P, _P]),
    "sq_compress_host_staging": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                   ctypes.c_int64]),
    "sq_compress_kv_host": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           ctypes.c_int64, _P, ctypes.POINTER(sq_cache), ctypes.POINTER(sq_cache),
                                           _P, ctypes.c_size_t, _P, _P]),
    "sq_decompress_kv": (ctypes.c_int, [_P, ctypes.POINTER(sq_cache), ctypes.c_int, ctypes.c_int64,
                                        ctypes.c_int64, ctypes.c_int, _P, _P, _P]),
    "sq_attn_workspace": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                            ctypes.c_int64]),
    "sq_attn_decode": (ctypes.c_int, [_P, _P, ctypes.POINTER(sq_cache), ctypes.POINTER(sq_cache), _P,
                                      ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64,
                                      _P, ctypes.c_int, ctypes.c_float, _P, ctypes.c_int, _P, _P,
                                      ctypes.c_size_t, _P, _P]),
    "sq_decode_step": (ctypes.c_int, [_P, _P, ctypes.POINTER(sq_cache), ctypes.POINTER(sq_cache), _P, _P, _P,
                                      ctypes.c_int, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int64, ctypes.c_float, _P, ctypes.c_int, _P, _P, ctypes.c_size_t, _P,
                                      _P]),
    "sq_attn_prefill_workspace": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                    ctypes.c_int64, ctypes.c_int64]),
    "sq_attn_prefill": (ctypes.c_int, [_P, _P, ctypes.POINTER(sq_cache), ctypes.POINTER(sq_cache), _P, ctypes.c_int,
                                       ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, _P,
                                       ctypes.c_int, ctypes.c_float, _P, ctypes.c_int, _P, ctypes.c_size_t, _P, _P]),
    "sq_attn_decode_noalloc": (ctypes.c_int, [_P, _P, ctypes.POINTER(sq_cache), ctypes.POINTER(sq_cache), _P,
                                              ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                              ctypes.c_int64, _P, ctypes.c_int, ctypes.c_float, _P, ctypes.c_int,
                                              _P, _P, _P]),
    "sq_kv4_page_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "sq_kv4_append": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P]),
    "sq_kv4_read": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P]),
    "sq_kv4_attn_workspace": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, _I64]),
    "sq_kv4_attn_decode": (ctypes.c_int, [_P, _P, ctypes.c_int, _I64, _P, ctypes.c_int, _I64, _I64, _P, ctypes.c_float,
                                          ctypes.c_int, _P, ctypes.c_int, _P, _P, ctypes.c_size_t, _P, _P]),
    "sq_kv4_decode_step": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_int, _I64, _I64, _I64, _I64, _I64, _I64, _P,
                                          ctypes.c_int, _I64, _P, ctypes.c_float, ctypes.c_int, _P, ctypes.c_int, _P,
                                          _P, ctypes.c_size_t, _P, _P]),
    "sq_kv4_attn_prefill_workspace": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, _I64]),
    "sq_kv4_attn_prefill": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, _I64, _P, ctypes.c_int, _I64, _I64, _P,
                                           ctypes.c_float, ctypes.c_int, _P, ctypes.c_int, _P, _P, ctypes.c_size_t, _P,
                                           _P]),
    "sq_wait_selftest": (ctypes.c_int, [ctypes.c_uint32, _P, _P]),
}

SQ_ATTN_NOALLOC_MAX_BYTES = 8 << 20


def lib() -> ctypes.CDLL:
    """The loaded libsq (raises if it is missing: build it with build.py)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libsq not built: {LIB_PATH} is missing "
                               "(run python -m compressed_attention_head_b200.build)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, what: str) -> None:
    if status != SQ_OK:
        raise SqError(status, what)


# --------------------------------------------------------------------------- host-only calls
def sq_abi_version() -> int:
    return lib().sq_abi_version()


def sq_status_str(status: int) -> str:
    return lib().sq_status_str(status).decode()


def sq_calib_bytes(d: int) -> int:
    return lib().sq_calib_bytes(d)


def calib_params(d, n_heads, avg_bits, is_key, qjl=True, normalize=True, d_eff_override=0, max_bits=8,
                 seed=42, max_sweeps=30, tol=1e-13, rotation=0, cumvar=0.0, codebooks=0,
                 fit_iters=0) -> sq_calib_params:
    """rotation: 0 calibrated eigenbasis, 1 random rotation (A/B baseline);
    cumvar: 0 participation-ratio d_eff, else the cumulative-variance fraction;
    codebooks: 0 shared Gaussian Lloyd-Max, 1 per-regime codebooks fitted to the
    calibration vectors (fit_iters Lloyd iterations, 0 = the library's 30)."""
    return sq_calib_params(d, n_heads, float(avg_bits), int(bool(is_key)), int(bool(qjl)), int(bool(normalize)),
                           int(d_eff_override), int(max_bits), int(seed) & ((1 << 64) - 1), int(max_sweeps),
                           float(tol), int(rotation), float(cumvar), int(codebooks), int(fit_iters))


def sq_record_words(params: sq_calib_params) -> int:
    return lib().sq_record_words(ctypes.byref(params))


def sq_codebook(b: int):
    """(levels, thresholds, D) of the library's b-bit Gaussian Lloyd-Max quantizer."""
    lv = np.zeros(1 << b)
    th = np.zeros((1 << b) - 1)
    dist = ctypes.c_double()
    _check(lib().sq_codebook(b, lv.ctypes.data, th.ctypes.data, ctypes.addressof(dist)), "sq_codebook")
    return lv, th, dist.value


def sq_calibrate_workspace(params: sq_calib_params, n_tokens: int) -> int:
    return lib().sq_calibrate_workspace(ctypes.byref(params), n_tokens)


def sq_attn_workspace(batch, n_q_heads, n_kv_heads, d, max_ctx) -> int:
    return lib().sq_attn_workspace(batch, n_q_heads, n_kv_heads, d, max_ctx)


# --------------------------------------------------------------------------- device buffers
@dataclass
class PackedCache:
    """Caller-owned device arrays of one packed cache (see sq_cache in sq.h)."""

    codes: torch.Tensor          # int32 [batch, n_heads, cap / 32, words, 32], read as uint32
    norm: torch.Tensor           # float32 [batch, n_heads, cap]
    rnorm: torch.Tensor | None   # float32 [batch, n_heads, cap] or None
    batch: int
    n_heads: int
    cap: int
    words: int

    def struct(self) -> sq_cache:
        return sq_cache(self.codes.data_ptr(), self.norm.data_ptr(),
                        self.rnorm.data_ptr() if self.rnorm is not None else None,
                        self.batch, self.n_heads, self.cap, self.words)

    def words_u32(self) -> np.ndarray:
        """The records as [batch, n_heads, cap, words] uint32 (undoing the 32-token interleave)."""
        c = self.codes.cpu().numpy().view(np.uint32)
        return np.ascontiguousarray(c.transpose(0, 1, 2, 4, 3)).reshape(self.batch, self.n_heads, self.cap,
                                                                        self.words)

    def tiled(self, rep_batch: int, rep_heads: int) -> "PackedCache":
        """A new cache holding this one repeated rep_batch times over the batch and
        rep_heads times over the heads (row (b, h) = this row (b % batch, h % n_heads))."""
        return PackedCache(self.codes.repeat(rep_batch, rep_heads, 1, 1, 1),
                           self.norm.repeat(rep_batch, rep_heads, 1),
                           self.rnorm.repeat(rep_batch, rep_heads, 1) if self.rnorm is not None else None,
                           self.batch * rep_batch, self.n_heads * rep_heads, self.cap, self.words)


def alloc_cache(batch, n_heads, cap, words, with_rnorm, device="cuda") -> PackedCache:
    """Zeroed packed cache; cap is rounded up to a multiple of 32."""
    cap = ((int(cap) + 31) // 32) * 32
    codes = torch.zeros(batch, n_heads, cap // 32, words, 32, dtype=torch.int32, device=device)
    norm = torch.zeros(batch, n_heads, cap, dtype=torch.float32, device=device)
    rnorm = torch.zeros_like(norm) if with_rnorm else None
    return PackedCache(codes, norm, rnorm, batch, n_heads, cap, words)


def alloc_records(n_heads: int, d: int, device="cuda") -> torch.Tensor:
    """Zeroed storage for n_heads calibration records (uint8, record after record)."""
    return torch.zeros(n_heads * sq_calib_bytes(d), dtype=torch.uint8, device=device)


# --------------------------------------------------------------------------- launching calls
def sq_init() -> None:
    _check(lib().sq_init(), "sq_init")


SQ_OPT_COMPRESS_PATH = 1
SQ_OPT_ATTN_PATH = 2
SQ_OPT_TC_ERROR_BOUND = 3


def sq_set_option(option: int, value: int) -> None:
    _check(lib().sq_set_option(option, value), "sq_set_option")


def sq_calibrate(params, x, n_tokens, stride_head, stride_tok, calib_out, ws, status=None, stream=None):
    _check(lib().sq_calibrate(ctypes.byref(params), _ptr(x), DTYPE_CODE[x.dtype], n_tokens, stride_head,
                              stride_tok, _ptr(calib_out), _ptr(ws), ws.numel() * ws.element_size(),
                              _ptr(status), _stream(stream)), "sq_calibrate")


def sq_calib_import(calib, n_heads, d, status=None, stream=None):
    _check(lib().sq_calib_import(_ptr(calib), n_heads, d, _ptr(status), _stream(stream)), "sq_calib_import")


def sq_compress_kv(calib_k, calib_v, k, v, batch, n_heads, d, n_tok, start_pos, kc, vc, flags=None,
                   stream=None):
    x = k if k is not None else v
    kcs = kc.struct() if kc is not None else None
    vcs = vc.struct() if vc is not None else None
    _check(lib().sq_compress_kv(_ptr(calib_k), _ptr(calib_v), _ptr(k), _ptr(v), DTYPE_CODE[x.dtype], batch,
                                n_heads, d, n_tok, _ptr(start_pos),
                                ctypes.byref(kcs) if kcs is not None else None,
                                ctypes.byref(vcs) if vcs is not None else None, _ptr(flags),
                                _stream(stream)), "sq_compress_kv")


def sq_compress_host_staging(batch, n_heads, d, dtype, n_tok) -> int:
    return lib().sq_compress_host_staging(batch, n_heads, d, DTYPE_CODE[dtype], n_tok)


def sq_compress_kv_host(calib_k, calib_v, k, v, batch, n_heads, d, n_tok, start_pos, kc, vc, staging, flags=None,
                        stream=None):
    """k, v: CPU tensors (pinned for overlapped copies); staging: a device uint8 tensor."""
    x = k if k is not None else v
    for t in (k, v):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise ValueError("sq_compress_kv_host takes contiguous host tensors")
    kcs = kc.struct() if kc is not None else None
    vcs = vc.struct() if vc is not None else None
    _check(lib().sq_compress_kv_host(_ptr(calib_k), _ptr(calib_v), _ptr(k), _ptr(v), DTYPE_CODE[x.dtype], batch,
                                     n_heads, d, n_tok, _ptr(start_pos),
                                     ctypes.byref(kcs) if kcs is not None else None,
                                     ctypes.byref(vcs) if vcs is not None else None, _ptr(staging),
                                     staging.numel() * staging.element_size() if staging is not None else 0,
                                     _ptr(flags), _stream(stream)), "sq_compress_kv_host")


def sq_decompress_kv(calib, cache, d, t0, n_tok, apply_qjl, out, flags=None, stream=None):
    cs = cache.struct()
    _check(lib().sq_decompress_kv(_ptr(calib), ctypes.byref(cs), d, t0, n_tok, int(bool(apply_qjl)), _ptr(out),
                                  _ptr(flags), _stream(stream)), "sq_decompress_kv")


def sq_attn_decode(calib_k, calib_v, kc, vc, seq_lens, batch, n_q_heads, n_kv_heads, d, max_ctx, q, scale, out,
                   scores_out=None, ws=None, flags=None, stream=None):
    kcs, vcs = kc.struct(), vc.struct()
    _check(lib().sq_attn_decode(_ptr(calib_k), _ptr(calib_v), ctypes.byref(kcs), ctypes.byref(vcs),
                                _ptr(seq_lens), batch, n_q_heads, n_kv_heads, d, max_ctx, _ptr(q),
                                DTYPE_CODE[q.dtype], float(scale), _ptr(out), DTYPE_CODE[out.dtype],
                                _ptr(scores_out), _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0,
                                _ptr(flags), _stream(stream)), "sq_attn_decode")


def sq_attn_prefill_workspace(batch, n_q_heads, n_kv_heads, d, n_qtok, max_ctx) -> int:
    return lib().sq_attn_prefill_workspace(batch, n_q_heads, n_kv_heads, d, n_qtok, max_ctx)


def sq_attn_prefill(calib_k, calib_v, kc, vc, start, batch, n_q_heads, n_kv_heads, d, n_qtok, max_ctx, q, scale, out,
                    ws, flags=None, stream=None):
    """Causal attention of q [batch, n_q, n_qtok, d] at positions start[b] + t (see sq.h)."""
    kcs, vcs = kc.struct(), vc.struct()
    _check(lib().sq_attn_prefill(_ptr(calib_k), _ptr(calib_v), ctypes.byref(kcs), ctypes.byref(vcs), _ptr(start),
                                 batch, n_q_heads, n_kv_heads, d, n_qtok, max_ctx, _ptr(q), DTYPE_CODE[q.dtype],
                                 float(scale), _ptr(out), DTYPE_CODE[out.dtype], _ptr(ws),
                                 ws.numel() * ws.element_size(), _ptr(flags), _stream(stream)), "sq_attn_prefill")


def sq_decode_step(calib_k, calib_v, kc, vc, k_new, v_new, q, pos, batch, n_q_heads, n_kv_heads, d, max_ctx, scale,
                   out, scores_out=None, ws=None, flags=None, stream=None):
    """Append the new token at pos[b] and attend over pos[b] + 1 tokens (see sq.h)."""
    kcs, vcs = kc.struct(), vc.struct()
    _check(lib().sq_decode_step(_ptr(calib_k), _ptr(calib_v), ctypes.byref(kcs), ctypes.byref(vcs), _ptr(k_new),
                                _ptr(v_new), _ptr(q), DTYPE_CODE[q.dtype], _ptr(pos), batch, n_q_heads, n_kv_heads, d,
                                max_ctx, float(scale), _ptr(out), DTYPE_CODE[out.dtype], _ptr(scores_out), _ptr(ws),
                                ws.numel() * ws.element_size() if ws is not None else 0, _ptr(flags),
                                _stream(stream)), "sq_decode_step")


def sq_attn_decode_noalloc(calib_k, calib_v, kc, vc, seq_lens, batch, n_q_heads, n_kv_heads, d, max_ctx, q, scale,
                           out, scores_out=None, flags=None, stream=None):
    """sq_attn_decode with the library's fixed scratch array instead of a workspace
    (for callers that cannot allocate device memory; see sq.h)."""
    kcs, vcs = kc.struct(), vc.struct()
    _check(lib().sq_attn_decode_noalloc(_ptr(calib_k), _ptr(calib_v), ctypes.byref(kcs), ctypes.byref(vcs),
                                        _ptr(seq_lens), batch, n_q_heads, n_kv_heads, d, max_ctx, _ptr(q),
                                        DTYPE_CODE[q.dtype], float(scale), _ptr(out), DTYPE_CODE[out.dtype],
                                        _ptr(scores_out), _ptr(flags), _stream(stream)), "sq_attn_decode_noalloc")


def sq_wait_selftest(limit_us, flags, stream=None):
    """One GPU thread waits on an mbarrier nothing arrives on for limit_us
    microseconds with the library's bounded-wait helper, then sets
    SQ_FLAG_TIMEOUT in flags (see sq.h)."""
    _check(lib().sq_wait_selftest(int(limit_us), _ptr(flags), _stream(stream)), "sq_wait_selftest")


# --------------------------------------------------------------------------- the paged 4-bit cache
# A decode step of one sequence takes the GPU about ten microseconds, so these bindings
# spend few on the host: addresses go as plain integers, and the structures of a cache
# and of a rotation table are made once and again when a field of theirs is set.
class _Described:
    """Keeps what struct() made of its fields until one of them is set, or a tensor of them moves or changes form."""

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__["_made"] = None

    def __getstate__(self):                       # what is kept names addresses: a copy makes its own
        return {**self.__dict__, "_made": None}

    def described(self):
        """(reference to the structure, the structure, its tensors' device, what it was made of); an address names its
        device too."""
        made, where = self._made, self.where()
        if made is None or made[3] != where:
            struct = self.struct()
            made = self.__dict__["_made"] = (ctypes.byref(struct), struct, self.device(), where)
        return made

    def ref(self):
        return self.described()[0]


@dataclass
class PagedKV4(_Described):
    """Caller-owned pool of pages and the page table of a batch (see sq_kv4_cache in sq.h)."""

    pages: torch.Tensor          # uint8 [n_pages, n_kv, page_tokens / 16, 16 d + 128]
    table: torch.Tensor          # int32 [batch, pages_per_row]; the rows may be strided, not share memory
    n_kv: int
    d: int
    page_tokens: int

    def __post_init__(self):
        self.check()

    def check(self):
        shape = (self.pages.shape[0], self.n_kv, self.page_tokens // 16, 16 * self.d + 128)
        if self.pages.dtype != torch.uint8 or tuple(self.pages.shape) != shape or not self.pages.is_contiguous():
            raise ValueError(f"pages: a contiguous uint8 tensor of shape {shape} is wanted")
        if self.table.dtype != torch.int32 or self.table.dim() != 2 or (self.table.shape[1] > 1
                                                                        and self.table.stride(1) != 1):
            raise ValueError("table: an int32 tensor [batch, pages_per_row] with rows of stride 1 is wanted")
        if self.table.shape[0] > 1 and self.table.stride(0) < self.table.shape[1]:
            raise ValueError("table: rows that share memory (an expanded table?) are not taken, make it contiguous")

    @property
    def batch(self) -> int:
        return self.table.shape[0]

    def device(self):
        return _kv4_device(self.pages.get_device(), self.pages, self.table)

    def where(self):
        p, t = self.pages, self.table
        return p.data_ptr(), p.numel(), p.is_contiguous(), t.data_ptr(), t.shape, t.stride(), t.dtype

    def struct(self) -> sq_kv4_cache:
        self.check()
        batch, per_row = self.table.shape
        return sq_kv4_cache(self.pages.data_ptr(), self.table.data_ptr(), self.pages.shape[0],
                            self.table.stride(0) if batch > 1 else per_row, batch, per_row, self.n_kv, self.d,
                            self.page_tokens)


@dataclass
class Rope(_Described):
    """Rotation table float32 [n_pos, rot_dim]: cosines of rot_dim / 2 angles, then their sines."""

    table: torch.Tensor
    interleaved: bool = False

    def __post_init__(self):
        self.check()

    def check(self):
        if self.table.dtype != torch.float32 or self.table.dim() != 2 or not self.table.is_contiguous():
            raise ValueError("rotation table: a contiguous float32 tensor [n_pos, rot_dim] is wanted")

    def device(self):
        return self.table.get_device()

    def where(self):
        t = self.table
        return t.data_ptr(), t.shape, t.is_contiguous(), t.dtype

    def struct(self) -> sq_rope:
        self.check()
        return sq_rope(self.table.data_ptr(), self.table.shape[0], self.table.shape[1], int(self.interleaved))


def rope_table(n_pos: int, rot_dim: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """The rotation table of angles pos * theta^(-2i / rot_dim), formed in float64."""
    i = torch.arange(0, rot_dim, 2, device=device, dtype=torch.float64)
    ang = torch.arange(n_pos, device=device, dtype=torch.float64)[:, None] * theta ** (-i / rot_dim)
    return torch.cat([torch.cos(ang), torch.sin(ang)], 1).float()


def sq_kv4_page_bytes(n_kv, d, page_tokens) -> int:
    return lib().sq_kv4_page_bytes(n_kv, d, page_tokens)


def alloc_kv4(n_pages, n_kv, d, page_tokens, table, device="cuda") -> PagedKV4:
    """A zeroed pool of n_pages pages behind the given page table."""
    if sq_kv4_page_bytes(n_kv, d, page_tokens) == 0:
        raise ValueError(f"unsupported paged cache: {n_kv} heads, head_dim {d}, {page_tokens} tokens a page")
    return PagedKV4(torch.zeros(n_pages, n_kv, page_tokens // 16, 16 * d + 128, dtype=torch.uint8, device=device),
                    table, n_kv, d, page_tokens)


def _kv4_device(dev, *tensors):
    """dev, the index of the device that every tensor (or None) is on."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"every tensor must be on the current device, got some on {t.device} and on device {dev}")
    return dev


def _kv4_call(cache, rope, stream, *tensors):
    """(the cache's reference and structure, the rotation's reference, the call's stream as an integer). Its tensors live on
    the current device: a kernel cannot read the others."""
    ref, made, dev, _ = cache.described()
    turn = None
    if rope:
        turn, _, on, _ = rope.described()
        if on != dev:
            raise ValueError(f"every tensor must be on the current device, got some on {rope.table.device} and on device {dev}")
    _kv4_device(dev, *tensors)
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"every tensor must be on the current device, got some on {cache.pages.device}")
    return ref, made, turn, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _kv4_ints(name, t, n):
    if t.numel() != n or t.dim() != 1 or t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 tensor of {n} elements is wanted")
    return t.data_ptr()


def _kv4_heads(name, t, heads, d, rows=None, dtype=None):
    """Address, token stride and head stride of a tensor [rows, heads, d] (heads None: any number); the stride of an
    axis of one element, which may be any number, is 0."""
    if t.dim() == 3:
        n, h, e = t.shape
        s0, s1, s2 = t.stride()
        if ((heads is None or h == heads) and e == d and s2 == 1 and t.dtype in DTYPE_CODE
                and (rows is None or n == rows) and (dtype is None or t.dtype == dtype)):
            return t.data_ptr(), s0 if n > 1 else 0, s1 if h > 1 else 0
    raise ValueError(f"{name}: a tensor [{'tokens' if rows is None else rows}, {'heads' if heads is None else heads}, {d}] "
                     f"of stride 1 along the last axis{'' if dtype is None else f' and type {dtype}'} is wanted")


def _kv4_apart(name, n, h, d, s0, s1):
    """Refuses an output [n, h, d] whose rows share memory: each stride steps over all that the smaller ones reach."""
    if (h == 1 or s1 >= d) and (n < 2 or s0 >= (h - 1) * s1 + d):
        return
    reach = d
    for stride, count in sorted(x for x in ((s0, n), (s1, h)) if x[1] > 1):
        if stride < reach:
            raise ValueError(f"{name}: an output whose rows share no memory is wanted")
        reach += (count - 1) * stride


def _kv4_out(out, lse, q):
    """Addresses of the outputs."""
    shape = q.shape
    if out.shape != shape or not out.is_contiguous() or out.dtype not in DTYPE_CODE:
        raise ValueError("out: a contiguous tensor of q's shape is wanted")
    if lse is None:
        return out.data_ptr(), None
    if lse.dtype != torch.float32 or lse.shape != shape[:2] or not lse.is_contiguous():
        raise ValueError("lse: a contiguous float32 tensor [tokens, n_q_heads] is wanted")
    return out.data_ptr(), lse.data_ptr()


def _kv4_at(flags):
    if flags is None:
        return None
    if flags.element_size() != 4 or flags.numel() < 1:
        raise ValueError("flags: a 32-bit word is wanted")
    return flags.data_ptr()


def _kv4_bytes(ws):
    if ws is None:
        return None, 0
    if not ws.is_contiguous():
        raise ValueError("ws: a contiguous tensor is wanted")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def sq_kv4_append(cache, k, v, start, cu=None, rope=None, flags=None, stream=None):
    """Append k, v [tokens, n_kv, d] (any strides but the last axis's) at positions start[b] + i (see sq.h)."""
    ref, made, turn, st = _kv4_call(cache, rope, stream, k, v, start, cu, flags)
    kp, k0, k1 = _kv4_heads("k", k, cache.n_kv, cache.d)
    n = k.shape[0]
    vp, v0, v1 = _kv4_heads("v", v, cache.n_kv, cache.d, n, k.dtype)
    batch = made.batch
    at = _kv4_ints("start", start, batch)
    cu = None if cu is None else _kv4_ints("cu", cu, batch + 1)
    _check(lib().sq_kv4_append(ref, kp, vp, DTYPE_CODE[k.dtype], k0, k1, v0, v1, n, cu, at, turn, _kv4_at(flags), st),
           "sq_kv4_append")


def sq_kv4_read(cache, start, cu, k_out, v_out, flags=None, stream=None):
    """The tokens at positions start[b] + i, as the cache holds them, into k_out, v_out [tokens, n_kv, d]."""
    ref, made, _, st = _kv4_call(cache, None, stream, k_out, v_out, start, cu, flags)
    kp, k0, k1 = _kv4_heads("k_out", k_out, cache.n_kv, cache.d)
    n = k_out.shape[0]
    vp, v0, v1 = _kv4_heads("v_out", v_out, cache.n_kv, cache.d, n, k_out.dtype)
    _kv4_apart("k_out", n, cache.n_kv, cache.d, k0, k1)
    _kv4_apart("v_out", n, cache.n_kv, cache.d, v0, v1)
    batch = made.batch
    at = _kv4_ints("start", start, batch)
    cu = None if cu is None else _kv4_ints("cu", cu, batch + 1)
    _check(lib().sq_kv4_read(ref, kp, vp, DTYPE_CODE[k_out.dtype], k0, k1, v0, v1, n, cu, at, _kv4_at(flags), st),
           "sq_kv4_read")


def sq_kv4_attn_workspace(batch, n_q_heads, n_kv_heads, d, max_ctx) -> int:
    return lib().sq_kv4_attn_workspace(batch, n_q_heads, n_kv_heads, d, max_ctx)


def sq_kv4_attn_decode(cache, seq_lens, q, scale, out, max_ctx, ws, rope=None, window=0, lse=None, flags=None,
                       stream=None):
    """Attention of q [batch, n_q_heads, d] over the first seq_lens[b] tokens of every sequence (see sq.h)."""
    ref, made, turn, st = _kv4_call(cache, rope, stream, q, out, seq_lens, lse, ws, flags)
    batch = made.batch
    qp, q0, q1 = _kv4_heads("q", q, None, cache.d, batch)
    op, lp = _kv4_out(out, lse, q)
    wp, wn = _kv4_bytes(ws)
    _check(lib().sq_kv4_attn_decode(ref, _kv4_ints("seq_lens", seq_lens, batch), q.shape[1], max_ctx, qp,
                                    DTYPE_CODE[q.dtype], q0, q1, turn, scale, window, op,
                                    DTYPE_CODE[out.dtype], lp, wp, wn, _kv4_at(flags), st), "sq_kv4_attn_decode")


def sq_kv4_decode_step(cache, k, v, q, pos, scale, out, max_ctx, ws, rope=None, window=0, lse=None, flags=None,
                       stream=None):
    """Append one token a sequence at pos[b], then attend over pos[b] + 1 tokens (see sq.h)."""
    ref, made, turn, st = _kv4_call(cache, rope, stream, k, v, q, out, pos, lse, ws, flags)
    batch, n_kv, d, dtype = made.batch, cache.n_kv, cache.d, q.dtype
    qp, q0, q1 = _kv4_heads("q", q, None, d, batch)
    kp, k0, k1 = _kv4_heads("k", k, n_kv, d, batch, dtype)
    vp, v0, v1 = _kv4_heads("v", v, n_kv, d, batch, dtype)
    op, lp = _kv4_out(out, lse, q)
    wp, wn = _kv4_bytes(ws)
    _check(lib().sq_kv4_decode_step(ref, kp, vp, qp, DTYPE_CODE[dtype], k0, k1, v0, v1, q0, q1,
                                    _kv4_ints("pos", pos, batch), q.shape[1], max_ctx, turn,
                                    scale, window, op, DTYPE_CODE[out.dtype], lp, wp, wn, _kv4_at(flags), st),
           "sq_kv4_decode_step")


def sq_kv4_attn_prefill_workspace(batch, n_q_heads, n_kv_heads, d, n_tok) -> int:
    return lib().sq_kv4_attn_prefill_workspace(batch, n_q_heads, n_kv_heads, d, n_tok)


def sq_kv4_attn_prefill(cache, start, cu, q, scale, out, ws, rope=None, window=0, lse=None, flags=None, stream=None):
    """Causal attention of q [tokens, n_q_heads, d], token cu[b] + i at position start[b] + i (see sq.h)."""
    ref, made, turn, st = _kv4_call(cache, rope, stream, q, out, start, cu, lse, ws, flags)
    batch = made.batch
    qp, q0, q1 = _kv4_heads("q", q, None, cache.d)
    op, lp = _kv4_out(out, lse, q)
    wp, wn = _kv4_bytes(ws)
    _check(lib().sq_kv4_attn_prefill(ref, _kv4_ints("cu", cu, batch + 1), _kv4_ints("start", start, batch),
                                     q.shape[1], q.shape[0], qp, DTYPE_CODE[q.dtype], q0, q1, turn,
                                     scale, window, op, DTYPE_CODE[out.dtype], lp, wp, wn, _kv4_at(flags), st),
           "sq_kv4_attn_prefill")
