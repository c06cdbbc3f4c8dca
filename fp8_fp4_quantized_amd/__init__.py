"""Python binding of ``libkvc.so``: the MI355X (gfx950) compressed-KV store
and gather for DeepSeek-V4.1 low-ratio layers (C ABI in ``include/kvc.h``).

Argument marshalling only.  Every step of the path runs in the HIP kernels of
``libkvc.so``; PyTorch provides device memory and the current stream.  There
is no fallback: importing this package without the built library raises.

Function names are those of the C ABI.  Tensors are CUDA (HIP) tensors:
bf16 rows may be ``torch.bfloat16`` or ``int16``/``uint16`` bit patterns;
caches are ``uint8`` tensors ``[num_pages, page_stride]``.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass

import torch  # noqa: F401  (loads the HIP runtime that libkvc.so then binds to)

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkvc.so")

KVC_OK, KVC_EINVAL, KVC_EUNSUPPORTED, KVC_ELAUNCH = 0, -1, -2, -3
LAYOUT_V4, LAYOUT_V41, LAYOUT_V41_FP4 = 0, 1, 2
LAYOUTS = {"V4": LAYOUT_V4, "V41": LAYOUT_V41, "V41_FP4": LAYOUT_V41_FP4}
MODE_PREFILL, MODE_DECODE, MODE_VERIFY = 0, 1, 2
STATUS_ID_RANGE, STATUS_PAGE_RANGE, STATUS_PT_RANGE = 1, 2, 4
STATUS_LATENT_RANGE, STATUS_POS_RANGE, STATUS_REQ_RANGE = 8, 16, 32
STATUS_TOKEN_RANGE = 64
STATUS_NO_PAGE = 128
ROPE_SCALING = {"none": 0, "linear": 1, "base": 2, "parts": 3}
WEIGH_FEW = 128        # (token, head) pairs a slot may have without a workspace
SELECT_NO_WORKSPACE = 32768   # weights a row may hold without a workspace


class KvcError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"kvc error {code}: {msg}")
        self.code = code


class kvc_layout_info(C.Structure):
    _fields_ = [("data_bytes", C.c_int32), ("scale_bytes", C.c_int32),
                ("row_bytes", C.c_int32), ("group", C.c_int32), ("quant_dims", C.c_int32)]


class kvc_cache(C.Structure):
    _fields_ = [("base", C.c_void_p), ("layout", C.c_int32), ("page_size", C.c_int32),
                ("page_stride", C.c_int64), ("num_pages", C.c_int64)]


class kvc_compress_args(C.Structure):
    _fields_ = [
        ("ratio", C.c_int32), ("mode", C.c_int32),
        ("kv", C.c_void_p), ("kv_stride", C.c_int64),
        ("score", C.c_void_p), ("score_stride", C.c_int64),
        ("num_slots", C.c_int32),
        ("offsets", C.c_void_p), ("start_pos", C.c_void_p),
        ("page_table", C.c_void_p), ("pt_stride", C.c_int64),
        ("out_loc", C.c_void_p), ("state", C.c_void_p),
        ("norm_w", C.c_void_p), ("eps", C.c_float),
        ("freqs", C.c_void_p), ("max_pos", C.c_int64),
        ("latent_out", C.c_void_p), ("latent_stride", C.c_int64), ("max_out_rows", C.c_int64),
        ("prequant_out", C.c_void_p), ("prequant_stride", C.c_int64),
        ("cache", kvc_cache), ("status", C.c_void_p),
        ("draft_len", C.c_int32), ("ring_slots", C.c_int32),
        ("dcp_world", C.c_int32), ("dcp_rank", C.c_int32), ("dcp_interleave", C.c_int32),
        ("tile_rows", C.c_int32), ("kv_rows", C.c_int64), ("pt_width", C.c_int64),
    ]


class kvc_slot_map_args(C.Structure):
    _fields_ = [
        ("ratio", C.c_int32), ("page_size", C.c_int32), ("num_pages", C.c_int64),
        ("num_slots", C.c_int32), ("token_stride", C.c_int32),
        ("lens", C.c_void_p), ("new_lens", C.c_void_p), ("depth", C.c_void_p),
        ("page_table", C.c_void_p), ("pt_stride", C.c_int64), ("pt_width", C.c_int64),
        ("free_pages", C.c_void_p), ("n_free", C.c_int64), ("max_tokens", C.c_int64),
        ("offsets", C.c_void_p), ("start_pos", C.c_void_p), ("out_loc", C.c_void_p),
        ("positions", C.c_void_p), ("token_to_req", C.c_void_p), ("totals", C.c_void_p),
        ("status", C.c_void_p),
    ]


class kvc_attend_args(C.Structure):
    _fields_ = [
        ("ratio", C.c_int32), ("num_heads", C.c_int32), ("num_slots", C.c_int32),
        ("draft_len", C.c_int32),
        ("q", C.c_void_p), ("q_stride", C.c_int64), ("q_head_stride", C.c_int64),
        ("q_rows", C.c_int64),
        ("offsets", C.c_void_p), ("start_pos", C.c_void_p),
        ("page_table", C.c_void_p), ("pt_stride", C.c_int64), ("pt_width", C.c_int64),
        ("tree", C.c_void_p), ("scale", C.c_float), ("sink", C.c_void_p),
        ("out", C.c_void_p), ("out_stride", C.c_int64), ("out_head_stride", C.c_int64),
        ("lse", C.c_void_p), ("cache", kvc_cache),
        ("workspace", C.c_void_p), ("workspace_bytes", C.c_int64), ("status", C.c_void_p),
    ]


class kvc_rope_table_args(C.Structure):
    _fields_ = [
        ("freqs", C.c_void_p), ("n", C.c_int64), ("first", C.c_int64), ("rot_dim", C.c_int32),
        ("scaling", C.c_int32), ("base", C.c_double), ("factor", C.c_double),
        ("original", C.c_double), ("beta_fast", C.c_double), ("beta_slow", C.c_double),
        ("mscale", C.c_double),
    ]


class kvc_rope_args(C.Structure):
    _fields_ = [
        ("dtype", C.c_int32), ("num_heads", C.c_int32), ("head_dim", C.c_int32),
        ("rot_dim", C.c_int32), ("offset", C.c_int32), ("half", C.c_int32),
        ("transpose", C.c_int32), ("tokens", C.c_int64),
        ("x", C.c_void_p), ("x_stride", C.c_int64), ("x_head_stride", C.c_int64),
        ("out", C.c_void_p), ("out_stride", C.c_int64), ("out_head_stride", C.c_int64),
        ("positions", C.c_void_p), ("freqs", C.c_void_p), ("max_pos", C.c_int64),
        ("status", C.c_void_p),
    ]


class kvc_weigh_args(C.Structure):
    _fields_ = [
        ("ratio", C.c_int32), ("num_heads", C.c_int32), ("num_slots", C.c_int32),
        ("draft_len", C.c_int32),
        ("q", C.c_void_p), ("q_stride", C.c_int64), ("q_head_stride", C.c_int64),
        ("q_rows", C.c_int64), ("lse", C.c_void_p),
        ("offsets", C.c_void_p), ("start_pos", C.c_void_p),
        ("page_table", C.c_void_p), ("pt_stride", C.c_int64), ("pt_width", C.c_int64),
        ("tree", C.c_void_p), ("scale", C.c_float), ("decay", C.c_float),
        ("prev", C.c_void_p), ("prev_stride", C.c_int64),
        ("weights", C.c_void_p), ("w_stride", C.c_int64), ("w_width", C.c_int64),
        ("cache", kvc_cache),
        ("workspace", C.c_void_p), ("workspace_bytes", C.c_int64), ("status", C.c_void_p),
    ]


class kvc_evict_args(C.Structure):
    _fields_ = [
        ("ratio", C.c_int32), ("num_slots", C.c_int32), ("lens", C.c_void_p),
        ("weights", C.c_void_p), ("w_stride", C.c_int64), ("w_width", C.c_int64),
        ("budget", C.c_int32), ("first", C.c_int32), ("recent", C.c_int32),
        ("budgets", C.c_void_p),
        ("kept", C.c_void_p), ("kept_stride", C.c_int64), ("kept_width", C.c_int64),
        ("counts", C.c_void_p), ("kept_weights", C.c_void_p), ("kw_stride", C.c_int64),
        ("workspace", C.c_void_p), ("workspace_bytes", C.c_int64), ("status", C.c_void_p),
    ]


class kvc_compact_args(C.Structure):
    _fields_ = [
        ("ratio", C.c_int32), ("num_slots", C.c_int32), ("lens", C.c_void_p),
        ("kept", C.c_void_p), ("kept_stride", C.c_int64), ("kept_width", C.c_int64),
        ("counts", C.c_void_p),
        ("page_table", C.c_void_p), ("pt_stride", C.c_int64), ("pt_width", C.c_int64),
        ("free_pages", C.c_void_p), ("n_free", C.c_int64),
        ("new_table", C.c_void_p), ("nt_stride", C.c_int64), ("new_lens", C.c_void_p),
        ("kept_weights", C.c_void_p), ("kw_stride", C.c_int64),
        ("weights", C.c_void_p), ("w_stride", C.c_int64), ("w_width", C.c_int64),
        ("freed", C.c_void_p), ("freed_cap", C.c_int64), ("totals", C.c_void_p),
        ("cache", kvc_cache), ("status", C.c_void_p),
    ]


# symbol -> (restype, argtypes); the same list as include/kvc.h
_VP, _I32, _I64 = C.c_void_p, C.c_int32, C.c_int64
SIGNATURES = {
    "kvc_layout_query": (C.c_int, [_I32, C.POINTER(kvc_layout_info)]),
    "kvc_store_rows": (C.c_int, [C.POINTER(kvc_cache), _VP, _I64, _VP, _I64, _VP, _VP]),
    "kvc_store_rows_rope": (C.c_int, [C.POINTER(kvc_cache), _VP, _I64, _VP, _VP, _I64, _VP, _I64,
                                      _VP, _VP]),
    "kvc_dcp_filter_ids": (C.c_int, [_VP, _I64, _I32, _I64, _VP, _I32, _VP, _I64, _I64, _VP, _I32,
                                     _I64, _I32, _I32, _I32, _VP, _I64, _VP, _VP, _VP]),
    "kvc_compress_store": (C.c_int, [C.POINTER(kvc_compress_args), _VP]),
    "kvc_dequant_gather": (C.c_int, [C.POINTER(kvc_cache), _VP, _I64, _VP, _I64, _VP, _I64, _VP, _VP]),
    "kvc_kvbuf_create": (_VP, []),
    "kvc_kvbuf_destroy": (None, [_VP]),
    "kvc_kvbuf_forget": (None, [_VP]),
    "kvc_kvbuf_begin_forward": (None, [_VP]),
    "kvc_dequant_gather_reuse": (C.c_int, [_VP, C.POINTER(kvc_cache), _VP, _I64, _VP, _I64, _VP,
                                           _I64, _VP, _VP, _VP]),
    "kvc_slot_map": (C.c_int, [C.POINTER(kvc_slot_map_args), _VP]),
    "kvc_attend_workspace": (C.c_int, [_I32, _I64, _I32, C.POINTER(_I64)]),
    "kvc_attend_prefill": (C.c_int, [C.POINTER(kvc_attend_args), _VP]),
    "kvc_attend_tree": (C.c_int, [C.POINTER(kvc_attend_args), _VP]),
    "kvc_rope_table": (C.c_int, [C.POINTER(kvc_rope_table_args), _VP]),
    "kvc_rope_rows": (C.c_int, [C.POINTER(kvc_rope_args), _VP]),
    "kvc_weigh_workspace": (C.c_int, [C.POINTER(_I64)]),
    "kvc_weigh_prefill": (C.c_int, [C.POINTER(kvc_weigh_args), _VP]),
    "kvc_weigh_tree": (C.c_int, [C.POINTER(kvc_weigh_args), _VP]),
    "kvc_evict_workspace": (C.c_int, [_I32, _I64, C.POINTER(_I64)]),
    "kvc_evict_select": (C.c_int, [C.POINTER(kvc_evict_args), _VP]),
    "kvc_cache_compact": (C.c_int, [C.POINTER(kvc_compact_args), _VP]),
    "kvc_last_error": (C.c_char_p, []),
    "kvc_version": (C.c_int, []),
}

_lib = None


def lib():
    """The loaded ``libkvc.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m fp8_fp4_quantized_amd.build` or __graft_entry__.build()")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


lib()   # fail loudly at import when the HIP library is missing


def _check(rc: int) -> None:
    if rc != KVC_OK:
        raise KvcError(rc, lib().kvc_last_error().decode())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


_INT32 = torch.int32
_I32_T = (_INT32,)
_F32_T = (torch.float32,)
_B16_T = (torch.bfloat16, torch.int16, torch.uint16)


def _dense(t, dtypes, name: str) -> int:
    """Pointer of a contiguous device tensor of one of ``dtypes``."""
    if not (t.is_cuda and t.dtype in dtypes and t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous device tensor of {dtypes}, got "
                         f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _rows(t, dtypes, name: str) -> int:
    """Pointer of a 2-D device tensor of ``dtypes`` whose rows are contiguous
    (any row stride)."""
    if not (t.is_cuda and t.dtype in dtypes and t.dim() == 2 and t.stride(1) == 1):
        raise ValueError(f"{name}: expected a 2-D device tensor of {dtypes} with contiguous "
                         f"rows, got {t.dtype} {tuple(t.shape)} strides {t.stride()}")
    return t.data_ptr()


def _opt(t, check, dtypes, name: str) -> int | None:
    return None if t is None else check(t, dtypes, name)


def _need(ok: bool, msg: str) -> None:
    """A size the library would trust (it reads or writes that many entries)
    that the tensor does not have: refused before anything is launched."""
    if not ok:
        raise ValueError(msg)


def _rows_of(t, name: str, min_cols: int = 512) -> int:
    """Row count of a 2-D row buffer holding at least ``min_cols`` columns."""
    _need(t.dim() == 2, f"{name}: expected a 2-D tensor, got shape {tuple(t.shape)}")
    _need(t.shape[1] >= min_cols, f"{name}: rows hold {t.shape[1]} columns, need {min_cols}")
    return t.shape[0]


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


@dataclass
class Cache:
    """A paged cache: ``data`` is a uint8 tensor ``[num_pages, page_stride]``."""
    data: torch.Tensor
    layout: int
    page_size: int

    def desc(self) -> kvc_cache:
        assert self.data.dtype == torch.uint8 and self.data.dim() == 2 and self.data.is_contiguous()
        lay = LAYOUTS[self.layout] if isinstance(self.layout, str) else int(self.layout)
        return kvc_cache(self.data.data_ptr(), lay, self.page_size,
                         self.data.shape[1], self.data.shape[0])


# --------------------------------------------------------------------- calls
def kvc_version() -> int:
    return lib().kvc_version()


def kvc_last_error() -> str:
    return lib().kvc_last_error().decode()


def kvc_layout_query(layout) -> kvc_layout_info:
    info = kvc_layout_info()
    lay = LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    _check(lib().kvc_layout_query(lay, C.byref(info)))
    return info


def kvc_store_rows(cache: Cache, rows: torch.Tensor, out_loc: torch.Tensor,
                   status: torch.Tensor | None = None, stream=None) -> None:
    """Quantize bf16 ``rows [n, >=512]`` into ``cache`` at ``out_loc [n]``."""
    n = _rows_of(rows, "rows")
    _need(out_loc.numel() >= n, f"out_loc: {out_loc.numel()} entries for {n} rows")
    d = cache.desc()
    _check(lib().kvc_store_rows(C.byref(d), _rows(rows, _B16_T, "rows"), rows.stride(0),
                                _dense(out_loc, _I32_T, "out_loc"), rows.shape[0],
                                _opt(status, _dense, _I32_T, "status"), _stream(stream)))


def kvc_store_rows_rope(cache: Cache, rows: torch.Tensor, positions: torch.Tensor,
                        freqs: torch.Tensor, out_loc: torch.Tensor,
                        status: torch.Tensor | None = None, stream=None) -> None:
    """Rotate the rope dims of bf16 ``rows [n, >=512]`` at ``positions [n]``
    (table ``freqs [max_pos, 64]`` fp32) and quantize them at ``out_loc``."""
    n = _rows_of(rows, "rows")
    _need(out_loc.numel() >= n, f"out_loc: {out_loc.numel()} entries for {n} rows")
    _need(positions.numel() >= n, f"positions: {positions.numel()} entries for {n} rows")
    _need(freqs.dim() == 2 and freqs.shape[1] == 64, f"freqs: shape {tuple(freqs.shape)}, "
                                                     "expected [max_pos, 64]")
    d = cache.desc()
    _check(lib().kvc_store_rows_rope(C.byref(d), _rows(rows, _B16_T, "rows"), rows.stride(0),
                                     _dense(positions, _I32_T, "positions"),
                                     _dense(freqs, _F32_T, "freqs"), freqs.shape[0],
                                     _dense(out_loc, _I32_T, "out_loc"), rows.shape[0],
                                     _opt(status, _dense, _I32_T, "status"), _stream(stream)))


def kvc_dcp_filter_ids(ids: torch.Tensor, token_to_req: torch.Tensor, block_table: torch.Tensor,
                       out_slots: torch.Tensor, out_lens: torch.Tensor, *, page_size: int,
                       num_pages: int, world: int, rank: int, interleave: int,
                       valid: torch.Tensor | None = None, status: torch.Tensor | None = None,
                       stream=None) -> None:
    """This rank's share of global compressed ids ``[T, k]``: physical slots
    compacted into ``out_slots [T, k]`` (-1 tail), counts into ``out_lens [T]``."""
    _need(ids.dim() == 2, f"ids: expected [T, k], got shape {tuple(ids.shape)}")
    T, k = ids.shape
    _need(token_to_req.numel() >= T, f"token_to_req: {token_to_req.numel()} entries for {T} rows")
    _need(valid is None or valid.numel() >= T, f"valid: fewer than {T} entries")
    _need(out_slots.dim() == 2 and out_slots.shape[0] >= T and out_slots.shape[1] >= k,
          f"out_slots: shape {tuple(out_slots.shape)}, need at least [{T}, {k}]")
    _need(out_lens.numel() >= T, f"out_lens: {out_lens.numel()} entries for {T} rows")
    _need(block_table.dim() == 2, f"block_table: expected [n_req, pages], got "
                                  f"{tuple(block_table.shape)}")
    _check(lib().kvc_dcp_filter_ids(_rows(ids, _I32_T, "ids"), T, k, ids.stride(0),
                                    _dense(token_to_req, _I32_T, "token_to_req"),
                                    block_table.shape[0], _rows(block_table, _I32_T, "block_table"),
                                    block_table.stride(0), block_table.shape[1],
                                    _opt(valid, _dense, _I32_T, "valid"),
                                    page_size, num_pages, world, rank, interleave,
                                    _rows(out_slots, _I32_T, "out_slots"), out_slots.stride(0),
                                    _dense(out_lens, _I32_T, "out_lens"),
                                    _opt(status, _dense, _I32_T, "status"), _stream(stream)))


def kvc_dequant_gather(cache: Cache, page_table: torch.Tensor | None, ids: torch.Tensor,
                       out: torch.Tensor, status: torch.Tensor | None = None, stream=None) -> None:
    """``out[j] = bf16 row of ids[j]`` (through ``page_table`` when given)."""
    _need(_rows_of(out, "out") >= ids.numel(), f"out: {out.shape[0]} rows for {ids.numel()} ids")
    d = cache.desc()
    n_pages = 0 if page_table is None else page_table.numel()
    _check(lib().kvc_dequant_gather(C.byref(d), _opt(page_table, _dense, _I32_T, "page_table"),
                                    n_pages, _dense(ids, _I32_T, "ids"), ids.numel(),
                                    _rows(out, _B16_T, "out"), out.stride(0),
                                    _opt(status, _dense, _I32_T, "status"), _stream(stream)))


class KVBuf:
    """Dequant-reuse head (``kvc_kvbuf``): a gather whose arguments match the
    last one it ran is skipped."""

    def __init__(self):
        self._h = lib().kvc_kvbuf_create()
        if not self._h:
            raise MemoryError("kvc_kvbuf_create")

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h and _lib is not None:
            _lib.kvc_kvbuf_destroy(h)

    def forget(self) -> None:
        lib().kvc_kvbuf_forget(self._h)

    def begin_forward(self) -> None:
        lib().kvc_kvbuf_begin_forward(self._h)

    def kvc_dequant_gather_reuse(self, cache: Cache, page_table, ids, out, status=None,
                                 stream=None) -> bool:
        _need(_rows_of(out, "out") >= ids.numel(),
              f"out: {out.shape[0]} rows for {ids.numel()} ids")
        d = cache.desc()
        hit = C.c_int32(0)
        n_pages = 0 if page_table is None else page_table.numel()
        _check(lib().kvc_dequant_gather_reuse(
            self._h, C.byref(d), _opt(page_table, _dense, _I32_T, "page_table"), n_pages,
            _dense(ids, _I32_T, "ids"), ids.numel(), _rows(out, _B16_T, "out"), out.stride(0),
            _opt(status, _dense, _I32_T, "status"), C.byref(hit), _stream(stream)))
        return bool(hit.value)


def _compress_args(*, ratio: int, mode: int, kv: torch.Tensor, score: torch.Tensor | None,
                       start_pos: torch.Tensor, cache: Cache, norm_w: torch.Tensor, eps: float,
                       freqs: torch.Tensor, latent_out: torch.Tensor, max_out_rows: int | None = None,
                       offsets: torch.Tensor | None = None, page_table: torch.Tensor | None = None,
                       out_loc: torch.Tensor | None = None, state: torch.Tensor | None = None,
                       prequant_out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                       draft_len: int = 1, ring_slots: int = 1, dcp_world: int = 1,
                       dcp_rank: int = 0, dcp_interleave: int = 1,
                       tile_rows: int = 0) -> kvc_compress_args:
    """The argument block of kvc_compress_store (every check done here).
    The fused compressor.  ``kv``/``score`` are 2-D views whose row stride
    is passed through (a fused ``|kv|score|`` buffer ``proj [T, 1024]`` is
    ``kv=proj[:, :512], score=proj[:, 512:]``).  ``state`` is ``[S,
    ring_slots, 2, 512]`` bf16 (``[S, 2, 512]`` for one entry).  A page
    table may be a column slice of a wider table: its width bounds the
    logical pages, its row stride addresses the rows."""
    S = start_pos.numel()
    D = draft_len if mode == MODE_VERIFY else 1
    kv_rows = _rows_of(kv, "kv")
    if score is not None:
        kv_rows = min(kv_rows, _rows_of(score, "score"))
    lat_rows = _rows_of(latent_out, "latent_out")
    if max_out_rows is None:
        max_out_rows = lat_rows
    _need(0 <= max_out_rows <= lat_rows,
          f"max_out_rows {max_out_rows}: latent_out holds {lat_rows} rows")
    _need(prequant_out is None or _rows_of(prequant_out, "prequant_out") >= max_out_rows,
          f"prequant_out: fewer than max_out_rows = {max_out_rows} rows")
    if mode != MODE_PREFILL:
        _need(max_out_rows >= S * D, f"max_out_rows {max_out_rows}: decode / verify write "
                                     f"latent rows up to {S * D}")
        _need(kv_rows >= S * D, f"kv: {kv_rows} token rows for {S} slots x {D} tokens")
        _need(out_loc is None or out_loc.numel() >= S * D,
              f"out_loc: {out_loc.numel() if out_loc is not None else 0} entries for {S * D} "
              "tokens")
    else:
        _need(offsets is not None and offsets.numel() >= 2 * S,
              f"offsets: expected [2, {S}] entries")
    if page_table is not None:
        _need(page_table.dim() == 2 and page_table.shape[0] >= S,
              f"page_table: shape {tuple(page_table.shape)}, need {S} rows")
    if ratio == 2:
        _need(state is not None and state.numel() >= S * max(ring_slots, 1) * 1024,
              f"state: need [{S}, {max(ring_slots, 1)}, 2, 512] bf16")
    _need(norm_w.numel() >= 512, "norm_w: expected 512 entries")
    _need(freqs.dim() == 2 and freqs.shape[1] == 64,
          f"freqs: shape {tuple(freqs.shape)}, expected [max_pos, 64]")
    a = kvc_compress_args()
    a.ratio, a.mode = ratio, mode
    a.kv, a.kv_stride = _rows(kv, _B16_T, "kv"), kv.stride(0)
    a.score = _opt(score, _rows, _B16_T, "score")
    a.score_stride = 0 if score is None else score.stride(0)
    a.num_slots = S
    a.kv_rows = kv_rows
    a.offsets = _opt(offsets, _dense, _I32_T, "offsets")
    a.start_pos = _dense(start_pos, _I32_T, "start_pos")
    a.page_table = _opt(page_table, _rows, _I32_T, "page_table")
    a.pt_stride = 0 if page_table is None else page_table.stride(0)
    a.pt_width = 0 if page_table is None else page_table.shape[1]
    a.out_loc = _opt(out_loc, _dense, _I32_T, "out_loc")
    a.state = _opt(state, _dense, _B16_T, "state")
    a.norm_w, a.eps = _dense(norm_w, _B16_T, "norm_w"), eps
    a.freqs, a.max_pos = _dense(freqs, _F32_T, "freqs"), freqs.shape[0]
    a.latent_out = _rows(latent_out, _B16_T, "latent_out")
    a.latent_stride = latent_out.stride(0)
    a.max_out_rows = max_out_rows
    a.prequant_out = _opt(prequant_out, _rows, _B16_T, "prequant_out")
    a.prequant_stride = 0 if prequant_out is None else prequant_out.stride(0)
    a.cache = cache.desc()
    a.status = _opt(status, _dense, _I32_T, "status")
    a.draft_len, a.ring_slots = draft_len, ring_slots
    a.dcp_world, a.dcp_rank, a.dcp_interleave = dcp_world, dcp_rank, dcp_interleave
    a.tile_rows = tile_rows
    return a


def kvc_compress_store(*, stream=None, **kw) -> None:
    """The fused compressor; keyword arguments as ``_compress_args``."""
    _check(lib().kvc_compress_store(C.byref(_compress_args(**kw)), _stream(stream)))


class Prepared:
    """A call whose arguments were checked and packed once: calling it
    launches on the given stream (default: the current one) with no Python
    work beyond the foreign call.  It keeps the tensors it points to alive;
    their contents may change between calls, their storage must not."""

    __slots__ = ("_fn", "_args", "_keep")

    def __init__(self, fn, args, keep):
        self._fn, self._args, self._keep = fn, args, keep

    def __call__(self, stream=None) -> None:
        _check(self._fn(*self._args, _stream(stream)))


def prepare_compress_store(**kw) -> Prepared:
    """kvc_compress_store with its argument block built once."""
    a = _compress_args(**kw)
    return Prepared(lib().kvc_compress_store, (C.byref(a),), (a, kw))


def prepare_dequant_gather(cache: Cache, page_table: torch.Tensor | None, ids: torch.Tensor,
                           out: torch.Tensor, status: torch.Tensor | None = None) -> Prepared:
    """kvc_dequant_gather with its arguments checked and packed once."""
    _need(_rows_of(out, "out") >= ids.numel(), f"out: {out.shape[0]} rows for {ids.numel()} ids")
    d = cache.desc()
    n_pages = 0 if page_table is None else page_table.numel()
    args = (C.byref(d), _opt(page_table, _dense, _I32_T, "page_table"), n_pages,
            _dense(ids, _I32_T, "ids"), ids.numel(), _rows(out, _B16_T, "out"), out.stride(0),
            _opt(status, _dense, _I32_T, "status"))
    return Prepared(lib().kvc_dequant_gather, args, (d, cache, page_table, ids, out, status))


# ------------------------------------------------------------------ slot map
def _one_device(dev, tensors) -> None:
    """Refuses (name, tensor) pairs that are on another device than ``dev``
    (None: left out)."""
    for name, t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"{name}: on {t.device}, other arguments on {dev}")


def _i32(t, n: int, name: str) -> int | None:
    """Pointer of a contiguous int32 device tensor of at least n entries, or
    None for None."""
    if t is None:
        return None
    if t.dtype is torch.int32 and t.numel() >= n and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    _need(t.numel() >= n, f"{name}: {t.numel()} entries, need {n}")
    return _dense(t, _I32_T, name)


def _i32_on(t, n: int, name: str, index: int) -> int | None:
    """``_i32`` of a tensor that must be on the device of that index."""
    if t is None:
        return None
    # (get_device: one call for being on a device and on which; a slot map's
    # kernel is as short as these checks)
    if (t.dtype is _INT32 and t.get_device() == index and t.is_contiguous()
            and (n == 0 or t.numel() >= n)):
        return t.data_ptr()
    if index >= 0:
        _one_device(torch.device("cuda", index), ((name, t),))
    return _i32(t, n, name)


def _pt_stride(page_table) -> int:
    """Entries between page-table rows (of a single row: its width, whatever
    stride the tensor carries)."""
    return page_table.stride(0) if page_table.shape[0] > 1 else page_table.shape[1]


def _rows_are(t, n: int, name: str) -> None:
    """Refuses a tensor of rows (two dims) that are not of n entries each, whose
    entries the library would take as rows of n; a flat one passes."""
    if t is not None and t.dim() > 1 and (t.dim() != 2 or t.shape[1] != n):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, need rows of {n}")


def _call_on(dev, stream, fn, args) -> None:
    """One call with ``dev`` as the current device, on ``stream`` (default:
    that device's current stream)."""
    index = dev.index
    # (the raw handle: torch.cuda.current_stream would build an object per call)
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        rc = fn(C.byref(args), handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(C.byref(args), handle)
    _check(rc)


def kvc_slot_map(*, ratio: int, page_size: int, num_pages: int, lens: torch.Tensor,
                 page_table: torch.Tensor, free_pages: torch.Tensor,
                 new_lens: torch.Tensor | None = None, token_stride: int = 0,
                 depth: torch.Tensor | None = None, offsets: torch.Tensor | None = None,
                 start_pos: torch.Tensor | None = None, out_loc: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, token_to_req: torch.Tensor | None = None,
                 totals: torch.Tensor | None = None, max_tokens: int | None = None,
                 status: torch.Tensor | None = None, stream=None) -> None:
    """The batch tables of one step from the request lengths ``lens [S]`` and
    ``new_lens [S]`` (default: ``token_stride`` each): new pages of
    ``free_pages`` entered in ``page_table [S, pages]``, and the outputs
    ``offsets [2, S]``, ``start_pos [S]``, ``out_loc`` / ``positions`` /
    ``token_to_req [max_tokens]``, ``totals [4]`` that are given.
    ``max_tokens`` defaults to the smallest per-token output."""
    S = lens.numel()
    per = max_tokens
    if max_tokens is None:
        max_tokens = min([t.numel() for t in (out_loc, positions, token_to_req, depth)
                          if t is not None], default=S * token_stride)
        per = 0                               # (no per-token tensor is shorter)
    on = lens.get_device()
    # (messages are made only where they are raised: one takes as long as three checks)
    if offsets is not None and offsets.dim() > 1 and offsets.shape != (2, S):
        raise ValueError(f"offsets: shape {tuple(offsets.shape)}, need (2, {S})")
    if depth is not None and token_stride > 0:
        _rows_are(depth, token_stride, "depth")
    lens_p = _i32(lens, S, "lens")            # (refuses one that is on no device)
    if page_table.get_device() != on:
        _one_device(lens.device, (("page_table", page_table),))
    table_p = _rows(page_table, _I32_T, "page_table")
    rows, width = page_table.shape
    if rows < S:
        raise ValueError(f"page_table: shape {tuple(page_table.shape)}, need {S} rows")
    _call_on(lens.device, stream, lib().kvc_slot_map, kvc_slot_map_args(
        ratio, page_size, num_pages, S, token_stride, lens_p,
        _i32_on(new_lens, S, "new_lens", on), _i32_on(depth, per, "depth", on), table_p,
        page_table.stride(0) if rows > 1 else width, width,
        _i32_on(free_pages, 0, "free_pages", on), free_pages.numel(), max_tokens,
        _i32_on(offsets, 2 * S, "offsets", on), _i32_on(start_pos, S, "start_pos", on),
        _i32_on(out_loc, per, "out_loc", on), _i32_on(positions, per, "positions", on),
        _i32_on(token_to_req, per, "token_to_req", on), _i32_on(totals, 4, "totals", on),
        _i32_on(status, 1, "status", on)))


# ----------------------------------------------------------------- attention
def kvc_attend_workspace(num_slots: int, tokens: int, num_heads: int) -> int:
    """Workspace bytes of an attention call (``tokens``: rows of q; for
    kvc_attend_tree, slots times draft_len)."""
    n = C.c_int64(0)
    _check(lib().kvc_attend_workspace(num_slots, tokens, num_heads, C.byref(n)))
    return n.value


def _attend(fn, cache: Cache, q, start_pos, page_table, out, *, slots, tokens, ratio, scale, sink, lse,
            workspace, status, stream, offsets=None, draft_len=0, tree=None) -> None:
    for name, t in (("q", q), ("out", out)):
        _need(t.is_cuda and t.dtype in _B16_T and t.dim() == 3 and t.shape[2] == 512 and
              t.stride(2) == 1, f"{name}: expected a [tokens, heads, 512] bf16 device tensor with "
                                f"contiguous rows, got {t.dtype} {tuple(t.shape)} strides {t.stride()}")
    T, H, _ = q.shape
    _need(out.shape == q.shape, f"out: shape {tuple(out.shape)}, q has {tuple(q.shape)}")
    dev = q.device
    _one_device(dev, (("out", out), ("cache", cache.data), ("start_pos", start_pos),
                      ("page_table", page_table), ("offsets", offsets), ("tree", tree),
                      ("sink", sink), ("lse", lse), ("workspace", workspace), ("status", status)))
    _need(page_table.dim() == 2 and page_table.shape[0] >= slots,
          f"page_table: shape {tuple(page_table.shape)}, need {slots} rows")
    _need(sink is None or sink.numel() >= H, f"sink: fewer than {H} entries")
    _need(lse is None or tuple(lse.shape) == (T, H), f"lse: expected shape [{T}, {H}]")
    # a written row must be its own
    s0, s1, _ = out.stride()
    _need(T <= 1 or H <= 1 or s0 >= (H - 1) * s1 + 512 or s1 >= (T - 1) * s0 + 512,
          f"out: overlapping rows (strides {out.stride()})")
    if workspace is None:
        # of the stream the call runs on: the allocator then reuses it in order
        n = kvc_attend_workspace(slots, tokens, H)
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    a = kvc_attend_args(
        ratio, H, slots, draft_len, q.data_ptr(), q.stride(0), q.stride(1), T,
        _i32(offsets, 2 * slots, "offsets"), _i32(start_pos, slots, "start_pos"),
        _rows(page_table, _I32_T, "page_table"), _pt_stride(page_table), page_table.shape[1],
        _opt(tree, _dense, (torch.int64, torch.uint64), "tree"), scale,
        _opt(sink, _dense, _F32_T, "sink"), out.data_ptr(), s0, s1,
        _opt(lse, _dense, _F32_T, "lse"), cache.desc(),
        _dense(workspace, (torch.uint8,), "workspace"), workspace.numel(),
        _i32(status, 1, "status"))
    _call_on(dev, stream, fn, a)


def kvc_attend_prefill(cache: Cache, q: torch.Tensor, offsets: torch.Tensor,
                       start_pos: torch.Tensor, page_table: torch.Tensor, out: torch.Tensor, *,
                       scale: float, ratio: int = 1, sink: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       status: torch.Tensor | None = None, stream=None) -> None:
    """Causal attention of packed tokens ``q [T, H, 512]`` (slot b's rows and
    count in ``offsets [2, S]``, first position in ``start_pos [S]``) over the
    cached rows; ``out [T, H, 512]``, ``lse [T, H]`` (base 2).  ``workspace``:
    a uint8 tensor of ``kvc_attend_workspace`` bytes (allocated per call
    where it is not given)."""
    S = start_pos.numel()
    _need(offsets.numel() == 2 * S, f"offsets: expected [2, {S}] entries")
    _rows_are(offsets, S, "offsets")
    _attend(lib().kvc_attend_prefill, cache, q, start_pos, page_table, out, slots=S,
            tokens=q.shape[0], ratio=ratio, scale=scale, sink=sink, lse=lse, workspace=workspace,
            status=status, stream=stream, offsets=offsets)


def kvc_attend_tree(cache: Cache, q: torch.Tensor, start_pos: torch.Tensor,
                    page_table: torch.Tensor, out: torch.Tensor, *, scale: float,
                    draft_len: int = 1, tree: torch.Tensor | None = None, ratio: int = 1,
                    sink: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                    stream=None) -> None:
    """Attention of ``draft_len`` tokens per slot, ``q [S * draft_len, H,
    512]``, over the cached rows: a chain, or a tree given by ancestor masks
    ``tree [S, draft_len]`` (int64 bit patterns).  Other arguments as
    kvc_attend_prefill."""
    S = start_pos.numel()
    _need(q.dim() == 3 and q.shape[0] >= S * draft_len,
          f"q: shape {tuple(q.shape)} for {S} slots x {draft_len} tokens")
    _need(tree is None or tree.numel() >= S * draft_len, f"tree: expected [{S}, {draft_len}] masks")
    _rows_are(tree, draft_len, "tree")
    _attend(lib().kvc_attend_tree, cache, q, start_pos, page_table, out, slots=S,
            tokens=S * draft_len, ratio=ratio, scale=scale, sink=sink, lse=lse,
            workspace=workspace, status=status, stream=stream, draft_len=draft_len, tree=tree)


# -------------------------------------------------------------------- rotary
_DTYPES = {torch.bfloat16: 0, torch.int16: 0, torch.uint16: 0, torch.float16: 1, torch.float32: 2}


def kvc_rope_table(out: torch.Tensor, *, first: int = 0, base: float = 10000.0,
                   scaling: str = "none", factor: float = 1.0, original: float = 0.0,
                   beta_fast: float = 32.0, beta_slow: float = 1.0, mscale: float = 1.0,
                   stream=None) -> None:
    """The rotary table of positions ``first ..`` into ``out [n, rot_dim]``
    (fp32, (cos, sin) pairs).  ``scaling``: "none", "linear", "base" or
    "parts" (by ``factor``; "parts" from an ``original`` context, between
    ``beta_fast`` and ``beta_slow`` turns); ``mscale`` multiplies the
    entries."""
    _need(out.dim() == 2, f"out: expected [positions, rot_dim], got shape {tuple(out.shape)}")
    _need(scaling in ROPE_SCALING, f"scaling: {scaling!r}, one of {sorted(ROPE_SCALING)}")
    a = kvc_rope_table_args(_dense(out, _F32_T, "out"), out.shape[0], first, out.shape[1],
                            ROPE_SCALING[scaling], base, factor, original, beta_fast, beta_slow,
                            mscale)
    _call_on(out.device, stream, lib().kvc_rope_table, a)


def _heads(t, name: str) -> None:
    """Refuses what is not a [tokens, heads, dims] or [tokens, dims] device
    tensor of heads."""
    if not (t.is_cuda and t.dtype in _DTYPES and t.dim() in (2, 3) and
            (t.stride(-1) == 1 or t.shape[-1] == 1)):
        raise ValueError(f"{name}: expected a [tokens, heads, dims] or [tokens, dims] device tensor of "
                         f"bf16, fp16 or fp32 with contiguous rows, got {t.dtype} {tuple(t.shape)} "
                         f"strides {t.stride()}")


def kvc_rope_rows(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor,
                  out: torch.Tensor | None = None, *, offset: int | None = None,
                  half: bool = False, transpose: bool = False,
                  status: torch.Tensor | None = None, stream=None) -> None:
    """Rotate ``x [T, H, D]`` or ``[T, D]`` (bf16, fp16 or fp32) at
    ``positions [T]`` by the table ``freqs [max_pos, rot_dim]`` into ``out``
    (default: in place).  The rotated dims are ``offset ..`` (default: the
    last ``rot_dim``), pairs of neighbours or of ``half``s; ``transpose`` is
    the inverse rotation, which is also the rotation's backward pass."""
    _heads(x, "x")
    on = x.get_device()
    shape, strides, at = x.shape, x.stride(), x.data_ptr()
    if len(shape) == 3:
        T, H, D = shape
        x0, x1, _ = strides
    else:
        (T, D), H, x0, x1 = shape, 1, strides[0], 0
    if out is None:
        o0, o1, to = x0, x1, at
    else:
        _heads(out, "out")
        if out.shape != shape or out.dtype != x.dtype:
            raise ValueError(f"out: {out.dtype} {tuple(out.shape)}, x is {x.dtype} {tuple(shape)}")
        if out.get_device() != on:
            _one_device(x.device, (("out", out),))
        to = out.data_ptr()
        o0, o1 = out.stride(0), out.stride(1) if len(shape) == 3 else 0
        if to != at and out.stride() == strides and abs(to - at) < D * x.element_size():
            raise ValueError("out: overlaps x without being x")
    # a written row must be its own
    if T > 1 and H > 1 and o0 < (H - 1) * o1 + D and o1 < (T - 1) * o0 + D:
        raise ValueError(f"out: overlapping rows (strides {o0}, {o1})")
    if freqs.dim() != 2 or freqs.get_device() != on:
        _one_device(x.device, (("freqs", freqs),))
        raise ValueError(f"freqs: shape {tuple(freqs.shape)}, expected [max_pos, rot_dim]")
    max_pos, rot = freqs.shape
    pos = _i32_on(positions, T, "positions", on)
    table = _dense(freqs, _F32_T, "freqs")
    flag = _i32_on(status, 1, "status", on)
    if T == 0 or H == 0:
        return
    _call_on(x.device, stream, lib().kvc_rope_rows, kvc_rope_args(
        _DTYPES[x.dtype], H, D, rot, D - rot if offset is None else offset, half, transpose, T, at,
        x0, x1, to, o0, o1, pos, table, max_pos, flag))


# ------------------------------------------------------------------ eviction
def _table(t, types, rows: int, width: int, name: str, index: int):
    """Pointer, row stride of a 2-D tensor of at least ``rows`` rows of ``width``
    entries on the device of that index, or (None, 0) for None."""
    if t is None:
        return None, 0
    if t.get_device() != index and index >= 0:
        _one_device(torch.device("cuda", index), ((name, t),))
    at = _rows(t, types, name)
    n, w = t.shape
    if n < rows or w < width:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, need at least [{rows}, {width}]")
    return at, t.stride(0) if n > 1 else w


def _bytes(workspace, name: str, index: int):
    """Pointer, size of a workspace on the device of that index."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != index:
        _one_device(torch.device("cuda", index), ((name, workspace),))
    return _dense(workspace, (torch.uint8,), name), workspace.numel()


def _cache_on(cache: Cache, index: int):
    if cache.data.get_device() != index:
        _one_device(torch.device("cuda", index), (("cache", cache.data),))
    return cache.desc()


def _scratch(n: int, dev, stream):
    """Workspace of n bytes, of the stream the call runs on (the allocator then
    reuses it in order)."""
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return torch.empty(n, dtype=torch.uint8, device=dev)


_weigh_bytes = None


def kvc_weigh_workspace() -> int:
    """Workspace bytes of a kvc_weigh_* call that needs one (a slot with more
    than ``WEIGH_FEW`` (token, head) pairs)."""
    global _weigh_bytes
    if _weigh_bytes is None:
        n = C.c_int64(0)
        _check(lib().kvc_weigh_workspace(C.byref(n)))
        _weigh_bytes = n.value
    return _weigh_bytes


def _weigh(fn, cache: Cache, q, lse, start_pos, page_table, weights, *, slots, pairs, ratio, scale,
           prev, decay, workspace, status, stream, offsets=None, draft_len=0, tree=None) -> None:
    if not (q.is_cuda and q.dtype in _B16_T and q.dim() == 3 and q.shape[2] == 512 and q.stride(2) == 1):
        raise ValueError(f"q: expected a [tokens, heads, 512] bf16 device tensor with contiguous rows, got "
                         f"{q.dtype} {tuple(q.shape)} strides {q.stride()}")
    T, H, _ = q.shape
    q0, q1, _ = q.stride()
    on = q.get_device()
    if lse.get_device() != on or (tree is not None and tree.get_device() != on):
        _one_device(q.device, (("lse", lse), ("tree", tree)))
    if lse.shape != (T, H):
        raise ValueError(f"lse: shape {tuple(lse.shape)}, expected [{T}, {H}]")
    table, pt_stride = _table(page_table, _I32_T, slots, 0, "page_table", on)
    w, w_stride = _table(weights, _F32_T, slots, 0, "weights", on)
    W = weights.shape[1]
    old, old_stride = _table(prev, _F32_T, slots, W, "prev", on)
    if pairs > WEIGH_FEW and workspace is None:
        workspace = _scratch(kvc_weigh_workspace(), q.device, stream)
    space, size = _bytes(workspace, "workspace", on)
    _call_on(q.device, stream, fn, kvc_weigh_args(
        ratio, H, slots, draft_len, q.data_ptr(), q0, q1, T, _dense(lse, _F32_T, "lse"),
        _i32_on(offsets, 2 * slots, "offsets", on), _i32_on(start_pos, slots, "start_pos", on), table,
        pt_stride, page_table.shape[1], _opt(tree, _dense, (torch.int64, torch.uint64), "tree"), scale,
        decay, old, old_stride, w, w_stride, W, _cache_on(cache, on), space, size,
        _i32_on(status, 1, "status", on)))


def kvc_weigh_prefill(cache: Cache, q: torch.Tensor, lse: torch.Tensor, offsets: torch.Tensor,
                      start_pos: torch.Tensor, page_table: torch.Tensor, weights: torch.Tensor, *,
                      scale: float, ratio: int = 1, prev: torch.Tensor | None = None,
                      decay: float = 1.0, workspace: torch.Tensor | None = None,
                      status: torch.Tensor | None = None, stream=None) -> None:
    """Attention weight that the cached rows collect from packed tokens: for
    every row its tokens see, ``weights [S, rows]`` becomes ``decay`` times
    ``prev`` (default: 0; may be ``weights``) plus the sum of the weights that
    ``kvc_attend_prefill`` gave the row, whose ``q [T, H, 512]`` and
    ``lse [T, H]`` these are.  ``workspace``: a uint8 tensor of
    ``kvc_weigh_workspace`` bytes (allocated per call where it is needed and
    not given)."""
    S = start_pos.numel()
    if offsets.numel() != 2 * S:
        raise ValueError(f"offsets: shape {tuple(offsets.shape)}, expected [2, {S}]")
    _rows_are(offsets, S, "offsets")
    _weigh(lib().kvc_weigh_prefill, cache, q, lse, start_pos, page_table, weights, slots=S,
           pairs=q.shape[0] * q.shape[1] if q.dim() == 3 else 0, ratio=ratio, scale=scale, prev=prev,
           decay=decay, workspace=workspace, status=status, stream=stream, offsets=offsets)


def kvc_weigh_tree(cache: Cache, q: torch.Tensor, lse: torch.Tensor, start_pos: torch.Tensor,
                   page_table: torch.Tensor, weights: torch.Tensor, *, scale: float,
                   draft_len: int = 1, tree: torch.Tensor | None = None, ratio: int = 1,
                   prev: torch.Tensor | None = None, decay: float = 1.0,
                   workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                   stream=None) -> None:
    """kvc_weigh_prefill for ``draft_len`` tokens per slot, ``q [S *
    draft_len, H, 512]`` and the ``lse`` that ``kvc_attend_tree`` gave: a
    chain, a tree of ancestor masks, or single tokens."""
    S = start_pos.numel()
    if q.dim() != 3 or q.shape[0] < S * draft_len:
        raise ValueError(f"q: shape {tuple(q.shape)} for {S} slots x {draft_len} tokens")
    if tree is not None and tree.numel() < S * draft_len:
        raise ValueError(f"tree: shape {tuple(tree.shape)}, expected [{S}, {draft_len}] masks")
    _rows_are(tree, draft_len, "tree")
    _weigh(lib().kvc_weigh_tree, cache, q, lse, start_pos, page_table, weights, slots=S,
           pairs=draft_len * q.shape[1], ratio=ratio, scale=scale, prev=prev, decay=decay,
           workspace=workspace, status=status, stream=stream, draft_len=draft_len, tree=tree)


def kvc_evict_workspace(num_slots: int, w_width: int) -> int:
    """Workspace bytes of kvc_evict_select over ``num_slots`` rows of
    ``w_width`` weights."""
    n = C.c_int64(0)
    _check(lib().kvc_evict_workspace(num_slots, w_width, C.byref(n)))
    return n.value


def _rows_32(n: int) -> int:
    """A number of rows as the 32 bits that the library takes: one past them is as
    many as there can be."""
    return min(max(n, -1), 0x7FFFFFFF)


def kvc_evict_select(lens: torch.Tensor, weights: torch.Tensor, kept: torch.Tensor,
                     counts: torch.Tensor, *, budget: int | None = None, ratio: int = 1,
                     first: int = 0, recent: int = 0, budgets: torch.Tensor | None = None,
                     kept_weights: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     stream=None) -> None:
    """The rows that stay of slots of ``lens [S]`` tokens: at most ``budget``
    (default: as many as ``kept`` holds) or ``budgets [S]`` rows, the
    ``first`` and the ``recent`` ones and, of the others, those with the
    greatest ``weights [S, rows]``.  Their numbers go to ``kept [S, K]``
    (ascending, then -1), their count to ``counts [S]`` (-1: an inactive or
    refused slot), their weights to ``kept_weights [S, K]``."""
    S = lens.numel()
    on = lens.get_device()
    lens_p = _i32(lens, S, "lens")            # (refuses one that is on no device)
    w, w_stride = _table(weights, _F32_T, S, 0, "weights", on)
    k, k_stride = _table(kept, _I32_T, S, 0, "kept", on)
    K, W = kept.shape[1], weights.shape[1]
    kw, kw_stride = _table(kept_weights, _F32_T, S, K, "kept_weights", on)
    if workspace is None and W > SELECT_NO_WORKSPACE and S > 0:
        workspace = _scratch(kvc_evict_workspace(S, W), lens.device, stream)
    space, size = _bytes(workspace, "workspace", on)
    _call_on(lens.device, stream, lib().kvc_evict_select, kvc_evict_args(
        ratio, S, lens_p, w, w_stride, W, K if budget is None else _rows_32(budget), _rows_32(first),
        _rows_32(recent), _i32_on(budgets, S, "budgets", on), k, k_stride, K, _i32_on(counts, S, "counts", on), kw,
        kw_stride, space, size, _i32_on(status, 1, "status", on)))


def kvc_cache_compact(cache: Cache, lens: torch.Tensor, kept: torch.Tensor, counts: torch.Tensor,
                      page_table: torch.Tensor, free_pages: torch.Tensor, new_table: torch.Tensor,
                      new_lens: torch.Tensor, *, ratio: int = 1,
                      kept_weights: torch.Tensor | None = None,
                      weights: torch.Tensor | None = None, freed: torch.Tensor | None = None,
                      totals: torch.Tensor | None = None, status: torch.Tensor | None = None,
                      stream=None) -> None:
    """Move the rows ``kept [S, K]`` (``counts [S]`` of them) of slots that drop
    some to pages of ``free_pages``: ``new_table [S, pages]`` and ``new_lens
    [S]`` say where the slots are afterwards, ``freed`` lists the pages given
    back, ``kept_weights [S, K]`` goes to the front of ``weights [S, rows]``,
    and ``totals [4]`` counts pages taken, pages given back, rows dropped and
    slots refused."""
    S = lens.numel()
    on = lens.get_device()
    lens_p = _i32(lens, S, "lens")            # (refuses one that is on no device)
    k, k_stride = _table(kept, _I32_T, S, 0, "kept", on)
    K = kept.shape[1]
    table, pt_stride = _table(page_table, _I32_T, S, 0, "page_table", on)
    width = page_table.shape[1]
    new, nt_stride = _table(new_table, _I32_T, S, width, "new_table", on)
    kw, kw_stride = _table(kept_weights, _F32_T, S, K, "kept_weights", on)
    w, w_stride = _table(weights, _F32_T, S, 0, "weights", on)
    # (an empty tensor has no address: the library would take it as none given)
    if freed is not None and freed.numel() == 0 and S > 0:
        raise ValueError("freed: holds no page")
    _call_on(lens.device, stream, lib().kvc_cache_compact, kvc_compact_args(
        ratio, S, lens_p, k, k_stride, K, _i32_on(counts, S, "counts", on), table, pt_stride, width,
        _i32_on(free_pages, 0, "free_pages", on), free_pages.numel(), new, nt_stride,
        _i32_on(new_lens, S, "new_lens", on), kw, kw_stride, w, w_stride,
        0 if weights is None else weights.shape[1], _i32_on(freed, 0, "freed", on),
        0 if freed is None else freed.numel(), _i32_on(totals, 4, "totals", on),
        _cache_on(cache, on), _i32_on(status, 1, "status", on)))
