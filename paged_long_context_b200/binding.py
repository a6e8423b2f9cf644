"""Thin Python binding of the C ABI in include/cfr_paged.h (ctypes).

Argument marshalling only: every step of the attention computation runs in the
CUDA kernels of libcfr_paged.so.  There is no fallback: if the library is not
built, or a call is rejected, the binding raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import synth

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcfr_paged.so")

CFR_OK = 0
STATUS = {0: "CFR_OK", 1: "CFR_ERR_INVALID_ARG", 2: "CFR_ERR_UNSUPPORTED", 3: "CFR_ERR_OVERFLOW",
          4: "CFR_ERR_PAGE_INDEX", 5: "CFR_ERR_CUDA", 6: "CFR_ERR_TIMEOUT", 7: "CFR_ERR_WORKSPACE"}
DEVERR_PAGE_ID, DEVERR_PAGE_FMT, DEVERR_SEQ_LEN, DEVERR_POOL, DEVERR_TIMEOUT = 0x1, 0x2, 0x4, 0x8, 0x10
DEVERR_SCHEDULE = 0x20
STATUS_CODES = {v: k for k, v in STATUS.items()}
PATH_CUDA_CORE, PATH_TENSOR_CORE, PATH_F32_TMA = 1, 2, 3

# every exported symbol the header declares
EXPORTS = ["cfr_paged_decode_workspace_size", "cfr_paged_decode", "cfr_paged_decode_phases",
           "cfr_merge_partials",
           "cfr_schedule_splits", "cfr_gather_pages", "cfr_paged_decode_path", "cfr_status_str",
           "cfr_paged_decode_static_workspace", "cfr_demote_pages", "cfr_append_kv",
           "cfr_paged_decode_sink_window", "cfr_paged_decode_multi", "cfr_wait_probe",
           "cfr_qk_norm_rope_append", "cfr_write_kv", "cfr_read_kv",
           "cfr_paged_decode_tree_workspace_size", "cfr_paged_decode_tree"]
FMT_COUNT = 5


def _header_static_workspace_bytes() -> int:
    """CFR_STATIC_WORKSPACE_BYTES as the header defines it (one source of truth)."""
    import re
    hdr = os.path.join(os.path.dirname(_PKG), "include", "cfr_paged.h")
    m = re.search(r"#define\s+CFR_STATIC_WORKSPACE_BYTES\s+\((\d+)u\s*<<\s*(\d+)\)",
                  open(hdr).read())
    if not m:
        raise RuntimeError("CFR_STATIC_WORKSPACE_BYTES not found in include/cfr_paged.h")
    return int(m.group(1)) << int(m.group(2))


STATIC_WORKSPACE_BYTES = _header_static_workspace_bytes()


class CfrError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class KvPool(ctypes.Structure):
    """Mirror of cfr_kv_pool."""
    _fields_ = [
        ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32),
        ("k_pool", ctypes.c_void_p * FMT_COUNT), ("v_pool", ctypes.c_void_p * FMT_COUNT),
        ("scales", ctypes.c_void_p * FMT_COUNT), ("pool_pages", ctypes.c_int64 * FMT_COUNT),
    ]


_lib = None
_VP, _I32, _I64, _SZ, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


def lib():
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m paged_long_context_b200.build` (no CPU fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        L.cfr_paged_decode_workspace_size.restype = _SZ
        L.cfr_paged_decode_workspace_size.argtypes = [_I32] * 6
        L.cfr_paged_decode.restype = ctypes.c_int
        L.cfr_paged_decode.argtypes = [_VP, _I32, ctypes.POINTER(KvPool), _VP, _I32, _VP, _I32, _VP,
                                       _I32, _I32, _VP, _VP, _F32, _VP, _VP, _VP, _SZ, _VP, _VP]
        L.cfr_paged_decode_phases.restype = ctypes.c_int
        L.cfr_paged_decode_phases.argtypes = L.cfr_paged_decode.argtypes + [ctypes.c_uint32]
        L.cfr_merge_partials.restype = ctypes.c_int
        L.cfr_merge_partials.argtypes = [_VP, _VP, _VP, _VP, _I32, _I32, _I32, _VP, _VP, _VP]
        L.cfr_schedule_splits.restype = ctypes.c_int
        L.cfr_schedule_splits.argtypes = [_VP, _I32, _I32, _I32, _I32, _VP, _VP, _I32, _VP, _VP, _VP]
        L.cfr_gather_pages.restype = ctypes.c_int
        L.cfr_gather_pages.argtypes = [ctypes.POINTER(KvPool), _VP, _VP, _I32, _I32, _I32, _I32,
                                       _I32, _I32, _VP, _VP, _I64, _VP, _VP]
        L.cfr_paged_decode_path.restype = _I32
        L.cfr_paged_decode_path.argtypes = [_I32, ctypes.POINTER(KvPool), _I32, _VP, _I32, _I32, _VP]
        L.cfr_paged_decode_static_workspace.restype = ctypes.c_int
        L.cfr_paged_decode_static_workspace.argtypes = [_VP, _I32, ctypes.POINTER(KvPool), _VP, _I32,
                                                        _VP, _I32, _VP, _I32, _I32, _VP, _VP, _F32,
                                                        _VP, _VP, _VP, _VP]
        L.cfr_paged_decode_sink_window.restype = ctypes.c_int
        L.cfr_paged_decode_sink_window.argtypes = L.cfr_paged_decode.argtypes + [_I32, _I32,
                                                                                  ctypes.c_uint32]
        L.cfr_paged_decode_multi.restype = ctypes.c_int
        L.cfr_paged_decode_multi.argtypes = [_VP, _I32, ctypes.POINTER(KvPool), _VP, _I32, _VP, _I32,
                                             _VP, _I32, _I32, _I32, _VP, _VP, _F32, _VP, _VP, _VP,
                                             _SZ, _VP, _VP, ctypes.c_uint32]
        L.cfr_demote_pages.restype = ctypes.c_int
        L.cfr_demote_pages.argtypes = [ctypes.POINTER(KvPool), _I32, _I32, _VP, _VP, _VP, _I64,
                                       _VP, _VP, _VP, _I32, _VP, _VP]
        L.cfr_append_kv.restype = ctypes.c_int
        L.cfr_append_kv.argtypes = [ctypes.POINTER(KvPool), _VP, _I32, _VP, _I32, _VP, _I32,
                                    _VP, _VP, _I32, _VP, _VP]
        L.cfr_qk_norm_rope_append.restype = ctypes.c_int
        L.cfr_qk_norm_rope_append.argtypes = [ctypes.POINTER(KvPool), _VP, _I32, _VP, _I32, _I32,
                                              _VP, _I64, _VP, _I64, _VP, _I64, _I32, _I32, _I32,
                                              _VP, _VP, _F32, _VP, _VP, _I32, _I32, _VP, _VP, _VP,
                                              _VP, _VP]
        L.cfr_write_kv.restype = ctypes.c_int
        L.cfr_write_kv.argtypes = [ctypes.POINTER(KvPool), _VP, _I32, _VP, _I32, _I32, _VP, _VP,
                                   _VP, _I64, _VP, _I64, _I32, _I32, _VP, _VP]
        L.cfr_read_kv.restype = ctypes.c_int
        L.cfr_read_kv.argtypes = L.cfr_write_kv.argtypes
        L.cfr_paged_decode_tree_workspace_size.restype = _SZ
        L.cfr_paged_decode_tree_workspace_size.argtypes = [_I32] * 5
        L.cfr_paged_decode_tree.restype = ctypes.c_int
        L.cfr_paged_decode_tree.argtypes = [_VP, _I32, ctypes.POINTER(KvPool), _VP, _I32, _VP, _I32,
                                            _VP, _I32, _I32, _I32, _VP, _VP, _VP, _VP, _VP, _F32,
                                            _F32, _VP, _I32, _VP, _VP, _SZ, _VP, _VP]
        L.cfr_wait_probe.restype = ctypes.c_int
        L.cfr_wait_probe.argtypes = [_I64, _I32, _VP, _VP, _VP]
        L.cfr_status_str.restype = ctypes.c_char_p
        L.cfr_status_str.argtypes = [ctypes.c_int]
        _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> Optional[ctypes.c_void_p]:
    if stream is None:
        if torch.cuda.is_available():
            return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        return None
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def status_str(status: int) -> str:
    return lib().cfr_status_str(status).decode()


def pool_struct(num_kv_heads: int, head_dim: int, page_tokens: int, k_pool: dict, v_pool: dict,
                scales: Optional[dict] = None) -> KvPool:
    """cfr_kv_pool from dicts format -> device tensor."""
    s = KvPool()
    s.num_kv_heads, s.head_dim, s.page_tokens = num_kv_heads, head_dim, page_tokens
    scales = scales or {}
    for f in range(FMT_COUNT):
        s.k_pool[f] = k_pool[f].data_ptr() if f in k_pool else None
        s.v_pool[f] = v_pool[f].data_ptr() if f in v_pool else None
        s.scales[f] = scales[f].data_ptr() if f in scales else None
        s.pool_pages[f] = int(k_pool[f].shape[0]) if f in k_pool else 0
    return s


def kv_pool_struct(case: "synth.DecodeCase") -> KvPool:
    return pool_struct(case.num_kv_heads, case.head_dim, case.page_tokens, case.k_pool,
                       case.v_pool, case.scales)


def workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_pages, page_tokens) -> int:
    return int(lib().cfr_paged_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                     max_pages, page_tokens))


def _head_map_host(case):
    if case.head_map is None:
        return None, None
    hm = case.head_map.detach().to("cpu", torch.int32).contiguous()
    return hm, ctypes.c_void_p(hm.data_ptr())


def decode_path(case) -> int:
    """1 = general CUDA-core kernel, 2 = tcgen05 kernel, 3 = fp32 TMA kernel,
    0 = the call would be rejected."""
    pool = kv_pool_struct(case)
    hm, hmp = _head_map_host(case)
    return int(lib().cfr_paged_decode_path(case.q_fmt, ctypes.byref(pool), case.max_pages,
                                           _p(case.page_fmt), case.uniform_fmt, case.num_q_heads,
                                           hmp))


class DecodeBuffers:
    """Caller-owned output and scratch buffers of one decode call (device)."""

    def __init__(self, case, device=None, with_lse=True):
        dev = device or case.device
        rows = case.num_q_heads * getattr(case, "num_queries", 1)   # [Q][Hq] query rows
        self.out = torch.empty((case.batch, rows, case.head_dim), dtype=torch.float32, device=dev)
        self.lse = torch.empty((case.batch, rows), dtype=torch.float32,
                               device=dev) if with_lse else None
        n = workspace_size(case.batch, rows, case.num_kv_heads, case.head_dim,
                           case.max_pages, case.page_tokens)
        if n == 0:
            raise CfrError(1, "cfr_paged_decode_workspace_size")
        self.workspace = torch.empty((n,), dtype=torch.uint8, device=dev)
        self.err = torch.zeros((1,), dtype=torch.int32, device=dev)


PHASE_SCHEDULE, PHASE_DECODE, PHASE_MERGE, PHASE_ALL = 0x1, 0x2, 0x4, 0x7


def paged_decode_raw(case, bufs: DecodeBuffers, stream=None, workspace_bytes=None,
                     phases: Optional[int] = None, sink_window: Optional[tuple] = None) -> int:
    """Call cfr_paged_decode (cfr_paged_decode_phases when ``phases`` is given,
    cfr_paged_decode_sink_window when ``sink_window`` = (sink_tokens, window_tokens)
    is given, cfr_paged_decode_multi when the case has several queries per
    sequence) on a case whose tensors live on the GPU; returns the status."""
    pool = kv_pool_struct(case)
    hm, hmp = _head_map_host(case)
    nbytes = bufs.workspace.numel() if workspace_bytes is None else workspace_bytes
    args = (_p(case.q), case.q_fmt, ctypes.byref(pool), _p(case.page_table), case.max_pages,
            _p(case.seq_lens), case.batch, _p(case.page_fmt), case.uniform_fmt, case.num_q_heads,
            hmp, _p(case.alibi_slopes), float(case.softmax_scale), _p(bufs.out), _p(bufs.lse),
            _p(bufs.workspace), nbytes, _p(bufs.err), _stream(stream))
    if getattr(case, "num_queries", 1) > 1:
        if sink_window is not None:
            raise ValueError("sink/window subsets take one query per sequence")
        return int(lib().cfr_paged_decode_multi(
            _p(case.q), case.q_fmt, ctypes.byref(pool), _p(case.page_table), case.max_pages,
            _p(case.seq_lens), case.batch, _p(case.page_fmt), case.uniform_fmt, case.num_q_heads,
            case.num_queries, hmp, _p(case.alibi_slopes), float(case.softmax_scale), _p(bufs.out),
            _p(bufs.lse), _p(bufs.workspace), nbytes, _p(bufs.err), _stream(stream),
            PHASE_ALL if phases is None else phases))
    if sink_window is not None:
        return int(lib().cfr_paged_decode_sink_window(*args, int(sink_window[0]),
                                                      int(sink_window[1]),
                                                      PHASE_ALL if phases is None else phases))
    if phases is None:
        return int(lib().cfr_paged_decode(*args))
    return int(lib().cfr_paged_decode_phases(*args, phases))


def paged_decode(case, bufs: Optional[DecodeBuffers] = None, stream=None,
                 sink_window: Optional[tuple] = None) -> DecodeBuffers:
    """Decode attention for every (sequence, query head), over all tokens or a
    (sink_tokens, window_tokens) subset; raises on a rejected call."""
    bufs = bufs or DecodeBuffers(case)
    st = paged_decode_raw(case, bufs, stream, sink_window=sink_window)
    if st != CFR_OK:
        raise CfrError(st, "cfr_paged_decode")
    return bufs


def merge_partials(part_acc, part_m, part_l, split_off, batch, num_q_heads, head_dim, out,
                   lse=None, stream=None) -> int:
    return int(lib().cfr_merge_partials(_p(part_acc), _p(part_m), _p(part_l), _p(split_off),
                                        batch, num_q_heads, head_dim, _p(out), _p(lse),
                                        _stream(stream)))


def schedule_splits(seq_lens, batch, page_tokens, max_pages, target_splits, split_off, splits,
                    max_splits, num_splits, err=None, stream=None) -> int:
    return int(lib().cfr_schedule_splits(_p(seq_lens), batch, page_tokens, max_pages,
                                         target_splits, _p(split_off), _p(splits), max_splits,
                                         _p(num_splits), _p(err), _stream(stream)))


def gather_pages(case, b, kv_head, n_tokens, k_out, v_out, pitch, err=None, stream=None) -> int:
    pool = kv_pool_struct(case)
    return int(lib().cfr_gather_pages(ctypes.byref(pool), _p(case.page_table), _p(case.page_fmt),
                                      case.uniform_fmt, case.batch, case.max_pages, b, kv_head,
                                      n_tokens,
                                      _p(k_out), _p(v_out), pitch, _p(err), _stream(stream)))


def paged_decode_static_workspace(case, out, lse=None, err=None, stream=None) -> int:
    """cfr_paged_decode_static_workspace: decode with the library's built-in scratch array
    (for callers that cannot allocate device memory); returns the status."""
    pool = kv_pool_struct(case)
    hm, hmp = _head_map_host(case)
    return int(lib().cfr_paged_decode_static_workspace(
        _p(case.q), case.q_fmt, ctypes.byref(pool), _p(case.page_table), case.max_pages,
        _p(case.seq_lens), case.batch, _p(case.page_fmt), case.uniform_fmt, case.num_q_heads, hmp,
        _p(case.alibi_slopes), float(case.softmax_scale), _p(out), _p(lse), _p(err),
        _stream(stream)))


def wait_probe(limit_cycles: int, arrive: bool, err=None, result=None, stream=None) -> int:
    """cfr_wait_probe: the decode kernels' bounded on-chip wait, run once with a
    short cycle limit on a barrier that is (arrive) or is not arrived on."""
    return int(lib().cfr_wait_probe(int(limit_cycles), 1 if arrive else 0, _p(err), _p(result),
                                    _stream(stream)))


def demote_pages(pool: KvPool, src_fmt: int, dst_fmt: int, dst_k, dst_v, dst_scales,
                 src_slots, dst_slots, valid_tokens=None, err=None, stream=None) -> int:
    """cfr_demote_pages: re-encode pages of the src_fmt pool described by ``pool`` into
    the destination pool tensors (device uint8 [slots][Hkv][P][row_bytes]); returns the status."""
    n = int(src_slots.numel())
    return int(lib().cfr_demote_pages(ctypes.byref(pool), src_fmt, dst_fmt, _p(dst_k), _p(dst_v),
                                      _p(dst_scales), int(dst_k.shape[0]), _p(src_slots),
                                      _p(dst_slots), _p(valid_tokens), n, _p(err),
                                      _stream(stream)))


def append_kv(pool: KvPool, page_table, page_fmt, uniform_fmt: int, positions, k_new, v_new,
              err=None, stream=None) -> int:
    """cfr_append_kv: write one token per sequence into its F32/BF16 page; returns the status."""
    new_fmt = synth.F32 if k_new.dtype == torch.float32 else synth.BF16
    return int(lib().cfr_append_kv(ctypes.byref(pool), _p(page_table), int(page_table.shape[1]),
                                   _p(page_fmt), uniform_fmt, _p(positions),
                                   int(positions.numel()), _p(k_new), _p(v_new), new_fmt, _p(err),
                                   _stream(stream)))



_I32S, _I64S, _U8S, _F32S, _F64S = (torch.int32,), (torch.int64, torch.uint64), (torch.uint8,), \
    (torch.float32,), (torch.float64,)
_HOT = (torch.float32, torch.bfloat16)


def _device() -> int:
    """The current CUDA device; -1, the device of host tensors, where there is none (the library's
    own checks can be called there, and it launches nothing)."""
    if torch.cuda.is_initialized():
        return torch._C._cuda_getDevice()
    return torch.cuda.current_device() if torch.cuda.is_available() else -1


def _raw_stream(stream, dev: int) -> int:
    """A cudaStream_t as a number; the current stream of the device when none is given."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else 0
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _refuse(name, t, dtypes, shape, dev, layout):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is required")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.dtype} where {' or '.join(map(str, dtypes))} is wanted")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} where {tuple(shape)} is wanted")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, where {'the host' if dev < 0 else f'cuda:{dev}, the current device,'} is wanted")
    raise ValueError(f"{name}: {layout}")


def _want(name, t, dtypes, shape, dev):
    """Address of a contiguous tensor argument, after the checks that the C ABI cannot make: its
    type, shape, layout and device (shape None: any)."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and (shape is None or t.shape == shape) \
            and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _refuse(name, t, dtypes, shape, dev, "must be contiguous")


def _may(name, t, dtypes, shape, dev):
    return None if t is None else _want(name, t, dtypes, shape, dev)


def _want_rows(name, t, dtypes, shape, dev):
    """Address and token stride (in values) of a [tokens][heads][head_dim] argument whose tokens may
    be any distance apart; each token's values are contiguous."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == dev:
        n, heads, d = shape
        st = t.stride()
        if n * heads == 0 or (st[2] == 1 and (heads == 1 or st[1] == d)):
            # (a single row's stride is free: its own size)
            return t.data_ptr(), st[0] if n > 1 else heads * d
    _refuse(name, t, dtypes, shape, dev, "each token's [heads][head_dim] values must be contiguous")


def _want_table(page_table, page_fmt, dev):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table: an int32 tensor [batch][max_pages] is wanted")
    return (_want("page_table", page_table, _I32S, page_table.shape, dev),
            _may("page_fmt", page_fmt, _U8S, page_table.shape, dev))


def qk_norm_rope_append(pool: KvPool, q, k, v, rope_positions, inv_freq, q_out, page_table, page_fmt,
                        uniform_fmt: int, seq_ids, token_ids, q_weight=None, k_weight=None,
                        eps: float = 1e-6, interleaved: bool = False, err=None, stream=None) -> int:
    """cfr_qk_norm_rope_append: norm and rotate a step's queries and keys, and write its K and V
    into F32 / BF16 pages; q, k, v are [tokens][heads][head_dim] (views of a packed projection are
    fine); returns the status."""
    dev = _device()
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q: a tensor [tokens][heads][head_dim] is wanted")
    n, hq, d = q.shape[0], q.shape[1], pool.head_dim
    like, kv_shape = (q.dtype,), (n, pool.num_kv_heads, d)
    table, fmts = _want_table(page_table, page_fmt, dev)
    qp, qs = _want_rows("q", q, _HOT, (n, hq, d), dev)
    kp, ks = _want_rows("k", k, like, kv_shape, dev)
    vp, vs = _want_rows("v", v, like, kv_shape, dev)
    rot = 0
    inv = pos = None
    if inv_freq is not None:
        inv = _want("inv_freq", inv_freq, _F64S, None, dev)
        pos = _want("rope_positions", rope_positions, _I32S, (n,), dev)
        rot = 2 * inv_freq.numel()
    st = lib().cfr_qk_norm_rope_append(
        ctypes.byref(pool), table, page_table.shape[1], fmts, uniform_fmt, page_table.shape[0], qp, qs,
        kp, ks, vp, vs, synth.F32 if q.dtype == torch.float32 else synth.BF16, n, hq,
        _may("q_weight", q_weight, _F32S, (d,), dev), _may("k_weight", k_weight, _F32S, (d,), dev), eps,
        pos, inv, rot, 1 if interleaved else 0, _want("q_out", q_out, like, (n, hq, d), dev),
        _want("seq_ids", seq_ids, _I32S, (n,), dev), _want("token_ids", token_ids, _I32S, (n,), dev),
        _may("err", err, _I32S, None, dev), _raw_stream(stream, dev))
    return int(st)


def _chunk(fn, pool, page_table, page_fmt, uniform_fmt, row_offsets, starts, a, b, names, err, stream):
    dev = _device()
    if not isinstance(a, torch.Tensor) or a.dim() != 3:
        raise ValueError(f"{names[0]}: a tensor [rows][kv heads][head_dim] is wanted")
    shape = (a.shape[0], pool.num_kv_heads, pool.head_dim)
    table, fmts = _want_table(page_table, page_fmt, dev)
    batch, max_pages = page_table.shape
    ap, sa = _want_rows(names[0], a, _HOT, shape, dev)
    bp, sb = _want_rows(names[1], b, (a.dtype,), shape, dev)
    return int(fn(ctypes.byref(pool), table, max_pages, fmts, uniform_fmt, batch,
                  _want("row_offsets", row_offsets, _I32S, (batch + 1,), dev),
                  _want("starts", starts, _I32S, (batch,), dev), ap, sa, bp, sb,
                  synth.F32 if a.dtype == torch.float32 else synth.BF16, shape[0],
                  _may("err", err, _I32S, None, dev), _raw_stream(stream, dev)))


def write_kv(pool: KvPool, page_table, page_fmt, uniform_fmt: int, row_offsets, starts, k_new, v_new,
             err=None, stream=None) -> int:
    """cfr_write_kv: store a ragged chunk of new tokens into pages of any format, quantising as it
    writes; k_new, v_new are [rows][kv heads][head_dim]; returns the status."""
    return _chunk(lib().cfr_write_kv, pool, page_table, page_fmt, uniform_fmt, row_offsets, starts,
                  k_new, v_new, ("k_new", "v_new"), err, stream)


def read_kv(pool: KvPool, page_table, page_fmt, uniform_fmt: int, row_offsets, starts, k_out, v_out,
            err=None, stream=None) -> int:
    """cfr_read_kv: cached tokens back as dense fp32 or bf16 rows; returns the status."""
    return _chunk(lib().cfr_read_kv, pool, page_table, page_fmt, uniform_fmt, row_offsets, starts,
                  k_out, v_out, ("k_out", "v_out"), err, stream)


def tree_workspace_size(batch, num_queries, num_q_heads, num_kv_heads, head_dim) -> int:
    return int(lib().cfr_paged_decode_tree_workspace_size(batch, num_queries, num_q_heads,
                                                          num_kv_heads, head_dim))


def paged_decode_tree(pool: KvPool, q, page_table, seq_lens, out, lse, workspace, page_fmt=None,
                      uniform_fmt: int = synth.BF16, q_lens=None, tree_mask=None, depths=None,
                      head_map=None, alibi_slopes=None, softmax_scale: float = 0.0,
                      logit_cap: float = 0.0, err=None, stream=None) -> int:
    """cfr_paged_decode_tree: attention of drafted tokens (q is [batch][queries][heads][head_dim])
    over the cache, under a tree mask of int64 bit rows [batch][queries]; returns the status.
    head_map is a host int32 tensor.  bf16 queries have their probabilities rounded to bf16 once, fp32
    queries keep them in fp32 (on a slower kernel)."""
    dev = _device()
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.shape[3] != pool.head_dim:
        raise ValueError("q: a tensor [batch][queries][heads][head_dim] is wanted")
    shape = q.shape
    batch, nq, hq, _ = shape
    table, fmts = _want_table(page_table, page_fmt, dev)
    if page_table.shape[0] != batch:
        raise ValueError(f"page_table: {page_table.shape[0]} rows for {batch} sequences")
    st = lib().cfr_paged_decode_tree(
        _want("q", q, _HOT, None, dev), synth.F32 if q.dtype == torch.float32 else synth.BF16,
        ctypes.byref(pool), table, page_table.shape[1], _want("seq_lens", seq_lens, _I32S, (batch,), dev),
        batch, fmts, uniform_fmt, hq, nq, _may("q_lens", q_lens, _I32S, (batch,), dev),
        _may("tree_mask", tree_mask, _I64S, (batch, nq), dev),
        _may("depths", depths, _I32S, (batch, nq), dev), _may("head_map", head_map, _I32S, (hq,), -1),
        _may("alibi_slopes", alibi_slopes, _F32S, (hq,), dev), softmax_scale, logit_cap,
        _want("out", out, _HOT, shape, dev), synth.F32 if out.dtype == torch.float32 else synth.BF16,
        _may("lse", lse, _F32S, (batch, nq, hq), dev), _want("workspace", workspace, _U8S, None, dev),
        workspace.numel(), _may("err", err, _I32S, None, dev), _raw_stream(stream, dev))
    return int(st)
