"""Thin Python binding of libhs (include/hs_api.h), same names as the C ABI.

Argument marshalling only: checks dtypes/devices, allocates output tensors
when the caller does not pass them, and forwards raw pointers plus the current
CUDA stream.  Every step of the path runs in the CUDA kernels of libhs.so;
there is no CPU fallback.  If the library cannot be loaded this module raises.
"""
import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

import torch

from . import _build

_lib = None
_binding = None  # the hot calls' extension module (csrc/hs_binding.cpp), if built

HS_OK = 0
STATUS_NAMES = {0: "HS_OK", 1: "HS_ERR_INVALID_ARG", 2: "HS_ERR_MISALIGNED", 3: "HS_ERR_CAPACITY",
                4: "HS_ERR_CUDA", 5: "HS_ERR_TIMEOUT", 6: "HS_ERR_BAD_INDEX",
                7: "HS_ERR_UNSUPPORTED"}


class HSError(RuntimeError):
    def __init__(self, name, code):
        super().__init__(f"{name} failed: {STATUS_NAMES.get(code, code)}")
        self.code = code


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F32 = ctypes.c_float

_SIGS = {
    "hs_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "hs_wait_selftest": ([_I32, ctypes.c_uint64, _P, _P, _P], ctypes.c_int),
    "hs_host_device_pointer": ([_P, ctypes.POINTER(_P)], ctypes.c_int),
    "hs_normalize_indices": ([_P, _I32, _I32, _I32, _I32, _P, _P, _P, _I64, _I32, _P, _I32, _I32,
                              _I32, _I32, _P, _P, _P, _P, _P], ctypes.c_int),
    "hs_hot_state_reset": ([_P, _P, _I32, _I32, _P], ctypes.c_int),
    "hs_normalize_lookup_assign": ([_P, _I32, _I32, _I32, _I32, _P, _P, _P, _I64, _I32, _P, _I32,
                                    _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _I32, _I64,
                                    _P, _P, _P, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "hs_hot_lookup_assign": ([_P, _P, _I32, _I32, _I32, _P, _P, _P, _I32, _I64, _P, _P, _P, _P,
                              _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "hs_layer_transfer": ([_P, _P, _I64, _I64, _I32, _I32, _I32, _I32, _I64, _I64, _P, _P, _I32,
                           _I64, _I32, _I32, _P, _P], ctypes.c_int),
    "hs_swap_in": ([_P, _I64, _P, _I64, _P, _P, _P, _I32, _I32, _P, _I32, _I64, _I32, _P, _P, _P],
                   ctypes.c_int),
    "hs_hot_lookup_swap_in": ([_P, _P, _I32, _I32, _I32, _P, _P, _P, _I32, _I64, _P, _P, _P, _P,
                               _P, _P, _P, _P, _P, _P, _I64, _P, _I64, _P], ctypes.c_int),
    "hs_backup": ([_P, _P, _P, _P, _I32, _I64, _I64, _P, _P], ctypes.c_int),
    "hs_sparse_decode_workspace_bytes": ([_I32, _I32, _I32, _I32, _I32, _I32], _I64),
    "hs_sparse_decode": ([_P, _P, _P, _I64, _I64, _I64, _P, _P, _I32, _I32, _I32, _I32, _I32,
                          _I32, _F32, _P, _P, _P, _I64, _P, _P], ctypes.c_int),
    "hs_merge_states": ([_P, _P, _P, _I32, _I32, _I32, _P, _P, _P], ctypes.c_int),
    "hs_sparse_decode_partial_splits": ([_I32, _I32, _I32, _I32, _I32, _I32], _I32),
    "hs_sparse_decode_partial": ([_P, _P, _P, _I64, _I64, _I64, _P, _P, _I32, _I32, _I32, _I32,
                                  _I32, _I32, _F32, _P, _P, _P, _I32, _I32, _P, _P],
                                 ctypes.c_int),
    "hs_sparse_decode_finish": ([_P, _P, _P, _I64, _I64, _I64, _P, _P, _I32, _I32, _I32, _I32,
                                 _I32, _I32, _F32, _P, _P, _P, _I32, _I32, _P, _P, _P, _P, _P],
                                ctypes.c_int),
    "hs_sparse_decode_noalloc": ([_P, _P, _P, _I64, _I64, _I64, _P, _P, _I32, _I32, _I32, _I32,
                                  _I32, _I32, _F32, _P, _P, _P, _P], ctypes.c_int),
    "hs_fp8ds_gather": ([_P, _I64, _I64, _P, _P, _I32, _I32, _P, _P, _P, _P], ctypes.c_int),
    "hs_sparse_decode_fp8ds_workspace_bytes": ([_I32, _I32, _I32], _I64),
    "hs_swap_in_fp8ds": ([_P, _I64, _I64, _P, _I64, _P, _P, _P, _I32, _I32, _P, _I32, _I64, _I32,
                          _P, _P, _P], ctypes.c_int),
    "hs_sparse_decode_fp8ds": ([_P, _P, _I64, _I64, _P, _P, _I32, _I32, _I32, _F32, _P, _P, _P,
                                _I64, _P, _P], ctypes.c_int),
    "hs_paged_decode_workspace_bytes": ([_I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32], _I64),
    "hs_paged_decode": ([_P, _I64, _I32, _P, _P, _I32, _I64, _I64, _I64, _I32, _I32, _P, _I64,
                         _I32, _I32, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P,
                         _I64, _F32, _P, _P, _P, _I64, _P, _P], ctypes.c_int),
    "hs_evict_select": ([_P, _I64, _P, _I64, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _I64, _P,
                         _I64, _P, _P, _P, _P, _I32, _P, _P], ctypes.c_int),
    "hs_evict_move": ([_P, _P, _I64, _I64, _I64, _I32, _I32, _I32, _I32, _P, _I64, _I32, _P, _P,
                       _P, _I32, _I32, _P, _P], ctypes.c_int),
    "hs_evict": ([_P, _I64, _P, _I64, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _I64, _P, _I64,
                  _P, _P, _P, _P, _I32, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32, _I32, _P,
                  _I64, _I32, _P, _P], ctypes.c_int),
}

NOALLOC_WORKSPACE_BYTES = 8 * 1024 * 1024  # HS_NOALLOC_WORKSPACE_BYTES

EXPORTS = tuple(_SIGS)


def lib_path():
    return _build.LIB


def lib():
    """Load libhs.so (building it first if it is missing or stale)."""
    global _lib
    if _lib is None:
        path = _build.build()
        L = ctypes.CDLL(path)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
        _load_binding()
    return _lib


def _load_binding():
    global _binding
    path = _build.binding_path()
    if path is None or not os.path.exists(path):
        return
    loader = importlib.machinery.ExtensionFileLoader("_hs_binding", path)
    try:
        mod = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("_hs_binding", loader))
        loader.exec_module(mod)
    except ImportError as e:  # every call has its way through ctypes
        warnings.warn(f"the extension of the hot calls does not load: {e}")
        return
    _binding = mod


def _ptr(t):
    """Device-visible address of a tensor argument: a CUDA tensor's own, or
    the mapped address of a pinned host tensor (the kernels then read or
    write host memory over the link)."""
    if t is None:
        return None
    if not t.is_cuda:
        return ctypes.c_void_p(host_device_pointer(t))
    return ctypes.c_void_p(t.data_ptr())


def device_address(t):
    """Device-visible address (int) of a CUDA tensor or a pinned host tensor."""
    return _ptr(t).value


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _raw_stream(device, stream=None):
    """As _stream, as an int, for the current stream of `device` (an index)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device)


def _call(name, *args):
    rc = getattr(lib(), name)(*args)
    if rc != HS_OK:
        raise HSError(name, rc)


def _check(t, dtype, name, cuda=True):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if cuda and not t.is_cuda and not t.is_pinned():
        raise ValueError(f"{name}: must be a CUDA tensor or pinned host memory")


def _check_workspace(t):
    """Scratch is one run of bytes: numel elements from the tensor's start."""
    if t is not None and not t.is_contiguous():
        raise ValueError("workspace: must be contiguous")


def wait_selftest(mode, timeout_ns, *, stream=None):
    """Bounded-wait self-test (hs_wait_selftest); returns (status, elapsed_ns)."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    elapsed = torch.zeros(1, dtype=torch.int64, device="cuda")
    _call("hs_wait_selftest", mode, timeout_ns, _ptr(status), _ptr(elapsed), _stream(stream))
    torch.cuda.synchronize()
    return int(status.item()), int(elapsed.item())


def status_string(code):
    return lib().hs_status_string(code).decode()


def host_device_pointer(t):
    """Device-visible address of a pinned host tensor."""
    if not t.is_pinned():
        raise ValueError("host memory must be pinned (pin_memory())")
    out = ctypes.c_void_p()
    _call("hs_host_device_pointer", ctypes.c_void_p(t.data_ptr()), ctypes.byref(out))
    return out.value


# ---------------------------------------------------------------------------
def normalize_indices(cand, row_req, seq_lens, block_table, page_size, *, window=0, num_sinks=0,
                      page_owner=None, num_pages, max_blocks=None, cap=None, out=None,
                      stream=None):
    """S1.  Returns (tok, slot, count, err) int32 tensors."""
    for t, n in ((cand, "cand"), (row_req, "row_req"), (seq_lens, "seq_lens"),
                 (block_table, "block_table"), (page_owner, "page_owner")):
        _check(t, torch.int32, n)
    rows, n_cand = cand.shape
    num_reqs, bt_stride = block_table.shape
    max_blocks = bt_stride if max_blocks is None else max_blocks
    cap = n_cand + window + num_sinks if cap is None else cap
    if out is None:
        dev = cand.device
        out = (torch.empty(rows, cap, dtype=torch.int32, device=dev),
               torch.empty(rows, cap, dtype=torch.int32, device=dev),
               torch.empty(rows, dtype=torch.int32, device=dev),
               torch.empty(rows, 4, dtype=torch.int32, device=dev))
    tok, slot, count, err = out
    _call("hs_normalize_indices", _ptr(cand), rows, n_cand, window, num_sinks, _ptr(row_req),
          _ptr(seq_lens), _ptr(block_table), bt_stride, max_blocks, _ptr(page_owner), num_reqs,
          num_pages, page_size, cap, _ptr(tok), _ptr(slot), _ptr(count), _ptr(err),
          _stream(stream))
    return tok, slot, count, err


def normalize_lookup_assign(cand, row_req, seq_lens, block_table, page_size, newest_slot, dgi,
                            lru, region_stride, stats, *, window=0, num_sinks=0, page_owner=None,
                            num_pages, max_blocks=None, cap=None, s1_out=None, s2_out=None,
                            stream=None):
    """S1 and S2 in one kernel (hs_normalize_lookup_assign).  Returns
    (s1_out, s2_out): (tok, slot, count, err) as normalize_indices and the
    8-tuple (hot_idx, miss_mask, miss_src, miss_dst, miss_count, err,
    hit_idx, miss_rows) as hot_lookup_assign with split lists."""
    for t, n in ((cand, "cand"), (row_req, "row_req"), (seq_lens, "seq_lens"),
                 (block_table, "block_table"), (page_owner, "page_owner"),
                 (newest_slot, "newest_slot"), (dgi, "dgi")):
        _check(t, torch.int32, n)
    _check(lru, torch.int16, "lru")
    _check(stats, torch.int64, "stats")
    rows, n_cand = cand.shape
    num_reqs, bt_stride = block_table.shape
    max_blocks = bt_stride if max_blocks is None else max_blocks
    cap = n_cand + window + num_sinks if cap is None else cap
    hot_size = dgi.shape[1]
    dev = cand.device
    i32 = dict(dtype=torch.int32, device=dev)
    if s1_out is None:
        s1_out = (torch.empty(rows, cap, **i32), torch.empty(rows, cap, **i32),
                  torch.empty(rows, **i32), torch.empty(rows, 4, **i32))
    if s2_out is None:
        s2_out = (torch.empty(rows, cap, **i32),
                  torch.empty(rows, cap, dtype=torch.uint8, device=dev),
                  torch.empty(rows, cap, **i32),
                  torch.empty(rows, cap, dtype=torch.int64, device=dev),
                  torch.empty(rows, **i32), torch.empty(rows, **i32),
                  torch.empty(rows, cap, **i32), torch.empty(rows, cap, **i32))
    tok, slot, count, err = s1_out
    hot_idx, miss_mask, miss_src, miss_dst, miss_count, lerr, hit_idx, miss_rows = s2_out
    _call("hs_normalize_lookup_assign", _ptr(cand), rows, n_cand, window, num_sinks,
          _ptr(row_req), _ptr(seq_lens), _ptr(block_table), bt_stride, max_blocks,
          _ptr(page_owner), num_reqs, num_pages, page_size, cap, _ptr(tok), _ptr(slot),
          _ptr(count), _ptr(err), _ptr(newest_slot), _ptr(dgi), _ptr(lru), hot_size,
          region_stride, _ptr(hot_idx), _ptr(miss_mask), _ptr(miss_src), _ptr(miss_dst),
          _ptr(miss_count), _ptr(stats), _ptr(lerr), _ptr(hit_idx), _ptr(miss_rows),
          _stream(stream))
    return s1_out, s2_out


def hot_state_reset(dgi, lru, stream=None):
    _check(dgi, torch.int32, "dgi")
    _check(lru, torch.int16, "lru")
    rows, hot_size = dgi.shape
    _call("hs_hot_state_reset", _ptr(dgi), _ptr(lru), rows, hot_size, _stream(stream))


def hot_lookup_assign(slot, count, newest_slot, dgi, lru, region_stride, stats, *,
                      num_real_rows=None, out=None, with_mask=True, with_split_lists=False,
                      swap=None, stream=None):
    """S2.  dgi/lru are updated in place; stats int64 [2] accumulates.
    Returns (hot_idx, miss_mask, miss_src, miss_dst, miss_count, err) and, with
    with_split_lists (or an 8-tuple `out`), also (hit_idx, miss_rows).
    swap=(host_pool_dev, host_rows, hot, row_bytes): the same kernel also
    copies the misses into the hot rows (hs_hot_lookup_swap_in)."""
    _check(slot, torch.int32, "slot")
    _check(count, torch.int32, "count")
    _check(newest_slot, torch.int32, "newest_slot")
    _check(dgi, torch.int32, "dgi")
    _check(lru, torch.int16, "lru")
    _check(stats, torch.int64, "stats")
    rows, cap = slot.shape
    hot_size = dgi.shape[1]
    if out is None:
        dev = slot.device
        out = (torch.empty(rows, cap, dtype=torch.int32, device=dev),
               torch.empty(rows, cap, dtype=torch.uint8, device=dev) if with_mask else None,
               torch.empty(rows, cap, dtype=torch.int32, device=dev),
               torch.empty(rows, cap, dtype=torch.int64, device=dev),
               torch.empty(rows, dtype=torch.int32, device=dev),
               torch.empty(rows, dtype=torch.int32, device=dev))
        if with_split_lists:
            out = out + (torch.empty(rows, cap, dtype=torch.int32, device=dev),
                         torch.empty(rows, cap, dtype=torch.int32, device=dev))
    hot_idx, miss_mask, miss_src, miss_dst, miss_count, err = out[:6]
    hit_idx, miss_rows = (out[6], out[7]) if len(out) == 8 else (None, None)
    nrr = rows if num_real_rows is None else num_real_rows
    if swap is None:
        _call("hs_hot_lookup_assign", _ptr(slot), _ptr(count), rows, cap, nrr,
              _ptr(newest_slot), _ptr(dgi), _ptr(lru), hot_size, region_stride, _ptr(hot_idx),
              _ptr(miss_mask), _ptr(miss_src), _ptr(miss_dst), _ptr(miss_count), _ptr(stats),
              _ptr(err), _ptr(hit_idx), _ptr(miss_rows), _stream(stream))
    else:
        host_pool_dev, host_rows, hot, row_bytes = swap
        _call("hs_hot_lookup_swap_in", _ptr(slot), _ptr(count), rows, cap, nrr,
              _ptr(newest_slot), _ptr(dgi), _ptr(lru), hot_size, region_stride, _ptr(hot_idx),
              _ptr(miss_mask), _ptr(miss_src), _ptr(miss_dst), _ptr(miss_count), _ptr(stats),
              _ptr(err), _ptr(hit_idx), _ptr(miss_rows), ctypes.c_void_p(host_pool_dev),
              host_rows, _ptr(hot), row_bytes, _stream(stream))
    return out


def swap_in(host_pool_dev, host_rows, hot, row_bytes, miss_src, miss_dst, miss_count, *,
            dgi=None, hot_size=0, region_stride=0, max_ctas=0, ticket=None, status=None,
            stream=None):
    """S3 SwapIn.  host_pool_dev: device-visible address (int) of the pinned pool.
    ticket: None, or int32 [2] device counters, zero on entry and left zero
    (groups claimed dynamically by the warps)."""
    _check(miss_src, torch.int32, "miss_src")
    _check(miss_dst, torch.int64, "miss_dst")
    _check(miss_count, torch.int32, "miss_count")
    _check(dgi, torch.int32, "dgi")
    _check(ticket, torch.int32, "ticket")
    _check(status, torch.int32, "status")
    if ticket is not None and ticket.numel() < 2:
        raise ValueError("ticket needs 2 int32 words")
    rows, cap = miss_src.shape
    _call("hs_swap_in", ctypes.c_void_p(host_pool_dev), host_rows, _ptr(hot), row_bytes,
          _ptr(miss_src), _ptr(miss_dst), _ptr(miss_count), rows, cap, _ptr(dgi), hot_size,
          region_stride, max_ctas, _ptr(ticket), _ptr(status), _stream(stream))


def layer_pointer_table(dev_pools):
    """Device pointer table for layer_transfer: dev_pools is a list over
    buffers (K, V; or one for MLA) of lists over layers of CUDA tensors
    [dev_tokens, ...] (row-major rows).  Build it once, outside graph capture."""
    ptrs = [t.data_ptr() for pools in dev_pools for t in pools]
    return torch.tensor(ptrs, dtype=torch.int64, device=dev_pools[0][0].device)


def layer_transfer(table, nbuf, layers, dev_tokens, row_bytes, host_pool, host_tokens,
                   src_idx, dst_idx, *, page_size, page_first, direction, max_ctas=0,
                   status=None, stream=None):
    """HiCache layer transfer (see hs_layer_transfer): table from
    layer_pointer_table; host_pool a pinned host tensor holding nbuf pools of
    host_tokens * layers rows; src_idx/dst_idx int32 or int64 CUDA tensors [n];
    direction 0 host -> device, 1 device -> host."""
    _check(table, torch.int64, "table")
    if src_idx.dtype not in (torch.int32, torch.int64) or dst_idx.dtype != src_idx.dtype:
        raise TypeError("src_idx/dst_idx: int32 or int64, the same dtype")
    _check(src_idx, src_idx.dtype, "src_idx")
    _check(dst_idx, dst_idx.dtype, "dst_idx")
    _check(status, torch.int32, "status")
    if table.numel() != nbuf * layers:
        raise ValueError("table holds nbuf * layers pointers")
    n = src_idx.numel()
    if dst_idx.numel() != n:
        raise ValueError("src_idx and dst_idx differ in length")
    hdev = host_device_pointer(host_pool)
    _call("hs_layer_transfer", _ptr(table), ctypes.c_void_p(hdev), host_tokens,
          host_tokens * layers * row_bytes, nbuf, layers, page_size, 1 if page_first else 0,
          dev_tokens, row_bytes, _ptr(src_idx), _ptr(dst_idx), src_idx.element_size(), n,
          direction, max_ctas, _ptr(status), _stream(stream))


def backup(src, src_rows, host_pool_dev, dst_slots, row_bytes, host_rows, *, status=None,
           stream=None):
    """BackUp: host_pool[dst_slots[i]] = src[src_rows[i]]."""
    _check(src_rows, torch.int64, "src_rows")
    _check(dst_slots, torch.int32, "dst_slots")
    _check(status, torch.int32, "status")
    _call("hs_backup", _ptr(src), _ptr(src_rows), ctypes.c_void_p(host_pool_dev),
          _ptr(dst_slots), dst_slots.numel(), row_bytes, host_rows, _ptr(status),
          _stream(stream))


def sparse_decode_workspace_bytes(rows, heads, kv_heads, cap, d_qk, d_v):
    return int(lib().hs_sparse_decode_workspace_bytes(rows, heads, kv_heads, cap, d_qk, d_v))


def sparse_decode(q, k_base, v_base, row_stride, kv_head_stride, num_kv_rows, kv_rows, count,
                  scale, d_v, *, out=None, lse=None, workspace=None, status=None, stream=None):
    """S4.  q bf16 [rows, heads, d_qk]; kv_rows int32 [rows, kv_heads, cap];
    count int32 [rows, kv_heads] or None.  Returns (out bf16, lse fp32)."""
    _check(q, torch.bfloat16, "q")
    _check(kv_rows, torch.int32, "kv_rows")
    _check(count, torch.int32, "count")
    _check(status, torch.int32, "status")
    rows, heads, d_qk = q.shape
    _, kv_heads, cap = kv_rows.shape
    if out is None:
        out = torch.empty(rows, heads, d_v, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(rows, heads, dtype=torch.float32, device=q.device)
    ws = sparse_decode_workspace_bytes(rows, heads, kv_heads, cap, d_qk, d_v)
    _check_workspace(workspace)
    if ws > 0 and (workspace is None or workspace.numel() * workspace.element_size() < ws):
        workspace = torch.empty(ws, dtype=torch.uint8, device=q.device)
    _call("hs_sparse_decode", _ptr(q), _ptr(k_base), _ptr(v_base), row_stride, kv_head_stride,
          num_kv_rows, _ptr(kv_rows), _ptr(count), rows, cap, heads, kv_heads, d_qk, d_v,
          float(scale), _ptr(out), _ptr(lse), _ptr(workspace) if ws > 0 else None,
          workspace.numel() * workspace.element_size() if (ws > 0) else 0, _ptr(status),
          _stream(stream))
    return out, lse


FP8DS_ROW_BYTES = 656


def fp8ds_gather(kv8, kv_rows, count, *, out=None, out_ids=None, status=None, stream=None):
    """Reconstruct fp8_ds_mla rows.  kv8 uint8 [num_kv_rows, row_bytes >= 656];
    kv_rows int32 [rows, cap]; count int32 [rows] or None.  Returns (out bf16
    [rows * cap, 576], out_ids int32 [rows * cap])."""
    _check(kv8, torch.uint8, "kv8")
    _check(kv_rows, torch.int32, "kv_rows")
    _check(count, torch.int32, "count")
    _check(status, torch.int32, "status")
    rows, cap = kv_rows.shape[0], kv_rows.shape[-1]
    if out is None:
        out = torch.empty(rows * cap, 576, dtype=torch.bfloat16, device=kv_rows.device)
    if out_ids is None:
        out_ids = torch.empty(rows * cap, dtype=torch.int32, device=kv_rows.device)
    _call("hs_fp8ds_gather", _ptr(kv8), kv8.shape[1], kv8.shape[0], _ptr(kv_rows), _ptr(count),
          rows, cap, _ptr(out), _ptr(out_ids), _ptr(status), _stream(stream))
    return out, out_ids


def swap_in_fp8ds(host_pool_dev, host_rows, host_row_bytes, hot, miss_src, miss_dst,
                  miss_count, *, dgi=None, hot_size=0, region_stride=0, max_ctas=0,
                  ticket=None, status=None, stream=None):
    """S3 SwapIn from a pool of fp8_ds_mla rows (device-visible address
    host_pool_dev) into bf16 hot rows [hot_rows, 576], reconstructing as the
    copy stores each row; arguments as for swap_in."""
    _check(hot, torch.bfloat16, "hot")
    _check(miss_src, torch.int32, "miss_src")
    _check(miss_dst, torch.int64, "miss_dst")
    _check(miss_count, torch.int32, "miss_count")
    _check(dgi, torch.int32, "dgi")
    _check(ticket, torch.int32, "ticket")
    _check(status, torch.int32, "status")
    if ticket is not None and ticket.numel() < 2:
        raise ValueError("ticket needs 2 int32 words")
    rows, cap = miss_src.shape
    _call("hs_swap_in_fp8ds", ctypes.c_void_p(host_pool_dev), host_rows, host_row_bytes,
          _ptr(hot), hot.shape[0], _ptr(miss_src), _ptr(miss_dst), _ptr(miss_count), rows, cap,
          _ptr(dgi), hot_size, region_stride, max_ctas, _ptr(ticket), _ptr(status),
          _stream(stream))


def sparse_decode_fp8ds_workspace_bytes(rows, heads, cap):
    return int(lib().hs_sparse_decode_fp8ds_workspace_bytes(rows, heads, cap))


def sparse_decode_fp8ds(q, kv8, kv_rows, count, scale, *, out=None, lse=None, workspace=None,
                        status=None, stream=None):
    """S4 over fp8_ds_mla rows (MLA shape).  q bf16 [rows, heads, 576]; kv8
    uint8 [num_kv_rows, row_bytes >= 656]; kv_rows int32 [rows, 1, cap] or
    [rows, cap]; count int32 [rows] / [rows, 1] or None.  Returns (out bf16
    [rows, heads, 512], lse fp32 [rows, heads])."""
    _check(q, torch.bfloat16, "q")
    _check(kv8, torch.uint8, "kv8")
    _check(kv_rows, torch.int32, "kv_rows")
    _check(count, torch.int32, "count")
    _check(status, torch.int32, "status")
    rows, heads, _ = q.shape
    cap = kv_rows.shape[-1]
    if out is None:
        out = torch.empty(rows, heads, 512, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(rows, heads, dtype=torch.float32, device=q.device)
    ws = sparse_decode_fp8ds_workspace_bytes(rows, heads, cap)
    _check_workspace(workspace)
    if workspace is None or workspace.numel() * workspace.element_size() < ws:
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=q.device)
    _call("hs_sparse_decode_fp8ds", _ptr(q), _ptr(kv8), kv8.shape[1], kv8.shape[0],
          _ptr(kv_rows), _ptr(count), rows, cap, heads, float(scale), _ptr(out), _ptr(lse),
          _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
          _stream(stream))
    return out, lse


def sparse_decode_partial_splits(rows, heads, kv_heads, cap, d_qk, d_v):
    return int(lib().hs_sparse_decode_partial_splits(rows, heads, kv_heads, cap, d_qk, d_v))


def sparse_decode_partial(q, k_base, v_base, row_stride, kv_head_stride, num_kv_rows, kv_rows,
                          count, scale, d_v, part_m, part_l, part_o, part_base, *, status=None,
                          stream=None):
    """S4 partial states into columns [part_base, part_base + P) of
    part_m/part_l fp32 [rows*heads, parts] and part_o fp32 [rows*heads, parts, d_v];
    returns P.  Combine with merge_states."""
    _check(q, torch.bfloat16, "q")
    _check(kv_rows, torch.int32, "kv_rows")
    _check(count, torch.int32, "count")
    for t, n in ((part_m, "part_m"), (part_l, "part_l"), (part_o, "part_o")):
        _check(t, torch.float32, n)
    _check(status, torch.int32, "status")
    rows, heads, d_qk = q.shape
    _, kv_heads, cap = kv_rows.shape
    parts = part_m.shape[-1]
    _call("hs_sparse_decode_partial", _ptr(q), _ptr(k_base), _ptr(v_base), row_stride,
          kv_head_stride, num_kv_rows, _ptr(kv_rows), _ptr(count), rows, cap, heads, kv_heads,
          d_qk, d_v, float(scale), _ptr(part_m), _ptr(part_l), _ptr(part_o), parts, part_base,
          _ptr(status), _stream(stream))
    return sparse_decode_partial_splits(rows, heads, kv_heads, cap, d_qk, d_v)


def sparse_decode_finish(q, k_base, v_base, row_stride, kv_head_stride, num_kv_rows, kv_rows,
                         count, scale, d_v, part_m, part_l, part_o, parts_used, *, sync=None,
                         out=None, lse=None, status=None, stream=None):
    """Attend over kv_rows, merge with partial columns [0, parts_used) and
    write the final (out bf16 [rows, heads, d_v], lse fp32 [rows, heads]).
    sync: optional int32 scratch of rows*heads words (lets the MLA kernel split
    the rows over several CTAs and merge in the last one)."""
    _check(q, torch.bfloat16, "q")
    _check(sync, torch.int32, "sync")
    _check(kv_rows, torch.int32, "kv_rows")
    _check(count, torch.int32, "count")
    for t, n in ((part_m, "part_m"), (part_l, "part_l"), (part_o, "part_o")):
        _check(t, torch.float32, n)
    _check(status, torch.int32, "status")
    rows, heads, d_qk = q.shape
    _, kv_heads, cap = kv_rows.shape
    if out is None:
        out = torch.empty(rows, heads, d_v, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(rows, heads, dtype=torch.float32, device=q.device)
    _call("hs_sparse_decode_finish", _ptr(q), _ptr(k_base), _ptr(v_base), row_stride,
          kv_head_stride, num_kv_rows, _ptr(kv_rows), _ptr(count), rows, cap, heads, kv_heads,
          d_qk, d_v, float(scale), _ptr(part_m), _ptr(part_l), _ptr(part_o), part_m.shape[-1],
          parts_used, _ptr(sync), _ptr(out), _ptr(lse), _ptr(status), _stream(stream))
    return out, lse


def merge_states(m, l, o, *, out=None, lse=None, stream=None):
    """Eq. (7) merge: m, l fp32 [n, parts] (m in log2 units); o fp32 [n, parts, d_v]."""
    for t, n in ((m, "m"), (l, "l"), (o, "o")):
        _check(t, torch.float32, n)
    n, parts, d_v = o.shape
    if out is None:
        out = torch.empty(n, d_v, dtype=torch.bfloat16, device=o.device)
    if lse is None:
        lse = torch.empty(n, dtype=torch.float32, device=o.device)
    _call("hs_merge_states", _ptr(m), _ptr(l), _ptr(o), n, parts, d_v, _ptr(out), _ptr(lse),
          _stream(stream))
    return out, lse


def sparse_decode_noalloc(q, k_base, v_base, row_stride, kv_head_stride, num_kv_rows, kv_rows,
                          count, scale, d_v, *, out, lse, status=None, stream=None):
    """S4 without a workspace argument: for callers that may not allocate
    device memory on the decode path (the library's built-in scratch array is
    used; see hs_sparse_decode_noalloc in hs_api.h).  `out` and `lse` must be
    passed in, so that this call allocates nothing."""
    _check(q, torch.bfloat16, "q")
    _check(kv_rows, torch.int32, "kv_rows")
    _check(count, torch.int32, "count")
    _check(out, torch.bfloat16, "out")
    _check(lse, torch.float32, "lse")
    _check(status, torch.int32, "status")
    rows, heads, d_qk = q.shape
    _, kv_heads, cap = kv_rows.shape
    _call("hs_sparse_decode_noalloc", _ptr(q), _ptr(k_base), _ptr(v_base), row_stride,
          kv_head_stride, num_kv_rows, _ptr(kv_rows), _ptr(count), rows, cap, heads, kv_heads,
          d_qk, d_v, float(scale), _ptr(out), _ptr(lse), _ptr(status), _stream(stream))
    return out, lse


# ---------------------------------------------------------------------------
# Paged caches.  These calls are short next to their argument checks.  The
# common case (contiguous tensors, everything given) is checked and called by
# the extension module, which returns None for any other; then each argument is
# compared with what it should be in one expression, and the checkers below,
# which say what is wrong, run where that fails.
_ELEMENT = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}  # HS_BF16, ..
_I, _F = torch.int32, torch.float32


def _check_cache(k_cache, v_cache, device):
    """Paged caches [num_pages, page_size, kv_heads, d], any strides with
    contiguous rows (a [pages, heads, page, d] cache is passed transposed)."""
    if k_cache.dim() != 4 or k_cache.stride(3) != 1:
        raise ValueError("k_cache: [num_pages, page_size, kv_heads, d] with contiguous rows")
    if k_cache.get_device() != device:
        raise ValueError(f"k_cache: on {k_cache.device}, expected cuda:{device}")
    if v_cache is not None:
        if v_cache.dtype != k_cache.dtype or v_cache.device != k_cache.device:
            raise TypeError("v_cache: the type and device of k_cache")
        if v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride():
            raise ValueError("v_cache: the shape and strides of k_cache")


def _check_rows(t, dtype, name, device, rows, cols=None):
    """A tensor of `rows` leading entries (and `cols` columns at least, rows a
    stride apart) on CUDA device `device`."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{device}")
    if t.dim() != (1 if cols is None else 2) or t.shape[0] != rows:
        raise ValueError(f"{name}: expected {rows} rows, got shape {tuple(t.shape)}")
    if cols is None:
        if t.numel() > 1 and t.stride(0) != 1:
            raise ValueError(f"{name}: must be contiguous")
    elif t.shape[1] < cols or (t.shape[1] > 1 and t.stride(1) != 1) or (
            rows > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"{name}: needs {cols} contiguous columns, its rows apart")


def _vector(t, dtype, name, device, n):
    """Address of a contiguous 1-D tensor of n entries, or None."""
    if t is None:
        return None
    if (t.dtype is not dtype or t.get_device() != device or t.shape != (n,)
            or not t.is_contiguous()):
        _check_rows(t, dtype, name, device, n)
    return t.data_ptr()


def _matrix(t, dtype, name, device, rows, cols):
    """(address, elements between rows) of a 2-D tensor of at least `cols`
    columns, or (None, 0)."""
    if t is None:
        return None, 0
    shape = t.shape
    if (t.dtype is dtype and t.get_device() == device and len(shape) == 2 and shape[0] == rows
            and shape[1] >= cols and t.is_contiguous()):
        return t.data_ptr(), shape[1]
    _check_rows(t, dtype, name, device, rows, cols)
    return t.data_ptr(), t.stride(0) if rows > 1 else shape[1]


def _output(t, dtype, name, device, shape):
    """Address of a contiguous tensor of exactly this shape."""
    if (t.dtype is not dtype or t.get_device() != device or t.shape != shape
            or not t.is_contiguous()):
        if t.dtype != dtype or t.get_device() != device:
            raise TypeError(f"{name}: expected {dtype} on cuda:{device}")
        raise ValueError(f"{name}: expected contiguous {tuple(shape)}")
    return t.data_ptr()


def _status_ptr(status, device):
    """Address of a status word on CUDA device `device` or in pinned host memory."""
    if status is None:
        return None
    if status.numel() < 1:
        raise ValueError("status: needs a word")
    if status.dtype is not _I or status.get_device() != device:
        _check(status, _I, "status")
        if status.is_cuda:
            raise ValueError(f"status: on {status.device}, expected cuda:{device}")
        return _ptr(status)
    return status.data_ptr()


def _cache_strides(c, unit):
    """Page, row and head strides in elements times `unit`; 0 for a dimension
    of one entry (its stride is never used and may be anything)."""
    (p, r, h, _), (np_, nr, nh, _) = c.stride(), c.shape
    return p * unit if np_ > 1 else 0, r * unit if nr > 1 else 0, h * unit if nh > 1 else 0


def _check_i32(**values):
    """Host integers that the C call takes as int32 (ctypes would wrap them)."""
    for name, v in values.items():
        if not -1 << 31 <= v < 1 << 31:
            raise ValueError(f"{name}: {v} is out of range")


def _used_on(stream, *tensors):
    """Tensors made here and used on a stream other than the current one: the
    allocator must not hand their memory out before that stream is done."""
    if stream is not None:
        for t in tensors:
            t.record_stream(stream)


def _current_device(t, name):
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: must be on the current CUDA device")
    return dev


def paged_decode_workspace_bytes(rows, heads, kv_heads, d, max_len, *, window=0, num_sinks=0,
                                 with_score=False):
    _check_i32(rows=rows, heads=heads, kv_heads=kv_heads, d=d, max_len=max_len, window=window,
               num_sinks=num_sinks)
    return int(lib().hs_paged_decode_workspace_bytes(rows, heads, kv_heads, d, max_len, window,
                                                     num_sinks, 1 if with_score else 0))


def paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale, *, window=0, num_sinks=0,
                 max_len=None, k_scale=None, v_scale=None, score=None, score_decay=1.0, out=None,
                 lse=None, workspace=None, status=None, stream=None):
    """One new token's attention over every cached token (hs_paged_decode).

    q [rows, heads, d] bf16 or fp16 (heads packed, rows may be strided);
    k_cache, v_cache [num_pages, page_size, kv_heads, d] of q's type or
    float8_e4m3fn (then k_scale, v_scale fp32 [kv_heads] or None), same
    strides; block_table int32 [rows, blocks]; seq_lens int32 [rows]; max_len
    bounds seq_lens (default: what block_table and score hold).  score fp32
    [rows, >= max_len]: running scores, updated in place with the tokens'
    attention weights summed over the heads.  workspace: a contiguous CUDA
    tensor, used if it is large enough (paged_decode_workspace_bytes).  Returns
    (out [rows, heads, d] of q's type, lse fp32 [rows, heads]).  A call with out,
    lse and workspace given takes the shortest way through the binding."""
    dev = torch._C._cuda_getDevice()
    if _binding is not None:
        rc = _binding.paged_decode(dev, _raw_stream(dev, stream), q, k_cache, v_cache,
                                   block_table, seq_lens, scale, window, num_sinks, max_len,
                                   k_scale, v_scale, score, score_decay, out, lse, workspace,
                                   status)
        if rc is not None:
            if rc != HS_OK:
                raise HSError("hs_paged_decode", rc)
            return out, lse
    if q.get_device() != dev:
        raise ValueError("q: must be on the current CUDA device")
    qt, kt = q.dtype, k_cache.dtype
    if qt is not torch.bfloat16 and qt is not torch.float16:
        raise TypeError(f"q: expected torch.bfloat16 or torch.float16, got {qt}")
    if kt not in _ELEMENT:
        raise TypeError(f"k_cache: unsupported {kt}")
    if v_cache is None:
        raise ValueError("v_cache: needed")
    qshape, kshape, kstride, tshape = q.shape, k_cache.shape, k_cache.stride(), block_table.shape
    if (len(kshape) != 4 or kstride[3] != 1 or k_cache.get_device() != dev
            or v_cache.dtype is not kt or v_cache.shape != kshape or v_cache.stride() != kstride
            or v_cache.get_device() != dev):
        _check_cache(k_cache, v_cache, dev)
    rows, heads, d = qshape
    num_pages, page_size, kv_heads, dc = kshape
    if dc != d:
        raise ValueError("k_cache: head size of q")
    if q.is_contiguous():
        q_stride = heads * d
    else:
        q_stride, *rest = q.stride()
        if rest != [d, 1]:
            raise ValueError("q: heads must be packed")
    if (block_table.dtype is not _I or seq_lens.dtype is not _I
            or block_table.get_device() != dev or seq_lens.get_device() != dev
            or seq_lens.shape != (rows,) or len(tshape) != 2 or tshape[0] != rows
            or not seq_lens.is_contiguous() or not block_table.is_contiguous()):
        _check_rows(block_table, _I, "block_table", dev, rows, 0)
        _check_rows(seq_lens, _I, "seq_lens", dev, rows)
    blocks = tshape[1]
    if max_len is None:
        max_len = blocks * page_size
        if score is not None and score.dim() == 2:
            max_len = min(max_len, score.shape[1])
    if not 0 <= max_len < 1 << 31:
        raise ValueError("max_len: 0 to 2^31 - 1")
    _check_i32(window=window, num_sinks=num_sinks)
    score_ptr, score_stride, k_scale_ptr, v_scale_ptr = None, 0, None, None
    if score is not None:
        score_ptr, score_stride = _matrix(score, _F, "score", dev, rows, max_len)
    if k_scale is not None:
        k_scale_ptr = _vector(k_scale, _F, "k_scale", dev, kv_heads)
    if v_scale is not None:
        v_scale_ptr = _vector(v_scale, _F, "v_scale", dev, kv_heads)
    if out is None:
        out = torch.empty(rows, heads, d, dtype=qt, device=q.device)
        _used_on(stream, out)
    elif (out.dtype is not qt or out.get_device() != dev or out.shape != qshape
          or not out.is_contiguous()):
        _output(out, qt, "out", dev, qshape)
    if lse is None:
        lse = torch.empty(rows, heads, dtype=_F, device=q.device)
        _used_on(stream, lse)
    elif (lse.dtype is not _F or lse.get_device() != dev or lse.shape != (rows, heads)
          or not lse.is_contiguous()):
        _output(lse, _F, "lse", dev, (rows, heads))
    # A dimension of one entry may have any stride: it is never used.
    ps, rs, hstr, _ = kstride
    if num_pages <= 1 or page_size <= 1 or kv_heads <= 1:
        ps, rs, hstr = _cache_strides(k_cache, 1)
    call = lib().hs_paged_decode
    for again in (False, True):
        ws, ws_bytes = None, 0
        if workspace is not None:
            if workspace.get_device() != dev:
                raise ValueError("workspace: must be on q's device")
            _check_workspace(workspace)
            ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
        rc = call(q.data_ptr(), q_stride, _ELEMENT[qt], k_cache.data_ptr(), v_cache.data_ptr(),
                  _ELEMENT[kt], ps, rs, hstr, num_pages, page_size, block_table.data_ptr(),
                  block_table.stride(0) if rows > 1 else blocks, blocks, max_len,
                  seq_lens.data_ptr(), k_scale_ptr, v_scale_ptr, rows, heads, kv_heads, d, window,
                  num_sinks, scale, score_ptr, score_stride, score_decay, out.data_ptr(),
                  lse.data_ptr(), ws, ws_bytes, None if status is None else _status_ptr(status, dev),
                  _raw_stream(dev, stream))
        if rc != 3 or again:
            break
        # HS_ERR_CAPACITY: the workspace is missing or too small.
        n = paged_decode_workspace_bytes(rows, heads, kv_heads, d, max_len, window=window,
                                         num_sinks=num_sinks, with_score=score is not None)
        if n < 0:
            break
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
        _used_on(stream, workspace)
    if rc != HS_OK:
        raise HSError("hs_paged_decode", rc)
    return out, lse


def _evict_args(score, seq_lens, budget, max_len, recent, num_sinks, positions, next_pos,
                score_out, positions_out, lens_out, moves, stream):
    """Device, checked arguments of hs_evict_select, and what evict_select
    returns."""
    dev = _current_device(score, "score")
    if score.dim() != 2:
        raise ValueError("score: [rows, tokens]")
    rows, width = score.shape
    if max_len is None:
        max_len = width
    _check_i32(max_len=max_len, budget=budget, recent=recent, num_sinks=num_sinks)
    score_ptr, score_stride = _matrix(score, _F, "score", dev, rows, max_len)
    pos_ptr, pos_stride = _matrix(positions, _I, "positions", dev, rows, max_len)
    lens_ptr = _vector(seq_lens, _I, "seq_lens", dev, rows)
    next_ptr = _vector(next_pos, _I, "next_pos", dev, rows)
    if score_out is None:
        score_out, so_ptr, so_stride = score, score_ptr, score_stride
    else:
        so_ptr, so_stride = _matrix(score_out, _F, "score_out", dev, rows, max_len)
    if positions_out is None:
        positions_out, po_ptr, po_stride = positions, pos_ptr, pos_stride
    else:
        po_ptr, po_stride = _matrix(positions_out, _I, "positions_out", dev, rows, max_len)
    if lens_out is None:
        lens_out, lo_ptr = seq_lens, lens_ptr
    else:
        lo_ptr = _vector(lens_out, _I, "lens_out", dev, rows)
    if moves is None:
        cap = max(0, min(budget, max_len - budget))
        i32 = dict(dtype=_I, device=score.device)
        moves = (torch.empty(rows, cap, **i32), torch.empty(rows, cap, **i32),
                 torch.empty(rows, **i32))
        _used_on(stream, *moves)
    src, dst, count = moves
    shape = src.shape
    if len(shape) != 2 or shape[0] != rows:
        raise ValueError(f"moves[0]: expected {rows} rows, got shape {tuple(shape)}")
    args = (score_ptr, score_stride, pos_ptr, pos_stride, lens_ptr, next_ptr, rows, max_len,
            budget, recent, num_sinks, so_ptr, so_stride, po_ptr, po_stride, lo_ptr,
            _output(src, _I, "moves[0]", dev, shape), _output(dst, _I, "moves[1]", dev, shape),
            _vector(count, _I, "moves[2]", dev, rows), shape[1])
    return dev, args, (score_out, positions_out, lens_out, moves)


def _move_args(k_cache, v_cache, block_table, rows, dev):
    shape, stride = k_cache.shape, k_cache.stride()
    if (len(shape) != 4 or stride[3] != 1 or k_cache.get_device() != dev
            or v_cache is not None and (v_cache.dtype is not k_cache.dtype
                                        or v_cache.shape != shape or v_cache.stride() != stride
                                        or v_cache.get_device() != dev)):
        _check_cache(k_cache, v_cache, dev)
    table, table_stride = _matrix(block_table, _I, "block_table", dev, rows, 0)
    num_pages, page_size, kv_heads, d = shape
    e = k_cache.element_size()
    ps, rs, hstr = _cache_strides(k_cache, e)
    return (k_cache.data_ptr(), None if v_cache is None else v_cache.data_ptr(), ps, rs, hstr,
            kv_heads, d * e, num_pages, page_size, table, table_stride, block_table.shape[1])


def evict_select(score, seq_lens, budget, *, max_len=None, recent=0, num_sinks=0, positions=None,
                 next_pos=None, score_out=None, positions_out=None, lens_out=None, moves=None,
                 status=None, stream=None):
    """Which tokens a request over its budget keeps (hs_evict_select).

    score fp32 [rows, >= max_len]; seq_lens int32 [rows]; positions int32
    [rows, >= max_len] or None; next_pos int32 [rows] or None; max_len
    defaults to score's width.  score_out, positions_out and lens_out default
    to the inputs (updated in place).  Returns (score_out, positions_out,
    lens_out, (move_src, move_dst int32 [rows, cap], move_count int32
    [rows]))."""
    dev, args, result = _evict_args(score, seq_lens, budget, max_len, recent, num_sinks,
                                    positions, next_pos, score_out, positions_out, lens_out,
                                    moves, stream)
    rc = lib().hs_evict_select(*args, _status_ptr(status, dev), _raw_stream(dev, stream))
    if rc != HS_OK:
        raise HSError("hs_evict_select", rc)
    return result


def evict_move(moves, k_cache, v_cache, block_table, *, status=None, stream=None):
    """Apply evict_select's moves to a paged cache [num_pages, page_size,
    kv_heads, d] of any type (v_cache None: one cache) (hs_evict_move)."""
    src, dst, count = moves
    dev = _current_device(src, "moves")
    shape = src.shape
    if len(shape) != 2:
        raise ValueError("moves[0]: [rows, cap]")
    rows, cap = shape
    lists = (_output(src, _I, "moves[0]", dev, shape), _output(dst, _I, "moves[1]", dev, shape),
             _vector(count, _I, "moves[2]", dev, rows))
    rc = lib().hs_evict_move(*_move_args(k_cache, v_cache, block_table, rows, dev), *lists, rows,
                             cap, _status_ptr(status, dev), _raw_stream(dev, stream))
    if rc != HS_OK:
        raise HSError("hs_evict_move", rc)


def evict(score, seq_lens, budget, k_cache, v_cache, block_table, *, max_len=None, recent=0,
          num_sinks=0, positions=None, next_pos=None, score_out=None, positions_out=None,
          lens_out=None, moves=None, status=None, stream=None):
    """evict_select, then evict_move on one layer's caches (hs_evict); same
    arguments and result as evict_select."""
    if _binding is not None:
        dev = torch._C._cuda_getDevice()
        rc = _binding.evict(dev, _raw_stream(dev, stream), score, seq_lens, budget, k_cache,
                            v_cache, block_table, max_len, recent, num_sinks, positions, next_pos,
                            score_out, positions_out, lens_out, moves, status)
        if rc is not None:
            if rc != HS_OK:
                raise HSError("hs_evict", rc)
            return (score if score_out is None else score_out,
                    positions if positions_out is None else positions_out,
                    seq_lens if lens_out is None else lens_out, moves)
    dev, args, result = _evict_args(score, seq_lens, budget, max_len, recent, num_sinks,
                                    positions, next_pos, score_out, positions_out, lens_out,
                                    moves, stream)
    rc = lib().hs_evict(*args, *_move_args(k_cache, v_cache, block_table, score.shape[0], dev),
                        _status_ptr(status, dev), _raw_stream(dev, stream))
    if rc != HS_OK:
        raise HSError("hs_evict", rc)
    return result
