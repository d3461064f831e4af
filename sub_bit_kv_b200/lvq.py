"""ctypes binding of liblvq (include/lvq.h), same names as the C ABI.

Argument marshalling only: every step of the codec and the attention runs in
the library's CUDA kernels.  torch supplies device memory and streams.  If the
library is missing, or the device is not sm_100, calls raise: there is no
fallback path.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblvq.so")

LVQ_OK, LVQ_EINVAL, LVQ_EUNSUPPORTED, LVQ_ECAPACITY, LVQ_ECUDA, LVQ_ETIMEOUT, LVQ_EDEVICE = range(7)


class LvqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class lvq_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_layers", "n_kv_heads", "n_q_heads", "head_dim", "T", "Tc", "G", "K", "n_sink", "n_recent",
        "page_tokens", "max_batch", "max_ctx", "max_splits")] + [("rope_base", ctypes.c_float)] + [
        ("pool_pages", ctypes.c_int32), ("reserved_", ctypes.c_int32), ("page_table", ctypes.c_void_p)]


class lvq_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "c", "n_groups", "n_blocks", "ring_tokens", "max_pages", "page_bytes", "rope_coarse",
        "page_table_stride")] + [
        ("idx_bytes", ctypes.c_size_t), ("idx_strides", ctypes.c_int64 * 8), ("page_table_bytes", ctypes.c_size_t),
        ("cb_bytes", ctypes.c_size_t), ("cb_strides", ctypes.c_int64 * 7),
        ("cbp_bytes", ctypes.c_size_t), ("cbp_strides", ctypes.c_int64 * 8),
        ("cb_norm_bytes", ctypes.c_size_t),
        ("sink_bytes", ctypes.c_size_t), ("sink_strides", ctypes.c_int64 * 7),
        ("ring_bytes", ctypes.c_size_t), ("ring_strides", ctypes.c_int64 * 7),
        ("rope_bytes", ctypes.c_size_t), ("workspace_bytes", ctypes.c_size_t)]


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_SIGS = {
    "lvq_cache_layout": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout)],
    "lvq_pack_codebooks": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _P, _P, _P, _P],
    "lvq_rope_table": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _P, _P],
    "lvq_encode_prefill": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _I32, _I32, _P,
                           ctypes.c_int64, _I32, _I32, _I32, _I32, _P, _P, _P, _P],
    "lvq_encode_page": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _I32, _P, _P, _P, _P, _P,
                        _P, _P, _P],
    "lvq_decode_attention": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _I32, _I32, _I32, _P,
                             _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P],
    "lvq_dequantize": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _I32, _I32, _I32, _I32, _P,
                       _P, _I32, _I32, _P, _P],
    "lvq_kmeans_update": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _I32, _I32, _P,
                          ctypes.c_int64, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P],
    "lvq_status_string": [_I32],
    "lvq_debug_faults": [ctypes.c_int64, _I32],
    "lvq_decode_max_ctas": [_I32],
    "lvq_decode_attention_noalloc": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _I32, _I32, _I32,
                                     _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _P],
    "lvq_pool_create": [_I32, ctypes.POINTER(_P)],
    "lvq_pool_destroy": [_P],
    "lvq_pool_alloc": [_P, _I32, ctypes.POINTER(_I32)],
    "lvq_pool_free": [_P, ctypes.POINTER(_I32), _I32],
    "lvq_pool_available": [_P],
    "lvq_pool_share": [_P, ctypes.POINTER(_I32), _I32],
    "lvq_pool_holders": [_P, _I32],
    "lvq_pool_renumber": [_P, ctypes.POINTER(_I32)],
    "lvq_plan_compaction": [_I32, _P, _I32, _P, _P, ctypes.POINTER(_I32)],
    "lvq_copy_pages": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _I32, _P, _P, _P, _P],
    "lvq_compact_pages": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _I32, _P, _P, _P, _P, _P, _P],
    "lvq_fork_requests": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _I32, _I32, ctypes.POINTER(_I32),
                          _I32, ctypes.POINTER(_I32), _P, _P, _P, _P, _P, _P, _P, _P],
    "lvq_decode_attention_shared": [ctypes.POINTER(lvq_config), ctypes.POINTER(lvq_layout), _I32, _I32, _I32, _P,
                                    _P, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _P],
}
EXPORTED = tuple(_SIGS)

_lib = None


def lib():
    """Loads liblvq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m sub_bit_kv_b200._build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(h, name)
            fn.argtypes = args
            fn.restype = {"lvq_status_string": ctypes.c_char_p, "lvq_pool_destroy": None}.get(name, ctypes.c_int)
        _lib = h
    return _lib


def status_string(s: int) -> str:
    return lib().lvq_status_string(int(s)).decode()


def _check(s: int, where: str):
    if s != LVQ_OK:
        raise LvqError(s, where)


def make_config(n_layers, n_kv_heads, n_q_heads, head_dim, T, Tc, G, n_sink, n_recent, max_batch, max_ctx,
                max_splits=64, rope_base=10000.0, K=256, page_tokens=8, pool_pages=0) -> lvq_config:
    """pool_pages > 0: pool mode (CodedCache allocates the page table and sets page_table)."""
    return lvq_config(n_layers, n_kv_heads, n_q_heads, head_dim, T, Tc, G, K, n_sink, n_recent, page_tokens,
                      max_batch, max_ctx, max_splits, rope_base, pool_pages, 0, None)


class PagePool:
    """The library's host-side page allocator (lvq_pool): physical page ids of a pool, handed
    out lowest first and taken back when a request ends."""

    def __init__(self, n_pages: int):
        h = _P()
        _check(lib().lvq_pool_create(int(n_pages), ctypes.byref(h)), "lvq_pool_create")
        self._h = h
        self.n_pages = int(n_pages)

    def alloc(self, n: int) -> list:
        ids = (_I32 * max(1, n))()
        _check(lib().lvq_pool_alloc(self._h, int(n), ids), "lvq_pool_alloc")
        return list(ids[:n])

    def free(self, ids) -> None:
        arr = (_I32 * max(1, len(ids)))(*ids)
        _check(lib().lvq_pool_free(self._h, arr, len(ids)), "lvq_pool_free")

    def available(self) -> int:
        return int(lib().lvq_pool_available(self._h))

    def share(self, ids) -> None:
        """One more holder of each page; each holder frees it once."""
        arr = (_I32 * max(1, len(ids)))(*ids)
        _check(lib().lvq_pool_share(self._h, arr, len(ids)), "lvq_pool_share")

    def holders(self, page: int) -> int:
        """Holders of a page (0: free, -1: no such page)."""
        return int(lib().lvq_pool_holders(self._h, int(page)))

    def renumber(self, new_id) -> None:
        """The pages take the ids of a compaction plan (new_id[old], -1 for free pages)."""
        new_id = torch.as_tensor(new_id, dtype=torch.int32, device="cpu").contiguous()
        if new_id.numel() != self.n_pages:
            raise ValueError(f"new_id holds {new_id.numel()} ids, the pool {self.n_pages} pages")
        _check(lib().lvq_pool_renumber(self._h, ctypes.cast(new_id.data_ptr(), ctypes.POINTER(_I32))),
               "lvq_pool_renumber")

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.lvq_pool_destroy(h)
            self._h = None


def lvq_cache_layout(cfg: lvq_config) -> lvq_layout:
    lay = lvq_layout()
    _check(lib().lvq_cache_layout(ctypes.byref(cfg), ctypes.byref(lay)), "lvq_cache_layout")
    return lay


def _ptr(t: Optional[torch.Tensor], name: str, dtype=None, min_bytes: int = 0, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() * t.element_size() < min_bytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, needs {min_bytes}")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:             # the same handle without a Stream object: 0.3 us instead of 3.2
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _current(stream):
    """Makes the call's stream the current one for torch's own allocations and copies."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(_stream(stream), device=torch.cuda.current_device()))


def lvq_pack_codebooks(cfg, lay, cb, cbp, cb_norm=None, stream=None):
    _check(lib().lvq_pack_codebooks(
        ctypes.byref(cfg), ctypes.byref(lay), _ptr(cb, "cb", torch.bfloat16, lay.cb_bytes),
        _ptr(cbp, "cbp", torch.bfloat16, lay.cbp_bytes),
        _ptr(cb_norm, "cb_norm", torch.float32, lay.cb_norm_bytes, optional=True), _stream(stream)),
        "lvq_pack_codebooks")


def lvq_rope_table(cfg, lay, rope, stream=None):
    _check(lib().lvq_rope_table(ctypes.byref(cfg), ctypes.byref(lay), _ptr(rope, "rope", torch.float32,
                                                                           lay.rope_bytes), _stream(stream)),
           "lvq_rope_table")


def lvq_encode_prefill(cfg, lay, layer, req, kv, tok_begin, n_tok, coded_offset, cb, idx, dev_status,
                       kv_tok_stride=None, stream=None):
    """kv: bf16 [2][T][N][Hkv][d] of one layer and request (contiguous); with layer = -1
    (every layer in one call) [n_layers][2][T][N][Hkv][d]."""
    if layer == -1:
        if kv.dim() != 6 or kv.shape[0] != cfg.n_layers:
            raise ValueError("layer = -1 takes kv as [n_layers][2][T][N][Hkv][d]")
        kv1 = kv[0]
    else:
        kv1 = kv
    if kv1.dim() != 5 or kv1.shape[0] != 2 or kv1.shape[1] != cfg.T:
        raise ValueError("kv must be [2][T][N][Hkv][d]")
    n_total = kv1.shape[2]
    stride = kv_tok_stride if kv_tok_stride is not None else kv1.shape[3] * kv1.shape[4]
    _check(lib().lvq_encode_prefill(
        ctypes.byref(cfg), ctypes.byref(lay), layer, req, _ptr(kv, "kv", torch.bfloat16), stride, n_total,
        tok_begin, n_tok, coded_offset, _ptr(cb, "cb", torch.bfloat16, lay.cb_bytes),
        _ptr(idx, "idx", torch.uint8, lay.idx_bytes), _ptr(dev_status, "dev_status", torch.int32, 4),
        _stream(stream)), "lvq_encode_prefill")


def lvq_kmeans_update(cfg, lay, layer, req, kv, tok_begin, n_tok, coded_offset, idx, cb, counts, dev_status,
                      kv_tok_stride=None, stream=None):
    """Update step of one k-means iteration after lvq_encode_prefill wrote the codes.
    kv: bf16 [2][T][N][Hkv][d] of one layer and request (contiguous); cb is updated in
    place; counts: None or int32 [2][n_blk][Hkv][n_g][256] (the library writes uint32)."""
    if kv.dim() != 5 or kv.shape[0] != 2 or kv.shape[1] != cfg.T:
        raise ValueError("kv must be [2][T][N][Hkv][d]")
    n_total = kv.shape[2]
    stride = kv_tok_stride if kv_tok_stride is not None else kv.shape[3] * kv.shape[4]
    n_counts = 2 * lay.n_blocks * cfg.n_kv_heads * lay.n_groups * 256
    _check(lib().lvq_kmeans_update(
        ctypes.byref(cfg), ctypes.byref(lay), layer, req, _ptr(kv, "kv", torch.bfloat16), stride, n_total,
        tok_begin, n_tok, coded_offset, _ptr(idx, "idx", torch.uint8, lay.idx_bytes),
        _ptr(cb, "cb", torch.bfloat16, lay.cb_bytes),
        _ptr(counts, "counts", torch.int32, 4 * n_counts, optional=True),
        _ptr(dev_status, "dev_status", torch.int32, 4), _stream(stream)), "lvq_kmeans_update")


def lvq_debug_faults(wait_iters: int = 0, fault_mask: int = 0):
    """Test hook: bound of every device-side wait (0: the normal bound) and copies that never
    happen (bit 0: decode's first code chunk, bit 1: k-means' first tile).  Process-global."""
    _check(lib().lvq_debug_faults(int(wait_iters), int(fault_mask)), "lvq_debug_faults")


def lvq_decode_max_ctas(max_ctas: int = 0):
    """Caps the CTAs of later lvq_decode_attention calls (0: one per work item); with more work
    items than the cap each CTA walks a run of them.  Process-global."""
    _check(lib().lvq_decode_max_ctas(int(max_ctas)), "lvq_decode_max_ctas")


def lvq_encode_page(cfg, lay, batch, ctx_len, coded_len, ring, cb, cb_norm, idx, dev_status, stream=None):
    _check(lib().lvq_encode_page(
        ctypes.byref(cfg), ctypes.byref(lay), batch, _ptr(ctx_len, "ctx_len", torch.int32, 4 * batch),
        _ptr(coded_len, "coded_len", torch.int32, 4 * batch), _ptr(ring, "ring", torch.bfloat16, lay.ring_bytes),
        _ptr(cb, "cb", torch.bfloat16, lay.cb_bytes), _ptr(cb_norm, "cb_norm", torch.float32, lay.cb_norm_bytes),
        _ptr(idx, "idx", torch.uint8, lay.idx_bytes),
        _ptr(dev_status, "dev_status", torch.int32, 4), _stream(stream)), "lvq_encode_page")


def lvq_decode_attention(cfg, lay, layer, step, batch, q, ctx_len, coded_len, sink, ring, idx, cbp, rope,
                         num_splits, workspace, out, lse, dev_status, split_lse=None, stream=None):
    d = cfg.head_dim
    _check(lib().lvq_decode_attention(
        ctypes.byref(cfg), ctypes.byref(lay), layer, step, batch,
        _ptr(q, "q", torch.bfloat16, 2 * batch * cfg.n_q_heads * d),
        _ptr(ctx_len, "ctx_len", torch.int32, 4 * batch), _ptr(coded_len, "coded_len", torch.int32, 4 * batch),
        _ptr(sink, "sink", torch.bfloat16, lay.sink_bytes), _ptr(ring, "ring", torch.bfloat16, lay.ring_bytes),
        _ptr(idx, "idx", torch.uint8, lay.idx_bytes), _ptr(cbp, "cbp", torch.bfloat16, lay.cbp_bytes),
        _ptr(rope, "rope", torch.float32, lay.rope_bytes), num_splits,
        _ptr(workspace, "workspace", torch.float32, lay.workspace_bytes),
        _ptr(out, "out", torch.float32, 4 * batch * cfg.n_q_heads * d),
        _ptr(lse, "lse", torch.float32, 4 * batch * cfg.n_q_heads),
        _ptr(split_lse, "split_lse", torch.float32, 4 * batch * cfg.n_q_heads * (num_splits + 1), optional=True),
        _ptr(dev_status, "dev_status", torch.int32, 4), _stream(stream)), "lvq_decode_attention")


def lvq_decode_attention_noalloc(cfg, lay, layer, step, batch, q, ctx_len, coded_len, sink, ring, idx, cbp, rope,
                                 num_splits, out, lse, dev_status, split_lse=None, stream=None):
    """lvq_decode_attention with the library's own 4 MiB device workspace (no workspace argument)."""
    d = cfg.head_dim
    _check(lib().lvq_decode_attention_noalloc(
        ctypes.byref(cfg), ctypes.byref(lay), layer, step, batch,
        _ptr(q, "q", torch.bfloat16, 2 * batch * cfg.n_q_heads * d),
        _ptr(ctx_len, "ctx_len", torch.int32, 4 * batch), _ptr(coded_len, "coded_len", torch.int32, 4 * batch),
        _ptr(sink, "sink", torch.bfloat16, lay.sink_bytes), _ptr(ring, "ring", torch.bfloat16, lay.ring_bytes),
        _ptr(idx, "idx", torch.uint8, lay.idx_bytes), _ptr(cbp, "cbp", torch.bfloat16, lay.cbp_bytes),
        _ptr(rope, "rope", torch.float32, lay.rope_bytes), num_splits,
        _ptr(out, "out", torch.float32, 4 * batch * cfg.n_q_heads * d),
        _ptr(lse, "lse", torch.float32, 4 * batch * cfg.n_q_heads),
        _ptr(split_lse, "split_lse", torch.float32, 4 * batch * cfg.n_q_heads * (num_splits + 1), optional=True),
        _ptr(dev_status, "dev_status", torch.int32, 4), _stream(stream)), "lvq_decode_attention_noalloc")


def _on(dev: int, t: Optional[torch.Tensor], name: str, dtype, min_bytes: int):
    """_ptr for the calls below, which also refuse a tensor of another device than `dev`, the current one."""
    if t is not None and t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.nbytes >= min_bytes:
        return t.data_ptr()
    _ptr(t, name, dtype, min_bytes)             # says what is wrong, unless it is the device
    raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")


def _table(cfg, lay, dev: int, page_table):
    if cfg.pool_pages > 0:
        return _on(dev, page_table, "page_table", torch.int32, lay.page_table_bytes)
    if page_table is not None:
        raise ValueError("page_table belongs to pool mode")
    return None


def lvq_decode_attention_shared(cfg, lay, layer, step, batch, q, ctx_len, coded_len, group_begin, group_tokens, sink,
                                ring, idx, cbp, rope, num_splits, workspace, out, lse, dev_status, stream=None):
    """lvq_decode_attention for groups of requests whose first coded tokens are the same: group i holds
    the requests group_begin[i] .. group_begin[i + 1] - 1 and shares group_tokens[i] coded tokens, which
    are restored once for every 16 (request, query head) rows of a KV head.  group_begin: int32 [n_groups + 1], group_tokens: int32 [n_groups],
    both on the device.  num_splits = 0: the library's choice."""
    d, hq, dev = cfg.head_dim, cfg.n_q_heads, torch.cuda.current_device()
    n_groups = 0 if group_tokens is None else group_tokens.numel()
    _check(lib().lvq_decode_attention_shared(
        ctypes.byref(cfg), ctypes.byref(lay), layer, step, batch,
        _on(dev, q, "q", torch.bfloat16, 2 * batch * hq * d),
        _on(dev, ctx_len, "ctx_len", torch.int32, 4 * batch), _on(dev, coded_len, "coded_len", torch.int32, 4 * batch),
        n_groups, _on(dev, group_begin, "group_begin", torch.int32, 4 * (n_groups + 1)),
        _on(dev, group_tokens, "group_tokens", torch.int32, 4 * n_groups),
        _on(dev, sink, "sink", torch.bfloat16, lay.sink_bytes), _on(dev, ring, "ring", torch.bfloat16, lay.ring_bytes),
        _on(dev, idx, "idx", torch.uint8, lay.idx_bytes), _on(dev, cbp, "cbp", torch.bfloat16, lay.cbp_bytes),
        _on(dev, rope, "rope", torch.float32, lay.rope_bytes), num_splits,
        _on(dev, workspace, "workspace", torch.float32, lay.workspace_bytes),
        _on(dev, out, "out", torch.float32, 4 * batch * hq * d), _on(dev, lse, "lse", torch.float32, 4 * batch * hq),
        _on(dev, dev_status, "dev_status", torch.int32, 4), _stream(stream)), "lvq_decode_attention_shared")


def lvq_copy_pages(cfg, lay, pairs, idx, dev_status, stream=None):
    """Copies pages of the pool in every (layer, block, head, K/V).  pairs: device int32 [n][2], (source,
    destination); no destination twice, none that is also a source."""
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [n][2]")
    dev, n = torch.cuda.current_device(), pairs.shape[0]
    _check(lib().lvq_copy_pages(
        ctypes.byref(cfg), ctypes.byref(lay), n, _on(dev, pairs, "pairs", torch.int32, 0),
        _on(dev, idx, "idx", torch.uint8, lay.idx_bytes), _on(dev, dev_status, "dev_status", torch.int32, 4),
        _stream(stream)), "lvq_copy_pages")


class CompactionPlan:
    """What lvq_plan_compaction writes: new_id (host int32 [n_pages], -1: not live), n_live, and the
    moves for lvq_compact_pages (host int32 [n_moves][2])."""

    def __init__(self, n_pages: int, order):
        if isinstance(order, torch.Tensor):
            order = order.to(device="cpu", dtype=torch.int32).contiguous()
            n, ids = order.numel(), order.data_ptr()
        else:
            order = array.array("i", order)     # (a quarter of the time that a tensor takes from a list)
            n, ids = len(order), order.buffer_info()[0]
        self.n_pages = int(n_pages)
        # one buffer, so that it goes to the device in one copy: the moves, then new_id
        self._room = 2 * (n + n // 2)
        self._host = torch.empty(self._room + max(1, self.n_pages), dtype=torch.int32, pin_memory=_has_cuda())
        k = _I32()
        base = self._host.data_ptr()
        _check(lib().lvq_plan_compaction(self.n_pages, ids if n else None, n, base + 4 * self._room,
                                         base if n else None, ctypes.byref(k)), "lvq_plan_compaction")
        self.n_moves = k.value

    @property
    def moves(self) -> torch.Tensor:
        return self._host[:2 * self.n_moves].view(-1, 2)

    @property
    def new_id(self) -> torch.Tensor:
        return self._host[self._room:]

    @property
    def n_live(self) -> int:
        return int((self.new_id >= 0).sum())


@functools.lru_cache(None)
def _has_cuda() -> bool:
    return torch.cuda.is_available()


def lvq_plan_compaction(n_pages, order) -> CompactionPlan:
    """Plans a compaction of a pool of n_pages pages: the pages in `order` (a list or a CPU tensor; a page
    named again keeps its first place) get the ids 0, 1, ...; host work only."""
    return CompactionPlan(n_pages, order)


def lvq_compact_pages(cfg, lay, plan: CompactionPlan, page_table, idx, dev_status, stream=None):
    """Carries out a compaction plan in place on the pool's codes and rewrites the page table.  Not under
    capture: a plan belongs to one state of the pool, a replay would apply it to another."""
    if plan.n_pages != cfg.pool_pages:
        raise ValueError(f"the plan is for a pool of {plan.n_pages} pages, the configuration has {cfg.pool_pages}")
    dev, raw = torch.cuda.current_device(), _stream(stream)
    table, codes = _table(cfg, lay, dev, page_table), _on(dev, idx, "idx", torch.uint8, lay.idx_bytes)
    status = _on(dev, dev_status, "dev_status", torch.int32, 4)
    with _current(stream):                      # (the plan's device copy belongs to the call's stream)
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("lvq_compact_pages cannot be captured: a plan belongs to one state of the pool")
        on_device = plan._host.cuda(non_blocking=True)
        base = on_device.data_ptr()
        _check(lib().lvq_compact_pages(ctypes.byref(cfg), ctypes.byref(lay), plan.n_moves, base, base + 4 * plan._room,
                                       table, codes, status, raw), "lvq_compact_pages")


def lvq_fork_requests(cfg, lay, parent, children, coded_tokens, tail_pages, ctx_len, coded_len, sink, ring, idx,
                      page_table, dev_status, stream=None):
    """Makes every request of `children` (a list) a copy of `parent`, which has coded_tokens coded tokens.
    tail_pages: in pool mode, where coded_tokens is not a multiple of 8, a page of its own for each child
    (else None).  CodedCache.fork also does the pool's bookkeeping."""
    dev, n = torch.cuda.current_device(), len(children)
    if tail_pages is not None and len(tail_pages) != n:
        raise ValueError(f"{len(tail_pages)} tail pages for {n} children")
    b = 4 * cfg.max_batch
    _check(lib().lvq_fork_requests(
        ctypes.byref(cfg), ctypes.byref(lay), parent, n, (_I32 * max(1, n))(*children), coded_tokens,
        None if tail_pages is None else (_I32 * max(1, n))(*tail_pages),
        _on(dev, ctx_len, "ctx_len", torch.int32, b), _on(dev, coded_len, "coded_len", torch.int32, b),
        _on(dev, sink, "sink", torch.bfloat16, lay.sink_bytes), _on(dev, ring, "ring", torch.bfloat16, lay.ring_bytes),
        _on(dev, idx, "idx", torch.uint8, lay.idx_bytes), _table(cfg, lay, dev, page_table),
        _on(dev, dev_status, "dev_status", torch.int32, 4), _stream(stream)), "lvq_fork_requests")


def lvq_dequantize(cfg, lay, layer, step, req, kv, idx, cbp, tok_begin, n_tok, out, stream=None):
    _check(lib().lvq_dequantize(
        ctypes.byref(cfg), ctypes.byref(lay), layer, step, req, kv, _ptr(idx, "idx", torch.uint8, lay.idx_bytes),
        _ptr(cbp, "cbp", torch.bfloat16, lay.cbp_bytes), tok_begin, n_tok,
        _ptr(out, "out", torch.bfloat16, 2 * n_tok * cfg.n_kv_heads * cfg.head_dim), _stream(stream)),
        "lvq_dequantize")


class CodedCache:
    """Device buffers of one configuration, allocated with torch to the sizes
    lvq_cache_layout gives (plumbing: the library itself allocates nothing)."""

    def __init__(self, cfg: lvq_config, device="cuda"):
        self.cfg = cfg
        self.lay = lay = lvq_cache_layout(cfg)
        dev = torch.device(device)
        self.idx = torch.zeros(lay.idx_bytes, dtype=torch.uint8, device=dev)
        self.cb = torch.zeros(lay.cb_bytes // 2, dtype=torch.bfloat16, device=dev)
        self.cbp = torch.zeros(lay.cbp_bytes // 2, dtype=torch.bfloat16, device=dev)
        self.cb_norm = torch.zeros(lay.cb_norm_bytes // 4, dtype=torch.float32, device=dev)
        self.sink = torch.zeros(lay.sink_bytes // 2, dtype=torch.bfloat16, device=dev)
        self.ring = torch.zeros(lay.ring_bytes // 2, dtype=torch.bfloat16, device=dev)
        self.rope = torch.zeros(lay.rope_bytes // 4, dtype=torch.float32, device=dev)
        self.workspace = torch.zeros(lay.workspace_bytes // 4, dtype=torch.float32, device=dev)
        self.ctx_len = torch.zeros(cfg.max_batch, dtype=torch.int32, device=dev)
        self.coded_len = torch.zeros(cfg.max_batch, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.pool = None
        if cfg.pool_pages > 0:
            # pool mode: the page table (every entry unassigned) and the host allocator; the
            # config carries the table's device address from here on
            self.page_table = torch.full((lay.page_table_bytes // 4,), -1, dtype=torch.int32, device=dev)
            cfg.page_table = self.page_table.data_ptr()
            self.pool = PagePool(cfg.pool_pages)
            self.pages = [[] for _ in range(cfg.max_batch)]       # host copy: physical page of logical page i

    # pool mode: pages of a request
    def assign_pages(self, b: int, n_pages: int) -> list:
        """Makes request b hold at least n_pages logical pages (new ones from the pool) and writes
        its page-table row.  Returns the request's physical pages."""
        have = self.pages[b]
        if n_pages > len(have):
            have += self.pool.alloc(n_pages - len(have))
            row = torch.tensor(have, dtype=torch.int32)
            self.page_table[b * self.lay.page_table_stride: b * self.lay.page_table_stride + len(have)].copy_(row)
        return list(have)

    def release(self, b: int) -> None:
        """Request b ends: its pages go back to the pool and its page-table row is cleared."""
        if self.pages[b]:
            self.pool.free(self.pages[b])
            self.pages[b] = []
            self.page_table[b * self.lay.page_table_stride:(b + 1) * self.lay.page_table_stride].fill_(-1)

    def fork(self, parent: int, children, coded_tokens: int, stream=None, check: bool = False) -> None:
        """Every request of `children` becomes a copy of request `parent`, which has coded_tokens coded
        tokens.  In pool mode the children hold the parent's full pages with it and get a page of their
        own for a partial last one; they must hold no pages before.

        The call does not wait: the children's page lists are filled on the caller's word.  Where the device
        finds otherwise (coded_len[parent] is not coded_tokens, the parent's counters or its partial page are
        bad), it writes the status and no child, and every child has to be released before it, assign_pages
        or compact is used on.  check=True waits for the fork and, refused, gives the pages back and raises
        LvqError (it reads a status word of its own; not under capture)."""
        children = list(children)
        tails = None
        status = self.status
        if self.pool is not None:
            if any(self.pages[c] for c in children):
                raise ValueError("a child holds pages: release it first")
            full, rest = divmod(coded_tokens, 8)
            if len(self.pages[parent]) < full + (rest > 0):
                raise ValueError(f"request {parent} holds {len(self.pages[parent])} pages, {coded_tokens} coded tokens need more")
            if rest:
                tails = self.pool.alloc(len(children))
        try:
            with _current(stream) if check else contextlib.nullcontext():
                if check:
                    if status.is_cuda and torch.cuda.is_current_stream_capturing():
                        raise RuntimeError("a captured fork cannot be checked")
                    status = torch.zeros_like(status)
                lvq_fork_requests(self.cfg, self.lay, parent, children, coded_tokens, tails, self.ctx_len, self.coded_len,
                                  self.sink, self.ring, self.idx, getattr(self, "page_table", None), status, stream)
                if check:
                    _check(int(status.item()), "lvq_fork_requests")
        except Exception:
            if tails:
                self.pool.free(tails)
            raise
        if self.pool is not None:
            for i, c in enumerate(children):
                self.pool.share(self.pages[parent][:full])
                self.pages[c] = self.pages[parent][:full] + ([tails[i]] if tails else [])

    def compact(self, stream=None) -> int:
        """Pool mode: the pages in use move to the lowest ids, each request's pages next to one another
        (a shared page with the first request that holds it), so that its reads form long runs.
        Returns the number of pages moved."""
        if self.pool is None:
            raise ValueError("compaction belongs to pool mode")
        plan = lvq_plan_compaction(self.cfg.pool_pages, [p for row in self.pages for p in row])
        self.pool.renumber(plan.new_id)         # refuses pages that are held outside the requests' lists
        try:
            lvq_compact_pages(self.cfg, self.lay, plan, self.page_table, self.idx, self.status, stream)
        except Exception:
            old = torch.full_like(plan.new_id, -1)
            live = plan.new_id >= 0
            old[plan.new_id[live].long()] = torch.arange(old.numel(), dtype=torch.int32)[live]
            self.pool.renumber(old)
            raise
        to = plan.new_id.tolist()
        self.pages = [[to[p] for p in row] for row in self.pages]
        return plan.n_moves

    # shaped views of the caller-owned buffers (layouts from lvq_cache_layout)
    def cb_view(self):
        c = self.cfg
        return self.cb.view(c.n_layers, 2, self.lay.n_blocks, c.n_kv_heads, self.lay.n_groups, 256, c.G)

    def sink_view(self):
        c = self.cfg
        return self.sink.view(c.n_layers, 2, c.T, c.max_batch, c.n_kv_heads, c.n_sink, c.head_dim)

    def ring_view(self):
        c = self.cfg
        return self.ring.view(c.n_layers, 2, c.T, c.max_batch, c.n_kv_heads, self.lay.ring_tokens, c.head_dim)

    def idx_view(self):
        c, l = self.cfg, self.lay
        if c.pool_pages > 0:       # [layer][n_blk][Hkv][kv][pool page][n_g][8]
            return self.idx.view(c.n_layers, l.n_blocks, c.n_kv_heads, 2, c.pool_pages, l.n_groups, 8)
        return self.idx.view(c.n_layers, l.n_blocks, c.max_batch, c.n_kv_heads, 2, l.max_pages, l.n_groups, 8)

    def check_status(self, where="device"):
        s = int(self.status.item())
        if s != LVQ_OK:
            self.status.zero_()
            raise LvqError(s, where)
