"""Thin Python binding of the C ABI in ``include/hs.h``.

Functions carry the C names and only marshal arguments: every step of the
resolve path runs in the CUDA kernels of ``libhs.so``.  Device buffers may be
passed as torch tensors (their ``data_ptr()`` is used) or as raw integer
addresses; streams as ``torch.cuda.Stream`` objects, raw handles, or ``None``
for torch's current stream.  A failing call raises :class:`HsError`.

:class:`Pool` wraps a pool handle with numpy views of the host records and
zero-copy torch views of the device metadata.
"""
from __future__ import annotations

import ctypes

import numpy as np

from . import _native

HS_OK = 0
HS_ERR_INVALID_ARG = -1
HS_ERR_CUDA = -2
HS_ERR_NOMEM = -3
HS_ERR_DEVICE_INPUT = -4
HS_ERR_TIMEOUT = -5
HS_ERR_UNSUPPORTED = -6

HS_HOST_ALLOC_AUTO = 0
HS_HOST_ALLOC_PINNED = 1
HS_HOST_ALLOC_VMM_NUMA = 2
HS_HOST_ALLOC_THP_REGISTERED = 3

HS_OVERLAP_AUTO = 0
HS_OVERLAP_ON = 1
HS_OVERLAP_OFF = 2

HS_STATUS_POS_RANGE = 0x1
HS_STATUS_POS_DUP = 0x2
HS_STATUS_REQ_RANGE = 0x4
HS_STATUS_REQ_BUSY = 0x8
HS_STATUS_PLAN = 0x10
HS_STATUS_META = 0x20


class HsError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {hs_strerror(code)} ({code})")


def _lib():
    return _native._lib or _native.load()


def _check(rc: int, what: str) -> None:
    if rc != HS_OK:
        raise HsError(rc, what)


def _ptr(x):
    if x is None or type(x) is int:
        return x
    try:
        return x.data_ptr()
    except AttributeError:
        pass
    if isinstance(x, int):
        return x
    if isinstance(x, np.ndarray):
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x).__name__}")


def _current_stream():
    """The handle of torch's current stream on the current device: by torch's
    raw query where it has one (a Stream object costs 2.8 us to make)."""
    global _current_stream
    import torch
    torch.cuda.current_stream()          # initialises CUDA
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    else:
        _current_stream = lambda: raw(device())  # noqa: E731
    return _current_stream()


def _stream(s):
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def hs_strerror(code: int) -> str:
    return _lib().hs_strerror(code).decode()


def hs_kernels_per_call() -> int:
    return int(_lib().hs_kernels_per_call())


def hs_plan_bytes(n_req: int, k: int) -> int:
    return int(_lib().hs_plan_bytes(n_req, k))


def hs_create_pool(n_requests, n_layers, n_positions, record_bytes, slots, max_k,
                   layer_anchor=None, host_limit_bytes=0, host_alloc=HS_HOST_ALLOC_AUTO,
                   launch_overlap=HS_OVERLAP_AUTO) -> int:
    anchors = None
    if layer_anchor is not None:
        anchors = (ctypes.c_int32 * len(layer_anchor))(*layer_anchor)
    d = _native.PoolDesc(n_requests, n_layers, n_positions, record_bytes, slots, max_k,
                         ctypes.cast(anchors, ctypes.c_void_p) if anchors is not None else None,
                         host_limit_bytes, host_alloc, launch_overlap)
    h = ctypes.c_void_p()
    _check(_lib().hs_create_pool(ctypes.byref(d), ctypes.byref(h)), "hs_create_pool")
    return h.value


def hs_destroy_pool(pool: int) -> None:
    _check(_lib().hs_destroy_pool(pool), "hs_destroy_pool")


def hs_host_records(pool: int, req: int, layer: int) -> int:
    p = ctypes.c_void_p()
    _check(_lib().hs_host_records(pool, req, layer, ctypes.byref(p)), "hs_host_records")
    return p.value


def hs_device_views(pool: int, layer: int) -> _native.Views:
    v = _native.Views()
    _check(_lib().hs_device_views(pool, layer, ctypes.byref(v)), "hs_device_views")
    return v


def hs_device_host_numa(device: int) -> int:
    """Host NUMA node closest to `device`, -1 when none is reported."""
    return int(_lib().hs_device_host_numa(device))


def hs_touch_records(pool: int, req: int = -1, layer: int = -1, stream=None) -> None:
    _check(_lib().hs_touch_records(pool, req, layer, _stream(stream)), "hs_touch_records")


def hs_warm_pool(pool: int) -> None:
    _check(_lib().hs_warm_pool(pool), "hs_warm_pool")


def hs_pool_info(pool: int) -> dict:
    i = _native.PoolInfo()
    _check(_lib().hs_pool_info(pool, ctypes.byref(i)), "hs_pool_info")
    return {f: int(getattr(i, f)) for f, _ in _native.PoolInfo._fields_}


def hs_resolve(pool, layer, n_req, req_ids, sel, k, out, plan=None, stream=None) -> None:
    _check(_lib().hs_resolve(pool, layer, n_req, _ptr(req_ids), _ptr(sel), k, _ptr(out),
                             _ptr(plan), _stream(stream)), "hs_resolve")


def hs_resolve_anchor(pool, layer, n_req, req_ids, sel, k, out, plan_out, stream=None) -> None:
    _check(_lib().hs_resolve_anchor(pool, layer, n_req, _ptr(req_ids), _ptr(sel), k, _ptr(out),
                                    _ptr(plan_out), _stream(stream)), "hs_resolve_anchor")


HS_MEASURE_NO_FETCH = 0x1
HS_STAMPS = ("ENTRY", "LOADED", "HASHED", "PROBED", "DECIDED", "CHECKED", "VERDICT", "COMMITTED",
             "F_ISSUE", "F_ISSUED", "F_WAITED", "F_LANDED", "F_STORED", "ATTEMPTS", "EXIT",
             "LEAD_FETCHED")
HS_STAMP = {name: i for i, name in enumerate(HS_STAMPS)}


def hs_measure_stamp_slots() -> int:
    return int(_lib().hs_measure_stamp_slots())


def hs_resolve_measure(pool, layer, n_req, req_ids, sel, k, out, flags=0, times=None,
                       stream=None) -> None:
    """Measurement variant of hs_resolve: HS_MEASURE_NO_FETCH skips the miss
    fetch; `times` (device u64 [n_req][hs_measure_stamp_slots()]) receives
    stage timestamps."""
    _check(_lib().hs_resolve_measure(pool, layer, n_req, _ptr(req_ids), _ptr(sel), k, _ptr(out),
                                     flags, _ptr(times), _stream(stream)), "hs_resolve_measure")


def hs_prefetch_plan(pool, anchor_layer, target_layer, n_req, req_ids, sel, k, plan,
                     stream=None) -> None:
    _check(_lib().hs_prefetch_plan(pool, anchor_layer, target_layer, n_req, _ptr(req_ids),
                                   _ptr(sel), k, _ptr(plan), _stream(stream)), "hs_prefetch_plan")


def hs_prefetch_copy(pool, target_layer, n_req, k, plan, stream=None) -> None:
    _check(_lib().hs_prefetch_copy(pool, target_layer, n_req, k, _ptr(plan), _stream(stream)),
           "hs_prefetch_copy")


def hs_stats(pool, layer: int = -1, check: bool = True) -> dict:
    """Counters of `layer` (-1: all).  With check=False a status error is
    returned in the dict instead of raised."""
    s = _native.Stats()
    rc = _lib().hs_stats(pool, layer, ctypes.byref(s))
    if rc not in (HS_OK, HS_ERR_DEVICE_INPUT) or (check and rc != HS_OK):
        raise HsError(rc, f"hs_stats (status 0x{s.status:x})")
    d = {f: int(getattr(s, f)) for f, _ in _native.Stats._fields_}
    d["rc"] = rc
    return d


def hs_reset(pool) -> None:
    _check(_lib().hs_reset(pool), "hs_reset")


def hs_link_probe(nbytes: int, reps: int = 10, record_bytes: int = 1152,
                  host_alloc: int = HS_HOST_ALLOC_AUTO):
    """(H2D memcpy GB/s, scattered-record GPU-load GB/s), best of `reps`,
    over a host buffer of `nbytes` allocated the `host_alloc` way."""
    a, b = ctypes.c_double(), ctypes.c_double()
    _check(_lib().hs_link_probe(nbytes, reps, record_bytes, host_alloc, ctypes.byref(a),
                                ctypes.byref(b)), "hs_link_probe")
    return a.value, b.value


def hs_sparse_attention(q, cache, cache_rows, idx, n_req, k, heads, scale, out,
                        stream=None) -> None:
    """Attention of q [n_req][heads][576] bf16 over the published rows idx
    [n_req][k] of a layer's cache; fp32 out [n_req][heads][512]."""
    _check(_lib().hs_sparse_attention(_ptr(q), _ptr(cache), cache_rows, _ptr(idx), n_req, k,
                                      heads, scale, _ptr(out), _stream(stream)),
           "hs_sparse_attention")


def hs_sparse_attention_heads(q, cache, cache_rows, idx, n_req, k, heads, scale, out,
                              stream=None) -> None:
    """Attention of q [n_req][heads][128] bf16 over the published rows idx
    [n_req][k] of a layer's cache of per-head token records (keys of every
    head, then values; heads * 512 bytes); fp32 out [n_req][heads][128]."""
    _check(_lib().hs_sparse_attention_heads(_ptr(q), _ptr(cache), cache_rows, _ptr(idx), n_req,
                                            k, heads, scale, _ptr(out), _stream(stream)),
           "hs_sparse_attention_heads")


HS_ATTN_STATUS_TIMEOUT = 0x1


def hs_attention_status() -> int:
    """HS_ATTN_STATUS_* bits set by attention calls since the last query
    (synchronises the device, clears the bits)."""
    v = ctypes.c_uint32()
    _check(_lib().hs_attention_status(ctypes.byref(v)), "hs_attention_status")
    return int(v.value)


def qk_desc(q_heads, heads, inv_freq, eps=1e-6, interleaved=False, q_stride=0, k_stride=0,
            v_stride=0) -> _native.QkDesc:
    """Descriptor of hs_qk_norm_rope: len(inv_freq) pairs are rotated
    (rot_dim = 2 * len(inv_freq)); strides in elements between tokens (0:
    dense)."""
    freq = [float(f) for f in inv_freq]
    if len(freq) > 64:
        raise ValueError("at most 64 rotated pairs in a head of 128")
    return _native.QkDesc(q_heads, heads, 2 * len(freq), int(interleaved), eps, q_stride,
                          k_stride, v_stride, (ctypes.c_double * 64)(*freq))


def hs_qk_norm_rope(desc, q, k, v, wq, wk, pos, n_tok, q_out, records, record_rows, rows=None,
                    stream=None) -> None:
    """Per-head RMS norm (weights wq, wk: bf16 [128] or None) and position
    rotation of n_tok tokens' queries and keys; q_out bf16
    [n_tok][q_heads][128], and each token's record (keys, then the values as
    they are) into row rows[i] (int64; None: row i) of `records`.  `desc` is
    a qk_desc."""
    _check(_lib().hs_qk_norm_rope(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(wq),
                                  _ptr(wk), _ptr(pos), n_tok, _ptr(q_out), _ptr(records),
                                  record_rows, _ptr(rows), _stream(stream)), "hs_qk_norm_rope")


def hs_prefix_attention_bytes(n_req: int, q_heads: int, heads: int, prefix_len: int,
                              k: int) -> int:
    """Workspace bytes of hs_prefix_attention (0: none needed)."""
    return int(_lib().hs_prefix_attention_bytes(n_req, q_heads, heads, prefix_len, k))


def hs_prefix_attention(q, prefix, prefix_len, cache, cache_rows, idx, n_req, k, q_heads, heads,
                        scale, out, work=None, work_bytes=0, stream=None) -> None:
    """Attention of q [n_req][q_heads][128] bf16 over prefix_len token records
    that all requests share and over each request's published rows idx
    [n_req][k] of `cache`; bf16 out [n_req][q_heads][128]."""
    _check(_lib().hs_prefix_attention(_ptr(q), _ptr(prefix), prefix_len, _ptr(cache), cache_rows,
                                      _ptr(idx), n_req, k, q_heads, heads, scale, _ptr(out),
                                      _ptr(work), work_bytes, _stream(stream)),
           "hs_prefix_attention")


def hs_attention_weights_bytes(n_req: int, q_heads: int, heads: int, k: int) -> int:
    """Workspace bytes of hs_sparse_attention_weights (0: none needed)."""
    return int(_lib().hs_attention_weights_bytes(n_req, q_heads, heads, k))


def hs_sparse_attention_weights(q, cache, cache_rows, idx, sel, n_req, k, q_heads, heads, scale,
                                out, weights, weight_rows, n_positions, work=None, work_bytes=0,
                                req_ids=None, stream=None) -> None:
    """Attention of q [n_req][q_heads][128] bf16 over the published rows idx
    [n_req][k]; bf16 out [n_req][q_heads][128].  Also adds to weights
    [weight_rows][n_positions] (fp32), at request req_ids[i] (None: i) and
    position sel[i][j], the attention weight of row j summed over the query
    heads."""
    _check(_lib().hs_sparse_attention_weights(_ptr(q), _ptr(cache), cache_rows, _ptr(idx),
                                              _ptr(sel), _ptr(req_ids), n_req, k, q_heads, heads,
                                              scale, _ptr(out), _ptr(weights), weight_rows,
                                              n_positions, _ptr(work), work_bytes,
                                              _stream(stream)),
           "hs_sparse_attention_weights")


def hs_select_heavy(weights, weight_rows, n_positions, lens, n_req, k, recent, sel, req_ids=None,
                    stream=None) -> None:
    """The k positions each request keeps, ascending, into sel [n_req][k]
    int32: the `recent` last of its lens[i] (None: n_positions) positions and
    those of the largest weights[req_ids[i]] among the others; -1 past the
    request's length."""
    _check(_lib().hs_select_heavy(_ptr(weights), weight_rows, n_positions, _ptr(req_ids),
                                  _ptr(lens), n_req, k, recent, _ptr(sel), _stream(stream)),
           "hs_select_heavy")


HS_LATENT_RECORD_BYTES = 1152
HS_PACKED_RECORD_BYTES = 416


def hs_rope_frequencies(rot_dim: int, base: float = 10000.0, factor: float = 1.0,
                        trained: int = 4096, fast: float = 32.0, slow: float = 1.0):
    """(inv_freq, magnitude) of a rotation of rot_dim dimensions for contexts
    `factor` times as long as the `trained` one: fast pairs as they are, slow
    ones slowed down, those between in parts.  The attention's scale is to be
    multiplied by magnitude ** 2."""
    freq, magnitude = (ctypes.c_double * 64)(), ctypes.c_double()
    _check(_lib().hs_rope_frequencies(rot_dim, base, factor, trained, fast, slow, freq,
                                      ctypes.byref(magnitude)), "hs_rope_frequencies")
    return list(freq[:rot_dim // 2]), magnitude.value


def latent_desc(q_heads, inv_freq, eps=1e-6, interleaved=False, magnitude=1.0, packed=False,
                shift=0, q_stride=0, q_head_stride=0, out_stride=0, out_head_stride=0,
                kv_stride=0) -> _native.LatentDesc:
    """Descriptor of hs_latent_norm_rope: 32 frequencies; strides in elements
    (0: dense)."""
    freq = [float(f) for f in inv_freq]
    if len(freq) != 32:
        raise ValueError("64 rotated dimensions have 32 pairs")
    return _native.LatentDesc(q_heads, int(interleaved), int(packed), shift, eps, magnitude,
                              q_stride, q_head_stride, out_stride, out_head_stride, kv_stride,
                              (ctypes.c_double * 32)(*freq))


def hs_latent_norm_rope(desc, q, kv, w, pos, n_tok, q_out, records, record_rows, rows=None,
                        stream=None) -> None:
    """RMS norm (weight w: bf16 [512] or None) of the 512 latent values of n_tok
    tokens' kv [n_tok][576] bf16 and the position rotation of the other 64 and
    of 64 dimensions of every query head, from q to q_out; each token's record
    (bf16, or packed) into row rows[i] (int64; None: row i) of `records`.
    `desc` is a latent_desc."""
    _check(_lib().hs_latent_norm_rope(ctypes.byref(desc), _ptr(q), _ptr(kv), _ptr(w), _ptr(pos),
                                      n_tok, _ptr(q_out), _ptr(records), record_rows, _ptr(rows),
                                      _stream(stream)), "hs_latent_norm_rope")


def hs_pack_records(records, n, shift, packed, packed_rows, rows=None, stream=None) -> None:
    """n bf16 latent records [n][576] to packed ones (416 bytes), record i into
    row rows[i] (int64; None: row i) of `packed`."""
    _check(_lib().hs_pack_records(_ptr(records), n, shift, _ptr(packed), packed_rows, _ptr(rows),
                                  _stream(stream)), "hs_pack_records")


def hs_unpack_records(packed, packed_rows, shift, records, n, rows=None, stream=None) -> None:
    """Rows rows[i] (int64; None: row i) of `packed` to n bf16 latent records
    [n][576]; zeros for a row outside the range."""
    _check(_lib().hs_unpack_records(_ptr(packed), packed_rows, shift, _ptr(records), n,
                                    _ptr(rows), _stream(stream)), "hs_unpack_records")


def hs_packed_attention_bytes(n_req: int, heads: int, k: int) -> int:
    """Workspace bytes of hs_packed_attention (0 so far: none needed)."""
    return int(_lib().hs_packed_attention_bytes(n_req, heads, k))


def hs_packed_attention(q, cache, cache_rows, idx, n_req, k, heads, scale, shift, out, work=None,
                        work_bytes=0, stream=None) -> None:
    """Attention of q [n_req][heads][576] bf16 over the published packed rows
    idx [n_req][k] of a layer's cache; bf16 out [n_req][heads][512]."""
    _check(_lib().hs_packed_attention(_ptr(q), _ptr(cache), cache_rows, _ptr(idx), n_req, k, heads,
                                      scale, shift, _ptr(out), _ptr(work), work_bytes,
                                      _stream(stream)), "hs_packed_attention")


def hs_latent_prefill_bytes(n_tok: int, n_keys: int, n_seq: int, heads: int) -> int:
    """Workspace bytes of hs_latent_prefill (0: none needed)."""
    return int(_lib().hs_latent_prefill_bytes(n_tok, n_keys, n_seq, heads))


def hs_latent_prefill(q, k, v, kr, q_starts, k_starts, n_seq, n_tok, n_keys, heads, scale, out,
                      work=None, work_bytes=0, kv_stride=0, kv_head_stride=0, kr_stride=0,
                      stream=None) -> None:
    """Causal attention of q [n_tok][heads][192] bf16 over keys k (128 a head)
    with kr (64, shared by the heads) and values v (128 a head); sequence s has
    the queries q_starts[s] .. q_starts[s + 1] and the keys k_starts[s] ..
    k_starts[s + 1], the queries being the last tokens; bf16 out
    [n_tok][heads][128].  Strides in elements (0: dense)."""
    _check(_lib().hs_latent_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(kr), kv_stride, kv_head_stride,
                                    kr_stride, _ptr(q_starts), _ptr(k_starts), n_seq, n_tok,
                                    n_keys, heads, scale, _ptr(out), _ptr(work), work_bytes,
                                    _stream(stream)), "hs_latent_prefill")


HS_NOALLOC_MAX_REQUESTS = 4096


def hs_resolve_noalloc(state: dict, n_req, req_ids, sel, k, out, status=None, stream=None) -> None:
    """Resolve one layer whose state the caller owns, allocating nothing.

    ``state`` maps the hs_layer_state fields to values: sizes as ints,
    arrays as torch tensors or device addresses.  See include/hs.h for the
    scratch array it shares between calls."""
    st = _native.LayerState(
        state["n_requests"], state["n_positions"], state["record_bytes"], state["slots"],
        _ptr(state["host_records"]), _ptr(state["cache"]), _ptr(state["page_table"]),
        _ptr(state["slot_pos"]), _ptr(state["stamps"]), _ptr(state["lru"]),
        _ptr(state["resolves"]))
    _check(_lib().hs_resolve_noalloc(ctypes.byref(st), n_req, _ptr(req_ids), _ptr(sel), k,
                                     _ptr(out), _ptr(status), _stream(stream)),
           "hs_resolve_noalloc")


class _CudaArray:
    def __init__(self, ptr, shape, typestr):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (ptr, False), "version": 3, "strides": None}


class Pool:
    """A pool handle plus host and device views."""

    def __init__(self, n_requests, n_layers, n_positions, record_bytes, slots, max_k,
                 layer_anchor=None, host_limit_bytes=0, host_alloc=HS_HOST_ALLOC_AUTO,
                 launch_overlap=HS_OVERLAP_AUTO):
        self.R, self.NL, self.L = n_requests, n_layers, n_positions
        self.W, self.B, self.max_k = record_bytes, slots, max_k
        self.handle = hs_create_pool(n_requests, n_layers, n_positions, record_bytes, slots,
                                     max_k, layer_anchor, host_limit_bytes, host_alloc,
                                     launch_overlap)

    @classmethod
    def for_workload(cls, w, host_limit_bytes=0, host_alloc=HS_HOST_ALLOC_AUTO,
                     launch_overlap=HS_OVERLAP_AUTO):
        return cls(w.n_requests, w.n_layers, w.n_positions, w.record_bytes, w.slots, w.k,
                   list(w.anchors), host_limit_bytes, host_alloc, launch_overlap)

    def info(self) -> dict:
        return hs_pool_info(self.handle)

    def touch(self, req=-1, layer=-1, stream=None):
        hs_touch_records(self.handle, req, layer, stream)

    def warm(self):
        """Touch every record, resolve synthetic steps, reset (before first use)."""
        hs_warm_pool(self.handle)

    def close(self):
        if self.handle:
            hs_destroy_pool(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def host_records(self, req, layer) -> np.ndarray:
        """numpy uint8 view [L][W] of the pinned host records of (req, layer)."""
        addr = hs_host_records(self.handle, req, layer)
        buf = (ctypes.c_uint8 * (self.L * self.W)).from_address(addr)
        return np.frombuffer(buf, np.uint8).reshape(self.L, self.W)

    def views(self, layer):
        """torch tensors (zero-copy) over the device arrays of `layer`."""
        import torch
        v = hs_device_views(self.handle, layer)
        R, B, L, W = self.R, self.B, self.L, self.W

        def t(ptr, shape, ts):
            return torch.as_tensor(_CudaArray(ptr, shape, ts), device="cuda")
        return {"cache": t(v.cache, (R * B, W), "|u1"),
                "page_table": t(v.page_table, (R, L), "<i4"),
                "slot_pos": t(v.slot_pos, (R, B), "<i4"),
                "stamps": t(v.stamps, (R, B), "<u4"),
                "lru": t(v.lru, (R, B), "<u2"),
                "resolves": t(v.resolves, (R,), "<u4")}

    def resolve(self, layer, sel, out, req_ids=None, plan=None, stream=None, n_req=None):
        n = sel.shape[0] if n_req is None else n_req
        hs_resolve(self.handle, layer, n, req_ids, sel, sel.shape[-1], out, plan, stream)

    def resolve_anchor(self, layer, sel, out, plan_out, req_ids=None, stream=None):
        hs_resolve_anchor(self.handle, layer, sel.shape[0], req_ids, sel, sel.shape[-1], out,
                          plan_out, stream)

    def resolve_measure(self, layer, sel, out, flags=0, times=None, req_ids=None, stream=None):
        hs_resolve_measure(self.handle, layer, sel.shape[0], req_ids, sel, sel.shape[-1], out,
                           flags, times, stream)

    def prefetch_plan(self, anchor_layer, target_layer, sel, plan, req_ids=None, stream=None):
        hs_prefetch_plan(self.handle, anchor_layer, target_layer, sel.shape[0], req_ids, sel,
                         sel.shape[-1], plan, stream)

    def prefetch_copy(self, target_layer, n_req, k, plan, stream=None):
        hs_prefetch_copy(self.handle, target_layer, n_req, k, plan, stream)

    def stats(self, layer=-1, check=True):
        return hs_stats(self.handle, layer, check)

    def reset(self):
        hs_reset(self.handle)
