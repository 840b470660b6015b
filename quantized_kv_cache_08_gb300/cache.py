"""A torch-facing holder for one kvq layer cache.

PyTorch only provides the device memory (uint8 / int32 tensors) and the
stream; every operation is one call through the C ABI (see _binding).
"""

from __future__ import annotations

import ctypes

import torch

from . import _binding as B


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dtype_code(t):
    if t.dtype == torch.float32:
        return B.KVQ_F32
    if t.dtype == torch.bfloat16:
        return B.KVQ_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: use float32 or bfloat16")


def _check_dev(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class KVCache:
    """n_seq sequences of one attention layer: q8_0 K plane and q5_1 V plane
    (fmt "q8_0/q5_1") or FP8 E4M3 K and V planes (fmt "e4m3"), device counters
    and the decode workspace, all caller-owned torch memory."""

    FORMATS = {"q8_0/q5_1": (B.KVQ_Q8_0, B.KVQ_Q5_1, 34, 24), "e4m3": (B.KVQ_FP8_E4M3, B.KVQ_FP8_E4M3, 32, 32)}

    def __init__(self, n_seq, n_kv_heads, head_dim, max_q_heads, max_t=1, max_rows=0,
                 window=0, ring=False, device=None, stream=None, fmt="q8_0/q5_1"):
        if fmt not in self.FORMATS:
            raise ValueError(f"fmt must be one of {sorted(self.FORMATS)}")
        k_fmt, v_fmt, _, _ = self.FORMATS[fmt]
        self.fmt = fmt
        self.cfg = B.make_config(n_seq, n_kv_heads, head_dim, max_q_heads, max_t, max_rows,
                                 window, ring, k_fmt, v_fmt)
        sz = B.kvq_required_bytes(self.cfg)
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.k_plane = torch.empty(sz.k_plane, dtype=torch.uint8, device=dev)
        self.v_plane = torch.empty(sz.v_plane, dtype=torch.uint8, device=dev)
        self.counters = torch.empty(sz.counters // 4, dtype=torch.int32, device=dev)
        self.workspace = torch.empty(max(sz.workspace, 16), dtype=torch.uint8, device=dev)
        self.n_seq, self.n_kv_heads, self.head_dim = n_seq, n_kv_heads, head_dim
        # the geometry as the library lays it out
        self.k_tok, self.v_tok, self.rows = sz.k_row_bytes, sz.v_row_bytes, sz.rows
        self.window, self.ring = window, bool(ring)
        self.handle = B.kvq_alloc(self.cfg, self.k_plane.data_ptr(), self.v_plane.data_ptr(),
                                  self.counters.data_ptr(), self.workspace.data_ptr(),
                                  _stream_handle(stream))

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None:
            B.kvq_free(h)
            self.handle = None

    # -- the calls of the path: append, decode, truncate (host or device counts)
    def append(self, k, v, seq_ids=None, stream=None):
        """k, v: [n, T, Hkv, D] float32/bfloat16 CUDA tensors."""
        _check_dev(k, "k")
        _check_dev(v, "v")
        if k.shape != v.shape or k.dtype != v.dtype or k.dim() != 4:
            raise ValueError("k and v must both be [n, T, Hkv, D] of one dtype")
        n = self.n_seq if seq_ids is None else len(seq_ids)
        if k.shape[0] != n or k.shape[2] != self.n_kv_heads or k.shape[3] != self.head_dim:
            raise ValueError(f"k shape {tuple(k.shape)} does not match the cache")
        B.kvq_append(self.handle, k.data_ptr(), v.data_ptr(), _dtype_code(k), k.shape[1],
                     seq_ids, _stream_handle(stream))

    def decode(self, q, sinks=None, scale=0.0, out=None, stream=None):
        """q: [n_seq, T, Hq, D] float32/bfloat16; returns float32 [n_seq, T, Hq, D]."""
        _check_dev(q, "q")
        if q.dim() != 4 or q.shape[0] != self.n_seq or q.shape[3] != self.head_dim:
            raise ValueError(f"q shape {tuple(q.shape)} does not match the cache")
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        _check_dev(out, "out")
        if out.dtype != torch.float32 or out.shape != q.shape:
            raise ValueError("out must be float32 with q's shape")
        sp = None
        if sinks is not None:
            _check_dev(sinks, "sinks")
            if sinks.dtype != torch.float32 or sinks.numel() != q.shape[2]:
                raise ValueError("sinks must be float32 [Hq]")
            sp = sinks.data_ptr()
        B.kvq_decode(self.handle, q.data_ptr(), _dtype_code(q), q.shape[1], q.shape[2], sp,
                     scale, out.data_ptr(), _stream_handle(stream))
        return out

    def truncate(self, new_len, stream=None):
        B.kvq_truncate(self.handle, list(new_len), _stream_handle(stream))

    def truncate_device(self, accept, T, stream=None):
        """Keep the first accept[b] of each sequence's last T rows; accept is a
        CUDA int32 tensor [n_seq] read when the kernel runs (no host wait)."""
        _check_dev(accept, "accept")
        if accept.dtype != torch.int32 or accept.numel() != self.n_seq:
            raise ValueError("accept must be int32 [n_seq]")
        B.kvq_truncate_device(self.handle, accept.data_ptr(), T, _stream_handle(stream))

    def sync_len(self, stream=None):
        """Wait for the stream and read the device lengths into the host mirror."""
        B.kvq_sync_len(self.handle, _stream_handle(stream))

    # -- host-side helpers
    def lens(self):
        return B.kvq_get_len(self.handle, self.n_seq)[0]

    def bases(self):
        return B.kvq_get_len(self.handle, self.n_seq)[1]

    def note_replayed(self, steps, T):
        B.kvq_note_replayed(self.handle, steps, T)

    def ring_headroom(self, T):
        return B.kvq_ring_headroom(self.handle, T)

    def physical_rows(self, seq, start, end):
        return B.kvq_physical_rows(self.handle, seq, start, end)

    def device_error(self, stream=None):
        return B.kvq_read_device_error(self.handle, _stream_handle(stream))

    def set_split_rows(self, rows):
        B.kvq_set_split_rows(self.handle, rows)

    def set_row_slices(self, slices):
        """Row slices per tile on the stream-K kernel: 0 automatic, 1 or 2."""
        B.kvq_set_row_slices(self.handle, slices)

    def set_softcap(self, softcap):
        """softcap > 0 caps scaled scores to softcap * tanh(s / softcap); 0 is off."""
        B.kvq_set_softcap(self.handle, softcap)

    def set_decode_path(self, path, query_bits=0):
        """path: 0 auto, 1 generic split kernel, 2 stream-K kernel."""
        B.kvq_set_decode_path(self.handle, path, query_bits)

    def k_rows(self, seq, phys_lo, phys_hi):
        """Raw K bytes of physical rows [phys_lo, phys_hi) of a sequence (a view)."""
        n = self.n_seq * self.rows * self.k_tok
        v = self.k_plane[:n].view(self.n_seq, self.rows, self.k_tok)
        return v[seq, phys_lo:phys_hi]

    def v_rows(self, seq, phys_lo, phys_hi):
        n = self.n_seq * self.rows * self.v_tok
        v = self.v_plane[:n].view(self.n_seq, self.rows, self.v_tok)
        return v[seq, phys_lo:phys_hi]


def _token_rows(t, heads, dim, name):
    """Address and row stride (in elements) of [..., heads, dim] rows that lie
    evenly apart in memory (dense, or slices of a wider projection)."""
    if t.shape[-2] != heads or t.shape[-1] != dim:
        raise ValueError(f"{name} shape {tuple(t.shape)} does not match the cache")
    st = t.stride()
    if t.numel() and (st[-1] != 1 or (heads > 1 and st[-2] != dim)):
        raise ValueError(f"{name} needs each row's heads side by side")
    if t.dim() == 3:
        stride = st[0] if t.shape[0] > 1 else heads * dim
    else:
        n, T = t.shape[0], t.shape[1]
        stride = st[1] if T > 1 else st[0] if n > 1 else heads * dim
        if n > 1 and T > 1 and st[0] != T * st[1]:
            raise ValueError(f"{name} rows must lie evenly apart")
    return t.data_ptr(), stride


_I32 = torch.int32
_DTYPE = {torch.float32: B.KVQ_F32, torch.bfloat16: B.KVQ_BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda index: torch.cuda.current_stream(index).cuda_stream
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


class PagedKVCache:
    """One attention layer's cache in pages: a pool of `n_pages` pages of
    `page_rows` rows, in the formats of KVCache.  The caller keeps, as int32
    CUDA tensors, a table of page numbers per sequence ([n, max_pages]) and the
    lengths ([n], counting the rows that a call appends or whose queries it
    takes), and passes both to every call; all calls read them on the device.

    rope_dim > 0: `append` rotates the first rope_dim elements of each head of
    its keys (and queries) by their positions.  rope_freq gives rope_dim / 2
    radians per position in place of rope_base^(-2i / rope_dim).  bounds: keep
    key bounds per page, which `select` scores.  pool and bounds_buf take over
    existing uint8 CUDA tensors of `sizes.pool` and `sizes.bounds` bytes.

    rope_axes: the axis of each of the rope_dim / 2 rotated pairs, for appends
    whose rows are given positions on several axes.  scores: keep an attention score per row and KV head in
    `scores` (float32 [n_pages, Hkv, page_rows], zeros at first; scores_buf takes over an existing
    tensor), which `decode_scored` adds to, `select_rows` goes by and `compact`
    moves; appended rows start at 0.  score_scratch: room beside it for the scores of a call of up to
    8 queries a KV head (or as many as max_q_heads, max_t and the keys' bytes allow; 4 bytes a row, KV head and query: 14 % of a
    pool of head_dim 128 for 8), which spares such calls of decode_scored a second pass over the keys."""

    def __init__(self, n_pages, page_rows, n_kv_heads, head_dim, max_q_heads, max_seqs, max_pages, max_t=1,
                 fmt="q8_0/q5_1", rope_dim=0, rope_base=10000.0, rope_interleaved=False, rope_freq=None, bounds=False,
                 pool=None, bounds_buf=None, device=None, stream=None, rope_axes=None, scores=False, scores_buf=None,
                 score_scratch=True):
        self.handle = None
        self._lib = B.lib()
        if fmt not in KVCache.FORMATS:
            raise ValueError(f"fmt must be one of {sorted(KVCache.FORMATS)}")
        k_fmt, v_fmt, _, _ = KVCache.FORMATS[fmt]
        self.fmt = fmt
        if rope_freq is not None and len(rope_freq) != rope_dim // 2:
            raise ValueError("rope_freq needs rope_dim / 2 values")
        if rope_axes is not None and len(rope_axes) != rope_dim // 2:
            raise ValueError("rope_axes needs rope_dim / 2 values")
        self.cfg = B.make_paged_config(n_pages, page_rows, n_kv_heads, head_dim, max_q_heads, max_seqs, max_pages,
                                       max_t, k_fmt, v_fmt, bounds, rope_dim, rope_interleaved, rope_base)
        self.sizes = sz = B.kvq_paged_required_bytes(self.cfg)
        if device is None:
            device = pool.device if pool is not None else "cuda"
        dev = torch.device(device)
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device, self.index = dev, dev.index
        self.n_kv_heads, self.head_dim, self.max_pages = n_kv_heads, head_dim, max_pages
        self.pool = self._buffer(pool, sz.pool, "pool")
        self.bounds = self._buffer(bounds_buf, sz.bounds, "bounds_buf") if bounds else None
        self.n_axes, self.scores, self.scratch = 1, None, None
        if scores or scores_buf is not None:
            shape = (n_pages, n_kv_heads, page_rows)
            if scores_buf is None:
                scores_buf = torch.zeros(shape, dtype=torch.float32, device=dev)
            if scores_buf.dtype != torch.float32 or tuple(scores_buf.shape) != shape or scores_buf.device != dev \
                    or not scores_buf.is_contiguous():
                raise ValueError(f"scores_buf must be a contiguous float32 {list(shape)} tensor on {dev}")
            self.scores = scores_buf
            # (a call keeps at most 8 queries' scores, and only where they are fewer bytes than a row's keys)
            key = head_dim // 32 * (32 if fmt == "e4m3" else 34)
            queries = min(8, max_q_heads // n_kv_heads * max_t, (key - 1) // 8)
            if score_scratch:
                self.scratch = torch.empty(n_pages * n_kv_heads * page_rows * queries, dtype=torch.float32, device=dev)
        self.workspace = torch.empty(sz.workspace, dtype=torch.uint8, device=dev)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream(dev))   # the workspace's memory may still be in use there
        with torch.cuda.device(dev):
            self.handle = B.kvq_paged_alloc(self.cfg, self.pool.data_ptr(),
                                            self.bounds.data_ptr() if bounds else None, self.workspace.data_ptr(),
                                            rope_freq, _stream_handle(stream))
        if rope_axes is not None:
            self.n_axes = max(rope_axes, default=0) + 1
            B.kvq_paged_set_axes(self.handle, rope_axes, self.n_axes)
        if self.scores is not None:
            B.kvq_paged_set_scores(self.handle, self.scores.data_ptr())
            if self.scratch is not None:
                B.kvq_paged_set_score_scratch(self.handle, self.scratch.data_ptr(), queries)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None:
            B.kvq_paged_free(h)
            self.handle = None

    def _buffer(self, t, size, name):
        if t is None:
            return torch.empty(size, dtype=torch.uint8, device=self.device)
        if t.dtype != torch.uint8 or t.numel() != size or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 tensor of {size} bytes on {self.device}")
        return t

    # The checks below run before every call of a decode step, so they ask each
    # tensor for as little as they can.
    def _bad_ints(self, t, shape, name):
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor on {self.device}")

    def _ints(self, t, shape, name):
        if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != self.index or not t.is_contiguous():
            self._bad_ints(t, shape, name)
        return t.data_ptr()

    def _batch(self, tables, lens):
        n = lens.shape[0] if lens.dim() == 1 else -1
        if tables.dtype is not _I32 or lens.dtype is not _I32 or tables.shape != (n, self.max_pages) \
                or tables.get_device() != self.index or lens.get_device() != self.index \
                or not tables.is_contiguous() or not lens.is_contiguous():
            self._ints(tables, (n, self.max_pages), "tables")
            self._bad_ints(lens, (n,), "lens")
        return n, tables.data_ptr(), lens.data_ptr()

    def _dense(self, t, name):
        if t.get_device() != self.index or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor on {self.device}")
        return t.data_ptr()

    def _rows(self, t, n, starts, name):
        """T, address of starts, rows of a [n, T, H, D] or packed [rows, H, D] tensor."""
        if starts is None:
            if t.dim() != 4 or t.shape[0] != n:
                raise ValueError(f"{name} must be [n, T, heads, dim] without starts")
            return t.shape[1], None, n * t.shape[1]
        if t.dim() != 3:
            raise ValueError(f"{name} must be [rows, heads, dim] with starts")
        return 0, self._ints(starts, (n + 1,), "starts"), t.shape[0]

    def _stream(self, stream):
        return _raw_stream(self.index) if stream is None else stream.cuda_stream

    def _call(self, fn, *args):
        """A call of the library with the cache's device current."""
        if _current_device() == self.index:
            st = fn(self.handle, *args)
        else:
            with torch.cuda.device(self.index):
                st = fn(self.handle, *args)
        if st:
            B._check(st)

    def _new(self, shape, dtype, stream):
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        # memory of the stream that writes it, kept for the one that asked for it
        with torch.cuda.stream(stream):
            out = torch.empty(shape, dtype=dtype, device=self.device)
        out.record_stream(torch.cuda.current_stream(self.device))
        return out

    def append(self, k, v, tables, lens, starts=None, q=None, q_out=None, stream=None, positions=None):
        """k, v: float32/bfloat16 [n, T, Hkv, D], or packed [rows, Hkv, D] with
        starts (int32 [n + 1]).  q (same form, up to max_q_heads heads) is rotated
        into q_out (made if None; q itself when dense), which is returned.
        positions (int32, k's rows, [n, T, axes] or [rows, axes]; with one axis
        the last dimension may be left out) take the place of each row's index."""
        n, tp, lp = self._batch(tables, lens)
        shape, dtype, hkv, dim, index = k.shape, k.dtype, self.n_kv_heads, self.head_dim, self.index
        code = _DTYPE.get(dtype)
        if code is None or v.dtype is not dtype or v.shape != shape or shape[-1] != dim or shape[-2] != hkv:
            raise ValueError(f"k {dtype} {tuple(shape)} and v {v.dtype} {tuple(v.shape)} must be float32 or bfloat16 "
                             "rows of the cache's heads, alike")
        if k.get_device() != index or v.get_device() != index:
            raise ValueError(f"k and v must be on {self.device}")
        T, sp, rows = self._rows(k, n, starts, "k")
        kp, ks = (k.data_ptr(), hkv * dim) if k.is_contiguous() else _token_rows(k, hkv, dim, "k")
        vp, vs = (v.data_ptr(), hkv * dim) if v.is_contiguous() else _token_rows(v, hkv, dim, "v")
        qp, qs, op, hq = None, 0, None, 0
        if q is not None:
            qshape = q.shape
            hq = qshape[-2]
            if q.dtype is not dtype or qshape[-1] != dim or qshape[:-2] != shape[:-2] or q.get_device() != index:
                raise ValueError("q must have k's rows, head_dim, dtype and device")
            qp, qs = (q.data_ptr(), hq * dim) if q.is_contiguous() else _token_rows(q, hq, dim, "q")
            if q_out is None:
                q_out = self._new(qshape, dtype, stream)
            elif q_out.dtype is not dtype or q_out.shape != qshape:
                raise ValueError("q_out must have q's shape and dtype")
            op = self._dense(q_out, "q_out")
        elif q_out is not None:
            raise ValueError("q_out without q")
        raw = _raw_stream(index) if stream is None else stream.cuda_stream
        if positions is None:
            self._call(self._lib.kvq_paged_append, kp, ks, vp, vs, qp, qs, op, hq, code, tp, lp, n, T, sp, rows, raw)
            return q_out
        want = (*shape[:-2], self.n_axes)
        if self.n_axes == 1 and positions.shape == shape[:-2]:
            want = shape[:-2]
        self._call(self._lib.kvq_paged_append_at, kp, ks, vp, vs, qp, qs, op, hq, code, tp, lp, n, T, sp, rows,
                   self._ints(positions, want, "positions"), raw)
        return q_out

    def read(self, tables, lens, k_out, v_out, starts=None, stream=None):
        """Each entry's last rows as values into k_out, v_out: float32/bfloat16
        [n, T, Hkv, D], or packed [rows, Hkv, D] with starts."""
        n, tp, lp = self._batch(tables, lens)
        shape, code, index = k_out.shape, _DTYPE.get(k_out.dtype), self.index
        if code is None or v_out.dtype is not k_out.dtype or v_out.shape != shape or shape[-1] != self.head_dim \
                or shape[-2] != self.n_kv_heads:
            raise ValueError("k_out and v_out must be float32 or bfloat16 rows of the cache's heads, alike")
        if k_out.get_device() != index or v_out.get_device() != index or not k_out.is_contiguous() \
                or not v_out.is_contiguous():
            raise ValueError(f"k_out and v_out must be contiguous tensors on {self.device}")
        T, sp, rows = self._rows(k_out, n, starts, "k_out")
        self._call(self._lib.kvq_paged_read, k_out.data_ptr(), v_out.data_ptr(), code, tp, lp, n, T, sp, rows,
                   _raw_stream(index) if stream is None else stream.cuda_stream)

    def update_bounds(self, tables, lens, T, stream=None):
        """Renew the key bounds of the pages that hold each sequence's last T
        rows (appends do this; for pages filled in another way)."""
        n, tp, lp = self._batch(tables, lens)
        self._call(self._lib.kvq_paged_bounds, tp, lp, n, T, None, n * T, self._stream(stream))

    def _query(self, q, tables, lens, sinks, scale, window, softcap, out, stream):
        n, tp, lp = self._batch(tables, lens)
        shape, code = q.shape, _DTYPE.get(q.dtype)
        if code is None or len(shape) != 4 or shape[0] != n or shape[3] != self.head_dim:
            raise ValueError(f"q {q.dtype} {tuple(shape)} does not match the cache and lens")
        if not 0 <= window < 1 << 31:
            raise ValueError("window must be >= 0 and fit an int32")
        qp = self._dense(q, "q")
        if out is None:
            out = torch.empty_like(q) if stream is None else self._new(shape, q.dtype, stream)
            op = out.data_ptr()
        else:
            if out.dtype is not q.dtype or out.shape != shape:
                raise ValueError("out must have q's shape and dtype")
            op = self._dense(out, "out")
        sk = None
        if sinks is not None:
            if sinks.dtype is not torch.float32 or sinks.numel() != shape[2]:
                raise ValueError("sinks must be float32 [Hq]")
            sk = self._dense(sinks, "sinks")
        return out, ctypes.byref(B.kvq_paged_query(qp, op, code, n, shape[1], shape[2], tp, lp, sk, scale, softcap, window))

    def decode(self, q, tables, lens, sinks=None, scale=0.0, window=0, softcap=0.0, out=None, stream=None):
        """q: float32/bfloat16 [n, T, Hq, D], the last T rows of each sequence;
        returns the attention outputs in q's shape and dtype."""
        out, a = self._query(q, tables, lens, sinks, scale, window, softcap, out, stream)
        self._call(self._lib.kvq_paged_decode, a, self._stream(stream))
        return out

    def decode_shared(self, q, tables, lens, group_start, prefix_lens, sinks=None, scale=0.0, window=0, softcap=0.0,
                      out=None, stream=None):
        """decode for a batch whose sequences group_start[i] .. group_start[i+1]
        share their first prefix_lens[i] rows, read once a group (int32 CUDA
        tensors [groups + 1] and [groups])."""
        out, a = self._query(q, tables, lens, sinks, scale, window, softcap, out, stream)
        g = prefix_lens.numel()
        self._call(self._lib.kvq_paged_decode_shared, a, self._ints(group_start, (g + 1,), "group_start"),
                   self._ints(prefix_lens, (g,), "prefix_lens"), g, self._stream(stream))
        return out

    def select(self, q, tables, lens, keep, n_first=1, n_last=1, pages=None, stream=None):
        """Indexes into each table of the `keep` pages that each query row and
        KV head reads: int32 [n, T, Hkv, keep], ascending, -1 behind the last."""
        if pages is None:
            pages = self._new((q.shape[0], q.shape[1], self.n_kv_heads, keep), torch.int32, stream)
        out, a = self._query(q, tables, lens, None, 0.0, 0, 0.0, q, stream)
        self._call(self._lib.kvq_paged_select, a, self._ints(pages, (q.shape[0], q.shape[1], self.n_kv_heads, keep), "pages"),
                   keep, n_first, n_last, self._stream(stream))
        return pages

    def decode_sparse(self, q, tables, lens, pages, sinks=None, scale=0.0, softcap=0.0, out=None, stream=None):
        """decode over the listed pages only (int32 [n, T, Hkv, keep])."""
        out, a = self._query(q, tables, lens, sinks, scale, 0, softcap, out, stream)
        keep = pages.shape[-1]
        self._call(self._lib.kvq_paged_decode_sparse, a,
                   self._ints(pages, (q.shape[0], q.shape[1], self.n_kv_heads, keep), "pages"), keep, self._stream(stream))
        return out

    def decode_scored(self, q, tables, lens, decay=1.0, sinks=None, scale=0.0, window=0, softcap=0.0, out=None,
                      stream=None):
        """decode, with the weights of each row added to its score: decay * score
        + the sum over the T query rows and the queries of the KV head (those of
        drafts that fall later too: nothing takes them off again)."""
        if not 0.0 <= decay <= 1.0:
            raise ValueError("decay must be in [0, 1]")
        out, a = self._query(q, tables, lens, sinks, scale, window, softcap, out, stream)
        self._call(self._lib.kvq_paged_decode_scored, a, decay, self._stream(stream))
        return out

    def select_rows(self, tables, lens, keep, n_first=0, n_last=0, rows=None, stream=None):
        """The rows that stay of each sequence and KV head: int32 [n, Hkv, keep],
        the first n_first, the last n_last and the best scored of the others,
        ascending, -1 behind the last."""
        n, tp, lp = self._batch(tables, lens)
        if rows is None:
            rows = torch.empty((n, self.n_kv_heads, keep), dtype=_I32, device=self.device) if stream is None else \
                self._new((n, self.n_kv_heads, keep), torch.int32, stream)
            rp = rows.data_ptr()
        else:
            rp = self._ints(rows, (n, self.n_kv_heads, keep), "rows")
        self._call(self._lib.kvq_paged_select_rows, tp, lp, n, keep, n_first, n_last, rp,
                   _raw_stream(self.index) if stream is None else stream.cuda_stream)
        return rows

    def compact(self, tables, lens, rows, lens_out=None, tables_out=None, stream=None):
        """Move the listed rows (int32 [n, Hkv, keep], ascending) to the front of
        their sequence's pages, or into those of tables_out; returns the new
        lengths (lens_out, made if None; may be lens)."""
        n, tp, lp = self._batch(tables, lens)
        keep = rows.shape[-1]
        rp = self._ints(rows, (n, self.n_kv_heads, keep), "rows")
        to = None if tables_out is None else self._ints(tables_out, (n, self.max_pages), "tables_out")
        if lens_out is None:
            lens_out = torch.empty_like(lens) if stream is None else self._new((n,), torch.int32, stream)
            op = lens_out.data_ptr()
        else:
            op = self._ints(lens_out, (n,), "lens_out")
        self._call(self._lib.kvq_paged_compact, tp, lp, n, rp, keep, to, op,
                   _raw_stream(self.index) if stream is None else stream.cuda_stream)
        return lens_out

    def device_error(self, stream=None):
        """0, or 1: a page number or length out of range, 2: a wait ran out (read and cleared)."""
        if _current_device() == self.index:
            return B.kvq_paged_read_error(self.handle, self._stream(stream))
        with torch.cuda.device(self.index):
            return B.kvq_paged_read_error(self.handle, self._stream(stream))


def verify(target, draft, tokens, uniform, lens=None, accept=None, next_tokens=None, stream=None):
    """Which drafted tokens stand, and each sequence's next token.

    target: float32/bfloat16 [n, T, V] probabilities behind each row of a T-row
    step; draft: [n, T - 1, V] that tokens (int32 [n, T - 1]; outside [0, V): no
    draft) were drawn from, or None (looked up: probability 1); uniform: float32
    [n, T] in [0, 1).  Rows may lie apart (strides), elements side by side.
    Returns (accept, next_tokens), int32 [n] each, made if None: accept counts the rows of the step
    that stay, as KVCache.truncate_device takes them; lens (int32 [n], the
    lengths of a paged cache) is lowered by the others."""
    dtype = target.dtype
    code = _DTYPE.get(dtype)
    if code is None or target.dim() != 3 or not target.is_cuda:
        raise ValueError("target must be a float32 or bfloat16 [n, T, V] CUDA tensor")
    n, T, V = target.shape
    index = target.get_device()
    ts, tr, te = target.stride()
    dp, ds, dr = None, 0, 0
    if draft is not None:
        if draft.dtype is not dtype or draft.shape != (n, T - 1, V) or draft.get_device() != index:
            raise ValueError(f"draft must be {dtype} {[n, T - 1, V]} on target's device")
        ds, dr, de = draft.stride()
        if de != 1 and V > 1 and T > 1:
            raise ValueError("draft needs each row's elements side by side")
        dp = draft.data_ptr()
    if te != 1 and V > 1:
        raise ValueError("target needs each row's elements side by side")
    if tokens.dtype is not _I32 or tokens.shape != (n, T - 1) or tokens.get_device() != index or not tokens.is_contiguous():
        raise ValueError(f"tokens must be a contiguous int32 {[n, T - 1]} tensor on target's device")
    if uniform.dtype is not torch.float32 or uniform.shape != (n, T) or uniform.get_device() != index \
            or not uniform.is_contiguous():
        raise ValueError(f"uniform must be a contiguous float32 {[n, T]} tensor on target's device")

    def counts(t, name):
        if t.dtype is not _I32 or t.shape != (n,) or t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 {[n]} tensor on target's device")
        return t.data_ptr()

    def make():
        with torch.cuda.stream(stream):
            t = torch.empty(n, dtype=_I32, device=target.device)
        t.record_stream(torch.cuda.current_stream(target.device))
        return t

    ap = counts(accept, "accept") if accept is not None else None
    np_ = counts(next_tokens, "next_tokens") if next_tokens is not None else None
    lp = counts(lens, "lens") if lens is not None else None
    if accept is None:
        accept = torch.empty(n, dtype=_I32, device=target.device) if stream is None else make()
        ap = accept.data_ptr()
    if next_tokens is None:
        next_tokens = torch.empty_like(accept) if stream is None else make()
        np_ = next_tokens.data_ptr()
    a = ctypes.byref(B.kvq_verify_args(target.data_ptr(), dp, tokens.data_ptr(), uniform.data_ptr(), code, n, T, V, ts, tr, ds,
                                       dr, ap, np_, lp))
    raw = _raw_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:
        st = B.lib().kvq_verify(a, raw)
    else:
        with torch.cuda.device(index):
            st = B.lib().kvq_verify(a, raw)
    if st:
        B._check(st)
    return accept, next_tokens
