"""Torch-level plans of the decode step: ``PagedAttention`` (attention of one new token, or of a
chunk of them, over a paged key-value cache, and eviction from that cache) and ``Sampler`` (the next
token from logits and given random numbers).

Both only marshal arguments to the C ABI (``include/ctr.h``: ``ctr_attn_*``, ``ctr_sampler_*``)
after checking them.  A call runs on ``stream`` (default: the current stream of the plan's
device, which has to be the current device).  When ``stream`` is another stream than the current
one, the caller orders the two, as for ``Plan``; the plan's own tensors and those that the call
allocates are then kept for that stream.
"""
from __future__ import annotations

import torch

import transposed_convolution_gb300 as _ctr


def _device_of(device):
    d = torch.device(device if device is not None else "cuda")
    if d.type != "cuda":
        raise ValueError("the plan needs a CUDA device, got %s" % d)
    return torch.device("cuda", torch.cuda.current_device() if d.index is None else d.index)


def _numel(shape):
    n = 1
    for v in shape[1:]:
        n *= v
    return n


class _DecodePlan:
    """A plan handle on one device, and the checks both plans make of their arguments."""

    handle = None
    _destroy = None
    _kept = ()              # tensors of the plan that its kernels use

    def _stream(self, stream, *made):
        """The raw stream of a call; tensors that the call made are kept for it."""
        current = torch._C._cuda_getCurrentRawStream(self._index)
        if stream is None or stream.cuda_stream == current:
            return current
        for t in made + self._kept:
            t.record_stream(stream)
        return stream.cuda_stream

    def _at(self, t, name, shape, dtype):
        """The address of a contiguous tensor, after its shape, type, device and layout have been
        checked: one expression, because small calls take as long as their checks."""
        if (t.shape != shape or t.dtype is not dtype or t.get_device() != self._index
                or not t.is_contiguous()):
            self._refuse(t, name, shape, dtype)
            raise ValueError("%s must be contiguous" % name)
        return t.data_ptr()

    def _heads_at(self, t, name, T, heads, D, dtype):
        """As _rows_at for rows of heads, [T, heads, D]: the address and row stride of what a fused
        projection leaves, in few steps."""
        if t.dim() == 3 and t.dtype is dtype and t.get_device() == self._index:
            shape, stride = t.shape, t.stride()
            if (shape[0] == T and shape[1] == heads and shape[2] == D and stride[2] == 1 and stride[1] == D
                    and T > 1):
                return t.data_ptr(), stride[0]
        return self._rows_at(t, name, (T, heads, D), dtype)

    def _rows_at(self, t, name, shape, dtype):
        """The address and the row stride of a tensor whose rows (of all but the first dimension)
        are contiguous and lie at any distance."""
        if t.is_contiguous():
            return self._at(t, name, shape, dtype), t.stride(0) if shape[0] > 1 else _numel(shape)
        self._refuse(t, name, shape, dtype)
        stride = t.stride()
        if len(shape) == 3 and shape[1] == 1:
            inner = stride[2] == 1
        else:
            inner = stride[1:] == ((1,) if len(shape) == 2 else (shape[2], 1))
        if not inner and not (shape[0] and t[0].is_contiguous()):
            raise ValueError("%s must be contiguous within a row" % name)
        # The stride of a single row is arbitrary.
        return t.data_ptr(), stride[0] if shape[0] > 1 else _numel(shape)

    def _refuse(self, t, name, shape, dtype):
        """Raises for a wrong shape, type or device."""
        if t.shape != shape:
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
        if t.dtype is not dtype:
            raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
        if t.get_device() != self._index:
            raise ValueError("%s is on %s, the plan on %s" % (name, t.device, self.device))

    def close(self):
        if self.handle:
            type(self)._destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedAttention(_DecodePlan):
    """Attention of one new token for each of ``B`` sequences over a paged cache.

    The cache is ``k_pages`` and ``v_pages``, [num_pages, H_kv, page_size, D] (``layout``
    "head") or [num_pages, page_size, H_kv, D] ("token"): given, or allocated (zeros) when only
    ``num_pages`` is.  Slot j of sequence b is row j % page_size of page
    ``tables[b, j // page_size]``.  ``window`` > 0 attends to the last that many slots;
    ``weights`` accumulates every slot's attention weight, for ``evict``; ``chunks`` makes room for
    ``forward_chunk``.
    """

    def __init__(self, B, H_q, H_kv, D, page_size, max_pages, num_pages=None, k_pages=None,
                 v_pages=None, dtype=None, layout="head", window=0, scale=None, weights=False,
                 device=None, chunks=False):
        if layout not in ("head", "token"):
            raise ValueError("layout must be 'head' or 'token'")
        if (k_pages is None) != (v_pages is None):
            raise ValueError("k_pages and v_pages belong together")
        if k_pages is None and num_pages is None:
            raise ValueError("give k_pages and v_pages, or num_pages")
        if k_pages is not None:
            device = k_pages.device if device is None else device
            dtype = k_pages.dtype if dtype is None else dtype
            num_pages = k_pages.shape[0] if num_pages is None else num_pages
        self.device = _device_of(device)
        self._index = self.device.index
        self.dtype = dtype if dtype is not None else torch.float32
        self.B, self.H_q, self.H_kv, self.D = int(B), int(H_q), int(H_kv), int(D)
        self.page_size, self.max_pages = int(page_size), int(max_pages)
        self.num_pages, self.capacity = int(num_pages), int(page_size) * int(max_pages)
        self.layout, self.window, self.weights = layout, int(window), bool(weights)
        self.chunks = bool(chunks)
        shape = ((self.num_pages, self.H_kv, self.page_size, self.D) if layout == "head" else
                 (self.num_pages, self.page_size, self.H_kv, self.D))
        self.handle = _ctr.ctr_attn_create(B, H_q, H_kv, D, page_size, max_pages,
                                           _ctr._dtype_code(self.dtype))
        try:
            if layout == "token":
                _ctr.ctr_attn_set_layout(self.handle, _ctr.CTR_CACHE_TOKEN_MAJOR)
            if self.window:
                _ctr.ctr_attn_set_window(self.handle, self.window)
            if scale is not None:
                _ctr.ctr_attn_set_scale(self.handle, scale)
            if self.weights:
                _ctr.ctr_attn_set_weights(self.handle, 1)
            if self.chunks:
                _ctr.ctr_attn_set_chunks(self.handle, 1)
            if k_pages is None:
                k_pages = torch.zeros(shape, dtype=self.dtype, device=self.device)
                v_pages = torch.zeros(shape, dtype=self.dtype, device=self.device)
            k = self._at(k_pages, "k_pages", shape, self.dtype)
            v = self._at(v_pages, "v_pages", shape, self.dtype)
            self.k_pages, self.v_pages = k_pages, v_pages
            _ctr.ctr_attn_bind_cache(self.handle, k, v, self.num_pages)
            self.workspace_bytes = _ctr.ctr_attn_workspace_bytes(self.handle)
            self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)
            self._kept = (self.workspace, self.k_pages, self.v_pages)
            _ctr.ctr_attn_bind_workspace(self.handle, self.workspace.data_ptr(),
                                         self.workspace_bytes)
            self._q_shape, self._kv_shape = (self.B, self.H_q, self.D), (self.B, self.H_kv, self.D)
            self._table_shape, self._lens_shape = (self.B, self.max_pages), (self.B,)
            self._weights_shape = (self.B, self.H_kv, self.capacity)
            self._forward = _ctr.load_library().ctr_attn_forward
            self._evict = _ctr.load_library().ctr_attn_evict
            self._forward_chunk = _ctr.load_library().ctr_attn_forward_chunk
            self._put = _ctr.load_library().ctr_attn_put
            self._starts_shape = (self.B + 1,)
            with torch.cuda.device(self.device):
                _ctr.ctr_attn_reset(self.handle, self._stream(None))
                # The plan may be used on any stream from here on.
                torch.cuda.current_stream().synchronize()
        except Exception:
            self.close()
            raise

    _destroy = staticmethod(lambda handle: _ctr.ctr_attn_destroy(handle))

    def forward(self, q, tables, lens, k_new=None, v_new=None, weights=None, weights_out=None,
                out=None, stream=None):
        """out [B, H_q, D] of q [B, H_q, D] over each sequence's cached tokens; with k_new and
        v_new [B, H_kv, D], which the call puts at slot lens[b], over those too.  q, k_new
        and v_new may be slices of a fused projection (any row stride).  tables [B, max_pages]
        and lens [B] are int32; lens[b] < 0 marks an idle row.  A plan with weights adds this
        step's to ``weights`` [B, H_kv, max_pages * page_size] (None: zeros) and writes the sums
        to ``weights_out`` (default: ``weights`` itself)."""
        q_ptr, q_stride = self._rows_at(q, "q", self._q_shape, self.dtype)
        k_ptr = v_ptr = wi_ptr = wo_ptr = None
        kv_stride = 0
        if k_new is not None and v_new is not None:
            k_ptr, kv_stride = self._rows_at(k_new, "k_new", self._kv_shape, self.dtype)
            v_ptr, v_stride = self._rows_at(v_new, "v_new", self._kv_shape, self.dtype)
            if v_stride != kv_stride:
                raise ValueError("k_new and v_new must have the same row stride")
        elif k_new is not None or v_new is not None:
            raise ValueError("k_new and v_new belong together")
        t_ptr = self._at(tables, "tables", self._table_shape, torch.int32)
        l_ptr = self._at(lens, "lens", self._lens_shape, torch.int32)
        if self.weights:
            if weights_out is None:
                weights_out = weights
            if weights_out is None:
                raise ValueError("a plan with weights needs weights or weights_out")
            if weights is not None:
                wi_ptr = self._at(weights, "weights", self._weights_shape, torch.float32)
            wo_ptr = self._at(weights_out, "weights_out", self._weights_shape, torch.float32)
        elif weights is not None or weights_out is not None:
            raise ValueError("the plan was made without weights")
        if out is None:
            out = torch.empty(self._q_shape, dtype=self.dtype, device=self.device)
            raw = self._stream(stream, out)
        else:
            raw = self._stream(stream)
        o_ptr = self._at(out, "out", self._q_shape, self.dtype)
        st = self._forward(self.handle, q_ptr, q_stride, k_ptr, v_ptr, kv_stride, t_ptr, l_ptr, wi_ptr,
                           wo_ptr, o_ptr, raw)
        if st:
            raise _ctr.CtrError(st, "ctr_attn_forward")
        return out

    def put(self, k, v, slots, q=None, positions=None, rotary=None, q_out=None, stream=None):
        """Put the K and V rows of new tokens, k and v [T, H_kv, D], into the cache at slots [T]
        (int64, page * page_size + row; negative: nowhere).  ``rotary`` (a ``Rotary`` plan of this D
        and dtype) turns K by positions [T] (int32) on the way, and q [T, H_q, D], which the call then
        returns turned (in q_out, which may be q).  k, v and q may be slices of a fused projection."""
        T = k.shape[0] if k.dim() else 0
        k_ptr, kv_stride = self._heads_at(k, "k", T, self.H_kv, self.D, self.dtype)
        v_ptr, v_stride = self._heads_at(v, "v", T, self.H_kv, self.D, self.dtype)
        if v_stride != kv_stride:
            raise ValueError("k and v must have the same row stride")
        s_ptr = self._at(slots, "slots", (T,), torch.int64)
        p_ptr = r_ptr = q_ptr = o_ptr = None
        q_stride = o_stride = 0
        made = ()
        if rotary is not None:
            if positions is None:
                raise ValueError("a rotary plan needs positions")
            if rotary.D != self.D or rotary.dtype is not self.dtype:
                raise ValueError("the rotary plan has D = %d, %s, the cache D = %d, %s"
                                 % (rotary.D, rotary.dtype, self.D, self.dtype))
            p_ptr = self._at(positions, "positions", (T,), torch.int32)
            r_ptr = rotary.handle
            if not r_ptr:
                # (The C call takes no plan for no rotation.)
                raise ValueError("the rotary plan is closed")
        elif positions is not None:
            raise ValueError("positions without a rotary plan")
        if q is not None:
            if rotary is None:
                raise ValueError("q without a rotary plan")
            shape = (T, self.H_q, self.D)
            q_ptr, q_stride = self._heads_at(q, "q", T, self.H_q, self.D, self.dtype)
            if q_out is None:
                q_out = torch.empty(shape, dtype=self.dtype, device=self.device)
                made = (q_out,)
            o_ptr, o_stride = self._heads_at(q_out, "q_out", T, self.H_q, self.D, self.dtype)
            if not T:
                q_ptr = o_ptr = None
        elif q_out is not None:
            raise ValueError("q_out without q")
        st = self._put(self.handle, r_ptr, q_ptr, q_stride, k_ptr, v_ptr, kv_stride, p_ptr, s_ptr, T,
                       o_ptr, o_stride, self._stream(stream, *made))
        if st:
            raise _ctr.CtrError(st, "ctr_attn_put")
        return q_out

    def forward_chunk(self, q, tables, lens, starts, out=None, stream=None):
        """out [T, H_q, D] of q [T, H_q, D], whose rows starts[b] .. starts[b + 1] - 1 are the new tokens
        of sequence b, at the slots from lens[b] on, where ``put`` has put their K and V: each attends
        to the slots up to its own (the last ``window`` of them).  tables [B, max_pages], lens [B] and
        starts [B + 1] are int32; lens[b] < 0 marks an idle sequence, whose rows give 0.  q may be a
        slice of a fused projection.  Rows of ``out`` that no sequence has are left as they are (anything,
        in a tensor that the call makes)."""
        T = q.shape[0] if q.dim() else 0
        shape = (T, self.H_q, self.D)
        q_ptr, q_stride = self._heads_at(q, "q", T, self.H_q, self.D, self.dtype)
        t_ptr = self._at(tables, "tables", self._table_shape, torch.int32)
        l_ptr = self._at(lens, "lens", self._lens_shape, torch.int32)
        s_ptr = self._at(starts, "starts", self._starts_shape, torch.int32)
        if out is None:
            out = torch.empty(shape, dtype=self.dtype, device=self.device)
            raw = self._stream(stream, out)
        else:
            raw = self._stream(stream)
        st = self._forward_chunk(self.handle, q_ptr, q_stride, T, t_ptr, l_ptr, s_ptr,
                                 self._at(out, "out", shape, self.dtype), raw)
        if st:
            raise _ctr.CtrError(st, "ctr_attn_forward_chunk")
        return out

    def evict(self, tables, lens, weights, dst_tables, budget, sinks=0, recent=0, slots=None,
              lens_out=None, weights_out=None, stream=None):
        """Keep ``budget`` slots of every (sequence, head) -- the first ``sinks``, the last
        ``recent`` and the heaviest others -- and copy them, in order, to the pages of
        ``dst_tables`` [B, >= ceil(budget / page_size)].  Returns (slots [B, H_kv, budget] int32,
        the kept slots then -1; lens_out [B] int32, the new lengths; weights_out [B, H_kv, >=
        budget], the kept weights in front).  The source pages stay as they are."""
        budget = int(budget)
        if dst_tables.dim() != 2 or dst_tables.shape[0] != self.B:
            raise ValueError("dst_tables must be [%d, pages]" % self.B)
        at, made = self._at, []
        shape = (self.B, self.H_kv, max(budget, 0))
        t_ptr = at(tables, "tables", self._table_shape, torch.int32)
        l_ptr = at(lens, "lens", self._lens_shape, torch.int32)
        w_ptr = at(weights, "weights", self._weights_shape, torch.float32)
        d_ptr = at(dst_tables, "dst_tables", dst_tables.shape, torch.int32)
        if slots is None:
            slots = torch.empty(shape, dtype=torch.int32, device=self.device)
            made.append(slots)
        if lens_out is None:
            lens_out = torch.empty(self._lens_shape, dtype=torch.int32, device=self.device)
            made.append(lens_out)
        clear = weights_out is None
        if clear:
            weights_out = torch.empty(shape, dtype=torch.float32, device=self.device)
            made.append(weights_out)
        if weights_out.dim() != 3:
            raise ValueError("weights_out must be [%d, %d, >= %d]" % (self.B, self.H_kv, budget))
        pitch = weights_out.shape[2]
        s_ptr = at(slots, "slots", shape, torch.int32)
        lo_ptr = at(lens_out, "lens_out", self._lens_shape, torch.int32)
        wo_ptr = at(weights_out, "weights_out", (self.B, self.H_kv, pitch), torch.float32)
        raw = self._stream(stream, *made)
        if clear:
            # On the call's own stream: on the current one it might run after the kernels.
            with torch.cuda.stream(stream):
                weights_out.zero_()
        st = self._evict(self.handle, t_ptr, l_ptr, w_ptr, d_ptr, dst_tables.shape[1], budget,
                         int(sinks), int(recent), s_ptr, lo_ptr, wo_ptr, pitch, raw)
        if st:
            raise _ctr.CtrError(st, "ctr_attn_evict")
        return slots, lens_out, weights_out

    def set_wait_limit_ns(self, ns):
        _ctr.ctr_attn_set_wait_limit_ns(self.handle, ns)

    def check(self, stream=None):
        """Wait for ``stream`` and raise CtrError when a call met a page number, a slot, a length or
        a start out of range, or a kernel gave up waiting for its own copies or products."""
        _ctr.ctr_attn_check(self.handle, self._stream(stream))

    def describe(self) -> str:
        return _ctr.ctr_attn_describe(self.handle)


class Sampler(_DecodePlan):
    """The next token of each of ``rows`` rows from logits over ``vocab`` tokens, with per-row
    temperature, top-k, top-p and min-p and given Exp(1) random numbers."""

    def __init__(self, rows, vocab, dtype=None, device=None):
        self.device = _device_of(device)
        self._index = self.device.index
        self.dtype = dtype if dtype is not None else torch.float32
        self.rows, self.vocab = int(rows), int(vocab)
        self._shape, self._row_shape = (self.rows, self.vocab), (self.rows,)
        self._forward = _ctr.load_library().ctr_sampler_forward
        self.handle = _ctr.ctr_sampler_create(rows, vocab, _ctr._dtype_code(self.dtype))

    _destroy = staticmethod(lambda handle: _ctr.ctr_sampler_destroy(handle))

    def forward(self, logits, noise, temperature=None, top_k=None, top_p=None, min_p=None,
                out=None, stream=None):
        """tokens [rows] int64 from logits [rows, vocab] and noise [rows, vocab] (float32, Exp(1)
        draws; both may have any row stride).  temperature, top_p, min_p (float32) and top_k
        (int32) are [rows] or None for 1, 1, 0 and 0 (off); temperature <= 0 is greedy."""
        at, shape = self._at, self._row_shape
        x_ptr, x_stride = self._rows_at(logits, "logits", self._shape, self.dtype)
        n_ptr, n_stride = self._rows_at(noise, "noise", self._shape, torch.float32)
        if out is None:
            out = torch.empty(shape, dtype=torch.int64, device=self.device)
            raw = self._stream(stream, out)
        else:
            raw = self._stream(stream)
        st = self._forward(
            self.handle, x_ptr, x_stride, n_ptr, n_stride,
            None if temperature is None else at(temperature, "temperature", shape, torch.float32),
            None if top_k is None else at(top_k, "top_k", shape, torch.int32),
            None if top_p is None else at(top_p, "top_p", shape, torch.float32),
            None if min_p is None else at(min_p, "min_p", shape, torch.float32),
            at(out, "out", shape, torch.int64), raw)
        if st:
            raise _ctr.CtrError(st, "ctr_sampler_forward")
        return out

    def describe(self) -> str:
        return _ctr.ctr_sampler_describe(self.handle)
