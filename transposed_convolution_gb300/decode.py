"""Torch-level plans of the decode step: ``PagedAttention`` (attention of one new token over a
paged key-value cache, and eviction from that cache) and ``Sampler`` (the next token from logits
and given random numbers).

Both only marshal arguments to the C ABI (``include/ctr.h``: ``ctr_attn_*``, ``ctr_sampler_*``)
after checking them.  A call runs on ``stream`` (default: the current stream of the plan's
device).  When ``stream`` is another stream than the current one, the caller orders the two, as
for ``Plan``; tensors that the call itself allocates are then kept for that stream.
"""
from __future__ import annotations

import torch

import transposed_convolution_gb300 as _ctr


def _device_of(device):
    d = torch.device(device if device is not None else "cuda")
    if d.type != "cuda":
        raise ValueError("the plan needs a CUDA device, got %s" % d)
    return torch.device("cuda", torch.cuda.current_device() if d.index is None else d.index)


class _DecodePlan:
    """A plan handle on one device, and the checks both plans make of their arguments."""

    handle = None
    _destroy = None

    def _stream(self, stream, *made):
        """The raw stream of a call; tensors that the call made are kept for it."""
        if stream is None:
            return torch.cuda.current_stream(self.device).cuda_stream
        if stream != torch.cuda.current_stream(self.device):
            for t in made:
                t.record_stream(stream)
        return stream.cuda_stream

    def _checked(self, t, name, shape, dtype, rows=False):
        """t's address, after its shape, type, device and layout have been checked.  With
        ``rows`` the first dimension may have any stride; otherwise t is contiguous."""
        if t.shape != shape:
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
        if t.dtype != dtype:
            raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
        if t.device != self.device:
            raise ValueError("%s is on %s, the plan on %s" % (name, t.device, self.device))
        if not (t.is_contiguous() or (rows and t.shape[0] and t[0].is_contiguous())):
            raise ValueError("%s must be contiguous%s" % (name, " within a row" if rows else ""))
        return t.data_ptr()

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
    ``weights`` accumulates every slot's attention weight, for ``evict``.
    """

    def __init__(self, B, H_q, H_kv, D, page_size, max_pages, num_pages=None, k_pages=None,
                 v_pages=None, dtype=None, layout="head", window=0, scale=None, weights=False,
                 device=None):
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
        self.dtype = dtype if dtype is not None else torch.float32
        self.B, self.H_q, self.H_kv, self.D = int(B), int(H_q), int(H_kv), int(D)
        self.page_size, self.max_pages = int(page_size), int(max_pages)
        self.num_pages, self.capacity = int(num_pages), int(page_size) * int(max_pages)
        self.layout, self.window, self.weights = layout, int(window), bool(weights)
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
            if k_pages is None:
                k_pages = torch.zeros(shape, dtype=self.dtype, device=self.device)
                v_pages = torch.zeros(shape, dtype=self.dtype, device=self.device)
            k = self._checked(k_pages, "k_pages", shape, self.dtype)
            v = self._checked(v_pages, "v_pages", shape, self.dtype)
            self.k_pages, self.v_pages = k_pages, v_pages
            _ctr.ctr_attn_bind_cache(self.handle, k, v, self.num_pages)
            self.workspace_bytes = _ctr.ctr_attn_workspace_bytes(self.handle)
            self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)
            _ctr.ctr_attn_bind_workspace(self.handle, self.workspace.data_ptr(),
                                         self.workspace_bytes)
            with torch.cuda.device(self.device):
                _ctr.ctr_attn_reset(self.handle, self._stream(None))
                # The plan may be used on any stream from here on.
                torch.cuda.current_stream().synchronize()
        except Exception:
            self.close()
            raise

    _destroy = staticmethod(lambda handle: _ctr.ctr_attn_destroy(handle))

    def _weights(self, t, name):
        return self._checked(t, name, (self.B, self.H_kv, self.capacity), torch.float32)

    def forward(self, q, tables, lens, k_new=None, v_new=None, weights=None, weights_out=None,
                out=None, stream=None):
        """out [B, H_q, D] of q [B, H_q, D] over each sequence's cached tokens; with k_new and
        v_new [B, H_kv, D], which the call puts at slot lens[b], over those too.  q, k_new
        and v_new may be slices of a fused projection (any row stride).  tables [B, max_pages]
        and lens [B] are int32; lens[b] < 0 marks an idle row.  A plan with weights adds this
        step's to ``weights`` [B, H_kv, max_pages * page_size] (None: zeros) and writes the sums
        to ``weights_out`` (default: ``weights`` itself)."""
        if (k_new is None) != (v_new is None):
            raise ValueError("k_new and v_new belong together")
        q_ptr = self._checked(q, "q", (self.B, self.H_q, self.D), self.dtype, rows=True)
        k_ptr = v_ptr = None
        kv_stride = 0
        if k_new is not None:
            shape = (self.B, self.H_kv, self.D)
            k_ptr = self._checked(k_new, "k_new", shape, self.dtype, rows=True)
            v_ptr = self._checked(v_new, "v_new", shape, self.dtype, rows=True)
            kv_stride = self._row_stride(k_new)
            if self._row_stride(v_new) != kv_stride:
                raise ValueError("k_new and v_new must have the same row stride")
        t_ptr = self._checked(tables, "tables", (self.B, self.max_pages), torch.int32)
        l_ptr = self._checked(lens, "lens", (self.B,), torch.int32)
        wi_ptr = wo_ptr = None
        if self.weights:
            if weights_out is None:
                weights_out = weights
            if weights_out is None:
                raise ValueError("a plan with weights needs weights or weights_out")
            wi_ptr = None if weights is None else self._weights(weights, "weights")
            wo_ptr = self._weights(weights_out, "weights_out")
        elif weights is not None or weights_out is not None:
            raise ValueError("the plan was made without weights")
        made = ()
        if out is None:
            out = torch.empty((self.B, self.H_q, self.D), dtype=self.dtype, device=self.device)
            made = (out,)
        o_ptr = self._checked(out, "out", (self.B, self.H_q, self.D), self.dtype)
        _ctr.ctr_attn_forward(self.handle, q_ptr, self._row_stride(q), k_ptr, v_ptr, kv_stride, t_ptr,
                              l_ptr, wi_ptr, wo_ptr, o_ptr, self._stream(stream, *made))
        return out

    @staticmethod
    def _row_stride(t):
        # The stride of a single row is arbitrary: any valid one will do.
        return t.stride(0) if t.shape[0] > 1 else t[0].numel()

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
        t_ptr = self._checked(tables, "tables", (self.B, self.max_pages), torch.int32)
        l_ptr = self._checked(lens, "lens", (self.B,), torch.int32)
        w_ptr = self._weights(weights, "weights")
        d_ptr = self._checked(dst_tables, "dst_tables", tuple(dst_tables.shape), torch.int32)
        made = []
        if slots is None:
            slots = torch.empty((self.B, self.H_kv, max(budget, 0)), dtype=torch.int32,
                                device=self.device)
            made.append(slots)
        if lens_out is None:
            lens_out = torch.empty((self.B,), dtype=torch.int32, device=self.device)
            made.append(lens_out)
        if weights_out is None:
            weights_out = torch.zeros((self.B, self.H_kv, max(budget, 0)), dtype=torch.float32,
                                      device=self.device)
            made.append(weights_out)
        if weights_out.dim() != 3:
            raise ValueError("weights_out must be [%d, %d, >= %d]" % (self.B, self.H_kv, budget))
        pitch = weights_out.shape[2]
        s_ptr = self._checked(slots, "slots", (self.B, self.H_kv, budget), torch.int32)
        lo_ptr = self._checked(lens_out, "lens_out", (self.B,), torch.int32)
        wo_ptr = self._checked(weights_out, "weights_out", (self.B, self.H_kv, pitch), torch.float32)
        _ctr.ctr_attn_evict(self.handle, t_ptr, l_ptr, w_ptr, d_ptr, dst_tables.shape[1], budget,
                            int(sinks), int(recent), s_ptr, lo_ptr, wo_ptr, pitch,
                            self._stream(stream, *made))
        return slots, lens_out, weights_out

    def check(self, stream=None):
        """Wait for ``stream`` and raise CtrError when a call met a page number or a length out
        of range."""
        _ctr.ctr_attn_check(self.handle, self._stream(stream))

    def describe(self) -> str:
        return _ctr.ctr_attn_describe(self.handle)


class Sampler(_DecodePlan):
    """The next token of each of ``rows`` rows from logits over ``vocab`` tokens, with per-row
    temperature, top-k, top-p and min-p and given Exp(1) random numbers."""

    def __init__(self, rows, vocab, dtype=None, device=None):
        self.device = _device_of(device)
        self.dtype = dtype if dtype is not None else torch.float32
        self.rows, self.vocab = int(rows), int(vocab)
        self.handle = _ctr.ctr_sampler_create(rows, vocab, _ctr._dtype_code(self.dtype))

    _destroy = staticmethod(lambda handle: _ctr.ctr_sampler_destroy(handle))

    def _per_row(self, t, name, dtype):
        return None if t is None else self._checked(t, name, (self.rows,), dtype)

    def forward(self, logits, noise, temperature=None, top_k=None, top_p=None, min_p=None,
                out=None, stream=None):
        """tokens [rows] int64 from logits [rows, vocab] and noise [rows, vocab] (float32, Exp(1)
        draws; both may have any row stride).  temperature, top_p, min_p (float32) and top_k
        (int32) are [rows] or None for 1, 1, 0 and 0 (off); temperature <= 0 is greedy."""
        shape = (self.rows, self.vocab)
        x_ptr = self._checked(logits, "logits", shape, self.dtype, rows=True)
        n_ptr = self._checked(noise, "noise", shape, torch.float32, rows=True)
        made = ()
        if out is None:
            out = torch.empty((self.rows,), dtype=torch.int64, device=self.device)
            made = (out,)
        o_ptr = self._checked(out, "out", (self.rows,), torch.int64)
        strides = [t.stride(0) if self.rows > 1 else self.vocab for t in (logits, noise)]
        _ctr.ctr_sampler_forward(self.handle, x_ptr, strides[0], n_ptr, strides[1],
                                 self._per_row(temperature, "temperature", torch.float32),
                                 self._per_row(top_k, "top_k", torch.int32),
                                 self._per_row(top_p, "top_p", torch.float32),
                                 self._per_row(min_p, "min_p", torch.float32), o_ptr,
                                 self._stream(stream, *made))
        return out

    def describe(self) -> str:
        return _ctr.ctr_sampler_describe(self.handle)
