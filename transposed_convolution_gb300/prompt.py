"""Torch-level plans of what a chunk of new tokens needs besides its attention: ``Rotary`` (rotary
positions) and ``PagePool`` (pages of the cache, slots and positions, reserved on the GPU).

They marshal arguments to the C ABI (``include/ctr.h``: ``ctr_rope_*``, ``ctr_pages_*``) after checking
them, under the rules of ``PagedAttention`` for streams and devices.
"""
from __future__ import annotations

import ctypes

import torch

import transposed_convolution_gb300 as _ctr

from .decode import _DecodePlan, _device_of

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {None: 0, "linear": 1, "parts": 2}


class Rotary(_DecodePlan):
    """Rotary positions for heads of D columns, of which the first ``rotary_dim`` (default: all) are
    turned, as pairs (i, i + rotary_dim / 2) (``layout`` "half") or (2i, 2i + 1) ("interleaved").

    Pair i turns by base ** (-2i / rotary_dim) radians a position.  ``scaling`` "linear" divides that
    by ``factor``; "parts" divides it for pairs that turn fewer than ``low`` times over ``original``
    positions, leaves those of more than ``high`` turns, and blends between, in proportion to the turns;
    ``frequencies`` gives all of them instead (for a blend in proportion to the pair's number, as many models
    were trained with: such a model's come out otherwise with "parts").  ``magnitude`` multiplies what is
    turned."""

    def __init__(self, D, rotary_dim=None, layout="half", base=10000.0, scaling=None, factor=1.0,
                 original=None, low=1.0, high=32.0, magnitude=1.0, frequencies=None, dtype=None,
                 device=None):
        if layout not in _LAYOUTS:
            raise ValueError("layout must be 'half' or 'interleaved'")
        if scaling not in _SCALINGS:
            raise ValueError("scaling must be None, 'linear' or 'parts'")
        if scaling == "parts" and original is None:
            raise ValueError("scaling 'parts' needs original")
        if frequencies is not None and scaling is not None:
            raise ValueError("frequencies are given as they are: no scaling")
        self.device = _device_of(device)
        self._index = self.device.index
        self.dtype = dtype if dtype is not None else torch.float32
        self.D = int(D)
        self.rotary_dim = self.D if rotary_dim is None else int(rotary_dim)
        self.handle = _ctr.ctr_rope_create(self.D, self.rotary_dim, _ctr._dtype_code(self.dtype))
        try:
            _ctr.ctr_rope_set_layout(self.handle, _LAYOUTS[layout])
            _ctr.ctr_rope_set_base(self.handle, base)
            _ctr.ctr_rope_set_scaling(self.handle, _SCALINGS[scaling], factor,
                                      0.0 if original is None else original, low, high)
            _ctr.ctr_rope_set_magnitude(self.handle, magnitude)
            if frequencies is not None:
                _ctr.ctr_rope_set_frequencies(self.handle, [float(f) for f in frequencies])
            self._forward = _ctr.load_library().ctr_rope_forward
        except Exception:
            self.close()
            raise

    _destroy = staticmethod(lambda handle: _ctr.ctr_rope_destroy(handle))

    @property
    def frequencies(self):
        """The rotary_dim / 2 frequencies, in radians a position."""
        return _ctr.ctr_rope_frequencies(self.handle, self.rotary_dim // 2)

    def forward(self, q, k, positions, q_out=None, k_out=None, stream=None):
        """(q_out, k_out) of q [T, H_q, D] and k [T, H_k, D] (either may be None) at positions [T]
        (int32; negative ones turn backwards: with the negated positions the call is its own
        gradient's).  q_out may be q, and k_out k; all may be slices with any row stride."""
        T = positions.shape[0] if positions.dim() else 0
        p_ptr = self._at(positions, "positions", (T,), torch.int32)
        made = ()
        q_ptr = k_ptr = qo_ptr = ko_ptr = None
        q_stride = k_stride = qo_stride = ko_stride = H_q = H_k = 0
        if q is not None:
            q_ptr, q_stride, H_q = self._rows_of(q, "q", T)
            if q_out is None:
                q_out = torch.empty((T, H_q, self.D), dtype=self.dtype, device=self.device)
                made = (q_out,)
                qo_ptr, qo_stride = q_out.data_ptr(), H_q * self.D
            else:
                qo_ptr, qo_stride = self._heads_at(q_out, "q_out", T, H_q, self.D, self.dtype)
        elif q_out is not None:
            raise ValueError("q_out without q")
        if k is not None:
            k_ptr, k_stride, H_k = self._rows_of(k, "k", T)
            if k_out is None:
                k_out = torch.empty((T, H_k, self.D), dtype=self.dtype, device=self.device)
                made += (k_out,)
                ko_ptr, ko_stride = k_out.data_ptr(), H_k * self.D
            else:
                ko_ptr, ko_stride = self._heads_at(k_out, "k_out", T, H_k, self.D, self.dtype)
        elif k_out is not None:
            raise ValueError("k_out without k")
        st = self._forward(self.handle, q_ptr, q_stride, H_q, k_ptr, k_stride, H_k, p_ptr, T, qo_ptr,
                           qo_stride, ko_ptr, ko_stride, self._stream(stream, *made))
        if st:
            raise _ctr.CtrError(st, "ctr_rope_forward")
        return q_out, k_out

    def _rows_of(self, x, name, T):
        if x.dim() != 3:
            raise ValueError("%s must be [%d, heads, %d]" % (name, T, self.D))
        heads = x.shape[1]
        ptr, stride = self._heads_at(x, name, T, heads, self.D, self.dtype)
        return ptr, stride, heads

    def describe(self) -> str:
        return _ctr.ctr_rope_describe(self.handle)


class PagePool(_DecodePlan):
    """The free pages of a cache of ``num_pages`` pages of ``page_size`` rows, for B sequences of up to
    ``max_pages`` pages: ``free`` [num_pages] int32, whose first ``count`` [1] int32 entries are
    free.  Both are allocated, with every page free, or given by the caller (who may share them
    between pools, or take them to the host and back)."""

    def __init__(self, B, page_size, max_pages, num_pages=None, free=None, count=None, device=None):
        if (free is None) != (count is None):
            raise ValueError("free and count belong together")
        if free is None and num_pages is None:
            raise ValueError("give num_pages, or free and count")
        if free is not None:
            device = free.device if device is None else device
            num_pages = free.shape[0] if num_pages is None else num_pages
        self.device = _device_of(device)
        self._index = self.device.index
        self.B, self.page_size, self.max_pages = int(B), int(page_size), int(max_pages)
        self.num_pages = int(num_pages)
        self.handle = _ctr.ctr_pages_create(B, page_size, max_pages)
        try:
            refill = free is None
            if refill:
                free = torch.empty(self.num_pages, dtype=torch.int32, device=self.device)
                count = torch.empty(1, dtype=torch.int32, device=self.device)
            f_ptr = self._at(free, "free", (self.num_pages,), torch.int32)
            c_ptr = self._at(count, "count", (1,), torch.int32)
            _ctr.ctr_pages_bind_list(self.handle, f_ptr, c_ptr, self.num_pages)
            self.free, self.count = free, count
            nbytes = _ctr.ctr_pages_workspace_bytes(self.handle)
            self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            self._kept = (self.workspace, self.free, self.count)
            _ctr.ctr_pages_bind_workspace(self.handle, self.workspace.data_ptr(), nbytes)
            self._table_shape, self._row_shape = (self.B, self.max_pages), (self.B,)
            self._starts_shape = (self.B + 1,)
            self._reserve = _ctr.load_library().ctr_pages_reserve
            self._release = _ctr.load_library().ctr_pages_release
            with torch.cuda.device(self.device):
                _ctr.ctr_pages_reset(self.handle, int(refill), self._stream(None))
                # The plan may be used on any stream from here on.
                torch.cuda.current_stream().synchronize()
        except Exception:
            self.close()
            raise

    _destroy = staticmethod(lambda handle: _ctr.ctr_pages_destroy(handle))

    def _or_empty(self, t, name, shape, dtype, made):
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=self.device)
            made.append(t)
            return t, t.data_ptr()
        return t, self._at(t, name, shape, dtype)

    def reserve(self, tables, lens, counts, rows, granted=None, starts=None, slots=None,
                positions=None, lens_out=None, stream=None):
        """Make room for counts [B] more tokens in each sequence: the pages that are missing go into
        tables [B, max_pages].  Returns (granted [B], the counts, or 0 for requests that do not fit
        behind the earlier ones; starts [B + 1], each sequence's first row; slots [rows] int64 and
        positions [rows], of the new tokens, -1 and 0 behind the last; lens_out [B], the lengths with
        them).  All int32 but the slots; lens is not changed, and lens[b] < 0 marks an idle one.

        The rows are those of the granted requests, one after the other: where one is refused, those behind it
        come earlier than in rows laid out by ``counts``, and the caller brings the two together (as
        ``rows_as_asked`` in examples/prompt_decode.py does, on the GPU) before ``put``."""
        rows, made = int(rows), []
        t_ptr = self._at(tables, "tables", self._table_shape, torch.int32)
        l_ptr = self._at(lens, "lens", self._row_shape, torch.int32)
        c_ptr = self._at(counts, "counts", self._row_shape, torch.int32)
        i32, shape = torch.int32, (max(rows, 0),)
        granted, g_ptr = self._or_empty(granted, "granted", self._row_shape, i32, made)
        starts, st_ptr = self._or_empty(starts, "starts", self._starts_shape, i32, made)
        slots, s_ptr = self._or_empty(slots, "slots", shape, torch.int64, made)
        positions, p_ptr = self._or_empty(positions, "positions", shape, i32, made)
        lens_out, lo_ptr = self._or_empty(lens_out, "lens_out", self._row_shape, i32, made)
        st = self._reserve(self.handle, t_ptr, l_ptr, c_ptr, rows, g_ptr, st_ptr, s_ptr, p_ptr, lo_ptr,
                           self._stream(stream, *made))
        if st:
            raise _ctr.CtrError(st, "ctr_pages_reserve")
        return granted, starts, slots, positions, lens_out

    def release(self, tables, lens, keep, lens_out=None, stream=None):
        """Give back the pages behind each sequence's first keep [B] tokens (int32; negative: all of
        them, and the sequence becomes idle).  Returns lens_out [B], the lengths that are left."""
        made = []
        t_ptr = self._at(tables, "tables", self._table_shape, torch.int32)
        l_ptr = self._at(lens, "lens", self._row_shape, torch.int32)
        k_ptr = self._at(keep, "keep", self._row_shape, torch.int32)
        lens_out, lo_ptr = self._or_empty(lens_out, "lens_out", self._row_shape, torch.int32, made)
        st = self._release(self.handle, t_ptr, l_ptr, k_ptr, lo_ptr, self._stream(stream, *made))
        if st:
            raise _ctr.CtrError(st, "ctr_pages_release")
        return lens_out

    def check(self, stream=None):
        """Wait for ``stream`` and raise CtrError when a call met a length, a count or a page number out
        of range, or gave back more pages than there are."""
        _ctr.ctr_pages_check(self.handle, self._stream(stream))

    def describe(self) -> str:
        return _ctr.ctr_pages_describe(self.handle)
