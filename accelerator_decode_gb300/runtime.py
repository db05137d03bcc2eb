"""Device-side plumbing around libg4: upload host weights with PyTorch, hold the borrowed
tensors alive, and marshal calls.  No decoder arithmetic happens here."""
import ctypes
import operator

import numpy as np
import torch

from . import g4 as _g4


def _dev(a, device):
    """Host numpy array (any integer dtype) -> CUDA tensor of the same bytes."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    elif a.dtype == np.uint32:
        a = a.view(np.int32)
    return torch.from_numpy(a).to(device, non_blocking=False)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def stream_handle(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class Decoder:
    """One libg4 handle.  `weights` is a host weight dict in the canonical format (synth).
    kv_format "bf16", "int8" or "int4" (cache rows); kv_page_size 0 (static rows) or a power of two
    (paged cache of kv_pages pages, 0 = as many as static rows would take).  Vocabulary
    tables given as int4 dicts (packed, scales) select the int4 table format."""

    def __init__(self, cfg, weights, max_batch, max_context, device=0, kv_format="bf16", kv_page_size=0,
                 kv_pages=0):
        t4 = [isinstance(weights[k], dict) for k in ("embed", "ple_table")]
        if t4[0] != t4[1]:
            raise ValueError("the token embedding and the per-layer table share one table format")
        self.cfg = cfg
        self.device = torch.device("cuda", device)
        self.max_batch, self.max_context = max_batch, max_context
        self.fmt = weights["fmt"]
        self.table_format = "w4a16" if t4[0] else "bf16"
        self.c = _g4.make_config(cfg, self.fmt, max_batch, max_context, kv_format, kv_page_size, kv_pages,
                                 self.table_format)
        keep, tmp = [], []

        def borrow(a):
            t = _dev(a, self.device)
            keep.append(t)
            return _ptr(t)

        def linear(x):
            lin = _g4.g4_linear()
            if "w" in x:
                t = _dev(x["w"], self.device)
                tmp.append(t)
                lin.w = t.data_ptr()
            else:
                t = _dev(x["packed"], self.device)
                s = _dev(x["scales"], self.device)
                tmp.extend([t, s])
                lin.w, lin.scales = t.data_ptr(), s.data_ptr()
            return lin

        L = cfg["num_layers"]
        layers = (_g4.g4_layer_weights * L)()
        for l, lw in enumerate(weights["layers"]):
            for n in _g4.LINEAR_NAMES:
                setattr(layers[l], n, linear(lw[n]))
            for n in _g4.NORM_NAMES:
                setattr(layers[l], n, borrow(lw[n]))
            layers[l].layer_scale = float(lw["layer_scale"])
        w = _g4.g4_weights()
        if self.table_format == "w4a16":
            w.embed = borrow(weights["embed"]["packed"])
            w.embed_scales = borrow(weights["embed"]["scales"])
            w.ple_table = borrow(weights["ple_table"]["packed"])
            w.ple_table_scales = borrow(weights["ple_table"]["scales"])
        else:
            w.embed = borrow(weights["embed"])
            w.ple_table = borrow(weights["ple_table"])
        w.ple_model_proj = linear(weights["ple_model_proj"])
        w.ple_proj_norm = borrow(weights["ple_proj_norm"])
        w.final_norm = borrow(weights["final_norm"])
        w.layers = layers
        torch.cuda.synchronize(self.device)
        self.h = _g4.g4_create(self.c, w, device)
        del tmp                         # linears were copied into the library's layout
        self._keep = keep               # embed, per-layer table and gains are borrowed
        self._trace = None
        torch.cuda.empty_cache()

    # -- calls -------------------------------------------------------------------------------
    def prefill(self, slots, prompts, start_pos=None, stream=None, want_logits=False):
        """prompts: list of host int arrays.  Returns (next ids [n] int32, logits [n, V] or None),
        both device tensors (valid after the stream synchronises)."""
        n = len(prompts)
        lens = [len(p) for p in prompts]
        offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        toks = torch.from_numpy(np.concatenate([np.asarray(p, np.int32) for p in prompts])).to(self.device)
        nxt = torch.empty(n, dtype=torch.int32, device=self.device)
        logits = torch.empty(n, self.cfg["vocab"], dtype=torch.float32, device=self.device) if want_logits else None
        start = [0] * n if start_pos is None else list(start_pos)
        _g4.g4_prefill(self.h, stream_handle(stream), list(slots), offsets.tolist(), start, _ptr(toks),
                       _ptr(nxt), _ptr(logits))
        self._last_prefill_tokens = toks   # keep alive until the stream runs
        return nxt, logits

    def decode_step(self, d_slots, d_tokens, d_positions, d_next, d_logits=None, stream=None):
        n = d_tokens.numel()
        _g4.g4_decode_step(self.h, stream_handle(stream), n, _ptr(d_slots), _ptr(d_tokens), _ptr(d_positions),
                           _ptr(d_next), _ptr(d_logits))

    def profile_step(self, d_slots, d_tokens, d_positions, d_next, d_logits=None, repeats=1, stream=None):
        return _g4.g4_profile_step(self.h, stream_handle(stream), d_tokens.numel(), _ptr(d_slots), _ptr(d_tokens),
                                   _ptr(d_positions), _ptr(d_next), _ptr(d_logits), repeats)

    def reserve(self, slot, n_positions, stream=None):
        """Paged cache: pages for positions [0, n_positions) of `slot` (no-op when static)."""
        _g4.g4_kv_reserve(self.h, stream_handle(stream), int(slot), int(n_positions))

    def release(self, slot, stream=None):
        """Paged cache: return the slot's pages to the pool."""
        _g4.g4_kv_release(self.h, stream_handle(stream), int(slot))

    def pages_free(self):
        return _g4.g4_kv_pages_free(self.h)

    def device_error(self, stream=None):
        return _g4.g4_get_device_error(self.h, stream_handle(stream))

    def set_trace(self, enable):
        c = self.cfg
        stride = max(c["hidden"], c["num_q_heads"] * max(c["head_dim_full"], c["head_dim_sliding"]))
        if enable:
            self._trace = torch.zeros(c["num_layers"], 2, self.max_batch, stride, dtype=torch.float32,
                                      device=self.device)
            _g4.g4_set_trace(self.h, _ptr(self._trace), self._trace.numel())
        else:
            _g4.g4_set_trace(self.h, None, 0)
            self._trace = None
        return self._trace

    def step_mode(self, n_seq=1):
        """1: persistent single-launch step; 0: one launch per phase."""
        return _g4.lib.g4_step_mode(self.h, n_seq)

    def set_step_mode(self, mode):
        """0 (default): one launch per phase; 1: persistent single-launch step for n_seq <= 2."""
        _g4.g4_set_step_mode(self.h, int(mode))

    def device_bytes(self):
        return _g4.lib.g4_device_bytes(self.h)

    def close(self):
        if getattr(self, "h", None) is not None:
            _g4.g4_free(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class LinearOp:
    """Standalone projection kernel (the decode step's GEMV) on one weight matrix."""

    def __init__(self, fmt, lin, device=0):
        self.device = torch.device("cuda", device)
        n_out, n_in = lin["shape"]
        self.n_out, self.n_in = n_out, n_in
        if fmt == "bf16":
            w = _dev(lin["w"], self.device)
            s = None
        else:
            w = _dev(lin["packed"], self.device)
            s = _dev(lin["scales"], self.device)
        h = ctypes.c_void_p()
        st = _g4.lib.g4_linear_create(device, _g4.G4_W4A16 if fmt == "w4a16" else _g4.G4_BF16, n_out, n_in,
                                      _ptr(w), _ptr(s), ctypes.byref(h))
        _g4.check(st, "g4_linear_create")
        self.h = h

    def __call__(self, x, stream=None):
        y = torch.empty(x.shape[0], self.n_out, dtype=torch.float32, device=self.device)
        _g4.check(_g4.lib.g4_linear_forward(self.h, stream_handle(stream), x.shape[0], _ptr(x), _ptr(y)),
                  "g4_linear_forward")
        return y

    def close(self):
        if getattr(self, "h", None) is not None:
            _g4.lib.g4_linear_free(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def argmax_rows(logits, stream=None):
    ids = torch.empty(logits.shape[0], dtype=torch.int32, device=logits.device)
    _g4.check(_g4.lib.g4_argmax_rows(logits.device.index, stream_handle(stream), logits.shape[0],
                                     logits.shape[1], _ptr(logits), _ptr(ids)), "g4_argmax_rows")
    return ids


def argmax_rows_static(logits, stream=None):
    """Allocation-free row argmax (fixed scratch inside the library; see include/g4.h)."""
    ids = torch.empty(logits.shape[0], dtype=torch.int32, device=logits.device)
    _g4.check(_g4.lib.g4_argmax_rows_static(logits.device.index, stream_handle(stream), logits.shape[0],
                                            logits.shape[1], _ptr(logits), _ptr(ids)), "g4_argmax_rows_static")
    return ids


_KV4_TYPES = {torch.float32: _g4.G4_DT_F32, torch.bfloat16: _g4.G4_DT_BF16, torch.float16: _g4.G4_DT_F16}


def _kv4_int(name, v):
    """A whole number that C's int32 holds (ctypes would pass its low 32 bits without a word)."""
    v = operator.index(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} is {v}: 32 bits do not hold it")
    return v


def _kv4_array(name, t, shape, dtype, index):
    """Checks a contiguous array on device `index`; its address (None: NULL)."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} has to be contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{index}")
    return t.data_ptr()


class KV4Cache:
    """A KV cache held in 4 bits (g4_kv4_* in include/g4.h): one layer's rows.

    slots, start, lens and counts are int32 device tensors with one entry per sequence.
    page_table: int32 [n_slots, ceil(capacity / page_size)] on the device (kept, and read by every
    call); n_pages defaults to its number of entries.  track: every row carries its position and
    accumulated attention weight, which `evict` goes by.  Calls run on `stream` (default: the
    current one), where their results are valid; calls on one cache have to be ordered, and come
    from one host thread at a time."""

    def __init__(self, n_slots, capacity, num_q_heads, num_kv_heads, head_dim, max_q_len=64, page_size=0,
                 page_table=None, n_pages=None, track=False, device=None):
        self.index = torch.cuda.current_device() if device is None else torch.device("cuda", device).index
        self.device = torch.device("cuda", self.index)
        n_slots, capacity, num_q_heads, num_kv_heads, head_dim, max_q_len, page_size = (
            _kv4_int(name, v) for name, v in (
                ("n_slots", n_slots), ("capacity", capacity), ("num_q_heads", num_q_heads),
                ("num_kv_heads", num_kv_heads), ("head_dim", head_dim), ("max_q_len", max_q_len), ("page_size", page_size)))
        if page_size:
            if page_table is None or page_size < 0:
                raise ValueError("a paged cache needs its page_table")
            _kv4_array("page_table", page_table, (n_slots, -(-capacity // page_size)), torch.int32, self.index)
        elif page_table is not None:
            raise ValueError("page_table without page_size")
        self.n_slots, self.capacity, self.track = n_slots, capacity, bool(track)
        self.num_q_heads, self.num_kv_heads, self.head_dim = num_q_heads, num_kv_heads, head_dim
        self._table = page_table
        c = _g4.g4_kv4_config(n_slots, capacity, num_q_heads, num_kv_heads, head_dim, max_q_len, page_size,
                              _kv4_int("n_pages", page_table.numel() if n_pages is None else n_pages) if page_size else 0,
                              int(track))
        h = ctypes.c_void_p()
        _g4.check(_g4.lib.g4_kv4_create(self.index, ctypes.byref(c), _ptr(page_table), ctypes.byref(h)),
                  "g4_kv4_create")
        self.h = h
        # the two tensor arguments of a call, filled in anew each time
        self._ta, self._tb = _g4.g4_kv4_tensor(), _g4.g4_kv4_tensor()
        self._pa, self._pb = ctypes.byref(self._ta), ctypes.byref(self._tb)

    # -- arguments ---------------------------------------------------------------------------
    def _dense(self, name, t, shape, into):
        """Checks a dense [sequences, rows, heads, head_dim] argument and describes it to C."""
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
        code = _KV4_TYPES.get(t.dtype)
        if code is None:
            raise TypeError(f"{name} is {t.dtype}: float32, bfloat16 or float16 is wanted")
        s = t.stride()
        if s[3] != 1:
            raise ValueError(f"{name}: the last dimension has to be contiguous")
        if t.get_device() != self.index:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")
        into.data, into.dtype = t.data_ptr(), code
        into.seq_stride, into.row_stride, into.head_stride = s[0], s[1], s[2]

    def _fresh(self, t, code, rows, heads, into):
        """Describes a contiguous result to C."""
        d = self.head_dim
        into.data, into.dtype = t.data_ptr(), code
        into.seq_stride, into.row_stride, into.head_stride = rows * heads * d, heads * d, d

    def _seq(self, name, t, n):
        return _kv4_array(name, t, (n,), torch.int32, self.index)

    def _stream(self, stream):
        """The stream's handle."""
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.index)
        if stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {self.device}")
        return stream.cuda_stream

    def _empty(self, shape, dtype, stream):
        """A result, made on the stream that fills it."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _done(self, status, name, stream, used):
        """Raises for an error; the caching allocator learns of the tensors used on a given stream."""
        if status:
            raise _g4.G4Error(status, name)
        if stream is not None:
            for t in used:
                if t is not None:
                    t.record_stream(stream)

    # -- calls -------------------------------------------------------------------------------
    def append(self, k, v, slots, start, counts=None, positions=None, weights=None, stream=None):
        """Code rows k, v [n, rows, num_kv_heads, head_dim] into rows start[i].. of slots[i].  With track,
        positions not given are counted on from the newest that the slot holds (from 0 at row 0)."""
        n, rows = slots.numel(), k.shape[1] if k.dim() == 4 else -1
        shape = (n, rows, self.num_kv_heads, self.head_dim)
        self._dense("k", k, shape, self._ta)
        self._dense("v", v, shape, self._tb)
        per = (n, self.num_kv_heads, rows)
        status = _g4.lib.g4_kv4_append(
            self.h, self._stream(stream), n, self._seq("slots", slots, n), self._seq("start", start, n),
            self._seq("counts", counts, n), rows, self._pa, self._pb,
            _kv4_array("positions", positions, per, torch.int32, self.index),
            _kv4_array("weights", weights, per, torch.float32, self.index))
        self._done(status, "g4_kv4_append", stream, (k, v, slots, start, counts, positions, weights))

    def read(self, slots, start, n_rows, counts=None, dtype=torch.bfloat16, stream=None):
        """(k, v) of rows start[i].. of slots[i], [n, n_rows, num_kv_heads, head_dim]; zeros where
        there is no row (at and beyond counts[i], on a missing page)."""
        n, n_rows = slots.numel(), _kv4_int("n_rows", n_rows)
        shape = (n, n_rows, self.num_kv_heads, self.head_dim)
        if dtype not in _KV4_TYPES:
            raise TypeError(f"rows cannot be given as {dtype}")
        args = (self._seq("slots", slots, n), self._seq("start", start, n), self._seq("counts", counts, n))
        k, v = self._empty(shape, dtype, stream), self._empty(shape, dtype, stream)
        self._fresh(k, _KV4_TYPES[dtype], n_rows, self.num_kv_heads, self._ta)
        self._fresh(v, _KV4_TYPES[dtype], n_rows, self.num_kv_heads, self._tb)
        status = _g4.lib.g4_kv4_read(self.h, self._stream(stream), n, *args, n_rows, 1, self._pa, self._pb)
        self._done(status, "g4_kv4_read", stream, (slots, start, counts))
        return k, v

    def account(self, slots, start, n_rows, counts=None, stream=None):
        """(positions, accumulated weights) of rows, [n, num_kv_heads, n_rows]; zeros where there is
        no row."""
        n, n_rows = slots.numel(), _kv4_int("n_rows", n_rows)
        shape = (n, self.num_kv_heads, n_rows)
        args = (self._seq("slots", slots, n), self._seq("start", start, n), self._seq("counts", counts, n))
        pos, weight = self._empty(shape, torch.int32, stream), self._empty(shape, torch.float32, stream)
        status = _g4.lib.g4_kv4_account(self.h, self._stream(stream), n, *args, n_rows, 1, pos.data_ptr(),
                                        weight.data_ptr())
        self._done(status, "g4_kv4_account", stream, (slots, start, counts))
        return pos, weight

    def attend(self, q, slots, lens, q_lens=None, scale=0.0, window=0, accumulate=False, out=None, stream=None):
        """Attention of q [n, q_len, num_q_heads, head_dim] over rows 0 .. lens[i] - 1 of slots[i], the
        query tokens being the newest rows.  Returns out: the given tensor, whose rows at and beyond
        q_lens[i] stay as they were, or a new one, where they are zeros."""
        n, q_len = slots.numel(), q.shape[1] if q.dim() == 4 else -1
        shape = (n, q_len, self.num_q_heads, self.head_dim)
        self._dense("q", q, shape, self._ta)
        window = _kv4_int("window", window)
        args = (self._seq("slots", slots, n), self._seq("lens", lens, n), q_len, self._seq("q_lens", q_lens, n))
        given = out is not None
        if given:
            self._dense("out", out, shape, self._tb)
        else:
            out = self._empty(shape, q.dtype, stream)
            self._fresh(out, self._ta.dtype, q_len, self.num_q_heads, self._tb)
        status = _g4.lib.g4_kv4_attend(self.h, self._stream(stream), n, *args, scale, window, bool(accumulate),
                                       not given, self._pa, self._pb)
        self._done(status, "g4_kv4_attend", stream, (q, out, slots, lens, q_lens))
        return out

    def evict(self, slots, lens, budget, recent=0, stream=None):
        """Keep `budget` rows of every slot (see g4_kv4_evict); returns the new lens."""
        n, budget, recent = slots.numel(), _kv4_int("budget", budget), _kv4_int("recent", recent)
        args = (self._seq("slots", slots, n), self._seq("lens", lens, n))
        new = self._empty((n,), torch.int32, stream)
        status = _g4.lib.g4_kv4_evict(self.h, self._stream(stream), n, *args, budget, recent, new.data_ptr())
        self._done(status, "g4_kv4_evict", stream, (slots, lens))
        return new

    def device_error(self, stream=None):
        """(status, word) of the sticky device error word, cleared."""
        w = ctypes.c_int32(0)
        return _g4.lib.g4_kv4_get_device_error(self.h, self._stream(stream), ctypes.byref(w)), w.value

    def device_bytes(self):
        return _g4.lib.g4_kv4_bytes(self.h)

    def close(self):
        if getattr(self, "h", None) is not None:
            _g4.lib.g4_kv4_free(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
