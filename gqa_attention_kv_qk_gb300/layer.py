"""DecodeLayer: one attention layer's KV cache and workspace on a CUDA device.

PyTorch allocates the device memory and supplies the stream; every step of the
method runs in libuaa through the C ABI (binding.py). This is the call a user
makes: build the layer, load or grow its cache, then `step(q, k_new, v_new)`.
"""
from __future__ import annotations

import contextlib

import torch

from . import binding as B
from . import workloads as W

_TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _require_cuda(device):
    if not torch.cuda.is_available():
        raise RuntimeError("DecodeLayer needs a CUDA device; libuaa has no CPU implementation")
    d = torch.device(device)
    return d if d.index is not None or d.type != "cuda" else torch.device("cuda", torch.cuda.current_device())


def _memory_of(stream, index):
    """The context in which new tensors take memory that is in order with `stream` (a
    stream object or a raw handle of device `index`; None: the current one). Memory of
    the current stream may have work pending there that another stream does not wait
    for, and goes back to it while the other's is."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(handle, index) if handle else torch.cuda.default_stream(index)
    return torch.cuda.stream(stream)


class DecodeLayer:
    """page_size: store the caches as pools of pages of that many positions;
    block_table ([batch][capacity / page_size] int32, default: sequence b takes
    pages b P .. b P + P - 1) maps each sequence's logical pages to pool pages, of
    which there are n_pages (default: just enough). max_q_len: the most tokens per
    sequence one step takes (q, k_new, v_new of shape [B][T][H][D]); the
    workspace is sized for it. cache: the caller's own tensors for some of k_cache,
    v_cache, k_scale, v_scale and seq_lens (a pool shared with other layers, a cache
    filled before), used in place instead of new ones. workspace: a uint8 tensor of
    B.uaa_workspace_size bytes and more, zeroed once, or another layer's ws_tensor:
    layers whose steps run one after another share one (prefill chunks over a 4-bit
    cache take up to 512 MiB of it, or the widened rows of one sequence)."""

    def __init__(self, cfg: dict, batch: int, capacity: int, device="cuda", page_size=None, block_table=None,
                 n_pages=None, max_q_len=1, cache=None, workspace=None):
        self.cfg = dict(cfg)
        self.device = _require_cuda(device)
        self._index = self.device.index
        self.batch = int(batch)
        self.capacity = int(capacity)
        self.desc = B.make_desc(cfg)
        Hq, Hkv, D = cfg["n_q_heads"], cfg["n_kv_heads"], cfg["head_dim"]
        kv = cfg.get("kv_dtype", "bf16")
        dev = self.device
        self.page_size = int(page_size or 0)
        if self.page_size:
            if capacity % self.page_size:
                raise ValueError(f"capacity {capacity} is not a multiple of page_size {self.page_size}")
            self.pages_per_seq = capacity // self.page_size
            if block_table is None:
                block_table = torch.arange(batch * self.pages_per_seq, dtype=torch.int32).reshape(batch, -1)
            self.block_table = torch.as_tensor(block_table, dtype=torch.int32).to(dev).contiguous()
            assert self.block_table.shape == (batch, self.pages_per_seq)
            self.n_pages = int(n_pages or batch * self.pages_per_seq)
            rows = (self.n_pages, Hkv, self.page_size)  # pools of pages
        else:
            self.pages_per_seq = self.n_pages = 0
            self.block_table = None
            rows = (batch, Hkv, capacity)
        cache = dict(cache or {})

        def tensor(name, shape, dtype):
            t = cache.pop(name, None)
            if t is None:
                return torch.zeros(shape, dtype=dtype, device=dev)
            if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous() or t.device != dev:
                raise ValueError(f"cache[{name!r}] is {tuple(t.shape)} {t.dtype} on {t.device}, the layer needs a "
                                 f"contiguous {tuple(shape)} {dtype} on its device")
            return t

        row_of = {"f32": (D, torch.float32), "bf16": (D, torch.bfloat16), "q8": (D, torch.int8),
                  "q4": (D // 2, torch.uint8)}
        for which in ("k", "v"):
            kind = ("bf16" if which == "k" else "q8") if kv == "vq8" else kv
            width, dt = row_of[kind]
            setattr(self, which + "_cache", tensor(which + "_cache", (*rows, width), dt))
            scale = {"q8": (rows, torch.float32), "q4": ((*rows, D // 32), torch.float16)}.get(kind)
            setattr(self, which + "_scale", tensor(which + "_scale", *scale) if scale else None)
        given = cache.get("seq_lens") is not None
        self.seq_lens = tensor("seq_lens", (batch,), torch.int32)
        if any(t is not None for t in cache.values()):
            raise ValueError(f"a {kv} layer has no cache tensor named {sorted(cache)}")
        self.max_len_hint = max(0, int(self.seq_lens.max())) if given and batch else 0
        self._args_cache = {}
        self._read_args = None
        self._reads = {}            # read_rows' tensors per row count
        self.out = torch.empty((batch, Hq, D), dtype=_TORCH_DTYPE[cfg.get("out_dtype", "f32")], device=dev)
        self._outs = {1: self.out}  # per tokens-per-step count: [B][Hq][D], or [B][T][Hq][D]
        self.q_len = 1              # tokens per sequence of the current step
        self.max_q_len = int(max_q_len)
        self.q_norm_w = self.k_norm_w = self.sink = None
        # workspace sized for the longest allowed sequence; zeroed once (status word)
        nbytes = B.uaa_workspace_size(self.desc, batch, capacity - 1, 0, self.max_q_len)
        if nbytes == 0:
            raise B.UaaError(B.UAA_ERR_UNSUPPORTED, B.last_error())
        w = torch.zeros((nbytes,), dtype=torch.uint8, device=dev) if workspace is None else workspace
        if w.dtype != torch.uint8 or w.dim() != 1 or not w.is_contiguous() or w.device != dev or w.numel() < nbytes:
            raise ValueError(f"workspace is {tuple(w.shape)} {w.dtype} on {w.device}, the layer needs {nbytes} "
                             f"contiguous bytes (uint8) on its device")
        self.ws_tensor = w
        self.ws = B.UaaWorkspace(w.data_ptr(), w.numel())

    @classmethod
    def for_case(cls, case: dict, device="cuda") -> "DecodeLayer":
        """A layer holding a host case of workloads.host_case (a vq8 / q8 cache is
        quantised on the device); a paged workload gets a pool with spare pages,
        assigned in seeded random order."""
        cfg = case["cfg"]
        ps = int(cfg.get("page_size", 0) or 0)
        T = int(cfg.get("q_len", 1) or 1)
        if ps:
            P = case["cap"] // ps
            n_pages = cfg["batch"] * P + max(2, cfg["batch"])
            layer = cls(cfg, cfg["batch"], case["cap"], device, page_size=ps,
                        block_table=W.block_table(cfg, P, n_pages), n_pages=n_pages, max_q_len=T)
        else:
            layer = cls(cfg, cfg["batch"], case["cap"], device, max_q_len=T)
        k = case["k_values"] if cfg.get("kv_dtype") in ("q8", "q4") else case["k_cache"]
        v = case["v_values"] if cfg.get("kv_dtype") in ("vq8", "q8", "q4") else case["v_cache"]
        layer.load_cache(k, v, case["lens"])
        layer.set_params(case["q_norm_w"], case["k_norm_w"], case["sink"])
        return layer

    # ------------------------------------------------------------ state
    def set_params(self, q_norm_w=None, k_norm_w=None, sink=None):
        D, Hq = self.cfg["head_dim"], self.cfg["n_q_heads"]
        for name, t, n in (("q_norm_w", q_norm_w, D), ("k_norm_w", k_norm_w, D), ("sink", sink, Hq)):
            if t is not None and t.numel() != n:
                raise ValueError(f"{name} has {t.numel()} values, the layer needs {n}")
        to = lambda t: None if t is None else t.to(device=self.device, dtype=torch.float32).contiguous()
        self.q_norm_w, self.k_norm_w, self.sink = to(q_norm_w), to(k_norm_w), to(sink)
        self._args_cache.clear()  # they hold the addresses of the ones before

    def _entries(self):
        """The block table's entries as one index per logical page, and which of them
        name a page (a trimmed, ended or fresh row holds -1)."""
        e = self.block_table.reshape(-1).long()
        return e, (e >= 0) & (e < self.n_pages)

    def _to_pool(self, logical, pool):
        """Logical rows [B][Hkv][cap][...] into a pool [n_pages][Hkv][page_size][...]; rows
        of absent pages go nowhere."""
        Bn, Hkv, ps, P = self.batch, logical.shape[1], self.page_size, self.pages_per_seq
        rest = tuple(logical.shape[3:])
        x = logical.reshape(Bn, Hkv, P, ps, *rest).transpose(1, 2).reshape(Bn * P, Hkv, ps, *rest)
        e, held = self._entries()
        pool.index_copy_(0, e[held], x.to(device=pool.device, dtype=pool.dtype)[held])

    def logical(self, name: str):
        """A cache tensor ("k_cache", "v_cache", "k_scale", "v_scale") as logical
        rows [B][Hkv][cap][...] (a gathered copy for a paged layer, zeros where the
        table has no page)."""
        t = getattr(self, name)
        if t is None or not self.page_size:
            return t
        Bn, P, ps = self.batch, self.pages_per_seq, self.page_size
        e, held = self._entries()
        x = t.index_select(0, e.masked_fill(~held, 0))
        x.masked_fill_(~held.reshape(-1, *[1] * (x.dim() - 1)), 0)
        Hkv, rest = x.shape[1], tuple(x.shape[3:])
        return x.reshape(Bn, P, Hkv, ps, *rest).transpose(1, 2).reshape(Bn, Hkv, P * ps, *rest)

    def load_cache(self, k, v, lens):
        """Copy host caches (logical rows [B][Hkv][cap][D]) in; rows on pages that a paged
        layer's table does not hold are left out. For a vq8 layer `v`
        holds fp32 values, and for a q8 or q4 layer `k` too, quantised on the device by
        uaa_vq8_quantize or uaa_q4_quantize (the append's own rules)."""
        D = self.cfg["head_dim"]
        s = B.call_stream(None, self._index)

        def put(vals, cache, scales):
            if scales is not None:  # codes and scales of the logical rows, then into place
                vals = vals.to(device=self.device, dtype=torch.float32).contiguous()
                codes = torch.empty((*vals.shape[:-1], cache.shape[-1]), dtype=cache.dtype, device=self.device)
                sc = torch.empty((*vals.shape[:-1], *scales.shape[3:]), dtype=scales.dtype, device=self.device)
                quantize = B.uaa_q4_quantize if cache.dtype == torch.uint8 else B.uaa_vq8_quantize
                quantize(vals.data_ptr(), B.DTYPE["f32"], vals.numel() // D, D, codes.data_ptr(), sc.data_ptr(), s)
                pairs = ((codes, cache), (sc, scales))
            else:
                pairs = ((vals, cache),)
            for src, dst in pairs:
                if self.page_size:
                    self._to_pool(src.to(self.device), dst)
                else:
                    dst.copy_(src)

        put(k, self.k_cache, self.k_scale)
        put(v, self.v_cache, self.v_scale)
        lens = torch.as_tensor(lens, dtype=torch.int32)
        self.seq_lens.copy_(lens)
        self.max_len_hint = max(0, int(lens.max())) if lens.numel() else 0

    def set_lengths(self, lens):
        lens = torch.as_tensor(lens, dtype=torch.int32)
        self.seq_lens.copy_(lens)
        self.max_len_hint = max(0, int(lens.max())) if lens.numel() else 0

    # ------------------------------------------------------------ calls
    def out_for(self, q_len: int, stream=None):
        """The layer's output rows for steps of q_len tokens per sequence (made for the
        given stream if there are none yet)."""
        o = self._outs.get(q_len)
        if o is None:
            with _memory_of(stream, self._index):
                o = self._outs[q_len] = torch.empty((self.batch, q_len, *self.out.shape[1:]), dtype=self.out.dtype,
                                                    device=self.device)
        return o

    def _begin(self, q, stream=None):
        """Tokens per sequence of a step's q ([B][Hq][D] or [B][T][Hq][D]); the step runs on `stream`."""
        T = int(q.shape[1]) if q.dim() == 4 else 1
        if T > self.max_q_len:
            raise ValueError(f"{T} tokens per sequence, the layer was built for max_q_len={self.max_q_len}")
        self.q_len = T
        if T not in self._outs:
            self.out_for(T, stream)
        return T

    def _bound(self, T, stream=None):
        """The bound on the lengths before a step of T tokens. max_len_hint grows with every
        step and knows nothing of rows that ended or went back to a shorter parent:
        where the capacity would end by it, the lengths themselves are read (which waits
        for the stream; not in a capture)."""
        if self.max_len_hint + T > self.capacity and self.batch:
            with _memory_of(stream, self._index):
                if not torch.cuda.is_current_stream_capturing():
                    self.max_len_hint = max(0, int(self.seq_lens.max()))
        return self.max_len_hint

    def args(self, q, k_new, v_new, max_seq_len=None, q_rot=None, out=None) -> B.UaaStepArgs:
        """The step's argument struct (a copy of one built once per distinct set of pointers)."""
        msl = self.max_len_hint if max_seq_len is None else int(max_seq_len)
        if out is None:
            out = self.out_for(self.q_len)
        # a copy: callers may change fields
        return B.UaaStepArgs.from_buffer_copy(self._args(q, k_new, v_new, msl, q_rot, out))

    def _args(self, q, k_new, v_new, msl, q_rot, out) -> B.UaaStepArgs:
        # what _build_args checks is part of the key: another tensor may come to lie there
        key = (msl, self.q_len,
               None if out is self._outs.get(self.q_len) else (out.data_ptr(), out.dtype, out.numel(), out.is_contiguous()),
               None if q is None else (q.data_ptr(), q.dtype, q.numel(), q.is_contiguous(),
                                       k_new.data_ptr(), k_new.dtype, k_new.numel(), k_new.is_contiguous(),
                                       v_new.data_ptr(), v_new.dtype, v_new.numel(), v_new.is_contiguous()),
               None if q_rot is None else (q_rot.data_ptr(), q_rot.dtype, q_rot.numel(), q_rot.is_contiguous()))
        a = self._args_cache.get(key)
        if a is None:
            if len(self._args_cache) > 64:
                self._args_cache.clear()
            a = self._args_cache[key] = self._build_args(q, k_new, v_new, msl, q_rot, out)
        return a

    def _build_args(self, q, k_new, v_new, max_seq_len, q_rot, out) -> B.UaaStepArgs:
        c = self.cfg
        io = _TORCH_DTYPE[c.get("io_dtype", "bf16")]
        for name, t, heads, dt in (("q", q, c["n_q_heads"], io), ("k_new", k_new, c["n_kv_heads"], io),
                                   ("v_new", v_new, c["n_kv_heads"], io),
                                   ("q_rot", q_rot, c["n_q_heads"], torch.float32),
                                   ("out", out, c["n_q_heads"], self.out.dtype)):
            if t is None:
                continue
            n = self.batch * self.q_len * heads * c["head_dim"]
            if t.dtype != dt or t.numel() != n or not t.is_contiguous() or t.get_device() != self._index:
                raise ValueError(f"{name} is {tuple(t.shape)} {t.dtype} on {t.device}, strides {tuple(t.stride())}; a step of "
                                 f"{self.q_len} token(s) needs {n} contiguous {dt} values on cuda:{self._index}")
        a = B.UaaStepArgs()
        a.batch = self.batch
        a.q, a.k_new, a.v_new = B.ptr(q), B.ptr(k_new), B.ptr(v_new)
        a.q_norm_w, a.k_norm_w, a.sink = B.ptr(self.q_norm_w), B.ptr(self.k_norm_w), B.ptr(self.sink)
        a.k_cache, a.v_cache, a.v_scale = B.ptr(self.k_cache), B.ptr(self.v_cache), B.ptr(self.v_scale)
        a.cache_capacity = self.capacity
        a.seq_lens = B.ptr(self.seq_lens)
        a.max_seq_len = max_seq_len
        a.out = B.ptr(self.out if out is None else out)
        a.q_rot = B.ptr(q_rot)
        a.k_scale = B.ptr(self.k_scale)
        a.q_len = self.q_len
        if self.page_size:
            a.block_table = B.ptr(self.block_table)
            a.page_size, a.pages_per_seq, a.n_pages = self.page_size, self.pages_per_seq, self.n_pages
        return a

    def step(self, q, k_new, v_new, stream=None, max_seq_len=None, advance_hint=True, q_rot=None, out=None):
        """One step (append, split-K partials, combine) on `stream` for q of one token
        per sequence ([B][Hq][D]) or T tokens ([B][T][Hq][D], causal within the
        chunk); the output rows ([B][Hq][D] or [B][T][Hq][D]) go to `out` if given.
        max_seq_len: a bound on the lengths before the step, for a capture or where the
        caller knows one (default: the layer's own, read from the device when the
        capacity would end by it)."""
        s = B.call_stream(stream, self._index)
        T = self._begin(q, stream)
        want = self._outs[T]
        if out is not None:
            assert out.shape == want.shape and out.dtype == want.dtype and out.is_contiguous()
        msl = self._bound(T, stream) if max_seq_len is None else int(max_seq_len)
        B.uaa_decode_attn(self.desc, self._args(q, k_new, v_new, msl, q_rot, want if out is None else out), self.ws, s)
        if advance_hint and max_seq_len is None:
            self.max_len_hint += T
        return want if out is None else out

    def read_rows(self, start, n, stream=None):
        """The cached keys and values of positions start[b] .. start[b] + n - 1 of every
        sequence (start: int32 tensor [B] on the device, or None for 0), as
        [B][n][Hkv][D] tensors in the layer's out dtype; any cache kind, paged or not.
        Positions outside the cache, or on absent pages, read as zeros. The tensors are
        the layer's own (a pair for each of the first 16 values of n; new ones for
        others), overwritten by the next read of n rows, as a step's output is by the
        next step; work on another stream than the read's waits for it, and keeps them
        (record_stream) for as long as it uses them."""
        s = B.call_stream(stream, self._index)
        if start is not None and (start.dtype is not torch.int32 or start.shape != self.seq_lens.shape
                                  or start.get_device() != self._index or not start.is_contiguous()):
            raise ValueError("start is not a contiguous int32 tensor [batch] on the device")
        got = self._reads.get(n)
        if got is None:
            shape = (self.batch, int(n), self.cfg["n_kv_heads"], self.cfg["head_dim"])
            with _memory_of(stream, self._index):
                got = tuple(torch.empty(shape, dtype=self.out.dtype, device=self.device) for _ in "kv")
            if len(self._reads) < 16:  # kept for good: a captured graph may write them
                self._reads[n] = got
        if self._read_args is None:
            self._read_args = self._build_args(None, None, None, 0, None, None)
        B.uaa_cache_read(self.desc, self._read_args, B.ptr(start), int(n), B.ptr(got[0]), B.ptr(got[1]), s)
        return got

    def append(self, q, k_new, v_new, stream=None, q_rot=None):
        s = B.call_stream(stream, self._index)
        self._bound(self._begin(q, stream), stream)
        B.uaa_rope_qk_norm_append(self.desc, self.args(q, k_new, v_new, q_rot=q_rot), self.ws, s)

    def append_partial(self, q, k_new, v_new, stream=None, q_rot=None):
        """Steps 1 and 2 (one fused kernel for bf16 / vq8 / q8 caches and one token);
        follow with combine()."""
        s = B.call_stream(stream, self._index)
        self._bound(self._begin(q, stream), stream)
        B.uaa_decode_attn_append_partial(self.desc, self.args(q, k_new, v_new, q_rot=q_rot), self.ws, s)

    def partial(self, stream=None):
        s = B.call_stream(stream, self._index)
        B.uaa_decode_attn_partial(self.desc, self.args(None, None, None), self.ws, s)

    def combine(self, stream=None):
        s = B.call_stream(stream, self._index)
        B.uaa_decode_attn_combine(self.desc, self.args(None, None, None), self.ws, s)
        self.max_len_hint += self.q_len
        return self.out_for(self.q_len)

    def layout(self, max_seq_len=None) -> B.UaaWorkspaceLayout:
        return B.uaa_get_workspace_layout(self.desc, self.batch,
                                          self.max_len_hint if max_seq_len is None else max_seq_len, 0, self.q_len)

    def device_status(self, stream=None) -> int:
        s = B.call_stream(stream, self._index)
        return B.uaa_device_status(self.ws, s)
