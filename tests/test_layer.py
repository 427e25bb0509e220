"""DecodeLayer around the step: reading and filling caches whose table has absent
pages, reads on another stream than the current one, length bounds of a loop."""
import pytest
import torch

from gqa_attention_kv_qk_gb300 import binding as B
from gqa_attention_kv_qk_gb300 import workloads as W


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gqa_attention_kv_qk_gb300 import build
    build.build()


def config(**kw):
    cfg = dict(n_q_heads=4, n_kv_heads=2, head_dim=64, kv_dtype="bf16", io_dtype="bf16", out_dtype="f32",
               rope_style="neox", rope_theta=10000.0, seed=51, batch=1, seq_len=64)
    cfg.update(kw)
    return cfg


# ---------------------------------------------------------------- tables with holes

def paged_stub(table, pool, page_size):
    """A paged layer's tensors on the host: what logical() and _to_pool() work on."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    layer = DecodeLayer.__new__(DecodeLayer)
    layer.block_table = torch.tensor(table, dtype=torch.int32)
    layer.batch, layer.pages_per_seq = layer.block_table.shape
    layer.page_size, layer.n_pages, layer.k_cache = page_size, pool.shape[0], pool
    return layer


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.uint8, torch.float16])
def test_absent_pages_on_the_host(dtype):
    """Entries of -1 (trimmed, ended, never given) and past the pool read as zeros and
    take no rows."""
    table = [[2, -1, 0], [-1, -1, -1], [5, 1, 6], [3, -2, 4]]  # 6 pages: entry 6 is none either
    pool = torch.randint(1, 100, (6, 2, 16, 8), generator=torch.Generator().manual_seed(1)).to(dtype)
    layer = paged_stub(table, pool.clone(), 16)
    got = layer.logical("k_cache")
    assert got.shape == (4, 2, 48, 8)
    for b, row in enumerate(table):
        for l, e in enumerate(row):
            want = pool[e] if 0 <= e < 6 else torch.zeros_like(pool[0])
            assert torch.equal(got[b, :, 16 * l:16 * l + 16], want)
    new = torch.randint(1, 100, (4, 2, 48, 8), generator=torch.Generator().manual_seed(2)).to(dtype)
    layer._to_pool(new, layer.k_cache)
    for b, row in enumerate(table):
        for l, e in enumerate(row):
            if 0 <= e < 6:
                assert torch.equal(layer.k_cache[e], new[b, :, 16 * l:16 * l + 16])


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["f32", "bf16", "vq8", "q8", "q4"])
def test_absent_pages(kv):
    """load_cache and logical() of a layer on a table with holes, against the reader."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    from tests import plain64
    cfg = config(kv_dtype=kv, io_dtype="f32" if kv == "f32" else "bf16", batch=3, seq_len=100, page_size=32)
    case = W.host_case(cfg, lens=[100, 7, 64])
    cap = case["cap"]
    table = torch.tensor([[3, -1, 5, 0] + [-1] * (cap // 32 - 4), [-1] * (cap // 32), [1, 2] + [-1] * (cap // 32 - 2)])
    layer = DecodeLayer(cfg, 3, cap, page_size=32, block_table=table, n_pages=6)
    k = case["k_values"] if kv in ("q8", "q4") else case["k_cache"]
    v = case["v_values"] if kv in ("vq8", "q8", "q4") else case["v_cache"]
    layer.load_cache(k, v, case["lens"])
    rows = layer.read_rows(None, cap)
    for got, x in zip(plain64.cached_values(layer), rows):
        assert ((got - x.transpose(1, 2).double().cpu()).abs() <= got.abs() * 2.0 ** -24).all()
        held = (table >= 0).repeat_interleave(32, 1)
        assert not got.transpose(1, 2)[~held].any() and bool(got.transpose(1, 2)[held][:64].any())
    full = DecodeLayer.for_case(case)  # the same rows with every page there
    for a, b in zip(plain64.cached_values(layer), plain64.cached_values(full)):
        assert torch.equal(a.transpose(1, 2)[held], b.transpose(1, 2)[held])
    assert layer.device_status() == 0


# ---------------------------------------------------------------- other streams

def test_new_tensors_belong_to_the_stream_that_writes_them(monkeypatch):
    """The tensors that a read or a step makes on first use are allocated in the context
    of the stream it was given: memory of the current stream may have work pending that
    the other does not wait for, and returns to it under the other's pending writes."""
    import contextlib

    from gqa_attention_kv_qk_gb300 import layer as L
    active, made = [], []

    @contextlib.contextmanager
    def entered(stream):
        active.append(stream)
        yield
        active.pop()

    empty = torch.empty

    def recorded(*shape, **kw):
        made.append(active[-1] if active else None)
        return empty(*shape, **kw)

    class Stream:
        cuda_stream = 0x1234

    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, index: (handle, index))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda index: ("default", index))
    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(B, "uaa_cache_read", lambda *a, **k: 0)
    monkeypatch.setattr(B, "uaa_decode_attn", lambda *a, **k: 0)
    monkeypatch.setattr(B, "call_stream", lambda stream, index: stream or 7)
    layer = L.DecodeLayer.__new__(L.DecodeLayer)
    layer.cfg, layer.batch, layer.max_q_len, layer._index, layer.device = config(), 1, 4, 0, torch.device("cpu")
    layer.out, layer._reads, layer._read_args, layer.seq_lens = empty(1, 4, 64), {}, object(), torch.zeros(1)
    layer.desc = layer.ws = None
    layer._outs, layer.max_len_hint, layer._args = {1: layer.out}, 0, lambda *a: None
    for n, stream, want in ((1, Stream(), (0x1234, 0)), (2, None, None), (3, 0x77, (0x77, 0)), (4, 0, ("default", 0))):
        layer.read_rows(None, n, stream=stream)
        assert made == [want, want], n
        made.clear()
        if n > 1:
            layer.step(torch.zeros(1, n, 4, 64), None, None, stream=stream, max_seq_len=5)
            assert made == [want], n
            made.clear()
    layer.read_rows(None, 3, stream=Stream())  # kept: no new ones
    assert not made


@pytest.mark.gpu
def test_reads_on_another_stream():
    """A read that is pending on a side stream owns its tensors: their memory is not
    handed out on the current stream meanwhile, and was not taken from under work
    pending there."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    layer = DecodeLayer.for_case(W.host_case(config(batch=2, seq_len=200), lens=[200, 150]))
    want = {n: [x.clone() for x in layer.read_rows(None, n)] for n in range(1, 60)}  # the first 16 counts are kept
    torch.cuda.synchronize()
    side, wait = torch.cuda.Stream(), 100_000_000  # about 50 ms
    for n in (40, 41, 42):
        with torch.cuda.stream(side):
            torch.cuda._sleep(wait)
        got = layer.read_rows(None, n, stream=side)
        shape, dtype = got[0].shape, got[0].dtype
        del got
        mine = [torch.full(shape, 7.0, dtype=dtype, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert all(bool((x == 7.0).all()) for x in mine)
        del mine
    for n in (50, 51, 52):
        old = [torch.empty(want[n][0].shape, device="cuda") for _ in range(4)]
        torch.cuda._sleep(wait)
        for x in old:
            x.fill_(9.0)
        del old, x
        got = layer.read_rows(None, n, stream=side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[n]))


# ---------------------------------------------------------------- length bounds

def test_length_bound_on_the_host(monkeypatch):
    """The bound that a step passes on: it grows by the step's tokens, and where the
    capacity would end by it, it is the lengths' own largest again."""
    from gqa_attention_kv_qk_gb300 import layer as L
    passed, capturing = [], [False]
    monkeypatch.setattr(B, "uaa_decode_attn", lambda *a, **k: 0)
    monkeypatch.setattr(B, "uaa_rope_qk_norm_append", lambda *a, **k: 0)
    monkeypatch.setattr(B, "call_stream", lambda stream, index: stream or 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    layer = L.DecodeLayer.__new__(L.DecodeLayer)
    layer.batch, layer.capacity, layer.max_q_len, layer._index, layer.device = 2, 64, 7, 0, torch.device("cpu")
    layer.out = torch.empty(2, 4, 64)
    layer._outs, layer.max_len_hint, layer.desc, layer.ws, layer.q_len = {1: layer.out}, 0, None, None, 1
    layer._args = lambda q, k, v, msl, q_rot, out: passed.append(msl)
    layer.args = lambda q, k, v, q_rot=None: passed.append(layer.max_len_hint)
    q = torch.zeros(2, 7, 4, 64)
    for i in range(40):  # rows that start over every third step
        layer.seq_lens = torch.tensor([i % 3 * 7, 0], dtype=torch.int32)
        layer.step(q, None, None)
        assert layer.seq_lens[0] <= passed[-1] <= 64 - 7
    assert passed[:9] == [7 * i for i in range(9)] and passed[9] == 0
    layer.max_len_hint = 60
    layer.append(q, None, None)
    assert passed[-1] == layer.seq_lens[0]
    layer.seq_lens, layer.max_len_hint = torch.tensor([60, 5], dtype=torch.int32), 63
    layer.step(q, None, None)
    assert passed[-1] == 60                     # full: refused by the call
    layer.seq_lens, layer.max_len_hint = torch.tensor([-1, -1], dtype=torch.int32), 63
    layer.step(q, None, None)
    assert passed[-1] == 0
    layer.max_len_hint, capturing[0] = 63, True
    layer.step(q, None, None)
    assert passed[-1] == 63                     # a capture does not wait


@pytest.mark.gpu
@pytest.mark.parametrize("entry", ["step", "split", "side"])
def test_loop_of_forks_outlives_the_capacity(entry):
    """Rows that end and start over take more steps than one sequence has room for: the
    step's bound on the lengths follows them. A row that is full is still refused.
    (Bar of fp32 outputs of values ~N(0, 1): 2e-3.)"""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    from gqa_attention_kv_qk_gb300.pages import PageTable
    from tests import plain64
    Bn, ps, P, T = 3, 16, 4, 7
    pages = PageTable(torch.full((Bn, P), -1), ps, 16)
    layer = DecodeLayer(config(batch=Bn), Bn, P * ps, page_size=ps, block_table=pages.block_table, n_pages=16,
                        max_q_len=T, cache=dict(seq_lens=pages.seq_lens))
    side = torch.cuda.Stream() if entry == "side" else None
    lens = [0] * Bn
    for i in range(40):
        parents = [-1 if lens[b] + T > P * ps or (i + b) % 5 == 4 else b for b in range(Bn)]
        lens = [n if p >= 0 else 0 for n, p in zip(lens, parents)]
        par = torch.tensor(parents, dtype=torch.int32, device="cuda")
        q, k, v = (torch.randn((Bn, T, h, 64), generator=torch.Generator().manual_seed(10 * i + h)).to(torch.bfloat16).cuda()
                   for h in (4, 2, 2))
        q_rot = torch.empty((Bn, T, 4, 64), device="cuda")
        torch.cuda.synchronize()
        pages.fork(par, stream=side)
        pages.reserve(T, stream=side)
        pages.copy_layer(layer, stream=side)
        if entry == "split":
            layer.append(q, k, v, q_rot=q_rot)
            layer.partial()
            out = layer.combine()
        else:
            out = layer.step(q, k, v, q_rot=q_rot, stream=side)
        torch.cuda.synchronize()
        assert layer.device_status() == 0 and pages.device_status() == 0
        kk, vv = plain64.cached_values(layer)
        want = plain64.attend(q_rot, kk, vv, lens)
        assert float((out.double().cpu() - want).abs().max()) <= 2e-3, i
        lens = [n + T for n in lens]
        assert pages.seq_lens.tolist() == lens
    layer.set_lengths([P * ps - T + 1, 0, 0])
    with pytest.raises(B.UaaError, match="does not fit cache_capacity=64"):
        layer.step(q, k, v)
    with pytest.raises(B.UaaError, match="does not fit cache_capacity=64"):
        layer.append(q, k, v)
    g = torch.cuda.CUDAGraph()  # in a capture the layer's bound stands as it is
    layer.set_lengths([0] * Bn)
    layer.max_len_hint = P * ps
    with pytest.raises(B.UaaError, match="does not fit"):
        with torch.cuda.graph(g):
            layer.step(q, k, v)


# ---------------------------------------------------------------- lengths outside the cache

def step_cases():
    for kv in ("f32", "bf16", "vq8", "q8", "q4"):
        for T in (1, 4, 70):  # one token, a short chunk, 140 rows per kv head
            for page in (0, 32):
                for win, first in ((0, 0), (50, 9)):
                    yield kv, T, page, win, first


def step_pair(kv, T, page, win, first, odd):
    """Two layers alike; in the second one, sequence 1 has the length `odd` (the first one's is 20)."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    lens = [130, 20, 57]
    cfg = config(kv_dtype=kv, io_dtype="f32" if kv == "f32" else "bf16", batch=3, seq_len=130, q_len=T, page_size=page,
                 window=win, first_tokens=first, reproducible=True)
    case = W.host_case(cfg, lens=lens)
    a, b = DecodeLayer.for_case(case), DecodeLayer.for_case(case)
    b.seq_lens[1] = odd
    b.out_for(T).fill_(7.0)
    return a, b, [case[k].cuda() for k in ("q", "k_new", "v_new")]


def compare_pair(a, b, T, odd, run):
    before = [t.clone() for t in (b.k_cache, b.v_cache)]
    want, got = run(a), run(b)
    torch.cuda.synchronize()
    assert a.device_status() == 0
    assert b.seq_lens.tolist() == [130 + T, odd, 57 + T]
    for x, y in ((a.logical("k_cache"), b.logical("k_cache")), (a.logical("v_cache"), b.logical("v_cache"))):
        assert torch.equal(x[::2], y[::2])
    for t, old in zip((b.logical("k_cache"), b.logical("v_cache")), before):
        if not b.page_size:
            assert torch.equal(t[1], old[1])
    # ranges are cut elsewhere: each side's weights are within 2^-11 (one fp16 part) or
    # 2^-16 (two parts) of the exact ones, and values within +-4.5
    eps = 2.0 ** -11 if a.desc.kv_dtype == B.DTYPE["q4"] else 2.0 ** -16
    assert float((got[::2] - want[::2]).abs().max()) <= 9 * eps
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("entry", ["step", "split"])
@pytest.mark.parametrize("odd", [2**31 - 1, 2**31 - 30, -2**31])
def test_lengths_at_the_ends_of_int32(entry, odd):
    """No sum of a length and a step's tokens wraps: such a sequence is not appended and
    the others are as they are alone; with a window it sees nothing."""
    for kv, T, page, win, first in step_cases():
        a, b, x = step_pair(kv, T, page, win, first, odd)

        def run(layer):
            if entry == "step":
                return layer.step(*x, max_seq_len=130, advance_hint=False)
            layer.append(*x)
            layer.partial()
            return layer.combine()

        got = compare_pair(a, b, T, odd, run)
        flags = b.device_status()
        assert odd < 0 or flags & B.UAA_DEVFLAG_CAPACITY, (kv, T, page, win)
        if odd < 0 or win:
            assert not got[1].any(), (kv, T, page, win)


@pytest.mark.gpu
@pytest.mark.parametrize("entry", ["step", "split"])
def test_idle_rows(entry):
    """A row of negative length: not appended, zero output rows, no flag."""
    for kv, T, page, win, first in step_cases():
        a, b, x = step_pair(kv, T, page, win, first, -1)

        def run(layer):
            if entry == "step":
                return layer.step(*x, max_seq_len=130, advance_hint=False)
            layer.append(*x)
            layer.partial()
            return layer.combine()

        got = compare_pair(a, b, T, -1, run)
        assert b.device_status() == 0 and not got[1].any(), (kv, T, page, win)
    b.set_lengths([-1, -1, -1])
    assert b.max_len_hint == 0 and not b.step(*x).any() and b.seq_lens.tolist() == [-1] * 3


# ---------------------------------------------------------------- another current device

def test_calls_of_another_device_are_refused(monkeypatch):
    """The library launches on the current device: a layer or table of another one says so
    before anything is launched, with its own stream or with a given one."""
    from gqa_attention_kv_qk_gb300 import layer as L
    from gqa_attention_kv_qk_gb300 import pages as P
    import gqa_attention_kv_qk_gb300.binding as binding

    def launched(*a, **k):
        raise AssertionError("a launch on the wrong device")

    for name in vars(binding).copy():
        if name.startswith("uaa_"):
            monkeypatch.setattr(binding, name, launched)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_several_devices", True)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 0)
    layer = L.DecodeLayer.__new__(L.DecodeLayer)
    layer.cfg, layer.batch, layer.max_q_len, layer._index, layer.device = config(), 1, 4, 1, torch.device("cuda", 1)
    layer.seq_lens, layer.capacity, layer.max_len_hint, layer.q_len = torch.zeros(1), 64, 0, 1
    layer.out = torch.empty(1, 4, 64)
    layer._outs, layer.args, layer.desc, layer.ws = {1: layer.out}, lambda *a, **k: None, None, None
    layer._reads, layer._read_args, layer._args = {1: (layer.out, layer.out)}, object(), lambda *a: None
    table = P.PageTable.__new__(P.PageTable)
    table._index, table.args, table.ws, table.n_pages = 1, None, None, 4

    class Parents:
        dtype, shape = torch.int32, table.__dict__.setdefault("seq_lens", torch.zeros(1)).shape
        get_device, is_contiguous, data_ptr = (lambda s: 1), (lambda s: True), (lambda s: 0)

    q = torch.zeros(1, 4, 64)
    for stream in (None, 0x77):
        for call in (lambda: layer.step(q, q, q, stream=stream), lambda: layer.append(q, q, q, stream=stream),
                     lambda: layer.append_partial(q, q, q, stream=stream), lambda: layer.partial(stream=stream),
                     lambda: layer.combine(stream=stream), lambda: layer.read_rows(None, 1, stream=stream),
                     lambda: layer.device_status(stream=stream), lambda: table.fork(Parents(), stream=stream),
                     lambda: table.trim(3, stream=stream), lambda: table.reserve(stream=stream),
                     lambda: table.compact(stream=stream), lambda: table.copy(stream=stream),
                     lambda: table.device_status(stream=stream)):
            with pytest.raises(RuntimeError, match="on cuda:1, and the current device is cuda:0"):
                call()
    layer._index = 0
    assert binding.call_stream(None, 0) == 0 and binding.call_stream(0x77, 0) == 0x77


# ---------------------------------------------------------------- tensors of a step

def test_tensors_that_do_not_fit_are_refused(monkeypatch):
    """A step's tensors reach the library as addresses: another type, size, device or
    stride would be read past or as something else."""
    from gqa_attention_kv_qk_gb300 import layer as L
    layer = L.DecodeLayer.__new__(L.DecodeLayer)
    layer.cfg, layer.batch, layer._index, layer.device = config(), 3, -1, torch.device("cpu")
    layer.q_len, layer.page_size, layer.capacity, layer._args_cache = 2, 0, 64, {}
    layer.out, layer._outs = torch.zeros(3, 4, 64), {}
    layer.q_norm_w = layer.k_norm_w = layer.sink = layer.k_scale = layer.v_scale = None
    layer.k_cache = layer.v_cache = layer.seq_lens = torch.zeros(4)
    bf, f4 = torch.bfloat16, torch.float32
    ok = dict(q=torch.zeros(3, 2, 4, 64, dtype=bf), k_new=torch.zeros(3, 2, 2, 64, dtype=bf),
              v_new=torch.zeros(3, 2, 2, 64, dtype=bf), q_rot=torch.zeros(3, 2, 4, 64), out=torch.zeros(3, 2, 4, 64))

    def build(**kw):
        x = {**ok, **kw}
        return layer._args(x["q"], x["k_new"], x["v_new"], 5, x["q_rot"], x["out"])

    assert build().q == ok["q"].data_ptr() and build(q_rot=None).q_rot in (None, 0)
    qkv = torch.zeros(3, 2, 8 * 64, dtype=bf)                        # a fused projection's output
    for name, bad in (("q", qkv[..., :256].unflatten(-1, (4, 64))), ("k_new", qkv[..., 256:384]), ("q", ok["q"].to(f4)),
                      ("q", ok["q"][:, :1]), ("v_new", ok["q"]), ("k_new", ok["k_new"].to(torch.float16)),
                      ("q_rot", ok["q_rot"].to(bf)), ("out", ok["out"].to(bf)), ("out", ok["out"][:2])):
        with pytest.raises(ValueError, match=f"^{name} is"):
            build(**{name: bad})
    layer._index = 0                                                 # of the device: these are the host's
    layer._args_cache.clear()
    with pytest.raises(ValueError, match="^q is .* on cuda:0"):
        build()
    for name, n in (("q_norm_w", 64), ("k_norm_w", 64), ("sink", 4)):
        layer.set_params(**{name: torch.ones(n)})
        with pytest.raises(ValueError, match=f"{name} has {n + 1} values, the layer needs {n}"):
            layer.set_params(**{name: torch.ones(n + 1)})
