"""The pages of a paged cache (fork, trim, reserve, compact, copy) against a plain
sequential model of them, on random tables; and a run of them together with the
step."""
import random

import pytest
import torch

from gqa_attention_kv_qk_gb300 import binding as B
from gqa_attention_kv_qk_gb300 import workloads as W
from tests import plain64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gqa_attention_kv_qk_gb300 import build
    build.build()


# ---------------------------------------------------------------- on the host

WS = B.UaaWorkspace(0x20000, 1 << 30)


def page_args(**kw):
    a = B.UaaPageArgs()
    a.batch, a.page_size, a.pages_per_seq, a.n_pages = 2, 32, 4, 16
    for f in ("block_table", "seq_lens", "page_refs", "moves", "counts"):
        setattr(a, f, 0x10000)  # aligned, never dereferenced
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status,fact", [
    (dict(batch=-1), B.UAA_ERR_INVALID_ARGUMENT, "batch=-1"),
    (dict(page_size=24), B.UAA_ERR_UNSUPPORTED, "page_size=24"),
    (dict(page_size=8192), B.UAA_ERR_UNSUPPORTED, "page_size=8192"),
    (dict(pages_per_seq=0), B.UAA_ERR_INVALID_ARGUMENT, "pages_per_seq=0"),
    (dict(n_pages=0), B.UAA_ERR_INVALID_ARGUMENT, "n_pages=0"),
    (dict(n_pages=2**30 + 1), B.UAA_ERR_UNSUPPORTED, "n_pages=1073741825"),
    (dict(pages_per_seq=2**29, batch=1), B.UAA_ERR_UNSUPPORTED, "exceeds 2^31 positions"),
    (dict(block_table=None), B.UAA_ERR_INVALID_ARGUMENT, "block_table is NULL"),
    (dict(seq_lens=0x10004), B.UAA_ERR_INVALID_ARGUMENT, "seq_lens is not 16-byte aligned"),
    (dict(page_refs=None), B.UAA_ERR_INVALID_ARGUMENT, "page_refs is NULL"),
    (dict(moves=None), B.UAA_ERR_INVALID_ARGUMENT, "moves is NULL"),
    (dict(counts=None), B.UAA_ERR_INVALID_ARGUMENT, "counts is NULL"),
])
def test_argument_refusals(kw, status, fact):
    a = page_args(**kw)
    big = B.UaaWorkspace(0x20000, 1 << 40)
    for call in (lambda: B.uaa_pages_fork(a, 0x10000, big, None, check=False),
                 lambda: B.uaa_pages_trim(a, 4, 0, big, None, check=False),
                 lambda: B.uaa_pages_reserve(a, 1, big, None, check=False),
                 lambda: B.uaa_pages_compact(a, big, None, check=False),
                 lambda: B.uaa_pages_copy(a, [0x10000], [512], big, None, check=False)):
        assert call() == status
        assert fact in B.last_error()


def test_call_refusals():
    a = page_args()
    small = B.UaaWorkspace(0x20000, B.uaa_pages_workspace_size(2, 4, 16) - 1)
    assert B.uaa_pages_compact(a, small, None, check=False) == B.UAA_ERR_INVALID_ARGUMENT
    assert "workspace has" in B.last_error()
    for call, status, fact in (
            (lambda: B.uaa_pages_fork(a, 0, WS, None, check=False), B.UAA_ERR_INVALID_ARGUMENT, "parents is NULL"),
            (lambda: B.uaa_pages_fork(a, 0x10002, WS, None, check=False), B.UAA_ERR_INVALID_ARGUMENT, "aligned"),
            (lambda: B.uaa_pages_trim(a, 0, 0, WS, None, check=False), B.UAA_ERR_UNSUPPORTED, "window=0"),
            (lambda: B.uaa_pages_trim(a, 5, -1, WS, None, check=False), B.UAA_ERR_UNSUPPORTED, "first_tokens=-1"),
            (lambda: B.uaa_pages_reserve(a, 0, WS, None, check=False), B.UAA_ERR_UNSUPPORTED, "q_len=0"),
            (lambda: B.uaa_pages_reserve(a, 1025, WS, None, check=False), B.UAA_ERR_UNSUPPORTED, "q_len=1025"),
            (lambda: B.uaa_pages_copy(a, [0x10000] * 9, [512] * 9, WS, None, check=False), B.UAA_ERR_UNSUPPORTED,
             "n_pools=9"),
            (lambda: B.uaa_pages_copy(a, [0x10000], [24], WS, None, check=False), B.UAA_ERR_UNSUPPORTED,
             "page_bytes[0]=24"),
            (lambda: B.uaa_pages_copy(a, [0x10008], [32], WS, None, check=False), B.UAA_ERR_INVALID_ARGUMENT,
             "pools[0] is not 16-byte aligned"),
            (lambda: B.uaa_pages_copy(a, [0], [32], WS, None, check=False), B.UAA_ERR_INVALID_ARGUMENT,
             "pools[0] is NULL")):
        assert call() == status
        assert fact in B.last_error()
    assert B.uaa_pages_workspace_size(4, 0, 5) == 0
    assert B.uaa_pages_fork(page_args(batch=0, block_table=None, seq_lens=None), 0, WS, None, check=False) == B.UAA_OK


# ---------------------------------------------------------------- the plain model

class Model:
    """The table one entry at a time, in order."""

    def __init__(self, table, lens, n_pages, page_size):
        self.table, self.lens = [list(r) for r in table], list(lens)
        self.N, self.ps = n_pages, page_size
        self.refs = [0] * n_pages
        for r in self.table:
            for e in r:
                if e >= 0:
                    self.refs[e] += 1
        self.moves = []

    def fork(self, parents):
        old, lens = [list(r) for r in self.table], list(self.lens)
        for b, p in enumerate(parents):
            for e in self.table[b]:
                if e >= 0:
                    self.refs[e] -= 1
            self.table[b] = list(old[p]) if p >= 0 else [-1] * len(old[b])
            self.lens[b] = lens[p] if p >= 0 else 0
            for e in self.table[b]:
                if e >= 0:
                    self.refs[e] += 1

    def trim(self, window, first):
        for b, r in enumerate(self.table):
            for l, e in enumerate(r):
                seen = any(j < first or j > self.lens[b] - window for j in range(l * self.ps, (l + 1) * self.ps))
                if e >= 0 and not seen:
                    r[l] = -1
                    self.refs[e] -= 1

    def reserve(self, q_len):
        """Returns whether the pool had enough."""
        asks = []
        for b, r in enumerate(self.table):
            L = self.lens[b]
            if L + q_len <= len(r) * self.ps:
                asks += [(b, l) for l in range(L // self.ps, (L + q_len - 1) // self.ps + 1)]
        by_page = {}
        for b, l in asks:
            by_page.setdefault(self.table[b][l], []).append((b, l))
        takes = []
        for b, l in asks:
            e = self.table[b][l]
            alone = e >= 0 and (self.refs[e] == 1 or (self.refs[e] == len(by_page[e]) and by_page[e][-1] == (b, l)))
            if not alone:
                takes.append((b, l))
        free = [p for p in range(self.N) if self.refs[p] == 0]
        self.moves = []
        self.takes = len(takes)
        if len(free) < len(takes):
            return False
        for (b, l), page in zip(takes, free):
            e = self.table[b][l]
            if e >= 0:
                self.refs[e] -= 1
                if l * self.ps < self.lens[b]:
                    self.moves.append((e, page))
            self.table[b][l] = page
            self.refs[page] = 1
        return True

    def compact(self):
        live = [p for p in range(self.N) if self.refs[p]]
        n = len(live)
        self.moves = list(zip([p for p in live if p >= n], [p for p in range(n) if not self.refs[p]]))
        to = dict(self.moves)
        self.table = [[to.get(e, e) for e in r] for r in self.table]
        for s, d in self.moves:
            self.refs[d], self.refs[s] = self.refs[s], 0
        return n


def random_state(seed, B_, P, ps, N):
    rng = random.Random(seed)
    free = list(range(N))
    rng.shuffle(free)
    table, lens = [[-1] * P for _ in range(B_)], [0] * B_
    for b in range(B_):
        n = rng.choice([0, 1, rng.randint(0, P * ps), rng.randint(0, P * ps), P * ps])
        need = -(-n // ps)
        if need > len(free) - N // 4:
            n, need = 0, 0
        lens[b] = n
        for l in range(need):
            table[b][l] = free.pop()
    return table, lens, rng


def same(pages, m, moves=True):
    assert pages.block_table.tolist() == m.table
    assert pages.seq_lens.tolist() == m.lens
    assert pages.page_refs.tolist() == m.refs
    if moves:
        n = int(pages.counts[0])
        assert [tuple(x) for x in pages.moves[:n].tolist()] == m.moves
    assert int(pages.ws_tensor[256:].numel()) > 0


def table_of(table, lens, ps, N):
    from gqa_attention_kv_qk_gb300.pages import PageTable
    return PageTable(torch.tensor(table, dtype=torch.int32), ps, N, seq_lens=torch.tensor(lens, dtype=torch.int32))


SHAPES = [(1, 1, 16, 1), (1, 3, 16, 7), (4, 5, 32, 33), (33, 7, 16, 400), (7, 300, 64, 5000), (300, 9, 128, 20000),
          (1100, 4, 16, 40001), (130, 70, 16, 30000), (1200, 3, 16, 1500), (20, 80, 16, 1700)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
def test_against_the_model(shape):
    """Rounds of every operation on the same table."""
    B_, P, ps, N = shape
    table, lens, rng = random_state(sum(shape), B_, P, ps, N)
    m = Model(table, lens, N, ps)
    pages = table_of(table, lens, ps, N)
    assert pages.page_refs.tolist() == m.refs
    for step in range(4):
        parents = [rng.choice([b, b, -1, rng.randrange(B_), rng.randrange(B_)]) for b in range(B_)]
        if step == 1:
            parents = [0] * B_           # everyone continues one row
        m.fork(parents)
        pages.fork(torch.tensor(parents, dtype=torch.int32, device="cuda"))
        same(pages, m, moves=False)
        q = rng.choice([1, 1, 2, ps, ps + 1, min(1024, 3 * ps + 5)])
        ok = m.reserve(q)
        pages.reserve(q)
        same(pages, m)
        assert int(pages.counts[2]) == m.takes
        assert pages.device_status() == (0 if ok else B.UAA_DEVFLAG_POOL)
        if ok:
            for b in range(B_):
                if m.lens[b] + q <= P * ps:
                    m.lens[b] += q
            pages.seq_lens.copy_(torch.tensor(m.lens, dtype=torch.int32))
        w, f = rng.randint(1, P * ps), rng.choice([0, 1, ps - 1, ps, ps + 1])
        if P * ps * B_ <= 200_000:
            m.trim(w, f)
            pages.trim(w, f)
            same(pages, m, moves=False)
        n = m.compact()
        pages.compact()
        same(pages, m)
        assert int(pages.counts[1]) == n == pages.held()
        assert pages.device_status() == 0


@pytest.mark.gpu
def test_pool_without_enough_pages():
    """All or none: a reserve that the pool cannot serve changes nothing, and the
    next one, after pages were freed, is served."""
    table, lens = [[0, 1], [2, -1], [3, -1]], [32, 16, 16]
    pages = table_of(table, lens, 16, 5)
    before = pages.page_refs.clone()
    pages.reserve(1)   # rows 1 and 2 ask for a page each; one is free; row 0 is full
    assert pages.device_status() == B.UAA_DEVFLAG_POOL
    assert pages.counts.tolist()[0] == 0 and int(pages.counts[2]) == 2
    assert pages.block_table.tolist() == table and torch.equal(pages.page_refs, before)
    pages.fork(torch.tensor([-1, 1, 2], dtype=torch.int32, device="cuda"))
    pages.reserve(1)
    assert pages.device_status() == 0
    assert pages.block_table.tolist() == [[0, -1], [2, 1], [3, 4]]


@pytest.mark.gpu
def test_without_sequences():
    """A table without rows: nothing to fork, trim or reserve, and pinned pages still move."""
    from gqa_attention_kv_qk_gb300.pages import PageTable
    pages = PageTable(torch.zeros((0, 3)), 16, 6, page_refs=torch.tensor([0, 1, 0, 0, 2, 0]))
    pages.fork(torch.zeros(0, dtype=torch.int32, device="cuda"))
    pages.trim(1, 0)
    pages.reserve(5)
    assert pages.counts.tolist()[0] == 0 and pages.counts.tolist()[2] == 0
    pages.compact()
    assert pages.device_status() == 0
    assert pages.page_refs.tolist() == [2, 1, 0, 0, 0, 0]
    assert pages.moves[:1].tolist() == [[4, 0]] and pages.counts.tolist()[:2] == [1, 2]


@pytest.mark.gpu
def test_bad_entries_are_flagged_and_left():
    pages = table_of([[0, 1], [2, -1]], [20, 5], 16, 8)
    pages.block_table[0, 1] = 99
    pages.trim(1, 0)
    assert pages.device_status() == B.UAA_DEVFLAG_PAGE
    pages.compact()
    assert pages.device_status() == B.UAA_DEVFLAG_PAGE
    assert pages.block_table.tolist()[0][1] == 99
    pages.reserve(1)
    assert pages.device_status() == B.UAA_DEVFLAG_PAGE
    pages.fork(torch.tensor([0, 7], dtype=torch.int32, device="cuda"))  # no such parent: the row stays
    assert pages.device_status() == B.UAA_DEVFLAG_PAGE
    pool = torch.zeros(8, 64, device="cuda")
    pages.moves[0, 0], pages.moves[0, 1], pages.counts[0] = 3, 8, 1
    pages.copy(pool)
    assert pages.device_status() == B.UAA_DEVFLAG_PAGE


@pytest.mark.gpu
@pytest.mark.parametrize("shape,dtype", [((9, 4), torch.float32), ((50, 3, 16, 64), torch.bfloat16),
                                         ((50, 7, 5, 16), torch.uint8), ((7, 70001, 8), torch.float16)])
def test_copy(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(4)
    pools = [torch.randint(0, 100, shape, generator=g, device="cuda").to(dtype) for _ in range(3)]
    pools.append(torch.randint(0, 100, (shape[0], 16), generator=g, device="cuda").to(torch.int8))
    N = shape[0]
    pages = table_of([[0]], [1], 16, N)
    src, dst = list(range(0, N, 2)), list(range(1, N, 2))
    pairs = list(zip(src, dst))
    pages.moves[:len(pairs)] = torch.tensor(pairs, dtype=torch.int32)
    for n in (0, 1, len(pairs)):
        pages.counts[0] = n
        want = [p.clone() for p in pools]
        for w in want:
            for s, d in pairs[:n]:
                w[d] = w[s]
        pages.copy(*pools)
        assert all(torch.equal(a, b) for a, b in zip(pools, want))
    with pytest.raises(ValueError, match="pool"):
        pages.copy(pools[0][1:])
    with pytest.raises(B.UaaError, match="page_bytes"):
        pages.copy(torch.zeros(N, 3, dtype=torch.uint8, device="cuda"))
    assert pages.device_status() == 0


def test_host_errors_need_no_gpu():
    if not torch.cuda.is_available():
        from gqa_attention_kv_qk_gb300.pages import PageTable
        with pytest.raises(RuntimeError, match="CUDA"):
            PageTable([[0]], 16, 1)


@pytest.mark.gpu
def test_table_refusals():
    from gqa_attention_kv_qk_gb300.pages import PageTable
    for bad in (dict(block_table=[[0, 9]], n_pages=4), dict(block_table=[[0, -2]], n_pages=4)):
        with pytest.raises(ValueError, match="outside"):
            PageTable(torch.tensor(bad["block_table"]), 16, bad["n_pages"])
    with pytest.raises(ValueError, match="dimensions"):
        PageTable(torch.tensor([0, 1]), 16, 4)
    with pytest.raises(ValueError, match="page_refs"):
        PageTable(torch.tensor([[0, 1]]), 16, 4, page_refs=torch.zeros(3))
    with pytest.raises(B.UaaError, match="n_pages=0"):
        PageTable(torch.tensor([[-1]]), 16, 0, page_refs=torch.zeros(0))
    pages = PageTable(torch.tensor([[0, 1]]), 16, 4)
    with pytest.raises(ValueError, match="parents"):
        pages.fork(torch.tensor([0], dtype=torch.int64, device="cuda"))
    with pytest.raises(B.UaaError, match="q_len=0"):
        pages.reserve(0)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "q4"])
@pytest.mark.parametrize("captured", [False, True])
def test_together(kv, captured):
    """Streams that branch, end, and run under a window with first tokens on one pool:
    every step's outputs are those of the sequences' own histories, kept apart in
    64 bits; the pool holds no more pages than the windows need."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    Bn, ps, P, T, win, first = 5, 32, 12, 3, 70, 20
    cfg = dict(n_q_heads=4, n_kv_heads=2, head_dim=64, kv_dtype=kv, io_dtype="bf16", out_dtype="f32",
               rope_style="neox", rope_theta=10000.0, window=win, first_tokens=first, seed=3, batch=Bn, seq_len=1)
    N = 40
    pages = table_of([[-1] * P for _ in range(Bn)], [0] * Bn, ps, N)
    layer = DecodeLayer(cfg, Bn, P * ps, page_size=ps, block_table=pages.block_table, n_pages=N, max_q_len=T,
                        cache=dict(seq_lens=pages.seq_lens))
    assert layer.block_table is pages.block_table and layer.seq_lens is pages.seq_lens
    rng = random.Random(11)
    hist = [([], []) for _ in range(Bn)]  # every row's keys and values so far, as the cache holds them
    buf = {n: torch.zeros((Bn, T, h, 64), dtype=torch.bfloat16, device="cuda") for n, h in
           (("q", 4), ("k", 2), ("v", 2))}
    par = torch.arange(Bn, dtype=torch.int32, device="cuda")
    q_rot = torch.empty((Bn, T, 4, 64), dtype=torch.float32, device="cuda")
    start = torch.zeros(Bn, dtype=torch.int32, device="cuda")
    got = {}

    def one_step():
        pages.fork(par)
        pages.reserve(T)
        pages.copy_layer(layer)
        start.copy_(layer.seq_lens)
        got["out"] = layer.step(buf["q"], buf["k"], buf["v"], max_seq_len=P * ps - T, advance_hint=False, q_rot=q_rot)
        got["rows"] = layer.read_rows(start, T)
        pages.trim(win, first)
        pages.compact()
        pages.copy_layer(layer)

    graph = None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            saved = [t.clone() for t in (pages.block_table, pages.page_refs, pages.seq_lens)]
            one_step()  # the kernels' first launches happen outside the capture
            for t, s in zip((pages.block_table, pages.page_refs, pages.seq_lens), saved):
                t.copy_(s)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                one_step()
        torch.cuda.current_stream().wait_stream(side)
    for step in range(60):
        lens = [len(h[0]) for h in hist]
        parents = list(range(Bn))
        if step and step % 4 == 0:
            parents = [rng.randrange(Bn) for _ in range(Bn)]
        if step % 13 == 12:
            parents[rng.randrange(Bn)] = -1
        par.copy_(torch.tensor(parents, dtype=torch.int32))
        for n, t in buf.items():
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(100 * step + len(n) + ord(n[0]))))
        hist = [([], []) if p < 0 else (list(hist[p][0]), list(hist[p][1])) for p in parents]
        lens = [len(h[0]) for h in hist]
        if graph is not None:
            graph.replay()
        else:
            one_step()
        torch.cuda.synchronize()
        assert layer.device_status() == 0 and pages.device_status() == 0
        rk, rv = (x.double().cpu() for x in got["rows"])
        for b in range(Bn):
            for t in range(T):
                hist[b][0].append(rk[b, t])
                hist[b][1].append(rv[b, t])
        assert pages.seq_lens.tolist() == [n + T for n in lens]
        for b in range(Bn):
            k, v = (torch.stack(x, 1).unsqueeze(0) for x in hist[b])
            want = plain64.attend(q_rot[b:b + 1], k, v, [lens[b]], win, first)
            err = (got["out"][b:b + 1].double().cpu() - want).abs()
            assert float(err.max()) <= 4e-3, (step, b)
        # first tokens' pages (1) and the window's (at most 4), and no hole below them
        held = pages.held()
        assert held <= Bn * 5
        assert bool((pages.page_refs[:held] > 0).all()) and bool((pages.page_refs[held:] == 0).all())


@pytest.mark.gpu
def test_two_layers_on_one_table():
    """Layers of different kinds share the table: the bookkeeping runs once, the copies
    for each, and both keep their sequences' rows through forks and compaction."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    Bn, ps, P, N = 4, 32, 6, 30
    base = dict(n_q_heads=4, n_kv_heads=2, head_dim=64, io_dtype="bf16", out_dtype="f32", rope_style="neox",
                rope_theta=10000.0, seed=3, batch=Bn, seq_len=1)
    pages = table_of([[-1] * P for _ in range(Bn)], [0] * Bn, ps, N)
    layers = [DecodeLayer(dict(base, kv_dtype=kv), Bn, P * ps, page_size=ps, block_table=pages.block_table, n_pages=N,
                          max_q_len=20) for kv in ("q4", "q8", "bf16", "f32", "vq8")]
    rng = random.Random(5)
    hist = [[([], []) for _ in range(Bn)] for _ in layers]
    for step in range(12):
        T = rng.choice([1, 2, 20])
        parents = [rng.randrange(Bn) for _ in range(Bn)] if step % 3 == 2 else list(range(Bn))
        pages.fork(torch.tensor(parents, dtype=torch.int32, device="cuda"))
        pages.reserve(T)
        start = pages.seq_lens.clone()
        assert pages.device_status() == 0
        for i, layer in enumerate(layers):
            pages.copy_layer(layer)
            layer.seq_lens.copy_(pages.seq_lens)
            shape = lambda h: (Bn, T, h, 64) if T > 1 else (Bn, h, 64)
            g = torch.Generator().manual_seed(1000 * step + i)
            q, k, v = (torch.randn(shape(h), generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))
            layer.step(q, k, v, max_seq_len=P * ps - 20)
            assert layer.device_status() == 0
            rk, rv = (x.clone() for x in layer.read_rows(start, T))
            hist[i] = [(list(hist[i][p][0]), list(hist[i][p][1])) for p in parents]
            for b in range(Bn):
                for t in range(T):
                    hist[i][b][0].append(rk[b, t])
                    hist[i][b][1].append(rv[b, t])
        pages.seq_lens.copy_(layers[0].seq_lens)
        if step % 2:
            pages.compact()
            for layer in layers:
                pages.copy_layer(layer)
        for i, layer in enumerate(layers):  # every row that a sequence has written, wherever it is now
            n = max(len(h[0]) for h in hist[i])
            rk, rv = layer.read_rows(None, n)
            for b in range(Bn):
                m = len(hist[i][b][0])
                assert torch.equal(rk[b, :m], torch.stack(hist[i][b][0])), (step, i, b)
                assert torch.equal(rv[b, :m], torch.stack(hist[i][b][1])), (step, i, b)
        if int(pages.seq_lens.max()) > P * ps - 45:
            break
    assert step >= 5


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 1500])  # more requests than one pass of the CTA takes
def test_idle_rows_ask_for_nothing(rows):
    """A row that ended and is marked idle holds no page and asks for none, through forks
    of it too; a pool with room for the others alone serves them. At length 0 it
    starts over."""
    live = rows // 3
    pages = table_of([[-1, -1]] * rows, [0] * rows, 16, 2 * live)
    par = torch.tensor([b if b < live else -1 for b in range(rows)], dtype=torch.int32, device="cuda")
    pages.fork(par)
    pages.seq_lens.masked_fill_(par < 0, -1)
    for step in range(2):
        pages.reserve(16)
        assert pages.device_status() == 0 and int(pages.counts[2]) == live
        pages.seq_lens[:live] += 16
        pages.trim(40, 1)
        par = torch.tensor([b if b < live else rows - 1 for b in range(rows)], dtype=torch.int32, device="cuda")
        pages.fork(par)
    assert pages.seq_lens.tolist() == [32] * live + [-1] * (rows - live)
    assert pages.block_table.tolist() == [[b, live + b] for b in range(live)] + [[-1, -1]] * (rows - live)
    pages.fork(torch.tensor([-1] + list(range(1, rows)), dtype=torch.int32, device="cuda"))
    pages.reserve(1)
    assert pages.block_table.tolist()[0] == [0, -1] and pages.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2, 3000])  # fork in one launch, and in two
@pytest.mark.parametrize("after", ["fork", "trim"])
def test_copy_after_fork_or_trim_does_nothing(after, rows):
    """The moves of a reserve are void once the table has changed: a copy that comes too
    late leaves the pages as the sequences have them now."""
    pages = table_of([[0, 1, -1]] + [[-1] * 3] * (rows - 1), [20] + [0] * (rows - 1), 16, 8)
    par = torch.tensor([0, 0] + [-1] * (rows - 2), dtype=torch.int32, device="cuda")
    pages.fork(par)
    pages.seq_lens[2:] = -1
    pages.reserve(1)
    assert pages.moves[:1].tolist() == [[1, 2]] and int(pages.counts[0]) == 1
    pool = torch.arange(8, device="cuda", dtype=torch.float32).unsqueeze(1).repeat(1, 64)
    pages.copy(pool)
    assert float(pool[2, 0]) == 1.0
    pool[2] = 50.0                    # the sequence that took page 2 writes it
    if after == "fork":
        pages.fork(torch.arange(rows, dtype=torch.int32, device="cuda"))
    else:
        pages.trim(100, 0)
    before = pool.clone()
    pages.copy(pool)
    assert torch.equal(pool, before) and int(pages.counts[0]) == 0 and pages.device_status() == 0


def marks(pages):
    """The per-page request marks in the workspace of the page operators."""
    al = lambda n: (4 * n + 255) // 256 * 256
    at = 256 + 2 * al(pages.batch * pages.pages_per_seq) + al(pages.batch)
    return pages.ws_tensor[at:at + 2 * al(pages.n_pages)].view(torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,q_len", [(6, 1), (6, 40), (600, 40)])
def test_requests_leave_no_marks(rows, q_len):
    """reserve counts who asks for which held page in the workspace, and leaves those
    counts at zero: after a served call, one in which the last holder keeps its page,
    and one that the pool could not serve."""
    table = [[0, 1, 2, -1]] + [[-1] * 4] * (rows - 1)
    pages = table_of(table, [40] + [0] * (rows - 1), 16, 8 * rows)
    assert marks(pages).numel() >= 2 * pages.n_pages
    pages.fork(torch.zeros(rows, dtype=torch.int32, device="cuda"))  # every row holds the same pages
    for pins in (True, False):
        if pins:
            pages.page_refs[3:].add_(1)   # no page is free: refused
        pages.reserve(q_len if q_len + 40 <= 64 else 20)
        assert pages.device_status() == (B.UAA_DEVFLAG_POOL if pins else 0)
        assert not marks(pages).any()
        if pins:
            pages.page_refs[3:].sub_(1)
    assert pages.block_table[-1, 2] == 2  # the last holder kept it
    assert len(set(pages.block_table[:, 2].tolist())) == rows
    pages.compact()
    assert not marks(pages).any() and pages.device_status() == 0
