"""The cache operators of the decode step and the cases they are measured on.

Three operators. Attention of one step (append of the new tokens, then softmax
attention) over a cache held in 4 bits; the same step under a sliding window with
a few first tokens that stay visible; and the pages of a paged cache: branching
(fork, reserve with copy-on-write, copy) and reclaiming (trim behind the window,
compact, copy).

`run` computes a case in plain torch operations, in 32 bits (angles in 64), or,
where `own` is true, makes the calls a user makes of the library. `exact`
computes the attention cases in 64 bits from the definition.

A 4-bit row of D values: groups of 32 dims, each with a scale s = max|x| / 7
rounded to 8 significant bits (bf16, then fp16; at most 2720), codes
c = rint(x / s) in [-7, 7], stored as nibbles c + 8, dim 2i in the low nibble of
byte i.
"""
import math
import random

import torch

own = False

MAX_SCALE = 2720.0  # 24 * s and 7 * s stay finite in fp16


# ---------------------------------------------------------------- the cases

def _attend(name, kv, B, Hq, Hkv, D, lo, hi, T=1, page=0, window=0, first=0, softcap=0.0, sink=False, norm=False):
    c = dict(kind="attend", kv=kv, B=B, Hq=Hq, Hkv=Hkv, D=D, lo=lo, hi=hi, T=T, page=page, window=window, first=first,
             softcap=softcap, sink=sink, norm=norm)
    return dict(name=name, **c) if name else c


def _pages(name, kind, B, Hkv, D, page, per_seq, n_pages, T=1, window=0, first=0):
    c = dict(kind=kind, B=B, Hkv=Hkv, D=D, page=page, per_seq=per_seq, n_pages=n_pages, T=T, window=window, first=first)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one short conversation on a small model: launch latency
        _attend("q4_decode_one", "q4", 1, 32, 8, 64, 256, 256),
        # a full batch of decode steps at 8K tokens
        _attend("q4_decode_8k", "q4", 16, 32, 8, 128, 8192, 8192),
        # a serving batch of mixed ages on a paged pool, per-head norm of q and k
        _attend("q4_decode_ragged_paged", "q4", 32, 32, 8, 128, 1024, 32768, page=64, norm=True),
        # draft tokens to verify, 8 query heads per kv head, sink logits, odd length
        _attend("q4_verify_g8_sink", "q4", 64, 64, 8, 64, 4095, 4095, T=3, sink=True),
        # a prefill chunk onto a 4-bit cache
        _attend("q4_prefill_chunk", "q4", 4, 32, 8, 128, 8000, 8192, T=256),
        # long conversations that keep 4 first tokens and the last 4096
        _attend("first_decode_32k", "bf16", 16, 32, 8, 128, 32768, 32768, window=4096, first=4),
        # the same idea on a paged 4-bit pool whose pages behind the window were freed, ragged
        _attend("first_paged_q4_ragged", "q4", 32, 32, 8, 128, 1, 20000, page=32, window=1000, first=65, norm=True),
        # a prefill chunk under a window with first tokens
        _attend("first_prefill_chunk", "bf16", 4, 32, 8, 128, 12345, 16384, T=512, window=2048, first=16),
        # a beam of 8 reorders and takes its next pages: latency
        _pages("branch_beam8", "branch", 8, 8, 128, 16, 64, 512),
        # 256 sequences fork, then each needs room for 4 tokens: many shared last pages to copy
        _pages("branch_batch256", "branch", 256, 8, 128, 64, 128, 16384, T=4),
        # a small pool is tidied
        _pages("reclaim_small", "reclaim", 8, 8, 128, 16, 64, 512, window=200, first=16),
        # a 4 GB pool is trimmed behind a window and compacted
        _pages("reclaim_pool", "reclaim", 128, 8, 128, 64, 256, 16384, window=4096, first=64),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng: random.Random):
    what = rng.choice(["q4", "q4", "first", "first", "branch", "reclaim"])
    if what in ("q4", "first"):
        D = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 8]) if D != 256 else rng.choice([1, 2, 4])
        T = rng.choice([1, 1, 1, rng.randint(2, 9), _log(rng, 16, 256)])
        hi = _log(rng, 1, 20000)
        # at most a quarter of the largest listed case's cache rows and score elements
        B = max(1, min(_log(rng, 1, 64), 500_000 // max(hi, 64) // Hkv, 60_000_000 // (Hkv * G * T * max(hi, 64))))
        lo = rng.randint(0, hi)
        page = rng.choice([0, 32, 64, 128, 256])
        kv = "q4" if what == "q4" else rng.choice(["bf16", "q4"])
        window = _log(rng, 1, 8192) if what == "first" or rng.random() < 0.3 else 0
        first = _log(rng, 1, 300) if what == "first" else 0
        return _attend(None, kv, B, Hkv * G, Hkv, D, lo, hi, T, page, window, first,
                       rng.choice([0.0, 0.0, 50.0]), rng.random() < 0.3, rng.random() < 0.3)
    page = rng.choice([16, 32, 64, 128])
    per_seq = _log(rng, 2, 128)
    B = _log(rng, 1, 200)
    n_pages = max(8, min(2 * B * per_seq + rng.randint(0, 99), 8192 * 64 // page))
    B = max(1, min(B, n_pages // 2))
    Hkv, D = rng.choice([1, 2, 8]), rng.choice([64, 128])
    if what == "branch":
        return _pages(None, "branch", B, Hkv, D, page, per_seq, n_pages, T=rng.choice([1, 1, 3, page + 1]))
    return _pages(None, "reclaim", B, Hkv, D, page, per_seq, n_pages, window=_log(rng, 1, per_seq * page),
                  first=rng.choice([0, 1, 4, page, 3 * page + 1]))


# ---------------------------------------------------------------- inputs

def _capacity(c):
    unit = max(64, c["page"])
    return (c["hi"] + c["T"] + unit - 1) // unit * unit


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quantize(x):
    """4-bit codes (two per byte) and fp16 scales of rows x [..., D]."""
    D = x.shape[-1]
    g = x.float().reshape(*x.shape[:-1], D // 32, 32)
    s = (g.abs().amax(-1) / 7.0).to(torch.bfloat16).float().clamp(max=MAX_SCALE).to(torch.float16)
    sf = s.float().unsqueeze(-1)
    code = torch.where(sf > 0, torch.round(g / sf.clamp(min=1e-30)).clamp(-7, 7), torch.zeros_like(g))
    u = (code + 8).to(torch.uint8).reshape(*x.shape[:-1], D // 2, 2)
    return u[..., 0] | (u[..., 1] << 4), s


def _values(codes, scales):
    """The values that codes and scales stand for, in 32 bits."""
    u = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    c = u.float() - 8.0
    return (c.reshape(*scales.shape, 32) * scales.float().unsqueeze(-1)).reshape(c.shape)


def prepare(case, seed):
    return _prepare_attend(case, seed) if case["kind"] == "attend" else _prepare_pages(case, seed)


def _prepare_attend(c, seed):
    g = _gen(seed)
    dev = "cuda"
    B, Hq, Hkv, D, T, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"], c["page"]
    cap = _capacity(c)
    lens = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    lens[0] = c["hi"]
    s = dict(case=c, cap=cap, lens0=lens, lens=lens.clone())
    if page:  # every sequence's pages, in random order over a pool with spare pages
        per_seq = cap // page
        n_pages = B * per_seq + max(2, B)
        table = torch.randperm(n_pages, generator=g, device=dev)[: B * per_seq].reshape(B, per_seq).to(torch.int32)
        # pages that no token can see any more were freed; pages past the new tokens are not there yet
        at = torch.arange(per_seq, device=dev).unsqueeze(0) * page
        n = lens.long().unsqueeze(1)
        gone = at >= n + T
        if c["window"]:
            gone |= (at >= c["first"]) & (at + page <= n - c["window"] + 1)
        s["table"] = torch.where(gone, torch.full_like(table, -1), table)
        s["n_pages"] = n_pages
        rows = (n_pages, Hkv, page)
    else:
        s["table"], s["n_pages"], rows = None, 0, (B, Hkv, cap)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    # a few dims of the keys are larger than the rest, as rotary models' caches have them
    gain = 1.0 + 3.0 * (torch.rand((D,), generator=g, device=dev) < 0.05).float()
    for n, w in (("k", gain), ("v", torch.ones_like(gain))):
        cache = torch.empty((*rows, D), dtype=torch.bfloat16, device=dev)
        if c["kv"] == "q4":
            codes = torch.empty((*rows, D // 2), dtype=torch.uint8, device=dev)
            scales = torch.empty((*rows, D // 32), dtype=torch.float16, device=dev)
        step = max(1, (1 << 26) // (rows[1] * rows[2] * D))
        for i in range(0, rows[0], step):
            x = normal(min(step, rows[0] - i), *rows[1:], D) * w
            if c["kv"] == "q4":
                codes[i:i + step], scales[i:i + step] = _quantize(x)
            else:
                cache[i:i + step] = x.to(torch.bfloat16)
        if c["kv"] == "q4":
            s[n + "_cache"], s[n + "_scale"] = codes, scales
        else:
            s[n + "_cache"], s[n + "_scale"] = cache, None
    tok = (T,) if T > 1 else ()
    s["q"] = normal(B, *tok, Hq, D).to(torch.bfloat16)
    s["k_new"] = (normal(B, *tok, Hkv, D) * gain).to(torch.bfloat16)
    s["v_new"] = normal(B, *tok, Hkv, D).to(torch.bfloat16)
    s["sink"] = normal(Hq) if c["sink"] else None
    s["q_norm_w"] = 0.5 + torch.rand((D,), generator=g, device=dev) if c["norm"] else None
    s["k_norm_w"] = 0.5 + torch.rand((D,), generator=g, device=dev) if c["norm"] else None
    return s


def _prepare_pages(c, seed):
    g = _gen(seed)
    dev = "cuda"
    B, P, ps, N = c["B"], c["per_seq"], c["page"], c["n_pages"]
    # lengths: some rows empty, the others anywhere up to the table's end (short of the new tokens)
    most = max(1, P * ps - c["T"])
    lens = torch.randint(0, most + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    lens[torch.rand((B,), generator=g, device=dev) < 0.1] = 0
    held = (lens.long() + ps - 1) // ps
    # sequences take pages at random places of the pool, as many as half of it gives
    most_held = (torch.cumsum(held, 0) <= N // 2)
    lens = torch.where(most_held, lens, torch.zeros_like(lens))
    held = torch.where(most_held, held, torch.zeros_like(held))
    perm = torch.randperm(N, generator=g, device=dev).to(torch.int32)
    start = torch.cumsum(held, 0) - held
    l = torch.arange(P, device=dev).unsqueeze(0)
    table = torch.where(l < held.unsqueeze(1), perm[(start.unsqueeze(1) + l).clamp(max=N - 1)],
                        torch.full((1, 1), -1, dtype=torch.int32, device=dev))
    refs = torch.bincount(table[table >= 0].long(), minlength=N).to(torch.int32)
    pool = (N, c["Hkv"], ps, c["D"])
    s = dict(case=c, table0=table.contiguous(), refs0=refs, lens0=lens, table=table.clone(), refs=refs.clone(),
             lens=lens.clone(),
             k_cache=torch.randn(pool, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16),
             v_cache=torch.randn(pool, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16))
    # the best beams' parents: some rows continue, some are replaced by others, some end
    par = torch.randint(0, B, (B,), generator=g, device=dev)
    keep = torch.rand((B,), generator=g, device=dev)
    par = torch.where(keep < 0.4, torch.arange(B, device=dev), par)
    s["parents"] = torch.where(keep > 0.95, torch.full_like(par, -1), par).to(torch.int32)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own_attend(state) if kind == "attend" else _own_pages(state)
    if kind == "attend":
        return _plain_attend(state)
    return _plain_branch(state) if kind == "branch" else _plain_reclaim(state)


THETA = 500000.0


def _config(c):
    return dict(n_q_heads=c["Hq"], n_kv_heads=c["Hkv"], head_dim=c["D"], kv_dtype=c["kv"], io_dtype="bf16",
                out_dtype="bf16", rope_style="neox", rope_theta=THETA, rope_scaling="none", qk_norm=c["norm"],
                norm_eps=1e-6, window=c["window"], first_tokens=c["first"], softcap=c["softcap"], has_sink=c["sink"])


def _own_attend(s):
    c = s["case"]
    layer = s.get("layer")
    if layer is None:  # what a program keeps: the layer, its workspace and its cache
        from gqa_attention_kv_qk_gb300.layer import DecodeLayer
        layer = DecodeLayer(_config(c), c["B"], s["cap"], page_size=c["page"], block_table=s["table"],
                            n_pages=s["n_pages"], max_q_len=c["T"],
                            cache=dict(k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"],
                                       v_scale=s["v_scale"], seq_lens=s["lens"]))
        layer.set_params(s["q_norm_w"], s["k_norm_w"], s["sink"])
        s["layer"] = layer
    layer.seq_lens.copy_(s["lens0"])
    out = layer.step(s["q"], s["k_new"], s["v_new"], max_seq_len=c["hi"])
    k, v = layer.read_rows(s["lens0"], c["T"])
    return dict(out=out, k_rows=k, v_rows=v, lens=layer.seq_lens)


def _own_pages(s):
    c = s["case"]
    pages = s.get("pages")
    if pages is None:
        from gqa_attention_kv_qk_gb300.pages import PageTable
        pages = s["pages"] = PageTable(s["table"], c["page"], c["n_pages"], page_refs=s["refs"], seq_lens=s["lens"])
    pages.block_table.copy_(s["table0"])
    pages.page_refs.copy_(s["refs0"])
    pages.seq_lens.copy_(s["lens0"])
    if c["kind"] == "branch":
        pages.fork(s["parents"])
        pages.reserve(c["T"])
    else:
        pages.trim(c["window"], c["first"])
        pages.compact()
    pages.copy(s["k_cache"], s["v_cache"])
    return dict(table=pages.block_table, refs=pages.page_refs, lens=pages.seq_lens, k=s["k_cache"], v=s["v_cache"])


def _rope(x, pos):
    """NeoX rotation of rows x [B, T, H, D] at positions pos [B, T]."""
    D = x.shape[-1]
    f = THETA ** (-torch.arange(0, D, 2, device=x.device, dtype=torch.float64) / D)
    ang = pos.double().unsqueeze(-1) * f
    cos, sin = ang.cos().float().unsqueeze(2), ang.sin().float().unsqueeze(2)
    a, b = x[..., : D // 2], x[..., D // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _norm(x, w):
    return x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w


def _places(s, pos):
    """Flat cache rows of positions pos [B, T], per kv head: [B, T, Hkv]."""
    c = s["case"]
    h = torch.arange(c["Hkv"], device=pos.device)
    if not c["page"]:
        b = torch.arange(c["B"], device=pos.device).reshape(-1, 1, 1)
        return (b * c["Hkv"] + h) * s["cap"] + pos.unsqueeze(-1)
    page = torch.gather(s["table"].long(), 1, pos // c["page"])
    return (page.unsqueeze(-1) * c["Hkv"] + h) * c["page"] + (pos % c["page"]).unsqueeze(-1)


def _logical(s, x):
    """Cache rows in order of their positions, [B, Hkv, cap, ...]; rows of absent pages are anything."""
    c = s["case"]
    if not c["page"]:
        return x
    y = x[s["table"].long().clamp(min=0)]  # [B, per_seq, Hkv, page, ...]
    return y.transpose(1, 2).reshape(c["B"], c["Hkv"], s["cap"], *x.shape[3:])


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"]
    G, cap = Hq // Hkv, s["cap"]
    s["lens"].copy_(s["lens0"])
    pos = s["lens"].long().unsqueeze(1) + torch.arange(T, device="cuda")
    q = _rope(_norm(s["q"].float().reshape(B, T, Hq, D), s["q_norm_w"]), pos)
    k = _rope(_norm(s["k_new"].float().reshape(B, T, Hkv, D), s["k_norm_w"]), pos)
    v = s["v_new"].float().reshape(B, T, Hkv, D)
    at = _places(s, pos).reshape(-1)
    got = []
    for name, x in (("k", k), ("v", v)):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        if c["kv"] == "q4":
            codes, sc = _quantize(x)
            cache.reshape(-1, D // 2)[at] = codes.reshape(-1, D // 2)
            scale.reshape(-1, D // 32)[at] = sc.reshape(-1, D // 32)
            got.append(_values(codes, sc).to(torch.bfloat16))
        else:
            x = x.to(torch.bfloat16)
            cache.reshape(-1, D)[at] = x.reshape(-1, D)
            got.append(x)
    s["lens"] += T
    if c["kv"] == "q4":
        keys = _values(_logical(s, s["k_cache"]), _logical(s, s["k_scale"]))
        vals = _values(_logical(s, s["v_cache"]), _logical(s, s["v_scale"]))
    else:
        keys, vals = _logical(s, s["k_cache"]).float(), _logical(s, s["v_cache"]).float()
    # [B, Hkv, T * G, cap]
    qg = q.reshape(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    z = torch.matmul(qg, keys.transpose(2, 3)) / math.sqrt(D)
    if c["softcap"]:
        z = c["softcap"] * torch.tanh(z / c["softcap"])
    j = torch.arange(cap, device="cuda")
    p = pos.repeat_interleave(G, 1).unsqueeze(-1)
    seen = j <= p
    if c["window"]:
        seen = seen & ((j > p - c["window"]) | (j < c["first"]))
    z = z.masked_fill(~seen.unsqueeze(1), -math.inf)
    m = z.amax(-1, keepdim=True)
    if c["sink"]:
        sink = s["sink"].reshape(Hkv, 1, G).expand(Hkv, T, G).reshape(1, Hkv, T * G, 1)
        m = torch.maximum(m, sink)
    e = torch.exp(z - m)
    den = e.sum(-1, keepdim=True)
    if c["sink"]:
        den = den + torch.exp(sink - m)
    o = torch.matmul(e, vals) / den
    o = o.reshape(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    shape = (B, T, Hq, D) if T > 1 else (B, Hq, D)
    return dict(out=o.reshape(shape).to(torch.bfloat16), k_rows=got[0], v_rows=got[1], lens=s["lens"])


def _count(table, n):
    return torch.bincount(table[table >= 0].long(), minlength=n).to(torch.int32)


def _plain_branch(s):
    """Rows take their parents' rows (-1: freed); then every sequence gets pages of
    its own for its next T tokens: the lowest free ones, in order of (sequence,
    page); a shared page that is written next is copied, and the last of its
    sequences keeps it where nothing else holds it."""
    c = s["case"]
    B, P, ps, N, T = c["B"], c["per_seq"], c["page"], c["n_pages"], c["T"]
    par = s["parents"].long()
    ended = par < 0
    old = s["table0"]
    table = torch.where(ended.unsqueeze(1), torch.full_like(old, -1), old[par.clamp(min=0)])
    lens = torch.where(ended, torch.zeros_like(s["lens0"]), s["lens0"][par.clamp(min=0)])
    refs = s["refs0"] - _count(old, N) + _count(table, N)
    l = torch.arange(P, device="cuda").unsqueeze(0)
    n = lens.long().unsqueeze(1)
    wanted = (l >= n // ps) & (l <= (n + T - 1) // ps) & (n + T <= P * ps)
    held = wanted & (table >= 0)
    asked = _count(torch.where(held, table, torch.full_like(table, -1)), N)
    at = torch.arange(B * P, device="cuda").reshape(B, P)
    last = torch.full((N,), -1, dtype=torch.long, device="cuda")
    last = last.scatter_reduce(0, table[held].long(), at[held], "amax")
    e = table.long().clamp(min=0)
    stays = held & ((refs[e] == 1) | ((refs[e] == asked[e]) & (last[e] == at)))
    takes = wanted & ~stays
    free = (refs == 0).nonzero().squeeze(1).to(torch.int32)
    if int(takes.sum()) <= free.numel():
        fresh = free[: int(takes.sum())]
        was = table[takes]
        kept = (held & takes & (l * ps < n))[takes]  # rows before the new tokens are copied
        refs = refs - _count(was, N)
        refs[fresh.long()] = 1
        table = table.clone()
        table[takes] = fresh
        src, dst = was[kept].long(), fresh[kept].long()
        s["k_cache"][dst] = s["k_cache"][src]
        s["v_cache"][dst] = s["v_cache"][src]
    s["table"].copy_(table)
    s["refs"].copy_(refs)
    s["lens"].copy_(lens)
    return dict(table=s["table"], refs=s["refs"], lens=s["lens"], k=s["k_cache"], v=s["v_cache"])


def _plain_reclaim(s):
    """Pages that no later token can see leave the table; then the pages that are
    held move to the front of the pool, the lowest first into the lowest hole."""
    c = s["case"]
    P, ps, N = c["per_seq"], c["page"], c["n_pages"]
    old, lens = s["table0"], s["lens0"]
    l = torch.arange(P, device="cuda").unsqueeze(0) * ps
    gone = (l >= c["first"]) & (l + ps <= lens.long().unsqueeze(1) - c["window"] + 1) & (old >= 0)
    table = torch.where(gone, torch.full_like(old, -1), old)
    refs = s["refs0"] - _count(torch.where(gone, old, torch.full_like(old, -1)), N)
    live = refs > 0
    n_live = int(live.sum())
    at = torch.arange(N, device="cuda")
    dst = ((~live) & (at < n_live)).nonzero().squeeze(1)
    src = (live & (at >= n_live)).nonzero().squeeze(1)
    to = at.clone()
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table = torch.where(table >= 0, to[table.long().clamp(min=0)].to(torch.int32), table)
    s["k_cache"][dst] = s["k_cache"][src]
    s["v_cache"][dst] = s["v_cache"][src]
    s["table"].copy_(table)
    s["refs"].copy_(refs)
    s["lens"].copy_(lens)
    return dict(table=s["table"], refs=s["refs"], lens=s["lens"], k=s["k_cache"], v=s["v_cache"])


# ---------------------------------------------------------------- what a pass cannot do without

def _seen(c, lens):
    """Keys read per sequence (the union over its new tokens), and (row, key) pairs per query head."""
    keys = pairs = 0
    for n in lens:
        end = n + c["T"]
        lo = max(0, n + 1 - c["window"]) if c["window"] else 0
        keys += end - lo + min(c["first"], lo)
        for p in (n, end - 1):
            lo = max(0, p + 1 - c["window"]) if c["window"] else 0
            pairs += (p + 1 - lo + min(c["first"], lo)) * c["T"] / 2
    return keys, pairs


def work(case):
    c = case
    if c["kind"] == "attend":
        # lengths are drawn evenly over [lo, hi], the first one is hi
        B = c["B"]
        lens = [c["hi"]] + [c["lo"] + (c["hi"] - c["lo"]) * (2 * i + 1) // (2 * max(1, B - 1)) for i in range(B - 1)]
        keys, pairs = _seen(c, lens)
        row = c["D"] * 2 if c["kv"] == "bf16" else c["D"] // 2 + c["D"] // 16
        io = B * c["T"] * (2 * c["Hq"] * c["D"] * 2 + 4 * c["Hkv"] * c["D"] * 2 + 2 * c["Hkv"] * row)
        return dict(bytes=2 * keys * c["Hkv"] * row + io, flops=4 * pairs * c["Hq"] * c["D"])
    B, P, N, ps = c["B"], c["per_seq"], c["n_pages"], c["page"]
    page_bytes = 2 * 2 * c["Hkv"] * ps * c["D"] * 2  # a page of both pools, read and written
    table = 2 * 4 * (B * P + N + B)
    held = min(N // 2, B * P // 2 * 9 // 10)
    if c["kind"] == "branch":
        return dict(bytes=table + page_bytes * max(1, B // 2), flops=B * P)
    alive = held * min(1.0, (c["window"] + c["first"] + ps) / max(1, P * ps / 2))
    return dict(bytes=int(table + page_bytes * max(1, alive * (1 - alive / N))), flops=B * P)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The attention cases by their definition, a sequence and a kv head at a time."""
    c = case
    if c["kind"] != "attend":
        return None  # integers and copies
    s = _prepare_attend(c, seed)
    B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"]
    G, f8 = Hq // Hkv, torch.float64
    if B * Hkv > 1024:
        return None
    out = torch.empty((B, T, Hq, D), dtype=f8, device="cuda")
    new = {n: torch.empty((B, T, Hkv, D), dtype=f8, device="cuda") for n in "kv"}
    half = D // 2
    freq = torch.pow(torch.tensor(THETA, dtype=f8, device="cuda"),
                     -2.0 * torch.arange(half, dtype=f8, device="cuda") / D)

    def turned(x, w, at):  # rows [T, H, D] as complex numbers, turned by their positions' angles
        if w is not None:
            x = x * w.to(f8) * torch.rsqrt(torch.mean(x * x, -1, keepdim=True) + 1e-6)
        turn = torch.polar(torch.ones((T, half), dtype=f8, device="cuda"), at.unsqueeze(1) * freq).unsqueeze(1)
        y = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
        return torch.cat((y.real, y.imag), -1)

    def stored(x):  # what a row is worth once it is in the cache
        if c["kv"] == "bf16":
            return x.to(torch.bfloat16).to(f8)
        grp = x.unflatten(-1, (D // 32, 32))
        sc = torch.clamp((grp.abs().max(-1, keepdim=True).values / 7).to(torch.bfloat16).to(f8), max=MAX_SCALE)
        sc = sc.to(torch.float16).to(f8)
        lev = torch.clamp(torch.round(grp / torch.where(sc > 0, sc, torch.ones_like(sc))), -7, 7)
        return (lev * sc).flatten(-2)

    def cached(n, b, h, upto):  # positions [0, upto) of one head
        x, sc = s[n + "_cache"], s[n + "_scale"]
        if c["page"]:
            pages = s["table"][b, : (upto + c["page"] - 1) // c["page"]].long().clamp(min=0)
            x = x[pages, h].flatten(0, 1)[:upto]
            sc = None if sc is None else sc[pages, h].flatten(0, 1)[:upto]
        else:
            x, sc = x[b, h, :upto], None if sc is None else sc[b, h, :upto]
        if sc is None:
            return x.to(f8)
        nib = torch.empty((upto, D), dtype=f8, device="cuda")
        nib[:, 0::2] = (x % 16).to(f8)
        nib[:, 1::2] = torch.div(x, 16, rounding_mode="floor").to(f8)
        return (nib - 8) * sc.to(f8).repeat_interleave(32, 1)

    for b in range(B):
        n = int(s["lens0"][b])
        at = torch.arange(n, n + T, device="cuda")
        qr = turned(s["q"][b].reshape(T, Hq, D).to(f8), s["q_norm_w"], at.to(f8))
        new["k"][b] = stored(turned(s["k_new"][b].reshape(T, Hkv, D).to(f8), s["k_norm_w"], at.to(f8)))
        new["v"][b] = stored(s["v_new"][b].reshape(T, Hkv, D).to(f8))
        j = torch.arange(n + T, device="cuda")
        hidden = j.unsqueeze(0) > at.unsqueeze(1)
        if c["window"]:
            hidden |= (j.unsqueeze(0) + c["window"] <= at.unsqueeze(1)) & (j.unsqueeze(0) >= c["first"])
        use = (~hidden).any(0).nonzero().squeeze(1)
        hidden = hidden[:, use]
        for h in range(Hkv):
            kk = torch.cat((cached("k", b, h, n), new["k"][b, :, h]))[use]
            vv = torch.cat((cached("v", b, h, n), new["v"][b, :, h]))[use]
            logit = torch.einsum("tgd,nd->tgn", qr[:, h * G:(h + 1) * G], kk) * D ** -0.5
            if c["softcap"]:
                logit = torch.tanh(logit / c["softcap"]) * c["softcap"]
            logit.masked_fill_(hidden.unsqueeze(1), -math.inf)
            lse = torch.logsumexp(logit, -1)
            if c["sink"]:
                lse = torch.logaddexp(lse, s["sink"][h * G:(h + 1) * G].to(f8).expand_as(lse))
            out[b, :, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", torch.exp(logit - lse.unsqueeze(-1)), vv)
    return dict(out=out if T > 1 else out[:, 0], k_rows=new["k"], v_rows=new["v"], lens=None)
