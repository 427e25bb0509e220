"""One workspace through steps of different geometry: what a launch leaves in it for
the next one survives the steps between, and its size covers every shorter step.

Tolerance of the fp32 cache: the parity bar of the attention outputs (max 2e-3, mean
2e-4 for values ~N(0, 1)); fp32 arithmetic over 700 keys is off by some 1e-6.
"""
import pytest
import torch

from gqa_attention_kv_qk_gb300 import binding as B
from tests import plain64

TOL_MAX, TOL_MEAN = 2e-3, 2e-4


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gqa_attention_kv_qk_gb300 import build
    build.build()


def config(**kw):
    cfg = dict(n_q_heads=32, n_kv_heads=8, head_dim=128, kv_dtype="f32", io_dtype="f32", out_dtype="f32",
               rope_style="neox", rope_theta=10000.0, seed=41, batch=1, seq_len=64)
    cfg.update(kw)
    return cfg


def filled_layer(cfg, batch, cap, n, max_q_len):
    """A layer of `batch` sequences holding n random rows each."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    layer = DecodeLayer(cfg, batch, cap, max_q_len=max_q_len)
    g = torch.Generator(device="cuda").manual_seed(n)
    for t in (layer.k_cache, layer.v_cache):
        t[:, :, :n] = torch.randn(t[:, :, :n].shape, generator=g, device="cuda")
    layer.set_lengths([n] * batch)
    return layer


def rows(cfg, batch, T, seed):
    g = torch.Generator().manual_seed(seed)
    shape = lambda h: (batch, T, h, cfg["head_dim"]) if T > 1 else (batch, h, cfg["head_dim"])
    dt = torch.float32 if cfg["io_dtype"] == "f32" else torch.bfloat16
    return [torch.randn(shape(h), generator=g).to(dt).cuda() for h in
            (cfg["n_q_heads"], cfg["n_kv_heads"], cfg["n_kv_heads"])]


def assert_step(layer, out, q_rot, n, what):
    k, v = plain64.cached_values(layer)
    want = plain64.attend(q_rot, k[:, :, :n + q_rot.shape[1]], v[:, :, :n + q_rot.shape[1]], [n] * layer.batch)
    err = (out.double().cpu().reshape(want.shape) - want).abs()
    assert float(err.max()) <= TOL_MAX and float(err.mean()) <= TOL_MEAN, (what, float(err.max()))


@pytest.mark.gpu
@pytest.mark.parametrize("batch,chunk", [(12, 3), (8, 64)])
def test_fp32_steps_between_chunks(batch, chunk):
    """The fp32 one-launch step merges a unit's splits when the last of them has counted
    in. A chunk's split records (3 tokens, 12 sequences) or q rows (64 tokens) lie
    where the shorter step has other arrays: the counts are still zero after it."""
    cfg, n = config(), 700
    layer = filled_layer(cfg, batch, 1024, n, chunk)
    lay = B.uaa_get_workspace_layout(layer.desc, batch, n, 0, 1)
    assert lay.step_splits > 1
    layer.out.fill_(float("nan"))
    for i, T in enumerate((chunk, 1, 1, chunk, 1)):
        q, k, v = rows(cfg, batch, T, 10 * i + batch)
        q_rot = torch.empty((batch, T, 32, 128), device="cuda")
        out = layer.step(q, k, v, q_rot=q_rot)
        torch.cuda.synchronize()
        assert layer.device_status() == 0
        assert_step(layer, out, q_rot, n, (i, T))
        n += T


@pytest.mark.gpu
def test_fp32_step_after_another_desc_in_the_built_in_scratch():
    """The same through uaa_decode_attn_static, whose one array serves every desc."""
    cfg, n, batch = config(), 700, 8
    layer = filled_layer(cfg, batch, 1024, n, 1)
    other_cfg = config(kv_dtype="bf16", io_dtype="bf16")
    other = filled_layer(other_cfg, batch, 256, 100, 40)
    for i in range(2):
        q, k, v = rows(other_cfg, batch, 40, i)  # its q rows take most of the array
        other._begin(q)
        B.uaa_decode_attn_static(other.desc, other.args(q, k, v), torch.cuda.current_stream())
        other.max_len_hint += 40
        layer.out.fill_(float("nan"))
        q, k, v = rows(cfg, batch, 1, 5 + i)
        q_rot = torch.empty((batch, 1, 32, 128), device="cuda")
        layer._begin(q)
        B.uaa_decode_attn_static(layer.desc, layer.args(q, k, v, q_rot=q_rot), torch.cuda.current_stream())
        layer.max_len_hint += 1
        torch.cuda.synchronize()
        assert_step(layer, layer.out, q_rot, n, i)
        n += 1


@pytest.mark.parametrize("kv", ["f32", "bf16", "vq8", "q8", "q4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_size_never_falls_with_longer_steps(kv, D):
    """A workspace sized for q_len serves every step of at most q_len tokens."""
    for G, Hkv, batch, n_sm, max_len in ((1, 1, 1, 152, 100), (1, 8, 3, 152, 100), (2, 4, 16, 148, 4095),
                                         (4, 8, 16, 152, 4095), (8, 8, 4, 148, 4095), (8, 1, 1030, 152, 8000),
                                         (16, 2, 2, 152, 300), (20, 1, 1, 152, 5)):
        d = B.make_desc(config(kv_dtype=kv, head_dim=D, n_q_heads=G * Hkv, n_kv_heads=Hkv))
        sizes = [B.uaa_workspace_size(d, batch, max_len, n_sm, t) for t in (*range(1, 140), 300, 1000)]
        assert sizes[0] > 0 and sizes == sorted(sizes), (G, Hkv, batch)
        for t in (1, 5, 40):
            assert B.uaa_get_workspace_layout(d, batch, max_len, n_sm, t).total_bytes == sizes[t - 1]


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv_heads,longest", [(64, 8, 4), (16, 4, 8), (2, 1, 16), (1, 1, 32)])
def test_shorter_steps_than_the_longest(heads, kv_heads, longest):
    """Over a 4-bit cache at head_dim 64, 17-24 rows take 24-row units and 25-32 rows
    16-row ones, in a smaller workspace: a layer made for the longer steps serves both.
    (One sequence: its q rows do not make up for the units. Bar: q' and P are one fp16
    part each, 4e-3 and 4e-4 for values ~N(0, 1).)"""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    cfg = config(kv_dtype="q4", io_dtype="bf16", head_dim=64, n_q_heads=heads, n_kv_heads=kv_heads)
    layer = DecodeLayer(cfg, 1, 512, max_q_len=longest)
    n, G = 0, heads // kv_heads
    for i, T in enumerate((longest, 24 // G, 1, longest, 17 // G + 1, 24 // G)):
        q, k, v = rows(cfg, 1, T, i)
        q_rot = torch.empty((1, T, heads, 64), device="cuda")
        out = layer.step(q, k, v, q_rot=q_rot)
        torch.cuda.synchronize()
        assert layer.device_status() == 0
        kk, vv = plain64.cached_values(layer)
        want = plain64.attend(q_rot, kk, vv, [n])
        err = (out.double().cpu().reshape(want.shape) - want).abs()
        assert float(err.max()) <= 4e-3 and float(err.mean()) <= 4e-4, T
        n += T


@pytest.mark.gpu
def test_layers_that_share_a_workspace():
    """Layers of every kind on one workspace, one step after another (single tokens,
    drafts and prefill chunks), give what they give on workspaces of their own."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    kinds = [dict(kv_dtype=kv, io_dtype="f32" if kv == "f32" else "bf16", head_dim=D, reproducible=True, **kw)
             for kv, D, kw in (("q4", 128, {}), ("f32", 64, {}), ("q4", 64, dict(window=90, first_tokens=5)),
                               ("bf16", 128, {}), ("q8", 256, {}), ("vq8", 64, {}))]
    cfgs = [config(n_q_heads=16, n_kv_heads=4, **k) for k in kinds]
    batch, cap, longest = 3, 1024, 40
    need = [B.uaa_workspace_size(B.make_desc(c), batch, cap - 1, 0, longest) for c in cfgs]
    shared = torch.zeros(max(need), dtype=torch.uint8, device="cuda")
    own = [DecodeLayer(c, batch, cap, max_q_len=longest) for c in cfgs]
    one = [DecodeLayer(c, batch, cap, max_q_len=longest, workspace=shared) for c in cfgs]
    assert all(x.ws_tensor is shared for x in one) and own[0].ws_tensor.numel() == need[0]
    assert DecodeLayer(cfgs[0], batch, cap, max_q_len=longest, workspace=own[0].ws_tensor).ws.bytes == need[0]
    for i, T in enumerate((40, 1, 3, 1, 1, 40, *[1] * 3, 40, 40, 40, 40, 40, 40, 40, 40, 40, 40, 40, 40, 1, 4, 1)):
        for a, b, cfg in zip(own, one, cfgs):
            x = rows(cfg, batch, T, i)
            assert torch.equal(a.step(*x), b.step(*x)), (cfg["kv_dtype"], i, T)
    for a, b in zip(own, one):
        assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.seq_lens, b.seq_lens)
        assert a.device_status() == 0 and b.device_status() == 0
    for bad in (shared[:need[0] - 1], shared.view(torch.int8), shared.cpu(), shared.repeat(2)[::2], shared.view(-1, 2)):
        with pytest.raises(ValueError, match="workspace"):
            DecodeLayer(cfgs[0], batch, cap, max_q_len=longest, workspace=bad)
    with pytest.raises(B.UaaError, match="16-byte aligned"):
        layer = DecodeLayer(cfgs[5], batch, cap, workspace=shared[8:])
        layer.step(*rows(cfgs[5], batch, 1, 0))


def test_fixed_parts_take_nothing_from_the_built_in_scratch():
    """Every step whose arrays fitted 8 MiB beside a range balance of its own size fits
    the built-in scratch, whose fixed parts are sized for the largest grid."""
    al = lambda x: (x + 255) // 256 * 256
    tight = 0
    for kv, D, heads, kv_heads in (("bf16", 128, 32, 8), ("q4", 64, 64, 8), ("vq8", 64, 64, 8), ("f32", 64, 32, 8),
                                   ("q8", 256, 16, 8)):
        d = B.make_desc(config(kv_dtype=kv, head_dim=D, n_q_heads=heads, n_kv_heads=kv_heads))
        for n_sm in (148, 152):
            for batch in range(1, 700):
                lay = B.uaa_get_workspace_layout(d, batch, 4000, n_sm, 1)
                P = lay.n_ctas
                own = 256 + 256 + al(8 * P) + 2 * al(4 * P) + al(4 * (P + 1)) + lay.total_bytes - lay.q_rot_offset
                if own <= 8 << 20:
                    assert lay.total_bytes <= B.UAA_STATIC_SCRATCH_BYTES
                    tight += lay.total_bytes > 8 << 20
    assert tight > 0
