"""The 4-bit cache (kv_dtype q4): its quantiser, the append's codes, attention over
it in every form, and the reader of cached rows, against plain64.

Attention tolerance: q' and the softmax weights enter the tensor core as one fp16
part each, a relative error of at most 2^-11 (fp16 eps / 2); keys and values are
exact (code * scale). A logit is a sum of D terms whose magnitudes add up to less
than about 8 here (D = 128: 128 E|q k| / sqrt(128) = 7.2), so it is off by at most
8 * 2^-11 = 4e-3, and by a few 1e-4 as the D errors average; an output row is off
by the weighted mean of those times values of size ~1, and by 2^-11 of itself for
the weights: 4e-3 at most, 4e-4 in the mean. A bf16 output adds half a step.
"""
import pytest
import torch

from gqa_attention_kv_qk_gb300 import binding as B
from gqa_attention_kv_qk_gb300 import workloads as W
from tests import plain64
from tests.test_abi_host import WS, fake_args

TOL_MAX, TOL_MEAN = 4e-3, 4e-4


def config(**kw):
    cfg = dict(n_q_heads=8, n_kv_heads=2, head_dim=128, kv_dtype="q4", io_dtype="bf16", out_dtype="f32",
               rope_style="neox", rope_theta=10000.0, seed=31, batch=1, seq_len=64)
    cfg.update(kw)
    return cfg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gqa_attention_kv_qk_gb300 import build
    build.build()


# ---------------------------------------------------------------- on the host

def test_step_refusals():
    d = B.make_desc(config())
    a = fake_args(k_scale=0x10000, v_scale=None)
    assert B.uaa_decode_attn(d, a, WS, None, check=False) == B.UAA_ERR_INVALID_ARGUMENT
    assert "v_scale is NULL" in B.last_error()
    a = fake_args(k_scale=None)
    assert B.uaa_decode_attn(d, a, WS, None, check=False) == B.UAA_ERR_INVALID_ARGUMENT
    assert "k_scale is NULL" in B.last_error()
    a = fake_args(k_scale=0x10000, block_table=0x10000, page_size=16, pages_per_seq=8, n_pages=16)
    assert B.uaa_decode_attn(d, a, WS, None, check=False) == B.UAA_ERR_UNSUPPORTED
    assert "page_size=16 is below 32" in B.last_error()
    # a stage of 256 keys that holds the last one must not pass 2^31
    d, cap = B.make_desc(config(n_kv_heads=1)), 2**31 - 256
    for a, fact in ((fake_args(k_scale=0x10000, batch=1, cache_capacity=cap), f"cache_capacity={cap}"),
                    (fake_args(k_scale=0x10000, block_table=0x10000, page_size=32, pages_per_seq=cap // 32, n_pages=8,
                               cache_capacity=cap), f"cache_capacity={cap}"),
                    (fake_args(k_scale=0x10000, batch=2, cache_capacity=cap // 2), "exceeds 2^31")):
        assert B.uaa_decode_attn(d, a, WS, None, check=False) == B.UAA_ERR_UNSUPPORTED
        assert fact in B.last_error()


def test_quantize_refusals():
    ok = (0x10000, 0, 4, 64, 0x10000, 0x10000)
    for bad, status, fact in (((0x10000, 0, 4, 96, 0x10000, 0x10000), B.UAA_ERR_UNSUPPORTED, "head_dim=96"),
                              ((0x10000, 4, 4, 64, 0x10000, 0x10000), B.UAA_ERR_UNSUPPORTED, "x_dtype=4"),
                              ((0x10000, 0, -1, 64, 0x10000, 0x10000), B.UAA_ERR_INVALID_ARGUMENT, "n_rows=-1"),
                              ((0, 0, 4, 64, 0x10000, 0x10000), B.UAA_ERR_INVALID_ARGUMENT, "NULL"),
                              ((0x10000, 0, 4, 64, 0x10008, 0x10000), B.UAA_ERR_INVALID_ARGUMENT, "aligned")):
        assert B.uaa_q4_quantize(*bad, None, check=False) == status
        assert fact in B.last_error()
    assert B.uaa_q4_quantize(*ok[:2], 0, *ok[3:], None, check=False) == B.UAA_OK


def test_read_refusals():
    d = B.make_desc(config())
    a = fake_args(k_scale=0x10000)
    for args, n, k, status, fact in ((a, -1, 0x10000, B.UAA_ERR_INVALID_ARGUMENT, "n_rows=-1"),
                                     (a, 1, 0x10004, B.UAA_ERR_INVALID_ARGUMENT, "outputs must be 16-byte aligned"),
                                     (fake_args(), 1, 0x10000, B.UAA_ERR_INVALID_ARGUMENT, "k_scale is NULL"),
                                     (fake_args(cache_capacity=6), 1, 0x10000, B.UAA_ERR_INVALID_ARGUMENT,
                                      "cache_capacity=6")):
        assert B.uaa_cache_read(d, args, 0x10000, n, k, 0x10000, None, check=False) == status
        assert fact in B.last_error()
    assert B.uaa_cache_read(d, a, 0, 0, 0x10000, 0x10000, None, check=False) == B.UAA_OK
    assert B.uaa_cache_read(d, a, 0, 5, 0, 0, None, check=False) == B.UAA_OK


def test_geometry():
    for D, keys, per_sm in ((64, 256, 2), (128, 256, 2), (256, 128, 1)):
        lay = B.uaa_get_workspace_layout(B.make_desc(config(head_dim=D)), 4, 100, 152)
        assert (lay.kernel, lay.stage_keys, lay.n_ctas) == (1, keys, 152 * per_sm)


def test_plain_values_are_within_half_a_step():
    x = torch.randn(50, 128, generator=torch.Generator().manual_seed(3)) * torch.logspace(-3, 3, 50).unsqueeze(1)
    codes, s = plain64.q4_quantize(x)
    step = s.double().repeat_interleave(32, -1)
    # a scale is rounded by up to 2^-9, so the largest value may lie 7 * 2^-9 steps beyond code 7.5's reach
    assert ((codes.double() * step - x.double()).abs() <= step * (0.5 + 7 * 2.0 ** -8)).all()


# ---------------------------------------------------------------- the quantiser

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,rows", [(64, 1), (64, 333), (128, 1000), (256, 77), (128, 200_001)])
def test_quantize(D, rows, dtype):
    g = torch.Generator().manual_seed(D + rows)
    x = torch.randn(rows, D, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    x[0, :32] = 0.0                                   # a group of zeros
    x[0, 32] = 7.0                                    # integers on the codes' grid, and ties
    x[0, 33:40] = torch.tensor([0.5, 1.5, -2.5, 3.5, 6.5, -6.5, 7.0])
    if rows > 9:
        x[1] *= 1e-9                                  # scales that are fp16 subnormals, or zero
        x[2] *= 1e-6
        x[3] = 1e6                                    # beyond the largest scale: saturates
        x[4, 5] = float("inf")
        x[5] = 0.0
        x[6, 0] = 1e-38
    x = x.to(dtype)
    dev = x.cuda()
    codes = torch.full((rows, D // 2), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, D // 32), 99.0, dtype=torch.float16, device="cuda")
    B.uaa_q4_quantize(dev.data_ptr(), B.DTYPE["f32" if dtype == torch.float32 else "bf16"], rows, D,
                      codes.data_ptr(), scales.data_ptr(), torch.cuda.current_stream())
    want, s = plain64.q4_quantize(x)
    assert torch.equal(scales.cpu(), s)
    assert torch.equal(plain64.q4_nibbles(codes), want)


# ---------------------------------------------------------------- the step

CASES = {
    "first-token": (dict(batch=3), [0, 1, 63], 1, 0),
    "tile-boundaries": (dict(batch=4), [63, 64, 127, 255], 1, 0),
    "last-slot": (dict(batch=2), [255, 127], 1, 0),
    "d64": (dict(head_dim=64), [500, 64, 3], 1, 0),
    "d64-long": (dict(head_dim=64, n_q_heads=16), [5000, 1], 1, 0),
    "d256": (dict(head_dim=256), [500, 64, 3], 1, 0),
    "mha": (dict(n_q_heads=4, n_kv_heads=4), [300, 77], 1, 0),
    "g8-bf16-out": (dict(n_q_heads=16, out_dtype="bf16"), [1000, 77], 1, 0),
    "g16": (dict(n_q_heads=32), [300, 77], 1, 0),
    "g20-two-groups": (dict(n_q_heads=20, n_kv_heads=1), [300, 77], 1, 0),
    "d256-g16": (dict(n_q_heads=16, n_kv_heads=1, head_dim=256), [300], 1, 0),
    "many": (dict(), [0, 5, 700, 64, 128, 129, 31, 32, 33, 1500, 2, 1], 1, 0),
    "window": (dict(window=100), [700, 100, 99, 20], 1, 0),
    "window-first": (dict(window=70, first_tokens=5), [700, 75, 76, 74, 20], 1, 0),
    "softcap-sink": (dict(softcap=5.0, has_sink=True), [700, 20], 1, 0),
    "qknorm-offset": (dict(qk_norm=True, norm_offset=True, norm_w_range=(-0.5, 0.5)), [300, 20], 1, 0),
    "interleaved": (dict(rope_style="interleaved"), [300, 0], 1, 0),
    "rotary96": (dict(rotary_dim=96), [300, 20], 1, 0),
    "rotary48-d64": (dict(rotary_dim=48, head_dim=64), [300, 20], 1, 0),
    "f32-io": (dict(io_dtype="f32"), [300, 20], 1, 0),
    "chunk2": (dict(), [0, 63, 300], 2, 0),
    "chunk4-window": (dict(window=3), [254, 2], 4, 0),
    "chunk5-first": (dict(window=70, first_tokens=66), [500, 136, 135], 5, 0),
    "chunk33-d64": (dict(head_dim=64, n_q_heads=16), [200, 0], 33, 0),
    # 24-row units (head_dim 64): one, a part of one, two, and a second one with a few rows
    "chunk3-d64-g8": (dict(head_dim=64, n_q_heads=16, has_sink=True), [700, 255, 0, 62], 3, 0),
    "chunk5-d64-g4-window": (dict(head_dim=64, window=9), [300, 4], 5, 0),
    "chunk6-d64-g8-first": (dict(head_dim=64, n_q_heads=16, window=100, first_tokens=30), [500, 130, 129], 6, 0),
    "chunk10-d64-g4-paged32": (dict(head_dim=64), [300, 60], 10, 32),
    "d64-mha-chunk20": (dict(head_dim=64, n_q_heads=2), [300, 60], 20, 0),
    "d64-g20": (dict(head_dim=64, n_q_heads=40, softcap=9.0), [300, 60], 1, 0),
    "chunk7-d256-norm": (dict(head_dim=256, qk_norm=True, norm_w_range=(0.5, 1.5)), [100, 3], 7, 0),
    "chunk3-interleaved-f32": (dict(rope_style="interleaved", io_dtype="f32", rotary_dim=64), [100, 3], 3, 0),
    "chunk3-rotary96": (dict(rotary_dim=96), [100, 3], 3, 0),     # halves of 48: the row-per-warp append
    "chunk3-rotary64": (dict(rotary_dim=64), [100, 3], 3, 0),     # halves of 32 and dims that pass
    "chunk160": (dict(n_q_heads=4), [90, 0], 160, 0),
    "paged32": (dict(), [500, 31, 32, 0], 1, 32),
    "paged32-d64-window": (dict(head_dim=64, window=37), [500, 20], 1, 32),
    "paged256-first": (dict(window=300, first_tokens=40), [1500, 340, 341], 1, 256),
    "paged64-chunk9-d256": (dict(head_dim=256), [300, 60], 9, 64),
    # 128 (token, head) rows and more per kv head: widened rows and the prefill kernel
    "prefill-window-sink": (dict(window=100, has_sink=True), [500, 0, 127], 40, 0),
    "prefill-first": (dict(window=150, first_tokens=100), [700, 250, 251, 252, 20], 33, 0),
    "prefill-d64-first-softcap": (dict(window=128, first_tokens=200, head_dim=64, softcap=20.0), [900, 328, 327], 64, 0),
    "prefill-paged32": (dict(), [300, 31, 0], 70, 32),
    "prefill-paged256-first-bf16": (dict(window=300, first_tokens=40, out_dtype="bf16"), [1500, 340, 341], 64, 256),
    "prefill-norm-interleaved": (dict(qk_norm=True, norm_w_range=(0.5, 1.5), rope_style="interleaved"), [130], 50, 0),
}


@pytest.mark.gpu
@pytest.mark.parametrize("entry", ["step", "split"])
@pytest.mark.parametrize("name", list(CASES))
def test_step(name, entry):
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    over, lens, T, page = CASES[name]
    cfg = config(**over)
    cfg.update(batch=len(lens), seq_len=max(lens), q_len=T, page_size=page)
    case = W.host_case(cfg, lens=lens)
    layer = DecodeLayer.for_case(case)
    win, first = cfg.get("window", 0), cfg.get("first_tokens", 0)
    if not page:  # scales of unused slots, and of rows that no token of the step sees, are NaN
        for b, n in enumerate(lens):
            lo = max(0, n + 1 - win) if win else 0
            for sc in (layer.k_scale, layer.v_scale):
                sc[b, :, n:] = float("nan")
                if lo > first:
                    sc[b, :, first:lo] = float("nan")
    before = {n: getattr(layer, n).clone() for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    dev = {k: case[k].cuda() for k in ("q", "k_new", "v_new")}
    Hq, Hkv, D = cfg["n_q_heads"], cfg["n_kv_heads"], cfg["head_dim"]
    shape = (len(lens), T, Hq, D)
    q_rot = torch.empty(shape, dtype=torch.float32, device="cuda")
    if entry == "step":
        out = layer.step(dev["q"], dev["k_new"], dev["v_new"], q_rot=q_rot)
    else:
        layer.append(dev["q"], dev["k_new"], dev["v_new"], q_rot=q_rot)
        layer.partial()
        out = layer.combine()
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    assert layer.seq_lens.cpu().tolist() == [n + T for n in lens]

    # the new rows: each value within half a step of the exact rotated row, its scale
    # within a bf16 rounding of max / 7 (fp32 rounding of the rotation on top: 2^-18)
    kn, qn = case["k_new"].reshape(len(lens), T, Hkv, D), case["q"].reshape(shape)
    if cfg.get("qk_norm"):
        off = 1.0 if cfg.get("norm_offset") else 0.0
        kn = plain64.rms_norm(kn, case["k_norm_w"], cfg.get("norm_eps", 1e-6), off)
        qn = plain64.rms_norm(qn, case["q_norm_w"], cfg.get("norm_eps", 1e-6), off)
    turn = dict(theta=cfg["rope_theta"], rotary_dim=cfg.get("rotary_dim", 0),
                interleaved=cfg["rope_style"] == "interleaved")
    kn, qn = plain64.rope_rows(kn, lens, **turn), plain64.rope_rows(qn, lens, **turn)
    assert torch.allclose(q_rot.double().cpu(), qn, rtol=2e-5, atol=2e-5)
    kv, vv = plain64.cached_values(layer)
    ks, vs = layer.logical("k_scale").double().cpu(), layer.logical("v_scale").double().cpu()
    vn = case["v_new"].reshape(len(lens), T, Hkv, D).double()
    for b, n in enumerate(lens):
        for got, sc, want in ((kv[b, :, n:n + T], ks[b, :, n:n + T], kn[b]), (vv[b, :, n:n + T], vs[b, :, n:n + T], vn[b])):
            want = want.transpose(0, 1)
            amax = want.unflatten(-1, (-1, 32)).abs().amax(-1)
            assert ((sc - amax / 7).abs() <= amax / 7 * (2.0 ** -8 + 2.0 ** -18)).all()
            step = sc.repeat_interleave(32, -1)
            # beyond code 7 by the scale's rounding: 7 * 2^-8 of a step
            assert ((got - want).abs() <= step * (0.5 + 7 * 2.0 ** -8) + want.abs() * 2.0 ** -18).all()
    # nothing else of the cache changed
    if not page:
        for b, n in enumerate(lens):
            for name_, old in before.items():
                new = getattr(layer, name_)
                keep = torch.ones(new.shape[2], dtype=torch.bool, device="cuda")
                keep[n:n + T] = False
                assert torch.equal(new[b][:, keep].view(torch.uint8 if new.dtype == torch.uint8 else torch.int16),
                                   old[b][:, keep].view(torch.uint8 if new.dtype == torch.uint8 else torch.int16))
    # the reader gives the rows as they are cached
    start = torch.tensor(lens, dtype=torch.int32, device="cuda")
    rk, rv = layer.read_rows(start, T)
    for b, n in enumerate(lens):
        half = torch.finfo(torch.bfloat16).eps / 2 if cfg["out_dtype"] == "bf16" else 0.0
        for got, x in ((rk, kv), (rv, vv)):
            w = x[b, :, n:n + T].transpose(0, 1)
            assert ((got[b].double().cpu() - w).abs() <= half * w.abs()).all()

    want = plain64.attend(q_rot, kv, vv, lens, win, first, cfg.get("softcap", 0.0), case["sink"])
    got = out.double().cpu().reshape(shape)
    assert torch.isfinite(got).all()
    err = (got - want).abs()
    if cfg["out_dtype"] == "bf16":
        err = (err - want.abs() * torch.finfo(torch.bfloat16).eps / 2).clamp(min=0)
    assert float(err.max()) <= TOL_MAX, float(err.max())
    assert float(err.mean()) <= TOL_MEAN, float(err.mean())


@pytest.mark.gpu
def test_prefill_in_batch_slices():
    """More widened rows than the workspace holds at once: the sequences go through it
    some at a time, and give what each gives alone."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    lens, T = [30, 0, 200, 64, 127, 128, 129, 1, 77], 40
    cfg = config(n_q_heads=32, n_kv_heads=8, batch=len(lens), seq_len=max(lens), q_len=T)
    lay = B.uaa_get_workspace_layout(B.make_desc(cfg), len(lens), 16000, 0, T)
    assert lay.kernel == 2 and lay.step_kernels == 1 + 2 * 2
    case = W.host_case(cfg, lens=lens)
    one = DecodeLayer.for_case(case)
    big = DecodeLayer(cfg, len(lens), 16000 + 64, max_q_len=T)
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        getattr(big, n)[:, :, :case["cap"]] = getattr(one, n)
    big.seq_lens.copy_(one.seq_lens)
    dev = {k: case[k].cuda() for k in ("q", "k_new", "v_new")}
    want = one.step(dev["q"], dev["k_new"], dev["v_new"]).clone()
    got = big.step(dev["q"], dev["k_new"], dev["v_new"], max_seq_len=16000)
    torch.cuda.synchronize()
    assert one.device_status() == 0 and big.device_status() == 0
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_prefill_beyond_the_length_bound():
    """A sequence longer than max_seq_len has no room for its widened rows: flagged, its
    rows are zero, the others as they are."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    lens, T = [500, 30], 64
    cfg = config(batch=2, seq_len=500, q_len=T)
    case = W.host_case(cfg, lens=lens)
    a, b = DecodeLayer.for_case(case), DecodeLayer.for_case(case)
    dev = {k: case[k].cuda() for k in ("q", "k_new", "v_new")}
    want = a.step(dev["q"], dev["k_new"], dev["v_new"]).clone()
    got = b.step(dev["q"], dev["k_new"], dev["v_new"], max_seq_len=100)
    torch.cuda.synchronize()
    assert a.device_status() == 0 and b.device_status() == B.UAA_DEVFLAG_LEN_HINT
    assert torch.equal(got[1], want[1]) and not got[0].any()
    assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.seq_lens, b.seq_lens)


@pytest.mark.gpu
def test_codes_of_the_append_and_the_quantiser_agree():
    """Value rows are stored as given: the append's codes are the quantiser's, bit for
    bit, from the fused step, the separate append and a chunk's append."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    for T, entry in ((1, "step"), (1, "append"), (5, "append")):
        cfg = config(batch=3, seq_len=100, q_len=T)
        case = W.host_case(cfg, lens=[100, 0, 63])
        layer = DecodeLayer.for_case(case)
        dev = {k: case[k].cuda() for k in ("q", "k_new", "v_new")}
        getattr(layer, entry)(dev["q"], dev["k_new"], dev["v_new"])
        torch.cuda.synchronize()
        want, s = plain64.q4_quantize(case["v_new"].reshape(3, T, 2, 128))
        for b, n in enumerate([100, 0, 63]):
            assert torch.equal(layer.v_scale[b, :, n:n + T].cpu(), s[b].transpose(0, 1))
            assert torch.equal(plain64.q4_nibbles(layer.v_cache[b, :, n:n + T]), want[b].transpose(0, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["f32", "bf16", "vq8", "q8", "q4"])
@pytest.mark.parametrize("page", [0, 32])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_read_rows(kv, page, out):
    """Every cache kind, positions that start before 0 or end past the capacity, and
    pages that are not in the table (zeros)."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    cfg = config(kv_dtype=kv, batch=3, seq_len=100, page_size=page, out_dtype=out,
                 io_dtype="f32" if kv == "f32" else "bf16", head_dim=64)
    case = W.host_case(cfg, lens=[100, 7, 64])
    layer = DecodeLayer.for_case(case)
    k, v = plain64.cached_values(layer)
    cap, n = case["cap"], 50
    if page:
        layer.block_table[0, 1] = -1
        layer.block_table[1, 0] = layer.n_pages
        k[0, :, 32:64] = v[0, :, 32:64] = 0.0
        k[1, :, :32] = v[1, :, :32] = 0.0
    start = [20, -3, cap - 10]
    rk, rv = layer.read_rows(torch.tensor(start, dtype=torch.int32, device="cuda"), n)
    assert rk.shape == (3, n, 2, 64) and rk.dtype == (torch.float32 if out == "f32" else torch.bfloat16)
    half = torch.finfo(torch.bfloat16).eps / 2 if out == "bf16" else 2.0 ** -24
    for b in range(3):
        for t in range(n):
            p = start[b] + t
            for got, x in ((rk, k), (rv, v)):
                w = x[b, :, p] if 0 <= p < cap else torch.zeros(2, 64, dtype=torch.float64)
                assert ((got[b, t].double().cpu() - w).abs() <= half * w.abs()).all()
    rk, rv = layer.read_rows(None, cap)  # whole caches from 0
    assert ((rk.transpose(1, 2).double().cpu() - k).abs() <= half * k.abs()).all()
    with pytest.raises(ValueError, match="start"):
        layer.read_rows(torch.zeros(2, dtype=torch.int32, device="cuda"), 1)


@pytest.mark.gpu
def test_reads_keep_their_tensors():
    """A captured read writes its pair at every replay, whatever was read since: the
    layer never lets go of a pair. Row counts past the sixteenth get new tensors."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    layer = DecodeLayer.for_case(W.host_case(config(batch=2, seq_len=60), lens=[60, 3]))
    first = layer.read_rows(None, 1)[0].data_ptr()
    pairs = [layer.read_rows(None, n) for n in range(1, 40)]
    assert layer.read_rows(None, 1)[0].data_ptr() == first and layer.read_rows(None, 16)[0] is pairs[15][0]
    a, b = layer.read_rows(None, 30), layer.read_rows(None, 30)
    assert a[0] is not b[0] and all(torch.equal(x, y) for x, y in zip(a, b))
    start = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="on the device"):
        layer.read_rows(start, 1)


@pytest.mark.gpu
def test_parameters_set_between_steps():
    """A step takes the sink and the norm weights of the last set_params."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    cfg = config(batch=2, seq_len=60, has_sink=True, qk_norm=True)
    case = W.host_case(cfg, lens=[60, 3])
    dev = {k: case[k].cuda() for k in ("q", "k_new", "v_new")}
    a, b = DecodeLayer.for_case(case), DecodeLayer.for_case(case)
    a.step(dev["q"], dev["k_new"], dev["v_new"], advance_hint=False)
    a.load_cache(case["k_values"], case["v_values"], case["lens"])
    other = dict(q_norm_w=case["q_norm_w"] * 0.5, k_norm_w=case["k_norm_w"] * 1.5, sink=case["sink"] + 2.0)
    for layer in (a, b):
        layer.set_params(**other)
    oa, ob = (x.step(dev["q"], dev["k_new"], dev["v_new"]) for x in (a, b))
    assert torch.allclose(oa, ob, atol=1e-6)  # ranges may be cut elsewhere


@pytest.mark.gpu
def test_own_cache_tensors():
    """A layer works on the caller's tensors in place, and refuses ones that do not fit."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    cfg = config(batch=2, seq_len=60)
    case = W.host_case(cfg, lens=[60, 3])
    a = DecodeLayer.for_case(case)
    own = {n: getattr(a, n).clone() for n in ("k_cache", "v_cache", "k_scale", "v_scale", "seq_lens")}
    b = DecodeLayer(cfg, 2, case["cap"], cache=own)
    dev = {k: case[k].cuda() for k in ("q", "k_new", "v_new")}
    assert b.max_len_hint == 60  # of the caller's lengths
    oa, ob = a.step(dev["q"], dev["k_new"], dev["v_new"]), b.step(dev["q"], dev["k_new"], dev["v_new"])
    assert torch.allclose(oa, ob, atol=1e-6)  # ranges may be cut elsewhere
    for n, t in own.items():
        assert getattr(b, n) is t and torch.equal(t, getattr(a, n))
    for name, bad in (("k_cache", own["k_cache"].view(torch.int8)), ("v_scale", own["v_scale"][:, :, :4]),
                      ("seq_lens", own["seq_lens"].cpu()), ("k_cache", own["k_cache"].transpose(2, 3))):
        with pytest.raises(ValueError, match=name):
            DecodeLayer(cfg, 2, case["cap"], cache={**own, name: bad})
    with pytest.raises(ValueError, match="k_scale"):
        DecodeLayer(dict(cfg, kv_dtype="bf16"), 2, case["cap"], cache=dict(k_scale=own["k_scale"]))


@pytest.mark.gpu
def test_captured_and_replayed():
    """Steps captured into a graph, on a side stream, give what eager ones give
    (uniform ranges: the same bits), also when another layer's graph is replayed
    between them."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    cfg = config(batch=3, seq_len=400, reproducible=True)
    case = W.host_case(cfg, lens=[390, 0, 64])
    eager, graph = DecodeLayer.for_case(case), DecodeLayer.for_case(case)
    other = DecodeLayer.for_case(case)
    dev = {k: case[k].cuda() for k in ("q", "k_new", "v_new")}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        for layer in (graph, other):
            lens0 = layer.seq_lens.clone()
            layer.step(dev["q"], dev["k_new"], dev["v_new"], max_seq_len=399, advance_hint=False)
            layer.seq_lens.copy_(lens0)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                layer.step(dev["q"], dev["k_new"], dev["v_new"], max_seq_len=399, advance_hint=False)
            graphs.append(g)
    torch.cuda.synchronize()
    for step in range(3):
        want = eager.step(dev["q"], dev["k_new"], dev["v_new"], max_seq_len=399, advance_hint=False)
        with torch.cuda.stream(stream):
            graphs[0].replay()
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(graph.out, want) and torch.equal(other.out, want)
        assert torch.equal(graph.seq_lens, eager.seq_lens)
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        assert torch.equal(getattr(graph, n), getattr(eager, n))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 64])
def test_steps_of_different_lengths_in_turn(D, page):
    """One layer and workspace through prefill chunks, draft tokens and single tokens
    (other kernels, grids and workspace layouts in turn), from an empty cache."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    Bn, cap = 3, 512
    cfg = config(batch=Bn, seq_len=0, head_dim=D, n_q_heads=16, first_tokens=9, window=200)
    layer = DecodeLayer(cfg, Bn, cap, page_size=page, max_q_len=150)
    g = torch.Generator().manual_seed(D + page)
    n = 0
    for T in (64, 1, 3, 2, 1, 150, 5, 1, 33, 8, 1, 1, 16):
        shape = lambda h: (Bn, T, h, D) if T > 1 else (Bn, h, D)
        q, k, v = (torch.randn(shape(h), generator=g).to(torch.bfloat16).cuda() for h in (16, 2, 2))
        q_rot = torch.empty((Bn, T, 16, D), dtype=torch.float32, device="cuda")
        out = layer.step(q, k, v, q_rot=q_rot)
        torch.cuda.synchronize()
        assert layer.device_status() == 0
        kk, vv = plain64.cached_values(layer)
        want = plain64.attend(q_rot, kk, vv, [n] * Bn, 200, 9)
        err = (out.double().cpu().reshape(want.shape) - want).abs()
        assert float(err.max()) <= TOL_MAX and float(err.mean()) <= TOL_MEAN, T
        n += T
        assert layer.seq_lens.tolist() == [n] * Bn


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3])
def test_static_scratch(T):
    """uaa_decode_attn_static over a 4-bit cache under a window with first tokens."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    cfg = config(batch=3, seq_len=300, q_len=T, window=100, first_tokens=7, reproducible=True)
    case = W.host_case(cfg, lens=[290, 0, 107])
    a, b = DecodeLayer.for_case(case), DecodeLayer.for_case(case)
    dev = {k: case[k].cuda() for k in ("q", "k_new", "v_new")}
    want = a.step(dev["q"], dev["k_new"], dev["v_new"])
    b._begin(dev["q"])
    B.uaa_decode_attn_static(b.desc, b.args(dev["q"], dev["k_new"], dev["v_new"]), torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(b.out_for(T), want) and torch.equal(a.k_cache, b.k_cache) and torch.equal(a.v_scale, b.v_scale)
    big = config(batch=3, seq_len=300, q_len=200)  # a prefill chunk's widened rows do not fit the built-in scratch
    c = DecodeLayer.for_case(W.host_case(big, lens=[9, 0, 7]))
    q = torch.zeros((3, 200, 8, 128), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((3, 200, 2, 128), dtype=torch.bfloat16, device="cuda")
    c._begin(q)
    args = c.args(q, kv, kv, max_seq_len=32000 - 200)
    args.cache_capacity = 32000
    st = B.uaa_decode_attn_static(c.desc, args, torch.cuda.current_stream(), check=False)
    assert st == B.UAA_ERR_INVALID_ARGUMENT and "built-in scratch" in B.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["prefill", "decode"])
def test_long_tail_behind_a_dominant_key(kind):
    """One key holds almost all of a row's mass and the rest lies in a long tail of equal
    weights of w = 2^-24.8 of it: fp16 weights relative to the dominant one would round
    each to 2^-24, 1.7 times as much.

    Values are 7 in the tail and 0 at the dominant key, so the output is 7 r / (1 + r)
    with r = n w. Tolerance: a tail weight's own rounding (2^-11 of it) and that of q'
    (2^-11 of a logit of 24.8 in log2, times ln 2: 17.2 times as much) move r by
    r 2^-11 18.2; fp32 sums of equal terms over 2^13 accumulations by r 2^-11 at most."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    if kind == "prefill":
        Bn, Hkv, n, T = 1, 1, 2 ** 17, 128     # the query-tiled kernel
    else:                                      # as many units as ranges: each range is a whole unit
        Hkv, n, T = 8, 2 ** 15, 1
        Bn = 2 * torch.cuda.get_device_properties(0).multi_processor_count // Hkv
    cfg = config(n_q_heads=Hkv, n_kv_heads=Hkv, head_dim=64, rotary_dim=2, batch=Bn, reproducible=True)
    layer = DecodeLayer(cfg, Bn, n + 128, max_q_len=T)
    assert B.uaa_get_workspace_layout(layer.desc, Bn, n, 0, T).kernel == (2 if T > 1 else 1)
    layer.k_cache.fill_(0x88)                  # code 0
    layer.k_cache[:, :, 0, 1] = 0x8F           # the first key: 7 in dim 2, which no position turns
    layer.v_cache.fill_(0xFF)                  # code 7
    layer.v_cache[:, :, 0] = 0x88
    layer.k_scale.fill_(1.0)
    layer.v_scale.fill_(1.0)
    layer.set_lengths([n] * Bn)
    shape = (Bn, T, Hkv, 64) if T > 1 else (Bn, Hkv, 64)
    q, k, v = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    q[..., 2] = 19.625                         # 19.625 * 7 / sqrt(64) log2(e) = 24.77
    v.fill_(7.0)
    out = layer.step(q, k, v)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    keys, values = (torch.zeros(1, 1, n + T, 64, dtype=torch.float64) for _ in range(2))
    keys[:, :, 0, 2], values[:, :, 1:] = 7.0, 7.0
    for t in sorted({0, T // 2, T - 1}):
        want = float(plain64.attend(q[:1].reshape(1, T, Hkv, 64)[:, t:t + 1, :1], keys, values, [n + t])[0, 0, 0, 0])
        r = want / (7.0 - want)
        assert 0.9 * (n + t) * 2.0 ** -24.8 < r < 1.1 * (n + t) * 2.0 ** -24.7
        got = out.double().cpu().reshape(Bn, T, Hkv, 64)[:, t]
        assert float((got - want).abs().max()) <= 7 * r * 2.0 ** -11 * 19.2, (t, want, float(got.min()), float(got.max()))


@pytest.mark.gpu
@pytest.mark.parametrize("T,page,D", [(1, 0, 64), (1, 32, 128), (3, 0, 64), (3, 32, 64), (64, 0, 64)])
def test_batches_of_more_than_one_slice(T, page, D):
    """1,030 sequences: two launches of the split-K kernel, with sequences of the second
    one at every place of a window with first tokens."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    n = 1030
    lens = [(7 * b) % 90 for b in range(n)]
    cfg = config(n_q_heads=2, n_kv_heads=1, head_dim=D, batch=n, seq_len=90, q_len=T, page_size=page, window=20,
                 first_tokens=3)
    case = W.host_case(cfg, lens=lens)
    layer = DecodeLayer.for_case(case)
    assert layer.layout().n_slices == 2
    q_rot = torch.empty((n, T, 2, D), device="cuda")
    out = layer.step(*(case[k].cuda() for k in ("q", "k_new", "v_new")), q_rot=q_rot)
    torch.cuda.synchronize()
    assert layer.device_status() == 0 and layer.seq_lens.tolist() == [x + T for x in lens]
    k, v = plain64.cached_values(layer)
    some = sorted({*range(0, n, 37), *range(1015, 1030)})
    want = plain64.attend(q_rot[some], k[some], v[some], [lens[b] for b in some], 20, 3)
    err = (out.double().cpu().reshape(n, T, 2, D)[some] - want).abs()
    assert float(err.max()) <= TOL_MAX and float(err.mean()) <= TOL_MEAN


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,page", [(1, 256, 0), (3, 256, 0), (40, 128, 0), (1, 256, 64), (64, 128, 64)])
def test_rows_past_4_gib(T, D, page):
    """Sequences whose codes lie past 2^32 bytes of the cache (or on such pages of a pool)
    give what they give in a small cache; so does the reader, and a copy of such pages."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    Bn, Hkv, cap = 3, 8, 1024
    cfg = config(n_q_heads=32, n_kv_heads=Hkv, head_dim=D, batch=Bn, seq_len=500, q_len=T, page_size=page,
                 reproducible=True)
    lens = [500, 0, 77]
    case = W.host_case(cfg, lens=lens, cap=cap)
    small = DecodeLayer.for_case(case)
    rows = 2 ** 32 // (D // 2) + 10 * Hkv * cap        # past 2^32 bytes of codes
    if page:
        n = rows // (Hkv * page)
        table = torch.arange(n - Bn * cap // page, n, dtype=torch.int32).flip(0).reshape(Bn, -1)
        big = DecodeLayer(cfg, Bn, cap, page_size=page, block_table=table, n_pages=n, max_q_len=T)
        at = lambda x: x
    else:
        n = rows // (Hkv * cap)
        big = DecodeLayer(dict(cfg, batch=n), n, cap, max_q_len=T)
        at = lambda x: x[n - Bn:]
        big.seq_lens.fill_(-1)
    at(big.seq_lens).copy_(small.seq_lens)
    big.max_len_hint = small.max_len_hint
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        x = small.logical(name)
        if page:
            big._to_pool(x, getattr(big, name))
        else:
            at(getattr(big, name)).copy_(x)
    assert big.k_cache.numel() > 2 ** 32
    dev = {k: case[k].cuda() for k in ("q", "k_new", "v_new")}
    want = small.step(*dev.values())
    if not page:                                        # the other sequences are idle
        dev = {k: torch.cat((torch.zeros((n - Bn, *x.shape[1:]), dtype=x.dtype, device="cuda"), x)) for k, x in dev.items()}
    got = big.step(*dev.values())
    torch.cuda.synchronize()
    assert small.device_status() == 0 and big.device_status() == 0
    assert float((at(got) - want).abs().max()) <= TOL_MAX  # ranges are cut elsewhere
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        assert torch.equal(at(big.logical(name)), small.logical(name))
    for a, b in zip(small.read_rows(None, 600), big.read_rows(None, 600)):
        assert torch.equal(at(b), a)
    if page:
        from gqa_attention_kv_qk_gb300.pages import PageTable
        pages = PageTable(big.block_table, page, n, seq_lens=big.seq_lens)
        assert pages.block_table is big.block_table
        pages.compact()
        pages.copy_layer(big)
        assert pages.block_table.max() < Bn * cap // page and pages.device_status() == 0
        for a, b in zip(small.read_rows(None, 600), big.read_rows(None, 600)):
            assert torch.equal(b, a)
