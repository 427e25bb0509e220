"""A sliding window whose first tokens stay visible (uaa_attn_desc.first_tokens):
every kernel that attends, against the definition in 64 bits.

Tolerances are the parity bar of the attention outputs (max 2e-3, mean 2e-4 for
fp32 outputs of values ~N(0, 1)): the tensor-core kernels split q' and P into two
bf16 or fp16 parts (2^-16 relative), so a logit of a few units is off by less
than 1e-4 and an output by less than 1e-3 times the values' size. A bf16 output
adds half a step, 2^-8 relative.
"""
import pytest
import torch

from gqa_attention_kv_qk_gb300 import binding as B
from gqa_attention_kv_qk_gb300 import workloads as W
from tests import plain64

TOL_MAX, TOL_MEAN = 2e-3, 2e-4


def config(**kw):
    cfg = dict(n_q_heads=8, n_kv_heads=2, head_dim=128, kv_dtype="bf16", io_dtype="bf16", out_dtype="f32",
               rope_style="neox", rope_theta=10000.0, seed=21, batch=1, seq_len=64)
    cfg.update(kw)
    return cfg


def test_refusals():
    from gqa_attention_kv_qk_gb300 import build
    build.build()
    d = B.make_desc(config(window=16, first_tokens=-1))
    assert B.uaa_workspace_size(d, 1, 64, 152) == 0
    assert "first_tokens=-1 is negative" in B.last_error()
    for w, f in ((0, 4), (16, 0), (16, 4), (2**31 - 1, 2**31 - 1)):
        assert B.uaa_workspace_size(B.make_desc(config(window=w, first_tokens=f)), 1, 64, 152, 1) > 0


def test_visible_is_the_union():
    assert plain64.visible(9, 3, 2) == [0, 1, 7, 8, 9]
    assert plain64.visible(3, 3, 2) == [0, 1, 2, 3]      # the two runs meet
    assert plain64.visible(9, 0, 2) == list(range(10))   # no window
    assert plain64.visible(5, 3, 99) == list(range(6))


# (config, lengths before the step, tokens, page size)
CASES = {
    # runs apart, touching, overlapping, in one tile; one first token; first tokens in several tiles
    "bf16-decode": (dict(window=70, first_tokens=4), [500, 74, 75, 73, 3, 0], 1, 0),
    "bf16-one-each": (dict(window=1, first_tokens=1), [300, 1, 2, 0], 1, 0),
    "bf16-first-129-of-one-tile-more": (dict(window=64, first_tokens=129), [1000, 193, 194, 192, 257], 1, 0),
    "bf16-same-tile": (dict(window=200, first_tokens=20), [230, 256, 219, 220, 221], 1, 0),
    "bf16-d64-sink-g8": (dict(window=100, first_tokens=65, head_dim=64, n_q_heads=16, has_sink=True),
                         [700, 165, 166, 8], 1, 0),
    "bf16-d256-softcap": (dict(window=33, first_tokens=7, head_dim=256, softcap=20.0), [400, 39, 41], 1, 0),
    "bf16-g16": (dict(window=100, first_tokens=10, n_q_heads=32), [600, 110], 1, 0),
    "bf16-window-wider": (dict(window=4096, first_tokens=10), [600, 110], 1, 0),
    "bf16-first-wider": (dict(window=50, first_tokens=100000), [600, 110], 1, 0),
    "bf16-no-window": (dict(window=0, first_tokens=10), [600, 110], 1, 0),
    "vq8-decode": (dict(window=70, first_tokens=5, kv_dtype="vq8"), [500, 90], 1, 0),
    "vq8-d64-stage256": (dict(window=300, first_tokens=70, kv_dtype="vq8", head_dim=64), [1500, 371, 369, 300], 1, 0),
    "q8-decode": (dict(window=200, first_tokens=130, kv_dtype="q8"), [1000, 331], 1, 0),
    "f32-one-launch": (dict(window=600, first_tokens=77, kv_dtype="f32", io_dtype="f32"), [1500, 676, 678, 2], 1, 0),
    "f32-d256": (dict(window=9, first_tokens=2, kv_dtype="f32", io_dtype="f32", head_dim=256), [100, 11], 1, 0),
    "f32-chunk": (dict(window=9, first_tokens=3, kv_dtype="f32", io_dtype="f32"), [200, 12, 0], 5, 0),
    # chunks: rows whose windows start at different keys, chunks longer than the window
    "bf16-chunk4": (dict(window=70, first_tokens=4), [500, 72, 73, 74, 75, 0], 4, 0),
    "bf16-chunk20-window3": (dict(window=3, first_tokens=2), [500, 0, 5], 20, 0),
    "q8-chunk3": (dict(window=70, first_tokens=80, kv_dtype="q8"), [500, 150, 149], 3, 0),
    "vq8-d64-chunk6": (dict(window=129, first_tokens=1, kv_dtype="vq8", head_dim=64), [700, 130], 6, 0),
    # the query-tiled prefill kernel (128 rows and more per kv head)
    "prefill-apart": (dict(window=100, first_tokens=4), [1000, 0], 40, 0),
    "prefill-same-block": (dict(window=150, first_tokens=100), [250, 251, 252, 20], 33, 0),
    "prefill-d64-first-200": (dict(window=128, first_tokens=200, head_dim=64, has_sink=True), [900, 328, 327], 64, 0),
    "prefill-long": (dict(window=60, first_tokens=17, out_dtype="bf16"), [700], 300, 0),
    # paged: the pages between the first tokens and the window are gone from the table
    "paged16-bf16": (dict(window=70, first_tokens=20), [500, 90, 15], 1, 16),
    "paged64-vq8": (dict(window=70, first_tokens=65, kv_dtype="vq8"), [900, 199], 1, 64),
    "paged32-q8-chunk": (dict(window=100, first_tokens=33, kv_dtype="q8"), [900, 134], 4, 32),
    "paged128-f32": (dict(window=100, first_tokens=129, kv_dtype="f32", io_dtype="f32"), [900, 400], 1, 128),
    "paged32-prefill-rows": (dict(window=100, first_tokens=33), [900, 134], 40, 32),
}


@pytest.mark.gpu
@pytest.mark.parametrize("entry", ["step", "split"])
@pytest.mark.parametrize("name", list(CASES))
def test_first_tokens(name, entry):
    from gqa_attention_kv_qk_gb300 import build
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    build.build()
    over, lens, T, page = CASES[name]
    cfg = config(batch=len(lens), seq_len=max(lens), q_len=T, page_size=page, **over)
    case = W.host_case(cfg, lens=lens, fill_unused="nan")
    win, first = cfg["window"], cfg["first_tokens"]
    # rows that no token of the step sees hold NaN
    kinds = [("k_cache", "k_values"), ("v_cache", "v_values")]
    for b, n in enumerate(lens):
        lo = max(0, n + 1 - win) if win else 0
        for a, c in kinds:
            x = case[a] if a in case else case[c]
            if lo > first:
                x[b, :, first:lo] = float("nan")
    layer = DecodeLayer.for_case(case)
    # pages without a visible position leave the table
    if page:
        table = layer.block_table.cpu()
        for b, n in enumerate(lens):
            lo = max(0, n + 1 - win)
            for p in range(table.shape[1]):
                if (p * page >= first and (p + 1) * page <= lo) or p * page >= n + T:
                    table[b, p] = -1
        layer.block_table.copy_(table)
    dev = {k: case[k].cuda() for k in ("q", "k_new", "v_new")}
    shape = (len(lens), T, cfg["n_q_heads"], cfg["head_dim"])
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
    if page:
        layer.block_table.clamp_(min=0)  # for reading back; absent pages' rows are not used
    k, v = plain64.cached_values(layer)
    want = plain64.attend(q_rot, k, v, lens, win, first, cfg.get("softcap", 0.0), case["sink"])
    got = out.double().cpu().reshape(shape)
    assert torch.isfinite(got).all()
    err = (got - want).abs()
    half_step = want.abs() * torch.finfo(torch.bfloat16).eps / 2 if cfg["out_dtype"] == "bf16" else 0.0
    assert ((err - half_step) <= TOL_MAX).all(), float(err.max())
    assert float((err - half_step).clamp(min=0).mean()) <= TOL_MEAN


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["vq8", "q8"])
def test_long_tail_behind_a_first_token(kv):
    """The first token holds almost all of a row's mass, the window a long tail of equal
    weights of w = 2^-24.8 of it: as fp16 numbers relative to the first token's, hi + lo
    parts both end at 2^-24, and every tail weight was 1.7 times as large.

    Values are 127 s in the tail and 0 at the first token, so the output is
    127 s r / (1 + r) with r = n w. Tolerance: rounding q' to 16 bits moves a logit of
    24.8 (log2) by 24.8 2^-16, fp32 rounding of the products below that: r by r 2^-11 at
    most; the weights' hi + lo parts and fp32 sums of 2^13 equal terms: r 2^-11."""
    from gqa_attention_kv_qk_gb300 import build
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    build.build()
    Hkv, n = 8, 2 ** 15
    Bn = 2 * torch.cuda.get_device_properties(0).multi_processor_count // Hkv  # a range per unit
    cfg = config(kv_dtype=kv, n_q_heads=Hkv, n_kv_heads=Hkv, head_dim=64, rotary_dim=2, batch=Bn, reproducible=True,
                 window=n - 100, first_tokens=1)
    layer = DecodeLayer(cfg, Bn, n + 128)
    s = 1.0 / 127
    if kv == "q8":
        layer.k_scale.fill_(7.0 / 127)
        layer.k_cache[:, :, 0, 2] = 127        # dim 2, which no position turns
        key = float(torch.tensor(7.0 / 127)) * 127
    else:
        layer.k_cache[:, :, 0, 2] = 7.0
        key = 7.0
    layer.v_cache.fill_(127)
    layer.v_cache[:, :, 0] = 0
    layer.v_scale.fill_(s)
    layer.set_lengths([n] * Bn)
    q, k, v = (torch.zeros((Bn, Hkv, 64), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    q[..., 2] = 19.625                         # 19.625 * 7 / sqrt(64) log2(e) = 24.77
    v.fill_(1.0)
    out = layer.step(q, k, v)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    keys, values = (torch.zeros(1, 1, n + 1, 64, dtype=torch.float64) for _ in range(2))
    keys[:, :, 0, 2], values[:, :, 1:] = key, float(torch.tensor(s)) * 127
    want = float(plain64.attend(q[:1, None, :1], keys, values, [n], n - 100, 1)[0, 0, 0, 0])
    r = want / (1.0 - want)
    assert 0.9 * n * 2.0 ** -24.8 < r < 1.1 * n * 2.0 ** -24.7
    assert float((out.double().cpu() - want).abs().max()) <= r * 2.0 ** -10, (want, float(out.min()), float(out.max()))


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1e-36, 1e-33, 1e-30, 1e30])
def test_values_of_extreme_size(size):
    """vq8 scales near the smallest fp32 numbers, where they are taken relative to the
    smallest normal one, and huge ones. Outputs are within 2^-10 of the largest value:
    the weights' parts (2^-16) and, for scales below 2^-112, half of fp32's smallest
    step against outputs 100 times as large and more."""
    from gqa_attention_kv_qk_gb300 import build
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    build.build()
    lens = [300, 5, 64]
    cfg = config(kv_dtype="vq8", batch=3, seq_len=300, window=90, first_tokens=3)
    case = W.host_case(cfg, lens=lens)
    case["v_values"] *= size
    layer = DecodeLayer.for_case(case)
    v_new = (case["v_new"].double() * size).to(torch.bfloat16).cuda()
    q_rot = torch.empty((3, 1, 8, 128), device="cuda")
    out = layer.step(case["q"].cuda(), case["k_new"].cuda(), v_new, q_rot=q_rot)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    k, v = plain64.cached_values(layer)
    want = plain64.attend(q_rot, k, v, lens, 90, 3)
    err = (out.double().cpu().reshape(want.shape) - want).abs()
    assert torch.isfinite(out).all() and float(err.max()) <= float(v.abs().max()) * 2.0 ** -10
