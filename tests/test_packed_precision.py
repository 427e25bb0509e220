"""How near the packed steps come to 64 bits: bf16 outputs against half a step of their own
rounding, appended keys against theirs, keys that are infinite."""
import math

import pytest
import torch

from tests import plain64
from tests.test_packed import expected, make_plan, make_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gqa_attention_kv_qk_gb300 import build
    build.build()


def half_step(x):
    """Half a bf16 step of values up to |x|: 2^-8 of the power of two at or below it."""
    return 2.0 ** -8 * 2.0 ** x.abs().clamp(min=1e-30).log2().floor()


def slack_before_rounding(cfg, s, q_rot):
    """A bound on the fp32 output's error, per element. With A the softmax's mean of |v|: the weights
    enter in two bf16 parts, off by less than 2^-14 of each, so by 2^-14 A together;
    q' enters in two bf16 parts, 2^-16, its rotation and the sums in fp32 are far below another
    2^-16, so a logit is off by at most z = 2^-15 sum |q k| / sqrt D, a weight by z of itself, and
    numerator and denominator together by 2 z A; exp2, the scales of 8-bit caches and the fp32 sums of
    a few dozen weights stay below 2^-18 A."""
    layer = s["layer"]
    keys, values = plain64.cached_values(layer)
    G, D = cfg["n_q_heads"] // cfg["n_kv_heads"], cfg["head_dim"]
    sink = layer.sink.cpu() if layer.sink is not None else None
    slack, r = torch.zeros_like(q_rot), 0
    for b, (n, T) in enumerate(zip(s["lens"], s["new"])):
        rows = slice(r, r + T)
        q = q_rot[rows]
        a = plain64.attend(q.unsqueeze(0), keys[b:b + 1, :, :n + T], values[b:b + 1, :, :n + T].abs(), [n], sink=sink)[0]
        k = keys[b, :, :n + T].abs().repeat_interleave(G, 0)  # [Hq][n + T][D]
        z = 2.0 ** -15 * torch.einsum("thd,hjd->thj", q.abs(), k).amax(-1, keepdim=True) / math.sqrt(D)
        slack[rows] = a * (2.0 ** -14 + 2.0 ** -18 + 2 * z)
        r += T
    return slack


@pytest.mark.parametrize("kv,D,G", [("bf16", 64, 4), ("bf16", 128, 4), ("vq8", 64, 8), ("q8", 128, 2), ("bf16", 128, 40)])
def test_bf16_outputs_are_rounded_once(kv, D, G):
    """Few keys a row, so that the roundings of single weights would show: an output is the 64-bit
    value rounded to bf16, but for the slack above. (One bf16 part of the weights leaves 7 to 23 %
    of the elements outside.)"""
    cfg = dict(n_q_heads=2 * G, n_kv_heads=2, head_dim=D, kv_dtype=kv, io_dtype="bf16", out_dtype="bf16", rope_theta=10000.0,
               has_sink=G == 8)
    requests = [(2, 1), (0, 3), (5, 2), (1, 1), (3, 6), (0, 2), (7, 1), (2, 2), (4, 1), (0, 9)]
    s = make_step(cfg, requests, 64, page=32, seed=D + G)
    plan = make_plan(s)
    out = s["layer"].step_packed(s["q"], s["k"], s["v"], plan).double().cpu()
    want, q_rot, _ = expected(cfg, s)
    slack = slack_before_rounding(cfg, s, q_rot)
    err = (out - want).abs()
    assert bool((err <= half_step(want.abs() + slack) + slack).all()), float((err > half_step(want.abs() + slack) + slack).double().mean())


@pytest.mark.parametrize("style", ["neox", "interleaved"])
def test_bf16_keys_with_a_norm_are_rounded_once(style):
    """A million appended elements: each the exact key rounded to bf16, but for the fp32 value's own
    error. cos and sin are sums of two floats within 2^-26, so the pair (a, b) is off by at most
    2^-26 (|a| + |b|) <= 2^-25 of its length; norm, products and sums of two floats are off by far less;
    and the value is rounded to fp32 first, 2^-24. (Norm and rotation in plain fp32 are off by some
    2^-22 of the length, and dozens of these elements land outside.)"""
    cfg = dict(n_q_heads=8, n_kv_heads=8, head_dim=128, kv_dtype="bf16", io_dtype="bf16", out_dtype="f32", rope_theta=10000.0,
               rope_style=style, qk_norm=True)
    s = make_step(cfg, [(0, 600), (400, 400)], 1024, page=32, seed=11)
    plan = make_plan(s)
    s["layer"].append_packed(s["q"], s["k"], s["v"], plan)
    k = s["layer"].read_packed(plan)[0].double().cpu()
    from tests.test_packed import pair_positions, turned
    r = 0
    for n, T in zip(s["lens"], s["new"]):
        exact = turned(cfg, s["k"][r:r + T], s["layer"].k_norm_w, pair_positions(cfg, s, r, n, T))
        if style == "neox":
            a, b = exact.chunk(2, -1)
            length = torch.sqrt(a * a + b * b).repeat(1, 1, 2)
        else:
            a, b = exact[..., ::2], exact[..., 1::2]
            length = torch.sqrt(a * a + b * b).repeat_interleave(2, -1)
        own = 2.0 ** -24 * 1.01 * exact.abs() + 2.0 ** -25 * length
        assert bool(((k[r:r + T] - exact).abs() <= half_step(exact.abs() + own) + own).all())
        r += T


@pytest.mark.parametrize("kv", ["bf16", "vq8"])
@pytest.mark.parametrize("style", ["neox", "interleaved"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_infinite_keys_stay_infinite(kv, style, io):
    """An infinite element turns into infinities of the formula's signs, a sum beyond the largest
    number into an infinity, a NaN stays one; other pairs are as they were."""
    cfg = dict(n_q_heads=4, n_kv_heads=2, head_dim=64, kv_dtype=kv, io_dtype=io, out_dtype="f32", rope_theta=10000.0, rope_style=style)
    s = make_step(cfg, [(1, 40), (100, 1), (30, 2)], 128, page=32, seed=6)
    k = s["k"]
    inf, big = float("inf"), 3.3e38
    k[3, 0, 5], k[3, 1, 40], k[17, 0, 0], k[40, 1, 63], k[41, 0, 9], k[42, 1, 10] = inf, -inf, -inf, inf, float("nan"), inf
    k[20, 0, [0, 1, 32, 33]] = big  # (pairs of either style: their sums pass the largest bf16)
    plan = make_plan(s)
    s["layer"].append_packed(s["q"], k, s["v"], plan)
    got = s["layer"].read_packed(plan)[0].double().cpu()
    from tests.test_packed import pair_positions, turned
    exact = torch.cat([turned(cfg, k[r:r + T], None, pair_positions(cfg, s, r, n, T)) for r, n, T in ((0, 1, 40), (40, 100, 1), (41, 30, 2))])
    # (numbers beyond the largest bf16, 2^128 - 2^120, and half a step more are infinities)
    exact = torch.where(exact.abs() >= 2.0 ** 128 - 2.0 ** 119, exact.sign() * inf, exact)
    assert int(torch.isinf(exact).sum()) >= 11 and int(torch.isnan(exact).sum()) == 2
    assert torch.equal(torch.isnan(got), torch.isnan(exact))
    assert torch.equal(torch.isinf(got), torch.isinf(exact)) and bool((got[torch.isinf(exact)] == exact[torch.isinf(exact)]).all())
    fine = torch.isfinite(exact)
    # 2^-8 relative and the rounding to fp32 of terms up to the pair's length, here 6 or big
    assert bool(((got - exact).abs()[fine] <= half_step(exact)[fine] + 2.0 ** -22 * torch.where(exact.abs() > 1e30, big, 6.0)[fine]).all())
