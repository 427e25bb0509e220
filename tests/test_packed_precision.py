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
