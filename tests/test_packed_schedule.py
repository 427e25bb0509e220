"""The packed attention's work list: batches whose pairs are cut into the most pieces."""
import math
import random

import pytest
import torch

from gqa_attention_kv_qk_gb300 import binding as B


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gqa_attention_kv_qk_gb300 import build
    build.build()


@pytest.mark.gpu
@pytest.mark.parametrize("kv,ragged", [("bf16", False), ("bf16", True), ("vq8", False)])
def test_many_long_requests_of_one_kv_head(kv, ragged):
    """Twice as many single tokens as SMs, less one, far behind: all but the first round of requests
    are cut along the keys, the last ones into the most pieces. They share the pages of one long text,
    and every output row is written and right (weights in two parts, 2^-14, and logits within
    2^-16 sum |q k| / sqrt D = 3e-4 on values up to 6: below 6 (2^-14 + 6e-4) = 4e-3, and 1e-4 on average)."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    from gqa_attention_kv_qk_gb300.packed import PackedPlan
    from gqa_attention_kv_qk_gb300.pages import PageTable
    n_sm = torch.cuda.get_device_properties(0).multi_processor_count
    Bn, G, D, ps, L = 2 * n_sm - 1, 8, 64, 64, 64000
    P = L // ps
    cfg = dict(n_q_heads=G, n_kv_heads=1, head_dim=D, kv_dtype=kv, io_dtype="bf16", out_dtype="f32", rope_theta=10000.0)
    rng, g = random.Random(1), torch.Generator(device="cuda").manual_seed(1)
    held = [rng.randint(P // 3, P) if ragged else P for _ in range(Bn)]
    lens = [ps * n for n in held]
    table = torch.full((Bn, P + 1), -1, dtype=torch.int32)
    for b in range(Bn):
        table[b, :held[b]] = torch.arange(held[b], dtype=torch.int32)
    pages = PageTable(table, ps, P + Bn, seq_lens=torch.tensor(lens, dtype=torch.int32))
    layer = DecodeLayer(cfg, Bn, (P + 1) * ps, page_size=ps, block_table=pages.block_table, n_pages=P + Bn,
                        cache=dict(seq_lens=pages.seq_lens), max_tokens=Bn)
    new = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    text = new(2, P, 1, ps, D)
    layer.k_cache[:P] = text[0].to(torch.bfloat16)
    if kv == "bf16":
        layer.v_cache[:P] = text[1].to(torch.bfloat16)
    else:
        layer.v_cache[:P] = (text[1] * 20).round().clamp(-127, 127).to(torch.int8)
        layer.v_scale[:P] = 0.05
    q, k, v = (new(Bn, h, D).to(torch.bfloat16) for h in (G, 1, 1))
    plan = PackedPlan(Bn, Bn)
    pages.plan(torch.ones(Bn, dtype=torch.int32, device="cuda"), plan)
    out = torch.full((Bn, G, D), 77.0, device="cuda")
    layer.append_packed(q, k, v, plan)
    for _ in range(2):  # (the counters start over)
        out.fill_(77.0)
        layer.attend_packed(plan, out)
        torch.cuda.synchronize()
        assert layer.device_status() == 0 and pages.device_status() == 0
        assert int((out == 77.0).sum()) == 0
    # the definition in 64 bits: the shared text's keys, and each request's own last one
    values = layer.v_cache.double() if kv == "bf16" else layer.v_cache.double() * layer.v_scale.double().unsqueeze(-1)
    keys, own = layer.k_cache.double().reshape(-1, D), torch.arange(P, P + Bn, device="cuda")
    values = values.reshape(-1, D)
    at = pages.block_table[torch.arange(Bn, device="cuda"), torch.tensor(held, device="cuda")].long() * ps
    assert torch.equal(at.sort().values, own * ps)
    f = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    ang = (torch.tensor(lens, dtype=torch.float64, device="cuda").unsqueeze(-1) * f).unsqueeze(1)
    a, b = q.double().chunk(2, -1)
    turned = torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1) / math.sqrt(D)
    worst, total = 0.0, 0.0
    for i in range(Bn):
        use = torch.cat([torch.arange(lens[i], device="cuda"), at[i:i + 1]])
        want = torch.softmax(turned[i] @ keys[use].T, -1) @ values[use]
        err = (out[i].double() - want).abs()
        worst, total = max(worst, float(err.max())), total + float(err.mean())
    assert worst <= 4e-3 and total / Bn <= 1e-4


@pytest.mark.parametrize("n_tokens,mib", [(1, 6), (16, 16), (64, 32), (1024, 150), (8192, 300)])
def test_workspace_grows_with_the_rows(n_tokens, mib):
    """A decode step's workspace of 32 / 8 heads holds what its rows can be cut into, not what a full
    batch's could (64 rows took 162 MiB)."""
    d = B.make_desc(dict(n_q_heads=32, n_kv_heads=8, head_dim=128, kv_dtype="bf16", io_dtype="bf16", out_dtype="bf16"))
    for batch in (1, 64):
        size = B.uaa_packed_workspace_size(d, batch, n_tokens, 152)
        assert 0 < size <= mib << 20
        assert size >= n_tokens * 32 * 128 * 4
    sizes = [B.uaa_packed_workspace_size(d, 64, n, 152) for n in (0, 1, 2, 63, 64, 65, 1000, 8192)]
    assert sizes == sorted(sizes)
