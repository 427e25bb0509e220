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
