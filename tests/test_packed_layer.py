"""DecodeLayer's packed steps: tensors it refuses, attention whose append was another's, and steps
of equal lengths that are captured after a packed one."""
import pytest
import torch

from gqa_attention_kv_qk_gb300 import binding as B
from tests.test_packed import check_out, expected, make_step

pytestmark = pytest.mark.gpu
CFG = dict(n_q_heads=8, n_kv_heads=2, head_dim=64, kv_dtype="bf16", io_dtype="bf16", out_dtype="f32", rope_theta=10000.0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gqa_attention_kv_qk_gb300 import build
    build.build()


def rows(n, heads, seed=0):
    return torch.randn((n, heads, 64), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
