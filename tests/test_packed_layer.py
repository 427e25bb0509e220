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


@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_tokens_that_share_one_row_are_refused(which):
    """expand() gives a stride of 0 between tokens, which the C entries take as dense rows."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    from gqa_attention_kv_qk_gb300.packed import PackedPlan
    layer, plan = DecodeLayer(CFG, 2, 128, max_tokens=8), PackedPlan(2, 8)
    x = dict(q=rows(8, 8), k=rows(8, 2), v=rows(8, 2))
    x[which] = x[which][:1].expand(8, -1, -1)
    with pytest.raises(ValueError, match="strides"):
        layer.step_packed(x["q"], x["k"], x["v"], plan)
    with pytest.raises(ValueError, match="strides"):
        layer.append_packed(x["q"], x["k"], x["v"], plan)
    # one token has no neighbour: its stride says nothing
    one = PackedPlan(2, 1)
    layer.plan(torch.tensor([1, 0], dtype=torch.int32, device="cuda"), one)
    layer.step_packed(rows(1, 8).expand(1, -1, -1), rows(1, 2), rows(1, 2), one)
    assert layer.seq_lens.tolist() == [1, 0]


@pytest.mark.parametrize("kv", ["bf16", "q4", "f32"])
def test_attention_after_another_append(kv):
    """attend_packed needs the layer's own append by the plan as it stands, the last one on its workspace."""
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    from gqa_attention_kv_qk_gb300.packed import PackedPlan
    cfg = dict(CFG, kv_dtype=kv)
    a = DecodeLayer(cfg, 2, 128, max_tokens=8)
    b = DecodeLayer(cfg, 2, 128, max_tokens=8, workspace=a.ws_tensor)
    view = DecodeLayer(cfg, 2, 128, max_tokens=8, workspace=a.ws_tensor[:])
    plan, out = PackedPlan(2, 8), torch.zeros((8, 8, 64), device="cuda")
    x = rows(8, 8), rows(8, 2, 1), rows(8, 2, 2)
    q_lens = torch.tensor([3, 5], dtype=torch.int32, device="cuda")
    a.plan(q_lens, plan)
    a.append_packed(*x, plan)
    assert a.attend_packed(plan, out) is out
    for other in (b, view):
        a.append_packed(*x, plan)
        other.append_packed(*x, plan)
        with pytest.raises(ValueError, match="append_packed"):
            a.attend_packed(plan, out)
        other.attend_packed(plan, out)
    a.append_packed(*x, plan)
    b.step(torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda"), rows(2, 2), rows(2, 2))
    with pytest.raises(ValueError, match="append_packed"):
        a.attend_packed(plan, out)
    a.step_packed(*x, plan)
    a.attend_packed(plan, out)
    a.plan(q_lens, plan)  # refilled, for other lengths by now
    with pytest.raises(ValueError, match="append_packed"):
        a.attend_packed(plan, out)
    a.append_packed(*x, plan)
    assert a.attend_packed(plan, out) is out and a.device_status() == 0
    # a workspace of its own is not concerned
    alone = DecodeLayer(cfg, 2, 128, max_tokens=8)
    alone.plan(q_lens, plan)
    alone.append_packed(*x, plan)
    b.step(torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda"), rows(2, 2), rows(2, 2))
    alone.attend_packed(plan, out)


@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_equal_steps_captured_after_a_packed_one(kv):
    """The bound on the lengths is not known then: the capture goes by what fits the cache."""
    cfg = dict(CFG, kv_dtype=kv)
    s = make_step(cfg, [(30, 20), (0, 9), (120, 4)], 128, seed=4)
    layer, plan = s["layer"], s["plan"]
    x = rows(3, 8, 5), rows(3, 2, 6), rows(3, 2, 7)
    layer.plan(s["q_lens"], plan)
    layer.step_packed(s["q"], s["k"], s["v"], plan)
    assert layer.seq_lens.tolist() == [50, 9, 124]
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.zeros((3, 8, 64), device="cuda")
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        layer.step(*x, out=out)
        layer.append(*x)
        layer.partial()
        layer.combine()
    s.update(N=3, new=[1, 1, 1], q=x[0], k=x[1], v=x[2])
    for lens in ([50, 9, 124], [52, 11, 126], [3, 0, 6]):
        layer.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert layer.seq_lens.tolist() == [n + 2 for n in lens] and layer.device_status() == 0
        s["lens"] = lens
        check_out(cfg, out, expected(cfg, s)[0])
        s["lens"] = [n + 1 for n in lens]
        check_out(cfg, layer.out, expected(cfg, s)[0])
    # a sequence without room is flagged, as ever
    layer.seq_lens.copy_(torch.tensor([5, 128, 7], dtype=torch.int32))
    graph.replay()
    assert layer.device_status() == B.UAA_DEVFLAG_CAPACITY and layer.seq_lens.tolist() == [7, 128, 9]
    # an eager step reads the lengths, and says so where there is no room
    layer.plan(torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda"), plan)
    layer.step_packed(*(t.repeat(11, 1, 1) for t in x), plan)
    with pytest.raises(B.UaaError, match="capacity"):
        layer.step(*x)


def test_equal_steps_of_no_sequences_after_a_packed_one():
    from gqa_attention_kv_qk_gb300.layer import DecodeLayer
    from gqa_attention_kv_qk_gb300.packed import PackedPlan
    layer, plan = DecodeLayer(CFG, 0, 128, max_tokens=4), PackedPlan(0, 4)
    layer.plan(torch.zeros(0, dtype=torch.int32, device="cuda"), plan)
    out = torch.full((4, 8, 64), 7.0, device="cuda")
    layer.step_packed(rows(4, 8), rows(4, 2), rows(4, 2), plan, out=out)
    assert bool((out == 7.0).all()) and tuple(layer.step(rows(0, 8), rows(0, 2), rows(0, 2)).shape) == (0, 8, 64)
