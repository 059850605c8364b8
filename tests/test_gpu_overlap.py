"""x and y as columns of one buffer: the same bits as apart, and refused where
they overlap."""
import pytest

from test_gpu_quant import make

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("C", [1, 6, 16, 50])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_columns_of_one_buffer(C, xt):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import routed_expert_fp4_amd as rf
    N, K, G = 70, 500, 64
    codes, scales, z, x, y = make(C, N, K, G, xt, "f32", True, 80)
    m = rf.QuantMatrix(codes, scales, K, G, z)
    ws = rf.QuantWorkspace(m, C, x.dtype)
    rf.moe_quant_linear(m, x, C, y, ws)
    both = torch.zeros((C, K + N + 3), dtype=x.dtype, device="cuda")
    both[:, 2:2 + K] = x
    rf.moe_quant_linear(m, both[:, 2:2 + K], C, both[:, 2 + K:2 + K + N], ws)
    assert torch.equal(both[:, 2 + K:2 + K + N], y) and torch.equal(both[:, 2:2 + K], x)
    before = both.clone()
    with pytest.raises(rf.MoeError):
        rf.moe_quant_linear(m, both[:, 2:2 + K], C, both[:, 1 + K:1 + K + N], ws)
    torch.cuda.synchronize()
    assert torch.equal(before, both)
