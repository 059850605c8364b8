"""One workspace, sized for the largest batch, through batches of other sizes:
the same bits as a workspace of each call's own."""
import pytest

from gpu_util import say
from test_gpu_load import fwd, make as make_load
from test_gpu_quant import make, run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("N,K,G,xt,largest", [(7168, 3584, 32, "bf16", 257), (3584, 7168, 128, "f32", 100),
                                              (1001, 4099, 64, "f16", 600)])
def test_dense_product_of_fewer_tokens(N, K, G, xt, largest):
    import routed_expert_fp4_amd as rf
    codes, scales, z, x, y = make(largest, N, K, G, xt, "bf16", True, 60)
    m = rf.QuantMatrix(codes, scales, K, G, z)
    ws = rf.QuantWorkspace(m, largest, x.dtype)
    for C in (largest, largest - 1, 256, 200, 129, 64, 65, 17, 16, 9, 8, 2, 1, largest):
        if C > largest:
            continue
        say(f"[quant] {C} of {largest} tokens x {N} x {K}")
        y[:C].fill_(float("nan"))
        rf.moe_quant_linear(m, x[:C], C, y[:C], ws)
        own = torch.full_like(y[:C], float("nan"))
        run(codes, scales, z, x[:C], own, K, G)
        assert torch.equal(y[:C], own), C


def test_balance_of_other_batches():
    """Batches of one slot and of many, and both sides of the number of
    workgroups from which arrivals are shared out over several tickets."""
    import routed_expert_fp4_amd as rf
    E, k = 896, 4
    ws = rf.BalanceWorkspace(40000, E, 60)
    for C, S in [(40000, 1), (32768, 1), (300, 47), (20, 1), (2047, 8), (900, 60), (2056, 9), (1000, 10), (32, 1),
                 (4111, 47), (33, 2), (40000, 1), (300, 47)]:
        say(f"[balance] {C} tokens, {S} sequences")
        logits, idx, seq, mask = make_load(C, E, k, S, True, seed=C)
        a, _ = fwd(logits, idx, E, 0.1, "sigmoid", seq, mask, S, ws)
        b, _ = fwd(logits, idx, E, 0.1, "sigmoid", seq, mask, S)
        for n in ("counts", "tokens", "probs", "loss"):
            assert torch.equal(a[n], b[n]), (C, S, n)
