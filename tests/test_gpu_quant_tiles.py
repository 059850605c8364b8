"""Every instance of the matrix kernel's tiles: each type of activations and
scales, each kind of group, over enough columns that its buffers and tables
come round several times, with odd sizes and partial tiles.

All results are compared with a 64-bit product; the tolerance is that of
test_gpu_quant.
"""
import pytest

from gpu_util import say
from test_gpu_quant import T, make

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def weights(codes, scales, z, K, G):
    q = torch.stack((codes & 15, codes >> 4), 2).reshape(codes.shape[0], -1)[:, :K].double()
    g = torch.arange(K, device=codes.device) // G
    return (q - (8.0 if z is None else z[:, g].double())) * scales[:, g].double()


def check_all(codes, scales, z, x, y, K, G, old=None):
    """y against x W^T (+ old), element by element, on the GPU in 64 bits."""
    W = weights(codes, scales, z, K, G).t().contiguous()
    xd = x.double().contiguous()
    want, size = xd @ W, xd.abs() @ W.abs()
    few = xd.abs().amax(1, keepdim=True) * W.abs().sum(0)[None, :]
    tol = (160 + K / 32 + 2) * 2.0 ** -24 * size + 2.0 ** -38 * few
    if old is not None:
        want = want + old.double()
        tol = tol + 2.0 ** -24 * want.abs()
    f = torch.finfo(y.dtype)
    off = (y.double() - want).abs() > (tol + f.eps / 2 * want.abs() + f.smallest_normal * f.eps) * 1.0001
    assert not bool(off.any()) and bool(torch.isfinite(y).all()), f"{int(off.sum())} of {off.numel()} off"


# the larger tile (fp32: 64 tokens x 256 rows where 128 workgroups come of it;
# 16 bits: 128 x 256 where the smaller tile has more than 512) and the smaller
@pytest.mark.parametrize("wide", [True, False], ids=["larger", "smaller"])
@pytest.mark.parametrize("G", [32, 64, 128, 384])
@pytest.mark.parametrize("st", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
def test_every_tile(xt, st, G, wide):
    import routed_expert_fp4_amd as rf
    zeros = st != "bf16"
    C, N = ((519, 4003) if xt == "f32" else (1003, 4219)) if wide else (201, 1003)
    K = {32: 2437, 64: 2560, 128: 2433, 384: 2688}[G] if wide else {32: 1664, 64: 1601, 128: 1667, 384: 1700}[G]
    say(f"[quant] {C} x {N} x {K}, groups of {G}, {xt}, scales {st}, zeros {zeros}")
    codes, scales, z, x, y = make(C, N, K, G, xt, st, zeros, 70, y_pad=1)
    m = rf.QuantMatrix(codes, scales, K, G, z)
    ws = rf.QuantWorkspace(m, C, x.dtype)
    y[:, :N] = float("nan")
    rf.moe_quant_linear(m, x, C, y[:, :N], ws)
    check_all(codes, scales, z, x, y[:, :N], K, G)
    old = torch.randn((C, N), device="cuda").to(T[xt])
    y[:, :N] = old
    rf.moe_quant_linear(m, x, C, y[:, :N], ws, accumulate=True)
    check_all(codes, scales, z, x, y[:, :N], K, G, old)
    assert bool((y[:, N:] == 7.0).all())


@pytest.mark.parametrize("xt,G,st", [("bf16", 128, "bf16"), ("bf16", 64, "bf16"), ("bf16", 32, "f16"),
                                     ("f32", 128, "bf16"), ("f32", 64, "f32"), ("f16", 32, "f32")])
def test_long_rows_in_the_larger_tile(xt, G, st):
    """7168 columns, whole rows of tiles, aligned outputs."""
    import routed_expert_fp4_amd as rf
    C, N, K = (512, 4096, 7168) if xt == "f32" else (1088, 4096, 7168)
    say(f"[quant] {C} x {N} x {K}, groups of {G}, {xt}, scales {st}")
    codes, scales, z, x, y = make(C, N, K, G, xt, st, True, 71)
    m = rf.QuantMatrix(codes, scales, K, G, z)
    rf.moe_quant_linear(m, x, C, y, rf.QuantWorkspace(m, C, x.dtype))
    check_all(codes, scales, z, x, y, K, G)
