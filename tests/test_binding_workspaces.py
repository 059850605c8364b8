"""The dense product and the balance loss keep state in their workspaces, so
each takes its own kind alone (no GPU: refused before anything is launched)."""
import pytest

torch = pytest.importorskip("torch")


class OnGpu:
    """Stands for a tensor of this shape and type on cuda:0, at a made-up address."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.is_cuda = dtype, torch.Size(shape), True

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def stride(self):
        return (self.shape[1], 1)

    def data_ptr(self):
        return 0x100000


def workspace(cls):
    ws = object.__new__(cls)
    ws.tensor, ws.nbytes, ws.device = OnGpu(torch.int32, 1 << 20), 1 << 22, 0
    return ws


@pytest.fixture()
def rf(monkeypatch):
    import routed_expert_fp4_amd as rf

    def launched(fn, *args):
        raise AssertionError(f"{fn} was launched")

    monkeypatch.setattr(rf, "_launch", launched)
    return rf


def calls(rf):
    f32, i32 = torch.float32, torch.int32
    m = object.__new__(rf.QuantMatrix)
    m.N, m.K, m.device, m.ref = 64, 256, 0, None

    def linear(ws):
        rf.moe_quant_linear(m, OnGpu(f32, 4, 256), 4, OnGpu(f32, 4, 64), ws)

    def balance(ws):
        rf.moe_balance_fwd(OnGpu(f32, 4, 16), OnGpu(i32, 4, 2), 4, 16, 2, 0.1, OnGpu(i32, 1, 16), OnGpu(i32, 1),
                           OnGpu(f32, 1, 16), OnGpu(f32, 1), ws)

    return {rf.QuantWorkspace: linear, rf.BalanceWorkspace: balance}


def test_each_takes_its_own_kind(rf):
    others = (rf.QuantWorkspace, rf.BalanceWorkspace, rf.Workspace, rf.LatentWorkspace, rf.MxMmaWorkspace)
    for own, call in calls(rf).items():
        with pytest.raises(AssertionError, match="was launched"):
            call(workspace(own))
        for cls in others:
            if cls is own:
                continue
            ws = object.__new__(cls)
            if cls in (rf.QuantWorkspace, rf.BalanceWorkspace):
                ws = workspace(cls)
            with pytest.raises(ValueError, match=own.__name__):
                call(ws)
        with pytest.raises(ValueError, match=own.__name__):
            call(None)
