"""Counts of packed batches whose sequences are uneven: right on both sides of
the number of choices from which a batch is shared out in slots, and no batch
takes many times as long as an even one."""
import numpy as np
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def cuts(kind, C, S, rng):
    if kind == "even":
        return np.linspace(0, C, S + 1).astype(np.int32)
    if kind == "drawn":
        return np.sort(rng.integers(0, C + 1, S + 1)).astype(np.int32)
    if kind == "first":                               # all but a few in the first one
        return np.concatenate([[1], C - np.arange(S)[::-1]]).astype(np.int32)
    seq = np.minimum(np.arange(S + 1), C - 2).astype(np.int32)
    seq[-1] = C - 1                                   # or in the last one
    return seq


@pytest.mark.parametrize("C,E,k,S", [(2048, 100, 32, 20), (2049, 100, 32, 20), (5000, 896, 16, 128),
                                     (9000, 1024, 8, 3), (40000, 64, 32, 700), (65535, 448, 16, 5000),
                                     (70000, 30, 1, 2), (30000, 17, 5, 20000)])
@pytest.mark.parametrize("kind", ["even", "drawn", "first", "last"])
def test_against_the_definition(C, E, k, S, kind):
    import routed_expert_fp4_amd as rf
    say(f"[counts] {C} tokens x {k} of {E}, {S} sequences, {kind}")
    rng = np.random.default_rng(C + S)
    seq = cuts(kind, C, S, rng)
    idx = rng.integers(-1, E + 1, (C, k)).astype(np.int32)          # some outside
    mask = (rng.random(C) < 0.8).astype(np.uint8)
    owner = np.searchsorted(seq, np.arange(C), side="right") - 1
    inside = (owner >= 0) & (owner < S) & (np.arange(C) < seq[-1])
    i, s, m = (torch.from_numpy(a).cuda() for a in (idx, seq, mask))
    for masked in (False, True):
        live = inside & (mask != 0) if masked else inside
        tok = np.bincount(owner[live], minlength=S)
        at = (owner[:, None] * E + idx)[live[:, None] & (idx >= 0) & (idx < E)]
        want = np.bincount(at, minlength=S * E).reshape(S, E)
        cnt = torch.full((S, E), 9, dtype=torch.int32, device="cuda")
        tk = torch.full((S,), 9, dtype=torch.int32, device="cuda")
        for again in range(2):
            rf.moe_expert_counts(i, C, E, k, cnt, tk, seq_offsets=s, S=S, token_mask=m if masked else None,
                                 accumulate=again > 0)
            assert np.array_equal(cnt.cpu().numpy(), want * (again + 1))
            assert np.array_equal(tk.cpu().numpy(), tok * (again + 1))
        cnt.fill_(4)
        rf.moe_expert_counts(i, C, E, k, cnt, None, seq_offsets=s, S=S, token_mask=m if masked else None)
        assert np.array_equal(cnt.cpu().numpy(), want)


def test_bad_offsets_stay_inside_the_batch():
    """Offsets outside [0, C] or falling, in a batch that is shared out: every
    count stays within the batch."""
    import routed_expert_fp4_amd as rf
    C, E, k, S = 9000, 33, 16, 5
    idx = torch.randint(0, E, (C, k), dtype=torch.int32, device="cuda")
    for seq in ([-5, 10, 90000, 20, 2 ** 31 - 1, 40], [9000, 4000, 3000, 2000, 1000, 0], [-2 ** 31] * 6, [7] * 6):
        cnt = torch.full((S, E), 9, dtype=torch.int32, device="cuda")
        s = torch.tensor(seq, dtype=torch.int64).clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32).cuda()
        rf.moe_expert_counts(idx, C, E, k, cnt, seq_offsets=s, S=S)
        assert int(cnt.min()) >= 0 and int(cnt.max()) <= C * k


def test_captured_into_a_graph():
    import routed_expert_fp4_amd as rf
    C, E, k, S = 9000, 200, 16, 40
    rng = np.random.default_rng(1)
    idx = torch.from_numpy(rng.integers(0, E, (C, k)).astype(np.int32)).cuda()
    seq = torch.from_numpy(cuts("drawn", C, S, rng)).cuda()
    cnt, tok, again, tok2 = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((S, E), (S,), (S, E), (S,)))
    rf.moe_expert_counts(idx, C, E, k, cnt, tok, seq_offsets=seq, S=S)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rf.moe_expert_counts(idx, C, E, k, again, tok2, seq_offsets=seq, S=S)
    for r in range(4):
        idx.copy_(torch.randint(0, E, (C, k), device="cuda"))
        again.fill_(7)
        tok2.fill_(7)
        graph.replay()
        rf.moe_expert_counts(idx, C, E, k, cnt, tok, seq_offsets=seq, S=S)
        torch.cuda.synchronize()
        assert torch.equal(cnt, again) and torch.equal(tok, tok2), r


def test_uneven_batches_take_about_as_long_as_even_ones():
    """One workgroup for the long sequence took 24 and 65 times as long."""
    import routed_expert_fp4_amd as rf
    E, rng = 448, np.random.default_rng(2)
    for C, k, S in ((65536, 16, 128), (65536, 16, 10000)):
        idx = torch.from_numpy(rng.integers(0, E, (C, k)).astype(np.int32)).cuda()
        cnt = torch.zeros((S, E), dtype=torch.int32, device="cuda")
        took = []
        for kind in ("even", "last"):
            seq = torch.from_numpy(cuts(kind, C, S, rng)).cuda()
            best = 1e9
            for _ in range(5):
                a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
                a.record()
                for _ in range(20):
                    rf.moe_expert_counts(idx, C, E, k, cnt, seq_offsets=seq, S=S)
                b.record()
                torch.cuda.synchronize()
                best = min(best, a.elapsed_time(b))
            took.append(best)
        assert took[1] < 6 * took[0], (C, k, S, took)
