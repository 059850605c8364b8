"""Device tensors and comparisons shared by the GPU tests of dropout, the adapters
and the gated block."""
import numpy as np
import torch

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def device(a, t, pad=0, off=0):
    """A matrix (or a stack of them) of type t in a wider tensor filled with NaN:
    rows `pad` elements further apart, the first `off` elements into it."""
    a = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(t)
    wide = torch.full((*a.shape[:-1], a.shape[-1] + pad + off), float("nan"), dtype=t, device="cuda")
    out = wide[..., off:off + a.shape[-1]]
    out.copy_(a)
    return out


def host(t):
    return t.double().cpu().numpy()


def check(got, want, tol, depth, what, rel=True, steps=1):
    """Element by element within `tol`, the rounding of the result and (where a
    16-bit type has lost its normals) a step of its smallest; and the 2-norm within
    what as many independent roundings give (`steps`: of how many roundings to the
    type, where operands are rounded to it too).  Infinities and NaN where they are
    wanted."""
    eps, tiny = torch.finfo(got.dtype).eps / 2, torch.finfo(got.dtype).smallest_normal
    g = host(got)
    fine = np.isfinite(want)
    assert (np.isnan(g) == np.isnan(want)).all(), f"{what}: NaN in other places"
    inf = np.isinf(want)
    assert (g[inf] == want[inf]).all(), f"{what}: infinities"
    off = np.where(fine, np.abs(g - np.where(fine, want, 0)), 0)
    bad = ~(off <= (tol + eps * np.abs(np.where(fine, want, 0)) + 2 * eps * tiny) * 1.0001)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {off.max():.3e} at {np.argwhere(bad)[0]}"
    if rel and fine.all():
        n = np.linalg.norm(want)
        assert np.linalg.norm(g - want) <= (steps * eps + 2 * np.sqrt(depth) * 2.0 ** -24) * n + 2 * eps * tiny * np.sqrt(want.size), \
            f"{what}: rel-L2 {np.linalg.norm(g - want) / max(n, 1e-300):.2e}"


def untouched(t, view):
    """What lies between and behind a view's rows is still NaN."""
    full = t._base if t._base is not None else t
    mask = torch.ones_like(full, dtype=torch.bool)
    mask.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool(torch.isnan(full.float())[mask].all())
