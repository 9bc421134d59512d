"""Helpers of the tests of what stands around the linear layers: element types,
rows with gaps, and the rounding a stored result may have."""

import numpy as np
import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# Half a unit in the last place of a result of size 1, and half the smallest
# step of the type (results that underflow).
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def type_of(q4lib, name):
    return {"f32": q4lib.Q4_TYPE_F32, "f16": q4lib.Q4_TYPE_F16, "bf16": q4lib.Q4_TYPE_BF16}[name]


GAP = 77.0


def rows(x, name, pad=0, shift=0):
    """`x` [m x d] on the device in its type, as rows `pad` elements further
    apart than they are long, the first `shift` elements into a buffer that is
    otherwise GAP."""
    m, d = x.shape
    buf = torch.full((m * (d + pad) + shift,), GAP, dtype=TYPES[name], device="cuda")
    v = buf[shift:shift + m * (d + pad)].view(m, d + pad)[:, :d]
    v.copy_(torch.as_tensor(np.asarray(x)) if not isinstance(x, torch.Tensor) else x)
    return v


def blank(m, d, name, pad=0, shift=0):
    return rows(torch.full((m, d), float("nan")), name, pad, shift)


def gaps_kept(v):
    """The elements between the rows of a view made by rows() are untouched."""
    if v.shape[0] == 0 or v.stride(0) == v.shape[1]:
        return True
    ld, d = v.stride(0), v.shape[1]
    whole = torch.as_strided(v, (v.shape[0], ld), (ld, 1), v.storage_offset())
    return bool((whole[:, d:].float() == GAP).all())


def f64(x):
    return x.detach().to(torch.float64).cpu().numpy()


def close(y, ref, tol, what=""):
    """|y - ref| <= tol elementwise; NaN and infinities in the same places."""
    y, ref = f64(y) if isinstance(y, torch.Tensor) else y, np.asarray(ref)
    assert y.shape == ref.shape, f"{what}: shape {y.shape}, not {ref.shape}"
    assert np.array_equal(np.isnan(y), np.isnan(ref)), f"{what}: NaN in other places"
    inf = np.isinf(ref)
    assert np.array_equal(y[inf], ref[inf]), f"{what}: infinities differ"
    ok = ~np.isnan(ref) & ~inf
    if not ok.any():
        return 0.0
    ratio = np.abs(y - ref)[ok] / np.broadcast_to(tol, ref.shape)[ok]
    assert ratio.max() <= 1.0, f"{what}: error {ratio.max():.3g} of the tolerance"
    return float(ratio.max())
