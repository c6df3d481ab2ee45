"""Shared helpers of the row-operator tests: routing, strided rows, tolerances."""
import numpy as np

DTYPES = ("bf16", "f16", "f32")


def torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def half_step(name):
    """Relative error of one rounding to the type: half a step."""
    import torch
    return torch.finfo(torch_dtype(name)).eps / 2


def floor(name):
    """Absolute error of one rounding near zero: half of the smallest subnormal."""
    import torch
    f = torch.finfo(torch_dtype(name))
    return f.smallest_normal * f.eps / 2


def routing(T, E, k, seed, masked=0.0, partial=False):
    """logits [T, E], selected experts [T, k] (-1: not routed) and positive weights [T, k]."""
    rng = np.random.default_rng(seed)
    logits = rng.normal(size=(T, E)).astype(np.float32)
    idx = np.argsort(-logits - 0.5 * rng.normal(size=E), axis=1, kind="stable")[:, :k]
    idx = idx.astype(np.int32)
    off = rng.random(T) < masked
    idx[off] = -1
    if partial:  # single slots of a token not routed
        idx[rng.random((T, k)) < 0.2] = -1
    w = rng.random((T, k)).astype(np.float32) + 0.1
    w[idx < 0] = 0
    return logits, idx, w


def rows(n, d, pad, dtype, seed, device="cuda"):
    """[n, d] of normal values, rows d + pad elements apart, in a buffer of the type."""
    import torch
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(n, d + pad, generator=g).to(torch_dtype(dtype)).to(device)
    return t[:, :d]


def filled(n, d, pad, dtype, value, device="cuda"):
    """A strided [n, d] view of a constant buffer, and the buffer."""
    import torch
    buf = torch.full((n, d + pad), value, dtype=torch_dtype(dtype), device=device)
    return buf[:, :d], buf


def f64(t):
    return t.detach().double().cpu().numpy()


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()
