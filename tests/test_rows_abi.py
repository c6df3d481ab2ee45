"""Row operators and 8-bit products: host-side argument checks (no GPU needed: these paths
return before any CUDA call) and the oracle's own checks."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import rows_oracle as R
from sparse_moe_layer_select_b200 import build as B
from sparse_moe_layer_select_b200 import moe as M
from tests.rows_common import routing

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, SHAPE, SMALL = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED_SHAPE, M.MOE_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def L():
    """The library with argument types for the calls below (ctypes would pass Python integers
    as 32-bit ones)."""
    B.build()
    lib = ctypes.CDLL(M.LIB_PATH)
    P, I, S, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    kinds = {"D": P, "p": P, "o": P, "q": P, "w": P, "W": P, "s": S, "c": S, "t": I, "z": Z}
    for name, spec in CALLS.items():
        getattr(lib, name).argtypes = [kinds[a[0]] for a in spec.split()] + [P]
    lib.moe_quantize_int8.argtypes = [I, I, I, P, S, P, P, S, P, P]
    lib.moe_matmul_int8.argtypes = [P, P, Z, P]
    return lib


def _dims(T=64, d=100, E=16, k=4):
    return M.make_dims(T, d, E, k, 0, 0)


# Fake device addresses: refused calls never reach the device.  Per call the good arguments;
# names say what each is (p: required pointer, o: optional one, s: row stride, t: dtype).
CALLS = {
    "moe_sort": "D p p p p p t:0 p s p s w z:1000000",
    "moe_dispatch": "D t:0 p s p p s W",
    "moe_dispatch_backward": "D t:0 p s p o s t:1 p s W",
    "moe_combine": "D t:0 p s p p o s t:2 p s W",
    "moe_combine_backward": "D t:0 p s p s p p q s p W",
    "moe_route_backward": "D p p p p W",
    "moe_dispatch_int8": "D t:0 p s p p c p W",
}


def _args(name, dims, change=None):
    out = []
    for i, a in enumerate(CALLS[name].split()):
        v = {"D": ctypes.byref(dims), "p": 1024 * (i + 1), "o": 1024 * (i + 1), "s": 104, "c": 112,
             "w": 4096, "W": 8192, "q": 512 * 1024}.get(a[0])
        if ":" in a:
            v = int(a.split(":")[1])
        out.append(v)
    if change:
        out[change[0]] = change[1]
    return out + [None]


@pytest.mark.parametrize("name", CALLS)
def test_argument_errors_return_before_any_launch(L, name):
    f = getattr(L, name)
    kinds = CALLS[name].split()
    for i, a in enumerate(kinds):
        if a in ("p", "q"):
            assert f(*_args(name, _dims(), (i, None))) == BAD, i       # missing
        if a in ("p", "q", "o"):
            assert f(*_args(name, _dims(), (i, 1024 + 8))) == BAD, i   # misaligned
        if a in ("s", "c"):
            assert f(*_args(name, _dims(), (i, 99))) == BAD, i         # shorter than a row
        if a == "c":
            assert f(*_args(name, _dims(), (i, 104))) == BAD           # not a multiple of 16
        if a[0] == "t":
            assert f(*_args(name, _dims(), (i, 3))) == BAD
            assert f(*_args(name, _dims(), (i, -1))) == BAD
        if a in ("w", "W"):
            assert f(*_args(name, _dims(), (i, 4096 + 16))) == BAD     # not 256-byte aligned
    for dims in (_dims(d=0), _dims(E=513), _dims(k=17, E=32), _dims(k=5, E=4), _dims(k=0),
                 _dims(T=1 << 28, k=8)):
        assert f(*_args(name, dims)) == SHAPE
    assert f(*_args(name, _dims(T=-1))) == BAD
    wrong = _dims()
    wrong.struct_size = 4
    assert f(*_args(name, wrong)) == BAD
    if name != "moe_sort":  # T = 0 needs no pointers
        empty = [None if a[0] in "poqwW" else v
                 for a, v in zip(CALLS[name].split(), _args(name, _dims(T=0)))]
        assert f(*empty, None) == M.MOE_OK


def test_every_declared_symbol_is_exported(L):
    with open(os.path.join(ROOT, "include", "moe_rows.h")) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", src)))
    assert sorted(M.ROWS_EXPORTED) == declared
    assert all(hasattr(L, name) for name in declared)


def test_sort_workspace(L):
    n = M.sort_workspace_size(_dims(32768, 2048, 256, 8))
    assert 256 <= n <= M.workspace_size(M.make_dims(32768, 2048, 256, 8, 512, 512))
    assert M.sort_workspace_size(_dims(T=1, d=1, E=1, k=1)) >= 256
    assert M.sort_workspace_size(_dims(E=513)) == 0
    a = _args("moe_sort", _dims(), (12, M.sort_workspace_size(_dims()) - 1))
    assert L.moe_sort(*a) == SMALL
    a = _args("moe_sort", _dims(), (9, None))   # x without x_perm
    assert L.moe_sort(*a) == BAD
    a = _args("moe_sort", _dims(), (11, None))  # no workspace
    assert L.moe_sort(*a) == BAD


def test_combine_backward_in_place_needs_one_stride(L):
    a = _args("moe_combine_backward", _dims())
    a[8], a[9] = a[4], 112
    assert L.moe_combine_backward(*a) == BAD


def test_quantize_int8_refusals(L):
    def call(rows=8, cols=100, dtype=0, x=1024, xs=100, n=None, codes=2048, cs=112, scales=4096):
        return L.moe_quantize_int8(rows, cols, dtype, x, xs, n, codes, cs, scales, None)
    for kw in (dict(rows=-1), dict(dtype=3), dict(x=None), dict(x=1032), dict(xs=99), dict(n=1026),
               dict(codes=None), dict(codes=2056), dict(cs=100), dict(cs=96), dict(scales=None),
               dict(scales=4100)):
        assert call(**kw) == BAD, kw
    assert call(cols=0) == SHAPE
    assert call(rows=0, x=None, codes=None, scales=None) == M.MOE_OK


def test_matmul_int8_refusals(L):
    def call(ws=4096, ws_bytes=256, size=None, **kw):
        v = dict(M=8, N=40, K=100, G=2, out_dtype=0, flags=0, a=1 << 20, a_stride=112,
                 a_scale=2 << 20, b=3 << 20, b_stride=112, b_scale=4 << 20, offsets=5 << 20,
                 out=6 << 20, out_stride=40)
        v.update(kw)
        m = M.moe_int8_matmul_t(size or ctypes.sizeof(M.moe_int8_matmul_t), *v.values())
        return L.moe_matmul_int8(ctypes.byref(m), ws, ws_bytes, None)
    for kw in (dict(size=8), dict(M=-1), dict(out_dtype=3), dict(flags=2), dict(offsets=None),
               dict(offsets=(5 << 20) + 2), dict(a=None), dict(a=(1 << 20) + 8), dict(b=None),
               dict(a_scale=None), dict(b_scale=8), dict(out=None), dict(a_stride=96),
               dict(a_stride=104), dict(b_stride=96), dict(b_stride=120), dict(out_stride=39),
               dict(ws=None), dict(ws=4096 + 128)):
        assert call(**kw) == BAD, kw
    for kw in (dict(N=0), dict(K=0), dict(K=131072), dict(G=0), dict(G=513),
               dict(N=1 << 30), dict(M=(1 << 31) - 1), dict(a_stride=1 << 40),
               dict(N=1 << 29, G=4)):
        assert call(**kw) == SHAPE, kw
    assert call(ws_bytes=128) == SMALL
    assert call(M=0, a=None, out=None, a_scale=None) == M.MOE_OK
    assert L.moe_matmul_int8(None, 4096, 256, None) == BAD


def test_binding_refusals_need_no_gpu(L):
    import torch
    M_ = M
    dims = _dims(4, 32, 4, 2)
    x, p = torch.zeros(4, 32), torch.zeros(8, 32)
    inv = torch.zeros(4, 2, dtype=torch.int32)
    q, s = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: M_.dispatch(dims, x, inv, p),                 # CPU tensors
                 lambda: M_.dispatch(dims, x[:3], inv, p),
                 lambda: M_.quantize_int8(x, p.to(torch.int8), s),
                 lambda: M_.quantize_int8(x, q, s, n_rows=torch.zeros(2, dtype=torch.int32)),
                 lambda: M_.matmul_int8(q, s, q[:, :16], s, x, q),     # K differs
                 lambda: M_.matmul_int8(q, s, q[:3], s[:3], x[:, :3], q, swiglu=True),
                 lambda: M_.matmul_int8(q, s, q, s, x[:, :4], q, offsets=inv[0])):
        with pytest.raises(M.MoeError) as e:
            call()
        assert e.value.code == BAD


# ---------------------------------------------------------------- the oracle itself

def test_oracle_gradients_against_differences():
    T, E, k, d = 12, 9, 3, 7
    logits, idx, w = routing(T, E, k, 1, 0.2, True)
    l = logits.astype(np.float64)
    rng = np.random.default_rng(2)
    inv = R.expert_order(idx, E)[3]
    o, dy, dw = rng.normal(size=(T * k, d)), rng.normal(size=(T, d)), rng.normal(size=(T, k))
    for norm in (False, True):
        g = R.route_backward(l, idx, dw, norm)
        for t, e in ((0, int(idx[0, 0])), (5, int(idx[5, 2])), (7, 4)):
            v = np.zeros_like(l)
            v[t, e] = 1e-6
            num = ((R.route_weights(l + v, idx, norm) - R.route_weights(l - v, idx, norm)) *
                   dw).sum() / 2e-6
            assert abs(num - g[t, e]) < 1e-8
    d_o, d_w, _ = R.combine_backward(dy, o, inv, w, 2.5)
    loss = lambda o_, w_: (R.to_tokens(o_, inv, w_, 2.5)[0] * dy).sum()  # noqa: E731
    on = np.argwhere(inv >= 0)
    for t, j in on[:: max(1, len(on) // 5)]:
        v = np.zeros_like(w, dtype=np.float64)
        v[t, j] = 1e-6
        assert abs((loss(o, w + v) - loss(o, w - v)) / 2e-6 - d_w[t, j]) < 1e-7
        v = np.zeros_like(o)
        v[inv[t, j], 3] = 1e-6
        assert abs((loss(o + v, w) - loss(o - v, w)) / 2e-6 - d_o[inv[t, j], 3]) < 1e-7
    assert np.all(np.isnan(d_o[int((inv >= 0).sum()):]))


def test_oracle_order_and_round_trip():
    _, idx, _ = routing(50, 8, 3, 4, 0.1, True)
    counts, offsets, perm, inv = R.expert_order(idx, 8)
    flat = idx.reshape(-1)
    assert list(perm) == sorted(np.flatnonzero(flat >= 0), key=lambda i: (flat[i], i))
    assert np.array_equal(counts, np.bincount(flat[flat >= 0], minlength=8))
    assert all(inv.reshape(-1)[p] == r for r, p in enumerate(perm))
    x = np.random.default_rng(5).normal(size=(50, 6))
    xp = R.dispatch(x, inv, np.zeros((150, 6)))
    back = R.to_tokens(xp, inv)[0]
    assert np.allclose(back, x * (idx >= 0).sum(1)[:, None])


def test_oracle_quantization():
    x = np.array([[1.0, -2.0, 127.0], [0, 0, 0], [1e-40, 0, -3e-41], [np.inf, 1, 2],
                  [np.nan, 1, 2], [0.5, -63.5, 62.0]], dtype=np.float32)
    q, s = R.quantize_int8(x)
    assert q[0].tolist() == [1, -2, 127] and s[0] == 1
    assert q[1].tolist() == [0, 0, 0] and s[1] == 1
    assert s[2] == 2.0 ** -126 and q[2].tolist() == [0, 0, 0]
    assert np.isnan(s[3]) and np.isnan(s[4]) and not q[3:5].any()
    assert s[5] == 0.5 and q[5].tolist() == [1, -127, 124]
    z = R.matmul_int8(q[:1], s[:1], q[None, 5:6], s[None, 5:6])
    assert z[0, 0] == (1 * 1 + 2 * 127 + 127 * 124) * 0.5
