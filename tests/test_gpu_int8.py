"""Rows quantized to 8 bits and products of such rows, against the oracle.

Codes and scales are compared exactly.  A product's integer sum is exact; converting it and
multiplying by two scales are three fp32 roundings, the output's type one more.
"""
import numpy as np
import pytest

from oracle import rows_oracle as R
from sparse_moe_layer_select_b200 import moe as M
from tests.rows_common import (DTYPES, dev, f64, filled, floor, half_step, routing, rows,
                               torch_dtype)

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    torch.cuda.set_device(0)
    from sparse_moe_layer_select_b200 import build as B
    B.build()
    yield


def _header():
    import torch
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def _status(ws):
    import torch
    torch.cuda.synchronize()
    return M.read_device_status(ws)


def _codes(n, d, value=77):
    import torch
    pitch = (d + 15) // 16 * 16 + 16
    buf = torch.full((n, pitch), value, dtype=torch.int8, device="cuda")
    return buf[:, :d], buf


# ---------------------------------------------------------------- quantization

@pytest.mark.parametrize("n,d,pad", [(1, 1, 0), (1, 2048, 0), (5, 7, 0), (5, 8, 1), (33, 1000, 0),
                                     (33, 1003, 5), (3, 4096, 0), (3, 4099, 5), (9, 1002, 2),
                                     (2, 9001, 7), (2, 40000, 0), (1500, 512, 0)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize(n, d, pad, dtype):
    import torch
    x = rows(n, d, pad, dtype, 1)
    if n > 2:
        x[1] = 0
        x[2] *= 1e-3
    codes, buf = _codes(n, d)
    scales = torch.full((n,), -7.0, device="cuda")
    M.quantize_int8(x, codes, scales)
    q, s = R.quantize_int8(f64(x))
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), q)
    assert torch.all(buf[:, d:] == 77)


def test_quantize_extremes():
    """Zeros, subnormals, the largest values, infinities and NaN, ties."""
    import torch
    x = torch.zeros(9, 40)
    x[1, 3], x[1, 5] = 1e-40, -2e-41
    x[2, 0], x[2, 1] = 3.3e38, -3.4e38
    x[3, 7] = float("inf")
    x[4, 9] = float("nan")
    x[5, 2], x[5, 3], x[5, 4], x[5, 5] = 127.0, 2.5, 3.5, -0.5
    x[6, 39] = float("-inf")
    x[7, :] = -1e-45
    x[8, :2] = torch.tensor([1e-38, 1.2e-36])
    x = x.cuda()
    codes, scales = M.alloc_codes(9, 40)
    M.quantize_int8(x, codes, scales)
    q, s = R.quantize_int8(f64(x))
    assert np.array_equal(codes.cpu().numpy(), q)
    assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    assert codes[5, 3:6].tolist() == [2, 4, 0] and np.isnan(s[[3, 4, 6]]).all()


@pytest.mark.parametrize("valid", [0, 1, 6, 10, 99, -3])
def test_quantize_only_the_first_rows(valid):
    import torch
    x = rows(10, 72, 0, "f16", 2)
    codes, buf = _codes(10, 72)
    scales = torch.full((10,), -7.0, device="cuda")
    offsets = torch.tensor([5, valid], dtype=torch.int32, device="cuda")
    M.quantize_int8(x, codes, scales, n_rows=offsets[1:])
    n = min(max(valid, 0), 10)
    q, s = R.quantize_int8(f64(x))
    assert np.array_equal(codes[:n].cpu().numpy(), q[:n])
    assert np.array_equal(scales[:n].cpu().numpy(), s[:n])
    assert torch.all(buf[n:] == 77) and torch.all(scales[n:] == -7)


@pytest.mark.parametrize("T,d,E,k,pad,masked", [(1, 2048, 256, 8, 0, 0.0), (64, 256, 16, 4, 0, 0.2),
                                                (37, 1003, 60, 6, 5, 0.2), (20, 77, 512, 16, 0, 0),
                                                (7, 5000, 8, 8, 2, 0.5), (300, 64, 8, 1, 0, 1.0)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_dispatch_int8(T, d, E, k, pad, masked, dtype):
    import torch
    _, idx, _ = routing(T, E, k, 3, masked, True)
    inv = R.expert_order(idx, E)[3]
    x = rows(T, d, pad, dtype, 4)
    x[0, 0] = float("nan")
    codes, buf = _codes(T * k, d)
    scales = torch.full((T * k,), -7.0, device="cuda")
    ws = _header()
    M.dispatch_int8(M.make_dims(T, d, E, k, 0, 0), x, dev(inv.astype(np.int32)), codes, scales, ws)
    assert _status(ws) == (0, 0)
    q, s = R.quantize_int8(f64(x))
    ref_q, ref_s = np.full((T * k, d), 77, dtype=np.int8), np.full(T * k, -7, dtype=np.float32)
    for j in range(k):
        on = inv[:, j] >= 0
        ref_q[inv[on, j]], ref_s[inv[on, j]] = q[on], s[on]
    assert np.array_equal(codes.cpu().numpy(), ref_q)
    assert np.array_equal(scales.cpu().numpy(), ref_s, equal_nan=True)
    assert torch.all(buf[:, d:] == 77)


# ---------------------------------------------------------------- products

def _matrix(n, k, seed, lo=-127):
    """int8 rows a multiple of 16 bytes apart, the bytes between them poisoned."""
    import torch
    rng = np.random.default_rng(seed)
    v = rng.integers(lo, 128, size=(n, k)).astype(np.int8)
    codes, _ = _codes(n, k, value=113)
    codes.copy_(torch.from_numpy(v))
    return v, codes


def _groups(codes, G):
    """[G * n, K] codes as [G, n, K], the same rows."""
    n, s = codes.shape[0] // G, codes.stride(0)
    return codes.as_strided((G, n, codes.shape[1]), (n * s, s, 1))


def _scales(n, seed):
    return (np.random.default_rng(seed).random(n).astype(np.float32) + 0.5) / 64


def _check(got, ref, dtype, extra=0.0):
    u = half_step(dtype)
    tol = (3 * U32 * (1 + u) + u) * np.abs(ref) + floor(dtype) + extra
    err = np.abs(got - ref)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:3].tolist())


def _swiglu_tol(gate, up, ref, dtype):
    """gate and up are off by three fp32 roundings each; the exponential of |g| by 2 + 1.2 |g|
    steps (its stated bound), relative to exp(-g), which is a share of the denominator; two more
    operations.  silu's own slope is at most 1 + |g| relative to its value."""
    u = half_step(dtype)
    return (2 * (8 + 4 * np.abs(gate)) * U32 + u) * np.abs(ref) + floor(dtype) + \
        1e-30 * np.abs(up)


@pytest.mark.parametrize("Mr,N,K", [(1, 1, 1), (1, 1024, 2048), (2, 16, 16), (16, 127, 31),
                                    (17, 128, 128), (31, 129, 129), (64, 256, 512),
                                    (127, 40, 1000), (128, 300, 256), (129, 1111, 160),
                                    (300, 64, 77), (513, 257, 384), (1025, 512, 640)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_matmul(Mr, N, K, dtype):
    import torch
    a, da = _matrix(Mr, K, 1, lo=-128)
    b, db = _matrix(N, K, 2, lo=-128)
    sa, sb = _scales(Mr, 3), _scales(N, 4)
    out, buf = filled(Mr, N, 3, dtype, -7.0)
    ws = _header()
    M.matmul_int8(da, dev(sa), db, dev(sb), out, ws)
    assert _status(ws) == (0, 0)
    _check(f64(out), R.matmul_int8(a, sa, b[None], sb[None]), dtype)
    assert torch.all(buf[:, N:] == -7)


def test_matmul_sums_are_exact_at_the_largest_length():
    """All codes -128 at the longest K the call takes: the sum is 128 * 128 * K < 2^31."""
    import torch
    K = 131071
    a = torch.full((3, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
    one = torch.ones(3, device="cuda")
    out, ws = torch.empty(3, 3, device="cuda"), _header()
    M.matmul_int8(a, one, a, one, out, ws)
    assert _status(ws) == (0, 0)
    assert torch.all(out == float(np.float32(128 * 128 * K)))


GROUPS = [([0, 0, 5, 5, 40, 40, 173, 300], 300),   # empty groups, one above a tile
          ([0, 300], 300),
          ([0, 0, 0, 300, 300], 300),              # every row in one group
          ([7, 20, 33, 290], 300),                 # rows before and behind the groups
          ([0] * 513, 40),                         # no rows at all
          (list(range(0, 513)), 512)]              # one row per group


@pytest.mark.parametrize("offsets,Mr", GROUPS, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("dtype,swiglu", [("bf16", False), ("f16", True), ("f32", False),
                                          ("f32", True)])
def test_grouped_matmul(offsets, Mr, dtype, swiglu):
    import torch
    G, N, K = len(offsets) - 1, (72 if len(offsets) < 20 else 24), 200
    rows_b = 2 * N if swiglu else N
    a, da = _matrix(Mr, K, 5)
    b, db = _matrix(G * rows_b, K, 6)
    sa, sb = _scales(Mr, 7), _scales(G * rows_b, 8).reshape(G, rows_b)
    sa = sa * np.float32(4 / np.sqrt(K))  # gate values of a few units
    out, buf = filled(Mr, N, 8, dtype, -7.0)
    ws = _header()
    M.matmul_int8(da, dev(sa), _groups(db, G), dev(sb), out, ws,
                  offsets=dev(np.array(offsets, dtype=np.int32)), swiglu=swiglu)
    assert _status(ws) == (0, 0)
    ref = R.matmul_int8(a, sa, b.reshape(G, rows_b, K), sb, offsets, swiglu)
    inside = np.zeros(Mr, dtype=bool)
    inside[offsets[0]:offsets[-1]] = True
    if swiglu:
        ref, gate, up = ref
        tol = _swiglu_tol(gate, up, ref, dtype)[inside]
        assert np.all(np.abs(f64(out) - ref)[inside] <= tol)
    else:
        _check(f64(out)[inside], ref[inside], dtype)
    assert np.all(f64(out)[~inside] == -7) and torch.all(buf[:, N:] == -7)


@pytest.mark.parametrize("N,K,pad", [(72, 200, 8), (300, 1300, 0), (257, 1040, 3)])
@pytest.mark.parametrize("dtype,swiglu", [("bf16", True), ("f16", False), ("f32", False),
                                          ("f32", True)])
def test_grouped_matmul_of_large_groups(N, K, pad, dtype, swiglu):
    """Groups that fill 256-row tiles, between an empty one and a small one; K below and above
    the depth at which the pipeline's shape changes."""
    import torch
    offsets, Mr = [0, 0, 257, 300, 1100, 1111], 1200
    G, rows_b = len(offsets) - 1, 2 * N if swiglu else N
    a, da = _matrix(Mr, K, 21)
    b, db = _matrix(G * rows_b, K, 22)
    sa, sb = _scales(Mr, 23), _scales(G * rows_b, 24).reshape(G, rows_b)
    sa = sa * np.float32(4 / np.sqrt(K))
    out, buf = filled(Mr, N, pad, dtype, -7.0)
    ws = _header()
    M.matmul_int8(da, dev(sa), _groups(db, G), dev(sb), out, ws,
                  offsets=dev(np.array(offsets, dtype=np.int32)), swiglu=swiglu)
    assert _status(ws) == (0, 0)
    ref = R.matmul_int8(a, sa, b.reshape(G, rows_b, K), sb, offsets, swiglu)
    n = offsets[-1]
    if swiglu:
        ref, gate, up = ref
        tol = _swiglu_tol(gate, up, ref, dtype)[:n]
        assert np.all(np.abs(f64(out) - ref)[:n] <= tol)
    else:
        _check(f64(out)[:n], ref[:n], dtype)
    assert np.all(f64(out)[n:] == -7) and torch.all(buf[:, N:] == -7)


def test_swiglu_far_from_zero():
    """Gates from -150 to 150: the activation neither overflows nor turns NaN."""
    import torch
    g = np.arange(-127, 128, 1)[:, None].astype(np.int8)
    sa = np.full(255, 1.2, dtype=np.float32)
    b, sb = np.array([[1], [1]], dtype=np.int8), np.ones(2, dtype=np.float32)
    codes, _ = _codes(255, 1)
    codes.copy_(torch.from_numpy(g))
    bc, _ = _codes(2, 1)
    bc.copy_(torch.from_numpy(b))
    out, ws = torch.empty(255, 1, device="cuda"), _header()
    M.matmul_int8(codes, dev(sa), bc, dev(sb), out, ws, swiglu=True)
    assert _status(ws) == (0, 0)
    ref, gate, up = R.matmul_int8(g, sa, b[None], sb[None], None, True)
    assert np.all(np.abs(f64(out) - ref) <= _swiglu_tol(gate, up, ref, "f32"))


def test_not_a_number_scales_and_the_fp16_range():
    import torch
    a, da = _matrix(4, 64, 9)
    b, db = _matrix(8, 64, 10)
    sa, sb = np.array([1, np.nan, 1e-3, 0], dtype=np.float32), np.ones(8, dtype=np.float32)
    out, ws = torch.zeros(4, 8, device="cuda"), _header()
    M.matmul_int8(da, dev(sa), db, dev(sb), out, ws)
    assert _status(ws) == (0, 0)
    got = f64(out)
    assert np.isnan(got[1]).all() and np.isfinite(got[[0, 2, 3]]).all() and not got[3].any()
    half = torch.zeros(4, 8, device="cuda", dtype=torch.float16)
    M.matmul_int8(da, dev(sa * 100), db, dev(sb), half, ws)  # sums of some 1e4, times 100
    assert _status(ws)[0] == M.MOE_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("Mr,N,K", [(1, 3, 5000), (1, 8192, 4100), (2, 129, 2049), (3, 64, 15),
                                    (5, 257, 513), (16, 100, 1000), (17, 100, 1000),
                                    (16, 4096, 1024), (40, 128, 4096), (95, 200, 2048),
                                    (33, 1200, 1500), (70, 2500, 6200), (300, 900, 600),
                                    (520, 1100, 300), (600, 1300, 300)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_few_rows(Mr, N, K, swiglu):
    """The sizes around which the product changes its kernel, with the end of the last row at
    the end of its allocation."""
    import torch
    rows_b = 2 * N if swiglu else N
    rng = np.random.default_rng(31)
    a = rng.integers(-127, 128, size=(Mr, K)).astype(np.int8)
    b = rng.integers(-127, 128, size=(rows_b, K)).astype(np.int8)
    pitch = (K + 15) // 16 * 16
    def tight(v):
        flat = torch.full(((v.shape[0] - 1) * pitch + K,), 99, dtype=torch.int8, device="cuda")
        t = flat.as_strided(v.shape, (pitch, 1))
        t.copy_(torch.from_numpy(v))
        return t
    sa, sb = _scales(Mr, 32) * np.float32(4 / np.sqrt(K)), _scales(rows_b, 33)
    out, buf = filled(Mr, N, 5, "f32", -7.0)
    ws = _header()
    M.matmul_int8(tight(a), dev(sa), tight(b), dev(sb), out, ws, swiglu=swiglu)
    assert _status(ws) == (0, 0)
    ref = R.matmul_int8(a, sa, b[None], sb[None], None, swiglu)
    if swiglu:
        ref, gate, up = ref
        assert np.all(np.abs(f64(out) - ref) <= _swiglu_tol(gate, up, ref, "f32"))
    else:
        _check(f64(out), ref, "f32")
    assert torch.all(buf[:, N:] == -7)


@pytest.mark.parametrize("Mr", [1, 8, 16])
@pytest.mark.parametrize("offsets", [None, [0, 0, 2, 2, 5, 16], [0, 16, 16, 16, 16, 16],
                                     [3, 4, 4, 6, 6, 7], [0, 9, 4, 30, 2, -1]], ids=str)
def test_few_rows_in_groups(Mr, offsets):
    """One expert's row each, empty groups, rows before and behind the groups, bad offsets."""
    import torch
    G, N, K = (300 if offsets is None else len(offsets) - 1), 40, 96
    if offsets is None:
        offsets = sorted(np.random.default_rng(34).integers(0, Mr + 1, size=G - 1).tolist())
        offsets = [0] + offsets + [Mr]
    a, da = _matrix(Mr, K, 35)
    b, db = _matrix(G * N, K, 36)
    out, _ = filled(Mr, N, 0, "f32", -7.0)
    ws = _header()
    M.matmul_int8(da, torch.ones(Mr, device="cuda"), _groups(db, G),
                  torch.ones(G * N, device="cuda"), out, ws,
                  offsets=dev(np.array(offsets, dtype=np.int32)))
    bad = any(o < 0 or o > Mr for o in offsets) or offsets != sorted(offsets)
    assert _status(ws)[0] == (M.MOE_ERR_DEVICE_BOUNDS if bad else M.MOE_OK)
    got = f64(out)
    for r in range(Mr):
        ends = np.clip(np.array(offsets[1:]), 0, Mr)
        g = next((i for i, e in enumerate(ends) if e > r), None)
        if r < offsets[0] or g is None:
            assert np.all(got[r] == -7), r
        else:
            ref = b[g * N:(g + 1) * N].astype(np.float64) @ a[r].astype(np.float64)
            assert np.array_equal(got[r], ref), r


@pytest.mark.parametrize("offsets", [[0, 30, 20, 40], [-5, 10, 20, 40], [0, 10, 20, 400],
                                     [40, 30, 20, 10], [0, 2 ** 31 - 1, -2 ** 31, 40]])
def test_bad_offsets_are_clamped_and_reported(offsets):
    import torch
    a, da = _matrix(40, 64, 11)
    b, db = _matrix(3 * 16, 64, 12)
    out, buf = filled(40, 16, 16, "f32", -7.0)
    ws = _header()
    one = torch.ones(48, device="cuda")
    M.matmul_int8(da, one[:40], _groups(db, 3), one, out, ws,
                  offsets=dev(np.array(offsets, dtype=np.int32)))
    assert _status(ws) == (M.MOE_ERR_DEVICE_BOUNDS, 23)
    assert torch.all(buf[:, 16:] == -7)
    # every row that was written holds the products with one group
    z = [R.matmul_int8(a, np.ones(40), b[None, 16 * g:16 * g + 16], np.ones((1, 16)))
         for g in range(3)]
    got = f64(out)
    for r in range(40):
        assert np.all(got[r] == -7) or any(np.array_equal(got[r], zg[r]) for zg in z)


@pytest.mark.parametrize("Mr,offsets,tile", [(17, [0, 9, 17], 128), (64, None, 256)])
def test_more_items_than_a_block_lists(Mr, offsets, tile):
    """Some 5 million channels: over 256 tiles for every block, the last ones of which are found
    by the search alone."""
    import torch
    N, K = tile * (148 if tile == 128 else 74) * 262, 16
    G = 1 if offsets is None else len(offsets) - 1
    g = torch.Generator(device="cuda").manual_seed(41)
    a = torch.randint(-127, 128, (Mr, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-127, 128, (G, N, K), generator=g, device="cuda", dtype=torch.int8)
    out, ws = torch.full((Mr, N), -7.0, device="cuda"), _header()
    M.matmul_int8(a, torch.ones(Mr, device="cuda"), b if offsets else b[0],
                  torch.ones(G * N, device="cuda"), out, ws,
                  offsets=offsets and dev(np.array(offsets, dtype=np.int32)))
    assert _status(ws) == (0, 0)
    for i, (lo, hi) in enumerate(zip(offsets or [0], (offsets or [0, Mr])[1:])):
        for c in range(0, N, 1 << 20):  # sums below 2^24: exact in float32
            want = a[lo:hi].float() @ b[i, c:c + (1 << 20)].float().t()
            assert torch.equal(out[lo:hi, c:c + (1 << 20)], want)


def test_zero_rows():
    import torch
    e, s = torch.empty(0, 32, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    M.quantize_int8(torch.empty(0, 32, device="cuda"), e, s)
    b = torch.zeros(16, 32, dtype=torch.int8, device="cuda")
    M.matmul_int8(e, s, b, torch.ones(16, device="cuda"), torch.empty(0, 16, device="cuda"),
                  _header())


def test_two_products_at_once_on_two_streams_and_captured():
    import torch
    a, da = _matrix(700, 512, 13)
    b, db = _matrix(640, 512, 14)
    sa, sb = dev(_scales(700, 15)), dev(_scales(640, 16))
    want = torch.empty(700, 640, device="cuda")
    M.matmul_int8(da, sa, db, sb, want, _header())
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(want) for _ in range(4)] for _ in streams]
    heads = [_header() for _ in streams]
    torch.cuda.synchronize()
    for i in range(4):
        for s, o, w in zip(streams, outs, heads):
            M.matmul_int8(da, sa, db, sb, o[i], w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for o in outs for t in o)
    live = torch.zeros_like(da)
    out, ws = torch.zeros_like(want), _header()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.matmul_int8(live, sa, db, sb, out, ws)
    live.copy_(da)
    graph.replay()
    assert _status(ws) == (0, 0) and torch.equal(out, want)
