"""Rows to expert order and back, and their gradients, against the float64 oracle.

Tolerances count roundings: u = half a step of the output type, 2^-24 one fp32 operation,
times the sum of the magnitudes that enter the sum.
"""
import numpy as np
import pytest

from oracle import rows_oracle as R
from sparse_moe_layer_select_b200 import moe as M
from tests.rows_common import (DTYPES, dev, f64, filled, floor, half_step, routing, rows,
                               torch_dtype)

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
SCALE = 2.5

# (T, d, E, k, row padding, share of padding tokens, single slots not routed)
SHAPES = [(1, 1, 1, 1, 0, 0.0, False),        # one element
          (1, 2048, 256, 8, 0, 0.0, False),   # one token
          (64, 2048, 256, 8, 0, 0.1, False),  # a decode batch
          (37, 1003, 60, 6, 5, 0.2, True),    # 16-byte rows (fp16/bf16), a ragged last chunk
          (129, 1003, 60, 6, 3, 0.1, True),   # rows at even offsets
          (50, 77, 512, 16, 0, 0.0, True),    # rows at odd offsets
          (5, 4224, 16, 16, 8, 0.5, False),
          (600, 64, 8, 8, 0, 0.0, False),     # more than one index chunk, every expert
          (3, 9000, 4, 2, 0, 1.0, False)]     # nothing routed at all


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    torch.cuda.set_device(0)
    from sparse_moe_layer_select_b200 import build as B
    B.build()
    yield


def _dims(T, d, E, k, norm=1, scale=SCALE):
    return M.make_dims(T, d, E, k, 0, 0, scale, norm)


def _status(ws):
    import torch
    torch.cuda.synchronize()
    return M.read_device_status(ws)


def _close(got, ref, tol):
    err = np.abs(got - ref)
    assert np.all(err <= tol), (float((err / np.maximum(tol, 1e-300)).max()),
                                np.argwhere(err > tol)[:3].tolist())


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", DTYPES)
def test_sort_and_dispatch(shape, dtype):
    import torch
    T, d, E, k, pad, masked, partial = shape
    _, idx, _ = routing(T, E, k, 1, masked, partial)
    dims = _dims(T, d, E, k)
    x = rows(T, d, pad, dtype, 2)
    x_perm, buf = filled(T * k, d, pad, dtype, -7.0)
    ws = M.alloc_sort_workspace(dims)
    out = M.alloc_sort(dims)
    out["perm"].fill_(-7)
    M.sort(dims, dev(idx), out, ws, x=x, x_perm=x_perm)
    assert _status(ws) == (0, 0)
    counts, offsets, perm, inv = R.expert_order(idx, E)
    n = len(perm)
    assert np.array_equal(out["counts"].cpu(), counts)
    assert np.array_equal(out["offsets"].cpu(), offsets)
    assert np.array_equal(out["perm"].cpu()[:n], perm)
    assert np.all(out["perm"].cpu().numpy()[n:] == -7)  # behind the last routed row
    assert np.array_equal(out["inv"].cpu(), inv)
    ref = R.dispatch(f64(x), inv, np.full((T * k, d), -7.0))
    assert np.array_equal(f64(x_perm), ref)
    assert torch.all(buf[:, d:] == -7.0)
    # the copy alone, from the inverse
    again, _ = filled(T * k, d, pad, dtype, -7.0)
    M.dispatch(dims, x, out["inv"], again, ws)
    assert _status(ws) == (0, 0)
    assert torch.equal(again, x_perm)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("f16", "bf16"), ("f16", "f16"),
                                             ("f32", "f32"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("with_add", [False, True])
def test_combine_and_dispatch_backward(shape, dtype, out_dtype, with_add):
    import torch
    T, d, E, k, pad, masked, partial = shape
    _, idx, w = routing(T, E, k, 3, masked, partial)
    inv = R.expert_order(idx, E)[3]
    n = int((inv >= 0).sum())
    dims = _dims(T, d, E, k)
    o = rows(T * k, d, pad, dtype, 4)
    o[n:] = float("nan")  # rows that no slot names are not read
    add = rows(T, d, pad, dtype, 5) if with_add else None
    ws = M.alloc_sort_workspace(dims)
    ref_add = f64(add) if with_add else None
    u = half_step(out_dtype)
    for weight in (w, None):
        y, buf = filled(T, d, pad, out_dtype, -7.0)
        if weight is None:
            M.dispatch_backward(dims, o, dev(inv.astype(np.int32)), y, ws, add=add)
        else:
            M.combine(dims, o, dev(inv.astype(np.int32)), dev(w), y, ws, shared=add)
        assert _status(ws) == (0, 0)
        ref, mag = R.to_tokens(f64(o), inv, weight, SCALE if weight is not None else 1.0, ref_add)
        # k products or sums, the scale and the addend in fp32, then one rounding
        _close(f64(y), ref, (k + 3) * U32 * mag * (1 + u) + u * np.abs(ref) + floor(out_dtype))
        assert torch.all(buf[:, d:] == -7.0)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", DTYPES)
def test_combine_backward(shape, dtype):
    import torch
    T, d, E, k, pad, masked, partial = shape
    _, idx, w = routing(T, E, k, 6, masked, partial)
    inv = R.expert_order(idx, E)[3]
    n = int((inv >= 0).sum())
    dims = _dims(T, d, E, k)
    dy, o = rows(T, d, pad, dtype, 7), rows(T * k, d, pad, dtype, 8)
    o[n:] = float("nan")
    d_o, buf = filled(T * k, d, pad, dtype, -7.0)
    d_w = torch.full((T, k), -7.0, device="cuda")
    ws = M.alloc_sort_workspace(dims)
    inv32 = dev(inv.astype(np.int32))
    M.combine_backward(dims, dy, o, inv32, dev(w), d_o, d_w, ws)
    assert _status(ws) == (0, 0)
    ref_o, ref_w, mag = R.combine_backward(f64(dy), f64(o), inv, w, SCALE)
    u = half_step(dtype)
    _close(f64(d_o)[:n], ref_o[:n], (2 * U32 * (1 + u) + u) * np.abs(ref_o[:n]) + floor(dtype))
    assert torch.all(d_o[n:] == -7.0) and torch.all(buf[:, d:] == -7.0)
    # a row's products are summed by 32 lanes at least: chains of d / 32 terms and a chunk's
    # rest, five sums over the lanes, the scale
    _close(f64(d_w), ref_w, (d / 32 + 16) * U32 * mag)
    # the gradient in place of the rows
    w2 = torch.empty_like(d_w)
    M.combine_backward(dims, dy, o, inv32, dev(w), o, w2, ws)
    torch.cuda.synchronize()
    assert torch.equal(o[:n], d_o[:n]) and torch.equal(w2, d_w)


@pytest.mark.parametrize("norm", [0, 1])
@pytest.mark.parametrize("T,E,k,masked,spread", [(1, 1, 1, 0.0, 1.0), (64, 256, 8, 0.1, 1.0),
                                                 (333, 61, 6, 0.2, 3.0), (40, 512, 16, 0.0, 10.0),
                                                 (5, 16, 16, 1.0, 1.0)])
def test_route_backward(norm, T, E, k, masked, spread):
    import torch
    logits, idx, _ = routing(T, E, k, 9, masked, T == 333)
    logits = logits * np.float32(spread)
    d_w = np.random.default_rng(10).normal(size=(T, k)).astype(np.float32)
    dims = _dims(T, 64, E, k, norm)
    out = torch.full((T, E), float("nan"), device="cuda")
    ws = M.alloc_sort_workspace(dims)
    M.route_backward(dims, dev(logits), dev(idx), dev(d_w), out, ws)
    assert _status(ws) == (0, 0)
    ref = R.route_backward(logits.astype(np.float64), idx, d_w.astype(np.float64), norm)
    w = R.route_weights(logits.astype(np.float64), idx, norm)
    mag = np.zeros((T, E))
    q = R.sigmoid(-logits.astype(np.float64))
    for j in range(k):
        on = idx[:, j] >= 0
        g = np.abs(d_w[on, j]) + (np.abs(d_w[on] * w[on]).sum(1) if norm else 0)
        mag[on, idx[on, j]] += w[on, j] * q[on, idx[on, j]] * g
    # exp of a log-sigmoid of magnitude up to |l|: |l| roundings' worth of relative error in the
    # weight, twice with the maximum's; some 16 operations of a step or two each
    worst = 16 * 2 + 4 * float(np.abs(logits).max())
    _close(f64(out), ref, worst * U32 * mag)
    assert np.all(f64(out)[ref == 0] == 0)


def test_route_backward_with_saturated_and_repeated_scores():
    """Scores that underflow as a row, a score of exactly 0 or 1, the same expert twice."""
    import torch
    dims = _dims(4, 64, 8, 2)
    logits = np.zeros((4, 8), dtype=np.float32)
    logits[0, :2] = [-300.0, -301.0]   # both scores are 0 in fp32; their weights are not
    logits[1, :2] = [200.0, -200.0]
    logits[2, :2] = [np.inf, -np.inf]
    idx = np.array([[0, 1], [0, 1], [0, 1], [3, 3]], dtype=np.int32)
    d_w = np.array([[1.0, -2.0], [1.0, 1.5], [1.0, 1.5], [1.0, 2.0]], dtype=np.float32)
    out = torch.full((4, 8), float("nan"), device="cuda")
    M.route_backward(dims, dev(logits), dev(idx), dev(d_w), out)
    got = f64(out)
    p = np.array([1.0, np.exp(-1.0)]) / (1 + np.exp(-1.0))
    assert np.allclose(got[0, :2], p * (d_w[0] - (d_w[0] * p).sum()), rtol=1e-5, atol=0)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got[1]) < 1e-30) and np.all(got[2] == 0)
    # each slot of the repeated expert has weight 1/2 and slope 1/2: the gradients cancel
    assert abs(got[3, 3]) < 1e-7 and np.all(np.delete(got[3], 3) == 0)


def test_gradients_against_differences():
    """The combine is linear in its rows and in its weights, so its gradients are its adjoint:
    <d_o, v> = <d_y, combine(v)>.  The router's gradient against central differences."""
    import torch
    T, d, E, k = 40, 160, 16, 4
    logits, idx, w = routing(T, E, k, 11, 0.1, True)
    inv = R.expert_order(idx, E)[3]
    inv32 = dev(inv.astype(np.int32))
    dims = _dims(T, d, E, k)
    dy, o, v = (rows(n, d, 0, "f32", s) for n, s in ((T, 12), (T * k, 13), (T * k, 14)))
    vw = np.random.default_rng(15).normal(size=(T, k)).astype(np.float32) * (idx >= 0)
    d_o, d_w = torch.zeros_like(o), torch.zeros(T, k, device="cuda")
    M.combine_backward(dims, dy, o, inv32, dev(w), d_o, d_w)
    y_v, y_w = torch.empty_like(dy), torch.empty_like(dy)
    M.combine(dims, v, inv32, dev(w), y_v)
    M.combine(dims, o, inv32, dev(vw), y_w)
    dx = torch.empty_like(dy)
    M.dispatch_backward(dims, v, inv32, dx)
    x_perm = torch.zeros_like(o)
    M.dispatch(dims, dy, inv32, x_perm)
    dot = lambda a, b: float((f64(a) * f64(b)).sum())  # noqa: E731
    size = float(np.linalg.norm(f64(dy)) * np.linalg.norm(f64(v)) * SCALE)
    assert abs(dot(d_o, v) - dot(dy, y_v)) <= 1e-6 * size
    assert abs(dot(d_w, torch.from_numpy(vw)) - dot(dy, y_w)) <= 1e-6 * size
    assert abs(dot(x_perm, v) - dot(dy, dx)) <= 1e-6 * size
    for norm in (0, 1):
        g = torch.empty(T, E, device="cuda")
        M.route_backward(_dims(T, d, E, k, norm), dev(logits), dev(idx), d_w, g)
        h, vl = 1e-6, np.random.default_rng(16).normal(size=(T, E))
        l = logits.astype(np.float64)
        diff = (R.route_weights(l + h * vl, idx, norm) - R.route_weights(l - h * vl, idx, norm))
        num = (diff / (2 * h) * f64(d_w)).sum(1)
        ana = (f64(g) * vl).sum(1)
        # differences: truncation of order h^2 and 1e-16 / h of cancellation; fp32 in g
        assert np.all(np.abs(num - ana) <= 1e-5 * np.abs(f64(d_w)).sum(1) + 1e-12)


def test_not_a_number_where_nothing_is_routed():
    """NaN in the weights, gradients and logits of slots and experts that do not count."""
    import torch
    T, d, E, k = 50, 136, 16, 4
    logits, idx, w = routing(T, E, k, 50, 0.3, True)
    off = idx < 0
    inv = R.expert_order(idx, E)[3]
    dims, ws = _dims(T, d, E, k), M.alloc_sort_workspace(_dims(T, d, E, k))
    o, dy = rows(T * k, d, 0, "bf16", 51), rows(T, d, 0, "bf16", 52)
    inv32, bad_w = dev(inv.astype(np.int32)), np.where(off, np.float32("nan"), w)
    both = []
    for weight in (w, bad_w):
        y, d_o = torch.empty_like(dy), torch.zeros_like(o)
        d_w = torch.empty(T, k, device="cuda")
        M.combine(dims, o, inv32, dev(weight), y, ws)
        M.combine_backward(dims, dy, o, inv32, dev(weight), d_o, d_w, ws)
        both.append((y, d_o, d_w))
    assert all(torch.equal(a, b) for a, b in zip(*both))
    g = both[0][2].clone()
    clean, dirty = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    M.route_backward(dims, dev(logits), dev(idx), g, clean, ws)
    chosen = np.zeros((T, E), dtype=bool)
    t, j = np.nonzero(~off)
    chosen[t, idx[t, j]] = True
    g[dev(off)] = float("nan")
    M.route_backward(dims, dev(np.where(chosen, logits, np.float32("nan"))), dev(idx), g, dirty, ws)
    assert torch.equal(clean, dirty) and _status(ws) == (0, 0)


@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("f32", 1)])
def test_sums_in_place_of_their_addend(dtype, pad):
    import torch
    T, d, E, k = 77, 200, 16, 4
    _, idx, w = routing(T, E, k, 60, 0.1)
    inv = dev(R.expert_order(idx, E)[3].astype(np.int32))
    dims = _dims(T, d, E, k)
    o, add = rows(T * k, d, pad, dtype, 61), rows(T, d, pad, dtype, 62)
    for call in (lambda y, a: M.combine(dims, o, inv, dev(w), y, shared=a),
                 lambda y, a: M.dispatch_backward(dims, o, inv, y, add=a)):
        apart = filled(T, d, pad, dtype, 0.0)[0]
        call(apart, add)
        same = filled(T, d, pad, dtype, 0.0)[0]
        same.copy_(add)
        call(same, same)
        assert torch.equal(apart, same)


def test_calls_on_two_streams_at_once():
    import torch
    T, d, E, k = 500, 512, 32, 4
    _, idx, w = routing(T, E, k, 70, 0.1)
    dims, di, dw = _dims(T, d, E, k), dev(idx), dev(w)
    x = rows(T, d, 0, "bf16", 71)
    work = []
    for _ in range(2):
        r, xp = M.alloc_sort(dims), torch.zeros(T * k, d, dtype=torch.bfloat16, device="cuda")
        work.append((torch.cuda.Stream(), M.alloc_sort_workspace(dims), r, xp, torch.zeros_like(x)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, ws, r, xp, y in work:
            M.sort(dims, di, r, ws, x=x, x_perm=xp, stream=s)
            M.combine(dims, xp, r["inv"], dw, y, ws, stream=s)
    torch.cuda.synchronize()
    (_, ws, r, xp, y), (_, ws2, r2, xp2, y2) = work
    assert _status(ws) == (0, 0) and _status(ws2) == (0, 0)
    n = int(r["offsets"][-1])
    assert torch.equal(r["inv"], r2["inv"]) and torch.equal(xp[:n], xp2[:n]) and torch.equal(y, y2)
    assert torch.equal(r["inv"].cpu(), torch.from_numpy(R.expert_order(idx, E)[3].astype(np.int32)))


def test_out_of_range_rows_and_experts_are_skipped_and_reported():
    import torch
    T, d, E, k = 6, 32, 4, 2
    dims = _dims(T, d, E, k)
    inv = np.arange(T * k, dtype=np.int32).reshape(T, k)
    bad = inv.copy()
    bad[2, 1], bad[4, 0] = T * k, -2
    kept = np.where((bad >= 0) & (bad < T * k), bad, -1)
    w = np.ones((T, k), dtype=np.float32)
    x, o = rows(T, d, 0, "f32", 20), rows(T * k, d, 0, "f32", 21)
    calls = [lambda i, ws, out: M.dispatch(dims, x, i, out[0], ws),
             lambda i, ws, out: M.combine(dims, o, i, dev(w), out[1], ws),
             lambda i, ws, out: M.dispatch_backward(dims, o, i, out[1], ws),
             lambda i, ws, out: M.combine_backward(dims, x, o, i, dev(w), out[0], out[2], ws),
             lambda i, ws, out: M.dispatch_int8(dims, x, i, out[3], out[4], ws)]
    for call in calls:
        got = []
        for i, code in ((bad, M.MOE_ERR_DEVICE_BOUNDS), (kept, M.MOE_OK)):
            ws = M.alloc_sort_workspace(dims)
            out = (torch.zeros(T * k, d, device="cuda"), torch.zeros(T, d, device="cuda"),
                   torch.zeros(T, k, device="cuda"),
                   torch.zeros(T * k, d, dtype=torch.int8, device="cuda"),
                   torch.zeros(T * k, device="cuda"))
            call(dev(i), ws, out)
            assert _status(ws)[0] == code
            got.append(out)
        assert all(torch.equal(a, b) for a, b in zip(*got))
    idx = np.array([[0, 1], [9, 2], [-3, 3], [1, 0], [2, 3], [0, 2]], dtype=np.int32)
    ws = M.alloc_sort_workspace(dims)
    g = torch.empty(T, E, device="cuda")
    M.route_backward(dims, torch.zeros(T, E, device="cuda"), dev(idx), dev(w), g, ws)
    assert _status(ws)[0] == M.MOE_ERR_DEVICE_BOUNDS
    ref = R.route_backward(np.zeros((T, E)), np.where((idx < 0) | (idx >= E), -1, idx), w, 1)
    assert np.allclose(f64(g), ref, atol=1e-6)
    # a run of calls on one header: the first error stays until moe_sort clears it
    M.dispatch(dims, x, dev(kept), torch.zeros(T * k, d, device="cuda"), ws)
    assert _status(ws)[0] == M.MOE_ERR_DEVICE_BOUNDS
    good = np.where((idx < 0) | (idx >= E), -1, idx).astype(np.int32)
    M.sort(dims, dev(good), M.alloc_sort(dims), ws)
    assert _status(ws) == (0, 0)


def test_zero_tokens():
    import torch
    dims = _dims(0, 64, 8, 2)
    out = M.alloc_sort(dims)
    out["counts"].fill_(5)
    out["offsets"].fill_(5)
    e = torch.empty(0, 64, device="cuda")
    i, w = torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda")
    M.sort(dims, i, out, M.alloc_sort_workspace(dims), x=e, x_perm=e)
    torch.cuda.synchronize()
    assert int(out["offsets"].abs().sum()) == 0 and int(out["counts"].abs().sum()) == 0
    M.dispatch(dims, e, i, e)
    M.combine(dims, e, i, w, e)
    M.dispatch_backward(dims, e, i, e)
    M.combine_backward(dims, e, e, i, w, e, w)
    M.route_backward(dims, torch.empty(0, 8, device="cuda"), i, w, torch.empty(0, 8, device="cuda"))


def _step(dims, idx, w, logits, x, dy, weights, buf, ws, stream=None):
    """A training step's routing around one linear map per expert, from the public calls."""
    r = buf["r"]
    E = dims.num_experts
    M.sort(dims, idx, r, ws, x=x, x_perm=buf["x_perm"], stream=stream)
    # the experts themselves: every row times every expert's matrix, its own kept
    e_of = (buf["row"][:, None] >= r["offsets"][None, 1:E + 1]).sum(1).clamp(max=E - 1)
    live = (buf["row"] < r["offsets"][E])[:, None]
    wt = weights[e_of]
    torch_o = (buf["x_perm"][:, None, :] @ wt)[:, 0] * live
    buf["o"].copy_(torch_o)
    M.combine(dims, buf["o"], r["inv"], w, buf["y"], ws, stream=stream)
    M.combine_backward(dims, dy, buf["o"], r["inv"], w, buf["d_o"], buf["d_w"], ws, stream=stream)
    buf["dxp"].copy_((buf["d_o"][:, None, :] @ wt.transpose(1, 2))[:, 0] * live)
    M.dispatch_backward(dims, buf["dxp"], r["inv"], buf["dx"], ws, stream=stream)
    M.route_backward(dims, logits, idx, buf["d_w"], buf["d_logits"], ws, stream=stream)


def test_training_step_against_autograd_in_64_bits_eager_captured_and_on_a_stream():
    import torch
    T, d, E, k = 96, 64, 16, 4
    logits, idx, _ = routing(T, E, k, 30, 0.1)
    dims = _dims(T, d, E, k)
    w = R.route_weights(logits.astype(np.float64), idx, True).astype(np.float32)
    g = torch.Generator().manual_seed(31)
    x, dy = torch.randn(T, d, generator=g).cuda(), torch.randn(T, d, generator=g).cuda()
    weights = (torch.randn(E, d, d, generator=g) / 8).cuda()
    new = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731

    def buffers():
        return {"r": M.alloc_sort(dims), "row": torch.arange(T * k, device="cuda"),
                "x_perm": new(T * k, d), "o": new(T * k, d), "y": new(T, d), "d_o": new(T * k, d),
                "d_w": new(T, k), "dxp": new(T * k, d), "dx": new(T, d), "d_logits": new(T, E)}

    di, dw, dl = dev(idx), dev(w), dev(logits)
    ws, buf = M.alloc_sort_workspace(dims), buffers()
    _step(dims, di, dw, dl, x, dy, weights, buf, ws)
    assert _status(ws) == (0, 0)

    # the same step in float64 autograd, on the CPU
    lx = torch.from_numpy(f64(x)).requires_grad_()
    ll = torch.from_numpy(logits.astype(np.float64)).requires_grad_()
    on = torch.from_numpy(idx >= 0)
    at = torch.from_numpy(np.where(idx >= 0, idx, 0).astype(np.int64))
    s = torch.sigmoid(torch.gather(ll, 1, at)) * on
    p = s / torch.where(on.any(1), s.sum(1), torch.ones(())).unsqueeze(1)
    full = torch.einsum("td,edf->tef", lx, weights.double().cpu())
    y = SCALE * (p.unsqueeze(-1) * torch.gather(full, 1, at.unsqueeze(-1).expand(-1, -1, d))).sum(1)
    y.backward(torch.from_numpy(f64(dy)))
    rel = lambda a, b: np.linalg.norm(f64(a) - b) / np.linalg.norm(b)  # noqa: E731
    # fp32 sums of d products twice over: far below 1e-5 in the norm
    assert rel(buf["y"], y.detach().numpy()) < 1e-5
    assert rel(buf["dx"], lx.grad.numpy()) < 1e-5
    assert rel(buf["d_logits"], ll.grad.numpy()) < 1e-5

    # captured once, replayed on other inputs; then on a stream of its own
    want = {n: t.clone() for n, t in buf.items() if n != "r"}
    cap = buffers()
    cx = torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(dims, di, dw, dl, cx, dy, weights, cap, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(dims, di, dw, dl, cx, dy, weights, cap, ws)
    cx.copy_(x)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for n in ("x_perm", "y", "d_o", "d_w", "dx", "d_logits"):
        assert torch.equal(cap[n], want[n]), n
    own = buffers()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # torch's products on the same stream
        _step(dims, di, dw, dl, x, dy, weights, own, ws, stream=side)
    side.synchronize()
    assert torch.equal(own["dx"], want["dx"]) and torch.equal(own["d_logits"], want["d_logits"])


def test_binding_refuses_what_does_not_fit():
    import torch
    T, d, E, k = 4, 32, 4, 2
    dims = _dims(T, d, E, k)
    x, inv = torch.zeros(T, d, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
    p = torch.zeros(T * k, d, device="cuda")
    for call in (lambda: M.dispatch(dims, x, inv, p[:-1]),                   # too few rows
                 lambda: M.dispatch(dims, x, inv, p.to(torch.bfloat16)),     # another type
                 lambda: M.dispatch(dims, x, inv.long(), p),
                 lambda: M.dispatch(dims, x.double(), inv, p.double()),
                 lambda: M.dispatch(dims, x.t().contiguous().t(), inv, p),   # rows not contiguous
                 lambda: M.dispatch(dims, x[:1].expand(T, d), inv, p),       # row stride 0
                 lambda: M.dispatch(dims, x.cpu(), inv, p),
                 lambda: M.dispatch(dims, x, inv, p, ws=torch.zeros(16, dtype=torch.uint8,
                                                                    device="cuda"))):
        with pytest.raises(M.MoeError) as e:
            call()
        assert e.value.code == M.MOE_ERR_INVALID_ARG


def test_large_offsets():
    """Row offsets past 2^31 elements: the last token's rows lie behind them."""
    import torch
    T, d, E, k = 33000, 8192, 16, 8   # 264000 rows of 16 KB: 4.3 GB, 2.16e9 elements
    dims = _dims(T, d, E, k)
    idx = torch.arange(k, dtype=torch.int32, device="cuda").repeat(T, 1)
    r, ws = M.alloc_sort(dims), M.alloc_sort_workspace(dims)
    x = torch.randn(T, d, device="cuda", dtype=torch.bfloat16)
    x_perm = torch.empty(T * k, d, device="cuda", dtype=torch.bfloat16)
    M.sort(dims, idx, r, ws, x=x, x_perm=x_perm)
    assert torch.equal(x_perm[-1], x[-1]) and torch.equal(x_perm[-T], x[0])
    y = torch.empty_like(x)
    w = torch.full((T, k), 1 / 8, device="cuda")
    M.combine(_dims(T, d, E, k, scale=1.0), x_perm, r["inv"], w, y)
    assert torch.equal(y, x)  # eight equal rows times 1/8: exact
    d_w = torch.empty_like(w)
    M.combine_backward(_dims(T, d, E, k, scale=8.0), x, x_perm, r["inv"], w, x_perm, d_w, ws)
    assert torch.equal(x_perm[-1], x[-1]) and torch.equal(x_perm[-T], x[0])
    assert _status(ws) == (0, 0)
