"""Row operators, 8-bit products and the layers on them at their limits: batches smaller
than the buffers were made for, row offsets past 2^31, scores that underflow."""
import types

import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import rows_oracle as R
from sparse_moe_layer_select_b200 import inputs as I
from sparse_moe_layer_select_b200 import moe as M
from tests import gpu_common as G
from tests.rows_common import dev, f64, routing, torch_dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    torch.cuda.set_device(0)
    from sparse_moe_layer_select_b200 import build as B
    B.build()
    yield


# ---------------------------------------------------------------- smaller batches

@pytest.mark.parametrize("T,most", [(5000, 8192), (6144, 6145), (12288, 12289), (1, 12289)])
def test_sort_of_a_smaller_batch_in_a_larger_ones_workspace(T, most):
    # 49152 and 98304 entries are the last with chunks of 1024 and 2048 entries
    E, k = 256, 8
    dims = M.make_dims(T, 64, E, k, 0, 0)
    ws = M.alloc_sort_workspace(M.make_dims(most, 64, E, k, 0, 0))
    _, idx, _ = routing(T, E, k, 1)
    out = M.alloc_sort(dims)
    M.sort(dims, dev(idx), out, ws)
    assert M.read_device_status(ws) == (0, 0)
    counts, offsets, perm, inv = R.expert_order(idx, E)
    for name, want in (("counts", counts), ("offsets", offsets), ("perm", perm), ("inv", inv)):
        assert np.array_equal(out[name].cpu(), want), name


def test_int8_layer_runs_every_smaller_batch():
    import torch
    w = I.get("c1_tiny").with_(T=12289)  # top-4: the chunks double behind 12288 tokens
    layers = [M.MoeLayer(G.host_to_device(I.host_inputs(w)), w.d_model, w.E, w.k, w.F, w.Fs,
                         w.routed_scaling_factor, max_tokens=most, int8=True)
              for most in (12289, 12288)]
    x = G.host_to_device(I.host_inputs(w))["x"]
    for T in (12288, 9000):
        a, b = (layer.forward(x[:T].contiguous()) for layer in layers)
        torch.cuda.synchronize()
        assert layers[0].device_status() == layers[1].device_status() == (0, 0)
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,most", [(2304, 2310), (9472, 9473)])
@pytest.mark.parametrize("int8", [False, True])
def test_layer_runs_a_batch_with_more_router_planes(T, most, int8):
    import torch
    # 2304 and 9472 tokens are the last that the router takes in four and two slices of d
    w = I.get("c1_tiny").with_(T=most, num_experts=256, num_experts_per_tok=2)
    h = I.host_inputs(w)
    ys = []
    for size in (most, T):
        layer = M.MoeLayer(G.host_to_device(h), w.d_model, w.E, w.k, w.F, w.Fs,
                           w.routed_scaling_factor, max_tokens=size, int8=int8)
        x = G.host_to_device({"x": h["x"][:T]})["x"]
        ys.append(layer.forward(x))
        assert layer.device_status() == (0, 0)
    assert torch.equal(*ys)


# ---------------------------------------------------------------- scores that underflow

@pytest.mark.parametrize("flag,T", [(M.MOE_FLAG_ROUTER_CUDA_CORE, 64), (M.MOE_FLAG_ROUTER_TENSOR, 1030)])
@pytest.mark.parametrize("selection_bias", [False, True])
def test_router_weights_and_gradient_of_scores_that_underflow(flag, T, selection_bias):
    """sigmoid(l) is 0 in fp32 below l = -88.7 and keeps few bits above; the normalised weights
    of such rows are those of their logits all the same."""
    import torch
    E, k, d = 32, 8, 64
    # token t has the logits of column t % d, exactly: distinct values, the largest at `top`
    top = np.array([-20, -43, -45, -80, -87, -88.5, -89, -104, -150, -300])[np.arange(d) % 10]
    rng = np.random.default_rng(4)
    step = np.where(top < -128, 2.0, 0.5)
    W = np.stack([t - s * rng.permutation(E) for t, s in zip(top, step)], 1).astype(np.float32)
    x = np.zeros((T, d), dtype=np.float32)
    x[np.arange(T), np.arange(T) % d] = 1.0
    dims = M.make_dims(T, d, E, k, 64, 0, 2.5, 1,
                       flag | (M.MOE_FLAG_BIAS_SELECTION_ONLY if selection_bias else 0))
    xb, wb = dev(x).bfloat16(), dev(W).bfloat16()
    assert np.array_equal(f64(wb), W)
    bias = rng.normal(size=E).astype(np.float32) if selection_bias else None
    ws = M.alloc_workspace(dims)
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), dtype=torch.float32, device="cuda")
    M.route(dims, xb, wb, None if bias is None else dev(bias), idx, w, ws)
    assert M.read_device_status(ws) == (0, 0)
    logits = W.T.astype(np.float64)[np.arange(T) % d]
    off = M.lib().moe_logits_offset(dims)
    got_l = ws[off:off + 4 * T * E].view(torch.float32).view(T, E)
    assert np.array_equal(f64(got_l), logits)
    sel = idx.cpu().numpy()
    if selection_bias:  # scores are nothing beside the bias, but for the rows at -20: 2e-9
        assert np.array_equal(np.sort(sel[top[np.arange(T) % d] < -40][0]), np.sort(np.argsort(-bias)[:k]))
    else:
        assert np.array_equal(sel, np.argsort(-logits, axis=1, kind="stable")[:, :k])
    l = np.take_along_axis(logits, sel.astype(np.int64), 1)
    s = O.sigmoid(l)
    want = s / s.sum(1, keepdims=True)
    # a difference of two logits (exact), an exponential of two units, twice; k sums, a division.
    # Above 2^-64 (the first two tops) the exponential's argument has no error either.
    tol = (4 + 4 + k + 2) * 2.0 ** -24
    assert np.all(np.abs(f64(w) - want) <= tol * want)
    # and back
    d_w = rng.normal(size=(T, k)).astype(np.float32)
    out = torch.full((T, E), float("nan"), device="cuda")
    M.route_backward(dims, got_l.contiguous(), idx, dev(d_w), out, ws)
    ref = R.route_backward(logits, sel, d_w.astype(np.float64), 1)
    p = R.route_weights(logits, sel, 1)
    mag = np.zeros((T, E))
    np.put_along_axis(mag, sel.astype(np.int64),
                      p * (np.abs(d_w) + (np.abs(d_w) * p).sum(1, keepdims=True)), 1)
    # (log sigmoid of magnitude |l|: |l| roundings of relative error in a weight, twice with the
    # maximum's; some 16 operations of a step or two each)
    worst = 16 * 2 + 4 * np.abs(logits).max(1, keepdims=True)
    assert np.all(np.abs(f64(out) - ref) <= worst * 2.0 ** -24 * mag)


# ---------------------------------------------------------------- weights without a scale

@pytest.mark.parametrize("name,at,value", [("w_gate", (3, 5, 7), np.inf), ("w_up", (15, 127, 255), np.nan),
                                           ("w_down", (0, 0, 0), -np.inf), ("ws_gate", (1, 1), np.nan),
                                           ("ws_up", (0, 255), np.inf), ("ws_down", (255, 0), np.nan)])
def test_int8_weights_with_an_infinity_or_nan_are_refused(name, at, value):
    import torch
    w = I.get("c1_tiny")
    W = G.host_to_device(I.host_inputs(w))
    W[name][at] = value
    raw = types.SimpleNamespace(cuda_stream=torch.cuda.Stream().cuda_stream)
    for stream in (None, torch.cuda.Stream(), raw):
        torch.cuda.synchronize()
        with pytest.raises(M.MoeError) as e:
            M.prepare_int8(W, stream)
        assert e.value.code == M.MOE_ERR_DEVICE_BOUNDS
    with pytest.raises(M.MoeError):
        M.MoeLayer(W, w.d_model, w.E, w.k, w.F, w.Fs, max_tokens=8, int8=True)
    W[name][at] = 1.0
    M.prepare_int8(W)


# ---------------------------------------------------------------- what a layer holds

@pytest.mark.parametrize("T,flag", [(64, 0), (2304, M.MOE_FLAG_ROUTER_TENSOR), (9473, 0)])
def test_router_writes_nothing_behind_its_workspace(T, flag):
    import torch
    w = I.get("c1_tiny").with_(T=T, num_experts=256, num_experts_per_tok=2)
    h = G.host_to_device(I.host_inputs(w))
    dims = M.dims_for(w, flags=flag)
    n = M.route_workspace_size(dims)
    whole = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    outs = []
    for ws in (whole[:n], M.alloc_workspace(dims)):
        idx = torch.empty((T, w.k), dtype=torch.int32, device="cuda")
        wt = torch.empty((T, w.k), device="cuda")
        M.route(dims, h["x"], h["w_router"], None, idx, wt, ws)
        assert M.read_device_status(ws) == (0, 0)
        outs.append((idx, wt))
    assert torch.all(whole[n:] == 0xAB)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("kind", [{}, {"fp8": True}, {"int8": True}])
def test_device_status_before_a_first_batch(kind):
    import torch
    w = I.get("c1_tiny")
    W = G.host_to_device(I.host_inputs(w))
    new = lambda: M.MoeLayer(W, w.d_model, w.E, w.k, w.F, w.Fs, max_tokens=64, **kind)  # noqa: E731
    layer = new()
    layer.ws.fill_(0xFF)  # its memory goes back and is given to the next layer
    del layer
    layer = new()
    assert layer.device_status() == (0, 0)


@pytest.mark.parametrize("kind", [{}, {"fp8": True}, {"int8": True}])
def test_layers_take_no_tokens(kind):
    import torch
    w = I.get("c1_tiny")
    W = G.host_to_device(I.host_inputs(w))
    layer = M.MoeLayer(W, w.d_model, w.E, w.k, w.F, w.Fs, max_tokens=64, **kind)
    before = layer.forward(W["x"])
    assert layer.forward(W["x"][:0]).shape == (0, w.d_model)
    y = torch.empty(0, w.d_model, dtype=torch.bfloat16, device="cuda")
    assert layer.forward(W["x"][:0], y) is y
    assert torch.equal(layer.forward(W["x"]), before) and layer.device_status() == (0, 0)


def test_int8_layer_holds_its_codes_and_not_the_weights():
    import torch
    w = I.get("c1_tiny")
    W = G.host_to_device(I.host_inputs(w))
    layer = M.MoeLayer(W, w.d_model, w.E, w.k, w.F, w.Fs, max_tokens=w.T, int8=True)
    assert layer.ws.numel() == M.route_workspace_size(layer.dims(w.T))
    assert layer.ws.numel() < M.workspace_size(layer.dims(w.T)) / 10
    x = W["x"]
    first = layer.forward(x)
    for n in G.WEIGHT_KEYS[1:]:  # gone or overwritten by their owner, to no effect
        W[n].fill_(float("nan"))
    W.clear()
    assert sorted(n for n, t in layer.W.items() if t is not None) == ["w_router"]
    assert torch.equal(layer.forward(x), first) and layer.device_status() == (0, 0)


# ---------------------------------------------------------------- the activation's error

@pytest.mark.parametrize("rows,grouped", [(16, False), (255, False), (255, True)])
def test_swiglu_error_in_units_of_the_last_place(rows, grouped):
    """The stated bound of silu, on each of the three product kernels: gates of -126 to 126 in
    steps of 1/128 and up values, all exact, so that only the activation and one product round."""
    import torch
    a = np.linspace(-127, 127, rows).round().astype(np.int8)[:, None]
    N = 127
    b = np.concatenate([np.arange(1, N + 1), np.ones(N)]).astype(np.int8)[:, None]
    qa, sa = M.alloc_codes(rows, 1)
    qb, sb = M.alloc_codes(2 * N, 1)
    qa.copy_(dev(a)), qb.copy_(dev(b))
    sa.fill_(1.0)
    sb.fill_(2.0 ** -7)
    out = torch.empty(rows, N, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    if grouped:
        offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        M.matmul_int8(qa, sa, qb[None], sb, out, ws, offsets=offsets, swiglu=True)
    else:
        M.matmul_int8(qa, sa, qb, sb, out, ws, swiglu=True)
    assert M.read_device_status(ws) == (0, 0)
    gate, up, got = a / 128.0 * b[:N].T.astype(np.float64), a / 128.0, f64(out)
    want = gate * R.sigmoid(gate) * up
    units = np.where(gate < 0, 5 + 1.2 * np.abs(gate), 6) + 0.5
    on = gate > -87
    # (a unit is at most 2^-23 of the value, and 2^-149 near zero)
    assert np.all(np.abs(got - want)[on] <= (units * 2.0 ** -23 * np.abs(want) + 2.0 ** -149)[on])
    assert np.all(got[gate < -88] == 0)


# ---------------------------------------------------------------- streams

def test_stream_arguments():
    """What is no stream of the tensors' device is refused, with no error left behind."""
    import torch
    x = torch.ones(4, 64, device="cuda")
    q, s = M.alloc_codes(4, 64)
    raw = torch.cuda.Stream().cuda_stream
    new = types.SimpleNamespace
    for bad in (0, "stream", new(), new(cuda_stream="0"), new(cuda_stream=None), new(cuda_stream=1.5),
                new(cuda_stream=raw, device_index=1)):
        s.fill_(-1.0)
        torch.cuda.synchronize()
        with pytest.raises(M.MoeError) as e:
            M.quantize_int8(x, q, s, stream=bad)
        assert e.value.code == M.MOE_ERR_INVALID_ARG and "stream" in str(e.value)
        torch.cuda.synchronize()
        assert torch.all(s == -1.0)  # nothing was launched
    for good in (None, torch.cuda.Stream(), new(cuda_stream=raw), new(cuda_stream=raw, device_index=0),
                 torch.cuda.default_stream()):
        s.fill_(-1.0)
        torch.cuda.synchronize()
        M.quantize_int8(x, q, s, stream=good)
        torch.cuda.synchronize()
        assert torch.all(s > 0) and torch.all(q == 127)


# ---------------------------------------------------------------- past 32 bits

def test_quantize_of_nearly_2_to_31_rows():
    import torch
    n = (1 << 31) - 2
    x = torch.ones(n, 1, dtype=torch.bfloat16, device="cuda")
    x[-3:, 0] = torch.tensor([2.0, -4.0, 0.0])
    q, s = M.alloc_codes(n, 1)
    s.fill_(-1.0)
    M.quantize_int8(x, q, s)
    one = np.float32(1) / np.float32(127)
    assert int((s == float(one)).sum()) == n - 3
    assert q[-4:, 0].tolist() == [127, 127, -127, 0]
    assert s[-4:].tolist() == [one, np.float32(2) / np.float32(127), np.float32(4) / np.float32(127), 1.0]


def _random_codes(rows, cols, pitch=None):
    """int8 codes [rows, cols] of an LCG over the element's place, rows `pitch` bytes apart."""
    import torch
    q = torch.empty(rows, pitch or (cols + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 28) // q.shape[1])
    c = torch.arange(cols, device="cuda", dtype=torch.int32) * 7919
    for r in range(0, rows, step):
        i = torch.arange(r, min(r + step, rows), device="cuda", dtype=torch.int32)[:, None]
        q[r:r + step, :cols] = (((i * 1103515245 + c) * 48271 >> 11) & 0xff).to(torch.int8)
    return q[:, :cols]


def _check_rows(out, a, sa, b, sb, rows, cols):
    """Elements [rows] x [cols] of a product against float64 (integer sums below 2^53 are
    exact): rounded to fp32, two scales, rounded to the output's type."""
    import torch
    got = out[rows][:, cols].double()
    want = (a[rows].double() @ b[cols].double().t()) * sa[rows].double()[:, None] * \
        sb[cols].double()
    u = torch.finfo(out.dtype).eps / 2
    assert torch.all((got - want).abs() <= (3 * 2.0 ** -24 * (1 + u) + u) * want.abs())


def test_dispatch_int8_past_2_to_31_bytes():
    import torch
    T, d, E, k = 70000, 4096, 16, 8
    dims = M.make_dims(T, d, E, k, 0, 0)
    assert T * k * d > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, d, generator=g, device="cuda", dtype=torch.bfloat16)
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int().contiguous()
    r, ws = M.alloc_sort(dims), M.alloc_sort_workspace(dims)
    M.sort(dims, idx, r, ws)
    q, s = M.alloc_codes(T * k, d)
    M.dispatch_int8(dims, x, r["inv"], q, s, ws)
    one, s1 = M.alloc_codes(T, d)
    M.quantize_int8(x, one, s1)
    assert M.read_device_status(ws) == (0, 0)
    for t in range(0, T, 5000):
        at = r["inv"][t:t + 5000].long()
        assert torch.all(q[at] == one[t:t + 5000, None])
        assert torch.all(s[at] == s1[t:t + 5000, None])


@pytest.mark.parametrize("rows,N,K,pitch", [(600000, 64, 4000, None),   # a past 2^31 bytes
                                            (300000, 8000, 16, None),   # out past 2^31 elements
                                            (300000, 8001, 16, None),   # and rows off 16 bytes
                                            (3000, 70, 100, 1 << 20)])  # rows far apart
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_product_past_2_to_31(rows, N, K, pitch, dtype):
    import torch
    a, b = _random_codes(rows, K, pitch), _random_codes(N, K, pitch)
    g = torch.Generator(device="cuda").manual_seed(2)
    sa, sb = (torch.rand(n, generator=g, device="cuda") + 0.5 for n in (rows, N))
    out = torch.empty(rows, N, device="cuda", dtype={"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    M.matmul_int8(a, sa, b, sb, out, ws)
    assert M.read_device_status(ws) == (0, 0)
    for r in (slice(0, 300), slice(rows // 2, rows // 2 + 300), slice(rows - 300, rows)):
        _check_rows(out, a, sa, b, sb, r, slice(0, N))


@pytest.mark.parametrize("G,rows,N,K", [(512, 28000, 80000, 16),  # out past 2^31 elements
                                        (300, 900, 2000, 4096),   # b past 2^31 bytes
                                        (300, 16, 2000, 4096),    # the same for a few rows
                                        (4, 1, 1 << 26, 16)])
def test_grouped_product_past_2_to_31(G, rows, N, K):
    import torch
    a, b = _random_codes(rows, K), _random_codes(G * N, K)
    g = torch.Generator(device="cuda").manual_seed(3)
    sa, sb = (torch.rand(n, generator=g, device="cuda") + 0.5 for n in (rows, G * N))
    # the last rows are the last group's; the first group has rows too where there are two
    ends = torch.linspace(0, rows, G + 1).round().int()
    if rows <= 16:
        ends = torch.full((G + 1,), rows // 2, dtype=torch.int32)
        ends[0], ends[G] = 0, rows
    out = torch.empty(rows, N, device="cuda", dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    M.matmul_int8(a, sa, b.view(G, N, K), sb, out, ws, offsets=ends.cuda())
    assert M.read_device_status(ws) == (0, 0)
    for e in {0, G // 2, G - 1}:
        lo, hi = int(ends[e]), min(int(ends[e + 1]), int(ends[e]) + 200)
        for c in (slice(0, 2000), slice(N - 2000, N)):
            _check_rows(out, a, sa, b[e * N:(e + 1) * N], sb[e * N:(e + 1) * N], slice(lo, hi), c)


# ---------------------------------------------------------------- the int8 layer's shapes

@pytest.mark.parametrize("T,d,E,k,F,Fs", [(130, 128, 60, 6, 192, 64),    # E off 16: CUDA-core router
                                          (1100, 192, 48, 5, 64, 320),   # rows on 256-row tiles
                                          (5, 64, 512, 16, 64, 0)])
def test_int8_layer_shapes(T, d, E, k, F, Fs):
    import torch
    from tests.test_gpu_int8_layer import _reference
    w = I.get("c1_tiny").with_(T=T, d_model=d, num_experts=E, num_experts_per_tok=k,
                               moe_intermediate_size=F, shared_intermediate_size=Fs)
    h = I.host_inputs(w)
    dv = G.host_to_device(h)
    layer = M.MoeLayer(dv, d, E, k, F, Fs, w.routed_scaling_factor, max_tokens=T // 2, int8=True)
    y = layer.forward(dv["x"])  # more than it was made for: it grows
    torch.cuda.synchronize()
    assert layer.device_status() == (0, 0) and layer.max_tokens == T
    idx, wt = (layer.routing[n].cpu().numpy().reshape(-1)[:T * k].reshape(T, k)
               for n in ("topk_idx", "topk_w"))
    ref = O.route(h["x"], h["w_router"], None, k)
    G.check_routing(idx, wt, {"topk_idx": ref[0], "topk_w": ref[1], "scores": ref[2]}, k)
    # as for the tiny layer: fp16 contributions, a bf16 sum, rarely a code across a border
    want = _reference(w, h, idx, wt, h["x"])
    assert np.linalg.norm(G.y_numpy(y) - want) <= 4e-3 * np.linalg.norm(want)


@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("Fs", [0, 128])
def test_int8_layer_with_no_token_routed_and_with_rows_that_are_not_numbers(T, Fs):
    import torch
    w = I.get("c1_tiny").with_(T=T, shared_intermediate_size=Fs)
    W = G.host_to_device(I.host_inputs(w))
    layer = M.MoeLayer(W, w.d_model, w.E, w.k, w.F, w.Fs, max_tokens=T, int8=True)
    x = W["x"]
    y = layer.forward(x)
    none = layer.forward(x, token_mask=torch.zeros(T, dtype=torch.uint8, device="cuda"))
    assert layer.device_status() == (0, 0)
    assert torch.isfinite(none).all() and int(layer.routing["offsets"][w.E]) == 0
    assert (none == 0).all() == (Fs == 0)  # the shared expert alone
    # a token that is not a number is its own loss only
    bad = x.clone()
    bad[T // 2, 3] = float("nan")
    got = layer.forward(bad)
    others = torch.arange(T, device="cuda") != T // 2
    assert torch.isnan(got[T // 2]).all() and torch.equal(got[others], y[others])
    bad[T // 2, 3] = float("inf")
    got = layer.forward(bad)
    assert torch.isnan(got[T // 2]).all() and torch.equal(got[others], y[others])
    assert torch.equal(layer.forward(x), y) and layer.device_status() == (0, 0)


# ---------------------------------------------------------------- long sums

@pytest.mark.parametrize("d", [8192, 32768, 32770, 32771])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_weight_gradient_of_long_rows(d, dtype):
    """Products of one sign and size, whose running sum rounds the same way again and again: the
    dot product of a row is summed in pieces, so that no chain of roundings is d / 32 long."""
    import torch
    T = 128
    dims = M.make_dims(T, d, 1, 1, 0, 0, 1.0)
    c = np.random.default_rng(6).uniform(0.5, 1.5, T).astype(np.float32)
    rows = dev(c)[:, None].expand(T, d).to(torch_dtype(dtype)).contiguous()
    inv = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
    d_w = torch.empty(T, 1, device="cuda")
    M.combine_backward(dims, rows, rows, inv, torch.ones(T, 1, device="cuda"),
                       torch.empty_like(rows), d_w)
    want = d * f64(rows)[:, 0] ** 2
    # elements of a lane's piece (up to 64 bytes, eight loads at most), its pieces, five sums
    # over the lanes and the scale: one rounding each
    size, chunk = rows.element_size(), 8 if d % 8 == 0 else 2 if d % 2 == 0 else 1
    piece = min(64 // size, 8 * chunk)
    steps = piece + -(-d // (32 * piece)) + 6
    assert np.all(np.abs(f64(d_w)[:, 0] - want) <= steps * 2.0 ** -24 * want)


# ---------------------------------------------------------------- more chunks than fit at once

def test_sort_of_more_slots_than_one_launch_takes():
    import torch
    T, E, k = 400001, 60, 8  # 782 chunks of 4096: histogram and scatter in two launches
    _, idx, _ = routing(T, E, k, 7, 0.1, True)
    dims = M.make_dims(T, 8, E, k, 0, 0)
    x = torch.arange(T, device="cuda", dtype=torch.float32)[:, None].expand(T, 8).contiguous()
    x_perm = torch.full((T * k, 8), -1.0, device="cuda")
    ws, out = M.alloc_sort_workspace(dims), M.alloc_sort(dims)
    ws.fill_(0xFF)
    M.sort(dims, dev(idx), out, ws, x=x, x_perm=x_perm)
    assert M.read_device_status(ws) == (0, 0)
    flat = idx.reshape(-1)
    counts = np.bincount(flat[flat >= 0], minlength=E)
    n = int(counts.sum())
    perm = np.argsort(np.where(flat < 0, E, flat), kind="stable")[:n]
    inv = np.full(T * k, -1)
    inv[perm] = np.arange(n)
    assert np.array_equal(out["counts"].cpu(), counts)
    assert np.array_equal(out["offsets"].cpu(), np.concatenate([[0], np.cumsum(counts)]))
    assert np.array_equal(out["perm"].cpu()[:n], perm)
    assert np.array_equal(out["inv"].cpu().reshape(-1), inv)
    assert np.array_equal(x_perm[:n, 3].cpu(), perm // k) and torch.all(x_perm[n:] == -1)
