"""The layer with int8 experts (MoeLayer(int8=True)) against the same method in float64."""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import rows_oracle as R
from sparse_moe_layer_select_b200 import inputs as I
from sparse_moe_layer_select_b200 import moe as M
from tests import gpu_common as G
from tests import parity as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    torch.cuda.set_device(0)
    from sparse_moe_layer_select_b200 import build as B
    B.build()
    yield


def _bf16(a):
    return (a.astype(np.uint32) << 16).view(np.float32)


def _ffn(q, s, gate, up, down):
    """Rows with codes q and scales s through one SwiGLU expert of bf16 weights, all four
    matrices quantized by rows (codes decided in fp32, products in float64)."""
    b, sb = R.quantize_int8(np.concatenate([_bf16(gate), _bf16(up)]))
    h = R.matmul_int8(q, s, b[None], sb[None], None, True)[0]
    hq, hs = R.quantize_int8(h)
    b, sb = R.quantize_int8(_bf16(down))
    return R.matmul_int8(hq, hs, b[None], sb[None])


def _reference(w, h, idx, wt, x):
    q, s = R.quantize_int8(_bf16(x))
    y = np.zeros((x.shape[0], w.d_model))
    for e in range(w.E):
        t, j = np.nonzero(idx == e)
        if len(t):
            o = _ffn(q[t], s[t], h["w_gate"][e], h["w_up"][e], h["w_down"][e])
            np.add.at(y, t, w.routed_scaling_factor * wt[t, j, None].astype(np.float64) * o)
    if w.Fs:
        y += _ffn(q, s, h["ws_gate"], h["ws_up"], h["ws_down"])
    return y


def _layer(w, dev, **kw):
    return M.MoeLayer(dev, w.d_model, w.E, w.k, w.F, w.Fs, w.routed_scaling_factor,
                      max_tokens=w.T, int8=True, **kw)


@pytest.mark.parametrize("T,Fs", [(64, 128), (1, 128), (300, 0)])
def test_layer_with_int8_experts(T, Fs):
    import torch
    w = I.get("c1_tiny").with_(T=T, shared_intermediate_size=Fs)
    h = I.host_inputs(w)
    dev = G.host_to_device(h)
    layer = _layer(w, dev)
    y = layer.forward(dev["x"])
    torch.cuda.synchronize()
    assert layer.device_status() == (0, 0)
    idx, wt = (layer.routing[n].cpu().numpy()[:T] for n in ("topk_idx", "topk_w"))
    ref = O.route(h["x"], h["w_router"], None, w.k)
    G.check_routing(idx, wt, {"topk_idx": ref[0], "topk_w": ref[1], "scores": ref[2]}, w.k)
    # fp16 contributions and a bf16 sum: half a step of bf16, 2^-9, in the norm, and rarely a
    # code of h on the other side of a border
    want = _reference(w, h, idx, wt, h["x"])
    assert np.linalg.norm(G.y_numpy(y) - want) <= 4e-3 * np.linalg.norm(want)
    # the quantized layer is near the layer itself: four quantizations of about 1% each
    full = G.oracle_forward(w, h)["y"]
    assert np.linalg.norm(want - full) <= 0.05 * np.linalg.norm(full)
    # smaller batches in the same buffers, tokens masked, captured and replayed
    if T == 300:
        mask = torch.ones(100, dtype=torch.uint8, device="cuda")
        mask[::3] = 0
        x = dev["x"][:100].contiguous()
        first = layer.forward(x, token_mask=mask)
        idx, wt = (layer.routing[n].cpu().numpy().reshape(-1)[:100 * w.k].reshape(100, w.k)
                   for n in ("topk_idx", "topk_w"))
        assert np.all(idx[::3] == -1) and not G.y_numpy(first)[::3].any()
        want = _reference(w, h, idx, wt, h["x"][:100])
        assert np.linalg.norm(G.y_numpy(first) - want) <= 4e-3 * np.linalg.norm(want)
        live, out = torch.zeros_like(x), torch.zeros_like(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.forward(live, out, token_mask=mask)
        live.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        assert layer.forward(dev["x"][:0]).shape == (0, w.d_model)


def test_one_kind_of_8_bit_experts():
    with pytest.raises(ValueError):
        M.MoeLayer({}, 256, 16, 4, 128, 128, fp8=True, int8=True)
