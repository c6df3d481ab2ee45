"""Row operators, 8-bit products and the layers on them at their limits: batches smaller
than the buffers were made for, row offsets past 2^31, scores that underflow."""
import numpy as np
import pytest

from oracle import rows_oracle as R
from sparse_moe_layer_select_b200 import inputs as I
from sparse_moe_layer_select_b200 import moe as M
from tests import gpu_common as G
from tests.rows_common import dev, routing

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
