"""Limits of the row operators, the 8-bit products and the layers on them: sizes of
workspaces, refused arguments (no GPU needed: these paths return before any CUDA call)."""
import ctypes
import os

import pytest

from sparse_moe_layer_select_b200 import build as B
from sparse_moe_layer_select_b200 import moe as M


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


@pytest.fixture(scope="module")
def L():
    """The library with 64-bit strides and addresses (ctypes passes plain integers as 32-bit)."""
    lib = ctypes.CDLL(M.LIB_PATH)
    P, I, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.moe_dispatch_backward.argtypes = [P, I, P, S, P, P, S, I, P, S, P, P]
    lib.moe_combine.argtypes = [P, I, P, S, P, P, P, S, I, P, S, P, P]
    lib.moe_combine_backward.argtypes = [P, I, P, S, P, S, P, P, P, S, P, P, P]
    lib.moe_dispatch.argtypes = [P, I, P, S, P, P, S, P, P]
    lib.moe_dispatch_int8.argtypes = [P, I, P, S, P, P, S, P, P, P]
    lib.moe_quantize_int8.argtypes = [I, I, I, P, S, P, P, S, P, P]
    return lib


BAD, SHAPE = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED_SHAPE


# ---------------------------------------------------------------- refused arguments

# addend: type and stride of the rows and of the output that replaces them (no call with
# matching ones here: it would be launched)
@pytest.mark.parametrize("in_type,in_stride,out_type,out_stride", [
    (0, 104, 2, 104), (0, 104, 0, 112), (2, 104, 1, 104), (1, 104, 0, 104), (2, 128, 2, 104)])
def test_sums_in_place_need_one_type_and_stride(L, in_type, in_stride, out_type, out_stride):
    dims = ctypes.byref(M.make_dims(64, 100, 16, 4, 0, 0))
    rows, inv, w, out = 1 << 20, 2 << 20, 3 << 20, 4 << 20  # never dereferenced
    assert L.moe_combine(dims, in_type, rows, 104, inv, w, out, in_stride, out_type, out,
                         out_stride, None, None) == BAD
    assert L.moe_dispatch_backward(dims, in_type, rows, 104, inv, out, in_stride, out_type, out,
                                   out_stride, None, None) == BAD


@pytest.mark.parametrize("T,d", [(1, (1 << 31) - 1), (1, (1 << 30) + 1), (((1 << 31) - 1) // 4, 1),
                                 ((1 << 29) - 1024, 1)])
def test_sizes_past_32_bit_numbers_are_refused(L, T, d):
    dims = ctypes.byref(M.make_dims(T, d, 16, 4, 0, 0))
    s = d + 16 - d % 16
    a = [i << 40 for i in range(1, 9)]  # never dereferenced
    assert L.moe_dispatch(dims, 0, a[0], s, a[1], a[2], s, None, None) == SHAPE
    assert L.moe_combine(dims, 0, a[0], s, a[1], a[2], None, 0, 0, a[3], s, None, None) == SHAPE
    assert L.moe_dispatch_backward(dims, 0, a[0], s, a[1], None, 0, 0, a[2], s, None, None) == SHAPE
    assert L.moe_combine_backward(dims, 0, a[0], s, a[1], s, a[2], a[3], a[4], s, a[5], None,
                                  None) == SHAPE
    assert L.moe_dispatch_int8(dims, 0, a[0], s, a[1], a[2], s, a[3], None, None) == SHAPE
    assert M.sort_workspace_size(M.make_dims(T, d, 16, 4, 0, 0)) == 0
    if T == 1:
        assert L.moe_quantize_int8(1, d, 0, a[0], s, None, a[1], s, a[2], None) == SHAPE


@pytest.mark.parametrize("flag", [M.MOE_FLAG_GEMM_SINGLE_CTA, M.MOE_FLAG_GEMM_PAIR,
                                  M.MOE_FLAG_FP8_EXPERTS, M.MOE_FLAG_COMBINE_REDUCE,
                                  M.MOE_FLAG_FUSED_EXPERTS])
def test_int8_layer_refuses_flags_it_has_no_use_for(flag):
    for flags in (flag, flag | M.MOE_FLAG_ROUTER_TENSOR):
        with pytest.raises(ValueError, match="flags"):  # before the (missing) weights are read
            M.MoeLayer({}, 256, 16, 4, 128, 128, flags=flags, int8=True)
    with pytest.raises(KeyError):
        M.MoeLayer({}, 256, 16, 4, 128, 128, flags=M.MOE_FLAG_ROUTER_TENSOR, int8=True)


# ---------------------------------------------------------------- workspaces

def _chunks(n):
    """Chunks of the index builder: one up to 4096 entries, above that the smallest of 1024,
    2048 and 4096 entries that gives at most 48 chunks (4096 if none does)."""
    if n <= 4096:
        return 1
    c = next((c for c in (1024, 2048) if 48 * c >= n), 4096)
    return -(-n // c)


def _sort_bytes(T, E, k):
    """Bytes that moe_sort uses for one batch: header, chunk histograms, tiles."""
    r = lambda b: (b + 255) // 256 * 256  # noqa: E731
    n = T * k
    return 256 + r(4 * E * _chunks(n)) + r(16 * (-(-n // 128) + E))


@pytest.mark.parametrize("E,k", [(1, 1), (16, 4), (256, 8), (512, 3), (512, 16)])
def test_sort_workspace_serves_every_smaller_batch(E, k):
    around = {0, 1, 2}
    for n in (4096, 49152, 98304, 196608):
        around |= {max(0, n // k + i) for i in (-1, 0, 1, 2)}
    Ts = sorted(around | set(range(1, 250000 // k, 997)))
    size = most = 0
    for T in Ts:
        n = M.sort_workspace_size(M.make_dims(T, 64, E, k, 0, 0))
        most = max(most, _sort_bytes(T, E, k))
        assert n >= size and n >= most, (T, n, size, most)
        size = n
    # one batch needs no more than the layer's own workspace for it
    assert _sort_bytes(5000, 256, 8) <= M.workspace_size(M.make_dims(5000, 64, 256, 8, 64, 0))


@pytest.mark.parametrize("E,k,d,F,Fs,flags", [
    (16, 4, 256, 128, 128, 0), (256, 8, 2048, 512, 512, M.MOE_FLAG_DOWN_F16),
    (256, 1, 64, 64, 0, M.MOE_FLAG_DOWN_F16), (512, 1, 64, 64, 0, M.MOE_FLAG_DOWN_F16),
    (256, 2, 128, 128, 0, M.MOE_FLAG_FUSED_EXPERTS | M.MOE_FLAG_DOWN_F16),
    (256, 2, 256, 64, 0, M.MOE_FLAG_ROUTER_TENSOR | M.MOE_FLAG_DOWN_F16),
    (256, 2, 256, 64, 0, M.MOE_FLAG_ROUTER_CUDA_CORE | M.MOE_FLAG_DOWN_F16)])
def test_layer_workspace_serves_every_smaller_batch(E, k, d, F, Fs, flags):
    dims = lambda T: M.make_dims(T, d, E, k, F, Fs, flags=flags)  # noqa: E731
    Ts = {1, 2, 3} | set(range(1, 250000 // k, 331))
    for t in (1024, 128 * 18, 128 * 37, 128 * 74, 4096 // k, 49152 // k, 98304 // k):
        Ts |= {max(1, t + i) for i in (-1, 0, 1, 2)}
    size = most = route = 0
    for T in sorted(Ts):
        most = max(most, M.workspace_size(dims(T)))
        # the router alone: header, index and logits, whatever follows them
        planes = (M.lib().moe_logits_offset(dims(T)) + 255) // 256 * 256 + 4 * T * E
        n = M.route_workspace_size(dims(T))
        assert max(planes, route) <= n <= M.workspace_size_upto(dims(T)), T
        route = n
        n = M.workspace_size_upto(dims(T))
        assert n == most and n >= size, T
        size = n
    assert M.workspace_size_upto(M.make_dims(64, 100, E, k, F, Fs)) == 0
    assert M.route_workspace_size(M.make_dims(64, 100, E, k, F, Fs)) == 0


def test_router_needs_no_room_for_the_experts(L):
    dims = M.make_dims(64, 2048, 256, 8, 512, 512)
    # header, histogram and tile lists, logits: no fp16 copy of the weights (537 MB)
    assert M.route_workspace_size(dims) < 200_000 < 500_000_000 < M.workspace_size(dims)
    n = M.route_workspace_size(M.make_dims(32768, 2048, 256, 8, 512, 512))
    assert n < 40_000_000
    L.moe_route.argtypes = [ctypes.c_void_p] * 7 + [ctypes.c_size_t, ctypes.c_void_p]
    assert L.moe_route(ctypes.byref(dims), 1 << 20, 2 << 20, None, 3 << 20, 4 << 20, 5 << 20,
                       M.route_workspace_size(dims) - 1, None) == M.MOE_ERR_WORKSPACE_TOO_SMALL


# ---------------------------------------------------------------- building

@pytest.mark.parametrize("missing", ["torch", "Python.h", "g++"])
def test_libraries_build_where_the_binding_cannot(missing, monkeypatch, capsys):
    run = []
    monkeypatch.setattr(B.subprocess, "run", lambda cmd, check: run.append(cmd))
    monkeypatch.setattr(B.os, "replace", lambda a, b: None)
    if missing == "torch":
        find = B.importlib.util.find_spec
        monkeypatch.setattr(B.importlib.util, "find_spec",
                            lambda n: None if n == "torch" else find(n))
    elif missing == "Python.h":
        monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": "/nowhere"})
    else:
        monkeypatch.setattr(B.shutil, "which", lambda n: None)
    moe, gen = B.build(force=True)
    assert moe.endswith("libmoe_b200.so") and gen.endswith("libmoe_gen.so")
    assert len(run) == 2 and all("nvcc" in cmd[0] for cmd in run)
    assert f"no {missing}" in capsys.readouterr().err


def test_binding_is_built_where_it_can_be(monkeypatch):
    run = []
    monkeypatch.setattr(B.subprocess, "run", lambda cmd, check: run.append(cmd))
    monkeypatch.setattr(B.os, "replace", lambda a, b: None)
    B.build(force=True)
    assert [os.path.basename(cmd[0]) for cmd in run] == ["nvcc", "nvcc", "g++"]
