"""The C ABI of the operators on unquantized and 4-bit integer experts on the
CPU: every bad argument is refused on the host, also under host
AddressSanitizer, and the binding refuses what the C ABI cannot see.  Device
pointers are fake, 16-byte aligned integers; no call here reaches a device."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from nvfp4_weight_only_moe_amd import binding as b

A = 0x10000000
STEP = 0x10000000


def at(i):
    return A + i * STEP


@pytest.fixture(scope="module")
def L():
    return b.lib()


OK, ARG, SHAPE, ALIGN, UNSUP, WS = 0, -1, -2, -3, -4, -7


def linear(L, x=at(0), X=8, K=64, w=at(1), E=4, N=32, off=at(2), slots=at(3), k=2, M=16, y=at(4), ws=at(8),
           ws_bytes=1 << 27):
    return L.moe_grouped_linear(x, X, K, w, E, N, off, slots, k, M, y, ws, ws_bytes, None)


def swiglu(L, x=at(0), X=8, K=64, g=at(1), u=at(2), E=4, N=32, off=at(3), slots=at(4), k=2, M=16, h=at(5), a=at(6),
           bb=at(7), ws=at(8), ws_bytes=1 << 27):
    return L.moe_grouped_swiglu(x, X, K, g, u, E, N, off, slots, k, M, h, a, bb, ws, ws_bytes, None)


def dgrad(L, dy=at(0), w=at(1), dy2=at(2), w2=at(3), M=16, N=32, E=4, K=64, off=at(4), dx=at(5), ws=at(8),
          ws_bytes=1 << 27):
    return L.moe_grouped_linear_dgrad(dy, w, dy2, w2, M, N, E, K, off, dx, ws, ws_bytes, None)


def sdgrad(L, dy=at(0), w=at(1), M=16, N=32, E=4, K=64, off=at(2), a=at(3), bb=at(4), da=at(5), db=at(6), ws=at(8),
           ws_bytes=1 << 27):
    return L.moe_grouped_swiglu_dgrad(dy, w, M, N, E, K, off, a, bb, da, db, ws, ws_bytes, None)


def wgrad(L, dy=at(0), M=16, N=32, x=at(1), X=8, K=64, E=4, off=at(2), slots=at(3), k=2, acc=0, dw=at(4), ws=at(5),
          ws_bytes=1 << 27):
    return L.moe_grouped_linear_wgrad(dy, M, N, x, X, K, E, off, slots, k, acc, dw, ws, ws_bytes, None)


@pytest.mark.parametrize("f", [linear, swiglu, dgrad, sdgrad])
def test_grouped_shapes(L, f):
    assert f(L, M=0) == OK                                # no-op
    assert f(L, M=-1) == SHAPE
    assert f(L, N=0) == SHAPE and f(L, K=0) == SHAPE and f(L, E=0) == SHAPE
    assert f(L, N=36) == SHAPE and f(L, K=60) == SHAPE    # multiples of 8
    assert f(L, N=(1 << 20) + 8) == SHAPE and f(L, K=(1 << 20) + 8) == SHAPE
    assert f(L, E=1025) == UNSUP
    assert f(L, off=0) == ARG and f(L, off=at(9) + 4) == ALIGN


def test_grouped_pointers(L):
    for f, names, outs in ((linear, ("x", "w", "y"), ("y",)), (swiglu, ("x", "g", "u", "h"), ("h", "a", "bb")),
                           (dgrad, ("dy", "w", "dx"), ("dx",)), (sdgrad, ("dy", "w", "a", "bb", "da", "db"), ("da", "db"))):
        for n in names:
            assert f(L, **{n: 0}) == ARG, (f.__name__, n)
            assert f(L, **{n: at(9) + 8}) == ALIGN, (f.__name__, n)
        for o in outs:                                    # outputs overlap an input or each other
            for i in range(5):
                if f(L, **{o: at(i) + 16}) == ARG:
                    break
            else:
                raise AssertionError((f.__name__, o))
    assert swiglu(L, a=0) == ARG and swiglu(L, bb=0) == ARG          # both or neither
    assert swiglu(L, a=at(7)) == ARG                                 # a is b
    assert sdgrad(L, da=at(6)) == ARG
    assert dgrad(L, dy2=0) == ARG and dgrad(L, w2=0) == ARG
    assert dgrad(L, dy2=at(9) + 8) == ALIGN
    assert dgrad(L, dx=at(2)) == ARG                                 # dx is dy2


@pytest.mark.parametrize("f,products", [(linear, 1), (swiglu, 3), (dgrad, 2), (sdgrad, 1)])
def test_grouped_workspace(L, f, products):
    """Few rows and a long sum take a workspace: required, large enough, aligned, apart from every buffer."""
    size = dict(M=16, N=64, K=8192, E=1) if f in (linear, swiglu) else dict(M=16, N=8192, K=64, E=1)
    need = L.moe_grouped_workspace_size(16, 1, 8192, 64, products)
    assert need >= 2 * 16 * 64 * 4
    assert f(L, **size, ws=0) == WS and f(L, **size, ws_bytes=need - 1) == WS
    assert f(L, **size, ws=at(8) + 8) == ALIGN
    for i in range(5):
        assert f(L, **size, ws=at(i)) == ARG, i
    assert L.moe_grouped_workspace_size(0, 1, 8192, 64, products) == 0
    assert L.moe_grouped_workspace_size(16, 1, 8192, 64, 4) == 0
    assert L.moe_grouped_workspace_size(1 << 20, 64, 4096, 4096, products) == 0    # many tiles: none


@pytest.mark.parametrize("f", [linear, swiglu, wgrad])
def test_gathered_rows(L, f):
    assert f(L, k=0) == SHAPE and f(L, k=33) == UNSUP
    assert f(L, X=-1) == SHAPE and f(L, X=0) == SHAPE
    assert f(L, slots=at(9) + 4) == ALIGN
    assert f(L, slots=0) == SHAPE                                    # X == M without slots
    assert f(L, X=1 << 25, K=128) == SHAPE                           # 32-bit offsets


def test_wgrad(L):
    for n in ("dy", "x", "off", "dw"):
        assert wgrad(L, **{n: 0}) == ARG, n
        assert wgrad(L, **{n: at(9) + 8}) == ALIGN, n
    assert wgrad(L, acc=2) == ARG
    assert wgrad(L, dw=at(1)) == ARG and wgrad(L, dw=at(3)) == ARG
    assert wgrad(L, N=36) == SHAPE and wgrad(L, M=-1) == SHAPE and wgrad(L, E=1025) == UNSUP
    big = dict(M=16384, N=256, K=5120, E=1, X=16384, slots=0)
    need = L.moe_grouped_linear_wgrad_workspace_size(16384, 256, 5120, 1)
    if need:
        assert wgrad(L, **big, ws=0) == WS and wgrad(L, **big, ws_bytes=need - 1) == WS
        assert wgrad(L, **big, ws=at(5) + 8) == ALIGN and wgrad(L, **big, ws=at(4) + 16) == ARG
    assert L.moe_grouped_linear_wgrad_workspace_size(-1, 256, 5120, 1) == 0
    assert L.moe_grouped_linear_wgrad_workspace_size(0, 256, 5120, 1) == 0


def tensor(E=1, N=32, K=256, group=64, codes=at(1), scales=at(2), zeros=at(3)):
    return b.Int4TensorC(E, N, K, group, codes, scales, zeros)


def int4(L, x=at(0), X=4, t=None, off=None, slots=None, k=1, M=4, out=at(5), **kw):
    t = tensor(**kw) if t is None else t
    return L.moe_int4_linear(x, X, ctypes.byref(t), off, slots, k, M, out, None)


def test_int4(L):
    assert int4(L, M=0, X=0) == OK
    assert L.moe_int4_linear(at(0), 4, None, None, None, 1, 4, at(5), None) == ARG
    assert int4(L, K=192) == SHAPE and int4(L, group=16) == SHAPE and int4(L, N=0) == SHAPE and int4(L, E=0) == SHAPE
    assert int4(L, E=1025, off=at(4)) == UNSUP
    assert int4(L, M=-1) == SHAPE and int4(L, M=5) == SHAPE          # X == M
    assert int4(L, M=1 << 29, X=1 << 29, out=1 << 60) == SHAPE         # more than 2^22 tiles
    assert int4(L, E=2) == ARG                                       # experts need offsets
    assert int4(L, slots=at(4)) == ARG                               # slots need offsets
    assert int4(L, off=at(4) + 4) == ALIGN
    assert int4(L, off=at(4), slots=at(6), k=0) == SHAPE and int4(L, off=at(4), slots=at(6), k=33) == UNSUP
    for n in ("x", "out", "codes", "scales"):
        assert int4(L, **{n: 0}) == ARG, n
        assert int4(L, **{n: at(9) + 8}) == ALIGN, n
    assert int4(L, zeros=at(9) + 8) == ALIGN
    for i in (0, 1, 2, 3):
        assert int4(L, out=at(i) + 16) == ARG, i
    t = tensor()
    assert L.moe_int4_quantize_pack(None, ctypes.byref(t), None) == ARG
    assert L.moe_int4_quantize_pack(at(2), ctypes.byref(t), None) == ARG
    assert L.moe_int4_quantize_pack(at(0) + 4, ctypes.byref(t), None) == ALIGN
    assert L.moe_int4_quantize_pack(at(0), ctypes.byref(tensor(K=64)), None) == SHAPE
    assert L.moe_int4_quantize_pack(at(0), ctypes.byref(tensor(scales=at(1))), None) == ARG
    assert L.moe_int4_dequantize(ctypes.byref(t), None, None) == ARG
    assert L.moe_int4_dequantize(ctypes.byref(t), at(1), None) == ARG


def combine(L, y=at(0), M=16, H=64, pos=at(1), w=at(2), T=8, k=2, out=at(3)):
    return L.moe_combine(y, M, H, pos, w, T, k, out, None)


def combine_bwd(L, dout=at(0), T=8, H=64, y=at(1), M=16, pos=at(2), w=at(3), ids=at(4), k=2, E=8, dy=at(5), dw=at(6),
                dl=at(7)):
    return L.moe_combine_backward(dout, T, H, y, M, pos, w, ids, k, E, dy, dw, dl, None)


@pytest.mark.parametrize("f", [combine, combine_bwd])
def test_combine_shapes(L, f):
    assert f(L, T=0) == OK
    assert f(L, T=-1) == SHAPE and f(L, M=-1) == SHAPE and f(L, k=0) == SHAPE
    assert f(L, H=60) == SHAPE and f(L, H=0) == SHAPE and f(L, H=(1 << 20) + 8) == SHAPE
    assert f(L, T=(1 << 22) + 1) == SHAPE and f(L, k=33) == UNSUP


def test_combine_pointers(L):
    for n in ("y", "pos", "out"):
        assert combine(L, **{n: 0}) == ARG, n
    for n in ("y", "pos", "out", "w"):
        assert combine(L, **{n: at(9) + 4}) == ALIGN, n
    assert combine(L, out=at(0)) == ARG and combine(L, out=at(2)) == ARG
    for n in ("dout", "y", "pos", "dy"):
        assert combine_bwd(L, **{n: 0}) == ARG, n
    for n in ("dout", "y", "pos", "w", "ids", "dy", "dw", "dl"):
        assert combine_bwd(L, **{n: at(9) + 4}) == ALIGN, n
    assert combine_bwd(L, w=0) == ARG and combine_bwd(L, ids=0) == ARG          # dlogits need both
    assert combine_bwd(L, E=0) == SHAPE and combine_bwd(L, E=1025) == UNSUP
    assert combine_bwd(L, dy=at(0)) == ARG and combine_bwd(L, dw=at(5)) == ARG and combine_bwd(L, dl=at(6)) == ARG


def test_binding_refuses_host_tensors_and_wrong_types():
    x, w, off = torch.zeros(4, 64), torch.zeros(1, 32, 64), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: b.moe_grouped_linear(x, w, off), lambda: b.moe_grouped_swiglu(x, w, w, off),
                 lambda: b.moe_grouped_linear_dgrad(x, w, off), lambda: b.moe_grouped_swiglu_dgrad(x, w, x, x, off),
                 lambda: b.moe_grouped_linear_wgrad(x, x, off), lambda: b.moe_combine(x, off, 1),
                 lambda: b.moe_int4_quantize_pack(w), lambda: b.moe_combine_backward(x, x, off, x),
                 lambda: b.moe_int4_linear(x, None), lambda: b.moe_int4_dequantize(None),
                 lambda: b.moe_grouped_linear("x", w, off), lambda: b.moe_grouped_linear(),
                 lambda: b.moe_grouped_linear(w=w, x=x, offsets=off), lambda: b.moe_int4_linear(w=None, x=x)):
        with pytest.raises(ValueError):
            call()


def test_under_host_asan():
    if os.environ.get("MOE_TEST_UNDER_ASAN"):
        pytest.skip("already the instrumented run")
    import test_abi_asan as asan
    from nvfp4_weight_only_moe_amd import build_lib
    lib = build_lib.build_asan()
    env = dict(os.environ, LD_PRELOAD=build_lib.asan_runtime(), HIP_VISIBLE_DEVICES="", MOE_TEST_UNDER_ASAN="1",
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1")
    code = asan.RUNNER.format(root=asan.ROOT, tests=os.path.join(asan.ROOT, "tests"), lib=lib, testfile=__file__)
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=600)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0 and "AddressSanitizer" not in r.stderr and " passed" in r.stdout, tail
