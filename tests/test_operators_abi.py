"""Host-side refusals of the vector-state scan, the 4-bit projection and the
8-bit state cache (no GPU: nothing is launched)."""
import ctypes

import pytest
import torch

import discrete_selective_ssm_b200 as naju

FAKE = ctypes.c_void_p(4096)
MIS = ctypes.c_void_p(4098)


@pytest.fixture(scope="module")
def L():
    return naju.lib()


def dims(Bt=2, seq=100, d=64, N=1, dtype=naju.F32, out=None):
    return naju.make_dims(Bt, seq, d, N, dtype, out, 0)


def test_vscan_workspace(L):
    dm = dims(2, 300, 200)
    n = L.naju_vscan_workspace_bytes(ctypes.byref(dm))
    assert n % 256 == 0 and n >= 2 * 5 * 200 * 4
    # one item per unit needs no flags and no aggregates
    assert L.naju_vscan_workspace_bytes(ctypes.byref(dims(2, 32, 200))) < 8192
    for bad in (dims(N=16), dims(Bt=0), dims(seq=0), dims(d=0), dims(dtype=7),
                dims(out=naju.BF16), dims(1 << 20, 1 << 26, 1)):
        assert L.naju_vscan_workspace_bytes(ctypes.byref(bad)) == 0
    assert L.naju_vscan_workspace_bytes(None) == 0


def test_vscan_refusals(L):
    dm = dims()
    n = 1 << 30
    f = lambda d, *a: L.naju_vscan_fwd(ctypes.byref(d) if d else None, *a)  # noqa: E731
    ok = [FAKE, FAKE, None, None, None, FAKE, None]
    assert f(None, *ok, FAKE, n, None) == 1
    assert f(dims(N=16), *ok, FAKE, n, None) == 2
    assert f(dm, None, *ok[1:], FAKE, n, None) == 1
    assert f(dm, MIS, *ok[1:], FAKE, n, None) == 1
    assert f(dm, FAKE, FAKE, MIS, None, None, FAKE, None, FAKE, n, None) == 1
    assert f(dm, FAKE, FAKE, None, None, None, None, None, FAKE, n, None) == 1
    assert f(dm, *ok, None, n, None) == 1
    assert f(dm, *ok, FAKE, 256, None) == 1
    assert f(dm, *ok, MIS, n, None) == 1
    b = lambda *a: L.naju_vscan_bwd(ctypes.byref(dm), *a)  # noqa: E731
    #           h     a     b     z     dy    dxf   dh    da    db    dz    dx0
    assert b(FAKE, FAKE, FAKE, None, FAKE, None, FAKE, FAKE, None, None, None, FAKE, n, None) == 1
    assert b(FAKE, FAKE, None, FAKE, FAKE, None, FAKE, FAKE, None, None, None, FAKE, n, None) == 1
    assert b(FAKE, FAKE, None, None, None, None, FAKE, FAKE, None, None, None, FAKE, n, None) == 1
    assert b(FAKE, FAKE, None, None, FAKE, None, FAKE, FAKE, None, None, None, FAKE, 16, None) == 1


def test_vscan_step_refusals(L):
    s = L.naju_vscan_step
    assert s(0, 8, 0, *[FAKE] * 6, None) == 1
    assert s(1, 8, 5, *[FAKE] * 6, None) == 2
    assert s(1, 8, 0, None, *[FAKE] * 5, None) == 1
    assert s(1, 8, 0, FAKE, FAKE, MIS, None, FAKE, FAKE, None) == 1


def test_vscan_binding_refuses_cpu_tensors():
    h = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        naju.vscan_fwd(h, h)
    with pytest.raises(ValueError):
        naju.vscan_fwd(h[0], h[0])
    with pytest.raises(ValueError):
        naju.vscan_step(torch.zeros(4, 8), h[0], h[0])
