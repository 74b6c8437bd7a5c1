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
    # (the status word and one item's checkpoints per unit)
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


def test_state_cache_refusals(L):
    ok = [FAKE] * 4
    for f in (L.naju_state_store, L.naju_state_load):
        assert f(0, 8, 16, 4, *ok, None) == 1
        assert f(65536, 8, 16, 4, *ok, None) == 1
        assert f(1, 0, 16, 4, *ok, None) == 1
        assert f(1, 8, 16, 0, *ok, None) == 1
        assert f(1, 8, 24, 4, *ok, None) == 2
        for i in range(4):
            a = list(ok)
            a[i] = None
            assert f(1, 8, 16, 4, *a, None) == 1
    assert L.naju_state_store(1, 8, 16, 4, MIS, FAKE, FAKE, FAKE, None) == 1
    assert L.naju_state_load(1, 8, 16, 4, MIS, FAKE, FAKE, FAKE, None) == 1


def test_state_cache_binding_refusals():
    q, s = naju.state_pool(3, 8, 16, "cpu")
    slots = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        naju.state_load(q, s, slots)
    with pytest.raises(ValueError):
        naju.state_load(q[0], s, slots)
    with pytest.raises(ValueError):
        naju.state_store(torch.zeros(1, 8, 16), slots[None], q, s)


def test_w4_refusals(L):
    q = lambda *a: L.naju_w4_quantize(*a, None)  # noqa: E731
    assert q(0, 64, 32, 0, FAKE, FAKE, FAKE) == 1
    assert q(8, 0, 32, 0, FAKE, FAKE, FAKE) == 1
    assert q(8, 64, 48, 0, FAKE, FAKE, FAKE) == 2
    assert q(8, 64, 32, 3, FAKE, FAKE, FAKE) == 2
    assert q(8, 64, 32, 0, None, FAKE, FAKE) == 1
    assert q(8, 64, 32, 0, FAKE, MIS, FAKE) == 1
    out = ctypes.c_void_p(8192)
    f = lambda *a: L.naju_w4_linear(*a[:-1], out if a[-1] is FAKE else a[-1], None)  # noqa: E731
    #        m  in  out  G  dt  x     wq    s     bias  res   y
    assert f(0, 64, 8, 32, 0, FAKE, FAKE, FAKE, None, None, FAKE) == 1
    assert f(1 << 21, 64, 8, 32, 0, FAKE, FAKE, FAKE, None, None, FAKE) == 1
    assert f(1, 64, 0, 32, 0, FAKE, FAKE, FAKE, None, None, FAKE) == 1
    assert f(1, 64, 8, 16, 0, FAKE, FAKE, FAKE, None, None, FAKE) == 2
    assert f(1, 64, 8, 32, 2, FAKE, FAKE, FAKE, None, None, FAKE) == 2
    assert f(1, 64, 8, 32, 0, MIS, FAKE, FAKE, None, None, FAKE) == 1
    assert f(1, 64, 8, 32, 0, FAKE, MIS, FAKE, None, None, FAKE) == 1
    assert f(1, 64, 8, 32, 0, FAKE, FAKE, None, None, None, FAKE) == 1
    assert f(1, 64, 8, 32, 0, FAKE, FAKE, FAKE, None, MIS, FAKE) == 1
    assert f(1, 64, 8, 32, 0, FAKE, FAKE, FAKE, None, None, None) == 1
    # the result over the input it is computed from
    assert L.naju_w4_linear(1, 64, 64, 32, 0, FAKE, FAKE, FAKE, None, None, FAKE, None) == 1


def test_w4_binding_refusals():
    with pytest.raises(ValueError):
        naju.w4_quantize(torch.zeros(8, 64))
    with pytest.raises(ValueError):
        naju.w4_quantize(torch.zeros(64))
    with pytest.raises(ValueError):
        naju.w4_linear(torch.zeros(1, 64), torch.zeros(8, 64, dtype=torch.uint8),
                       torch.zeros(8, 1, dtype=torch.bfloat16))


@pytest.mark.parametrize("dtype,e", [(naju.F32, 4), (naju.BF16, 2)])
def test_w4_results_over_inputs_are_refused(L, dtype, e):
    """y anywhere over an input, but for the residual's own place."""
    m, K, O, G = 3, 256, 64, 32
    p = lambda v: ctypes.c_void_p(v)  # noqa: E731
    names = ("x", "wq", "scales", "bias", "residual")
    size = dict(x=m * K * e, wq=O * K // 2, scales=2 * O * K // G, bias=4 * O, residual=m * O * e)
    at = {n: (1 << 20) * (i + 1) for i, n in enumerate(names)}
    out = m * O * e
    f = lambda y: L.naju_w4_linear(m, K, O, G, dtype, *(p(at[n]) for n in names), p(y), None)  # noqa: E731
    for n in names:
        for y in (at[n] + 16, at[n] - 16, at[n] + size[n] - 16, at[n] - out + 16):
            assert f(y) == 1, (n, y - at[n])
    for n in names:
        if n != "residual":
            assert f(at[n]) == 1, n
