"""The 4-bit projections against the definition in 64 bits.

Bound, element by element: every product (q - 8) x is exact, a group's sum of G
of them and the sum over groups round by at most half a step (u = 2^-24) per
addition, and the tensor cores' own additions by at most a whole one; so y is
off by at most 2 u (n_in + 4) of the sum of |terms|.  A bf16 y adds half a
bf16 step, 2^-8 of the value.
"""
import math

import numpy as np
import pytest
import torch

import discrete_selective_ssm_b200 as naju

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def unpack(wq, K):
    """q [n_out, K] from the packed words, word by word."""
    w = wq.cpu().numpy().view("<u4")
    O = w.shape[0]
    q = np.zeros((O, w.shape[1] // 16 * 128), dtype=np.int64)
    for b in range(w.shape[1] // 16):
        for c in range(4):
            for j in range(4):
                word = w[:, 16 * b + 4 * c + j]
                for e in range(8):
                    nibble = e // 2 + 4 * (e % 2)
                    q[:, 128 * b + 32 * j + 8 * c + e] = (word >> np.uint32(4 * nibble)) & 15
    assert (q[:, K:] == 8).all()
    return q[:, :K]


def weights(wq, scales, K, G):
    s = np.repeat(scales.double().cpu().numpy(), G, 1)[:, :K]
    return (unpack(wq, K) - 8) * s


def make(m, K, O, G, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(O, K, generator=g) / math.sqrt(K)
    x = torch.randn(m, K, generator=g).to(DT[dtype]).cuda()
    wq, scales = naju.w4_quantize(W.cuda(), G)
    return x, W, wq, scales


def check(x, wq, scales, G, bias=None, residual=None, **kw):
    K = x.shape[-1]
    y = naju.w4_linear(x, wq, scales, G, bias=bias, residual=residual, **kw)
    W = weights(wq, scales, K, G)
    xd = x.double().cpu().numpy()
    want, size = xd @ W.T, np.abs(xd) @ np.abs(W).T
    for t in (bias, residual):
        if t is not None:
            want, size = want + t.double().cpu().numpy(), size + t.double().abs().cpu().numpy()
    allow = 2 * U * (K + 4) * size + 1e-30
    if x.dtype == torch.bfloat16:
        allow = allow + 2.0 ** -8 * np.abs(want)
    err = np.abs(y.double().cpu().numpy() - want)
    assert y.dtype == x.dtype and np.isfinite(err).all()
    k = np.unravel_index(np.argmax(err - allow), err.shape)
    assert err[k] <= allow[k], f"{k}: off by {err[k]:.3e}, allowed {allow[k]:.3e}"
    return y


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 3, 8, 9, 16, 17, 32, 33, 64, 65, 130, 256])
def test_rows(m, G, dtype):
    x, _, wq, scales = make(m, 520, 200, G, dtype, m + G)
    check(x, wq, scales, G)


@pytest.mark.parametrize("K", [1, 7, 31, 32, 33, 127, 128, 129, 1000, 2048, 2500])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_inputs(K, dtype):
    for m, G in ((1, 128), (11, 32), (40, 64)):
        x, _, wq, scales = make(m, K, 37, G, dtype, K + m)
        check(x, wq, scales, G)


@pytest.mark.parametrize("O", [1, 15, 16, 17, 127, 129, 1111])
def test_outputs(O):
    for m in (1, 20, 70):
        x, _, wq, scales = make(m, 384, O, 64, "bf16", O + m)
        check(x, wq, scales, 64)


@pytest.mark.parametrize("m,K,O", [(1, 8192, 64), (4, 8192, 300), (64, 8192, 130), (200, 4096, 64)])
def test_long_rows(m, K, O):
    """Few rows of weights: the inputs are shared out over a cluster."""
    for dtype in ("bf16", "f32"):
        x, _, wq, scales = make(m, K, O, 128, dtype, K + O)
        y = check(x, wq, scales, 128)
        assert torch.equal(y, naju.w4_linear(x, wq, scales, 128))  # a fixed order of sums


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bias_and_residual(dtype):
    for m in (1, 12, 100):
        x, _, wq, scales = make(m, 300, 150, 32, dtype, m)
        bias = torch.randn(150, device="cuda")
        res = torch.randn(m, 150, device="cuda").to(DT[dtype])
        check(x, wq, scales, 32, bias=bias)
        check(x, wq, scales, 32, residual=res)
        y = check(x, wq, scales, 32, bias=bias, residual=res)
        assert torch.equal(naju.w4_linear(x, wq, scales, 32, bias=bias, residual=res, y=res), y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_quantize(G, dtype):
    """scale = bf16(max / 7) and q = the nearest, per group, ragged last group."""
    g = torch.Generator().manual_seed(G)
    W = (torch.randn(30, 333, generator=g) * torch.randn(30, 1, generator=g).exp()).to(DT[dtype])
    W[3] = 0
    W[4, :40] = 0
    wq, scales = naju.w4_quantize(W.cuda(), G)
    q = unpack(wq, 333)
    Wd = W.double().numpy()
    for i in range(scales.shape[1]):
        blk = Wd[:, G * i:G * (i + 1)]
        m = torch.from_numpy(np.abs(blk).max(1)).float()
        s = (m / 7).bfloat16()
        assert torch.equal(s, scales[:, i].cpu())
        sd = s.double().numpy()[:, None]
        live = sd[:, 0] > 0
        # fp32 quotients: within half a step of a border either neighbour is right
        off = np.abs(np.clip(blk[live] / sd[live], -8, 7) - (q[live, G * i:G * (i + 1)] - 8))
        assert (off <= 0.5 + 8 * U).all()
        assert (q[~live, G * i:G * (i + 1)] == 8).all()


def test_quantize_non_finite():
    W = torch.randn(4, 256)
    W[1, 5] = math.inf
    W[2, 200] = math.nan
    wq, scales = naju.w4_quantize(W.cuda(), 128)
    bad = torch.isnan(scales).cpu()
    assert bad.tolist() == [[False, False], [True, False], [False, True], [False, False]]
    y = naju.w4_linear(torch.ones(1, 256, device="cuda"), wq, scales, 128)
    assert torch.isnan(y)[0].tolist() == [False, True, True, False]


def test_infinite_and_extreme_inputs():
    """An infinity meets q = 8 (weight 0) as NaN and others as infinities; the
    largest fp32 values split without overflow."""
    x, _, wq, scales = make(2, 128, 16, 128, "f32", 5)
    W = weights(wq, scales, 128, 128)
    x.zero_()
    x[0, 3] = math.inf
    x[1, 4] = 3.0e38
    y = naju.w4_linear(x, wq, scales, 128).cpu().numpy()
    for o in range(16):
        w = W[o, 3]
        assert np.isnan(y[0, o]) if w == 0 else y[0, o] == math.copysign(math.inf, w)
        assert abs(y[1, o] - 3.0e38 * W[o, 4]) <= 4 * U * 3.0e38 * abs(W[o, 4])


def test_rows_of_any_leading_shape_and_streams():
    x, _, wq, scales = make(6, 256, 64, 128, "bf16", 9)
    y = naju.w4_linear(x, wq, scales)
    assert torch.equal(naju.w4_linear(x.view(2, 3, 256), wq, scales), y.view(2, 3, 64))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z = naju.w4_linear(x, wq, scales)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(z, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z = naju.w4_linear(x, wq, scales)
    x.copy_(torch.randn(6, 256).bfloat16())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, naju.w4_linear(x, wq, scales))


def test_neighbours_stay():
    x, _, wq, scales = make(9, 200, 33, 64, "bf16", 11)
    buf = torch.full((9 * 33 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    naju.w4_linear(x, wq, scales, 64, y=buf[:9 * 33].view(9, 33))
    torch.cuda.synchronize()
    assert bool((buf[9 * 33:] == 7.0).all())


def test_refusals():
    x, _, wq, scales = make(2, 128, 16, 128, "bf16")
    with pytest.raises(naju.NajuError):
        naju.w4_linear(x, wq, scales, 100)
    with pytest.raises(naju.NajuError):
        naju.w4_linear(x[:0], wq, scales)
    with pytest.raises(ValueError):
        naju.w4_linear(x, wq, scales, 64)
    with pytest.raises(ValueError):
        naju.w4_linear(x[:, :100].contiguous(), wq[:, :32].contiguous(), scales)
    with pytest.raises(TypeError):
        naju.w4_linear(x.half(), wq, scales)
    with pytest.raises(ValueError):
        naju.w4_linear(x, wq, scales, bias=torch.zeros(15, device="cuda"))


@pytest.fixture(params=[1, 2], ids=["warp", "tcgen05"])
def impl(request):
    naju.testing_set_w4_impl(request.param)
    yield request.param
    naju.testing_set_w4_impl(0)


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 300])
def test_each_form_rows(impl, m, G):
    x, _, wq, scales = make(m, 520, 200, G, "bf16", m + G + 1)
    check(x, wq, scales, G)


@pytest.mark.parametrize("K", [136, 256, 264, 384, 1000, 1920, 4096])
@pytest.mark.parametrize("O", [1, 127, 128, 129, 400])
def test_each_form_sizes(impl, K, O):
    for m, G in ((5, 128), (40, 32)):
        x, _, wq, scales = make(m, K, O, G, "bf16", K + O)
        bias = torch.randn(O, device="cuda")
        res = torch.randn(m, O, device="cuda").bfloat16()
        y = check(x, wq, scales, G, bias=bias, residual=res)
        assert torch.equal(y, naju.w4_linear(x, wq, scales, G, bias=bias, residual=res))


def test_each_form_extremes(impl):
    """The largest bf16 values stay finite until the result, a NaN scale and an
    infinite input reach their own results only."""
    x, _, wq, scales = make(20, 512, 160, 128, "bf16", 3)
    W = weights(wq, scales, 512, 128)
    x.zero_()
    x[1, 4] = 3.0e38
    scales[7, 2] = math.nan
    x[3, 100] = math.inf
    y = naju.w4_linear(x, wq, scales, 128).double().cpu().numpy()
    for o in range(160):
        if o == 7:
            assert np.isnan(y[:, o]).all()
            continue
        want = float(x[1, 4]) * W[o, 4]
        assert abs(y[1, o] - want) <= 2.0 ** -8 * abs(want)
        w = W[o, 100]
        assert np.isnan(y[3, o]) if w == 0 else y[3, o] == math.copysign(math.inf, w)
        assert (y[[0, 2] + list(range(4, 20)), o] == 0).all()


def test_large_batch_takes_the_tensor_cores():
    x, _, wq, scales = make(256, 1024, 1100, 64, "bf16", 21)
    check(x, wq, scales, 64)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 2])
@pytest.mark.parametrize("K,O", [(8193, 9), (9216, 700), (20000, 33), (33000, 5)])
def test_inputs_longer_than_the_stage(m, K, O, dtype):
    """One and two rows of x that come into shared memory in several parts."""
    x, _, wq, scales = make(m, K, O, 128, dtype, K + m)
    check(x, wq, scales, 128)


def test_result_over_its_input_is_refused():
    x, _, wq, scales = make(1, 128, 128, 128, "bf16")
    with pytest.raises(naju.NajuError):
        naju.w4_linear(x, wq, scales, y=x)


def test_two_calls_at_once():
    """Two streams, the same weights: neither call keeps anything of its own."""
    a, _, wq, scales = make(200, 1024, 2048, 64, "bf16", 31)
    b = torch.randn(200, 1024, device="cuda").bfloat16()
    want = [naju.w4_linear(t, wq, scales, 64) for t in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        got = []
        for t, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(naju.w4_linear(t, wq, scales, 64))
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("m", [1, 9, 40])
def test_offsets_past_32_bits(m):
    """Weights of more than 2^31 bytes: the last rows equal a product with them
    alone."""
    K, O, tail = 16384, 263000, 129
    g = torch.Generator(device="cuda").manual_seed(1)
    wq = torch.randint(0, 256, (O, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    assert wq.numel() > 2 ** 31
    scales = torch.rand(O, K // 128, generator=g, device="cuda").add_(0.5).bfloat16()
    x = torch.randn(m, K, generator=g, device="cuda").bfloat16()
    y = naju.w4_linear(x, wq, scales)
    for impl in (0, 1, 2):
        naju.testing_set_w4_impl(impl)
        try:
            last = naju.w4_linear(x, wq[-tail:].contiguous(), scales[-tail:].contiguous())
        finally:
            naju.testing_set_w4_impl(0)
        # the order of the sums may differ: two roundings to bf16
        err = (y[:, -tail:].double() - last.double()).abs()
        assert bool((err <= 2.0 ** -7 * last.double().abs() + 1e-2).all())
