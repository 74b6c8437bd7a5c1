"""The entry points' `stream` argument: a call on a stream that is not the
current one, its results, workspace and inputs dropped at once while the
stream is still busy, and memory of those sizes taken and filled on the
current stream."""
import pytest
import torch

import discrete_selective_ssm_b200 as naju

pytestmark = pytest.mark.gpu
BUSY = 20_000_000  # clock ticks (about 10 ms) that hold the given stream back


def rn(*shape, mean=0.0, dt=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) + mean).to(dt).cuda()


def vscan(stream):
    t = [rn(2, 3000, 256, mean=m, seed=k) for k, m in enumerate((0.0, 5.0, -2.0, 0.0, 0.0))]
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            torch.cuda._sleep(BUSY)
    h, a, b, z, dy = t
    y, xf, ws = naju.vscan_fwd(h, a, b, z=z, stream=stream)
    g = naju.vscan_bwd(dy, h, a, b, ws, z=z, stream=stream)
    return [ws], [y, xf, *g.values()]


def vscan_forward_alone(stream):
    ws, (y, xf, *_) = vscan(stream)
    t = [rn(2, 3000, 256, mean=m, seed=k) for k, m in enumerate((0.0, 5.0))]
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    y2, xf2, _ = naju.vscan_fwd(*t, stream=stream)  # its workspace is gone at once
    return ws, [y, xf, y2, xf2]


def matrix_scan(stream):
    Bt, L, d, N = 2, 500, 128, 64
    h, a, b, z, dy = (rn(Bt, L, d, mean=m, seed=k) for k, m in enumerate((0.0, 5.0, -2.0, 0.0, 0.0)))
    B, C = rn(Bt, L, N, seed=7), rn(Bt, L, N, seed=8)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            torch.cuda._sleep(BUSY)
    y, xf, ws = naju.scan_fwd(h, a, b, B, C, z=z, stream=stream)
    g = naju.scan_bwd(dy, h, a, b, B, C, ws, z=z, stream=stream)
    return [ws], [y, xf, *(v for v in g.values() if v is not None)]


def projection(stream):
    W, x, res = rn(700, 512), rn(40, 512, dt=torch.bfloat16), rn(40, 700, dt=torch.bfloat16)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            torch.cuda._sleep(BUSY)
    wq, scales = naju.w4_quantize(W, 64, stream=stream)
    return [wq, scales], [naju.w4_linear(x, wq, scales, 64, residual=res, stream=stream)]


def cache(stream):
    state = rn(4, 300, 64)
    slots = torch.tensor([3, 0, 5, 1], dtype=torch.int32, device="cuda")
    pq, ps = naju.state_pool(6, 300, 64, "cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            torch.cuda._sleep(BUSY)
    naju.state_store(state, slots, pq, ps, stream=stream)
    return [], [naju.state_load(pq, ps, slots, stream=stream)]


def steps(stream):
    h, a, b, z = (rn(8, 512, mean=m, seed=k) for k, m in enumerate((0.0, 5.0, -2.0, 0.0)))
    state, conv = rn(8, 512, seed=5), rn(8, 512, 3, seed=6)
    w = rn(512, 4, seed=9)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            torch.cuda._sleep(BUSY)
    u = naju.conv_silu_step(conv, h, w, stream=stream)
    y = naju.vscan_step(state, u, a, b, z, stream=stream)
    return [u], [y, state, conv]


@pytest.mark.parametrize("use", [vscan, vscan_forward_alone, matrix_scan, projection, cache, steps])
def test_everything_is_dropped_at_once(use):
    """Results on a given stream equal those of the current one, although the
    inputs and the intermediate tensors are gone when the call's kernels run and
    their sizes are allocated and filled anew on the current stream."""
    _, want = use(None)
    want = [t.clone() for t in want]
    sizes = [2 * 3000 * 256 * 4, 2 * 500 * 128 * 4, 2 * 500 * 64 * 4, 4 * 300 * 64 * 4, 700 * 512 * 4,
             40 * 512 * 2, 40 * 700 * 2, 8 * 512 * 4, 8 * 512 * 3 * 4, 512 * 4 * 4]
    side = torch.cuda.Stream()
    gone, got = use(side)
    sizes += [t.numel() * t.element_size() for t in gone]
    old = {t.data_ptr() for t in gone}
    del gone
    refill = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
    assert not old & {t.data_ptr() for t in refill}  # still the given stream's
    torch.cuda.current_stream().wait_stream(side)
    for w, g in zip(want, got):
        assert torch.equal(w, g)


def test_results_read_late_by_the_caller_stay():
    """A result dropped while the current stream still reads it: the given
    stream's next call of that size does not write over it."""
    h, a = rn(2, 3000, 256), rn(2, 3000, 256, mean=5.0)
    nothing = torch.zeros_like(h)
    want = naju.vscan_fwd(h, a)[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = naju.vscan_fwd(h, a, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    kept = y + 0.0
    del y
    other = [naju.vscan_fwd(nothing, a, stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and len(other) == 3


def test_the_current_stream_given():
    h, a = rn(1, 100, 64), rn(1, 100, 64, mean=5.0)
    y = naju.vscan_fwd(h, a)[0]
    assert torch.equal(naju.vscan_fwd(h, a, stream=torch.cuda.current_stream())[0], y)
    with pytest.raises(AttributeError):
        naju.vscan_fwd(h, a, stream=3)


def test_the_default_stream_given_on_another():
    """The default stream's handle is zero."""
    h, a = rn(1, 100, 64), rn(1, 100, 64, mean=5.0)
    state, row = rn(4, 64), rn(4, 64, seed=1)
    w = rn(64, 128)
    y, (wq, sc) = naju.vscan_fwd(h, a)[0], naju.w4_quantize(w)
    step = naju.vscan_step(state.clone(), row, row)
    torch.cuda.synchronize()
    default = torch.cuda.default_stream()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = naju.vscan_fwd(h, a, stream=default)[0]
        got_wq, got_sc = naju.w4_quantize(w, stream=default)
        got_step = naju.vscan_step(state, row, row, stream=torch.cuda.ExternalStream(0))
        torch.cuda.current_stream().wait_stream(default)
        assert torch.equal(got, y) and torch.equal(got_wq, wq) and torch.equal(got_sc, sc)
        assert torch.equal(got_step, step)
    torch.cuda.synchronize()
