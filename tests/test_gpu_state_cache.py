"""The 8-bit state cache against its definition in 64 bits.  A stored value is
exact in the format's own terms, so q and scale are compared for equality; what
reads back is one fp32 product (half a step, 2^-24) and within half a quantum
of what was stored."""
import numpy as np
import pytest
import torch

import discrete_selective_ssm_b200 as naju

pytestmark = pytest.mark.gpu


def reference(x):
    """q and scale of rows (last axis) in 64 bits; scale rounded to fp32."""
    x = x.double().cpu()
    scale = (x.abs().amax(-1) / 127).float()
    s = scale.double()
    q = torch.round(x / torch.where(s > 0, s, 1.0)[..., None])
    q[s == 0] = 0
    return q.clamp(-127, 127).to(torch.int8), scale


def states(n, d, N, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    row = (torch.randn(n, d, 1, generator=g) * spread).exp()
    return (torch.randn(n, d, N, generator=g) * row).cuda()


@pytest.mark.parametrize("N", [16, 32, 64, 128])
@pytest.mark.parametrize("n,d", [(1, 1), (3, 7), (2, 129), (5, 640)])
def test_store_and_load(n, d, N):
    x = states(n, d, N, n * d + N)
    S = n + 3
    pq, ps = naju.state_pool(S, d, N, "cuda")
    pq.fill_(5)
    ps.fill_(2.0)
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(N))[:n].int().cuda()
    naju.state_store(x, slots, pq, ps)
    q, s = reference(x)
    idx = slots.long().cpu()
    assert torch.equal(pq.cpu()[idx], q) and torch.equal(ps.cpu()[idx], s)
    rest = [i for i in range(S) if i not in idx.tolist()]  # other slots keep their values
    assert bool((pq.cpu()[rest] == 5).all()) and bool((ps.cpu()[rest] == 2.0).all())
    back = naju.state_load(pq, ps, slots)
    assert torch.equal(back.cpu(), s[..., None] * q.float())
    err = (back.double() - x.double()).abs()
    assert bool((err <= (0.5 + 127 * 2.0 ** -23) * ps[slots.long()].double()[..., None]).all())


def test_borders_are_exact():
    """Values on and next to the middles between two quanta."""
    d, N = 64, 128
    g = torch.Generator().manual_seed(3)
    top = torch.rand(1, d, 1, generator=g) * 3 + 0.5
    s = (top / 127).float()
    k = torch.randint(-126, 126, (1, d, N), generator=g).float() + 0.5
    x = (k.double() * s.double()).float()
    x = torch.where(torch.rand(x.shape, generator=g) < 0.3, torch.nextafter(x, x * 2), x)
    x = torch.where(torch.rand(x.shape, generator=g) < 0.3, torch.nextafter(x, x * 0), x)
    x[..., :1] = top
    # a power-of-two scale makes the middles themselves representable
    x[0, :8, 1:] = k[0, :8, 1:] / 1024
    x[0, :8, 0] = 127 / 1024
    pq, ps = naju.state_pool(1, d, N, "cuda")
    naju.state_store(x.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), pq, ps)
    q, s = reference(x)
    assert torch.equal(ps.cpu(), s) and torch.equal(pq.cpu(), q)


def test_extreme_rows():
    """All zero, one large value, tiny (subnormal) and the largest values,
    infinities and NaN."""
    d, N = 10, 16
    x = torch.zeros(1, d, N)
    x[0, 1, 3] = 1e30
    x[0, 2] = torch.linspace(-1, 1, N) * 1e-40
    x[0, 3] = torch.linspace(-1, 1, N) * 3.4e38
    x[0, 4, 0] = float("inf")
    x[0, 5, 7] = float("-inf")
    x[0, 6, 15] = float("nan")
    x[0, 7] = 1e-45
    x[0, 8] = -2.5
    x[0, 9] = torch.linspace(-1, 1, N) * 2e-38
    pq, ps = naju.state_pool(1, d, N, "cuda")
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    naju.state_store(x.cuda(), slot, pq, ps)
    back = naju.state_load(pq, ps, slot).cpu()
    assert bool((back[0, 0] == 0).all()) and bool((back[0, 7] == 0).all())
    assert bool(torch.isnan(back[0, 4:7]).all())
    fine = [1, 2, 3, 8, 9]
    q, s = reference(x[:, fine])
    assert torch.equal(ps.cpu()[:, fine], s) and torch.equal(pq.cpu()[:, fine], q)
    assert torch.equal(back[:, fine], s[..., None] * q.float())


def test_slots_outside_and_named_twice():
    n, d, N = 6, 100, 32
    x = states(n, d, N, 5)
    pq, ps = naju.state_pool(4, d, N, "cuda")
    slots = torch.tensor([2, -1, 2, 4, 0, 2], dtype=torch.int32, device="cuda")
    for _ in range(3):
        naju.state_store(x, slots, pq, ps)
        q, s = reference(x)
        assert torch.equal(pq[2].cpu(), q[5]) and torch.equal(ps[2].cpu(), s[5])
        assert torch.equal(pq[0].cpu(), q[4])
        assert float(ps[1].abs().max()) == 0 and float(ps[3].abs().max()) == 0
    state = torch.full((n, d, N), 9.0, device="cuda")
    back = naju.state_load(pq, ps, slots, state=state)
    assert back is state
    assert bool((back[1] == 0).all()) and bool((back[3] == 0).all())
    assert torch.equal(back[0], back[5]) and torch.equal(back[0], back[2])


def test_captured_and_on_another_stream():
    n, d, N = 4, 200, 64
    x, y = states(n, d, N, 7), states(n, d, N, 8)
    pq, ps = naju.state_pool(6, d, N, "cuda")
    slots = torch.tensor([5, 1, 0, 3], dtype=torch.int32, device="cuda")
    want = naju.state_pool(6, d, N, "cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        naju.state_store(y, slots, *want)
        out = naju.state_load(*want, slots)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        naju.state_store(x, slots, pq, ps)
        back = naju.state_load(pq, ps, slots)
    x.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(pq, want[0]) and torch.equal(ps, want[1]) and torch.equal(back, out)


def test_a_session_parked_and_resumed():
    """Decode steps before and after a store and load, in another batch place:
    y differs from the uninterrupted run by the rounding of the state alone."""
    n, d, N = 3, 64, 64
    g = torch.Generator().manual_seed(9)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    state = rn(n, d, N)
    a, b, h, B, C, D = rn(n, d) + 5, rn(n, d) - 2, rn(n, d), rn(n, N), rn(n, N), rn(d)
    straight = state.clone()
    pq, ps = naju.state_pool(8, d, N, "cuda")
    slots = torch.tensor([7, 2, 4], dtype=torch.int32, device="cuda")
    naju.state_store(state, slots, pq, ps)
    order = [2, 0, 1]
    resumed = naju.state_load(pq, ps, slots[order].contiguous())
    y1 = naju.scan_step(straight, h, a, b, B, C, D=D)
    pick = lambda t: t[order].contiguous()  # noqa: E731
    y2 = naju.scan_step(resumed, pick(h), pick(a), pick(b), pick(B), pick(C), D=D)
    f = torch.sigmoid(a.double())
    quantum = ps[slots.long()].double()[..., None] * 0.5
    allow = (f * (quantum * C.double().abs()[:, None]).sum(-1) / N ** 0.5)[order]
    err = (y2.double() - y1.double()[order]).abs()
    # half a quantum of every state value, decayed and read out; 1e-5: fp32 sums
    assert bool((err <= allow + 1e-5 * (1 + y1.double().abs()[order])).all())
    assert float(np.abs(np.asarray(err.cpu())).max()) > 0


def test_offsets_past_32_bits():
    d, N, S = 2048, 64, 16500
    assert S * d * N > 2 ** 31
    pq, ps = naju.state_pool(S, d, N, "cuda")
    x = states(2, d, N, 12)
    slots = torch.tensor([S - 1, 16390], dtype=torch.int32, device="cuda")
    naju.state_store(x, slots, pq, ps)
    q, s = reference(x)
    assert torch.equal(pq[slots.long()].cpu(), q) and torch.equal(ps[slots.long()].cpu(), s)
    assert torch.equal(naju.state_load(pq, ps, slots).cpu(), s[..., None] * q.float())
    assert int(pq[:4].abs().max()) == 0  # (where an offset cut to 32 bits would land)


def test_scale_is_the_rounded_quotient():
    """Maxima of every size, subnormal ones among them, and the largest values'
    neighbours: the stored scale is max / 127, rounded once."""
    n, d, N = 4, 65536, 16
    g = torch.Generator().manual_seed(17)
    bits = torch.randint(0, 0x7f800000, (n, d), generator=g, dtype=torch.int64).int()
    bits[0, :4096] = torch.arange(4096, dtype=torch.int32)               # the smallest
    bits[1, :4096] = 0x7f7fffff - torch.arange(4096, dtype=torch.int32)  # the largest
    bits[2, :] = 0x3f800000 + torch.randint(0, 1 << 23, (d,), generator=g, dtype=torch.int64).int()
    top = bits.view(torch.float32)
    x = torch.zeros(n, d, N)
    x[..., 5] = -top
    x[..., 9] = top / 3
    pq, ps = naju.state_pool(n, d, N, "cuda")
    naju.state_store(x.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"), pq, ps)
    q, s = reference(x)
    want = torch.from_numpy(top.numpy() / np.float32(127))  # IEEE division
    assert torch.equal(s, want) and torch.equal(ps.cpu(), want)
    fine = want >= 2.0 ** -126  # (a scale below the normal range is itself coarse)
    assert torch.equal(pq.cpu()[fine], q[fine])
