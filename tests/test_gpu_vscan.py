"""The vector-state scan (forward, backward, decode step) against the fp64
definition in vscan_ref.

Bounds, element by element.  Every operation of the kernels rounds by at most
half a step (u = 2^-24 relative); a gate value is off by at most 6 u of itself
(base-2 exponential 2 steps, its argument, the sum, the reciprocal), times a
further |logit| u where it is the small one.  A term of x_t passes at most
t + 1 gates and additions, so x_t is off by at most 8 u (t + 8) of the same
recurrence over |h| and |x0|; a gradient is such a product of a forward and a
reverse recurrence: 8 u (L + 16 + max|logit|) of the gradient formed of absolute
values.  bf16 outputs add half a bf16 step, 2^-8 of the value.
"""
import math

import numpy as np
import pytest
import torch

import discrete_selective_ssm_b200 as naju
import vscan_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(Bt, L, d, dtype="f32", coupled=False, z=True, x0=True, seed=0, a=(5.0, 1.0),
         b=(-2.0, 1.0)):
    g = torch.Generator().manual_seed(1000 + seed)

    def rn(shape, mean=0.0, std=1.0, dt=DT[dtype]):
        return (torch.randn(shape, generator=g) * std + mean).to(dt).cuda()

    act = (Bt, L, d)
    return {"h": rn(act), "a": rn(act, *a), "b": None if coupled else rn(act, *b),
            "z": rn(act) if z else None, "dy": rn(act),
            "x0": rn((Bt, d), dt=torch.float32) if x0 else None,
            "dx_final": rn((Bt, d), dt=torch.float32) if x0 else None}


def bounds(t):
    """Sums of absolute values: (y, x_final) and the gradients."""
    ab = lambda v: None if v is None else v.double().abs()  # noqa: E731
    h, a, b, z, x0, dy, dxf = (t[k] for k in ("h", "a", "b", "z", "x0", "dy", "dx_final"))
    _, xf, xs = ref.fwd(ab(h), a, b, None, ab(x0))
    av, zv = ref.f64(a), ref.f64(z)
    f, fc = ref.sigmoid(av), ref.sigmoid(-av)
    i = fc if b is None else ref.sigmoid(ref.f64(b))
    ic = None if b is None else ref.sigmoid(-ref.f64(b))
    y, dyv, out = xs[:, 1:], np.abs(ref.f64(dy)), {}
    dx = dyv
    if z is not None:
        s = ref.sigmoid(zv)
        y = y * np.abs(zv) * s
        out["dz"] = dyv * xs[:, 1:] * (s + np.abs(zv) * s * (1 - s))
        dx = dyv * np.abs(zv) * s
    g = np.zeros_like(dx)
    r = np.zeros_like(xf) if dxf is None else np.abs(ref.f64(dxf))
    for k in range(dx.shape[1] - 1, -1, -1):
        g[:, k] = dx[:, k] + r
        r = f[:, k] * g[:, k]
    hv = np.abs(ref.f64(h))
    out["dx0"], out["dh"] = r, g * i
    out["da"] = g * (xs[:, :-1] + (hv if b is None else 0.0)) * f * fc
    if b is not None:
        out["db"] = g * hv * i * ic
    return y, xf, out


def factor(t):
    m = max(float(t[k].float().nan_to_num(posinf=0, neginf=0).abs().max())
            for k in ("a", "b", "z") if t[k] is not None)
    return 8 * U * (t["h"].shape[1] + 16 + m)


def near(got, want, allow, name):
    g = ref.f64(got)
    assert g.shape == want.shape, name
    assert np.all(np.isfinite(g)), f"{name}: non-finite values"
    if got.dtype == torch.bfloat16:
        allow = allow + 2.0 ** -8 * np.abs(want)
    over = np.abs(g - want) - allow - 1e-30
    k = np.unravel_index(np.argmax(over), over.shape)
    assert over[k] <= 0, f"{name} at {k}: got {g[k]!r}, want {want[k]!r}, allowed {allow[k]:.3e}"


def run(t, out_dtype=None, **kw):
    y, xf, ws = naju.vscan_fwd(t["h"], t["a"], t["b"], z=t["z"], x0=t["x0"],
                               out_dtype=out_dtype, **kw)
    g = naju.vscan_bwd(t["dy"], t["h"], t["a"], t["b"], ws, z=t["z"], dx_final=t["dx_final"],
                       out_dtype=out_dtype)
    assert naju.last_device_status(ws) == 0
    return y, xf, g


def check(t, out_dtype=None):
    y, xf, g = run(t, out_dtype)
    ry, rx, _ = ref.fwd(t["h"], t["a"], t["b"], t["z"], t["x0"])
    rg = ref.bwd(t["dy"], t["h"], t["a"], t["b"], t["z"], t["x0"], t["dx_final"])
    by, bx, bg = bounds(t)
    k = factor(t)
    near(y, ry, k * by, "y")
    near(xf, rx, k * bx, "x_final")
    for n in ("dh", "da", "db", "dz", "dx0"):
        assert (g[n] is None) == (rg[n] is None), n
        if g[n] is not None:
            near(g[n], rg[n], 2 * k * bg[n], n)
    return y, xf, g


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parity(dtype, z, coupled):
    check(make(2, 300, 200, dtype, coupled, z), naju.F32)


@pytest.mark.parametrize("L", [1, 2, 7, 8, 63, 64, 65, 127, 129, 640])
@pytest.mark.parametrize("d", [1, 63, 64, 130])
def test_lengths_and_widths(L, d):
    check(make(3, L, d, "bf16", seed=L + d))


@pytest.mark.parametrize("d", [1, 31, 32, 33, 100])
def test_widths_f32(d):
    check(make(2, 97, d, "f32", coupled=True, seed=d))


def test_no_initial_state_and_no_final_gradient():
    check(make(2, 130, 48, "f32", x0=False))


def test_one_long_sequence():
    """Many items of one unit: many rounds of a full cluster."""
    check(make(1, 20000, 40, "f32", seed=9))


def test_long_memory():
    """f within 1e-4 of one: the state sums thousands of tokens."""
    check(make(2, 3000, 32, "f32", seed=3, a=(9.0, 0.5)))


def test_saturated_gates():
    """Logits far out on both sides: neither gate loses its small part."""
    check(make(2, 200, 64, "f32", seed=4, a=(0.0, 12.0), b=(0.0, 12.0)))
    check(make(2, 200, 64, "f32", seed=4, a=(0.0, 12.0), coupled=True))
    check(make(2, 200, 64, "bf16", seed=4, a=(0.0, 30.0), b=(0.0, 30.0)))


def lowest(dt):
    return torch.finfo(dt).min


@pytest.mark.parametrize("far", ["inf", "lowest"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_and_padded(dtype, far):
    """a = -inf starts afresh: the documents of a packed row equal their own
    runs, and no gradient crosses.  a = +inf, b = -inf keeps the state."""
    big = math.inf if far == "inf" else -lowest(DT[dtype])
    t = make(1, 150, 64, dtype, x0=False, seed=6)
    cut = 70
    t["a"][:, cut] = -big
    y, xf, g = run(t)
    s = {k: None if v is None else v[:, cut:].contiguous() for k, v in t.items()}
    y2, xf2, g2 = run(s)
    ab, bb = t["a"].clone(), t["b"].clone()
    ab[:, cut] = -700.0  # the definition's e^{-a} stays finite there
    ry, rx, _ = ref.fwd(t["h"], ab, t["b"], t["z"], None)
    by, bx, _ = bounds({**t, "a": ab})
    near(y, ry, factor(t) * by, "y")
    near(y2, ry[:, cut:], factor(t) * by[:, cut:], "own run")
    assert float(g["da"][:, cut].abs().max()) == 0.0
    for n in ("dh", "da", "db", "dz"):
        near(g[n][:, cut:], ref.f64(g2[n]), 2 ** -7 * np.abs(ref.f64(g2[n])) + 1e-5, n)
    p = make(2, 100, 64, dtype, seed=7)
    q = {k: None if v is None else v[:, :60].contiguous() if v.dim() == 3 else v
         for k, v in p.items()}
    p["a"][:, 60:] = big
    p["b"][:, 60:] = -big
    p["dy"][:, 60:] = 0
    y, xf, g = run(p)
    y2, xf2, g2 = run(q)
    assert torch.equal(y[:, :60], y2)
    assert float(g["db"][:, 60:].abs().max()) == 0.0 and float(g["da"][:, 60:].abs().max()) == 0.0
    _, rx, _ = ref.fwd(q["h"], q["a"], q["b"], None, q["x0"])
    _, bx, bg = bounds(q)
    near(xf, rx, factor(p) * bx, "x_final")
    near(g["dx0"], ref.bwd(q["dy"], q["h"], q["a"], q["b"], q["z"], q["x0"],
                           q["dx_final"])["dx0"], 2 * factor(p) * bg["dx0"], "dx0")


def test_nan_logit_stays():
    t = make(1, 80, 64, "f32", x0=False)
    t["a"][0, 10, 3] = math.nan
    y, xf, _ = naju.vscan_fwd(t["h"], t["a"], t["b"], z=t["z"])
    assert torch.isnan(y[0, 10:, 3]).all() and torch.isnan(xf[0, 3])
    assert torch.isfinite(y[0, :10]).all() and torch.isfinite(y[0, :, :3]).all()


def test_gradients_against_differences():
    t = make(1, 90, 33, "f32", seed=8)
    _, _, g = run(t)

    def loss(s):
        y, xf, _ = ref.fwd(s["h"], s["a"], s["b"], s["z"], s["x0"])
        return float((y * ref.f64(t["dy"])).sum() + (xf * ref.f64(t["dx_final"])).sum())

    for k, n in (("h", "dh"), ("a", "da"), ("b", "db"), ("z", "dz"), ("x0", "dx0")):
        v = torch.randn(t[k].shape, generator=torch.Generator().manual_seed(5)).double()
        e = 1e-5
        hi = loss({**t, k: t[k].double().cpu() + e * v})
        lo = loss({**t, k: t[k].double().cpu() - e * v})
        got = float((g[n].double().cpu() * v).sum())
        size = float((g[n].double().cpu() * v).abs().sum())
        # fp32 gradients (8 u (L + 16) of their terms) and the difference's e^2
        assert abs(got - (hi - lo) / (2 * e)) <= 1e-4 * size, n


def test_bitwise_repeatable():
    """The order in which items finish never changes a result."""
    t = make(2, 9000, 256, "f32", seed=11)
    first = run(t)
    for _ in range(5):
        again = run(t)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        for n in ("dh", "da", "db", "dz", "dx0"):
            assert torch.equal(first[2][n], again[2][n]), n


def test_steps_equal_the_forward():
    t = make(3, 70, 129, "f32", seed=12)
    state = t["x0"].clone()
    ys = [naju.vscan_step(state, *(t[k][:, i].contiguous() for k in ("h", "a", "b", "z")))
          for i in range(70)]
    ry, rx, _ = ref.fwd(t["h"], t["a"], t["b"], t["z"], t["x0"])
    by, bx, _ = bounds(t)
    near(torch.stack(ys, 1), ry, factor(t) * by, "y")
    near(state, rx, factor(t) * bx, "state")


@pytest.mark.parametrize("Bt,d", [(1, 1), (1, 7), (5, 13), (256, 2048), (3, 1000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("coupled", [False, True])
def test_step(Bt, d, dtype, coupled):
    t = make(Bt, 1, d, dtype, coupled, z=not coupled, seed=d)
    one = {k: None if v is None else v.view(Bt, d) for k, v in t.items()}
    state = one["x0"].clone()
    y = naju.vscan_step(state, one["h"], one["a"], one["b"], one["z"])
    ry, rx, _ = ref.fwd(t["h"], t["a"], t["b"], t["z"], t["x0"])
    by, bx, _ = bounds(t)
    near(y, ry[:, 0], factor(t) * by[:, 0], "y")
    near(state, rx, factor(t) * bx, "state")


def test_outputs_stay_inside_their_tensors():
    """Neighbours of every output keep their values (odd width, ragged end)."""
    t = make(1, 67, 33, "bf16", seed=13)
    n = 67 * 33
    bufs = {k: torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
            for k in ("y", "dh", "da", "db", "dz")}
    view = {k: v[:n].view(1, 67, 33) for k, v in bufs.items()}
    y, _, ws = naju.vscan_fwd(t["h"], t["a"], t["b"], z=t["z"], x0=t["x0"], y=view["y"])
    g = {k: view[k] for k in ("dh", "da", "db", "dz")}
    naju.vscan_bwd(t["dy"], t["h"], t["a"], t["b"], ws, z=t["z"], grads=g)
    torch.cuda.synchronize()
    for k, v in bufs.items():
        assert bool((v[n:] == 7.0).all()), k


def test_another_stream_and_a_graph():
    """On a side stream, and captured (forward and backward together) and
    replayed on new inputs while eager results live."""
    t, s = make(2, 500, 64, "f32", seed=14), make(2, 500, 64, "f32", seed=15)
    want = run(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2]["da"], want[2]["da"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, xf, ws = naju.vscan_fwd(t["h"], t["a"], t["b"], z=t["z"], x0=t["x0"])
        g = naju.vscan_bwd(t["dy"], t["h"], t["a"], t["b"], ws, z=t["z"],
                           dx_final=t["dx_final"])
    for k in t:
        t[k].copy_(s[k])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(xf, want[1])
    for n in ("dh", "da", "db", "dz", "dx0"):
        assert torch.equal(g[n], want[2][n]), n


def test_bounded_wait_reports():
    """An item that never publishes its state: the waits run out, the call
    returns, and the next call is right."""
    t = make(1, 300, 32, "f32", seed=16)
    naju.testing_set_wait_limit(200)
    naju.testing_set_skip_publish(True)
    try:
        _, _, ws = naju.vscan_fwd(t["h"], t["a"], t["b"])
        assert naju.last_device_status(ws) == 4
        assert naju.last_device_status(ws) == 0
        naju.vscan_bwd(t["dy"], t["h"], t["a"], t["b"], ws)
        assert naju.last_device_status(ws) == 4
    finally:
        naju.testing_set_wait_limit(0)
        naju.testing_set_skip_publish(False)
    check(t)


def test_refusals_on_device_tensors():
    t = make(1, 10, 32, "f32")
    with pytest.raises(ValueError):
        naju.vscan_fwd(t["h"], t["a"][:, :9])
    with pytest.raises(TypeError):
        naju.vscan_fwd(t["h"], t["a"].bfloat16())
    with pytest.raises(ValueError):
        naju.vscan_fwd(t["h"].transpose(1, 2).contiguous().transpose(1, 2), t["a"])
    with pytest.raises(naju.NajuError):
        naju.vscan_fwd(t["h"][:, :0], t["a"][:, :0])
    with pytest.raises(naju.NajuError):
        naju.vscan_fwd(t["h"], t["a"], out_dtype=naju.BF16)
    with pytest.raises(naju.NajuError):
        naju.vscan_fwd(t["h"], t["a"], workspace=torch.empty(256, dtype=torch.uint8,
                                                             device="cuda"))


@pytest.mark.parametrize("cluster", [1, 2, 3, 4, 8, 13, 16])
def test_blocks_per_unit(cluster):
    """Every cluster size walks the same items: more blocks than items, a last
    round that is not full, and one block alone."""
    naju.testing_set_vscan_cluster(cluster)
    try:
        check(make(1, 700, 72, "bf16", seed=cluster))
        check(make(2, 33, 31, "f32", seed=cluster, coupled=True))
    finally:
        naju.testing_set_vscan_cluster(0)


def test_the_cluster_size_changes_no_more_than_rounding():
    t = make(1, 1500, 64, "f32", seed=30)
    naju.testing_set_vscan_cluster(1)
    try:
        one = run(t)
    finally:
        naju.testing_set_vscan_cluster(0)
    many = run(t)
    by, _, bg = bounds(t)
    near(many[0], ref.f64(one[0]), 2 * factor(t) * by, "y")
    near(many[2]["da"], ref.f64(one[2]["da"]), 4 * factor(t) * bg["da"], "da")


def test_long_rows_of_every_width_path():
    """Widths without 16-byte rows take the plain loads, in both directions."""
    for d, dt in ((65, "bf16"), (66, "bf16"), (33, "f32")):
        check(make(1, 900, d, dt, seed=d))


@pytest.mark.parametrize("d,dtype", [(8, "bf16"), (16, "bf16"), (24, "bf16"), (4, "f32"),
                                     (8, "f32"), (36, "f32")])
def test_rows_narrower_than_a_tile(d, dtype):
    check(make(2, 100, d, dtype, seed=d))


def test_batches_of_short_sequences():
    """Many units of one item or less (the whole batch in one round)."""
    check(make(200, 5, 72, "bf16", seed=40))
    check(make(300, 1, 33, "f32", seed=41, coupled=True))


def test_two_workspaces_at_once():
    """Two streams with a workspace each; one workspace used by one call after
    the other."""
    s, t = make(2, 800, 64, "f32", seed=42), make(2, 800, 64, "f32", seed=43)
    want = [run(s), run(t)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for q in streams:
        q.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for v, q in zip((s, t), streams):
            with torch.cuda.stream(q):
                y, xf, ws = naju.vscan_fwd(v["h"], v["a"], v["b"], z=v["z"], x0=v["x0"])
                g = naju.vscan_bwd(v["dy"], v["h"], v["a"], v["b"], ws, z=v["z"],
                                   dx_final=v["dx_final"])
                got.append((y, xf, g))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[2]["da"], b[2]["da"])
    _, _, ws = naju.vscan_fwd(s["h"], s["a"], s["b"], z=s["z"], x0=s["x0"])
    y, _, ws2 = naju.vscan_fwd(t["h"], t["a"], t["b"], z=t["z"], x0=t["x0"], workspace=ws)
    g = naju.vscan_bwd(t["dy"], t["h"], t["a"], t["b"], ws, z=t["z"], dx_final=t["dx_final"])
    assert ws2 is ws and torch.equal(y, want[1][0]) and torch.equal(g["dh"], want[1][2]["dh"])


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last tokens equal their own run from the
    state before them, and so do their gradients."""
    L, d, cut = 1_049_000, 2048, 1_048_900
    assert L * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    rn = lambda: torch.randn(1, L, d, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    h, a = rn(), rn().add_(4.0)
    y, xf, ws = naju.vscan_fwd(h, a)
    assert naju.last_device_status(ws) == 0
    tail = lambda t: t[:, cut:].contiguous()  # noqa: E731
    before = naju.vscan_fwd(h[:, :cut].contiguous(), a[:, :cut].contiguous())[1]
    y2, xf2, ws2 = naju.vscan_fwd(tail(h), tail(a), x0=before)
    # a state of at most about one, summed in another order; bf16 results
    assert float((xf - xf2).abs().max()) <= 1e-5
    assert float((tail(y).float() - y2.float()).abs().max()) <= 2.0 ** -7 * float(y2.abs().max())
    grads = naju.vscan_bwd(h, h, a, None, ws, want_dx0=False)
    grads2 = naju.vscan_bwd(tail(h), tail(h), tail(a), None, ws2)
    for n in ("dh", "da"):
        one, two = tail(grads[n]).float(), grads2[n].float()
        assert float((one - two).abs().max()) <= 2.0 ** -7 * float(two.abs().max()), n


@pytest.mark.parametrize("a", [math.inf, 60.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_saturated_gate_keeps_the_state(dtype, a):
    """sigmoid(a) is one to fp32's last place: with h = 0 the state passes any
    number of tokens bit for bit, whatever the write gate is, in the forward,
    in steps, and as the adjoint of the backward."""
    t = make(2, 20000, 64, dtype, z=False, seed=50, b=(0.0, 3.0))
    t["h"].zero_()
    t["dy"].zero_()
    t["a"].fill_(a)
    t["b"][:, :, 32:] = t["b"][:, :1, 32:]  # half of the channels: one value throughout
    y, xf, g = run(t, naju.F32)
    assert torch.equal(xf, t["x0"])
    assert torch.equal(y, t["x0"][:, None].expand_as(y))
    assert torch.equal(g["dx0"], t["dx_final"])
    state = t["x0"].clone()
    for k in range(20):
        naju.vscan_step(state, *(t[n][:, k].contiguous() for n in ("h", "a", "b")))
    assert torch.equal(state, t["x0"])


def test_a_flag_without_a_truth_value_is_refused():
    t = make(1, 10, 32, "f32")
    neither = torch.ones(2)
    with pytest.raises(RuntimeError, match="ambiguous"):
        naju.vscan_fwd(t["h"], t["a"], want_final=neither)
    _, _, ws = naju.vscan_fwd(t["h"], t["a"])
    with pytest.raises(RuntimeError, match="ambiguous"):
        naju.vscan_bwd(t["dy"], t["h"], t["a"], None, ws, want_dx0=neither)


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_each_gate_by_itself(dtype, coupled):
    """One token from a state of one with nothing written leaves f, from no
    state with h = 1 the write gate.  The smaller side s of a gate is off by
    at most (1.5 |a| + 10) u of itself (constant and argument of the
    exponential |a| u and 0.3 |a| u, the exponential 2^-22.5, sum u, reciprocal
    2 u, three products), the larger by that of s and half a place below one
    (2^-25); a coupled gate of bf16 logits takes the reciprocal itself (2 u)."""
    n = 8192
    a = torch.linspace(-30.0, 30.0, n).to(DT[dtype]).cuda().view(1, 1, n)
    b = a.flip(-1).contiguous()
    zero, one = torch.zeros_like(a), torch.ones_like(a)
    x1 = torch.ones(1, n, device="cuda")
    write = -a if coupled else b
    half = 2 * U if coupled and dtype == "bf16" else U / 2
    for h, x0, logit in ((zero, x1, a), (one, None, write)):
        _, got, _ = naju.vscan_fwd(h, a, None if coupled else b, x0=x0)
        v = ref.f64(logit).reshape(n)
        s = ref.sigmoid(-np.abs(v))
        allow = s * (1.5 * np.abs(v) + 10) * U + np.where(v >= 0, half, 0.0)
        err = np.abs(ref.f64(got).reshape(n) - ref.sigmoid(v))
        k = int(np.argmax(err - allow))
        assert err[k] <= allow[k], f"logit {v[k]}: off by {err[k] / U:.2f} u, allowed {allow[k] / U:.2f} u"
    state = x1.clone()
    naju.vscan_step(state, zero[0], a[0], None if coupled else b[0])
    v = ref.f64(a).reshape(n)
    allow = ref.sigmoid(-np.abs(v)) * (1.5 * np.abs(v) + 10) * U + np.where(v >= 0, U / 2, 0.0)
    assert (np.abs(ref.f64(state).reshape(n) - ref.sigmoid(v)) <= allow).all()
