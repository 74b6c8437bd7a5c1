"""The block with a vector state against its fp64 definition, and the block's
decode path (prefill, step, 4-bit projections, parked states) against the
forward and against fp64 arithmetic on the weights it really uses."""
import numpy as np
import pytest
import torch

import discrete_selective_ssm_b200 as naju
import vscan_ref as ref
from discrete_selective_ssm_b200.block import EPS, PARAMS, VECTOR_PARAMS, NajuBlock, init_params
from naju_check import TOL_F32, assert_close
from oracle import block as ob
from oracle import conv_silu_bwd, conv_silu_fwd
from test_gpu_w4 import weights

pytestmark = pytest.mark.gpu


def flat(t):
    return t.reshape(-1, t.shape[-1])


def vector_fwd(x, p, coupled):
    """fp64 block with a vector state: returns (out, final state, cache)."""
    p = {k: np.asarray(v, np.float64) for k, v in p.items()}
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + EPS)
    n = x * r
    xn = n * p["norm_w"]
    uz = xn @ p["W_in"]
    di = p["W_in"].shape[1] // 2
    u, z = uz[..., :di], uz[..., di:]
    h = conv_silu_fwd(u, p["conv_w"], p["conv_b"])
    a = h @ p["W_a"] + p["b_a"]
    b = None if coupled else h @ p["W_b"] + p["b_b"]
    y, xl, _ = ref.fwd(h, a, b, z)
    return x + y @ p["W_out"], xl, dict(r=r, n=n, xn=xn, u=u, z=z, h=h, a=a, b=b, y=y, p=p)


def vector_bwd(c, dout, coupled):
    p, g = c["p"], {}
    g["W_out"] = flat(c["y"]).T @ flat(dout)
    sg = ref.bwd(dout @ p["W_out"].T, c["h"], c["a"], c["b"], c["z"])
    dh = sg["dh"] + sg["da"] @ p["W_a"].T
    g["W_a"], g["b_a"] = flat(c["h"]).T @ flat(sg["da"]), flat(sg["da"]).sum(0)
    if not coupled:
        dh = dh + sg["db"] @ p["W_b"].T
        g["W_b"], g["b_b"] = flat(c["h"]).T @ flat(sg["db"]), flat(sg["db"]).sum(0)
    du, g["conv_w"], g["conv_b"] = conv_silu_bwd(c["u"], p["conv_w"], p["conv_b"], dh)
    duz = np.concatenate([du, sg["dz"]], axis=-1)
    g["W_in"] = flat(c["xn"]).T @ flat(duz)
    dxn = duz @ p["W_in"].T
    g["norm_w"] = flat(dxn * c["n"]).sum(0)
    dn = dxn * p["norm_w"]
    return dout + c["r"] * (dn - c["n"] * np.mean(dn * c["n"], axis=-1, keepdims=True)), g


@pytest.mark.parametrize("coupled", [False, True])
def test_vector_state_block(coupled):
    """fp32 against fp64 at the existing block's tolerance (same projections)."""
    Bt, L, dm, di = 2, 150, 48, 72
    params = init_params(dm, di, 1, seed=21)
    assert set(params) == set(VECTOR_PARAMS) and set(init_params(dm, di, 16)) == set(PARAMS)
    blk = NajuBlock(dm, di, 1, "cuda", dtype=torch.float32, params=params, coupled=coupled)
    gen = torch.Generator().manual_seed(22)
    x, dout = torch.randn(Bt, L, dm, generator=gen), torch.randn(Bt, L, dm, generator=gen)
    out, ctx = blk.forward(x.cuda())
    dx, g = blk.backward(ctx, dout.cuda())
    ro, _, c = vector_fwd(x.numpy(), params, coupled)
    rdx, rg = vector_bwd(c, dout.double().numpy(), coupled)
    assert_close(out, ro, TOL_F32, name="out")
    assert_close(dx, rdx, TOL_F32, name="dx")
    for k, v in rg.items():
        assert_close(g[k], v, TOL_F32, name=k)
    if coupled:
        assert float(g["W_b"].abs().max()) == 0.0


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("N", [1, 16, 64])
@pytest.mark.parametrize("prompt", [1, 2, 3, 40])
def test_steps_go_on_from_a_prefill(prompt, N, coupled):
    """Prefill and steps give the outputs of one forward over all tokens."""
    Bt, L, dm, di = 3, 48, 40, 56
    blk = NajuBlock(dm, di, N, "cuda", dtype=torch.float32, seed=N, coupled=coupled)
    x = torch.randn(Bt, L, dm, generator=torch.Generator().manual_seed(3)).cuda()
    whole, _ = blk.forward(x)
    out, state = blk.prefill(x[:, :prompt].contiguous())
    outs = [out] + [blk.step(x[:, t].contiguous(), state)[:, None] for t in range(prompt, L)]
    assert_close(torch.cat(outs, 1), whole.cpu().numpy(), TOL_F32, name="out")
    state = blk.new_state(Bt)
    outs = [blk.step(x[:, t].contiguous(), state) for t in range(4)]
    assert_close(torch.stack(outs, 1), whole[:, :4].cpu().numpy(), TOL_F32, name="from nothing")


def read_back(blk):
    """Parameters with every 4-bit projection as it reads back (fp64)."""
    p = {k: v.double().cpu().numpy() for k, v in blk.p.items()}
    for k, (wq, scales, group) in blk.q.items():
        n_in = blk.d_model if k == "W_in" else blk.d_inner
        w = weights(wq, scales, n_in, group).T
        if k == "W_BC":
            p["W_B"], p["W_C"] = w[:, :blk.d_state], w[:, blk.d_state:]
        else:
            p[k] = w
    return p


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("N", [1, 32])
@pytest.mark.parametrize("Bt", [1, 5, 20])
def test_quantised_steps(Bt, N, coupled):
    """Steps on 4-bit projections equal the fp64 block on the weights that the
    4 bits stand for."""
    dm, di, L = 136, 168, 12
    blk = NajuBlock(dm, di, N, "cuda", dtype=torch.float32, seed=5, coupled=coupled)
    blk.quantize(group=32)
    x = torch.randn(Bt, L, dm, generator=torch.Generator().manual_seed(4))
    state = blk.new_state(Bt)
    outs = torch.stack([blk.step(x[:, t].cuda().contiguous(), state) for t in range(L)], 1)
    p = read_back(blk)
    if N == 1:
        want, xl, _ = vector_fwd(x.numpy(), p, coupled)
        assert_close(state["state"], xl, TOL_F32, name="state")
    else:
        want, _ = ob.block_fwd(x.numpy(), p, coupled)
    assert_close(outs, want, TOL_F32, name="out")


def test_a_served_session():
    """A batch as it is served in bf16: prompts prefilled, decoded on 4-bit
    projections, parked, resumed in other places with a new session among
    them, and decoded on.  Every output is compared with the same block at
    fp32 from the same states (bf16 rounding of a handful of intermediate
    vectors, each off by at most 2^-9 of its largest value)."""
    Bt, dm, di, N = 6, 256, 512, 64
    blk = NajuBlock(dm, di, N, "cuda", dtype=torch.bfloat16, seed=8)
    blk.quantize()
    full = NajuBlock(dm, di, N, "cuda", dtype=torch.float32,
                     params={k: v.float() for k, v in blk.p.items()})
    full.q = blk.q
    g = torch.Generator().manual_seed(6)
    x = torch.randn(Bt, 30, dm, generator=g).bfloat16().cuda()
    _, state = blk.prefill(x[:, :20].contiguous())
    clone = lambda s: {k: v.clone() for k, v in s.items()}  # noqa: E731

    def both(t, st):
        other = clone(st)
        y = blk.step(t, st)
        assert y.dtype == torch.bfloat16
        assert_close(y, full.step(t.float(), other).cpu().numpy(), 2e-2, name="step")

    for t in range(20, 25):
        both(x[:, t].contiguous(), state)
    pq, ps = naju.state_pool(9, di, N, "cuda")
    slots = torch.tensor([3, 8, 0, 5, 1, 7], dtype=torch.int32, device="cuda")
    naju.state_store(state["state"], slots, pq, ps)
    places = [4, 2, 0]  # three come back, the last place is a new session
    back = torch.tensor([slots[i].item() for i in places] + [-1], dtype=torch.int32,
                        device="cuda")
    conv = torch.cat([state["conv"][places], torch.zeros_like(state["conv"][:1])])
    resumed = {"state": naju.state_load(pq, ps, back), "conv": conv.contiguous()}
    half = ps[slots.long()][places] * 0.5
    err = (resumed["state"][:3] - state["state"][places]).abs().amax(-1)
    assert bool((err <= half * (1 + 1e-4)).all())
    assert float(resumed["state"][3].abs().max()) == 0.0
    for t in range(25, 30):
        both(x[:4, t].contiguous(), resumed)


def test_bf16_gradients_of_the_vector_block_run():
    blk = NajuBlock(64, 128, 1, "cuda", seed=9)
    x = torch.randn(2, 70, 64, device="cuda", dtype=torch.bfloat16)
    out, ctx = blk.forward(x)
    dx, g = blk.backward(ctx, torch.ones_like(out))
    assert set(g) == set(VECTOR_PARAMS)
    for t in (out, dx, *g.values()):
        assert bool(torch.isfinite(t.float()).all())


def test_a_wider_residual_keeps_its_bits():
    """fp32 inputs to a bf16 block: the residual is added in fp32, as in forward."""
    blk = NajuBlock(64, 128, 16, "cuda", seed=10)
    x = torch.randn(2, 1, 64, device="cuda")
    out, _ = blk.forward(x)
    for quantised in (False, True):
        if quantised:
            blk.quantize()
        y = blk.step(x[:, 0].contiguous(), blk.new_state(2))
        assert y.dtype == torch.float32
        # what the block adds is rounded to bf16, the sum is not
        added = (y - x[:, 0]).double().cpu().numpy()
        assert float(np.abs((x[:, 0] + (y - x[:, 0]).bfloat16() - y).cpu().numpy()).max()) <= 1e-6
        if not quantised:
            assert_close(y, out[:, 0].cpu().numpy(), 1e-2, name="out")
        assert np.abs(added).max() > 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [1, 16])
def test_steps_take_strided_tokens(N, dtype):
    """Tokens cut out of a prompt, and with the batch as the inner dimension,
    on the full and on the 4-bit projections."""
    blk = NajuBlock(64, 128, N, "cuda", dtype=dtype, seed=11)
    x = torch.randn(3, 5, 64, generator=torch.Generator().manual_seed(12)).to(dtype).cuda()
    for quantised in (False, True):
        if quantised:
            blk.quantize(group=32)
        want = blk.step(x[:, 2].contiguous(), blk.new_state(3))
        assert not x[:, 2].is_contiguous()
        assert torch.equal(blk.step(x[:, 2], blk.new_state(3)), want)
        inner = x[:, 2].t().contiguous().t()
        assert torch.equal(blk.step(inner, blk.new_state(3)), want)
