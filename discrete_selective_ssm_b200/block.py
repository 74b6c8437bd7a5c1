"""The full Naju block around the library (Naju reproduction README, block
flowchart): normalized token -> input projection (u, z) -> causal depthwise
conv + SiLU (h) -> gate logits a, b and token directions B, C projected from
h -> native-discrete state scan with readout and feedthrough -> SiLU(z)
output modulation -> output projection -> residual.

The dense parts (RMSNorm, the projections: cuBLAS GEMMs through torch) are
plain library calls; the conv, the scan and their gradients run in this
package's kernels (h-mode scan, so the projections of h can add their own
gradient to dh before the conv backward).  Readings where the pages are
silent: RMSNorm with eps 1e-6; a, b, B, C are linear maps of h, with the
preserve-first biases forget_bias = 5 on a and write_bias = -2 on b (README
"Core equations") and no bias on B, C or the output projection.
`coupled=True` drops the b projection: i = 1 - f.  d_state = 1 keeps one state
value per channel instead of a row (the vector-state scan: no B, C and D).

Decoding: prefill(x) runs a prompt and returns the state it leaves, step(x,
state) one token from there.  quantize() lays the projections out in 4 bits
for step(); the state's matrices park in a pool of the package's 8-bit state
cache (state_pool, state_store, state_load).
"""
from __future__ import annotations

import math

import torch

from . import _native as nj

EPS = 1e-6
PARAMS = ("norm_w", "W_in", "conv_w", "conv_b", "W_a", "b_a", "W_b", "b_b", "W_B", "W_C",
          "D", "W_out")
# parameters of a block with a vector state (d_state 1)
VECTOR_PARAMS = tuple(k for k in PARAMS if k not in ("W_B", "W_C", "D"))
# parameters kept in fp32 whatever the activation dtype
_FP32 = ("norm_w", "conv_w", "conv_b", "b_a", "b_b", "D")


class NajuBlock:
    """Parameters live in `self.p` (CUDA tensors).  forward(x) returns
    (out, ctx); backward(ctx, dout) returns (dx, grads) with one gradient per
    parameter (fp32 for the fp32 parameters, the activation dtype otherwise)."""

    def __init__(self, d_model: int, d_inner: int, d_state: int, device, dtype=torch.bfloat16,
                 params: dict | None = None, seed: int = 0, coupled: bool = False):
        self.d_model, self.d_inner, self.d_state = d_model, d_inner, d_state
        self.dtype, self.coupled = dtype, coupled
        self.q = None  # 4-bit projections of step(), set by quantize()
        if params is None:
            params = init_params(d_model, d_inner, d_state, seed)
        self.p = {k: torch.as_tensor(v).to(device=device,
                                           dtype=torch.float32 if k in _FP32 else dtype)
                  .contiguous() for k, v in params.items()}

    # ------------------------------------------------------------ forward
    def forward(self, x: torch.Tensor):
        out, _, ctx = self._forward(x, False)
        return out, ctx

    def _forward(self, x: torch.Tensor, want_final: bool):
        p, dt = self.p, self.dtype
        xf = x.float()
        r = torch.rsqrt(xf.pow(2).mean(-1, keepdim=True) + EPS)
        n = xf * r
        xn = (n * p["norm_w"]).to(dt)
        uz = xn @ p["W_in"]
        di = self.d_inner
        u, z = uz[..., :di].contiguous(), uz[..., di:].contiguous()
        h = nj.conv_silu_fwd(u, p["conv_w"], p["conv_b"])
        a = (h @ p["W_a"] + p["b_a"]).to(dt)
        b = None if self.coupled else (h @ p["W_b"] + p["b_b"]).to(dt)
        B = C = None
        if self.d_state == 1:
            y, xf_, ws = nj.vscan_fwd(h, a, b, z=z, want_final=want_final)
        else:
            B = (h @ p["W_B"]).contiguous()
            C = (h @ p["W_C"]).contiguous()
            y, xf_, ws = nj.scan_fwd(h, a, b, B, C, z=z, D=p["D"], want_final=want_final)
        out = (xf + (y @ p["W_out"]).float()).to(x.dtype)
        ctx = dict(x=x, r=r, n=n, xn=xn, u=u, z=z, h=h, a=a, b=b, B=B, C=C, y=y, ws=ws)
        return out, xf_, ctx

    # ----------------------------------------------------------- backward
    def backward(self, ctx: dict, dout: torch.Tensor):
        p, dt, c = self.p, self.dtype, ctx
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        g = {}
        do = dout.to(dt)
        g["W_out"] = flat(c["y"]).t() @ flat(do)
        dy = (do @ p["W_out"].t()).contiguous()
        if self.d_state == 1:
            sg = nj.vscan_bwd(dy, c["h"], c["a"], c["b"], c["ws"], z=c["z"], want_dx0=False)
            dh = sg["dh"].float() + (sg["da"] @ p["W_a"].t()).float()
        else:
            sg = nj.scan_bwd(dy, c["h"], c["a"], c["b"], c["B"], c["C"], c["ws"], z=c["z"],
                             D=p["D"], want_dx0=False)
            g["D"] = sg["dD"]
            dh = sg["dhu"].float() + (sg["da"] @ p["W_a"].t()).float() \
                + (sg["dB"] @ p["W_B"].t()).float() + (sg["dC"] @ p["W_C"].t()).float()
        g["W_a"] = flat(c["h"]).t() @ flat(sg["da"])
        g["b_a"] = flat(sg["da"]).float().sum(0)
        if self.coupled:
            g["W_b"] = torch.zeros_like(p["W_b"])
            g["b_b"] = torch.zeros_like(p["b_b"])
        else:
            dh = dh + (sg["db"] @ p["W_b"].t()).float()
            g["W_b"] = flat(c["h"]).t() @ flat(sg["db"])
            g["b_b"] = flat(sg["db"]).float().sum(0)
        if self.d_state != 1:
            g["W_B"] = flat(c["h"]).t() @ flat(sg["dB"])
            g["W_C"] = flat(c["h"]).t() @ flat(sg["dC"])
        du, g["conv_w"], g["conv_b"] = nj.conv_silu_bwd(c["u"], p["conv_w"], p["conv_b"],
                                                        dh.to(dt).contiguous())
        duz = torch.cat([du, sg["dz"]], dim=-1)
        g["W_in"] = flat(c["xn"]).t() @ flat(duz)
        dxn = (duz @ p["W_in"].t()).float()
        g["norm_w"] = flat(dxn * c["n"]).sum(0)
        dn = dxn * p["norm_w"]
        dx = c["r"] * (dn - c["n"] * (dn * c["n"]).mean(-1, keepdim=True))
        return (dout.float() + dx).to(dout.dtype), g

    # ------------------------------------------------------------- decode
    def new_state(self, batch: int) -> dict:
        """The state of `batch` sessions before their first token."""
        dev = self.p["W_in"].device
        row = (self.d_inner,) if self.d_state == 1 else (self.d_inner, self.d_state)
        return {"state": torch.zeros((batch, *row), dtype=torch.float32, device=dev),
                "conv": torch.zeros((batch, self.d_inner, 3), dtype=torch.float32, device=dev)}

    def prefill(self, x: torch.Tensor):
        """forward over a prompt [batch, L, d_model]; returns (out, state) with
        the state that step() goes on from."""
        out, state, ctx = self._forward(x, True)
        conv = torch.zeros((*state.shape[:2], 3), dtype=torch.float32, device=x.device)
        last = ctx["u"][:, -3:].float().transpose(1, 2)  # the last three inputs, oldest first
        conv[:, :, 3 - last.shape[2]:] = last
        return out, {"state": state, "conv": conv}

    def quantize(self, group: int = 128) -> None:
        """Lays the projections out in 4 bits with one scale per `group` inputs;
        step() then reads those.  The full weights stay as they are (forward,
        prefill and backward use them); after they change, call this again."""
        p = self.p
        mats = {"W_in": p["W_in"], "W_a": p["W_a"], "W_out": p["W_out"]}
        if not self.coupled:
            mats["W_b"] = p["W_b"]
        if self.d_state != 1:
            mats["W_BC"] = torch.cat([p["W_B"], p["W_C"]], 1)
        self.q = {k: (*nj.w4_quantize(w.t().contiguous(), group), group) for k, w in mats.items()}

    def _project(self, name: str, x, bias=None, residual=None):
        if self.q is not None:
            wq, scales, group = self.q[name]
            return nj.w4_linear(x, wq, scales, group, bias=bias, residual=residual)
        w = torch.cat([self.p["W_B"], self.p["W_C"]], 1) if name == "W_BC" else self.p[name]
        y = x @ w
        if bias is not None:
            y = y + bias
        if residual is not None:
            y = residual.float() + y.float()
        return y.to(x.dtype)

    def step(self, x: torch.Tensor, state: dict) -> torch.Tensor:
        """One token x [batch, d_model] of every session; `state` (new_state or
        prefill) is updated in place.  Returns the block's output."""
        p, dt, di = self.p, self.dtype, self.d_inner
        x = x.contiguous()  # (tokens of a prompt, x[:, t], are strided)
        xf = x.float()
        r = torch.rsqrt(xf.pow(2).mean(-1, keepdim=True) + EPS)
        uz = self._project("W_in", (xf * r * p["norm_w"]).to(dt))
        u, z = uz[:, :di].contiguous(), uz[:, di:].contiguous()
        h = nj.conv_silu_step(state["conv"], u, p["conv_w"], p["conv_b"])
        a = self._project("W_a", h, bias=p["b_a"])
        b = None if self.coupled else self._project("W_b", h, bias=p["b_b"])
        if self.d_state == 1:
            y = nj.vscan_step(state["state"], h, a, b, z)
        else:
            bc = self._project("W_BC", h)
            y = nj.scan_step(state["state"], h, a, b, bc[:, :self.d_state].contiguous(),
                             bc[:, self.d_state:].contiguous(), z, p["D"])
        if x.dtype == dt:
            return self._project("W_out", y, residual=x)
        return (xf + self._project("W_out", y).float()).to(x.dtype)


def init_params(d_model: int, d_inner: int, d_state: int, seed: int = 0) -> dict:
    """Seeded fp32 parameters (CPU tensors), scaled so activations stay O(1);
    without W_B, W_C and D for a vector state (d_state 1)."""
    gen = torch.Generator().manual_seed(seed)
    s_in, s_h = 1.0 / math.sqrt(d_model), 1.0 / math.sqrt(d_inner)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    params = {
        "norm_w": 1.0 + 0.1 * rn(d_model),
        "W_in": rn(d_model, 2 * d_inner) * s_in,
        "conv_w": rn(d_inner, 4) * 0.5,
        "conv_b": rn(d_inner) * 0.1,
        "W_a": rn(d_inner, d_inner) * s_h,
        "b_a": torch.full((d_inner,), 5.0),
        "W_b": rn(d_inner, d_inner) * s_h,
        "b_b": torch.full((d_inner,), -2.0),
        "W_B": rn(d_inner, d_state) * s_h,
        "W_C": rn(d_inner, d_state) * s_h,
        "D": rn(d_inner),
        "W_out": rn(d_inner, d_model) * s_h,
    }
    return {k: v for k, v in params.items() if d_state != 1 or k in VECTOR_PARAMS}
