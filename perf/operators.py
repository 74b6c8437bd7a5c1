"""The vector-state scan, the 4-bit projection and the 8-bit state cache, as
cases that can be run and timed: `run` computes a case in its plain form
(elementary torch operations, 32 bits or more) or, where `own` is true, makes
the calls that a user makes of this package.

Vector-state scan (the gates of the native-discrete recurrence with one state
value per channel; b absent: the coupled gate i = 1 - f):
    x_t = f_t x_{t-1} + i_t h_t,   f = sigmoid(a), i = sigmoid(b) or 1 - f,
    y_t = x_t SiLU(z_t)            (z optional)
4-bit projection (q in 0..15, one bf16 scale per group of G inputs of a row):
    y = x W^T + bias + residual,   W[o, k] = scale[o, k / G] (q[o, k] - 8)
8-bit state cache (one fp32 scale per row of N state values):
    scale = max|x| / 127 (rounded to fp32), q = round(x / scale) of the exact
    quotient, ties to even; read back as scale q
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def _scan(op, name, Bt, L, d, dtype, z=True, coupled=False, x0=False):
    c = {"op": op, "Bt": Bt, "L": L, "d": d, "dtype": dtype, "z": z, "coupled": coupled, "x0": x0}
    return dict(c, name=name) if name else c


def _w4(name, M, n_in, n_out, group, dtype, bias=False, residual=False):
    c = {"op": "w4", "M": M, "n_in": n_in, "n_out": n_out, "group": group, "dtype": dtype,
         "bias": bias, "residual": residual}
    return dict(c, name=name) if name else c


def _cache(name, n, d, N, slots):
    c = {"op": "cache", "n": n, "d": d, "N": N, "slots": slots}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short fp32 sequence (tiny_fwd_f32's sizes): the call's own latency
        _scan("prefill", "prefill_short", 1, 256, 64, "f32", z=False, x0=True),
        # one long prompt taken in at once: few rows, a long time axis
        _scan("prefill", "prefill_long", 1, 65536, 2048, "bf16", x0=True),
        # a small model's training step (small_lm's sizes), fp32, coupled gate
        _scan("train", "train_small", 8, 512, 192, "f32", coupled=True),
        # a full training step (throughput_train's sizes)
        _scan("train", "train_large", 16, 4096, 2048, "bf16"),
        # one token of one session, and of a full decode batch
        _scan("step", "step_one", 1, 1, 2048, "bf16"),
        _scan("step", "step_batch", 256, 1, 8192, "bf16"),
        # a block's input projection for one session (d_model 1024, d_inner 2048)
        _w4("w4_one", 1, 1024, 4096, 128, "bf16"),
        # a wide projection for one session: the weights come from HBM
        _w4("w4_one_wide", 1, 8192, 28672, 128, "bf16"),
        # gate logits of a small decode batch, odd sizes, fp32, small groups
        _w4("w4_odd", 13, 1000, 1111, 32, "f32", bias=True),
        # a block's input projection for a full decode batch
        _w4("w4_batch", 256, 2048, 4096, 64, "bf16", residual=True),
        # one small session parked and resumed
        _cache("cache_one", 1, 192, 16, 8),
        # a decode batch (throughput_decode's sizes) parked and resumed
        _cache("cache_batch", 256, 2048, 64, 320),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "step", "w4", "w4", "w4", "cache"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("prefill", "train"):
        while True:
            Bt, L, d = _log(rng, 1, 16), _log(rng, 1, 65536), _log(rng, 8, 4096)
            if Bt * L * d <= (1 << (27 if dtype == "bf16" else 26)):
                break
        if rng.random() < 0.5:
            d = max(8, d // 8 * 8)
        return _scan(op, None, Bt, L, d, dtype, rng.random() < 0.5, rng.random() < 0.5,
                     rng.random() < 0.5)
    if op == "step":
        return _scan(op, None, _log(rng, 1, 256), 1, _log(rng, 64, 8192), dtype,
                     rng.random() < 0.5, rng.random() < 0.5, True)
    if op == "w4":
        while True:
            M, n_in, n_out = _log(rng, 1, 256), _log(rng, 64, 8192), _log(rng, 64, 28672)
            if M * n_in * n_out <= (1 << 31) and n_in * n_out <= (1 << 27):
                break
        if rng.random() < 0.5:
            n_in, n_out = max(64, n_in // 64 * 64), max(64, n_out // 64 * 64)
        return _w4(None, M, n_in, n_out, rng.choice([32, 64, 128]), dtype, rng.random() < 0.5,
                   rng.random() < 0.5)
    while True:
        n, d, N = _log(rng, 1, 256), _log(rng, 64, 4096), rng.choice([16, 32, 64, 128])
        if n * d * N <= (1 << 25):
            break
    return _cache(None, n, d, N, n + rng.randrange(1, 65))


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 1000003 + 17)

    def normal(shape, mean=0.0, std=1.0, dt=torch.float32):
        t = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)
        return t.mul_(std).add_(mean).to(dt)

    s = dict(case)
    if case["op"] in ("prefill", "train", "step"):
        Bt, L, d, dt = case["Bt"], case["L"], case["d"], _DT[case["dtype"]]
        act = (Bt, d) if case["op"] == "step" else (Bt, L, d)
        s["h"] = normal(act, dt=dt)
        s["a"] = normal(act, 5.0, 1.0, dt)       # preserve-first biases
        s["b_"] = None if case["coupled"] else normal(act, -2.0, 1.0, dt)
        s["z_"] = normal(act, dt=dt) if case["z"] else None
        if case["op"] == "step":
            s["state"] = normal((Bt, d))
        else:
            s["x0_"] = normal((Bt, d)) if case["x0"] else None
        if case["op"] == "train":
            s["dy"] = normal(act, dt=dt)
        return s
    if case["op"] == "w4":
        M, K, O, G, dt = (case["M"], case["n_in"], case["n_out"], case["group"],
                          _DT[case["dtype"]])
        s["x"] = normal((M, K), dt=dt)
        # packed words: rows padded to whole blocks of 128 inputs with q = 8
        q = normal((O, K), 8.0, 2.5).round_().clamp_(0, 15).to(torch.uint8)
        s["wq"] = _pack(q)
        s["scales"] = (normal((O, -(-K // G))).abs_().add_(0.5) / (3.0 * math.sqrt(K))).to(
            torch.bfloat16)
        s["bias_"] = normal((O,)) if case["bias"] else None
        s["residual_"] = normal((M, O), dt=dt) if case["residual"] else None
        return s
    n, d, N, slots = case["n"], case["d"], case["N"], case["slots"]
    row = normal((n, d, 1)).exp_()               # channels of different size
    s["state"] = normal((n, d, N)).mul_(row)
    perm = torch.randperm(slots, generator=gen, device=dev)[:n].to(torch.int32)
    if n > 3:
        perm[n // 2] = -1                        # a batch place without a session
    s["slots_"] = perm
    s["pool_q"] = torch.zeros((slots, d, N), dtype=torch.int8, device=dev)
    s["pool_s"] = torch.zeros((slots, d), dtype=torch.float32, device=dev)
    return s


def _order(device):
    """Place of input k of a 128-block among its 128 nibbles (byte 0's low
    nibble first): word 4c + j of the block (32 bits, little-endian) holds
    inputs 32j + 8c .. 32j + 8c + 7, the even ones in its nibbles 0-3, the odd
    ones in its nibbles 4-7."""
    k = torch.arange(128, device=device)
    j, c, e = k // 32, k % 32 // 8, k % 8
    return (4 * c + j) * 8 + (e % 2) * 4 + e // 2


def _pack(q):
    """q [out, in] uint8 in 0..15 -> the packed words [out, ceil(in / 128) * 64]."""
    O, K = q.shape
    nb = -(-K // 128)
    full = torch.full((O, nb * 128), 8, dtype=torch.uint8, device=q.device)
    full[:, :K] = q
    nib = torch.empty_like(full).view(O, nb, 128)
    nib[:, :, _order(q.device)] = full.view(O, nb, 128)
    nib = nib.view(O, nb, 64, 2)
    return (nib[..., 0] | (nib[..., 1] << 4)).reshape(O, nb * 64).contiguous()


# -------------------------------------------------------------------- runs
def run(s):
    if own:
        return _RUN_OWN[s["op"]](s)
    return _RUN_PLAIN[s["op"]](s)


def _prefill_own(s):
    import discrete_selective_ssm_b200 as naju
    y, x_final, _ = naju.vscan_fwd(s["h"], s["a"], s["b_"], z=s["z_"], x0=s["x0_"])
    return {"y": y, "x_final": x_final}


def _train_own(s):
    import discrete_selective_ssm_b200 as naju
    y, x_final, ws = naju.vscan_fwd(s["h"], s["a"], s["b_"], z=s["z_"], x0=s["x0_"])
    g = naju.vscan_bwd(s["dy"], s["h"], s["a"], s["b_"], ws, z=s["z_"])
    return {"y": y, "x_final": x_final, **{k: v for k, v in g.items() if v is not None}}


def _step_own(s):
    import discrete_selective_ssm_b200 as naju
    y = naju.vscan_step(s["state"], s["h"], s["a"], s["b_"], z=s["z_"])
    return {"y": y, "state": s["state"]}


def _w4_own(s):
    import discrete_selective_ssm_b200 as naju
    return naju.w4_linear(s["x"], s["wq"], s["scales"], group=s["group"], bias=s["bias_"],
                          residual=s["residual_"])


def _cache_own(s):
    import discrete_selective_ssm_b200 as naju
    naju.state_store(s["state"], s["slots_"], s["pool_q"], s["pool_s"])
    back = naju.state_load(s["pool_q"], s["pool_s"], s["slots_"])
    return {"state": back, "scales": s["pool_s"]}


def _gates(s):
    """h, f, 1 - f and the write gate in 32 bits."""
    a = s["a"].float()
    f, fc = torch.sigmoid(a), torch.sigmoid(-a)
    i = fc if s["b_"] is None else torch.sigmoid(s["b_"].float())
    return s["h"].float(), f, fc, i


def _recur(f, v):
    """x_t = f_t x_{t-1} + v_t over dimension 1, by doubling spans (v and f
    are overwritten; x_{-1} = 0)."""
    span, L = 1, v.shape[1]
    while span < L:
        v[:, span:] += f[:, span:] * v[:, :-span]
        f[:, span:] *= f[:, :-span].clone()
        span *= 2
    return v


def _forward_plain(s):
    h, f, fc, i = _gates(s)
    v = i * h
    if s["x0_"] is not None:
        v[:, 0] += f[:, 0] * s["x0_"]
    x = _recur(f.clone(), v)
    y = x if s["z_"] is None else x * s["z_"].float() * torch.sigmoid(s["z_"].float())
    return h, f, fc, i, x, y


def _prefill_plain(s):
    *_, x, y = _forward_plain(s)
    return {"y": y.to(s["h"].dtype), "x_final": x[:, -1].contiguous()}


def _train_plain(s):
    dt = s["h"].dtype
    h, f, fc, i, x, y = _forward_plain(s)
    dx = s["dy"].float()
    out = {"y": y.to(dt), "x_final": x[:, -1].contiguous()}
    if s["z_"] is not None:
        z = s["z_"].float()
        sz = torch.sigmoid(z)
        out["dz"] = (dx * x * sz * (1 + z * (1 - sz))).to(dt)
        dx = dx * z * sz
    # adjoint: g_t = dx_t + f_{t+1} g_{t+1}
    fn = torch.cat([f[:, 1:], torch.zeros_like(f[:, :1])], 1).flip(1)
    g = _recur(fn, dx.flip(1)).flip(1)
    out["dx0"] = f[:, 0] * g[:, 0]
    first = torch.zeros_like(x[:, :1]) if s["x0_"] is None else s["x0_"][:, None]
    df = g * torch.cat([first, x[:, :-1]], 1)
    out["dh"] = (g * i).to(dt)
    if s["b_"] is None:
        df -= g * h
    else:
        out["db"] = (g * h * i * torch.sigmoid(-s["b_"].float())).to(dt)
    out["da"] = (df * f * fc).to(dt)
    return out


def _step_plain(s):
    h, f, _, i = _gates(s)
    x = s["state"]
    x.mul_(f).add_(i * h)
    y = x if s["z_"] is None else x * s["z_"].float() * torch.sigmoid(s["z_"].float())
    return {"y": y.to(s["h"].dtype), "state": x}


def _w4_plain(s):
    wq, K, G = s["wq"], s["n_in"], s["group"]
    O = wq.shape[0]
    nib = torch.stack([wq & 15, wq >> 4], -1).view(O, -1, 128)
    q = nib[:, :, _order(wq.device)].reshape(O, -1)[:, :K].float() - 8.0
    w = q * s["scales"].float().repeat_interleave(G, 1)[:, :K]
    y = s["x"].float() @ w.t()
    if s["bias_"] is not None:
        y += s["bias_"]
    if s["residual_"] is not None:
        y += s["residual_"].float()
    return y.to(s["x"].dtype)


def _cache_plain(s):
    x, slots, pq, ps = s["state"], s["slots_"].long(), s["pool_q"], s["pool_s"]
    scale = x.abs().amax(-1) / 127.0
    # the quotient in 64 bits: in 32 it lands on the other side of some borders
    q = torch.round(x.double() / torch.where(scale > 0, scale, 1.0).double()[..., None])
    live = slots >= 0
    pq[slots[live]] = q[live].to(torch.int8)
    ps[slots[live]] = scale[live]
    back = pq[slots].float() * ps[slots][..., None]
    return {"state": back * live[:, None, None], "scales": ps}


_RUN_OWN = {"prefill": _prefill_own, "train": _train_own, "step": _step_own, "w4": _w4_own,
            "cache": _cache_own}
_RUN_PLAIN = {"prefill": _prefill_plain, "train": _train_plain, "step": _step_plain,
              "w4": _w4_plain, "cache": _cache_plain}


# -------------------------------------------------------------------- work
def work(case):
    """Every input read once, every output written once."""
    e = 2 if case.get("dtype") == "bf16" else 4
    op = case["op"]
    if op in ("prefill", "train", "step"):
        Bt, L, d = case["Bt"], case["L"], case["d"]
        n, ins = Bt * L * d, 2 + (not case["coupled"]) + case["z"]
        if op == "step":
            return {"bytes": n * (e * (ins + 1) + 8), "flops": n * 20}
        fwd = n * e * (ins + 1) + Bt * d * 4 * (1 + case["x0"])
        if op == "prefill":
            return {"bytes": fwd, "flops": n * 20}
        # forward, then the inputs and dy again and one gradient per input
        return {"bytes": fwd + n * e * (2 * ins + 1) + Bt * d * 4, "flops": n * 60}
    if op == "w4":
        M, K, O, G = case["M"], case["n_in"], case["n_out"], case["group"]
        b = O * (K / 2 + 2 * -(-K // G)) + M * K * e + M * O * e
        return {"bytes": b + 4 * O * case["bias"] + M * O * e * case["residual"],
                "flops": 2 * M * K * O}
    n = case["n"] * case["d"]
    return {"bytes": 2 * n * (4 * case["N"] + case["N"] + 4) + 8 * case["n"],
            "flops": 6 * n * case["N"]}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """From the definitions, in 64 bits: the recurrences token by token, the
    product with the unpacked weights, the cache value by value."""
    s = prepare(case, seed)
    up = lambda t: None if t is None else t.double()  # noqa: E731
    op = case["op"]
    if op == "w4":
        K, G = case["n_in"], case["group"]
        word = s["wq"].view(torch.int32).long().view(case["n_out"], -1, 4, 4)  # [o, block, c, j]
        W = torch.empty((case["n_out"], word.shape[1], 4, 4, 8), dtype=torch.float64,
                        device=word.device)                                   # [o, block, j, c, e]
        for e in range(8):
            W[..., e] = ((word >> (4 * (e // 2 + 4 * (e % 2)))) & 15).transpose(2, 3)
        W = W.view(case["n_out"], -1)[:, :K] - 8
        W *= up(s["scales"])[:, torch.arange(K, device=W.device) // G]
        y = up(s["x"]) @ W.t()
        for t in (s["bias_"], s["residual_"]):
            y = y if t is None else y + t.double()
        return y
    if op == "cache":
        x = up(s["state"])
        scale = (x.abs().amax(-1) / 127).float().double()    # as the cache holds it
        back = torch.round(x / scale[..., None]) * scale[..., None]
        back[s["slots_"] < 0] = 0
        pool = torch.zeros_like(s["pool_s"], dtype=torch.float64)
        for k, slot in enumerate(s["slots_"].tolist()):
            if slot >= 0:
                pool[slot] = scale[k]
        return {"state": back, "scales": pool}
    step = op == "step"
    h, a, b, z = (t if t is None or not step else t[:, None]
                  for t in (up(s["h"]), up(s["a"]), up(s["b_"]), up(s["z_"])))
    f = 1 / (1 + torch.exp(-a))
    i = 1 - f if b is None else 1 / (1 + torch.exp(-b))
    x0 = up(s["state"] if step else s["x0_"])
    x0 = torch.zeros_like(f[:, 0]) if x0 is None else x0
    x = torch.empty_like(f)
    cur = x0
    for t in range(f.shape[1]):
        cur = torch.addcmul(i[:, t] * h[:, t], f[:, t], cur)
        x[:, t] = cur
    gate = torch.ones_like(x) if z is None else z / (1 + torch.exp(-z))
    y = x * gate
    if step:
        return {"y": y[:, 0], "state": cur}
    out = {"y": y, "x_final": cur}
    if op == "prefill":
        return out
    dy = up(s["dy"])
    g = torch.empty_like(f)
    back = torch.zeros_like(cur)
    for t in range(f.shape[1] - 1, -1, -1):
        torch.addcmul(back, dy[:, t], gate[:, t], out=g[:, t])
        back = f[:, t] * g[:, t]
    out["dx0"] = back
    before = torch.cat([x0[:, None], x[:, :-1]], 1)
    out["dh"] = g * i
    if b is None:
        out["da"] = g * (before - h) / (2 + torch.exp(a) + torch.exp(-a))
    else:
        out["da"] = g * before / (2 + torch.exp(a) + torch.exp(-a))
        out["db"] = g * h / (2 + torch.exp(b) + torch.exp(-b))
    if z is not None:
        sz = 1 / (1 + torch.exp(-z))
        out["dz"] = dy * x * (sz + z * sz * (1 - sz))
    return out
