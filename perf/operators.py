"""Cases of the layer's norm, 8-bit input projection, short convolution and
selective state space scan: inputs, the operators in plain torch, the
framework's calls, the work of one pass and 64-bit results.

``own`` picks what ``run`` does: False computes the operators from elementary
torch operations in fp32, True makes the framework's calls."""
import math

import torch

own = False

HD = 64        # head dimension of the framework's layers
E4M3_MAX = 448.0


def listed():
    return [
        # the pre-norm of a 1.3B-wide layer over a training batch: residual stream in and out
        dict(name="norm_prompt", op="norm", rows=4 * 8192, width=2048, dtype="bf16", residual=True),
        # the same norm in front of the 8-bit projection, one token of 256 streams
        dict(name="norm_f8_step", op="norm_f8", rows=256, width=2048, dtype="bf16", residual=True),
        # training, 125M-wide layer: the norm's backward
        dict(name="norm_backward", op="norm_bwd", rows=8 * 2048, width=768, dtype="bf16", residual=True),
        # q, k, v and the gate of a 1.3B layer's prompt from 8-bit activations and weights
        dict(name="proj_f8_prompt", op="proj_f8", batch=4, length=8192, width=2048, heads=32),
        # the same for one token of 61 streams of a 125M layer
        dict(name="proj_f8_step", op="proj_f8", batch=61, length=1, width=768, heads=12),
        # the short convolution over q, k or v of a 1.3B layer's prompt, keeping the state for decoding
        dict(name="conv_prompt", op="conv", batch=4, heads=32, length=8192, dim=64, taps=4,
             dtype="bf16", silu=True, state=False),
        # one token of 256 streams
        dict(name="conv_step", op="conv_step", batch=256, heads=32, dim=64, taps=4, dtype="bf16",
             silu=True),
        # training, 125M layer
        dict(name="conv_backward", op="conv_bwd", batch=8, heads=12, length=2048, dim=64, taps=4,
             dtype="bf16", silu=True),
        # the scan over a 1.3B layer's prompt, every head its own b and c
        dict(name="ssm_prompt", op="ssm", batch=4, heads=32, groups=32, length=8192, n=64,
             dtype="bf16", skip=True, state=False),
        # fp32 data, few streams, an odd length, heads sharing b and c, a prompt's continuation
        dict(name="ssm_fp32_odd", op="ssm", batch=1, heads=6, groups=2, length=1003, n=128,
             dtype="f32", skip=True, state=True),
        # one token of 256 streams
        dict(name="ssm_step", op="ssm_step", batch=256, heads=32, groups=32, n=64, dtype="bf16",
             skip=True),
        # training, 125M layer
        dict(name="ssm_backward", op="ssm_bwd", batch=8, heads=12, groups=12, length=2048, n=64,
             dtype="bf16", skip=True, state=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_f8", "norm_bwd", "proj_f8", "conv", "conv_step", "conv_bwd",
                     "ssm", "ssm", "ssm_step", "ssm_bwd", "ssm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        width = 8 * _log(rng, 8, 1024)
        rows = _log(rng, 1, min(32768, (1 << 26) // width))
        return dict(op=op, rows=rows, width=width, dtype=dtype, residual=rng.random() < 0.7)
    if op == "proj_f8":
        heads, width = _log(rng, 1, 32), 64 * _log(rng, 1, 32)
        batch = _log(rng, 1, 64)
        return dict(op=op, batch=batch, length=_log(rng, 1, 16384 // batch), width=width,
                    heads=heads)
    taps = rng.choice([2, 3, 4])
    if op == "conv_step":
        return dict(op=op, batch=_log(rng, 1, 256), heads=_log(rng, 1, 32),
                    dim=rng.choice([32, 64, 128]), taps=taps, dtype=dtype, silu=rng.random() < 0.7)
    n = rng.choice([32, 64, 128])
    groups, share = rng.choice([(1, 8), (2, 3), (4, 1), (12, 1), (3, 5), (1, 1), (8, 4)])
    if op == "ssm_step":
        return dict(op=op, batch=_log(rng, 1, 200), heads=groups * share, groups=groups, n=n,
                    dtype=dtype, skip=rng.random() < 0.5)
    batch = _log(rng, 1, 8)
    most = {"ssm": 1 << 18, "ssm_bwd": 1 << 17}.get(op, 1 << 19)
    if dtype == "f32" or n == 128:
        most //= 2
    length = _log(rng, 1, min(16384, most // (batch * groups * share)))
    if op.startswith("conv"):
        return dict(op=op, batch=batch, heads=groups * share, length=length,
                    dim=rng.choice([32, 64, 128]), taps=taps, dtype=dtype, silu=rng.random() < 0.7,
                    **({"state": rng.random() < 0.5} if op == "conv" else {}))
    return dict(op=op, batch=batch, heads=groups * share, groups=groups, length=length, n=n,
                dtype=dtype, skip=rng.random() < 0.5, state=rng.random() < 0.5)


def _dtype(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, shift=0.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev).mul_(scale).add_(shift).to(dtype)

    op, dt_ = case["op"], _dtype(case)
    s = {"case": case}
    if op.startswith("norm"):
        shape = (case["rows"], case["width"])
        s["x"] = normal(*shape, dtype=dt_)
        s["weight"] = normal(case["width"], scale=0.1, shift=1.0)
        if op == "norm_bwd":
            s["dy"] = normal(*shape, dtype=dt_)
            s["dr"] = normal(*shape, dtype=dt_) if case["residual"] else None
        else:
            # a residual stream is wider than one layer's output
            s["residual"] = normal(*shape, scale=3.0, dtype=dt_) if case["residual"] else None
        return s
    if op == "proj_f8":
        B, T, D, H = case["batch"], case["length"], case["width"], case["heads"]
        x = normal(B, T, D)
        s["x_scale"] = x.abs().amax(-1) / E4M3_MAX
        s["x"] = (x / s["x_scale"][..., None]).to(torch.float8_e4m3fn)
        w = torch.cat([normal(3 * H * HD, D, scale=1 / math.sqrt(D * HD)),
                       normal(H, D, scale=1 / math.sqrt(D))])
        s["w_scale"] = w.abs().amax(-1) / E4M3_MAX
        s["w"] = (w / s["w_scale"][:, None]).to(torch.float8_e4m3fn)
        s["b_eta"] = normal(H, scale=0.1)
        return s
    if op.startswith("conv"):
        B, H, d, K = case["batch"], case["heads"], case["dim"], case["taps"]
        shape = (B, H, d) if op == "conv_step" else (B, H, case["length"], d)
        s["x"] = normal(*shape, dtype=dt_)
        s["w"] = normal(H, K, d, scale=1 / math.sqrt(K))
        s["bias"] = normal(H, d, scale=0.1)
        if op == "conv_step" or case.get("state"):
            s["state"] = normal(B, H, K - 1, d, dtype=dt_)
        if op == "conv_bwd":
            s["dy"] = normal(*shape, dtype=dt_)
        return s
    B, H, G, N = case["batch"], case["heads"], case["groups"], case["n"]
    t = () if op == "ssm_step" else (case["length"],)
    s["x"] = normal(B, H, *t, HD, dtype=dt_)
    s["b"] = normal(B, G, *t, N, scale=N ** -0.25, dtype=dt_)
    s["c"] = normal(B, G, *t, N, scale=N ** -0.25, dtype=dt_)
    # steps between 1e-3 and 1e-1, decay rates between 1 and 16 per unit of step
    s["dt"] = torch.exp(torch.rand((B, H, *t), generator=g, device=dev) * math.log(100.0)
                        + math.log(1e-3))
    s["a"] = -(1.0 + 15.0 * torch.rand((H,), generator=g, device=dev))
    s["d_skip"] = normal(H, scale=0.1, shift=1.0) if case["skip"] else None
    if op == "ssm_step" or case["state"]:
        s["state"] = normal(B, H, N, HD, scale=0.1)
    if op == "ssm_bwd":
        s["dy"] = normal(*s["x"].shape, dtype=dt_)
        s["dstate"] = normal(B, H, N, HD, scale=0.1) if case["state"] else None
    return s


# ---- the framework's calls --------------------------------------------------

def _run_own(s):
    import linear_rnn_ttt_amd as fw
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return fw.ttt_rms_norm_forward(s["x"], s["weight"], s["residual"])
    if op == "norm_f8":
        return fw.ttt_rms_norm_forward_f8(s["x"], s["weight"], s["residual"])
    if op == "norm_bwd":
        return fw.ttt_rms_norm_backward(s["x"], s["weight"], s["dy"], s["dr"])
    if op == "proj_f8":
        return fw.ttt_input_projection_f8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["b_eta"],
                                          heads=case["heads"], eta_base=1 / HD)
    if op == "conv":
        return fw.ttt_conv_forward(s["x"], s["w"], s["bias"], state0=s.get("state"),
                                   silu=case["silu"], return_state=True)
    if op == "conv_step":
        y = fw.ttt_conv_decode_step(s["x"], s["w"], s["bias"], s["state"], silu=case["silu"])
        return y, s["state"]     # moved on in place
    if op == "conv_bwd":
        return fw.ttt_conv_backward(s["x"], s["w"], s["bias"], s["dy"], silu=case["silu"])[:3]
    if op == "ssm":
        return fw.ttt_ssm_forward(s["x"], s["dt"], s["a"], s["b"], s["c"], s["d_skip"],
                                  state0=s.get("state"))
    if op == "ssm_step":
        y = fw.ttt_ssm_decode_step(s["x"], s["dt"], s["a"], s["b"], s["c"], s["state"],
                                   s["d_skip"])
        return y, s["state"]     # moved on in place
    return fw.ttt_ssm_backward(s["x"], s["dt"], s["a"], s["b"], s["c"], s["dy"], s["d_skip"],
                               state0=s.get("state"), dstate=s["dstate"])


# ---- plain torch ------------------------------------------------------------

def _plain_norm(s):
    f8 = s["case"]["op"] == "norm_f8"
    x = s["x"].float()
    r = x if s["residual"] is None else x + s["residual"].float()
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + 1e-6) * s["weight"]
    kept = None if s["residual"] is None else r.to(s["x"].dtype)
    if not f8:
        return y.to(s["x"].dtype), kept
    scale = y.abs().amax(-1) / E4M3_MAX
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (y / scale[:, None]).to(torch.float8_e4m3fn), scale, kept


def _plain_norm_bwd(s):
    r, dy, w = s["x"].float(), s["dy"].float(), s["weight"]
    rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + 1e-6)
    xh = r * rstd
    u = dy * w
    dr = rstd * (u - xh * (u * xh).mean(-1, keepdim=True))
    if s["dr"] is not None:
        dr = dr + s["dr"].float()
    return dr.to(s["x"].dtype), (dy * xh).sum(0)


def _plain_proj(s):
    H = s["case"]["heads"]
    x = s["x"].float()
    B, T, D = x.shape
    y = x.view(B * T, D) @ s["w"].float().t()
    y = (y * s["x_scale"].view(-1, 1) * s["w_scale"]).view(B, T, -1)
    qkv = [y[..., i * H * HD:(i + 1) * H * HD].reshape(B, T, H, HD).transpose(1, 2)
           .contiguous().to(torch.bfloat16) for i in range(3)]
    gate = y[..., 3 * H * HD:] + s["b_eta"]
    eta = (1 / HD) / (1 + torch.exp(-gate))
    return (*qkv, eta.transpose(1, 2).contiguous())


def _taps(xp, w, T):
    """bias-free convolution of the padded fp32 xp [B,H,T+K-1,d] with w [H,K,d]."""
    K = w.shape[1]
    if K == 2:
        return xp[:, :, :T] * w[:, None, 0] + xp[:, :, 1:T + 1] * w[:, None, 1]
    y = (xp[:, :, :T] * w[:, None, 0] + xp[:, :, 1:T + 1] * w[:, None, 1]
         + xp[:, :, 2:T + 2] * w[:, None, 2])
    return y if K == 3 else y + xp[:, :, 3:T + 3] * w[:, None, 3]


def _padded(s):
    x = s["x"].float()
    if x.dim() == 3:
        x = x[:, :, None]
    K = s["w"].shape[1]
    first = s.get("state")
    first = (torch.zeros(x.shape[:2] + (K - 1, x.shape[3]), device=x.device) if first is None
             else first.float())
    return torch.cat([first, x], 2), x.shape[2]


def _plain_conv(s):
    xp, T = _padded(s)
    y = _taps(xp, s["w"], T) + s["bias"][:, None]
    if s["case"]["silu"]:
        y = y / (1 + torch.exp(-y))
    y = y.to(s["x"].dtype).view(s["x"].shape)
    last = xp[:, :, T:].to(s["x"].dtype)
    if s["case"]["op"] == "conv_step":   # the stream's state moves on in place
        return y, s["state"].copy_(last)
    return y, last.contiguous()


def _plain_conv_bwd(s):
    xp, T = _padded(s)
    w = s["w"]
    K = w.shape[1]
    du = s["dy"].float()
    if s["case"]["silu"]:
        u = _taps(xp, w, T) + s["bias"][:, None]
        sig = 1 / (1 + torch.exp(-u))
        du = du * sig * (1 + u * (1 - sig))
    dup = torch.nn.functional.pad(du, (0, 0, 0, K - 1))
    dx = _taps(dup, w.flip(1), T)
    dw = torch.stack([(du * xp[:, :, j:j + T]).sum((0, 2)) for j in range(K)], 1)
    return dx.to(s["x"].dtype), dw, du.sum((0, 2))


def _ssm_pieces(x, dt, a, b, c, S0, L=64):
    """y without the skip and the final state, in fp32 (decays from fp64 sums),
    by tiles of L tokens: products inside a tile, and the state between them."""
    B, H, T, _ = x.shape
    G, N = b.shape[1], b.shape[3]
    nc = -(-T // L)
    pad = nc * L - T

    def tiles(v):
        v = torch.nn.functional.pad(v, (0, 0, 0, pad))
        return v.reshape(v.shape[0], v.shape[1], nc, L, v.shape[3])

    xt = tiles(x)
    bt, ct = tiles(b), tiles(c)
    bt = bt[:, :, None].expand(B, G, H // G, nc, L, N).reshape(B, H, nc, L, N)
    ct = ct[:, :, None].expand(B, G, H // G, nc, L, N).reshape(B, H, nc, L, N)
    dtt = tiles(dt[..., None])[..., 0]
    cum = torch.cumsum(dtt.double() * a.double()[:, None, None], -1)        # [B,H,nc,L]
    low = torch.ones(L, L, device=x.device, dtype=torch.bool).tril()
    gap = (cum[..., :, None] - cum[..., None, :]).masked_fill(~low, -math.inf)
    M = torch.matmul(ct, bt.transpose(-1, -2)) * torch.exp(gap).float() * dtt[..., None, :]
    y = torch.matmul(M, xt)
    left = torch.exp(cum[..., -1:] - cum).float() * dtt                     # to the tile's end
    added = torch.matmul((bt * left[..., None]).transpose(-1, -2), xt)      # [B,H,nc,N,P]
    # state before each tile (and after the last): a triangular product over tiles
    whole = torch.nn.functional.pad(torch.cumsum(cum[..., -1], -1), (1, 0))  # [B,H,nc+1]
    lowc = torch.ones(nc + 1, nc + 1, device=x.device, dtype=torch.bool).tril()
    span = (whole[..., :, None] - whole[..., None, :]).masked_fill(~lowc, -math.inf)
    first = torch.zeros_like(added[:, :, :1]) if S0 is None else S0[:, :, None]
    into = torch.cat([first, added], 2).flatten(3)
    S = torch.matmul(torch.exp(span).float(), into).view(B, H, nc + 1, N, -1)
    y = y + torch.matmul(ct, S[:, :, :-1]) * torch.exp(cum).float()[..., None]
    return y.reshape(B, H, nc * L, -1)[:, :, :T], S[:, :, -1]


def _plain_ssm(s):
    x = s["x"].float()
    y, S = _ssm_pieces(x, s["dt"], s["a"], s["b"].float(), s["c"].float(), s.get("state"))
    if s["d_skip"] is not None:
        y = y + x * s["d_skip"][:, None, None]
    return y.to(s["x"].dtype), S.contiguous()


def _plain_ssm_step(s):
    x, b, c = s["x"].float(), s["b"].float(), s["c"].float()
    H, G = x.shape[1], b.shape[1]
    b, c = b.repeat_interleave(H // G, 1), c.repeat_interleave(H // G, 1)
    S = s["state"]                       # the stream's state moves on in place
    S.mul_(torch.exp(s["dt"] * s["a"])[..., None, None])
    S.add_((s["dt"][..., None] * b)[..., None] * x[:, :, None])
    y = (c[..., None] * S).sum(2)
    if s["d_skip"] is not None:
        y = y + x * s["d_skip"][:, None]
    return y.to(s["x"].dtype), S


def _plain_ssm_bwd(s):
    names = ["x", "dt", "a", "b", "c"]
    leaves = [s[k].float().detach().requires_grad_() for k in names]
    extra = [s[k].detach().requires_grad_() if s.get(k) is not None else None
             for k in ("d_skip", "state")]
    with torch.enable_grad():
        y, S = _ssm_pieces(*leaves, extra[1])
        if extra[0] is not None:
            y = y + leaves[0] * extra[0][:, None, None]
        outs, cots = [y], [s["dy"].float()]
        if s["dstate"] is not None:
            outs, cots = outs + [S], cots + [s["dstate"]]
        wanted = leaves + [e for e in extra if e is not None]
        grads = list(torch.autograd.grad(outs, wanted, cots))
    found = [g.to(s[k].dtype) for g, k in zip(grads, names)]
    rest = iter(grads[5:])
    return (*found, *(next(rest) if e is not None else None for e in extra))


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op in ("norm", "norm_f8"):
        return _plain_norm(state)
    if op == "norm_bwd":
        return _plain_norm_bwd(state)
    if op == "proj_f8":
        return _plain_proj(state)
    if op in ("conv", "conv_step"):
        return _plain_conv(state)
    if op == "conv_bwd":
        return _plain_conv_bwd(state)
    if op == "ssm":
        return _plain_ssm(state)
    if op == "ssm_step":
        return _plain_ssm_step(state)
    return _plain_ssm_bwd(state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    es = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if op.startswith("norm"):
        n = case["rows"] * case["width"]
        if op == "norm_bwd":     # r, dy [, dr] in, dr out
            return {"bytes": n * es * (4 if case["residual"] else 3) + case["width"] * 8,
                    "flops": 9 * n}
        moved = n * es * (3 if case["residual"] else 1)
        moved += n + 4 * case["rows"] if op == "norm_f8" else n * es
        return {"bytes": moved + case["width"] * 4, "flops": 5 * n}
    if op == "proj_f8":
        M, D, H = case["batch"] * case["length"], case["width"], case["heads"]
        cols = 3 * H * HD + H
        return {"bytes": M * D + 4 * M + cols * (D + 4) + M * H * (3 * HD * 2 + 4),
                "flops": 2.0 * M * D * cols}
    B, H = case["batch"], case["heads"]
    if op.startswith("conv"):
        d, K, T = case["dim"], case["taps"], case.get("length", 1)
        n = B * H * T * d
        tails = B * H * (K - 1) * d * es
        if op == "conv_bwd":
            return {"bytes": 3 * n * es + 8 * H * (K + 1) * d, "flops": n * (6 * K + 10)}
        known = 2 if op == "conv_step" or case["state"] else 1
        return {"bytes": 2 * n * es + known * tails + 4 * H * (K + 1) * d,
                "flops": n * (2 * K + 6)}
    G, N, T = case["groups"], case["n"], case.get("length", 1)
    heads, shared, states = B * H * T, B * G * T * N * es, B * H * N * HD * 4
    if op == "ssm_step":
        return {"bytes": 2 * heads * HD * es + 2 * shared + 4 * heads + 2 * states,
                "flops": heads * N * HD * 5.0}
    # the recurrence itself, two operations each for its decay-and-add, its input and its output
    if op == "ssm":
        return {"bytes": 2 * heads * HD * es + 2 * shared + 4 * heads
                + states * (2 if case["state"] else 1), "flops": heads * N * HD * 6.0}
    return {"bytes": 3 * heads * HD * es + 4 * shared + 8 * heads
            + (3 * states if case["state"] else 0), "flops": heads * N * HD * 16.0}


# ---- 64 bits ----------------------------------------------------------------

def _exact_ssm(s, backward):
    """The recurrence, token by token."""
    x, dt, a, b, c = (s[k].double() for k in ("x", "dt", "a", "b", "c"))
    B, H, T, P = x.shape
    G, N = b.shape[1], b.shape[3]
    if T * B * H * N * P * 8 > (40e9 if backward else 1e14) or T > 20000:
        return None
    skip = None if s["d_skip"] is None else s["d_skip"].double()
    share = H // G
    S = (torch.zeros((B, H, N, P), dtype=torch.float64, device=x.device)
         if s.get("state") is None else s["state"].double())
    fade = torch.exp(dt * a[:, None])
    kept = [S]
    y = torch.empty_like(x)
    for t in range(T):
        bt = b[:, :, t].repeat_interleave(share, 1)
        ct = c[:, :, t].repeat_interleave(share, 1)
        S = S * fade[:, :, t, None, None] + (bt * dt[:, :, t, None])[..., None] * x[:, :, t, None]
        y[:, :, t] = (ct[..., None] * S).sum(2)
        if backward:
            kept.append(S)
    if not backward:
        return (y if skip is None else y + x * skip[:, None, None]), S
    dy = s["dy"].double()
    adj = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()
    dx, ddt = torch.empty_like(x), torch.empty_like(dt)
    db, dc = torch.zeros_like(b), torch.zeros_like(c)
    da = torch.zeros_like(dt)
    for t in range(T - 1, -1, -1):
        bt = b[:, :, t].repeat_interleave(share, 1)
        ct = c[:, :, t].repeat_interleave(share, 1)
        dc[:, :, t] = (kept[t + 1] * dy[:, :, t, None]).sum(3).view(B, G, share, N).sum(2)
        adj = adj + ct[..., None] * dy[:, :, t, None]
        adx = (adj * x[:, :, t, None]).sum(3)                       # [B,H,N]
        db[:, :, t] = (adx * dt[:, :, t, None]).view(B, G, share, N).sum(2)
        dx[:, :, t] = (adj * bt[..., None]).sum(2) * dt[:, :, t, None]
        through = (adj * kept[t]).sum((2, 3)) * fade[:, :, t]       # d of a dt
        ddt[:, :, t] = (adx * bt).sum(2) + through * a
        da[:, :, t] = through * dt[:, :, t]
        adj = adj * fade[:, :, t, None, None]
    dskip = None
    if skip is not None:
        dx = dx + dy * skip[:, None, None]
        dskip = (dy * x).sum((0, 2, 3))
    return dx, ddt, da.sum((0, 2)), db, dc, dskip, (None if s.get("state") is None else adj)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("ssm", "ssm_bwd"):
        return _exact_ssm(s, op == "ssm_bwd")
    x = s["x"].double()
    if op.startswith("norm"):
        w = s["weight"].double()
        r = x if s.get("residual") is None else x + s["residual"].double()
        length = torch.sqrt(r.square().sum(-1, keepdim=True) / case["width"] + 1e-6)
        if op == "norm_bwd":
            dy = s["dy"].double()
            lead = dy * w / length
            dr = lead - r * (lead * r).sum(-1, keepdim=True) / (case["width"] * length.square())
            return (dr if s["dr"] is None else dr + s["dr"].double()), (dy * r / length).sum(0)
        y = r / length * w
        kept = None if s["residual"] is None else r
        if op == "norm":
            return y, kept
        top = y.abs().amax(-1) / E4M3_MAX
        return y / top[:, None], top, kept
    if op == "proj_f8":
        H, (B, T, D) = case["heads"], x.shape
        xs, ws = s["x_scale"].double(), s["w_scale"].double()
        y = torch.matmul(x * xs[..., None], (s["w"].double() * ws[:, None]).t())
        heads = y[..., :3 * H * HD].reshape(B, T, 3, H, HD).permute(2, 0, 3, 1, 4)
        eta = torch.sigmoid(y[..., 3 * H * HD:] + s["b_eta"].double()).permute(0, 2, 1) / HD
        return heads[0], heads[1], heads[2], eta
    if op.startswith("conv"):
        B, H, K, d = x.shape[0], case["heads"], case["taps"], case["dim"]
        x = x.view(B, H, -1, d)
        T = x.shape[2]
        w, bias = s["w"].double(), s["bias"].double()
        old = s.get("state")
        old = x.new_zeros(B, H, K - 1, d) if old is None else old.double()
        seq = torch.cat([old, x], 2)
        u = torch.einsum("bhtdk,hkd->bhtd", seq.unfold(2, K, 1), w) + bias[:, None]
        if op != "conv_bwd":
            y = u * torch.sigmoid(u) if case["silu"] else u
            return y.view(s["x"].shape), seq[:, :, T:]
        du = s["dy"].double()
        if case["silu"]:
            sg = torch.sigmoid(u)
            du = du * (sg + u * sg * (1 - sg))
        dseq = torch.zeros_like(seq)
        for j in range(K):
            dseq[:, :, j:j + T] += du * w[:, None, j]
        dw = torch.stack([(seq[:, :, j:j + T] * du).sum((0, 2)) for j in range(K)], 1)
        return dseq[:, :, K - 1:], dw, du.sum((0, 2))
    # one step of the scan
    share = case["heads"] // case["groups"]
    b = s["b"].double().repeat_interleave(share, 1)
    c = s["c"].double().repeat_interleave(share, 1)
    dt = s["dt"].double()
    S = (s["state"].double() * torch.exp(dt * s["a"].double())[..., None, None]
         + torch.einsum("bhn,bhp->bhnp", b * dt[..., None], x))
    y = torch.einsum("bhn,bhnp->bhp", c, S)
    return (y if s["d_skip"] is None else y + x * s["d_skip"].double()[:, None]), S
