"""Plain fp64 references of the RMS norm, the 8-bit input projection, the short
convolution and the selective state space scan, straight from their formulas
(include/ttt.h), token by token where there is a recurrence.  torch float64
tensors in, dicts of float64 tensors out, on the inputs' device.

Beside each result ``name`` stands ``name_mag``: the same sum with every term
replaced by its magnitude.  A computation whose terms carry relative errors of
at most eps is off by at most eps * mag, whatever cancels."""
from __future__ import annotations

import torch


def rms_norm(x, weight, residual=None, eps=1e-6):
    r = x if residual is None else x + residual
    rstd = 1.0 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    mag = x.abs() if residual is None else x.abs() + residual.abs()
    return {"y": r * rstd * weight, "y_mag": mag * rstd * weight.abs(), "r": r, "r_mag": mag}


def rms_norm_backward(r, weight, dy, dr=None, eps=1e-6):
    rstd = 1.0 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    xh, u = r * rstd, dy * weight
    mean = (u * xh).mean(-1, keepdim=True)
    dx = rstd * (u - xh * mean)
    mag = rstd * (u.abs() + xh.abs() * (u * xh).abs().mean(-1, keepdim=True))
    if dr is not None:
        dx, mag = dx + dr, mag + dr.abs()
    flat = (dy * xh).reshape(-1, r.shape[-1])
    return {"dx": dx, "dx_mag": mag, "dweight": flat.sum(0), "dweight_mag": flat.abs().sum(0)}


def input_f8(x, x_scale, w, w_scale, b_eta, heads, eta_base, d=64):
    B, T, D = x.shape
    H = heads
    xs, ws = x * x_scale[..., None], w * w_scale[:, None]
    y, mag = xs @ ws.t(), xs.abs() @ ws.abs().t()
    out = {}
    for i, name in enumerate("qkv"):
        for key, v in ((name, y), (name + "_mag", mag)):
            out[key] = v[..., i * H * d:(i + 1) * H * d].reshape(B, T, H, d).transpose(1, 2)
    gate = y[..., 3 * H * d:] + b_eta
    out["eta"] = (eta_base / (1.0 + torch.exp(-gate))).transpose(1, 2)
    out["gate_mag"] = (mag[..., 3 * H * d:] + b_eta.abs()).transpose(1, 2)
    return out


def _window(x, state0, K):
    B, H, T, d = x.shape
    first = torch.zeros((B, H, K - 1, d), dtype=x.dtype, device=x.device) \
        if state0 is None else state0
    return torch.cat([first, x], 2)


def conv(x, w, bias=None, state0=None, silu=True):
    K, T = w.shape[1], x.shape[2]
    seq = _window(x, state0, K)
    u = sum(seq[:, :, j:j + T] * w[:, None, j] for j in range(K))
    mag = sum((seq[:, :, j:j + T] * w[:, None, j]).abs() for j in range(K))
    if bias is not None:
        u, mag = u + bias[:, None], mag + bias.abs()[:, None]
    y = u * torch.sigmoid(u) if silu else u
    return {"y": y, "y_mag": mag, "state": seq[:, :, T:]}


def conv_backward(x, w, bias, dy, state0=None, dstate=None, silu=True):
    K, T = w.shape[1], x.shape[2]
    seq = _window(x, state0, K)
    u = sum(seq[:, :, j:j + T] * w[:, None, j] for j in range(K))
    umag = sum((seq[:, :, j:j + T] * w[:, None, j]).abs() for j in range(K))
    if bias is not None:
        u, umag = u + bias[:, None], umag + bias.abs()[:, None]
    du, dumag = dy, dy.abs()
    if silu:
        s = torch.sigmoid(u)
        du = dy * s * (1 + u * (1 - s))
        dumag = dy.abs() * (1 + umag)     # an error of u counts at most so much
    out = {"dbias": du.sum((0, 2)), "dbias_mag": dumag.sum((0, 2))}
    for suffix, g, ww, xx in (("", du, w, seq), ("_mag", dumag, w.abs(), seq.abs())):
        dseq = torch.zeros_like(seq)
        for j in range(K):
            dseq[:, :, j:j + T] += g * ww[:, None, j]
        if dstate is not None:
            dseq[:, :, T:] += dstate if not suffix else dstate.abs()
        out["dx" + suffix] = dseq[:, :, K - 1:]
        out["dstate0" + suffix] = dseq[:, :, :K - 1]
        out["dw" + suffix] = torch.stack(
            [(xx[:, :, j:j + T] * g).sum((0, 2)) for j in range(K)], 1)
    return out


def _spread(v, H):
    return v.repeat_interleave(H // v.shape[1], 1)


def _fades(dt, a):
    """exp(a dt) per token, and its exponent's size: an exponent in error by
    2^-24 of itself moves the decay by that times its size."""
    return torch.exp(dt * a[:, None])


def ssm(x, dt, a, b, c, d_skip=None, state0=None):
    B, H, T, P = x.shape
    N = b.shape[-1]
    b, c, fade = _spread(b, H), _spread(c, H), _fades(dt, a)
    out = {}
    for suffix, f in (("", lambda v: v), ("_mag", torch.abs)):
        S = torch.zeros((B, H, N, P), dtype=x.dtype, device=x.device) \
            if state0 is None else f(state0)
        y = torch.empty_like(x)
        for t in range(T):
            add = f(dt[:, :, t, None] * b[:, :, t])[..., None] * f(x[:, :, t])[:, :, None]
            S = S * fade[:, :, t, None, None] + add
            y[:, :, t] = (f(c[:, :, t])[..., None] * S).sum(2)
        if d_skip is not None:
            y = y + f(x * d_skip[:, None, None])
        out["y" + suffix], out["state" + suffix] = y, S
    return out


def ssm_backward(x, dt, a, b, c, dy, d_skip=None, state0=None, dstate=None, tile=64):
    """tile: tokens over which the kernels sum c.dc - b.db, for ddt_mag alone."""
    B, H, T, P = x.shape
    G, N = b.shape[1], b.shape[-1]
    b, c, fade = _spread(b, H), _spread(c, H), _fades(dt, a)
    out = {}
    for suffix, f in (("", lambda v: v), ("_mag", torch.abs)):
        S = torch.zeros((B, H, N, P), dtype=x.dtype, device=x.device) \
            if state0 is None else f(state0)
        S = S.clone()
        states = [S]
        for t in range(T):
            add = f(dt[:, :, t, None] * b[:, :, t])[..., None] * f(x[:, :, t])[:, :, None]
            S = S * fade[:, :, t, None, None] + add
            states.append(S)
        A = torch.zeros_like(S) if dstate is None else f(dstate)
        dx, ddt, e = torch.empty_like(x), torch.empty_like(dt), torch.empty_like(dt)
        db, dc = torch.empty_like(b), torch.empty_like(c)
        run = torch.zeros_like(dt[:, :, 0])
        for t in range(T - 1, -1, -1):
            if suffix and ((t + 1) % tile == 0 or t == T - 1):
                run = (states[t + 1] * A).sum((2, 3))      # behind the tile
            dc[:, :, t] = (states[t + 1] * f(dy[:, :, t])[:, :, None]).sum(3)
            A = A + f(c[:, :, t])[..., None] * f(dy[:, :, t])[:, :, None]
            ax = (A * f(x[:, :, t])[:, :, None]).sum(3)
            db[:, :, t] = ax * f(dt[:, :, t])[..., None]
            dx[:, :, t] = (A * f(b[:, :, t])[..., None]).sum(2) * f(dt[:, :, t])[..., None]
            direct = (ax * f(b[:, :, t])).sum(2)
            if suffix:
                run = run + (f(c[:, :, t]) * dc[:, :, t]).sum(2) + f(dt[:, :, t]) * direct
                e[:, :, t] = run
            else:
                e[:, :, t] = (A * states[t]).sum((2, 3)) * fade[:, :, t]
            ddt[:, :, t] = direct + f(a) * e[:, :, t]
            A = A * fade[:, :, t, None, None]
        if d_skip is not None:
            dx = dx + f(dy) * f(d_skip)[:, None, None]
            out["dd" + suffix] = (f(dy) * f(x)).sum((0, 2, 3))
        out["dx" + suffix], out["ddt" + suffix] = dx, ddt
        out["da" + suffix] = (f(dt) * e).sum((0, 2))
        out["dstate0" + suffix] = A
        for name, v in (("db", db), ("dc", dc)):
            out[name + suffix] = v.view(B, G, H // G, T, N).sum(2)
    return out
