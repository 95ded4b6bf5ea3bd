"""The fp64 references of oracle/block.py against torch's own functions, against
autograd and against central differences (CPU)."""
import pytest
import torch

from oracle import block


def rnd(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=g, dtype=torch.float64) * scale


def close(a, b, tol=1e-11):
    assert a.shape == b.shape
    assert float((a - b).abs().max()) <= tol * max(1.0, float(b.abs().max()))


def directional(loss, args, grads, seed):
    """(difference of the loss along one random direction, the gradients' value for it)."""
    h, want, plus, minus = 1e-6, 0.0, [], []
    for i, (v, g) in enumerate(zip(args, grads)):
        d = rnd(*v.shape, seed=seed + i)
        plus.append(v + h * d)
        minus.append(v - h * d)
        want = want + float((d * g).sum())
    return float(loss(*plus) - loss(*minus)) / (2 * h), want


@pytest.mark.parametrize("rows,width,res", [(1, 8, True), (5, 24, False)])
def test_norm(rows, width, res):
    x, w, dy = rnd(rows, width), 1 + 0.1 * rnd(width), rnd(rows, width, seed=3)
    r = rnd(rows, width, seed=1) if res else None
    got = block.rms_norm(x, w, r)
    full = x + r if res else x
    close(got["y"], torch.nn.functional.rms_norm(full, (width,), w, 1e-6))
    dr = rnd(rows, width, seed=4)
    g = block.rms_norm_backward(full, w, dy, dr)
    diff, want = directional(
        lambda v, u: (block.rms_norm(v, u)["y"] * dy).sum() + (v * dr).sum(), (full, w),
        (g["dx"], g["dweight"]), 7)
    assert abs(diff - want) <= 1e-7 * max(1.0, abs(want))


@pytest.mark.parametrize("T,K,silu,state", [(1, 4, True, True), (2, 4, True, True),
                                            (9, 3, False, False), (7, 2, True, False)])
def test_conv(T, K, silu, state):
    B, H, d = 2, 3, 8
    x, w, bias, dy = rnd(B, H, T, d), rnd(H, K, d), rnd(H, d), rnd(B, H, T, d, seed=5)
    s0 = rnd(B, H, K - 1, d, seed=2) if state else None
    ds = rnd(B, H, K - 1, d, seed=9)
    got = block.conv(x, w, bias, s0, silu)
    pad = torch.zeros(B, H, K - 1, d, dtype=torch.float64) if s0 is None else s0
    flat = torch.cat([pad, x], 2).permute(0, 1, 3, 2).reshape(B, H * d, T + K - 1)
    u = torch.nn.functional.conv1d(flat, w.permute(0, 2, 1).reshape(H * d, 1, K),
                                   bias.reshape(-1), groups=H * d)
    u = torch.nn.functional.silu(u) if silu else u
    close(got["y"], u.view(B, H, d, T).permute(0, 1, 3, 2))
    g = block.conv_backward(x, w, bias, dy, s0, ds, silu)

    def loss(x, w, bias, s0):
        o = block.conv(x, w, bias, s0, silu)
        return (o["y"] * dy).sum() + (o["state"] * ds).sum()
    diff, want = directional(loss, (x, w, bias, pad),
                             [g[k] for k in ("dx", "dw", "dbias", "dstate0")], 3)
    assert abs(diff - want) <= 1e-6 * max(1.0, abs(want))


@pytest.mark.parametrize("B,H,G,T,N", [(1, 1, 1, 1, 4), (2, 4, 2, 5, 3), (1, 3, 3, 9, 8)])
def test_ssm(B, H, G, T, N):
    P = 6
    x, b, c = rnd(B, H, T, P), rnd(B, G, T, N, seed=1), rnd(B, G, T, N, seed=2)
    dt, a = rnd(B, H, T, seed=3).abs() * 0.3, -rnd(H, seed=4).abs() - 0.2
    dsk, s0, dy = rnd(H, seed=5), rnd(B, H, N, P, seed=6), rnd(B, H, T, P, seed=7)
    dS = rnd(B, H, N, P, seed=8)
    out = block.ssm(x, dt, a, b, c, dsk, s0)
    # the sum that the recurrence stands for
    for h in range(H):
        cum = torch.cumsum(dt[:, h] * a[h], -1)
        g = h // (H // G)
        y = x[:, h] * dsk[h] + torch.exp(cum)[..., None] * (c[:, g] @ s0[:, h])
        for t in range(T):
            for s in range(t + 1):
                w = (c[:, g, t] * b[:, g, s]).sum(-1) * torch.exp(cum[:, t] - cum[:, s])
                y[:, t] += (w * dt[:, h, s])[:, None] * x[:, h, s]
        close(out["y"][:, h], y)
    grads = block.ssm_backward(x, dt, a, b, c, dy, dsk, s0, dS)

    def loss(x, dt, a, b, c, dsk, s0):
        o = block.ssm(x, dt, a, b, c, dsk, s0)
        return (o["y"] * dy).sum() + (o["state"] * dS).sum()
    keys = ("dx", "ddt", "da", "db", "dc", "dd", "dstate0")
    diff, want = directional(loss, (x, dt, a, b, c, dsk, s0), [grads[k] for k in keys], 11)
    assert abs(diff - want) <= 1e-6 * max(1.0, abs(want))
    leaves = [v.clone().requires_grad_() for v in (x, dt, a, b, c, dsk, s0)]
    S, ys = leaves[6], []
    for t in range(T):
        bt = leaves[3][:, :, t].repeat_interleave(H // G, 1)
        ct = leaves[4][:, :, t].repeat_interleave(H // G, 1)
        S = S * torch.exp(leaves[1][:, :, t] * leaves[2])[..., None, None] + \
            (leaves[1][:, :, t, None] * bt)[..., None] * leaves[0][:, :, t, None]
        ys.append((ct[..., None] * S).sum(2) + leaves[0][:, :, t] * leaves[5][:, None])
    auto = torch.autograd.grad([torch.stack(ys, 2), S], leaves, [dy, dS])
    for k, v in zip(keys, auto):
        close(grads[k], v, 1e-10)
    for k in keys:   # magnitudes bound their values
        assert bool((grads[k].abs() <= grads[k + "_mag"] * (1 + 1e-9) + 1e-12).all()), k


def test_input_f8():
    B, T, D, H = 2, 3, 16, 2
    x, w = rnd(B, T, D), rnd(3 * H * 4 + H, D, seed=1)
    xs, ws, be = rnd(B, T, seed=2).abs(), rnd(3 * H * 4 + H, seed=3).abs(), rnd(H, seed=4)
    out = block.input_f8(x, xs, w, ws, be, H, 0.25, d=4)
    y = torch.einsum("btj,nj->btn", x * xs[..., None], w * ws[:, None])
    close(out["k"][1, 1, 2], y[1, 2, H * 4 + 4:H * 4 + 8])
    close(out["eta"][0, 1, 1], 0.25 * torch.sigmoid(y[0, 1, 3 * H * 4 + 1] + be[1]))
