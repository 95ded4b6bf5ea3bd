"""The block's calls together and at their edges, on the GPU: a training step's
gradients through norm, convolution and scan; refusals that need a GPU tensor;
what a NaN reaches; large decays and steps."""
import pytest
import torch

import linear_rnn_ttt_amd as fw
from oracle import block

from _block import d64, held, rnd

pytestmark = pytest.mark.gpu


def test_training_step_gradients_reach_the_residual_stream():
    """fp32 data: residual stream -> norm -> a projection (torch) -> convolutions
    -> scan -> loss, and back through each backward, against autograd of the
    same step in fp64.  Each call is within 2^-15 of its sums of magnitudes,
    which for these normal inputs stay below 16 times the values: for four
    calls 4 * 16 * 2^-15 = 2^-9 of a gradient's largest value."""
    B, T, D, H, K = 2, 90, 128, 2, 4
    x, res = rnd(B, T, D, seed=1), rnd(B, T, D, seed=2, scale=2.0)
    weight = rnd(D, seed=3, scale=0.1, shift=1.0)
    W = rnd(3 * H * 64, D, seed=4, scale=D ** -0.5)
    taps = [rnd(H, K, 64, seed=5 + i, scale=0.5) for i in range(3)]
    bias = [rnd(H, 64, seed=8 + i, scale=0.1) for i in range(3)]
    dt = torch.exp(rnd(B, H, T, seed=11) - 3)
    a, skip = -torch.exp(rnd(H, seed=12)), rnd(H, seed=13)
    dy, dr = rnd(B, H, T, 64, seed=14), rnd(B, T, D, seed=15)

    y, r = fw.ttt_rms_norm_forward(x, weight, res)
    heads = (y.view(B * T, D) @ W.t()).view(B, T, 3, H, 64).permute(2, 0, 3, 1, 4).contiguous()
    u = [fw.ttt_conv_forward(h, w, b)[0] for h, w, b in zip(heads, taps, bias)]
    z, _ = fw.ttt_ssm_forward(u[2], dt, a, u[1], u[0], skip, return_state=False)
    dx, ddt, da, db, dc, dd, _ = fw.ttt_ssm_backward(u[2], dt, a, u[1], u[0], dy, skip)
    back = [fw.ttt_conv_backward(h, w, b, g) for h, w, b, g in zip(heads, taps, bias, (dc, db, dx))]
    dheads = torch.stack([b[0] for b in back]).permute(1, 3, 0, 2, 4).reshape(B * T, -1)
    dnorm = (dheads @ W).view(B, T, D)
    dres, dweight = fw.ttt_rms_norm_backward(r, weight, dnorm, dr)

    lx, lr, lw, la, ls, ldt, lW = (t.double().requires_grad_()
                                   for t in (x, res, weight, a, skip, dt, W))
    lt = [t.double().requires_grad_() for t in taps]
    s = lx + lr
    n = s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-6) * lw
    h = (n.view(B * T, D) @ lW.t()).view(B, T, 3, H, 64).permute(2, 0, 3, 1, 4)
    v = [block.conv(h[i], lt[i], bias[i].double())["y"] for i in range(3)]
    S, ys = torch.zeros(B, H, 64, 64, dtype=torch.float64, device="cuda"), []
    for t in range(T):
        S = S * torch.exp(ldt[:, :, t] * la)[..., None, None] + \
            (ldt[:, :, t, None] * v[1][:, :, t])[..., None] * v[2][:, :, t, None]
        ys.append((v[0][:, :, t, :, None] * S).sum(2) + v[2][:, :, t] * ls[:, None])
    loss = (torch.stack(ys, 2) * dy).sum() + (s * dr).sum()
    want = torch.autograd.grad(loss, [lx, lr, lw, la, ls, ldt, *lt])
    got = [dres, dres, dweight, da, dd, ddt] + [b[1] for b in back]
    for i, (g, w) in enumerate(zip(got, want)):
        err = float((g.double() - w).abs().max() / w.abs().max())
        print("gradient %d: %.2e" % (i, err), flush=True)
        assert err <= 2.0 ** -9, i


def test_refusals():
    x = rnd(2, 4, 32, 64, dtype=torch.bfloat16)
    b = rnd(2, 2, 32, 64, dtype=torch.bfloat16)
    dt, a, w = torch.ones(2, 4, 32, device="cuda"), torch.ones(4, device="cuda"), rnd(4, 4, 64)
    ones = torch.ones(64, device="cuda")
    bad = [
        lambda: fw.ttt_rms_norm_forward(x.half(), ones),
        lambda: fw.ttt_rms_norm_forward(x, ones.bfloat16()),
        lambda: fw.ttt_rms_norm_forward(x.transpose(1, 2), ones),
        lambda: fw.ttt_rms_norm_forward(x, ones, x.float()),
        lambda: fw.ttt_rms_norm_forward(x, ones, res_out=x.clone()),
        lambda: fw.ttt_rms_norm_forward(x[..., :12].contiguous(), ones[:12]),   # width 12
        lambda: fw.ttt_rms_norm_forward(x, ones, eps=-1.0),
        lambda: fw.ttt_rms_norm_forward(x[:0], ones),
        lambda: fw.ttt_rms_norm_forward(x, ones, y=x),
        lambda: fw.ttt_rms_norm_forward_f8(x, ones, scale=torch.ones(2, device="cuda")),
        lambda: fw.ttt_rms_norm_backward(x, ones, x[:1]),
        lambda: fw.ttt_rms_norm_backward(x, ones, x, workspace=torch.empty(
            16, dtype=torch.uint8, device="cuda")),
        lambda: fw.ttt_conv_forward(x, w[:2]),
        lambda: fw.ttt_conv_forward(x, rnd(4, 5, 64)),
        lambda: fw.ttt_conv_forward(x, w, rnd(4, 32)),
        lambda: fw.ttt_conv_forward(x, w, state0=x[:, :, :2].contiguous()),
        lambda: fw.ttt_conv_forward(x, w, y=x),
        lambda: fw.ttt_conv_decode_step(x, w, None, x),
        lambda: fw.ttt_conv_decode_step(x[:, :, 0].contiguous(), w, None,
                                        x[:, :, :3].float().contiguous()),
        lambda: fw.ttt_conv_backward(x, w, None, x.float()),
        lambda: fw.ttt_ssm_forward(x, dt.double(), a, b, b),
        lambda: fw.ttt_ssm_forward(x, dt, a[:2], b, b),
        lambda: fw.ttt_ssm_forward(x, dt, a, b[:, :, :16].contiguous(), b),
        lambda: fw.ttt_ssm_forward(x, dt, a, b, b[..., :32].contiguous()),
        lambda: fw.ttt_ssm_forward(x, dt, a, *(2 * [rnd(2, 3, 32, 64, dtype=torch.bfloat16)])),
        lambda: fw.ttt_ssm_forward(x, dt, a, *(2 * [b[..., :16].contiguous()])),
        lambda: fw.ttt_ssm_forward(x, dt, a, b, b, state0=torch.ones(2, 4, 64, 32, device="cuda")),
        lambda: fw.ttt_ssm_forward(x, dt, a, b.float(), b.float()),
        lambda: fw.ttt_ssm_decode_step(x, dt, a, b, b, torch.ones(2, 4, 64, 64, device="cuda")),
        lambda: fw.ttt_ssm_backward(x, dt, a, b, b, x[:, :, :5].contiguous()),
        lambda: fw.ttt_input_projection_f8(x, dt, b, dt, a, heads=4, eta_base=1.0),
        # 2 bytes off a 16-byte boundary
        lambda: fw.ttt_conv_forward(rnd(1, 1, 9 * 64, 8, dtype=torch.bfloat16).view(-1)[1:513]
                                    .view(1, 1, 64, 8), rnd(1, 4, 8)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("case %d was not refused" % i, flush=True)


def test_a_nan_reaches_its_tile_and_what_comes_after():
    x = rnd(1, 2, 300, 64, seed=1, dtype=torch.bfloat16)
    b, c = (rnd(1, 2, 300, 64, seed=s, scale=0.3, dtype=torch.bfloat16) for s in (2, 3))
    dt, a = torch.full((1, 2, 300), 0.05, device="cuda"), -torch.ones(2, device="cuda")
    y, S = fw.ttt_ssm_forward(x, dt, a, b, c)
    x2 = x.clone()
    x2[0, 0, 150, 7] = float("nan")
    y2, S2 = fw.ttt_ssm_forward(x2, dt, a, b, c)
    assert torch.equal(y2[0, 1], y[0, 1]) and torch.equal(S2[0, 1], S[0, 1])
    assert torch.equal(y2[0, 0, :128], y[0, 0, :128])
    assert bool(torch.isnan(y2[0, 0, 150:, 7]).all()) and bool(torch.isnan(S2[0, 0, :, 7]).all())
    # the other features never meet it
    keep = torch.arange(64, device="cuda") != 7
    assert torch.equal(y2[0, 0][:, keep], y[0, 0][:, keep])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_decays_from_none_to_total_and_a_growing_state(dtype):
    """Steps of 0 (nothing happens), decays that underflow at once, and a state
    that grows by e^0.02 a token."""
    for a, dt in ((-1.0, 0.0), (-1e4, 1.0), (-1e-6, 1e3), (2.0, 0.01)):
        x = rnd(1, 2, 150, 64, seed=4, dtype=dtype)
        b, c = (rnd(1, 1, 150, 32, seed=s, scale=0.3, dtype=dtype) for s in (5, 6))
        A, D = torch.full((2,), a, device="cuda"), torch.full((1, 2, 150), dt, device="cuda")
        s0 = rnd(1, 2, 32, 64, seed=7)
        dy = rnd(1, 2, 150, 64, seed=8, dtype=dtype)
        y, S = fw.ttt_ssm_forward(x, D, A, b, c, state0=s0)
        want = block.ssm(*d64(x, D, A, b, c, None, s0))
        held("y", y, want["y"], want["y_mag"], 2.0 ** -14)
        held("state", S, want["state"], want["state_mag"], 2.0 ** -15)
        got = fw.ttt_ssm_backward(x, D, A, b, c, dy, state0=s0)
        want = block.ssm_backward(*d64(x, D, A, b, c, dy, None, s0),
                                  tile=64 if dtype == torch.bfloat16 else 32)
        for name, t in zip(("dx", "ddt", "da", "db", "dc", None, "dstate0"), got):
            if name:
                held(name, t, want[name], want[name + "_mag"], 2.0 ** -14)


def test_a_stream_of_its_own_and_a_stream_argument():
    x = rnd(2, 3, 200, 64, dtype=torch.bfloat16)
    b = rnd(2, 1, 200, 64, scale=0.3, dtype=torch.bfloat16)
    dt, a = torch.full((2, 3, 200), 0.1, device="cuda"), -torch.ones(3, device="cuda")
    y, S = fw.ttt_ssm_forward(x, dt, a, b, b)
    g = fw.ttt_ssm_backward(x, dt, a, b, b, y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y2, S2 = fw.ttt_ssm_forward(x, dt, a, b, b)
        g2 = fw.ttt_ssm_backward(x, dt, a, b, b, y2)
    y3, S3 = fw.ttt_ssm_forward(x, dt, a, b, b, stream=s)
    s.synchronize()
    for u, v in ((y2, y), (S2, S), (y3, y), (S3, S)):
        assert torch.equal(u, v)
    for u, v in zip(g2, g):
        assert (u is None and v is None) or torch.equal(u, v)


def test_offsets_past_32_bits():
    """More than 2^31 values in one tensor: the last unit (row) is what it is alone."""
    H, T = 9, 1 << 22
    x = torch.empty(1, H, T, 64, dtype=torch.bfloat16, device="cuda")
    x.normal_()
    w, bias = rnd(H, 4, 64, scale=0.5), rnd(H, 64)
    y, tail = fw.ttt_conv_forward(x, w, bias, return_state=True)
    y1, tail1 = fw.ttt_conv_forward(x[:, -1:].contiguous(), w[-1:], bias[-1:], return_state=True)
    assert torch.equal(y[:, -1:], y1) and torch.equal(tail[:, -1:], tail1)
    dx, dw, db, _ = fw.ttt_conv_backward(x, w, bias, y)
    dx1, dw1, db1, _ = fw.ttt_conv_backward(x[:, -1:].contiguous(), w[-1:], bias[-1:], y1)
    assert torch.equal(dx[:, -1:], dx1) and torch.equal(dw[-1:], dw1) and torch.equal(db[-1:], db1)
    del dx, dx1, y1
    rows = x.view(-1, 8192)
    weight = torch.ones(8192, device="cuda")
    n, r = fw.ttt_rms_norm_forward(rows, weight, y.view(-1, 8192))
    n1, r1 = fw.ttt_rms_norm_forward(rows[-3000:].contiguous(), weight,
                                     y.view(-1, 8192)[-3000:].contiguous())
    assert torch.equal(n[-3000:], n1) and torch.equal(r[-3000:], r1)
    del n, r, y
    # the scan: the last unit from a state in its middle is the whole scan's end
    dt = torch.full((1, H, T), 0.05, device="cuda")
    a = -torch.ones(H, device="cuda")
    b = torch.empty(1, H, T, 32, dtype=torch.bfloat16, device="cuda")
    b.normal_(std=0.3)
    y, S = fw.ttt_ssm_forward(x, dt, a, b, b)
    part = [t[:, -1:, -576:].contiguous() for t in (x, dt, b)]
    want = block.ssm(*d64(part[0], part[1], a[-1:], part[2], part[2], None, None))
    # what came before the last 576 tokens has faded to e^-29, and to e^-14 300 tokens from the end
    held("state", S[:, -1:], want["state"], want["state_mag"] + 1.0, 2.0 ** -15)
    held("y", y[:, -1:, -300:], want["y"][:, :, -300:], want["y_mag"][:, :, -300:] + 1.0,
         2.0 ** -14)
    dy = torch.flip(y, [2])
    del y
    got = fw.ttt_ssm_backward(x, dt, a, b, b, dy)
    g = block.ssm_backward(*d64(part[0], part[1], a[-1:], part[2], part[2],
                                dy[:, -1:, -576:].contiguous(), None, None, None))
    for name, t in zip(("dx", "ddt"), got):
        held(name, t[:, -1:, -300:], g[name][:, :, -300:], g[name + "_mag"][:, :, -300:] + 1.0,
             2.0 ** -14)


def test_projection_offsets_past_32_bits():
    """More than 2^31 values of x and of each of q, k, v (T itself is at most 2^22)."""
    T, D, H = (1 << 21) + 300, 512, 9
    x = torch.empty(2, T, D, dtype=torch.float8_e4m3fn, device="cuda")
    x.view(torch.uint8).random_(0, 0x78)      # every positive finite value but the top binade's
    xs = torch.full((2, T), 2.0 ** -10, device="cuda")
    w = rnd(3 * H * 64 + H, D, seed=60).to(torch.float8_e4m3fn)
    ws = torch.full((3 * H * 64 + H,), 2.0 ** -5, device="cuda")
    be = rnd(H, seed=61, scale=0.1)
    got = fw.ttt_input_projection_f8(x, xs, w, ws, be, heads=H, eta_base=1 / 64)
    want = block.input_f8(*d64(x[1:, -300:], xs[1:, -300:], w, ws, be), H, 1 / 64)
    for name, t in zip("qkv", got):
        held(name, t[1:, :, -300:], want[name], want[name + "_mag"], 2.0 ** -15)
    gate = want["gate_mag"] * (D / 32 + 40) * 2.0 ** -24
    held("eta", got[3][1:, :, -300:], want["eta"], want["eta"] * (gate + 2.0 ** -20), 1.0)
