"""GPU input projection from 8-bit operands against oracle/block.py, and the
layer's calls run together: norm, projection, convolution, scan.

coef: q, k, v come from the 8-bit matrix product, whose sums of 128 exact
products were measured to be off by up to 7e-4 where they are about 11 in size
and their magnitudes sum to about 80 (9e-6 of the magnitudes): 2^-15 with room;
then three fp32 products.  The gate's sums are fp32: D / 32 steps of 32, below
(D / 32 + 40) 2^-24; through the sigmoid eta moves by at most that times eta
(its slope is below its value), and its own exponential, sum and division are
off by a few 2^-24: 2^-20."""
import pytest
import torch

from linear_rnn_ttt_amd import (ttt_conv_decode_step, ttt_conv_forward, ttt_input_projection,
                                ttt_input_projection_f8, ttt_linear_forward,
                                ttt_rms_norm_forward, ttt_rms_norm_forward_f8,
                                ttt_ssm_decode_step, ttt_ssm_forward)
from oracle import block

from _block import d64, held, replayed, rnd

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def rows_f8(v):
    s = v.abs().amax(-1).clamp(min=1e-20) / 448.0
    return (v / s[..., None]).to(F8), s


def make(B, T, D, H, seed=0):
    x, xs = rows_f8(rnd(B, T, D, seed=seed))
    w, ws = rows_f8(torch.cat([rnd(3 * H * 64, D, seed=seed + 1, scale=(D * 64) ** -0.5),
                               rnd(H, D, seed=seed + 2, scale=D ** -0.5)]))
    return x, xs, w, ws, rnd(H, seed=seed + 3, scale=0.1)


def check(got, want, D):
    for name, t in zip("qkv", got):
        held(name, t, want[name], want[name + "_mag"], 2.0 ** -15)
    gate = want["gate_mag"] * (D / 32 + 40) * 2.0 ** -24
    held("eta", got[3], want["eta"], want["eta"] * (gate + 2.0 ** -20), 1.0)


@pytest.mark.parametrize("B,T,D,H", [(1, 1, 64, 1), (2, 100, 128, 2), (3, 257, 192, 3),
                                     (1, 300, 768, 12), (2, 33, 64, 5), (61, 1, 768, 12),
                                     (1, 513, 2048, 2), (4, 300, 320, 40),
                                     # enough 256 x 256 tiles for the larger workgroup, with
                                     # one step of D, a half step behind one, and several
                                     (1, 2300, 64, 40), (3, 767, 192, 40), (2, 1100, 512, 41)],
                         ids=lambda v: str(v))
def test_matches_the_oracle(B, T, D, H):
    x, xs, w, ws, be = make(B, T, D, H)
    got = ttt_input_projection_f8(x, xs, w, ws, be, heads=H, eta_base=1 / 64)
    check(got, block.input_f8(*d64(x, xs, w, ws, be), H, 1 / 64), D)


def test_gate_extremes_and_rows_of_zeros():
    x, xs, w, ws, be = make(1, 70, 128, 4)
    x[0, 3] = torch.zeros(128, device="cuda").to(F8)
    be = torch.tensor([30.0, -30.0, 0.0, 2.0], device="cuda")
    got = ttt_input_projection_f8(x, xs, w, ws, be, heads=4, eta_base=0.5)
    check(got, block.input_f8(*d64(x, xs, w, ws, be), 4, 0.5), 128)
    assert all(bool((t[0, :, 3] == 0).all()) for t in got[:3])


def test_captured_and_replayed():
    x, xs, w, ws, be = make(2, 300, 256, 3)
    replayed(lambda: ttt_input_projection_f8(x, xs, w, ws, be, heads=3, eta_base=1 / 64),
             ("q", "k", "v", "eta"))


def layer(D=256, H=4, K=4):
    return dict(norm=rnd(D, seed=31, scale=0.1, shift=1.0), be=rnd(H, seed=32, scale=0.1),
                w=torch.cat([rnd(3 * H * 64, D, seed=33, scale=(D * 64) ** -0.5),
                             rnd(H, D, seed=34, scale=D ** -0.5)]),
                conv=[rnd(H, K, 64, seed=35 + i, scale=K ** -0.5) for i in range(3)],
                bias=[rnd(H, 64, seed=38 + i, scale=0.1) for i in range(3)],
                a=-torch.exp(rnd(H, seed=41)), skip=rnd(H, seed=42))


@pytest.mark.parametrize("eight", [True, False], ids=["8bit", "bf16"])
def test_a_layer_prompt_then_steps(eight):
    """Norm with the residual, projection, convolutions, scan over a prompt, then
    token by token with the states: the steps continue the prompt as a longer
    prompt would, and each call agrees with its reference on its own inputs."""
    B, T, D, H, more = 2, 75, 256, 4, 3
    L = layer(D, H)
    x = rnd(B, T + more, D, seed=50, dtype=torch.bfloat16)
    res = rnd(B, T + more, D, seed=51, dtype=torch.bfloat16)
    if eight:
        w8, ws = rows_f8(L["w"])

    def front(x, res):
        if eight:
            y, s, r = ttt_rms_norm_forward_f8(x, L["norm"], res)
            return ttt_input_projection_f8(y, s, w8, ws, L["be"], heads=H, eta_base=1 / 64)
        y, r = ttt_rms_norm_forward(x, L["norm"], res)
        return ttt_input_projection(y, L["w"].bfloat16(), L["be"], heads=H, eta_base=1 / 64)

    def prompt(n):
        q, k, v, eta = front(x[:, :n].contiguous(), res[:, :n].contiguous())
        conv = [ttt_conv_forward(t, w, b, return_state=True)
                for t, w, b in zip((q, k, v), L["conv"], L["bias"])]
        c, b, u = (o[0] for o in conv)
        y, S = ttt_ssm_forward(u, eta, L["a"], b, c, L["skip"])
        return y, S, [o[1] for o in conv], (u, eta, b, c), (q, k, v)

    full, Sfull, tails_full, (u, eta, b, c), (q, k, v) = prompt(T + more)
    want = block.ssm(*d64(u, eta, L["a"], b, c, L["skip"]))
    held("scan", full, want["y"], want["y_mag"], 2.0 ** -14)
    # the TTT scan takes the same inputs
    z, _ = ttt_linear_forward(q, k, v, eta, rnd(H, 64, 64, seed=60, scale=0.02),
                              torch.ones(H, 64, device="cuda"), torch.zeros(H, 64, device="cuda"))
    assert bool(torch.isfinite(z.float()).all())

    _, S, tails, _, _ = prompt(T)
    for t in range(T, T + more):
        q, k, v, eta = front(x[:, t:t + 1].contiguous(), res[:, t:t + 1].contiguous())
        c, b, u = (ttt_conv_decode_step(p.view(B, H, 64), w, bi, s)
                   for p, w, bi, s in zip((q, k, v), L["conv"], L["bias"], tails))
        y = ttt_ssm_decode_step(u, eta.view(B, H), L["a"], b, c, S, L["skip"])
        held("token %d" % t, y, want["y"][:, :, t], want["y_mag"][:, :, t], 2.0 ** -14)
    for one, other in zip(tails, tails_full):
        assert torch.equal(one, other)
    held("state", S, want["state"], want["state_mag"], 2.0 ** -15)
