"""GPU selective state space scan (forward, step, backward) against oracle/block.py.

coef, relative to the sum of magnitudes.  A decay exp2(e) made from an fp32
exponent is off by 0.7 |e| 2^-24 of itself, at most 2^-17 before it underflows
(|e| < 127); sums of up to 128 + 64 terms in fp32 by less than 2^-16.4.  fp32
data (24-bit operands): together below 2^-15.6, taken as 2^-15.  bf16 data
carry M and S (W1, W2, A and S) in 16 bits, 2^-16 for each of two factors at
most: 2^-14.  The state's own operands have 24 bits, so its bound is that of
fp32 data in both.  Exponents here stay small, and the observed errors far
below: the bound is what every input is promised."""
import math

import pytest
import torch

from linear_rnn_ttt_amd import ttt_ssm_backward, ttt_ssm_decode_step, ttt_ssm_forward
from oracle import block

from _block import d64, held, replayed, rnd

pytestmark = pytest.mark.gpu
COEF = {torch.bfloat16: 2.0 ** -14, torch.float32: 2.0 ** -15}
STATE = 2.0 ** -15
TILE = {torch.bfloat16: 64, torch.float32: 32}
TYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]


def make(B, H, G, T, N, dtype, seed=0, reset=False):
    x = rnd(B, H, T, 64, seed=seed, dtype=dtype)
    b = rnd(B, G, T, N, seed=seed + 1, scale=N ** -0.25, dtype=dtype)
    c = rnd(B, G, T, N, seed=seed + 2, scale=N ** -0.25, dtype=dtype)
    dt = torch.exp(rnd(B, H, T, seed=seed + 3) - 3.0)
    if reset:     # some tokens forget everything before them, some change nothing
        dt.view(-1)[::7] = 40.0
        dt.view(-1)[3::11] = 0.0
    a = -torch.exp(rnd(H, seed=seed + 4))
    return x, dt, a, b, c, rnd(H, seed=seed + 5), rnd(B, H, N, 64, seed=seed + 6, scale=0.2)


CASES = [(1, 1, 1, 1, 32), (2, 2, 1, 2, 64), (1, 3, 3, 17, 128), (2, 4, 2, 63, 32),
         (1, 2, 2, 64, 64), (1, 2, 1, 65, 128), (2, 3, 1, 130, 64), (1, 4, 4, 321, 32),
         (1, 6, 2, 200, 128)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("B,H,G,T,N", CASES)
def test_forward(B, H, G, T, N, dtype):
    for i, (skip, first) in enumerate(((True, True), (False, False))):
        x, dt, a, b, c, d, s0 = make(B, H, G, T, N, dtype, seed=i, reset=i == 1)
        d, s0 = d if skip else None, s0 if first else None
        y, S = ttt_ssm_forward(x, dt, a, b, c, d, state0=s0)
        want = block.ssm(*d64(x, dt, a, b, c, d, s0))
        held("y", y, want["y"], want["y_mag"], COEF[dtype])
        held("state", S, want["state"], want["state_mag"], STATE)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("B,H,G,T,N", CASES)
def test_backward(B, H, G, T, N, dtype):
    names = ("dx", "ddt", "da", "db", "dc", "dd", "dstate0")
    for i, full in enumerate((True, False)):
        x, dt, a, b, c, d, s0 = make(B, H, G, T, N, dtype, seed=10 + i, reset=i == 1)
        dy = rnd(B, H, T, 64, seed=20, dtype=dtype)
        dS = rnd(B, H, N, 64, seed=21) if full else None
        if not full:
            d = s0 = None
        got = ttt_ssm_backward(x, dt, a, b, c, dy, d, state0=s0, dstate=dS)
        want = block.ssm_backward(*d64(x, dt, a, b, c, dy, d, s0, dS), tile=TILE[dtype])
        for name, g in zip(names, got):
            if name in ("dd", "dstate0") and not full:
                assert g is None
                continue
            held(name, g, want[name], want[name + "_mag"],
                 STATE if name == "dstate0" else COEF[dtype])
            if g.dtype == torch.float32:   # beside the sums' bound, the fp32 tolerance of the scans
                err = float((g.double() - want[name]).abs().max())
                assert err <= 1e-4 * float(want[name].abs().max()), (name, err)


def test_a_reset_leaves_later_tokens_exact():
    """A step of decay -4e4 inside a tile: the tokens behind it see only each
    other, with decays as exact as without it."""
    x, dt, a, b, c, d, s0 = make(1, 2, 2, 50, 64, torch.float32, seed=3)
    a = -torch.ones_like(a)
    dt = dt.clamp(max=0.01)
    dt[:, :, 20] = 4e4
    y, S = ttt_ssm_forward(x, dt, a, b, c, d, state0=s0)
    x2 = x.clone()
    b2, dt2 = b.clone(), dt.clone()
    want = block.ssm(*d64(x, dt, a, b, c, d, s0))
    # exponents of the tokens behind are below 0.3: no 2^-17 term
    held("y", y[:, :, 21:], want["y"][:, :, 21:], want["y_mag"][:, :, 21:], 2.0 ** -18)
    held("state", S, want["state"], want["state_mag"], 2.0 ** -18)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("B,H,G,N", [(1, 1, 1, 32), (3, 4, 2, 64), (2, 6, 1, 128)])
def test_step_by_step(B, H, G, N, dtype):
    T = 5
    x, dt, a, b, c, d, s0 = make(B, H, G, T, N, dtype, seed=2)
    want = block.ssm(*d64(x, dt, a, b, c, d, s0))
    for skip in (d, None):
        S = s0.clone()
        for t in range(T):
            y = ttt_ssm_decode_step(*(v[:, :, t].contiguous() for v in (x, dt)), a,
                                    *(v[:, :, t].contiguous() for v in (b, c)), S, skip)
            ref, mag = want["y"][:, :, t], want["y_mag"][:, :, t]
            if skip is None:
                ref = ref - (x[:, :, t] * d[:, None]).double()
            # fp32 throughout: N + 8 roundings of a sum
            held("y", y, ref, mag, (N + 8 + 8 * t) * 2.0 ** -24)
        held("state", S, want["state"], want["state_mag"], 2.0 ** -19)


def test_prompt_cut_in_two_and_in_place_state():
    x, dt, a, b, c, d, s0 = make(2, 2, 1, 150, 64, torch.bfloat16, seed=5)
    want = block.ssm(*d64(x, dt, a, b, c, d, s0))
    S = s0.clone()
    y1, _ = ttt_ssm_forward(*(v[:, :, :70].contiguous() for v in (x, dt)), a,
                            *(v[:, :, :70].contiguous() for v in (b, c)), d, state0=S,
                            state_out=S)
    y2, _ = ttt_ssm_forward(*(v[:, :, 70:].contiguous() for v in (x, dt)), a,
                            *(v[:, :, 70:].contiguous() for v in (b, c)), d, state0=S,
                            state_out=S)
    held("y", torch.cat([y1, y2], 2), want["y"], want["y_mag"], COEF[torch.bfloat16])
    held("state", S, want["state"], want["state_mag"], STATE)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T", [90, 250, 700])
def test_in_place_state_of_any_number_of_segments(T, dtype):
    """The final state written over state0, which other workgroups of the unit
    read: bit for bit the state and outputs of a call with two tensors."""
    x, dt, a, b, c, d, s0 = make(2, 3, 1, T, 64, dtype, seed=17)
    y, want = ttt_ssm_forward(x, dt, a, b, c, d, state0=s0)
    for _ in range(4):
        S = s0.clone()
        y2, S2 = ttt_ssm_forward(x, dt, a, b, c, d, state0=S, state_out=S)
        assert S2 is S and torch.equal(S, want) and torch.equal(y2, y)


def test_steps_of_zero_leave_the_state():
    """A padded batch: tokens with dt = 0 behind a sequence's end."""
    x, dt, a, b, c, d, s0 = make(2, 3, 1, 140, 64, torch.bfloat16, seed=6)
    dt[1, :, 90:] = 0.0
    _, S = ttt_ssm_forward(x, dt, a, b, c, d, state0=s0)
    want = block.ssm(*d64(*(v[1:, :, :90] for v in (x, dt)), a, *(v[1:, :, :90] for v in (b, c)),
                          d, s0[1:]))
    held("state", S[1:], want["state"], want["state_mag"], STATE)


def test_many_units_take_one_segment_each():
    """As many units as make one segment: the scan's single launch."""
    x, dt, a, b, c, d, s0 = make(40, 32, 1, 70, 32, torch.bfloat16, seed=7)
    y, S = ttt_ssm_forward(x, dt, a, b, c, d, state0=s0)
    got = ttt_ssm_backward(x, dt, a, b, c, y, d, state0=s0, dstate=S)
    pick = slice(17, 19)
    sub = [v[pick] for v in (x, dt)] + [a] + [v[pick] for v in (b, c)]
    want = block.ssm(*d64(*sub, d, s0[pick]))
    held("y", y[pick], want["y"], want["y_mag"], COEF[torch.bfloat16])
    held("state", S[pick], want["state"], want["state_mag"], STATE)
    g = block.ssm_backward(*d64(*sub, y[pick], d, s0[pick], S[pick]))
    for name, t in zip(("dx", "ddt", None, "db", "dc", None, "dstate0"), got):
        if name:
            held(name, t[pick], g[name], g[name + "_mag"], COEF[torch.bfloat16])


def test_long_sequence_of_one_unit_and_odd_segments():
    x, dt, a, b, c, d, s0 = make(1, 1, 1, 5003, 64, torch.bfloat16, seed=8)
    y, S = ttt_ssm_forward(x, dt, a, b, c, d, state0=s0)
    want = block.ssm(*d64(x, dt, a, b, c, d, s0))
    held("y", y, want["y"], want["y_mag"], COEF[torch.bfloat16])
    held("state", S, want["state"], want["state_mag"], STATE)
    dy = rnd(1, 1, 5003, 64, seed=9, dtype=torch.bfloat16)
    got = ttt_ssm_backward(x, dt, a, b, c, dy, d, state0=s0)
    g = block.ssm_backward(*d64(x, dt, a, b, c, dy, d, s0))
    for name, t in zip(("dx", "ddt", "da", "db", "dc", "dd", "dstate0"), got):
        held(name, t, g[name], g[name + "_mag"], COEF[torch.bfloat16])


def test_gradients_against_differences_of_the_gpu_forward():
    """fp32 data: the loss's change along a random direction of every input.
    The forward's own error (2^-20 of magnitudes summing to some 1e4 here) over
    a step of 2^-6 in each direction is below 1 %; the difference's curvature
    is made small by the central form."""
    x, dt, a, b, c, d, s0 = make(1, 2, 1, 90, 32, torch.float32, seed=12)
    dy = rnd(1, 2, 90, 64, seed=13)
    dS = rnd(1, 2, 32, 64, seed=14)
    args = [x, dt, a, b, c, d, s0]
    grads = ttt_ssm_backward(x, dt, a, b, c, dy, d, state0=s0, dstate=dS)
    for i, g in enumerate(grads):
        h = 2.0 ** -6 * float(args[i].abs().mean())
        way = torch.sign(g)
        loss = []
        for sgn in (1.0, -1.0):
            v = list(args)
            v[i] = (v[i] + sgn * h * way).contiguous()
            y, S = ttt_ssm_forward(*v[:6], state0=v[6])
            loss.append(float((y.double() * dy).sum() + (S.double() * dS).sum()))
        diff, want = (loss[0] - loss[1]) / (2 * h), float(g.double().abs().sum())
        print("input %d: difference %.6g, gradient %.6g" % (i, diff, want), flush=True)
        assert abs(diff - want) <= 0.01 * want


def test_captured_and_replayed_repeatable_and_two_workspaces():
    x, dt, a, b, c, d, s0 = make(2, 4, 2, 700, 64, torch.bfloat16, seed=15)
    dy = rnd(2, 4, 700, 64, seed=16, dtype=torch.bfloat16)
    replayed(lambda: ttt_ssm_forward(x, dt, a, b, c, d, state0=s0), ("y", "state"))
    replayed(lambda: ttt_ssm_backward(x, dt, a, b, c, dy, d, state0=s0),
             ("dx", "ddt", "da", "db", "dc", "dd", "dstate0"))
    want = ttt_ssm_forward(x, dt, a, b, c, d, state0=s0)
    torch.cuda.synchronize()
    # two calls at once, each under its own stream
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        got.append(ttt_ssm_forward(x, dt, a, b, c, d, state0=s0, stream=s))
    for s in streams:
        s.synchronize()
    for g in got:
        for u, v in zip(g, want):
            assert torch.equal(u, v)
