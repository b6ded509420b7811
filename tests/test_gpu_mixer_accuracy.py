"""GPU: fp32 operands keep fp32's accuracy where exponentials are far from 1:
strong decays, gates that are nearly shut, and SiLU far below zero, where a
rounding of the exponent's argument would show as |x| half steps.

Tolerances.  Scan: half a step and the oracle's bound (2^-20 of every term),
with one token a sequence, so that nothing else hides an error.  SiLU, relative
to its value: exp 2^-22 + 2^-23, 1 + e 2^-24, the reciprocal 2^-23, the product
2^-24: below 3 * 2^-22.  Its derivative times dy has the factor 1 + z (1 - s) in
place of z, which rounds once more and for z <= -4 carries 4/3 of the error of
1 - s (s < 0.02, so 2^-24 and 0.02 of the above), and one more product: 2^-24
each, below 2^-20 in all."""
import numpy as np
import pytest
import torch

from chunk_gated_delta_02_b200 import carve
from oracle import mixer

from _mixer import close, cuda, np64

pytestmark = pytest.mark.gpu

N = 400


def spread(lo, hi):
    """N values between, none of them round."""
    gen = torch.Generator().manual_seed(7)
    return torch.linspace(lo, hi, N) + (hi - lo) / N * torch.rand(N, generator=gen) * 0.9


def check_scan(raw, scale, comp, x, h0):
    """One token a sequence, forward and backward and as a single step."""
    g = raw.view(-1, 1, 8).cuda()
    x, h0 = torch.full_like(g, x), torch.full_like(g[:, 0], h0)
    d_h, dh_T = torch.full_like(g, 0.7), torch.zeros_like(h0)
    opt = dict(decay_scale=scale, complement=comp)
    h, h_T, ws = carve.scan_fwd(x, g, h0, training=True, **opt)
    gr = carve.scan_bwd(x, g, d_h, ws, dh_T=dh_T, **opt)
    state = h0.clone()
    o = carve.scan_step(x[:, 0], g[:, 0], state, **opt)
    for b in range(len(g)):
        args = [np64(t[b]) for t in (x, g)] + [np64(h0[b])]
        ref, last, e = mixer.scan_fwd(*args, scale, comp)
        for got, what in ((h[b], "h"), (h_T[b:b + 1], "h_T"), (o[b:b + 1], "o"),
                          (state[b:b + 1], "state")):
            close(got, ref, e, what)
        r = mixer.scan_bwd(*args, np64(d_h[b]), np64(dh_T[b]), scale, comp)
        for name in ("dx", "dg"):
            close(gr[name][b], *r[name], name)
        close(gr["dh0"][b], *r["dh0"], "dh0")


def test_strong_decays():
    check_scan(-spread(0.05, 80.0), 0.0, False, 0.0, 1.3)


@pytest.mark.parametrize("comp", [False, True])
def test_gates_nearly_shut(comp):
    check_scan(-spread(0.1, 80.0), 1.0, comp, 1.7, 0.0)


def test_gates_wide_open():
    # (beyond, the rounding of the log-decay itself counts: |u| 2^-24 of the decay)
    check_scan(spread(0.1, 4.0), 1.0, True, 0.0, 1.3)


def test_packed_and_long_walks_share_it():
    """The other instances: sequences of more than one segment, packed."""
    raw = -spread(10.0, 80.0).view(50, 8).cuda()
    cu = torch.arange(51, dtype=torch.int32, device="cuda")
    x, zero = torch.full_like(raw, 1.7), torch.zeros(50, 8, device="cuda")
    h, _, _ = carve.scan_fwd(x, raw, zero, cu, decay_scale=1.0, complement=True)
    for t in range(50):
        ref, _, e = mixer.scan_fwd(np64(x[t:t + 1]), np64(raw[t:t + 1]), np.zeros(8), 1.0, True)
        close(h[t:t + 1], ref, e, "packed")


def test_silu_far_below_zero():
    z = -spread(4.0, 80.0).view(-1, 8)
    x = z.cuda()[None]
    w = cuda([[0.0, 1.0]] * 8)
    y, _ = carve.conv_fwd(x, w, silu=True)
    gr = carve.conv_bwd(x, w, torch.full_like(x, 0.7), silu=True)
    step = carve.conv_step(x[0], w, torch.zeros(x.shape[1], 1, 8, device="cuda"), silu=True)
    v = np64(z)
    s = 1 / (1 + np.exp(-v))
    dy = float(np.float32(0.7))
    for got, ref, tol in ((y[0], v * s, 3 * 2.0 ** -22), (step, v * s, 3 * 2.0 ** -22),
                          (gr["dx"][0], dy * s * (1 + v * (1 - s)), 2.0 ** -20)):
        assert (np.abs(np64(got) - ref) <= tol * np.abs(ref)).all()
