"""GPU: states and gradients that are infinite or NaN stay in their sequence,
and a log-decay of -inf forgets what is finite (0 times infinity is NaN, here as
in the recurrence)."""
import pytest
import torch

from chunk_gated_delta_02_b200 import carve

from _mixer import DT, offsets

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def draw(T, C, N, dt):
    gen = torch.Generator().manual_seed(T + C)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, d_h = rn(T, C).to(DT[dt]).cuda(), rn(T, C).to(DT[dt]).cuda()
    return x, (-0.1 * rn(T, C).abs()).to(DT[dt]).cuda(), d_h, rn(N, C).cuda(), rn(N, C).cuda()


LENGTHS = [[37, 64, 100], [5, 3, 2, 1, 1, 7, 200], [1000, 1, 1500], [128, 128, 128], [70, 0, 70]]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [INF, -INF, NAN], ids=["inf", "-inf", "nan"])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: "-".join(map(str, v)))
def test_states_that_are_not_finite_stay_in_their_sequence(lengths, value, dt):
    T, N, C = sum(lengths), len(lengths), 72
    x, g, d_h, h0, dh_T = draw(T, C, N, dt)
    cu = offsets(lengths)
    at = [sum(lengths[:i]) for i in range(N + 1)]
    h, h_T, ws = carve.scan_fwd(x, g, h0, cu, training=True)
    gr = carve.scan_bwd(x, g, d_h, ws, dh_T=dh_T, cu_seqlens=cu)
    for i in range(N):
        bad, bad_T = h0.clone(), dh_T.clone()
        bad[i], bad_T[i] = value, value
        h2, h_T2, ws2 = carve.scan_fwd(x, g, bad, cu, training=True)
        gr2 = carve.scan_bwd(x, g, d_h, ws2, dh_T=dh_T, cu_seqlens=cu)
        gr3 = carve.scan_bwd(x, g, d_h, ws, dh_T=bad_T, cu_seqlens=cu)
        rows = torch.ones(T, dtype=torch.bool, device="cuda")
        rows[at[i]:at[i + 1]] = False
        seqs = torch.arange(N, device="cuda") != i
        for got, want in ((h2, h), (gr2["dx"], gr["dx"]), (gr2["dg"], gr["dg"]),
                          (gr3["dx"], gr["dx"]), (gr3["dg"], gr["dg"])):
            assert torch.equal(got[rows], want[rows])
        for got, want in ((h_T2, h_T), (gr2["dh0"], gr["dh0"]), (gr3["dh0"], gr["dh0"])):
            assert torch.equal(got[seqs], want[seqs])
        # where it belongs it shows: the first row and the first gradient
        assert not h_T2[i].isfinite().any() and not gr3["dh0"][i].isfinite().any()
        if lengths[i]:
            assert not h2[at[i]].isfinite().any()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_decay_of_minus_infinity(dt):
    x, g, _, _, _ = draw(300, 64, 1, dt)
    x, g = x[None], g[None]
    g[0, 150] = -INF
    h0 = torch.ones(1, 64, device="cuda")
    h, _, _ = carve.scan_fwd(x, g, h0)
    other, _, _ = carve.scan_fwd(x, g, 1e30 * h0)
    assert torch.equal(h[0, 150:], other[0, 150:])  # finite states are forgotten
    assert torch.equal(h[0, 150], x[0, 150])
    h, h_T, _ = carve.scan_fwd(x, g, INF * h0)
    assert (h[0, :150] == INF).all() and h[0, 150:].isnan().all() and h_T.isnan().all()
    h, h_T, _ = carve.scan_fwd(x, g, NAN * h0)
    assert h.isnan().all() and h_T.isnan().all()
