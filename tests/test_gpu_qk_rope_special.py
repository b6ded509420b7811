"""GPU: rows of the norms and the rotation that hold NaN, infinities or
nothing but tiny values."""
import pytest
import torch

from chunk_gated_delta_02_b200 import carve

from _mixer import DT

pytestmark = pytest.mark.gpu

N, H, RD = 11, 3, 32


def draw(D, dt, seed):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen).to(DT[dt]).cuda()  # noqa: E731
    pos = torch.arange(N, dtype=torch.int32, device="cuda") + 900
    return rn(N, H, D), rn(N, H, D), rn(D), pos, carve.rope_freqs(RD)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("l2norm", [False, True], ids=["mean", "l2"])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [32, 80, 128])
def test_a_nan_makes_its_row_nan_and_no_other(D, dt, l2norm, eps):
    q, dy, w, pos, freqs = draw(D, dt, D)
    opt = dict(eps=eps, l2norm=l2norm)
    want, _ = carve.qk_rope_fwd(q, None, pos, freqs, w, **opt)
    grad = carve.qk_rope_bwd(q, None, pos, freqs, dy, None, w, **opt)["dq"]
    bad = q.clone()
    rows = [(0, 1, 0), (4, 0, D - 1), (10, 2, RD // 2)]
    for n, h, i in rows:
        bad[n, h, i] = float("nan")
    y, _ = carve.qk_rope_fwd(bad, None, pos, freqs, w, **opt)
    gr = carve.qk_rope_bwd(bad, None, pos, freqs, dy, None, w, **opt)
    hit = torch.zeros(N, H, dtype=torch.bool, device="cuda")
    for n, h, _ in rows:
        hit[n, h] = True
    for got, whole in ((y, want), (gr["dq"], grad)):
        assert got[hit].isnan().all()
        assert torch.equal(got[~hit], whole[~hit])
    assert gr["dw_q"].isnan().all()  # the sums over all rows


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_rows_of_norm_zero(dt):
    """Zeros, and values whose squares fp32 does not hold, give zeros with
    eps = 0; with eps > 0 the latter keep their direction."""
    q, dy, w, pos, freqs = draw(64, dt, 1)
    q[2] = 0
    q[5] = 1e-30 * q[5].sign()
    for l2norm in (False, True):
        y, _ = carve.qk_rope_fwd(q, None, pos, freqs, w, eps=0.0, l2norm=l2norm)
        gr = carve.qk_rope_bwd(q, None, pos, freqs, dy, None, w, eps=0.0, l2norm=l2norm)
        for n in (2, 5):
            assert (y[n] == 0).all() and (gr["dq"][n] == 0).all()
        assert y.isfinite().all() and gr["dw_q"].isfinite().all()
    y, _ = carve.qk_rope_fwd(q, None, None, None, eps=1e-6)
    assert torch.equal(y[5].sign(), q[5].sign())
