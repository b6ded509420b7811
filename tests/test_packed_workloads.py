"""The plain forms of perf/operators.py on packed batches, and the library's
calls there: rows behind the last sequence belong to none, so that they are
zero and every other row is the oracle's."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import mixer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ops():
    spec = importlib.util.spec_from_file_location(
        "workloads", os.path.join(ROOT, "perf", "operators.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def state(lengths, behind, mode):
    """What the scan's plain form takes, on the CPU in fp32."""
    gen = torch.Generator().manual_seed(len(lengths) + behind)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    T, N, H, D = sum(lengths) + behind, len(lengths), 2, 8
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    return dict(case=dict(op="scan", mode=mode, ragged=True, dtype="fp32", complement=True),
                x=rn(T, H, D), g=-0.1 * rn(T, H, D).abs(), scale=0.0, h0=rn(N, H, D), cu=cu,
                longest=max(lengths), d_h=rn(T, H, D), dh_T=rn(N, H, D))


@pytest.mark.parametrize("lengths, behind", [([9, 0, 17], 5), ([1, 2], 40), ([30], 1), ([8, 3], 0)])
def test_plain_packed_scan_is_the_oracle(ops, lengths, behind):
    s = state(lengths, behind, "train")
    n64 = {k: v.double().reshape(len(v), -1).numpy() for k, v in s.items()
           if k in ("x", "g", "h0", "d_h", "dh_T")}
    h, h_T, dx, dg, dh0 = (t.reshape(len(t), -1).double().numpy() for t in ops._plain_scan(s))
    end = sum(lengths)
    for t in (h, dx, dg):
        assert (t[end:] == 0).all()
    at = 0
    for i, n in enumerate(lengths):
        rows = [n64[k][at:at + n] for k in ("x", "g")]
        want, last, e = mixer.scan_fwd(*rows, n64["h0"][i], complement=True)
        # the doubled products and sums round once more for every level: a
        # bound of 2^-20 a step takes those of 8 levels
        assert (np.abs(h[at:at + n] - want) <= e + 2.0 ** -24 * np.abs(want)).all()
        assert np.allclose(h_T[i], last, rtol=0, atol=1e-5)
        r = mixer.scan_bwd(*rows, n64["h0"][i], n64["d_h"][at:at + n], n64["dh_T"][i],
                           complement=True)
        for got, key in ((dx[at:at + n], "dx"), (dg[at:at + n], "dg"), (dh0[i], "dh0")):
            assert (np.abs(got - r[key][0]) <= r[key][1] + 2.0 ** -24 * np.abs(r[key][0])).all(), key
        at += n


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["fwd", "train"])
@pytest.mark.parametrize("T, B", [(64 * 3 + 41, 3), (700, 2), (158, 2)])
def test_packed_scan_behind_the_last_sequence(ops, mode, T, B):
    case = dict(op="scan", mode=mode, B=B, T=T, H=2, D=16, dtype="fp32", ragged=True, raw=True,
                complement=False)
    end = int(ops.prepare(case, 3)["cu"][-1])
    assert end < T
    plain = ops.run(ops.prepare(case, 3))
    ops.own = True
    try:
        own = ops.run(ops.prepare(case, 3))
    finally:
        ops.own = False
    rows = [0] if mode == "fwd" else [0, 2, 3]
    for i in rows:
        for out in (plain, own, ops.exact(case, 3)):
            assert (out[i][end:] == 0).all()
