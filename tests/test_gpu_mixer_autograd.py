"""GPU: the operators around the core under autograd: tensors that a later
call overwrites, packed batches, workspaces handed on by the wrappers."""
import pytest
import torch

from chunk_gated_delta_02_b200 import carve
from oracle import mixer

from _mixer import close, np64, offsets

pytestmark = pytest.mark.gpu


def rn(*shape, seed=1, dtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=gen).to(dtype).cuda()


def leaf(t):
    return t.clone().requires_grad_()


def writes(t):
    """Calls that write into t, a [2, 3, 16] tensor."""
    x, w, q = rn(2, 16), rn(16, 4), rn(2, 3, 16)
    neg = -q.abs()
    ws = carve.scan_fwd(q, neg, training=True)[2]
    return {
        "conv_step state": lambda: carve.conv_step(x, w, t),
        "scan_step state": lambda: carve.scan_step(q, neg, t),
        "scan_step o": lambda: carve.scan_step(q, neg, q.clone(), o=t),
        "scan_fwd h": lambda: carve.scan_fwd(q, neg, h=t),
        "scan_bwd dg": lambda: carve.scan_bwd(q, neg, q, ws, out=dict(
            dx=torch.empty_like(q), dg=t, dh0=None)),
        "qk_rope_fwd q_out": lambda: carve.qk_rope_fwd(q, None, None, None, q_out=t),
        "qk_rope_bwd dq": lambda: carve.qk_rope_bwd(q, None, None, None, q, None, out=dict(dq=t)),
        "conv_fwd y": lambda: carve.conv_fwd(q, w, y=t),
        "conv_bwd dx": lambda: carve.conv_bwd(q, w, q, out=dict(
            dx=t, dw=torch.empty(16, 4, device="cuda"))),
    }


@pytest.mark.parametrize("name", [
    "conv_step state", "scan_step state", "scan_step o", "scan_fwd h", "scan_bwd dg",
    "qk_rope_fwd q_out", "qk_rope_bwd dq", "conv_fwd y", "conv_bwd dx"])
def test_a_kept_tensor_that_was_overwritten_is_noticed(name):
    t, other = rn(2, 3, 16), leaf(rn(2, 3, 16, seed=2))
    loss = (t * other).sum()  # keeps t
    writes(t)[name]()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_the_state_of_a_convolution_that_was_overwritten_is_noticed():
    x, w, state = leaf(rn(2, 5, 16)), rn(16, 4), rn(2, 3, 16, seed=2)
    y, _ = carve.conv(x, w, state=state, silu=True)
    carve.conv_step(rn(2, 16), w, state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_tensors_of_inference_mode_are_written_as_before():
    with torch.inference_mode():
        state, x, w = rn(2, 3, 16), rn(2, 16), rn(16, 4)
        want = torch.cat([state[:, 1:], x[:, None]], 1)
        carve.conv_step(x, w, state)
    assert torch.equal(state, want)
    carve.conv_step(x, w, state)  # outside of it too, as any kernel of the library
    assert torch.equal(state[:, -2], state[:, -1])


PACKED = [([40, 0, 3, 85], 0, 0), ([1] * 20, 2, 5), ([300], 0, 33)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("lengths, lead, tail", PACKED, ids=["4", "20", "1"])
def test_scan_packed(lengths, lead, tail, dtype):
    """carve.scan over a packed batch is its entry points, and sequence by
    sequence the fp64 oracle."""
    T, N, C = lead + sum(lengths) + tail, len(lengths), 24
    cu = offsets(lengths, lead)
    x, raw, d_h = (rn(T, C, seed=i, dtype=dtype) for i in (1, 2, 3))
    h0, dh_T = rn(N, C, seed=4), rn(N, C, seed=5)
    opt = dict(decay_scale=0.3, complement=True)
    leaves = [leaf(t) for t in (x, raw, h0)]
    ws = carve.scan_workspace(x, cu)
    h, h_T = carve.scan(*leaves, cu_seqlens=cu, workspace=ws, **opt)
    grads = torch.autograd.grad([h, h_T], leaves, [d_h, dh_T])
    assert carve.get_status(ws) == 0
    want, want_T, ws2 = carve.scan_fwd(x, raw, h0, cu, training=True, **opt)
    gr = carve.scan_bwd(x, raw, d_h, ws2, dh_T=dh_T, cu_seqlens=cu, **opt)
    assert torch.equal(h, want) and torch.equal(h_T, want_T)
    for got, name in zip(grads, ("dx", "dg", "dh0")):
        assert torch.equal(got, gr[name]), name
    at = lead
    for i, n in enumerate(lengths):
        args = [np64(t) for t in (x[at:at + n], raw[at:at + n], h0[i])]
        hs, last, bound = mixer.scan_fwd(*args, 0.3, True)
        close(h[at:at + n], hs, bound, "h")
        close(h_T[i], last, bound[-1] if n else 0, "h_T")
        r = mixer.scan_bwd(*args, np64(d_h[at:at + n]), np64(dh_T[i]), 0.3, True)
        close(grads[0][at:at + n], *r["dx"], "dx")
        close(grads[1][at:at + n], *r["dg"], "dg")
        close(grads[2][i], *r["dh0"], "dh0")
        at += n
    for t in (h, *grads[:2]):
        assert (t[:lead] == 0).all() and (t[T - tail:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("lengths, lead, tail", PACKED, ids=["4", "20", "1"])
def test_conv_packed(lengths, lead, tail, dtype):
    T, N, C = lead + sum(lengths) + tail, len(lengths), 24
    cu = offsets(lengths, lead)
    x, dy = rn(T, C, dtype=dtype), rn(T, C, seed=2, dtype=dtype)
    w, bias = rn(C, 4, seed=3, dtype=dtype), rn(C, seed=4, dtype=dtype)
    state, dstate_T = rn(N, 3, C, seed=5, dtype=dtype), rn(N, 3, C, seed=6, dtype=dtype)
    leaves = [leaf(t) for t in (x, w, bias, state)]
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    y, state_T = carve.conv(*leaves, cu_seqlens=cu, silu=True, workspace=ws)
    grads = torch.autograd.grad([y, state_T], leaves, [dy, dstate_T])
    assert carve.get_status(ws) == 0
    want, want_T = carve.conv_fwd(x, w, bias, state, cu, True)
    gr = carve.conv_bwd(x, w, dy, bias, state, dstate_T, cu, True)
    assert torch.equal(y, want) and torch.equal(state_T, want_T)
    for got, name in zip(grads, ("dx", "dw", "dbias", "dstate")):
        assert torch.equal(got, gr[name].to(dtype)), name
    at = lead
    for i, n in enumerate(lengths):
        args = [np64(t) for t in (x[at:at + n], w, bias, state[i])]
        ref, kept, e = mixer.conv_fwd(*args, True)
        close(y[at:at + n], ref, e, "y")
        r = mixer.conv_bwd(*args, np64(dy[at:at + n]), np64(dstate_T[i]), True)
        close(grads[0][at:at + n], *r["dx"], "dx")
        close(grads[3][i], *r["dstate"], "dstate")
        at += n
    for t in (y, grads[0]):
        assert (t[:lead] == 0).all() and (t[T - tail:] == 0).all()


def test_bad_offsets_show_in_a_workspace_handed_on():
    x, w = leaf(rn(50, 16)), rn(16, 4)
    cu = torch.tensor([0, 30, 20, 50], dtype=torch.int32, device="cuda")
    ws, wc = carve.scan_workspace(x, cu), torch.zeros(256, dtype=torch.uint8, device="cuda")
    h, _ = carve.scan(x, -x.detach().abs(), cu_seqlens=cu, workspace=ws)
    h.sum().backward()
    carve.conv(x, w, cu_seqlens=cu, workspace=wc)[0].sum().backward()
    for t in (ws, wc):
        assert carve.STATUS[carve.get_status(t)] == "CARVE_ERR_INVALID_ARG"


def test_workspace_used_again_before_the_backward_is_noticed():
    x = leaf(rn(2, 90, 16))
    g = -x.detach().abs()
    ws = carve.scan_workspace(x)
    h, _ = carve.scan(x, g, workspace=ws)
    carve.scan(x.detach(), g, workspace=ws)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        h.sum().backward()
    # without training it holds the status word alone
    small = carve.scan_workspace(x, training=False)
    assert small.numel() == 256
    h2, _ = carve.scan(x.detach(), g, workspace=small)
    assert torch.equal(h, h2) and carve.get_status(small) == 0
    with pytest.raises(ValueError, match="workspace"):
        carve.scan(x, g, workspace=small)
    with pytest.raises(carve.CarveError):
        carve.scan_workspace(x[..., :12])
