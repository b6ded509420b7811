"""GPU: the operators around the core under autograd: tensors that a later
call overwrites, packed batches, workspaces handed on by the wrappers."""
import pytest
import torch

from chunk_gated_delta_02_b200 import carve

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
