"""GPU: the status word that the operators around the core leave in a
workspace (no GPU fault is involved: bounded waits run out through the
test-only knobs of the library, on good memory)."""
import pytest
import torch

from chunk_gated_delta_02_b200 import carve

from _mixer import offsets

pytestmark = pytest.mark.gpu


def status(ws):
    return carve.STATUS[carve.get_status(ws)]


def rn(*shape, dtype=torch.float32, seed=1):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=gen).to(dtype).cuda()


def stall(monkeypatch, on):
    """Block 1 keeps its pair of tile 1 to itself: its cluster's waits run out
    after 2e5 cycles."""
    for name, value in (("CARVE_TEST_WAIT_CYCLES", "200000"), ("CARVE_TEST_STALL_BLOCK", "1")):
        monkeypatch.setenv(name, value) if on else monkeypatch.delenv(name)


@pytest.mark.parametrize("packed", [False, True], ids=["dense", "packed"])
def test_backward_keeps_the_forwards_error(monkeypatch, packed):
    x, g = rn(1, 4096, 64), -0.1 * rn(1, 4096, 64, seed=2).abs()
    cu = None
    if packed:
        x, g, cu = x[0], g[0], offsets([4096])
    stall(monkeypatch, True)
    _, _, ws = carve.scan_fwd(x, g, cu_seqlens=cu, training=True)
    torch.cuda.synchronize()
    stall(monkeypatch, False)
    gr = carve.scan_bwd(x, g, x, ws, cu_seqlens=cu)
    assert status(ws) == "CARVE_ERR_TIMEOUT"
    assert gr["dg"].isnan().any()  # of the states that the forward kept
    # a forward starts anew
    carve.scan_fwd(x, g, cu_seqlens=cu, training=True, workspace=ws)
    carve.scan_bwd(x, g, x, ws, cu_seqlens=cu)
    assert status(ws) == "CARVE_OK"


def used(n=256):
    """A workspace that something else has been in."""
    return torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")


def test_inference_scan_reports_to_a_workspace_it_is_given(monkeypatch):
    x, g, ws = rn(1, 4096, 64), -0.1 * rn(1, 4096, 64, seed=2).abs(), used()
    stall(monkeypatch, True)
    h, _, got = carve.scan_fwd(x, g, workspace=ws)
    torch.cuda.synchronize()
    stall(monkeypatch, False)
    assert got is ws and h.isnan().any() and status(ws) == "CARVE_ERR_TIMEOUT"
    h, _, _ = carve.scan_fwd(x, g, workspace=ws)
    assert h.isfinite().all() and status(ws) == "CARVE_OK"
    empty, ws = x[:, :0], used()
    carve.scan_fwd(empty, empty, workspace=ws)
    assert status(ws) == "CARVE_OK"
    for bad in (used(255), ws.cpu()):
        with pytest.raises(ValueError, match="workspace"):
            carve.scan_fwd(x, g, workspace=bad)
    with pytest.raises(carve.CarveError, match="WORKSPACE"):  # not on 16 bytes
        carve.scan_fwd(x, g, workspace=used(264)[8:])


@pytest.mark.parametrize("T", [0, 30])
@pytest.mark.parametrize("packed", [False, True], ids=["dense", "packed"])
def test_convolution_writes_the_word(packed, T):
    x, w, cu = rn(2, T, 16), rn(16, 4), None
    if packed:
        x, cu = x.reshape(2 * T, 16), offsets([T, T])
    size = carve.lib().carve_conv_workspace_bytes
    shape = carve.ConvShape(2, x.shape[-2], 16, 4, carve.CARVE_FP32, 0, 0, 0, 0)
    ws, wb = used(size(shape, int(packed), 0)), used(size(shape, int(packed), 1))
    y, _ = carve.conv_fwd(x, w, cu_seqlens=cu, workspace=ws)
    assert status(ws) == "CARVE_OK" and y.shape == x.shape
    gr = carve.conv_bwd(x, w, x, cu_seqlens=cu, workspace=wb)
    assert status(wb) == "CARVE_OK"
    assert T or (gr["dw"] == 0).all()


def test_convolution_without_tokens_captured():
    """A copy and a memset in front of a kernel."""
    x, w, s = rn(2, 0, 16), rn(16, 4), rn(2, 3, 16)
    ws, wb = used(), used(4096)
    call = lambda: (carve.conv_fwd(x, w, None, s, workspace=ws)[1],  # noqa: E731
                    carve.conv_bwd(x, w, x, None, s, 2 * s, workspace=wb))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        state, gr = call()
    for t in (state, gr["dstate"], gr["dw"]):
        t.fill_(7)
    for t in (ws, wb):
        t.fill_(0x55)
    graph.replay()
    assert torch.equal(state, s) and torch.equal(gr["dstate"], 2 * s) and (gr["dw"] == 0).all()
    assert status(ws) == status(wb) == "CARVE_OK"


@pytest.mark.parametrize("N", [0, 50])
def test_rotations_backward_writes_the_word(N):
    """Through the C entry point: the binding keeps this workspace to itself."""
    lib, f32 = carve.lib(), carve.CARVE_FP32
    q, w, d = rn(N, 2, 32), rn(32, seed=2), rn(N, 2, 32, seed=3)
    want = carve.qk_rope_bwd(q, None, None, None, d, None, w)
    shape = carve.RopeShape(N, 2, 0, 32, 0, f32, 1e-6, 0, 0, 0, 0)
    ws = used(lib.carve_qk_rope_workspace_bytes(shape) + 256)
    dq, dw = torch.empty_like(q), torch.empty(32, device="cuda")
    p = lambda t: t.data_ptr() or None  # noqa: E731
    rc = lib.carve_qk_rope_bwd(shape, p(q), None, None, None, p(w), None, p(d), None, p(ws),
                               ws.numel() - 256, p(dq), None, p(dw), None,
                               torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and status(ws) == "CARVE_OK"
    assert torch.equal(dq, want["dq"]) and torch.equal(dw, want["dw_q"])
    assert (ws[-256:] == 0x55).all()


def test_workspace_over_an_input_is_refused():
    """One allocation, seen as bytes and as what a call reads."""
    raw = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    x = raw[4096:4096 + 2 * 70 * 16 * 4].view(torch.float32).view(2, 70, 16)
    clear, w = rn(2, 70, 16), rn(16, 4)
    over, beside = raw[:8192], raw[40000:]
    state = raw[:2 * 3 * 16 * 4].view(torch.float32).view(2, 3, 16)
    calls = [lambda ws: carve.scan_fwd(x, clear, workspace=ws),
             lambda ws: carve.scan_fwd(clear, x, training=True, workspace=ws),
             lambda ws: carve.conv_fwd(x, w, workspace=ws),
             lambda ws: carve.conv_fwd(clear, w, state=state, workspace=ws),
             lambda ws: carve.conv_bwd(clear, w, x, workspace=ws),
             lambda ws: carve.conv_bwd(clear, w, clear, state=state, workspace=ws),
             lambda ws: carve.scan_bwd(clear, -clear.abs(), x, ws)]
    carve.scan_fwd(clear, -clear.abs(), training=True, workspace=beside)
    for call in calls:
        with pytest.raises(ValueError, match="workspace overlaps"):
            call(over)
        call(beside)
