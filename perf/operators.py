"""Workloads of the operators around the chunk core: the gated linear scan,
the per-head q / k norms with the position rotation, and the short causal
convolution.

    listed(), draw(rng)   the cases (dicts of plain values)
    prepare(case, seed)   what a user's program holds before the call
    run(state)            one pass: the plain form, or, with ``own`` true,
                          the library's entry points
    exact(case, seed)     the same outputs from the definitions in fp64
    work(case)            bytes and flops one pass cannot do without

The plain forms are elementary torch operations in fp32 (fp64 for the
rotation angles), rounded once at the end.  Sequences are handled packed:
a dense batch is B sequences of T tokens laid end to end.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
TAPS = 4


def listed():
    layer = dict(B=8, T=4096, H=16, D=128, dtype="bf16")  # the 1.3B-layer shape
    return [
        # one new token for each of 8 sequences: launch latency
        dict(name="scan_step", op="scan", mode="step", B=8, T=1, H=16, D=128,
             dtype="bf16", ragged=False, raw=True, complement=True),
        # a prefill batch of 33 packed sequences of very different lengths
        dict(name="scan_packed", op="scan", mode="fwd", B=33, T=16384, H=16,
             D=128, dtype="bf16", ragged=True, raw=False, complement=False),
        # one long context: few channels, the split over time counts
        dict(name="scan_long", op="scan", mode="fwd", B=1, T=65536, H=16,
             D=128, dtype="bf16", ragged=False, raw=False, complement=False),
        # a training step of one layer, gates fused
        dict(layer, name="scan_train", op="scan", mode="train", ragged=False,
             raw=True, complement=True),
        # fp32 training at odd sizes
        dict(name="scan_train_fp32", op="scan", mode="train", B=3, T=1021,
             H=5, D=208, dtype="fp32", ragged=False, raw=False,
             complement=False),
        # q and k of one new token per sequence, far into its context
        dict(name="rope_step", op="rope", mode="fwd", B=8, T=1, HQ=16, HK=16,
             D=128, RD=128, dtype="bf16", fused=False, weights=True,
             l2norm=True, interleaved=False, first=1000003),
        # a long prefill: q and k as slices of one fused projection
        dict(name="rope_prefill", op="rope", mode="fwd", B=1, T=65536, HQ=16,
             HK=16, D=128, RD=128, dtype="bf16", fused=True, weights=True,
             l2norm=True, interleaved=False, first=0),
        # a training step of one layer
        dict(name="rope_train", op="rope", mode="train", B=8, T=4096, HQ=16,
             HK=16, D=128, RD=128, dtype="bf16", fused=False, weights=True,
             l2norm=False, interleaved=False, first=0),
        # fp32, fewer key heads than query heads, a head half rotated
        dict(name="rope_train_fp32", op="rope", mode="train", B=2, T=777,
             HQ=6, HK=2, D=80, RD=32, dtype="fp32", fused=True, weights=True,
             l2norm=False, interleaved=True, first=5),
        # one new token for each of 64 sequences, q, k and v channels together
        dict(name="conv_step", op="conv", mode="step", B=64, T=1, C=6144,
             dtype="bf16", ragged=False, silu=True, bias=True),
        # packed prefill of the same projection
        dict(name="conv_packed", op="conv", mode="fwd", B=33, T=16384, C=6144,
             dtype="bf16", ragged=True, silu=True, bias=False),
        # a training step of one layer
        dict(name="conv_train", op="conv", mode="train", B=8, T=4096, C=6144,
             dtype="bf16", ragged=False, silu=True, bias=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Sequences of one token to 65536, 1 to 64 of them, channels 16 to 6144;
    at most as many elements as the largest listed case of the operator."""
    op = rng.choice(["scan", "rope", "conv"])
    mode = rng.choice(["step", "fwd", "fwd", "train", "train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    B = _log_int(rng, 1, 64)
    D = 16 * _log_int(rng, 1, 16)
    H = _log_int(rng, 1, 24)
    cap = {"scan": 8 * 4096 * 2048, "rope": 8 * 4096 * 4096,
           "conv": 8 * 4096 * 6144}[op]
    if op == "conv":
        H, D = 1, 8 * _log_int(rng, 2, 768)
    elif op == "rope":
        hk = rng.choice([h for h in range(1, H + 1) if H % h == 0])
    heads = H + hk if op == "rope" else H
    T = _log_int(rng, 1, max(1, min(65536, cap // (2 * B * heads * D))))
    case = dict(op=op, mode=mode, B=B, T=T, dtype=dtype)
    if op == "rope":
        case.update(mode="fwd" if mode == "step" else mode, HQ=H, HK=hk, D=D,
                    T=1 if mode == "step" else T,
                    RD=16 * rng.randint(0, D // 16), fused=rng.random() < .5,
                    weights=rng.random() < .7, l2norm=rng.random() < .5,
                    interleaved=rng.random() < .5,
                    first=_log_int(rng, 1, 4000000))
        return case
    ragged = mode != "step" and rng.random() < .5
    case.update(T=1 if mode == "step" else max(T, B) if ragged else T,
                ragged=ragged)
    if ragged:  # T is the packed total
        case["T"] = max(B, min(65536, case["T"] * _log_int(rng, 1, B)))
    if op == "scan":
        case.update(H=H, D=D, raw=rng.random() < .5,
                    complement=rng.random() < .5)
    else:
        case.update(C=D, silu=rng.random() < .7, bias=rng.random() < .5)
    return case


# ---------------------------------------------------------------- inputs

def _lengths(case, gen):
    """Packed lengths: about log-uniform, one empty sequence where there are
    several, and up to 63 rows behind the last sequence."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    u = torch.rand(B, generator=gen).mul(4).exp().double()
    if B > 2:
        u[1] = 0
    rest = T % 64 if T > 64 * B else 0
    n = (u / u.sum() * (T - rest)).floor().long()
    n[0] += T - rest - int(n.sum())
    return n.tolist()


def prepare(case, seed):
    host = torch.Generator().manual_seed(int(seed))
    gen = torch.Generator("cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    randn = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    s = dict(case=case)
    if case["op"] == "rope":
        B, T, HQ, HK, D, RD = (case[k] for k in ("B", "T", "HQ", "HK", "D", "RD"))
        wide = HQ + 2 * HK if case["fused"] else 0
        if wide:
            qkv = randn(B, T, wide * D).to(dt)
            s["q"] = qkv[..., :HQ * D].view(B, T, HQ, D)
            s["k"] = qkv[..., HQ * D:(HQ + HK) * D].view(B, T, HK, D)
        else:
            s["q"], s["k"] = randn(B, T, HQ, D).to(dt), randn(B, T, HK, D).to(dt)
        ahead = torch.randint(0, 64, (B, 1), generator=host)
        s["pos"] = (case["first"] + ahead + torch.arange(T)).to(torch.int32).cuda()
        s["freqs"] = (10000.0 ** (-torch.arange(0, RD, 2, dtype=torch.float64) / max(RD, 1))).cuda()
        s["w_q"] = (1 + 0.1 * randn(D)).to(dt) if case["weights"] else None
        s["w_k"] = (1 + 0.1 * randn(D)).to(dt) if case["weights"] else None
        if case["mode"] == "train":
            s["dq"], s["dk"] = randn(B, T, HQ, D).to(dt), randn(B, T, HK, D).to(dt)
        return s
    B, T = case["B"], case["T"]
    n = _lengths(case, host)
    cu = torch.tensor([0] + n, dtype=torch.int64).cumsum(0)
    s["cu"] = cu.to(torch.int32).cuda()
    s["longest"] = max(n)
    if case["op"] == "scan":
        H, D = case["H"], case["D"]
        lead = (T,) if case["ragged"] else (B,) if case["mode"] == "step" else (B, T)
        s["x"] = randn(*lead, H, D).to(dt)
        # channels of short and of long memory
        logits = randn(*lead, H, D) + torch.linspace(-4, 1, H * D, device="cuda").view(H, D)
        s["g"] = (logits if case["raw"] else -0.1 * torch.nn.functional.softplus(logits)).to(dt)
        s["scale"] = 0.1 if case["raw"] else 0.0
        s["h0"] = randn(B, H, D)
        if case["mode"] == "train":
            s["d_h"], s["dh_T"] = randn(*lead, H, D).to(dt), randn(B, H, D)
        return s
    C = case["C"]
    lead = (T,) if case["ragged"] else (B,) if case["mode"] == "step" else (B, T)
    s["x"] = randn(*lead, C).to(dt)
    s["w"] = (randn(C, TAPS) * 0.5).to(dt)
    s["bias"] = (randn(C) * 0.1).to(dt) if case["bias"] else None
    s["state"] = randn(B, TAPS - 1, C).to(dt)
    if case["mode"] == "train":
        s["dy"] = randn(*lead, C).to(dt)
        s["dstate_T"] = randn(B, TAPS - 1, C).to(dt)
    return s


# ------------------------------------------------------- the library's calls

def _own(s):
    from chunk_gated_delta_02_b200 import carve
    c = s["case"]
    train = c["mode"] == "train"
    if c["op"] == "rope":
        opt = dict(w_q=s["w_q"], w_k=s["w_k"], l2norm=c["l2norm"],
                   interleaved=c["interleaved"])
        out = carve.qk_rope_fwd(s["q"], s["k"], s["pos"], s["freqs"], **opt)
        if not train:
            return out
        gr = carve.qk_rope_bwd(s["q"], s["k"], s["pos"], s["freqs"], s["dq"],
                               s["dk"], **opt)
        return out + tuple(gr[n] for n in ("dq", "dk", "dw_q", "dw_k"))
    cu = s["cu"] if c["ragged"] else None
    if c["op"] == "scan":
        opt = dict(decay_scale=s["scale"], complement=c["complement"])
        if c["mode"] == "step":
            return carve.scan_step(s["x"], s["g"], s["h0"], **opt), s["h0"]
        h, h_T, ws = carve.scan_fwd(s["x"], s["g"], s["h0"], cu_seqlens=cu,
                                    training=train, **opt)
        if not train:
            return h, h_T
        gr = carve.scan_bwd(s["x"], s["g"], s["d_h"], ws, dh_T=s["dh_T"],
                            cu_seqlens=cu, **opt)
        return h, h_T, gr["dx"], gr["dg"], gr["dh0"]
    if c["mode"] == "step":
        return carve.conv_step(s["x"], s["w"], s["state"], s["bias"],
                               silu=c["silu"]), s["state"]
    y, state_T = carve.conv_fwd(s["x"], s["w"], s["bias"], s["state"],
                                cu_seqlens=cu, silu=c["silu"])
    if not train:
        return y, state_T
    gr = carve.conv_bwd(s["x"], s["w"], s["dy"], s["bias"], s["state"],
                        dstate_T=s["dstate_T"], cu_seqlens=cu, silu=c["silu"])
    return y, state_T, gr["dx"], gr["dw"], gr["dbias"], gr["dstate"]


# ------------------------------------------------------------ the plain forms

def _rotation(pos, freqs):
    """cos and sin of pos * freqs, the angle in fp64: [..., 1, RD / 2]."""
    angle = pos.double().unsqueeze(-1) * freqs
    return angle.cos().float().unsqueeze(-2), angle.sin().float().unsqueeze(-2)


def _halves(x, rd, interleaved):
    return (x[..., 0:rd:2], x[..., 1:rd:2]) if interleaved else (x[..., :rd // 2], x[..., rd // 2:rd])


def _rotate(x, cos, sin, interleaved):
    rd = 2 * cos.shape[-1]
    a, b = _halves(x, rd, interleaved)
    y = x.clone()
    ya, yb = _halves(y, rd, interleaved)
    ya.copy_(a * cos - b * sin)
    yb.copy_(a * sin + b * cos)
    return y


def _inverse_norm(x, l2norm, eps=1e-6):
    ss = x.square().sum(-1, keepdim=True)
    return torch.rsqrt((ss if l2norm else ss / x.shape[-1]) + eps)


def _plain_rope(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    cos, sin = _rotation(s["pos"], s["freqs"])

    def forward(x, w):
        x = x.float()
        y = x * _inverse_norm(x, c["l2norm"])
        return _rotate(y if w is None else y * w.float(), cos, sin, c["interleaved"]).to(dt)

    def backward(x, w, d):
        x, d = x.float(), _rotate(d.float(), cos, -sin, c["interleaved"])
        r = _inverse_norm(x, c["l2norm"])
        dw = None if w is None else (d * x * r).sum((0, 1, 2))
        d = d if w is None else d * w.float()
        dot = (d * x).sum(-1, keepdim=True) * r * r
        return (r * (d - x * (dot if c["l2norm"] else dot / x.shape[-1]))).to(dt), dw

    out = forward(s["q"], s["w_q"]), forward(s["k"], s["w_k"])
    if c["mode"] != "train":
        return out
    dq, dwq = backward(s["q"], s["w_q"], s["dq"])
    dk, dwk = backward(s["k"], s["w_k"], s["dk"])
    return out + (dq, dk, dwq, dwk)


def _scan_in_place(a, b, longest):
    """b_t <- a_t b_{t-1} + b_t over dim 0 by doubling (a is used up)."""
    d = 1
    while d < longest:
        b[d:] += a[d:] * b[:-d]
        a[d:] = a[d:] * a[:-d]
        d *= 2
    return b


def _decay(g, scale):
    """exp of the log-decay, 1 minus it, and d(log-decay) / dg."""
    if not scale:
        return g.exp(), -torch.expm1(g), None
    u = -scale * torch.nn.functional.softplus(g)
    return u.exp(), -torch.expm1(u), -scale * torch.sigmoid(g)


def _plain_scan(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    x, g = s["x"].float(), s["g"].float()
    a, rest, slope = _decay(g, s["scale"])
    if c["mode"] == "step":
        s["h0"].copy_(a * s["h0"] + (rest * x if c["complement"] else x))
        return s["h0"].to(dt), s["h0"]
    shape, row = x.shape, x.shape[-2:]
    a, x, rest = a.reshape(-1, *row), x.reshape(-1, *row), rest.reshape(-1, *row)
    cu = s["cu"].long()
    some = (cu[1:] > cu[:-1]).nonzero().flatten()  # sequences that are not empty
    first, last = cu[:-1][some], cu[1:][some] - 1
    end = int(cu[-1])
    xi = rest * x if c["complement"] else x.clone()
    xi[first] += a[first] * s["h0"][some]
    ac = a.clone()
    ac[first] = 0
    ac[end:] = 0  # rows of no sequence: no state runs on through them
    xi[end:] = 0
    h = _scan_in_place(ac, xi, s["longest"])
    h_T = s["h0"].clone()
    h_T[some] = h[last]
    if c["mode"] == "fwd":
        return h.to(dt).view(shape), h_T
    # lambda_t = d_h_t + a_{t+1} lambda_{t+1}, the scan of the reversed axis
    lam = s["d_h"].float().reshape(-1, *row).clone()
    lam[end:] = 0
    lam[last] += s["dh_T"][some]
    an = torch.zeros_like(a)
    an[:-1] = a[1:]
    an[last] = 0
    lam = _scan_in_place(an.flip(0), lam.flip(0), s["longest"]).flip(0)
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[first] = s["h0"][some]
    dx = lam * rest if c["complement"] else lam
    dg = a * lam * (before - x if c["complement"] else before)
    if slope is not None:
        dg = dg * slope.reshape(-1, *row)
    dg[end:] = 0
    dh0 = s["dh_T"].clone()
    dh0[some] = a[first] * lam[first]
    return h.to(dt).view(shape), h_T, dx.to(dt).view(shape), dg.to(dt).view(shape), dh0


def _silu(z):
    return z * torch.sigmoid(z)


def _plain_conv(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    w, taps = s["w"].float(), s["w"].shape[1]
    bias = 0.0 if s["bias"] is None else s["bias"].float()
    state = s["state"]
    n, cu = state.shape[0], s["cu"].long()
    x = s["x"].float()
    if c["mode"] == "step":
        window = torch.cat([state.float(), x.unsqueeze(1)], 1)
        z = (window * w.t()).sum(1) + bias
        state.copy_(window[:, 1:])
        return (_silu(z) if c["silu"] else z).to(dt), state
    shape, C = x.shape, x.shape[-1]
    # rows of the inputs, then of the states; tap j of token t reads row at[j, t]
    rows = torch.cat([x.reshape(-1, C), state.float().reshape(-1, C)])
    total = rows.shape[0] - n * (taps - 1)
    end = int(cu[-1])
    t = torch.arange(end, device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True)
    where = lambda p, q, begin: torch.where(p >= begin, p, total + q * (taps - 1) + p - begin + taps - 1)  # noqa: E731
    at = [where(t - taps + 1 + j, seq, cu[seq]) for j in range(taps)]
    back = torch.arange(1 - taps, 0, device="cuda")
    kept = where(cu[1:, None] + back, torch.arange(n, device="cuda")[:, None], cu[:-1, None])
    z = sum(w[:, j] * rows[at[j]] for j in range(taps)) + bias
    y = torch.zeros(total, C, device="cuda")
    y[:end] = _silu(z) if c["silu"] else z
    out = y.to(dt).view(shape), rows[kept].to(dt)
    if c["mode"] == "fwd":
        return out
    dz = s["dy"].float().reshape(-1, C)[:end]
    if c["silu"]:
        sg = torch.sigmoid(z)
        dz = dz * sg * (1 + z * (1 - sg))
    dw = torch.stack([(dz * rows[at[j]]).sum(0) for j in range(taps)], 1)
    drows = torch.zeros_like(rows)
    drows.index_add_(0, kept.flatten(), s["dstate_T"].float().reshape(-1, C))
    for j in range(taps):
        drows[at[j]] += w[:, j] * dz
    return out + (drows[:total].to(dt).view(shape), dw,
                  None if s["bias"] is None else dz.sum(0),
                  drows[total:].to(dt).view(n, taps - 1, C))


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "scan": _plain_scan, "conv": _plain_conv}[state["case"]["op"]](state)


# --------------------------------------------------------- fp64 definitions

def _exact_rope(s):
    c = s["case"]
    D, RD = c["D"], c["RD"]
    ang = (s["pos"].double()[..., None] * s["freqs"]).unsqueeze(-2)
    rot = torch.polar(torch.ones_like(ang), ang)  # unit complex numbers

    def pairs(x):
        p = x[..., :RD]
        p = p.unflatten(-1, (RD // 2, 2)) if c["interleaved"] else p.unflatten(-1, (2, RD // 2)).transpose(-1, -2)
        return torch.view_as_complex(p.contiguous())

    def turned(x, r):
        if not RD:
            return x
        p = torch.view_as_real(pairs(x) * r)
        p = p.flatten(-2) if c["interleaved"] else p.transpose(-1, -2).flatten(-2)
        return torch.cat([p, x[..., RD:]], -1)

    def one(x, w, d):
        x = x.double()
        w = 1.0 if w is None else w.double()
        size = (x.pow(2).sum(-1, keepdim=True) / (1 if c["l2norm"] else D) + 1e-6).sqrt()
        unit = x / size
        y = turned(unit * w, rot)
        if d is None:
            return y, None, None
        dn = turned(d.double(), rot.conj())
        du = dn * w
        along = (du * unit).sum(-1, keepdim=True) / (1 if c["l2norm"] else D)
        return y, (du - unit * along) / size, (dn * unit).flatten(0, 2).sum(0)

    yq, dq, dwq = one(s["q"], s["w_q"], s.get("dq"))
    yk, dk, dwk = one(s["k"], s["w_k"], s.get("dk"))
    if c["mode"] != "train":
        return yq, yk
    return yq, yk, dq, dk, dwq if c["weights"] else None, dwk if c["weights"] else None


def _table(s):
    """Token rows as a [longest, sequences] table: row numbers and a mask."""
    cu = s["cu"].long()
    t = torch.arange(s["longest"], device="cuda")[:, None]
    live = t < (cu[1:] - cu[:-1])
    return torch.where(live, cu[:-1] + t, 0), live


def _exact_scan(s):
    c = s["case"]
    if c["mode"] == "step":
        at = torch.arange(c["B"], device="cuda")[None]
        live = torch.ones_like(at, dtype=torch.bool)
    else:
        at, live = _table(s)
    row = s["x"].shape[-2:]
    flat = lambda v: v.reshape(-1, *row)  # noqa: E731
    xs, gs = flat(s["x"]), flat(s["g"])
    scale, live = s["scale"], live[..., None, None]

    def token(t):
        raw, x = gs[at[t]].double(), xs[at[t]].double()
        u = -scale * torch.logaddexp(raw, torch.zeros_like(raw)) if scale else raw
        return raw, u, x

    h, keep = s["h0"].double(), torch.empty(len(at), *s["h0"].shape, device="cuda", dtype=torch.float64)
    for t in range(len(at)):
        raw, u, x = token(t)
        keep[t] = h
        h = torch.where(live[t], torch.exp(u) * h - (torch.expm1(u) * x if c["complement"] else -x), h)
    if c["mode"] == "step":
        return h, h
    ys = torch.cat([keep[1:], h[None]])
    out = torch.zeros(xs.shape, device="cuda", dtype=torch.float64)
    mask = live[..., 0, 0]
    out[at[mask]] = ys[mask]
    if c["mode"] == "fwd":
        return out.view(s["x"].shape), h
    dx, dg = torch.zeros_like(out), torch.zeros_like(out)
    ds, back = flat(s["d_h"]), s["dh_T"].double()
    for t in reversed(range(len(at))):
        raw, u, x = token(t)
        lam = back + ds[at[t]].double()
        m = live[t, :, 0, 0]
        i = at[t][m]
        dx[i] = (-torch.expm1(u) * lam if c["complement"] else lam)[m]
        d = torch.exp(u) * lam * (keep[t] - x if c["complement"] else keep[t])
        dg[i] = (d * (-scale / (1 + torch.exp(-raw))) if scale else d)[m]
        back = torch.where(live[t], torch.exp(u) * lam, back)
    return out.view(s["x"].shape), h, dx.view(s["x"].shape), dg.view(s["x"].shape), back


def _exact_conv(s):
    c = s["case"]
    w, n, C = s["w"].double(), c["B"], c["C"]
    bias = 0.0 if s["bias"] is None else s["bias"].double()
    act = (lambda z: z / (1 + torch.exp(-z))) if c["silu"] else (lambda z: z)
    slope = (lambda z: (1 + torch.exp(-z) * (1 + z)) / (1 + torch.exp(-z)) ** 2) if c["silu"] else torch.ones_like
    if c["mode"] == "step":
        rows = torch.cat([s["state"].double(), s["x"].double()[:, None]], 1)
        return act(torch.einsum("btc,ct->bc", rows, w) + bias), rows[:, 1:]
    xs = s["x"].reshape(-1, C)
    train = c["mode"] == "train"
    y = torch.zeros(xs.shape, device="cuda", dtype=torch.float64)
    kept, dstate = [], []
    dx = torch.zeros_like(y) if train else None
    dw, db = torch.zeros_like(w), torch.zeros(C, device="cuda", dtype=torch.float64)
    cu = s["cu"].tolist()
    for i in range(n):  # one sequence at a time, its state before it
        rows = torch.cat([s["state"][i], xs[cu[i]:cu[i + 1]]]).double()
        T = cu[i + 1] - cu[i]
        z = torch.nn.functional.conv1d(rows.t()[None], w[:, None], groups=C)[0].t() + bias if T else rows[:0]
        y[cu[i]:cu[i + 1]] = act(z)
        kept.append(rows[T:])
        if train:
            dz = s["dy"].reshape(-1, C)[cu[i]:cu[i + 1]].double() * slope(z)
            dr = torch.zeros_like(rows)
            dr[T:] = s["dstate_T"][i].double()
            for j in range(TAPS):
                dr[j:j + T] += w[:, j] * dz
                dw[:, j] += (rows[j:j + T] * dz).sum(0)
            db += dz.sum(0)
            dx[cu[i]:cu[i + 1]] = dr[TAPS - 1:]
            dstate.append(dr[:TAPS - 1])
    out = y.view(s["x"].shape), torch.stack(kept)
    if not train:
        return out
    return out + (dx.view(s["x"].shape), dw, None if s["bias"] is None else db, torch.stack(dstate))


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "scan": _exact_scan, "conv": _exact_conv}[case["op"]](s)


# ---------------------------------------------------------------- the work

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    train = case["mode"] == "train"
    B, T = case["B"], case["T"]
    if case["op"] == "rope":
        e = B * T * (case["HQ"] + case["HK"]) * case["D"]
        # q, k (and their output gradients) in; outputs (and gradients) out
        return {"bytes": e * size * (4 if train else 2) + 4 * B * T,
                "flops": e * (18 if train else 7)}
    tokens = T if case["ragged"] or case["mode"] == "step" else B * T
    tokens = B if case["mode"] == "step" else tokens
    if case["op"] == "scan":
        C = case["H"] * case["D"]
        state = 8 * B * C * (2 if train else 1)
        return {"bytes": tokens * C * size * (6 if train else 3) + state,
                "flops": tokens * C * (12 if train else 4)}
    C = case["C"]
    state = 2 * B * (TAPS - 1) * C * size * (2 if train else 1)
    return {"bytes": tokens * C * size * (4 if train else 2) + state + C * (TAPS + 1) * size,
            "flops": tokens * C * (12 + 30 * train)}
