"""dma_prep and dma_prep_bwd on the GPU against the formula in float64.

Tolerances, from the arithmetic.  With u = 2^-24 (half a step of float32): the square sum of d <= 128
terms (tree of 8 sequential terms and 4 levels) is off by at most 13 u, the root by half of that and two
roundings more, the products with the norm factor and weight by 3 u, the angle's cos and sin by 2 u in
absolute terms (of |cos|, |sin| <= 1), the two products and the sum of the rotation by 3 u.  A rotated
channel is therefore within 20 u of |a| + |b|, the pair's members; an output is then rounded once: half
a step of its type, relative (bf16 2^-8, float32 2^-24).  The backward's row adds a second sum of the
same length, against the sum of its terms' magnitudes: 40 u of the row's magnitudes covers it."""
import numpy as np
import pytest

from gpu_common import lib, torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _types(dtype):
    torch = torch_cuda()
    return torch, torch.bfloat16 if dtype == "bf16" else torch.float32


def _rotation(pos, freq, inter, d):
    """R [tokens, d, d] in float64."""
    rot = 2 * freq.shape[0]
    R = np.zeros(pos.shape + (d, d))
    R[..., np.arange(d), np.arange(d)] = 1.0
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        ang = pos.astype(np.float64) * np.float64(freq[i])
        R[..., a, a] = R[..., b, b] = np.cos(ang)
        R[..., b, a], R[..., a, b] = np.sin(ang), -np.sin(ang)
    return R


def _forward(x, w, R, eps):
    """x [B, N, heads, d] float64 -> (out, magnitude of what was summed) [B, N, heads, d]."""
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return np.einsum("bnij,bnhj->bnhi", R, y), np.einsum("bnij,bnhj->bnhi", np.abs(R), np.abs(y))


def _backward(x, w, R, eps, dy):
    g = np.einsum("bnji,bnhj->bnhi", R, dy)
    gm = np.einsum("bnji,bnhj->bnhi", np.abs(R), np.abs(dy))
    if w is None:
        return g, gm, None, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dx = r * (g * w) - x * r ** 3 * (x * g * w).mean(-1, keepdims=True)
    mag = r * (gm * np.abs(w)) + np.abs(x) * r ** 3 * (np.abs(x) * gm * np.abs(w)).mean(-1, keepdims=True)
    return dx, mag, (g * x * r).sum((0, 1, 2)), (gm * np.abs(x) * r).sum((0, 1, 2))


def _np(t):
    return t.double().cpu().numpy()


def _freq(torch, rot, base=10000.0):
    if rot == 0:
        return None
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def _case(B, N, H, Hkv, d, dtype, rot, inter, qn, kn, layout="packed", pos=None, seed=0, scale=1.0):
    torch, t = _types(dtype)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g, device="cuda") * scale

    if layout == "packed":         # one projection: [B, N, H + 2 Hkv, d]
        qkv = normal(B, N, H + 2 * Hkv, d).to(t)
        q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    elif layout == "heads":        # head-major: [B, heads, N, d]
        q, k, v = (normal(B, h, N, d).to(t).transpose(1, 2) for h in (H, Hkv, Hkv))
    else:                          # positions outermost: [N, B, heads, d], rows with a gap behind them
        q, k, v = (normal(N, B, h, d + 64).to(t)[..., :d].transpose(0, 1) for h in (H, Hkv, Hkv))
    qw = (1 + 0.1 * normal(d)).to(t) if qn else None
    kw = (1 + 0.1 * normal(d)).to(t) if kn else None
    if pos == "far":
        pos = torch.randint(-5, 1 << 24, (B, N), generator=g, device="cuda", dtype=torch.int32)
    return dict(q=q, k=k, v=v, qw=qw, kw=kw, pos=pos, freq=_freq(torch, rot), inter=inter, t=t, torch=torch,
                normal=normal, rot=rot)


def _R(c, B, N, d, first=0):
    pos = c["pos"].cpu().numpy() if c["pos"] is not None else np.broadcast_to(first + np.arange(N), (B, N))
    freq = c["freq"].cpu().numpy() if c["rot"] else np.zeros(0, np.float32)
    return _rotation(pos, freq, c["inter"], d)


CASES = [
    # B, N, H, Hkv, d, dtype, rot, inter, q norm, k norm, layout, pos
    (1, 1, 2, 1, 64, "bf16", 64, False, True, True, "packed", None),
    (2, 3, 32, 8, 128, "bf16", 128, False, True, True, "packed", "far"),
    (1, 9, 16, 8, 128, "bf16", 128, True, True, True, "heads", None),
    (3, 37, 6, 2, 64, "f32", 48, True, True, True, "packed", "far"),
    (2, 130, 7, 7, 128, "f32", 112, False, True, False, "gaps", "far"),
    (1, 77, 12, 4, 64, "bf16", 16, False, False, True, "heads", None),
    (2, 41, 5, 1, 128, "bf16", 0, False, True, True, "gaps", None),
    (1, 19, 3, 3, 64, "f32", 0, True, False, False, "packed", None),
    (1, 2100, 2, 1, 64, "bf16", 32, True, True, True, "packed", None),
]


@pytest.mark.parametrize("B,N,H,Hkv,d,dtype,rot,inter,qn,kn,layout,pos", CASES)
def test_forward(B, N, H, Hkv, d, dtype, rot, inter, qn, kn, layout, pos):
    dma = lib()
    c = _case(B, N, H, Hkv, d, dtype, rot, inter, qn, kn, layout, pos, seed=N)
    torch, t = c["torch"], c["t"]
    p = dma.make_params(B, H, Hkv, N, d, 1, dtype=dtype)
    r = dma.make_prep(c["freq"], c["qw"], c["kw"], eps=1e-5, positions=c["pos"], first=11, interleaved=inter)
    Q = torch.full((B, H, N, d), float("nan"), dtype=t, device="cuda")
    K = torch.full((B, Hkv, N, d), float("nan"), dtype=t, device="cuda")
    V = torch.full((B, Hkv, N, d), float("nan"), dtype=t, device="cuda")
    dma.prep(p, r, c["q"], c["k"], c["v"], Q, K, V)
    torch.cuda.synchronize()
    assert torch.equal(V, c["v"].transpose(1, 2))
    R = _R(c, B, N, d, first=11)
    for got, x, w in ((Q, c["q"], c["qw"]), (K, c["k"], c["kw"])):
        ref, mag = _forward(_np(x), None if w is None else _np(w), R, np.float64(np.float32(1e-5)))
        err = np.abs(_np(got).transpose(0, 2, 1, 3) - ref)
        assert (err <= HALF[dtype] * np.abs(ref) + 20 * U * mag * (1 + HALF[dtype])).all(), err.max()


@pytest.mark.parametrize("B,N,H,Hkv,d,dtype,rot,inter,qn,kn,layout,pos", CASES)
def test_backward(B, N, H, Hkv, d, dtype, rot, inter, qn, kn, layout, pos):
    dma = lib()
    c = _case(B, N, H, Hkv, d, dtype, rot, inter, qn, kn, layout, pos, seed=N + 1)
    torch, t = c["torch"], c["t"]
    p = dma.make_params(B, H, Hkv, N, d, 1, dtype=dtype)
    r = dma.make_prep(c["freq"], c["qw"], c["kw"], eps=1e-5, positions=c["pos"], first=11, interleaved=inter)
    dQ, dK, dV = (c["normal"](B, h, N, d).to(t) for h in (H, Hkv, Hkv))
    dVg = c["normal"](B, Hkv, N, d)
    wide = torch.full((B, N, H + 2 * Hkv, d + 64), -77.0, dtype=t, device="cuda")   # gaps must stay
    gq, gk, gv = wide[:, :, :H, :d], wide[:, :, H:H + Hkv, :d], wide[:, :, H + Hkv:, :d]
    dqw = torch.full((d,), float("nan"), device="cuda") if qn else None
    dkw = torch.full((d,), float("nan"), device="cuda") if kn else None
    ws = dma.alloc_prep_workspace(p, r)
    q, k = c["q"] if qn else None, c["k"] if kn else None
    dma.prep_bwd(p, r, q, k, dQ, dK, dV, dVg, gq, gk, gv, dqw, dkw, ws)
    torch.cuda.synchronize()
    assert (wide[..., d:] == -77.0).all()
    R = _R(c, B, N, d, first=11)
    for got, x, w, dy, gw in ((gq, c["q"], c["qw"], dQ, dqw), (gk, c["k"], c["kw"], dK, dkw)):
        ref, mag, rw, mw = _backward(_np(x), None if w is None else _np(w), R, np.float64(np.float32(1e-5)),
                                     _np(dy).transpose(0, 2, 1, 3))
        err = np.abs(_np(got) - ref)
        assert (err <= HALF[dtype] * np.abs(ref) + 40 * U * mag * (1 + HALF[dtype])).all(), err.max()
        if gw is not None:
            # a lane adds up to rows / lanes terms one after the other; here at most 2100 * 2 rows in all
            assert (np.abs(_np(gw) - rw) <= (40 + B * N * 2) * U * mw).all()
    ref = _np(dV).transpose(0, 2, 1, 3) + _np(dVg).transpose(0, 2, 1, 3)
    assert (np.abs(_np(gv) - ref) <= (HALF[dtype] + U) * np.abs(ref)).all()
    # again, without the gate's share, the weights' gradients or the values: the rows keep their bits
    first = wide.clone()
    dma.prep_bwd(p, r, q, k, dQ, dK, None, None, gq, gk, None, None, None, ws)
    assert torch.equal(wide, first)
    dma.prep_bwd(p, r, q, k, dQ, dK, dV, None, gq, gk, gv, None, None, ws)
    assert torch.equal(gv, dV.transpose(1, 2))


def test_gradient_against_differences():
    """Directional differences of the formula in float64 against the kernel's float32 gradients."""
    dma = lib()
    B, N, H, Hkv, d = 1, 5, 2, 1, 64
    c = _case(B, N, H, Hkv, d, "f32", 32, False, True, True, seed=3)
    torch = c["torch"]
    p = dma.make_params(B, H, Hkv, N, d, 1, dtype="f32")
    r = dma.make_prep(c["freq"], c["qw"], c["kw"], eps=1e-5)
    dQ, dK = c["normal"](B, H, N, d), c["normal"](B, Hkv, N, d)
    gq, gk = torch.empty(B, N, H, d, device="cuda"), torch.empty(B, N, Hkv, d, device="cuda")
    dqw, dkw = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    dma.prep_bwd(p, r, c["q"], c["k"], dQ, dK, None, None, gq, gk, None, dqw, dkw, dma.alloc_prep_workspace(p, r))
    R = _R(c, B, N, d)
    rng = np.random.default_rng(0)
    for x, w, dy, gx, gw in ((c["q"], c["qw"], dQ, gq, dqw), (c["k"], c["kw"], dK, gk, dkw)):
        x, w, dy = _np(x), _np(w), _np(dy).transpose(0, 2, 1, 3)
        ux, uw, h = rng.standard_normal(x.shape), rng.standard_normal(w.shape), 1e-5

        def f(s):
            return (_forward(x + s * ux, w + s * uw, R, np.float64(np.float32(1e-5)))[0] * dy).sum()
        diff = (f(h) - f(-h)) / (2 * h)
        terms = np.concatenate([(_np(gx) * ux).ravel(), (_np(gw) * uw).ravel()])
        _, mag, _, mw = _backward(x, w, R, np.float64(np.float32(1e-5)), dy)
        # the kernel's rounding as above; the differences' own error (h^2 of the third derivative, 2^-53 / h
        # of the sum's terms) is below 1e-8 of the terms
        tol = 40 * U * (mag * np.abs(ux)).sum() + (40 + 2 * N * B) * U * (mw * np.abs(uw)).sum()
        assert abs(diff - terms.sum()) <= tol + 1e-8 * np.abs(terms).sum()


def test_sums_do_not_depend_on_the_run_and_rows_of_zeros():
    dma = lib()
    B, N, H, Hkv, d = 2, 3000, 8, 8, 64
    c = _case(B, N, H, Hkv, d, "bf16", 64, False, True, True, seed=9)
    torch = c["torch"]
    c["q"][:, ::3] = 0
    p = dma.make_params(B, H, Hkv, N, d, 1)
    r = dma.make_prep(c["freq"], c["qw"], c["kw"], eps=1e-6)
    out = [torch.empty((B, h, N, d), dtype=c["t"], device="cuda") for h in (H, Hkv, Hkv)]
    dma.prep(p, r, c["q"], c["k"], c["v"], *out)
    assert (out[0][:, :, ::3] == 0).all() and torch.isfinite(out[0].float()).all()
    ws = dma.alloc_prep_workspace(p, r)
    grads = []
    for _ in range(3):
        g = [torch.empty_like(c["q"]), torch.empty_like(c["k"]), torch.empty(d, device="cuda"),
             torch.empty(d, device="cuda")]
        dma.prep_bwd(p, r, c["q"], c["k"], out[0], out[1], None, None, g[0], g[1], None, g[2], g[3], ws)
        grads.append(g)
        ws.fill_(255)
    for g in grads[1:]:
        for a, b in zip(g, grads[0]):
            assert torch.equal(a, b)
    assert all(torch.isfinite(x.float()).all() for x in grads[0])


def test_values_pass_bit_for_bit_and_unrotated_channels_keep_infinities():
    dma = lib()
    torch, t = _types("bf16")
    B, N, H, Hkv, d = 1, 4, 2, 1, 64
    qkv = torch.randn(B, N, H + 2 * Hkv, d, device="cuda").to(t)
    qkv[0, 1, :, 40] = float("inf")
    qkv[0, 2, 3, 0] = float("nan")
    p = dma.make_params(B, H, Hkv, N, d, 1)
    r = dma.make_prep(_freq(torch, 32))
    out = [torch.empty((B, h, N, d), dtype=t, device="cuda") for h in (H, Hkv, Hkv)]
    dma.prep(p, r, qkv[:, :, :H], qkv[:, :, H:H + 1], qkv[:, :, H + 1:], *out)
    assert torch.equal(out[2].view(torch.int16), qkv[:, :, H + 1:].transpose(1, 2).contiguous().view(torch.int16))
    for o in out[:2]:
        assert (o[0, :, 1, 40] == float("inf")).all()
        rest = o[0, :, 1].clone()
        rest[:, 40] = 0
        assert torch.isfinite(rest.float()).all()


def test_other_stream_and_captured_graph():
    dma = lib()
    B, N, H, Hkv, d = 2, 65, 4, 2, 128
    c = _case(B, N, H, Hkv, d, "bf16", 128, False, True, True, seed=4)
    torch, t = c["torch"], c["t"]
    p = dma.make_params(B, H, Hkv, N, d, 1)
    r = dma.make_prep(c["freq"], c["qw"], c["kw"])
    ws = dma.alloc_prep_workspace(p, r)

    def bufs():
        return ([torch.zeros((B, h, N, d), dtype=t, device="cuda") for h in (H, Hkv, Hkv)],
                [torch.zeros((B, N, h, d), dtype=t, device="cuda") for h in (H, Hkv, Hkv)],
                [torch.zeros(d, device="cuda") for _ in range(2)])

    def both(o, g, w, stream=None):
        dma.prep(p, r, c["q"], c["k"], c["v"], *o, stream=stream)
        dma.prep_bwd(p, r, c["q"], c["k"], *o, None, *g, *w, ws, stream=stream)

    want = bufs()
    both(*want)
    torch.cuda.synchronize()
    other = bufs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    both(*other, stream=s)
    s.synchronize()
    graph, got = torch.cuda.CUDAGraph(), bufs()
    with torch.cuda.graph(graph):
        both(*got)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a in (other, got):
        for x, y in zip(sum(want, []), sum(a, [])):
            assert torch.equal(x, y)


def test_calls_that_the_binding_refuses():
    dma = lib()
    torch, t = _types("bf16")
    p = dma.make_params(2, 4, 2, 10, 64, 1)
    q, k = torch.zeros(2, 10, 4, 64, dtype=t, device="cuda"), torch.zeros(2, 10, 2, 64, dtype=t, device="cuda")
    Q, K = torch.zeros(2, 4, 10, 64, dtype=t, device="cuda"), torch.zeros(2, 2, 10, 64, dtype=t, device="cuda")
    r = dma.make_prep(_freq(torch, 64))
    good = dict(q=q, k=k, v=k, Q=Q, K=K, V=torch.zeros_like(K))
    dma.prep(p, r, *good.values())
    for name, bad in (("q", q.float()), ("q", q[:, :9]), ("k", k.cpu()), ("Q", Q.transpose(1, 2)),
                      ("Q", Q.transpose(1, 2).contiguous().transpose(1, 2)), ("K", K[..., :32]),
                      ("q", torch.zeros(2, 10, 64, 4, dtype=t, device="cuda").transpose(2, 3))):
        with pytest.raises(ValueError, match=name):
            dma.prep(p, r, *{**good, name: bad}.values())
    for kw in (dict(q_weight=torch.zeros(64, device="cuda")), dict(k_weight=torch.zeros(32, dtype=t, device="cuda")),
               dict(positions=torch.zeros(2, 10, device="cuda")),
               dict(positions=torch.zeros(2, 9, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            dma.prep(p, dma.make_prep(_freq(torch, 64), **kw), *good.values())
    with pytest.raises(ValueError):
        dma.prep(p, dma.make_prep(_freq(torch, 64).cpu()), *good.values())
    odd = torch.zeros(2 * 10 * 4 * 64 + 4, dtype=t, device="cuda")[4:].view(2, 10, 4, 64)   # 8 bytes off
    with pytest.raises(dma.DmaError) as e:
        dma.prep(p, r, odd, *list(good.values())[1:])
    assert e.value.code == 1


def test_training_step_from_projections_and_back():
    """Projections -> prep -> gate -> selection -> attention, and the gradients all the way back to the
    projections.  Each stage is held to its own tolerance on the inputs the GPU gave it; the last (prep_bwd) to the
    whole: the attention's 2e-2 + 1e-2 |x| on its gradients, carried through the rows' Jacobian in magnitudes."""
    import oracle
    from gpu_common import assert_close
    dma = lib()
    B, N, H, Hkv, d, w = 1, 200, 4, 2, 64, 48
    c = _case(B, N, H, Hkv, d, "bf16", 64, False, True, True, seed=12)
    torch, t = c["torch"], c["t"]
    p = dma.make_params(B, H, Hkv, N, d, w)
    r = dma.make_prep(c["freq"], c["qw"], c["kw"], eps=1e-5)
    Q, K, V = (torch.empty((B, h, N, d), dtype=t, device="cuda") for h in (H, Hkv, Hkv))
    Delta, A = (0.05 * c["normal"](Hkv * d, H)).to(t), -torch.rand(H, device="cuda")
    dma.prep(p, r, c["q"], c["k"], c["v"], Q, K, V)
    fwd = dma.forward(p, Q, K, V, Delta, A)
    dO = c["normal"](B, H, N, d).to(t)
    bwd = dma.backward(p, Q, K, V, Delta, A, fwd, dO)
    grad = torch.empty(B, N, H + 2 * Hkv, d, dtype=t, device="cuda")
    gq, gk, gv = grad[:, :, :H], grad[:, :, H:H + Hkv], grad[:, :, H + Hkv:]
    dqw, dkw = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    dma.prep_bwd(p, r, c["q"], c["k"], bwd["dQ"], bwd["dK"], bwd["dV"], bwd["dV_gate"], gq, gk, gv, dqw, dkw,
                 dma.alloc_prep_workspace(p, r))
    torch.cuda.synchronize()
    # the oracle on the inputs that prep made
    delta = fwd["delta"].cpu().numpy()
    evict = np.stack([oracle.topw_eviction(delta[0, h], w) for h in range(H)])[None]
    Qn, Kn, Vn = _np(Q), _np(K), _np(V)
    O, _ = oracle.attn_fwd(Qn, Kn, Vn, delta.astype(np.float64), evict)
    assert_close(fwd["O"].float().cpu().numpy(), O, "O")
    rQ, rK, rV, rd = oracle.attn_bwd(Qn, Kn, Vn, delta.astype(np.float64), evict, _np(dO))
    _, _, rVg = oracle.gate_bwd(Vn, _np(Delta), _np(A), bwd["d_delta"].cpu().numpy().astype(np.float64))
    R = _R(c, B, N, d)
    eps = np.float64(np.float32(1e-5))
    for got, gw, x, wt, dy in ((gq, dqw, c["q"], c["qw"], rQ), (gk, dkw, c["k"], c["kw"], rK)):
        x, wt, dy = _np(x), _np(wt), dy.transpose(0, 2, 1, 3)
        ref, mag, rw, mw = _backward(x, wt, R, eps, dy)
        _, slack, _, slack_w = _backward(x, wt, R, eps, 2e-2 + 1e-2 * np.abs(dy))
        assert (np.abs(_np(got) - ref) <= slack + 2.0 ** -8 * (np.abs(ref) + slack) + 40 * U * mag).all()
        assert (np.abs(_np(gw) - rw) <= slack_w + (40 + 2 * N) * U * mw).all()
    ref = rV.transpose(0, 2, 1, 3) + rVg.transpose(0, 2, 1, 3)
    tol = 2e-2 + 1e-2 * np.abs(rV.transpose(0, 2, 1, 3)) + 2e-2 + 1e-2 * np.abs(rVg.transpose(0, 2, 1, 3))
    assert (np.abs(_np(gv) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol)).all()
