"""dma_prep_bwd's weight gradients, row by row.

With a single row of dQ (dK) that is not zero the sum over all rows is that row's own term, however the rows are
shared out: every other addition adds a zero.  The term dy x r is off by what its factors are (see
test_gpu_prep.py): 40 u of (|a| + |b|) |x| r, a and b the pair that was rotated into dy, covers them, and the final
rounding to float32 one u more."""
import numpy as np
import pytest

from gpu_common import lib
from test_gpu_prep import U, _backward, _case, _np, _R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,N,H,Hkv,d,dtype,rot,inter", [
    (2, 5000, 6, 3, 64, "bf16", 64, False),     # several tokens a warp
    (1, 9001, 5, 1, 128, "f32", 96, True),
    (1, 700, 16, 8, 128, "bf16", 128, False),   # a token's chunks spread over warps
    (1, 1, 33, 11, 64, "bf16", 32, True),
])
def test_every_row_counts_once(B, N, H, Hkv, d, dtype, rot, inter):
    dma = lib()
    c = _case(B, N, H, Hkv, d, dtype, rot, inter, True, True, seed=N)
    torch, t = c["torch"], c["t"]
    p = dma.make_params(B, H, Hkv, N, d, 1, dtype=dtype)
    r = dma.make_prep(c["freq"], c["qw"], c["kw"], eps=1e-5, interleaved=inter)
    ws = dma.alloc_prep_workspace(p, r)
    gq, gk = torch.empty((B, N, H, d), dtype=t, device="cuda"), torch.empty((B, N, Hkv, d), dtype=t, device="cuda")
    rng = np.random.default_rng(N)
    tokens = {0, N - 1, N // 2, min(N - 1, 2367), min(N - 1, 2368), min(N - 1, 4736)} | set(rng.integers(0, N, 6).tolist())
    dQ, dK = torch.zeros((B, H, N, d), dtype=t, device="cuda"), torch.zeros((B, Hkv, N, d), dtype=t, device="cuda")
    eps = np.float64(np.float32(1e-5))
    for i, n in enumerate(sorted(tokens)):
        b, hq, hk = (B - 1) * (i & 1), (H - 1, 0, int(rng.integers(H)))[i % 3], (Hkv - 1, 0, int(rng.integers(Hkv)))[i % 3]
        row = [c["normal"](d).to(t) for _ in range(2)]
        dQ[b, hq, n], dK[b, hk, n] = row
        dqw, dkw = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        dma.prep_bwd(p, r, c["q"], c["k"], dQ, dK, None, None, gq, gk, None, dqw, dkw, ws)
        one = dict(c, pos=torch.tensor([[n]], dtype=torch.int32))
        R = _R(one, 1, 1, d)
        for got, x, w, dy, h in ((dqw, c["q"], c["qw"], row[0], hq), (dkw, c["k"], c["kw"], row[1], hk)):
            x, dy = _np(x[b, n, h]), _np(dy)
            _, _, ref, _ = _backward(x[None, None, None], _np(w), R, eps, dy[None, None, None])
            pairs = np.abs(dy) @ (R[0, 0] != 0)
            mag = pairs * np.abs(x) / np.sqrt((x * x).mean() + eps)
            err = np.abs(_np(got) - ref)
            assert (err <= 41 * U * mag).all(), (n, h, (err / mag).max() / U)
        # the row's own gradient is the only one
        assert torch.count_nonzero(gq.abs().sum(-1)) == 1 and torch.count_nonzero(gk.abs().sum(-1)) == 1
        assert gq[b, n, hq].any() and gk[b, n, hk].any()
        dQ[b, hq, n], dK[b, hk, n] = 0, 0


def test_backward_calls_in_flight_share_a_workspace():
    """The sums of one call are read while the next call is already being launched."""
    dma = lib()
    B, N, H, Hkv, d = 2, 3000, 8, 4, 64
    c = _case(B, N, H, Hkv, d, "bf16", 64, False, True, True, seed=5)
    torch = c["torch"]
    p = dma.make_params(B, H, Hkv, N, d, 1)
    r = dma.make_prep(c["freq"], c["qw"], c["kw"])
    ws = dma.alloc_prep_workspace(p, r)
    grads = [[c["normal"](B, h, N, d).to(c["t"]) for h in (H, Hkv)] for _ in range(3)]
    results = []
    for wait in (True, False):
        out = [[torch.empty_like(c["q"]), torch.empty_like(c["k"]), torch.empty(d, device="cuda"),
                torch.empty(d, device="cuda")] for _ in range(12)]
        torch.cuda.synchronize()
        for i, o in enumerate(out):
            dma.prep_bwd(p, r, c["q"], c["k"], *grads[i % 3], None, None, o[0], o[1], None, o[2], o[3], ws)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        results.append(out)
    for a, b in zip(*results):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
