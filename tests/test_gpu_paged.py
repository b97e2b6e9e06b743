"""Paged cache on the GPU (dma_paged_append, dma_paged_topk, dma_paged_attn) against the definitions in
float64.

Selections are compared position by position.  Tolerances of the attention, with u = 2^-24: a score is a sum
of d products, at most 16 of them (and 4 levels) one after the other, then delta is added: off by at most
(20 A + |s|) u, A the sum of the products' magnitudes (scaled).  Its exponential is taken of a difference
s - m: 2 |s - m| u more, and 2^-22 relative for the instruction; past |s - m| = 104 it is 0 in float32.  A
weight is therefore within (20 A + |s| + 2 |s - m| + 8) u, relative, the weighted sum adds at most 32
products in a row, 8 groups and one partial result for each 256 keys, and the quotient doubles it:
  |o - o'| <= 2 max_j(...) u sum_j w_j |v_j| + half a step of the output's type,
  |LSE - LSE'| <= max_j(...) u + 2 u |LSE|.
With a shared prefix the weights are also split into two bf16 parts for the tensor cores, which leaves
2^-16 of each."""
import numpy as np
import pytest

from gpu_common import lib, torch_cuda
from test_gpu_prep import _forward, _freq, _rotation

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


class Cache:
    """A paged cache with pages in random order, and its float64 view."""

    def __init__(self, lens, H, Hkv, d, page, dtype, w, seed=0, prefix=0, N=None, delta="gate", spare=3, w_heads=None):
        torch = torch_cuda()
        self.torch, self.dma = torch, lib()
        self.t = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.lens_host, self.H, self.Hkv, self.d, self.page, self.dtype, self.w = lens, H, Hkv, d, page, dtype, w
        self.G, self.prefix, self.w_heads = H // Hkv, prefix, w_heads
        S = len(lens)
        self.N = N or max(max(lens), 1)
        per = -(-self.N // page)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.gen = g
        np_ = prefix // page
        n_pages = np_ + S * (per - np_) + spare
        ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.empty((S, per), dtype=torch.int32, device="cuda")
        self.table[:, :np_] = ids[:np_]
        self.table[:, np_:] = ids[np_:np_ + S * (per - np_)].view(S, -1)
        self.unused = ids[np_ + S * (per - np_):]
        self.K = self.normal(n_pages, Hkv, page, d).to(self.t)
        self.V = self.normal(n_pages, Hkv, page, d).to(self.t)
        if delta == "gate":
            self.delta = torch.exp(-torch.rand((n_pages, H, page), generator=g, device="cuda"))
        elif delta == "levels":
            self.delta = torch.randint(0, 5, (n_pages, H, page), generator=g, device="cuda").float() - 2
            self.delta[self.delta == 0] = -0.0
            self.delta[:, :, ::3] = self.delta[:, :, ::3].abs()
        elif delta == "constant":
            self.delta = torch.full((n_pages, H, page), 0.25, device="cuda")
        else:                       # any float32 pattern that is a number
            bits = torch.randint(-(1 << 31), 1 << 31, (n_pages, H, page), generator=g, device="cuda").to(torch.int32)
            f = bits.view(torch.float32)
            self.delta = torch.where(torch.isnan(f), torch.ones_like(f), f).contiguous()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        wh = None if w_heads is None else torch.tensor(w_heads, dtype=torch.int32, device="cuda")
        self.wh = wh
        self.p = self.dma.make_params(S, H, Hkv, self.N, d, w, Nq=1, dtype=dtype, w_heads=wh)
        self.c = self.dma.make_pages(self.p, self.K, self.V, self.delta, self.table, self.lens, prefix=prefix)
        self.ws = self.dma.alloc_paged_workspace(self.p, self.c)
        self.ws[256:].fill_(0xA5)   # nothing may rely on what a workspace holds

    def normal(self, *s):
        return self.torch.randn(s, generator=self.gen, device="cuda")

    def window(self, h):
        return self.w if self.w_heads is None else min(max(self.w_heads[h], 1), self.w)

    def row(self, s, n=None):
        """K, V [Hkv, n, d] and delta [H, n] of sequence s in float64."""
        n = self.lens_host[s] if n is None else n
        j = np.arange(n)
        pg, sl = self.table[s].cpu().numpy()[j // self.page], j % self.page
        pg, sl = self.torch.from_numpy(pg).long().cuda(), self.torch.from_numpy(sl).long().cuda()
        return [x[pg, :, sl].double().cpu().numpy().swapaxes(0, 1) for x in (self.K, self.V)] + [
            self.delta[pg, :, sl].cpu().numpy().T]

    def chosen(self, delta, h):
        n = delta.shape[0]
        order = np.lexsort((np.arange(n), -delta.astype(np.float64)))
        return np.sort(order[:self.window(h)])

    def region(self, off, shape, dtype=np.int32):
        n = int(np.prod(shape)) * np.dtype(dtype).itemsize
        return self.ws[off:off + n].cpu().numpy().view(dtype).reshape(shape)

    def selected(self):
        """Positions the GPU selected for every row, from the workspace."""
        lay = self.dma.paged_layout(self.p, self.c)
        S, H = len(self.lens_host), self.H
        rows = self.region(lay.off_rows, (S, H, 4))
        sel = self.region(lay.off_sel, (S, H, lay.sel_len))
        out = [[sel[s, h, :rows[s, h, 0]] for h in range(H)] for s in range(S)]
        if lay.cand_len:
            cand = self.region(lay.off_cand, (H, lay.cand_len))
            _, _, dp = self.row(0, self.prefix)
            for h in range(H):
                n = min(self.window(h), self.prefix)
                f = dp[h][cand[h, :n]]
                u = np.where(f == 0, np.float32(0), f).astype(np.float32).view(np.uint32)
                key = np.where(u >> 31 == 1, ~u, u | np.uint32(1 << 31)).astype(np.uint32)
                for s in range(S):
                    edge, cut = np.uint32(rows[s, h, 1].view(np.uint32)), rows[s, h, 2]
                    take = (key > edge) | ((key == edge) & (np.arange(n) < cut))
                    assert take.sum() == rows[s, h, 3], (s, h)
                    out[s][h] = np.concatenate([cand[h, :n][take], out[s][h]])
        return out

    def check_selection(self):
        got = self.selected()
        for s, n in enumerate(self.lens_host):
            _, _, delta = self.row(s)
            for h in range(self.H):
                np.testing.assert_array_equal(got[s][h], self.chosen(delta[h], h), err_msg=f"{s} {h}")

    def attend(self, Q, scale=None):
        """(O, LSE, bounds of both) in float64."""
        S, H, d = len(self.lens_host), self.H, self.d
        O, L = np.zeros((S, H, d)), np.full((S, H), -np.inf)
        bO, bL = np.zeros((S, H, d)), np.zeros((S, H))
        Q = Q.double().cpu().numpy()
        scale = np.float64(np.float32(d ** -0.5)) if scale is None else np.float64(np.float32(scale))
        for s, n in enumerate(self.lens_host):
            if n == 0:
                continue
            K, V, delta = self.row(s)
            for h in range(H):
                j = self.chosen(delta[h], h)
                k, v, dl = K[h // self.G][j], V[h // self.G][j], delta[h][j].astype(np.float64)
                x = k @ Q[s, h] * scale + dl
                m = x.max()
                if m == -np.inf:
                    continue
                e = np.exp(x - m)
                O[s, h], L[s, h] = e @ v / e.sum(), m + np.log(e.sum())
                A = np.abs(k) @ np.abs(Q[s, h]) * scale
                rel = 20 * A + np.abs(dl) + A + 2 * np.minimum(m - x, 104) + 8
                rel = (rel[np.isfinite(dl)].max() + 32 + 8 + self.w / 256 + 2) * U
                if self.prefix and self.dtype == "bf16":
                    rel += 2.0 ** -16
                bO[s, h] = 2 * rel * (e @ np.abs(v)) / e.sum() + HALF[self.dtype] * np.abs(O[s, h]) * (1 + 2 * rel)
                bL[s, h] = rel + 2 * U * abs(L[s, h])
        return O, L, bO, bL

    def run(self, Q=None, stream=None):
        torch, S = self.torch, len(self.lens_host)
        Q = self.normal(S, self.H, self.d).to(self.t) if Q is None else Q
        O = torch.full((S, self.H, self.d), float("nan"), dtype=self.t, device="cuda")
        L = torch.full((S, self.H), float("nan"), device="cuda")
        self.dma.paged_topk(self.p, self.c, self.ws, stream)
        self.dma.paged_attn(self.p, self.c, Q, self.ws, O, L, stream)
        return Q, O, L

    def check(self, Q, O, L):
        rO, rL, bO, bL = self.attend(Q)
        O, L = O.double().cpu().numpy(), L.double().cpu().numpy()
        assert (np.isinf(L) == np.isinf(rL)).all()
        ok = np.isfinite(rL)
        assert (O[~ok] == 0).all()
        assert (np.abs(O - rO) <= bO).all(), (np.abs(O - rO) - bO).max()
        assert (np.abs(L[ok] - rL[ok]) <= bL[ok]).all(), (np.abs(L[ok] - rL[ok]) - bL[ok]).max()
        assert self.dma.check_device_status(self.p, self.ws) == 0


CASES = {
    # lens, H, Hkv, d, page, dtype, w, further arguments
    "one": ([1], 1, 1, 64, 16, "f32", 1, {}),
    "short": ([1, 0, 2, 16, 17], 2, 1, 64, 16, "bf16", 16, {}),
    "window": ([63, 64, 65, 300, 0], 6, 2, 128, 64, "bf16", 64, {}),
    "ties": ([500, 33, 129], 4, 4, 64, 32, "f32", 100, dict(delta="levels")),
    "constant": ([1000, 77], 3, 1, 128, 128, "bf16", 257, dict(delta="constant")),
    "any_bits": ([3001, 12, 2999], 5, 5, 64, 16, "f32", 700, dict(delta="bits")),
    "ragged": ([5000, 1, 4097, 2048, 2049, 0, 3], 8, 2, 128, 16, "bf16", 2048, {}),
    "heads": ([900, 40], 4, 2, 64, 16, "bf16", 300, dict(w_heads=[300, 1, 0, 999])),
    "room": ([130, 5], 2, 2, 128, 1024, "f32", 4096, dict(N=7000)),
    "long": ([70001, 65536], 2, 1, 64, 64, "bf16", 1000, {}),
}

# enough long rows for the selection that sieves: lengths that sieve at every group size and that do not,
# values alike so that the sieve's list overflows, a few large values among many (a wide range of keys)
SIEVED = {
    "lengths": ([20000, 17001, 150, 8 * 150, 8 * 150 - 1, 2400, 4801, 0, 1, 19999, 12345, 16384], "gate"),
    "ties": ([20000] * 6 + [19000 + i for i in range(6)], "levels"),
    "constant": ([18000, 20000, 19001, 400] * 3, "constant"),
    "any_bits": ([20000 - 117 * i for i in range(12)], "bits"),
}


@pytest.mark.parametrize("name", SIEVED)
def test_selection_of_many_long_rows(name):
    lens, kind = SIEVED[name]
    c = Cache(lens, 16, 1, 64, 64, "bf16", 150, seed=31, delta=kind)
    if kind == "gate":   # the best keys all in one place, as where a gate follows the content
        c.delta[c.table[0, 100:103].long()] += 1.0
    c.dma.paged_topk(c.p, c.c, c.ws)
    c.torch.cuda.synchronize()
    c.check_selection()
    assert c.dma.check_device_status(c.p, c.ws) == 0


def test_sieve_over_clusters_with_short_rows():
    # few rows, long enough for clusters of several CTAs each; a short row leaves most of them without a key
    c = Cache([140_000, 16, 17, 139_999, 20_000], 18, 1, 64, 64, "bf16", 1, seed=33, delta="gate")
    c.dma.paged_topk(c.p, c.c, c.ws)
    c.torch.cuda.synchronize()
    c.check_selection()


def test_sieved_row_with_a_bad_page():
    c = Cache([20000] * 12, 16, 1, 64, 64, "bf16", 150, seed=32)
    c.table[3, 200] = -5
    c.dma.paged_topk(c.p, c.c, c.ws)
    assert c.dma.check_device_status(c.p, c.ws) == 0x10000000
    got = c.selected()
    assert all(got[3][h].size == 0 for h in range(16))
    _, _, delta = c.row(4)
    np.testing.assert_array_equal(got[4][0], c.chosen(delta[0], 0))


@pytest.mark.parametrize("name", CASES)
def test_selection_and_attention(name):
    lens, H, Hkv, d, page, dtype, w, more = CASES[name]
    c = Cache(lens, H, Hkv, d, page, dtype, w, seed=len(name), **more)
    if more.get("delta") == "bits":
        c.dma.paged_topk(c.p, c.c, c.ws)
        c.torch.cuda.synchronize()
        c.check_selection()
        return
    out = c.run()
    c.torch.cuda.synchronize()
    c.check_selection()
    c.check(*out)
    # the same selection serves another query
    Q2 = c.normal(len(lens), H, d).to(c.t)
    O2, L2 = c.torch.empty_like(out[1]), c.torch.empty_like(out[2])
    c.dma.paged_attn(c.p, c.c, Q2, c.ws, O2, L2)
    c.check(Q2, O2, L2)


PREFIXED = {
    # lens, prefix, H, Hkv, d, page, dtype, w, further arguments
    "two": ([64, 65], 64, 2, 1, 64, 16, "bf16", 16, {}),
    "few": ([320, 333, 0, 500, 320], 320, 4, 2, 128, 64, "bf16", 100, {}),
    "wide": ([48 + 7 * i for i in range(19)], 48, 3, 3, 64, 16, "bf16", 64, {}),
    "window_over_prefix": ([128, 1000, 200], 128, 2, 1, 128, 128, "bf16", 300, {}),
    "ties": ([256 + 50 * i for i in range(33)], 256, 2, 1, 64, 32, "bf16", 90, dict(delta="levels")),
    "constant": ([160, 170, 480], 160, 1, 1, 64, 32, "bf16", 80, dict(delta="constant")),
    "heads": ([512, 700, 513], 512, 4, 2, 64, 16, "bf16", 200, dict(w_heads=[200, 1, 0, 999])),
    "batch": ([4096 + i for i in range(70)], 4096, 4, 2, 128, 64, "bf16", 600, {}),
    "batch_33": ([320 + 5 * (i % 9) for i in range(33)], 320, 3, 1, 64, 32, "bf16", 100, {}),
    "batch_64": ([2048 + i % 50 for i in range(64)], 2048, 2, 2, 128, 64, "bf16", 1500, dict(w_heads=[1500, 513])),
    "batch_65_ties": ([1024 + 3 * i for i in range(65)], 1024, 2, 1, 64, 64, "bf16", 400, dict(delta="levels")),
    "batch_all": ([640 + i for i in range(40)], 640, 2, 1, 128, 64, "bf16", 900, {}),
    "batch_small": ([0 if i % 7 == 3 else 16 + i for i in range(48)], 16, 2, 1, 128, 16, "bf16", 5, {}),
    "many_33": ([1280 + 7 * (i % 9) for i in range(33)], 1280, 16, 4, 64, 64, "bf16", 1200, {}),
    "many_ties": ([1024 + 3 * i for i in range(65)], 1024, 10, 2, 64, 64, "bf16", 1000, dict(delta="levels")),
    "many_all": ([2432 + i for i in range(40)], 2432, 8, 8, 128, 64, "bf16", 3000, {}),
    "many_130": ([0 if i % 7 == 3 else 1024 + i for i in range(130)], 1024, 8, 2, 128, 32, "bf16", 800, {}),
    "many_windows": ([2048 + i for i in range(40)], 2048, 16, 2, 128, 64, "bf16", 1200,
                     dict(w_heads=[1200, 1, 2, 64, 127, 128, 129, 256, 257, 511, 512, 513, 640, 1100, 1199, 3])),
    "long": ([40960, 50001], 40960, 2, 1, 128, 64, "bf16", 2048, {}),
    "crossing": ([4096, 4700, 4200, 4097, 4150], 4096, 2, 1, 64, 64, "bf16", 512, {}),
    "crossing_ties": ([1024 + 40 * i for i in range(12)], 1024, 2, 1, 64, 64, "bf16", 400, dict(delta="levels")),
    "tiny_window": ([512, 600, 513, 530], 512, 2, 1, 64, 16, "bf16", 3, {}),
    "idle_first": ([0, 100, 96], 96, 2, 2, 64, 32, "bf16", 40, {}),
    "float": ([64, 100, 90], 64, 2, 1, 64, 16, "f32", 30, {}),
    "alone": ([90], 64, 2, 1, 64, 16, "bf16", 30, {}),
}


@pytest.mark.parametrize("name", PREFIXED)
def test_shared_prefix(name):
    lens, prefix, H, Hkv, d, page, dtype, w, more = PREFIXED[name]
    c = Cache(lens, H, Hkv, d, page, dtype, w, seed=len(name), prefix=prefix, **more)
    lay = c.dma.paged_layout(c.p, c.c)
    assert (lay.cand_len > 0) == (dtype == "bf16" and len(lens) > 1)
    out = c.run()
    c.torch.cuda.synchronize()
    c.check_selection()
    c.check(*out)
    again = c.run(out[0])
    for x, y in zip(out, again):
        assert c.torch.equal(x, y)


def test_shared_prefix_any_bits_and_many_that_pass():
    """Selections alone: any float32 pattern, and own keys that push out more candidates than are kept in order."""
    for kind, seed in (("bits", 41), ("bits", 42), ("gate", 43)):
        c = Cache([2048, 2100, 2048 + 900, 2049, 0, 2700], 6, 6, 64, 32, "bf16", 300, seed=seed, prefix=2048, delta=kind)
        if kind == "gate":
            c.delta[c.table[2, 64:].long()] += 0.4
            c.delta[c.table[5, 64:66].long()] += 0.4
        c.dma.paged_topk(c.p, c.c, c.ws)
        c.torch.cuda.synchronize()
        c.check_selection()


def test_shared_prefix_masked_places_may_hold_anything():
    """Candidates that one sequence selects and another does not hold infinities: only the first sees them."""
    c = Cache([192, 320, 200], 2, 1, 64, 32, "bf16", 32, seed=3, prefix=192)
    torch = c.torch
    c.delta[c.table[1, 6:].long()] = 2.0 + torch.arange(32, device="cuda") / 64   # sequence 1 selects none of the prefix
    Q, O, L = c.run()
    assert all((x < 192).all() for x in c.selected()[0]) and all((x >= 192).all() for x in c.selected()[1])
    for s in range(3):
        c.K[c.table[s, :6].long()] = float("nan")
        c.V[c.table[s, :6].long()] = -float("inf")
    _, O2, L2 = c.run(Q)
    assert torch.equal(O[1], O2[1]) and torch.equal(L[1], L2[1])
    assert torch.isnan(O2[0].float()).all() and torch.isnan(L2[0]).all()
    # an infinite value among finite keys reaches those who selected it, and no other channel
    c = Cache([192, 320, 200], 1, 1, 64, 32, "bf16", 32, seed=3, prefix=192)
    c.delta[c.table[1, 6:].long()] = 2.0 + torch.arange(32, device="cuda") / 64
    want = c.run()
    j = int(c.selected()[0][0][-1])
    assert j in c.selected()[2][0]
    c.V[c.table[0, j // 32].long(), 0, j % 32, 5] = float("inf")
    got = c.run(want[0])
    for s in (0, 2):
        assert got[1][s, 0, 5] == float("inf")
        other = torch.arange(64, device="cuda") != 5
        assert (got[1][s, 0, other].float() - want[1][s, 0, other].float()).abs().max() <= 2.0 ** -8 * 4
    assert torch.equal(got[1][1], want[1][1]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,w", [(1, 700), (16, 1200)])
def test_shared_prefix_of_many_masked_places_may_hold_anything(H, w, d):
    """As above, for batches that fill both kernels: infinities in the first, a middle and the last tile."""
    B, prefix = 40, 1280
    c = Cache([prefix + 64] + [prefix + 1 + i for i in range(1, B - 1)] + [prefix + 1300], H, 1, d, 64, "bf16", w, seed=d,
              prefix=prefix)
    torch = c.torch
    last = c.table[B - 1, 20:].long()
    c.delta[last] = 2.0 + torch.rand(c.delta[last].shape, generator=c.gen, device="cuda")   # it selects none of the prefix
    want = c.run()
    sel = c.selected()
    assert (sel[B - 1][0] >= prefix).all()
    pick = [int(sel[0][0][k]) for k in (1, 300, 600)]
    assert all(j < prefix for j in pick)
    channel = (5, d - 1, 0)
    for j, ch, v in zip(pick, channel, (1.0, -1.0, 1.0)):
        c.V[c.table[0, j // 64].long(), 0, j % 64, ch] = v * float("inf")
    got = c.run(want[0])
    assert torch.equal(got[1][B - 1], want[1][B - 1]) and torch.equal(got[2], want[2])
    for s in range(B - 1):
        other = torch.ones(d, dtype=torch.bool, device="cuda")
        for j, ch, v in zip(pick, channel, (1.0, -1.0, 1.0)):
            if j in sel[s][0]:
                assert got[1][s, 0, ch] == v * float("inf")
                other[ch] = False
        assert (got[1][s, 0, other].float() - want[1][s, 0, other].float()).abs().max() <= 2.0 ** -8 * 4
    for s in range(B):
        c.K[c.table[s, :20].long()] = float("nan")
    got = c.run(want[0])
    assert torch.equal(got[1][B - 1], want[1][B - 1]) and torch.equal(got[2][B - 1], want[2][B - 1])
    assert torch.isnan(got[1][:B - 1].float()).all() and torch.isnan(got[2][:B - 1]).all()


def test_shared_prefix_bad_pages_and_short_lengths():
    c = Cache([64, 100, 80], 2, 1, 64, 16, "bf16", 20, seed=4, prefix=64)
    dma = c.dma
    c.lens[2] = 63                       # shorter than the prefix it is said to share
    Q, O, L = c.run()
    assert dma.check_device_status(c.p, c.ws) == 0x10000000
    assert (O[2] == 0).all() and (L[2] == -float("inf")).all()
    dma.clear_device_status(c.p, c.ws)
    c.lens_host = [64, 100, 0]
    c.check(Q, O, L)
    c.table[0, 1] = -7                   # sequence 0's row names the prefix
    _, O, L = c.run(Q)
    assert dma.check_device_status(c.p, c.ws) == 0x10000000
    assert (O == 0).all() and (L == -float("inf")).all()


def test_selection_longer_than_a_cluster_holds():
    # 8 x 49152 values stay on chip; the rest of the row is read again in every round
    c = Cache([500_003], 1, 1, 64, 64, "bf16", 5000, delta="bits")
    c.dma.paged_topk(c.p, c.c, c.ws)
    c.torch.cuda.synchronize()
    c.check_selection()


def test_masked_places_may_hold_anything():
    """Keys that are not selected, slots behind the last position and unused pages: NaN and infinities."""
    c = Cache([300, 40, 17], 2, 1, 64, 32, "bf16", 32, seed=2)
    torch = c.torch
    c.delta[c.unused.long()] = float("nan")
    for x in (c.K, c.V):
        x[c.unused.long()] = float("inf")
    want = c.run()
    keep = torch.zeros((c.K.shape[0], c.page), dtype=torch.bool, device="cuda")
    used = torch.zeros_like(keep)
    for s, n in enumerate(c.lens_host):
        _, _, delta = c.row(s)
        j = np.unique(np.concatenate([c.chosen(delta[h], h) for h in range(2)]))
        pages = c.table[s].long()
        keep[pages[torch.from_numpy(j // 32).cuda()], torch.from_numpy(j % 32).cuda()] = True
        i = torch.arange(n, device="cuda")
        used[pages[i // 32], i % 32] = True
    for x, bad in ((c.K, float("nan")), (c.V, float("inf"))):
        x.copy_(torch.where(keep[:, None, :, None], x, torch.full_like(x, bad)))
    c.delta.copy_(torch.where(used[:, None, :], c.delta, torch.full_like(c.delta, float("nan"))))
    got = c.run(want[0])
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_lowest_and_infinite_gate_values():
    c = Cache([40, 40, 40], 1, 1, 64, 16, "f32", 64, seed=5)
    low = np.finfo(np.float32).min
    pages = c.table.long()
    c.delta[pages[0]] = float(low)              # all alike: the scores drown, every key weighs the same
    c.delta[pages[1]] = -float("inf")           # nothing left
    c.delta[pages[2]] = -float("inf")
    c.delta[pages[2, 1], 0, 3] = 0.5            # one key left, at position 19
    Q, O, L = c.run()
    c.check_selection()
    _, V, _ = c.row(0)
    np.testing.assert_allclose(O[0, 0].cpu().numpy(), V[0].mean(0), atol=1e-5)
    assert L[0, 0].item() == low
    assert (O[1] == 0).all() and L[1, 0].item() == -float("inf")
    assert torch_cuda().equal(O[2, 0], c.V[pages[2, 1], 0, 3])


def test_pages_and_lengths_out_of_range_are_skipped_and_reported():
    c = Cache([100, 100, 100, 100], 2, 1, 64, 16, "bf16", 50, seed=6)
    dma, torch = c.dma, c.torch
    c.table[1, 3] = c.K.shape[0]
    c.table[2, 0] = -1
    c.lens[3] = 101
    Q, O, L = c.run()
    torch.cuda.synchronize()
    with pytest.raises(Exception):
        dma.check("dma_check_device_status", 5)
    assert dma.check_device_status(c.p, c.ws) == 0x10000000
    assert (O[1:] == 0).all() and (L[1:] == -float("inf")).all()
    dma.clear_device_status(c.p, c.ws)
    c.lens_host = [100, 0, 0, 0]
    c.check(Q, O, L)
    # a page behind a sequence's length is never looked at
    c.lens_host = [100, 48, 0, 100]
    c.lens.copy_(torch.tensor(c.lens_host))
    c.check(*c.run(Q))


# ---------------------------------------------------------------- append

APPENDS = {
    # lens (after), tokens appended (None: one each), H, Hkv, d, page, dtype, rot, interleaved, norms
    "step": ([1, 17, 0, 64, 65], None, 4, 2, 64, 16, "bf16", 64, False, True),
    "prompts": ([70, 5, 33, 129], [70, 0, 20, 129], 16, 8, 128, 32, "bf16", 128, False, True),
    "one_head_f32": ([19, 3], [7, 3], 1, 1, 64, 16, "f32", 32, True, True),
    "wide_f32": ([40, 16, 2], [40, 1, 2], 33, 11, 128, 16, "f32", 128, False, False),
    "odd_heads": ([37, 200], [36, 64], 12, 4, 64, 64, "bf16", 16, True, True),
    "no_turn": ([50], [50], 64, 8, 64, 16, "bf16", 0, False, True),
    "wide_rows": ([21, 9], [3, 9], 32, 32, 128, 16, "bf16", 128, False, True),
    "many": ([1, 2, 3] * 23, None, 32, 8, 128, 64, "bf16", 128, False, True),
}


def _append(c, cnt, rot, inter, norms, layout="packed", pad=3, base=10000.0):
    """Appends to cache c; returns the tokens' float64 inputs and what the call was given."""
    torch, dma = c.torch, c.dma
    H, Hkv, d = c.H, c.Hkv, c.d
    step = cnt is None
    cnt = [1] * len(c.lens_host) if step else cnt
    T = sum(cnt) + (0 if step else pad)      # behind the last sequence: padding
    if layout == "packed":
        qkv = c.normal(T, H + 2 * Hkv, d).to(c.t)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    else:                                    # head-major
        q, k, v = (c.normal(h, T, d).to(c.t).transpose(0, 1) for h in (H, Hkv, Hkv))
    qw = (1 + 0.1 * c.normal(d)).to(c.t) if norms else None
    kw = (1 + 0.1 * c.normal(d)).to(c.t) if norms else None
    r = dma.make_prep(_freq(torch, rot, base), qw, kw, eps=1e-5, interleaved=inter)
    Delta = (0.05 * c.normal(Hkv * d, H)).to(c.t)
    A = -torch.rand(H, generator=c.gen, device="cuda")
    starts = None if step else torch.tensor(np.concatenate([[0], np.cumsum(cnt)]), dtype=torch.int32, device="cuda")
    Qo = torch.full((T, H, d), 9.0, dtype=c.t, device="cuda")
    return dict(q=q, k=k, v=v, qw=qw, kw=kw, r=r, Delta=Delta, A=A, starts=starts, Q=Qo, cnt=cnt, T=T)


def _check_append(c, a, rot, inter, before, base=10000.0):
    """The whole cache and Q against the definition; before: the cache as it was."""
    d = c.d
    K, V, D = (x.double().cpu().numpy() for x in before)
    freq = _freq(c.torch, rot, base).cpu().numpy() if rot else np.zeros(0, np.float32)
    table, t = c.table.cpu().numpy(), 0
    f64 = {n: a[n].double().cpu().numpy() for n in "qkv"}
    w = {n: None if a[n] is None else a[n].double().cpu().numpy() for n in ("qw", "kw")}
    Del, A = a["Delta"].double().cpu().numpy(), a["A"].double().cpu().numpy()
    Q = np.full((a["T"], c.H, d), 9.0)
    bK, bQ, bD = np.zeros(K.shape), np.zeros(Q.shape), np.zeros(D.shape)
    half, eps = HALF[c.dtype], np.float64(np.float32(1e-5))
    for s, n in enumerate(a["cnt"]):
        for i in range(n):
            pos = c.lens_host[s] - n + i
            if pos >= 0:
                R = _rotation(np.array([[pos]]), freq, inter, d)
                pg, sl = table[s, pos // c.page], pos % c.page
                for out, b, name, at in ((K, bK, "k", (pg, slice(None), sl)), (Q, bQ, "q", (t,))):
                    y, mag = _forward(f64[name][t][None, None], w[name + "w"], R, eps)
                    out[at] = y[0, 0]
                    b[at] = half * np.abs(y[0, 0]) + 20 * U * mag[0, 0] * (1 + half)
                V[pg, :, sl] = f64["v"][t]
                x = f64["v"][t].reshape(-1) @ Del
                # float32 sums of K products (K / 8 at most in a row), then softplus and exp
                mag = np.abs(f64["v"][t].reshape(-1)) @ np.abs(Del)
                D[pg, :, sl] = np.exp(A * np.logaddexp(0, x))
                K_ = f64["v"][t].size
                bD[pg, :, sl] = D[pg, :, sl] * (np.abs(A) * ((K_ / 8 + 16) * mag + 8 * np.logaddexp(0, x)) + 8) * U
            t += 1
    assert np.array_equal(c.V.double().cpu().numpy(), V)
    for got, ref, b in ((c.K, K, bK), (c.delta, D, bD), (a["Q"], Q, bQ)):
        err = np.abs(got.double().cpu().numpy() - ref)
        assert (err <= b).all(), ((err - b).max(), np.unravel_index((err - b).argmax(), err.shape))


@pytest.mark.parametrize("layout", ["packed", "heads"])
@pytest.mark.parametrize("name", APPENDS)
def test_append(name, layout):
    lens, cnt, H, Hkv, d, page, dtype, rot, inter, norms = APPENDS[name]
    c = Cache(lens, H, Hkv, d, page, dtype, 8, seed=len(name), N=max(lens) + 5)
    a = _append(c, cnt, rot, inter, norms, layout)
    before = [x.clone() for x in (c.K, c.V, c.delta)]
    c.dma.paged_append(c.p, c.c, a["r"], a["q"], a["k"], a["v"], a["Delta"], a["A"], a["Q"], c.ws, starts=a["starts"])
    _check_append(c, a, rot, inter, before)
    assert c.dma.check_device_status(c.p, c.ws) == 0
    # without queries the cache gets the same bits
    again = [x.clone() for x in (c.K, c.V, c.delta)]
    for x, y in zip((c.K, c.V, c.delta), before):
        x.copy_(y)
    c.dma.paged_append(c.p, c.c, a["r"], None, a["k"], a["v"], a["Delta"], a["A"], None, c.ws, starts=a["starts"])
    for x, y in zip((c.K, c.V, c.delta), again):
        assert c.torch.equal(x, y)


@pytest.mark.parametrize("B", [31, 32, 33, 70])
def test_append_to_many_sequences(B):
    """Sequences are looked up in two ways, for fewer than 32 and for more; some append nothing."""
    cnt = [(7 * b) % 5 if b % 3 else 0 for b in range(B)]
    c = Cache([n + 3 * b % 40 for b, n in enumerate(cnt)], 4, 2, 64, 16, "bf16", 8, seed=B, N=64)
    a = _append(c, cnt, 64, False, True, pad=37)
    before = [x.clone() for x in (c.K, c.V, c.delta)]
    c.dma.paged_append(c.p, c.c, a["r"], a["q"], a["k"], a["v"], a["Delta"], a["A"], a["Q"], c.ws, starts=a["starts"])
    _check_append(c, a, 64, False, before)
    assert c.dma.check_device_status(c.p, c.ws) == 0


def test_append_skips_what_has_no_place():
    c = Cache([30, 30, 30], 2, 1, 64, 16, "bf16", 8, N=32, seed=8)
    dma, torch = c.dma, c.torch
    a = _append(c, [4, 4, 40], 64, False, True)   # sequence 2 appends more tokens than it is long
    c.table[1, 1] = c.K.shape[0] + 7              # sequence 1's tokens lie in a page that does not exist
    before = [x.clone() for x in (c.K, c.V, c.delta)]
    dma.paged_append(c.p, c.c, a["r"], a["q"], a["k"], a["v"], a["Delta"], a["A"], a["Q"], c.ws, starts=a["starts"])
    assert dma.check_device_status(c.p, c.ws) == 0x10000000
    dma.clear_device_status(c.p, c.ws)
    Q = a["Q"].clone()
    assert (Q[4:8] == 9).all() and (Q[8:18] == 9).all() and (Q[48:] == 9).all()
    for s in (1, 2):   # what is written is right, what is skipped stays: compare with those tokens left out
        c.lens_host[s] = 30
    pg = c.table.clone()
    c.table[1, 1] = int(c.unused[0])
    keep = [x[c.unused.long()].clone() for x in before]
    for x, y in zip((c.K, c.V, c.delta), keep):
        assert torch.equal(x[c.unused.long()], y)
    a["cnt"][1] = 0
    for n in "qkv":
        a[n] = torch.cat([a[n][:4], a[n][8:]])
    a["Q"], a["T"] = torch.cat([Q[:4], Q[8:]]), a["T"] - 4
    _check_append(c, a, 64, False, before)
    c.table.copy_(pg)
    # longer than N: the whole sequence is skipped
    c.lens[0] = 33
    now = [x.clone() for x in (c.K, c.V, c.delta)]
    dma.paged_append(c.p, c.c, a["r"], a["q"][:3], a["k"][:3], a["v"][:3], a["Delta"], a["A"], a["Q"][:3], c.ws,
                     starts=torch.tensor([0, 3, 3, 3], dtype=torch.int32, device="cuda"))
    assert dma.check_device_status(c.p, c.ws) == 0x10000000
    for x, y in zip((c.K, c.V, c.delta), now):
        assert torch.equal(x, y)


def test_serving_loop_against_the_dense_path_and_in_a_graph():
    """Prompts, then decode steps with lengths that grow on the device: a captured step replayed equals the
    calls made one by one, and each step's attention is that of the dense cache through dma_attn_fwd."""
    lens = [40, 7, 100]
    H, Hkv, d, page, w, steps = 4, 2, 64, 16, 32, 5
    caches, outs = [], []
    for mode in ("calls", "graph"):
        c = Cache(lens, H, Hkv, d, page, "bf16", w, seed=11, N=128)
        dma, torch = c.dma, c.torch
        a = _append(c, list(lens), 64, False, True, pad=0)
        dma.paged_append(c.p, c.c, a["r"], a["q"], a["k"], a["v"], a["Delta"], a["A"], a["Q"], c.ws, starts=a["starts"])
        tok = [c.normal(3, H + 2 * Hkv, d).to(c.t) for _ in range(steps)]
        x = torch.empty_like(tok[0])
        q = torch.empty((3, H, d), dtype=c.t, device="cuda")
        O, L = torch.empty_like(q), torch.empty((3, H), device="cuda")

        def step():
            c.lens.add_(1)
            dma.paged_append(c.p, c.c, a["r"], x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], a["Delta"], a["A"], q, c.ws)
            dma.paged_topk(c.p, c.c, c.ws)
            dma.paged_attn(c.p, c.c, q, c.ws, O, L)

        if mode == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        got = []
        for i in range(steps):
            x.copy_(tok[i])
            graph.replay() if mode == "graph" else step()
            got.append((O.clone(), L.clone(), q.clone()))
            c.lens_host = [n + i + 1 for n in lens]
            if mode == "calls":
                c.check(q, O, L)
                c.check_selection()
        outs.append(got)
        caches.append(c)
        assert c.lens.tolist() == [n + steps for n in lens]
    for a_, b_ in zip(*outs):
        for x_, y_ in zip(a_, b_):
            assert torch.equal(x_, y_)
    # the last step of each sequence through the dense decode
    c = caches[0]
    for s, n in enumerate(c.lens_host):
        K, V, delta = (torch.from_numpy(np.ascontiguousarray(y)).cuda() for y in c.row(s))
        p = dma.make_params(1, H, Hkv, n, d, w, Nq=1)
        ws = dma.alloc_workspace(p)
        Kd, Vd, dd = K.to(c.t)[None].contiguous(), V.to(c.t)[None].contiguous(), delta.float()[None].contiguous()
        dma.topk_mask(p, dd, None, ws)
        o, l = torch.empty((1, H, 1, d), dtype=c.t, device="cuda"), torch.empty((1, H, 1), device="cuda")
        dma.attn_fwd(p, outs[0][-1][2][s][None, :, None].contiguous(), Kd, Vd, dd, None, ws, o, l)
        # two bf16 roundings apart at most, and the dense path's own approximate exponentials
        assert (o[0, :, 0].float() - outs[0][-1][0][s].float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()
        assert (l[0, :, 0] - outs[0][-1][1][s]).abs().max() <= 1e-4


def test_two_streams_and_graphs_that_share_a_workspace():
    a = Cache([500, 3, 77], 4, 2, 64, 16, "bf16", 64, seed=20)
    b = Cache([64, 900], 2, 2, 128, 32, "f32", 128, seed=21)
    torch = a.torch
    want = [a.run(), b.run()]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        with torch.cuda.stream(s1):
            ra = a.run(want[0][0])
        with torch.cuda.stream(s2):
            rb = b.run(want[1][0])
        got.append((ra, rb))
    torch.cuda.synchronize()
    for ra, rb in got:
        for x, y in list(zip(want[0], ra)) + list(zip(want[1], rb)):
            assert torch.equal(x, y)
    # two graphs on one workspace, replayed in turn, selection and attention in either
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    Q2 = a.normal(3, 4, 64).to(a.t)
    w2 = a.run(Q2)
    with torch.cuda.graph(g1):
        r1 = a.run(want[0][0])
    with torch.cuda.graph(g2):
        r2 = a.run(Q2)
    for _ in range(3):
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    for x, y in list(zip(want[0], r1)) + list(zip(w2, r2)):
        assert torch.equal(x, y)


def test_large_shared_batch_in_a_graph_beside_another_stream():
    """The tcgen05 kernel captured and replayed as lengths change, while the same call runs on another stream."""
    prefix = 1280
    c = Cache([prefix + 1 + i % 20 for i in range(40)], 16, 4, 64, 64, "bf16", 1200, seed=5, prefix=prefix, N=prefix + 64)
    torch, dma = c.torch, c.dma
    Q, O, L = c.run()
    full = [x.clone() for x in (O, L)]
    lens = c.lens.clone()
    side, ws2 = torch.cuda.Stream(), dma.alloc_paged_workspace(c.p, c.c)
    O2, L2 = torch.empty_like(O), torch.empty_like(L)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dma.paged_topk(c.p, c.c, c.ws)
        dma.paged_attn(c.p, c.c, Q, c.ws, O, L)
    for grow in (30, 0, 7):
        c.lens.copy_(lens + grow)
        c.lens[3] = 0
        torch.cuda.synchronize()
        O.fill_(float("nan"))
        L.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            dma.paged_topk(c.p, c.c, ws2)
            dma.paged_attn(c.p, c.c, Q, ws2, O2, L2)
        torch.cuda.synchronize()
        assert torch.equal(O, O2) and torch.equal(L, L2)
        assert (O[3] == 0).all() and (L[3] == -float("inf")).all()
        if grow == 0:
            keep = torch.arange(40, device="cuda") != 3
            assert torch.equal(O[keep], full[0][keep]) and torch.equal(L[keep], full[1][keep])
    assert dma.check_device_status(c.p, c.ws) == 0


def test_many_rows_of_any_lengths():
    """Rows that take several rounds are taken in the order of lengths, equal ones and idle ones among them."""
    lens = [(i * 977) % 4300 for i in range(60)] + [0, 0, 4300, 4300, 1, 1, 2]
    c = Cache(lens, 12, 4, 64, 16, "bf16", 40, seed=6)
    c.dma.paged_topk(c.p, c.c, c.ws)
    c.torch.cuda.synchronize()
    c.check_selection()


def test_calls_that_the_binding_refuses():
    c = Cache([40, 7], 4, 2, 64, 16, "bf16", 8, seed=50)
    dma, torch = c.dma, c.torch
    Q, O, L = c.run()
    for bad in ((Q.float(), O, L), (Q[:1], O, L), (Q, O.float(), L), (Q, O, L[:, :2]), (Q, O.transpose(0, 1), L),
                (Q.cpu(), O, L)):
        with pytest.raises(ValueError):
            dma.paged_attn(c.p, c.c, bad[0], c.ws, bad[1], bad[2])
    with pytest.raises(ValueError):
        dma.paged_topk(c.p, c.c, c.ws.cpu())
    with pytest.raises(dma.DmaError) as e:
        dma.paged_topk(c.p, c.c, c.ws[:1024])
    assert e.value.code == 3
    for name, bad in (("K", c.K.float()), ("K", c.K[:, :1]), ("V", c.V[:-1]), ("delta", c.delta.to(c.t)),
                      ("table", c.table.long()), ("table", c.table[:1]), ("lens", c.lens.float())):
        args = dict(K=c.K, V=c.V, delta=c.delta, table=c.table, lens=c.lens)
        args[name] = bad
        with pytest.raises(ValueError):
            dma.make_pages(c.p, **args)
    a = _append(c, [3, 2], 64, False, True)
    call = lambda **kw: dma.paged_append(c.p, c.c, a["r"], *[kw.get(n, a[n]) for n in ("q", "k", "v", "Delta", "A", "Q")],
                                         c.ws, starts=kw.get("starts", a["starts"]))
    before = [x.clone() for x in (c.K, c.V, c.delta)]
    for kw in (dict(v=a["v"][:-1]), dict(Delta=a["Delta"].float()), dict(A=a["A"][:2]), dict(Q=a["Q"][:-1]),
               dict(starts=a["starts"].long()), dict(starts=a["starts"][:-1]), dict(k=a["k"].cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(dma.DmaError):
        call(starts=None)                        # eight tokens are not one for each of two sequences
    empty = [a[n][:0] for n in ("q", "k", "v")]
    dma.paged_append(c.p, c.c, a["r"], *empty, a["Delta"], a["A"], a["Q"][:0], c.ws,
                     starts=torch.zeros(3, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for x, y in zip((c.K, c.V, c.delta), before):
        assert torch.equal(x, y)


def test_tables_may_name_the_same_page_twice():
    """Two sequences over the same pages, and one page at two places of a sequence: reading does not care."""
    c = Cache([48, 48, 70], 2, 1, 64, 16, "bf16", 20, seed=51)
    c.table[1] = c.table[0]
    c.table[2, 3] = c.table[2, 1]
    Q = c.normal(3, 2, 64).to(c.t)
    Q[1] = Q[0]
    out = c.run(Q)
    c.torch.cuda.synchronize()
    c.check_selection()
    c.check(*out)
    assert c.torch.equal(out[1][0], out[1][1]) and c.torch.equal(out[2][0], out[2][1])


def test_rows_far_into_a_large_cache():
    """Slots whose byte offset passes 32 bits (cache of 4.3 GB): the last pages, at both ends of a table row."""
    torch = torch_cuda()
    dma = lib()
    H, Hkv, d, page, n_pages = 2, 1, 128, 64, 262144 + 8
    K = torch.zeros((n_pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    delta = torch.zeros((n_pages, H, page), device="cuda")
    lens = torch.tensor([150, 64], dtype=torch.int32, device="cuda")
    table = torch.tensor([[n_pages - 1, 0, n_pages - 2], [n_pages - 3, -9, -9]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    p = dma.make_params(2, H, Hkv, 192, d, 100, Nq=1)
    pages = dma.make_pages(p, K, V, delta, table, lens)
    ws = dma.alloc_paged_workspace(p, pages)
    qkv = torch.randn((214, H + 2 * Hkv, d), generator=g, device="cuda").to(K.dtype)
    Delta = (0.05 * torch.randn((Hkv * d, H), generator=g, device="cuda")).to(K.dtype)
    A = -torch.rand(H, generator=g, device="cuda")
    starts = torch.tensor([0, 150, 214], dtype=torch.int32, device="cuda")
    Qo = torch.empty((214, H, d), dtype=K.dtype, device="cuda")
    r = dma.make_prep(None)
    dma.paged_append(p, pages, r, qkv[:, :H], qkv[:, H:H + 1], qkv[:, H + 1:], Delta, A, Qo, ws, starts=starts)
    assert torch.equal(K[n_pages - 1, 0], qkv[:64, H]) and torch.equal(V[n_pages - 3, 0], qkv[150:, H + 1])
    assert torch.equal(K[n_pages - 2, 0, :22], qkv[128:150, H]) and (K[1:n_pages - 3] == 0).all()
    Q = torch.randn((2, H, d), generator=g, device="cuda").to(K.dtype)
    O, L = torch.empty_like(Q), torch.empty((2, H), device="cuda")
    dma.paged_topk(p, pages, ws)
    dma.paged_attn(p, pages, Q, ws, O, L)
    assert dma.check_device_status(p, ws) == 0
    # the same rows in a small cache give the same bits
    small = [x[[0, n_pages - 1, n_pages - 2, n_pages - 3]].contiguous() for x in (K, V, delta)]
    t2 = torch.tensor([[1, 0, 2], [3, -9, -9]], dtype=torch.int32, device="cuda")
    pages2 = dma.make_pages(p, *small, t2, lens)
    O2, L2 = torch.empty_like(O), torch.empty_like(L)
    dma.paged_topk(p, pages2, ws)
    dma.paged_attn(p, pages2, Q, ws, O2, L2)
    assert torch.equal(O, O2) and torch.equal(L, L2)


def test_prefix_that_is_everything():
    """No position behind the prefix, for any sequence or for all that the problem allows."""
    for N in (96, 128):
        c = Cache([96, 96, 0, 96], 4, 2, 64, 32, "bf16", 40, seed=52, prefix=96, N=N)
        out = c.run()
        c.torch.cuda.synchronize()
        c.check_selection()
        c.check(*out)
