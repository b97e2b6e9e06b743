"""Calls of the paged cache that its documentation allows or refuses, beside the cases of test_gpu_paged.py."""
import numpy as np
import pytest

from test_gpu_paged import Cache, _append, _check_append

pytestmark = pytest.mark.gpu


def _call(c, a):
    c.dma.paged_append(c.p, c.c, a["r"], a["q"], a["k"], a["v"], a["Delta"], a["A"], a["Q"], c.ws, starts=a["starts"])


@pytest.mark.parametrize("dtype,B,step", [("bf16", 4, True), ("bf16", 5, False), ("bf16", 40, False), ("f32", 4, False)])
def test_append_to_a_length_below_the_prefix_is_skipped(dtype, B, step):
    """A length between 0 and the prefix would lead into the pages that the whole batch shares."""
    prefix, cnt = 64, [1] * B if step else [1 + b % 3 for b in range(B)]
    lens = [prefix + 4 + b % 5 for b in range(B)]
    c = Cache(lens, 4, 2, 64, 16, dtype, 8, seed=B, prefix=prefix, N=96)
    a = _append(c, None if step else cnt, 64, False, True)
    short = {1: prefix - 1, B - 2: 3, B - 1: cnt[B - 1]}
    for b, n in short.items():
        c.lens[b] = n
    before = [x.clone() for x in (c.K, c.V, c.delta)]
    _call(c, a)
    assert c.dma.check_device_status(c.p, c.ws) == 0x10000000
    shared = c.table[0, :prefix // 16].long()
    for x, y in zip((c.K, c.V, c.delta), before):
        assert c.torch.equal(x[shared], y[shared])
    first = np.concatenate([[0], np.cumsum(cnt)])
    for b in short:
        assert (a["Q"][first[b]:first[b + 1]] == 9).all()
    # the others are written as if the short ones had appended nothing
    keep = [t for t in range(a["T"]) if t >= first[-1] or np.searchsorted(first, t, "right") - 1 not in short]
    for n in ("q", "k", "v", "Q"):
        a[n] = a[n][keep]
    a["cnt"], a["T"] = [0 if b in short else n for b, n in enumerate(cnt)], len(keep)
    _check_append(c, a, 64, False, before)


def test_append_fills_the_prefix_through_one_sequence():
    """Lengths that reach the prefix append into it like anywhere else: sequence 0 writes the prompt that all
    share, the others nothing yet."""
    prefix = 64
    c = Cache([prefix, prefix, 0, prefix], 4, 2, 64, 16, "bf16", 8, seed=3, prefix=prefix, N=96)
    a = _append(c, [prefix, 0, 0, 0], 64, False, True)
    before = [x.clone() for x in (c.K, c.V, c.delta)]
    _call(c, a)
    assert c.dma.check_device_status(c.p, c.ws) == 0
    _check_append(c, a, 64, False, before)


SHAPES = {
    "rows": ([700, 0, 33, 512, 90], 0, 4, 2, 64, 16, "bf16", 64),
    "few_behind_prefix": ([320, 333, 0, 500, 320], 320, 4, 2, 128, 64, "bf16", 100),
    "many_behind_prefix": ([1280 + 7 * (i % 9) for i in range(40)], 1280, 16, 4, 64, 64, "bf16", 1200),
    "long_rows": ([20000 - 117 * i for i in range(12)], 0, 16, 1, 64, 64, "bf16", 150),
}


def _make(name, seed=71):
    lens, prefix, H, Hkv, d, page, dtype, w = SHAPES[name]
    return Cache(lens, H, Hkv, d, page, dtype, w, seed=seed, prefix=prefix, N=max(lens) + 64)


@pytest.mark.parametrize("name", SHAPES)
def test_steps_in_flight_equal_steps_one_by_one(name):
    """Lengths, gate values and queries change from call to call while earlier calls on the same workspace
    still run."""
    c = _make(name)
    torch, dma = c.torch, c.dma
    S, lens0 = len(c.lens_host), c.lens.clone()
    deltas = [c.delta.clone(), c.delta.flip(0).contiguous(), (c.delta * 0.5).contiguous()]
    Q = [c.normal(S, c.H, c.d).to(c.t) for _ in range(2)]
    grow = [(lens0 + g) * (lens0 > 0) for g in (0, 40, 17, 63)]
    results = []
    for wait in (True, False):
        out = [(torch.empty_like(Q[0]), torch.empty((S, c.H), device="cuda")) for _ in range(24)]
        torch.cuda.synchronize()
        for i, (O, L) in enumerate(out):
            c.delta.copy_(deltas[i % 3])
            c.lens.copy_(grow[i % 4])
            dma.paged_topk(c.p, c.c, c.ws)
            dma.paged_attn(c.p, c.c, Q[i % 2], c.ws, O, L)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        results.append(out)
    for a, b in zip(*results):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert dma.check_device_status(c.p, c.ws) == 0


@pytest.mark.parametrize("name", SHAPES)
def test_calls_captured_behind_another_streams_work(name):
    """In a captured graph the calls follow copies and kernels of another stream, and run on a forked one."""
    c = _make(name)
    torch, dma = c.torch, c.dma
    S = len(c.lens_host)
    src = dict(delta=c.delta.flip(0).contiguous(), lens=(c.lens + 9) * (c.lens > 0),
               Q=c.normal(S, c.H, c.d).to(c.t))
    old = dict(delta=c.delta.clone(), lens=c.lens.clone())
    Q = torch.zeros_like(src["Q"])
    c.delta.copy_(src["delta"])
    c.lens.copy_(src["lens"])
    want = c.run(src["Q"])[1:]
    want = [x.clone() for x in want]
    O, L = torch.empty_like(want[0]), torch.empty_like(want[1])
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            c.delta.copy_(src["delta"])       # a copy
            Q.copy_(src["Q"])
        torch.mul(src["lens"], 1, out=c.lens)  # a kernel
        main.wait_stream(side)                # the selection follows both
        dma.paged_topk(c.p, c.c, c.ws)
        O.zero_()
        side.wait_stream(main)
        with torch.cuda.stream(side):         # the attention on the forked stream
            dma.paged_attn(c.p, c.c, Q, c.ws, O, L)
        main.wait_stream(side)
    for _ in range(3):
        c.delta.copy_(old["delta"])
        c.lens.copy_(old["lens"])
        Q.zero_()
        L.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, want[0]) and torch.equal(L, want[1])
    assert dma.check_device_status(c.p, c.ws) == 0


def test_calls_from_two_host_threads():
    import threading
    a, b = _make("few_behind_prefix"), _make("rows", seed=72)
    torch = a.torch
    want = [a.run(), b.run()]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i, c):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(50):
                    got[i] = c.run(want[i][0])
            s.synchronize()
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i, c)) for i, c in enumerate((a, b))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for w, g in zip(want, got):
        for x, y in zip(w, g):
            assert torch.equal(x, y)


@pytest.mark.parametrize("B", [79, 80, 81, 130])
def test_rows_of_several_rounds(B):
    """More rows than the GPU takes at once, with and without an order by lengths: long, equal, idle and bad ones."""
    lens = [(i * 977) % 4300 for i in range(B - 7)] + [0, 0, 4300, 4300, 1, 1, 2]
    c = Cache(lens, 12, 4, 64, 16, "bf16", 40, seed=B)
    c.lens[3] = 4301
    c.dma.paged_topk(c.p, c.c, c.ws)
    c.torch.cuda.synchronize()
    assert c.dma.check_device_status(c.p, c.ws) == 0x10000000
    c.lens_host[3] = 0
    c.check_selection()


@pytest.mark.parametrize("d,Hkv,prefix,w,most", [(64, 2, 8192, 1024, 304), (128, 8, 4096, 512, 400), (128, 1, 4096, 512, 600)])
def test_many_rows_behind_a_prefix(d, Hkv, prefix, w, most):
    """Rows enough for lists of one warp each (and, where they are longer, not): none, few, and more own keys than one
    partial result holds."""
    B, H = 80, 16
    lens = [0 if b % 13 == 5 else prefix + (b * 37) % most for b in range(B - 2)] + [prefix + most, prefix]
    c = Cache(lens, H, Hkv, d, 16, "bf16", w, seed=d + Hkv, prefix=prefix, N=prefix + most,
              w_heads=[w, 1, 0, 17, 64, 255, 256, 300, w - 1] + [w] * 7)
    for b in (1, 7, B - 2):   # all their own keys pass
        c.delta[c.table[b, prefix // 16:].long()] += 1.0
    out = c.run()
    c.torch.cuda.synchronize()
    rows = c.region(c.dma.paged_layout(c.p, c.c).off_rows, (B, H, 4))
    assert rows[B - 2, 0, 0] == min(w, most) and rows[B - 1, 0, 0] == 0
    got = c.selected()
    again = c.run(out[0])
    for x, y in zip(out, again):
        assert c.torch.equal(x, y)
    # the definition, for some of the sequences
    some = sorted({*range(0, B, 9), 1, 5, 7, B - 2, B - 1})
    c.lens_host, c.table = [lens[b] for b in some], c.table[some]
    for i, b in enumerate(some):
        _, _, delta = c.row(i)
        for h in range(H):
            np.testing.assert_array_equal(got[b][h], c.chosen(delta[h], h), err_msg=f"{b} {h}")
    c.check(out[0][some], out[1][some], out[2][some])


@pytest.mark.parametrize("H,Hkv,d,dtype", [(16, 4, 64, "bf16"), (32, 2, 64, "bf16"), (48, 2, 64, "bf16"), (64, 8, 128, "bf16"),
                                           (33, 3, 64, "f32")])
def test_a_prompt_in_parts_is_the_prompt_at_once(H, Hkv, d, dtype):
    """Tokens enough for several rounds of CTAs, against the same tokens in calls of a few: the same bits."""
    lens = [3500, 0, 1621]
    c = Cache(lens, H, Hkv, d, 64, dtype, 8, seed=H, N=3600)
    torch = c.torch
    a = _append(c, lens, d, False, True, pad=5)
    before = [x.clone() for x in (c.K, c.V, c.delta)]
    _call(c, a)
    whole = [x.clone() for x in (c.K, c.V, c.delta, a["Q"])]
    for x, y in zip((c.K, c.V, c.delta), before):
        x.copy_(y)
    Q, at, first = torch.full_like(a["Q"], 9.0), [0, 0, 0], [0, 3500, 3500]
    for n in (1, 700, 37, 2000, 64, 3500):
        take = [min(n, lens[b] - at[b]) for b in range(3)]
        tok = torch.cat([torch.arange(first[b] + at[b], first[b] + at[b] + take[b], device="cuda") for b in range(3)])
        at = [x + t for x, t in zip(at, take)]
        c.lens.copy_(torch.tensor(at, dtype=torch.int32))
        part = dict(a, starts=torch.tensor(np.concatenate([[0], np.cumsum(take)]), dtype=torch.int32, device="cuda"),
                    Q=torch.empty((tok.numel(), H, d), dtype=c.t, device="cuda"), **{k: a[k][tok] for k in "qkv"})
        _call(c, part)
        Q[tok] = part["Q"]
    assert at == lens and c.dma.check_device_status(c.p, c.ws) == 0
    for x, y in zip(whole, (c.K, c.V, c.delta, Q)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("name,N", [("rows", 5000), ("rows", 70_000), ("rows", 400_000), ("few_behind_prefix", 5000),
                                    ("few_behind_prefix", 40_000), ("few_behind_prefix", 200_000),
                                    ("many_behind_prefix", 3000), ("many_behind_prefix", 20_000),
                                    ("many_behind_prefix", 120_000), ("long_rows", 80_000), ("long_rows", 600_000)])
def test_a_limit_far_above_the_lengths(name, N):
    """N chooses the kernels (other block sizes, clusters nearly all without a key, the sieve), not the results."""
    c = _make(name)
    torch, dma = c.torch, c.dma
    per = -(-N // c.page)
    table = torch.full((len(c.lens_host), per), -1, dtype=torch.int32, device="cuda")   # nothing behind a row's pages
    table[:, :c.table.shape[1]] = c.table
    c.table, c.N = table, N
    c.p = dma.make_params(len(c.lens_host), c.H, c.Hkv, N, c.d, c.w, Nq=1, dtype=c.dtype)
    c.c = dma.make_pages(c.p, c.K, c.V, c.delta, table, c.lens, prefix=c.prefix)
    c.ws = dma.alloc_paged_workspace(c.p, c.c)
    c.ws[256:].fill_(0xA5)
    out = c.run()
    torch.cuda.synchronize()
    c.check_selection()
    c.check(*out)
    again = c.run(out[0])
    for x, y in zip(out, again):
        assert torch.equal(x, y)
