"""Measured cases of the operators around the attention: from the projections to its inputs and back
(prep, prep_bwd), and serving from a paged cache (append, decode, decode over a shared prefix).

`run` computes an operator in its plain form (torch, 32 bits, rounded once at the end) or, with
`own`, through trainable_dynamic_mask_b200; `exact` restates the definition in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 10000.0
DEV = "cuda"


def listed():
    return [
        # the training workload's projections (B2 N8192, 16 query heads on 8) on their way into the attention
        dict(name="prep_train", op="prep", B=2, N=8192, H=16, Hkv=8, d=128, dtype="bf16", rot=128, inter=False,
             norm=True, far=False),
        # one decode step of eight sequences, each at its own position: launch latency
        dict(name="prep_step", op="prep", B=8, N=1, H=32, Hkv=8, d=128, dtype="bf16", rot=128, inter=False, norm=True,
             far=True),
        # odd length, three heads to a group, float32, part of the channels rotated in neighbouring pairs
        dict(name="prep_odd_f32", op="prep", B=3, N=1237, H=6, Hkv=2, d=64, dtype="f32", rot=48, inter=True, norm=True,
             far=True),
        # the training workload's gradients on their way back to the projections
        dict(name="prep_bwd_train", op="prep_bwd", B=2, N=8192, H=16, Hkv=8, d=128, dtype="bf16", rot=128, inter=False,
             norm=True, far=False),
        # the same at an odd length, in float32
        dict(name="prep_bwd_odd_f32", op="prep_bwd", B=1, N=331, H=6, Hkv=2, d=64, dtype="f32", rot=32, inter=False,
             norm=True, far=True),
        # one token for each of 64 sequences of different lengths: every decode step of a server
        dict(name="append_step", op="append", S=64, longest=512, page=64, H=32, Hkv=8, d=128, dtype="bf16", step=True,
             rot=128, inter=False, norm=True, mix=1),
        # prompts of five sequences, about 8000 tokens together, packed
        dict(name="append_prompts", op="append", S=5, longest=3001, page=64, H=16, Hkv=8, d=128, dtype="bf16",
             step=False, rot=128, inter=False, norm=True, mix=2),
        # the decode workload (8 rows of 65536 positions, window 2048) in pages
        dict(name="decode_long", op="decode", S=8, longest=65536, shortest=65536, prefix=0, page=64, H=32, Hkv=8, d=128,
             w=2048, dtype="bf16", mix=3),
        # a running batch of mixed lengths, some shorter than the window, one finished (length 0)
        dict(name="decode_ragged", op="decode", S=48, longest=8192, shortest=0, prefix=0, page=16, H=16, Hkv=8, d=128,
             w=1024, dtype="bf16", mix=4),
        # one short sequence: launch latency
        dict(name="decode_one", op="decode", S=1, longest=1000, shortest=1000, prefix=0, page=64, H=2, Hkv=1, d=64, w=64,
             dtype="f32", mix=5),
        # 64 continuations of one long prompt
        dict(name="decode_prefix", op="decode", S=64, longest=33000, shortest=32768, prefix=32768, page=64, H=32, Hkv=8,
             d=128, w=2048, dtype="bf16", mix=6),
        # eight samples of one short prompt
        dict(name="decode_prefix_few", op="decode", S=8, longest=2311, shortest=2048, prefix=2048, page=32, H=16, Hkv=8,
             d=64, w=512, dtype="bf16", mix=7),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["prep", "prep_bwd", "append", "decode", "prefix"])
    H, Hkv = rng.choice([(2, 1), (6, 2), (8, 8), (12, 4), (16, 8), (32, 8)])
    d = rng.choice([64, 128])
    c = dict(H=H, Hkv=Hkv, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]), mix=rng.randrange(1 << 20))
    turn = dict(rot=rng.choice([16, 32, d // 2, d - 16, d, d]), inter=rng.random() < 0.4, norm=rng.random() < 0.8)
    if op in ("prep", "prep_bwd"):
        B = rng.choice([1, 2, 3, 4])
        most = 16384 * 24 * 128 * 2 // ((H + Hkv) * d * (2 if c["dtype"] == "bf16" else 4))
        c.update(op=op, B=B, N=_log(rng, 1, min(8192, most // B)), far=rng.random() < 0.5, **turn)
    elif op == "append":
        step = rng.random() < 0.5
        S = _log(rng, 1, 64) if step else rng.choice([1, 2, 3, 5, 7])
        c.update(op=op, S=S, longest=_log(rng, 16, 512) if step else _log(rng, 16, 8000 // S), step=step,
                 page=rng.choice([16, 32, 64, 128]), **turn)
    elif op == "decode":
        S = _log(rng, 1, 48)
        longest = _log(rng, 1, min(65536, 180000 // S))
        c.update(op=op, S=S, longest=longest, shortest=rng.choice([0, longest // 2, longest]), prefix=0,
                 page=rng.choice([16, 32, 64, 128]), w=_log(rng, 16, 2048))
    else:
        page = rng.choice([16, 32, 64, 128])
        prefix = page * _log(rng, 1, 16384 // page)
        c.update(op="decode", S=_log(rng, 2, 64), longest=prefix + _log(rng, 1, 600), shortest=prefix, prefix=prefix,
                 page=page, w=_log(rng, 16, 2048))
    return c


# ---------------------------------------------------------------- what follows from a case alone

def _lens(c):
    """Cache lengths of a serving case (the tokens being appended included)."""
    rng = random.Random(c["mix"])
    low = c.get("shortest", 1)
    n = [rng.randint(low, c["longest"]) for _ in range(c["S"])]
    n[0] = c["longest"]
    if c["S"] > 1:
        n[1] = low
    return n


def _counts(c):
    """Tokens appended to each sequence: one (a decode step), or a whole prompt behind what is there."""
    lens = _lens(c)
    if c["step"]:
        return [1] * c["S"]
    rng = random.Random(c["mix"] + 1)
    return [n if i == 0 else rng.randint((n + 1) // 2, n) for i, n in enumerate(lens)]


def _size(c):
    return 2 if c["dtype"] == "bf16" else 4


def _type(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def work(case):
    c = case
    e, d, H, Hkv = _size(c), c["d"], c["H"], c["Hkv"]
    if c["op"] == "prep":
        rows = c["B"] * c["N"] * (H + 2 * Hkv)
        return {"bytes": 2 * rows * d * e, "flops": 8 * rows * d}
    if c["op"] == "prep_bwd":
        tok = c["B"] * c["N"]
        return {"bytes": tok * d * ((H + Hkv) * 3 * e + Hkv * (2 * e + 4)), "flops": 16 * tok * (H + Hkv) * d}
    if c["op"] == "append":
        tok = sum(_counts(c))
        return {"bytes": tok * (2 * (H + 2 * Hkv) * d * e + 4 * H) + Hkv * d * H * e,
                "flops": 2 * tok * Hkv * d * H + 8 * tok * (H + Hkv) * d}
    lens, w, P = _lens(c), c["w"], c["prefix"]
    G = H // Hkv

    def union(n, k):   # rows that G independent choices of k of n rows touch
        return n * (1.0 - (1.0 - k / n) ** G) if n > 0 else 0.0

    nbytes = 4 * H * P + (2 * Hkv * d * e * union(P, min(w, P)) if P else 0)
    flops = 0
    for n in lens:
        kept = min(w, n)
        nbytes += 4 * H * (n - P) + 2 * H * d * e
        rest = n - P
        nbytes += 2 * Hkv * d * e * union(rest, kept * rest / n if n else 0)
        flops += 4 * d * H * kept
    return {"bytes": int(nbytes), "flops": flops}


# ---------------------------------------------------------------- inputs

def _inv_freq(rot):
    i = torch.arange(0, rot, 2, device=DEV, dtype=torch.float64)
    return (BASE ** (-i / max(rot, 1))).float()


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _gate_values(V, Delta, A):
    """Gate values of pages V [n, Hkv, page, d]: delta [n, H, page]."""
    n, Hkv, page, d = V.shape
    out = torch.empty((n, Delta.shape[1], page), dtype=torch.float32, device=DEV)
    for i in range(0, n, 512):
        x = V[i:i + 512].permute(0, 2, 1, 3).reshape(-1, Hkv * d).float() @ Delta.float()
        out[i:i + 512] = torch.exp(A * torch.nn.functional.softplus(x)).view(-1, page, x.shape[1]).transpose(1, 2)
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    t, H, Hkv, d = _type(c), c["H"], c["Hkv"], c["d"]
    st = {"c": c}
    if "rot" in c:
        st["freq"] = _inv_freq(c["rot"])
        st["qw"] = _normal(g, (d,), torch.float32, 0.1).add_(1).to(t) if c["norm"] else None
        st["kw"] = _normal(g, (d,), torch.float32, 0.1).add_(1).to(t) if c["norm"] else None
    if c["op"] in ("prep", "prep_bwd"):
        B, N = c["B"], c["N"]
        qkv = _normal(g, (B, N, H + 2 * Hkv, d), t)   # one projection's output, heads side by side
        st.update(q=qkv[:, :, :H], k=qkv[:, :, H:H + Hkv], v=qkv[:, :, H + Hkv:])
        st["pos"] = None
        if c["far"]:
            st["pos"] = torch.randint(0, 1 << 20, (B, N), generator=g, device=DEV, dtype=torch.int32)
        heads = dict(Q=(B, H, N, d), K=(B, Hkv, N, d), V=(B, Hkv, N, d))
        if c["op"] == "prep_bwd":
            for n, s in heads.items():
                st["d" + n] = _normal(g, s, t)
            st["dVg"] = _normal(g, heads["V"], torch.float32, 0.1)
        if own:
            import trainable_dynamic_mask_b200 as dma
            st["p"] = dma.make_params(B, H, Hkv, N, d, 1, Nq=N, dtype=c["dtype"])
            st["r"] = dma.make_prep(st["freq"], q_weight=st["qw"], k_weight=st["kw"], eps=EPS, positions=st["pos"],
                                    interleaved=c["inter"])
            if c["op"] == "prep":
                for n, s in heads.items():
                    st[n + "o"] = torch.empty(s, dtype=t, device=DEV)
            else:
                st["grad"] = torch.empty_like(qkv)
                st["dqw"] = torch.empty(d, device=DEV) if c["norm"] else None
                st["dkw"] = torch.empty(d, device=DEV) if c["norm"] else None
                st["ws"] = dma.alloc_prep_workspace(st["p"], st["r"])
        return st
    S, page, lens, P = c["S"], c["page"], _lens(c), c.get("prefix", 0)
    st["lens_host"] = lens
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    # pages in arbitrary order; a shared prefix's pages stand in every sequence's table
    per = -(-c["longest"] // page)
    np_ = P // page
    n_pages = np_ + S * (per - np_) + 3
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.empty((S, per), dtype=torch.int32, device=DEV)
    table[:, :np_] = ids[:np_]
    table[:, np_:] = ids[np_:np_ + S * (per - np_)].view(S, per - np_)
    st["table"] = table
    st["Kp"] = torch.empty((n_pages, Hkv, page, d), dtype=t, device=DEV)
    st["Vp"] = torch.empty((n_pages, Hkv, page, d), dtype=t, device=DEV)
    for i in range(0, n_pages, 1024):
        for x in (st["Kp"], st["Vp"]):
            x[i:i + 1024] = _normal(g, x[i:i + 1024].shape, t)
    st["Delta"] = _normal(g, (Hkv * d, H), t, 0.02)
    st["A"] = -torch.rand(H, generator=g, device=DEV)
    st["dp"] = _gate_values(st["Vp"], st["Delta"], st["A"])
    if c["op"] == "append":
        cnt = _counts(c)
        T = sum(cnt)
        seq = [s for s in range(S) for _ in range(cnt[s])]
        pos = [lens[s] - cnt[s] + i for s in range(S) for i in range(cnt[s])]
        st["seq"] = torch.tensor(seq, device=DEV)
        st["pos"] = torch.tensor(pos, device=DEV)
        starts = [0]
        for n in cnt:
            starts.append(starts[-1] + n)
        st["starts"] = None if c["step"] else torch.tensor(starts, dtype=torch.int32, device=DEV)
        qkv = _normal(g, (T, H + 2 * Hkv, d), t)
        st.update(q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:])
        st["Qo"] = torch.empty((T, H, d), dtype=t, device=DEV)
    else:
        st["Q"] = _normal(g, (S, H, d), t)
        st["O"] = torch.empty((S, H, d), dtype=t, device=DEV)
        st["LSE"] = torch.empty((S, H), dtype=torch.float32, device=DEV)
    if own:
        import trainable_dynamic_mask_b200 as dma
        st["p"] = dma.make_params(S, H, Hkv, c["longest"], d, c.get("w", 1), Nq=1, dtype=c["dtype"])
        st["pages"] = dma.make_pages(st["p"], st["Kp"], st["Vp"], st["dp"], table, st["lens"], prefix=P)
        st["ws"] = dma.alloc_paged_workspace(st["p"], st["pages"])
        if c["op"] == "append":
            st["r"] = dma.make_prep(st["freq"], q_weight=st["qw"], k_weight=st["kw"], eps=EPS, interleaved=c["inter"])
    return st


# ---------------------------------------------------------------- the plain form

def _halves(x, rot, inter):
    """The two members of every rotated pair: [..., rot / 2] each."""
    if inter:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _joined(a, b, rest, inter):
    if inter:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _turned(x, pos, freq, inter, back=False):
    """x [..., heads, d] rotated by the angles pos x freq (pos [...]); back: by the opposite angles."""
    rot = 2 * freq.numel()
    a = pos.double()[..., None, None] * freq.double()
    co, si = a.cos().float(), a.sin().float()
    if back:
        si = -si
    u, v = _halves(x, rot, inter)
    return _joined(u * co - v * si, v * co + u * si, x[..., rot:], inter)


def _normed(x, weight):
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _positions(st):
    c = st["c"]
    if st["pos"] is not None:
        return st["pos"]
    return torch.arange(c["N"], device=DEV).expand(c["B"], c["N"])


def _plain_prep(st):
    c = st["c"]
    pos = _positions(st)
    out = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        y = _turned(_normed(x.float(), w), pos, st["freq"], c["inter"])
        out.append(y.to(x.dtype).transpose(1, 2).contiguous())
    return out + [st["v"].transpose(1, 2).contiguous()]


def _plain_prep_bwd(st):
    c = st["c"]
    pos = _positions(st)
    rows, weights = [], []
    for x, w, dy in ((st["q"], st["qw"], st["dQ"]), (st["k"], st["kw"], st["dK"])):
        gy = _turned(dy.float().transpose(1, 2), pos, st["freq"], c["inter"], back=True)
        if w is None:
            rows.append(gy.to(x.dtype))
            continue
        xf = x.float()
        r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
        gw = gy * w.float()
        rows.append((r * gw - xf * r.pow(3) * (xf * gw).mean(-1, keepdim=True)).to(x.dtype))
        weights.append((gy * xf * r).sum((0, 1, 2), dtype=torch.float64).float())
    rows.append((st["dV"].float() + st["dVg"]).to(st["dV"].dtype).transpose(1, 2))
    return [torch.cat(rows, 2)] + weights


def _plain_append(st):
    c = st["c"]
    k = _turned(_normed(st["k"].float(), st["kw"]), st["pos"], st["freq"], c["inter"])
    q = _turned(_normed(st["q"].float(), st["qw"]), st["pos"], st["freq"], c["inter"])
    x = st["v"].float().flatten(1) @ st["Delta"].float()
    delta = torch.exp(st["A"] * (torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))))
    page = st["table"][st["seq"], st["pos"] // c["page"]].long()
    slot = st["pos"] % c["page"]
    st["Kp"][page, :, slot] = k.to(st["Kp"].dtype)
    st["Vp"][page, :, slot] = st["v"]
    st["dp"][page, :, slot] = delta
    return [q.to(st["q"].dtype), st["Kp"], st["Vp"], st["dp"]]


def _plain_decode(st):
    c = st["c"]
    H, Hkv, d, page = c["H"], c["Hkv"], c["d"], c["page"]
    group = torch.arange(H, device=DEV)[:, None] // (H // Hkv)
    outs, lses = [], []
    for s, n in enumerate(st["lens_host"]):
        if n == 0:
            outs.append(torch.zeros((H, d), device=DEV))
            lses.append(torch.full((H,), float("-inf"), device=DEV))
            continue
        pages = st["table"][s].long()
        delta = st["dp"][pages].transpose(0, 1).reshape(H, -1)[:, :n]
        val, idx = torch.sort(delta, dim=1, descending=True, stable=True)
        val, idx = val[:, :c["w"]], idx[:, :c["w"]]
        where = pages[idx // page]
        k = st["Kp"][where, group, idx % page].float()
        v = st["Vp"][where, group, idx % page].float()
        x = (k @ st["Q"][s].float()[:, :, None]).squeeze(2) / math.sqrt(d) + val
        m = x.max(1, keepdim=True).values
        e = torch.exp(x - m)
        total = e.sum(1, keepdim=True)
        outs.append(((e / total)[:, None] @ v).squeeze(1))
        lses.append((m + total.log()).squeeze(1))
    return [torch.stack(outs).to(st["Q"].dtype), torch.stack(lses)]


# ---------------------------------------------------------------- the framework's calls

def _own(st):
    import trainable_dynamic_mask_b200 as dma
    c = st["c"]
    if c["op"] == "prep":
        dma.prep(st["p"], st["r"], st["q"], st["k"], st["v"], st["Qo"], st["Ko"], st["Vo"])
        return [st["Qo"], st["Ko"], st["Vo"]]
    if c["op"] == "prep_bwd":
        H, Hkv = c["H"], c["Hkv"]
        gr = st["grad"]
        dma.prep_bwd(st["p"], st["r"], st["q"], st["k"], st["dQ"], st["dK"], st["dV"], st["dVg"], gr[:, :, :H],
                     gr[:, :, H:H + Hkv], gr[:, :, H + Hkv:], st["dqw"], st["dkw"], st["ws"])
        return [gr] + ([st["dqw"], st["dkw"]] if c["norm"] else [])
    if c["op"] == "append":
        dma.paged_append(st["p"], st["pages"], st["r"], st["q"], st["k"], st["v"], st["Delta"], st["A"], st["Qo"],
                         st["ws"], starts=st["starts"])
        return [st["Qo"], st["Kp"], st["Vp"], st["dp"]]
    dma.paged_topk(st["p"], st["pages"], st["ws"])
    dma.paged_attn(st["p"], st["pages"], st["Q"], st["ws"], st["O"], st["LSE"])
    return [st["O"], st["LSE"]]


def run(state):
    if own:
        return _own(state)
    return {"prep": _plain_prep, "prep_bwd": _plain_prep_bwd, "append": _plain_append,
            "decode": _plain_decode}[state["c"]["op"]](state)


# ---------------------------------------------------------------- the definition in 64 bits

def _matrix(pos, freq, inter, d):
    """Rotation matrices R [..., d, d] of the positions (y = R x)."""
    rot = 2 * freq.numel()
    R = torch.eye(d, dtype=torch.float64, device=DEV).expand(*pos.shape, d, d).clone()
    for i in range(freq.numel()):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        ang = pos.double() * freq[i].double()
        R[..., a, a] = R[..., b, b] = torch.cos(ang)
        R[..., b, a] = torch.sin(ang)
        R[..., a, b] = -torch.sin(ang)
    return R


def _by_chunks(fn, pos, *rows):
    """fn over at most 2048 flattened positions at a time (the rotation matrices are d x d each)."""
    return torch.cat([fn(pos[i:i + 2048], *(r[i:i + 2048] for r in rows)) for i in range(0, pos.numel(), 2048)])


def _exact_rows(x, weight, pos, freq, inter):
    """x [tokens, heads, d] normed and rotated."""
    def part(p, v):
        v = v.double()
        if weight is not None:
            v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + EPS) * weight.double()
        return torch.einsum("tij,thj->thi", _matrix(p, freq, inter, v.shape[-1]), v)
    return _by_chunks(part, pos, x)


def _exact_grad(x, weight, dy, pos, freq, inter):
    """Gradients of the inputs [tokens, heads, d] and of the weight, through the Jacobian of the norm."""
    sums = []

    def part(p, v, g):
        v, g = v.double(), g.double()
        d = v.shape[-1]
        g = torch.einsum("tij,thi->thj", _matrix(p, freq, inter, d), g)
        if weight is None:
            return g
        n = torch.sqrt((v * v).sum(-1, keepdim=True) / d + EPS)
        unit = v / n
        sums.append((g * unit).sum((0, 1)))
        gw = g * weight.double()
        return (gw - unit * ((unit * gw).sum(-1, keepdim=True) / d)) / n
    out = _by_chunks(part, pos, x, dy)
    return out, sum(sums) if sums else None


def _exact_decode(st):
    c = st["c"]
    H, Hkv, d, page, w = c["H"], c["Hkv"], c["d"], c["page"], c["w"]
    O = torch.zeros((c["S"], H, d), dtype=torch.float64, device=DEV)
    L = torch.full((c["S"], H), float("-inf"), dtype=torch.float64, device=DEV)
    for s, n in enumerate(st["lens_host"]):
        if n == 0:
            continue
        i = torch.arange(n, device=DEV)
        pg, sl = st["table"][s].long()[i // page], i % page
        k = st["Kp"][pg, :, sl].transpose(0, 1).double()      # [Hkv, n, d]
        v = st["Vp"][pg, :, sl].transpose(0, 1).double()
        delta = st["dp"][pg, :, sl].t().double()              # [H, n]
        # kept: more than w - 1 positions may not come before it (a larger delta, or an equal one earlier)
        if n > w:
            edge = torch.topk(delta, w, dim=1).values[:, -1:]
            above, equal = delta > edge, delta == edge
            keep = above | (equal & (equal.cumsum(1) <= w - above.sum(1, keepdim=True)))
        else:
            keep = torch.ones_like(delta, dtype=torch.bool)
        q = st["Q"][s].double().view(Hkv, H // Hkv, d)
        x = torch.bmm(q, k.transpose(1, 2)).view(H, n) * d ** -0.5 + delta
        x = x.masked_fill(~keep, float("-inf"))
        L[s] = torch.logsumexp(x, 1)
        a = torch.exp(x - L[s][:, None]).view(Hkv, H // Hkv, n)
        O[s] = torch.bmm(a, v).view(H, d)
    return [O, L]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["op"] == "decode":
        return _exact_decode(st)
    if c["op"] == "append":
        pos = st["pos"]
        q = _exact_rows(st["q"], st["qw"], pos, st["freq"], c["inter"])
        k = _exact_rows(st["k"], st["kw"], pos, st["freq"], c["inter"])
        x = torch.einsum("tr,rh->th", st["v"].double().reshape(pos.numel(), -1), st["Delta"].double())
        gate = torch.exp(st["A"].double() * torch.logaddexp(x, torch.zeros_like(x)))
        Kp, Vp, dp = st["Kp"].double(), st["Vp"].double(), st["dp"].double()
        pg, sl = st["table"][st["seq"], pos // c["page"]].long(), pos % c["page"]
        Kp[pg, :, sl], Vp[pg, :, sl], dp[pg, :, sl] = k, st["v"].double(), gate
        return [q, Kp, Vp, dp]
    B, N, d = c["B"], c["N"], c["d"]
    pos = _positions(st).reshape(-1)
    if c["op"] == "prep":
        out = [_exact_rows(st[n].reshape(B * N, -1, d), st[n + "w"], pos, st["freq"], c["inter"]) for n in "qk"]
        out.append(st["v"].double().reshape(B * N, -1, d))
        return [o.view(B, N, -1, d).transpose(1, 2) for o in out]
    rows, weights = [], []
    for n in "qk":
        dy = st["d" + n.upper()].transpose(1, 2).reshape(B * N, -1, d)
        g, gw = _exact_grad(st[n].reshape(B * N, -1, d), st[n + "w"], dy, pos, st["freq"], c["inter"])
        rows.append(g)
        weights.append(gw)
    rows.append((st["dV"].double() + st["dVg"].double()).transpose(1, 2).reshape(B * N, -1, d))
    grad = torch.cat(rows, 1).view(B, N, -1, d)
    return [grad] + (weights if c["norm"] else [])
