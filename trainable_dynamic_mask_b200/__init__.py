"""Dynamic Mask Attention hot path on B200 (sm_100a): Python binding of libdma.

Every function here marshals arguments and calls the C ABI declared in
include/dma.h; all computation runs in the library's CUDA kernels.  PyTorch is
used for device memory and streams only.  Functions raise DmaError when the
library returns a status other than DMA_OK.

Method: "Trainable Dynamic Mask Sparse Attention" (HF blog "dmattn"):
gate delta = exp(softplus(v Delta) A), causal top-w mask, masked attention
softmax(q k^T / sqrt(d) + m) v, with its backward.
"""
from __future__ import annotations

import ctypes

from ._lib import (BLOCK_Q, DMA_BF16, DMA_F32, DMA_FLAG_FORWARD_ONLY, DmaCpLayout, DmaError, DmaPagedLayout, DmaPages,
                   DmaParams, DmaPrep, DmaPrepStrides, DmaWsLayout, LIB_PATH, check, exported_names, load)

__all__ = [
    "BLOCK_Q", "DMA_BF16", "DMA_F32", "DmaError", "DmaParams", "LIB_PATH", "load", "exported_names",
    "make_params", "workspace_size", "workspace_layout", "gate", "topk_mask", "topk_append", "gate_append",
    "attn_fwd", "attn_bwd",
    "gate_bwd", "gate_bwd_noalloc", "check_device_status", "clear_device_status", "selftest_bounded_wait",
    "abi_version", "alloc_workspace", "forward",
    "backward", "cp_layout", "cp_candidates", "cp_compact",
    "DmaPrep", "make_prep", "prep", "prep_bwd", "prep_workspace_size", "alloc_prep_workspace",
    "DmaPages", "make_pages", "paged_layout", "paged_append", "paged_topk", "paged_attn", "alloc_paged_workspace",
]


def make_params(B, H, Hkv, N, d, w, Nq=None, scale=0.0, dtype="bf16", w_heads=None,
                forward_only=False) -> DmaParams:
    """dma_params_t for a problem (Nq defaults to N; Nq=1 is decode).

    forward_only: no backward follows (DMA_FLAG_FORWARD_ONLY): the forward keeps
    nothing for it in the workspace.

    w_heads: None, or per-head windows as a device int32 tensor of H values (or its
    device address); w must then be the largest of them.  The caller keeps the
    tensor alive for as long as the parameters are used."""
    dt = {"bf16": DMA_BF16, "f32": DMA_F32}[dtype] if isinstance(dtype, str) else int(dtype)
    return DmaParams(B=B, H=H, Hkv=Hkv, N=N, Nq=N if Nq is None else Nq, d=d, w=w,
                     scale=float(scale), dtype=dt, flags=DMA_FLAG_FORWARD_ONLY if forward_only else 0,
                     w_heads=_ptr(w_heads))


def abi_version() -> int:
    return int(load().dma_abi_version())


def workspace_size(p: DmaParams) -> int:
    n = ctypes.c_size_t(0)
    check("dma_workspace_size", load().dma_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


def workspace_layout(p: DmaParams) -> DmaWsLayout:
    lay = DmaWsLayout()
    check("dma_workspace_layout", load().dma_workspace_layout(ctypes.byref(p), ctypes.byref(lay)))
    return lay


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to libdma must be contiguous")
    return t.data_ptr()


def _nbytes(t):
    return 0 if t is None else t.nbytes


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def gate(p, V, Delta, A, delta, x_save=None, workspace=None, stream=None):
    check("dma_gate", load().dma_gate(ctypes.byref(p), _ptr(V), _ptr(Delta), _ptr(A), _ptr(delta),
                                      _ptr(x_save), _ptr(workspace), _nbytes(workspace), _stream(stream)))


def topk_mask(p, delta, evict, workspace, stream=None):
    check("dma_topk_mask", load().dma_topk_mask(ctypes.byref(p), _ptr(delta), _ptr(evict),
                                                _ptr(workspace), _nbytes(workspace), _stream(stream)))


def topk_append(p, delta, workspace, stream=None):
    """Decode selection after one key is appended (p.N = the new cache length)."""
    check("dma_topk_append", load().dma_topk_append(ctypes.byref(p), _ptr(delta), _ptr(workspace),
                                                    _nbytes(workspace), _stream(stream)))


def gate_append(p, V, Delta, A, delta, x_save=None, stream=None):
    """Gate of the last key position only (delta[:, :, p.N - 1])."""
    check("dma_gate_append", load().dma_gate_append(ctypes.byref(p), _ptr(V), _ptr(Delta), _ptr(A), _ptr(delta),
                                                    _ptr(x_save), _stream(stream)))


def attn_fwd(p, Q, K, V, delta, evict, workspace, O, LSE, stream=None):
    check("dma_attn_fwd", load().dma_attn_fwd(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(delta),
                                              _ptr(evict), _ptr(workspace), _nbytes(workspace), _ptr(O),
                                              _ptr(LSE), _stream(stream)))


def attn_bwd(p, Q, K, V, delta, evict, workspace, O, LSE, dO, dQ, dK, dV, d_delta, stream=None):
    check("dma_attn_bwd", load().dma_attn_bwd(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(delta),
                                              _ptr(evict), _ptr(workspace), _nbytes(workspace), _ptr(O),
                                              _ptr(LSE), _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV),
                                              _ptr(d_delta), _stream(stream)))


def gate_bwd(p, V, Delta, A, x_save, delta, d_delta, dDelta, dA, dV_gate, workspace, stream=None):
    check("dma_gate_bwd", load().dma_gate_bwd(ctypes.byref(p), _ptr(V), _ptr(Delta), _ptr(A),
                                              _ptr(x_save), _ptr(delta), _ptr(d_delta), _ptr(dDelta),
                                              _ptr(dA), _ptr(dV_gate), _ptr(workspace), _nbytes(workspace),
                                              _stream(stream)))


def gate_bwd_noalloc(p, V, Delta, A, x_save, delta, d_delta, dDelta, dA, dV_gate, stream=None):
    """dma_gate_bwd without a workspace, for callers that may not allocate device
    memory; its scratch is a fixed array inside the library (see include/dma.h)."""
    check("dma_gate_bwd_noalloc", load().dma_gate_bwd_noalloc(ctypes.byref(p), _ptr(V), _ptr(Delta), _ptr(A),
                                                              _ptr(x_save), _ptr(delta), _ptr(d_delta),
                                                              _ptr(dDelta), _ptr(dA), _ptr(dV_gate),
                                                              _stream(stream)))


def check_device_status(p, workspace, stream=None) -> int:
    code = ctypes.c_int32(0)
    load().dma_check_device_status(ctypes.byref(p), _ptr(workspace), _stream(stream), ctypes.byref(code))
    return int(code.value)


def selftest_bounded_wait(p, workspace, limit_cycles=1_000_000, stream=None):
    """Launch the device-side bounded-wait check (a wait that must give up and report)."""
    check("dma_selftest_bounded_wait", load().dma_selftest_bounded_wait(ctypes.byref(p), _ptr(workspace),
                                                                        _nbytes(workspace), int(limit_cycles),
                                                                        _stream(stream)))


def clear_device_status(p, workspace, stream=None):
    check("dma_clear_device_status", load().dma_clear_device_status(ctypes.byref(p), _ptr(workspace),
                                                                    _stream(stream)))


# ---------------------------------------------------------------- context-parallel prefill

def cp_layout(p, prefix_len, n_prev) -> DmaCpLayout:
    """Candidate-buffer and workspace sizes of shard problem p (see trainable_dynamic_mask_b200.cp)."""
    lay = DmaCpLayout()
    check("dma_cp_layout", load().dma_cp_layout(ctypes.byref(p), int(prefix_len), int(n_prev), ctypes.byref(lay)))
    return lay


def cp_candidates(p, shard_start, delta, K, V, cand, workspace, stream=None):
    check("dma_cp_candidates", load().dma_cp_candidates(ctypes.byref(p), int(shard_start), _ptr(delta), _ptr(K),
                                                        _ptr(V), _ptr(cand), _nbytes(cand), _ptr(workspace),
                                                        _nbytes(workspace), _stream(stream)))


def cp_compact(p, prefix_len, n_prev, cands, delta, K, V, delta_c, Kc, Vc, pos_c, workspace, stream=None):
    check("dma_cp_compact", load().dma_cp_compact(ctypes.byref(p), int(prefix_len), int(n_prev), _ptr(cands),
                                                  _nbytes(cands), _ptr(delta), _ptr(K), _ptr(V), _ptr(delta_c),
                                                  _ptr(Kc), _ptr(Vc), _ptr(pos_c), _ptr(workspace),
                                                  _nbytes(workspace), _stream(stream)))


# ---------------------------------------------------------------- projections to inputs

class _Torch:
    """What every call needs of torch, looked up once (a small call takes about as long as its checks)."""
    ready = False

    @classmethod
    def get(cls):
        import torch
        torch.cuda.current_device()   # CUDA is up, or this says why not
        cls.types = {DMA_BF16: torch.bfloat16, DMA_F32: torch.float32}
        cls.f32, cls.i32 = torch.float32, torch.int32
        cls.device = staticmethod(torch._C._cuda_getDevice)
        cls.stream = staticmethod(torch._C._cuda_getCurrentRawStream)   # its address: no Stream object is made
        cls.ready = True
        return cls


def _torch():
    return _Torch if _Torch.ready else _Torch.get()


def _dense(name, t, shape, dtype, dev):
    """Address of a dense tensor of that shape and type on the current device dev (None: NULL)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(name, t, shape, dtype, dev)
    raise ValueError(f"{name} must be contiguous")


def _rows(name, t, shape, dtype, dev, out):
    """Address of rows [B, N, heads, d] (or [T, heads, d]) at any strides; those of all but the channels go
    into out (of a dimension of one element, which has no stride to speak of, 0)."""
    if t is None:
        return None
    st = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or st[-1] != 1:
        _refuse(name, t, shape, dtype, dev)
        raise ValueError(f"{name}: the channels of a row must be contiguous")
    if len(st) == 4:
        out[:] = (st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else 0, st[2] if shape[2] > 1 else 0)
    else:
        out[:] = (0, st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else 0)
    return t.data_ptr()


def _refuse(name, t, shape, dtype, dev):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current device (cuda:{dev}), not {t.device}")


def make_prep(inv_freq, q_weight=None, k_weight=None, eps=1e-6, positions=None, first=0, interleaved=False) -> DmaPrep:
    """dma_prep_t: the norm and rotation between the projections and the attention.

    inv_freq: device float32 [rot / 2] (radians per position), rotating the first rot
    channels; None: no rotation.  q_weight, k_weight: [d] in the storage type; None: no
    norm.  positions: device int32 [B, N]; None: first, first + 1, ...  interleaved: the
    pairs are neighbouring channels instead of the two halves.  The result keeps the
    tensors alive."""
    r = DmaPrep(inv_freq=_ptr(inv_freq), positions=_ptr(positions), q_weight=_ptr(q_weight), k_weight=_ptr(k_weight),
                eps=float(eps), rot=0 if inv_freq is None else 2 * inv_freq.numel(),
                interleaved=1 if interleaved else 0, first=int(first))
    r.tensors = (inv_freq, q_weight, k_weight, positions)
    r.fits = None
    return r


def _check_prep_tensors(p, r, dev):
    """The weights and positions of r fit p (looked at again when p's sizes change)."""
    key = (p.B, p.N, p.d, p.dtype, dev)
    if r.fits != key:
        tt = _torch()
        freq, qw, kw, pos = r.tensors
        _dense("inv_freq", freq, (r.rot // 2,), tt.f32, dev)
        _dense("q_weight", qw, (p.d,), tt.types[p.dtype], dev)
        _dense("k_weight", kw, (p.d,), tt.types[p.dtype], dev)
        _dense("positions", pos, (p.B, p.N), tt.i32, dev)
        r.fits = key


def prep(p, r, q, k, v, Q, K, V, stream=None):
    """Projections q [B, N, H, d], k, v [B, N, Hkv, d] (any strides) to the attention's inputs
    Q [B, H, N, d], K, V [B, Hkv, N, d]: per-head norm, rotation and transposition in one pass.
    v and V may be None together."""
    call, tt = load().dma_prep, _torch()
    dev, t = tt.device(), tt.types[p.dtype]
    B, H, Hkv, N, d = p.B, p.H, p.Hkv, p.N, p.d
    _check_prep_tensors(p, r, dev)
    st = DmaPrepStrides()
    check("dma_prep", call(
        p, r, st, _rows("q", q, (B, N, H, d), t, dev, st.q), _rows("k", k, (B, N, Hkv, d), t, dev, st.k),
        _rows("v", v, (B, N, Hkv, d), t, dev, st.v), _dense("Q", Q, (B, H, N, d), t, dev),
        _dense("K", K, (B, Hkv, N, d), t, dev), _dense("V", V, (B, Hkv, N, d), t, dev),
        tt.stream(dev) if stream is None else _stream(stream)))


def prep_workspace_size(p, r) -> int:
    n = ctypes.c_size_t(0)
    check("dma_prep_workspace_size", load().dma_prep_workspace_size(p, r, n))
    return int(n.value)


def prep_bwd(p, r, q, k, dQ, dK, dV, dV_gate, dq, dk, dv, dq_weight, dk_weight, workspace, stream=None):
    """Gradients of prep's inputs from those of its outputs: dq, dk, dv are written at their own
    strides ([B, N, heads, d]), dV_gate (float32, or None) is added to dV, dq_weight and dk_weight are
    float32 [d] (None: not wanted); q, k as in prep (None where there is no weight)."""
    call, tt = load().dma_prep_bwd, _torch()
    dev, t, f = tt.device(), tt.types[p.dtype], tt.f32
    B, H, Hkv, N, d = p.B, p.H, p.Hkv, p.N, p.d
    _check_prep_tensors(p, r, dev)
    st, gst = DmaPrepStrides(), DmaPrepStrides()
    sq, sk, hq, hk = (B, N, H, d), (B, N, Hkv, d), (B, H, N, d), (B, Hkv, N, d)
    check("dma_prep_bwd", call(
        p, r, st, gst, _rows("q", q, sq, t, dev, st.q), _rows("k", k, sk, t, dev, st.k), _dense("dQ", dQ, hq, t, dev),
        _dense("dK", dK, hk, t, dev), _dense("dV", dV, hk, t, dev), _dense("dV_gate", dV_gate, hk, f, dev),
        _rows("dq", dq, sq, t, dev, gst.q), _rows("dk", dk, sk, t, dev, gst.k), _rows("dv", dv, sk, t, dev, gst.v),
        _dense("dq_weight", dq_weight, (d,), f, dev), _dense("dk_weight", dk_weight, (d,), f, dev),
        _workspace(workspace, dev), _nbytes(workspace), tt.stream(dev) if stream is None else _stream(stream)))


def _workspace(ws, dev):
    """Address of a workspace on the current device dev."""
    if ws is None:
        return None
    if ws.get_device() != dev:
        raise ValueError(f"the workspace must be on the current device (cuda:{dev}), not {ws.device}")
    return _ptr(ws)


# ---------------------------------------------------------------- paged cache

def make_pages(p, K, V, delta, table, lens, prefix=0) -> DmaPages:
    """dma_pages_t: the paged cache of p's sequences.  K, V [n_pages, Hkv, page, d], delta
    [n_pages, H, page] float32, table int32 [B, max_pages], lens int32 [B] (device tensors, which the
    result keeps alive; they may be written to between calls).  prefix: leading positions that every
    sequence shares, a multiple of the page length.  The calls below take these pages with parameters of the
    same heads, channels and type, for as many sequences or fewer (the first ones)."""
    if K.dim() != 4 or table.dim() != 2:
        raise ValueError("K must be [n_pages, Hkv, page, d] and table [B, max_pages]")
    tt = _torch()
    dev, t = tt.device(), tt.types[p.dtype]
    n, page = K.shape[0], K.shape[2]
    rows = (n, p.Hkv, page, p.d)
    c = DmaPages(K=_dense("K", K, rows, t, dev), V=_dense("V", V, rows, t, dev),
                 delta=_dense("delta", delta, (n, p.H, page), tt.f32, dev),
                 table=_dense("table", table, (p.B, table.shape[1]), tt.i32, dev),
                 lens=_dense("lens", lens, (p.B,), tt.i32, dev), n_pages=n, page=page,
                 max_pages=table.shape[1], prefix=int(prefix))
    c.tensors, c.device = (K, V, delta, table, lens), dev
    c.sequences, c.rows, c.fits = p.B, (p.H, p.Hkv, p.d, p.dtype), (None, None)
    return c


def _same_problem(p, c):
    """p reads pages as they were made: the same heads, channels and type, and no more sequences (the library
    sees addresses alone)."""
    if p.B > c.sequences or (p.H, p.Hkv, p.d, p.dtype) != c.rows:
        raise ValueError(f"the pages were made for B <= {c.sequences} and (H, Hkv, d, dtype) = {c.rows}, not for "
                         f"B = {p.B} and {(p.H, p.Hkv, p.d, p.dtype)}")


def _check_pages(p, c, dev):
    """(B, H, Hkv, d, storage type) of p, whose pages fit it (looked at again when any field of p changes) and
    are on the current device dev."""
    if c.device != dev:
        raise ValueError(f"the pages are on cuda:{c.device}, the current device is cuda:{dev}")
    key, fits = bytes(p), c.fits
    if fits[0] != key:
        _same_problem(p, c)
        c.fits = fits = key, (p.B, p.H, p.Hkv, p.d, _torch().types[p.dtype])
    return fits[1]


def paged_layout(p, c) -> DmaPagedLayout:
    call = load().dma_paged_layout
    if hasattr(c, "rows"):   # pages described by hand are their maker's responsibility
        _same_problem(p, c)
    lay = DmaPagedLayout()
    check("dma_paged_layout", call(p, c, lay))
    return lay


def paged_append(p, c, r, q, k, v, Delta, A, Q, workspace, starts=None, stream=None):
    """Appends tokens to the cache from their projections q [T, H, d], k, v [T, Hkv, d] (any strides),
    as the last positions of c.lens: K normed and rotated, V, the gate values; Q [T, H, d] receives the
    normed and rotated queries (q and Q may be None together).  starts: device int32 [B + 1], the
    sequences' token ranges; None: one token each."""
    call, tt = load().dma_paged_append, _torch()
    dev, f, T = tt.device(), tt.f32, k.shape[0]
    B, H, Hkv, d, t = _check_pages(p, c, dev)
    _check_prep_tensors(p, r, dev)
    st = DmaPrepStrides()
    check("dma_paged_append", call(
        p, c, r, st, T, _dense("starts", starts, (B + 1,), tt.i32, dev),
        _rows("q", q, (T, H, d), t, dev, st.q), _rows("k", k, (T, Hkv, d), t, dev, st.k),
        _rows("v", v, (T, Hkv, d), t, dev, st.v), _dense("Delta", Delta, (Hkv * d, H), t, dev),
        _dense("A", A, (H,), f, dev), _dense("Q", Q, (T, H, d), t, dev), _workspace(workspace, dev),
        _nbytes(workspace), tt.stream(dev) if stream is None else _stream(stream)))


def paged_topk(p, c, workspace, stream=None):
    """Selection of every (sequence, head) over its cache, into the workspace."""
    call, tt = load().dma_paged_topk, _torch()
    dev = tt.device()
    _check_pages(p, c, dev)
    check("dma_paged_topk", call(p, c, _workspace(workspace, dev), _nbytes(workspace),
                                 tt.stream(dev) if stream is None else _stream(stream)))


def paged_attn(p, c, Q, workspace, O, LSE, stream=None):
    """Attention of one query [B, H, d] for each sequence over the keys paged_topk selected."""
    call, tt = load().dma_paged_attn, _torch()
    dev = tt.device()
    B, H, _, d, t = _check_pages(p, c, dev)
    shape = (B, H, d)
    check("dma_paged_attn", call(
        p, c, _dense("Q", Q, shape, t, dev), _workspace(workspace, dev), _nbytes(workspace),
        _dense("O", O, shape, t, dev), _dense("LSE", LSE, (B, H), tt.f32, dev),
        tt.stream(dev) if stream is None else _stream(stream)))


# ---------------------------------------------------------------- convenience (torch allocation)

def alloc_paged_workspace(p, c, device="cuda"):
    """A workspace for the paged calls (torch allocation, status word cleared)."""
    import torch
    return torch.zeros(paged_layout(p, c).bytes, dtype=torch.uint8, device=device)


def alloc_prep_workspace(p, r, device="cuda"):
    """A workspace for prep_bwd (torch allocation)."""
    import torch
    return torch.empty(prep_workspace_size(p, r), dtype=torch.uint8, device=device)


def alloc_workspace(p, device="cuda", stream=None):
    """A workspace for problem p (torch allocation) with its status word cleared."""
    import torch
    ws = torch.empty(workspace_size(p), dtype=torch.uint8, device=device)
    clear_device_status(p, ws, stream)
    return ws


def forward(p, Q, K, V, Delta, A, workspace=None, stream=None):
    """gate -> top-w mask -> attention forward.  Allocates the outputs (and the
    workspace if none is given) with torch on Q's device; returns a dict with
    delta, x, evict (None for decode), O, LSE, workspace."""
    import torch
    dev = Q.device
    ws = workspace if workspace is not None else alloc_workspace(p, dev, stream)
    f32 = torch.float32
    delta = torch.empty((p.B, p.H, p.N), dtype=f32, device=dev)
    x = torch.empty((p.B, p.H, p.N), dtype=f32, device=dev)
    decode = p.Nq == 1 and p.N > 1
    evict = None if decode else torch.empty((p.B, p.H, p.N), dtype=torch.int32, device=dev)
    O = torch.empty((p.B, p.H, p.Nq, p.d), dtype=Q.dtype, device=dev)
    LSE = torch.empty((p.B, p.H, p.Nq), dtype=f32, device=dev)
    gate(p, V, Delta, A, delta, x, ws, stream)
    topk_mask(p, delta, evict, ws, stream)
    attn_fwd(p, Q, K, V, delta, evict, ws, O, LSE, stream)
    return {"delta": delta, "x": x, "evict": evict, "O": O, "LSE": LSE, "workspace": ws}


def backward(p, Q, K, V, Delta, A, fwd, dO, stream=None):
    """Attention backward then gate backward for the outputs of forward().
    Returns dQ, dK, dV (attention part), dV_gate, d_delta, dDelta, dA."""
    import torch
    dev = Q.device
    f32 = torch.float32
    ws = fwd["workspace"]
    dQ = torch.empty_like(Q)
    dK = torch.empty_like(K)
    dV = torch.empty_like(V)
    dd = torch.empty((p.B, p.H, p.N), dtype=f32, device=dev)
    attn_bwd(p, Q, K, V, fwd["delta"], fwd["evict"], ws, fwd["O"], fwd["LSE"], dO, dQ, dK, dV, dd, stream)
    dDelta = torch.empty(tuple(Delta.shape), dtype=f32, device=dev)
    dA = torch.empty((p.H,), dtype=f32, device=dev)
    dVg = torch.empty(tuple(V.shape), dtype=f32, device=dev)
    gate_bwd(p, V, Delta, A, fwd["x"], fwd["delta"], dd, dDelta, dA, dVg, ws, stream)
    return {"dQ": dQ, "dK": dK, "dV": dV, "d_delta": dd, "dDelta": dDelta, "dA": dA, "dV_gate": dVg}
