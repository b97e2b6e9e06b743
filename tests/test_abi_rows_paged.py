"""Argument checks of the calls between the projections and the attention (dma_prep, dma_prep_bwd) and of
the paged cache (dma_paged_*), all on the host: every call below is refused, or asks for sizes only.  No
test here touches a GPU."""
import ctypes
import os
import subprocess
import sys

import pytest

import trainable_dynamic_mask_b200 as dma
from trainable_dynamic_mask_b200 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 1 << 20   # 16-byte aligned, never dereferenced on the host


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    if not os.path.exists(_lib.LIB_PATH):
        from trainable_dynamic_mask_b200 import build
        build.build()
    return dma.load()


def _prep(**kw):
    f = dict(inv_freq=FAKE, positions=None, q_weight=FAKE, k_weight=FAKE, eps=1e-6, rot=64, interleaved=0, first=0)
    f.update(kw)
    return _lib.DmaPrep(**f)


def _pages(**kw):
    f = dict(K=FAKE, V=FAKE, delta=FAKE, table=FAKE, lens=FAKE, n_pages=100, page=16, max_pages=20, prefix=0)
    f.update(kw)
    return _lib.DmaPages(**f)


@pytest.mark.parametrize("kw,expect", [
    (dict(), OK),
    (dict(rot=0, inv_freq=None), OK),
    (dict(rot=0), INVALID),                       # frequencies without channels
    (dict(inv_freq=None), INVALID),
    (dict(rot=80), INVALID),                      # more than d
    (dict(rot=-16), INVALID),
    (dict(rot=24), UNSUPPORTED),                  # not a multiple of 16
    (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(interleaved=2), INVALID),
    (dict(q_weight=FAKE + 4), INVALID),
    (dict(positions=FAKE + 8), INVALID),
    (dict(positions=None, first=2**31 - 256), OK),
    (dict(positions=None, first=2**31 - 255), INVALID),   # the last position would not be an int32
])
def test_prep_description(kw, expect):
    p = dma.make_params(1, 2, 1, 256, 64, 1)
    n = ctypes.c_size_t(0)
    assert dma.load().dma_prep_workspace_size(ctypes.byref(p), ctypes.byref(_prep(**kw)), ctypes.byref(n)) == expect
    assert n.value > 0 or expect != OK


@pytest.mark.parametrize("kw,expect", [
    (dict(N=1 << 24), OK),                        # the attention's row limit does not apply
    (dict(N=(1 << 24) + 1), UNSUPPORTED),
    (dict(N=1 << 24, B=128), UNSUPPORTED),        # B N = 2^31
    (dict(Nq=5), INVALID),
    (dict(d=96), UNSUPPORTED),
    (dict(H=3, Hkv=2), INVALID),
    (dict(B=0), INVALID),
    (dict(B=40000, N=1), UNSUPPORTED),            # B H > 65535
])
def test_prep_problem(kw, expect):
    f = dict(B=1, H=2, Hkv=1, N=256, d=64, w=1)
    f.update(kw)
    n = ctypes.c_size_t(0)
    r = _prep()
    assert dma.load().dma_prep_workspace_size(ctypes.byref(dma.make_params(**f)), ctypes.byref(r),
                                              ctypes.byref(n)) == expect


def _paged(pkw=None, **kw):
    f = dict(B=3, H=4, Hkv=2, N=320, d=64, w=50, Nq=1)
    f.update(pkw or {})
    lay = _lib.DmaPagedLayout()
    p = dma.make_params(**f)
    return dma.load().dma_paged_layout(ctypes.byref(p), ctypes.byref(_pages(**kw)), ctypes.byref(lay)), lay


@pytest.mark.parametrize("pkw,kw,expect", [
    (dict(), dict(), OK),
    (dict(N=321), dict(), INVALID),               # longer than a table row
    (dict(N=1), dict(max_pages=1), OK),
    (dict(Nq=2), dict(), INVALID),
    (dict(w=0), dict(), INVALID),
    (dict(d=80), dict(), UNSUPPORTED),
    (dict(), dict(page=8), UNSUPPORTED),
    (dict(), dict(page=24), UNSUPPORTED),
    (dict(), dict(page=2048), UNSUPPORTED),
    (dict(), dict(page=0), INVALID),
    (dict(), dict(n_pages=0), INVALID),
    (dict(), dict(n_pages=1 << 27), UNSUPPORTED),                  # 2^31 positions
    (dict(H=64, Hkv=8, B=1), dict(n_pages=1 << 25), UNSUPPORTED),  # 2^31 rows of gate values
    (dict(), dict(prefix=48), OK),
    (dict(), dict(prefix=40), INVALID),           # not whole pages
    (dict(), dict(prefix=336), INVALID),
    (dict(), dict(prefix=-16), INVALID),
    (dict(), dict(K=None), INVALID),
    (dict(), dict(lens=FAKE + 4), INVALID),
    (dict(), dict(table=None), INVALID),
    (dict(w=300000, N=300000), dict(max_pages=20000), UNSUPPORTED),   # min(w, N) > 4096 d, as for decode
])
def test_paged_problem(pkw, kw, expect):
    assert _paged(pkw, **kw)[0] == expect


def test_paged_layout():
    st, lay = _paged()
    assert st == OK and lay.sel_len == 50 and lay.cand_len == 0
    st, lay = _paged(dict(N=30))
    assert lay.sel_len == 30
    st, lay = _paged(prefix=304)                  # shared: candidates of the prefix, the rest row by row
    assert lay.sel_len == 16 and lay.cand_len == 50
    for off in (lay.off_status, lay.off_rows, lay.off_sel, lay.off_cand):
        assert off % 256 == 0
    assert lay.off_sel >= lay.off_rows + 3 * 4 * 16 and lay.bytes > lay.off_cand + 4 * 50 * 4
    assert _paged(dict(B=1), prefix=304)[1].cand_len == 0          # one sequence shares with nobody
    assert _paged(dict(dtype="f32"), prefix=304)[1].cand_len == 0  # float32 is computed row by row
    assert _paged(dict(N=304), prefix=304)[1].sel_len == 1


_FAKE_CHECKS = r"""
import ctypes, sys
sys.path.insert(0, %(root)r)
import trainable_dynamic_mask_b200 as dma
from trainable_dynamic_mask_b200 import _lib
OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4
F = 1 << 20
lib = dma.load()

def prep(**kw):
    f = dict(inv_freq=F, positions=None, q_weight=F, k_weight=F, eps=1e-6, rot=64, interleaved=0, first=0)
    f.update(kw)
    return _lib.DmaPrep(**f)

def strides(q=(64 * 4 * 100, 64 * 4, 64), k=None, v=None):
    a = _lib.DmaPrepStrides()
    for name, s in (("q", q), ("k", k or q), ("v", v or q)):
        for i in range(3):
            getattr(a, name)[i] = s[i]
    return a

p = dma.make_params(2, 4, 4, 100, 64, 1)
# dma_prep(p, r, st, q, k, v, Q, K, V, stream)
assert lib.dma_prep(p, prep(), strides(), F, F, F, F, F, F, None) == CUDA      # passes every check, no device here
assert lib.dma_prep(p, prep(), strides(), F, F, None, F, F, None, None) == CUDA
for i in range(6):
    a = [F] * 6
    a[i] = F + 4
    assert lib.dma_prep(p, prep(), strides(), *a, None) == INVALID, i
    a[i] = None
    assert lib.dma_prep(p, prep(), strides(), *a, None) == INVALID, i          # v and V only together
assert lib.dma_prep(p, prep(), None, *([F] * 6), None) == INVALID
assert lib.dma_prep(p, prep(), strides(q=(25600, 260, 64)), *([F] * 6), None) == INVALID   # 520 bytes
assert lib.dma_prep(p, prep(), strides(q=(25600, -256, 64)), *([F] * 6), None) == INVALID
assert lib.dma_prep(p, prep(), strides(k=(0, 0, 0)), *([F] * 6), None) == CUDA             # one row for all: read only
assert lib.dma_prep(p, prep(rot=24), strides(), *([F] * 6), None) == UNSUPPORTED

# dma_prep_bwd(p, r, st, gst, q, k, dQ, dK, dV, dV_gate, dq, dk, dv, dqw, dkw, ws, bytes, stream)
n = ctypes.c_size_t(0)
assert lib.dma_prep_workspace_size(p, prep(), n) == OK
def bwd(r=None, st=None, gst=None, ws=F, nb=None, **kw):
    a = dict(q=F, k=F, dQ=F, dK=F, dV=F, dVg=F, dq=F, dk=F, dv=F, dqw=F, dkw=F)
    a.update(kw)
    return lib.dma_prep_bwd(p, r or prep(), st or strides(), gst or strides(), a["q"], a["k"], a["dQ"], a["dK"], a["dV"],
                            a["dVg"], a["dq"], a["dk"], a["dv"], a["dqw"], a["dkw"], ws, n.value if nb is None else nb, None)
assert bwd() == CUDA
assert bwd(dV=None, dVg=None, dv=None) == CUDA
assert bwd(dVg=None, dqw=None, dkw=None) == CUDA
assert bwd(r=prep(q_weight=None, k_weight=None), q=None, k=None, dqw=None, dkw=None) == CUDA
assert bwd(q=None) == INVALID and bwd(k=None) == INVALID                        # read where there is a weight
assert bwd(r=prep(q_weight=None), q=None) == INVALID                            # a gradient for no weight
assert bwd(dV=None) == INVALID and bwd(dv=None) == INVALID and bwd(dV=None, dv=None) == INVALID
for name in ("q", "k", "dQ", "dK", "dV", "dVg", "dq", "dk", "dv", "dqw", "dkw"):
    assert bwd(**{name: F + 8}) == INVALID, name
for name in ("dQ", "dK", "dq", "dk"):
    assert bwd(**{name: None}) == INVALID, name
assert bwd(nb=n.value - 1) == WORKSPACE and bwd(ws=None) == WORKSPACE and bwd(ws=F + 4) == WORKSPACE
assert bwd(gst=strides(q=(0, 256, 64))) == INVALID             # batch rows on top of one another
assert bwd(gst=strides(q=(25600, 256, 32))) == INVALID         # heads that overlap
assert bwd(gst=strides(k=(25600, 64, 64))) == INVALID          # positions on top of heads
assert bwd(gst=strides(q=(4 * 100 * 64, 64, 100 * 64))) == CUDA   # head-major
assert bwd(gst=strides(q=(64, 2 * 4 * 64, 2 * 64))) == CUDA       # batch innermost
assert bwd(st=strides(q=(0, 256, 64))) == CUDA                    # inputs may be shared

# paged
def pages(**kw):
    f = dict(K=F, V=F, delta=F, table=F, lens=F, n_pages=100, page=16, max_pages=20, prefix=0)
    f.update(kw)
    return _lib.DmaPages(**f)
pd = dma.make_params(3, 4, 2, 320, 64, 50, Nq=1)
lay = _lib.DmaPagedLayout()
assert lib.dma_paged_layout(pd, pages(), lay) == OK
assert lib.dma_paged_layout(pd, pages(), None) == INVALID
nb = lay.bytes
assert lib.dma_paged_topk(pd, pages(), F, nb, None) == CUDA
assert lib.dma_paged_topk(pd, pages(), F, nb - 1, None) == WORKSPACE
assert lib.dma_paged_topk(pd, pages(), F + 4, nb, None) == WORKSPACE
assert lib.dma_paged_topk(pd, None, F, nb, None) == INVALID
assert lib.dma_paged_attn(pd, pages(), F, F, nb, F, F, None) == CUDA
for i in range(3):
    a = [F, F, F]
    a[i] = None if i else F + 2
    assert lib.dma_paged_attn(pd, pages(), a[0], F, nb, a[1], a[2], None) == INVALID
assert lib.dma_paged_attn(pd, pages(), F, None, nb, F, F, None) == WORKSPACE
# dma_paged_append(p, c, r, st, T, starts, q, k, v, Delta, A, Q, ws, bytes, stream)
def app(pp=pd, c=None, r=None, st=None, T=7, starts=F, ws=F, size=nb, **kw):
    a = dict(q=F, k=F, v=F, Delta=F, A=F, Q=F)
    a.update(kw)
    return lib.dma_paged_append(pp, c or pages(), r or prep(), st or strides(), T, starts, a["q"], a["k"], a["v"],
                                a["Delta"], a["A"], a["Q"], ws, size, None)
assert app() == CUDA and app(T=3, starts=None) == CUDA and app(q=None, Q=None) == CUDA
assert app(T=0) == OK and app(T=0, k=None, v=None) == OK
assert app(T=4, starts=None) == INVALID and app(T=-1) == INVALID
assert app(starts=F + 4) == INVALID
assert app(r=prep(positions=F)) == INVALID                     # positions are the cache's
assert app(r=prep(rot=128)) == INVALID
assert app(q=None) == INVALID and app(Q=None) == INVALID
for name in ("q", "k", "v", "Delta", "A", "Q"):
    assert app(**{name: F + 8}) == INVALID, name
for name in ("k", "v", "Delta", "A"):
    assert app(**{name: None}) == INVALID, name
assert app(st=strides(v=(0, 130, 64))) == INVALID
assert app(size=nb - 1) == WORKSPACE and app(ws=None) == WORKSPACE
ph = dma.make_params(1, 72, 8, 320, 64, 50, Nq=1)
assert lib.dma_paged_layout(ph, pages(), lay) == OK
assert app(pp=ph, size=lay.bytes) == UNSUPPORTED               # the gate holds at most 64 heads
print("ok")
"""


def test_calls_are_refused_before_any_launch():
    # in a child process that sees no GPU: a call that passes every check ends with DMA_ERR_CUDA there
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", _FAKE_CHECKS % {"root": ROOT}], env=env, capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


_MISSING = r"""
import sys
sys.path.insert(0, %(root)r)
import trainable_dynamic_mask_b200 as dma
from trainable_dynamic_mask_b200 import _lib
_lib.LIB_PATH = %(missing)r
_lib._lib = None
p = dma.make_params(1, 2, 1, 256, 64, 64)
r = dma.make_prep(None)
c = _lib.DmaPages()
for name, fn in {
    "prep": lambda: dma.prep(p, r, *([None] * 6)),
    "prep_bwd": lambda: dma.prep_bwd(p, r, *([None] * 12)),
    "prep_workspace_size": lambda: dma.prep_workspace_size(p, r),
    "paged_layout": lambda: dma.paged_layout(p, c),
    "paged_append": lambda: dma.paged_append(p, c, r, *([None] * 7)),
    "paged_topk": lambda: dma.paged_topk(p, c, None),
    "paged_attn": lambda: dma.paged_attn(p, c, *([None] * 4)),
}.items():
    try:
        fn()
    except RuntimeError as e:
        assert "no fallback" in str(e) and "build" in str(e), (name, str(e))
    else:
        raise AssertionError(name + " ran without libdma.so")
print("ok")
"""


def test_entry_points_raise_without_the_library():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    missing = os.path.join(ROOT, "no_such_dir", "libdma.so")
    r = subprocess.run([sys.executable, "-c", _MISSING % {"root": ROOT, "missing": missing}], env=env,
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
