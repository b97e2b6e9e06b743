"""The binding holds pages to the problem they were made for.  On the CPU, with CPU tensors and a library that
only records which calls reach it: the sizes of tensors are not known behind the C interface."""
import pytest
import torch

import trainable_dynamic_mask_b200 as dma
from trainable_dynamic_mask_b200 import _lib


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


class _Here:
    """What the binding asks of torch, on the CPU (get_device() of a CPU tensor is -1)."""
    types = {dma.DMA_BF16: torch.bfloat16, dma.DMA_F32: torch.float32}
    f32, i32 = torch.float32, torch.int32
    device = staticmethod(lambda: -1)
    stream = staticmethod(lambda dev: 0)


B, H, Hkv, N, d, W = 3, 4, 2, 64, 64, 8


@pytest.fixture
def lib(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(_lib, "_lib", r)
    monkeypatch.setattr(dma, "_torch", lambda: _Here)
    return r


def _params(**kw):
    f = dict(B=B, H=H, Hkv=Hkv, N=N, d=d, w=W, Nq=1)
    f.update(kw)
    return dma.make_params(**f)


def _pages(p):
    rows = torch.zeros(9, Hkv, 16, d, dtype=torch.bfloat16)
    return dma.make_pages(p, rows, rows.clone(), torch.zeros(9, H, 16), torch.zeros(B, 4, dtype=torch.int32),
                          torch.zeros(B, dtype=torch.int32))


def _calls(p, c):
    """Every paged call, with tensors that fit p."""
    t = torch.bfloat16 if p.dtype == dma.DMA_BF16 else torch.float32
    q, kv = torch.zeros(p.B, p.H, p.d, dtype=t), torch.zeros(p.B, p.Hkv, p.d, dtype=t)
    ws, r = torch.zeros(64, dtype=torch.uint8), dma.make_prep(None)
    Delta, A = torch.zeros(p.Hkv * p.d, p.H, dtype=t), torch.zeros(p.H)
    return {
        "dma_paged_layout": lambda: dma.paged_layout(p, c),
        "dma_paged_append": lambda: dma.paged_append(p, c, r, q, kv, kv, Delta, A, torch.empty_like(q), ws),
        "dma_paged_topk": lambda: dma.paged_topk(p, c, ws),
        "dma_paged_attn": lambda: dma.paged_attn(p, c, q, ws, torch.empty_like(q), torch.zeros(p.B, p.H)),
    }


NAMES = ["dma_paged_layout", "dma_paged_append", "dma_paged_topk", "dma_paged_attn"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("kw", [dict(), dict(N=48), dict(w=20), dict(scale=0.5), dict(B=2), dict(B=1)])
def test_pages_serve_problems_that_they_hold(lib, name, kw):
    # other limits, and the leading sequences alone
    c = _pages(_params())
    _calls(_params(**kw), c)[name]()
    assert lib.calls == [name]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("kw", [dict(B=4), dict(H=8), dict(H=2), dict(H=4, Hkv=4), dict(Hkv=1), dict(d=128),
                                dict(dtype="f32")])
def test_pages_of_another_problem_are_refused(lib, name, kw):
    c = _pages(_params())
    with pytest.raises(ValueError, match="pages"):
        _calls(_params(**kw), c)[name]()
    assert lib.calls == []


def test_pages_of_another_device_are_refused(lib, monkeypatch):
    c = _pages(_params())
    monkeypatch.setattr(_Here, "device", staticmethod(lambda: 1))
    with pytest.raises(ValueError, match="cuda:1"):
        dma.paged_topk(_params(), c, torch.zeros(64, dtype=torch.uint8))
    assert lib.calls == []


@pytest.mark.parametrize("name", NAMES)
def test_parameters_are_looked_at_again_when_they_change(lib, name):
    p = _params()
    c = _pages(p)
    _calls(p, c)[name]()
    p.B = 4
    with pytest.raises(ValueError, match="pages"):
        _calls(p, c)[name]()
    assert lib.calls == [name]
    p.B = 2
    _calls(p, c)[name]()
    assert lib.calls == [name, name]
