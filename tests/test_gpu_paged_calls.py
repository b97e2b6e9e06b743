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
