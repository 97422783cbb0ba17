"""The grouped products at the borders of what they take (needs an MI355X): ends of any
value and order, more experts than a wave has lanes, strides past 31 bits, reductions of
length zero, gradients larger than the caches. Bounds as in test_gpu_grouped.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import swiglu_activation_amd as sw
from tests.test_gpu_grouped import OPS, _ends, _inputs, _run, _say, _verify

pytestmark = pytest.mark.gpu


def _given(ends):
    return torch.tensor(ends, dtype=torch.int32, device="cuda")


# direct, general, split (whole vectors and others), tiles; the last two with more than 64 experts
ANY_ENDS = [(9, 3, 72, 200), (50, 3, 35, 77), (300, 3, 512, 4096), (300, 3, 511, 4095), (2000, 3, 512, 1024),
            (200, 70, 72, 136), (9000, 100, 512, 768)]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("shape", ANY_ENDS, ids=lambda c: "-".join(map(str, c)))
def test_ends_of_any_value_and_order(op, shape):
    """A group begins at the largest end before it. Ends that decrease, are negative or past
    the rows give the bits of the ends in order that they amount to, within a workspace of
    exactly the size asked for."""
    rows, experts, n, k = shape
    gen = torch.Generator().manual_seed(rows + n)
    t, f, scale = _inputs(op, rows, experts, n, k, 0, gen)
    rng = np.random.default_rng(rows)
    top = 2 ** 31 - 1
    turns = [rows if e % 2 == 0 else 0 for e in range(experts)]
    cases = [turns, turns[::-1], sorted(rng.integers(0, rows + 1, experts).tolist(), reverse=True),
             rng.integers(-rows, 2 * rows + 1, experts).tolist(), [top, -top - 1] * (experts // 2) + [5] * (experts % 2),
             [-1] * experts]
    need = sw.swiglu_grouped_workspace_size({"dgrad": "mm_dgrad", "wgrad": "mm_wgrad"}.get(op, op), rows, experts, n, k)
    guard = 1 << 20
    ws = torch.full((need + guard,), 0x5a, dtype=torch.uint8, device="cuda")
    for i, ends in enumerate(cases):
        _say(f"[grouped bounds] {op} {shape} ends {i}, workspace {need}")
        fixed = np.maximum.accumulate(np.clip(np.array(ends, dtype=np.int64), 0, rows)).tolist()
        sizes = np.diff([0] + fixed).tolist()
        want = _run(op, t, f, _given(fixed), scale)
        got = _run(op, t, f, _given(ends), scale, workspace=ws[:need] if need else None)
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
        assert bool((ws[need:] == 0x5a).all()), i
        if i in (0, 3):
            _verify(op, got, t, f, sizes, scale, f"{op} ends {i}")
        whole = _run(op, t, f, _given(ends), scale, workspace=False)
        _verify(op, whole, t, f, sizes, scale, f"{op} ends {i} without workspace")


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("shape", [(6600, 66, 512, 768), (9000, 130, 768, 640)], ids=lambda c: "-".join(map(str, c)))
def test_more_experts_than_lanes(op, shape):
    """Groups of about 100 rows in tiles of 128 and 256, the experts around the 64th (and the 128th) empty."""
    rows, experts, n, k = shape
    _say(f"[grouped bounds] {op} {shape}")
    gen = torch.Generator().manual_seed(experts)
    rng = np.random.default_rng(experts)
    p = rng.dirichlet(np.ones(experts) * 2)
    for e in (62, 63, 64, 65, 127, 128):
        if e < experts - 1:
            p[e] = 0
    sizes = rng.multinomial(rows, p / p.sum()).tolist()
    t, f, scale = _inputs(op, rows, experts, n, k, 5, gen)
    got = _run(op, t, f, _ends(sizes), scale)
    _verify(op, got, t, f, sizes, scale, op)


@pytest.mark.parametrize("op", ["mm", "fc1", "dgrad"])
@pytest.mark.parametrize("n,k", [(24, 40), (19, 37)])
def test_strides_past_31_bits(op, n, k):
    """Few rows whose strides, and their weights', put a row a multiple of 2^31 or 2^32
    bytes from the first: 2^30 elements between token rows, 2^27 between weight rows
    (the 8th feature of a tile is 2^31 bytes from the first)."""
    _say(f"[grouped bounds] {op} long strides, n {n} k {k}")
    gen = torch.Generator().manual_seed(n)
    sizes = [3]
    t, f, scale = _inputs(op, 3, 1, n, k, 0, gen)
    big = torch.zeros((2 << 30) + 64, dtype=torch.bfloat16, device="cuda")
    tv = big.as_strided((3, t.shape[1]), (1 << 30, 1))
    tv.copy_(t)
    _verify(op, _run(op, tv, f, _ends(sizes), scale), t, f, sizes, scale, op + " token rows far apart")
    del tv, big
    rows = f.shape[1]
    big = torch.zeros(((rows - 1) << 27) + 64, dtype=torch.bfloat16, device="cuda")
    fv = big.as_strided((1, rows, f.shape[2]), (big.numel(), 1 << 27, 1))
    fv.copy_(f)
    _verify(op, _run(op, t, fv, _ends(sizes), scale), t, f, sizes, scale, op + " weight rows far apart")


@pytest.mark.parametrize("rows,experts,n", [(5, 2, 16), (3000, 4, 4096), (70000, 4, 1024)])
def test_a_reduction_of_length_zero_gives_zeros(rows, experts, n):
    """Whatever the rows' scales are."""
    _say(f"[grouped bounds] fc1 of no columns, rows {rows} n {n}")
    a = torch.empty(rows, 0, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(experts, 2 * n, 0, dtype=torch.bfloat16, device="cuda")
    scale = torch.full((rows,), float("nan"), device="cuda")
    scale[::2] = float("inf")
    ends = _given([rows // experts * (e + 1) for e in range(experts)])
    assert not bool(sw.swiglu_grouped_fc1(a, w, ends, scale).any())
    assert not bool(sw.swiglu_grouped_mm(a, w, ends).any())


@pytest.mark.parametrize("dtype,k", [(torch.bfloat16, 4096), (torch.float32, 2048), (torch.float32, 4104),
                                     (torch.bfloat16, 4104)])
def test_weight_gradients_larger_than_the_caches(dtype, k):
    """Short groups and more than 256 MiB of gradients: rows of whole 128-byte lines are
    stored past the caches, others through them. Some experts have no rows."""
    experts, n = 44, 1000
    _say(f"[grouped bounds] wgrad {dtype} {experts} x {n} x {k}")
    gen = torch.Generator().manual_seed(k)
    sizes = np.random.default_rng(k).multinomial(1900, np.arange(experts) % 5 / (np.arange(experts) % 5).sum()).tolist()
    assert experts * n * k * dtype.itemsize > 256 << 20 and 0 in sizes
    t, f, _ = _inputs("wgrad", 1900, experts, n, k, 7, gen)
    got = _run("wgrad", t, f, _ends(sizes), None, dtype)
    _verify("wgrad", got, t, f, sizes, None, f"wgrad {dtype}")
    assert torch.equal(got, _run("wgrad", t, f, _ends(sizes), None, dtype)), "two calls differ"
