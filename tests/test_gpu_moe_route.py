"""Tokens sorted by expert, back with weights applied, and the gradients, on the GPU against the
FP64 oracle.

The maps and the gathered rows are exact. A 16-bit output y of FP32 sums over terms x_j is within
half a step of its type, eps / 2 |y|, plus the FP32 sums' error: k terms, each product and sum
rounded to 24 bits, at most (k + 1) 2^-24 sum |x_j|, and the type's smallest step for fp16
subnormals. FP32 sums over H products: at most (H / 32 + 10) 2^-24 sum |x| (H / 32 per lane at most
in four chains, then 5 + 2 additions; the products of two 16-bit values are rounded once at most).
"""
import numpy as np
import pytest
import torch

from oracle import routed
from weight_only_int4_07_b200 import native

pytestmark = pytest.mark.gpu
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    native.lib()
    torch.cuda.set_device(0)


def _ids(T, k, E, seed, kind):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if kind == "one":
        ids[:] = E - 1
    elif kind == "drop":
        ids[torch.rand(T, k, generator=g) < 0.3] = -1
        ids[torch.rand(T, k, generator=g) < 0.1] = E + 5
    elif kind == "none":
        ids[:] = -1
    elif kind == "sorted":
        ids = ids.view(-1).sort(descending=True).values.view(T, k)
    return ids.contiguous()


def _rows(n, H, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, H, generator=g).to(dtype)


def _f64(t):
    return t.detach().cpu().double().numpy()


SHAPES = [(1, 1, 1, 8, "any"), (1, 8, 64, 4096, "any"), (3, 2, 8, 72, "any"), (5, 3, 4, 8, "none"),
          (16, 4, 64, 2048, "drop"), (77, 4, 9, 1032, "drop"), (300, 32, 1024, 16, "any"), (513, 2, 2, 264, "one"),
          (1021, 8, 128, 64, "any"), (1025, 8, 16, 64, "drop"), (3001, 7, 1000, 24, "sorted"), (9000, 1, 3, 40, "one")]


@pytest.mark.parametrize("T,k,E,H,kind", SHAPES)
def test_sort_maps_and_rows(T, k, E, H, kind):
    ids = _ids(T, k, E, T + k, kind)
    X = _rows(T, H, torch.bfloat16, 5)
    want_off, want_rows, want_slots = routed.sort(ids.numpy(), E)
    R = int(want_off[E])
    d = ids.cuda()
    keep = dict(rows=torch.full((T * k,), -77, dtype=torch.int32, device="cuda"),
                Xs=torch.full((T * k, H), 3.5, dtype=torch.bfloat16, device="cuda"))
    offsets, rows, slots, Xs = native.w4a16_moe_sort(d, E, X=X.cuda(), **keep)
    assert np.array_equal(offsets.cpu().numpy(), want_off)
    assert np.array_equal(slots.cpu().numpy(), want_slots)
    assert np.array_equal(rows.cpu().numpy()[:R], want_rows)
    assert bool((rows[R:] == -77).all()) and bool((Xs[R:] == 3.5).all())   # left as they were
    assert torch.equal(Xs[:R].cpu(), X[torch.from_numpy(want_rows // k)])
    maps = native.w4a16_moe_sort(d, E)
    assert maps[3] is None and torch.equal(maps[0], offsets) and torch.equal(maps[2], slots)
    assert torch.equal(maps[1][:R], rows[:R])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,E,H,kind", SHAPES[:9])
def test_combine_and_gradients(T, k, E, H, kind, weighted, dtype):
    ids = _ids(T, k, E, T + k, kind)
    off, rows_np, slots_np = routed.sort(ids.numpy(), E)
    R = int(off[E])
    n = T * k
    slots = torch.from_numpy(slots_np.astype(np.int32)).cuda()
    g = torch.Generator().manual_seed(9)
    w = torch.rand(T, k, generator=g) if weighted else None
    Ys, dY, dXs = (_rows(m, H, dtype, s) for m, s in ((n, 1), (T, 2), (n, 3)))
    # a choice without a row adds nothing, whatever stands in its place
    if weighted:
        w[torch.from_numpy(slots_np < 0)] = float("nan")
    Ys[R:] = float("nan")
    dXs[R:] = float("inf")
    half = torch.finfo(dtype).eps / 2
    wn = None if w is None else w.numpy()
    wd = None if w is None else w.cuda()

    Y = native.w4a16_moe_combine(Ys.cuda(), slots, wd)
    ref, mag = routed.combine(_f64(Ys), slots_np, wn)
    assert (np.abs(_f64(Y) - ref) <= half * np.abs(ref) + (k + 1) * 2.0 ** -24 * (1 + half) * mag + TINY[dtype]).all()

    dX = native.w4a16_moe_sort_grad(dXs.cuda(), slots)
    ref, mag = routed.combine(_f64(dXs), slots_np, None)
    assert (np.abs(_f64(dX) - ref) <= half * np.abs(ref) + (k + 1) * 2.0 ** -24 * (1 + half) * mag + TINY[dtype]).all()

    dYs = torch.full((n, H), 7.0, dtype=dtype, device="cuda")
    got, dw = native.w4a16_moe_combine_grad(dY.cuda(), Ys.cuda(), slots, wd, dYs=dYs)
    assert got is dYs
    want, dwref, dwmag = routed.combine_grad(_f64(dY), _f64(Ys), slots_np, wn)
    out = _f64(dYs)
    for s in range(R):
        # the FP32 product of a 16-bit value and the weight, then the type
        assert (np.abs(out[s] - want[s]) <= (half * (1 + 2.0 ** -24) + 2.0 ** -24) * np.abs(want[s]) + TINY[dtype]).all()
    assert (out[R:] == 7.0).all()
    assert (np.abs(_f64(dw) - dwref) <= (H / 32 + 10) * 2.0 ** -24 * dwmag).all()
    assert (_f64(dw)[slots_np < 0] == 0).all()
    alone, none = native.w4a16_moe_combine_grad(dY.cuda(), None, slots, wd, dYs=torch.full_like(dYs, 7.0))
    assert none is None and torch.equal(alone, dYs)


def test_results_repeat_and_hold_in_a_captured_graph():
    """Sort, combine and gradients captured once, replayed on other inputs and on another stream."""
    T, k, E, H = 1300, 8, 32, 128
    dev = dict(device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int32, **dev)
    X = torch.zeros(T, H, dtype=torch.float16, **dev)
    w = torch.zeros(T, k, **dev)
    bufs = dict(offsets=torch.zeros(E + 1, dtype=torch.int32, **dev), rows=torch.zeros(T * k, dtype=torch.int32, **dev),
                slots=torch.zeros(T, k, dtype=torch.int32, **dev), Xs=torch.zeros(T * k, H, dtype=torch.float16, **dev),
                workspace=torch.empty(native.w4a16_moe_sort_workspace_bytes(T, k, E), dtype=torch.uint8, **dev))
    Y, dX = torch.zeros_like(X), torch.zeros_like(X)
    dYs, dw = torch.zeros_like(bufs["Xs"]), torch.zeros_like(w)

    def step():
        _, _, slots, Xs = native.w4a16_moe_sort(ids, E, X=X, **bufs)
        native.w4a16_moe_combine(Xs, slots, w, Y=Y)
        native.w4a16_moe_combine_grad(X, Xs, slots, w, dYs=dYs, dweights=dw)
        native.w4a16_moe_sort_grad(dYs, slots, dX=dX)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        ids.copy_(_ids(T, k, E, seed, "any"))
        X.copy_(_rows(T, H, torch.float16, seed))
        w.copy_(torch.rand(T, k, generator=torch.Generator().manual_seed(seed)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (bufs["offsets"], bufs["rows"], bufs["slots"], bufs["Xs"], Y, dYs, dw, dX)]
        with torch.cuda.stream(side):
            for t in (Y, dX, dYs, dw):
                t.zero_()
            step()
        torch.cuda.synchronize()
        for a, b in zip(got, (bufs["offsets"], bufs["rows"], bufs["slots"], bufs["Xs"], Y, dYs, dw, dX)):
            assert torch.equal(a, b)
        # Y = (sum of weights) X, row by row
        ref = w.double().sum(1, keepdim=True) * X.double()
        assert (Y.double() - ref).abs().max() <= 2.0 ** -10 * ref.abs().max()


@pytest.mark.parametrize("T,k,E,kind", [(40000, 8, 1024, "any"), (33000, 9, 1023, "drop"), (300000, 1, 1024, "one")])
def test_maps_of_many_ids(T, k, E, kind):
    """A hundred and more histograms of 1024 bins, added up by every CTA."""
    ids = _ids(T, k, E, T, kind)
    want_off, want_rows, want_slots = routed.sort(ids.numpy(), E)
    offsets, rows, slots, _ = native.w4a16_moe_sort(ids.cuda(), E)
    assert np.array_equal(offsets.cpu().numpy(), want_off) and np.array_equal(slots.cpu().numpy(), want_slots)
    assert np.array_equal(rows.cpu().numpy()[:len(want_rows)], want_rows)
