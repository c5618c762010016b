"""The experts' INT4 products on sorted rows, against the FP64 oracle's layer of every expert.

Bound of one output y, s = sum_k |a_k w_k|, h = eps / 2 of the 16-bit type: the dequantized weight
rounded once to the type (h s; no such rounding in the forms that scale FP32 sums), FP32 sums of K
products (K 2^-23 s), the output's own rounding (h |y|), the type's smallest step. Those errors
are independent, so the 2-norm of all errors is also within h times the outputs' 2-norm: two
roundings of relative size at most h, whose mean square is below h^2 / 3 each.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import routed
from weight_only_int4_07_b200 import native, synthetic

pytestmark = pytest.mark.gpu
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
KERNELS = [native.KERNEL_AUTO, native.KERNEL_GEMV, native.KERNEL_TC]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    native.lib()
    torch.cuda.set_device(0)


_cache = {}


def experts(E, K, N, group, sym):
    """(per expert: oracle codes, scales, zeros), the tiled buffers [E, bytes] on the GPU."""
    key = (E, K, N, group, sym)
    if key not in _cache:
        packed, tiled = [], []
        for e in range(E):
            st, c, s, z = oracle.quantize(synthetic.weights_normal(K, N, seed=70 + e), group, sym)
            assert st == oracle.OK
            packed.append((c, s, z))
            tiled.append(torch.from_numpy(oracle.repack(c, s, z, K, N, group, sym)))
        _cache[key] = packed, torch.stack(tiled).cuda()
    return _cache[key]


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)


def activations(R, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(R, K, generator=g).to(dtype)


def bits(t):
    return t.contiguous().view(torch.int16).numpy().view(np.uint16)


def check(C, A, off, packed, K, N, group, sym, skip=()):
    dt = 0 if A.dtype == torch.float16 else 1
    h = torch.finfo(A.dtype).eps / 2
    C = C.cpu().double().numpy()
    num = den = 0.0
    for e, (c, s, z) in enumerate(packed):
        rows = [i for i in range(int(off[e]), int(off[e + 1])) if i not in skip]
        if not rows:
            continue
        Y, mag = oracle.linear(bits(A[rows]), dt, c, s, z, N, group, sym)
        err = np.abs(C[rows] - Y)
        assert (err <= (h + K * 2.0 ** -23) * mag + h * np.abs(Y) + TINY[A.dtype]).all(), e
        num, den = num + float((err ** 2).sum()), den + float((Y ** 2).sum())
    assert num <= h * h * den


CASES = [  # counts per expert, K, N, group, sym, dtype: every tile height, empty experts, one row, ragged runs
    ([1], 128, 128, 128, 0, torch.float16),
    ([0, 1, 0, 1], 256, 256, 128, 0, torch.bfloat16),
    ([2, 0, 1, 3, 0, 0, 9, 1], 1024, 384, 128, 0, torch.float16),
    ([2, 0, 1, 3, 0, 0, 9, 1], 512, 128, 32, 1, torch.bfloat16),
    ([8, 0, 25, 1, 0, 0, 7, 3, 0, 2], 128, 512, 64, 0, torch.float16),
    ([0, 0, 16, 0, 0, 0, 0, 20], 384, 1280, 128, 1, torch.float16),
    ([1] * 40 + [0] * 23 + [17], 256, 128, 128, 0, torch.bfloat16),
    ([17, 1, 40, 0, 16, 2], 512, 256, 64, 0, torch.float16),
    ([33, 1, 100, 0, 16, 2], 384, 256, 32, 0, torch.bfloat16),
    ([0, 150, 64, 65], 640, 384, 128, 1, torch.bfloat16),
    ([129, 300, 0, 77], 256, 640, 64, 1, torch.float16),
    ([600, 0, 257], 1024, 256, 128, 0, torch.bfloat16),
    ([0, 0, 0], 256, 128, 128, 0, torch.float16),
]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("counts,K,N,group,sym,dtype", CASES)
def test_every_run_meets_its_own_weight(counts, K, N, group, sym, dtype, kernel):
    E, off = len(counts), offsets_of(counts)
    n = int(off[E])
    R = n + 3                                          # rows behind the last run: not used
    if kernel == native.KERNEL_GEMV and R > 8 * max(1, E):
        pytest.skip("more rows per expert than the decode kernel accepts")
    packed, tiled = experts(E, K, N, group, sym)
    A = activations(R, K, dtype, 3)
    A[n:] = float("nan")
    C = torch.full((R, N), 5.0, dtype=dtype, device="cuda")
    ws = torch.zeros(native.w4a16_moe_workspace_bytes(R, E, N, K, group), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (A.cuda(), off.cuda(), tiled, N, group, sym)
    native.w4a16_moe_gemm(*args, C=C, workspace=ws, kernel=kernel, dev_status=status)
    first = C.clone()
    native.w4a16_moe_gemm(*args, C=C, workspace=ws, kernel=kernel, dev_status=status)
    assert int(status) == 0 and not bool(ws[:65536].any())     # the counters are zero again
    assert torch.equal(first, C)                               # and the sums' order is fixed
    assert bool((C[n:] == 5.0).all())                          # left as they were
    check(C, A, off, packed, K, N, group, sym)


# the tensor cores' tiles whole (one or several to a CTA), each in ranges of its own, or cut evenly
CUTS = [([30, 40, 0, 35], 768, 1280, 32, 1, torch.bfloat16), ([30] * 20, 256, 2304, 128, 0, torch.float16),
        ([60, 70], 4096, 384, 128, 0, torch.bfloat16), ([300, 1], 2048, 256, 64, 1, torch.float16),
        ([10, 14], 4096, 384, 64, 0, torch.float16), ([2, 3, 0, 4], 2560, 256, 128, 0, torch.bfloat16),
        ([45] * 10, 5120, 1024, 128, 0, torch.bfloat16), ([12] * 10, 5120, 1024, 128, 0, torch.float16)]


@pytest.mark.parametrize("counts,K,N,group,sym,dtype", CUTS)
def test_tiles_whole_in_ranges_of_their_own_or_cut_evenly(counts, K, N, group, sym, dtype):
    test_every_run_meets_its_own_weight(counts, K, N, group, sym, dtype, native.KERNEL_TC)


# the down projections' input lengths; an expert with most of the rows beside many with few or none
LONG = [([1, 0, 3], 14336, 128, 128, 0, torch.bfloat16), ([2, 1], 28672, 128, 128, 1, torch.float16),
        ([0, 9, 4, 1], 14336, 128, 32, 1, torch.float16), ([12, 30], 28672, 128, 64, 0, torch.bfloat16)]
UNEVEN = [([1] * 60 + [300] + [2] * 40 + [0] * 20 + [15] * 5 + [1, 0], 256, 128, 128, 0, torch.bfloat16),
          ([0] * 127 + [384], 256, 128, 32, 0, torch.float16),
          ([1] * 31 + [90], 384, 256, 64, 1, torch.bfloat16)]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("counts,K,N,group,sym,dtype", LONG + UNEVEN)
def test_long_inputs_and_uneven_routing(counts, K, N, group, sym, dtype, kernel):
    test_every_run_meets_its_own_weight(counts, K, N, group, sym, dtype, kernel)


@pytest.mark.parametrize("kernel,most,dtype", [(native.KERNEL_GEMV, 6, torch.float16), (native.KERNEL_GEMV, 6, torch.bfloat16),
                                               (native.KERNEL_AUTO, 2, torch.bfloat16), (native.KERNEL_TC, 6, torch.float16),
                                               (native.KERNEL_TC, 30, torch.float16), (native.KERNEL_TC, 80, torch.bfloat16),
                                               (native.KERNEL_TC, 180, torch.bfloat16), (native.KERNEL_TC, 300, torch.float16)])
def test_as_many_experts_as_a_call_takes(kernel, most, dtype):
    """1024 experts (the runs' table takes 12 KB of shared memory) at every tile height; 0 to `most` rows
    each, the first and the last expert with some. Experts' outputs are checked on a sample of them."""
    E, K, N, group, sym = 1024, 128, 128, 32, 0
    packed, tiled = experts(E, K, N, group, sym)
    counts = torch.randint(0, most + 1, (E,), generator=torch.Generator().manual_seed(most))
    counts[[0, 517, E - 1]] = most
    counts[[1, 516, E - 2]] = 0
    off = offsets_of(counts.tolist())
    n = int(off[E])
    A = activations(n + 2, K, dtype, 9)
    C = torch.full((n + 2, N), 5.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.w4a16_moe_gemm(A.cuda(), off.cuda(), tiled, N, group, sym, C=C, kernel=kernel, dev_status=status)
    assert int(status) == 0 and bool((C[n:] == 5.0).all())
    dt, h = (0 if dtype == torch.float16 else 1), torch.finfo(dtype).eps / 2
    for e in [0, 2, 3, 515, 517, 518, E - 3, E - 1] + list(range(7, E, 61)):
        rows = slice(int(off[e]), int(off[e + 1]))
        if rows.start == rows.stop:
            continue
        Y, mag = oracle.linear(bits(A[rows]), dt, *packed[e], N, group, sym)
        err = np.abs(C[rows].cpu().double().numpy() - Y)
        assert (err <= (h + K * 2.0 ** -23) * mag + h * np.abs(Y) + TINY[dtype]).all(), e


@pytest.mark.parametrize("kernel", KERNELS)
def test_offsets_outside_the_rows_are_clamped(kernel):
    K, N, group, sym = 256, 256, 128, 0
    packed, tiled = experts(4, K, N, group, sym)
    A = activations(20, K, torch.float16, 4)
    off = torch.tensor([-7, 5, 3, 9, 1 << 30], dtype=torch.int32)   # runs [0, 5), none, [3, 9), [9, 20)
    C = native.w4a16_moe_gemm(A.cuda(), off.cuda(), tiled, N, group, sym, kernel=kernel).cpu()
    for e, lo, hi in ((0, 0, 3), (2, 5, 9), (3, 9, 20)):            # (rows 3 and 4 stand in two runs)
        c, s, z = packed[e]
        Y, mag = oracle.linear(bits(A[lo:hi]), 0, c, s, z, N, group, sym)
        assert (np.abs(C[lo:hi].double().numpy() - Y) <= 2.0 ** -10 * mag).all()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_row_that_is_not_finite_stays_by_itself(dtype, kernel):
    K, N, group, sym = 512, 256, 128, 0
    counts = [3, 2, 4]
    packed, tiled = experts(3, K, N, group, sym)
    off = offsets_of(counts)
    A = activations(9, K, dtype, 5)
    A[1, 7], A[4, 0], A[8, 100] = float("nan"), float("inf"), float("-inf")
    C = native.w4a16_moe_gemm(A.cuda(), off.cuda(), tiled, N, group, sym, kernel=kernel)
    check(C, A, off, packed, K, N, group, sym, skip=(1, 4, 8))
    assert not torch.isfinite(C[1]).any()


@pytest.mark.parametrize("kernel", KERNELS)
def test_wide_bf16_rows(kernel):
    """bf16 rows whose values span more binades than fp16 holds, and rows far outside its range: the
    bound grows with the row's largest product, as for any FP32 sum."""
    K, N, group, sym = 512, 256, 128, 0
    packed, tiled = experts(2, K, N, group, sym)
    off = offsets_of([4, 3])
    A = activations(7, K, torch.bfloat16, 6)
    A[0] *= 1e30
    A[1] *= 1e-30
    A[2, ::2] *= 1e20
    A[5, 17] = 1e30
    A[6, 128:256] *= 1e-12
    C = native.w4a16_moe_gemm(A.cuda(), off.cuda(), tiled, N, group, sym, kernel=kernel)
    check(C, A, off, packed, K, N, group, sym)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("e", [-110, -118, -122, -128])
def test_bf16_rows_at_the_low_end(kernel, e):
    """bf16 rows near and below the type's smallest normal value, 2^-126: as exact as any others (below
    it the output's own steps of 2^-133 count)."""
    K, N, group, sym = 1024, 256, 128, 0
    packed, tiled = experts(2, K, N, group, sym)
    off = offsets_of([4, 3])
    A = (activations(7, K, torch.float64, 8) * 2.0 ** e).bfloat16()
    A[1] = 0
    A[5, 128:] *= 2.0 ** 12
    C = native.w4a16_moe_gemm(A.cuda(), off.cuda(), tiled, N, group, sym, kernel=kernel)
    if e > -128:
        check(C, A, off, packed, K, N, group, sym)
    for x, (c, s, z) in enumerate(packed):
        rows = slice(int(off[x]), int(off[x + 1]))
        Y, mag = oracle.linear(bits(A[rows]), 1, c, s, z, N, group, sym)
        err = np.abs(C[rows].cpu().double().numpy() - Y)
        assert (err <= (2.0 ** -8 + K * 2.0 ** -23) * mag + 2.0 ** -8 * np.abs(Y) + TINY[torch.bfloat16]).all()


def test_routing_experts_and_back_in_a_captured_graph():
    """A mixture layer as it is used: sort, two expert products with a gate between, back; captured
    once and replayed on other tokens, against the oracle and the same calls made eagerly."""
    T, k, E, K, N, group, sym = 24, 2, 8, 256, 384, 128, 0
    up, tup = experts(E, K, N, group, sym)
    down, tdown = experts(E, N, K, group, sym)
    dev = dict(device="cuda")
    ids, w = torch.zeros(T, k, dtype=torch.int32, **dev), torch.zeros(T, k, **dev)
    X, Y = (torch.zeros(T, K, dtype=torch.bfloat16, **dev) for _ in range(2))
    Xs = torch.zeros(T * k, K, dtype=torch.bfloat16, **dev)
    Hs = torch.zeros(T * k, N, dtype=torch.bfloat16, **dev)
    Ys = torch.zeros(T * k, K, dtype=torch.bfloat16, **dev)
    maps = dict(offsets=torch.zeros(E + 1, dtype=torch.int32, **dev), rows=torch.zeros(T * k, dtype=torch.int32, **dev),
                slots=torch.zeros(T, k, dtype=torch.int32, **dev))
    need = max(native.w4a16_moe_workspace_bytes(T * k, E, N, K, group), native.w4a16_moe_workspace_bytes(T * k, E, K, N, group))

    def layer(ws):
        offsets, _, slots, _ = native.w4a16_moe_sort(ids, E, X=X, Xs=Xs, **maps)
        native.w4a16_moe_gemm(Xs, offsets, tup, N, group, sym, C=Hs, workspace=ws)
        Hs.clamp_(min=0)
        native.w4a16_moe_gemm(Hs, offsets, tdown, K, group, sym, C=Ys, workspace=ws)
        native.w4a16_moe_combine(Ys, slots, w, Y=Y)

    def workspace():
        return torch.zeros(need, dtype=torch.uint8, **dev)

    layer(workspace())
    torch.cuda.synchronize()
    graph, ws = torch.cuda.CUDAGraph(), workspace()
    with torch.cuda.graph(graph):
        layer(ws)
    side, ws_side = torch.cuda.Stream(), workspace()
    torch.cuda.synchronize()
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        ids.copy_(torch.randint(0, E, (T, k), generator=g, dtype=torch.int32))
        ids[5] = -1                                            # a padded token
        X.copy_(torch.randn(T, K, generator=g).bfloat16())
        w.copy_(torch.rand(T, k, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        hs, ys, y = Hs.clone(), Ys.clone(), Y.clone()
        for t in (Hs, Ys, Y):
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            layer(ws_side)
        torch.cuda.synchronize()
        off, rows, slots = routed.sort(ids.cpu().numpy(), E)
        n = int(off[E])
        assert torch.equal(hs[:n], Hs[:n]) and torch.equal(ys[:n], Ys[:n]) and torch.equal(y, Y)
        check(ys[:n], hs[:n].cpu(), off, down, N, K, group, sym)
        ref, mag = routed.combine(ys.cpu().double().numpy(), slots, w.cpu().numpy())
        assert (np.abs(y.cpu().double().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * mag).all()
        assert not bool(y[5].any())


def test_the_way_back_through_experts_in_16_bits():
    """A mixture layer's gradients as a program forms them: combine's, each expert's product with its
    dequantized weight (a library product: the layer's own way back is not this library's), sort's.
    Against the formulas in 64 bits; h = eps / 2: one rounding each of dYs, of dXs and of dX, and of
    Ys in dw, beside FP32 sums."""
    T, k, E, K, N, group, sym = 40, 3, 6, 256, 128, 128, 0
    packed, tiled = experts(E, K, N, group, sym)
    g = torch.Generator().manual_seed(4)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[3], ids[7, 1] = -1, -1
    X, dY = (torch.randn(T, n, generator=g).half() for n in (K, N))
    w = torch.rand(T, k, generator=g)
    offsets, _, slots, Xs = native.w4a16_moe_sort(ids.cuda(), E, X=X.cuda())
    Ys = native.w4a16_moe_gemm(Xs, offsets, tiled, N, group, sym)
    dYs, dw = native.w4a16_moe_combine_grad(dY.cuda(), Ys, slots, w.cuda())
    weights = [oracle.dequant(*packed[e], K, N, group, sym) for e in range(E)]
    dXs = torch.zeros_like(Xs)
    off = offsets.tolist()
    for e in range(E):
        W = torch.from_numpy(weights[e]).cuda()
        dXs[off[e]:off[e + 1]] = (dYs[off[e]:off[e + 1]].double() @ W.t()).half()
    dX = native.w4a16_moe_sort_grad(dXs, slots).cpu().double().numpy()
    h = 2.0 ** -11
    Xd, dYd, wd, ys = X.double().numpy(), dY.double().numpy(), w.double().numpy(), Ys.cpu().double().numpy()
    dw, sl = dw.cpu().double().numpy(), slots.cpu().numpy()
    for t in range(T):
        ref, mag = np.zeros(K), np.zeros(K)
        for j in range(k):
            e = int(ids[t, j])
            if e < 0:
                assert dw[t, j] == 0
                continue
            ref += wd[t, j] * (weights[e] @ dYd[t])
            mag += wd[t, j] * (np.abs(weights[e]) @ np.abs(dYd[t]))
            y, ymag = Xd[t] @ weights[e], np.abs(Xd[t]) @ np.abs(weights[e])
            # Ys as the layer leaves it, within its own bound; dw a sum of N products of it
            bound = ((h + K * 2.0 ** -23) * ymag + h * np.abs(y) + TINY[torch.float16]) @ np.abs(dYd[t])
            assert abs(dw[t, j] - y @ dYd[t]) <= bound + N * 2.0 ** -24 * (np.abs(ys[sl[t, j]]) @ np.abs(dYd[t]))
        assert (np.abs(dX[t] - ref) <= 2 * h * (1 + h) * mag + h * np.abs(ref) + (k + 1) * (2.0 ** -23 * mag + TINY[torch.float16])).all()
