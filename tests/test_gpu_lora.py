"""The layer with low-rank adapters against the FP64 oracle.

Bound of one output y = b + d (layer and adapter), h = eps / 2 of the 16-bit type, |.| of the terms
summed: layer as in the experts' test, (h + K 2^-23) sum |a w|; T_j in FP32, K 2^-23 of its terms,
through |s Lb|; T_j as two 16-bit values, 2^-16 of it (bf16; fp16 2^-22, and 2^-38 of the row's
largest) and FP32 sums of r products, r 2^-22, through |s Lb|; the output's rounding h |y|.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import routed
from weight_only_int4_07_b200 import native, synthetic

pytestmark = pytest.mark.gpu
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    native.lib()
    torch.cuda.set_device(0)


_cache = {}


def layer(K, N, group, sym):
    key = (K, N, group, sym)
    if key not in _cache:
        st, c, s, z = oracle.quantize(synthetic.weights_normal(K, N, seed=40), group, sym)
        assert st == oracle.OK
        _cache[key] = (c, s, z), torch.from_numpy(oracle.repack(c, s, z, K, N, group, sym)).cuda()
    return _cache[key]


def make(M, K, N, r, L, dtype, ids, seed=1):
    g = torch.Generator().manual_seed(seed)
    A = torch.randn(M, K, generator=g).to(dtype)
    La = (torch.randn(L, r, K, generator=g) / K ** 0.5).to(dtype)
    Lb = (torch.randn(L, N, r, generator=g) * 0.05).to(dtype)
    scale = torch.rand(L, generator=g) + 0.5
    if isinstance(ids, str):
        n = torch.randint(-1, L, (M,), generator=g)
        ids = {"any": n, "runs": n.sort().values, "none": torch.full((M,), -1), "one": torch.full((M,), L - 1),
               "wild": torch.where(n < 0, torch.tensor(1 << 30), n)}[ids]
    return A, La, Lb, scale, ids.to(torch.int32)


def bits(t):
    return t.contiguous().view(torch.int16).numpy().view(np.uint16)


def check(C, A, La, Lb, scale, ids, packed, N, group, sym, cols=None):
    dt = 0 if A.dtype == torch.float16 else 1
    h = torch.finfo(A.dtype).eps / 2
    K, r = A.shape[1], La.shape[1]
    c, s, z = packed
    base, mag = oracle.linear(bits(A), dt, c, s, z, N, group, sym, cols=cols)
    sel = slice(None) if cols is None else cols
    d, d1, d2, d3 = routed.lora(A.double().numpy(), La.double().numpy(), Lb.double().numpy()[:, sel], scale.numpy(),
                                ids.numpy())
    y = C.cpu().double().numpy()[:, sel]
    ref = base + d
    bound = ((h + K * 2.0 ** -23) * mag + K * 2.0 ** -23 * d2 + (2.0 ** -16 + r * 2.0 ** -22) * d1 + 2.0 ** -38 * d3
             + h * np.abs(ref) + TINY[A.dtype])
    assert (np.abs(y - ref) <= bound).all(), float((np.abs(y - ref) / bound).max())
    assert ((y - ref) ** 2).sum() <= h * h * (ref ** 2).sum()


CASES = [  # M, K, N, group, sym, dtype, rank, adapters, ids
    (1, 128, 128, 128, 0, torch.float16, 8, 1, "one"),
    (1, 4096, 256, 128, 0, torch.bfloat16, 16, 5, "one"),
    (1, 512, 256, 64, 1, torch.float16, 64, 2, "none"),
    (3, 1024, 384, 32, 0, torch.bfloat16, 24, 2, "any"),
    (8, 8192, 384, 128, 0, torch.float16, 32, 3, "any"),          # K slices in the decode kernel
    (8, 8192, 384, 128, 0, torch.bfloat16, 64, 9, "any"),
    (2, 2048, 1152, 32, 0, torch.float16, 64, 2, "any"),
    (7, 4096, 128, 64, 1, torch.bfloat16, 8, 7, "wild"),
    (5, 1024, 256, 128, 0, torch.float16, 16, 4, "any"),          # too many products for the decode kernel
    (16, 640, 256, 128, 1, torch.bfloat16, 40, 16, "wild"),
    (16, 4096, 128, 128, 0, torch.float16, 256, 2, "one"),        # the tensor-core layer, 16 rows
    (17, 256, 128, 128, 0, torch.bfloat16, 8, 4, "any"),
    (45, 1024, 640, 64, 0, torch.float16, 72, 7, "any"),
    (100, 384, 256, 32, 1, torch.bfloat16, 136, 1024, "any"),
    (257, 512, 384, 128, 0, torch.float16, 64, 3, "runs"),
    (300, 256, 256, 128, 0, torch.bfloat16, 16, 2, "none"),
    (13, 4096, 256, 128, 0, torch.bfloat16, 48, 13, "any"),       # 16-row tiles, scaled per unit
    (64, 128, 1280, 32, 0, torch.float16, 16, 64, "any"),         # a weight unit and many low-rank units
    (130, 256, 2560, 64, 0, torch.bfloat16, 32, 33, "any"),
    (520, 128, 384, 128, 1, torch.float16, 8, 5, "runs"),
]


@pytest.mark.parametrize("M,K,N,group,sym,dtype,r,L,ids", CASES)
def test_rows_with_their_adapters(M, K, N, group, sym, dtype, r, L, ids):
    packed, tiled = layer(K, N, group, sym)
    A, La, Lb, scale, rows = make(M, K, N, r, L, dtype, ids)
    ws = torch.zeros(native.w4a16_lora_workspace_bytes(M, N, K, group, r, L), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (A.cuda(), tiled, N, group, sym, La.cuda(), Lb.cuda(), scale.cuda(), rows.cuda())
    C = native.w4a16_lora_gemm(*args, workspace=ws, dev_status=status)
    check(C, A, La, Lb, scale, rows, packed, N, group, sym)
    again = native.w4a16_lora_gemm(*args, workspace=ws, dev_status=status)
    assert torch.equal(C, again) and int(status) == 0 and not bool(ws[:65536].any())


def test_pieces_of_a_long_batch():
    """More rank products than are held at a time: 256 rows of up to 256 adapters of rank 256, twice,
    then 88."""
    M, K, N, group, sym, r, L = 600, 128, 128, 128, 0, 256, 300
    packed, tiled = layer(K, N, group, sym)
    for dtype in (torch.float16, torch.bfloat16):
        A, La, Lb, scale, rows = make(M, K, N, r, L, dtype, "any")
        C = native.w4a16_lora_gemm(A.cuda(), tiled, N, group, sym, La.cuda(), Lb.cuda(), scale.cuda(), rows.cuda())
        check(C, A, La, Lb, scale, rows, packed, N, group, sym)


# one row block: its tiles whole (one or several to a CTA), each in ranges of its own, or cut evenly
CUTS = [(100, 512, 2304, 32, 1, torch.bfloat16, 16, 3, "any"), (40, 256, 20480, 128, 0, torch.float16, 8, 2, "any"),
        (200, 4096, 384, 128, 0, torch.bfloat16, 64, 8, "any"), (30, 4096, 256, 64, 1, torch.float16, 32, 9, "any"),
        (12, 4096, 640, 128, 0, torch.bfloat16, 24, 6, "any"), (70, 5120, 10240, 128, 0, torch.bfloat16, 16, 4, "any"),
        (20, 5120, 10240, 64, 0, torch.float16, 16, 4, "any")]


@pytest.mark.parametrize("M,K,N,group,sym,dtype,r,L,ids", CUTS)
def test_tiles_whole_in_ranges_of_their_own_or_cut_evenly(M, K, N, group, sym, dtype, r, L, ids):
    test_rows_with_their_adapters(M, K, N, group, sym, dtype, r, L, ids)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_stretches_of_rows_without_adapters(dtype):
    """Blocks of rows with many adapters, one or none, in one batch; the slices of K that the rank
    products are summed in go by how many there are, on the device."""
    M, K, N, group, sym, r, L = 230, 2048, 256, 128, 0, 40, 40
    packed, tiled = layer(K, N, group, sym)
    A, La, Lb, scale, rows = make(M, K, N, r, L, dtype, "any")
    ws = torch.zeros(native.w4a16_lora_workspace_bytes(M, N, K, group, r, L), dtype=torch.uint8, device="cuda")
    args = (A.cuda(), tiled, N, group, sym, La.cuda(), Lb.cuda(), scale.cuda())
    for gaps in ([(0, 32), (64, 128), (200, 230)], [(0, 225)], [(1, 230)], [(0, 0)]):
        ids = rows.clone()
        ids[128:160] = 7
        for lo, hi in gaps:
            ids[lo:hi] = -1
        C = native.w4a16_lora_gemm(*args, ids.cuda(), workspace=ws)
        check(C, A, La, Lb, scale, ids, packed, N, group, sym)


@pytest.mark.parametrize("M", [1, 6, 13, 40, 300])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_an_adapter_that_is_not_finite_stays_with_its_rows(M, dtype):
    K, N, group, sym, r, L = 1024, 256, 128, 0, 24, 4
    packed, tiled = layer(K, N, group, sym)
    A, La, Lb, scale, rows = make(M, K, N, r, L, dtype, torch.arange(M) % (L + 1) - 1)
    Lb[1, 77, 3] = float("inf")
    Lb[2, 5, 23] = float("nan")
    La[3, 1, 9] = float("nan")
    C = native.w4a16_lora_gemm(A.cuda(), tiled, N, group, sym, La.cuda(), Lb.cuda(), scale.cuda(), rows.cuda())
    good = (rows <= 0).nonzero().view(-1)
    check(C.cpu()[good], A[good], La, Lb, scale, rows[good], packed, N, group, sym)
    C = C.cpu()
    for a, ch in ((1, 77), (2, 5)):
        mine = (rows == a).nonzero().view(-1)
        assert not C[mine][:, ch].isfinite().any()
        others = [n for n in range(N) if n != ch]
        assert C[mine][:, others].isfinite().all()
    assert C[rows == 3].isnan().all()


@pytest.mark.parametrize("M", [5, 40])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rows_of_any_size_keep_to_themselves(M, dtype):
    """Rows and adapters far from one in size, a zero row, a row that is not finite."""
    K, N, group, sym, r, L = 256, 256, 128, 0, 16, 4
    packed, tiled = layer(K, N, group, sym)
    A, La, Lb, scale, rows = make(M, K, N, r, L, dtype, "any")
    A[0] *= 2.0 ** 12
    A[1] *= 2.0 ** -10
    A[2] = 0
    La[1] *= 2.0 ** -8
    scale[2] = 2.0 ** 10
    La[3, 5] = 0
    C = native.w4a16_lora_gemm(A.cuda(), tiled, N, group, sym, La.cuda(), Lb.cuda(), scale.cuda(), rows.cuda())
    check(C, A, La, Lb, scale, rows, packed, N, group, sym)
    bad = A.clone()
    bad[3, 9] = float("nan")
    D = native.w4a16_lora_gemm(bad.cuda(), tiled, N, group, sym, La.cuda(), Lb.cuda(), scale.cuda(), rows.cuda())
    # the decode kernel picks its bf16 arithmetic from all rows that a CTA stages (a row that is not
    # finite counts as too wide for fp16), so the other rows' sums may be formed in another order:
    # they are held to the same bound instead of to the same bits
    keep = torch.arange(M) != 3
    check(D.cpu()[keep], A[keep], La, Lb, scale, rows[keep], packed, N, group, sym)
    assert bool(D[3].isnan().all())


def test_without_adapters_it_is_the_layer():
    """No row with an adapter: the outputs of w4a16_gemm, bit for bit (one rounding of the same sums)."""
    for M, K, N, dtype in ((1, 512, 256, torch.float16), (7, 8192, 256, torch.bfloat16), (64, 512, 256, torch.bfloat16)):
        _, tiled = layer(K, N, 128, 0)
        A, La, Lb, scale, rows = make(M, K, N, 16, 2, dtype, "none")
        C = native.w4a16_lora_gemm(A.cuda(), tiled, N, 128, 0, La.cuda(), Lb.cuda(), scale.cuda(), rows.cuda())
        D = native.w4a16_gemm(A.cuda(), tiled, None, None, N, 128, 0, layout=native.LAYOUT_TILED)
        assert torch.equal(C, D)


@pytest.mark.parametrize("M", [4, 50])
def test_captured_and_replayed_on_other_rows(M):
    K, N, group, sym, r, L = 512, 384, 128, 0, 16, 6
    packed, tiled = layer(K, N, group, sym)
    A, La, Lb, scale, rows = (t.cuda() for t in make(M, K, N, r, L, torch.float16, "any"))
    C = torch.zeros(M, N, dtype=torch.float16, device="cuda")
    need = native.w4a16_lora_workspace_bytes(M, N, K, group, r, L)
    ws, ws2 = (torch.zeros(need, dtype=torch.uint8, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    native.w4a16_lora_gemm(A, tiled, N, group, sym, La, Lb, scale, rows, C=C, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        native.w4a16_lora_gemm(A, tiled, N, group, sym, La, Lb, scale, rows, C=C, workspace=ws)
    for seed in (5, 6):
        new = make(M, K, N, r, L, torch.float16, "any", seed=seed)
        for dst, src in zip((A, La, Lb, scale, rows), new):
            dst.copy_(src)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):   # at the same time, on its own workspace
            D = native.w4a16_lora_gemm(A, tiled, N, group, sym, La, Lb, scale, rows, workspace=ws2)
        torch.cuda.synchronize()
        assert torch.equal(C, D)
        check(C, *new, packed, N, group, sym)


@pytest.mark.parametrize("M", [1, 5])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_part_of_the_input_that_is_zero_or_tiny(M, dtype):
    """A CTA of the decode kernel stages a part of K: rows that are zero (or, bf16, tiny) there while their
    rank products are not, and a product far above the layer's (bf16: 2^34; fp16: 2^10)."""
    K, N, group, sym, r, L = 1024, 128, 128, 0, 16, 2
    packed, tiled = layer(K, N, group, sym)
    for lo, hi, by in ((0, 128, 0.0), (0, 512, 0.0), (512, 1024, 0.0), (0, 512, 2.0 ** -90), (0, 1024, 0.0)):
        if dtype == torch.float16 and by:
            continue
        for up in (1.0, 2.0 ** 16 if dtype == torch.bfloat16 else 2.0 ** 4):
            A, La, Lb, scale, rows = make(M, K, N, r, L, dtype, "one")
            A[:, lo:hi] *= by
            La, Lb = La * up, Lb * up
            C = native.w4a16_lora_gemm(A.cuda(), tiled, N, group, sym, La.cuda(), Lb.cuda(), scale.cuda(), rows.cuda())
            check(C, A, La, Lb, scale, rows, packed, N, group, sym)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_slices_of_k_where_rows_are_zero(dtype):
    """8 rows of 8192 inputs, which the decode kernel takes in slices of K: rows that are zero in the first or
    in the last slices, one row all zero."""
    M, K, N, group, sym, r, L = 8, 8192, 256, 128, 0, 16, 3
    packed, tiled = layer(K, N, group, sym)
    A, La, Lb, scale, rows = make(M, K, N, r, L, dtype, "any")
    A[:3, :K // 2] = 0
    A[3:6, K // 2:] = 0
    A[6] = 0
    C = native.w4a16_lora_gemm(A.cuda(), tiled, N, group, sym, La.cuda(), Lb.cuda(), scale.cuda(), rows.cuda())
    check(C, A, La, Lb, scale, rows, packed, N, group, sym)


# the down projections' input lengths, of which a CTA of the decode kernel stages a part
LONG = [(1, 14336, 256, 128, 0, torch.float16, 16, 2, "one"), (1, 28672, 128, 128, 1, torch.bfloat16, 64, 3, "one"),
        (3, 14336, 128, 64, 0, torch.bfloat16, 32, 3, "any"), (8, 28672, 128, 128, 0, torch.bfloat16, 16, 5, "any"),
        (8, 14336, 384, 128, 0, torch.float16, 64, 8, "any"), (7, 28672, 256, 32, 0, torch.float16, 8, 4, "wild"),
        (16, 28672, 128, 128, 0, torch.bfloat16, 32, 9, "any"), (40, 14336, 256, 128, 1, torch.bfloat16, 16, 7, "any"),
        (40, 28672, 128, 32, 0, torch.float16, 40, 3, "runs")]


@pytest.mark.parametrize("M,K,N,group,sym,dtype,r,L,ids", LONG)
def test_long_inputs(M, K, N, group, sym, dtype, r, L, ids):
    test_rows_with_their_adapters(M, K, N, group, sym, dtype, r, L, ids)


# several hundred rows in no order: every block of 256 meets most adapters
UNORDERED = [(542, 1152, 384, 128, 0, torch.float16, 112, 36, "any"), (700, 512, 256, 64, 1, torch.bfloat16, 64, 64, "any"),
             (384, 2048, 256, 128, 0, torch.bfloat16, 128, 40, "wild"), (900, 256, 128, 32, 0, torch.float16, 16, 300, "any")]


@pytest.mark.parametrize("M,K,N,group,sym,dtype,r,L,ids", UNORDERED)
def test_many_rows_in_no_order(M, K, N, group, sym, dtype, r, L, ids):
    test_rows_with_their_adapters(M, K, N, group, sym, dtype, r, L, ids)
