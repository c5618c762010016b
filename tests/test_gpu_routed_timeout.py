"""The routed layers' bounded waits run out on purpose, and the device stays usable.

As for the dense layer: w4a16_set_wait_limit_ns(1) makes the tensor-core kernel's first pipeline waits
run out, and counters that start far below zero make the CTA that sums a cut tile wait for a count
it never sees (limit 1 ms). Nothing faults or traps: the kernel records W4A16_ETIMEOUT, lets its copies
and MMAs land and returns; the next call, on a zeroed workspace, is exact against the oracle.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import routed
from weight_only_int4_07_b200 import native, synthetic

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    native.lib()
    torch.cuda.set_device(0)
    yield
    native.w4a16_set_wait_limit_ns(0)


def _layer(K, N, seed):
    st, c, s, z = oracle.quantize(synthetic.weights_normal(K, N, seed), 128, 0)
    assert st == oracle.OK
    return (c, s, z), torch.from_numpy(oracle.repack(c, s, z, K, N, 128, 0)).cuda()


def _bits(t):
    return t.contiguous().view(torch.int16).numpy().view(np.uint16)


def _times_out_then_recovers(call, ws, how):
    """`call(status)` with waits that run out, then with the default limit on a zeroed workspace."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if how == "counters":
        ws[:65536] = 0x80
    torch.cuda.synchronize()
    prev = native.w4a16_set_wait_limit_ns(1 if how == "limit" else 1_000_000)
    try:
        call(status)
        torch.cuda.synchronize()            # the launch returned: no wait was left without a limit
    finally:
        native.w4a16_set_wait_limit_ns(prev)
    assert int(status) == native.ETIMEOUT
    ws.zero_()
    status.zero_()
    out = call(status)
    torch.cuda.synchronize()
    assert int(status) == 0 and not bool(ws[:65536].any())
    return out


@pytest.mark.parametrize("kernel,how", [(native.KERNEL_GEMV, "counters"), (native.KERNEL_TC, "counters"),
                                        (native.KERNEL_TC, "limit")])
def test_expert_products(kernel, how):
    E, K, N = 3, 4096, 2048
    layers = [_layer(K, N, 50 + e) for e in range(E)]
    off = torch.tensor([0, 5, 5, 9], dtype=torch.int32)
    A = torch.randn(9, K, generator=torch.Generator().manual_seed(1)).bfloat16()
    ws = torch.zeros(native.w4a16_moe_workspace_bytes(9, E, N, K, 128), dtype=torch.uint8, device="cuda")
    args = (A.cuda(), off.cuda(), torch.stack([t for _, t in layers]), N, 128, 0)
    C = _times_out_then_recovers(lambda s: native.w4a16_moe_gemm(*args, workspace=ws, kernel=kernel, dev_status=s), ws, how)
    for e in (0, 2):
        lo, hi = int(off[e]), int(off[e + 1])
        Y, mag = oracle.linear(_bits(A[lo:hi]), 1, *layers[e][0], N, 128, 0)
        # the weight's and the output's rounding to bf16, and FP32 sums
        assert (np.abs(C[lo:hi].cpu().double().numpy() - Y) <= (2.0 ** -8 + K * 2.0 ** -23) * mag + 2.0 ** -8 * np.abs(Y)).all()


@pytest.mark.parametrize("M,how", [(4, "counters"), (40, "counters"), (40, "limit"), (300, "limit")])
def test_adapters(M, how):
    K, N, r, L = 4096, 2048, 16, 3
    packed, tiled = _layer(K, N, 60)
    g = torch.Generator().manual_seed(2)
    A = torch.randn(M, K, generator=g).bfloat16()
    La = (torch.randn(L, r, K, generator=g) / 64).bfloat16()
    Lb = (torch.randn(L, N, r, generator=g) * 0.05).bfloat16()
    scale, ids = torch.ones(L), (torch.arange(M) % L).to(torch.int32)
    ws = torch.zeros(native.w4a16_lora_workspace_bytes(M, N, K, 128, r, L), dtype=torch.uint8, device="cuda")
    args = (A.cuda(), tiled, N, 128, 0, La.cuda(), Lb.cuda(), scale.cuda(), ids.cuda())
    C = _times_out_then_recovers(lambda s: native.w4a16_lora_gemm(*args, workspace=ws, dev_status=s), ws, how)
    cols = synthetic.column_sample(N, 64, seed=M)
    Y, mag = oracle.linear(_bits(A), 1, *packed, N, 128, 0, cols=cols)
    d, d1, d2, _ = routed.lora(A.double().numpy(), La.double().numpy(), Lb.double().numpy()[:, cols], scale.numpy(), ids.numpy())
    err = np.abs(C.cpu().double().numpy()[:, cols] - Y - d)
    # the terms of the bound of the adapters' tests, in bf16
    assert (err <= (2.0 ** -8 + K * 2.0 ** -23) * mag + K * 2.0 ** -23 * d2 + (2.0 ** -16 + r * 2.0 ** -22) * d1
            + 2.0 ** -8 * np.abs(Y + d)).all()
