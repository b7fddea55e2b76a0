"""The adapters' part of the 4-bit projection: s A x reaches the expand with more bits than y has.

Tolerance, an element before its rounding: (n / 16 + 64) 2^-24 of the absolute
products for a sum of n of them in fp32 (base and shrink over K, expand over 2
R: two bf16 an element of s A x), and 2^-17 of the expand's absolute products
for the two bf16. The result has to lie between the bf16 roundings of the two
ends. (With one bf16 for s A x a tenth of the elements and more lie outside.)"""
import numpy as np
import pytest
import torch

import rank_delta_gb300 as rd
from rank_delta_gb300 import torch_helpers as th
from tests.test_gpu_mx4 import PATHS, Setup, lib, nibbles, values  # noqa: F401

pytestmark = pytest.mark.gpu


def deep(n):
    return (n / 16 + 64) * 2.0 ** -24


def check(s, y):
    x = s.x.double().cpu().numpy()
    W = values(nibbles(s.codes), s.scales.cpu().numpy())
    want, tol = x @ W.T, deep(s.K) * (np.abs(x) @ np.abs(W).T)
    for slot, d in enumerate(s.delta):
        rows = np.nonzero(s.slots == slot)[0]
        if d is None or not len(rows):
            continue
        A, B, scale = d
        h, hb = x[rows] @ A.T, np.abs(x[rows]) @ np.abs(A).T
        want[rows] += scale * (h @ B.T)
        tol[rows] += scale * ((2.0 ** -17 + deep(2 * s.R)) * np.abs(h) @ np.abs(B).T + deep(s.K) * hb @ np.abs(B).T)
    got = y.double().cpu().numpy()
    low, high = [torch.tensor(v).to(torch.float32).to(torch.bfloat16).double().numpy() for v in (want - tol, want + tol)]
    bad = ~((low <= got) & (got <= high))
    assert not bad.any(), (bad.mean(), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("M,K,N,L,R", [
    (1, 256, 256, 1, 16), (3, 2080, 130, 3, 64), (4, 512, 300, 4, 200), (7, 1056, 257, 4, 24), (20, 512, 128, 20, 256),
    (48, 512, 150, 80, 16), (64, 4096, 384, 8, 32), (64, 4096, 1100, 16, 64), (150, 4096, 1100, 16, 24), (256, 2048, 2048, 8, 16),
    (256, 4224, 300, 32, 64), (300, 800, 200, 24, 72), (2304, 2080, 16, 24, 32), (2100, 96, 72, 2, 136)])
@pytest.mark.parametrize("path", PATHS)
def test_adapters_lose_no_bits_on_either_path(path, M, K, N, L, R):
    s = Setup(M, K, N, L, R, seed=M + K + R)
    s.slots = (np.arange(M, dtype=np.int32) * 7) % L
    check(s, s.run(path))
    assert s.flags == 0


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("M", [2, 70])
def test_adapters_at_the_ends_of_the_range(path, M):
    """s A x past the largest bf16 but not past fp32, tiny, and infinite: y is what B makes of it."""
    K, N, R = 64, 40, 16
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    route = th.DeviceRoute(3, R, K, N)
    largest = float(torch.finfo(torch.bfloat16).max)
    for slot, (a, b) in enumerate([((largest, 0.75 * 2.0 ** 120), 2.0 ** -120), ((2.0 ** -60, 2.0 ** -72), 2.0 ** 30),
                                   ((float("inf"), 1.0), 0.5)]):
        A = torch.zeros(1, K, dtype=torch.bfloat16)
        A[0, 0], A[0, 1] = a
        rd.lora_pool_pack(route.rt, slot, A.cuda(), torch.full((N, 1), b, dtype=torch.bfloat16, device="cuda"), 1, 0.0, False, 1.0)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[:, :2] = 1.0
    slots = torch.arange(M, dtype=torch.int32, device="cuda") % 4 - 1
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = th.workspace(rd.lora_mx4_proj_workspace_bytes(M, route.rt))
    rd.lora_mx4_proj_apply(x, K, codes, scales, M, K, N, slots, route.rt, y, N, ws, ws.numel(), torch.cuda.current_stream(), path)
    torch.cuda.synchronize()
    assert rd.lora_status_get(ws) == 0
    want = torch.tensor([0.0, (largest + 0.75 * 2.0 ** 120) * 2.0 ** -120, (2.0 ** -60 + 2.0 ** -72) * 2.0 ** 30, float("inf")],
                        dtype=torch.float64).to(torch.float32).to(torch.bfloat16).cuda()
    assert torch.equal(y, want[(slots + 1).long()][:, None].expand(M, N))
