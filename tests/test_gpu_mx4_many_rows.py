"""The 4-bit projection at the ends of its row counts and strides: more chunks of 64 rows than a
grid's last dimension has, and one row with any stride.

Tolerance as in test_gpu_mx4_adapters: the fp32 sums, 2^-17 of the adapter's part,
and one rounding of y to bf16, 2^-8 of it."""
import pytest
import torch

import rank_delta_gb300 as rd
from rank_delta_gb300 import torch_helpers as th
from tests.test_gpu_mx4 import Setup, lib, nibbles, quantise, values  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [4_200_001, 65535 * 64 + 1])
def test_millions_of_rows(M):
    K, N, L, R = 32, 8, 3, 8
    gen = torch.Generator(device="cuda").manual_seed(M)
    normal = lambda *n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    codes, scales = quantise(normal(N, K) / 6)
    W = torch.tensor(values(nibbles(codes), scales.cpu().numpy())).cuda()
    route = th.DeviceRoute(L, R, K, N)
    x = normal(M, K).bfloat16()
    slots = torch.randint(-1, L, (M,), generator=gen, device="cuda", dtype=torch.int32)
    want, size = x.double() @ W.t(), x.double().abs() @ W.abs().t()
    for s in range(L):
        A, B = (normal(R, K) / 6).bfloat16(), normal(N, R).bfloat16()
        rd.lora_pool_pack(route.rt, s, A, B, R, 0.0, False, 1.0)
        mine = (slots == s)[:, None]
        want += torch.where(mine, (x.double() @ A.double().t()) @ B.double().t(), 0.0)
        size += torch.where(mine, (x.double().abs() @ A.double().abs().t()) @ B.double().abs().t(), 0.0)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = th.workspace(rd.lora_mx4_proj_workspace_bytes(M, route.rt))
    rd.lora_mx4_proj_apply(x, K, codes, scales, M, K, N, slots, route.rt, y, N, ws, ws.numel(), torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert rd.lora_status_get(ws) == 0
    bad = (y.double() - want).abs() > 2.0 ** -8 * want.abs() + (2.0 ** -16 + 66 * 2.0 ** -24) * size
    assert not bool(bad.any()), (int(bad.sum()), torch.nonzero(bad)[:3].tolist())


@pytest.mark.parametrize("path", [rd.LORA_MX4_PATH_ROWS, rd.LORA_MX4_PATH_TILES])
@pytest.mark.parametrize("stride", [1 << 39, 1 << 50])
def test_one_row_may_have_any_stride(path, stride):
    s = Setup(1, 512, 200, 2, 16, seed=4)
    want = s.run(path)
    y, ws = torch.empty_like(want), th.workspace(rd.lora_mx4_proj_workspace_bytes(1, s.route.rt))
    rd.lora_mx4_proj_apply(s.x, stride, s.codes, s.scales, 1, 512, 200, torch.tensor(s.slots).cuda(), s.route.rt, y, stride + 1, ws,
                           ws.numel(), None, path)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
