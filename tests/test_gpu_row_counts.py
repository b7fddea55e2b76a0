"""A workspace of lora_sample or lora_distill whose first words went back to what they were, with the words behind them
left as a call put them: memory that is handed out again, or a caller that clears the front. Nothing of the earlier call
counts in the next one."""
import pytest
import torch

import rank_delta_gb300 as rd
from tests.test_gpu_sample import lib, tag  # noqa: F401
from tests.test_gpu_sample_rows import BF16, on_device

pytestmark = pytest.mark.gpu


def fresh(fill=0):
    return torch.full((256,), fill, dtype=torch.uint8, device="cuda")


def draw(x, s, ws):
    M, V = x.shape
    out = [torch.full((M,), 123, dtype=d, device="cuda") for d in (torch.int32, torch.float32, torch.int32)]
    rd.lora_sample(x, tag(x.dtype), V, M, V, *s, *out, ws, 256)
    torch.cuda.synchronize()
    return out


def go_back(ws, how, epoch):
    words = ws.view(torch.int32)
    if how == "front":
        words[:4] = 0
    else:
        words[2] = epoch


# rows by CTAs of two and eight warps, by clusters, and (from 600 on) through the three kernels of many rows
@pytest.mark.parametrize("M,V", [(3000, 500), (1500, 20000), (40, 60000), (700, 4001), (2000, 2500)])
@pytest.mark.parametrize("how", ["front", "epoch"])
def test_rows_are_all_drawn(M, V, how):
    gen = torch.Generator().manual_seed(M)
    x = (torch.randn(M, V, generator=gen) * 0.5).cuda().bfloat16()  # flat: many rows are left open
    s = on_device(M, gen)
    want = draw(x, s, fresh())
    ws = fresh()
    for turn in range(3):
        epoch = int(ws.view(torch.int32)[2])
        got = draw(x, s, ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), turn
        assert int(ws.view(torch.int32)[2]) == epoch + 1  # the status was written
        go_back(ws, how, epoch)


@pytest.mark.parametrize("M,V", [(3000, 500), (40, 60000), (700, 4001)])
@pytest.mark.parametrize("how", ["front", "epoch"])
def test_flags_of_both_operators(M, V, how):
    gen = torch.Generator().manual_seed(M)
    x = torch.randn(M, V, generator=gen).cuda().bfloat16()
    u = torch.full((M,), 0.5, device="cuda")
    u[M // 2] = 2.0
    ids = torch.full((M, 4), V, dtype=torch.int32, device="cuda")
    teacher, loss = torch.zeros(M, 4, device="cuda"), torch.empty(M, device="cuda")
    ws = fresh()
    for _ in range(3):
        epoch = int(ws.view(torch.int32)[2])
        draw(x, (u, None, None, None, None), ws)
        assert rd.lora_status_get(ws) == rd.LORA_FLAG_SETTING_RANGE
        go_back(ws, how, epoch)
        rd.lora_distill(x, tag(BF16), V, M, V, 1.0, ids, teacher, 4, rd.LORA_DISTILL_REST, loss, None, None, None, 0, ws, 256)
        assert rd.lora_status_get(ws) == rd.LORA_FLAG_TOKEN_RANGE
        go_back(ws, how, epoch)
