"""The rows kernel of the 4-bit projection (one to four rows) where it goes round its rings.

A CTA takes many steps (few features a step and more of them than the device
has SMs), a warp one or two boxes of 256 k a step, all warps or some; scale
rows lie on 8-byte boundaries or not; ranks from 8 to 256. Up to 8192 k and
four rows LORA_MX4_PATH_ROWS takes that kernel. Tolerance as in
test_gpu_mx4_adapters."""
import numpy as np
import pytest
import torch

import rank_delta_gb300 as rd
from tests.test_gpu_mx4 import Setup, lib  # noqa: F401
from tests.test_gpu_mx4_adapters import check

pytestmark = pytest.mark.gpu

ROWS = rd.LORA_MX4_PATH_ROWS


@pytest.mark.parametrize("M,K,N,L,R", [
    (1, 4096, 32000, 2, 64), (3, 4096, 10007, 4, 16), (4, 4096, 10007, 5, 256), (2, 4352, 5000, 3, 8), (4, 4352, 9001, 4, 24),
    (1, 8192, 9001, 2, 128), (4, 8192, 9001, 5, 64), (3, 4128, 7003, 4, 40), (2, 8160, 9001, 3, 16), (4, 256, 80001, 4, 8),
    (1, 32, 160001, 2, 8), (4, 2080, 10007, 3, 104)])
def test_many_steps_a_cta(M, K, N, L, R):
    s = Setup(M, K, N, L, R, seed=M + K + N)
    check(s, s.run(ROWS, y_pad=M % 2))
    assert s.flags == 0


@pytest.mark.parametrize("K,N", [(1056, 300), (8192, 5001)])
@pytest.mark.parametrize("order", [(-1, 0, 1, 6), (2, 3, -1, 4), (5, 1, 1, 2), (-1, 7, 3, 0)])
def test_rows_without_a_delta_keep_the_base_product(K, N, order):
    """None, an empty slot (1), one of scale 0 (2) and ones out of range (6, 7), each beside rows with one."""
    s = Setup(4, K, N, 6, 16, seed=3)
    base = s.run(ROWS, np.full(4, -1, np.int32))
    s.slots = np.array(order, np.int32)
    y = s.run(ROWS)
    assert s.flags == (rd.LORA_FLAG_SLOT_RANGE if max(order) >= 6 else 0)
    check(s, y)
    off = torch.tensor(np.isin(s.slots, (-1, 1, 2, 6, 7))).cuda()
    assert torch.equal(y[off].view(torch.int16), base[off].view(torch.int16))


def test_a_stack_of_adapters():
    s = Setup(3, 512, 3000, 1, 32, seed=5)
    rng = np.random.default_rng(9)
    bf = lambda a: torch.tensor(a).to(torch.bfloat16).cuda()  # noqa: E731
    A = [bf(rng.standard_normal((r, 512)) / 22) for r in (8, 5)]
    B = [bf(rng.standard_normal((3000, r)) * 0.2) for r in (8, 5)]
    rd.lora_pool_pack_stack(s.route.rt, 0, A, B, [8, 5], [0.0, 0.0], [False, False], [2.0, -0.5])
    s.delta[0] = (torch.cat(A).double().cpu().numpy(), torch.cat((2.0 * B[0].double(), -0.5 * B[1].double()), 1).cpu().numpy(), 1.0)
    s.slots[:] = 0, -1, 0
    check(s, s.run(ROWS))


@pytest.mark.parametrize("M,K,N", [(4, 4096, 10007), (2, 8192, 9001), (1, 4096, 32000)])
def test_the_same_bytes_on_every_run_and_on_another_stream(M, K, N):
    s = Setup(M, K, N, 4, 32, seed=7)
    first = s.run(ROWS).view(torch.int16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, None, side):
        assert torch.equal(s.run(ROWS, stream=stream).view(torch.int16), first)
