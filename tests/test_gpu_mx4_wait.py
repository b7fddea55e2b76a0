"""Bounded waits of the 4-bit projection that run out (GPU only; nothing faults or hangs).

Through the test hook the limit is cut to 200 us, and one kind of barrier
counts an arrival that never comes: the adapters' stages (tiles) or a step's
sums (rows kernel), or the base's stages. The call must return and report
LORA_FLAG_WAIT_TIMEOUT, whichever role gives up first, and the next normal
call on other buffers must give the bytes that one before it gave. The shapes
have one, two and four segments of 16 ranks a stage and fewer and more stages
than there are places for, one and several parts of K, and all three tile
heights."""
import numpy as np
import pytest
import torch

import rank_delta_gb300 as rd
from tests.test_gpu_mx4 import Setup, lib  # noqa: F401

pytestmark = pytest.mark.gpu

ROWS, TILES = rd.LORA_MX4_PATH_ROWS, rd.LORA_MX4_PATH_TILES


@pytest.mark.parametrize("path,M,K,N,L,R", [
    (ROWS, 1, 4096, 10007, 2, 16), (ROWS, 4, 5120, 300, 4, 64), (TILES, 8, 256, 130, 1, 16), (TILES, 40, 4096, 600, 16, 64),
    (TILES, 64, 1024, 30000, 16, 64), (TILES, 128, 2080, 1100, 24, 64), (TILES, 256, 4096, 1100, 32, 64), (TILES, 600, 512, 520, 40, 40)])
@pytest.mark.parametrize("never", [1, 2])
def test_a_wait_that_runs_out_is_reported(path, M, K, N, L, R, never):
    s = Setup(M, K, N, L, R, seed=M + N)
    s.slots = np.arange(M, dtype=np.int32) % L
    s.slots[s.slots == 1] = 0 if L > 2 else 1  # slot 1 of several is empty
    want = s.run(path)
    assert s.flags == 0
    rd.lora_test_wait_hook(200_000, never)
    try:
        s.run(path)
        flags = s.flags
    finally:
        rd.lora_test_wait_hook(0, 0)
    assert flags & rd.LORA_FLAG_WAIT_TIMEOUT, f"status {flags:#x}"
    again = s.run(path)
    assert s.flags == 0, f"the next call reports {s.flags:#x}"
    assert torch.equal(again.view(torch.int16), want.view(torch.int16))
