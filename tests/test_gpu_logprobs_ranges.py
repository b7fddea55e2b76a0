"""lora_logprobs at the ends of its ranges: alternatives whose log probability is beyond fp32.

Definition, tolerances and placing as in test_gpu_logprobs; what the
definition gives is rounded to fp32 first, past its range to infinity."""
import numpy as np
import pytest
import torch

from tests.test_gpu_logprobs import INF, check, define, forward, lib, place  # noqa: F401

pytestmark = pytest.mark.gpu


def in_fp32(want):
    with np.errstate(over="ignore"):
        return {k: v.astype(np.float32).astype(np.float64) if v.dtype.kind == "f" else v for k, v in want.items()}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V", [(6, 40), (6, 5003), (6, 40000), (520, 9000), (3000, 257)])
@pytest.mark.parametrize("inv_t,k", [(1.25, 32), (2.0, 5), (1.0, 20)])
def test_elements_of_the_lowest_value_are_alternatives(dtype, M, V, inv_t, k):
    """A row, a warp and a cluster a row: rows with fewer elements above the type's lowest value than alternatives asked for."""
    rng = np.random.default_rng(M + V)
    x = rng.standard_normal((M, V)) * 3
    low = float(torch.finfo(dtype).min)
    for i in range(M):
        keep = rng.choice(V, i % 4, replace=False)  # none, for a uniform row, to three
        mask = np.ones(V, bool)
        mask[keep] = False
        x[i, mask] = low
    x[1::6, ::2] = -INF  # of these, none is an alternative
    x[5::6, V // 2:] = -INF
    t = place(torch.tensor(x), dtype, 1, 2)
    tokens = rng.integers(-1, V, M).astype(np.int32)
    check(forward(t, torch.tensor(tokens).cuda(), inv_t, k), in_fp32(define(t, tokens, inv_t, k)), V)
