"""Whole rows of log probabilities by CTAs that take five or more, one after another.

The rows are too long for a warp's and there are more than five times as many as
CTAs stay resident (three an SM), so what a CTA's reading threads leave for its
finishing warps is written over again and again, and two finishing warps take turns.
The rows that a CTA takes differ in kind. Definition and tolerances as in
test_gpu_logprobs."""
import numpy as np
import pytest
import torch

from tests.test_gpu_logprobs import INF, check, define, forward, lib, place  # noqa: F401

pytestmark = pytest.mark.gpu

V, KINDS, INV_T = 9001, 11, 0.75


@pytest.fixture(scope="module", params=[torch.bfloat16, torch.float32])
def rows(request):
    dtype = request.param
    M = 15 * torch.cuda.get_device_properties(0).multi_processor_count + 23
    rng = np.random.default_rng(11)
    x = rng.standard_normal((M, V)).astype(np.float32) * 3
    e = 8 if dtype == torch.bfloat16 else 4
    low = float(torch.finfo(dtype).min)
    kind = np.arange(M) % KINDS
    x[kind == 1] = 1.5                                    # equal
    x[kind == 2] = rng.integers(0, 3, (int((kind == 2).sum()), V))
    x[kind == 3] = np.arange(V) / 64                      # the best at the end
    x[np.ix_(kind == 4, np.arange(V) // e % 256 == 77)] += 25  # one thread's
    x[np.ix_(kind == 5, np.arange(200, 270))] += 20       # together
    x[np.ix_(kind == 6, np.arange(7, V))] = -INF          # seven left
    x[kind == 7] = -INF
    x[kind == 8, V - 1] = np.nan
    x[kind == 9, 3] = INF
    x[np.ix_(kind == 10, np.arange(4, V))] = low
    t = place(torch.tensor(x), dtype, 3, 1)
    tokens = rng.integers(-1, V, M).astype(np.int32)
    return t, tokens, define(t, tokens, INV_T, 32)


@pytest.mark.parametrize("k", [0, 1, 3, 8, 9, 20, 32])
def test_rows_of_different_kinds(rows, k):
    t, tokens, want = rows
    want = dict(want, top_ids=want["top_ids"][:, :k], top_logprobs=want["top_logprobs"][:, :k])
    got = forward(t, torch.tensor(tokens).cuda(), INV_T, k)
    check(got, want, V)
    assert got["flags"] == 0
    again = forward(t, torch.tensor(tokens).cuda(), INV_T, k)
    for name in ("logprob", "entropy", "stats", "top_logprobs"):
        assert torch.equal(got[name].view(torch.int32), again[name].view(torch.int32)), name
