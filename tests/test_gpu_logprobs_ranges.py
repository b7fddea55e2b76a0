"""Log probabilities and their gradient at the ends of their ranges: alternatives whose log
probability is beyond fp32, tokens that dominate their rows.

Definition, tolerances and placing as in test_gpu_logprobs; what the
definition gives is rounded to fp32 first, past its range to infinity."""
import numpy as np
import pytest
import torch

import rank_delta_gb300 as rd
from tests.test_gpu_logprobs import INF, LOG_TOL, check, define, forward, lib, place  # noqa: F401

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [37, 4099, 40001])
@pytest.mark.parametrize("g,h", [(0.7, None), (-1.5, None), (None, 0.3), (0.9, -0.4)])
def test_the_gradient_of_a_token_that_dominates_its_row(dtype, V, g, h):
    """1 - p from 1e-2 to 1e-7, a row each: the token's element relative to its own terms. 1 - p and H are as good
    as log S is relative to itself (LOG_TOL, see test_gpu_logprobs); the products and the function are good to 2^-21."""
    M, inv_t = 24, 0.75
    rng = np.random.default_rng(V)
    x = rng.standard_normal((M, V))
    at = rng.integers(0, V, M)
    x[np.arange(M), at] = (np.log(V) + np.linspace(4.6, 16.1, M)) / inv_t
    t = place(torch.tensor(x), dtype, 3, 1)
    x = t.double().cpu().numpy()
    d = (x - x.max(1, keepdims=True)) * inv_t
    assert (d.argmax(1) == at).all()
    others = np.exp(d)
    others[np.arange(M), at] = 0.0
    rest = others.sum(1)
    log_p, p, one_less = -np.log1p(rest), 1 / (1 + rest), rest / (1 + rest)
    entropy = np.log1p(rest) - (others * d).sum(1) / (1 + rest)
    token = torch.tensor(at.astype(np.int32)).cuda()
    f = forward(t, token, inv_t, 0)
    full = lambda v: None if v is None else torch.full((M,), v, device="cuda")  # noqa: E731
    out = torch.empty(M, V, dtype=dtype, device="cuda")
    rd.lora_logprobs_grad(t, rd.LORA_DTYPE_F32 if dtype == torch.float32 else rd.LORA_DTYPE_BF16, t.stride(0), M, V, token, inv_t,
                          f["stats"], f["entropy"] if h is not None else None, full(g), full(h), out, V)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()[np.arange(M), at]
    terms = inv_t * (g or 0.0) * one_less, -inv_t * (h or 0.0) * p * (log_p + entropy)
    want, size = terms[0] + terms[1], np.abs(terms[0]) + np.abs(terms[1])
    unit = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
    bad = ~(np.abs(got - want) <= (2 * LOG_TOL + 2.0 ** -21) * size + unit * np.abs(want))
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], one_less[bad][:4])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V", [(2, 40000), (3, 300), (3000, 257)])
@pytest.mark.parametrize("inv_t", [2.0 ** 127, 1e30, 2.0 ** -149])
def test_inverse_temperatures_at_their_ends(dtype, M, V, inv_t):
    """Greedy choice, with ties, and a uniform one."""
    rng = np.random.default_rng(V)
    t = place(torch.tensor(rng.integers(-9, 9, (M, V)).astype(np.float64)), dtype, 1, 0)
    tokens = rng.integers(0, V, M).astype(np.int32)
    check(forward(t, torch.tensor(tokens).cuda(), inv_t, 5), in_fp32(define(t, tokens, inv_t, 5)), V)
