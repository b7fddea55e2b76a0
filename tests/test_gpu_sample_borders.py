"""lora_sample by exact sums alone, and next to the border of min-p.

Log probabilities as in test_gpu_sample.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import lib, place, sample  # noqa: F401
from tests.test_gpu_sample_rows import BF16, F32, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["plain", "q"])
@pytest.mark.parametrize("M,V", [(30, 70000), (16, 131072), (304, 33000)])
def test_exact_sums_by_clusters(M, V, how):
    """A uniform of 0 is told by exact sums alone: rows of clusters whose CTAs take parts of unlike work, many times. The
    first element weighs something in each, so it is the token; how many are kept, and the sum, are each part's."""
    gen = torch.Generator().manual_seed(M)
    x = torch.full((M, V), -30.0)
    x[:, 0] = 0.0
    x[:, V // 2] = 1.0
    for i in range(M):  # all that is kept lies in one part
        a = V // 8 * (i % 8)
        x[i, a:a + V // 8] = torch.maximum(x[i, a:a + V // 8], torch.randn(V // 8, generator=gen) * 0.1)
    x = place(x, BF16)
    q = None if how == "plain" else [0.1] * M
    w = torch.exp(x.double() - x.double().max(1, keepdim=True).values)
    keep = torch.ones_like(w, dtype=torch.bool) if q is None else w >= float(np.float32(0.1))
    kept = keep.sum(1).cpu().numpy()
    lp = (w[:, 0].log() - (w * keep).sum(1).log()).cpu().numpy()
    for _ in range(40):
        tok, got_lp, got_kept, flags = sample(x, [0.0] * M, None, None, None, q)
        assert flags == 0 and (tok == 0).all() and (got_kept == kept).all()
        assert np.abs(got_lp - lp).max() <= 6e-6 + 2.0 ** -21 * np.abs(lp).max()


def around(q, t, m):
    """The f32 that lies nearest to m + log(q) / t, and the three on either side."""
    x = np.float32(m + np.log(q) / t)
    out = [x]
    for way in (-np.inf, np.inf):
        y = x
        for _ in range(3):
            y = np.nextafter(y, np.float32(way))
            out.append(y)
    return [float(a) for a in out]


# short rows, a CTA a row, clusters, and many rows
PATHS = [(9, 2, 0), (12, 100, 5), (470, 700, 5), (12, 5001, 5), (6, 70000, 5), (630, 2100, 5)]


@pytest.mark.parametrize("m", [0.0, -6.5, 1000.0])
@pytest.mark.parametrize("M,V,others", PATHS)
def test_elements_a_few_steps_from_the_border(M, V, others, m):
    """min-p of 2^-5 to 2^-39, elements of f32 up to three steps on either side of its border: 1e-6 of their weight and
    less, where a unit of 2^-53 is up to 2^-14 of it."""
    gen = torch.Generator().manual_seed(V)
    x = torch.full((M, V), m - 200.0)
    qs, ts, us = [], [], torch.rand(M, generator=gen).tolist()
    for i in range(M):
        q, t = 2.0 ** -[39, 25, 15, 5][i % 4], float(np.float32([1.0, 0.75, 1.3][i % 3]))
        at = torch.randperm(V, generator=gen)[:2 + others].tolist()
        near = around(q, t, m)
        x[i, at[0]] = m
        for j, v in enumerate(at[1:]):
            x[i, v] = near[(i + j) % len(near)]
        qs.append(q)
        ts.append(t)
    assert compare(place(x, F32, 1, 1), us, ts, None, None, qs) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,V,others", PATHS)
def test_a_setting_a_step_from_an_element(M, V, others, dtype):
    """min_p is the weight of an element as fp32 has it, or one of the two numbers beside: 2^-24 of it apart."""
    gen = torch.Generator().manual_seed(V + 1)
    x = torch.full((M, V), -300.0)
    qs, us = [], torch.rand(M, generator=gen).tolist()
    for i in range(M):
        at = torch.randperm(V, generator=gen)[:2 + others].tolist()
        d = float(torch.tensor([-3.7, -9.3, -14.6, -26.9][i % 4]).to(dtype))
        x[i, at[0]] = 0.0
        x[i, at[1:]] = d
        q = np.float32(np.exp(d))
        qs.append(float([np.nextafter(q, np.float32(0)), q, np.nextafter(q, np.float32(1))][i % 3]))
    assert compare(place(x, dtype, 1, 1), us, None, None, None, qs) == 0


@pytest.mark.parametrize("M,V", [(3, 100), (6, 70000), (630, 2100)])
def test_min_p_of_1_keeps_the_equals_of_the_best_alone(M, V):
    """Elements a step below the best, at temperatures that bring their weights within 2^-60 of 1."""
    x = torch.full((M, V), 8.0)
    x[:, 1::2] = float(np.nextafter(np.float32(8.0), np.float32(0)))
    ts = [[1.0, 2.0 ** -10, 2.0 ** -40][i % 3] for i in range(M)]
    assert compare(place(x, F32, 0, 1), [0.7] * M, ts, None, None, [1.0] * M) == 0


@pytest.mark.parametrize("M,V", [(4, 100), (4, 70000), (630, 2100)])
def test_the_border_of_huge_logits(M, V):
    """m = 2^30, elements 64 apart, min_p as near e^-64 as fp32 numbers come: m + log min_p has no such digits in 64 bits
    (they end at 2^-22), the difference of an element and m has."""
    m = 2.0 ** 30
    q = np.float32(np.exp(-64.0))
    near = [np.nextafter(q, np.float32(0)), q, np.nextafter(q, np.float32(1))]
    x = torch.full((M, V), m - 640.0)
    x[:, V // 2] = m
    x[:, V // 3] = m - 64.0
    want = lambda row, u, t, k, p, q: (V // 2, 0.0, 1 + int(-64.0 >= np.log(q)))  # noqa: E731
    assert compare(place(x, F32), [0.5] * M, None, None, None, [float(near[i % 3]) for i in range(M)], want_of=want) == 0


@pytest.mark.parametrize("few", [2, 100, 128, 129, 700])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,V", [(12, 1500), (12, 5000), (6, 70000), (630, 2100)])
def test_rows_with_nothing_but_the_lowest_value(M, V, dtype, few):
    """All that is not masked by -infinity has the type's lowest value: equal weights, of which top-k keeps the first, and
    top-p and min-p of those."""
    gen = torch.Generator().manual_seed(V + few)
    x = torch.full((M, V), -np.inf)
    for i in range(M):
        x[i, torch.randperm(V, generator=gen)[:few]] = torch.finfo(dtype).min
    r = torch.rand(3, M, generator=gen).tolist()
    k = [[5, 0, 64, 1000][i % 4] for i in range(M)]
    p = [[0.5, 0.9, 1.0][i % 3] for i in range(M)]
    q = [[0.0, 0.3][i % 2] for i in range(M)]
    assert compare(place(x, dtype, 1, 1), r[0], [0.5 + a for a in r[1]], k, p, q) == 0
