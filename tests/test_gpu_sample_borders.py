"""lora_sample by exact sums alone, and next to the border of min-p.

Log probabilities as in test_gpu_sample.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import lib, place, sample  # noqa: F401
from tests.test_gpu_sample_rows import BF16

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
