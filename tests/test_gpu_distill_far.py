"""lora_distill and lora_distill_grad where a row has no distribution and nothing is left beside what is named.

Tolerances as in test_gpu_distill.py."""
import pytest
import torch

from tests.test_gpu_distill import INF, NAN, REST, RENORM, check, distill, lib, place  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [RENORM, REST])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [12, 3000, 70000])
def test_no_distribution_and_nothing_beside_what_is_named(dtype, V, mode):
    """A NaN or an infinity among the logits or the entries makes every element of the gradient NaN, masked ones too."""
    n = 6
    x = torch.full((6, V), -INF)
    ids = torch.arange(n, dtype=torch.int32).repeat(6, 1)
    teacher = torch.full((6, n), -2.0)
    x[0, :n] = torch.arange(n) * 1.0
    x[0, 2] = NAN                       # a named one
    x[1, :n] = 1.0
    x[1, 3] = INF
    x[2, :n] = 1.0
    teacher[2, 4] = NAN                 # an entry, the rest masked
    teacher[3, 0] = INF                 # an entry, all masked
    x[4, n:] = 0.5
    teacher[4, 1] = NAN                 # an entry, nothing masked
    x[5, V - 1] = NAN                   # one that nobody names
    x, ids, teacher = place(x, dtype, 1), ids.cuda(), teacher.cuda()
    check(x, ids, teacher, mode, 1.0)
    g = torch.ones(6, device="cuda")
    dx = torch.zeros_like(x)
    loss, _, _ = distill(x, ids, teacher, mode, 1.0, g, dx)
    assert loss.isnan().all() and dx.isnan().all()
