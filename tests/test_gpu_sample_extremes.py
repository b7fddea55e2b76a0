"""Whole calls of lora_sample against the definition in torch's doubles, with uniforms next to 0 and 1 and top-p next to
0 and 1 beside ordinary ones: the sums that decide there are the ones that fp32 and fine weights leave open most often.

Every row is compared. A count or a token may be another than the doubles' only where the border that parts the two
lies within 2^-40 of the sum, which is what the call promises; doubles' own sums are off by 2^-48 of it at most
(131072 additions in a tree's order, 2^-53 each)."""
import pytest
import torch

import rank_delta_gb300 as rd
from tests.test_gpu_sample import lib, tag  # noqa: F401
from tests.test_gpu_sample_rows import BF16, F32

pytestmark = pytest.mark.gpu

NEAR = 2.0 ** -40


def numbers(M, gen, ends):
    """Uniform numbers, every second of them one of `ends`."""
    u = torch.rand(M, generator=gen, device="cuda")
    at = torch.randint(len(ends), (M,), generator=gen, device="cuda")
    return torch.where(torch.arange(M, device="cuda") % 2 == 0, torch.tensor(ends, device="cuda")[at], u)


def check(x, u, t, k, p):
    M, V = x.shape
    tok, kept = (torch.full((M,), 123, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.full((256,), 0xAB, dtype=torch.uint8, device="cuda")
    rd.lora_sample(x, tag(x.dtype), V, M, V, u, t, k, p, None, tok, None, kept, ws, 256)
    assert rd.lora_status_get(ws) == 0
    rows = x.double()
    down, order = torch.sort(rows, dim=1, descending=True, stable=True)
    w = torch.exp((down - down[:, :1]) * t.double()[:, None])
    place = torch.arange(V, device="cuda")
    if k is not None:
        w = torch.where((place < k[:, None]) | (k[:, None] <= 0), w, 0.0)
    c = torch.cumsum(w, 1)
    limit = (w > 0).sum(1)
    n = kept.long()
    assert ((n >= 1) & (n <= V)).all()
    if p is None:
        want = torch.full((M,), V, device="cuda") if k is None else torch.where(k > 0, k.long().clamp(max=V), V)
        assert torch.equal(n, want)
    else:
        z = c[:, -1]
        share = p.double() * z
        up_to = torch.gather(c, 1, (n - 1)[:, None])[:, 0]
        before = torch.where(n > 1, torch.gather(c, 1, (n - 2).clamp(min=0)[:, None])[:, 0], -1.0)
        bad = ~((n == 1) | (before < share + NEAR * z)) | ~((up_to >= share - NEAR * z) | (n >= limit))
        assert not bad.any(), (bad.nonzero()[:4, 0].tolist(), n[bad][:4], p[bad][:4])
    # the draw, from the tokens that the call keeps
    inside = torch.zeros((M, V), dtype=torch.bool, device="cuda").scatter_(1, order, place < n[:, None])
    w = torch.where(inside, torch.exp((rows - down[:, :1]) * t.double()[:, None]), 0.0)
    c = torch.cumsum(w, 1)
    total, at = c[:, -1], tok.long()[:, None]
    assert ((at >= 0) & (at < V)).all() and torch.gather(inside, 1, at).all()
    target = u.double() * total
    hi = torch.gather(c, 1, at)[:, 0]
    lo = hi - torch.gather(w, 1, at)[:, 0]
    bad = (lo > target + NEAR * total) | (hi < target - NEAR * total)
    assert not bad.any(), (bad.nonzero()[:4, 0].tolist(), tok[bad][:4], u[bad][:4])
    return (tok.long() != (c <= target[:, None]).sum(1).clamp(max=V - 1)).sum().item()


# many rows read through registers (few of them open, and hundreds), clusters, a CTA a row, short rows
@pytest.mark.parametrize("M,V,dtype,wide", [(2048, 32000, BF16, 3.0), (1000, 20011, F32, 1.0), (96, 131072, BF16, 2.0), (24, 50257, F32, 1.5),
                                            (500, 9001, F32, 2.0), (3000, 1000, BF16, 2.0), (3000, 333, F32, 1.0)])
@pytest.mark.parametrize("how", ["plain", "p", "k", "kp"])
def test_against_doubles(M, V, dtype, wide, how):
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(1000 * V + seed)
        x = torch.randn(M, V, generator=gen, device="cuda") * (wide * (0.02 + torch.rand(M, 1, generator=gen, device="cuda")))
        u = numbers(M, gen, [2.0 ** -39, 2.0 ** -30, 2.0 ** -24, 1.0 - 2.0 ** -24, 1.0 - 2.0 ** -20])
        t = 0.5 + 1.5 * torch.rand(M, generator=gen, device="cuda")
        p = k = None
        if "p" in how and how != "plain":
            p = numbers(M, gen, [1.0 - 2.0 ** -24, 1.0 - 2.0 ** -20, 1.0 - 2.0 ** -12, 2.0 ** -20, 0.999])
        if "k" in how:
            k = (V ** torch.rand(M, generator=gen, device="cuda")).int()
        differ = check(x.to(dtype), u, t, k, p)
        assert differ <= 2 + M * V * 2.0 ** -39, differ  # (so many borders may lie that near)
