"""lora_logprobs and lora_logprobs_grad against their definitions in 64 bits.

Tolerances. The kernels sum in fp32: a thread's terms one after another (at
most V / 256 + 32 of them), then joins of a depth of at most 5 + 8 + 8, each
term 2^x of an argument that three roundings of 2^-24 relative went into and
with an error of 2^-22 of its own. For the V of these tests log S is then
within (V / 256 + 56) 2^-24 + 2^-21 < 2.5e-5, and the weighted means behind
the entropy within that times 1 + the largest |log p| that weighs in, which is
below 1 + log V + 4. Differences d are good to |d| 2^-22."""
import numpy as np
import pytest
import torch

import rank_delta_gb300 as rd
from rank_delta_gb300 import build as rdbuild

pytestmark = pytest.mark.gpu

LOG_TOL = 2.5e-5
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    rdbuild.build()
    assert torch.cuda.is_available()
    return rd.lib()


def tag(dtype):
    return rd.LORA_DTYPE_F32 if dtype == torch.float32 else rd.LORA_DTYPE_BF16


def place(values, dtype, lead, pad):
    """The rows at an offset of `lead` elements from a 16-byte boundary, `pad` elements apart."""
    M, V = values.shape
    buf = torch.zeros(lead + M * (V + pad) + 8, dtype=dtype, device="cuda")
    rows = buf[lead:lead + M * (V + pad)].view(M, V + pad)[:, :V]
    rows.copy_(values)
    return rows


def forward(x, tokens, inv_t, k, stream=None):
    M, V = x.shape
    new = lambda *n, dt=torch.float32: torch.full(n, 123, dtype=dt, device="cuda")  # noqa: E731
    out = dict(logprob=new(M), entropy=new(M), stats=new(M, 2), top_ids=new(M, k, dt=torch.int32), top_logprobs=new(M, k))
    ws = torch.full((rd.lora_logprobs_workspace_bytes(M, V, k),), 7, dtype=torch.uint8, device="cuda")
    rd.lora_logprobs(x, tag(x.dtype), x.stride(0), M, V, tokens, inv_t, k, out["logprob"], out["entropy"], out["stats"],
                     out["top_ids"], out["top_logprobs"], ws, ws.numel(), stream)
    torch.cuda.synchronize()
    out["flags"] = rd.lora_status_get(ws)
    return out


def define(x, tokens, inv_t, k):
    """The definition, a row at a time in 64 bits."""
    x = x.double().cpu().numpy()
    M, V = x.shape
    o = dict(logprob=np.zeros(M), entropy=np.zeros(M), stats=np.zeros((M, 2)), top_ids=np.full((M, k), -1),
             top_logprobs=np.full((M, k), -INF), lp=np.full((M, V), -INF))
    for i, row in enumerate(x):
        if np.isnan(row).any() or (row == INF).any():
            for a in ("entropy", "stats", "top_logprobs", "lp"):
                o[a][i] = np.nan
            o["logprob"][i] = np.nan if 0 <= tokens[i] < V else 0.0
            continue
        top = row.max()
        if top == -INF:
            o["stats"][i] = (-INF, 0.0)
            o["logprob"][i] = -INF if 0 <= tokens[i] < V else 0.0
            continue
        d = (row - top) * inv_t
        S = np.exp(d).sum()
        lp = d - np.log(S)
        p = np.exp(lp)
        some = p > 0
        o["lp"][i] = lp
        o["entropy"][i] = -(p[some] * lp[some]).sum()
        o["stats"][i] = (top, np.log(S))
        if 0 <= tokens[i] < V:
            o["logprob"][i] = lp[tokens[i]]
        order = np.lexsort((np.arange(V), -row))[:k]
        order = order[row[order] > -INF]
        o["top_ids"][i, :len(order)] = order
        o["top_logprobs"][i, :len(order)] = lp[order]
    return o


def check(got, want, V):
    def near(name, tol):
        g, w = got[name].double().cpu().numpy(), want[name]
        same = (g == w) | (np.isnan(g) & np.isnan(w))
        with np.errstate(invalid="ignore"):
            ok = same | (np.abs(g - w) <= tol + np.where(np.isfinite(w), np.abs(w), 0) * 2.0 ** -22)
        assert ok.all(), (name, np.argwhere(~ok)[:3].tolist(), g[~ok][:3], w[~ok][:3])

    near("stats", LOG_TOL)
    near("logprob", LOG_TOL)
    near("entropy", LOG_TOL * (5 + np.log(V)))
    near("top_logprobs", LOG_TOL)
    assert np.array_equal(got["top_ids"].cpu().numpy(), want["top_ids"])


def both(x, tokens, inv_t, k):
    got = forward(x, torch.tensor(tokens, dtype=torch.int32, device="cuda"), inv_t, k)
    check(got, define(x, tokens, inv_t, k), x.shape[1])
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V,lead,pad,k,inv_t", [
    (1, 1, 0, 0, 1, 1.0), (3, 2, 1, 0, 2, 1.0), (2, 7, 3, 1, 5, 0.5), (5, 8, 0, 0, 8, 1.0), (4, 33, 2, 4, 32, 2.0),
    (1, 1000, 0, 0, 0, 1.0), (3, 2049, 5, 0, 32, 1.25), (70, 4099, 0, 1, 3, 1.0), (1, 32000, 0, 0, 20, 1.0),
    (2, 70001, 7, 2, 32, 1.0), (400, 513, 1, 0, 1, 1.0), (160, 9000, 0, 8, 7, 0.25)])
def test_sizes_and_alignments(dtype, M, V, lead, pad, k, inv_t):
    gen = torch.Generator().manual_seed(M * 1000 + V)
    x = place(torch.randn(M, V, generator=gen) * 4, dtype, lead, pad)
    tokens = torch.randint(V, (M,), generator=gen).tolist()
    if M > 2:
        tokens[1] = -1
    got = both(x, tokens, inv_t, k)
    assert got["flags"] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [40, 5003, 40000])
def test_masks_ties_and_values_without_a_distribution(dtype, V):
    gen = torch.Generator().manual_seed(V)
    rows = torch.randn(14, V, generator=gen) * 3
    low = torch.finfo(dtype).min
    rows[0] = -INF                      # nothing left
    rows[1, 1:] = -INF                  # one element left
    rows[2, ::2] = -INF
    rows[3] = low                       # uniform
    rows[4, 3:] = low
    rows[5] = 1.5                       # ties everywhere
    rows[6] = (rows[6] > 0).float()     # two values
    rows[7, V // 2] = float("nan")
    rows[8, V - 1] = INF
    rows[9] = torch.arange(V) / V * 50  # the best at the end
    rows[10] = -torch.arange(V) / V * 50
    rows[11] = -0.0
    rows[11, ::3] = 0.0                 # equal to the others
    rows[12] = -INF
    rows[12, V - 2] = low
    step = 8 if dtype == torch.bfloat16 else 4
    share = (torch.arange(V) // step) % 256 == 17  # one thread's elements are the best
    rows[13, share] += 100
    x = place(rows, dtype, 0, 0)
    tokens = [0, 0, 1, V - 1, 0, 7, 3, 2, 5, V - 1, 0, 1, V - 2, 3]
    both(x, tokens, 1.0, 32)
    both(x, tokens, 1.0, 3)


def test_token_past_the_vocabulary_sets_the_flag_and_counts_as_none():
    x = torch.randn(3, 100, device="cuda")
    got = both(x, [100, -5, 99], 1.0, 1)
    assert got["flags"] == rd.LORA_FLAG_TOKEN_RANGE
    assert got["logprob"][:2].tolist() == [0.0, 0.0]
    assert both(x, [1, 2, 3], 1.0, 1)["flags"] == 0


def test_outputs_may_be_left_out():
    x = torch.randn(4, 3000, device="cuda")
    full = forward(x, torch.zeros(4, dtype=torch.int32, device="cuda"), 1.0, 2)
    ent = torch.empty(4, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    rd.lora_logprobs(x, rd.LORA_DTYPE_F32, 3000, 4, 3000, None, 1.0, 0, None, ent, None, None, None, ws, 256)
    torch.cuda.synchronize()
    assert torch.equal(ent, full["entropy"])
    rd.lora_logprobs(x, rd.LORA_DTYPE_F32, 3000, 0, 3000, None, 1.0, 0, None, None, None, None, None, None, 0)


def test_same_bytes_on_every_run_other_streams_and_in_a_graph():
    x = (torch.randn(6, 50021, device="cuda") * 3).to(torch.bfloat16)
    tok = torch.arange(6, dtype=torch.int32, device="cuda")
    first = forward(x, tok, 0.7, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for again in (forward(x, tok, 0.7, 16), forward(x, tok, 0.7, 16, side)):
        for name in ("logprob", "entropy", "stats", "top_ids", "top_logprobs"):
            assert torch.equal(first[name], again[name]), name
    out, ws = torch.zeros(6, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rd.lora_logprobs(x, rd.LORA_DTYPE_BF16, x.stride(0), 6, 50021, tok, 0.7, 0, out, None, None, None, None, ws, 256,
                         torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first["logprob"])


def test_rows_past_32_bit_offsets():
    V, stride = 1001, (1 << 30) + 8  # rows 2 GB apart in bf16: the third begins past 2^32 bytes
    buf = torch.zeros(2 * stride + V, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (3, V), (stride, 1))
    x.copy_(torch.randn(3, V) * 3)
    got = both(x, [3, 500, 1000], 1.0, 4)
    g = torch.ones(3, device="cuda")
    d = torch.empty(3, V, dtype=torch.bfloat16, device="cuda")
    rd.lora_logprobs_grad(x, rd.LORA_DTYPE_BF16, stride, 3, V, torch.tensor([3, 500, 1000], dtype=torch.int32, device="cuda"),
                          1.0, got["stats"], None, g, None, d, V)
    torch.cuda.synchronize()
    assert d[2, 1000] > 0 and d[0, 3] > 0


# ---------------------------------------------------------------- gradient


def define_grad(x, tokens, inv_t, g, h):
    o = define(x, tokens, inv_t, 0)
    lp = o["lp"]
    p = np.where(np.isnan(lp), np.nan, np.exp(lp))
    V = x.shape[1]
    want, scale = np.zeros(lp.shape), np.zeros(lp.shape)
    for i in range(len(lp)):
        if o["stats"][i, 0] == -INF:
            continue
        gi = g[i] if g is not None and 0 <= tokens[i] < V else 0.0
        hi = h[i] if h is not None else 0.0
        at = np.zeros(V)
        if 0 <= tokens[i] < V:
            at[tokens[i]] = 1.0
        with np.errstate(invalid="ignore"):
            inner = np.where(p[i] > 0, lp[i] + o["entropy"][i], 0.0)
            want[i] = inv_t * (gi * (at - p[i]) - hi * p[i] * inner)
            # what p, log p and H may be off by (see above), and one unit of the sum's roundings
            off = LOG_TOL + np.where(p[i] > 0, np.abs(lp[i]), 0.0) * 2.0 ** -21
            scale[i] = inv_t * (abs(gi) * (p[i] * off + at * 2.0 ** -23) +
                                abs(hi) * p[i] * (np.abs(inner) * off + off + LOG_TOL * (5 + np.log(V))))
        if np.isnan(lp[i]).any():
            want[i] = np.nan
    return o, want, scale


def run_grad(x, tokens, inv_t, g, h, d):
    tok = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    f = forward(x, tok, inv_t, 0)
    cu = lambda a: None if a is None else torch.tensor(a, dtype=torch.float32, device="cuda")  # noqa: E731
    rd.lora_logprobs_grad(x, tag(x.dtype), x.stride(0), x.shape[0], x.shape[1], tok, inv_t, f["stats"],
                          f["entropy"] if h is not None else None, cu(g), cu(h), d, d.stride(0))
    torch.cuda.synchronize()
    return d


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V,lead,pad,dlead,use", [
    (1, 1, 0, 0, 0, "gh"), (3, 2, 1, 0, 1, "g"), (2, 9, 0, 3, 2, "h"), (5, 33, 3, 0, 0, "gh"), (7, 4099, 1, 0, 1, "gh"),
    (2, 40001, 0, 0, 0, "g"), (40, 1003, 2, 2, 2, "h")])
def test_gradient_against_the_formula(dtype, M, V, lead, pad, dlead, use):
    rng = np.random.default_rng(M * 31 + V)
    x = place(torch.tensor(rng.standard_normal((M, V)) * 3), dtype, lead, pad)
    if V > 8:
        x[0, ::3] = -INF
        x[1] = -INF
    if M > 4:
        x[2, 5] = float("nan")
        x[3] = torch.finfo(dtype).min
    tokens = rng.integers(0, V, M).tolist()
    tokens[-1] = -1 if M > 1 else 0
    g = rng.standard_normal(M).astype(np.float32) if "g" in use else None
    h = rng.standard_normal(M).astype(np.float32) if "h" in use else None
    inv_t = 0.75
    o, want, scale = define_grad(x, tokens, inv_t, g, h)
    d = place(torch.full((M, V), 9.0), dtype, dlead, pad)
    got = run_grad(x, tokens, inv_t, g, h, d).double().cpu().numpy()
    rounding = 2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 2.0 ** -23 * np.abs(want)
    ok = (np.isnan(got) & np.isnan(want)) | (np.abs(got - want) <= scale * 1.01 + rounding + 1e-37)
    assert ok.all(), (np.argwhere(~ok)[:3].tolist(), got[~ok][:3], want[~ok][:3], scale[~ok][:3])


def test_gradient_over_the_logits_themselves():
    x = torch.randn(3, 5001, device="cuda")
    keep = x.clone()
    g = np.ones(3, np.float32)
    want = run_grad(keep, [1, 2, 3], 1.0, g, None, torch.empty_like(x))
    got = run_grad(x, [1, 2, 3], 1.0, g, None, x)
    assert torch.equal(got, want)


def test_gradient_against_differences_of_the_forward_kernel():
    """Central differences of fp32 outputs with steps of 2^-5: the truncation is
    step^2 / 6 times a third derivative of at most 2 (|g| + |h| (1 + H + |log p|)) < 40, that is 0.0065; the
    outputs' rounding, LOG_TOL * 7 over a step, is below 0.0055 in the worst case."""
    V, step = 9, 2.0 ** -5
    x = torch.randn(1, V, device="cuda")
    g, h, tok = np.array([0.8], np.float32), np.array([-0.6], np.float32), [4]
    d = run_grad(x, tok, 1.0, g, h, torch.empty_like(x))[0].cpu().numpy()
    t = torch.tensor(tok * (2 * V), dtype=torch.int32, device="cuda")
    moved = x.repeat(2 * V, 1)
    for v in range(V):
        moved[2 * v, v] += step
        moved[2 * v + 1, v] -= step
    f = forward(moved, t, 1.0, 0)
    val = (g[0] * f["logprob"].double() + h[0] * f["entropy"].double()).cpu().numpy()
    diff = (val[0::2] - val[1::2]) / (2 * step)
    assert np.abs(diff - d).max() < 0.012


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("k", [9, 20, 32])
def test_many_rows_whose_best_lie_together(dtype, k):
    """Whole rows by one CTA: the best in one thread's share, in a run, all equal, few distinct values, rising, masked but for
    fewer than k, one value apart; a CTA takes more than one row."""
    M, V = 700, 2500
    rng = np.random.default_rng(k)
    x = rng.standard_normal((M, V)).astype(np.float32)
    e = 16 // (2 if dtype == torch.bfloat16 else 4) * 8  # a vector of every eighth
    x[0::9] = 1.5
    x[1::9] = rng.integers(0, 3, x[1::9].shape)
    x[2::9] = np.arange(V) / 64
    x[3::9] = -np.arange(V) / 64
    x[4::9, 100:160] += 20
    x[5::9, ::e] += 20
    x[6::9, 5:] = -INF
    x[7::9] = np.finfo(np.float32).min if dtype == torch.float32 else -3.3895313892515355e38
    x[7::9, -1] = 0.0
    t = place(torch.tensor(x), dtype, 1, 3)
    tokens = rng.integers(-1, V, M).astype(np.int32)
    check(forward(t, torch.tensor(tokens).cuda(), 1.0, k), define(t, tokens, 1.0, k), V)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V", [(4, 32000), (400, 6000), (3, 131072)])
def test_rows_that_one_element_dominates(dtype, M, V):
    """Log S and the entropy relative to themselves, down to some 1e-4: 1 is left out of S before it is summed, so the
    tolerance of the sums of the others holds for them."""
    gen = torch.Generator().manual_seed(V)
    x = torch.randn(M, V, generator=gen)
    at = torch.randint(V, (M,), generator=gen)
    x[torch.arange(M), at] = 14 + 12 * torch.rand(M, generator=gen)
    x[::3, 5] = x[::3].amax(1) - 9  # a second one, far above the rest, 1e-4 of it
    t = place(x, dtype, 0, 0)
    tokens = at.to(torch.int32).cuda()
    got, want = forward(t, tokens, 1.0, 1), define(t, at.numpy(), 1.0, 1)
    for name, w in (("stats", want["stats"][:, 1]), ("entropy", want["entropy"]), ("logprob", want["logprob"])):
        g = got[name].double().cpu().numpy()
        g = g[:, 1] if name == "stats" else g
        if name == "stats":  # the sums of the others in 64 bits: log1p keeps what log of the whole loses
            d = t.double().cpu().numpy()
            d = np.exp(d - d.max(1, keepdims=True))
            d[np.arange(M), d.argmax(1)] = 0.0
            w = np.log1p(d.sum(1))
        elif name == "logprob":
            w = -np.log1p(d.sum(1))
        assert (np.abs(g - w) <= LOG_TOL * np.abs(w)).all(), (name, g[:4], w[:4])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V", [(520, 9000), (3000, 257), (1000, 4)])
@pytest.mark.parametrize("k", [0, 3, 20])
def test_many_rows_of_different_lengths(dtype, M, V, k):
    """Whole rows by CTAs that take several, and by warps; ties, masks, rows without a distribution, shares held by one thread."""
    k = min(k, V)
    rng = np.random.default_rng(M + k)
    x = rng.standard_normal((M, V)).astype(np.float32) * 3
    x[0::11] = -1.5
    x[1::11] = rng.integers(0, 2, x[1::11].shape)
    x[2::11] = np.arange(V) / 32
    x[3::11, V // 3:V // 3 + 70] += 15
    x[4::11, 1:] = -INF
    x[5::11] = -INF
    x[6::11, V - 1] = np.nan
    x[7::11, 0] = INF
    e = 16 // (2 if dtype == torch.bfloat16 else 4)
    x[8::11, ::32 * e] += 30
    t = place(torch.tensor(x), dtype, 3, 1)
    tokens = rng.integers(-1, V, M).astype(np.int32)
    got = forward(t, torch.tensor(tokens).cuda(), 0.75, k)
    check(got, define(t, tokens, 0.75, k), V)
    assert got["flags"] == 0
