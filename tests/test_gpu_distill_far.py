"""lora_distill and lora_distill_grad where a row has no distribution and nothing is left beside what is named, and
where what no entry names is far below the rest of the row.

Tolerances as in test_gpu_distill.py; lora_distill_grad takes a row's rest apart by itself where its log p is below
-256, so no digits of p / p_r hang on the statistics there, and the bound is the one-pass gradient's, whatever log p_r
is."""
import numpy as np
import pytest
import torch

from tests.test_gpu_distill import INF, NAN, REST, RENORM, check, define, distill, gradient, lib, place, same  # noqa: F401

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


def far_rows(V, n, dtype, values, gen):
    """Rows whose named tokens have ordinary values and whose others have one of `values`, or two a step apart."""
    M = 2 * len(values)
    x = torch.empty(M, V)
    ids = torch.stack([torch.randperm(V, generator=gen)[:n] for _ in range(M)]).int()
    for i, value in enumerate(values):
        x[2 * i] = value
        x[2 * i + 1] = value
        x[2 * i + 1, ::3] = value * 1.5 if abs(value) < 1e38 else value / 2
        if value > -1e9:
            x[2 * i + 1] += torch.randn(V, generator=gen)
    x.scatter_(1, ids.long(), torch.randn(M, n, generator=gen) * 2)
    teacher = torch.log_softmax(torch.randn(M, n + 1, generator=gen), -1)[:, :n].contiguous()  # a share is left for the rest
    return x, ids.cuda(), teacher.cuda()


@pytest.mark.parametrize("mode", [RENORM, REST])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,n,t,lead", [(40, 6, 1.0, 0), (5003, 20, 0.75, 3), (40000, 256, 1.25, 1), (131072, 20, 2.0, 0)])
def test_the_rest_far_below(dtype, V, n, t, lead, mode):
    gen = torch.Generator().manual_seed(V)
    low = torch.finfo(dtype).min
    x, ids, teacher = far_rows(V, n, dtype, [-100.0, -300.0, -1e4, -1e6, -1e9, -1e20, low / 4, low], gen)
    x = place(x, dtype, lead, 1)
    M = x.shape[0]
    want = define(x.double().cpu().numpy(), ids.cpu().numpy(), teacher.double().cpu().numpy(), mode, t)
    rows = x.double().cpu().numpy()
    for i in range(M):  # p / p_r from the rest alone: log p_r of -1e20 leaves no digits of log p - log p_r, in 64 bits either
        rest = rows[i].copy()
        rest[ids[i].cpu().numpy()] = -INF
        share = np.exp((rest - rest.max()) * t)
        share /= share.sum()
        log_rest, qr, Q = want["stats"][i, 2:5]
        other = rest > -INF
        want["dx"][i, other] = t * (Q * np.exp(log_rest) - qr) * share[other]
        want["terms"][i, other] = t * (Q * np.exp(log_rest) + qr) * share[other]
    g = torch.linspace(-1.0, 2.0, M, device="cuda")
    f64 = lambda a: a.double().cpu().numpy()  # noqa: E731
    dx = place(torch.full((M, V), 5.0), dtype, lead, 1)
    loss, stats, _ = distill(x, ids, teacher, mode, t, g, dx)
    big = (want["stats"][:, 2] < -3.4029e38) & (mode == REST)  # a log probability beyond fp32, whose largest is 3.40283e38
    assert same(f64(loss), want["loss"], want["slack"])[~big].all() and (f64(loss)[big] == INF).all()
    by = f64(g)[:, None] * want["dx"]
    tol = 2e-5 * np.abs(f64(g))[:, None] * want["terms"] + torch.finfo(dtype).eps / 2 * 1.01 * np.abs(by) + 1e-37
    logs = np.abs(want["stats"][:, 2]) + want["stats"][:, 1]
    near = np.where(logs < 300, logs, 0.0)[:, None]  # only there the statistics' digits
    from_stats = 2.0 ** -22 * near * np.abs(f64(g))[:, None] * want["terms"]
    for what, have, slack in (("step", dx, 0.0), ("grad", gradient(x, ids, teacher, mode, stats, g, torch.full_like(dx, 5.0), t), from_stats),
                              ("elsewhere in a vector", gradient(x, ids, teacher, mode, stats, g, place(torch.zeros(M, V), dtype, lead + 1, 3), t),
                               from_stats),
                              ("over the logits", (lambda c: gradient(c, ids, teacher, mode, stats, g, c, t))(place(x, dtype, lead, 1)), from_stats)):
        ok = same(f64(have), by, tol + slack)
        assert ok.all(), (what, np.argwhere(~ok)[:5].tolist(), f64(have)[~ok][:5], by[~ok][:5], tol[~ok][:5])


@pytest.mark.parametrize("mode", [RENORM, REST])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,n", [(1, 3), (50, 50), (5003, 20), (40000, 100)])
def test_tokens_beside_which_nothing_is_left_with_little_of_the_teacher(dtype, V, n, mode):
    """Q, the teacher's sum over them, is e^-1 to e^-25 and up to e^3, and a slope is Q p - q: of Q's size, not of p's."""
    gen = torch.Generator().manual_seed(V + n)
    sums = torch.tensor([3.0, 0.1, 0.0, -1e-6, -1.0, -5.0, -10.0, -17.0, -25.0])
    M = len(sums)
    x = torch.full((M, V), -INF)
    ids = torch.stack([torch.randperm(V, generator=gen)[:min(n, V)] for _ in range(M)])
    own = torch.randn(M, ids.shape[1], generator=gen) * 2
    x.scatter_(1, ids, own)
    teacher = torch.log_softmax(own + 0.01 * torch.randn(own.shape, generator=gen), 1) + sums[:, None]
    x, ids, teacher = place(x, dtype, 1, 1), ids.int().cuda(), teacher.cuda()
    f64 = lambda a: a.double().cpu().numpy()  # noqa: E731
    want = define(f64(x), ids.cpu().numpy(), f64(teacher), mode, 1.0)
    g = torch.linspace(-1.0, 2.0, M, device="cuda")
    dx = torch.zeros_like(x)
    loss, stats, _ = distill(x, ids, teacher, mode, 1.0, g, dx)
    assert same(f64(loss), want["loss"], want["slack"]).all()
    # a share is an integer of 2^-53, off by half of one, and Q the sum of n of them
    units = ids.shape[1] * 2.0 ** -54
    Q = want["stats"][:, 4]
    assert (np.abs(f64(stats[:, 4]) - Q) <= 2.0 ** -23 * Q + units).all()
    by = f64(g)[:, None] * want["dx"]
    tol = np.abs(f64(g))[:, None] * (2e-5 * want["terms"] + units) + torch.finfo(dtype).eps / 2 * 1.01 * np.abs(by) + 1e-37
    for what, have in (("step", dx), ("grad", gradient(x, ids, teacher, mode, stats, g, torch.full_like(dx, 5.0)))):
        ok = same(f64(have), by, tol)
        assert ok.all(), (what, np.argwhere(~ok)[:5].tolist(), f64(have)[~ok][:5], by[~ok][:5], tol[~ok][:5])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V,n", [(40, 3000, 2), (12, 32003, 8), (4, 131072, 20), (700, 5000, 3)])
def test_a_near_teacher_that_names_little_of_a_flat_row(dtype, M, V, n):
    """The rest has nearly all on both sides, so the loss is a small difference: log q_r and log p_r go by what they lack
    of 1. A row's sum is good to 4e-6 of itself, which is 4e-6 (1 - p_r) in log p_r; a named term to 4e-6 of its share
    (its logarithms of up to 16 have 2^-21 of them, 8e-6 of the share); the two logarithms of the rest to 2^-22 each."""
    gen = torch.Generator().manual_seed(V)
    x = place(torch.randn(M, V, generator=gen) * 0.5, dtype, 1, 1)
    ids = torch.stack([torch.randperm(V, generator=gen)[:n] for _ in range(M)])
    near = x.double().cpu() + 0.1 * torch.randn(M, V, generator=gen)
    teacher = torch.gather(torch.log_softmax(near, 1), 1, ids).float()
    f64 = lambda a: a.double().cpu().numpy()  # noqa: E731
    want = define(f64(x), ids.numpy(), f64(teacher), REST, 1.0)
    loss, stats, _ = distill(x, ids.int().cuda(), teacher.cuda(), REST)
    log_rest, qr, Q = want["stats"][:, 2], want["stats"][:, 3], want["stats"][:, 4]
    tol = 4e-6 * -np.expm1(log_rest) + 2.0 ** -22 * np.abs(log_rest)
    assert (np.abs(f64(stats[:, 2]) - log_rest) <= tol).all()
    off = np.abs(f64(loss) - want["loss"])
    tol += 1.2e-5 * (Q - qr) + 2.0 ** -22 * np.abs(np.log(qr)) + 2.0 ** -50
    assert (off <= tol).all(), (off.max(), tol[off.argmax()], want["loss"][off.argmax()])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [0.0, 64.0, -1024.0, 2.0 ** 13])
def test_a_teacher_of_plain_logits_far_from_0(dtype, offset):
    """LORA_DISTILL_RENORM takes values up to a constant. Those of this test are multiples of 2^-9, so that they are exact with
    each offset, and so is what the call makes of them: the share's logarithm is (val - best) - log of a sum, each
    within 2^-21 of up to 16, and so is log p; a share is off by 2^-21 of itself more, and times |log q - log p|. The
    loss is a sum of such terms."""
    gen = torch.Generator().manual_seed(6)
    M, V, n = 64, 3000, 30
    ids = torch.stack([torch.randperm(V, generator=gen)[:n] for _ in range(M)])
    teacher = (torch.randn(M, n, generator=gen) * 512).round() / 512
    x = torch.randn(M, V, generator=gen) - 12.0
    x.scatter_(1, ids, teacher + 0.05 * torch.randn(M, n, generator=gen))  # a near student
    x = place(x, dtype, 1, 1)
    f64 = lambda a: a.double().cpu().numpy()  # noqa: E731
    want = define(f64(x), ids.numpy(), f64(teacher), RENORM, 1.0)
    g = torch.ones(M, device="cuda")
    dx = torch.zeros_like(x)
    loss, _, _ = distill(x, ids.int().cuda(), (teacher + offset).cuda(), RENORM, 1.0, g, dx)
    off = np.abs(f64(loss) - want["loss"])
    assert off.max() <= 4e-6, (off.max(), want["loss"][off.argmax()])
    tol = 2e-5 * want["terms"] + torch.finfo(dtype).eps / 2 * 1.01 * np.abs(want["dx"]) + 1e-37
    assert same(f64(dx), want["dx"], tol).all()
