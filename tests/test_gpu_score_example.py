"""The example that scores tokens under a 4-bit head with adapters, against
64-bit sums of the same steps.

Tolerances. Logits: one bf16 rounding, 2^-8 of the value, and s h rounded to
bf16 in it, 2^-8 of the expand's absolute products, on top of fp32 sums that
are far closer. Scores and gradient, from the very logits that the example
kept: fp32 sums of V terms in at most 64 dependent steps, 1e-5 of the largest
term; the gradient is rounded to bf16 once, 2^-8 of the value."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import rank_delta_gb300 as rd
from rank_delta_gb300 import build as rdbuild

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,hidden,vocab,adapters,rank,top", [(1, 256, 1000, 2, 8, 3), (70, 1024, 3000, 5, 12, 20)])
def test_scores_and_gradient(rows, hidden, vocab, adapters, rank, top):
    rdbuild.build()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "score_tokens.py")
    spec = importlib.util.spec_from_file_location("score_tokens", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.main(["--rows", str(rows), "--hidden", str(hidden), "--vocab", str(vocab), "--adapters", str(adapters),
                      "--rank", str(rank), "--top", str(top)])
    head, f64 = r["head"], lambda t: t.double().cpu().numpy()  # noqa: E731
    back = torch.empty_like(r["weight"])
    rd.lora_mx4_dequantize(head.codes, head.scales, vocab, hidden, back, rd.LORA_DTYPE_BF16, back.stride(0))
    x, slots = f64(r["x"]), r["slots"].cpu().numpy()
    want = x @ f64(back).T
    slack = 2.0 ** -8 * np.abs(want) + 1e-4
    for s, (a, b, scale) in enumerate(r["adapters"]):
        i = slots == s
        h = scale * x[i] @ f64(a).T
        want[i] += h @ f64(b).T
        slack[i] += 2.0 ** -8 * (np.abs(want[i]) + np.abs(h) @ np.abs(f64(b)).T)
    got = f64(r["logits"])
    assert (np.abs(got - want) <= slack).all()

    z = got - got.max(1, keepdims=True)
    p = np.exp(z)
    logp = z - np.log(p.sum(1, keepdims=True))
    p = np.exp(logp)
    entropy = -(p * logp).sum(1)
    tokens = r["tokens"].cpu().numpy()
    at = np.arange(rows), tokens
    assert np.abs(f64(head.logprob) - logp[at]).max() <= 1e-5 * np.abs(logp).max()
    assert np.abs(f64(head.entropy) - entropy).max() <= 1e-5 * np.abs(logp).max()
    ids = head.top_ids.cpu().numpy()
    order = np.lexsort((np.arange(vocab)[None].repeat(rows, 0), -got))[:, :top]  # ties: the lower id
    assert np.array_equal(ids, order)
    assert np.abs(f64(head.top_logprobs) - np.take_along_axis(logp, order, 1)).max() <= 1e-5 * np.abs(logp).max()
    adv = f64(r["advantage"])
    loss = -(adv * logp[at]).sum() - r["bonus"] * entropy.sum()
    assert abs(float(r["loss"]) - loss) <= 1e-5 * (np.abs(adv) * np.abs(logp).max() + r["bonus"] * entropy.max()).sum()
    hot = np.zeros_like(p)
    hot[at] = 1.0
    grad = -adv[:, None] * (hot - p) + r["bonus"] * p * (logp + entropy[:, None])
    terms = np.abs(adv)[:, None] * (hot + p) + r["bonus"] * p * (np.abs(logp) + entropy[:, None])
    assert (np.abs(f64(r["grad"]) - grad) <= 2.0 ** -8 * np.abs(grad) + 1e-5 * terms + 2.0 ** -133).all()
