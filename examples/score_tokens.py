"""The answering end of a multi-adapter server, and the training step on it.

A 4-bit output head serves rows of several adapters: its weight is quantised
once, each row's adapter is added in the projection that gives the logits, and
the tokens are scored from them: log probability, entropy and the best
alternatives. The same logits then give the gradient of a policy-gradient
loss with an entropy bonus,

    loss = -sum_i advantage_i * logprob_i - bonus * sum_i entropy_i,

written over the logits. Everything runs on one stream, without a copy to the
host between the calls:

    python examples/score_tokens.py [--rows 64] [--hidden 4096] [--vocab 32000] [--adapters 8] [--rank 16] [--top 5]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import rank_delta_gb300 as rd  # noqa: E402
from rank_delta_gb300 import torch_helpers as th  # noqa: E402


class Head:
    """A head [vocab][hidden] in 4 bits with its adapters, and the buffers of `rows` rows."""

    def __init__(self, weight: torch.Tensor, adapters, rows: int, top: int, stream):
        self.vocab, self.hidden = weight.shape
        dtype = rd.LORA_DTYPE_F32 if weight.dtype == torch.float32 else rd.LORA_DTYPE_BF16
        dev = weight.device
        self.codes = torch.empty(rd.lora_mx4_code_bytes(self.vocab, self.hidden), dtype=torch.uint8, device=dev)
        self.scales = torch.empty(rd.lora_mx4_scale_bytes(self.vocab, self.hidden), dtype=torch.uint8, device=dev)
        rd.lora_mx4_quantize(weight, dtype, weight.stride(0), self.vocab, self.hidden, self.codes, self.scales, stream)
        rank = max(8, -(-max(a.shape[0] for a, _, _ in adapters) // 8) * 8)
        self.route = th.DeviceRoute(len(adapters), rank, self.hidden, self.vocab, device=dev, stream=stream)
        for slot, (a, b, scale) in enumerate(adapters):
            rd.lora_pool_pack(self.route.rt, slot, a, b, a.shape[0], 0.0, False, scale, stream)
        self.top = top
        self.ws = th.workspace(rd.lora_mx4_proj_workspace_bytes(rows, self.route.rt), dev)
        self.score_ws = th.workspace(rd.lora_logprobs_workspace_bytes(rows, self.vocab, top), dev)
        new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        self.logits = new(rows, self.vocab, dtype=torch.bfloat16)
        self.logprob, self.entropy, self.stats = new(rows), new(rows), new(rows, 2)
        self.top_ids, self.top_logprobs = new(rows, top, dtype=torch.int32), new(rows, top)

    def score(self, x, slots, tokens, stream, inv_temperature: float = 1.0) -> None:
        """Logits of x [rows][hidden] under each row's adapter, and the scores of tokens."""
        m, y = x.shape[0], self.logits
        rd.lora_mx4_proj_apply(x, x.stride(0), self.codes, self.scales, m, self.hidden, self.vocab, slots, self.route.rt, y,
                               y.stride(0), self.ws, self.ws.numel(), stream)
        rd.lora_logprobs(y, rd.LORA_DTYPE_BF16, y.stride(0), m, self.vocab, tokens, inv_temperature, self.top, self.logprob,
                         self.entropy, self.stats, self.top_ids, self.top_logprobs, self.score_ws, self.score_ws.numel(), stream)

    def backward(self, m, tokens, grad_logprob, grad_entropy, stream, inv_temperature: float = 1.0) -> torch.Tensor:
        """The gradient with respect to the logits, over them."""
        y = self.logits
        rd.lora_logprobs_grad(y, rd.LORA_DTYPE_BF16, y.stride(0), m, self.vocab, tokens, inv_temperature, self.stats, self.entropy,
                              grad_logprob, grad_entropy, y, y.stride(0), stream)
        return y[:m]


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("rows", 64), ("hidden", 4096), ("vocab", 32000), ("adapters", 8), ("rank", 16), ("top", 5)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--bonus", type=float, default=0.01)
    a = ap.parse_args(argv)
    rng = torch.Generator(device="cuda").manual_seed(7)
    normal = lambda *shape: torch.randn(shape, generator=rng, device="cuda")  # noqa: E731
    weight = (normal(a.vocab, a.hidden) / a.hidden ** 0.5).bfloat16()
    adapters = [((normal(a.rank, a.hidden) / a.hidden ** 0.5).bfloat16(), (0.3 * normal(a.vocab, a.rank)).bfloat16(), 1.0)
                for _ in range(a.adapters)]
    x = normal(a.rows, a.hidden).bfloat16()
    slots = torch.arange(a.rows, dtype=torch.int32, device="cuda") % (a.adapters + 1) - 1  # -1: no adapter
    tokens = torch.randint(0, a.vocab, (a.rows,), generator=rng, device="cuda", dtype=torch.int32)
    advantage = normal(a.rows)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        head = Head(weight, adapters, a.rows, a.top, stream)
        head.score(x, slots, tokens, stream)
        logits = head.logits.clone()
        loss = -(advantage * head.logprob).sum() - a.bonus * head.entropy.sum()
        grad = head.backward(a.rows, tokens, -advantage, torch.full_like(advantage, -a.bonus), stream)
    stream.synchronize()
    for ws in (head.ws, head.score_ws):
        assert rd.lora_status_get(ws, stream) == 0
    print("loss %.4f, mean logprob %.4f, mean entropy %.4f" % (float(loss), float(head.logprob.mean()), float(head.entropy.mean())))
    for i in range(min(3, a.rows)):
        best = ["%d: %.3f" % t for t in zip(head.top_ids[i].tolist(), head.top_logprobs[i].tolist())]
        print("row %d (adapter %d) token %d %.3f; best %s" % (i, slots[i], tokens[i], head.logprob[i], ", ".join(best)))
    return {"head": head, "weight": weight, "adapters": adapters, "x": x, "slots": slots, "tokens": tokens,
            "advantage": advantage, "bonus": a.bonus, "logits": logits, "loss": loss, "grad": grad}


if __name__ == "__main__":
    main()
