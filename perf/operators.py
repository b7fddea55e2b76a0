"""The operators of the answering end of a multi-adapter server, as measured cases.

A request's last steps: hidden states go through a base matrix kept in
microscaled 4-bit floating point with each row's own adapter on top, and the
logits that come out are turned into log probabilities (to sample from, to
score a prompt, or to train on):

* quantise   -- a bf16 or f32 matrix to 4-bit codes with one power-of-two scale
                for 32 of them, and the values read back;
* project    -- y = dq(W) x + s B (A x) with W in that form, an adapter a row;
* logprobs   -- log probability of a given token a row, the row's entropy, the
                statistics of its softmax, and its best alternatives;
* grad       -- the gradient of the log probability and the entropy with
                respect to the logits.

``run`` computes a pass either in plain torch (32-bit arithmetic, rounded
once), or, where ``own`` is set, through rank_delta_gb300.
"""
import math

import torch

own = False

BLOCK = 32  # values that share a scale
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of the codes 0..7; code 8 + c is -MAGNITUDES[c]


def listed():
    return [
        # a decode-sized square projection's weight, as it is loaded
        dict(name="quantise 4096x4096", op="quantise", rows=4096, K=4096, f32=False, pad=0),
        # an f32 master copy with rows that are not packed, an odd number of rows
        dict(name="quantise f32 strided", op="quantise", rows=2047, K=2080, f32=True, pad=5),
        # a gate/up weight
        dict(name="quantise 14336x4096", op="quantise", rows=14336, K=4096, f32=False, pad=0),
        # one request decoding
        dict(name="project 1 row", op="project", M=1, K=4096, N=4096, L=16, R=64),
        # a decode batch, sixteen adapters in it
        dict(name="project 64 rows", op="project", M=64, K=4096, N=4096, L=16, R=64),
        # a fused q/k/v projection of a larger batch, many small adapters
        dict(name="project 256 rows qkv", op="project", M=256, K=4096, N=6144, L=32, R=16),
        # eight prompts of 1024 tokens through gate/up, an adapter each
        dict(name="project 8192 rows", op="project", M=8192, K=4096, N=14336, L=8, R=64),
        # one request's next token with its best twenty
        dict(name="logprobs 1 row", op="logprobs", M=1, V=32000, pad=0, f32=False, top=20, inv_t=1.25),
        # a decode batch from f32 logits, a vocabulary of odd size without padding
        dict(name="logprobs 64 rows f32", op="logprobs", M=64, V=32003, pad=0, f32=True, top=5, inv_t=1.0),
        # eight prompts of 1024 tokens scored
        dict(name="logprobs 8192 rows", op="logprobs", M=8192, V=32000, pad=0, f32=False, top=1, inv_t=1.0),
        # a small training batch with an entropy bonus, odd rows
        dict(name="grad 96 rows", op="grad", M=96, V=32003, pad=0, f32=True, bonus=True, inv_t=1.0),
        # a training batch of eight sequences
        dict(name="grad 8192 rows", op="grad", M=8192, V=32000, pad=0, f32=False, bonus=False, inv_t=1.0),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("quantise", "project", "project", "logprobs", "logprobs", "grad"))
    if op == "quantise":
        while True:
            case = dict(op=op, rows=_spread(rng, 16, 16384), K=BLOCK * _spread(rng, 8, 256), f32=rng.random() < 0.3,
                        pad=rng.choice((0, 0, 8, 3)))
            if case["rows"] * case["K"] * (4 if case["f32"] else 2) <= 14336 * 4096 * 2:
                return case
    if op == "project":
        while True:
            case = dict(op=op, M=_spread(rng, 1, 8192), K=BLOCK * _spread(rng, 16, 256), N=_spread(rng, 250, 16384),
                        L=rng.randint(1, 32), R=8 * _spread(rng, 1, 8))
            if case["M"] * case["K"] * case["N"] <= 8192 * 4096 * 14336 // 2:
                return case
    while True:
        case = dict(op=op, M=_spread(rng, 1, 8192), V=_spread(rng, 1000, 131072), pad=rng.choice((0, 0, 1, 8)),
                    f32=rng.random() < 0.5, inv_t=rng.choice((1.0, 1.0, 0.5, 1.25)))
        if case["M"] * case["V"] * (2 if case["f32"] else 1) <= 8192 * 32000:
            break
    if op == "logprobs":
        case["top"] = rng.choice((0, 1, 5, 20, 32))
    else:
        case["bonus"] = rng.random() < 0.5
    return case


def work(case):
    if case["op"] == "quantise":
        n = case["rows"] * case["K"]
        size = 4 if case["f32"] else 2
        return {"bytes": n * 2 * size + 2 * (n // 2 + n // BLOCK), "flops": 3 * n}
    if case["op"] == "project":
        M, K, N, L, R = (case[k] for k in "MKNLR")
        return {"bytes": N * K // 2 + N * K // BLOCK + 2 * M * (K + N) + 2 * min(M, L) * R * (K + N) + 4 * M,
                "flops": 2 * M * K * N + 2 * M * R * (K + N)}
    n = case["M"] * case["V"]
    size = 4 if case["f32"] else 2
    if case["op"] == "logprobs":
        return {"bytes": n * size + case["M"] * (4 + 16 + 8 * case["top"]), "flops": 5 * n}
    return {"bytes": 2 * n * size + 24 * case["M"], "flops": 5 * n}


# ------------------------------------------------------------------ plain forms


def _power(byte):
    """2^(byte - 127) in f32 (byte 0: the subnormal 2^-127; 255: NaN)."""
    bits = torch.where(byte == 0, torch.full_like(byte, 1 << 22), byte << 23)
    p = bits.view(torch.float32)
    return torch.where(byte == 255, torch.full_like(p, math.nan), p)


def _quantise(w):
    """(codes 0..15 [rows][K], scale bytes [rows][K/32]), both int32."""
    f = w.float().view(w.shape[0], -1, BLOCK)
    amax = f.abs().amax(-1)
    byte = torch.frexp(amax)[1] + (127 - 1 - 2)  # floor(log2 amax) - 2, biased
    byte = torch.where(amax == 0, torch.zeros_like(byte), byte.clamp(0, 254))
    byte = torch.where(torch.isfinite(amax), byte, torch.full_like(byte, 255))
    m = f.abs() * ((254 - byte.clamp(max=253)) << 23).view(torch.float32)[..., None]
    code = (m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    code = torch.where((byte == 255)[..., None], torch.zeros_like(code), code + 8 * torch.signbit(f))
    return code.view(w.shape), byte


def _pack(code):
    """Two codes a byte, the even one in the low half."""
    return (code[:, 0::2] + (code[:, 1::2] << 4)).to(torch.uint8)


def _values(code, byte):
    table = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), device=code.device)
    v = table[code.long()].view(code.shape[0], -1, BLOCK)
    return (v * _power(byte)[..., None]).view(code.shape)


def _unpack(codes):
    c = codes.int()
    return torch.stack((c & 15, c >> 4), -1).view(codes.shape[0], -1)


def _plain_quantise(s):
    code, byte = _quantise(s["w"])
    return {"values": _values(code, byte).to(s["w"].dtype), "scales": byte.to(torch.uint8)}


def _plain_project(s):
    x = s["x"].float()
    M, (L, R, K) = x.shape[0], s["A"].shape
    h = (x @ s["A"].float().view(L * R, K).t()).view(M, L, R)
    mine = s["slots"][:, None] == torch.arange(L, device=x.device)
    h = h * (mine * s["scale"])[..., None]
    y = x @ _values(_unpack(s["codes"]), s["scales"].int()).t()
    y = y + h.view(M, L * R) @ s["B"].float().permute(0, 2, 1).reshape(L * R, -1)
    return {"y": y.to(torch.bfloat16)}


def _softmax(logits, inv_t):
    """(z - max z, exp of it, [row maximum, log of the exps' sum], whether the row has any)."""
    x = logits.float()
    top = x.amax(-1, keepdim=True)
    some = top != -math.inf
    d = (x - torch.where(some, top, torch.zeros_like(top))) * inv_t
    e = torch.exp(d)
    total = e.sum(-1, keepdim=True)
    logsum = torch.where(some, torch.log(total), torch.zeros_like(total))
    return d, e, torch.cat((top, logsum), -1), some


def _entropy(d, e, stats, some):
    mean = torch.where(e > 0, e * d, torch.zeros_like(d)).sum(-1) / torch.where(some, e.sum(-1, keepdim=True), 1.0)[:, 0]
    return stats[:, 1] - mean


def _plain_logprobs(s):
    logits, tokens, k = s["logits"], s["tokens"].long(), s["top"]
    d, e, stats, some = _softmax(logits, s["inv_t"])
    given = torch.gather(d, 1, tokens.clamp(min=0)[:, None])[:, 0] - stats[:, 1]
    out = {"logprob": torch.where(tokens >= 0, given, torch.zeros_like(given)), "entropy": _entropy(d, e, stats, some),
           "stats": stats}
    if k:
        bits = (logits.float() + 0.0).view(torch.int32)
        bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        column = torch.arange(logits.shape[1], device=logits.device)
        ids = 0xFFFFFFFF - (torch.topk((bits << 32) + (0xFFFFFFFF - column), k).values & 0xFFFFFFFF)
        best = torch.gather(d, 1, ids) - stats[:, 1:]
        out["top_logprobs"] = best
        out["top_ids"] = torch.where(best == -math.inf, -1, ids).int()
    return out


def _plain_grad(s):
    x, stats = s["logits"].float(), s["stats"]
    some = stats[:, :1] != -math.inf
    lp = (x - torch.where(some, stats[:, :1], 0.0)) * s["inv_t"] - stats[:, 1:]
    p = torch.exp(lp)
    at = torch.arange(x.shape[1], device=x.device) == s["tokens"][:, None]
    g = torch.where(s["tokens"] >= 0, s["g_logprob"], 0.0)[:, None]
    d = g * (at.float() - p)
    if s["g_entropy"] is not None:
        d = d - torch.where(p > 0, s["g_entropy"][:, None] * p * (lp + s["entropy"][:, None]), 0.0)
    return {"dlogits": torch.where(some, d * s["inv_t"], 0.0).to(s["logits"].dtype)}


# ------------------------------------------------------------------ inputs


def _logits(case, gen):
    """Rows as a model's head gives them: a wide bulk, a few likely tokens, some
    tokens masked in some rows (by -inf, or by the type's lowest value), one row
    of a larger batch masked altogether."""
    M, V, device = case["M"], case["V"], "cuda"
    dtype = torch.float32 if case["f32"] else torch.bfloat16
    buf = torch.empty((M, V + case["pad"]), dtype=dtype, device=device)
    x = buf[:, :V]
    for a in range(0, M, 512):
        b = min(M, a + 512)
        x[a:b] = torch.randn((b - a, V), generator=gen, device=device) * 2.5 - 4.0
    likely = torch.randint(V, (M, 8), generator=gen, device=device)
    x.scatter_(1, likely, (torch.randn((M, 8), generator=gen, device=device) * 3.0 + 9.0).to(dtype))
    tokens = torch.where(torch.rand(M, generator=gen, device=device) < 0.6, likely[:, 0],
                         torch.randint(V, (M,), generator=gen, device=device))
    hidden = torch.rand(V, generator=gen, device=device) < 0.5
    x[3::7] = torch.where(hidden, -math.inf, x[3::7].float()).to(dtype)
    x[4::11] = torch.where(hidden, torch.finfo(dtype).min, x[4::11].float()).to(dtype)
    x[4::11].scatter_(1, likely[4::11], 9.0)  # what is asked for there is not masked
    tokens[4::11] = likely[4::11, 0]
    if M > 16:
        x[5] = -math.inf
        tokens[6::16] = -1  # padding
    return x, tokens.int()


def _routes(case, s):
    """The packed adapter pool that a server keeps."""
    import rank_delta_gb300 as rd
    from rank_delta_gb300 import torch_helpers as th
    route = th.DeviceRoute(case["L"], case["R"], case["K"], case["N"])
    for slot, r in enumerate(s["ranks"]):
        rd.lora_pool_pack(route.rt, slot, s["A"][slot, :r].contiguous(), s["B"][slot, :, :r].contiguous(), r, 16.0,
                          False, 1.0)
    return route, th.workspace(rd.lora_mx4_proj_workspace_bytes(case["M"], route.rt))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"op": case["op"]}
    if case["op"] == "quantise":
        rows, K, dtype = case["rows"], case["K"], torch.float32 if case["f32"] else torch.bfloat16
        buf = torch.zeros((rows, K + case["pad"]), dtype=dtype, device="cuda")
        w = buf[:, :K]
        w.copy_(torch.randn((rows, K), generator=gen, device="cuda") / math.sqrt(K))
        w[1::64, :BLOCK] = 0  # blocks of zeros
        w[2::64] *= 2.0 ** 20  # rows of another size
        w[3::64] *= 2.0 ** -110
        s.update(w=w, rows=rows, K=K, codes=torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda"),
                 scales=torch.empty((rows, K // BLOCK), dtype=torch.uint8, device="cuda"),
                 back=torch.empty((rows, K), dtype=dtype, device="cuda"))
        return s
    if case["op"] == "project":
        M, K, N, L, R = (case[k] for k in "MKNLR")
        rand = lambda *n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
        code, byte = _quantise(rand(N, K) / math.sqrt(K))
        ranks = [R if i % 2 == 0 else max(1, R // 2) for i in range(L)]
        kept = (torch.arange(R) < torch.tensor(ranks)[:, None]).float().cuda()
        s.update(M=M, K=K, N=N, codes=_pack(code), scales=byte.to(torch.uint8), x=rand(M, K).to(torch.bfloat16), ranks=ranks,
                 A=(rand(L, R, K) / math.sqrt(K) * kept[:, :, None]).to(torch.bfloat16),
                 B=(rand(L, N, R) * 0.1 * kept[:, None, :]).to(torch.bfloat16),
                 scale=torch.tensor([16.0] * L, device="cuda") / torch.tensor(ranks, dtype=torch.float32, device="cuda"),
                 y=torch.empty((M, N), dtype=torch.bfloat16, device="cuda"))
        if M >= 1024:  # prompts: runs of rows with one adapter
            slots = (torch.arange(M, device="cuda") * L) // M
        else:
            slots = torch.randint(-1 if M > 1 else 0, L, (M,), generator=gen, device="cuda")
        s["slots"] = slots.int()
        if own:  # the route and the workspace belong to the program, as the weights do
            s["route"], s["ws"] = _routes(case, s)
        return s
    s["logits"], s["tokens"] = _logits(case, gen)
    s.update(M=case["M"], V=case["V"], inv_t=case["inv_t"], stride=case["V"] + case["pad"])
    M = case["M"]
    if case["op"] == "logprobs":
        s["top"] = case["top"]
        s.update(logprob=torch.empty(M, device="cuda"), entropy=torch.empty(M, device="cuda"),
                 stats=torch.empty((M, 2), device="cuda"), ws=torch.empty(256, dtype=torch.uint8, device="cuda"),
                 top_ids=torch.empty((M, s["top"]), dtype=torch.int32, device="cuda"),
                 top_logprobs=torch.empty((M, s["top"]), device="cuda"))
        return s
    stats, entropy = [], []
    for a in range(0, M, 1024):  # what the forward pass left
        d, e, st, some = _softmax(s["logits"][a:a + 1024], case["inv_t"])
        stats.append(st)
        entropy.append(_entropy(d, e, st, some))
    s["stats"], s["entropy"] = torch.cat(stats), torch.cat(entropy)
    s["g_logprob"] = -torch.rand(M, generator=gen, device="cuda") - 0.1
    s["g_entropy"] = torch.randn(M, generator=gen, device="cuda") * 0.05 if case["bonus"] else None
    s["dlogits"] = torch.empty((M, case["V"]), dtype=s["logits"].dtype, device="cuda")
    return s


def run(s):
    if not own:
        return {"quantise": _plain_quantise, "project": _plain_project, "logprobs": _plain_logprobs,
                "grad": _plain_grad}[s["op"]](s)
    import rank_delta_gb300 as rd
    stream = torch.cuda.current_stream()
    if s["op"] == "quantise":
        w, back = s["w"], s["back"]
        dtype = rd.LORA_DTYPE_F32 if w.dtype == torch.float32 else rd.LORA_DTYPE_BF16
        rd.lora_mx4_quantize(w, dtype, w.stride(0), s["rows"], s["K"], s["codes"], s["scales"], stream)
        rd.lora_mx4_dequantize(s["codes"], s["scales"], s["rows"], s["K"], back, dtype, back.stride(0), stream)
        return {"values": back, "scales": s["scales"]}
    if s["op"] == "project":
        x, y, ws = s["x"], s["y"], s["ws"]
        rd.lora_mx4_proj_apply(x, x.stride(0), s["codes"], s["scales"], s["M"], s["K"], s["N"], s["slots"], s["route"].rt,
                               y, y.stride(0), ws, ws.numel(), stream)
        return {"y": y}
    logits = s["logits"]
    dtype = rd.LORA_DTYPE_F32 if logits.dtype == torch.float32 else rd.LORA_DTYPE_BF16
    if s["op"] == "logprobs":
        top = s["top"]
        rd.lora_logprobs(logits, dtype, s["stride"], s["M"], s["V"], s["tokens"], s["inv_t"], top, s["logprob"],
                         s["entropy"], s["stats"], s["top_ids"], s["top_logprobs"], s["ws"], 256, stream)
        out = {"logprob": s["logprob"], "entropy": s["entropy"], "stats": s["stats"]}
        return dict(out, top_logprobs=s["top_logprobs"], top_ids=s["top_ids"]) if top else out
    rd.lora_logprobs_grad(logits, dtype, s["stride"], s["M"], s["V"], s["tokens"], s["inv_t"], s["stats"], s["entropy"],
                          s["g_logprob"], s["g_entropy"], s["dlogits"], s["V"], stream)
    return {"dlogits": s["dlogits"]}


# ------------------------------------------------------------------ 64 bits


def _exact_matrix(codes, scales):
    """Each nibble's value from its own sign, exponent and mantissa bits."""
    c = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        n = ((codes >> (4 * half)) & 15).double()
        sign = 1.0 - 2.0 * (n >= 8).double()
        n = n - 8.0 * (n >= 8).double()
        e = torch.floor(n / 2)
        c[:, half::2] = sign * torch.where(e > 0, (1 + (n - 2 * e) / 2) * torch.exp2(e - 1), n / 2)
    return c * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        w = s["w"].double().view(case["rows"], -1, BLOCK)
        out = torch.empty_like(w)
        for a in range(0, w.shape[0], 2048):
            b = w[a:a + 2048]
            e = torch.floor(torch.log2(b.abs().amax(-1, keepdim=True))).clamp(min=-125.0) - 2
            m = b / torch.exp2(e)
            step = torch.exp2(torch.floor(torch.log2(m.abs().clamp(min=1.0))) - 1)
            out[a:a + 2048] = (torch.round(m / step) * step).clamp(-6, 6) * torch.exp2(e)
        return {"values": out.view(case["rows"], -1), "scales": None}
    if case["op"] == "project":
        x, slots = s["x"].double(), s["slots"]
        y = x @ _exact_matrix(s["codes"], s["scales"]).t()
        for slot, r in enumerate(s["ranks"]):
            rows = torch.nonzero(slots == slot)[:, 0]
            h = x[rows] @ s["A"][slot, :r].double().t()
            y[rows] += 16.0 / r * (h @ s["B"][slot, :, :r].double().t())
        return {"y": y}
    M, V, inv_t, lowest = case["M"], case["V"], case["inv_t"], -math.inf
    parts = []
    for a in range(0, M, 1024):
        x = s["logits"][a:a + 1024].double()
        t = s["tokens"][a:a + 1024].long()
        row = torch.arange(x.shape[0], device=x.device)
        top = x.max(-1).values
        empty = top == lowest
        z = (x - torch.where(empty, 0.0, top)[:, None]) * inv_t
        logsum = torch.where(empty, 0.0, torch.logsumexp(z, -1))
        lp = z - logsum[:, None]
        p = lp.exp()
        H = -torch.where(p > 0, p * lp, 0.0).sum(-1)
        if case["op"] == "logprobs":
            d = {"logprob": torch.where(t >= 0, lp[row, t.clamp(min=0)], 0.0), "entropy": H,
                 "stats": torch.stack((top, logsum), -1)}
            if case["top"]:
                d["top_logprobs"] = torch.sort(lp, -1, descending=True).values[:, :case["top"]]
                d["top_ids"] = None
        else:
            st, H = s["stats"][a:a + 1024].double(), s["entropy"][a:a + 1024].double()
            lp = (x - torch.where(empty, 0.0, st[:, 0])[:, None]) * inv_t - st[:, 1:]
            p = lp.exp()
            g = s["g_logprob"][a:a + 1024].double() * (t >= 0)
            dz = -g[:, None] * p
            dz[row, t.clamp(min=0)] += g
            if s["g_entropy"] is not None:
                dz -= torch.where(p > 0, p * (lp + H[:, None]), 0.0) * s["g_entropy"][a:a + 1024].double()[:, None]
            dz[empty] = 0.0
            d = {"dlogits": dz * inv_t}
        parts.append(d)
    return {k: None if parts[0][k] is None else torch.cat([p[k] for p in parts]) for k in parts[0]}
