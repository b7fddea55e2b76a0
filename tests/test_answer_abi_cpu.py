"""Argument checks of the calls at the answering end: refused on the host, before any CUDA call."""
import math

import pytest

import rank_delta_gb300 as rd
from rank_delta_gb300 import build as rdbuild
from tests.test_abi_cpu import expect


@pytest.fixture(scope="module", autouse=True)
def built():
    rdbuild.build()
    return rd.lib()


def test_logprobs_refusals():
    good = dict(logits=4096, dtype=rd.LORA_DTYPE_BF16, stride=100, M=4, V=100, tokens=256, inv_t=1.0, k=3, logprob=256,
                entropy=256, stats=256, ids=256, lps=256, ws=512, n=256)

    def call(**kw):
        a = dict(good, **kw)
        return lambda: rd.lora_logprobs(a["logits"], a["dtype"], a["stride"], a["M"], a["V"], a["tokens"], a["inv_t"], a["k"],
                                        a["logprob"], a["entropy"], a["stats"], a["ids"], a["lps"], a["ws"], a["n"])

    assert rd.lora_logprobs_workspace_bytes(4, 100, 3) == 256
    expect(rd.LORA_ERR_RANGE, call(dtype=2), contains=("dtype 2",))
    expect(rd.LORA_ERR_SHAPE, call(M=-1), contains=("M -1",))
    expect(rd.LORA_ERR_SHAPE, call(V=0))
    expect(rd.LORA_ERR_SHAPE, call(stride=99), contains=("stride 99", "V 100"))
    for t in (0.0, -1.0, math.inf, math.nan):
        expect(rd.LORA_ERR_RANGE, call(inv_t=t), contains=("inv_temperature",))
    expect(rd.LORA_ERR_RANGE, call(k=33), contains=("top_k 33", "32"))
    expect(rd.LORA_ERR_RANGE, call(k=-1))
    expect(rd.LORA_ERR_RANGE, call(k=20, V=10), contains=("top_k 20", "10"))
    expect(rd.LORA_ERR_NULL, call(logits=0))
    expect(rd.LORA_ERR_NULL, call(ids=0))
    expect(rd.LORA_ERR_NULL, call(lps=0))
    expect(rd.LORA_ERR_NULL, call(tokens=0), contains=("tokens",))
    expect(rd.LORA_ERR_NULL, call(ws=0))
    expect(rd.LORA_ERR_ALIGN, call(ws=520))
    expect(rd.LORA_ERR_ALIGN, call(logits=4097))
    expect(rd.LORA_ERR_ALIGN, call(logits=4098, dtype=rd.LORA_DTYPE_F32))
    expect(rd.LORA_ERR_WORKSPACE, call(n=128), contains=("128", "256"))
    expect(rd.LORA_ERR_UNSUPPORTED, call(V=(1 << 30) + 1, stride=1 << 31))
    call(M=0, logits=0, ws=0, n=0)()


def test_logprobs_grad_refusals():
    good = dict(logits=4096, dtype=rd.LORA_DTYPE_F32, stride=100, M=4, V=100, tokens=256, inv_t=1.0, stats=256, entropy=256,
                g=256, h=256, d=8192, ds=100)

    def call(**kw):
        a = dict(good, **kw)
        return lambda: rd.lora_logprobs_grad(a["logits"], a["dtype"], a["stride"], a["M"], a["V"], a["tokens"], a["inv_t"],
                                             a["stats"], a["entropy"], a["g"], a["h"], a["d"], a["ds"])

    expect(rd.LORA_ERR_RANGE, call(dtype=7))
    expect(rd.LORA_ERR_SHAPE, call(ds=99), contains=("d_stride 99",))
    expect(rd.LORA_ERR_SHAPE, call(stride=50))
    expect(rd.LORA_ERR_SHAPE, call(d=4096, ds=101), contains=("same stride",))
    expect(rd.LORA_ERR_NULL, call(stats=0))
    expect(rd.LORA_ERR_NULL, call(d=0))
    expect(rd.LORA_ERR_NULL, call(g=0, h=0), contains=("neither",))
    expect(rd.LORA_ERR_NULL, call(tokens=0), contains=("tokens",))
    expect(rd.LORA_ERR_NULL, call(entropy=0), contains=("entropy",))
    expect(rd.LORA_ERR_ALIGN, call(d=8194))
    expect(rd.LORA_ERR_RANGE, call(inv_t=0.0))
    call(M=0)()


def test_mx4_sizes_and_refusals():
    assert rd.lora_mx4_code_bytes(10, 64) == 320 and rd.lora_mx4_scale_bytes(10, 64) == 20
    assert rd.lora_mx4_code_bytes(10, 65) == 0 and rd.lora_mx4_scale_bytes(0, 64) == 0
    assert rd.lora_mx4_code_bytes(1 << 32, 64) == 32 << 32
    good = dict(w=4096, dtype=rd.LORA_DTYPE_BF16, stride=64, rows=4, K=64, codes=512, scales=77)

    def quant(**kw):
        a = dict(good, **kw)
        return lambda: rd.lora_mx4_quantize(a["w"], a["dtype"], a["stride"], a["rows"], a["K"], a["codes"], a["scales"])

    def back(**kw):
        a = dict(good, **kw)
        return lambda: rd.lora_mx4_dequantize(a["codes"], a["scales"], a["rows"], a["K"], a["w"], a["dtype"], a["stride"])

    for call in (quant, back):
        expect(rd.LORA_ERR_RANGE, call(dtype=3), contains=("dtype 3",))
        expect(rd.LORA_ERR_SHAPE, call(rows=-1))
        for K in (0, 16, 40):
            expect(rd.LORA_ERR_SHAPE, call(K=K), contains=(f"K {K}", "32"))
        expect(rd.LORA_ERR_SHAPE, call(stride=63), contains=("w_stride 63",))
        for name in ("w", "codes", "scales"):
            expect(rd.LORA_ERR_NULL, call(**{name: 0}))
        expect(rd.LORA_ERR_ALIGN, call(codes=520))
        expect(rd.LORA_ERR_ALIGN, call(w=4097))
        expect(rd.LORA_ERR_ALIGN, call(w=4098, dtype=rd.LORA_DTYPE_F32))
        expect(rd.LORA_ERR_UNSUPPORTED, call(rows=1 << 60), contains=("K 64",))
        call(rows=0, w=0, codes=0, scales=0)()


def test_mx4_projection_refusals():
    from tests.test_abi_cpu import fake_route
    rt = fake_route(L=4, R=8, K=256, N=256)
    need = rd.lora_mx4_proj_workspace_bytes(8, rt)
    assert need > 0
    assert rd.lora_mx4_proj_workspace_bytes(8, fake_route(kind=rd.LORA_ROUTE_EMBED)) == 0
    good = dict(x=4096, xs=256, codes=8192, scales=513, M=8, K=256, N=256, slots=4096, rt=rt, y=4096, ys=256, ws=1 << 20,
                n=need, path=0)

    def call(**kw):
        a = dict(good, **kw)
        return lambda: rd.lora_mx4_proj_apply(a["x"], a["xs"], a["codes"], a["scales"], a["M"], a["K"], a["N"], a["slots"],
                                              a["rt"], a["y"], a["ys"], a["ws"], a["n"], None, a["path"])

    expect(rd.LORA_ERR_NOT_INIT, call(rt=rd.lora_route()))
    expect(rd.LORA_ERR_UNSUPPORTED, call(rt=fake_route(kind=rd.LORA_ROUTE_EMBED)))
    expect(rd.LORA_ERR_SHAPE, call(M=-1))
    expect(rd.LORA_ERR_RANGE, call(path=9), contains=("path 9",))
    expect(rd.LORA_ERR_SHAPE, call(K=512), contains=("K 512", "n_in 256"))
    expect(rd.LORA_ERR_SHAPE, call(rt=fake_route(K=264), K=264, xs=264), contains=("K 264", "32"))
    for name in ("codes", "scales", "x", "slots", "y", "ws"):
        expect(rd.LORA_ERR_NULL, call(**{name: 0}))
    expect(rd.LORA_ERR_ALIGN, call(codes=8200))
    expect(rd.LORA_ERR_ALIGN, call(x=4098))
    expect(rd.LORA_ERR_ALIGN, call(xs=260))
    expect(rd.LORA_ERR_SHAPE, call(ys=255))
    expect(rd.LORA_ERR_ALIGN, call(ws=(1 << 20) + 16))
    expect(rd.LORA_ERR_WORKSPACE, call(n=need - 1), contains=(str(need), str(need - 1)))
    call(M=0, x=0, codes=0, ws=0, n=0)()
