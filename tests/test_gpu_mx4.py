"""Microscaled 4-bit matrices: quantisation and reading back against the
format's definition (equal, code for code), and the projection with such a
base against 64-bit sums.

Tolerance of the projection, an element before its rounding: the fp32
accumulation, whose partial sums follow one another at most K / 16 + 64 deep,
(K / 16 + 64) 2^-24 times the sum of the absolute products; and for the
adapter the same over its own two sums, plus 2^-8 of the expand's absolute
products for the paths that round s h to bf16. The result's own rounding has
no tolerance: it has to lie between the roundings of the two ends."""
import numpy as np
import pytest
import torch

import rank_delta_gb300 as rd
from rank_delta_gb300 import build as rdbuild
from rank_delta_gb300 import torch_helpers as th

pytestmark = pytest.mark.gpu

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
PATHS = [rd.LORA_MX4_PATH_ROWS, rd.LORA_MX4_PATH_TILES]


@pytest.fixture(scope="module", autouse=True)
def lib():
    rdbuild.build()
    assert torch.cuda.is_available()
    return rd.lib()


def tag(dtype):
    return rd.LORA_DTYPE_F32 if dtype == torch.float32 else rd.LORA_DTYPE_BF16


def define(w):
    """(codes [rows][K], scale bytes [rows][K/32]) of float64 values, from the definition."""
    b = w.reshape(w.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    m = np.where(bad, 1.0, np.abs(b).max(-1))
    e = np.full(m.shape, -10000)
    e[m > 0] = np.frexp(m[m > 0])[1] - 1
    byte = np.where(bad, 255, np.where(m == 0, 0, np.maximum(e - 2 + 127, 0)))
    v = np.abs(np.where(bad[..., None], 0.0, b)) / np.exp2(np.where(bad, 127, byte) - 127.0)[..., None]
    d = np.abs(np.minimum(v, 6.0)[..., None] - GRID)
    near = d == d.min(-1, keepdims=True)  # ties: the even code
    code = np.where(near[..., ::2].any(-1), 2 * near[..., ::2].argmax(-1), near.argmax(-1))
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(b))
    return code.reshape(w.shape).astype(np.uint8), byte.astype(np.uint8)


def values(code, byte):
    v = np.where(code >= 8, -1.0, 1.0) * GRID[code & 7]
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)


def quantise(w):
    rows, K = w.shape
    codes = torch.full((rows, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, K // 32), 0xEE, dtype=torch.uint8, device="cuda")
    assert codes.numel() == rd.lora_mx4_code_bytes(rows, K) and scales.numel() == rd.lora_mx4_scale_bytes(rows, K)
    rd.lora_mx4_quantize(w, tag(w.dtype), w.stride(0), rows, K, codes, scales, torch.cuda.current_stream())
    return codes, scales


def nibbles(codes):
    c = codes.cpu().numpy()
    return np.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K,pad,lead", [(1, 32, 0, 0), (3, 64, 0, 1), (5, 96, 3, 0), (33, 1056, 8, 0), (700, 4096, 0, 0),
                                             (17, 8192, 1, 3)])
def test_quantise_is_the_definition(dtype, rows, K, pad, lead):
    rng = np.random.default_rng(rows + K)
    w = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-20, 20, (rows, K // 32))).repeat(32, axis=1)
    buf = torch.zeros(lead + rows * (K + pad), dtype=dtype, device="cuda")
    t = buf[lead:].view(rows, K + pad)[:, :K]
    t.copy_(torch.tensor(w))
    codes, scales = quantise(t)
    want, byte = define(t.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), byte)
    assert np.array_equal(nibbles(codes), want)
    back = torch.zeros(lead + rows * (K + pad), dtype=dtype, device="cuda")
    b = back[lead:].view(rows, K + pad)[:, :K]
    rd.lora_mx4_dequantize(codes, scales, rows, K, b, tag(dtype), b.stride(0))
    torch.cuda.synchronize()
    assert np.array_equal(b.double().cpu().numpy(), values(want, byte))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantise_edges(dtype):
    """Zeros, ties at every midpoint, block maxima just below and at powers of
    two, subnormals, the type's largest value, infinities and NaN."""
    rows = torch.zeros(12, 64, dtype=torch.float64)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.0, 4.0])
    for r, s in ((1, 1.0), (2, 2.0 ** -30), (3, 2.0 ** 60)):
        rows[r, :10] = mid * s
        rows[r, 32:42] = -mid * s
    big, tiny = float(torch.finfo(dtype).max), 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149
    rows[4, :3] = torch.tensor([big, -big, big / 2])
    rows[5, :4] = torch.tensor([tiny, -tiny, 3 * tiny, 2.0 ** -127])
    rows[6, :3] = torch.tensor([2.0 ** -126, 2.0 ** -125, -(2.0 ** -124)])
    rows[7, 3] = float("inf")
    rows[8, 40] = float("nan")
    rows[9, :2] = torch.tensor([-0.0, -1e-30])
    rows[9, 31] = 1.0
    rows[10, :2] = torch.tensor([1.9921875, 0.1])
    rows[11, :2] = torch.tensor([2.0, 0.1])
    t = rows.to(dtype).cuda()
    codes, scales = quantise(t)
    want, byte = define(t.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), byte)
    assert np.array_equal(nibbles(codes), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_reading_back_every_code_and_scale(dtype):
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    byte = np.arange(256, dtype=np.uint8)[:, None]
    packed = torch.tensor(code[:, 0::2] | code[:, 1::2] << 4).cuda()
    out = torch.zeros(256, 32, dtype=dtype, device="cuda")
    rd.lora_mx4_dequantize(packed, torch.tensor(byte).cuda(), 256, 32, out, tag(dtype), 32)
    torch.cuda.synchronize()
    want = torch.tensor(values(code, byte)).to(torch.float32).to(dtype)  # past the type's range: infinity
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(out.cpu().float(), 0.0), torch.nan_to_num(want.float(), 0.0))


# -------------------------------------------------------------- projection


class Setup:
    def __init__(self, M, K, N, L, R, seed, x_pad=0):
        rng = np.random.default_rng(seed)
        self.M, self.K, self.N, self.L, self.R = M, K, N, L, R
        bf = lambda a: torch.tensor(a).to(torch.bfloat16).cuda()  # noqa: E731
        self.x = bf(rng.standard_normal((M, K + x_pad)))[:, :K]
        w = torch.tensor(rng.standard_normal((N, K)) / np.sqrt(K)).float().cuda()
        self.codes, self.scales = quantise(w)
        self.route = th.DeviceRoute(L, R, K, N)
        self.delta = []  # (A, B, s) of each slot, or None
        for s in range(L):
            if s == 1 and L > 2:
                self.delta.append(None)  # an empty slot
                continue
            r = max(1, R - s)
            A, B = bf(rng.standard_normal((r, K)) / np.sqrt(K)), bf(rng.standard_normal((N, r)) * 0.2)
            scale = 0.0 if s == 2 and L > 4 else 1.0 + s % 3
            rd.lora_pool_pack(self.route.rt, s, A, B, r, 0.0, False, scale)
            self.delta.append((A.double().cpu().numpy(), B.double().cpu().numpy(), scale))
        self.slots = rng.integers(-1, L, M).astype(np.int32)

    def run(self, path, slots=None, y_pad=0, stream=None):
        slots = torch.tensor(self.slots if slots is None else slots).cuda()
        y = torch.full((self.M, self.N + y_pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        ws = torch.full((rd.lora_mx4_proj_workspace_bytes(self.M, self.route.rt),), 0x5A, dtype=torch.uint8,
                        device="cuda")
        rd.lora_mx4_proj_apply(self.x, self.x.stride(0), self.codes, self.scales, self.M, self.K, self.N, slots,
                               self.route.rt, y, y.stride(0), ws, ws.numel(), stream, path)
        torch.cuda.synchronize()
        self.flags = rd.lora_status_get(ws)
        assert bool(torch.isnan(y[:, self.N:]).all()), "written past a row"
        return y[:, :self.N]

    def check(self, y, slots=None):
        slots = self.slots if slots is None else slots
        x = self.x.double().cpu().numpy()
        W = values(nibbles(self.codes), self.scales.cpu().numpy())
        want, big = x @ W.T, np.abs(x) @ np.abs(W).T
        deep = lambda n: (n / 16 + 64) * 2.0 ** -24  # noqa: E731
        tol = deep(self.K) * big
        for s, d in enumerate(self.delta):
            rows = np.nonzero(slots == s)[0]
            if d is None or not len(rows):
                continue
            A, B, scale = d
            h = x[rows] @ A.T
            want[rows] += scale * (h @ B.T)
            hb = np.abs(x[rows]) @ np.abs(A).T
            tol[rows] += scale * ((2.0 ** -8 + deep(self.R)) * np.abs(h) @ np.abs(B).T + deep(self.K) * hb @ np.abs(B).T)
        got = y.double().cpu().numpy()
        ends = [torch.tensor(v).to(torch.float32).to(torch.bfloat16).double().numpy() for v in (want - tol, want + tol)]
        bad = ~((ends[0] <= got) & (got <= ends[1]))
        assert not bad.any(), (np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], tol[bad][:4], int(bad.sum()))


SHAPES = [  # M, K, N, L, R
    (1, 32, 1, 1, 8), (1, 96, 17, 2, 8), (2, 256, 256, 4, 16), (8, 4096, 130, 3, 64), (9, 1056, 257, 4, 24),
    (16, 8224, 48, 5, 8), (17, 160, 500, 6, 40), (33, 2080, 129, 16, 64), (64, 4096, 384, 8, 32), (65, 544, 300, 4, 16),
    (200, 1024, 640, 6, 64), (1, 20000, 64, 2, 16), (300, 4096, 257, 3, 8), (64, 12288, 128, 4, 128)]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("M,K,N,L,R", SHAPES)
def test_projection_against_64_bits(path, M, K, N, L, R):
    s = Setup(M, K, N, L, R, seed=M + K + N, x_pad=8 * (M % 3))
    s.check(s.run(path, y_pad=M % 2))
    assert s.flags == 0


@pytest.mark.parametrize("M", [1, 5, 40, 130])
def test_auto_takes_every_row_count(M):
    s = Setup(M, 512, 200, 4, 16, seed=M)
    s.check(s.run(rd.LORA_MX4_PATH_AUTO))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("M", [6, 70])
def test_rows_without_a_delta_are_the_base_product_byte_for_byte(path, M):
    s = Setup(M, 1056, 300, 6, 16, seed=3)
    slots = np.arange(M, dtype=np.int32) % 8 - 1  # -1, 0, 1 (empty), 2 (scale 0), 3, 4, 5, 6 (out of range)
    base = s.run(path, np.full(M, -1, np.int32))
    y = s.run(path, slots)
    assert s.flags == (rd.LORA_FLAG_SLOT_RANGE if (slots >= 6).any() else 0)
    s.check(y, slots)
    off = torch.tensor(np.isin(slots, (-1, 1, 2, 6))).cuda()
    assert torch.equal(y[off].view(torch.int16), base[off].view(torch.int16))


@pytest.mark.parametrize("path", PATHS)
def test_stack_of_adapters_in_a_slot(path):
    s = Setup(20, 512, 160, 1, 32, seed=5)
    rng = np.random.default_rng(9)
    bf = lambda a: torch.tensor(a).to(torch.bfloat16).cuda()  # noqa: E731
    A = [bf(rng.standard_normal((r, 512)) / 22) for r in (8, 5)]
    B = [bf(rng.standard_normal((160, r)) * 0.2) for r in (8, 5)]
    rd.lora_pool_pack_stack(s.route.rt, 0, A, B, [8, 5], [0.0, 0.0], [False, False], [2.0, -0.5])
    s.delta[0] = (torch.cat(A).double().cpu().numpy(),
                  torch.cat((2.0 * B[0].double(), -0.5 * B[1].double()), 1).cpu().numpy(), 1.0)
    s.check(s.run(path))


@pytest.mark.parametrize("path", PATHS)
def test_scales_at_the_ends_of_their_range(path):
    """Blocks scaled by 2^20 and beyond, tiny ones, and a NaN block: the widened weight is exact bf16."""
    s = Setup(3, 128, 64, 1, 8, seed=11)
    s.scales[:8] = 127 + 20
    s.scales[8:16] = 127 + 60
    s.scales[16:24] = 1
    s.scales[24:32] = 0
    s.slots[:] = -1
    y = s.run(path)
    s.check(y)
    s.scales[40, 1] = 255
    y = s.run(path)
    assert bool(torch.isnan(y[:, 40]).all()) and bool(torch.isfinite(y[:, 41]).all())


@pytest.mark.parametrize("path", PATHS)
def test_same_bytes_on_every_run_and_on_another_stream(path):
    s = Setup(48, 4096, 520, 8, 32, seed=7)
    a, b = s.run(path), s.run(path)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = s.run(path, stream=side)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(a.view(torch.int16), c.view(torch.int16))


# More slots than a chunk of rows has, ranks that end inside a segment of 16, one slot with every row, every
# adapter in a tile, several parts of K with a tail, one and two tiles of rows.
LARGER = [
    (48, 512, 150, 80, 16), (40, 384, 130, 200, 8), (230, 1024, 300, 1, 64), (130, 768, 260, 40, 40), (20, 512, 128, 20, 256),
    (256, 4224, 300, 32, 64), (150, 4096, 1100, 16, 24), (256, 2048, 2048, 8, 16), (64, 4096, 520, 16, 56), (192, 1056, 130, 64, 64),
    (300, 800, 200, 24, 72)]


@pytest.mark.parametrize("M,K,N,L,R", LARGER)
def test_many_adapters_and_large_ranks(M, K, N, L, R):
    s = Setup(M, K, N, L, R, seed=M + R)
    s.check(s.run(rd.LORA_MX4_PATH_TILES, y_pad=8 * (M % 2)))
    assert s.flags == 0


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("M", [3, 40, 150])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_an_adapter_that_is_not_finite_stays_with_its_rows(path, M, value):
    """Slot 0 with such values in A and in B: rows of the other slots get what they should, those of none the same bytes."""
    s = Setup(M, 1024, 300, 4, 24, seed=M)
    slots = np.arange(M, dtype=np.int32) % 5 - 1  # -1 .. 3
    clean = s.run(path, slots)
    rng = np.random.default_rng(1)
    bf = lambda a: torch.tensor(a).to(torch.bfloat16).cuda()  # noqa: E731
    A, B = bf(rng.standard_normal((24, 1024)) / 32), bf(rng.standard_normal((300, 24)))
    A[3, 5] = value
    B[7, 2] = B[299, 23] = value
    rd.lora_pool_pack(s.route.rt, 0, A, B, 24, 0.0, False, 1.0)
    y = s.run(path, slots)
    own = torch.tensor(slots == 0).cuda()
    assert not bool(torch.isfinite(y[own].float()).any())
    s.check(torch.where(own[:, None], clean, y), slots)
    none = torch.tensor(slots == -1).cuda()
    assert torch.equal(y[none].view(torch.int16), clean[none].view(torch.int16))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("M", [2, 70])
def test_bases_that_no_tile_load_takes(path, M):
    """Scales on an odd address, a base of y that is 2 bytes off, K with a tail."""
    s = Setup(M, 2080, 200, 4, 16, seed=M)
    odd = torch.empty(s.scales.numel() + 1, dtype=torch.uint8, device="cuda")[1:].view_as(s.scales)
    odd.copy_(s.scales)
    s.scales = odd
    s.check(s.run(path, y_pad=3))


@pytest.mark.parametrize("M", [1, 64, 200])
def test_replayed_from_a_graph(M):
    s = Setup(M, 1024, 384, 8, 32, seed=M)
    want = s.run(rd.LORA_MX4_PATH_AUTO)
    y = torch.empty(M, 384, dtype=torch.bfloat16, device="cuda")
    ws = th.workspace(rd.lora_mx4_proj_workspace_bytes(M, s.route.rt))
    slots = torch.tensor(s.slots).cuda()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(2):
            rd.lora_mx4_proj_apply(s.x, s.x.stride(0), s.codes, s.scales, M, 1024, 384, slots, s.route.rt, y, 384, ws, ws.numel(),
                                   torch.cuda.current_stream())
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("M,K,N,L,R,runs", [(2048, 288, 40, 5, 64, True), (2050, 320, 24, 300, 24, False), (2500, 96, 72, 2, 136, True),
                                            (2304, 2080, 16, 24, 32, False)])
def test_calls_of_thousands_of_rows(M, K, N, L, R, runs):
    """Slots in runs as prefill has them, and rows of any slot; chunks with more slots than CTAs, a last chunk that ends early."""
    s = Setup(M, K, N, L, R, seed=M)
    if runs:
        s.slots = np.repeat(np.arange(-1, L, dtype=np.int32), -(-M // (L + 1)))[:M].copy()
    s.check(s.run(rd.LORA_MX4_PATH_AUTO))
    assert s.flags == 0
