// Microscaled 4-bit matrices: quantisation, reading back, and the projection
//   y[i, :] = dq(W) x_i + s B_s (A_s x_i)
// with the base W in that form and each row's adapter in bf16.
//
// quantize   a thread takes a block: its scale is 2^(floor(log2 max) - 2), read
//            off the exponent field, so the largest code is 4 or 6; codes are
//            rounded to nearest even and saturate.
// dequantize the reverse, eight values a thread and step.
// shrink     h = A_s x_i for the rows of each slot, on the tensor cores straight
//            from memory: 16 rank rows by up to 32 of the slot's rows a CTA and
//            pass (64 rows, 16 slots of rank 64, K = 4096: 6.4 us, latency); for
//            thousands of rows 64 by 64 through shared memory. The projection
//            kernels start behind it at once and wait for h only where they need
//            it.
// rows       the product for up to four rows, on the tensor cores' registers
//            (mma.sync): a warp's 16 weight rows need not pass through shared
//            memory a second time once they are widened.
#include <algorithm>

#include "behind.cuh"
#include "lora_mx4.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace rd {

namespace {

constexpr int Q_THREADS = 256;
constexpr int Q_UNROLL = 4;

__device__ __forceinline__ float absmax_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

// Two fp32 values to E2M1 codes, `lo` in the low half of the byte.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi)
{
    uint16_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u16.u8 %0, t;\n\t}"
        : "=h"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// Eight elements from p; `vec`: p is 16-byte aligned.
__device__ __forceinline__ void load8(const uint16_t *p, bool vec, float (&f)[8])
{
    if (vec) {
        const uint4 q = ld_nc_16(p);
        f[0] = bf_lo(q.x); f[1] = bf_hi(q.x); f[2] = bf_lo(q.y); f[3] = bf_hi(q.y);
        f[4] = bf_lo(q.z); f[5] = bf_hi(q.z); f[6] = bf_lo(q.w); f[7] = bf_hi(q.w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = __uint_as_float((uint32_t)p[i] << 16);
    }
}
__device__ __forceinline__ void load8(const float *p, bool vec, float (&f)[8])
{
    if (vec) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = p[i];
    }
}

// Element offset of unit u (8 values) of a matrix of K / 8 = upr units a row.
__device__ __forceinline__ int64_t unit_offset(int64_t u, int upr, int64_t stride, bool packed)
{
    if (packed)
        return u * 8;
    const int64_t row = u / upr;
    return row * stride + (u - row * upr) * 8;
}

} // namespace

namespace {

// The scale byte of a block whose largest magnitude has exponent field e (255:
// the block holds an infinity or a NaN).
__device__ __forceinline__ uint32_t scale_byte(uint32_t e) { return e == 255u ? 255u : (e > 2u ? e - 2u : 0u); }

// Eight values, scaled by 2^(127 - byte), to codes.
__device__ __forceinline__ uint32_t codes8(const float (&f)[8], uint32_t byte)
{
    const float up = __uint_as_float((254u - (byte < 254u ? byte : 253u)) << 23);
    uint32_t c = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c |= e2m1_pair(f[2 * i] * up, f[2 * i + 1] * up) << (8 * i);
    return byte == 255u ? 0u : c;
}

// A block of 32 values in bf16 pairs -> its codes and scale byte. Magnitudes
// are compared as integers (a NaN is the largest), scaling is an addition to
// their exponents, and what the exponent has left fits fp16, whose pairs
// convert in one instruction. Values below 2^-15 of the scale become 0, as
// they would be rounded. Elements that are subnormal in bf16 have no such
// exponent; they matter in blocks of byte <= 2, which take the way of fp32.
__device__ __forceinline__ uint4 quantize_block(const uint32_t (&w)[16], uint32_t &byte)
{
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    byte = scale_byte(max(m >> 16, m & 0xFFFFu) >> 7);
    const uint32_t down = (uint32_t)((15 - (int)byte) * 128) & 0xFFFFu, both = down | down << 16;
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (byte <= 2u) {
            const float f[8] = {bf_lo(w[4 * j]), bf_hi(w[4 * j]), bf_lo(w[4 * j + 1]), bf_hi(w[4 * j + 1]),
                                bf_lo(w[4 * j + 2]), bf_hi(w[4 * j + 2]), bf_lo(w[4 * j + 3]), bf_hi(w[4 * j + 3])};
            c[j] = codes8(f, byte);
            continue;
        }
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = w[4 * j + i];
            const uint32_t h = (__viaddmax_s16x2(v & 0x7FFF7FFFu, both, 0u) << 3) | (v & 0x80008000u);
            uint16_t r;
            asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f16x2 t, %1;\n\tcvt.u16.u8 %0, t;\n\t}" : "=h"(r) : "r"(h));
            b[i] = r;
        }
        c[j] = byte == 255u ? 0u : (b[0] | b[1] << 8) | (b[2] | b[3] << 8) << 16;
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}

} // namespace

// bf16 rows on 16-byte boundaries: a block of 32 values a thread, whose 16
// bytes of codes and scale byte are neighbours of the next thread's.
// 14336x4096: 23 us, 6.4 TB/s (four threads a block, through fp32: 40 us).
__global__ void __launch_bounds__(Q_THREADS) mx4_quantize_blocks_kernel(Mx4QuantParams p)
{
    begin_behind();
    const int bpr = p.K / 32;
    const int64_t b = (int64_t)blockIdx.x * Q_THREADS + threadIdx.x;
    if (b >= p.rows * bpr)
        return;
    const uint16_t *src = static_cast<const uint16_t *>(p.w) + (p.w_stride == p.K ? b * 32 : b / bpr * p.w_stride + b % bpr * 32);
    uint32_t v[16], byte;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 q = ld_nc_16(src + 8 * i);
        v[4 * i] = q.x;
        v[4 * i + 1] = q.y;
        v[4 * i + 2] = q.z;
        v[4 * i + 3] = q.w;
    }
    reinterpret_cast<uint4 *>(p.codes)[b] = quantize_block(v, byte);
    p.scales[b] = (uint8_t)byte;
}

// fp32 (a block would be 128 bytes a thread: 57 us for 14336x4096 against 39 us,
// 6.8 TB/s) and rows on any boundary: four threads a block.
template <typename T> __global__ void __launch_bounds__(Q_THREADS) mx4_quantize_kernel(Mx4QuantParams p, int vec)
{
    begin_behind();
    const int upr = p.K / 8;
    const int64_t total = p.rows * upr; // a multiple of 4: the threads of a block go together
    const bool packed = p.w_stride == p.K;
    const T *w = static_cast<const T *>(p.w);
    const int64_t u0 = (int64_t)blockIdx.x * (Q_THREADS * 2) + threadIdx.x;
    float f[2][8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int64_t u = u0 + q * Q_THREADS;
        if (u < total) {
            load8(w + unit_offset(u, upr, p.w_stride, packed), vec, f[q]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[q][i] = 0.0f;
        }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int64_t u = u0 + q * Q_THREADS;
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = absmax_nan(m, f[q][i]);
        m = absmax_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = absmax_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t byte = scale_byte(__float_as_uint(m) >> 23), c = codes8(f[q], byte);
        if (u < total) {
            reinterpret_cast<uint32_t *>(p.codes)[u] = c;
            if ((u & 3) == 0)
                p.scales[u >> 2] = (uint8_t)byte;
        }
    }
}

namespace {

// What a thread reads back at a time, 16 bytes of values: 8 codes of bf16, 4 of fp32.
template <typename T> struct Back;
template <> struct Back<uint16_t> {
    using Codes = uint32_t;
    static __device__ __forceinline__ void store(uint16_t *p, bool vec, uint32_t codes, uint32_t byte)
    {
        uint32_t o[4], f1, f2;
        mx4_unpack8(codes, o);
        mx4_factors(byte, f1, f2);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = mul_bf16x2(mul_bf16x2(o[i], f1), f2);
        if (vec) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[2 * i] = (uint16_t)o[i];
                p[2 * i + 1] = (uint16_t)(o[i] >> 16);
            }
        }
    }
};
template <> struct Back<float> {
    using Codes = uint16_t;
    static __device__ __forceinline__ void store(float *p, bool vec, uint32_t codes, uint32_t byte)
    {
        uint32_t o[4];
        mx4_unpack8(codes, o);
        // times 2^126, then 2^(byte - 127); byte 0 is the subnormal 2^-127
        const float s = byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte == 0u ? 1u << 22 : byte << 23);
        const float up = __uint_as_float((126u + 127u) << 23);
        const float4 f = make_float4(bf_lo(o[0]) * up * s, bf_hi(o[0]) * up * s, bf_lo(o[1]) * up * s, bf_hi(o[1]) * up * s);
        if (vec) {
            *reinterpret_cast<float4 *>(p) = f;
        } else {
            p[0] = f.x;
            p[1] = f.y;
            p[2] = f.z;
            p[3] = f.w;
        }
    }
};

} // namespace

// 14336x4096 to bf16: 23 us, 6.4 TB/s.
template <typename T> __global__ void __launch_bounds__(Q_THREADS) mx4_dequantize_kernel(Mx4DequantParams p, int vec)
{
    using Codes = typename Back<T>::Codes;
    constexpr int EACH = 2 * sizeof(Codes); // values
    begin_behind();
    const int upr = p.K / EACH;
    const int64_t total = p.rows * upr;
    const bool packed = p.w_stride == p.K;
    T *w = static_cast<T *>(p.w);
    const int64_t u0 = (int64_t)blockIdx.x * (Q_THREADS * Q_UNROLL) + threadIdx.x;
    uint32_t c[Q_UNROLL], b[Q_UNROLL];
#pragma unroll
    for (int q = 0; q < Q_UNROLL; ++q) {
        const int64_t u = u0 + q * Q_THREADS;
        c[q] = u < total ? __ldg(reinterpret_cast<const Codes *>(p.codes) + u) : 0u;
        b[q] = u < total ? __ldg(p.scales + u / (32 / EACH)) : 0u;
    }
#pragma unroll
    for (int q = 0; q < Q_UNROLL; ++q) {
        const int64_t u = u0 + q * Q_THREADS;
        if (u < total) {
            const int64_t row = packed ? 0 : u / upr;
            Back<T>::store(w + (packed ? u * EACH : row * p.w_stride + (u - row * upr) * EACH), vec, c[q], b[q]);
        }
    }
}

namespace {

// Blocks of threads for `items`, a thread taking `each` (the host has checked
// that they are a grid's worth).
unsigned grid_for(int64_t items, int each)
{
    return (unsigned)((items + (int64_t)Q_THREADS * each - 1) / ((int64_t)Q_THREADS * each));
}

template <typename T> bool vec_rows(const void *w, int64_t stride)
{
    return (reinterpret_cast<uintptr_t>(w) & 15u) == 0 && (stride * sizeof(T)) % 16 == 0;
}

} // namespace

cudaError_t launch_mx4_quantize(const Mx4QuantParams &p, int dtype, cudaStream_t st)
{
    const unsigned pairs = grid_for(p.rows * (p.K / 8), 2);
    if (dtype == LORA_DTYPE_F32)
        return launch_behind(mx4_quantize_kernel<float>, dim3(pairs), Q_THREADS, 0, 1, st, p, (int)vec_rows<float>(p.w, p.w_stride));
    if (vec_rows<uint16_t>(p.w, p.w_stride))
        return launch_behind(mx4_quantize_blocks_kernel, dim3(grid_for(p.rows * (p.K / 32), 1)), Q_THREADS, 0, 1, st, p);
    return launch_behind(mx4_quantize_kernel<uint16_t>, dim3(pairs), Q_THREADS, 0, 1, st, p, 0);
}

cudaError_t launch_mx4_dequantize(const Mx4DequantParams &p, int dtype, cudaStream_t st)
{
    if (dtype == LORA_DTYPE_F32)
        return launch_behind(mx4_dequantize_kernel<float>, dim3(grid_for(p.rows * (p.K / 4), Q_UNROLL)), Q_THREADS, 0, 1, st, p,
                             (int)vec_rows<float>(p.w, p.w_stride));
    return launch_behind(mx4_dequantize_kernel<uint16_t>, dim3(grid_for(p.rows * (p.K / 8), Q_UNROLL)), Q_THREADS, 0, 1, st, p,
                         (int)vec_rows<uint16_t>(p.w, p.w_stride));
}

// ------------------------------------------------------------------ shrink
namespace {

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int SH_WARPS = 16;     // they share K
constexpr int SH_THREADS = SH_WARPS * 32;
constexpr int SH_ROWS = 64;      // a CTA takes, of the 64 or 256 rows of a chunk
constexpr int SH_PAIR = 16;      // rows whose sums are joined at a time

// The call's status, by one CTA.
__device__ __forceinline__ void open_status(const Mx4ProjParams &p, int tid)
{
    int bad = 0;
    for (int i = tid; i < p.M; i += SH_THREADS)
        bad |= p.seq_slot[i] >= p.L;
    bad = __syncthreads_or(bad);
    if (tid == 0)
        status_begin(p.status, bad ? (uint32_t)LORA_FLAG_SLOT_RANGE : 0u);
}

// The u-th slot that a chunk of up to ROWS rows may have, and what is in it; -1:
// there are not as many. With more slots than rows it is the u-th distinct one
// of the rows (`mine`: this thread's). Whole CTA.
template <int ROWS>
__device__ __forceinline__ int shrink_slot(const Mx4ProjParams &p, int u, int mine, int tid, uint32_t *present, int &slot_s,
                                           SlotInfo &si)
{
    if (p.L <= min(p.M, ROWS)) {
        si = slot_info(p.tab, u, p.L);
        return u;
    }
    const int lane = tid & 31;
    present[lane] = 0u;
    if (tid == 0)
        slot_s = -1;
    __syncthreads();
    if (mine >= 0 && mine < p.L)
        atomicOr(&present[mine >> 5], 1u << (mine & 31));
    __syncthreads();
    if (tid < 32) {
        const uint32_t w = present[lane];
        int incl = __popc(w);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        const int before = incl - __popc(w);
        if (u >= before && u < incl) {
            uint32_t rest = w;
            for (int i = before; i < u; ++i)
                rest &= rest - 1;
            slot_s = lane * 32 + __ffs(rest) - 1;
        }
    }
    __syncthreads();
    if (slot_s >= 0)
        si = slot_info(p.tab, slot_s, p.L);
    return slot_s;
}

// NT * 8 rows of the slot (from i0; past the last they repeat it) against 16
// rank rows over the warp's blocks of 32 k, `AHEAD` blocks' loads in flight.
template <int NT, int AHEAD>
__device__ __forceinline__ void shrink_tile(const Mx4ProjParams &p, const uint16_t *ra, const uint16_t *rb, const int *rows,
                                            int count, int i0, int b0, int b1, int g, int t, float (&acc)[NT][4])
{
    const uint16_t *x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        x[n] = p.x + (int64_t)rows[min(i0 + n * 8 + g, count - 1)] * p.x_stride + t * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[n][i] = 0.0f;
    }
    for (int b = b0; b < b1; b += AHEAD) {
        uint4 va[AHEAD], vb[AHEAD], vx[AHEAD][NT];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const bool have = b + a < b1;
            const uint4 z = make_uint4(0, 0, 0, 0);
            va[a] = have ? ld_nc_16(ra + (b + a) * 32) : z;
            vb[a] = have ? ld_nc_16(rb + (b + a) * 32) : z;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                vx[a][n] = have ? ld_nc_16(x[n] + (b + a) * 32) : z;
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_16816(acc[n], va[a].x, vb[a].x, va[a].y, vb[a].y, vx[a][n].x, vx[a][n].y);
                mma_16816(acc[n], va[a].z, vb[a].z, va[a].w, vb[a].w, vx[a][n].z, vx[a][n].w);
            }
    }
}

} // namespace

// Grid: 16-rank groups, by slots (or, where there are more of them than rows in a
// chunk, the u-th distinct slot of the chunk), by chunks of CHUNK rows and `takes` CTAs
// for 64 rows of the slot each. Each thread multiplies 8
// consecutive k of two rank rows and of the slot's rows at a time: which k a
// fragment's slots mean is free as long as both operands agree. (16 warps have 128
// registers a thread; 56 bytes more are in local memory.)
template <int CHUNK> __global__ void __launch_bounds__(SH_THREADS) mx4_shrink_kernel(Mx4ProjParams p, int takes)
{
    __shared__ uint32_t present[MAX_BUCKETS / 32];
    __shared__ int slot_s, rows_s[SH_ROWS];
    __shared__ float red[SH_WARPS][16][SH_PAIR + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int r0 = blockIdx.x * 16, u = blockIdx.y, c0 = (int)blockIdx.z / takes * CHUNK, from = (int)blockIdx.z % takes * SH_ROWS;
    // Launched early behind whatever the stream ran before; nothing is read
    // until that is complete, and only then may the projection kernel start.
    begin_behind();
    const int mine = tid < CHUNK && c0 + tid < p.M ? p.seq_slot[c0 + tid] : -1;
    if (blockIdx.x == 0 && u == 0 && blockIdx.z == 0)
        open_status(p, tid);
    SlotInfo si;
    const int slot = shrink_slot<CHUNK>(p, u, mine, tid, present, slot_s, si);
    if (slot < 0 || !si.on || r0 >= si.rank)
        return;
    const uint32_t match = __ballot_sync(0xffffffffu, mine == slot);
    __syncthreads(); // slot_s and the distinct slots have been read
    if (lane == 0 && warp < CHUNK / 32)
        present[warp] = match;
    __syncthreads();
    int before = 0, total = 0; // the slot's rows of the chunk, in order
#pragma unroll
    for (int w = 0; w < CHUNK / 32; ++w) {
        const int n = __popc(present[w]);
        before += w < warp ? n : 0;
        total += n;
    }
    const int count = min(total - from, SH_ROWS), at = before + __popc(match & ((1u << lane) - 1u)) - from;
    if (count <= 0)
        return;
    if (mine == slot && at >= 0 && at < SH_ROWS)
        rows_s[at] = c0 + tid;
    __syncthreads();
    const int nb = p.K / 32;
    const int b0 = (int)((int64_t)nb * warp / SH_WARPS), b1 = (int)((int64_t)nb * (warp + 1) / SH_WARPS); // this warp's blocks of 32 k
    // rank rows past the rank read the last one; what comes of them is dropped
    const uint16_t *ra = si.a + (size_t)min(r0 + g, si.rank - 1) * p.K + t * 8;
    const uint16_t *rb = si.a + (size_t)min(r0 + g + 8, si.rank - 1) * p.K + t * 8;
    const float *comp = p.tab.comp_table + (size_t)slot * LORA_COMP_STRIDE;

    // the warps' sums of two tiles of 8 rows, in warp order, to h
    auto join = [&](int i0, const float (&a)[4], const float (&b)[4]) {
        red[warp][g][2 * t] = a[0];
        red[warp][g][2 * t + 1] = a[1];
        red[warp][g + 8][2 * t] = a[2];
        red[warp][g + 8][2 * t + 1] = a[3];
        red[warp][g][8 + 2 * t] = b[0];
        red[warp][g][8 + 2 * t + 1] = b[1];
        red[warp][g + 8][8 + 2 * t] = b[2];
        red[warp][g + 8][8 + 2 * t + 1] = b[3];
        __syncthreads();
        for (int i = tid; i < 16 * SH_PAIR; i += SH_THREADS) {
            const int q = i & 15, row = i >> 4;
            if (i0 + row < count && r0 + q < p.R) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < SH_WARPS; ++w)
                    v += red[w][q][row];
                v = r0 + q < si.rank ? si.scale * __ldg(comp + r0 + q) * v : 0.0f;
                store_h(p, (size_t)rows_s[i0 + row] * p.R + r0 + q, v);
            }
        }
        __syncthreads();
    };
    const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (count <= 8) {
        float acc[1][4];
        shrink_tile<1, 8>(p, ra, rb, rows_s, count, 0, b0, b1, g, t, acc);
        join(0, acc[0], none);
        return;
    }
    int i0 = 0;
    for (; count - i0 > 16; i0 += 32) {
        float acc[4][4];
        shrink_tile<4, 4>(p, ra, rb, rows_s, count, i0, b0, b1, g, t, acc);
        join(i0, acc[0], acc[1]);
        join(i0 + 16, acc[2], acc[3]);
    }
    if (i0 < count) {
        float acc[2][4];
        shrink_tile<2, 6>(p, ra, rb, rows_s, count, i0, b0, b1, g, t, acc);
        join(i0, acc[0], acc[1]);
    }
}

namespace {

constexpr int SM_CHUNK = 256;              // rows that a group of CTAs sorts by slot
constexpr int SM_ROWS = 64, SM_RANKS = 64; // of a product, by slabs of 64 k
constexpr int SM_STAGES = 12;
constexpr int SM_MOST = 16;                // CTAs of a chunk, at most
constexpr uint32_t SM_TILE = 64 * 128, SM_BYTES = SM_STAGES * 2 * SM_TILE + 1024;

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

} // namespace

// The same for many rows. The CTAs of a chunk of 256 rows sort it by slot and take
// turns with what that gives: up to 64 rows of a slot against up to 64 ranks, both
// through shared memory, so x is read once and A once for 64 rows. A warp has 32
// ranks by 32 rows of one k16 of each slab (16 by 16 of all four, which reads shared
// memory twice as often: 4 us longer for 8192 rows). (A grid over
// slots would be mostly empty CTAs: 8192 rows of 16 slots, 8192 of them.)
// Grid: groups of 64 ranks, CTAs of a chunk, chunks.
__global__ void __launch_bounds__(SH_THREADS, 1) mx4_shrink_many_kernel(Mx4ProjParams p)
{
    extern __shared__ uint8_t sm_raw[];
    __shared__ alignas(16) int slots_s[SM_CHUNK]; // read four at a time
    __shared__ int sorted_s[SM_CHUNK], unit_s[SM_CHUNK];
    __shared__ uint32_t starts_s[SM_CHUNK / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int r0 = blockIdx.x * SM_RANKS, c0 = (int)blockIdx.z * SM_CHUNK;
    begin_behind();
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
        open_status(p, tid);
    int mine = -1;
    if (tid < SM_CHUNK) {
        mine = c0 + tid < p.M ? p.seq_slot[c0 + tid] : -1;
        mine = mine < p.L ? mine : -1;
        slots_s[tid] = mine;
    }
    if (tid < SM_CHUNK / 32)
        starts_s[tid] = 0u;
    __syncthreads();
    int less = 0, before = 0, all = 0; // rows of lower slots, earlier rows of this one, rows of this one
    if (tid < SM_CHUNK) {
#pragma unroll 4
        for (int j = 0; j < SM_CHUNK; j += 4) {
            const int4 v = *reinterpret_cast<const int4 *>(slots_s + j);
            less += (v.x < mine) + (v.y < mine) + (v.z < mine) + (v.w < mine);
            const int e[4] = {v.x == mine, v.y == mine, v.z == mine, v.w == mine};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                all += e[i];
                before += e[i] && j + i < tid;
            }
        }
        const int at = less + before;
        sorted_s[at] = c0 + tid;
        if (mine >= 0 && before % SM_ROWS == 0) // a unit begins
            atomicOr(&starts_s[at >> 5], 1u << (at & 31));
    }
    __syncthreads();
    int units = 0, nth = 0;
#pragma unroll
    for (int w = 0; w < SM_CHUNK / 32; ++w) {
        const int n = __popc(starts_s[w]);
        nth += w < (less + before) >> 5 ? n : 0;
        units += n;
    }
    if (mine >= 0 && before % SM_ROWS == 0)
        unit_s[nth + __popc(starts_s[(less + before) >> 5] & ((1u << ((less + before) & 31)) - 1u))] =
            mine << 16 | (less + before) << 8 | (min(all - before, SM_ROWS) - 1);
    __syncthreads();

    const uint32_t raw = smem_u32(sm_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const smem = sm_raw + (base - raw);
    const int row = tid >> 3, piece = tid & 7, slabs = (p.K + 63) / 64;
    const uint32_t into = (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4));
    const int rg = (warp & 1) * 32, xg = (warp >> 1 & 1) * 32, k16 = warp >> 2;
    const int lr = lane & 7, lm = lane >> 3; // row and matrix of a load
    const int a_row = rg + lr + (lm & 1) * 8, x_row = xg + lr + (lm >> 1) * 8;
    const uint32_t a_at = SM_TILE + (uint32_t)(a_row * 128 + (((k16 * 2 + (lm >> 1)) ^ (a_row & 7)) << 4)),
                   x_at = (uint32_t)(x_row * 128 + (((k16 * 2 + (lm & 1)) ^ (x_row & 7)) << 4));
    for (int unit = blockIdx.y; unit < units; unit += gridDim.y) {
        const int slot = unit_s[unit] >> 16, count = (unit_s[unit] & 255) + 1;
        const int *const rows_s = sorted_s + (unit_s[unit] >> 8 & 255);
        const SlotInfo si = slot_info(p.tab, slot, p.L);
        if (!si.on || r0 >= si.rank)
            continue;
        const bool have_x = row < count, have_a = r0 + row < si.rank;
        const uint16_t *xr = p.x + (int64_t)rows_s[have_x ? row : 0] * p.x_stride + piece * 8;
        const uint16_t *ar = si.a + (size_t)(have_a ? r0 + row : 0) * p.K + piece * 8;
        auto load = [&](int b) {
            if (b < slabs) {
                uint8_t *const to = smem + (uint32_t)(b % SM_STAGES) * 2 * SM_TILE + into;
                const bool in = b * 64 + piece * 8 < p.K;
                const int k = in ? b * 64 : 0;
                cp_async_16(to, in ? xr + k : p.x, in && have_x ? 16u : 0u);
                cp_async_16(to + SM_TILE, in ? ar + k : p.x, in && have_a ? 16u : 0u);
            }
            cp_async_commit();
        };
        __syncthreads(); // the unit before has been read
        for (int b = 0; b < SM_STAGES - 1; ++b)
            load(b);
        const bool work = r0 + rg < si.rank && xg < count;
        float acc[2][4][4] = {};
        for (int b = 0; b < slabs; ++b) {
            cp_async_wait_group<SM_STAGES - 2>();
            __syncthreads(); // slab b is there, and slab b - 1 has been read
            load(b + SM_STAGES - 1);
            if (work) {
                const uint32_t at = base + (uint32_t)(b % SM_STAGES) * 2 * SM_TILE;
                uint32_t a[2][4], x[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) { // 16 rows further: 2048 bytes, turned alike
                    ldmatrix_x4(at + a_at + (uint32_t)i * 2048, a[i]);
                    ldmatrix_x4(at + x_at + (uint32_t)i * 2048, x[i]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        mma_16816(acc[i][n], a[i][0], a[i][1], a[i][2], a[i][3], x[n >> 1][(n & 1) * 2], x[n >> 1][(n & 1) * 2 + 1]);
            }
        }
        // the four k16's sums, in order, where the slabs were
        __syncthreads();
        float *const red = reinterpret_cast<float *>(smem);
        constexpr int RED_ROW = SM_ROWS + 1, RED = SM_RANKS * RED_ROW;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    red[k16 * RED + (rg + i * 16 + g + (j >> 1) * 8) * RED_ROW + xg + n * 8 + 2 * t + (j & 1)] = acc[i][n][j];
        __syncthreads();
        const float *comp = p.tab.comp_table + (size_t)slot * LORA_COMP_STRIDE;
        const int ranks = min(p.R - r0, SM_RANKS);
        for (int i = tid; i < count * SM_RANKS; i += SH_THREADS) {
            const int r = i & (SM_RANKS - 1), q = i / SM_RANKS;
            if (r < ranks) {
                const float *v = red + r * RED_ROW + q;
                const float h = r0 + r < si.rank ? si.scale * __ldg(comp + r0 + r) * (v[0] + v[RED] + v[2 * RED] + v[3 * RED]) : 0.0f;
                store_h(p, (size_t)rows_s[q] * p.R + r0 + r, h);
            }
        }
    }
}

cudaError_t launch_mx4_shrink(const Mx4ProjParams &p, int num_sms, cudaStream_t st)
{
    // Many rows and more than 16 ranks, of which the other kernel reads x for each:
    // a call of K = N = 4096, 16 slots of rank 64 (then 32 of rank 16), takes
    //   rows  2048         4096          8192
    //   many  63.6  61.8   112.7 111.9   203.3 202.9 us
    //   other 69.6  57.7   132.2 111.6   248.4 209.0
    // (and of more than 65535 times 64 rows the other's chunks are not a grid's)
    if (p.M >= 2048 && (p.R > 16 || p.M > 65535 * SH_ROWS)) {
        static std::atomic<uint64_t> raised{0};
        const cudaError_t e = raise_smem_limit(raised, mx4_shrink_many_kernel, (int)SM_BYTES);
        if (e != cudaSuccess)
            return e;
        // some two CTAs an SM; a chunk of one slot has four units, of many more
        const int groups = (p.R + SM_RANKS - 1) / SM_RANKS, chunks = (p.M + SM_CHUNK - 1) / SM_CHUNK;
        const int each = std::max(4, std::min(SM_MOST, 2 * num_sms / (groups * chunks)));
        return launch_behind(mx4_shrink_many_kernel, dim3((unsigned)groups, (unsigned)each, (unsigned)chunks), SH_THREADS, SM_BYTES, 1,
                             st, p);
    }
    // A CTA takes all registers of its SM, and the projection's have to wait for it: the
    // fewer have work the better. Chunks of 64 and of 256 rows, 16 adapters of rank 64 at
    // N = 4096, then 32 of rank 64 and 32 of rank 16 at N = 6144:
    //   128 rows   18.5  18.3   30.3  28.6   22.2  21.5 us
    //   256 rows   25.3  23.1   40.8  37.6   27.5  27.3
    //   512 rows   36.3  32.2   62.0  55.6   37.5  35.3
    const int chunk = p.M > SH_ROWS ? 256 : SH_ROWS;
    const int takes = std::min((p.M + SH_ROWS - 1) / SH_ROWS, chunk / SH_ROWS);
    return launch_behind(chunk == 256 ? mx4_shrink_kernel<256> : mx4_shrink_kernel<SH_ROWS>,
                         dim3((unsigned)((p.R + 15) / 16), (unsigned)std::min(p.L, std::min(p.M, chunk)),
                              (unsigned)((p.M + chunk - 1) / chunk * takes)),
                         SH_THREADS, 0, 1, st, p, takes);
}

// -------------------------------------------------------------------- rows
namespace {

constexpr int RW_WARPS = 16, RW_FINISH = 4;  // compute, finish
constexpr int RW_THREADS = (RW_WARPS + RW_FINISH) * 32;
constexpr int RW_ROWS = 4;                   // batch rows: half the n of one mma
constexpr uint32_t RW_BOX = 16 * 128;        // codes of 16 weight rows x 256 k
constexpr int RW_BUFS = 3;                   // steps whose partial sums may wait to be finished
constexpr uint32_t RW_PART = 16 * RW_ROWS;   // floats of a warp's partial tile, [feature][row]
constexpr int RW_MAX_DEPTH = 4;
constexpr uint32_t RW_SMEM = 226 * 1024;
constexpr int RW_X = 1, RW_H = 2; // named barriers

// How the warps share the work: a team of `team` warps splits K (boxes of 256)
// of 16 features, and the CTA's teams take neighbouring features.
struct RowsShape {
    int boxes, team, depth;
    uint32_t x_bytes, smem;
};
inline RowsShape rows_shape(int K, int R)
{
    RowsShape r;
    r.boxes = (K + 255) / 256;
    r.team = 1;
    while (r.team < RW_WARPS && r.team < r.boxes)
        r.team *= 2;
    r.x_bytes = (uint32_t)r.boxes * 512u * RW_ROWS;
    const uint32_t fixed = 1024u + r.x_bytes + RW_BUFS * RW_WARPS * RW_PART * 4 + RW_ROWS * (uint32_t)R * 4 +
                           RW_WARPS / (uint32_t)r.team * 16u * RW_ROWS * 4u;
    r.depth = 0;
    while (r.depth < RW_MAX_DEPTH && fixed + (uint32_t)(r.depth + 1) * RW_WARPS * RW_BOX <= RW_SMEM)
        ++r.depth;
    r.smem = fixed + (uint32_t)r.depth * RW_WARPS * RW_BOX;
    return r;
}

__device__ __forceinline__ uint4 lds_16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// mx4_unpack8 with the pairs (0, 4), (1, 5), (2, 6), (3, 7): codes four apart lie
// in the two halves of a word as they are, so none are moved.
__device__ __forceinline__ void unpack8_apart(uint32_t w, uint32_t (&o)[4])
{
    const uint32_t v = w >> 8;
    o[0] = ((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
    o[1] = ((w & 0x00F000F0u) * 0x0104u) & 0x81C081C0u;
    o[2] = ((v & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
    o[3] = ((v & 0x00F000F0u) * 0x0104u) & 0x81C081C0u;
}
// Eight values of x in the same pairs.
__device__ __forceinline__ uint4 pairs_apart(uint4 v)
{
    return make_uint4(prmt<0x5410>(v.x, v.z), prmt<0x7632>(v.x, v.z), prmt<0x5410>(v.y, v.w), prmt<0x7632>(v.y, v.w));
}

// Eight codes of two weight rows -> bf16 pairs, times their blocks' scales.
__device__ __forceinline__ void widen_pair(uint32_t a, uint32_t b, uint32_t fa, uint32_t fb, uint32_t (&u)[4], uint32_t (&v)[4])
{
    unpack8_apart(a, u);
    unpack8_apart(b, v);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        u[q] = mul_bf16x2(u[q], fa);
        v[q] = mul_bf16x2(v[q], fb);
    }
}

} // namespace

// A CTA an SM; step s of CTA c takes the features of 16 * teams from
// (s * gridDim + c) * 16 * teams on. Each compute warp has a ring of its own
// of code boxes that its lane 0 keeps asking for by TMA, steps ahead, so
// nothing in a CTA waits for anything but its own boxes; partial sums of a
// step go to shared memory, and four more warps add them in order, add the
// adapters and write y while the next steps are in work. x (4 rows, all of K)
// stays in shared memory; within 64 bytes its 16-byte pieces are turned by
// the row and the block so that the eight lanes of a load phase meet different
// bank groups. Which k a fragment's slots mean is free as long as
// both operands agree: thread t of four supplies the block t of 128 k.
// 1x4096x32000 takes 30 us (2.3 TB/s of codes), 1x4096x4096 8.7 with its shrink. Issue
// and waits bound it: 62 % of the issue slots are used, and half of the 17.7 million
// instructions of a warp of the former call widen, 17 for 8 codes.
__global__ void __launch_bounds__(RW_THREADS, 1)
    mx4_rows_kernel(const __grid_constant__ CUtensorMap codes, const __grid_constant__ Mx4ProjParams p, RowsShape shape)
{
    extern __shared__ uint8_t rw_raw[];
    __shared__ uint64_t full[RW_WARPS][RW_MAX_DEPTH], part_full[RW_BUFS], part_free[RW_BUFS];
    __shared__ const uint16_t *brow[RW_ROWS]; // B of the row's slot, nullptr: no delta
    __shared__ int bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t raw = smem_u32(rw_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const smem = rw_raw + (base - raw);
    const uint32_t ring = base, xs = base + (uint32_t)shape.depth * RW_WARPS * RW_BOX, xrow = (uint32_t)shape.boxes * 512u;
    float *const part = reinterpret_cast<float *>(smem + (xs - base) + shape.x_bytes);
    float *const hs = part + RW_BUFS * RW_WARPS * RW_PART, *const delta = hs + RW_ROWS * p.R; // s h; a step's B (s h)
    const int T = shape.team, teams = RW_WARPS / T, nblk = p.K / 32;
    const int tiles = (p.N + 15) / 16, groups = (tiles + teams - 1) / teams; // of 16 features, of a step's
    const int steps = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    if (tid < RW_WARPS * RW_MAX_DEPTH)
        mbar_init(&full[tid / RW_MAX_DEPTH][tid % RW_MAX_DEPTH], 1 + (p.never > 1));
    if (tid == 0) {
        for (int b = 0; b < RW_BUFS; ++b) {
            mbar_init(&part_full[b], RW_WARPS + (p.never == 1));
            mbar_init(&part_free[b], RW_FINISH);
        }
        bad = 0;
    }
    fence_barrier_init();
    __syncthreads();

    if (warp < RW_WARPS) {
        const int wk = warp % T, team = warp / T, g = lane >> 2, t = lane & 3;
        const int per = wk < shape.boxes ? (shape.boxes - wk + T - 1) / T : 0; // boxes of a step, 0 to 2
        const int units = steps * per, depth = shape.depth;
        const uint32_t mine = ring + (uint32_t)(warp * depth) * RW_BOX;
        auto feature = [&](int s) { return ((s * (int)gridDim.x + (int)blockIdx.x) * teams + team) * 16; };
        auto ask = [&](int u, int slot) {
            const int s = per == 2 ? u >> 1 : u, box = wk + (per == 2 ? (u & 1) * T : 0);
            mbar_arrive_expect_tx(&full[warp][slot], RW_BOX);
            tma_load_2d(smem + (warp * depth + slot) * RW_BOX, &codes, box * 128, feature(s), &full[warp][slot]);
        };
        // scale bytes of a box: rows g and g + 8, blocks t and t + 4
        const bool eights = nblk % 8 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 7u) == 0;
        const int jump = (int)gridDim.x * teams * 16; // features from a step to the next
        int sf = feature(0) + g, sk = 0;              // where the next are
        const int byte_at = eights ? 8 * t : 0;
        // The bytes are cut out where they are used: here the cut would wait for
        // the load, a quarter of the time of a step.
        auto next_scales = [&](uint2 (&sc)[2]) {
            const int b0 = (wk + sk * T) * 8;
#pragma unroll
            for (int r = 0; r < 2; ++r) { // rows past N repeat the last; their sums are dropped
                const uint8_t *row = p.scales + (size_t)min(sf + 8 * r, p.N - 1) * nblk + b0;
                if (eights)
                    sc[r] = __ldg(reinterpret_cast<const uint2 *>(row));
                else {
                    sc[r].x = b0 + t < nblk ? __ldg(row + t) : 0u;
                    sc[r].y = b0 + 4 + t < nblk ? __ldg(row + 4 + t) : 0u;
                }
            }
            if (++sk == per) {
                sk = 0;
                sf += jump;
            }
        };
        if (elected())
            for (int u = 0; u < min(depth, units); ++u)
                ask(u, u);
        __syncwarp();
        uint2 next[2] = {};
        if (units > 0)
            next_scales(next);
        // x, zeros past K and M
        for (int i = tid; i < RW_ROWS * shape.boxes * 32; i += RW_WARPS * 32) {
            const int row = i / (shape.boxes * 32), piece = i - row * (shape.boxes * 32), block = piece >> 2;
            const bool have = row < p.M && piece * 8 < p.K;
            const int turn = (block >> 1 & 1) | (row & 1) << 1;
            const uint4 v = pairs_apart(have ? ld_nc_16(p.x + (int64_t)row * p.x_stride + piece * 8) : make_uint4(0, 0, 0, 0));
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(xs + (uint32_t)row * xrow + (uint32_t)block * 64u +
                                                                         (uint32_t)((piece & 3) ^ turn) * 16u),
                         "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                         : "memory");
        }
        named_bar_sync(RW_X, RW_WARPS * 32);

        const uint32_t xg = xs + (uint32_t)(g & (RW_ROWS - 1)) * xrow + (uint32_t)t * 64u; // columns 4 to 7 repeat
        const uint32_t turn = (uint32_t)((t >> 1) | (g & 1) << 1) << 4;
        const uint32_t row_at = (uint32_t)g * 128u; // of a box; row g + 8 is 1024 further and turned alike
        int slot = 0, u = 0;
        uint32_t parity = 0;
        bool ok = true; // no wait gave up
        for (int s = 0; s < steps; ++s) {
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int k = 0; k < per; ++k, ++u) {
                const int box = wk + k * T;
                uint32_t sc[4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    sc[r] = next[r].x >> byte_at & 255u;
                    sc[2 + r] = next[r].y >> byte_at & 255u;
                }
                if (u + 1 < units)
                    next_scales(next);
                if (!(ok = warp_wait(&full[warp][slot], parity, &bad, p.wait_ns)))
                    break;
                const uint32_t at = mine + (uint32_t)slot * RW_BOX + row_at;
                const bool twice = __any_sync(0xffffffffu, max(max(sc[0], sc[1]), max(sc[2], sc[3])) > MX4_ONE_FACTOR);
#pragma unroll
                for (int h = 0; h < 2; ++h) { // 128 k
                    const uint32_t piece = (uint32_t)(((h * 4 + t) ^ (g & 7)) << 4);
                    const uint4 a = lds_16(at + piece), b = lds_16(at + 1024u + piece);
                    uint32_t fa = mx4_factor(sc[2 * h]), fb = mx4_factor(sc[2 * h + 1]), fa2 = 0u, fb2 = 0u;
                    if (twice) {
                        mx4_factors(sc[2 * h], fa, fa2);
                        mx4_factors(sc[2 * h + 1], fb, fb2);
                    }
                    const uint32_t xa = xg + (uint32_t)(box * 8 + h * 4) * 64u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 xv = lds_16(xa + (((uint32_t)j << 4) ^ turn));
                        uint32_t w[4], v[4];
                        widen_pair(j == 0 ? a.x : j == 1 ? a.y : j == 2 ? a.z : a.w, j == 0 ? b.x : j == 1 ? b.y : j == 2 ? b.z : b.w,
                                   fa, fb, w, v);
                        if (twice) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                w[q] = mul_bf16x2(w[q], fa2);
                                v[q] = mul_bf16x2(v[q], fb2);
                            }
                        }
                        mma_16816(acc, w[0], v[0], w[1], v[1], xv.x, xv.y);
                        mma_16816(acc, w[2], v[2], w[3], v[3], xv.z, xv.w);
                    }
                }
                __syncwarp(); // every lane has read the box
                if (u + depth < units && elected())
                    ask(u + depth, slot);
                if (++slot == depth) {
                    slot = 0;
                    parity ^= 1u;
                }
            }
            const int buf = s % RW_BUFS, use = s / RW_BUFS;
            if (ok && use > 0) // the step that used the buffer before has been finished
                ok = warp_wait(&part_free[buf], (uint32_t)(use - 1) & 1u, &bad, p.wait_ns);
            if (!ok)
                break;
            float *to = part + (size_t)(buf * RW_WARPS + warp) * RW_PART;
            if (t < RW_ROWS / 2) {
                *reinterpret_cast<float2 *>(to + g * RW_ROWS + 2 * t) = make_float2(acc[0], acc[1]);
                *reinterpret_cast<float2 *>(to + (g + 8) * RW_ROWS + 2 * t) = make_float2(acc[2], acc[3]);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&part_full[buf]);
        }
        if (!ok) // the boxes on their way land before the CTA ends
            for (int v = u; v < min(u + depth, units); ++v)
                mbar_wait(&full[warp][v % depth], (uint32_t)(v / depth) & 1u, p.wait_ns);
    } else {
        // ---- finish: the rows' slots, s h, then step by step
        const int ft = tid - RW_WARPS * 32;
        if (ft < RW_ROWS) {
            const SlotInfo si = ft < p.M ? slot_info(p.tab, p.seq_slot[ft], p.L) : SlotInfo{nullptr, nullptr, 0.0f, 0, 0};
            brow[ft] = si.on ? si.b : nullptr;
        }
        named_bar_sync(RW_H, RW_FINISH * 32);
        grid_dependency_wait(); // h is complete, and the call's status open
        for (int i = ft; i < p.M * p.R; i += RW_FINISH * 32) {
            const int row = i / p.R, r = i - row * p.R;
            float v = 0.0f;
            if (brow[row] != nullptr && r < p.tab.rank_table[p.seq_slot[row]])
                v = __ldcg(p.h + i);
            hs[i] = v;
        }
        named_bar_sync(RW_H, RW_FINISH * 32);
        // the adapter's part of an output takes `lanes` lanes, a 16-byte piece of its
        // B row each; then a thread adds the team's partial sums of an output
        // (a step's first pieces are asked for while the step before is in work)
        const int pieces = p.R / 8, sums = min(T, shape.boxes), width = teams * 16, outs = width * p.M;
        const int wide = 31 - __clz(width); // a power of two
        int lanes = 1;
        while (lanes < pieces)
            lanes *= 2;
        const int sub = lane & (lanes - 1), each = 32 / lanes, first = (ft >> 5) * each + lane / lanes;
        constexpr int AT_ONCE = 4;
        uint4 b[AT_ONCE];
        auto ask = [&](int s, int o0) {
            const int f0 = (s * (int)gridDim.x + (int)blockIdx.x) * width;
#pragma unroll
            for (int a = 0; a < AT_ONCE; ++a) {
                const int o = o0 + a * RW_FINISH * each + first, r = o >> wide, f = f0 + (o & (width - 1));
                b[a] = make_uint4(0, 0, 0, 0);
                if (o < outs && f < p.N && sub < pieces && brow[r] != nullptr)
                    b[a] = ld_nc_16(brow[r] + (size_t)f * p.R + sub * 8);
            }
        };
        if (steps > 0)
            ask(0, 0);
        for (int s = 0; s < steps; ++s) {
            const int buf = s % RW_BUFS, f0 = (s * (int)gridDim.x + (int)blockIdx.x) * width;
            for (int o0 = 0; o0 < outs; o0 += RW_FINISH * each * AT_ONCE) {
                if (o0 > 0)
                    ask(s, o0);
#pragma unroll
                for (int a = 0; a < AT_ONCE; ++a) {
                    if (o0 + a * RW_FINISH * each >= outs) // none of the warp's lanes has one
                        break;
                    const int o = o0 + a * RW_FINISH * each + first;
                    float d = 0.0f;
                    if (o < outs && sub < pieces) {
                        const float4 *h = reinterpret_cast<const float4 *>(hs + (o >> wide) * p.R + sub * 8);
                        d = dot8_bf_f32(0.0f, b[a], h[0], h[1]);
                    }
                    for (int i = lanes / 2; i > 0; i >>= 1)
                        d += __shfl_xor_sync(0xffffffffu, d, i);
                    if (sub == 0 && o < outs)
                        delta[o] = d;
                }
            }
            if (s + 1 < steps)
                ask(s + 1, 0);
            named_bar_sync(RW_H, RW_FINISH * 32);
            wait_or_note(&part_full[buf], (uint32_t)(s / RW_BUFS) & 1u, &bad, p.wait_ns); // goes on with what there is
            const float *from = part + (size_t)buf * RW_WARPS * RW_PART;
            for (int i = ft; i < 2 * outs; i += RW_FINISH * 32) { // two threads an output
                const int o = i >> 1, row = o >> wide, f = o & (width - 1);
                const float *q = from + (size_t)((f >> 4) * T) * RW_PART + (f & 15) * RW_ROWS + row;
                float v = 0.0f;
#pragma unroll 8
                for (int w = i & 1; w < sums; w += 2)
                    v += q[w * RW_PART];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                if (brow[row] != nullptr) // else the base product to the bit
                    v += delta[o];
                if ((i & 1) == 0 && f0 + f < p.N)
                    p.y[(int64_t)row * p.y_stride + f0 + f] = f32_to_bf16_bits(v);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&part_free[buf]);
            named_bar_sync(RW_H, RW_FINISH * 32); // delta is written again
        }
        if (ft == 0 && *reinterpret_cast<volatile int *>(&bad) != 0)
            atomicOr(p.status, (uint32_t)LORA_FLAG_WAIT_TIMEOUT);
    }
}

// Whether a call can take the rows kernel: x and two boxes a warp have to fit.
bool mx4_rows_fit(int M, int K, int R) { return M <= RW_ROWS && K <= 512 * RW_WARPS && rows_shape(K, R).depth >= 2; }

cudaError_t launch_mx4_rows(const Mx4ProjParams &p, const CUtensorMap &codes, int num_sms, cudaStream_t st)
{
    const RowsShape shape = rows_shape(p.K, p.R);
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = raise_smem_limit(raised, mx4_rows_kernel, (int)RW_SMEM);
    if (e != cudaSuccess)
        return e;
    const int step = 16 * (RW_WARPS / shape.team), groups = (p.N + step - 1) / step;
    return launch_behind(mx4_rows_kernel, dim3((unsigned)(groups < num_sms ? groups : num_sms)), RW_THREADS, shape.smem, 1, st, codes, p,
                         shape);
}

} // namespace rd
