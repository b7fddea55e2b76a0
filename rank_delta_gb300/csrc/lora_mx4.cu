// Microscaled 4-bit matrices: quantisation, reading back, and the projection
//   y[i, :] = dq(W) x_i + s B_s (A_s x_i)
// with the base W in that form and each row's adapter in bf16.
//
// quantize   a thread takes a block: its scale is 2^(floor(log2 max) - 2), read
//            off the exponent field, so the largest code is 4 or 6; codes are
//            rounded to nearest even and saturate.
// dequantize the reverse, eight values a thread and step.
// shrink     h = A_s x_i for the rows of each slot, on the tensor cores straight
//            from memory: 16 rank rows by up to 16 of the slot's rows a CTA and
//            pass. The projection kernels start behind it at once and wait for
//            h only where they need it.
// stream     the product for few rows. The weight's 16-row fragments go from
//            memory to the tensor cores' registers: a thread copies 16 bytes
//            (one block of 32 codes) of two weight rows, 128 k of the tile's 16
//            rows a warp and step, into a ring of its own in shared memory (no
//            barrier: it reads back what it copied itself), widens them to bf16
//            exactly, and multiplies. Which k a fragment's slots mean is free as
//            long as both operands agree, so the codes stay in their natural
//            order and x is read to match.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "lora_mx4.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace rd {

namespace cg = cooperative_groups;

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
// 14336x4096: 24 us, 6.1 TB/s (four threads a block, through fp32: 40 us).
__global__ void __launch_bounds__(Q_THREADS) mx4_quantize_blocks_kernel(Mx4QuantParams p)
{
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

// 14336x4096 to bf16: 24 us, 6.3 TB/s.
template <typename T> __global__ void __launch_bounds__(Q_THREADS) mx4_dequantize_kernel(Mx4DequantParams p, int vec)
{
    using Codes = typename Back<T>::Codes;
    constexpr int EACH = 2 * sizeof(Codes); // values
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
        mx4_quantize_kernel<float><<<pairs, Q_THREADS, 0, st>>>(p, vec_rows<float>(p.w, p.w_stride));
    else if (vec_rows<uint16_t>(p.w, p.w_stride))
        mx4_quantize_blocks_kernel<<<grid_for(p.rows * (p.K / 32), 1), Q_THREADS, 0, st>>>(p);
    else
        mx4_quantize_kernel<uint16_t><<<pairs, Q_THREADS, 0, st>>>(p, 0);
    return cudaGetLastError();
}

cudaError_t launch_mx4_dequantize(const Mx4DequantParams &p, int dtype, cudaStream_t st)
{
    if (dtype == LORA_DTYPE_F32)
        mx4_dequantize_kernel<float>
            <<<grid_for(p.rows * (p.K / 4), Q_UNROLL), Q_THREADS, 0, st>>>(p, vec_rows<float>(p.w, p.w_stride));
    else
        mx4_dequantize_kernel<uint16_t>
            <<<grid_for(p.rows * (p.K / 8), Q_UNROLL), Q_THREADS, 0, st>>>(p, vec_rows<uint16_t>(p.w, p.w_stride));
    return cudaGetLastError();
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
constexpr int SH_ROWS = 64;      // rows a CTA looks through for its slot
constexpr int SH_PAIR = 16;      // rows whose sums are joined at a time

__device__ __forceinline__ void grid_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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

// Grid: 16-rank groups, by slots (or, for more than SH_ROWS of them, the u-th
// distinct slot of the chunk), by 64-row chunks. Each thread multiplies 8
// consecutive k of two rank rows and of the slot's rows at a time: which k a
// fragment's slots mean is free as long as both operands agree.
__global__ void __launch_bounds__(SH_THREADS) mx4_shrink_kernel(Mx4ProjParams p)
{
    __shared__ uint32_t present[MAX_BUCKETS / 32];
    __shared__ int slot_s, rows_s[SH_ROWS];
    __shared__ float red[SH_WARPS][16][SH_PAIR + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int r0 = blockIdx.x * 16, u = blockIdx.y, c0 = blockIdx.z * SH_ROWS;
    // Launched early behind whatever the stream ran before; nothing is read
    // until that is complete, and only then may the projection kernel start.
    grid_dependency_wait();
    grid_dependents_launch();
    const int mine = tid < SH_ROWS && c0 + tid < p.M ? p.seq_slot[c0 + tid] : -1;
    SlotInfo si;
    int slot = u;
    if (p.L <= SH_ROWS)
        si = slot_info(p.tab, slot, p.L); // on its way with the rows' slots
    if (blockIdx.x == 0 && u == 0 && c0 == 0) { // the call's status
        int bad = 0;
        for (int i = tid; i < p.M; i += SH_THREADS)
            bad |= p.seq_slot[i] >= p.L;
        bad = __syncthreads_or(bad);
        if (tid == 0)
            status_begin(p.status, bad ? (uint32_t)LORA_FLAG_SLOT_RANGE : 0u);
    }
    if (p.L > SH_ROWS) { // the u-th distinct slot among the chunk's rows
        present[lane] = 0u;
        if (tid == 0)
            slot_s = -1;
        __syncthreads();
        if (mine >= 0 && mine < p.L)
            atomicOr(&present[mine >> 5], 1u << (mine & 31));
        __syncthreads();
        if (warp == 0) {
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
        slot = slot_s;
        if (slot < 0)
            return;
        si = slot_info(p.tab, slot, p.L);
    }
    if (!si.on || r0 >= si.rank)
        return;
    if (tid < SH_ROWS) { // the slot's rows, in order
        const uint32_t m = __ballot_sync(0xffffffffu, mine == slot);
        if (lane == 0)
            present[warp] = m;
    }
    __syncthreads();
    if (tid < SH_ROWS && mine == slot)
        rows_s[(warp == 1 ? __popc(present[0]) : 0) + __popc(present[warp] & ((1u << lane) - 1u))] = c0 + tid;
    const int count = __popc(present[0]) + __popc(present[1]);
    __syncthreads();
    if (count == 0)
        return;
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
                const size_t at = (size_t)rows_s[i0 + row] * p.R + r0 + q;
                p.h[at] = v;
                p.hs[at] = f32_to_bf16_bits(v);
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

cudaError_t launch_mx4_shrink(const Mx4ProjParams &p, cudaStream_t st)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int distinct = p.M < SH_ROWS ? p.M : SH_ROWS; // at most, in a chunk
    cfg.gridDim = dim3((unsigned)((p.R + 15) / 16), (unsigned)(p.L <= SH_ROWS ? p.L : distinct),
                       (unsigned)((p.M + SH_ROWS - 1) / SH_ROWS));
    cfg.blockDim = dim3(SH_THREADS);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mx4_shrink_kernel, p);
}

// ------------------------------------------------------------------ stream
namespace {

constexpr int ST_THREADS = 256;           // 8 warps, 16 features each
constexpr int ST_FEATURES = 128;
constexpr int ST_DEPTH = 6;               // 128-wide k chunks of codes in flight
constexpr uint32_t ST_RING = ST_DEPTH * 2 * ST_THREADS * 16;
constexpr uint32_t ST_X_BYTES = 96 * 1024; // x of a pass over part of K, at most
constexpr int ST_TILE = ST_FEATURES + 4;  // floats of a token's row of the partial tile

// Bytes of a token's x row over `chunks` chunks: every 64-byte block is
// followed by 16 spare bytes, and rows lie 4 (mod 8) 16-byte units apart, so
// that the eight lanes of a load phase touch eight different bank groups.
__host__ __device__ inline uint32_t st_x_stride(int chunks)
{
    uint32_t u = (uint32_t)chunks * 20u;
    u += (4u + 8u - u % 8u) % 8u;
    return u * 16u;
}

// Chunks of K a pass may stage for nt token tiles of 8.
inline int st_pass_chunks(int nt)
{
    int c = 1;
    while (c < 64 && (uint32_t)(nt * 8) * st_x_stride(c + 1) <= ST_X_BYTES)
        ++c;
    return c;
}

__device__ __forceinline__ uint4 lds_16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Scale bytes of 128 weight rows, blocks [b0, b0 + n) of each (zero past K), to
// sc[row][n padded to 4]; W bytes an access, which the caller has checked for
// alignment. Eight accesses of a thread are in flight at a time.
template <typename W>
__device__ __forceinline__ void stage_scales(const uint8_t *scales, int nblk, int N, int f0, int b0, int n, uint8_t *sc,
                                             int scs, int tid)
{
    constexpr int B = sizeof(W);
    const int each = (n + B - 1) / B, total = ST_FEATURES * each;
    for (int i0 = tid; i0 < total; i0 += 8 * ST_THREADS) {
        W v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * ST_THREADS, r = i / each, b = (i - r * each) * B;
            v[u] = W{};
            if (i < total && b0 + b < nblk)
                v[u] = __ldg(reinterpret_cast<const W *>(scales + (size_t)min(f0 + r, N - 1) * nblk + b0 + b));
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * ST_THREADS, r = i / each, b = (i - r * each) * B;
            if (i < total)
                *reinterpret_cast<W *>(sc + r * scs + b) = v[u];
        }
    }
}

// Two blocks' worth of a row pair's codes in registers -> bf16, times their scales.
struct Widen {
    uint32_t fa1, fa2, fb1, fb2;
    bool twice;
    __device__ __forceinline__ Widen(uint32_t sa, uint32_t sb)
    {
        mx4_factors(sa, fa1, fa2);
        mx4_factors(sb, fb1, fb2);
        twice = __any_sync(0xffffffffu, sa > MX4_ONE_FACTOR || sb > MX4_ONE_FACTOR);
    }
    __device__ __forceinline__ void operator()(uint32_t a, uint32_t b, uint32_t (&u)[4], uint32_t (&v)[4]) const
    {
        mx4_unpack8(a, u);
        mx4_unpack8(b, v);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            u[q] = mul_bf16x2(u[q], fa1);
            v[q] = mul_bf16x2(v[q], fb1);
        }
        if (twice) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                u[q] = mul_bf16x2(u[q], fa2);
                v[q] = mul_bf16x2(v[q], fb2);
            }
        }
    }
};

} // namespace

// Grid: (feature tiles of 128) x kparts, by token tiles of 8 NT; the kparts
// CTAs of a tile are a cluster, and each finishes 128 / kparts features.
template <int NT>
__global__ void __launch_bounds__(ST_THREADS) mx4_stream_kernel(Mx4ProjParams p, int kparts, int pass_chunks)
{
    constexpr int TOK = NT * 8;
    extern __shared__ __align__(128) uint8_t st_smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int part = blockIdx.x % kparts, f0 = (blockIdx.x / kparts) * ST_FEATURES, t0 = blockIdx.y * TOK;
    const int nblk = p.K / 32, nch = (nblk + 3) / 4, per = (nch + kparts - 1) / kparts;
    const int cb = min(nch, part * per), ce = min(nch, cb + per);
    const int fs = ST_FEATURES / kparts, fb = part * fs; // the features this CTA finishes
    const uint32_t xstr = st_x_stride(pass_chunks);
    const uint32_t smem = smem_u32(st_smem);
    const uint32_t ring = smem + tid * 16;
    const uint32_t xs = smem + ST_RING;
    uint8_t *sc = st_smem + ST_RING + (uint32_t)TOK * xstr; // [128][4 pass_chunks] scale bytes
    const int scs = (4 * pass_chunks + 15) & ~15;

    // this thread's two weight rows (rows past N repeat the last; their sums are dropped)
    const int fa = f0 + warp * 16 + g;
    const uint8_t *wa = p.codes + (size_t)min(fa, p.N - 1) * (p.K / 2) + t * 16;
    const uint8_t *wb = p.codes + (size_t)min(fa + 8, p.N - 1) * (p.K / 2) + t * 16;
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[n][i] = 0.0f;

    auto fetch = [&](int c, int slot) { // codes of chunk c, zeros past K
        const uint32_t have = c * 4 + t < nblk ? 16u : 0u;
        const uint32_t d = ring + (uint32_t)slot * (2 * ST_THREADS * 16);
        cp16(d, have ? wa + (size_t)c * 64 : p.codes, have);
        cp16(d + ST_THREADS * 16, have ? wb + (size_t)c * 64 : p.codes, have);
    };

    for (int c0 = cb; c0 < ce; c0 += pass_chunks) {
        const int nc = min(pass_chunks, ce - c0);
        // the first chunks of codes, a group a chunk, also where there is none; x of
        // the pass (zeros past K and M) goes with the first
#pragma unroll
        for (int d = 0; d < ST_DEPTH - 1; ++d) {
            if (d < nc)
                fetch(c0 + d, d);
            if (d == 0) {
                for (int i = tid; i < TOK * nc * 16; i += ST_THREADS) {
                    const int tok = i / (nc * 16), q = i - tok * (nc * 16); // 16-byte piece q of the row
                    const int k = c0 * 128 + q * 8;
                    const bool have = t0 + tok < p.M && k < p.K;
                    cp16(xs + (uint32_t)tok * xstr + (uint32_t)((q >> 2) * 80 + (q & 3) * 16),
                         have ? p.x + (int64_t)(t0 + tok) * p.x_stride + k : p.x, have ? 16u : 0u);
                }
            }
            cp_async_commit();
        }
        if (nblk % 16 == 0 && nc % 4 == 0 && c0 % 4 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 15u) == 0)
            stage_scales<uint4>(p.scales, nblk, p.N, f0, c0 * 4, nc * 4, sc, scs, tid);
        else if (nblk % 4 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 3u) == 0)
            stage_scales<uint32_t>(p.scales, nblk, p.N, f0, c0 * 4, nc * 4, sc, scs, tid);
        else
            stage_scales<uint8_t>(p.scales, nblk, p.N, f0, c0 * 4, nc * 4, sc, scs, tid);
        cp_async_wait_group<ST_DEPTH - 2>();
        __syncthreads();
        for (int i = 0, slot = 0; i < nc; ++i) {
            cp_async_wait_group<ST_DEPTH - 2>();
            const uint4 a = lds_16(ring + (uint32_t)slot * (2 * ST_THREADS * 16));
            const uint4 b = lds_16(ring + (uint32_t)slot * (2 * ST_THREADS * 16) + ST_THREADS * 16);
            const int ahead = i + ST_DEPTH - 1;
            if (ahead < nc)
                fetch(c0 + ahead, slot == 0 ? ST_DEPTH - 1 : slot - 1);
            cp_async_commit();
            slot = slot + 1 == ST_DEPTH ? 0 : slot + 1;
            const Widen widen(sc[(warp * 16 + g) * scs + i * 4 + t], sc[(warp * 16 + g + 8) * scs + i * 4 + t]);
            const uint32_t xa = xs + (uint32_t)g * xstr + (uint32_t)(i * 4 + t) * 80;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t u[4], v[4];
                widen(j == 0 ? a.x : j == 1 ? a.y : j == 2 ? a.z : a.w, j == 0 ? b.x : j == 1 ? b.y : j == 2 ? b.z : b.w, u, v);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 xb = lds_16(xa + (uint32_t)(n * 8) * xstr + (uint32_t)j * 16);
                    mma_16816(acc[n], u[0], v[0], u[1], v[1], xb.x, xb.y);
                    mma_16816(acc[n], u[2], v[2], u[3], v[3], xb.z, xb.w);
                }
            }
        }
        __syncthreads(); // x and the scales are overwritten
    }
    cp_async_wait_all();
    __syncthreads();

    // ---- partial tile, [token][128 + 4]; then s comp h of the tile's rows, [token][R], and the delta, [token][fs]
    float *tile = reinterpret_cast<float *>(st_smem);
    float *hs = tile + TOK * ST_TILE;
    float *delta = hs + TOK * p.R;
    __shared__ const uint16_t *brow_s[TOK]; // B of a row's slot, nullptr: no delta
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int f = warp * 16 + g, tok = n * 8 + 2 * t;
        tile[tok * ST_TILE + f] = acc[n][0];
        tile[(tok + 1) * ST_TILE + f] = acc[n][1];
        tile[tok * ST_TILE + f + 8] = acc[n][2];
        tile[(tok + 1) * ST_TILE + f + 8] = acc[n][3];
    }
    if (kparts > 1)
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    grid_dependency_wait(); // h is complete
    const int rows = min(TOK, p.M - t0);
#pragma unroll 4
    for (int i = tid; i < rows * p.R; i += ST_THREADS) {
        const int tok = i / p.R, r = i - tok * p.R, slot = p.seq_slot[t0 + tok];
        const SlotInfo si = slot_info(p.tab, slot, p.L);
        if (r == 0)
            brow_s[tok] = si.on ? si.b : nullptr;
        float v = 0.0f;
        if (si.on && r < si.rank)
            v = __ldcg(p.h + (size_t)(t0 + tok) * p.R + r);
        hs[i] = v;
    }
    __syncthreads();
    // a B row is `pieces` 16-byte pieces, a lane each: one row, or several
    const int pieces = p.R / 8;
    int lanes = 1;
    while (lanes < pieces)
        lanes *= 2;
    const int sub = lane & (lanes - 1), each = 32 / lanes;
    constexpr int AT_ONCE = 8;
    for (int i0 = warp * each; i0 < rows * fs; i0 += (ST_THREADS / 32) * each * AT_ONCE) {
        uint4 b[AT_ONCE];
        int tok[AT_ONCE];
#pragma unroll
        for (int a = 0; a < AT_ONCE; ++a) {
            const int i = i0 + a * (ST_THREADS / 32) * each + lane / lanes, f = i % fs;
            tok[a] = i / fs;
            const uint16_t *base = i < rows * fs && f0 + fb + f < p.N && sub < pieces ? brow_s[tok[a]] : nullptr;
            b[a] = make_uint4(0, 0, 0, 0);
            tok[a] = base != nullptr ? tok[a] : -1;
            if (base != nullptr)
                b[a] = ld_nc_16(base + (size_t)(f0 + fb + f) * p.R + sub * 8);
        }
#pragma unroll
        for (int a = 0; a < AT_ONCE; ++a) {
            const int i = i0 + a * (ST_THREADS / 32) * each + lane / lanes;
            float d = 0.0f;
            if (tok[a] >= 0) {
                const float4 *hp = reinterpret_cast<const float4 *>(hs + tok[a] * p.R + sub * 8);
                d = dot8_bf_f32(0.0f, b[a], hp[0], hp[1]);
            }
            for (int o = lanes / 2; o > 0; o >>= 1)
                d += __shfl_xor_sync(0xffffffffu, d, o);
            if (i < rows * fs && sub == 0)
                delta[i] = d;
        }
    }
    __syncthreads();
    if (kparts > 1)
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // ---- sum over the K parts (part order), the row's adapter, one rounding
    for (int i = tid; i < rows * fs; i += ST_THREADS) {
        const int tok = i / fs, f = i - tok * fs;
        if (f0 + fb + f >= p.N)
            continue;
        float v = 0.0f;
        if (kparts > 1) {
            cg::cluster_group cl = cg::this_cluster();
            for (int r = 0; r < kparts; ++r)
                v += cl.map_shared_rank(tile, r)[tok * ST_TILE + fb + f];
        } else {
            v = tile[tok * ST_TILE + f];
        }
        if (brow_s[tok] != nullptr) // else the base product to the bit
            v += delta[i];
        p.y[(int64_t)(t0 + tok) * p.y_stride + f0 + fb + f] = f32_to_bf16_bits(v);
    }
    if (kparts > 1)
        cg::this_cluster().sync(); // the parts' tiles are read until here
}

template <int NT> cudaError_t launch_st(const Mx4ProjParams &p, int num_sms, cudaStream_t st)
{
    const int tiles = (p.N + ST_FEATURES - 1) / ST_FEATURES, nch = (p.K / 32 + 3) / 4;
    const int ttiles = (p.M + NT * 8 - 1) / (NT * 8);
    int kparts = 1;
    while (kparts < 8 && tiles * kparts * ttiles < num_sms && nch >= 4 * kparts)
        kparts *= 2;
    int pass = st_pass_chunks(NT);
    const int per = (nch + kparts - 1) / kparts;
    pass = pass < per ? pass : per;
    uint32_t smem = ST_RING + (uint32_t)(NT * 8) * st_x_stride(pass) + ST_FEATURES * ((4 * (uint32_t)pass + 15) & ~15u);
    const uint32_t end = (uint32_t)(NT * 8) * (ST_TILE + p.R + ST_FEATURES / kparts) * 4;
    smem = smem > end ? smem : end;
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = raise_smem_limit(raised, mx4_stream_kernel<NT>, 224 * 1024);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)kparts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * kparts), (unsigned)ttiles);
    cfg.blockDim = dim3(ST_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mx4_stream_kernel<NT>, p, kparts, pass);
}

cudaError_t launch_mx4_stream(const Mx4ProjParams &p, int num_sms, cudaStream_t st)
{
    if (p.M <= 8)
        return launch_st<1>(p, num_sms, st);
    if (p.M <= 16)
        return launch_st<2>(p, num_sms, st);
    if (p.M <= 32)
        return launch_st<4>(p, num_sms, st);
    return launch_st<8>(p, num_sms, st);
}

} // namespace rd
