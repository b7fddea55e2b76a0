// Microscaled 4-bit matrices: quantisation, reading back, and the projection
//   y[i, :] = dq(W) x_i + s B_s (A_s x_i)
// with the base W in that form and each row's adapter in bf16.
//
// quantize   a thread takes 8 consecutive values, four threads share a block:
//            its scale is 2^(floor(log2 max) - 2), read off the exponent field,
//            so the largest code is 4 or 6; codes are rounded to nearest even
//            and saturate. One pass: bound by HBM.
// dequantize the reverse, one 16-byte store a thread and step.
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

template <typename T> struct In8;
template <> struct In8<uint16_t> {
    static __device__ __forceinline__ void load(const uint16_t *p, bool vec, float (&f)[8])
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
    static __device__ __forceinline__ void store(uint16_t *p, bool vec, const float (&f)[8])
    {
        if (vec) {
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
            *reinterpret_cast<uint4 *>(p) = make_uint4(r[0], r[1], r[2], r[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i] = f32_to_bf16_bits(f[i]);
        }
    }
};
template <> struct In8<float> {
    static __device__ __forceinline__ void load(const float *p, bool vec, float (&f)[8])
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
    static __device__ __forceinline__ void store(float *p, bool vec, const float (&f)[8])
    {
        if (vec) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i] = f[i];
        }
    }
};

// Element offset of unit u (8 values) of a matrix of K / 8 = upr units a row.
__device__ __forceinline__ int64_t unit_offset(int64_t u, int upr, int64_t stride, bool packed)
{
    if (packed)
        return u * 8;
    const int64_t row = u / upr;
    return row * stride + (u - row * upr) * 8;
}

} // namespace

template <typename T> __global__ void __launch_bounds__(Q_THREADS) mx4_quantize_kernel(Mx4QuantParams p, int vec)
{
    const int upr = p.K / 8;
    const int64_t total = p.rows * upr; // a multiple of 4: the threads of a block go together
    const bool packed = p.w_stride == p.K;
    const T *w = static_cast<const T *>(p.w);
    for (int64_t u0 = (int64_t)blockIdx.x * (Q_THREADS * Q_UNROLL) + threadIdx.x; u0 - threadIdx.x < total;
         u0 += (int64_t)gridDim.x * (Q_THREADS * Q_UNROLL)) {
        float f[Q_UNROLL][8];
#pragma unroll
        for (int q = 0; q < Q_UNROLL; ++q) {
            const int64_t u = u0 + q * Q_THREADS;
            if (u < total) {
                In8<T>::load(w + unit_offset(u, upr, p.w_stride, packed), vec, f[q]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    f[q][i] = 0.0f;
            }
        }
#pragma unroll
        for (int q = 0; q < Q_UNROLL; ++q) {
            const int64_t u = u0 + q * Q_THREADS;
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = absmax_nan(m, f[q][i]);
            m = absmax_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = absmax_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t e = __float_as_uint(m) >> 23; // 255: an infinity or a NaN
            const uint32_t byte = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
            const float up = __uint_as_float((254u - byte) << 23); // 2^(127 - byte); byte <= 252 here
            uint32_t c = 0u;
            if (byte != 255u) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    c |= e2m1_pair(f[q][2 * i] * up, f[q][2 * i + 1] * up) << (8 * i);
            }
            if (u < total) {
                reinterpret_cast<uint32_t *>(p.codes)[u] = c;
                if ((u & 3) == 0)
                    p.scales[u >> 2] = (uint8_t)byte;
            }
        }
    }
}

template <typename T> __global__ void __launch_bounds__(Q_THREADS) mx4_dequantize_kernel(Mx4DequantParams p, int vec)
{
    const int upr = p.K / 8;
    const int64_t total = p.rows * upr;
    const bool packed = p.w_stride == p.K;
    T *w = static_cast<T *>(p.w);
    for (int64_t u0 = (int64_t)blockIdx.x * (Q_THREADS * Q_UNROLL) + threadIdx.x; u0 < total;
         u0 += (int64_t)gridDim.x * (Q_THREADS * Q_UNROLL)) {
        uint32_t c[Q_UNROLL], b[Q_UNROLL];
#pragma unroll
        for (int q = 0; q < Q_UNROLL; ++q) {
            const int64_t u = u0 + q * Q_THREADS;
            c[q] = u < total ? __ldg(reinterpret_cast<const uint32_t *>(p.codes) + u) : 0u;
            b[q] = u < total ? __ldg(p.scales + (u >> 2)) : 0u;
        }
#pragma unroll
        for (int q = 0; q < Q_UNROLL; ++q) {
            const int64_t u = u0 + q * Q_THREADS;
            if (u >= total)
                break;
            // 2^(byte - 127); byte 0 is the subnormal 2^-127
            const float s = b[q] == 255u ? __uint_as_float(0x7FC00000u)
                                         : __uint_as_float(b[q] == 0u ? 1u << 22 : b[q] << 23);
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) { // fp16's layout: exponent bias 15
                const uint32_t n = (c[q] >> (4 * i)) & 15u;
                const uint32_t mag = n & 7u;
                const float v = mag < 2u ? 0.5f * (float)mag
                                         : __uint_as_float(((126u + (mag >> 1)) << 23) | ((mag & 1u) << 22));
                f[i] = (n & 8u ? -v : v) * s;
            }
            In8<T>::store(w + unit_offset(u, upr, p.w_stride, packed), vec, f);
        }
    }
}

namespace {

int quant_blocks(int64_t units, int num_sms)
{
    const int64_t need = (units + Q_THREADS * Q_UNROLL - 1) / (Q_THREADS * Q_UNROLL);
    const int64_t cap = (int64_t)num_sms * 8;
    return (int)(need < cap ? need : cap);
}

template <typename T> bool vec_rows(const void *w, int64_t stride)
{
    return (reinterpret_cast<uintptr_t>(w) & 15u) == 0 && (stride * sizeof(T)) % 16 == 0;
}

} // namespace

cudaError_t launch_mx4_quantize(const Mx4QuantParams &p, int dtype, int num_sms, cudaStream_t st)
{
    const int blocks = quant_blocks(p.rows * (p.K / 8), num_sms);
    if (dtype == LORA_DTYPE_F32)
        mx4_quantize_kernel<float><<<blocks, Q_THREADS, 0, st>>>(p, vec_rows<float>(p.w, p.w_stride));
    else
        mx4_quantize_kernel<uint16_t><<<blocks, Q_THREADS, 0, st>>>(p, vec_rows<uint16_t>(p.w, p.w_stride));
    return cudaGetLastError();
}

cudaError_t launch_mx4_dequantize(const Mx4DequantParams &p, int dtype, int num_sms, cudaStream_t st)
{
    const int blocks = quant_blocks(p.rows * (p.K / 8), num_sms);
    if (dtype == LORA_DTYPE_F32)
        mx4_dequantize_kernel<float><<<blocks, Q_THREADS, 0, st>>>(p, vec_rows<float>(p.w, p.w_stride));
    else
        mx4_dequantize_kernel<uint16_t><<<blocks, Q_THREADS, 0, st>>>(p, vec_rows<uint16_t>(p.w, p.w_stride));
    return cudaGetLastError();
}

// ------------------------------------------------------------------ stream
namespace {

constexpr int ST_THREADS = 256;           // 8 warps, 16 features each
constexpr int ST_FEATURES = 128;
constexpr int ST_DEPTH = 6;               // 128-wide k chunks of codes in flight
constexpr uint32_t ST_RING = ST_DEPTH * 2 * ST_THREADS * 16;
constexpr uint32_t ST_X_BYTES = 96 * 1024; // x of a pass over part of K, at most

// Bytes of a token's x row over `chunks` chunks: every 64-byte block is
// followed by 16 spare bytes, and rows lie 4 (mod 8) 16-byte units apart, so
// that the eight lanes of a load phase touch eight different bank groups.
__host__ __device__ inline uint32_t st_x_stride(int chunks)
{
    uint32_t u = (uint32_t)chunks * 20u;
    u += (4u + 8u - u % 8u) % 8u;
    return u * 16u;
}

// Chunks of K a pass may stage for nt tokens tiles of 8.
inline int st_pass_chunks(int nt)
{
    int c = 1;
    while (c < 64 && (uint32_t)(nt * 8) * st_x_stride(c + 1) <= ST_X_BYTES)
        ++c;
    return c;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds_16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

} // namespace

// Grid: (feature tiles of 128) x kparts, by token tiles of 8 NT; the kparts
// CTAs of a tile are a cluster, and each finishes 128 / kparts features.
template <int NT>
__global__ void __launch_bounds__(ST_THREADS) mx4_stream_kernel(Mx4ProjParams p, int kparts, int pass_chunks)
{
    extern __shared__ __align__(128) uint8_t st_smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int part = blockIdx.x % kparts, f0 = (blockIdx.x / kparts) * ST_FEATURES, t0 = blockIdx.y * (NT * 8);
    const int nblk = p.K / 32, nch = (nblk + 3) / 4, per = (nch + kparts - 1) / kparts;
    const int cb = min(nch, part * per), ce = min(nch, cb + per);
    const uint32_t xstr = st_x_stride(pass_chunks);
    const uint32_t smem = smem_u32(st_smem);
    const uint32_t ring = smem + tid * 16;
    const uint32_t xs = smem + ST_RING;
    uint8_t *sc = st_smem + ST_RING + (uint32_t)(NT * 8) * xstr; // [128][4 pass_chunks] scale bytes
    const int scs = 4 * pass_chunks;

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
        const size_t o = (size_t)c * 64;
        const uint32_t d = ring + (uint32_t)slot * (2 * ST_THREADS * 16);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(have ? wa + o : p.codes), "r"(have) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + ST_THREADS * 16), "l"(have ? wb + o : p.codes), "r"(have) : "memory");
    };

    for (int c0 = cb; c0 < ce; c0 += pass_chunks) {
        const int nc = min(pass_chunks, ce - c0);
        // x of the pass (zeros past K and M), then the first chunks of codes
        for (int i = tid; i < NT * 8 * nc * 16; i += ST_THREADS) {
            const int tok = i / (nc * 16), q = i - tok * (nc * 16); // 16-byte piece q of the row
            const int k = c0 * 128 + q * 8;
            const bool have = t0 + tok < p.M && k < p.K;
            const uint16_t *src = have ? p.x + (int64_t)(t0 + tok) * p.x_stride + k : p.x;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             xs + (uint32_t)tok * xstr + (uint32_t)((q >> 2) * 80 + (q & 3) * 16)),
                         "l"(src), "r"(have ? 16u : 0u)
                         : "memory");
        }
        cp_async_commit();
#pragma unroll
        for (int d = 0; d < ST_DEPTH - 1; ++d) { // a group a chunk, also where there is none
            if (d < nc)
                fetch(c0 + d, d);
            cp_async_commit();
        }
        for (int i = tid; i < ST_FEATURES * nc * 4; i += ST_THREADS) {
            const int r = i / (nc * 4), b = i - r * (nc * 4);
            sc[r * scs + b] = c0 * 4 + b < nblk ? p.scales[(size_t)min(f0 + r, p.N - 1) * nblk + c0 * 4 + b] : (uint8_t)0;
        }
        cp_async_wait_group<ST_DEPTH - 1>();
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
            uint32_t fa1, fa2, fb1, fb2;
            const uint32_t sa = sc[(warp * 16 + g) * scs + i * 4 + t], sb = sc[(warp * 16 + g + 8) * scs + i * 4 + t];
            mx4_factors(sa, fa1, fa2);
            mx4_factors(sb, fb1, fb2);
            const bool twice = sa > 142u || sb > 142u;
            const uint32_t xa = xs + (uint32_t)g * xstr + (uint32_t)(i * 4 + t) * 80;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t u[4], v[4];
                mx4_unpack8(j == 0 ? a.x : j == 1 ? a.y : j == 2 ? a.z : a.w, u);
                mx4_unpack8(j == 0 ? b.x : j == 1 ? b.y : j == 2 ? b.z : b.w, v);
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

    // ---- partial tile to shared memory: [token][128 + 4]
    float *tile = reinterpret_cast<float *>(st_smem);
    constexpr int TS = ST_FEATURES + 4;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int f = warp * 16 + g, tok = n * 8 + 2 * t;
        tile[tok * TS + f] = acc[n][0];
        tile[(tok + 1) * TS + f] = acc[n][1];
        tile[tok * TS + f + 8] = acc[n][2];
        tile[(tok + 1) * TS + f + 8] = acc[n][3];
    }
    if (kparts > 1)
        cg::this_cluster().sync();
    else
        __syncthreads();
    // ---- sum over the K parts (part order), the row's adapter, one rounding
    const int fs = ST_FEATURES / kparts;
    for (int tok = warp; tok < NT * 8; tok += ST_THREADS / 32) {
        const int row = t0 + tok;
        if (row >= p.M)
            break;
        const int slot = p.seq_slot[row];
        const SlotInfo si = slot_info(p.tab, slot, p.L);
        const float *cr = p.tab.comp_table + (size_t)(si.on ? slot : 0) * LORA_COMP_STRIDE;
        for (int q = lane; q < fs; q += 32) {
            const int f = part * fs + q;
            if (f0 + f >= p.N)
                break;
            float v = 0.0f;
            if (kparts > 1) {
                cg::cluster_group cl = cg::this_cluster();
                for (int r = 0; r < kparts; ++r)
                    v += cl.map_shared_rank(tile, r)[tok * TS + f];
            } else {
                v = tile[tok * TS + f];
            }
            if (si.on) {
                const uint16_t *brow = si.b + (size_t)(f0 + f) * p.R;
                float d = 0.0f;
                for (int k = 0; k < si.rank; k += 8) {
                    float4 h0 = make_float4(0, 0, 0, 0), h1 = h0;
                    for (int u = 0; u < p.kp; ++u) {
                        const float4 *hp = reinterpret_cast<const float4 *>(p.h + ((size_t)u * p.M + row) * p.R + k);
                        const float4 a = hp[0], b = hp[1];
                        h0.x += a.x; h0.y += a.y; h0.z += a.z; h0.w += a.w;
                        h1.x += b.x; h1.y += b.y; h1.z += b.z; h1.w += b.w;
                    }
                    const float4 c0 = __ldg(reinterpret_cast<const float4 *>(cr + k));
                    const float4 c1 = __ldg(reinterpret_cast<const float4 *>(cr + k + 4));
                    h0.x *= c0.x; h0.y *= c0.y; h0.z *= c0.z; h0.w *= c0.w;
                    h1.x *= c1.x; h1.y *= c1.y; h1.z *= c1.z; h1.w *= c1.w;
                    d = dot8_bf_f32(d, ld_nc_16(brow + k), h0, h1);
                }
                v += si.scale * d;
            }
            p.y[(int64_t)row * p.y_stride + f0 + f] = f32_to_bf16_bits(v);
        }
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
    uint32_t smem = ST_RING + (uint32_t)(NT * 8) * st_x_stride(pass) + ST_FEATURES * 4 * (uint32_t)pass;
    const uint32_t tile = (uint32_t)(NT * 8) * (ST_FEATURES + 4) * 4;
    smem = smem > tile ? smem : tile;
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = raise_smem_limit(raised, mx4_stream_kernel<NT>, 224 * 1024);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)kparts;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * kparts), (unsigned)ttiles);
    cfg.blockDim = dim3(ST_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
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
