// Microscaled 4-bit matrices (lora_mx4.cu): what the host ABI hands to the
// kernels, and the conversions they share.
//
// A value is an E2M1 code (sign, two exponent bits, one mantissa bit: 0, 0.5,
// 1, 1.5, 2, 3, 4, 6) times the power of two 2^(byte - 127) that 32
// consecutive values of a row share. Byte 255 makes its block NaN.
#pragma once
#include "lora_internal.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace rd {

struct Mx4QuantParams {
    const void *w; // rows of K, row stride in elements
    int64_t w_stride;
    int64_t rows;
    int K;
    uint8_t *codes;  // [rows][K / 2]
    uint8_t *scales; // [rows][K / 32]
};

struct Mx4DequantParams {
    const uint8_t *codes, *scales;
    int64_t rows;
    int K;
    void *w;
    int64_t w_stride;
};

struct Mx4ProjParams {
    const uint16_t *x;
    int64_t x_stride;
    const uint8_t *codes, *scales;
    int M, K, N, L, R;
    const int32_t *seq_slot;
    Tables tab;
    // s comp (A_s x_i) of every adapted row, [M][R]: in fp32 for the rows kernel, or for
    // tiles (h null) as two bf16 whose sum it is to 2^-17 of itself
    float *h;
    uint16_t *hs, *ls;
    uint16_t *y;
    int64_t y_stride;
    uint32_t *status;
    // limit of a wait; test hook: 1, the adapters' stages (rows kernel: the steps' sums) wait
    // for an arrival that never comes; more, the base's do
    uint64_t wait_ns;
    int never;
};

cudaError_t launch_mx4_quantize(const Mx4QuantParams &p, int dtype, cudaStream_t st);
cudaError_t launch_mx4_dequantize(const Mx4DequantParams &p, int dtype, cudaStream_t st);
cudaError_t launch_mx4_shrink(const Mx4ProjParams &p, int num_sms, cudaStream_t st);
// Most rows of a call: tiles of rows, and chunks of the shrink, are a grid's y and z.
constexpr int MX4_MAX_ROWS = 65535 * 256;
// The product for up to four rows; `codes`: bytes [N][K / 2], boxes of 128 bytes x 16 rows, 128-byte swizzle.
bool mx4_rows_fit(int M, int K, int R);
cudaError_t launch_mx4_rows(const Mx4ProjParams &p, const CUtensorMap &codes, int num_sms, cudaStream_t st);
// The tiles of a tensor-core launch: rows of a token tile (the host encodes x
// in boxes of 64 k by that many rows) and K parts.
struct Mx4TcPlan {
    int tn, kparts;
};
Mx4TcPlan plan_mx4_tc(const Mx4ProjParams &p, int num_sms);
struct Mx4TcMaps {
    CUtensorMap x;      // boxes of 64 k x tn rows, 128-byte swizzle
    CUtensorMap codes;  // bytes [N][K / 2], boxes of 128 bytes x 128 rows, 128-byte swizzle
    CUtensorMap scales; // bytes [N][K / 32], boxes of 16 bytes x 128 rows, when rows lie 16 bytes apart
    int scales_ok;      // 1: encoded
};
cudaError_t launch_mx4_tc(const Mx4ProjParams &p, const Mx4TcPlan &plan, const Mx4TcMaps &maps, cudaStream_t st);

// An element of h to where the call's product takes it from. One bf16 would be
// 2^-9 off, as much as the rounding of y itself; the second takes that up. (A value past
// the largest bf16 stays finite; an infinity or a NaN is in the first alone.)
__device__ __forceinline__ void store_h(const Mx4ProjParams &p, size_t at, float v)
{
    if (p.h != nullptr) {
        p.h[at] = v;
        return;
    }
    uint16_t hi = f32_to_bf16_bits(v);
    const bool finite = (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
    if (finite && (hi & 0x7FFFu) == 0x7F80u)
        --hi;
    p.hs[at] = hi;
    p.ls[at] = finite ? f32_to_bf16_bits(v - __uint_as_float((uint32_t)hi << 16)) : (uint16_t)0;
}

// Wait for a phase, at most `limit` ns, or (`heed`) until another wait of the CTA has given
// up; false: not complete, and noted. The clock is read only every 256 polls
// from the first on (a read of it takes longer than a stage).
__device__ __forceinline__ bool wait_or_note(uint64_t *bar, uint32_t parity, int *bad, uint64_t limit, bool heed = true)
{
    const uint32_t a = smem_u32(bar);
    uint64_t t0 = 0;
    for (uint32_t i = 1; !mbar_try_wait(a, parity); ++i) {
        if ((i & 255u) != 0)
            continue;
        const uint64_t t = globaltimer_ns();
        t0 = t0 == 0 ? t : t0;
        if (t - t0 > limit || (heed && *reinterpret_cast<volatile int *>(bad) != 0)) {
            *reinterpret_cast<volatile int *>(bad) = 1;
            return false;
        }
    }
    return true;
}
// The same for a whole warp, which goes on together.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int *bad, uint64_t limit)
{
    const uint32_t a = smem_u32(bar);
    uint64_t t0 = 0;
    for (uint32_t i = 1; !__all_sync(0xffffffffu, mbar_try_wait(a, parity)); ++i) {
        if ((i & 255u) != 0)
            continue;
        const uint64_t t = globaltimer_ns();
        t0 = t0 == 0 ? t : t0;
        if (__any_sync(0xffffffffu, t - t0 > limit || *reinterpret_cast<volatile int *>(bad) != 0)) {
            *reinterpret_cast<volatile int *>(bad) = 1;
            return false;
        }
    }
    return true;
}

// One lane of the converged warp, by the instruction that tells the compiler so:
// what follows in its branch needs no loop over lanes that might differ (with
// lane == 0 instead a product took 80 cycles to issue, and 8192x4096x14336 8 % longer).
__device__ __forceinline__ bool elected()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.b32 %0, 1, 0, e;\n\t}" : "=r"(one));
    return one != 0u;
}

// The bf16 factors that turn value * 2^-126 (what mx4_unpack8 gives) into value
// * 2^(byte - 127). The second is 1 unless the first would leave bf16's range
// (byte > MX4_ONE_FACTOR).
constexpr uint32_t MX4_ONE_FACTOR = 128;
__device__ __forceinline__ void mx4_factors(uint32_t byte, uint32_t &f1, uint32_t &f2)
{
    const uint32_t e = byte + 126u;
    const uint32_t a = e < 254u ? e : 254u;
    f1 = a << 7;
    f2 = (127u + e - a) << 7;
    if (byte == 255u)
        f1 = 0x7FC0u;
    f1 |= f1 << 16;
    f2 |= f2 << 16;
}

// The first of them alone, for byte <= MX4_ONE_FACTOR: twice (byte + 126) << 7.
__device__ __forceinline__ uint32_t mx4_factor(uint32_t byte) { return byte * 0x00800080u + 0x3F003F00u; }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <uint32_t SELECT> __device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "n"(SELECT));
    return r;
}

// Eight codes (the lowest four bits first) as bf16 pairs in order, each value
// times 2^-126: a code's three magnitude bits become the two lowest exponent
// bits and the highest fraction bit (0.5 is a subnormal), its sign bit 15. The
// even and the odd codes are set apart, a pair's two are put at the bottom of
// the halves of a word (byte selectors 8.. replicate a sign bit, here zeros),
// and one product by 2^12 + 2^6 brings both to both places.
__device__ __forceinline__ void mx4_unpack8(uint32_t w, uint32_t (&o)[4])
{
    const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
    o[0] = prmt<0x8480>(even, odd);
    o[1] = prmt<0x8581>(even, odd);
    o[2] = prmt<0x8682>(even, odd);
    o[3] = prmt<0x8783>(even, odd);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = (o[i] * 0x1040u) & 0x81C081C0u;
}

} // namespace rd
