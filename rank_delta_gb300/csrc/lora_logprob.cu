// Log probabilities of given tokens, entropy, softmax statistics and the best
// alternatives of rows of logits, and the gradient of the first two.
//
// With z_v = x_v t (t = inv_temperature), m = max x, d_v = (x_v - m) t:
//   S = sum e^{d_v},  log p_v = d_v - log S,  H = log S - (sum e^{d_v} d_v) / S
// (S is carried as 1 + the rest, the 1 one element that is the maximum),
//   dx_v = t [ g (1[v = token] - p_v) - g_H p_v (log p_v + H) ].
//
// A row is read once: every thread keeps its maximum, and S and sum e^d d
// relative to a reference that trails the maximum by at most 2^8 (so both are
// rescaled rarely). Sums are fp32, e^d is the hardware's 2^x (about 2^-22
// relative). While one group of vectors is summed the next one, or the next
// row's first, is on its way.
//
// The best alternatives cost the pass nothing but the maximum it needs anyway:
// of the threads' own best elements the k-th largest is a lower bound of the
// row's k-th best, so only the (at most k) threads whose best reaches it can
// hold any of the k, and their shares, V / threads elements each, are read
// again from L2. Elements are compared by (value, lowest index first) packed
// into 64 bits, which orders them totally; -0 equals +0. What reaches the
// bound, k elements and a few, is then put in order.
//
// logprob_rows_kernel   many rows or short ones: a CTA takes whole rows, one after another;
//     eight warps read, a ninth (and tenth) finishes the row before while they are in the
//     next one, so neither the joins nor the alternatives stop the loads.
// logprob_short_kernel  many short rows: a warp takes a row.
// logprob_split_kernel  few long rows: a row is spread over a cluster of up to 8
//     CTAs, all warps finish it together, and the parts are joined through
//     distributed shared memory. Nothing depends on timing in either.
#include <cooperative_groups.h>

#include "behind.cuh"
#include "lora_logprob.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace rd {

namespace cg = cooperative_groups;

namespace {

constexpr int LP_THREADS = 256;     // gradient, and rows spread over a cluster
constexpr int LP_WARPS = LP_THREADS / 32;
// Whole rows: reading threads of a CTA (one warp more finishes), CTAs resident
// a SM and 16-byte vectors of a thread in flight. 256 x 3 x 4 reads 8192 rows
// of 32000 bf16 in 91 us; 128 x 6 took 68 % longer, 192 x 4 9, 384 x 2 16, 512 x
// 2 65 (small groups scatter the reads, large ones leave a row two steps).
constexpr int ROW_READERS = 256;
constexpr int ROW_THREADS = ROW_READERS + 32;
constexpr int ROW_CTAS = 3;
constexpr int LP_UNROLL = 4;
constexpr int SHORT_VECS = 1024;    // of a row that one warp takes where there are many
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7fc00000u); }

// max that lets a NaN through (a row that holds one has no distribution)
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float exp2_fast(float a)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}

// Two fp32 operations an instruction.
struct f2 {
    unsigned long long v;
};
__device__ __forceinline__ f2 make_f2(float a, float b)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split_f2(f2 p, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ f2 add_f2(f2 a, f2 b)
{
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 mul_f2(f2 a, f2 b)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 fma_f2(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// A 16-byte vector of T: E elements, widened to fp32.
template <typename T> struct Vec;
template <> struct Vec<uint16_t> {
    static constexpr int E = 8;
    static __device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ void unpack(const uint4 &q, float (&f)[8])
    {
        f[0] = bf_lo(q.x); f[1] = bf_hi(q.x); f[2] = bf_lo(q.y); f[3] = bf_hi(q.y);
        f[4] = bf_lo(q.z); f[5] = bf_hi(q.z); f[6] = bf_lo(q.w); f[7] = bf_hi(q.w);
    }
    static __device__ __forceinline__ uint32_t pair(float lo, float hi)
    {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8])
    {
        return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
    }
    static __device__ __forceinline__ uint16_t narrow(float v) { return f32_to_bf16_bits(v); }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float largest(const uint4 &q)
    {
        const uint32_t m = max2(max2(q.x, q.y), max2(q.z, q.w));
        return max_nan(bf_lo(m), bf_hi(m));
    }
};
template <> struct Vec<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ float widen(float v) { return v; }
    static __device__ __forceinline__ void unpack(const uint4 &q, float (&f)[4])
    {
        f[0] = __uint_as_float(q.x); f[1] = __uint_as_float(q.y);
        f[2] = __uint_as_float(q.z); f[3] = __uint_as_float(q.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4])
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ float narrow(float v) { return v; }
    static __device__ __forceinline__ float largest(const uint4 &q)
    {
        return max_nan(max_nan(__uint_as_float(q.x), __uint_as_float(q.y)),
                       max_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
    }
};

// Elements of a row's first 16-byte vector that lie before the row.
template <typename T> __device__ __forceinline__ int row_lead(const T *row)
{
    return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

// Vector c of a row (elements [c E - lead, c E - lead + E)), read past L1;
// elements outside the row are -infinity and not read.
template <typename T> __device__ __forceinline__ uint4 load_vec(const T *row, int V, int lead, int c)
{
    constexpr int E = Vec<T>::E;
    const int i0 = c * E - lead;
    if (i0 >= 0 && i0 + E <= V) {
        uint4 q;
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                     : "l"(row + i0));
        return q;
    }
    float f[E];
#pragma unroll
    for (int q = 0; q < E; ++q)
        f[q] = i0 + q >= 0 && i0 + q < V ? Vec<T>::widen(row[i0 + q]) : neg_inf();
    return Vec<T>::pack(f); // exact: the values came from T
}

template <typename T> __device__ __forceinline__ uint4 empty_vec()
{
    const uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(w, w, w, w);
}

// (value, index) as one number: larger value first, then the lower index. 0
// is below every finite element.
__device__ __forceinline__ unsigned long long order_key(float v, int idx)
{
    const uint32_t b = __float_as_uint(v + 0.0f); // -0 -> +0
    const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
    return (unsigned long long)k << 32 | (0xFFFFFFFFu - (uint32_t)idx);
}
__device__ __forceinline__ float key_value(unsigned long long c)
{
    const uint32_t k = (uint32_t)(c >> 32);
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ int key_index(unsigned long long c) { return (int)(0xFFFFFFFFu - (uint32_t)c); }

__device__ __forceinline__ unsigned long long warp_max_key(unsigned long long c)
{
    const uint32_t hi = (uint32_t)(c >> 32);
    const uint32_t mh = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t ml = __reduce_max_sync(0xffffffffu, hi == mh ? (uint32_t)c : 0u);
    return (unsigned long long)mh << 32 | ml;
}

// The lanes' keys in descending order.
__device__ __forceinline__ unsigned long long warp_sort_desc(unsigned long long c, int lane)
{
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const unsigned long long o = __shfl_xor_sync(0xffffffffu, c, j);
            const bool want_max = ((lane & j) == 0) == ((lane & k) == 0);
            c = want_max == (o > c) ? o : c;
        }
    return c;
}

// Statistics of part of a row: maximum, sum of 2^a and sum of 2^a a with
// a = (x - maximum) t log2 e.
struct Stat {
    float m, s, u;
};

// Factor and shift of a part with maximum m in a whole with maximum top.
__device__ __forceinline__ void rescale(Stat &st, float top, float c)
{
    const float mm = top == neg_inf() ? 0.0f : top;
    // a part without elements (m = -inf) holds s = u = 0
    const float d = st.m == neg_inf() ? 0.0f : max_nan((st.m - mm) * c, -1000.0f);
    const float f = exp2_fast(d);
    st.u = f * (st.u + d * st.s);
    st.s *= f;
    st.m = top;
}

__device__ __forceinline__ float warp_max_nan(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The lanes' parts as one, where a part's s leaves out one element that is its maximum (1
// itself): in a row that one element dominates, the sum of the others keeps its
// digits, log S is log1p of it, and the entropy, which is as small, is as good.
__device__ __forceinline__ Stat warp_join_rest(Stat st, float c)
{
    const float top = warp_max_nan(st.m);
    const int holder = __ffs(__ballot_sync(0xffffffffu, st.m == top)) - 1;
    if (st.m == neg_inf()) // no elements
        st.s = st.u = 0.0f;
    else if ((int)(threadIdx.x & 31) != holder) {
        st.s += 1.0f;
        rescale(st, top, c);
    }
    return Stat{top, warp_sum(st.s), warp_sum(st.u)};
}

// What a thread has summed of its elements, relative to a reference `at` that
// is one of them and trails the maximum `m` by at most 2^SLACK. For bf16 the
// difference to the reference and the scaling are one fused operation,
// a = x c - ref with ref = fl(at c), and masked elements are raised, two at a
// time, to a value whose power of two is 0 (so that 0 times their a is 0):
// that holds while at c is small enough for ref's rounding to be put right
// afterwards to first order and the raised value lies far enough below. Other
// rows (and fp32, which has half the elements a byte) take the difference
// first and clamp a.
constexpr float SLACK = 8.0f;

template <typename T> struct Sums {
    float m, at, limit, ref, c, drop, slack;
    bool fused;
    uint32_t low;         // the raised value, twice
    f2 s, u; // two sums each

    __device__ __forceinline__ void scale(float c_)
    {
        c = c_;
        drop = 400.0f / c_;
        slack = SLACK / c_;
    }
    __device__ __forceinline__ void clear()
    {
        m = at = limit = neg_inf();
        ref = 0.0f;
        fused = false;
        low = 0u;
        s = u = make_f2(0.0f, 0.0f);
    }
    // ref - at c, what the sums' origin is off by
    __device__ __forceinline__ float origin() const { return fused ? fmaf(-at, c, ref) : 0.0f; }

    // a new reference
    __device__ __forceinline__ void raise(float top)
    {
        const float old = origin(), from = at;
        at = top;
        ref = at * c;
        limit = at + slack;
        if (sizeof(T) == 2) {
            const uint32_t b = f32_to_bf16_bits(at - drop);
            const float raised = __uint_as_float(b << 16);
            low = b | b << 16;
            fused = fabsf(ref) <= 4096.0f && (raised - at) * c <= -150.0f && raised > neg_inf();
        }
        if (from != neg_inf()) {
            const float d = max_nan((from - at) * c + (old - origin()), -1000.0f);
            const float w = exp2_fast(d);
            const f2 d2 = make_f2(d, d), w2 = make_f2(w, w);
            u = mul_f2(w2, fma_f2(d2, s, u));
            s = mul_f2(w2, s);
        }
    }
    __device__ __forceinline__ void add_pair(f2 a)
    {
        float a0, a1;
        split_f2(a, a0, a1);
        const f2 e = make_f2(exp2_fast(a0), exp2_fast(a1));
        s = add_f2(s, e);
        u = fma_f2(e, a, u);
    }
    template <int N> __device__ __forceinline__ void add(const uint4 (&v)[N])
    {
        constexpr int E = Vec<T>::E;
        if (sizeof(T) == 2 && fused) {
            const f2 c2 = make_f2(c, c), r2 = make_f2(-ref, -ref);
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t x;
                    asm("max.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w[i]), "r"(low));
                    add_pair(fma_f2(make_f2(bf_lo(x), bf_hi(x)), c2, r2));
                }
            }
        } else {
            const float aa = at == neg_inf() ? 0.0f : at;
#pragma unroll
            for (int q = 0; q < N; ++q) {
                float f[E];
                Vec<T>::unpack(v[q], f);
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    add_pair(make_f2(max_nan((f[e] - aa) * c, -1000.0f), max_nan((f[e + 1] - aa) * c, -1000.0f)));
            }
        }
    }
    __device__ __forceinline__ Stat stat() const // relative to `at`
    {
        float s0, s1, u0, u1;
        split_f2(s, s0, s1);
        split_f2(u, u0, u1);
        Stat st{at, s0 + s1, u0 + u1};
        const float d = origin(); // at most 2^-13: 2^d is 1 + d ln 2
        st.u += d * st.s;
        st.u = fmaf(d * LN2, st.u, st.u);
        st.s = fmaf(d * LN2, st.s, st.s);
        return st;
    }
};

using Key = unsigned long long;
constexpr int FEW = 8; // up to so many alternatives are taken one by one, more are sorted

// How many of a descending list of 32 come before `k`.
__device__ __forceinline__ int count_before(const Key *list, Key k)
{
    int n = 0;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
        if (list[n + s - 1] > k)
            n += s;
    return n + (list[n] > k ? 1 : 0);
}

// The place of key [own][at] among all lists.
__device__ __forceinline__ int place(const Key (*lists)[32], int own, int at, Key k)
{
    int n = at;
#pragma unroll
    for (int l = 0; l < LP_WARPS; ++l)
        if (l != own)
            n += count_before(lists[l], k);
    return n;
}

// The k largest of the lanes' keys in descending order, lane by lane: for few
// by taking the largest k times, else by sorting.
__device__ __forceinline__ Key warp_top(Key c, int k, int lane)
{
    if (k > FEW)
        return warp_sort_desc(c, lane);
    Key mine = 0ull;
    for (int i = 0; i < k; ++i) {
        const Key best = warp_max_key(c);
        mine = lane == i ? best : mine;
        c = c == best ? 0ull : c; // keys are unique, or 0
    }
    return mine;
}

// The 32 largest of two descending lists.
__device__ __forceinline__ Key merge_desc(Key a, Key b, int lane)
{
    const Key r = __shfl_sync(0xffffffffu, b, 31 - lane);
    Key c = a > r ? a : r; // the 32 largest, rising then falling
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) {
        const Key o = __shfl_xor_sync(0xffffffffu, c, j);
        c = ((lane & j) == 0) == (o > c) ? o : c;
    }
    return c;
}

// One row as a CTA sees it: its vectors [vb, ve).
template <typename T> struct Part {
    const T *x;
    int V, lead, vb, ve;
};

// The first vector that a lane takes of thread `who`'s share, for share_rest.
template <int THREADS, typename T> __device__ __forceinline__ uint4 share_first(const Part<T> &r, int who, int lane)
{
    const int v = r.vb + who + lane * THREADS;
    return v < r.ve ? load_vec(r.x, r.V, r.lead, v) : empty_vec<T>();
}
// What thread `who` of THREADS sums of its share, but relative to `top`, which is its
// maximum, and with one element that is it left out; over the lanes. (This, instead
// of taking 1 from the sum, costs 8192 rows of 32000 bf16 3 us, and keeps log S and the
// entropy of a row of entropy 0.001 within 6e-7 of themselves instead of 6e-5.)
template <int THREADS, typename T>
__device__ __forceinline__ Stat share_rest(const Part<T> &r, int who, uint4 raw, float top, float c, int lane)
{
    constexpr int E = Vec<T>::E;
    Stat st{top, 0.0f, 0.0f};
    int equal = 0;
    for (int v = r.vb + who + lane * THREADS; v < r.ve;) {
        float f[E];
        Vec<T>::unpack(raw, f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const bool is = f[e] == top;
            const float d = is ? -1000.0f : max_nan((f[e] - top) * c, -1000.0f), w = exp2_fast(d);
            equal += is;
            st.s += w;
            st.u = fmaf(w, d, st.u);
        }
        v += 32 * THREADS;
        if (v < r.ve)
            raw = load_vec(r.x, r.V, r.lead, v);
    }
    const int first = __ffs(__ballot_sync(0xffffffffu, equal > 0)) - 1;
    st.s += (float)(equal - (lane == first));
    return st;
}

// The elements that reach `bound` in the shares of `npicked` of THREADS
// threads, the k best in descending order (of those this warp takes: vectors
// i0, i0 + step, ... of them, 32 at a time). Lane l's `who` is the l-th picked
// thread.
template <int THREADS, typename T>
__device__ __forceinline__ Key gather_top(const Part<T> &r, int who, int npicked, int i0, int step, Key bound, int k,
                                          Key *held, int lane)
{
    constexpr int E = Vec<T>::E, AHEAD = 5;
    const int share = (r.ve - r.vb + THREADS - 1) / THREADS, items = npicked * share;
    Key list = 0ull, floor = bound;
    int n = 0;
    for (; i0 < items; i0 += AHEAD * step) {
        uint4 raw[AHEAD];
        int at[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int i = i0 + a * step + lane, pick = min(i / share, 31);
            const int v = r.vb + __shfl_sync(0xffffffffu, who, pick) + (i - pick * share) * THREADS;
            at[a] = v * E - r.lead;
            raw[a] = i < items && v < r.ve ? load_vec(r.x, r.V, r.lead, v) : empty_vec<T>();
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            float f[E];
            Vec<T>::unpack(raw[a], f);
            const float least = floor == 1ull ? neg_inf() : key_value(floor);
            uint32_t mine = 0u; // this lane's elements that may reach the floor
#pragma unroll
            for (int e = 0; e < E; ++e)
                mine |= f[e] >= least && f[e] > neg_inf() ? 1u << e : 0u;
            while (__any_sync(0xffffffffu, mine != 0u)) { // one of each lane at a time
                const int e = __ffs(mine) - 1;
                float x = f[0];
#pragma unroll
                for (int j = 1; j < E; ++j)
                    x = e == j ? f[j] : x;
                const Key key = order_key(x, at[a] + e);
                const bool in = mine != 0u && key >= floor;
                mine &= mine - 1u;
                const uint32_t all = __ballot_sync(0xffffffffu, in);
                if (in)
                    held[n + __popc(all & ((1u << lane) - 1u))] = key;
                n += __popc(all);
                if (n >= 32) {
                    __syncwarp();
                    const Key c = held[lane], rest = held[32 + lane];
                    __syncwarp();
                    held[lane] = rest;
                    __syncwarp();
                    n -= 32;
                    list = merge_desc(list, warp_sort_desc(c, lane), lane);
                    const Key kth = __shfl_sync(0xffffffffu, list, k - 1);
                    floor = kth > floor ? kth : floor;
                }
            }
        }
    }
    __syncwarp();
    const Key rest = lane < n ? held[lane] : 0ull;
    __syncwarp(); // held is written again for the next row
    if (!__any_sync(0xffffffffu, list != 0ull))
        return warp_top(rest, k, lane);
    return merge_desc(list, warp_sort_desc(rest, lane), lane);
}

// What a warp keeps of the shares it looks through: vectors with an element
// that may reach the bound, and the elements that do.
struct Finds {
    static constexpr int VECS = 64, KEYS = 96;
    uint4 raw[VECS];
    int at[VECS];
    Key key[KEYS];
};

// gather_top for a warp by itself where no more than that reaches the bound (else
// false): a key's place is how many precede it.
template <int THREADS, typename T>
__device__ __forceinline__ bool gather_few(const Part<T> &r, int who, int npicked, Key bound, Finds &f, int lane, Key &top)
{
    constexpr int E = Vec<T>::E, AHEAD = 5;
    const int share = (r.ve - r.vb + THREADS - 1) / THREADS, items = npicked * share;
    const float least = bound == 1ull ? neg_inf() : key_value(bound);
    const uint32_t before = (1u << lane) - 1u;
    int vecs = 0, keys = 0;
    for (int i0 = 0; i0 < items; i0 += AHEAD * 32) {
        uint4 raw[AHEAD];
        int at[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int i = i0 + a * 32 + lane, pick = min(i / share, 31);
            const int v = r.vb + __shfl_sync(0xffffffffu, who, pick) + (i - pick * share) * THREADS;
            at[a] = v * E - r.lead;
            raw[a] = i < items && v < r.ve ? load_vec(r.x, r.V, r.lead, v) : empty_vec<T>();
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const float most = Vec<T>::largest(raw[a]);
            const bool hit = most >= least && most > neg_inf();
            const uint32_t all = __ballot_sync(0xffffffffu, hit);
            const int n = vecs + __popc(all);
            if (n > Finds::VECS)
                return false;
            if (hit) {
                const int to = vecs + __popc(all & before);
                f.raw[to] = raw[a];
                f.at[to] = at[a];
            }
            vecs = n;
        }
    }
    __syncwarp();
    for (int g = 0; g < vecs; g += 32) {
        const bool have = g + lane < vecs;
        const uint4 raw = have ? f.raw[g + lane] : empty_vec<T>();
        const int at = have ? f.at[g + lane] : 0;
        float x[E];
        Vec<T>::unpack(raw, x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const Key k = x[e] > neg_inf() ? order_key(x[e], at + e) : 0ull;
            const bool in = k >= bound;
            const uint32_t all = __ballot_sync(0xffffffffu, in);
            const int n = keys + __popc(all);
            if (n > Finds::KEYS)
                return false;
            if (in)
                f.key[keys + __popc(all & before)] = k;
            keys = n;
        }
    }
    __syncwarp();
    Key k[Finds::KEYS / 32];
    int to[Finds::KEYS / 32];
#pragma unroll
    for (int q = 0; q < Finds::KEYS / 32; ++q) {
        k[q] = q * 32 + lane < keys ? f.key[q * 32 + lane] : 0ull;
        to[q] = 0;
    }
#pragma unroll 4
    for (int i = 0; i < keys; ++i) {
        const Key other = f.key[i];
#pragma unroll
        for (int q = 0; q < Finds::KEYS / 32; ++q)
            to[q] += other > k[q];
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < Finds::KEYS / 32; ++q)
        if (k[q] != 0ull && to[q] < 32)
            f.key[to[q]] = k[q];
    __syncwarp();
    top = lane < keys ? f.key[lane] : 0ull;
    __syncwarp(); // the lists are written again for the next row
    return true;
}

// The key that every element has to reach: the last element of the vector of
// the k-th best thread (its vector may hold the value more than once), or any
// element where fewer than k threads hold one.
template <typename T> __device__ __forceinline__ Key bound_of(Key kth, int lead)
{
    return kth != 0ull ? order_key(key_value(kth), key_index(kth) * Vec<T>::E - lead + Vec<T>::E - 1) : 1ull;
}

// One thread's pass over its share of a row's vectors [vb, ve), with the next
// group always on its way.
template <typename T, int THREADS> struct Reader {
    static constexpr int E = Vec<T>::E, GROUP = LP_UNROLL * THREADS;
    const LogprobParams &p;
    int tid;
    Part<T> r;
    int safe_from, safe_to; // vectors that lie in the row entirely
    uint4 next[LP_UNROLL];

    __device__ __forceinline__ void fetch(int g0)
    {
        if (g0 >= safe_from && g0 + GROUP <= min(safe_to, r.ve)) {
            const uint4 *v = reinterpret_cast<const uint4 *>(r.x - r.lead) + (g0 + tid);
#pragma unroll
            for (int q = 0; q < LP_UNROLL; ++q)
                asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(next[q].x), "=r"(next[q].y), "=r"(next[q].z), "=r"(next[q].w)
                             : "l"(v + q * THREADS));
        } else {
#pragma unroll
            for (int q = 0; q < LP_UNROLL; ++q) {
                const int v = g0 + tid + q * THREADS;
                next[q] = v < r.ve ? load_vec(r.x, r.V, r.lead, v) : empty_vec<T>();
            }
        }
    }
    // row `row`, part `part` of `parts`; its first group is asked for
    __device__ __forceinline__ void enter(int row, int part, int parts)
    {
        r.x = static_cast<const T *>(p.logits) + (int64_t)row * p.stride;
        r.V = p.V;
        r.lead = row_lead(r.x);
        const int nvec = (int)(((int64_t)r.lead + p.V + E - 1) / E), per = (nvec + parts - 1) / parts;
        r.vb = min(nvec, part * per);
        r.ve = min(nvec, r.vb + per);
        safe_from = r.lead > 0 ? 1 : 0;
        safe_to = (int)(((int64_t)r.lead + p.V) / E);
        if (r.vb < r.ve)
            fetch(r.vb);
    }
    // the row entered; then(), called while its last group is summed, may enter another
    template <bool TOP, typename Then>
    __device__ __forceinline__ void read(Sums<T> &sums, int &best_vec, Then then)
    {
        const int vb = r.vb, ve = r.ve;
        best_vec = -1;
        for (int g0 = vb; g0 < ve; g0 += GROUP) {
            uint4 cur[LP_UNROLL];
#pragma unroll
            for (int q = 0; q < LP_UNROLL; ++q)
                cur[q] = next[q];
            if (g0 + GROUP < ve)
                fetch(g0 + GROUP);
            else
                then();
            float vm[LP_UNROLL], gm;
#pragma unroll
            for (int q = 0; q < LP_UNROLL; ++q) {
                vm[q] = Vec<T>::largest(cur[q]);
                gm = q == 0 ? vm[0] : max_nan(gm, vm[q]);
            }
            if (!(gm <= sums.limit))
                sums.raise(gm);
            const bool up = !(gm <= sums.m);
            sums.m = up ? gm : sums.m;
            if (TOP) {
                int q = LP_UNROLL - 1;
#pragma unroll
                for (int j = LP_UNROLL - 2; j >= 0; --j)
                    q = vm[j] == gm ? j : q;
                best_vec = up ? g0 + tid + q * THREADS : best_vec;
            }
            sums.add(cur);
        }
        if (vb >= ve)
            then();
    }
};

// The row's results, by one warp: lane i holds the i-th best element.
template <typename T, bool TOP>
__device__ __forceinline__ void write_row(const LogprobParams &p, int row, int token, float given, const Stat &st,
                                          Key top, int lane)
{
    const bool empty = st.m == neg_inf();
    // NaN when the row holds one, in the sums if not in the maximum, or +infinity
    const float logsum = empty ? 0.0f : st.m < -neg_inf() ? log1pf(st.s) : quiet_nan();
    const bool none = !(logsum == logsum);
    if (lane == 0) {
        if (p.stats != nullptr) {
            p.stats[2 * (int64_t)row] = none ? quiet_nan() : st.m;
            p.stats[2 * (int64_t)row + 1] = logsum;
        }
        if (p.entropy != nullptr)
            p.entropy[row] = empty ? 0.0f : logsum - LN2 * (st.u / (1.0f + st.s));
        if (p.logprob != nullptr) {
            float lp = 0.0f;
            if (token >= 0 && token < p.V)
                lp = empty ? neg_inf() : (given - st.m) * p.inv_t - logsum;
            p.logprob[row] = lp;
        }
    }
    if (TOP && lane < p.top_k) {
        // an element is one also where its log probability leaves fp32's range
        const bool one = top != 0ull && !none;
        const float lp = one ? (key_value(top) - st.m) * p.inv_t - logsum : neg_inf();
        p.top_logprobs[(int64_t)row * p.top_k + lane] = none ? quiet_nan() : lp;
        p.top_ids[(int64_t)row * p.top_k + lane] = one ? key_index(top) : -1;
    }
}

// The call's status, by `threads` threads of one CTA: any token past the vocabulary.
__device__ __forceinline__ void open_status(const LogprobParams &p, int tid, int threads)
{
    int bad = 0;
    if (p.tokens != nullptr)
        for (int i = tid; i < p.M; i += threads)
            bad |= p.tokens[i] >= p.V;
    bad = __syncthreads_or(bad);
    if (tid == 0)
        status_begin(p.status, bad ? (uint32_t)LORA_FLAG_TOKEN_RANGE : 0u);
}

constexpr int BAR_FULL = 1, BAR_FREE = 3; // named barriers, two of each

// What the reading threads leave of a row: maximum, reference and the sums
// relative to it; and (maximum, vector that holds it), which differ between
// threads since the vectors are their own.
template <bool TOP> struct Left {
    float4 sums[ROW_READERS];
    Key best[TOP ? ROW_READERS : 1];
};

} // namespace

// 8192 x 32000 bf16: 91 us, 5.7 TB/s, and 109 with the best element; issue slots
// and the exponentials bound it. 4096 x 32000 f32: 80 us, 6.6 TB/s, HBM. FIN warps
// finish rows in turn: with more than FEW alternatives that takes longer than
// reading, and two are worth the registers they take from the others (the best
// 20: 151 us, some 35 more with one; the best 5: 128, some 13 more with two). What does
// not fit the registers of three CTAs an SM is in local memory: up to 48 bytes a thread
// with one of them, 144 with two.
template <typename T, bool TOP, int FIN>
__global__ void __launch_bounds__(ROW_READERS + FIN * 32, ROW_CTAS) logprob_rows_kernel(LogprobParams p)
{
    constexpr int PER = ROW_READERS / 32; // threads a lane of the last warp answers for
    __shared__ Left<TOP> left[2];
    __shared__ Finds finds[TOP ? FIN : 1];
    begin_behind();
    const int tid = threadIdx.x, lane = tid & 31, step = gridDim.x;
    const float c = p.inv_t * LOG2E;
    if (blockIdx.x == 0)
        open_status(p, tid, ROW_READERS + FIN * 32);
    if (tid < ROW_READERS) {
        Reader<T, ROW_READERS> reader{p, tid};
        reader.enter(blockIdx.x, 0, 1);
        Sums<T> sums;
        sums.scale(c);
        for (int row = blockIdx.x, turn = 0; row < p.M; row += step, ++turn) {
            int best_vec;
            sums.clear();
            reader.template read<TOP>(sums, best_vec, [&] {
                if (row + step < p.M)
                    reader.enter(row + step, 0, 1);
            });
            const Stat st = sums.stat();
            Left<TOP> &l = left[turn & 1];
            if (turn >= 2) // the row before last has been finished
                named_bar_sync(BAR_FREE + (turn & 1), ROW_THREADS);
            l.sums[tid] = make_float4(sums.m, st.m, st.s, st.u);
            if (TOP) {
                Key best = best_vec >= 0 && sums.m > neg_inf() ? order_key(sums.m, best_vec) : 0ull;
                if (FIN == 2)
                    best = warp_sort_desc(best, tid & 31); // a warp's share of what would keep the last warp too long
                l.best[tid] = best;
            }
            named_bar_arrive(BAR_FULL + (turn & 1), ROW_THREADS);
        }
        return;
    }
    const int fin = (tid - ROW_READERS) / 32;
    Finds &found = finds[TOP ? fin : 0];
    for (int row = blockIdx.x + fin * step, turn = fin; row < p.M; row += FIN * step, turn += FIN) {
        Left<TOP> &l = left[turn & 1];
        Part<T> r;
        r.x = static_cast<const T *>(p.logits) + (int64_t)row * p.stride;
        r.V = p.V;
        r.lead = row_lead(r.x);
        r.vb = 0;
        r.ve = (int)(((int64_t)r.lead + p.V + Vec<T>::E - 1) / Vec<T>::E);
        // what the results need besides, on its way before the wait
        const int token = p.logprob != nullptr ? p.tokens[row] : -1;
        const float given = token >= 0 && token < p.V ? Vec<T>::widen(r.x[token]) : 0.0f;
        named_bar_sync(BAR_FULL + (turn & 1), ROW_THREADS);
        float4 q[PER];
        Key key[TOP ? PER : 1], best = 0ull;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            q[i] = l.sums[i * 32 + lane];
            if (TOP)
                key[i] = l.best[i * 32 + lane];
        }
        if (row + 2 * (int64_t)step < p.M)
            named_bar_arrive(BAR_FREE + (turn & 1), ROW_THREADS);
        float m = q[0].x;
#pragma unroll
        for (int i = 1; i < PER; ++i)
            m = max_nan(m, q[i].x);
        m = warp_max_nan(m);
        int holder = 0; // the thread whose maximum it is
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) {
            const uint32_t is = __ballot_sync(0xffffffffu, q[i].x == m);
            holder = is != 0u ? i * 32 + __ffs(is) - 1 : holder;
        }
        const uint4 raw = share_first<ROW_READERS>(r, holder, lane);
        Key top = 0ull;
        if (TOP) { // the k best threads, lane by lane
            if (FIN == 1) { // top_k <= FEW
                for (int i = 0; i < p.top_k; ++i) {
                    Key mine = key[0];
#pragma unroll
                    for (int j = 1; j < PER; ++j)
                        mine = key[j] > mine ? key[j] : mine;
                    const Key one = warp_max_key(mine);
                    best = lane == i ? one : best;
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        key[j] = key[j] == one ? 0ull : key[j];
                }
            } else {
#pragma unroll
                for (int w = 1; w < PER; w *= 2)
#pragma unroll
                    for (int j = 0; j + w < PER; j += 2 * w)
                        key[j] = merge_desc(key[j], key[j + w], lane);
                best = lane < p.top_k ? key[0] : 0ull;
            }
            const int npicked = __popc(__ballot_sync(0xffffffffu, best != 0ull));
            const Key bound = bound_of<T>(__shfl_sync(0xffffffffu, best, p.top_k - 1), r.lead);
            const int who = best != 0ull ? key_index(best) % ROW_READERS : 0;
            // for a few the one pass is shorter; else only where a share holds much of the best
            if (FIN == 1 || !gather_few<ROW_READERS>(r, who, npicked, bound, found, lane, top))
                top = gather_top<ROW_READERS>(r, who, npicked, 0, 32, bound, p.top_k, found.key, lane);
        }
        Stat st = share_rest<ROW_READERS>(r, holder, raw, m, c, lane);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            Stat one{q[i].y, q[i].z, q[i].w};
            rescale(one, m, c);
            if (i * 32 + lane != holder) {
                st.s += one.s;
                st.u += one.u;
            }
        }
        st.s = warp_sum(st.s);
        st.u = warp_sum(st.u);
        write_row<T, TOP>(p, row, token, given, st, top, lane);
    }
}

// Many short rows: a row a warp, which reads and finishes it, so the finishing, which
// takes longer than reading, goes on in all warps of an SM. Latency and issue bound it:
// 8170 x 3188 bf16 in 16 us, 26 with the best five.
template <typename T, bool TOP> __global__ void __launch_bounds__(LP_THREADS) logprob_short_kernel(LogprobParams p)
{
    __shared__ Finds finds[TOP ? LP_WARPS : 1];
    begin_behind();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t at = (int64_t)blockIdx.x * LP_WARPS + warp;
    const float c = p.inv_t * LOG2E;
    if (blockIdx.x == 0)
        open_status(p, tid, LP_THREADS);
    if (at >= p.M)
        return;
    const int row = (int)at;
    Reader<T, 32> reader{p, lane};
    reader.enter(row, 0, 1);
    const Part<T> r = reader.r;
    const int token = p.logprob != nullptr ? p.tokens[row] : -1;
    const float given = token >= 0 && token < p.V ? Vec<T>::widen(r.x[token]) : 0.0f;
    Sums<T> sums;
    int best_vec;
    sums.scale(c);
    sums.clear();
    reader.template read<TOP>(sums, best_vec, [] {});
    const float m = warp_max_nan(sums.m);
    const int holder = max(__ffs(__ballot_sync(0xffffffffu, sums.m == m)) - 1, 0);
    const uint4 raw = share_first<32>(r, holder, lane);
    Key top = 0ull;
    if (TOP) {
        Key best = warp_top(best_vec >= 0 && sums.m > neg_inf() ? order_key(sums.m, best_vec) : 0ull, p.top_k, lane);
        best = lane < p.top_k ? best : 0ull;
        const int npicked = __popc(__ballot_sync(0xffffffffu, best != 0ull));
        const Key bound = bound_of<T>(__shfl_sync(0xffffffffu, best, p.top_k - 1), r.lead);
        const int who = best != 0ull ? key_index(best) % 32 : 0;
        if (!gather_few<32>(r, who, npicked, bound, finds[warp], lane, top))
            top = gather_top<32>(r, who, npicked, 0, 32, bound, p.top_k, finds[warp].key, lane);
    }
    Stat one = sums.stat(), st = share_rest<32>(r, holder, raw, m, c, lane);
    rescale(one, m, c);
    st.s = warp_sum(st.s + (lane != holder ? one.s : 0.0f));
    st.u = warp_sum(st.u + (lane != holder ? one.u : 0.0f));
    write_row<T, TOP>(p, row, token, given, st, top, lane);
}

namespace {

constexpr int CAND = 256; // elements that reach the bound, gathered by the whole CTA

template <bool TOP> struct SplitShared {
    Stat warp[LP_WARPS], cta;
    Key lists[TOP ? LP_WARPS : 1][32]; // the warps' best (value, vector), descending
    Key found[TOP ? CAND : 1];
    Key fin[32], last[32]; // the CTA's best, the row's
    Key held[TOP ? LP_WARPS : 1][64];
    Key bound;
    int picked[32];
    int nfound;
};

} // namespace

// Latency bounds it. 1 x 32000 bf16: 4 us, 8.7 with the best 20; 64 x 32003 f32 with
// the best 20: 9 us.
template <typename T, bool TOP>
__global__ void __launch_bounds__(LP_THREADS, 4) logprob_split_kernel(LogprobParams p, int parts)
{
    constexpr int E = Vec<T>::E;
    __shared__ SplitShared<TOP> sm;
    begin_behind();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = blockIdx.x % parts, row = blockIdx.x / parts;
    const float c = p.inv_t * LOG2E;
    Reader<T, LP_THREADS> reader{p, tid};
    reader.enter(row, part, parts);
    const Part<T> r = reader.r;
    if (blockIdx.x == 0)
        open_status(p, tid, LP_THREADS);
    if (TOP && tid < 32) {
        sm.picked[tid] = -1;
        sm.fin[tid] = sm.last[tid] = 0ull;
        if (tid == 0) {
            sm.bound = 1ull; // with fewer than k threads that hold any element, every element counts
            sm.nfound = 0;
        }
    }
    const int token = p.logprob != nullptr ? p.tokens[row] : -1;
    const float given = token >= 0 && token < p.V ? Vec<T>::widen(r.x[token]) : 0.0f;
    Sums<T> sums;
    int best_vec;
    sums.scale(c);
    sums.clear();
    reader.template read<TOP>(sums, best_vec, [] {});
    Stat ws{warp_max_nan(sums.m), 0.0f, 0.0f};
    const int holder = max(__ffs(__ballot_sync(0xffffffffu, sums.m == ws.m)) - 1, 0);
    const uint4 raw = share_first<LP_THREADS>(r, warp * 32 + holder, lane);
    Key best = 0ull;
    if (TOP) {
        best = warp_top(best_vec >= 0 && sums.m > neg_inf() ? order_key(sums.m, best_vec) : 0ull, p.top_k, lane);
        sm.lists[warp][lane] = best;
    }
    {
        Stat one = sums.stat();
        rescale(one, ws.m, c);
        const Stat rest = share_rest<LP_THREADS>(r, warp * 32 + holder, raw, ws.m, c, lane);
        ws.s = warp_sum(rest.s + (lane != holder ? one.s : 0.0f));
        ws.u = warp_sum(rest.u + (lane != holder ? one.u : 0.0f));
        if (lane == 0)
            sm.warp[warp] = ws;
    }
    __syncthreads();
    if (TOP) {
        const int at = best != 0ull && lane < p.top_k ? place(sm.lists, warp, lane, best) : 32;
        if (at < p.top_k) // the thread whose best it is
            sm.picked[at] = (key_index(best) - r.vb) % LP_THREADS;
        if (at == p.top_k - 1)
            sm.bound = bound_of<T>(best, r.lead);
        __syncthreads();
        const Key bound = sm.bound;
        const int share = (r.ve - r.vb + LP_THREADS - 1) / LP_THREADS;
        const int who = sm.picked[lane], npicked = __popc(__ballot_sync(0xffffffffu, who >= 0));
        for (int i = tid; i < npicked * share; i += LP_THREADS) {
            const int pick = i / share, v = r.vb + sm.picked[pick] + (i - pick * share) * LP_THREADS;
            if (v >= r.ve)
                continue;
            const uint4 raw = load_vec(r.x, r.V, r.lead, v);
            if (order_key(Vec<T>::largest(raw), 0) < bound) // all below it by value
                continue;
            float f[E];
            Vec<T>::unpack(raw, f);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const Key k = f[e] > neg_inf() ? order_key(f[e], v * E - r.lead + e) : 0ull;
                if (k >= bound) {
                    const int n = atomicAdd(&sm.nfound, 1); // in any order: they are put in order below
                    if (n < CAND)
                        sm.found[n] = k;
                }
            }
        }
        __syncthreads();
        const int nfound = sm.nfound;
        if (nfound <= CAND) { // a key's place is how many precede it
            if (tid < nfound) {
                const Key k = sm.found[tid];
                int to = 0;
                for (int i = 0; i < nfound; ++i)
                    to += sm.found[i] > k;
                if (to < p.top_k)
                    sm.fin[to] = k;
            }
        } else { // a share holds much of the best: sorted lists instead
            const Key list = gather_top<LP_THREADS>(r, max(who, 0), npicked, warp * 32, LP_THREADS, bound, p.top_k, sm.held[warp],
                                                     lane);
            sm.lists[warp][lane] = list;
            __syncthreads();
            const int to = list != 0ull && lane < p.top_k ? place(sm.lists, warp, lane, list) : 32;
            if (to < p.top_k)
                sm.fin[to] = list;
        }
        __syncthreads();
    }

    // ---- join: warps, then the cluster's parts
    Stat st{neg_inf(), 0.0f, 0.0f};
    if (warp == 0) {
        if (lane < LP_WARPS)
            st = sm.warp[lane];
        st = warp_join_rest(st, c);
        if (lane == 0)
            sm.cta = st;
    }
    Key top = 0ull;
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    if (part == 0) {
        if (warp == 0) {
            st = lane < parts ? cl.map_shared_rank(&sm, lane)->cta : Stat{neg_inf(), 0.0f, 0.0f};
            st = warp_join_rest(st, c);
        }
        if (TOP) {
            const Key k = warp < parts && lane < p.top_k ? cl.map_shared_rank(&sm, warp)->fin[lane] : 0ull;
            sm.lists[warp][lane] = k;
            __syncthreads();
            const int at = k != 0ull ? place(sm.lists, warp, lane, k) : 32;
            if (at < p.top_k)
                sm.last[at] = k;
            __syncthreads();
            top = sm.last[lane];
        }
        if (warp == 0)
            write_row<T, TOP>(p, row, token, given, st, top, lane);
    }
    cl.sync(); // the parts' shared memory is read until here
}

// A CTA takes LP_UNROLL * LP_THREADS vectors of one row of dlogits. With
// a = log2 p and one factor for each row, an element is
//   dx = 2^a (q + r a),  q = -t (g + g_H H),  r = -t g_H ln 2,
// but the token's own, whose g (1 - p) is -g expm1(log p): where p is near 1 the
// difference of g and g p would keep few digits. a = x c - (m c + log S log2 e), the
// latter held as two fp32 numbers so that p is as good as fp32 allows.
// 8192 x 32000 bf16: 150 us, 7.0 TB/s, HBM; 96 x 32003 f32 with entropy 4.5 us.
template <typename T, bool BONUS>
__global__ void __launch_bounds__(LP_THREADS, 6) logprob_grad_kernel(LogprobGradParams p, int segs)
{
    constexpr int E = Vec<T>::E;
    begin_behind();
    const int row = blockIdx.x / segs, seg = blockIdx.x % segs;
    const T *x = static_cast<const T *>(p.logits) + (int64_t)row * p.stride;
    T *dx = static_cast<T *>(p.dlogits) + (int64_t)row * p.d_stride;
    const int lead = row_lead(dx);
    const bool same = row_lead(x) == lead; // both rows split into the same vectors
    const int nvec = (int)(((int64_t)lead + p.V + E - 1) / E);
    const int v0 = seg * (LP_UNROLL * LP_THREADS) + threadIdx.x;
    uint4 raw[LP_UNROLL];
#pragma unroll
    for (int q = 0; q < LP_UNROLL; ++q) {
        const int v = v0 + q * LP_THREADS, i0 = v * E - lead;
        if (v < nvec) {
            if (same && i0 >= 0 && i0 + E <= p.V) { // not through the read-only path: dlogits may be logits
                asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(raw[q].x), "=r"(raw[q].y), "=r"(raw[q].z), "=r"(raw[q].w)
                             : "l"(x + i0)
                             : "memory");
            } else {
                float f[E];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    f[e] = i0 + e >= 0 && i0 + e < p.V ? Vec<T>::widen(x[i0 + e]) : neg_inf();
                raw[q] = Vec<T>::pack(f);
            }
        }
    }
    const float m = p.stats[2 * (int64_t)row], logsum = p.stats[2 * (int64_t)row + 1];
    int t = p.tokens != nullptr ? p.tokens[row] : -1;
    t = t < p.V ? t : -1;
    const float g = t >= 0 && p.g_logprob != nullptr ? p.g_logprob[row] : 0.0f;
    const float gh = BONUS ? p.g_entropy[row] : 0.0f;
    const float H = BONUS ? p.entropy[row] : 0.0f;
    const bool empty = m == neg_inf();
    const float c = p.inv_t * LOG2E;
    const float qf = -p.inv_t * (g + gh * H), rf = -p.inv_t * gh * LN2;
    // m c + logsum log2 e in two parts; rows of huge values take the difference first
    const float mc = m * c, ml = fmaf(m, c, -mc), ls = logsum * LOG2E;
    const float hi = mc + ls, part = hi - mc, lo = ((mc - (hi - part)) + (ls - part)) + ml;
    const bool huge = !(fabsf(mc) <= 65536.0f);
    const f2 c2 = make_f2(c, c), hi2 = make_f2(-hi, -hi), lo2 = make_f2(-lo, -lo), q2 = make_f2(qf, qf), r2 = make_f2(rf, rf);
    const f2 nm2 = make_f2(-m, -m), ls2 = make_f2(-ls, -ls);
    bool mine = false; // this thread has the token's element, which is xt
    float xt = 0.0f;
#pragma unroll
    for (int q = 0; q < LP_UNROLL; ++q) {
        const int v = v0 + q * LP_THREADS, i0 = v * E - lead;
        if (v >= nvec)
            break;
        float f[E];
        Vec<T>::unpack(raw[q], f);
        if (t >= max(i0, 0) && t < i0 + E) { // none, -1, may lie before the row in its first vector
            mine = true;
#pragma unroll
            for (int e = 0; e < E; ++e)
                xt = i0 + e == t ? f[e] : xt;
        }
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const f2 x2 = make_f2(f[e], f[e + 1]);
            f2 a2;
            if (huge)
                a2 = add_f2(mul_f2(add_f2(x2, nm2), c2), ls2);
            else
                a2 = add_f2(fma_f2(x2, c2, hi2), lo2);
            float a0, a1;
            split_f2(a2, a0, a1);
            f2 d2;
            if (BONUS) { // 0 log 0 is 0
                a0 = max_nan(a0, -1000.0f);
                a1 = max_nan(a1, -1000.0f);
                d2 = fma_f2(make_f2(a0, a1), r2, q2);
            } else {
                d2 = q2;
            }
            d2 = mul_f2(make_f2(exp2_fast(a0), exp2_fast(a1)), d2);
            split_f2(d2, f[e], f[e + 1]);
        }
        if (empty) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                f[e] = 0.0f;
        }
        if (i0 >= 0 && i0 + E <= p.V) {
            *reinterpret_cast<uint4 *>(dx + i0) = Vec<T>::pack(f);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (i0 + e >= 0 && i0 + e < p.V)
                    dx[i0 + e] = Vec<T>::narrow(f[e]);
        }
    }
    // Over what was stored there. The row's numbers are read again: kept through the loop
    // they took registers that it needs (8192 x 32000 bf16 with entropy: 169 us, 155).
    if (mine && !empty) {
        const float lp = (xt - p.stats[2 * (int64_t)row]) * p.inv_t - p.stats[2 * (int64_t)row + 1];
        float d = p.g_logprob != nullptr ? -p.inv_t * p.g_logprob[row] * expm1f(lp) : 0.0f;
        if (BONUS) {
            const float l = max_nan(lp, -700.0f);
            d = fmaf(exp2_fast(l * LOG2E), -p.inv_t * p.g_entropy[row] * (l + p.entropy[row]), d);
        }
        dx[t] = Vec<T>::narrow(d);
    }
}

template <typename T> cudaError_t launch_lp(const LogprobParams &p, int num_sms, cudaStream_t st)
{
    // Parts of a row, each at least one vector a thread: none of a row that a CTA is
    // through with before a cluster has met, else enough CTAs for one an SM, and for
    // two where a part is longer than `longest`. us for the best 0, 5 and 20 with two for
    // all, one for all, and this:
    //    90 x   8000 bf16   3.9  8.1  8.6   3.9  8.1  8.6   2.7  5.1  6.4
    //    64 x  32000 f32    4.2  9.6 10.2   4.1  8.0  8.4   4.0  7.1  8.5
    //   200 x  32000 f32    7.6 12.0 13.4   7.5 10.1 15.3   7.6 10.1 13.4
    //    90 x 131072 f32   10.9 15.6 17.8  14.2 18.8 21.1  10.8 15.7 17.9
    // Around `shortest`, us for the best 1, 5 and 20 with 1, 2, 4 and 8 parts (f32):
    //     1 x  32003    6.2  7.4 12.2   8.0  8.3  9.2   7.4  7.8  8.2   7.2  7.7  8.0
    //    64 x  32003    6.5  7.9 12.8   8.4  8.5  9.6   8.1  8.5  9.0   9.6 10.2 10.8
    //     1 x  50000    7.5  9.4 16.1   8.6  8.9  9.7   7.9  8.1  8.8   7.4  7.8  8.2
    //    64 x  50000    8.3  9.4 16.6   9.0  9.0 10.1   8.8  9.1 10.1  10.3 10.9 11.7
    //   200 x  65536   15.3 17.9 27.4  15.8 16.5 18.5  22.5 23.3 25.8  29.7 31.1 33.3
    // (Rows of 256 KB in bf16 would rather stay whole in a call of 200 with up to eight
    // alternatives: 200 x 131072 16.4 and 19.1 us whole, 20.8 and 21.6 in two parts.)
    const bool few = p.top_k > 0 && p.top_k <= FEW;
    const int64_t shortest = few ? 140 << 10 : 40 << 10, longest = p.top_k > FEW ? 112 << 10 : 224 << 10;
    const int64_t nvec = ((int64_t)p.V + Vec<T>::E - 1) / Vec<T>::E;
    int parts = 1;
    while (parts < 8 && nvec * 16 > shortest && nvec >= 2 * parts * LP_THREADS &&
           ((int64_t)p.M * parts < num_sms || ((int64_t)p.M * parts < 2 * num_sms && nvec * 16 / parts > longest)))
        parts *= 2;
    // More short rows than CTAs that take whole ones: a warp each. us for the best 0, 1, 5
    // and 20, whole rows by CTAs and by warps:
    //   1000 x  8000 bf16   7.5 13.8 15.4 15.2    6.8  8.5  8.8 13.0
    //   8170 x  3188 bf16  41.4 73.2 82.4 87.9   15.5 24.8 26.3 34.4
    //   1000 x 14000 bf16  10.1 16.7 18.6 20.0   12.5 14.0 15.7 22.7
    //   2000 x 14000 bf16  16.3 25.8 29.3 32.0   14.9 20.2 23.0 34.6
    //   8170 x 14000 bf16  57.9 84.7 98.0  102   43.2 53.4 62.8 96.5
    //   8170 x 20000 bf16  73.9 96.3  110  126   61.0 72.9 96.6  183
    //   2000 x  8000 f32   13.5 20.3 23.9 25.5   15.2 17.2 20.1 33.9
    //   8170 x  8000 f32   42.3 66.0 80.6 79.7   45.1 55.2 68.1  120
    //    700 x  8000 bf16   6.3  9.6 10.6 11.9    6.5  7.8  8.4 12.5
    //    700 x  4000 f32    5.2  7.8  8.9  9.6    5.5  6.9  7.5 11.5
    // The cut is at 16 KB, below which warps take down to a third of the time; but rows of
    // more than 12 KB, of which no CTA has more than two, are left to CTAs without
    // alternatives and with more than 16 (the best nine of 700: 11.5 and 9.6 us, 9.3 and
    // 8.7). Between 16 and 40 KB thousands of rows with few alternatives would be up to 37 %
    // shorter by warps, hundreds of rows or twenty alternatives up to half as long again.
    const int at_once = ROW_CTAS * num_sms;
    const bool two = nvec > SHORT_VECS * 3 / 4 && p.M <= 2 * at_once && (p.top_k == 0 || p.top_k > 2 * FEW);
    if (parts == 1 && nvec <= SHORT_VECS && p.M > at_once && !two)
        return launch_behind(p.top_k > 0 ? logprob_short_kernel<T, true> : logprob_short_kernel<T, false>,
                             dim3((unsigned)(((int64_t)p.M + LP_WARPS - 1) / LP_WARPS)), LP_THREADS, 0, 1, st, p);
    if (parts == 1) { // as many CTAs as stay resident, each with rows one after another
        const dim3 grid((unsigned)(p.M < at_once ? p.M : at_once));
        return launch_behind(p.top_k > FEW  ? logprob_rows_kernel<T, true, 2>
                             : p.top_k > 0 ? logprob_rows_kernel<T, true, 1>
                                           : logprob_rows_kernel<T, false, 1>,
                             grid, p.top_k > FEW ? ROW_THREADS + 32 : ROW_THREADS, 0, 1, st, p);
    }
    return launch_behind(p.top_k > 0 ? logprob_split_kernel<T, true> : logprob_split_kernel<T, false>, dim3((unsigned)(p.M * parts)),
                         LP_THREADS, 0, (unsigned)parts, st, p, parts);
}

cudaError_t launch_logprob(const LogprobParams &p, int dtype, int num_sms, cudaStream_t st)
{
    return dtype == LORA_DTYPE_F32 ? launch_lp<float>(p, num_sms, st) : launch_lp<uint16_t>(p, num_sms, st);
}

template <typename T> cudaError_t launch_grad(const LogprobGradParams &p, cudaStream_t st)
{
    // one vector more than V fills, for rows that start inside one
    const int64_t nvec = ((int64_t)p.V + Vec<T>::E - 1) / Vec<T>::E + 1;
    const int segs = (int)((nvec + LP_UNROLL * LP_THREADS - 1) / (LP_UNROLL * LP_THREADS));
    return launch_behind(p.g_entropy != nullptr ? logprob_grad_kernel<T, true> : logprob_grad_kernel<T, false>,
                         dim3((unsigned)(p.M * segs)), LP_THREADS, 0, 1, st, p, segs);
}

cudaError_t launch_logprob_grad(const LogprobGradParams &p, int dtype, cudaStream_t st)
{
    return dtype == LORA_DTYPE_F32 ? launch_grad<float>(p, st) : launch_grad<uint16_t>(p, st);
}

} // namespace rd
