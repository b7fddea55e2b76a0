// Log probabilities of given tokens, entropy, softmax statistics and the best
// alternatives of rows of logits, and the gradient of the first two.
//
// With z_v = x_v t (t = inv_temperature), m = max x, d_v = (x_v - m) t:
//   S = sum e^{d_v},  log p_v = d_v - log S,  H = log S - (sum e^{d_v} d_v) / S,
//   dx_v = t [ g (1[v = token] - p_v) - g_H p_v (log p_v + H) ].
//
// logprob_kernel reads a row once: every thread keeps a running maximum with
// S and sum e^d d relative to it and rescales both when a group of its
// elements raises the maximum (rare after the first group). Sums are fp32, e^d
// is the hardware's 2^x (about 2^-22 relative). While one group is summed the
// next one, or the next row's first, is on its way: the kernel is bound by HBM
// as long as its loads never stop.
//
// The best alternatives cost the pass nothing but the maximum it needs anyway:
// of the threads' own best elements the k-th largest is a lower bound of the
// row's k-th best, so only the (at most k) threads whose best reaches it can
// hold any of the k, and their shares, V / threads elements each, are read
// again from L2. Elements are compared by (value, lowest index first) packed
// into 64 bits, which orders them totally; -0 equals +0. Sorted lists of the
// warps are merged by counting: a key's place is its place in its own list
// plus, by binary search, how many of each other list precede it.
//
// A row is split over a cluster of up to 8 CTAs when there are too few rows to
// fill the SMs; the parts are joined through distributed shared memory in
// part order, so results do not depend on timing.
#include <cooperative_groups.h>

#include "lora_logprob.cuh"
#include "vec.cuh"

namespace rd {

namespace cg = cooperative_groups;

namespace {

constexpr int LP_THREADS = 256;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_UNROLL = 4;        // 16-byte vectors of a thread in flight
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

__device__ __forceinline__ Stat join(Stat a, Stat b, float c)
{
    const float top = max_nan(a.m, b.m);
    rescale(a, top, c);
    rescale(b, top, c);
    return Stat{top, a.s + b.s, a.u + b.u};
}

__device__ __forceinline__ Stat warp_join(Stat st, float c)
{
    float top = st.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    rescale(st, top, c);
    st.s = warp_sum(st.s);
    st.u = warp_sum(st.u);
    return st;
}

// What a thread has summed of its elements. For bf16 the difference to the
// maximum and the scaling are one fused operation, a = x c - ref with ref =
// fl(m c), and masked elements are raised, two at a time, to a value whose
// power of two is 0 (so that 0 times their a is 0): that holds while m c is
// small enough for ref's rounding to be put right afterwards to first order
// and the raised value lies far enough below m. Other rows (and fp32, which
// has half the elements a byte) take the difference first and clamp a.
template <typename T> struct Sums {
    float m, ref, c;
    bool fused;
    uint32_t low; // the raised value, twice
    f2 s, u;

    __device__ __forceinline__ void clear(float c_)
    {
        m = neg_inf();
        ref = 0.0f;
        c = c_;
        fused = false;
        low = 0u;
        s = u = make_f2(0.0f, 0.0f);
    }
    // ref - m c, what the sums' origin is off by
    __device__ __forceinline__ float origin() const { return fused ? fmaf(-m, c, ref) : 0.0f; }

    __device__ __forceinline__ void raise(float top)
    {
        const float old = origin(), from = m;
        m = top;
        ref = m * c;
        if (sizeof(T) == 2) {
            const uint32_t b = f32_to_bf16_bits(m - 400.0f / c);
            const float raised = __uint_as_float(b << 16);
            low = b | b << 16;
            fused = fabsf(ref) <= 4096.0f && (raised - m) * c <= -150.0f && raised > neg_inf();
        }
        if (from != neg_inf()) {
            const float d = max_nan((from - m) * c + (old - origin()), -1000.0f);
            const float w = exp2_fast(d);
            const f2 d2 = make_f2(d, d), w2 = make_f2(w, w);
            u = mul_f2(w2, fma_f2(d2, s, u));
            s = mul_f2(w2, s);
        }
    }
    __device__ __forceinline__ void add_pair(f2 a2)
    {
        float a0, a1;
        split_f2(a2, a0, a1);
        const f2 e2 = make_f2(exp2_fast(a0), exp2_fast(a1));
        s = add_f2(s, e2);
        u = fma_f2(e2, a2, u);
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
            const float nm = m == neg_inf() ? 0.0f : -m;
            const f2 c2 = make_f2(c, c), nm2 = make_f2(nm, nm);
#pragma unroll
            for (int q = 0; q < N; ++q) {
                float f[E];
                Vec<T>::unpack(v[q], f);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    float a0, a1;
                    split_f2(mul_f2(add_f2(make_f2(f[e], f[e + 1]), nm2), c2), a0, a1);
                    add_pair(make_f2(max_nan(a0, -1000.0f), max_nan(a1, -1000.0f)));
                }
            }
        }
    }
    __device__ __forceinline__ Stat stat() const
    {
        float a, b;
        Stat st;
        st.m = m;
        split_f2(s, a, b);
        st.s = a + b;
        split_f2(u, a, b);
        st.u = a + b;
        const float d = origin(); // at most 2^-13: 2^d is 1 + d ln 2
        st.u += d * st.s;
        st.u = fmaf(d * LN2, st.u, st.u);
        st.s = fmaf(d * LN2, st.s, st.s);
        return st;
    }
};

using Key = unsigned long long;

struct LpShared {
    Stat warp[2][LP_WARPS]; // by row parity: a warp may be a row ahead
    Stat cta;
    Key lists[LP_WARPS][32];  // descending
    Key found[LP_WARPS][32];
    Key fin[32], last[32];    // the CTA's best, the row's
    Key bound;
    int picked[32];
};

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

} // namespace

template <typename T, bool TOP>
__global__ void __launch_bounds__(LP_THREADS, 4) logprob_kernel(LogprobParams p, int parts)
{
    constexpr int E = Vec<T>::E, GROUP = LP_UNROLL * LP_THREADS;
    __shared__ LpShared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = blockIdx.x % parts, row_step = gridDim.x / parts;
    const float c = p.inv_t * LOG2E;

    // a row and the vectors [vb, ve) of it that this CTA takes
    int row = blockIdx.x / parts;
    const T *x;
    int lead, vb, ve;
    auto enter = [&](int r) {
        x = static_cast<const T *>(p.logits) + (int64_t)r * p.stride;
        lead = row_lead(x);
        const int nvec = (int)(((int64_t)lead + p.V + E - 1) / E), per = (nvec + parts - 1) / parts;
        vb = min(nvec, part * per);
        ve = min(nvec, vb + per);
    };
    uint4 next[LP_UNROLL];
    auto fetch = [&](int v0) {
#pragma unroll
        for (int q = 0; q < LP_UNROLL; ++q) {
            const int v = v0 + q * LP_THREADS;
            next[q] = v < ve ? load_vec(x, p.V, lead, v) : empty_vec<T>();
        }
    };
    enter(row);
    fetch(vb + tid);

    if (blockIdx.x == 0) { // the call's status: any token past the vocabulary
        int bad = 0;
        if (p.tokens != nullptr)
            for (int i = tid; i < p.M; i += LP_THREADS)
                bad |= p.tokens[i] >= p.V;
        bad = __syncthreads_or(bad);
        if (tid == 0)
            status_begin(p.status, bad ? (uint32_t)LORA_FLAG_TOKEN_RANGE : 0u);
    }

    for (int parity = 0; row < p.M; parity ^= 1) {
        // ---- the pass
        const T *const rx = x;
        const int rlead = lead, rvb = vb, rve = ve, rrow = row;
        Sums<T> sums;
        sums.clear(c);
        int best_vec = -1; // the vector that holds the thread's maximum
        for (int g0 = rvb; g0 < rve; g0 += GROUP) {
            uint4 cur[LP_UNROLL];
#pragma unroll
            for (int q = 0; q < LP_UNROLL; ++q)
                cur[q] = next[q];
            if (g0 + GROUP < rve) {
                fetch(g0 + GROUP + tid);
            } else if ((row += row_step) < p.M) {
                enter(row);
                fetch(vb + tid);
            }
            float vm[LP_UNROLL], gm;
#pragma unroll
            for (int q = 0; q < LP_UNROLL; ++q) {
                vm[q] = Vec<T>::largest(cur[q]);
                gm = q == 0 ? vm[0] : max_nan(gm, vm[q]);
            }
            if (!(gm <= sums.m)) {
                sums.raise(gm);
                if (TOP) {
#pragma unroll
                    for (int q = LP_UNROLL - 1; q >= 0; --q)
                        if (vm[q] == gm)
                            best_vec = g0 + tid + q * LP_THREADS;
                }
            }
            sums.add(cur);
        }
        if (row == rrow && (row += row_step) < p.M) { // a part without vectors
            enter(row);
            fetch(vb + tid);
        }

        // ---- the warps' statistics and best elements
        const Stat ws = warp_join(sums.stat(), c);
        if (lane == 0)
            sm.warp[parity][warp] = ws;
        Key sorted = 0ull;
        if (TOP) {
            if (best_vec >= 0 && sums.m > neg_inf()) {
                float f[E];
                Vec<T>::unpack(load_vec(rx, p.V, rlead, best_vec), f);
#pragma unroll
                for (int e = E - 1; e >= 0; --e) // the lowest index last
                    if (f[e] == sums.m)
                        sorted = order_key(f[e], best_vec * E - rlead + e);
            }
            sorted = warp_sort_desc(sorted, lane);
            sm.lists[warp][lane] = sorted;
            if (tid < 32) {
                sm.picked[tid] = -1;
                sm.fin[tid] = 0ull;
                if (tid == 0)
                    sm.bound = 1ull; // fewer than k threads hold any element: every element counts
            }
        }
        __syncthreads();
        if (TOP) {
            const int at = sorted != 0ull && lane < p.top_k ? place(sm.lists, warp, lane, sorted) : 32;
            if (p.top_k == 1) { // the best of the bests needs no second look
                if (at == 0)
                    sm.fin[0] = sorted;
            } else {
                if (at < p.top_k) // the thread whose best it is
                    sm.picked[at] = ((key_index(sorted) + rlead) / E - rvb) % LP_THREADS;
                if (at == p.top_k - 1)
                    sm.bound = sorted;
                __syncthreads();
                // ---- the picked threads' shares again, a warp each
                Key list = 0ull, floor = sm.bound; // lane i: the i-th best so far
                for (int i = warp; i < p.top_k && sm.picked[i] >= 0; i += LP_WARPS) {
                    for (int w0 = rvb + sm.picked[i]; w0 < rve; w0 += 32 * LP_THREADS) {
                        const int v = w0 + lane * LP_THREADS;
                        const uint4 raw = v < rve ? load_vec(rx, p.V, rlead, v) : empty_vec<T>();
                        float f[E];
                        Vec<T>::unpack(raw, f);
                        // whether any lane has a candidate at all (by value; ties are settled below)
                        if (!__any_sync(0xffffffffu, order_key(Vec<T>::largest(raw), 0) >= floor))
                            continue;
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const Key k = f[e] > neg_inf() ? order_key(f[e], v * E - rlead + e) : 0ull;
                            uint32_t who = __ballot_sync(0xffffffffu, k >= floor);
                            while (who != 0u) {
                                const int src = __ffs(who) - 1;
                                who &= who - 1;
                                const Key n = __shfl_sync(0xffffffffu, k, src);
                                if (n >= floor) { // uniform; the floor may have risen since the vote
                                    const int to = __popc(__ballot_sync(0xffffffffu, list > n));
                                    const Key up = __shfl_up_sync(0xffffffffu, list, 1);
                                    list = lane < to ? list : (lane == to ? n : up);
                                    const Key kth = __shfl_sync(0xffffffffu, list, p.top_k - 1);
                                    floor = kth > floor ? kth : floor;
                                }
                            }
                        }
                    }
                }
                sm.found[warp][lane] = list;
                __syncthreads();
                if (list != 0ull && lane < p.top_k) {
                    const int to = place(sm.found, warp, lane, list);
                    if (to < p.top_k)
                        sm.fin[to] = list;
                }
            }
            __syncthreads();
        }

        // ---- join: warps, then the cluster's parts
        Stat st;
        if (warp == 0) {
            st = sm.warp[parity][0];
            for (int w = 1; w < LP_WARPS; ++w)
                st = join(st, sm.warp[parity][w], c);
        }
        const Key *fin = sm.fin;
        if (parts > 1) {
            cg::cluster_group cl = cg::this_cluster();
            if (tid == 0)
                sm.cta = st;
            cl.sync();
            if (part == 0) {
                if (warp == 0)
                    for (int r = 1; r < parts; ++r)
                        st = join(st, cl.map_shared_rank(&sm, r)->cta, c);
                if (TOP) {
                    const Key k = warp < parts ? cl.map_shared_rank(&sm, warp)->fin[lane] : 0ull;
                    sm.lists[warp][lane] = k;
                    if (tid < 32)
                        sm.last[tid] = 0ull;
                    __syncthreads();
                    const int at = k != 0ull ? place(sm.lists, warp, lane, k) : 32;
                    if (at < p.top_k)
                        sm.last[at] = k;
                    __syncthreads();
                    fin = sm.last;
                }
            }
        }
        if (part == 0 && warp == 0) {
            const bool empty = st.m == neg_inf();
            const float logsum = empty ? 0.0f : logf(st.s); // NaN when the row holds a NaN or +infinity
            const bool none = !(logsum == logsum);
            if (lane == 0) {
                if (p.stats != nullptr) {
                    p.stats[2 * (int64_t)rrow] = none ? quiet_nan() : st.m;
                    p.stats[2 * (int64_t)rrow + 1] = logsum;
                }
                if (p.entropy != nullptr)
                    p.entropy[rrow] = empty ? 0.0f : logsum - LN2 * (st.u / st.s);
                if (p.logprob != nullptr) {
                    const int t = p.tokens[rrow];
                    float lp = 0.0f;
                    if (t >= 0 && t < p.V)
                        lp = empty ? neg_inf() : (Vec<T>::widen(rx[t]) - st.m) * p.inv_t - logsum;
                    p.logprob[rrow] = lp;
                }
            }
            if (TOP && lane < p.top_k) {
                const Key k = fin[lane];
                const float lp = k != 0ull ? (key_value(k) - st.m) * p.inv_t - logsum : neg_inf();
                p.top_logprobs[(int64_t)rrow * p.top_k + lane] = none ? quiet_nan() : lp;
                p.top_ids[(int64_t)rrow * p.top_k + lane] = lp > neg_inf() ? key_index(k) : -1;
            }
        }
        if (parts > 1)
            cg::this_cluster().sync(); // the parts' shared memory is read until here
    }
}

// A CTA takes LP_UNROLL * LP_THREADS vectors of one row of dlogits. With
// a = log2 p and one factor for each row, an element is
//   dx = 2^a (q + r a),  q = -t (g + g_H H),  r = -t g_H ln 2,
// and the token's own gets t g on top. a = x c - (m c + log S log2 e), the
// latter held as two fp32 numbers so that p is as good as fp32 allows.
template <typename T, bool BONUS>
__global__ void __launch_bounds__(LP_THREADS, 6) logprob_grad_kernel(LogprobGradParams p, int segs)
{
    constexpr int E = Vec<T>::E;
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
    const float qf = -p.inv_t * (g + gh * H), rf = -p.inv_t * gh * LN2, own = p.inv_t * g;
    // m c + logsum log2 e in two parts; rows of huge values take the difference first
    const float mc = m * c, ml = fmaf(m, c, -mc), ls = logsum * LOG2E;
    const float hi = mc + ls, part = hi - mc, lo = ((mc - (hi - part)) + (ls - part)) + ml;
    const bool huge = !(fabsf(mc) <= 65536.0f);
    const f2 c2 = make_f2(c, c), hi2 = make_f2(-hi, -hi), lo2 = make_f2(-lo, -lo), q2 = make_f2(qf, qf), r2 = make_f2(rf, rf);
    const f2 nm2 = make_f2(-m, -m), ls2 = make_f2(-ls, -ls);
#pragma unroll
    for (int q = 0; q < LP_UNROLL; ++q) {
        const int v = v0 + q * LP_THREADS, i0 = v * E - lead;
        if (v >= nvec)
            break;
        float f[E];
        Vec<T>::unpack(raw[q], f);
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
        if (t >= i0 && t < i0 + E) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                f[e] += i0 + e == t ? own : 0.0f;
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
}

template <typename T> cudaError_t launch_lp(const LogprobParams &p, int num_sms, cudaStream_t st)
{
    // parts of a row: enough CTAs for two a SM, each part at least one vector a thread
    const int nvec = (int)(((int64_t)p.V + Vec<T>::E - 1) / Vec<T>::E);
    int parts = 1;
    while (parts < 8 && (int64_t)p.M * parts < 2 * num_sms && nvec >= 2 * parts * LP_THREADS)
        parts *= 2;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)parts;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    // whole rows: as many CTAs as stay resident, each with several rows one after another
    cfg.gridDim = dim3((unsigned)(parts > 1 || p.M < 4 * num_sms ? p.M * parts : 4 * num_sms));
    cfg.blockDim = dim3(LP_THREADS);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = parts > 1 ? 1 : 0;
    return p.top_k > 0 ? cudaLaunchKernelEx(&cfg, logprob_kernel<T, true>, p, parts)
                       : cudaLaunchKernelEx(&cfg, logprob_kernel<T, false>, p, parts);
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
    if (p.g_entropy != nullptr)
        logprob_grad_kernel<T, true><<<(unsigned)(p.M * segs), LP_THREADS, 0, st>>>(p, segs);
    else
        logprob_grad_kernel<T, false><<<(unsigned)(p.M * segs), LP_THREADS, 0, st>>>(p, segs);
    return cudaGetLastError();
}

cudaError_t launch_logprob_grad(const LogprobGradParams &p, int dtype, cudaStream_t st)
{
    return dtype == LORA_DTYPE_F32 ? launch_grad<float>(p, st) : launch_grad<uint16_t>(p, st);
}

} // namespace rd
