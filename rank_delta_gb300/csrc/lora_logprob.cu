// Log probabilities of given tokens, entropy, softmax statistics and the best
// alternatives of rows of logits, and the gradient of the first two.
//
// With z_v = x_v t (t = inv_temperature), m = max x, d_v = (x_v - m) t:
//   S = sum e^{d_v},  log p_v = d_v - log S,  H = log S - (sum e^{d_v} d_v) / S,
//   dx_v = t [ g (1[v = token] - p_v) - g_H p_v (log p_v + H) ].
//
// logprob_kernel reads a row once: every thread keeps a running maximum with
// S and sum e^d d relative to it and rescales both when a group of its
// elements raises the maximum (rare after the first group). Differences are
// taken before the scaling by t (a row of the type's lowest values is a
// uniform row, and nothing overflows but what is masked), sums are fp32, e^d
// is the hardware's 2^x (about 2^-22 relative).
//
// The best alternatives cost the pass nothing but the maximum it needs anyway:
// of the threads' own best elements the k-th largest is a lower bound of the
// row's k-th best, so only the (exactly k) threads whose best reaches it can
// hold any of the k, and their shares, V / threads elements each, are read
// again from L2. Elements are compared by (value, lowest index first) packed
// into 64 bits, which orders them totally; -0 equals +0.
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
};

// Elements of a row's first 16-byte vector that lie before the row.
template <typename T> __device__ __forceinline__ int row_lead(const T *row)
{
    return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

// Vector c of a row (elements [c E - lead, c E - lead + E)); elements outside
// the row are -infinity and not read.
template <typename T> __device__ __forceinline__ void load_vec(const T *row, int V, int lead, int c, float (&f)[Vec<T>::E])
{
    constexpr int E = Vec<T>::E;
    const int i0 = c * E - lead;
    if (i0 >= 0 && i0 + E <= V) {
        Vec<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(row + i0)), f);
    } else {
#pragma unroll
        for (int q = 0; q < E; ++q)
            f[q] = i0 + q >= 0 && i0 + q < V ? Vec<T>::widen(row[i0 + q]) : neg_inf();
    }
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

// The running statistics of part of a row: maximum, sum of 2^a and sum of
// 2^a a with a = (x - maximum) t log2 e.
struct Stat {
    float m, s, u;
};

__device__ __forceinline__ Stat join(Stat a, Stat b, float c)
{
    Stat r;
    r.m = max_nan(a.m, b.m);
    const float mm = r.m == neg_inf() ? 0.0f : r.m;
    // a part without elements (m = -inf) holds s = u = 0
    const float da = a.m == neg_inf() ? 0.0f : max_nan((a.m - mm) * c, -1000.0f);
    const float db = b.m == neg_inf() ? 0.0f : max_nan((b.m - mm) * c, -1000.0f);
    const float fa = exp2_fast(da), fb = exp2_fast(db);
    r.s = fa * a.s + fb * b.s;
    r.u = fa * (a.u + da * a.s) + fb * (b.u + db * b.s);
    return r;
}

struct LpShared {
    Stat warp[LP_WARPS];
    Stat cta;
    unsigned long long lists[LP_WARPS][32];
    unsigned long long fin[32]; // the CTA's best, descending
    unsigned long long bound;
    int picked[LP_THREADS];
    int npicked;
};

// The k best of n <= 32 descending lists of 32 (0 = no element), by one warp:
// lane l holds the head of list l. out(i, key) is called by every lane.
template <typename At, typename Out>
__device__ __forceinline__ void merge_lists(int n, int k, int lane, At at, Out out)
{
    int pos = 0;
    unsigned long long head = lane < n ? at(lane, 0) : 0ull;
    for (int i = 0; i < k; ++i) {
        const unsigned long long best = warp_max_key(head);
        out(i, best);
        if (best != 0ull && head == best) {
            ++pos;
            head = pos < 32 ? at(lane, pos) : 0ull;
        }
    }
}

} // namespace

template <typename T, bool TOP>
__global__ void __launch_bounds__(LP_THREADS) logprob_kernel(LogprobParams p, int parts)
{
    constexpr int E = Vec<T>::E;
    __shared__ LpShared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / parts, part = blockIdx.x % parts;
    const T *x = static_cast<const T *>(p.logits) + (int64_t)row * p.stride;
    const int lead = row_lead(x);
    const int nvec = (int)(((int64_t)lead + p.V + E - 1) / E);
    const int per = (nvec + parts - 1) / parts;
    const int vb = part * per, ve = min(nvec, vb + per);
    const float c = p.inv_t * LOG2E;

    if (blockIdx.x == 0) { // the call's status: any token past the vocabulary
        int bad = 0;
        if (p.tokens != nullptr)
            for (int i = tid; i < p.M; i += LP_THREADS)
                bad |= p.tokens[i] >= p.V;
        bad = __syncthreads_or(bad);
        if (tid == 0)
            status_begin(p.status, bad ? (uint32_t)LORA_FLAG_TOKEN_RANGE : 0u);
    }

    // ---- the pass
    float m = neg_inf();
    int best_vec = -1; // first vector of the group that set the maximum
    f2 s2 = make_f2(0.0f, 0.0f), u2 = s2;
    const f2 c2 = make_f2(c, c);
    for (int v0 = vb + tid; v0 < ve; v0 += LP_UNROLL * LP_THREADS) {
        float f[LP_UNROLL][E];
#pragma unroll
        for (int q = 0; q < LP_UNROLL; ++q) {
            const int v = v0 + q * LP_THREADS;
            if (v < ve) {
                load_vec(x, p.V, lead, v, f[q]);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    f[q][e] = neg_inf();
            }
        }
        float gm = neg_inf();
#pragma unroll
        for (int q = 0; q < LP_UNROLL; ++q) {
            float vm = f[q][0];
#pragma unroll
            for (int e = 1; e < E; ++e)
                vm = max_nan(vm, f[q][e]);
            gm = max_nan(gm, vm);
        }
        if (!(gm <= m)) {
            if (m != neg_inf()) { // rescale what has been summed
                const float d = max_nan((m - gm) * c, -1000.0f);
                const float w = exp2_fast(d);
                const f2 d2 = make_f2(d, d), w2 = make_f2(w, w);
                u2 = mul_f2(w2, fma_f2(d2, s2, u2));
                s2 = mul_f2(w2, s2);
            }
            m = gm;
            best_vec = v0;
        }
        const float nm = m == neg_inf() ? 0.0f : -m;
        const f2 nm2 = make_f2(nm, nm);
#pragma unroll
        for (int q = 0; q < LP_UNROLL; ++q)
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                float a0, a1;
                split_f2(mul_f2(add_f2(make_f2(f[q][e], f[q][e + 1]), nm2), c2), a0, a1);
                // masked elements add nothing: 2^-1000 is 0, and so is its product
                const f2 a2 = make_f2(max_nan(a0, -1000.0f), max_nan(a1, -1000.0f));
                split_f2(a2, a0, a1);
                const f2 e2 = make_f2(exp2_fast(a0), exp2_fast(a1));
                s2 = add_f2(s2, e2);
                u2 = fma_f2(e2, a2, u2);
            }
    }
    Stat st;
    float h0, h1;
    st.m = m;
    split_f2(s2, h0, h1);
    st.s = h0 + h1;
    split_f2(u2, h0, h1);
    st.u = h0 + h1;

    // ---- this thread's best element, the warp's in order
    if (TOP) {
        unsigned long long mine = 0ull;
        if (m > neg_inf()) {
            for (int q = LP_UNROLL - 1; q >= 0; --q) { // the lowest index is found last
                const int v = best_vec + q * LP_THREADS;
                if (v < ve) {
                    float f[E];
                    load_vec(x, p.V, lead, v, f);
#pragma unroll
                    for (int e = E - 1; e >= 0; --e)
                        if (f[e] == m)
                            mine = order_key(m, v * E - lead + e);
                }
            }
        }
        sm.lists[warp][lane] = warp_sort_desc(mine, lane);
        if (tid == 0)
            sm.npicked = 0;
        __syncthreads();
        if (warp == 0) {
            unsigned long long kth = 0ull;
            merge_lists(LP_WARPS, p.top_k, lane, [&](int l, int i) { return sm.lists[l][i]; },
                        [&](int, unsigned long long k) { kth = k; });
            if (lane == 0)
                sm.bound = kth != 0ull ? kth : 1ull; // fewer than k threads hold any: every element counts
        }
        __syncthreads();
        const unsigned long long bound = sm.bound;
        if (mine >= bound)
            sm.picked[atomicAdd(&sm.npicked, 1)] = tid; // any order: what comes of it is ordered by key
        __syncthreads();
        // ---- the picked threads' shares again, a warp each
        unsigned long long list = 0ull, floor = bound; // lane i: the i-th best so far
        for (int i = warp; i < sm.npicked; i += LP_WARPS) {
            const int first = vb + sm.picked[i];
            for (int w0 = first; w0 < ve; w0 += 32 * LP_THREADS) {
                const int v = w0 + lane * LP_THREADS;
                float f[E];
                if (v < ve) {
                    load_vec(x, p.V, lead, v, f);
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        f[e] = neg_inf();
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const unsigned long long k = f[e] > neg_inf() ? order_key(f[e], v * E - lead + e) : 0ull;
                    uint32_t who = __ballot_sync(0xffffffffu, k >= floor);
                    while (who != 0u) {
                        const int src = __ffs(who) - 1;
                        who &= who - 1;
                        const unsigned long long n = __shfl_sync(0xffffffffu, k, src);
                        if (n >= floor) { // uniform; the floor may have risen since the vote
                            const int at = __popc(__ballot_sync(0xffffffffu, list > n));
                            const unsigned long long up = __shfl_up_sync(0xffffffffu, list, 1);
                            list = lane < at ? list : (lane == at ? n : up);
                            const unsigned long long kth = __shfl_sync(0xffffffffu, list, p.top_k - 1);
                            floor = kth > floor ? kth : floor;
                        }
                    }
                }
            }
        }
        sm.lists[warp][lane] = list;
    }

    // ---- join: lanes, warps, then the cluster's parts
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Stat b;
        b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
        b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
        b.u = __shfl_xor_sync(0xffffffffu, st.u, o);
        st = lane & o ? join(b, st, c) : join(st, b, c); // the same order in both lanes
    }
    if (lane == 0)
        sm.warp[warp] = st;
    __syncthreads();
    if (warp == 0) {
        st = sm.warp[0];
        for (int w = 1; w < LP_WARPS; ++w)
            st = join(st, sm.warp[w], c);
        if (lane == 0)
            sm.cta = st;
        if (TOP && parts > 1)
            merge_lists(LP_WARPS, p.top_k, lane, [&](int l, int i) { return sm.lists[l][i]; },
                        [&](int i, unsigned long long k) {
                            if (lane == 0)
                                sm.fin[i] = k;
                        });
        if (TOP && parts > 1 && lane >= p.top_k)
            sm.fin[lane] = 0ull;
    }
    if (parts > 1) {
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        if (part == 0 && warp == 0)
            for (int r = 1; r < parts; ++r)
                st = join(st, cl.map_shared_rank(&sm, r)->cta, c);
    }
    if (part == 0 && warp == 0) {
        const bool empty = st.m == neg_inf();
        const float logsum = empty ? 0.0f : logf(st.s); // NaN when the row holds a NaN or +infinity
        const bool none = !(logsum == logsum);
        if (lane == 0) {
            if (p.stats != nullptr) {
                p.stats[2 * (int64_t)row] = none ? quiet_nan() : st.m;
                p.stats[2 * (int64_t)row + 1] = logsum;
            }
            if (p.entropy != nullptr)
                p.entropy[row] = empty ? 0.0f : logsum - LN2 * (st.u / st.s);
            if (p.logprob != nullptr) {
                const int t = p.tokens[row];
                float lp = 0.0f;
                if (t >= 0 && t < p.V)
                    lp = empty ? neg_inf() : (Vec<T>::widen(x[t]) - st.m) * p.inv_t - logsum;
                p.logprob[row] = lp;
            }
        }
        if (TOP) {
            auto put = [&](int i, unsigned long long k) {
                if (lane == 0) {
                    const float lp = k != 0ull ? (key_value(k) - st.m) * p.inv_t - logsum : neg_inf();
                    const bool some = k != 0ull && lp > neg_inf();
                    p.top_logprobs[(int64_t)row * p.top_k + i] = none ? quiet_nan() : lp;
                    p.top_ids[(int64_t)row * p.top_k + i] = some ? key_index(k) : -1;
                }
            };
            if (parts > 1) {
                cg::cluster_group cl = cg::this_cluster();
                merge_lists(parts, p.top_k, lane,
                            [&](int l, int i) { return cl.map_shared_rank(&sm, l)->fin[i]; }, put);
            } else {
                merge_lists(LP_WARPS, p.top_k, lane, [&](int l, int i) { return sm.lists[l][i]; }, put);
            }
        }
    }
    if (parts > 1)
        cg::this_cluster().sync(); // the parts' shared memory is read until here
}

// A CTA takes LP_UNROLL * LP_THREADS vectors of one row of dlogits.
template <typename T>
__global__ void __launch_bounds__(LP_THREADS) logprob_grad_kernel(LogprobGradParams p, int segs)
{
    constexpr int E = Vec<T>::E;
    const int row = blockIdx.x / segs, seg = blockIdx.x % segs;
    const T *x = static_cast<const T *>(p.logits) + (int64_t)row * p.stride;
    T *dx = static_cast<T *>(p.dlogits) + (int64_t)row * p.d_stride;
    const int lead = row_lead(dx);
    const bool same = row_lead(x) == lead; // both rows split into the same vectors
    const float m = p.stats[2 * (int64_t)row], logsum = p.stats[2 * (int64_t)row + 1];
    int t = p.tokens != nullptr ? p.tokens[row] : -1;
    const float g = t >= 0 && t < p.V && p.g_logprob != nullptr ? p.g_logprob[row] : 0.0f;
    const float gh = p.g_entropy != nullptr ? p.g_entropy[row] : 0.0f;
    const float H = p.g_entropy != nullptr ? p.entropy[row] : 0.0f;
    const bool empty = m == neg_inf();
    const int nvec = (int)(((int64_t)lead + p.V + E - 1) / E);
    const int v0 = seg * (LP_UNROLL * LP_THREADS) + threadIdx.x;
    float f[LP_UNROLL][E];
#pragma unroll
    for (int q = 0; q < LP_UNROLL; ++q) {
        const int v = v0 + q * LP_THREADS, i0 = v * E - lead;
        if (v < nvec) {
            if (same && i0 >= 0 && i0 + E <= p.V) {
                Vec<T>::unpack(*reinterpret_cast<const uint4 *>(x + i0), f[q]);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    f[q][e] = i0 + e >= 0 && i0 + e < p.V ? Vec<T>::widen(x[i0 + e]) : neg_inf();
            }
        }
    }
#pragma unroll
    for (int q = 0; q < LP_UNROLL; ++q) {
        const int v = v0 + q * LP_THREADS, i0 = v * E - lead;
        if (v >= nvec)
            break;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float lp = (f[q][e] - m) * p.inv_t - logsum;
            const float pr = exp2_fast(lp * LOG2E);
            float d = g * ((i0 + e == t ? 1.0f : 0.0f) - pr);
            d -= pr != 0.0f ? gh * pr * (lp + H) : 0.0f; // 0 log 0 is 0
            f[q][e] = empty ? 0.0f : d * p.inv_t;
        }
        if (i0 >= 0 && i0 + E <= p.V) {
            *reinterpret_cast<uint4 *>(dx + i0) = Vec<T>::pack(f[q]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (i0 + e >= 0 && i0 + e < p.V)
                    dx[i0 + e] = Vec<T>::narrow(f[q][e]);
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
    cfg.gridDim = dim3((unsigned)(p.M * parts));
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
    logprob_grad_kernel<T><<<(unsigned)(p.M * segs), LP_THREADS, 0, st>>>(p, segs);
    return cudaGetLastError();
}

cudaError_t launch_logprob_grad(const LogprobGradParams &p, int dtype, cudaStream_t st)
{
    return dtype == LORA_DTYPE_F32 ? launch_grad<float>(p, st) : launch_grad<uint16_t>(p, st);
}

} // namespace rd
