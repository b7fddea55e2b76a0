// The next token of each row of logits, from a given uniform number, under the
// row's own temperature, top-k, top-p and min-p.
//
// With m = max x and weights w_v = e^{(x_v - m) t}, the elements in the order
// (x descending, index ascending): top-k keeps the first k, top-p the shortest
// prefix of those with p of their weight, min-p those with w >= min_p. Each is a
// prefix, so what is kept is a prefix too: a value and how many of the elements
// equal to it. The token is the first kept one, in index order, at which the
// running sum of weights exceeds u times their sum.
//
// Tokens are compared, not rounded, so every decision has to be that of exact
// arithmetic. Weights that decide are computed to about 2^-43 of themselves and
// summed as 64-bit integers, whose sums do not depend on their order. Sums over
// the whole vocabulary are first taken in fp32 with a bound on their error; only
// a row whose decision lies within the bound is gone through again exactly.
//
// A row lies in shared memory, spread over a cluster where it is long or rows
// are few (row_team.cuh). Of the threads' own maxima, which cost nothing, those that
// top-k or top-p need give a bound that every kept element reaches; the few
// elements that do are listed, and one warp sorts them while the others are at the
// next row (in a cluster, the leading CTA counts each its place). A row of which
// more may be kept than the list holds, or that the list leaves open, is gone through
// by fine_row: top-k by counting in bins of the values' order-preserving bits, top-p
// in bins of the exponent, whose one bin that the border lies in is listed, sums in
// fp32 with the exponent's rounding put right. What that leaves open exact_row
// decides, by exact sums in bins of the values' bits, as often as it takes to reach
// one value. Rows are taken as teams get through, since those take several times
// as long. Hundreds of rows are read through registers instead, by warps that do
// nothing else.
//
// Times below are of calls one after another on a GB300, on rows as perf/more_operators.py
// makes them for the sizes and settings named (seed 1), unless they say otherwise.
#include <cooperative_groups.h>

#include "behind.cuh"
#include "lora_sample.cuh"
#include "row_team.cuh"

namespace rd {

namespace cg = cooperative_groups;

namespace {

constexpr int LIST = 128;       // elements that may be kept, listed
constexpr int REDO = 4;
constexpr int BINS = 256;
constexpr int GUIDE = 64;       // bins of the threads' maxima, two a lane
constexpr int LIST_SCALE = 53;  // a listed weight w is the integer w 2^53: LIST of them fit
constexpr int BAR_TEAM = 1, BAR_LIST = 2, BAR_GIVEN = 3, BAR_TAKEN = 4;

struct __align__(16) Entry {
    float x;
    int i;
    u64 w;
};

// One row's settings.
struct Settings {
    float u, t, p, least;
    int k;

    // Nothing lies at 1 of the sum; NaN and what is out of range stay what they are.
    static __device__ __forceinline__ float below_one(float u) { return u == 1.0f ? 0x1.fffffep-1f : u; }
    // One of the five on its way into shared memory, by thread `at`; valid for all once it has waited and they have met.
    static __device__ __forceinline__ void fetch(const SampleParams &a, int row, int at, uint32_t *to)
    {
        const uint32_t *from = reinterpret_cast<const uint32_t *>(at == 0   ? a.uniform
                                                                  : at == 1 ? a.inv_t
                                                                  : at == 2 ? a.top_p
                                                                  : at == 3 ? a.min_p
                                                                            : reinterpret_cast<const float *>(a.top_k));
        if (from != nullptr)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to + at)), "l"(from + row) : "memory");
        else
            to[at] = at == 1 || at == 2 ? 0x3f800000u : 0u; // 1, or nothing
    }
    __device__ __forceinline__ void take(const uint32_t *from)
    {
        u = below_one(__uint_as_float(from[0]));
        t = __uint_as_float(from[1]);
        p = __uint_as_float(from[2]);
        least = __uint_as_float(from[3]);
        k = (int)from[4];
    }
    __device__ __forceinline__ void read(const SampleParams &a, int row)
    {
        u = below_one(a.uniform[row]);
        t = a.inv_t != nullptr ? a.inv_t[row] : 1.0f;
        p = a.top_p != nullptr ? a.top_p[row] : 1.0f;
        least = a.min_p != nullptr ? a.min_p[row] : 0.0f;
        k = a.top_k != nullptr ? a.top_k[row] : 0;
    }
    __device__ __forceinline__ bool bad() const
    {
        return !(t >= 0x1p-64f) || !(u >= 0.0f && u <= 1.0f) || !(p == p) || !(least == least);
    }
    __device__ __forceinline__ bool greedy() const { return k == 1 || t > 0x1p64f || p <= 0.0f || least > 1.0f; }
    __device__ __forceinline__ int limit(int V) const { return k <= 0 || k >= V ? 0 : k; }
};

// What a row's list is worked out with.
struct ListTask {
    int n, k, equal;
    u64 rest;         // fp32 sum over the vocabulary but `equal` maxima, 2^43 times, where top-p is of all
    float margin;
    bool by_p, least_bound; // what min-p keeps is listed in whole, and no more
    int row;
    Settings a;
    Scale s;
};

template <int W> struct Shared {
    static constexpr int SLOTS = MAX_PARTS * W;
    u64 powers[32];
    uint64_t bars[W];
    // the team's warps write these for all its CTAs; rows take turns at two of each
    float maxima[2][SLOTS], minima[2][SLOTS];
    u64 rest[2][SLOTS];
    int equal[2][SLOTS];
    int alive[2]; // the leading CTA's
    int next[2], open[2]; // the row after next; the turn of a row that was left open
    int first[2];
    alignas(8) uint32_t guide[2][GUIDE]; // counts, or weights in 2^-20
    uint32_t settings[2][5];
    int listed;
    ListTask task, taken; // to be worked out; the ninth warp's copy
    Entry few[LIST];
    int redo[REDO], redone[2]; // rows it left open, and how many so far; as many as are known at a row's maximum
    int left_open, out_of_range, late;
    // of a row that is gone through exactly
    u64 sums[6][W], cta_sum[6];
    int firsts[W], cta_first;
    float top[W], cta_top, least;
    u64 warp_mass[W], cta_mass;
    int warp_ties[W], cta_ties;
    struct {
        int bin, count, ties;
        u64 mass;
    } cross;
    u64 scan_mass[W];
    int scan_count[W];
    float queue[W][64];
    union {
        Entry list[LIST];
        struct {
            uint32_t low[BINS], high[BINS], count[BINS]; // a sum of weights as two words, how many
        } bins;
    };
};

// p as a fraction of 2^64, for 0 <= p < 1, and the product with an integer, rounded up.
__device__ __forceinline__ u64 fraction(float p) { return (u64)(p * 18446744073709551616.0f); }
__device__ __forceinline__ u64 share_up(u64 f, u64 z) { return __umul64hi(f, z) + (f * z != 0ull); }

__device__ __forceinline__ Scale scale_of(float m, float t)
{
    constexpr float L_HI = 0x1.715476p+0f, L_LO = 0x1.4ae0c0p-26f; // log2 e
    Scale s;
    s.m = m;
    s.c = __fmul_rn(t, L_HI);
    s.c_low = fmaf(t, L_HI, -s.c) + t * L_LO;
    return s;
}

// How near a border a draw may be told from sums that are off by `margin`, all of it
// in `rest` of the `total`: what precedes the border, less u of the total, is (1 - u)
// of what precedes it less u of what follows. Only what was summed once does so: sums
// that are taken apart again to look into them may come to `apart` more or less in parts.
// Each of V numbers loses up to a unit when it becomes an integer.
__device__ __forceinline__ u64 draw_slack(float u, u64 total, u64 rest, float margin, float apart, int V)
{
    const float t = (float)total, r = fmaxf((float)rest, 1.0f);
    const float part = ((1.0f - u) * fminf(r, u * t) + u * fminf(r, (1.0f - u) * t)) / r;
    return (u64)((margin * part + apart) * 1.001f * SUM_UNITS) + (u64)V + 4ull;
}

// What sums of fp32 weights over V elements are off by, that come to `sum`. Each weight
// is off by 3 roundings of its exponent, 2^-24 |a| ln 2 each, and 2^-22; its part of the
// sum by `adds` more. Weighted, |a| is on average at most log2 of V / min(1, sum),
// since entropy is at most log V.
__device__ __forceinline__ float sum_margin(float sum, int V, float adds)
{
    return sum * 0x1p-24f * (2.3f * (log2f((float)V) + fmaxf(0.0f, -log2f(fmaxf(sum, 1e-30f)))) + 5.0f + adds) + (float)V * SUM_UNIT;
}

// A value below which a weight is less than 2^a, a < 0, whatever is rounded on the way.
__device__ __forceinline__ float value_at(const Scale &s, float a)
{
    const float d = -a / s.c;
    return (s.m - d) - (fabsf(s.m) + d) * 0x1p-21f;
}

// The CTA's W warps.
template <int W> __device__ __forceinline__ void cta_sync()
{
    __syncwarp();
    named_bar_sync(BAR_TEAM, W * 32);
}

// All of the team's, and what they wrote.
template <int W> __device__ __forceinline__ void team_sync(int parts)
{
    __syncwarp();
    if (parts > 1) {
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    } else {
        named_bar_sync(BAR_TEAM, W * 32);
    }
}

// The sum of a value over all threads of the team, by way of place AT. The others' CTAs
// read this one's after the team has met: a place is written again only behind another
// meeting of the team (a sum at another place, say), not behind barriers of a CTA alone.
template <int AT, int W> __device__ __forceinline__ u64 team_sum(Shared<W> &sm, u64 v, int parts)
{
    const int lane = threadIdx.x & 31;
    v = warp_sum64(v);
    if (lane == 0)
        sm.sums[AT][threadIdx.x >> 5] = v;
    cta_sync<W>();
    v = 0ull;
#pragma unroll
    for (int w = 0; w < W; ++w)
        v += sm.sums[AT][w];
    if (parts > 1) {
        cg::cluster_group cl = cg::this_cluster();
        if (threadIdx.x == 0)
            sm.cta_sum[AT] = v;
        team_sync<W>(parts);
        v = warp_sum64(lane < parts ? cl.map_shared_rank(&sm, lane)->cta_sum[AT] : 0ull);
    }
    return v;
}

// The lowest index in the team.
template <int W> __device__ __forceinline__ int team_first(Shared<W> &sm, int i, int parts)
{
    const int lane = threadIdx.x & 31;
    i = __reduce_min_sync(0xffffffffu, i);
    if (lane == 0)
        sm.firsts[threadIdx.x >> 5] = i;
    cta_sync<W>();
#pragma unroll
    for (int w = 0; w < W; ++w)
        i = min(i, sm.firsts[w]);
    if (parts > 1) {
        cg::cluster_group cl = cg::this_cluster();
        if (threadIdx.x == 0)
            sm.cta_first = i;
        team_sync<W>(parts);
        i = __reduce_min_sync(0xffffffffu, lane < parts ? cl.map_shared_rank(&sm, lane)->cta_first : 0x7fffffff);
    }
    return i;
}

template <typename T, int W> __device__ __forceinline__ float element(const Row<T, W> &r, int v, int e)
{
    return Vec<T>::widen(reinterpret_cast<const T *>(r.vec + v)[e]);
}

// The first of this thread's elements that is at least `bound`.
template <typename T, int W> __device__ __forceinline__ int first_from(const Row<T, W> &r, float bound)
{
    constexpr int E = Vec<T>::E;
    for (int v = r.w0 + r.lane; v < r.w1; v += 32) {
        const uint4 raw = r.vec[v];
        if (Vec<T>::largest(raw) >= bound) {
            float f[E];
            Vec<T>::unpack(raw, f);
            int at = 0x7fffffff;
#pragma unroll
            for (int e = E - 1; e >= 0; --e)
                at = f[e] >= bound ? r.first + v * E + e : at;
            return at;
        }
    }
    return 0x7fffffff;
}

// How many of this thread's elements are not masked.
template <typename T, int W> __device__ __forceinline__ int alive_of(const Row<T, W> &r)
{
    constexpr int E = Vec<T>::E;
    int n = 0;
#pragma unroll 2
    for (int v = r.w0 + r.lane; v < r.w1; v += 32) {
        const uint4 raw = r.vec[v];
        if (Vec<T>::smallest(raw) > neg_inf()) {
            n += E;
        } else {
            float f[E];
            Vec<T>::unpack(raw, f);
#pragma unroll
            for (int e = 0; e < E; ++e)
                n += f[e] > neg_inf();
        }
    }
    return n;
}

// f(x) for each element of the warp's run in [from, to], 32 of them at a time;
// f is called by the whole warp, with -infinity where a lane has none.
template <typename T, int W, typename F>
__device__ __forceinline__ void each_between(const Row<T, W> &r, float *queue, float from, float to, F f)
{
    constexpr int E = Vec<T>::E;
    if (from <= LEAST) { // nearly all; f leaves out what is above `to`
        for (int v0 = r.w0; v0 < r.w1; v0 += 32) {
            float x[E];
            Vec<T>::unpack(v0 + r.lane < r.w1 ? r.vec[v0 + r.lane] : empty_vec<T>(), x);
#pragma unroll
            for (int e = 0; e < E; ++e)
                f(x[e]);
        }
        return;
    }
    int held = 0;
    for (int v0 = r.w0; v0 < r.w1; v0 += 32) {
        const int v = v0 + r.lane;
        const uint4 raw = v < r.w1 ? r.vec[v] : empty_vec<T>();
        uint32_t hits = 0u;
        if (Vec<T>::largest(raw) >= from) {
            float x[E];
            Vec<T>::unpack(raw, x);
#pragma unroll
            for (int e = 0; e < E; ++e)
                hits |= x[e] >= from && x[e] <= to ? 1u << e : 0u;
        }
        uint32_t any;
        while ((any = __ballot_sync(0xffffffffu, hits != 0u)) != 0u) {
            if (hits != 0u)
                queue[held + __popc(any & ((1u << r.lane) - 1u))] = element(r, v, __ffs(hits) - 1);
            hits &= hits - 1u;
            held += __popc(any);
            __syncwarp();
            if (held >= 32) {
                const float x = queue[r.lane], rest = queue[32 + r.lane];
                __syncwarp();
                queue[r.lane] = rest;
                held -= 32;
                __syncwarp();
                f(x);
            }
        }
    }
    __syncwarp();
    if (held > 0)
        f(r.lane < held ? queue[r.lane] : neg_inf());
    __syncwarp();
}

// The lowest value that min-p keeps, min_p at most 1: the first of m + log(min_p) / t upwards. That sum may be
// rounded past a neighbour; the difference of a value and m is exact, or so long that its last digits say nothing.
__device__ __noinline__ float least_kept(float m, float t, float min_p)
{
    const double d = log((double)min_p) / (double)t, v = (double)m + d;
    float x = v < (double)LEAST ? LEAST : __double2float_ru(v);
    if (x < m && (double)x - (double)m < d)
        x = nextafterf(x, m);
    const float below = nextafterf(x, neg_inf());
    return x > LEAST && (double)below - (double)m >= d ? below : x;
}

// What is kept: elements above `x`, and the first `ties` of those equal to it.
struct Cut {
    float x;
    int ties;
};

// A drawn element, as one lane found it.
struct Drawn {
    int i;
    float x;
    u64 before, w;
};

// The element of the warp's run at which the running sum of fp32 weights exceeds
// `target` (less than the run's sum), by the lane that finds it.
template <typename T, int W>
__device__ __forceinline__ bool walk(const Row<T, W> &r, const Scale &s, u64 target, Drawn &d)
{
    constexpr int E = Vec<T>::E;
    u64 before = 0ull;
    for (int v0 = r.w0; v0 < r.w1; v0 += 128) {
        u64 mine[4], all[4], sum = 0ull;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int v = v0 + 32 * j + r.lane;
            int equal = 0;
            mine[j] = as_fixed(vector_rest<T, true>(v < r.w1 ? r.vec[v] : empty_vec<T>(), s, equal), SUM_SCALE);
            mine[j] += (u64)equal << SUM_SCALE;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sum += all[j] = warp_sum64(mine[j]);
        if (target >= before + sum) {
            before += sum;
            continue;
        }
        int j = 0; // the 32 vectors that it lies in
        u64 own = mine[0];
#pragma unroll
        for (int q = 0; q < 3; ++q)
            if (j == q && target >= before + all[q]) {
                before += all[q];
                j = q + 1;
                own = mine[q + 1];
            }
        u64 upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 n = __shfl_up_sync(0xffffffffu, upto, o);
            upto += r.lane >= o ? n : 0ull;
        }
        const u64 at = before + upto - own;
        const bool here = target >= at && target < at + own;
        if (here) {
            const int v = v0 + 32 * j + r.lane;
            u64 run = at;
            d = Drawn{0, s.m, at, 0ull};
            for (int e = 0; e < E; ++e) {
                const float x = element(r, v, e);
                const u64 w = x == s.m ? 1ull << SUM_SCALE : as_fixed(exp2_fast(__fmul_rn(x - s.m, s.c)), SUM_SCALE);
                if (w > 0ull)
                    d = Drawn{r.first + v * E + e, x, run, w};
                run += w;
                if (run > target)
                    break;
            }
        }
        return here;
    }
    return false;
}

// The same of exact weights of what is kept.
template <typename T, int W>
__device__ __forceinline__ bool walk_exact(const Row<T, W> &r, const Scale &s, Cut cut, int bits, u64 tie_weight, const u64 *powers,
                                           u64 target, Drawn &d)
{
    constexpr int E = Vec<T>::E;
    u64 before = 0ull;
    for (int v0 = r.w0; v0 < r.w1; v0 += 32) {
        const int v = v0 + r.lane;
        const bool any = v < r.w1 && Vec<T>::largest(r.vec[v]) >= cut.x;
        if (!__any_sync(0xffffffffu, any))
            continue;
        u64 mine = 0ull;
        int ties = 0;
        if (any) {
            float x[E];
            Vec<T>::unpack(r.vec[v], x);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const u64 w = weight(s, x[e], bits, powers);
                mine += x[e] > cut.x ? w : 0ull;
                ties += x[e] == cut.x;
            }
        }
        // of the lanes in order
        int upto_ties = ties;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, upto_ties, o);
            upto_ties += r.lane >= o ? n : 0;
        }
        int allowed = min(max(cut.ties - (upto_ties - ties), 0), ties);
        mine += (u64)allowed * tie_weight;
        cut.ties -= min(cut.ties, __shfl_sync(0xffffffffu, upto_ties, 31));
        u64 upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 n = __shfl_up_sync(0xffffffffu, upto, o);
            upto += r.lane >= o ? n : 0ull;
        }
        const u64 all = __shfl_sync(0xffffffffu, upto, 31);
        if (target >= before + all) {
            before += all;
            continue;
        }
        const u64 at = before + upto - mine;
        const bool here = target >= at && target < at + mine;
        if (here) {
            u64 run = at;
            d = Drawn{0, s.m, at, 0ull};
            for (int e = 0; e < E; ++e) {
                const float x = element(r, v, e);
                u64 w = 0ull;
                if (x > cut.x)
                    w = weight(s, x, bits, powers);
                else if (x == cut.x && allowed > 0) {
                    w = tie_weight;
                    --allowed;
                }
                if (w > 0ull)
                    d = Drawn{r.first + v * E + e, x, run, w};
                run += w;
                if (run > target)
                    break;
            }
        }
        return here;
    }
    return false;
}

// The thread's bins, over the team, and where the running count (or weight) over
// the bins reaches `target`: written to sm.cross by the thread that has the bin.
template <bool BY_MASS, int W> __device__ __forceinline__ void cross_bins(Shared<W> &sm, int above, u64 above_mass, u64 target, int parts)
{
    constexpr int OWN = BINS / (W * 32);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cg::cluster_group cl = cg::this_cluster();
    team_sync<W>(parts); // the bins are counted
    int c[OWN], uc = 0;
    u64 m[OWN], um = 0ull;
#pragma unroll
    for (int b = 0; b < OWN; ++b) {
        c[b] = (int)sm.bins.count[OWN * tid + b];
        m[b] = BY_MASS ? (u64)sm.bins.high[OWN * tid + b] << 32 | sm.bins.low[OWN * tid + b] : 0ull;
        if (parts > 1) { // the others', all on their way at once
            const int part = (int)cl.block_rank();
#pragma unroll
            for (int q = 1; q < MAX_PARTS; ++q) {
                const auto &o = cl.map_shared_rank(&sm, (part + q) & (parts - 1))->bins;
                c[b] += q < parts ? (int)o.count[OWN * tid + b] : 0;
                if (BY_MASS)
                    m[b] += q < parts ? (u64)o.high[OWN * tid + b] << 32 | o.low[OWN * tid + b] : 0ull;
            }
        }
        uc += c[b];
        um += m[b];
    }
    const int own_c = uc;
    const u64 own_m = um;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int nc = __shfl_up_sync(0xffffffffu, uc, o);
        uc += lane >= o ? nc : 0;
        if (BY_MASS) {
            const u64 nm = __shfl_up_sync(0xffffffffu, um, o);
            um += lane >= o ? nm : 0ull;
        }
    }
    if (lane == 31) {
        sm.scan_count[warp] = uc;
        sm.scan_mass[warp] = um;
    }
    cta_sync<W>();
    uc += above - own_c;
    um += above_mass - own_m;
    for (int w = 0; w < warp; ++w) {
        uc += sm.scan_count[w];
        um += sm.scan_mass[w];
    }
#pragma unroll
    for (int b = 0; b < OWN; ++b) {
        const u64 from = BY_MASS ? um : (u64)uc, size = BY_MASS ? m[b] : (u64)c[b];
        if (from < target && from + size >= target) { // one bin of one thread
            sm.cross.bin = OWN * tid + b;
            sm.cross.count = uc;
            sm.cross.ties = c[b];
            sm.cross.mass = um;
        }
        uc += c[b];
        um += m[b];
    }
    team_sync<W>(parts); // and read
}

template <int W> __device__ __forceinline__ void clear_bins(Shared<W> &sm)
{
    for (int b = threadIdx.x; b < BINS; b += W * 32)
        sm.bins.low[b] = sm.bins.high[b] = sm.bins.count[b] = 0u;
    if (threadIdx.x == 0)
        sm.cross.bin = -1;
    cta_sync<W>();
}

// Bits that take `width` into BINS bins.
__device__ __forceinline__ int bin_shift(uint32_t width) { return max(0, 32 - __clz((int)width) - 8); }

// Where the running count (or weight) over the elements in descending order reaches
// `target`: the value, what lies above it and how many equal it. Only elements in
// [low, high] are looked at; `above` and `above_mass` say what lies above those.
// False where they do not reach it.
struct Crossing {
    float x;
    int above, ties;
    u64 above_mass;
};
template <bool BY_MASS, typename T, int W>
__device__ __noinline__ bool descend(Shared<W> &sm, const Row<T, W> r, const Scale s, int bits, u64 target, float low, float high,
                                     int parts, Crossing &out)
{
    constexpr int DROP = sizeof(T) == 2 ? 16 : 0; // bits that say nothing
    constexpr uint32_t NOTHING = (1u << DROP) - 1u;
    uint32_t most = order_bits(high), least = order_bits(low), hi = most >> DROP, lo = least >> DROP;
    for (;;) {
        const int shift = bin_shift(hi - lo);
        clear_bins(sm);
        each_between(r, sm.queue[r.warp], order_value(least), order_value(most), [&](float x) {
            const uint32_t k = order_bits(x);
            if (k < least || k > most)
                return;
            const uint32_t bin = (hi - (k >> DROP)) >> shift;
            atomicAdd(&sm.bins.count[bin], 1u);
            if (BY_MASS) {
                const u64 w = weight(s, x, bits, sm.powers);
                const uint32_t l = (uint32_t)w, was = atomicAdd(&sm.bins.low[bin], l);
                const uint32_t h = (uint32_t)(w >> 32) + (was + l < l ? 1u : 0u);
                if (h != 0u)
                    atomicAdd(&sm.bins.high[bin], h);
            }
        });
        cross_bins<BY_MASS>(sm, out.above, out.above_mass, target, parts);
        const int bin = sm.cross.bin;
        if (bin < 0)
            return false;
        out.above = sm.cross.count;
        out.above_mass = sm.cross.mass;
        out.ties = sm.cross.ties;
        cta_sync<W>(); // cross is written again
        const uint32_t top = hi - ((uint32_t)bin << shift);
        lo = top - min(top - lo, (1u << shift) - 1u);
        hi = top;
        if (shift == 0) { // one value: of 16 bits, those that are not there are ones below 0
            out.x = order_value(hi << DROP | ((hi << DROP) & 0x80000000u ? 0u : NOTHING));
            return true;
        }
        most = min(most, hi << DROP | NOTHING);
        least = max(least, lo << DROP);
    }
}

// One row, which the team has in shared memory, with every sum that decides exact,
// for any number of elements that are kept.
template <typename T, int W>
__device__ __noinline__ void exact_row(Shared<W> &sm, const Row<T, W> r, const SampleParams &p, int row, int part, int parts)
{
    constexpr int E = Vec<T>::E;
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = r.lane;
    float *const queue = sm.queue[r.warp];
    Settings a;
    a.read(p, row);
    const int k = a.limit(p.V);
    const bool by_p = a.p < 1.0f, zero = a.u < 0x1p-40f;
    int group;
    const float mine = max_of(r, group);
    float m = warp_top(mine);
    if (lane == 0)
        sm.top[r.warp] = m;
    cta_sync<W>();
#pragma unroll
    for (int w = 0; w < W; ++w)
        m = fmaxf(m, sm.top[w]);
    if (tid == 0) {
        sm.cta_top = m;
        sm.least = neg_inf();
    }
    team_sync<W>(parts);
    if (parts > 1)
        m = warp_top(lane < parts ? cl.map_shared_rank(&sm, lane)->cta_top : neg_inf());
    if (a.least > 0.0f && tid == 0)
        sm.least = least_kept(m, a.t, a.least);
    const Scale s = scale_of(m, a.t);
    // An exact weight w is the integer w 2^bits, in 2^62 the sum of all: a unit, by which each may be off in half, is
    // then below 2^-42 of the mean weight, whether a few elements have it all or all have as much.
    int equal;
    const u64 rest = team_sum<1>(sm, rest_of(r, s, mine, group, equal), parts);
    equal = (int)team_sum<2>(sm, (u64)equal, parts);
    const float whole = (float)rest * SUM_UNIT + (float)equal;
    const int bits = min(58, 61 - ((int)(__float_as_uint(whole * 1.001f) >> 23) - 127));
    const float floor0 = fmaxf(m - 1000.0f / s.c, LEAST);
    Cut cut{LEAST, 0x7fffffff}; // all
    bool all = true;
    u64 z = 0ull;
    Crossing at;
    if (k > 0) {
        // first among those above a bound that a few hundred reach, then among all
        float low = value_at(s, -24.0f);
        for (;;) {
            at.above = 0;
            at.above_mass = 0ull;
            if (descend<false>(sm, r, s, bits, (u64)k, fmaxf(low, LEAST), m, parts, at)) {
                cut = Cut{at.x, k - at.above};
                all = false;
                break;
            }
            if (!(low > LEAST))
                break;
            low = LEAST;
        }
        if (!all && by_p) {
            u64 sum = 0ull;
            each_between(r, queue, cut.x, -LEAST, [&](float x) { sum += x > cut.x ? weight(s, x, bits, sm.powers) : 0ull; });
            z = team_sum<0>(sm, sum, parts) + (u64)cut.ties * weight(s, cut.x, bits, sm.powers);
        }
    }
    if (by_p) {
        const u64 f = fraction(a.p);
        bool done = false;
        if (all) {
            // Of the fp32 weights the bin in which they reach p; what lies above it exactly, what lies below it
            // in fp32, whose error counts the less the more p keeps.
            const float low = fmaxf(value_at(s, log2f((1.0f - a.p) * whole / (float)p.V) - 0.01f), LEAST);
            const uint32_t hi = order_bits(m), lo = order_bits(low);
            const int shift = bin_shift(hi - lo);
            const float unit = __uint_as_float((uint32_t)(127 + 30 - (32 - __clz((int)whole + 1))) << 23); // all of them fit
            clear_bins(sm);
            for (int v = r.w0 + lane; v < r.w1; v += 32) {
                const uint4 raw = r.vec[v];
                if (!(Vec<T>::largest(raw) >= low))
                    continue;
                float x[E];
                Vec<T>::unpack(raw, x);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (x[e] >= low && x[e] <= m) // above it only after a copy's wait gave up
                        atomicAdd(&sm.bins.low[(hi - order_bits(x[e])) >> shift], (uint32_t)(exp2_fast((x[e] - m) * s.c) * unit + 0.5f));
            }
            cross_bins<true>(sm, 0, 0ull, (u64)(a.p * whole * unit), parts);
            const int bin = sm.cross.bin;
            cta_sync<W>();
            if (bin >= 0) {
                const uint32_t top = hi - ((uint32_t)bin << shift), bottom = top - min(top - lo, (1u << shift) - 1u);
                const float high = order_value(top), deep = order_value(bottom);
                u64 sum = 0ull, in = 0ull, tail = 0ull;
                each_between(r, queue, deep, -LEAST, [&](float x) {
                    const u64 w = weight(s, x, bits, sm.powers);
                    sum += x > high ? w : 0ull;
                    in += x > high ? 0ull : w;
                });
                for (int v = r.w0 + lane; v < r.w1; v += 32) {
                    float x[E], t[E];
                    Vec<T>::unpack(r.vec[v], x);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        t[e] = x[e] < deep ? exp2_fast((x[e] - m) * s.c) : 0.0f;
#pragma unroll
                    for (int w = 1; w < E; w *= 2)
#pragma unroll
                        for (int e = 0; e + w < E; e += 2 * w)
                            t[e] += t[e + w];
                    tail += as_fixed(t[0], SUM_SCALE);
                }
                sum = team_sum<3>(sm, sum, parts);
                in = team_sum<4>(sm, in, parts);
                tail = team_sum<5>(sm, tail, parts);
                const float margin = sum_margin((float)tail * SUM_UNIT, p.V, 5.0f);
                const u64 mg = (u64)(margin * SUM_UNITS) + 1ull;
                const u64 z_low = sum + in + ((tail > mg ? tail - mg : 0ull) << (bits - SUM_SCALE));
                const u64 z_high = sum + in + ((tail + mg) << (bits - SUM_SCALE));
                const u64 t_low = share_up(f, z_low), t_high = share_up(f, z_high);
                at.above = 0;
                at.above_mass = sum;
                if (t_low > sum && t_high <= sum + in && descend<true>(sm, r, s, bits, t_low, deep, high, parts, at)) {
                    const u64 w = weight(s, at.x, bits, sm.powers);
                    const u64 n = (t_low - at.above_mass + w - 1ull) / w, n_high = (t_high - at.above_mass + w - 1ull) / w;
                    if (n == n_high) {
                        cut = Cut{at.x, (int)n};
                        done = true;
                    }
                }
            }
            if (!done) { // the whole exactly
                u64 sum = 0ull;
                each_between(r, queue, LEAST, -LEAST, [&](float x) { sum += weight(s, x, bits, sm.powers); });
                cta_sync<W>();
                z = team_sum<0>(sm, sum, parts);
            }
        }
        if (!done) {
            const u64 target = max(1ull, share_up(f, z));
            float low = fmaxf(cut.x, all ? value_at(s, log2f((1.0f - a.p) * whole / (float)p.V) - 0.01f) : LEAST);
            for (;;) {
                at.above = 0;
                at.above_mass = 0ull;
                if (descend<true>(sm, r, s, bits, target, low, m, parts, at)) {
                    const u64 w = weight(s, at.x, bits, sm.powers), n = (target - at.above_mass + w - 1ull) / w; // enough to reach it
                    cut = Cut{at.x, (int)(n < (u64)at.ties ? n : (u64)at.ties)};
                    break;
                }
                if (!(low > cut.x))
                    break;
                low = cut.x;
            }
        }
    }
    cta_sync<W>(); // sm.least is there
    if (sm.least > cut.x)
        cut = Cut{sm.least, 0x7fffffff};
    const u64 tie_weight = weight(s, cut.x, bits, sm.powers);
    // what each warp has of them, those equal to the cut apart
    u64 own = 0ull;
    int ties = 0, above = 0;
    each_between(r, queue, cut.x, -LEAST, [&](float x) {
        if (x > cut.x) {
            own += weight(s, x, bits, sm.powers);
            ++above;
        } else {
            ties += x == cut.x;
        }
    });
    own = warp_sum64(own);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) {
        sm.warp_mass[r.warp] = own;
        sm.warp_ties[r.warp] = ties;
    }
    // and a barrier; not by place 2, which others may still read where nothing was cut by rank or sum since
    above = (int)team_sum<5>(sm, (u64)above, parts);
    u64 before = 0ull, total = 0ull;
    int ties_before = 0, ties_all = 0;
    for (int w = 0; w < W; ++w) {
        if (w < r.warp) {
            before += sm.warp_mass[w];
            ties_before += sm.warp_ties[w];
        }
        total += sm.warp_mass[w];
        ties_all += sm.warp_ties[w];
    }
    if (parts > 1) {
        if (tid == 0) {
            sm.cta_mass = total;
            sm.cta_ties = ties_all;
        }
        team_sync<W>(parts);
        const u64 om = lane < parts ? cl.map_shared_rank(&sm, lane)->cta_mass : 0ull;
        const int ot = lane < parts ? cl.map_shared_rank(&sm, lane)->cta_ties : 0;
        before += warp_sum64(lane < part ? om : 0ull);
        ties_before += __reduce_add_sync(0xffffffffu, lane < part ? ot : 0);
        total = warp_sum64(om);
        ties_all = __reduce_add_sync(0xffffffffu, ot);
    }
    const int tied = min(ties_all, cut.ties), here = min(ties, max(0, cut.ties - ties_before));
    total += (u64)tied * tie_weight;
    before += (u64)min(ties_before, cut.ties) * tie_weight;
    own += (u64)here * tie_weight;
    const u64 target = __umul64hi(fraction(a.u), total);
    const float logsum = log1pf((float)(total - (1ull << bits)) / (float)(1ull << bits));
    if (zero) {
        const int first = team_first(sm, first_from(r, fmaxf(cut.x, floor0)), parts);
        for (int v = r.w0 + lane; v < r.w1; v += 32)
            if (first >= max(r.first + v * E, 0) && first < r.first + v * E + E) {
                p.tokens[row] = first;
                if (p.logprob != nullptr)
                    p.logprob[row] = (element(r, v, first - r.first - v * E) - m) * a.t - logsum;
            }
    } else if (target >= before && target < before + own) {
        Drawn d;
        if (walk_exact(r, s, Cut{cut.x, here}, bits, tie_weight, sm.powers, target - before, d)) {
            p.tokens[row] = d.i;
            if (p.logprob != nullptr)
                p.logprob[row] = (d.x - m) * a.t - logsum;
        }
    }
    if (p.kept != nullptr && tid == 0 && part == 0)
        p.kept[row] = above + tied;
    team_sync<W>(parts); // shared memory is read until here, by others too
}

// fp32 weights good to their last bits but what 2^x itself is off by: the
// exponent's rounding errors go in to first order. With the sum over a vector,
// within FINE of themselves: 2^-22 and two roundings, and three of the sum.
constexpr float FINE = 10.0f * 0x1p-24f;
__device__ __forceinline__ f2 sub_f2(f2 a, f2 b) { return fma_f2(b, make_f2(-1.0f, -1.0f), a); }
template <int E> __device__ __forceinline__ void fine_weights(const Scale &s, const float (&x)[E], float (&w)[E])
{
    const f2 m = make_f2(s.m, s.m), c = make_f2(s.c, s.c), minus_c = make_f2(-s.c, -s.c), c_low = make_f2(s.c_low, s.c_low);
    const f2 ln2 = make_f2(LN2, LN2);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const f2 v = make_f2(x[e], x[e + 1]), d = sub_f2(v, m), t = sub_f2(d, v);
        const f2 d_low = sub_f2(sub_f2(v, sub_f2(d, t)), add_f2(m, t)); // x - m = d + d_low
        const f2 b = mul_f2(d, minus_c);                              // -a
        const f2 low = fma_f2(d_low, c, fma_f2(d, c_low, fma_f2(d, c, b)));
        float b0, b1, w0, w1;
        split_f2(b, b0, b1);
        const f2 g = make_f2(exp2_fast(-b0), exp2_fast(-b1));
        split_f2(fma_f2(mul_f2(g, ln2), low, g), w0, w1);
        w[e] = b0 < 126.0f ? w0 : 0.0f; // nothing of an infinite difference
        w[e + 1] = b1 < 126.0f ? w1 : 0.0f;
    }
}
template <int E> __device__ __forceinline__ float sum_of(const float (&x)[E])
{
    float t[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        t[e] = x[e];
#pragma unroll
    for (int w = 1; w < E; w *= 2)
#pragma unroll
        for (int e = 0; e + w < E; e += 2 * w)
            t[e] += t[e + w];
    return t[0];
}

// What lies above `high`, and below `deep` and above `floor`, of this thread's part in exact weights.
template <typename T, int W>
__device__ __noinline__ void exact_parts(const Row<T, W> r, const Scale s, float high, float deep, float floor, const u64 *powers, u64 &own,
                                         u64 &tail)
{
    constexpr int E = Vec<T>::E;
    u64 up = 0ull, down = 0ull;
#pragma unroll 1
    for (int v = r.w0 + r.lane; v < r.w1; v += 32) {
        float x[E];
        Vec<T>::unpack(r.vec[v], x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const u64 w = weight(s, x[e], SUM_SCALE, powers);
            up += x[e] > high ? w : 0ull;
            down += x[e] < deep && x[e] > floor ? w : 0ull;
        }
    }
    own = up;
    tail = down;
}

// One row, which the team has in shared memory, for any number of elements that are
// kept, by sums of fine weights: false where those leave it open. Where top-p ends is
// what they do most often, and exact sums of the two parts tell it.
template <typename T, int W>
__device__ __noinline__ bool fine_row(Shared<W> &sm, const Row<T, W> r, const SampleParams &p, int row, int part, int parts)
{
    constexpr int E = Vec<T>::E;
    cg::cluster_group cl = cg::this_cluster();
    Shared<W> *const lead = parts > 1 ? cl.map_shared_rank(&sm, 0) : &sm;
    const int tid = threadIdx.x, lane = r.lane;
    Settings a;
    a.read(p, row);
    if (a.u < 0x1p-40f)
        return false;
    const int k = a.limit(p.V);
    const bool by_p = a.p < 1.0f;
    int group;
    const float mine = max_of(r, group);
    float m = warp_top(mine);
    if (lane == 0)
        sm.top[r.warp] = m;
    cta_sync<W>();
#pragma unroll
    for (int w = 0; w < W; ++w)
        m = fmaxf(m, sm.top[w]);
    if (tid == 0) {
        sm.cta_top = m;
        sm.least = neg_inf();
        sm.listed = 0;
    }
    team_sync<W>(parts);
    if (parts > 1)
        m = warp_top(lane < parts ? cl.map_shared_rank(&sm, lane)->cta_top : neg_inf());
    if (a.least > 0.0f && tid == 0)
        sm.least = least_kept(m, a.t, a.least);
    const Scale s = scale_of(m, a.t);
    Cut cut{LEAST, 0x7fffffff}; // all
    bool all = true;            // a cut by rank may lie at the lowest value too
    float tie_weight = 0.0f;
    if (k > 0) { // exactly, by counting; first among those above a bound that most rows' first thousands reach
        Crossing at;
        float low = value_at(s, -24.0f);
        for (;;) {
            at.above = 0;
            at.above_mass = 0ull;
            if (descend<false>(sm, r, s, SUM_SCALE, (u64)k, fmaxf(low, LEAST), m, parts, at)) {
                cut = Cut{at.x, k - at.above};
                all = false;
                break;
            }
            if (!(low > LEAST))
                break;
            low = LEAST;
        }
        tie_weight = (float)weight(s, cut.x, SUM_SCALE, sm.powers) * SUM_UNIT;
    }
    u64 own = 0ull, exact = 0ull; // this thread's part of what is kept, and what of it was listed
    int above = 0, ties = 0;
    bool sure = true, summed = false;
    if (by_p) {
        // ---- roughly: the weight of the whole, and in which of BINS steps of the exponent p of it is reached
        float rough = 0.0f;
        for (int v = r.w0 + lane; v < r.w1; v += 32) {
            float x[E];
            Vec<T>::unpack(r.vec[v], x);
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[e] = x[e] > cut.x || all ? exp2_fast((x[e] - m) * s.c) : 0.0f;
            rough += sum_of(x);
        }
        const float whole = (float)team_sum<0>(sm, as_fixed(rough, SUM_SCALE), parts) * SUM_UNIT + (all ? 0.0f : (float)cut.ties * tie_weight);
        float a_low = all ? log2f((1.0f - a.p) * whole / (float)p.V) - 0.02f : (cut.x - m) * s.c - 0.01f, a_high = 0.0f;
        float taken = 0.0f; // the weight above a_high
        // a weight takes 22 bits and all of them 31 (equal elements are rounded alike: what 22 bits for all leave of
        // each put 3 % of rows' ends of 8192 x 32000 bf16 into a neighbour's bin)
        const float unit = __uint_as_float((uint32_t)(127 + min(22, 31 - (32 - __clz((int)whole + 1)))) << 23);
        float high = m, deep = LEAST;
        int n = LIST + 1;
        u64 tail = 0ull;
        for (int round = 0; round < 3 && n > LIST && sure; ++round) {
            const float steps = (float)BINS / (a_high - a_low), x_low = value_at(s, a_low);
            clear_bins(sm);
            for (int v = r.w0 + lane; v < r.w1; v += 32) {
                const uint4 raw = r.vec[v];
                if (!(Vec<T>::largest(raw) >= x_low))
                    continue;
                float x[E];
                Vec<T>::unpack(raw, x);
                // numbers become integers by adding 2^23, whose bits end in them; those beyond the bins come out large
                const f2 nm = make_f2(-m, -m), c2 = make_f2(s.c, s.c), down = make_f2(-steps, -steps), from = make_f2(a_high * steps + 0x1p23f, a_high * steps + 0x1p23f);
                const f2 unit2 = make_f2(unit, unit), magic = make_f2(0x1p23f, 0x1p23f);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const f2 z = mul_f2(add_f2(make_f2(x[e], x[e + 1]), nm), c2);
                    float z0, z1, b0, b1, q0, q1;
                    split_f2(z, z0, z1);
                    split_f2(fma_f2(z, down, from), b0, b1);
                    split_f2(fma_f2(make_f2(exp2_fast(z0), exp2_fast(z1)), unit2, magic), q0, q1);
                    const uint32_t bin0 = __float_as_uint(b0) - 0x4B000000u, bin1 = __float_as_uint(b1) - 0x4B000000u;
                    if (bin0 < (uint32_t)BINS)
                        atomicAdd(&sm.bins.low[bin0], __float_as_uint(q0) - 0x4B000000u);
                    if (bin1 < (uint32_t)BINS)
                        atomicAdd(&sm.bins.low[bin1], __float_as_uint(q1) - 0x4B000000u);
                }
            }
            cross_bins<true>(sm, 0, 0ull, (u64)fmaxf((a.p * whole - taken) * unit, 1.0f), parts);
            const int bin = sm.cross.bin;
            cta_sync<W>();
            if (bin < 0) {
                sure = false;
                break;
            }
            const float top = a_high;
            // bins are about whole numbers of steps; the narrow ones of a bin that held too many are less than the sums so
            // far are off by
            const float beside = round == 0 ? 0.5f : 12.5f;
            a_high = fminf(0.0f, top - ((float)bin - beside) / steps);
            a_low = top - ((float)bin + beside) / steps;
            high = a_high >= 0.0f ? m : m + a_high / s.c;
            deep = m + a_low / s.c;
            if (!all && deep <= cut.x) {
                sure = false;
                break;
            }
            // ---- finely: what lies above that step, what lies below it; the elements in it are listed
            own = tail = 0ull;
            above = 0;
            for (int v = r.w0 + lane; v < r.w1; v += 32) {
                float x[E], w[E], t[E];
                Vec<T>::unpack(r.vec[v], x);
                fine_weights(s, x, w);
                uint32_t in = 0u;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const bool up = x[e] > high, down = x[e] < deep;
                    above += up;
                    in |= !up && !down ? 1u << e : 0u;
                    t[e] = down && (all || x[e] > cut.x) ? w[e] : 0.0f;
                    w[e] = up ? w[e] : 0.0f;
                }
                own += as_fixed(sum_of(w), SUM_SCALE);
                tail += as_fixed(sum_of(t), SUM_SCALE);
                if (in != 0u) {
                    int to = atomicAdd(&lead->listed, __popc(in));
                    for (; in != 0u; in &= in - 1u, ++to)
                        if (to < LIST) {
                            const int e = __ffs(in) - 1;
                            lead->list[to].x = element(r, v, e);
                            lead->list[to].i = r.first + v * E + e;
                        }
                }
            }
            team_sync<W>(parts);
            n = lead->listed;
            team_sync<W>(parts);
            if (n > LIST) {
                taken = (float)team_sum<5>(sm, own, parts) * SUM_UNIT;
                if (tid == 0)
                    sm.listed = 0; // bins take the list's place again
            }
        }
        sure = sure && n <= LIST;
        if (sure) {
            Entry *const list = parts > 1 ? sm.few : sm.list; // at hand
            if (parts > 1)
                for (int j = tid; j < n; j += W * 32)
                    sm.few[j] = lead->list[j];
            cta_sync<W>();
            for (int j = tid; j < n; j += W * 32)
                list[j].w = weight(s, list[j].x, SUM_SCALE, sm.powers);
            cta_sync<W>();
            u64 listed = 0ull;
            for (int j = 0; j < n; ++j)
                listed += list[j].w;
            for (float off = FINE;; off = 0x1p-40f) {
                const u64 high_sum = team_sum<1>(sm, own, parts), tail_sum = team_sum<2>(sm, tail, parts) +
                                                                              (all ? 0ull : (u64)cut.ties * weight(s, cut.x, SUM_SCALE, sm.powers));
                // An entry is kept where what is listed before it is less than p (high + listed + tail) - high, whose
                // error is that of (1 - p) high and p tail.
                const float q = 1.0f - a.p, hf = (float)high_sum * SUM_UNIT, tf = (float)tail_sum * SUM_UNIT;
                const long long slack = (long long)((off * (q * hf + a.p * tf) + (float)p.V * SUM_UNIT) * SUM_UNITS) + 2;
                const u64 share = share_up(fraction(a.p), high_sum + listed + tail_sum);
                const long long target = (long long)(share - high_sum);
                bool doubt = target <= slack || target + slack > (long long)listed;
                if (tid == 0)
                    sm.cross.bin = 0; // doubts
                cta_sync<W>();
                for (int j = tid; j < n; j += W * 32) {
                    const Entry e = list[j];
                    u64 before = 0ull;
                    int equals = 0;
                    for (int o = 0; o < n; ++o) {
                        const Entry f = list[o];
                        const bool tie = f.x == e.x && f.i < e.i;
                        before += f.x > e.x || tie ? f.w : 0ull;
                        equals += tie;
                    }
                    const long long gap = target - (long long)before;
                    doubt |= gap <= slack && gap > -slack;
                    if (gap > 0 && gap <= (long long)e.w) { // the last one
                        sm.cross.ties = equals + 1;
                        sm.scan_mass[0] = (u64)order_bits(e.x);
                    }
                }
                if (doubt)
                    atomicOr(&sm.cross.bin, 1);
                cta_sync<W>();
                sure = sm.cross.bin == 0; // the same in every CTA
                if (sure || off != FINE)
                    break;
                exact_parts(r, s, high, deep, all ? neg_inf() : cut.x, sm.powers, own, tail);
                exact = own;
            }
            cut = Cut{order_value((uint32_t)sm.scan_mass[0]), sm.cross.ties};
            tie_weight = (float)weight(s, cut.x, SUM_SCALE, sm.powers) * SUM_UNIT;
            // the kept entries are the threads' that hold them: by warps' runs
            if (sure && !(sm.least > cut.x)) {
                summed = true;
                for (int j = lane; j < n; j += 32) {
                    const Entry e = list[j];
                    if (e.i >= max(r.first + r.w0 * E, 0) && e.i < r.first + r.w1 * E) {
                        const u64 w = e.x > cut.x ? e.w : 0ull;
                        own += w;
                        exact += w;
                        above += e.x > cut.x;
                        ties += e.x == cut.x;
                    }
                }
                exact = warp_sum64(exact);
            }
        }
        team_sync<W>(parts); // the list and the crossing have been read
        if (tid == 0)
            sm.listed = 0;
    }
    cta_sync<W>(); // sm.least is there
    if (sm.least > cut.x)
        cut = Cut{sm.least, 0x7fffffff};
    const u64 tie_units = weight(s, cut.x, SUM_SCALE, sm.powers);
    if (!summed) {
        own = 0ull;
        above = ties = 0;
    }
    if (sure && !summed)
        for (int v = r.w0 + lane; v < r.w1; v += 32) {
            float x[E], w[E];
            if (!(Vec<T>::largest(r.vec[v]) >= cut.x))
                continue;
            Vec<T>::unpack(r.vec[v], x);
            fine_weights(s, x, w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                above += x[e] > cut.x;
                ties += x[e] == cut.x;
                w[e] = x[e] > cut.x ? w[e] : 0.0f;
            }
            own += as_fixed(sum_of(w), SUM_SCALE);
        }
    own = warp_sum64(own);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) {
        sm.warp_mass[r.warp] = own;
        sm.warp_ties[r.warp] = ties;
    }
    above = (int)team_sum<3>(sm, (u64)above, parts); // and a barrier
    u64 before = 0ull, total = 0ull;
    int ties_before = 0, ties_all = 0;
    for (int w = 0; w < W; ++w) {
        if (w < r.warp) {
            before += sm.warp_mass[w];
            ties_before += sm.warp_ties[w];
        }
        total += sm.warp_mass[w];
        ties_all += sm.warp_ties[w];
    }
    if (parts > 1) {
        if (tid == 0) {
            sm.cta_mass = total;
            sm.cta_ties = ties_all;
        }
        team_sync<W>(parts);
        const u64 om = lane < parts ? cl.map_shared_rank(&sm, lane)->cta_mass : 0ull;
        const int ot = lane < parts ? cl.map_shared_rank(&sm, lane)->cta_ties : 0;
        before += warp_sum64(lane < part ? om : 0ull);
        ties_before += __reduce_add_sync(0xffffffffu, lane < part ? ot : 0);
        total = warp_sum64(om);
        ties_all = __reduce_add_sync(0xffffffffu, ot);
    }
    const int tied = min(ties_all, cut.ties), here = min(ties, max(0, cut.ties - ties_before));
    total += (u64)tied * tie_units;
    before += (u64)min(ties_before, cut.ties) * tie_units;
    own += (u64)here * tie_units;
    const u64 target = __umul64hi(fraction(a.u), total);
    // the warp that looks into its own adds other parts of vectors up (three roundings each way, three of the last vector's
    // elements), and has what was listed by fine weights
    const u64 slack = draw_slack(a.u, total, total, FINE * ((float)total * SUM_UNIT),
                                 (9.0f * 0x1p-24f * (float)own + FINE * (float)exact) * SUM_UNIT, p.V);
    bool drawn = false;
    if (sure && target >= before && target < before + own) {
        // ---- in the warp that the target lies in
        u64 want = target - before, run = 0ull;
        int left = here; // equal ones that are kept
        for (int g0 = r.w0; g0 < r.w1; g0 += 128) {
            // ---- which 32 of 128 vectors
            u64 part_of[4];
            int equal_of[4], v0 = -1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int v = g0 + 32 * j + lane;
                float x[E], w[E];
                Vec<T>::unpack(v < r.w1 ? r.vec[v] : empty_vec<T>(), x);
                fine_weights(s, x, w);
                equal_of[j] = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    equal_of[j] += x[e] == cut.x;
                    w[e] = x[e] > cut.x ? w[e] : 0.0f;
                }
                part_of[j] = as_fixed(sum_of(w), SUM_SCALE);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                part_of[j] = warp_sum64(part_of[j]);
                equal_of[j] = __reduce_add_sync(0xffffffffu, equal_of[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int kept = min(left, equal_of[j]);
                const u64 whole = part_of[j] + (u64)kept * tie_units;
                if (v0 < 0 && want >= run + whole) {
                    run += whole;
                    left -= kept;
                } else if (v0 < 0) {
                    v0 = g0 + 32 * j;
                }
            }
            if (v0 < 0)
                continue;
            // ---- which of them, and which element
            const int v = v0 + lane;
            float x[E], w[E];
            Vec<T>::unpack(v < r.w1 ? r.vec[v] : empty_vec<T>(), x);
            fine_weights(s, x, w);
            int equal = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                equal += x[e] == cut.x;
                w[e] = x[e] > cut.x ? w[e] : 0.0f;
            }
            int upto_equal = equal;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int n = __shfl_up_sync(0xffffffffu, upto_equal, o);
                upto_equal += lane >= o ? n : 0;
            }
            int allowed = min(max(left - (upto_equal - equal), 0), equal);
            const u64 mass = as_fixed(sum_of(w), SUM_SCALE) + (u64)allowed * tie_units;
            u64 upto = mass;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 n = __shfl_up_sync(0xffffffffu, upto, o);
                upto += lane >= o ? n : 0ull;
            }
            u64 at = run + upto - mass;
            if (want >= at && want < at + mass) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    u64 one = as_fixed(w[e], SUM_SCALE);
                    if (x[e] == cut.x && allowed > 0) {
                        one = tie_units;
                        --allowed;
                    }
                    if (!drawn && want >= at + slack && want + slack < at + one) {
                        drawn = true;
                        p.tokens[row] = r.first + v * E + e;
                        if (p.logprob != nullptr)
                            p.logprob[row] = (x[e] - m) * a.t - log1pf((float)(total - (1ull << SUM_SCALE)) * SUM_UNIT);
                    }
                    at += one;
                }
            }
            break;
        }
    }
    const bool done = team_sum<4>(sm, drawn ? 1ull : 0ull, parts) != 0ull;
    if (done && p.kept != nullptr && tid == 0 && part == 0)
        p.kept[row] = above + tied;
    team_sync<W>(parts); // shared memory is read until here, by others too
    return done;
}

// Where it is needed once a row: code that has to be fetched costs more than the call.
__device__ __noinline__ u64 weight_once(const Scale s, float x, int bits, const u64 *powers) { return weight(s, x, bits, powers); }

// min_p in the unit 2^-scale of listed weights, upwards; and whether a weight w in that unit is so near it that
// its rounding may decide: half a unit and 2^-43 of w it is off by, up to a unit is `least`. Such a row is left open,
// for the ways that compare values instead.
__device__ __forceinline__ u64 min_p_units(float min_p, int scale)
{
    const float mp = min_p * __uint_as_float((uint32_t)(127 + scale) << 23);
    return (u64)mp + ((float)(u64)mp < mp ? 1ull : 0ull);
}
__device__ __forceinline__ bool at_border(u64 w, u64 least)
{
    const u64 off = 2ull + (w >> 40);
    return w + off >= least && w <= least + off;
}

// A bound for what is kept, from the threads' own maxima: at least `need` of them
// (or of their weight, in 2^-20) lie above it. -infinity where they do not suffice.
__device__ __forceinline__ float guide_bound(uint32_t first_bin, uint32_t second_bin, uint32_t need, float m, float lowest, float per_bin, int lane)
{
    const uint32_t own = first_bin + second_bin;
    uint32_t upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t n = __shfl_up_sync(0xffffffffu, upto, o);
        upto += lane >= o ? n : 0u;
    }
    const uint32_t reach = __ballot_sync(0xffffffffu, upto >= need);
    if (reach == 0u)
        return neg_inf();
    const int l = __ffs(reach) - 1;
    const bool early = __shfl_sync(0xffffffffu, upto - own + first_bin, l) >= need;
    const int bin = 2 * l + (early ? 0 : 1);
    if (bin == GUIDE - 1)
        return lowest;
    const float d = (float)(bin + 1) * per_bin;
    return fmaxf(lowest, (m - d) - (fabsf(m) + d) * 0x1p-21f); // below the bin for all roundings
}

// The running sum over 32 PER numbers, lane by lane and then register by register.
template <int PER> __device__ __forceinline__ void running(const u64 (&v)[PER], u64 (&before)[PER], u64 &all, int lane)
{
    all = 0ull;
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        u64 upto = v[r];
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const u64 n = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? n : 0ull;
        }
        before[r] = all + upto - v[r];
        all += __shfl_sync(0xffffffffu, upto, 31);
    }
}
// 32 PER keys in descending order (32-bit ones in ascending order): number r 32 + lane
// is register r's. Rolled up: a warp goes through this once a row, and what it
// waits for is the code, not its latency.
template <int PER, typename K> __device__ __forceinline__ void sort_keys(K (&k)[PER], int lane)
{
    constexpr bool DOWN = sizeof(K) == 8;
#pragma unroll 1
    for (int size = 2; size <= 32 * PER; size <<= 1) {
        if (PER > 2 && size == 128) { // registers 64 apart
#pragma unroll
            for (int r = 0; r < PER / 2; ++r) {
                const K a = k[r], b = k[(r + PER / 2) % PER];
                const bool swap = DOWN == (b > a);
                k[r] = swap ? b : a;
                k[(r + PER / 2) % PER] = swap ? a : b;
            }
        }
        if (PER > 1 && size >= 64) { // registers 32 apart
#pragma unroll
            for (int r = 0; r + 1 < PER; r += 2) {
                const K a = k[r], b = k[r + 1];
                const bool swap = (DOWN == (((r * 32) & size) == 0)) == (b > a);
                k[r] = swap ? b : a;
                k[r + 1] = swap ? a : b;
            }
        }
#pragma unroll 1
        for (int j = min(size >> 1, 16); j > 0; j >>= 1) {
#pragma unroll
            for (int r = 0; r < PER; ++r) {
                const K o = __shfl_xor_sync(0xffffffffu, k[r], j);
                const bool up = ((r * 32 + lane) & size) == 0, lower = (lane & j) == 0;
                const bool want_big = DOWN == (up == lower);
                k[r] = want_big == (o > k[r]) ? o : k[r];
            }
        }
    }
}

// The listed elements: top-k, top-p of what it left, min-p, and the draw, by one warp.
// False where the sums leave it open.
template <int PER>
__device__ __noinline__ bool finish_warp(const u64 *powers, Entry *list, const SampleParams &p, const ListTask &q)
{
    const int lane = threadIdx.x & 31, n = q.n;
    const float u = q.a.u, min_p = q.a.least;
    const Scale s = q.s;
    const bool ordered = q.k > 0 || q.by_p; // else min-p alone, which the best passes (it is at most 1)
    const int scale = min(LIST_SCALE, 62 - (32 - __clz((int)((q.rest >> SUM_SCALE) + (u64)q.equal + 1ull))));
    u64 key[PER], w[PER], before[PER], all;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int at = r * 32 + lane;
        key[r] = at < n ? (u64)order_bits(list[at].x) << 32 | (0xFFFFFFFFu - (uint32_t)list[at].i) : 0ull;
    }
    if (ordered)
        sort_keys<PER>(key, lane);
#pragma unroll
    for (int r = 0; r < PER; ++r)
        w[r] = r * 32 + lane < n ? weight_once(s, order_value((uint32_t)(key[r] >> 32)), scale, powers) : 0ull;
    running<PER>(w, before, all, lane);
    bool keep[PER], open = min_p > 0.0f && min_p < 0x1p-40f; // beneath the weights' unit
#pragma unroll
    for (int r = 0; r < PER; ++r)
        keep[r] = r * 32 + lane < n && (q.k == 0 || r * 32 + lane < q.k);
    if (q.by_p) {
        u64 z_low, z_high;
        if (q.k == 0) {
            const u64 z = q.rest + ((u64)q.equal << SUM_SCALE), mg = (u64)(q.margin * SUM_UNITS) + 1ull;
            z_low = (z - mg) << (scale - SUM_SCALE);
            z_high = (z + mg) << (scale - SUM_SCALE);
        } else { // of the first k
            u64 sum = 0ull;
#pragma unroll
            for (int r = 0; r < PER; ++r)
                sum += keep[r] ? w[r] : 0ull;
            z_low = z_high = warp_sum64(sum);
        }
        const u64 f = fraction(q.a.p), t_low = share_up(f, z_low), t_high = share_up(f, z_high);
        open |= q.k == 0 && all < t_high && !q.least_bound;
#pragma unroll
        for (int r = 0; r < PER; ++r) {
            const bool first = r * 32 + lane == 0, in = before[r] < t_low || first;
            open |= keep[r] && in != (before[r] < t_high || first);
            keep[r] = keep[r] && in;
        }
    }
    if (min_p > 0.0f) { // w >= min_p
        const u64 least = min_p_units(min_p, scale);
#pragma unroll
        for (int r = 0; r < PER; ++r) {
            const bool best = order_value((uint32_t)(key[r] >> 32)) == s.m; // its w = 1 is exact
            open |= keep[r] && !best && at_border(w[r], least);
            keep[r] = keep[r] && (w[r] >= least || (ordered && r * 32 + lane == 0));
        }
    }
    const bool zero = u < 0x1p-40f;
    const float floor0 = fmaxf(s.m - 1000.0f / s.c, LEAST);
    int kept = 0;
    uint32_t by_index[PER]; // kept elements' index and place; below 2^19 and 2^7
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int at = r * 32 + lane;
        const float x = order_value((uint32_t)(key[r] >> 32));
        kept += keep[r];
        by_index[r] = keep[r] && !(zero && x < floor0) ? (0xFFFFFFFFu - (uint32_t)key[r]) << 7 | at : 0xFFFFFFFFu;
    }
    if (__any_sync(0xffffffffu, open))
        return false;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        Entry e;
        e.x = order_value((uint32_t)(key[r] >> 32));
        e.i = (int)(0xFFFFFFFFu - (uint32_t)key[r]);
        e.w = w[r];
        list[r * 32 + lane] = e;
    }
    __syncwarp();
    kept = __reduce_add_sync(0xffffffffu, kept);
    sort_keys<PER>(by_index, lane);
#pragma unroll
    for (int r = 0; r < PER; ++r)
        w[r] = by_index[r] != 0xFFFFFFFFu ? list[by_index[r] & 127u].w : 0ull;
    u64 total;
    running<PER>(w, before, total, lane);
    if (zero) { // what had no weight left was not among them
        u64 sum = 0ull;
#pragma unroll
        for (int r = 0; r < PER; ++r)
            sum += keep[r] ? list[r * 32 + lane].w : 0ull;
        total = warp_sum64(sum);
    }
    const u64 target = __umul64hi(fraction(u), total);
#pragma unroll
    for (int r = 0; r < PER; ++r)
        if (zero ? r == 0 && lane == 0 : target >= before[r] && target - before[r] < w[r]) {
            const Entry e = list[by_index[r] & 127u];
            p.tokens[q.row] = e.i;
            if (p.logprob != nullptr)
                p.logprob[q.row] = (e.x - s.m) * q.a.t - log1pf((float)(total - (1ull << scale)) / (float)(1ull << scale));
        }
    if (lane == 0 && p.kept != nullptr)
        p.kept[q.row] = kept;
    __syncwarp();
    return true;
}
static_assert(LIST <= 128 && LORA_MAX_VOCAB < 1 << 19, "an index and a place in 26 bits");
__device__ __forceinline__ bool finish_any(const u64 *powers, Entry *list, const SampleParams &p, const ListTask &q)
{
    return q.n <= 32   ? finish_warp<1>(powers, list, p, q)
           : q.n <= 64 ? finish_warp<2>(powers, list, p, q)
                       : finish_warp<LIST / 32>(powers, list, p, q);
}

// The listed elements: top-k, top-p of what it left, min-p, and the draw, by the CTA's W
// warps. An element is that of up to eight threads side by side, which count what
// precedes it together. False where the sums leave it open. Clusters' lists are worked out so: their rows are
// few, and what counts is how long one takes. One row of 32000 bf16 with every setting 12.5 us, 13.5 with the
// sort in one warp; 8 rows 14.2 and 16.3, 64 rows 18.7 and 19.9. Where one more warp
// works out the lists of many rows beside the others, the sort takes less of the SM.
template <int W> __device__ __noinline__ bool finish_list(Shared<W> &sm, Entry *list, const SampleParams &p, const ListTask &q)
{
    constexpr int THREADS = W * 32;
    const int tid = threadIdx.x % THREADS, n = q.n, row = q.row;
    const Settings a = q.a;
    const Scale s = q.s;
    int ways = 1;
    while (ways < 8 && 2 * ways * n <= THREADS)
        ways *= 2;
    const int id = tid / ways, sub = tid & (ways - 1);
    auto sync = [&] { named_bar_sync(BAR_LIST, THREADS); };
    auto sum_of = [&](u64 v, int at) {
        v = warp_sum64(v);
        if ((tid & 31) == 0)
            sm.sums[at][tid >> 5] = v;
        sync();
        v = 0ull;
#pragma unroll
        for (int w = 0; w < W; ++w)
            v += sm.sums[at][w];
        return v;
    };
    const int scale = min(LIST_SCALE, 62 - (32 - __clz((int)((q.rest >> SUM_SCALE) + (u64)q.equal + 1ull))));
    float x = neg_inf();
    int i = 0x7fffffff, ahead = 0;
    u64 w = 0ull, before = 0ull;
    if (id < n) {
        x = list[id].x;
        i = list[id].i;
        w = weight_once(s, x, scale, sm.powers);
        if (sub == 0)
            list[id].w = w;
    }
    sync();
    const bool ordered = q.k > 0 || q.by_p; // else min-p alone, which the best passes (it is at most 1)
    const bool busy = (tid & ~31) < n * ways;
    if (busy && ordered) {
#pragma unroll 4
        for (int j = sub; j < n; j += ways) { // their places in the order
            const Entry e = list[j];
            const bool is = e.x > x || (e.x == x && e.i < i);
            ahead += is;
            before += is ? e.w : 0ull;
        }
        for (int o = 1; o < ways; o *= 2) {
            ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
            before += __shfl_xor_sync(0xffffffffu, before, o);
        }
    }
    bool keep = id < n && sub == 0 && (q.k == 0 || ahead < q.k);
    bool open = a.least > 0.0f && a.least < 0x1p-40f; // beneath the weights' unit
    if (q.by_p) {
        const u64 listed = sum_of(keep ? w : 0ull, 0), f = fraction(a.p);
        u64 z_low = listed, z_high = listed;
        if (q.k == 0) {
            const u64 z = q.rest + ((u64)q.equal << SUM_SCALE), mg = (u64)(q.margin * SUM_UNITS) + 1ull;
            z_low = (z - mg) << (scale - SUM_SCALE);
            z_high = (z + mg) << (scale - SUM_SCALE);
        }
        const u64 t_low = share_up(f, z_low), t_high = share_up(f, z_high);
        const bool in = before < t_low || ahead == 0;
        open |= q.k == 0 && listed < t_high && !q.least_bound;
        open |= keep && in != (before < t_high || ahead == 0);
        keep = keep && in;
    }
    if (a.least > 0.0f) { // w >= min_p
        const u64 least = min_p_units(a.least, scale);
        open |= keep && x != s.m && at_border(w, least); // w = 1 of the best and its equals is exact
        keep = keep && (w >= least || (ordered && ahead == 0));
    }
    // the count, and in the upper half whether any is open
    int kept = __reduce_add_sync(0xffffffffu, (int)keep);
    kept |= __any_sync(0xffffffffu, open) ? 1 << 20 : 0;
    if ((tid & 31) == 0)
        sm.firsts[tid >> 5] = kept;
    const u64 total = sum_of(keep ? w : 0ull, 1); // and all are through with the list's weights
    kept = 0;
#pragma unroll
    for (int v = 0; v < W; ++v)
        kept += sm.firsts[v];
    if (kept >> 20 != 0)
        return false;
    const u64 target = __umul64hi(fraction(a.u), total);
    const bool zero = a.u < 0x1p-40f;
    int first = 0x7fffffff;
    if (zero) { // the first with a weight above e^-693
        const float floor0 = fmaxf(s.m - 1000.0f / s.c, LEAST);
        first = __reduce_min_sync(0xffffffffu, keep && x >= floor0 ? i : 0x7fffffff);
        sync();
        if ((tid & 31) == 0)
            sm.firsts[tid >> 5] = first;
        sync();
#pragma unroll
        for (int v = 0; v < W; ++v)
            first = min(first, sm.firsts[v]);
    } else { // the first, in index order, past u of their sum
        before = 0ull;
        if (id < n && sub == 0)
            list[id].w = keep ? w : 0ull;
        sync();
        if (busy) {
#pragma unroll 4
            for (int j = sub; j < n; j += ways) {
                const Entry e = list[j];
                before += e.i < i ? e.w : 0ull;
            }
            for (int o = 1; o < ways; o *= 2)
                before += __shfl_xor_sync(0xffffffffu, before, o);
        }
    }
    if (keep && (zero ? i == first : target >= before && target - before < w)) {
        p.tokens[row] = i;
        if (p.logprob != nullptr)
            p.logprob[row] = (x - s.m) * a.t - log1pf((float)(total - (1ull << scale)) / (float)(1ull << scale));
    }
    if (tid == 0 && p.kept != nullptr)
        p.kept[row] = kept;
    return true;
}

} // namespace

// TEAM: rows spread over clusters, a leading CTA of which works the lists out with
// all its warps. Else one more warp does, while the others are at the next row, and
// a row that it leaves open is gone through again when that is known. Latency bounds
// it: one row of 32000 takes 12 us (top 50, top-p and min-p, a cluster of eight), of which
// its copy takes 3; 590 x 32000 bf16 of top 50 32 us. 64 rows of 32003 f32 with settings of
// every kind take 18 to 39 us, as rows that the list leaves open, or their exact sums, come
// up or not. The registers that the CTAs an SM may have do not hold it all: 250 to 450 bytes a
// thread are stored to local memory and 340 to 940 loaded (-Xptxas -v), most with four warps.
template <typename T, int W, bool TEAM>
__global__ void __launch_bounds__(W * 32 + (TEAM ? 0 : 32), W == 8 ? 3 : 8) sample_kernel(SampleParams p, int parts_)
{
    constexpr int E = Vec<T>::E;
    extern __shared__ uint4 slice[];
    __shared__ Shared<W> sm;
    begin_behind();
    cg::cluster_group cl = cg::this_cluster();
    const int parts = TEAM ? parts_ : 1;
    const int tid = threadIdx.x, lane = tid & 31;
    const int part = TEAM ? (int)blockIdx.x % parts : 0, teams = TEAM ? (int)gridDim.x / parts : (int)gridDim.x;
    const T *logits = static_cast<const T *>(p.logits);
    if (tid == 0) {
        sm.listed = sm.alive[0] = sm.alive[1] = sm.left_open = sm.redone[0] = sm.redone[1] = sm.out_of_range = sm.late = 0;
        sm.open[0] = sm.open[1] = -1;
        sm.first[0] = sm.first[1] = 0x7fffffff;
    }
    if (tid < 32)
        sm.powers[tid] = POWERS[tid];
    for (int i = tid; i < GUIDE; i += W * 32)
        sm.guide[0][i] = 0u;
    if (!TEAM && tid >= W * 32) {
        __syncthreads();
        for (;;) {
            named_bar_sync(BAR_GIVEN, 64);
            if (sm.task.row < 0)
                break;
            static_assert(sizeof(ListTask) % 4 == 0 && sizeof(ListTask) <= 128, "a word a lane");
            if (lane < (int)sizeof(ListTask) / 4)
                reinterpret_cast<uint32_t *>(&sm.taken)[lane] = reinterpret_cast<const uint32_t *>(&sm.task)[lane];
#pragma unroll
            for (int i = 0; i < LIST; i += 32)
                sm.few[i + lane] = sm.list[i + lane];
            __syncwarp();
            const ListTask &q = sm.taken;
            named_bar_arrive(BAR_TAKEN, W * 32 + 32);
            const bool ok = finish_any(sm.powers, sm.few, p, q);
            if (!ok && lane == 0) {
                sm.redo[sm.left_open % REDO] = q.row;
                __threadfence_block();
                *reinterpret_cast<volatile int *>(&sm.left_open) += 1;
            }
            __syncwarp();
        }
        named_bar_arrive(BAR_TAKEN, W * 32 + 32);
        return;
    }
    Row<T, W> r;
    r.open(slice, sm.bars);
    int row = TEAM ? (int)blockIdx.x / parts : (int)blockIdx.x; // the first two are given; what follows is claimed two rows ahead
    int next = row + teams;
    r.load(logits + (int64_t)row * p.stride, p.V, part, parts);
    if (tid < 5)
        Settings::fetch(p, row, tid, sm.settings[0]);
    if (tid == 0)
        CallCounts().open<2>(p.status);
    Shared<W> *const told = TEAM && lane < parts ? cl.map_shared_rank(&sm, lane) : &sm; // a lane for each CTA of the team
    Shared<W> *const lead = TEAM ? cl.map_shared_rank(&sm, 0) : &sm;                    // keeps the team's list
    const int place = part * W + r.warp, slots = parts * W;
    if (TEAM)
        team_sync<W>(parts);
    else
        __syncthreads();
    int last = -1, redone = 0, turn = 0;
    bool given = false;   // the ninth warp has a list that it may not have taken yet
    bool resumed = false; // the row was begun before
    enum { END, HERE, BACK };
    for (;;) {
        int slow;
        for (;; ++turn) {
            const int h = turn & 1;
            const bool have = row < p.M;
            int group = 0;
            float mine = neg_inf();
            if (have) {
                uint32_t claimed = 0u;
                if (tid == 0 && part == 0 && !resumed)
                    claimed = CallCounts::of(p.status).next_row();
                if (tid < 5)
                    cp_async_wait_all(); // the row's settings
                r.wait();
                if (next < p.M)
                    r.prefetch(logits + (int64_t)next * p.stride, p.V);

                // ---- the row's maximum; the lowest of the threads' own
                mine = max_of(r, group);
                const float top = warp_top(mine);
                const uint32_t low = __reduce_min_sync(0xffffffffu, mine > neg_inf() ? order_bits(mine) : 0xffffffffu);
                const int after = __shfl_sync(0xffffffffu, (int)claimed + 2 * teams, 0);
                if (lane < parts) {
                    told->maxima[h][place] = top;
                    told->minima[h][place] = low == 0xffffffffu ? -neg_inf() : order_value(low);
                    if (place == 0 && !resumed)
                        told->next[h] = after;
                }
            } else if (!TEAM) { // the ninth warp is told to go, and what it has left open is known
                if (given)
                    named_bar_sync(BAR_TAKEN, W * 32 + 32);
                given = false;
                if (!resumed) {
                    if (r.warp == 0) {
                        if (lane == 0)
                            sm.task.row = -1;
                        __syncwarp();
                        named_bar_arrive(BAR_GIVEN, 64);
                    }
                    named_bar_sync(BAR_TAKEN, W * 32 + 32);
                }
            }
            if (!TEAM && tid == 0) {
                sm.redone[h] = *reinterpret_cast<volatile int *>(&sm.left_open);
                __threadfence_block();
            }
            resumed = false;
            team_sync<W>(parts);
            if (TEAM ? last >= 0 && sm.open[h ^ 1] == turn - 1 : last >= 0 && (redone < sm.redone[h] || sm.open[h ^ 1] == turn - 1)) {
                slow = BACK;
                break;
            }
            if (!have) {
                slow = END;
                break;
            }
            float m, lowest;
            {
                const bool one = lane < slots, two = TEAM && lane + 32 < slots;
                const float x = one ? sm.maxima[h][lane] : neg_inf(), y = two ? sm.maxima[h][lane + 32] : neg_inf();
                m = warp_top(max_nan(x, y));
                const float v = fminf(one ? sm.minima[h][lane] : -neg_inf(), two ? sm.minima[h][lane + 32] : -neg_inf());
                lowest = order_value(__reduce_min_sync(0xffffffffu, order_bits(v)));
            }
            for (int i = tid; i < GUIDE; i += W * 32)
                sm.guide[h ^ 1][i] = 0u;
            if (tid == 0) // all have read what the row before listed, and list again behind the next barrier
                sm.listed = 0;
            Settings a;
            a.take(sm.settings[h]);
            if (tid < 5 && next < p.M)
                Settings::fetch(p, next, tid, sm.settings[h ^ 1]);
            const bool bad = a.bad(), empty = m == neg_inf(), none = bad || !(m < -neg_inf());
            if (bad && tid == 0)
                sm.out_of_range = 1;
            bool loaded = false; // the next row was asked for
            if (empty || none) {
                if (tid == 0 && part == 0) {
                    p.tokens[row] = -1;
                    if (p.logprob != nullptr)
                        p.logprob[row] = none ? quiet_nan() : neg_inf();
                    if (p.kept != nullptr)
                        p.kept[row] = 0;
                }
            } else if (a.greedy()) {
                if (mine == m) // few threads
                    atomicMin(&lead->first[h], first_from(r, m));
                team_sync<W>(parts);
                if (tid == 0 && part == 0) {
                    p.tokens[row] = sm.first[h];
                    sm.first[h] = 0x7fffffff;
                    if (p.logprob != nullptr)
                        p.logprob[row] = 0.0f;
                    if (p.kept != nullptr)
                        p.kept[row] = 1;
                }
            } else {
                const Scale s = scale_of(m, a.t);
                const int k = a.limit(p.V);
                const bool by_p = a.p < 1.0f, plain = k == 0 && !by_p && !(a.least > 0.0f), whole = k == 0 && (by_p || plain);

                // ---- the threads' maxima, in bins from the row's down to their lowest
                const float per_bin = fminf(m - lowest, 60.0f / s.c) * (1.0f / (GUIDE - 1));
                if (!plain && (k > 0 || by_p) && mine > neg_inf()) {
                    const float bins = per_bin > 0.0f ? 1.0f / per_bin : 0.0f;
                    const int bin = min(GUIDE - 1, (int)((m - mine) * bins));
                    atomicAdd(&sm.guide[h][bin], k > 0 ? 1u : (uint32_t)(exp2_fast((mine - m) * s.c) * 0x1p20f));
                }
                // ---- fp32 sum over the vocabulary, where nothing else bounds what is kept
                u64 own = 0ull, own_rest = 0ull, rest = 0ull;
                int equal = 0;
                if (whole) {
                    own = warp_sum64(rest_of(r, s, mine, group, equal));
                    equal = __reduce_add_sync(0xffffffffu, equal);
                    if (plain && p.kept != nullptr) {
                        const int alive = __reduce_add_sync(0xffffffffu, alive_of(r));
                        if (lane == 0 && alive != 0)
                            atomicAdd(&lead->alive[h], alive);
                    }
                    if (lane < parts) {
                        told->rest[h][place] = own;
                        told->equal[h][place] = equal;
                    }
                    own_rest = own;
                    own += (u64)equal << SUM_SCALE;
                }
                team_sync<W>(parts);
                float margin = 0.0f;
                u64 before = 0ull; // of the warps in front
                if (whole) {
                    const bool one = lane < slots, two = TEAM && lane + 32 < slots;
                    const u64 r0 = one ? sm.rest[h][lane] : 0ull, r1 = two ? sm.rest[h][lane + 32] : 0ull;
                    const int e0 = one ? sm.equal[h][lane] : 0, e1 = two ? sm.equal[h][lane + 32] : 0;
                    rest = warp_sum64(r0 + r1);
                    equal = __reduce_add_sync(0xffffffffu, e0 + e1);
                    if (plain)
                        before = warp_sum64((lane < place ? r0 + ((u64)e0 << SUM_SCALE) : 0ull) +
                                            (lane + 32 < place ? r1 + ((u64)e1 << SUM_SCALE) : 0ull));
                    margin = sum_margin((float)rest * SUM_UNIT, p.V, 5.0f);
                }
                if (plain) {
                    // ---- in the warp that the target lies in, by fp32 sums
                    const u64 total = rest + ((u64)equal << SUM_SCALE);
                    const u64 target = __umul64hi(fraction(a.u), total);
                    if (target >= before && target < before + own) {
                        Drawn d;
                        bool sure = false;
                        if (walk(r, s, target - before, d)) {
                            // the same weights, four vectors' sums of which have five roundings, and now three
                            const u64 mg = draw_slack(a.u, total, rest, margin, 8.0f * 0x1p-24f * (float)own_rest * SUM_UNIT, p.V);
                            const u64 at = target - before - d.before;
                            sure = at >= mg && at + mg < d.w && !(a.u < 0x1p-40f);
                            if (sure) {
                                p.tokens[row] = d.i;
                                if (p.logprob != nullptr)
                                    p.logprob[row] = (d.x - m) * a.t - log1pf((float)(total - (1ull << SUM_SCALE)) * SUM_UNIT);
                            }
                        }
                        sure = __any_sync(0xffffffffu, sure);
                        if (!sure && lane < parts)
                            told->open[h] = turn;
                    }
                    if (p.kept != nullptr && tid == 0 && part == 0) { // all that are not masked
                        p.kept[row] = sm.alive[h];
                        sm.alive[h] = 0;
                    }
                } else {
                    // ---- a bound that all of them reach
                    const float low = a.least > 0.0f ? value_at(s, log2f(a.least) - 0.01f) : neg_inf();
                    float bound = neg_inf();
                    if (k > 0 || by_p) {
                        uint32_t g0, g1;
                        if (!TEAM) {
                            g0 = sm.guide[h][2 * lane];
                            g1 = sm.guide[h][2 * lane + 1];
                        } else {
                            uint2 g[MAX_PARTS]; // all on their way at once
#pragma unroll
                            for (int q = 0; q < MAX_PARTS; ++q)
                                g[q] = q < parts ? *reinterpret_cast<const uint2 *>(&cl.map_shared_rank(&sm, q)->guide[h][2 * lane]) : make_uint2(0u, 0u);
                            g0 = g1 = 0u;
#pragma unroll
                            for (int q = 0; q < MAX_PARTS; ++q) {
                                g0 += g[q].x;
                                g1 += g[q].y;
                            }
                        }
                        const float z = (float)(rest + ((u64)equal << SUM_SCALE)) * SUM_UNIT;
                        const float need = fminf(z * a.p * 1.0001f * 0x1p20f + 4096.0f, 4e9f);
                        bound = guide_bound(g0, g1, k > 0 ? (uint32_t)k : (uint32_t)need, m, lowest, per_bin, lane);
                        if (k == 0) // elements below 1 - p of the whole's mean do not reach 1 - p together
                            bound = fmaxf(bound, value_at(s, log2f((1.0f - a.p) * z / (float)p.V) - 0.01f));
                    }
                    bool least_bound = false;
                    if (k == 0 || !by_p) { // what top-p takes a share of has to be listed in whole
                        least_bound = low > bound;
                        bound = fmaxf(bound, low);
                    }
                    bound = fmaxf(bound, LEAST);

                    // ---- list them, where the bound leaves anything out
                    const bool listing = bound > LEAST || p.V <= LIST;
                    if (!TEAM && given) { // the list before is out of the way
                        named_bar_sync(BAR_TAKEN, W * 32 + 32);
                        given = false;
                    }
                    if (listing && __any_sync(0xffffffffu, mine >= bound)) // the warp has any
                        for (int v0 = r.w0; v0 < r.w1; v0 += 1024) {       // 32 vectors a lane
                            const int v1 = min(r.w1, v0 + 1024);
                            uint32_t near = 0u; // of them, those that reach it
                            if (mine >= bound)
#pragma unroll 4
                                for (int v = v0 + lane, j = 0; v < v1; v += 32, ++j)
                                    near |= Vec<T>::largest(r.vec[v]) >= bound ? 1u << j : 0u;
                            int n = 0;
                            for (uint32_t left = near; left != 0u; left &= left - 1u) {
                                float f[E];
                                Vec<T>::unpack(r.vec[v0 + 32 * (__ffs(left) - 1) + lane], f);
#pragma unroll
                                for (int e = 0; e < E; ++e)
                                    n += f[e] >= bound;
                            }
                            int upto = n;
#pragma unroll
                            for (int o = 1; o < 32; o <<= 1) {
                                const int u = __shfl_up_sync(0xffffffffu, upto, o);
                                upto += lane >= o ? u : 0;
                            }
                            int base = 0;
                            if (lane == 31 && upto > 0)
                                base = atomicAdd(&lead->listed, upto);
                            base = __shfl_sync(0xffffffffu, base, 31);
                            if (base > LIST) // too many
                                break;
                            int to = base + upto - n;
                            for (uint32_t left = near; left != 0u; left &= left - 1u) {
                                const int v = v0 + 32 * (__ffs(left) - 1) + lane;
                                float f[E];
                                Vec<T>::unpack(r.vec[v], f);
#pragma unroll
                                for (int e = 0; e < E; ++e)
                                    if (f[e] >= bound) {
                                        if (to < LIST) {
                                            lead->list[to].x = f[e];
                                            lead->list[to].i = r.first + v * E + e;
                                        }
                                        ++to;
                                    }
                            }
                        }
                    team_sync<W>(parts);
                    const int n = listing ? lead->listed : LIST + 1;
                    if (n > LIST) {
                        slow = HERE;
                        break;
                    }
                    if (next < p.M) { // the list has what is needed of this one
                        r.load(logits + (int64_t)next * p.stride, p.V, part, parts);
                        loaded = true;
                    }
                    if (part == 0) {
                        if (tid == 0) {
                            ListTask &q = sm.task;
                            q.n = n;
                            q.k = k;
                            q.equal = equal;
                            q.rest = rest;
                            q.margin = margin;
                            q.by_p = by_p;
                            q.least_bound = least_bound;
                            q.row = row;
                            q.a = a;
                            q.s = s;
                        }
                        if (!TEAM) {
                            if (r.warp == 0) {
                                __syncwarp();
                                named_bar_arrive(BAR_GIVEN, 64);
                            }
                            given = true;
                        } else {
                            cta_sync<W>(); // the task is there
                            const bool ok = finish_list(sm, sm.list, p, sm.task);
                            if (!ok && r.warp == 0 && lane < parts)
                                told->open[h] = turn;
                        }
                    }
                }
            }
            if (!loaded && next < p.M)
                r.load(logits + (int64_t)next * p.stride, p.V, part, parts);
            last = row;
            row = next;
            next = sm.next[h];
        }
        if (slow == END)
            break;
        if (slow == HERE) { // more than the list holds
            team_sync<W>(parts); // all have read how many
            if (tid == 0)
                sm.listed = 0;
            if (!fine_row(sm, r, p, row, part, parts))
                exact_row(sm, r, p, row, part, parts);
            if (next < p.M)
                r.load(logits + (int64_t)next * p.stride, p.V, part, parts);
            last = row;
            row = next;
            next = sm.next[turn & 1];
            ++turn;
        } else { // rows that were left open, by the ninth warp or by the team
            const int known = TEAM ? 0 : sm.redone[turn & 1];
            bool again = sm.open[(turn & 1) ^ 1] == turn - 1;
            if (given)
                named_bar_sync(BAR_TAKEN, W * 32 + 32);
            given = false;
            while (redone < known || again) {
                int back = last;
                if (redone < known)
                    back = sm.redo[redone++ % REDO];
                else
                    again = false;
                r.load(logits + (int64_t)back * p.stride, p.V, part, parts);
                r.wait();
                if (!fine_row(sm, r, p, back, part, parts))
                    exact_row(sm, r, p, back, part, parts);
            }
            if (tid == 0)
                sm.open[(turn & 1) ^ 1] = -1;
            if (row < p.M)
                r.load(logits + (int64_t)row * p.stride, p.V, part, parts);
            resumed = true;
        }
    }
    if (TEAM)
        team_sync<W>(parts); // others may still read this CTA's
    if (r.late)
        sm.late = 1;
    r.close();
    cta_sync<W>();
    if (tid == 0)
        CallCounts::of(p.status).close((sm.out_of_range ? (uint32_t)LORA_FLAG_SETTING_RANGE : 0u) |
                                           (sm.late ? (uint32_t)LORA_FLAG_WAIT_TIMEOUT : 0u), gridDim.x);
}

namespace {

// ---------------------------------------------------------------- many rows

// Where there are many rows, they are not kept: eight warps of a CTA read one after
// another, each thread with its maximum and, where no setting bounds what is kept,
// each warp with the sum of each of its runs of 128 vectors relative to a reference
// that trails the maximum; and four warps finish them in turn. The threads whose
// maximum reaches the bound are few, and their shares are read again from L2; a draw
// from the whole vocabulary reads the run that it falls into. Nothing the finishing
// warps do stops the loads. What they leave open is marked in `tokens`, for the
// kernels behind. 8192 x 32000 bf16 (77 us by its bytes), whole calls: 137 us of min-p, where
// the maxima bound it; 180 where nothing is cut, with some 70 rows for the kernels behind;
// 185 of top-p at temperature 0.5, 241 of top 50, where the finishing warps do.
constexpr int READERS = 256, READ_WARPS = READERS / 32, FINISHERS = 4, AHEAD = 4;
constexpr int READ_THREADS = READERS + 32 * FINISHERS;
constexpr int GROUP = AHEAD * READERS;                                 // vectors that a CTA reads at once,
constexpr int MAX_GROUPS = 48;                                         // a run of 128 a warp
constexpr int BAR_FULL = 1, BAR_FREE = 1 + FINISHERS;                  // of each finishing warp
constexpr int OPEN = (int)0x80000000;
constexpr float TRAIL = 8.0f;  // log2 of what a reference may trail the maximum by

struct ReadShared {
    u64 powers[32];
    float2 left[FINISHERS][READERS];                  // a thread's maximum and the first vector with it
    float2 runs[FINISHERS][MAX_GROUPS * READ_WARPS];  // a run's sum and its reference
    Entry list[FINISHERS][LIST];
    uint4 near[FINISHERS][LIST]; // vectors with an element that reaches the bound, and where they begin
    int near_at[FINISHERS][LIST];
    uint32_t guide[FINISHERS][GUIDE];
    uint16_t picked[FINISHERS][READERS];
    ListTask task[FINISHERS];
};

// As load_vec, for any v.
template <typename T> __device__ __forceinline__ uint4 reload(const T *x, int V, int lead, int v, int nvec)
{
    return v < nvec ? load_vec(x, V, lead, v) : empty_vec<T>();
}

// The vectors of a thread, AHEAD of a group at a time.
__device__ __forceinline__ int own_vector(int thread, int group, int q)
{
    return group * GROUP + (thread >> 5) * (32 * AHEAD) + q * 32 + (thread & 31);
}
template <typename T> struct Stream {
    static constexpr int E = Vec<T>::E;
    const T *x;
    int lead, nvec;
    uint4 next[AHEAD];

    __device__ __forceinline__ void fetch(int group, int V)
    {
        const int v0 = own_vector((int)threadIdx.x, group, 0), run = v0 - (int)(threadIdx.x & 31); // the warp's
        if ((run > 0 || lead == 0) && run + 32 * AHEAD <= (lead + V) / E) {
            const uint4 *v = reinterpret_cast<const uint4 *>(x - lead) + v0;
#pragma unroll
            for (int q = 0; q < AHEAD; ++q)
                asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(next[q].x), "=r"(next[q].y), "=r"(next[q].z), "=r"(next[q].w)
                             : "l"(v + q * 32));
        } else {
#pragma unroll
            for (int q = 0; q < AHEAD; ++q)
                next[q] = reload(x, V, lead, v0 + q * 32, nvec);
        }
    }
    __device__ __forceinline__ void enter(const T *row, int V)
    {
        x = row;
        lead = row_lead(x);
        nvec = (lead + V + E - 1) / E;
        fetch(0, V);
    }
};

// The token of a row that nothing cuts, by one warp, from the sums of its runs. False
// where fp32 sums leave it open.
template <typename T>
__device__ __forceinline__ bool draw_from_all(const ReadShared &sm, int which, const SampleParams &p, int row, const Settings &a, const Scale &s)
{
    constexpr int E = Vec<T>::E;
    const T *x = static_cast<const T *>(p.logits) + (int64_t)row * p.stride;
    const int lead = row_lead(x), nvec = (lead + p.V + E - 1) / E, lane = threadIdx.x & 31;
    const int runs = (nvec + 32 * AHEAD - 1) / (32 * AHEAD);
    if (a.u < 0x1p-40f)
        return false;
    auto sum_of_run = [&](int i) { // at least 0, and the same every time
        const float2 f = sm.runs[which][i];
        return f.x > 0.0f ? as_fixed(f.x * exp2_fast((f.y - s.m) * s.c), SUM_SCALE) : 0ull;
    };
    u64 total = 0ull;
    for (int i = lane; i < runs; i += 32)
        total += sum_of_run(i);
    total = warp_sum64(total);
    const u64 target = __umul64hi(fraction(a.u), total);
    u64 before = 0ull, own_run = 0ull;
    int run = -1;
    for (int i0 = 0; i0 < runs; i0 += 32) {
        const u64 own = i0 + lane < runs ? sum_of_run(i0 + lane) : 0ull;
        u64 upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 n = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? n : 0ull;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, before + upto > target);
        if (past != 0u) {
            const int l = __ffs(past) - 1;
            run = i0 + l;
            before += __shfl_sync(0xffffffffu, upto - own, l);
            own_run = __shfl_sync(0xffffffffu, own, l);
            break;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    // a thread adds 4 AHEAD pairs, a warp 5 more; the sum is rescaled; then those of the run that is looked into
    constexpr float adds = 4.0f * AHEAD + 5.0f + 12.0f;
    const u64 slack = draw_slack(a.u, total, total, sum_margin((float)total * SUM_UNIT, p.V, adds),
                                 2.0f * sum_margin((float)own_run * SUM_UNIT, p.V, adds), p.V);
    uint4 raw[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
        raw[j] = reload(x, p.V, lead, run >= 0 ? run * (32 * AHEAD) + 32 * j + lane : nvec, nvec);
    bool drawn = false, past = false;
    float lp = 0.0f;
    int token = 0;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
        int none;
        const u64 own = as_fixed(vector_rest<T, false>(raw[j], s, none), SUM_SCALE);
        u64 upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 n = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? n : 0ull;
        }
        const u64 all = __shfl_sync(0xffffffffu, upto, 31);
        u64 at = before + upto - own;
        if (!past && target >= at && target < at + own) {
            float f[E];
            Vec<T>::unpack(raw[j], f);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const u64 w = as_fixed(exp2_fast(__fmul_rn(f[e] - s.m, s.c)), SUM_SCALE);
                if (target >= at + slack && target + slack < at + w && !drawn) {
                    drawn = true;
                    token = (run * (32 * AHEAD) + 32 * j + lane) * E - lead + e;
                    lp = (f[e] - s.m) * a.t - log1pf((float)(total - (1ull << SUM_SCALE)) * SUM_UNIT);
                }
                at += w;
            }
        }
        past |= target < before + all;
        before += all;
    }
    if (drawn) {
        p.tokens[row] = token;
        if (p.logprob != nullptr)
            p.logprob[row] = lp;
    }
    return __any_sync(0xffffffffu, drawn);
}

// A row that has been read, by one warp. False where it is left open.
template <typename T>
__device__ __forceinline__ bool finish_row(ReadShared &sm, const SampleParams &p, int row, int which)
{
    constexpr int E = Vec<T>::E, PER = READERS / 32;
    const int lane = threadIdx.x & 31;
    const T *x = static_cast<const T *>(p.logits) + (int64_t)row * p.stride;
    const int lead = row_lead(x), nvec = (lead + p.V + E - 1) / E, groups = (nvec + GROUP - 1) / GROUP;
    Settings a;
    a.read(p, row);
    for (int i = lane; i < GUIDE; i += 32)
        sm.guide[which][i] = 0u;
    named_bar_sync(BAR_FULL + which, READERS + 32);
    float own[PER], m, lowest = -neg_inf();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        own[i] = sm.left[which][i * 32 + lane].x;
        m = i == 0 ? own[0] : max_nan(m, own[i]);
        lowest = fminf(lowest, own[i] > neg_inf() ? own[i] : -neg_inf());
    }
    m = warp_top(m);
    lowest = order_value(__reduce_min_sync(0xffffffffu, order_bits(lowest)));
    const bool bad = a.bad(), empty = m == neg_inf(), none = bad || !(m < -neg_inf());
    if (empty || none) {
        if (lane == 0) {
            p.tokens[row] = -1;
            if (p.logprob != nullptr)
                p.logprob[row] = none ? quiet_nan() : neg_inf();
            if (p.kept != nullptr)
                p.kept[row] = 0;
            if (bad) // the status is written by the last kernel
                CallCounts::of(p.status).flag((uint32_t)LORA_FLAG_SETTING_RANGE);
        }
        return true;
    }
    if (a.greedy()) {
        int v = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            v = own[i] == m ? min(v, __float_as_int(sm.left[which][i * 32 + lane].y)) : v;
        v = __reduce_min_sync(0xffffffffu, v);
        if (lane == 0) {
            float f[E];
            Vec<T>::unpack(load_vec(x, p.V, lead, v), f);
            int at = 0;
#pragma unroll
            for (int e = E - 1; e >= 0; --e)
                at = f[e] == m ? e : at;
            p.tokens[row] = v * E - lead + at;
            if (p.logprob != nullptr)
                p.logprob[row] = 0.0f;
            if (p.kept != nullptr)
                p.kept[row] = 1;
        }
        return true;
    }
    const Scale s = scale_of(m, a.t);
    const int k = a.limit(p.V);
    const bool by_p = a.p < 1.0f;
    if (k == 0 && !by_p && !(a.least > 0.0f)) {
        if (p.kept != nullptr) { // the readers have counted them
            int n = 0;
            for (int i = lane; i < READERS; i += 32)
                n += __float_as_int(sm.left[which][i].y);
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0)
                p.kept[row] = n;
        }
        return draw_from_all<T>(sm, which, p, row, a, s);
    }
    // ---- the bound, as in sample_kernel
    const float low = a.least > 0.0f ? value_at(s, log2f(a.least) - 0.01f) : neg_inf();
    float bound = neg_inf(), sum = 0.0f, margin = 0.0f;
    if (k == 0 && by_p) {
        for (int i = lane; i < groups * READ_WARPS; i += 32) {
            const float2 f = sm.runs[which][i];
            sum += f.x > 0.0f ? f.x * exp2_fast((f.y - m) * s.c) : 0.0f;
        }
        sum = warp_sum(sum);
        margin = sum_margin(sum, p.V, 4.0f * AHEAD + 5.0f + 12.0f + (float)(groups * READ_WARPS) * (1.0f / 32) + 5.0f);
    }
    if (k > 0 || by_p) {
        const float per_bin = fminf(m - lowest, 60.0f / s.c) * (1.0f / (GUIDE - 1)), bins = per_bin > 0.0f ? 1.0f / per_bin : 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (own[i] > neg_inf())
                atomicAdd(&sm.guide[which][min(GUIDE - 1, (int)((m - own[i]) * bins))],
                          k > 0 ? 1u : (uint32_t)(exp2_fast((own[i] - m) * s.c) * 0x1p20f));
        __syncwarp();
        const float need = fminf(sum * a.p * 1.0001f * 0x1p20f + 4096.0f, 4e9f);
        bound = guide_bound(sm.guide[which][2 * lane], sm.guide[which][2 * lane + 1], k > 0 ? (uint32_t)k : (uint32_t)need, m, lowest, per_bin, lane);
        if (k == 0)
            bound = fmaxf(bound, value_at(s, log2f((1.0f - a.p) * sum / (float)p.V) - 0.01f));
    }
    bool least_bound = false;
    if (k == 0 || !by_p) {
        least_bound = low > bound;
        bound = fmaxf(bound, low);
    }
    bound = fmaxf(bound, LEAST);
    if (!(bound > LEAST))
        return false;
    // ---- the threads with any, and of their shares the vectors with what reaches it
    const uint32_t ahead_of = (1u << lane) - 1u;
    int picked = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool is = own[i] >= bound;
        const uint32_t all = __ballot_sync(0xffffffffu, is);
        if (is)
            sm.picked[which][picked + __popc(all & ahead_of)] = (uint16_t)(i * 32 + lane);
        picked += __popc(all);
    }
    if (picked > LIST)
        return false;
    __syncwarp();
    const int share = groups * AHEAD, items = picked * share; // below 2^16
    const uint32_t over = 0xffffffffu / (uint32_t)share + 1u; // i / share is the upper word of i over
    int vecs = 0;
    uint4 coming[AHEAD];
    int coming_at[AHEAD];
    auto ask = [&](int i0) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int i = i0 + 32 * j + lane, pick = (int)__umulhi((uint32_t)i, over), r = i - pick * share;
            const int v = i < items ? own_vector((int)sm.picked[which][pick], r / AHEAD, r % AHEAD) : nvec;
            coming_at[j] = v * E - lead;
            coming[j] = reload(x, p.V, lead, v, nvec);
        }
    };
    ask(0);
    for (int i0 = 0; i0 < items; i0 += 32 * AHEAD) {
        uint4 raw[AHEAD];
        int at[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            raw[j] = coming[j];
            at[j] = coming_at[j];
        }
        if (i0 + 32 * AHEAD < items)
            ask(i0 + 32 * AHEAD);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const bool hit = Vec<T>::largest(raw[j]) >= bound;
            const uint32_t all = __ballot_sync(0xffffffffu, hit);
            const int to = vecs + __popc(all & ahead_of);
            if (hit && to < LIST) {
                sm.near[which][to] = raw[j];
                sm.near_at[which][to] = at[j];
            }
            vecs += __popc(all);
        }
        if (vecs > LIST)
            return false;
    }
    __syncwarp();
    // ---- and the elements
    Entry *const list = sm.list[which];
    int n = 0;
    for (int g = 0; g < vecs; g += 32) {
        const bool have = g + lane < vecs;
        float f[E];
        Vec<T>::unpack(have ? sm.near[which][g + lane] : empty_vec<T>(), f);
        const int at = have ? sm.near_at[which][g + lane] : 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const bool hit = f[e] >= bound;
            const uint32_t all = __ballot_sync(0xffffffffu, hit);
            const int to = n + __popc(all & ahead_of);
            if (hit && to < LIST) {
                list[to].x = f[e];
                list[to].i = at + e;
            }
            n += __popc(all);
        }
    }
    if (n > LIST)
        return false;
    ListTask &task = sm.task[which];
    if (lane == 0) {
        task.n = n;
        task.k = k;
        task.equal = 0;
        task.rest = as_fixed(sum, SUM_SCALE);
        task.margin = margin;
        task.by_p = by_p;
        task.least_bound = least_bound;
        task.row = row;
        task.a = a;
        task.s = s;
    }
    __syncwarp();
    return finish_any(sm.powers, list, p, task);
}

} // namespace

template <typename T> __global__ void __launch_bounds__(READ_THREADS, 2) read_rows_kernel(SampleParams p)
{
    constexpr int E = Vec<T>::E;
    __shared__ ReadShared sm;
    begin_behind();
    const int tid = threadIdx.x, lane = tid & 31, step = gridDim.x;
    const T *logits = static_cast<const T *>(p.logits);
    if (tid < 32)
        sm.powers[tid] = POWERS[tid];
    if (tid == 0)
        CallCounts().open<5>(p.status);
    __syncthreads();
    if (tid < READERS) {
        Stream<T> in;
        in.enter(logits + (int64_t)blockIdx.x * p.stride, p.V);
        const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
        float t, next_t;
        int sums, next_sums; // whether the row's sum is needed: 2 where nothing cuts it
        auto settings = [&](int row, float &t, int &sums) {
            t = p.inv_t != nullptr ? p.inv_t[row] : 1.0f;
            const int k = p.top_k != nullptr ? p.top_k[row] : 0;
            const float top = p.top_p != nullptr ? p.top_p[row] : 1.0f, least = p.min_p != nullptr ? p.min_p[row] : 0.0f;
            sums = (k > 0 && k < p.V) || top <= 0.0f ? 0 : top < 1.0f ? 1 : least > 0.0f ? 0 : 2;
        };
        settings(blockIdx.x, t, sums);
        for (int row = blockIdx.x, turn = 0; row < p.M; row += step, ++turn) {
            const int nvec = in.nvec, which = turn % FINISHERS;
            const float c = __fmul_rn(t, 0x1.715476p+0f), trail = TRAIL / c;
            if (row + step < p.M)
                settings(row + step, next_t, next_sums);
            float m = neg_inf(), at = neg_inf(), limit = neg_inf();
            int best = 0, alive = 0;
            if (turn >= FINISHERS) // the row that used the place is done
                named_bar_sync(BAR_FREE + which, READERS + 32);
            for (int group = 0; group * GROUP < nvec; ++group) {
                uint4 cur[AHEAD];
#pragma unroll
                for (int q = 0; q < AHEAD; ++q)
                    cur[q] = in.next[q];
                if ((group + 1) * GROUP < nvec)
                    in.fetch(group + 1, p.V);
                else if (row + step < p.M)
                    in.enter(logits + (int64_t)(row + step) * p.stride, p.V);
                float vm[AHEAD], gm;
#pragma unroll
                for (int q = 0; q < AHEAD; ++q) {
                    vm[q] = Vec<T>::largest(cur[q]);
                    gm = q == 0 ? vm[0] : max_nan(gm, vm[q]);
                }
                if (!(gm <= m)) {
                    m = max_nan(m, gm);
                    int q = AHEAD - 1;
#pragma unroll
                    for (int j = AHEAD - 2; j >= 0; --j)
                        q = vm[j] == gm ? j : q;
                    best = own_vector(tid, group, q);
                }
                if (sums != 0) { // the same for all
                    if (__any_sync(0xffffffffu, !(gm <= limit))) { // a new reference for the warp
                        at = max_nan(at, warp_top(gm));
                        limit = at + trail;
                    }
                    const float a = at == neg_inf() ? 0.0f : at;
                    const f2 na = make_f2(-a, -a), c2 = make_f2(c, c);
                    f2 s0 = make_f2(0.0f, 0.0f), s1 = s0;
#pragma unroll
                    for (int q = 0; q < AHEAD; ++q) {
                        float f[E];
                        Vec<T>::unpack(cur[q], f);
#pragma unroll
                        for (int e = 0; e < E; e += 2) {
                            float a0, a1;
                            split_f2(mul_f2(add_f2(make_f2(f[e], f[e + 1]), na), c2), a0, a1);
                            f2 &to = e & 2 ? s1 : s0;
                            to = add_f2(to, make_f2(exp2_fast(a0), exp2_fast(a1)));
                        }
                        if (sums == 2 && p.kept != nullptr) {
                            if (Vec<T>::smallest(cur[q]) > neg_inf()) {
                                alive += E;
                            } else {
#pragma unroll
                                for (int e = 0; e < E; ++e)
                                    alive += f[e] > neg_inf();
                            }
                        }
                    }
                    float s0a, s0b;
                    split_f2(add_f2(s0, s1), s0a, s0b);
                    const float sum = warp_sum(s0a + s0b);
                    if (lane == 0)
                        sm.runs[which][group * READ_WARPS + warp] = make_float2(sum, at);
                }
            }
            sm.left[which][tid] = make_float2(m, __int_as_float(sums == 2 && !(t > 0x1p64f) ? alive : best));
            t = next_t;
            sums = next_sums;
            named_bar_arrive(BAR_FULL + which, READERS + 32);
        }
        return;
    }
    const int which = (tid - READERS) / 32;
    for (int row = blockIdx.x + which * step; row < p.M; row += FINISHERS * step) {
        if (!finish_row<T>(sm, p, row, which) && lane == 0) {
            p.tokens[row] = OPEN;
            CallCounts::of(p.status).left_open(CallCounts::OPENED, row);
        }
        __syncwarp();
        if (row + FINISHERS * step < p.M) // the place is used again
            named_bar_arrive(BAR_FREE + which, READERS + 32);
    }
}

// The rows that read_rows_kernel left open. Up to `most` of them are gone through by
// the call's last kernel, each by a cluster of the most parts; of more, by the kernel
// in front of it, by teams as large as they have to be, and the last one has those that
// fine sums leave open too. A few are in the workspace's list, others have to be
// looked for among `some` rows at a time. The last kernel writes the call's status.
// Of 8192 x 32000 bf16, top-p 0.95 at temperature 1 (571 us a call), some 2400 rows come here
// and take more than half of it by three CTAs an SM: maximum, rough sum, bins, fine sums and
// draw one after another in shared memory, whose barriers 24 warps do not hide.
template <typename T, bool TEAM>
__global__ void __launch_bounds__(256, 3) open_rows_kernel(SampleParams p, int parts_, int some, int most, int last)
{
    constexpr int W = 8;
    extern __shared__ uint4 slice[];
    __shared__ Shared<W> sm;
    begin_behind();
    cg::cluster_group cl = cg::this_cluster();
    const int parts = TEAM ? parts_ : 1, part = TEAM ? (int)blockIdx.x % parts : 0, tid = threadIdx.x, lane = tid & 31;
    const int team = (int)blockIdx.x / parts, teams = (int)gridDim.x / parts;
    const CallCounts counts = CallCounts::of(p.status);
    const int opened = counts.count(CallCounts::OPENED);
    const bool again = last && opened > most;
    if (!last && opened <= most)
        return;
    const int mine = again ? counts.count(CallCounts::AGAIN) : opened;
    Row<T, W> r;
    r.open(slice, sm.bars);
    if (tid < 32)
        sm.powers[tid] = POWERS[tid];
    if (tid == 0)
        sm.late = 0;
    Shared<W> *const told = TEAM && lane < parts ? cl.map_shared_rank(&sm, lane) : &sm;
    int chunk = 0;      // rows from here on
    uint32_t open = 0u; // of them, those that are open
    if (TEAM)
        team_sync<W>(parts); // all of the cluster are there
    for (int turn = 0; mine > 0; ++turn) {
        if (part == 0 && r.warp == 0) {
            int row = p.M;
            if (last && mine <= CallCounts::LISTED) {
                const int at = team + turn * teams;
                row = at < mine ? counts.listed(at) : p.M;
                row = (uint32_t)row < (uint32_t)p.M ? row : p.M; // whatever else was written there
            } else {
                while (open == 0u) {
                    int c = 0;
                    if (lane == 0)
                        c = (int)counts.add(again ? CallCounts::NEXT_AGAIN : CallCounts::NEXT);
                    c = __shfl_sync(0xffffffffu, c, 0);
                    if ((int64_t)c * some >= p.M)
                        break;
                    chunk = c * some;
                    open = __ballot_sync(0xffffffffu, lane < some && chunk + lane < p.M && p.tokens[chunk + lane] == OPEN);
                }
                row = open != 0u ? chunk + __ffs(open) - 1 : p.M;
                open &= open - 1u;
            }
            if (lane < parts)
                told->next[turn & 1] = row;
        }
        team_sync<W>(parts);
        const int row = sm.next[turn & 1];
        if (row >= p.M)
            break;
        r.load(static_cast<const T *>(p.logits) + (int64_t)row * p.stride, p.V, part, parts);
        r.wait();
        if (!again && fine_row(sm, r, p, row, part, parts))
            continue;
        if (last)
            exact_row(sm, r, p, row, part, parts);
        else if (part == 0 && tid == 0)
            counts.left_open(CallCounts::AGAIN, row);
    }
    if (TEAM)
        team_sync<W>(parts);
    if (r.late)
        sm.late = 1;
    r.close();
    __syncthreads();
    if (tid == 0) {
        if (last)
            counts.close(sm.late ? (uint32_t)LORA_FLAG_WAIT_TIMEOUT : 0u, gridDim.x);
        else if (sm.late)
            counts.flag((uint32_t)LORA_FLAG_WAIT_TIMEOUT);
    }
}

template <typename T, int W, bool TEAM> cudaError_t launch_as(const SampleParams &p, const TeamPlan &t, cudaStream_t st)
{
    const cudaError_t e = allow_smem<sample_kernel<T, W, TEAM>>();
    if (e != cudaSuccess)
        return e;
    return launch_behind(sample_kernel<T, W, TEAM>, dim3((unsigned)(t.teams * t.parts)), W * 32 + (TEAM ? 0 : 32), t.smem, (unsigned)t.parts,
                         st, p, t.parts);
}
template <typename T> cudaError_t launch_typed(const SampleParams &p, int num_sms, cudaStream_t st)
{
    // Read through registers, rows get along without a cluster's barriers, but wait for the other kernels of the call.
    // 600 rows: (512 and 590) x 32000 bf16 of top 50 take 37.5 and 37.6 us there and 30.5 and 32.2 here, x 9000 30.1
    // and 30.2 against 23.6 and 24.6, and of top-p at temperature 0.5 23.6 and 23.8 against 20.4 and 21.2, but x 32000
    // 37 and 62 us against 51 and 67. A row that nothing cuts is summed there in runs, few of which have to be looked
    // into: 152 x 131072 86 us against 121, 64 x 32000 45 against 47, but 152 x 32000 31 against 29, 64 x 131072 40
    // against 33, and 152 x 4000 16 against 11. Which settings rows have is not known here, only which arrays there are:
    // 256 and 512 x 131072 of mixed settings take 277 and 358 us, and would take 199 and 237 there.
    const bool plain = p.top_k == nullptr && p.top_p == nullptr && p.min_p == nullptr;
    const int many_rows = plain && p.V >= 16384 ? 64 : 600;

    if (p.M >= many_rows && p.V >= 2048 && p.V <= (MAX_GROUPS * GROUP - 1) * Vec<T>::E) {
        cudaError_t e = allow_smem<open_rows_kernel<T, true>>();
        if (e == cudaSuccess)
            e = allow_smem<open_rows_kernel<T, false>>();
        if (e != cudaSuccess)
            return e;
        const unsigned at_once = 2u * (unsigned)num_sms;
        e = launch_behind(read_rows_kernel<T>, dim3((unsigned)p.M < at_once ? (unsigned)p.M : at_once), READ_THREADS, 0, 1, st, p);
        if (e != cudaSuccess)
            return e;
        // One open row a cluster of eight: it takes a row a fifth of the time that a CTA does, but three times the SMs' time.
        // (8192 x 32000 bf16 of which nothing is cut: 180 us, with up to six rows a cluster 194. 1000 x 32000 of top-p at
        // temperature 1: 168 us, with up to six 270.) The few that fine sums leave open again are theirs in any case.
        const int64_t nvec = ((int64_t)p.V + Vec<T>::E - 1) / Vec<T>::E + 1;
        const int wide = num_sms * 3 / MAX_PARTS, most = wide;
        const size_t smem = (size_t)((nvec + MAX_PARTS - 1) / MAX_PARTS) * 16;
        auto some = [&](int64_t teams) { // rows that a team looks for open ones among at a time
            const int64_t each = p.M / (8 * teams);
            return each < 1 ? 1 : each > 32 ? 32 : (int)each;
        };
        if (p.M > most) {
            const TeamPlan t = plan_teams<T, 8>(p.M, p.V, num_sms, sizeof(Shared<8>));
            e = launch_behind(t.parts > 1 ? open_rows_kernel<T, true> : open_rows_kernel<T, false>, dim3((unsigned)(t.teams * t.parts)), 256, t.smem,
                              (unsigned)t.parts, st, p, t.parts, some(t.teams), most, 0);
            if (e != cudaSuccess)
                return CallCounts::give_up(e, p.status, st);
        }
        e = launch_behind(open_rows_kernel<T, true>, dim3((unsigned)(wide * MAX_PARTS)), 256, smem, (unsigned)MAX_PARTS, st, p, MAX_PARTS,
                          some(wide), most, 1);
        return e == cudaSuccess ? e : CallCounts::give_up(e, p.status, st);
    }
    // Two warps a short row (8192 x 1000 bf16 of which nothing is cut 66 us, of top-p 65; four 78 and 81, eight 112 and
    // 128), four where top-k has to guess a bound from the threads' maxima, of which 64 are too few (top 50: 86 us, with
    // two warps 145, with eight 144), but not of the shortest rows (500 elements: 172 us, with two 137).
    if (short_rows<T>(p.M, p.V, num_sms)) {
        if (p.top_k != nullptr && p.V >= 96 * Vec<T>::E)
            return launch_as<T, 4, false>(p, plan_teams<T, 4>(p.M, p.V, num_sms, sizeof(Shared<4>)), st);
        return launch_as<T, 2, false>(p, plan_teams<T, 2>(p.M, p.V, num_sms, sizeof(Shared<2>)), st);
    }
    const TeamPlan t = plan_teams<T, 8>(p.M, p.V, num_sms, sizeof(Shared<8>));
    return t.parts > 1 ? launch_as<T, 8, true>(p, t, st) : launch_as<T, 8, false>(p, t, st);
}

cudaError_t launch_sample(const SampleParams &p, int dtype, int num_sms, cudaStream_t st)
{
    return dtype == LORA_DTYPE_F32 ? launch_typed<float>(p, num_sms, st) : launch_typed<uint16_t>(p, num_sms, st);
}

} // namespace rd
