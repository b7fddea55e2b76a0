// The divergence of rows of logits from a teacher's distribution that is known
// on its best tokens only, and the gradient over the logits.
//
// With p = softmax(x t), m = max x, entries j (token v_j, teacher's share q_j), and
// r the elements that no entry names, p_r their sum:
//   loss = sum_j q_j (log q_j - log p_{v_j}) + q_r (log q_r - log p_r)
//   dx_v = t g (Q p_v - q_v)            v named
//   dx_v = t g (Q p_r - q_r) p_v / p_r  v not named, Q = sum_j q_j + q_r
// where either the q_j sum to 1 and q_r = 0, or q_r = 1 - sum_j q_j. A softmax of the
// rest by itself, with its own maximum, keeps p_v / p_r and log p_r good however
// little the rest has; so the named elements are taken out of the row first.
//
// distill_kernel       loss, statistics and, where rows' weights are given, the
//     gradient, with the row in shared memory (row_team.cuh): it is read once.
// distill_grad_kernel  the gradient by itself from the statistics: one pass.
#include <cooperative_groups.h>

#include "behind.cuh"
#include "lora_distill.cuh"
#include "row_team.cuh"

namespace rd {

namespace cg = cooperative_groups;

namespace {

constexpr int SHARE_SCALE = 53; // a share of the teacher is an integer of 2^-53: LORA_MAX_TEACHER of them fit
constexpr int BAR_MAX = 1, BAR_SUM = 2, BAR_ACROSS = 3;

// A row's entries, ready for use: id -1 where there is none.
struct __align__(16) Entries {
    int id[LORA_MAX_TEACHER];
    float val[LORA_MAX_TEACHER];
    u64 shares; // the sum of e^val 2^53, over e^best where they are to sum to 1
    float norm, norm_low; // log q = val - norm - norm_low: a teacher's plain logits may lie far from 0
    int spoilt;
};

// What the warps of a team have found in a row.
template <int W> struct Found {
    float rest_max[MAX_PARTS * W], named_max[MAX_PARTS * W];
    u64 rest[MAX_PARTS * W], named[MAX_PARTS * W];
    int equal[MAX_PARTS * W]; // of the rest's maximum, and 2^20 times of the row's among the named
};

template <int W> struct Shared {
    u64 powers[32];
    uint64_t bars[W];
    int late; // a copy was not there in time
    Found<W> found[2];
    Entries entries[3];           // the next row's are prepared while the last one's may still be read
    float x[2][LORA_MAX_TEACHER]; // the named elements, taken out of the row
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// log of an integer of 2^-bits that is at least 1.
__device__ __forceinline__ float log_fixed(u64 v, int bits)
{
    return log1pf((float)(v - (1ull << bits)) / (float)(1ull << bits));
}

// The numbers of a row that its sums give.
struct Numbers {
    float m, rest_max;
    bool none, empty, no_rest;
    float rest_sum, rest_equal, below, others; // the rest's over its maximum; log of that over the row's; S - 1
    float named;                               // what S has of the named ones
    float q_rest, total;

    template <int W> __device__ __forceinline__ void maxima(const Found<W> &f, int parts, bool spoilt, int lane)
    {
        static_assert(MAX_PARTS * W <= 32, "a lane for each");
        const bool one = lane < parts * W;
        rest_max = warp_top(one ? f.rest_max[lane] : neg_inf());
        m = max_nan(rest_max, warp_top(one ? f.named_max[lane] : neg_inf()));
        none = spoilt || !(m < -neg_inf());
        empty = !none && m == neg_inf();
        no_rest = !none && rest_max == neg_inf();
    }
    template <int W> __device__ __forceinline__ void sums(const Found<W> &f, const Entries &en, const DistillParams &p, int parts, int lane)
    {
        u64 r = 0ull, n = 0ull;
        int e = 0;
        if (lane < parts * W) {
            r = f.rest[lane];
            n = f.named[lane];
            e = f.equal[lane];
        }
        r = warp_sum64(r);
        n = warp_sum64(n);
        e = __reduce_add_sync(0xffffffffu, e);
        rest_equal = (float)(e & 0xFFFFF);
        rest_sum = (float)r * SUM_UNIT;
        below = no_rest || empty ? 0.0f : (rest_max - m) * p.inv_t;
        const int of_rest = rest_max == m; // one of the maxima is left out, of the rest where it has one
        const float at_rest = no_rest ? 0.0f : expf(below) * ((rest_equal - (float)of_rest) + rest_sum);
        others = fmaxf(at_rest + (float)((e >> 20) - (1 - of_rest)) + (float)n * 0x1p-53f, 0.0f);
        named = (float)(e >> 20) + (float)n * 0x1p-53f;
        q_rest = 0.0f;
        if (p.rest) {
            const u64 one = 1ull << SHARE_SCALE;
            if (!no_rest && en.shares < one)
                q_rest = (float)(one - en.shares) * 0x1p-53f;
            total = (float)(no_rest || en.shares > one ? en.shares : one) * 0x1p-53f;
        } else {
            total = en.shares != 0ull ? 1.0f : 0.0f;
        }
    }
    __device__ __forceinline__ float log_s() const { return none || empty ? 0.0f : log1pf(others); }
    // log p_r by the ratio of the named ones to the rest, whose digits it keeps where p_r is near 1: the difference of two
    // logarithms of 4 has 2^-22 of them at best. Where the rest is far below, by that.
    __device__ __forceinline__ float log_rest(float log_s) const
    {
        if (no_rest)
            return neg_inf();
        if (below > -64.0f)
            return -log1pf(named / (expf(below) * (rest_equal + rest_sum)));
        return below + (log1pf((rest_equal - 1.0f) + rest_sum) - log_s);
    }
};

// log q - log p of an entry, as good as its parts: the products and differences as two numbers each.
__device__ __forceinline__ float log_ratio(const Numbers &a, const Entries &en, float log_s, float t, float x, float val)
{
    if (!(x > neg_inf()))
        return -x; // a masked element
    if (!(val > neg_inf()))
        return val; // no share
    const float d = x - a.m, v = d - x, d_low = (x - (d - v)) - (a.m + v);
    const float z = __fmul_rn(d, t);
    if (!(z > neg_inf()))
        return -z; // beyond fp32
    const float z_low = fmaf(d, t, -z) + d_low * t;
    const float q = val - en.norm, w = q - val, q_low = (val - (q - w)) - (en.norm + w);
    const float g = q - z, y = g - q, g_low = (q - (g - y)) - (z + y);
    const float h = g + log_s, u = h - g, h_low = (g - (h - u)) + (log_s - u);
    return h + ((g_low + h_low) + ((q_low - en.norm_low) - z_low));
}

// The entries of a row, by one warp.
__device__ __forceinline__ bool prepare(Entries &en, const DistillParams &p, int row, const u64 *powers, int lane)
{
    const int32_t *ids = p.ids + (int64_t)row * p.n;
    const float *teacher = p.teacher + (int64_t)row * p.n;
    bool past = false, spoilt = false;
    float best = neg_inf();
    for (int c = 0; c < p.n; c += 32) {
        const int j = c + lane;
        int id = j < p.n ? ids[j] : -1;
        float val = j < p.n ? teacher[j] : neg_inf();
        past |= id >= p.V;
        id = id < p.V ? id : -1;
        // a token's first entry counts
        if ((__match_any_sync(0xffffffffu, id) & ((1u << lane) - 1u)) != 0u)
            id = -1;
        for (int o = 0; o < c; o += 4) {
            const int4 e = *reinterpret_cast<const int4 *>(en.id + o);
            if (id == e.x || id == e.y || id == e.z || id == e.w)
                id = -1;
        }
        if (id >= 0)
            spoilt |= !(val < -neg_inf());
        if (p.rest)
            val = val > 0.0f ? 0.0f : val;
        val = id >= 0 ? val : neg_inf();
        best = fmaxf(best, val);
        en.id[j] = id;
        en.val[j] = val;
        __syncwarp();
    }
    best = warp_max_nan(best);
    const float high = p.rest || best == neg_inf() ? 0.0f : best;
    constexpr float L_HI = 0x1.715476p+0f, L_LO = 0x1.4ae0c0p-26f; // log2 e
    u64 shares = 0ull;
    for (int c = 0; c < p.n; c += 32)
        shares += weight(Scale{high, L_HI, L_LO}, en.val[c + lane], SHARE_SCALE, powers);
    shares = warp_sum64(shares);
    spoilt = __any_sync(0xffffffffu, spoilt);
    if (lane == 0) {
        en.shares = shares;
        const bool plain = p.rest || shares == 0ull || spoilt;
        const float from = plain ? 0.0f : high, sum = plain ? 0.0f : log_fixed(shares, SHARE_SCALE);
        const float norm = from + sum, v = norm - from;
        en.norm = norm;
        en.norm_low = (from - (norm - v)) + (sum - v);
        en.spoilt = spoilt;
    }
    return past;
}

// The row's loss and statistics, by one warp.
template <int W> __device__ __forceinline__ void finish(const Found<W> &f, const Entries &en, const float *x, const DistillParams &p, int row, int parts, int lane)
{
    Numbers a{};
    a.maxima(f, parts, en.spoilt != 0, lane);
    a.sums(f, en, p, parts, lane);
    const float log_s = a.log_s();
    const float log_rest = a.log_rest(log_s);
    float loss = 0.0f;
    for (int c = 0; c < p.n; c += 32) {
        const float val = en.val[c + lane], q = expf((val - en.norm) - en.norm_low);
        if (q > 0.0f && val > neg_inf())
            loss = fmaf(q, a.empty ? -neg_inf() : log_ratio(a, en, log_s, p.inv_t, x[c + lane], val), loss);
    }
    loss = warp_sum(loss);
    if (lane == 0) {
        if (a.q_rest > 0.0f) { // near 1, as p_r may be: by what it lacks of 1
            const float others = (float)en.shares * 0x1p-53f;
            loss = fmaf(a.q_rest, (others < 0.5f ? log1pf(-others) : logf(a.q_rest)) - log_rest, loss);
        }
        const float n = quiet_nan();
        p.loss[row] = a.none ? n : loss;
        if (p.stats != nullptr) {
            float *st = p.stats + (int64_t)row * LORA_DISTILL_STATS;
            st[0] = a.none ? n : a.m;
            st[1] = a.none ? n : log_s;
            st[2] = a.none ? n : log_rest;
            st[3] = a.none ? n : a.q_rest;
            st[4] = a.none ? n : a.total;
            st[5] = a.none ? n : en.norm;
        }
    }
}

// dx of a named element over t g: Q p - q from their logarithms, good where they are near; `gap` is log p - log q. Q is
// far from 1 where the teacher gives little, or more than 1, to tokens beside which nothing is left.
__device__ __forceinline__ float named_slope(float log_p, float log_q, float gap, float total)
{
    const float near = gap + logf(total);
    const float d = near > 0.0f ? -total * expf(log_p) * expm1f(-near) : expf(log_q) * expm1f(near);
    return total == 0.0f ? 0.0f : d;
}

} // namespace

// W warps go through the row; one more prepares the next row's entries and writes
// the last one's loss meanwhile. Four warps, three of whose CTAs' rows of 64 KB an SM holds,
// two for short rows. 8192 x 32000 bf16: the loss 117 us, 4.5 TB/s; with the gradient, reading
// and writing, 217 us, 4.8 TB/s. Neither memory nor issue bounds these (half of DRAM's rate, 54 and 53 % of the
// issue slots, 26 and 28 % of the exponentials' unit): a CTA waits for its own row's copy,
// maxima and sums in turn, and three of them an SM do not hide that. Only the gradient needs the
// row to stay. A row of few vectors is latency: 64 x 32003 f32 9.3 us.
// Long rows meet twice in a cluster: 1000 x 131072 bf16 with gradient and 128 entries 201 us.
template <typename T, int W, bool GRAD>
__global__ void __launch_bounds__(W * 32 + 32, W == 4 ? 4 : 8) distill_kernel(DistillParams p, int parts)
{
    constexpr int E = Vec<T>::E;
    extern __shared__ uint4 slice[];
    __shared__ Shared<W> sm;
    begin_behind();
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = (int)blockIdx.x % parts, team = (int)blockIdx.x / parts, teams = (int)gridDim.x / parts;
    if (tid < 32)
        sm.powers[tid] = POWERS[tid];
    if (tid == 0)
        sm.late = 0;
    const T *logits = static_cast<const T *>(p.logits);
    Row<T, W> r;
    if (warp < W) {
        r.open(slice, sm.bars);
        r.load(logits + (int64_t)team * p.stride, p.V, part, parts);
        if (parts > 1)
            cl.sync();
        else
            __syncthreads();
    }

    if (warp == W) {
        CallCounts counts;
        if (lane == 0)
            counts.open<1>(p.status);
        __syncwarp();
        // the powers are this warp's to wait for, too
        const u64 *powers = POWERS;
        bool past = prepare(sm.entries[0], p, team, powers, lane);
        if (parts > 1)
            cl.sync();
        else
            __syncthreads();
        int last = -1, turn = 0;
        for (int row = team; row < p.M; row += teams, ++turn) {
            if (parts > 1)
                cluster_arrive(); // the maxima are there
            if (last >= 0 && part == 0)
                finish(sm.found[(turn - 1) & 1], sm.entries[(turn - 1) % 3], sm.x[(turn - 1) & 1], p, last, parts, lane);
            if (row + teams < p.M)
                past |= prepare(sm.entries[(turn + 1) % 3], p, row + teams, sm.powers, lane);
            __syncwarp();
            if (parts > 1) {
                cluster_wait();
                cluster_arrive(); // the sums are there
                cluster_wait();
            } else {
                named_bar_sync(BAR_SUM, W * 32 + 32);
            }
            last = row;
        }
        if (part == 0)
            finish(sm.found[(turn - 1) & 1], sm.entries[(turn - 1) % 3], sm.x[(turn - 1) & 1], p, last, parts, lane);
        past = __any_sync(0xffffffffu, past);
        if (lane == 0)
            counts.close((past ? (uint32_t)LORA_FLAG_TOKEN_RANGE : 0u) | (sm.late ? (uint32_t)LORA_FLAG_WAIT_TIMEOUT : 0u), gridDim.x);
        return;
    }

    constexpr float L_HI = 0x1.715476p+0f, L_LO = 0x1.4ae0c0p-26f; // log2 e
    Scale s;
    s.c = __fmul_rn(p.inv_t, L_HI);
    s.c_low = fmaf(p.inv_t, L_HI, -s.c) + p.inv_t * L_LO;
    // where this warp's findings go: one lane for each CTA of the team
    Shared<W> *const told = parts > 1 && lane < parts ? cl.map_shared_rank(&sm, lane) : &sm;
    Shared<W> *const lead = parts > 1 ? cl.map_shared_rank(&sm, 0) : &sm;
    const int place = part * W + warp;
    int turn = 0;
    for (int row = team; row < p.M; row += teams, ++turn) {
        const Entries &en = sm.entries[turn % 3];
        float *const taken = sm.x[turn & 1];
        const float g = GRAD ? p.g[row] : 0.0f;
        r.wait();
        if (row + teams < p.M)
            r.prefetch(logits + (int64_t)(row + teams) * p.stride, p.V);

        // ---- named elements of the warp's run are taken out of the row
        const int e0 = r.first + r.w0 * E, e1 = r.first + r.w1 * E;
        float named_max = neg_inf();
        uint32_t chunks = 0u; // of 32 entries, those of which this lane has one: in few turns, since each lane takes its own
        for (int c = 0; c < p.n; c += 32) {
            const int id = en.id[c + lane];
            const bool mine = id >= max(e0, 0) && id < e1;
            if (mine) {
                T *at = reinterpret_cast<T *>(slice) + (id - r.first);
                const float x = Vec<T>::widen(*at);
                *at = Vec<T>::narrow(neg_inf());
                taken[c + lane] = x;
                if (parts > 1)
                    lead->x[turn & 1][c + lane] = x;
                named_max = max_nan(named_max, x);
            }
            chunks |= mine ? 1u << (c / 32) : 0u;
        }
        const bool any = __any_sync(0xffffffffu, chunks != 0u);
        __syncwarp();

        // ---- maxima
        int group;
        const float own = max_of(r, group), rest_own = warp_top(own);
        if (any)
            named_max = warp_top(named_max);
        if (lane < parts) {
            Found<W> &f = told->found[turn & 1];
            f.rest_max[place] = rest_own;
            f.named_max[place] = named_max;
        }
        __syncwarp();
        if (parts > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            named_bar_sync(BAR_MAX, W * 32);
        }
        Numbers a{};
        a.maxima(sm.found[turn & 1], parts, en.spoilt != 0, lane);

        if (r.late)
            sm.late = 1;
        // ---- sums of the rest and of the named ones, the maxima's own 1 apart
        s.m = a.no_rest || a.none ? 0.0f : a.rest_max;
        u64 rest = 0ull, named = 0ull;
        int equal = 0;
        if (!a.none && !a.no_rest)
            rest = rest_of(r, s, own, group, equal);
        if (!GRAD && row + teams < p.M) // this thread is through with its vectors
            r.load(logits + (int64_t)(row + teams) * p.stride, p.V, part, parts);
        if (!a.none && !a.empty)
            for (uint32_t left = chunks; left != 0u; left &= left - 1u) {
                const float x = taken[(__ffs(left) - 1) * 32 + lane];
                named += x == a.m ? 0ull : weight(Scale{a.m, s.c, s.c_low}, x, SHARE_SCALE, sm.powers);
                equal += x == a.m ? 1 << 20 : 0;
            }
        rest = warp_sum64(rest);
        if (any)
            named = warp_sum64(named);
        equal = __reduce_add_sync(0xffffffffu, equal);
        if (lane < parts) {
            Found<W> &f = told->found[turn & 1];
            f.rest[place] = rest;
            f.named[place] = named;
            f.equal[place] = equal;
        }
        __syncwarp();
        if (parts > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            named_bar_sync(BAR_SUM, W * 32 + 32);
        }
        if (!GRAD)
            continue;

        // ---- the others' slopes: over t g, (Q p_r - q_r) / sum over the rest's softmax, where p_r over its sum is
        // e^below / S
        a.sums(sm.found[turn & 1], en, p, parts, lane);
        const float tg = p.inv_t * g;
        const float slope = a.empty || a.no_rest ? 0.0f : a.none ? quiet_nan()
                            : tg * (a.total * expf(a.below) / (1.0f + a.others) - a.q_rest / (a.rest_equal + a.rest_sum));
        const float shift = s.m;
        T *dx = static_cast<T *>(p.dlogits) + (int64_t)row * p.d_stride;
        const bool zero = a.empty || a.no_rest;
        const f2 nm = make_f2(-shift, -shift), c2 = make_f2(s.c, s.c), k2 = make_f2(slope, slope);
        const bool same = row_lead(dx) == row_lead(logits + (int64_t)row * p.stride);
        if (zero) {
            const int from = max(e0, 0), to = min(e1, p.V);
            for (int i = from + lane; i < to; i += 32)
                dx[i] = Vec<T>::narrow(0.0f);
        } else if (same) { // both rows split into the same vectors
#pragma unroll 2
            for (int v = r.w0 + lane; v < r.w1; v += 32) {
                const int i0 = r.first + v * E;
                float f[E];
                Vec<T>::unpack(r.vec[v], f);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    float a0, a1;
                    split_f2(mul_f2(add_f2(make_f2(f[e], f[e + 1]), nm), c2), a0, a1);
                    split_f2(mul_f2(make_f2(exp2_fast(a0), exp2_fast(a1)), k2), f[e], f[e + 1]);
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
        } else { // a vector of dx lies across two of the row, and may across two runs
            const T *have = reinterpret_cast<const T *>(slice);
            const int from = max(r.first, 0), to = min(r.first + r.count * E, p.V), lead_in = row_lead(dx);
            for (int v = (from + lead_in) / E + tid; v * E - lead_in < to; v += W * 32) {
                const int i0 = v * E - lead_in;
                float f[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = i0 + e;
                    f[e] = i >= from && i < to ? Vec<T>::widen(have[i - r.first]) : neg_inf();
                }
#pragma unroll
                for (int e = 0; e < E; ++e)
                    f[e] = exp2_fast((f[e] - shift) * s.c) * slope;
                if (i0 >= from && i0 + E <= to) {
                    *reinterpret_cast<uint4 *>(dx + i0) = Vec<T>::pack(f);
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (i0 + e >= from && i0 + e < to)
                            dx[i0 + e] = Vec<T>::narrow(f[e]);
                }
            }
        }
        if (!zero && !same)
            named_bar_sync(BAR_ACROSS, W * 32); // over what other warps stored there; the slice is free
        else
            __syncwarp(); // over what the warp stored there
        if (any) {
            const float log_s = a.log_s();
            for (uint32_t left = chunks; left != 0u; left &= left - 1u) {
                const int j = (__ffs(left) - 1) * 32 + lane;
                const float x = taken[j], val = en.val[j];
                const float gap = -log_ratio(a, en, log_s, p.inv_t, x, val);
                float d = tg * named_slope((x - a.m) * p.inv_t - log_s, (val - en.norm) - en.norm_low, gap, a.total);
                d = a.none ? quiet_nan() : a.empty || x == neg_inf() ? 0.0f : d;
                dx[en.id[j]] = Vec<T>::narrow(d);
            }
        }
        if (row + teams < p.M)
            r.load(logits + (int64_t)(row + teams) * p.stride, p.V, part, parts);
    }
    r.close();
}

namespace {

constexpr int DG_THREADS = 256, DG_UNROLL = 4;

// Statistics have log p_r to 2^-24 of itself, which is what p_v / p_r is off by (6e-5 at -256, all of it at -1e9, where
// the others are masked by a finite value). Below this, a row whose rest has a share finds its rest's softmax again, by its first CTA.
constexpr float FAR_REST = -256.0f;

// The whole row of dx, by one CTA: -k times the softmax of the others, `own` for the thread's named element (`id`,
// or -1). dx may be x.
template <typename T> __device__ __noinline__ void far_rest(const T *x, T *dx, int V, int id, float own, float t, float k)
{
    __shared__ float tops[DG_THREADS / 32];
    __shared__ u64 sums[DG_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (dx != x)
        for (int i = tid; i < V; i += DG_THREADS)
            dx[i] = x[i];
    __syncthreads();
    if (id >= 0)
        dx[id] = Vec<T>::narrow(neg_inf());
    __syncthreads();
    float top = neg_inf();
    for (int i = tid; i < V; i += DG_THREADS)
        top = fmaxf(top, Vec<T>::widen(dx[i]));
    top = warp_top(top);
    if (lane == 0)
        tops[warp] = top;
    __syncthreads();
    top = warp_top(tops[lane % (DG_THREADS / 32)]);
    const float c = t * LOG2E, shift = top > neg_inf() ? top : 0.0f;
    u64 sum = 0ull;
    for (int i = tid; i < V; i += DG_THREADS)
        sum += as_fixed(exp2_fast((Vec<T>::widen(dx[i]) - shift) * c), SUM_SCALE);
    sum = warp_sum64(sum);
    if (lane == 0)
        sums[warp] = sum;
    __syncthreads();
    sum = warp_sum64(lane < DG_THREADS / 32 ? sums[lane] : 0ull);
    const float each = sum != 0ull ? -k / ((float)sum * SUM_UNIT) : 0.0f;
    for (int i = tid; i < V; i += DG_THREADS)
        dx[i] = Vec<T>::narrow(exp2_fast((Vec<T>::widen(dx[i]) - shift) * c) * each);
    __syncthreads();
    if (id >= 0)
        dx[id] = Vec<T>::narrow(own);
}

} // namespace

// A CTA takes DG_UNROLL * DG_THREADS vectors of one row of dlogits; named elements
// that lie among them are written over what the pass stored there. 8192 x 32000 bf16 179 us,
// 5.9 TB/s: 68 % of DRAM's rate and 61 % of the issue slots. The gradient of the log probabilities,
// which names one token a row, is at 7.0 TB/s; without the named elements this one was 3 % faster, so most of the
// difference is elsewhere and not explained. Other shapes were slower: eight vectors a thread 225 us,
// two 213, 512 threads 216.
template <typename T, bool REST> __global__ void __launch_bounds__(DG_THREADS, 6) distill_grad_kernel(DistillParams p, int segs)
{
    constexpr int E = Vec<T>::E;
    begin_behind();
    const int row = blockIdx.x / segs, seg = blockIdx.x % segs, tid = threadIdx.x;
    const T *x = static_cast<const T *>(p.logits) + (int64_t)row * p.stride;
    T *dx = static_cast<T *>(p.dlogits) + (int64_t)row * p.d_stride;
    const int lead = row_lead(dx);
    const bool same = row_lead(x) == lead; // both rows split into the same vectors
    const int nvec = (int)(((int64_t)lead + p.V + E - 1) / E);
    const int first = seg * (DG_UNROLL * DG_THREADS), v0 = first + tid;
    uint4 raw[DG_UNROLL];
#pragma unroll
    for (int q = 0; q < DG_UNROLL; ++q) {
        const int v = v0 + q * DG_THREADS, i0 = v * E - lead;
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
    const float *st = p.stats + (int64_t)row * LORA_DISTILL_STATS;
    const float m = st[0], log_s = st[1], log_rest = st[2], q_rest = REST ? st[3] : 0.0f, total = st[4], norm = REST ? 0.0f : st[5];
    const float tg = p.inv_t * p.g[row];
    // The named elements of this segment, an entry a thread (n <= DG_THREADS)
    __shared__ int ids[LORA_MAX_TEACHER];
    int id = -1;
    float xn = 0.0f, val = 0.0f;
    if (tid < p.n) {
        id = p.ids[(int64_t)row * p.n + tid];
        val = p.teacher[(int64_t)row * p.n + tid];
        ids[tid] = id;
    }
    __syncthreads();
    const bool far = REST && q_rest > 0.0f && !(log_rest >= FAR_REST);
    if (id >= 0) {
        const int64_t at = ((int64_t)id + lead) / E;
        if (id >= p.V || (!far && (at < first || at >= first + DG_UNROLL * DG_THREADS)))
            id = -1;
        for (int j = 0; j < tid && id >= 0; ++j)
            id = ids[j] == id ? -1 : id; // a token's first entry counts
        if (id >= 0)
            xn = Vec<T>::widen(x[id]);
        if (REST)
            val = val > 0.0f && val < -neg_inf() ? 0.0f : val;
    }
    if (far || p.dlogits == p.logits)
        __syncthreads(); // every element is read before any is written
    const bool empty = m == neg_inf(), none = !(m == m), no_rest = log_rest == neg_inf();
    auto named = [&] {
        const double log_p = ((double)xn - (double)m) * (double)p.inv_t - (double)log_s;
        const double log_q = (double)val - (double)norm;
        const float d = tg * named_slope((float)log_p, (float)log_q, (float)(log_p - log_q), total);
        return none ? quiet_nan() : xn == neg_inf() ? 0.0f : d;
    };
    if (far) {
        if (seg == 0) // the row is its first CTA's
            far_rest<T>(x, dx, p.V, id, id >= 0 ? named() : 0.0f, p.inv_t, tg * q_rest);
        return;
    }
    const bool zero = empty || (no_rest && !none);
    // Where the rest has no share, its slopes are t g Q p_v, and p_r is not taken apart.
    const float of_rest = q_rest > 0.0f ? log_rest : 0.0f;
    const float slope = none ? quiet_nan() : zero ? 0.0f : tg * (total * expf(of_rest) - q_rest);
    const float c = p.inv_t * LOG2E;
    // 2^a with a = x c - (m c + (log S + log p_r) log2 e), the latter in two parts; rows of huge values take the
    // difference first
    const float mc = m * c, ml = fmaf(m, c, -mc), ls = (log_s + of_rest) * LOG2E;
    const float hi = mc + ls, pt = hi - mc, lo = ((mc - (hi - pt)) + (ls - pt)) + ml;
    const bool huge = !(fabsf(mc) <= 65536.0f);
    const f2 c2 = make_f2(c, c), hi2 = make_f2(-hi, -hi), lo2 = make_f2(-lo, -lo), k2 = make_f2(slope, slope);
    const f2 nm2 = make_f2(-m, -m), ls2 = make_f2(-ls, -ls);
#pragma unroll
    for (int q = 0; q < DG_UNROLL; ++q) {
        const int v = v0 + q * DG_THREADS, i0 = v * E - lead;
        if (v >= nvec)
            break;
        float f[E];
        Vec<T>::unpack(raw[q], f);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const f2 x2 = make_f2(f[e], f[e + 1]);
            const f2 a2 = huge ? add_f2(mul_f2(add_f2(x2, nm2), c2), ls2) : add_f2(fma_f2(x2, c2, hi2), lo2);
            float a0, a1;
            split_f2(a2, a0, a1);
            split_f2(mul_f2(make_f2(exp2_fast(a0), exp2_fast(a1)), k2), f[e], f[e + 1]);
        }
        if (zero) {
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
    __syncthreads(); // over what was stored there
    if (id >= 0)
        dx[id] = Vec<T>::narrow(named());
}

template <typename T, int W, bool GRAD> cudaError_t launch_team(const DistillParams &p, int num_sms, cudaStream_t st)
{
    const TeamPlan t = plan_teams<T, W>(p.M, p.V, num_sms, sizeof(Shared<W>));
    const cudaError_t e = allow_smem<distill_kernel<T, W, GRAD>>();
    if (e != cudaSuccess)
        return e;
    return launch_behind(distill_kernel<T, W, GRAD>, dim3((unsigned)(t.teams * t.parts)), W * 32 + 32, t.smem, (unsigned)t.parts, st, p,
                         t.parts);
}
template <typename T> cudaError_t launch_typed(const DistillParams &p, int num_sms, cudaStream_t st)
{
    if (short_rows<T>(p.M, p.V, num_sms))
        return p.dlogits != nullptr ? launch_team<T, 2, true>(p, num_sms, st) : launch_team<T, 2, false>(p, num_sms, st);
    return p.dlogits != nullptr ? launch_team<T, 4, true>(p, num_sms, st) : launch_team<T, 4, false>(p, num_sms, st);
}

cudaError_t launch_distill(const DistillParams &p, int dtype, int num_sms, cudaStream_t st)
{
    return dtype == LORA_DTYPE_F32 ? launch_typed<float>(p, num_sms, st) : launch_typed<uint16_t>(p, num_sms, st);
}

template <typename T> cudaError_t launch_grad(const DistillParams &p, cudaStream_t st)
{
    // one vector more than V fills, for rows that start inside one
    const int64_t nvec = ((int64_t)p.V + Vec<T>::E - 1) / Vec<T>::E + 1;
    const int segs = (int)((nvec + DG_UNROLL * DG_THREADS - 1) / (DG_UNROLL * DG_THREADS));
    return launch_behind(p.rest ? distill_grad_kernel<T, true> : distill_grad_kernel<T, false>, dim3((unsigned)(p.M * segs)), DG_THREADS, 0,
                         1, st, p, segs);
}

cudaError_t launch_distill_grad(const DistillParams &p, int dtype, cudaStream_t st)
{
    return dtype == LORA_DTYPE_F32 ? launch_grad<float>(p, st) : launch_grad<uint16_t>(p, st);
}

} // namespace rd
