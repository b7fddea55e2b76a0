// A row of logits in shared memory, spread over a team (a CTA, or a cluster of
// them), and exponentials of its elements: fp32 sums over all of them, and single
// weights to about 2^-43 of themselves.
#pragma once
#include <atomic>

#include "logit_rows.cuh"
#include "lora_internal.cuh"

namespace rd {

namespace {

typedef unsigned long long u64;

constexpr int MAX_PARTS = 8;
constexpr int SUM_SCALE = 43; // sums of weights over a vocabulary, below 2^19 elements, are integers of 2^-43
constexpr float SUM_UNIT = 0x1p-43f, SUM_UNITS = 0x1p43f;
constexpr float LEAST = -3.402823466e38f; // the lowest finite value

// Counts that a call's CTAs share, in the words 4 to 13 of its workspace: numbers, each
// with the call's tag above it, that count from 0 wherever they hold another tag;
// and from there on rows that were counted. Every CTA of the call's first kernel
// opens them before it uses them; the epoch that the tag is made of moves on when
// the last CTA of its last kernel has been counted, after all have read it. That CTA
// clears them first: the epoch lies in the workspace too, and where it goes back (memory
// handed out again, a caller that clears the front), counts that stood under a tag
// would pass for the next call's own.
struct CallCounts {
    static constexpr int LISTED = 50; // 64 words
    enum { ENDED = 4, NEXT = 6, OPENED = 8, AGAIN = 10, NEXT_AGAIN = 12, ROWS = 14 };
    uint32_t *st;

    template <int NUMBERS> __device__ __forceinline__ void open(uint32_t *status) // the first of them, by one thread
    {
        st = status;
        const uint32_t tag = status_tag(reinterpret_cast<volatile uint32_t *>(st)[2]);
#pragma unroll
        for (int i = 0; i < NUMBERS; ++i) {
            u64 *w = reinterpret_cast<u64 *>(st + ENDED) + i;
            const u64 seen = *reinterpret_cast<volatile u64 *>(w);
            if ((uint32_t)(seen >> 32) != tag)
                atomicCAS(w, seen, (u64)tag << 32); // fails where another CTA did it
        }
    }
    static __device__ __forceinline__ CallCounts of(uint32_t *status)
    {
        CallCounts c;
        c.st = status;
        return c;
    }
    __device__ __forceinline__ uint32_t add(int word) const { return (uint32_t)atomicAdd(reinterpret_cast<u64 *>(st + word), 1ull); }
    // A row left for a later kernel, once (OPENED) or again (AGAIN): the list has the last of the two.
    __device__ __forceinline__ void left_open(int word, int row) const
    {
        const uint32_t at = add(word);
        if (at < (uint32_t)LISTED)
            st[ROWS + at] = (uint32_t)row;
    }
    __device__ __forceinline__ int count(int word) const { return (int)reinterpret_cast<volatile uint32_t *>(st)[word]; }
    __device__ __forceinline__ int listed(int at) const { return (int)reinterpret_cast<volatile uint32_t *>(st)[ROWS + at]; }
    __device__ __forceinline__ uint32_t next_row() const { return add(NEXT); }
    __device__ __forceinline__ void flag(uint32_t flags) const { atomicOr(reinterpret_cast<u64 *>(st + ENDED), (u64)flags << 24); }
    // The same thread, when its CTA is through: the last of them writes the status word.
    __device__ __forceinline__ void close(uint32_t flags, uint32_t ctas) const
    {
        u64 *w = reinterpret_cast<u64 *>(st + ENDED);
        if (flags != 0u)
            flag(flags);
        const uint32_t was = (uint32_t)atomicAdd(w, 1ull);
        if ((was & 0xFFFFFFu) + 1u == ctas) {
            clear();
            status_begin(st, was >> 24);
        }
    }
    __device__ __forceinline__ void clear() const
    {
#pragma unroll
        for (int word = ENDED; word < ROWS; word += 2)
            *reinterpret_cast<volatile u64 *>(st + word) = 0ull;
    }
    // A call whose kernels could not all be launched: what the first has counted ends here, since nothing moves its epoch on.
    static cudaError_t give_up(cudaError_t e, uint32_t *status, cudaStream_t stream)
    {
        cudaMemsetAsync(status + ENDED, 0, (ROWS - ENDED) * sizeof(uint32_t), stream);
        return e;
    }
};

// 2^(j/32) 2^62, to the nearest integer.
__device__ const u64 POWERS[32] = {
    0x4000000000000000ull, 0x4166c34c5615d0ecull, 0x42d561b3e6243d8aull, 0x444c0740496d4294ull,
    0x45cae0f1f545eb73ull, 0x47521cc5a2e6a9e0ull, 0x48e1e9b9d588e19bull, 0x4a7a77d47f7b84b1ull,
    0x4c1bf828c6dc54b8ull, 0x4dc69cdceaa72a9cull, 0x4f7a993048d088d7ull, 0x513821818624b40cull,
    0x52ff6b54d8a89c75ull, 0x54d0ad5a753e077cull, 0x56ac1f752150a563ull, 0x5891fac0e95612c8ull,
    0x5a827999fcef3242ull, 0x5c7dd7a3b17dcf75ull, 0x5e8451cfac061b5full, 0x6096266533384a2bull,
    0x62b39508aa836d6full, 0x64dcdec3371793d1ull, 0x6712460a8fc24072ull, 0x69540ec8f895722dull,
    0x6ba27e656b4eb57aull, 0x6dfddbcbed791babull, 0x70666f76154a7089ull, 0x72dc8373be41a454ull,
    0x75606373ee921c97ull, 0x77f25ccdee6d7ae6ull, 0x7a92be8a92436616ull, 0x7d41d96db915019dull};

// Bits in the order of the values (-0 as +0); of a NaN they may be any.
__device__ __forceinline__ uint32_t order_bits(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// The largest of the lanes' values, a NaN above all.
__device__ __forceinline__ float warp_top(float v)
{
    return order_value(__reduce_max_sync(0xffffffffu, v == v ? order_bits(v) : 0xffffffffu));
}

__device__ __forceinline__ u64 warp_sum64(u64 v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The row's scale, and what a weight needs of it: a = (x - m) c log2, c = t log2 e as two numbers.
struct Scale {
    float m, c, c_low;
};

// e^{(x - m) t} 2^bits as an integer, within about 2^-43 of itself (and half a
// unit): the exponent as the sum of two fp32 numbers, 2^(j/32) from the table, and
// e^y of the rest, |y| < 0.0109, by its series to y^5.
__device__ __forceinline__ u64 weight(const Scale &s, float x, int bits, const u64 *powers)
{
    const float d = x - s.m;
    const float a = __fmul_rn(d, s.c);
    if (!(a > -63.0f))
        return 0ull;
    const float v = d - x, d_low = (x - (d - v)) - (s.m + v); // x - m = d + d_low
    const float a_low = fmaf(d, s.c, -a) + fmaf(d, s.c_low, d_low * s.c);
    const float j = rintf(a * 32.0f);
    const float r = fmaf(j, -0.03125f, a); // exact
    constexpr float LN2_HI = 0x1.62e430p-1f, LN2_LO = -0x1.05c610p-29f;
    const float y = __fmul_rn(r, LN2_HI);
    const float y_low = fmaf(r, LN2_HI, -y) + fmaf(r, LN2_LO, a_low * LN2_HI);
    const float z = __fmul_rn(y, y), z_low = fmaf(y, y, -z) + 2.0f * y * y_low;
    const float tail = y * z * fmaf(y, fmaf(y, 1.0f / 120.0f, 1.0f / 24.0f), 1.0f / 6.0f);
    const float half = 0.5f * z, h = y + half;
    const float h_low = ((y - h) + half) + (y_low + fmaf(0.5f, z_low, tail));
    const long long q = (long long)(h * 0x1p62f) + (long long)(h_low * 0x1p62f); // (e^y - 1) 2^62
    const int ji = (int)j;
    const u64 base = powers[ji & 31];
    const u64 w = base + (u64)(__mul64hi((long long)base, q) << 2);
    const int sh = 62 - bits - (ji >> 5);
    return sh > 63 ? 0ull : (w + ((1ull << sh) >> 1)) >> sh;
}

// One row as a CTA of its team has it, each warp with a contiguous run of vectors
// of its own: it copies them (one bulk copy, counted on the warp's barrier), and
// nobody else goes through them. The runs are the same wherever a row begins inside a
// vector, since a warp asks for the next row while others are still at theirs.
template <typename T, int W> struct Row { // W warps a CTA
    static constexpr int E = Vec<T>::E;
    uint4 *vec;    // the CTA's vectors
    uint64_t *bar; // the warp's
    uint32_t phase;
    bool late;     // a copy was not there in time
    int lane, warp;
    int into;      // elements before the row in its first vector
    int first;     // index of the first element of vec[0] (negative where the row begins inside a vector)
    int count;     // how many vectors
    int w0, w1;    // this warp's run
    int in0, in1;  // of it, those that the row fills

    __device__ __forceinline__ void open(uint4 *vec_, uint64_t *bars)
    {
        vec = vec_;
        lane = threadIdx.x & 31;
        warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); // as one number a warp
        bar = bars + warp;
        phase = 0u;
        late = false;
        into = -1;
        if (lane == 0) {
            mbar_init(bar, 1);
            fence_barrier_init();
        }
        __syncwarp();
    }
    // Where the row's vectors lie (`parts` is a power of two): as those of the row before where it begins as far
    // into a vector.
    __device__ __forceinline__ void place(int lead, int V, int part, int parts)
    {
        into = lead;
        const int nvec = (lead + V + E - 1) / E, most = (E - 1 + V + E - 1) / E, per = (most + parts - 1) >> (__ffs(parts) - 1);
        const int vb = min(nvec, part * per);
        count = min(nvec, vb + per) - vb;
        const int run = (max(0, min(most, (part + 1) * per) - part * per) + W - 1) / W; // of every row
        first = vb * E - lead;
        w0 = min(count, warp * run);
        w1 = min(count, w0 + run);
        in0 = max(w0, first < 0 ? 1 : 0);
        in1 = max(in0, min(w1, (V - first) / E));
    }
    // Asks for a row; the warp is through with the one that it has. The row's first and last vector may hold elements
    // that are not the row's: those two are not copied in bulk.
    __device__ __forceinline__ void load(const T *x, int V, int part, int parts)
    {
        const int lead = row_lead(x);
        if (lead != into)
            place(lead, V, part, parts);
        if (late)
            return;
        __syncwarp();
        if (lane == 0) {
            fence_proxy_async_smem();
            const uint32_t bytes = (uint32_t)(in1 - in0) * 16u;
            mbar_arrive_expect_tx(bar, bytes);
            if (bytes != 0u)
                bulk_load_1d(vec + in0, x + first + in0 * E, bytes, bar);
        }
        if (in1 - in0 < w1 - w0) {
            if (lane == 0 && w0 < in0 && w0 < w1)
                vec[w0] = load_vec(x, V, -first, w0);
            if (lane == 1 && in1 < w1)
                vec[in1] = load_vec(x, V, -first, in1);
        }
    }
    // It is there, or, for ever after a wait that gave up, nothing more is copied.
    __device__ __forceinline__ void wait()
    {
        if (late)
            return;
        late = __any_sync(0xffffffffu, !mbar_wait(bar, phase));
        phase ^= late ? 0u : 1u;
        __syncwarp(); // the vectors that were not copied in bulk
    }
    // Before the CTA ends: no copy is left on its way.
    __device__ __forceinline__ void close()
    {
        if (late)
            mbar_wait(bar, phase);
    }
    // Another row's vectors of this warp's on their way into L2 (about: it may begin elsewhere in a vector).
    __device__ __forceinline__ void prefetch(const T *x, int V) const
    {
        if (lane == 0 && in1 - in0 > 2)
            bulk_prefetch_l2(x - row_lead(x) + into + first + (in0 + 1) * E, (uint32_t)(in1 - in0 - 2) * 16u);
    }
};

// Parts of a row, each a CTA's share of it in shared memory: enough of them that three
// CTAs a SM hold theirs, and where rows are few, enough CTAs for one a SM.
struct TeamPlan {
    int parts;
    size_t smem; // bytes of a part
    int64_t teams;
};
template <typename T, int W> TeamPlan plan_teams(int M, int V, int num_sms, size_t fixed)
{
    const int64_t nvec = ((int64_t)V + Vec<T>::E - 1) / Vec<T>::E + 1; // one more for a row that begins inside one
    TeamPlan t;
    t.parts = 1;
    while (t.parts < MAX_PARTS &&
           (nvec * 16 / t.parts > (66 << 10) || ((int64_t)M * t.parts < num_sms && nvec >= 2 * t.parts * W * 32)))
        t.parts *= 2;
    t.smem = (size_t)((nvec + t.parts - 1) / t.parts) * 16;
    int resident = (int)((228 << 10) / (t.smem + fixed + 1024)); // 1 KB a CTA is the system's
    resident = resident < 1 ? 1 : resident > (W == 8 ? 3 : 8) ? (W == 8 ? 3 : 8) : resident; // registers
    t.teams = (int64_t)num_sms * resident / t.parts;
    t.teams = M < t.teams ? M : t.teams;
    return t;
}

// Many rows of few vectors: a CTA of two warps a row, of which an SM holds more.
template <typename T> bool short_rows(int M, int V, int num_sms)
{
    return (int64_t)V <= 1024 * Vec<T>::E && M > 3 * num_sms;
}

// A kernel's dynamic shared memory as large as it gets, once a device.
template <auto kernel> cudaError_t allow_smem()
{
    static std::atomic<unsigned long long> done{0ull};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1ull)))
        return e;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (227 << 10) - (int)fa.sharedSizeBytes);
    if (e == cudaSuccess && dev < 64)
        done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

// 2^a of the elements of a vector but those equal to the maximum; how many are.
template <typename T, bool CAREFUL>
__device__ __forceinline__ float vector_rest(const uint4 &raw, const Scale &s, int &equal)
{
    constexpr int E = Vec<T>::E;
    float f[E];
    Vec<T>::unpack(raw, f);
    const f2 nm = make_f2(-s.m, -s.m), c = make_f2(s.c, s.c);
    f2 sum[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        float a0, a1;
        split_f2(mul_f2(add_f2(make_f2(f[e], f[e + 1]), nm), c), a0, a1);
        a0 = exp2_fast(a0);
        a1 = exp2_fast(a1);
        if (CAREFUL) {
            const bool is0 = f[e] == s.m, is1 = f[e + 1] == s.m;
            a0 = is0 ? 0.0f : a0;
            a1 = is1 ? 0.0f : a1;
            equal += is0 + is1;
        }
        sum[e / 2] = make_f2(a0, a1);
    }
#pragma unroll
    for (int w = 1; w < E / 2; w *= 2)
#pragma unroll
        for (int j = 0; j + w < E / 2; j += 2 * w)
            sum[j] = add_f2(sum[j], sum[j + w]);
    float a, b;
    split_f2(sum[0], a, b);
    return a + b;
}

__device__ __forceinline__ u64 as_fixed(float v, int bits) { return (u64)(v * __uint_as_float((uint32_t)(127 + bits) << 23)); }

// The largest of this thread's elements, and the first of the (up to four) vectors, 32 apart, one of which holds it.
template <typename T, int W> __device__ __forceinline__ float max_of(const Row<T, W> &r, int &group)
{
    float m = neg_inf();
    int v = r.w0 + r.lane;
    group = v;
    for (; v + 96 < r.w1; v += 128) {
        const float a = Vec<T>::largest(r.vec[v]), b = Vec<T>::largest(r.vec[v + 32]);
        const float c = Vec<T>::largest(r.vec[v + 64]), d = Vec<T>::largest(r.vec[v + 96]);
        const float g = max_nan(max_nan(a, b), max_nan(c, d));
        group = g > m ? v : group;
        m = max_nan(m, g);
    }
    for (; v < r.w1; v += 32) {
        const float g = Vec<T>::largest(r.vec[v]);
        group = g > m ? v : group;
        m = max_nan(m, g);
    }
    return m;
}

// This thread's fp32 sum of 2^a over its vectors, 2^43 times. Where it has the maximum,
// the vector that holds it is taken by itself, and the maxima in it (`equal`) count
// 1 each beside the sum.
template <typename T, int W> __device__ __forceinline__ u64 rest_of(const Row<T, W> &r, const Scale &s, float mine, int group, int &equal)
{
    u64 sum = 0ull;
    equal = 0;
    int held = -1;
    uint4 kept;
    if (mine == s.m)
        for (int v = group; v < r.w1; v += 32)
            if (Vec<T>::largest(r.vec[v]) == s.m) {
                held = v;
                break;
            }
    if (held >= 0) { // it is there, but for a copy that comes after its wait gave up
        kept = r.vec[held];
        r.vec[held] = empty_vec<T>();
        sum = as_fixed(vector_rest<T, true>(kept, s, equal), SUM_SCALE);
    }
    __syncwarp();
    int none, v = r.w0 + r.lane;
    for (; v + 96 < r.w1; v += 128) {
        const float a = vector_rest<T, false>(r.vec[v], s, none), b = vector_rest<T, false>(r.vec[v + 32], s, none);
        const float c = vector_rest<T, false>(r.vec[v + 64], s, none), d = vector_rest<T, false>(r.vec[v + 96], s, none);
        sum += as_fixed((a + b) + (c + d), SUM_SCALE);
    }
    for (; v < r.w1; v += 32)
        sum += as_fixed(vector_rest<T, false>(r.vec[v], s, none), SUM_SCALE);
    if (held >= 0)
        r.vec[held] = kept;
    return sum;
}

} // namespace

} // namespace rd
