// The projection with a microscaled 4-bit base on the 5th-generation tensor
// cores: y[i, :] = dq(W) x_i + s B_s (A_s x_i) for batches of more than a few
// rows.
//
// A CTA takes 128 features by one tile of up to 256 rows and a part of K.
// The codes come by TMA, 256 k of 128 rows a box; sixteen warps widen them to
// bf16 exactly and store them in tensor memory, where tcgen05.mma takes its first
// operand from (a thread has a row there as it has here: no swizzle, no fence, and
// shared memory is left to x); x comes by TMA, and one thread issues the products.
// The weight is widened once for all rows of the tile. With tiles of 256 rows
// the tensor cores and what a tile takes before and after them bound it
// (8192x4096x14336: 598 us, 550 without adapters, 1.75 PFLOP/s; a stage of 64 k
// takes 515 to 555 cycles, its products 512); with fewer rows it is the widening and what a
// call takes in any case, shrink, set-up and epilogue (64x4096x4096: 15.7 us, 10.1
// without adapters). Many adapters in a tile are as much work as the base: each of
// them is multiplied with all rows (512x4096x6144 with 32 of rank 64: 55 us, 28 without).
//
// The adapters are more K: s h of the tile's rows (as two bf16, whose sum is good to
// 2^-17; the sums stay fp32) against the B rows of each slot in the tile,
// a row's columns zero for every slot but its own, into an accumulator of
// their own, which is added to the rows that have an adapter: the others keep
// the base product to the bit. Where that sum is not finite, the row's part is
// computed alone, so that no adapter reaches another's rows.
//
// With few feature tiles K is split over a cluster of CTAs, whose partial
// tiles are exchanged through distributed shared memory: each part sums and writes
// some of the features.
#include <algorithm>

#include "lora_mx4.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace rd {

namespace {

constexpr int BM = 128;             // features of a tile: the UMMA M
constexpr int TEAMS = 2;            // of the widening warps, that copy the adapters' rows
// 16-rank segments of the adapters in a sub-tile of 64 k: of h the first bf16 of SEGS
// segments, then the second; of B the segments alone, once for both.
constexpr int SEGS = 2;
// The rings between TMA, the widening warps and the products. A stage is SUB
// sub-tiles of 64 k. There are S of them: widened weights in tensor memory (32
// columns a sub-tile, from column A_COL on) and tn rows of x in shared memory (tn
// 128 bytes a sub-tile), with one barrier for "both are there" and one for "the
// products are through". CS steps of codes (256 k of 128 rows, and 16 scale
// bytes a row) and DS slots of the adapters' rows come besides, S of
// them with the codes' place once those are widened. Groups of four
// warps (128 rows) widen, sub-tile m by group m mod GROUPS, and drain the
// accumulators.
//
// 64 k take 2 tn cycles of the tensor cores. Up to about 128 rows that is less
// than a stage's waits and commits, so a stage has two sub-tiles there
// (64x4096x14336: 6 % longer with one); above, two would leave two stages
// only (256x4096x14336: 19 % longer with two).
//
// Up to 128 rows the widened weights lie behind both accumulators; above it
// they take the columns of the adapters' accumulator (ALIAS), which is not written
// before the last base product has read them.
template <int MAX_ROWS_, int SUB_, int S_, int CS_, int DS_, int A_COL_, bool ALIAS_> struct Rings {
    static constexpr int MAX_ROWS = MAX_ROWS_; // of a tile
    static constexpr int SUB = SUB_, S = S_, CS = CS_, DS = DS_, A_COL = A_COL_;
    static constexpr bool ALIAS = ALIAS_;
    static constexpr int GROUPS = 4, WARPS = GROUPS * 4, THREADS = (WARPS + 4) * 32;
    // A group that waits for its stage's slot has been told, by the wait for its
    // stage before (GROUPS / SUB stages earlier), that the slot's use before the
    // last is through; were that still open, the parity of the last use would
    // not tell the two apart.
    // (The adapters' stages: the group that copies to stage d, of team d mod TEAMS, has
    // widened for stage d - 4 / SUB or a later one, as bases are whole steps.)
    static_assert(S >= GROUPS / SUB && S >= TEAMS, "parity of a slot's last use");
    static_assert(DS + CS / SUB >= S, "slots of the adapters' rows: one a stage");
    static_assert(A_COL + S * SUB * 32 <= 512, "tensor memory");
};
constexpr int MAX_RING = 16, MAX_KPARTS = 8;
constexpr uint32_t CODE_BYTES = BM * 128, SCALE_BYTES = BM * 16;
constexpr uint32_t A_BYTES = BM * 128;
constexpr int MAX_TN = 256;

struct TcShared {
    uint64_t full[MAX_RING], free[MAX_RING], c_full[MAX_RING], c_free[MAX_RING], d_full[MAX_RING], routed, base_done, done, joined;
    uint32_t tmem;
    int bad;                          // a wait gave up
    int verdict;                      // whether the adapters are taken: 0 not decided, 1, 2 not
    int x_asked, codes_asked;         // stages of x and steps of codes that were asked for
    int nseg;
    uint32_t present[MAX_BUCKETS / 32];
    int16_t tok_slot[MAX_TN];         // the row's slot, -1: no delta
    uint32_t adapted[MAX_TN / 32];    // bit of a row: it has a delta
    int16_t slot_id[MAX_TN];          // distinct slots of the tile, ascending
    int seg_start[MAX_TN + 1];        // their first 16-rank segment
    int nslot;
    const uint16_t *slot_b[MAX_TN];
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 lds_16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_2(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}
// Byte offset of 16-byte piece c (0..7) of row r in a swizzled 128-byte-row tile.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// umma_bf16 with A in tensor memory: 128 lanes, two k a column.
__device__ __forceinline__ void umma_bf16_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}
// The shared-memory address of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// `bytes` (a multiple of 16) from this CTA's shared memory to another's, whose barrier they complete on.
__device__ __forceinline__ void copy_to_cluster(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "r"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// Features that each of `kparts` parts of K finishes (the last has what is left).
__host__ __device__ constexpr int part_features(int kparts) { return (BM / 8 + kparts - 1) / kparts * 8; }
__host__ __device__ constexpr int part_owns(int kparts, int part)
{
    const int fs = part_features(kparts), left = BM - part * fs;
    return left < 0 ? 0 : left < fs ? left : fs;
}

// An adapter's part of y over segments q0 .. q1 of the tile, row tok and feature
// f, once more by itself: the zeros that keep a slot's B from the other slots'
// rows make a NaN of an infinity or a NaN in it.
__device__ __noinline__ float delta_alone(const Mx4ProjParams &p, const TcShared &sh, int t0, int tok, int f, int q0, int q1)
{
    int i = 0;
    while (i + 1 < sh.nslot && sh.slot_id[i] != sh.tok_slot[tok])
        ++i;
    const int begin = max(q0, sh.seg_start[i]) - sh.seg_start[i], end = min(q1, sh.seg_start[i + 1]) - sh.seg_start[i];
    const uint16_t *b = sh.slot_b[i] + (size_t)min(f, p.N - 1) * p.R;
    const size_t h = (size_t)(t0 + tok) * p.R;
    float sum = 0.0f;
    for (int r = begin * 16; r < min(end * 16, p.R); ++r)
        sum = fmaf(bf_lo(p.hs[h + r]) + bf_lo(p.ls[h + r]), bf_lo(b[r]), sum);
    return sum;
}

// 16 lanes x 16 columns as four 8 x 8 fragments: thread t has columns 2 (t % 4)
// and the next of lane t / 4 in r[0], r[1], of lane t / 4 + 8 in r[2], r[3], and
// of the next eight columns in r[4..7]. Valid after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
// Four 8 x 8 matrices of 16-bit values, transposed; lane l has the address of
// row l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
// 32 columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                 "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
                 "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
                 "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two blocks of a row, 32 codes each, and their scale bytes -> 64 k in bf16.
__device__ __forceinline__ void widen(const uint4 (&codes)[2], uint32_t s0, uint32_t s1, uint32_t (&out)[32])
{
    uint32_t f1[2] = {mx4_factor(s0), mx4_factor(s1)}, f2[2] = {0u, 0u};
    const bool twice = __any_sync(0xffffffffu, s0 > MX4_ONE_FACTOR || s1 > MX4_ONE_FACTOR);
    if (twice) {
        mx4_factors(s0, f1[0], f2[0]);
        mx4_factors(s1, f1[1], f2[1]);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint32_t w[4] = {codes[b].x, codes[b].y, codes[b].z, codes[b].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t o[4];
            mx4_unpack8(w[j], o);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                out[b * 16 + j * 4 + q] = mul_bf16x2(o[q], f1[b]);
        }
    }
    if (twice) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            out[i] = mul_bf16x2(out[i], f2[i / 16]);
    }
}

// Eight bf16 values to y, of which `left` are wanted (0 or less: none), by one
// store where y is 16-byte aligned (`vec`).
__device__ __forceinline__ void store_8(uint16_t *y, uint4 v, int left, bool vec)
{
    if (vec && left >= 8) {
        *reinterpret_cast<uint4 *>(y) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < left)
            y[k] = (uint16_t)(w[k >> 1] >> (k & 1) * 16);
}

// The tile's rows and slots, by one warp: each row's slot, the distinct slots
// in ascending order with their B and their 16-rank segments.
__device__ __forceinline__ void route_tile(const Mx4ProjParams &p, TcShared &sh, int t0, int tn, int lane)
{
    sh.present[lane] = 0u;
    __syncwarp();
    for (int i0 = 0; i0 < tn; i0 += 32) {
        const int i = i0 + lane;
        int slot = -1;
        if (i < tn && t0 + i < p.M) {
            const int s = p.seq_slot[t0 + i];
            if (slot_info(p.tab, s, p.L).on) {
                slot = s;
                atomicOr(&sh.present[s >> 5], 1u << (s & 31));
            }
        }
        sh.tok_slot[i] = (int16_t)slot;
        __syncwarp();
        const uint32_t on = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0)
            sh.adapted[i0 >> 5] = on;
    }
    __syncwarp();
    const uint32_t w = sh.present[lane];
    int segs = 0;
    for (uint32_t b = w; b != 0u; b &= b - 1)
        segs += (p.tab.rank_table[lane * 32 + __ffs(b) - 1] + 15) / 16;
    int slots_before = __popc(w), segs_before = segs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, slots_before, o), b = __shfl_up_sync(0xffffffffu, segs_before, o);
        if (lane >= o) {
            slots_before += a;
            segs_before += b;
        }
    }
    if (lane == 31) {
        sh.nslot = slots_before;
        sh.nseg = segs_before;
        sh.seg_start[slots_before] = segs_before;
    }
    slots_before -= __popc(w);
    segs_before -= segs;
    for (uint32_t b = w; b != 0u; b &= b - 1) {
        const int s = lane * 32 + __ffs(b) - 1;
        sh.slot_id[slots_before] = (int16_t)s;
        sh.slot_b[slots_before] = p.tab.b_table[s];
        sh.seg_start[slots_before] = segs_before;
        segs_before += (p.tab.rank_table[s] + 15) / 16;
        ++slots_before;
    }
    __syncwarp();
}

} // namespace

template <typename RINGS>
__global__ void __launch_bounds__(RINGS::THREADS, 1)
    mx4_tc_kernel(const __grid_constant__ Mx4TcMaps maps, const __grid_constant__ Mx4ProjParams p, int tn, int kparts)
{
    constexpr int SUB = RINGS::SUB, S = RINGS::S, CS = RINGS::CS, DS = RINGS::DS, GROUPS = RINGS::GROUPS, WIDEN_WARPS = RINGS::WARPS;
    extern __shared__ uint8_t tc_smem_raw[];
    __shared__ TcShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t raw = smem_u32(tc_smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const smem = tc_smem_raw + (base - raw);
    const uint32_t x_bytes = (uint32_t)tn * 128u;
    const uint32_t d_at = base, x_at = base + DS * SUB * A_BYTES, codes_at = x_at + S * SUB * x_bytes,
                   scales_at = codes_at + CS * CODE_BYTES;
    const int part = blockIdx.x % kparts, f0 = (blockIdx.x / kparts) * BM, t0 = blockIdx.y * tn;
    const int nblk = p.K / 32, nst = (nblk + 1) / 2, nsteps = (nst + 3) / 4; // blocks of 32 k, sub-tiles of 64, steps of 256
    const int j0 = (int)((int64_t)nsteps * part / kparts), j1 = (int)((int64_t)nsteps * (part + 1) / kparts);
    // sub-tiles of the part: whole steps (past K both operands are zeros)
    const int m0 = 4 * j0, mbase = 4 * (j1 - j0), nbase = mbase / SUB;
    constexpr uint32_t cols = 512; // no second CTA fits on the SM by its shared memory

    // the loads of a stage of x, and of a step of codes and scales
    auto load_x = [&](int n) {
        const int s = n % S;
        mbar_arrive_expect_tx(&sh.full[s], SUB * x_bytes);
        for (int h = 0; h < SUB; ++h)
            tma_load_2d(smem + DS * SUB * A_BYTES + (uint32_t)(s * SUB + h) * x_bytes, &maps.x, (m0 + n * SUB + h) * 64, t0,
                        &sh.full[s]);
    };
    auto load_codes = [&](int j) {
        const int cs = j % CS;
        uint8_t *at = smem + DS * SUB * A_BYTES + S * SUB * x_bytes;
        mbar_arrive_expect_tx(&sh.c_full[cs], CODE_BYTES + (maps.scales_ok ? SCALE_BYTES : 0u));
        tma_load_2d(at + (uint32_t)cs * CODE_BYTES, &maps.codes, (j0 + j) * 128, f0, &sh.c_full[cs]);
        if (maps.scales_ok) // the 16 bytes that hold the step's eight
            tma_load_2d(at + CS * CODE_BYTES + (uint32_t)cs * SCALE_BYTES, &maps.scales, ((j0 + j) * 8) & ~15, f0, &sh.c_full[cs]);
    };

    // The first loads are on their way before anything else is set up.
    if (warp == WIDEN_WARPS + 2 && elected()) {
        prefetch_tmap(&maps.codes);
        prefetch_tmap(&maps.x);
        for (int s = 0; s < S; ++s) {
            mbar_init(&sh.full[s], 1 + 4 * SUB + (p.never > 1)); // x, and the groups' warps
            mbar_init(&sh.free[s], 1);
        }
        for (int s = 0; s < S; ++s)
            mbar_init(&sh.d_full[s], WIDEN_WARPS / TEAMS * 32 + (p.never == 1));
        for (int s = 0; s < CS; ++s) {
            mbar_init(&sh.c_full[s], 1);
            mbar_init(&sh.c_free[s], 16); // four warps for each of the step's four stages
        }
        mbar_init(&sh.routed, 1);
        mbar_init(&sh.base_done, 1);
        mbar_init(&sh.done, 1);
        mbar_init(&sh.joined, 1);
        sh.bad = sh.verdict = 0;
        fence_barrier_init();
        if (kparts > 1 && part_owns(kparts, part) > 0)
            mbar_arrive_expect_tx(&sh.joined, (uint32_t)((kparts - 1) * part_owns(kparts, part) * (tn + 1)) * 4u);
        for (int j = 0; j < CS && j < j1 - j0; ++j)
            load_codes(j);
        for (int n = 0; n < S && n < nbase; ++n)
            load_x(n);
    }
    if (warp == WIDEN_WARPS + 1)
        tmem_alloc(&sh.tmem, cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    auto d_slot = [&](int s) { return s < DS ? d_at + (uint32_t)(s * SUB) * A_BYTES : codes_at + (uint32_t)((s - DS) * SUB) * A_BYTES; };
    // stage n's products are through (stage n - S is known to be)
    auto stage_free = [&](int n) { return wait_or_note(&sh.free[n % S], (uint32_t)(n / S) & 1u, &sh.bad, p.wait_ns); };
    auto warp_stage_free = [&](int n) { return warp_wait(&sh.free[n % S], (uint32_t)(n / S) & 1u, &sh.bad, p.wait_ns); };
    // A role leaves its loop where a wait gives up, and what it left is seen to at the end.
    int m = warp >> 2;       // a widening warp's next sub-tile
    bool adapters = false;   // the widening warps': the adapters are taken
    if (warp < WIDEN_WARPS) {
        // ---- widen: every GROUPS-th sub-tile
        const int group = warp >> 2, row = (warp & 3) * 32 + lane;
        const int rowi = min(f0 + row, p.N - 1); // rows past N repeat the last; their sums are dropped
        const uint8_t *srow = p.scales + (size_t)rowi * nblk;
        auto byte_scales = [&](int m) { // rows of scales that TMA cannot take
            const int b0 = (m0 + m) * 2;
            return (b0 < nblk ? (uint32_t)__ldg(srow + b0) : 0u) | (b0 + 1 < nblk ? (uint32_t)__ldg(srow + b0 + 1) << 8 : 0u);
        };
        uint32_t sc_next = !maps.scales_ok && group < mbase ? byte_scales(group) : 0u;
        const uint32_t own = sw128(row, 0);
        bool ok = true;
        for (; m < mbase; m += GROUPS) {
            const int j = m >> 2, cs = j % CS, quarter = m & 3;
            if (!(ok = warp_wait(&sh.c_full[cs], (uint32_t)(j / CS) & 1u, &sh.bad, p.wait_ns)))
                break;
            const uint32_t at = codes_at + (uint32_t)cs * CODE_BYTES;
            const uint4 c[2] = {lds_16((at + own) ^ (uint32_t)(quarter << 5)), lds_16((at + own) ^ (uint32_t)(quarter << 5 | 16))};
            uint32_t sc = sc_next;
            if (maps.scales_ok)
                sc = lds_2(scales_at + (uint32_t)cs * SCALE_BYTES + row * 16 + ((m0 + m) * 2 & 15));
            else if (m + GROUPS < mbase)
                sc_next = byte_scales(m + GROUPS);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.c_free[cs]);
            const int n = m / SUB, s = n % S;
            if (n >= S && !(ok = warp_stage_free(n - S)))
                break;
            tc_fence_after();
            uint32_t out[32];
            widen(c, sc & 255u, (sc >> 8) & 255u, out);
            tmem_st32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(RINGS::A_COL + (s * SUB + m % SUB) * 32), out);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.full[s]);
        }

        // ---- the adapters' operands: SEGS SUB segments of 16 ranks a stage. Eight
        // lanes copy a row's 128 bytes of h in a sub-tile, four a row's 64 of B, so a warp's
        // copy meets 8 pieces of memory (a row a lane, 32: 64x4096x14336 took 10 % longer)
        ok = ok && warp_wait(&sh.routed, 0, &sh.bad, p.wait_ns);
        // The warps meet at a barrier below, so all of them take the answer of the first to
        // get here. Where it is yes, the routing was seen to be complete.
        int verdict = 0;
        if (lane == 0) {
            __threadfence_block();
            verdict = atomicCAS(&sh.verdict, 0, ok ? 1 : 2);
            if (verdict == 0)
                verdict = ok ? 1 : 2;
            __threadfence_block();
        }
        adapters = __shfl_sync(0xffffffffu, verdict, 0) == 1;
        __syncwarp();
        const int q0 = adapters ? sh.nseg * part / kparts : 0, q1 = adapters ? sh.nseg * (part + 1) / kparts : 0;
        const int ndelta = (q1 - q0 + SEGS * SUB - 1) / (SEGS * SUB);
        // The warps work in teams, a stage each: finding its slot and waiting take
        // as long as the copies (256x4096x14336: 2 % longer with all on every stage).
        constexpr int TEAM_WARPS = WIDEN_WARPS / TEAMS;
        constexpr int SUB_WARPS = TEAM_WARPS / SUB, ROWS = SUB_WARPS * 4; // that copy a sub-tile, rows at a time
        const int team = warp / TEAM_WARPS, sub = warp % TEAM_WARPS / SUB_WARPS, piece = lane & 7, half = piece >> 2,
                  first = (warp % SUB_WARPS) * 4 + (lane >> 3);
        const int own_seg = sub * SEGS + (piece >> 1 & 1); // of a stage
        constexpr int AT_ONCE = RINGS::MAX_ROWS / ROWS, B_AT_ONCE = BM / ROWS / 2;
        size_t b_row[B_AT_ONCE]; // element offsets of the rows this thread copies
#pragma unroll
        for (int i = 0; i < B_AT_ONCE; ++i)
            b_row[i] = (size_t)min(f0 + first + (2 * i + half) * ROWS, p.N - 1) * p.R;
        int h_slot[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
            h_slot[i] = adapters && first + i * ROWS < tn ? sh.tok_slot[first + i * ROWS] : -1;
        // rows ROWS further are swizzled alike
        const uint32_t into = sw128(first, piece), b_into = sw128(first, piece & 3) + (uint32_t)(half * ROWS * 128);
        const uint16_t *const plane = half == 0 ? p.hs : p.ls;
        // the slot of this thread's segment, the lo-th, its segments, and the slot that
        // had the stage's place before
        int lo = -1, begin = 0, end = 0, slot = -1, lo_before = -1, end_before = 0, before = -1;
        const uint16_t *slot_b = nullptr;
        auto find = [&](int q) {
            if (q >= end) { // another slot
                do {
                    begin = end;
                    end = sh.seg_start[++lo + 1];
                } while (q >= end);
                slot = sh.slot_id[lo];
                slot_b = sh.slot_b[lo];
            }
            return (q - begin) * 16 + (piece & 1) * 8; // the rank
        };
        auto copy_b = [&](int s, int r) {
            const uint32_t at = d_slot(s) + (uint32_t)sub * A_BYTES + b_into;
            const uint16_t *b = slot_b + (r < p.R ? r : 0);
#pragma unroll
            for (int i = 0; i < B_AT_ONCE; ++i)
                cp16(at + (uint32_t)(2 * i * ROWS * 128), b + b_row[i], r < p.R ? 16u : 0u); // else zeros
        };
        // B of the stages that have their places from the start, or from when all codes
        // are widened, is copied while h is waited for
        static_assert(DS >= TEAMS && S <= 2 * TEAMS, "a team's first stage, and one more");
        int rank0 = 0, rank1 = 0, slot0 = -1;
        const int q_first = q0 + SEGS * SUB * team + own_seg, q_second = q_first + SEGS * SUB * TEAMS;
        if (ok && team < ndelta && q_first < q1) {
            rank0 = find(q_first);
            slot0 = slot;
            copy_b(team, rank0);
        }
        if (ndelta > DS) // the further places are where the codes were
            named_bar_sync(5u, WIDEN_WARPS * 32);
        if (ok && team + TEAMS < min(ndelta, S) && q_second < q1) {
            rank1 = find(q_second);
            copy_b(team + TEAMS, rank1);
        }
        if (ndelta > 0)
            grid_dependency_wait(); // h is complete
        for (int d = team; ok && d < ndelta; d += TEAMS) {
            const int n = nbase + d, s = d % S, xslot = n % S;
            if (n >= S && !(ok = warp_stage_free(n - S)))
                break;
            const int q = q0 + SEGS * SUB * d + own_seg;
            if (q < q1) {
                int r = d == team ? rank0 : rank1;
                if (d >= min(team + 2 * TEAMS, S)) {
                    r = find(q);
                    copy_b(s, r);
                }
                const int now = d == team ? slot0 : slot;
                // rows of x that are not the slot's are zeros: all of a slot at first, then
                // those that the stage S before had
                if (d >= S && q - SEGS * SUB * S >= end_before) {
                    do
                        end_before = sh.seg_start[++lo_before + 1];
                    while (q - SEGS * SUB * S >= end_before);
                    before = sh.slot_id[lo_before];
                }
                const uint32_t xt = x_at + (uint32_t)(xslot * SUB + sub) * x_bytes + into, have = r < p.R ? 16u : 0u;
                const uint16_t *h = plane + (size_t)(t0 + first) * p.R + (have ? r : 0);
#pragma unroll
                for (int i = 0; i < AT_ONCE; ++i)
                    if (first + i * ROWS < tn) {
                        const bool mine = h_slot[i] == now;
                        if (mine || d < S || h_slot[i] == before)
                            cp16(xt + (uint32_t)(i * ROWS * 128), mine ? h + i * ROWS * p.R : p.hs, mine ? have : 0u);
                    }
            }
            cp_async_mbar_arrive_noinc(&sh.d_full[s]); // when this thread's copies have landed
        }
        wait_or_note(&sh.done, 0, &sh.bad, p.wait_ns, false); // the products end whether or not a wait gave up
        __syncwarp();
    } else if (warp == WIDEN_WARPS) {
        // ---- x
        if (elected()) {
            int n = S;
            for (; n < nbase && stage_free(n - S); ++n)
                load_x(n);
            sh.x_asked = min(n, nbase);
        }
        __syncwarp();
    } else if (warp == WIDEN_WARPS + 1) {
        // ---- products
        const uint32_t idesc = idesc_bf16_f32(BM, (uint32_t)tn);
        const uint64_t xdesc = sw128_kmajor_desc(x_at);
        const uint32_t widened = tmem + RINGS::A_COL, delta = tmem + (uint32_t)(RINGS::ALIAS ? MAX_TN : tn);
        int s = 0;
        uint32_t parity = 0;
        auto x_of = [&] { return xdesc + (uint64_t)((uint32_t)(s * SUB) * (x_bytes >> 4)); };
        auto next = [&] {
            if (++s == S) {
                s = 0;
                parity ^= 1u;
            }
        };
        bool ok = true;
        for (int n = 0; n < nbase; ++n) {
            if (!(ok = warp_wait(&sh.full[s], parity, &sh.bad, p.wait_ns)))
                break;
            __syncwarp();
            tc_fence_after();
            const uint64_t xd = x_of();
            if (elected()) {
#pragma unroll
                for (int j = 0; j < 4 * SUB; ++j)
                    umma_bf16_tmem(tmem, widened + (uint32_t)(s * SUB * 32 + j * 8),
                                   xd + (uint64_t)((uint32_t)(j >> 2) * (x_bytes >> 4) + (uint32_t)(j & 3) * 2u), idesc,
                                   n == 0 && j == 0 ? 0u : 1u);
                umma_commit(&sh.free[s]);
            }
            __syncwarp();
            next();
        }
        ok = ok && warp_wait(&sh.routed, 0, &sh.bad, p.wait_ns);
        const int q0 = ok ? sh.nseg * part / kparts : 0, q1 = ok ? sh.nseg * (part + 1) / kparts : 0;
        if (RINGS::ALIAS && q1 > q0) {
            __syncwarp();
            if (elected())
                umma_commit(&sh.base_done);
            __syncwarp();
            ok = warp_wait(&sh.base_done, 0, &sh.bad, p.wait_ns);
            tc_fence_after();
        }
        for (int q = q0, d = 0; ok && q < q1; q += SEGS * SUB, ++d) {
            const int ds = d % S;
            if (!(ok = warp_wait(&sh.d_full[ds], (uint32_t)(d / S) & 1u, &sh.bad, p.wait_ns)))
                break;
            __syncwarp();
            fence_proxy_async_smem(); // cp.async (generic proxy) wrote both operands
            tc_fence_after();
            const uint64_t dd = sw128_kmajor_desc(d_slot(ds)), xd = x_of();
            if (elected()) {
#pragma unroll
                for (int j = 0; j < 4 * SUB; ++j) // both parts of h against the same segment of B
                    if ((j >> 2) * SEGS + (j & 1) < q1 - q)
                        umma_bf16(delta, dd + (uint64_t)((j >> 2) * (A_BYTES >> 4) + (j & 1) * 2),
                                  xd + (uint64_t)((uint32_t)(j >> 2) * (x_bytes >> 4) + (uint32_t)(j & 3) * 2u), idesc,
                                  d == 0 && j == 0 ? 0u : 1u);
                umma_commit(&sh.free[s]);
            }
            __syncwarp();
            next();
        }
        if (elected())
            umma_commit(&sh.done);
        __syncwarp();
    } else if (warp == WIDEN_WARPS + 2) {
        // ---- codes and scales
        if (elected()) {
            int j = CS;
            for (; j < j1 - j0 && wait_or_note(&sh.c_free[j % CS], (uint32_t)(j / CS - 1) & 1u, &sh.bad, p.wait_ns); ++j)
                load_codes(j);
            sh.codes_asked = min(j, j1 - j0);
        }
        __syncwarp();
    } else {
        route_tile(p, sh, t0, tn, lane);
        if (lane == 0)
            mbar_arrive(&sh.routed);
        grid_dependency_wait(); // a call is not over before its shrink is
        __syncwarp();
    }

    // Where a wait gave up: everything on its way ends (with the same limit) before the
    // CTA does. The stages whose x was asked for get the arrivals that the widening
    // warps still owe them. Whole CTA, behind a barrier that all waits lie before.
    auto unwind = [&] {
        if (warp < WIDEN_WARPS) {
            cp_async_wait_all();
            if (lane == 0)
                for (; m < mbase && m / SUB < sh.x_asked; m += GROUPS)
                    mbar_arrive(&sh.full[m / SUB % S]);
        }
        __syncthreads();
        if (tid == 0) {
            for (int n = max(0, sh.x_asked - S); n < sh.x_asked; ++n)
                mbar_wait(&sh.full[n % S], (uint32_t)(n / S) & 1u, p.wait_ns);
            for (int j = max(0, sh.codes_asked - CS); j < sh.codes_asked; ++j)
                mbar_wait(&sh.c_full[j % CS], (uint32_t)(j / CS) & 1u, p.wait_ns);
            mbar_wait(&sh.done, 0, p.wait_ns); // the products
            grid_dependency_wait();            // the call's status is open
            atomicOr(p.status, (uint32_t)LORA_FLAG_WAIT_TIMEOUT);
        }
        __syncthreads();
    };
    const int rows = min(tn, p.M - t0);
    const bool vec = (reinterpret_cast<uintptr_t>(p.y) & 15u) == 0 && p.y_stride % 8 == 0;
    const uint32_t delta_col = (uint32_t)(RINGS::ALIAS ? MAX_TN : tn);
    if (kparts == 1) {
        // ---- the accumulators, turned by stmatrix into rows of 128 features in
        // bf16, 272 bytes apart in shared memory, which every product has left;
        // a group of four warps has 16 rows at a time, every GROUPS-th. (Through
        // fp32 a tile of 256 rows took 8100 cycles.)
        if (warp < WIDEN_WARPS) {
            constexpr uint32_t Y_ROW = BM * 2 + 16;
            const int group = warp >> 2;
            const bool adapted = adapters && sh.nseg > 0;
            const uint32_t quad = (uint32_t)(warp & 3) * 32;
            // the lane's row of the four 8 x 8 matrices of a store: 8 features of a batch row
            const uint32_t to = base + (uint32_t)((lane >> 4) * 8 + (lane & 7)) * Y_ROW + (quad + (uint32_t)(lane >> 3 & 1) * 8) * 2;
            tc_fence_after();
            for (int c = group; c < tn / 16; c += GROUPS) {
                uint32_t v[2][8], d[2][8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t at = tmem + ((quad + (uint32_t)h * 16) << 16) + (uint32_t)(c * 16);
                    tmem_ld_16x16(at, v[h]);
                    if (adapted)
                        tmem_ld_16x16(at + delta_col, d[h]);
                }
                const uint32_t on = adapted ? sh.adapted[c >> 1] >> ((c & 1) * 16 + (lane & 3) * 2) : 0u;
                tmem_wait_ld();
                if (adapted) {
                    float probe = 0.0f; // NaN if a delta is not finite
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        probe = fmaf(__uint_as_float(d[j >> 3][j & 7]), 0.0f, probe);
                    if (probe != probe) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (on >> ((j >> 2 & 1) * 8 + (j & 1)) & 1u && isnan(__uint_as_float(d[j >> 3][j & 7])))
                                d[j >> 3][j & 7] = __float_as_uint(
                                    delta_alone(p, sh, t0, c * 16 + (j >> 2 & 1) * 8 + (lane & 3) * 2 + (j & 1),
                                                f0 + (int)quad + (j >> 3) * 16 + (lane >> 2) + (j >> 1 & 1) * 8, 0, sh.nseg));
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) { // rows 2 (lane % 4) and the next of 8: the first 8, features 0 and 8; the second
                        float a = __uint_as_float(v[h][2 * q]), b = __uint_as_float(v[h][2 * q + 1]);
                        if (on >> (q >> 1) * 8 & 1u)
                            a += __uint_as_float(d[h][2 * q]);
                        if (on >> (q >> 1) * 8 & 2u)
                            b += __uint_as_float(d[h][2 * q + 1]);
                        o[q] = pack2(a, b);
                    }
                    stmatrix_x4_trans(to + (uint32_t)(c * 16) * Y_ROW + (uint32_t)h * 32, o);
                }
            }
            named_bar_sync(1u + (uint32_t)group, 128);
            if (!vec) { // a feature a thread: a warp's stores lie in one piece
                const int f = tid & 127;
                if (f0 + f < p.N)
                    for (int c = group; c < tn / 16; c += GROUPS)
#pragma unroll 8
                        for (int tok = c * 16; tok < min(c * 16 + 16, rows); ++tok)
                            p.y[(int64_t)(t0 + tok) * p.y_stride + f0 + f] = (uint16_t)lds_2(base + (uint32_t)tok * Y_ROW + (uint32_t)f * 2);
            } else {
                for (int i = tid & 127; i < tn / GROUPS * 16 + 256; i += 128) {
                    const int tok = ((i >> 8) * GROUPS + group) * 16 + (i >> 4 & 15), f = (i & 15) * 8, feature = f0 + f;
                    if (tok >= rows)
                        break;
                    const uint4 o = lds_16(base + (uint32_t)tok * Y_ROW + (uint32_t)f * 2);
                    store_8(p.y + (int64_t)(t0 + tok) * p.y_stride + feature, o, p.N - feature, vec);
                }
            }
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (sh.bad)
            unwind();
        if (warp == WIDEN_WARPS + 1)
            tmem_dealloc(tmem, cols);
        return;
    }

    // ---- the accumulators, [feature][row + 1] floats in shared memory. Each part
    // finishes fs features: it gets the others' sums of them as one bulk copy from
    // each, once its own products have left their rings. (The cluster's
    // barriers order no memory: the copies complete on a barrier of their own.)
    const int fs = part_features(kparts), own = part_owns(kparts, part), stride = tn + 1;
    const uint32_t chunk = (uint32_t)(fs * stride) * 4u, recv = base + (uint32_t)(BM * stride) * 4u;
    cluster_arrive();
    if (warp < WIDEN_WARPS) {
        tc_fence_after();
        const bool adapted = adapters && sh.nseg * (part + 1) / kparts > sh.nseg * part / kparts;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        float *const to = reinterpret_cast<float *>(smem) + ((warp & 3) * 32 + lane) * stride;
        for (int c = warp >> 2; c < tn / 16; c += GROUPS) {
            uint32_t v[16], d[16];
            tmem_ld16_nowait(tmem + lanes + (uint32_t)(c * 16), v);
            if (adapted)
                tmem_ld16_nowait(tmem + lanes + delta_col + (uint32_t)(c * 16), d);
            const uint32_t on = adapted ? sh.adapted[c >> 1] >> ((c & 1) * 16) : 0u;
            tmem_wait_ld();
            if (adapted) {
                float probe = 0.0f; // NaN if a delta is not finite
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    probe = fmaf(__uint_as_float(d[i]), 0.0f, probe);
                if (probe != probe) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (on >> i & 1u && isnan(__uint_as_float(d[i])))
                            d[i] = __float_as_uint(delta_alone(p, sh, t0, c * 16 + i, f0 + (warp & 3) * 32 + lane,
                                                               sh.nseg * part / kparts, sh.nseg * (part + 1) / kparts));
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float o = __uint_as_float(v[i]);
                if (on >> i & 1u)
                    o += __uint_as_float(d[i]);
                to[c * 16 + i] = o;
            }
        }
        fence_proxy_async_smem();
    }
    __syncthreads();
    cluster_wait();
    if (warp == WIDEN_WARPS && lane < kparts && lane != part && part_owns(kparts, lane) > 0)
        copy_to_cluster(cluster_addr(recv + (uint32_t)(part - (part > lane)) * chunk, (uint32_t)lane), base + (uint32_t)lane * chunk,
                        (uint32_t)(part_owns(kparts, lane) * stride) * 4u, cluster_addr(smem_u32(&sh.joined), (uint32_t)lane));
    __syncwarp();
    // ---- the parts' sum, in part order, and one rounding; 8 features of a row at a time
    if (own > 0)
        wait_or_note(&sh.joined, 0, &sh.bad, p.wait_ns, false); // so do the copies come
    __syncwarp();
    cluster_arrive(); // this part has its copies
    {
        const int eights = own / 8;
        const float *const tile = reinterpret_cast<const float *>(smem);
        for (int i = tid; i < rows * eights; i += RINGS::THREADS) {
            const int tok = i / eights, u = i - tok * eights, feature = f0 + part * fs + u * 8;
            float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            for (int r = 0; r < kparts; ++r) {
                const int at = r == part ? part * fs : BM + (r - (r > part)) * fs;
                const float *src = tile + (at + u * 8) * stride + tok;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] += src[k * stride];
            }
            store_8(p.y + (int64_t)(t0 + tok) * p.y_stride + feature,
                    make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])), p.N - feature, vec);
        }
    }
    cluster_wait(); // every part has its copies, which read the others' shared memory
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sh.bad)
        unwind();
    if (warp == WIDEN_WARPS + 1)
        tmem_dealloc(tmem, cols);
}

namespace {

constexpr uint32_t SMEM_LIMIT = 217 * 1024; // besides TcShared
// The rings, and later the exchange.
template <typename RINGS> uint32_t smem_bytes(int tn, int kparts)
{
    const uint32_t rings = RINGS::SUB * (RINGS::DS * A_BYTES + RINGS::S * (uint32_t)tn * 128u) + RINGS::CS * (CODE_BYTES + SCALE_BYTES);
    const uint32_t exchange = kparts > 1 ? (uint32_t)((BM + (kparts - 1) * part_features(kparts)) * (tn + 1)) * 4u : 0u;
    return 1024u + (rings > exchange ? rings : exchange);
}

// The cluster of the kernel's grid, and that it may begin before the call's shrink is through.
struct TcLaunch {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg;
    template <typename RINGS> cudaError_t fill(int tn, int kparts, dim3 grid, cudaStream_t st)
    {
        static std::atomic<uint64_t> raised{0};
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)kparts;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3((unsigned)RINGS::THREADS);
        cfg.dynamicSmemBytes = smem_bytes<RINGS>(tn, kparts);
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return raise_smem_limit(raised, mx4_tc_kernel<RINGS>, (int)SMEM_LIMIT);
    }
};

// How many clusters of `kparts` CTAs the current device runs at a time: its SMs come
// in groups that a cluster does not cross. Asked once a device; an answer that could
// not be had (0) is asked for again.
constexpr int MAX_DEVICES = 64;
template <typename RINGS> int clusters_at_once(int kparts, int num_sms)
{
    static std::atomic<int> known[MAX_DEVICES][MAX_KPARTS + 1];
    int dev = -1, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) {
        (void)cudaGetLastError();
        return 0;
    }
    if ((n = known[dev][kparts].load()) > 0)
        return n;
    TcLaunch l;
    if (l.fill<RINGS>(16, kparts, dim3((unsigned)(kparts * num_sms)), nullptr) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, mx4_tc_kernel<RINGS>, &l.cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    known[dev][kparts].store(n);
    return n;
}

template <typename RINGS>
cudaError_t launch(const Mx4ProjParams &p, const Mx4TcPlan &plan, const Mx4TcMaps &maps, cudaStream_t st)
{
    TcLaunch l;
    const cudaError_t e = l.fill<RINGS>(plan.tn, plan.kparts,
                                        dim3((unsigned)((p.N + BM - 1) / BM * plan.kparts), (unsigned)((p.M + plan.tn - 1) / plan.tn)), st);
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&l.cfg, mx4_tc_kernel<RINGS>, maps, p, plan.tn, plan.kparts);
}

// Whether clusters of k parts for all tiles run at once, and their exchange fits.
template <typename RINGS> bool fits(int tn, int k, int64_t ctas, int num_sms)
{
    return smem_bytes<RINGS>(tn, k) <= SMEM_LIMIT && clusters_at_once<RINGS>(k, num_sms) >= ctas;
}

// What fits in 227 KB of shared memory and 512 columns of tensor memory.
using Rings64 = Rings<64, 2, 4, 4, 2, 128, false>;
using Rings128 = Rings<128, 2, 3, 3, 2, 256, false>;
using Rings256 = Rings<256, 1, 4, 2, 2, 256, true>;

} // namespace

// The tiles' rows and the parts of K, by an estimate of the cycles of the CTAs that
// an SM runs one after another: set-up, what 64 k take (the widening up to 64
// rows, the products from some 170 on), and the epilogue, with the exchange if
// there is one. Measured where it decides, 16 adapters of rank 64:
// 256x4096x4096 26.0 us as 256 rows in two parts, 22.9 as twice 128;
// 512x4096x6144 with 32 adapters 57.4 us as twice 256, 54.8 as three times 176.
// Where the fewest tiles are more CTAs than SMs it is no guide to heights that differ
// by little: the shrink's CTAs take SMs from the first wave, and tiles that begin in the
// middle of an adapter's run of rows meet more of them. Only tiles of up to 256 and of
// up to 128 rows are compared there. Us with adapters, these and any height by the estimate:
//   rows       1100       1536        2048        4096        6000
//   N  4096    54.6 54.5  64.4  63.0  63.4  76.4  112.7 126.3 165.2 169.3
//   N  6144    54.2 56.6  63.9  63.8  81.3  85.2  155.8 160.4 216.9 214.5
//   N 14336   105.7 105.8 131.8 142.8 170.9 170.8
Mx4TcPlan plan_mx4_tc(const Mx4ProjParams &p, int num_sms)
{
    const int ftiles = (p.N + BM - 1) / BM, nst = (p.K / 32 + 1) / 2, nsteps = (nst + 3) / 4;
    Mx4TcPlan plan{0, 1};
    int64_t least = 0;
    const int fewest = (p.M + MAX_TN - 1) / MAX_TN;
    const bool waves = (int64_t)ftiles * fewest > num_sms;
    const int last = waves ? std::min((p.M + 127) / 128, 65535) : 4 * fewest;
    for (int t = fewest; t <= last; t = waves && t < last ? last : t + 1) {
        const int each = (p.M + t - 1) / t, tn = (each + 15) / 16 * 16;
        const int64_t ctas = (int64_t)ftiles * ((p.M + tn - 1) / tn);
        const int sub = tn <= 128 ? 335 + (tn > 64 ? (tn - 64) * 7 / 8 : 0) : 2 * tn + 5 > 390 ? 2 * tn + 5 : 390;
        for (int k = 1; k <= MAX_KPARTS && k <= nsteps && (k == 1 || ctas * k <= num_sms); ++k) {
            const int64_t waves = (ctas * k + num_sms - 1) / num_sms;
            const int64_t cost = waves * (4000 + (int64_t)((nsteps + k - 1) / k) * 4 * sub + (k > 1 ? 2700 + 28 * tn : 600 + 15 * tn));
            if ((plan.tn == 0 || cost < least) &&
                (k == 1 || (tn <= 64    ? fits<Rings64>(tn, k, ctas, num_sms)
                            : tn <= 128 ? fits<Rings128>(tn, k, ctas, num_sms)
                                        : fits<Rings256>(tn, k, ctas, num_sms)))) {
                least = cost;
                plan.tn = tn;
                plan.kparts = k;
            }
        }
        if (tn <= 16)
            break;
    }
    return plan;
}

cudaError_t launch_mx4_tc(const Mx4ProjParams &p, const Mx4TcPlan &plan, const Mx4TcMaps &maps, cudaStream_t st)
{
    return plan.tn <= 64    ? launch<Rings64>(p, plan, maps, st)
           : plan.tn <= 128 ? launch<Rings128>(p, plan, maps, st)
                            : launch<Rings256>(p, plan, maps, st);
}

} // namespace rd
