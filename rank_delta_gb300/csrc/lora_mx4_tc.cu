// The projection with a microscaled 4-bit base on the 5th-generation tensor
// cores: y[i, :] = dq(W) x_i + s B_s (A_s x_i) for batches of more than a few
// rows.
//
// A CTA takes 128 features by one tile of up to 256 rows and a part of K.
// The codes come by TMA, 256 k of 128 rows a box; sixteen warps widen them to
// bf16 exactly and store them as the swizzled K-major operand of tcgen05.mma; x
// comes by TMA in the same layout; one thread issues the products into TMEM. The
// weight is widened once for all rows of the tile. With tiles of 256 rows the
// tensor cores bound it (8192x4096x14336: 733 us without adapters, 1.31 PFLOP/s);
// with fewer rows it is the widening and what a call takes in any case, shrink,
// set-up and epilogue (one row of K = 1024: 7.2 us; 64x4096x4096: 16.6 us;
// 256x4096x6144: 28.5 us).
//
// The adapters are more K: s h of the tile's rows (rounded to bf16, as y
// itself is; the sums stay fp32) against the B rows of each slot in the tile,
// a row's columns zero for every slot but its own, into an accumulator of
// their own, which is added to the rows that have an adapter: the others keep
// the base product to the bit.
//
// With few feature tiles K is split over a cluster of CTAs, whose partial
// tiles are summed in part order through distributed shared memory.
#include <cooperative_groups.h>

#include "lora_mx4.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace rd {

namespace cg = cooperative_groups;

namespace {

constexpr int BM = 128;             // features of a tile: the UMMA M
// Three rings between TMA, the widening warps and the products. A stage is SUB
// sub-tiles of 64 k: AS slots of widened weights (16 KB a sub-tile), XS slots of
// tn rows of x (tn 128 bytes), CS steps of codes (256 k of 128 rows, and 16 scale
// bytes a row). Groups of four warps (128 rows) widen, sub-tile m by group m mod
// GROUPS, and drain the accumulators.
//
// The thread that issues the products spends some 100 cycles on each wait and
// more on a commit, which is longer than the products of 64 k take for up to
// about 128 rows: there a stage has two sub-tiles.
template <int SUB_, int AS_, int XS_, int CS_> struct Rings {
    static constexpr int SUB = SUB_, AS = AS_, XS = XS_, CS = CS_;
    static constexpr int GROUPS = SUB == 1 && AS < 4 ? AS : 4, WARPS = GROUPS * 4, THREADS = (WARPS + 4) * 32;
    // A group that waits for its stage's slot has been told, by the wait for its
    // stage before (GROUPS / SUB stages earlier), that the slot's use before the
    // last is through; were that still open, the parity of the last use would
    // not tell the two apart.
    static_assert(AS >= GROUPS / SUB && XS >= AS, "parity of a slot's last use");
};
constexpr int MAX_RING = 16;
constexpr uint32_t CODE_BYTES = BM * 128, SCALE_BYTES = BM * 16;
constexpr uint32_t A_BYTES = BM * 128;
constexpr int MAX_TN = 256;

struct TcShared {
    uint64_t x_full[MAX_RING], x_free[MAX_RING], a_full[MAX_RING], a_free[MAX_RING], c_full[MAX_RING], c_free[MAX_RING];
    uint64_t d_full[MAX_RING], routed, done;
    uint32_t tmem;
    int bad;                          // a wait gave up
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
__device__ __forceinline__ void sts_16(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
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

// umma_bf16 and umma_commit by the lanes with lead != 0.
__device__ __forceinline__ void umma_bf16_by(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.b32 q, %5, 0;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
                 : "memory");
}
__device__ __forceinline__ void umma_commit_by(uint32_t lead, uint64_t *bar)
{
    asm volatile("{\n\t.reg .pred q;\n\t"
                 "setp.ne.b32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
                 "r"(lead)
                 : "memory");
}

// Two blocks of a row, 32 codes each, and their scale bytes -> the row's 128
// bytes of bf16. row_at is where its piece 0 lies: the swizzle's exclusive or
// with the row goes into the address once.
__device__ __forceinline__ void widen_store(const uint4 (&codes)[2], uint32_t s0, uint32_t s1, uint32_t row_at)
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
                o[q] = mul_bf16x2(o[q], f1[b]);
            if (twice) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    o[q] = mul_bf16x2(o[q], f2[b]);
            }
            sts_16(row_at ^ (uint32_t)((b * 4 + j) << 4), make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
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
    constexpr int SUB = RINGS::SUB, AS = RINGS::AS, XS = RINGS::XS, CS = RINGS::CS, GROUPS = RINGS::GROUPS, WIDEN_WARPS = RINGS::WARPS;
    extern __shared__ uint8_t tc_smem_raw[];
    __shared__ TcShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t raw = smem_u32(tc_smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const smem = tc_smem_raw + (base - raw);
    const uint32_t x_bytes = (uint32_t)tn * 128u;
    const uint32_t a_at = base, x_at = base + AS * SUB * A_BYTES, codes_at = x_at + XS * SUB * x_bytes,
                   scales_at = codes_at + CS * CODE_BYTES;
    const int part = blockIdx.x % kparts, f0 = (blockIdx.x / kparts) * BM, t0 = blockIdx.y * tn;
    const int nblk = p.K / 32, nst = (nblk + 1) / 2, nsteps = (nst + 3) / 4; // blocks of 32 k, sub-tiles of 64, steps of 256
    const int j0 = (int)((int64_t)nsteps * part / kparts), j1 = (int)((int64_t)nsteps * (part + 1) / kparts);
    // sub-tiles of the part, whole stages (past K both operands are zeros)
    const int m0 = 4 * j0, mbase = (min(nst, 4 * j1) - m0 + SUB - 1) / SUB * SUB, nbase = mbase / SUB;
    uint32_t cols = 32;
    while ((int)cols < 2 * tn)
        cols *= 2;

    if (tid == 0) {
        for (int s = 0; s < XS; ++s) {
            mbar_init(&sh.x_full[s], 1);
            mbar_init(&sh.x_free[s], 1);
        }
        for (int s = 0; s < AS; ++s) {
            mbar_init(&sh.a_full[s], 4 * SUB); // the groups' warps
            mbar_init(&sh.a_free[s], 1);
            mbar_init(&sh.d_full[s], WIDEN_WARPS * 32);
        }
        for (int s = 0; s < CS; ++s) {
            mbar_init(&sh.c_full[s], 1);
            mbar_init(&sh.c_free[s], 16); // four warps for each of the step's four stages
        }
        mbar_init(&sh.routed, 1);
        mbar_init(&sh.done, 1);
        sh.bad = 0;
        fence_barrier_init();
    }
    if (warp == WIDEN_WARPS + 1)
        tmem_alloc(&sh.tmem, cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

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
        for (int m = group; m < mbase; m += GROUPS) {
            const int j = m >> 2, cs = j % CS, quarter = m & 3;
            wait_or_note(&sh.c_full[cs], (uint32_t)(j / CS) & 1u, &sh.bad);
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
            const int n = m / SUB, s = n % AS, use = n / AS;
            if (use > 0)
                wait_or_note(&sh.a_free[s], (uint32_t)(use - 1) & 1u, &sh.bad);
            __syncwarp();
            widen_store(c, sc & 255u, (sc >> 8) & 255u, a_at + (uint32_t)(s * SUB + m % SUB) * A_BYTES + own);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.a_full[s]);
        }

        // ---- the adapters' operands: 4 SUB segments of 16 ranks a stage, every
        // GROUPS-th by this group
        wait_or_note(&sh.routed, 0, &sh.bad);
        const int q0 = sh.nseg * part / kparts, q1 = sh.nseg * (part + 1) / kparts;
        const int ndelta = __any_sync(0xffffffffu, *reinterpret_cast<volatile int *>(&sh.bad) != 0)
                               ? 0
                               : (q1 - q0 + 4 * SUB - 1) / (4 * SUB);
        const int rows = min(tn, p.M - t0);
        if (ndelta > 0)
            grid_dependency_wait(); // h is complete
        int q = q0 + group, lo = 0; // this group's next segment, and the slot it belongs to
        for (int d = 0; d < ndelta; ++d) {
            const int n = nbase + d, s = n % AS, use = n / AS, xslot = n % XS, xuse = n / XS;
            if (use > 0)
                wait_or_note(&sh.a_free[s], (uint32_t)(use - 1) & 1u, &sh.bad);
            if (xuse > 0)
                wait_or_note(&sh.x_free[xslot], (uint32_t)(xuse - 1) & 1u, &sh.bad);
            for (; q < min(q1, q0 + 4 * SUB * (d + 1)); q += GROUPS) {
                const int j = q - q0 - 4 * SUB * d;
                while (lo + 1 < sh.nslot && sh.seg_start[lo + 1] <= q)
                    ++lo;
                const int r = (q - sh.seg_start[lo]) * 16, slot = sh.slot_id[lo];
                const uint32_t two = r + 8 < p.R ? 16u : 0u, at = a_at + (uint32_t)(s * SUB + (j >> 2)) * A_BYTES,
                               xt = x_at + (uint32_t)(xslot * SUB + (j >> 2)) * x_bytes;
                const uint16_t *b = sh.slot_b[lo] + (size_t)rowi * p.R + r;
                cp16(at + sw128(row, 2 * (j & 3)), b, 16u);
                cp16(at + sw128(row, 2 * (j & 3) + 1), two ? b + 8 : b, two);
                for (int tok = row; tok < tn; tok += 128) { // zeros for the other slots' rows
                    const bool mine = sh.tok_slot[tok] == slot;
                    const uint16_t *h = p.hs + (size_t)(t0 + (mine ? tok : 0)) * p.R + r;
                    cp16(xt + sw128(tok, 2 * (j & 3)), h, mine ? 16u : 0u);
                    cp16(xt + sw128(tok, 2 * (j & 3) + 1), two ? h + 8 : h, mine ? two : 0u);
                }
            }
            cp_async_mbar_arrive_noinc(&sh.d_full[s]); // when this thread's copies have landed
        }
        wait_or_note(&sh.done, 0, &sh.bad);
        __syncwarp();
    } else if (warp == WIDEN_WARPS) {
        // ---- x
        if (lane == 0) {
            prefetch_tmap(&maps.x);
            for (int n = 0; n < nbase; ++n) {
                const int s = n % XS, use = n / XS;
                if (use > 0)
                    wait_or_note(&sh.x_free[s], (uint32_t)(use - 1) & 1u, &sh.bad);
                mbar_arrive_expect_tx(&sh.x_full[s], SUB * x_bytes);
                for (int h = 0; h < SUB; ++h)
                    tma_load_2d(smem + AS * SUB * A_BYTES + (uint32_t)(s * SUB + h) * x_bytes, &maps.x, (m0 + n * SUB + h) * 64,
                                t0, &sh.x_full[s]);
            }
        }
        __syncwarp();
    } else if (warp == WIDEN_WARPS + 1) {
        // ---- products: the whole warp goes along, so that what the instructions
        // take is known to be the same in all lanes; lane 0 issues
        const uint32_t lead = lane == 0 ? 1u : 0u, idesc = idesc_bf16_f32(BM, (uint32_t)tn);
        const uint64_t adesc = sw128_kmajor_desc(a_at), xdesc = sw128_kmajor_desc(x_at);
        auto stage = [&](uint32_t d_tmem, int s, int xslot, int steps, bool first) {
            const uint64_t ad = adesc + (uint64_t)(uint32_t)(s * SUB) * (A_BYTES >> 4);
            const uint64_t xd = xdesc + (uint64_t)((uint32_t)(xslot * SUB) * (x_bytes >> 4));
#pragma unroll
            for (int j = 0; j < 4 * SUB; ++j)
                if (j < steps)
                    umma_bf16_by(lead, d_tmem, ad + (uint64_t)((j >> 2) * (A_BYTES >> 4) + (j & 3) * 2),
                                 xd + (uint64_t)((uint32_t)(j >> 2) * (x_bytes >> 4) + (uint32_t)(j & 3) * 2u), idesc,
                                 first && j == 0 ? 0u : 1u);
            umma_commit_by(lead, &sh.a_free[s]);
            umma_commit_by(lead, &sh.x_free[xslot]);
        };
        int s = 0, xslot = 0;
        uint32_t a_parity = 0, x_parity = 0;
        auto advance = [&] {
            if (++s == AS) {
                s = 0;
                a_parity ^= 1u;
            }
            if (++xslot == XS) {
                xslot = 0;
                x_parity ^= 1u;
            }
        };
        for (int n = 0; n < nbase; ++n) {
            // both polls on their way at once
            const bool x_in = mbar_try_wait(smem_u32(&sh.x_full[xslot]), x_parity), a_in = mbar_try_wait(smem_u32(&sh.a_full[s]), a_parity);
            if (!x_in)
                wait_or_note(&sh.x_full[xslot], x_parity, &sh.bad);
            if (!a_in)
                wait_or_note(&sh.a_full[s], a_parity, &sh.bad);
            tc_fence_after();
            stage(tmem, s, xslot, 4 * SUB, n == 0);
            advance();
        }
        wait_or_note(&sh.routed, 0, &sh.bad);
        const int q0 = sh.nseg * part / kparts, q1 = sh.nseg * (part + 1) / kparts;
        for (int q = q0; q < q1 && !__any_sync(0xffffffffu, *reinterpret_cast<volatile int *>(&sh.bad) != 0); q += 4 * SUB) {
            wait_or_note(&sh.d_full[s], (uint32_t)((q - q0) / (4 * SUB) / AS) & 1u, &sh.bad);
            fence_proxy_async_smem(); // cp.async (generic proxy) wrote both operands
            tc_fence_after();
            stage(tmem + (uint32_t)tn, s, xslot, q1 - q, q == q0);
            advance();
        }
        umma_commit_by(lead, &sh.done);
        __syncwarp();
    } else if (warp == WIDEN_WARPS + 2) {
        // ---- codes and scales
        if (lane == 0) {
            for (int j = 0; 4 * j < mbase; ++j) {
                const int cs = j % CS, use = j / CS;
                if (use > 0)
                    wait_or_note(&sh.c_free[cs], (uint32_t)(use - 1) & 1u, &sh.bad);
                mbar_arrive_expect_tx(&sh.c_full[cs], CODE_BYTES + (maps.scales_ok ? SCALE_BYTES : 0u));
                uint8_t *at = smem + AS * SUB * A_BYTES + XS * SUB * x_bytes;
                tma_load_2d(at + (uint32_t)cs * CODE_BYTES, &maps.codes, (j0 + j) * 128, f0, &sh.c_full[cs]);
                if (maps.scales_ok) // the 16 bytes that hold the step's eight
                    tma_load_2d(at + CS * CODE_BYTES + (uint32_t)cs * SCALE_BYTES, &maps.scales, ((j0 + j) * 8) & ~15, f0,
                                &sh.c_full[cs]);
            }
        }
        __syncwarp();
    } else {
        route_tile(p, sh, t0, tn, lane);
        if (lane == 0)
            mbar_arrive(&sh.routed);
        __syncwarp();
    }

    // ---- the accumulators: each part finishes 128 / kparts features, and gets
    // them from every part in its shared memory, [part][row][features + 4]
    cg::cluster_group cl = cg::this_cluster();
    if (kparts > 1)
        cl.sync(); // every part's products have read their operands
    else
        __syncthreads();
    const int fs = BM / kparts, stride = fs + 4, rows = min(tn, p.M - t0);
    float *const tile = reinterpret_cast<float *>(smem);
    if (warp < WIDEN_WARPS) {
        tc_fence_after();
        const bool adapted = sh.nseg * (part + 1) / kparts > sh.nseg * part / kparts;
        const int f = (warp & 3) * 32 + lane, owner = f / fs;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        float *const to = (kparts > 1 ? cl.map_shared_rank(tile, owner) : tile) + (size_t)part * tn * stride + (f - owner * fs);
        for (int c = warp >> 2; c < tn / 16; c += GROUPS) {
            uint32_t v[16], d[16];
            tmem_ld16_nowait(tmem + lanes + (uint32_t)(c * 16), v);
            if (adapted)
                tmem_ld16_nowait(tmem + lanes + (uint32_t)(tn + c * 16), d);
            const uint32_t on = adapted ? sh.adapted[c >> 1] >> ((c & 1) * 16) : 0u;
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float o = __uint_as_float(v[i]);
                if (on >> i & 1u)
                    o += __uint_as_float(d[i]);
                to[(c * 16 + i) * stride] = o;
            }
        }
    }
    if (kparts > 1)
        cl.sync();
    else
        __syncthreads();
    // ---- the parts' sum, in part order, and one rounding; 8 features of a row at a time
    {
        const int eights = fs / 8, log_eights = 31 - __clz(eights), b0 = part * fs;
        const bool vec = (reinterpret_cast<uintptr_t>(p.y) & 15u) == 0 && p.y_stride % 8 == 0;
#pragma unroll 4
        for (int i = tid; i < rows * eights; i += RINGS::THREADS) {
            const int tok = i >> log_eights, f = (i & (eights - 1)) * 8, feature = f0 + b0 + f;
            float v[8];
            const float4 *src = reinterpret_cast<const float4 *>(tile + tok * stride + f);
            const float4 first = src[0], second = src[1];
            v[0] = first.x; v[1] = first.y; v[2] = first.z; v[3] = first.w;
            v[4] = second.x; v[5] = second.y; v[6] = second.z; v[7] = second.w;
            for (int r = 1; r < kparts; ++r) {
                const float4 *more = src + r * (tn * stride / 4);
                const float4 a = more[0], b = more[1];
                v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
                v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
            }
            uint16_t *y = p.y + (int64_t)(t0 + tok) * p.y_stride + feature;
            if (vec && feature + 8 <= p.N) {
                *reinterpret_cast<uint4 *>(y) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (feature + k < p.N)
                        y[k] = f32_to_bf16_bits(v[k]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == WIDEN_WARPS + 1)
        tmem_dealloc(tmem, cols);
    if (tid == 0 && sh.bad) {
        grid_dependency_wait(); // the call's status is open
        atomicOr(p.status, (uint32_t)LORA_FLAG_WAIT_TIMEOUT);
    }
}

namespace {

template <typename RINGS>
cudaError_t launch(const Mx4ProjParams &p, const Mx4TcPlan &plan, const Mx4TcMaps &maps, cudaStream_t st)
{
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = raise_smem_limit(raised, mx4_tc_kernel<RINGS>, 217 * 1024);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)plan.kparts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.N + BM - 1) / BM * plan.kparts), (unsigned)((p.M + plan.tn - 1) / plan.tn));
    cfg.blockDim = dim3((unsigned)RINGS::THREADS);
    cfg.dynamicSmemBytes = 1024u + RINGS::SUB * (RINGS::AS * A_BYTES + RINGS::XS * (uint32_t)plan.tn * 128u) +
                           RINGS::CS * (CODE_BYTES + SCALE_BYTES);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mx4_tc_kernel<RINGS>, maps, p, plan.tn, plan.kparts);
}

} // namespace

Mx4TcPlan plan_mx4_tc(const Mx4ProjParams &p, int num_sms)
{
    Mx4TcPlan plan;
    const int tiles = (p.M + MAX_TN - 1) / MAX_TN, each = (p.M + tiles - 1) / tiles;
    plan.tn = (each + 15) / 16 * 16;
    const int ctas = (p.N + BM - 1) / BM * tiles, nst = (p.K / 32 + 1) / 2;
    plan.kparts = 1;
    while (plan.kparts < 8 && ctas * plan.kparts * 2 <= num_sms && nst >= 8 * plan.kparts)
        plan.kparts *= 2;
    return plan;
}

cudaError_t launch_mx4_tc(const Mx4ProjParams &p, const Mx4TcPlan &plan, const Mx4TcMaps &maps, cudaStream_t st)
{
    if (plan.tn <= 64)
        return launch<Rings<2, 3, 4, 3>>(p, plan, maps, st); // what fits in 227 KB
    return plan.tn <= 128 ? launch<Rings<2, 2, 3, 3>>(p, plan, maps, st) : launch<Rings<1, 3, 4, 2>>(p, plan, maps, st);
}

} // namespace rd
