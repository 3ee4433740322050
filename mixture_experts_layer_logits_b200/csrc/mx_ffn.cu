// mx_ffn.cu -- products grouped by expert of E4M3 token rows with E2M1 weights (both in
// microscaled blocks of 32 with E8M0 scales), alone and as the two products of the
// expert FFN, on block-scaled tcgen05 tensor cores:
//   D[f, j] = sum_b 2^(sw[f, b] + sa[j, b] - 254) sum_{i in block b} w[f, i] a[j, i]
// in fp32.  Products of codes and their power-of-two scales are exact, so only the
// fp32 sums round.
//
// Two launches of one persistent, warp-specialised kernel make the FFN:
//   MODE 0  act[p, f] = MX(silu(gate) * up) of x[rows[p] / k] with w13[e] rows f and I + f
//   MODE 1  y[rows[p] or p, f] = w[e] row f dotted with act (or any E4M3 rows) [p]
//
// The MMA's M = 128 rows are weight rows and its N columns the token rows of one
// expert, rounded up to 16 per tile: few tokens cost few columns, and a ragged group
// costs at most 15 padded ones.  MODE 0's 128 weight rows are 64 gate rows and their
// 64 up rows.
//
// Warp roles: 0 TMA; 1 TMEM and MMA issue; 2-3 scales; 4-11 epilogue; MODE 0: 12-15
// gather of token rows.
//   - Token rows: MODE 1 loads them by TMA with the weights; MODE 0 gathers x rows with
//     16-byte cp.async copies straight to their swizzled places.  (26 gather4 TMA loads a
//     stage, one per lane, issue too slowly: prefill's w13 took 1.70 ms instead of 0.97.)
//   - Weights: TMA unpacks the 4-bit codes to the byte-wide slots that a mixed
//     E2M1 x E4M3 MMA reads, so HBM and L2 move half a byte an element.
//   - Scales: a K tile of 128 has 4 scale bytes per row.  They are copied 4 bytes at
//     a time (cp.async) from the row-major scale matrices into the 512-byte layout
//     that tcgen05.cp spreads over tensor memory (row r at 16 (r % 32) + 4 (r / 32)).
//     Each ring stage has its own scale columns in tensor memory, so a stage's copy
//     never waits for another stage's MMAs.
//   - Tiles are derived from expert_offsets by every CTA itself (a prefix sum in
//     shared memory), so there is no tile list and no launch for one.
// Every mbarrier wait is bounded (mbar_wait); on a timeout the kernel records the
// error word, stops issuing, drains what it issued and frees TMEM.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gemm_common.cuh"
#include "kernels.h"
#include "mx_common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

using gemm::named_bar_or;
using gemm::named_bar_sync;
using gemm::silu_mul;

constexpr int kBM = 128;                  // weight rows per tile (MMA M)
constexpr int kBK = 128;                  // K elements per stage: one 128-byte swizzle row
constexpr int kATile = kBM * kBK;         // bytes in shared memory (one per element)
constexpr int kATxBytes = kATile / 2;     // an unpacking TMA load counts its packed bytes
constexpr int kMaxExperts = 1024;
constexpr int kScaleWarps = 2, kGatherWarps = 4, kEpiWarps = 8;
constexpr int kScaleWarp0 = 2, kEpiWarp0 = 4, kGatherWarp0 = 12;
constexpr int kMaxStages = 12;

// Instruction descriptor of kind::mxf8f6f4: E2M1 A (code 5), E4M3 B (code 0), both
// K-major, E8M0 scales.
__device__ __forceinline__ uint32_t idesc_mx(int M, int N)
{
    return (5u << 7) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}

// Its bits that select the scale byte of K block kb, 0..3, for B and A.
__device__ __forceinline__ constexpr uint32_t idesc_kb(int kb)
{
    return ((uint32_t)kb << 4) | ((uint32_t)kb << 29);
}

// CG: CTAs that work on one MMA (cta_group::1 or ::2).
template <int CG>
__device__ __forceinline__ void umma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate)
{
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, "
            "[%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, "
            "[%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// Shared-memory descriptor of 512 bytes of scales: 32 rows of 16 bytes, no swizzle,
// groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem)
{
    return (uint64_t)((smem >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(128 >> 4) << 32) |
           ((uint64_t)1 << 46);
}

// Copies them to 4 TMEM columns, the same 32 lanes' worth in every lane quarter.
// Ordered before later MMAs of this thread.
// With CG = 2 each of the two CTAs copies from its own shared memory to its own TMEM.
template <int CG>
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc)
{
    if constexpr (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                     : "memory");
}

// Arrive on `bar` (with CG = 2: on the barrier at this address in both CTAs) when every
// tensor instruction issued so far by this thread is done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar)
{
    if constexpr (CG == 1)
        umma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
            "[%0], %1;" ::"r"(smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_acquire(uint32_t* dst, uint32_t cols)
{
    if constexpr (CG == 1) {
        tmem_alloc(dst, cols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(dst)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CG>
__device__ __forceinline__ void tmem_release(uint32_t taddr, uint32_t cols)
{
    if constexpr (CG == 1)
        tmem_dealloc(taddr, cols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
                     : "memory");
}

// 16 TMEM lanes x 8 columns: lane i gets columns 2 (i % 4) and the next of TMEM lanes i / 4
// (r[0], r[1]) and i / 4 + 8 (r[2], r[3]).
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t* r)
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
}

// Four 8x8 matrices of 16-bit elements, transposed: lane i's register m holds rows 2 (i % 4)
// and the next of column i / 4 of matrix m, and its address is that of row i % 8 of
// matrix i / 8.
__device__ __forceinline__ void store_matrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                                      uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\t"
        "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrive on the barrier that lies at this address in CTA 0 of the cluster.  It carries
// only the fact.  What it stands for is in the arriving CTA: scales in its shared
// memory, written and fenced towards the async proxy before, which the tensor core of
// that CTA's own SM reads; or its TMEM, read out before tcgen05.wait::ld.  So the default
// release (CTA scope) is enough.  A release at cluster scope waits for the L2: 1200
// cycles a stage, prefill 2.66 ms instead of 1.56.
__device__ __forceinline__ void arrive_leader(uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// Address of the same shared-memory location in CTA 0 of the cluster.
__device__ __forceinline__ uint32_t in_leader(const void* p)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}

// 2D TMA load of a box at (c, row) into this CTA's shared memory whose bytes count on
// `bar`.  CG = 2: `bar` may lie in the other CTA of the pair.
template <int CG>
__device__ __forceinline__ void tma_box(uint32_t dst, const void* tmap, uint32_t bar, int c, int row,
                                        uint64_t policy)
{
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c), "r"(row), "l"(policy)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            ".cta_group::2.L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c), "r"(row), "l"(policy)
            : "memory");
}

// mbar_wait for a barrier that the other CTA of the cluster arrives on.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity,
                                                  volatile int* abort)
{
    uint64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((n & 255u) == 0) {
            if (*abort) return false;
            const uint64_t t = globaltimer_ns();
            if (!t0) t0 = t;
            if (t - t0 > 2000000000ull) return false;
        }
    }
}

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// One lane of a converged warp, the same one every time.  The loops of the TMA and
// MMA warps run in all 32 lanes and only the issue is the elected lane's: the
// descriptors then stay in uniform registers, which the tensor instructions take
// their operands from (a loop inside `if (lane == 0)` took 60 cycles to issue one MMA).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// n / d and n % d for 0 <= n < 2^31 by a multiplication with m = floor(2^32 / d) + 1
// (d = 1: m = 0).  The product can be one too large where n d is large; that is put right.
__device__ __forceinline__ int div_by(int n, int d, uint32_t m)
{
    int q = d == 1 ? n : (int)__umulhi((uint32_t)n, m);
    if (q * d > n) --q;
    return q;
}

// NT: the most token rows of a tile (the MMA's N).
template <int MODE, int NT, int CG>
struct Cfg {
    static constexpr int kThreads = 32 * (MODE == 0 ? kGatherWarp0 + kGatherWarps : kGatherWarp0);
    static constexpr int kBRows = NT / CG;                       // token rows in one CTA's B tile
    static constexpr int kBTile = kBRows * kBK;
    static constexpr int kSfbCols = 4 * ((NT + 127) / 128);      // TMEM columns of B's scales
    static constexpr int kSfCols = 4 + kSfbCols;
    static constexpr int kSfBytes = kSfCols * 128;
    static constexpr int kStageBytes = (kATile + kBTile + kSfBytes + 1023) & ~1023;
    // epilogue: 8 warps x 2 buffers, MODE 0 of 4 columns x 32 lanes of fp32, MODE 1 of 8
    // token rows x 32 bf16
    static constexpr int kStaging = 8192;
    static constexpr int kTables = 2 * (kMaxExperts + 1) * 4 + 8 + 128;
    static constexpr int kAux = 512;
    static constexpr int kFixed = 1024 + kStaging + kTables + kAux;
    static constexpr int kNBuf = NT <= 64 ? 4 : 2;               // accumulators in flight
    static constexpr int kSfCol0 = kNBuf * NT;                   // first scale column
    static constexpr int kStagesSmem = (232448 - kFixed) / kStageBytes;
    static constexpr int kStagesTmem = (512 - kSfCol0) / kSfCols;
    static constexpr int kStagesRaw = kStagesSmem < kStagesTmem ? kStagesSmem : kStagesTmem;
    static constexpr int kStages = kStagesRaw > kMaxStages ? kMaxStages : kStagesRaw;
    static constexpr int kSmem = kFixed + kStages * kStageBytes;
    static constexpr int kUsedCols = kSfCol0 + kStages * kSfCols;
    static constexpr int kTmemCols = kUsedCols <= 128 ? 128 : kUsedCols <= 256 ? 256 : 512;
    static constexpr int kGroupCols = NT / 2;                    // token columns per epilogue group
    static constexpr int kGIters = (kBRows * 8 + kGatherWarps * 32 - 1) / (kGatherWarps * 32);
    static constexpr int kSIters = (NT + kScaleWarps * 32 - 1) / (kScaleWarps * 32);
    static constexpr int kFeatures = CG * (MODE == 0 ? 64 : 128);  // output features per unit
    static_assert(NT % 16 == 0 && NT >= 16 && NT <= 256, "MMA N tile");
    static_assert(kStages >= 2 && kUsedCols <= 512 && kSmem <= 232448, "resources");
};

struct Aux {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t tfull[4];
    uint64_t tempty[4];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int warp_sum[16];
};

// One tile of a group: `rows` token rows from `row`, the feature block `fb` of `expert`.
struct Unit {
    int expert, fb, row, rows;
};

template <int MODE, int NT, int CG>
__global__ void __launch_bounds__(Cfg<MODE, NT, CG>::kThreads, 1)
    mx_grouped_kernel(const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_a, const MxArgs g)
{
    using C = Cfg<MODE, NT, CG>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t* staging = ring + C::kStages * C::kStageBytes;
    Aux* aux = reinterpret_cast<Aux*>(staging + C::kStaging);
    static_assert(sizeof(Aux) <= C::kAux, "aux area");
    int* first = reinterpret_cast<int*>(staging + C::kStaging + C::kAux);  // [E + 1] tiles before e
    int* start = first + kMaxExperts + 1;                                  // [E + 1] rows before e

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            // the expect_tx, and one arrival per scale warp and per gather warp (CG = 2:
            // CTA 0's barrier is the one that counts, for both CTAs)
            mbar_init(&aux->full[s], 1 + CG * (kScaleWarps + (MODE == 0 ? kGatherWarps : 0)));
            mbar_init(&aux->empty[s], 1);
        }
        for (int b = 0; b < C::kNBuf; ++b) {
            mbar_init(&aux->tfull[b], 1);
            mbar_init(&aux->tempty[b], CG * kEpiWarps);
        }
        mbar_init(&aux->drain, 1);
        aux->abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_w);
        if (MODE == 1) tma_prefetch_desc(&tm_a);
    }
    if (warp == 1) {
        tmem_acquire<CG>(&aux->tmem_base, C::kTmemCols);
    }
    // The second product of the FFN (g.early) takes only act from the launch before it;
    // expert_offsets, rows and weights were complete before that launch passed its own
    // wait, so the tables and the first weight tiles need not wait for it.
    if (!g.early) pdl_wait();
    pdl_launch_dependents();

    // tiles before each expert (exclusive prefix sums), offsets clamped to 0 .. R and
    // ascending, so that no offset leads outside the operands
    {
        constexpr int kPer = (kMaxExperts + C::kThreads - 1) / C::kThreads;
        int tiles[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x * kPer + i;
            tiles[i] = 0;
            if (e < g.E) {
                const int a = min(max(__ldcg(g.offsets + e), 0), g.R);
                const int b = min(max(__ldcg(g.offsets + e + 1), a), g.R);
                start[e] = a;
                if (e == g.E - 1) start[g.E] = b;
                tiles[i] = (b - a + NT - 1) / NT;
            }
            sum += tiles[i];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) aux->warp_sum[warp] = incl;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        int before = incl - sum;
        for (int w = 0; w < warp; ++w) before += aux->warp_sum[w];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x * kPer + i;
            if (e < g.E) first[e] = before;
            before += tiles[i];
            if (e == g.E - 1) first[g.E] = before;
        }
        if constexpr (CG == 2)
            cluster_sync();  // barriers initialised and TMEM allocated in both CTAs
        else
            __syncthreads();
    }
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int unit0 = (int)blockIdx.x / CG, stride = (int)gridDim.x / CG;
    const uint32_t tmem_base = aux->tmem_base;
    volatile int* abort_flag = &aux->abort;
    auto flag_error = [&] {
        atomicExch(g.err, kDeviceErrorMagic);
        aux->abort = 1;
    };

    const int fbs = g.fb_count;
    const int units = first[g.E] * fbs;
    const int num_kt = g.K / kBK;
    // unit u: experts in order; within one, feature block major and tile minor, so the
    // tiles that share a weight block run at the same time on neighbouring CTAs and
    // share it in L2.  A group of c rows in t tiles is cut evenly (to 16 rows).
    // All 32 lanes decode together; `e` is the expert of this warp's unit before (a
    // CTA's units ascend, so the search starts there, 32 experts at a time).
    auto decode = [&](int u, int& e) {
        const int rest = div_by(u, fbs, g.fb_magic);
        for (;;) {  // to the last e with first[e] <= rest
            const int at = e + 1 + lane;
            const uint32_t past = __ballot_sync(0xffffffffu, at > g.E || first[min(at, g.E)] > rest);
            if (past) {
                e += __ffs(past) - 1;
                break;
            }
            e += 32;
        }
        const int local = u - first[e] * fbs, count = first[e + 1] - first[e];
        const int rows = start[e + 1] - start[e];
        Unit t;
        t.expert = e;
        t.fb = local;
        t.row = start[e];
        t.rows = rows;
        if (count > 1) {
            const int per = ((rows + count - 1) / count + 15) & ~15;
            t.fb = local / count;
            const int at = (local - t.fb * count) * per;
            t.row += at;
            t.rows = min(per, rows - at);
        }
        return t;
    };
    // first output feature of this CTA's part of a unit
    auto first_feature = [&](const Unit& t) {
        return t.fb * C::kFeatures + (int)rank * (C::kFeatures / CG);
    };
    // first weight row of its tile, of the [E * rows, K] weight matrix; MODE 0's up rows
    // are N further on.  MODE 1: a pair's second tile may begin past N; it then
    // reads the first instead, and none of it is stored.
    auto weight_row = [&](const Unit& t) {
        const int f = first_feature(t);
        return MODE == 0 ? t.expert * 2 * g.N + f : t.expert * g.N + (f < g.N ? f : 0);
    };
    // the MMA's N, and the first of this CTA's token rows in the tile
    auto padded = [](int rows) { return (rows + 15) & ~15; };
    auto first_token = [&](const Unit& t) { return CG == 2 ? (int)rank * (padded(t.rows) / 2) : 0; };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        const uint64_t wpol = g.stream_weights ? l2_policy_evict_first() : l2_policy_evict_normal();
        const uint64_t tpol = l2_policy_evict_last();  // token rows are read again per feature block
        const uint32_t ring0 = smem_u32(ring);
        int stage = 0, fills = 0, e = 0;
        uint32_t phase = 0;
        bool ok = true, dep = !(MODE == 1 && g.early);
        const uint32_t bytes = CG * (kATxBytes + (MODE == 1 ? C::kBTile : 0));
        for (int u = unit0; u < units && ok; u += stride) {
            const Unit t = decode(u, e);
            const int row = weight_row(t), trow = t.row + first_token(t);
            for (int kt = 0; kt < num_kt; ++kt) {
                ok = __all_sync(0xffffffffu, mbar_wait(&aux->empty[stage], phase ^ 1u, abort_flag));
                if (!ok) break;
                const uint32_t st = ring0 + stage * C::kStageBytes;
                const uint32_t bar = CG == 2 ? in_leader(&aux->full[stage]) : smem_u32(&aux->full[stage]);
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&aux->full[stage], bytes);
                    tma_box<CG>(st, &tm_w, bar, kt * kBK, row, wpol);
                    tma_box<CG>(st + kATile / 2, &tm_w, bar, kt * kBK, row + (MODE == 0 ? g.N : kBM / 2),
                                wpol);
                }
                if (MODE == 1) {
                    if (!dep) {
                        pdl_wait();
                        dep = true;
                    }
                    if (elect_one()) tma_box<CG>(st + kATile, &tm_a, bar, kt * kBK, trow, tpol);
                }
                __syncwarp();
                ++fills;
                if (++stage == C::kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!dep) pdl_wait();  // (no unit here) the grid still depends on it
        if (!ok || *abort_flag) {
            if (lane == 0) flag_error();
            // let every TMA load already issued land before the CTA (CG = 2: the pair) can exit
            for (int s = 0; s < C::kStages && rank == 0; ++s) {
                const int n = fills > s ? (fills - s + C::kStages - 1) / C::kStages : 0;
                if (n > 0) {
                    volatile int never = 0;
                    mbar_wait(&aux->full[s], (uint32_t)((n - 1) & 1), &never, 500000000ull);
                }
            }
        }
    } else if (warp == 1 && rank == 1) {
        // the first CTA of the pair issues the MMAs of both
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        int stage = 0, lu = 0, e = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t ring0 = smem_u32(ring);
        for (int u = unit0; u < units && ok; u += stride, ++lu) {
            const Unit t = decode(u, e);
            const int b = lu % C::kNBuf;
            const uint32_t bphase = (uint32_t)((lu / C::kNBuf) & 1) ^ 1u;
            ok = __all_sync(0xffffffffu, CG == 2 ? mbar_wait_cluster(&aux->tempty[b], bphase, abort_flag)
                                                 : mbar_wait(&aux->tempty[b], bphase, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const int n = padded(t.rows);
            const uint32_t d = tmem_base + (uint32_t)(b * NT), idesc = idesc_mx(CG * kBM, n);
            for (int kt = 0; kt < num_kt; ++kt) {
                ok = __all_sync(0xffffffffu, CG == 2 ? mbar_wait_cluster(&aux->full[stage], phase, abort_flag)
                                                     : mbar_wait(&aux->full[stage], phase, abort_flag));
                if (!ok) break;
                tc_fence_after();
                const uint32_t sa = ring0 + stage * C::kStageBytes;
                const uint32_t sb = sa + kATile, sf = sb + C::kBTile;
                const uint32_t tsf = tmem_base + (uint32_t)(C::kSfCol0 + stage * C::kSfCols);
                const uint64_t da = umma_desc_sw128(sa), db = umma_desc_sw128(sb);
                const uint64_t ds = scale_desc(sf);
                if (elect_one()) {
                    if (CG == 1) fence_proxy_async_smem();  // scales and gathered rows came by cp.async
                    scales_to_tmem<CG>(tsf, ds);
#pragma unroll
                    for (int i = 0; i < C::kSfbCols / 4; ++i)
                        if (i * 128 < n) scales_to_tmem<CG>(tsf + 4 + 4 * i, ds + (512 >> 4) * (1 + i));
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk)  // 32 bytes along K
                        umma_mx<CG>(d, da + 2 * kk, db + 2 * kk, idesc | idesc_kb(kk), tsf, tsf + 4,
                                    (kt | kk) ? 1u : 0u);
                    commit<CG>(&aux->empty[stage]);
                    if (kt + 1 == num_kt) commit<CG>(&aux->tfull[b]);
                }
                __syncwarp();
                if (++stage == C::kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) flag_error();
        // all MMAs and copies issued by this warp are complete before TMEM is freed
        if (elect_one()) commit<CG>(&aux->drain);
        __syncwarp();
        volatile int never = 0;
        if (!mbar_wait(&aux->drain, 0, &never, 500000000ull)) atomicExch(g.err, kDeviceErrorMagic);
    } else if (warp < kEpiWarp0) {
        // ------------------------------------------------------------ scales
        // Thread i handles weight rows i and i + 64 and token rows i, i + 64, ... of a tile; a
        // row's 4 bytes of a K tile go to place(row) of the stage.
        const int i0 = threadIdx.x - kScaleWarp0 * 32;
        const size_t ld = (size_t)g.K / 32;
        if (MODE == 1 && g.early) pdl_wait();  // act's scales
        auto place = [](int r) { return (uint32_t)((r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4); };
        constexpr int kRows = 2 + C::kSIters;
        // index of token row j of the tile (0 past its end, where any scale will do)
        auto token_row = [&](const Unit& t, int j) {
            int r = t.row + min(j, t.rows - 1);
            if (MODE == 0) {
                r = g.rows[r];
                if (!debug_in_range(r, 0, g.R, g.err)) r = 0;
            }
            return r;
        };
        auto weight_src = [&](const Unit& t, int i) {
            // MODE 1: the last block's rows may lie past N; theirs are never stored
            const int row = MODE == 0 ? weight_row(t) + i * g.N + i0
                                      : t.expert * g.N + min(first_feature(t) + i * 64 + i0, g.N - 1);
            return g.w_scale + (size_t)row * ld;
        };
        auto token_src = [&](int r) {
            return g.a_scale + (size_t)(MODE == 0 ? div_by(r, g.k, g.k_magic) : r) * ld;
        };
        int q = 0, e = 0;
        bool ok = true;
        auto wait_empty = [&](int stage) {
            const uint32_t phase = (uint32_t)((q / C::kStages) & 1);
            ok = __all_sync(0xffffffffu, mbar_wait(&aux->empty[stage], phase ^ 1u, abort_flag));
            if (!ok && lane == 0) flag_error();
            return ok;
        };
        if constexpr (CG == 1) {
            // Few token rows, many stages in flight: 4-byte cp.async copies, which arrive on the
            // stage's barrier when they land.
            Unit t = {};
            int tok[C::kSIters];
            if (unit0 < units) {
                t = decode(unit0, e);
#pragma unroll
                for (int i = 0; i < C::kSIters; ++i) tok[i] = token_row(t, i0 + i * 64);
            }
            for (int u = unit0; u < units && ok; u += stride) {
                const int rows = t.rows;
                const uint8_t* src[kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i) src[i] = i < 2 ? weight_src(t, i) : token_src(tok[i - 2]);
                if (u + stride < units) {  // the next unit's rows are on their way during this one
                    t = decode(u + stride, e);
#pragma unroll
                    for (int i = 0; i < C::kSIters; ++i) tok[i] = token_row(t, i0 + i * 64);
                }
                for (int kt = 0; kt < num_kt; ++kt, ++q) {
                    const int stage = q % C::kStages;
                    if (!wait_empty(stage)) break;
                    const uint32_t sf = smem_u32(ring + stage * C::kStageBytes + kATile + C::kBTile);
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
                        if (i < 2 || i0 + (i - 2) * 64 < rows)
                            cp_async_4(sf + (i < 2 ? place(i0 + i * 64) : 512 + place(i0 + (i - 2) * 64)),
                                       src[i] + kt * 4);
                    cp_async_mbar_arrive(&aux->full[stage]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&aux->full[stage]);
                }
            }
            cp_async_commit();
            cp_async_wait<0>();  // no copy is still in flight when the CTA exits
        } else {
            // Many token rows: a 4-byte copy is one L1 line lookup a row and K tile.  So rows are
            // read a group of 4 K tiles at a time (16 bytes where the row pitch allows it), kAhead
            // groups before they are stored from registers.
            constexpr int kAhead = 2;
            const int align = (int)(ld & 15);  // 0: 16-byte rows, 8: 8-byte, else 4-byte
            auto load = [&](uint32_t (&w)[4], const uint8_t* p, int kt) {
                p += kt * 4;
                if (align == 0) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
                    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                } else if (align == 8) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
                    w[0] = v.x, w[1] = v.y;
                    if (kt + 2 < num_kt) {
                        const uint2 x = __ldg(reinterpret_cast<const uint2*>(p) + 1);
                        w[2] = x.x, w[3] = x.y;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (kt + j < num_kt) w[j] = __ldg(reinterpret_cast<const uint32_t*>(p) + j);
                }
            };
            // The reader: the next group to load, and (one unit further) the rows of the unit after.
            const uint8_t* src[kRows];
            int tok[C::kSIters], ru = unit0, rkt = 0;
            Unit rt = {};
            auto next_rows = [&](int u) {
                if (u >= units) return;
                rt = decode(u, e);
#pragma unroll
                for (int i = 0; i < C::kSIters; ++i) tok[i] = token_row(rt, i0 + i * 64);
            };
            auto read_group = [&](uint32_t (&w)[kRows][4]) {
                if (ru >= units) return;
                if (rkt == 0) {
#pragma unroll
                    for (int i = 0; i < kRows; ++i) src[i] = i < 2 ? weight_src(rt, i) : token_src(tok[i - 2]);
                    next_rows(ru + stride);
                }
#pragma unroll
                for (int i = 0; i < kRows; ++i) load(w[i], src[i], rkt);
                rkt += 4;
                if (rkt >= num_kt) {
                    rkt = 0;
                    ru += stride;
                }
            };
            uint32_t w[kAhead][kRows][4];
            next_rows(unit0);
#pragma unroll
            for (int a = 0; a < kAhead; ++a) read_group(w[a]);
            for (int u = unit0; u < units && ok; u += stride) {
                for (int kt = 0; kt < num_kt && ok; kt += 4) {
                    uint32_t cur[kRows][4];
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            cur[i][j] = w[0][i][j];
#pragma unroll
                            for (int a = 0; a + 1 < kAhead; ++a) w[a][i][j] = w[a + 1][i][j];
                        }
                    read_group(w[kAhead - 1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (kt + j >= num_kt) break;
                        const int stage = q % C::kStages;
                        if (!wait_empty(stage)) break;
                        uint8_t* sf = ring + stage * C::kStageBytes + kATile + C::kBTile;
#pragma unroll
                        for (int i = 0; i < kRows; ++i)
                            if (i < 2 || i0 + (i - 2) * 64 < NT)
                                *reinterpret_cast<uint32_t*>(
                                    sf + (i < 2 ? place(i0 + i * 64) : 512 + place(i0 + (i - 2) * 64))) =
                                    cur[i][j];
                        fence_proxy_async_smem();  // read by tcgen05.cp
                        __syncwarp();
                        if (lane == 0) arrive_leader(&aux->full[stage]);
                        ++q;
                    }
                }
            }
        }
    } else if (MODE == 0 && warp >= kGatherWarp0) {
        // ------------------------------------------------------------ gather (MODE 0)
        // Thread i copies the 16-byte chunks i, i + 128, ... of this CTA's token rows (8 chunks a
        // row).  CG = 1: the copies arrive on the stage's barrier themselves.  CG = 2: that
        // cannot reach the other CTA's barrier, so a warp waits for its copies of kLag stages
        // ago, fences them towards the async proxy and arrives there.
        constexpr int kLag = 3;
        static_assert(kLag < C::kStages, "a stage is filled before its ring slot comes round");
        const int i0 = threadIdx.x - kGatherWarp0 * 32;
        const uint64_t pol = l2_policy_evict_last();  // token rows are read again per feature block
        int q = 0, e = 0;
        bool ok = true;
        Unit t = {};
        int r[C::kGIters];
        auto next_rows = [&](int u) {
            if (u >= units) return;
            t = decode(u, e);
#pragma unroll
            for (int i = 0; i < C::kGIters; ++i) {
                const int j = (i0 + i * 128) >> 3;
                r[i] = -1;
                if (j < C::kBRows && first_token(t) + j < t.rows) {
                    r[i] = g.rows[t.row + first_token(t) + j];
                    if (!debug_in_range(r[i], 0, g.R, g.err)) r[i] = 0;
                }
            }
        };
        auto arrive = [&](int stage) {  // CG = 2
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive_leader(&aux->full[stage]);
        };
        next_rows(unit0);
        for (int u = unit0; u < units && ok; u += stride) {
            const uint8_t* src[C::kGIters];
#pragma unroll
            for (int i = 0; i < C::kGIters; ++i)
                src[i] = r[i] < 0 ? nullptr
                                  : g.a + (size_t)div_by(r[i], g.k, g.k_magic) * g.K + (i0 & 7) * 16;
            next_rows(u + stride);  // on their way during this unit
            for (int kt = 0; kt < num_kt; ++kt, ++q) {
                const int stage = q % C::kStages;
                const uint32_t phase = (uint32_t)((q / C::kStages) & 1);
                ok = __all_sync(0xffffffffu, mbar_wait(&aux->empty[stage], phase ^ 1u, abort_flag));
                if (!ok) {
                    if (lane == 0) flag_error();
                    break;
                }
                const uint32_t sb = smem_u32(ring + stage * C::kStageBytes + kATile);
#pragma unroll
                for (int i = 0; i < C::kGIters; ++i) {
                    const int c = i0 + i * 128, j = c >> 3;
                    if (src[i])
                        cp_async_16_hint(sb + j * 128 + (((c & 7) ^ (j & 7)) << 4), src[i] + kt * kBK, pol);
                }
                if constexpr (CG == 1) {
                    cp_async_mbar_arrive(&aux->full[stage]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&aux->full[stage]);
                } else {
                    cp_async_commit();
                    if (q >= kLag) {
                        cp_async_wait<kLag>();
                        arrive((q - kLag) % C::kStages);
                    }
                }
            }
        }
        cp_async_commit();
        cp_async_wait<0>();  // no copy is still in flight when the CTA exits
        if constexpr (CG == 2)
            for (int p = max(q - kLag, 0); p < q && ok; ++p) arrive(p % C::kStages);
    } else {
        // ------------------------------------------------------------ epilogue
        const int grp = (warp - kEpiWarp0) >> 2;     // token-column group
        const int lq = warp & 3;                     // TMEM lane quarter
        int lu = 0, chunk = 0, e = 0;
        auto release = [&](int b) {  // this warp has read accumulator b
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2)
                    arrive_leader(&aux->tempty[b]);
                else
                    mbar_arrive(&aux->tempty[b]);
            }
        };
        for (int u = unit0; u < units; u += stride, ++lu) {
            const Unit t = decode(u, e);
            const int b = lu % C::kNBuf;
            const int jbeg = grp * C::kGroupCols, jend = min(t.rows, jbeg + C::kGroupCols);
            // MODE 1: lane i holds the y rows of the group's columns i, i + 32, ...
            int yrow[(C::kGroupCols + 31) / 32] = {};
            if (MODE == 1) {
#pragma unroll
                for (int i = 0; i < (C::kGroupCols + 31) / 32; ++i) {
                    const int j = jbeg + i * 32 + lane;
                    if (j < jend) {
                        yrow[i] = g.rows ? g.rows[t.row + j] : t.row + j;
                        if (!debug_in_range(yrow[i], 0, g.R, g.err)) yrow[i] = 0;
                    }
                }
            }
            const bool got = mbar_wait(&aux->tfull[b], (uint32_t)((lu / C::kNBuf) & 1), abort_flag);
            if (!got) flag_error();
            if (named_bar_or(1 + grp, 128, !got || *abort_flag)) break;  // same in all 4 warps
            tc_fence_after();
            const uint32_t acc = tmem_base + ((uint32_t)(lq * 32) << 16) + (uint32_t)(b * NT);
            if constexpr (MODE == 0) {
                // Lanes 0-63 hold gate rows, 64-127 the up rows of the same features.  Warps lq
                // and lq ^ 2 exchange 4 of every 8 columns through shared memory: the gate
                // warp finishes the first 4, the up warp the others.  A warp's 32 lanes are
                // then one MX block of act for each of its columns.
                const bool up = lq >= 2;
                const int feature = first_feature(t) + (lq & 1) * 32;
                float* mine = reinterpret_cast<float*>(staging) + (warp - kEpiWarp0) * 256;
                const float* other = reinterpret_cast<float*>(staging) + ((warp ^ 2) - kEpiWarp0) * 256;
                for (int j0 = jbeg; j0 < jend; j0 += 8, ++chunk) {
                    uint32_t v[8];
                    tmem_ld8(acc + j0, v);
                    tmem_ld_wait();
                    const int buf = (chunk & 1) * 128;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mine[buf + i * 32 + lane] = __uint_as_float(up ? v[i] : v[4 + i]);
                    named_bar_sync(3 + grp * 2 + (lq & 1), 64);
                    float a[4];
                    uint32_t code[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float o = other[buf + i * 32 + lane];
                        const float own = __uint_as_float(up ? v[4 + i] : v[i]);
                        a[i] = up ? silu_mul(o, own) : silu_mul(own, o);
                        const uint32_t m = __reduce_max_sync(0xffffffffu,
                                                             __float_as_uint(a[i]) & 0x7FFFFFFFu);
                        code[i] = mx::scale_code(m, mx::kEmaxE4M3);
                        a[i] *= mx::inverse_scale(min(code[i], 254u));
                    }
                    const uint32_t q4 = mx::e4m3x4(a[0], a[1], a[2], a[3]);
                    const int j = j0 + (up ? 4 : 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (j + i < jend) {
                            const size_t p = (size_t)(t.row + j + i);
                            g.act[p * g.N + feature + lane] =
                                code[i] == mx::kNanScale ? 0x7F : (uint8_t)(q4 >> (8 * i));
                            if (lane == i)
                                g.act_scale[p * (g.N / 32) + feature / 32] = (uint8_t)code[i];
                        }
                    }
                }
                release(b);
            } else {
                // Drain this group's columns into registers as packed bf16 and hand them back,
                // then transpose 8 token rows of this warp's 32 features at a time through
                // its own 512 bytes of shared memory and store 16 bytes a lane.  The 16x256b
                // load gives a lane two tokens of feature lane / 4, which is the fragment that
                // a transposing stmatrix takes; 16-byte chunk c of row r lies at c ^ (r / 2), so
                // neither its 8 rows nor the reads share a bank.  No barrier but the warp's.
                uint32_t pk[C::kGroupCols / 2];
                constexpr int kBatch = 4;  // column blocks per wait
#pragma unroll
                for (int c0 = 0; c0 < C::kGroupCols / 8; c0 += kBatch) {
                    uint32_t v[kBatch][8];
#pragma unroll
                    for (int c = c0; c < c0 + kBatch && c < C::kGroupCols / 8; ++c)
                        if (jbeg + c * 8 < jend) {
                            tmem_ld_16x256(acc + jbeg + c * 8, v[c - c0]);
                            tmem_ld_16x256(acc + (16u << 16) + jbeg + c * 8, v[c - c0] + 4);
                        }
                    tmem_ld_wait();
#pragma unroll
                    for (int c = c0; c < c0 + kBatch && c < C::kGroupCols / 8; ++c)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(
                                __uint_as_float(v[c - c0][2 * i]), __uint_as_float(v[c - c0][2 * i + 1]));
                            pk[c * 4 + i] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                }
                release(b);
                const int f = first_feature(t) + lq * 32 + (lane & 3) * 8;
                __nv_bfloat16* const y = static_cast<__nv_bfloat16*>(g.y) + f;
                uint8_t* const mine = staging + (warp - kEpiWarp0) * 1024;
                const uint32_t put = smem_u32(mine) + (lane & 7) * 64 + (((lane >> 3) ^ ((lane & 7) >> 1)) << 4);
                const uint8_t* const get = mine + (lane >> 2) * 64 + (((lane & 3) ^ (lane >> 3)) << 4);
#pragma unroll
                for (int c = 0; c < C::kGroupCols / 8; ++c) {
                    if (jbeg + c * 8 < jend) {
                        const int buf = (c & 1) * 512;
                        store_matrix_x4_trans(put + buf, pk[c * 4], pk[c * 4 + 1], pk[c * 4 + 2], pk[c * 4 + 3]);
                        __syncwarp();
                        const uint4 val = *reinterpret_cast<const uint4*>(get + buf);
                        const int j = c * 8 + (lane >> 2);
                        const int row = __shfl_sync(0xffffffffu, yrow[c / 4], j & 31);
                        if (jbeg + j < jend && f < g.N)
                            *reinterpret_cast<uint4*>(y + (size_t)row * g.N) = val;
                    }
                }
                __syncwarp();  // the buffers are free again
            }
        }
    }

    tc_fence_before();
    if constexpr (CG == 2)
        cluster_sync();  // neither CTA leaves while the other may arrive on its barriers
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_release<CG>(tmem_base, C::kTmemCols);
    }
}

// ------------------------------------------------------------------ host side

// E2M1 codes [rows, cols / 2]: a box of box_rows x 128 elements, unpacked to one byte slot
// an element with the 128-byte swizzle.
cudaError_t tmap_e2m1(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows)
{
    gemm::EncodeTiledFn fn = gemm::get_encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols / 2};
    const cuuint32_t box[2] = {(cuuint32_t)kBK, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<void*>(base), dims,
                          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int MODE, int NT, int CG = 1>
cudaError_t launch_nt(MxArgs g, cudaStream_t st)
{
    using C = Cfg<MODE, NT, CG>;
    g.fb_count = (g.N + C::kFeatures - 1) / C::kFeatures;
    auto magic = [](int d) { return d > 1 ? (uint32_t)((1ull << 32) / (unsigned)d + 1) : 0u; };
    g.fb_magic = magic(g.fb_count);
    g.k_magic = magic(g.k);
    CUtensorMap tw, ta;
    cudaError_t e = tmap_e2m1(&tw, g.w, (uint64_t)g.E * g.N * (MODE == 0 ? 2 : 1), (uint64_t)g.K, 64);
    if (e == cudaSuccess)
        e = MODE == 1 ? gemm::make_tmap_u8(&ta, g.a, (uint64_t)g.R, (uint64_t)g.K, C::kBRows, kBK)
                      : (ta = tw, e);
    if (e != cudaSuccess) return e;
    auto kern = mx_grouped_kernel<MODE, NT, CG>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(device_sms() / CG * CG);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, tw, ta, g);
}

template <int MODE>
cudaError_t launch_mode(const MxArgs& g, int most, cudaStream_t st)
{
    if (most <= 16) return launch_nt<MODE, 16>(g, st);
    if (most <= 32) return launch_nt<MODE, 32>(g, st);
    if (most <= 64) return launch_nt<MODE, 64>(g, st);
    if (g.R < 64 * g.E) return launch_nt<MODE, 128>(g, st);
    return launch_nt<MODE, 208, 2>(g, st);
}

}  // namespace

cudaError_t launch_mx_grouped(const MxArgs& args, int mode, cudaStream_t st)
{
    MxArgs g = args;
    // the most rows that one expert can have: a token picks an expert at most once
    const int most = mode == 2 ? g.R : g.R / g.k;
    g.early = mode == 1;
    g.stream_weights = most <= 64;
    if (mode == 2) {
        g.rows = nullptr;
        g.k = 1;
    }
    return mode == 0 ? launch_mode<0>(g, most, st) : launch_mode<1>(g, most, st);
}

}  // namespace moe
