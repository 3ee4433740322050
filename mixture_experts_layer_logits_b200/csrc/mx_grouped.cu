// mx_grouped.cu -- products grouped by expert of E4M3 token rows with E2M1 weights, both in
// microscaled blocks, alone and as the two products of the expert FFN, on block-scaled tcgen05
// tensor cores.
//
//   MODE 0  act[p, f] = MX(silu(gate) * up) of x[rows[p] / k] with w13[e] rows f and I + f
//   MODE 1  y[rows[p] or p, f] = w[e] row f dotted with act (or any E4M3 rows) [p]
//
// Two CTAs of a cluster work on one MMA (cta_group::2): its M = 256 rows are weight rows, 128 per
// CTA, its N columns an expert's token rows, rounded up to 16 per tile, so few tokens cost few
// columns and a ragged group at most 15 padded ones.  Why this shape (cycles per K tile of 128,
// i.e. 4 MMAs and the scale copies; an SM streaming 128 packed weight rows of it at its share of
// HBM takes 380):
//   - one CTA, M = 128, N = 16: 502; the pair 409 for twice the rows.  An MMA takes 90 cycles or
//     more to read its M operand, and a scale copy in between costs the pair less.
//   - token rows as the M operand, N = 256 weight rows: 523 for 256 rows a CTA, so HBM-bound; but an
//     MMA then multiplies 128 rows however few are tokens, and the power that takes lowers the
//     clock: T = 64, E = 256, skewed, H = 7168, I = 2048 took 136 us under sustained load (114 in
//     a burst), the pair 108 (94).
//   - many tokens: a pair reads each weight row and each token row once, half of both per CTA.
//     One CTA with N = 128 was bound by its reads from L2 (T = 8192, E = 128, k = 8, H = 4096,
//     I = 1536: 2.11 ms, the pair 1.2 in a burst and 1.34 under the power cap of sustained load).
//
// Warp roles: 0 TMA; 1 TMEM, and in CTA 0 MMA issue for both; 2-3 and 12-13 scales; 4-11
// epilogue; MODE 0: 14-15 gather of token rows.
//   - MODE 1 loads token rows by TMA with the weights; MODE 0 gathers x rows with 16-byte
//     cp.async copies straight to their swizzled places.  (26 gather4 TMA loads a stage, one
//     per lane, issue too slowly: w13 took 1.70 ms instead of 0.97.)
//   - Both CTAs' loads count on CTA 0's full barriers; the commit of a stage's MMAs frees it
//     in both.
// Every mbarrier wait is bounded; on a timeout the kernel records the error word, stops
// issuing, drains what it issued and frees TMEM.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_gemm.cuh"

namespace moe {

namespace {

using namespace mx;
using gemm::named_bar_or;
using gemm::named_bar_sync;

constexpr int kBM = 128;                  // weight rows of one CTA's tile
constexpr int kATile = kBM * kBK;
// weight rows of one TMA box (MODE 0 loads gate and up rows of 32 features in turn)
template <int MODE>
constexpr int kWBoxRows = MODE == 0 ? 32 : kBM;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8, kGatherWarp0 = 14, kGatherWarps = 2;
constexpr int kThreads = 32 * (kGatherWarp0 + kGatherWarps);  // whole warpgroups; MODE 1 leaves two warps idle
constexpr int kMaxStages = 12;
// epilogue shared memory per warp: MODE 0, 2 buffers of 8 columns x 32 lanes of fp32 to swap; MODE 1,
// 2 buffers of 8 token rows x 32 bf16
constexpr int kWarpStaging = 2 * 1024;

// NT: the most token rows of a tile.
template <int MODE, int NT>
struct Cfg {
    static constexpr int kBRows = NT / 2;                        // token rows in one CTA's B tile
    static constexpr int kBTile = kBRows * kBK;
    static constexpr int kTokenScales = NT > 128 ? 1024 : 512;   // bytes a stage
    static constexpr int kStageBytes = (kATile + kBTile + 512 + kTokenScales + 1023) & ~1023;
    static constexpr int kStaging = kEpiWarps * (MODE == 0 ? kWarpStaging : 1024);
    static constexpr int kFixed = 1024 + kStaging + 512 + kTableBytes;
    static constexpr int kNBuf = NT <= 64 ? 4 : 2;               // accumulators in flight
    static constexpr int kSfCol0 = kNBuf * NT;                   // first scale column
    static constexpr int kSfCols = NT > 128 ? 16 : 8;            // per stage; 4 of weights, 4 or 8 of tokens
    static constexpr int kStagesSmem = (232448 - kFixed) / kStageBytes;
    static constexpr int kStagesTmem = (512 - kSfCol0) / kSfCols;
    static constexpr int kStagesRaw = kStagesSmem < kStagesTmem ? kStagesSmem : kStagesTmem;
    static constexpr int kStages = kStagesRaw < kMaxStages ? kStagesRaw : kMaxStages;
    static constexpr int kSmem = kFixed + kStages * kStageBytes;
    static constexpr int kTmemCols = kSfCol0 + kStages * kSfCols <= 256 ? 256 : 512;
    static constexpr int kFeatures = MODE == 0 ? 64 : 128;       // output features of one CTA
    static constexpr int kGroupCols = NT / 2;                    // token columns per epilogue group of four warps
    static constexpr int kGIters = (kBRows * 8 + kGatherWarps * 32 - 1) / (kGatherWarps * 32);
    static_assert(NT % 16 == 0 && NT <= 256 && kStages >= 4 && kSmem <= 232448, "tile");
};

struct Aux {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t gathered[kMaxStages];  // MODE 0: this CTA's gathered rows of the stage have landed
    uint64_t tfull[4];
    uint64_t tempty[4];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

// Arrive on the barrier at this address in both CTAs when every tensor instruction issued so
// far by this thread is done.
__device__ __forceinline__ void commit(uint64_t* bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Address of the same shared-memory location in CTA 0 of the cluster.
__device__ __forceinline__ uint32_t in_leader(const void* p)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}

// Arrive on the barrier that lies at this address in CTA 0 of the cluster.  It carries
// only the fact.  What it stands for is in the arriving CTA: scales and gathered rows in its
// shared memory, written and fenced towards the async proxy before, which the tensor core
// of that CTA's own SM reads; or its TMEM, read out before tcgen05.wait::ld.  So the default
// release (CTA scope) is enough.  A release at cluster scope waits for the L2: 1200 cycles
// a stage, prefill 2.66 ms instead of 1.52.  The waits on such barriers acquire at CTA scope alike.
__device__ __forceinline__ void arrive_leader(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_leader(bar)) : "memory");
}

// Whether the phase with this parity is complete.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Arrives on the barrier once every cp.async this thread issued so far has landed: one of the
// arrivals that the barrier counts.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
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

// silu(g) u = g u / (1 + 2^(-g log2 e)), exponential and reciprocal one instruction each.  The
// rounding of the exponent makes the power off by up to |g| units of 2^-24, and instructions and
// products add a few of 2^-23: far inside the rounding to E4M3.  From g = -64 down 1 / (1 + e^-g) is
// e^g to fp32's precision and is taken as the square of 2^(g log2 e / 2), one factor of it with u.
// The reciprocal would be subnormal from g = -87.3 on, hence zero; this holds to g = -174,
// where e^g = 2^-251.  It costs the prompt's FFN 0.3% (T = 8192: 1311 and 1316 us).
__device__ __forceinline__ float swiglu(float g, float u)
{
    const bool far = !(g > -64.0f);
    float p, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(g * (far ? 0.72134752f : -1.44269504f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + p));
    return g * (far ? p : r) * (far ? p * u : u);
}

// The largest magnitude of four, NaN if one of them is.
__device__ __forceinline__ float max_abs4(float a, float b, float c, float d)
{
    float m;
    asm("{\n\t.reg .f32 t;\n\t"
        "max.NaN.f32 t, %1, %2;\n\t"
        "max.NaN.f32 %0, %3, %4;\n\t"
        "max.NaN.f32 %0, %0, t;\n\t}"
        : "=&f"(m)
        : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)), "f"(fabsf(d)));
    return m;
}

// 4 x 4 bytes transposed over the lanes whose l differs in its lower 2 bits (lanes 4 apart): byte i
// of the lane with l % 4 = b goes to byte b of the one with l % 4 = i.
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t q, int l)
{
    uint32_t o = __shfl_xor_sync(0xffffffffu, q, 4);
    q = __byte_perm(q, o, l & 1 ? 0x3715 : 0x6240);
    o = __shfl_xor_sync(0xffffffffu, q, 8);
    return __byte_perm(q, o, l & 2 ? 0x3276 : 0x5410);
}

template <int MODE, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    mx_grouped_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
                      const MxArgs g)
{
    using C = Cfg<MODE, NT>;
    constexpr int kStages = C::kStages, kStageBytes = C::kStageBytes, kBTile = C::kBTile;
    constexpr int kGroupCols = C::kGroupCols, kNBuf = C::kNBuf;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t* staging = ring + kStages * kStageBytes;
    Aux* aux = reinterpret_cast<Aux*>(staging + C::kStaging);
    static_assert(sizeof(Aux) <= 512, "aux area");

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    // The second product of the FFN (g.early) takes only act from the launch before it;
    // expert_offsets, rows and weights were complete before that launch passed its own
    // wait, so the tables and the first weight tiles need not wait for it.
    Offsets<kThreads> offsets;
    if (g.early) offsets.read(g);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            // CTA 0's counts: the expect_tx, one arrival per scale warp of both CTAs, and CTA 1's
            // relayed one for its gathered rows
            mbar_init(&aux->full[s], 1 + 2 * kScaleWarps + (MODE == 0 ? 1 : 0));
            mbar_init(&aux->empty[s], 1);
            mbar_init(&aux->gathered[s], 32 * kGatherWarps);
        }
        for (int b = 0; b < kNBuf; ++b) {
            mbar_init(&aux->tfull[b], 1);
            mbar_init(&aux->tempty[b], 2 * kEpiWarps);
        }
        mbar_init(&aux->drain, 1);
        aux->abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_w);
        if (MODE == 1) tma_prefetch_desc(&tm_a);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&aux->tmem_base)),
                     "r"(C::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_arrive();  // barriers initialised, TMEM allocated
    if (!g.early) {
        pdl_wait();
        offsets.read(g);
    }
    pdl_launch_dependents();
    const Groups groups = build_groups<kThreads>(
        g, offsets, NT, reinterpret_cast<int*>(staging + C::kStaging + 512));
    cluster_wait();    // ... in the other CTA too
    tc_fence_after();

    uint32_t rank;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int unit0 = (int)blockIdx.x / 2, stride = (int)gridDim.x / 2;
    const uint32_t tmem_base = aux->tmem_base;
    volatile int* abort_flag = &aux->abort;
    auto flag_error = [&] {
        atomicExch(g.err, kDeviceErrorMagic);
        aux->abort = 1;
    };
    const int fbs = g.fb_count;
    const int units = groups.first[g.E] * fbs;
    const int num_kt = g.K / kBK;
    Units list(groups, fbs, g.fb_magic, unit0, stride);
    auto padded = [](int rows) { return (rows + 15) & ~15; };  // the MMA's N
    // this CTA's part of a unit: its first output feature, and its first token row in the tile.
    // MODE 1: the second CTA's features may begin past N; it then works on the first ones
    // again, and stores none of them.
    auto first_feature = [&](const Unit& t) { return (t.fb * 2 + (int)rank) * C::kFeatures; };
    auto first_token = [&](const Unit& t) { return (int)rank * (padded(t.rows) / 2); };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        // Weights that one tile reads once leave L2 first (T = 8, E = 128: 11.8 us for the down
        // product, 12.1 without); where several tiles share them they stay (T = 8192: 384 us, 391
        // with evict_first).  Token rows are read again per feature block (11.8 us; 16.0 with the
        // default policy).
        const uint64_t wpol = g.stream_weights ? l2_policy_evict_first() : l2_policy_evict_normal();
        const uint64_t tpol = l2_policy_evict_last();
        const uint32_t ring0 = smem_u32(ring);
        const uint32_t bytes = 2 * (kBM * kRowTx + (MODE == 1 ? kBTile : 0));
        const uint32_t full0 = in_leader(&aux->full[0]);
        int stage = 0, fills = 0;
        uint32_t phase = 0;
        bool ok = true, dep = !(MODE == 1 && g.early);
        for (int u = unit0; u < units && ok; u += stride) {
            const Unit t = list.next();
            const int f = first_feature(t);
            const int row = MODE == 0 ? t.expert * 2 * g.N + f : t.expert * g.N + (f < g.N ? f : 0);
            const int trow = t.row + first_token(t);
            for (int kt = 0; kt < num_kt; ++kt) {
                ok = warp_agrees(mbar_wait(&aux->empty[stage], phase ^ 1u, abort_flag));
                if (!ok) break;
                const uint32_t st = ring0 + stage * kStageBytes;
                const uint32_t bar = full0 + stage * 8;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&aux->full[stage], bytes);
#pragma unroll
                    for (int r = 0; r < kBM; r += kWBoxRows<MODE>)
                        tma_2d(st + r * kBK, &tm_w, bar, kt * kBK,
                               row + (MODE == 0 ? tile_feature(r) + (tile_row_is_up(r) ? g.N : 0) : r), wpol);
                }
                if (MODE == 1) {
                    if (!dep) {
                        pdl_wait();
                        dep = true;
                    }
                    __syncwarp();
                    if (elect_one()) tma_2d(st + kATile, &tm_a, bar, kt * kBK, trow, tpol);
                }
                __syncwarp();
                ++fills;
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!dep) pdl_wait();  // (no unit here) the grid still depends on it
        if (!ok || *abort_flag) {
            if (lane == 0) flag_error();
            // let every TMA load already issued land before the pair can exit
            for (int s = 0; s < kStages && rank == 0; ++s) {
                const int n = fills > s ? (fills - s + kStages - 1) / kStages : 0;
                if (n > 0) {
                    volatile int never = 0;
                    mbar_wait(&aux->full[s], (uint32_t)((n - 1) & 1), &never, 500000000ull);
                }
            }
        }
    } else if (warp == 1 && rank == 1) {
        // ------------------------------------------------------------ relay (MODE 0)
        // CTA 0 issues the MMAs of both: tell it when a stage's gathered rows are here.
        if (MODE == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = unit0; u < units && ok; u += stride)
                for (int kt = 0; kt < num_kt; ++kt) {
                    ok = warp_agrees(mbar_wait(&aux->gathered[stage], phase, abort_flag));
                    if (!ok) break;
                    if (elect_one()) {
                        fence_proxy_async_smem();
                        arrive_leader(&aux->full[stage]);
                    }
                    __syncwarp();
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            if (!ok && lane == 0) flag_error();
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        int stage = 0, lu = 0, ready = 0;  // ready: stages from this one on known to be full
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t ring0 = smem_u32(ring);
        for (int u = unit0; u < units && ok; u += stride, ++lu) {
            const Unit t = list.next();
            const int b = lu % kNBuf;
            ok = warp_agrees(
                mbar_wait(&aux->tempty[b], (uint32_t)((lu / kNBuf) & 1) ^ 1u, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const int n = padded(t.rows);
            const uint32_t d = tmem_base + (uint32_t)(b * NT);
            const uint32_t idesc = idesc_mx(2 * kBM, n);
            for (int kt = 0; kt < num_kt; ++kt) {
                // MODE 0 has two barriers to pass, and a read of one takes some 100 cycles while MMAs
                // and TMA use the shared memory: the lanes look at those of 4 stages at once (FFN of 8
                // tokens 31.6 us, 33.6 one by one; with a single barrier it costs, 12.2 and 11.9 us).
                if (MODE == 0 && ready == 0) {
                    const bool wraps = stage + lane >= kStages;
                    const int at = stage + lane - (wraps ? kStages : 0);
                    const uint32_t parity = phase ^ (wraps ? 1u : 0u);
                    const bool there =
                        lane < 4 && mbar_test(&aux->gathered[at], parity) && mbar_test(&aux->full[at], parity);
                    ready = __ffs(~__ballot_sync(0xffffffffu, there)) - 1;
                    __syncwarp();
                }
                if (ready == 0)
                    ok = warp_agrees((MODE == 1 || mbar_wait(&aux->gathered[stage], phase, abort_flag)) &&
                                     mbar_wait(&aux->full[stage], phase, abort_flag));
                else
                    --ready;
                if (!ok) break;
                tc_fence_after();
                const uint32_t sa = ring0 + stage * kStageBytes;
                const uint32_t sb = sa + kATile, sf = sb + kBTile;
                const uint32_t tsf = tmem_base + (uint32_t)(C::kSfCol0 + stage * C::kSfCols);
                const uint64_t da = umma_desc_sw128(sa), db = umma_desc_sw128(sb);
                const uint64_t ds = scale_desc(sf);
                if (elect_one()) {
                    if (MODE == 0) fence_proxy_async_smem();  // this CTA's rows came by cp.async
                    scales_to_tmem(tsf, ds);
                    scales_to_tmem(tsf + 4, ds + (512 >> 4));
                    if (NT > 128 && n > 128) scales_to_tmem(tsf + 8, ds + (1024 >> 4));
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk)  // 32 bytes along K
                        umma_mx(d, da + 2 * kk, db + 2 * kk, idesc | idesc_kb(kk), tsf, tsf + 4,
                                (kt | kk) ? 1u : 0u);
                    commit(&aux->empty[stage]);
                    if (kt + 1 == num_kt) commit(&aux->tfull[b]);
                }
                __syncwarp();
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) flag_error();
        __syncwarp();
        // all MMAs and copies issued by this warp are complete before TMEM is freed
        if (elect_one()) commit(&aux->drain);
        __syncwarp();
        volatile int never = 0;
        if (!mbar_wait(&aux->drain, 0, &never, 500000000ull)) atomicExch(g.err, kDeviceErrorMagic);
    } else if (warp == 2 || warp == 3 || warp == 12 || warp == 13) {
        // ------------------------------------------------------------ scales
        // Thread i handles weight row i of this CTA's tile and token rows i and i + 128 of the
        // whole tile (each CTA needs them all).
        const int i0 = (warp < 4 ? warp - 2 : warp - 10) * 32 + lane;
        const size_t ld = (size_t)g.K / 32;
        if (MODE == 1 && g.early) pdl_wait();  // act's scales
        constexpr int kTok = NT > 128 ? 2 : 1, kRows = 1 + kTok;
        int put[kRows] = {(int)scale_place(i0)};
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            put[1 + i] = i0 + i * 128 < NT ? (int)(512 + scale_place(i0 + i * 128)) : -1;
        int tok[kTok];
        Unit next;
        auto fetch = [&](int u) {
            next = list.next();
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                // past the tile's end any scale will do
                tok[i] = next.row + min(i0 + i * 128, next.rows - 1);
                if (MODE == 0) {
                    tok[i] = g.rows[tok[i]];
                    if (!debug_in_range(tok[i], 0, g.R, g.err)) tok[i] = 0;
                }
            }
        };
        auto sources = [&](int, const uint8_t* (&src)[kRows]) {
            // MODE 1: rows past N belong to features that are never stored
            const int f = first_feature(next);
            const int row = MODE == 0 ? next.expert * 2 * g.N + f + tile_feature(i0) +
                                            (tile_row_is_up(i0) ? g.N : 0)
                                      : next.expert * g.N + min(f + i0, g.N - 1);
            src[0] = g.w_scale + (size_t)row * ld;
#pragma unroll
            for (int i = 0; i < kTok; ++i)
                src[1 + i] = g.a_scale + (size_t)(MODE == 0 ? div_by(tok[i], g.k, g.k_magic) : tok[i]) * ld;
        };
        run_scales<kRows>(
            unit0, stride, units, num_kt, (int)ld, put, fetch, sources,
            [&](int q) {
                const bool ok = warp_agrees(mbar_wait(&aux->empty[q % kStages],
                                                                  (uint32_t)((q / kStages) & 1) ^ 1u,
                                                                  abort_flag));
                if (!ok && lane == 0) flag_error();
                return ok;
            },
            [&](int q) { return ring + (q % kStages) * kStageBytes + kATile + kBTile; },
            [&](int q) {
                if (lane == 0) arrive_leader(&aux->full[q % kStages]);
            });
    } else if (MODE == 0 && warp >= kGatherWarp0) {
        // ------------------------------------------------------------ gather (MODE 0)
        // Thread i copies the 16-byte chunks i, i + 64, ... of this CTA's token rows (8 chunks a
        // row).  The copies arrive on this CTA's own barrier when they land (they cannot on the
        // other CTA's); CTA 0's MMA warp waits for that, CTA 1's warp 1 relays it.
        const int i0 = threadIdx.x - kGatherWarp0 * 32;
        const uint64_t pol = l2_policy_evict_last();
        int q = 0;
        bool ok = true;
        int r[C::kGIters];
        auto next_rows = [&](int u) {
            if (u >= units) return;
            const Unit t = list.next();
#pragma unroll
            for (int i = 0; i < C::kGIters; ++i) {
                const int j = (i0 + i * kGatherWarps * 32) >> 3;
                r[i] = -1;
                if (j < C::kBRows && first_token(t) + j < t.rows) {
                    r[i] = g.rows[t.row + first_token(t) + j];
                    if (!debug_in_range(r[i], 0, g.R, g.err)) r[i] = 0;
                }
            }
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
                const int stage = q % kStages;
                const uint32_t phase = (uint32_t)((q / kStages) & 1);
                ok = warp_agrees(mbar_wait(&aux->empty[stage], phase ^ 1u, abort_flag));
                if (!ok) {
                    if (lane == 0) flag_error();
                    break;
                }
                const uint32_t sb = smem_u32(ring + stage * kStageBytes + kATile);
#pragma unroll
                for (int i = 0; i < C::kGIters; ++i) {
                    const int c = i0 + i * kGatherWarps * 32, j = c >> 3;
                    if (src[i])
                        cp_async_16_hint(sb + j * 128 + (((c & 7) ^ (j & 7)) << 4), src[i] + kt * kBK, pol);
                }
                cp_async_arrive(&aux->gathered[stage]);
            }
        }
        cp_async_commit();
        cp_async_wait<0>();  // no copy is still in flight when the CTA exits
    } else if (warp >= kEpiWarp0 && warp < kEpiWarp0 + kEpiWarps) {
        // ------------------------------------------------------------ epilogue
        const int grp = (warp - kEpiWarp0) >> 2;     // token-column group
        const int lq = warp & 3;                     // TMEM lane quarter
        const int jbeg = grp * kGroupCols;
        constexpr int kBlocks = kGroupCols / 8;      // column blocks of 8
        auto release = [&](int b) {  // this warp has read accumulator b
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(&aux->tempty[b]);
        };
        int lu = 0;
        bool stopped = false;
        for (int u = unit0; u < units; u += stride, ++lu) {
            const Unit t = list.next();
            const int b = lu % kNBuf;
            const int jend = min(t.rows, jbeg + kGroupCols);
            // MODE 1: lane i holds the y rows of the group's columns i, i + 32, ...
            int yrow[(kGroupCols + 31) / 32] = {};
            if (MODE == 1) {
#pragma unroll
                for (int i = 0; i < (kGroupCols + 31) / 32; ++i) {
                    const int j = jbeg + i * 32 + lane;
                    if (j < jend) {
                        yrow[i] = g.rows ? g.rows[t.row + j] : t.row + j;
                        if (!debug_in_range(yrow[i], 0, g.R, g.err)) yrow[i] = 0;
                    }
                }
            }
            const bool got = mbar_wait(&aux->tfull[b], (uint32_t)((lu / kNBuf) & 1), abort_flag);
            if (!got) flag_error();
            // same in all 4 warps; also: the group is done with the unit before's staging
            stopped = named_bar_or(1 + grp, 128, !got || *abort_flag);
            if (stopped) break;
            __syncwarp();
            tc_fence_after();
            const uint32_t acc = tmem_base + ((uint32_t)(lq * 32) << 16) + (uint32_t)(b * NT);
            if constexpr (MODE == 0) {
                // Warps 0 and 2 of a group hold the gates of 32 features, an MX block of act, and
                // warps 1 and 3 their ups.  Of every two column blocks the gate warp finishes the
                // first and the up warp the second: they swap the other halves through shared
                // memory.  A lane then has features lane / 4 + 0, 8, 16, 24 of tokens 2 (lane % 4)
                // and the next.
                const int up = lq & 1;
                uint8_t* const ex = staging + (warp - kEpiWarp0) * kWarpStaging;
                const uint8_t* const other = staging + ((warp ^ 1) - kEpiWarp0) * kWarpStaging;
                const int f = first_feature(t) + (lq >> 1) * 32;
                for (int c = 0; c < kBlocks && jbeg + c * 8 < jend; c += 2) {
                    // (past the last block the loads only keep the warps alike)
                    const int cb = c + up;                    // the block that this warp finishes
                    const int cg = min(c + 1 - up, kBlocks - 1);  // the one that it gives away
                    const uint32_t mine = acc + jbeg + min(cb, kBlocks - 1) * 8, give = acc + jbeg + cg * 8;
                    uint32_t own[8], gift[8];
                    tmem_ld_16x256(give, gift);
                    tmem_ld_16x256(give + (16u << 16), gift + 4);
                    tmem_ld_16x256(mine, own);
                    tmem_ld_16x256(mine + (16u << 16), own + 4);
                    tmem_ld_wait();
                    const int buf = (c & 2) * 512;
                    reinterpret_cast<uint4*>(ex + buf)[lane] = make_uint4(gift[0], gift[1], gift[2], gift[3]);
                    reinterpret_cast<uint4*>(ex + buf)[32 + lane] = make_uint4(gift[4], gift[5], gift[6], gift[7]);
                    named_bar_sync(3 + grp * 2 + (lq >> 1), 64);
                    const uint4 o0 = reinterpret_cast<const uint4*>(other + buf)[lane];
                    const uint4 o1 = reinterpret_cast<const uint4*>(other + buf)[32 + lane];
                    const uint32_t got8[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
                    if (cb >= kBlocks || jbeg + cb * 8 >= jend) continue;  // warp-uniform
                    float a[8];  // even: the first token
                    if (up) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            a[i] = swiglu(__uint_as_float(got8[i]), __uint_as_float(own[i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            a[i] = swiglu(__uint_as_float(own[i]), __uint_as_float(got8[i]));
                    }
                    // the largest magnitude's exponent is all that the scale takes: the upper halves
                    // of both tokens' maxima go through the reduction as one register
                    const uint32_t m0 = __float_as_uint(max_abs4(a[0], a[2], a[4], a[6]));
                    const uint32_t m1 = __float_as_uint(max_abs4(a[1], a[3], a[5], a[7]));
                    uint32_t m = __byte_perm(m0, m1, 0x7632);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const uint32_t s0 = scale_code(m << 16, kEmaxE4M3), s1 = scale_code(m & 0xFFFF0000u, kEmaxE4M3);
                    const float i0 = inverse_scale(min(s0, 254u)), i1 = inverse_scale(min(s1, 254u));
                    uint32_t q0 = e4m3x4(a[0] * i0, a[2] * i0, a[4] * i0, a[6] * i0);
                    uint32_t q1 = e4m3x4(a[1] * i1, a[3] * i1, a[5] * i1, a[7] * i1);
                    if (s0 == kNanScale) q0 = 0x7F7F7F7Fu;
                    if (s1 == kNanScale) q1 = 0x7F7F7F7Fu;
                    // Byte i of q0 and q1 is feature lane / 4 + 8 i.  Transposed over the 4 lanes
                    // whose lane / 4 differs in its lower 2 bits, a lane has 4 consecutive features
                    // from 8 (lane / 4 % 4) + 4 (lane / 16), and the warp stores whole 32-byte rows.
                    q0 = transpose_bytes(q0, lane >> 2), q1 = transpose_bytes(q1, lane >> 2);
                    const int j = jbeg + cb * 8 + (lane & 3) * 2;
                    uint8_t* const put = g.act + (size_t)(t.row + j) * g.N + f + (lane >> 2 & 3) * 8 + (lane >> 4) * 4;
                    if (j < jend) *reinterpret_cast<uint32_t*>(put) = q0;
                    if (j + 1 < jend) *reinterpret_cast<uint32_t*>(put + g.N) = q1;
                    if (lane < 4) {
                        uint8_t* const sc = g.act_scale + (size_t)(t.row + j) * (g.N / 32) + f / 32;
                        if (j < jend) sc[0] = (uint8_t)s0;
                        if (j + 1 < jend) sc[g.N / 32] = (uint8_t)s1;
                    }
                }
                __syncwarp();
                release(b);
            } else {
                // Drain this group's columns into registers as packed bf16 and hand them back,
                // then transpose 8 token rows of this warp's 32 features at a time through
                // its own 512 bytes of shared memory and store 16 bytes a lane.  The 16x256b
                // load gives a lane two tokens of feature lane / 4, which is the fragment that
                // a transposing stmatrix takes; 16-byte chunk c of row r lies at c ^ (r / 2), so
                // neither its 8 rows nor the reads share a bank.  No barrier but the warp's.
                uint32_t pk[kBlocks * 4];
                constexpr int kBatch = 4;  // column blocks per wait
#pragma unroll
                for (int c0 = 0; c0 < kBlocks; c0 += kBatch) {
                    uint32_t v[kBatch][8];
#pragma unroll
                    for (int c = c0; c < c0 + kBatch && c < kBlocks; ++c)
                        if (jbeg + c * 8 < jend) {
                            tmem_ld_16x256(acc + jbeg + c * 8, v[c - c0]);
                            tmem_ld_16x256(acc + (16u << 16) + jbeg + c * 8, v[c - c0] + 4);
                        }
                    tmem_ld_wait();
#pragma unroll
                    for (int c = c0; c < c0 + kBatch && c < kBlocks; ++c)
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
                for (int c = 0; c < kBlocks; ++c) {
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
        if (warp == kEpiWarp0) {
            // CTA 0 commits to both CTAs, and nothing else waits for the last arrivals in CTA 1, nor
            // for the ring's last ones in either: they must be in before the shared memory goes to
            // another CTA.  A lane for each stage's last fill and one for the last commit of all.
            // (After an abort the number of fills is not known; the last commit comes all the same,
            // at most one bounded wait after this CTA's own.)
            volatile int never = 0;
            const int fills = lu * num_kt;
            bool in = true;
            if (lane < kStages && !stopped && fills > lane)
                in = mbar_wait(&aux->empty[lane], (uint32_t)(((fills - lane - 1) / kStages) & 1), &never);
            if (lane == kStages) in = mbar_wait(&aux->drain, 0, &never, 3000000000ull);
            if (!in) flag_error();
            __syncwarp();
        }
    }

    // Neither CTA leaves before the other's threads have made their last arrival in it; tensor-core
    // arrivals are no thread's, and were waited for above.
    tc_fence_before();
    cluster_arrive();
    cluster_wait();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(C::kTmemCols)
                     : "memory");
    }
}

template <int MODE, int NT>
cudaError_t launch_nt(MxArgs g, cudaStream_t st)
{
    using C = Cfg<MODE, NT>;
    g.fb_count = (g.N + 2 * C::kFeatures - 1) / (2 * C::kFeatures);
    g.fb_magic = magic(g.fb_count);
    CUtensorMap tw, ta;
    cudaError_t e = weights_map(&tw, g.w, (uint64_t)g.E * g.N * (MODE == 0 ? 2 : 1), (uint64_t)g.K,
                                kWBoxRows<MODE>);
    if (e == cudaSuccess)
        e = MODE == 1 ? gemm::make_tmap_u8(&ta, g.a, (uint64_t)g.R, (uint64_t)g.K, C::kBRows, kBK)
                      : (ta = tw, e);
    if (e != cudaSuccess) return e;
    return launch_pairs<mx_grouped_kernel<MODE, NT>>(device_sms() / 2 * 2, kThreads, C::kSmem, st, tw, ta, g);
}

// Token rows per tile.  A tile that holds all of an expert's rows reads its weights once, and a
// wider tile than needed costs little (E = 32, N = K = 2048, 2 rows an expert: NT = 16 15.9 us,
// 64 16.1, 128 16.3, 208 18.5); beyond 64 the average decides: 64 rows an expert 128 19.8 us, 208
// 22.4; 128 rows 22.4 and 25.2; 160 rows 30.0 and 26.1; 256 rows 36.4 and 39.0; 400 rows 60.3 and 48.5.
// From 209 to 256 rows an expert both widths cut a group in two and 128 is the faster; the rule
// does not tell these from the rest above 128.
template <int MODE>
cudaError_t launch_mode(const MxArgs& g, int most, cudaStream_t st)
{
    if (most <= 16) return launch_nt<MODE, 16>(g, st);
    if (most <= 32) return launch_nt<MODE, 32>(g, st);
    if (most <= 64) return launch_nt<MODE, 64>(g, st);
    if (g.R <= 128LL * g.E) return launch_nt<MODE, 128>(g, st);
    return launch_nt<MODE, 208>(g, st);
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
    g.k_magic = magic(g.k);
    return mode == 0 ? launch_mode<0>(g, most, st) : launch_mode<1>(g, most, st);
}

}  // namespace moe
