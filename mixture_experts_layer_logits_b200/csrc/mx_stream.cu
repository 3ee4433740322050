// mx_stream.cu -- microscaled grouped products for few token rows per expert, where streaming
// the weights is the work.
//
//   MODE 0  act[p, f] = MX(silu(gate) * up) of x[rows[p] / k] with w13[e] rows f and I + f
//   MODE 1  y[rows[p] or p, f] = w[e] row f dotted with act (or any E4M3 rows) [p]
//
// Token rows are the M operand of the MMA and weight rows its N = 128 .. 256.  An MMA takes 90
// cycles or more to read its M operand, 131 for N = 256: weights as the M operand would stream
// at most 2 KB of packed codes per 125 cycles (with the scale copies), which is 4.5 TB/s for the
// card and was 36 us for T = 8, E = 128, k = 8, H = 2048, I = 768; as the N operand 4 KB per 131,
// above what HBM gives.  Only the first NT rows of the M = 128 operand are token rows.  The others
// are whatever follows in the stage (its weight codes): they end in accumulator lanes that
// nothing reads.
//
// One accumulator lane is one token, so a thread holds a token's features in its columns: SwiGLU,
// the MX blocks of act and the rows of y need no exchange between threads.
//
// Warp roles: 0 TMA; 1 TMEM and MMA issue; 2-3 and 12-13 scales; 4-11 epilogue;
// MODE 0: 14-15 gather of token rows (16-byte cp.async copies).
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
using gemm::silu_mul;

constexpr int kSfBytes = 512 + 1024;      // scales of the token rows and of the weight rows
constexpr int kTmemCols = 512;
constexpr int kAccCols = 192;             // two accumulators of up to 192 columns, or one of 256
constexpr int kSfCol0 = 2 * kAccCols;     // first scale column
constexpr int kEpiWarp0 = 4, kEpiWarps = 8, kGatherWarp0 = 14, kGatherWarps = 2;
constexpr int kThreads = 32 * (kGatherWarp0 + kGatherWarps);  // whole warpgroups; MODE 1 leaves two warps idle
constexpr int kMaxStages = 6;

// NT: token rows of a tile (128: all of M).
template <int MODE, int NT>
struct Cfg {
    // the most weight rows of a tile; 128 token rows leave room for five stages of 192 only
    static constexpr int kMaxN = NT == 128 ? 192 : 256;
    static constexpr int kWidths = kMaxN / 64 - 1;               // 256, 192, 128
    static constexpr int kATile = NT * kBK;
    static constexpr int kBTile = kMaxN * kBK;
    static constexpr int kStageBytes = (kATile + kBTile + kSfBytes + 1023) & ~1023;
    static constexpr int kFixed = 1024 + 512 + kTableBytes;
    static constexpr int kStagesRaw = (232448 - kFixed) / kStageBytes;
    static constexpr int kStages = kStagesRaw > kMaxStages ? kMaxStages : kStagesRaw;
    static constexpr int kSmem = kFixed + kStages * kStageBytes;
    static constexpr int kGIters = (NT * 8 + kGatherWarps * 32 - 1) / (kGatherWarps * 32);
    static_assert(kATile + kBTile >= 128 * kBK, "the M operand's 128 rows lie inside the stage");
    static_assert(kSfCol0 + kStages * kSfCols <= kTmemCols, "TMEM");
    static_assert(kStages >= 4 && NT % 16 == 0 && NT <= 128, "tile");
};

struct Aux {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

// Warp-wide load of 32 consecutive 32-bit TMEM columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
        "%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

template <int MODE, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    mx_stream_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
                     const MxArgs g)
{
    using C = Cfg<MODE, NT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    Aux* aux = reinterpret_cast<Aux*>(ring + C::kStages * C::kStageBytes);
    static_assert(sizeof(Aux) <= 512, "aux area");

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            // the expect_tx, one arrival per scale warp and per gather warp
            mbar_init(&aux->full[s], 1 + kScaleWarps + (MODE == 0 ? kGatherWarps : 0));
            mbar_init(&aux->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&aux->tfull[b], 1);
            mbar_init(&aux->tempty[b], kEpiWarps);
        }
        mbar_init(&aux->drain, 1);
        aux->abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_w);
        if (MODE == 1) tma_prefetch_desc(&tm_a);
    }
    if (warp == 1) {
        tmem_alloc(&aux->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    // The second product of the FFN (g.early) takes only act from the launch before it;
    // expert_offsets, rows and weights were complete before that launch passed its own
    // wait, so the tables and the first weight tiles need not wait for it.
    if (!g.early) pdl_wait();
    pdl_launch_dependents();
    tc_fence_before();
    const Groups groups = build_groups<kThreads>(
        g, NT, reinterpret_cast<int*>(ring + C::kStages * C::kStageBytes + 512));
    tc_fence_after();

    const uint32_t tmem_base = aux->tmem_base;
    volatile int* abort_flag = &aux->abort;
    auto flag_error = [&] {
        atomicExch(g.err, kDeviceErrorMagic);
        aux->abort = 1;
    };
    // Weight rows per tile, 256, 192 or 128: the fewest rounds of the grid, each as long as its
    // rows take to stream.  Per K tile that is about 2.95 cycles a row (all SMs sharing
    // HBM), and no less than 525, which the MMAs and the scale copies take whatever N.
    // T = 8, E = 128, k = 8, I = 768: 52 experts x 6 tiles of 256 are 3 rounds, x 8 of 192 also,
    // a quarter shorter.  One accumulator of 256 columns cannot take the next tile's MMAs
    // while it is read out, two of 192 can.
    const int tiles = groups.first[g.E];
    int nsel = 0;
    {
        int best = INT32_MAX;
#pragma unroll
        for (int i = 0; i < C::kWidths; ++i) {
            const int rounds = (tiles * g.fb_count[i] + (int)gridDim.x - 1) / (int)gridDim.x;
            const int cost = rounds * max(C::kMaxN - 64 * i, 178);
            if (cost < best) {
                best = cost;
                nsel = i;
            }
        }
    }
    const int n = C::kMaxN - 64 * nsel;               // weight rows per tile
    const int features = MODE == 0 ? n / 2 : n;    // output features per tile
    const int nbuf = n <= kAccCols ? 2 : 1;        // accumulators in flight
    const int fbs = nsel == 0 ? g.fb_count[0] : nsel == 1 ? g.fb_count[1] : g.fb_count[2];
    const uint32_t fb_magic = nsel == 0 ? g.fb_magic[0] : nsel == 1 ? g.fb_magic[1] : g.fb_magic[2];
    const int unit0 = (int)blockIdx.x, stride = (int)gridDim.x, units = tiles * fbs;
    const int num_kt = g.K / kBK;
    auto unit = [&](int u, int& e) { return groups.unit(u, fbs, fb_magic, e); };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        const uint64_t wpol = g.stream_weights ? l2_policy_evict_first() : l2_policy_evict_normal();
        const uint64_t tpol = l2_policy_evict_last();  // token rows are read again per feature block
        const uint32_t ring0 = smem_u32(ring);
        const uint32_t bytes = n * kRowTx + (MODE == 1 ? C::kATile : 0);
        int stage = 0, fills = 0, e = 0;
        uint32_t phase = 0;
        bool ok = true, dep = !(MODE == 1 && g.early);
        for (int u = unit0; u < units && ok; u += stride) {
            const Unit t = unit(u, e);
            const int f = t.fb * features;
            for (int kt = 0; kt < num_kt; ++kt) {
                ok = warp_agrees(mbar_wait(&aux->empty[stage], phase ^ 1u, abort_flag));
                if (!ok) break;
                const uint32_t st = ring0 + stage * C::kStageBytes;
                const uint32_t bar = smem_u32(&aux->full[stage]);
                if (elect_one()) {
                    mbar_arrive_expect_tx(&aux->full[stage], bytes);
#pragma unroll
                    for (int r = 0; r < C::kMaxN; r += kWBox<MODE>) {
                        if (r >= n) break;
                        // Rows past the expert's last are another's or zeros, and never stored;
                        // MODE 0's boxes past its last feature read its first ones instead.
                        int row = t.expert * g.N + f + r;
                        if (MODE == 0) {
                            const int at = f + tile_feature(r);
                            row = t.expert * 2 * g.N + (at < g.N ? at : 0) + (tile_row_is_up(r) ? g.N : 0);
                        }
                        tma_2d<1>(st + C::kATile + r * kBK, &tm_w, bar, kt * kBK, row, wpol);
                    }
                }
                if (MODE == 1) {
                    if (!dep) {
                        pdl_wait();
                        dep = true;
                    }
                    __syncwarp();
                    if (elect_one()) tma_2d<1>(st, &tm_a, bar, kt * kBK, t.row, tpol);
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
            // let every TMA load already issued land before the CTA can exit
            for (int s = 0; s < C::kStages; ++s) {
                const int k = fills > s ? (fills - s + C::kStages - 1) / C::kStages : 0;
                if (k > 0) {
                    volatile int never = 0;
                    mbar_wait(&aux->full[s], (uint32_t)((k - 1) & 1), &never, 500000000ull);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        int stage = 0, lu = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t ring0 = smem_u32(ring);
        const uint32_t idesc = idesc_formats(false) | idesc_shape(128, n);
        for (int u = unit0; u < units && ok; u += stride, ++lu) {
            const int b = nbuf == 2 ? lu & 1 : 0, use = nbuf == 2 ? lu >> 1 : lu;
            ok = warp_agrees(mbar_wait(&aux->tempty[b], (uint32_t)(use & 1) ^ 1u, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem_base + (uint32_t)(b * kAccCols);
            for (int kt = 0; kt < num_kt; ++kt) {
                ok = warp_agrees(mbar_wait(&aux->full[stage], phase, abort_flag));
                if (!ok) break;
                tc_fence_after();
                const uint32_t sa = ring0 + stage * C::kStageBytes;
                const uint32_t sb = sa + C::kATile, sf = sb + C::kBTile;
                const uint32_t tsf = tmem_base + (uint32_t)(kSfCol0 + stage * kSfCols);
                const uint64_t da = umma_desc_sw128(sa), db = umma_desc_sw128(sb);
                const uint64_t ds = scale_desc(sf);
                if (elect_one()) {
                    if (MODE == 0) fence_proxy_async_smem();  // the token rows came by cp.async
                    scales_to_tmem<1>(tsf, ds);
                    scales_to_tmem<1>(tsf + 4, ds + (512 >> 4));
                    if (n > 128) scales_to_tmem<1>(tsf + 8, ds + (1024 >> 4));
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk)  // 32 bytes along K
                        umma<1>(d, da + 2 * kk, db + 2 * kk, idesc | idesc_kb(kk), tsf, tsf + 4,
                                (kt | kk) ? 1u : 0u);
                    umma_commit(&aux->empty[stage]);
                    if (kt + 1 == num_kt) umma_commit(&aux->tfull[b]);
                }
                __syncwarp();
                if (++stage == C::kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) flag_error();
        __syncwarp();
        // all MMAs and copies issued by this warp are complete before TMEM is freed
        if (elect_one()) umma_commit(&aux->drain);
        __syncwarp();
        volatile int never = 0;
        if (!mbar_wait(&aux->drain, 0, &never, 500000000ull)) atomicExch(g.err, kDeviceErrorMagic);
    } else if (warp == 2 || warp == 3 || warp == 12 || warp == 13) {
        // ------------------------------------------------------------ scales
        // Thread i handles weight rows i and i + 128 of the tile and token row i.
        const int i0 = (warp < 4 ? warp - 2 : warp - 10) * 32 + lane;
        const size_t ld = (size_t)g.K / 32;
        if (MODE == 1 && g.early) pdl_wait();  // act's scales
        constexpr int kRows = 3;
        const int put[kRows] = {(int)(512 + scale_place(i0)), i0 + 128 < n ? (int)(512 + scale_place(i0 + 128)) : -1,
                                i0 < NT ? (int)scale_place(i0) : -1};
        int e = 0, tok;
        Unit next;
        auto fetch = [&](int u) {
            next = unit(u, e);
            // past the tile's end any scale will do
            tok = next.row + min(i0, next.rows - 1);
            if (MODE == 0) {
                tok = g.rows[tok];
                if (!debug_in_range(tok, 0, g.R, g.err)) tok = 0;
            }
        };
        auto sources = [&](int, const uint8_t* (&src)[kRows]) {
            // rows past the expert's last belong to features that are never stored
            const int f = next.fb * features;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = i0 + i * 128;
                const int row = MODE == 0 ? next.expert * 2 * g.N + min(f + tile_feature(r), g.N - 1) +
                                                (tile_row_is_up(r) ? g.N : 0)
                                          : next.expert * g.N + min(f + r, g.N - 1);
                src[i] = g.w_scale + (size_t)row * ld;
            }
            src[2] = g.a_scale + (size_t)(MODE == 0 ? div_by(tok, g.k, g.k_magic) : tok) * ld;
        };
        run_scales<kRows>(
            unit0, stride, units, num_kt, (int)ld, put, fetch, sources,
            [&](int q) {
                const bool ok = warp_agrees(mbar_wait(&aux->empty[q % C::kStages],
                                                                  (uint32_t)((q / C::kStages) & 1) ^ 1u,
                                                                  abort_flag));
                if (!ok && lane == 0) flag_error();
                return ok;
            },
            [&](int q) { return ring + (q % C::kStages) * C::kStageBytes + C::kATile + C::kBTile; },
            [&](int q) {
                if (lane == 0) mbar_arrive(&aux->full[q % C::kStages]);
            });
    } else if (MODE == 0 && warp >= kGatherWarp0) {
        // ------------------------------------------------------------ gather (MODE 0)
        // Thread i copies the 16-byte chunks i, i + 64, ... of the tile's token rows (8 chunks a
        // row) to their swizzled places; the copies arrive on the stage's barrier when they
        // land, and the MMA warp fences the async proxy.
        const int i0 = threadIdx.x - kGatherWarp0 * 32;
        const uint64_t pol = l2_policy_evict_last();
        int q = 0, e = 0;
        bool ok = true;
        int r[C::kGIters];
        auto next_rows = [&](int u) {
            if (u >= units) return;
            const Unit t = unit(u, e);
#pragma unroll
            for (int i = 0; i < C::kGIters; ++i) {
                const int j = (i0 + i * kGatherWarps * 32) >> 3;
                r[i] = -1;
                if (j < t.rows) {
                    r[i] = g.rows[t.row + j];
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
                const int stage = q % C::kStages;
                const uint32_t phase = (uint32_t)((q / C::kStages) & 1);
                ok = warp_agrees(mbar_wait(&aux->empty[stage], phase ^ 1u, abort_flag));
                if (!ok) {
                    if (lane == 0) flag_error();
                    break;
                }
                const uint32_t sa = smem_u32(ring + stage * C::kStageBytes);
#pragma unroll
                for (int i = 0; i < C::kGIters; ++i) {
                    const int c = i0 + i * kGatherWarps * 32, j = c >> 3;
                    if (src[i])
                        cp_async_16_hint(sa + j * 128 + (((c & 7) ^ (j & 7)) << 4), src[i] + kt * kBK, pol);
                }
                cp_async_mbar_arrive(&aux->full[stage]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&aux->full[stage]);
            }
        }
        cp_async_commit();
        cp_async_wait<0>();  // no copy is still in flight when the CTA exits
    } else if (warp >= kEpiWarp0 && warp < kEpiWarp0 + kEpiWarps) {
        // ------------------------------------------------------------ epilogue
        // Two warps per lane quarter take the column blocks in turn.
        const int grp = (warp - kEpiWarp0) >> 2;
        const int lq = warp & 3;
        const int j = lq * 32 + lane;  // token row of the tile
        int lu = 0, e = 0;
        for (int u = unit0; u < units; u += stride, ++lu) {
            const Unit t = unit(u, e);
            const int b = nbuf == 2 ? lu & 1 : 0, use = nbuf == 2 ? lu >> 1 : lu;
            const bool live = j < t.rows;
            int p = t.row + min(j, t.rows - 1);
            if (MODE == 1 && g.rows) {
                p = g.rows[p];
                if (!debug_in_range(p, 0, g.R, g.err)) p = 0;
            }
            const bool got = mbar_wait(&aux->tfull[b], (uint32_t)(use & 1), abort_flag);
            if (!warp_agrees(got)) {
                if (lane == 0) flag_error();
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem_base + ((uint32_t)(lq * 32) << 16) + (uint32_t)(b * kAccCols);
            const int f0 = t.fb * features;
            if (lq * 32 < t.rows) {  // warp-uniform
                if constexpr (MODE == 0) {
                    // 64 columns are 32 features, one MX block: 32 gates, then 32 ups
                    for (int blk = grp; blk * 64 < n; blk += 2) {
                        if (f0 + blk * 32 >= g.N) break;
                        float act[32];
                        uint32_t m = 0;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t v[16], w[16];
                            tmem_ld16(acc + blk * 64 + h * 16, v);
                            tmem_ld16(acc + blk * 64 + 32 + h * 16, w);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float a = silu_mul(__uint_as_float(v[i]), __uint_as_float(w[i]));
                                act[h * 16 + i] = a;
                                m = max(m, __float_as_uint(a) & 0x7FFFFFFFu);
                            }
                        }
                        const uint32_t code = scale_code(m, kEmaxE4M3);
                        const float inv = inverse_scale(min(code, 254u));
                        uint32_t q[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            q[i] = code == kNanScale ? 0x7F7F7F7Fu
                                                     : e4m3x4(act[4 * i] * inv, act[4 * i + 1] * inv,
                                                              act[4 * i + 2] * inv, act[4 * i + 3] * inv);
                        if (live) {
                            uint4* const dst = reinterpret_cast<uint4*>(g.act + (size_t)p * g.N + f0 + blk * 32);
                            dst[0] = make_uint4(q[0], q[1], q[2], q[3]);
                            dst[1] = make_uint4(q[4], q[5], q[6], q[7]);
                            g.act_scale[(size_t)p * (g.N / 32) + f0 / 32 + blk] = (uint8_t)code;
                        }
                        __syncwarp();
                    }
                } else {
                    for (int c = grp * 32; c < n; c += 64) {
                        if (f0 + c >= g.N) break;
                        uint32_t v[32];
                        tmem_ld32(acc + c, v);
                        tmem_ld_wait();
                        __nv_bfloat16* const dst = static_cast<__nv_bfloat16*>(g.y) + (size_t)p * g.N + f0 + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(
                                    __uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
                                w[k] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                            if (live && f0 + c + i < g.N)
                                *reinterpret_cast<uint4*>(dst + i) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        __syncwarp();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&aux->tempty[b]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

template <int MODE, int NT>
cudaError_t launch_nt(MxArgs g, cudaStream_t st)
{
    using C = Cfg<MODE, NT>;
    for (int i = 0; i < C::kWidths; ++i) {
        const int features = (C::kMaxN - 64 * i) / (MODE == 0 ? 2 : 1);
        g.fb_count[i] = (g.N + features - 1) / features;
        g.fb_magic[i] = magic(g.fb_count[i]);
    }
    CUtensorMap tw, ta;
    cudaError_t e = weights_map(&tw, g.w, (uint64_t)g.E * g.N * (MODE == 0 ? 2 : 1), (uint64_t)g.K,
                                kWBox<MODE>);
    if (e == cudaSuccess)
        e = MODE == 1 ? gemm::make_tmap_u8(&ta, g.a, (uint64_t)g.R, (uint64_t)g.K, NT, kBK) : (ta = tw, e);
    if (e != cudaSuccess) return e;
    return launch<mx_stream_kernel<MODE, NT>>(device_sms(), 1, kThreads, C::kSmem, st, tw, ta, g);
}

template <int MODE>
cudaError_t launch_mode(const MxArgs& g, int most, cudaStream_t st)
{
    if (most <= 16) return launch_nt<MODE, 16>(g, st);
    if (most <= 32) return launch_nt<MODE, 32>(g, st);
    if (most <= 64) return launch_nt<MODE, 64>(g, st);
    return launch_nt<MODE, 128>(g, st);
}

}  // namespace

cudaError_t launch_mx_pair(const MxArgs& g, int mode, cudaStream_t st);

cudaError_t launch_mx_grouped(const MxArgs& args, int mode, cudaStream_t st)
{
    MxArgs g = args;
    // the most rows that one expert can have: a token picks an expert at most once
    const int most = mode == 2 ? g.R : g.R / g.k;
    g.early = mode == 1;
    g.stream_weights = most <= 128;
    if (mode == 2) {
        g.rows = nullptr;
        g.k = 1;
    }
    g.k_magic = magic(g.k);
    if (g.R >= 128 * g.E) return launch_mx_pair(g, mode == 0 ? 0 : 1, st);
    return mode == 0 ? launch_mode<0>(g, most, st) : launch_mode<1>(g, most, st);
}

}  // namespace moe
