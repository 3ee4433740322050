// mx_gemm.cuh -- building blocks of the microscaled grouped products (mx_grouped.cu): block-scaled
// MMA wrappers, the tiles of the groups, the scale loader, tensor maps and the launch.
//
//   D[f, j] = sum_b 2^(sw[f, b] + sa[j, b] - 254) sum_{i in block b} w[f, i] a[j, i]
//
// with E2M1 weights w, E4M3 token rows a, blocks of 32 and E8M0 scales.  Products of codes and
// their power-of-two scales are exact, so only the fp32 sums round.
//
// Weights lie in shared memory one byte an element: TMA unpacks the 4-bit codes to the
// slots that a mixed E2M1 x E4M3 MMA reads, so HBM and L2 move half a byte an element.
//
// A K tile of 128 has 4 scale bytes per row.  They are laid out as tcgen05.cp spreads them
// over tensor memory (row r of 128 at byte 16 (r % 32) + 4 (r / 32) of 512).  Every ring
// stage has its own scale columns in tensor memory, so a stage's copy never has to wait for
// another stage's MMAs.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "gemm_common.cuh"
#include "kernels.h"
#include "mx_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace mx {

constexpr int kBK = 128;                    // K elements per stage: one 128-byte swizzle row
constexpr int kMaxExperts = 1024;
constexpr int kRowTx = kBK / 2;             // an unpacking TMA load counts its packed bytes
constexpr int kTableBytes = 2 * (kMaxExperts + 1) * 4 + 120;

// ------------------------------------------------------------------ PTX

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

// The outcome of a wait that every lane of a warp polled for itself, agreed on by all.  The
// lanes may leave their polling loops at different times, and neither the loop nor the vote
// promises that the warp runs converged afterwards, which elect.sync and the .aligned
// tensor instructions after it need: hence the __syncwarp.
__device__ __forceinline__ bool warp_agrees(bool ok)
{
    ok = __all_sync(0xffffffffu, ok);
    __syncwarp();
    return ok;
}

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

// D (+)= A B^T with scales, one MMA of a pair of CTAs (cta_group::2).
__device__ __forceinline__ void umma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate)
{
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

// Copies them to 4 TMEM columns, the same 32 lanes' worth in every lane quarter, ordered
// before later MMAs of this thread.  Each CTA of the pair copies from its own shared memory to
// its own TMEM.
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// 2D TMA load of a box at (c, row) into this CTA's shared memory, whose bytes count on `bar`,
// which may lie in the other CTA of the pair.
__device__ __forceinline__ void tma_2d(uint32_t dst, const void* tmap, uint32_t bar, int c, int row,
                                       uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2.L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c), "r"(row), "l"(policy)
        : "memory");
}

// ------------------------------------------------------------------ groups and tiles

// n / d for 0 <= n < 2^31 by a multiplication with m = floor(2^32 / d) + 1 (d = 1: m = 0).
// The product can be one too large where n d is large; that is put right.
__device__ __forceinline__ int div_by(int n, int d, uint32_t m)
{
    int q = d == 1 ? n : (int)__umulhi((uint32_t)n, m);
    if (q * d > n) --q;
    return q;
}

// A tile: `rows` token rows from `row`, the feature block `fb` of `expert`.
struct Unit {
    int expert, fb, row, rows;
};

// The groups of a call, derived from expert_offsets by every CTA itself, so that there is no
// tile list and no launch for one.
struct Groups {
    const int* first;  // [E + 1] tiles before each expert
    const int* start;  // [E + 1] rows before each expert
    int E;
};

// The units u0, u0 + stride, ... of tiles x fbs, one after the other: experts in order; within one,
// feature block major and tile minor, so the tiles that share a weight block run at the same time
// on neighbouring CTAs and share it in L2.  A group of c rows in t tiles is cut evenly (to 16 rows).
// The lanes look 32 units up at once and hand them out by shuffles: one look-up is a chain of
// shared-memory reads and divisions of some 600 cycles, more than a K tile's MMAs take.
struct Units {
    Groups g;
    int fbs, units, stride, u;
    uint32_t fb_magic;
    int at;     // 0 .. 31: next lane to hand out
    Unit mine;

    __device__ __forceinline__ Units(const Groups& groups, int fb_count, uint32_t magic, int u0, int step)
        : g(groups), fbs(fb_count), units(groups.first[groups.E] * fb_count), stride(step), u(u0), fb_magic(magic),
          at(32)
    {
    }

    // All 32 lanes take part.  (Past the last unit: the last one again.)
    __device__ __forceinline__ Unit next()
    {
        if (at == 32) {
            look_up(min(u + (int)(threadIdx.x & 31) * stride, units - 1));
            u = min(u + 32 * stride, units - 1);
            at = 0;
        }
        Unit t;
        t.expert = __shfl_sync(0xffffffffu, mine.expert, at);
        t.fb = __shfl_sync(0xffffffffu, mine.fb, at);
        t.row = __shfl_sync(0xffffffffu, mine.row, at);
        t.rows = __shfl_sync(0xffffffffu, mine.rows, at);
        ++at;
        return t;
    }

    __device__ __forceinline__ void look_up(int v)
    {
        const int rest = div_by(v, fbs, fb_magic);
        int e = 0;  // to the last e with first[e] <= rest
        for (int step = 1 << (31 - __clz(g.E)); step; step >>= 1)
            if (e + step < g.E && g.first[e + step] <= rest) e += step;
        const int local = v - g.first[e] * fbs, count = g.first[e + 1] - g.first[e];
        const int rows = g.start[e + 1] - g.start[e];
        mine.expert = e;
        mine.fb = local;
        mine.row = g.start[e];
        mine.rows = rows;
        if (count > 1) {
            const int per = ((rows + count - 1) / count + 15) & ~15;
            mine.fb = local / count;
            const int from = (local - mine.fb * count) * per;
            mine.row += from;
            mine.rows = min(per, rows - from);
        }
    }
};

// A thread's share of expert_offsets: those of experts threadIdx.x * kPer + i, and the next.
// Read on their own so that their way from L2 passes under the rest of the prologue.
template <int kThreads>
struct Offsets {
    static constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
    int v[kPer + 1];

    __device__ __forceinline__ void read(const MxArgs& g)
    {
#pragma unroll
        for (int i = 0; i <= kPer; ++i) {
            const int e = threadIdx.x * kPer + i;
            v[i] = e <= g.E ? __ldcg(g.offsets + e) : 0;
        }
    }
};

// Fills first / start (kTableBytes of shared memory at `tables`) for tiles of up to nt rows.
// Offsets are clamped to 0 .. R and to ascending order, so that none leads outside the
// operands.  All kThreads threads call it; it ends with a barrier.
template <int kThreads>
__device__ __forceinline__ Groups build_groups(const MxArgs& g, const Offsets<kThreads>& off, int nt,
                                               int* tables)
{
    int* first = tables;
    int* start = tables + kMaxExperts + 1;
    int* warp_sum = start + kMaxExperts + 1;
    constexpr int kPer = Offsets<kThreads>::kPer;
    static_assert(kThreads / 32 * 4 <= 120, "warp_sum");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int tiles[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        tiles[i] = 0;
        if (e < g.E) {
            const int a = min(max(off.v[i], 0), g.R);
            const int b = min(max(off.v[i + 1], a), g.R);
            start[e] = a;
            if (e == g.E - 1) start[g.E] = b;
            tiles[i] = (b - a + nt - 1) / nt;
        }
        sum += tiles[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int ws = lane < kThreads / 32 ? warp_sum[lane] : 0, wincl = ws;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, wincl, o);
        if (lane >= o) wincl += v;
    }
    int before = incl - sum + __shfl_sync(0xffffffffu, wincl - ws, warp);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        if (e < g.E) first[e] = before;
        before += tiles[i];
        if (e == g.E - 1) first[g.E] = before;
    }
    __syncthreads();
    return Groups{first, start, g.E};
}

// ------------------------------------------------------------------ scales

// Byte of row r's 4 scales in a K tile's layout.
__device__ __forceinline__ uint32_t scale_place(int r)
{
    return (uint32_t)((r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4);
}

// Feature of row r of a MODE 0 tile, without the feature block's part, and whether the row is its
// up row: 32 gate rows, their 32 up rows, and so on.
__device__ __forceinline__ int tile_feature(int r) { return r / 64 * 32 + r % 32; }
__device__ __forceinline__ bool tile_row_is_up(int r) { return r / 32 % 2; }

// The kScaleWarps warps that bring scales into the ring.  Reading 4 bytes a row and K tile costs one
// L1 line lookup and a 32-byte sector each time (as cp.async copies that was 0.58 of the 2.53 ms
// of the FFN at T = 8192), so a row is read a group of 8 K tiles at a time (32 bytes; in 16-byte loads
// where the row pitch allows it) into registers, one group ahead, and stored 4 bytes a stage.
// The rows are split over four warps: a stage costs a warp some 200 cycles whatever it stores (the
// wait, the fence towards tcgen05.cp's proxy, the arrival), and the fence waits for the loads ahead
// too, 440 cycles a stage in all at T = 8192 (where a K tile takes 540 to 580).  Loads later in the
// group cost 10%, several stages under one fence 4% (T = 64, E = 256).
//   units       unit0, unit0 + stride, ... below `units`, each of num_kt K tiles
//   kRows       rows of this thread; put[i]: where row i's bytes go within a stage's scales,
//               or -1
//   fetch(u)    starts reading what sources(u) needs
//   sources(u, src)  sets the rows' first scale bytes for unit u
//   wait(q)     waits until ring fill q may be written (false: give up)
//   stage(q)    shared memory of that fill's scales
//   arrive(q)   called by every lane after its warp's stores are fenced
// The launch before, which may still run when this one begins, may have written the scales (act's, or
// those of a quantised matrix), so the loads are coherent ones; they follow the wait for that launch.
constexpr int kScaleWarps = 4;
template <int kRows, typename Fetch, typename Sources, typename Wait, typename Stage, typename Arrive>
__device__ __forceinline__ void run_scales(int unit0, int stride, int units, int num_kt, int row_bytes,
                                           const int (&put)[kRows], Fetch fetch, Sources sources, Wait wait,
                                           Stage stage, Arrive arrive)
{
    if (unit0 >= units) return;
    const int align = row_bytes & 15;  // 0: 16-byte rows, 8: 8-byte, else 4-byte
    const uint8_t* src[kRows];
    uint32_t next[kRows][8];
    auto read = [&](int kt) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (put[i] < 0) continue;
            const uint8_t* s = src[i] + kt * 4;
            if (align == 0) {
#pragma unroll
                for (int j = 0; j < 8; j += 4)
                    if (kt + j < num_kt) {
                        const uint4 v = __ldca(reinterpret_cast<const uint4*>(s + 4 * j));
                        next[i][j] = v.x, next[i][j + 1] = v.y, next[i][j + 2] = v.z, next[i][j + 3] = v.w;
                    }
            } else if (align == 8) {
#pragma unroll
                for (int j = 0; j < 8; j += 2)
                    if (kt + j < num_kt) {
                        const uint2 v = __ldca(reinterpret_cast<const uint2*>(s + 4 * j));
                        next[i][j] = v.x, next[i][j + 1] = v.y;
                    }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (kt + j < num_kt) next[i][j] = __ldca(reinterpret_cast<const uint32_t*>(s + 4 * j));
            }
        }
    };
    fetch(unit0);
    sources(unit0, src);
    read(0);
    int q = 0;
    for (int u = unit0; u < units; u += stride) {
        if (u + stride < units) fetch(u + stride);
        for (int kt = 0; kt < num_kt; kt += 8) {
            uint32_t cur[kRows][8];
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) cur[i][j] = next[i][j];
            if (kt + 8 < num_kt) {
                read(kt + 8);
            } else if (u + stride < units) {
                sources(u + stride, src);
                read(0);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (kt + j >= num_kt) break;
                if (!wait(q)) return;
                uint8_t* const sf = stage(q);
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (put[i] >= 0) *reinterpret_cast<uint32_t*>(sf + put[i]) = cur[i][j];
                fence_proxy_async_smem();
                __syncwarp();
                arrive(q);
                ++q;
            }
        }
    }
}

// ------------------------------------------------------------------ host side

inline uint32_t magic(int d) { return d > 1 ? (uint32_t)((1ull << 32) / (unsigned)d + 1) : 0u; }

// E2M1 codes [rows, cols / 2]: boxes of box_rows x 128 elements, unpacked to one byte slot an
// element with the 128-byte swizzle.
inline cudaError_t weights_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols,
                               uint32_t box_rows)
{
    gemm::EncodeTiledFn fn = gemm::get_encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols / 2};
    const cuuint32_t box[2] = {(cuuint32_t)kBK, box_rows};
    const cuuint32_t ones[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<void*>(base), dims,
                          strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Launches kern as pairs of CTAs.
template <auto kern>
cudaError_t launch_pairs(int grid, int threads, int smem, cudaStream_t st, const CUtensorMap& tw,
                         const CUtensorMap& ta, const MxArgs& g)
{
    // the attribute stays with the kernel (one `done` per instantiation), so it is set once a device
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(done.load(std::memory_order_relaxed) & bit) || !bit) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, tw, ta, g);
}

}  // namespace mx
}  // namespace moe
