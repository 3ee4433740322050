// mx_quant.cu -- the HBM-bound producers of microscaled rows: quantisation of a
// matrix, and the residual addition with root-mean-square norm.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "mx_common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

__device__ __forceinline__ void unpack_bf16x8(const uint4& q, float (&v)[8])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------------ quantisation

// A matrix whose columns are a multiple of 32 is a run of blocks, whatever its rows:
// four consecutive threads hold one block, 8 elements each.  HBM-bound; a thread has U
// chunks' loads in flight before it uses the first (201 M bf16 elements to E2M1: U = 1
// 104 us, 2 86 us, 4 78.5 us, which is the measured copy rate, 8 80 us).  An fp32 chunk is two
// loads and needs no more (134 M elements to E4M3: U = 1 98.9 us, the measured copy rate, 2 100.8).
// The launch before, which may still run when this one begins, may write the inputs of both kernels
// here: their loads are coherent ones behind pdl_wait, never read-only ones.
template <bool E2M1, typename Src, int U>
__global__ void __launch_bounds__(256)
    quantize_kernel(const Src* src, long chunks, uint8_t* __restrict__ codes,
                    uint8_t* __restrict__ scales)
{
    pdl_launch_dependents();
    pdl_wait();
    const long c0 = (long)blockIdx.x * (256 * U) + threadIdx.x;  // 8-element chunks c0 + 256 u
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long c = min(c0 + 256 * u, chunks - 1);
        if constexpr (sizeof(Src) == 2) {
            unpack_bf16x8(__ldcs(reinterpret_cast<const uint4*>(src) + c), v[u]);
        } else {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(src) + 2 * c);
            const float4 b = __ldcs(reinterpret_cast<const float4*>(src) + 2 * c + 1);
            v[u][0] = a.x, v[u][1] = a.y, v[u][2] = a.z, v[u][3] = a.w;
            v[u][4] = b.x, v[u][5] = b.y, v[u][6] = b.z, v[u][7] = b.w;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long c = c0 + 256 * u;
        uint2 q;
        const uint32_t s = mx::quantize8<E2M1>(v[u], mx::max_bits(v[u]), q);
        if (c >= chunks) continue;
        if constexpr (E2M1)
            reinterpret_cast<uint32_t*>(codes)[c] = q.x;
        else
            reinterpret_cast<uint2*>(codes)[c] = q;
        if ((c & 3) == 0) scales[c >> 2] = (uint8_t)s;
    }
}

// ------------------------------------------------------------------ norm

// The sum of v over the CTA, in every thread.  `part`: 32 floats of shared memory.
__device__ __forceinline__ float block_sum(float v, float* part)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < (blockDim.x >> 5) ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One row per CTA.  h = x + residual rounded to bf16 (that is what the next layer
// reads, so the norm is the norm of the stored sum), r = 1 / sqrt(mean(h^2) + eps),
// n = (h * weight) * r: the product of two bf16 values is exact in fp32, so n carries
// the rounding of r and of one product.  Sums are fp32.  A row whose mean square is not
// 2^-24 .. 2^24, or whose weights are so large that h * weight overflows, is done again: h first
// takes the power of two that brings the root mean square to 2^-14 .. 2^-13, and r the opposite
// one, so that h * weight is out of fp32's range only where n is, or is below bf16's.
template <int C>
__global__ void __launch_bounds__(1024, C <= 4 ? 2 : 1)
    rmsnorm_kernel(const uint4* x, const uint4* residual, const uint4* weight, int chunks, float inv_h, float eps,
                   uint4* sum, uint4* __restrict__ out, uint8_t* __restrict__ codes,
                   uint8_t* __restrict__ scales)
{
    __shared__ float part[32];
    pdl_launch_dependents();
    pdl_wait();
    const size_t base = (size_t)blockIdx.x * chunks;
    uint4 h[C];
    float ss = 0.f;
    // Chunks whose loads are in flight together (8192 x 4096 with residual: one by one 51.1 us, two
    // 46.6).  More of them take registers that CTAs need (32768 columns: 740 rows 42.2 us, with four
    // and half the CTAs 40.5, but 296 rows 16.0 and 17.4).
    constexpr int kBatch = C < 2 ? C : 2;
#pragma unroll
    for (int i0 = 0; i0 < C; i0 += kBatch) {
        uint4 add[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int c = threadIdx.x + (i0 + i) * blockDim.x;
            if (c >= chunks) continue;
            h[i0 + i] = __ldcg(x + base + c);
            if (residual) add[i] = __ldcg(residual + base + c);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int c = threadIdx.x + (i0 + i) * blockDim.x;
            if (c >= chunks) continue;
            float v[8];
            unpack_bf16x8(h[i0 + i], v);
            if (residual) {
                float r[8];
                unpack_bf16x8(add[i], r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += r[j];
                h[i0 + i] = pack_bf16x8(v);
                sum[base + c] = h[i0 + i];
                unpack_bf16x8(h[i0 + i], v);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
        }
    }
    float m = fmaf(block_sum(ss, part), inv_h, eps);
    auto put = [&](int c, bool live, const float (&v)[8]) {  // whether n's chunk c has a NaN or an infinity
        if (live && out) out[base + c] = pack_bf16x8(v);
        if (!codes) return mx::max_bits(v) >= 0x7F800000u;
        uint2 q;
        const uint32_t s = mx::quantize8<false>(v, mx::max_bits(v), q);
        if (live) {
            reinterpret_cast<uint2*>(codes)[base + c] = q;
            if ((c & 3) == 0) scales[(base + c) >> 2] = (uint8_t)s;
        }
        return s == mx::kNanScale;
    };
    if (m >= 0x1p-24f && m <= 0x1p24f) {  // the same in every thread
        const float r = 1.0f / sqrtf(m);
        bool over = false;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            const bool live = c < chunks;
            float v[8] = {};
            if (live) {
                float w[8];
                unpack_bf16x8(h[i], v);
                unpack_bf16x8(__ldca(weight + c), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = v[j] * w[j] * r;
            }
            over |= put(c, live, v);
        }
        if (!__any_sync(0xffffffffu, over)) return;
    }

    // Rows and weights of any size, from memory again: this costs the rows above no registers.
    const uint4* const row = (residual ? sum : x) + base;
    float scale = 1.0f;
    if (!(m >= 0x1p-100f && m < INFINITY)) {  // the same in every thread
        // Squares left the range of fp32, or they and eps lie so low that what underflowed would
        // count: once more for the row times a power of two (a NaN or an infinity stays one).
        scale = m < 1.0f ? 0x1p80f : 0x1p-80f;
        ss = 0.f;
#pragma unroll 1
        for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
            float v[8];
            unpack_bf16x8(__ldcg(row + c), v);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[j] * scale, v[j] * scale, ss);
        }
        __syncthreads();  // `part` has been read
        m = fmaf(block_sum(ss, part), inv_h, eps * scale * scale);
    }
    // m = f 4^k with f in [1/4, 1).  The 2^-13 keeps `down` in range for a row of one element 2^-133.
    const int k = ((int)(__float_as_uint(m) >> 23 & 255) - 127 + 2) >> 1;
    const float down = scale * __uint_as_float((uint32_t)(127 - 13 - k) << 23);
    const float r = 1.0f / sqrtf(m) * __uint_as_float((uint32_t)(127 + 13 + k) << 23);
#pragma unroll 1
    for (int i = 0; i < C; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        const bool live = c < chunks;
        float v[8] = {};
        if (live) {
            float w[8];
            unpack_bf16x8(__ldcg(row + c), v);
            unpack_bf16x8(__ldca(weight + c), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = v[j] * down * w[j] * r;
        }
        put(c, live, v);
    }
}

template <int C>
cudaError_t launch_norm(const NormArgs& a, int threads, cudaStream_t st)
{
    return launch_pdl(rmsnorm_kernel<C>, dim3(a.T), dim3(threads), 0, st,
                      static_cast<const uint4*>(a.x), static_cast<const uint4*>(a.residual),
                      static_cast<const uint4*>(a.weight), a.H / 8, 1.0f / (float)a.H, a.eps,
                      static_cast<uint4*>(a.sum), static_cast<uint4*>(a.out), a.codes, a.scales);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t st)
{
    const int chunks = a.H / 8;
    // Chunks of 8 elements a thread: one where there are few rows, two where rows fill the SMs several
    // times and a CTA keeps 128 threads or more (with residual and blocks, one and two: 64 x 7168 2.9 and
    // 3.1 us, 740 x 4096 6.1 and 6.5, 888 x 4096 6.8 and 7.0, 1184 x 4096 8.4 and 7.6, 1036 x 7168 13.4 and
    // 11.0, 4096 x 7168 50.4 and 42.3), more only as 1024 threads cannot do without.
    const bool many = a.T >= 7 * device_sms() && chunks > 256;
    const int c = max((chunks + 1023) / 1024, many ? 2 : 1);
    const int cc = c <= 2 ? c : c <= 4 ? 4 : 8;
    const int threads = ((chunks + cc - 1) / cc + 31) & ~31;
    if (cc == 1) return launch_norm<1>(a, threads, st);
    if (cc == 2) return launch_norm<2>(a, threads, st);
    if (cc == 4) return launch_norm<4>(a, threads, st);
    return launch_norm<8>(a, threads, st);
}

template <bool E2M1, typename Src, int U>
static cudaError_t launch_quantize(const void* src, long chunks, uint8_t* codes, uint8_t* scales,
                                   cudaStream_t st)
{
    return launch_pdl(quantize_kernel<E2M1, Src, U>, dim3((unsigned)((chunks + 256 * U - 1) / (256 * U))),
                      dim3(256), 0, st, static_cast<const Src*>(src), chunks, codes, scales);
}

template <typename Src, int U>
static cudaError_t launch_quantize(const void* src, long chunks, bool e2m1, uint8_t* codes,
                                   uint8_t* scales, cudaStream_t st)
{
    return e2m1 ? launch_quantize<true, Src, U>(src, chunks, codes, scales, st)
                : launch_quantize<false, Src, U>(src, chunks, codes, scales, st);
}

cudaError_t launch_quantize_mx(const void* src, bool f32, long n, bool e2m1, uint8_t* codes,
                               uint8_t* scales, cudaStream_t st)
{
    const long chunks = n / 8;
    // Several chunks a thread pay once the grid fills the SMs for all that (bf16 to E4M3, U = 1 and
    // 4: 2.1 M elements 1.8 and 3.0 us, 5.2 M 3.8 and 3.8, 8.4 M 5.6 and 5.1, 134 M 73.7 and 60.6).
    const bool many = chunks > 4096L * device_sms();
    if (f32) return launch_quantize<float, 1>(src, chunks, e2m1, codes, scales, st);
    return many ? launch_quantize<uint16_t, 4>(src, chunks, e2m1, codes, scales, st)
                : launch_quantize<uint16_t, 1>(src, chunks, e2m1, codes, scales, st);
}

}  // namespace moe
