// mx_ffn.cu -- products grouped by expert of E4M3 rows with E2M1 weights (both in
// microscaled blocks), alone and as the two products of the expert FFN.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kernels.h"
#include "mx_common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float e8m0(uint32_t c)
{
    return c == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(c ? c << 23 : 1u << 22);
}

__device__ __forceinline__ float e4m3(uint32_t c)
{
    const uint32_t e = (c >> 3) & 15, m = c & 7;
    float v = e ? __uint_as_float(((e + 120) << 23) | (m << 20)) : (float)m * 0.001953125f;
    if ((c & 127) == 127) v = __uint_as_float(0x7FC00000u);
    return c & 128 ? -v : v;
}

__device__ __forceinline__ float e2m1(uint32_t c)
{
    const uint32_t e = (c >> 1) & 3, m = c & 1;
    const float v = e ? __uint_as_float(((e + 126) << 23) | (m << 22)) : (float)m * 0.5f;
    return c & 8 ? -v : v;
}

// The dot product of one row of a and one of w, block by block.
__device__ float dot(const uint8_t* a, const uint8_t* sa, const uint8_t* w, const uint8_t* sw, int K)
{
    float acc = 0.f;
    for (int b = 0; b < K / 32; ++b) {
        float s = 0.f;
        for (int i = 0; i < 16; ++i) {
            const uint32_t q = w[b * 16 + i];
            s = fmaf(e4m3(a[b * 32 + 2 * i]), e2m1(q & 15), s);
            s = fmaf(e4m3(a[b * 32 + 2 * i + 1]), e2m1(q >> 4), s);
        }
        acc = fmaf(s * e8m0(sa[b]), e8m0(sw[b]), acc);
    }
    return acc;
}

// One thread per output (feature f of row p); a warp holds one MX block of act.
template <int MODE>
__global__ void __launch_bounds__(128) mx_grouped_kernel(const MxArgs g)
{
    pdl_launch_dependents();
    pdl_wait();
    const int p = blockIdx.y + blockIdx.z * gridDim.y, f = blockIdx.x * 128 + threadIdx.x;
    if (p >= min(g.R, g.offsets[g.E])) return;
    int lo = 0, hi = g.E;  // the expert of row p: the last e with offsets[e] <= p
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (g.offsets[mid] <= p) lo = mid; else hi = mid;
    }
    const int r = MODE == 2 ? p : g.rows[p];
    const size_t arow = MODE == 0 ? r / g.k : p;
    const uint8_t* a = g.a + arow * g.K;
    const uint8_t* sa = g.a_scale + arow * (g.K / 32);
    const size_t wrow = (size_t)lo * (MODE == 0 ? 2 * g.N : g.N) + f;
    if (f >= g.N) return;
    float v = dot(a, sa, g.w + wrow * (g.K / 2), g.w_scale + wrow * (g.K / 32), g.K);
    if (MODE == 0) {
        const size_t up = wrow + g.N;
        const float u = dot(a, sa, g.w + up * (g.K / 2), g.w_scale + up * (g.K / 32), g.K);
        v = v / (1.0f + expf(-v)) * u;
        uint32_t m = __float_as_uint(v) & 0x7FFFFFFFu;
        for (int o = 16; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t code = mx::scale_code(m, mx::kEmaxE4M3);
        const float q = v * mx::inverse_scale(min(code, 254u));
        g.act[(size_t)p * g.N + f] = code == 255 ? 0x7F : (uint8_t)mx::e4m3x4(q, q, q, q);
        if ((f & 31) == 0) g.act_scale[(size_t)p * (g.N / 32) + f / 32] = (uint8_t)code;
    } else {
        static_cast<__nv_bfloat16*>(g.y)[(size_t)r * g.N + f] = __float2bfloat16(v);
    }
}

template <int MODE>
cudaError_t launch_mode(const MxArgs& g, cudaStream_t st)
{
    const int ry = g.R < 32768 ? g.R : 32768;
    return launch_pdl(mx_grouped_kernel<MODE>, dim3((g.N + 127) / 128, ry, (g.R + ry - 1) / ry),
                      dim3(128), 0, st, g);
}

}  // namespace

cudaError_t launch_mx_grouped(const MxArgs& g, int mode, cudaStream_t st)
{
    return mode == 0 ? launch_mode<0>(g, st) : mode == 1 ? launch_mode<1>(g, st) : launch_mode<2>(g, st);
}

}  // namespace moe
