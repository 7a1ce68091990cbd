// The routed experts of a few tokens over 8-bit floating-point weights
// (include/q2k.h, fp8_moe).
#include <algorithm>

#include "q2k_common.cuh"
#include "q2k_internal.h"

namespace q2k {

namespace {

__device__ __forceinline__ float e4m3_f(uint32_t code)
{
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(code));
    return half_lo_f(h);
}

// A row of a block-scaled matrix times a bf16 row, by a warp.
__device__ __forceinline__ float row_dot(const uint8_t* w, const float* scales, const uint16_t* x, int K)
{
    float s = 0.f;
    for (int k = (int)(threadIdx.x & 31); k < K; k += 32)
        s = fmaf(e4m3_f(w[k]) * scales[k / 128], bf16_bits_f(x[k]), s);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// h of a pair (token, choice), a warp a value.
__global__ void __launch_bounds__(256) fp8_moe_up_kernel(const Fp8Moe a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int p = blockIdx.y, e = a.ids[p], dim = (int)a.dim, inter = (int)a.inter;
    const int r = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (e < 0 || e >= a.E || r >= inter)
        return;
    const int kb = (dim + 127) / 128, rb = (inter + 127) / 128;
    float v[2];
    for (int j = 0; j < 2; ++j) {
        const int64_t at = (int64_t)e * 2 + j;
        v[j] = row_dot(a.gate_up + (at * inter + r) * dim, a.gate_up_scales + (at * rb + r / 128) * kb,
                       a.x + p / a.topk * a.ldx, dim);
    }
    const float h = __fdiv_rn(v[0], 1.0f + expf(-v[0])) * v[1];
    if ((threadIdx.x & 31) == 0)
        static_cast<uint16_t*>(a.workspace)[(int64_t)p * inter + r] = __bfloat16_as_ushort(__float2bfloat16_rn(h));
}

__global__ void __launch_bounds__(256) fp8_moe_down_kernel(const Fp8Moe a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.y, dim = (int)a.dim, inter = (int)a.inter;
    const int r = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= dim)
        return;
    const int kb = (inter + 127) / 128, rb = (dim + 127) / 128;
    float y = 0.f;
    for (int j = 0; j < a.topk; ++j) {
        const int64_t p = (int64_t)t * a.topk + j, e = a.ids[p];
        if (e < 0 || e >= a.E)
            continue;
        const float v = row_dot(a.down + (e * dim + r) * inter, a.down_scales + (e * rb + r / 128) * kb,
                                static_cast<const uint16_t*>(a.workspace) + p * inter, inter);
        y = fmaf(a.route_w[p], v, y);
    }
    if ((threadIdx.x & 31) == 0) {
        if (a.y_bf16)
            static_cast<uint16_t*>(a.y)[t * a.ldy + r] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
        else
            static_cast<float*>(a.y)[t * a.ldy + r] = y;
    }
}

}  // namespace

size_t fp8_moe_workspace(int64_t m, int64_t topk, int64_t dim, int64_t inter)
{
    (void)dim;
    return (size_t)((m * topk * inter * 2 + 255) / 256 * 256);
}

cudaError_t launch_fp8_moe(const Fp8Moe& p, cudaStream_t s)
{
    cudaError_t e = launch_pdl(fp8_moe_up_kernel, dim3((unsigned)((p.inter + 7) / 8), (unsigned)(p.m * p.topk)), dim3(256),
                               0, s, p);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(fp8_moe_down_kernel, dim3((unsigned)((p.dim + 7) / 8), (unsigned)p.m), dim3(256), 0, s, p);
}

}  // namespace q2k
