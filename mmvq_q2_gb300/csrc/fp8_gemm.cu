// The product of 8-bit floating-point operands (include/q2k.h, fp8_gemm).
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

// A thread a value of y.
__global__ void __launch_bounds__(256) fp8_gemm_kernel(const Fp8Gemm a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t n = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const int64_t t = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5);
    if (n >= a.N || t >= a.m)
        return;
    const int64_t blocks = (a.K + 127) / 128;
    float y = 0.f;
    for (int64_t b = 0; b < blocks; ++b) {
        float s = 0.f;
        for (int64_t k = b * 128; k < min(a.K, b * 128 + 128); ++k)
            s = fmaf(e4m3_f(a.x[t * a.ldx + k]), e4m3_f(a.W[n * a.K + k]), s);
        y = fmaf(s, a.x_scales[t * a.ld_xs + b] * a.w_scales[n / 128 * blocks + b], y);
    }
    if (a.y_bf16)
        static_cast<uint16_t*>(a.y)[t * a.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
    else
        static_cast<float*>(a.y)[t * a.ldy + n] = y;
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8Gemm& p, cudaStream_t s)
{
    if (fp8_stream_supported(p))
        return launch_fp8_gemm_stream(p, s);
    return launch_pdl(fp8_gemm_kernel, dim3((unsigned)((p.N + 31) / 32), (unsigned)((p.m + 7) / 8)), dim3(256), 0, s, p);
}

}  // namespace q2k
