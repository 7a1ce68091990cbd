// Encoders of 8-bit floating-point operands (include/q2k.h, fp8_quantize and
// swiglu_fp8_rows): e4m3 codes with an fp32 scale for each 128 values of a
// row or each 128 x 128 values of a matrix.
//
// One pass, bound by memory: a block's values stay in registers between the
// read that finds their largest and the write of their codes.  The largest is
// taken over the bits of |x|, which order like the numbers with infinity and
// NaN above all, so both reach the scale.
#include <algorithm>

#include "q2k_common.cuh"
#include "q2k_internal.h"

namespace q2k {

namespace {

constexpr int kEncThreads = 256;
constexpr int kRowGroup = 8;                         // lanes that share a block of a row: 16 values each
constexpr int kRowGroups = kEncThreads / kRowGroup;  // of a thread block
constexpr int kEncGroup = 16;                        // lanes of a row of a 128 x 128 block: 8 values each
constexpr int kEncGroups = kEncThreads / kEncGroup;

struct EncArgs {
    const void* x;
    uint8_t* q;
    float* scales;
    int64_t rows, ldx, ldq, ld_scales;
    int K, blocks, x_bf16, swiglu;
    int row_shift;  // log2 of the groups that share a row
};

// 448 * (1 / c), and the scale c / 448, of a block whose largest |x| has these bits.
__device__ __forceinline__ float enc_factor(uint32_t top_bits, float* scale)
{
    float c = fmaxf(__uint_as_float(top_bits), 0x1.cp-112f);  // 448 * 2^-120
    if (top_bits >= 0x7f800000u)
        c = __uint_as_float(0x7fffffffu);
    *scale = __fdiv_rn(c, 448.0f);
    return __fmul_rn(448.0f, __frcp_rn(c));
}

__device__ __forceinline__ uint32_t enc4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// g / (1 + e^-g) * u, within 8 units of the last place of h.  e^-g is the hardware's 2^t (2^-22 off) of t = -g log2(e) as
// a product, and what its rounding and log2(e)'s left as a factor 1 + t' ln 2, a quarter of it here.  Both are taken of a
// gate cut at 128, where e^-g no longer counts: past 2.36e38 the product is infinite and what it left is, too.  The
// division is one of a quarter by a quarter, by the hardware's reciprocal (2^-23 off), which past 2^126 would be 0 and
// lose what a large u shows; so h is right to g = -88.7, below which e^-g is past fp32's range.  The sigmoid meets u
// before g, so that a gate near or below fp32's smallest normal value loses no bits to a factor below 1: 1 + e^-g of a gate
// so small is 2, and u is large where h is not lost in any case.  (8191 rows of 2048 16.7 us; with expf and a quick
// division 19.8, with a rounded one 28.)
__device__ __forceinline__ float swiglu1(float g, float u)
{
    const float c = fminf(g, 128.0f);  // (128 for NaN, which the products keep)
    const float hi = __fmul_rn(c, -0x1.715476p+0f);
    const float lo = fmaf(c, -0x1.4ae0cp-26f, fmaf(c, -0x1.715476p+0f, -hi));
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(hi));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, fmaf(lo, 0x1.62e43p-3f, 0.25f), 0.25f)));
    return 0.25f * r * u * g;
}

// 8 values as they lie in memory, and as numbers.
template <bool BF16>
struct Enc8 {
    uint4 w[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void* p, int64_t i)
    {
        const uint4* at = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (BF16 ? 2 : 4));
#pragma unroll
        for (int k = 0; k < (BF16 ? 1 : 2); ++k)
            w[k] = at[k];
    }
    __device__ __forceinline__ float at(int j) const
    {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
        if (BF16)
            return __uint_as_float(j & 1 ? u[j >> 1] & 0xffff0000u : u[j >> 1] << 16);
        return __uint_as_float(u[j]);
    }
};

__device__ __forceinline__ void enc_store8(uint8_t* q, const float (&v)[8], float f)
{
    *reinterpret_cast<uint2*>(q) = make_uint2(enc4(v[0] * f, v[1] * f, v[2] * f, v[3] * f),
                                              enc4(v[4] * f, v[5] * f, v[6] * f, v[7] * f));
}

// 16 of a block's values: chunks of 16 bytes, a lane's one behind those of the 8 lanes' before it.
template <bool BF16>
struct Enc16 {
    static constexpr int kChunk = BF16 ? 8 : 4, kChunks = 16 / kChunk;  // values of a chunk
    uint4 w[kChunks];
    // n values of the block are there, a multiple of kChunk
    __device__ __forceinline__ void load(const void* p, int64_t first, int lane, int n)
    {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = (c * kRowGroup + lane) * kChunk;
            w[c] = k < n ? *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + (first + k) * (BF16 ? 2 : 4))
                         : make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ float at(int i) const
    {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
        if (BF16)
            return __uint_as_float(i & 1 ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);
        return __uint_as_float(u[i]);
    }
};

// Rows on 16-byte boundaries, K a multiple of 8: 8 lanes a block of 128, the
// groups of a thread block side by side along a row (2^row_shift of them) and
// over rows.  (8 values a lane instead of 16 had the scale worked out twice as
// often: 22 us for 8191 x 4096 in bf16.)
template <bool BF16, bool SWIGLU>
__global__ void __launch_bounds__(kEncThreads) fp8_rows_kernel(const EncArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    using X = Enc16<BF16>;
    const int group = threadIdx.x / kRowGroup, lane = threadIdx.x % kRowGroup;
    const int across = 1 << a.row_shift;
    const int64_t row = (int64_t)blockIdx.x * (kRowGroups >> a.row_shift) + (group >> a.row_shift);
    for (int b0 = 0; b0 < a.blocks; b0 += across) {
        const int b = b0 + (group & (across - 1));
        const int n = row < a.rows ? min(128, a.K - b * 128) : 0;  // (none past the last block)
        X x, up;
        x.load(a.x, row * a.ldx + b * 128, lane, n);
        if (SWIGLU)
            up.load(a.x, row * a.ldx + a.K + b * 128, lane, n);
        float v[16];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            v[i] = SWIGLU ? swiglu1(x.at(i), up.at(i)) : x.at(i);
            top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
        }
#pragma unroll
        for (int o = kRowGroup / 2; o >= 1; o >>= 1)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        float scale;
        const float f = enc_factor(top, &scale);
        uint8_t* const q = a.q + row * a.ldq + b * 128;
#pragma unroll
        for (int c = 0; c < X::kChunks; ++c) {
            const int k = (c * kRowGroup + lane) * X::kChunk;
            const float* const w = v + c * X::kChunk;
            const uint32_t lo = enc4(w[0] * f, w[1] * f, w[2] * f, w[3] * f);
            if (k < n) {
                if (BF16)
                    *reinterpret_cast<uint2*>(q + k) = make_uint2(lo, enc4(w[BF16 ? 4 : 0] * f, w[BF16 ? 5 : 0] * f, w[BF16 ? 6 : 0] * f, w[BF16 ? 7 : 0] * f));
                else
                    *reinterpret_cast<uint32_t*>(q + k) = lo;
            }
        }
        if (lane == 0 && n > 0)
            a.scales[row * a.ld_scales + b] = scale;
    }
}

__device__ __forceinline__ float enc_load1(const EncArgs& a, int64_t i)
{
    return a.x_bf16 ? bf16_bits_f(static_cast<const uint16_t*>(a.x)[i]) : static_cast<const float*>(a.x)[i];
}

// Any K, stride and alignment: a warp a block of 128, value by value.
__global__ void __launch_bounds__(kEncThreads) fp8_rows_any_kernel(const EncArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 31;
    for (int b = threadIdx.x >> 5; b < a.blocks; b += kEncThreads / 32) {
        float v[4];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = b * 128 + j * 32 + lane;
            v[j] = 0.f;
            if (k < a.K)
                v[j] = a.swiglu ? swiglu1(enc_load1(a, row * a.ldx + k), enc_load1(a, row * a.ldx + a.K + k))
                                : enc_load1(a, row * a.ldx + k);
            top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
        }
        float scale;
        const float f = enc_factor(__reduce_max_sync(0xffffffffu, top), &scale);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = b * 128 + j * 32 + lane;
            if (k < a.K)
                a.q[row * a.ldq + k] = (uint8_t)enc4(v[j] * f, 0.f, 0.f, 0.f);
        }
        if (lane == 0)
            a.scales[row * a.ld_scales + b] = scale;
    }
}

// The largest of a thread block's values, the same in every thread.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* part)
{
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < kEncThreads / 32 ? part[threadIdx.x & 31] : 0u);
}

// A thread block a 128 x 128 block, all of it on its way at once (64 values a thread).
template <bool BF16>
__global__ void __launch_bounds__(kEncThreads) fp8_blocks_kernel(const EncArgs a)
{
    __shared__ uint32_t part[kEncThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    constexpr int R = 128 / kEncGroups;
    const int group = threadIdx.x / kEncGroup, lane = threadIdx.x % kEncGroup;
    const int64_t row0 = (int64_t)blockIdx.x * 128 + group;
    const int k = (int)blockIdx.y * 128 + lane * 8;
    Enc8<BF16> x[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (row0 + r * kEncGroups < a.rows && k < a.K)
            x[r].load(a.x, (row0 + r * kEncGroups) * a.ldx + k);
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (row0 + r * kEncGroups < a.rows && k < a.K) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = max(top, __float_as_uint(x[r].at(j)) & 0x7fffffffu);
        }
    float scale;
    const float f = enc_factor(block_max(top, part), &scale);
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (row0 + r * kEncGroups < a.rows && k < a.K) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = x[r].at(j);
            enc_store8(a.q + (row0 + r * kEncGroups) * a.ldq + k, v, f);
        }
    if (threadIdx.x == 0)
        a.scales[(int64_t)blockIdx.x * a.ld_scales + blockIdx.y] = scale;
}

__global__ void __launch_bounds__(kEncThreads) fp8_blocks_any_kernel(const EncArgs a)
{
    __shared__ uint32_t part[kEncThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row0 = (int64_t)blockIdx.x * 128 + (threadIdx.x >> 7);
    const int k = (int)blockIdx.y * 128 + (threadIdx.x & 127);
    uint32_t top = 0;
    for (int r = 0; r < 128; r += kEncThreads / 128)
        if (row0 + r < a.rows && k < a.K)
            top = max(top, __float_as_uint(enc_load1(a, (row0 + r) * a.ldx + k)) & 0x7fffffffu);
    float scale;
    const float f = enc_factor(block_max(top, part), &scale);
    for (int r = 0; r < 128; r += kEncThreads / 128)
        if (row0 + r < a.rows && k < a.K)
            a.q[(row0 + r) * a.ldq + k] = (uint8_t)enc4(enc_load1(a, (row0 + r) * a.ldx + k) * f, 0.f, 0.f, 0.f);
    if (threadIdx.x == 0)
        a.scales[(int64_t)blockIdx.x * a.ld_scales + blockIdx.y] = scale;
}

bool on(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

cudaError_t launch_fp8_encode(const Fp8Encode& p, cudaStream_t s)
{
    EncArgs a{};
    a.x = p.x;
    a.q = p.q;
    a.scales = p.scales;
    a.rows = p.rows;
    a.ldx = p.ldx;
    a.ldq = p.ldq;
    a.ld_scales = p.ld_scales;
    a.K = (int)p.K;
    a.blocks = (a.K + 127) / 128;
    a.x_bf16 = p.x_bf16;
    a.swiglu = p.swiglu;
    const int64_t per16 = p.x_bf16 ? 8 : 4;
    const bool vec = p.K % 8 == 0 && on(p.x, 16) && p.ldx % per16 == 0 && on(p.q, 8) && p.ldq % 8 == 0;
    if (p.block_rows == 128) {
        const dim3 grid((unsigned)((p.rows + 127) / 128), (unsigned)a.blocks);
        auto* kernel = !vec ? fp8_blocks_any_kernel : p.x_bf16 ? fp8_blocks_kernel<true> : fp8_blocks_kernel<false>;
        return launch_pdl(kernel, grid, dim3(kEncThreads), 0, s, a);
    }
    if (!vec)
        return launch_pdl(fp8_rows_any_kernel, dim3((unsigned)p.rows), dim3(kEncThreads), 0, s, a);
    while ((1 << a.row_shift) < std::min(a.blocks, kRowGroups))
        ++a.row_shift;
    const int64_t rows = kRowGroups >> a.row_shift;  // of a thread block
    auto* kernel = p.swiglu ? (p.x_bf16 ? fp8_rows_kernel<true, true> : fp8_rows_kernel<false, true>)
                            : (p.x_bf16 ? fp8_rows_kernel<true, false> : fp8_rows_kernel<false, false>);
    return launch_pdl(kernel, dim3((unsigned)((p.rows + rows - 1) / rows)), dim3(kEncThreads), 0, s, a);
}

}  // namespace q2k
