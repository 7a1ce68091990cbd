// Between the products of a decode layer: the norms around a block fused
// with its gate and residual scale, and the route of the experts
// (include/q2k.h, norm_gate_residual and moe_route_topk).
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "q2k_common.cuh"
#include "q2k_internal.h"
#include "q2k_q8.cuh"

namespace q2k {

namespace {

// ---- norm_gate_residual --------------------------------------------------------
//
// h = residual + alpha * gate * norm(y), n = norm(h): two sums over a row,
// the second of values that need the first.  Bound by memory: a row stays in
// registers (8 values a run, one or two runs a thread) from its one read to
// its one write.

struct NormArgs {
    const void *y, *gate, *residual;
    void *residual_out, *out_q8;
    uint16_t* out;
    const float *post_w, *pre_w;
    int64_t ld_y, ld_gate, ld_res, ld_ro, ld_out, T;
    float alpha, eps;
    int dim, y_bf16, stream_bf16;
};

__device__ __forceinline__ float load1(const void* p, int64_t i, int bf16)
{
    return bf16 ? bf16_bits_f(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void load8(const void* p, int64_t i, int bf16, float (&v)[8])
{
    if (bf16) {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    } else {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = f[0], b = f[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

// (One instruction for two; a conversion alone goes through a slower unit.)
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ void store8(void* p, int64_t i, int bf16, const float (&v)[8])
{
    if (bf16)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
            make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
    else {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        f[0] = make_float4(v[0], v[1], v[2], v[3]);
        f[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// Sum over the block, the same bits in every thread (fixed order).
__device__ __forceinline__ float block_sum(float v, float* part)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    const int nw = (int)(blockDim.x >> 5);
    if (nw == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = (int)(threadIdx.x & 31) < nw ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// The q8_1 rows of the bf16 row in shared memory.
__device__ __forceinline__ void encode_row(const uint16_t* n_row, int dim, uint8_t* out)
{
    for (int i0 = 0; i0 < dim; i0 += 4 * (int)blockDim.x) {
        const int i = i0 + 4 * (int)threadIdx.x;
        const bool live = i < dim;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (live) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = bf16_bits_f(n_row[i + j]);
        }
        q8_1_encode_group(v, out + (i / kQ8Values) * kQ8Bytes, (int)threadIdx.x & 7, live);
    }
}

// 8 values of a row as they lie in memory: a load of 16 bytes, of fp32 two (a
// row's start need only be on 16 bytes).
template <bool BF16>
struct Raw8 {
    uint4 w[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void* p, int64_t i)
    {
        const char* at = static_cast<const char*>(p) + i * (BF16 ? 2 : 4);
#pragma unroll
        for (int k = 0; k < (BF16 ? 1 : 2); ++k)
            w[k] = reinterpret_cast<const uint4*>(at)[k];
    }
    __device__ __forceinline__ float at(int j) const
    {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
        if (BF16)
            return __uint_as_float(j & 1 ? u[j >> 1] & 0xffff0000u : u[j >> 1] << 16);
        return __uint_as_float(u[j]);
    }
};

// NR runs of 8 values a thread, rows and pointers on 16-byte boundaries.  A
// block takes rows blockIdx.x, + gridDim.x, ...: where it has more than one,
// the weights wait in shared memory (read again for every row they were 32 of
// 72 KB of a row's traffic from L2), and the next row is on its way while
// this one is summed.  Where two runs a thread pay (launch_norm_vec), half the
// warps meet at a barrier, and more blocks share an SM to work meanwhile.
// 8192 rows of 4096, all bf16, a gate per token: 60 us, 5.6 TB/s; all fp32:
// 92 us, 6.5 TB/s.
constexpr int kNormVecDim = 8 * 1024;

template <int NR, bool YB, bool SB>
__global__ void __launch_bounds__(NR == 1 ? 1024 : 256, NR == 1 ? 1 : 3) norm_vec_kernel(const NormArgs a)
{
    extern __shared__ __align__(16) uint8_t norm_smem[];
    __shared__ float part[2][2][32];
    pdl_launch_dependents();
    pdl_wait();
    const bool many = gridDim.x < a.T;
    float* const w_smem = reinterpret_cast<float*>(norm_smem);
    uint16_t* const n_row = reinterpret_cast<uint16_t*>(norm_smem + (many ? (size_t)a.dim * 8 : 0));  // with out_q8
    const float* pre_w = many ? w_smem : a.pre_w;
    const float* post_w = many ? w_smem + a.dim : a.post_w;
    const bool has_y = a.y != nullptr, has_gate = a.gate != nullptr, has_post = a.post_w != nullptr;
    Raw8<SB> res[NR];
    Raw8<YB> y[NR], gate[NR];
    auto at = [&](int r) { return (r * (int)blockDim.x + (int)threadIdx.x) * 8; };
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int r = 0; r < NR; ++r)
            if (at(r) < a.dim && t < a.T) {
                res[r].load(a.residual, t * a.ld_res + at(r));
                if (has_y)
                    y[r].load(a.y, t * a.ld_y + at(r));
                if (has_gate)
                    gate[r].load(a.gate, t * a.ld_gate + at(r));
            }
    };
    int64_t t = blockIdx.x;
    fetch(t);
    if (many) {
        for (int i = (int)threadIdx.x * 4; i < a.dim; i += (int)blockDim.x * 4) {
            *reinterpret_cast<float4*>(w_smem + i) = *reinterpret_cast<const float4*>(a.pre_w + i);
            if (has_post)
                *reinterpret_cast<float4*>(w_smem + a.dim + i) = *reinterpret_cast<const float4*>(a.post_w + i);
        }
        __syncthreads();
    }
    for (int odd = 0; t < a.T; t += gridDim.x, odd ^= 1) {
        float h[NR][8], u[NR][8];
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const bool live = at(r) < a.dim;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[r][j] = live ? res[r].at(j) : 0.f;
                u[r][j] = live && has_y ? y[r].at(j) : 0.f;
                s = fmaf(u[r][j], u[r][j], s);
            }
        }
        if (has_post) {
            const float inv = 1.0f / sqrtf(block_sum(s, part[odd][0]) / (float)a.dim + a.eps);
#pragma unroll
            for (int r = 0; r < NR; ++r)
                if (at(r) < a.dim) {
                    float w[8];
                    load8(post_w, at(r), 0, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        u[r][j] = u[r][j] * inv * w[j];
                }
        }
        s = 0.f;
#pragma unroll
        for (int r = 0; r < NR; ++r)
            if (at(r) < a.dim) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (has_y)
                        h[r][j] = fmaf(a.alpha, has_gate ? u[r][j] * gate[r].at(j) : u[r][j], h[r][j]);
                    s = fmaf(h[r][j], h[r][j], s);
                }
                if (a.residual_out)
                    store8(a.residual_out, t * a.ld_ro + at(r), SB, h[r]);
            }
        fetch(t + gridDim.x);
        if (!a.out && !a.out_q8)
            continue;
        const float inv = 1.0f / sqrtf(block_sum(s, part[odd][1]) / (float)a.dim + a.eps);
#pragma unroll
        for (int r = 0; r < NR; ++r)
            if (at(r) < a.dim) {
                float w[8];
                load8(pre_w, at(r), 0, w);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    h[r][j] = h[r][j] * inv * w[j];
                if (a.out)
                    store8(a.out, t * a.ld_out + at(r), 1, h[r]);
                if (a.out_q8)
                    store8(n_row, at(r), 1, h[r]);
            }
        if (a.out_q8) {
            __syncthreads();
            encode_row(n_row, a.dim, static_cast<uint8_t*>(a.out_q8) + t * (a.dim / kQ8Values) * kQ8Bytes);
            __syncthreads();
        }
    }
}

// Any dim, stride and alignment: the row waits in shared memory as fp32.
__global__ void __launch_bounds__(256) norm_any_kernel(const NormArgs a)
{
    extern __shared__ float smem[];
    float* part = smem;          // [2][32]
    float* row = smem + 64;      // [dim]
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = blockIdx.x;
    float inv = 1.f;
    if (a.post_w) {
        float s = 0.f;
        for (int i = (int)threadIdx.x; i < a.dim; i += (int)blockDim.x) {
            const float v = load1(a.y, t * a.ld_y + i, a.y_bf16);
            s = fmaf(v, v, s);
        }
        inv = 1.0f / sqrtf(block_sum(s, part) / (float)a.dim + a.eps);
    }
    float s = 0.f;
    for (int i = (int)threadIdx.x; i < a.dim; i += (int)blockDim.x) {
        float h = load1(a.residual, t * a.ld_res + i, a.stream_bf16);
        if (a.y) {
            float u = load1(a.y, t * a.ld_y + i, a.y_bf16);
            if (a.post_w)
                u = u * inv * a.post_w[i];
            if (a.gate)
                u *= load1(a.gate, t * a.ld_gate + i, a.y_bf16);
            h = fmaf(a.alpha, u, h);
        }
        row[i] = h;
        if (a.residual_out) {
            if (a.stream_bf16)
                static_cast<uint16_t*>(a.residual_out)[t * a.ld_ro + i] = __bfloat16_as_ushort(__float2bfloat16_rn(h));
            else
                static_cast<float*>(a.residual_out)[t * a.ld_ro + i] = h;
        }
        s = fmaf(h, h, s);
    }
    if (!a.out && !a.out_q8)
        return;
    inv = 1.0f / sqrtf(block_sum(s, part + 32) / (float)a.dim + a.eps);
    uint16_t* n_row = reinterpret_cast<uint16_t*>(row + a.dim);
    for (int i = (int)threadIdx.x; i < a.dim; i += (int)blockDim.x) {
        const uint16_t n = __bfloat16_as_ushort(__float2bfloat16_rn(row[i] * inv * a.pre_w[i]));
        if (a.out)
            a.out[t * a.ld_out + i] = n;
        if (a.out_q8)
            n_row[i] = n;
    }
    if (a.out_q8) {
        __syncthreads();
        encode_row(n_row, a.dim, static_cast<uint8_t*>(a.out_q8) + t * (a.dim / kQ8Values) * kQ8Bytes);
    }
}

// ---- moe_route_topk ------------------------------------------------------------
//
// One warp a token, expert e in lane e % 32: the scores stay in registers.
// The choice works on whole numbers that order like the floats, so that a
// maximum over the warp is one redux instruction and a tie falls to the
// lowest index exactly.  What bounds it is the number of instructions (256
// experts: 1 KB to read, 840 instructions of a warp).  So a lane keeps
// its two best at hand and looks its scores through again only when both are
// gone; and a softmax without bias or groups is chosen by its exponentials,
// since dividing all by one sum keeps their order: the scores are worked out
// for the chosen and the next one alone.  (Two of them may round to one
// score; the token then takes the full way.)  16384 tokens of 256 experts,
// 8 each: 21.7 us with every score divided and every round through all.

struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    const int64_t* expert_ptrs;
    int64_t* ptrs_out;
    int64_t m, ld;
    int E, sigmoid, n_group, topk_group, topk, renorm;
    int share;          // log2 of the lanes that a group gets
    uint32_t per_size;  // 2^20 / (experts of a group), rounded up: e * per_size >> 20 is e / size for e and size to 1024
    float scale;
};

// Orders like the float; NaN below -inf, 0 is left for "taken".
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 becomes 0
    if (v != v)
        return 1u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// The choice of the largest keys, one a call, from the warp's NE * 32; a key
// that is taken is not given again, and equal ones come by rising expert.
template <int NE>
struct Best {
    uint32_t k1, k2;  // the lane's best two
    int j1, j2;
    bool have2;       // k2 is known
    __device__ __forceinline__ explicit Best(const uint32_t (&key)[NE]) : k1(0), k2(0), j1(0), j2(0), have2(true)
    {
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const bool first = key[j] > k1, second = key[j] > k2;
            k2 = first ? k1 : second ? key[j] : k2;
            j2 = first ? j1 : second ? j : j2;
            k1 = first ? key[j] : k1;
            j1 = first ? j : j1;
        }
    }
    // The expert with the largest key, and the key, the same in every lane.
    __device__ __forceinline__ uint32_t take(const uint32_t (&key)[NE], uint32_t& best)
    {
        const int lane = threadIdx.x & 31;
        best = __reduce_max_sync(0xffffffffu, k1);
        const uint32_t mine = (uint32_t)(j1 * 32 + lane);
        const uint32_t e = __reduce_min_sync(0xffffffffu, k1 == best ? mine : 0xffffffffu);
        const bool owner = e == mine;
        const uint32_t pk = k1;
        const int pj = j1;
        if (owner) {
            k1 = k2;
            j1 = j2;
        }
        if (__any_sync(0xffffffffu, owner && !have2)) {
            // the best of what comes after the key just taken
            uint32_t k = 0;
            int at = 0;
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                const bool after = key[j] < pk || (key[j] == pk && j > pj);
                if (after && key[j] > k) {
                    k = key[j];
                    at = j;
                }
            }
            if (owner && !have2) {
                k1 = k;
                j1 = at;
            }
        }
        if (owner)
            have2 = false;
        return e;
    }
};

template <int NE, bool BF16>
__global__ void __launch_bounds__(128) moe_route_kernel(const RouteArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (t >= a.m)
        return;
    float s[NE];
    uint32_t key[NE];
    float top = -FLT_MAX;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int e = j * 32 + lane;
        float x = -INFINITY;
        if (e < a.E)
            x = BF16 ? bf16_bits_f(static_cast<const uint16_t*>(a.logits)[t * a.ld + e])
                     : static_cast<const float*>(a.logits)[t * a.ld + e];
        s[j] = fminf(fmaxf(x, -INFINITY), FLT_MAX);  // the maximum of NaN and x is x
        top = fmaxf(top, s[j]);
    }
    float sum = 0.f;  // softmax: of the exponentials
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < NE; ++j)
            s[j] = __fdiv_rn(1.0f, 1.0f + expf(-s[j]));
    } else {
        top = key_value(__reduce_max_sync(0xffffffffu, order_key(top)));
        // Each e <= 1 as a multiple of 2^-12 and the rest: the former sum up
        // without rounding, the latter are below 2^-13, so the sum is that of
        // 36 bits and more, rounded once: a choice between near equals does
        // not depend on the order of the sum.
        float hi = 0.f, lo = 0.f;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            s[j] = expf(s[j] - top);
            const float h = __fadd_rn(__fadd_rn(s[j], 0x1.8p11f), -0x1.8p11f);
            hi = __fadd_rn(hi, h);
            lo = __fadd_rn(lo, __fadd_rn(s[j], -h));
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            hi = __fadd_rn(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            lo = __fadd_rn(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        }
        sum = __shfl_sync(0xffffffffu, __fadd_rn(hi, lo), 0);
    }
    auto finish = [&](float w, int id) {  // lane i: score and expert of choice i
        if (a.renorm) {
            float all = lane < a.topk ? w : 0.f;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1)
                all += __shfl_xor_sync(0xffffffffu, all, o);
            w = w / (all + 1e-20f);
        }
        if (lane < a.topk) {
            a.ids[t * a.topk + lane] = id;
            a.weights[t * a.topk + lane] = w * a.scale;
            if (a.ptrs_out) {
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    a.ptrs_out[(t * 3 + i) * a.topk + lane] = a.expert_ptrs[(int64_t)i * a.E + id];
            }
        }
    };
    if (!a.sigmoid && !a.bias && a.n_group == 1 && a.topk < 32) {
        // the bits of numbers from 0 on order like the numbers
#pragma unroll
        for (int j = 0; j < NE; ++j)
            key[j] = j * 32 + lane < a.E ? __float_as_uint(s[j]) + 1u : 0u;
        Best<NE> best(key);
        const int rounds = min(a.topk + 1, a.E);
        float v = 0.f;
        int id = 0;
        for (int i = 0; i < rounds; ++i) {
            uint32_t k;
            const uint32_t e = best.take(key, k);
            if (lane == i) {
                v = __uint_as_float(k - 1u);
                id = (int)e;
            }
        }
        const float w = sum > 0.f ? __fdiv_rn(v, sum) : 0.f;
        const float v2 = __shfl_down_sync(0xffffffffu, v, 1), w2 = __shfl_down_sync(0xffffffffu, w, 1);
        if (!__any_sync(0xffffffffu, lane + 1 < rounds && w == w2 && v != v2)) {
            finish(w, id);
            return;
        }
    }
    if (!a.sigmoid) {
#pragma unroll
        for (int j = 0; j < NE; ++j)
            s[j] = sum > 0.f ? __fdiv_rn(s[j], sum) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int e = j * 32 + lane;
        key[j] = e < a.E ? order_key(a.bias ? __fadd_rn(s[j], a.bias[e]) : s[j]) : 0u;
    }
    if (a.n_group > 1) {
        // A group's best two, by 2^share lanes of its own from shared memory.
        // (By the whole warp, group after group: 16384 tokens of 256 experts in
        // 8 groups 27.4 us against 20.1, of 160 in 8 32.1 against 20.1, one
        // token 6.1 against 4.6.)
        __shared__ uint32_t sh_key[4][NE * 33];
        uint32_t* k = sh_key[threadIdx.x >> 5];
#pragma unroll
        for (int j = 0; j < NE; ++j)
            k[j * 33 + lane] = key[j];
        __syncwarp();
        const int size = a.E / a.n_group, g = lane >> a.share;
        uint32_t gkey = 0;  // group g's score
        {
            uint32_t k1 = 0, k2 = 0;
            if (g < a.n_group)
                for (int e = g * size + lane - (g << a.share); e < (g + 1) * size; e += 1 << a.share) {
                    const uint32_t x = k[e + (e >> 5)];
                    k2 = max(k2, min(k1, x));
                    k1 = max(k1, x);
                }
            for (int o = 1; o < 1 << a.share; o <<= 1) {
                const uint32_t b1 = __shfl_xor_sync(0xffffffffu, k1, o), b2 = __shfl_xor_sync(0xffffffffu, k2, o);
                k2 = max(min(k1, b1), max(k2, b2));
                k1 = max(k1, b1);
            }
            if (g < a.n_group)
                gkey = order_key(size > 1 ? key_value(k1) + key_value(k2) : key_value(k1));
        }
        uint32_t kept = 0;
        for (int i = 0; i < a.topk_group; ++i) {
            const uint32_t best = __reduce_max_sync(0xffffffffu, gkey);
            const int first = (__ffs(__ballot_sync(0xffffffffu, gkey == best)) - 1) >> a.share;
            kept |= 1u << first;
            if (g == first)
                gkey = 0;
        }
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const uint32_t e = (uint32_t)(j * 32 + lane);
            if (e < (uint32_t)a.E && !(kept >> (e * a.per_size >> 20) & 1u))  // e / size
                key[j] = 0;
        }
    }
    Best<NE> best(key);
    int id = 0;
    for (int i = 0; i < a.topk; ++i) {
        uint32_t k;
        const uint32_t e = best.take(key, k);
        if (lane == i)
            id = (int)e;
    }
    float w = 0.f;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const float v = __shfl_sync(0xffffffffu, s[j], id & 31);
        w = id >> 5 == j ? v : w;
    }
    finish(w, id);
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <int NR, bool YB, bool SB>
cudaError_t launch_norm_runs(const NormArgs& a, const DeviceInfo& di, cudaStream_t s)
{
    auto* kernel = norm_vec_kernel<NR, YB, SB>;
    const int threads = (a.dim / 8 + NR * 32 - 1) / (NR * 32) * 32;
    const size_t row = a.out_q8 ? (size_t)a.dim * 2 : 0, weights = (size_t)a.dim * 8;
    // weights and the bf16 row: at most 80 KB
    static std::atomic<unsigned long long> devs{0};
    static std::atomic<int> fits[33];  // blocks an SM by warps a block, once asked
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!(devs.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormVecDim * 10);
        if (e != cudaSuccess)
            return e;
        devs.fetch_or(bit, std::memory_order_acq_rel);
    }
    int blocks = fits[threads / 32].load(std::memory_order_relaxed);
    if (blocks == 0) {
        // (the same on every device: the library runs on one kind)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kernel, threads, (size_t)threads * NR * 80);
        if (e != cudaSuccess)
            return e;
        blocks = std::max(1, blocks);
        fits[threads / 32].store(blocks, std::memory_order_relaxed);
    }
    const unsigned grid = (unsigned)std::min<int64_t>(a.T, (int64_t)di.sm_count * blocks);
    return launch_pdl(kernel, dim3(grid), dim3(threads), row + (grid < a.T ? weights : 0), s, a);
}

template <bool YB, bool SB>
cudaError_t launch_norm_vec(const NormArgs& a, const DeviceInfo& di, cudaStream_t s)
{
    // Two runs a thread: 60 us against 68 (8192 rows of 4096, all bf16) and 43
    // against 57 (of 2880).  With fp32 rows a run is twice the bytes and two
    // of them spill (108 us against 92), and few rows want many threads each
    // (300 rows of 4096: 5.0 us against 4.0).
    if constexpr (YB && SB)
        if (a.dim >= 2048 && a.dim <= 4096 && a.T > 4 * di.sm_count)
            return launch_norm_runs<2, YB, SB>(a, di, s);
    return launch_norm_runs<1, YB, SB>(a, di, s);
}

}  // namespace

cudaError_t launch_norm_gate_residual(const NormProblem& p, cudaStream_t s)
{
    NormArgs a{};
    a.y = p.y;
    a.gate = p.gate;
    a.residual = p.residual;
    a.residual_out = p.residual_out;
    a.out_q8 = p.out_q8;
    a.out = p.out;
    a.post_w = p.post_w;
    a.pre_w = p.pre_w;
    a.ld_y = p.ld_y;
    a.ld_gate = p.ld_gate;
    a.ld_res = p.ld_res;
    a.ld_ro = p.ld_ro;
    a.ld_out = p.ld_out;
    a.T = p.T;
    a.alpha = p.alpha;
    a.eps = p.eps;
    a.dim = (int)p.dim;
    a.y_bf16 = p.y_bf16;
    a.stream_bf16 = p.stream_bf16;
    const int y16 = p.y_bf16 ? 8 : 4, s16 = p.stream_bf16 ? 8 : 4;  // elements of 16 bytes
    const bool vec = a.dim % 8 == 0 && on16(a.y) && on16(a.gate) && on16(a.residual) && on16(a.residual_out) &&
                     on16(a.out) && on16(a.post_w) && on16(a.pre_w) && (!a.y || a.ld_y % y16 == 0) &&
                     a.ld_gate % y16 == 0 && a.ld_res % s16 == 0 && (!a.residual_out || a.ld_ro % s16 == 0) &&
                     (!a.out || a.ld_out % 8 == 0);
    if (!vec || a.dim > kNormVecDim) {
        static std::atomic<unsigned long long> smem_devs{0};
        cudaError_t e = allow_max_smem(norm_any_kernel, smem_devs);
        if (e != cudaSuccess)
            return e;
        return launch_pdl(norm_any_kernel, dim3((unsigned)a.T), dim3(256),
                          (size_t)(64 + a.dim) * sizeof(float) + (a.out_q8 ? (size_t)a.dim * 2 : 0), s, a);
    }
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess)
        return e;
    if (a.y_bf16)
        return a.stream_bf16 ? launch_norm_vec<true, true>(a, di, s) : launch_norm_vec<true, false>(a, di, s);
    return a.stream_bf16 ? launch_norm_vec<false, true>(a, di, s) : launch_norm_vec<false, false>(a, di, s);
}

cudaError_t launch_moe_route(const RouteProblem& p, cudaStream_t s)
{
    RouteArgs a{};
    a.logits = p.logits;
    a.bias = p.bias;
    a.ids = p.ids;
    a.weights = p.weights;
    a.expert_ptrs = p.expert_ptrs;
    a.ptrs_out = p.ptrs_out;
    a.m = p.m;
    a.ld = p.ld;
    a.E = (int)p.E;
    a.sigmoid = p.sigmoid;
    a.n_group = p.n_group;
    a.topk_group = p.topk_group;
    a.topk = p.topk;
    a.renorm = p.renorm;
    a.scale = p.scale;
    for (int lanes = 32; lanes >= 2 * a.n_group; lanes /= 2)
        ++a.share;
    const uint32_t size = (uint32_t)(a.E / a.n_group);
    a.per_size = ((1u << 20) + size - 1) / size;
    const int ne = (a.E + 31) / 32;
    auto pick = [&](auto bf16) {
        constexpr bool B = decltype(bf16)::value;
        return ne <= 1 ? moe_route_kernel<1, B> : ne <= 2 ? moe_route_kernel<2, B> : ne <= 4 ? moe_route_kernel<4, B>
             : ne <= 8 ? moe_route_kernel<8, B> : ne <= 16 ? moe_route_kernel<16, B> : moe_route_kernel<32, B>;
    };
    auto* kernel = p.bf16 ? pick(std::true_type{}) : pick(std::false_type{});
    return launch_pdl(kernel, dim3((unsigned)((p.m + 3) / 4)), dim3(128), 0, s, a);
}

}  // namespace q2k
