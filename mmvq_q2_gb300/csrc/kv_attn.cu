// Attention of new tokens over the paged cache (include/q2k.h,
// kv_attention_bf16).
#include <algorithm>
#include <cmath>

#include "q2k_common.cuh"
#include "q2k_internal.h"

namespace q2k {

__device__ int g_attn_error = 0;

namespace {

constexpr int kErrBadPage = 2;

struct AttnArgs {
    const uint16_t *q, *k, *v;
    uint16_t* out;
    float* lse;
    const int32_t *table, *cu_q, *seq_lens;
    int64_t ld_q, ld_o, ld_table, max_pages, n_pages, page_stride;
    int T, Hq, Hkv, D, n_req, shift, window;
    float scale;
};

// One warp a (token, head): 32 keys at a time, a key's score in each lane,
// then the lanes share the values' columns.  Running maximum and sum.
__global__ void __launch_bounds__(128) kv_attn_kernel(const AttnArgs a)
{
    __shared__ float q_s[4][128];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + warp;
    if (row >= (int64_t)a.T * a.Hq)
        return;
    const int t = (int)(row / a.Hq), head = (int)(row % a.Hq), kvh = head / (a.Hq / a.Hkv);
    if (t >= a.cu_q[a.n_req])
        return;
    int r = 0, hi_r = a.n_req;
    while (hi_r - r > 1) {
        const int mid = (r + hi_r) / 2;
        if (a.cu_q[mid] <= t)
            r = mid;
        else
            hi_r = mid;
    }
    const int p = a.seq_lens[r] - (a.cu_q[r + 1] - t);
    const int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
    for (int d = lane; d < a.D; d += 32)
        q_s[warp][d] = bf16_bits_f(a.q[t * a.ld_q + (int64_t)head * a.D + d]) * a.scale;
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = lo; j0 <= p; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY;
        int64_t at = -1;
        if (j <= p) {
            const int col = j >> a.shift;
            const int page = col < a.max_pages ? a.table[r * a.ld_table + col] : -1;
            s = 0.f;
            if (page >= 0 && page < a.n_pages) {
                at = page * a.page_stride + (((int64_t)kvh << a.shift) + (j & ((1 << a.shift) - 1))) * a.D;
                for (int d = 0; d < a.D; ++d)
                    s = fmaf(q_s[warp][d], bf16_bits_f(a.k[at + d]), s);
            } else {
                atomicOr(&g_attn_error, kErrBadPage);
            }
        }
        float top = s;
#pragma unroll
        for (int i = 16; i >= 1; i >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
        const float mn = fmaxf(m, top);
        const float shrink = expf(m - mn), e = expf(s - mn);
        l *= shrink;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            o[c] *= shrink;
        m = mn;
        float sum = e;
#pragma unroll
        for (int i = 16; i >= 1; i >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, i);
        l += sum;
        for (int i = 0; i < 32 && j0 + i <= p; ++i) {
            const float w = __shfl_sync(0xffffffffu, e, i);
            const int64_t src = __shfl_sync(0xffffffffu, at, i);
            if (src >= 0) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c * 32 + lane < a.D)
                        o[c] = fmaf(w, bf16_bits_f(a.v[src + c * 32 + lane]), o[c]);
            }
        }
    }
    const float inv = l > 0.f ? 1.0f / l : 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (c * 32 + lane < a.D)
            a.out[t * a.ld_o + (int64_t)head * a.D + c * 32 + lane] =
                __bfloat16_as_ushort(__float2bfloat16_rn(o[c] * inv));
    if (a.lse && lane == 0)
        a.lse[(int64_t)t * a.Hq + head] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t kv_attention_workspace(int64_t, int64_t, int64_t, int64_t) { return 16; }

cudaError_t launch_kv_attention(const AttnProblem& p, cudaStream_t s)
{
    AttnArgs a{};
    a.q = p.q;
    a.k = p.k_cache;
    a.v = p.v_cache;
    a.out = p.out;
    a.lse = p.lse;
    a.table = p.block_table;
    a.cu_q = p.cu_q;
    a.seq_lens = p.seq_lens;
    a.ld_q = p.ld_q;
    a.ld_o = p.ld_o;
    a.max_pages = p.max_pages;
    a.ld_table = p.ld_table;
    a.n_pages = p.n_pages;
    a.page_stride = p.page_stride;
    a.T = (int)p.T;
    a.Hq = (int)p.Hq;
    a.Hkv = (int)p.Hkv;
    a.D = (int)p.D;
    a.n_req = (int)p.n_req;
    a.window = (int)std::min<int64_t>(p.window, 0x7fffffff);
    a.scale = p.scale;
    while ((1 << a.shift) < p.page_size)
        ++a.shift;
    return launch_pdl(kv_attn_kernel, dim3((unsigned)((p.T * p.Hq + 3) / 4)), dim3(128), 0, s, a);
}

cudaError_t attn_error_word(int32_t* out, bool clear)
{
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_error, sizeof(int));
    if (e != cudaSuccess)
        return e;
    *out = v;
    if (clear) {
        int z = 0;
        e = cudaMemcpyToSymbol(g_attn_error, &z, sizeof(int));
    }
    return e;
}

}  // namespace q2k
