// The paged cache's bookkeeping and its writer (include/q2k.h,
// kv_page_plan and kv_rope_store).
#include <algorithm>
#include <climits>

#include "q2k_common.cuh"
#include "q2k_internal.h"

namespace q2k {

namespace {

// ---- kv_page_plan --------------------------------------------------------------
//
// All whole numbers: the sums of the new tokens and of the pages they open
// over the requests, then one table lookup per token.  What bounds it is
// latency (a step's lengths are a few KB), so there is one launch and no
// block waits for another: each block scans all lengths itself, keeps both
// prefix sums in shared memory and fills its share of the tokens and of the
// new pages by binary search.  (Without a token to place a call takes 1.8 us
// for up to 128 requests, 3.1 for 1000, 35 for 16384; with a token for each
// 2.6, 5.0 and 37.  A launch of its own for the sums would take the same scan
// and come before the other.)  Slots in a page opened by this very call
// come from the free list, not from the table, so blocks do not depend on
// one another's writes.

constexpr int kPlanThreads = 512;

struct PlanArgs {
    const int32_t *ctx, *add, *free_pages, *free_head;
    int32_t *table, *cu_q, *seq_lens, *positions, *token_req, *slot_map, *head_out, *err;
    int64_t max_pages, ld_table, n_free;
    int n, shift, max_tokens;
};

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int shift) { return (tokens + (1 << shift) - 1) >> shift; }

// The last r with sums[r] <= i (sums[0] = 0, sums[n] > i).
__device__ __forceinline__ int find_request(const int32_t* sums, int n, int i)
{
    int lo = 0, hi = n;  // sums[lo] <= i < sums[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) kv_page_plan_kernel(const PlanArgs a)
{
    extern __shared__ int64_t plan_smem[];
    int64_t* warp_new = plan_smem;                    // one sum a warp
    int64_t* warp_need = plan_smem + kPlanThreads / 32;
    int32_t* cu = reinterpret_cast<int32_t*>(plan_smem + kPlanThreads / 16);  // [n + 1] new tokens before request r, cut at max_tokens
    int32_t* need = cu + a.n + 1;                                             // [n + 1] pages opened before request r, cut at INT_MAX
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    if (threadIdx.x == 0)
        cu[0] = need[0] = 0;
    int err = 0;
    int64_t base_new, base_need;
    // Where there are more new tokens than max_tokens, once more for those
    // that are kept: lengths, pages and positions then fit one another, and
    // the rest can be the next step.
    bool cut = false;
    for (;;) {
        base_new = base_need = 0;
        for (int r0 = 0; r0 < a.n; r0 += kPlanThreads) {
            const int r = r0 + (int)threadIdx.x;
            int64_t nw = 0, nd = 0;
            if (r < a.n) {
                int c = a.ctx[r], w = a.add[r];
                if (c < 0 || w < 0)
                    err |= 4;
                c = max(c, 0);
                w = cut ? cu[r + 1] - cu[r] : max(w, 0);
                const int64_t seq = (int64_t)c + w;
                if (blockIdx.x == 0)
                    a.seq_lens[r] = (int32_t)min(seq, (int64_t)INT_MAX);
                if (w > 0 && seq > (a.max_pages << a.shift))
                    err |= 2;
                nw = w;
                // pages past the table's row cannot be recorded and are not taken
                nd = min(pages_of(seq, a.shift), a.max_pages) - min(pages_of(c, a.shift), a.max_pages);
            }
            int64_t sn = nw, sd = nd;  // inclusive sums over the block
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, sn, o), v = __shfl_up_sync(0xffffffffu, sd, o);
                if (lane >= o) {
                    sn += u;
                    sd += v;
                }
            }
            if (lane == 31) {
                warp_new[warp] = sn;
                warp_need[warp] = sd;
            }
            __syncthreads();
            int64_t tn = 0, td = 0;
            for (int w = 0; w < kPlanThreads / 32; ++w) {
                if (w == warp) {
                    sn += base_new + tn;
                    sd += base_need + td;
                }
                tn += warp_new[w];
                td += warp_need[w];
            }
            if (r < a.n) {
                cu[r + 1] = (int32_t)min(sn, (int64_t)a.max_tokens);
                need[r + 1] = (int32_t)min(sd, (int64_t)INT_MAX);
                if (blockIdx.x == 0)
                    a.cu_q[r + 1] = cu[r + 1];
            }
            base_new += tn;
            base_need += td;
            __syncthreads();
        }
        if (base_new <= a.max_tokens)
            break;
        cut = true;
        err &= ~2;  // asked again of what is kept
    }
    int head = a.free_head ? *a.free_head : 0;
    if (head < 0) {
        head = 0;
        err |= 4;
    }
    if (threadIdx.x == 0) {
        if (cut)
            err |= 8;
        if (head + base_need > a.n_free && base_need > 0)
            err |= 1;
        if (blockIdx.x == 0) {
            a.cu_q[0] = 0;
            *a.head_out = (int32_t)max((int64_t)head, min(head + base_need, min(a.n_free, (int64_t)INT_MAX)));
        }
    }
    if (blockIdx.x == 0 && a.err && err)
        atomicOr(a.err, err);
    __syncthreads();

    const int stride = (int)(gridDim.x * blockDim.x);
    const int first = (int)(blockIdx.x * blockDim.x + threadIdx.x);
    const int total = cu[a.n], pages = need[a.n];
    for (int64_t i = first; i < pages; i += stride) {
        const int r = find_request(need, a.n, (int)i);
        const int64_t col = pages_of(max(a.ctx[r], 0), a.shift) + (i - need[r]);
        const int64_t at = head + i;
        if (col < a.max_pages)
            a.table[r * a.ld_table + col] = at < a.n_free ? a.free_pages[at] : -1;
    }
    for (int64_t t = first; t < a.max_tokens; t += stride) {
        int pos = -1, slot = -1, r = -1;
        if (t < total) {
            r = find_request(cu, a.n, (int)t);
            const int c = max(a.ctx[r], 0);
            const int64_t p = (int64_t)c + (t - cu[r]);
            pos = (int)min(p, (int64_t)INT_MAX);
            const int64_t col = p >> a.shift, have = pages_of(c, a.shift);
            int page = -1;
            if (col < have) {
                if (col < a.max_pages)
                    page = a.table[r * a.ld_table + col];
            } else if (col < a.max_pages) {
                const int64_t at = (int64_t)head + need[r] + (col - have);
                if (at < a.n_free)
                    page = a.free_pages[at];
            }
            if (page >= 0 && page <= (INT_MAX >> a.shift))
                slot = (page << a.shift) + (int)(p & ((1 << a.shift) - 1));
        }
        a.positions[t] = pos;
        a.token_req[t] = r;
        a.slot_map[t] = slot;
    }
}

// ---- kv_rope_store -------------------------------------------------------------
//
// Bound by memory: every value is read once (fp32 or bf16) and written once
// (bf16).  The angles of a token are the same for all heads, so a block
// takes whole tokens, computes rot/2 sines and cosines per token into shared
// memory (accurate sincosf: positions reach far beyond 2 pi) while its first
// values are already on their way to registers, and turns them from there.

struct RopeArgs {
    const void *q, *k, *v;
    int64_t ld_q, ld_k, ld_v, ld_qo;
    const int32_t *positions, *slot_map;
    const float* inv_freq;
    uint16_t *q_out, *k_cache, *v_cache;
    int32_t* err;
    int64_t T, n_slots, page_stride;
    int Hq, Hkv, D, half, interleaved, shift;
    int sec0, sec1;  // pairs below sec0 turn by axis 0, below sec1 by axis 1, others by axis 2
    int tokens;      // tokens of one block
};

__device__ __forceinline__ void rope_angles(const RopeArgs& a, int64_t t0, float2* cs)
{
    const int tid = (int)(threadIdx.y * blockDim.x + threadIdx.x), nt = (int)(blockDim.x * blockDim.y);
    for (int i = tid; i < a.tokens * a.half; i += nt) {
        const int t = a.tokens == 1 ? 0 : i / a.half, p = i - t * a.half;
        if (t0 + t >= a.T)
            break;
        const int axis = p < a.sec0 ? 0 : p < a.sec1 ? 1 : 2;
        const float ang = __fmul_rn((float)a.positions[axis * a.T + t0 + t], a.inv_freq[p]);
        float s, c;
        sincosf(ang, &s, &c);
        cs[i] = make_float2(c, s);
    }
}

// Where head `row` (q heads, then k, then v) of token t is read and written;
// dst is NULL where the token is not stored.
template <typename T>
__device__ __forceinline__ void rope_row(const RopeArgs& a, int64_t t, int row, const T*& src, uint16_t*& dst)
{
    if (row < a.Hq) {
        src = static_cast<const T*>(a.q) + t * a.ld_q + (int64_t)row * a.D;
        dst = a.q_out + t * a.ld_qo + (int64_t)row * a.D;
        return;
    }
    const bool is_v = row >= a.Hq + a.Hkv;
    const int h = row - a.Hq - (is_v ? a.Hkv : 0);
    src = is_v ? static_cast<const T*>(a.v) + t * a.ld_v + (int64_t)h * a.D
               : static_cast<const T*>(a.k) + t * a.ld_k + (int64_t)h * a.D;
    const int slot = a.slot_map[t];
    dst = nullptr;
    if (slot < 0)
        return;
    if (slot >= a.n_slots) {
        if (a.err)
            *a.err = 1;
        return;
    }
    const int64_t page = slot >> a.shift, off = slot & ((1 << a.shift) - 1);
    dst = (is_v ? a.v_cache : a.k_cache) + page * a.page_stride + (((int64_t)h << a.shift) + off) * a.D;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(uint16_t v) { return bf16_bits_f(v); }
__device__ __forceinline__ uint16_t to_bf16(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// 32 bytes in one load where they are aligned so: two of 16 touch every
// sector twice.
__device__ __forceinline__ void load8(const float* p, float (&v)[8])
{
    if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
        asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "l"(p));
        return;
    }
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8])
{
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // two values an instruction
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The 8 pairs of a rotated part: (u, w) value by value, or side by side.
__device__ __forceinline__ void turn16(const RopeArgs& a, const float2* p, float (&u)[8], float (&w)[8])
{
    if (!a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = u[i], y = w[i];
            u[i] = x * p[i].x - y * p[i].y;
            w[i] = y * p[i].x + x * p[i].y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = u[2 * i], y = u[2 * i + 1];
            u[2 * i] = x * p[i].x - y * p[i].y;
            u[2 * i + 1] = y * p[i].x + x * p[i].y;
            const float z = w[2 * i], z2 = w[2 * i + 1];
            w[2 * i] = z * p[4 + i].x - z2 * p[4 + i].y;
            w[2 * i + 1] = z2 * p[4 + i].x + z * p[4 + i].y;
        }
    }
}

// 16 values a thread: threadIdx.x is the part of the head (D / 16 of them),
// threadIdx.y the head of one of the block's tokens.
template <typename T>
__global__ void __launch_bounds__(512, 2) kv_rope_vec_kernel(const RopeArgs a)
{
    extern __shared__ float2 cs[];  // [tokens][half] cosine, sine
    pdl_launch_dependents();
    pdl_wait();
    const int heads = a.Hq + 2 * a.Hkv;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int part = (int)threadIdx.x;
    const int rot_parts = a.half / 8;
    bool ready = false;
    for (int y = (int)threadIdx.y; y < a.tokens * heads || !ready; y += (int)blockDim.y) {
        const int tl = a.tokens == 1 ? 0 : y / heads, row = y - tl * heads;
        const int64_t t = t0 + tl;
        const bool live = y < a.tokens * heads && t < a.T;
        const T* src = nullptr;
        uint16_t* dst = nullptr;
        float u[8], w[8];
        const bool turn = row < a.Hq + a.Hkv && part < rot_parts;
        // the two runs of 8 values: a rotated part holds 8 pairs
        const int o1 = turn && !a.interleaved ? part * 8 : part * 16;
        const int o2 = turn && !a.interleaved ? a.half + part * 8 : part * 16 + 8;
        if (live) {
            rope_row<T>(a, t, row, src, dst);
            if (dst) {
                load8(src + o1, u);
                load8(src + o2, w);
            }
        }
        if (!ready) {
            rope_angles(a, t0, cs);
            __syncthreads();
            ready = true;
        }
        if (!live || !dst)
            continue;
        if (turn)
            turn16(a, cs + tl * a.half + part * 8, u, w);
        store8(dst + o1, u);
        store8(dst + o2, w);
    }
}

// The same for many tokens where a token fills a block: a thread keeps its
// part of its head through kRopeGroup tokens, whose angles are worked out at
// once (one token a block, the block waited for its sines longer than for
// its values), with the next token's values on their way.
constexpr int kRopeGroup = 4;

template <typename T>
__global__ void __launch_bounds__(512, 2) kv_rope_group_kernel(const RopeArgs a)
{
    extern __shared__ float2 cs[];  // [kRopeGroup][half] cosine, sine
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * kRopeGroup;
    const int n = (int)min((int64_t)kRopeGroup, a.T - t0);
    const int part = (int)threadIdx.x, row = (int)threadIdx.y;
    const bool turn = row < a.Hq + a.Hkv && part < a.half / 8;
    const int o1 = turn && !a.interleaved ? part * 8 : part * 16;
    const int o2 = turn && !a.interleaved ? a.half + part * 8 : part * 16 + 8;
    float u[8], w[8], u2[8], w2[8];
    uint16_t *dst = nullptr, *dst2 = nullptr;
    auto fetch = [&](int tl, float (&x)[8], float (&y)[8], uint16_t*& to) {
        const T* src;
        rope_row<T>(a, t0 + tl, row, src, to);
        if (to) {
            load8(src + o1, x);
            load8(src + o2, y);
        }
    };
    fetch(0, u, w, dst);
    rope_angles(a, t0, cs);
    __syncthreads();
    for (int tl = 0; tl < n; ++tl) {
        if (tl + 1 < n)
            fetch(tl + 1, u2, w2, dst2);
        if (dst) {
            if (turn)
                turn16(a, cs + tl * a.half + part * 8, u, w);
            store8(dst + o1, u);
            store8(dst + o2, w);
        }
        dst = dst2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u[i] = u2[i];
            w[i] = w2[i];
        }
    }
}

// Any D, rot and alignment: a value (or pair) a step, threads over the head.
template <typename T>
__global__ void __launch_bounds__(256) kv_rope_any_kernel(const RopeArgs a)
{
    extern __shared__ float2 cs[];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = blockIdx.x;
    rope_angles(a, t, cs);
    __syncthreads();
    const int heads = a.Hq + 2 * a.Hkv;
    for (int row = (int)threadIdx.y; row < heads; row += (int)blockDim.y) {
        const T* src;
        uint16_t* dst;
        rope_row<T>(a, t, row, src, dst);
        if (!dst)
            continue;
        const int pairs = row < a.Hq + a.Hkv ? a.half : 0;
        for (int i = (int)threadIdx.x; i < pairs; i += (int)blockDim.x) {
            const int i1 = a.interleaved ? 2 * i : i, i2 = a.interleaved ? 2 * i + 1 : i + a.half;
            const float x = to_f(src[i1]), y = to_f(src[i2]);
            dst[i1] = to_bf16(x * cs[i].x - y * cs[i].y);
            dst[i2] = to_bf16(y * cs[i].x + x * cs[i].y);
        }
        for (int i = 2 * pairs + (int)threadIdx.x; i < a.D; i += (int)blockDim.x)
            dst[i] = to_bf16(to_f(src[i]));
    }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

cudaError_t launch_kv_page_plan(const PagePlan& p, cudaStream_t s)
{
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess)
        return e;
    PlanArgs a{};
    a.ctx = p.ctx_lens;
    a.add = p.new_lens;
    a.free_pages = p.free_pages;
    a.free_head = p.free_head;
    a.table = p.block_table;
    a.cu_q = p.cu_q;
    a.seq_lens = p.seq_lens;
    a.positions = p.positions;
    a.token_req = p.token_req;
    a.slot_map = p.slot_map;
    a.head_out = p.free_head_out;
    a.err = p.err_flag;
    a.max_pages = p.max_pages;
    a.ld_table = p.ld_table;
    a.n_free = p.n_free;
    a.n = (int)p.n_req;
    a.max_tokens = (int)p.max_tokens;
    while ((1 << a.shift) < p.page_size)
        ++a.shift;
    static std::atomic<unsigned long long> smem_devs{0};
    if ((e = allow_max_smem(kv_page_plan_kernel, smem_devs)) != cudaSuccess)
        return e;
    const size_t smem = (size_t)kPlanThreads / 16 * sizeof(int64_t) + (size_t)(a.n + 1) * 2 * sizeof(int32_t);
    // two tokens a thread: more blocks only repeat the scan
    const int64_t want = (p.max_tokens + 2 * kPlanThreads - 1) / (2 * kPlanThreads);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(want, di.sm_count));
    return launch_pdl(kv_page_plan_kernel, dim3(grid), dim3(kPlanThreads), smem, s, a);
}

cudaError_t launch_kv_rope_store(const RopeStore& p, cudaStream_t s)
{
    RopeArgs a{};
    a.q = p.q;
    a.k = p.k;
    a.v = p.v;
    a.ld_q = p.ld_q;
    a.ld_k = p.ld_k;
    a.ld_v = p.ld_v;
    a.ld_qo = p.ld_qo;
    a.positions = p.positions;
    a.slot_map = p.slot_map;
    a.inv_freq = p.inv_freq;
    a.q_out = p.q_out;
    a.k_cache = p.k_cache;
    a.v_cache = p.v_cache;
    a.err = p.err_flag;
    a.T = p.T;
    a.n_slots = p.n_pages * p.page_size;
    a.page_stride = p.page_stride;
    a.Hq = p.q ? (int)p.Hq : 0;
    a.Hkv = (int)p.Hkv;
    a.D = (int)p.D;
    a.half = (int)p.rot / 2;
    a.interleaved = p.interleaved;
    a.sec0 = p.sections[0];
    a.sec1 = p.sections[0] + p.sections[1];
    while ((1 << a.shift) < p.page_size)
        ++a.shift;
    const int heads = a.Hq + 2 * a.Hkv;
    const int in8 = p.x_bf16 ? 8 : 4;  // elements of 16 bytes
    const bool vec = a.D % 16 == 0 && p.rot % 16 == 0 && on16(a.k) && on16(a.v) && on16(a.k_cache) && on16(a.v_cache) &&
                     a.ld_k % in8 == 0 && a.ld_v % in8 == 0 &&
                     (!a.Hq || (on16(a.q) && on16(a.q_out) && a.ld_q % in8 == 0 && a.ld_qo % 8 == 0));
    if (vec) {
        const int parts = a.D / 16;
        DeviceInfo di;
        cudaError_t e = device_info(&di);
        if (e != cudaSuccess)
            return e;
        // groups where they are enough for two waves of two blocks an SM
        if (parts * heads > 128 && parts * heads <= 512 && p.T >= (int64_t)4 * kRopeGroup * di.sm_count) {
            a.tokens = kRopeGroup;
            return launch_pdl(p.x_bf16 ? kv_rope_group_kernel<uint16_t> : kv_rope_group_kernel<float>,
                              dim3((unsigned)((p.T + kRopeGroup - 1) / kRopeGroup)), dim3(parts, heads),
                              (size_t)kRopeGroup * a.half * sizeof(float2), s, a);
        }
        // whole tokens to about 256 threads; a token of more heads takes up to 512 and then loops
        a.tokens = (int)std::max<int64_t>(1, std::min<int64_t>(256 / (parts * heads), p.T));
        const int rows = std::min(a.tokens * heads, 512 / parts);
        const size_t smem = (size_t)a.tokens * a.half * sizeof(float2);
        const unsigned grid = (unsigned)((p.T + a.tokens - 1) / a.tokens);
        return launch_pdl(p.x_bf16 ? kv_rope_vec_kernel<uint16_t> : kv_rope_vec_kernel<float>, dim3(grid),
                          dim3(parts, rows), smem, s, a);
    }
    a.tokens = 1;
    return launch_pdl(p.x_bf16 ? kv_rope_any_kernel<uint16_t> : kv_rope_any_kernel<float>, dim3((unsigned)p.T),
                      dim3(32, 8), (size_t)a.half * sizeof(float2), s, a);
}

}  // namespace q2k
