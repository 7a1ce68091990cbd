// Products of few tokens over 8-bit floating-point weights (include/q2k.h):
// fp8_gemm for up to 32 rows, and fp8_moe, the routed experts of a few tokens.
//
// Bound by memory: each weight is read once and used for a handful of tokens.
// A persistent CTA an SM walks items of 32 weight rows.  One warp copies the
// rows, 512 values at a time, into a ring of shared-memory stages, a tensor
// copy each (with a bulk copy a row, 73 cycles each, their issue was the
// bound: 2.0 TB/s).  Two groups of four warps take turns at the stages; a
// warp feeds its 128 values of all 32 rows to the tensor cores as they are
// (mma.sync m16n8k32 on e4m3, weights as the 16 rows, tokens as the 8
// columns), scales each block's sums in fp32 and adds them up.  Three more
// warps join the eight through shared memory and store, while those go on
// with the next item (with the eight doing it themselves, fp8_moe's second
// launch, with its counters, took twice the time).  (The
// 5th-generation tensor cores would want 128 weight rows or tokens a tile; at
// these sizes the MMAs take a few percent of the time either way.)
//
// A thread needs 4 values of a row for each MMA.  Since the order along K is
// free as long as both operands share it, it takes 16 neighbouring bytes of
// its row and feeds them to two MMAs: one 16-byte load a row and 64 values.
// The copies swizzle lines of 128 bytes, so that the loads of two rows meet no
// bank twice; rows that are no multiple of 128 bytes cannot be cut into such
// lines and lie as they are (loads then take twice the cycles).
//
// bf16 tokens (fp8_moe) enter as two columns of e4m3 each: with a power of
// two that brings a block's largest below 256, the upper 4 bits of a value
// are one e4m3 number and what is left, times 16, another.  Together they are
// the bf16 value exactly, where it is within 2^-13 of the block's largest (and
// off by less than 2^-20 of that below).  The weights need no conversion that
// way: expanding them to bf16 costs 2 to 4 instructions a pair, more than the
// streaming leaves room for.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "q2k_common.cuh"
#include "q2k_internal.h"

namespace q2k {

__device__ int g_fp8_stream_error = 0;

namespace {

constexpr int kWarps = 8;                      // that compute, in two groups; one more copies
constexpr int kEndWarps = 3;                   // that join and store
constexpr int kThreads = (kWarps + 1 + kEndWarps) * 32;
constexpr int kRows = 32;                      // weight rows of an item
constexpr int kChunk = 512;                    // values of a row in a stage
constexpr int kWStage = kRows * kChunk;
constexpr int kMaxPairs = 1024, kMaxExperts = 1024;

enum Mode : int { GEMM = 0, UP = 1, DOWN = 2 };

struct StreamArgs {
    const uint8_t* W;
    const float* w_scales;
    int K, blocks;      // blocks of 128 along K
    int rows;           // weight rows: N; inter (UP); dim (DOWN)
    int row_blocks;     // of w_scales
    int tiles;          // items of one matrix
    int stages, stage_bytes;  // stages: an even number, so that a stage is always the same group's
    int swizzled;             // lines of 128 bytes
    int k_step, block_step;   // coordinates of a chunk: (0, 4 blocks) swizzled, (128 words, 0) otherwise
    int m;
    // GEMM
    const uint8_t* x;
    const float* x_scales;
    int64_t ldx, ld_xs;
    // fp8_moe
    const uint16_t* xb;     // bf16 rows: tokens (UP) or h of the pairs (DOWN)
    const int32_t* ids;
    const float* route_w;
    int topk, E;
    uint16_t* h;            // [pairs, inter]
    float* part;            // [pairs, dim]
    int* done;              // [tiles of dim]
    int done_count;
    // results
    void* y;
    int64_t ldy;
    int y_bf16;
};

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two floats as e4m3, and back.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t v)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
    return make_float2(half_lo_f(h), half_hi_f(h));
}

// The computing warps among themselves, and those that end items.
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }
__device__ __forceinline__ void enders_sync() { asm volatile("bar.sync 6, %0;" ::"n"(kEndWarps * 32) : "memory"); }
// Between the two: buffer `buf` is full, or free again; one side arrives, the other waits.
constexpr int kBothSides = (kWarps + kEndWarps) * 32;
__device__ __forceinline__ void pair_arrive(int id) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kBothSides) : "memory"); }
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kBothSides) : "memory"); }
constexpr int kBarFull = 2, kBarFree = 4;

// The experts that have a token, as passes of up to CAP (token, choice) pairs.
struct Lists {
    int ids[kMaxPairs];
    uint16_t rank[kMaxPairs], list[kMaxPairs];                         // pairs by expert, in order
    uint16_t v_expert[kMaxPairs], v_first[kMaxPairs], v_count[kMaxPairs];  // passes
    uint16_t count[kMaxExperts];
    int passes;
};

// By all threads; ends with a barrier.
__device__ void build_lists(Lists& l, const StreamArgs& a, int cap)
{
    const int pairs = a.m * a.topk, tid = threadIdx.x;
    for (int i = tid; i < a.E; i += kThreads)
        l.count[i] = 0;
    for (int i = tid; i < pairs; i += kThreads)
        l.ids[i] = a.ids[i];
    __syncthreads();
    if (tid < 32) {
        // a pair's place among those of its expert, 32 pairs at a time
        for (int i0 = 0; i0 < pairs; i0 += 32) {
            const int i = i0 + tid;
            const int e = i < pairs ? l.ids[i] : -1;
            const bool valid = e >= 0 && e < a.E;
            const uint32_t same = __match_any_sync(0xffffffffu, valid ? e : -1);
            const int before = valid ? l.count[e] : 0;
            __syncwarp();
            if (valid) {
                l.rank[i] = (uint16_t)(before + __popc(same & ((1u << tid) - 1u)));
                if ((same >> tid) == 1u)  // the last of them
                    l.count[e] = (uint16_t)(before + __popc(same));
            }
            __syncwarp();
        }
        // each lane a run of experts: first pair and first pass of each
        const int run = (a.E + 31) / 32, e0 = tid * run, e1 = min(a.E, e0 + run);
        int n = 0, v = 0;
        for (int e = e0; e < e1; ++e) {
            n += l.count[e];
            v += (l.count[e] + cap - 1) / cap;
        }
        int n_at = n, v_at = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int pn = __shfl_up_sync(0xffffffffu, n_at, o), pv = __shfl_up_sync(0xffffffffu, v_at, o);
            if (tid >= o) {
                n_at += pn;
                v_at += pv;
            }
        }
        if (tid == 31)
            l.passes = v_at;
        n_at -= n;
        v_at -= v;
        for (int e = e0; e < e1; ++e) {
            const int c = l.count[e];
            l.count[e] = (uint16_t)n_at;  // from here on the expert's first place
            for (int at = 0; at < c; at += cap, ++v_at) {
                l.v_expert[v_at] = (uint16_t)e;
                l.v_first[v_at] = (uint16_t)(n_at + at);
                l.v_count[v_at] = (uint16_t)min(cap, c - at);
            }
            n_at += c;
        }
    }
    __syncthreads();
    for (int i = tid; i < pairs; i += kThreads) {
        const int e = l.ids[i];
        if (e >= 0 && e < a.E)
            l.list[l.count[e] + l.rank[i]] = (uint16_t)i;
    }
    __syncthreads();
}

// A block of 128 bf16 values, 4 a lane, as two rows of e4m3 and their scale.
__device__ __forceinline__ void split_block(const float (&v)[4], uint8_t* upper, uint8_t* lower, float* scale)
{
    const uint32_t top = __reduce_max_sync(
        0xffffffffu, max(max(__float_as_uint(v[0]) & 0x7fffffffu, __float_as_uint(v[1]) & 0x7fffffffu),
                         max(__float_as_uint(v[2]) & 0x7fffffffu, __float_as_uint(v[3]) & 0x7fffffffu)));
    // 2^(7 - e) of the largest's exponent e, within fp32's powers of two for it and its inverse
    const uint32_t e = min(max(top >> 23, 20u), 254u);
    const float f = __uint_as_float((261u - e) << 23), inv = __uint_as_float((e - 7u) << 23);
    float w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = v[j] * f;
        if ((__float_as_uint(v[j]) & 0x7fffffffu) >= 0x7f800000u)
            w[j] = __uint_as_float(0x7fffffffu);  // infinity too: e4m3 has none
    }
    const uint32_t u0 = e4m3x2(w[0], w[1]), u1 = e4m3x2(w[2], w[3]);
    const float2 r0 = from_e4m3x2(u0), r1 = from_e4m3x2(u1);
    const uint32_t l0 = e4m3x2((w[0] - r0.x) * 16.f, (w[1] - r0.y) * 16.f);
    const uint32_t l1 = e4m3x2((w[2] - r1.x) * 16.f, (w[3] - r1.y) * 16.f);
    *reinterpret_cast<uint32_t*>(upper) = u0 | u1 << 16;
    *reinterpret_cast<uint32_t*>(lower) = l0 | l1 << 16;
    if ((threadIdx.x & 31) == 0)
        *scale = inv;
}

// A box of 512 bytes by rows, by gate and up, by expert.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int k, int block, int row, int expert, uint32_t bar,
                                         uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(block), "r"(row), "r"(0), "r"(expert), "r"(bar), "l"(policy)
        : "memory");
}

template <int MODE, int NT>
struct Shared {
    static constexpr int kTok = MODE == GEMM ? 8 * NT : 4 * NT;  // tokens of a pass
    uint64_t full[16], empty[16];
    static constexpr int kBufs = MODE == GEMM && NT == 4 ? 1 : 2;
    int abort_flag, issued, last;
    float red[kBufs][2][kWarps][kTok * 20];  // [buffer][row tile][warp]: 16 rows of a token, 20 apart
    Lists lists[MODE == GEMM ? 0 : 1];
};

template <int MODE, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_stream_kernel(const StreamArgs a, const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx)
{
    using Sh = Shared<MODE, NT>;
    constexpr int TOK = Sh::kTok;
    extern __shared__ __align__(1024) uint8_t smem[];
    // the 128-byte swizzle repeats every 1024 bytes: stages start on 1024
    uint8_t* const ring = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u);
    Sh& sh = *reinterpret_cast<Sh*>(ring + (size_t)a.stages * a.stage_bytes);
    constexpr int kFixed = ((int)sizeof(Sh) + 127) / 128 * 128;
    float* const xs = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(&sh) + kFixed);  // [blocks][TOK]
    uint8_t* const cols = reinterpret_cast<uint8_t*>(xs) + (a.blocks * TOK * 4 + 127) / 128 * 128;
    const int col_pitch = a.blocks * 128 + 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), kWarps / 2);
        }
        sh.abort_flag = 0;
        sh.issued = 0;
        fence_mbar_init();
    }
    // UP lets DOWN start only once what came before is complete: DOWN reads ids
    // and weights before it waits for UP.
    if (MODE != DOWN)
        pdl_wait();
    pdl_launch_dependents();
    int passes = 1;
    if constexpr (MODE != GEMM) {
        build_lists(sh.lists[0], a, TOK);
        passes = sh.lists[0].passes;
    } else {
        for (int i = threadIdx.x; i < a.blocks * TOK; i += kThreads) {
            const int b = i / TOK, t = i % TOK;
            xs[i] = t < a.m ? a.x_scales[t * a.ld_xs + b] : 0.f;
        }
        __syncthreads();
    }
    const int total = passes * a.tiles;
    const int first = (int)((int64_t)blockIdx.x * total / gridDim.x);
    const int end = (int)((int64_t)(blockIdx.x + 1) * total / gridDim.x);
    const int n_chunks = (a.K + kChunk - 1) / kChunk;

    volatile int* const abort_flag = &sh.abort_flag;
    auto give_up = [&]() {
        atomicOr(&g_fp8_stream_error, Q2K_ERR_BIT_WAIT_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp == kWarps) {
        if (lane == 0) {  // copies
            const uint64_t wpol = l2_policy_evict_first(), xpol = l2_policy_evict_last();
            int slot = 0, use = 0;
            bool ok = true;
            for (int it = first; it < end && ok; ++it) {
                const int v = it / a.tiles, tile = it - v * a.tiles;
                const int row = tile * (MODE == UP ? 16 : kRows);
                const int expert = MODE == GEMM ? 0 : sh.lists[0].v_expert[v];
                for (int c = 0; c < n_chunks; ++c) {
                    if (use > 0 && !mbar_wait_bounded(smem_u32(&sh.empty[slot]), (uint32_t)(use - 1) & 1u, abort_flag)) {
                        give_up();
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_u32(&sh.full[slot]);
                    const uint32_t dst = smem_u32(ring + (size_t)slot * a.stage_bytes);
                    mbar_arrive_expect_tx(bar, (uint32_t)a.stage_bytes);
                    copy_box(dst, &tw, c * a.k_step, c * a.block_step, row, expert, bar, wpol);
                    if (MODE == GEMM)
                        copy_box(dst + kWStage, &tx, c * a.k_step, c * a.block_step, 0, 0, bar, xpol);
                    sh.issued = sh.issued + 1;
                    if (++slot == a.stages) {
                        slot = 0;
                        ++use;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp < kWarps) {
        if (MODE == DOWN)
            pdl_wait();
        const int kb = warp & 3, group = warp >> 2, g = lane >> 2, c4 = lane & 3;
        int slot = group, use = 0, turn = 0, cur_v = -1, n_tok = a.m, buf = 0;
        // where this thread's 16 bytes of a row's two halves lie
        int at[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            at[h] = kb * 128 + 16 * (a.swizzled ? (4 * h + c4) ^ (kb | (g & 1) << 2) : 4 * h + c4);
        // scale of this warp's block of chunk `lane`, fetched an item ahead
        auto scale_of = [&](int it, int chunk, int part) {
            const int b = chunk * 4 + kb;
            if (it >= end || b >= a.blocks)
                return 0.f;
            const int v = it / a.tiles, tile = it - v * a.tiles;
            int64_t row_block;
            if (MODE == GEMM)
                row_block = tile * kRows / 128;
            else if (MODE == UP)
                row_block = ((int64_t)sh.lists[0].v_expert[v] * 2 + part) * a.row_blocks + tile * 16 / 128;
            else
                row_block = (int64_t)sh.lists[0].v_expert[v] * a.row_blocks + tile * kRows / 128;
            return a.w_scales[row_block * a.blocks + b];
        };
        // (gate and up have scales of their own; otherwise both row tiles share one)
        float next_ws[2] = {scale_of(first, lane, 0), MODE == UP ? scale_of(first, lane, 1) : 0.f};
        const int col_step = MODE == GEMM ? kChunk : col_pitch;
        for (int it = first; it < end; ++it) {
            const int v = it / a.tiles;
            float ws_lane[2] = {next_ws[0], next_ws[1]};
            next_ws[0] = scale_of(it + 1, lane, 0);
            if (MODE == UP)
                next_ws[1] = scale_of(it + 1, lane, 1);
            if constexpr (MODE != GEMM) {
                if (v != cur_v) {
                    cur_v = v;
                    consumers_sync();  // the columns are no longer read
                    const Lists& l = sh.lists[0];
                    n_tok = l.v_count[v];
                    const uint16_t* pairs = l.list + l.v_first[v];
                    const int64_t ld = MODE == UP ? a.ldx : a.K;
                    const bool wide = (reinterpret_cast<uintptr_t>(a.xb) & 7u) == 0 && ld % 4 == 0;
                    constexpr int U = 4;
                    const int work = n_tok * a.blocks;
                    for (int i0 = warp; i0 < work; i0 += U * kWarps) {
                        float val[U][4];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int i = i0 + u * kWarps, t = i / a.blocks, k = (i - t * a.blocks) * 128 + lane * 4;
                            val[u][0] = val[u][1] = val[u][2] = val[u][3] = 0.f;
                            if (i < work && k < a.K) {
                                const int pair = pairs[t];
                                const uint16_t* p = a.xb + (int64_t)(MODE == UP ? pair / a.topk : pair) * ld + k;
                                if (wide) {
                                    const uint2 w = *reinterpret_cast<const uint2*>(p);
                                    val[u][0] = __uint_as_float(w.x << 16);
                                    val[u][1] = __uint_as_float(w.x & 0xffff0000u);
                                    val[u][2] = __uint_as_float(w.y << 16);
                                    val[u][3] = __uint_as_float(w.y & 0xffff0000u);
                                } else {
#pragma unroll
                                    for (int j = 0; j < 4; ++j)
                                        val[u][j] = bf16_bits_f(p[j]);
                                }
                            }
                        }
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int i = i0 + u * kWarps;
                            if (i < work) {
                                const int t = i / a.blocks, b = i - t * a.blocks;
                                uint8_t* col = cols + (size_t)(2 * t) * col_pitch + b * 128 + lane * 4;
                                split_block(val[u], col, col + col_pitch, &xs[b * TOK + t]);
                            }
                        }
                    }
                    consumers_sync();
                }
            }
            const int n_nt = MODE == GEMM ? NT : (n_tok + 3) / 4;
            float acc[2][NT][4];
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i)
                acc[i / NT][i % NT][0] = acc[i / NT][i % NT][1] = acc[i / NT][i % NT][2] = acc[i / NT][i % NT][3] = 0.f;
            for (int c = 0; c < n_chunks; ++c, turn ^= 1) {
                if (MODE == GEMM && c > 0 && (c & 31) == 0)
                    ws_lane[0] = scale_of(it, c + lane, 0);
                if (turn != group)
                    continue;
                const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&sh.full[slot]), (uint32_t)use & 1u, abort_flag));
                if (!ok) {
                    if (lane == 0)
                        give_up();
                } else if (c * 4 + kb < a.blocks) {
                    const uint8_t* st = ring + (size_t)slot * a.stage_bytes;
                    uint4 w[2][2][2];  // [row tile][rows g and g + 8][half]
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[i >> 2][(i >> 1) & 1][i & 1] =
                            *reinterpret_cast<const uint4*>(st + (g + (i >> 1) * 8) * kChunk + at[i & 1]);
                    const float ws0 = __shfl_sync(0xffffffffu, ws_lane[0], c & 31);
                    const float ws1 = MODE == UP ? __shfl_sync(0xffffffffu, ws_lane[1], c & 31) : ws0;
                    const float* px = xs + (c * 4 + kb) * TOK;
                    const uint8_t* pb = (MODE == GEMM ? st + kWStage : cols + c * kChunk + kb * 128 + c4 * 16) + g * col_step;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (MODE != GEMM && n >= n_nt)
                            break;
                        float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 x = *reinterpret_cast<const uint4*>(pb + n * 8 * col_step + (MODE == GEMM ? at[h] : 64 * h));
#pragma unroll
                            for (int t = 0; t < 2; ++t)
                                mma_e4m3(d[t], w[t][0][h].x, w[t][1][h].x, w[t][0][h].y, w[t][1][h].y, x.x, x.y);
#pragma unroll
                            for (int t = 0; t < 2; ++t)
                                mma_e4m3(d[t], w[t][0][h].z, w[t][1][h].z, w[t][0][h].w, w[t][1][h].w, x.z, x.w);
                        }
                        if (MODE == GEMM) {
                            const float2 s = *reinterpret_cast<const float2*>(px + n * 8 + 2 * c4);
                            const float s0 = ws0 * s.x, s1 = ws0 * s.y;
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                acc[t][n][0] = fmaf(d[t][0], s0, acc[t][n][0]);
                                acc[t][n][1] = fmaf(d[t][1], s1, acc[t][n][1]);
                                acc[t][n][2] = fmaf(d[t][2], s0, acc[t][n][2]);
                                acc[t][n][3] = fmaf(d[t][3], s1, acc[t][n][3]);
                            }
                        } else {  // columns 2t and 2t + 1 are token t's upper and lower part
                            const float sx = px[n * 4 + c4];
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                const float s = (t ? ws1 : ws0) * sx;
                                acc[t][n][0] = fmaf(fmaf(d[t][1], 0.0625f, d[t][0]), s, acc[t][n][0]);
                                acc[t][n][2] = fmaf(fmaf(d[t][3], 0.0625f, d[t][2]), s, acc[t][n][2]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sh.empty[slot]));
                if ((slot += 2) >= a.stages) {
                    slot = group;
                    ++use;
                }
            }
            if (it - first >= Sh::kBufs)
                pair_sync(kBarFree + buf);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float* red = sh.red[buf][t][warp];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (MODE == GEMM) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            red[(n * 8 + 2 * c4 + (j & 1)) * 20 + g + (j >> 1) * 8] = acc[t][n][j];
                    } else if (n < n_nt) {
                        red[(n * 4 + c4) * 20 + g] = acc[t][n][0];
                        red[(n * 4 + c4) * 20 + g + 8] = acc[t][n][2];
                    }
                }
            }
            pair_arrive(kBarFull + buf);
            buf ^= Sh::kBufs - 1;
        }
    } else {
        if (MODE == DOWN)
            pdl_wait();
        const int tid = (int)threadIdx.x - (kWarps + 1) * 32;
        if (MODE == UP && blockIdx.x == 0)
            for (int i = tid; i < a.done_count; i += kEndWarps * 32)
                a.done[i] = 0;
        int buf = 0;
        for (int it = first; it < end; ++it) {
            const int v = it / a.tiles, tile = it - v * a.tiles;
            const int n_tok = MODE == GEMM ? a.m : sh.lists[0].v_count[v];
            pair_sync(kBarFull + buf);
            auto total_of = [&](int tile16, int t, int r) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    v += sh.red[buf][tile16][w][t * 20 + r];
                return v;
            };
            if constexpr (MODE == GEMM) {
                for (int o = tid; o < a.m * kRows; o += kEndWarps * 32) {
                    const int t = o >> 5, r = o & 31, n = tile * kRows + r;
                    if (n < a.rows) {
                        const float yv = total_of(r >> 4, t, r & 15);
                        if (a.y_bf16)
                            static_cast<uint16_t*>(a.y)[t * a.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(yv));
                        else
                            static_cast<float*>(a.y)[t * a.ldy + n] = yv;
                    }
                }
            } else if constexpr (MODE == UP) {
                const Lists& l = sh.lists[0];
                for (int o = tid; o < n_tok * 16; o += kEndWarps * 32) {
                    const int t = o >> 4, r = o & 15, row = tile * 16 + r;
                    if (row < a.rows) {
                        const float gate = total_of(0, t, r), up = total_of(1, t, r);
                        const float hv = __fdiv_rn(gate, 1.0f + expf(-gate)) * up;
                        a.h[(int64_t)l.list[l.v_first[v] + t] * a.rows + row] = __bfloat16_as_ushort(__float2bfloat16_rn(hv));
                    }
                }
            } else {
                const Lists& l = sh.lists[0];
                for (int o = tid; o < n_tok * kRows; o += kEndWarps * 32) {
                    const int t = o >> 5, r = o & 31, row = tile * kRows + r;
                    if (row < a.rows)
                        a.part[(int64_t)l.list[l.v_first[v] + t] * a.rows + row] = total_of(r >> 4, t, r & 15);
                }
                // The pass that finishes a tile last adds up its tokens' choices, in their order.
                __threadfence();
                enders_sync();
                if (tid == 0)
                    sh.last = atomicAdd(&a.done[tile], 1) == passes - 1;
                enders_sync();
                if (sh.last) {
                    __threadfence();
                    for (int o = tid; o < a.m * kRows; o += kEndWarps * 32) {
                        const int t = o >> 5, row = tile * kRows + (o & 31);
                        if (row >= a.rows)
                            continue;
                        float yv = 0.f;
                        for (int j = 0; j < a.topk; ++j) {
                            const int p = t * a.topk + j, e = l.ids[p];
                            if (e >= 0 && e < a.E)
                                yv = fmaf(a.route_w[p], __ldcg(a.part + (int64_t)p * a.rows + row), yv);
                        }
                        if (a.y_bf16)
                            static_cast<uint16_t*>(a.y)[t * a.ldy + row] = __bfloat16_as_ushort(__float2bfloat16_rn(yv));
                        else
                            static_cast<float*>(a.y)[t * a.ldy + row] = yv;
                    }
                }
            }
            if (it + Sh::kBufs < end)
                pair_arrive(kBarFree + buf);
            buf ^= Sh::kBufs - 1;
        }
        if (MODE == DOWN && passes == 0)  // no token has an expert
            for (int64_t o = (int64_t)blockIdx.x * kEndWarps * 32 + tid; o < (int64_t)a.m * a.rows;
                 o += (int64_t)gridDim.x * kEndWarps * 32) {
                const int64_t at = o / a.rows * a.ldy + o % a.rows;
                if (a.y_bf16)
                    static_cast<uint16_t*>(a.y)[at] = 0;
                else
                    static_cast<float*>(a.y)[at] = 0.f;
            }
    }
    __syncthreads();
    if (sh.abort_flag && threadIdx.x == 0)  // let the copies that were issued land before the CTA exits
        for (int i = max(0, sh.issued - a.stages); i < sh.issued; ++i)
            mbar_wait_bounded(smem_u32(&sh.full[i % a.stages]), (uint32_t)(i / a.stages) & 1u, nullptr);
}

PFN_cuTensorMapEncodeTiled_v12000 stream_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// [experts, parts, rows, K] codes, rows ld bytes apart.  A box is 512 bytes of K, zeros past the edges: as lines of 128
// bytes where K is cut into such, as words otherwise.
bool encode_rows(CUtensorMap* map, const void* base, bool lines, int64_t K, int64_t rows, int64_t ld, int64_t parts,
                 int64_t experts, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = stream_encoder();
    const cuuint64_t k = (cuuint64_t)K, l = (cuuint64_t)ld, r = (cuuint64_t)rows, p = (cuuint64_t)parts;
    const cuuint64_t dims[5] = {lines ? 128 : k / 4, lines ? k / 128 : 1, r, p, (cuuint64_t)experts};
    const cuuint64_t strides[4] = {lines ? 128 : l, l, l * r, l * r * p};
    const cuuint32_t box[5] = {128, lines ? 4u : 1u, (cuuint32_t)box_rows, (cuuint32_t)parts, 1};
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return enc && enc(map, lines ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT32, 5, const_cast<void*>(base),
                      dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      lines ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int NT>
cudaError_t launch_stream(StreamArgs a, int items, cudaStream_t s)
{
    using Sh = Shared<MODE, NT>;
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess)
        return e;
    static std::atomic<unsigned long long> devs{0};
    if ((e = allow_max_smem(fp8_stream_kernel<MODE, NT>, devs)) != cudaSuccess)
        return e;
    a.blocks = (a.K + 127) / 128;
    a.stage_bytes = kWStage + (MODE == GEMM ? 8 * NT * kChunk : 0);
    a.swizzled = a.K % 128 == 0;
    a.k_step = a.swizzled ? 0 : kChunk / 4;
    a.block_step = a.swizzled ? 4 : 0;
    const int parts = MODE == UP ? 2 : 1;
    CUtensorMap tw{}, tx{};
    if (!encode_rows(&tw, a.W, a.swizzled, a.K, a.rows, a.K, parts, std::max(a.E, 1), kRows / parts) ||
        (MODE == GEMM && !encode_rows(&tx, a.x, a.swizzled, a.K, a.m, a.ldx, 1, 1, 8 * NT)))
        return cudaErrorInvalidValue;
    const size_t fixed = 1024 + (sizeof(Sh) + 127) / 128 * 128 + (size_t)(a.blocks * Sh::kTok * 4 + 127) / 128 * 128 +
                         (MODE == GEMM ? 0 : (size_t)(8 * NT) * (a.blocks * 128 + 64));
    if (fixed + 2 * (size_t)a.stage_bytes > (size_t)di.smem_optin)
        return cudaErrorInvalidConfiguration;
    a.stages = (int)std::min<size_t>(16, ((size_t)di.smem_optin - fixed) / a.stage_bytes) & ~1;
    return launch_pdl(fp8_stream_kernel<MODE, NT>, dim3((unsigned)std::min(items, di.sm_count)), dim3(kThreads),
                      fixed + (size_t)a.stages * a.stage_bytes, s, a, tw, tx);
}

size_t part_bytes(size_t n) { return (n + 255) / 256 * 256; }

// Columns of 8 that a pass of the experts has: 4 tokens each.
int moe_columns(int64_t m, int64_t K)
{
    // 4 tiles of 8 columns where they leave room for a ring, fewer for few tokens or long rows
    const int fit = K <= 2048 ? 4 : K <= 6144 ? 2 : 1;
    const int want = m <= 4 ? 1 : m <= 8 ? 2 : 4;
    return std::min(fit, want);
}

template <int MODE>
cudaError_t launch_moe(const StreamArgs& a, int items, cudaStream_t s)
{
    switch (moe_columns(a.m, a.K)) {
    case 1: return launch_stream<MODE, 1>(a, items, s);
    case 2: return launch_stream<MODE, 2>(a, items, s);
    default: return launch_stream<MODE, 4>(a, items, s);
    }
}

}  // namespace

bool fp8_encoder_there() { return stream_encoder() != nullptr; }

bool fp8_stream_supported(const Fp8Gemm& p)
{
    // the scales of x lie in shared memory, 32 KB at most
    return p.m <= 32 && (p.K + 127) / 128 * ((p.m + 7) / 8 * 8) <= 8192 && p.N <= (1 << 30);
}

cudaError_t launch_fp8_gemm_stream(const Fp8Gemm& p, cudaStream_t s)
{
    StreamArgs a{};
    a.W = p.W;
    a.w_scales = p.w_scales;
    a.K = (int)p.K;
    a.rows = (int)p.N;
    a.tiles = (a.rows + kRows - 1) / kRows;
    a.m = (int)p.m;
    a.x = p.x;
    a.x_scales = p.x_scales;
    a.ldx = p.ldx;
    a.ld_xs = p.ld_xs;
    a.y = p.y;
    a.ldy = p.ldy;
    a.y_bf16 = p.y_bf16;
    if (a.m <= 8)
        return launch_stream<GEMM, 1>(a, a.tiles, s);
    return a.m <= 16 ? launch_stream<GEMM, 2>(a, a.tiles, s) : launch_stream<GEMM, 4>(a, a.tiles, s);
}

size_t fp8_moe_workspace(int64_t m, int64_t topk, int64_t dim, int64_t inter)
{
    const size_t pairs = (size_t)(m * topk);
    return part_bytes(pairs * inter * 2) + part_bytes(pairs * dim * 4) + part_bytes((size_t)(dim + kRows - 1) / kRows * 4);
}

cudaError_t launch_fp8_moe(const Fp8Moe& p, cudaStream_t s)
{
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess)
        return e;
    const size_t pairs = (size_t)(p.m * p.topk);
    uint8_t* ws = static_cast<uint8_t*>(p.workspace);
    StreamArgs a{};
    a.m = (int)p.m;
    a.ids = p.ids;
    a.route_w = p.route_w;
    a.topk = p.topk;
    a.E = p.E;
    a.h = reinterpret_cast<uint16_t*>(ws);
    a.part = reinterpret_cast<float*>(ws + part_bytes(pairs * p.inter * 2));
    a.done = reinterpret_cast<int*>(ws + part_bytes(pairs * p.inter * 2) + part_bytes(pairs * p.dim * 4));
    a.done_count = (int)((p.dim + kRows - 1) / kRows);
    a.y = p.y;
    a.ldy = p.ldy;
    a.y_bf16 = p.y_bf16;

    StreamArgs up = a;
    up.W = p.gate_up;
    up.w_scales = p.gate_up_scales;
    up.K = (int)p.dim;
    up.rows = (int)p.inter;
    up.row_blocks = (up.rows + 127) / 128;
    up.tiles = (up.rows + 15) / 16;
    up.xb = p.x;
    up.ldx = p.ldx;
    // passes are known on the device alone: a CTA on every SM
    if ((e = launch_moe<UP>(up, di.sm_count, s)) != cudaSuccess)
        return e;

    StreamArgs down = a;
    down.W = p.down;
    down.w_scales = p.down_scales;
    down.K = (int)p.inter;
    down.rows = (int)p.dim;
    down.row_blocks = (down.rows + 127) / 128;
    down.tiles = a.done_count;
    down.xb = a.h;
    return launch_moe<DOWN>(down, di.sm_count, s);
}

cudaError_t fp8_stream_error_word(int32_t* out, bool clear)
{
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp8_stream_error, sizeof(int));
    if (e != cudaSuccess)
        return e;
    *out = v;
    if (clear) {
        int z = 0;
        e = cudaMemcpyToSymbol(g_fp8_stream_error, &z, sizeof(int));
    }
    return e;
}

}  // namespace q2k
