// Products of few tokens over 8-bit floating-point weights (include/q2k.h):
// fp8_gemm for up to 32 rows, and fp8_moe, the routed experts of a few tokens.
//
// Bound by memory: each weight is read once and used for a handful of tokens.
// So the weights' way is short: three warps copy tiles of 2 x 128 values of K by
// up to 128 rows into a ring of shared-memory stages (tensor copies, 128-byte
// swizzled; a warp takes 390 cycles from one stage's copy to the next's, so
// one alone was the bound), another issues tcgen05.mma kind::f8f6f4 on them as
// they are, weight rows as M = 128, tokens as N = 16 to 64 columns.  The scales
// change every 128 values of K, so each block of a stage has an accumulator of
// its own in tensor memory, and four warps read them back, scale them and add
// them up in fp32, a thread a row; that frees the stage.  (mma.sync, eight warps at the same
// ring: it is made of conversions to f16 and f16 MMAs here, and was bound by
// its instructions' latency: 16 rows of 16384 x 16384 52 to 59 us, experts of
// 8 tokens 278 us.  A bulk copy a row, 512 bytes, was bound by their issue, 73
// cycles each.)
//
// A persistent CTA an SM.  Rows are shared out evenly: a tile has as many
// rows, up to 128, as make the tiles a whole number for each SM, or for each
// cluster of 2 or 4 that then share a tile along K and join through distributed
// shared memory (an MMA takes its 39 cycles whatever rows the tile has, so
// tiles are kept large).  fp8_moe's first launch (gate and up) gives each CTA an equal
// run of units of 16 + 16 rows, expert after expert, up to four units a tile;
// its second (down) gives each cluster its rows of y, of every expert in
// turn, so that the sum over a token's experts stays with the cluster.  (Joined
// by whoever finished a tile last, the fences alone took 10000 cycles an item.)
//
// Tokens of fp8_moe enter as columns of e5m2: with a power of two that brings
// a block's largest below 2^16, a bf16 value is an fp16 number, whose upper
// byte is an e5m2 one; what is left, times 8, is the next, and once more.
// Together the three are the bf16 value exactly, where it is within 2^-30 of
// the block's largest (and off by less than 2^-37 of that below).  (Two columns
// of e4m3 are exact within 2^-13 alone; with two more for the blocks that need
// them, as many of h's do, 32 tokens of 8 experts took 117 us where these take
// 61.)  h, which is fp32 between the launches, enters as four: rounded to fp16
// beside the power of two, that number exactly.  (In bf16 and three, as x, its
// rounding was off as far as that of y to bf16 is, and the experts of one token
// took 40.6 us where they take 40.0.)  Four warps write the columns into the
// stages, every fourth token each, the next stage's values on their way.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "fp8_common.cuh"
#include "q2k_internal.h"

namespace q2k {

__device__ int g_fp8_stream_error = 0;

namespace {

constexpr int kRowsMax = 128;  // weight rows of a tile: the MMA's M
constexpr int kBlock = 128;    // values of K that share a scale: a swizzle row
constexpr int kPair = 2;       // such blocks in a stage
constexpr int kUnit = 16;      // UP: rows of gate, and of up, in a unit
constexpr int kMaxStages = 16;
constexpr int kCopyWarps = 3, kSplitWarps = 4;
constexpr int kMaxPairs = 1024, kMaxExperts = 1024;

enum Mode : int { GEMM = 0, UP = 1, DOWN = 2 };

// Warps: one for the MMAs, three for copies, four that add up (tensor memory lanes by warp % 4), four for columns.
constexpr int threads_of(int mode) { return mode == GEMM ? 256 : 384; }

// Columns that a token enters as; tokens of a pass, and rows of them in a block of a stage.
constexpr int planes_of(int mode) { return mode == GEMM ? 1 : mode == UP ? 3 : 4; }
constexpr int tokens_of(int mode, int columns) { return mode == GEMM ? columns : columns / planes_of(mode) / 8 * 8; }
constexpr int x_rows_of(int mode, int columns) { return planes_of(mode) * tokens_of(mode, columns); }

// Columns of tensor memory that an accumulator is given, and stages that have theirs in its 512.
constexpr int acc_columns(int columns) { return columns <= 32 ? columns : 64; }
constexpr int stages_of(int columns) { return 512 / (kPair * acc_columns(columns)); }

struct StreamArgs {
    const float* w_scales;
    int K, blocks, pairs;     // blocks of 128 along K, and pairs of them
    int rows;                 // weight rows: N; inter (UP); dim (DOWN)
    int row_blocks;           // of w_scales
    int tile_rows, tiles;     // rows of a tile (UP: of a unit), tiles of one matrix
    int box_bytes;            // of one copy of weights
    int stages, w_bytes;      // of weights in a block of a stage
    int m;
    // GEMM
    const float* x_scales;
    int64_t ld_xs;
    // fp8_moe
    const uint16_t* xb;       // UP: tokens, bf16 rows
    int64_t ldx;
    const int32_t* ids;
    const float* route_w;
    int topk, E;
    float* h;                 // [pairs, inter]
    // results
    void* y;
    int64_t ldy;
    int y_bf16;
};

// 16 fp32 columns of this warp's 32 lanes; complete after settle().
__device__ __forceinline__ void tmem_load16(uint32_t taddr, float* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}

// 8 of them.
__device__ __forceinline__ void tmem_load8(uint32_t taddr, float* v)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr));
}

// Two floats as fp16.
__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// What is left of two fp16 numbers without their upper bytes, times 8: exact.
__device__ __forceinline__ uint32_t left8(uint32_t h)
{
    uint32_t r;
    asm("{\n\t.reg .b32 u;\n\tand.b32 u, %1, 0xff00ff00;\n\tsub.rn.f16x2 u, %1, u;\n\tmul.rn.f16x2 %0, u, %2;\n\t}"
        : "=r"(r)
        : "r"(h), "r"(0x48004800u));
    return r;
}

// A box of 128 bytes by rows, by gate and up, by expert.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int k, int row, int expert, uint32_t bar,
                                         uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(row), "r"(0), "r"(expert), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void store_peer(uint32_t addr, uint32_t rank, float v)
{
    asm volatile("{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %0, %1;\n\tst.shared::cluster.f32 [p], %2;\n\t}" ::"r"(addr),
                 "r"(rank), "f"(v)
                 : "memory");
}

__device__ __forceinline__ float load_peer(uint32_t addr, uint32_t rank)
{
    float v;
    asm volatile("{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %1, %2;\n\tld.shared::cluster.f32 %0, [p];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

// The experts that have a token, as passes of up to CAP (token, choice) pairs.
struct Lists {
    uint16_t list[kMaxPairs];                                              // pairs by expert, in order
    uint16_t v_expert[kMaxPairs], v_first[kMaxPairs], v_count[kMaxPairs];  // passes
    uint16_t token[kMaxPairs];  // of list's entries, and their weights
    float weight[kMaxPairs];
    int passes;

    __device__ __forceinline__ void put(const StreamArgs& a, int place, int pair)
    {
        list[place] = (uint16_t)pair;
        token[place] = (uint16_t)(pair / a.topk);
        weight[place] = a.route_w[pair];
    }
};

// What they are made with, where the first stage's columns are written later.
struct ListScratch {
    alignas(16) int ids[kMaxPairs];
    alignas(16) uint16_t count[kMaxExperts];
    uint16_t rank[kMaxPairs];
};

constexpr int kFewPairs = 256;

// The lists of up to 256 pairs: a pair's place is the number of pairs before it, by expert and then by pair, which each
// thread counts for itself; likewise a pass's.  (2.2 us with the other way, for 8 pairs of 256 experts.)
template <int kThreads>
__device__ __forceinline__ void build_few_lists(Lists& l, ListScratch& s, const StreamArgs& a, int cap)
{
    static_assert(kThreads >= kFewPairs, "a thread a pair");
    constexpr int kNone = 0x7fffffff;
    int* const starts = reinterpret_cast<int*>(s.count);  // the expert where a pair starts a pass
    const int pairs = a.m * a.topk, i = threadIdx.x, whole = (pairs + 3) & ~3;
    int e = kNone;
    if (i < whole) {
        if (i < pairs)
            e = a.ids[i];
        e = e >= 0 && e < a.E ? e : kNone;
        s.ids[i] = e;
    }
    __syncthreads();
    int place = 0, before = 0, same = 0;
    if (i < whole) {
        for (int j = 0; j < whole; j += 4) {
            const int4 v = *reinterpret_cast<const int4*>(s.ids + j);
            const int o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool eq = o[u] == e, first = eq && j + u < i;
                place += o[u] < e || first;
                before += first;
                same += eq;
            }
        }
        starts[i] = e != kNone && before % cap == 0 ? e : kNone;
        if (e != kNone)
            l.put(a, place, i);
    }
    const bool start = i < whole && e != kNone && before % cap == 0;
    const int passes = __syncthreads_count(start);
    if (start) {
        int v = 0;
        for (int j = 0; j < whole; j += 4) {
            const int4 w = *reinterpret_cast<const int4*>(starts + j);
            const int o[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int u = 0; u < 4; ++u)
                v += o[u] < e || (o[u] == e && j + u < i);
        }
        l.v_expert[v] = (uint16_t)e;
        l.v_first[v] = (uint16_t)place;
        l.v_count[v] = (uint16_t)min(cap, same - before);
    }
    if (i == 0)
        l.passes = passes;
    __syncthreads();
}

// By all threads; ends with a barrier.
template <int kThreads>
__device__ void build_lists(Lists& l, ListScratch& s, const StreamArgs& a, int cap)
{
    const int pairs = a.m * a.topk, tid = threadIdx.x;
    if (pairs <= kFewPairs)
        return build_few_lists<kThreads>(l, s, a, cap);
    for (int i = tid; i < a.E; i += kThreads)
        s.count[i] = 0;
    for (int i = tid; i < pairs; i += kThreads)
        s.ids[i] = a.ids[i];
    __syncthreads();
    if (tid < 32) {
        // a pair's place among those of its expert, 32 pairs at a time
        for (int i0 = 0; i0 < pairs; i0 += 32) {
            const int i = i0 + tid;
            const int e = i < pairs ? s.ids[i] : -1;
            const bool valid = e >= 0 && e < a.E;
            const uint32_t same = __match_any_sync(0xffffffffu, valid ? e : -1);
            const int before = valid ? s.count[e] : 0;
            __syncwarp();
            if (valid) {
                s.rank[i] = (uint16_t)(before + __popc(same & ((1u << tid) - 1u)));
                if ((same >> tid) == 1u)  // the last of them
                    s.count[e] = (uint16_t)(before + __popc(same));
            }
            __syncwarp();
        }
        // each lane a run of experts: first pair and first pass of each
        const int run = (a.E + 31) / 32, e0 = tid * run, e1 = min(a.E, e0 + run);
        int n = 0, v = 0;
        for (int e = e0; e < e1; ++e) {
            n += s.count[e];
            v += (s.count[e] + cap - 1) / cap;
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
            const int c = s.count[e];
            s.count[e] = (uint16_t)n_at;  // from here on the expert's first place
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
        const int e = s.ids[i];
        if (e >= 0 && e < a.E)
            l.put(a, s.count[e] + s.rank[i], i);
    }
    __syncthreads();
}

// A lane's four values of a block: bf16 of a token, fp32 of h.
template <int MODE>
using Raw = std::conditional_t<MODE == DOWN, uint4, uint2>;

// N blocks of 128 values, 4 a lane, each as e5m2 rows (128-byte swizzled: t[n] of the block's first TOK rows, of those after
// them, ...), and its scale.  All at once: each is a chain of its own.  A NaN or an infinity leaves NaN.
template <int MODE, int N, int TOK>
__device__ __forceinline__ void split_blocks(const Raw<MODE> (&raw)[N], uint8_t* const (&tile)[N], const int (&t)[N], float* const (&scale)[N])
{
    const int lane = threadIdx.x & 31;
    // The exponent that the block's largest has at most: h's rounding to fp16 may carry into the next.
    constexpr uint32_t kTop = MODE == DOWN ? 14 : 15;
    uint32_t top[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        // the largest magnitude, as a whole number
        if constexpr (MODE == DOWN) {
            top[n] = max(max(raw[n].x & 0x7fffffffu, raw[n].y & 0x7fffffffu), max(raw[n].z & 0x7fffffffu, raw[n].w & 0x7fffffffu));
        } else {
            const uint32_t a = raw[n].x & 0x7fff7fffu, b = raw[n].y & 0x7fff7fffu;
            top[n] = max(max(a & 0xffffu, a >> 16), max(b & 0xffffu, b >> 16)) << 16;
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
        top[n] = __reduce_max_sync(0xffffffffu, top[n]);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        // 2^(kTop - e) of the largest's exponent e, within fp32's powers of two for it and its inverse
        const uint32_t e = min(max(top[n] >> 23, 20u), 254u);
        const float f = __uint_as_float((254u + kTop - e) << 23);
        uint32_t h0, h1;
        if constexpr (MODE == DOWN) {
            h0 = f16x2(__uint_as_float(raw[n].x) * f, __uint_as_float(raw[n].y) * f);
            h1 = f16x2(__uint_as_float(raw[n].z) * f, __uint_as_float(raw[n].w) * f);
        } else {
            h0 = f16x2(__uint_as_float(raw[n].x << 16) * f, __uint_as_float(raw[n].x & 0xffff0000u) * f);
            h1 = f16x2(__uint_as_float(raw[n].y << 16) * f, __uint_as_float(raw[n].y & 0xffff0000u) * f);
        }
        uint8_t* const at = tile[n] + t[n] * kBlock + (((lane >> 2) ^ (t[n] & 7)) << 4) + ((lane & 3) << 2);
#pragma unroll
        for (int p = 0; p < planes_of(MODE); ++p) {
            *reinterpret_cast<uint32_t*>(at + p * TOK * kBlock) = __byte_perm(h0, h1, 0x7531);  // the upper bytes
            if (p + 1 < planes_of(MODE)) {
                h0 = left8(h0);
                h1 = left8(h1);
            }
        }
        if (lane == 0)
            *scale[n] = __uint_as_float((e - kTop) << 23);
    }
}

template <int MODE, int NC>
struct Shared {
    uint64_t full[kMaxStages], done[kMaxStages], freed[kMaxStages];  // of a stage: copied; multiplied; added up
    uint32_t tmem;
    int abort_flag;
    alignas(16) float scales[MODE == GEMM ? 1 : kMaxStages][kPair][tokens_of(MODE, NC)];  // of a stage's columns; read four at a time
    Lists lists[MODE == GEMM ? 0 : 1];
};

// What a CTA works on: pieces of a tile and a run of blocks along K, one after another.
template <int MODE, int S>
struct Walk {
    int tiles, pairs, passes, rank;
    int at, end, tile_at;                 // UP: units; else pairs of blocks of all passes
    int pass, tile, units, k, k_end;      // the piece, k in pairs of blocks
    bool last;                            // of its tile

    __device__ __forceinline__ Walk(const StreamArgs& a, int n_passes) : tiles(a.tiles), pairs(a.pairs), passes(n_passes)
    {
        rank = S > 1 ? (int)blockIdx.x % S : 0;
        tile_at = (int)blockIdx.x / S;
        if (MODE == UP) {
            const int64_t total = (int64_t)passes * tiles;
            at = (int)(blockIdx.x * total / gridDim.x);
            end = (int)((blockIdx.x + 1) * total / gridDim.x);
        } else {
            range();
        }
        pass = tile = k = k_end = 0;
        units = 1;
        last = true;
    }
    __device__ __forceinline__ void range()
    {
        const int total = passes * pairs;  // at most 1024 * 64
        at = rank * total / S;
        end = (rank + 1) * total / S;
    }
    __device__ __forceinline__ bool next()
    {
        if (MODE == UP) {
            if (at >= end)
                return false;
            pass = at / tiles;
            tile = at - pass * tiles;
            units = min(min(4, tiles - tile), end - at);
            at += units;
            k = 0;
            k_end = pairs;
            return true;
        }
        if (tile_at >= tiles || at >= end)
            return false;
        tile = tile_at;
        pass = MODE == GEMM ? 0 : at / pairs;
        k = at - pass * pairs;
        k_end = min(pairs, k + end - at);
        at += k_end - k;
        last = at >= end;
        if (last) {  // the next tile, if there is one
            tile_at += (int)gridDim.x / S;
            range();
        }
        return true;
    }
};

template <int MODE, int NC, int S>
__global__ void __launch_bounds__(threads_of(MODE), 1)
    fp8_stream_kernel(const StreamArgs a, const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx)
{
    using Sh = Shared<MODE, NC>;
    constexpr int kThreads = threads_of(MODE);
    constexpr int TOK = tokens_of(MODE, NC), kPlane = planes_of(MODE);
    constexpr uint32_t kXBytes = x_rows_of(MODE, NC) * kBlock;  // of tokens in a block of a stage
    constexpr int kAcc = acc_columns(NC);
    constexpr uint32_t kTmem = 512;
    extern __shared__ __align__(1024) uint8_t smem[];
    // The 128-byte swizzle repeats every 1024 bytes: stages start on 1024.  (An MMA reads 128 rows of weights whatever
    // the tile has, and NC of tokens: past them, and past the rings' ends, lie other bytes of this CTA, whose sums
    // nothing uses.)
    uint8_t* const ring = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u);
    uint8_t* const x_ring = ring + (size_t)a.stages * kPair * a.w_bytes;
    Sh& sh = *reinterpret_cast<Sh*>(x_ring + (size_t)a.stages * kPair * kXBytes);
    // [m][128] sums of a tile (DOWN), or the cluster's of the tokens that are this CTA's (GEMM): [S][m / S][128]
    float* const y_sum = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(&sh) + (sizeof(Sh) + 127) / 128 * 128);
    float* const xs = y_sum + (S > 1 ? (a.m + S - 1) * kRowsMax : 0);  // GEMM: [2 pairs][NC]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // (a lane a stage: one thread for all takes 0.1 us more, of 5.5 for a row of 4096 x 4096)
    if (threadIdx.x < a.stages) {
        mbar_init(smem_u32(&sh.full[threadIdx.x]), MODE == GEMM ? 1 : 1 + kSplitWarps);
        mbar_init(smem_u32(&sh.done[threadIdx.x]), 1);
        mbar_init(smem_u32(&sh.freed[threadIdx.x]), 4);
        fence_mbar_init();
    }
    if (threadIdx.x == 96)
        sh.abort_flag = 0;
    if (threadIdx.x == 32) {
        prefetch_map(&tw);
        if (MODE == GEMM)
            prefetch_map(&tx);
    }
    __syncwarp();
    if (S > 1)
        cluster_arrive();  // this CTA has started
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // UP lets DOWN start only once what came before is complete: DOWN reads ids
    // and weights before it waits for UP.
    if (MODE != DOWN)
        pdl_wait();
    pdl_launch_dependents();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    int passes = 1;
    if constexpr (MODE != GEMM) {
        build_lists<kThreads>(sh.lists[0], *reinterpret_cast<ListScratch*>(x_ring), a, TOK);
        passes = sh.lists[0].passes;
    } else {
        __syncthreads();
    }
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = sh.tmem;
    const Lists& l = sh.lists[0];

    volatile int* const abort_flag = &sh.abort_flag;
    auto give_up = [&]() {
        atomicOr(&g_fp8_stream_error, Q2K_ERR_BIT_WAIT_TIMEOUT);
        *abort_flag = 1;
    };
    // by a whole warp
    auto wait = [&](uint64_t* bar, int use) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait_near(smem_u32(bar), (uint32_t)use & 1u, abort_flag));
        if (!ok && lane == 0)
            give_up();
        return ok;
    };
    auto store = [&](int64_t t, int row, float v) {
        if (a.y_bf16)
            static_cast<uint16_t*>(a.y)[t * a.ldy + row] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        else
            static_cast<float*>(a.y)[t * a.ldy + row] = v;
    };
    Walk<MODE, S> work(a, passes);
    const int q = warp & 3;  // of the warps that add up: their lanes, 32 rows
    const int rank = S > 1 ? (int)blockIdx.x % S : 0, share = (a.m + S - 1) / S;

    if (warp == 0) {
        // ---- MMAs
        constexpr uint32_t idesc = instr_desc_e4m3(NC) | (MODE == GEMM ? 0u : kBIsE5m2);
        const uint32_t w_bytes = (uint32_t)a.w_bytes, ring_at = smem_u32(ring), x_at = smem_u32(x_ring);
        int slot = 0, use = 0;
        bool ok = true, ready = false;
        while (ok && work.next())
            for (int k = work.k; k < work.k_end; ++k) {
                if (!ready && !wait(&sh.full[slot], use)) {
                    ok = false;
                    break;
                }
                const int slot1 = slot + 1 == a.stages ? 0 : slot + 1, use1 = use + (slot1 == 0);
                const bool full1 = mbar_ready(smem_u32(&sh.full[slot1]), (uint32_t)use1 & 1u);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t s0 = uniform((uint32_t)slot);
                const uint32_t sa = ring_at + s0 * kPair * w_bytes, sb = x_at + s0 * kPair * kXBytes, d = tmem + s0 * kPair * kAcc;
                if (elect_one()) {
#pragma unroll
                    for (int p = 0; p < kPair; ++p)
#pragma unroll
                        for (int i = 0; i < kBlock / 32; ++i)  // K = 32 an MMA: 32 bytes along the swizzled row
                            umma_e4m3(d + p * kAcc, desc_at(sa + p * w_bytes + 32 * i), desc_at(sb + p * kXBytes + 32 * i), idesc, i > 0);
                    umma_commit(smem_u32(&sh.done[0]) + 8 * s0);
                }
                ready = __all_sync(0xffffffffu, full1);
                slot = slot1;
                use = use1;
            }
    } else if (warp <= kCopyWarps) {
        // ---- copies: of every third stage
        if (lane == 0) {
            const uint64_t wpol = l2_policy_evict_first(), xpol = l2_policy_evict_last();
            int slot = 0, use = 0, turn = 0, last_slot = -1, last_use = 0;
            bool ok = true;
            while (ok && work.next()) {
                const int expert = MODE == GEMM ? 0 : l.v_expert[work.pass];
                for (int k = work.k; k < work.k_end; ++k) {
                    if (turn == warp - 1) {
                        if (use > 0 && !mbar_wait_near(smem_u32(&sh.freed[slot]), (uint32_t)(use - 1) & 1u, abort_flag)) {
                            give_up();
                            ok = false;
                            break;
                        }
                        const uint32_t bar = smem_u32(&sh.full[slot]);
                        uint32_t dst = smem_u32(ring + (size_t)slot * kPair * a.w_bytes);
                        mbar_arrive_expect_tx(bar, kPair * ((uint32_t)(work.units * a.box_bytes) + (MODE == GEMM ? kXBytes : 0u)));
#pragma unroll
                        for (int p = 0; p < kPair; ++p, dst += (uint32_t)a.w_bytes) {
                            const int at = (k * kPair + p) * kBlock;
                            for (int u = 0; u < work.units; ++u)
                                copy_box(dst + u * a.box_bytes, &tw, at, (work.tile + u) * a.tile_rows, expert, bar, wpol);
                            if (MODE == GEMM)
                                copy_box(smem_u32(x_ring + (slot * kPair + p) * kXBytes), &tx, at, 0, 0, bar, xpol);
                        }
                        last_slot = slot;
                        last_use = use;
                    }
                    if (++turn == kCopyWarps)
                        turn = 0;
                    if (++slot == a.stages) {
                        slot = 0;
                        ++use;
                    }
                }
            }
            if (last_slot >= 0 && *abort_flag) {  // let the copies that were issued land before the CTA exits
                const volatile int never = 0;
                mbar_wait_near(smem_u32(&sh.full[last_slot]), (uint32_t)last_use & 1u, &never);
            }
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ---- sums
        if (MODE == DOWN)
            pdl_wait();
        const uint32_t t_addr = tmem + ((uint32_t)(32 * q) << 16);
        const bool mine = 32 * q < a.tile_rows || MODE == UP;  // has rows
        if (MODE == DOWN)
            for (int t = 0; t < a.m; ++t)
                y_sum[t * kRowsMax + 32 * q + lane] = 0.f;
        if constexpr (MODE == GEMM) {
            for (int i = (int)threadIdx.x - 128; i < a.pairs * kPair * NC; i += 128) {
                const int b = i / NC, t = i % NC;
                xs[i] = t < a.m && b < a.blocks ? a.x_scales[t * a.ld_xs + b] : 0.f;
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
        }
        int slot = 0, use = 0;
        // The scales of a piece's blocks, 32 at a time, a lane each: of rows before `cut` the first, else the second.
        struct Scales {
            float v[2];
            int cut;
        };
        auto scales_of = [&](const Walk<MODE, S>& w, int k0) {
            Scales s{{0.f, 0.f}, 32};
            int64_t first, second;
            if (MODE == UP) {
                first = (int64_t)l.v_expert[w.pass] * 2 * a.row_blocks + min((w.tile + q) * kUnit / 128, a.row_blocks - 1);
                second = first + a.row_blocks;
                s.cut = kUnit;
            } else {
                const int row = w.tile * a.tile_rows + 32 * q;
                const int64_t e = MODE == DOWN ? (int64_t)l.v_expert[w.pass] * a.row_blocks : 0;
                first = e + min(row / 128, a.row_blocks - 1);
                second = e + min(row / 128 + 1, a.row_blocks - 1);
                s.cut = (row / 128 + 1) * 128 - row;
            }
            if (k0 + lane < min(a.blocks, w.k_end * kPair)) {
                s.v[0] = a.w_scales[first * a.blocks + k0 + lane];
                if (s.cut < 32)
                    s.v[1] = a.w_scales[second * a.blocks + k0 + lane];
            }
            return s;
        };
        // GEMM, S > 1: token t's sums go to CTA t % S, into the place that it has for this CTA's
        bool pushed = false;
        auto push = [&](const float (&v)[TOK]) {
            __syncwarp();
            if (!pushed)
                cluster_wait();  // all have started
            pushed = true;
            const uint32_t at = smem_u32(y_sum + rank * share * kRowsMax + 32 * q + lane);
#pragma unroll
            for (int t = 0; t < TOK; ++t)
                if (t < a.m)
                    store_peer(at + (uint32_t)(t / S) * (kRowsMax * 4), t % S, v[t]);
        };
        bool ready = false;
        bool more = work.next();
        Scales next{{0.f, 0.f}, 32};
        if (more)
            next = scales_of(work, work.k * kPair);
        while (more) {
            const Walk<MODE, S> piece = work;
            Scales ws = next;
            if ((more = work.next()))
                next = scales_of(work, work.k * kPair);  // (a piece ahead)
            const int n_tok = MODE == GEMM ? a.m : l.v_count[piece.pass];
            float acc[TOK];
#pragma unroll
            for (int t = 0; t < TOK; ++t)
                acc[t] = 0.f;
            for (int k = piece.k; k < piece.k_end; ++k) {
                const int j = (k - piece.k) * kPair & 31;
                if (j == 0 && k > piece.k)
                    ws = scales_of(piece, k * kPair);
                float w[kPair];
#pragma unroll
                for (int p = 0; p < kPair; ++p) {
                    const float w0 = __shfl_sync(0xffffffffu, ws.v[0], j + p), w1 = __shfl_sync(0xffffffffu, ws.v[1], j + p);
                    w[p] = lane < ws.cut ? w0 : w1;
                }
                // (what filled the stage has the columns' scales with it)
                if (!ready && !(wait(&sh.done[slot], use) && wait(&sh.full[slot], use)))
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const int slot1 = slot + 1 == a.stages ? 0 : slot + 1, use1 = use + (slot1 == 0);
                // Both blocks at once or, where registers do not suffice (16 tokens of fp8_moe), one after the other.
                constexpr int R = TOK * kPlane, kAtOnce = kPair * R <= 64 ? kPair : 1;
#pragma unroll
                for (int p0 = 0; p0 < kPair; p0 += kAtOnce) {
                    float d[kAtOnce * R], sx[kAtOnce][TOK];
                    if (mine) {
#pragma unroll
                        for (int p = 0; p < kAtOnce; ++p) {
                            const uint32_t from = t_addr + slot * kPair * kAcc + (p0 + p) * kAcc;
#pragma unroll
                            for (int c = 0; c < R; c += 16)
                                if (c + 16 <= R)
                                    tmem_load16(from + c, d + p * R + c);
                                else
                                    tmem_load8(from + c, d + p * R + c);
                        }
#pragma unroll
                        for (int p = 0; p < kAtOnce; ++p) {
                            const float* px = MODE == GEMM ? xs + (k * kPair + p0 + p) * NC : sh.scales[slot][p0 + p];
#pragma unroll
                            for (int t = 0; t < TOK; t += 4) {
                                if (MODE != GEMM && t >= n_tok)
                                    break;
                                const float4 v = *reinterpret_cast<const float4*>(px + t);
                                sx[p][t] = v.x, sx[p][t + 1] = v.y, sx[p][t + 2] = v.z, sx[p][t + 3] = v.w;
                            }
                        }
                    }
                    bool done1 = false, full1 = false;
                    if (p0 + kAtOnce == kPair) {
                        done1 = mbar_ready(smem_u32(&sh.done[slot1]), (uint32_t)use1 & 1u);
                        full1 = mbar_ready(smem_u32(&sh.full[slot1]), (uint32_t)use1 & 1u);
                    }
                    settle(d);
                    if (p0 + kAtOnce == kPair) {
                        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                        ready = __all_sync(0xffffffffu, done1 && full1);
                        if (lane == 0)
                            mbar_arrive(smem_u32(&sh.freed[slot]));
                    }
                    if (mine) {
#pragma unroll
                        for (int p = 0; p < kAtOnce; ++p)
#pragma unroll
                            for (int t = 0; t < TOK; ++t) {
                                if (MODE != GEMM && (t & 3) == 0 && t >= n_tok)
                                    break;
                                const float f = w[p0 + p] * sx[p][t], *v = d + p * R + t;
                                float all = v[(kPlane - 1) * TOK];
#pragma unroll
                                for (int c = kPlane - 2; c >= 0; --c)
                                    all = fmaf(all, 0.125f, v[c * TOK]);
                                acc[t] = fmaf(all, f, acc[t]);
                            }
                    }
                }
                slot = slot1;
                use = use1;
            }
            if constexpr (MODE == GEMM) {
                const int r = 32 * q + lane, row = piece.tile * a.tile_rows + r;
                if (S > 1) {
                    push(acc);
                } else if (r < a.tile_rows && row < a.rows && !*abort_flag) {
#pragma unroll
                    for (int t = 0; t < TOK; ++t)
                        if (t < a.m)
                            store(t, row, acc[t]);
                }
            } else if constexpr (MODE == UP) {
                const int row = (piece.tile + q) * kUnit + (lane & 15);
#pragma unroll
                for (int t = 0; t < TOK; ++t) {
                    if (t >= n_tok)
                        break;
                    const float gate = acc[t], up = __shfl_down_sync(0xffffffffu, acc[t], 16);
                    if (q < piece.units && lane < 16 && row < a.rows) {
                        const float hv = __fdiv_rn(gate, 1.0f + expf(-gate)) * up;
                        a.h[(int64_t)l.list[l.v_first[piece.pass] + t] * a.rows + row] = hv;
                    }
                }
            } else {
                // (a row of y_sum's columns is this thread's alone)
                const int r = 32 * q + lane, row = piece.tile * a.tile_rows + r;
#pragma unroll
                for (int t = 0; t < TOK; ++t) {
                    if (t >= n_tok)
                        break;
                    const int at = l.v_first[piece.pass] + t;
                    float& to = y_sum[l.token[at] * kRowsMax + r];
                    to = fmaf(l.weight[at], acc[t], to);
                }
                if (S == 1 && piece.last)
                    for (int t = 0; t < a.m; ++t) {
                        if (r < a.tile_rows && row < a.rows && !*abort_flag)
                            store(t, row, y_sum[t * kRowsMax + r]);
                        y_sum[t * kRowsMax + r] = 0.f;
                    }
            }
        }
        if (MODE == GEMM && S > 1 && !pushed) {  // fewer pairs of blocks than CTAs
            const float none[TOK] = {};
            push(none);
        }
        if (MODE == DOWN && S == 1 && passes == 0)  // no token has an expert
            for (int tile = (int)blockIdx.x; tile < a.tiles; tile += (int)gridDim.x)
                for (int t = 0; t < a.m; ++t) {
                    const int r = 32 * q + lane, row = tile * a.tile_rows + r;
                    if (r < a.tile_rows && row < a.rows)
                        store(t, row, 0.f);
                }
    } else if constexpr (MODE != GEMM) {
        // ---- columns
        if (MODE == DOWN)
            pdl_wait();
        const int sw = warp - 8;
        const bool wide = (reinterpret_cast<uintptr_t>(a.xb) & 7u) == 0 && a.ldx % 4 == 0;
        using R4 = Raw<MODE>;
        using Value = std::conditional_t<MODE == UP, uint16_t, float>;
        auto load4 = [&](const Value* row, int k) {  // four values from lane * 4 on; zeros past K
            R4 r{};
            if (k + lane * 4 >= a.K)
                return r;
            const Value* const v = row + k;
            if constexpr (MODE == DOWN)  // (rows of h are whole 64 bytes)
                r = *reinterpret_cast<const uint4*>(v);
            else if (wide)
                r = *reinterpret_cast<const uint2*>(v);
            else
                r = make_uint2(v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16);
            return r;
        };
        // Every fourth token of a stage is this warp's; the next stage's values are on their way.
        constexpr int G = TOK / kSplitWarps;
        const Value* row[G] = {};
        R4 ahead[G][kPair];
        int pass = -1, count = 0;
        auto fetch = [&]() {
            if (work.pass != pass) {
                pass = work.pass;
                count = (l.v_count[pass] - sw + kSplitWarps - 1) / kSplitWarps;
#pragma unroll
                for (int g = 0; g < G; ++g)
                    if (g < count) {
                        const int at = l.v_first[pass] + sw + g * kSplitWarps;
                        if constexpr (MODE == UP)
                            row[g] = a.xb + (int64_t)l.token[at] * a.ldx + lane * 4;
                        else
                            row[g] = a.h + (int64_t)l.list[at] * a.K + lane * 4;
                    }
            }
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int p = 0; p < kPair; ++p)
                    ahead[g][p] = g < count ? load4(row[g], (work.k * kPair + p) * kBlock) : R4{};
        };
        bool live = work.next();
        if (live)
            fetch();
        int slot = 0, use = 0;
        while (live) {
            R4 now[G][kPair];
#pragma unroll
            for (int i = 0; i < G * kPair; ++i)
                now[i / kPair][i % kPair] = ahead[i / kPair][i % kPair];
            const int n_now = count;
            live = ++work.k < work.k_end || work.next();
            if (live)
                fetch();
            if (use > 0 && !wait(&sh.freed[slot], use - 1))
                break;
            uint8_t* const tile = x_ring + slot * kPair * kXBytes;
            auto split = [&](auto tokens) {  // of so many tokens
                constexpr int N = decltype(tokens)::value;
                R4 raw[N * kPair];
                uint8_t* tiles[N * kPair];
                int t[N * kPair];
                float* scale[N * kPair];
#pragma unroll
                for (int i = 0; i < N * kPair; ++i) {
                    raw[i] = now[i / kPair][i % kPair];
                    tiles[i] = tile + i % kPair * kXBytes;
                    t[i] = sw + i / kPair * kSplitWarps;
                    scale[i] = &sh.scales[slot][i % kPair][t[i]];
                }
                split_blocks<MODE, N * kPair, TOK>(raw, tiles, t, scale);
            };
            if (n_now == 1)
                split(std::integral_constant<int, 1>{});
            else if (n_now > 1)
                split(std::integral_constant<int, G>{});
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sh.full[slot]));
            if (++slot == a.stages) {
                slot = 0;
                ++use;
            }
        }
    }
    if constexpr (S > 1) {
        const bool adds = warp >= 4 && warp < 8;
        __syncwarp();
        if (MODE != GEMM || !adds)
            cluster_wait();  // (the pushing warps have)
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        const int r = 32 * q + lane, row = (int)blockIdx.x / S * a.tile_rows + r;
        if (adds && r < a.tile_rows && row < a.rows && !*abort_flag)
            for (int t = rank; t < a.m; t += S) {
                float v = 0.f;
#pragma unroll
                for (int c = 0; c < S; ++c)  // in the order of K
                    v += MODE == GEMM ? y_sum[(c * share + t / S) * kRowsMax + r] : load_peer(smem_u32(y_sum + t * kRowsMax + r), c);
                store(t, row, v);
            }
        __syncwarp();
        if (MODE != GEMM) {
            cluster_sync();  // nobody reads this CTA's sums any more
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
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

// [experts, parts, rows, K] codes, rows ld bytes apart.  A box is 128 values of K by box_rows rows by all parts, zeros
// past the edges.
bool encode_rows(CUtensorMap* map, const void* base, int64_t K, int64_t rows, int64_t ld, int64_t parts, int64_t experts,
                 int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = stream_encoder();
    const cuuint64_t l = (cuuint64_t)ld, r = (cuuint64_t)rows, p = (cuuint64_t)parts;
    const cuuint64_t dims[4] = {(cuuint64_t)K, r, p, (cuuint64_t)experts};
    const cuuint64_t strides[3] = {l, l * r, l * r * p};
    const cuuint32_t box[4] = {kBlock, (cuuint32_t)box_rows, (cuuint32_t)parts, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows a tile: as many, up to 128, as give each of `teams` the same number of tiles.
int balanced_rows(int64_t rows, int teams)
{
    const int64_t rounds = (rows + (int64_t)kRowsMax * teams - 1) / ((int64_t)kRowsMax * teams);
    return (int)((rows + rounds * teams - 1) / (rounds * teams));
}

// Clusters of S such CTAs that the device runs at once (the same on every device: the library runs on one kind).
template <int MODE, int NC, int S>
cudaError_t clusters_of(const DeviceInfo& di, int* n)
{
    static std::atomic<int> known{0};
    *n = known.load(std::memory_order_relaxed);
    if (*n > 0)
        return cudaSuccess;
    static std::atomic<unsigned long long> devs{0};
    cudaError_t e = allow_max_smem(fp8_stream_kernel<MODE, NC, S>, devs);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(di.sm_count / S * S));
    cfg.blockDim = dim3(threads_of(MODE));
    cfg.dynamicSmemBytes = (size_t)di.smem_optin;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(n, fp8_stream_kernel<MODE, NC, S>, &cfg);
    if (e != cudaSuccess)
        return e;
    if (*n < 1)
        return cudaErrorInvalidConfiguration;
    known.store(*n, std::memory_order_relaxed);
    return cudaSuccess;
}

template <int MODE, int NC, int S>
cudaError_t launch_stream(StreamArgs a, const void* W, const void* x, const DeviceInfo& di, cudaStream_t s)
{
    using Sh = Shared<MODE, NC>;
    auto* kernel = fp8_stream_kernel<MODE, NC, S>;
    static std::atomic<unsigned long long> devs{0};
    cudaError_t e = allow_max_smem(kernel, devs);
    if (e != cudaSuccess)
        return e;
    a.blocks = (a.K + kBlock - 1) / kBlock;
    a.pairs = (a.blocks + kPair - 1) / kPair;
    a.row_blocks = (a.rows + 127) / 128;
    int teams = di.sm_count / S;
    if (S > 2 && (e = clusters_of<MODE, NC, S>(di, &teams)) != cudaSuccess)
        return e;
    a.tile_rows = MODE == UP ? kUnit : balanced_rows(a.rows, teams);
    a.tiles = (a.rows + a.tile_rows - 1) / a.tile_rows;
    const int parts = MODE == UP ? 2 : 1;
    a.box_bytes = a.tile_rows * parts * kBlock;
    a.w_bytes = MODE == UP ? kRowsMax * kBlock : (a.box_bytes + 1023) / 1024 * 1024;
    const size_t rest = (sizeof(Sh) + 127) / 128 * 128 + (MODE == DOWN || S > 1 ? (size_t)(a.m + S - 1) * kRowsMax * 4 : 0) +
                        (MODE == GEMM ? (size_t)a.pairs * kPair * NC * 4 : 0);
    const size_t past = (size_t)(kRowsMax * kBlock - a.w_bytes);  // what an MMA may read behind the last stage
    constexpr size_t kXBytes = (size_t)x_rows_of(MODE, NC) * kBlock;
    static_assert(sizeof(Sh) >= NC * kBlock - kXBytes, "an MMA reads so much behind the last stage's tokens");
    const size_t stage = kPair * (a.w_bytes + kXBytes), room = (size_t)di.smem_optin - 1024;
    a.stages = (int)std::min<size_t>(stages_of(NC), rest < room ? (room - rest) / stage : 0);
    size_t bytes = (size_t)a.stages * stage + rest;
    if (a.stages * kPair * kXBytes + rest < past)
        bytes = (size_t)a.stages * kPair * a.w_bytes + past;
    if (a.stages < 2 || bytes > room)
        return cudaErrorInvalidConfiguration;
    CUtensorMap tw{}, tx{};
    if (!encode_rows(&tw, W, a.K, a.rows, a.K, parts, std::max(a.E, 1), a.tile_rows) ||
        (MODE == GEMM && !encode_rows(&tx, x, a.K, a.m, a.ldx, 1, 1, NC)))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    // (UP: the passes are known on the device alone, so a CTA on every SM)
    cfg.gridDim = dim3((unsigned)(MODE == UP ? di.sm_count : std::min(a.tiles, teams) * S));
    cfg.blockDim = dim3(threads_of(MODE));
    cfg.dynamicSmemBytes = alone_on_sm(1024 + bytes, (size_t)di.smem_optin);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, tw, tx);
}

template <int MODE, int NC>
cudaError_t launch_stream(const StreamArgs& a, const void* W, const void* x, cudaStream_t s)
{
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess)
        return e;
    // Clusters along K as long as the tiles of all of them at once cover the rows.  (With clusters of 4, 8 of 152 SMs are
    // left out, which costs less than tiles of half the rows.)
    if constexpr (MODE != UP) {
        int teams = 0;
        if ((e = clusters_of<MODE, NC, 4>(di, &teams)) != cudaSuccess)
            return e;
        if (a.rows <= kRowsMax * teams)
            return launch_stream<MODE, NC, 4>(a, W, x, di, s);
        if (a.rows <= kRowsMax * (di.sm_count / 2))
            return launch_stream<MODE, NC, 2>(a, W, x, di, s);
    }
    return launch_stream<MODE, NC, 1>(a, W, x, di, s);
}

}  // namespace

bool fp8_encoder_there() { return stream_encoder() != nullptr; }

bool fp8_stream_supported(const Fp8Gemm& p)
{
    // the scales of x lie in shared memory, 32 KB at most
    const int64_t columns = p.m <= 16 ? 16 : 32;
    return p.m <= 32 && (p.K + 127) / 128 * columns <= 8192;
}

cudaError_t launch_fp8_gemm_stream(const Fp8Gemm& p, cudaStream_t s)
{
    StreamArgs a{};
    a.w_scales = p.w_scales;
    a.K = (int)p.K;
    a.rows = (int)p.N;
    a.m = (int)p.m;
    a.x_scales = p.x_scales;
    a.ldx = p.ldx;
    a.ld_xs = p.ld_xs;
    a.y = p.y;
    a.ldy = p.ldy;
    a.y_bf16 = p.y_bf16;
    return a.m <= 16 ? launch_stream<GEMM, 16>(a, p.W, p.x, s) : launch_stream<GEMM, 32>(a, p.W, p.x, s);
}

size_t fp8_moe_workspace(int64_t m, int64_t topk, int64_t inter)
{
    return (size_t)(m * topk * inter * 4 + 255) / 256 * 256;
}

cudaError_t launch_fp8_moe(const Fp8Moe& p, cudaStream_t s)
{
    StreamArgs a{};
    a.m = (int)p.m;
    a.ids = p.ids;
    a.route_w = p.route_w;
    a.topk = p.topk;
    a.E = p.E;
    a.h = static_cast<float*>(p.workspace);
    a.y = p.y;
    a.ldy = p.ldy;
    a.y_bf16 = p.y_bf16;

    StreamArgs up = a;
    up.w_scales = p.gate_up_scales;
    up.K = (int)p.dim;
    up.rows = (int)p.inter;
    up.xb = p.x;
    up.ldx = p.ldx;

    StreamArgs down = a;
    down.w_scales = p.down_scales;
    down.K = (int)p.inter;
    down.rows = (int)p.dim;

    // 8 tokens a pass, 16 where experts, about evenly chosen, often have more
    const double mean = (double)p.m * p.topk / p.E;
    const bool many = std::min<double>((double)p.m, mean + 2 * std::sqrt(mean)) > 8;
    cudaError_t e = many ? launch_stream<UP, 48>(up, p.gate_up, nullptr, s) : launch_stream<UP, 32>(up, p.gate_up, nullptr, s);
    if (e != cudaSuccess)
        return e;
    return many ? launch_stream<DOWN, 64>(down, p.down, nullptr, s) : launch_stream<DOWN, 32>(down, p.down, nullptr, s);
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
