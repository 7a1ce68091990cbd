// Attention of new tokens over the paged cache (include/q2k.h,
// kv_attention_bf16) on the 5th-generation tensor cores.
//
//   S = Q K^T,  P = 2^(c S - c m),  O = P V / l,   c = scale * log2(e)
//
// with the running maximum m and sum l of each row: one pass over the keys.
//
// Rows.  The query heads of one kv head read the same keys, so a row is a
// (token, head) pair: g = Hq / Hkv heads of floor(128 / g) tokens fill a
// tile of 128 rows, from one new token (g rows) to long prompts.
//
// Work.  An item is a request's block of two row tiles on one kv head, its
// units its tiles of 128 keys and, in calls of some size, two for its start
// and end.  Every CTA (one per SM) sums the units of all requests from the
// lengths on the device and takes an equal run of them, wherever it starts
// and ends: a long decode is split over the whole GPU, a batch of ragged ones
// and causal prompts balance, and the host needs to know no length.  An item
// that one CTA finishes is written at once; the pieces of a split one go to
// the workspace, and a second launch joins them in a fixed order.
//
// One CTA, twelve warps:
//   warp 0       copies Q and K tiles (64 values of D by 128 rows, 128-byte
//                swizzle) into shared memory, a TMA box per page;
//   warp 3       works out the items and copies the V tiles;
//   warps 1, 2   issue the MMAs of streams 0 and 1: S into tensor memory, and
//                O += P V with P read from tensor memory (in S's place) and V
//                as it lies;
//   warps 4..7   softmax of stream 0, one row a thread,
//   warps 8..11  of stream 1.
// Two streams, so that the tensor cores work for one while the other's
// softmax runs: the two row tiles of a block over the same keys, or, where
// a block has a single tile (decode), every other key tile of it, merged at
// the item's end.
//
// P is relative to a reference that follows a row's maximum loosely: only
// when a score has passed it by more than 8 (P above 2^8; bf16 and the fp32
// sums hold large values as well as those below 1, and the division by l
// makes the result the same) does the reference move, and O is rescaled in
// tensor memory.  So the exponentials of a tile need not wait for its
// maximum; a tile that would pass 2^64 is done again with the maximum first.
// P is rounded to bf16 because the product wants both operands of one 16-bit
// type: V's is bf16, and 2^64 is past fp16.  Sums and maxima are fp32.  Against
// 64 bits the result is off by 2.3e-3 of its norm, where rounding it to bf16
// alone gives 1.7e-3.
//
// Rows of V that no row of the block may see (past the sequence's end, or
// before a window) are cleared in shared memory: a probability of zero
// times what an unused slot holds could be NaN.  Table entries that are not
// needed are never read; what is not needed of a tile is filled with zeros
// by reading past the cache.
//
// Every wait is bounded: on a timeout the kernel sets its error word, lets
// the copies in flight land, frees its tensor memory and returns.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <mutex>

#include "q2k_common.cuh"
#include "q2k_internal.h"
#include "q2k_umma.cuh"

namespace q2k {

__device__ int g_attn_error = 0;

namespace {

constexpr int kErrBadPage = 2, kErrSetup = 4;
constexpr int kThreads = 384;
constexpr int kMaxCtas = 160;
constexpr int kRows = 128;                  // rows of a tile, keys of a tile
constexpr int kHalfBytes = kRows * 128;     // 128 rows of 64 values
constexpr int kMaxStages = 12;
constexpr int kItems = 4;                   // items worked out ahead
constexpr float kGrow = 8.0f;               // log2 of how far P may pass 1 before its reference moves
constexpr int kTurnMmas = 2;                // MMAs of S within a turn
constexpr float kRange = 64.0f;             // and of how far within one tile

// A split item whose last piece CTA x wrote (its first slot): what the join
// needs to know, in one read.
struct alignas(16) Head {
    int first;      // CTA of the item's first piece (its second slot); -1: nothing to join
    int t0, n, h;   // first token, tokens, kv head
};

struct AttnArgs {
    uint16_t* out;
    float* lse;
    const int32_t *table, *cu_q, *seq_lens;
    int64_t ld_o, ld_table, max_pages, n_pages;
    int T, Hq, Hkv, D, n_req, shift, window;
    int g, tq;         // query heads of a kv head, tokens of a row tile
    int nst;           // ring stages
    int row_cap;       // rows of a piece in the workspace
    float c;           // scale * log2(e)
    int out_align;     // of the rows of out: 32, 16 or 2 bytes
    Head* heads;       // [gridDim.x] what each CTA's first item ended, if it did
    float* part_o;     // [2 * gridDim.x][D / 8][row_cap][8]
    float2* part_ml;   // [2 * gridDim.x][row_cap] maximum (times c) and sum
};

// What of its item a run holds: the first key tile, the last.
constexpr int kFirst = 1, kLast = 2;

// ---- the work ------------------------------------------------------------------

struct Request {
    int t0, n, base;  // first token, new tokens, position of the first
};

__device__ __forceinline__ Request load_request(const AttnArgs& a, int r)
{
    Request q;
    q.t0 = min(max(a.cu_q[r], 0), a.T);
    q.n = min(max(a.cu_q[r + 1], q.t0), a.T) - q.t0;
    q.base = min(max(a.seq_lens[r], 0), 1 << 30) - q.n;
    return q;
}

__device__ __forceinline__ int blocks_of(const AttnArgs& a, const Request& q) { return (q.n + 2 * a.tq - 1) / (2 * a.tq); }

// First key that a row at position p sees.
__device__ __forceinline__ int first_key(const AttnArgs& a, int p) { return a.window > 0 ? max(0, p - a.window + 1) : 0; }

// Key tiles [lo, hi] that tokens i0..i1-1 of a request see (one, wholly
// masked, where they see nothing).
__device__ __forceinline__ void key_tiles(const AttnArgs& a, const Request& q, int i0, int i1, int& lo, int& hi)
{
    lo = first_key(a, q.base + i0) / kRows;
    hi = max(q.base + i1 - 1, 0) / kRows;
    lo = min(lo, hi);
}

__device__ __forceinline__ int tiles_of(const AttnArgs& a, const Request& q, int j)
{
    int lo, hi;
    key_tiles(a, q, j * 2 * a.tq, min(q.n, (j + 1) * 2 * a.tq), lo, hi);
    return hi - lo + 1;
}

// An item counts as its key tiles and some more, its first units, for its
// start and end: without them the CTAs with many short items (the first
// blocks of a prompt) end last, and a cut near an item's first tile makes two
// items of one.  Two units: 64 decodes of 4100 tokens 189.8 us without, 179.4
// with one, 173.2 with two, 174.8 with five; 1346 tokens of 64 heads 54.1,
// 48.0, 46.7, 50.8; 8192 tokens over 4096 802, 792, 788, 794.  None where
// there are less than two tiles a CTA: then what counts is the most tiles of
// one (1500 tokens of 8 heads, window 323: 17.4 us without, 19.5 with two).
constexpr int kItemCost = 2;

__device__ __forceinline__ int cost_of_item(int64_t tiles) { return tiles >= 2 * (int64_t)gridDim.x ? kItemCost : 0; }

// Items of one row tile, no more of them than CTAs (and at most 32 requests),
// are not split where none has more than four key tiles above a CTA's share:
// such an item takes less time than its join, and counts as one unit.  One
// token over 200, 300, 450 (32 heads of 128): 14.6, 14.4, 14.6 us split, 10.6,
// 12.6, 13.7 whole (600: 15.0, 15.7); 16 tokens over 200, 500 each: 17.4, 21.7
// split, 14.0, 19.2 whole.
constexpr int kWholeTiles = 4;

// One item, or the part of it that lies in this CTA's run of units.
struct Item {
    int r, h, j;
    int t0, n, p0;   // first token (of all), tokens, position of the first
    int k0, k1;      // this CTA's key tiles [k0, k1); none: the run is over
    int lo;          // the item's first key tile
    int first[2], last[2];  // the tiles of the run that a stream works on
    int kind;
    int two;         // two row tiles (else one, its key tiles dealt to both streams)
};

// Where a CTA's run starts: item (r, h, j), its unit off, and the run's units.
struct Start {
    int r, h, j, off;
    int cost;   // units of an item before its first tile
    int whole;  // an item is one unit
    int64_t units;
    Request q;
};

// The items of a run, one after the other.
struct Walk {
    int r, h, j, off, cost, whole, blocks;
    int64_t left;
    Request q;

    __device__ __forceinline__ Walk(const AttnArgs& a, const Start& s)
        : r(s.r), h(s.h), j(s.j), off(s.off), cost(s.cost), whole(s.whole), blocks(blocks_of(a, s.q)), left(s.units), q(s.q)
    {
    }
    __device__ __forceinline__ void next(const AttnArgs& a, Item& it)
    {
        it.k0 = it.k1 = 0;
        if (left <= 0)
            return;
        it.r = r;
        it.h = h;
        it.j = j;
        const int i0 = j * 2 * a.tq, i1 = min(q.n, i0 + 2 * a.tq);
        it.t0 = q.t0 + i0;
        it.n = i1 - i0;
        it.p0 = q.base + i0;
        it.two = it.n > a.tq;
        int lo, hi;
        key_tiles(a, q, i0, i1, lo, hi);
        it.lo = lo;
        const int end = (int)min((int64_t)(whole ? 1 : hi - lo + 1 + cost), off + left);
        it.k0 = lo + max(0, off - cost);
        it.k1 = whole ? hi + 1 : lo + max(0, end - cost);  // k0 where the run ends before the first tile
        it.kind = (it.k0 == lo ? kFirst : 0) | (it.k1 == hi + 1 ? kLast : 0);
        for (int s = 0; s < 2; ++s) {
            it.first[s] = it.k0;
            it.last[s] = it.k1 - 1;
            if (it.two) {  // a row tile may see fewer keys than its block
                int l, x;
                key_tiles(a, q, s ? i0 + a.tq : i0, s ? i1 : i0 + a.tq, l, x);
                it.first[s] = max(it.k0, l);
                it.last[s] = min(it.k1 - 1, x);
            }
        }
        left -= end - off;
        off = 0;
        if (left > 0 && ++j >= blocks) {
            j = 0;
            if (++h >= a.Hkv) {
                h = 0;
                do
                    q = load_request(a, ++r);
                while (q.n == 0);
                blocks = blocks_of(a, q);
            }
        }
    }
};

// One warp, a request a lane (n = 0 where there is none): its key tiles on one kv head.
__device__ __forceinline__ int64_t tiles_of(const AttnArgs& a, const Request& q)
{
    const int lane = threadIdx.x & 31, nb = blocks_of(a, q);
    int64_t tiles = 0;
    if (nb <= 8)
        for (int j = 0; j < nb; ++j)
            tiles += tiles_of(a, q, j);
    for (uint32_t big = __ballot_sync(0xffffffffu, nb > 8); big; big &= big - 1) {
        const int src = __ffs(big) - 1;
        const Request b{__shfl_sync(0xffffffffu, q.t0, src), __shfl_sync(0xffffffffu, q.n, src),
                        __shfl_sync(0xffffffffu, q.base, src)};
        const int n = blocks_of(a, b);
        int64_t mine = 0;
        for (int j = lane; j < n; j += 32)
            mine += tiles_of(a, b, j);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            mine += __shfl_xor_sync(0xffffffffu, mine, o);
        if (lane == src)
            tiles = mine;
    }
    return tiles;
}

// The sum over the lanes up to this one.
__device__ __forceinline__ int64_t sum_to_lane(int64_t v)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if ((int)(threadIdx.x & 31) >= o)
            v += x;
    }
    return v;
}

// All threads: the units before each request into sums[0..n_req] (shared
// memory), with warp_sums as scratch; returns cost_of_item.
__device__ __forceinline__ int sum_units(const AttnArgs& a, int64_t* sums, int64_t* warp_sums)
{
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // requests side by side go to different warps: a long one keeps a whole warp
    int64_t all = 0;
    for (int r0 = 0; r0 < a.n_req; r0 += kThreads) {
        const int r = r0 + lane * kWarps + warp;
        const int64_t tiles = tiles_of(a, r < a.n_req ? load_request(a, r) : Request{0, 0, 0}) * a.Hkv;
        if (r < a.n_req)
            sums[r + 1] = tiles;
        all += tiles;
    }
    all = sum_to_lane(all);
    if (lane == 31)
        warp_sums[warp] = all;
    if (threadIdx.x == 0)
        sums[0] = 0;
    __syncthreads();
    all = 0;
    for (int w = 0; w < kWarps; ++w)
        all += warp_sums[w];
    const int cost = cost_of_item(all);
    __syncthreads();
    int64_t base = 0;
    for (int r0 = 0; r0 < a.n_req; r0 += kThreads) {
        const int r = r0 + (int)threadIdx.x;
        int64_t units = 0;
        if (r < a.n_req)
            units = sums[r + 1] + (int64_t)cost * a.Hkv * blocks_of(a, load_request(a, r));
        units = sum_to_lane(units);
        if (lane == 31)
            warp_sums[warp] = units;
        __syncthreads();
        int64_t before = base;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp)
                before += warp_sums[w];
            base += warp_sums[w];
        }
        if (r < a.n_req)
            sums[r + 1] = before + units;
        __syncthreads();
    }
    return cost;
}

// CTA c of n takes the units [run_start(c), run_start(c + 1)), one at least: n
// is the grid, or the units where they are fewer.
// (A 64-bit division is a long piece of code, and few calls have 2^23 units.)
__device__ __forceinline__ int64_t run_start(int64_t total, int c, int n)
{
    return total < 1 << 23 ? (int64_t)((uint32_t)total * (uint32_t)c / (uint32_t)n) : total * c / n;
}

// One warp: the request that unit `at` belongs to, from all sums.
__device__ __forceinline__ int find_request(const AttnArgs& a, const int64_t* sums, int64_t at)
{
    int lo = 0, hi = a.n_req;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= at)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// One warp: the item and the unit in it of unit rem of request r, which has
// per_head of them on each kv head; s.cost and s.whole are set.
__device__ __forceinline__ void find_start(const AttnArgs& a, int r, const Request& q, int64_t per_head, int64_t rem,
                                           Start& s)
{
    const int lane = threadIdx.x & 31;
    s.r = r;
    s.q = q;
    s.h = rem < 1ll << 31 && per_head < 1ll << 31 ? (int)((uint32_t)rem / (uint32_t)per_head) : (int)(rem / per_head);
    rem -= s.h * per_head;
    const int nb = blocks_of(a, q);
    s.j = 0;
    s.off = 0;
    for (int j0 = 0; j0 < nb; j0 += 32) {
        const int n = j0 + lane < nb ? s.whole ? 1 : tiles_of(a, q, j0 + lane) + s.cost : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o)
                sum += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, sum > rem);
        if (past) {
            const int src = __ffs(past) - 1;
            s.j = j0 + src;
            s.off = (int)(rem - __shfl_sync(0xffffffffu, sum - n, src));
            return;
        }
        rem -= __shfl_sync(0xffffffffu, sum, 31);
    }
}

// A place in the ring of stages and the parity of its use.
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void skip(int n, int nst)  // n <= nst
    {
        if ((s += n) >= nst) {
            s -= nst;
            phase ^= 1u;
        }
    }
    __device__ __forceinline__ void next(int nst) { skip(1, nst); }
};

// ---- PTX -----------------------------------------------------------------------

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Shared-memory matrix descriptors, the address in the low word, the rest
// here.  Q and K: rows of 64 values of D (128 bytes, swizzled), groups of 8
// rows 1024 bytes apart.  V as it lies: the same rows are 64 values along N,
// K going down them, and the next 64 values of N lie one half tile further.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
constexpr uint32_t kDescLoQK = 1u << 16, kDescLoV = (uint32_t)(kHalfBytes >> 4) << 16;

__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lo) { return (addr >> 4) | lo; }

// The MMAs of q2k_umma.cuh with descriptors put together from words.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "n"(kDescHi), "r"((uint32_t)acc)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 y, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b), "r"(idesc), "n"(kDescHi), "r"((uint32_t)acc)
        : "memory");
}

// The same value in every lane, known to the compiler as such.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

constexpr uint32_t kTransposeB = 1u << 16;

// 32 fp32 columns of this warp's TMEM lanes into v[OFF..]; complete after tcgen05.wait::ld.
template <int OFF, int N>
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[N])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[OFF + 0]), "=f"(v[OFF + 1]), "=f"(v[OFF + 2]), "=f"(v[OFF + 3]), "=f"(v[OFF + 4]), "=f"(v[OFF + 5]),
          "=f"(v[OFF + 6]), "=f"(v[OFF + 7]), "=f"(v[OFF + 8]), "=f"(v[OFF + 9]), "=f"(v[OFF + 10]),
          "=f"(v[OFF + 11]), "=f"(v[OFF + 12]), "=f"(v[OFF + 13]), "=f"(v[OFF + 14]), "=f"(v[OFF + 15]),
          "=f"(v[OFF + 16]), "=f"(v[OFF + 17]), "=f"(v[OFF + 18]), "=f"(v[OFF + 19]), "=f"(v[OFF + 20]),
          "=f"(v[OFF + 21]), "=f"(v[OFF + 22]), "=f"(v[OFF + 23]), "=f"(v[OFF + 24]), "=f"(v[OFF + 25]),
          "=f"(v[OFF + 26]), "=f"(v[OFF + 27]), "=f"(v[OFF + 28]), "=f"(v[OFF + 29]), "=f"(v[OFF + 30]),
          "=f"(v[OFF + 31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// mbar_wait_bounded with its clock read only after many polls: here most
// waits are short, and each lies on the path from one product to the next.
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity, const volatile int* abort_flag)
{
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity))
            return true;
        if ((it & 63u) == 63u) {
            if (*abort_flag)
                return false;
            const uint64_t t = global_timer_ns();
            if (t0 == 0)
                t0 = t;
            else if (t - t0 > 2000000000ull)
                return false;
        }
    }
}

template <int N>
__device__ __forceinline__ void set_regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// ---- the kernel ----------------------------------------------------------------

struct Shared {
    uint64_t q_full, q_empty, mma_done, s_full[2], p_ready[2], o_done[2], traded, read;
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t item_full[kItems], item_empty[kItems];
    Item items[kItems];
    int64_t warp_sums[kThreads / 32];
    Start start;
    int64_t total;
    float2 ml[2][kRows];  // one-tile items: each stream's maximum (times c) and sum
    uint32_t tmem;
    int abort_flag, turn;
    int loads[2], q_loads;  // K, V and Q tiles asked for, for the clean-up
};

__device__ __forceinline__ void store_32b(void* dst, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 16 fp32 values of a row of a piece, which lies in blocks of 8 columns, so
// that the rows of a warp are side by side.  (Row after row, the stores of an
// item took 2600 cycles: 12 chunks in a window 51.2 us against 48.0, 3744
// tokens of D = 96 33.4 against 28.6.)
__device__ __forceinline__ void store_part16(float* dst, int block, const float* v)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = __float_as_uint(v[8 * h + i]);
        store_32b(dst + h * block, w);
    }
}

// 16 values of a row of out, a sector in one store where it is aligned.
__device__ __forceinline__ void store_out16(uint16_t* dst, const float* v, float f, int align)
{
    if (align >= 16) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = pack_bf16(v[2 * i] * f, v[2 * i + 1] * f);
        if (align >= 32) {
            store_32b(dst, w);
        } else {
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            dst[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i] * f));
    }
}

// A row's maximum (times c) and sum, over all keys or some.  No key: the
// maximum is -inf and the sum 0, exactly; keys of score -inf alone leave a sum
// of 0 under a finite maximum (max_c); a sum of NaN (a score of NaN or +inf)
// is passed on.  So a sum is asked for being 0, never for being above it.
__device__ __forceinline__ float max_c(float m, float c, bool has_key) { return has_key ? fmaxf(m * c, -FLT_MAX) : -INFINITY; }

// What a part counts in a whole of the given maximum.
__device__ __forceinline__ float part_weight(float2 ml, float top) { return ml.y == 0.f ? 0.f : exp2_approx(ml.x - top); }

// 1 / l; zero for a row without a key.
__device__ __forceinline__ float inverse(float top, float l) { return top == -INFINITY && l == 0.f ? 0.f : 1.0f / l; }

__device__ __forceinline__ float lse_of(float mc, float l)
{
    return l == 0.f ? -INFINITY : (mc + log2f(l)) * 0.6931471805599453f;
}

template <int DB>  // halves of 64 values of D
__global__ void __launch_bounds__(kThreads, 1)
    kv_attn_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv)
{
    extern __shared__ __align__(1024) uint8_t smem[];  // two Q tiles, the ring, Shared
    constexpr int kTile = DB * kHalfBytes;
    pdl_launch_dependents();
    Shared& sh = *reinterpret_cast<Shared*>(smem + (size_t)(2 + a.nst) * kTile);
    const uint32_t q_smem = smem_u32(smem), ring = q_smem + 2 * kTile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &sh.abort_flag;

    if (smem_u32(smem) & 1023u) {  // the swizzle repeats every 1024 bytes
        pdl_wait();
        if (threadIdx.x == 0) {
            a.heads[blockIdx.x].first = -1;  // nothing to join
            atomicOr(&g_attn_error, kErrSetup);
        }
        return;
    }
    if (threadIdx.x == 32) {
        prefetch_map(&tq);
        prefetch_map(&tk);
        prefetch_map(&tv);
    }
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&sh.q_full), 1);
        mbar_init(smem_u32(&sh.q_empty), 2);
        mbar_init(smem_u32(&sh.mma_done), 2);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&sh.s_full[s]), 1);
            mbar_init(smem_u32(&sh.p_ready[s]), 4);
            mbar_init(smem_u32(&sh.o_done[s]), 1);
        }
        mbar_init(smem_u32(&sh.traded), 8);
        mbar_init(smem_u32(&sh.read), 8);
        for (int s = 0; s < a.nst; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), 2);
        }
        sh.abort_flag = sh.turn = 0;
        for (int s = 0; s < kItems; ++s) {
            mbar_init(smem_u32(&sh.item_full[s]), 1);
            mbar_init(smem_u32(&sh.item_empty[s]), 12);  // every working warp
        }
        sh.loads[0] = sh.loads[1] = sh.q_loads = 0;
        fence_mbar_init();
    }
    pdl_wait();
    // this CTA's run of units (the sums lie where the ring will be)
    int64_t* sums = reinterpret_cast<int64_t*>(smem + 2 * kTile);
    const bool few = a.n_req <= 32;
    Request req{0, 0, 0};
    int64_t upto = 0, per_head = 0, total;
    int cost;
    bool whole = false;
    if (few) {  // every warp for itself, a request a lane: no barrier
        if (lane < a.n_req)
            req = load_request(a, lane);
        per_head = tiles_of(a, req);
        upto = sum_to_lane(per_head * a.Hkv);
        const int64_t tiles = __shfl_sync(0xffffffffu, upto, 31);
        const uint32_t with = __ballot_sync(0xffffffffu, req.n > 0);
        whole = __all_sync(0xffffffffu, req.n <= a.tq && (per_head - kWholeTiles) * gridDim.x <= tiles) &&
                __popc(with) * a.Hkv <= (int)gridDim.x;
        cost = whole ? 0 : cost_of_item(tiles);
        if (whole) {
            per_head = with >> lane & 1u;
            upto = __popc(with & ((2u << lane) - 1u)) * a.Hkv;
        } else if (cost) {
            per_head += (int64_t)cost * blocks_of(a, req);
            upto = sum_to_lane(per_head * a.Hkv);
        }
        total = __shfl_sync(0xffffffffu, upto, 31);
    } else {
        cost = sum_units(a, sums, sh.warp_sums);
        total = sums[a.n_req];
    }
    const int runs = (int)min(total, (int64_t)gridDim.x);
    if (threadIdx.x == 0) {
        a.heads[blockIdx.x].first = -1;
        sh.total = total;
    }
    if ((int)blockIdx.x >= runs)
        return;
    const int64_t from = run_start(total, blockIdx.x, runs), to = run_start(total, blockIdx.x + 1, runs);
    if (warp == 0) {
        Start s;
        s.cost = cost;
        s.whole = whole;
        if (few) {
            const int r = __ffs(__ballot_sync(0xffffffffu, upto > from)) - 1;
            const int64_t rem = from - (upto - per_head * a.Hkv);
            find_start(a, r,
                       Request{__shfl_sync(0xffffffffu, req.t0, r), __shfl_sync(0xffffffffu, req.n, r),
                               __shfl_sync(0xffffffffu, req.base, r)},
                       __shfl_sync(0xffffffffu, per_head, r), __shfl_sync(0xffffffffu, rem, r), s);
        } else {
            const int r = find_request(a, sums, from);
            find_start(a, r, load_request(a, r), (sums[r + 1] - sums[r]) / a.Hkv, from - sums[r], s);
        }
        s.units = to - from;
        if (lane == 0)
            sh.start = s;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the sums are read; copies may overwrite them
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem;

    auto wait = [&](uint64_t& bar, uint32_t parity) {
        if (mbar_wait_short(smem_u32(&bar), parity & 1u, abort_flag))
            return true;
        atomicOr(&g_attn_error, Q2K_ERR_BIT_WAIT_TIMEOUT);
        *abort_flag = 1;
        return false;
    };
    auto warp_wait = [&](uint64_t& bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };

    // The items, from warp 3 to every warp (itself too): next_item() gives the
    // next one, done_item() hands its place back.
    Ring item_at;
    auto next_item = [&](const Item*& it) {
        it = &sh.items[item_at.s];
        return warp_wait(sh.item_full[item_at.s], item_at.phase) && it->k0 < it->k1;
    };
    auto done_item = [&]() {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(&sh.item_empty[item_at.s]));
        item_at.next(kItems);
    };
    const Item* it;
    bool ok = true;
    // 384 threads started with 168 registers each: 4 warps give up 80, 8 take 40 more
    if (warp < 4) {
        set_regs_down<88>();
        if (warp == 0 || warp == 3) {
            // ---- copies ----
            // Warp 0 takes K (and Q), warp 3 V: with pages of 16 a tile is 16
            // boxes, and one warp issued them too slowly (64 decodes of 4100
            // tokens: 220 us, 196 us with pages of 32).
            const bool is_v = warp == 3;
            const CUtensorMap* map = is_v ? &tv : &tk;
            const int box_rows = min(1 << a.shift, kRows), boxes = kRows / box_rows;
            Ring at, item_in;  // the stage of the next tile; the place of the next item to work out
            if (is_v)
                at.next(a.nst);
            int loads = 0, items = 0, put = 0;
            Walk walk(a, sh.start);
            auto put_item = [&]() {  // warp 3
                if (put >= kItems && !warp_wait(sh.item_empty[item_in.s], item_in.phase ^ 1u))
                    return false;
                ++put;
                Item x;
                walk.next(a, x);
                if (lane == 0) {
                    sh.items[item_in.s] = x;
                    mbar_arrive(smem_u32(&sh.item_full[item_in.s]));
                }
                __syncwarp();
                item_in.next(kItems);
                return true;
            };
            if (is_v)
                ok = put_item() && put_item();
            while (ok && next_item(it)) {
                if (is_v) {
                    if (!(ok = put_item()))
                        break;
                } else {
                    if (items > 0 && !(ok = warp_wait(sh.q_empty, (uint32_t)(items - 1))))
                        break;
                    if (lane == 0) {
                        const int tiles = it->two ? 2 : 1;
                        mbar_arrive_expect_tx(smem_u32(&sh.q_full), (uint32_t)(tiles * DB * a.g * a.tq * 128));
                        sh.q_loads = items + 1;
                        for (int s = 0; s < tiles; ++s)
#pragma unroll
                            for (int b = 0; b < DB; ++b)
                                tma_load_3d(q_smem + s * kTile + b * kHalfBytes, &tq, b * 64, it->h * a.g,
                                            it->t0 + s * a.tq, smem_u32(&sh.q_full));
                    }
                    __syncwarp();
                    ++items;
                }
                const int key_lo = first_key(a, it->p0), key_hi = it->p0 + it->n - 1, h = it->h, k1 = it->k1;
                const int32_t* table = a.table + it->r * a.ld_table;
                // the page that holds this lane's box of key tile k, or one past the cache where no row needs it
                auto page_of = [&](int k) -> int {
                    const int key = k * kRows + lane * box_rows;
                    if (lane >= boxes || key > key_hi || key + box_rows <= key_lo)
                        return (int)a.n_pages;
                    const int col = key >> a.shift;
                    const int page = col < a.max_pages ? table[col] : -1;
                    if (page >= 0 && page < a.n_pages)
                        return page;
                    atomicOr(&g_attn_error, kErrBadPage);
                    return (int)a.n_pages;
                };
                int here = page_of(it->k0);
                for (int k = it->k0; k < k1; ++k) {
                    const int page = here;
                    if (k + 1 < k1)
                        here = page_of(k + 1);  // on its way while this tile's stage is awaited
                    const int s = at.s;
                    if (2 * loads + is_v >= a.nst && !(ok = warp_wait(sh.empty[s], at.phase ^ 1u)))
                        break;
                    ++loads;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(smem_u32(&sh.full[s]), kTile);
                        sh.loads[is_v] = loads;
                    }
                    __syncwarp();
                    if (lane < boxes) {
                        const uint32_t dst = ring + (uint32_t)s * kTile + (uint32_t)(lane * box_rows * 128);
                        const int row = (k * kRows + lane * box_rows) & ((1 << a.shift) - 1);
#pragma unroll
                        for (int b = 0; b < DB; ++b)
                            tma_load_4d(dst + b * kHalfBytes, map, b * 64, row, h, page, smem_u32(&sh.full[s]));
                    }
                    at.skip(2, a.nst);
                }
                done_item();
            }
        } else {
            // ---- MMAs ----
            // Warp 1 issues for stream 0, warp 2 for stream 1: one warp keeps
            // few MMAs in flight (87 cycles or more for one of 128 x 128 x 16,
            // 70 to 80 from two warps; 64 would be the tensor cores' rate).
            // The whole warp runs the loop and one elected lane issues, so
            // that descriptors stay in warp-uniform registers.
            const int s = warp - 1;
            const uint32_t idesc_s = instr_desc(kRows), idesc_o = instr_desc(a.D) | kTransposeB;
            const uint32_t t_s = uniform(tmem + s * 256), t_o = t_s + 128;
            const uint32_t s_bar = uniform(smem_u32(&sh.s_full[s])), o_bar = uniform(smem_u32(&sh.o_done[s]));
            Ring at;  // the place of the item's first K tile; its V tile lies behind it, and so on
            uint32_t q_phase = 0, p_phase = 0;
            while (ok && next_item(it)) {
                if (!(ok = warp_wait(sh.q_full, q_phase)))
                    break;
                q_phase ^= 1u;
                const int first = it->first[s], last = it->last[s], k0 = it->k0, k1 = it->k1;
                const int v_lo = first_key(a, it->p0), v_hi = it->p0 + it->n;
                const bool two = it->two;
                done_item();
                const uint32_t qd = uniform(desc_lo(q_smem + (two ? s * kTile : 0), kDescLoQK));
                // Both streams work on every tile of a block of two row tiles; of
                // a block of one, this stream works on every other tile.  It
                // waits for the stages of the tiles between all the same, and
                // frees them: a warp that left out a use of a stage could take
                // the parity of an earlier one for its own.
                const int hop = two ? 1 : 2;
                int k = two ? k0 : k0 + s;
                Ring ks = at;  // K tile k's place
                auto pass = [&](Ring r) {  // the K and V stages from r on
                    for (int x = 0; x < 2; ++x) {
                        if (!warp_wait(sh.full[r.s], r.phase))
                            return false;
                        if (lane == 0)
                            mbar_arrive(smem_u32(&sh.empty[r.s]));
                        r.next(a.nst);
                    }
                    return true;
                };
                if (!two && s == 1) {
                    if (!(ok = pass(ks)))
                        break;
                    ks.skip(2, a.nst);
                }
                // Two row tiles, D above 64: a stream takes a turn for its O += P V
                // and the first MMAs of its next S.  Without turns the streams'
                // products interleave and end together, both softmaxes then run
                // at once and the tensor cores wait (8192 new tokens over 4096:
                // 876 us without, 787 with; none to six MMAs of S in the turn
                // give 782 to 790).  At D <= 64 the products are half as long and
                // the softmaxes bind: 12 chunks in a window take 45.4 us without
                // turns, 47.6 with them.
                bool mine = false;
                auto take_turn = [&]() {
                    bool got = true;
                    if (lane == 0) {
                        uint64_t t0 = 0;
                        for (uint32_t n = 0; atomicCAS(&sh.turn, 0, 1) != 0; ++n) {
                            if ((n & 63u) == 63u) {
                                const uint64_t now = global_timer_ns();
                                t0 = t0 ? t0 : now;
                                if (*abort_flag || now - t0 > 2000000000ull) {
                                    got = false;
                                    break;
                                }
                            }
                        }
                    }
                    mine = __all_sync(0xffffffffu, got);
                    return mine;
                };
                auto end_turn = [&]() {
                    __syncwarp();
                    if (mine && lane == 0)
                        atomicExch(&sh.turn, 0);
                    mine = false;
                };
                auto score = [&]() {  // S of tile k
                    if (!warp_wait(sh.full[ks.s], ks.phase))
                        return false;
                    fence_after();
                    const bool act = k >= first && k <= last;
                    const uint32_t kd = uniform(desc_lo(ring + (uint32_t)ks.s * kTile, kDescLoQK));
                    const uint32_t bar = uniform(smem_u32(&sh.empty[ks.s]));
                    if (elect_one()) {
                        if (act) {
                            // columns past D are zero in both tiles
#pragma unroll
                            for (int x = 0; x < DB * 4; ++x) {
                                const uint32_t off = (uint32_t)((x >> 2) * (kHalfBytes >> 4) + (x & 3) * 2);
                                if (x == kTurnMmas && mine)
                                    atomicExch(&sh.turn, 0);
                                mma_ss(t_s, qd + off, kd + off, idesc_s, x > 0);
                            }
                            umma_commit(s_bar);
                        }
                        umma_commit(bar);
                    }
                    __syncwarp();
                    return true;
                };
                bool begun = false;  // O holds a product of this item
                if (k < k1)
                    ok = score();
                while (ok && k < k1) {
                    Ring vs = ks;
                    vs.next(a.nst);
                    if (k + hop >= k1 && elect_one())
                        umma_commit(smem_u32(&sh.q_empty));  // this was the last S of the item
                    __syncwarp();
                    if (!(ok = warp_wait(sh.full[vs.s], vs.phase)))
                        break;
                    const bool act = k >= first && k <= last;
                    if (act) {
                        // clear the rows that no row of the block sees (the other stream may write the same zeros)
                        const int z_lo = max(0, min(kRows, v_lo - k * kRows));
                        const int z_hi = max(0, min(kRows, v_hi - k * kRows));
                        if (z_lo > 0 || z_hi < kRows) {
                            for (int i = lane; i < kRows * 8; i += 32) {
                                const int row = i >> 3;
                                if (row < z_lo || row >= z_hi) {
                                    uint8_t* p = smem + (size_t)(2 + vs.s) * kTile + i * 16;
#pragma unroll
                                    for (int b = 0; b < DB; ++b)
                                        *reinterpret_cast<uint4*>(p + b * kHalfBytes) = make_uint4(0, 0, 0, 0);
                                }
                            }
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                        }
                        if (!(ok = warp_wait(sh.p_ready[s], p_phase)))
                            break;
                        p_phase ^= 1u;
                        if (two && DB == 2) {
                            // nothing is waited for during a turn: the next K tile
                            // may need a stage that the other stream has yet to free
                            Ring ns = vs;
                            ns.next(a.nst);
                            if (!(ok = (k + 1 >= k1 || warp_wait(sh.full[ns.s], ns.phase)) && take_turn()))
                                break;
                        }
                        fence_after();
                    }
                    const uint32_t vd = uniform(desc_lo(ring + (uint32_t)vs.s * kTile, kDescLoV));
                    const uint32_t bar = uniform(smem_u32(&sh.empty[vs.s]));
                    if (elect_one()) {
                        if (act) {
#pragma unroll
                            for (int x = 0; x < kRows / 16; ++x)
                                mma_ts(t_o, t_s + x * 8, vd + (uint32_t)(x * (2048 >> 4)), idesc_o, begun || x > 0);
                            if (k + hop > last)
                                umma_commit(o_bar);  // O is complete
                        }
                        umma_commit(bar);
                    }
                    __syncwarp();
                    begun |= act;
                    ks.skip(2, a.nst);
                    if (!two) {
                        if (k + 1 < k1 && !(ok = pass(ks)))
                            break;
                        ks.skip(2, a.nst);
                    }
                    k += hop;
                    if (k < k1)
                        ok = score();
                    if (!(k < k1 && k >= first && k <= last))
                        end_turn();  // no S to end it
                    mine = false;
                }
                if (k0 + (two ? 0 : s) >= k1 && lane == 0)
                    mbar_arrive(smem_u32(&sh.q_empty));  // no tile of this item was this stream's
                const int used = 2 * (k1 - k0), rounds = used / a.nst;
                at.phase ^= (uint32_t)rounds & 1u;
                at.skip(used - rounds * a.nst, a.nst);
            }
            // every product and arrival has landed before the CTA can exit
            if (elect_one())
                umma_commit(smem_u32(&sh.mma_done));
            __syncwarp();
            mbar_wait_bounded(smem_u32(&sh.mma_done), 0u, nullptr);
            __syncwarp();
        }
    } else {
        set_regs_up<208>();
        // ---- softmax ----
        const int s = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16), t_s = lanes + s * 256, t_o = t_s + 128;
        const int ti = row / a.g, head = row - ti * a.g;
        uint32_t phase = 0, done = 0, trade = 0;
        while (ok && next_item(it)) {
            const bool two = it->two;
            const int i = ti + (two && s ? a.tq : 0);  // token of the block
            const bool live = row < a.g * a.tq && i < it->n;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int p = it->p0 + i;
            const int k_max = live ? p : INT_MAX, k_min = live ? first_key(a, p) : 0;
            float m = -INFINITY, l = 0.f;  // m: what P is relative to
            float m_next = -INFINITY;
            bool pending = false;          // m_next takes over with the next tile
            int count = 0;
            const int k_last = it->last[s], stride = two ? 1 : 2;
            for (int k = it->first[s] + (two ? 0 : s); k <= k_last; k += stride) {
                if (!(ok = warp_wait(sh.s_full[s], phase)))
                    break;
                fence_after();
                if (warp_live) {
                    // P against a new reference from here on.  S of this tile
                    // is complete, and with it the product issued before it.
                    auto move_to = [&](float m_new) {
                        const float f = m_new == m ? 1.f : exp2_approx((m - m_new) * a.c);
                        m = m_new;
                        if (count > 0) {
                            l *= f;
                            for (int x = 0; x < a.D; x += 16) {
                                float o[16];
                                uint32_t w[16];
                                tmem_ld16(t_o + x, o);
#pragma unroll
                                for (int y = 0; y < 16; ++y)
                                    w[y] = __float_as_uint(o[y] * f);
                                tmem_st16(t_o + x, w);
                            }
                        }
                    };
                    if (pending) {
                        move_to(m_next);
                        pending = false;
                    }
                    const int key0 = k * kRows;
                    const bool edge = __any_sync(0xffffffffu, key0 + kRows - 1 > k_max || key0 < k_min);
                    const float2 c2 = make_float2(a.c, a.c);
                    float top = -INFINITY;
                    bool redo = edge || count == 0;
                    if (!redo) {
                        float v[kRows];
                        tmem_ld32<0>(t_s, v);
                        tmem_ld32<32>(t_s + 32, v);
                        tmem_ld32<64>(t_s + 64, v);
                        tmem_ld32<96>(t_s + 96, v);
                        tmem_wait_ld();
                        // Against the reference as it stands, with the maximum
                        // taken on the way: it only has to catch what passes
                        // the range, and moves the reference for the next tile.
                        const float mc = m == -INFINITY ? 0.f : m * a.c;
                        const float2 mc2 = make_float2(-mc, -mc);
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                        float t2[2] = {-INFINITY, -INFINITY};
                        uint32_t w[kRows / 2];
#pragma unroll
                        for (int y = 0; y < kRows / 2; ++y) {
                            const float x0 = v[2 * y], x1 = v[2 * y + 1];
                            t2[y & 1] = max3(t2[y & 1], x0, x1);
                            float2 e = fma2(make_float2(x0, x1), c2, mc2);
                            e.x = exp2_approx(e.x);
                            e.y = exp2_approx(e.y);
                            sum[y & 1] = add2(sum[y & 1], e);
                            w[y] = pack_bf16(e.x, e.y);
                        }
                        top = fmaxf(t2[0], t2[1]);
                        const float up = live ? (top - m) * a.c : 0.f;
                        redo = __any_sync(0xffffffffu, up > kRange);
                        if (!redo) {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                tmem_st16(t_s + x * 16, reinterpret_cast<const uint32_t(&)[16]>(w[x * 16]));
                            sum[0] = add2(sum[0], sum[1]);
                            l += sum[0].x + sum[0].y;
                            pending = __any_sync(0xffffffffu, up > kGrow);
                            m_next = fmaxf(m, top);
                        }
                    }
                    if (redo) {
                        // Columns that some row of the warp sees, and those that all do:
                        // of an edge tile most are one or the other.
                        int some_lo = 0, some_hi = kRows - 1, all_lo = 0, all_hi = kRows - 1;
                        const int lo = k_min - key0, hi = k_max - key0;
                        if (edge) {
                            some_lo = __reduce_min_sync(0xffffffffu, live ? lo : INT_MAX);
                            some_hi = __reduce_max_sync(0xffffffffu, live ? hi : INT_MIN);
                            all_lo = __reduce_max_sync(0xffffffffu, live ? lo : INT_MIN);
                            all_hi = __reduce_min_sync(0xffffffffu, live ? hi : INT_MAX);
                        }
                        // 32 columns at a time, in loops that stay loops: this is
                        // the first code that a short call runs, and its time there
                        // is that of fetching it (unrolled: one token over 2047 17.2 us
                        // against 16.1, 12 chunks in a window 53.3 against 51.0, 8192
                        // tokens 829 against 809).
                        auto unseen = [&](int x) { return x > some_hi || x + 31 < some_lo; };
                        auto load = [&](int x, float(&u)[32]) {
                            tmem_ld32<0>(t_s + x, u);
                            tmem_wait_ld();
                            if (x < all_lo || x + 31 > all_hi) {
                                const int from = lo - x, to = hi - x;
#pragma unroll
                                for (int y = 0; y < 32; ++y)
                                    u[y] = y <= to && y >= from ? u[y] : -INFINITY;
                            }
                        };
                        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                        for (int x = 0; x < kRows; x += 32) {
                            if (unseen(x))
                                continue;
                            float u[32];
                            load(x, u);
#pragma unroll
                            for (int y = 0; y < 32; y += 8) {
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    t4[z] = max3(t4[z], u[y + z], u[y + 4 + z]);
                            }
                        }
                        top = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
                        // false for -inf - -inf
                        if (__any_sync(0xffffffffu, live && (top - m) * a.c > kGrow))
                            move_to(fmaxf(m, top));
                        const float mc = m == -INFINITY ? 0.f : m * a.c;
                        const float2 mc2 = make_float2(-mc, -mc);
                        float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
                        for (int x = 0; x < kRows; x += 32) {
                            uint32_t w[16] = {};
                            if (!unseen(x)) {
                                float u[32];
                                load(x, u);
#pragma unroll
                                for (int y = 0; y < 16; ++y) {
                                    float2 e = fma2(make_float2(u[2 * y], u[2 * y + 1]), c2, mc2);
                                    e.x = exp2_approx(e.x);
                                    e.y = exp2_approx(e.y);
                                    sum = add2(sum, e);
                                    w[y] = pack_bf16(e.x, e.y);
                                }
                            }
                            tmem_st16(t_s + x / 2, w);
                        }
                        l += sum.x + sum.y;
                    }
                    tmem_wait_st();
                }
                fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sh.p_ready[s]));
                phase ^= 1u;
                ++count;
            }
            if (!ok)
                break;
            // ---- the item's result ----
            const int kind = it->kind;
            const bool whole = (kind & kFirst) && (kind & kLast);
            const int slot = 2 * blockIdx.x + ((kind & kFirst) ? 1 : 0);
            if (!(kind & kFirst) && (kind & kLast) && warp == 4 && lane == 0) {
                // the CTA whose run holds the item's first tile
                const int64_t tot = sh.total;
                const int runs = (int)min(tot, (int64_t)gridDim.x);
                const int64_t unit = run_start(tot, blockIdx.x, runs) - (it->k0 - it->lo);
                int c = (int)((float)unit / (float)tot * (float)runs);
                while (run_start(tot, c + 1, runs) <= unit)
                    ++c;
                while (run_start(tot, c, runs) > unit)
                    --c;
                a.heads[blockIdx.x] = Head{c, it->t0, it->n, it->h};
            }
            const int64_t out_row = (int64_t)(it->t0 + i);
            const int out_head = it->h * a.g + head;
            done_item();
            uint16_t* dst = a.out + out_row * a.ld_o + (int64_t)out_head * a.D;
            float* part = a.part_o + (int64_t)slot * a.row_cap * a.D + ((two ? s * kRows : 0) + row) * 8;
            const float mc = max_c(m, a.c, live && p >= 0);
            if (count > 0) {
                if (!(ok = warp_wait(sh.o_done[s], done)))
                    break;
                done ^= 1u;
            }
            float f0 = 1.f, f1 = 0.f, top = mc, sum = l;
            if (!two) {
                // both streams hold a part of the same rows: each joins every other 32 columns
                sh.ml[s][row] = make_float2(mc, l);
                fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sh.traded));
                if (!(ok = warp_wait(sh.traded, trade)))
                    break;
                const float2 e0 = sh.ml[0][row], e1 = sh.ml[1][row];
                top = fmaxf(e0.x, e1.x);
                f0 = part_weight(e0, top);
                f1 = part_weight(e1, top);
                sum = e0.y * f0 + e1.y * f1;
            } else if (l == 0.f) {
                f0 = 0.f;  // a row without a key is zero, whatever O holds
            }
            fence_after();
            if (warp_live) {
                const float inv = whole ? inverse(top, sum) : 1.f;
                for (int x = two ? 0 : s * 32; x < a.D; x += two ? 32 : 64) {
                    float o[32];
                    tmem_ld32<0>((two ? t_o : lanes + 128) + x, o);
                    if (!two) {
                        float o1[32];
                        tmem_ld32<0>(lanes + 384 + x, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            o[y] = (f0 == 0.f ? 0.f : o[y] * f0) + (f1 == 0.f ? 0.f : o1[y] * f1);
                    } else {
                        tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            o[y] = f0 == 0.f ? 0.f : o[y];
                    }
                    if (live) {
#pragma unroll
                        for (int y = 0; y < 32; y += 16)
                            if (x + y < a.D) {
                                if (whole)
                                    store_out16(dst + x + y, o + y, inv, a.out_align);
                                else
                                    store_part16(part + (x + y) * a.row_cap, 8 * a.row_cap, o + y);
                            }
                    }
                }
                if (live && (two || s == 0)) {
                    if (!whole)
                        a.part_ml[(int64_t)slot * a.row_cap + (two ? s * kRows : 0) + row] = make_float2(top, sum);
                    else if (a.lse)
                        a.lse[out_row * a.Hq + out_head] = lse_of(top, sum);
                }
            }
            fence_before();
            if (!two) {
                // O and ml are free again once both streams have read them
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sh.read));
                if (!(ok = warp_wait(sh.read, trade)))
                    break;
                trade ^= 1u;
            }
        }
    }
    fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) {
        // let the copies that were issued land before the CTA exits
        for (int v = 0; v < 2; ++v)
            for (int i = max(0, sh.loads[v] - a.nst); i < sh.loads[v]; ++i)
                mbar_wait_bounded(smem_u32(&sh.full[(2 * i + v) % a.nst]), (uint32_t)((2 * i + v) / a.nst) & 1u, nullptr);
        if (sh.q_loads > 0)
            mbar_wait_bounded(smem_u32(&sh.q_full), (uint32_t)(sh.q_loads - 1) & 1u, nullptr);
    }
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// Joins the pieces of split items: block x takes the item whose last piece
// CTA x of the first launch wrote, in the order of the keys.  What bounds it
// is latency: what it has to know comes in one read, and a row's next pieces
// are on their way together with their maxima.  Where there are many rows,
// which then mostly have two pieces, a lane takes 16 columns of a row, so
// that a warp reads the blocks as they lie; where there are few, which have
// many pieces, a warp takes a row.
constexpr int kJoinWarps = 8, kJoinY = kRows / 16;

struct JoinRow {
    int in, i;  // row of its tile, token of the block
    bool live;
    __device__ __forceinline__ JoinRow(const AttnArgs& a, const Head& head, int row) : in(row & 127)
    {
        const int ti = in / a.g;
        i = (row >> 7) * a.tq + ti;
        live = in < a.g * a.tq && i < head.n;
        in -= ti * a.g;  // now the head of the group
    }
};

// A piece's first row in the workspace.
__device__ __forceinline__ int64_t piece_row(const AttnArgs& a, int c, int first)
{
    return (int64_t)(2 * c + (c == first)) * a.row_cap;
}

__device__ __forceinline__ void load_32b(const float* src, float* v)
{
    uint32_t w[8];
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(src)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = __uint_as_float(w[i]);
}

__device__ __forceinline__ void join_columns(const AttnArgs& a, const Head& head, int first, int last)
{
    const int row = (int)threadIdx.x, x = (int)blockIdx.y * 16;
    if (row >= (head.n > a.tq ? 2 * kRows : kRows) || x >= a.D)
        return;
    const JoinRow r(a, head, row);
    if (!r.live)
        return;
    struct Piece {
        float v[16];
        float2 ml;
    };
    auto fetch = [&](int c, Piece& p) {
        if (c > last)
            return;
        const int64_t at = piece_row(a, c, first);
        p.ml = a.part_ml[at + row];
        const float* src = a.part_o + at * a.D + ((x >> 3) * a.row_cap + row) * 8;
        load_32b(src, p.v);
        load_32b(src + a.row_cap * 8, p.v + 8);
    };
    constexpr int kAhead = 2;
    Piece p[kAhead] = {};
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        fetch(first + i, p[i]);
    float top = -INFINITY, sum = 0.f, o[16];
#pragma unroll
    for (int y = 0; y < 16; ++y)
        o[y] = 0.f;
#pragma unroll 4
    for (int c = first; c <= last; ++c)
        top = fmaxf(top, a.part_ml[piece_row(a, c, first) + row].x);
    for (int c0 = first; c0 <= last; c0 += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (c0 + i > last)
                break;
            // a piece without a key for this row holds zeros
            const float f = part_weight(p[i].ml, top);
            sum = fmaf(p[i].ml.y, f, sum);
#pragma unroll
            for (int y = 0; y < 16; ++y)
                o[y] = fmaf(p[i].v[y], f, o[y]);
            fetch(c0 + i + kAhead, p[i]);
        }
    }
    const int64_t t = head.t0 + r.i;
    const int h = head.h * a.g + r.in;
    store_out16(a.out + t * a.ld_o + (int64_t)h * a.D + x, o, inverse(top, sum), a.out_align);
    if (a.lse && x == 0)
        a.lse[t * a.Hq + h] = lse_of(top, sum);
}

__device__ __forceinline__ void join_rows(const AttnArgs& a, const Head& head, int first, int last)
{
    constexpr int kAhead = 4;
    const int lane = threadIdx.x & 31, col = lane * 4;
    const int rows = head.n > a.tq ? 2 * kRows : kRows;
    for (int row = (int)blockIdx.y * kJoinWarps + (threadIdx.x >> 5); row < rows; row += kJoinWarps * (int)gridDim.y) {
        const JoinRow r(a, head, row);
        if (!r.live)
            continue;
        struct Pieces {
            float4 v[kAhead];
            float2 ml[kAhead];
        };
        Pieces now, next;
        auto fetch = [&](Pieces& p, int c) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const bool there = c + j <= last;
                const int64_t at = piece_row(a, c + j, first);
                p.ml[j] = there ? a.part_ml[at + row] : make_float2(-INFINITY, 0.f);
                p.v[j] = there && col < a.D ? *reinterpret_cast<const float4*>(
                                                  a.part_o + at * a.D + ((col >> 3) * a.row_cap + row) * 8 + (col & 7))
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        };
        fetch(now, first);
        // the maximum of all pieces, 32 at a time
        float top = -INFINITY;
        for (int c = first + lane; c <= last; c += 32)
            top = fmaxf(top, a.part_ml[piece_row(a, c, first) + row].x);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = first; c <= last; c += kAhead) {
            fetch(next, c + kAhead);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float f = part_weight(now.ml[j], top);
                sum = fmaf(now.ml[j].y, f, sum);
                o.x = fmaf(now.v[j].x, f, o.x);
                o.y = fmaf(now.v[j].y, f, o.y);
                o.z = fmaf(now.v[j].z, f, o.z);
                o.w = fmaf(now.v[j].w, f, o.w);
            }
            now = next;
        }
        const float inv = inverse(top, sum);
        const int64_t t = head.t0 + r.i;
        const int h = head.h * a.g + r.in;
        if (col < a.D) {
            uint16_t* dst = a.out + t * a.ld_o + (int64_t)h * a.D + col;
            const uint32_t lo = pack_bf16(o.x * inv, o.y * inv), hi = pack_bf16(o.z * inv, o.w * inv);
            if (a.out_align >= 16) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
            } else {
                dst[0] = (uint16_t)lo;
                dst[1] = (uint16_t)(lo >> 16);
                dst[2] = (uint16_t)hi;
                dst[3] = (uint16_t)(hi >> 16);
            }
        }
        if (a.lse && lane == 0)
            a.lse[t * a.Hq + h] = lse_of(top, sum);
    }
}

__global__ void __launch_bounds__(kJoinWarps * 32, 4) kv_attn_join_kernel(const AttnArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int last = (int)blockIdx.x;
    const Head head = a.heads[last];
    if (head.first < 0)
        return;
    if (head.n * a.g > 64)
        join_columns(a, head, head.first, last);
    else
        join_rows(a, head, head.first, last);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

bool encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box,
                      estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace: piece headers, then sums and maxima, then rows of O.
struct Layout {
    int64_t row_cap;
    size_t ml, o, bytes;
};

Layout layout_of(int64_t T, int64_t Hq, int64_t Hkv, int64_t D)
{
    const int64_t g = Hq / Hkv, tq = kRows / g;
    Layout w{};
    w.row_cap = T <= tq ? std::max<int64_t>(1, T * g) : 2 * kRows;
    w.ml = (size_t)kMaxCtas * sizeof(Head);
    w.o = w.ml + ((size_t)2 * kMaxCtas * w.row_cap * sizeof(float2) + 31) / 32 * 32;
    w.bytes = w.o + (size_t)2 * kMaxCtas * w.row_cap * D * sizeof(float);
    return w;
}

template <int DB>
cudaError_t launch_tc(AttnArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                      int smem_optin, cudaStream_t s)
{
    constexpr size_t tile = DB * kHalfBytes;
    static std::atomic<unsigned long long> devs{0};
    cudaError_t e = allow_max_smem(kv_attn_kernel<DB>, devs);
    if (e != cudaSuccess)
        return e;
    a.nst = (int)std::min<size_t>(kMaxStages, ((size_t)smem_optin - sizeof(Shared)) / tile - 2);
    if (a.nst < 5 || (size_t)a.nst * tile < ((size_t)a.n_req + 1) * sizeof(int64_t))
        return cudaErrorInvalidConfiguration;
    const size_t smem = (2 + (size_t)a.nst) * tile + sizeof(Shared);
    if ((e = launch_pdl(kv_attn_kernel<DB>, dim3(grid), dim3(kThreads), smem, s, a, tq, tk, tv)) != cudaSuccess)
        return e;
    const int y = a.row_cap <= 64 ? (a.row_cap + kJoinWarps - 1) / kJoinWarps : kJoinY;
    return launch_pdl(kv_attn_join_kernel, dim3(grid, y), dim3(kJoinWarps * 32), 0, s, a);
}

}  // namespace

bool attn_supported() { return encoder() != nullptr; }

size_t kv_attention_workspace(int64_t T, int64_t Hq, int64_t Hkv, int64_t D) { return layout_of(T, Hq, Hkv, D).bytes; }

cudaError_t launch_kv_attention(const AttnProblem& p, cudaStream_t s)
{
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess)
        return e;
    AttnArgs a{};
    a.out = p.out;
    a.lse = p.lse;
    a.table = p.block_table;
    a.cu_q = p.cu_q;
    a.seq_lens = p.seq_lens;
    a.ld_o = p.ld_o;
    a.max_pages = p.max_pages;
    a.ld_table = p.ld_table;
    a.n_pages = p.n_pages;
    a.T = (int)p.T;
    a.Hq = (int)p.Hq;
    a.Hkv = (int)p.Hkv;
    a.D = (int)p.D;
    a.n_req = (int)p.n_req;
    a.window = (int)std::min<int64_t>(p.window, 0x7fffffff);
    while ((1 << a.shift) < p.page_size)
        ++a.shift;
    a.g = a.Hq / a.Hkv;
    a.tq = kRows / a.g;
    a.c = p.scale * 1.4426950408889634f;
    const uintptr_t out_bits = reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.ld_o * 2);
    a.out_align = out_bits % 32 == 0 ? 32 : out_bits % 16 == 0 ? 16 : 2;
    const Layout w = layout_of(p.T, p.Hq, p.Hkv, p.D);
    uint8_t* ws = static_cast<uint8_t*>(p.workspace);
    a.row_cap = (int)w.row_cap;
    a.heads = reinterpret_cast<Head*>(ws);
    a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
    a.part_o = reinterpret_cast<float*>(ws + w.o);

    CUtensorMap tq{}, tk{}, tv{};
    const cuuint64_t qd[3] = {(cuuint64_t)p.D, (cuuint64_t)p.Hq, (cuuint64_t)p.T};
    const cuuint64_t qs[2] = {(cuuint64_t)p.D * 2, (cuuint64_t)p.ld_q * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)a.g, (cuuint32_t)a.tq};
    const cuuint64_t kd[4] = {(cuuint64_t)p.D, (cuuint64_t)p.page_size, (cuuint64_t)p.Hkv, (cuuint64_t)p.n_pages};
    const cuuint64_t ks[3] = {(cuuint64_t)p.D * 2, (cuuint64_t)(p.page_size * p.D * 2), (cuuint64_t)p.page_stride * 2};
    const cuuint32_t kb[4] = {64, (cuuint32_t)std::min<int64_t>(p.page_size, kRows), 1, 1};
    if (!encode(&tq, p.q, 3, qd, qs, qb) || !encode(&tk, p.k_cache, 4, kd, ks, kb) ||
        !encode(&tv, p.v_cache, 4, kd, ks, kb))
        return cudaErrorInvalidValue;
    const int grid = std::min(di.sm_count, kMaxCtas);
    return p.D <= 64 ? launch_tc<1>(a, tq, tk, tv, grid, di.smem_optin, s)
                     : launch_tc<2>(a, tq, tk, tv, grid, di.smem_optin, s);
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
