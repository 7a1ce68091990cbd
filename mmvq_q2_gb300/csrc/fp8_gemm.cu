// The product of 8-bit floating-point operands for many rows (include/q2k.h,
// fp8_gemm; up to 32 rows go to fp8_stream.cu) on the 5th-generation tensor
// cores: tcgen05.mma kind::f8f6f4 on e4m3, fp32 accumulators in tensor memory.
//
// The scales change every 128 values along K, so an accumulator holds one such
// block alone: four MMAs of K = 32 fill one of two to eight accumulators while
// another is read back, multiplied by its rows' and its block's scale and added
// to fp32 sums in registers.  A tile is 128 rows of x (a tensor memory lane
// each, so a thread has one row and its scale is one number) by BN rows of W
// (half of BN to a group of four warps; within one block of 128, so W's scale
// is one number too):
//   warps 0,2,3  copy tiles of 128 values of K (128-byte swizzled) into a ring
//                of shared-memory stages, a stage in turn;
//   warp 1       issues the MMAs;
//   warps 4..11  read back, scale, add; at the end they leave y in shared
//                memory for tensor copies to store (8191 x 8192 x 4096 213 us;
//                stored by the warps 222).
// What bounds a block of K at BN = 256, 920 to 940 cycles where its MMAs take 510:
// the way round an accumulator (until the adding warps are awake 1121, read back
// 487, until the next issue 246) is two blocks, for two accumulators.  192
// columns, read back at once, took 254 us; pairs of SMs on one tile 220.
// CTAs walk the tiles, 16 tiles of x at a time, so that what runs together
// shares operands in L2.  Where there are fewer tiles than SMs, the CTAs of a
// cluster share a tile along K and add their sums through shared memory, in
// the order of K (no atomics: a call repeats bit for bit).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "fp8_common.cuh"
#include "q2k_internal.h"

namespace q2k {

__device__ int g_fp8_gemm_error = 0;

namespace {

constexpr int kThreads = 384;
constexpr int kTM = 128;             // rows of x in a tile
constexpr int kTK = 128;             // values of K in a stage: one swizzle row, one block of the scales
constexpr int kXTile = kTM * kTK;
constexpr int kMaxStages = 12;
constexpr int kGroup = 16;           // tiles of x that are walked together

struct GemmArgs {
    const float *x_scales, *w_scales;
    void* y;
    int64_t ld_xs, ldy;
    int m, N, blocks;  // blocks of 128 along K
    int tiles_m, tiles_n, stages;
    int bulk_store;     // y by tensor copies
    int y_bf16, align;  // bytes that the start of every 32 values of y is aligned to: 32, 16 or less
};

struct GemmShared {
    uint64_t full[kMaxStages], done[kMaxStages];  // of a stage: copied; multiplied
    uint64_t acc_empty[8];                        // of an accumulator: read back
    uint32_t tmem;
    int abort_flag;
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

// acc += v * f of 16 values, two an instruction (one at a time 229 us for 8191 x 8192 x 4096 against 219).
__device__ __forceinline__ void fma_pairs(float* acc, const float* v, float f)
{
#pragma unroll
    for (int i = 0; i < 16; i += 2)
        asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%0, %1};\n\t"
            "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
            : "+f"(acc[i]), "+f"(acc[i + 1])
            : "f"(v[i]), "f"(v[i + 1]), "f"(f));
}

__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// The 32 bytes at dst where they are aligned to `align`, a sector in one store if that is 32.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8], int align)
{
    if (align >= 32) {
        store32(dst, w);
    } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// n values of a row of y from column `col` on, 8 at a time (n a multiple of 8).
template <int n>
__device__ __forceinline__ void store_row(const GemmArgs& a, int64_t row, int col, const float* v)
{
    if (a.y_bf16) {
        uint16_t* y = static_cast<uint16_t*>(a.y) + row * a.ldy + col;
        if (n % 16 == 0 && a.align >= 16 && col + n <= a.N) {
#pragma unroll
            for (int i = 0; i < n; i += 16) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[i + 2 * j + 1]), "f"(v[i + 2 * j]));
                store32(y + i, w, a.align);
            }
        } else {
#pragma unroll
            for (int i = 0; i < n; ++i)
                if (col + i < a.N)
                    y[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
        }
    } else {
        float* y = static_cast<float*>(a.y) + row * a.ldy + col;
        if (a.align >= 16 && col + n <= a.N) {
#pragma unroll
            for (int i = 0; i < n; i += 8) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = __float_as_uint(v[i + j]);
                store32(y + i, w, a.align);
            }
        } else {
#pragma unroll
            for (int i = 0; i < n; ++i)
                if (col + i < a.N)
                    y[i] = v[i];
        }
    }
}

// A box of 128 bytes by 32 rows of y from shared memory; lane 0 of the warp that has it.
__device__ __forceinline__ void store_box(const CUtensorMap* map, int x, int y, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}

// n columns of a warp's 32 rows by such boxes, through its one buffer (two would cost a stage of the ring, and more time
// than they save).
template <int n, bool BF16>
__device__ __forceinline__ void store_boxes(const GemmArgs& a, const CUtensorMap* map, uint8_t* buf, int row0, int col, const float* v)
{
    constexpr int kCols = BF16 ? 64 : 32;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int b = 0; b < n / kCols; ++b) {
        if (row0 >= a.m || col + b * kCols >= a.N)
            break;  // nothing of the box, or of those after it, is in y
        if (lane == 0)  // the buffer's last store has read it
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // 16 bytes of the row, where the swizzle has them
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (BF16)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                        : "=r"(w[i])
                        : "f"(v[b * kCols + 8 * j + 2 * i + 1]), "f"(v[b * kCols + 8 * j + 2 * i]));
                else
                    w[i] = __float_as_uint(v[b * kCols + 4 * j + i]);
            }
            *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0)
            store_box(map, col + b * kCols, row0, smem_u32(buf));
    }
}

__device__ __forceinline__ void store_peer(uint32_t addr, uint32_t rank, float v)
{
    asm volatile("{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %0, %1;\n\tst.shared::cluster.f32 [p], %2;\n\t}" ::"r"(addr),
                 "r"(rank), "f"(v)
                 : "memory");
}

constexpr int kBox = 128 * 32, kBoxes = 8 * kBox;  // of y, one a warp

// S CTAs of a cluster share a tile along K.
template <int BN, int S>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const GemmArgs a, const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw,
                    const __grid_constant__ CUtensorMap ty)
{
    constexpr int WGC = BN / 2;     // columns of a group of four warps
    constexpr int kAccs = 512 / BN;  // accumulators in tensor memory
    constexpr uint32_t kStage = (uint32_t)(kXTile + BN * kTK);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    pdl_launch_dependents();
    // the 128-byte swizzle repeats every 1024 bytes: stages start on 1024
    uint8_t* const ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float* const red = reinterpret_cast<float*>(ring + (size_t)a.stages * kStage);  // S > 1: [S][BN / S][128]
    uint8_t* const boxes = reinterpret_cast<uint8_t*>(red);                         // S == 1
    GemmShared& sh = *reinterpret_cast<GemmShared*>(boxes + (S > 1 ? BN * 512 : kBoxes));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)blockIdx.x % S : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.done[s]), 1);
        }
        for (int b = 0; b < kAccs; ++b) {
            mbar_init(smem_u32(&sh.acc_empty[b]), 8);
        }
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (S > 1)
        cluster_sync();  // every CTA of the cluster has started
    const uint32_t tmem = sh.tmem;
    volatile int* const abort_flag = &sh.abort_flag;
    auto give_up = [&]() {
        atomicOr(&g_fp8_gemm_error, Q2K_ERR_BIT_WAIT_TIMEOUT);
        *abort_flag = 1;
    };
    const int tiles = a.tiles_m * a.tiles_n;
    const int tile0 = (int)blockIdx.x / S, step = (int)gridDim.x / S;
    const int k_first = rank * a.blocks / S, k_end = (rank + 1) * a.blocks / S;
    auto place = [&](int t, int& m0, int& n0) {
        const int per = kGroup * a.tiles_n, group = t / per, in = t - group * per;
        const int high = min(kGroup, a.tiles_m - group * kGroup);
        m0 = (group * kGroup + in % high) * kTM;
        n0 = in / high * BN;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp != 1) {
            if (lane == 0) {  // copies: of every third stage
                const uint64_t pol = l2_policy_evict_last();
                const int me = warp == 0 ? 0 : warp - 1;
                int slot = 0, use = 0, turn = 0, last_slot = -1, last_use = 0;
                bool ok = true;
                for (int t = tile0; t < tiles && ok; t += step) {
                    int m0, n0;
                    place(t, m0, n0);
                    for (int k = k_first; k < k_end; ++k) {
                        if (turn == me) {
                            if (use > 0 && !mbar_wait_near(smem_u32(&sh.done[slot]), (uint32_t)(use - 1) & 1u, abort_flag)) {
                                give_up();
                                ok = false;
                                break;
                            }
                            const uint32_t bar = smem_u32(&sh.full[slot]), dst = smem_u32(ring + (size_t)slot * kStage);
                            mbar_arrive_expect_tx(bar, kStage);
                            tma_load_2d(dst, &tx, k * kTK, m0, bar, pol);
                            tma_load_2d(dst + kXTile, &tw, k * kTK, n0, bar, pol);
                            last_slot = slot;
                            last_use = use;
                        }
                        if (++turn == 3)
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
        } else {  // MMAs
            constexpr uint32_t idesc = instr_desc_e4m3(BN);
            const uint32_t ring_at = smem_u32(ring);
            int slot = 0, use = 0, n = 0;
            bool ok = true;
            for (int t = tile0; t < tiles && ok; t += step)
                for (int k = k_first; k < k_end; ++k, ++n) {
                    const int b = n % kAccs;
                    const uint32_t s0 = uniform((uint32_t)slot), b0 = uniform((uint32_t)b);
                    const uint32_t sa = ring_at + s0 * kStage, d = tmem + b0 * BN;
                    if (!mbar_wait_near(smem_u32(&sh.full[slot]), (uint32_t)use & 1u, abort_flag) ||
                        (n >= kAccs && !mbar_wait_near(smem_u32(&sh.acc_empty[b]), (uint32_t)(n / kAccs - 1) & 1u, abort_flag)))
                        ok = false;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) {
                        if (lane == 0)
                            give_up();
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < kTK / 32; ++i)  // K = 32 an MMA: 32 bytes along the swizzled row
                            umma_e4m3(d, desc_at(sa + 32 * i), desc_at(sa + kXTile + 32 * i), idesc, i > 0);
                        // One commit, 115 cycles, tells both that the accumulator is full and that the stage is free.
                        // So there have to be as many stages as accumulators: block n + stages then waits for the
                        // accumulator of block n or a later one to be read back, hence until all who add have seen
                        // this stage's barrier turn; with fewer it could turn twice before they look.
                        umma_commit(smem_u32(&sh.done[0]) + 8 * s0);
                    }
                    __syncwarp();
                    if (++slot == a.stages) {
                        slot = 0;
                        ++use;
                    }
                }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int q = warp & 3, wg = (warp - 4) >> 2;
        const uint32_t t_addr = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(wg * WGC);
        int n = 0, slot = 0, use = 0;
        for (int t = tile0; t < tiles; t += step) {
            int m0, n0;
            place(t, m0, n0);
            const int row = m0 + 32 * q + lane, col = n0 + wg * WGC;
            const float* xs = a.x_scales + (int64_t)min(row, a.m - 1) * a.ld_xs;
            const float* ws = a.w_scales + (int64_t)(min(col, a.N - 1) / 128) * a.blocks;
            float acc[WGC];
#pragma unroll
            for (int i = 0; i < WGC; ++i)
                acc[i] = 0.f;
            // a block's scale, the next one's on its way
            float fx = k_first < k_end ? xs[k_first] : 0.f, fw = k_first < k_end ? ws[k_first] : 0.f;
            for (int k = k_first; k < k_end; ++k, ++n) {
                const int buf = n % kAccs;
                const float f = fx * fw;
                if (k + 1 < k_end) {
                    fx = xs[k + 1];
                    fw = ws[k + 1];
                }
                const bool ok = __all_sync(
                    0xffffffffu, mbar_wait_near(smem_u32(&sh.done[slot]), (uint32_t)use & 1u, abort_flag));
                if (!ok) {
                    if (lane == 0)
                        give_up();
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                // All columns at once as far as registers go, else 16 on their way while 16 are added up (with 32 they do
                // not suffice: 256 us for 8191 x 8192 x 4096 against 219).  The accumulator is free once the last have
                // landed.
                auto free_it = [&]() {
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&sh.acc_empty[buf]));
                };
                if constexpr (WGC <= 64) {
                    float v[WGC];
#pragma unroll
                    for (int c = 0; c < WGC; c += 16)
                        tmem_load16(t_addr + buf * BN + c, v + c);
                    settle(v);
                    free_it();
#pragma unroll
                    for (int c = 0; c < WGC; c += 16)
                        fma_pairs(acc + c, v + c, f);
                } else {
                    float v[2][16];
                    tmem_load16(t_addr + buf * BN, v[0]);
#pragma unroll
                    for (int c = 0; c < WGC; c += 16) {
                        settle(v[c / 16 & 1]);
                        if (c + 16 < WGC)
                            tmem_load16(t_addr + buf * BN + c + 16, v[(c / 16 + 1) & 1]);
                        else
                            free_it();
                        fma_pairs(acc + c, v[c / 16 & 1], f);
                    }
                }
                if (++slot == a.stages) {
                    slot = 0;
                    ++use;
                }
            }
            if constexpr (S == 1) {
                if (*abort_flag)
                    continue;
                if (a.bulk_store) {
                    uint8_t* const mine = boxes + (warp - 4) * kBox;
                    if (a.y_bf16)
                        store_boxes<WGC, true>(a, &ty, mine, m0 + 32 * q, col, acc);
                    else
                        store_boxes<WGC, false>(a, &ty, mine, m0 + 32 * q, col, acc);
                } else if (row < a.m) {
                    store_row<WGC>(a, row, col, acc);
                }
            } else {
                // slice r of the columns is added up and stored by CTA r
                constexpr int SC = WGC / S;
                const uint32_t at = smem_u32(red) + (uint32_t)(((rank * 2 + wg) * SC * 128 + 32 * q + lane) * 4);
#pragma unroll
                for (int i = 0; i < WGC; ++i)
                    store_peer(at + (uint32_t)(i % SC) * 512u, (uint32_t)(i / SC), acc[i]);
            }
        }
    }
    if (S == 1 && warp >= 4 && lane == 0)
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if constexpr (S > 1) {
        cluster_sync();
        if (warp >= 4) {
            constexpr int SC = WGC / S;
            const int q = warp & 3, wg = (warp - 4) >> 2;
            int m0, n0;
            place(tile0, m0, n0);
            const int row = m0 + 32 * q + lane;
            float sum[SC];
#pragma unroll
            for (int i = 0; i < SC; ++i) {
                sum[i] = red[(wg * SC + i) * 128 + 32 * q + lane];
#pragma unroll
                for (int r = 1; r < S; ++r)
                    sum[i] += red[((r * 2 + wg) * SC + i) * 128 + 32 * q + lane];
            }
            if (row < a.m && !*abort_flag)
                store_row<SC>(a, row, n0 + wg * WGC + rank * SC, sum);
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

PFN_cuTensorMapEncodeTiled_v12000 gemm_encoder()
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

// [rows, cols] values of `size` bytes, rows ld apart; a box is 128 bytes by box_rows, 128-byte swizzled, zeros past the
// edges (stores are cut there).
bool encode_boxes(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base, int64_t rows, int64_t cols, int64_t ld,
                  int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = gemm_encoder();
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(ld * size)};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows};
    const cuuint32_t ones[2] = {1, 1};
    return enc && enc(map, type, 2, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The shared memory that a block may have on the one kind of device that this library runs on.
constexpr size_t kSharedBytes = 232448;

constexpr size_t extra_bytes(int bn, int split)
{
    return 1024 + sizeof(GemmShared) + (split > 1 ? (size_t)bn * 512 : (size_t)kBoxes);
}

// Stages that fit into `bytes` of shared memory; 0 where they are fewer than the accumulators.
constexpr int stages_in(size_t bytes, int bn, int split)
{
    const size_t extra = extra_bytes(bn, split), n = bytes < extra ? 0 : (bytes - extra) / (size_t)(kXTile + bn * kTK);
    return n < (size_t)(512 / bn) ? 0 : n < (size_t)kMaxStages ? (int)n : kMaxStages;
}

template <int BN, int S>
cudaError_t launch_tiles(GemmArgs a, const Fp8Gemm& p, const DeviceInfo& di, cudaStream_t s)
{
    constexpr size_t kStage = kXTile + BN * kTK;
    auto* kernel = fp8_gemm_kernel<BN, S>;
    static std::atomic<unsigned long long> devs{0};
    cudaError_t e = allow_max_smem(kernel, devs);
    if (e != cudaSuccess)
        return e;
    a.tiles_m = (a.m + kTM - 1) / kTM;
    a.tiles_n = (a.N + BN - 1) / BN;
    static_assert(stages_in(kSharedBytes, BN, S) > 0, "fewer stages than accumulators");
    a.stages = stages_in((size_t)di.smem_optin, BN, S);
    if (a.stages == 0)
        return cudaErrorInvalidConfiguration;
    CUtensorMap tx{}, tw{}, ty{};
    if (!encode_boxes(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.x, p.m, p.K, p.ldx, kTM) ||
        !encode_boxes(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.W, p.N, p.K, p.K, BN))
        return cudaErrorInvalidValue;
    // (a tensor copy stores 16 bytes at a time: a row that ends inside them would have what follows it overwritten)
    a.bulk_store = S == 1 && a.align >= 16 && p.N * (p.y_bf16 ? 2 : 4) % 16 == 0 && p.ldy < ((int64_t)1 << 36);
    if (a.bulk_store && !(p.y_bf16 ? encode_boxes(&ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.y, p.m, p.N, p.ldy, 32)
                                   : encode_boxes(&ty, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, p.y, p.m, p.N, p.ldy, 32)))
        return cudaErrorInvalidValue;
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
    if (tiles * S > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(S > 1 ? tiles * S : std::min<int64_t>(tiles, di.sm_count)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = alone_on_sm(extra_bytes(BN, S) + (size_t)a.stages * kStage, (size_t)di.smem_optin);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, tx, tw, ty);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8Gemm& p, cudaStream_t s)
{
    if (fp8_stream_supported(p))
        return launch_fp8_gemm_stream(p, s);
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess)
        return e;
    GemmArgs a{};
    a.x_scales = p.x_scales;
    a.w_scales = p.w_scales;
    a.y = p.y;
    a.ld_xs = p.ld_xs;
    a.ldy = p.ldy;
    a.m = (int)p.m;
    a.N = (int)p.N;
    a.blocks = (int)((p.K + kTK - 1) / kTK);
    a.y_bf16 = p.y_bf16;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.y) | (uintptr_t)(p.ldy * (p.y_bf16 ? 2 : 4));
    a.align = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 1;
    // What each choice of tile and split takes, in cycles, as measured at 48 to 1024 rows of 512 to 16384 x 2048 to 4096:
    // once, and for each block of K of a tile.  (128 columns over 4 CTAs, 128 rows of 4096 x 4096: 8.4 us against 12.6
    // alone; 128 over 2, 5000 x 4112: 11.8 against 15.4; 64 over 2, 2048 x 2048: 5.9 against 6.7 for 128 over 4; 256
    // alone, 203 rows of 16384 x 4096: 19.6 against 24.0 for 128.)
    struct Option {
        int bn, split, once, block;
    };
    constexpr Option options[5] = {{256, 1, 5700, 800}, {128, 1, 6000, 540}, {128, 2, 9200, 560}, {128, 4, 11000, 330}, {64, 2, 7400, 475}};
    auto cost = [&](const Option& o) {
        const int64_t tiles = (int64_t)((a.m + kTM - 1) / kTM) * ((a.N + o.bn - 1) / o.bn);
        const int64_t at_once = o.split == 4 ? di.sm_count / 4 - 2 : di.sm_count / o.split;  // (some SMs are left out)
        const int64_t rounds = (tiles + at_once - 1) / at_once;
        return o.once + rounds * ((a.blocks + o.split - 1) / o.split) * o.block + (rounds - 1) * 2000;
    };
    int best = 0;
    for (int i = 1; i < 5; ++i)
        if (options[i].split <= a.blocks && cost(options[i]) < cost(options[best]))
            best = i;
    switch (best) {
    case 0: return launch_tiles<256, 1>(a, p, di, s);
    case 1: return launch_tiles<128, 1>(a, p, di, s);
    case 2: return launch_tiles<128, 2>(a, p, di, s);
    case 3: return launch_tiles<128, 4>(a, p, di, s);
    default: return launch_tiles<64, 2>(a, p, di, s);
    }
}

cudaError_t fp8_gemm_error_word(int32_t* out, bool clear)
{
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp8_gemm_error, sizeof(int));
    if (e != cudaSuccess)
        return e;
    *out = v;
    if (clear) {
        int z = 0;
        e = cudaMemcpyToSymbol(g_fp8_gemm_error, &z, sizeof(int));
    }
    return e;
}

}  // namespace q2k
