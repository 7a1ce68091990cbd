// C ABI entry points (include/q2k.h): argument validation before any CUDA
// call, then dispatch to the kernel translation units.  Validation mirrors
// the pages' `ensure!` checks that run before any launch
// (engram_v41/apply.rs `apply`, engram_v41.rs `rows_from_q2k`,
// moe_v41/init.rs `MoeV41::new`).
#include "../../include/q2k.h"
#include "q2k_common.cuh"
#include "q2k_internal.h"

#include <mutex>

namespace q2k {

namespace {
constexpr int kMaxDevices = 64;
DeviceInfo g_info[kMaxDevices];
bool g_info_ok[kMaxDevices];
std::mutex g_info_mu;
thread_local int t_last_cuda_error = 0;

int fail_cuda(cudaError_t e)
{
    t_last_cuda_error = (int)e;
    return Q2K_ERR_CUDA;
}
}  // namespace

cudaError_t device_info(DeviceInfo* out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(g_info_mu);
        if (g_info_ok[dev]) {
            *out = g_info[dev];
            return cudaSuccess;
        }
    }
    DeviceInfo d{};
    if ((e = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    if ((e = cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess)
        return e;
    if ((e = cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess)
        return e;
    if ((e = cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess)
        return e;
    std::lock_guard<std::mutex> lk(g_info_mu);
    g_info[dev] = d;
    g_info_ok[dev] = true;
    *out = d;
    return cudaSuccess;
}

}  // namespace q2k

using namespace q2k;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Device check: compute capability 10.3 (the library carries sm_103a code only).
int check_device()
{
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess)
        return fail_cuda(e);
    if (di.cc_major != 10 || di.cc_minor != 3)
        return Q2K_ERR_UNSUPPORTED;
    return Q2K_OK;
}

int finish(cudaError_t e) { return e == cudaSuccess ? Q2K_OK : fail_cuda(e); }

// Largest K the library accepts (weights rows up to 1 MiB of blocks).
constexpr int64_t kMaxK = 1 << 20;

// Cache slots are int32.
constexpr int64_t kMaxSlots = (int64_t)1 << 31;

bool type_ok(int t) { return t == Q2K_F32 || t == Q2K_BF16; }

// int32 arrays of na and nb entries share an address.
bool overlap(const int32_t* a, int64_t na, const int32_t* b, int64_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na > 0 && nb > 0 && x < y + (uintptr_t)nb * 4 && y < x + (uintptr_t)na * 4;
}

bool page_size_ok(int64_t p) { return p >= 16 && p <= 1024 && (p & (p - 1)) == 0; }

bool cache_ok(int64_t n_pages, int64_t page_size, int64_t page_stride, int64_t Hkv, int64_t D)
{
    return page_size_ok(page_size) && n_pages >= 1 && n_pages <= kMaxSlots / page_size &&
           page_stride >= Hkv * page_size * D && page_stride % 8 == 0 && page_stride < ((int64_t)1 << 36);
}

int64_t fp8_blocks(int64_t K) { return (K + 127) / 128; }

bool fp8_moe_shape_ok(int64_t m, int64_t topk, int64_t dim, int64_t inter)
{
    return m >= 0 && m <= 128 && topk >= 1 && topk <= 32 && m * topk <= 1024 && dim >= 16 && dim <= 16384 &&
           dim % 16 == 0 && inter >= 16 && inter <= 16384 && inter % 16 == 0;
}

bool attn_heads_ok(int64_t Hq, int64_t Hkv, int64_t D)
{
    return Hkv >= 1 && Hkv <= 4096 && Hq >= Hkv && Hq % Hkv == 0 && Hq / Hkv <= 128 && D >= 16 && D <= 128 && D % 16 == 0;
}

}  // namespace

extern "C" {

size_t q2k_row_bytes(int64_t K)
{
    if (K <= 0 || K % kBlockWeights)
        return 0;
    return (size_t)(K / kBlockWeights) * kBlockBytes;
}

size_t q3k_row_bytes(int64_t K)
{
    if (K <= 0 || K % kBlockWeights)
        return 0;
    return (size_t)(K / kBlockWeights) * 110;
}

size_t q8_1_row_bytes(int64_t K)
{
    if (K <= 0 || K % kQ8Values)
        return 0;
    return (size_t)(K / kQ8Values) * kQ8Bytes;
}

const char* q2k_status_string(int status)
{
    switch (status) {
    case Q2K_OK: return "ok";
    case Q2K_ERR_NULL_ARG: return "null argument";
    case Q2K_ERR_BAD_SHAPE: return "bad shape";
    case Q2K_ERR_MISALIGNED: return "misaligned pointer";
    case Q2K_ERR_CUDA: return "cuda runtime error";
    case Q2K_ERR_UNSUPPORTED: return "unsupported device (needs compute capability 10.3)";
    case Q2K_ERR_WORKSPACE: return "workspace missing or too small";
    default: return "unknown status";
    }
}

int q2k_last_cuda_error(void) { return t_last_cuda_error; }

int q2k_device_error(int32_t* host_out, int clear)
{
    if (!host_out)
        return Q2K_ERR_NULL_ARG;
    int32_t a = 0, b = 0, c = 0, d = 0, q = 0, o = 0, mq = 0, q3t = 0, at = 0, fs = 0, fg = 0;
    cudaError_t e = mv_error_word(&a, clear != 0);
    if (e == cudaSuccess)
        e = m1_error_word(&o, clear != 0);
    if (e == cudaSuccess)
        e = mmq_error_word(&mq, clear != 0);
    if (e == cudaSuccess)
        e = gemm_error_word(&b, clear != 0);
    if (e == cudaSuccess)
        e = mt_error_word(&c, clear != 0);
    if (e == cudaSuccess)
        e = umma_error_word(&d, clear != 0);
    if (e == cudaSuccess)
        e = q3_error_word(&q, clear != 0);
    if (e == cudaSuccess)
        e = q3mt_error_word(&q3t, clear != 0);
    if (e == cudaSuccess)
        e = attn_error_word(&at, clear != 0);
    if (e == cudaSuccess)
        e = fp8_stream_error_word(&fs, clear != 0);
    if (e == cudaSuccess)
        e = fp8_gemm_error_word(&fg, clear != 0);
    if (e != cudaSuccess)
        return fail_cuda(e);
    *host_out = a | b | c | d | q | o | mq | q3t | at | fs | fg;
    return Q2K_OK;
}

int q2k_dequant_rows(const void* table, int64_t n_table_rows, int64_t K, const int32_t* ids, int64_t n_rows,
                     uint16_t* out_bf16, int32_t* err_flag, q2k_stream_t stream)
{
    if (!table || !out_bf16)
        return Q2K_ERR_NULL_ARG;
    if (K <= 0 || K % kBlockWeights || K > kMaxK || n_rows < 0 || n_table_rows <= 0)
        return Q2K_ERR_BAD_SHAPE;
    if (!ids && n_rows > n_table_rows)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(table, 4) || !aligned(out_bf16, 2) || (ids && !aligned(ids, 4)) || (err_flag && !aligned(err_flag, 4)))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (n_rows == 0)
        return Q2K_OK;
    return finish(launch_dequant_rows(table, n_table_rows, K, ids, n_rows, out_bf16, err_flag,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

int q2k_engram_hash(const int64_t* token_map, int64_t vocab, int64_t* cache, int64_t max_seq,
                    const uint32_t* input_ids, int64_t seqlen, int64_t start_pos, int64_t max_ngram,
                    int64_t n_layers, int64_t n_heads, const int64_t* multipliers, const int64_t* primes,
                    const int64_t* offsets, int64_t pad_id, int64_t* out, int32_t* layer_ids,
                    int64_t layer_index, int32_t* err_flag, q2k_stream_t stream)
{
    if (!token_map || !cache || (seqlen > 0 && !input_ids) || !multipliers || !primes || !offsets ||
        (seqlen > 0 && !out))
        return Q2K_ERR_NULL_ARG;
    if (vocab <= 0 || max_seq <= 0 || seqlen < 0 || start_pos < 0 || start_pos + seqlen > max_seq ||
        max_ngram < 2 || max_ngram > 16 || n_layers < 1 || n_layers > 1024 || n_heads < 1 || n_heads > 1024 ||
        (layer_ids && (layer_index < 0 || layer_index >= n_layers)))
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(token_map, 8) || !aligned(cache, 8) || !aligned(input_ids, 4) || !aligned(multipliers, 8) ||
        !aligned(primes, 8) || !aligned(offsets, 8) || !aligned(out, 8) || !aligned(layer_ids, 4) ||
        !aligned(err_flag, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (seqlen == 0)
        return Q2K_OK;
    return finish(launch_engram_hash(token_map, vocab, cache, input_ids, seqlen, start_pos, (int)max_ngram,
                                     (int)n_layers, (int)n_heads, multipliers, primes, offsets, pad_id, out, layer_ids,
                                     (int)layer_index, err_flag, reinterpret_cast<cudaStream_t>(stream)));
}

int q2k_engram_gate(float* streams, const float* kv, int64_t ld_kv, const float* qk, int64_t tokens, int64_t hc,
                    int64_t dim, float eps, float* gates, q2k_stream_t stream)
{
    if (tokens > 0 && (!streams || !kv || !qk))
        return Q2K_ERR_NULL_ARG;
    if (tokens < 0 || tokens > (1 << 30) || hc < 1 || hc > 4 || dim < 1 || dim > kMaxK || ld_kv < (hc + 1) * dim ||
        !(eps >= 0.f) || eps > 3.0e38f)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(streams, 4) || !aligned(kv, 4) || !aligned(qk, 4) || (gates && !aligned(gates, 4)))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (tokens == 0)
        return Q2K_OK;
    return finish(launch_engram_gate(streams, kv, ld_kv, qk, tokens, (int)hc, (int)dim, eps, gates,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

int q8_1_quantize_rows(const uint16_t* x_bf16, int64_t m, int64_t K, int64_t ldx, void* out_q8_1,
                       q2k_stream_t stream)
{
    if (!x_bf16 || !out_q8_1)
        return Q2K_ERR_NULL_ARG;
    if (m < 0 || K <= 0 || K % kQ8Values || ldx < K || K > kMaxK)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(x_bf16, 2) || !aligned(out_q8_1, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (m == 0)
        return Q2K_OK;
    return finish(launch_q8_1_quantize(x_bf16, m, K, ldx, out_q8_1, reinterpret_cast<cudaStream_t>(stream)));
}

int q2k_gemv_bf16(const void* W, int64_t N, int64_t K, const uint16_t* x, int64_t m, int64_t ldx, float* y,
                  int64_t ldy, q2k_stream_t stream)
{
    if (!W || !x || !y)
        return Q2K_ERR_NULL_ARG;
    if (N <= 0 || K <= 0 || K % kBlockWeights || K > kMaxK || m < 1 || m > 8 || ldx < K || ldy < N)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(W, 4) || !aligned(x, 2) || !aligned(y, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    MvProblem p{};
    p.act = ACT_BF16;
    p.m = (int)m;
    p.K = K;
    p.n_seg = 1;
    p.W[0] = W;
    p.N[0] = N;
    p.y[0] = y;
    p.ldy[0] = ldy;
    p.x = x;
    p.x_tok_stride = ldx * 2;
    return finish(launch_mv(p, reinterpret_cast<cudaStream_t>(stream)));
}

int q2k_mmvq_q8_1(const void* W, int64_t N, int64_t K, const void* xq, int64_t m, float* y, int64_t ldy,
                  q2k_stream_t stream)
{
    if (!W || !xq || !y)
        return Q2K_ERR_NULL_ARG;
    if (N <= 0 || K <= 0 || K % kBlockWeights || K > kMaxK || m < 1 || m > 8 || ldy < N)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(W, 4) || !aligned(xq, 4) || !aligned(y, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    MvProblem p{};
    p.act = ACT_Q8;
    p.m = (int)m;
    p.K = K;
    p.n_seg = 1;
    p.W[0] = W;
    p.N[0] = N;
    p.y[0] = y;
    p.ldy[0] = ldy;
    p.x = xq;
    p.x_tok_stride = (int64_t)q8_1_row_bytes(K);
    return finish(launch_mv(p, reinterpret_cast<cudaStream_t>(stream)));
}

int q2k_mmvq_pair(const void* Wa, int64_t Na, float* ya, const void* Wb, int64_t Nb, float* yb, int64_t K,
                  const void* xq, int64_t m, q2k_stream_t stream)
{
    if (!Wa || !Wb || !ya || !yb || !xq)
        return Q2K_ERR_NULL_ARG;
    if (Na <= 0 || Nb <= 0 || K <= 0 || K % kBlockWeights || K > kMaxK || m < 1 || m > 8)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(Wa, 4) || !aligned(Wb, 4) || !aligned(ya, 4) || !aligned(yb, 4) || !aligned(xq, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    MvProblem p{};
    p.act = ACT_Q8;
    p.m = (int)m;
    p.K = K;
    p.n_seg = 2;
    p.W[0] = Wa;
    p.W[1] = Wb;
    p.N[0] = Na;
    p.N[1] = Nb;
    p.y[0] = ya;
    p.y[1] = yb;
    p.ldy[0] = Na;
    p.ldy[1] = Nb;
    p.x = xq;
    p.x_tok_stride = (int64_t)q8_1_row_bytes(K);
    return finish(launch_mv(p, reinterpret_cast<cudaStream_t>(stream)));
}

int q2k_mmvq_pair_bf16(const void* Wa, int64_t Na, float* ya, const void* Wb, int64_t Nb, float* yb, int64_t K,
                       const uint16_t* x_bf16, int64_t m, void* xq_out, q2k_stream_t stream)
{
    if (!Wa || !Wb || !ya || !yb || !x_bf16 || !xq_out)
        return Q2K_ERR_NULL_ARG;
    if (Na <= 0 || Nb <= 0 || K <= 0 || K % kBlockWeights || K > kMaxK || m < 1 || m > 8)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(Wa, 4) || !aligned(Wb, 4) || !aligned(ya, 4) || !aligned(yb, 4) || !aligned(x_bf16, 2) ||
        !aligned(xq_out, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    MvProblem p{};
    p.act = ACT_Q8;
    p.m = (int)m;
    p.K = K;
    p.n_seg = 2;
    p.W[0] = Wa;
    p.W[1] = Wb;
    p.N[0] = Na;
    p.N[1] = Nb;
    p.y[0] = ya;
    p.y[1] = yb;
    p.ldy[0] = Na;
    p.ldy[1] = Nb;
    p.x_tok_stride = (int64_t)q8_1_row_bytes(K);
    p.x = xq_out;
    if (m == 1 && aligned(x_bf16, 16) && !m1_supported(p)) {
        // one launch: every CTA encodes the row, the first also stores it.
        // (Where the row-team kernel takes the pair, a separate encoding
        // launch ahead of it measured faster: 4.5 vs 6.0 us at cfg2.)
        p.x = x_bf16;
        p.x_prep = 1;
        p.x_out = xq_out;
        return finish(launch_mv(p, s));
    }
    cudaError_t e = launch_q8_1_quantize(x_bf16, m, K, K, xq_out, s);
    if (e != cudaSuccess)
        return fail_cuda(e);
    p.x = xq_out;
    return finish(launch_mv(p, s));
}

int q2k_mmvq_grouped(const void* W, int64_t groups, int64_t rows_per_group, int64_t K_group, const void* xq,
                     int64_t m, float* y, q2k_stream_t stream)
{
    if (!W || !xq || !y)
        return Q2K_ERR_NULL_ARG;
    if (groups <= 0 || groups > 4096 || rows_per_group <= 0 || K_group <= 0 || K_group % kBlockWeights ||
        K_group > kMaxK || m < 1 || m > 8 || groups * rows_per_group > (1 << 30))
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(W, 4) || !aligned(xq, 4) || !aligned(y, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    MvProblem p{};
    p.act = ACT_Q8;
    p.m = (int)m;
    p.K = K_group;
    p.n_seg = (int)groups;
    p.W[0] = W;  // group g: rows g*rows_per_group.. of W
    p.w_seg_stride = rows_per_group * (int64_t)q2k_row_bytes(K_group);
    p.N[0] = rows_per_group;
    p.y_exp = y;  // y[t, g*rows_per_group + r]
    p.ldy_exp = groups * rows_per_group;
    p.seg_major = 1;  // each group gets CTAs of its own, its slice staged once
    p.x = xq;
    p.x_tok_stride = (int64_t)q8_1_row_bytes(groups * K_group);
    p.x_seg_stride = (int64_t)q8_1_row_bytes(K_group);  // group g's blocks of each token's row
    return finish(launch_mv(p, reinterpret_cast<cudaStream_t>(stream)));
}

int q2k_mmvq_experts(const void* const* W_table, int64_t n_mat, int64_t N, int64_t K, const void* xq,
                     int x_per_matrix, float* y, const float* route_w, float* y_sum, q2k_stream_t stream)
{
    if (!W_table || !xq || (!y && !y_sum) || (y_sum && !route_w))
        return Q2K_ERR_NULL_ARG;
    if (n_mat <= 0 || n_mat > 4096 || N <= 0 || K <= 0 || K % kBlockWeights || K > kMaxK ||
        (x_per_matrix != 0 && x_per_matrix != 1))
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(W_table, 8) || !aligned(xq, 4) || (y && !aligned(y, 4)) || (route_w && !aligned(route_w, 4)) ||
        (y_sum && !aligned(y_sum, 4)))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    MvProblem p{};
    p.act = ACT_Q8;
    p.m = 1;
    p.K = K;
    p.n_seg = (int)n_mat;
    p.W_table = W_table;
    p.N[0] = N;
    p.y_exp = y;
    p.route_w = route_w;
    p.y_sum = y_sum;
    p.x = xq;
    p.x_tok_stride = (int64_t)q8_1_row_bytes(K);
    p.x_seg_stride = x_per_matrix ? (int64_t)q8_1_row_bytes(K) : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (y) {
        // each matrix gets CTAs of its own (full reduction units, its input
        // row staged once); the route-weighted sum, if asked for, is a
        // second pass over y
        p.seg_major = 1;
        p.y_sum = nullptr;
        cudaError_t e = launch_mv(p, s);
        if (e != cudaSuccess || !y_sum)
            return e != cudaSuccess ? fail_cuda(e) : finish(e);
        return finish(launch_expert_sum(y, route_w, n_mat, N, y_sum, s));
    }
    // the fused sum keeps every matrix's partial sums of a CTA's rows in
    // shared memory: refuse, before any launch, a problem whose partials do
    // not fit (per-matrix outputs in y are then the workspace it needs)
    if (!mv_plan_ok(p))
        return Q2K_ERR_WORKSPACE;
    return finish(launch_mv(p, s));
}

int q3k_mmvq_q8_1(const void* W, int64_t N, int64_t K, const void* xq, int64_t m, float* y, int64_t ldy,
                  q2k_stream_t stream)
{
    if (!W || !xq || !y)
        return Q2K_ERR_NULL_ARG;
    if (N <= 0 || N > (1 << 30) || K <= 0 || K % kBlockWeights || K > kMaxK || m < 1 || m > 8 || ldy < N)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(W, 4) || !aligned(xq, 4) || !aligned(y, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    Q3Problem p{};
    p.W = W;
    p.n_seg = 1;
    p.N = N;
    p.K = K;
    p.m = (int)m;
    p.x = xq;
    p.x_tok_stride = (int64_t)q8_1_row_bytes(K);
    p.y = y;
    p.ldy = ldy;
    return finish(launch_q3k_mv(p, reinterpret_cast<cudaStream_t>(stream)));
}

int q3k_mmvq_experts(const void* const* W_table, int64_t n_mat, int64_t N, int64_t K, const void* xq,
                     int x_per_matrix, float* y, const float* route_w, float* y_sum, q2k_stream_t stream)
{
    if (!W_table || !xq || !y || (y_sum && !route_w))
        return Q2K_ERR_NULL_ARG;
    if (n_mat <= 0 || n_mat > 4096 || N <= 0 || N > (1 << 30) || K <= 0 || K % kBlockWeights || K > kMaxK ||
        (x_per_matrix != 0 && x_per_matrix != 1))
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(W_table, 8) || !aligned(xq, 4) || !aligned(y, 4) || (route_w && !aligned(route_w, 4)) ||
        (y_sum && !aligned(y_sum, 4)))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    Q3Problem p{};
    p.W_table = W_table;
    p.n_seg = (int)n_mat;
    p.N = N;
    p.K = K;
    p.m = 1;
    p.x = xq;
    p.x_tok_stride = (int64_t)q8_1_row_bytes(K);
    p.x_seg_stride = x_per_matrix ? (int64_t)q8_1_row_bytes(K) : 0;
    p.y = y;
    p.ldy = N;
    p.y_seg_stride = N;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_q3k_mv(p, s);
    if (e != cudaSuccess || !y_sum)
        return e != cudaSuccess ? fail_cuda(e) : finish(e);
    return finish(launch_expert_sum(y, route_w, n_mat, N, y_sum, s));
}

int swiglu_q8_1_rows(const float* gate_up, int64_t E, int64_t N, void* h_q8, uint16_t* h_bf16, q2k_stream_t stream)
{
    if (!gate_up || !h_q8)
        return Q2K_ERR_NULL_ARG;
    if (E <= 0 || N <= 0 || N % kQ8Values || N > kMaxK)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(gate_up, 4) || !aligned(h_q8, 4) || (h_bf16 && !aligned(h_bf16, 2)))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    return finish(launch_swiglu_q8_1(gate_up, E, N, h_q8, h_bf16, reinterpret_cast<cudaStream_t>(stream)));
}

static size_t round256(size_t v) { return (v + 255) / 256 * 256; }

size_t q2k_moe_m1_workspace_bytes(int64_t E, int64_t dim, int64_t inter)
{
    if (E <= 0 || dim <= 0 || inter <= 0 || dim % kBlockWeights || inter % kBlockWeights)
        return 0;
    return round256(q8_1_row_bytes(dim)) + round256((size_t)2 * E * inter * sizeof(float)) +
           round256((size_t)E * q8_1_row_bytes(inter)) + round256((size_t)E * dim * sizeof(float));
}

int q2k_moe_m1(const void* const* ptrs, int64_t E, int64_t dim, int64_t inter, const uint16_t* x_bf16,
               const float* route_w, float* y, void* workspace, size_t workspace_bytes, q2k_stream_t stream)
{
    if (!ptrs || !x_bf16 || !route_w || !y)
        return Q2K_ERR_NULL_ARG;
    if (E <= 0 || E > 1024 || dim <= 0 || inter <= 0 || dim % kBlockWeights || inter % kBlockWeights ||
        dim > kMaxK || inter > kMaxK)
        return Q2K_ERR_BAD_SHAPE;
    const size_t need = q2k_moe_m1_workspace_bytes(E, dim, inter);
    if (!workspace || workspace_bytes < need)
        return Q2K_ERR_WORKSPACE;
    if (!aligned(ptrs, 8) || !aligned(x_bf16, 2) || !aligned(route_w, 4) || !aligned(y, 4) || !aligned(workspace, 256))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    void* xq = ws;
    float* gate_up = reinterpret_cast<float*>(ws + round256(q8_1_row_bytes(dim)));
    void* h_q8 = ws + round256(q8_1_row_bytes(dim)) + round256((size_t)2 * E * inter * sizeof(float));
    float* down_out = reinterpret_cast<float*>(static_cast<uint8_t*>(h_q8) + round256((size_t)E * q8_1_row_bytes(inter)));
    // A 16-byte aligned x is quantised inside the gate/up GEMV (each CTA
    // encodes it; the first also stores it in the workspace), and SwiGLU +
    // q8_1 of h run inside the down GEMV the same way: three launches, the
    // same bits as the five separate steps.
    const bool fuse_x = aligned(x_bf16, 16);
    cudaError_t e = cudaSuccess;
    if (!fuse_x && (e = launch_q8_1_quantize(x_bf16, 1, dim, dim, xq, s)) != cudaSuccess)
        return fail_cuda(e);
    MvProblem p{};
    p.act = ACT_Q8;
    p.m = 1;
    p.K = dim;
    p.n_seg = (int)(2 * E);
    p.W_table = ptrs;
    p.N[0] = inter;
    p.y_exp = gate_up;
    p.seg_major = 1;  // each gate/up matrix gets CTAs of its own
    p.x = fuse_x ? static_cast<const void*>(x_bf16) : xq;
    p.x_tok_stride = (int64_t)q8_1_row_bytes(dim);
    p.x_seg_stride = 0;
    if (fuse_x) {
        p.x_prep = 1;
        p.x_out = xq;
    }
    if ((e = launch_mv(p, s)) != cudaSuccess)
        return fail_cuda(e);
    MvProblem d{};
    d.act = ACT_Q8;
    d.m = 1;
    d.K = inter;
    d.n_seg = (int)E;
    d.W_table = ptrs + 2 * E;
    d.N[0] = dim;
    d.y_exp = down_out;  // one expert per CTA, then the route-weighted sum
    d.seg_major = 1;
    d.x = h_q8;
    d.x_tok_stride = (int64_t)q8_1_row_bytes(inter);
    d.x_seg_stride = (int64_t)q8_1_row_bytes(inter);
    d.x_prep = 2;  // h = SwiGLU(gate, up) -> q8_1 per CTA, also stored in h_q8
    d.gu = gate_up;
    d.gu_E = E;
    d.x_out = h_q8;
    if ((e = launch_mv(d, s)) != cudaSuccess)
        return fail_cuda(e);
    return finish(launch_expert_sum(down_out, route_w, E, dim, y, s));
}

size_t q2k_mmq_q8_1_workspace_bytes(int64_t m, int64_t K)
{
    if (m < 1 || m > (1 << 24) || K <= 0 || K % 1024 || K > kMaxK)
        return 0;
    return mmq_q8_1_workspace(m, K);
}

int q2k_mmq_bf16(const void* W, int64_t N, int64_t K, const uint16_t* x, int64_t m, int64_t ldx, float* y,
                 int64_t ldy, q2k_stream_t stream)
{
    if (!W || !x || !y)
        return Q2K_ERR_NULL_ARG;
    if (N < 1 || N > (1 << 30) || K <= 0 || K % 1024 || K > kMaxK || m < 1 || m > (1 << 24) || ldx < K || ldx % 8 ||
        ldy < N)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(W, 16) || !aligned(x, 16) || !aligned(y, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (!mmq_supported(m, N, K))
        return Q2K_ERR_UNSUPPORTED;  // no tensor-map encoder in this driver
    return finish(launch_mmq_bf16(W, N, K, x, m, ldx, y, ldy, reinterpret_cast<cudaStream_t>(stream)));
}

int q2k_mmq_q8_1(const void* W, int64_t N, int64_t K, const void* xq, int64_t m, float* y, int64_t ldy,
                 void* workspace, size_t workspace_bytes, q2k_stream_t stream)
{
    if (!W || !xq || !y)
        return Q2K_ERR_NULL_ARG;
    if (N < 1 || N > (1 << 30) || K <= 0 || K % 1024 || K > kMaxK || m < 1 || m > (1 << 24) || ldy < N)
        return Q2K_ERR_BAD_SHAPE;
    if (!workspace || workspace_bytes < q2k_mmq_q8_1_workspace_bytes(m, K))
        return Q2K_ERR_WORKSPACE;
    if (!aligned(W, 16) || !aligned(xq, 4) || !aligned(y, 4) || !aligned(workspace, 16))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (!mmq_supported(m, N, K))
        return Q2K_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint16_t* xb = static_cast<uint16_t*>(workspace);
    cudaError_t e = launch_q8_1_to_bf16(xq, m, K, xb, s);
    if (e != cudaSuccess)
        return fail_cuda(e);
    return finish(launch_mmq_bf16(W, N, K, xb, m, K, y, ldy, s));
}

int dense_gemm_bf16(const uint16_t* x, int64_t m, int64_t K, int64_t ldx, const uint16_t* W, int64_t N, float* y,
                    int64_t ldy, q2k_stream_t stream)
{
    if (!x || !W || !y)
        return Q2K_ERR_NULL_ARG;
    if (m < 1 || K <= 0 || K % 8 || N <= 0 || ldx < K || ldx % 8 || ldy < N || K > (1 << 30) / 2 ||
        N > (1 << 30) || m > (1 << 24))
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(y, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    return finish(launch_dense_gemm(x, m, K, ldx, W, N, y, ldy, reinterpret_cast<cudaStream_t>(stream)));
}

int kv_page_plan(const int32_t* ctx_lens, const int32_t* new_lens, int64_t n_req, int64_t page_size,
                 const int32_t* free_pages, int64_t n_free, const int32_t* free_head, int32_t* block_table,
                 int64_t max_pages, int64_t ld_table, int32_t* cu_q, int32_t* seq_lens, int32_t* positions, int32_t* token_req,
                 int32_t* slot_map, int64_t max_tokens, int32_t* free_head_out, int32_t* err_flag,
                 q2k_stream_t stream)
{
    if (!ctx_lens || !new_lens || (n_free > 0 && !free_pages) || !block_table || !cu_q || !seq_lens ||
        (max_tokens > 0 && (!positions || !token_req || !slot_map)) || !free_head_out)
        return Q2K_ERR_NULL_ARG;
    if (n_req < 1 || n_req > 16384 || !page_size_ok(page_size) || n_free < 0 || n_free > kMaxSlots || max_pages < 1 ||
        max_pages > kMaxSlots || ld_table < max_pages || max_tokens < 0 || max_tokens > (1 << 30) || free_head == free_head_out)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) || !aligned(free_head, 4) ||
        !aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(seq_lens, 4) || !aligned(positions, 4) ||
        !aligned(token_req, 4) || !aligned(slot_map, 4) || !aligned(free_head_out, 4) || !aligned(err_flag, 4))
        return Q2K_ERR_MISALIGNED;
    // every block reads the inputs, at any time: none may be written meanwhile
    const struct {
        const int32_t* p;
        int64_t n;
    } in[] = {{ctx_lens, n_req}, {new_lens, n_req}, {free_pages, n_free}, {free_head, 1}},
      out[] = {{cu_q, n_req + 1},     {seq_lens, n_req},      {positions, max_tokens}, {token_req, max_tokens},
               {slot_map, max_tokens}, {free_head_out, 1}, {err_flag, 1}};
    for (const auto& i : in)
        for (const auto& o : out)
            if (overlap(i.p, i.n, o.p, o.n))
                return Q2K_ERR_BAD_SHAPE;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    PagePlan p{};
    p.ctx_lens = ctx_lens;
    p.new_lens = new_lens;
    p.n_req = n_req;
    p.page_size = page_size;
    p.free_pages = free_pages;
    p.n_free = n_free;
    p.free_head = free_head;
    p.block_table = block_table;
    p.max_pages = max_pages;
    p.ld_table = ld_table;
    p.cu_q = cu_q;
    p.seq_lens = seq_lens;
    p.positions = positions;
    p.token_req = token_req;
    p.slot_map = slot_map;
    p.max_tokens = max_tokens;
    p.free_head_out = free_head_out;
    p.err_flag = err_flag;
    return finish(launch_kv_page_plan(p, reinterpret_cast<cudaStream_t>(stream)));
}

int kv_rope_store(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v, int x_type,
                  int64_t T, int64_t Hq, int64_t Hkv, int64_t D, const int32_t* positions, int64_t n_axes,
                  const int32_t* sections, const float* inv_freq, int64_t rot, int interleaved,
                  const int32_t* slot_map, uint16_t* q_out, int64_t ld_qo, uint16_t* k_cache, uint16_t* v_cache,
                  int64_t n_pages, int64_t page_size, int64_t page_stride, int32_t* err_flag, q2k_stream_t stream)
{
    if (!sections || (!q) != (!q_out) ||
        (T > 0 && (!k || !v || !slot_map || !k_cache || !v_cache || (rot > 0 && (!positions || !inv_freq)))))
        return Q2K_ERR_NULL_ARG;
    if (!type_ok(x_type) || T < 0 || T > (1 << 30) || Hkv < 1 || Hkv > 4096 || (q && (Hq < 1 || Hq > 4096)) || D < 1 ||
        D > 512 || rot < 0 || rot > D || rot % 2 || n_axes < 1 || n_axes > 3 || (interleaved != 0 && interleaved != 1) ||
        ld_k < Hkv * D || ld_v < Hkv * D || (q && (ld_q < Hq * D || ld_qo < Hq * D)) ||
        !cache_ok(n_pages, page_size, page_stride, Hkv, D))
        return Q2K_ERR_BAD_SHAPE;
    int64_t pairs = 0;
    for (int64_t i = 0; i < n_axes; ++i) {
        if (sections[i] < 0)
            return Q2K_ERR_BAD_SHAPE;
        pairs += sections[i];
    }
    if (pairs != rot / 2)
        return Q2K_ERR_BAD_SHAPE;
    const uintptr_t es = x_type == Q2K_BF16 ? 2 : 4;
    if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(positions, 4) || !aligned(inv_freq, 4) ||
        !aligned(slot_map, 4) || !aligned(q_out, 2) || !aligned(k_cache, 2) || !aligned(v_cache, 2) ||
        !aligned(err_flag, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (T == 0)
        return Q2K_OK;
    RopeStore p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.ld_q = ld_q;
    p.ld_k = ld_k;
    p.ld_v = ld_v;
    p.x_bf16 = x_type == Q2K_BF16;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.positions = positions;
    for (int64_t i = 0; i < n_axes; ++i)
        p.sections[i] = sections[i];
    p.inv_freq = inv_freq;
    p.rot = rot;
    p.interleaved = interleaved;
    p.slot_map = slot_map;
    p.q_out = q_out;
    p.ld_qo = ld_qo;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.n_pages = n_pages;
    p.page_size = page_size;
    p.page_stride = page_stride;
    p.err_flag = err_flag;
    return finish(launch_kv_rope_store(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kv_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D)
{
    if (T < 0 || T > (1 << 24) || !attn_heads_ok(Hq, Hkv, D))
        return 0;
    return kv_attention_workspace(T, Hq, Hkv, D);
}

int kv_attention_bf16(const uint16_t* q, int64_t ld_q, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                      const uint16_t* k_cache, const uint16_t* v_cache, int64_t n_pages, int64_t page_size,
                      int64_t page_stride, const int32_t* block_table, int64_t max_pages, int64_t ld_table,
                      const int32_t* cu_q, const int32_t* seq_lens, int64_t n_req, float scale, int64_t window,
                      uint16_t* out, int64_t ld_o, float* lse, void* workspace, size_t workspace_bytes, q2k_stream_t stream)
{
    if ((T != 0 && (!q || !out || !k_cache || !v_cache)) || (T != 0 && n_req != 0 && (!block_table || !cu_q || !seq_lens)))
        return Q2K_ERR_NULL_ARG;
    if (T < 0 || T > (1 << 24) || !attn_heads_ok(Hq, Hkv, D) || ld_q < Hq * D || ld_q % 8 || ld_o < Hq * D ||
        !cache_ok(n_pages, page_size, page_stride, Hkv, D) || max_pages < 1 || max_pages > kMaxSlots || ld_table < max_pages || n_req < 0 ||
        n_req > 16384 || !(scale > 0.f) || scale > 3.0e38f || window < 0)
        return Q2K_ERR_BAD_SHAPE;
    if (T != 0 && (!workspace || workspace_bytes < kv_attention_workspace_bytes(T, Hq, Hkv, D)))
        return Q2K_ERR_WORKSPACE;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_table, 4) ||
        !aligned(cu_q, 4) || !aligned(seq_lens, 4) || !aligned(out, 2) || !aligned(lse, 4) || !aligned(workspace, 32))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (T == 0 || n_req == 0)
        return Q2K_OK;
    if (!attn_supported())
        return Q2K_ERR_UNSUPPORTED;  // no tensor-map encoder in this driver
    AttnProblem p{};
    p.q = q;
    p.ld_q = ld_q;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.n_pages = n_pages;
    p.page_size = page_size;
    p.page_stride = page_stride;
    p.block_table = block_table;
    p.max_pages = max_pages;
    p.ld_table = ld_table;
    p.cu_q = cu_q;
    p.seq_lens = seq_lens;
    p.n_req = n_req;
    p.scale = scale;
    p.window = window;
    p.out = out;
    p.ld_o = ld_o;
    p.lse = lse;
    p.workspace = workspace;
    return finish(launch_kv_attention(p, reinterpret_cast<cudaStream_t>(stream)));
}

int norm_gate_residual(const void* y, int y_type, int64_t ld_y, const float* post_w, const void* gate,
                       int64_t ld_gate, const void* residual, int stream_type, int64_t ld_res, float alpha,
                       const float* pre_w, float eps, int64_t T, int64_t dim, void* residual_out, int64_t ld_ro,
                       uint16_t* out, int64_t ld_out, void* out_q8, q2k_stream_t stream)
{
    if (T != 0 && (!residual || !pre_w || (!out && !out_q8 && !residual_out) || (!y && (post_w || gate))))
        return Q2K_ERR_NULL_ARG;
    if (!type_ok(y_type) || !type_ok(stream_type) || T < 0 || T > (1 << 30) || dim < 1 || dim > 32768 ||
        (y && ld_y < dim) || (gate && ld_gate != 0 && ld_gate < dim) || ld_res < dim ||
        (residual_out && ld_ro < dim) || (out && ld_out < dim) || (out_q8 && dim % kQ8Values) || !(eps >= 0.f) ||
        eps > 3.0e38f || !(alpha >= -3.0e38f && alpha <= 3.0e38f))
        return Q2K_ERR_BAD_SHAPE;
    const uintptr_t ys = y_type == Q2K_BF16 ? 2 : 4, ss = stream_type == Q2K_BF16 ? 2 : 4;
    if (!aligned(y, ys) || !aligned(gate, ys) || !aligned(post_w, 4) || !aligned(pre_w, 4) || !aligned(residual, ss) ||
        !aligned(residual_out, ss) || !aligned(out, 2) || !aligned(out_q8, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (T == 0)
        return Q2K_OK;
    NormProblem p{};
    p.y = y;
    p.y_bf16 = y_type == Q2K_BF16;
    p.ld_y = ld_y;
    p.post_w = post_w;
    p.gate = gate;
    p.ld_gate = ld_gate;
    p.residual = residual;
    p.stream_bf16 = stream_type == Q2K_BF16;
    p.ld_res = ld_res;
    p.alpha = alpha;
    p.pre_w = pre_w;
    p.eps = eps;
    p.T = T;
    p.dim = dim;
    p.residual_out = residual_out;
    p.ld_ro = ld_ro;
    p.out = out;
    p.ld_out = ld_out;
    p.out_q8 = out_q8;
    return finish(launch_norm_gate_residual(p, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_route_topk(const void* logits, int type, int64_t m, int64_t E, int64_t ld, const float* bias, int score,
                   int64_t n_group, int64_t topk_group, int64_t topk, int renorm, float scale, int32_t* ids,
                   float* weights, const int64_t* expert_ptrs, int64_t* ptrs_out, q2k_stream_t stream)
{
    if (m != 0 && (!logits || !ids || !weights || (!expert_ptrs) != (!ptrs_out)))
        return Q2K_ERR_NULL_ARG;
    if (!type_ok(type) || m < 0 || m > (1 << 30) || E < 1 || E > 1024 || ld < E ||
        (score != Q2K_ROUTE_SOFTMAX && score != Q2K_ROUTE_SIGMOID) || n_group < 1 || n_group > 32 || E % n_group ||
        topk_group < 1 || topk_group > n_group || topk < 1 || topk > 32 || topk > topk_group * (E / n_group) ||
        (renorm != 0 && renorm != 1) || !(scale >= -3.0e38f && scale <= 3.0e38f))
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(logits, type == Q2K_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
        !aligned(expert_ptrs, 8) || !aligned(ptrs_out, 8))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (m == 0)
        return Q2K_OK;
    RouteProblem p{};
    p.logits = logits;
    p.bf16 = type == Q2K_BF16;
    p.m = m;
    p.E = E;
    p.ld = ld;
    p.bias = bias;
    p.sigmoid = score == Q2K_ROUTE_SIGMOID;
    p.n_group = (int)n_group;
    p.topk_group = (int)topk_group;
    p.topk = (int)topk;
    p.renorm = renorm;
    p.scale = scale;
    p.ids = ids;
    p.weights = weights;
    p.expert_ptrs = expert_ptrs;
    p.ptrs_out = ptrs_out;
    return finish(launch_moe_route(p, reinterpret_cast<cudaStream_t>(stream)));
}

int fp8_quantize(const void* x, int x_type, int64_t rows, int64_t K, int64_t ldx, int64_t block_rows, uint8_t* q,
                 int64_t ldq, float* scales, int64_t ld_scales, q2k_stream_t stream)
{
    if (rows != 0 && (!x || !q || !scales))
        return Q2K_ERR_NULL_ARG;
    if (!type_ok(x_type) || rows < 0 || rows > (1 << 30) || K < 1 || K > kMaxK || (block_rows != 1 && block_rows != 128) ||
        ldx < K || ldq < K || ld_scales < fp8_blocks(K))
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(x, x_type == Q2K_BF16 ? 2 : 4) || !aligned(scales, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (rows == 0)
        return Q2K_OK;
    Fp8Encode p{};
    p.x = x;
    p.x_bf16 = x_type == Q2K_BF16;
    p.block_rows = (int)block_rows;
    p.rows = rows;
    p.K = K;
    p.ldx = ldx;
    p.q = q;
    p.ldq = ldq;
    p.scales = scales;
    p.ld_scales = ld_scales;
    return finish(launch_fp8_encode(p, reinterpret_cast<cudaStream_t>(stream)));
}

int swiglu_fp8_rows(const void* gate_up, int type, int64_t rows, int64_t N, int64_t ld, uint8_t* q, int64_t ldq,
                    float* scales, int64_t ld_scales, q2k_stream_t stream)
{
    if (rows != 0 && (!gate_up || !q || !scales))
        return Q2K_ERR_NULL_ARG;
    if (!type_ok(type) || rows < 0 || rows > (1 << 30) || N < 1 || N > kMaxK / 2 || ld < 2 * N || ldq < N ||
        ld_scales < fp8_blocks(N))
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(gate_up, type == Q2K_BF16 ? 2 : 4) || !aligned(scales, 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (rows == 0)
        return Q2K_OK;
    Fp8Encode p{};
    p.x = gate_up;
    p.x_bf16 = type == Q2K_BF16;
    p.swiglu = 1;
    p.block_rows = 1;
    p.rows = rows;
    p.K = N;
    p.ldx = ld;
    p.q = q;
    p.ldq = ldq;
    p.scales = scales;
    p.ld_scales = ld_scales;
    return finish(launch_fp8_encode(p, reinterpret_cast<cudaStream_t>(stream)));
}

int fp8_gemm(const uint8_t* x, int64_t m, int64_t K, int64_t ldx, const float* x_scales, int64_t ld_xs,
             const uint8_t* W, int64_t N, const float* w_scales, void* y, int y_type, int64_t ldy, q2k_stream_t stream)
{
    if (!W || !w_scales || (m != 0 && (!x || !x_scales || !y)))
        return Q2K_ERR_NULL_ARG;
    if (!type_ok(y_type) || m < 0 || m >= (1 << 30) || N < 1 || N >= (1 << 30) || K < 16 || K > kMaxK || K % 16 ||
        ldx < K || ldx % 16 || ldx >= ((int64_t)1 << 36) || ld_xs < fp8_blocks(K) || ldy < N)
        return Q2K_ERR_BAD_SHAPE;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) ||
        !aligned(y, y_type == Q2K_BF16 ? 2 : 4))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (m == 0)
        return Q2K_OK;
    if (!fp8_encoder_there())
        return Q2K_ERR_UNSUPPORTED;  // no tensor-map encoder in this driver
    Fp8Gemm p{};
    p.x = x;
    p.m = m;
    p.K = K;
    p.ldx = ldx;
    p.x_scales = x_scales;
    p.ld_xs = ld_xs;
    p.W = W;
    p.N = N;
    p.w_scales = w_scales;
    p.y = y;
    p.y_bf16 = y_type == Q2K_BF16;
    p.ldy = ldy;
    return finish(launch_fp8_gemm(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fp8_moe_workspace_bytes(int64_t m, int64_t topk, int64_t dim, int64_t inter)
{
    if (!fp8_moe_shape_ok(m, topk, dim, inter))
        return 0;
    return fp8_moe_workspace(m, topk, inter);
}

int fp8_moe(const uint16_t* x, int64_t m, int64_t dim, int64_t ldx, const int32_t* ids, const float* route_w,
            int64_t topk, int64_t E, const uint8_t* gate_up, const float* gate_up_scales, const uint8_t* down,
            const float* down_scales, int64_t inter, void* y, int y_type, int64_t ldy, void* workspace,
            size_t workspace_bytes, q2k_stream_t stream)
{
    if (!gate_up || !gate_up_scales || !down || !down_scales || (m != 0 && (!x || !ids || !route_w || !y)))
        return Q2K_ERR_NULL_ARG;
    if (!fp8_moe_shape_ok(m, topk, dim, inter) || !type_ok(y_type) || E < 1 || E > 1024 || ldx < dim || ldy < dim)
        return Q2K_ERR_BAD_SHAPE;
    if (m != 0 && (!workspace || workspace_bytes < fp8_moe_workspace(m, topk, inter)))
        return Q2K_ERR_WORKSPACE;
    if (!aligned(x, 2) || !aligned(ids, 4) || !aligned(route_w, 4) || !aligned(gate_up, 16) || !aligned(down, 16) ||
        !aligned(gate_up_scales, 4) || !aligned(down_scales, 4) || !aligned(y, y_type == Q2K_BF16 ? 2 : 4) ||
        !aligned(workspace, 256))
        return Q2K_ERR_MISALIGNED;
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    if (m == 0)
        return Q2K_OK;
    if (!fp8_encoder_there())
        return Q2K_ERR_UNSUPPORTED;  // no tensor-map encoder in this driver
    Fp8Moe p{};
    p.x = x;
    p.m = m;
    p.dim = dim;
    p.ldx = ldx;
    p.ids = ids;
    p.route_w = route_w;
    p.topk = (int)topk;
    p.E = (int)E;
    p.gate_up = gate_up;
    p.gate_up_scales = gate_up_scales;
    p.down = down;
    p.down_scales = down_scales;
    p.inter = inter;
    p.y = y;
    p.y_bf16 = y_type == Q2K_BF16;
    p.ldy = ldy;
    p.workspace = workspace;
    return finish(launch_fp8_moe(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// ---- routed experts without any allocation -------------------------------------
//
// Some callers cannot hand the library a workspace: a host program that links
// only this library and has no device allocator of its own, or a decode loop
// whose memory is planned once up front and must not allocate (or make its
// allocator grow) between steps.  For them this entry point runs the same
// launches as q2k_moe_m1 on a fixed scratch buffer that lives in the
// library's own device image.  The scratch is a file-scope __device__ array,
// so it is reserved when the module loads: nothing is allocated or freed here.
//
// Every byte of the scratch is written before it is read within one call
// (the q8_1 x, the fp32 gate/up outputs and the q8_1 h are produced in full
// by their launches), so nothing has to be cleared.  Calls that overlap on
// one device (two streams, or two threads) share this buffer and race; keep
// them on one stream.

namespace {
__device__ __align__(256) unsigned char g_moe_scratch[Q2K_MOE_M1_STATIC_SCRATCH_BYTES];

void* g_moe_scratch_ptr[kMaxDevices];
std::mutex g_moe_scratch_mu;

// The scratch's device address on the current device, looked up once per
// device (the first call on a device does this; it may load the module).
// The cached address belongs to the device's context at that time: after a
// cudaDeviceReset the module loads again, possibly elsewhere, and the cached
// address is stale, so a process that resets a device must not call this
// entry point on it afterwards.
cudaError_t moe_scratch(void** out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(g_moe_scratch_mu);
    if (!g_moe_scratch_ptr[dev]) {
        void* p = nullptr;
        if ((e = cudaGetSymbolAddress(&p, g_moe_scratch)) != cudaSuccess)
            return e;
        g_moe_scratch_ptr[dev] = p;
    }
    *out = g_moe_scratch_ptr[dev];
    return cudaSuccess;
}
}  // namespace

extern "C" int q2k_moe_m1_static_scratch(const void* const* ptrs, int64_t E, int64_t dim, int64_t inter,
                                         const uint16_t* x_bf16, const float* route_w, float* y,
                                         q2k_stream_t stream)
{
    if (!ptrs || !x_bf16 || !route_w || !y)
        return Q2K_ERR_NULL_ARG;
    // the shapes q2k_moe_m1 refuses are refused here the same way; only a
    // valid problem that needs more than the fixed scratch is a WORKSPACE error
    if (E <= 0 || E > 1024 || dim <= 0 || inter <= 0 || dim % kBlockWeights || inter % kBlockWeights ||
        dim > kMaxK || inter > kMaxK)
        return Q2K_ERR_BAD_SHAPE;
    const size_t need = q2k_moe_m1_workspace_bytes(E, dim, inter);
    if (need > (size_t)Q2K_MOE_M1_STATIC_SCRATCH_BYTES)
        return Q2K_ERR_WORKSPACE;  // the problem does not fit the fixed scratch
    int st = check_device();
    if (st != Q2K_OK)
        return st;
    void* ws = nullptr;
    cudaError_t e = moe_scratch(&ws);
    if (e != cudaSuccess)
        return fail_cuda(e);
    return q2k_moe_m1(ptrs, E, dim, inter, x_bf16, route_w, y, ws, (size_t)Q2K_MOE_M1_STATIC_SCRATCH_BYTES, stream);
}

