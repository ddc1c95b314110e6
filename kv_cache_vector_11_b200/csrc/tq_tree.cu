// Attention of the newest tokens of every request over its paged, packed cache
// (tq_tree_attention): one CTA per (node, head), online softmax in fp32.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <climits>
#include <cmath>

#include "tq_device.cuh"

namespace tq {
namespace {

constexpr int kTaThreads = 128;
constexpr int kTaMaxNodes = 256;

struct TreeArgs {
    const void * q;
    int32_t q_dtype;
    const int32_t * cu;
    int32_t batch, n_rows, max_nodes;
    const int32_t * lens;
    int64_t max_len;
    const uint64_t * mask;
    int32_t mask_words;
    int32_t n_q_heads, n_kv_heads;
    int32_t page_shift, n_pages, max_pages;
    const int32_t * table;
    const uint32_t * k_codes;
    const uint16_t * k_norms;
    const uint32_t * v_codes;
    const uint16_t * v_norms;
    float scale;
    int32_t dense;              // HAAR rotation (rot_f32) instead of Walsh-Hadamard
    const float * rot_f32;
    uint32_t d1_bits[8], d2_bits[8];
    float kc[kMaxLevels], vc[kMaxLevels];
    void * out;
    uint32_t * status;
};

__device__ __forceinline__ float load_el(const void * p, int dt, int64_t i) {
    if (dt == TQ_DTYPE_F32) return static_cast<const float *>(p)[i];
    if (dt == TQ_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    return __half2float(static_cast<const __half *>(p)[i]);
}
__device__ __forceinline__ void store_el(void * p, int dt, int64_t i, float v) {
    if (dt == TQ_DTYPE_F32) static_cast<float *>(p)[i] = v;
    else if (dt == TQ_DTYPE_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half *>(p)[i] = __float2half_rn(v);
}
__device__ __forceinline__ float sgn(const uint32_t * bits, int i) {
    return ((bits[i >> 5] >> (i & 31)) & 1u) ? -1.0f : 1.0f;
}

template <int D>
__device__ void fwht(float * v) {
    for (int h = 1; h < D; h <<= 1) {
        __syncthreads();
        for (int k = threadIdx.x; k < D / 2; k += kTaThreads) {
            const int i = (k / h) * 2 * h + (k % h);
            const float x = v[i], y = v[i + h];
            v[i] = x + y;
            v[i + h] = x - y;
        }
    }
    __syncthreads();
}

template <int D, int KB, int VB>
__global__ void __launch_bounds__(kTaThreads) tree_simple_kernel(const __grid_constant__ TreeArgs a) {
    constexpr int NB = D / 32, W = kTaThreads / 32;
    __shared__ float raw[D], qr[D], part[W][D], ml[W][2];
    const int row = blockIdx.x / a.n_q_heads, h = blockIdx.x % a.n_q_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= row) lo = mid; else hi = mid;
    }
    const int r0 = max(a.cu[lo], 0), r1 = min(a.cu[lo + 1], a.n_rows);
    if (row < r0 || row >= r1 || row - r0 >= a.max_nodes) return;
    const int node = row - r0, n = min(r1 - r0, a.max_nodes);
    const int64_t len = min((int64_t)max(a.lens[lo], 0), a.max_len);
    const int64_t base = (int64_t)(row * (int64_t)a.n_q_heads + h) * D;
    for (int i = threadIdx.x; i < D; i += kTaThreads) raw[i] = load_el(a.q, a.q_dtype, base + i);
    __syncthreads();
    if (!a.dense) {
        for (int i = threadIdx.x; i < D; i += kTaThreads) qr[i] = raw[i] * sgn(a.d2_bits, i);
        fwht<D>(qr);
        for (int i = threadIdx.x; i < D; i += kTaThreads) qr[i] *= rsqrtf((float)D) * sgn(a.d1_bits, i);
    } else {
        for (int e = threadIdx.x; e < D; e += kTaThreads) {
            float s = 0.0f;
            for (int i = 0; i < D; ++i) s = fmaf(a.rot_f32[e * D + i], raw[i], s);
            qr[e] = s;
        }
    }
    __syncthreads();
    const int hk = h / (a.n_q_heads / a.n_kv_heads);
    const int64_t ctx0 = len - n;
    float q[NB], o[NB];
    for (int b = 0; b < NB; ++b) { q[b] = qr[32 * b + lane] * a.scale; o[b] = 0.0f; }
    float m = -CUDART_INF_F, l = 0.0f;
    for (int64_t t = warp; t < len; t += W) {
        const int64_t j = t - ctx0;
        if (j >= 0) {
            if (a.mask != nullptr) {
                if (!((a.mask[(int64_t)row * a.mask_words + (j >> 6)] >> (j & 63)) & 1u)) continue;
            } else if (j > node) {
                continue;
            }
        }
        const int pg = min(max(a.table[(int64_t)lo * a.max_pages + (t >> a.page_shift)], 0), a.n_pages - 1);
        const int64_t r = (((int64_t)pg * a.n_kv_heads + hk) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
        float s = 0.0f;
        for (int b = 0; b < NB; ++b) {
            const uint32_t c = extract_code<KB>(a.k_codes + (r * NB + b) * KB, lane);
            s = fmaf(q[b], a.kc[c] * half_bits_to_float(a.k_norms[r * NB + b]), s);
        }
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s);
        const float c = m == -CUDART_INF_F ? 0.0f : expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * c + p;
        for (int b = 0; b < NB; ++b) {
            const uint32_t vi = extract_code<VB>(a.v_codes + (r * NB + b) * VB, lane);
            o[b] = o[b] * c + p * a.vc[vi] * half_bits_to_float(a.v_norms[r * NB + b]);
        }
    }
    for (int b = 0; b < NB; ++b) part[warp][32 * b + lane] = o[b];
    if (lane == 0) { ml[warp][0] = m; ml[warp][1] = l; }
    __syncthreads();
    float M = -CUDART_INF_F, L = 0.0f;
    for (int w = 0; w < W; ++w) M = fmaxf(M, ml[w][0]);
    for (int w = 0; w < W; ++w) L += ml[w][0] == -CUDART_INF_F ? 0.0f : expf(ml[w][0] - M) * ml[w][1];
    for (int i = threadIdx.x; i < D; i += kTaThreads) {
        float t = 0.0f;
        for (int w = 0; w < W; ++w) t += ml[w][0] == -CUDART_INF_F ? 0.0f : expf(ml[w][0] - M) * part[w][i];
        raw[i] = L != 0.0f ? t / L : 0.0f;
    }
    __syncthreads();
    if (!a.dense) {
        for (int i = threadIdx.x; i < D; i += kTaThreads) raw[i] *= sgn(a.d1_bits, i);
        fwht<D>(raw);
        for (int i = threadIdx.x; i < D; i += kTaThreads)
            store_el(a.out, a.q_dtype, base + i, raw[i] * rsqrtf((float)D) * sgn(a.d2_bits, i));
    } else {
        for (int i = threadIdx.x; i < D; i += kTaThreads) {
            float s = 0.0f;
            for (int e = 0; e < D; ++e) s = fmaf(a.rot_f32[e * D + i], raw[e], s);
            store_el(a.out, a.q_dtype, base + i, s);
        }
    }
}

template <int D, int KB>
int launch_tree_v(const TreeArgs & a, int vb, cudaStream_t st) {
    const unsigned grid = (unsigned)((int64_t)a.n_rows * a.n_q_heads);
    if (vb == 2) tree_simple_kernel<D, KB, 2><<<grid, kTaThreads, 0, st>>>(a);
    else if (vb == 3) tree_simple_kernel<D, KB, 3><<<grid, kTaThreads, 0, st>>>(a);
    else tree_simple_kernel<D, KB, 4><<<grid, kTaThreads, 0, st>>>(a);
    return (int)cudaGetLastError();
}

template <int D>
int launch_tree(const TreeArgs & a, int kb, int vb, cudaStream_t st) {
    return kb == 2 ? launch_tree_v<D, 2>(a, vb, st) : kb == 3 ? launch_tree_v<D, 3>(a, vb, st)
                                                             : launch_tree_v<D, 4>(a, vb, st);
}

bool tree_sizes_ok(int32_t batch, int32_t n_rows, int32_t max_nodes, int32_t n_q_heads, int32_t n_kv_heads,
                   int64_t max_len, int32_t head_dim, const char ** why) {
    *why = nullptr;
    if (!supported_dim(head_dim)) *why = "head_dim must be 64, 128 or 256";
    else if (batch < 1 || n_rows < 0 || max_len < 0) *why = "batch must be >= 1, n_rows and max_len >= 0";
    else if (max_nodes < 1 || max_nodes > kTaMaxNodes) *why = "max_nodes must be in [1, 256]";
    else if (n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads != 0)
        *why = "n_q_heads must be a positive multiple of n_kv_heads";
    else if ((int64_t)n_rows * n_q_heads > INT32_MAX / 2) *why = "more than 2^30 rows times heads";
    else if (max_len > INT32_MAX) *why = "max_len above 2^31 - 1";
    return *why == nullptr;
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" size_t tq_tree_workspace_size(int32_t batch, int32_t n_rows, int32_t max_nodes, int32_t n_q_heads,
                                         int32_t n_kv_heads, int64_t max_len, int32_t head_dim) {
    const char * why;
    if (!tree_sizes_ok(batch, n_rows, max_nodes, n_q_heads, n_kv_heads, max_len, head_dim, &why)) return 0;
    return 256;
}

extern "C" tq_status tq_tree_attention(const tq_rotation * rot, int32_t k_bits, int32_t v_bits, int32_t block,
                                       const float * k_centroids, const float * v_centroids, const void * q,
                                       tq_dtype q_dtype, const int32_t * cu_nodes, int32_t batch, int32_t n_rows,
                                       int32_t max_nodes, const int32_t * lens, int64_t max_len,
                                       const uint64_t * tree_mask, int32_t mask_words, int32_t n_q_heads,
                                       int32_t n_kv_heads, int32_t head_dim, int32_t page_size, int32_t n_pages,
                                       const int32_t * block_table, int32_t max_pages, const uint32_t * k_codes,
                                       const uint16_t * k_norms, const uint32_t * v_codes, const uint16_t * v_norms,
                                       float scale, void * out, void * workspace, size_t workspace_bytes,
                                       uint32_t * status_dev, void * stream) {
    tq_status st = check_rotation(rot, head_dim);
    if (st != TQ_OK) return st;
    const char * why;
    if (!tree_sizes_ok(batch, n_rows, max_nodes, n_q_heads, n_kv_heads, max_len, head_dim, &why))
        return fail(TQ_ERR_INVALID_ARG, why);
    if (!supported_bits(k_bits) || !supported_bits(v_bits))
        return fail(TQ_ERR_UNSUPPORTED, "k_bits and v_bits must be 2, 3 or 4");
    if (block != kBlock) return fail(TQ_ERR_UNSUPPORTED, "paged caches hold block 32 (fp16 norms)");
    if (q_dtype != TQ_DTYPE_F32 && q_dtype != TQ_DTYPE_BF16 && q_dtype != TQ_DTYPE_F16)
        return fail(TQ_ERR_INVALID_ARG, "unknown q dtype");
    if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
        return fail(TQ_ERR_UNSUPPORTED, "page_size must be a power of two in [16, 65536]");
    if (n_pages < 1 || max_pages < 1) return fail(TQ_ERR_INVALID_ARG, "n_pages and max_pages must be >= 1");
    if (max_len > (int64_t)max_pages * page_size)
        return fail(TQ_ERR_INVALID_ARG, "max_len exceeds max_pages * page_size");
    if (tree_mask && (mask_words < (max_nodes + 63) / 64))
        return fail(TQ_ERR_INVALID_ARG, "mask_words below ceil(max_nodes / 64)");
    if (std::isnan(scale) || std::isinf(scale)) return fail(TQ_ERR_INVALID_ARG, "scale is not finite");
    CodebookParams kcb, vcb;
    if ((st = build_codebook_params(k_bits, k_centroids, nullptr, &kcb, false)) != TQ_OK) return st;
    if ((st = build_codebook_params(v_bits, v_centroids, nullptr, &vcb, false)) != TQ_OK) return st;
    if (n_rows == 0) return TQ_OK;
    if (!q || !out || !cu_nodes || !lens || !block_table || !k_codes || !k_norms || !v_codes || !v_norms)
        return fail(TQ_ERR_INVALID_ARG, "null q / out / cu_nodes / lens / block_table / cache");
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_codes, 16) || !aligned(k_norms, 16) ||
        !aligned(v_codes, 16) || !aligned(v_norms, 16))
        return fail(TQ_ERR_INVALID_ARG, "q, out and the cache must be 16-byte aligned");
    if (!aligned(cu_nodes, 4) || !aligned(lens, 4) || !aligned(block_table, 4) || !aligned(tree_mask, 8) ||
        !aligned(status_dev, 4))
        return fail(TQ_ERR_INVALID_ARG, "int32 arrays 4-byte, tree_mask 8-byte aligned");
    const size_t need = tq_tree_workspace_size(batch, n_rows, max_nodes, n_q_heads, n_kv_heads, max_len, head_dim);
    if (!workspace || workspace_bytes < need)
        return fail(TQ_ERR_INVALID_ARG, "workspace missing or smaller than tq_tree_workspace_size");
    if (!aligned(workspace, 256)) return fail(TQ_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    TreeArgs a{};
    a.q = q;
    a.q_dtype = q_dtype;
    a.cu = cu_nodes;
    a.batch = batch;
    a.n_rows = n_rows;
    a.max_nodes = max_nodes;
    a.lens = lens;
    a.max_len = max_len;
    a.mask = tree_mask;
    a.mask_words = mask_words;
    a.n_q_heads = n_q_heads;
    a.n_kv_heads = n_kv_heads;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.n_pages = n_pages;
    a.max_pages = max_pages;
    a.table = block_table;
    a.k_codes = k_codes;
    a.k_norms = k_norms;
    a.v_codes = v_codes;
    a.v_norms = v_norms;
    a.scale = scale > 0.0f ? scale : 1.0f / std::sqrt((float)head_dim);
    a.dense = rot->kind == TQ_ROT_HAAR;
    a.rot_f32 = rot->dev_f32;
    for (int i = 0; i < 8; ++i) {
        a.d1_bits[i] = rot->d1_bits[i];
        a.d2_bits[i] = rot->d2_bits[i];
    }
    for (int i = 0; i < kMaxLevels; ++i) {
        a.kc[i] = kcb.centroid[i];
        a.vc[i] = vcb.centroid[i];
    }
    a.out = out;
    a.status = status_dev;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int e = head_dim == 64 ? launch_tree<64>(a, k_bits, v_bits, s)
                : head_dim == 128 ? launch_tree<128>(a, k_bits, v_bits, s) : launch_tree<256>(a, k_bits, v_bits, s);
    return cuda_status(e, "tree attention launch");
}
