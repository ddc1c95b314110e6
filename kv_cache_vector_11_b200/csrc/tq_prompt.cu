// Causal attention of packed sequences over their unquantized keys and values
// (tq_prompt_attention): one warp per (query, head), online softmax in fp32.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <climits>
#include <cmath>

#include "tq_device.cuh"

namespace tq {
namespace {

constexpr int kPaThreads = 128;

struct PromptArgs {
    const void * q;
    const void * k;
    const void * v;
    const int32_t * cu_q;
    const int32_t * cu_k;
    int32_t batch;
    int64_t total_q, total_k;
    int32_t n_q_heads, n_kv_heads;
    int64_t q_stride, k_stride, v_stride;
    float scale;
    void * out;
    uint32_t * status;
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16 * o) { *o = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(float x, __half * o) { *o = __float2half_rn(x); }

__device__ __forceinline__ int64_t clamp_to(int64_t x, int64_t lo, int64_t hi) { return min(max(x, lo), hi); }

template <int D, typename T>
__global__ void __launch_bounds__(kPaThreads) prompt_simple_kernel(const __grid_constant__ PromptArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (kPaThreads / 32) + (threadIdx.x >> 5);
    const int64_t tok = w / a.n_q_heads;
    const int h = (int)(w % a.n_q_heads);
    if (tok >= a.total_q) return;
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_q[mid] <= tok) lo = mid; else hi = mid;
    }
    const int64_t q0 = clamp_to(a.cu_q[lo], 0, a.total_q), q1 = clamp_to(a.cu_q[lo + 1], q0, a.total_q);
    if (tok < q0 || tok >= q1) return;
    const int64_t k0 = clamp_to(a.cu_k[lo], 0, a.total_k), k1 = clamp_to(a.cu_k[lo + 1], k0, a.total_k);
    const int64_t n = clamp_to(tok - q0 + (k1 - k0) - (q1 - q0) + 1, 0, k1 - k0);
    const int hk = h / (a.n_q_heads / a.n_kv_heads);
    constexpr int E = D / 32;
    float q[E], o[E];
    const T * qp = static_cast<const T *>(a.q) + tok * a.q_stride + (int64_t)h * D;
    for (int e = 0; e < E; ++e) { q[e] = to_f32(qp[lane + 32 * e]) * a.scale; o[e] = 0.0f; }
    float m = -CUDART_INF_F, l = 0.0f;
    for (int64_t j = k0; j < k0 + n; ++j) {
        const T * kp = static_cast<const T *>(a.k) + j * a.k_stride + (int64_t)hk * D;
        const T * vp = static_cast<const T *>(a.v) + j * a.v_stride + (int64_t)hk * D;
        float s = 0.0f;
        for (int e = 0; e < E; ++e) s = fmaf(q[e], to_f32(kp[lane + 32 * e]), s);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s);
        const float c = m == -CUDART_INF_F ? 0.0f : expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * c + p;
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * to_f32(vp[lane + 32 * e]);
    }
    T * op = static_cast<T *>(a.out) + (tok * a.n_q_heads + h) * D;
    for (int e = 0; e < E; ++e) from_f32(n > 0 ? o[e] / l : 0.0f, op + lane + 32 * e);
}

template <int D, typename T>
int launch_prompt_t(const PromptArgs & a, cudaStream_t st) {
    const int64_t warps = a.total_q * a.n_q_heads, per = kPaThreads / 32;
    prompt_simple_kernel<D, T><<<(unsigned)((warps + per - 1) / per), kPaThreads, 0, st>>>(a);
    return (int)cudaGetLastError();
}

template <int D>
int launch_prompt(const PromptArgs & a, tq_dtype dtype, cudaStream_t st) {
    return dtype == TQ_DTYPE_BF16 ? launch_prompt_t<D, __nv_bfloat16>(a, st) : launch_prompt_t<D, __half>(a, st);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" tq_status tq_prompt_attention(const void * q, const void * k, const void * v, tq_dtype dtype,
                                         const int32_t * cu_q, const int32_t * cu_k, int32_t batch,
                                         int64_t total_q, int64_t total_k, int32_t n_q_heads,
                                         int32_t n_kv_heads, int32_t head_dim, int64_t q_stride,
                                         int64_t k_stride, int64_t v_stride, float scale, void * out,
                                         uint32_t * status_dev, void * stream) {
    if (!supported_dim(head_dim)) return fail(TQ_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
    if (dtype != TQ_DTYPE_BF16 && dtype != TQ_DTYPE_F16)
        return fail(TQ_ERR_UNSUPPORTED, "prompt attention takes bf16 or fp16 rows");
    if (n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads != 0)
        return fail(TQ_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of n_kv_heads");
    if (n_q_heads > 65535) return fail(TQ_ERR_UNSUPPORTED, "more than 65535 query heads");
    if (batch < 1 || total_q < 0 || total_k < 0)
        return fail(TQ_ERR_INVALID_ARG, "batch must be >= 1, total_q and total_k >= 0");
    if (total_q > INT32_MAX || total_k > INT32_MAX)
        return fail(TQ_ERR_UNSUPPORTED, "more than 2^31 - 1 packed tokens");
    if (std::isnan(scale) || std::isinf(scale)) return fail(TQ_ERR_INVALID_ARG, "scale is not finite");
    if (q_stride < (int64_t)n_q_heads * head_dim || k_stride < (int64_t)n_kv_heads * head_dim ||
        v_stride < (int64_t)n_kv_heads * head_dim || ((q_stride | k_stride | v_stride) & 7) != 0)
        return fail(TQ_ERR_INVALID_ARG, "token strides must be multiples of 8 elements, at least one row");
    if (total_q == 0) return TQ_OK;
    if (!q || !out || !cu_q || (total_k > 0 && (!k || !v)))
        return fail(TQ_ERR_INVALID_ARG, "null q / k / v / out / cu_q");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu_q, 4) ||
        !aligned(cu_k, 4) || !aligned(status_dev, 4))
        return fail(TQ_ERR_INVALID_ARG, "q, k, v and out must be 16-byte aligned, offsets 4-byte");
    PromptArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.cu_q = cu_q;
    a.cu_k = cu_k ? cu_k : cu_q;
    a.batch = batch;
    a.total_q = total_q;
    a.total_k = total_k;
    a.n_q_heads = n_q_heads;
    a.n_kv_heads = n_kv_heads;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.scale = scale > 0.0f ? scale : 1.0f / std::sqrt((float)head_dim);
    a.out = out;
    a.status = status_dev;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int e = head_dim == 64 ? launch_prompt<64>(a, dtype, st)
                : head_dim == 128 ? launch_prompt<128>(a, dtype, st) : launch_prompt<256>(a, dtype, st);
    return cuda_status(e, "prompt attention launch");
}
