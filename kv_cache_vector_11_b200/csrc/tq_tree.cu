// Attention of the newest tokens of every request over its paged, packed cache
// (tq_tree_attention), on the tensor cores.
//
//   out = R^T sum_t p_t v^_t / sum_t p_t,   p_t = 2^(mul <q~, k^_t> - ref),   q~ = R q
//
// Three launches: the queries are rotated into fp16 rows (tree_prep_kernel),
// every CTA takes an equal share of the key tiles of all requests
// (tree_kernel), and the shares of a row are merged and rotated back
// (tree_combine_kernel).
//
// A row is a (node, head of the group) pair, heads inner; the rows of one
// request and KV head attend the same cached tokens, so a tile of 128 keys is
// unpacked once for all of them.  The unit of work is one key tile against one
// set of rows, counted request by request; the grid is one CTA per SM and CTA c
// takes the units [c W / C, (c + 1) W / C): long caches are split over many
// CTAs, short ones share one.  Where a CTA's range starts inside a set's tiles
// it writes its part of the sum into a slot of its own, all other parts go to
// the rows' own slots, so a row has one own slot and one more per further CTA.
//
// In the CTA one warpgroup unpacks keys and one values into swizzled operand tiles
// (shared memory, a ring of buffers each), two warps issue the MMAs, one softmax
// thread per row turns scores into weights (tq_fmha.cuh).  Which rows share a CTA:
//   PAIR:   two row tiles (256 rows) against the same key tile: unpacking is
//           paid once for both, the tensor core works on one while the softmax
//           warps of the other run;
//   STREAM: one row tile (at most 128 rows), the even key tiles and the odd
//           ones with a softmax and an accumulator each.  Taken when no request
//           can have more than 128 rows;
//   WIDE:   d = 256, one row tile whose accumulator fills half of TMEM, the
//           scores of the next key tile under way during a softmax.
// At most 8 rows take a kernel of their own (tree_few_kernel).
//
// Unpacking: centroids are 16-bit table entries, looked up four at a time with
// byte permutes (a table of 8 bytes in two registers; the low and the high
// bytes of four entries, interleaved), times the block's norm in fp16.
//
// What bounds it: the integer pipe, which byte permutes, masks and the maxima of
// the softmax share.  A key tile of 128 tokens takes the two unpacking warpgroups
// about 3000 cycles (d = 128, 4-bit keys and 3-bit values), its products 1280 a
// row tile; 8 x 128K trees of 64 nodes, 4 heads a group: 1.21 ms on the same inputs
// again and again, 0.91 PFLOP/s; 1.39 ms on inputs that change, 0.79 PFLOP/s.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <climits>
#include <cmath>

#include "tq_device.cuh"
#include "tq_fmha.cuh"

namespace tq {
namespace {

using fm::kTile;

constexpr int kTaMaxNodes = 256;
constexpr int kFewRows = 8;          // rows that share a key tile in tree_few_kernel

enum TreeMode { PAIR = 0, STREAM = 1, WIDE = 2 };

struct TreeArgs {
    const void * q;
    int32_t q_dtype;
    const int32_t * cu;
    int32_t batch, n_rows, max_nodes;
    const int32_t * lens;
    int64_t max_len;
    const uint64_t * mask;
    int32_t mask_words;
    int32_t n_q_heads, n_kv_heads, group;
    int32_t page_shift, n_pages, max_pages;
    const int32_t * table;
    const uint32_t * k_codes;
    const uint16_t * k_norms;
    const uint32_t * v_codes;
    const uint16_t * v_norms;
    int32_t k_bits, v_bits;
    float scale;
    int32_t dense;              // HAAR rotation (rot_f32) instead of Walsh-Hadamard
    const float * rot_f32;
    uint32_t d1_bits[8], d2_bits[8];
    // fp16 centroids: low bytes of entries 0..15 (4 words), high bytes (4 words)
    uint32_t k_table[8], v_table[8];
    void * out;
    uint32_t * status;
    int32_t rows_per_set;       // rows that share a CTA: 256 (PAIR) or 128
    int32_t streams;            // own slots of a row: 2 (STREAM) or 1
    int32_t n_ctas;             // sharers of the units: CTAs, or warps where few rows share a tile
    int32_t more_rows;          // rows of a sharer in `more`: 256, or 8
    // workspace
    int64_t * unit0;            // [batch + 1] units before a request
    int32_t * row_request;      // [n_rows] the request of a row, -1 for padding
    __half * q_rows;            // [n_rows * n_q_heads][d], by request, KV head, node, head
    float * q_mul;              // what a row's scores are multiplied by
    int64_t own_rows;           // n_rows * n_q_heads, up to a multiple of 32
    float * own;                // partial sums of streams x own_rows rows (part_at)
    float2 * own_ml;            //   their (ref, sum of weights)
    float * more;               // of n_ctas x more_rows rows, parts of sets that began with an earlier sharer
    float2 * more_ml;
};

// Request b: its first row, the nodes that are computed, the tokens before its
// nodes (negative where some are not cached) and all its cached tokens, clamped as
// the entry point says.  The nodes lie behind `ctx` also where max_nodes leaves
// out the last of them.
struct Request {
    int32_t r0, n, ctx, len;
};
__device__ __forceinline__ Request request_of(const TreeArgs & a, int b) {
    Request q;
    q.r0 = min(max(a.cu[b], 0), a.n_rows);
    const int32_t nodes = min(max(a.cu[b + 1], q.r0), a.n_rows) - q.r0;
    q.n = min(nodes, a.max_nodes);
    q.len = (int32_t)min((int64_t)max(a.lens[b], 0), a.max_len);
    q.ctx = q.len - nodes;
    return q;
}
// Whether something of request b was clamped.
__device__ __forceinline__ bool past_limits(const TreeArgs & a, int b) {
    const int32_t r0 = a.cu[b], r1 = a.cu[b + 1], len = a.lens[b];
    return r0 < 0 || r1 < r0 || r1 > a.n_rows || r1 - r0 > a.max_nodes || len < 0 || len > a.max_len;
}
__device__ __forceinline__ int sets_of(const TreeArgs & a, int n) {
    return (n * a.group + a.rows_per_set - 1) / a.rows_per_set;
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// The CTAs that share the units (no more than there are), the first unit of
// CTA c, and the CTA whose range holds unit u.
__device__ __forceinline__ int64_t sharers(const TreeArgs & a, int64_t units) { return min((int64_t)a.n_ctas, units); }
__device__ __forceinline__ int64_t first_unit(int64_t c, int64_t units, int64_t n) { return n > 0 ? units * min(c, n) / n : 0; }
__device__ __forceinline__ int cta_of(int64_t u, int64_t units, int64_t n) {
    const int64_t x = (u + 1) * n - 1;
    // (a 32-bit division where it does: the 64-bit one takes some 500 cycles)
    return (x | units) <= 0xFFFFFFFFll ? (int)((uint32_t)x / (uint32_t)units) : (int)(x / units);
}

// Where column `col` (a multiple of 4) of row `row` of the partial sums lies:
// 32 rows take turns, four columns each, since a thread has a row and a warp
// then writes 512 bytes in a piece (stored row by row, 16 bytes of 32 rows at a
// time, tree_kernel took 130 us for 16 trees over up to 32K tokens, this way 114).
template <int D>
__device__ __forceinline__ int64_t part_at(int64_t row, int col) {
    return ((row >> 5) * (D / 4) + (col >> 2)) * 128 + (row & 31) * 4;
}

// Reference and sum of a part.  A reference of -inf says that no key was attended
// and the sums are not to be read; NaN scores, which no maximum sees, leave one
// beside a NaN sum, and must be.
__device__ __forceinline__ float2 part_ml(float ref, float sum) { return make_float2(isnan(sum) ? sum : ref, sum); }

// The parts of this CTA's range, one per (request, KV head, row set).
struct Part {
    int b, hk, set, tile0, tiles;    // key tiles [tile0, tile0 + tiles)
    Request rq;
    int rows;                        // rows of the set (> 0)
    int64_t row_id;                  // of the set's first row
};
struct PartIter {
    int64_t u, end;
    int b;
    __device__ __forceinline__ void start(const TreeArgs & a, int b0) {
        const int64_t units = a.unit0[a.batch];
        const int64_t n = sharers(a, units);
        u = first_unit(blockIdx.x, units, n);
        end = first_unit(blockIdx.x + 1, units, n);
        b = b0;
    }
    __device__ __forceinline__ bool next(const TreeArgs & a, Part & p) {
        if (u >= end) return false;
        while (u >= a.unit0[b + 1]) ++b;
        p.b = b;
        p.rq = request_of(a, b);
        const int sets = sets_of(a, p.rq.n), tiles = tiles_of(p.rq.len);
        const int64_t rel = u - a.unit0[b];
        const int64_t s = rel / tiles;
        p.tile0 = (int)(rel - s * tiles);
        p.hk = (int)(s / sets);
        p.set = (int)(s - (int64_t)p.hk * sets);
        p.tiles = (int)min((int64_t)(tiles - p.tile0), end - u);
        p.rows = min(a.rows_per_set, p.rq.n * a.group - p.set * a.rows_per_set);
        p.row_id = (int64_t)p.rq.r0 * a.n_q_heads + (int64_t)p.hk * p.rq.n * a.group + (int64_t)p.set * a.rows_per_set;
        u += p.tiles;
        return true;
    }
};

// ---------------------------------------------------------------------------
// Rotation of the queries
// ---------------------------------------------------------------------------

constexpr int kTpThreads = 256;

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
// E consecutive elements from a multiple of E on (2, 4 or 8 of them), as one or
// two wide accesses.
template <int BYTES>
struct Words {
    uint32_t w[BYTES / 4];
};
template <int BYTES>
__device__ __forceinline__ Words<BYTES> load_words(const void * p) {
    Words<BYTES> r;
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            const uint4 u = static_cast<const uint4 *>(p)[i];
            r.w[4 * i] = u.x; r.w[4 * i + 1] = u.y; r.w[4 * i + 2] = u.z; r.w[4 * i + 3] = u.w;
        }
    } else if constexpr (BYTES == 8) {
        const uint2 u = *static_cast<const uint2 *>(p);
        r.w[0] = u.x; r.w[1] = u.y;
    } else {
        r.w[0] = *static_cast<const uint32_t *>(p);
    }
    return r;
}
template <int BYTES>
__device__ __forceinline__ void store_words(void * p, const Words<BYTES> & r) {
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i)
            static_cast<uint4 *>(p)[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
    } else if constexpr (BYTES == 8) {
        *static_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
    } else {
        *static_cast<uint32_t *>(p) = r.w[0];
    }
}
template <int E>
__device__ __forceinline__ void load_vec(const void * p, int dt, int64_t at, float * v) {
    if (dt == TQ_DTYPE_F32) {
        const Words<4 * E> r = load_words<4 * E>(static_cast<const float *>(p) + at);
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = __uint_as_float(r.w[k]);
        return;
    }
    const Words<2 * E> r = load_words<2 * E>(static_cast<const uint16_t *>(p) + at);
#pragma unroll
    for (int k = 0; k < E; k += 2) {
        if (dt == TQ_DTYPE_BF16) {
            v[k] = bf16_lo(r.w[k / 2]);
            v[k + 1] = bf16_hi(r.w[k / 2]);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[k / 2]));
            v[k] = f.x;
            v[k + 1] = f.y;
        }
    }
}
template <int E>
__device__ __forceinline__ void store_vec(void * p, int dt, int64_t at, const float * v) {
    if (dt == TQ_DTYPE_F32) {
        Words<4 * E> r;
#pragma unroll
        for (int k = 0; k < E; ++k) r.w[k] = __float_as_uint(v[k]);
        store_words<4 * E>(static_cast<float *>(p) + at, r);
        return;
    }
    Words<2 * E> r;
#pragma unroll
    for (int k = 0; k < E; k += 2)
        r.w[k / 2] = dt == TQ_DTYPE_BF16 ? fm::pack2<true>(v[k], v[k + 1]) : fm::pack2<false>(v[k], v[k + 1]);
    store_words<2 * E>(static_cast<uint16_t *>(p) + at, r);
}
__device__ __forceinline__ float signed_by(const uint32_t * bits, int i, float v) {
    return ((bits[i >> 5] >> (i & 31)) & 1u) ? -v : v;
}

// Walsh-Hadamard transform of a vector held by a warp, lane l with elements
// E l .. E l + E - 1, scaled by 1 / sqrt(32 E).
template <int E>
__device__ __forceinline__ void warp_fwht(float * v, int lane) {
#pragma unroll
    for (int h = 1; h < E; h <<= 1)
#pragma unroll
        for (int i = 0; i < E; ++i)
            if ((i & h) == 0) {
                const float x = v[i], y = v[i + h];
                v[i] = x + y;
                v[i + h] = x - y;
            }
#pragma unroll
    for (int h = 1; h < 32; h <<= 1)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float o = __shfl_xor_sync(0xffffffffu, v[i], h);
            v[i] = (lane & h) ? o - v[i] : v[i] + o;
        }
    const float sc = rsqrtf(32.0f * E);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= sc;
}

// The request of a row, the last one that starts at or before it, by a whole
// warp: 32 starts a step (one read in sequence for up to 32 requests, two for up
// to 1024).
__device__ __forceinline__ int request_of_row(const TreeArgs & a, int row, int lane) {
    int lo = 0, n = a.batch;
    while (n > 1) {
        const int step = (n + 31) >> 5, at = lo + lane * step;
        const unsigned before = __ballot_sync(0xffffffffu, lane * step < n && a.cu[min(at, a.batch)] <= row);
        const int k = max(__popc(before) - 1, 0) * step;
        lo += k;
        n = min(step, n - k);
    }
    return lo;
}

// Programmatic dependent launch: the next kernel of the stream may start its
// prologue / the kernel in front is complete and its results are visible.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Block 0: the units before every request.  The others: one warp per (row,
// head), q~ = R q times a power of two that brings the row's largest
// coordinate into [1, 2) (from 2^127 on into [2, 4): the factor 2^-127 would be
// subnormal, and its bits here those of 0), so that fp16 neither overflows nor
// loses the row; q_mul carries the inverse, the softmax scale and log2 e.
template <int D>
__global__ void __launch_bounds__(kTpThreads) tree_prep_kernel(const __grid_constant__ TreeArgs a) {
    constexpr int E = D / 32, NW = kTpThreads / 32;
    __shared__ float x_s[NW][D];
    __shared__ int64_t sums[NW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    let_next_start();
    if (blockIdx.x == 0) {
        int64_t before = 0;
        for (int b0 = 0; b0 < a.batch; b0 += kTpThreads) {
            const int b = b0 + tid;
            int64_t n = 0;
            if (b < a.batch) {
                const Request q = request_of(a, b);
                n = (int64_t)a.n_kv_heads * sets_of(a, q.n) * tiles_of(q.len);
                if (a.status != nullptr && past_limits(a, b)) atomicOr(a.status, TQ_STATUS_LIMIT);
            }
            int64_t incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += u;
            }
            __syncthreads();
            if (lane == 31) sums[warp] = incl;
            __syncthreads();
            int64_t all = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                if (w < warp) incl += sums[w];
                all += sums[w];
            }
            if (b < a.batch) a.unit0[b] = before + incl - n;
            before += all;
        }
        if (tid == 0) a.unit0[a.batch] = before;
        return;
    }
    const int64_t vec = (int64_t)(blockIdx.x - 1) * NW + warp;
    if (vec >= (int64_t)a.n_rows * a.n_q_heads) return;
    const int row = (int)(vec / a.n_q_heads), h = (int)(vec - (int64_t)row * a.n_q_heads);
    const int b = request_of_row(a, row, lane);
    const Request q = request_of(a, b);
    const int node = row - q.r0;
    const bool is_row = node >= 0 && node < q.n;
    if (h == 0 && lane == 0) a.row_request[row] = is_row ? b : -1;
    if (!is_row) return;
    float v[E];
    if (a.dense) {
        for (int i = lane; i < D; i += 32) x_s[warp][i] = load_el(a.q, a.q_dtype, vec * D + i);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const float4 * r = reinterpret_cast<const float4 *>(a.rot_f32 + (int64_t)(E * lane + k) * D);
            float s = 0.0f;
            for (int i = 0; i < D / 4; ++i) {
                const float4 w = __ldg(r + i), x = reinterpret_cast<const float4 *>(x_s[warp])[i];
                s = fmaf(w.x, x.x, fmaf(w.y, x.y, fmaf(w.z, x.z, fmaf(w.w, x.w, s))));
            }
            v[k] = s;
        }
    } else {
        load_vec<E>(a.q, a.q_dtype, vec * D + E * lane, v);
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = signed_by(a.d2_bits, E * lane + k, v[k]);
        warp_fwht<E>(v, lane);
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = signed_by(a.d1_bits, E * lane + k, v[k]);
    }
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < E; ++k) top = fmaxf(top, fabsf(v[k]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    int e = (int)(__float_as_uint(top) >> 23) - 127;
    e = e == 128 ? 0 : min(max(e, -120), 126);           // (infinite or NaN rows stay so)
    const float f = __uint_as_float((uint32_t)(127 - e) << 23);
    const int hk = h / a.group, g = h - hk * a.group;
    const int64_t id = (int64_t)q.r0 * a.n_q_heads + (int64_t)hk * q.n * a.group + (int64_t)node * a.group + g;
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] *= f;
    store_vec<E>(a.q_rows, TQ_DTYPE_F16, id * D + E * lane, v);
    // (not 0, which times the -inf of a masked key is NaN; products with the
    // smallest normal number are below 2^-90 as well)
    if (lane == 0) a.q_mul[id] = fmaxf(a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23), 0x1p-126f);
}

// ---------------------------------------------------------------------------
// Unpacking
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, __half2 b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), b);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// 8 codes of a block (their nibbles in `x`) -> 4 fp16 pairs, times `norm`.
// TOP: codes above 7 exist (4 bits); bit 3 of a code chooses between the
// lookups in the lower and the upper half of the table.
template <bool TOP>
__device__ __forceinline__ uint4 lookup8(uint32_t x, const uint32_t * tab, __half2 norm) {
    const uint32_t sel = TOP ? x & 0x77777777u : x, x4 = TOP ? x << 4 : 0u;
    uint32_t o[4];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const uint32_t s = p ? sel >> 16 : sel;
        uint32_t lo = __byte_perm(tab[0], tab[1], s), hi = __byte_perm(tab[4], tab[5], s);
        if constexpr (TOP) {
            uint32_t m;      // byte i: bit 3 of code i, replicated
            if (p == 0) asm("prmt.b32 %0, %1, %2, 0xD9C8;" : "=r"(m) : "r"(x4), "r"(x));
            else asm("prmt.b32 %0, %1, %2, 0xFBEA;" : "=r"(m) : "r"(x4), "r"(x));
            lo = (__byte_perm(tab[2], tab[3], s) & m) | (lo & ~m);
            hi = (__byte_perm(tab[6], tab[7], s) & m) | (hi & ~m);
        }
        o[2 * p] = hmul2_u(__byte_perm(lo, hi, 0x5140), norm);
        o[2 * p + 1] = hmul2_u(__byte_perm(lo, hi, 0x7362), norm);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Block `blk` of a row of an operand buffer: BITS words (the first of w), the
// norm twice.
template <int BITS>
__device__ __forceinline__ void unpack_block(const uint32_t * w, uint32_t nn, const uint32_t * tab, unsigned char * dst, int blk,
                                             int swz) {
    const __half2 norm = *reinterpret_cast<const __half2 *>(&nn);
    dst += (blk >> 1) * (kTile * 128);
    const int c0 = (4 * (blk & 1)) ^ swz;                // 16-byte chunk of the 128-byte row, swizzled
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t x;
        if constexpr (BITS == 4) {
            x = w[k];
        } else if constexpr (BITS == 3) {
            // 24 bits -> 8 nibbles (a step keeps the lower part and takes the rest
            // from the shifted word; what it takes too much the last step drops)
            const int wi = 24 * k / 32, sh = 24 * k % 32;
            x = sh + 24 <= 32 ? w[wi] >> sh : __funnelshift_r(w[wi], w[wi < 2 ? wi + 1 : 2], sh);
            x = (x & 0x00000FFFu) | ((x * 16u) & ~0x00000FFFu);
            x = (x & 0x003F003Fu) | ((x * 4u) & ~0x003F003Fu);
            x = (x & 0x07070707u) | ((x * 2u) & 0x70707070u);
        } else {
            // 16 bits -> 8 nibbles
            x = (w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu;
            x = (x | (x * 256u)) & 0x00FF00FFu;
            x = (x | (x * 16u)) & 0x0F0F0F0Fu;
            x = (x | (x * 4u)) & 0x33333333u;
        }
        *reinterpret_cast<uint4 *>(dst + 16 * (c0 ^ k)) = lookup8<BITS == 4>(x, tab, norm);
    }
}

// A row: NB blocks, U of them to a pass of the loop.  One at a time the words move
// down a register per block; unrolled, the three widths are 30 KB of instructions.
// Beside one row tile that gains (16 trees over up to 32K tokens 133 -> 128 us, four
// with d = 256 76 -> 75), beside two, whose softmax fills the rest of the cycles, it
// loses (8 trees over 128K tokens 1.21 -> 1.34 ms).
template <int BITS, int NB, int U>
__device__ __forceinline__ void unpack_row(uint32_t * w, const uint32_t * norms, const uint32_t * tab, unsigned char * dst, int swz) {
    uint64_t n = norms[0];
    if constexpr (NB == 4) n |= (uint64_t)norms[1] << 32;
#pragma unroll U
    for (int blk = 0; blk < NB; ++blk) {
        unpack_block<BITS>(w, __byte_perm((uint32_t)n, 0u, 0x1010), tab, dst, blk, swz);
        n >>= 16;
#pragma unroll
        for (int i = 0; i + BITS < BITS * NB; ++i) w[i] = w[i + BITS];
    }
}

// The bits of a row's mask for 32 consecutive tokens, the first of them node j0
// (negative: that many tokens before the nodes, which every node attends).
__device__ __forceinline__ uint32_t mask32(const TreeArgs & a, const uint64_t * words, int node, int j0) {
    if (j0 <= -32) return 0xFFFFFFFFu;
    uint32_t bits;
    if (words != nullptr) {
        const int from = max(j0, 0), w = from >> 6;
        if (w >= a.mask_words) return 0u;
        uint64_t x = words[w] >> (from & 63);
        if ((from & 63) > 32 && w + 1 < a.mask_words) x |= words[w + 1] << (64 - (from & 63));
        bits = (uint32_t)x;
    } else {
        const int c = node + 1 - max(j0, 0);             // nodes 0 .. node
        bits = c >= 32 ? 0xFFFFFFFFu : c <= 0 ? 0u : (1u << c) - 1u;
    }
    return j0 >= 0 ? bits : (bits << -j0) | ((1u << -j0) - 1u);
}

// ---------------------------------------------------------------------------
// The key tiles
// ---------------------------------------------------------------------------

template <int D, int MODE>
struct TaCfg {
    static constexpr int WGS = MODE == WIDE ? 1 : 2;     // softmax warpgroups
    static constexpr int NH = D == 256 ? 2 : 1;          // buffers of a key or value tile
    static constexpr int W = D / NH;                     // columns of a buffer
    static constexpr int NB = W / 32;                    // norm blocks of a buffer's row
    static constexpr int SLICE = kTile * 128;            // 64 columns of 128 rows
    static constexpr int BUF = W / 64 * SLICE;
    static constexpr int QT = MODE == PAIR ? 2 : 1;      // row tiles
    // one ring of key buffers and one of value buffers; STREAM: three of values,
    // so that a thread that takes every other tile sees each buffer's uses in order
    static constexpr int OFF_RING = QT * NH * BUF;
    static constexpr int NK = D == 64 ? 4 : 2, NV = D == 64 ? 4 : MODE == STREAM ? 3 : 2;
    static constexpr int STAGES = NK + NV;
    static constexpr int THREADS = 128 * (WGS + 3);      // softmax, unpacking keys and values, the issuing threads
    // packed rows on their way, one thread a row: codes as 4 chunks x 128 threads
    // x CHUNK bytes, the norms, and (keys) the norms of the values
    static constexpr int CHUNK = 4 * NB, NORMS = 2 * NB;
    static constexpr int OFF_PACKED = OFF_RING + STAGES * BUF;
    static constexpr int PACKED = kTile * (4 * CHUNK + 2 * NORMS);
    // mbarriers: full[STAGES], empty[STAGES], s_full[2][2], p_full[2][2],
    // o_done[2][2], o_last[2], o_free[2], s_free[2], drained[2], q_full, q_free
    static constexpr int OFF_BAR = OFF_PACKED + 2 * PACKED;
    static constexpr int N_BAR = 2 * STAGES + 22;
    static constexpr int OFF_BAD = (OFF_BAR + 8 * N_BAR + 15) / 16 * 16;    // 8 tiles x 128 bits: keys with a bad norm
    static constexpr int OFF_MISC = OFF_BAD + 128;                           // TMEM address, error flag, first request
    static constexpr int SMEM = OFF_MISC + 16 + 1024;                       // + alignment of the base
    static_assert(SMEM <= 232448, "shared memory of a CTA");
    // registers a thread: 96 at launch (640 threads) or 128 (512)
    static constexpr int R_SOFTMAX = WGS == 2 ? 136 : 168;
    static constexpr int R_UNPACK = WGS == 2 ? 80 : 120;
    static constexpr int R_MMA = WGS == 2 ? 48 : 104;
    static constexpr int R_LAUNCH = WGS == 2 ? 96 : 128;
    static_assert(WGS * R_SOFTMAX + 2 * R_UNPACK + R_MMA <= (WGS + 3) * R_LAUNCH, "no more than the launch holds");
};

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }

// Asynchronous copy of N bytes into shared memory, zeros where !live.
template <int N>
__device__ __forceinline__ void copy_or_zero(uint32_t dst, const void * src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" :: "r"(dst), "l"(src), "n"(N), "r"(live ? N : 0) : "memory");
}

template <int D, int MODE>
__global__ void __launch_bounds__(TaCfg<D, MODE>::THREADS, 1) tree_kernel(const __grid_constant__ TreeArgs a,
                                                                           const __grid_constant__ CUtensorMap qmap) {
    using C = TaCfg<D, MODE>;
    constexpr int WGS = C::WGS, NH = C::NH, NB = C::NB, ST = C::STAGES;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char * smem = smem_raw + (sbase - raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t full = sbase + (uint32_t)C::OFF_BAR, empty = full + 8u * ST, s_full = empty + 8u * ST,
                   p_full = s_full + 32u, o_done = p_full + 32u, o_last = o_done + 32u, o_free = o_last + 16u,
                   s_free = o_free + 16u, drained = s_free + 16u, q_full = drained + 16u, q_free = q_full + 8u;
    volatile uint32_t * s_bad = reinterpret_cast<volatile uint32_t *>(smem + C::OFF_BAD);
    uint32_t * s_tmem = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int * s_err = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    int * s_first = reinterpret_cast<int *>(smem + C::OFF_MISC + 8);

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            tc::mbar_init(full + 8u * i, 4);
            tc::mbar_init(empty + 8u * i, MODE == PAIR ? 2 : 1);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(s_full + 8u * i, 1);
            tc::mbar_init(p_full + 8u * i, 128);
            tc::mbar_init(o_done + 8u * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(o_last + 8u * i, 1);
            tc::mbar_init(o_free + 8u * i, 128);
            tc::mbar_init(s_free + 8u * i, 1);
            tc::mbar_init(drained + 8u * i, 1);
        }
        tc::mbar_init(q_full, 1);
        tc::mbar_init(q_free, MODE == WIDE ? 1 : 2);
        *s_err = 0;
    }
    if (warp == 0) tc::tmem_alloc(sbase + (uint32_t)C::OFF_MISC, 512);
    let_next_start();
    wait_for_previous();
    {
        // the request of this CTA's first unit
        const int64_t units = a.unit0[a.batch], u0 = first_unit(blockIdx.x, units, sharers(a, units));
        for (int b = tid; b < a.batch; b += C::THREADS)
            if (a.unit0[b] <= u0 && u0 < a.unit0[b + 1]) *s_first = b;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);
    PartIter it;
    it.start(a, *s_first);
    Part p;

    if (warp >= 4 * (WGS + 2)) {
        regs_down<C::R_MMA>();
        // ---- MMAs, issued by two threads (as in the prompt kernel): PAIR and
        // STREAM one per score slot, WIDE one for the scores and one for the
        // products; a third warp loads the row tiles ----
        const int t = warp - 4 * (WGS + 2);
        if (t == 2 && lane == 0) {
            // (the rotated rows were written by plain stores of the kernel in front)
            asm volatile("fence.proxy.async;" ::: "memory");
            bool ok = true;
            for (int part = 0; ok && it.next(a, p); ++part) {
                if (part > 0) ok = fm::wait(q_free, (uint32_t)((part - 1) & 1));
                if (!ok) break;
                const int tiles = MODE == PAIR && p.rows > kTile ? 2 : 1;
                tc::mbar_arrive_expect_tx(q_full, (uint32_t)(tiles * (D / 64) * C::SLICE));
                for (int i = 0; i < tiles; ++i)
                    for (int c = 0; c < D / 64; ++c)
                        tc::tma_load_2d(sbase + (uint32_t)((i * (D / 64) + c) * C::SLICE), &qmap, 64 * c,
                                        (int)p.row_id + i * kTile, q_full);
                // (also before this thread ends)
                ok = fm::wait(q_full, (uint32_t)(part & 1));
            }
            if (!ok) *s_err = 1;
        } else if (t < 2) {
            const uint32_t lead = fm::elected();
            constexpr uint32_t id_qk = fm::idesc(false, kTile, false), id_qk64 = fm::idesc(false, 64, false),
                               id_pv = fm::idesc(false, C::W, true);
            const uint64_t ring_desc = tc::smem_desc_sw128(sbase + (uint32_t)C::OFF_RING);
            const uint64_t v_desc = fm::smem_desc_sw128_mn(sbase + (uint32_t)C::OFF_RING, (uint32_t)C::SLICE);
            // scores of row tile i and the columns h of the key tile in buffer b
            // into slot s, keys from row `key` of the tile on
            auto qk = [&](int i, int s, int h, uint32_t b, int key, uint32_t id) {
                const uint64_t qd = fm::opaque(tc::smem_desc_sw128(sbase + (uint32_t)((i * NH + h) * C::BUF)));
                const uint64_t kd = ring_desc + (uint64_t)(b * (uint32_t)(C::BUF >> 4) + 8u * (uint32_t)key);
#pragma unroll
                for (int ks = 0; ks < C::W / 16; ++ks) {
                    const uint64_t off = (uint64_t)(((ks >> 2) * C::SLICE + (ks & 3) * 32) >> 4);
                    fm::mma_ss(lead, tmem + (uint32_t)s * fm::kSlotCols + (uint32_t)key, qd + off, kd + off, id, h > 0 || ks > 0 ? 1u : 0u);
                }
            };
            // weights of half g of slot s times the columns h of the value tile in
            // buffer b onto accumulator w
            auto pv = [&](int w, int s, int h, uint32_t b, int g, bool acc) {
                const uint64_t vd = v_desc + (uint64_t)(b * (uint32_t)(C::BUF >> 4) + 512u * (uint32_t)g);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    fm::mma_ts(lead, tmem + fm::kOutCol + (uint32_t)(w * D + h * C::W),
                               tmem + (uint32_t)s * fm::kSlotCols + (uint32_t)g * fm::kHalfCols + 8u * k, vd + 128u * k, id_pv,
                               acc || k > 0 ? 1u : 0u);
            };
            fm::Ring<C::NK> kr;                              // the next key and value buffer
            fm::Ring<C::NV> vr;
            const uint32_t v_full = full + 8u * C::NK, v_empty = empty + 8u * C::NK;
            bool ok = true;
            uint32_t use = 0, finished = 0;                  // key tiles and parts of this thread so far
            const uint32_t sf = s_full + 16u * t, pf = p_full + 16u * t, od = o_done + 16u * t;
            for (int part = 0; ok && it.next(a, p); ++part) {
                // (every part in turn, also one that this thread has no share in)
                ok = fm::wait_warp(q_full, (uint32_t)(part & 1));
                if (!ok) break;
                if constexpr (MODE != WIDE) {
                    // Slot t: PAIR row tile t against every key tile; STREAM the one row
                    // tile against the key tiles t, t + 2, ...; the buffers between are
                    // the other thread's, and filled in order, so that the buffer waited
                    // for is at its use or the one before.
                    const bool takes = MODE == PAIR ? t * kTile < p.rows : t < p.tiles;
                    const int i = MODE == PAIR ? t : 0, stride = MODE == PAIR ? 1 : 2;
                    if (!takes) {
                        for (int j = 0; j < p.tiles && ok; ++j) {
                            if constexpr (MODE == PAIR) {
                                ok = fm::wait_warp(full + 8u * kr.at, kr.parity);
                                if (lane == 0) tc::mbar_arrive(empty + 8u * kr.at);
                                ok = ok && fm::wait_warp(v_full + 8u * vr.at, vr.parity);
                                if (lane == 0) tc::mbar_arrive(v_empty + 8u * vr.at);
                            }
                            kr.step();
                            vr.step();
                        }
                        if (lane == 0) tc::mbar_arrive(q_free);
                        continue;
                    }
                    if (MODE == STREAM && t == 1) {
                        kr.step();
                        vr.step();
                    }
                    ok = fm::wait_warp(full + 8u * kr.at, kr.parity);
                    if (!ok) break;
                    tc::fence_after_sync();
                    for (int g = 0; g < 2; ++g) {
                        qk(i, t, 0, kr.at, 64 * g, id_qk64);
                        fm::commit(lead, sf + 8u * g);
                    }
                    fm::commit(lead, empty + 8u * kr.at);
                    bool first = true;
                    int j = MODE == STREAM ? t : 0;
                    for (; j < p.tiles; j += stride) {
                        const bool more = j + stride < p.tiles;
                        if (!more) fm::commit(lead, q_free);     // (behind the part's last scores)
                        kr.step();                               // to key tile j + stride
                        if (MODE == STREAM && j + 1 < p.tiles) kr.step();
                        ok = fm::wait_warp(v_full + 8u * vr.at, vr.parity);
                        if (more) ok = ok && fm::wait_warp(full + 8u * kr.at, kr.parity);
                        // the accumulator of the part before has been read
                        if (first && finished > 0) ok = ok && fm::wait_warp(o_free + 8u * t, (finished - 1) & 1u);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            ok = ok && fm::wait_warp(pf + 8u * g, use & 1u);
                            if (!ok) break;
                            tc::fence_after_sync();
                            pv(t, t, 0, C::NK + vr.at, g, !first || g > 0);
                            if (more) {
                                qk(i, t, 0, kr.at, 64 * g, id_qk64);
                                fm::commit(lead, sf + 8u * g);
                            }
                            fm::commit(lead, od + 8u * g);
                        }
                        if (!ok) break;
                        fm::commit(lead, v_empty + 8u * vr.at);
                        if (more) fm::commit(lead, empty + 8u * kr.at);
                        vr.step();
                        if (MODE == STREAM && j + 1 < p.tiles) vr.step();
                        first = false;
                        ++use;
                    }
                    if (!ok) break;
                    fm::commit(lead, o_last + 8u * t);
                    ++finished;
                } else if (t == 0) {
                    for (int j = 0; j < p.tiles && ok; ++j, ++use) {
                        // slot use & 1 is free behind the products of two tiles before
                        if (use > 1) ok = fm::wait_warp(s_free + 8u * (use & 1u), ((use >> 1) - 1) & 1u);
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            ok = ok && fm::wait_warp(full + 8u * kr.at, kr.parity);
                            if (!ok) break;
                            tc::fence_after_sync();
                            qk(0, (int)(use & 1u), h, kr.at, 0, id_qk);
                            fm::commit(lead, empty + 8u * kr.at);
                            kr.step();
                        }
                        if (!ok) break;
                        for (int g = 0; g < 2; ++g) fm::commit(lead, s_full + 8u * (2 * (use & 1u) + g));
                        if (j + 1 == p.tiles) fm::commit(lead, q_free);
                    }
                } else {
                    for (int j = 0; j < p.tiles && ok; ++j, ++use) {
                        uint32_t b[NH];
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            b[h] = vr.at;
                            ok = ok && fm::wait_warp(v_full + 8u * vr.at, vr.parity);
                            vr.step();
                        }
                        if (j == 0 && finished > 0) ok = ok && fm::wait_warp(o_free, (finished - 1) & 1u);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            ok = ok && fm::wait_warp(p_full + 16u * (use & 1u) + 8u * g, (use >> 1) & 1u);
                            if (!ok) break;
                            tc::fence_after_sync();
#pragma unroll
                            for (int h = 0; h < NH; ++h) {
                                pv(0, (int)(use & 1u), h, C::NK + b[h], g, j > 0 || g > 0);
                                if (g == 1) fm::commit(lead, v_empty + 8u * b[h]);
                            }
                            fm::commit(lead, o_done + 8u * g);
                        }
                        if (ok) fm::commit(lead, s_free + 8u * (use & 1u));
                    }
                    if (!ok) break;
                    fm::commit(lead, o_last);
                    ++finished;
                }
            }
            if (!ok) {
                // the MMAs in flight end before their columns are freed
                *s_err = 1;
                fm::commit(lead, drained + 8u * t);
                fm::wait_warp(drained + 8u * t, 0u);
            }
        }
        __syncwarp();
    } else if (warp >= 4 * WGS) {
        // ---- unpacking: one warpgroup the keys, one the values (side by side
        // rather than on the same tile, so that one looks up while the other waits
        // or copies); thread r has row r of every buffer ----
        regs_down<C::R_UNPACK>();
        const int r = tid & (kTile - 1);
        const bool values = warp >= 4 * (WGS + 1);
        const int bits = values ? a.v_bits : a.k_bits;
        const uint32_t * codes = values ? a.v_codes : a.k_codes;
        const uint16_t * norms = values ? a.v_norms : a.k_norms;
        uint32_t tab[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) tab[i] = values ? a.v_table[i] : a.k_table[i];
        const uint32_t packed = sbase + (uint32_t)(C::OFF_PACKED + (values ? C::PACKED : 0));
        const unsigned char * src = smem + C::OFF_PACKED + (values ? C::PACKED : 0);
        const uint32_t ring0 = values ? C::NK : 0u, n_ring = values ? C::NV : C::NK;

        // Cache row of this thread's token in key tile `tile` of the part, kNone
        // past the last token (32 bits: the host refuses larger storage); its page
        // was read a tile earlier, the read takes a while.
        constexpr uint32_t kNone = 0xFFFFFFFFu;
        int page = 0;
        auto read_page = [&](int tile) {
            const int t = (p.tile0 + tile) * kTile + r;
            if (tile < p.tiles && t < p.rq.len) page = __ldg(a.table + (int64_t)p.b * a.max_pages + (t >> a.page_shift));
        };
        auto tile_row = [&](int tile) {
            const int t = (p.tile0 + tile) * kTile + r;
            const uint32_t pg = (uint32_t)min(max(page, 0), a.n_pages - 1);
            return t >= p.rq.len ? kNone
                                 : ((pg * (uint32_t)a.n_kv_heads + (uint32_t)p.hk) << a.page_shift) +
                                       ((uint32_t)t & ((1u << a.page_shift) - 1u));
        };
        // The packed words and norms of a buffer's row on their way into shared
        // memory; every thread reads back only what it copied itself.
        auto fetch = [&](uint32_t row, int half) {
            const bool live = row != kNone;
            const uint64_t at = live ? row : 0u;
            const uint32_t * c = codes + at * (uint32_t)(D / 32 * bits) + (uint32_t)(half * NB * bits);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < bits) copy_or_zero<C::CHUNK>(packed + (uint32_t)((i * kTile + r) * C::CHUNK), c + i * NB, live);
            const uint64_t nat = at * (D / 32) + (uint32_t)(half * NB);
            const uint32_t nd = packed + (uint32_t)(kTile * 4 * C::CHUNK + r * C::NORMS);
            copy_or_zero<C::NORMS>(nd, norms + nat, live);
            if (!values) copy_or_zero<C::NORMS>(nd + (uint32_t)(kTile * C::NORMS), a.v_norms + nat, live);
        };
        uint32_t row = kNone;
        int step = 0, half = 0, tile = 0;                // step, half: of the item on its way
        bool more = it.next(a, p);
        auto start_part = [&] {
            step = 0;
            read_page(0);
            row = tile_row(0);
            read_page(1);
        };
        if (more) {
            start_part();
            fetch(row, 0);
        }
        uint32_t at = 0, parity = 1;                     // buffer of the ring, parity of its last release
        while (more) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            uint32_t w[4 * NB], norm[NB / 2], other[NB / 2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (NB == 4) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(src + (i * kTile + r) * 16);
                    w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(src + (i * kTile + r) * 8);
                    w[2 * i] = x.x; w[2 * i + 1] = x.y;
                }
            }
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) {
                const uint32_t * n = reinterpret_cast<const uint32_t *>(src + kTile * 4 * C::CHUNK + r * C::NORMS) + i;
                norm[i] = n[0];
                other[i] = n[kTile * C::NORMS / 4];
            }
            // a key with an infinite or NaN norm marks its readers' sums, and takes
            // no part in the products
            uint32_t bad = 0u;
#pragma unroll
            for (int i = 0; i < NB / 2; ++i)
                bad |= ((norm[i] & 0x7C007C00u) + 0x04000400u) | (values ? 0u : (other[i] & 0x7C007C00u) + 0x04000400u);
            bad &= 0x80008000u;
            const int this_half = half;
            if (!values) {
                const uint32_t keys = __ballot_sync(0xffffffffu, bad != 0u);
                if (lane == 0) {
                    volatile uint32_t * word = s_bad + 4 * (tile & 7) + (warp - 4 * WGS);
                    *word = this_half == 0 ? keys : *word | keys;
                }
                if (this_half == NH - 1) ++tile;
            }
            if (bad != 0u) {
#pragma unroll
                for (int i = 0; i < NB / 2; ++i) norm[i] = 0u;
            }
            // the next item
            if (NH == 2 && half == 0) {
                half = 1;
            } else {
                half = 0;
                if (++step < p.tiles) {
                    row = tile_row(step);
                    read_page(step + 1);
                } else {
                    more = it.next(a, p);
                    if (more) start_part();
                }
            }
            if (more) fetch(row, half);
            // (a fresh barrier counts as released: its phase before the first has parity 1)
            const uint32_t s = ring0 + at;
            const bool ok = fm::wait(empty + 8u * s, parity);
            if (!__all_sync(0xffffffffu, ok)) {
                *s_err = 1;
                break;
            }
            unsigned char * dst = smem + C::OFF_RING + s * C::BUF + r * 128;
            constexpr int U = MODE == PAIR ? 1 : NB;
            if (bits == 4) unpack_row<4, NB, U>(w, norm, tab, dst, r & 7);
            else if (bits == 3) unpack_row<3, NB, U>(w, norm, tab, dst, r & 7);
            else unpack_row<2, NB, U>(w, norm, tab, dst, r & 7);
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(full + 8u * s);
            if (++at == n_ring) {
                at = 0;
                parity ^= 1u;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ---- softmax: warpgroup w, one thread per row ----
        regs_up<C::R_SOFTMAX>();
        const int w = warp >> 2;
        const int r = tid & 127;
        const uint32_t lane_tm = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t o_tm = lane_tm + fm::kOutCol + (uint32_t)(w * D);
        bool ok = true;
        int tile0 = 0;                       // key tiles of the parts before
        int mine = 0, done = 0;              // tiles and parts that this warpgroup has done
        while (ok && it.next(a, p)) {
            const int in_set = MODE == PAIR ? w * kTile + r : r;       // row of the set
            const bool valid = in_set < p.rows;
            const bool takes = MODE == PAIR ? w * kTile < p.rows : MODE == STREAM ? w < p.tiles : true;
            const int64_t id = p.row_id + in_set;
            const bool own = p.tile0 == 0;
            const int slot_row = w * kTile + r;
            const int64_t part_row = own ? (MODE == STREAM ? w * a.own_rows : 0) + id : (int64_t)blockIdx.x * a.more_rows + slot_row;
            float2 * ml = (own ? a.own_ml : a.more_ml) + part_row;
            if (!takes) {
                if (MODE == STREAM && valid) *ml = make_float2(-CUDART_INF_F, 0.0f);
                tile0 += p.tiles;
                continue;
            }
            const int in_req = p.set * a.rows_per_set + in_set;
            const int node = in_req / a.group;
            const uint64_t * words = a.mask != nullptr && valid ? a.mask + (int64_t)(p.rq.r0 + node) * a.mask_words : nullptr;
            const float mul = valid ? a.q_mul[id] : 0.0f;
            const int ctx0 = p.rq.ctx;                                 // tokens before the nodes
            const bool warp_valid = (MODE == PAIR ? w * kTile : 0) + (r & ~31) < p.rows;
            fm::RowState st{-CUDART_INF_F, 0.0f};
            bool first = true;
            for (int j = MODE == STREAM ? w : 0; j < p.tiles && ok; j += MODE == STREAM ? 2 : 1) {
                const int slot = MODE == WIDE ? (tile0 + j) & 1 : w;
                const uint32_t use = MODE == WIDE ? (uint32_t)(tile0 + j) >> 1 : (uint32_t)mine;
                const int t0 = (p.tile0 + j) * kTile;
                const bool edge = t0 + kTile > ctx0;
                uint32_t allowed[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
                if (edge && warp_valid) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int c = p.rq.len - (t0 + 32 * x);    // tokens left
                        const uint32_t in = c >= 32 ? 0xFFFFFFFFu : c <= 0 ? 0u : (1u << c) - 1u;
                        allowed[x] = valid ? in & (in != 0u ? mask32(a, words, node, t0 + 32 * x - ctx0) : 0u) : 0u;
                    }
                }
#pragma unroll 1
                for (int g = 0; g < 2; ++g) {
                    // (the scores that follow in this half wait for these weights)
                    const bool scored = fm::wait(s_full + 8u * (2 * slot + g), use & 1u);
                    ok = __all_sync(0xffffffffu, ok && scored);
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (warp_valid) {
                        // products so far: half 1 of the tile before -- its scores were behind
                        // those of the tile in front, or WIDE two in front -- then, in this
                        // half 1, those of half 0
                        auto scale_acc = [&](float f) {
                            bool r = first || fm::wait(o_done + 8u * (2 * w + 1), (uint32_t)((mine - 1) & 1));
                            if (g == 1) r = r && fm::wait(o_done + 8u * (2 * w), (uint32_t)(mine & 1));
                            // (the accumulator's loads and stores want a converged warp, and the
                            // votes that follow the same answer in all its lanes)
                            r = __all_sync(0xffffffffu, r);
                            fm::rescale(o_tm, D, f);
                            return r;
                        };
                        const uint32_t half = lane_tm + (uint32_t)slot * fm::kSlotCols + (uint32_t)g * fm::kHalfCols;
                        const uint32_t al[2] = {g == 0 ? allowed[0] : allowed[2], g == 0 ? allowed[1] : allowed[3]};
                        if (edge) ok = fm::softmax_half<false, true>(half, first && g == 0, mul, al, st, scale_acc);
                        else ok = fm::softmax_half<false, false>(half, first && g == 0, mul, nullptr, st, scale_acc);
                        const volatile uint32_t * bad = s_bad + 4 * ((tile0 + j) & 7) + 2 * g;
                        if (((bad[0] & al[0]) | (bad[1] & al[1])) != 0u) st.sum = CUDART_NAN_F;
                    }
                    tc::mbar_arrive(p_full + 8u * (2 * slot + g));
                }
                first = false;
                ++mine;
            }
            tile0 += p.tiles;
            ok = ok && fm::wait(o_last + 8u * w, (uint32_t)(done & 1));
            ++done;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc::fence_after_sync();
            if (warp_valid) {
                float * dst = own ? a.own : a.more;
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    fm::tmem_ld32(o_tm + (uint32_t)c, o);
                    if (valid) {
#pragma unroll
                        for (int x = 0; x < 32; x += 4)
                            *reinterpret_cast<uint4 *>(dst + part_at<D>(part_row, c + x)) = make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
                    }
                }
                if (valid) *ml = part_ml(st.ref, st.sum);
            }
            tc::fence_before_sync();
            tc::mbar_arrive(o_free + 8u * w);
        }
        if (!ok) *s_err = 1;
    }
    __syncthreads();
    tc::fence_after_sync();
    if (*s_err != 0 && tid == 0 && a.status != nullptr) atomicOr(a.status, TQ_STATUS_TIMEOUT);
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Few rows: at most 8 rows share a key tile (single tokens, small groups)
// ---------------------------------------------------------------------------

// A tile of 128 rows would be nearly empty, and its unpacking into shared memory
// the whole cost.  Here every warp streams 16 tokens at a time for itself and
// unpacks them into the registers of m16n8k16 MMAs, which hold the tokens (or
// the output coordinates) in their 16 rows and the query rows in their 8 columns:
//
//   scores: A = 16 tokens x 16 coordinates of keys, lane 4 g + t with tokens g,
//     g + 8 and the coordinates t D/4 .. (t + 1) D/4 - 1, a run of the packed row;
//   values: A = 16 coordinates x 16 tokens, lane 4 g + t with the coordinates
//     4 g .. 4 g + 3 of each block and the tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9;
//     B = the weights, transposed by movmatrix.
//
// Pairs of codes become pairs of fp16 centroids by one shared-memory lookup (a
// copy of the table per lane, so no two lanes meet in a bank), times the norm.
// The units are shared among the warps of the grid as they are among its CTAs
// elsewhere.
//
// 64 single tokens over 1 .. 32K tokens (133 MB of packed rows, 20 us of HBM time):
// 66 us, 214 us with tree_kernel.  Bound by the issue slots (77 % busy: some 600
// instructions per 16 tokens, a third of them lookups); the ring keeps three
// slabs a warp on their way.
template <int D>
struct FewCfg {
    static constexpr int NB = D / 32, SEG = D / 4;       // blocks; coordinates of a lane's run of keys
    static constexpr int WARPS = D == 256 ? 8 : 16;
    static constexpr int STAGES = 3;
    static constexpr int SLAB = 16 * (2 * D / 2 + 4 * NB);   // packed bytes of 16 tokens at 4 bits: codes, norms
    static constexpr int OFF_VC = 16 * D / 2, OFF_KN = 2 * OFF_VC, OFF_VN = OFF_KN + 32 * NB;
    static constexpr int OFF_RING = 2 * 256 * 128;       // behind the two tables
    static constexpr int SMEM = OFF_RING + WARPS * STAGES * SLAB;
    static_assert(SMEM <= 232448, "shared memory of a CTA");
};

__device__ __forceinline__ void mma_16816(float * d, const uint32_t * a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// The pair tables: entry e (two codes, the first in its low bits) at byte 256 e,
// keys in the lower half, values in the upper, one word a lane.  Offset of the
// pair at bit `sh` of x: the pair's bits at bit 8 on, the lane's word below; for
// 4-bit codes, whose pairs are bytes, one byte permute.
template <int BITS>
__device__ __forceinline__ uint32_t pair_at(uint32_t x, int sh, uint32_t lane4) {
    if constexpr (BITS == 4) {
        return __byte_perm(x, lane4, 0x7704u | ((uint32_t)(sh >> 3) << 4));
    } else {
        constexpr uint32_t MASK = ((1u << (2 * BITS)) - 1u) << 8;
        return ((sh >= 8 ? x >> (sh - 8) : x << (8 - sh)) & MASK) | lane4;
    }
}

// Scores of 16 tokens: acc += keys x queries.  `codes`: the slab's packed keys,
// qf: the lane's query words (B fragments in order).
template <int D, int BITS>
__device__ __forceinline__ void few_scores(float * acc, const unsigned char * codes, const __half * norms, const uint32_t * qf,
                                           const unsigned char * tables, uint32_t lane4, int g, int t) {
    constexpr int NB = D / 32, SEG = D / 4, ROW = D / 8 * BITS;
    constexpr int PIECE = SEG < 32 ? SEG : 32;           // codes taken at a time: a block, or half of one
#pragma unroll
    for (int b = 0; b < SEG / PIECE; ++b) {
        const int blk = D == 64 ? t >> 1 : t * (SEG / 32) + b;
        uint32_t w[2][BITS + 1];
        __half2 norm[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t * row = reinterpret_cast<const uint32_t *>(codes + (g + 8 * r) * ROW) + blk * BITS;
#pragma unroll
            for (int i = 0; i < BITS; ++i) w[r][i] = row[i];
            w[r][BITS] = 0u;
            if (D == 64 && (t & 1)) {                     // the second half of the block
#pragma unroll
                for (int i = 0; i < BITS; ++i) {
                    const int lo = i + BITS / 2;
                    w[r][i] = lo < BITS ? (BITS % 2 ? __funnelshift_r(w[r][lo], w[r][lo + 1 <= BITS ? lo + 1 : BITS], 16) : w[r][lo]) : 0u;
                }
            }
            norm[r] = __half2half2(norms[(g + 8 * r) * NB + blk]);
        }
#pragma unroll
        for (int k = 0; k < PIECE / 4; ++k) {             // 4 codes of each token: one MMA
            uint32_t a[4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int bit = 2 * BITS * (2 * k + h), wi = bit >> 5, sh = bit & 31;
                    const uint32_t at = sh + 2 * BITS <= 32 ? pair_at<BITS>(w[r][wi], sh, lane4)
                                                            : pair_at<BITS>(__funnelshift_r(w[r][wi], w[r][wi + 1], sh - 8), 8, lane4);
                    a[2 * h + r] = hmul2_u(*reinterpret_cast<const uint32_t *>(tables + at), norm[r]);
                }
            mma_16816(acc, a, qf[2 * (b * (PIECE / 4) + k)], qf[2 * (b * (PIECE / 4) + k) + 1]);
        }
    }
}

// Output of 16 tokens: o += values x weights (b0, b1: the lane's weights).
template <int D, int BITS>
__device__ __forceinline__ void few_values(float (*o)[4], const unsigned char * codes, const __half * norms, uint32_t b0, uint32_t b1,
                                           const unsigned char * tables, uint32_t lane4, int g, int t) {
    constexpr int NB = D / 32, ROW = D / 8 * BITS;
    const int bit = 4 * BITS * g, wi = bit >> 5, sh = bit & 31;       // the lane's 4 codes of a block
    // norms of the four tokens, all blocks, two to a word
    uint32_t nw[4][NB / 2];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < NB / 2; ++i)
            nw[k][i] = reinterpret_cast<const uint32_t *>(norms + (2 * t + (k & 1) + 8 * (k >> 1)) * NB)[i];
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
        uint32_t lo[4], hi[4];                            // (coordinate 0, 1) and (2, 3) of the four tokens
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int tok = 2 * t + (k & 1) + 8 * (k >> 1);
            const uint32_t * row = reinterpret_cast<const uint32_t *>(codes + tok * ROW) + blk * BITS;
            uint32_t x = row[wi];
            if (BITS == 3) x = __funnelshift_r(x, row[min(wi + 1, 2)], sh);
            else x >>= sh;
            lo[k] = *reinterpret_cast<const uint32_t *>(tables + 128 + pair_at<BITS>(x, 0, lane4));
            hi[k] = *reinterpret_cast<const uint32_t *>(tables + 128 + pair_at<BITS>(x, 2 * BITS, lane4));
        }
        uint32_t a0[4], a1[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {                     // tokens 2 t, 2 t + 1; then those 8 on
            const uint32_t nn = __byte_perm(nw[2 * h][blk >> 1], nw[2 * h + 1][blk >> 1], blk & 1 ? 0x7632 : 0x5410);
            const __half2 norm = *reinterpret_cast<const __half2 *>(&nn);
            a0[2 * h] = hmul2_u(__byte_perm(lo[2 * h], lo[2 * h + 1], 0x5410), norm);
            a0[2 * h + 1] = hmul2_u(__byte_perm(lo[2 * h], lo[2 * h + 1], 0x7632), norm);
            a1[2 * h] = hmul2_u(__byte_perm(hi[2 * h], hi[2 * h + 1], 0x5410), norm);
            a1[2 * h + 1] = hmul2_u(__byte_perm(hi[2 * h], hi[2 * h + 1], 0x7632), norm);
        }
        mma_16816(o[2 * blk], a0, b0, b1);
        mma_16816(o[2 * blk + 1], a1, b0, b1);
    }
}

template <int D>
__global__ void __launch_bounds__(32 * FewCfg<D>::WARPS, 1) tree_few_kernel(const __grid_constant__ TreeArgs a) {
    using C = FewCfg<D>;
    constexpr int NB = C::NB;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    let_next_start();
    // the pair tables
    for (int i = threadIdx.x; i < 2 * 256 * 32; i += 32 * C::WARPS) {
        const bool v = (i & 32) != 0;
        const int e = i >> 6, bits = v ? a.v_bits : a.k_bits;
        const uint32_t * tab = v ? a.v_table : a.k_table;
        auto entry = [&](int c) {
            return ((tab[c >> 2] >> (8 * (c & 3))) & 0xFFu) | ((tab[4 + (c >> 2)] >> (8 * (c & 3))) & 0xFFu) << 8;
        };
        reinterpret_cast<uint32_t *>(smem)[i] = entry(e & ((1 << bits) - 1)) | entry((e >> bits) & ((1 << bits) - 1)) << 16;
    }
    wait_for_previous();
    __syncthreads();
    const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t lane4 = 4u * (uint32_t)lane;
    const uint32_t ring = (uint32_t)(C::OFF_RING + warp * C::STAGES * C::SLAB);

    // this warp's units
    const int64_t units = a.unit0[a.batch], n = sharers(a, units);
    const int worker = blockIdx.x * C::WARPS + warp;
    PartIter it;
    it.u = first_unit(worker, units, n);
    it.end = first_unit(worker + 1, units, n);
    if (it.u >= it.end) return;
    {
        // the request of the first one
        int lo = 0, len = a.batch;
        while (len > 1) {
            const int step = (len + 31) >> 5, at = lo + lane * step;
            const unsigned before = __ballot_sync(0xffffffffu, lane * step < len && a.unit0[min(at, a.batch)] <= it.u);
            const int k = max(__popc(before) - 1, 0) * step;
            lo += k;
            len = min(step, len - k);
        }
        it.b = lo;
    }
    Part p;
    while (it.next(a, p)) {
        const int t0 = p.tile0 * kTile, n_slabs = (min(p.rq.len - t0, p.tiles * kTile) + 15) >> 4;
        const int ctx0 = p.rq.ctx;
        // 16 tokens lie in one page, one behind the other; the page of the slab to
        // be fetched next was read a slab earlier
        int page = 0;
        auto read_page = [&](int s) {
            if (s < n_slabs) page = __ldg(a.table + (int64_t)p.b * a.max_pages + ((t0 + 16 * s) >> a.page_shift));
        };
        auto fetch = [&](int s) {
            if (s < n_slabs) {
                const uint32_t pg = (uint32_t)min(max(page, 0), a.n_pages - 1);
                const uint64_t row = ((pg * (uint32_t)a.n_kv_heads + (uint32_t)p.hk) << a.page_shift) +
                                     ((uint32_t)(t0 + 16 * s) & ((1u << a.page_shift) - 1u));
                const uint32_t dst = sbase + ring + (uint32_t)((s % C::STAGES) * C::SLAB);
                const int kb = 2 * D * a.k_bits, vb = 2 * D * a.v_bits;          // bytes of codes
                const unsigned char * kc = reinterpret_cast<const unsigned char *>(a.k_codes) + row * (uint32_t)(D / 8 * a.k_bits);
                const unsigned char * vc = reinterpret_cast<const unsigned char *>(a.v_codes) + row * (uint32_t)(D / 8 * a.v_bits);
#pragma unroll
                for (int i = 0; i < (8 * D + 511) / 512; ++i) {
                    const int at = 512 * i + 16 * lane;
                    if (at < kb) tc::cp_async16(dst + (uint32_t)at, kc + at);
                    if (at < vb) tc::cp_async16(dst + (uint32_t)(C::OFF_VC + at), vc + at);
                }
                if (lane < 2 * NB) {
                    tc::cp_async16(dst + (uint32_t)(C::OFF_KN + 16 * lane), reinterpret_cast<const unsigned char *>(a.k_norms + row * NB) + 16 * lane);
                    tc::cp_async16(dst + (uint32_t)(C::OFF_VN + 16 * lane), reinterpret_cast<const unsigned char *>(a.v_norms + row * NB) + 16 * lane);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int s = 0; s < C::STAGES; ++s) {
            read_page(s);
            fetch(s);
        }
        read_page(C::STAGES);

        // queries: row g, the lane's run of coordinates
        uint32_t qf[D / 8];
        if (g < p.rows) {
            const uint4 * q = reinterpret_cast<const uint4 *>(a.q_rows + (p.row_id + g) * D + t * C::SEG);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 u = q[i];
                qf[4 * i] = u.x; qf[4 * i + 1] = u.y; qf[4 * i + 2] = u.z; qf[4 * i + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) qf[i] = 0u;
        }
        // this lane's columns of the scores and of the output: rows 2 t and 2 t + 1
        float mul[2], ref[2] = {-CUDART_INF_F, -CUDART_INF_F}, sum[2] = {0.0f, 0.0f};
        int node[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = 2 * t + c;
            mul[c] = r < p.rows ? a.q_mul[p.row_id + r] : 0.0f;
            node[c] = (p.set * a.rows_per_set + min(r, p.rows - 1)) / a.group;
        }
        float o[2 * NB][4];
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;

        for (int s = 0; s < n_slabs; ++s) {
            asm volatile("cp.async.wait_group %0;" :: "n"(C::STAGES - 1) : "memory");
            __syncwarp();
            unsigned char * slab = smem + ring + (s % C::STAGES) * C::SLAB;
            const __half * kn = reinterpret_cast<const __half *>(slab + C::OFF_KN);
            const __half * vn = reinterpret_cast<const __half *>(slab + C::OFF_VN);
            // tokens with an infinite or NaN norm: their readers' sums are marked, and
            // they take no part in the products
            unsigned bad = 0u;
            {
                uint32_t x = 0u;
                const uint32_t * kw = reinterpret_cast<const uint32_t *>(kn) + (lane & 15) * (NB / 2);
                const uint32_t * vw = reinterpret_cast<const uint32_t *>(vn) + (lane & 15) * (NB / 2);
                for (int i = 0; i < NB / 2; ++i) x |= ((kw[i] & 0x7C007C00u) + 0x04000400u) | ((vw[i] & 0x7C007C00u) + 0x04000400u);
                bad = __ballot_sync(0xffffffffu, lane < 16 && (x & 0x80008000u) != 0u);
                if (__builtin_expect(bad != 0u, 0)) {
                    if ((bad >> lane) & 1u)
                        for (int i = 0; i < NB / 2; ++i) {
                            reinterpret_cast<uint32_t *>(slab + C::OFF_KN)[lane * (NB / 2) + i] = 0u;
                            reinterpret_cast<uint32_t *>(slab + C::OFF_VN)[lane * (NB / 2) + i] = 0u;
                        }
                    __syncwarp();
                }
            }
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};        // tokens g, g + 8 (k >> 1) of rows 2 t, 2 t + 1 (k & 1)
            if (a.k_bits == 4) few_scores<D, 4>(x, slab, kn, qf, smem, lane4, g, t);
            else if (a.k_bits == 3) few_scores<D, 3>(x, slab, kn, qf, smem, lane4, g, t);
            else few_scores<D, 2>(x, slab, kn, qf, smem, lane4, g, t);
            const int tok0 = t0 + 16 * s;
            if (__builtin_expect(tok0 + 16 > ctx0 || bad != 0u, 0)) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int tok = tok0 + g + 8 * (k >> 1), nd = node[k & 1];
                    bool ok = tok < p.rq.len;
                    if (ok && tok >= ctx0) {
                        const uint64_t * words = a.mask != nullptr ? a.mask + (int64_t)(p.rq.r0 + nd) * a.mask_words : nullptr;
                        ok = (mask32(a, words, nd, tok - ctx0) & 1u) != 0u;
                    }
                    if (!ok) x[k] = -CUDART_INF_F;
                    else if ((bad >> (g + 8 * (k >> 1))) & 1u) sum[k & 1] = CUDART_NAN_F;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] *= mul[k & 1];
            // (a row with multiplier 0 is none: -inf times 0 stays in its own column)
            const bool raise = fmaxf(x[0], x[2]) > ref[0] + fm::kLazy || fmaxf(x[1], x[3]) > ref[1] + fm::kLazy;
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = fmaxf(x[c], x[2 + c]);
#pragma unroll
                    for (int i = 4; i < 32; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
                    if (top > ref[c] + fm::kLazy) {
                        const float f = ref[c] == -CUDART_INF_F ? 0.0f : fm::ex2(ref[c] - top);
                        ref[c] = top;
                        sum[c] *= f;
#pragma unroll
                        for (int i = 0; i < 2 * NB; ++i) {
                            o[i][c] *= f;
                            o[i][2 + c] *= f;
                        }
                    }
                }
            }
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float rf = ref[k & 1];
                w[k] = fm::ex2(x[k] - (rf == -CUDART_INF_F ? 0.0f : rf) + fm::kShift<false>);
                sum[k & 1] += w[k];
            }
            const uint32_t b0 = transpose_8x8(fm::pack2<false>(w[0], w[1])), b1 = transpose_8x8(fm::pack2<false>(w[2], w[3]));
            const unsigned char * vc = slab + C::OFF_VC;
            if (a.v_bits == 4) few_values<D, 4>(o, vc, vn, b0, b1, smem, lane4, g, t);
            else if (a.v_bits == 3) few_values<D, 3>(o, vc, vn, b0, b1, smem, lane4, g, t);
            else few_values<D, 2>(o, vc, vn, b0, b1, smem, lane4, g, t);
            __syncwarp();                                 // the slab has been read
            fetch(s + C::STAGES);
            read_page(s + C::STAGES + 1);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        const bool own = p.tile0 == 0;
        float * parts = own ? a.own : a.more;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float total = sum[c];
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) total += __shfl_xor_sync(0xffffffffu, total, i);
            const int r = 2 * t + c;
            if (r >= p.rows) continue;
            const int64_t at = own ? p.row_id + r : (int64_t)worker * a.more_rows + r;
            if (g == 0) (own ? a.own_ml : a.more_ml)[at] = part_ml(ref[c], total);
#pragma unroll
            for (int b = 0; b < NB; ++b)
                *reinterpret_cast<float4 *>(parts + part_at<D>(at, 32 * b + 4 * g)) =
                    make_float4(o[2 * b][c], o[2 * b][2 + c], o[2 * b + 1][c], o[2 * b + 1][2 + c]);
        }
    }
}

// ---------------------------------------------------------------------------
// Merge and rotation back: R rows a CTA
// ---------------------------------------------------------------------------

constexpr int kTmThreads = 256;

// First the lanes of a warp have R rows and 32 / R groups of four columns, so
// that the parts are read as they were written (part_at); the sums meet in shared
// memory, and the warps rotate the rows back.  R = 8 where few rows share a key
// tile: their parts are many (one per warp of the grid that shared the tiles), so
// more CTAs read them, eight reads of a thread at a time (rotation and
// merge of 64 single tokens: 36 us with R = 32, 20 us with 8).  R = 8 also where
// an SM gets no more than one such CTA (the call for 5 nodes of 8 heads, with the
// dense rotation: 22.6 us with 32, 20.5 with 8); with more rows 32 is the faster
// one (620 nodes of 16 heads, d = 256: 69 us against 72).
template <int D, int R>
__global__ void __launch_bounds__(kTmThreads) tree_combine_kernel(const __grid_constant__ TreeArgs a) {
    constexpr int E = D / 32, NW = kTmThreads / 32, GP = 32 / R, LD = D + 4, RW = R / NW;
    constexpr int CH = D / 4 >= NW * GP ? D / 4 / (NW * GP) : 1;
    __shared__ __align__(16) float y_s[R][LD];
    __shared__ int64_t out_s[R];                         // where a row's output starts, -1: no row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int my_row = lane % R, my_col = 4 * (warp * GP + lane / R);      // and every 4 NW GP columns on
    const bool active = my_col < D;
    const int64_t id = (int64_t)blockIdx.x * R + my_row;
    wait_for_previous();
    // the row: its request, place in the request, and parts
    int64_t dst = -1, u0 = 0;
    int tiles = 0, in_set = 0;
    if (id < (int64_t)a.n_rows * a.n_q_heads) {
        const int b = a.row_request[(uint32_t)id / (uint32_t)a.n_q_heads];
        if (b >= 0) {
            const Request q = request_of(a, b);
            const int rem = (int)id - q.r0 * a.n_q_heads;    // (rows times heads fit 30 bits)
            if (rem >= 0 && rem < q.n * a.n_q_heads) {
                const int per = q.n * a.group, hk = rem / per, in_req = rem - hk * per;
                const int node = in_req / a.group, set = in_req / a.rows_per_set;
                in_set = in_req - set * a.rows_per_set;
                tiles = tiles_of(q.len);
                u0 = a.unit0[b] + ((int64_t)hk * sets_of(a, q.n) + set) * tiles;
                dst = ((int64_t)(q.r0 + node) * a.n_q_heads + hk * a.group + in_req - node * a.group) * D;
            }
        }
    }
    if (warp == 0 && lane < R) out_s[lane] = dst;
    const int64_t units = a.unit0[a.batch], n = sharers(a, units);
    int c0 = 0, c1 = -1;                                 // the CTAs that share the row's tiles
    if (tiles > 0) {
        c0 = cta_of(u0, units, n);
        c1 = cta_of(u0 + tiles - 1, units, n);
    }
    // its parts, U at a time: their reads do not wait for one another
    constexpr int U = R == 8 ? 8 : D == 256 ? 2 : 4;
    const int n_parts = active ? (c1 - c0 + 1) * a.streams : 0;
    float ref = -CUDART_INF_F, sum = 0.0f;
    float4 acc[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p0 = 0; p0 < n_parts; p0 += U) {
        float2 ml[U];
        float4 x[U][CH];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ml[u] = make_float2(-CUDART_INF_F, 0.0f);
            if (p0 + u < n_parts) {
                const int at_c = a.streams == 2 ? (p0 + u) >> 1 : p0 + u, s = a.streams == 2 ? (p0 + u) & 1 : 0;
                const int64_t at = at_c == 0 ? s * a.own_rows + id : (int64_t)(c0 + at_c) * a.more_rows + s * kTile + in_set;
                const float * parts = at_c == 0 ? a.own : a.more;
                ml[u] = (at_c == 0 ? a.own_ml : a.more_ml)[at];
#pragma unroll
                for (int k = 0; k < CH; ++k) x[u][k] = *reinterpret_cast<const float4 *>(parts + part_at<D>(at, my_col + 4 * NW * GP * k));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (ml[u].x == -CUDART_INF_F) continue;      // no key attended (what its part holds is not read)
            const float top = fmaxf(ref, ml[u].x);       // (a NaN stays in the sums)
            const float fa = ref == -CUDART_INF_F ? 0.0f : fm::ex2(ref - top), fb = fm::ex2(ml[u].x - top);
            ref = top;
            sum = sum * fa + ml[u].y * fb;
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                acc[k].x = acc[k].x * fa + x[u][k].x * fb;
                acc[k].y = acc[k].y * fa + x[u][k].y * fb;
                acc[k].z = acc[k].z * fa + x[u][k].z * fb;
                acc[k].w = acc[k].w * fa + x[u][k].w * fb;
            }
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // a node that attends nothing: zeros
#pragma unroll
    for (int k = 0; k < CH; ++k) acc[k] = make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv);
    // (a row marked by a NaN sum is NaN whatever its parts hold)
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        if (isnan(sum)) acc[k] = make_float4(sum, sum, sum, sum);
        if (active) *reinterpret_cast<float4 *>(&y_s[my_row][my_col + 4 * NW * GP * k]) = acc[k];
    }
    __syncthreads();
    if (a.dense) {
        float x[RW][E];
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int k = 0; k < E; ++k) x[r][k] = 0.0f;
        for (int e = 0; e < D; ++e) {
            float y[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r) y[r] = y_s[RW * warp + r][e];
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float w = __ldg(a.rot_f32 + (int64_t)e * D + 32 * k + lane);
#pragma unroll
                for (int r = 0; r < RW; ++r) x[r][k] = fmaf(w, y[r], x[r][k]);
            }
        }
#pragma unroll
        for (int r = 0; r < RW; ++r)
            if (out_s[RW * warp + r] >= 0)
#pragma unroll
                for (int k = 0; k < E; ++k) store_el(a.out, a.q_dtype, out_s[RW * warp + r] + 32 * k + lane, x[r][k]);
    } else {
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const int64_t to = out_s[RW * warp + r];
            if (to < 0) continue;
            float v[E];
#pragma unroll
            for (int k = 0; k < E; ++k) v[k] = signed_by(a.d1_bits, E * lane + k, y_s[RW * warp + r][E * lane + k]);
            warp_fwht<E>(v, lane);
#pragma unroll
            for (int k = 0; k < E; ++k) v[k] = signed_by(a.d2_bits, E * lane + k, v[k]);
            store_vec<E>(a.out, a.q_dtype, to + E * lane, v);
        }
    }
}

// A launch that may start while the kernel in front of it is still running.
template <typename K, typename... Args>
int launch_dependent(K kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t st, const Args &... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int MODE>
int launch_tree_main(const TreeArgs & a, cudaStream_t st) {
    using C = TaCfg<D, MODE>;
    CUtensorMap qmap;
    if (!encode_tensor_map_2d(&qmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.q_rows, (uint64_t)D,
                              (uint64_t)a.n_rows * a.n_q_heads, (uint64_t)D * 2, 64u, (uint32_t)kTile,
                              CU_TENSOR_MAP_SWIZZLE_128B))
        return (int)cudaErrorInvalidValue;
    auto k = tree_kernel<D, MODE>;
    // a build that gives the kernel fewer registers would wait for good where the
    // softmax warps take theirs
    static const int regs = [] {
        cudaFuncAttributes fa{};
        return cudaFuncGetAttributes(&fa, tree_kernel<D, MODE>) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs < C::R_LAUNCH) return (int)cudaErrorInvalidConfiguration;
    if (int e = ensure_dynamic_smem(reinterpret_cast<const void *>(k), C::SMEM)) return e;
    return launch_dependent(k, (unsigned)a.n_ctas, C::THREADS, C::SMEM, st, a, qmap);
}

template <int D>
int launch_tree(TreeArgs & a, cudaStream_t st) {
    const unsigned vecs = (unsigned)(((int64_t)a.n_rows * a.n_q_heads + 7) / 8);
    tree_prep_kernel<D><<<vecs + 1, kTpThreads, 0, st>>>(a);
    if (int e = (int)cudaGetLastError()) return e;
    int e;
    if (a.rows_per_set == kFewRows) {
        using C = FewCfg<D>;
        auto k = tree_few_kernel<D>;
        if (int f = ensure_dynamic_smem(reinterpret_cast<const void *>(k), C::SMEM)) return f;
        e = launch_dependent(k, (unsigned)(a.n_ctas / C::WARPS), 32 * C::WARPS, C::SMEM, st, a);
    } else if constexpr (D == 256) e = launch_tree_main<D, WIDE>(a, st);
    else e = a.streams == 2 ? launch_tree_main<D, STREAM>(a, st) : launch_tree_main<D, PAIR>(a, st);
    if (e) return e;
    // (a.n_ctas: the SMs, or their warps)
    return a.own_rows <= 8 * (int64_t)a.n_ctas || a.rows_per_set == kFewRows ? launch_dependent(tree_combine_kernel<D, 8>, (unsigned)(a.own_rows / 8), kTmThreads, 0, st, a)
                                      : launch_dependent(tree_combine_kernel<D, 32>, (unsigned)(a.own_rows / 32), kTmThreads, 0, st, a);
}

int64_t own_rows_of(int64_t vecs) { return (vecs + 31) / 32 * 32; }

// Workspace sections, each from a 256-byte boundary.
struct TreeSpace {
    size_t unit0, row_request, q_rows, q_mul, own, own_ml, more, more_ml, total;
};
TreeSpace tree_space(int64_t batch, int64_t n_rows, int64_t vecs, int d, int n_ctas) {
    TreeSpace s;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    s.unit0 = take((size_t)(batch + 1) * 8);
    s.row_request = take((size_t)n_rows * 4);
    s.q_rows = take((size_t)vecs * d * 2);
    s.q_mul = take((size_t)vecs * 4);
    s.own = take((size_t)own_rows_of(vecs) * 2 * d * 4);
    s.own_ml = take((size_t)own_rows_of(vecs) * 2 * 8);
    // (16 warps with 8 rows each take half of what two row tiles do)
    s.more = take((size_t)n_ctas * 2 * kTile * d * 4);
    s.more_ml = take((size_t)n_ctas * 2 * kTile * 8);
    s.total = at;
    return s;
}

// fp16 bits of the centroids as byte tables (entries above 2^bits - 1 repeat the last)
void centroid_table(const CodebookParams & cb, int bits, uint32_t * tab) {
    for (int i = 0; i < 8; ++i) tab[i] = 0u;
    for (int i = 0; i < 16; ++i) {
        const __half_raw h = __float2half_rn(cb.centroid[i < (1 << bits) ? i : (1 << bits) - 1]);
        tab[i >> 2] |= (uint32_t)(h.x & 0xFFu) << (8 * (i & 3));
        tab[4 + (i >> 2)] |= (uint32_t)(h.x >> 8) << (8 * (i & 3));
    }
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
    else if (max_len > INT32_MAX - 255) *why = "max_len above 2^31 - 256";
    return *why == nullptr;
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" size_t tq_tree_workspace_size(int32_t batch, int32_t n_rows, int32_t max_nodes, int32_t n_q_heads,
                                         int32_t n_kv_heads, int64_t max_len, int32_t head_dim) {
    const char * why;
    if (!tree_sizes_ok(batch, n_rows, max_nodes, n_q_heads, n_kv_heads, max_len, head_dim, &why)) return 0;
    return tree_space(batch, n_rows, (int64_t)n_rows * n_q_heads, head_dim, device_sm_count()).total;
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
    if ((int64_t)n_pages * n_kv_heads > (int64_t)(0xFFFFFFFFu / (uint32_t)page_size))
        return fail(TQ_ERR_UNSUPPORTED, "2^32 cache rows or more");
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
    a.k_bits = k_bits;
    a.v_bits = v_bits;
    centroid_table(kcb, k_bits, a.k_table);
    centroid_table(vcb, v_bits, a.v_table);
    a.group = n_q_heads / n_kv_heads;
    a.n_ctas = device_sm_count();
    const bool few = (int64_t)max_nodes * a.group <= kFewRows;
    a.streams = !few && head_dim < 256 && (int64_t)max_nodes * a.group <= kTile ? 2 : 1;
    a.rows_per_set = few ? kFewRows : head_dim < 256 && a.streams == 1 ? 2 * kTile : kTile;
    a.more_rows = few ? kFewRows : 2 * kTile;
    unsigned char * ws = static_cast<unsigned char *>(workspace);
    const TreeSpace sp = tree_space(batch, n_rows, (int64_t)n_rows * n_q_heads, head_dim, a.n_ctas);
    if (few) a.n_ctas *= head_dim == 256 ? FewCfg<256>::WARPS : FewCfg<128>::WARPS;
    a.unit0 = reinterpret_cast<int64_t *>(ws + sp.unit0);
    a.row_request = reinterpret_cast<int32_t *>(ws + sp.row_request);
    a.q_rows = reinterpret_cast<__half *>(ws + sp.q_rows);
    a.q_mul = reinterpret_cast<float *>(ws + sp.q_mul);
    a.own_rows = own_rows_of((int64_t)n_rows * n_q_heads);
    a.own = reinterpret_cast<float *>(ws + sp.own);
    a.own_ml = reinterpret_cast<float2 *>(ws + sp.own_ml);
    a.more = reinterpret_cast<float *>(ws + sp.more);
    a.more_ml = reinterpret_cast<float2 *>(ws + sp.more_ml);
    a.out = out;
    a.status = status_dev;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int e = head_dim == 64 ? launch_tree<64>(a, s) : head_dim == 128 ? launch_tree<128>(a, s) : launch_tree<256>(a, s);
    return cuda_status(e, "tree attention launch");
}
