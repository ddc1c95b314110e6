// Causal attention of packed sequences over their unquantized keys and values
// (tq_prompt_attention), on the tensor cores.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = 2^(mul <q_i, k_j> - ref_i),   j <= i + nk - nq
//
// A CTA takes one or two tiles of 128 rows of one sequence and one KV head.  A
// row is a (query, head of the group) pair, heads inner, so a tile holds
// 128 / GP consecutive queries: grouped heads share every key tile that is
// loaded, and the tiles cut by the causal edge are GP times fewer.  Key and
// value tiles (128 keys) arrive by TMA into one ring of buffers, from the last
// key tile to the first; two threads issue the MMAs, one softmax thread per row
// reads its scores from TMEM and writes the weights back over them (tq_fmha.cuh).
//
//  d <= 128: two row tiles; the tensor core works on one tile while the
//    softmax warps of the other run, and the pair shares the key ring.
//  d = 256: one row tile (its accumulator fills half of TMEM); the scores of
//    key tile j + 1 are computed into the second slot during the softmax of j.
//    The head dimension is cut into halves of 128 columns, one buffer each.
//
// Values at keys that a row may not attend meet a zero weight, which a NaN or
// an infinity would turn into NaN.  Such pairs exist only in the tiles at the
// causal edge and at the sequence's end.  There a warp looks over the value
// tile before the second product: rows past the sequence are zeroed, and a
// non-finite value inside it makes the CTA compute its rows again on the CUDA
// cores, with the keys that a row attends and no others.
//
// What bounds it (8192 tokens, 32 / 8 heads, d = 128, bf16: 0.418 ms on the same
// inputs again and again, 1.32 PFLOP/s, 0.80 of the measured burst rate of a GEMM;
// 0.494 ms on inputs that change, 1.11 PFLOP/s, 0.79 of its sustained rate): the
// issue and wake-up latencies between the softmax and the tensor core, whose pipe is
// active 66 % of the cycles; leaving the exponentials out gains 4 %, half the score
// products 10 %.  Taking turns between the two issuing threads cost 7 %, score tiles
// of 128 keys at once (instead of two halves) 13 %.  Short sequences are bound by a
// block's way in and out, 4 us of loads, one softmax and the stores that nothing
// overlaps (16 prompts of 64 .. 2048 tokens: 0.161 ms on the same inputs, of which
// 0.06 ms; 0.176 ms on inputs that change).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <climits>
#include <cmath>
#include <type_traits>

#include "tq_device.cuh"
#include "tq_fmha.cuh"

namespace tq {
namespace {

using fm::kTile;

constexpr int kPaMaxHeads = 32;      // heads of a group in one row tile

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
    int32_t heads, queries;          // GP; queries of a row tile (128 / GP)
    float scale;
    void * out;
    uint32_t * status;
};

template <int D>
struct PaCfg {
    static constexpr int NQ = D == 256 ? 1 : 2;          // row tiles of a CTA
    static constexpr int NH = D == 256 ? 2 : 1;          // buffers of a key or value tile
    static constexpr int W = D / NH;                     // columns of a buffer
    static constexpr int SLICE = kTile * 128;            // 64 columns of 128 rows
    static constexpr int BUF = W / 64 * SLICE;
    static constexpr int STAGES = D == 64 ? 8 : 5;
    static constexpr int THREADS = 128 * NQ + 128;
    static constexpr int OFF_KV = NQ * NH * BUF;
    static constexpr int OFF_BAR = OFF_KV + STAGES * BUF;
    // mbarriers: q, full[STAGES], empty[STAGES], s_full[2][2], p_full[2][2],
    // o_done[2][2], o_last[2], s_free[2], drained[2], scanned; then the
    // TMEM address, error and redo flags, the tile, and the sums of the search
    // for it
    static constexpr int N_BAR = 2 * STAGES + 20;
    static constexpr int OFF_MISC = OFF_BAR + 8 * N_BAR;
    static constexpr int SMEM = OFF_MISC + 32 + 4 * (THREADS / 32) + 1024;   // + alignment of the base
    static_assert(SMEM <= 232448, "shared memory of a CTA");
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16 * o) { *o = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(float x, __half * o) { *o = __float2half_rn(x); }

__device__ __forceinline__ int clamp_to(int x, int lo, int hi) { return min(max(x, lo), hi); }

// One row by one warp on the CUDA cores: the first n keys from row k0 on.
template <int D, typename T>
__device__ __noinline__ void prompt_row(const PromptArgs & a, int64_t tok, int h, int hk, int64_t k0, int64_t n) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float q[E], o[E];
    const T * qp = static_cast<const T *>(a.q) + tok * a.q_stride + (int64_t)h * D;
    for (int e = 0; e < E; ++e) {
        q[e] = to_f32(qp[lane + 32 * e]) * a.scale;
        o[e] = 0.0f;
    }
    float m = -CUDART_INF_F, l = 0.0f;
    for (int64_t j = k0; j < k0 + n; ++j) {
        const T * kp = static_cast<const T *>(a.k) + j * a.k_stride + (int64_t)hk * D;
        const T * vp = static_cast<const T *>(a.v) + j * a.v_stride + (int64_t)hk * D;
        float s = 0.0f;
        for (int e = 0; e < E; ++e) s = fmaf(q[e], to_f32(kp[lane + 32 * e]), s);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s);
        // (a score of -inf has weight 0, also in front of the first finite one; a
        // row with no other divides 0 by 0)
        const float c = m == -CUDART_INF_F ? 0.0f : expf(m - mn);
        const float p = s == -CUDART_INF_F && mn == s ? 0.0f : expf(s - mn);
        m = mn;
        l = l * c + p;
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * to_f32(vp[lane + 32 * e]);
    }
    T * op = static_cast<T *>(a.out) + (tok * a.n_q_heads + h) * D;
    for (int e = 0; e < E; ++e) from_f32(n > 0 ? o[e] / l : 0.0f, op + lane + 32 * e);
}

// Out of line: rare, and away from the softmax's instructions.
template <int D>
__device__ __noinline__ void scale_row(uint32_t o_tm, float f) { fm::rescale(o_tm, D, f); }

template <int D, bool BF16>
__global__ void __launch_bounds__(PaCfg<D>::THREADS, 1)
prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap qmap,
              const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using C = PaCfg<D>;
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    constexpr int NQ = C::NQ, NH = C::NH, SW = C::W / 64, ST = C::STAGES, NT = C::THREADS;
    extern __shared__ unsigned char smem_raw[];
    // the swizzled tiles need 1024-byte alignment
    const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char * smem = smem_raw + (sbase - raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t bar = sbase + (uint32_t)C::OFF_BAR;
    const uint32_t q_full = bar, full = bar + 8u, empty = full + 8u * ST, s_full = empty + 8u * ST,
                   p_full = s_full + 32u, o_done = p_full + 32u, o_last = o_done + 32u, s_free = o_last + 16u,
                   drained = s_free + 16u, scanned = drained + 16u;
    uint32_t * s_tmem = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int * s_err = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    volatile int * s_redo = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 8);
    int * s_seq = reinterpret_cast<int *>(smem + C::OFF_MISC + 12);      // sequence, tile
    int * s_sums = reinterpret_cast<int *>(smem + C::OFF_MISC + 32);

    const int ctrl = warp - 4 * NQ;                       // 0 and 3: MMAs, 1: copies, 2: value scan

    // Barriers (by the thread that copies, which is the first to use them) and
    // TMEM first, beside the search for the tile.
    if (ctrl == 1 && lane == 0) {
        tc::mbar_init(q_full, 1);
        for (int i = 0; i < ST; ++i) {
            tc::mbar_init(full + 8u * i, 1);
            tc::mbar_init(empty + 8u * i, NQ);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(s_full + 8u * i, 1);
            tc::mbar_init(p_full + 8u * i, 128);
            tc::mbar_init(o_done + 8u * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(o_last + 8u * i, 1);
            tc::mbar_init(s_free + 8u * i, 1);
            tc::mbar_init(drained + 8u * i, 1);
        }
        tc::mbar_init(scanned, 32);
        *s_err = 0;
        *s_redo = 0;
        s_seq[0] = -1;
    }
    if (warp == 0) tc::tmem_alloc(sbase + (uint32_t)C::OFF_MISC, 512);
    if (ctrl == 1 && lane < 3)
        asm volatile("prefetch.tensormap [%0];" :: "l"(lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap) : "memory");

    // Which sequence and tile: the tiles of all sequences are counted one sequence
    // after another, a sequence's last tile first (it has the most keys); blocks of
    // one tile and all heads follow each other.
    const int n_groups = a.n_q_heads / a.heads;
    const int tau = (int)(blockIdx.x / (unsigned)n_groups);
    const int hg = (int)(blockIdx.x - (unsigned)tau * (unsigned)n_groups);
    const int cta_queries = NQ * a.queries;
    auto tiles_of = [&](int b) {
        if (b >= a.batch) return 0;
        const int r0 = clamp_to(a.cu_q[b], 0, (int)a.total_q), r1 = clamp_to(a.cu_q[b + 1], r0, (int)a.total_q);
        return (int)((unsigned)(r1 - r0 + cta_queries - 1) / (unsigned)cta_queries);
    };
    auto warp_scan = [&](int n) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += u;
        }
        return n;
    };
    // Query i attends the keys below i + shift + 1, counted from where the sequence
    // starts to where its offsets say that it ends, also behind the arrays: rows that
    // are there then attend the same keys as they would if all were.
    auto shift_of = [&](int b, int r0, int c0) { return (max(a.cu_k[b + 1], c0) - c0) - (max(a.cu_q[b + 1], r0) - r0); };
    int seq = -1, tile = 0, shift = 0;
    int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
    if (a.batch <= 128) {
        // every warp for itself, without a barrier
        int before = 0;
        for (int b0 = 0; b0 < a.batch && seq < 0; b0 += 32) {
            const int b = min(b0 + lane, a.batch - 1);
            const int r0 = clamp_to(a.cu_q[b], 0, (int)a.total_q), r1 = clamp_to(a.cu_q[b + 1], r0, (int)a.total_q);
            const int c0 = clamp_to(a.cu_k[b], 0, (int)a.total_k), c1 = clamp_to(a.cu_k[b + 1], c0, (int)a.total_k);
            const int nt = b0 + lane < a.batch ? (int)((unsigned)(r1 - r0 + cta_queries - 1) / (unsigned)cta_queries) : 0;
            const int end = before + warp_scan(nt);
            const unsigned hit = __ballot_sync(0xffffffffu, tau < end);
            if (hit != 0u) {
                const int at = __ffs((int)hit) - 1;
                seq = b0 + at;
                // (inside the sequence whatever the offsets are)
                tile = max(min(__shfl_sync(0xffffffffu, end, at) - 1 - tau, __shfl_sync(0xffffffffu, nt, at) - 1), 0);
                q0 = __shfl_sync(0xffffffffu, r0, at);
                q1 = __shfl_sync(0xffffffffu, r1, at);
                k0 = __shfl_sync(0xffffffffu, c0, at);
                k1 = __shfl_sync(0xffffffffu, c1, at);
                shift = __shfl_sync(0xffffffffu, shift_of(b, r0, c0), at);
            }
            before = __shfl_sync(0xffffffffu, end, 31);
        }
    } else {
        int before = 0;
        for (int b0 = 0; b0 < a.batch && before <= tau; b0 += NT) {
            const int n = tiles_of(b0 + tid);
            int end = warp_scan(n);
            __syncthreads();
            if (lane == 31) s_sums[warp] = end;
            __syncthreads();
            int all = 0;
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) {
                const int x = s_sums[w];
                if (w < warp) end += x;
                all += x;
            }
            end += before;
            if (tau < end && tau >= end - n) {
                s_seq[0] = b0 + tid;
                s_seq[1] = end - 1 - tau;
            }
            before += all;
        }
        __syncthreads();
        seq = s_seq[0];
        tile = s_seq[1];
        if (seq >= 0) {
            q0 = clamp_to(a.cu_q[seq], 0, (int)a.total_q);
            q1 = clamp_to(a.cu_q[seq + 1], q0, (int)a.total_q);
            k0 = clamp_to(a.cu_k[seq], 0, (int)a.total_k);
            k1 = clamp_to(a.cu_k[seq + 1], k0, (int)a.total_k);
            shift = shift_of(seq, q0, k0);
        }
    }
    const int nq = q1 - q0, nk = k1 - k0;
    const int i0 = tile * cta_queries;                    // first query of this CTA
    const int i_last = min(i0 + cta_queries, nq) - 1;
    const int n_keys = min(max(i_last + shift + 1, 0), nk);
    // key tiles, taken from the last to the first; none past the last row tile
    const int n = seq < 0 ? 0 : (n_keys + kTile - 1) / kTile;
    const int full_keys = min(max(i0 + shift + 1, 0), nk);    // keys that every row attends
    const int n_edge = n - full_keys / kTile;             // tiles with a key that some row does not attend
    const int slots = NQ == 2 && i0 + a.queries < nq ? 2 : 1;
    const int h0 = hg * a.heads, hk = h0 / (a.n_q_heads / a.n_kv_heads);

    // The copies into empty buffers start here, while the others meet.  Copy `it`:
    // the buffers of a key tile, then of its values.
    const int n_copies = 2 * NH * n;
    int last = n_copies;                                  // copies that were started
    auto copy_buffer = [&](int it) {
        const int j = it / (2 * NH), h = it % NH, s = it % ST;
        const CUtensorMap * map = (it / NH) % 2 == 0 ? &kmap : &vmap;
        tc::mbar_arrive_expect_tx(full + 8u * s, (uint32_t)C::BUF);
        for (int c = 0; c < SW; ++c)
            tc::tma_load_3d(sbase + (uint32_t)(C::OFF_KV + s * C::BUF + c * C::SLICE), map, 64 * (h * SW + c), hk,
                            k0 + (n - 1 - j) * kTile, full + 8u * s);
    };
    if (n > 0 && ctrl == 1 && lane == 0) {
        // queries: boxes of 64 columns, GP heads, 128 / GP tokens
        const uint32_t rows = (uint32_t)(a.heads * a.queries);
        tc::mbar_arrive_expect_tx(q_full, (uint32_t)slots * (D / 64) * rows * 128u);
        for (int i = 0; i < slots; ++i)
            for (int c = 0; c < D / 64; ++c)
                tc::tma_load_3d(sbase + (uint32_t)((i * (D / 64) + c) * C::SLICE), &qmap, 64 * c, h0,
                                q0 + i0 + i * a.queries, q_full);
        for (int it = 0; it < min(ST, n_copies); ++it) copy_buffer(it);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);

    if (n > 0 && ctrl == 1) {
        if (lane == 0) {
            bool ok = true;
            for (int it = ST; it < n_copies && ok; ++it) {
                ok = fm::wait(empty + 8u * (it % ST), (uint32_t)((it / ST - 1) & 1));
                if (ok) copy_buffer(it);
                else last = it;
            }
            if (!ok) *s_err = 1;
            // the last copy into every buffer lands before the CTA ends
            fm::wait(q_full, 0u);
            for (int t = max(0, last - ST); t < last; ++t)
                fm::wait(full + 8u * (t % ST), (uint32_t)((t / ST) & 1));
        }
        __syncwarp();
    } else if (n > 0 && (ctrl == 0 || ctrl == 3)) {
        // ---- MMAs, issued by two threads.  An MMA holds its thread about as long
        // as the tensor core works on it, a wait or a commit costs some 100 cycles
        // more; with two threads those of one overlap the products of the other
        // (8192-token prompt, d = 128: 0.579 ms with one thread, 0.475 ms with two;
        // 0.433 ms when the warps run converged, see fm::elected). ----
        const int t = ctrl == 0 ? 0 : 1;                  // (the same in all lanes)
        if (NQ == 1 || t < slots) {
            const uint32_t lead = fm::elected();
            constexpr uint32_t id_qk = fm::idesc(BF16, kTile, false), id_qk64 = fm::idesc(BF16, 64, false), id_pv = fm::idesc(BF16, C::W, true);
            const uint64_t kv_desc = tc::smem_desc_sw128(sbase + (uint32_t)C::OFF_KV);
            const uint64_t v_desc = fm::smem_desc_sw128_mn(sbase + (uint32_t)C::OFF_KV, (uint32_t)C::SLICE);
            // scores of row tile i and the columns h of the key tile in buffer b
            // into slot s, keys from row `key` of the tile on
            auto qk = [&](int i, int s, int h, uint32_t b, int key, uint32_t id) {
                const uint64_t qd = fm::opaque(tc::smem_desc_sw128(sbase + (uint32_t)((i * NH + h) * C::BUF)));
                const uint64_t kd = kv_desc + (uint64_t)(b * (uint32_t)(C::BUF >> 4) + 8u * (uint32_t)key);
#pragma unroll
                for (int ks = 0; ks < C::W / 16; ++ks) {
                    const uint64_t off = (uint64_t)(((ks >> 2) * C::SLICE + (ks & 3) * 32) >> 4);
                    fm::mma_ss(lead, tmem + (uint32_t)s * fm::kSlotCols + (uint32_t)key, qd + off, kd + off, id, h > 0 || ks > 0 ? 1u : 0u);
                }
            };
            // weights of half g of slot s times the columns h of the value tile in
            // buffer b onto accumulator i
            auto pv = [&](int i, int s, int h, uint32_t b, int g, bool acc) {
                const uint64_t vd = v_desc + (uint64_t)(b * (uint32_t)(C::BUF >> 4) + 512u * (uint32_t)g);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    fm::mma_ts(lead, tmem + fm::kOutCol + (uint32_t)(i * D + h * C::W),
                               tmem + (uint32_t)s * fm::kSlotCols + (uint32_t)g * fm::kHalfCols + 8u * k, vd + 128u * k, id_pv,
                               acc || k > 0 ? 1u : 0u);
            };
            bool ok = fm::wait_warp(q_full, 0u);
            fm::Ring<ST> ring;                            // the next buffer
            if constexpr (NQ == 2) {
                // thread t: row tile t.  The scores of a half come behind the
                // products that read the weights they overwrite.
                auto release = [&](uint32_t b) {              // for the other thread too, if it has no share
                    fm::commit(lead, empty + 8u * b);
                    if (slots == 1) fm::commit(lead, empty + 8u * b);
                };
                const uint32_t sf = s_full + 16u * t, pf = p_full + 16u * t, od = o_done + 16u * t;
                ok = ok && fm::wait_warp(full, 0u);
                if (ok) {
                    for (int g = 0; g < 2; ++g) {
                        qk(t, t, 0, 0u, 64 * g, id_qk64);
                        fm::commit(lead, sf + 8u * g);
                    }
                    release(0u);
                }
                ring.step();
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t v = ring.at, vp = ring.parity;
                    ring.step();
                    const uint32_t k = ring.at, kp = ring.parity;
                    ring.step();
                    const bool more = j + 1 < n;
                    ok = fm::wait_warp(full + 8u * v, vp);
                    if (j < n_edge) ok = ok && fm::wait_warp(scanned, (uint32_t)(j & 1));
                    if (more) ok = ok && fm::wait_warp(full + 8u * k, kp);
                    ok = ok && fm::wait_warp(pf, (uint32_t)(j & 1));
                    if (!ok) break;
                    tc::fence_after_sync();
                    pv(t, t, 0, v, 0, j > 0);
                    if (more) {
                        qk(t, t, 0, k, 0, id_qk64);
                        fm::commit(lead, sf);
                    }
                    fm::commit(lead, od);
                    ok = fm::wait_warp(pf + 8u, (uint32_t)(j & 1));
                    if (!ok) break;
                    tc::fence_after_sync();
                    pv(t, t, 0, v, 1, true);
                    if (more) {
                        qk(t, t, 0, k, 64, id_qk64);
                        fm::commit(lead, sf + 8u);
                        release(k);
                    }
                    fm::commit(lead, od + 8u);
                    release(v);
                }
                if (ok) fm::commit(lead, o_last + 8u * t);
            } else if (t == 0) {
                // scores: slot j & 1 is free again behind the products of tile j - 2
                for (int j = 0; j < n && ok; ++j) {
                    if (j > 1) ok = fm::wait_warp(s_free + 8u * (j & 1), (uint32_t)(((j >> 1) - 1) & 1));
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        ok = ok && fm::wait_warp(full + 8u * ring.at, ring.parity);
                        if (!ok) break;
                        tc::fence_after_sync();
                        qk(0, j & 1, h, ring.at, 0, id_qk);
                        fm::commit(lead, empty + 8u * ring.at);
                        ring.step();
                    }
                    for (int h = 0; h < NH; ++h) ring.step();                 // (the values)
                    for (int g = 0; g < 2 && ok; ++g) fm::commit(lead, s_full + 8u * (2 * (j & 1) + g));
                }
            } else {
                // products
                for (int j = 0; j < n && ok; ++j) {
                    for (int h = 0; h < NH; ++h) ring.step();                 // (the keys)
                    uint32_t b[NH];
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        b[h] = ring.at;
                        ok = ok && fm::wait_warp(full + 8u * ring.at, ring.parity);
                        ring.step();
                    }
                    if (j < n_edge) ok = ok && fm::wait_warp(scanned, (uint32_t)(j & 1));
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        ok = ok && fm::wait_warp(p_full + 8u * (2 * (j & 1) + g), (uint32_t)((j >> 1) & 1));
                        if (!ok) break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            pv(0, j & 1, h, b[h], g, j > 0 || g > 0);
                            if (g == 1) fm::commit(lead, empty + 8u * b[h]);
                        }
                        fm::commit(lead, o_done + 8u * g);
                    }
                    if (ok) fm::commit(lead, s_free + 8u * (j & 1));
                }
                if (ok) fm::commit(lead, o_last);
            }
            if (!ok) {
                // the MMAs in flight end before their columns are freed
                *s_err = 1;
                fm::commit(lead, drained + 8u * t);
                fm::wait_warp(drained + 8u * t, 0u);
            }
        }
        __syncwarp();
    } else if (n > 0 && ctrl == 2) {
        // values of the edge tiles: thread t looks over every 32nd row from t
        const int t = lane;
        bool ok = true;
        for (int j = 0; j < n_edge && ok; ++j) {
            bool bad = false;
            for (int h = 0; h < NH && ok; ++h) {
                const int it = 2 * NH * j + NH + h;
                ok = fm::wait(full + 8u * (it % ST), (uint32_t)((it / ST) & 1));
                if (!ok) break;
                unsigned char * vb = smem + C::OFF_KV + (it % ST) * C::BUF;
                for (int r = t; r < kTile; r += 32) {
                    uint32_t non = 0u;
                    for (int c = 0; c < C::W / 8; ++c) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(vb + (c >> 3) * C::SLICE + r * 128 + 16 * ((c & 7) ^ (r & 7)));
                        // an exponent of all ones carries into the bit above it
                        constexpr uint32_t E = BF16 ? 0x7F807F80u : 0x7C007C00u, ONE = BF16 ? 0x00800080u : 0x04000400u;
                        non |= ((u.x & E) + ONE) | ((u.y & E) + ONE) | ((u.z & E) + ONE) | ((u.w & E) + ONE);
                    }
                    if ((non & 0x80008000u) == 0u) continue;
                    if ((n - 1 - j) * kTile + r < nk) {
                        bad = true;
                    } else {
                        for (int c = 0; c < C::W / 8; ++c)
                            *reinterpret_cast<uint4 *>(vb + (c >> 3) * C::SLICE + r * 128 + 16 * (c & 7)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
            }
            if (bad) *s_redo = 1;
            // one tile ahead of the products at most: `scanned` must not pass
            // a phase that an issuing thread has not waited for
            for (int i = 0; i < slots && j > 0; ++i)
                ok = ok && fm::wait(o_done + 8u * (2 * i + 1), (uint32_t)((j - 1) & 1));
            if (!ok) {
                *s_err = 1;
                break;
            }
            tc::fence_proxy_async();
            tc::mbar_arrive(scanned);
        }
    } else if (ctrl < 0) {
        const int i = warp >> 2;                          // row tile
        const int r = tid & 127;
        const int g = r % a.heads, qt = r / a.heads;
        const int qi = i0 + i * a.queries + qt;
        const bool valid = seq >= 0 && qt < a.queries && qi < nq;
        const int lim = valid ? min(max(qi + shift + 1, 0), nk) : 0;      // keys of this row
        T * op = static_cast<T *>(a.out) + ((int64_t)(q0 + qi) * a.n_q_heads + h0 + g) * D;
        if (n > 0 && i < slots) {
            const uint32_t lane_tm = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
            const uint32_t o_tm = lane_tm + fm::kOutCol + (uint32_t)(i * D);
            const float mul = a.scale * 1.4426950408889634f;
            fm::RowState st{-CUDART_INF_F, 0.0f};
            bool ok = true;
            for (int j = 0; j < n && ok; ++j) {
                const int slot = NQ == 2 ? i : (j & 1), use = NQ == 2 ? j : (j >> 1);
                const uint32_t s_tm = lane_tm + (uint32_t)slot * fm::kSlotCols;
                uint32_t allowed[4];
                if (j < n_edge) {
                    const int left = lim - (n - 1 - j) * kTile;           // columns of this tile to keep
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int c = left - 32 * x;
                        allowed[x] = c >= 32 ? 0xFFFFFFFFu : c <= 0 ? 0u : (1u << c) - 1u;
                    }
                }
#pragma unroll 1
                for (int g = 0; g < 2 && ok; ++g) {
                    // (the scores that follow in this half wait for these weights)
                    ok = fm::wait(s_full + 8u * (2 * slot + g), (uint32_t)(use & 1));
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc::fence_after_sync();
                    // products so far: the second half of the tile before -- d = 256
                    // had the scores of this tile behind those of tile j - 2 at the
                    // latest -- then, in this half 1, those of half 0
                    auto scale_acc = [&](float f) {
                        bool r = j == 0 || fm::wait(o_done + 8u * (2 * i + 1), (uint32_t)((j - 1) & 1));
                        if (g == 1) r = r && fm::wait(o_done + 8u * (2 * i), (uint32_t)(j & 1));
                        // (the accumulator's loads and stores want a converged warp, and the
                        // votes that follow the same answer in all its lanes)
                        r = __all_sync(0xffffffffu, r);
                        if (r) scale_row<D>(o_tm, f);
                        return r;
                    };
                    const uint32_t half = s_tm + (uint32_t)g * fm::kHalfCols;
                    if (j < n_edge) {
                        const uint32_t al[2] = {g == 0 ? allowed[0] : allowed[2], g == 0 ? allowed[1] : allowed[3]};
                        ok = fm::softmax_half<BF16, true>(half, j + g == 0, mul, al, st, scale_acc);
                    } else {
                        ok = fm::softmax_half<BF16, false>(half, j + g == 0, mul, nullptr, st, scale_acc);
                    }
                    tc::mbar_arrive(p_full + 8u * (2 * slot + g));
                }
            }
            ok = ok && fm::wait(o_last + 8u * i, 0u);
            if (!ok) *s_err = 1;
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                tc::fence_after_sync();
                const float inv = lim > 0 ? 1.0f / st.sum : 0.0f;
                // The rows go through shared memory (the row tile of the queries, which
                // nothing reads any more; each warp has its rows' share), so that a
                // store covers whole rows: row by row from their threads, 16 bytes of 32
                // rows at a time, they take 5000 cycles, this way 3000.
                constexpr int RB = 2 * D, PER = 512 / RB, CH = RB / 16;      // bytes of a row, rows of a store, chunks of a row
                unsigned char * mine = smem + i * NH * C::BUF + (warp & 3) * (32 * RB);
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    fm::tmem_ld32(o_tm + (uint32_t)c, o);
#pragma unroll
                    for (int x = 0; x < 32; x += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            w[y] = lim > 0 ? fm::pack2<BF16>(__uint_as_float(o[x + 2 * y]) * inv, __uint_as_float(o[x + 2 * y + 1]) * inv) : 0u;
                        *reinterpret_cast<uint4 *>(mine + lane * RB + 16 * (((c + x) >> 3) ^ (lane & 7))) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
                const uint64_t to = valid ? reinterpret_cast<uint64_t>(op) : 0u;
#pragma unroll 4
                for (int k = 0; k < 32; k += PER) {
                    const int row = k + lane / CH, c = lane % CH;
                    const uint64_t dst = __shfl_sync(0xffffffffu, to, row);
                    const uint4 w = *reinterpret_cast<const uint4 *>(mine + row * RB + 16 * (c ^ (row & 7)));
                    if (dst != 0u) *reinterpret_cast<uint4 *>(dst + 16u * (uint32_t)c) = w;
                }
                tc::fence_before_sync();
            }
        } else if (valid && n == 0) {
            for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4 *>(op + c) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    __syncthreads();
    tc::fence_after_sync();
    if (*s_err != 0 && tid == 0 && a.status != nullptr) atomicOr(a.status, TQ_STATUS_TIMEOUT);
    if (blockIdx.x == gridDim.x - 1 && a.status != nullptr) {        // (seldom has a tile)
        for (int b = tid; b < a.batch; b += NT)
            if (a.cu_q[b] < 0 || a.cu_q[b + 1] < a.cu_q[b] || a.cu_q[b + 1] > a.total_q || a.cu_k[b] < 0 ||
                a.cu_k[b + 1] < a.cu_k[b] || a.cu_k[b + 1] > a.total_k)
                atomicOr(a.status, TQ_STATUS_LIMIT);
    }
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
    if (*s_redo != 0) {
        __syncthreads();
        for (int r = warp; r < NQ * a.queries * a.heads; r += NT / 32) {
            const int qi = i0 + r / a.heads;
            if (qi >= nq) break;
            prompt_row<D, T>(a, q0 + qi, h0 + r % a.heads, hk, k0, min(max(qi + shift + 1, 0), nk));
        }
    }
}

template <int D, bool BF16>
tq_status launch_prompt_t(PromptArgs a, cudaStream_t st) {
    using C = PaCfg<D>;
    // heads of a row tile: the largest divisor of the group up to 32
    const int group = a.n_q_heads / a.n_kv_heads;
    a.heads = 1;
    for (int g = 2; g <= kPaMaxHeads; ++g)
        if (group % g == 0) a.heads = g;
    a.queries = kTile / a.heads;
    // every sequence adds at most one tile that is not full
    const int64_t tiles = a.total_q / ((int64_t)C::NQ * a.queries) + a.batch;
    const int64_t grid = tiles * (a.n_q_heads / a.heads);
    if (grid > INT32_MAX) return fail(TQ_ERR_UNSUPPORTED, "more than 2^31 - 1 row tiles");
    CUtensorMap qmap, kmap, vmap;
    const CUtensorMapDataType dt = BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    auto encode = [&](CUtensorMap * m, const void * base, int64_t tokens, int heads, int64_t stride, int box_heads,
                      int box_tokens) {
        const uint64_t dims[3] = {(uint64_t)D, (uint64_t)heads, (uint64_t)tokens};
        const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)stride * 2};
        const uint32_t box[3] = {64u, (uint32_t)box_heads, (uint32_t)box_tokens};
        return encode_tensor_map_3d(m, dt, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    bool ok = encode(&qmap, a.q, a.total_q, a.n_q_heads, a.q_stride, a.heads, a.queries);
    if (a.total_k > 0) {
        ok = ok && encode(&kmap, a.k, a.total_k, a.n_kv_heads, a.k_stride, 1, kTile) &&
             encode(&vmap, a.v, a.total_k, a.n_kv_heads, a.v_stride, 1, kTile);
    } else {
        kmap = vmap = qmap;                  // (no tile is read)
    }
    if (!ok) return fail(TQ_ERR_UNSUPPORTED, "tensor maps of q, k and v rejected (token stride too large?)");
    auto k = prompt_kernel<D, BF16>;
    if (int e = ensure_dynamic_smem(reinterpret_cast<const void *>(k), C::SMEM))
        return cuda_status(e, "prompt attention shared memory");
    k<<<(unsigned)grid, C::THREADS, C::SMEM, st>>>(a, qmap, kmap, vmap);
    return cuda_status((int)cudaGetLastError(), "prompt attention launch");
}

template <int D>
tq_status launch_prompt(const PromptArgs & a, tq_dtype dtype, cudaStream_t st) {
    return dtype == TQ_DTYPE_BF16 ? launch_prompt_t<D, true>(a, st) : launch_prompt_t<D, false>(a, st);
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
    if (total_q > INT32_MAX - 255 || total_k > INT32_MAX - 255)
        return fail(TQ_ERR_UNSUPPORTED, "more than 2^31 - 256 packed tokens");
    if (std::isnan(scale) || std::isinf(scale)) return fail(TQ_ERR_INVALID_ARG, "scale is not finite");
    if (q_stride < (int64_t)n_q_heads * head_dim || k_stride < (int64_t)n_kv_heads * head_dim ||
        v_stride < (int64_t)n_kv_heads * head_dim || ((q_stride | k_stride | v_stride) & 7) != 0)
        return fail(TQ_ERR_INVALID_ARG, "token strides must be multiples of 8 elements, at least one row");
    if (total_q == 0) return TQ_OK;
    if (!q || !out || !cu_q || (total_k > 0 && (!k || !v)))
        return fail(TQ_ERR_INVALID_ARG, "null q / k / v / out / cu_q");
    if (out == q || out == k || out == v) return fail(TQ_ERR_INVALID_ARG, "out must not be q, k or v");
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
    return head_dim == 64 ? launch_prompt<64>(a, dtype, st)
         : head_dim == 128 ? launch_prompt<128>(a, dtype, st) : launch_prompt<256>(a, dtype, st);
}
