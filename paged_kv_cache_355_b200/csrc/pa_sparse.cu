// pa_sparse.cu -- decode attention over a list of chosen blocks of each row
// and kv head, instead of over the whole context.
//
// For each row r and query head h of kv head g, over the tokens t < L of the
// blocks that selected[r][g] lists:
//   out[r][h] = sum_t softmax(scale * <q[r][h], K_t>)_t V_t.
// One pass with a running maximum and sum (log2 domain, fp32).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct SparseParams {
    const void *q, *k_pool, *v_pool;
    const int32_t *block_tables, *seq_ids, *context_lens, *selected;
    int max_blocks_per_seq, batch, max_selected, block_size;
    void* out;
    int out_bf16;
    float scale_log2;
    int64_t num_rows;
    int num_q_heads, num_kv_heads;
    int64_t num_blocks;
    int* err;
};

__device__ __forceinline__ void store_out(const SparseParams& p, int64_t at, float x) {
    if (p.out_bf16)
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(x);
    else
        static_cast<float*>(p.out)[at] = x;
}

constexpr int kSimtWarps = 8;

// CUDA-core form.  One CTA per (row, kv head, G query heads); its warps take
// the listed blocks in turn.  D / 8 lanes hold one token's row; each such lane
// group keeps its own running maximum, sum and output, joined at the end.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kSimtWarps * 32) sparse_simt_kernel(const SparseParams p, int head_slices) {
    constexpr int kLanes = D / kChunk;
    constexpr int kRows = 32 / kLanes;
    constexpr int kStates = kSimtWarps * kRows;
    __shared__ float s_m[kStates][G], s_l[kStates][G];
    __shared__ float s_o[kSimtWarps][G][D];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t unit = blockIdx.x;
    const int64_t rg = unit / head_slices;  // (row, kv head)
    const int slice = (int)(unit - rg * head_slices);
    const int64_t row = rg / p.num_kv_heads;
    const int h = (int)(rg - row * p.num_kv_heads);
    const int head0 = h * (p.num_q_heads / p.num_kv_heads) + slice * G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / kLanes, chunk = lane % kLanes;

    const int64_t seq = p.seq_ids ? (int64_t)p.seq_ids[row] : row;
    const int L = p.context_lens[row];
    bool row_ok = seq >= 0 && seq < p.batch && L >= 0 && L <= (int64_t)p.max_blocks_per_seq * p.block_size;
    if (!row_ok && threadIdx.x == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
    const int32_t* table = p.block_tables + (row_ok ? seq : 0) * p.max_blocks_per_seq;
    const int32_t* list = p.selected + rg * p.max_selected;

    float q[G][kChunk], o[G][kChunk], m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        Chunk<T> raw;
        raw.load(static_cast<const T*>(p.q) + (row * p.num_q_heads + head0 + g) * D + chunk * kChunk);
        raw.to_f32(q[g]);
        m[g] = __int_as_float(0xff800000);
        l[g] = 0.f;
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
            q[g][e] *= p.scale_log2;
            o[g][e] = 0.f;
        }
    }
    for (int i = warp; row_ok && i < p.max_selected; i += kSimtWarps) {
        const int j = list[i];
        if (j < 0) continue;
        int64_t blk = -1;
        if ((int64_t)j * p.block_size < L) blk = table[j];
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
            continue;
        }
        const int held = min(p.block_size, L - j * p.block_size);
        const int64_t base = ((blk * p.num_kv_heads + h) * p.block_size) * D + chunk * kChunk;
        for (int t0 = 0; t0 < held; t0 += kRows) {
            const int t = t0 + sub;
            const bool in = t < held;
            float k[kChunk] = {}, v[kChunk] = {};
            if (in) {
                Chunk<T> raw;
                raw.load(static_cast<const T*>(p.k_pool) + base + t * D);
                raw.to_f32(k);
                raw.load(static_cast<const T*>(p.v_pool) + base + t * D);
                raw.to_f32(v);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < kChunk; ++e) s = fmaf(q[g][e], k[e], s);
#pragma unroll
                for (int x = kLanes / 2; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
                if (!in) continue;
                const float top = fmaxf(m[g], s);
                const float base_m = top == __int_as_float(0xff800000) ? 0.f : top;
                const float keep = exp2f(m[g] - base_m), w = exp2f(s - base_m);
                m[g] = top;
                l[g] = l[g] * keep + w;
#pragma unroll
                for (int e = 0; e < kChunk; ++e) o[g][e] = fmaf(w, v[e], o[g][e] * keep);
            }
        }
    }
    // join the lane groups and warps
    const int state = warp * kRows + sub;
    if (chunk == 0) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            s_m[state][g] = m[g];
            s_l[state][g] = l[g];
        }
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float top = __int_as_float(0xff800000);
        for (int x = 0; x < kStates; ++x) top = fmaxf(top, s_m[x][g]);
        const float base_m = top == __int_as_float(0xff800000) ? 0.f : top;
        const float w = exp2f(m[g] - base_m);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
            float x = o[g][e] * w;
#pragma unroll
            for (int y = kLanes; y < 32; y <<= 1) x += __shfl_xor_sync(0xffffffffu, x, y);
            if (sub == 0) s_o[warp][g][chunk * kChunk + e] = x;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += kSimtWarps * 32) {
        const int g = i / D, d = i - g * D;
        float top = __int_as_float(0xff800000);
        for (int x = 0; x < kStates; ++x) top = fmaxf(top, s_m[x][g]);
        const float base_m = top == __int_as_float(0xff800000) ? 0.f : top;
        float sum = 0.f, acc = 0.f;
        for (int x = 0; x < kStates; ++x) sum += s_l[x][g] * exp2f(s_m[x][g] - base_m);
#pragma unroll
        for (int x = 0; x < kSimtWarps; ++x) acc += s_o[x][g][d];
        // nothing attended: a zero row (a NaN sum stays NaN)
        store_out(p, (row * p.num_q_heads + head0 + g) * D + d, sum == 0.f ? 0.f : acc / sum);
    }
}

template <typename T, int D>
int launch_simt(const SparseParams& p, cudaStream_t st) {
    const int group = p.num_q_heads / p.num_kv_heads;
    const int slices = group > 8 ? group / 8 : 1;
    const int64_t grid = p.num_rows * p.num_kv_heads * slices;
    if (grid > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    const dim3 g((unsigned)grid), b(kSimtWarps * 32);
    switch (group / slices) {
        case 1: return launch_pdl(sparse_simt_kernel<T, D, 1>, g, b, 0, st, p, slices);
        case 2: return launch_pdl(sparse_simt_kernel<T, D, 2>, g, b, 0, st, p, slices);
        case 4: return launch_pdl(sparse_simt_kernel<T, D, 4>, g, b, 0, st, p, slices);
        case 8: return launch_pdl(sparse_simt_kernel<T, D, 8>, g, b, 0, st, p, slices);
    }
    return PA_ERR_UNSUPPORTED;
}

// ---------------------------------------------------------------------------
// bf16: matrix instructions
// ---------------------------------------------------------------------------
// A warp takes 16 tokens at a time (two half-tiles of 8, so that blocks of 8,
// 16 and 32 tokens are all whole half-tiles) through a ring of shared memory of
// its own, filled by asynchronous copies: warps never wait for one another
// until the end.  Both products are m16n8k16 with the few query heads on the
// 8-wide side: S^T = K Q^T over 16 tokens, O^T = V^T P^T over 16 channels at a
// time, so no row of an instruction is padding.  P^T's fragment is S^T's
// accumulator, rounded and transposed in 8x8 matrices between the lanes.
// 16-byte chunk c of a row lies at c ^ (row & 7), so that the eight rows of a
// matrix load touch all banks.
// P is split into a bf16 value and a bf16 remainder (two products), so that
// its rounding, 2^-17 of P, stays far below the fp32 output's use; rounding P
// once (2^-9) would be half of a bf16 output's own error.
constexpr int kMmaWarps = 4;
constexpr int kMaxSplits = 8;  // the portable cluster size

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// A float of the shared memory of CTA `rank` of the cluster, at the address
// that p has in this one.
__device__ __forceinline__ float load_cluster(const float* p, uint32_t rank) {
    uint32_t at;
    float x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    return x;
}

// One cluster of `splits` CTAs per (row, kv head): its splits * 4 warps take
// the tiles of the list in turn, each with its own running maximum and sum, and
// the states are joined through the cluster's shared memory, so that a long
// list of few rows fills the GPU without a workspace or a second launch.
// NT: 8-wide tiles of query heads (2 for a group of 16).
template <int D, int NT, int kStages>
__global__ void __launch_bounds__(kMmaWarps * 32, 3) sparse_mma_kernel(const SparseParams p, int splits) {
    constexpr int kHeads = 8 * NT;             // query heads, the group padded with zero rows
    constexpr int kRowBytes = 2 * D;
    constexpr int kTile = 16 * kRowBytes;      // K or V of one tile of 16 tokens
    constexpr int kStage = 2 * kTile;
    constexpr int kSteps = D / 16;
    constexpr int kRowLanes = D / 8;           // lanes that copy one row
    constexpr int kCopyRows = 32 / kRowLanes;  // rows of one copy instruction
    extern __shared__ __align__(1024) uint8_t ring[];  // [warp][stage][K, V][16 tokens][D], later the states
    __shared__ float s_m[kMmaWarps][kHeads], s_l[kMmaWarps][kHeads], c_m[kHeads], c_l[kHeads];
    const float kNegInf = __int_as_float(0xff800000);
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t rank = splits > 1 ? cluster_rank() : 0;
    const int64_t unit = blockIdx.x / splits;
    const int64_t row = unit / p.num_kv_heads;
    const int h = (int)(unit - row * p.num_kv_heads);
    const int group = p.num_q_heads / p.num_kv_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;

    // this warp's tiles, 16 at a time; lanes 2 i and 2 i + 1 look up the two
    // half-tiles of the i-th.  The list is read one chunk ahead, the first time
    // beside the row's length.
    const int per_block = p.block_size / 8;  // half-tiles
    const int shift = per_block == 1 ? 0 : per_block == 2 ? 1 : 2;
    const int64_t halves = (int64_t)p.max_selected * per_block;
    const int step = splits * kMmaWarps;     // warps of the cluster
    const int64_t tiles = (halves + 1) / 2;
    const int32_t* list = p.selected + unit * p.max_selected;
    int64_t first = (int64_t)rank * kMmaWarps + warp;
    int64_t half = (first + (int64_t)(lane >> 1) * step) * 2 + (lane & 1);
    int entry = half < halves ? list[half >> shift] : -1;

    const int64_t seq = p.seq_ids ? (int64_t)p.seq_ids[row] : row;
    const int L = p.context_lens[row];
    const bool row_ok = seq >= 0 && seq < p.batch && L >= 0 && L <= (int64_t)p.max_blocks_per_seq * p.block_size;
    if (!row_ok && threadIdx.x == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
    const int32_t* table = p.block_tables + (row_ok ? seq : 0) * p.max_blocks_per_seq;

    // the lane's part of the copies: one chunk of one row in every kCopyRows
    const int copy_row = lane / kRowLanes, copy_chunk = lane % kRowLanes;
    const __nv_bfloat16* k_pool = static_cast<const __nv_bfloat16*>(p.k_pool) + copy_row * D + copy_chunk * 8;
    const __nv_bfloat16* v_pool = static_cast<const __nv_bfloat16*>(p.v_pool) + copy_row * D + copy_chunk * 8;
    const uint32_t slots = smem_addr(ring) + warp * (kStages * kStage);
    const uint32_t copy_dst = slots + copy_row * kRowBytes + ((copy_chunk ^ copy_row) << 4);
    // matrix loads: lane = (matrix, row).  K's matrices are (chunk of the
    // k-step, half-tile), V's, transposed, (half-tile, chunk of the 16 channels)
    const uint32_t mat_row = lane & 7, mat_lo = (lane >> 3) & 1, mat_hi = lane >> 4;
    const uint32_t k_mat = slots + (mat_lo * 8 + mat_row) * kRowBytes + ((mat_hi ^ mat_row) << 4);
    const uint32_t v_mat = slots + kTile + (mat_hi * 8 + mat_row) * kRowBytes + ((mat_lo ^ mat_row) << 4);

    uint32_t q[NT][kSteps][2];  // head 8 n + g as a column of Q^T
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int head = 8 * n + g;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (row * p.num_q_heads + h * group + head) * D + 2 * t;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                q[n][i][c] = head < group ? *reinterpret_cast<const uint32_t*>(src + 16 * i + 8 * c) : 0u;
    }
    float o[NT][kSteps][4] = {};     // channels 16 i + g (+ 8), heads 8 n + 2 t (+ 1)
    float m[NT][2], l[NT][2] = {};   // of heads 8 n + 2 t (+ 1); l over this lane's tokens
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = kNegInf;

    for (; first < tiles && row_ok; first += (int64_t)step * 16) {
        uint32_t at = 0;  // the half-tile's place in the pools, in rows of 8 tokens
        int held = 0;     // its tokens below L
        const int j = entry, sub = (int)(half & (per_block - 1));
        half += (int64_t)step * 32;
        entry = half < halves ? list[half >> shift] : -1;
        if (j >= 0) {
            int64_t blk = -1;
            if ((int64_t)j * p.block_size < L) blk = table[j];
            if (blk < 0 || blk >= p.num_blocks) {
                record_error(p.err, PA_ERR_BAD_BLOCK_ID);
            } else {
                held = min(8, max(0, L - j * p.block_size - 8 * sub));
                at = (uint32_t)((blk * p.num_kv_heads + h) * per_block + sub);
            }
        }
        unsigned todo = __ballot_sync(0xffffffffu, held > 0);
        todo = (todo | (todo >> 1)) & 0x55555555u;

        auto fetch = [&](int lead, int stage) {
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const int left = __shfl_sync(0xffffffffu, held, lead + a) - copy_row;
                const size_t off = (size_t)__shfl_sync(0xffffffffu, at, lead + a) * (8 * D);
#pragma unroll
                for (int u = 0; u < 8 / kCopyRows; ++u) {
                    const uint32_t dst = (copy_dst ^ ((u * kCopyRows) << 4)) + stage * kStage +
                                         (a * 8 + u * kCopyRows) * kRowBytes;
                    const bool in = u * kCopyRows < left;
                    copy_async16(dst, k_pool + off + u * kCopyRows * D, in);
                    copy_async16(dst + kTile, v_pool + off + u * kCopyRows * D, in);
                }
            }
        };
        unsigned ahead = todo;  // tiles still to be fetched
#pragma unroll
        for (int st = 0; st < kStages; ++st) {
            if (ahead) fetch(__ffs(ahead) - 1, st);
            ahead &= ahead - 1;
            copy_async_commit();
        }
        for (int stage = 0; todo; todo &= todo - 1, stage = stage + 1 == kStages ? 0 : stage + 1) {
            const int lead = __ffs(todo) - 1;
            copy_async_wait<kStages - 1>();
            __syncwarp();  // every lane's copies are in
            float s[NT][2][4] = {};  // tokens g, g + 8; heads 2 t, 2 t + 1; two chains
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                uint32_t k[4];
                ldmatrix_x4((k_mat ^ (i << 5)) + stage * kStage, k[0], k[1], k[2], k[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16_16816(s[n][i & 1], k, q[n][i][0], q[n][i][1]);
            }
            const bool in0 = g < __shfl_sync(0xffffffffu, held, lead), in1 = g < __shfl_sync(0xffffffffu, held, lead + 1);

            // p = 2^(x - m).  m is a maximum of earlier scores, not the running
            // one: it moves only when a score passes it by 8, so that most tiles
            // need no maximum across lanes and no rescale, and p stays below 2^8.
            float x[NT][4];
            bool over = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    x[n][c] = (c < 2 ? in0 : in1) ? (s[n][0][c] + s[n][1][c]) * p.scale_log2 : kNegInf;
                    over |= x[n][c] > m[n][c & 1] + 8.f;
                }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float top = fmaxf(m[n][c], fmaxf(x[n][c], x[n][c + 2]));
#pragma unroll
                        for (int y = 4; y < 32; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
                        const float keep = exp2_approx(m[n][c] - (top == kNegInf ? 0.f : top));
                        m[n][c] = top;
                        l[n][c] *= keep;
#pragma unroll
                        for (int i = 0; i < kSteps; ++i) {
                            o[n][i][c] *= keep;
                            o[n][i][c + 2] *= keep;
                        }
                    }
            }
            uint32_t hi[NT][2], lo[NT][2];  // P^T, tokens 0..7 and 8..15 of the tile
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float b0 = m[n][0] == kNegInf ? 0.f : m[n][0], b1 = m[n][1] == kNegInf ? 0.f : m[n][1];
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const float p0 = exp2_approx(x[n][2 * a] - b0), p1 = exp2_approx(x[n][2 * a + 1] - b1);
                    l[n][0] += p0;
                    l[n][1] += p1;
                    const uint32_t v = pack_bf16x2(p0, p1);
                    hi[n][a] = movmatrix_trans(v);
                    lo[n][a] = movmatrix_trans(pack_bf16x2(p0 - bf16_lo_to_f32(v), p1 - bf16_hi_to_f32(v)));
                }
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                uint32_t v[4];
                ldmatrix_x4_trans((v_mat ^ (i << 5)) + stage * kStage, v[0], v[1], v[2], v[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_bf16_16816(o[n][i], v, hi[n][0], hi[n][1]);
                    mma_bf16_16816(o[n][i], v, lo[n][0], lo[n][1]);
                }
            }
            __syncwarp();  // every lane has read the stage
            if (ahead) fetch(__ffs(ahead) - 1, stage);
            ahead &= ahead - 1;
            copy_async_commit();
        }
    }

    // the warps' states, in the ring's place, joined to the CTA's; then the
    // cluster's, each CTA finishing its share of the outputs
    copy_async_wait<0>();
    __syncthreads();
    float(*s_o)[kHeads][D] = reinterpret_cast<float(*)[kHeads][D]>(ring);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int head = 8 * n + 2 * t + c;
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], y);
            if (g == 0) {
                s_m[warp][head] = m[n][c];
                s_l[warp][head] = l[n][c];
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                s_o[warp][head][16 * i + g] = o[n][i][c];
                s_o[warp][head][16 * i + g + 8] = o[n][i][c + 2];
            }
        }
    __syncthreads();
    const bool alone = splits == 1;
    for (int i = threadIdx.x; i < group * D; i += kMmaWarps * 32) {
        const int head = i / D, d = i % D;
        float top = kNegInf;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) top = fmaxf(top, s_m[w][head]);
        const float base = top == kNegInf ? 0.f : top;
        float sum = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) {
            const float weight = exp2f(s_m[w][head] - base);
            sum = fmaf(s_l[w][head], weight, sum);
            acc = fmaf(s_o[w][head][d], weight, acc);
        }
        if (alone) {
            // nothing attended: a zero row (a NaN sum stays NaN)
            store_out(p, (row * p.num_q_heads + h * group + head) * D + d, sum == 0.f ? 0.f : acc / sum);
        } else {
            s_o[0][head][d] = acc;  // read by this thread alone until here
            if (d == 0) {
                c_m[head] = top;
                c_l[head] = sum;
            }
        }
    }
    if (alone) return;
    cluster_sync();
    for (int i = rank * (kMmaWarps * 32) + threadIdx.x; i < group * D; i += splits * (kMmaWarps * 32)) {
        const int head = i / D, d = i % D;
        float ms[kMaxSplits], ls[kMaxSplits], os[kMaxSplits];
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c) {
            ms[c] = c < splits ? load_cluster(&c_m[head], c) : kNegInf;
            ls[c] = c < splits ? load_cluster(&c_l[head], c) : 0.f;
            os[c] = c < splits ? load_cluster(&s_o[0][head][d], c) : 0.f;
        }
        float top = kNegInf;
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c) top = fmaxf(top, ms[c]);
        const float base = top == kNegInf ? 0.f : top;
        float sum = 0.f, acc = 0.f;
#pragma unroll
        for (int c = 0; c < kMaxSplits; ++c) {
            const float weight = exp2f(ms[c] - base);
            sum = fmaf(ls[c], weight, sum);
            acc = fmaf(os[c], weight, acc);
        }
        store_out(p, (row * p.num_q_heads + h * group + head) * D + d, sum == 0.f ? 0.f : acc / sum);
    }
    cluster_sync();  // the shared memory lives until the cluster has read it
}

template <int D, int NT>
int launch_mma(const SparseParams& p, cudaStream_t st) {
    constexpr int kStages = D == 128 ? 2 : 4;  // 16 KB in flight a warp
    constexpr size_t kSmem = (size_t)kMmaWarps * kStages * (D / 8) * 512;
    static_assert(kSmem >= (size_t)kMmaWarps * NT * 8 * D * 4, "the states fit in the ring");
    auto kernel = sparse_mma_kernel<D, NT, kStages>;
    static std::atomic<unsigned long long> configured{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
            return PA_ERR_CUDA;
        configured.fetch_or(bit);
    }
    const int64_t units = p.num_rows * p.num_kv_heads;
    // half-tiles are counted in 32 bits (a pool that needs more is 4 TB)
    if (p.num_blocks > (1ll << 32) / (p.num_kv_heads * (p.block_size / 8))) return PA_ERR_UNSUPPORTED;
    // One CTA a list keeps its four warps longest in their stream, and is best
    // as soon as the lists fill the SMs: at 2048 lists of 64 blocks of 16 tokens
    // 156 us (6.85 TB/s) against 165 with two CTAs and 190 with four; at 128
    // lists 15.6 against 17.8 and 21.3.  Below that, as many as give each SM
    // one (16 lists of 512 blocks: 72.8 us with one, 16.9 with eight); and three
    // an SM, which is what its shared memory holds, where each warp then still
    // has 16 tiles (128 lists of 256 blocks: 49.3 us with one, 47.6 with three).
    const int64_t tiles = ((int64_t)p.max_selected * p.block_size + 15) / 16;
    const int64_t fill = num_sms() / units, hold = 3 * num_sms() / units;
    int64_t splits = std::max(fill, std::min(hold, tiles / (kMmaWarps * 16)));
    splits = std::min(splits, std::min((int64_t)kMaxSplits, (tiles + kMmaWarps - 1) / kMmaWarps));
    splits = std::max(splits, (int64_t)1);
    if (units * splits > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * splits));
    cfg.blockDim = dim3(kMmaWarps * 32);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, p, (int)splits) != cudaSuccess) {
        (void)cudaGetLastError();
        return PA_ERR_CUDA;
    }
    return launch_status();
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_paged_attention_decode_sparse(const void* q, const void* k_pool, const void* v_pool,
                                                const int32_t* block_tables, int max_blocks_per_seq,
                                                const int32_t* seq_ids, const int32_t* context_lens,
                                                const int32_t* selected, int max_selected, float scale,
                                                int block_size, void* out, int out_dtype, int64_t num_rows,
                                                int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                int64_t num_blocks, int kv_dtype, void* stream) {
    PA_NVTX_RANGE("pa_paged_attention_decode_sparse");
    if (num_rows < 0 || batch < 0 || max_blocks_per_seq < 0 || max_selected <= 0 || num_q_heads <= 0 ||
        num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0 || !valid_dtype(kv_dtype) ||
        !valid_dtype(out_dtype) || num_q_heads % num_kv_heads != 0)
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size) ||
        !supported_group(num_q_heads / num_kv_heads, kv_dtype))
        return PA_ERR_UNSUPPORTED;
    if (!seq_ids && num_rows > batch) return PA_ERR_INVALID_ARG;
    if (num_rows == 0) return PA_OK;
    if (!q || !k_pool || !v_pool || !block_tables || !context_lens || !selected || !out || !aligned16(q) ||
        !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
        return PA_ERR_INVALID_ARG;
    SparseParams p = {};
    p.q = q;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.block_tables = block_tables;
    p.seq_ids = seq_ids;
    p.context_lens = context_lens;
    p.selected = selected;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.batch = batch;
    p.max_selected = max_selected;
    p.block_size = block_size;
    p.out = out;
    p.out_bf16 = out_dtype == PA_BF16;
    p.scale_log2 = scale * kLog2e;
    p.num_rows = num_rows;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.num_blocks = num_blocks;
    p.err = error_word_ptr();
    if (!p.err) return PA_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (kv_dtype == PA_BF16) {
        if (num_q_heads / num_kv_heads == 16)
            return head_dim == 128 ? launch_mma<128, 2>(p, st) : launch_mma<64, 2>(p, st);
        return head_dim == 128 ? launch_mma<128, 1>(p, st) : launch_mma<64, 1>(p, st);
    }
    return head_dim == 128 ? launch_simt<float, 128>(p, st) : launch_simt<float, 64>(p, st);
}
