// pa_sparse.cu -- decode attention over a list of chosen blocks of each row
// and kv head, instead of over the whole context.
//
// For each row r and query head h of kv head g, over the tokens t < L of the
// blocks that selected[r][g] lists:
//   out[r][h] = sum_t softmax(scale * <q[r][h], K_t>)_t V_t.
// One pass with a running maximum and sum (log2 domain, fp32).  Bound by the
// read of K and V: a block's tokens of one kv head are contiguous, blocks are
// scattered.
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

// Warps of a CTA, each with a ring of 16 KB.  bf16: six, two CTAs an SM, while
// all lists' CTAs fit the GPU at once, else four, three CTAs an SM, which end
// more evenly (256 lists of 128 blocks of 16 tokens: 47.0 us with six, 52.1 with
// four; 320 of 64: 38.3 and 32.4; 2048 of 16: 61.5 and 51.1).  fp32: twelve, one
// CTA an SM, since a warp computes longer on what it has (128 lists of 128: 50
// us; with four warps and each list split in three, 53).
constexpr int kF32Warps = 12;
constexpr int kRingBytes = 16384;
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

// What both kernels know of their (row, kv head), and of the half-tiles of 8
// tokens that its list names.
struct Row {
    int64_t unit, row;
    int h, group, L;
    bool ok;
    const int32_t *table, *list;
    uint32_t rank;  // of the CTA in the list's cluster

    // Reads the list's entry of half-tile `half` beside the row's length.
    __device__ __forceinline__ int open(const SparseParams& p, int splits, int64_t half, int64_t halves, int shift) {
        const uint32_t u = blockIdx.x / splits;
        unit = u;
        row = u / p.num_kv_heads;
        h = (int)(u % p.num_kv_heads);
        group = p.num_q_heads / p.num_kv_heads;
        list = p.selected + unit * p.max_selected;
        const int entry = half < halves ? list[half >> shift] : -1;
        const int64_t seq = p.seq_ids ? (int64_t)p.seq_ids[row] : row;
        L = p.context_lens[row];
        ok = seq >= 0 && seq < p.batch && L >= 0 && L <= (int64_t)p.max_blocks_per_seq * p.block_size;
        if (!ok && threadIdx.x == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
        table = p.block_tables + (ok ? seq : 0) * p.max_blocks_per_seq;
        return entry;
    }
    // The place in the pools, in rows of 8 tokens, of the sub-th half-tile of
    // listed block j, and its tokens below L (0: nothing to read).
    __device__ __forceinline__ int place(const SparseParams& p, int j, int sub, int per_block, uint32_t& at) const {
        at = 0;
        if (j < 0) return 0;
        int64_t blk = -1;
        if ((int64_t)j * p.block_size < L) blk = table[j];
        if (blk < 0 || blk >= p.num_blocks) {
            record_error(p.err, PA_ERR_BAD_BLOCK_ID);
            return 0;
        }
        at = (uint32_t)((blk * p.num_kv_heads + h) * per_block + sub);
        return min(8, max(0, L - j * p.block_size - 8 * sub));
    }
};

// Joins the states (running maximum, sum and output of each head) that the
// CTA's threads left in shared memory, then those of the cluster's CTAs, each
// CTA finishing its share of the outputs.
template <int STATES, int HEADS, int D, int WARPS>
__device__ __forceinline__ void join_states(const SparseParams& p, const Row& r, int splits, float (*s_o)[HEADS][D],
                                            float (*s_m)[HEADS], float (*s_l)[HEADS], float* c_m, float* c_l) {
    const float kNegInf = __int_as_float(0xff800000);
    constexpr int kThreads = WARPS * 32;
    const int64_t out0 = (r.row * p.num_q_heads + r.h * r.group) * D;
    __syncthreads();
    for (int i = threadIdx.x; i < r.group * D; i += kThreads) {
        const int head = i / D, d = i % D;
        float top = kNegInf;
#pragma unroll
        for (int w = 0; w < STATES; ++w) top = fmaxf(top, s_m[w][head]);
        const float base = top == kNegInf ? 0.f : top;
        float sum = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < STATES; ++w) {
            const float weight = exp2f(s_m[w][head] - base);
            sum = fmaf(s_l[w][head], weight, sum);
            acc = fmaf(s_o[w][head][d], weight, acc);
        }
        if (splits == 1) {
            // nothing attended: a zero row (a NaN sum stays NaN)
            store_out(p, out0 + i, sum == 0.f ? 0.f : acc / sum);
        } else {
            s_o[0][head][d] = acc;  // read by this thread alone until here
            if (d == 0) {
                c_m[head] = top;
                c_l[head] = sum;
            }
        }
    }
    if (splits == 1) return;
    cluster_sync();
    for (int i = r.rank * kThreads + threadIdx.x; i < r.group * D; i += splits * kThreads) {
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
        store_out(p, out0 + i, sum == 0.f ? 0.f : acc / sum);
    }
    cluster_sync();  // the shared memory lives until the cluster has read it
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
// P enters its product in 32 bits: as a bf16 value and two bf16 remainders (three
// products; rounded once it is off by 2^-8, with one remainder by 2^-17), and each
// tile's products are summed by themselves, smallest first, and added to the
// running output by rounded additions, since the matrix instruction cuts off what
// does not fit its sum: through a running sum of 43 tiles a warp, an fp32 output was
// 2.9e-6 (relative, in norm) below the definition, and is 2.5e-7 off it now, as in
// the fp32 kernel.  This costs 1 % on streams of long lists (45.7 to 46.3 us), 5 %
// on one context (6.1 to 6.5 us), 7 % with a group of 16 (51.0 to 54.5 us).
// (An infinite V that meets a remainder of the other sign, or zero, gives NaN.)
// Measured: 16 contexts, 64 / 8 heads of 128, 256 blocks of 16 tokens each (269
// MB): 46.3 us, 5.80 TB/s, 0.88 of a copy, with one CTA on 128 of the 148 SMs;
// 2048 lists of 64 blocks 160 us, 6.7 TB/s; one context of 128 blocks 6.5 us; a
// group of 16, 128 lists of 256 blocks, 4.9 TB/s.
// One cluster of `splits` CTAs per (row, kv head): its splits * WARPS warps take
// the tiles of the list in turn, each with its own running maximum and sum, and
// the states are joined through the cluster's shared memory, so that a long
// list of few rows fills the GPU without a workspace or a second launch.
// NT: 8-wide tiles of query heads (2 for a group of 16).
template <int D, int NT, int kStages, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 12 / WARPS) sparse_mma_kernel(const SparseParams p, int splits) {
    constexpr int kHeads = 8 * NT;             // query heads, the group padded with zero rows
    constexpr int kRowBytes = 2 * D;
    constexpr int kTile = 16 * kRowBytes;      // K or V of one tile of 16 tokens
    constexpr int kStage = 2 * kTile;
    constexpr int kSteps = D / 16;
    constexpr int kRowLanes = D / 8;           // lanes that copy one row
    constexpr int kCopyRows = 32 / kRowLanes;  // rows of one copy instruction
    extern __shared__ __align__(1024) uint8_t ring[];  // [warp][stage][K, V][16 tokens][D], later the states
    __shared__ float s_m[WARPS][kHeads], s_l[WARPS][kHeads], c_m[kHeads], c_l[kHeads];
    const float kNegInf = __int_as_float(0xff800000);
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;

    // this warp's tiles, 16 at a time; lanes 2 i and 2 i + 1 look up the two
    // half-tiles of the i-th.  The list is read one chunk ahead, the first time
    // beside the row's length.
    const int per_block = p.block_size / 8;  // half-tiles
    const int shift = per_block == 1 ? 0 : per_block == 2 ? 1 : 2;
    const int64_t halves = (int64_t)p.max_selected * per_block;
    const int step = splits * WARPS;  // warps of the cluster
    const int64_t tiles = (halves + 1) / 2;
    Row r;
    r.rank = splits > 1 ? cluster_rank() : 0;
    int64_t first = (int64_t)r.rank * WARPS + warp;
    int64_t half = (first + (int64_t)(lane >> 1) * step) * 2 + (lane & 1);
    int entry = r.open(p, splits, half, halves, shift);

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
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (r.row * p.num_q_heads + r.h * r.group + head) * D + 2 * t;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                q[n][i][c] = head < r.group ? *reinterpret_cast<const uint32_t*>(src + 16 * i + 8 * c) : 0u;
    }
    float o[NT][kSteps][4] = {};     // channels 16 i + g (+ 8), heads 8 n + 2 t (+ 1)
    float m[NT][2], l[NT][2] = {};   // of heads 8 n + 2 t (+ 1); l over this lane's tokens
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = kNegInf;

    for (; first < tiles && r.ok; first += (int64_t)step * 16) {
        uint32_t at;
        const int held = r.place(p, entry, (int)(half & (per_block - 1)), per_block, at);
        half += (int64_t)step * 32;
        entry = half < halves ? r.list[half >> shift] : -1;
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
            // 8 heads at a time, V's fragments loaded for each: with all 16 heads' P
            // held at once registers spill (63 us for the 128 lists)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t pt[3][2];  // P^T's three parts, tokens 0..7 and 8..15 of the tile
                const float b0 = m[n][0] == kNegInf ? 0.f : m[n][0], b1 = m[n][1] == kNegInf ? 0.f : m[n][1];
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    float r0 = exp2_approx(x[n][2 * a] - b0), r1 = exp2_approx(x[n][2 * a + 1] - b1);
                    l[n][0] += r0;
                    l[n][1] += r1;
#pragma unroll
                    for (int c = 0; c < 3; ++c) {
                        const uint32_t v = pack_bf16x2(r0, r1);
                        pt[c][a] = movmatrix_trans(v);
                        r0 -= bf16_lo_to_f32(v);
                        r1 -= bf16_hi_to_f32(v);
                    }
                }
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    uint32_t v[4];
                    ldmatrix_x4_trans((v_mat ^ (i << 5)) + stage * kStage, v[0], v[1], v[2], v[3]);
                    float sum[4] = {};
#pragma unroll
                    for (int c = 2; c >= 0; --c) mma_bf16_16816(sum, v, pt[c][0], pt[c][1]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[n][i][c] += sum[c];
                }
            }
            __syncwarp();  // every lane has read the stage
            if (ahead) fetch(__ffs(ahead) - 1, stage);
            ahead &= ahead - 1;
            copy_async_commit();
        }
    }

    // the warps' states take the ring's place
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
    join_states<WARPS, kHeads, D, WARPS>(p, r, splits, s_o, s_m, s_l, c_m, c_l);
}

// ---------------------------------------------------------------------------
// fp32: CUDA cores
// ---------------------------------------------------------------------------
// D / 4 lanes hold a token's row, 4 channels each (one row of D 128, two of
// D 64 side by side), through the same rings, a half-tile of 8 tokens a stage;
// a lane reads back only what it copied.  Four tokens of a lane group at a
// time: the products of 4 G scores are summed over the lanes by one
// reduce-scatter (about 4 G shuffles instead of 4 G log2(D / 4)), so that each
// weight is computed by one lane or few, and reaches the others through shared
// memory.  Measured: 128 equal lists of 128 blocks of 16 tokens, D 128: one query
// head 6.0 TB/s, eight 5.4 TB/s.
template <int D, int G, int kStages>
__global__ void __launch_bounds__(kF32Warps * 32, 1) sparse_f32_kernel(const SparseParams p, int splits) {
    constexpr int kLanes = D / 4;
    constexpr int kRows = 32 / kLanes;        // tokens side by side
    constexpr int kOwn = 8 / kRows;           // tokens of a lane group in a half-tile
    constexpr int kStage = 2 * 8 * D * 4;     // K and V of a half-tile
    constexpr int kStates = kF32Warps * kRows;
    constexpr int kValues = 4 * G;            // scores of 4 tokens
    constexpr int kHeld = kValues > kLanes ? kValues / kLanes : 1;  // of them in a lane
    extern __shared__ __align__(1024) uint8_t ring[];  // [warp][stage][K, V][row][lane], later the states
    __shared__ float s_m[kStates][G], s_l[kStates][G], c_m[G], c_l[G];
    __shared__ __align__(16) float s_p[kF32Warps][kRows][kValues];
    const float kNegInf = __int_as_float(0xff800000);
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / kLanes, x = lane % kLanes;

    const int per_block = p.block_size / 8;
    const int shift = per_block == 1 ? 0 : per_block == 2 ? 1 : 2;
    const int64_t halves = (int64_t)p.max_selected * per_block;
    const int step = splits * kF32Warps;
    Row r;
    r.rank = splits > 1 ? cluster_rank() : 0;
    int64_t first = (int64_t)r.rank * kF32Warps + warp;  // this warp's half-tiles, 32 at a time
    int64_t half = first + (int64_t)lane * step;
    int entry = r.open(p, splits, half, halves, shift);

    const float* k_pool = static_cast<const float*>(p.k_pool) + sub * D + 4 * x;
    const float* v_pool = static_cast<const float*>(p.v_pool) + sub * D + 4 * x;
    uint8_t* mine = ring + warp * (kStages * kStage) + lane * 16;
    float4 q[G], o[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
        q[i] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) +
                                                (r.row * p.num_q_heads + r.h * G + i) * D + 4 * x);
        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // the lane's scores are values x * kValues / kLanes + i, of token value / G
    // and head value % G; m and l are of those heads, l over its own tokens
    const int value0 = x * kValues / kLanes;
    float m[kHeld], l[kHeld] = {};
#pragma unroll
    for (int i = 0; i < kHeld; ++i) m[i] = kNegInf;

    for (; first < halves && r.ok; first += (int64_t)step * 32) {
        uint32_t at;
        const int held = r.place(p, entry, (int)(half & (per_block - 1)), per_block, at);
        half += (int64_t)step * 32;
        entry = half < halves ? r.list[half >> shift] : -1;
        unsigned todo = __ballot_sync(0xffffffffu, held > 0);

        auto fetch = [&](int lead, int stage) {
            const int left = __shfl_sync(0xffffffffu, held, lead) - sub;
            const size_t off = (size_t)__shfl_sync(0xffffffffu, at, lead) * (8 * D);
            const uint32_t dst = smem_addr(mine) + stage * kStage;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                copy_async16(dst + i * 512, k_pool + off + i * kRows * D, i * kRows < left);
                copy_async16(dst + kStage / 2 + i * 512, v_pool + off + i * kRows * D, i * kRows < left);
            }
        };
        unsigned ahead = todo;
#pragma unroll
        for (int st = 0; st < kStages; ++st) {
            if (ahead) fetch(__ffs(ahead) - 1, st);
            ahead &= ahead - 1;
            copy_async_commit();
        }
        for (int stage = 0; todo; todo &= todo - 1, stage = stage + 1 == kStages ? 0 : stage + 1) {
            const int n = __shfl_sync(0xffffffffu, held, __ffs(todo) - 1);
            copy_async_wait<kStages - 1>();
            const float4* rows = reinterpret_cast<const float4*>(mine + stage * kStage);
#pragma unroll
            for (int t0 = 0; t0 < kOwn; t0 += 4) {
                float s[kValues];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float4 k = rows[(t0 + t) * 32];
#pragma unroll
                    for (int i = 0; i < G; ++i)
                        s[t * G + i] = fmaf(q[i].x, k.x, q[i].y * k.y) + fmaf(q[i].z, k.z, q[i].w * k.w);
                }
                reduce_scatter<kValues, kLanes>(s);
                // as in the bf16 kernel, m moves only when a score passes it by 8
                bool over = false;
                float y[kHeld];
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
                    const int t = (t0 + (value0 + i) / G) * kRows + sub;
                    y[i] = t < n ? s[i] * p.scale_log2 : kNegInf;
                    over |= y[i] > m[i] + 8.f;
                }
                if (__any_sync(0xffffffffu, over)) {
                    float keep[kHeld];
#pragma unroll
                    for (int i = 0; i < kHeld; ++i) {
                        float top = fmaxf(m[i], y[i]);  // over the four tokens
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, kLanes / 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, kLanes / 2));
                        keep[i] = exp2_approx(m[i] - (top == kNegInf ? 0.f : top));
                        m[i] = top;
                        l[i] *= keep[i];
                    }
#pragma unroll
                    for (int i = 0; i < G; ++i) {
                        const float w = __shfl_sync(0xffffffffu, keep[kHeld == 1 ? 0 : i % kHeld],
                                                    kHeld == 1 ? i * kLanes / kValues : i / kHeld, kLanes);
                        o[i].x *= w; o[i].y *= w; o[i].z *= w; o[i].w *= w;
                    }
                }
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
                    const float w = exp2_approx(y[i] - (m[i] == kNegInf ? 0.f : m[i]));
                    l[i] += w;
                    s_p[warp][sub][value0 + i] = w;  // the same from every lane that has it
                }
                __syncwarp();
                float w[kValues];
#pragma unroll
                for (int i = 0; i < kValues; i += 4)
                    *reinterpret_cast<float4*>(&w[i]) = *reinterpret_cast<const float4*>(&s_p[warp][sub][i]);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float4 v = rows[kStage / 32 + (t0 + t) * 32];
#pragma unroll
                    for (int i = 0; i < G; ++i) {
                        o[i].x = fmaf(w[t * G + i], v.x, o[i].x);
                        o[i].y = fmaf(w[t * G + i], v.y, o[i].y);
                        o[i].z = fmaf(w[t * G + i], v.z, o[i].z);
                        o[i].w = fmaf(w[t * G + i], v.w, o[i].w);
                    }
                }
                __syncwarp();  // s_p is read
            }
            if (ahead) fetch(__ffs(ahead) - 1, stage);
            ahead &= ahead - 1;
            copy_async_commit();
        }
    }

    copy_async_wait<0>();
    __syncthreads();
    float(*s_o)[G][D] = reinterpret_cast<float(*)[G][D]>(ring);
    const int state = warp * kRows + sub;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], kLanes / 4);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], kLanes / 2);
        if (x < kLanes / 4) {  // token 0's lanes
            s_m[state][value0 + i] = m[i];
            s_l[state][value0 + i] = l[i];
        }
    }
#pragma unroll
    for (int i = 0; i < G; ++i) *reinterpret_cast<float4*>(&s_o[state][i][4 * x]) = o[i];
    join_states<kStates, G, D, kF32Warps>(p, r, splits, s_o, s_m, s_l, c_m, c_l);
}

// `step_tokens`: tokens that a warp takes at a time.
int launch_sparse(const SparseParams& p, void (*kernel)(SparseParams, int), std::atomic<unsigned long long>& configured,
                  int warps, int step_tokens, cudaStream_t st) {
    const int smem = warps * kRingBytes;
    int dev = 0;
    cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return PA_ERR_CUDA;
        configured.fetch_or(bit);
    }
    const int64_t units = p.num_rows * p.num_kv_heads;
    // half-tiles are counted in 32 bits (a pool that needs more is 4 TB)
    if (p.num_blocks > (1ll << 32) / (p.num_kv_heads * (p.block_size / 8))) return PA_ERR_UNSUPPORTED;
    // One CTA a list keeps its warps longest in their stream: at 128 lists of 256
    // blocks of 16 tokens 46.3 us, against 48.9 with two and 54.1 with three.
    // Fewer lists are split over as many CTAs as leave each SM one (64 lists of
    // 128 blocks: 20.7 us with one, 18.1 with two; 8 lists: 17.3 with one, 6.5
    // with eight).
    const int64_t steps = ((int64_t)p.max_selected * p.block_size + step_tokens - 1) / step_tokens;
    int64_t splits = std::min(num_sms() / units, std::min((int64_t)kMaxSplits, (steps + warps - 1) / warps));
    splits = std::max(splits, (int64_t)1);
    if (units > 0x7fffffff / splits) return PA_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * splits));
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = smem;
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

template <int D, int NT, int WARPS>
int launch_mma_warps(const SparseParams& p, cudaStream_t st) {
    constexpr int kStages = kRingBytes / (2 * 16 * 2 * D);
    static_assert(NT * 8 * D * 4 <= kRingBytes, "the states fit in the ring");
    static std::atomic<unsigned long long> configured{0};
    return launch_sparse(p, sparse_mma_kernel<D, NT, kStages, WARPS>, configured, WARPS, 16, st);
}

template <int D, int NT>
int launch_mma(const SparseParams& p, cudaStream_t st) {
    return p.num_rows * p.num_kv_heads <= 2 * num_sms() ? launch_mma_warps<D, NT, 6>(p, st)
                                                        : launch_mma_warps<D, NT, 4>(p, st);
}

template <int D, int G>
int launch_f32(const SparseParams& p, cudaStream_t st) {
    constexpr int kStages = kRingBytes / (2 * 8 * 4 * D);
    static_assert((128 / D) * G * D * 4 <= kRingBytes, "the states fit in the ring");
    static std::atomic<unsigned long long> configured{0};
    return launch_sparse(p, sparse_f32_kernel<D, G, kStages>, configured, kF32Warps, 8, st);
}

template <int D>
int launch_f32_group(const SparseParams& p, cudaStream_t st) {
    switch (p.num_q_heads / p.num_kv_heads) {
        case 1: return launch_f32<D, 1>(p, st);
        case 2: return launch_f32<D, 2>(p, st);
        case 4: return launch_f32<D, 4>(p, st);
        case 8: return launch_f32<D, 8>(p, st);
    }
    return PA_ERR_UNSUPPORTED;
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
        !supported_group(num_q_heads / num_kv_heads, kv_dtype) || num_rows > 0x7fffffff)
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
    return head_dim == 128 ? launch_f32_group<128>(p, st) : launch_f32_group<64>(p, st);
}
