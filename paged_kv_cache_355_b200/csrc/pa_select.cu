// pa_select.cu -- choosing the blocks a query attends to: per-block key
// bounds, a block score from them, and the choice of the best blocks.
//
// bounds: for each block and kv head, per channel the smallest and the largest
//   key value over the block's tokens.
// score:  for each query row, kv head and block, the largest over the group's
//   query heads of  sum_d max(q_d * lo_d, q_d * hi_d), which no dot product of
//   q with a key of the block exceeds.
// select: the first and the last blocks of the row, then those of the largest
//   score; equal scores go to the lower block.
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

constexpr int kWarps = 4;

// ---------------------------------------------------------------------------
// key bounds
// ---------------------------------------------------------------------------
struct BoundsParams {
    const void* k_pool;
    void* key_bounds;
    const int32_t* block_tables;
    int max_blocks_per_seq;
    const int32_t* context_lens;
    const int32_t* query_start;  // NULL: one new token a sequence
    int max_query_len, batch, num_kv_heads, block_size;
    int64_t num_blocks;
    int max_touched;  // blocks that max_query_len new tokens can lie in
    int heads_per_warp, parts;  // parts: warps for a block's heads
    int* err;
};

// The running minimum and maximum of a lane's 16 bytes of channels, NaN kept.
template <typename T>
struct Range;

__device__ __forceinline__ uint32_t min2_nan(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

template <>
struct Range<__nv_bfloat16> {
    uint32_t lo[4], hi[4];  // pairs of channels
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = 0x7f807f80u;  // +inf
            hi[i] = 0xff80ff80u;
        }
    }
    __device__ __forceinline__ void take(const uint4& c) {
        const uint32_t x[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = min2_nan(lo[i], x[i]);
            hi[i] = max2_nan(hi[i], x[i]);
        }
    }
    __device__ __forceinline__ void join(int lanes) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = min2_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], lanes));
            hi[i] = max2_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], lanes));
        }
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p, bool high) const {
        *reinterpret_cast<uint4*>(p) =
            high ? make_uint4(hi[0], hi[1], hi[2], hi[3]) : make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
};

template <>
struct Range<float> {
    float lo[4], hi[4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = __int_as_float(0x7f800000);
            hi[i] = __int_as_float(0xff800000);
        }
    }
    __device__ __forceinline__ void take(const uint4& c) {
        const uint32_t x[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = min_nan(lo[i], __uint_as_float(x[i]));
            hi[i] = max_nan(hi[i], __uint_as_float(x[i]));
        }
    }
    __device__ __forceinline__ void join(int lanes) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = min_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], lanes));
            hi[i] = max_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], lanes));
        }
    }
    __device__ __forceinline__ void store(float* p, bool high) const {
        *reinterpret_cast<float4*>(p) =
            high ? make_float4(hi[0], hi[1], hi[2], hi[3]) : make_float4(lo[0], lo[1], lo[2], lo[3]);
    }
};

// One warp per (sequence, block with new tokens, part of the kv heads): it takes
// the rows of the block's tokens head by head, through a ring of four pieces of
// 4 KB that asynchronous copies fill, and joins the lanes' ranges by shuffles.
// Bound by the read of the keys: one pass, 2 D values written for BS * D read;
// a lane reads back only what it copied itself, so no barrier is needed.  The
// whole block is read again for every new token rather than its bounds updated,
// so that the call can be repeated and follows a copied or rewritten block.
// Measured: eight prompts, 299k tokens, 8 kv heads of 128, bf16 (688 MB): 104
// us, 6.6 TB/s, the rate of a copy; fp32 6.7 TB/s; the last blocks of 64
// sequences (5.6 MB): 3.3 us.
constexpr int kPieces = 4;
constexpr int kPieceBytes = 4096;

template <typename T, int D, int BS>
__global__ void __launch_bounds__(kWarps * 32) key_bounds_kernel(const BoundsParams p) {
    constexpr int kElems = 16 / sizeof(T);                    // channels of a lane
    constexpr int kLanes = D / kElems;                        // lanes of one row
    constexpr int kRows = 32 / kLanes;                        // rows side by side
    constexpr int kOwn = BS / kRows;                          // rows of one lane
    constexpr int kBatch = kOwn < kPieceBytes / 512 ? kOwn : kPieceBytes / 512;  // of a piece
    constexpr int kPerHead = kOwn / kBatch;                   // pieces of one head
    extern __shared__ __align__(1024) uint8_t ring[];         // [warp][piece][row][lane]
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const uint32_t per_seq = (uint32_t)p.max_touched * p.parts;
    const int64_t b = unit / per_seq;
    if (b >= p.batch) return;
    const uint32_t rem = unit % per_seq;
    const int i = (int)(rem / p.parts), part = (int)(rem % p.parts);
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, chunk = lane % kLanes;

    const int L = p.context_lens[b];
    int64_t n = L > 0 ? 1 : 0;
    if (p.query_start) n = (int64_t)p.query_start[b + 1] - p.query_start[b];
    if (L < 0 || n < 0 || n > L || n > p.max_query_len || L > (int64_t)p.max_blocks_per_seq * BS) {
        if (rem == 0 && lane == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
        return;
    }
    if (n == 0) return;
    const int64_t j = (L - n) / BS + i;
    if (j > (L - 1) / BS) return;
    const int64_t blk = p.block_tables[b * p.max_blocks_per_seq + j];
    if (blk < 0 || blk >= p.num_blocks) {
        if (part == 0 && lane == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
        return;
    }
    const int64_t left = L - j * BS;
    const int held = left < BS ? (int)left : BS;  // tokens of the block
    const int h0 = part * p.heads_per_warp, h1 = min(h0 + p.heads_per_warp, p.num_kv_heads);
    const int64_t row = blk * p.num_kv_heads + h0;
    const T* src = static_cast<const T*>(p.k_pool) + row * (BS * D) + sub * D + chunk * kElems;
    T* dst = static_cast<T*>(p.key_bounds) + row * (2 * D) + (sub & 1) * D + chunk * kElems;
    uint8_t* mine = ring + (threadIdx.x >> 5) * (kPieces * kPieceBytes) + lane * 16;

    const int pieces = (h1 - h0) * kPerHead;
    int fetched = 0;
    auto fetch = [&]() {
        if (fetched < pieces) {
            const int t0 = fetched % kPerHead * kBatch;
            const uint32_t to = smem_addr(mine) + fetched % kPieces * kPieceBytes;
#pragma unroll
            for (int t = 0; t < kBatch; ++t)
                copy_async16(to + t * 512, src + (t0 + t) * kRows * D, (t0 + t) * kRows + sub < held);
            ++fetched;
            if (fetched % kPerHead == 0) src += BS * D;
        }
        copy_async_commit();
    };
#pragma unroll
    for (int f = 0; f < kPieces; ++f) fetch();
    Range<T> r;
    for (int done = 0; done < pieces; ++done) {
        copy_async_wait<kPieces - 1>();
        if (kPerHead == 1 || done % kPerHead == 0) r.clear();
        const int t0 = done % kPerHead * kBatch;
        const uint8_t* from = mine + done % kPieces * kPieceBytes;
        uint4 rows[kBatch];
#pragma unroll
        for (int t = 0; t < kBatch; ++t) rows[t] = *reinterpret_cast<const uint4*>(from + t * 512);
#pragma unroll
        for (int t = 0; t < kBatch; ++t)
            if ((t0 + t) * kRows + sub < held) r.take(rows[t]);
        fetch();
        if (kPerHead == 1 || (done + 1) % kPerHead == 0) {
#pragma unroll
            for (int m = kLanes; m < 32; m <<= 1) r.join(m);
            if (kRows == 1) {
                r.store(dst, false);
                r.store(dst + D, true);
            } else if (sub < 2) {
                r.store(dst, sub == 1);
            }
            dst += 2 * D;
        }
    }
    copy_async_wait<0>();
}

template <typename T, int D>
int launch_bounds(BoundsParams p, cudaStream_t st) {
    constexpr int kSmem = kWarps * kPieces * kPieceBytes;
    // a warp takes as many kv heads of a block as leave 64 warps an SM
    const int64_t all = (int64_t)p.batch * p.max_touched * p.num_kv_heads;
    const int64_t heads = std::max((int64_t)1, std::min((int64_t)p.num_kv_heads, all / ((int64_t)num_sms() * 64)));
    p.parts = (int)((p.num_kv_heads + heads - 1) / heads);
    p.heads_per_warp = (p.num_kv_heads + p.parts - 1) / p.parts;
    const int64_t per_seq = (int64_t)p.max_touched * p.parts;
    if (per_seq > 0x7fffffff / p.batch) return PA_ERR_UNSUPPORTED;  // warps are counted in 32 bits
    const int64_t blocks = (p.batch * per_seq + kWarps - 1) / kWarps;
    auto kernel = p.block_size == 8    ? key_bounds_kernel<T, D, 8>
                  : p.block_size == 16 ? key_bounds_kernel<T, D, 16>
                                       : key_bounds_kernel<T, D, 32>;
    static std::atomic<unsigned long long> configured{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        const void* const kernels[] = {(const void*)key_bounds_kernel<T, D, 8>, (const void*)key_bounds_kernel<T, D, 16>,
                                       (const void*)key_bounds_kernel<T, D, 32>};
        for (const void* k : kernels)
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
                return PA_ERR_CUDA;
        configured.fetch_or(bit);
    }
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kWarps * 32), kSmem, st, p);
}

// ---------------------------------------------------------------------------
// block scores
// ---------------------------------------------------------------------------
struct ScoreParams {
    const void *q, *key_bounds;
    const int32_t *block_tables, *seq_ids, *context_lens;
    int max_blocks_per_seq, batch, max_context_len, block_size;
    float* scores;
    int64_t score_stride;  // blocks of one (row, kv head) of scores
    int64_t num_rows;
    int num_q_heads, num_kv_heads;
    int64_t num_blocks;
    // a CTA's warps take head_warps kv heads side by side, each tiles_per_warp
    // tiles of 16 blocks: `parts` CTAs for a row's heads, `chunks` for its tiles
    int head_warps, tiles_per_warp, parts, chunks;
    int* err;
};

// This warp's part of a row: one kv head of `tiles_per_warp` tiles of 16
// blocks, `stride` tiles apart.
struct WarpTiles {
    const int32_t* table;
    int64_t row;
    int h, blocks, first, end, stride;
    bool named, recorder;  // the row's sequence exists; this thread reports a bad row
};

// Where the warp is, without the row's length: its table may be read beside it.
__device__ __forceinline__ WarpTiles warp_tiles(const ScoreParams& p) {
    WarpTiles w;
    const uint32_t unit = blockIdx.x / p.chunks;
    const int chunk = (int)(blockIdx.x % p.chunks), warp = threadIdx.x >> 5;
    w.row = unit / p.parts;
    w.h = (int)(unit % p.parts) * p.head_warps + (warp & (p.head_warps - 1));
    const int64_t seq = p.seq_ids ? (int64_t)p.seq_ids[w.row] : w.row;
    w.named = seq >= 0 && seq < p.batch;
    w.recorder = chunk == 0 && w.h == 0 && threadIdx.x == 0;
    w.table = p.block_tables + (w.named ? seq : 0) * p.max_blocks_per_seq;
    w.stride = kWarps / p.head_warps;
    w.first = chunk * w.stride * p.tiles_per_warp + warp / p.head_warps;
    w.end = w.h < p.num_kv_heads ? w.first + w.stride * p.tiles_per_warp : 0;
    w.blocks = 0;
    return w;
}

// Block j's table entry, read whether or not the row is that long.
__device__ __forceinline__ int32_t entry_of(const ScoreParams& p, const WarpTiles& w, int j) {
    return w.named && j < p.max_blocks_per_seq ? w.table[j] : -1;
}

// The row's length, which ends the warp's tiles.
__device__ __forceinline__ void end_tiles(const ScoreParams& p, WarpTiles& w) {
    const int L = p.context_lens[w.row];
    if (!w.named || L < 0 || L > p.max_context_len) {
        if (w.recorder) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
    } else {
        w.blocks = (int)(((int64_t)L + p.block_size - 1) >> block_shift(p.block_size));
    }
    w.end = min(w.end, (w.blocks + 15) / 16);
}

// The physical block of the row's block j from its entry; -1 past the row's
// blocks and (recorded) where it is bad.
__device__ __forceinline__ int32_t block_of(const ScoreParams& p, const WarpTiles& w, int j, int32_t entry) {
    if (j >= w.blocks) return -1;
    if (entry < 0 || entry >= p.num_blocks) {
        record_error(p.err, PA_ERR_BAD_BLOCK_ID);
        return -1;
    }
    return entry;
}

// The table entries of a warp's tiles, looked up two tiles (a pair) at a time:
// lane i holds block i % 16 of tile 2 * pair + i / 16 of the warp's sequence,
// e0 of the pair being scored, e1 of the next one, which is being fetched.
struct Entries {
    int32_t e0, e1;
    int j, last, pair;
    int apart;  // blocks between a lane's blocks of two pairs

    // Reads beside the row's length; false where the warp has no tile.
    __device__ __forceinline__ bool open(const ScoreParams& p, WarpTiles& w) {
        const int lane = threadIdx.x & 31;
        j = (w.first + (lane >> 4) * w.stride) * 16 + (lane & 15);
        apart = 2 * 16 * w.stride;
        e0 = entry_of(p, w, j);
        e1 = entry_of(p, w, j + apart);
        end_tiles(p, w);
        if (w.first >= w.end) return false;
        last = w.end * 16;  // blocks of other CTAs lie behind
        e0 = j < last ? block_of(p, w, j, e0) : -1;
        j += apart;
        e1 = j < last ? block_of(p, w, j, e1) : -1;
        pair = 0;
        return true;
    }
    __device__ __forceinline__ int32_t at(int tile, int block) const {  // of the warp's sequence
        return __shfl_sync(0xffffffffu, (tile >> 1) == pair ? e0 : e1, (tile & 1) * 16 + block);
    }
    __device__ __forceinline__ void next_pair(const ScoreParams& p, const WarpTiles& w) {
        ++pair;
        e0 = e1;
        j += apart;
        e1 = j < last ? block_of(p, w, j, entry_of(p, w, j)) : -1;
    }
};

// bf16.  max(q lo, q hi) is q hi where q >= 0 and q lo where q < 0, so a score
// is the dot product of (q-, q+) with (lo, hi) over 2 D terms, all of whose
// products are exact: a matrix product (m16n8k16) of 16 blocks with the group's
// heads, padded to 8 by repeats, which leave the maximum alone.  Bound by the
// read of the bounds: a block's two rows are 4 D contiguous bytes, copied
// asynchronously into a ring of one or two tiles that belongs to the warp alone.
// 16-byte chunk c of block b lies at c ^ (b & 7), so that the eight rows of a
// matrix load touch all banks.
// Measured: 16 contexts of 32k to 131k tokens, 64 / 8 heads of 128 (313 MB): 49
// us, 6.4 TB/s, 0.97 of a copy; 256 of up to 4096 tokens, 32 / 8 heads (50 MB):
// 13.3 us.
template <int D, int NT, int STAGES>
__global__ void __launch_bounds__(kWarps * 32, STAGES == 1 ? (NT == 1 ? 5 : 4) : 3) block_scores_mma_kernel(const ScoreParams p) {
    constexpr int kRowBytes = 4 * D;            // lo and hi of one block
    constexpr int kTile = 16 * kRowBytes;
    constexpr int kRowLanes = D / 4;            // lanes that copy one block
    constexpr int kCopyRows = 32 / kRowLanes;
    constexpr int kSteps = D / 16;
    extern __shared__ __align__(1024) uint8_t ring[];  // [warp][stage][16 blocks][lo, hi]
    griddep_wait();
    griddep_launch_dependents();
    WarpTiles w = warp_tiles(p);
    Entries e;
    if (!e.open(p, w)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int tiles = (w.end - w.first + w.stride - 1) / w.stride;

    const int group = p.num_q_heads / p.num_kv_heads;
    const int copy_row = lane / kRowLanes, copy_chunk = lane % kRowLanes;
    const __nv_bfloat16* bounds = static_cast<const __nv_bfloat16*>(p.key_bounds) + (int64_t)w.h * 2 * D + 8 * copy_chunk;
    const int64_t block_stride = (int64_t)p.num_kv_heads * 2 * D;
    const uint32_t slots = smem_addr(ring) + warp * (STAGES * kTile);
    const uint32_t copy_dst = slots + copy_row * kRowBytes;
    int fetched = 0;
    auto fetch = [&](int stage) {
        if (fetched < tiles) {
#pragma unroll
            for (int u = 0; u < 16; u += kCopyRows) {
                const int32_t blk = e.at(fetched, u + copy_row);
                const uint32_t dst = copy_dst + stage * kTile + u * kRowBytes + ((copy_chunk ^ ((u + copy_row) & 7)) << 4);
                copy_async16(dst, bounds + (blk < 0 ? 0 : blk) * block_stride, blk >= 0);
            }
            ++fetched;
        }
        copy_async_commit();
    };
#pragma unroll
    for (int st = 0; st < STAGES; ++st) fetch(st);

    // column 8 n + g of Q^T; its negative values (side 0) meet lo, the others hi
    uint32_t q[2][NT][kSteps][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const __nv_bfloat16* src =
            static_cast<const __nv_bfloat16*>(p.q) + (w.row * p.num_q_heads + w.h * group + (8 * n + g) % group) * D + 2 * t;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint32_t x = *reinterpret_cast<const uint32_t*>(src + 16 * i + 8 * c);
                uint32_t neg;  // the sign of each half, all over it
                asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(neg) : "r"(x));
                q[0][n][i][c] = x & neg;
                q[1][n][i][c] = x & ~neg;
            }
    }
    // matrix loads: lane = (matrix, row), the matrices (8 blocks, chunk of 8 channels)
    const uint32_t mat_row = lane & 7, mat_lo = (lane >> 3) & 1, mat_hi = lane >> 4;
    const uint32_t mat = slots + (mat_lo * 8 + mat_row) * kRowBytes + ((mat_hi ^ mat_row) << 4);
    float* out = p.scores + (w.row * p.num_kv_heads + w.h) * p.score_stride + w.first * 16;
    int stage = 0;
    for (int tile = 0; tile < tiles; ++tile, stage ^= STAGES - 1, out += w.stride * 16) {
        const unsigned have = __ballot_sync(0xffffffffu, e.e0 >= 0) >> (16 * (tile & 1));
        copy_async_wait<STAGES - 1>();
        __syncwarp();  // every lane's copies are in
        float s[2][NT][4] = {};
#pragma unroll
        for (int side = 0; side < 2; ++side)
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                uint32_t a[4];
                ldmatrix_x4((mat ^ (i << 5)) + stage * kTile + side * 2 * D, a[0], a[1], a[2], a[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16_16816(s[side][n], a, q[side][n][i][0], q[side][n][i][1]);
            }
        __syncwarp();  // every lane has read the stage
        fetch(stage);
        // heads 2 t, 2 t + 1 (+ 8) of blocks g and g + 8
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            float best = max_nan(s[0][0][2 * a] + s[1][0][2 * a], s[0][0][2 * a + 1] + s[1][0][2 * a + 1]);
            if (NT == 2)
                best = max_nan(best, max_nan(s[0][NT - 1][2 * a] + s[1][NT - 1][2 * a],
                                             s[0][NT - 1][2 * a + 1] + s[1][NT - 1][2 * a + 1]));
            best = max_nan(best, __shfl_xor_sync(0xffffffffu, best, 1));
            best = max_nan(best, __shfl_xor_sync(0xffffffffu, best, 2));
            if (t == a && (have >> (g + 8 * a) & 1)) out[g + 8 * a] = best;
        }
        if (tile & 1) e.next_pair(p, w);
    }
    copy_async_wait<0>();
}

// fp32, on the CUDA cores: D / 4 lanes hold the two rows of a block, four
// channels each, four blocks of a lane group at a time, through a ring of four
// such pieces (a lane reads back only what it copied); their sums over the
// lanes by one reduce-scatter.  Measured: one query head a kv head 6.3 TB/s,
// eight 5.2 TB/s, bound there by the 16 multiply-adds an 8-byte pair of bounds.
template <int D, int G>
__global__ void __launch_bounds__(kWarps * 32, 3) block_scores_f32_kernel(const ScoreParams p) {
    constexpr int kLanes = D / 4;
    constexpr int kRows = 32 / kLanes;        // blocks side by side
    constexpr int kBlocks = 4;                // of one lane in a piece
    constexpr int kPiece = kBlocks * 2 * 512;
    constexpr int kPerTile = 16 / (kBlocks * kRows);
    constexpr int kStages = 4;
    constexpr int kHeld = kBlocks * G > kLanes ? kBlocks * G / kLanes : 1;  // sums in a lane
    extern __shared__ __align__(1024) uint8_t ring[];  // [warp][stage][block][lo, hi][lane]
    griddep_wait();
    griddep_launch_dependents();
    WarpTiles w = warp_tiles(p);
    Entries e;
    if (!e.open(p, w)) return;
    const int lane = threadIdx.x & 31, sub = lane / kLanes, x = lane % kLanes;
    const int tiles = (w.end - w.first + w.stride - 1) / w.stride;
    float4 neg[G], pos[G];  // q's negative values, which meet lo, and the others
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) +
                                                          (w.row * p.num_q_heads + w.h * G + i) * D + 4 * x);
        neg[i] = make_float4(q.x < 0.f ? q.x : 0.f, q.y < 0.f ? q.y : 0.f, q.z < 0.f ? q.z : 0.f, q.w < 0.f ? q.w : 0.f);
        pos[i] = make_float4(q.x < 0.f ? 0.f : q.x, q.y < 0.f ? 0.f : q.y, q.z < 0.f ? 0.f : q.z, q.w < 0.f ? 0.f : q.w);
    }
    const float* bounds = static_cast<const float*>(p.key_bounds) + (int64_t)w.h * 2 * D + 4 * x;
    const int64_t block_stride = (int64_t)p.num_kv_heads * 2 * D;
    uint8_t* mine = ring + (threadIdx.x >> 5) * (kStages * kPiece) + lane * 16;
    int f_tile = 0, f_part = 0;
    auto fetch = [&](int stage) {
        if (f_tile < tiles) {
            const uint32_t dst = smem_addr(mine) + stage * kPiece;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int32_t blk = e.at(f_tile, (f_part * kBlocks + b) * kRows + sub);
                const float* src = bounds + (blk < 0 ? 0 : blk) * block_stride;
                copy_async16(dst + b * 1024, src, blk >= 0);
                copy_async16(dst + b * 1024 + 512, src + D, blk >= 0);
            }
            if (++f_part == kPerTile) {
                f_part = 0;
                ++f_tile;
            }
        }
        copy_async_commit();
    };
#pragma unroll
    for (int st = 0; st < kStages; ++st) fetch(st);
    float* out = p.scores + (w.row * p.num_kv_heads + w.h) * p.score_stride + w.first * 16;
    int stage = 0;
    for (int tile = 0; tile < tiles; ++tile, out += w.stride * 16) {
        const unsigned have = __ballot_sync(0xffffffffu, e.e0 >= 0) >> (16 * (tile & 1));
        for (int part = 0; part < kPerTile; ++part, stage = (stage + 1) % kStages) {
            copy_async_wait<kStages - 1>();
            const float4* rows = reinterpret_cast<const float4*>(mine + stage * kPiece);
            float v[kBlocks * G];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const float4 lo = rows[b * 64], hi = rows[b * 64 + 32];
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    float a = neg[i].x * lo.x, c = pos[i].x * hi.x;
                    a = fmaf(neg[i].y, lo.y, a);
                    c = fmaf(pos[i].y, hi.y, c);
                    a = fmaf(neg[i].z, lo.z, a);
                    c = fmaf(pos[i].z, hi.z, c);
                    a = fmaf(neg[i].w, lo.w, a);
                    c = fmaf(pos[i].w, hi.w, c);
                    v[b * G + i] = a + c;
                }
            }
            fetch(stage);
            reduce_scatter<kBlocks * G, kLanes>(v);
            // lane x holds heads of block x / (kLanes / kBlocks)
            float best = v[0];
#pragma unroll
            for (int i = 1; i < kHeld; ++i) best = max_nan(best, v[i]);
#pragma unroll
            for (int m = kLanes / kBlocks / 2; m; m >>= 1) best = max_nan(best, __shfl_xor_sync(0xffffffffu, best, m));
            const int block = (part * kBlocks + x / (kLanes / kBlocks)) * kRows + sub;
            if (x % (kLanes / kBlocks) == 0 && (have >> block & 1)) out[block] = best;
        }
        if (tile & 1) e.next_pair(p, w);
    }
    copy_async_wait<0>();
}

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------
struct SelectParams {
    const float* scores;
    int64_t score_stride;
    const int32_t* context_lens;
    int max_context_len, block_size;
    int32_t* selected;
    int max_selected, num_first, num_last;
    int64_t num_rows;
    int num_kv_heads;
    int* err;
};

// A score as an integer of the same order: NaN above +inf, -0 equal to +0.  No
// score gives 0, which marks what is not to be chosen from.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int sum_lanes(int x) { return __reduce_add_sync(0xffffffffu, x); }
__device__ __forceinline__ uint32_t min_lanes(uint32_t x) { return __reduce_min_sync(0xffffffffu, x); }
__device__ __forceinline__ uint32_t max_lanes(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }

// The row of one (row, kv head) as the selection sees it.
struct SelectRow {
    int32_t* out;
    int blocks;      // of the row
    int last;        // the first of its last num_last blocks
    int num_first, want;  // want: blocks to choose besides the first and last
    __device__ __forceinline__ bool always(int j) const { return j < num_first || j >= last; }
    __device__ __forceinline__ uint32_t key(int j, float score) const {
        return j < blocks && !always(j) ? score_key(score) : 0u;
    }
};

// False where the row is already written: no more blocks than max_selected
// (all of them), or a bad length (none).  Called by `threads` threads.
__device__ __forceinline__ bool select_row(const SelectParams& p, uint32_t unit, int thread, int threads, SelectRow& r) {
    const uint32_t row = unit / p.num_kv_heads;
    const int L = p.context_lens[row];
    r.out = p.selected + (int64_t)unit * p.max_selected;
    r.blocks = 0;
    if (L < 0 || L > p.max_context_len) {
        if (unit == row * p.num_kv_heads && thread == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
    } else {
        r.blocks = (int)(((int64_t)L + p.block_size - 1) >> block_shift(p.block_size));
    }
    if (r.blocks <= p.max_selected) {
        for (int i = thread; i < p.max_selected; i += threads) r.out[i] = i < r.blocks ? i : -1;
        return false;
    }
    r.num_first = p.num_first;
    r.last = r.blocks - p.num_last;
    r.want = p.max_selected - p.num_first - p.num_last;
    return true;
}

// Short rows, at most 32 * kShortItems blocks: one warp a row, its keys in
// registers.  The value of the last key to be taken is found by bisection, a
// count over the warp a step, which ends early at any value that exactly
// max_selected keys reach.  Bound by latency: 2048 rows of up to 256 blocks, 64
// kept, 5.3 us.
constexpr int kShortItems = 8;

__global__ void __launch_bounds__(kWarps * 32) select_short_kernel(const SelectParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= p.num_rows * p.num_kv_heads) return;
    const int lane = threadIdx.x & 31;
    // the scores are read beside the row's length, whether or not it is that long
    const float* scores = p.scores + unit * p.score_stride;
    float score[kShortItems];
#pragma unroll
    for (int i = 0; i < kShortItems; ++i) score[i] = 32 * i + lane < p.score_stride ? scores[32 * i + lane] : 0.f;
    SelectRow r;
    if (!select_row(p, unit, lane, 32, r)) return;
    uint32_t key[kShortItems], lo = 0xffffffffu, hi = 0;
#pragma unroll
    for (int i = 0; i < kShortItems; ++i) {
        key[i] = r.key(32 * i + lane, score[i]);
        hi = max(hi, key[i]);
        if (key[i]) lo = min(lo, key[i]);
    }
    lo = min_lanes(lo);
    hi = max_lanes(hi);
    // every key above hi is taken, none below lo; `want` of those in lo .. hi
    int want = r.want;
    if (want == 0) {
        lo = hi = 0xffffffffu;
    } else {
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            int n = 0;
#pragma unroll
            for (int i = 0; i < kShortItems; ++i) n += key[i] >= mid && key[i] <= hi;
            n = sum_lanes(n);
            if (n == want) {
                lo = mid;
                break;
            }
            if (n > want) {
                lo = mid;
            } else {
                want -= n;
                hi = mid - 1;
            }
        }
    }
    int at = 0;
    const unsigned below = (1u << lane) - 1u;
#pragma unroll
    for (int i = 0; i < kShortItems; ++i) {
        const int j = 32 * i + lane;
        const unsigned edge = __ballot_sync(0xffffffffu, want > 0 && key[i] >= lo && key[i] <= hi);
        const bool sure = (j < r.blocks && r.always(j)) || key[i] > hi;
        const bool take = sure || ((edge >> lane & 1u) && __popc(edge & below) < want);
        const unsigned taken = __ballot_sync(0xffffffffu, take);
        if (take) r.out[at + __popc(taken & below)] = j;
        at += __popc(taken);
        want -= min(want, __popc(edge));
    }
}

// Long rows: one CTA a row.  The range of keys that holds the last one to be
// taken is narrowed by histograms of kBins equal parts of it, until all of the
// range is to be taken or it is one value; scores lie close together, so parts
// of their own range tell them apart where the leading bits of a radix select
// would all be the same (and the counters' atomics would collide).  Counts are
// integers: the order of the atomics changes nothing.  Rows of up to THREADS *
// kItems blocks are read once, longer ones once a pass.  Bound by latency and
// barriers: 128 rows of 2048 to 8192 blocks, 256 kept, 7.6 us.
constexpr int kBins = 2048;

template <int THREADS, int kItems>
__global__ void __launch_bounds__(THREADS) select_long_kernel(const SelectParams p) {
    constexpr int kW = THREADS / 32;
    constexpr int kOwn = kBins / THREADS;  // bins of one thread
    __shared__ int hist[kBins];
    __shared__ uint32_t s_lo[kW], s_hi[kW];
    __shared__ int s_sum[kW], s_edge[kW];
    __shared__ int s_bin, s_above, s_count;
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // warp w's part of a chunk is contiguous, item i its i-th 32 blocks; the first
    // chunk is read beside the row's length, whether or not it is that long
    const float* scores = p.scores + blockIdx.x * p.score_stride;
    auto first_of = [&](int chunk) { return chunk * THREADS * kItems + warp * 32 * kItems + lane; };
    float score[kItems];
    auto read = [&](int chunk) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int j = first_of(chunk) + 32 * i;
            score[i] = j < p.score_stride ? scores[j] : 0.f;
        }
    };
    read(0);
    SelectRow r;
    if (!select_row(p, blockIdx.x, tid, THREADS, r)) return;
    const int chunks = (r.blocks + THREADS * kItems - 1) / (THREADS * kItems);
    uint32_t key[kItems];
    auto load = [&](int chunk) {
        if (chunk > 0 || chunks > 1) read(chunk);
#pragma unroll
        for (int i = 0; i < kItems; ++i) key[i] = r.key(first_of(chunk) + 32 * i, score[i]);
    };
#pragma unroll
    for (int i = 0; i < kOwn; ++i) hist[tid * kOwn + i] = 0;
    uint32_t lo = 0xffffffffu, hi = 0;
    for (int c = 0; c < chunks; ++c) {
        load(c);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            hi = max(hi, key[i]);
            if (key[i]) lo = min(lo, key[i]);
        }
    }
    lo = min_lanes(lo);
    hi = max_lanes(hi);
    if (lane == 0) {
        s_lo[warp] = lo;
        s_hi[warp] = hi;
    }
    __syncthreads();
    lo = min_lanes(s_lo[lane % kW]);
    hi = max_lanes(s_hi[lane % kW]);

    // every key above hi is taken, none below lo; `want` of the `count` in lo .. hi
    int want = r.want, count = r.blocks - p.num_first - p.num_last;
    if (want == 0) lo = hi = 0xffffffffu;
    while (want > 0 && want < count && lo < hi) {
        const int shift = max(0, 21 - __clz(hi - lo));  // (hi - lo) >> shift < kBins
        for (int c = 0; c < chunks; ++c) {
            if (chunks > 1) load(c);
#pragma unroll
            for (int i = 0; i < kItems; ++i)
                if (key[i] >= lo && key[i] <= hi) atomicAdd(&hist[(key[i] - lo) >> shift], 1);
        }
        __syncthreads();
        // thread t owns bins top - t * kOwn and below; sums from the top
        int own[kOwn], sum = 0;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int b = kBins - 1 - (tid * kOwn + i);
            own[i] = hist[b];
            hist[b] = 0;
            sum += own[i];
        }
        int upto = sum;  // of this warp's threads up to this one
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += x;
        }
        if (lane == 31) s_sum[warp] = upto;
        __syncthreads();
        int above = upto - sum + sum_lanes(lane < warp ? s_sum[lane % kW] : 0);
        if (above < want && above + sum >= want) {  // one thread
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                if (above < want && above + own[i] >= want) {
                    s_bin = kBins - 1 - (tid * kOwn + i);
                    s_above = above;
                    s_count = own[i];
                }
                above += own[i];
            }
        }
        __syncthreads();
        want -= s_above;
        count = s_count;
        lo += (uint32_t)s_bin << shift;
        hi = min(hi - lo, (1u << shift) - 1u) + lo;
    }

    // in ascending order: those surely taken, and the first `want` of lo .. hi
    int done = 0, edges = 0;
    const unsigned below = (1u << lane) - 1u;
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) load(c);
        unsigned sure[kItems], edge[kItems];
        int n_sure = 0, n_edge = 0;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int j = first_of(c) + 32 * i;
            sure[i] = __ballot_sync(0xffffffffu, (j < r.blocks && r.always(j)) || key[i] > hi);
            edge[i] = __ballot_sync(0xffffffffu, want > 0 && key[i] >= lo && key[i] <= hi);
            n_sure += __popc(sure[i]);
            n_edge += __popc(edge[i]);
        }
        __syncthreads();
        if (lane == 0) {
            s_sum[warp] = n_sure;
            s_edge[warp] = n_edge;
        }
        __syncthreads();
        const int all_sure = sum_lanes(lane < kW ? s_sum[lane] : 0), all_edge = sum_lanes(lane < kW ? s_edge[lane] : 0);
        int a = done + sum_lanes(lane < warp ? s_sum[lane % kW] : 0);
        int e = edges + sum_lanes(lane < warp ? s_edge[lane % kW] : 0);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const bool is_sure = sure[i] >> lane & 1u, is_edge = edge[i] >> lane & 1u;
            const int rank = e + __popc(edge[i] & below);
            if (is_sure || (is_edge && rank < want))
                r.out[a + __popc(sure[i] & below) + min(rank, want)] = first_of(c) + 32 * i;
            a += __popc(sure[i]);
            e += __popc(edge[i]);
        }
        done += all_sure;
        edges += all_edge;
    }
}

constexpr int kScoresSmem = kWarps * 16384;  // rings of 16 KB a warp (8 KB for bf16 of D 64)

int launch_scores_kernel(const ScoreParams& p, void (*kernel)(ScoreParams), std::atomic<unsigned long long>& configured,
                         int smem, cudaStream_t st) {
    int dev = 0;
    cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return PA_ERR_CUDA;
        configured.fetch_or(bit);
    }
    const int64_t grid = p.num_rows * p.parts;
    if (grid > 0x7fffffff / p.chunks) return PA_ERR_UNSUPPORTED;
    return launch_pdl(kernel, dim3((unsigned)(grid * p.chunks)), dim3(kWarps * 32), smem, st, p);
}

template <int D, int NT>
int launch_scores_mma(const ScoreParams& p, bool brief, cudaStream_t st) {
    constexpr int kTile = kWarps * 16 * 4 * D;
    static std::atomic<unsigned long long> one{0}, two{0};
    return brief ? launch_scores_kernel(p, block_scores_mma_kernel<D, NT, 1>, one, kTile, st)
                 : launch_scores_kernel(p, block_scores_mma_kernel<D, NT, 2>, two, 2 * kTile, st);
}

template <int D, int G>
int launch_scores_f32(const ScoreParams& p, cudaStream_t st) {
    static std::atomic<unsigned long long> configured{0};
    return launch_scores_kernel(p, block_scores_f32_kernel<D, G>, configured, kScoresSmem, st);
}

int launch_scores(ScoreParams p, int head_dim, int dtype, cudaStream_t st) {
    const int64_t tiles = ((int64_t)p.max_context_len + 16 * p.block_size - 1) / (16 * p.block_size);
    const int64_t all = p.num_rows * p.num_kv_heads * tiles, sms = num_sms();
    // A CTA's warps take heads side by side: they share a row's look-ups, and a
    // row of one tile has work for all of them (256 rows of one tile, 8 kv
    // heads: 4.4 us, against 7.1 with a head's tiles side by side).  Up to
    // four tiles a warp as long as that leaves 12 warps an SM (16 contexts of 32k
    // to 131k tokens: 59 us with one, 50 with four or eight; 256 of up to 4096:
    // 18.5 with one, 13.4 with four, 15.8 with eight; 256 of 700: 12.0 with one,
    // 10.9 with three; 64 of 2000: 7.8 with two, 8.4 with one).
    p.head_warps = p.num_kv_heads > 2 ? kWarps : p.num_kv_heads;
    const int per_cta = kWarps / p.head_warps;  // tiles side by side
    p.parts = (p.num_kv_heads + p.head_warps - 1) / p.head_warps;
    p.tiles_per_warp = (int)std::max((int64_t)1, std::min((int64_t)4, all / (sms * 12)));
    p.chunks = (int)((tiles + per_cta * p.tiles_per_warp - 1) / (per_cta * p.tiles_per_warp));
    // A ring of two tiles pays only where all warps have several: 49.1 against
    // 50.0 us for the 16 long contexts.  In a batch of shorter rows, ragged as a
    // rule, most have fewer, and five CTAs an SM with one tile each do better
    // than three with two (256 rows of up to 16k tokens: 31.0 against 34.6 us,
    // of 700 tokens 10.9 against 12.5).
    const bool brief = tiles <= 128 || p.tiles_per_warp == 1;
    const int group = p.num_q_heads / p.num_kv_heads;
    const bool wide = head_dim == 128;
    if (dtype == PA_BF16) {
        if (group == 16) return wide ? launch_scores_mma<128, 2>(p, brief, st) : launch_scores_mma<64, 2>(p, brief, st);
        return wide ? launch_scores_mma<128, 1>(p, brief, st) : launch_scores_mma<64, 1>(p, brief, st);
    }
    switch (group) {
        case 1: return wide ? launch_scores_f32<128, 1>(p, st) : launch_scores_f32<64, 1>(p, st);
        case 2: return wide ? launch_scores_f32<128, 2>(p, st) : launch_scores_f32<64, 2>(p, st);
        case 4: return wide ? launch_scores_f32<128, 4>(p, st) : launch_scores_f32<64, 4>(p, st);
        case 8: return wide ? launch_scores_f32<128, 8>(p, st) : launch_scores_f32<64, 8>(p, st);
    }
    return PA_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_update_key_bounds(const void* k_pool, void* key_bounds, const int32_t* block_tables,
                                    int max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_start,
                                    int max_query_len, int batch, int num_kv_heads, int head_dim, int block_size,
                                    int64_t num_blocks, int dtype, void* stream) {
    PA_NVTX_RANGE("pa_update_key_bounds");
    if (batch < 0 || max_blocks_per_seq < 0 || max_query_len < 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        block_size <= 0 || num_blocks < 0 || !valid_dtype(dtype) || (!query_start && max_query_len < 1))
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size)) return PA_ERR_UNSUPPORTED;
    if (batch == 0 || max_query_len == 0) return PA_OK;
    if (!k_pool || !key_bounds || !block_tables || !context_lens || !aligned16(k_pool) || !aligned16(key_bounds))
        return PA_ERR_INVALID_ARG;
    BoundsParams p = {};
    p.k_pool = k_pool;
    p.key_bounds = key_bounds;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.max_query_len = query_start ? max_query_len : 1;
    p.batch = batch;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    // n tokens that end anywhere lie in at most (n - 2) / bs + 2 blocks
    p.max_touched = (int)(((int64_t)p.max_query_len + block_size - 2) / block_size) + 1;
    if (p.max_touched > max_blocks_per_seq) p.max_touched = max_blocks_per_seq > 0 ? max_blocks_per_seq : 1;
    p.err = error_word_ptr();
    if (!p.err) return PA_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == PA_BF16)
        return head_dim == 128 ? launch_bounds<__nv_bfloat16, 128>(p, st) : launch_bounds<__nv_bfloat16, 64>(p, st);
    return head_dim == 128 ? launch_bounds<float, 128>(p, st) : launch_bounds<float, 64>(p, st);
}

extern "C" int pa_block_scores(const void* q, const void* key_bounds, const int32_t* block_tables,
                               int max_blocks_per_seq, const int32_t* seq_ids, const int32_t* context_lens,
                               int max_context_len, int block_size, float* scores, int64_t score_stride,
                               int64_t num_rows, int batch, int num_q_heads, int num_kv_heads, int head_dim,
                               int64_t num_blocks, int dtype, void* stream) {
    PA_NVTX_RANGE("pa_block_scores");
    if (num_rows < 0 || batch < 0 || max_blocks_per_seq < 0 || max_context_len < 0 || num_q_heads <= 0 ||
        num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0 || !valid_dtype(dtype) ||
        num_q_heads % num_kv_heads != 0)
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size) ||
        !supported_group(num_q_heads / num_kv_heads, dtype) || num_rows > 0x7fffffff)
        return PA_ERR_UNSUPPORTED;
    const int64_t max_blocks = ((int64_t)max_context_len + block_size - 1) / block_size;
    if (max_context_len > (int64_t)max_blocks_per_seq * block_size || score_stride < max_blocks ||
        (!seq_ids && num_rows > batch))
        return PA_ERR_INVALID_ARG;
    if (num_rows == 0 || max_context_len == 0) return PA_OK;
    if (!q || !key_bounds || !block_tables || !context_lens || !scores || !aligned16(q) || !aligned16(key_bounds) ||
        !aligned16(scores))
        return PA_ERR_INVALID_ARG;
    ScoreParams p = {};
    p.q = q;
    p.key_bounds = key_bounds;
    p.block_tables = block_tables;
    p.seq_ids = seq_ids;
    p.context_lens = context_lens;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.batch = batch;
    p.max_context_len = max_context_len;
    p.block_size = block_size;
    p.scores = scores;
    p.score_stride = score_stride;
    p.num_rows = num_rows;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.num_blocks = num_blocks;
    p.err = error_word_ptr();
    if (!p.err) return PA_ERR_CUDA;
    return launch_scores(p, head_dim, dtype, static_cast<cudaStream_t>(stream));
}

extern "C" int pa_select_blocks(const float* scores, int64_t score_stride, const int32_t* context_lens,
                                int max_context_len, int block_size, int32_t* selected, int max_selected,
                                int num_first, int num_last, int64_t num_rows, int num_kv_heads, void* stream) {
    PA_NVTX_RANGE("pa_select_blocks");
    if (num_rows < 0 || num_kv_heads <= 0 || max_context_len < 0 || block_size <= 0 || max_selected <= 0 ||
        num_first < 0 || num_last < 0 || (int64_t)num_first + num_last > max_selected)
        return PA_ERR_INVALID_ARG;
    if (!supported_block_size(block_size) || num_rows > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    if (score_stride < ((int64_t)max_context_len + block_size - 1) / block_size) return PA_ERR_INVALID_ARG;
    if (num_rows == 0) return PA_OK;
    // scores without columns (max_context_len 0) may have no address: nothing of them is read
    if ((!scores && score_stride > 0) || !context_lens || !selected || !aligned16(scores) || !aligned16(selected))
        return PA_ERR_INVALID_ARG;
    const int64_t grid = num_rows * num_kv_heads;
    if (grid > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    SelectParams p = {};
    p.scores = scores;
    p.score_stride = score_stride;
    p.context_lens = context_lens;
    p.max_context_len = max_context_len;
    p.block_size = block_size;
    p.selected = selected;
    p.max_selected = max_selected;
    p.num_first = num_first;
    p.num_last = num_last;
    p.num_rows = num_rows;
    p.num_kv_heads = num_kv_heads;
    p.err = error_word_ptr();
    if (!p.err) return PA_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // by the longest row that may come: a warp a row while its keys fit the
    // warp's registers, then a CTA of 512 threads with four blocks each (512 rows
    // of up to 1000 blocks: 9.9 us, with 256 threads 10.3, with 1024 14.0), or of
    // 1024 with eight (128 rows of 2048 to 8192 blocks: 7.6 us, 8.1 with 512)
    const int64_t blocks = ((int64_t)max_context_len + block_size - 1) / block_size;
    if (blocks <= 32 * kShortItems)
        return launch_pdl(select_short_kernel, dim3((unsigned)((grid + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0, st, p);
    if (blocks <= 2048) return launch_pdl(select_long_kernel<512, 4>, dim3((unsigned)grid), dim3(512), 0, st, p);
    return launch_pdl(select_long_kernel<1024, 8>, dim3((unsigned)grid), dim3(1024), 0, st, p);
}
