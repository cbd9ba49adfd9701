// The projections of project.cu for many tokens: compute-bound, on CTA pairs.
//
// A tile is 256 tokens x 256 (or 128) accumulator columns, computed by a pair
// of CTAs with cta_group::2 products: each CTA loads its half of the tokens
// and its half of the W rows (for the gated form one CTA loads gate rows, the
// other the up rows of the same outputs, so the two halves of a tile's columns
// are act's argument and its factor), and holds the accumulator of its own 128
// tokens in TMEM, twice, so the epilogue of one tile runs under the products
// of the next.  One warp per CTA loads by TMA into a ring, one warp of the pair
// issues the products, eight warps of each CTA read the accumulator, add the
// bias, the activation, the factor and the residual in fp32, round, and send
// boxes of 32 tokens to y by TMA.  The pairs are persistent and walk the tiles
// in groups of eight token tiles, so that the tiles in flight share both
// operands in L2.
//
// A 64-column chunk of a wide tile takes 505 cycles, the products' own time;
// beyond a few milliseconds of work the board's power limit sets the clock
// (1.2-1.5 GHz of 1.97), which then bounds the call together with the last
// round, in which not all pairs have a tile: 4096 tokens, 11008 -> 4096, 295-313
// us (1.18-1.25 PFLOP/s; 3.46 rounds run as 4; a library's plain product 279 us),
// 2001 tokens through the 7B gate and up, 276-283 us (1.28-1.31 PFLOP/s; 9.3
// rounds run as 10).
//
// fp32 outputs take a fresh accumulator every 512 columns of d_in, added up in
// the epilogue's registers (the tensor core's rounding towards zero adds up
// over long sums, see project.cu).
#include <algorithm>
#include <atomic>

#include "act.cuh"
#include "project.h"
#include "ptx_ops.cuh"

namespace af {
namespace {

constexpr int kTileThreads = 320;               // producer, MMA, eight epilogue warps
constexpr int kEpiWarps = 8;
constexpr int kPairTokens = 256;
constexpr int kGroup = 8;                       // token tiles per group of the walk
constexpr uint32_t kTileSmem = 226 * 1024;      // the whole SM: no other tcgen05 kernel beside a pair
constexpr uint32_t kBox = 32 * 128;             // a warp's box of outputs: 32 rows of up to 128 bytes
constexpr uint32_t kBoxBytes = kEpiWarps * kBox;
constexpr uint32_t kXBytes = 128 * kChunkK * 2; // a CTA's tokens of a chunk

// A stage holds one chunk of a wide tile, two of a narrow one: the waits and
// the commit of a stage, with four products of 128 columns, took the issuing
// warp 500 cycles, as long as four of 256 columns take the tensor core.
template <int kCols>
struct Ring {
    static constexpr int kPer = kCols == 128 ? 2 : 1;              // chunks per stage
    static constexpr uint32_t kWBytes = kCols / 2 * kChunkK * 2;
    static constexpr uint32_t kChunk = kXBytes + kWBytes;
    static constexpr uint32_t kStage = kPer * kChunk;
    static constexpr int kStages = (int)((kTileSmem - 1024 - kBoxBytes) / kStage);
};

struct TileArgs : ProjectArgs {
    int32_t m_tiles, n_tiles, out_cols;         // outputs per tile
    int32_t part;                               // chunks per accumulator
    uint32_t tiles;
};

// Adds p[0 .. N) (bf16, 16-byte aligned) to v; groups of 8 from `limit` on are not read.
template <int N>
__device__ __forceinline__ void add_bf16(float (&v)[N], const uint16_t* p, int limit)
{
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        if (i < limit) {
            const uint4 w = *reinterpret_cast<const uint4*>(p + i);
            v[i] += bf16lo(w.x); v[i + 1] += bf16hi(w.x); v[i + 2] += bf16lo(w.y); v[i + 3] += bf16hi(w.y);
            v[i + 4] += bf16lo(w.z); v[i + 5] += bf16hi(w.z); v[i + 6] += bf16lo(w.w); v[i + 7] += bf16hi(w.w);
        }
    }
}

template <int N>
__device__ __forceinline__ void load_cols(uint32_t taddr, float (&v)[N])
{
    static_assert(N == 32, "one load");
    uint32_t r[32];
    tc_ld_x32(taddr, r);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ uint4 pack8(const float* v)
{
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

// Where a warp puts its outputs on their way to y: a box of 32 tokens x kRow
// bytes in shared memory, in the layout that the tensor map of y swizzles, so
// that lanes that write a row each meet no bank twice.
template <int kRow>
struct Box {
    static_assert(kRow == 128 || kRow == 64, "a swizzled row");
    uint8_t* at;
    // 16 bytes of the lane's row
    __device__ __forceinline__ void put(int piece, uint4 w) const
    {
        const int r = threadIdx.x & 31, turned = kRow == 128 ? piece ^ (r & 7) : piece ^ ((r >> 1) & 3);
        *reinterpret_cast<uint4*>(at + r * kRow + turned * 16) = w;
    }
    // the box may be written again once the copy of its last contents has read it
    __device__ __forceinline__ void wait() const
    {
        bulk_wait_group_read<0>();
        __syncwarp();
    }
    __device__ __forceinline__ void send(const CUtensorMap* y, int o, int t) const
    {
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) tma_store_2d(y, at, o, t);
        bulk_commit_group();
    }
};

__device__ __forceinline__ void add_bf16(float (&v)[32], const uint4 (&w)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[8 * i] += bf16lo(w[i].x); v[8 * i + 1] += bf16hi(w[i].x);
        v[8 * i + 2] += bf16lo(w[i].y); v[8 * i + 3] += bf16hi(w[i].y);
        v[8 * i + 4] += bf16lo(w[i].z); v[8 * i + 5] += bf16hi(w[i].z);
        v[8 * i + 6] += bf16lo(w[i].w); v[8 * i + 7] += bf16hi(w[i].w);
    }
}

// 32 residuals of a lane's token, outputs o .., loaded ahead of their use.
struct Residual {
    uint4 w[4];
    __device__ __forceinline__ void load(const ProjectArgs& a, int64_t t, int o)
    {
        if (!a.residual || t >= a.T) return;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (o + 8 * i < a.N) w[i] = *reinterpret_cast<const uint4*>(a.residual + t * a.ldr + o + 8 * i);
    }
    __device__ __forceinline__ void add(const ProjectArgs& a, float (&v)[32]) const
    {
        if (a.residual) add_bf16(v, w);
    }
};

// Puts 32 finished columns of the lane's token into the box.
template <bool kF32, int kRow>
__device__ __forceinline__ void put32(const float (&v)[32], Box<kRow> box, int piece)
{
    if constexpr (kF32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            box.put(piece + i, make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                          __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) box.put(piece + i, pack8(v + 8 * i));
    }
}

// Bytes of a row of a box.
template <int kCols, bool kGated, bool kF32>
__host__ __device__ constexpr int box_row()
{
    return kGated && kCols == 128 ? 64 : 128;
}

// kCols: accumulator columns of a tile.  kF32: fp32 outputs (never gated).
template <int kCols, bool kGated, bool kF32>
__global__ void __launch_bounds__(kTileThreads, 1) tile_kernel(const __grid_constant__ CUtensorMap xmap,
                                                               const __grid_constant__ CUtensorMap wmap,
                                                               const __grid_constant__ CUtensorMap umap,
                                                               const __grid_constant__ CUtensorMap ymap,
                                                               const TileArgs a)
{
    using R = Ring<kCols>;
    constexpr int kStages = R::kStages;
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t full[kStages], empty[kStages], accfull[2], accempty[2], done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    uint8_t* boxes = ring + (size_t)kStages * R::kStage;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const uint32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (warp == 2 && elect_one()) {
        prefetch_map(&xmap);
        prefetch_map(kGated && rank ? &umap : &wmap);
    }
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accempty[i], 2 * kEpiWarps);
        }
        mbar_init(&done, 1);
        fence_mbar_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 1) {
        tmem_alloc_pair(&tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // tile i of the walk: groups of kGroup token tiles, token tiles fastest (in
    // 32 bits: three 64-bit divisions by variables took 3000 cycles of every tile)
    const auto tile_at = [&](uint32_t i, int& m, int& n) {
        const uint32_t per = (uint32_t)(kGroup * a.n_tiles);
        const uint32_t g = i / per;
        const uint32_t rows = (uint32_t)min(kGroup, a.m_tiles - (int)g * kGroup);
        const uint32_t j = i - g * per;
        n = (int)(j / rows);
        m = (int)(g * kGroup + (j - (uint32_t)n * rows));
    };

    if (warp == 0) {
        // The whole warp walks the loop and one elected lane issues the copies
        // (and, below, the products: issued from a branch of one lane, with the
        // others parked, a 64-column chunk of a 256 x 256 tile took 705 cycles
        // instead of the 505 that its products take).
        int64_t it = 0;             // stages so far
        int s = 0;                  // the ring's next stage
        uint32_t lap = 1;           // parity that its `empty` completes with when free (the first lap: at once)
        bool stop = false;
        for (uint32_t i = pair; i < a.tiles && !stop; i += pairs) {
            int m, n;
            tile_at(i, m, n);
            const int t = m * kPairTokens + rank * 128;
            const int row = kGated ? n * a.out_cols : n * a.out_cols + rank * (kCols / 2);
            const CUtensorMap* w = kGated && rank ? &umap : &wmap;
            for (int c = 0; c < a.chunks; c += R::kPer, ++it) {
                if (!mbar_wait_warp(&empty[s], lap, &abort_flag)) {
                    stop = true;
                    break;
                }
                if (!(a.stall && blockIdx.x == 0 && it == 0) && elect_one()) {      // test hook: the first never arrives
                    uint8_t* p = ring + (size_t)s * R::kStage;
                    const uint32_t bar = cluster_map(smem_u32(&full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * R::kStage);
#pragma unroll
                    for (int j = 0; j < R::kPer; ++j) {         // past the last column: zeros
                        tma_load_2d_pair(p + j * R::kChunk, &xmap, bar, (c + j) * kChunkK, t);
                        tma_load_2d_pair(p + j * R::kChunk + kXBytes, w, bar, (c + j) * kChunkK, row);
                    }
                }
                __syncwarp();
                if (++s == kStages) { s = 0; lap ^= 1; }
            }
        }
        // Every stage's last products have signalled before the CTA leaves;
        // after an abort, what is in flight has landed.
        const int64_t from = max((int64_t)0, it - kStages);
        for (int64_t j = from; j < it; ++j)
            if (!mbar_wait_warp(&empty[j % kStages], (uint32_t)(j / kStages) & 1, &abort_flag)) break;
        if (rank == 0 && __any_sync(0xffffffffu, *(volatile int*)&abort_flag))
            for (int64_t j = from; j < it; ++j)
                if (!(a.stall && blockIdx.x == 0 && j == 0))
                    mbar_wait_landed(&full[j % kStages], (uint32_t)(j / kStages) & 1);
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t idesc = make_idesc_bf16(256, kCols, 0u, 0u);
            int s = 0;                  // the ring's next stage
            uint32_t lap = 0;           // parity that its `full` completes with
            uint32_t use = 0;           // accumulators so far
            const uint64_t xdesc = make_sdesc(smem_u32(ring), 16u, 1024u, kLayoutSw128);
            const uint64_t wdesc = make_sdesc(smem_u32(ring) + kXBytes, 16u, 1024u, kLayoutSw128);
            bool stop = false;
            for (uint32_t i = pair; i < a.tiles && !stop; i += pairs) {
                int left = 0;           // stages until the next accumulator
                for (int c = 0; c < a.chunks; c += R::kPer) {
                    const bool fresh = left == 0;
                    if (fresh) {
                        if (!mbar_wait_warp(&accempty[use & 1], ((use >> 1) & 1) ^ 1u, &abort_flag)) {
                            stop = true;
                            break;
                        }
                        tc_fence_after();
                        left = (min(kF32 ? a.part : a.chunks, a.chunks - c) + R::kPer - 1) / R::kPer;
                    }
                    if (!mbar_wait_warp(&full[s], lap, &abort_flag)) {
                        stop = true;
                        break;
                    }
                    --left;
                    if (elect_one()) {
                        const uint32_t d = tmem + (use & 1) * kCols;
                        const uint64_t at = (uint64_t)(s * (int)(R::kStage >> 4));
#pragma unroll
                        for (int j = 0; j < R::kPer; ++j)
#pragma unroll
                            for (int kk = 0; kk < kChunkK / 16; ++kk) {
                                const uint64_t off = at + (uint64_t)(j * (R::kChunk >> 4) + kk * 2);
                                tc_mma_bf16_pair(d, xdesc + off, wdesc + off, idesc, fresh && j + kk == 0 ? 0u : 1u);
                            }
                        tc_commit_pair(&empty[s]);
                        if (left == 0) tc_commit_pair(&accfull[use & 1]);
                    }
                    __syncwarp();
                    if (left == 0) ++use;
                    if (++s == kStages) { s = 0; lap ^= 1; }
                }
            }
            __syncwarp();
            if (elect_one()) tc_commit_pair(&done);         // in both CTAs, also after an abort
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;
        using B = Box<box_row<kCols, kGated, kF32>()>;
        const B box{boxes + (warp - 2) * kBox};
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        const uint32_t free0 = cluster_map(smem_u32(&accempty[0]), 0), free1 = cluster_map(smem_u32(&accempty[1]), 0);
        uint32_t use = 0;
        bool ok = true;
        // waits for the next accumulator; gives it back
        const auto take = [&]() {
            ok = mbar_wait_warp(&accfull[use & 1], (use >> 1) & 1, &abort_flag);
            tc_fence_after();
            return ok;
        };
        const auto give = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(use & 1 ? free1 : free0);
            ++use;
        };
        for (uint32_t i = pair; i < a.tiles; i += pairs) {
            int m, n;
            tile_at(i, m, n);
            const int64_t t0 = (int64_t)m * kPairTokens + rank * 128 + q * 32;
            if constexpr (kGated) {
                constexpr int kMine = kCols / 4;            // outputs per warp
                const int o0 = n * a.out_cols + half * kMine;
                if (!take()) break;
                const uint32_t d = lanes + (uint32_t)(use & 1) * kCols + half * kMine;
                box.wait();
#pragma unroll
                for (int c = 0; c < kMine; c += 32) {
                    float v[32], u[32];
                    load_cols(d + c, v);
                    load_cols(d + kCols / 2 + c, u);
                    if (a.bias) add_bf16(v, a.bias + o0 + c, a.N - o0 - c);
                    if (a.bias_up) add_bf16(u, a.bias_up + o0 + c, a.N - o0 - c);
                    activate_all(v, a.act);
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= u[j];
                    put32<false>(v, box, c / 8);
                }
                if (o0 < a.N && t0 < a.T) box.send(&ymap, o0, (int)t0);
                give();
            } else if constexpr (!kF32) {
                constexpr int kMine = kCols / 2;
                const int o0 = n * a.out_cols + half * kMine;
                Residual ahead;             // of the next step
                ahead.load(a, t0 + lane, o0);
                uint4 bias[4];
                const auto load_bias = [&](int o) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (a.bias && o + 8 * i < a.N) bias[i] = *reinterpret_cast<const uint4*>(a.bias + o + 8 * i);
                };
                load_bias(o0);
                if (!take()) break;
                const uint32_t d = lanes + (uint32_t)(use & 1) * kCols + half * kMine;
#pragma unroll
                for (int c = 0; c < kMine; c += 32) {
                    float v[32];
                    load_cols(d + c, v);
                    if (a.bias) add_bf16(v, bias);
                    if (c + 32 < kMine) load_bias(o0 + c + 32);
                    activate_all(v, a.act);
                    ahead.add(a, v);
                    if (c + 32 < kMine) ahead.load(a, t0 + lane, o0 + c + 32);
                    if (!(c & 32)) box.wait();
                    put32<false>(v, box, (c & 32) / 8);
                    if ((c & 32) && o0 + c - 32 < a.N && t0 < a.T) box.send(&ymap, o0 + c - 32, (int)t0);
                }
                give();
            } else {
                constexpr int kMine = kCols / 2, kParts = kMine / 32;
                const int o0 = n * a.out_cols + half * kMine;
                float v[kParts][32];
                for (int c0 = 0; c0 < a.chunks; c0 += a.part) {
                    if (!take()) break;
                    const uint32_t d = lanes + (uint32_t)(use & 1) * kCols + half * kMine;
#pragma unroll
                    for (int c = 0; c < kParts; ++c) {
                        float p[32];
                        load_cols(d + c * 32, p);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[c][j] = c0 ? v[c][j] + p[j] : p[j];
                    }
                    give();
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < kParts; ++c) {
                    const int o = o0 + c * 32;
                    Residual now;
                    now.load(a, t0 + lane, o);
                    if (a.bias) add_bf16(v[c], a.bias + o, a.N - o);
                    activate_all(v[c], a.act);
                    now.add(a, v[c]);
                    box.wait();
                    put32<true>(v[c], box, 0);
                    if (o < a.N && t0 < a.T) box.send(&ymap, o, (int)t0);
                }
            }
        }
    }
    if (warp >= 2) bulk_wait_group<0>();
    __syncthreads();
    if (threadIdx.x == 0 && *(volatile int*)&abort_flag && a.status) atomicOr(a.status, ADAFUSE_STATUS_TIMEOUT);
    // A CTA may leave once nothing of the other can still reach it: the products
    // have all signalled (after an abort too), and the second CTA's arrivals on
    // `accempty`, of which nobody waits for the last two, are released here.
    if (warp == 1) {
        mbar_wait_landed(&done, 0);
        __syncwarp();
    }
    cluster_sync_release();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// Tensor map of y: boxes of 32 tokens x `row` bytes, swizzled by the row's length.
bool encode_outputs(CUtensorMap* m, const ProjectArgs& a, int row)
{
    const cuuint64_t size = a.y_f32 ? 4 : 2;
    cuuint64_t dims[2] = {(cuuint64_t)a.N, (cuuint64_t)a.T};
    cuuint64_t strides[1] = {(cuuint64_t)(a.T > 1 ? a.ldy : (a.N + 7) / 8 * 8) * size};
    cuuint32_t box[2] = {(cuuint32_t)(row / size), 32};
    cuuint32_t estr[2] = {1, 1};
    return tensor_map_encoder()(m, a.y_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.y,
                                dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kCols, bool kGated, bool kF32>
int launch_tiles(ProjectCall& c, int pairs)
{
    TileArgs a{c.a};
    a.out_cols = kGated ? kCols / 2 : kCols;
    a.m_tiles = (int)((a.T + kPairTokens - 1) / kPairTokens);
    a.n_tiles = (a.N + a.out_cols - 1) / a.out_cols;
    const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
    if (tiles > 0x7fffffff || a.n_tiles > 0x7fffffff / kGroup) return ADAFUSE_ERR_UNSUPPORTED;
    a.tiles = (uint32_t)tiles;
    a.part = kPartCols / kChunkK;
    auto kernel = tile_kernel<kCols, kGated, kF32>;
    static std::atomic<uint64_t> ready{0};          // devices whose kernel may use all shared memory
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ADAFUSE_ERR_DEVICE;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTileSmem) != cudaSuccess)
            return ADAFUSE_ERR_CUDA;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    CUtensorMap xm, wm, um, ym;
    if (!encode_rows(&xm, c.x, a.T, c.K, c.ldx, 128) || !encode_rows(&wm, c.W, a.N, c.K, c.ldw, kCols / 2))
        return ADAFUSE_ERR_UNSUPPORTED;
    if (!kGated) um = wm;
    else if (!encode_rows(&um, c.W_up, a.N, c.K, c.ldw, kCols / 2)) return ADAFUSE_ERR_UNSUPPORTED;
    if (!encode_outputs(&ym, a, box_row<kCols, kGated, kF32>())) return ADAFUSE_ERR_UNSUPPORTED;
    const int64_t n = std::min<int64_t>(tiles, pairs);
    return launch_pdl_cluster(kernel, dim3((unsigned)(2 * n)), dim3(kTileThreads), kTileSmem, 2, c.s, xm, wm, um, ym, a);
}

}  // namespace

namespace {

// Rounds that the device's pairs take for the tiles of so many columns.
int64_t rounds_of(const ProjectCall& c, int cols)
{
    const int pairs = std::max(1, device_sms() / 2), out = c.W_up ? cols / 2 : cols;
    return ((c.a.T + kPairTokens - 1) / kPairTokens * ((c.a.N + out - 1) / out) + pairs - 1) / pairs;
}

// A chunk of a narrow tile takes 0.65 of a wide one's time: narrow tiles where
// the last round of wide ones would leave many pairs idle (512 tokens, 4096 ->
// 4096: 18.0 us narrow, 25.4 wide; 768: 29.4 and 28.1).  The fp32 form keeps 64
// sums per lane beside the epilogue's own values; 128 would not fit.
bool wide_tiles(const ProjectCall& c) { return !c.a.y_f32 && rounds_of(c, 256) <= 0.65 * rounds_of(c, 128); }

}  // namespace

// Measured: a chunk of a round takes 545 cycles wide, 355 narrow, 450 in the
// gated form and 480 with fp32 outputs (which drain an accumulator every eight
// chunks); the rest of a call about 9500.
double project_tile_cost(const ProjectCall& c)
{
    const bool wide = wide_tiles(c);
    const double chunk = wide ? 545 : c.W_up ? 450 : c.a.y_f32 ? 480 : 355;
    return (double)rounds_of(c, wide ? 256 : 128) * c.a.chunks * chunk + (c.a.y_f32 ? 12500 : 9500);
}

int launch_project_tile(ProjectCall& c)
{
    const int pairs = device_sms() / 2;
    const bool gated = c.W_up != nullptr, wide = wide_tiles(c);
    if (gated) return wide ? launch_tiles<256, true, false>(c, pairs) : launch_tiles<128, true, false>(c, pairs);
    if (c.a.y_f32) return launch_tiles<128, false, true>(c, pairs);
    return wide ? launch_tiles<256, false, false>(c, pairs) : launch_tiles<128, false, false>(c, pairs);
}

}  // namespace af
