// Projections with their epilogue:
//   y = act(x W^T + bias) + residual                                (project)
//   y = act(x W_gate^T + bias_gate) * (x W_up^T + bias_up)          (gated)
// for x [T, d_in] and weights [d_out, d_in], everything in fp32 up to the one
// rounding of y.
//
// stream_kernel (decode batches, and long prompts of few outputs; otherwise the
// tiles of project_tile.cu): W streams past a tile of tokens.  A unit is 128
// rows of W (and the same 128 of W_up) against a tile of up to 256 (128)
// tokens, with the W rows as the M side of the tensor-core product and the
// tokens, padded to 16, as its N side, so that a single token costs one pass
// over W.  A unit's d_in is split over the CTAs of a cluster: one warp loads
// the CTA's range of 64-column chunks through a ring of shared memory by TMA,
// two issue tcgen05.mma into TMEM, then the partial sums go to shared memory
// (token by token), each CTA gets the others' sums of its share of the tokens
// by bulk copies, adds them in rank order, applies the epilogue and writes y.
// No workspace, no counters, no atomics.  TMEM is freed before a CTA waits for
// its cluster, so no CTA ever waits for another while it holds TMEM that the
// other needs.
//
// Bound by W's bytes: one token through 4096 -> 11008 gate and up (180 MB) 31
// us, 5.8 TB/s; 64 tokens through 5120 -> 13824 (283 MB) 50-53 us, 5.4-5.7 TB/s.
// A single 4096 x 4096 layer (33.5 MB, 5.1 us) takes 8.4-8.8: the launch, the
// first load's way (1.2 us) and the sum over the cluster (1 us) are not hidden.
//
// The tensor core rounds each step of an accumulator towards zero, which adds
// up over long sums: about 1e-9 d_in of the result (measured against 64 bits:
// 4.4e-6 at d_in = 4096, 1.6e-5 at 13824, 1.2e-4 at 131072, where all products
// have one sign).  bf16 outputs, off by 2^-9 to 2^-8 from their one rounding,
// keep one accumulator per multiplying warp, and d_in is limited to kMaxSum for
// them, where the sums' error is a sixteenth of that; fp32 outputs accumulate
// parts of at most 512 columns in accumulators of their own, added up in
// registers, for any d_in.
#include <algorithm>
#include <atomic>
#include <cstring>

#include "act.cuh"
#include "ops.h"
#include "project.h"
#include "ptx_ops.cuh"

namespace af {

bool encode_rows(CUtensorMap* m, const void* p, int64_t rows, int32_t cols, int64_t ld, int box_rows)
{
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? ld : cols) * 2};
    cuuint32_t box[2] = {kChunkK, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box,
                                estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int kStreamThreads = 256;                     // one warp loads, two multiply; all finish
constexpr int kMaxRing = 12;                            // stages of at least 18 KB
constexpr int kMaxSplits = 8;
constexpr int32_t kMaxSum = 131072;                     // most columns of a bf16 output's sum
constexpr uint32_t kWTile = kTileM * kChunkK * 2;       // 16 KB

struct StreamArgs : ProjectArgs {
    int32_t tile;           // tokens per unit: a multiple of 16
    int32_t n_tt;           // token tiles
    int32_t splits, ring, parts;
    uint32_t tmem_cols, stage_bytes;
};

__device__ __forceinline__ void add_bf16x4(float (&v)[4], uint2 w)
{
    v[0] += bf16lo(w.x); v[1] += bf16hi(w.x); v[2] += bf16lo(w.y); v[3] += bf16hi(w.y);
}

// bias, activation, product and residual of 4 consecutive outputs, and their store
template <bool kGated>
__device__ __forceinline__ void finish4(const StreamArgs& a, float (&v)[4], float (&u)[4], uint2 bias, uint2 bias_up,
                                        uint2 residual, int64_t t, int o)
{
    if (a.bias) add_bf16x4(v, bias);
    activate_all(v, a.act);
    if constexpr (kGated) {
        if (a.bias_up) add_bf16x4(u, bias_up);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= u[i];
    } else {
        if (a.residual) add_bf16x4(v, residual);
    }
    if (!kGated && a.y_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.y) + t * a.ldy + o) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + t * a.ldy + o) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// v += 4 floats in shared memory
__device__ __forceinline__ void add4(float (&v)[4], uint32_t at)
{
    const uint4 x = ld_shared_v4(at);
    v[0] += __uint_as_float(x.x); v[1] += __uint_as_float(x.y);
    v[2] += __uint_as_float(x.z); v[3] += __uint_as_float(x.w);
}

// v = the sum, in rank order, of the 4 floats at `mine` (this CTA's) and those
// of the cluster's other CTAs, `step` bytes apart from `theirs` on.
__device__ __forceinline__ void sum_ranks(float (&v)[4], uint32_t mine, uint32_t theirs, uint32_t step, int rank, int splits)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxSplits; ++r) {
        if (r >= splits) break;
        add4(v, r == rank ? mine : theirs + (uint32_t)(r < rank ? r : r - 1) * step);
    }
}

template <bool kGated>
__global__ void __launch_bounds__(kStreamThreads, 2) stream_kernel(const __grid_constant__ CUtensorMap xmap,
                                                                const __grid_constant__ CUtensorMap wmap,
                                                                const __grid_constant__ CUtensorMap umap,
                                                                const StreamArgs a)
{
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t full[kMaxRing], empty[kMaxRing], done, joined;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = a.splits > 1 ? (int)cluster_rank() : 0;
    const int unit = (int)blockIdx.x / a.splits;
    const int row0 = unit / a.n_tt * kTileM;
    const int64_t t0 = (int64_t)(unit % a.n_tt) * a.tile;
    const int ntok = (int)min((int64_t)a.tile, a.T - t0);
    const int c0 = (int)((int64_t)a.chunks * rank / a.splits);
    const int n = (int)((int64_t)a.chunks * (rank + 1) / a.splits) - c0;

    if (warp == 0 && elect_one()) {
        prefetch_map(&wmap);
        prefetch_map(&xmap);
        if constexpr (kGated) prefetch_map(&umap);
        for (int i = 0; i < min(n, a.ring); ++i) {
            tma_prefetch_2d(&wmap, (c0 + i) * kChunkK, row0);
            if constexpr (kGated) tma_prefetch_2d(&umap, (c0 + i) * kChunkK, row0);
        }
    }
    if (threadIdx.x == 32) {
        abort_flag = 0;
        for (int i = 0; i < a.ring; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kGated ? 2 : 1);
        }
        mbar_init(&done, 2);
        mbar_init(&joined, 1);
        fence_mbar_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 1) {
        tmem_alloc(&tmem_slot, a.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == 0) {
        // The whole warp walks the loop, one elected lane issues the copies.
        int s = 0, issued = 0;
        uint32_t lap = 1;               // parity that the stage's `empty` completes with when free (the first lap: at once)
        for (int i = 0; i < n; ++i) {
            if (!mbar_wait_warp(&empty[s], lap, &abort_flag)) break;
            if (!(a.stall && blockIdx.x == 0 && i == 0) && elect_one()) {       // test hook: the first never arrives
                uint8_t* p = ring + (size_t)s * a.stage_bytes;
                const int k = (c0 + i) * kChunkK;
                mbar_arrive_expect_tx(&full[s], a.stage_bytes);
                tma_load_2d(p, &wmap, &full[s], k, row0);
                if constexpr (kGated) tma_load_2d(p + kWTile, &umap, &full[s], k, row0);
                tma_load_2d(p + (kGated ? 2 : 1) * kWTile, &xmap, &full[s], k, (int)t0);
            }
            __syncwarp();
            issued = i + 1;
            if (++s == a.ring) { s = 0; lap ^= 1; }
        }
        // a wait gave up: what is in flight has to land before shared memory is given back
        if (__any_sync(0xffffffffu, *(volatile int*)&abort_flag))
            for (int i = max(0, issued - a.ring); i < issued; ++i)
                if (!(a.stall && blockIdx.x == 0 && i == 0))
                    mbar_wait_landed(&full[i % a.ring], (uint32_t)(i / a.ring) & 1);
        __syncwarp();
    } else if (warp <= 2) {
        // Two warps multiply, into accumulators of their own (added up below;
        // for the gated form one has W_gate, the other W_up): the waits, the
        // four products and the commit of a chunk take one warp 540 cycles,
        // 34 bytes of W a cycle, where an SM's share of the memory can be more.
        // A plain unit's warps take the chunks in turn, so its ring has an even
        // number of stages: each stage then belongs to one warp, which sees
        // every phase of its barrier.  (A warp that came back to a stage two
        // laps later would take the phase before last for the last one.)
        const int me = warp - 1;
        const uint32_t idesc = make_idesc_bf16(kTileM, (uint32_t)a.tile, 0u, 0u);
        const uint64_t desc = make_sdesc(smem_u32(ring), 16u, 1024u, kLayoutSw128);
        const uint32_t woff = kGated ? (uint32_t)me * (kWTile >> 4) : 0u, xoff = ((kGated ? 2 : 1) * kWTile) >> 4;
        const int mine = kGated ? n : (n + 1 - me) / 2;         // chunks: all, or every other
        int s = kGated ? 0 : me, part = 0, until = 0;           // the part that chunk i belongs to ends before chunk `until`
        uint32_t lap = 0;
        for (int i = 0; i < mine; ++i) {
            if (!mbar_wait_warp(&full[s], lap, &abort_flag)) break;
            const bool fresh = i == until;
            if (fresh) {
                if (i) ++part;
                until = (int)((int64_t)mine * (part + 1) / a.parts);
            }
            if (elect_one()) {
                const uint64_t at = desc + (uint64_t)(s * (int)(a.stage_bytes >> 4));
                const uint64_t w = at + woff, x = at + xoff;
                const uint32_t d = tmem + (uint32_t)((me * a.parts + part) * a.tile);
#pragma unroll
                for (int kk = 0; kk < kChunkK / 16; ++kk)
                    tc_mma_bf16(d, w + kk * 2, x + kk * 2, idesc, fresh && kk == 0 ? 0u : 1u);
                tc_commit(&empty[s]);
            }
            __syncwarp();
            s += kGated ? 1 : 2;
            if (s >= a.ring) { s -= a.ring; lap ^= 1; }
        }
        if (elect_one()) tc_commit(&done);          // at once where nothing was issued
        if (__any_sync(0xffffffffu, *(volatile int*)&abort_flag)) mbar_wait_landed(&done, 0);
        __syncwarp();
    }

    // The partial sums, [token][128 rows] fp32, over the ring: every load has
    // been consumed once the last product is done.  A warp takes its quarter of
    // the accumulator's lanes and every other 16 tokens.
    float* part = reinterpret_cast<float*>(ring);
    const bool ok = mbar_wait_hot(&done, 0, &abort_flag) && !*(volatile int*)&abort_flag;
    if (__all_sync(0xffffffffu, ok)) {
        tc_fence_after();
        const int q = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
#pragma unroll
        for (int m = 0; m < (kGated ? 2 : 1); ++m) {
            const int sums = kGated ? 1 : n > 1 ? 2 * a.parts : 1;
            float* p = part + m * a.tile * kTileM + q * 32 + lane;
            for (int t = (warp >> 2) * 16; t < ntok; t += 32) {
                uint32_t v[16];
                float sum[16];
                tc_ld_x16(lanes + (uint32_t)(m * a.tile + t), v);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[i] = __uint_as_float(v[i]);
                for (int j = 1; j < sums; ++j) {
                    tc_ld_x16(lanes + (uint32_t)(j * a.tile + t), v);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[i] += __uint_as_float(v[i]);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) p[(t + i) * kTileM] = sum[i];
            }
        }
        tc_fence_before();
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, a.tmem_cols);
    }

    // Each CTA of the cluster finishes its share of the tokens: the others copy
    // their partial sums of them behind its own, one bulk copy each (remote
    // loads by its threads brought 12 bytes a cycle).
    constexpr int kParts = kGated ? 2 : 1;
    const int own = (a.tile + a.splits - 1) / a.splits;
    const uint32_t sums = smem_u32(part), theirs = sums + (uint32_t)(kParts * a.tile * kTileM) * 4u;
    const uint32_t step = (uint32_t)(kParts * own * kTileM) * 4u;        // of one other CTA's sums
    const auto tokens_of = [&](int r) { return max(0, min(own, ntok - r * own)); };
    const int here = tokens_of(rank);
    bool ours = true;
    // A warp takes a token's 128 outputs, four per lane, and every eighth of its
    // CTA's tokens.  What the epilogue reads from memory is under way while the
    // sums come together, then four tokens ahead.
    constexpr int kWarps = kStreamThreads / 32, kAhead = 4;
    const int o = row0 + lane * 4;
    const auto read4 = [](const uint16_t* p, int64_t at) { return *reinterpret_cast<const uint2*>(p + at); };
    uint2 bias = {}, bias_up = {}, residual[kAhead] = {};
    const auto read_residuals = [&](int i) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (!kGated && a.residual && o < a.N && i + j * kWarps < here)
                residual[j] = read4(a.residual, (t0 + rank * own + i + j * kWarps) * a.ldr + o);
    };
    if (o < a.N) {
        if (a.bias) bias = read4(a.bias, o);
        if (kGated && a.bias_up) bias_up = read4(a.bias_up, o);
    }
    read_residuals(warp);
    if (a.splits > 1) {
        if (threadIdx.x == 0 && here)
            mbar_arrive_expect_tx(&joined, (uint32_t)((a.splits - 1) * kParts * here * kTileM) * 4u);
        cluster_sync();             // every ring is free, every partial sum written
        if (warp == 0 && elect_one())
            for (int r = 0; r < a.splits; ++r) {
                const int count = tokens_of(r);
                if (r == rank || !count) continue;
                const uint32_t to = cluster_map(theirs + (uint32_t)(rank < r ? rank : rank - 1) * step, (uint32_t)r);
                for (int m = 0; m < kParts; ++m)
                    bulk_copy_cluster(to + (uint32_t)(m * own * kTileM) * 4u,
                                      sums + (uint32_t)((m * a.tile + r * own) * kTileM) * 4u,
                                      (uint32_t)(count * kTileM) * 4u, cluster_map(smem_u32(&joined), (uint32_t)r));
            }
        __syncwarp();
        // also after an abort: the copies have to land before the CTA may leave
        ours = !here || mbar_wait_hot(&joined, 0, &abort_flag) || mbar_wait_landed(&joined, 0);
        cluster_arrive();           // what came here has left the others
    }
    const bool fine = ours && !*(volatile int*)&abort_flag;
    if (fine && o < a.N)
        for (int i0 = warp; i0 < here; i0 += kAhead * kWarps) {
            if (i0 != warp) read_residuals(i0);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = i0 + j * kWarps;
                if (i >= here) break;
                float v[4], u[4];
                const uint32_t at = (uint32_t)(i * kTileM + lane * 4) * 4u;
                const uint32_t mine = sums + (uint32_t)(rank * own * kTileM) * 4u + at;
                sum_ranks(v, mine, theirs + at, step, rank, a.splits);
                if constexpr (kGated)
                    sum_ranks(u, mine + (uint32_t)(a.tile * kTileM) * 4u,
                              theirs + (uint32_t)(own * kTileM) * 4u + at, step, rank, a.splits);
                finish4<kGated>(a, v, u, bias, bias_up, residual[j], t0 + rank * own + i, o);
            }
        }
    if (threadIdx.x == 0 && !fine && a.status) atomicOr(a.status, ADAFUSE_STATUS_TIMEOUT);
    if (a.splits > 1) cluster_wait();       // the others' copies of this CTA's sums are done
}

// ------------------------------------------------------------------ host side

// Shared memory per CTA of the two ways to run the stream kernel: two CTAs on
// an SM, or one.
constexpr uint32_t kSmemHalf = 111 * 1024, kSmemFull = 225 * 1024;

// Clusters of `splits` CTAs, one CTA per SM, that the device runs at a time,
// asked once.  (For CTAs of half an SM the runtime gives the same number, but
// two do share an SM: 157 of them, 20000 outputs, end in one round.)
template <bool kGated>
int clusters_at_once(int dev, int splits)
{
    static std::atomic<int> known[16][kMaxSplits + 1];
    std::atomic<int>* slot = dev < 16 ? &known[dev][splits] : nullptr;
    int v = slot ? slot->load(std::memory_order_relaxed) : 0;
    if (v > 0) return v;
    auto kernel = stream_kernel<kGated>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemFull) != cudaSuccess)
        return 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)splits);
    cfg.blockDim = dim3(kStreamThreads);
    cfg.dynamicSmemBytes = kSmemFull;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&v, kernel, &cfg) != cudaSuccess || v < 1) return 0;
    if (slot) slot->store(v, std::memory_order_relaxed);
    return v;
}

// How a call runs on the stream kernel.
struct StreamForm {
    int tile = 0, n_tt = 0, splits = 0, ring = 0;
    int parts = 1;              // accumulators of each multiplying warp (plain)
    bool half = false;
    double cost = 0;            // estimated cycles
};

// The cheapest form, if there is one: tiles of up to 128 tokens (gated 64) or
// twice that (fp32: from 32 on, as more parts need more accumulators); one
// CTA per SM with a deep ring, or two (where a ring and the partial sums fit
// half of shared memory); and the split of d_in.  Measured: a chunk takes a CTA
// 365 cycles (gated 500), more for tall tiles; memory gives W's bytes at 3400 a
// cycle where two thirds of the SMs' places are taken, less below; the sum over
// the splits, and each further round of clusters, cost their part.  (4096 ->
// 11008, one token: 17.6 us as two CTAs per SM in three splits, 19.6 as one
// without; 64 tokens: 20.8 and 22.7; 5120 -> 13824, 32 tokens: 28.7 and 27.4.
// 256 tokens, 4096 -> 4096: 16.2 us as two tiles, 19.2 as one; 4096 -> 11008:
// 48 and 43.)
template <bool kGated>
StreamForm stream_form(const ProjectCall& c, int dev)
{
    StreamForm best;
    const ProjectArgs& a = c.a;
    const double places = device_sms();
    constexpr int kMats = kGated ? 2 : 1;
    int64_t last = 0;
    for (int most = a.y_f32 ? 32 : 128 / kMats; most <= 256 / kMats; most *= 2) {
        StreamForm f;
        f.n_tt = (int)((a.T + most - 1) / most);
        if (f.n_tt == last) continue;
        last = f.n_tt;
        f.tile = (int)(((a.T + f.n_tt - 1) / f.n_tt + 15) / 16 * 16);       // of equal height
        f.n_tt = (int)((a.T + f.tile - 1) / f.tile);
        const uint32_t stage = kMats * kWTile + (uint32_t)f.tile * kChunkK * 2;
        const int64_t blocks = (int64_t)((a.N + kTileM - 1) / kTileM) * f.n_tt;
        const double tall = f.tile * kMats;
        const double chunk = kGated ? std::max(500., 4 * tall) : std::max(365., 2.9 * tall);
        const double memory = 2. * ((double)kMats * a.N * c.K + (double)a.T * (c.K + a.N)) / 3400;
        for (int two = 0; two < 2; ++two)
            for (int S = 1; S <= kMaxSplits && S <= a.chunks; ++S) {
                // its own and the others' partial sums lie over the ring in the end
                const uint32_t room = (two ? kSmemHalf : kSmemFull) - 1024;
                const uint32_t sums = (uint32_t)(f.tile + (f.tile + S - 1) / S * (S - 1)) * kTileM * 4 * kMats;
                f.ring = (int)std::min<uint32_t>(kMaxRing, room / stage);
                if (!kGated) f.ring &= ~1;              // even, see the multiplying warps
                if (sums > room || f.ring < (kGated ? 3 : 4)) continue;
                if (a.y_f32) {                          // as many accumulators as its parts need
                    f.parts = ((a.chunks + S - 1) / S + 1) / 2;
                    f.parts = (f.parts * kChunkK + kPartCols - 1) / kPartCols;
                    if (f.parts * 2 * f.tile > (two ? 256 : 512)) continue;
                }
                const int at_once = clusters_at_once<kGated>(dev, S) * (1 + two);
                if (!at_once || blocks * S > 0x7fffffff) continue;
                const int64_t rounds = (blocks + at_once - 1) / at_once;
                const double taken = (double)blocks * S / (rounds * places * (1 + two));
                const double work = (double)rounds * ((a.chunks + S - 1) / S) * chunk * (two ? 1.6 : 1.);
                const double stream = memory / std::min(1., taken / 0.67);
                f.cost = std::max(work, stream) + std::min(work, stream) / 8 + (300 + 3 * tall) * S +
                         (double)rounds * (6500 + 45 * tall) + two * 2500;
                f.splits = S;
                f.half = two;
                if (!best.splits || f.cost < best.cost) best = f;
            }
    }
    return best;
}

template <bool kGated>
int launch_stream(ProjectCall& c, const StreamForm& f)
{
    StreamArgs a{c.a};
    a.tile = f.tile;
    a.n_tt = f.n_tt;
    a.splits = f.splits;
    a.ring = f.ring;
    a.stage_bytes = (kGated ? 2 : 1) * kWTile + (uint32_t)a.tile * kChunkK * 2;
    const int64_t blocks = (int64_t)((a.N + kTileM - 1) / kTileM) * a.n_tt;
    a.parts = std::max(1, std::min(f.parts, a.chunks / a.splits / 2));         // a part has a chunk at least
    a.tmem_cols = 32;
    while ((int)a.tmem_cols < a.tile * a.parts * 2) a.tmem_cols *= 2;

    CUtensorMap xm, wm, um;
    if (!encode_rows(&xm, c.x, a.T, c.K, c.ldx, a.tile) || !encode_rows(&wm, c.W, a.N, c.K, c.ldw, kTileM))
        return ADAFUSE_ERR_UNSUPPORTED;
    if (!kGated) um = wm;
    else if (!encode_rows(&um, c.W_up, a.N, c.K, c.ldw, kTileM)) return ADAFUSE_ERR_UNSUPPORTED;
    return launch_pdl_cluster(stream_kernel<kGated>, dim3((unsigned)(blocks * a.splits)), dim3(kStreamThreads),
                              f.half ? kSmemHalf : kSmemFull, a.splits, c.s, xm, wm, um, a);
}

// W streams past the tokens, or tiles of tokens and outputs on CTA pairs, by the
// lower estimate (256 tokens, 4096 -> 4096: 16.2 us streamed, 17.8 in tiles;
// 384: 21.5 and 18.0; 256, 4096 -> 11008: 40.7 and 28.3; 2869, 6888 -> 144: 29
// and 37, as only the stream splits d_in).
template <bool kGated>
int launch_project(ProjectCall& c)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ADAFUSE_ERR_DEVICE;
    const StreamForm f = stream_form<kGated>(c, dev);
    if (!f.splits || f.cost > project_tile_cost(c)) return launch_project_tile(c);
    return launch_stream<kGated>(c, f);
}

int check(ProjectCall& c, const void* bias, const void* bias_up, bool gated, uint32_t flags)
{
    ProjectArgs& a = c.a;
    const uint32_t act = flags & ADAFUSE_ACT_MASK;
    if (flags & ~(ADAFUSE_ACT_MASK | ADAFUSE_TEST_STALL | (gated ? 0u : ADAFUSE_OUT_F32))) return ADAFUSE_ERR_INVALID_ARG;
    if (a.T < 0 || c.K < 1 || a.N < 1) return ADAFUSE_ERR_INVALID_ARG;
    if (act > ADAFUSE_ACT_GELU_TANH || c.K % 8 || a.N % 8 || a.T > 0x7fffff00 || a.N > 0x7fffff00 ||
        c.K > (flags & ADAFUSE_OUT_F32 ? 0x7fffff00 : kMaxSum)) return ADAFUSE_ERR_UNSUPPORTED;
    if (a.T == 0) return ADAFUSE_OK;
    if (!c.x || !c.W || !a.y || (gated && !c.W_up)) return ADAFUSE_ERR_INVALID_ARG;
    a.y_f32 = flags & ADAFUSE_OUT_F32 ? 1 : 0;
    const int64_t size = a.y_f32 ? 4 : 2;
    if (a.T == 1) { c.ldx = c.K; a.ldy = a.ldr = a.N; }
    if (a.N == 1) c.ldw = c.K;
    if (!a.residual) a.ldr = 0;
    if (c.ldx < c.K || c.ldw < c.K || a.ldy < a.N || (a.ldr != 0 && a.ldr < a.N)) return ADAFUSE_ERR_INVALID_ARG;
    for (const void* p : {c.x, c.W, c.W_up, (const void*)a.y, (const void*)a.residual, bias, bias_up})
        if (!aligned_to(p, 16)) return ADAFUSE_ERR_UNSUPPORTED;
    if (c.ldx % 8 || c.ldw % 8 || a.ldr % 8 || a.ldy % (a.y_f32 ? 4 : 8)) return ADAFUSE_ERR_UNSUPPORTED;
    for (const int64_t ld : {c.ldx, c.ldw, a.ldr, a.ldy})
        if (!plain_stride(ld)) return ADAFUSE_ERR_UNSUPPORTED;
    const RowSpan y{a.y, a.T, a.N * size, a.ldy * size};
    const RowSpan in[] = {{c.x, a.T, 2ll * c.K, 2 * c.ldx}, {c.W, a.N, 2ll * c.K, 2 * c.ldw},
                          {c.W_up, a.N, 2ll * c.K, 2 * c.ldw}, {bias, 1, 2ll * a.N, 2ll * a.N},
                          {bias_up, 1, 2ll * a.N, 2ll * a.N}, {a.residual, a.T, 2ll * a.N, 2 * a.ldr}};
    for (const RowSpan& r : in) {
        const bool in_place = &r == &in[5] && r.base == a.y && !a.y_f32 && a.ldr == a.ldy;
        if (r.base && !in_place && rows_overlap(y, r)) return ADAFUSE_ERR_INVALID_ARG;
    }
    a.bias = static_cast<const uint16_t*>(bias);
    a.bias_up = static_cast<const uint16_t*>(bias_up);
    a.act = act;
    a.chunks = (c.K + kChunkK - 1) / kChunkK;
    a.stall = flags & ADAFUSE_TEST_STALL ? 1 : 0;
    if (!device_sms()) return ADAFUSE_ERR_DEVICE;
    if (!tensor_map_encoder()) return ADAFUSE_ERR_CUDA;
    return ADAFUSE_OK;
}

}  // namespace
}  // namespace af

using namespace af;

extern "C" int adafuse_project(const void* x, int64_t T, int32_t d_in, int64_t x_row_stride, const void* W,
                               int32_t d_out, int64_t w_row_stride, const void* bias, const void* residual,
                               int64_t r_row_stride, void* y, int64_t y_row_stride, uint32_t flags, int32_t* status,
                               adafuse_stream_t stream)
{
    ProjectCall c{x, W, nullptr, x_row_stride, w_row_stride, d_in, {}, (cudaStream_t)stream};
    c.a.y = y;
    c.a.residual = static_cast<const uint16_t*>(residual);
    c.a.ldy = y_row_stride;
    c.a.ldr = r_row_stride;
    c.a.T = T;
    c.a.N = d_out;
    c.a.status = status;
    const int rc = check(c, bias, nullptr, false, flags);
    if (rc || T == 0) return rc;
    return launch_project<false>(c);
}

extern "C" int adafuse_gated_project(const void* x, int64_t T, int32_t d_in, int64_t x_row_stride,
                                     const void* W_gate, const void* W_up, int32_t d_out, int64_t w_row_stride,
                                     const void* bias_gate, const void* bias_up, void* y, int64_t y_row_stride,
                                     uint32_t flags, int32_t* status, adafuse_stream_t stream)
{
    ProjectCall c{x, W_gate, W_up, x_row_stride, w_row_stride, d_in, {}, (cudaStream_t)stream};
    c.a.y = y;
    c.a.ldy = y_row_stride;
    c.a.T = T;
    c.a.N = d_out;
    c.a.status = status;
    const int rc = check(c, bias_gate, bias_up, true, flags);
    if (rc || T == 0) return rc;
    return launch_project<true>(c);
}
