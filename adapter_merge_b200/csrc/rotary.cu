// Rotation of queries and keys by their positions, after an optional RMS norm
// of each head, in one pass over the heads.
//
// Angles.  Pair i of the token at position p turns by p * freq[i] radians.
// For far positions that product loses its fraction in fp32 (at p = 2^20 an
// fp32 angle is off by up to 1/32 rad), so the frequency is taken as a
// fraction of a turn with 64 bits after the point, F = freq / (2 pi) * 2^64,
// and p * F modulo 2^64 is the exact fraction of the last turn, for positions
// of either sign: one 64-bit integer product instead of a range reduction.
// The fraction goes to sincospif.
//
// HBM-bound for long prompts (each element read and written once), latency
// for a decode batch.  A CTA takes a few tokens, computes their sines and
// cosines once into shared memory (rot/2 per token, shared by all heads), then
// its lanes rotate the heads: an item is a vector of V elements together with
// the vector of its partners (one vector that holds both in the interleaved
// layout, one unrotated vector past `rot`), and 2^n lanes share a head, one
// item each, so that the norm's sum is a shuffle among them.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace af {
namespace {

constexpr int kRotThreads = 256;
constexpr int kMaxHeadDim = 1024;

struct Heads {
    const uint16_t* in;
    uint16_t* out;
    const uint16_t* weight;
    int64_t its, ihs, ots, ohs;
};

struct RotArgs {
    Heads q, k;
    const void* pos;
    const double* freq;
    int64_t T;
    int32_t Hq, H;          // query heads, all heads
    int32_t D, rot, half;
    int32_t lanes;          // lanes per head: a power of two
    int32_t items;          // items per head
    int32_t tokens;         // tokens per CTA
    int32_t pairs, pos32;
    float factor, eps, inv_d;
};

template <int V>
struct Vec {
    float v[V];
    __device__ __forceinline__ void load(const uint16_t* p)
    {
        if constexpr (V == 8) {
            const uint4 a = *reinterpret_cast<const uint4*>(p);
            v[0] = bf16lo(a.x); v[1] = bf16hi(a.x); v[2] = bf16lo(a.y); v[3] = bf16hi(a.y);
            v[4] = bf16lo(a.z); v[5] = bf16hi(a.z); v[6] = bf16lo(a.w); v[7] = bf16hi(a.w);
        } else if constexpr (V == 4) {
            const uint2 a = *reinterpret_cast<const uint2*>(p);
            v[0] = bf16lo(a.x); v[1] = bf16hi(a.x); v[2] = bf16lo(a.y); v[3] = bf16hi(a.y);
        } else {
            v[0] = __uint_as_float((uint32_t)*p << 16);
        }
    }
    __device__ __forceinline__ void store(uint16_t* p) const
    {
        if constexpr (V == 8)
            *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        else if constexpr (V == 4)
            *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        else
            *p = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    }
    __device__ __forceinline__ float squares() const
    {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s += v[i] * v[i];
        return s;
    }
};

// Item j of a head: its first vector's offset, its second's (-1: none), and
// the first of its pairs (-1: not rotated).
template <int V>
struct Item {
    int o1, o2, pair;
    __device__ __forceinline__ Item(const RotArgs& a, int j)
    {
        const bool split = !a.pairs || V == 1;          // partners in two vectors
        const int rotated = (split ? a.half : a.rot) / V;
        if (j >= rotated) {
            o1 = a.rot + (j - rotated) * V;
            o2 = pair = -1;
        } else if (!split) {
            o1 = j * V;
            o2 = -1;
            pair = j * (V / 2);
        } else {
            o1 = a.pairs ? 2 * j : j * V;
            o2 = a.pairs ? 2 * j + 1 : a.half + j * V;
            pair = j * V;
        }
    }
};

template <int V>
__device__ __forceinline__ void scale(Vec<V>& x, const uint16_t* w, float r)
{
    Vec<V> g;
    g.load(w);
#pragma unroll
    for (int i = 0; i < V; ++i) x.v[i] = x.v[i] * r * g.v[i];
}

template <int V>
__device__ __forceinline__ void rotate_item(const RotArgs& a, const Item<V>& it, const float2* cs, Vec<V>& x, Vec<V>& y)
{
    if (it.pair < 0) return;
    if (it.o2 >= 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 c = cs[it.pair + i];
            const float p = x.v[i], q = y.v[i];
            x.v[i] = p * c.x - q * c.y;
            y.v[i] = p * c.y + q * c.x;
        }
    } else if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 c = cs[it.pair + i];
            const float p = x.v[2 * i], q = x.v[2 * i + 1];
            x.v[2 * i] = p * c.x - q * c.y;
            x.v[2 * i + 1] = p * c.y + q * c.x;
        }
    }
}

// kOne: a head has no more items than lanes, so its values stay in registers
// between the norm's sum and the rotation; otherwise they are read again.
template <int V, bool kOne>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotArgs a)
{
    extern __shared__ float2 cs[];          // [tokens][half]: cosine, sine, times the factor
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int tokens = (int)min((int64_t)a.tokens, a.T - t0);
    for (int i = threadIdx.x; i < tokens * a.half; i += kRotThreads) {
        const int tl = i / a.half, f = i - tl * a.half;
        const int64_t p = a.pos32 ? (int64_t)static_cast<const int32_t*>(a.pos)[t0 + tl]
                                  : static_cast<const int64_t*>(a.pos)[t0 + tl];
        double turn = a.freq[f] * 0.15915494309189533577;       // 1 / (2 pi)
        turn -= floor(turn);
        const uint64_t frac = __double2ull_rn(turn * 18446744073709551616.0);     // 2^64 itself wraps to 0 below
        const int64_t at = (int64_t)((uint64_t)p * (turn < 1.0 ? frac : 0ull));
        float s, c;
        sincospif((float)at * 1.08420217248550443401e-19f, &s, &c);               // 2^-63 half turns
        cs[i] = make_float2(c * a.factor, s * a.factor);
    }
    __syncthreads();

    const int lane = threadIdx.x & (a.lanes - 1);
    const int per = kRotThreads / a.lanes;          // heads at a time
    const int tasks = tokens * a.H;
    // Every lane of a warp takes the same number of steps (the shuffles need
    // all of them); a step past the end does nothing.
    for (int first = 0; first < tasks; first += per) {
        const int task = first + (int)(threadIdx.x / a.lanes);
        const bool live = task < tasks;
        const int tl = live ? task / a.H : 0;
        const int h = live ? task - tl * a.H : 0;
        const bool is_q = h < a.Hq;
        const Heads& m = is_q ? a.q : a.k;
        const int hh = is_q ? h : h - a.Hq;
        const uint16_t* in = m.in + (t0 + tl) * m.its + hh * m.ihs;
        uint16_t* out = m.out + (t0 + tl) * m.ots + hh * m.ohs;
        const float2* c = cs + tl * a.half;
        Vec<V> x, y;
        if constexpr (kOne) {
            const Item<V> it(a, lane);
            const bool mine = live && lane < a.items;
            if (mine) {
                x.load(in + it.o1);
                if (it.o2 >= 0) y.load(in + it.o2);
            }
            if (a.q.weight || a.k.weight) {
                float sum = mine ? x.squares() + (it.o2 >= 0 ? y.squares() : 0.f) : 0.f;
                for (int d = a.lanes / 2; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (mine && m.weight) {
                    const float r = rsqrtf(sum * a.inv_d + a.eps);
                    scale<V>(x, m.weight + it.o1, r);
                    if (it.o2 >= 0) scale<V>(y, m.weight + it.o2, r);
                }
            }
            if (mine) {
                rotate_item<V>(a, it, c, x, y);
                x.store(out + it.o1);
                if (it.o2 >= 0) y.store(out + it.o2);
            }
        } else {
            float r = 1.f;
            if (a.q.weight || a.k.weight) {
                float sum = 0.f;
                for (int j = lane; live && j < a.items; j += a.lanes) {
                    const Item<V> it(a, j);
                    x.load(in + it.o1);
                    sum += x.squares();
                    if (it.o2 >= 0) {
                        y.load(in + it.o2);
                        sum += y.squares();
                    }
                }
                for (int d = a.lanes / 2; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                r = rsqrtf(sum * a.inv_d + a.eps);
            }
            for (int j = lane; live && j < a.items; j += a.lanes) {
                const Item<V> it(a, j);
                x.load(in + it.o1);
                if (it.o2 >= 0) y.load(in + it.o2);
                if (m.weight) {
                    scale<V>(x, m.weight + it.o1, r);
                    if (it.o2 >= 0) scale<V>(y, m.weight + it.o2, r);
                }
                rotate_item<V>(a, it, c, x, y);
                x.store(out + it.o1);
                if (it.o2 >= 0) y.store(out + it.o2);
            }
        }
    }
}

// Whether vectors of V elements fit the heads' layout.
bool vectors_fit(const adafuse_heads* m, int V, int T)
{
    if (!m) return true;
    const int64_t mask = V - 1;
    if (T > 1 && ((m->in_token_stride | m->out_token_stride) & mask)) return false;
    if (m->heads > 1 && ((m->in_head_stride | m->out_head_stride) & mask)) return false;
    return aligned_to(m->in, 2 * V) && aligned_to(m->out, 2 * V) && aligned_to(m->weight, 2 * V);
}

int64_t span(int64_t T, int64_t ts, int32_t heads, int64_t hs, int32_t D)
{
    return (T - 1) * ts + (int64_t)(heads - 1) * hs + D;
}

// Whether two sets of heads can share an element.  Sets whose address ranges
// cross are told apart where they have the same token stride and each token's
// heads lie within it (columns of one buffer).
bool heads_overlap(const void* p, int64_t pts, int64_t phs, int32_t ph, const void* q, int64_t qts, int64_t qhs,
                   int32_t qh, int64_t T, int32_t D)
{
    return rows_overlap(RowSpan{p, T, 2 * span(1, 0, ph, phs, D), 2 * pts},
                        RowSpan{q, T, 2 * span(1, 0, qh, qhs, D), 2 * qts});
}

int check_heads(const adafuse_heads* m, int64_t T, int32_t D)
{
    if (!m->in || !m->out || m->heads < 1) return ADAFUSE_ERR_INVALID_ARG;
    if (m->heads > 65536) return ADAFUSE_ERR_UNSUPPORTED;
    if (!aligned_to(m->in, 2) || !aligned_to(m->out, 2) || !aligned_to(m->weight, 2)) return ADAFUSE_ERR_INVALID_ARG;
    if (m->in_token_stride < 0 || m->in_head_stride < 0 || m->out_token_stride < 0 || m->out_head_stride < 0)
        return ADAFUSE_ERR_INVALID_ARG;
    // the outputs of two heads or tokens may not meet: either axis may be the outer one
    const int64_t ts = m->out_token_stride, hs = m->out_head_stride;
    const bool token_outer = (m->heads == 1 || hs >= D) && (T == 1 || ts >= span(1, 0, m->heads, hs, D));
    const bool head_outer = (T == 1 || ts >= D) && (m->heads == 1 || hs >= (T - 1) * ts + D);
    if (!token_outer && !head_outer) return ADAFUSE_ERR_INVALID_ARG;
    return ADAFUSE_OK;
}

}  // namespace
}  // namespace af

using namespace af;

extern "C" int adafuse_rotary(const adafuse_heads* q, const adafuse_heads* k, int64_t T, int32_t head_dim,
                              int32_t rot, const void* positions, const double* freq, float factor, float eps,
                              uint32_t flags, adafuse_stream_t stream)
{
    if (flags & ~(ADAFUSE_PAIRS | ADAFUSE_POS_I32)) return ADAFUSE_ERR_INVALID_ARG;
    if (!q || T < 0 || head_dim < 1 || rot < 0) return ADAFUSE_ERR_INVALID_ARG;
    if (rot % 2 || rot > head_dim || head_dim > kMaxHeadDim) return ADAFUSE_ERR_UNSUPPORTED;
    if (T == 0) return ADAFUSE_OK;
    int rc = check_heads(q, T, head_dim);
    if (!rc && k) rc = check_heads(k, T, head_dim);
    if (rc) return rc;
    const uintptr_t ps = flags & ADAFUSE_POS_I32 ? 4 : 8;
    if (rot && (!positions || !freq || !aligned_to(positions, ps) || !aligned_to(freq, 8)))
        return ADAFUSE_ERR_INVALID_ARG;
    const adafuse_heads* all[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        const adafuse_heads* o = all[i];
        if (!o) continue;
        const RowSpan mine{o->out, T, 2 * span(1, 0, o->heads, o->out_head_stride, head_dim), 2 * o->out_token_stride};
        for (int j = 0; j < 2; ++j) {
            const adafuse_heads* m = all[j];
            if (!m) continue;
            const bool same = i == j && m->in == o->out && m->in_token_stride == o->out_token_stride &&
                              m->in_head_stride == o->out_head_stride;
            if (!same && heads_overlap(o->out, o->out_token_stride, o->out_head_stride, o->heads, m->in,
                                       m->in_token_stride, m->in_head_stride, m->heads, T, head_dim))
                return ADAFUSE_ERR_INVALID_ARG;
            if (m->weight && rows_overlap(mine, RowSpan{m->weight, 1, 2 * head_dim, 2 * head_dim}))
                return ADAFUSE_ERR_INVALID_ARG;
        }
        if (rot && (rows_overlap(mine, RowSpan{positions, 1, (int64_t)ps * T, (int64_t)ps * T}) ||
                    rows_overlap(mine, RowSpan{freq, 1, 4 * (int64_t)rot, 4 * (int64_t)rot})))
            return ADAFUSE_ERR_INVALID_ARG;
    }
    if (k && heads_overlap(q->out, q->out_token_stride, q->out_head_stride, q->heads, k->out, k->out_token_stride,
                           k->out_head_stride, k->heads, T, head_dim))
        return ADAFUSE_ERR_INVALID_ARG;

    const auto heads = [](const adafuse_heads* m) {
        return Heads{static_cast<const uint16_t*>(m->in), static_cast<uint16_t*>(m->out),
                     static_cast<const uint16_t*>(m->weight), m->in_token_stride, m->in_head_stride,
                     m->out_token_stride, m->out_head_stride};
    };
    RotArgs a{};
    a.q = heads(q);
    if (k) a.k = heads(k);
    a.pos = positions;
    a.freq = freq;
    a.T = T;
    a.Hq = q->heads;
    a.H = q->heads + (k ? k->heads : 0);
    a.D = head_dim;
    a.rot = rot;
    a.half = rot / 2;
    a.pairs = flags & ADAFUSE_PAIRS ? 1 : 0;
    a.pos32 = flags & ADAFUSE_POS_I32 ? 1 : 0;
    a.factor = factor;
    a.eps = eps;
    a.inv_d = 1.f / (float)head_dim;

    // The widest vectors that the layout allows; a head's items one per lane
    // where 32 lanes are enough.
    const int edge = a.pairs ? rot : a.half;        // vectors may not cross from rotated to unrotated elements
    const auto fits = [&](int V) {
        return head_dim % V == 0 && edge % V == 0 && rot % V == 0 && vectors_fit(q, V, (int)std::min<int64_t>(T, 2)) &&
               vectors_fit(k, V, (int)std::min<int64_t>(T, 2));
    };
    const auto items = [&](int V) { return (a.pairs && V > 1 ? rot : a.half) / V + (head_dim - rot) / V; };
    int V = fits(8) && items(8) <= 32 ? 8 : fits(4) ? 4 : 1;
    a.items = items(V);
    const bool one = V > 1 && a.items <= 32;
    a.lanes = 1;
    while (a.lanes < 32 && a.lanes < a.items) a.lanes *= 2;
    const int sms = device_sms();
    if (!sms) return ADAFUSE_ERR_DEVICE;
    // Tokens per CTA: one while that leaves SMs without eight CTAs, up to four.
    a.tokens = (int)std::max<int64_t>(1, std::min<int64_t>(4, T / ((int64_t)sms * 8)));
    const int64_t blocks = (T + a.tokens - 1) / a.tokens;
    if (blocks > 0x7fffffff) return ADAFUSE_ERR_UNSUPPORTED;
    auto kernel = V == 8 ? rotary_kernel<8, true> : one ? rotary_kernel<4, true>
                : V == 4 ? rotary_kernel<4, false> : rotary_kernel<1, false>;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kRotThreads), (size_t)a.tokens * a.half * sizeof(float2),
                      (cudaStream_t)stream, a);
}
