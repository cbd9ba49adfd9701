// Rotation of queries and keys by their positions, after an optional RMS norm
// of each head, in one pass over the heads.
//
// Angles.  Pair i of the token at position p turns by p * freq[i] radians.
// For far positions that product loses its fraction in fp32 (at p = 2^20 an
// fp32 angle is off by up to 1/32 rad) and in the end in fp64 (by 0.06 rad at
// 2^50).  So the frequency is taken as a fraction of a turn with 128 bits after
// the point, F = freq / (2 pi) modulo 1, from a product with 1 / (2 pi) in two
// doubles (off by at most 2^-105 of freq / (2 pi)), and the upper 64 bits of
// p * F modulo 1 are two integer products, for positions of either sign and no
// range reduction.  They go to sincospif.
//
// HBM-bound for long prompts (each element read and written once), latency
// for a decode batch.  One warp, or several, take a token: each computes the
// token's sines and cosines into shared memory (rot/2, shared by all heads; a
// lane then keeps those of its own elements), then its lanes rotate the heads:
// an item is a vector of V elements together with the vector of its partners
// (one vector that holds both in the interleaved layout, one unrotated vector
// past `rot`), and as many neighbouring lanes as a head has items share it, so
// that the norm's sum is a shuffle among them.  A lane loads its next heads' items before it
// rotates those it has.  No barrier across warps.
#include <cuda_bf16.h>

#include "ops.h"
#include "ptx_ops.cuh"

namespace af {
namespace {

constexpr int kRotThreads = 128;
constexpr int kRotWarps = kRotThreads / 32;
// Heads that a lane loads ahead of those it rotates.  8192 tokens of 32 + 8
// heads of 128 with norms: 33.3 us with two, 36.9 with one (34.3-34.8 now, with
// angles of 128 bits); 4097 tokens of 80 heads, interleaved: 30.8-31.5 with two
// (of one vector each).
__host__ __device__ constexpr int flight(bool pairs, bool norm) { return (norm ? 2 : 1) * (pairs ? 2 : 1); }
constexpr int kLaneHeads = 20;          // most heads of a prompt's token per lane
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
    int32_t lanes;          // lanes per head
    int32_t first_step;     // half of the next power of two
    int32_t items;          // items per head
    int32_t warps, warps_log2;      // warps per token: a power of two
    int32_t pairs, pos32;
    float factor, eps, inv_d;
};

// V bf16 elements as they come from memory.
template <int V>
struct Raw {
    uint32_t w[V == 1 ? 1 : V / 2];
    __device__ __forceinline__ void load(const uint16_t* p)
    {
        if constexpr (V == 8) {
            const uint4 a = *reinterpret_cast<const uint4*>(p);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        } else if constexpr (V == 4) {
            const uint2 a = *reinterpret_cast<const uint2*>(p);
            w[0] = a.x; w[1] = a.y;
        } else {
            w[0] = *p;
        }
    }
};

template <int V>
struct Vec {
    float v[V];
    __device__ __forceinline__ void from(const Raw<V>& r)
    {
        if constexpr (V == 1) {
            v[0] = bf16lo(r.w[0]);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                v[2 * i] = bf16lo(r.w[i]);
                v[2 * i + 1] = bf16hi(r.w[i]);
            }
        }
    }
    __device__ __forceinline__ void load(const uint16_t* p)
    {
        Raw<V> r;
        r.load(p);
        from(r);
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

// The sum over the lanes that share a head, in all of them: lane `sub` of a
// group of any size adds up those behind it, the first one's sum goes to all.
__device__ __forceinline__ float head_sum(const RotArgs& a, float v, int sub, int group)
{
    for (int d = a.first_step; d; d >>= 1) {
        const float w = __shfl_down_sync(0xffffffffu, v, d);
        if (sub + d < a.lanes) v += w;
    }
    return __shfl_sync(0xffffffffu, v, group * a.lanes & 31);
}

// A frequency of f >= 0 radians as turns modulo 1, 128 bits after the point.
struct Turns {
    uint64_t hi, lo;
    __device__ __forceinline__ explicit Turns(double f)
    {
        constexpr double kC = 0.15915494309189535, kCLow = -9.839338337591243e-18;     // 1 / (2 pi) and what is left of it
        constexpr double k2p64 = 18446744073709551616.0;
        double t = f * kC, e = __fma_rn(f, kCLow, __fma_rn(f, kC, -t));                 // t + e turns
        t -= floor(t);                          // both exact
        e -= rint(e);
        const double a = t * k2p64, b = e * k2p64, below = floor(b);
        hi = __double2ull_rd(a);
        lo = __double2ull_rd((a - (double)hi) * k2p64);
        const uint64_t add = __double2ull_rd((b - below) * k2p64);
        lo += add;
        hi += (uint64_t)(int64_t)below + (lo < add ? 1u : 0u);
    }
    // the last turn of p times it, in 2^-64 turns
    __device__ __forceinline__ int64_t times(int64_t p) const
    {
        return (int64_t)((uint64_t)p * hi + __umul64hi((uint64_t)p, lo) - (p < 0 ? lo : 0ull));
    }
};

// The token's sines and cosines times the factor, by one warp.
__device__ __forceinline__ void turn_token(const RotArgs& a, int64_t t, float* cosv, float* sinv)
{
    if (!a.half) return;
    const int64_t p = a.pos32 ? (int64_t)static_cast<const int32_t*>(a.pos)[t] : static_cast<const int64_t*>(a.pos)[t];
    for (int i = threadIdx.x & 31; i < a.half; i += 32) {
        const double f = a.freq[i];
        float s, c;
        sincospif((float)Turns(fabs(f)).times(p) * 1.08420217248550443401e-19f, &s, &c);        // 2^-63 half turns
        if (!isfinite(f)) s = c = __int_as_float(0x7fffffff);   // NaN, as the formula has it, at every position
        cosv[i] = c * a.factor;
        sinv[i] = (f < 0 ? -s : s) * a.factor;
    }
    __syncwarp();
}

// Two fp32 values and the arithmetic on both at once.
struct Two {
    uint64_t v;
    __device__ __forceinline__ Two() {}
    __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ float2 get() const
    {
        float2 r;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
        return r;
    }
};
__device__ __forceinline__ Two operator*(Two a, Two b)
{
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Two unpack2(uint32_t w) { return Two(bf16lo(w), bf16hi(w)); }
__device__ __forceinline__ uint32_t pack2(Two a)
{
    const float2 f = a.get();
    return pack_bf16x2(f.x, f.y);
}

template <int V>
__device__ __forceinline__ void store_raw(const Raw<V>& r, uint16_t* p)
{
    if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
}

// The heads of one kind of a token, whose items (j of every head) one lane
// holds: heads h0, h0 + stride, ...; the same number of steps for all lanes.
// A pair turns as (p, q) -> (p a - q b, p c + q d); the coefficients hold the
// weights, so a norm costs its sum and one factor more.  All arithmetic is on
// two neighbouring elements at a time: two pairs, or, interleaved, the two
// elements of one.
template <int V, bool kPairs, bool kNorm>
__device__ __forceinline__ void rotate_heads(const RotArgs& a, const Heads& m, int n, int64_t t, int h0, int stride,
                                             int group, int sub, const Item<V>& it, bool mine, const float* cosv,
                                             const float* sinv)
{
    constexpr int H = V / 2;                        // words of a vector
    constexpr int F = flight(kPairs, kNorm);
    const bool turns = it.pair >= 0, two = !kPairs && it.o2 >= 0;
    // half: first' = first A - second B, second' = first C + second D, of two pairs
    // interleaved: (p', q') = (p, q) A + (q, p) B, of one pair
    Two A[H], B[H], C[H], D[H];
    if (mine) {
        Raw<V> w0, w1;
#pragma unroll
        for (int i = 0; i < H; ++i) w0.w[i] = w1.w[i] = 0x3f803f80u;        // ones
        if constexpr (kNorm) {
            w0.load(m.weight + it.o1);
            if (two) w1.load(m.weight + it.o2);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float p0 = bf16lo(w0.w[i]), p1 = bf16hi(w0.w[i]), q0 = bf16lo(w1.w[i]), q1 = bf16hi(w1.w[i]);
            if constexpr (kPairs) {
                const float c = turns ? cosv[it.pair + i] : 1.f, s = turns ? sinv[it.pair + i] : 0.f;
                A[i] = Two(c * p0, c * p1);
                B[i] = Two(-s * p1, s * p0);
            } else {
                const float c0 = turns ? cosv[it.pair + 2 * i] : 1.f, s0 = turns ? sinv[it.pair + 2 * i] : 0.f;
                const float c1 = turns ? cosv[it.pair + 2 * i + 1] : 1.f, s1 = turns ? sinv[it.pair + 2 * i + 1] : 0.f;
                A[i] = Two(c0 * p0, c1 * p1);
                B[i] = Two(-s0 * q0, -s1 * q1);
                C[i] = Two(s0 * p0, s1 * p1);
                D[i] = Two(c0 * q0, c1 * q1);
            }
        }
    }
    const uint16_t* in = m.in + t * m.its + h0 * m.ihs;
    uint16_t* out = m.out + t * m.ots + h0 * m.ohs;
    const int64_t din = stride * m.ihs, dout = stride * m.ohs;
    Raw<V> nx[F], ny[F];
    const auto fetch = [&](int h) {
#pragma unroll
        for (int j = 0; j < F; ++j) {
            if (mine && h + j * stride < n) {
                nx[j].load(in + it.o1);
                if (two) ny[j].load(in + it.o2);
            }
            in += din;
        }
    };
    fetch(h0);
    for (int h = h0; h - group < n; h += F * stride) {
        Raw<V> rx[F], ry[F];
#pragma unroll
        for (int j = 0; j < F; ++j) {
            rx[j] = nx[j];
            ry[j] = ny[j];
        }
        fetch(h + F * stride);
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const bool live = mine && h + j * stride < n;
            Two r(1.f, 1.f);
            if constexpr (kNorm) {
                float sum = 0.f;
                if (live) {
                    Two s(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const Two x = unpack2(rx[j].w[i]);
                        s = fma2(x, x, s);
                    }
                    if (two) {
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            const Two y = unpack2(ry[j].w[i]);
                            s = fma2(y, y, s);
                        }
                    }
                    const float2 f = s.get();
                    sum = f.x + f.y;
                }
                const float f = rsqrtf(head_sum(a, sum, sub, group) * a.inv_d + a.eps);
                r = Two(f, f);
            }
            if (live) {
                if (turns) {
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const Two x = unpack2(rx[j].w[i]);
                        if constexpr (kPairs) {
                            Two u = fma2(Two(bf16hi(rx[j].w[i]), bf16lo(rx[j].w[i])), B[i], x * A[i]);
                            if (kNorm) u = u * r;
                            rx[j].w[i] = pack2(u);
                        } else {
                            const Two y = unpack2(ry[j].w[i]);
                            Two u = fma2(y, B[i], x * A[i]), v = fma2(y, D[i], x * C[i]);
                            if (kNorm) {
                                u = u * r;
                                v = v * r;
                            }
                            rx[j].w[i] = pack2(u);
                            ry[j].w[i] = pack2(v);
                        }
                    }
                } else if constexpr (kNorm) {
#pragma unroll
                    for (int i = 0; i < H; ++i) rx[j].w[i] = pack2(unpack2(rx[j].w[i]) * A[i] * r);
                }
                store_raw(rx[j], out + it.o1);
                if (two) store_raw(ry[j], out + it.o2);
            }
            out += dout;
        }
    }
}

// Heads of at most as many items as lanes share them.
template <int V, bool kPairs, bool kNorm>
__global__ void __launch_bounds__(kRotThreads, 5) rotary_kernel(const RotArgs a)
{
    extern __shared__ float angles[];       // per warp: rot/2 cosines, rot/2 sines
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kRotWarps + warp, t = w >> a.warps_log2;
    if (t >= a.T) return;
    float* cosv = angles + warp * 2 * a.half;
    float* sinv = cosv + a.half;
    turn_token(a, t, cosv, sinv);
    const int group = lane / a.lanes, sub = lane - group * a.lanes;
    const int per = 32 / a.lanes, stride = per * a.warps;
    const int first = ((int)w & (a.warps - 1)) * per + group;
    const Item<V> it(a, sub);
    const bool mine = group < per;          // lanes past the last whole head idle
    if (kNorm && a.q.weight)
        rotate_heads<V, kPairs, true>(a, a.q, a.Hq, t, first, stride, group, sub, it, mine, cosv, sinv);
    else
        rotate_heads<V, kPairs, false>(a, a.q, a.Hq, t, first, stride, group, sub, it, mine, cosv, sinv);
    if (kNorm && a.k.weight)
        rotate_heads<V, kPairs, true>(a, a.k, a.H - a.Hq, t, first, stride, group, sub, it, mine, cosv, sinv);
    else
        rotate_heads<V, kPairs, false>(a, a.k, a.H - a.Hq, t, first, stride, group, sub, it, mine, cosv, sinv);
}

// Any head: a warp walks its items, twice for a norm.
template <int V>
__global__ void __launch_bounds__(kRotThreads) rotary_any_kernel(const RotArgs a)
{
    extern __shared__ float angles[];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kRotWarps + warp, t = w >> a.warps_log2;
    if (t >= a.T) return;
    float* cosv = angles + warp * 2 * a.half;
    float* sinv = cosv + a.half;
    turn_token(a, t, cosv, sinv);
    const int group = lane / a.lanes, sub = lane - group * a.lanes;
    const int per = 32 / a.lanes;
    for (int h = ((int)w & (a.warps - 1)) * per + group; h - group < a.H; h += per * a.warps) {
        const bool live = h < a.H && group < per;
        const Heads& m = h < a.Hq ? a.q : a.k;
        const int64_t hh = !live ? 0 : h < a.Hq ? h : h - a.Hq;
        const uint16_t* in = m.in + t * m.its + hh * m.ihs;
        uint16_t* out = m.out + t * m.ots + hh * m.ohs;
        Vec<V> x, y, w;
        float sum = 0.f;
        for (int j = sub; live && m.weight && j < a.items; j += a.lanes) {
            const Item<V> it(a, j);
            x.load(in + it.o1);
            sum += x.squares();
            if (it.o2 >= 0) {
                y.load(in + it.o2);
                sum += y.squares();
            }
        }
        const float r = rsqrtf(head_sum(a, sum, sub, group) * a.inv_d + a.eps);
        for (int j = sub; live && j < a.items; j += a.lanes) {
            const Item<V> it(a, j);
            x.load(in + it.o1);
            if (it.o2 >= 0) y.load(in + it.o2);
            if (m.weight) {
                w.load(m.weight + it.o1);
#pragma unroll
                for (int i = 0; i < V; ++i) x.v[i] *= r * w.v[i];
                if (it.o2 >= 0) {
                    w.load(m.weight + it.o2);
#pragma unroll
                    for (int i = 0; i < V; ++i) y.v[i] *= r * w.v[i];
                }
            }
            if (it.o2 >= 0) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float c = cosv[it.pair + i], s = sinv[it.pair + i], p = x.v[i], q = y.v[i];
                    x.v[i] = p * c - q * s;
                    y.v[i] = p * s + q * c;
                }
            } else if (V > 1 && it.pair >= 0) {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float c = cosv[it.pair + i], s = sinv[it.pair + i], p = x.v[2 * i], q = x.v[2 * i + 1];
                    x.v[2 * i] = p * c - q * s;
                    x.v[2 * i + 1] = p * s + q * c;
                }
            }
            x.store(out + it.o1);
            if (it.o2 >= 0) y.store(out + it.o2);
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

// Elements from a token's first head to the end of its last.
int64_t token_span(int32_t heads, int64_t head_stride, int32_t D) { return (int64_t)(heads - 1) * head_stride + D; }

// Heads as the overlap checks see them.
struct Span {
    const void* base;
    int64_t token_stride, head_stride;
    int32_t heads;
};

// Whether two sets of heads can share an element.  Sets whose address ranges
// cross are told apart where they have the same token stride and each token's
// heads lie within it (columns of one buffer), or the same head stride, of
// which the token stride is a multiple (q, k and v of a head side by side).
bool heads_overlap(const Span& p, const Span& q, int64_t T, int32_t D)
{
    if (!rows_overlap(RowSpan{p.base, T, 2 * token_span(p.heads, p.head_stride, D), 2 * p.token_stride},
                      RowSpan{q.base, T, 2 * token_span(q.heads, q.head_stride, D), 2 * q.token_stride}))
        return false;
    const int64_t hs = p.head_stride;
    if (hs != q.head_stride || hs < 2 * D || p.token_stride % hs || q.token_stride % hs) return true;
    const int64_t gap = (int64_t)(reinterpret_cast<uintptr_t>(q.base) - reinterpret_cast<uintptr_t>(p.base));
    const int64_t d = (gap % (2 * hs) + 2 * hs) % (2 * hs);
    return d < 2 * D || d + 2 * D > 2 * hs;
}

int check_heads(const adafuse_heads* m, int64_t T, int32_t D)
{
    if (!m->in || !m->out || m->heads < 1) return ADAFUSE_ERR_INVALID_ARG;
    if (m->heads > 65536) return ADAFUSE_ERR_UNSUPPORTED;
    if (!aligned_to(m->in, 2) || !aligned_to(m->out, 2) || !aligned_to(m->weight, 2)) return ADAFUSE_ERR_INVALID_ARG;
    if (m->in_token_stride < 0 || m->in_head_stride < 0 || m->out_token_stride < 0 || m->out_head_stride < 0)
        return ADAFUSE_ERR_INVALID_ARG;
    for (const int64_t ld : {m->in_token_stride, m->in_head_stride, m->out_token_stride, m->out_head_stride})
        if (!plain_stride(ld)) return ADAFUSE_ERR_UNSUPPORTED;
    // the outputs of two heads or tokens may not meet: either axis may be the outer one
    const int64_t ts = m->out_token_stride, hs = m->out_head_stride;
    const bool token_outer = (m->heads == 1 || hs >= D) && (T == 1 || ts >= token_span(m->heads, hs, D));
    const bool head_outer = (T == 1 || ts >= D) && (m->heads == 1 || hs >= (__int128)(T - 1) * ts + D);
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
    if (rot % 2 || rot > head_dim || head_dim > kMaxHeadDim || T > 0x7fffffff) return ADAFUSE_ERR_UNSUPPORTED;
    if (T == 0) return ADAFUSE_OK;
    int rc = check_heads(q, T, head_dim);
    if (!rc && k) rc = check_heads(k, T, head_dim);
    if (rc) return rc;
    const uintptr_t ps = flags & ADAFUSE_POS_I32 ? 4 : 8;
    if (rot && (!positions || !freq || !aligned_to(positions, ps) || !aligned_to(freq, 8)))
        return ADAFUSE_ERR_INVALID_ARG;
    const adafuse_heads* all[2] = {q, k};
    const auto span_of = [T, head_dim](const adafuse_heads* m, bool out) {      // strides that are not used: as if dense
        Span s{out ? m->out : m->in, out ? m->out_token_stride : m->in_token_stride,
               out ? m->out_head_stride : m->in_head_stride, m->heads};
        if (m->heads == 1) s.head_stride = head_dim;
        if (T == 1) s.token_stride = m->heads * s.head_stride;
        return s;
    };
    for (int i = 0; i < 2; ++i) {
        const adafuse_heads* o = all[i];
        if (!o) continue;
        const Span so = span_of(o, true);
        const RowSpan mine{o->out, T, 2 * token_span(o->heads, so.head_stride, head_dim), 2 * so.token_stride};
        for (int j = 0; j < 2; ++j) {
            const adafuse_heads* m = all[j];
            if (!m) continue;
            const Span si = span_of(m, false);
            const bool same = i == j && si.base == so.base && si.token_stride == so.token_stride &&
                              si.head_stride == so.head_stride;
            if (!same && heads_overlap(so, si, T, head_dim)) return ADAFUSE_ERR_INVALID_ARG;
            if (m->weight && rows_overlap(mine, RowSpan{m->weight, 1, 2 * head_dim, 2 * head_dim}))
                return ADAFUSE_ERR_INVALID_ARG;
        }
        if (rot && (rows_overlap(mine, RowSpan{positions, 1, (int64_t)ps * T, (int64_t)ps * T}) ||
                    rows_overlap(mine, RowSpan{freq, 1, 4 * (int64_t)rot, 4 * (int64_t)rot})))
            return ADAFUSE_ERR_INVALID_ARG;
    }
    if (k && heads_overlap(span_of(q, true), span_of(k, true), T, head_dim)) return ADAFUSE_ERR_INVALID_ARG;

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
    a.lanes = std::min(32, a.items);
    while (2 * a.first_step < a.lanes) a.first_step = std::max(1, 2 * a.first_step);
    const int sms = device_sms();
    if (!sms) return ADAFUSE_ERR_DEVICE;
    // Warps per token: one while a lane has at most kLaneHeads heads (each
    // warp computes the token's sines again: 4097 tokens of 80 heads took 32 us
    // with 20 heads per lane, 41 us with five), but enough to give every SM
    // its warps, as long as each has a head for its groups of lanes.
    a.warps = 1;
    while (a.warps * (32 / a.lanes) < a.H &&
           (T * a.warps < (int64_t)sms * 16 || a.H > kLaneHeads * a.warps * (32 / a.lanes))) a.warps *= 2;
    while ((1 << a.warps_log2) < a.warps) ++a.warps_log2;
    const int64_t blocks = (T * a.warps + kRotWarps - 1) / kRotWarps;
    if (blocks > 0x7fffffff) return ADAFUSE_ERR_UNSUPPORTED;
    const bool norm = q->weight || (k && k->weight);
    auto kernel = rotary_any_kernel<1>;
    if (one && V == 8)
        kernel = a.pairs ? (norm ? rotary_kernel<8, true, true> : rotary_kernel<8, true, false>)
                         : (norm ? rotary_kernel<8, false, true> : rotary_kernel<8, false, false>);
    else if (one)
        kernel = a.pairs ? (norm ? rotary_kernel<4, true, true> : rotary_kernel<4, true, false>)
                         : (norm ? rotary_kernel<4, false, true> : rotary_kernel<4, false, false>);
    else if (V == 4)
        kernel = rotary_any_kernel<4>;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kRotThreads), (size_t)kRotWarps * rot * sizeof(float),
                      (cudaStream_t)stream, a);
}
