// The projections' epilogue on outputs that exist already:
//   out = act(y + bias) * up + residual,
// e.g. silu(y_gate) * y_up of an unmerged apply, or the one rounding of a
// row-parallel layer's all-reduced fp32 sums together with its bias and the
// residual stream.
//
// HBM-bound: every operand is read and written once.  A thread takes one group
// of eight consecutive elements of a row (16 bytes of bf16, two 16-byte
// accesses of fp32) where every operand's address and row stride allow it, one
// element otherwise, and loads all its operands before it uses the first.
// 2047 rows of 5120 fp32 sums with bias and residual: 13.9 us (6.0 TB/s); two
// groups a thread 21 us, a loop over a few thousand threads 16.9 us.
#include <cuda_bf16.h>

#include "act.cuh"
#include "ops.h"
#include "ptx_ops.cuh"

namespace af {
namespace {

constexpr int kEpiThreads = 128;

struct EpiArgs {
    const void* y;
    const uint16_t* bias;
    const void* up;
    const uint16_t* res;
    void* out;
    int64_t ldy, ldu, ldr, ldo, T;
    int32_t n;          // columns
    uint32_t act;
};

template <int V, bool kF32>
__device__ __forceinline__ void load_group(const void* p, int64_t at, float (&v)[V])
{
    if constexpr (kF32) {
        const float* f = static_cast<const float*>(p) + at;
        if constexpr (V == 8) {
            const float4 a = *reinterpret_cast<const float4*>(f), b = *reinterpret_cast<const float4*>(f + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            v[0] = *f;
        }
    } else {
        const uint16_t* h = static_cast<const uint16_t*>(p) + at;
        if constexpr (V == 8) {
            const uint4 a = *reinterpret_cast<const uint4*>(h);
            v[0] = bf16lo(a.x); v[1] = bf16hi(a.x); v[2] = bf16lo(a.y); v[3] = bf16hi(a.y);
            v[4] = bf16lo(a.z); v[5] = bf16hi(a.z); v[6] = bf16lo(a.w); v[7] = bf16hi(a.w);
        } else {
            v[0] = __uint_as_float((uint32_t)*h << 16);
        }
    }
}

template <int V, bool kF32>
__device__ __forceinline__ void store_group(void* p, int64_t at, const float (&v)[V])
{
    if constexpr (kF32) {
        float* f = static_cast<float*>(p) + at;
        if constexpr (V == 8) {
            *reinterpret_cast<float4*>(f) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(f + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *f = v[0];
        }
    } else {
        uint16_t* h = static_cast<uint16_t*>(p) + at;
        if constexpr (V == 8)
            *reinterpret_cast<uint4*>(h) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        else
            *h = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    }
}

// Ten CTAs an SM: left alone the compiler takes 40 registers, with which not all
// of a thread's loads are under way at once (2047 x 5120 in graph replay: 13.7 us,
// 12.55 with 48).
template <int V, bool kInF32, bool kOutF32>
__global__ void __launch_bounds__(kEpiThreads, 10) epilogue_kernel(const EpiArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t groups = a.n / V, total = groups * a.T;
    const int64_t g = (int64_t)blockIdx.x * kEpiThreads + threadIdx.x;
    if (g >= total) return;
    const int64_t row = total <= 0x7fffffff ? (int64_t)((uint32_t)g / (uint32_t)groups) : g / groups;
    const int64_t col = (g - row * groups) * V;
    float v[V], b[V], u[V], r[V];
    load_group<V, kInF32>(a.y, row * a.ldy + col, v);
    if (a.up) load_group<V, kInF32>(a.up, row * a.ldu + col, u);
    if (a.res) load_group<V, false>(a.res, row * a.ldr + col, r);
    if (a.bias) {
        load_group<V, false>(a.bias, col, b);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += b[i];
    }
    activate_all(v, a.act);
    if (a.up) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= u[i];
    }
    if (a.res) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += r[i];
    }
    store_group<V, kOutF32>(a.out, row * a.ldo + col, v);
}

template <int V>
int launch_epilogue(const EpiArgs& a, bool in_f32, bool out_f32, cudaStream_t s)
{
    if (!device_sms()) return ADAFUSE_ERR_DEVICE;
    const int64_t groups = (int64_t)(a.n / V) * a.T;
    const int64_t blocks = (groups + kEpiThreads - 1) / kEpiThreads;
    if (blocks > 0x7fffffff) return ADAFUSE_ERR_UNSUPPORTED;
    auto kernel = in_f32 ? (out_f32 ? epilogue_kernel<V, true, true> : epilogue_kernel<V, true, false>)
                         : (out_f32 ? epilogue_kernel<V, false, true> : epilogue_kernel<V, false, false>);
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kEpiThreads), 0, s, a);
}

}  // namespace
}  // namespace af

using namespace af;

extern "C" int adafuse_epilogue(const void* y, int64_t T, int64_t n, int64_t y_row_stride, const void* bias,
                                const void* up, int64_t up_row_stride, const void* residual, int64_t r_row_stride,
                                void* out, int64_t out_row_stride, uint32_t flags, adafuse_stream_t stream)
{
    const uint32_t act = flags & ADAFUSE_ACT_MASK;
    if (flags & ~(ADAFUSE_ACT_MASK | ADAFUSE_IN_F32 | ADAFUSE_OUT_F32)) return ADAFUSE_ERR_INVALID_ARG;
    if (T < 0 || n < 1) return ADAFUSE_ERR_INVALID_ARG;
    if (act > ADAFUSE_ACT_GELU_TANH || n > 0x7fffffff || T > 0x7fffffff) return ADAFUSE_ERR_UNSUPPORTED;
    if (T == 0) return ADAFUSE_OK;
    if (!y || !out) return ADAFUSE_ERR_INVALID_ARG;
    if (!up) up_row_stride = 0;
    if (!residual) r_row_stride = 0;
    if (T == 1) y_row_stride = out_row_stride = up_row_stride = r_row_stride = n;
    const auto fits = [n](int64_t ld) { return ld == 0 || ld >= n; };
    if (!fits(y_row_stride) || !fits(up_row_stride) || !fits(r_row_stride) || out_row_stride < n)
        return ADAFUSE_ERR_INVALID_ARG;
    for (const int64_t ld : {y_row_stride, up_row_stride, r_row_stride, out_row_stride})
        if (!plain_stride(ld)) return ADAFUSE_ERR_UNSUPPORTED;
    const bool in_f32 = flags & ADAFUSE_IN_F32, out_f32 = flags & ADAFUSE_OUT_F32;
    const int64_t si = in_f32 ? 4 : 2, so = out_f32 ? 4 : 2;
    if (!aligned_to(y, si) || !aligned_to(up, si) || !aligned_to(out, so) || !aligned_to(bias, 2) ||
        !aligned_to(residual, 2))
        return ADAFUSE_ERR_INVALID_ARG;
    const RowSpan o{out, T, n * so, out_row_stride * so};
    const auto clash = [&](const void* p, int64_t ld, int64_t size) {
        if (!p || (p == out && ld == out_row_stride && size == so)) return false;
        return rows_overlap(o, RowSpan{p, T, n * size, ld * size});
    };
    if (clash(y, y_row_stride, si) || clash(up, up_row_stride, si) || clash(residual, r_row_stride, 2) ||
        (bias && rows_overlap(o, RowSpan{bias, 1, n * 2, n * 2})))
        return ADAFUSE_ERR_INVALID_ARG;
    const EpiArgs a{y, static_cast<const uint16_t*>(bias), up, static_cast<const uint16_t*>(residual), out,
                    y_row_stride, up_row_stride, r_row_stride, out_row_stride, T, (int32_t)n, act};
    const bool wide = n % 8 == 0 && y_row_stride % 8 == 0 && up_row_stride % 8 == 0 && r_row_stride % 8 == 0 &&
                      out_row_stride % 8 == 0 && aligned_to(y, 16) && aligned_to(up, 16) && aligned_to(out, 16) &&
                      aligned_to(bias, 16) && aligned_to(residual, 16);
    return wide ? launch_epilogue<8>(a, in_f32, out_f32, (cudaStream_t)stream)
                : launch_epilogue<1>(a, in_f32, out_f32, (cudaStream_t)stream);
}
