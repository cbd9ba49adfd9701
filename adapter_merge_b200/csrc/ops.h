// Host-side helpers of the operators between the adapted linears: overlap,
// stride and alignment checks, the tensor-map encoder, cluster launches.
#pragma once

#include <cudaTypedefs.h>

#include "internal.h"

namespace af {

// A strided set of rows in device memory, for the overlap checks.
struct RowSpan {
    const void* base;
    int64_t rows, row_bytes, pitch;    // pitch 0: one row that every index reads
};

// Whether two row sets can share a byte.  Sets whose address ranges cross are
// told apart only where both have one pitch (columns of one buffer).
inline bool rows_overlap(RowSpan a, RowSpan b)
{
    if (a.pitch == 0) a.rows = 1;
    if (b.pitch == 0) b.rows = 1;
    if (a.rows < 1 || b.rows < 1) return false;
    const int64_t pa = reinterpret_cast<int64_t>(a.base), pb = reinterpret_cast<int64_t>(b.base);
    const __int128 ea = (__int128)(a.rows - 1) * a.pitch + pa + a.row_bytes;
    const __int128 eb = (__int128)(b.rows - 1) * b.pitch + pb + b.row_bytes;
    if (ea <= pb || eb <= pa) return false;
    if (a.rows == 1 && b.rows == 1) return true;
    const int64_t pitch = a.rows == 1 ? b.pitch : a.pitch;
    if (b.rows > 1 && b.pitch != pitch) return true;
    if (a.row_bytes > pitch || b.row_bytes > pitch) return true;
    const int64_t d = ((pb - pa) % pitch + pitch) % pitch;     // b's first byte within a's pitch
    return d < a.row_bytes || d + b.row_bytes > pitch;
}

// Strides that the operators take, in elements; their byte offsets fit 64 bits
// with any number of rows that memory holds.
inline bool plain_stride(int64_t ld) { return ld >= 0 && ld < (1ll << 38); }

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The driver's tensor-map encoder, resolved once (thread-safe static
// initialisation); null if the driver does not provide it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// SMs of the current device (asked once per device), or 0 without a usable one.
int device_sms();

// As launch_pdl, in clusters of `cluster` CTAs along x.
template <typename... Params, typename... Args>
inline int launch_pdl_cluster(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, int cluster,
                              cudaStream_t s, Args&&... args)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_err(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...));
}

}  // namespace af
