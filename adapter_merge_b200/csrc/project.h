// What the projections' two kernels share: the call as the entry points have
// checked it, and the tensor maps of its operands.
#pragma once

#include "ops.h"

namespace af {

struct ProjectArgs {
    void* y;
    const uint16_t* residual;
    const uint16_t* bias;
    const uint16_t* bias_up;
    int32_t* status;
    int64_t ldy, ldr, T;
    int32_t N;              // d_out
    int32_t chunks;         // of kChunkK columns of d_in
    uint32_t act;
    int32_t y_f32, stall;
};

struct ProjectCall {
    const void *x, *W, *W_up;       // W_up: null for a plain projection
    int64_t ldx, ldw;
    int32_t K;
    ProjectArgs a;
    cudaStream_t s;
};

// Columns per accumulator of an fp32 output.
constexpr int kPartCols = 512;

// Tensor map of bf16 [rows, cols], rows `ld` elements apart: boxes of kChunkK
// columns x box_rows rows, 128-byte swizzle.
bool encode_rows(CUtensorMap* m, const void* p, int64_t rows, int32_t cols, int64_t ld, int box_rows);

int launch_project_tile(ProjectCall& c);
double project_tile_cost(const ProjectCall& c);     // estimated cycles

}  // namespace af
