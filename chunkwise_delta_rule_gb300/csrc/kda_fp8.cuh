// e4m3 values with a scale for each group of 128: the quantiser (kda_quant8.cu) and the product (kda_mm8.cu).
#pragma once

#include <cuda_fp8.h>

#include "kda_layer.cuh"

namespace kda {

constexpr int FP8_GROUP = 128;
constexpr float FP8_MAX = 448.f;

struct Quant8Args {
    int rows, D, blocks;
    int64_t ldx, ldq, ldqt;
    const void* x;
    uint8_t *q, *qt;
    float *scale, *scale_t;
};
cudaError_t launch_quant8(const Quant8Args& a, int bf16, cudaStream_t st);

struct Mm8Args {
    int M, N, K, groups, b_rows, f32;
    int64_t lda, ldb;
    const uint8_t *a, *b;
    const float *sa, *sb;
    void* y;
    int32_t* err;
};
// Bytes of workspace: copies of operands whose rows do not start every 16 bytes.
size_t mm8_align_bytes(const Mm8Args& a);
cudaError_t launch_mm8(Mm8Args a, void* ws, cudaStream_t st);

}  // namespace kda
