// Matrix product of e4m3 values with a scale for each 128 columns (include/kda.h), on CUDA cores:
//     y[m, n] = sum_g sa[m, g] sb[n, g] sum_{c in g} a[m, c] b[n, c].
// A group's sum is formed in fp32, then scaled and added to the output's.
#include "kda_fp8.cuh"

namespace kda {
namespace {

constexpr int NT = 256, TM = 64, TK = 32;

__device__ __forceinline__ float value(uint8_t x) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(x, __NV_E4M3)));
}

__global__ void __launch_bounds__(NT) k_mm8(Mm8Args a) {
    __shared__ __align__(16) float as[TK][TM + 4], bs[TK][TM + 4];
    const int m0 = blockIdx.x * TM, n0 = blockIdx.y * TM, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {}, part[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += TK) {
        __syncthreads();
        for (int x = threadIdx.x; x < TM * TK; x += NT) {
            const int r = x / TK, c = x - r * TK;
            as[c][r] = m0 + r < a.M && k0 + c < a.K ? value(a.a[(int64_t)(m0 + r) * a.lda + k0 + c]) : 0.f;
            bs[c][r] = n0 + r < a.N && k0 + c < a.K ? value(a.b[(int64_t)(n0 + r) * a.ldb + k0 + c]) : 0.f;
        }
        __syncthreads();
#pragma unroll 8
        for (int c = 0; c < TK; ++c) {
            const float4 x = *reinterpret_cast<const float4*>(&as[c][ty * 4]), y = *reinterpret_cast<const float4*>(&bs[c][tx * 4]);
            const float xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) part[i][j] = fmaf(xa[i], ya[j], part[i][j]);
        }
        const int g = k0 / FP8_GROUP;
        if ((k0 + TK) % FP8_GROUP && k0 + TK < a.K) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + ty * 4 + i;
            const float sa = m < a.M ? a.sa[(size_t)m * a.groups + g] : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx * 4 + j;
                if (n < a.N) acc[i][j] = fmaf(part[i][j], sa * a.sb[(size_t)(a.b_rows ? n : n / FP8_GROUP) * a.groups + g], acc[i][j]);
                part[i][j] = 0.f;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= a.M || n >= a.N) continue;
            if (a.f32) static_cast<float*>(a.y)[(size_t)m * a.N + n] = acc[i][j];
            else static_cast<__nv_bfloat16*>(a.y)[(size_t)m * a.N + n] = __float2bfloat16_rn(acc[i][j]);
        }
}

}  // namespace

cudaError_t launch_mm8(const Mm8Args& a, cudaStream_t st) {
    const dim3 grid((a.M + TM - 1) / TM, (a.N + TM - 1) / TM);
    return traced_launch("k_mm8", st, [&] { k_mm8<<<grid, NT, 0, st>>>(a); });
}

}  // namespace kda
