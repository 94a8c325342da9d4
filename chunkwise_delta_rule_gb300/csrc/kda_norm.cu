// Root-mean-square norm of the residual stream, with the residual's addition in
// front and an optional 8-bit output for the projection behind it:
//     h = x + residual,  r = (mean h^2 + eps)^(-1/2),  y = h r w
// The sum h is kept in fp32 for the norm and rounded once where it is stored.
// e4m3 output: per group of `group` columns (0: the row) scale = amax |y| / 448 and
// q = e4m3(y 448 / amax), to nearest even; a group of zeros has scale 0, and one
// that holds a NaN or an infinity has a NaN or infinite scale.
// Backward, from the stored h: with u = h r,
//     dx = r (w dy - u mean(u w dy)) + dres,   dw = sum over rows of dy u
// (the 8-bit rounding passes its gradient through unchanged).
// A row is held in registers by one warp or one CTA: each tensor is read once.
#include <cuda_fp8.h>

#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr float E4M3_MAX = 448.f;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
    return x;
}
// The larger magnitude; a NaN stays.
__device__ __forceinline__ float amax2(float a, float b) { return a > b || a != a ? a : b; }

// Sum (or NaN-keeping maximum) over the CTA's NT threads; every thread gets it. buf: NT / 32 floats.
template <int NT, bool MAX>
__device__ __forceinline__ float cta_reduce(float x, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(FULL, x, o);
        x = MAX ? amax2(x, y) : x + y;
    }
    if (NT == 32) return x;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    x = buf[0];
#pragma unroll
    for (int i = 1; i < NT / 32; ++i) x = MAX ? amax2(x, buf[i]) : x + buf[i];
    __syncthreads();
    return x;
}

// Columns of chunk k of a thread: chunks of 8 (CH = 8), or single columns side by side (CH = 1) for rows whose
// width is no multiple of 8, which keeps a warp's accesses together.
template <int NT, int CH>
__device__ __forceinline__ int col_of(int k) { return (k * NT + threadIdx.x) * CH; }

// One CTA of NT threads per row, NC chunks per thread.
template <typename TI, int NT, int NC, int CH, bool Q8>
__global__ void __launch_bounds__(NT) k_norm_fwd(NormArgs a, int vec) {
    __shared__ float buf[NT / 32];
    const size_t row = blockIdx.x;
    const TI* x = static_cast<const TI*>(a.x) + row * a.D;
    float h[NC][CH];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = col_of<NT, CH>(k);
#pragma unroll
        for (int i = 0; i < CH; ++i) h[k][i] = 0.f;
        if (c < a.D) load_row<CH>(x + c, h[k], a.D - c, vec);
    }
    if (a.residual) {
        const TI* res = static_cast<const TI*>(a.residual) + row * a.D;
        TI* ho = static_cast<TI*>(a.h) + row * a.D;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = col_of<NT, CH>(k);
            if (c >= a.D) continue;
            float r[CH];
            load_row<CH>(res + c, r, a.D - c, vec);
#pragma unroll
            for (int i = 0; i < CH; ++i) h[k][i] += r[i];
            store_row<CH>(ho + c, h[k], a.D - c, vec);
        }
    }
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < CH; ++i) ss = fmaf(h[k][i], h[k][i], ss);
    ss = cta_reduce<NT, false>(ss, buf);
    const float r = 1.f / sqrtf(ss / (float)a.D + a.eps);
    float rowmax = 0.f;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = col_of<NT, CH>(k);
        float w[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) w[i] = 0.f;
        if (c < a.D) load_row<CH>(a.weight + c, w, a.D - c, vec);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            h[k][i] = h[k][i] * r * w[i];
            if (Q8 && c + i < a.D) rowmax = amax2(fabsf(h[k][i]), rowmax);
        }
        if (!Q8 && c < a.D) store_row<CH>(static_cast<TI*>(a.y) + row * a.D + c, h[k], a.D - c, vec);
    }
    if (!Q8) return;
    uint8_t* q = static_cast<uint8_t*>(a.y) + row * a.D;
    float* sc = a.scale + row * a.ngroups;
    if (!a.group) rowmax = cta_reduce<NT, true>(rowmax, buf);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = col_of<NT, CH>(k);
        float m = rowmax;
        if (a.group) {
            m = 0.f;
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (c + i < a.D) m = amax2(fabsf(h[k][i]), m);
            for (int o = a.group / (2 * CH); o > 0; o >>= 1) m = amax2(m, __shfl_xor_sync(FULL, m, o));
        }
        if (c >= a.D) continue;
        if (a.group ? c % a.group == 0 : c == 0) sc[a.group ? c / a.group : 0] = m / E4M3_MAX;
        // 448 / m overflows below 1.4e-36: such groups are brought up by 2^64 first
        const float lift = m < 1e-30f ? 0x1p64f : 1.f;
        const float inv = m > 0.f ? E4M3_MAX / (m * lift) : (m == 0.f ? 0.f : m);
        uint32_t out[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < CH; ++i)
            out[i >> 2] |= (uint32_t)__nv_cvt_float_to_fp8(h[k][i] * lift * inv, __NV_SATFINITE, __NV_E4M3) << (8 * (i & 3));
        if (vec) {
            *reinterpret_cast<uint2*>(q + c) = make_uint2(out[0], out[1]);
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (c + i < a.D) q[c + i] = (uint8_t)(out[i >> 2] >> (8 * (i & 3)));
        }
    }
}

// CTA p takes rows p, p + parts, ...; each thread keeps its columns' dw sums.
template <typename TI, int NT, int NC, int CH>
__global__ void __launch_bounds__(NT) k_norm_bwd(NormArgs a, int vec) {
    __shared__ float buf[NT / 32];
    float w[NC][CH], dw[NC][CH];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = col_of<NT, CH>(k);
#pragma unroll
        for (int i = 0; i < CH; ++i) w[k][i] = dw[k][i] = 0.f;
        if (c < a.D) load_row<CH>(a.weight + c, w[k], a.D - c, vec);
    }
    for (int rw = blockIdx.x; rw < a.rows; rw += a.parts) {
        const size_t o = (size_t)rw * a.D;
        float h[NC][CH], d[NC][CH];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = col_of<NT, CH>(k);
#pragma unroll
            for (int i = 0; i < CH; ++i) h[k][i] = d[k][i] = 0.f;
            if (c < a.D) {
                load_row<CH>(static_cast<const TI*>(a.x) + o + c, h[k], a.D - c, vec);
                load_row<CH>(static_cast<const TI*>(a.dy) + o + c, d[k], a.D - c, vec);
            }
        }
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                ss = fmaf(h[k][i], h[k][i], ss);
                dot = fmaf(h[k][i] * w[k][i], d[k][i], dot);
            }
        ss = cta_reduce<NT, false>(ss, buf);
        dot = cta_reduce<NT, false>(dot, buf);
        const float r = 1.f / sqrtf(ss / (float)a.D + a.eps);
        const float m = dot * r * r / (float)a.D;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = col_of<NT, CH>(k);
            float g[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) g[i] = 0.f;
            if (c < a.D && a.dres) load_row<CH>(static_cast<const TI*>(a.dres) + o + c, g, a.D - c, vec);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                dw[k][i] = fmaf(d[k][i], h[k][i] * r, dw[k][i]);
                g[i] = fmaf(r, fmaf(w[k][i], d[k][i], -h[k][i] * m), g[i]);
            }
            if (c < a.D) store_row<CH>(static_cast<TI*>(a.dx) + o + c, g, a.D - c, vec);
        }
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = col_of<NT, CH>(k);
        if (c < a.D) store_row<CH>(a.part + (size_t)blockIdx.x * a.D + c, dw[k], a.D - c, vec);
    }
}

// dweight: the CTAs' sums in order.
__global__ void k_norm_sum(NormArgs a) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= a.D) return;
    float s = 0.f;
    for (int p = 0; p < a.parts; ++p) s += a.part[(size_t)p * a.D + d];
    a.dweight[d] = s;
}

template <typename TI, int NT, int NC, int CH, bool BWD>
void run_one(const NormArgs& a, int vec, cudaStream_t st) {
    if (BWD) k_norm_bwd<TI, NT, NC, CH><<<a.parts, NT, 0, st>>>(a, vec);
    else if (a.out) k_norm_fwd<TI, NT, NC, CH, true><<<a.rows, NT, 0, st>>>(a, vec);
    else k_norm_fwd<TI, NT, NC, CH, false><<<a.rows, NT, 0, st>>>(a, vec);
}

// Threads and elements per thread by the row's width.
template <typename TI, int CH, bool BWD>
void run_width(const NormArgs& a, int vec, cudaStream_t st) {
    if (a.D <= 256) run_one<TI, 32, 8 / CH, CH, BWD>(a, vec, st);
    else if (a.D <= 1024) run_one<TI, 128, 8 / CH, CH, BWD>(a, vec, st);
    else if (a.D <= 2048) run_one<TI, 256, 8 / CH, CH, BWD>(a, vec, st);
    else if (a.D <= 4096) run_one<TI, 256, 16 / CH, CH, BWD>(a, vec, st);
    else if (a.D <= 8192) run_one<TI, 512, 16 / CH, CH, BWD>(a, vec, st);
    else run_one<TI, 1024, 16 / CH, CH, BWD>(a, vec, st);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

int norm_bwd_parts(int rows) { return rows < 2 * sm_count() ? (rows > 0 ? rows : 1) : 2 * sm_count(); }

cudaError_t launch_norm_fwd(const NormArgs& a, int bf16, cudaStream_t st) {
    const int vec = a.D % 8 == 0 && aligned16(a.x) && aligned16(a.residual) && aligned16(a.weight) && aligned16(a.y) &&
                    aligned16(a.h);
    return traced_launch("k_norm_fwd", st, [&] {
        // an 8-bit output packs 8 columns per thread and forms its groups' maxima over them
        if (vec || a.out) bf16 ? run_width<__nv_bfloat16, 8, false>(a, vec, st) : run_width<float, 8, false>(a, vec, st);
        else bf16 ? run_width<__nv_bfloat16, 1, false>(a, 0, st) : run_width<float, 1, false>(a, 0, st);
    });
}

cudaError_t launch_norm_bwd(const NormArgs& a, int bf16, cudaStream_t st) {
    const int vec = a.D % 8 == 0 && aligned16(a.x) && aligned16(a.dy) && aligned16(a.weight) && aligned16(a.dres) &&
                    aligned16(a.dx);
    cudaError_t e = traced_launch("k_norm_bwd", st, [&] {
        if (vec) bf16 ? run_width<__nv_bfloat16, 8, true>(a, vec, st) : run_width<float, 8, true>(a, vec, st);
        else bf16 ? run_width<__nv_bfloat16, 1, true>(a, 0, st) : run_width<float, 1, true>(a, 0, st);
    });
    if (e != cudaSuccess) return e;
    return traced_launch("k_norm_sum", st, [&] { k_norm_sum<<<(a.D + 127) / 128, 128, 0, st>>>(a); });
}

}  // namespace kda
