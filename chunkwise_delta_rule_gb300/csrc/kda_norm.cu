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
// A CTA holds a row in registers, so each tensor is read once; it walks rows with the
// weight (and its gradient's sums) kept in registers and the next row's loads in
// flight while the present row is summed and written.
#include <cuda_fp8.h>

#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr float E4M3_MAX = 448.f;

// The larger of a and |b|; a NaN stays.
__device__ __forceinline__ float amax(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

// K sums (or one NaN-keeping maximum) over the CTA's NT threads; every thread gets them. buf alternates between two
// halves by `turn`, so that one barrier per call is enough.
template <int NT, int K, bool MAX>
__device__ __forceinline__ void cta_reduce(float (&x)[K], float (*buf)[K][NT / 32], int turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float y = __shfl_xor_sync(FULL, x[k], o);
            x[k] = MAX ? amax(x[k], y) : x[k] + y;
        }
    if (NT == 32) return;
    float(*b)[NT / 32] = buf[turn & 1];
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) b[k][threadIdx.x >> 5] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float v[NT / 32];
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) v[i] = b[k][i];
#pragma unroll
        for (int n = NT / 64; n > 0; n /= 2)
#pragma unroll
            for (int i = 0; i < n; ++i) v[i] = MAX ? amax(v[i], v[i + n]) : v[i] + v[i + n];
        x[k] = v[0];
    }
}

// A chunk of CH columns as it lies in memory: 16-byte accesses, or element by element up to `valid`.
template <typename TI, int CH>
struct Chunk {
    Raw<TI, CH> r;
    __device__ __forceinline__ void load(const TI* p, int valid, bool vec) {
        if (CH > 1 && vec) {
            constexpr int N = sizeof(TI) * CH / 16 > 0 ? sizeof(TI) * CH / 16 : 1;
#pragma unroll
            for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(&r)[i] = reinterpret_cast<const uint4*>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) r.v[i] = i < valid ? p[i] : TI(0.f);
        }
    }
};

// Columns of chunk k of a thread: chunks of 8 (CH = 8), or single columns side by side (CH = 1) for rows whose
// width is no multiple of 8, which keeps a warp's accesses together.
template <int NT, int CH>
__device__ __forceinline__ int col_of(int k) { return (k * NT + threadIdx.x) * CH; }

template <int NT, int NC, int CH>
__device__ __forceinline__ void load_weight(const NormArgs& a, bool vec, float (&w)[NC][CH]) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = col_of<NT, CH>(k);
#pragma unroll
        for (int i = 0; i < CH; ++i) w[k][i] = 0.f;
        if (c < a.D) load_row<CH>(a.weight + c, w[k], a.D - c, CH > 1 && vec);
    }
}

// CTA p of NT threads takes rows p, p + parts, ...; NC chunks per thread.
template <typename TI, int NT, int NC, int CH, bool Q8>
__global__ void __launch_bounds__(NT) k_norm_fwd(NormArgs a, int vec) {
    __shared__ __align__(16) float buf[2][1][NT / 32], bufm[2][1][NT / 32];
    Chunk<TI, CH> nx[NC], nr[NC];
    auto fetch = [&](int rw) {
        const size_t o = (size_t)rw * a.D;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = col_of<NT, CH>(k);
            if (c >= a.D) continue;
            nx[k].load(static_cast<const TI*>(a.x) + o + c, a.D - c, vec);
            if (a.residual) nr[k].load(static_cast<const TI*>(a.residual) + o + c, a.D - c, vec);
        }
    };
    fetch(blockIdx.x);
    const float inv_d = 1.f / (float)a.D;
    float w[NC][CH];
    load_weight<NT, NC, CH>(a, vec, w);
    for (int rw = blockIdx.x, turn = 0; rw < a.rows; rw += a.parts, ++turn) {
        const size_t o = (size_t)rw * a.D;
        float h[NC][CH], ss[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = col_of<NT, CH>(k);
            if (c < a.D) {
                unpack<CH>(nx[k].r, h[k]);
                if (a.residual) {
                    float r[CH];
                    unpack<CH>(nr[k].r, r);
#pragma unroll
                    for (int i = 0; i < CH; ++i) h[k][i] += r[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < CH; ++i) h[k][i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) ss[0] = fmaf(h[k][i], h[k][i], ss[0]);
        }
        if (rw + a.parts < a.rows) fetch(rw + a.parts);
        if (a.residual) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const int c = col_of<NT, CH>(k);
                if (c < a.D) store_row<CH>(static_cast<TI*>(a.h) + o + c, h[k], a.D - c, CH > 1 && vec);
            }
        }
        cta_reduce<NT, 1, false>(ss, buf, turn);
        const float r = rsqrtf(fmaf(ss[0], inv_d, a.eps));
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < CH; ++i) h[k][i] *= r * w[k][i];
        if (!Q8) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const int c = col_of<NT, CH>(k);
                if (c < a.D) store_row<CH>(static_cast<TI*>(a.y) + o + c, h[k], a.D - c, CH > 1 && vec);
            }
            continue;
        }
        float m[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) {   // columns past D are zero: their weight is
            m[k] = 0.f;
#pragma unroll
            for (int i = 0; i < CH; ++i) m[k] = amax(m[k], h[k][i]);
        }
        if (a.group) {
#pragma unroll
            for (int s = 64 / CH; s > 0; s >>= 1)
                if (a.group >= 2 * CH * s)
#pragma unroll
                    for (int k = 0; k < NC; ++k) m[k] = amax(m[k], __shfl_xor_sync(FULL, m[k], s));
        } else {
            float all[1] = {m[0]};
#pragma unroll
            for (int k = 1; k < NC; ++k) all[0] = amax(all[0], m[k]);
            cta_reduce<NT, 1, true>(all, bufm, turn);
#pragma unroll
            for (int k = 0; k < NC; ++k) m[k] = all[0];
        }
        uint8_t* q = static_cast<uint8_t*>(a.y) + o;
        float* sc = a.scale + (size_t)rw * a.ngroups;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = col_of<NT, CH>(k);
            if (c >= a.D) continue;
            if (a.group ? (c & (a.group - 1)) == 0 : c == 0) sc[a.group ? c >> (31 - __clz(a.group)) : 0] = m[k] * (1.f / E4M3_MAX);
            if (m[k] < 1e-30f) {   // 448 / m may overflow: such a group is brought up by 2^64 first
                m[k] *= 0x1p64f;
#pragma unroll
                for (int i = 0; i < CH; ++i) h[k][i] *= 0x1p64f;
            }
            const float inv = m[k] > 0.f ? __fdividef(E4M3_MAX, m[k]) : m[k];   // 0 and NaN as they are
            uint32_t out[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < CH; i += 2) {
                const float2 v = make_float2(h[k][i] * inv, h[k][CH > 1 ? i + 1 : 0] * inv);
                out[i >> 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3) << (8 * (i & 3));
            }
            if (vec) {
                *reinterpret_cast<uint2*>(q + c) = make_uint2(out[0], out[1]);
            } else {
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (c + i < a.D) q[c + i] = (uint8_t)(out[i >> 2] >> (8 * (i & 3)));
            }
        }
    }
}

// CTA p takes rows p, p + parts, ...; each thread keeps its columns' dw sums.
template <typename TI, int NT, int NC, int CH>
__global__ void __launch_bounds__(NT) k_norm_bwd(NormArgs a, int vec) {
    __shared__ __align__(16) float buf[2][2][NT / 32];
    const float inv_d = 1.f / (float)a.D;
    Chunk<TI, CH> nh[NC], nd[NC], ng[NC];
    auto fetch = [&](int rw) {
        const size_t o = (size_t)rw * a.D;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = col_of<NT, CH>(k);
            if (c >= a.D) continue;
            nh[k].load(static_cast<const TI*>(a.x) + o + c, a.D - c, vec);
            nd[k].load(static_cast<const TI*>(a.dy) + o + c, a.D - c, vec);
            if (a.dres) ng[k].load(static_cast<const TI*>(a.dres) + o + c, a.D - c, vec);
        }
    };
    if (blockIdx.x < a.rows) fetch(blockIdx.x);
    float w[NC][CH], dw[NC][CH];
    load_weight<NT, NC, CH>(a, vec, w);
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < CH; ++i) dw[k][i] = 0.f;
    for (int rw = blockIdx.x, turn = 0; rw < a.rows; rw += a.parts, ++turn) {
        const size_t o = (size_t)rw * a.D;
        Chunk<TI, CH> ch[NC], cd[NC], cg[NC];
        float sums[2] = {0.f, 0.f};   // h h, h w dy
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            if (col_of<NT, CH>(k) >= a.D) continue;
            ch[k] = nh[k];
            cd[k] = nd[k];
            cg[k] = ng[k];
            float h[CH], d[CH];
            unpack<CH>(ch[k].r, h);
            unpack<CH>(cd[k].r, d);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                sums[0] = fmaf(h[i], h[i], sums[0]);
                sums[1] = fmaf(h[i] * w[k][i], d[i], sums[1]);
            }
        }
        if (rw + a.parts < a.rows) fetch(rw + a.parts);
        cta_reduce<NT, 2, false>(sums, buf, turn);
        // correctly rounded: for rows of a few columns the two parts of dx all but cancel
        const float r = 1.f / sqrtf(fmaf(sums[0], inv_d, a.eps));
        const float m = sums[1] * inv_d * r * r;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = col_of<NT, CH>(k);
            if (c >= a.D) continue;
            float h[CH], d[CH], g[CH];
            unpack<CH>(ch[k].r, h);
            unpack<CH>(cd[k].r, d);
#pragma unroll
            for (int i = 0; i < CH; ++i) g[i] = 0.f;
            if (a.dres) unpack<CH>(cg[k].r, g);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                dw[k][i] = fmaf(d[i], h[i] * r, dw[k][i]);
                g[i] = fmaf(r, fmaf(w[k][i], d[i], -h[i] * m), g[i]);
            }
            store_row<CH>(static_cast<TI*>(a.dx) + o + c, g, a.D - c, CH > 1 && vec);
        }
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = col_of<NT, CH>(k);
        if (c < a.D) store_row<CH>(a.part + (size_t)blockIdx.x * a.D + c, dw[k], a.D - c, CH > 1 && vec);
    }
}

// dweight: the CTAs' sums in order.
__global__ void __launch_bounds__(256) k_norm_sum(NormArgs a) {
    float sum;
    const int d = sum_parts(a.part, a.parts, a.D, sum);
    if (d >= 0) a.dweight[d] = sum;
}

template <typename TI, int NT, int NC, int CH, bool BWD>
void run_one(NormArgs a, int vec, cudaStream_t st) {
    if constexpr (BWD) {
        k_norm_bwd<TI, NT, NC, CH><<<a.parts, NT, 0, st>>>(a, vec);
    } else {
        // as many CTAs as are resident together, about 1024 threads per SM
        const int most = sm_count() * (NT >= 1024 ? 1 : 1024 / NT < 16 ? 1024 / NT : 16);
        a.parts = a.rows < most ? a.rows : most;
        if (a.out) k_norm_fwd<TI, NT, NC, CH, true><<<a.parts, NT, 0, st>>>(a, vec);
        else k_norm_fwd<TI, NT, NC, CH, false><<<a.parts, NT, 0, st>>>(a, vec);
    }
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
    return traced_launch("k_norm_sum", st, [&] { k_norm_sum<<<(a.D + 31) / 32, 256, 0, st>>>(a); });
}

}  // namespace kda
