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
// Bound by HBM, 16384 rows of 4096, bf16: forward with residual and e4m3 output 82 us,
// 5.7 TB/s (85% of the copy rate; 1024 threads per SM at 64 registers: at 72 registers
// three CTAs per SM instead of four, 118 us); backward 101 us, 5.3 TB/s (78%). Sums and
// the row are fp32 throughout.
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
    static_assert(K == 1 || (K == 2 && !MAX), "one value, or two sums");
    const int lane = threadIdx.x & 31;
    float v0 = x[0];
    if (K == 2) {   // each half of the warp goes on with one of the sums
        const float send = lane & 16 ? x[0] : x[K - 1];
        v0 = (lane & 16 ? x[K - 1] : x[0]) + __shfl_xor_sync(FULL, send, 16);
    }
#pragma unroll
    for (int o = K == 2 ? 8 : 16; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(FULL, v0, o);
        v0 = MAX ? amax(v0, y) : v0 + y;
    }
    if (NT == 32) {
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] = K == 2 ? __shfl_sync(FULL, v0, 16 * k) : v0;
        return;
    }
    float(*b)[NT / 32] = buf[turn & 1];
    if ((lane & (K == 2 ? 15 : 31)) == 0) b[lane >> 4][threadIdx.x >> 5] = v0;
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
            if (!(m[k] >= 1e-30f && m[k] <= 1e30f)) {
                // 448 / m may overflow, or m be above 2^126, where the fast division gives 0: such a group is brought to
                // the middle of the range first
                const float by = m[k] < 1.f ? 0x1p64f : 0x1p-64f;
                m[k] *= by;
#pragma unroll
                for (int i = 0; i < CH; ++i) h[k][i] *= by;
            }
            // The fast division's two units do not show: of 2e8 values (bf16, 4096 columns) 125 are not the nearest 8-bit
            // ones, 112 with a correctly rounded one, 135 in elementary fp32 operations; its registers would leave three
            // CTAs of four on an SM (82 against 122 us).
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

// Rows on their way of the backward: a thread's chunks of h, dy and dres, `STAGES` rows in a ring in shared memory
// copied asynchronously (chunks of 8), or one row ahead in registers (single columns).
template <typename TI, int NT, int NC, int CH>
struct Rows {
    static constexpr bool ASYNC = CH > 1;
    static constexpr int ROW = 3 * NC * NT * CH * (int)sizeof(TI);
    static constexpr int STAGES = ROW <= 72 * 1024 ? 3 : ROW <= 100 * 1024 ? 2 : 1;   // 216 KB at most
    static constexpr int BYTES = ASYNC ? STAGES * ROW : 0;
    using C = Chunk<TI, CH>;
    C next[ASYNC ? 1 : 3][ASYNC ? 1 : NC];
    __device__ __forceinline__ static C* place(void* smem, int stage, int which, int k) {
        return static_cast<C*>(smem) + ((stage * 3 + which) * NC + k) * NT + threadIdx.x;
    }
    __device__ __forceinline__ void fetch(const NormArgs& a, void* smem, int rw, int stage) {
        if (rw < a.rows) {
            const TI* src[3] = {static_cast<const TI*>(a.x), static_cast<const TI*>(a.dy), static_cast<const TI*>(a.dres)};
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                if (!src[q]) continue;
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const int c = col_of<NT, CH>(k);
                    if (c >= a.D) continue;
                    const TI* p = src[q] + (size_t)rw * a.D + c;
                    if constexpr (ASYNC) {
#pragma unroll
                        for (int i = 0; i < (int)sizeof(C) / 16; ++i)
                            copy_async(reinterpret_cast<uint4*>(place(smem, stage, q, k)) + i, reinterpret_cast<const uint4*>(p) + i);
                    } else {
                        next[q][k].load(p, a.D - c, false);
                    }
                }
            }
        }
        copies_commit();
    }
    __device__ __forceinline__ void get(void* smem, int stage, int which, int k, float (&x)[CH]) const {
        if constexpr (ASYNC) unpack<CH>(place(smem, stage, which, k)->r, x);
        else unpack<CH>(next[which][k].r, x);
    }
};

// CTA p takes rows p, p + parts, ...; each thread keeps its columns' dw sums.
template <typename TI, int NT, int NC, int CH>
__global__ void __launch_bounds__(NT, NT == 256 && CH > 1 && sizeof(TI) == 2 ? 3 : 1) k_norm_bwd(NormArgs a) {
    using R = Rows<TI, NT, NC, CH>;
    constexpr int AHEAD = R::ASYNC ? R::STAGES - 1 : 1;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ __align__(16) float buf[2][2][NT / 32];
    const float inv_d = 1.f / (float)a.D;
    R rows;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) rows.fetch(a, ring, blockIdx.x + i * a.parts, i);
    float w[NC][CH], dw[NC][CH];
    load_weight<NT, NC, CH>(a, CH > 1, w);
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < CH; ++i) dw[k][i] = 0.f;
    int stage = 0;
    for (int rw = blockIdx.x, turn = 0; rw < a.rows; rw += a.parts, ++turn) {
        if (R::ASYNC) {   // the row after those in flight goes where the previous row lay
            rows.fetch(a, ring, rw + AHEAD * a.parts, stage == 0 ? R::STAGES - 1 : stage - 1);
            copies_wait<R::STAGES - 1>();
        }
        float h[NC][CH], d[NC][CH], g[R::ASYNC ? 1 : NC][CH];
        float sums[2] = {0.f, 0.f};   // h h, h w dy
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            if (col_of<NT, CH>(k) >= a.D) continue;
            rows.get(ring, stage, 0, k, h[k]);
            rows.get(ring, stage, 1, k, d[k]);
            if (!R::ASYNC) rows.get(ring, stage, 2, k, g[R::ASYNC ? 0 : k]);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                sums[0] = fmaf(h[k][i], h[k][i], sums[0]);
                sums[1] = fmaf(h[k][i] * w[k][i], d[k][i], sums[1]);
            }
        }
        if (!R::ASYNC) rows.fetch(a, ring, rw + a.parts, 0);
        cta_reduce<NT, 2, false>(sums, buf, turn);
        // correctly rounded: for rows of a few columns the two parts of dx all but cancel
        const float r = 1.f / sqrtf(fmaf(sums[0], inv_d, a.eps));
        const float m = sums[1] * inv_d * r * r;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = col_of<NT, CH>(k);
            if (c >= a.D) continue;
            float o[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) o[i] = 0.f;
            if (a.dres) {
                if constexpr (R::ASYNC) {
                    rows.get(ring, stage, 2, k, o);
                } else {
#pragma unroll
                    for (int i = 0; i < CH; ++i) o[i] = g[k][i];
                }
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                dw[k][i] = fmaf(d[k][i], h[k][i] * r, dw[k][i]);
                o[i] = fmaf(r, fmaf(w[k][i], d[k][i], -h[k][i] * m), o[i]);
            }
            store_row<CH>(static_cast<TI*>(a.dx) + (size_t)rw * a.D + c, o, a.D - c, CH > 1);
        }
        stage = stage + 1 == R::STAGES ? 0 : stage + 1;
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = col_of<NT, CH>(k);
        if (c < a.D) store_row<CH>(a.part + (size_t)blockIdx.x * a.D + c, dw[k], a.D - c, CH > 1);
    }
}

// dweight: the CTAs' sums in order.
__global__ void __launch_bounds__(256) k_norm_sum(NormArgs a) {
    float sum;
    const int d = sum_parts(a.part, a.parts, a.D, sum);
    if (d >= 0) a.dweight[d] = sum;
}

template <typename TI, int NT, int NC, int CH, bool BWD>
cudaError_t run_one(NormArgs a, int vec, cudaStream_t st) {
    if constexpr (BWD) {
        constexpr int smem = Rows<TI, NT, NC, CH>::BYTES;
        static SmemLimit limit;
        const cudaError_t e = limit.set(reinterpret_cast<const void*>(k_norm_bwd<TI, NT, NC, CH>), smem);
        if (e != cudaSuccess) return e;
        k_norm_bwd<TI, NT, NC, CH><<<a.parts, NT, smem, st>>>(a);
    } else {
        // as many CTAs as are resident together, about 1024 threads per SM
        const int most = sm_count() * (NT >= 1024 ? 1 : 1024 / NT < 16 ? 1024 / NT : 16);
        a.parts = a.rows < most ? a.rows : most;
        if constexpr (CH > 1) {   // an 8-bit output takes chunks at every width
            if (a.out) {
                k_norm_fwd<TI, NT, NC, CH, true><<<a.parts, NT, 0, st>>>(a, vec);
                return cudaSuccess;
            }
        }
        k_norm_fwd<TI, NT, NC, CH, false><<<a.parts, NT, 0, st>>>(a, vec);
    }
    return cudaSuccess;
}

// Threads and elements per thread by the row's width, so that about 1024 threads of an SM share its rows. Measured forward,
// 16384 rows, bf16, e4m3 output, taken against the other side: D = 256 with 32 threads 6.2 us against 11.6 with 128; 2048
// with 256 x 8 42.3 against 56.9 with 128 x 16; 4096 with 256 x 16 80.5 against 82.4 with 512 x 8; 8192 with 1024 x 8 175
// against 234 with 512 x 16, 5120 150 against 212, 6144 158 against 217, 7168 166 against 226.
template <typename TI, int CH, bool BWD>
cudaError_t run_width(const NormArgs& a, int vec, cudaStream_t st) {
    if (a.D <= 256) return run_one<TI, 32, 8 / CH, CH, BWD>(a, vec, st);
    if (a.D <= 1024) return run_one<TI, 128, 8 / CH, CH, BWD>(a, vec, st);
    if (a.D <= 2048) return run_one<TI, 256, 8 / CH, CH, BWD>(a, vec, st);
    if (a.D <= 4096) return run_one<TI, 256, 16 / CH, CH, BWD>(a, vec, st);
    // (the forward's registers leave only one CTA of 512 threads on an SM)
    if (a.D <= 8192) return run_one<TI, BWD ? 512 : 1024, (BWD ? 16 : 8) / CH, CH, BWD>(a, vec, st);
    return run_one<TI, 1024, 16 / CH, CH, BWD>(a, vec, st);
}
template <bool BWD>
cudaError_t run_norm(const char* name, const NormArgs& a, int bf16, bool chunks, int vec, cudaStream_t st) {
    cudaError_t r = cudaSuccess;
    const cudaError_t e = traced_launch(name, st, [&] {
        if (chunks) r = bf16 ? run_width<__nv_bfloat16, 8, BWD>(a, vec, st) : run_width<float, 8, BWD>(a, vec, st);
        else r = bf16 ? run_width<__nv_bfloat16, 1, BWD>(a, 0, st) : run_width<float, 1, BWD>(a, 0, st);
    });
    return r != cudaSuccess ? r : e;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

int norm_bwd_parts(int rows, int D) {
    // the CTAs resident together: about 768 threads per SM
    const int nt = D <= 256 ? 32 : D <= 1024 ? 128 : D <= 4096 ? 256 : D <= 8192 ? 512 : 1024;
    const int most = sm_count() * (nt >= 512 ? 1 : nt == 32 ? 8 : 768 / nt);
    return rows < most ? (rows > 0 ? rows : 1) : most;
}

cudaError_t launch_norm_fwd(const NormArgs& a, int bf16, cudaStream_t st) {
    const int vec = a.D % 8 == 0 && aligned16(a.x) && aligned16(a.residual) && aligned16(a.weight) && aligned16(a.y) &&
                    aligned16(a.h);
    // an 8-bit output packs 8 columns per thread and forms its groups' maxima over them
    return run_norm<false>("k_norm_fwd", a, bf16, vec || a.out, vec, st);
}

cudaError_t launch_norm_bwd(const NormArgs& a, int bf16, cudaStream_t st) {
    const int vec = a.D % 8 == 0 && aligned16(a.x) && aligned16(a.dy) && aligned16(a.weight) && aligned16(a.dres) &&
                    aligned16(a.dx);
    const cudaError_t e = run_norm<true>("k_norm_bwd", a, bf16, vec, vec, st);
    if (e != cudaSuccess) return e;
    return traced_launch("k_norm_sum", st, [&] { k_norm_sum<<<(a.D + 31) / 32, 256, 0, st>>>(a); });
}

}  // namespace kda
