// Linear attention with a decay for each head on CUDA cores: every type, width and alignment, and single tokens.
// A CTA holds a head's state (K rows x a slice of value columns) in registers, each warp a block of rows, and takes the
// tokens in groups of TG. With S the state entering a group of n tokens and a its decay, for its token i (forwards)
//     o_i = s (a^(i+1) q_i S + sum_{j<=i} a^(i-j) w (q_i k_j) v_j),   S <- a^n S + sum_j w a^(n-1-j) k_j v_j^T
// (backwards: a^i, and a^(n-j)). The state is rounded once per group instead of once per token, and a token costs two
// multiply-adds per state element instead of four.
// Sums are fp32; the outputs are rounded once.
#include "kda_lin.cuh"

namespace kda {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int NT = 256, NW = NT / 32;

template <typename TI>
__device__ __forceinline__ float as_float(TI x);
template <>
__device__ __forceinline__ float as_float(float x) { return x; }
template <>
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// KR rows of the state per warp (K <= 8 KR), VEC neighbouring value columns per lane, TG tokens per group.
template <typename TI, int KR, int VEC, int TG>
__global__ void __launch_bounds__(NT) k_lin(LinArgs a, int local) {
    constexpr int KM = NW * KR, SL = 32 * VEC;
    const LinCall& c = a.c[blockIdx.y];
    const int slices = (c.V + SL - 1) / SL;
    int at = blockIdx.x;
    const int slice = at % slices;
    at /= slices;
    const int h = at % a.HV;
    const int unit = at / a.HV;
    if (unit >= a.ax.rows * a.units_row) return;
    const int row = unit / a.units_row, u = unit - row * a.units_row;

    __shared__ __align__(16) float sq[TG][KM], sk[TG][KM], sv[TG][SL], part[TG][NW][SL];
    __shared__ float P[TG][TG];
    __shared__ float2 pw[TG + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k0 = warp * KR;
    const int v0 = slice * SL, vl = v0 + lane * VEC;       // this lane's columns
    const int t0 = u * a.unit_len, t1 = min(a.ax.len, t0 + a.unit_len);
    const float g = a.decay ? a.decay[h] : 0.f;
    const size_t KV = (size_t)c.K * c.V;
    if (blockIdx.x == 0 && blockIdx.y == 0 && !local) axis_check(a.ax, a.err);

    float S[KR][VEC];
    // One access per row where the columns lie side by side and start on the access's size.
    const bool vec = VEC > 1 && c.V % VEC == 0 && !c.transposed &&
                     ((reinterpret_cast<uintptr_t>(c.s0) | reinterpret_cast<uintptr_t>(c.s1)) & (4 * VEC - 1)) == 0;
    const size_t rk = c.transposed ? 1 : c.V, rv = c.transposed ? c.K : 1;
    auto load_state = [&](const float* p, bool wide, size_t dk, size_t dv) {
#pragma unroll
        for (int r = 0; r < KR; ++r) {
            if (k0 + r < c.K && vl < c.V) {
                const float* x = p + (k0 + r) * dk + vl * dv;
                if (VEC > 1 && wide) {
                    const Raw<float, VEC> y = load_raw<float, VEC>(x);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) S[r][i] = y.v[i];
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) S[r][i] = vl + i < c.V ? x[i * dv] : 0.f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) S[r][i] = 0.f;
            }
        }
    };
    auto store_state = [&](float* p, bool wide) {
#pragma unroll
        for (int r = 0; r < KR; ++r) {
            if (k0 + r >= c.K || vl >= c.V) continue;
            float* x = p + (size_t)(k0 + r) * c.V + vl;
            if (VEC > 1 && wide) {
                store_values<VEC>(x, S[r]);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (vl + i < c.V) x[i] = S[r][i];
            }
        }
    };
    // The state that sequence n starts from.
    auto start_state = [&](int n) {
        if (c.s0) {
            load_state(c.s0 + ((size_t)n * a.HV + h) * KV, vec, rk, rv);
        } else {
#pragma unroll
            for (int r = 0; r < KR; ++r)
#pragma unroll
                for (int i = 0; i < VEC; ++i) S[r][i] = 0.f;
        }
    };

    // final states of sequences without tokens
    if (u == 0 && !local && c.s1) {
        if (!a.ax.cu) {
            if (a.ax.len == 0) {
                start_state(row);
                store_state(c.s1 + ((size_t)row * a.HV + h) * KV, vec);
            }
        } else {
            for (int n = 0; n < a.ax.N; ++n) {
                if (axis_cu(a.ax, n + 1) > axis_cu(a.ax, n)) continue;
                start_state(n);
                store_state(c.s1 + ((size_t)n * a.HV + h) * KV, vec);
            }
        }
    }
    if (t0 >= t1) return;

    int t = t0;
    Seq s;
    if (local) {   // only the sequence that goes on behind the window
        s = lin_seq(a.ax, row, t1 - 1, c.back);
        if (s.end <= t1) return;
        t = max(t0, s.first);
    } else {
        s = lin_seq(a.ax, row, t, c.back);
    }
    bool first = true;
    while (t < t1) {
        const int end = min(s.end, t1);
        if (local) {
#pragma unroll
            for (int r = 0; r < KR; ++r)
#pragma unroll
                for (int i = 0; i < VEC; ++i) S[r][i] = 0.f;
        } else {
            start_state(s.n);
            if (s.first < t) {   // it came through earlier windows
                for (int e = s.first / a.unit_len; e < u; ++e) {
                    const float f = lin_power(g, (e + 1) * a.unit_len - max(s.first, e * a.unit_len));
                    const float* p = c.local + ((size_t)(unit - u + e) * a.HV + h) * KV;
#pragma unroll
                    for (int r = 0; r < KR; ++r)
#pragma unroll
                        for (int i = 0; i < VEC; ++i)
                            if (k0 + r < c.K && vl + i < c.V) S[r][i] = fmaf(S[r][i], f, p[(size_t)(k0 + r) * c.V + vl + i]);
                }
            }
        }
        if (first && warp == NW - 1 && lane <= TG) pw[lane] = lin_power2(g, lane);
        first = false;
        for (; t < end; t += TG) {
            const int n = min(TG, end - t);
            __syncthreads();   // the last group's readers are done
            for (int x = threadIdx.x; x < n * KM; x += NT) {
                const int i = x / KM, d = x - i * KM;
                const size_t tok = (size_t)row * a.ax.len + (c.back ? a.ax.len - 1 - (t + i) : t + i);
                sk[i][d] = d < c.K ? as_float(static_cast<const TI*>(c.k)[tok * c.ldk + (size_t)(h / c.gk) * c.K + d]) : 0.f;
                if (!local) sq[i][d] = d < c.K ? as_float(static_cast<const TI*>(c.q)[tok * c.ldq + (size_t)(h / c.gq) * c.K + d]) : 0.f;
            }
            for (int x = threadIdx.x; x < n * SL; x += NT) {
                const int i = x / SL, d = x - i * SL;
                const size_t tok = (size_t)row * a.ax.len + (c.back ? a.ax.len - 1 - (t + i) : t + i);
                sv[i][d] = v0 + d < c.V ? as_float(static_cast<const TI*>(c.v)[tok * c.ldv + (size_t)(h / c.gv) * c.V + v0 + d]) : 0.f;
            }
            __syncthreads();
            if (!local) {
                for (int x = warp; x < n * n; x += NW) {
                    const int i = x / n, j = x - i * n;
                    if (j > i) continue;
                    float d = 0.f;
                    for (int y = lane; y < c.K; y += 32) d = fmaf(sq[i][y], sk[j][y], d);
#pragma unroll
                    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(FULL, d, o);
                    if (lane == 0) P[i][j] = d * pw[i - j].x * (c.s * c.w);
                }
#pragma unroll
                for (int i = 0; i < TG; ++i) {
                    if (i >= n) break;
                    float o[VEC];
#pragma unroll
                    for (int y = 0; y < VEC; ++y) o[y] = 0.f;
#pragma unroll
                    for (int r = 0; r < KR; r += 4) {
                        const float4 qv = *reinterpret_cast<const float4*>(&sq[i][k0 + r]);
                        const float qa[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
                        for (int z = 0; z < 4; ++z)
#pragma unroll
                            for (int y = 0; y < VEC; ++y) o[y] = fmaf(qa[z], S[r + z][y], o[y]);
                    }
#pragma unroll
                    for (int y = 0; y < VEC; ++y) part[i][warp][lane * VEC + y] = o[y];
                }
            }
            // the state behind the group
            const float2 an = pw[n];
#pragma unroll
            for (int r = 0; r < KR; ++r)
#pragma unroll
                for (int y = 0; y < VEC; ++y) S[r][y] = an.x == 1.f ? S[r][y] : fmaf(S[r][y], an.x, S[r][y] * an.y);
#pragma unroll
            for (int j = 0; j < TG; ++j) {
                if (j >= n) break;
                const float e = c.w * pw[c.back ? n - j : n - 1 - j].x;
                float vj[VEC];
#pragma unroll
                for (int y = 0; y < VEC; ++y) vj[y] = e * sv[j][lane * VEC + y];
#pragma unroll
                for (int r = 0; r < KR; r += 4) {
                    const float4 kv = *reinterpret_cast<const float4*>(&sk[j][k0 + r]);
                    const float ka[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
                    for (int z = 0; z < 4; ++z)
#pragma unroll
                        for (int y = 0; y < VEC; ++y) S[r + z][y] = fmaf(ka[z], vj[y], S[r + z][y]);
                }
            }
            if (local) continue;
            __syncthreads();
            for (int x = threadIdx.x; x < n * SL; x += NT) {
                const int i = x / SL, d = x - i * SL;
                if (v0 + d >= c.V) continue;
                float o = 0.f;
#pragma unroll
                for (int y = 0; y < NW; ++y) o += part[i][y][d];
                o *= c.s * pw[c.back ? i : i + 1].x;
                for (int j = 0; j <= i; ++j) o = fmaf(P[i][j], sv[j][d], o);
                const size_t tok = (size_t)row * a.ax.len + (c.back ? a.ax.len - 1 - (t + i) : t + i);
                const size_t to = (tok * a.HV + h) * c.V + v0 + d;
                if (c.o_f32) static_cast<float*>(c.o)[to] = o;
                else static_cast<TI*>(c.o)[to] = TI(o);
            }
        }
        t = end;
        if (local) {
            store_state(c.local + ((size_t)unit * a.HV + h) * KV, VEC > 1 && c.V % VEC == 0);
            return;
        }
        if (end == s.end && c.s1) store_state(c.s1 + ((size_t)s.n * a.HV + h) * KV, vec);
        if (t < t1) s = lin_seq(a.ax, row, t, c.back);
    }
}

template <typename TI, int KR, int VEC, int TG>
cudaError_t run(const LinArgs& a, cudaStream_t st) {
    int vmax = 1;
    for (int i = 0; i < a.calls; ++i) vmax = a.c[i].V > vmax ? a.c[i].V : vmax;
    const long long ctas = (long long)a.ax.rows * a.units_row * a.HV * ((vmax + 32 * VEC - 1) / (32 * VEC));
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)ctas, a.calls);
    if (a.units_row > 1) {
        const cudaError_t e = traced_launch("k_lin_windows", st, [&] { k_lin<TI, KR, VEC, TG><<<grid, NT, 0, st>>>(a, 1); });
        if (e != cudaSuccess) return e;
    }
    return traced_launch("k_lin", st, [&] { k_lin<TI, KR, VEC, TG><<<grid, NT, 0, st>>>(a, 0); });
}

template <typename TI>
cudaError_t pick(const LinArgs& a, cudaStream_t st) {
    int kmax = 1, vmax = 1;
    for (int i = 0; i < a.calls; ++i) {
        kmax = a.c[i].K > kmax ? a.c[i].K : kmax;
        vmax = a.c[i].V > vmax ? a.c[i].V : vmax;
    }
    if (kmax <= 64) return vmax <= 64 ? run<TI, 8, 2, 8>(a, st) : run<TI, 8, 4, 8>(a, st);
    if (kmax <= 128) return vmax <= 64 ? run<TI, 16, 2, 8>(a, st) : run<TI, 16, 4, 8>(a, st);
    return run<TI, 32, 2, 4>(a, st);
}

template <typename TI>
__global__ void __launch_bounds__(256) k_lin_heads(const float* part, TI* out, int64_t n, int group, int width) {
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (x >= n) return;
    const int64_t row = x / width;
    const int d = (int)(x - row * width);
    float s = 0.f;
    for (int i = 0; i < group; ++i) s += part[(row * group + i) * width + d];
    out[x] = TI(s);
}

}  // namespace

// Windows per row: as many as keep `ctas` per window below two CTAs on each SM, of 64 tokens at least.
int lin_units(int rows, int len, int ctas) {
    const long long all = (long long)rows * ctas;
    int n = (int)(2LL * sm_count() / (all > 0 ? all : 1));
    if (n > len / 64) n = len / 64;
    return n > 1 ? n : 1;
}

cudaError_t launch_lin(const LinArgs& a, int bf16, cudaStream_t st) {
    return bf16 ? pick<__nv_bfloat16>(a, st) : pick<float>(a, st);
}

cudaError_t launch_lin_heads(const float* part, void* out, int64_t rows, int group, int width, int bf16, cudaStream_t st) {
    const int64_t n = rows * width, blocks = (n + 255) / 256;
    if (n == 0) return cudaSuccess;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return traced_launch("k_lin_heads", st, [&] {
        if (bf16) k_lin_heads<<<(unsigned)blocks, 256, 0, st>>>(part, static_cast<__nv_bfloat16*>(out), n, group, width);
        else k_lin_heads<<<(unsigned)blocks, 256, 0, st>>>(part, static_cast<float*>(out), n, group, width);
    });
}

}  // namespace kda
