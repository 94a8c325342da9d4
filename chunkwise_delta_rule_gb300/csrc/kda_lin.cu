// Linear attention with a decay for each head on CUDA cores: every type, width and alignment, and single tokens.
// A CTA holds a head's state (K rows x a slice of value columns) in registers, each warp a block of rows, and takes the
// tokens in groups of TG. With S the state entering a group of n tokens and a its decay, for its token i (forwards)
//     o_i = s (a^(i+1) q_i S + sum_{j<=i} a^(i-j) w (q_i k_j) v_j),   S <- a^n S + sum_j w a^(n-1-j) k_j v_j^T
// (backwards: a^i, and a^(n-j)). The state is rounded once per group instead of once per token, and a token costs two
// multiply-adds per state element instead of four.
// Sums are fp32; the outputs are rounded once. Bound by the instructions around its multiply-adds: groups of 8 tokens pass
// three barriers, two CTAs to an SM (fp32, 3 x 777 tokens, 10 heads of 40 x 72, forward and backward: 438 us; 1002 before the
// groups' values were fetched ahead and the slices went by the widths, 484 before multiply-adds took pairs of rows and the
// windows filled whole rounds of the SMs).
// One token per sequence has a kernel of its own, k_lin_step: 64 sequences of 32 heads of 128 x 128 take 43.6 us, 6.2 TB/s
// (92% of the copy rate; 115 us through the group kernel).
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
__global__ void __launch_bounds__(NT, KR * VEC >= 64 ? 1 : 2) k_lin(LinArgs a, int local) {
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

    constexpr int LD = KM + 4;   // rows of q and k four words apart in the banks
    constexpr int NK = TG * KM / NT, NV = TG * SL / NT > 0 ? TG * SL / NT : 1;   // a thread's values of a group
    __shared__ __align__(16) float sq[TG][LD], sk[TG][LD], sv[TG][SL], part[TG][NW][SL];
    __shared__ __align__(16) float P[TG][TG];
    __shared__ float2 pw[TG + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k0 = warp * KR;
    const int v0 = slice * SL, vl = v0 + lane * VEC;       // this lane's columns
    const int t0 = u * a.unit_len, t1 = min(a.ax.len, t0 + a.unit_len);
    const float g = a.decay ? a.decay[h] : 0.f;
    const size_t KV = (size_t)c.K * c.V;
    if (blockIdx.x == 0 && blockIdx.y == 0 && !local) axis_check(a.ax, a.err);

    float2 S[KR / 2][VEC];   // two neighbouring rows each: a multiply-add takes a pair
    // One access per row where the columns lie side by side and start on the access's size.
    const bool vec = VEC > 1 && c.V % VEC == 0 && !c.transposed &&
                     ((reinterpret_cast<uintptr_t>(c.s0) | reinterpret_cast<uintptr_t>(c.s1)) & (4 * VEC - 1)) == 0;
    const size_t rk = c.transposed ? 1 : c.V, rv = c.transposed ? c.K : 1;
    auto load_state = [&](const float* p, bool wide, size_t dk, size_t dv) {
#pragma unroll
        for (int r = 0; r < KR; ++r) {
            float z[VEC];
            if (k0 + r < c.K && vl < c.V) {
                const float* x = p + (k0 + r) * dk + vl * dv;
                if (VEC > 1 && wide) {
                    const Raw<float, VEC> y = load_raw<float, VEC>(x);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) z[i] = y.v[i];
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) z[i] = vl + i < c.V ? x[i * dv] : 0.f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) z[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) (r & 1 ? S[r / 2][i].y : S[r / 2][i].x) = z[i];
        }
    };
    auto store_state = [&](float* p, bool wide) {
#pragma unroll
        for (int r = 0; r < KR; ++r) {
            if (k0 + r >= c.K || vl >= c.V) continue;
            float* x = p + (size_t)(k0 + r) * c.V + vl;
            float z[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) z[i] = r & 1 ? S[r / 2][i].y : S[r / 2][i].x;
            if (VEC > 1 && wide) {
                store_values<VEC>(x, z);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (vl + i < c.V) x[i] = z[i];
            }
        }
    };
    // The state that sequence n starts from.
    auto start_state = [&](int n) {
        if (c.s0) {
            load_state(c.s0 + ((size_t)n * a.HV + h) * KV, vec, rk, rv);
        } else {
#pragma unroll
            for (int r = 0; r < KR / 2; ++r)
#pragma unroll
                for (int i = 0; i < VEC; ++i) S[r][i] = make_float2(0.f, 0.f);
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
            for (int r = 0; r < KR / 2; ++r)
#pragma unroll
                for (int i = 0; i < VEC; ++i) S[r][i] = make_float2(0.f, 0.f);
        } else {
            // (in the first window nothing has, whatever inconsistent offsets say)
            if (first && u > 0 && s.first < t) load_state(c.local + ((size_t)(unit - 1) * a.HV + h) * KV, VEC > 1 && c.V % VEC == 0, c.V, 1);   // it came through earlier windows
            else start_state(s.n);
        }
        if (first && warp == NW - 1 && lane <= TG) pw[lane] = lin_power2(g, lane);
        first = false;
        // the next group's values are on their way while a group is worked on
        float nq[NK], nk[NK], nv[NV];
        auto fetch = [&](int at) {
            const int64_t base = (int64_t)row * a.ax.len;
#pragma unroll
            for (int x = 0; x < NK; ++x) {
                const int i = (threadIdx.x + x * NT) / KM, d = (threadIdx.x + x * NT) % KM;
                const bool on = at + i < end && d < c.K;
                const int64_t tok = base + (c.back ? a.ax.len - 1 - (at + i) : at + i);
                nk[x] = on ? as_float(static_cast<const TI*>(c.k)[tok * c.ldk + (int64_t)(h / c.gk) * c.K + d]) : 0.f;
                nq[x] = on && !local ? as_float(static_cast<const TI*>(c.q)[tok * c.ldq + (int64_t)(h / c.gq) * c.K + d]) : 0.f;
            }
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                const int i = (threadIdx.x + x * NT) / SL, d = (threadIdx.x + x * NT) % SL;
                const int64_t tok = base + (c.back ? a.ax.len - 1 - (at + i) : at + i);
                nv[x] = i < TG && at + i < end && v0 + d < c.V
                            ? as_float(static_cast<const TI*>(c.v)[tok * c.ldv + (int64_t)(h / c.gv) * c.V + v0 + d]) : 0.f;
            }
        };
        fetch(t);
        for (; t < end; t += TG) {
            const int n = min(TG, end - t);
            __syncthreads();   // the last group's readers are done
#pragma unroll
            for (int x = 0; x < NK; ++x) {
                const int i = (threadIdx.x + x * NT) / KM, d = (threadIdx.x + x * NT) % KM;
                sk[i][d] = nk[x];
                if (!local) sq[i][d] = nq[x];
            }
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                const int i = (threadIdx.x + x * NT) / SL, d = (threadIdx.x + x * NT) % SL;
                if (i < TG) sv[i][d] = nv[x];
            }
            __syncthreads();
            if (t + TG < end) fetch(t + TG);
            if (!local) {
                {   // the group's scores, four threads to a pair of tokens
                    const int pair = threadIdx.x >> 2, i = pair / TG, j = pair % TG, y0 = (threadIdx.x & 3) * 4;
                    float d = 0.f;
                    if (pair < TG * TG && j <= i && i < n) {
                        for (int y = y0; y < c.K; y += 16) {   // (the rows hold zeros behind K)
                            const float4 x = *reinterpret_cast<const float4*>(&sq[i][y]), z = *reinterpret_cast<const float4*>(&sk[j][y]);
                            d = fmaf(x.x, z.x, fmaf(x.y, z.y, fmaf(x.z, z.z, fmaf(x.w, z.w, d))));
                        }
                    }
                    d += __shfl_xor_sync(FULL, d, 1);
                    d += __shfl_xor_sync(FULL, d, 2);
                    if ((threadIdx.x & 3) == 0 && pair < TG * TG && j <= i && i < n) P[i][j] = d * pw[i - j].x * (c.s * c.w);
                }
#pragma unroll
                for (int i = 0; i < TG; ++i) {
                    if (i >= n) break;
                    float2 o[VEC];
#pragma unroll
                    for (int y = 0; y < VEC; ++y) o[y] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int r = 0; r < KR; r += 4) {
                        const float4 qv = *reinterpret_cast<const float4*>(&sq[i][k0 + r]);
#pragma unroll
                        for (int y = 0; y < VEC; ++y) o[y] = fma2(make_float2(qv.x, qv.y), S[r / 2][y], o[y]);
#pragma unroll
                        for (int y = 0; y < VEC; ++y) o[y] = fma2(make_float2(qv.z, qv.w), S[r / 2 + 1][y], o[y]);
                    }
#pragma unroll
                    for (int y = 0; y < VEC; ++y) part[i][warp][lane * VEC + y] = o[y].x + o[y].y;
                }
            }
            // the state behind the group
            const float2 an = pw[n];
            if (an.x != 1.f) {
#pragma unroll
                for (int r = 0; r < KR / 2; ++r)
#pragma unroll
                    for (int y = 0; y < VEC; ++y)
                        S[r][y] = fma2(S[r][y], make_float2(an.x, an.x), mul2(S[r][y], make_float2(an.y, an.y)));
            }
#pragma unroll
            for (int j = 0; j < TG; ++j) {
                if (j >= n) break;
                const float e = c.w * pw[c.back ? n - j : n - 1 - j].x;
                float2 vj[VEC];
#pragma unroll
                for (int y = 0; y < VEC; ++y) {
                    const float x = e * sv[j][lane * VEC + y];
                    vj[y] = make_float2(x, x);
                }
#pragma unroll
                for (int r = 0; r < KR; r += 4) {
                    const float4 kv = *reinterpret_cast<const float4*>(&sk[j][k0 + r]);
#pragma unroll
                    for (int y = 0; y < VEC; ++y) S[r / 2][y] = fma2(make_float2(kv.x, kv.y), vj[y], S[r / 2][y]);
#pragma unroll
                    for (int y = 0; y < VEC; ++y) S[r / 2 + 1][y] = fma2(make_float2(kv.z, kv.w), vj[y], S[r / 2 + 1][y]);
                }
            }
            if (local) continue;
            __syncthreads();
            const int d = threadIdx.x % SL;   // this thread's column, of every NT / SL-th token
            if (v0 + d >= c.V) continue;
            float vd[TG];
#pragma unroll
            for (int j = 0; j < TG; ++j) vd[j] = sv[j][d];
#pragma unroll
            for (int x = 0; x < TG * SL / NT; ++x) {
                const int i = x * (NT / SL) + threadIdx.x / SL;
                if (i >= n) break;
                float o = 0.f;
#pragma unroll
                for (int y = 0; y < NW; ++y) o += part[i][y][d];
                o *= c.s * pw[c.back ? i : i + 1].x;
#pragma unroll
                for (int j = 0; j < TG; j += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&P[i][j]);
                    if (j <= i) o = fmaf(f.x, vd[j], o);
                    if (j + 1 <= i) o = fmaf(f.y, vd[j + 1], o);
                    if (j + 2 <= i) o = fmaf(f.z, vd[j + 2], o);
                    if (j + 3 <= i) o = fmaf(f.w, vd[j + 3], o);
                }
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

// One token of every sequence: S <- a S + k v^T, o = s q S, each state read and written once, 16 bytes at a time. A CTA
// has a head's K rows of up to 128 columns, VL lanes to a row, NR rows to a thread, all of them requested before the
// token's own values are waited for. Bound by HBM.
template <typename TI, int VL, int NR>
__global__ void __launch_bounds__(NT) k_lin_step(LinArgs a) {
    constexpr int STEP = NT / VL, SL = VL * 4;   // rows side by side, columns
    const LinCall& c = a.c[0];
    const int slices = (c.V + SL - 1) / SL, slice = blockIdx.x % slices, h = blockIdx.x / slices % a.HV, n = blockIdx.x / slices / a.HV;
    __shared__ __align__(16) float sq[STEP * NR], sk[STEP * NR], sv[SL], part[STEP][SL], dots[NW];
    __shared__ float2 an;
    const int r0 = threadIdx.x / VL, v = threadIdx.x % VL * 4, v0 = slice * SL;
    const bool cols = v0 + v < c.V;
    const size_t at = ((size_t)n * a.HV + h) * c.K * c.V + v0 + v;
    float4 S[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int k = r0 + i * STEP;
        S[i] = c.s0 && cols && k < c.K ? __ldcs(reinterpret_cast<const float4*>(c.s0 + at + (size_t)k * c.V)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float dot = 0.f;
    for (int k = threadIdx.x; k < STEP * NR; k += NT) {
        const bool on = k < c.K;
        const float q = on ? as_float(static_cast<const TI*>(c.q)[n * c.ldq + (int64_t)(h / c.gq) * c.K + k]) : 0.f;
        const float y = on ? as_float(static_cast<const TI*>(c.k)[n * c.ldk + (int64_t)(h / c.gk) * c.K + k]) : 0.f;
        sq[k] = q;
        sk[k] = y;
        dot = fmaf(q, y, dot);
    }
    if (threadIdx.x < SL) sv[threadIdx.x] = v0 + threadIdx.x < c.V ? as_float(static_cast<const TI*>(c.v)[n * c.ldv + (int64_t)h * c.V + v0 + threadIdx.x]) : 0.f;
    if (threadIdx.x == NT - 1) an = lin_power2(a.decay ? a.decay[h] : 0.f, 1);
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(FULL, dot, o);
    if ((threadIdx.x & 31) == 0) dots[threadIdx.x >> 5] = dot;
    __syncthreads();
    const float4 y = *reinterpret_cast<const float4*>(&sv[v]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int k = r0 + i * STEP;
        const float q = sq[k], x = sk[k];
        const auto one = [&](float& e, float& sum, float val) {
            sum = fmaf(q, e, sum);
            e = fmaf(e, an.x, fmaf(e, an.y, x * val));
        };
        one(S[i].x, o.x, y.x);
        one(S[i].y, o.y, y.y);
        one(S[i].z, o.z, y.z);
        one(S[i].w, o.w, y.w);
        if (c.s1 && cols && k < c.K) __stcs(reinterpret_cast<float4*>(c.s1 + at + (size_t)k * c.V), S[i]);
    }
    *reinterpret_cast<float4*>(&part[r0][v]) = o;
    __syncthreads();
    const int d = threadIdx.x;
    if (d < SL && v0 + d < c.V) {
        float sum = 0.f, qk = 0.f;
#pragma unroll
        for (int i = 0; i < STEP; ++i) sum += part[i][d];
#pragma unroll
        for (int i = 0; i < NW; ++i) qk += dots[i];
        sum = c.s * fmaf(sum, an.x, qk * sv[d]);
        static_cast<TI*>(c.o)[((size_t)n * a.HV + h) * c.V + v0 + d] = TI(sum);
    }
}

// Whether a call is one token of every sequence in whole accesses.
bool is_step(const LinArgs& a) {
    const LinCall& c = a.c[0];
    return a.calls == 1 && !a.ax.cu && a.ax.len == 1 && c.K <= 128 && c.V % 4 == 0 &&
           ((reinterpret_cast<uintptr_t>(c.s0) | reinterpret_cast<uintptr_t>(c.s1)) & 15) == 0;
}
template <typename TI>
cudaError_t run_step(const LinArgs& a, cudaStream_t st) {
    const LinCall& c = a.c[0];
    const int sl = c.V <= 32 ? 32 : c.V <= 64 ? 64 : 128;
    const long long ctas = (long long)a.ax.rows * a.HV * ((c.V + sl - 1) / sl);
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const unsigned g = (unsigned)ctas;
    return traced_launch("k_lin_step", st, [&] {
        if (sl == 32) c.K <= 64 ? k_lin_step<TI, 8, 2><<<g, NT, 0, st>>>(a) : k_lin_step<TI, 8, 4><<<g, NT, 0, st>>>(a);
        else if (sl == 64) c.K <= 64 ? k_lin_step<TI, 16, 4><<<g, NT, 0, st>>>(a) : k_lin_step<TI, 16, 8><<<g, NT, 0, st>>>(a);
        else c.K <= 64 ? k_lin_step<TI, 32, 8><<<g, NT, 0, st>>>(a) : k_lin_step<TI, 32, 16><<<g, NT, 0, st>>>(a);
    });
}

template <typename TI, int KR, int VEC, int TG>
cudaError_t run(const LinArgs& a, cudaStream_t st) {
    int vmax = 1;
    for (int i = 0; i < a.calls; ++i) vmax = a.c[i].V > vmax ? a.c[i].V : vmax;
    const long long ctas = (long long)a.ax.rows * a.units_row * a.HV * ((vmax + 32 * VEC - 1) / (32 * VEC));
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)ctas, a.calls);
    if (a.units_row > 1) {
        cudaError_t e = traced_launch("k_lin_windows", st, [&] { k_lin<TI, KR, VEC, TG><<<grid, NT, 0, st>>>(a, 1); });
        if (e != cudaSuccess || (e = launch_lin_join(a, st)) != cudaSuccess) return e;
    }
    return traced_launch("k_lin", st, [&] { k_lin<TI, KR, VEC, TG><<<grid, NT, 0, st>>>(a, 0); });
}

template <typename TI>
cudaError_t pick(const LinArgs& a, cudaStream_t st) {
    if (is_step(a)) return run_step<TI>(a, st);
    int kmax = 1, widths[3];
    for (int i = 0; i < a.calls; ++i) {
        kmax = a.c[i].K > kmax ? a.c[i].K : kmax;
        widths[i] = a.c[i].V;
    }
    const bool narrow = lin_slice(kmax, widths, a.calls) == 64;
    if (kmax <= 64) return narrow ? run<TI, 8, 2, 8>(a, st) : run<TI, 8, 4, 8>(a, st);
    if (kmax <= 96) return narrow ? run<TI, 12, 2, 8>(a, st) : run<TI, 12, 4, 8>(a, st);
    if (kmax <= 128) return narrow ? run<TI, 16, 2, 8>(a, st) : run<TI, 16, 4, 8>(a, st);
    return run<TI, 32, 2, 4>(a, st);
}

// One state element of a head through a row's windows, the next 8 windows' values on their way: behind window e the state
// is a^n (the state that entered, or that the sequence started from) + the window's own, n its tokens of the sequence. The
// powers are in two parts (a state meets one per window) and formed once per CTA, a thread for each window.
__global__ void __launch_bounds__(256) k_lin_join(LinArgs a) {
    const LinCall& c = a.c[blockIdx.z];
    const int row = blockIdx.y / a.HV, h = blockIdx.y % a.HV;
    const int x = blockIdx.x * 256 + threadIdx.x, KV = c.K * c.V;
    const size_t step = (size_t)a.HV * KV;
    float* p = c.local + ((size_t)row * a.units_row * a.HV + h) * KV + x;
    const int last = a.units_row - 1;
    constexpr int AHEAD = 8, GOES_ON = -1, ENDS = -2;
    float own[AHEAD], next[AHEAD];
    const auto fetch = [&](int e0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) next[i] = e0 + i < last && x < KV ? p[(size_t)(e0 + i) * step] : 0.f;
    };
    fetch(0);
    __shared__ float2 powers[2], power[LIN_MAX_WINDOWS];   // of a token and of a whole window; of each window's tokens
    __shared__ int enters[LIN_MAX_WINDOWS];                // the sequence whose initial state enters, or one of the two above
    const int mine = threadIdx.x;
    int n = 0;
    if (mine < last) {
        const int t0 = mine * a.unit_len, t1 = t0 + a.unit_len;
        const Seq s = lin_seq(a.ax, row, t1 - 1, c.back);
        if (s.end > t1) n = t1 - max(s.first, t0);
        enters[mine] = s.end <= t1 ? ENDS : s.first >= t0 ? s.n : GOES_ON;
    }
    if (mine == 0 || mine == 32) powers[mine >> 5] = lin_power2(a.decay ? a.decay[h] : 0.f, mine ? a.unit_len : 1);
    __syncthreads();
    if (n > 0) power[mine] = n == a.unit_len ? powers[1] : lin_raise(powers[0], n);
    __syncthreads();
    if (x >= KV) return;
    const int from = c.transposed ? x % c.V * c.K + x / c.V : x;   // in s0
    float S = 0.f;
    for (int e0 = 0; e0 < last; e0 += AHEAD) {
        float start[AHEAD];   // does not need the state
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            own[i] = next[i];
            const int seq = e0 + i < last ? enters[e0 + i] : ENDS;
            start[i] = seq >= 0 && c.s0 ? c.s0[((size_t)seq * a.HV + h) * KV + from] : 0.f;
        }
        fetch(e0 + AHEAD);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int e = e0 + i;
            if (e >= last || enters[e] == ENDS) continue;
            if (enters[e] >= 0) S = start[i];
            const float2 f = power[e];
            S = fmaf(S, f.x, fmaf(S, f.y, own[i]));
            p[(size_t)e * step] = S;
        }
    }
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

// Value columns of a CTA: 128, or 64 where slices of those walk fewer columns in all, or keys are wide.
int lin_slice(int kmax, const int* widths, int calls) {
    long long narrow = 0, wide = 0;
    for (int i = 0; i < calls; ++i) {
        narrow += (widths[i] + 63) / 64 * 64;
        wide += (widths[i] + 127) / 128 * 128;
    }
    return kmax > 128 || narrow < wide ? 64 : 128;
}

// The cheapest number of windows n of a row, in groups' times (some 5.7 us where two CTAs share an SM, or one of the widest
// has it): the CTAs over the SMs, a quarter of a round more for the uneven end of several; 0.65 more for each group where
// the windows' own states are formed first, 3 for a window's states, and windows cost two launches and a join. (Measured, us:
// fp32, 3 x 777 tokens, 10 heads of 40 x 72, forward in 1, 5, 10, 12 windows 366, 135, 112, 132, backward 452, 321, 335, 329; 300
// tokens, 4 heads of 64, forward in 1, 4, 10, 24: 105, 57, 35, 29; 2 x 4096 tokens, 16 heads of 128, backward in 1, 4, 24: 2928,
// 3081, 3186; bf16, 4 x 1000 tokens, 8 heads of 200, forward in 1, 2: 1253, 1674.)
int lin_window(int rows, int len, int ctas, int kmax, int slice) {
    const int groups = (len + 7) / 8;
    const double sms = sm_count(), fit = sms * (kmax > 128 || (kmax > 96 && slice == 128) ? 1 : 2);   // CTAs at once
    double least = 0;
    int best = groups > 0 ? groups : 1;
    for (int n = 1; n <= LIN_MAX_WINDOWS && n <= groups; ++n) {
        const int each = (groups + n - 1) / n;
        const double all = (double)rows * ctas * n;
        const double rounds = all > fit ? all / fit + 0.25 : all > sms || fit == sms ? 1. : 0.95;
        const double cost = rounds * (each * (n > 1 ? 1.65 : 1.) + 3.) + (n > 1 ? 4. + 0.1 * n : 0.);
        if (n == 1 || cost < least) {
            least = cost;
            best = each;
        }
    }
    return best * 8;
}

cudaError_t launch_lin(const LinArgs& a, int bf16, cudaStream_t st) {
    return bf16 ? pick<__nv_bfloat16>(a, st) : pick<float>(a, st);
}

cudaError_t launch_lin_join(const LinArgs& a, cudaStream_t st) {
    int most = 0;
    for (int i = 0; i < a.calls; ++i) most = a.c[i].K * a.c[i].V > most ? a.c[i].K * a.c[i].V : most;
    if ((long long)a.ax.rows * a.HV > 65535) return cudaErrorInvalidConfiguration;
    return traced_launch("k_lin_join", st, [&] { k_lin_join<<<dim3((most + 255) / 256, a.ax.rows * a.HV, a.calls), 256, 0, st>>>(a); });
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
