// Selective state space scan (diagonal, input-dependent step), forward:
//     delta = softplus(dt + dt_bias),  a = exp(-delta exp(A_log)),  u = delta x
//     h_t = a h_{t-1} + u B_t,   y_t = (sum_n C_t[n] h_t[n] + d_skip x_t) silu(z_t)
// Four lanes share a channel and hold its states in registers; a CTA of 128 threads
// walks 32 channels through a time piece, tile by tile: the tile's steps are formed
// once per (token, channel) in shared memory, the recurrence runs over them, and
// the outputs are gated and stored from shared memory.
// A long row is cut into time pieces when its channels alone do not fill the GPU:
// a first pass forms each piece's end state from zero and its sum of delta (the
// piece's decay is exp(A sum delta)); in the second pass each piece joins the
// states of the pieces before it and runs its outputs.
#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int TT = 32;   // tokens per tile
constexpr int YP = 40;   // row stride of the shared outputs (conflict-free for 4 tokens x 8 channels)

enum { OUT = 0, OUT_CKPT = 1, CKPT = 2, PIECE = 3 };

template <typename TI, int EL, int MODE>
__global__ void __launch_bounds__(SSM_T) k_ssm_fwd(SsmArgs a) {
    constexpr int NP = 4 * EL;
    constexpr bool HAS_Y = MODE == OUT || MODE == OUT_CKPT, HAS_CK = MODE == OUT_CKPT || MODE == CKPT;
    __shared__ float2 s_du[TT][SSM_CH];
    __shared__ __align__(16) float s_b[TT][NP];
    __shared__ __align__(16) float s_c[HAS_Y ? TT : 1][NP];
    __shared__ float s_y[HAS_Y ? TT : 1][YP];
    if (blockIdx.x == 0 && MODE != PIECE) axis_check(a.ax, a.err);
    const SsmPlace pl = ssm_place(a);
    const int tid = threadIdx.x, l = tid & 3, ch = tid >> 2, n0 = l * EL;
    const int d = pl.c0 + ch;
    const bool on = ch < pl.nch;
    const size_t tok0 = (size_t)pl.row * a.ax.len;
    const size_t DS = (size_t)a.D * a.S;
    float A2[EL], h[EL], sd = 0.f;
    load_states<EL>(a.A_log + (size_t)d * a.S, n0, a.S, on, A2);
#pragma unroll
    for (int e = 0; e < EL; ++e) A2[e] = on && n0 + e < a.S ? -expf(A2[e]) * LOG2E : 0.f;
    const float* h0 = a.h0 ? a.h0 + (size_t)d * a.S : nullptr;
    float* ht = a.ht && MODE != PIECE ? a.ht + (size_t)d * a.S : nullptr;
    auto init_state = [&](int n) {
        if (h0) {
            load_states<EL>(h0 + n * DS, n0, a.S, on, h);
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) h[e] = 0.f;
        }
    };
    if (ht && a.ax.cu) {   // sequences without tokens
        const int units = gridDim.x / (((a.D / a.G + SSM_CH - 1) / SSM_CH) * a.G);
        for (int n = pl.unit; n < a.ax.N; n += units) {
            if (axis_cu(a.ax, n + 1) > axis_cu(a.ax, n)) continue;
            init_state(n);
            store_states<EL>(ht + n * DS, n0, a.S, on, h);
        }
        if (pl.lo >= pl.hi) return;
    }
    int t = pl.lo;
    Seq s;
    if (MODE == PIECE) {
        // the part of the piece that reaches past its end
        s = seq_at(a.ax, pl.row, pl.hi - 1);
        if (s.end <= pl.hi) return;
        t = max(pl.lo, s.first);
        if (s.first >= pl.lo) init_state(s.n);
        else {
#pragma unroll
            for (int e = 0; e < EL; ++e) h[e] = 0.f;
        }
    } else {
        s = seq_at(a.ax, pl.row, t);
        if (t == s.first) {
            init_state(s.n);
        } else {
            // the state entering this piece: the earlier pieces of its sequence, joined in order
            const int q = s.first / a.unit_len;
#pragma unroll
            for (int e = 0; e < EL; ++e) h[e] = 0.f;
            for (int r = q; r < pl.u; ++r) {
                const size_t ru = (size_t)pl.row * a.units_row + r;
                float hl[EL];
                load_states<EL>(a.hloc + ru * DS + (size_t)d * a.S, n0, a.S, on, hl);
                const float sum = on ? a.sdt[ru * a.D + d] : 0.f;
#pragma unroll
                for (int e = 0; e < EL; ++e) h[e] = r == q ? hl[e] : fmaf(ex2(A2[e] * sum), h[e], hl[e]);
            }
        }
    }
    // this thread's part of a tile: one token, 8 channels
    const int ptok = tid >> 2, pc = (tid & 3) * 8, pvalid = pl.nch - pc;
    const TI* xp = static_cast<const TI*>(a.x) + tok0 * a.ldx + pl.c0 + pc;
    const TI* dp = static_cast<const TI*>(a.dt) + tok0 * a.lddt + pl.c0 + pc;
    const TI* zp = a.z ? static_cast<const TI*>(a.z) + tok0 * a.ldz + pl.c0 + pc : nullptr;
    const TI* bp = static_cast<const TI*>(a.b) + tok0 * a.ldb + (size_t)pl.g * a.S;
    const TI* cp = static_cast<const TI*>(a.c) + tok0 * a.ldc + (size_t)pl.g * a.S;
    const bool wide = pvalid >= 8;
    float bias[8], skip[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bias[i] = a.dt_bias && i < pvalid ? a.dt_bias[pl.c0 + pc + i] : 0.f;
        skip[i] = a.d_skip && i < pvalid ? a.d_skip[pl.c0 + pc + i] : 0.f;
    }
    for (int tb = t; tb < pl.hi; tb += TT) {
        const int te = min(tb + TT, pl.hi);
        float x[8], dt[8];
        const bool in = tb + ptok < te && pvalid > 0;
        if (in) {
            load_row<8>(xp + (size_t)(tb + ptok) * a.ldx, x, pvalid, wide && (a.vec & SSM_VEC_X));
            load_row<8>(dp + (size_t)(tb + ptok) * a.lddt, dt, pvalid, wide && (a.vec & SSM_VEC_DT));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float dl = 0.f;
            if (in) {
                dl = dt[i] + bias[i];
                if (a.softplus) dl = ssm_softplus(dl);
            } else {
                x[i] = 0.f;
            }
            s_du[ptok][pc + i] = make_float2(dl, dl * x[i]);
        }
        constexpr int NC = NP / 8;   // chunks of 8 states per row
        for (int i = tid; i < TT * NC * (HAS_Y ? 2 : 1); i += SSM_T) {
            const bool isc = i >= TT * NC;
            const int j = isc ? i - TT * NC : i, tok = j / NC, k = (j - tok * NC) * 8;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
            if (tb + tok < te) {
                if (isc) load_row<8>(cp + (size_t)(tb + tok) * a.ldc + k, v, a.S - k, a.S - k >= 8 && (a.vec & SSM_VEC_C));
                else load_row<8>(bp + (size_t)(tb + tok) * a.ldb + k, v, a.S - k, a.S - k >= 8 && (a.vec & SSM_VEC_B));
            }
            float* dst = isc ? &s_c[HAS_Y ? tok : 0][k] : &s_b[tok][k];
            reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        __syncthreads();
        t = tb;
        while (t < te) {
            if (MODE != PIECE && t == s.end) {
                if (ht) store_states<EL>(ht + s.n * DS, n0, a.S, on, h);
                s = seq_at(a.ax, pl.row, t);
                init_state(s.n);
            }
            if (HAS_CK && t % SSM_CKPT == 0) {
                const size_t slot = (size_t)pl.row * ((a.ax.len + SSM_CKPT - 1) / SSM_CKPT) + t / SSM_CKPT;
                store_states<EL>(a.ckpt + slot * DS + (size_t)d * a.S, n0, a.S, on, h);
            }
            int run = MODE == PIECE ? te : min(te, s.end);
            if (HAS_CK) run = min(run, (t | (SSM_CKPT - 1)) + 1);
            for (; t < run; t += 4) {
                float acc[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[i] = 0.f;
                    if (t + i >= run) continue;
                    const float2 du = s_du[t + i - tb][ch];
                    float b[EL], c[EL];
                    lds_states<EL>(&s_b[t + i - tb][n0], b);
                    if (HAS_Y) lds_states<EL>(&s_c[HAS_Y ? t + i - tb : 0][n0], c);
#pragma unroll
                    for (int e = 0; e < EL; ++e) {
                        h[e] = fmaf(ex2(du.x * A2[e]), h[e], du.y * b[e]);
                        if (HAS_Y) acc[i] = fmaf(h[e], c[e], acc[i]);
                    }
                    if (MODE == PIECE) sd += du.x;
                }
                if (HAS_Y) {
                    // lane l of a channel's four keeps token l's sum
                    halve<4>(acc, l, 2);
                    halve<2>(acc, l, 1);
                    if (t + l < run) s_y[HAS_Y ? t + l - tb : 0][ch] = acc[0];
                }
            }
            t = run;
        }
        __syncthreads();
        if (HAS_Y && in) {
            float o[8], z[8];
            if (zp) load_row<8>(zp + (size_t)(tb + ptok) * a.ldz, z, pvalid, wide && (a.vec & SSM_VEC_Z));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = fmaf(skip[i], x[i], s_y[HAS_Y ? ptok : 0][pc + i]);
                if (zp) o[i] *= z[i] * sigmoid_fast(z[i]);
            }
            store_row<8>(static_cast<TI*>(a.y) + (tok0 + tb + ptok) * a.D + pl.c0 + pc, o, pvalid, wide && (a.vec & SSM_VEC_OUT));
        }
    }
    if (MODE == PIECE) {
        store_states<EL>(a.hloc + pl.unit * DS + (size_t)d * a.S, n0, a.S, on, h);
        if (on && l == 0) a.sdt[(size_t)pl.unit * a.D + d] = sd;
    } else if (ht && pl.hi == s.end) {
        store_states<EL>(ht + s.n * DS, n0, a.S, on, h);
    }
}

template <typename TI, int EL>
void run_mode(const SsmArgs& a, int mode, unsigned grid, cudaStream_t st) {
    switch (mode) {
        case OUT: k_ssm_fwd<TI, EL, OUT><<<grid, SSM_T, 0, st>>>(a); break;
        case OUT_CKPT: k_ssm_fwd<TI, EL, OUT_CKPT><<<grid, SSM_T, 0, st>>>(a); break;
        case CKPT: k_ssm_fwd<TI, EL, CKPT><<<grid, SSM_T, 0, st>>>(a); break;
        default: k_ssm_fwd<TI, EL, PIECE><<<grid, SSM_T, 0, st>>>(a); break;
    }
}
template <typename TI>
void run_states(const SsmArgs& a, int mode, cudaStream_t st) {
    const unsigned grid = (unsigned)(a.ax.rows * a.units_row) * ssm_channel_tiles(a.D, a.G);
    if (a.S <= 8) run_mode<TI, 2>(a, mode, grid, st);
    else if (a.S <= 16) run_mode<TI, 4>(a, mode, grid, st);
    else if (a.S <= 32) run_mode<TI, 8>(a, mode, grid, st);
    else run_mode<TI, 16>(a, mode, grid, st);
}

}  // namespace

int ssm_channel_tiles(int D, int G) { return (D / G + SSM_CH - 1) / SSM_CH * G; }

int ssm_units(int rows, int len, int D, int G, int S, bool backward) {
    // pieces only while the channels and rows alone leave SMs idle; a piece is at least 128 tokens
    const long long ctas = (long long)rows * ssm_channel_tiles(D, G), want = 4LL * sm_count();
    long long units = ctas >= sm_count() ? 1 : want / ctas;
    const long long most = (len + 127) / 128;
    if (units > most) units = most;
    return units < 1 ? 1 : (int)units;
}

cudaError_t launch_ssm_fwd(const SsmArgs& a, int bf16, int mode, cudaStream_t st) {
    return traced_launch(mode == CKPT ? "k_ssm_ckpt" : "k_ssm_fwd", st, [&] {
        bf16 ? run_states<__nv_bfloat16>(a, mode, st) : run_states<float>(a, mode, st);
    });
}

cudaError_t launch_ssm_pieces(const SsmArgs& a, int bf16, cudaStream_t st) {
    return traced_launch("k_ssm_pieces", st, [&] {
        bf16 ? run_states<__nv_bfloat16>(a, PIECE, st) : run_states<float>(a, PIECE, st);
    });
}

}  // namespace kda
