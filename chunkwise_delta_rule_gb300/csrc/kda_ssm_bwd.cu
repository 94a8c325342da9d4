// Selective state space scan, backward. With d0_t = dy_t silu(z_t), A = -exp(A_log),
// a_t = exp(delta_t A) and g_t the adjoint of h_t:
//     g_t = C_t d0_t + a_{t+1} g_{t+1}
//     dC_t = sum_d d0 h,  dB_t = sum_d u g,  s1 = sum_n g B,  s2 = sum_n A a g h_{t-1}
//     dx = delta s1 + d_skip d0,  ddelta = x s1 + s2,  dA = sum_t delta a g h_{t-1}
//     dz = dy y0 silu'(z) with y0 = sum_n C h + d_skip x,  dh0 = a_1 g_1
// A CTA walks 32 channels backwards through a time piece in tiles of 16 tokens: the
// states inside a tile are recomputed from the checkpoint the forward left at its
// first token (L tokens at a time in registers), then the adjoint runs over them.
// dB and dC are summed over the warp's channels by halving exchanges, over the CTA
// in shared memory and over the CTAs' rows in a second kernel, in a fixed order;
// the parameters' gradients go the same way, so nothing depends on timing.
#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int TB = SSM_CKPT;   // tokens per tile
constexpr int YP = 40;

template <int EL>
struct BwdShape {
    static constexpr int NP = 4 * EL;
    static constexpr int L = EL <= 4 ? 16 : 64 / EL;      // tokens whose states are held at once
    static constexpr int NSUB = TB / L;
    static constexpr int VB = 2 * EL;                     // dB and dC values of a lane
    static constexpr int KEEP = VB >= 8 ? VB / 8 : 1;     // ... it holds after the sum over 8 channels
    struct Smem {
        float4 in[TB][SSM_CH];            // delta, u, d0, x
        float s1[TB][YP], s2[TB][YP], yc[TB][YP];
        float b[TB][NP], c[TB][NP];
        float red[4][TB][2 * NP];
        float sub[NSUB > 1 ? NSUB - 1 : 1][EL][SSM_T];
    };
};

template <typename TI, int EL>
__global__ void __launch_bounds__(SSM_T) k_ssm_bwd(SsmArgs a) {
    using Sh = BwdShape<EL>;
    constexpr int NP = Sh::NP, L = Sh::L, NSUB = Sh::NSUB, VB = Sh::VB, KEEP = Sh::KEEP;
    extern __shared__ __align__(16) unsigned char raw[];
    typename Sh::Smem& sm = *reinterpret_cast<typename Sh::Smem*>(raw);
    const SsmPlace pl = ssm_place<SSM_CH>(a);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = tid & 3, ch = tid >> 2, n0 = l * EL;
    const int d = pl.c0 + ch;
    const bool on = ch < pl.nch;
    const size_t tok0 = (size_t)pl.row * a.ax.len;
    const size_t DS = (size_t)a.D * a.S;
    float A2[EL], r[EL], dA[EL];
    load_states<EL>(a.A_log + (size_t)d * a.S, n0, a.S, on, A2);
#pragma unroll
    for (int e = 0; e < EL; ++e) {
        A2[e] = on && n0 + e < a.S ? -expf(A2[e]) * LOG2E : 0.f;
        r[e] = dA[e] = 0.f;
    }
    auto state_of = [&](const float* base, int n, float(&v)[EL]) {
        if (base) {
            load_states<EL>(base + n * DS + (size_t)d * a.S, n0, a.S, on, v);
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) v[e] = 0.f;
        }
    };
    if (a.dh0 && (a.ax.cu || a.ax.len == 0)) {   // sequences without tokens: their adjoint passes through
        for (int n = pl.unit; n < a.ax.N; n += pl.units) {
            if (a.ax.cu && axis_cu(a.ax, n + 1) > axis_cu(a.ax, n)) continue;
            float v[EL];
            state_of(a.dht, n, v);
            store_states<EL>(a.dh0 + n * DS + (size_t)d * a.S, n0, a.S, on, v);
        }
    }
    // this thread's part of a tile: one token, 4 channels
    const int ptok = tid >> 3, pc = (tid & 7) * 4, pvalid = pl.nch - pc;
    const TI* xp = static_cast<const TI*>(a.x) + tok0 * a.ldx + pl.c0 + pc;
    const TI* dp = static_cast<const TI*>(a.dt) + tok0 * a.lddt + pl.c0 + pc;
    const TI* zp = a.z ? static_cast<const TI*>(a.z) + tok0 * a.ldz + pl.c0 + pc : nullptr;
    const TI* yp = static_cast<const TI*>(a.dy) + tok0 * a.D + pl.c0 + pc;
    const TI* bp = static_cast<const TI*>(a.b) + tok0 * a.ldb + (size_t)pl.g * a.S;
    const TI* cp = static_cast<const TI*>(a.c) + tok0 * a.ldc + (size_t)pl.g * a.S;
    float bias[4], skip[4], dskip[4], dbias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = a.dt_bias && i < pvalid ? a.dt_bias[pl.c0 + pc + i] : 0.f;
        skip[i] = a.d_skip && i < pvalid ? a.d_skip[pl.c0 + pc + i] : 0.f;
        dskip[i] = dbias[i] = 0.f;
    }
    Seq s{0, 0, 0};
    if (pl.hi > pl.lo) {
        s = seq_at(a.ax, pl.row, pl.hi - 1);
        if (s.end > pl.hi) {
            // the adjoint entering this piece from the later pieces of its sequence, joined in order
            const int q = min((s.end - 1) / a.unit_len, a.units_row - 1);
            for (int v = q; v > pl.u; --v) {
                const size_t ru = (size_t)pl.row * a.units_row + v;
                float rl[EL];
                load_states<EL>(a.rloc + ru * DS + (size_t)d * a.S, n0, a.S, on, rl);
                const float sum = on ? a.sdt[ru * a.D + d] : 0.f;
#pragma unroll
                for (int e = 0; e < EL; ++e) r[e] = v == q ? rl[e] : fmaf(ex2(A2[e] * sum), r[e], rl[e]);
            }
        }
    }
    const int last = pl.hi > pl.lo ? (pl.hi - 1) / TB * TB : pl.lo - TB;
    for (int tb = last; tb >= pl.lo; tb -= TB) {
        const int te = min(tb + TB, pl.hi), nt = te - tb;
        const int t = tb + ptok;
        const bool in = t < te && pvalid > 0;
        // steps and gated gradients of the tile
        float x[4], raw_dt[4], z[4], dy[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = raw_dt[i] = z[i] = dy[i] = 0.f;
        if (in) {
            load_row<4>(xp + (size_t)t * a.ldx, x, pvalid, false);
            load_row<4>(dp + (size_t)t * a.lddt, raw_dt, pvalid, false);
            load_row<4>(yp + (size_t)t * a.D, dy, pvalid, false);
            if (zp) load_row<4>(zp + (size_t)t * a.ldz, z, pvalid, false);
        }
        float d0[4], dl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            raw_dt[i] += bias[i];
            dl[i] = !in || i >= pvalid ? 0.f : a.softplus ? ssm_softplus(raw_dt[i]) : raw_dt[i];
            d0[i] = zp ? dy[i] * z[i] * sigmoid_fast(z[i]) : dy[i];
            sm.in[ptok][pc + i] = make_float4(dl[i], dl[i] * x[i], d0[i], x[i]);
        }
        constexpr int NC = NP / 8;
        for (int i = tid; i < 2 * TB * NC; i += SSM_T) {
            const bool isc = i >= TB * NC;
            const int j = isc ? i - TB * NC : i, tok = j / NC, k = (j - tok * NC) * 8;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
            if (tb + tok < te) {
                if (isc) load_row<8>(cp + (size_t)(tb + tok) * a.ldc + k, v, a.S - k, a.S - k >= 8 && !(a.how >> SSM_C & 3));
                else load_row<8>(bp + (size_t)(tb + tok) * a.ldb + k, v, a.S - k, a.S - k >= 8 && !(a.how >> SSM_B & 3));
            }
            float* dst = isc ? &sm.c[tok][k] : &sm.b[tok][k];
            reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        // first and last tokens of sequences inside the tile
        uint32_t starts = 0, ends = 0;
        for (int p = te - 1;;) {
            if (p < s.first || p >= s.end) s = seq_at(a.ax, pl.row, p);
            if (s.end <= te && s.end > tb) ends |= 1u << (s.end - 1 - tb);
            if (s.first < tb) break;
            starts |= 1u << (s.first - tb);
            if (s.first == tb) break;
            p = s.first - 1;
        }
        __syncthreads();
        float hstart[EL];
        {
            const size_t slot = (size_t)pl.row * ((a.ax.len + TB - 1) / TB) + tb / TB;
            load_states<EL>(a.ckpt + slot * DS + (size_t)d * a.S, n0, a.S, on, hstart);
        }
        // one token of the recurrence
        auto step = [&](int i, float(&h)[EL]) {
            if (i > 0 && (starts >> i & 1)) state_of(a.h0, seq_at(a.ax, pl.row, tb + i).n, h);
            const float4 v = sm.in[i][ch];
            float b[EL];
            lds_states<EL>(&sm.b[i][n0], b);
#pragma unroll
            for (int e = 0; e < EL; ++e) h[e] = fmaf(ex2(v.x * A2[e]), h[e], v.y * b[e]);
        };
        if (NSUB > 1) {
            // states at the sub-blocks' starts
            float h[EL];
#pragma unroll
            for (int e = 0; e < EL; ++e) h[e] = hstart[e];
            for (int i = 0; i < min(nt, TB - L); ++i) {
                step(i, h);
                if ((i + 1) % L == 0)
#pragma unroll
                    for (int e = 0; e < EL; ++e) sm.sub[(i + 1) / L - 1][e][tid] = h[e];
            }
        }
        for (int k = NSUB - 1; k >= 0; --k) {
            const int i0 = k * L;
            if (i0 >= nt) continue;
            float hs[L][EL], h[EL], hk[EL];
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                hk[e] = k == 0 ? hstart[e] : sm.sub[k > 0 ? k - 1 : 0][e][tid];
                h[e] = hk[e];
            }
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (i0 + i < nt) step(i0 + i, h);
#pragma unroll
                for (int e = 0; e < EL; ++e) hs[i][e] = h[e];
            }
#pragma unroll
            for (int q = L / 4 - 1; q >= 0; --q) {
                float p1[4], p2[4], py[4];
#pragma unroll
                for (int j = 3; j >= 0; --j) {
                    const int i = 4 * q + j, it = i0 + i;
                    p1[j] = p2[j] = py[j] = 0.f;
                    if (it >= nt) continue;
                    if (ends >> it & 1) state_of(a.dht, seq_at(a.ax, pl.row, tb + it).n, r);
                    float hp[EL];
#pragma unroll
                    for (int e = 0; e < EL; ++e) hp[e] = i > 0 ? hs[i > 0 ? i - 1 : 0][e] : hk[e];
                    const bool start = starts >> it & 1;
                    if (start && it > 0) state_of(a.h0, seq_at(a.ax, pl.row, tb + it).n, hp);
                    const float4 v = sm.in[it][ch];
                    float b[EL], c[EL], bc[VB];
                    lds_states<EL>(&sm.b[it][n0], b);
                    lds_states<EL>(&sm.c[it][n0], c);
#pragma unroll
                    for (int e = 0; e < EL; ++e) {
                        const float g = fmaf(c[e], v.z, r[e]);
                        py[j] = fmaf(hs[i][e], c[e], py[j]);
                        bc[EL + e] = v.z * hs[i][e];
                        bc[e] = v.y * g;
                        p1[j] = fmaf(g, b[e], p1[j]);
                        r[e] = ex2(v.x * A2[e]) * g;
                        const float w = r[e] * hp[e];
                        p2[j] = fmaf(w, A2[e], p2[j]);
                        dA[e] = fmaf(w, v.x, dA[e]);
                    }
                    if (start) {
                        if (a.dh0) {
                            const int n = seq_at(a.ax, pl.row, tb + it).n;
                            store_states<EL>(a.dh0 + n * DS + (size_t)d * a.S, n0, a.S, on, r);
                        }
#pragma unroll
                        for (int e = 0; e < EL; ++e) r[e] = 0.f;
                    }
                    // over the warp's 8 channels: lane bits 2, 3, 4
                    int first = 0;
                    halve<VB>(bc, lane, 4);
                    first += lane & 4 ? VB / 2 : 0;
                    halve<VB / 2>(bc, lane, 8);
                    first += lane & 8 ? VB / 4 : 0;
                    if (VB >= 8) {
                        halve<(VB >= 8 ? VB / 4 : 2)>(bc, lane, 16);
                        first += lane & 16 ? VB / 8 : 0;
                    } else {
                        bc[0] += __shfl_xor_sync(SSM_FULL, bc[0], 16);
                    }
                    // value f of a lane: dB of its state f, or dC of state f - EL
#pragma unroll
                    for (int f = 0; f < KEEP; ++f) {
                        const int w = first + f;
                        sm.red[warp][it][w < EL ? n0 + w : NP + n0 + w - EL] = bc[f];
                    }
                }
                halve<4>(p1, l, 2); halve<2>(p1, l, 1);
                halve<4>(p2, l, 2); halve<2>(p2, l, 1);
                halve<4>(py, l, 2); halve<2>(py, l, 1);
                const int it = i0 + 4 * q + l;
                if (it < nt) {
                    sm.s1[it][ch] = p1[0];
                    sm.s2[it][ch] = p2[0];
                    sm.yc[it][ch] = py[0];
                }
            }
        }
        __syncthreads();
        if (in) {
            float ox[4], od[4], oz[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float s1 = sm.s1[ptok][pc + i];
                ox[i] = fmaf(dl[i], s1, skip[i] * d0[i]);
                float g = fmaf(x[i], s1, sm.s2[ptok][pc + i] * (1.f / LOG2E));
                if (a.softplus) g *= 1.f / (1.f + expf(-raw_dt[i]));
                od[i] = g;
                const float y0 = fmaf(skip[i], x[i], sm.yc[ptok][pc + i]), sg = sigmoid_fast(z[i]);
                oz[i] = dy[i] * y0 * sg * fmaf(z[i], 1.f - sg, 1.f);
                if (i < pvalid) {
                    dskip[i] = fmaf(d0[i], x[i], dskip[i]);
                    dbias[i] += g;
                }
            }
            const size_t o = (tok0 + t) * a.D + pl.c0 + pc;
            store_row<4>(static_cast<TI*>(a.dx) + o, ox, pvalid, false);
            store_row<4>(static_cast<TI*>(a.ddt) + o, od, pvalid, false);
            if (zp) store_row<4>(static_cast<TI*>(a.dz) + o, oz, pvalid, false);
        }
        for (int i = tid; i < nt * 2 * NP; i += SSM_T) {
            const int tok = i / (2 * NP), f = i - tok * (2 * NP), which = f / NP, n = f - which * NP;
            if (n >= a.S) continue;
            const float v = (sm.red[0][tok][f] + sm.red[1][tok][f]) + (sm.red[2][tok][f] + sm.red[3][tok][f]);
            const size_t tokens = (size_t)a.ax.rows * a.ax.len;
            a.pbc[((pl.tile * tokens + tok0 + tb + tok) * 2 + which) * a.S + n] = v;
        }
        __syncthreads();
    }
    // parameters: this piece's sums
    store_states<EL>(a.pA + pl.unit * DS + (size_t)d * a.S, n0, a.S, on, dA);
    float* red = &sm.red[0][0][0];   // [16 tokens][32 channels]
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) red[ptok * SSM_CH + pc + i] = which ? dbias[i] : dskip[i];
        __syncthreads();
        if (tid < pl.nch) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < TB; ++i) v += red[i * SSM_CH + tid];
            a.pv[((size_t)pl.unit * 2 + which) * a.D + pl.c0 + tid] = v;
        }
    }
}

// Local adjoint leaving a time piece's first token: from dht where the piece's sequence ends inside it, else from zero.
template <typename TI, int EL>
__global__ void __launch_bounds__(SSM_T) k_ssm_bwd_pieces(SsmArgs a) {
    constexpr int NP = 4 * EL;
    __shared__ float2 s_in[TB][SSM_CH];
    __shared__ __align__(16) float s_c[TB][NP];
    const SsmPlace pl = ssm_place<SSM_CH>(a);
    if (pl.lo >= pl.hi) return;
    const Seq s = seq_at(a.ax, pl.row, pl.lo);
    if (s.first >= pl.lo) return;
    const int tid = threadIdx.x, l = tid & 3, ch = tid >> 2, n0 = l * EL, d = pl.c0 + ch;
    const bool on = ch < pl.nch;
    const size_t tok0 = (size_t)pl.row * a.ax.len;
    const size_t DS = (size_t)a.D * a.S;
    float A2[EL], r[EL], sd = 0.f;
    load_states<EL>(a.A_log + (size_t)d * a.S, n0, a.S, on, A2);
#pragma unroll
    for (int e = 0; e < EL; ++e) A2[e] = on && n0 + e < a.S ? -expf(A2[e]) * LOG2E : 0.f;
    const int hi = min(pl.hi, s.end);
    if (s.end <= pl.hi && a.dht) {
        load_states<EL>(a.dht + s.n * DS + (size_t)d * a.S, n0, a.S, on, r);
    } else {
#pragma unroll
        for (int e = 0; e < EL; ++e) r[e] = 0.f;
    }
    const int ptok = tid >> 3, pc = (tid & 7) * 4, pvalid = pl.nch - pc;
    const TI* dp = static_cast<const TI*>(a.dt) + tok0 * a.lddt + pl.c0 + pc;
    const TI* zp = a.z ? static_cast<const TI*>(a.z) + tok0 * a.ldz + pl.c0 + pc : nullptr;
    const TI* yp = static_cast<const TI*>(a.dy) + tok0 * a.D + pl.c0 + pc;
    const TI* cp = static_cast<const TI*>(a.c) + tok0 * a.ldc + (size_t)pl.g * a.S;
    for (int tb = (hi - 1) / TB * TB; tb >= pl.lo; tb -= TB) {
        const int te = min(tb + TB, hi), t = tb + ptok;
        const bool in = t < te && pvalid > 0;
        float dt[4], z[4], dy[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) dt[i] = z[i] = dy[i] = 0.f;
        if (in) {
            load_row<4>(dp + (size_t)t * a.lddt, dt, pvalid, false);
            load_row<4>(yp + (size_t)t * a.D, dy, pvalid, false);
            if (zp) load_row<4>(zp + (size_t)t * a.ldz, z, pvalid, false);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = dt[i] + (a.dt_bias && i < pvalid ? a.dt_bias[pl.c0 + pc + i] : 0.f);
            const float dl = !in || i >= pvalid ? 0.f : a.softplus ? ssm_softplus(v) : v;
            s_in[ptok][pc + i] = make_float2(dl, zp ? dy[i] * z[i] * sigmoid_fast(z[i]) : dy[i]);
        }
        constexpr int NC = NP / 8;
        for (int i = tid; i < TB * NC; i += SSM_T) {
            const int tok = i / NC, k = (i - tok * NC) * 8;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
            if (tb + tok < te)
                load_row<8>(cp + (size_t)(tb + tok) * a.ldc + k, v, a.S - k, a.S - k >= 8 && !(a.how >> SSM_C & 3));
            reinterpret_cast<float4*>(&s_c[tok][k])[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(&s_c[tok][k])[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        __syncthreads();
        for (int i = te - tb - 1; i >= 0; --i) {
            const float2 v = s_in[i][ch];
            float c[EL];
            lds_states<EL>(&s_c[i][n0], c);
#pragma unroll
            for (int e = 0; e < EL; ++e) r[e] = ex2(v.x * A2[e]) * fmaf(c[e], v.y, r[e]);
            sd += v.x;
        }
        __syncthreads();
    }
    store_states<EL>(a.rloc + pl.unit * DS + (size_t)d * a.S, n0, a.S, on, r);
    if (on && l == 0) a.sdt[(size_t)pl.unit * a.D + d] = sd;
}

// db and dc: the channel tiles' sums in tile order (the first `nbc` CTAs); then the parameters' sums over the pieces.
template <typename TI>
__global__ void k_ssm_sums(SsmArgs a, unsigned nbc) {
    const size_t tokens = (size_t)a.ax.rows * a.ax.len;
    if (blockIdx.x < nbc) {
        const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;   // token, which, group, state
        const int GS = a.G * a.S;
        if (i >= tokens * 2 * GS) return;
        const size_t tok = i / (2 * GS);
        const int f = (int)(i - tok * 2 * GS), which = f / GS, gs = f - which * GS, g = gs / a.S, n = gs - g * a.S;
        const int tpg = (a.D / a.G + SSM_CH - 1) / SSM_CH;
        float v = 0.f;
        for (int k = 0; k < tpg; ++k) v += a.pbc[(((size_t)(g * tpg + k) * tokens + tok) * 2 + which) * a.S + n];
        st(static_cast<TI*>(which ? a.dc : a.db) + tok * GS + gs, v);
        return;
    }
    const size_t i = (size_t)(blockIdx.x - nbc) * blockDim.x + threadIdx.x;
    const size_t DS = (size_t)a.D * a.S;
    const int units = a.ax.rows * a.units_row;
    if (i < DS) {
        float v = 0.f;
        for (int u = 0; u < units; ++u) v += a.pA[u * DS + i];
        a.dA_log[i] = -expf(a.A_log[i]) * v;
    } else if (i < DS + 2 * (size_t)a.D) {
        const int f = (int)(i - DS), which = f >= a.D, d = which ? f - a.D : f;
        float* out = which ? a.ddt_bias : a.dd_skip;
        if (!out) return;
        float v = 0.f;
        for (int u = 0; u < units; ++u) v += a.pv[((size_t)u * 2 + which) * a.D + d];
        out[d] = v;
    }
}

template <typename TI, int EL>
cudaError_t run_bwd(const SsmArgs& a, unsigned grid, cudaStream_t st) {
    const size_t smem = sizeof(typename BwdShape<EL>::Smem);
    static SmemLimit limit;
    const cudaError_t e = limit.set(reinterpret_cast<const void*>(k_ssm_bwd<TI, EL>), (int)smem);
    if (e != cudaSuccess) return e;
    k_ssm_bwd<TI, EL><<<grid, SSM_T, smem, st>>>(a);
    return cudaSuccess;
}
template <typename TI, bool PIECES>
cudaError_t run_states(const SsmArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)(a.ax.rows * a.units_row) * ssm_channel_tiles(a.D, a.G);
    if (PIECES) {
        if (a.S <= 8) k_ssm_bwd_pieces<TI, 2><<<grid, SSM_T, 0, st>>>(a);
        else if (a.S <= 16) k_ssm_bwd_pieces<TI, 4><<<grid, SSM_T, 0, st>>>(a);
        else if (a.S <= 32) k_ssm_bwd_pieces<TI, 8><<<grid, SSM_T, 0, st>>>(a);
        else k_ssm_bwd_pieces<TI, 16><<<grid, SSM_T, 0, st>>>(a);
        return cudaSuccess;
    }
    if (a.S <= 8) return run_bwd<TI, 2>(a, grid, st);
    if (a.S <= 16) return run_bwd<TI, 4>(a, grid, st);
    if (a.S <= 32) return run_bwd<TI, 8>(a, grid, st);
    return run_bwd<TI, 16>(a, grid, st);
}

}  // namespace

int ssm_channel_tiles(int D, int G) { return (D / G + SSM_CH - 1) / SSM_CH * G; }

cudaError_t launch_ssm_bwd_pieces(const SsmArgs& a, int bf16, cudaStream_t st) {
    return traced_launch("k_ssm_bwd_pieces", st, [&] {
        bf16 ? run_states<__nv_bfloat16, true>(a, st) : run_states<float, true>(a, st);
    });
}

cudaError_t launch_ssm_bwd(const SsmArgs& a, int bf16, cudaStream_t st) {
    cudaError_t r = cudaSuccess;
    const cudaError_t e = traced_launch("k_ssm_bwd", st, [&] {
        r = bf16 ? run_states<__nv_bfloat16, false>(a, st) : run_states<float, false>(a, st);
    });
    return r != cudaSuccess ? r : e;
}

cudaError_t launch_ssm_bwd_sums(const SsmArgs& a, int bf16, cudaStream_t st) {
    const size_t bc = (size_t)a.ax.rows * a.ax.len * 2 * a.G * a.S, params = (size_t)a.D * (a.S + 2);
    const unsigned nbc = (unsigned)((bc + 255) / 256), np = (unsigned)((params + 255) / 256);
    return traced_launch("k_ssm_sums", st, [&] {
        if (bf16) k_ssm_sums<__nv_bfloat16><<<nbc + np, 256, 0, st>>>(a, nbc);
        else k_ssm_sums<float><<<nbc + np, 256, 0, st>>>(a, nbc);
    });
}

}  // namespace kda
