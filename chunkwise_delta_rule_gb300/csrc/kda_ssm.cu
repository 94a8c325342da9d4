// Selective state space scan (diagonal, input-dependent step), forward:
//     delta = softplus(dt + dt_bias),  a = exp(-delta exp(A_log)),  u = delta x
//     h_t = a h_{t-1} + u B_t,   y_t = (sum_n C_t[n] h_t[n] + d_skip x_t) silu(z_t)
// Four lanes share a channel and hold its states in registers; a CTA walks 32 channels
// through a time piece in tiles of 32 tokens. Four warps run the recurrence, four
// others work around it, so that the recurrence never waits for them: while tile k
// runs they copy tiles ahead into shared memory (asynchronously, each thread its own 8
// channels of one token and 8 states of one row), form tile k + 1's steps once per
// (token, channel), and sum, gate and store tile k - 1's outputs. One barrier per tile.
// Per four states and token the recurrence takes 4 exponentials (16 cycles of a
// scheduler's share at 32 per cycle and SM) and 8 paired multiply-adds (16 cycles):
// both pipes are full, which bounds the kernel, not memory.
// A long row is cut into time pieces when its channels alone do not fill the GPU:
// a first pass forms each piece's end state from zero and its sum of delta (the
// piece's decay is exp(A sum delta)); in the second pass each piece joins the
// states of the pieces before it and runs its outputs.
#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int TT = 32;   // tokens per tile

enum { OUT = 0, OUT_CKPT = 1, CKPT = 2, PIECE = 3 };

constexpr int FT = 2 * SSM_T;   // threads: 128 for the recurrence, 128 around it

template <typename TI, int EL, int MODE>
struct FwdShape {
    static constexpr int NP = 4 * EL;
    static constexpr bool HAS_Y = MODE == OUT || MODE == OUT_CKPT, HAS_CK = MODE == OUT_CKPT || MODE == CKPT;
    static constexpr int ROWS = HAS_Y ? 2 * TT : TT;                    // rows of b (and c) in a tile
    static constexpr int NBC = (ROWS * (NP / 8) + SSM_T - 1) / SSM_T;   // their chunks of 8 per thread
    static constexpr int NTOK = HAS_Y ? 3 : 2;                          // x, dt (and z)
    // tiles in flight: the previous (its x and z), the current, the next, and those copied ahead
    static constexpr int STAGES = sizeof(TI) == 2 ? (NP <= 32 ? 6 : 5) : (NP <= 16 ? 5 : 4);
    struct Smem {
        TI raw[STAGES][NTOK + NBC][SSM_T][8];
        float4 du[2][TT][SSM_CH / 2];          // (delta, u) of two channels; see du_at
        float b[2][TT][NP];
        float c[2][HAS_Y ? TT : 1][NP];
        float y[2][HAS_Y ? TT : 1][SSM_CH][4]; // the four lanes' parts; see y_at
    };
};

// Places of channel pairs and of channels in a token's row, permuted so that the eight threads of a quarter warp that
// hold (two tokens) x (four groups of 8 channels) reach distinct banks.
__device__ __forceinline__ int du_at(int tok, int pair) { return pair ^ ((pair >> 3) | (tok & 1) << 1); }
__device__ __forceinline__ int y_at(int tok, int ch) { return ch ^ ((ch >> 3) | (tok & 1) << 2); }

template <typename TI, int EL, int MODE>
__global__ void __launch_bounds__(FT, 2) k_ssm_fwd(SsmArgs a) {
    using Sh = FwdShape<TI, EL, MODE>;
    constexpr int NP = Sh::NP, NBC = Sh::NBC, STAGES = Sh::STAGES, P = EL / 2;
    constexpr bool HAS_Y = Sh::HAS_Y, HAS_CK = Sh::HAS_CK;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    typename Sh::Smem& sm = *reinterpret_cast<typename Sh::Smem*>(smem_raw);
    if (blockIdx.x == 0 && MODE != PIECE) axis_check(a.ax, a.err);
    const SsmPlace pl = ssm_place<SSM_CH>(a);
    const size_t tok0 = (size_t)pl.row * a.ax.len;
    const size_t DS = (size_t)a.D * a.S;
    int t = pl.lo;
    Seq s{0, 0, 0};
    if (pl.lo < pl.hi || !a.ax.cu) {
        if (MODE == PIECE) {
            // the part of the piece that reaches past its end
            s = seq_at(a.ax, pl.row, pl.hi - 1);
            if (s.end <= pl.hi) return;
            t = max(pl.lo, s.first);
        } else {
            s = seq_at(a.ax, pl.row, t);
        }
    }
    const int first_tile = t, ntiles = (pl.hi - t + TT - 1) / TT;
    const int tid = threadIdx.x & (SSM_T - 1);

    if (threadIdx.x >= SSM_T) {
        // ---------------------------------------------------------------- around the recurrence
        // this thread's part of a tile: one token, 8 channels; NBC chunks of 8 states of b's and c's rows
        const int ptok = tid >> 2, pc = (tid & 3) * 8, pvalid = pl.nch - pc;
        const TI* xp = static_cast<const TI*>(a.x) + tok0 * a.ldx + pl.c0 + pc;
        const TI* dp = static_cast<const TI*>(a.dt) + tok0 * a.lddt + pl.c0 + pc;
        const TI* zp = a.z ? static_cast<const TI*>(a.z) + tok0 * a.ldz + pl.c0 + pc : nullptr;
        const TI* bp = static_cast<const TI*>(a.b) + tok0 * a.ldb + (size_t)pl.g * a.S;
        const TI* cp = static_cast<const TI*>(a.c) + tok0 * a.ldc + (size_t)pl.g * a.S;
        constexpr int NC = NP / 8;
        auto fetch = [&](int k) {   // tile k of the piece into its stage
            const int tb = first_tile + k * TT;
            if (k < ntiles) {
                TI(*raw)[SSM_T][8] = sm.raw[k % STAGES];
                const size_t tt = min(tb + ptok, pl.hi - 1);
                const int n = tb + ptok < pl.hi ? pvalid : 0;
                copy8_async(raw[0][tid], xp + tt * a.ldx, n, a.how >> SSM_X & 3);
                copy8_async(raw[1][tid], dp + tt * a.lddt, n, a.how >> SSM_DT & 3);
                if (HAS_Y && zp) copy8_async(raw[2][tid], zp + tt * a.ldz, n, a.how >> SSM_Z & 3);
#pragma unroll
                for (int j = 0; j < NBC; ++j) {
                    const int i = tid + j * SSM_T;
                    if (i >= Sh::ROWS * NC) break;
                    const bool isc = i >= TT * NC;
                    const int r = isc ? i - TT * NC : i, tok = r / NC, k8 = (r - tok * NC) * 8;
                    const size_t tr = min(tb + tok, pl.hi - 1);
                    const int m = tb + tok < pl.hi ? a.S - k8 : 0;
                    const TI* src = isc ? cp + tr * a.ldc : bp + tr * a.ldb;
                    copy8_async(raw[Sh::NTOK + j][tid], src + (m > 0 ? k8 : 0), m, a.how >> (isc ? SSM_C : SSM_B) & 3);
                }
            }
            copies_commit();
        };
        for (int k = 0; k < STAGES - 2; ++k) fetch(k);
        float bias[8], skip[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            bias[i] = a.dt_bias && i < pvalid ? a.dt_bias[pl.c0 + pc + i] : 0.f;
            skip[i] = HAS_Y && a.d_skip && i < pvalid ? a.d_skip[pl.c0 + pc + i] : 0.f;
        }
        // step k: tile k + 1's steps, tile k - 1's outputs (k = -1: the first tile's steps alone)
        for (int k = -1; k <= ntiles; ++k) {
            if (k + 1 < ntiles) {
                const int w = (k + 1) & 1;
                copies_wait<STAGES - 3>();
                TI(*raw)[SSM_T][8] = sm.raw[(k + 1) % STAGES];
                float x[8], dt[8];
                load_row<8>(raw[0][tid], x, 8, true);
                load_row<8>(raw[1][tid], dt, 8, true);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    float2 dl = make_float2(dt[i] + bias[i], dt[i + 1] + bias[i + 1]);
                    if (a.softplus) dl = ssm_softplus2(dl);
                    const float2 u = mul2(dl, make_float2(x[i], x[i + 1]));
                    sm.du[w][ptok][du_at(ptok, (pc + i) >> 1)] = make_float4(dl.x, u.x, dl.y, u.y);
                }
#pragma unroll
                for (int j = 0; j < NBC; ++j) {
                    const int i = tid + j * SSM_T;
                    if (i >= Sh::ROWS * NC) break;
                    const bool isc = i >= TT * NC;
                    const int r = isc ? i - TT * NC : i, tok = r / NC, k8 = (r - tok * NC) * 8;
                    float v[8];
                    load_row<8>(raw[Sh::NTOK + j][tid], v, 8, true);
                    float4* dst = reinterpret_cast<float4*>(isc ? &sm.c[w][HAS_Y ? tok : 0][k8] : &sm.b[w][tok][k8]);
                    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                }
            }
            if (HAS_Y && k > 0) {
                const int tok = first_tile + (k - 1) * TT + ptok, w = (k - 1) & 1;
                if (tok < pl.hi && pvalid > 0) {
                    TI(*raw)[SSM_T][8] = sm.raw[(k - 1) % STAGES];
                    float o[8], x[8], z[8];
                    load_row<8>(raw[0][tid], x, 8, true);
                    if (zp) load_row<8>(raw[HAS_Y ? 2 : 0][tid], z, 8, true);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 v = *reinterpret_cast<const float4*>(sm.y[w][HAS_Y ? ptok : 0][y_at(ptok, pc + i)]);
                        o[i] = fmaf(skip[i], x[i], (v.x + v.y) + (v.z + v.w));
                        if (zp) o[i] *= z[i] * sigmoid_fast(z[i]);
                    }
                    store_row<8>(static_cast<TI*>(a.y) + (tok0 + tok) * a.D + pl.c0 + pc, o, pvalid,
                                 pvalid >= 8 && !(a.how >> SSM_OUT & 3));
                }
            }
            fetch(k + STAGES - 1);   // into the stage of tile k - 1, which was read last
            if (k < ntiles) __syncthreads();
        }
        return;
    }

    // -------------------------------------------------------------------- the recurrence
    const int l = tid & 3, ch = tid >> 2, n0 = l * EL, d = pl.c0 + ch;
    const bool on = ch < pl.nch;
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
        for (int n = pl.unit; n < a.ax.N; n += pl.units) {
            if (axis_cu(a.ax, n + 1) > axis_cu(a.ax, n)) continue;
            init_state(n);
            store_states<EL>(ht + n * DS, n0, a.S, on, h);
        }
    }
    // the state entering this piece
    if (MODE == PIECE ? s.first >= pl.lo : t == s.first) {
        init_state(s.n);
    } else {
#pragma unroll
        for (int e = 0; e < EL; ++e) h[e] = 0.f;
        if (MODE != PIECE) {
            // the earlier pieces of its sequence, joined in order
            const int q = s.first / a.unit_len;
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
    constexpr int N = EL <= 4 ? 4 : 16 / EL;   // tokens whose operands are in registers together
    struct Operands {
        float2 du[N], b[N][P], c[HAS_Y ? N : 1][P];
    };
    auto load = [&](int w, int i, int n, Operands& o) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (j >= n) break;
            o.du[j] = reinterpret_cast<const float2*>(&sm.du[w][i + j][du_at(i + j, ch >> 1)])[ch & 1];
            float v[EL];
            lds_states<EL>(&sm.b[w][i + j][n0], v);
#pragma unroll
            for (int e = 0; e < P; ++e) o.b[j][e] = make_float2(v[2 * e], v[2 * e + 1]);
            if (HAS_Y) {
                lds_states<EL>(&sm.c[w][HAS_Y ? i + j : 0][n0], v);
#pragma unroll
                for (int e = 0; e < P; ++e) o.c[HAS_Y ? j : 0][e] = make_float2(v[2 * e], v[2 * e + 1]);
            }
        }
    };
    auto run_tokens = [&](int w, int i, int n, const Operands& o) {
        float2 acc[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (j >= n) break;
            const float2 dl = make_float2(o.du[j].x, o.du[j].x), u = make_float2(o.du[j].y, o.du[j].y);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float2 g = mul2(dl, make_float2(A2[2 * e], A2[2 * e + 1]));
                const float2 hn = fma2(make_float2(ex2(g.x), ex2(g.y)), make_float2(h[2 * e], h[2 * e + 1]), mul2(u, o.b[j][e]));
                h[2 * e] = hn.x;
                h[2 * e + 1] = hn.y;
                if (HAS_Y) acc[j] = e == 0 ? mul2(hn, o.c[HAS_Y ? j : 0][e]) : fma2(hn, o.c[HAS_Y ? j : 0][e], acc[j]);
            }
            if (MODE == PIECE) sd += o.du[j].x;
        }
        if (HAS_Y) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j < n) sm.y[w][HAS_Y ? i + j : 0][y_at(i + j, ch)][l] = acc[j].x + acc[j].y;
        }
    };
    auto checkpoint = [&](int tok) {
        const size_t slot = (size_t)pl.row * ((a.ax.len + SSM_CKPT - 1) / SSM_CKPT) + tok / SSM_CKPT;
        store_states<EL>(a.ckpt + slot * DS + (size_t)d * a.S, n0, a.S, on, h);
    };
    __syncthreads();   // the first tile's steps
    for (int k = 0; k < ntiles; ++k) {
        const int tb = first_tile + k * TT, te = min(tb + TT, pl.hi), w = k & 1;
        t = tb;
        if (MODE != PIECE && t == s.end) {
            if (ht) store_states<EL>(ht + s.n * DS, n0, a.S, on, h);
            s = seq_at(a.ax, pl.row, t);
            init_state(s.n);
        }
        if (te - tb == TT && (MODE == PIECE || s.end >= te)) {
            // a whole tile of one sequence: the next tokens' operands are read while these run
            Operands o[2];
            load(w, 0, N, o[0]);
#pragma unroll
            for (int i = 0; i < TT; i += N) {
                if (HAS_CK && i % SSM_CKPT == 0) checkpoint(tb + i);
                if (i + N < TT) load(w, i + N, N, o[(i / N + 1) & 1]);
                run_tokens(w, i, N, o[(i / N) & 1]);
            }
        } else {
            while (t < te) {
                if (MODE != PIECE && t == s.end) {
                    if (ht) store_states<EL>(ht + s.n * DS, n0, a.S, on, h);
                    s = seq_at(a.ax, pl.row, t);
                    init_state(s.n);
                }
                if (HAS_CK && t % SSM_CKPT == 0) checkpoint(t);
                int run = MODE == PIECE ? te : min(te, s.end);
                if (HAS_CK) run = min(run, (t | (SSM_CKPT - 1)) + 1);
                Operands o;
                if (t + N <= run) {
                    load(w, t - tb, N, o);
                    run_tokens(w, t - tb, N, o);
                    t += N;
                } else {
                    load(w, t - tb, 1, o);
                    run_tokens(w, t - tb, 1, o);
                    ++t;
                }
            }
        }
        __syncthreads();
    }
    if (pl.lo >= pl.hi && a.ax.cu) return;
    if (MODE == PIECE) {
        store_states<EL>(a.hloc + pl.unit * DS + (size_t)d * a.S, n0, a.S, on, h);
        if (on && l == 0) a.sdt[(size_t)pl.unit * a.D + d] = sd;
    } else if (ht && pl.hi == s.end) {
        store_states<EL>(ht + s.n * DS, n0, a.S, on, h);
    }
}

// A lane's EL states of a row of b or c: one access of EL elements where the row is aligned to it.
template <int EL, typename TI>
__device__ __forceinline__ void load_lane(const TI* p, int n, bool aligned, float (&x)[EL]) {
    if (aligned && n >= EL && EL >= 4) {
        struct alignas(sizeof(TI) * EL > 16 ? 16 : sizeof(TI) * EL) Pack { TI v[EL]; };
        const Pack k = *reinterpret_cast<const Pack*>(p);
#pragma unroll
        for (int e = 0; e < EL; ++e) x[e] = ld(&k.v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < EL; ++e) x[e] = e < n ? ld(p + e) : 0.f;
    }
}

// A few tokens of each sequence (decoding): the state is the traffic, 8 bytes per value against 8 per channel for the
// token. The same four lanes per channel, NS sequences per thread so that their states are in flight together and A is
// formed once; everything is read directly, and after the exchange over the four lanes lane i holds sequence i's output.
template <typename TI, int EL, int NS>
__global__ void __launch_bounds__(SSM_T) k_ssm_step(SsmArgs a) {
    static_assert(NS == 1 || NS == 4, "sequences per thread");
    const int M = a.D / a.G, tpg = (M + SSM_CH - 1) / SSM_CH, tiles = tpg * a.G;
    const int sb = blockIdx.x / tiles, tile = blockIdx.x - sb * tiles, g = tile / tpg, tg = tile - g * tpg;
    const int l = threadIdx.x & 3, ch = threadIdx.x >> 2, n0 = l * EL, d = g * M + tg * SSM_CH + ch;
    const bool on = ch < M - tg * SSM_CH;
    const size_t DS = (size_t)a.D * a.S;
    const int B = a.ax.N, T = a.ax.len, s0 = sb * NS;
    float A2[EL], h[NS][EL];
    load_states<EL>(a.A_log + (size_t)d * a.S, n0, a.S, on, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        if (a.h0 && s0 + i < B) {
            load_states<EL>(a.h0 + (s0 + i) * DS + (size_t)d * a.S, n0, a.S, on, h[i]);
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) h[i][e] = 0.f;
        }
    }
    const float bias = a.dt_bias && on ? a.dt_bias[d] : 0.f, skip = a.d_skip && on ? a.d_skip[d] : 0.f;
    for (int t = 0; t < T; ++t) {
        float x[NS], dt[NS], b[NS][EL], c[NS][EL], acc[NS];
        const int mine = s0 + (NS == 4 ? l : 0);   // the sequence whose output this lane stores
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const bool in = on && s0 + i < B;
            const size_t tok = (size_t)(s0 + i) * T + t;
            x[i] = in ? ld(static_cast<const TI*>(a.x) + tok * a.ldx + d) : 0.f;
            dt[i] = in ? ld(static_cast<const TI*>(a.dt) + tok * a.lddt + d) : 0.f;
            const int n = s0 + i < B ? a.S - n0 : 0;
            load_lane<EL>(static_cast<const TI*>(a.b) + tok * a.ldb + (size_t)g * a.S + n0, n, !(a.how >> SSM_B & 3), b[i]);
            load_lane<EL>(static_cast<const TI*>(a.c) + tok * a.ldc + (size_t)g * a.S + n0, n, !(a.how >> SSM_C & 3), c[i]);
        }
        const bool store = on && mine < B && (NS == 4 || l == 0);
        if (a.z && store) z = ld(static_cast<const TI*>(a.z) + ((size_t)mine * T + t) * a.ldz + d);
        if (t == 0) {
#pragma unroll
            for (int e = 0; e < EL; ++e) A2[e] = on && n0 + e < a.S ? -expf(A2[e]) * LOG2E : 0.f;
        }
        float xm = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float dl = dt[i] + bias;
            if (a.softplus) dl = ssm_softplus(dl);
            const float u = dl * x[i];
            acc[i] = 0.f;
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                h[i][e] = fmaf(ex2(dl * A2[e]), h[i][e], u * b[i][e]);
                acc[i] = fmaf(h[i][e], c[i][e], acc[i]);
            }
            if (i == 0 || l == i) xm = x[i];
        }
        if (NS == 4) {
            halve<4>(acc, l, 2);
            halve<2>(acc, l, 1);
        } else {
            acc[0] += __shfl_xor_sync(SSM_FULL, acc[0], 2);
            acc[0] += __shfl_xor_sync(SSM_FULL, acc[0], 1);
        }
        if (store) {
            float o = fmaf(skip, xm, acc[0]);
            if (a.z) o *= z * sigmoid_fast(z);
            st(static_cast<TI*>(a.y) + ((size_t)mine * T + t) * a.D + d, o);
        }
    }
    if (a.ht) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (s0 + i < B) store_states<EL>(a.ht + (s0 + i) * DS + (size_t)d * a.S, n0, a.S, on, h[i]);
    }
}

int fwd_tiles(int D, int G) { return (D / G + SSM_CH - 1) / SSM_CH * G; }

template <typename TI, int EL>
void run_step(const SsmArgs& a, cudaStream_t st) {
    const unsigned tiles = fwd_tiles(a.D, a.G);
    // four sequences per thread once that still leaves every SM two CTAs
    if ((long long)tiles * (a.ax.N / 4) >= 2 * sm_count()) k_ssm_step<TI, EL, 4><<<tiles * ((a.ax.N + 3) / 4), SSM_T, 0, st>>>(a);
    else k_ssm_step<TI, EL, 1><<<tiles * a.ax.N, SSM_T, 0, st>>>(a);
}

template <typename TI, int EL, int MODE>
cudaError_t run_one(const SsmArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)(a.ax.rows * a.units_row) * fwd_tiles(a.D, a.G);
    const int smem = (int)sizeof(typename FwdShape<TI, EL, MODE>::Smem);
    static SmemLimit limit;
    const cudaError_t e = limit.set(reinterpret_cast<const void*>(k_ssm_fwd<TI, EL, MODE>), smem);
    if (e != cudaSuccess) return e;
    k_ssm_fwd<TI, EL, MODE><<<grid, FT, smem, st>>>(a);
    return cudaSuccess;
}
template <typename TI, int EL>
cudaError_t run_mode(const SsmArgs& a, int mode, cudaStream_t st) {
    switch (mode) {
        case OUT: return run_one<TI, EL, OUT>(a, st);
        case OUT_CKPT: return run_one<TI, EL, OUT_CKPT>(a, st);
        case CKPT: return run_one<TI, EL, CKPT>(a, st);
        default: return run_one<TI, EL, PIECE>(a, st);
    }
}
template <typename TI>
cudaError_t run_states(const SsmArgs& a, int mode, cudaStream_t st) {
    if (a.S <= 8) return run_mode<TI, 2>(a, mode, st);
    if (a.S <= 16) return run_mode<TI, 4>(a, mode, st);
    if (a.S <= 32) return run_mode<TI, 8>(a, mode, st);
    return run_mode<TI, 16>(a, mode, st);
}
template <typename TI>
void run_step_states(const SsmArgs& a, cudaStream_t st) {
    if (a.S <= 8) run_step<TI, 2>(a, st);
    else if (a.S <= 16) run_step<TI, 4>(a, st);
    else if (a.S <= 32) run_step<TI, 8>(a, st);
    else run_step<TI, 16>(a, st);
}
// Tokens per sequence up to which everything is read directly: past it the tiles' prefetch pays.
constexpr int STEP_TOKENS = 4;

cudaError_t launch(const char* name, const SsmArgs& a, int bf16, int mode, cudaStream_t st) {
    cudaError_t r = cudaSuccess;
    const cudaError_t e = traced_launch(name, st, [&] {
        r = bf16 ? run_states<__nv_bfloat16>(a, mode, st) : run_states<float>(a, mode, st);
    });
    return r != cudaSuccess ? r : e;
}

}  // namespace

int ssm_units(int rows, int len, int D, int G, int S, bool backward) {
    // pieces only while the channels and rows alone leave SMs idle; a piece is at least 128 tokens
    const long long ctas = (long long)rows * (backward ? ssm_bwd_tiles(D, G, S) : fwd_tiles(D, G));
    const long long full = backward ? 2 * sm_count() / 3 : sm_count(), want = (backward ? 2LL : 4LL) * sm_count();
    long long units = ctas >= full ? 1 : want / ctas;
    const long long most = (len + 127) / 128;
    if (units > most) units = most;
    return units < 1 ? 1 : (int)units;
}

cudaError_t launch_ssm_fwd(const SsmArgs& a, int bf16, int mode, cudaStream_t st) {
    if (mode == OUT && !a.ax.cu && a.ax.len > 0 && a.ax.len <= STEP_TOKENS)
        return traced_launch("k_ssm_step", st, [&] {
            bf16 ? run_step_states<__nv_bfloat16>(a, st) : run_step_states<float>(a, st);
        });
    return launch(mode == CKPT ? "k_ssm_ckpt" : "k_ssm_fwd", a, bf16, mode, st);
}

cudaError_t launch_ssm_pieces(const SsmArgs& a, int bf16, cudaStream_t st) {
    return launch("k_ssm_pieces", a, bf16, PIECE, st);
}

}  // namespace kda
