// Selective state space scan, backward. With d0_t = dy_t silu(z_t), A = -exp(A_log),
// a_t = exp(delta_t A) and g_t the adjoint of h_t:
//     g_t = C_t d0_t + a_{t+1} g_{t+1}
//     dC_t = sum_d d0 h,  dB_t = sum_d u g,  s1 = sum_n g B,  s2 = sum_n A a g h_{t-1}
//     dx = delta s1 + d_skip d0,  ddelta = x s1 + s2,  dA = sum_t delta a g h_{t-1}
//     dz = dy y0 silu'(z) with y0 = sum_n C h + d_skip x,  dh0 = a_1 g_1
// A CTA walks its channels backwards through a time piece in tiles of 16 tokens. Eight
// warps (four for more than 16 states) run the recurrences, four lanes per channel:
// the states inside a tile are recomputed from the checkpoint the forward left at its
// first token and held in registers (L tokens at a time), then the adjoint runs over
// them. Four others work around them, one tile apart, as in the forward: they copy
// tiles ahead, form the steps and gated gradients, and turn s1, s2 and sum C h into dx,
// ddelta and dz. dB and dC are summed over a warp's channels by
// halving exchanges, over the CTA's warps in shared memory and over the CTAs' rows in
// a second kernel, in a fixed order; the parameters' gradients go the same way, so
// nothing depends on timing.
// Measured, four rows of 2048 tokens, 2048 channels of 16 states, bf16: 418 us (and 16
// for the second kernel), beside a floor of 55 us for the bytes and about 100 for the
// multiply-adds. As in the forward the bound is instruction dispatch (0.63 instructions
// per cycle on the busiest scheduler, a fifth of them paired ones that hold it twice):
// about 45 instructions per token of a warp's adjoint, 27 for recomputing its states 1.5
// times (L = 8 of 16 tokens at once), 16 for the sums over channels (28 before the
// states' order made their choices unnecessary: 458 to 427 us).
#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int TB = SSM_CKPT;   // tokens per tile
constexpr int HT = 128;        // threads around the recurrences

template <typename TI, int EL>
struct BwdShape {
    static constexpr int NP = 4 * EL, P = EL / 2;
    static constexpr int RT = EL <= 4 ? 256 : 128;        // threads of the recurrences
    static constexpr int CH = RT / 4, RW = RT / 32;       // their channels, their warps
    static constexpr int CP = CH / 8;                     // channels of a token per thread around them
    // tokens whose states are held at once: more would save recomputed steps, but the unrolled loop over them (about 100
    // instructions each) has to stay in the instruction cache
    static constexpr int L = EL <= 4 ? 8 : 64 / EL;
    static constexpr int NSUB = TB / L;
    static constexpr int KEEP = EL >= 4 ? EL / 4 : 1;     // dB and dC values a lane holds after the sum over 8 channels
    // copies of the rows b and c, each in an order of its own inside four states (see the sums over channels)
    static constexpr int NVER = EL == 4 ? 4 : EL == 16 ? 1 : 2;
    static constexpr int NBC = (TB * 2 * (NP / 8) + HT - 1) / HT;   // chunks of 8 states of b and c per thread
    static constexpr int STAGES = 5;                      // tiles: the one after, the present, the one before, two on their way
    struct Smem {
        TI tok[STAGES][4][HT][CP];            // x, dt, dy, z
        TI bc[STAGES][NBC][HT][8];
        float4 in[2][TB][CH + CH / 8];               // delta, u, d0
        float4 out[2][TB][CH + CH / 8];              // s1, s2 (in log2 units), sum C h
        float b[2][NVER][TB * NP + 16], c[2][NVER][TB * NP + 16];   // the copies start in other banks
        float red[2][RW][TB][2 * NP];
        float sub[NSUB > 1 ? NSUB - 1 : 1][EL][RT];
    };
};

// Place of a channel in a token's row, spaced so that the eight threads of a quarter warp, of eight (or four)
// neighbouring channels each, reach distinct banks.
__device__ __forceinline__ int in_at(int ch) { return ch + (ch >> 3); }

__device__ __forceinline__ void named_barrier(int id, int count) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

template <typename TI, int EL>
__global__ void __launch_bounds__(BwdShape<TI, EL>::RT + HT, 1) k_ssm_bwd(SsmArgs a) {
    using Sh = BwdShape<TI, EL>;
    constexpr int NP = Sh::NP, P = Sh::P, RT = Sh::RT, CH = Sh::CH, RW = Sh::RW, CP = Sh::CP, L = Sh::L, NSUB = Sh::NSUB,
                  KEEP = Sh::KEEP, NVER = Sh::NVER, NBC = Sh::NBC, STAGES = Sh::STAGES;
    extern __shared__ __align__(16) unsigned char raw_smem[];
    typename Sh::Smem& sm = *reinterpret_cast<typename Sh::Smem*>(raw_smem);
    if (blockIdx.x == 0) axis_check(a.ax, a.err);
    const SsmPlace pl = ssm_place<CH>(a);
    const size_t tok0 = (size_t)pl.row * a.ax.len;
    const size_t DS = (size_t)a.D * a.S;
    // tile k = 0 is the piece's last one
    const int ntiles = (pl.hi - pl.lo + TB - 1) / TB;
    auto tile_begin = [&](int k) { return pl.lo + (ntiles - 1 - k) * TB; };

    if (threadIdx.x >= RT) {
        // ---------------------------------------------------------------- around the recurrences
        const int tid = threadIdx.x - RT;
        const int ptok = tid >> 3, pc = (tid & 7) * CP, pvalid = pl.nch - pc;   // one token, CP channels
        const size_t ld[4] = {a.ldx, a.lddt, (size_t)a.D, a.ldz};
        constexpr int SHIFT[4] = {SSM_X, SSM_DT, SSM_DY, SSM_Z};
        const bool gate = a.z != nullptr;
        constexpr int NC = NP / 8;
        // the rows of the next tile to fetch (tiles run backwards); whole ones of a whole tile need no checks
        const int first = tile_begin(0);
        const TI *tok_src[4], *bc_src[NBC];
        bool whole_rows = pvalid >= CP;
        auto input = [&](int q) { return q == 0 ? a.x : q == 1 ? a.dt : q == 2 ? a.dy : a.z; };
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            tok_src[q] = static_cast<const TI*>(input(q)) + (tok0 + first + ptok) * ld[q] + pl.c0 + pc;
            whole_rows = whole_rows && ((q == 3 && !gate) || !(a.how >> SHIFT[q] & 3));
        }
#pragma unroll
        for (int j = 0; j < NBC; ++j) {
            const int i = tid + j * HT, isc = i >= TB * NC, r = isc ? i - TB * NC : i, tok = r / NC, k8 = (r - tok * NC) * 8;
            bc_src[j] = static_cast<const TI*>(isc ? a.c : a.b) + (tok0 + first + tok) * (isc ? a.ldc : a.ldb) + (size_t)pl.g * a.S + k8;
            whole_rows = whole_rows && (i >= 2 * TB * NC || (k8 + 8 <= a.S && !(a.how >> (isc ? SSM_C : SSM_B) & 3)));
        }
        auto fetch = [&](int k) {
            const int tb = tile_begin(k), st = k % STAGES;
            if (k < ntiles && whole_rows && tb + TB <= pl.hi) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (q < 3 || gate) copy_whole_async<TI, CP>(sm.tok[st][q][tid], tok_src[q]);
#pragma unroll
                for (int j = 0; j < NBC; ++j)
                    if (tid + j * HT < 2 * TB * NC) copy_whole_async<TI, 8>(sm.bc[st][j][tid], bc_src[j]);
            } else if (k < ntiles) {
                // a row that is not there is a copy of no bytes from its own tensor's start: the access that `how` names has
                // to be aligned all the same, and another tensor's start need not be
                const int n = tb + ptok < pl.hi ? pvalid : 0;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (q < 3 || gate)
                        copy_row_async<TI, CP>(sm.tok[st][q][tid], n > 0 ? tok_src[q] : static_cast<const TI*>(input(q)), n, a.how >> SHIFT[q] & 3);
#pragma unroll
                for (int j = 0; j < NBC; ++j) {
                    const int i = tid + j * HT;
                    if (i >= 2 * TB * NC) break;
                    const bool isc = i >= TB * NC;
                    const int r = isc ? i - TB * NC : i, tok = r / NC, k8 = (r - tok * NC) * 8;
                    const int m = tb + tok < pl.hi ? a.S - k8 : 0;
                    copy8_async(sm.bc[st][j][tid], m > 0 ? bc_src[j] : static_cast<const TI*>(isc ? a.c : a.b), m, a.how >> (isc ? SSM_C : SSM_B) & 3);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) tok_src[q] -= TB * ld[q];
#pragma unroll
            for (int j = 0; j < NBC; ++j) bc_src[j] -= TB * (tid + j * HT >= TB * NC ? a.ldc : a.ldb);
            copies_commit();
        };
        for (int k = 0; k < STAGES - 2; ++k) fetch(k);
        // of dB and dC each thread sums one state's (or row's) place over the warps, for every ROWS-th token
        constexpr int ROWS = HT / (2 * NP);
        const int sum_f = tid % (2 * NP), sum_tok = tid / (2 * NP), sum_n = sum_f % NP;
        float* sums = a.pbc + ((pl.tile * (size_t)a.ax.rows * a.ax.len + tok0 + first + sum_tok) * 2 + sum_f / NP) * a.S + sum_n;
        float bias[CP], skip[CP], dskip[CP], dbias[CP];
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            bias[i] = a.dt_bias && i < pvalid ? a.dt_bias[pl.c0 + pc + i] : 0.f;
            skip[i] = a.d_skip && i < pvalid ? a.d_skip[pl.c0 + pc + i] : 0.f;
            dskip[i] = dbias[i] = 0.f;
        }
        // step k: tile k - 1's outputs, tile k + 1's inputs (in the place of tile k - 1's)
        for (int k = -1; k <= ntiles; ++k) {
            if (k > 0) {
                const int w = (k - 1) & 1, st = (k - 1) % STAGES, tb = tile_begin(k - 1), nt = min(TB, pl.hi - tb);
                if (ptok < nt && pvalid > 0) {
                    float x[CP], dt[CP], dy[CP], z[CP], ox[CP], od[CP], oz[CP];
                    load_row<CP>(sm.tok[st][0][tid], x, CP, true);
                    load_row<CP>(sm.tok[st][1][tid], dt, CP, true);
                    load_row<CP>(sm.tok[st][2][tid], dy, CP, true);
                    if (gate) load_row<CP>(sm.tok[st][3][tid], z, CP, true);
#pragma unroll
                    for (int i = 0; i < CP; ++i) {
                        const float4 in = sm.in[w][ptok][in_at(pc + i)];
                        const float4 v = sm.out[w][ptok][in_at(pc + i)];
                        const float y0 = fmaf(skip[i], x[i], v.z);
                        ox[i] = fmaf(in.x, v.x, skip[i] * in.z);
                        od[i] = fmaf(x[i], v.x, v.y * (1.f / LOG2E));
                        if (a.softplus) od[i] *= sigmoid_fast(dt[i] + bias[i]);
                        if (gate) {
                            const float sg = sigmoid_fast(z[i]);
                            oz[i] = dy[i] * y0 * sg * fmaf(z[i], 1.f - sg, 1.f);
                        }
                        if (i < pvalid) {
                            dskip[i] = fmaf(in.z, x[i], dskip[i]);
                            dbias[i] += od[i];
                        }
                    }
                    const size_t o = (tok0 + tb + ptok) * a.D + pl.c0 + pc;
                    const bool whole = pvalid >= CP && !(a.how >> SSM_OUT & 3);
                    store_part<TI, CP>(static_cast<TI*>(a.dx) + o, ox, pvalid, whole);
                    store_part<TI, CP>(static_cast<TI*>(a.ddt) + o, od, pvalid, whole);
                    if (gate) store_part<TI, CP>(static_cast<TI*>(a.dz) + o, oz, pvalid, whole);
                }
#pragma unroll
                for (int j = 0; j < TB; j += ROWS) {
                    float v = 0.f;
#pragma unroll
                    for (int r = 0; r < RW; ++r) v += sm.red[w][r][j + sum_tok][sum_f];
                    if (j + sum_tok < nt && sum_n < a.S) sums[(size_t)j * 2 * a.S] = v;
                }
                sums -= (size_t)TB * 2 * a.S;
            }
            if (k + 1 < ntiles) {
                const int w = (k + 1) & 1, st = (k + 1) % STAGES;
                copies_wait<STAGES - 3>();
                float x[CP], dt[CP], dy[CP], z[CP];
                load_row<CP>(sm.tok[st][0][tid], x, CP, true);
                load_row<CP>(sm.tok[st][1][tid], dt, CP, true);
                load_row<CP>(sm.tok[st][2][tid], dy, CP, true);
                if (gate) load_row<CP>(sm.tok[st][3][tid], z, CP, true);
#pragma unroll
                for (int i = 0; i < CP; i += 2) {
                    float2 dl = make_float2(dt[i] + bias[i], dt[i + 1] + bias[i + 1]);
                    if (a.softplus) dl = ssm_softplus2(dl);
                    const float2 u = mul2(dl, make_float2(x[i], x[i + 1]));
                    float2 d0 = make_float2(dy[i], dy[i + 1]);
                    if (gate) d0 = make_float2(d0.x * z[i] * sigmoid_fast(z[i]), d0.y * z[i + 1] * sigmoid_fast(z[i + 1]));
                    sm.in[w][ptok][in_at(pc + i)] = make_float4(dl.x, u.x, d0.x, 0.f);
                    sm.in[w][ptok][in_at(pc + i + 1)] = make_float4(dl.y, u.y, d0.y, 0.f);
                }
#pragma unroll
                for (int j = 0; j < NBC; ++j) {
                    const int i = tid + j * HT;
                    if (i >= 2 * TB * NC) break;
                    const bool isc = i >= TB * NC;
                    const int r = isc ? i - TB * NC : i, tok = r / NC, k8 = (r - tok * NC) * 8;
                    float v[8];
                    load_row<8>(sm.bc[st][j][tid], v, 8, true);
#pragma unroll
                    for (int ver = 0; ver < NVER; ++ver) {
                        const int x = EL == 8 ? 2 * ver : ver;
                        float4* dst = reinterpret_cast<float4*>((isc ? sm.c[w][ver] : sm.b[w][ver]) + tok * NP + k8);
                        dst[0] = make_float4(v[x], v[1 ^ x], v[2 ^ x], v[3 ^ x]);
                        dst[1] = make_float4(v[4 + x], v[4 + (1 ^ x)], v[4 + (2 ^ x)], v[4 + (3 ^ x)]);
                    }
                }
            }
            fetch(k + STAGES - 1);   // into the stage of tile k - 1, which was read last
            if (k < ntiles) __syncthreads();
        }
        // this piece's sums for d_skip and dt_bias
        float* red = &sm.red[0][0][0][0];   // [16 tokens][CH]
        for (int which = 0; which < 2; ++which) {
            named_barrier(1, HT);
#pragma unroll
            for (int i = 0; i < CP; ++i) red[ptok * CH + pc + i] = which ? dbias[i] : dskip[i];
            named_barrier(1, HT);
            if (tid < pl.nch) {
                float v = 0.f;
#pragma unroll
                for (int i = 0; i < TB; ++i) v += red[i * CH + tid];
                a.pv[((size_t)pl.unit * 2 + which) * a.D + pl.c0 + tid] = v;
            }
        }
        return;
    }

    // -------------------------------------------------------------------- the recurrences
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = tid & 3, ch = tid >> 2, n0 = l * EL;
    const int d = pl.c0 + ch;
    const bool on = ch < pl.nch;
    float A2[EL], r[EL], dA[EL], total[EL];
    load_states<EL>(a.A_log + (size_t)d * a.S, n0, a.S, on, A2);
#pragma unroll
    for (int e = 0; e < EL; ++e) {
        A2[e] = on && n0 + e < a.S ? -expf(A2[e]) * LOG2E : 0.f;
        r[e] = dA[e] = total[e] = 0.f;
    }
    // The sums over a warp's channels halve a lane's values at each exchange. So that nothing has to be chosen between,
    // a lane's states are held in the order n0 + (e ^ order), where lanes that exchange differ in the part of `order`
    // they exchange by: each sends the upper half of its registers and adds what arrives to its lower half.
    constexpr int O1 = EL / 2, O2 = EL >= 4 ? EL / 4 : 0;
    const int order = (lane & 8 ? O1 : 0) | (lane & 16 ? O2 : 0);
    const int my_ver = EL == 8 ? (order & 3) >> 1 : order & 3, my_n0 = n0 + (order & ~3);
    auto reorder = [&](float(&v)[EL]) {   // to that order or back
#pragma unroll
        for (int e = 0; e < EL; ++e)
            if (!(e & O1)) {
                const float x = v[e], y = v[e ^ O1];
                v[e] = lane & 8 ? y : x;
                v[e ^ O1] = lane & 8 ? x : y;
            }
#pragma unroll
        for (int e = 0; e < EL; ++e)
            if (O2 && !(e & O2)) {
                const float x = v[e], y = v[e ^ O2];
                v[e] = lane & 16 ? y : x;
                v[e ^ O2] = lane & 16 ? x : y;
            }
    };
    auto lds_row = [&](const float* row, float(&v)[EL]) {
        if (EL == 2) {
            const float2 q = *reinterpret_cast<const float2*>(row + n0);
            v[0] = q.x;
            v[EL > 1 ? 1 : 0] = q.y;
        } else {
#pragma unroll
            for (int e = 0; e + 3 < EL; e += 4) {
                const float4 q = *reinterpret_cast<const float4*>(row + (EL > 4 ? n0 + (e ^ (order & ~3)) : my_n0));
                v[e] = q.x; v[e + 1] = q.y; v[e + 2] = q.z; v[e + 3] = q.w;
            }
        }
    };
    auto state_of = [&](const float* base, int n, float(&v)[EL]) {
        if (base) {
            load_states<EL>(base + n * DS + (size_t)d * a.S, n0, a.S, on, v);
            reorder(v);
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) v[e] = 0.f;
        }
    };
    auto put_states = [&](float* base, int n, const float(&v)[EL]) {
        float x[EL];
#pragma unroll
        for (int e = 0; e < EL; ++e) x[e] = v[e];
        reorder(x);
        store_states<EL>(base + n * DS + (size_t)d * a.S, n0, a.S, on, x);
    };
    if (a.dh0 && (a.ax.cu || a.ax.len == 0)) {   // sequences without tokens: their adjoint passes through
        for (int n = pl.unit; n < a.ax.N; n += pl.units) {
            if (a.ax.cu && axis_cu(a.ax, n + 1) > axis_cu(a.ax, n)) continue;
            float v[EL];
            state_of(a.dht, n, v);
            put_states(a.dh0, n, v);
        }
    }
    Seq s{0, 0, 0};
    if (ntiles > 0) {
        s = seq_at(a.ax, pl.row, pl.hi - 1);
        if (s.end > pl.hi) {
            // the adjoint entering this piece from the later pieces of its sequence, joined in order
            const int q = min((s.end - 1) / a.unit_len, a.units_row - 1);
            join_pieces<EL>(a, a.rloc, pl.row, q, pl.u, -1, d, n0, on, A2, r);
        }
    }
    reorder(A2);
    reorder(r);
    const size_t slot0 = (size_t)pl.row * ((a.ax.len + TB - 1) / TB);
    float hnext[EL];   // the next tile's checkpoint, on its way
    if (ntiles > 0) load_states<EL>(a.ckpt + (slot0 + tile_begin(0) / TB) * DS + (size_t)d * a.S, n0, a.S, on, hnext);
    const int my_in = in_at(ch);
    // the first of the values a lane holds after the sums over channels: dB of a state, or its dC in lanes with bit 2
    const int my_red = (lane & 4 ? NP : 0) + n0 + order;
    __syncthreads();   // the first tile's inputs
    for (int k = 0; k < ntiles; ++k) {
        const int tb = tile_begin(k), te = min(tb + TB, pl.hi), nt = te - tb, w = k & 1;
        float hstart[EL];
#pragma unroll
        for (int e = 0; e < EL; ++e) hstart[e] = hnext[e];
        reorder(hstart);
        if (k + 1 < ntiles) load_states<EL>(a.ckpt + (slot0 + tile_begin(k + 1) / TB) * DS + (size_t)d * a.S, n0, a.S, on, hnext);
        // first and last tokens of sequences inside the tile
        uint32_t starts = 0, ends = 0;
        Seq last{0, 0, 0};   // the tile's last sequence; s becomes its first
        for (int p = te - 1;;) {
            if (p < s.first) s = seq_prev(a.ax, pl.row, s);
            if (p == te - 1) last = s;
            if (s.end <= te && s.end > tb) ends |= 1u << (s.end - 1 - tb);
            if (s.first < tb) break;
            starts |= 1u << (s.first - tb);
            if (s.first == tb) break;
            p = s.first - 1;
        }
        // one token of the forward recurrence
        auto step = [&](int i, float(&h)[EL]) {
            const float2 v = *reinterpret_cast<const float2*>(&sm.in[w][i][my_in]);
            float b[EL];
            lds_row(sm.b[w][my_ver] + i * NP, b);
            const float2 dl = make_float2(v.x, v.x), u = make_float2(v.y, v.y);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float2 g = ssm_exponent2(dl, make_float2(A2[2 * e], A2[2 * e + 1]));
                const float2 hn = fma2(make_float2(ex2(g.x), ex2(g.y)), make_float2(h[2 * e], h[2 * e + 1]),
                                       mul2(u, make_float2(b[2 * e], b[2 * e + 1])));
                h[2 * e] = hn.x;
                h[2 * e + 1] = hn.y;
            }
        };
        // one token of the adjoint, from its state h and the one before it
        auto reverse = [&](int it, const float(&h)[EL], const float(&hp)[EL]) {
            const float4 v = sm.in[w][it][my_in];
            float b[EL], c[EL], db[EL], dc[EL];
            lds_row(sm.b[w][my_ver] + it * NP, b);
            lds_row(sm.c[w][my_ver] + it * NP, c);
            const float2 dl = make_float2(v.x, v.x), u = make_float2(v.y, v.y), d0 = make_float2(v.z, v.z);
            float2 p1, p2, py;
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float2 cc = make_float2(c[2 * e], c[2 * e + 1]), hh = make_float2(h[2 * e], h[2 * e + 1]);
                const float2 AA = make_float2(A2[2 * e], A2[2 * e + 1]), bb = make_float2(b[2 * e], b[2 * e + 1]);
                const float2 g = fma2(cc, d0, make_float2(r[2 * e], r[2 * e + 1]));
                const float2 x = ssm_exponent2(dl, AA);
                const float2 dcv = mul2(d0, hh), dbv = mul2(u, g);
                const float2 rn = mul2(make_float2(ex2(x.x), ex2(x.y)), g);
                const float2 wv = mul2(rn, make_float2(hp[2 * e], hp[2 * e + 1]));
                py = e == 0 ? mul2(hh, cc) : fma2(hh, cc, py);
                p1 = e == 0 ? mul2(g, bb) : fma2(g, bb, p1);
                p2 = e == 0 ? mul2(wv, AA) : fma2(wv, AA, p2);
                const float2 da = fma2(wv, dl, make_float2(dA[2 * e], dA[2 * e + 1]));
                dA[2 * e] = da.x;
                dA[2 * e + 1] = da.y;
                r[2 * e] = rn.x;
                r[2 * e + 1] = rn.y;
                db[2 * e] = dbv.x;
                db[2 * e + 1] = dbv.y;
                dc[2 * e] = dcv.x;
                dc[2 * e + 1] = dcv.y;
            }
            // over the channel's four lanes: lane 0 keeps s1, lane 1 s2, lane 2 sum C h
            float pv[4] = {p1.x + p1.y, p2.x + p2.y, py.x + py.y, 0.f};
            halve<4>(pv, l, 2);
            halve<2>(pv, l, 1);
            reinterpret_cast<float*>(&sm.out[w][it][my_in])[l] = pv[0];
            // over the warp's 8 channels: lane bits 3 and 4 by the states' order, bit 2 with dB against dC
#pragma unroll
            for (int e = 0; e < O1; ++e) {
                db[e] += __shfl_xor_sync(SSM_FULL, db[e + O1], 8);
                dc[e] += __shfl_xor_sync(SSM_FULL, dc[e + O1], 8);
            }
#pragma unroll
            for (int e = 0; e < O2; ++e) {
                db[e] += __shfl_xor_sync(SSM_FULL, db[e + O2], 16);
                dc[e] += __shfl_xor_sync(SSM_FULL, dc[e + O2], 16);
            }
#pragma unroll
            for (int f = 0; f < KEEP; ++f) {
                float v = (lane & 4 ? dc[f] : db[f]) + __shfl_xor_sync(SSM_FULL, lane & 4 ? db[f] : dc[f], 4);
                if (!O2) v += __shfl_xor_sync(SSM_FULL, v, 16);
                sm.red[w][warp][it][my_red + f] = v;
            }
        };
        auto leave = [&](int n) {   // at the first token of sequence n its state's adjoint goes out
            if (a.dh0) put_states(a.dh0, n, r);
#pragma unroll
            for (int e = 0; e < EL; ++e) r[e] = 0.f;
        };
        if (nt == TB && !(starts & ~1u) && !(ends & ~(1u << (TB - 1)))) {
            // a whole tile of one sequence
            if (ends) state_of(a.dht, last.n, r);
            if (NSUB > 1) {
                // states at the sub-blocks' starts
                float h[EL];
#pragma unroll
                for (int e = 0; e < EL; ++e) h[e] = hstart[e];
#pragma unroll 1
                for (int sb = 1; sb < NSUB; ++sb) {
#pragma unroll
                    for (int i = 0; i < L; ++i) step((sb - 1) * L + i, h);
#pragma unroll
                    for (int e = 0; e < EL; ++e) sm.sub[NSUB > 1 ? sb - 1 : 0][e][tid] = h[e];
                }
            }
#pragma unroll 1
            for (int sb = NSUB - 1; sb >= 0; --sb) {
                float hs[L][EL], h[EL], hk[EL];
#pragma unroll
                for (int e = 0; e < EL; ++e) {
                    hk[e] = NSUB == 1 || sb == 0 ? hstart[e] : sm.sub[NSUB > 1 && sb > 0 ? sb - 1 : 0][e][tid];
                    h[e] = hk[e];
                }
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    step(sb * L + i, h);
#pragma unroll
                    for (int e = 0; e < EL; ++e) hs[i][e] = h[e];
                }
#pragma unroll
                for (int i = L - 1; i >= 0; --i) reverse(sb * L + i, hs[i], i > 0 ? hs[i > 0 ? i - 1 : 0] : hk);
            }
            if (starts) leave(s.n);
        } else {
            // sequences begin or end inside, or tokens are missing: the state before each token in the thread's own memory
            // (such tiles are rare, and unrolled this would not fit the instruction cache beside the other path)
            float before[TB][EL], h[EL];
            Seq q = s;
#pragma unroll
            for (int e = 0; e < EL; ++e) h[e] = hstart[e];
#pragma unroll 1
            for (int it = 0; it < nt; ++it) {
                if (it > 0 && (starts >> it & 1)) {
                    q = seq_next(a.ax, pl.row, q);
                    state_of(a.h0, q.n, h);
                }
#pragma unroll
                for (int e = 0; e < EL; ++e) before[it][e] = h[e];
                step(it, h);
            }
#pragma unroll 1
            for (int it = nt - 1; it >= 0; --it) {
                if (ends >> it & 1) state_of(a.dht, last.n, r);
                float hp[EL];
#pragma unroll
                for (int e = 0; e < EL; ++e) h[e] = hp[e] = before[it][e];
                step(it, h);
                reverse(it, h, hp);
                if (starts >> it & 1) {
                    leave(last.n);
                    if (it > 0) last = seq_prev(a.ax, pl.row, last);
                }
            }
        }
        // by tiles: one token after another each of thousands of addends would be rounded at the whole sum's size (dA_log of
        // rows of 2048 tokens 9.9e-7 from 64 bits, 5.9e-7 so, for 2 us of 428)
#pragma unroll
        for (int e = 0; e < EL; ++e) {
            total[e] += dA[e];
            dA[e] = 0.f;
        }
        __syncthreads();
    }
    put_states(a.pA, pl.unit, total);
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
    float bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = a.dt_bias && i < pvalid ? a.dt_bias[pl.c0 + pc + i] : 0.f;
    constexpr int NC = NP / 8, NPT = (TB * NC + SSM_T - 1) / SSM_T;
    float dt[4], z[4], dy[4], cv[NPT][8];
    auto fetch = [&](int tb) {   // a tile's rows, as far as they are there
        const int te = min(tb + TB, hi), t = tb + ptok;
        const int n = t < te && tb >= pl.lo ? pvalid : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) dt[i] = z[i] = dy[i] = 0.f;
        if (n > 0) {
            load_row<4>(dp + (size_t)t * a.lddt, dt, n, false);
            load_row<4>(yp + (size_t)t * a.D, dy, n, false);
            if (zp) load_row<4>(zp + (size_t)t * a.ldz, z, n, false);
        }
#pragma unroll
        for (int j = 0; j < NPT; ++j) {
            const int i = tid + j * SSM_T, tok = i / NC, k = (i - tok * NC) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) cv[j][e] = 0.f;
            if (i < TB * NC && tb + tok < te && tb >= pl.lo)
                load_row<8>(cp + (size_t)(tb + tok) * a.ldc + k, cv[j], a.S - k, a.S - k >= 8 && !(a.how >> SSM_C & 3));
        }
    };
    const int top = (hi - 1) / TB * TB;
    fetch(top);
    for (int tb = top; tb >= pl.lo; tb -= TB) {
        const int te = min(tb + TB, hi);
        const bool in = tb + ptok < te;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = dt[i] + bias[i];
            const float dl = !in || i >= pvalid ? 0.f : a.softplus ? ssm_softplus(v) : v;
            s_in[ptok][pc + i] = make_float2(dl, zp ? dy[i] * z[i] * sigmoid_fast(z[i]) : dy[i]);
        }
#pragma unroll
        for (int j = 0; j < NPT; ++j) {
            const int i = tid + j * SSM_T, tok = i / NC, k = (i - tok * NC) * 8;
            if (i >= TB * NC) break;
            reinterpret_cast<float4*>(&s_c[tok][k])[0] = make_float4(cv[j][0], cv[j][1], cv[j][2], cv[j][3]);
            reinterpret_cast<float4*>(&s_c[tok][k])[1] = make_float4(cv[j][4], cv[j][5], cv[j][6], cv[j][7]);
        }
        __syncthreads();
        fetch(tb - TB);
        auto token = [&](int i) {
            const float2 v = s_in[i][ch];
            float c[EL];
            lds_states<EL>(&s_c[i][n0], c);
#pragma unroll
            for (int e = 0; e < EL; ++e) r[e] = ssm_decay(v.x, A2[e]) * fmaf(c[e], v.y, r[e]);
            sd += v.x;
        };
        if (te - tb == TB) {
#pragma unroll 8
            for (int i = TB - 1; i >= 0; --i) token(i);
        } else {
#pragma unroll 1
            for (int i = te - tb - 1; i >= 0; --i) token(i);
        }
        __syncthreads();
    }
    store_states<EL>(a.rloc + pl.unit * DS + (size_t)d * a.S, n0, a.S, on, r);
    if (on && l == 0) a.sdt[(size_t)pl.unit * a.D + d] = sd;
}

__host__ __device__ constexpr int bwd_channels(int S) { return S <= 16 ? 64 : 32; }   // channels per CTA

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
        const int CH = bwd_channels(a.S), tpg = (a.D / a.G + CH - 1) / CH;
        float v = 0.f;
#pragma unroll 8
        for (int k = 0; k < tpg; ++k) v += a.pbc[(((size_t)(g * tpg + k) * tokens + tok) * 2 + which) * a.S + n];
        st(static_cast<TI*>(which ? a.dc : a.db) + tok * GS + gs, v);
        return;
    }
    const size_t i = (size_t)(blockIdx.x - nbc) * blockDim.x + threadIdx.x;
    const size_t DS = (size_t)a.D * a.S;
    const int units = a.ax.rows * a.units_row;
    if (i < DS) {
        float v = 0.f;
#pragma unroll 8
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
cudaError_t run_bwd(const SsmArgs& a, cudaStream_t st) {
    using Sh = BwdShape<TI, EL>;
    const unsigned grid = (unsigned)(a.ax.rows * a.units_row) * ((a.D / a.G + Sh::CH - 1) / Sh::CH) * a.G;
    static SmemLimit limit;
    const cudaError_t e = limit.set(reinterpret_cast<const void*>(k_ssm_bwd<TI, EL>), (int)sizeof(typename Sh::Smem));
    if (e != cudaSuccess) return e;
    k_ssm_bwd<TI, EL><<<grid, Sh::RT + HT, sizeof(typename Sh::Smem), st>>>(a);
    return cudaSuccess;
}
template <typename TI, int EL>
cudaError_t run_pieces(const SsmArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)(a.ax.rows * a.units_row) * ((a.D / a.G + SSM_CH - 1) / SSM_CH) * a.G;
    k_ssm_bwd_pieces<TI, EL><<<grid, SSM_T, 0, st>>>(a);
    return cudaSuccess;
}
template <bool PIECES, typename TI>
cudaError_t run_states(const SsmArgs& a, cudaStream_t st) {
    if (a.S <= 8) return PIECES ? run_pieces<TI, 2>(a, st) : run_bwd<TI, 2>(a, st);
    if (a.S <= 16) return PIECES ? run_pieces<TI, 4>(a, st) : run_bwd<TI, 4>(a, st);
    if (a.S <= 32) return PIECES ? run_pieces<TI, 8>(a, st) : run_bwd<TI, 8>(a, st);
    return PIECES ? run_pieces<TI, 16>(a, st) : run_bwd<TI, 16>(a, st);
}
template <bool PIECES>
cudaError_t launch(const char* name, const SsmArgs& a, int bf16, cudaStream_t st) {
    cudaError_t r = cudaSuccess;
    const cudaError_t e = traced_launch(name, st, [&] {
        r = bf16 ? run_states<PIECES, __nv_bfloat16>(a, st) : run_states<PIECES, float>(a, st);
    });
    return r != cudaSuccess ? r : e;
}

}  // namespace

int ssm_bwd_tiles(int D, int G, int S) { return (D / G + bwd_channels(S) - 1) / bwd_channels(S) * G; }

cudaError_t launch_ssm_bwd_pieces(const SsmArgs& a, int bf16, cudaStream_t st) {
    return launch<true>("k_ssm_bwd_pieces", a, bf16, st);
}

cudaError_t launch_ssm_bwd(const SsmArgs& a, int bf16, cudaStream_t st) { return launch<false>("k_ssm_bwd", a, bf16, st); }

cudaError_t launch_ssm_bwd_sums(const SsmArgs& a, int bf16, cudaStream_t st) {
    const size_t bc = (size_t)a.ax.rows * a.ax.len * 2 * a.G * a.S, params = (size_t)a.D * (a.S + 2);
    const unsigned nbc = (unsigned)((bc + 255) / 256), np = (unsigned)((params + 255) / 256);
    return traced_launch("k_ssm_sums", st, [&] {
        if (bf16) k_ssm_sums<__nv_bfloat16><<<nbc + np, 256, 0, st>>>(a, nbc);
        else k_ssm_sums<float><<<nbc + np, 256, 0, st>>>(a, nbc);
    });
}

}  // namespace kda
