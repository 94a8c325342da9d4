// Linear attention with a decay for each head on the tensor cores: bf16, K <= 128, in chunks of C = 128 tokens.
// With a the head's decay, S the state entering a chunk of n tokens and the call's s and w (kda_lin.cuh), forwards
//     P_ij = s w a^(i-j) (q_i k_j) for j <= i,   o_i = s a^(i+1) q_i S + sum_j P_ij v_j
//     S <- a^n S + K^T V',   V'_j = w a^(n-1-j) v_j
// and backwards in time (rows are tokens in memory order, the last one comes first)
//     P_ij = s w a^(j-i) (q_i k_j) for j >= i,   o_i = s a^(n-1-i) q_i S + sum_j P_ij v_j,   V'_j = w a^(j+1) v_j.
// A CTA walks a head's 64 value columns through a time window; the serial chain from chunk to chunk is one multiply-add
// per state element in registers, everything else runs ahead of it. Roles: one warp loads (TMA, two chunks deep), one
// issues the four products Q K^T, Q S, K^T V' and P V, four turn scores into P (TMEM to TMEM) and then write the outputs,
// eight keep the state and four form V'.
// Roundings: V' is three bf16 parts, 24 bits, so that the fp32 state is a sum of exact products (each chunk's is summed
// by the tensor core from zero and added once), or two, 2^-16, in calls that return no state; P and the copy of S that the
// queries meet are bf16; the output is rounded once.
// Powers of a: |i - j| = (i - block end) + (block end - j) for columns left of the row's block of 32, so that a score
// costs two products and no exponential; on the diagonal block a row's 32 powers stay in registers.
// Measured (bf16, K = V = 128): 2 x 8192 tokens of 32 heads 141 us, 3.8 TB/s of 537 MB (57% of the copy rate); 4 x 4096 tokens
// of 16 heads 76 us and their backward, three such calls in one launch, 222. What bounds it: a chunk takes some 4000
// cycles of its CTA, where HBM would take 2300 and the tensor cores are busy in 37%; the hand-overs Q K^T, P, P V one behind
// the other, and the roles' instructions, which run once a chunk and have to be fetched anew each time (V' unrolled by
// four 159 us, by two 141.5, not at all 139.5; two parts of V' in place of three 141.3). Kept out after measuring (the 2 x
// 8192 tokens above, against 140 to 141 us in the same call): outputs by the state's warps 160, the same with P V behind the
// next Q K^T 161; P in units of 16 columns, 152 against 150; K^T V' before Q S in quarters of V', 5700 cycles a chunk.
// The state lies over eight warps rather than four for the same reason (32768 tokens of 4 heads of 64 in time windows: 83
// us against 115).
// Rows of the tiles behind a sequence's end belong to its neighbour: K, V and V' are zeroed there, so that whatever they
// hold adds nothing; P is chosen, not multiplied, where masked.
#include "kda_lin.cuh"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int C = 128, VB = 64;                 // tokens of a chunk, value columns of a CTA
constexpr int NTHR = 18 * 32, LOADER = 16, ISSUER = 17;   // warps of the last two roles
constexpr int SV = 32;                          // columns of the state that a thread keeps
constexpr int ATOM = C * 128;                   // bytes of 128 rows of 64 bf16
constexpr int OFF_K = 2 * ATOM, OFF_V = 4 * ATOM, STAGE = 5 * ATOM;
constexpr int OFF_VP = 2 * STAGE, OFF_S = OFF_VP + 3 * ATOM, OFF_END = OFF_S + ATOM;
constexpr int T_SC = 0, T_P = 128, T_O1 = 192, T_O2 = 256, T_KV = 320;   // TMEM columns

struct Shared {
    float pw[C + 1];            // a^m
    float2 one, whole;          // a and a^C in two parts
    alignas(16) float col[32];  // a block's column's power: to the block's end forwards, from its start backwards
    uint64_t full[2], k_free[2], v_free[2], o_ready[2], sc_full, sc_free, p_full, pv_done, v_full, kv_done, s_full, o_free, drain;
    uint32_t tmem;
    int dead;
};
constexpr int SMEM = OFF_END + (int)sizeof(Shared) + 1024;
static_assert(SMEM <= 232448, "shared memory above the per-block limit");

struct LinTc {
    CUtensorMap map[4], out[3];
    LinArgs a;
    int mq[3], mk[3], mv[3];    // each call's maps
};

__device__ __forceinline__ bool wait(Shared& sm, uint64_t* bar, uint32_t parity) { return tc::warp_wait(bar, parity, &sm.dead); }

// The chunks of a window, the same for every role.
struct Chunks {
    const LinArgs& a;
    int row, t, t1, back;
    Seq s;
    __device__ Chunks(const LinArgs& a_, int row_, int t0, int t1_, int back_, bool local) : a(a_), row(row_), t(t0), t1(t1_), back(back_) {
        if (t >= t1) return;
        if (local) {   // only the sequence that goes on behind the window
            s = lin_seq(a.ax, row, t1 - 1, back);
            t = s.end <= t1 ? t1 : max(t0, s.first);
        } else {
            s = lin_seq(a.ax, row, t, back);
        }
    }
    __device__ __forceinline__ bool more() const { return t < t1; }
    __device__ __forceinline__ int n() const { return min(C, min(s.end, t1) - t); }
    // the packed token of the tile's first row
    __device__ __forceinline__ int64_t token(int n) const { return (int64_t)row * a.ax.len + (back ? a.ax.len - t - n : t); }
    __device__ __forceinline__ void next(int n) {
        t += n;
        if (t < t1 && t == s.end) s = lin_seq(a.ax, row, t, back);
    }
};

// Row j of V' from row j of V: e v in NP parts of 8 bits, the leading ones of what is left cut off, the last one rounded
// (the third is the rest). A row behind the chunk's n tokens becomes zeros in V, V' and the keys' KA tiles.
template <int NP>
__device__ __forceinline__ void spread(unsigned char* v, unsigned char* vp, unsigned char* k, int KA, int j, int n, float e) {
    v += j * 128;
    vp += j * 128;
    if (j < n) {
#pragma unroll 1
        for (int ch = 0; ch < 8; ++ch) {
            const uint32_t o = (ch ^ (j & 7)) << 4;
            const uint4 x4 = *reinterpret_cast<const uint4*>(v + o);
            const uint32_t in[4] = {x4.x, x4.y, x4.z, x4.w};
            uint32_t out[NP][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 x = mul2(make_float2(e, e), make_float2(__uint_as_float(in[i] << 16), __uint_as_float(in[i] & 0xffff0000u)));
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const uint32_t lo = __float_as_uint(x.x), hi = __float_as_uint(x.y);
                    out[p][i] = p == NP - 1 ? tc::pack_bf16(x.x, x.y) : __byte_perm(lo, hi, 0x7632);
                    x = add2(x, make_float2(-__uint_as_float(lo & 0xffff0000u), -__uint_as_float(hi & 0xffff0000u)));
                }
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) *reinterpret_cast<uint4*>(vp + p * ATOM + o) = make_uint4(out[p][0], out[p][1], out[p][2], out[p][3]);
        }
    } else {
        const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (int ch = 0; ch < 8; ++ch) {
            *reinterpret_cast<uint4*>(v + 16 * ch) = z;
#pragma unroll
            for (int p = 0; p < NP; ++p) *reinterpret_cast<uint4*>(vp + p * ATOM + 16 * ch) = z;
            for (int p = 0; p < KA; ++p) *reinterpret_cast<uint4*>(k + p * ATOM + j * 128 + 16 * ch) = z;
        }
    }
}
// This thread's SV columns of the state behind a chunk: an S + the chunk's sums, NP parts of them in TMEM.
template <int NP>
__device__ __forceinline__ void advance(float (&S)[SV], uint32_t sums, float2 an) {
#pragma unroll
    for (int v = 0; v < SV; v += 8) {
        float x[NP][8];
#pragma unroll
        for (int i = 0; i < NP; ++i) tc::tmem_ld8(sums + VB * i + v, x[i]);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float2 y = make_float2(x[1][i], x[1][i + 1]);
            if (NP == 3) y = add2(y, make_float2(x[NP - 1][i], x[NP - 1][i + 1]));
            y = add2(make_float2(x[0][i], x[0][i + 1]), y);
            const float2 z = make_float2(S[v + i], S[v + i + 1]);
            y = fma2(z, make_float2(an.x, an.x), fma2(z, make_float2(an.y, an.y), y));
            S[v + i] = y.x;
            S[v + i + 1] = y.y;
        }
    }
}
// Stores the first `cols` (a multiple of 8, or none) of them.
__device__ __forceinline__ void store_columns(float* p, const float (&S)[SV], int cols) {
    const bool vec = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
#pragma unroll
    for (int v = 0; v < SV; v += 4) {
        if (v >= cols) break;
        if (vec) {
            *reinterpret_cast<float4*>(p + v) = make_float4(S[v], S[v + 1], S[v + 2], S[v + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[v + i] = S[v + i];
        }
    }
}
// NP: parts of V'.
template <int NP>
__global__ void __launch_bounds__(NTHR, 1) k_lin_tc(const __grid_constant__ LinTc g) {
    extern __shared__ unsigned char raw[];
    const uint32_t base = (tc::smem_u32(raw) + 1023u) & ~1023u;
    unsigned char* mem = raw + (base - tc::smem_u32(raw));
    Shared& sm = *reinterpret_cast<Shared*>(mem + OFF_END);
    const LinArgs& a = g.a;
    const LinCall& c = a.c[blockIdx.y];
    const int blocks = (c.V + VB - 1) / VB;
    int at = blockIdx.x;
    const int v0 = at % blocks * VB;
    at /= blocks;
    const int h = at % a.HV, unit = at / a.HV;
    if (unit >= a.ax.rows * a.units_row) return;
    const int row = unit / a.units_row, u = unit - row * a.units_row;
    const int t0 = u * a.unit_len, t1 = min(a.ax.len, t0 + a.unit_len);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, role = warp < 4 ? 0 : warp < 12 ? 1 : warp < 16 ? 2 : 3, q32 = (warp & 3) * 32;
    const int KA = c.K > 64 ? 2 : 1;
    const float decay = a.decay ? a.decay[h] : 0.f;

    const bool back = c.back != 0;

    // The loader's copies of one chunk (lane 0); they arrive together. The first two chunks' start here.
    const CUtensorMap *mq = &g.map[g.mq[blockIdx.y]], *mk = &g.map[g.mk[blockIdx.y]], *mv = &g.map[g.mv[blockIdx.y]];
    const int hq = h / c.gq, hk = h / c.gk, hv = h / c.gv;
    const auto load_q = [&](int st, int z) {
        for (int p = 0; p < KA; ++p) tc::tma_load3(base + st * STAGE + p * ATOM, mq, 64 * p, hq, z, &sm.full[st]);
    };
    const auto load_k = [&](int st, int z) {
        tc::mbar_arrive_expect_tx(&sm.full[st], (2 * KA + 1) * ATOM);
        for (int p = 0; p < KA; ++p) tc::tma_load3(base + st * STAGE + OFF_K + p * ATOM, mk, 64 * p, hk, z, &sm.full[st]);
    };
    const auto load_v = [&](int st, int z) { tc::tma_load3(base + st * STAGE + OFF_V, mv, v0, hv, z, &sm.full[st]); };
    if (warp == LOADER) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                tc::mbar_init(&sm.full[i], 1);
                tc::mbar_init(&sm.k_free[i], 1);
                tc::mbar_init(&sm.v_free[i], 1);
                tc::mbar_init(&sm.o_ready[i], 4);
            }
            tc::mbar_init(&sm.sc_full, 1);
            tc::mbar_init(&sm.pv_done, 1);
            tc::mbar_init(&sm.kv_done, 1);
            tc::mbar_init(&sm.drain, 1);
            tc::mbar_init(&sm.sc_free, 4);
            tc::mbar_init(&sm.p_full, 4);
            tc::mbar_init(&sm.v_full, 4);
            tc::mbar_init(&sm.s_full, 8);
            tc::mbar_init(&sm.o_free, 4);
            sm.dead = 0;
            tc::fence_mbar_init();
            Chunks k(a, row, t0, t1, back, false);
            for (int i = 0; i < 2 && k.more(); ++i) {
                const int n = k.n(), z = (int)k.token(n);
                load_k(i, z);
                load_q(i, z);
                load_v(i, z);
                k.next(n);
            }
        }
        __syncwarp();
    }
    if (warp == ISSUER) {
        tc::tmem_alloc(&sm.tmem, 512);
        tc::tmem_relinquish();
    }
    // (64-bit exponentials: by one thread each, beside the set-up. 64 sequences of 128 tokens, 32 heads of 128, forward and backward:
    // 328 and 660 us; 348 and 746 with one in each of the state's warps, behind it.)
    if (threadIdx.x == 13 * 32) sm.whole = lin_power2(decay, C);
    if (threadIdx.x == 14 * 32) sm.one = lin_power2(decay, 1);
    for (int m = threadIdx.x; m <= C; m += NTHR) sm.pw[m] = lin_power(decay, m);
    if (threadIdx.x < 32) sm.col[threadIdx.x] = lin_power(decay, back ? threadIdx.x : 31 - threadIdx.x);
    if (KA == 1)   // the second half of the key rows: nothing, in every chunk
        for (int i = threadIdx.x; i < 2 * ATOM / 16; i += NTHR)
            *reinterpret_cast<uint4*>(mem + (i >= ATOM / 16) * STAGE + OFF_K + ATOM + i % (ATOM / 16) * 16) = make_uint4(0, 0, 0, 0);
    tc::fence_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tb = sm.tmem;

    if (role == 0) {
        // ---------------------------------------------------------------- scores to P; this thread's row i
        const int i = q32 + lane, w = warp;
        const float sw = c.s * c.w;
        const uint32_t tp = tc::taddr(tb, q32, T_P), ts = tc::taddr(tb, q32, T_SC);
        const uint32_t tri = back ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);   // the diagonal block's columns that row i meets
        if (blockIdx.x == 0 && blockIdx.y == 0 && a.err && a.ax.cu) {   // as axis_check, by these warps
            bool bad = false;
            for (int n = i; n < a.ax.N; n += 128) bad |= a.ax.cu[n + 1] < a.ax.cu[n];
            if (i == 0) bad |= a.ax.cu[0] != 0 || a.ax.cu[a.ax.N] != a.ax.len;
            if (bad) atomicOr(a.err, 1);
        }
        const uint32_t t1a = tc::taddr(tb, q32, T_O1), t2a = tc::taddr(tb, q32, T_O2);
        {
            uint32_t z[16];
#pragma unroll
            for (int m = 0; m < 16; ++m) z[m] = 0;
            for (int b = 0; b < 4; ++b) tc::tmem_st16u(tp + 16 * b, z);
            tc::tmem_wait_st();
        }
        uint32_t ph = 0, stage = 0;
        for (Chunks k(a, row, t0, t1, back, false); k.more(); ph ^= 1, stage ^= 1) {
            const int n = k.n();
            if (!wait(sm, &sm.sc_full, ph)) break;
            tc::fence_after_sync();
            // (Loops as short as they get: a warp is alone on its scheduler with this code, and long straight runs of it
            // wait for instructions.)
#pragma unroll 1
            for (int b = back ? w : 0; b <= (back ? 3 : w); ++b) {
                float x[2][16];
                tc::tmem_ld16(ts + 32 * b, x[0]);
                tc::tmem_ld16(ts + 32 * b + 16, x[1]);
                const int left = min(max(n - 32 * b, 0), 32);   // columns of tokens that the chunk has
                uint32_t mask = left == 32 ? 0xffffffffu : (1u << left) - 1u, p[16];
                if (b == w) {
                    mask &= tri;
                    float f[32];
#pragma unroll
                    for (int m = 0; m < 32; ++m) f[m] = sw * sm.pw[abs(lane - m)];
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int m = 0; m < 32; ++m) x[m >> 4][m & 15] = mask >> m & 1 ? x[m >> 4][m & 15] * f[m] : 0.f;
                } else {
                    const float rowf = sw * sm.pw[back ? 32 * b - i : i - 32 * b - 31];
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int m = 0; m < 32; m += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(&sm.col[m]);
                        float* y = &x[m >> 4][m & 15];
                        const float2 r = make_float2(rowf, rowf);
                        const float2 lo = mul2(make_float2(y[0], y[1]), mul2(r, make_float2(f.x, f.y)));
                        const float2 hi = mul2(make_float2(y[2], y[3]), mul2(r, make_float2(f.z, f.w)));
                        y[0] = lo.x;
                        y[1] = lo.y;
                        y[2] = hi.x;
                        y[3] = hi.y;
                    }
                    if (back && left < 32) {
#pragma unroll
                        for (int m = 0; m < 32; ++m) x[m >> 4][m & 15] = mask >> m & 1 ? x[m >> 4][m & 15] : 0.f;
                    }
                }
#pragma unroll
                for (int m = 0; m < 16; ++m) p[m] = tc::pack_bf16(x[m >> 3][2 * m & 15], x[m >> 3][(2 * m & 15) + 1]);
                tc::tmem_st16u(tp + 16 * b, p);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&sm.sc_free);
                tc::mbar_arrive(&sm.p_full);
            }
            // The outputs: a whole chunk's go through the tile of its queries, which every product has read, to one copy by
            // the loader; others row by row, as the rows behind the chunk are another sequence's.
            const bool there = i < n, whole = n == C;
            unsigned char* tile = mem + stage * STAGE + i * 128;
            const float gam = c.s * sm.pw[there ? (back ? n - 1 - i : i + 1) : 0];
            const size_t to = ((size_t)(k.token(n) + (there ? i : 0)) * a.HV + h) * c.V + v0;
            if (!wait(sm, &sm.pv_done, ph)) break;
            tc::fence_after_sync();
#pragma unroll 1
            for (int v = 0; v < VB; v += 16) {
                float x[16], y[16];
                tc::tmem_ld16(t1a + v, x);
                tc::tmem_ld16(t2a + v, y);
                tc::tmem_wait_ld();
                if (v == VB - 16) {
                    tc::fence_before_sync();
                    tc::warp_arrive(&sm.o_free);
                }
#pragma unroll
                for (int m = 0; m < 16; m += 2) {
                    const float2 r = fma2(make_float2(gam, gam), make_float2(x[m], x[m + 1]), make_float2(y[m], y[m + 1]));
                    x[m] = r.x;
                    x[m + 1] = r.y;
                }
                uint32_t bits[8];
#pragma unroll
                for (int m = 0; m < 8; ++m) bits[m] = tc::pack_bf16(x[2 * m], x[2 * m + 1]);
                if (whole && !c.o_f32) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        *reinterpret_cast<uint4*>(tile + (((v / 8 + m) ^ (i & 7)) << 4)) =
                            make_uint4(bits[4 * m], bits[4 * m + 1], bits[4 * m + 2], bits[4 * m + 3]);
                } else if (whole) {
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        *reinterpret_cast<float4*>(tile + v / 32 * ATOM + (((v % 32 / 4 + m) ^ (i & 7)) << 4)) =
                            make_float4(x[4 * m], x[4 * m + 1], x[4 * m + 2], x[4 * m + 3]);
                } else if (c.o_f32) {
                    float* p = static_cast<float*>(c.o) + to + v;
#pragma unroll
                    for (int m = 0; m < 16; m += 4)
                        if (there && v0 + v + m < c.V) *reinterpret_cast<float4*>(p + m) = make_float4(x[m], x[m + 1], x[m + 2], x[m + 3]);
                } else {
                    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(c.o) + to + v;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        if (there && v0 + v + 8 * m < c.V)
                            *reinterpret_cast<uint4*>(p + 8 * m) = make_uint4(bits[4 * m], bits[4 * m + 1], bits[4 * m + 2], bits[4 * m + 3]);
                }
            }
            if (whole) tc::fence_async_smem();
            tc::warp_arrive(&sm.o_ready[stage]);
            k.next(n);
        }
    } else if (role == 1) {
        // ---------------------------------------------------------------- the state; this thread's key row, 32 columns
        const int kk = q32 + lane, s0 = v0 + (warp < 8 ? 0 : SV);
        const size_t KV = (size_t)c.K * c.V, mine = (size_t)kk * c.V + s0;   // a state's elements, and this row's place in it
        const int cols = kk < c.K ? min(SV, c.V - s0) : 0;                   // a multiple of 8, or less than 0
        float S[SV];
        if (u == 0 && c.s1) {   // final states of sequences without tokens
            for (int n = a.ax.cu ? 0 : row; n < (a.ax.cu ? a.ax.N : row + 1); ++n) {
                if (a.ax.cu ? axis_cu(a.ax, n + 1) > axis_cu(a.ax, n) : a.ax.len > 0) continue;
                const size_t to = ((size_t)n * a.HV + h) * KV + mine;
#pragma unroll 1
                for (int v = 0; v < cols; ++v) c.s1[to + v] = c.s0 ? c.s0[to + v] : 0.f;   // (a call with s1 has natural states)
            }
        }
        const float2 one = sm.one, whole = sm.whole;
        uint32_t ph = 0;
        int seq = -1;
        const uint32_t tk = tc::taddr(tb, q32, T_KV + s0 - v0);
        unsigned char* sb = mem + OFF_S + kk * 128;
        for (Chunks k(a, row, t0, t1, back, false); k.more(); ph ^= 1) {
            const int n = k.n();
            if (seq < 0 || k.t == k.s.first) {   // a sequence that came through earlier windows goes on from the state joined there
                const bool joined = seq < 0 && u > 0 && k.s.first < k.t;   // (in the first window none, whatever inconsistent offsets say)
                const size_t rk = c.transposed && !joined ? 1 : c.V, rv = c.transposed && !joined ? c.K : 1;
                const float* p = (joined ? c.local + ((size_t)(unit - 1) * a.HV + h) * KV : c.s0 + ((size_t)k.s.n * a.HV + h) * KV) + kk * rk + s0 * rv;
                const bool has = joined || c.s0;
#pragma unroll
                for (int v = 0; v < SV; ++v) {
                    S[v] = has && v < cols ? *p : 0.f;
                    p += rv;
                }
            }
            seq = k.s.n;
#pragma unroll
            for (int v = 0; v < SV; v += 8) {
                uint4 x;
                x.x = tc::pack_bf16(S[v], S[v + 1]);
                x.y = tc::pack_bf16(S[v + 2], S[v + 3]);
                x.z = tc::pack_bf16(S[v + 4], S[v + 5]);
                x.w = tc::pack_bf16(S[v + 6], S[v + 7]);
                *reinterpret_cast<uint4*>(sb + (((((s0 - v0 + v) >> 3)) ^ (kk & 7)) << 4)) = x;
            }
            tc::fence_async_smem();
            tc::fence_before_sync();
            tc::warp_arrive(&sm.s_full);
            const float2 an = n == C ? whole : lin_raise(one, n);   // a partial chunk meets the state as often as a whole one
            if (!wait(sm, &sm.kv_done, ph)) break;
            tc::fence_after_sync();
            advance<NP>(S, tk, an);
            if (k.t + n == k.s.end && c.s1) store_columns(c.s1 + ((size_t)k.s.n * a.HV + h) * KV + mine, S, cols);
            k.next(n);
        }
    } else if (role == 2) {
        // ------------------------------------------------ V' in its parts; this thread's token row
        const int j = q32 + lane;
        uint32_t ph = 0, stage = 0, fph = 0;
        bool first = true;
        for (Chunks k(a, row, t0, t1, back, false); k.more();) {
            const int n = k.n();
            unsigned char* st = mem + stage * STAGE;
            if (!wait(sm, &sm.full[stage], fph)) break;
            if (!first && !wait(sm, &sm.kv_done, ph ^ 1)) break;
            first = false;
            spread<NP>(st + OFF_V, mem + OFF_VP, st + OFF_K, KA, j, n, c.w * sm.pw[j < n ? (back ? j + 1 : n - 1 - j) : 0]);
            tc::fence_async_smem();
            tc::warp_arrive(&sm.v_full);
            ph ^= 1;
            stage ^= 1;
            fph ^= stage == 0;
            k.next(n);
        }
    } else if (warp == LOADER) {
        // ------------------------------------------------ loads, from the third chunk on, and whole chunks' outputs
        int n1 = 0, n2 = 0, z1 = 0, z2 = 0, issued = 0;   // the last two chunks' tokens and first rows
        const auto give = [&](int i, int n, int z) {      // the outputs of chunk i
            if (!wait(sm, &sm.o_ready[i & 1], (i >> 1) & 1)) return false;
            if (n == C && lane == 0) {
                const uint32_t tile = base + (i & 1) * STAGE;
                const CUtensorMap* mo = &g.out[blockIdx.y];
                tc::tma_store3(mo, v0, h, z, tile);
                if (c.o_f32 && v0 + 32 < c.V) tc::tma_store3(mo, v0 + 32, h, z, tile + ATOM);
                tc::bulk_commit();
                tc::bulk_wait_read();
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        Chunks k(a, row, t0, t1, back, false);
        for (; k.more(); ++issued) {
            const int n = k.n(), z = (int)k.token(n), st = issued & 1;
            if (issued > 1) {
                const uint32_t ph = ((issued >> 1) - 1) & 1;
                if (lane < KA) tc::tma_prefetch3(mq, 64 * lane, hq, z);   // their place is free last
                if (!(ok = wait(sm, &sm.k_free[st], ph))) break;
                if (lane == 0) load_k(st, z);
                ok = wait(sm, &sm.v_free[st], ph);
                if (lane == 0) load_v(st, z);   // (the chunk's bytes are announced: all its copies are made)
                ok = give(issued - 2, n2, z2) && ok;
                if (lane == 0) load_q(st, z);
                __syncwarp();
            }
            n2 = n1;
            z2 = z1;
            n1 = n;
            z1 = z;
            if (!ok) {
                ++issued;
                break;
            }
            k.next(n);
        }
        if (ok && issued > 1) ok = give(issued - 2, n2, z2);
        if (ok && issued > 0) ok = give(issued - 1, n1, z1);
        // no copy is in flight when the CTA ends, after a failure either
        if (lane == 0) tc::bulk_wait_all();
        for (int i = max(0, issued - 2); i < issued; ++i) tc::mbar_wait(&sm.full[i & 1], (i >> 1) & 1);
    } else if (warp == ISSUER) {
        // ---------------------------------------------------------------- products
        constexpr uint32_t I_SC = tc::idesc_bf16(C, C), I_O = tc::idesc_bf16_bmn(C, VB), I_KV = tc::idesc_bf16_abmn(C, NP * VB);
        uint32_t stage = 0, fph = 0, ph = 0;
        bool first = true, ok = true;
        const uint64_t dvp = tc::sdesc_mn(base + OFF_VP, ATOM, 0), dsb = tc::sdesc_mn(base + OFF_S, ATOM, 0);
        for (Chunks k(a, row, t0, t1, back, false); k.more();) {
            const int n = k.n();
            const uint32_t st = base + stage * STAGE;
            const uint64_t dq = tc::sdesc_k(st, C, 0), dk = tc::sdesc_k(st + OFF_K, C, 0);
            ok = wait(sm, &sm.full[stage], fph);
            if (ok && !first) ok = wait(sm, &sm.sc_free, ph ^ 1);
            if (!ok) break;
            tc::fence_after_sync();
            tc::mma4_bf16_w<false, false>(tb + T_SC, dq, dk, I_SC, 0);
            if (KA > 1) tc::mma4_bf16_w<false, false>(tb + T_SC, tc::kstep_k(dq, C, 4), tc::kstep_k(dk, C, 4), I_SC, 1);
            tc::mma_commit_w(&sm.sc_full);
            ok = wait(sm, &sm.s_full, ph);
            if (ok && !first) ok = wait(sm, &sm.o_free, ph ^ 1);
            if (!ok) break;
            tc::fence_after_sync();
            tc::mma4_bf16_w<false, true>(tb + T_O1, dq, dsb, I_O, 0);
            if (KA > 1) tc::mma4_bf16_w<false, true>(tb + T_O1, tc::kstep_k(dq, C, 4), tc::kstep_mn(dsb, 4), I_O, 1);
            ok = wait(sm, &sm.v_full, ph);
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t dkt = tc::sdesc_mn(st + OFF_K, ATOM, 0), dv = tc::sdesc_mn(st + OFF_V, ATOM, 0);
            tc::mma4_bf16_w<true, true>(tb + T_KV, dkt, dvp, I_KV, 0);
            tc::mma4_bf16_w<true, true>(tb + T_KV, tc::kstep_mn(dkt, 4), tc::kstep_mn(dvp, 4), I_KV, 1);
            tc::mma_commit_w(&sm.kv_done);
            tc::mma_commit_w(&sm.k_free[stage]);
            ok = wait(sm, &sm.p_full, ph);
            if (!ok) break;
            tc::fence_after_sync();
            tc::mma4_bf16_ts_w(tb + T_O2, tb + T_P, dv, I_O, 0);
            tc::mma4_bf16_ts_w(tb + T_O2, tb + T_P + 32, tc::kstep_mn(dv, 4), I_O, 1);
            tc::mma_commit_w(&sm.pv_done);
            tc::mma_commit_w(&sm.v_free[stage]);
            first = false;
            ph ^= 1;
            stage ^= 1;
            fph ^= stage == 0;
            k.next(n);
        }
        // every product is done before the tensor memory goes back (after a failure, too)
        tc::mma_commit_w(&sm.drain);
        if (!tc::mbar_wait(&sm.drain, 0)) sm.dead = 1;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (threadIdx.x == 0 && sm.dead && a.err) atomicOr(a.err, 2);
    if (warp == ISSUER) tc::tmem_dealloc(tb, 512);
}

// ------------------------------------------------------------------ the windows' own states
// End states of the windows' own tokens, from zero: only the state's half of a chunk's work, two chunks at once (the
// scores' warps form every other V', which has two places, as the sums have). Bound by V' and the products behind it
// (32768 tokens of 16 heads of 128 in four windows: 223 us in all; 243 with K and V loaded together, 247 with the main
// kernel's loop).
constexpr int W_V = 2 * ATOM, W_STAGE = 3 * ATOM, W_VP = 2 * W_STAGE, W_END = W_VP + 6 * ATOM;
struct WindowShared {
    float pw[C + 1];
    float2 one, whole;
    uint64_t k_in[2], v_in[2], v_full[2], kv_done[2], kv_free[2], drain;
    uint32_t tmem;
    int dead;
};
constexpr int W_SMEM = W_END + (int)sizeof(WindowShared) + 1024;
static_assert(W_SMEM <= 232448, "shared memory above the per-block limit");

template <int NP>
__global__ void __launch_bounds__(NTHR, 1) k_lin_tc_windows(const __grid_constant__ LinTc g) {
    extern __shared__ unsigned char raw[];
    const uint32_t base = (tc::smem_u32(raw) + 1023u) & ~1023u;
    unsigned char* mem = raw + (base - tc::smem_u32(raw));
    WindowShared& sm = *reinterpret_cast<WindowShared*>(mem + W_END);
    const LinArgs& a = g.a;
    const LinCall& c = a.c[blockIdx.y];
    const int blocks = (c.V + VB - 1) / VB;
    int at = blockIdx.x;
    const int v0 = at % blocks * VB;
    at /= blocks;
    const int h = at % a.HV, unit = at / a.HV;
    if (unit >= a.ax.rows * a.units_row) return;
    const int row = unit / a.units_row, u = unit - row * a.units_row;
    if (u == a.units_row - 1) return;   // nothing comes behind a row's last window
    const int t0 = u * a.unit_len, t1 = min(a.ax.len, t0 + a.unit_len);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q32 = (warp & 3) * 32, KA = c.K > 64 ? 2 : 1;
    const float decay = a.decay ? a.decay[h] : 0.f;
    const bool back = c.back != 0;
    {
        const Chunks k(a, row, t0, t1, back, true);
        if (!k.more()) return;   // its last sequence ends with it
    }
    const CUtensorMap *mk = &g.map[g.mk[blockIdx.y]], *mv = &g.map[g.mv[blockIdx.y]];
    const int hk = h / c.gk, hv = h / c.gv;
    const auto load_k = [&](int st, int z) {
        tc::mbar_arrive_expect_tx(&sm.k_in[st], KA * ATOM);
        for (int p = 0; p < KA; ++p) tc::tma_load3(base + st * W_STAGE + p * ATOM, mk, 64 * p, hk, z, &sm.k_in[st]);
    };
    const auto load_v = [&](int st, int z) {
        tc::mbar_arrive_expect_tx(&sm.v_in[st], ATOM);
        tc::tma_load3(base + st * W_STAGE + W_V, mv, v0, hv, z, &sm.v_in[st]);
    };
    if (warp == LOADER) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                tc::mbar_init(&sm.k_in[i], 1);
                tc::mbar_init(&sm.v_in[i], 1);
                tc::mbar_init(&sm.v_full[i], 4);
                tc::mbar_init(&sm.kv_done[i], 1);
                tc::mbar_init(&sm.kv_free[i], 8);
            }
            tc::mbar_init(&sm.drain, 1);
            sm.dead = 0;
            tc::fence_mbar_init();
            Chunks k(a, row, t0, t1, back, true);
            for (int i = 0; i < 2 && k.more(); ++i) {
                const int n = k.n();
                load_v(i, (int)k.token(n));
                load_k(i, (int)k.token(n));
                k.next(n);
            }
        }
        __syncwarp();
    }
    if (warp == ISSUER) {
        tc::tmem_alloc(&sm.tmem, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 13 * 32) sm.whole = lin_power2(decay, C);
    if (threadIdx.x == 14 * 32) sm.one = lin_power2(decay, 1);
    for (int m = threadIdx.x; m <= C; m += NTHR) sm.pw[m] = lin_power(decay, m);
    if (KA == 1)   // the second half of the key rows: nothing, in every chunk
        for (int i = threadIdx.x; i < 2 * ATOM / 16; i += NTHR)
            *reinterpret_cast<uint4*>(mem + (i >= ATOM / 16) * W_STAGE + ATOM + i % (ATOM / 16) * 16) = make_uint4(0, 0, 0, 0);
    tc::fence_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tb = sm.tmem;

    if (warp < 4 || (warp >= 12 && warp < 16)) {
        // ------------------------------------------------ V' of every other chunk; this thread's token row
        const int j = q32 + lane, mine = warp < 4 ? 0 : 1;
        int i = 0;
        for (Chunks k(a, row, t0, t1, back, true); k.more(); ++i) {
            const int n = k.n();
            if ((i & 1) == mine) {
                const uint32_t ph = i >> 1 & 1;
                if (!tc::warp_wait(&sm.v_in[mine], ph, &sm.dead)) break;
                if (n < C && !tc::warp_wait(&sm.k_in[mine], ph, &sm.dead)) break;   // its rows behind the chunk are cleared
                if (i > 1 && !tc::warp_wait(&sm.kv_done[mine], ph ^ 1, &sm.dead)) break;
                unsigned char* st = mem + mine * W_STAGE;
                spread<NP>(st + W_V, mem + W_VP + mine * 3 * ATOM, st, KA, j, n, c.w * sm.pw[j < n ? (back ? j + 1 : n - 1 - j) : 0]);
                tc::fence_async_smem();
                tc::warp_arrive(&sm.v_full[mine]);
            }
            k.next(n);
        }
    } else if (warp < 12) {
        // ------------------------------------------------ the state; this thread's key row, 32 columns
        const int kk = q32 + lane, s0 = v0 + (warp < 8 ? 0 : SV), cols = kk < c.K ? min(SV, c.V - s0) : 0;
        float S[SV];
#pragma unroll
        for (int v = 0; v < SV; ++v) S[v] = 0.f;
        const float2 one = sm.one, whole = sm.whole;
        int i = 0;
        for (Chunks k(a, row, t0, t1, back, true); k.more(); ++i) {
            const int n = k.n();
            const float2 an = n == C ? whole : lin_raise(one, n);
            if (!tc::warp_wait(&sm.kv_done[i & 1], i >> 1 & 1, &sm.dead)) break;
            tc::fence_after_sync();
            advance<NP>(S, tc::taddr(tb, q32, (i & 1) * 256 + s0 - v0), an);
            tc::fence_before_sync();
            tc::warp_arrive(&sm.kv_free[i & 1]);
            k.next(n);
        }
        store_columns(c.local + (((size_t)unit * a.HV + h) * c.K + kk) * c.V + s0, S, cols);
    } else if (warp == LOADER) {
        int issued = 0;
        bool ok = true;
        for (Chunks k(a, row, t0, t1, back, true); k.more(); ++issued) {
            const int n = k.n();
            if (issued > 1) {
                const uint32_t ph = ((issued >> 1) - 1) & 1;
                if (!tc::warp_wait(&sm.v_full[issued & 1], ph, &sm.dead)) break;   // V has been read
                if (lane == 0) load_v(issued & 1, (int)k.token(n));
                ok = tc::warp_wait(&sm.kv_done[issued & 1], ph, &sm.dead);
                if (lane == 0) load_k(issued & 1, (int)k.token(n));
                __syncwarp();
                if (!ok) {
                    ++issued;
                    break;
                }
            }
            k.next(n);
        }
        // no copy is in flight when the CTA ends, after a failure either
        for (int i = max(0, issued - 2); i < issued; ++i) {
            tc::mbar_wait(&sm.v_in[i & 1], (i >> 1) & 1);
            tc::mbar_wait(&sm.k_in[i & 1], (i >> 1) & 1);
        }
    } else {
        constexpr uint32_t I_KV = tc::idesc_bf16_abmn(C, NP * VB);
        int i = 0;
        for (Chunks k(a, row, t0, t1, back, true); k.more(); ++i) {
            const int n = k.n(), b = i & 1;
            const uint32_t ph = i >> 1 & 1;
            if (!tc::warp_wait(&sm.k_in[b], ph, &sm.dead) || !tc::warp_wait(&sm.v_full[b], ph, &sm.dead)) break;
            if (i > 1 && !tc::warp_wait(&sm.kv_free[b], ph ^ 1, &sm.dead)) break;
            tc::fence_after_sync();
            const uint64_t dk = tc::sdesc_mn(base + b * W_STAGE, ATOM, 0), dv = tc::sdesc_mn(base + W_VP + b * 3 * ATOM, ATOM, 0);
            tc::mma4_bf16_w<true, true>(tb + b * 256, dk, dv, I_KV, 0);
            tc::mma4_bf16_w<true, true>(tb + b * 256, tc::kstep_mn(dk, 4), tc::kstep_mn(dv, 4), I_KV, 1);
            tc::mma_commit_w(&sm.kv_done[b]);
            k.next(n);
        }
        // every product is done before the tensor memory goes back (after a failure, too)
        tc::mma_commit_w(&sm.drain);
        if (!tc::mbar_wait(&sm.drain, 0)) sm.dead = 1;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (threadIdx.x == 0 && sm.dead && a.err) atomicOr(a.err, 2);
    if (warp == ISSUER) tc::tmem_dealloc(tb, 512);
}

template <int NP>
cudaError_t run(const LinTc& g, cudaStream_t st) {
    int vmax = 1;
    for (int i = 0; i < g.a.calls; ++i) vmax = g.a.c[i].V > vmax ? g.a.c[i].V : vmax;
    const long long ctas = (long long)g.a.ax.rows * g.a.units_row * g.a.HV * ((vmax + VB - 1) / VB);
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)ctas, g.a.calls);
    if (g.a.units_row > 1) {
        static SmemLimit limit;
        cudaError_t e = limit.set(reinterpret_cast<const void*>(&k_lin_tc_windows<NP>), W_SMEM);
        if (e != cudaSuccess) return e;
        e = traced_launch("k_lin_tc_windows", st, [&] { k_lin_tc_windows<NP><<<grid, NTHR, W_SMEM, st>>>(g); });
        if (e != cudaSuccess || (e = launch_lin_join(g.a, st)) != cudaSuccess) return e;
    }
    static SmemLimit limit;
    const cudaError_t e = limit.set(reinterpret_cast<const void*>(&k_lin_tc<NP>), SMEM);
    if (e != cudaSuccess) return e;
    return traced_launch("k_lin_tc", st, [&] { k_lin_tc<NP><<<grid, NTHR, SMEM, st>>>(g); });
}

}  // namespace

bool lin_tc_call(const LinCall& c) {
    const auto on = [](const void* p, int64_t ld, int w) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && w % 8 == 0; };
    return c.K <= C && on(c.q, c.ldq, c.K) && on(c.k, c.ldk, c.K) && on(c.v, c.ldv, c.V) && (reinterpret_cast<uintptr_t>(c.o) & 15) == 0;
}

// The cheapest number of windows n of a row, in chunks' times (2 us): every round of CTAs over the SMs takes a window's
// chunks, 0.6 of a chunk's time more for each where the windows' own states are formed first, and 3 to start; windows cost
// two launches more, and a little each where they are joined. (Measured, us: 32768 tokens, 16 heads of 128, 32 CTAs a
// window: one 524, two 407, four 223, eight 246; 8192 tokens, 2 x 24 CTAs backwards: one 134, two 144, three 96, four 118;
// 2 x 4096 tokens, 64 CTAs: one 74, two 79.)
int lin_tc_window(int rows, int len, int ctas) {
    const int chunks = (len + C - 1) / C;
    double least = 0;
    int best = chunks > 0 ? chunks : 1;
    for (int n = 1; n <= chunks && n <= LIN_MAX_WINDOWS; ++n) {
        const int each = (chunks + n - 1) / n;
        const long long all = (long long)rows * ctas * n, rounds = (all + sm_count() - 1) / sm_count();
        const double cost = rounds * (each * (n > 1 ? 1.6 : 1.) + 3.) + (n > 1 ? 10. + 0.06 * n : 0.);
        if (n == 1 || cost < least) {
            least = cost;
            best = each;
        }
    }
    return best * C;
}

cudaError_t launch_lin_tc(const LinArgs& a, cudaStream_t st) {
    LinTc g;
    g.a = a;
    const int64_t tokens = (int64_t)a.ax.rows * a.ax.len;
    int maps = 0;
    struct { const void* p; int64_t ld; int group, width; } seen[4];
    const auto map = [&](const void* p, int64_t ld, int group, int width, int& to) {
        for (to = 0; to < maps; ++to)   // the same tensor in another role
            if (seen[to].p == p && seen[to].ld == ld && seen[to].group == group && seen[to].width == width) return true;
        if (maps == 4) return false;
        seen[maps] = {p, ld, group, width};
        return tmap_tokens_bf16(&g.map[maps++], p, tokens, a.HV / group, width, ld, C);
    };
    for (int i = 0; i < a.calls; ++i) {
        const LinCall& c = a.c[i];
        if (!map(c.q, c.ldq, c.gq, c.K, g.mq[i]) || !map(c.k, c.ldk, c.gk, c.K, g.mk[i]) || !map(c.v, c.ldv, c.gv, c.V, g.mv[i]))
            return cudaErrorInvalidValue;
        if (!(c.o_f32 ? tmap_tokens_f32(&g.out[i], c.o, tokens, a.HV, c.V, C) : tmap_tokens_bf16(&g.out[i], c.o, tokens, a.HV, c.V, (int64_t)a.HV * c.V, C)))
            return cudaErrorInvalidValue;
    }
    bool states = false;   // they are fp32 results: all their bits are kept
    for (int i = 0; i < a.calls; ++i) states = states || a.c[i].s1;
    return states ? run<3>(g, st) : run<2>(g, st);
}

}  // namespace kda
