// Selective state space scan (diagonal, input-dependent step), forward:
//     delta = softplus(dt + dt_bias),  a = exp(-delta exp(A_log)),  u = delta x
//     h_t = a h_{t-1} + u B_t,   y_t = (sum_n C_t[n] h_t[n] + d_skip x_t) silu(z_t)
// Four lanes share a channel and hold its states in registers; a CTA walks 64 channels
// through a time piece in tiles of up to 32 tokens. Eight warps run the recurrence; four
// in front of it copy tiles ahead into shared memory (asynchronously, each thread its own
// share) and form a tile's steps once per (token, channel); four behind it sum, gate and
// store the outputs. Two tiles of buffers and an mbarrier per hand-over let the three
// run apart, and each warp of the recurrence on its own (with one barrier for all per
// tile, the latencies of the three added up: 461 against 444 us for two sequences of
// 8192 tokens and 4096 channels).
// Every lane needs its states' values of the rows b_t and c_t, the same for all
// channels. Read from shared memory they bound the kernel: a load fills 128 bytes of
// registers per cycle however few addresses it has, and the two rows are three quarters
// of what the recurrence reads. So the tensor core spreads them: with A[m][k] = 1 where
// k = m mod 4 and B[k][(token, e)] = the row's state 4 k' + e of lane group k, the product
// holds in tensor memory, in each lane's own row, that lane's values of every token of
// the tile, from where a warp reads 32 columns in one instruction. The product is exact:
// a bf16 value has one non-zero term, an fp32 one is split into three bf16 parts that
// add up to its 24 bits.
// Per four states and token the recurrence takes 4 exponentials (16 cycles of a
// scheduler's share at 32 per cycle and SM) and 8 paired multiply-adds (16 cycles).
// Measured, two rows of 8192 tokens, 4096 channels of 16 states, bf16: 406 us, 1.3 TB/s
// of the tensors' bytes (20% of the copy rate). The bound is instruction dispatch: on
// the 128 SMs that two rows of 64 channel tiles fill, a scheduler spends 106 cycles on
// four tokens of a warp's recurrence however many warps it has (a paired multiply-add
// holds it for two), 1700 of the 3100 cycles of a tile of 32 tokens; the steps, the
// gate and the copies are most of the rest. So what helps is fewer instructions: two
// tokens per shared access, rows spaced instead of permuted, copies without checks took
// it from 444 to 408. Two channels per lane (509), 8-token batches of operands (470, with
// registers moved between the warp groups) and exponentials one batch ahead (473) do not.
// A long row is cut into time pieces when its channels alone do not fill the GPU:
// a first pass forms each piece's end state from zero and its sum of delta (the
// piece's decay is exp(A sum delta)); in the second pass each piece joins the
// states of the pieces before it and runs its outputs.
#include "kda_ssm.cuh"
#include "tc.cuh"

namespace kda {
namespace {

enum { OUT = 0, OUT_CKPT = 1, CKPT = 2, PIECE = 3 };

constexpr int RT = 256;         // threads of the recurrence: 64 channels x 4 lanes
constexpr int CH = RT / 4;
constexpr int PT = 128;         // threads in front of it, and as many behind it

template <typename TI, int EL, int MODE>
struct FwdShape {
    static constexpr bool HAS_Y = MODE == OUT || MODE == OUT_CKPT, HAS_CK = MODE == OUT_CKPT || MODE == CKPT;
    static constexpr int THREADS = RT + (HAS_Y ? 2 : 1) * PT;
    static constexpr int NROW = HAS_Y ? 2 : 1;           // rows of a token: b (and c)
    // tokens per tile: at most 256 columns of spread rows, two tiles of them in the SM's 512; fp32 tiles are half as long
    // for their shared memory
    static constexpr int MOST = sizeof(TI) == 2 ? 32 : 16, TT = 128 / EL < MOST ? 128 / EL : MOST;
    static constexpr int COLS = TT * NROW * EL;          // columns of a tile
    static constexpr int ALLOC = 2 * COLS < 32 ? 32 : 2 * COLS;
    static constexpr int IT = 2, CP = TT * CH / PT / IT; // a thread's share around the recurrence: CP channels of two successive tokens
    static constexpr int PIECES = TT * NROW * 4;         // (token, row, lane group) of EL states
    static constexpr int PP = (PIECES + PT - 1) / PT;    // per thread
    static constexpr int STAGES = 4;                     // tiles in copies
    static constexpr int ATOM = 16 * 128;                // 16 k-rows of 64 columns
    static constexpr int OPB = (COLS + 63) / 64 * ATOM;  // bytes of a B operand
    struct Smem {
        unsigned char a[2 * ATOM];                       // 128 rows of ones
        unsigned char b[2][OPB];
        TI front[STAGES][2][IT][PT][CP];                 // x, dt
        TI back[HAS_Y ? STAGES : 1][2][IT][PT][CP];      // x, z
        TI bc[STAGES][PP][PT][EL];
        float4 du[2][TT / 2][CH + CH / 8];               // delta, u of two tokens; see du_at
        float4 y[2][HAS_Y ? TT / 2 : 1][2 * CH + CH / 8]; // two lanes' parts of two tokens; see y_at
        uint64_t full[2], done[2], yfree[2];             // hand-overs of a tile's buffers
        uint32_t tmem;
    };
    static_assert(CP % 2 == 0 && sizeof(Smem) + 1024 <= 227 * 1024, "tile shape");
};

// Places of a channel in the rows of two tokens' steps, and of its lanes 2 half and 2 half + 1 in those of their outputs,
// spaced so that the eight threads of a quarter warp, which hold a few neighbouring channels each, reach distinct banks
// (and so that a thread's places are a constant apart: permuted ones took an instruction each).
__device__ __forceinline__ int du_at(int ch) { return ch + (ch >> 3); }
__device__ __forceinline__ int y_at(int ch, int half) { return 2 * ch + half + (ch >> 3); }

// Byte of column n of k-row k in an operand whose columns are contiguous (128-byte swizzle).
__device__ __forceinline__ int op_at(int k, int n) {
    const int byte = (n & 63) * 2;
    return (n >> 6) * (16 * 128) + k * 128 + ((((byte >> 4) ^ (k & 7)) << 4) | (byte & 15));
}

// N columns of a warp's 32 lanes from tensor memory; the values are there after tmem_wait_ld.
template <int N>
__device__ __forceinline__ void spread_load(uint32_t addr, uint32_t (&r)[N]) {
    static_assert(N == 16 || N == 32, "columns per load");
    if constexpr (N == 32) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16 % N]),
              "=r"(r[17 % N]), "=r"(r[18 % N]), "=r"(r[19 % N]), "=r"(r[20 % N]), "=r"(r[21 % N]), "=r"(r[22 % N]),
              "=r"(r[23 % N]), "=r"(r[24 % N]), "=r"(r[25 % N]), "=r"(r[26 % N]), "=r"(r[27 % N]), "=r"(r[28 % N]),
              "=r"(r[29 % N]), "=r"(r[30 % N]), "=r"(r[31 % N])
            : "r"(addr));
    } else {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(addr));
    }
}
// A piece of EL states into k-rows l (bf16) or l, 4 + l, 8 + l (the three bf16 parts of fp32) from column n.
template <int EL>
__device__ __forceinline__ void put_piece(unsigned char* op, int l, int n, const __nv_bfloat16* v) {
    constexpr int W = EL < 8 ? EL : 8;   // elements of one access
    struct alignas(2 * W) Pack { uint32_t w[W / 2]; };
#pragma unroll
    for (int e = 0; e < EL; e += W) *reinterpret_cast<Pack*>(op + op_at(l, n + e)) = *reinterpret_cast<const Pack*>(v + e);
}
template <int EL>
__device__ __forceinline__ void put_piece(unsigned char* op, int l, int n, const float* v) {
#pragma unroll
    for (int e = 0; e < EL; e += 2) {
        float x0 = v[e], x1 = v[e + 1];
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            // the upper 16 bits, exact, and what is left of the value (an infinity is whole in its first part)
            const uint32_t h0 = __float_as_uint(x0) & 0xffff0000u, h1 = __float_as_uint(x1) & 0xffff0000u;
            *reinterpret_cast<uint32_t*>(op + op_at(4 * j + l, n + e)) = h0 >> 16 | h1;
            x0 = isinf(x0) ? 0.f : x0 - __uint_as_float(h0);
            x1 = isinf(x1) ? 0.f : x1 - __uint_as_float(h1);
        }
    }
}

// Copies of a thread's share of a tile: CP channels of IT tokens of two tensors, in a ring of STAGES tiles.
template <typename TI, typename Sh>
struct Share {
    static constexpr int CP = Sh::CP, IT = Sh::IT, PER = CH / CP;   // threads per token
    const TI* src[2][IT];
    size_t step[2];
    int how[2], tok[IT], pc, valid, left;   // left: tokens from the next tile to fetch on
    bool whole;                             // all CP channels are there, in rows that are aligned
    __device__ __forceinline__ void start(int tid, const SsmPlace& pl, int first, const void* s0, size_t ld0, int how0,
                                          const void* s1, size_t ld1, int how1, size_t row0) {
        pc = (tid % PER) * CP;
        valid = pl.nch - pc;
        left = pl.hi - first;
        how[0] = how0;
        how[1] = how1;
        whole = valid >= CP && how0 == 0 && (how1 == 0 || !s1);
        step[0] = Sh::TT * ld0;
        step[1] = Sh::TT * ld1;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            tok[i] = tid / PER * IT + i;
            src[0][i] = static_cast<const TI*>(s0) + (row0 + first + tok[i]) * ld0 + pl.c0 + pc;
            src[1][i] = s1 ? static_cast<const TI*>(s1) + (row0 + first + tok[i]) * ld1 + pl.c0 + pc : nullptr;
        }
    }
    __device__ __forceinline__ void fetch(TI (*stage)[IT][PT][CP], int tid) {
        if (whole && left >= Sh::TT) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                copy_whole_async<TI, CP>(stage[0][i][tid], src[0][i]);
                src[0][i] += step[0];
                if (src[1][i]) {
                    copy_whole_async<TI, CP>(stage[1][i][tid], src[1][i]);
                    src[1][i] += step[1];
                }
            }
            left -= Sh::TT;
        } else if (left > 0) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int n = tok[i] < left ? valid : 0;
                copy_row_async<TI, CP>(stage[0][i][tid], src[0][i], n, how[0]);
                src[0][i] += step[0];
                if (src[1][i]) {
                    copy_row_async<TI, CP>(stage[1][i][tid], src[1][i], n, how[1]);
                    src[1][i] += step[1];
                }
            }
            left -= Sh::TT;
        }
    }
};

template <typename TI, int EL, int MODE>
__global__ void __launch_bounds__(FwdShape<TI, EL, MODE>::THREADS, 1) k_ssm_fwd(SsmArgs a) {
    using Sh = FwdShape<TI, EL, MODE>;
    constexpr int NROW = Sh::NROW, STAGES = Sh::STAGES, P = EL / 2, TT = Sh::TT, CP = Sh::CP, IT = Sh::IT, COLS = Sh::COLS, PP = Sh::PP;
    constexpr bool HAS_Y = Sh::HAS_Y, HAS_CK = Sh::HAS_CK;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    typename Sh::Smem& sm = *reinterpret_cast<typename Sh::Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    if (blockIdx.x == 0 && MODE != PIECE) axis_check(a.ax, a.err);
    const SsmPlace pl = ssm_place<CH>(a);
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
    // tensor memory, hand-overs, the operands' constant parts
    if (threadIdx.x < 32) {
        tc::tmem_alloc(&sm.tmem, Sh::ALLOC);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            tc::mbar_init(&sm.full[w], PT / 32 + 1);   // the warps' steps and the spread rows
            tc::mbar_init(&sm.done[w], RT / 32);
            tc::mbar_init(&sm.yfree[w], PT / 32);
        }
        tc::fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 16 * 128; i += Sh::THREADS) {
        const int k = i >> 7, m = i & 127;
        *reinterpret_cast<__nv_bfloat16*>(sm.a + op_at(k, m)) = __float2bfloat16_rn(k < 12 && (m & 3) == (k & 3) ? 1.f : 0.f);
    }
    for (int i = threadIdx.x; i < 2 * Sh::OPB / 16; i += Sh::THREADS) reinterpret_cast<uint4*>(&sm.b[0][0])[i] = make_uint4(0, 0, 0, 0);
    tc::fence_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem;
    // A wait that gives up (a lost hand-over) is recorded where the caller gave an error word, and no further one is tried:
    // the results are not valid then.
    bool lost = false;
    auto await = [&](uint64_t* bar, int phase) {
        if (!lost && !tc::mbar_wait(bar, phase & 1)) {
            lost = true;
            if (a.err) atomicOr(a.err, 2);
        }
    };
    auto hand_over = [&](uint64_t* bar) {   // this warp's part
        __syncwarp();
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
    };

    if (threadIdx.x >= RT + PT) {
        // ---------------------------------------------------------------- behind the recurrence
        const int tid = threadIdx.x - RT - PT;
        Share<TI, Sh> sh;
        sh.start(tid, pl, first_tile, a.x, a.ldx, a.how >> SSM_X & 3, a.z, a.ldz, a.how >> SSM_Z & 3, tok0);
        const bool gate = a.z != nullptr, whole = sh.valid >= CP && !(a.how >> SSM_OUT & 3);
        float skip[CP];
#pragma unroll
        for (int i = 0; i < CP; ++i) skip[i] = a.d_skip && i < sh.valid ? a.d_skip[pl.c0 + sh.pc + i] : 0.f;
        for (int k = 0; k < STAGES - 1; ++k) {
            sh.fetch(sm.back[HAS_Y ? k : 0], tid);
            copies_commit();
        }
        for (int k = 0; k < ntiles; ++k) {
            const int w = k & 1, st = HAS_Y ? k % STAGES : 0;
            sh.fetch(sm.back[HAS_Y ? (k + STAGES - 1) % STAGES : 0], tid);
            copies_commit();
            copies_wait<STAGES - 1>();
            await(&sm.done[w], k >> 1);
            const int row = sh.tok[0], tok = first_tile + k * TT + row;
            if (tok < pl.hi && sh.valid > 0) {
                float2 sum[CP];   // over the lanes, of the two tokens
#pragma unroll
                for (int i = 0; i < CP; ++i) {
                    const float4 p = sm.y[w][HAS_Y ? row / 2 : 0][y_at(sh.pc + i, 0)], q = sm.y[w][HAS_Y ? row / 2 : 0][y_at(sh.pc + i, 1)];
                    sum[i] = add2(add2(make_float2(p.x, p.y), make_float2(p.z, p.w)), add2(make_float2(q.x, q.y), make_float2(q.z, q.w)));
                }
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    if (tok + it >= pl.hi) break;
                    float o[CP], x[CP], z[CP];
                    load_part<CP>(sm.back[st][0][it][tid], x);
                    if (gate) load_part<CP>(sm.back[st][1][it][tid], z);
#pragma unroll
                    for (int i = 0; i < CP; ++i) o[i] = fmaf(skip[i], x[i], it ? sum[i].y : sum[i].x);
                    if (gate) {
#pragma unroll
                        for (int i = 0; i < CP; ++i) o[i] *= z[i] * sigmoid_fast(z[i]);
                    }
                    store_part<TI, CP>(static_cast<TI*>(a.y) + (tok0 + tok + it) * a.D + pl.c0 + sh.pc, o, sh.valid, whole);
                }
            }
            hand_over(&sm.yfree[w]);
        }
    } else if (threadIdx.x >= RT) {
        // ---------------------------------------------------------------- in front of the recurrence
        const int tid = threadIdx.x - RT;
        Share<TI, Sh> sh;
        sh.start(tid, pl, first_tile, a.x, a.ldx, a.how >> SSM_X & 3, a.dt, a.lddt, a.how >> SSM_DT & 3, tok0);
        float bias[CP];
#pragma unroll
        for (int i = 0; i < CP; ++i) bias[i] = a.dt_bias && i < sh.valid ? a.dt_bias[pl.c0 + sh.pc + i] : 0.f;
        // pieces of b's and c's rows: a quarter's thread has the same lane group and row in each
        const int bl = tid & 3, brow = (tid / 4) % NROW, bvalid = a.S - bl * EL, bhow = a.how >> (brow ? SSM_C : SSM_B) & 3;
        const size_t bld = brow ? a.ldc : a.ldb;
        const TI* bsrc = static_cast<const TI*>(brow ? a.c : a.b) + (tok0 + first_tile) * bld + (size_t)pl.g * a.S + bl * EL;
        int bleft = pl.hi - first_tile;
        const bool bwhole = bvalid >= EL && bhow == 0 && EL * sizeof(TI) >= 4;
        size_t boff[PP];
#pragma unroll
        for (int p = 0; p < PP; ++p) boff[p] = (tid + p * PT) / (4 * NROW) * bld;
        auto fetch = [&](int k) {
            const int st = k % STAGES;
            sh.fetch(sm.front[st], tid);
            if (bwhole && bleft >= TT) {
#pragma unroll
                for (int p = 0; p < PP; ++p)
                    if (tid + p * PT < Sh::PIECES) copy_whole_async<TI, EL>(sm.bc[st][p][tid], bsrc + boff[p]);
                bsrc += TT * bld;
                bleft -= TT;
            } else if (bleft > 0) {
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    const int btok = (tid + p * PT) / (4 * NROW);
                    if (tid + p * PT < Sh::PIECES) copy_row_async<TI, EL>(sm.bc[st][p][tid], bsrc + btok * bld, btok < bleft ? bvalid : 0, bhow);
                }
                bsrc += TT * bld;
                bleft -= TT;
            }
            copies_commit();
        };
        for (int k = 0; k < STAGES - 1; ++k) fetch(k);
        constexpr uint32_t idesc = tc::idesc_bf16_abmn(128, COLS);
        const uint64_t adesc = tc::sdesc_mn(tc::smem_u32(sm.a), Sh::ATOM, 0);
        for (int k = 0; k < ntiles; ++k) {
            const int w = k & 1, st = k % STAGES;
            fetch(k + STAGES - 1);
            copies_wait<STAGES - 1>();
            if (k >= 2) await(&sm.done[w], (k >> 1) - 1);   // the buffers of tile k - 2
#pragma unroll
            for (int p = 0; p < PP; ++p)
                if (tid + p * PT < Sh::PIECES)
                    put_piece<EL>(sm.b[w], bl, ((tid + p * PT) / (4 * NROW) * NROW + brow) * EL, sm.bc[st][p][tid]);
            tc::fence_async_smem();
            tc::named_sync(1, PT);
            if (threadIdx.x < RT + 32) {
                tc::fence_after_sync();
                tc::mma_bf16_w(tmem + w * COLS, adesc, tc::sdesc_mn(tc::smem_u32(sm.b[w]), Sh::ATOM, 0), idesc, 0);
                tc::mma_commit_w(&sm.full[w]);
            }
            float2 dl[IT][CP / 2], u[IT][CP / 2];
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                float x[CP], dt[CP];
                load_part<CP>(sm.front[st][0][it][tid], x);
                load_part<CP>(sm.front[st][1][it][tid], dt);
#pragma unroll
                for (int i = 0; i < CP / 2; ++i) {
                    dl[it][i] = make_float2(dt[2 * i] + bias[2 * i], dt[2 * i + 1] + bias[2 * i + 1]);
                    if (a.softplus) dl[it][i] = ssm_softplus2(dl[it][i]);
                    u[it][i] = mul2(dl[it][i], make_float2(x[2 * i], x[2 * i + 1]));
                }
            }
            float4* du = sm.du[w][sh.tok[0] / 2];
#pragma unroll
            for (int i = 0; i < CP / 2; ++i) {
                du[du_at(sh.pc + 2 * i)] = make_float4(dl[0][i].x, u[0][i].x, dl[1][i].x, u[1][i].x);
                du[du_at(sh.pc + 2 * i + 1)] = make_float4(dl[0][i].y, u[0][i].y, dl[1][i].y, u[1][i].y);
            }
            hand_over(&sm.full[w]);
        }
        // The products are complete before the tensor memory goes back. The recurrence waits for them as well, but no longer
        // after a wait that gave up.
        if (threadIdx.x < RT + 32)
            for (int k = max(ntiles - 2, 0); k < ntiles; ++k)
                if (!tc::mbar_wait(&sm.full[k & 1], (k >> 1) & 1) && a.err) atomicOr(a.err, 2);
    } else {
        // ---------------------------------------------------------------- the recurrence
        const int tid = threadIdx.x, l = tid & 3, ch = tid >> 2, n0 = l * EL, d = pl.c0 + ch;
        const bool on = ch < pl.nch;
        const uint32_t lanes = tmem + ((uint32_t)((tid >> 5) & 3) << 21);   // this warp's quarter of the tensor memory's lanes
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
            // the earlier pieces of its sequence
            if (MODE != PIECE) join_pieces<EL>(a, a.hloc, pl.row, s.first / a.unit_len, pl.u, 1, d, n0, on, A2, h);
        }
        constexpr int N = 16 / EL;              // tokens of a batch of operands
        constexpr int NCOL = N * NROW * EL;     // their columns
        const int my_du = du_at(ch), my_y = y_at(ch, l >> 1);
        // PAIR: from an even tile row
        auto load_du = [&](bool pair, int w, int i, float2(&du)[N]) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (pair) {
                    if (j & 1) continue;
                    const float4 v = sm.du[w][(i + j) / 2][my_du];
                    du[j] = make_float2(v.x, v.y);
                    du[j + 1 < N ? j + 1 : j] = make_float2(v.z, v.w);
                } else {
                    du[j] = reinterpret_cast<const float2*>(&sm.du[w][(i + j) / 2][my_du])[(i + j) & 1];
                }
            }
        };
        // the first n tokens of a batch from tile row i
        auto run_tokens = [&](bool pair, int w, int i, int n, const float2(&du)[N], const uint32_t(&bc)[NCOL]) {
            float2 acc[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (j >= n) break;
                const float2 dl = make_float2(du[j].x, du[j].x), u = make_float2(du[j].y, du[j].y);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const int col = j * NROW * EL + 2 * e;
                    const float2 b = make_float2(__uint_as_float(bc[col]), __uint_as_float(bc[col + 1]));
                    const float2 g = ssm_exponent2(dl, make_float2(A2[2 * e], A2[2 * e + 1]));
                    const float2 hn = fma2(make_float2(ex2(g.x), ex2(g.y)), make_float2(h[2 * e], h[2 * e + 1]), mul2(u, b));
                    h[2 * e] = hn.x;
                    h[2 * e + 1] = hn.y;
                    if (HAS_Y) {
                        const int cc = HAS_Y ? col + EL : 0;
                        const float2 c = make_float2(__uint_as_float(bc[cc]), __uint_as_float(bc[cc + 1]));
                        acc[j] = e == 0 ? mul2(hn, c) : fma2(hn, c, acc[j]);
                    }
                }
                if (MODE == PIECE) sd += du[j].x;
            }
            if (HAS_Y) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (j >= n) break;
                    float* to = reinterpret_cast<float*>(&sm.y[w][HAS_Y ? (i + j) / 2 : 0][my_y]) + 2 * (l & 1);
                    if (pair) {
                        const int o = j + 1 < N ? j + 1 : j;
                        if (!(j & 1)) *reinterpret_cast<float2*>(to) = make_float2(acc[j].x + acc[j].y, acc[o].x + acc[o].y);
                    } else {
                        to[(i + j) & 1] = acc[j].x + acc[j].y;
                    }
                }
            }
        };
        auto checkpoint = [&](int tok) {
            const size_t slot = (size_t)pl.row * ((a.ax.len + SSM_CKPT - 1) / SSM_CKPT) + tok / SSM_CKPT;
            store_states<EL>(a.ckpt + slot * DS + (size_t)d * a.S, n0, a.S, on, h);
        };
        for (int k = 0; k < ntiles; ++k) {
            const int tb = first_tile + k * TT, te = min(tb + TT, pl.hi), w = k & 1;
            await(&sm.full[w], k >> 1);
            if (HAS_Y && k >= 2) await(&sm.yfree[w], (k >> 1) - 1);
            __syncwarp();
            tc::fence_after_sync();
            const uint32_t cols = lanes + w * COLS;
            t = tb;
            if (MODE != PIECE && t == s.end) {
                if (ht) store_states<EL>(ht + s.n * DS, n0, a.S, on, h);
                s = seq_next(a.ax, pl.row, s);
                init_state(s.n);
            }
            if (te - tb == TT && (MODE == PIECE || s.end >= te)) {
                // a whole tile of one sequence: the next tokens' operands are read while these run
                uint32_t bc[2][NCOL];
                float2 du[2][N];
                spread_load<NCOL>(cols, bc[0]);
                constexpr bool pair = N % 2 == 0;
                load_du(pair, w, 0, du[0]);
#pragma unroll
                for (int i = 0; i < TT; i += N) {
                    const int cur = (i / N) & 1;
                    if (HAS_CK && i % SSM_CKPT == 0 && (TT >= SSM_CKPT || (tb + i) % SSM_CKPT == 0)) checkpoint(tb + i);
                    tc::tmem_wait_ld();
                    if (i + N < TT) {
                        spread_load<NCOL>(cols + (i + N) * NROW * EL, bc[cur ^ 1]);
                        load_du(pair, w, i + N, du[cur ^ 1]);
                    }
                    run_tokens(pair, w, i, N, du[cur], bc[cur]);
                }
            } else {
                while (t < te) {
                    if (MODE != PIECE && t == s.end) {
                        if (ht) store_states<EL>(ht + s.n * DS, n0, a.S, on, h);
                        s = seq_next(a.ax, pl.row, s);
                        init_state(s.n);
                    }
                    if (HAS_CK && t % SSM_CKPT == 0) checkpoint(t);
                    int run = MODE == PIECE ? te : min(te, s.end);
                    if (HAS_CK) run = min(run, (t | (SSM_CKPT - 1)) + 1);
                    uint32_t bc[NCOL];
                    float2 du[N];
                    // a batch that starts near the tile's end would read past its columns: it starts earlier there
                    const int at = min(t - tb, TT - N);
                    spread_load<NCOL>(cols + at * NROW * EL, bc);
                    load_du(false, w, at, du);
                    tc::tmem_wait_ld();
                    const int skip = t - tb - at;
                    if (skip == 0 && t + N <= run) {
                        run_tokens(false, w, at, N, du, bc);
                        t += N;
                    } else {
                        // one token: the batch's entry `skip` brought to its front
#pragma unroll
                        for (int j = 1; j < N; ++j)
                            if (j == skip) {
                                du[0] = du[j];
#pragma unroll
                                for (int e = 0; e < NROW * EL; ++e) bc[e] = bc[j * NROW * EL + e];
                            }
                        run_tokens(false, w, t - tb, 1, du, bc);
                        ++t;
                    }
                }
            }
            tc::fence_before_sync();
            hand_over(&sm.done[w]);
        }
        if (pl.lo < pl.hi || !a.ax.cu) {
            if (MODE == PIECE) {
                store_states<EL>(a.hloc + pl.unit * DS + (size_t)d * a.S, n0, a.S, on, h);
                if (on && l == 0) a.sdt[(size_t)pl.unit * a.D + d] = sd;
            } else if (ht && pl.hi == s.end) {
                store_states<EL>(ht + s.n * DS, n0, a.S, on, h);
            }
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) tc::tmem_dealloc(tmem, Sh::ALLOC);
}

// A few tokens of each sequence (decoding): the state is the traffic, 8 bytes per value against 8 per channel for the
// token. The same four lanes per channel, NS sequences per thread so that their states are in flight together and A is
// formed once; everything is read directly. Of four sequences lane i forms sequence i's step for the channel's lanes, and
// after the exchange over them holds its output. WHOLE: the states fill the lanes and every row is aligned.
template <typename TI, int EL, int NS, bool WHOLE>
__global__ void __launch_bounds__(SSM_T, EL <= 4 ? (WHOLE ? 8 : 5) : 1) k_ssm_step(SsmArgs a) {
    static_assert(NS == 1 || NS == 4, "sequences per thread");
    constexpr int SC = SSM_T / 4;   // channels per CTA
    const int M = a.D / a.G, tpg = (M + SC - 1) / SC, tiles = tpg * a.G;
    const int sb = blockIdx.x / tiles, tile = blockIdx.x - sb * tiles, g = tile / tpg, tg = tile - g * tpg;
    const int l = threadIdx.x & 3, ch = threadIdx.x >> 2, n0 = l * EL, d = g * M + tg * SC + ch;
    const bool on = ch < M - tg * SC;
    const size_t DS = (size_t)a.D * a.S;
    const int B = a.ax.N, T = a.ax.len, s0 = sb * NS, valid = on ? a.S - n0 : 0;
    auto states = [&](const float* p, float(&v)[EL]) {
        if (WHOLE && EL >= 4) {
#pragma unroll
            for (int e = 0; e + 3 < EL; e += 4) {
                const float4 q = on ? *reinterpret_cast<const float4*>(p + e) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[e] = q.x; v[e + 1] = q.y; v[e + 2] = q.z; v[e + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) v[e] = e < valid ? p[e] : 0.f;
        }
    };
    auto row = [&](const TI* p, bool in, float(&v)[EL]) {
        if (WHOLE) {
            Raw<TI, EL> r;
            if (in) {
                constexpr int N = sizeof(r) > 16 ? sizeof(r) / 16 : 1;
                if (sizeof(r) > 16) {
#pragma unroll
                    for (int q = 0; q < N; ++q) reinterpret_cast<uint4*>(&r)[q] = reinterpret_cast<const uint4*>(p)[q];
                } else {
                    r = load_raw<TI, EL>(p);
                }
            } else {
#pragma unroll
                for (int e = 0; e < EL; ++e) r.v[e] = TI(0.f);
            }
            unpack<EL>(r, v);
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) v[e] = in && n0 + e < a.S ? ld(p + e) : 0.f;
        }
    };
    float A2[EL], h[NS][EL];
    const size_t base = (size_t)d * a.S + n0;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        if (a.h0 && s0 + i < B) {
            states(a.h0 + (s0 + i) * DS + base, h[i]);
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) h[i][e] = 0.f;
        }
    }
    states(a.A_log + base, A2);
    const float bias = a.dt_bias && on ? a.dt_bias[d] : 0.f, skip = a.d_skip && on ? a.d_skip[d] : 0.f;
    const int mine = s0 + (NS == 4 ? l : 0);   // the sequence whose step this lane forms and whose output it stores
    const bool own = on && mine < B;
    const TI* bp = static_cast<const TI*>(a.b) + (size_t)g * a.S + n0;
    const TI* cp = static_cast<const TI*>(a.c) + (size_t)g * a.S + n0;
    for (int t = 0; t < T; ++t) {
        const size_t tok = (size_t)mine * T + t;
        const float x = own ? ld(static_cast<const TI*>(a.x) + tok * a.ldx + d) : 0.f;
        const float dt = own ? ld(static_cast<const TI*>(a.dt) + tok * a.lddt + d) : 0.f;
        const float z = own && a.z ? ld(static_cast<const TI*>(a.z) + tok * a.ldz + d) : 0.f;
        float b[NS][EL], c[NS][EL], acc[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const size_t ti = (size_t)(s0 + i) * T + t;
            row(bp + ti * a.ldb, s0 + i < B, b[i]);
            row(cp + ti * a.ldc, s0 + i < B, c[i]);
        }
        if (t == 0) {
#pragma unroll
            for (int e = 0; e < EL; ++e) A2[e] = e < valid ? -expf(A2[e]) * LOG2E : 0.f;
        }
        float dl = dt + bias;
        if (a.softplus) dl = ssm_softplus(dl);
        const float u = dl * x;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const float di = NS == 4 ? __shfl_sync(SSM_FULL, dl, i, 4) : dl, ui = NS == 4 ? __shfl_sync(SSM_FULL, u, i, 4) : u;
            acc[i] = 0.f;
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                h[i][e] = fmaf(ssm_decay(di, A2[e]), h[i][e], ui * b[i][e]);
                acc[i] = fmaf(h[i][e], c[i][e], acc[i]);
            }
        }
        if (NS == 4) {
            halve<4>(acc, l, 2);
            halve<2>(acc, l, 1);
        } else {
            acc[0] += __shfl_xor_sync(SSM_FULL, acc[0], 2);
            acc[0] += __shfl_xor_sync(SSM_FULL, acc[0], 1);
        }
        if (own && (NS == 4 || l == 0)) {
            float o = fmaf(skip, x, acc[0]);
            if (a.z) o *= z * sigmoid_fast(z);
            st(static_cast<TI*>(a.y) + tok * a.D + d, o);
        }
    }
    if (a.ht) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            if (s0 + i >= B || !on) continue;
            float* p = a.ht + (s0 + i) * DS + base;
            if (WHOLE && EL >= 4) {
#pragma unroll
                for (int e = 0; e + 3 < EL; e += 4) *reinterpret_cast<float4*>(p + e) = make_float4(h[i][e], h[i][e + 1], h[i][e + 2], h[i][e + 3]);
            } else {
#pragma unroll
                for (int e = 0; e < EL; ++e)
                    if (e < valid) p[e] = h[i][e];
            }
        }
    }
}

int fwd_tiles(int D, int G) { return (D / G + CH - 1) / CH * G; }

template <typename TI, int EL, bool WHOLE>
void run_step_form(const SsmArgs& a, cudaStream_t st) {
    const unsigned tiles = (a.D / a.G + SSM_CH - 1) / SSM_CH * a.G;
    // four sequences per thread once that still leaves every SM two CTAs (4096 channels of 16 states: 64 sequences 7.6 us
    // against 12.6 with one per thread, 4 sequences 2.6 with one against 2.9)
    if ((long long)tiles * (a.ax.N / 4) >= 2 * sm_count())
        k_ssm_step<TI, EL, 4, WHOLE><<<tiles * ((a.ax.N + 3) / 4), SSM_T, 0, st>>>(a);
    else
        k_ssm_step<TI, EL, 1, WHOLE><<<tiles * a.ax.N, SSM_T, 0, st>>>(a);
}
template <typename TI, int EL>
void run_step(const SsmArgs& a, cudaStream_t st) {
    auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    const bool whole = a.S == 4 * EL && al(a.h0) && al(a.ht) && al(a.A_log) && !(a.how >> SSM_B & 3) && !(a.how >> SSM_C & 3);
    whole ? run_step_form<TI, EL, true>(a, st) : run_step_form<TI, EL, false>(a, st);
}

template <typename TI, int EL, int MODE>
cudaError_t run_one(const SsmArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)(a.ax.rows * a.units_row) * fwd_tiles(a.D, a.G);
    const int smem = (int)sizeof(typename FwdShape<TI, EL, MODE>::Smem) + 1024;
    static SmemLimit limit;
    const cudaError_t e = limit.set(reinterpret_cast<const void*>(k_ssm_fwd<TI, EL, MODE>), smem);
    if (e != cudaSuccess) return e;
    k_ssm_fwd<TI, EL, MODE><<<grid, FwdShape<TI, EL, MODE>::THREADS, smem, st>>>(a);
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
// Tokens per sequence up to which k_ssm_step takes them: it pays no start of tiles (5 us a wave of CTAs), the forward
// nothing for a token's latency. Measured, 4096 channels of 16 states: one sequence of 6 tokens 5.2 against 6.0 us, of 8
// 6.4 against 5.9; 8 sequences of 24 20.9 against 25.7, of 32 27 against 22; 64 of 24 104 against 165. 64 sequences, 1024
// channels of 64 states: 8 tokens 30 against 39, 16 tokens 52 against 47. The rule is coarse between the two: 3 sequences of
// 8 tokens (192 CTAs of the forward) 9.3 against 12.6, of 24 18.6 against 14.6; 5 of 8 9.1 against 17.1, of 24 18.7 against 20.7.
int step_tokens(const SsmArgs& a) {
    if ((long long)a.ax.rows * fwd_tiles(a.D, a.G) < 3 * sm_count()) return 6;
    return a.S <= 16 ? 24 : 12;
}

cudaError_t launch(const char* name, const SsmArgs& a, int bf16, int mode, cudaStream_t st) {
    cudaError_t r = cudaSuccess;
    const cudaError_t e = traced_launch(name, st, [&] {
        r = bf16 ? run_states<__nv_bfloat16>(a, mode, st) : run_states<float>(a, mode, st);
    });
    return r != cudaSuccess ? r : e;
}

}  // namespace

// Time pieces of a row. One CTA walks `len` tokens, and CTAs beyond the SMs wait for a further wave; with pieces each
// token is walked about twice (the pass for the pieces' states costs three quarters of the main one) and a CTA joins the
// pieces before its own. In units of a token's step: a CTA's fixed cost is about 64, a joined piece's about 2. The shortest
// pieces are 32 tokens. (Two rows of 1688 tokens and 32 channels, forward and backward: 98 us in pieces of 128 tokens joined
// one by one, 69 us so chosen and joined eight at a time.)
int ssm_units(int rows, int len, int D, int G, int S, bool backward) {
    const long long ctas = (long long)rows * (backward ? ssm_bwd_tiles(D, G, S) : fwd_tiles(D, G)), sms = sm_count();
    auto waves = [&](long long units) { return (ctas * units + sms - 1) / sms; };
    if (len <= 32 || ctas <= 0 || ctas > sms) return 1;
    long long best = 1, least = 4 * waves(1) * (len + 64);
    for (int wave = 1; wave <= 2; ++wave)
        for (int piece = 32; piece <= 128; piece *= 2) {
            const long long fit = wave * sms / ctas, most = (len + piece - 1) / piece, tried = fit < most ? fit : most;
            if (tried < 2) continue;
            const long long tokens = ((len + tried - 1) / tried + 31) / 32 * 32, units = (len + tokens - 1) / tokens;
            const long long cost = 7 * waves(units) * (tokens + 64) + 8 * units;
            if (cost < least) {
                least = cost;
                best = units;
            }
        }
    return (int)best;
}

cudaError_t launch_ssm_fwd(const SsmArgs& a, int bf16, int mode, cudaStream_t st) {
    if (mode == OUT && !a.ax.cu && a.ax.len > 0 && a.ax.len <= step_tokens(a))
        return traced_launch("k_ssm_step", st, [&] {
            bf16 ? run_step_states<__nv_bfloat16>(a, st) : run_step_states<float>(a, st);
        });
    return launch(mode == CKPT ? "k_ssm_ckpt" : "k_ssm_fwd", a, bf16, mode, st);
}

cudaError_t launch_ssm_pieces(const SsmArgs& a, int bf16, cudaStream_t st) {
    return launch("k_ssm_pieces", a, bf16, PIECE, st);
}

}  // namespace kda
