// Matrix product of e4m3 values with a scale for each 128 columns (include/kda.h):
//     y[m, n] = sum_g sa[m, g] sb[n, g] sum_{c in g} a[m, c] b[n, c].
// The scales vary along the contraction, so the tensor core sums one group at a time (four steps of K = 32 bytes, from
// zero, in TMEM) and warps add it, scaled, to the output's sums in registers, while the next groups are summed.
//
// Few rows (up to 64, or few tiles), k_mm8_rows: the tensor core's 128 rows are rows of b, its N are TN rows of a (16 to
// 128), so that the weights go once through the SM whatever the number of tokens; the contraction is cut over a cluster of
// up to 8 CTAs, whose sums meet in shared memory, in order. 64 x 4096 x 4096: 9.8 us on the device (floor 2.5: 17 MB), 1 x
// 4096 x 4096: 5.6; the launch, one load's latency and the meeting take most of the latter, the additions of 64 columns per
// group the rest.
// Many rows, k_mm8_pair: 16384 x 4096 x 4096 in 218 to 242 us, 2.3 to 2.5 PFLOP/s; with a scale per row of b (4096 x 4096 x
// 16384, fp32) 358. A group takes some 1000 cycles, of them 57% on the tensor cores: two sets of sums are all that fits
// TMEM, and a set is free again only when its warps have read all of it, 16 columns and one wait at a time. Kept out after
// measuring (us, against 225 to 240): the next 16 columns read ahead 287, 32 at a time 275 (both spill); sixteen warps of 64
// columns 284 against 222 (before the outputs went by TMA).
#include "kda_fp8.cuh"
#include "tc.cuh"

namespace kda {
namespace {

constexpr int G = FP8_GROUP;

struct Maps {
    CUtensorMap a, b, y;
};

// ------------------------------------------------------------------ rows that no tensor map takes
// Rows of K bytes, ld apart, to rows `pitch` apart (a multiple of 16; the bytes behind K are never read), 16 bytes to a
// thread: five whole words around them, shifted; byte by byte where those would reach behind the row.
__global__ void __launch_bounds__(256) k_mm8_align(const uint8_t* src, int64_t ld, uint8_t* dst, int64_t pitch, int K) {
    const uint8_t* s = src + (int64_t)blockIdx.x * ld;
    uint8_t* d = dst + (int64_t)blockIdx.x * pitch;
    const uint32_t off = reinterpret_cast<uintptr_t>(s) & 3;
    for (int c = threadIdx.x * 16; c < K; c += 256 * 16) {
        uint32_t w[5];
        if (c + 20 <= K) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(s + c - off);
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = q[i];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], off * 8);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) w[i] |= (c + 4 * i + k < K ? (uint32_t)s[c + 4 * i + k] : 0u) << (8 * k);
            }
        }
        *reinterpret_cast<uint4*>(d + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ------------------------------------------------------------------ few rows of a
constexpr int SB = 8;   // groups of scales brought in at a time

template <int TN>
struct Rows {
    static constexpr int BUF = TN <= 64 ? 4 : 2;                       // group sums in TMEM
    static constexpr int COLS = BUF * TN < 32 ? 32 : BUF * TN;         // TMEM columns (a power of two)
    static constexpr int STAGE = (G + TN) * 128;
    static constexpr int STAGES = 100 * 1024 / STAGE;                  // two CTAs on an SM
    static constexpr int PITCH = G + 4;                                // floats of a token's sums in shared memory
    struct Shared {
        float sa[4][4][TN];   // of four groups, each warp's own
        uint64_t full[STAGES], empty[STAGES], sum[BUF], free[BUF], drain;
        uint32_t tmem;
        int dead;
    };
    static constexpr int OFF = STAGES * STAGE;
    static constexpr int SMEM = OFF + (int)sizeof(Shared) + 1024;
    static_assert(TN * PITCH * 4 <= OFF, "the sums take the stages' place");
    static_assert(SMEM <= 232448, "shared memory above the per-block limit");
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 peer_load(uint32_t addr, uint32_t rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

// Grid: (contraction pieces, tiles of 128 rows of b, tiles of TN rows of a); a cluster is one tile's pieces. Four warps
// scale and add, one loads, one issues the products.
template <int TN>
__global__ void __launch_bounds__(192, 2) k_mm8_rows(const __grid_constant__ Maps maps, Mm8Args p) {
    using R = Rows<TN>;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (tc::smem_u32(raw) + 1023u) & ~1023u;
    unsigned char* mem = raw + (base - tc::smem_u32(raw));
    typename R::Shared& sm = *reinterpret_cast<typename R::Shared*>(mem + R::OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.y * G, m0 = blockIdx.z * TN;
    const int parts = gridDim.x, part = blockIdx.x;
    const int g0 = (int)((int64_t)p.groups * part / parts), g1 = (int)((int64_t)p.groups * (part + 1) / parts);
    if (warp == 4) {
        if (lane == 0) {
            for (int i = 0; i < R::STAGES; ++i) {
                tc::mbar_init(&sm.full[i], 1);
                tc::mbar_init(&sm.empty[i], 1);
            }
            for (int i = 0; i < R::BUF; ++i) {
                tc::mbar_init(&sm.sum[i], 1);
                tc::mbar_init(&sm.free[i], 4);
            }
            tc::mbar_init(&sm.drain, 1);
            sm.dead = 0;
            tc::fence_mbar_init();
        }
        __syncwarp();
    }
    const auto load = [&](int g) {   // lane 0 of the loader
        const int st = (g - g0) % R::STAGES;
        tc::mbar_arrive_expect_tx(&sm.full[st], R::STAGE);
        tc::tma_load2(base + st * R::STAGE, &maps.b, g * G, n0, &sm.full[st]);
        tc::tma_load2(base + st * R::STAGE + G * 128, &maps.a, g * G, m0, &sm.full[st]);
    };
    if (warp == 4 && lane == 0)
        for (int g = g0; g < g1 && g < g0 + R::STAGES; ++g) load(g);
    if (warp == 5) {
        tc::tmem_alloc(&sm.tmem, R::COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tb = sm.tmem;

    float acc[TN];
    if (warp < 4) {
#pragma unroll
        for (int t = 0; t < TN; ++t) acc[t] = 0.f;
        const int n = n0 + warp * 32 + lane;
        const float* sb = p.sb + (size_t)(p.b_rows ? min(n, p.N - 1) : blockIdx.y) * p.groups;
        for (int g = g0; g < g1; ++g) {
            const int i = g - g0, buf = i % R::BUF;
            if (i % 4 == 0) {
                __syncwarp();
                for (int t = lane; t < TN; t += 32) {
                    const float* sa = p.sa + (size_t)min(m0 + t, p.M - 1) * p.groups + g;
#pragma unroll
                    for (int k = 0; k < 4; ++k) sm.sa[warp][k][t] = g + k < g1 ? sa[k] : 0.f;
                }
                __syncwarp();
            }
            const float s = sb[g];
            if (!tc::warp_wait(&sm.sum[buf], (i / R::BUF) & 1, &sm.dead)) break;
            tc::fence_after_sync();
            const float* row = sm.sa[warp][i % 4];
#pragma unroll
            for (int c = 0; c < TN; c += 16) {
                float x[16];
                tc::tmem_ld16(tc::taddr(tb, warp * 32, buf * TN + c), x);
                tc::tmem_wait_ld();
#pragma unroll
                for (int t = 0; t < 16; t += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(row + c + t);
                    const float2 lo = fma2(make_float2(x[t], x[t + 1]), mul2(make_float2(s, s), make_float2(f.x, f.y)),
                                           make_float2(acc[c + t], acc[c + t + 1]));
                    const float2 hi = fma2(make_float2(x[t + 2], x[t + 3]), mul2(make_float2(s, s), make_float2(f.z, f.w)),
                                           make_float2(acc[c + t + 2], acc[c + t + 3]));
                    acc[c + t] = lo.x;
                    acc[c + t + 1] = lo.y;
                    acc[c + t + 2] = hi.x;
                    acc[c + t + 3] = hi.y;
                }
            }
            tc::fence_before_sync();
            tc::warp_arrive(&sm.free[buf]);
        }
    } else if (warp == 4) {
        int issued = min(g1 - g0, R::STAGES);
        for (; issued < g1 - g0; ++issued) {
            if (!tc::warp_wait(&sm.empty[issued % R::STAGES], (issued / R::STAGES - 1) & 1, &sm.dead)) break;
            if (lane == 0) load(g0 + issued);
            __syncwarp();
        }
        // no copy is in flight when the sums take the stages' place, after a failure either
        for (int i = max(0, issued - R::STAGES); i < issued; ++i) tc::mbar_wait(&sm.full[i % R::STAGES], (i / R::STAGES) & 1);
    } else {
        constexpr uint32_t I = tc::idesc_e4m3(G, TN);
        for (int g = g0; g < g1; ++g) {
            const int i = g - g0, buf = i % R::BUF, st = i % R::STAGES;
            if (!tc::warp_wait(&sm.full[st], (i / R::STAGES) & 1, &sm.dead)) break;
            if (i >= R::BUF && !tc::warp_wait(&sm.free[buf], (i / R::BUF - 1) & 1, &sm.dead)) break;
            tc::fence_after_sync();
            const uint32_t at = base + st * R::STAGE;
            tc::mma4_e4m3_w(tb + buf * TN, tc::sdesc(at), tc::sdesc(at + G * 128), I);
            tc::mma_commit_w(&sm.sum[buf]);
            tc::mma_commit_w(&sm.empty[st]);
        }
        // every product is done before the tensor memory goes back (after a failure, too)
        tc::mma_commit_w(&sm.drain);
        if (!tc::mbar_wait(&sm.drain, 0)) sm.dead = 1;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 5) tc::tmem_dealloc(tb, R::COLS);
    if (threadIdx.x == 0 && sm.dead && p.err) atomicOr(p.err, 2);

    // this CTA's sums as [token][row of b]; the cluster's added up in order
    float* sums = reinterpret_cast<float*>(mem);
    if (warp < 4) {
#pragma unroll
        for (int t = 0; t < TN; ++t) sums[t * R::PITCH + threadIdx.x] = acc[t];
    }
    cluster_sync();
    if (warp < 4) {
        const uint32_t rank = cluster_rank(), size = cluster_size();
        const int nq = n0 + lane * 4;
        const bool wide = p.N % 4 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15) == 0;
        for (int t = rank * 4 + warp; t < TN; t += 4 * size) {
            const int m = m0 + t;
            if (m >= p.M) break;
            const uint32_t at = base + (t * R::PITCH + lane * 4) * 4;
            float4 x[8];   // all of them on their way at once
#pragma unroll
            for (uint32_t r = 0; r < 8; ++r)
                if (r < size) x[r] = peer_load(at, r);
            float4 s = x[0];
#pragma unroll
            for (uint32_t r = 1; r < 8; ++r)
                if (r < size) {
                    s.x += x[r].x;
                    s.y += x[r].y;
                    s.z += x[r].z;
                    s.w += x[r].w;
                }
            const size_t to = (size_t)m * p.N + nq;
            if (wide && nq < p.N) {
                if (p.f32) *reinterpret_cast<float4*>(static_cast<float*>(p.y) + to) = s;
                else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + to) = make_uint2(tc::pack_bf16(s.x, s.y), tc::pack_bf16(s.z, s.w));
            } else {
                const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (nq + i >= p.N) break;
                    if (p.f32) static_cast<float*>(p.y)[to + i] = v[i];
                    else static_cast<__nv_bfloat16*>(p.y)[to + i] = __float2bfloat16_rn(v[i]);
                }
            }
        }
    }
    cluster_sync();   // no CTA ends while its sums are read
}

template <int TN>
cudaError_t run_rows(const Mm8Args& p, cudaStream_t st) {
    using R = Rows<TN>;
    Maps maps;
    if (!tmap_rows_u8(&maps.a, p.a, p.M, p.K, p.lda, TN) || !tmap_rows_u8(&maps.b, p.b, p.N, p.K, p.ldb, G)) return cudaErrorInvalidValue;
    static SmemLimit limit;
    const cudaError_t e = limit.set(reinterpret_cast<const void*>(&k_mm8_rows<TN>), R::SMEM);
    if (e != cudaSuccess) return e;
    const int tn = (p.N + G - 1) / G, tm = (p.M + TN - 1) / TN;
    int parts = 1;   // pieces of two groups at least, while they fit one round of the SMs, two on each
    while (parts < 8 && 4 * parts <= p.groups && (long long)parts * tn * tm <= sm_count()) parts *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(parts, tn, tm);
    cfg.blockDim = dim3(192);
    cfg.dynamicSmemBytes = R::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = parts;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    cudaError_t launched = cudaSuccess;
    const cudaError_t last = traced_launch("k_mm8_rows", st, [&] { launched = cudaLaunchKernelEx(&cfg, k_mm8_rows<TN>, maps, p); });
    return launched != cudaSuccess ? launched : last;
}

// ------------------------------------------------------------------ many rows of a
// Two CTAs share a tile of 256 x 256: each loads its 128 rows of a and 128 of b, the tensor cores read the other's rows of b
// over the pair, so that an SM's shared memory carries 64 KB per group in place of 96 (a tile of 128 x 256 by itself), for 512
// cycles of products. A CTA's sums are 128 rows x 256 columns, 128 columns
// of one row to a thread of eight warps.
constexpr int P_STAGES = 5, P_STAGE = 2 * G * 128, P_COLS = 256, P_W = 128, P_ADDERS = 8;   // columns of an adding thread, adding warps
constexpr int P_LOADER = 8, P_ISSUER = 9, P_SCALES = 10, P_THREADS = 12 * 32;   // (the twelfth completes a warpgroup)
constexpr int P_REGS_ADD = 208, P_REGS_REST = 88;   // 2 x 208 + 88 = 3 x 168, what a block of 384 threads starts with
constexpr int P_OUT = 32 * 128;                     // bytes of outputs on their way, for each adding warp
struct PairShared {
    float sa[2][SB][G + 4], sb[2][SB][P_COLS + 4];   // scales of SB groups: of this CTA's rows of a, of the tile's rows of b (or, one
                                             // for 128 of them, in the first two places)
    uint64_t full[P_STAGES], empty[P_STAGES], sum[2], free[2], s_full[2], s_free[2];
    uint32_t tmem;
    int dead;
};
constexpr int P_OFF_OUT = P_STAGES * P_STAGE, P_OFF = P_OFF_OUT + P_ADDERS * P_OUT, P_SMEM = P_OFF + (int)sizeof(PairShared) + 1024;
static_assert(P_SMEM <= 232448, "shared memory above the per-block limit");

// BROWS: a scale per row of b, else per 128 rows. Clusters of two walk the tiles.
template <bool BROWS>
__global__ void __launch_bounds__(P_THREADS, 1) k_mm8_pair(const __grid_constant__ Maps maps, Mm8Args p, int tiles_m, int tiles, int tma_out) {
    extern __shared__ unsigned char raw[];
    const uint32_t base = (tc::smem_u32(raw) + 1023u) & ~1023u;
    unsigned char* mem = raw + (base - tc::smem_u32(raw));
    PairShared& sm = *reinterpret_cast<PairShared*>(mem + P_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < P_STAGES; ++i) {
            tc::mbar_init(&sm.full[i], 1);
            tc::mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sm.sum[i], 1);
            tc::mbar_init(&sm.free[i], 2 * P_ADDERS);
            tc::mbar_init(&sm.s_full[i], 1);
            tc::mbar_init(&sm.s_free[i], P_ADDERS);
        }
        sm.dead = 0;
        tc::fence_mbar_init();
    }
    if (warp == P_ISSUER) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_u32(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers are set up
    tc::fence_after_sync();
    const uint32_t tb = sm.tmem;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (warp < P_ADDERS) {
        tc::regs_more<P_REGS_ADD>();
        const int quad = warp & 3, part = warp >> 2;
        const uint32_t ta = tc::taddr(tb, quad * 32, part * P_W), lead = tc::peer_smem(tc::smem_u32(sm.free), 0);
        uint32_t i = 0, round = 0;   // groups, and rounds of scales, so far
        const uint32_t out = P_OFF_OUT + warp * P_OUT;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            const int m = t % tiles_m * 256 + rank * 128 + quad * 32 + lane, n0 = t / tiles_m * 256 + part * P_W;
            float acc[P_W];
#pragma unroll
            for (int c = 0; c < P_W; ++c) acc[c] = 0.f;
            const float* sa = p.sa + (size_t)min(m, p.M - 1) * p.groups;
            const float* sb = p.sb + (size_t)(BROWS ? 0 : min(n0, p.N - 1) / G) * p.groups;
            const auto scale = [&](uint32_t from, int g) {   // of this row, and of b's rows where they share one
                return BROWS ? sm.sa[from][g % SB][quad * 32 + lane] : sa[g] * sb[g];
            };
            float s = BROWS ? 0.f : scale(0, 0);   // the present group's: read while the group before it is added
            for (int g = 0; g < p.groups; ++g, ++i) {
                const uint32_t buf = i & 1, from = round & 1;
                if (BROWS && g % SB == 0) {
                    if (!(ok = tc::warp_wait(&sm.s_full[from], round >> 1 & 1, &sm.dead))) break;
                    s = scale(from, g);
                }
                const float* col = &sm.sb[from][g % SB][part * P_W];
                const float2 s2 = make_float2(s, s);
                if (!BROWS && g + 1 < p.groups) s = scale(0, g + 1);
                if (!(ok = tc::warp_wait(&sm.sum[buf], i >> 1 & 1, &sm.dead))) break;
                tc::fence_after_sync();
#pragma unroll
                for (int c = 0; c < P_W; c += 16) {
                    float y[16];
                    tc::tmem_ld16(ta + buf * P_COLS + c, y);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        float2 lo = s2, hi = s2;
                        if (BROWS) {
                            const float4 f = *reinterpret_cast<const float4*>(col + c + k);
                            lo = mul2(s2, make_float2(f.x, f.y));
                            hi = mul2(s2, make_float2(f.z, f.w));
                        }
                        lo = fma2(make_float2(y[k], y[k + 1]), lo, make_float2(acc[c + k], acc[c + k + 1]));
                        hi = fma2(make_float2(y[k + 2], y[k + 3]), hi, make_float2(acc[c + k + 2], acc[c + k + 3]));
                        acc[c + k] = lo.x;
                        acc[c + k + 1] = lo.y;
                        acc[c + k + 2] = hi.x;
                        acc[c + k + 3] = hi.y;
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                const bool last = g % SB == SB - 1 || g + 1 == p.groups;
                if (lane == 0) {
                    tc::peer_arrive(lead + 8 * buf);
                    if (BROWS && last) tc::mbar_arrive(&sm.s_free[from]);
                }
                if (BROWS && !last) s = scale(from, g + 1);
                round += last;
            }
            if (!ok) break;
            if (tma_out) {   // 128 bytes of the warp's 32 rows at a time
                const auto piece = [&](int c, auto&& words) {
                    if (lane == 0) tc::bulk_wait_read();
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(mem + out + lane * 128 + ((k ^ (lane & 7)) << 4)) = words(k);
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (n0 + c < p.N && m < p.M) tc::tma_store2(&maps.y, n0 + c, m, base + out);
                        tc::bulk_commit();
                    }
                };
                if (p.f32) {
#pragma unroll
                    for (int c = 0; c < P_W; c += 32)
                        piece(c, [&](int k) {
                            const float* v = acc + c + 4 * k;
                            return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
                        });
                } else {
#pragma unroll
                    for (int c = 0; c < P_W; c += 64)
                        piece(c, [&](int k) {
                            const float* v = acc + c + 8 * k;
                            return make_uint4(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]), tc::pack_bf16(v[4], v[5]), tc::pack_bf16(v[6], v[7]));
                        });
                }
            } else if (m < p.M) {   // rows that no tensor map takes
                const int left = p.N - n0;
                if (p.f32) {
                    float* y = static_cast<float*>(p.y) + (size_t)m * p.N + n0;
#pragma unroll
                    for (int c = 0; c < P_W; ++c)
                        if (c < left) y[c] = acc[c];
                } else {
                    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + (size_t)m * p.N + n0;
#pragma unroll
                    for (int c = 0; c < P_W; ++c)
                        if (c < left) y[c] = __float2bfloat16_rn(acc[c]);
                }
            }
        }
        if (lane == 0) tc::bulk_wait_all();
        __syncwarp();
    } else {
        tc::regs_less<P_REGS_REST>();
    }
    if (warp == P_LOADER) {
        uint32_t i = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            const int m0 = t % tiles_m * 256 + rank * 128, n0 = t / tiles_m * 256 + rank * 128;
            for (int g = 0; g < p.groups; ++g, ++i) {
                const uint32_t st = i % P_STAGES;
                if (i >= P_STAGES && !(ok = tc::warp_wait(&sm.empty[st], (i / P_STAGES - 1) & 1, &sm.dead))) break;
                if (lane == 0) {
                    // the pair's products wait for both CTAs' rows on one barrier, that of rank 0
                    if (rank == 0) tc::mbar_arrive_expect_tx(&sm.full[st], 2 * P_STAGE);
                    const uint32_t bar = tc::peer_smem(tc::smem_u32(&sm.full[st]), 0);
                    tc::tma_load2_pair(base + st * P_STAGE, &maps.a, g * G, m0, bar);
                    tc::tma_load2_pair(base + st * P_STAGE + G * 128, &maps.b, g * G, n0, bar);
                }
                __syncwarp();
            }
        }
        // every copy has been read when the CTA ends (a failure's have had this wait's second to land)
        for (uint32_t k = i > P_STAGES ? i - P_STAGES : 0; k < i; ++k) tc::mbar_wait(&sm.empty[k % P_STAGES], (k / P_STAGES) & 1);
    } else if (warp == P_ISSUER && rank == 0) {
        constexpr uint32_t I = tc::idesc_e4m3(256, 256);
        uint32_t i = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step)
            for (int g = 0; g < p.groups; ++g, ++i) {
                const uint32_t st = i % P_STAGES, buf = i & 1;
                if (!(ok = tc::warp_wait(&sm.full[st], (i / P_STAGES) & 1, &sm.dead))) break;
                if (i >= 2 && !(ok = tc::warp_wait(&sm.free[buf], ((i >> 1) - 1) & 1, &sm.dead))) break;
                tc::fence_after_sync();
                const uint32_t at = base + st * P_STAGE;
                tc::mma4_e4m3_pair_w(tb + buf * P_COLS, tc::sdesc(at), tc::sdesc(at + G * 128), I);
                tc::mma_commit_pair_w(&sm.sum[buf]);
                tc::mma_commit_pair_w(&sm.empty[st]);
            }
    } else if (warp == P_SCALES && BROWS) {
        uint32_t round = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            const int m0 = t % tiles_m * 256 + rank * 128, n0 = t / tiles_m * 256;
            for (int g = 0; g < p.groups; g += SB, ++round) {
                if (round >= 2 && !(ok = tc::warp_wait(&sm.s_free[round & 1], ((round >> 1) - 1) & 1, &sm.dead))) break;
                // 8 lanes read a row's SB neighbouring scales, 4 rows at a time, 64 rows in flight; rows of the copies are 4
                // words off a bank's multiple, so that the lanes' words lie in banks of their own
                static_assert(SB == 8, "a row's scales are 8 lanes'");
                const int k = lane & 7, r4 = lane >> 3;
                const auto copy = [&](const float* from, int row, int rows, float* to, int pitch) {
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        v[i] = g + k < p.groups ? from[(size_t)min(row + 4 * i + r4, rows - 1) * p.groups + g + k] : 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[k * pitch + 4 * i + r4] = v[i];
                };
                for (int r = 0; r < G; r += 64) copy(p.sa, m0 + r, p.M, &sm.sa[round & 1][0][r], G + 4);
                for (int r = 0; r < P_COLS; r += 64) copy(p.sb, n0 + r, p.N, &sm.sb[round & 1][0][r], P_COLS + 4);
                tc::warp_arrive(&sm.s_full[round & 1]);
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();   // neither CTA's memory goes back while the other uses it
    tc::fence_after_sync();
    if (threadIdx.x == 0 && sm.dead && p.err) atomicOr(p.err, 2);
    if (warp == P_ISSUER) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tb) : "memory");
}

template <bool BROWS>
cudaError_t run_pair(const Mm8Args& p, cudaStream_t st) {
    Maps maps;
    if (!tmap_rows_u8(&maps.a, p.a, p.M, p.K, p.lda, G) || !tmap_rows_u8(&maps.b, p.b, p.N, p.K, p.ldb, G)) return cudaErrorInvalidValue;
    static SmemLimit limit;
    const cudaError_t e = limit.set(reinterpret_cast<const void*>(&k_mm8_pair<BROWS>), P_SMEM);
    if (e != cudaSuccess) return e;
    const int tma_out = tmap_matrix(&maps.y, p.y, p.M, p.N, p.f32, 32) ? 1 : 0;
    const int tm = (p.M + 255) / 256, tn = (p.N + 255) / 256, tiles = tm * tn;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(P_THREADS);
    cfg.dynamicSmemBytes = P_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    static std::atomic<int> fit[64];   // pairs that the device runs at once (not every SM has a partner)
    int dev = 0, pairs = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
    if (dev < 64) pairs = fit[dev].load(std::memory_order_relaxed);
    if (!pairs) {
        if (cudaOccupancyMaxActiveClusters(&pairs, k_mm8_pair<BROWS>, &cfg) != cudaSuccess || pairs < 1) {
            (void)cudaGetLastError();
            pairs = sm_count() / 2;
        }
        if (dev < 64) fit[dev].store(pairs, std::memory_order_relaxed);
    }
    cfg.gridDim = dim3(2 * (tiles < pairs ? tiles : pairs));
    cudaError_t launched = cudaSuccess;
    const cudaError_t last = traced_launch("k_mm8_pair", st, [&] { launched = cudaLaunchKernelEx(&cfg, k_mm8_pair<BROWS>, maps, p, tm, tiles, tma_out); });
    return launched != cudaSuccess ? launched : last;
}

bool on16(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 16 == 0; }
size_t pitch_of(int K) { return ((size_t)K + 15) / 16 * 16; }

}  // namespace

size_t mm8_align_bytes(const Mm8Args& p) {
    return (on16(p.a, p.lda) ? 0 : ((size_t)p.M * pitch_of(p.K) + 255) / 256 * 256) + (on16(p.b, p.ldb) ? 0 : (size_t)p.N * pitch_of(p.K));
}

cudaError_t launch_mm8(Mm8Args p, void* ws, cudaStream_t st) {
    uint8_t* free = static_cast<uint8_t*>(ws);
    const auto align = [&](const uint8_t*& x, int64_t& ld, int rows) {
        if (on16(x, ld)) return cudaSuccess;
        const int64_t pitch = (int64_t)pitch_of(p.K);
        const uint8_t* src = x;
        uint8_t* dst = free;
        const cudaError_t e = traced_launch("k_mm8_align", st, [&] { k_mm8_align<<<rows, 256, 0, st>>>(src, ld, dst, pitch, p.K); });
        x = dst;
        ld = pitch;
        free += ((size_t)rows * pitch + 255) / 256 * 256;
        return e;
    };
    cudaError_t e = align(p.a, p.lda, p.M);
    if (e != cudaSuccess || (e = align(p.b, p.ldb, p.N)) != cudaSuccess) return e;
    // Tiles of 256 x 256 for pairs of SMs from 17 of them on, if a has more than 64 rows: fewer leave most of a tile empty, at
    // the time of a whole one. (us, tiles of 128 rows of b against pairs, b from HBM. K 4096, blocks, bf16: M 1, N 2048 6.1
    // against 17.0, N 8192 9.3, 18.2, N 131072 84, 161; M 64, N 4096 10.6, 17.6, N 8192 13.1, 17.9, N 16384 19.5, 18.9, N
    // 131072 118, 105; M 128, N 4096 14.7, 18.5, N 8192 19.2, 18.8, N 16384 30.8, 20.0; M 256, N 4096 18.9, 18.6, N 8192 30.4,
    // 18.9; M 512, N 2048 18.6, 18.4, N 4096 30.0, 18.7. K 1024: M 64, N 8192 7.9, 8.7, N 131072 46, 36; M 256, N 4096 10.5,
    // 8.8. K 16384: M 64, N 8192 31, 55; M 256, N 4096 50, 58; M 1280, N 1280, rows, fp32 99, 93. Rows, fp32, K 4096: M 64, N
    // 32768 37, 54; M 128, N 8192 20.5, 30.7, N 16384 33.1, 31.8; M 256, N 4096 19.8, 31.1, N 8192 32.1, 31.2.)
    if (p.M > 64 && (long long)((p.M + 255) / 256) * ((p.N + 255) / 256) * 9 >= sm_count()) return p.b_rows ? run_pair<true>(p, st) : run_pair<false>(p, st);
    if (p.M <= 16) return run_rows<16>(p, st);
    if (p.M <= 32) return run_rows<32>(p, st);
    if (p.M <= 64) return run_rows<64>(p, st);
    return run_rows<128>(p, st);
}

}  // namespace kda
