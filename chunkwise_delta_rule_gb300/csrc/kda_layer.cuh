// Shared declarations of the layer operators around the delta rule: the short
// causal convolution (kda_conv.cu), the selective state space scan (kda_ssm.cu,
// kda_ssm_bwd.cu) and the root-mean-square norm (kda_norm.cu).
#pragma once

#include <atomic>

#include "kda_internal.cuh"

namespace kda {

// Tracing hooks of kda_api.cu (kda_profile_begin): a pair of events around one launch; -1 when tracing
// is off.
int trace_open(const char* name, cudaStream_t st);
void trace_close(int id, cudaStream_t st);

template <class F>
cudaError_t traced_launch(const char* name, cudaStream_t st, F&& launch) {
    const int id = trace_open(name, st);
    launch();
    trace_close(id, st);
    return cudaGetLastError();
}

// A kernel's dynamic shared memory limit, raised once per device.
struct SmemLimit {
    std::atomic<uint64_t> done{0};
    cudaError_t set(const void* kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
};

// The token axis: equal-length sequences are `rows` rows of `len` tokens, one sequence each; packed
// sequences are one row of all tokens, cut by the N + 1 offsets in cu.
struct TokenAxis {
    const int32_t* cu;
    int N;      // sequences
    int rows, len;
};

// Offset cu[n], kept inside the token axis whatever the caller's array holds.
__device__ __forceinline__ int axis_cu(const TokenAxis& ax, int n) { return min(max(ax.cu[n], 0), ax.len); }

// Packed axis: the sequence that holds token t (the first n with cu[n + 1] > t; the last sequence when
// inconsistent offsets leave t to none).
__device__ __forceinline__ int axis_find(const TokenAxis& ax, int t) {
    int lo = 0, hi = ax.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (axis_cu(ax, mid + 1) > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

struct Seq {
    int n, first, end;    // sequence, its first token and its end on the row
};

// The sequence holding token t of the row; first <= t < end whatever the offsets hold.
__device__ __forceinline__ Seq seq_at(const TokenAxis& ax, int row, int t) {
    if (!ax.cu) return {row, 0, ax.len};
    Seq s;
    s.n = axis_find(ax, t);
    s.first = min(axis_cu(ax, s.n), t);
    s.end = axis_cu(ax, s.n + 1);
    if (s.end <= t) s.end = ax.len;
    return s;
}

// The sequences behind and before s on its row (which has tokens there): the neighbour's one offset where it has tokens,
// instead of a search of the offsets.
__device__ __forceinline__ Seq seq_next(const TokenAxis& ax, int row, const Seq& s) {
    if (ax.cu && s.n + 1 < ax.N) {
        const int end = axis_cu(ax, s.n + 2);
        if (end > s.end) return {s.n + 1, s.end, end};
    }
    return seq_at(ax, row, s.end);
}
__device__ __forceinline__ Seq seq_prev(const TokenAxis& ax, int row, const Seq& s) {
    if (ax.cu && s.n > 0) {
        const int first = axis_cu(ax, s.n - 1);
        if (first < s.first) return {s.n - 1, first, s.first};
    }
    return seq_at(ax, row, s.first - 1);
}

// Packed axis: sets bit 0 of *err when cu does not start at 0, decreases, or does not end at the token
// count. Called by one whole CTA.
__device__ __forceinline__ void axis_check(const TokenAxis& ax, int32_t* err) {
    if (!ax.cu || !err) return;
    bool bad = false;
    for (int n = threadIdx.x; n < ax.N; n += blockDim.x) bad |= ax.cu[n + 1] < ax.cu[n];
    if (threadIdx.x == 0) bad |= ax.cu[0] != 0 || ax.cu[ax.N] != ax.len;
    if (bad) atomicOr(err, 1);
}

// 2^x (2^-22 relative; the argument already carries one fp32 rounding) and 1 / x.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp(1.f + ex2(-LOG2E * x)); }

// Packed pairs of fp32 (one instruction for two lanes of work).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return d;
}

// V consecutive elements of a row as fp32: 16-byte accesses when `vec` (V elements, aligned), else
// element by element with the ones past `valid` read as zero (not stored).
template <int V>
__device__ __forceinline__ void load_row(const float* p, float (&x)[V], int valid, bool vec) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 v = reinterpret_cast<const float4*>(p)[i];
            x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < valid ? p[i] : 0.f;
    }
}
template <int V>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&x)[V], int valid, bool vec) {
    if (V >= 8 && vec) {
#pragma unroll
        for (int i = 0; i < V / 8; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < valid ? __bfloat162float(p[i]) : 0.f;
    }
}
template <int V>
__device__ __forceinline__ void store_row(float* p, const float (&x)[V], int valid, bool vec) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < valid) p[i] = x[i];
    }
}
template <int V>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&x)[V], int valid, bool vec) {
    if (V >= 8 && vec) {
#pragma unroll
        for (int i = 0; i < V / 8; ++i) {
            uint4 v;
            __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
            reinterpret_cast<uint4*>(p)[i] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < valid) p[i] = __float2bfloat16_rn(x[i]);
    }
}

// Asynchronous copies of a thread's own data into shared memory: n elements of a row of V (zeros past n), in one or two
// whole accesses (`how` 0), 4-byte ones (1) or, for odd 16-bit addresses, plain ones (2).
// (The slow forms stay out of line: in line at every call they pushed the callers' loops out of the instruction cache.)
template <typename TI, int V>
__device__ __noinline__ void copy_row_slow(TI* dst, const TI* src, int n, int how) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if (how <= 1) {
        constexpr int PER = 4 / sizeof(TI);
#pragma unroll
        for (int i = 0; i < V / PER; ++i) {
            const int left = min(max(n - i * PER, 0), PER) * (int)sizeof(TI);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d + 4 * i), "l"(src + (left > 0 ? i * PER : 0)), "r"(left) : "memory");
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) dst[i] = i < n ? src[i] : TI(0.f);
    }
}
template <typename TI, int V>
__device__ __forceinline__ void copy_row_async(TI* dst, const TI* src, int n, int how) {
    constexpr int BYTES = V * (int)sizeof(TI), ONE = BYTES < 16 ? BYTES : 16;
    if (how == 0 && (n >= V || n <= 0)) {
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
        const char* p = reinterpret_cast<const char*>(src);
        const int full = n > 0 ? ONE : 0;
#pragma unroll
        for (int i = 0; i < BYTES / ONE; ++i) {
            if (ONE == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + 16 * i), "l"(p + (n > 0 ? 16 * i : 0)), "r"(full) : "memory");
            else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(p), "n"(ONE < 16 ? ONE : 8), "r"(full) : "memory");
        }
    } else {
        copy_row_slow<TI, V>(dst, src, n, how);
    }
}
// The same of a row that is there and aligned.
template <typename TI, int V>
__device__ __forceinline__ void copy_whole_async(TI* dst, const TI* src) {
    constexpr int BYTES = V * (int)sizeof(TI), ONE = BYTES < 16 ? BYTES : 16;
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
#pragma unroll
    for (int i = 0; i < BYTES; i += ONE) {
        if (ONE == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + i), "l"(reinterpret_cast<const char*>(src) + i) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d + i), "l"(reinterpret_cast<const char*>(src) + i), "n"(ONE < 16 ? ONE : 8) : "memory");
    }
}
template <typename TI>
__device__ __forceinline__ void copy8_async(TI* dst, const TI* src, int n, int how) { copy_row_async<TI, 8>(dst, src, n, how); }
// One aligned access of 4, 8 or 16 bytes, asynchronously.
template <typename R>
__device__ __forceinline__ void copy_async(R* dst, const void* src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if (sizeof(R) == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(sizeof(R) == 16 ? 8 : sizeof(R)) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// V elements of a row as they lie in memory (one access of up to 16 bytes when V > 1), and their values as pairs.
template <typename TI, int V>
struct alignas(sizeof(TI) * V > 16 ? 16 : sizeof(TI) * V) Raw {
    TI v[V];
};
template <int V>
__device__ __forceinline__ void unpack(const Raw<float, V>& r, float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = r.v[i];
}
template <int V>
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, V>& r, float (&x)[V]) {
    if (V == 1) {
        x[0] = __bfloat162float(r.v[0]);
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <typename TI, int V>
__device__ __forceinline__ Raw<TI, V> load_raw(const TI* p) { return *reinterpret_cast<const Raw<TI, V>*>(p); }
template <int V>
__device__ __forceinline__ void store_values(float* p, const float (&x)[V]) {
    Raw<float, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = x[i];
    *reinterpret_cast<Raw<float, V>*>(p) = r;
}
template <int V>
__device__ __forceinline__ void store_values(__nv_bfloat16* p, const float (&x)[V]) {
    Raw<__nv_bfloat16, V> r;
    if (V == 1) {
        r.v[0] = __float2bfloat16_rn(x[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[V > 1 ? 2 * i + 1 : 0]);
            reinterpret_cast<__nv_bfloat162*>(&r)[i] = h;
        }
    }
    *reinterpret_cast<Raw<__nv_bfloat16, V>*>(p) = r;
}

// Sums over `parts` rows of `n` columns in a fixed order: a CTA of 32 columns x 8 groups of rows (a group's rows in
// order, then the groups in order). Returns the total to the threads of group 0 (column -1 elsewhere).
__device__ __forceinline__ int sum_parts(const float* part, int parts, size_t n, float& total) {
    __shared__ float red[8][32];
    const int lx = threadIdx.x & 31, ly = threadIdx.x >> 5;
    const size_t c = (size_t)blockIdx.x * 32 + lx;
    float s = 0.f;
    if (c < n) {
#pragma unroll 8
        for (int p = ly; p < parts; p += 8) s += part[p * n + c];
    }
    red[ly][lx] = s;
    __syncthreads();
    total = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) total += red[k][lx];
    return ly == 0 && c < n ? (int)c : -1;
}

// ------------------------------------------------------------------ launchers
struct ConvArgs {
    TokenAxis ax;
    int D, W, silu, tile, ntiles, groups;   // tokens per thread; tiles of all rows; channel groups of V channels
    int tiles_row;                          // tiles per row
    int gx;                                 // channel groups side by side in a CTA (a power of two)
    size_t ldx;
    const void *x, *h0;
    const float *weight, *bias;
    void *y, *final_state;
    int32_t* err;
    // backward
    const void *dy, *dfinal;
    void *dx, *dinit;
    float *dweight, *dbias, *part;          // part: [parts][W + 1][D] sums of blocks of tiles
    int parts;
};
// Channels per thread (4 on the vector path, else 1), tokens per thread and block counts.
void conv_shape(ConvArgs& a, bool vec, bool backward);
cudaError_t launch_conv_fwd(ConvArgs a, int bf16, bool vec, cudaStream_t st);
cudaError_t launch_conv_bwd(ConvArgs a, int bf16, bool vec, cudaStream_t st);

struct NormArgs {
    int rows, D, out, group, ngroups;   // out: 0 the I/O type, 1 e4m3 with scales
    float eps;
    const void *x, *residual;
    const float* weight;
    void *y, *h;
    float* scale;
    // backward
    const void *dy, *dres;
    void* dx;
    float *dweight, *part;
    int parts;
};
int norm_bwd_parts(int rows, int D);
constexpr int NORM_MAX_D = 16384;
cudaError_t launch_norm_fwd(const NormArgs& a, int bf16, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormArgs& a, int bf16, cudaStream_t st);

// Checkpoint interval of the scan's saved states, in tokens.
constexpr int SSM_CKPT = 16;

// How the scan reaches the rows of its tensors, two bits each: 0 in 16-byte accesses, 1 in 4-byte ones, 2 element by
// element (see copy_row_async).
enum { SSM_X = 0, SSM_DT = 2, SSM_Z = 4, SSM_B = 6, SSM_C = 8, SSM_DY = 10, SSM_OUT = 12 };

struct SsmArgs {
    TokenAxis ax;
    int D, S, G, softplus;     // channels, states per channel, groups of b, c
    int how;                   // access to each tensor's rows (SSM_X ...)
    int units_row, unit_len;   // time pieces per row and their tokens (a multiple of 32)
    size_t ldx, lddt, ldz, ldb, ldc;
    const void *x, *dt, *z, *b, *c;
    const float *A_log, *d_skip, *dt_bias, *h0;
    void* y;
    float* ht;
    int32_t* err;
    float* ckpt;               // [rows][ceil(len / SSM_CKPT)][D][S]: state entering every 16th token
    float *hloc, *sdt;         // pieces: [rows * units_row][D][S] local end states, [..][D] sums of delta
    // backward
    const void* dy;
    const float* dht;
    void *dx, *ddt, *dz, *db, *dc;
    float *dA_log, *dd_skip, *ddt_bias, *dh0;
    float *rloc;               // pieces: [rows * units_row][D][S] local adjoints leaving the piece's start
    float *pA, *pv;            // [units][D][S]; [units][2][D] (skip, dt_bias)
    float* pbc;                // [channel tiles][rows * len][2][S]
};
int ssm_bwd_tiles(int D, int G, int S);   // the backward's channel tiles of all groups
int ssm_units(int rows, int len, int D, int G, int S, bool backward);
cudaError_t launch_ssm_fwd(const SsmArgs& a, int bf16, int mode, cudaStream_t st);   // 0 outputs, 1 + checkpoints, 2 checkpoints only
cudaError_t launch_ssm_pieces(const SsmArgs& a, int bf16, cudaStream_t st);          // local end states of every piece
cudaError_t launch_ssm_bwd_pieces(const SsmArgs& a, int bf16, cudaStream_t st);
cudaError_t launch_ssm_bwd(const SsmArgs& a, int bf16, cudaStream_t st);
cudaError_t launch_ssm_bwd_sums(const SsmArgs& a, int bf16, cudaStream_t st);

}  // namespace kda
