// Rounding to e4m3 with a scale for each group of 128 (include/kda.h): per group m = max |x|, scale = m / 448,
// q = e4m3(x 448 / m), to nearest even.
// A CTA takes a tile of 128 x 128 values and reads it once into registers: a thread has 8 neighbouring columns of 8
// neighbouring rows, so that a row's maximum is an exchange of 16 lanes, a column's one of a thread's own rows, a
// lane and eight warps, a row of q leaves in 8-byte pieces, and a column's 8 values are one 8-byte piece of qt. Those
// pieces turn in shared memory, piece p of column c at place p ^ (c / 8), which spreads both sides over all banks.
// 16384 x 4096 bf16 with both copies 61 us, 4.4 TB/s (66% of the copy rate); 4096 x 4096 fp32 in blocks 22.6 us. Bound by
// instructions (2.5 of 4 a cycle) rather than by HBM: two roundings of each value and the exchanges around them. Its
// factors are formed once per group, by one lane or thread, and handed round (each thread forming its own: 88 us); bf16
// maxima go two at a time (99 us before).
#include "kda_fp8.cuh"

namespace kda {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int NT = 256, TILE = FP8_GROUP, PER = 8;

// The larger of a and |b|; a NaN stays.
__device__ __forceinline__ float amax(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}
// What a group's values are multiplied by. 448 / m may overflow, or m be above the range in which its quotient is normal;
// such a group (`by` is not 1) is brought to the middle of the range first.
struct Factor {
    float by, inv;
};
__device__ __forceinline__ Factor factor(float m) {
    const float by = m >= 1e-30f && m <= 1e30f ? 1.f : m < 1.f ? 0x1p64f : 0x1p-64f;
    const float v = m * by;
    return {by, v > 0.f ? FP8_MAX / v : v};   // 0 and NaN as they are
}
// Four values of a group, rounded.
__device__ __forceinline__ uint32_t round4(float2 a, float2 b, const Factor& f) {
    if (f.by != 1.f) {
        a = mul2(a, make_float2(f.by, f.by));
        b = mul2(b, make_float2(f.by, f.by));
    }
    a = mul2(a, make_float2(f.inv, f.inv));
    b = mul2(b, make_float2(f.inv, f.inv));
    return (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) | (uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16;
}
// |x| of two bf16 values, and the larger ones of two pairs; a NaN stays.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b & 0x7fff7fffu));
    return r;
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Maxima of |x| over the rows (all 8 values of each) and over the columns of a thread's 8 x 8 values.
template <bool R, bool C>
__device__ __forceinline__ void maxima(const Raw<__nv_bfloat16, 8> (&raw)[8], float (&rm)[8], float (&cm)[8]) {
    uint32_t c[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw[i]);
        if (R) {
            const uint32_t m = max_bf16x2(max_bf16x2(max_bf16x2(max_bf16x2(0u, w[0]), w[1]), w[2]), w[3]);
            rm[i] = amax(low(m), high(m));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (C) c[j] = max_bf16x2(c[j], w[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (C) {
            cm[2 * j] = low(c[j]);
            cm[2 * j + 1] = high(c[j]);
        }
}
template <bool R, bool C>
__device__ __forceinline__ void maxima(const Raw<float, 8> (&raw)[8], float (&rm)[8], float (&cm)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) cm[j] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        rm[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (R) rm[i] = amax(rm[i], raw[i].v[j]);
            if (C) cm[j] = amax(cm[j], raw[i].v[j]);
        }
    }
}
// ROWS: q is wanted, COLS: qt.
template <typename TI, bool BLOCKS, bool ROWS, bool COLS>
__global__ void __launch_bounds__(NT, sizeof(TI) == 2 ? 3 : 2) k_quant8(Quant8Args a, int vecx, int vecq, int vect) {
    __shared__ __align__(16) uint2 turn[COLS ? TILE : 1][COLS ? TILE / PER : 1];
    __shared__ __align__(16) float cmax[COLS && !BLOCKS ? NT / 32 : 1][COLS && !BLOCKS ? TILE : 1];   // then row 0: the columns' 448 / m
    __shared__ float bmax[NT / 32];
    const int lx = threadIdx.x & 15, ty = threadIdx.x >> 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r0 = blockIdx.y * TILE + ty * PER, c0 = blockIdx.x * TILE + lx * PER;   // this thread's values
    const int gd = (a.D + TILE - 1) / TILE, gr = (a.rows + TILE - 1) / TILE;
    const int cols = min(max(a.D - c0, 0), PER);
    Raw<TI, PER> raw[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const TI* p = static_cast<const TI*>(a.x) + (int64_t)(r0 + i) * a.ldx + c0;
        if (r0 + i < a.rows && cols == PER && vecx) {
#pragma unroll
            for (int j = 0; j < (int)sizeof(raw[0]) / 16; ++j)
                reinterpret_cast<uint4*>(&raw[i])[j] = reinterpret_cast<const uint4*>(p)[j];
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j) raw[i].v[j] = r0 + i < a.rows && j < cols ? p[j] : TI(0.f);
        }
    }
    float rm[PER], cm[PER];   // maxima of the rows and of the columns
    Factor rf[PER], cf[PER];  // and their groups' factors
    bool odd_rows = false;
    maxima<BLOCKS || ROWS, COLS && !BLOCKS>(raw, rm, cm);
    if (BLOCKS) {
        float m = rm[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) m = amax(m, rm[i]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = amax(m, __shfl_xor_sync(FULL, m, o));
        if (lane == 0) bmax[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) m = amax(m, bmax[w]);
        const Factor f = factor(m);
#pragma unroll
        for (int i = 0; i < PER; ++i) rf[i] = cf[i] = f;
        if (threadIdx.x == 0) {
            if (ROWS) a.scale[(size_t)blockIdx.y * gd + blockIdx.x] = m / FP8_MAX;
            if (COLS) a.scale_t[(size_t)blockIdx.x * gr + blockIdx.y] = m / FP8_MAX;
        }
    } else {
        if (ROWS) {
            // 8 maxima over 16 lanes: at each exchange a lane goes on with half of the rows, until it has one
            float m4[4], m2[2];
            const bool b3 = lx & 8, b2 = lx & 4, b1 = lx & 2;
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = amax(b3 ? rm[4 + i] : rm[i], __shfl_xor_sync(FULL, b3 ? rm[i] : rm[4 + i], 8));
#pragma unroll
            for (int i = 0; i < 2; ++i) m2[i] = amax(b2 ? m4[2 + i] : m4[i], __shfl_xor_sync(FULL, b2 ? m4[i] : m4[2 + i], 4));
            float m = amax(b1 ? m2[1] : m2[0], __shfl_xor_sync(FULL, b1 ? m2[0] : m2[1], 2));
            m = amax(m, __shfl_xor_sync(FULL, m, 1));
            const int i = lx >> 1;   // this lane's row
            if (!(lx & 1) && r0 + i < a.rows) a.scale[(size_t)(r0 + i) * gd + blockIdx.x] = m / FP8_MAX;
            const Factor f = factor(m);
            odd_rows = __any_sync(FULL, f.by != 1.f);
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                rf[k].inv = __shfl_sync(FULL, f.inv, (lane & 16) | 2 * k);
                rf[k].by = odd_rows ? __shfl_sync(FULL, f.by, (lane & 16) | 2 * k) : 1.f;
            }
        }
        if (COLS) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                cm[j] = amax(cm[j], __shfl_xor_sync(FULL, cm[j], 16));
                if (lane < 16) cmax[warp][lx * PER + j] = cm[j];
            }
            __syncthreads();
            int odd = 0;
            if (threadIdx.x < TILE) {
                float m = cmax[0][threadIdx.x];
#pragma unroll
                for (int w = 1; w < NT / 32; ++w) m = amax(m, cmax[w][threadIdx.x]);
                const int c = blockIdx.x * TILE + threadIdx.x;
                if (c < a.D) a.scale_t[(size_t)c * gr + blockIdx.y] = m / FP8_MAX;
                const Factor f = factor(m);
                cmax[0][threadIdx.x] = f.inv;
                cmax[1][threadIdx.x] = f.by;
                odd = f.by != 1.f;
            }
            odd = __syncthreads_or(odd);
#pragma unroll
            for (int j = 0; j < PER; ++j) cf[j] = {odd ? cmax[1][lx * PER + j] : 1.f, cmax[0][lx * PER + j]};
        }
    }
    if (ROWS) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const Factor f = rf[i];
            float v[PER];
            unpack<PER>(raw[i], v);
            uint32_t w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) w[j] = round4(make_float2(v[4 * j], v[4 * j + 1]), make_float2(v[4 * j + 2], v[4 * j + 3]), f);
            if (r0 + i >= a.rows) continue;
            uint8_t* q = a.q + (int64_t)(r0 + i) * a.ldq + c0;
            if (cols == PER && vecq) {
                *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
            } else {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (j < cols) q[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
            }
        }
    }
    if (COLS) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const Factor f = cf[j];
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    float v[PER];
                    unpack<PER>(raw[4 * i + z], v);
                    x[z] = v[j];
                }
                w[i] = round4(make_float2(x[0], x[1]), make_float2(x[2], x[3]), f);
            }
            turn[lx * PER + j][ty ^ lx] = make_uint2(w[0], w[1]);
        }
        __syncthreads();
        const int p = threadIdx.x & 15;   // piece: rows 8 p .. 8 p + 7 of the tile
        const int rt = blockIdx.y * TILE + p * PER, n = min(max(a.rows - rt, 0), PER);
#pragma unroll
        for (int k = 0; k < TILE / 16; ++k) {
            const int c = k * 16 + (threadIdx.x >> 4), col = blockIdx.x * TILE + c;
            if (col >= a.D) break;
            const uint2 w = turn[c][p ^ (c >> 3)];
            uint8_t* q = a.qt + (int64_t)col * a.ldqt + rt;
            if (n == PER && vect) {
                *reinterpret_cast<uint2*>(q) = w;
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (i < n) q[i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
            }
        }
    }
}

template <typename TI, bool BLOCKS>
void run(const Quant8Args& a, cudaStream_t st) {
    const auto on = [](const void* p, int64_t ld, int n) { return (reinterpret_cast<uintptr_t>(p) % n == 0 && ld % n == 0) ? 1 : 0; };
    const int vecx = on(a.x, a.ldx * (int64_t)sizeof(TI), 16), vecq = on(a.q, a.ldq, 8), vect = on(a.qt, a.ldqt, 8);
    const dim3 grid((a.D + TILE - 1) / TILE, (unsigned)(((int64_t)a.rows + TILE - 1) / TILE));
    if (a.q && a.qt) k_quant8<TI, BLOCKS, true, true><<<grid, NT, 0, st>>>(a, vecx, vecq, vect);
    else if (a.q) k_quant8<TI, BLOCKS, true, false><<<grid, NT, 0, st>>>(a, vecx, vecq, vect);
    else k_quant8<TI, BLOCKS, false, true><<<grid, NT, 0, st>>>(a, vecx, vecq, vect);
}

}  // namespace

cudaError_t launch_quant8(const Quant8Args& a, int bf16, cudaStream_t st) {
    return traced_launch("k_quant8", st, [&] {
        if (bf16) a.blocks ? run<__nv_bfloat16, true>(a, st) : run<__nv_bfloat16, false>(a, st);
        else a.blocks ? run<float, true>(a, st) : run<float, false>(a, st);
    });
}

}  // namespace kda
