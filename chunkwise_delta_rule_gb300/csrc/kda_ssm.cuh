// Device helpers shared by the scan's forward and backward.
#pragma once

#include "kda_layer.cuh"

namespace kda {

// A compile-time number as a lambda's argument.
template <int N>
struct Int {
    static constexpr int value = N;
};

constexpr unsigned SSM_FULL = 0xffffffffu;
constexpr int SSM_T = 128;    // threads of the recurrence per CTA: 32 channels x 4 lanes
constexpr int SSM_CH = 32;    // channels per CTA

// log(1 + e^v) without overflow: max(v, 0) + log(1 + e) with e = e^-|v| in (0, 1]. With s = e / (2 + e) <= 1/3 the
// logarithm is 2 atanh(s), whose quotient by s is a smooth function of q = s^2 in [0, 1/9]: the polynomial interpolates
// it at the five Chebyshev points of that interval (8e-9 relative with fp32 coefficients), so that a step of 1e-3
// is as exact relative to itself as one of 1.
__device__ __forceinline__ float2 ssm_softplus2(float2 v) {
    const float2 e = make_float2(ex2(-LOG2E * fabsf(v.x)), ex2(-LOG2E * fabsf(v.y)));
    const float2 s = mul2(e, make_float2(rcp(2.f + e.x), rcp(2.f + e.y))), q = mul2(s, s);
    float2 p = make_float2(0.281577796f, 0.281577796f);
    p = fma2(p, q, make_float2(0.279651582f, 0.279651582f));
    p = fma2(p, q, make_float2(0.400245965f, 0.400245965f));
    p = fma2(p, q, make_float2(0.666663229f, 0.666663229f));
    p = fma2(p, q, make_float2(2.f, 2.f));
    return fma2(p, s, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float ssm_softplus(float v) { return ssm_softplus2(make_float2(v, v)).x; }

// Decays 2^(delta A) of exponents in log2 units. The hardware's 2^x lies below the value on the average: 1.7e-8 to 3.2e-8
// of it for exponents of -2^-8 .. -1, 5e-9 to 9e-9 for smaller ones (measured against 64 bits), and a state multiplies
// the decays of all the tokens that it remembers. A constant in the exponent, added by the product's own instruction,
// leaves at most 1.2e-8 and is itself lost in 1: a token of step 0 leaves the state as it is (training four rows of 2048 tokens, 2048 channels: dA_log 1.5e-6 from 64 bits without it, 1.0e-6 with it).
constexpr float SSM_EX2_MEAN = 2.5e-8f;
__device__ __forceinline__ float2 ssm_exponent2(float2 dl, float2 A2) { return fma2(dl, A2, make_float2(SSM_EX2_MEAN, SSM_EX2_MEAN)); }
__device__ __forceinline__ float ssm_decay(float dl, float A2) { return ex2(fmaf(dl, A2, SSM_EX2_MEAN)); }

// A CTA's place: time piece `unit` of `units` (tokens [lo, hi) of row `row`), nch <= CH channels from c0 of group g.
struct SsmPlace {
    int unit, units, row, u, lo, hi, tile, g, c0, nch;
};
template <int CH>
__device__ __forceinline__ SsmPlace ssm_place(const SsmArgs& a) {
    SsmPlace p;
    const int M = a.D / a.G, tpg = (M + CH - 1) / CH, tiles = tpg * a.G;
    p.unit = blockIdx.x / tiles;
    p.units = gridDim.x / tiles;
    p.tile = blockIdx.x - p.unit * tiles;
    p.g = p.tile / tpg;
    const int tg = p.tile - p.g * tpg;
    p.c0 = p.g * M + tg * CH;
    p.nch = min(CH, M - tg * CH);
    p.row = p.unit / a.units_row;
    p.u = p.unit - p.row * a.units_row;
    p.lo = p.u * a.unit_len;
    p.hi = min(p.lo + a.unit_len, a.ax.len);
    return p;
}

// A lane's EL states of channel d (states n0 .. n0 + EL - 1 of S), zero past S or for an absent channel.
template <int EL>
__device__ __forceinline__ void load_states(const float* p, int n0, int S, bool on, float (&x)[EL]) {
    const bool vec = on && S == 4 * EL && EL >= 4 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
    if (vec) {
#pragma unroll
        for (int e = 0; e + 3 < EL; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + n0 + e);
            x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < EL; ++e) x[e] = on && n0 + e < S ? p[n0 + e] : 0.f;
    }
}
template <int EL>
__device__ __forceinline__ void store_states(float* p, int n0, int S, bool on, const float (&x)[EL]) {
    const bool vec = S == 4 * EL && EL >= 4 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
    if (!on) return;
    if (vec) {
#pragma unroll
        for (int e = 0; e + 3 < EL; e += 4)
            *reinterpret_cast<float4*>(p + n0 + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < EL; ++e)
            if (n0 + e < S) p[n0 + e] = x[e];
    }
}

// One halving step of a sum over lanes: each lane keeps half of its V values and adds the partner's copy of them.
template <int V>
__device__ __forceinline__ void halve(float* v, int lane, int mask) {
    const bool up = lane & mask;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float send = up ? v[i] : v[i + V / 2];
        const float keep = up ? v[i + V / 2] : v[i];
        v[i] = keep + __shfl_xor_sync(SSM_FULL, send, mask);
    }
}

// The EL states of a lane's row in a shared [..][4 * EL] tile.
template <int EL>
__device__ __forceinline__ void lds_states(const float* p, float (&x)[EL]) {
    if (EL % 4 == 0) {
#pragma unroll
        for (int e = 0; e + 3 < EL; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + e);
            x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
        }
    } else {
        const float2 v = *reinterpret_cast<const float2*>(p);
        x[0] = v.x; x[1] = v.y;
    }
}

// A thread's V channels of a token: from its place in shared memory, and to a row of an output.
template <int V, typename TI>
__device__ __forceinline__ void load_part(const TI* p, float (&x)[V]) {
    if constexpr (V * sizeof(TI) >= 16) load_row<V>(p, x, V, true);
    else unpack<V>(load_raw<TI, V>(p), x);
}
template <typename TI, int V>
__device__ __forceinline__ void store_part(TI* p, const float (&x)[V], int valid, bool whole) {
    if (whole) {
        store_values<V>(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < valid) st(p + i, x[i]);
    }
}

// The state (or adjoint) h behind the time pieces from, from + dir, .. before `to` of a row: each piece's local one plus
// the decay exp(A sum delta) times what enters it. Several pieces' values are on their way together: one after another,
// each costs the memory's latency (0.3 us a piece).
template <int EL>
__device__ __forceinline__ void join_pieces(const SsmArgs& a, const float* local, int row, int from, int to, int dir, int d,
                                            int n0, bool on, const float (&A2)[EL], float (&h)[EL]) {
    constexpr int J = EL <= 4 ? 8 : 32 / EL;
    const int count = (to - from) * dir;
    for (int r = 0; r < count; r += J) {
        float hl[J][EL], sum[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool in = on && r + j < count;
            const size_t u = (size_t)row * a.units_row + from + (in ? r + j : 0) * dir;
            load_states<EL>(local + (u * a.D + d) * a.S, n0, a.S, in, hl[j]);
            sum[j] = in ? a.sdt[u * a.D + d] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < EL; ++e) h[e] = fmaf(ssm_decay(sum[j], A2[e]), h[e], hl[j][e]);
    }
}

}  // namespace kda
