// Linear attention with a decay for each head: what its kernels share. One recurrence serves the forward and the
// three gradients (include/kda.h has the operator):
//     forwards in time    S <- a S + w k v^T,  o = s q S       (o: (q, k, v);  dq: (do, v, k), the state transposed)
//     backwards in time   R <- R + w k v^T,  o = s q R,  R <- a R    (dv: (k, q, do);  dk: (v, do, q), transposed)
// with a = exp(decay of the head). A LinCall is one of them; its q, k, v are the roles, not the caller's tensors.
// "Mirrored" tokens: a call that runs backwards counts its tokens, and its windows, from the row's end.
#pragma once

#include "kda_layer.cuh"

namespace kda {

struct LinCall {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;     // elements between tokens
    int gq, gk, gv;            // value heads to a head of each
    int K, V;                  // widths of q, k and of v, o
    void* o;                   // [tokens][HV][V]
    int o_f32;                 // fp32 instead of the I/O type (partial sums of shared heads)
    const float* s0;           // [N][HV] states or NULL
    float* s1;                 // final states or NULL (natural order only)
    int transposed;            // s0 is [V][K]
    int back;
    float s, w;                // the formulas' s and w
    float* local;              // [windows][HV][K][V]: end states of the windows' own tokens, then the states they hand on
};

struct LinArgs {
    TokenAxis ax;
    int HV;
    const float* decay;        // [HV] or NULL
    int units_row, unit_len;   // windows per row and their tokens
    int32_t* err;
    int calls;
    LinCall c[3];
};

// The sequence that holds mirrored token t of the row, in mirrored tokens.
__device__ __forceinline__ Seq lin_seq(const TokenAxis& ax, int row, int t, int back) {
    if (!back) return seq_at(ax, row, t);
    const Seq s = seq_at(ax, row, ax.len - 1 - t);
    return {s.n, ax.len - s.end, ax.len - s.first};
}

// a^m = exp(g m): the product's rounding goes on as its low part, so that the power is within expf's two units.
__device__ __forceinline__ float lin_power(float g, int m) {
    if (m == 0) return 1.f;
    const float x = g * (float)m, low = fmaf(g, (float)m, -x);
    const float e = expf(x);
    return e > 0.f && e < 3e38f ? fmaf(e, low, e) : e;
}
// The same as a sum of two fp32 values, to 2^-48: a state meets this factor once per step, and its error would grow
// with the tokens that the state remembers.
__device__ __forceinline__ float2 lin_power2(float g, int m) {
    if (m == 0) return make_float2(1.f, 0.f);
    const double e = exp((double)g * m);
    const float hi = (float)e;
    return make_float2(hi, isfinite(hi) ? (float)(e - hi) : 0.f);
}
// The same from `one`, a^1 in two parts, for m >= 1 and without 64 bits, which a whole warp has no room for: squares and
// products of two-part values, each off by some 2^-46, so that a^m is off by m 2^-47 (2^-40 for a chunk of 128 tokens).
__device__ __forceinline__ float2 lin_mul2(float2 a, float2 b) {
    const float hi = __fmul_rn(a.x, b.x);
    if (!isfinite(hi)) return make_float2(hi, 0.f);
    const float lo = __fadd_rn(fmaf(a.x, b.x, -hi), fmaf(a.x, b.y, a.y * b.x)), sum = __fadd_rn(hi, lo);
    return make_float2(sum, __fadd_rn(lo, -__fadd_rn(sum, -hi)));
}
__device__ __forceinline__ float2 lin_raise(float2 one, int m) {
    float2 r = one;
#pragma unroll 1
    for (int b = 30 - __clz(m); b >= 0; --b) {
        r = lin_mul2(r, r);
        if (m >> b & 1) r = lin_mul2(r, one);
    }
    return r;
}

constexpr int LIN_MAX_W = 256;    // widest key or value
constexpr int LIN_MAX_WINDOWS = 256;   // time windows of a row

// The kernel on CUDA cores: value columns of a CTA for calls of these widths; the tokens of its time windows where a window
// is `ctas` CTAs.
int lin_slice(int kmax, const int* widths, int calls);
int lin_window(int rows, int len, int ctas, int kmax, int slice);
cudaError_t launch_lin(const LinArgs& a, int bf16, cudaStream_t st);
// The tensor cores' kernel: from this many tokens per sequence on (in the mean); the tokens of its time windows where a window is
// `ctas` CTAs; whether a bf16 call's widths and rows fit it.
// (64 sequences of 32 heads of 128, us, tensor cores against the kernel on CUDA cores: forward 8 tokens 371 against 230, 16
// 381 against 377, 32 368 against 670; backward 8 tokens 816 against 762, 16 830 against 1148.)
constexpr int LIN_TC_TOKENS = 16, LIN_TC_TOKENS_BACK = 10;
// Packed sequences lie one behind the other in a window, and each of them costs its CTA 7 to 12 us there however short it is,
// while the CUDA cores' windows spread a call of few heads over the SMs: such calls, of less than a third of the SMs' CTAs a
// window, need a higher mean. (us, tensor cores against CUDA cores, states carried; n x t: n sequences of t tokens, n + t: n
// single tokens beside one of t. Forward, 4 heads of 64: 16 x 32 115, 30, 16 x 64 110, 46, 16 x 128 20, 54, 64 + 4000 495,
// 230; 8 heads of 128: 12 x 24 128, 50, 12 x 64 121, 96, 64 x 24 670, 152, 64 x 48 100, 272, 64 + 1200 724, 440; 16 heads of
// 128: 64 x 32 692, 383, 64 x 64 189, 703, 64 + 4000 777, 1281; 32 heads of 128: 12 x 16 130, 74, 64 x 32 698, 771, 64 + 1200
// 756, 1022; 64 heads of 128: 12 x 16 132, 178, 64 + 1200 759, 1335. Backward, 4 heads of 64: 16 x 32 114, 46, 64 x 64 59,
// 142, 64 + 1000 491, 238; 8 heads of 128: 64 x 16 684, 301, 64 x 48 257, 710, 64 + 1200 734, 1084; 16 heads of 128: 64 x 16
// 694, 635, 64 + 1000 736, 1457.)
constexpr int LIN_TC_PACKED = 48, LIN_TC_PACKED_BACK = 24;
int lin_tc_window(int rows, int len, int ctas);
bool lin_tc_call(const LinCall& c);
cudaError_t launch_lin_tc(const LinArgs& a, cudaStream_t st);
// Turns the windows' own end states into the states that the next windows' first sequences enter with.
cudaError_t launch_lin_join(const LinArgs& a, cudaStream_t st);
// out[t][h][:] = sum over the group's value heads of part[t][h * group + i][:], in order.
cudaError_t launch_lin_heads(const float* part, void* out, int64_t rows, int group, int width, int bf16, cudaStream_t st);

}  // namespace kda
