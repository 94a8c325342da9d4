// Short causal convolution, one filter of W taps per channel, over the packed
// token axis, with the mixer's SiLU in its epilogue:
//     s_t = bias + sum_j w[j] x_{t-W+1+j},   y_t = s_t  or  s_t sigmoid(s_t)
// Tokens before a sequence's first come from its carried state, the last W - 1
// inputs of what came before (oldest first; zero without one). The backward
// recomputes s, forms d_t = dy_t act'(s_t), and gathers
//     dx_t = sum_j w[j] d_{t+W-1-j},  dw[j] = sum_t d_t x_{t-W+1+j},  dbias = sum_t d_t
// A thread owns 16 bytes of neighbouring channels and walks a tile of tokens with
// the window in registers, so each input is read once plus W - 1 rows per tile.
#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr int CT = 128;   // threads of the forward
constexpr int CB = 256;   // threads of the backward
constexpr int CU = 4;     // tokens whose loads are in flight together

template <int W, int V>
__device__ __forceinline__ void load_weights(const ConvArgs& a, int c0, float (&w)[V][W], float (&bias)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[v][j] = a.weight[(size_t)(c0 + v) * W + j];
        bias[v] = a.bias ? a.bias[c0 + v] : 0.f;
    }
}

// The W - 1 inputs before token t (oldest first).
template <typename TI, int W, int V>
__device__ __forceinline__ void load_window(const ConvArgs& a, const Seq& s, const TI* x, int t, int c0,
                                            float (&win)[W - 1][V]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int p = t - (W - 1) + j;
        if (p >= s.first) {
            load_row<V>(x + (size_t)p * a.ldx, win[j], V, V > 1);
        } else if (a.h0) {
            load_row<V>(static_cast<const TI*>(a.h0) + ((size_t)s.n * (W - 1) + (p - s.first) + (W - 1)) * a.D + c0,
                        win[j], V, V > 1);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) win[j][v] = 0.f;
        }
    }
}

// Sequences without tokens: dst rows = src rows (zero without src).
template <typename TI, int W, int V>
__device__ __forceinline__ void copy_empty(const ConvArgs& a, int tile_id, int row, int c0, const void* src, void* dst) {
    if (!dst || (a.ax.cu == nullptr && a.ax.len > 0)) return;
    for (int n = a.ax.cu ? tile_id : row; n < a.ax.N; n += a.ntiles) {
        if (a.ax.cu && axis_cu(a.ax, n + 1) > axis_cu(a.ax, n)) continue;
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            const size_t o = ((size_t)n * (W - 1) + r) * a.D + c0;
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = 0.f;
            if (src) load_row<V>(static_cast<const TI*>(src) + o, v, V, V > 1);
            store_row<V>(static_cast<TI*>(dst) + o, v, V, V > 1);
        }
    }
}

template <typename TI, int W, int V, bool SILU>
__global__ void __launch_bounds__(CT) k_conv_fwd(ConvArgs a) {
    if (blockIdx.x == 0) axis_check(a.ax, a.err);
    const size_t item = (size_t)blockIdx.x * CT + threadIdx.x;
    const int tile_id = (int)(item / a.groups);
    if (tile_id >= a.ntiles) return;
    const int c0 = (int)(item - (size_t)tile_id * a.groups) * V;
    const int row = tile_id / a.tiles_row;
    int t = (tile_id - row * a.tiles_row) * a.tile;
    const int t1 = min(t + a.tile, a.ax.len);
    const size_t tok0 = (size_t)row * a.ax.len;
    const TI* x = static_cast<const TI*>(a.x) + tok0 * a.ldx + c0;
    TI* y = static_cast<TI*>(a.y) + tok0 * a.D + c0;
    float w[V][W], bias[V], win[W - 1][V];
    load_weights<W, V>(a, c0, w, bias);
    copy_empty<TI, W, V>(a, tile_id, row, c0, a.h0, a.final_state);
    while (t < t1) {
        const Seq s = seq_at(a.ax, row, t);
        load_window<TI, W, V>(a, s, x, t, c0, win);
        if (t == s.first && a.final_state) {
            // the final state, by the thread that has the initial one in its window: the two may be one buffer
            const int len = s.end - s.first;
#pragma unroll
            for (int r = 0; r < W - 1; ++r) {
                const int p = len - (W - 1) + r;
                float f[V];
                if (p >= 0) {
                    load_row<V>(x + (size_t)(s.first + p) * a.ldx, f, V, V > 1);
                } else {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
                        if (k == len + r) {
#pragma unroll
                            for (int v = 0; v < V; ++v) f[v] = win[k][v];
                        }
                }
                store_row<V>(static_cast<TI*>(a.final_state) + ((size_t)s.n * (W - 1) + r) * a.D + c0, f, V, V > 1);
            }
        }
        const int run = min(t1, s.end);
        for (; t < run; t += CU) {
            float xt[CU][V];
#pragma unroll
            for (int u = 0; u < CU; ++u)
                if (t + u < run) load_row<V>(x + (size_t)(t + u) * a.ldx, xt[u], V, V > 1);
#pragma unroll
            for (int u = 0; u < CU; ++u) {
                if (t + u >= run) break;
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float acc = bias[v];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) acc = fmaf(w[v][j], win[j][v], acc);
                    acc = fmaf(w[v][W - 1], xt[u][v], acc);
                    o[v] = SILU ? acc * sigmoid_fast(acc) : acc;
#pragma unroll
                    for (int j = 0; j < W - 2; ++j) win[j][v] = win[j + 1][v];
                    win[W - 2][v] = xt[u][v];
                }
                store_row<V>(y + (size_t)(t + u) * a.D, o, V, V > 1);
            }
        }
        t = run;
    }
}

// The final states alone, one thread per sequence and channel group: for a state updated in place when other
// threads of the forward read the initial one (launched after it).
template <typename TI, int W, int V>
__global__ void __launch_bounds__(CT) k_conv_state(ConvArgs a) {
    const size_t item = (size_t)blockIdx.x * CT + threadIdx.x;
    const int n = (int)(item / a.groups);
    if (n >= a.ax.N) return;
    const int c0 = (int)(item - (size_t)n * a.groups) * V;
    int first = 0, end = a.ax.len;
    if (a.ax.cu) {
        first = axis_cu(a.ax, n);
        end = max(axis_cu(a.ax, n + 1), first);
    }
    const TI* x = static_cast<const TI*>(a.x) + (a.ax.cu ? 0 : (size_t)n * a.ax.len) * a.ldx + c0;
    const size_t o = (size_t)n * (W - 1) * a.D + c0;
    float f[W - 1][V];
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        const int p = end - (W - 1) + r;
#pragma unroll
        for (int v = 0; v < V; ++v) f[r][v] = 0.f;
        if (p >= first) load_row<V>(x + (size_t)p * a.ldx, f[r], V, V > 1);
        else if (a.h0) load_row<V>(static_cast<const TI*>(a.h0) + o + (size_t)(end - first + r) * a.D, f[r], V, V > 1);
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r) store_row<V>(static_cast<TI*>(a.final_state) + o + (size_t)r * a.D, f[r], V, V > 1);
}

// Block of gx channel groups by gy tiles; the tiles' parameter sums are added in tile order.
template <typename TI, int W, int V, bool SILU>
__global__ void __launch_bounds__(CB) k_conv_bwd(ConvArgs a, int gx) {
    extern __shared__ float red[];   // [gy][gx * V]
    const int gy = CB / gx;
    const int lx = threadIdx.x % gx, ly = threadIdx.x / gx;
    const int nbx = (a.groups + gx - 1) / gx;
    const int part = blockIdx.x / nbx, bx = blockIdx.x - part * nbx;
    const int cg = bx * gx + lx, c0 = cg * V;
    const int tile_id = part * gy + ly;
    const bool on = cg < a.groups && tile_id < a.ntiles;
    float dw[V][W], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[v][j] = 0.f;
    }
    if (on) {
        const int row = tile_id / a.tiles_row;
        int t = (tile_id - row * a.tiles_row) * a.tile;
        const int t1 = min(t + a.tile, a.ax.len);
        const size_t tok0 = (size_t)row * a.ax.len;
        const TI* x = static_cast<const TI*>(a.x) + tok0 * a.ldx + c0;
        const TI* dy = static_cast<const TI*>(a.dy) + tok0 * a.D + c0;
        TI* dx = static_cast<TI*>(a.dx) + tok0 * a.D + c0;
        const TI* df = static_cast<const TI*>(a.dfinal);
        float w[V][W], bias[V];
        load_weights<W, V>(a, c0, w, bias);
        copy_empty<TI, W, V>(a, tile_id, row, c0, a.dfinal, a.dinit);
        while (t < t1) {
            const Seq s = seq_at(a.ax, row, t);
            const int run = min(t1, s.end), len = s.end - s.first;
            const bool start = t == s.first;
            float win[W - 1][V], dwin[W - 1][V];   // x before the token (oldest first); d before it (newest first)
            load_window<TI, W, V>(a, s, x, t, c0, win);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) dwin[j][v] = 0.f;
            // W - 1 tokens past the run: their d reaches back into it (zero past the sequence)
            for (int tb = t; tb < run + W - 1; tb += CU) {
                float xt[CU][V], dt[CU][V];
#pragma unroll
                for (int u = 0; u < CU; ++u) {
                    const int tt = tb + u;
                    if (tt < min(run + W - 1, s.end)) {
                        load_row<V>(x + (size_t)tt * a.ldx, xt[u], V, V > 1);
                        load_row<V>(dy + (size_t)tt * a.D, dt[u], V, V > 1);
                    }
                }
#pragma unroll
                for (int u = 0; u < CU; ++u) {
                    const int tt = tb + u;
                    if (tt >= run + W - 1) break;
                    float e[V];
                    const bool own = tt < run, real = tt < s.end;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float d = 0.f;
                        if (real) {
                            d = dt[u][v];
                            if (SILU) {
                                float pre = bias[v];
#pragma unroll
                                for (int j = 0; j < W - 1; ++j) pre = fmaf(w[v][j], win[j][v], pre);
                                pre = fmaf(w[v][W - 1], xt[u][v], pre);
                                const float sg = sigmoid_fast(pre);
                                d *= sg * fmaf(pre, 1.f - sg, 1.f);
                            }
                            if (own) {
                                db[v] += d;
#pragma unroll
                                for (int j = 0; j < W - 1; ++j) dw[v][j] = fmaf(d, win[j][v], dw[v][j]);
                                dw[v][W - 1] = fmaf(d, xt[u][v], dw[v][W - 1]);
                            }
#pragma unroll
                            for (int j = 0; j < W - 2; ++j) win[j][v] = win[j + 1][v];
                            win[W - 2][v] = xt[u][v];
                        }
                        float acc = w[v][0] * d;
#pragma unroll
                        for (int j = 1; j < W; ++j) acc = fmaf(w[v][j], dwin[j - 1][v], acc);
                        e[v] = acc;
#pragma unroll
                        for (int j = W - 2; j > 0; --j) dwin[j][v] = dwin[j - 1][v];
                        dwin[0][v] = d;
                    }
                    const int q = tt - (W - 1);   // the token whose gradient is complete
                    int r = -1;                   // the final state's row that reads it
                    TI* dst = nullptr;
                    if (q >= t) {
                        dst = dx + (size_t)q * a.D;
                        if (q >= s.end - (W - 1)) r = q - (s.end - (W - 1));
                    } else if (start && a.dinit) {
                        const int i = tt - t;     // the initial state's row
                        dst = static_cast<TI*>(a.dinit) + ((size_t)s.n * (W - 1) + i) * a.D + c0;
                        if (i >= len) r = i - len;
                    }
                    if (dst) {
                        if (df && r >= 0) {
                            float f[V];
                            load_row<V>(df + ((size_t)s.n * (W - 1) + r) * a.D + c0, f, V, V > 1);
#pragma unroll
                            for (int v = 0; v < V; ++v) e[v] += f[v];
                        }
                        store_row<V>(dst, e, V, V > 1);
                    }
                }
            }
            t = run;
        }
    }
    // the block's sums, tap by tap
    const int ncol = gx * V;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) red[ly * ncol + lx * V + v] = j < W ? dw[v][j < W ? j : 0] : db[v];
        __syncthreads();
        for (int c = threadIdx.x; c < ncol; c += CB) {
            if (bx * ncol + c >= a.D) continue;
            float sum = 0.f;
            for (int k = 0; k < gy; ++k) sum += red[k * ncol + c];
            a.part[((size_t)part * (W + 1) + j) * a.D + bx * ncol + c] = sum;
        }
    }
}

// dweight and dbias: the blocks' sums in block order.
__global__ void k_conv_sum(ConvArgs a) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    const int j = i / a.D, d = i - j * a.D;
    if (j > a.W) return;
    float sum = 0.f;
    for (int p = 0; p < a.parts; ++p) sum += a.part[((size_t)p * (a.W + 1) + j) * a.D + d];
    if (j < a.W) a.dweight[(size_t)d * a.W + j] = sum;
    else if (a.dbias) a.dbias[d] = sum;
}

int bwd_gx(int groups) {
    int gx = 1;
    while (gx < 32 && gx < groups) gx *= 2;
    return gx;
}

template <typename TI, int W, int V>
void run_fwd(const ConvArgs& a, cudaStream_t st) {
    const size_t items = (size_t)a.ntiles * a.groups;
    const unsigned grid = (unsigned)((items + CT - 1) / CT);
    if (a.silu) k_conv_fwd<TI, W, V, true><<<grid, CT, 0, st>>>(a);
    else k_conv_fwd<TI, W, V, false><<<grid, CT, 0, st>>>(a);
}
template <typename TI, int W, int V>
void run_state(const ConvArgs& a, cudaStream_t st) {
    const size_t items = (size_t)a.ax.N * a.groups;
    k_conv_state<TI, W, V><<<(unsigned)((items + CT - 1) / CT), CT, 0, st>>>(a);
}
template <typename TI, int W, int V>
void run_bwd(const ConvArgs& a, cudaStream_t st) {
    const int gx = bwd_gx(a.groups);
    const unsigned grid = (unsigned)a.parts * ((a.groups + gx - 1) / gx);
    const size_t smem = sizeof(float) * CB * V;
    if (a.silu) k_conv_bwd<TI, W, V, true><<<grid, CB, smem, st>>>(a, gx);
    else k_conv_bwd<TI, W, V, false><<<grid, CB, smem, st>>>(a, gx);
}
enum { FWD, STATE, BWD };
template <int OP, typename TI, int W, int V>
void run_op(const ConvArgs& a, cudaStream_t st) {
    if (OP == FWD) run_fwd<TI, W, V>(a, st);
    else if (OP == STATE) run_state<TI, W, V>(a, st);
    else run_bwd<TI, W, V>(a, st);
}
template <int OP, typename TI, int V>
void run_w(const ConvArgs& a, cudaStream_t st) {
    switch (a.W) {
        case 2: run_op<OP, TI, 2, V>(a, st); break;
        case 3: run_op<OP, TI, 3, V>(a, st); break;
        default: run_op<OP, TI, 4, V>(a, st); break;
    }
}
template <int OP>
void run_conv(const ConvArgs& a, int bf16, bool vec, cudaStream_t st) {
    if (bf16) vec ? run_w<OP, __nv_bfloat16, 8>(a, st) : run_w<OP, __nv_bfloat16, 1>(a, st);
    else vec ? run_w<OP, float, 4>(a, st) : run_w<OP, float, 1>(a, st);
}

}  // namespace

void conv_shape(ConvArgs& a, int bf16, bool vec, bool backward) {
    const int V = vec ? (bf16 ? 8 : 4) : 1;
    a.groups = a.D / V;
    // tokens per thread: long tiles re-read fewer window rows, short ones fill the GPU
    const long long want = 152LL * 1024;
    int tile = backward ? 64 : 32;
    while (tile > 1 && (long long)a.groups * a.ax.rows * ((a.ax.len + tile - 1) / tile) < want) tile /= 2;
    if (backward && tile < 8) tile = 8;
    a.tile = tile;
    a.tiles_row = a.ax.len > 0 ? (a.ax.len + tile - 1) / tile : 1;
    a.ntiles = a.ax.rows * a.tiles_row;
    const int gy = CB / bwd_gx(a.groups);
    a.parts = (a.ntiles + gy - 1) / gy;
}

cudaError_t launch_conv_fwd(ConvArgs a, int bf16, bool vec, cudaStream_t st) {
    // a state updated in place: the thread that starts a sequence writes its final state, which is safe unless a
    // second tile reads initial rows too (tiles shorter than the window, or packed offsets anywhere in a tile)
    void* in_place = nullptr;
    if (a.final_state && a.final_state == a.h0 && (a.ax.cu || (a.tiles_row > 1 && a.tile < a.W - 1))) {
        in_place = a.final_state;
        a.final_state = nullptr;
    }
    cudaError_t e = traced_launch("k_conv_fwd", st, [&] { run_conv<FWD>(a, bf16, vec, st); });
    if (e != cudaSuccess || !in_place) return e;
    a.final_state = in_place;
    return traced_launch("k_conv_state", st, [&] { run_conv<STATE>(a, bf16, vec, st); });
}

cudaError_t launch_conv_bwd(ConvArgs a, int bf16, bool vec, cudaStream_t st) {
    cudaError_t e = traced_launch("k_conv_bwd", st, [&] { run_conv<BWD>(a, bf16, vec, st); });
    if (e != cudaSuccess) return e;
    const int n = (a.W + 1) * a.D;
    return traced_launch("k_conv_sum", st, [&] { k_conv_sum<<<(n + 127) / 128, 128, 0, st>>>(a); });
}

}  // namespace kda
