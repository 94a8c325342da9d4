// Short causal convolution, one filter of W taps per channel, over the packed
// token axis, with the mixer's SiLU in its epilogue:
//     s_t = bias + sum_j w[j] x_{t-W+1+j},   y_t = s_t  or  s_t sigmoid(s_t)
// Tokens before a sequence's first come from its carried state, the last W - 1
// inputs of what came before (oldest first; zero without one). The backward
// recomputes s, forms d_t = dy_t act'(s_t), and gathers
//     dx_t = sum_j w[j] d_{t+W-1-j},  dw[j] = sum_t d_t x_{t-W+1+j},  dbias = sum_t d_t
// A thread owns four neighbouring channels and walks a tile
// of tokens with the window in registers, so each input is read once plus W - 1 rows
// per tile. Each thread copies its own rows ahead into shared memory asynchronously (a
// dozen tokens; held in registers they cost the warps that hide the latency). The
// filters pass through shared memory too: read directly, each lane's values lie apart
// from its neighbour's and cost more than the tile's inputs.
// Bound by HBM where the tensors are large, bf16, 4096 channels, four taps: forward of
// 32768 packed tokens 93 us, 5.8 TB/s (85% of the copy rate); backward of two rows of
// 8192 98 us, 4.1 TB/s (61%: neither the memory nor the issue slots, 0.57 instructions
// per cycle and scheduler, are full; its rings and its sums' registers leave two CTAs on
// an SM, 22% of the warps). A token of each of 64 sequences of 12288 channels takes 3.3
// us on the device, where the launch is what it waits for.
#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr int CT = 128;   // threads of the forward
constexpr int CB = 256;   // threads of the backward
constexpr int VC = 4;     // channels per thread
constexpr int CU = 4;     // tokens of a group of copies, forward
constexpr int CD = 4;     // groups of copies in flight or in use

// ... and backward: as many as the window holds, so that a group's first tokens are the next one's window.
template <int W>
constexpr int BWD_U = W == 4 ? 3 : 2;

// The block's filters to shared memory, tap by tap: sw[j * ncol + c] = weight[first + c][j], row W the bias.
template <int W, int NT>
__device__ __forceinline__ void stage_weights(const ConvArgs& a, float* sw, int first, int ncol) {
    for (int i = threadIdx.x; i < ncol * W; i += NT) {
        const int c = i / W, j = i - c * W;
        sw[j * ncol + c] = first + c < a.D ? a.weight[(size_t)first * W + i] : 0.f;
    }
    for (int c = threadIdx.x; c < ncol; c += NT) sw[W * ncol + c] = a.bias && first + c < a.D ? a.bias[first + c] : 0.f;
    __syncthreads();
}
// A thread's filters, taps of neighbouring channels paired.
template <int W, int V>
__device__ __forceinline__ void read_weights(const float* sw, int ncol, int c, float (&w)[W][V], float (&bias)[V]) {
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        float v[V];
        unpack<V>(load_raw<float, V>(sw + j * ncol + c), v);
#pragma unroll
        for (int i = 0; i < V; ++i) (j < W ? w[j < W ? j : 0][i] : bias[i]) = v[i];
    }
}

// acc + w x over V channels, in pairs.
template <int V>
__device__ __forceinline__ void fma_v(const float (&w)[V], const float (&x)[V], float (&acc)[V]) {
    if (V == 1) {
        acc[0] = fmaf(w[0], x[0], acc[0]);
    } else {
#pragma unroll
        for (int i = 0; i + 1 < V; i += 2) {
            const float2 r = fma2(make_float2(w[i], w[i + 1]), make_float2(x[i], x[i + 1]), make_float2(acc[i], acc[i + 1]));
            acc[i] = r.x;
            acc[i + 1] = r.y;
        }
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
            unpack<V>(load_raw<TI, V>(x + (size_t)p * a.ldx), win[j]);
        } else if (a.h0) {
            unpack<V>(load_raw<TI, V>(static_cast<const TI*>(a.h0) + ((size_t)s.n * (W - 1) + (p - s.first) + (W - 1)) * a.D + c0),
                      win[j]);
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
            if (src) unpack<V>(load_raw<TI, V>(static_cast<const TI*>(src) + o), v);
            store_values<V>(static_cast<TI*>(dst) + o, v);
        }
    }
}

// A thread's rows on their way: groups of U tokens, CD of them in a ring in shared memory (for single 16-bit elements,
// which have no asynchronous copy, one group ahead in registers).
template <typename TI, int V, int U, int NT>
struct Ring {
    static constexpr bool ASYNC = sizeof(TI) * V >= 4;
    static constexpr int BYTES = ASYNC ? CD * U * NT * (int)sizeof(TI) * V : 0;
    using R = Raw<TI, V>;
    R* mine;
    const TI* src;      // token 0 of the run
    size_t ld;
    int n;              // tokens of the run
    R next[ASYNC ? 1 : U];
    __device__ __forceinline__ void start(void* smem, const TI* p, size_t stride, int tokens) {
        mine = static_cast<R*>(smem) + threadIdx.x;
        src = p;
        ld = stride;
        n = tokens;
    }
    __device__ __forceinline__ void fetch(int g) {
        const TI* p = src + (size_t)(g * U) * ld;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (g * U + u >= n) break;
            if constexpr (ASYNC) copy_async(mine + ((g % CD) * U + u) * NT, p + u * ld);
            else next[u] = load_raw<TI, V>(p + u * ld);
        }
    }
    __device__ __forceinline__ R get(int g, int u) const {
        if constexpr (ASYNC) return mine[((g % CD) * U + u) * NT];
        else return next[u];
    }
};

// Output of one token; the window moves on.
template <int W, int V, bool SILU>
__device__ __forceinline__ void conv_token(const float (&w)[W][V], const float (&bias)[V], float (&win)[W - 1][V],
                                           const float (&x)[V], float (&o)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = bias[v];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) fma_v<V>(w[j], win[j], o);
    fma_v<V>(w[W - 1], x, o);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (SILU) o[v] *= sigmoid_fast(o[v]);
#pragma unroll
        for (int j = 0; j < W - 2; ++j) win[j][v] = win[j + 1][v];
        win[W - 2][v] = x[v];
    }
}

// Block of gx channel groups by gy tiles.
template <typename TI, int W, int V, bool SILU>
__global__ void __launch_bounds__(CT) k_conv_fwd(ConvArgs a) {
    extern __shared__ __align__(16) float sw[];   // the filters, the ring
    if (blockIdx.x == 0) axis_check(a.ax, a.err);
    const int lx = threadIdx.x & (a.gx - 1), ly = threadIdx.x / a.gx, gy = CT / a.gx;
    const int nbx = (a.groups + a.gx - 1) / a.gx;
    const int by = blockIdx.x / nbx, bx = blockIdx.x - by * nbx;
    stage_weights<W, CT>(a, sw, bx * a.gx * V, a.gx * V);
    const int cg = bx * a.gx + lx, tile_id = by * gy + ly, c0 = cg * V;
    if (cg >= a.groups || tile_id >= a.ntiles) return;
    const int row = tile_id / a.tiles_row;
    int t = (tile_id - row * a.tiles_row) * a.tile;
    const int t1 = min(t + a.tile, a.ax.len);
    const size_t tok0 = (size_t)row * a.ax.len;
    const TI* x = static_cast<const TI*>(a.x) + tok0 * a.ldx + c0;
    TI* y = static_cast<TI*>(a.y) + tok0 * a.D + c0;
    float w[W][V], bias[V], win[W - 1][V];
    read_weights<W, V>(sw, a.gx * V, lx * V, w, bias);
    copy_empty<TI, W, V>(a, tile_id, row, c0, a.h0, a.final_state);
    while (t < t1) {
        const Seq s = seq_at(a.ax, row, t);
        const int run = min(t1, s.end);
        Ring<TI, V, CU, CT> ring;
        ring.start(sw + (W + 1) * a.gx * V, x + (size_t)t * a.ldx, a.ldx, run - t);
        constexpr int AHEAD = ring.ASYNC ? CD - 1 : 1;
#pragma unroll
        for (int g = 0; g < AHEAD; ++g) {
            ring.fetch(g);
            copies_commit();
        }
        load_window<TI, W, V>(a, s, x, t, c0, win);
        if (t == s.first && a.final_state) {
            // the final state, by the thread that has the initial one in its window: the two may be one buffer
            const int len = s.end - s.first;
#pragma unroll
            for (int r = 0; r < W - 1; ++r) {
                const int p = len - (W - 1) + r;
                float f[V];
                if (p >= 0) {
                    unpack<V>(load_raw<TI, V>(x + (size_t)(s.first + p) * a.ldx), f);
                } else {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
                        if (k == len + r) {
#pragma unroll
                            for (int v = 0; v < V; ++v) f[v] = win[k][v];
                        }
                }
                store_values<V>(static_cast<TI*>(a.final_state) + ((size_t)s.n * (W - 1) + r) * a.D + c0, f);
            }
        }
        TI* yp = y + (size_t)t * a.D;
        for (int g = 0; t < run; ++g, t += CU) {
            Raw<TI, V> cur[CU];
            if (ring.ASYNC) {
                ring.fetch(g + AHEAD);
                copies_commit();
                copies_wait<CD - 1>();
            }
#pragma unroll
            for (int u = 0; u < CU; ++u) cur[u] = ring.get(g, u);
            if (!ring.ASYNC) ring.fetch(g + AHEAD);
            if (t + CU <= run) {
#pragma unroll
                for (int u = 0; u < CU; ++u) {
                    float xt[V], o[V];
                    unpack<V>(cur[u], xt);
                    conv_token<W, V, SILU>(w, bias, win, xt, o);
                    store_values<V>(yp + (size_t)u * a.D, o);
                }
            } else {
#pragma unroll
                for (int u = 0; u < CU - 1; ++u) {
                    if (t + u >= run) break;
                    float xt[V], o[V];
                    unpack<V>(cur[u], xt);
                    conv_token<W, V, SILU>(w, bias, win, xt, o);
                    store_values<V>(yp + (size_t)u * a.D, o);
                }
            }
            yp += (size_t)CU * a.D;
        }
        t = run;
    }
}

// One token per sequence (decoding): a thread takes its channels of RB sequences, every row in flight together and the
// filters read once for all of them.
template <typename TI, int W, int V, bool SILU, int RB>
__global__ void __launch_bounds__(CT) k_conv_step(ConvArgs a) {
    const size_t item = (size_t)blockIdx.x * CT + threadIdx.x;
    const int n0 = (int)(item / a.groups) * RB;
    if (n0 >= a.ax.N) return;
    const int c0 = (int)(item % a.groups) * V;
    Raw<TI, V> x[RB], win[RB][W - 1];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        if (n0 + r >= a.ax.N) break;
        x[r] = load_raw<TI, V>(static_cast<const TI*>(a.x) + (size_t)(n0 + r) * a.ldx + c0);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (a.h0) {
                win[r][j] = load_raw<TI, V>(static_cast<const TI*>(a.h0) + ((size_t)(n0 + r) * (W - 1) + j) * a.D + c0);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) win[r][j].v[v] = TI(0.f);
            }
        }
    }
    float w[W][V], bias[V];
    {
        Raw<float, V> q[W];   // V channels of W taps: W accesses of V values
        const bool wide = (reinterpret_cast<uintptr_t>(a.weight) & 15) == 0;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            if (wide) {
                q[k] = load_raw<float, V>(a.weight + (size_t)c0 * W + k * V);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) q[k].v[v] = a.weight[(size_t)c0 * W + k * V + v];
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][v] = q[(v * W + j) / V].v[(v * W + j) % V];
            bias[v] = a.bias ? a.bias[c0 + v] : 0.f;
        }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        if (n0 + r >= a.ax.N) break;
        float xt[V], h[W - 1][V], o[V];
        unpack<V>(x[r], xt);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) unpack<V>(win[r][j], h[j]);
        conv_token<W, V, SILU>(w, bias, h, xt, o);
        store_values<V>(static_cast<TI*>(a.y) + (size_t)(n0 + r) * a.D + c0, o);
        if (a.final_state) {
            TI* f = static_cast<TI*>(a.final_state) + (size_t)(n0 + r) * (W - 1) * a.D + c0;
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                *reinterpret_cast<Raw<TI, V>*>(f + (size_t)j * a.D) = j < W - 2 ? win[r][j < W - 2 ? j + 1 : 0] : x[r];
        }
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
        if (p >= first) unpack<V>(load_raw<TI, V>(x + (size_t)p * a.ldx), f[r]);
        else if (a.h0) unpack<V>(load_raw<TI, V>(static_cast<const TI*>(a.h0) + o + (size_t)(end - first + r) * a.D), f[r]);
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r) store_values<V>(static_cast<TI*>(a.final_state) + o + (size_t)r * a.D, f[r]);
}

// Block of gx channel groups by gy tiles; the tiles' parameter sums are added in tile order.
template <typename TI, int W, int V, bool SILU>
__global__ void __launch_bounds__(CB, 2) k_conv_bwd(ConvArgs a) {
    constexpr int BU = BWD_U<W>;
    extern __shared__ __align__(16) float smem[];   // the filters, [gy][gx * V] sums, the rings of x and dy
    char* const ring = reinterpret_cast<char*>(smem + (W + 1) * a.gx * V + CB * V);
    const int gx = a.gx, gy = CB / gx;
    const int lx = threadIdx.x & (gx - 1), ly = threadIdx.x / gx;
    const int nbx = (a.groups + gx - 1) / gx;
    const int part = blockIdx.x / nbx, bx = blockIdx.x - part * nbx;
    const int cg = bx * gx + lx, c0 = cg * V;
    const int tile_id = part * gy + ly;
    const bool on = cg < a.groups && tile_id < a.ntiles;
    stage_weights<W, CB>(a, smem, bx * gx * V, gx * V);
    float dw[W][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
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
        float w[W][V], bias[V];
        read_weights<W, V>(smem, gx * V, lx * V, w, bias);
        copy_empty<TI, W, V>(a, tile_id, row, c0, a.dfinal, a.dinit);
        while (t < t1) {
            const Seq s = seq_at(a.ax, row, t);
            const int run = min(t1, s.end), len = s.end - s.first, lim = min(run + W - 1, s.end);
            const bool start = t == s.first;
            Ring<TI, V, BU, CB> rx, rd;
            rx.start(ring, x + (size_t)t * a.ldx, a.ldx, lim - t);
            rd.start(ring + rx.BYTES, dy + (size_t)t * a.D, a.D, lim - t);
            constexpr int AHEAD = rx.ASYNC ? CD - 1 : 1;
#pragma unroll
            for (int g = 0; g < AHEAD; ++g) {
                rx.fetch(g);
                rd.fetch(g);
                copies_commit();
            }
            float win[W - 1][V], dwin[W - 1][V];   // x before the token (oldest first); d before it (newest first)
            load_window<TI, W, V>(a, s, x, t, c0, win);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) dwin[j][v] = 0.f;
            // the gradient of a token's s, and its part of the filters' sums
            auto gradient = [&](const float(&xt)[V], float(&d)[V]) {
                if (!SILU) return;
                float pre[V];
#pragma unroll
                for (int v = 0; v < V; ++v) pre[v] = bias[v];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) fma_v<V>(w[j], win[j], pre);
                fma_v<V>(w[W - 1], xt, pre);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float sg = sigmoid_fast(pre[v]);
                    d[v] *= sg * fmaf(pre[v], 1.f - sg, 1.f);
                }
            };
            auto add_sums = [&](const float(&xt)[V], const float(&d)[V]) {
#pragma unroll
                for (int v = 0; v < V; ++v) db[v] += d[v];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) fma_v<V>(d, win[j], dw[j]);
                fma_v<V>(d, xt, dw[W - 1]);
            };
            auto next_x = [&](const float(&xt)[V]) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int j = 0; j < W - 2; ++j) win[j][v] = win[j + 1][v];
                    win[W - 2][v] = xt[v];
                }
            };
            // dx of the token W - 1 back, complete with this one's d
            auto gather = [&](const float(&d)[V], float(&e)[V]) {
#pragma unroll
                for (int v = 0; v < V; ++v) e[v] = w[0][v] * d[v];
#pragma unroll
                for (int j = 1; j < W; ++j) fma_v<V>(w[j], dwin[j - 1], e);
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int j = W - 2; j > 0; --j) dwin[j][v] = dwin[j - 1][v];
                    dwin[0][v] = d[v];
                }
            };
            // W - 1 tokens past the run: their d reaches back into it (zero past the sequence)
            for (int tb = t, g = 0; tb < run + W - 1; tb += BU, ++g) {
                Raw<TI, V> cx[BU], cd[BU];
                if (rx.ASYNC) {
                    rx.fetch(g + AHEAD);
                    rd.fetch(g + AHEAD);
                    copies_commit();
                    copies_wait<CD - 1>();
                }
#pragma unroll
                for (int u = 0; u < BU; ++u) {
                    cx[u] = rx.get(g, u);
                    cd[u] = rd.get(g, u);
                }
                if (!rx.ASYNC) {
                    rx.fetch(g + AHEAD);
                    rd.fetch(g + AHEAD);
                }
                if (tb >= t + W - 1 && tb + BU <= run && tb + BU <= s.end - (df ? 1 : 0)) {
                    // inside the run: no case to tell apart
                    TI* dst = dx + (size_t)(tb - (W - 1)) * a.D;
#pragma unroll
                    for (int u = 0; u < BU; ++u) {
                        float xt[V], d[V], e[V];
                        unpack<V>(cx[u], xt);
                        unpack<V>(cd[u], d);
                        gradient(xt, d);
                        add_sums(xt, d);
                        next_x(xt);
                        gather(d, e);
                        store_values<V>(dst + (size_t)u * a.D, e);
                    }
                    continue;
                }
#pragma unroll
                for (int u = 0; u < BU; ++u) {
                    const int tt = tb + u;
                    if (tt >= run + W - 1) break;
                    float d[V], e[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) d[v] = 0.f;
                    if (tt < lim) {
                        float xt[V];
                        unpack<V>(cx[u], xt);
                        unpack<V>(cd[u], d);
                        gradient(xt, d);
                        if (tt < run) add_sums(xt, d);
                        next_x(xt);
                    }
                    gather(d, e);
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
                            unpack<V>(load_raw<TI, V>(df + ((size_t)s.n * (W - 1) + r) * a.D + c0), f);
#pragma unroll
                            for (int v = 0; v < V; ++v) e[v] += f[v];
                        }
                        store_values<V>(dst, e);
                    }
                }
            }
            t = run;
        }
    }
    // the block's sums, tap by tap
    const int ncol = gx * V;
    float* red = smem + (W + 1) * ncol;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) red[ly * ncol + lx * V + v] = j < W ? dw[j < W ? j : 0][v] : db[v];
        __syncthreads();
        for (int c = threadIdx.x; c < ncol; c += CB) {
            if (bx * ncol + c >= a.D) continue;
            float sum = 0.f;
            for (int k = 0; k < gy; ++k) sum += red[k * ncol + c];
            a.part[((size_t)part * (W + 1) + j) * a.D + bx * ncol + c] = sum;
        }
    }
}

// dweight and dbias from the blocks' sums.
__global__ void __launch_bounds__(256) k_conv_sum(ConvArgs a) {
    float sum;
    const int i = sum_parts(a.part, a.parts, (size_t)(a.W + 1) * a.D, sum);
    if (i < 0) return;
    const int j = i / a.D, d = i - j * a.D;
    if (j < a.W) a.dweight[(size_t)d * a.W + j] = sum;
    else if (a.dbias) a.dbias[d] = sum;
}

template <typename TI, int W, int V>
void run_fwd(const ConvArgs& a, cudaStream_t st) {
    const int gy = CT / a.gx;
    const unsigned grid = (unsigned)((a.ntiles + gy - 1) / gy) * ((a.groups + a.gx - 1) / a.gx);
    const size_t smem = sizeof(float) * (W + 1) * a.gx * V + Ring<TI, V, CU, CT>::BYTES;
    if (a.silu) k_conv_fwd<TI, W, V, true><<<grid, CT, smem, st>>>(a);
    else k_conv_fwd<TI, W, V, false><<<grid, CT, smem, st>>>(a);
}
template <typename TI, int W, int V, int RB>
void run_step_rows(const ConvArgs& a, cudaStream_t st) {
    const size_t items = (size_t)((a.ax.N + RB - 1) / RB) * a.groups;
    const unsigned grid = (unsigned)((items + CT - 1) / CT);
    if (a.silu) k_conv_step<TI, W, V, true, RB><<<grid, CT, 0, st>>>(a);
    else k_conv_step<TI, W, V, false, RB><<<grid, CT, 0, st>>>(a);
}
template <typename TI, int W, int V>
void run_step(const ConvArgs& a, cudaStream_t st) {
    // four sequences per thread once that leaves every SM a CTA
    if ((size_t)(a.ax.N / 4) * a.groups >= (size_t)sm_count() * CT) run_step_rows<TI, W, V, 4>(a, st);
    else run_step_rows<TI, W, V, 1>(a, st);
}
template <typename TI, int W, int V>
void run_state(const ConvArgs& a, cudaStream_t st) {
    const size_t items = (size_t)a.ax.N * a.groups;
    k_conv_state<TI, W, V><<<(unsigned)((items + CT - 1) / CT), CT, 0, st>>>(a);
}
constexpr int SMEM_MOST = 112 * 1024;   // two CTAs per SM
template <typename TI, int W, int V>
cudaError_t run_bwd(const ConvArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)a.parts * ((a.groups + a.gx - 1) / a.gx);
    const size_t smem = sizeof(float) * ((W + 1) * a.gx * V + CB * V) + 2 * Ring<TI, V, BWD_U<W>, CB>::BYTES;
    static SmemLimit limit[2];
    if (a.silu) {
        const cudaError_t e = limit[1].set(reinterpret_cast<const void*>(k_conv_bwd<TI, W, V, true>), SMEM_MOST);
        if (e != cudaSuccess) return e;
        k_conv_bwd<TI, W, V, true><<<grid, CB, smem, st>>>(a);
    } else {
        const cudaError_t e = limit[0].set(reinterpret_cast<const void*>(k_conv_bwd<TI, W, V, false>), SMEM_MOST);
        if (e != cudaSuccess) return e;
        k_conv_bwd<TI, W, V, false><<<grid, CB, smem, st>>>(a);
    }
    return cudaSuccess;
}

enum { FWD, STEP, STATE, BWD };
template <int OP, typename TI, int W, int V>
cudaError_t run_op(const ConvArgs& a, cudaStream_t st) {
    if constexpr (OP == FWD) run_fwd<TI, W, V>(a, st);
    else if constexpr (OP == STEP) run_step<TI, W, V>(a, st);
    else if constexpr (OP == STATE) run_state<TI, W, V>(a, st);
    else return run_bwd<TI, W, V>(a, st);
    return cudaSuccess;
}
template <int OP, typename TI, int V>
cudaError_t run_w(const ConvArgs& a, cudaStream_t st) {
    switch (a.W) {
        case 2: return run_op<OP, TI, 2, V>(a, st);
        case 3: return run_op<OP, TI, 3, V>(a, st);
        default: return run_op<OP, TI, 4, V>(a, st);
    }
}
template <int OP>
cudaError_t run_conv(const char* name, const ConvArgs& a, int bf16, bool vec, cudaStream_t st) {
    cudaError_t r = cudaSuccess;
    const cudaError_t e = traced_launch(name, st, [&] {
        if (bf16) r = vec ? run_w<OP, __nv_bfloat16, VC>(a, st) : run_w<OP, __nv_bfloat16, 1>(a, st);
        else r = vec ? run_w<OP, float, VC>(a, st) : run_w<OP, float, 1>(a, st);
    });
    return r != cudaSuccess ? r : e;
}

}  // namespace

void conv_shape(ConvArgs& a, bool vec, bool backward) {
    const int V = vec ? VC : 1;
    a.groups = a.D / V;
    a.gx = 1;
    const int most = backward ? 32 : CT;
    while (a.gx < most && a.gx < a.groups) a.gx *= 2;
    // Tokens per thread: long tiles re-read fewer window rows and filters, short ones fill the GPU. (Forward, 64 packed
    // tokens of 1024 channels: 4.9 us so chosen, 19.9 in tiles of 64; backward, 2 x 128 of 512: 8.7 us so chosen, 24.4 in
    // tiles of 256.)
    int tile;
    if (backward) {
        // whole waves of CTAs (two per SM) of at most 256 tokens per thread, and no fewer than 8
        const long long nbx = (a.groups + a.gx - 1) / a.gx, gy = CB / a.gx, tokens = (long long)a.ax.rows * a.ax.len;
        long long parts = 0;
        do parts += 2LL * sm_count() / nbx > 0 ? 2LL * sm_count() / nbx : 1;
        while (tokens > parts * gy * 256);
        const long long per_row = parts * gy / a.ax.rows > 0 ? parts * gy / a.ax.rows : 1;
        tile = (int)((a.ax.len + per_row - 1) / per_row);
        if (tile < 8) tile = 8;
    } else {
        tile = 64;
        while (tile > 1 && (long long)a.groups * a.ax.rows * ((a.ax.len + tile - 1) / tile) < sm_count() * 1024LL) tile /= 2;
    }
    a.tile = tile;
    a.tiles_row = a.ax.len > 0 ? (a.ax.len + tile - 1) / tile : 1;
    a.ntiles = a.ax.rows * a.tiles_row;
    const int gy = CB / a.gx;
    a.parts = (a.ntiles + gy - 1) / gy;
}

cudaError_t launch_conv_fwd(ConvArgs a, int bf16, bool vec, cudaStream_t st) {
    if (!a.ax.cu && a.ax.len == 1) return run_conv<STEP>("k_conv_step", a, bf16, vec, st);
    // a state updated in place: the thread that starts a sequence writes its final state, which is safe unless a
    // second tile reads initial rows too (tiles shorter than the window, or packed offsets anywhere in a tile)
    void* in_place = nullptr;
    if (a.final_state && a.final_state == a.h0 && (a.ax.cu || (a.tiles_row > 1 && a.tile < a.W - 1))) {
        in_place = a.final_state;
        a.final_state = nullptr;
    }
    cudaError_t e = run_conv<FWD>("k_conv_fwd", a, bf16, vec, st);
    if (e != cudaSuccess || !in_place) return e;
    a.final_state = in_place;
    return run_conv<STATE>("k_conv_state", a, bf16, vec, st);
}

cudaError_t launch_conv_bwd(ConvArgs a, int bf16, bool vec, cudaStream_t st) {
    cudaError_t e = run_conv<BWD>("k_conv_bwd", a, bf16, vec, st);
    if (e != cudaSuccess) return e;
    const unsigned n = (unsigned)((a.W + 1) * a.D);
    return traced_launch("k_conv_sum", st, [&] { k_conv_sum<<<(n + 31) / 32, 256, 0, st>>>(a); });
}

}  // namespace kda
