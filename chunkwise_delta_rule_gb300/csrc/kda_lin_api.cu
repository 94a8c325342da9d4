// C entry points of linear attention with a decay for each head: argument
// validation, workspace layout, launch order. Contracts in include/kda.h.
#include "kda_api.cuh"
#include "kda_lin.cuh"

namespace {

using namespace kda::api;

struct Lin {
    kda::LinArgs a{};
    int H, K, V, bf16;
    int64_t ldq, ldk, ldv;
    float scale;
};

kda_status lin_args(const kda_lin_problem* p, Lin& l) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "problem is NULL");
    const kda_status st = make_axis(p->B, p->T, p->N, p->cu_seqlens, p->K, p->io, l.a.ax);
    if (st != KDA_OK) return st;
    if (p->H < 1 || p->V < 1) return fail(KDA_ERR_INVALID_ARG, "H and V must be >= 1");
    if (p->K > kda::LIN_MAX_W || p->V > kda::LIN_MAX_W) return fail(KDA_ERR_UNSUPPORTED, "K and V must be at most 256");
    const int HV = p->HV ? p->HV : p->H;
    if (HV < p->H || HV % p->H) return fail(KDA_ERR_INVALID_ARG, "HV must be a multiple of H");
    if (HV > (1 << 16)) return fail(KDA_ERR_UNSUPPORTED, "more than 2^16 value heads");
    const int64_t wk = (int64_t)p->H * p->K, wv = (int64_t)HV * p->V;
    if ((p->ldq && p->ldq < wk) || (p->ldk && p->ldk < wk) || (p->ldv && p->ldv < wv))
        return fail(KDA_ERR_INVALID_ARG, "a leading dimension is shorter than its row");
    if (!(p->scale <= 3e38f)) return fail(KDA_ERR_INVALID_ARG, "scale must be finite");
    l.H = p->H;
    l.K = p->K;
    l.V = p->V;
    l.bf16 = p->io == KDA_BF16;
    l.ldq = p->ldq ? p->ldq : wk;
    l.ldk = p->ldk ? p->ldk : wk;
    l.ldv = p->ldv ? p->ldv : wv;
    l.scale = p->scale > 0.f ? p->scale : 1.f / sqrtf((float)p->K);
    l.a.HV = HV;
    l.a.decay = p->decay;
    return KDA_OK;
}

size_t state_bytes(const Lin& l, size_t n) { return up(sizeof(float) * n * l.a.HV * l.K * l.V); }
// CTAs of a time window on the tensor cores.
int tc_ctas(const Lin& l, bool backward) {
    const int blocks = (l.V + 63) / 64, kblocks = (l.K + 63) / 64;
    return l.a.HV * (backward ? blocks + 2 * kblocks : blocks);
}
// Whether sizes alone let a call run on the tensor cores (its rows' alignment has to, too).
bool tc_sizes(const Lin& l, bool backward) {
    if (!l.bf16 || l.K % 8 || l.V % 8 || l.K > 128 || (backward && l.V > 128)) return false;
    const bool spread = l.a.ax.cu && 3ll * tc_ctas(l, backward) < kda::sm_count();
    const int least = spread ? (backward ? kda::LIN_TC_PACKED_BACK : kda::LIN_TC_PACKED) : (backward ? kda::LIN_TC_TOKENS_BACK : kda::LIN_TC_TOKENS);
    return (int64_t)l.a.ax.rows * l.a.ax.len >= (int64_t)least * l.a.ax.N;
}
void set_windows(Lin& l, bool backward, bool tc) {
    int len;
    if (tc) {
        len = kda::lin_tc_window(l.a.ax.rows, l.a.ax.len, tc_ctas(l, backward));
    } else {
        const int widths[3] = {l.V, l.K, l.K}, calls = backward ? 3 : 1;
        const int kmax = backward && l.V > l.K ? l.V : l.K, slice = kda::lin_slice(kmax, widths, calls);
        int ctas = 0;
        for (int i = 0; i < calls; ++i) ctas += l.a.HV * ((widths[i] + slice - 1) / slice);
        len = kda::lin_window(l.a.ax.rows, l.a.ax.len, ctas, kmax, slice);
    }
    l.a.unit_len = len > 0 ? len : 64;
    l.a.units_row = l.a.ax.len > 0 ? (l.a.ax.len + l.a.unit_len - 1) / l.a.unit_len : 1;
}
struct Layout {
    size_t local = 0, alias = 0, dq = 0, dk = 0;
    size_t all(bool backward) const { return backward ? 3 * local + dq + dk : local + alias; }
};
Layout layout(const Lin& l, bool backward) {
    Layout y;
    if (l.a.units_row > 1) {
        y.local = state_bytes(l, (size_t)l.a.ax.rows * l.a.units_row);
        y.alias = state_bytes(l, l.a.ax.N);
    }
    if (backward && l.a.HV != l.H) y.dq = y.dk = up(sizeof(float) * (size_t)l.a.ax.rows * l.a.ax.len * l.a.HV * l.K);
    return y;
}
// The larger of the two paths' workspaces: which one runs goes by the pointers' alignment, too.
size_t most_bytes(Lin l, bool backward) {
    size_t most = 0;
    for (int tc = 0; tc < 2; ++tc) {
        if (tc && !tc_sizes(l, backward)) continue;
        set_windows(l, backward, tc);
        const size_t b = layout(l, backward).all(backward);
        most = b > most ? b : most;
    }
    return most;
}

}  // namespace

extern "C" {

size_t kda_lin_workspace_size(const kda_lin_problem* p, int for_backward) {
    Lin l;
    if (lin_args(p, l) != KDA_OK) return 0;
    return most_bytes(l, for_backward != 0);
}

kda_status kda_lin_fwd(const kda_lin_problem* p, void* o, float* ht, void* ws, size_t ws_bytes, int32_t* err,
                       kda_stream_t stream) {
    Lin l;
    kda_status st = lin_args(p, l);
    if (st != KDA_OK) return st;
    if (l.a.ax.len > 0 && (!p->q || !p->k || !p->v || !o)) return fail(KDA_ERR_INVALID_ARG, "q, k, v and o must be non-NULL");
    if ((st = check_ws(ws, ws_bytes, most_bytes(l, false), "workspace")) != KDA_OK) return st;
    Carver cw{static_cast<char*>(ws)};
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const int G = l.a.HV / l.H;
    l.a.err = err;
    l.a.calls = 1;
    kda::LinCall& c = l.a.c[0];
    c = {p->q, p->k, p->v, l.ldq, l.ldk, l.ldv, G, G, 1, l.K, l.V, o, 0, p->h0, ht, 0, 0, l.scale, 1.f, nullptr};
    const bool tc = tc_sizes(l, false) && kda::lin_tc_call(c);
    set_windows(l, false, tc);
    const Layout y = layout(l, false);
    c.local = cw.take<float>(y.local);
    // the last window of a sequence would overwrite the state that its other windows read
    if (y.alias && ht && ht == p->h0) c.s1 = cw.take<float>(y.alias);
    if ((st = cuda_result(tc ? kda::launch_lin_tc(l.a, cs) : kda::launch_lin(l.a, l.bf16, cs), "linear attention")) != KDA_OK) return st;
    if (c.s1 != ht)
        return cuda_result(cudaMemcpyAsync(ht, c.s1, sizeof(float) * (size_t)l.a.ax.N * l.a.HV * l.K * l.V,
                                           cudaMemcpyDeviceToDevice, cs), "copy of the final states");
    return KDA_OK;
}

kda_status kda_lin_bwd(const kda_lin_problem* p, const void* dout, const float* dht, void* dq, void* dk, void* dv,
                       float* dh0, void* ws, size_t ws_bytes, int32_t* err, kda_stream_t stream) {
    Lin l;
    kda_status st = lin_args(p, l);
    if (st != KDA_OK) return st;
    if (l.a.ax.len > 0 && (!p->q || !p->k || !p->v || !dout || !dq || !dk || !dv))
        return fail(KDA_ERR_INVALID_ARG, "q, k, v, dout, dq, dk and dv must be non-NULL");
    if (dh0 && (dh0 == dht || dh0 == p->h0)) return fail(KDA_ERR_INVALID_ARG, "dh0 must have a buffer of its own");
    if ((st = check_ws(ws, ws_bytes, most_bytes(l, true), "workspace")) != KDA_OK) return st;
    Carver cw{static_cast<char*>(ws)};
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const int G = l.a.HV / l.H, K = l.K, V = l.V;
    const int64_t ldo = (int64_t)l.a.HV * V;
    const size_t part = layout(l, true).dq;   // the same on both paths
    float* pq = cw.take<float>(part);
    float* pk = cw.take<float>(part);
    l.a.err = err;
    l.a.calls = 3;
    l.a.c[0] = {dout, p->v, p->k, ldo, l.ldv, l.ldk, 1, 1, G, V, K, pq ? pq : dq, pq != nullptr, p->h0, nullptr, 1, 0, l.scale, 1.f, nullptr};
    l.a.c[1] = {p->v, dout, p->q, l.ldv, ldo, l.ldq, 1, 1, G, V, K, pk ? pk : dk, pk != nullptr, dht, nullptr, 1, 1, 1.f, l.scale, nullptr};
    l.a.c[2] = {p->k, p->q, dout, l.ldk, l.ldq, ldo, G, G, 1, K, V, dv, 0, dht, dh0, 0, 1, 1.f, l.scale, nullptr};
    bool tc = tc_sizes(l, true);
    for (const kda::LinCall& c : l.a.c) tc = tc && kda::lin_tc_call(c);
    set_windows(l, true, tc);
    const Layout y = layout(l, true);
    for (kda::LinCall& c : l.a.c) c.local = cw.take<float>(y.local);
    if ((st = cuda_result(tc ? kda::launch_lin_tc(l.a, cs) : kda::launch_lin(l.a, l.bf16, cs), "linear attention backward")) != KDA_OK) return st;
    if (!pq) return KDA_OK;
    const int64_t rows = (int64_t)l.a.ax.rows * l.a.ax.len * l.H;
    if ((st = cuda_result(kda::launch_lin_heads(pq, dq, rows, G, K, l.bf16, cs), "linear attention backward (heads)")) != KDA_OK) return st;
    return cuda_result(kda::launch_lin_heads(pk, dk, rows, G, K, l.bf16, cs), "linear attention backward (heads)");
}

}  // extern "C"
