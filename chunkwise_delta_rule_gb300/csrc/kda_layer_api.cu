// C entry points of the layer operators (short convolution, selective state space
// scan, root-mean-square norm): argument validation, workspace layout, launch
// order. Contracts in include/kda.h.
#include "kda_api.cuh"

namespace {

using namespace kda::api;

// ------------------------------------------------------------------ convolution
kda_status conv_args(const kda_conv_problem* p, kda::ConvArgs& a) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "problem is NULL");
    a = kda::ConvArgs{};
    const kda_status st = make_axis(p->B, p->T, p->N, p->cu_seqlens, p->D, p->io, a.ax);
    if (st != KDA_OK) return st;
    if (p->W < 2 || p->W > 4) return fail(KDA_ERR_UNSUPPORTED, "W must be 2, 3 or 4");
    if (p->silu != 0 && p->silu != 1) return fail(KDA_ERR_INVALID_ARG, "silu must be 0 or 1");
    if (p->ldx != 0 && p->ldx < p->D) return fail(KDA_ERR_INVALID_ARG, "ldx must be 0 or at least D");
    a.D = p->D;
    a.W = p->W;
    a.silu = p->silu;
    a.ldx = p->ldx ? (size_t)p->ldx : (size_t)p->D;
    a.x = p->x;
    a.h0 = p->h0;
    a.weight = p->weight;
    a.bias = p->bias;
    return KDA_OK;
}
kda_status conv_pointers(const kda::ConvArgs& a) {
    if (!a.weight) return fail(KDA_ERR_INVALID_ARG, "weight must be non-NULL");
    if (a.ax.len > 0 && !a.x) return fail(KDA_ERR_INVALID_ARG, "x must be non-NULL");
    return KDA_OK;
}
// Whether rows take accesses of four channels.
bool conv_vec(const kda::ConvArgs& a) {
    return a.D % 4 == 0 && a.ldx % 4 == 0 && aligned16(a.x) && aligned16(a.h0) && aligned16(a.y) &&
           aligned16(a.final_state) && aligned16(a.dy) && aligned16(a.dfinal) && aligned16(a.dx) && aligned16(a.dinit);
}
// The partial sums' bytes, whichever path the pointers' alignment will select.
size_t conv_part_bytes(kda::ConvArgs a) {
    size_t most = 0;
    for (int vec = 0; vec < 2; ++vec) {
        if (vec && a.D % 4) continue;
        kda::conv_shape(a, vec, true);
        const size_t b = sizeof(float) * (size_t)a.parts * (a.W + 1) * a.D;
        most = b > most ? b : most;
    }
    return up(most);
}

// ------------------------------------------------------------------ scan
struct SsmLayout {
    size_t pieces = 0;   // local end states and sums of delta (forward and backward passes share the sums)
    size_t alias = 0;    // final states of a call that updates them in place in several pieces
    size_t ckpt = 0;
    size_t rloc = 0, pA = 0, pv = 0, pbc = 0;
};

kda_status ssm_args(const kda_ssm_problem* p, kda::SsmArgs& a) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "problem is NULL");
    a = kda::SsmArgs{};
    const kda_status st = make_axis(p->B, p->T, p->N, p->cu_seqlens, p->D, p->io, a.ax);
    if (st != KDA_OK) return st;
    if (p->S < 1) return fail(KDA_ERR_INVALID_ARG, "S must be >= 1");
    if (p->S > 64) return fail(KDA_ERR_UNSUPPORTED, "more than 64 states per channel");
    if (p->G < 1 || p->D % p->G) return fail(KDA_ERR_INVALID_ARG, "G must divide D");
    if (p->dt_softplus != 0 && p->dt_softplus != 1) return fail(KDA_ERR_INVALID_ARG, "dt_softplus must be 0 or 1");
    if (p->save_policy != 0 && p->save_policy != 1) return fail(KDA_ERR_INVALID_ARG, "save_policy must be 0 or 1");
    const int64_t GS = (int64_t)p->G * p->S;
    if ((p->ldx && p->ldx < p->D) || (p->lddt && p->lddt < p->D) || (p->ldz && p->ldz < p->D) ||
        (p->ldb && p->ldb < GS) || (p->ldc && p->ldc < GS))
        return fail(KDA_ERR_INVALID_ARG, "a leading dimension is shorter than its row");
    a.D = p->D;
    a.S = p->S;
    a.G = p->G;
    a.softplus = p->dt_softplus;
    a.ldx = p->ldx ? p->ldx : p->D;
    a.lddt = p->lddt ? p->lddt : p->D;
    a.ldz = p->ldz ? p->ldz : p->D;
    a.ldb = p->ldb ? p->ldb : GS;
    a.ldc = p->ldc ? p->ldc : GS;
    a.x = p->x;
    a.dt = p->dt;
    a.z = p->z;
    a.b = p->b;
    a.c = p->c;
    a.A_log = p->A_log;
    a.d_skip = p->d_skip;
    a.dt_bias = p->dt_bias;
    a.h0 = p->h0;
    return KDA_OK;
}
kda_status ssm_pointers(const kda::SsmArgs& a) {
    if (!a.A_log) return fail(KDA_ERR_INVALID_ARG, "A_log must be non-NULL");
    if (a.ax.len > 0 && (!a.x || !a.dt || !a.b || !a.c)) return fail(KDA_ERR_INVALID_ARG, "x, dt, b and c must be non-NULL");
    return KDA_OK;
}
void ssm_pieces(kda::SsmArgs& a, bool backward) {
    const int units = kda::ssm_units(a.ax.rows, a.ax.len, a.D, a.G, a.S, backward);
    int len = (a.ax.len + units - 1) / units;
    len = (len + 31) / 32 * 32;
    a.unit_len = len > 0 ? len : 32;
    a.units_row = a.ax.len > 0 ? (a.ax.len + a.unit_len - 1) / a.unit_len : 1;
}
// Access to the rows of p, `ld` elements apart; whether the groups inside a row start on 16 (4) bytes.
int ssm_how(const void* p, size_t ld, bool groups16, bool groups4, int es, int shift) {
    const uintptr_t q = reinterpret_cast<uintptr_t>(p);
    const int how = groups16 && q % 16 == 0 && ld * es % 16 == 0 ? 0 : groups4 && q % 4 == 0 && ld * es % 4 == 0 ? 1 : 2;
    return how << shift;
}
void ssm_access(kda::SsmArgs& a, int es, const void* dy, const void* o0, const void* o1, const void* o2) {
    // a group's channels and states start D / G and S elements after the previous group's
    const bool c16 = a.G == 1 || (size_t)(a.D / a.G) * es % 16 == 0, c4 = a.G == 1 || (size_t)(a.D / a.G) * es % 4 == 0;
    const bool s16 = a.G == 1 || (size_t)a.S * es % 16 == 0, s4 = a.G == 1 || (size_t)a.S * es % 4 == 0;
    const bool out = c16 && (size_t)a.D * es % 16 == 0 && aligned16(o0) && aligned16(o1) && aligned16(o2);
    a.how = ssm_how(a.x, a.ldx, c16, c4, es, kda::SSM_X) | ssm_how(a.dt, a.lddt, c16, c4, es, kda::SSM_DT) |
            ssm_how(a.z, a.ldz, c16, c4, es, kda::SSM_Z) | ssm_how(a.b, a.ldb, s16, s4, es, kda::SSM_B) |
            ssm_how(a.c, a.ldc, s16, s4, es, kda::SSM_C) | ssm_how(dy, a.D, c16, c4, es, kda::SSM_DY) |
            (out ? 0 : 2) << kda::SSM_OUT;
}
size_t ssm_state_bytes(const kda::SsmArgs& a, size_t n) { return up(sizeof(float) * n * a.D * a.S); }
size_t ssm_ckpt_bytes(const kda::SsmArgs& a) {
    return ssm_state_bytes(a, (size_t)a.ax.rows * ((a.ax.len + kda::SSM_CKPT - 1) / kda::SSM_CKPT));
}
// Bytes of each part for the pieces already in `a`.
SsmLayout ssm_layout(const kda::SsmArgs& a, bool backward, int save) {
    SsmLayout L;
    const size_t units = (size_t)a.ax.rows * a.units_row, tokens = (size_t)a.ax.rows * a.ax.len;
    if (a.units_row > 1) L.pieces = ssm_state_bytes(a, units) + up(sizeof(float) * units * a.D);
    if (!backward) {
        if (a.units_row > 1) L.alias = ssm_state_bytes(a, a.ax.N);
        return L;
    }
    if (!save) L.ckpt = ssm_ckpt_bytes(a);
    if (a.units_row > 1) L.rloc = ssm_state_bytes(a, units);
    L.pA = ssm_state_bytes(a, units);
    L.pv = up(sizeof(float) * units * 2 * a.D);
    L.pbc = up(sizeof(float) * kda::ssm_bwd_tiles(a.D, a.G, a.S) * tokens * 2 * a.S);
    return L;
}

// ------------------------------------------------------------------ norm
kda_status norm_args(const kda_norm_problem* p, kda::NormArgs& a) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "problem is NULL");
    a = kda::NormArgs{};
    if (p->rows < 0 || p->D < 1) return fail(KDA_ERR_INVALID_ARG, "rows must be >= 0 and D >= 1");
    // the kernels' row counters step over the last row by a grid's rows
    if (p->rows > (1 << 30)) return fail(KDA_ERR_UNSUPPORTED, "more than 2^30 rows");
    if (p->D > kda::NORM_MAX_D) return fail(KDA_ERR_UNSUPPORTED, "rows wider than 16384");
    if (p->io != KDA_BF16 && p->io != KDA_FP32) return fail(KDA_ERR_INVALID_ARG, "unknown io dtype");
    if (p->out != 0 && p->out != 1) return fail(KDA_ERR_INVALID_ARG, "out must be 0 or 1");
    if (p->group != 0 && p->group != 32 && p->group != 64 && p->group != 128)
        return fail(KDA_ERR_UNSUPPORTED, "group must be 0, 32, 64 or 128");
    if (!(p->eps >= 0.f)) return fail(KDA_ERR_INVALID_ARG, "eps must be >= 0");
    a.rows = p->rows;
    a.D = p->D;
    a.out = p->out;
    a.group = p->group;
    a.ngroups = p->group ? (p->D + p->group - 1) / p->group : 1;
    a.eps = p->eps;
    a.x = p->x;
    a.residual = p->residual;
    a.weight = p->weight;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_conv_fwd(const kda_conv_problem* p, void* y, void* final_state, int32_t* err, kda_stream_t stream) {
    kda::ConvArgs a;
    kda_status st = conv_args(p, a);
    if (st != KDA_OK || (st = conv_pointers(a)) != KDA_OK) return st;
    if (a.ax.len > 0 && !y) return fail(KDA_ERR_INVALID_ARG, "y must be non-NULL");
    a.y = y;
    a.final_state = final_state;
    a.err = err;
    const int bf16 = p->io == KDA_BF16;
    const bool vec = conv_vec(a);
    kda::conv_shape(a, vec, false);
    return cuda_result(kda::launch_conv_fwd(a, bf16, vec, reinterpret_cast<cudaStream_t>(stream)), "short convolution");
}

size_t kda_conv_workspace_size(const kda_conv_problem* p) {
    kda::ConvArgs a;
    return conv_args(p, a) == KDA_OK ? conv_part_bytes(a) : 0;
}

kda_status kda_conv_bwd(const kda_conv_problem* p, const void* dy, const void* dfinal, void* dx, float* dweight,
                        float* dbias, void* dinit, void* ws, size_t ws_bytes, kda_stream_t stream) {
    kda::ConvArgs a;
    kda_status st = conv_args(p, a);
    if (st != KDA_OK || (st = conv_pointers(a)) != KDA_OK) return st;
    if (!dweight || (a.ax.len > 0 && (!dy || !dx))) return fail(KDA_ERR_INVALID_ARG, "dy, dx and dweight must be non-NULL");
    const int bf16 = p->io == KDA_BF16;
    if ((st = check_ws(ws, ws_bytes, conv_part_bytes(a), "workspace")) != KDA_OK) return st;
    a.dy = dy;
    a.dfinal = dfinal;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dinit = dinit;
    a.part = static_cast<float*>(ws);
    const bool vec = conv_vec(a);
    kda::conv_shape(a, vec, true);
    return cuda_result(kda::launch_conv_bwd(a, bf16, vec, reinterpret_cast<cudaStream_t>(stream)),
                       "short convolution backward");
}

size_t kda_ssm_workspace_size(const kda_ssm_problem* p, int for_backward) {
    kda::SsmArgs a;
    if (ssm_args(p, a) != KDA_OK) return 0;
    ssm_pieces(a, for_backward != 0);
    const SsmLayout L = ssm_layout(a, for_backward != 0, p->save_policy);
    return L.pieces + L.alias + L.ckpt + L.rloc + L.pA + L.pv + L.pbc;
}

size_t kda_ssm_saved_size(const kda_ssm_problem* p) {
    kda::SsmArgs a;
    return ssm_args(p, a) == KDA_OK && p->save_policy ? ssm_ckpt_bytes(a) : 0;
}

kda_status kda_ssm_fwd(const kda_ssm_problem* p, void* y, float* ht, void* saved, void* ws, size_t ws_bytes,
                       int32_t* err, kda_stream_t stream) {
    kda::SsmArgs a;
    kda_status st = ssm_args(p, a);
    if (st != KDA_OK || (st = ssm_pointers(a)) != KDA_OK) return st;
    if (a.ax.len > 0 && !y) return fail(KDA_ERR_INVALID_ARG, "y must be non-NULL");
    ssm_pieces(a, false);
    const SsmLayout L = ssm_layout(a, false, p->save_policy);
    if ((st = check_ws(ws, ws_bytes, L.pieces + L.alias, "workspace")) != KDA_OK) return st;
    if (p->save_policy && (st = check_ws(saved, ssm_ckpt_bytes(a), ssm_ckpt_bytes(a), "saved buffer")) != KDA_OK) return st;
    const int bf16 = p->io == KDA_BF16;
    ssm_access(a, esize(p->io), nullptr, y, nullptr, nullptr);
    a.y = y;
    a.err = err;
    a.ckpt = p->save_policy ? static_cast<float*>(saved) : nullptr;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    float* target = ht;
    if (a.units_row > 1) {
        const size_t units = (size_t)a.ax.rows * a.units_row;
        Carver cw{static_cast<char*>(ws)};
        a.hloc = cw.take<float>(ssm_state_bytes(a, units));
        a.sdt = cw.take<float>(up(sizeof(float) * units * a.D));
        // the last piece of a sequence would overwrite the state that its first one reads
        if (ht && ht == a.h0) target = cw.take<float>(L.alias);
        if ((st = cuda_result(kda::launch_ssm_pieces(a, bf16, cs), "scan (pieces)")) != KDA_OK) return st;
    }
    a.ht = target;
    if ((st = cuda_result(kda::launch_ssm_fwd(a, bf16, p->save_policy ? 1 : 0, cs), "scan")) != KDA_OK) return st;
    if (target != ht)
        return cuda_result(cudaMemcpyAsync(ht, target, sizeof(float) * (size_t)a.ax.N * a.D * a.S,
                                           cudaMemcpyDeviceToDevice, cs), "copy of the final states");
    return KDA_OK;
}

kda_status kda_ssm_bwd(const kda_ssm_problem* p, const void* dy, const float* dht, const void* saved,
                       const kda_ssm_grads* g, void* ws, size_t ws_bytes, kda_stream_t stream) {
    return kda_ssm_bwd_err(p, dy, dht, saved, g, ws, ws_bytes, nullptr, stream);
}

kda_status kda_ssm_bwd_err(const kda_ssm_problem* p, const void* dy, const float* dht, const void* saved,
                           const kda_ssm_grads* g, void* ws, size_t ws_bytes, int32_t* err, kda_stream_t stream) {
    kda::SsmArgs a;
    kda_status st = ssm_args(p, a);
    if (st != KDA_OK || (st = ssm_pointers(a)) != KDA_OK) return st;
    if (!g || !g->dA_log) return fail(KDA_ERR_INVALID_ARG, "dA_log must be non-NULL");
    if (a.ax.len > 0 && (!dy || !g->dx || !g->ddt || !g->db || !g->dc || (a.z && !g->dz)))
        return fail(KDA_ERR_INVALID_ARG, "dy, dx, ddt, db, dc (and dz with z) must be non-NULL");
    ssm_pieces(a, true);
    const SsmLayout L = ssm_layout(a, true, p->save_policy);
    if ((st = check_ws(ws, ws_bytes, L.pieces + L.ckpt + L.rloc + L.pA + L.pv + L.pbc, "workspace")) != KDA_OK) return st;
    if (p->save_policy && (st = check_ws(saved, ssm_ckpt_bytes(a), ssm_ckpt_bytes(a), "saved buffer")) != KDA_OK) return st;
    const int bf16 = p->io == KDA_BF16;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const size_t units = (size_t)a.ax.rows * a.units_row;
    Carver cw{static_cast<char*>(ws)};
    if (L.pieces) {
        a.hloc = cw.take<float>(ssm_state_bytes(a, units));
        a.sdt = cw.take<float>(up(sizeof(float) * units * a.D));
    }
    a.ckpt = L.ckpt ? cw.take<float>(L.ckpt) : const_cast<float*>(static_cast<const float*>(saved));
    a.rloc = cw.take<float>(L.rloc);
    a.pA = cw.take<float>(L.pA);
    a.pv = cw.take<float>(L.pv);
    a.pbc = cw.take<float>(L.pbc);
    ssm_access(a, esize(p->io), dy, g->dx, g->ddt, g->dz);
    a.err = err;
    if (!p->save_policy && a.ax.len > 0) {
        if (a.units_row > 1 && (st = cuda_result(kda::launch_ssm_pieces(a, bf16, cs), "scan (pieces)")) != KDA_OK) return st;
        if ((st = cuda_result(kda::launch_ssm_fwd(a, bf16, 2, cs), "scan (recompute)")) != KDA_OK) return st;
    }
    a.dy = dy;
    a.dht = dht;
    a.dx = g->dx;
    a.ddt = g->ddt;
    a.dz = g->dz;
    a.db = g->db;
    a.dc = g->dc;
    a.dA_log = g->dA_log;
    a.dd_skip = g->dd_skip;
    a.ddt_bias = g->ddt_bias;
    a.dh0 = g->dh0;
    if (a.units_row > 1 && (st = cuda_result(kda::launch_ssm_bwd_pieces(a, bf16, cs), "scan backward (pieces)")) != KDA_OK) return st;
    if ((st = cuda_result(kda::launch_ssm_bwd(a, bf16, cs), "scan backward")) != KDA_OK) return st;
    return cuda_result(kda::launch_ssm_bwd_sums(a, bf16, cs), "scan backward (sums)");
}

kda_status kda_norm_fwd(const kda_norm_problem* p, void* y, float* scale, void* h, kda_stream_t stream) {
    kda::NormArgs a;
    const kda_status st = norm_args(p, a);
    if (st != KDA_OK) return st;
    if (a.rows == 0) return KDA_OK;
    if (!a.x || !a.weight || !y) return fail(KDA_ERR_INVALID_ARG, "x, weight and y must be non-NULL");
    if (a.out && !scale) return fail(KDA_ERR_INVALID_ARG, "an 8-bit output needs scale");
    if (a.residual && !h) return fail(KDA_ERR_INVALID_ARG, "h must be non-NULL with a residual");
    a.y = y;
    a.scale = scale;
    a.h = h;
    return cuda_result(kda::launch_norm_fwd(a, p->io == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)), "norm");
}

size_t kda_norm_workspace_size(const kda_norm_problem* p) {
    kda::NormArgs a;
    return norm_args(p, a) == KDA_OK ? up(sizeof(float) * (size_t)kda::norm_bwd_parts(a.rows, a.D) * a.D) : 0;
}

kda_status kda_norm_bwd(const kda_norm_problem* p, const void* dy, const void* dres, void* dx, float* dweight,
                        void* ws, size_t ws_bytes, kda_stream_t stream) {
    kda::NormArgs a;
    kda_status st = norm_args(p, a);
    if (st != KDA_OK) return st;
    if (a.residual) return fail(KDA_ERR_INVALID_ARG, "the backward takes the stored sum as x and no residual");
    if (!a.weight || !dweight || (a.rows > 0 && (!a.x || !dy || !dx)))
        return fail(KDA_ERR_INVALID_ARG, "x, weight, dy, dx and dweight must be non-NULL");
    a.parts = kda::norm_bwd_parts(a.rows, a.D);
    if ((st = check_ws(ws, ws_bytes, sizeof(float) * (size_t)a.parts * a.D, "workspace")) != KDA_OK) return st;
    a.dy = dy;
    a.dres = dres;
    a.dx = dx;
    a.dweight = dweight;
    a.part = static_cast<float*>(ws);
    return cuda_result(kda::launch_norm_bwd(a, p->io == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)), "norm backward");
}

}  // extern "C"
