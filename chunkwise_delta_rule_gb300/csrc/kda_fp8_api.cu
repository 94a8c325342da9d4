// C entry points of the 8-bit quantiser and product: argument validation,
// workspace layout, launch order. Contracts in include/kda.h.
#include "kda_api.cuh"
#include "kda_fp8.cuh"

namespace {

using namespace kda::api;

constexpr int MAX_ROWS = 1 << 22, MAX_COLS = 1 << 20;   // a grid has at most 65535 tiles of 128 rows on its second and third axes

kda_status quant8_args(const kda_quant8_problem* p, kda::Quant8Args& a) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "problem is NULL");
    a = kda::Quant8Args{};
    if (p->rows < 0 || p->D < 1) return fail(KDA_ERR_INVALID_ARG, "rows must be >= 0 and D >= 1");
    if (p->rows > MAX_ROWS || p->D > MAX_COLS) return fail(KDA_ERR_UNSUPPORTED, "more than 2^22 rows or 2^20 columns");
    if (p->io != KDA_BF16 && p->io != KDA_FP32) return fail(KDA_ERR_INVALID_ARG, "unknown io dtype");
    if (p->blocks != 0 && p->blocks != 1) return fail(KDA_ERR_INVALID_ARG, "blocks must be 0 or 1");
    if ((p->ldx && p->ldx < p->D) || (p->ldq && p->ldq < p->D) || (p->ldqt && p->ldqt < p->rows))
        return fail(KDA_ERR_INVALID_ARG, "a leading dimension is shorter than its row");
    a.rows = p->rows;
    a.D = p->D;
    a.blocks = p->blocks;
    a.ldx = p->ldx ? p->ldx : p->D;
    a.ldq = p->ldq ? p->ldq : p->D;
    a.ldqt = p->ldqt ? p->ldqt : p->rows;
    a.x = p->x;
    return KDA_OK;
}

kda_status mm8_args(const kda_mm8_problem* p, kda::Mm8Args& a) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "problem is NULL");
    a = kda::Mm8Args{};
    if (p->M < 0 || p->N < 1 || p->K < 1) return fail(KDA_ERR_INVALID_ARG, "M must be >= 0, N and K >= 1");
    if (p->M > MAX_ROWS || p->N > MAX_COLS || p->K > MAX_ROWS)   // (the columns of a transposed copy are its rows)
        return fail(KDA_ERR_UNSUPPORTED, "more than 2^22 rows of a or columns, or 2^20 rows of b");
    if (p->out != KDA_BF16 && p->out != KDA_FP32) return fail(KDA_ERR_INVALID_ARG, "unknown output dtype");
    if (p->b_rows != 0 && p->b_rows != 1) return fail(KDA_ERR_INVALID_ARG, "b_rows must be 0 or 1");
    if ((p->lda && p->lda < p->K) || (p->ldb && p->ldb < p->K))
        return fail(KDA_ERR_INVALID_ARG, "a leading dimension is shorter than its row");
    a.M = p->M;
    a.N = p->N;
    a.K = p->K;
    a.groups = (p->K + kda::FP8_GROUP - 1) / kda::FP8_GROUP;
    a.b_rows = p->b_rows;
    a.f32 = p->out == KDA_FP32;
    a.lda = p->lda ? p->lda : p->K;
    a.ldb = p->ldb ? p->ldb : p->K;
    a.a = static_cast<const uint8_t*>(p->a);
    a.b = static_cast<const uint8_t*>(p->b);
    a.sa = p->scale_a;
    a.sb = p->scale_b;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_quant8(const kda_quant8_problem* p, void* q, float* scale, void* qt, float* scale_t, kda_stream_t stream) {
    kda::Quant8Args a;
    const kda_status st = quant8_args(p, a);
    if (st != KDA_OK || a.rows == 0) return st;
    if (!q && !qt) return fail(KDA_ERR_INVALID_ARG, "one of q and qt must be non-NULL");
    if ((q != nullptr) != (scale != nullptr) || (qt != nullptr) != (scale_t != nullptr))
        return fail(KDA_ERR_INVALID_ARG, "q comes with scale, qt with scale_t");
    if (!a.x) return fail(KDA_ERR_INVALID_ARG, "x must be non-NULL");
    a.q = static_cast<uint8_t*>(q);
    a.scale = scale;
    a.qt = static_cast<uint8_t*>(qt);
    a.scale_t = scale_t;
    return cuda_result(kda::launch_quant8(a, p->io == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)), "rounding to 8 bits");
}

size_t kda_mm8_workspace_size(const kda_mm8_problem* p) {
    kda::Mm8Args a;
    return mm8_args(p, a) == KDA_OK ? up(kda::mm8_align_bytes(a)) : 0;
}

kda_status kda_mm8(const kda_mm8_problem* p, void* y, void* ws, size_t ws_bytes, int32_t* err, kda_stream_t stream) {
    kda::Mm8Args a;
    kda_status st = mm8_args(p, a);
    if (st != KDA_OK) return st;
    if (a.M == 0) return KDA_OK;
    if (!a.a || !a.b || !a.sa || !a.sb || !y) return fail(KDA_ERR_INVALID_ARG, "a, b, their scales and y must be non-NULL");
    if ((st = check_ws(ws, ws_bytes, kda_mm8_workspace_size(p), "workspace")) != KDA_OK) return st;
    a.y = y;
    a.err = err;
    return cuda_result(kda::launch_mm8(a, ws, reinterpret_cast<cudaStream_t>(stream)), "8-bit product");
}

}  // extern "C"
