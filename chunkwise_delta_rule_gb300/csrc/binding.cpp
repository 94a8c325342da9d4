// Python binding of the layer operators (include/kda.h): argument checks, output
// allocation and the call, in one step each. A decoding step takes a few
// microseconds on the device; the same marshalling written in Python takes 10 to
// 20 microseconds of host time per call and bounds it.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <climits>
#include <optional>

#include "../../include/kda.h"

namespace py = pybind11;
using at::Tensor;
using OptT = std::optional<Tensor>;

namespace {

void need(bool ok, const char* msg) {
    if (!ok) throw py::value_error(msg);
}
// A size as the C interface holds it.
int size(int64_t v, const char* name) {
    if (v < INT_MIN || v > INT_MAX) throw py::value_error(std::string(name) + " is beyond 32 bits");
    return (int)v;
}
[[noreturn]] void refuse(const char* name, const char* what, at::IntArrayRef shape, at::ScalarType type) {
    std::ostringstream s;
    s << name << " must be a " << what << "CUDA tensor " << shape << ", " << type;
    throw py::value_error(s.str());
}
// Every tensor of a call lies on one device, x's.
void same_device(const Tensor& t, const char* name, const Tensor& x) {
    if (t.device() != x.device()) throw py::value_error(std::string(name) + " must be on x's device");
}

// An io type's kda_dtype.
kda_dtype io_of(const Tensor& t, const char* msg) {
    const at::ScalarType s = t.scalar_type();
    need(s == at::kBFloat16 || s == at::kFloat, msg);
    return s == at::kBFloat16 ? KDA_BF16 : KDA_FP32;
}

void* dense(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, const Tensor& x) {
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_cuda() || !t.is_contiguous()) refuse(name, "contiguous ", shape, type);
    same_device(t, name, x);
    return t.data_ptr();
}
void* dense(const OptT& t, const char* name, at::IntArrayRef shape, at::ScalarType type, const Tensor& x) {
    return t ? dense(*t, name, shape, type, x) : nullptr;
}
float* f32(const OptT& t, const char* name, at::IntArrayRef shape, const Tensor& x) {
    return static_cast<float*>(dense(t, name, shape, at::kFloat, x));
}

// Checks a [B, T, ...] input and returns the elements between its tokens (0: contiguous).
int64_t rows(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, const Tensor& x) {
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_cuda()) refuse(name, "", shape, type);
    same_device(t, name, x);
    if (t.is_contiguous()) return 0;
    int64_t width = 1;
    for (int64_t i = (int64_t)shape.size() - 1; i >= 2; --i) {
        if (shape[i] != 1 && t.stride(i) != width) throw py::value_error(std::string(name) + "'s rows must be dense");
        width *= shape[i];
    }
    const int64_t B = shape[0], T = shape[1];
    const int64_t ld = T > 1 ? t.stride(1) : B > 1 ? t.stride(0) : width;
    if (ld < width || (B > 1 && T > 1 && t.stride(0) != T * ld)) throw py::value_error(std::string(name) + "'s tokens must be evenly spaced");
    return ld;
}

// Sequences; packed ones' count and offsets.
int64_t axis(const OptT& cu, int64_t B, int& N, const int32_t*& p, const Tensor& x) {
    N = 0;
    p = nullptr;
    if (!cu) return B;
    need(cu->scalar_type() == at::kInt && cu->is_cuda() && cu->dim() == 1 && cu->is_contiguous() && cu->numel() >= 2,
         "cu_seqlens must be an int32 CUDA vector");
    same_device(*cu, "cu_seqlens", x);
    need(B == 1, "packed sequences need B == 1");
    N = size(cu->numel() - 1, "the number of sequences");
    p = cu->data_ptr<int32_t>();
    return N;
}
int32_t* error_word(const OptT& err, const Tensor& x) {
    if (!err) return nullptr;
    need(err->scalar_type() == at::kInt && err->is_cuda() && err->numel() >= 1, "err must be an int32 CUDA tensor");
    same_device(*err, "err", x);
    return err->data_ptr<int32_t>();
}
// The device of a call, x's, and its stream: the current one, or one the caller names. A named one is current while the
// call allocates, so that a block's earlier users, and the later ones of a workspace dropped at the call's end, are
// ordered with its kernels. What the two sides hand each other is recorded, so that its memory waits for both when it
// is freed.
class OnStream {
    c10::cuda::OptionalCUDAGuard device_;   // unset where x's device is the current one already
    c10::cuda::CUDAStream caller_, mine_;
    c10::cuda::OptionalCUDAStreamGuard guard_;
    bool other_ = false;
    void record(const Tensor& t, const c10::cuda::CUDAStream& s) {
        if (other_ && t.is_cuda() && t.numel()) t.record_stream(s.unwrap());
    }

public:
    OnStream(const py::object& stream, const Tensor& x)
        : caller_(c10::cuda::getCurrentCUDAStream(x.get_device())), mine_(caller_) {
        if (c10::cuda::current_device() != x.get_device()) device_.set_device(x.device());
        if (stream.is_none()) return;
        if (py::hasattr(stream, "device_index"))
            need(stream.attr("device_index").cast<int>() == x.get_device(), "stream must be on x's device");
        const auto handle = reinterpret_cast<cudaStream_t>(stream.attr("cuda_stream").cast<uintptr_t>());
        if (handle == caller_.stream()) return;
        other_ = true;
        mine_ = c10::cuda::getStreamFromExternal(handle, x.get_device());
        guard_.reset_stream(mine_);
    }
    operator kda_stream_t() const { return reinterpret_cast<kda_stream_t>(mine_.stream()); }
    // Tensors of the caller's that the kernels use, and tensors made here that the caller gets.
    template <class... T>
    void takes(const T&... t) { (each(t, mine_), ...); }
    template <class... T>
    void gives(const T&... t) { (each(t, caller_), ...); }

private:
    void each(const Tensor& t, const c10::cuda::CUDAStream& s) { record(t, s); }
    void each(const OptT& t, const c10::cuda::CUDAStream& s) {
        if (t) record(*t, s);
    }
};
void check(kda_status st, const char* where) {
    if (st != KDA_OK) py::module_::import("chunkwise_delta_rule_gb300._lib").attr("check")((int)st, where);
}
Tensor like(const Tensor& t) { return at::empty(t.sizes(), t.options()); }
OptT like(const OptT& t) { return t ? OptT(like(*t)) : OptT(); }
void* ptr(const OptT& t) { return t ? t->data_ptr() : nullptr; }
size_t bytes(const OptT& t) { return t ? t->nbytes() : 0; }
// The given buffer if it is large enough, else a new one (nothing for no bytes).
OptT buffer(size_t n, const char* name, const Tensor& x, const OptT& given) {
    if (given) {
        if (!given->is_cuda() || !given->is_contiguous()) throw py::value_error(std::string(name) + " must be a contiguous CUDA tensor");
        same_device(*given, name, x);
    }
    if (n == 0 || (given && given->nbytes() >= n)) return given;
    return at::empty({(int64_t)n}, x.options().dtype(at::kByte));
}

// ------------------------------------------------------------------ convolution
struct Conv {
    kda_conv_problem c{};
    Tensor x, weight;
    OptT bias, h0, cu;
    std::vector<int64_t> state;
    Conv(Tensor x_, Tensor w, OptT b, bool silu, OptT h, OptT cu_) : x(x_), weight(w), bias(b), h0(h), cu(cu_) {
        need(x.dim() == 3, "x must be [B, T, D], bf16 or fp32");
        c.io = io_of(x, "x must be [B, T, D], bf16 or fp32");
        need(weight.dim() == 2, "weight must be [D, W]");
        const int64_t B = x.size(0), T = x.size(1), D = x.size(2), W = weight.size(1);
        c.B = size(B, "B"); c.T = size(T, "T"); c.D = size(D, "D"); c.W = size(W, "W");
        c.ldx = rows(x, "x", x.sizes(), x.scalar_type(), x);
        const int64_t n = axis(cu, B, c.N, c.cu_seqlens, x);
        state = {n, W - 1, D};
        c.silu = silu;
        c.x = x.data_ptr();
        c.weight = static_cast<float*>(dense(weight, "weight", {D, W}, at::kFloat, x));
        c.bias = f32(bias, "bias", {D}, x);
        c.h0 = dense(h0, "initial_state", state, x.scalar_type(), x);
    }
};
py::tuple conv_fwd(const Conv& p, bool out_final, OptT final_state, OptT err, py::object stream) {
    OnStream on(stream, p.x);
    on.takes(p.x, p.weight, p.bias, p.h0, p.cu, final_state, err);
    Tensor y = like(p.x);
    if (!final_state && out_final) final_state = at::empty(p.state, p.x.options());
    void* f = dense(final_state, "final_state", p.state, p.x.scalar_type(), p.x);
    check(kda_conv_fwd(&p.c, y.data_ptr(), f, error_word(err, p.x), on), "kda_conv_fwd");
    on.gives(y, final_state);
    return py::make_tuple(y, final_state);
}
py::tuple conv_bwd(const Conv& p, Tensor dy, OptT dfinal, OptT ws, py::object stream, std::optional<bool> need_dinit) {
    OnStream on(stream, p.x);
    on.takes(p.x, p.weight, p.bias, p.h0, p.cu, dy, dfinal, ws);
    void* pdy = dense(dy, "dy", p.x.sizes(), p.x.scalar_type(), p.x);
    void* pdf = dense(dfinal, "dfinal", p.state, p.x.scalar_type(), p.x);
    Tensor dx = like(p.x), dw = like(p.weight);
    OptT db = like(p.bias), dinit;
    if (need_dinit ? *need_dinit : p.h0.has_value()) dinit = at::empty(p.state, p.x.options());
    ws = buffer(kda_conv_workspace_size(&p.c), "workspace", p.x, ws);
    check(kda_conv_bwd(&p.c, pdy, pdf, dx.data_ptr(), dw.data_ptr<float>(), static_cast<float*>(ptr(db)), ptr(dinit), ptr(ws),
                       bytes(ws), on), "kda_conv_bwd");
    on.gives(dx, dw, db, dinit);
    return py::make_tuple(dx, dw, db, dinit);
}

// ------------------------------------------------------------------ scan
struct Ssm {
    kda_ssm_problem c{};
    Tensor x, dt, A_log, b, cm;
    OptT d_skip, z, dt_bias, h0, cu;
    std::vector<int64_t> state;
    Ssm(Tensor x_, Tensor dt_, Tensor A, Tensor b_, Tensor c_, OptT skip, OptT z_, OptT bias, bool softplus, OptT h, OptT cu_, int save)
        : x(x_), dt(dt_), A_log(A), b(b_), cm(c_), d_skip(skip), z(z_), dt_bias(bias), h0(h), cu(cu_) {
        need(x.dim() == 3, "x must be [B, T, D], bf16 or fp32");
        c.io = io_of(x, "x must be [B, T, D], bf16 or fp32");
        need(b.dim() == 4, "b must be [B, T, G, S]");
        const int64_t B = x.size(0), T = x.size(1), D = x.size(2), G = b.size(2), S = b.size(3);
        const at::ScalarType type = x.scalar_type();
        const std::array<int64_t, 4> bc{B, T, G, S};
        c.B = size(B, "B"); c.T = size(T, "T"); c.D = size(D, "D"); c.S = size(S, "S"); c.G = size(G, "G");
        const int64_t n = axis(cu, B, c.N, c.cu_seqlens, x);
        state = {n, D, S};
        c.dt_softplus = softplus;
        c.save_policy = save;
        c.ldx = rows(x, "x", x.sizes(), type, x);
        c.lddt = rows(dt, "dt", x.sizes(), type, x);
        if (z) c.ldz = rows(*z, "z", x.sizes(), type, x);
        c.ldb = rows(b, "b", bc, type, x);
        c.ldc = rows(cm, "c", bc, type, x);
        c.x = x.data_ptr();
        c.dt = dt.data_ptr();
        c.z = ptr(z);
        c.b = b.data_ptr();
        c.c = cm.data_ptr();
        c.A_log = static_cast<float*>(dense(A_log, "A_log", {D, S}, at::kFloat, x));
        c.d_skip = f32(d_skip, "d_skip", {D}, x);
        c.dt_bias = f32(dt_bias, "dt_bias", {D}, x);
        c.h0 = f32(h0, "initial_state", state, x);
    }
};
py::tuple ssm_fwd(const Ssm& p, bool out_final, OptT ht, OptT saved, OptT ws, OptT err, py::object stream) {
    OnStream on(stream, p.x);
    on.takes(p.x, p.dt, p.A_log, p.b, p.cm, p.d_skip, p.z, p.dt_bias, p.h0, p.cu, ht, saved, ws, err);
    Tensor y = like(p.x);
    if (!ht && out_final) ht = at::empty(p.state, p.x.options().dtype(at::kFloat));
    float* h = f32(ht, "ht", p.state, p.x);
    ws = buffer(kda_ssm_workspace_size(&p.c, 0), "workspace", p.x, ws);
    OptT sv = p.c.save_policy ? buffer(kda_ssm_saved_size(&p.c), "saved", p.x, saved) : OptT();
    check(kda_ssm_fwd(&p.c, y.data_ptr(), h, ptr(sv), ptr(ws), bytes(ws), error_word(err, p.x), on), "kda_ssm_fwd");
    on.gives(y, ht, sv);
    return py::make_tuple(y, ht, sv);
}
py::tuple ssm_bwd(const Ssm& p, Tensor dy, OptT dht, OptT saved, OptT ws, py::object stream, std::optional<bool> need_dh0, OptT err) {
    OnStream on(stream, p.x);
    on.takes(p.x, p.dt, p.A_log, p.b, p.cm, p.d_skip, p.z, p.dt_bias, p.h0, p.cu, dy, dht, saved, ws, err);
    void* pdy = dense(dy, "dy", p.x.sizes(), p.x.scalar_type(), p.x);
    float* pdh = f32(dht, "dht", p.state, p.x);
    if (p.c.save_policy) {
        need(bytes(saved) >= kda_ssm_saved_size(&p.c), "save_policy 1 needs the forward's saved buffer");
        saved = buffer(0, "saved", p.x, saved);
    } else {
        saved = OptT();
    }
    Tensor dx = like(p.x), ddt = like(p.dt), dA = like(p.A_log), db = like(p.b), dc = like(p.cm);
    OptT dskip = like(p.d_skip), dz = like(p.z), dbias = like(p.dt_bias), dh0;
    if (need_dh0 ? *need_dh0 : p.h0.has_value()) dh0 = at::empty(p.state, p.x.options().dtype(at::kFloat));
    kda_ssm_grads g{};
    g.dx = dx.data_ptr();
    g.ddt = ddt.data_ptr();
    g.dz = ptr(dz);
    g.db = db.data_ptr();
    g.dc = dc.data_ptr();
    g.dA_log = dA.data_ptr<float>();
    g.dd_skip = static_cast<float*>(ptr(dskip));
    g.ddt_bias = static_cast<float*>(ptr(dbias));
    g.dh0 = static_cast<float*>(ptr(dh0));
    ws = buffer(kda_ssm_workspace_size(&p.c, 1), "workspace", p.x, ws);
    check(kda_ssm_bwd_err(&p.c, pdy, pdh, ptr(saved), &g, ptr(ws), bytes(ws), error_word(err, p.x), on), "kda_ssm_bwd");
    on.gives(dx, ddt, dA, db, dc, dskip, dz, dbias, dh0);
    return py::make_tuple(dx, ddt, dA, db, dc, dskip, dz, dbias, dh0);
}

// ------------------------------------------------------------------ norm
struct Norm {
    kda_norm_problem c{};
    Tensor x, weight;
    OptT residual;
    std::vector<int64_t> scales;   // shape of the scales of an 8-bit output
    Norm(Tensor x_, Tensor w, OptT r, double eps, const std::string& out, int64_t group) : x(x_), weight(w), residual(r) {
        need(x.dim() >= 1, "x must be bf16 or fp32 rows");
        c.io = io_of(x, "x must be bf16 or fp32 rows");
        need(out == "io" || out == "e4m3", "out must be \"io\" or \"e4m3\"");
        const int64_t D = x.size(-1);
        c.rows = D ? size(x.numel() / D, "the number of rows") : 0;
        c.D = size(D, "D");
        c.out = out == "e4m3";
        c.group = size(group, "group");
        c.eps = (float)eps;
        c.x = dense(x, "x", x.sizes(), x.scalar_type(), x);
        c.residual = dense(residual, "residual", x.sizes(), x.scalar_type(), x);
        c.weight = static_cast<float*>(dense(weight, "weight", {D}, at::kFloat, x));
        if (c.out) {
            scales.assign(x.sizes().begin(), x.sizes().end());
            scales.back() = group > 0 ? (D + group - 1) / group : 1;
        }
    }
};
py::tuple norm_fwd(const Norm& p, OptT h, py::object stream) {
    OnStream on(stream, p.x);
    on.takes(p.x, p.weight, p.residual, h);
    Tensor y = p.c.out ? at::empty(p.x.sizes(), p.x.options().dtype(at::kFloat8_e4m3fn)) : like(p.x);
    OptT scale;
    if (p.c.out) scale = at::empty(p.scales, p.x.options().dtype(at::kFloat));
    if (!p.residual) h = p.x;
    else if (!h) h = like(p.x);
    else dense(h, "h", p.x.sizes(), p.x.scalar_type(), p.x);
    check(kda_norm_fwd(&p.c, y.data_ptr(), static_cast<float*>(ptr(scale)), h->data_ptr(), on), "kda_norm_fwd");
    on.gives(y, scale, h);
    return py::make_tuple(y, scale, h);
}
py::tuple norm_bwd(const Norm& p, Tensor dy, OptT dres, OptT ws, py::object stream) {
    OnStream on(stream, p.x);
    on.takes(p.x, p.weight, dy, dres, ws);
    void* pdy = dense(dy, "dy", p.x.sizes(), p.x.scalar_type(), p.x);
    void* pdr = dense(dres, "dres", p.x.sizes(), p.x.scalar_type(), p.x);
    Tensor dx = like(p.x), dw = like(p.weight);
    ws = buffer(kda_norm_workspace_size(&p.c), "workspace", p.x, ws);
    check(kda_norm_bwd(&p.c, pdy, pdr, dx.data_ptr(), dw.data_ptr<float>(), ptr(ws), bytes(ws), on), "kda_norm_bwd");
    on.gives(dx, dw);
    return py::make_tuple(dx, dw);
}

}  // namespace

PYBIND11_MODULE(_binding, m) {
    m.doc() = "Argument checks and calls of the layer operators; see layer.py for their documentation.";
    py::class_<Conv>(m, "ConvProblem", "A validated convolution call plus the tensors it points to.")
        .def(py::init<Tensor, Tensor, OptT, bool, OptT, OptT>())
        .def_readonly("x", &Conv::x)
        .def_readonly("state_shape", &Conv::state);
    py::class_<Ssm>(m, "SsmProblem", "A validated scan call plus the tensors it points to.")
        .def(py::init<Tensor, Tensor, Tensor, Tensor, Tensor, OptT, OptT, OptT, bool, OptT, OptT, int>())
        .def_readonly("x", &Ssm::x)
        .def_readonly("state_shape", &Ssm::state);
    py::class_<Norm>(m, "NormProblem", "A validated norm call plus the tensors it points to.")
        .def(py::init<Tensor, Tensor, OptT, double, const std::string&, int64_t>())
        .def_readonly("x", &Norm::x);
    m.def("conv_fwd", &conv_fwd);
    m.def("conv_bwd", &conv_bwd);
    m.def("conv_workspace_size", [](const Conv& p) {
        const c10::cuda::CUDAGuard device(p.x.device());   // sizes go by the device's SMs
        return kda_conv_workspace_size(&p.c);
    });
    m.def("ssm_fwd", &ssm_fwd);
    m.def("ssm_bwd", &ssm_bwd);
    m.def("ssm_workspace_size", [](const Ssm& p, bool backward) {
        const c10::cuda::CUDAGuard device(p.x.device());
        return kda_ssm_workspace_size(&p.c, backward);
    });
    m.def("ssm_saved_size", [](const Ssm& p) { return kda_ssm_saved_size(&p.c); });
    m.def("norm_fwd", &norm_fwd);
    m.def("norm_bwd", &norm_bwd);
    m.def("norm_workspace_size", [](const Norm& p) {
        const c10::cuda::CUDAGuard device(p.x.device());
        return kda_norm_workspace_size(&p.c);
    });
}
