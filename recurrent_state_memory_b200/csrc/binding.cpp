// binding.cpp -- host side of the Python calls of the scan, the layer norm, the beam selection and the
// state reorder: checks of the tensors, outputs, descriptors, the C call of include/gdr.h on the
// tensors' device and stream.  These calls' kernels take a few microseconds at serving sizes, as
// long as a handful of Python statements; the same steps in Python cost 8 to 17 us a call.
#include <dlfcn.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/extension.h>

#include "gdr.h"

namespace {

using at::Tensor;
using MaybeTensor = std::optional<Tensor>;

// The library's entry points, of the file that gdr.lib() has loaded.
struct Api {
    decltype(&gdr_scan_fwd) scan_fwd;
    decltype(&gdr_scan_bwd) scan_bwd;
    decltype(&gdr_scan_step) scan_step;
    decltype(&gdr_layernorm_fwd) layernorm_fwd;
    decltype(&gdr_layernorm_bwd) layernorm_bwd;
    decltype(&gdr_layernorm_bwd_workspace_bytes) layernorm_bwd_workspace_bytes;
    decltype(&gdr_beam_select) beam_select;
    decltype(&gdr_beam_select_workspace_bytes) beam_select_workspace_bytes;
    decltype(&gdr_state_reorder) state_reorder;
} api;

template <typename F> void resolve(void* lib, F& f, const char* name) {
    f = reinterpret_cast<F>(dlsym(lib, name));
    if (!f) throw std::runtime_error(std::string("the library has no ") + name);
}

void load(const std::string& path) {
    void* lib = dlopen(path.c_str(), RTLD_NOW | RTLD_LOCAL);
    if (!lib) throw std::runtime_error(dlerror());
    resolve(lib, api.scan_fwd, "gdr_scan_fwd");
    resolve(lib, api.scan_bwd, "gdr_scan_bwd");
    resolve(lib, api.scan_step, "gdr_scan_step");
    resolve(lib, api.layernorm_fwd, "gdr_layernorm_fwd");
    resolve(lib, api.layernorm_bwd, "gdr_layernorm_bwd");
    resolve(lib, api.layernorm_bwd_workspace_bytes, "gdr_layernorm_bwd_workspace_bytes");
    resolve(lib, api.beam_select, "gdr_beam_select");
    resolve(lib, api.beam_select_workspace_bytes, "gdr_beam_select_workspace_bytes");
    resolve(lib, api.state_reorder, "gdr_state_reorder");
}

// gdr.GdrError with the library's detail.
void check(gdr_status s, const char* where) {
    if (s != GDR_OK) py::module_::import("recurrent_state_memory_b200.gdr").attr("_check")(static_cast<int>(s), where);
}

std::string str(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}
std::string str(at::ScalarType t) { return "torch." + std::string(t == at::kFloat ? "float32" : t == at::kBFloat16 ? "bfloat16" : t == at::kInt ? "int32" : t == at::kBool ? "bool" : at::toString(t)); }

gdr_dtype code(at::ScalarType t) {
    if (t == at::kBFloat16) return GDR_BF16;
    if (t == at::kFloat) return GDR_F32;
    throw py::type_error("unsupported dtype " + str(t) + " (bf16 or fp32)");
}

void on_gpu(const Tensor& t, const char* name) {
    if (!t.is_cuda()) throw py::value_error(std::string(name) + " must be a CUDA tensor");
}
void dense(const Tensor& t, const char* name) {
    if (!t.is_contiguous()) throw py::value_error(std::string(name) + " must be contiguous");
}
void on(const Tensor& t, const char* name, at::Device dev) {
    if (t.device() != dev) throw py::value_error(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
}
// Contiguous, on dev, of this shape and (unless Undefined) type.
void want(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    dense(t, name);
    if (type != at::ScalarType::Undefined && t.scalar_type() != type)
        throw py::type_error(std::string(name) + " must be " + str(type) + ", got " + str(t.scalar_type()));
    on(t, name, dev);
    if (t.sizes() != shape) throw py::value_error(std::string(name) + " must have the shape " + str(shape) + ", got " + str(t.sizes()));
}
void want(const MaybeTensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    if (t) want(*t, name, shape, type, dev);
}

// Its bytes are the memory that it has: an expanded or strided tensor has less, or other.
void want_workspace(const MaybeTensor& t, at::Device dev) {
    if (!t) return;
    dense(*t, "workspace");
    on(*t, "workspace", dev);
}

// Elements between the rows of t (dense: 0), whose rows are dense and evenly spaced (a slice along the
// last dimension of a wider contiguous tensor is).  What a dimension of one has for a stride is nothing.
int64_t row_stride(const Tensor& t, const char* name) {
    if (t.is_contiguous()) return 0;
    const auto st = t.strides(), sh = t.sizes();
    const int64_t n = t.dim();
    bool ok = n >= 2 && (st[n - 1] == 1 || sh[n - 1] == 1);
    int64_t row = -1, next = 0;             // the rows' distance, once known, and what the next dimension outwards must have
    for (int64_t d = n - 2; ok && d >= 0; --d) {
        if (sh[d] == 1) continue;
        if (row < 0) row = next = st[d];
        ok = st[d] == next;
        next *= sh[d];
    }
    if (!ok || row < sh[n - 1])
        throw py::value_error(std::string(name) + " must be contiguous, or a slice of a contiguous tensor along its last dimension");
    return row;
}

// A call: its device, current while this lives, and its stream, the given one or the current one.  With
// a given stream, memory is allocated on it (nothing that is queued on the current one uses it
// still), and none of the call's tensors gives its memory away before that stream, and for outputs
// the current one, are done with it.
class Call {
public:
    gdr_stream_t stream;
    Call(at::Device dev, const py::object& given)
        : dev_(dev), device_(dev), here_(c10::cuda::getCurrentCUDAStream(dev.index())) {
        stream = reinterpret_cast<void*>(here_.stream());
        if (given.is_none()) return;
        stream = reinterpret_cast<void*>(given.attr("cuda_stream").cast<intptr_t>());
        if (stream == reinterpret_cast<void*>(here_.stream())) return;
        there_.emplace(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(stream), dev.index()));
    }
    // The caller's tensors of the call.
    template <typename... T> void uses(const T&... t) const { if (there_) (used_on(t, there_->current_stream()), ...); }
    Tensor scratch(at::IntArrayRef shape, at::ScalarType type) const {
        return at::detail::empty_cuda(shape, type, dev_, std::nullopt);
    }
    Tensor output(at::IntArrayRef shape, at::ScalarType type) const {
        Tensor t = scratch(shape, type);
        if (there_) used_on(t, here_);
        return t;
    }

private:
    static void used_on(const Tensor& t, c10::Stream s) {
        c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), c10::cuda::CUDAStream(s));
    }
    static void used_on(const MaybeTensor& t, c10::Stream s) { if (t) used_on(*t, s); }
    const at::Device dev_;
    const c10::cuda::CUDAGuard device_;
    const c10::cuda::CUDAStream here_;
    std::optional<c10::cuda::CUDAStreamGuard> there_;
};

template <typename T = void> T* at_(const MaybeTensor& t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }
template <typename T = void> T* at_(const Tensor& t) { return static_cast<T*>(t.data_ptr()); }

at::ScalarType dtype_of(const py::object& d, at::ScalarType otherwise) {
    if (d.is_none()) return otherwise;
    if (!THPDtype_Check(d.ptr())) throw py::type_error("out_dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype*>(d.ptr())->scalar_type;
}

int size32(int64_t n, const char* name) {
    if (n > INT32_MAX) throw py::value_error(std::string(name) + " is too large");
    return static_cast<int>(n);
}

// ---------------------------------------------------------------- scan ----

at::Device scan_check(const Tensor& x, const Tensor& g, int64_t dims, const MaybeTensor& lengths) {
    on_gpu(x, "x");
    if (x.dim() != dims || g.sizes() != x.sizes())
        throw py::value_error(dims == 3 ? "x and g must have the same shape, [B, T, D]" : "x and g must have the same shape, [N, D]");
    on(g, "g", x.device());
    want(lengths, "lengths", {x.size(0)}, at::kInt, x.device());
    return x.device();
}

gdr_scan_desc scan_desc(const Tensor& x, const Tensor& g, int64_t T, at::ScalarType out, int gate_mode, bool tied) {
    gdr_scan_desc d;
    d.B = size32(x.size(0), "B"); d.T = size32(T, "T"); d.D = size32(x.size(-1), "D");
    d.x_row = row_stride(x, "x"); d.g_row = row_stride(g, "g");
    d.x_dtype = code(x.scalar_type()); d.g_dtype = code(g.scalar_type()); d.out_dtype = code(out);
    d.gate_mode = static_cast<gdr_gate_mode>(gate_mode); d.tied = tied;
    return d;
}

py::tuple scan_fwd(const Tensor& x, const Tensor& g, const MaybeTensor& h0, int gate_mode, bool tied,
                   const MaybeTensor& lengths, const py::object& out_dtype, bool want_state, bool want_ckpt,
                   const py::object& stream) {
    const at::Device dev = scan_check(x, g, 3, lengths);
    const int64_t B = x.size(0), T = x.size(1), D = x.size(2);
    want(h0, "h0", {B, D}, at::kFloat, dev);
    const at::ScalarType out = dtype_of(out_dtype, x.scalar_type());
    const gdr_scan_desc d = scan_desc(x, g, T, out, gate_mode, tied);
    const Call call(dev, stream);
    call.uses(x, g, h0, lengths);
    Tensor h = call.output({B, T, D}, out);
    MaybeTensor h_T, ckpt;
    if (want_state) h_T = call.output({B, D}, at::kFloat);
    if (want_ckpt) ckpt = call.output({B, (T + GDR_SCAN_CKPT - 1) / GDR_SCAN_CKPT, D}, at::kFloat);
    check(api.scan_fwd(&d, at_(x), at_(g), at_<float>(h0), at_<int>(lengths), at_(h), at_<float>(h_T), at_<float>(ckpt),
                       call.stream), "gdr_scan_fwd");
    return want_ckpt ? py::make_tuple(h, h_T, ckpt) : py::make_tuple(h, h_T);
}

py::dict scan_bwd(const Tensor& x, const Tensor& g, const Tensor& ckpt, const MaybeTensor& dh, const MaybeTensor& dh_T,
                  int gate_mode, bool tied, const MaybeTensor& lengths, bool want_dh0, const py::object& stream) {
    const at::Device dev = scan_check(x, g, 3, lengths);
    const int64_t B = x.size(0), T = x.size(1), D = x.size(2);
    want(ckpt, "ckpt", {B, (T + GDR_SCAN_CKPT - 1) / GDR_SCAN_CKPT, D}, at::kFloat, dev);
    want(dh, "dh", {B, T, D}, at::ScalarType::Undefined, dev);
    want(dh_T, "dh_T", {B, D}, at::kFloat, dev);
    const gdr_scan_desc d = scan_desc(x, g, T, dh ? dh->scalar_type() : x.scalar_type(), gate_mode, tied);
    const Call call(dev, stream);
    call.uses(x, g, ckpt, dh, dh_T, lengths);
    Tensor dx = call.output({B, T, D}, x.scalar_type()), dg = call.output({B, T, D}, g.scalar_type());
    MaybeTensor dh0;
    if (want_dh0) dh0 = call.output({B, D}, at::kFloat);
    check(api.scan_bwd(&d, at_(x), at_(g), at_<float>(ckpt), at_<int>(lengths), at_(dh), at_<float>(dh_T), at_(dx),
                       at_(dg), at_<float>(dh0), call.stream), "gdr_scan_bwd");
    py::dict r;
    r["x"] = dx; r["g"] = dg; r["h0"] = dh0;
    return r;
}

Tensor scan_step(const Tensor& x, const Tensor& g, const Tensor& h, int gate_mode, bool tied, const py::object& out_dtype,
                 const MaybeTensor& o, const py::object& stream) {
    const at::Device dev = scan_check(x, g, 2, {});
    want(h, "h", x.sizes(), at::kFloat, dev);
    const at::ScalarType out = dtype_of(out_dtype, x.scalar_type());
    want(o, "o", x.sizes(), out, dev);
    const gdr_scan_desc d = scan_desc(x, g, 1, out, gate_mode, tied);
    const Call call(dev, stream);
    call.uses(x, g, h, o);
    const Tensor to = o ? *o : call.output(x.sizes(), out);
    check(api.scan_step(&d, at_(x), at_(g), at_<float>(h), at_(to), call.stream), "gdr_scan_step");
    return to;
}

// ---------------------------------------------------------- layer norm ----

gdr_norm_desc norm_desc(const Tensor& x, at::ScalarType y, const MaybeTensor& weight, const MaybeTensor& bias, double eps) {
    on_gpu(x, "x");
    if (x.dim() < 1) throw py::value_error("x must have at least one dimension");
    dense(x, "x");
    const int64_t D = x.size(-1);
    const at::ScalarType w = weight ? weight->scalar_type() : bias ? bias->scalar_type() : at::kFloat;
    want(weight, "weight", {D}, w, x.device());
    want(bias, "bias", {D}, w, x.device());
    gdr_norm_desc d;
    d.rows = D ? x.numel() / D : 0; d.D = size32(D, "D");
    d.x_dtype = code(x.scalar_type()); d.y_dtype = code(y); d.w_dtype = code(w);
    d.eps = static_cast<float>(eps);
    return d;
}

py::tuple layernorm_fwd(const Tensor& x, const MaybeTensor& weight, const MaybeTensor& bias, double eps,
                        const py::object& out_dtype, bool want_stats, const py::object& stream) {
    const at::ScalarType out = dtype_of(out_dtype, x.scalar_type());
    const gdr_norm_desc d = norm_desc(x, out, weight, bias, eps);
    const at::Device dev = x.device();
    const Call call(dev, stream);
    call.uses(x, weight, bias);
    Tensor y = call.output(x.sizes(), out);
    MaybeTensor mean, rstd;
    if (want_stats) {
        mean = call.output(x.sizes().slice(0, x.dim() - 1), at::kFloat);
        rstd = call.output(x.sizes().slice(0, x.dim() - 1), at::kFloat);
    }
    check(api.layernorm_fwd(&d, at_(x), at_(weight), at_(bias), at_(y), at_<float>(mean), at_<float>(rstd), call.stream),
          "gdr_layernorm_fwd");
    return py::make_tuple(y, mean, rstd);
}

py::dict layernorm_bwd(const Tensor& x, const Tensor& dy, const Tensor& mean, const Tensor& rstd, const MaybeTensor& weight,
                       bool with_bias, bool want_dx, const MaybeTensor& workspace, const py::object& stream) {
    const gdr_norm_desc d = norm_desc(x, dy.scalar_type(), weight, {}, 0.0);
    const at::Device dev = x.device();
    const auto rows = x.sizes().slice(0, x.dim() - 1);
    want(dy, "dy", x.sizes(), at::ScalarType::Undefined, dev);
    want(mean, "mean", rows, at::kFloat, dev);
    want(rstd, "rstd", rows, at::kFloat, dev);
    want_workspace(workspace, dev);
    const Call call(dev, stream);
    call.uses(x, dy, mean, rstd, weight, workspace);
    MaybeTensor dx, dw, db;
    if (want_dx) dx = call.output(x.sizes(), x.scalar_type());
    if (weight) dw = call.output({x.size(-1)}, at::kFloat);
    if (with_bias) db = call.output({x.size(-1)}, at::kFloat);
    const size_t need = api.layernorm_bwd_workspace_bytes(&d, dw.has_value(), with_bias);
    const MaybeTensor ws = workspace ? workspace : need ? MaybeTensor(call.scratch({static_cast<int64_t>(need)}, at::kByte)) : MaybeTensor();
    check(api.layernorm_bwd(&d, at_(x), at_(dy), at_(weight), at_<float>(mean), at_<float>(rstd), at_(dx), at_<float>(dw),
                            at_<float>(db), at_(ws), ws ? ws->nbytes() : 0, call.stream), "gdr_layernorm_bwd");
    py::dict r;
    r["x"] = dx; r["weight"] = dw; r["bias"] = db;
    return r;
}

// ---------------------------------------------------------- beam search ----

py::tuple beam_select(const Tensor& logits, const Tensor& scores, const std::optional<int64_t>& n_out,
                      const MaybeTensor& finished, int64_t eos, const MaybeTensor& workspace, const py::object& stream) {
    on_gpu(logits, "logits");
    if (logits.dim() != 3) throw py::value_error("logits must be [G, K, V]");
    const at::Device dev = logits.device();
    const int64_t G = logits.size(0), K = logits.size(1), M = n_out.value_or(K);
    want(scores, "scores", {G, K}, at::kFloat, dev);
    want(finished, "finished", {G, K}, at::kBool, dev);
    want_workspace(workspace, dev);
    gdr_beam_desc d;
    d.G = size32(G, "G"); d.K = size32(K, "K"); d.V = size32(logits.size(2), "V"); d.M = size32(std::max<int64_t>(M, 0), "n_out");
    d.row = row_stride(logits, "logits");
    d.x_dtype = code(logits.scalar_type());
    d.eos = eos < 0 || eos > INT32_MAX ? -1 : static_cast<int>(eos);
    const Call call(dev, stream);
    call.uses(logits, scores, finished, workspace);
    const size_t need = api.beam_select_workspace_bytes(&d);
    if (!need)      // nothing to do, or sizes that are refused, before outputs of them are allocated
        check(api.beam_select(&d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, call.stream), "gdr_beam_select");
    Tensor out = call.output({G, d.M}, at::kFloat), parent = call.output({G, d.M}, at::kInt), token = call.output({G, d.M}, at::kInt);
    const MaybeTensor ws = workspace ? workspace : need ? MaybeTensor(call.scratch({static_cast<int64_t>(need)}, at::kByte)) : MaybeTensor();
    check(api.beam_select(&d, at_(logits), at_<float>(scores), at_<unsigned char>(finished), at_<float>(out), at_<int>(parent),
                          at_<int>(token), at_(ws), ws ? ws->nbytes() : 0, call.stream), "gdr_beam_select");
    return py::make_tuple(out, parent, token);
}

Tensor state_reorder(const Tensor& S, const Tensor& parent, bool layers, const py::object& stream) {
    on_gpu(S, "S");
    dense(S, "S");
    const at::Device dev = S.device();
    const int64_t at = layers ? 1 : 0;
    if (parent.dim() != 2 || S.dim() < 1 + at)
        throw py::value_error("parent must be [G, K] and S [G * K, ...] (layers: [L, G * K, ...])");
    want(parent, "parent", parent.sizes(), at::kInt, dev);
    const int64_t G = parent.size(0), K = parent.size(1), L = layers ? S.size(0) : 1, n = L * G * K;
    if (S.size(at) != G * K)
        throw py::value_error("S must hold G * K = " + std::to_string(G * K) + " states, got " + std::to_string(S.size(at)));
    gdr_reorder_desc d;
    d.L = size32(L, "L"); d.G = size32(G, "G"); d.K = size32(K, "K");
    d.state_bytes = n ? S.nbytes() / n : 0;
    const Call call(dev, stream);
    call.uses(S, parent);
    check(api.state_reorder(&d, at_(S), at_<int>(parent), call.stream), "gdr_state_reorder");
    return S;
}

}  // namespace

PYBIND11_MODULE(_binding, m) {
    m.attr("torch_version") = GDR_BUILT_WITH_TORCH;
    m.def("load", &load);
    m.def("row_stride", &row_stride);
    m.def("scan_fwd", &scan_fwd);
    m.def("scan_bwd", &scan_bwd);
    m.def("scan_step", &scan_step);
    m.def("layernorm_fwd", &layernorm_fwd);
    m.def("layernorm_bwd", &layernorm_bwd);
    m.def("beam_select", &beam_select);
    m.def("state_reorder", &state_reorder);
}
