// binding.cpp -- the torch-tensor forms of the operators around the attention (recurrence, rotary
// positions, group norm) as a compiled Python module.
//
// Argument checks, output allocation and the call into the C ABI, nothing else.  Compiled because
// these calls are short: a decoding step's kernel takes 1 to 3 us, and marshalling it through
// ctypes took 12 us on the host where this takes 6 (B8 H16 d128).
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <climits>

#include "la_chunked.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;
using OptStream = std::optional<int64_t>;

[[noreturn]] void fail(int status, const char *what)
{
    const py::object cls = py::module_::import("chunkwise_causal_linear_gb300").attr("LAError");
    PyErr_SetObject(cls.ptr(), cls(status, what).ptr());
    throw py::error_already_set();
}

std::string text(at::IntArrayRef shape)
{
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + ")";
}

void check(const Tensor &t, at::IntArrayRef shape, at::ScalarType type, const at::Device &device, const char *name)
{
    if (t.sizes() != shape)
        throw py::value_error(std::string(name) + " must be " + text(shape) + ", got " + text(t.sizes()));
    if (t.scalar_type() != type || t.device() != device)
        throw py::type_error(std::string(name) + " must be " + at::toString(type) + " on " + device.str() + ", got " +
                             at::toString(t.scalar_type()) + " on " + t.device().str());
}

// A contiguous tensor of that shape and type; NULL where there is none.
template <typename T>
T *dense(const OptTensor &t, at::IntArrayRef shape, at::ScalarType type, const at::Device &device, const char *name)
{
    if (!t) return nullptr;
    if (t->sizes() != shape || t->scalar_type() != type || t->device() != device || !t->is_contiguous())
        throw py::value_error(std::string(name) + " must be contiguous " + at::toString(type) + " " + text(shape) +
                              " on " + device.str() + ", got " + at::toString(t->scalar_type()) + " " +
                              text(t->sizes()) + " on " + t->device().str());
    return (T *)t->data_ptr();
}

// Strides of a [B, H, L, d] tensor, or of a [B, L, H d] one whose heads are d apart.
struct Strides {
    la_strides s{};
    const la_strides *p = nullptr;
    Strides() = default;
    Strides(const Tensor &t, at::IntArrayRef shape, at::ScalarType type, const at::Device &device, const char *name,
            int64_t d = 0)
    {
        check(t, shape, type, device, name);
        if (t.is_contiguous()) return;
        const at::IntArrayRef st = t.strides();
        if (st.back() != 1 && shape.back() > 1)
            throw py::value_error(std::string(name) + ": the channels (last axis) must be adjacent");
        s = d ? la_strides{st[0], d, st[1]} : la_strides{st[0], st[1], st[2]};
        p = &s;
    }
    Strides(const Strides &) = delete;  // p points into the object
};

int code(const Tensor &t)
{
    if (t.scalar_type() == at::kBFloat16) return LA_BF16;
    if (t.scalar_type() == at::kFloat) return LA_F32;
    throw py::type_error(std::string("unsupported dtype ") + at::toString(t.scalar_type()));
}

void *ptr(const OptTensor &t) { return t ? t->data_ptr() : nullptr; }

// The tensors' device made current, and the stream.  A stream that the caller names is made current
// too: what is allocated here belongs to it, and memory that is given back, as the workspace is at
// the end of the call, is not handed to another stream while the kernels still use it.
struct Place {
    c10::cuda::OptionalCUDAGuard guard;
    c10::cuda::OptionalCUDAStreamGuard stream_guard;
    void *stream;
    Place(const at::Device &device, const OptStream &s, const char *what)
    {
        if (!device.is_cuda())
            throw py::value_error(std::string(what) + ": CUDA tensors are needed, got " + device.str());
        guard.set_device(device);
        if (s) {
            // torch knows the legacy default stream by 0 only
            const cudaStream_t given = *s == (int64_t)(intptr_t)cudaStreamLegacy ? nullptr : (cudaStream_t)*s;
            stream_guard.reset_stream(c10::cuda::getStreamFromExternal(given, device.index()));
            stream = given;
        } else {
            stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        }
    }
};

// Axes of an input, each of a length that the C ABI's ints hold.
void axes(const Tensor &t, int n, const char *name)
{
    if (t.dim() != n)
        throw py::value_error(std::string(name) + " must have " + std::to_string(n) + " axes, got " + text(t.sizes()));
    for (const int64_t len : t.sizes())
        if (len > INT_MAX) throw py::value_error(std::string(name) + " is too long: " + text(t.sizes()));
}

py::object recurrence_fwd(const Tensor &x, const Tensor &gate, const OptTensor &h0, int gate_kind, bool complement,
                          const OptTensor &lengths, bool save_chunks, const OptTensor &out_, const OptStream &stream)
{
    const char *what = "la_recurrence_fwd";
    axes(x, 4, "x");
    const at::Device dev = x.device();
    const at::ScalarType type = x.scalar_type();
    const int64_t B = x.size(0), H = x.size(1), L = x.size(2), d = x.size(3);
    const int dtype = code(x), gtype = code(gate);
    const Place place(dev, stream, what);
    const Strides sx(x, x.sizes(), type, dev, "x"), sg(gate, x.sizes(), gate.scalar_type(), dev, "gate");
    const float *h = dense<float>(h0, {B, H, d}, at::kFloat, dev, "h0");
    const int *n = dense<int>(lengths, {B}, at::kInt, dev, "lengths");
    const auto f32 = x.options().dtype(at::kFloat);
    const Tensor out = out_ ? *out_ : at::empty(x.sizes(), x.options()), last = at::empty({B, H, d}, f32);
    const Strides so(out, x.sizes(), type, dev, "out");
    Tensor chunks;
    if (save_chunks) chunks = at::empty({B, H, (L + LA_RECURRENCE_CHUNK - 1) / LA_RECURRENCE_CHUNK, d}, f32);
    const int rc = la_recurrence_fwd(x.data_ptr(), gate.data_ptr(), h, n, out.data_ptr(), (float *)last.data_ptr(),
                                     save_chunks ? (float *)chunks.data_ptr() : nullptr, (int)B, (int)H, (int)L, (int)d,
                                     sx.p, sg.p, so.p, gate_kind, complement, dtype, gtype, place.stream);
    if (rc != LA_OK) fail(rc, what);
    if (save_chunks) return py::make_tuple(out, last, chunks);
    return py::make_tuple(out, last);
}

py::tuple recurrence_bwd(const Tensor &x, const Tensor &gate, const Tensor &chunk_states, const Tensor &dout,
                         const OptTensor &dh_last, int gate_kind, bool complement, const OptTensor &lengths,
                         const OptTensor &dx_, const OptTensor &dgate_, const OptStream &stream)
{
    const char *what = "la_recurrence_bwd";
    axes(x, 4, "x");
    const at::Device dev = x.device();
    const at::ScalarType type = x.scalar_type(), gate_type = gate.scalar_type();
    const int64_t B = x.size(0), H = x.size(1), L = x.size(2), d = x.size(3);
    const int dtype = code(x), gtype = code(gate);
    const Place place(dev, stream, what);
    const at::IntArrayRef shape = x.sizes();
    const Strides sx(x, shape, type, dev, "x"), sg(gate, shape, gate_type, dev, "gate"), sd(dout, shape, type, dev, "dout");
    const float *chunks = dense<float>(chunk_states, {B, H, (L + LA_RECURRENCE_CHUNK - 1) / LA_RECURRENCE_CHUNK, d},
                                       at::kFloat, dev, "chunk_states");
    const float *dl = dense<float>(dh_last, {B, H, d}, at::kFloat, dev, "dh_last");
    const int *n = dense<int>(lengths, {B}, at::kInt, dev, "lengths");
    const Tensor dx = dx_ ? *dx_ : at::empty(shape, x.options()), dgate = dgate_ ? *dgate_ : at::empty(shape, gate.options());
    const Tensor dh0 = at::empty({B, H, d}, x.options().dtype(at::kFloat));
    const Strides sdx(dx, shape, type, dev, "dx"), sdg(dgate, shape, gate_type, dev, "dgate");
    const int rc = la_recurrence_bwd(x.data_ptr(), gate.data_ptr(), chunks, n, dout.data_ptr(), dl, dx.data_ptr(),
                                     dgate.data_ptr(), (float *)dh0.data_ptr(), (int)B, (int)H, (int)L, (int)d, sx.p, sg.p,
                                     sd.p, sdx.p, sdg.p, gate_kind, complement, dtype, gtype, place.stream);
    if (rc != LA_OK) fail(rc, what);
    return py::make_tuple(dx, dgate, dh0);
}

Tensor recurrence_step(const Tensor &x, const Tensor &gate, const Tensor &state, int gate_kind, bool complement,
                       const OptTensor &out_, const OptStream &stream)
{
    const char *what = "la_recurrence_step";
    axes(x, 3, "x");
    const at::Device dev = x.device();
    const int dtype = code(x), gtype = code(gate);
    const Place place(dev, stream, what);
    const at::IntArrayRef shape = x.sizes();
    const Tensor out = out_ ? *out_ : at::empty(shape, x.options());
    const int rc = la_recurrence_step(dense<void>(x, shape, x.scalar_type(), dev, "x"),
                                      dense<void>(gate, shape, gate.scalar_type(), dev, "gate"),
                                      dense<float>(state, shape, at::kFloat, dev, "state"),
                                      dense<void>(out, shape, x.scalar_type(), dev, "out"), (int)x.size(0),
                                      (int)x.size(1), (int)x.size(2), gate_kind, complement, dtype, gtype, place.stream);
    if (rc != LA_OK) fail(rc, what);
    return out;
}

py::tuple rotary(const Tensor &q, const OptTensor &k, const Tensor &turns, int64_t rot, double amplitude,
                 const OptTensor &positions, int64_t offset, int layout, bool inverse, const OptTensor &q_out_,
                 const OptTensor &k_out_, const OptStream &stream)
{
    const char *what = "la_rotary";
    axes(q, 4, "q");
    if (k_out_ && !k) throw py::value_error("k_out is given without k");
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const int64_t B = q.size(0), H = q.size(1), L = q.size(2), d = q.size(3);
    const int dtype = code(q);
    const Place place(dev, stream, what);
    const Strides sq(q, q.sizes(), type, dev, "q");
    const Tensor q_out = q_out_ ? *q_out_ : at::empty(q.sizes(), q.options());
    const Strides sqo(q_out, q.sizes(), type, dev, "q_out");
    int64_t Hk = 0;
    OptTensor k_out;
    std::optional<Strides> sk, sko;
    if (k) {
        axes(*k, 4, "k");
        Hk = k->size(1);
        const std::array<int64_t, 4> shape{B, Hk, L, d};
        sk.emplace(*k, shape, type, dev, "k");
        k_out = k_out_ ? *k_out_ : at::empty(shape, k->options());
        sko.emplace(*k_out, shape, type, dev, "k_out");
    }
    const int rc = la_rotary(q.data_ptr(), ptr(k), q_out.data_ptr(), ptr(k_out),
                             dense<unsigned long long>(turns, {rot / 2}, at::kLong, dev, "table"),
                             dense<int>(positions, {B, L}, at::kInt, dev, "positions"), offset, (int)B, (int)H, (int)Hk,
                             (int)L, (int)d, (int)rot, sq.p, sk ? sk->p : nullptr, sqo.p, sko ? sko->p : nullptr, layout,
                             inverse, (float)amplitude, dtype, place.stream);
    if (rc != LA_OK) fail(rc, what);
    return py::make_tuple(q_out, k_out);
}

Tensor group_norm_fwd(const Tensor &x, const OptTensor &weight, const OptTensor &bias, const OptTensor &gate, double eps,
                      int activation, bool center, const OptTensor &out_, const OptStream &stream)
{
    const char *what = "la_group_norm_fwd";
    axes(x, 4, "x");
    const at::Device dev = x.device();
    const at::ScalarType type = x.scalar_type();
    const int64_t B = x.size(0), H = x.size(1), L = x.size(2), d = x.size(3);
    const int dtype = code(x);
    const Place place(dev, stream, what);
    const std::array<int64_t, 3> last{B, L, H * d};
    const Strides sx(x, x.sizes(), type, dev, "x");
    const float *w = dense<float>(weight, {H * d}, at::kFloat, dev, "weight");
    const float *b = dense<float>(bias, {H * d}, at::kFloat, dev, "bias");
    std::optional<Strides> sg;
    if (gate) sg.emplace(*gate, last, type, dev, "gate", d);
    const Tensor out = out_ ? *out_ : at::empty(last, x.options());
    const Strides so(out, last, type, dev, "out", d);
    const int rc = la_group_norm_fwd(x.data_ptr(), w, b, ptr(gate), out.data_ptr(), (int)B, (int)H, (int)L, (int)d, sx.p,
                                     sg ? sg->p : nullptr, so.p, center, activation, (float)eps, dtype, place.stream);
    if (rc != LA_OK) fail(rc, what);
    return out;
}

py::tuple group_norm_bwd(const Tensor &x, const Tensor &dout, const OptTensor &weight, const OptTensor &bias,
                         const OptTensor &gate, double eps, int activation, bool center, const OptTensor &dx_,
                         const OptTensor &dgate_, const OptTensor &workspace_, const OptStream &stream)
{
    const char *what = "la_group_norm_bwd";
    axes(x, 4, "x");
    if (dgate_ && !gate) throw py::value_error("dgate is given without gate");
    const at::Device dev = x.device();
    if (workspace_ && (workspace_->device() != dev || !workspace_->is_contiguous()))
        throw py::value_error("workspace must be contiguous on " + dev.str());
    const at::ScalarType type = x.scalar_type();
    const int64_t B = x.size(0), H = x.size(1), L = x.size(2), d = x.size(3);
    const int dtype = code(x);
    const Place place(dev, stream, what);
    const std::array<int64_t, 3> last{B, L, H * d};
    const Strides sx(x, x.sizes(), type, dev, "x"), sd(dout, last, type, dev, "dout", d);
    const float *w = dense<float>(weight, {H * d}, at::kFloat, dev, "weight");
    const float *b = dense<float>(bias, {H * d}, at::kFloat, dev, "bias");
    const Tensor dx = dx_ ? *dx_ : at::empty(x.sizes(), x.options());
    const Strides sdx(dx, x.sizes(), type, dev, "dx");
    OptTensor dgate, dw, db, workspace = workspace_;
    std::optional<Strides> sg, sdg;
    if (gate) {
        sg.emplace(*gate, last, type, dev, "gate", d);
        dgate = dgate_ ? *dgate_ : at::empty(last, x.options());
        sdg.emplace(*dgate, last, type, dev, "dgate", d);
    }
    const auto f32 = x.options().dtype(at::kFloat);
    if (weight) dw = at::empty({H * d}, f32);
    if (bias) db = at::empty({H * d}, f32);
    size_t need = 0;
    if (weight || bias) {
        need = la_group_norm_bwd_workspace_bytes((int)B, (int)H, (int)L, (int)d);
        if (!workspace || workspace->nbytes() < need) workspace = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
    }
    const int rc = la_group_norm_bwd(x.data_ptr(), w, b, ptr(gate), dout.data_ptr(), dx.data_ptr(), ptr(dgate),
                                     (float *)ptr(dw), (float *)ptr(db), (int)B, (int)H, (int)L, (int)d, sx.p,
                                     sg ? sg->p : nullptr, sd.p, sdx.p, sdg ? sdg->p : nullptr, center, activation,
                                     (float)eps, dtype, need ? ptr(workspace) : nullptr, need, place.stream);
    if (rc != LA_OK) fail(rc, what);
    return py::make_tuple(dx, dgate, dw, db);
}

}  // namespace

PYBIND11_MODULE(_layer, m)
{
    m.def("recurrence_fwd", &recurrence_fwd);
    m.def("recurrence_bwd", &recurrence_bwd);
    m.def("recurrence_step", &recurrence_step);
    m.def("rotary", &rotary);
    m.def("group_norm_fwd", &group_norm_fwd);
    m.def("group_norm_bwd", &group_norm_bwd);
}
