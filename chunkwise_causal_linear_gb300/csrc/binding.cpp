// binding.cpp -- the torch-tensor forms of the gated attention and of the operators around the attention
// (recurrence, rotary positions, group norm, norms around a block) as a compiled Python module.
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

// log_decay: fp32 [H], [B, H, L] or (without L) [B, H].
la_strides gate_strides(const Tensor &g, int64_t B, int64_t H, int64_t L, const at::Device &dev)
{
    if (g.scalar_type() != at::kFloat || g.device() != dev)
        throw py::type_error("log_decay must be Float on " + dev.str() + ", got " + at::toString(g.scalar_type()) + " on " +
                             g.device().str());
    if (g.dim() == 1 && g.size(0) == H) return {0, g.stride(0), 0};
    if (L < 0 && g.dim() == 2 && g.size(0) == B && g.size(1) == H) return {g.stride(0), g.stride(1), 0};
    if (L >= 0 && g.dim() == 3 && g.size(0) == B && g.size(1) == H && g.size(2) == L)
        return {g.stride(0), g.stride(1), g.stride(2)};
    throw py::value_error("log_decay must have one value per head or per token and head, got " + text(g.sizes()));
}

void *room(OptTensor &workspace, size_t need, const at::Device &dev)
{
    if (workspace && (workspace->device() != dev || !workspace->is_contiguous()))
        throw py::value_error("workspace must be contiguous on " + dev.str());
    if (!need) return nullptr;
    if (!workspace || workspace->nbytes() < need)
        workspace = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(dev));
    return workspace->data_ptr();
}

py::tuple gated_fwd(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &log_decay, double scale,
                    const OptTensor &state0, const OptTensor &lengths, const OptTensor &slots, const OptTensor &state_,
                    const OptTensor &out_, OptTensor workspace, const OptStream &stream, int path)
{
    const char *what = "la_gated_fwd";
    axes(q, 4, "q");
    axes(k, 4, "k");
    axes(v, 4, "v");
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const int64_t B = q.size(0), H = q.size(1), L = q.size(2), d = q.size(3), Hk = k.size(1), e = v.size(3);
    const int dtype = code(q);
    const Place place(dev, stream, what);
    const std::array<int64_t, 4> kshape{B, Hk, L, d}, vshape{B, Hk, L, e}, oshape{B, H, L, e};
    const Strides sq(q, q.sizes(), type, dev, "q"), sk(k, kshape, type, dev, "k"), sv(v, vshape, type, dev, "v");
    const la_strides sg = gate_strides(log_decay, B, H, L, dev);
    const int *n = dense<int>(lengths, {B}, at::kInt, dev, "lengths"), *at_ = dense<int>(slots, {B}, at::kInt, dev, "slots");
    OptTensor state = state_;
    int64_t pool = B;
    if (slots) {
        if (!state0 && !state) throw py::value_error("slots are given without a pool of states");
        const Tensor &p = state ? *state : *state0;
        axes(p, 4, "state");
        pool = p.size(0);
    } else if (!state) {
        state = at::empty({B, H, d, e}, q.options().dtype(at::kFloat));
    }
    const float *s0 = dense<float>(state0, {pool, H, d, e}, at::kFloat, dev, "state0");
    float *s1 = dense<float>(state, {pool, H, d, e}, at::kFloat, dev, "state");
    const Tensor out = out_ ? *out_ : at::empty(oshape, q.options());
    const Strides so(out, oshape, type, dev, "out");
    const size_t need = la_gated_workspace_bytes((int)B, (int)H, (int)L, (int)d, (int)e, dtype);
    void *ws = room(workspace, need, dev);
    const int rc = la_gated_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), (const float *)log_decay.data_ptr(), s0, s1, at_,
                                n, out.data_ptr(), (int)B, (int)H, (int)Hk, (int)L, (int)d, (int)e, (int)pool, sq.p, sk.p,
                                sv.p, &sg, so.p, (float)scale, dtype, ws, need, place.stream, path);
    if (rc != LA_OK) fail(rc, what);
    return py::make_tuple(out, state);
}

py::tuple gated_bwd(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &log_decay, const Tensor &dout,
                    double scale, const OptTensor &state0, const OptTensor &lengths, const OptTensor &dstate,
                    const OptTensor &dq_, const OptTensor &dk_, const OptTensor &dv_, bool decay_grad, OptTensor workspace,
                    const OptStream &stream, int path)
{
    const char *what = "la_gated_bwd";
    axes(q, 4, "q");
    axes(k, 4, "k");
    axes(v, 4, "v");
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const int64_t B = q.size(0), H = q.size(1), L = q.size(2), d = q.size(3), Hk = k.size(1), e = v.size(3);
    const int dtype = code(q);
    const Place place(dev, stream, what);
    const std::array<int64_t, 4> kshape{B, Hk, L, d}, vshape{B, Hk, L, e}, oshape{B, H, L, e};
    const Strides sq(q, q.sizes(), type, dev, "q"), sk(k, kshape, type, dev, "k"), sv(v, vshape, type, dev, "v"),
        so(dout, oshape, type, dev, "dout");
    const la_strides sg = gate_strides(log_decay, B, H, L, dev);
    const int *n = dense<int>(lengths, {B}, at::kInt, dev, "lengths");
    const float *s0 = dense<float>(state0, {B, H, d, e}, at::kFloat, dev, "state0"),
                *ds = dense<float>(dstate, {B, H, d, e}, at::kFloat, dev, "dstate");
    const Tensor dq = dq_ ? *dq_ : at::empty(q.sizes(), q.options()), dk = dk_ ? *dk_ : at::empty(kshape, q.options()),
                 dv = dv_ ? *dv_ : at::empty(vshape, q.options());
    const Strides sdq(dq, q.sizes(), type, dev, "dq"), sdk(dk, kshape, type, dev, "dk"), sdv(dv, vshape, type, dev, "dv");
    const auto f32 = q.options().dtype(at::kFloat);
    const bool heads = log_decay.dim() == 1;
    OptTensor dg;
    if (decay_grad) dg = heads ? at::empty({H}, f32) : at::empty({B, H, L}, f32);
    const Tensor dstate0 = at::empty({B, H, d, e}, f32);
    const size_t need = la_gated_bwd_workspace_bytes((int)B, (int)H, (int)Hk, (int)L, (int)d, (int)e, dtype);
    void *ws = room(workspace, need, dev);
    const int rc = la_gated_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), (const float *)log_decay.data_ptr(), s0, n,
                                dout.data_ptr(), ds, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                heads ? nullptr : (float *)ptr(dg), heads ? (float *)ptr(dg) : nullptr,
                                (float *)dstate0.data_ptr(), (int)B, (int)H, (int)Hk, (int)L, (int)d, (int)e, sq.p, sk.p, sv.p,
                                &sg, so.p, sdq.p, sdk.p, sdv.p, (float)scale, dtype, ws, need, place.stream, path);
    if (rc != LA_OK) fail(rc, what);
    return py::make_tuple(dq, dk, dv, dg, dstate0);
}

// Strides of a [B, H, d] tensor.
la_strides step_strides(const Tensor &t, at::IntArrayRef shape, at::ScalarType type, const at::Device &dev, const char *name)
{
    check(t, shape, type, dev, name);
    if (t.stride(2) != 1 && shape[2] > 1) throw py::value_error(std::string(name) + ": the channels (last axis) must be adjacent");
    return {t.stride(0), t.stride(1), 0};
}

Tensor gated_step(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &log_decay, const Tensor &state,
                  double scale, const OptTensor &slots, const OptTensor &out_, const OptStream &stream)
{
    const char *what = "la_gated_step";
    axes(q, 3, "q");
    axes(k, 3, "k");
    axes(v, 3, "v");
    axes(state, 4, "state");
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const int64_t B = q.size(0), H = q.size(1), d = q.size(2), Hk = k.size(1), e = v.size(2);
    const int dtype = code(q);
    const Place place(dev, stream, what);
    const la_strides sq = step_strides(q, q.sizes(), type, dev, "q"), sk = step_strides(k, {B, Hk, d}, type, dev, "k"),
                     sv = step_strides(v, {B, Hk, e}, type, dev, "v"), sg = gate_strides(log_decay, B, H, -1, dev);
    const int *at_ = dense<int>(slots, {B}, at::kInt, dev, "slots");
    const int64_t pool = slots ? state.size(0) : B;
    float *s = dense<float>(state, {pool, H, d, e}, at::kFloat, dev, "state");
    const Tensor out = out_ ? *out_ : at::empty({B, H, e}, q.options());
    void *o = dense<void>(out, {B, H, e}, type, dev, "out");
    const int rc = la_gated_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), (const float *)log_decay.data_ptr(), s, at_, o,
                                 (int)B, (int)H, (int)Hk, (int)d, (int)e, (int)pool, &sq, &sk, &sv, &sg, (float)scale, dtype,
                                 place.stream);
    if (rc != LA_OK) fail(rc, what);
    return out;
}

// Strides of a [B, L, d] tensor.
struct RowStrides {
    la_strides s{};
    const la_strides *p = nullptr;
    RowStrides(const OptTensor &t, at::IntArrayRef shape, at::ScalarType type, const at::Device &dev, const char *name)
    {
        if (!t) return;
        check(*t, shape, type, dev, name);
        if (t->is_contiguous()) return;
        if (t->stride(2) != 1 && shape[2] > 1)
            throw py::value_error(std::string(name) + ": the channels (last axis) must be adjacent");
        s = {t->stride(0), 0, t->stride(1)};
        p = &s;
    }
    RowStrides(const RowStrides &) = delete;
};

py::tuple block_norm_fwd(const Tensor &y, const Tensor &residual, const OptTensor &gate, int activation, int post,
                         const OptTensor &post_w, const OptTensor &post_b, int pre, const OptTensor &pre_w,
                         const OptTensor &pre_b, double rs, double bs, double eps, const OptTensor &h_, const OptTensor &n_,
                         const OptStream &stream)
{
    const char *what = "la_block_norm_fwd";
    axes(y, 3, "y");
    const at::Device dev = y.device();
    const at::ScalarType type = y.scalar_type(), rtype = residual.scalar_type();
    const int dtype = code(y), rcode = code(residual);
    const Place place(dev, stream, what);
    const at::IntArrayRef shape = y.sizes();
    const int64_t d = shape[2];
    if (pre == LA_NORM_NONE && (n_ || pre_w || pre_b)) throw py::value_error("n or its weights are given without a norm");
    const RowStrides sy(y, shape, type, dev, "y"), sr(residual, shape, rtype, dev, "residual"), sg(gate, shape, type, dev, "gate");
    const float *w1 = dense<float>(post_w, {d}, at::kFloat, dev, "post_weight"), *b1 = dense<float>(post_b, {d}, at::kFloat, dev, "post_bias"),
                *w2 = dense<float>(pre_w, {d}, at::kFloat, dev, "pre_weight"), *b2 = dense<float>(pre_b, {d}, at::kFloat, dev, "pre_bias");
    const Tensor h = h_ ? *h_ : at::empty(shape, residual.options());
    OptTensor n = n_;
    if (!n && pre != LA_NORM_NONE) n = at::empty(shape, y.options());
    const RowStrides sh(h, shape, rtype, dev, "h"), sn(n, shape, type, dev, "n");
    const int rc = la_block_norm_fwd(y.data_ptr(), residual.data_ptr(), ptr(gate), w1, b1, w2, b2, h.data_ptr(), ptr(n),
                                     (int)shape[0], (int)shape[1], (int)d, sy.p, sr.p, sg.p, sh.p, sn.p, post, pre, activation,
                                     (float)rs, (float)bs, (float)eps, dtype, rcode, place.stream);
    if (rc != LA_OK) fail(rc, what);
    return py::make_tuple(h, n);
}

py::dict block_norm_bwd(const Tensor &y, const Tensor &residual, const OptTensor &dh, const OptTensor &dn, const OptTensor &gate,
                        int activation, int post, const OptTensor &post_w, const OptTensor &post_b, int pre,
                        const OptTensor &pre_w, const OptTensor &pre_b, double rs, double bs, double eps, const OptTensor &dr_,
                        const OptTensor &dy_, const OptTensor &dgate_, OptTensor workspace, const OptStream &stream)
{
    const char *what = "la_block_norm_bwd";
    axes(y, 3, "y");
    if (dgate_ && !gate) throw py::value_error("dgate is given without gate");
    if (pre == LA_NORM_NONE && (dn || pre_w || pre_b)) throw py::value_error("dn or its weights are given without a norm");
    const at::Device dev = y.device();
    const at::ScalarType type = y.scalar_type(), rtype = residual.scalar_type();
    const int dtype = code(y), rcode = code(residual);
    const Place place(dev, stream, what);
    const at::IntArrayRef shape = y.sizes();
    const int64_t B = shape[0], L = shape[1], d = shape[2];
    const RowStrides sy(y, shape, type, dev, "y"), sr(residual, shape, rtype, dev, "residual"), sg(gate, shape, type, dev, "gate"),
        sdh(dh, shape, rtype, dev, "dh"), sdn(dn, shape, type, dev, "dn");
    const float *w1 = dense<float>(post_w, {d}, at::kFloat, dev, "post_weight"), *b1 = dense<float>(post_b, {d}, at::kFloat, dev, "post_bias"),
                *w2 = dense<float>(pre_w, {d}, at::kFloat, dev, "pre_weight"), *b2 = dense<float>(pre_b, {d}, at::kFloat, dev, "pre_bias");
    const Tensor dr = dr_ ? *dr_ : at::empty(shape, residual.options()), dy = dy_ ? *dy_ : at::empty(shape, y.options());
    OptTensor dgate, dw1, db1, dw2, db2;
    if (gate) dgate = dgate_ ? *dgate_ : at::empty(shape, y.options());
    const RowStrides sdr(dr, shape, rtype, dev, "dr"), sdy(dy, shape, type, dev, "dy"), sdg(dgate, shape, type, dev, "dgate");
    const auto f32 = y.options().dtype(at::kFloat);
    if (post_w) dw1 = at::empty({d}, f32);
    if (post_b) db1 = at::empty({d}, f32);
    if (pre_w && dn) dw2 = at::empty({d}, f32);
    if (pre_b && dn) db2 = at::empty({d}, f32);
    const size_t need = dw1 || db1 || dw2 || db2 ? la_block_norm_bwd_workspace_bytes((int)B, (int)L, (int)d) : 0;
    void *ws = room(workspace, need, dev);
    const int rc = la_block_norm_bwd(y.data_ptr(), residual.data_ptr(), ptr(gate), w1, b1, w2, b2, ptr(dh), ptr(dn), dr.data_ptr(),
                                     dy.data_ptr(), ptr(dgate), (float *)ptr(dw1), (float *)ptr(db1), (float *)ptr(dw2),
                                     (float *)ptr(db2), (int)B, (int)L, (int)d, sy.p, sr.p, sg.p, sdh.p, sdn.p, sdr.p, sdy.p, sdg.p,
                                     post, pre, activation, (float)rs, (float)bs, (float)eps, dtype, rcode, ws, need, place.stream);
    if (rc != LA_OK) fail(rc, what);
    py::dict out;
    out["dy"] = dy;
    out["dr"] = dr;
    out["dgate"] = dgate;
    out["dpost_w"] = dw1;
    out["dpost_b"] = db1;
    out["dpre_w"] = dw2;
    out["dpre_b"] = db2;
    return out;
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
    m.def("block_norm_fwd", &block_norm_fwd);
    m.def("block_norm_bwd", &block_norm_bwd);
    m.def("gated_fwd", &gated_fwd);
    m.def("gated_bwd", &gated_bwd);
    m.def("gated_step", &gated_step);
}
