// recurrence.cu -- gated linear recurrence h_t = a_t h_{t-1} + w_t x_t, its gradients and its
// decoding step (sm_103a).
//
// One thread per channel walks its sequence.  The gradients run backwards over the sequence,
// e_t = dout_t + a_{t+1} e_{t+1}; they need h_{t-1}, which each 128-row chunk recomputes in
// fp32 from the state before it (left by the forward).
#include "layer.cuh"

namespace la {

namespace {

constexpr int RC = LA_RECURRENCE_CHUNK;
constexpr int REC_THREADS = 128;

struct RecArgs {
    const void *x, *g, *dout;
    void *out, *dx, *dg;
    const float *h0, *dh_last, *chunks_in;
    float *h_last, *dh0, *chunks;
    const int *lengths;
    View vx, vg, vo, vdx, vdg;  // vo: out, or dout
    int B, H, L, d;
};

// a, w and da/dg from the gate input.  1 - a comes from its own formula where a is close to 1.
template <int KIND, bool COMP>
__device__ __forceinline__ void gate_of(float g, float &a, float &w, float &slope)
{
    if (KIND == LA_GATE_VALUE) {
        a = g;
        w = COMP ? 1.f - g : 1.f;
        slope = 1.f;
    } else if (KIND == LA_GATE_LOG) {
        a = expf(g);
        w = COMP ? -expm1f(g) : 1.f;
        slope = a;
    } else {
        // sigmoid(g) and sigmoid(-g) from e^-|g|, which never overflows
        const float e = expf(-fabsf(g)), r = 1.f / (1.f + e), s = e * r;
        a = g >= 0.f ? r : s;
        const float c = g >= 0.f ? s : r;
        w = COMP ? c : 1.f;
        slope = a * c;
    }
}

// One row of the recurrence: the state times the gate, a gate of 0 forgetting infinities and NaN
// as well.
__device__ __forceinline__ float forget(float a, float h) { return a == 0.f ? 0.f : a * h; }

__device__ __forceinline__ int rows_of(const RecArgs &a, int b)
{
    return a.lengths ? max(0, min(a.lengths[b], a.L)) : a.L;
}

template <typename T, typename G, int KIND, bool COMP>
__global__ void __launch_bounds__(REC_THREADS) rec_fwd_kernel(const RecArgs a)
{
    const int bh = blockIdx.x, b = bh / a.H, hd = bh % a.H;
    const int c = blockIdx.y * REC_THREADS + threadIdx.x;
    if (c >= a.d) return;
    const T *x = (const T *)a.x + row_of(a.vx, b, hd, 0) + c;
    const G *g = (const G *)a.g + row_of(a.vg, b, hd, 0) + c;
    T *out = (T *)a.out + row_of(a.vo, b, hd, 0) + c;
    const int n = rows_of(a, b), nc = (a.L + RC - 1) / RC;
    float h = a.h0 ? a.h0[(size_t)bh * a.d + c] : 0.f;
    for (int t = 0; t < a.L; ++t) {
        if (a.chunks && t % RC == 0) a.chunks[((size_t)bh * nc + t / RC) * a.d + c] = h;
        if (t < n) {
            float ga, w, sl;
            gate_of<KIND, COMP>(to_f32(g[t * a.vg.l]), ga, w, sl);
            h = forget(ga, h) + w * to_f32(x[t * a.vx.l]);
        }
        out[t * a.vo.l] = from_f32<T>(t < n ? h : 0.f);
    }
    if (a.h_last) a.h_last[(size_t)bh * a.d + c] = h;
}

template <typename T, typename G, int KIND, bool COMP>
__global__ void __launch_bounds__(REC_THREADS) rec_bwd_kernel(const RecArgs a)
{
    const int bh = blockIdx.x, b = bh / a.H, hd = bh % a.H;
    const int c = blockIdx.y * REC_THREADS + threadIdx.x;
    if (c >= a.d) return;
    const T *x = (const T *)a.x + row_of(a.vx, b, hd, 0) + c;
    const G *g = (const G *)a.g + row_of(a.vg, b, hd, 0) + c;
    const T *dout = (const T *)a.dout + row_of(a.vo, b, hd, 0) + c;
    T *dx = (T *)a.dx + row_of(a.vdx, b, hd, 0) + c;
    G *dg = (G *)a.dg + row_of(a.vdg, b, hd, 0) + c;
    const int n = rows_of(a, b), nc = (a.L + RC - 1) / RC;
    float carry = a.dh_last ? a.dh_last[(size_t)bh * a.d + c] : 0.f;  // a_{t+1} e_{t+1}
    float hs[RC];
    for (int k = nc - 1; k >= 0; --k) {
        const int t0 = k * RC, rows = min(RC, a.L - t0);
        float h = a.chunks_in[((size_t)bh * nc + k) * a.d + c];
        for (int i = 0; i < rows && t0 + i < n; ++i) {
            const int t = t0 + i;
            float ga, w, sl;
            gate_of<KIND, COMP>(to_f32(g[t * a.vg.l]), ga, w, sl);
            hs[i] = h;
            h = forget(ga, h) + w * to_f32(x[t * a.vx.l]);
        }
        for (int i = rows - 1; i >= 0; --i) {
            const int t = t0 + i;
            float rx = 0.f, rg = 0.f;
            if (t < n) {
                float ga, w, sl;
                gate_of<KIND, COMP>(to_f32(g[t * a.vg.l]), ga, w, sl);
                const float e = carry + to_f32(dout[t * a.vo.l]);
                rx = w * e;
                rg = forget(sl, e * (COMP ? hs[i] - to_f32(x[t * a.vx.l]) : hs[i]));
                carry = forget(ga, e);
            }
            dx[t * a.vdx.l] = from_f32<T>(rx);
            dg[t * a.vdg.l] = from_f32<G>(rg);
        }
    }
    if (a.dh0) a.dh0[(size_t)bh * a.d + c] = carry;
}

template <typename T, typename G, int KIND, bool COMP>
__global__ void __launch_bounds__(REC_THREADS) rec_step_kernel(const T *x, const G *g, float *state,
                                                               T *out, long long n)
{
    const long long i = (long long)blockIdx.x * REC_THREADS + threadIdx.x;
    if (i >= n) return;
    float ga, w, sl;
    gate_of<KIND, COMP>(to_f32(g[i]), ga, w, sl);
    const float h = forget(ga, state[i]) + w * to_f32(x[i]);
    state[i] = h;
    out[i] = from_f32<T>(h);
}

// Calls f.template operator()<T, G, KIND, COMP>() for the runtime choice.
template <typename F>
int dispatch(int dtype, int gate_dtype, int kind, int comp, F f)
{
    auto by_kind = [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        if (kind == LA_GATE_VALUE) return comp ? f.template operator()<T, G, LA_GATE_VALUE, true>()
                                               : f.template operator()<T, G, LA_GATE_VALUE, false>();
        if (kind == LA_GATE_LOG) return comp ? f.template operator()<T, G, LA_GATE_LOG, true>()
                                             : f.template operator()<T, G, LA_GATE_LOG, false>();
        return comp ? f.template operator()<T, G, LA_GATE_SIGMOID, true>()
                    : f.template operator()<T, G, LA_GATE_SIGMOID, false>();
    };
    if (dtype == LA_F32)
        return gate_dtype == LA_F32 ? by_kind(float(), float()) : by_kind(float(), __nv_bfloat16());
    return gate_dtype == LA_F32 ? by_kind(__nv_bfloat16(), float())
                                : by_kind(__nv_bfloat16(), __nv_bfloat16());
}

struct LaunchFwd {
    const RecArgs &a;
    cudaStream_t s;
    template <typename T, typename G, int KIND, bool COMP> int operator()() const
    {
        const dim3 grid((unsigned)(a.B * a.H), (unsigned)((a.d + REC_THREADS - 1) / REC_THREADS));
        rec_fwd_kernel<T, G, KIND, COMP><<<grid, REC_THREADS, 0, s>>>(a);
        return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    }
};

struct LaunchBwd {
    const RecArgs &a;
    cudaStream_t s;
    template <typename T, typename G, int KIND, bool COMP> int operator()() const
    {
        const dim3 grid((unsigned)(a.B * a.H), (unsigned)((a.d + REC_THREADS - 1) / REC_THREADS));
        rec_bwd_kernel<T, G, KIND, COMP><<<grid, REC_THREADS, 0, s>>>(a);
        return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    }
};

struct LaunchStep {
    const void *x, *g;
    float *state;
    void *out;
    long long n;
    cudaStream_t s;
    template <typename T, typename G, int KIND, bool COMP> int operator()() const
    {
        const unsigned grid = (unsigned)((n + REC_THREADS - 1) / REC_THREADS);
        rec_step_kernel<T, G, KIND, COMP><<<grid, REC_THREADS, 0, s>>>((const T *)x, (const G *)g, state, (T *)out, n);
        return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    }
};

int check_kinds(int gate_kind, int dtype, int gate_dtype)
{
    if (!dtype_ok(dtype) || !dtype_ok(gate_dtype)) return LA_ERR_UNSUPPORTED;
    if (gate_kind < LA_GATE_VALUE || gate_kind > LA_GATE_SIGMOID) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

int la_recurrence_fwd(const void *x, const void *gate, const float *h0, const int *lengths,
                      void *out, float *h_last, float *chunk_states, int B, int H, int L, int d,
                      const la_strides *x_strides, const la_strides *gate_strides,
                      const la_strides *out_strides, int gate_kind, int complement, int dtype,
                      int gate_dtype, void *stream)
{
    if (!x || !gate || !out) return LA_ERR_NULL;
    if (!sizes_ok(B, H, L, d)) return LA_ERR_SHAPE;
    const int rc = check_kinds(gate_kind, dtype, gate_dtype);
    if (rc != LA_OK) return rc;
    RecArgs a = {};
    a.x = x; a.g = gate; a.out = out;
    a.h0 = h0; a.h_last = h_last; a.chunks = chunk_states; a.lengths = lengths;
    a.B = B; a.H = H; a.L = L; a.d = d;
    a.vx = make_view(x_strides, H, L, d);
    a.vg = make_view(gate_strides, H, L, d);
    a.vo = make_view(out_strides, H, L, d);
    if (!input_view_ok(a.vx, B, H, L) || !input_view_ok(a.vg, B, H, L) || !output_view_ok(a.vo, B, H, L, d))
        return LA_ERR_ARG;
    const size_t e = dtype_size(dtype);
    if (!aligned(x, e) || !aligned(out, e) || !aligned(gate, dtype_size(gate_dtype)) || !aligned(h0, 4) ||
        !aligned(h_last, 4) || !aligned(chunk_states, 4) || !aligned(lengths, 4))
        return LA_ERR_ARG;
    return dispatch(dtype, gate_dtype, gate_kind, complement != 0, LaunchFwd{a, (cudaStream_t)stream});
}

int la_recurrence_bwd(const void *x, const void *gate, const float *chunk_states,
                      const int *lengths, const void *dout, const float *dh_last, void *dx,
                      void *dgate, float *dh0, int B, int H, int L, int d,
                      const la_strides *x_strides, const la_strides *gate_strides,
                      const la_strides *dout_strides, const la_strides *dx_strides,
                      const la_strides *dgate_strides, int gate_kind, int complement, int dtype,
                      int gate_dtype, void *stream)
{
    if (!x || !gate || !chunk_states || !dout || !dx || !dgate) return LA_ERR_NULL;
    if (!sizes_ok(B, H, L, d)) return LA_ERR_SHAPE;
    const int rc = check_kinds(gate_kind, dtype, gate_dtype);
    if (rc != LA_OK) return rc;
    RecArgs a = {};
    a.x = x; a.g = gate; a.dout = dout; a.dx = dx; a.dg = dgate;
    a.chunks_in = chunk_states; a.dh_last = dh_last; a.dh0 = dh0; a.lengths = lengths;
    a.B = B; a.H = H; a.L = L; a.d = d;
    a.vx = make_view(x_strides, H, L, d);
    a.vg = make_view(gate_strides, H, L, d);
    a.vo = make_view(dout_strides, H, L, d);
    a.vdx = make_view(dx_strides, H, L, d);
    a.vdg = make_view(dgate_strides, H, L, d);
    if (!input_view_ok(a.vx, B, H, L) || !input_view_ok(a.vg, B, H, L) || !input_view_ok(a.vo, B, H, L) ||
        !output_view_ok(a.vdx, B, H, L, d) || !output_view_ok(a.vdg, B, H, L, d))
        return LA_ERR_ARG;
    const size_t e = dtype_size(dtype), eg = dtype_size(gate_dtype);
    if (!aligned(x, e) || !aligned(dout, e) || !aligned(dx, e) || !aligned(gate, eg) || !aligned(dgate, eg) ||
        !aligned(chunk_states, 4) || !aligned(dh_last, 4) || !aligned(dh0, 4) || !aligned(lengths, 4))
        return LA_ERR_ARG;
    return dispatch(dtype, gate_dtype, gate_kind, complement != 0, LaunchBwd{a, (cudaStream_t)stream});
}

int la_recurrence_step(const void *x, const void *gate, float *state, void *out, int B, int H,
                       int d, int gate_kind, int complement, int dtype, int gate_dtype,
                       void *stream)
{
    if (!x || !gate || !state || !out) return LA_ERR_NULL;
    if (!sizes_ok(B, H, 1, d)) return LA_ERR_SHAPE;
    const long long n = (long long)B * H * d;
    if (n > (long long)INT_MAX * 64) return LA_ERR_SHAPE;
    const int rc = check_kinds(gate_kind, dtype, gate_dtype);
    if (rc != LA_OK) return rc;
    const size_t e = dtype_size(dtype);
    if (!aligned(x, e) || !aligned(out, e) || !aligned(gate, dtype_size(gate_dtype)) || !aligned(state, 4))
        return LA_ERR_ARG;
    return dispatch(dtype, gate_dtype, gate_kind, complement != 0,
                    LaunchStep{x, gate, state, out, n, (cudaStream_t)stream});
}

}  // extern "C"
