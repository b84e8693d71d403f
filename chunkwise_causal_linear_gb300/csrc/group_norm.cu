// group_norm.cu -- group norm over one head's channels of one token, with weight, bias and an
// activation or a gate, and its gradients (sm_103a).
//
// One warp per group.  The weight gradients sum over all tokens: a second kernel walks the
// rows per channel with the statistics the first one left in the workspace.
#include <math.h>

#include "layer.cuh"

namespace la {

namespace {

constexpr int GN_THREADS = 256;

struct GnArgs {
    const void *x, *gate, *dout;
    void *out, *dx, *dgate;
    const float *w, *b;
    float *dw, *db, *stats;  // stats: mean and rstd per (b, t, h)
    View vx, vg, vo, vdx, vdg;
    int B, H, L, d, center, act;
    float eps;
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// act(z) and act'(z)
__device__ __forceinline__ float act_of(int act, float z, float &slope)
{
    if (act == LA_ACT_NONE) {
        slope = 1.f;
        return z;
    }
    const float s = sigmoid(z);
    slope = s * (1.f + z * (1.f - s));
    return z * s;
}

template <typename T>
__device__ void group_stats(const GnArgs &a, const T *x, int lane, float &mean, float &rstd)
{
    mean = 0.f;
    if (a.center) {
        float s = 0.f;
        for (int c = lane; c < a.d; c += 32) s += to_f32(x[c]);
        mean = warp_sum(s) / a.d;
    }
    float v = 0.f;
    for (int c = lane; c < a.d; c += 32) {
        const float e = to_f32(x[c]) - mean;
        v = fmaf(e, e, v);
    }
    rstd = rsqrtf(warp_sum(v) / a.d + a.eps);
}

// group i of B * L * H, heads fastest
struct Place {
    int b, h, t;
};
__device__ __forceinline__ Place place_of(const GnArgs &a, long long i)
{
    return Place{(int)(i / a.H / a.L), (int)(i % a.H), (int)(i / a.H % a.L)};
}

template <typename T>
__global__ void __launch_bounds__(GN_THREADS) gn_fwd_kernel(const GnArgs a)
{
    const long long i = ((long long)blockIdx.x * GN_THREADS + threadIdx.x) / 32;
    const int lane = threadIdx.x & 31;
    if (i >= (long long)a.B * a.L * a.H) return;
    const Place p = place_of(a, i);
    const T *x = (const T *)a.x + row_of(a.vx, p.b, p.h, p.t);
    const T *g = a.gate ? (const T *)a.gate + row_of(a.vg, p.b, p.h, p.t) : nullptr;
    T *out = (T *)a.out + row_of(a.vo, p.b, p.h, p.t);
    float mean, rstd, sl;
    group_stats(a, x, lane, mean, rstd);
    for (int c = lane; c < a.d; c += 32) {
        const int wc = p.h * a.d + c;
        const float y = (to_f32(x[c]) - mean) * rstd * (a.w ? a.w[wc] : 1.f) + (a.b ? a.b[wc] : 0.f);
        out[c] = from_f32<T>(g ? y * act_of(a.act, to_f32(g[c]), sl) : act_of(a.act, y, sl));
    }
}

// dy of one channel (and dgate)
template <typename T>
__device__ __forceinline__ float grad_y(const GnArgs &a, float xh, float w, float b, const T *g, float dout, int c,
                                        float &dgate)
{
    const float y = xh * w + b;
    float sl;
    if (g) {
        const float act = act_of(a.act, to_f32(g[c]), sl);
        dgate = dout * y * sl;
        return dout * act;
    }
    act_of(a.act, y, sl);
    dgate = 0.f;
    return dout * sl;
}

template <typename T>
__global__ void __launch_bounds__(GN_THREADS) gn_bwd_kernel(const GnArgs a)
{
    const long long i = ((long long)blockIdx.x * GN_THREADS + threadIdx.x) / 32;
    const int lane = threadIdx.x & 31;
    if (i >= (long long)a.B * a.L * a.H) return;
    const Place p = place_of(a, i);
    const T *x = (const T *)a.x + row_of(a.vx, p.b, p.h, p.t);
    const T *g = a.gate ? (const T *)a.gate + row_of(a.vg, p.b, p.h, p.t) : nullptr;
    const T *dout = (const T *)a.dout + row_of(a.vo, p.b, p.h, p.t);
    T *dx = (T *)a.dx + row_of(a.vdx, p.b, p.h, p.t);
    T *dg = a.gate ? (T *)a.dgate + row_of(a.vdg, p.b, p.h, p.t) : nullptr;
    float mean, rstd, dgv;
    group_stats(a, x, lane, mean, rstd);
    float s1 = 0.f, s2 = 0.f;
    for (int c = lane; c < a.d; c += 32) {
        const int wc = p.h * a.d + c;
        const float xh = (to_f32(x[c]) - mean) * rstd, w = a.w ? a.w[wc] : 1.f;
        const float e = grad_y(a, xh, w, a.b ? a.b[wc] : 0.f, g, to_f32(dout[c]), c, dgv) * w;
        s1 += e;
        s2 = fmaf(e, xh, s2);
    }
    s1 = a.center ? warp_sum(s1) / a.d : 0.f;
    s2 = warp_sum(s2) / a.d;
    for (int c = lane; c < a.d; c += 32) {
        const int wc = p.h * a.d + c;
        const float xh = (to_f32(x[c]) - mean) * rstd, w = a.w ? a.w[wc] : 1.f;
        const float e = grad_y(a, xh, w, a.b ? a.b[wc] : 0.f, g, to_f32(dout[c]), c, dgv) * w;
        dx[c] = from_f32<T>(rstd * (e - s1 - xh * s2));
        if (dg) dg[c] = from_f32<T>(dgv);
    }
    if (a.stats && lane == 0) {
        a.stats[2 * i] = mean;
        a.stats[2 * i + 1] = rstd;
    }
}

// one block per 32 channels of a head: 8 warps walk the tokens
template <typename T>
__global__ void __launch_bounds__(GN_THREADS) gn_weight_kernel(const GnArgs a)
{
    __shared__ float sw[8][32], sb[8][32];
    const int h = blockIdx.x, c = blockIdx.y * 32 + (threadIdx.x & 31), warp = threadIdx.x / 32;
    const bool on = c < a.d;
    const int wc = h * a.d + c;
    const float w = on && a.w ? a.w[wc] : 1.f, bias = on && a.b ? a.b[wc] : 0.f;
    float aw = 0.f, ab = 0.f, dgv;
    if (on)
        for (long long r = warp; r < (long long)a.B * a.L; r += 8) {
            const int b = (int)(r / a.L), t = (int)(r % a.L);
            const T *x = (const T *)a.x + row_of(a.vx, b, h, t);
            const T *g = a.gate ? (const T *)a.gate + row_of(a.vg, b, h, t) : nullptr;
            const T *dout = (const T *)a.dout + row_of(a.vo, b, h, t);
            const float xh = (to_f32(x[c]) - a.stats[2 * (r * a.H + h)]) * a.stats[2 * (r * a.H + h) + 1];
            const float dy = grad_y(a, xh, w, bias, g, to_f32(dout[c]), c, dgv);
            aw = fmaf(dy, xh, aw);
            ab += dy;
        }
    sw[warp][threadIdx.x & 31] = aw;
    sb[warp][threadIdx.x & 31] = ab;
    __syncthreads();
    if (warp == 0 && on) {
        for (int i = 1; i < 8; ++i) {
            aw += sw[i][threadIdx.x];
            ab += sb[i][threadIdx.x];
        }
        if (a.dw) a.dw[wc] = aw;
        if (a.db) a.db[wc] = ab;
    }
}

int check_act(int activation, float eps, int dtype)
{
    if (!dtype_ok(dtype)) return LA_ERR_UNSUPPORTED;
    if (activation != LA_ACT_NONE && activation != LA_ACT_SILU) return LA_ERR_UNSUPPORTED;
    if (!(eps > 0.f) || !isfinite(eps)) return LA_ERR_ARG;
    return LA_OK;
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

int la_group_norm_fwd(const void *x, const float *weight, const float *bias, const void *gate,
                      void *out, int B, int H, int L, int d, const la_strides *x_strides,
                      const la_strides *gate_strides, const la_strides *out_strides, int center,
                      int activation, float eps, int dtype, void *stream)
{
    if (!x || !out) return LA_ERR_NULL;
    if (!sizes_ok(B, H, L, d)) return LA_ERR_SHAPE;
    const int rc = check_act(activation, eps, dtype);
    if (rc != LA_OK) return rc;
    GnArgs a = {};
    a.x = x; a.w = weight; a.b = bias; a.gate = gate; a.out = out;
    a.B = B; a.H = H; a.L = L; a.d = d;
    a.center = center ? 1 : 0; a.act = activation; a.eps = eps;
    a.vx = make_view(x_strides, H, L, d);
    a.vg = make_view(gate_strides, H, L, d, false);
    a.vo = make_view(out_strides, H, L, d, false);
    if (!input_view_ok(a.vx, B, H, L) || (gate && !input_view_ok(a.vg, B, H, L)) || !output_view_ok(a.vo, B, H, L, d))
        return LA_ERR_ARG;
    const size_t e = dtype_size(dtype);
    if (!aligned(x, e) || !aligned(gate, e) || !aligned(out, e) || !aligned(weight, 4) || !aligned(bias, 4))
        return LA_ERR_ARG;
    const long long blocks = ((long long)B * L * H + GN_THREADS / 32 - 1) / (GN_THREADS / 32);
    if (blocks > INT_MAX) return LA_ERR_SHAPE;
    if (dtype == LA_BF16)
        gn_fwd_kernel<__nv_bfloat16><<<(unsigned)blocks, GN_THREADS, 0, (cudaStream_t)stream>>>(a);
    else
        gn_fwd_kernel<float><<<(unsigned)blocks, GN_THREADS, 0, (cudaStream_t)stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

size_t la_group_norm_bwd_workspace_bytes(int B, int H, int L, int d)
{
    if (!sizes_ok(B, H, L, d)) return 0;
    return (size_t)B * H * L * 2 * sizeof(float);
}

int la_group_norm_bwd(const void *x, const float *weight, const float *bias, const void *gate,
                      const void *dout, void *dx, void *dgate, float *dweight, float *dbias,
                      int B, int H, int L, int d, const la_strides *x_strides,
                      const la_strides *gate_strides, const la_strides *dout_strides,
                      const la_strides *dx_strides, const la_strides *dgate_strides, int center,
                      int activation, float eps, int dtype, void *workspace,
                      size_t workspace_bytes, void *stream)
{
    if (!x || !dout || !dx || (gate == nullptr) != (dgate == nullptr)) return LA_ERR_NULL;
    if (!sizes_ok(B, H, L, d)) return LA_ERR_SHAPE;
    const int rc = check_act(activation, eps, dtype);
    if (rc != LA_OK) return rc;
    GnArgs a = {};
    a.x = x; a.w = weight; a.b = bias; a.gate = gate; a.dout = dout;
    a.dx = dx; a.dgate = dgate; a.dw = dweight; a.db = dbias;
    a.B = B; a.H = H; a.L = L; a.d = d;
    a.center = center ? 1 : 0; a.act = activation; a.eps = eps;
    a.vx = make_view(x_strides, H, L, d);
    a.vg = make_view(gate_strides, H, L, d, false);
    a.vo = make_view(dout_strides, H, L, d, false);
    a.vdx = make_view(dx_strides, H, L, d);
    a.vdg = make_view(dgate_strides, H, L, d, false);
    if (!input_view_ok(a.vx, B, H, L) || (gate && !input_view_ok(a.vg, B, H, L)) || !input_view_ok(a.vo, B, H, L) ||
        !output_view_ok(a.vdx, B, H, L, d) || (gate && !output_view_ok(a.vdg, B, H, L, d)))
        return LA_ERR_ARG;
    const size_t e = dtype_size(dtype);
    if (!aligned(x, e) || !aligned(gate, e) || !aligned(dout, e) || !aligned(dx, e) || !aligned(dgate, e) ||
        !aligned(weight, 4) || !aligned(bias, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return LA_ERR_ARG;
    if (dweight || dbias) {
        if (!workspace || workspace_bytes < la_group_norm_bwd_workspace_bytes(B, H, L, d)) return LA_ERR_WORKSPACE;
        if (!aligned(workspace, 4)) return LA_ERR_ARG;
        a.stats = (float *)workspace;
    }
    const long long blocks = ((long long)B * L * H + GN_THREADS / 32 - 1) / (GN_THREADS / 32);
    if (blocks > INT_MAX) return LA_ERR_SHAPE;
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == LA_BF16)
        gn_bwd_kernel<__nv_bfloat16><<<(unsigned)blocks, GN_THREADS, 0, s>>>(a);
    else
        gn_bwd_kernel<float><<<(unsigned)blocks, GN_THREADS, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return LA_ERR_CUDA;
    if (a.stats) {
        const dim3 grid((unsigned)H, (unsigned)((d + 31) / 32));
        if (dtype == LA_BF16)
            gn_weight_kernel<__nv_bfloat16><<<grid, GN_THREADS, 0, s>>>(a);
        else
            gn_weight_kernel<float><<<grid, GN_THREADS, 0, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return LA_ERR_CUDA;
    }
    return LA_OK;
}

}  // extern "C"
