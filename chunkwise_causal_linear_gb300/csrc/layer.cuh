// layer.cuh -- strided [B, H, L, d] views and their checks, and packed fp32 arithmetic, shared by
// the operators that stand around the attention (recurrence, rotary positions, group norm).
#pragma once

#include <limits.h>

#include "common.cuh"

namespace la {

int device_sms();  // SMs of the current device, 0 on an error (api.cu)
int *err_ptr();    // its device error word, NULL on an error

// Element (b, h, t, i) at b * b_ + h * h_ + t * l_ + i.
struct View {
    long long b, h, l;
};

__host__ __device__ inline long long row_of(const View &v, int b, int h, int t)
{
    return b * v.b + h * v.h + t * v.l;
}

// Contiguous [B, H, L, d] (head_major) or [B, L, H, d] where no strides are given.
inline View make_view(const la_strides *s, int H, int L, int d, bool head_major = true)
{
    if (s) return View{s->b, s->h, s->l};
    if (head_major) return View{(long long)H * L * d, (long long)L * d, d};
    return View{(long long)H * L * d, d, (long long)H * d};
}

// Sizes every one of these operators takes: positive, below 2^30 heads in all and 2^20 channels
// (grid limits), and element counts that 64-bit offsets hold with room to spare.
inline bool sizes_ok(int B, int H, int L, int d)
{
    if (B <= 0 || H <= 0 || L <= 0 || d <= 0 || d > (1 << 20)) return false;
    if (L > INT_MAX - (1 << 16)) return false;  // row numbers of a last, partial tile stay ints
    return (double)B * H * L * d < 4.6e18 && (double)B * H < (double)(INT_MAX / 2);
}

inline size_t dtype_size(int dtype) { return dtype == LA_F32 ? 4 : 2; }

inline bool dtype_ok(int dtype) { return dtype == LA_BF16 || dtype == LA_F32; }

inline bool aligned(const void *p, size_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

// Strides of an input: not negative, offsets inside 2^60 elements.
inline bool input_view_ok(const View &v, int B, int H, int L)
{
    const long long s[3] = {v.b, v.h, v.l};
    const int n[3] = {B, H, L};
    __int128 top = 0;
    for (int i = 0; i < 3; ++i) {
        if (s[i] < 0) return false;
        top += (__int128)s[i] * (n[i] - 1);
    }
    return top < ((__int128)1 << 60);
}

// Strides of an output: also no two elements in one place.  Sorted by stride, each axis must
// step over everything the axes below it span.
inline bool output_view_ok(const View &v, int B, int H, int L, int d)
{
    if (!input_view_ok(v, B, H, L)) return false;
    long long s[3] = {v.b, v.h, v.l};
    int n[3] = {B, H, L};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                const long long ts = s[i];
                s[i] = s[j];
                s[j] = ts;
                const int tn = n[i];
                n[i] = n[j];
                n[j] = tn;
            }
    __int128 span = d;  // elements the axes so far span
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (s[i] < span) return false;
        span += (__int128)s[i] * (n[i] - 1);
    }
    return true;
}

// All rows of the view start on `bytes`-byte boundaries.
inline bool rows_aligned(const void *p, const View &v, int B, int H, int L, size_t elem, size_t bytes)
{
    auto ok = [&](long long s, int n) { return n == 1 || (s * (long long)elem) % (long long)bytes == 0; };
    return aligned(p, bytes) && ok(v.b, B) && ok(v.h, H) && ok(v.l, L);
}

// A launch's own status, and no error left behind for the next call to find.
inline int status_of(cudaError_t e)
{
    if (e == cudaSuccess) return LA_OK;
    (void)cudaGetLastError();
    return LA_ERR_CUDA;
}
template <typename... P, typename... A>
inline int launch(void (*kern)(P...), dim3 grid, int block, size_t smem, cudaStream_t stream, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    return status_of(cudaLaunchKernelEx(&cfg, kern, args...));
}

// ---- arithmetic ----------------------------------------------------------------------------
// 2^x and 1/x by the special function unit: relative error 2^-22 and 2^-23, results below the
// normal range flushed to 0.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// V neighbouring values of a thread; pairs use the packed fp32 instructions.
template <int V> struct Ch {
    float v[V];
};
template <int V> __device__ __forceinline__ Ch<V> all(float x)
{
    Ch<V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = x;
    return r;
}
__device__ __forceinline__ Ch<1> fma(Ch<1> a, Ch<1> b, Ch<1> c) { return {{fmaf(a.v[0], b.v[0], c.v[0])}}; }
__device__ __forceinline__ Ch<1> mul(Ch<1> a, Ch<1> b) { return {{a.v[0] * b.v[0]}}; }
__device__ __forceinline__ Ch<1> add(Ch<1> a, Ch<1> b) { return {{a.v[0] + b.v[0]}}; }
__device__ __forceinline__ Ch<2> fma(Ch<2> a, Ch<2> b, Ch<2> c)
{
    Ch<2> r;
    asm("{ .reg .b64 x, y, z, w;\n"
        "mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7};\n"
        "fma.rn.f32x2 w, x, y, z; mov.b64 {%0, %1}, w; }"
        : "=f"(r.v[0]), "=f"(r.v[1])
        : "f"(a.v[0]), "f"(a.v[1]), "f"(b.v[0]), "f"(b.v[1]), "f"(c.v[0]), "f"(c.v[1]));
    return r;
}
__device__ __forceinline__ Ch<2> mul(Ch<2> a, Ch<2> b)
{
    Ch<2> r;
    asm("{ .reg .b64 x, y, w;\n"
        "mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5};\n"
        "mul.rn.f32x2 w, x, y; mov.b64 {%0, %1}, w; }"
        : "=f"(r.v[0]), "=f"(r.v[1]) : "f"(a.v[0]), "f"(a.v[1]), "f"(b.v[0]), "f"(b.v[1]));
    return r;
}
__device__ __forceinline__ Ch<2> add(Ch<2> a, Ch<2> b)
{
    Ch<2> r;
    asm("{ .reg .b64 x, y, w;\n"
        "mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5};\n"
        "add.rn.f32x2 w, x, y; mov.b64 {%0, %1}, w; }"
        : "=f"(r.v[0]), "=f"(r.v[1]) : "f"(a.v[0]), "f"(a.v[1]), "f"(b.v[0]), "f"(b.v[1]));
    return r;
}

__device__ __forceinline__ float min_nan(float x, float y)  // a NaN stays
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float max_nan(float x, float y)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
// e^x to 5 u (u = 2^-24) for x of [-150, 88.7] (or NaN): the power of two 4 u, and what the rounding of
// its argument left out, |x| u and more, multiplied in.
template <int V> __device__ __forceinline__ Ch<V> exp_fine(const Ch<V> &x)
{
    constexpr float LOG2E = 1.44269504f, LN2 = 0.693147182f, LN2_REST = -1.90465432e-9f;  // log 2 = LN2 + LN2_REST
    // e^x = 2^t e^(x - t log 2), whose last exponent is below 2^-16
    const Ch<V> t = mul(x, all<V>(LOG2E)), rest = fma(t, all<V>(-LN2_REST), fma(t, all<V>(-LN2), x));
    Ch<V> e;
#pragma unroll
    for (int v = 0; v < V; ++v) e.v[v] = ex2(t.v[v]);
    return fma(e, rest, e);
}

}  // namespace la
