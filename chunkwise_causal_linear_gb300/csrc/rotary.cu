// rotary.cu -- rotary positions: pairs of channels of q and k turned by position times
// frequency (sm_103a).
//
// A frequency is kept as a 64-bit fraction of a full turn per position, so the angle of
// position p is p * turns modulo 2^64: one integer product, exact however far p is.  An fp32
// product p * theta would be off by a radian at p ~ 2^24.
#include <math.h>

#include "layer.cuh"

namespace la {

namespace {

constexpr int ROT_THREADS = 256;

struct RotArgs {
    const void *q, *k;
    void *qo, *ko;
    const unsigned long long *turns;
    const int *pos;
    long long offset;
    View vq, vk, vqo, vko;
    int B, H, Hk, L, d, rot;
    int layout, inverse;
    float amp;
};

// Sine and cosine of 2 pi f / 2^64.  The nearest quarter turn is taken off in integers; what is
// left, at most an eighth of a turn, is exact to an fp32 rounding.
__device__ __forceinline__ void turn_sincos(unsigned long long f, float &s, float &c)
{
    const unsigned q = (unsigned)((f + (1ull << 61)) >> 62);
    const long long r = (long long)(f - ((unsigned long long)q << 62));
    float sr, cr;
    sincospif((float)r * 0x1p-63f, &sr, &cr);
    s = (q & 1) ? cr : sr;
    c = (q & 1) ? sr : cr;
    if (q & 2) s = -s;
    if ((q + 1) & 2) c = -c;
}

template <typename T>
__global__ void __launch_bounds__(ROT_THREADS) rotary_kernel(const RotArgs a)
{
    const int units = a.rot / 2 + (a.d - a.rot);
    const long long n = (long long)a.B * a.L * units;
    const long long i = (long long)blockIdx.x * ROT_THREADS + threadIdx.x;
    if (i >= n) return;
    const int u = (int)(i % units), t = (int)(i / units % a.L), b = (int)(i / units / a.L);
    float s = 0.f, c = 0.f;
    const bool pair = u < a.rot / 2;
    if (pair) {
        const long long p = a.pos ? (long long)a.pos[(size_t)b * a.L + t] : a.offset + t;
        turn_sincos((unsigned long long)p * a.turns[u], s, c);
        s *= a.inverse ? -a.amp : a.amp;
        c *= a.amp;
    }
    const int c0 = pair ? (a.layout == LA_ROTARY_HALF ? u : 2 * u) : a.rot / 2 + u;
    const int c1 = a.layout == LA_ROTARY_HALF ? u + a.rot / 2 : 2 * u + 1;
    for (int h = 0; h < a.H + a.Hk; ++h) {
        const bool isq = h < a.H;
        const int hd = isq ? h : h - a.H;
        const T *in = isq ? (const T *)a.q + row_of(a.vq, b, hd, t) : (const T *)a.k + row_of(a.vk, b, hd, t);
        T *out = isq ? (T *)a.qo + row_of(a.vqo, b, hd, t) : (T *)a.ko + row_of(a.vko, b, hd, t);
        if (pair) {
            const float x = to_f32(in[c0]), y = to_f32(in[c1]);
            out[c0] = from_f32<T>(x * c - y * s);
            out[c1] = from_f32<T>(x * s + y * c);
        } else {
            out[c0] = in[c0];
        }
    }
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

int la_rotary_table(int rot, double base, int scaling, double factor, double original_length,
                    double fast, double slow, unsigned long long *turns)
{
    if (!turns) return LA_ERR_NULL;
    if (rot <= 0 || (rot & 1)) return LA_ERR_SHAPE;
    if (scaling < LA_ROTARY_PLAIN || scaling > LA_ROTARY_PARTS) return LA_ERR_UNSUPPORTED;
    if (!(base > 0.0) || !isfinite(base)) return LA_ERR_ARG;
    if (scaling != LA_ROTARY_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return LA_ERR_ARG;
    if (scaling == LA_ROTARY_PARTS && (!(original_length > 0.0) || !isfinite(original_length) || !(slow > 0.0) ||
                                       !(fast > slow) || !isfinite(fast)))
        return LA_ERR_ARG;
    // 1 / (2 pi) as a sum of two doubles
    const double inv_hi = 0.15915494309189535, inv_lo = -9.839338337591243e-18;
    for (int j = 0; j < rot / 2; ++j) {
        double theta = pow(base, -2.0 * j / rot);
        if (scaling == LA_ROTARY_LINEAR) theta /= factor;
        if (scaling == LA_ROTARY_PARTS) {
            const double r = original_length * theta * inv_hi;  // turns over the original length
            const double keep = fmin(1.0, fmax(0.0, (r - slow) / (fast - slow)));
            theta = theta * keep + theta / factor * (1.0 - keep);
        }
        // theta / (2 pi) to more than a double's digits: the product and its rounding error
        const double hi = theta * inv_hi, lo = fma(theta, inv_hi, -hi) + theta * inv_lo;
        const double whole = floor(hi);
        if (!(whole < 9.0e15)) return LA_ERR_ARG;  // more than 2^53 turns per position
        const double top = (hi - whole) * 0x1p32, top_i = floor(top);
        turns[j] = ((unsigned long long)top_i << 32) + (unsigned long long)((top - top_i) * 0x1p32) +
                   (unsigned long long)llrint(lo * 0x1p64);
    }
    return LA_OK;
}

int la_rotary(const void *q, const void *k, void *q_out, void *k_out,
              const unsigned long long *turns, const int *positions, long long offset, int B,
              int H, int Hk, int L, int d, int rot, const la_strides *q_strides,
              const la_strides *k_strides, const la_strides *q_out_strides,
              const la_strides *k_out_strides, int layout, int inverse, float amplitude,
              int dtype, void *stream)
{
    if (!q || !q_out || (k == nullptr) != (k_out == nullptr)) return LA_ERR_NULL;
    if (rot > 0 && !turns) return LA_ERR_NULL;
    if (!k) Hk = 0;
    if (!sizes_ok(B, H, L, d) || (k && !sizes_ok(B, Hk, L, d))) return LA_ERR_SHAPE;
    if (rot < 0 || rot > d || (rot & 1)) return LA_ERR_SHAPE;
    if (!dtype_ok(dtype)) return LA_ERR_UNSUPPORTED;
    if (layout != LA_ROTARY_HALF && layout != LA_ROTARY_INTERLEAVED) return LA_ERR_UNSUPPORTED;
    if (!isfinite(amplitude)) return LA_ERR_ARG;
    RotArgs a = {};
    a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
    a.turns = turns; a.pos = positions; a.offset = offset;
    a.B = B; a.H = H; a.Hk = Hk; a.L = L; a.d = d; a.rot = rot;
    a.layout = layout; a.inverse = inverse ? 1 : 0;
    a.amp = amplitude;
    a.vq = make_view(q_strides, H, L, d);
    a.vqo = make_view(q_out_strides, H, L, d);
    if (!input_view_ok(a.vq, B, H, L) || !output_view_ok(a.vqo, B, H, L, d)) return LA_ERR_ARG;
    if (k) {
        a.vk = make_view(k_strides, Hk, L, d);
        a.vko = make_view(k_out_strides, Hk, L, d);
        if (!input_view_ok(a.vk, B, Hk, L) || !output_view_ok(a.vko, B, Hk, L, d)) return LA_ERR_ARG;
    }
    const size_t e = dtype_size(dtype);
    if (!aligned(q, e) || !aligned(k, e) || !aligned(q_out, e) || !aligned(k_out, e) || !aligned(turns, 8) ||
        !aligned(positions, 4))
        return LA_ERR_ARG;
    const long long n = (long long)B * L * (rot / 2 + (d - rot)), blocks = (n + ROT_THREADS - 1) / ROT_THREADS;
    if (blocks > INT_MAX) return LA_ERR_SHAPE;
    if (dtype == LA_BF16)
        rotary_kernel<__nv_bfloat16><<<(unsigned)blocks, ROT_THREADS, 0, (cudaStream_t)stream>>>(a);
    else
        rotary_kernel<float><<<(unsigned)blocks, ROT_THREADS, 0, (cudaStream_t)stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // extern "C"
