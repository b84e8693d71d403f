// rotary.cu -- rotary positions: pairs of channels of q and k turned by position times
// frequency (sm_103a).
//
// A frequency is kept as a 64-bit fraction of a full turn per position, so the angle of
// position p is p * turns modulo 2^64: one integer product without a rounding, off by p times what
// the frequency is off (2^-54 of a turn, that of its 64-bit arithmetic).  An fp32 product p * theta
// would be off by a radian at p ~ 2^24.
//
// Bound by memory: every element is read and written once.  A thread holds the sines and cosines
// of VEC pairs (16-byte vectors) of one token and goes over up to 16 heads of q and k with them;
// the first heads' loads are on the way while the sines (~30 instructions a pair) are computed.
#include <math.h>

#include <algorithm>

#include "layer.cuh"

namespace la {

namespace {

constexpr int ROT_THREADS = 256;
constexpr int ROT_HEADS = 16;  // heads of a thread at most (B8 H16 L8192 d128: 167 us, with 8 or 32 171)

// Heads whose loads are on the way together: with 16-byte vectors two (with four the registers leave
// two blocks an SM, 226 us), with single elements four.
template <int VEC> constexpr int ROT_AT_ONCE = VEC > 1 ? 2 : 4;

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
    int heads;  // heads of a thread, q's first, then k's
};

// Sine and cosine of 2 pi f / 2^64, f rounded to 32 bits of a turn.  The nearest quarter turn is
// taken off in integers; what is left, x at most an eighth of a turn, is exact to an fp32
// rounding, and the series of sine and cosine to x^9 and x^10 are off by less than 2e-9 there.
__device__ __forceinline__ void turn_sincos(unsigned long long f, float &s, float &c)
{
    const unsigned hi = (unsigned)((f + 0x80000000ull) >> 32), q = (hi + (1u << 29)) >> 30;
    const float x = (float)(int)(hi - (q << 30)) * (float)(6.283185307179586 / 4294967296.0), z = x * x;
    float p = fmaf(z, 1.f / 362880, -1.f / 5040);
    p = fmaf(z, p, 1.f / 120);
    p = fmaf(z, p, -1.f / 6);
    const float sr = fmaf(x * z, p, x);
    float r = fmaf(z, -1.f / 3628800, 1.f / 40320);
    r = fmaf(z, r, -1.f / 720);
    r = fmaf(z, r, 1.f / 24);
    r = fmaf(z, r, -0.5f);
    const float cr = fmaf(z, r, 1.f);
    s = (q & 1) ? cr : sr;
    c = (q & 1) ? sr : cr;
    if (q & 2) s = -s;
    if ((q + 1) & 2) c = -c;
}

// VEC neighbouring elements as they are stored
template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Vec {
    T v[VEC];
};

// The rows of a token head by head, q's and then k's.
template <typename T> struct HeadRows {
    T *p, *k;
    long long step, kstep;
    int left;  // heads of q still to come
    __device__ HeadRows(const void *q, const View &vq, const void *k_, const View &vk, int H, int b, int t, int h)
        : k((T *)k_ + row_of(vk, b, 0, t)), kstep(vk.h), left(H - h)
    {
        p = left > 0 ? (T *)q + row_of(vq, b, h, t) : k + (h - H) * kstep;
        step = left > 0 ? vq.h : kstep;
    }
    __device__ __forceinline__ void next()
    {
        p += step;
        if (--left == 0) {
            p = k;
            step = kstep;
        }
    }
};

// Unit u of a token: VEC pairs of the rotated channels, or two vectors of the copied ones.
template <typename T, int VEC>
__global__ void __launch_bounds__(ROT_THREADS, 3) rotary_kernel(const RotArgs a)
{
    using V = Vec<T, VEC>;
    const int pair_units = a.rot / (2 * VEC), units = pair_units + (a.d - a.rot + 2 * VEC - 1) / (2 * VEC);
    const unsigned long long n = (unsigned long long)a.B * a.L * units;
    const unsigned long long i = (unsigned long long)blockIdx.x * ROT_THREADS + threadIdx.x;
    if (i >= n) return;
    int u, t, b;
    if (n >> 32) {
        u = (int)(i % units);
        t = (int)(i / units % a.L);
        b = (int)(i / units / a.L);
    } else {
        const unsigned row = (unsigned)i / (unsigned)units;
        u = (int)((unsigned)i - row * units);
        b = (int)(row / (unsigned)a.L);
        t = (int)(row - (unsigned)b * a.L);
    }
    const bool pair = u < pair_units;
    const int h0 = blockIdx.y * a.heads, h1 = min(h0 + a.heads, a.H + a.Hk);
    HeadRows<const T> in(a.q, a.vq, a.k, a.vk, a.H, b, t, h0);
    HeadRows<T> out(a.qo, a.vqo, a.ko, a.vko, a.H, b, t, h0);
    const bool half = a.layout == LA_ROTARY_HALF;
    // the unit's two vectors, half of the turned or copied channels apart, so that neighbouring
    // threads have neighbouring vectors; the elements of a pair where a vector is one
    int c0, c1;
    bool two = true;
    if (pair) {
        const bool apart = half || VEC > 1;
        c0 = apart ? u * VEC : 2 * u;
        c1 = apart ? c0 + a.rot / 2 : c0 + 1;
    } else {
        c0 = a.rot + (u - pair_units) * VEC;
        c1 = c0 + (units - pair_units) * VEC;
        two = c1 < a.d;
        if (!two) c1 = c0;
    }
    constexpr int AT_ONCE = ROT_AT_ONCE<VEC>;
    V x[AT_ONCE], y[AT_ONCE];
    auto fetch = [&](int h) {
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
            if (h + j < h1) {
                x[j] = *(const V *)(in.p + c0);
                y[j] = *(const V *)(in.p + c1);
                in.next();
            }
    };
    fetch(h0);
    float s[VEC], c[VEC];
    if (pair) {
        const unsigned long long p = (unsigned long long)(a.pos ? (long long)a.pos[(size_t)b * a.L + t] : a.offset + t);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            // interleaved vectors hold VEC / 2 pairs each
            const int j = half || VEC == 1 ? u * VEC + e : ((e < VEC / 2 ? c0 : c1 - VEC) >> 1) + e;
            turn_sincos(p * a.turns[j], s[e], c[e]);
            s[e] *= a.inverse ? -a.amp : a.amp;
            c[e] *= a.amp;
        }
    }
    for (int h = h0; h < h1; h += AT_ONCE) {
        if (h != h0) fetch(h);
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
            if (h + j < h1) {
                if (pair && half) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float p = to_f32(x[j].v[e]), q = to_f32(y[j].v[e]);
                        x[j].v[e] = from_f32<T>(p * c[e] - q * s[e]);
                        y[j].v[e] = from_f32<T>(p * s[e] + q * c[e]);
                    }
                } else if (pair) {
                    // elements 2e, 2e + 1 of x then y
                    auto turn = [&](T &m, T &n, int e) {
                        const float p = to_f32(m), q = to_f32(n);
                        m = from_f32<T>(p * c[e] - q * s[e]);
                        n = from_f32<T>(p * s[e] + q * c[e]);
                    };
                    if constexpr (VEC == 1) {
                        turn(x[j].v[0], y[j].v[0], 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < VEC / 2; ++e) {
                            turn(x[j].v[2 * e], x[j].v[2 * e + 1], e);
                            turn(y[j].v[2 * e], y[j].v[2 * e + 1], VEC / 2 + e);
                        }
                    }
                }
                *(V *)(out.p + c0) = x[j];
                if (two) *(V *)(out.p + c1) = y[j];
                out.next();
            }
    }
}

template <typename T, int VEC> int launch_rotary(RotArgs &a, int sms, cudaStream_t s)
{
    const int units = a.rot / (2 * VEC) + (a.d - a.rot + 2 * VEC - 1) / (2 * VEC);
    const long long blocks = ((long long)a.B * a.L * units + ROT_THREADS - 1) / ROT_THREADS;
    if (blocks > INT_MAX) return LA_ERR_SHAPE;
    // heads of a thread: at most ROT_HEADS, in even groups, or half of them, a quarter, ...: where the
    // waves of three blocks an SM, a thread's heads and its sines (as two heads) each, are the least.
    // B1 H8 L4096 d128: 8.6 us with 8 heads, 10 with 4, 15 with 1; B2 H12 L16383 d64: 37.5 with 6 in
    // 4.5 waves, 39 with 12 in 2.2
    const int all = a.H + a.Hk, even = (all + ROT_HEADS - 1) / ROT_HEADS;
    a.heads = (all + even - 1) / even;
    auto groups = [&] { return (all + a.heads - 1) / a.heads; };
    auto cost = [&] { return (blocks * groups() + 3ll * sms - 1) / (3ll * sms) * (a.heads + 2); };
    int best = a.heads;
    for (long long least = cost(); a.heads > 1;) {
        a.heads = (a.heads + 1) / 2;
        if (cost() < least) {
            least = cost();
            best = a.heads;
        }
    }
    a.heads = best;
    while (groups() > 65535) a.heads *= 2;  // limit of the grid
    const int ny = groups();
    return launch(rotary_kernel<T, VEC>, dim3((unsigned)blocks, (unsigned)ny), ROT_THREADS, 0, s, a);
}

template <typename T, int VEC> bool whole_vectors(const RotArgs &a)
{
    auto ok = [&](const void *p, const View &v, int H) {
        return !p || rows_aligned(p, v, a.B, H, a.L, sizeof(T), sizeof(T) * VEC);
    };
    return a.rot % (2 * VEC) == 0 && a.d % VEC == 0 && ok(a.q, a.vq, a.H) && ok(a.qo, a.vqo, a.H) &&
           ok(a.k, a.vk, a.Hk) && ok(a.ko, a.vko, a.Hk);
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
        if (!(whole < 0x1p50)) return LA_ERR_ARG;  // beyond, lo 2^64 leaves 64 bits
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
    const int sms = device_sms();
    if (sms <= 0) return LA_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == LA_F32)
        return whole_vectors<float, 4>(a) ? launch_rotary<float, 4>(a, sms, s) : launch_rotary<float, 1>(a, sms, s);
    if (whole_vectors<__nv_bfloat16, 8>(a)) return launch_rotary<__nv_bfloat16, 8>(a, sms, s);
    return whole_vectors<__nv_bfloat16, 4>(a) ? launch_rotary<__nv_bfloat16, 4>(a, sms, s)
                                              : launch_rotary<__nv_bfloat16, 1>(a, sms, s);
}

}  // extern "C"
