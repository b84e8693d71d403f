// block_norm.cu -- the norms around a block, fused with its gate and the residual sum (sm_103a):
//
//     h = residual_scale r + branch_scale act(gate) (norm(y) w_post + b_post),
//     n = norm(h) w_pre + b_pre,
//
// and the gradients of both. norm is the root mean square's (x / sqrt(mean(x^2) + eps)), the layer's
// (centred first) or none (y as it is: w_post is a layer scale then).
//
// Bound by memory: y, r and gate are read once, h and n written once; apart, the two norms, the gate and the
// sum would read and write h and the norm's output once more each. A row is held in the registers of NT
// threads, 8 channels each (16 in rows above 1536), so that its statistics, centred variance and
// both norms come from that one read. Each thread copies its channels of the next rows ahead into places of
// its own in shared memory (cp.async, a ring of rows, no barrier), which costs no registers and hides the
// sums' barriers; rows that cannot be read 16 bytes at a time are loaded one row ahead, forwards. The gradients
// recompute the statistics from y and r (32-bit sums; h before its rounding) instead of reading them, and keep
// the sums for the weights' gradients in the threads' registers; the groups' sums are joined by a second kernel in a
// fixed order. Forwards the copies bind (B8 L8192 d2048 229 us, 86% of the measured copy rate), the gradients are bound
// by up to five sums over the row's threads, one after the other, and their instructions (480 us, 66%; of the schedulers'
// slots 45% are used).
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "layer.cuh"
#include "tc_common.cuh"

namespace la {

namespace {

constexpr int BN_MAX_D = 8192;
constexpr int BN_SIGMOID = LA_ACT_SIGMOID;

struct BnArgs {
    const void *y, *r, *gate, *dh, *dn;
    void *h, *n, *dr, *dy, *dgate;
    const float *post_w, *post_b, *pre_w, *pre_b;
    float *part;  // [blocks][4][d]: sums for post_w, pre_w, post_b, pre_b
    int sums;     // bit k: the k-th of them is wanted
    View vy, vr, vg, vh, vn, vdh, vdn, vdr, vdy, vdg;
    long long rows;
    int L, d, post, pre, act;
    float rs, bs, eps, inv_d;
};

// ---- VEC neighbouring channels as they lie in memory, and as fp32 ------------------------------
template <typename T, int VEC> struct Raw;
template <> struct Raw<__nv_bfloat16, 8> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *(const uint4 *)p; }
    __device__ __forceinline__ void get(float *f) const
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = tcc::bf_lo(u[i]);
            f[2 * i + 1] = tcc::bf_hi(u[i]);
        }
    }
};
template <> struct Raw<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = ((const float4 *)p)[0];
        b = ((const float4 *)p)[1];
    }
    __device__ __forceinline__ void get(float *f) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};
template <typename T> struct Raw<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void get(float *f) const { f[0] = to_f32(v); }
};
template <int VEC> __device__ __forceinline__ void put(__nv_bfloat16 *p, const float *f)
{
    if constexpr (VEC == 8) {
        *(uint4 *)p = make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]), ptx::pack_bf16x2(f[4], f[5]),
                                 ptx::pack_bf16x2(f[6], f[7]));
    } else {
        *p = __float2bfloat16_rn(f[0]);
    }
}
template <int VEC> __device__ __forceinline__ void put(float *p, const float *f)
{
    if constexpr (VEC == 8) {
        ((float4 *)p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        ((float4 *)p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *p = f[0];
    }
}
// VEC values of a vector of weights, `one` where there is none
template <int VEC> __device__ __forceinline__ void weights(const float *w, int c, float one, float *f)
{
    if (!w) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = one;
    } else if constexpr (VEC == 8) {
        const float4 a = __ldg((const float4 *)(w + c)), b = __ldg((const float4 *)(w + c) + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        f[0] = __ldg(w + c);
    }
}

// A thread's N channels as pairs for the packed instructions, or one by one.
template <int VEC> constexpr int WIDTH = VEC > 1 ? 2 : 1;
template <int W> __device__ __forceinline__ Ch<W> less(const Ch<W> &x, const Ch<W> &y) { return fma(y, all<W>(-1.f), x); }
template <int W, int M> __device__ __forceinline__ float over(const Ch<W> (&x)[M])  // sum
{
    Ch<W> s = x[0];
#pragma unroll
    for (int i = 1; i < M; ++i) s = add(s, x[i]);
    return W == 2 ? s.v[0] + s.v[W - 1] : s.v[0];
}
template <int W, int M> __device__ __forceinline__ float over(const Ch<W> (&x)[M], const Ch<W> (&y)[M])  // of products
{
    Ch<W> s = mul(x[0], y[0]);
#pragma unroll
    for (int i = 1; i < M; ++i) s = fma(x[i], y[i], s);
    return W == 2 ? s.v[0] + s.v[W - 1] : s.v[0];
}

// ---- sums over the threads of a row, the same in every one of them -----------------------------
// Two places in turn, so that one barrier a sum is enough: who writes a place again has passed the
// barrier behind the sum that everyone read it for.
template <int NT, bool WHOLE> struct Sums {  // WHOLE: the row's threads are the block
    float *sm;  // [2][NT / 32][2]
    int turn = 0;
    template <int N> __device__ __forceinline__ void operator()(float (&v)[N])
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if constexpr (NT > 32) {
            constexpr int W = NT / 32;
            const int t = threadIdx.x % NT;
            float *p = sm + turn * W * 2;
            turn ^= 1;
            if ((t & 31) == 0) *(float2 *)(p + (t >> 5) * 2) = make_float2(v[0], N > 1 ? v[N - 1] : 0.f);
            if constexpr (WHOLE) __syncthreads();
            else ptx::named_bar(1 + threadIdx.x / NT, NT);
            Ch<2> s = all<2>(0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float2 q = *(const float2 *)(p + w * 2);
                s = add(s, Ch<2>{{q.x, q.y}});
            }
            v[0] = s.v[0];
            if (N > 1) v[N - 1] = s.v[1];
        }
    }
};

// s = 1 / (1 + e^-z) and 1 - s, both from e^-|z|: the smaller one is e / (1 + e), so neither is a difference, and a slope of
// s (1 - s) is as exact far out as near 0. For fp32 by the exact division and exponential; for bf16, whose outputs are
// rounded by up to 2^-8, to (5 + |z|) 2^-23, and 0 where e^-|z| is below the normal range (|z| > 87.3). Without a SLOPE to
// form bf16 needs no e^-|z|: s is as exact from e^-z, and takes less (B8 L8192 d2048 forward 228 us, 231 otherwise).
template <typename T, bool SLOPE> __device__ __forceinline__ void sigmoid(float z, float &s, float &rest)
{
    if constexpr (!SLOPE && !std::is_same<T, float>::value) {
        s = rcp(1.f + ex2(-1.44269504f * z));
        return;
    }
    float e, large;
    if constexpr (std::is_same<T, float>::value) {
        e = expf(-fabsf(z));
        large = 1.f / (1.f + e);
    } else {
        e = ex2(-1.44269504f * fabsf(z));
        large = rcp(1.f + e);
    }
    const float small = e * large;
    s = z < 0.f ? small : large;
    rest = z < 0.f ? large : small;
}

// Channels of chunks that are not there, back to 0.
template <int VEC, int W, int M, int NC> __device__ __forceinline__ void clear(Ch<W> (&x)[M], const bool (&in)[NC])
{
#pragma unroll
    for (int i = 0; i < M; ++i)
        if (!in[i * W / VEC]) x[i] = all<W>(0.f);
}

// A row's 1/deviation; x centred in place where the kind asks for it.
template <int VEC, int W, int M, int NC, typename S>
__device__ __forceinline__ float statistics(Ch<W> (&x)[M], const bool (&in)[NC], int kind, const BnArgs &a, S &sum)
{
    if (kind == LA_NORM_LAYER) {
        float m[1] = {over(x)};
        sum(m);
        const Ch<W> mean = all<W>(m[0] * a.inv_d);
#pragma unroll
        for (int i = 0; i < M; ++i) x[i] = less(x[i], mean);
        clear<VEC>(x, in);
    }
    float s[1] = {over(x, x)};
    sum(s);
    return rsqrtf(fmaf(s[0], a.inv_d, a.eps));
}

// Row numbers b, t of B x L stepping by a fixed number of rows, without a division a row.
struct RowAt {
    int b, t;
    __device__ __forceinline__ RowAt(long long row, int L) : b((int)(row / L)), t((int)(row % L)) {}
    __device__ __forceinline__ void next(int step_b, int step_t, int L)
    {
        b += step_b;
        t += step_t;
        if (t >= L) {
            t -= L;
            ++b;
        }
    }
};

template <int NT, bool BWD> constexpr int bn_block = BWD ? (128 % NT == 0 ? 128 : NT) : 256 % NT == 0 ? 256 : NT < 192 ? 192 : NT;
// Threads of the gradients' kernel that an SM is to hold, and with that the registers of each (128 or 168): 16 channels
// of a row of up to 2048 spill at 128 with the biases' sums (B8 L8192 d2048 580 us, 711 at 128; fp32 d2048 without them 585 and
// 627; bf16 without them fit: 480 and 450), longer rows are waited for too long with one block (B4 L4096 d4096 240 us with
// two of 256, 335 with one).
template <int NT, int NC> constexpr int bn_threads = NC == 1 || (NC == 2 && NT >= 256) ? 512 : 384;
template <int NT, int NC>
constexpr int bn_held = bn_threads<NT, NC> < bn_block<NT, true> ? 1 : bn_threads<NT, NC> / bn_block<NT, true>;

// Rows on their way to a thread: three, or what the threads of an SM can have of its shared memory.
template <int VEC, int STAGE, int BLOCK, int THREADS = 384>
constexpr int AHEAD = VEC != 8 ? 1 : 3 * STAGE <= std::min(BLOCK * (221184 / THREADS), 204800) ? 3
                               : 2 * STAGE <= std::min(BLOCK * (221184 / THREADS), 204800) ? 2 : 1;

__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A thread's channels of a tensor, some rows ahead: ring places in shared memory for vectors, registers one
// row ahead for single channels.
template <typename X, int VEC, int NC, int BLOCK> struct Ahead {
    static constexpr int BYTES = VEC == 8 ? NC * BLOCK * 8 * (int)sizeof(X) : 0;  // of one row of the block
    Raw<X, VEC> raw[VEC == 8 ? 1 : NC];
    uint32_t base;  // this thread's place in the ring's first row
    int step;       // bytes between rows of the ring
    __device__ __forceinline__ void place(uint32_t smem, int stage_bytes)
    {
        base = smem + threadIdx.x * 16;
        step = stage_bytes;
    }
    __device__ __forceinline__ void fetch(const X *p, int slot, const int (&at)[NC], int d)
    {
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (at[c] < d) {
                if constexpr (VEC == 8) {
#pragma unroll
                    for (int h = 0; h < (int)sizeof(X) / 2; ++h)
                        copy16(base + slot * step + (c * (int)sizeof(X) / 2 + h) * BLOCK * 16, p + at[c] + h * 4);
                } else {
                    raw[c].load(p + at[c]);
                }
            }
    }
    __device__ __forceinline__ void get(float *f, int slot, int c) const
    {
        if constexpr (VEC == 8) {
            const uint32_t a = base + slot * step + c * ((int)sizeof(X) / 2) * BLOCK * 16;
            const uint4 u = ptx::lds128(a);
            Raw<X, 8> r;
            if constexpr (sizeof(X) == 2) {
                r.w = u;
            } else {
                const uint4 v = ptx::lds128(a + BLOCK * 16);
                r.a = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
                r.b = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
            }
            r.get(f);
        } else {
            raw[c].get(f);
        }
    }
};
template <int VEC> __device__ __forceinline__ void row_issued()
{
    if constexpr (VEC == 8) asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int VEC, int PF> __device__ __forceinline__ void row_arrived()
{
    if constexpr (VEC == 8) asm volatile("cp.async.wait_group %0;" ::"n"(PF - 1) : "memory");
}

// What both kernels begin with: the row group's first row, its channels, and the gate's activation.
#define BN_ROWS(STEP_ROWS)                                                                                             \
    constexpr int N = VEC * NC, W = WIDTH<VEC>, M = N / W, GROUPS = BLOCK / NT;                                         \
    __shared__ __align__(16) float sm[GROUPS * 2 * (NT / 32) * 2];                                                       \
    const int tid = threadIdx.x % NT, group = threadIdx.x / NT;                                                        \
    Sums<NT, GROUPS == 1> sum{sm + group * 2 * (NT / 32) * 2};                                                          \
    const long long first = (long long)blockIdx.x * GROUPS + group, STEP_ROWS = (long long)gridDim.x * GROUPS;          \
    const int step_b = (int)(STEP_ROWS / a.L), step_t = (int)(STEP_ROWS % a.L);                                         \
    int at[NC];                                                                                                         \
    bool in[NC];                                                                                                        \
    _Pragma("unroll") for (int c = 0; c < NC; ++c)                                                                      \
    {                                                                                                                   \
        at[c] = (c * NT + tid) * VEC;                                                                                   \
        in[c] = at[c] < a.d;                                                                                            \
    }

// V channels of a chunk at f as pairs
template <int W, int M> __device__ __forceinline__ float *flat(Ch<W> (&x)[M], int i) { return &x[i / W].v[i % W]; }

// act(z), and its slope where it is not 1.
template <typename T, bool SLOPE, int W, int M>
__device__ __forceinline__ void activate(const Ch<W> (&z)[M], Ch<W> (&slope)[M], Ch<W> (&act)[M], const BnArgs &a)
{
#pragma unroll
    for (int i = 0; i < M; ++i) {
        if (!a.gate) {
            act[i] = all<W>(1.f);
        } else if (a.act == LA_ACT_NONE) {
            act[i] = z[i];
        } else {
            Ch<W> s, rest;
#pragma unroll
            for (int u = 0; u < W; ++u) sigmoid<T, SLOPE>(z[i].v[u], s.v[u], rest.v[u]);
            act[i] = a.act == LA_ACT_SILU ? mul(z[i], s) : s;
            if constexpr (SLOPE) slope[i] = mul(s, a.act == LA_ACT_SILU ? fma(z[i], rest, all<W>(1.f)) : rest);
        }
    }
}

template <typename T, typename R, int VEC, int NT, int NC>
__global__ void __launch_bounds__(bn_block<NT, false>, 1) bn_fwd_kernel(const BnArgs a)
{
    constexpr int BLOCK = bn_block<NT, false>;
    BN_ROWS(step)
    extern __shared__ __align__(16) uint8_t ring[];
    constexpr int BT = Ahead<T, VEC, NC, BLOCK>::BYTES, BR = Ahead<R, VEC, NC, BLOCK>::BYTES, STAGE = 2 * BT + BR,
                  PF = AHEAD<VEC, STAGE, BLOCK>;
    Ahead<T, VEC, NC, BLOCK> ry, rg;
    Ahead<R, VEC, NC, BLOCK> rr;
    const uint32_t ring_at = ptx::smem_u32(ring);
    ry.place(ring_at, STAGE);
    rg.place(ring_at + BT, STAGE);
    rr.place(ring_at + 2 * BT, STAGE);
    RowAt ahead(first, a.L), now(first, a.L);
    auto fetch = [&](long long row, int slot) {
        if (row < a.rows) {
            ry.fetch((const T *)a.y + row_of(a.vy, ahead.b, 0, ahead.t), slot, at, a.d);
            rr.fetch((const R *)a.r + row_of(a.vr, ahead.b, 0, ahead.t), slot, at, a.d);
            if (a.gate) rg.fetch((const T *)a.gate + row_of(a.vg, ahead.b, 0, ahead.t), slot, at, a.d);
        }
        ahead.next(step_b, step_t, a.L);
        row_issued<VEC>();
    };
#pragma unroll
    for (int i = 0; i < PF; ++i) fetch(first + i * step, i);
    int slot = 0;
    for (long long row = first; row < a.rows; row += step, slot = slot + 1 == PF ? 0 : slot + 1) {
        Ch<W> u[M], h[M], act[M];
        {
            Ch<W> z[M], slope[M];
#pragma unroll
            for (int i = 0; i < M; ++i) u[i] = h[i] = z[i] = all<W>(0.f);
            row_arrived<VEC, PF>();
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (in[c]) {
                    ry.get(flat(u, c * VEC), slot, c);
                    rr.get(flat(h, c * VEC), slot, c);
                    if (a.gate) rg.get(flat(z, c * VEC), slot, c);
                }
            fetch(row + PF * step, slot);
            activate<T, false>(z, slope, act, a);
        }
        const Ch<W> k1 = all<W>(a.bs * (a.post == LA_NORM_NONE ? 1.f : statistics<VEC>(u, in, a.post, a, sum))), bs = all<W>(a.bs),
                    rs = all<W>(a.rs);
        R *const ho = (R *)a.h + row_of(a.vh, now.b, 0, now.t);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (in[c]) {
                Ch<W> w[VEC / W], bias[VEC / W];
                weights<VEC>(a.post_w, at[c], 1.f, w[0].v);
                if (a.post_b) weights<VEC>(a.post_b, at[c], 0.f, bias[0].v);
#pragma unroll
                for (int i = 0; i < VEC / W; ++i) {
                    const int m = c * VEC / W + i;
                    Ch<W> x = mul(mul(u[m], k1), w[i]);
                    if (a.post_b) x = fma(bias[i], bs, x);
                    h[m] = fma(act[m], x, mul(rs, h[m]));
                }
                put<VEC>(ho + at[c], flat(h, c * VEC));
            }
        if (a.n) {
            const Ch<W> k2 = all<W>(statistics<VEC>(h, in, a.pre, a, sum));
            T *const no = (T *)a.n + row_of(a.vn, now.b, 0, now.t);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (in[c]) {
                    Ch<W> w[VEC / W], bias[VEC / W], o[VEC / W];
                    weights<VEC>(a.pre_w, at[c], 1.f, w[0].v);
                    weights<VEC>(a.pre_b, at[c], 0.f, bias[0].v);
#pragma unroll
                    for (int i = 0; i < VEC / W; ++i) o[i] = fma(mul(h[c * VEC / W + i], k2), w[i], bias[i]);
                    put<VEC>(no + at[c], o[0].v);
                }
        }
        now.next(step_b, step_t, a.L);
    }
}

// dx of x/deviation (centred) from dxh, in place, with xh: (dxh - xh mean(dxh xh) [- mean(dxh)]) k.
template <int VEC, int W, int M, int NC, typename S>
__device__ __forceinline__ void norm_back(Ch<W> (&dxh)[M], const Ch<W> (&xh)[M], const bool (&in)[NC], float k, int kind, const BnArgs &a,
                                          S &sum)
{
    float s[2] = {over(dxh, xh), kind == LA_NORM_LAYER ? over(dxh) : 0.f};
    sum(s);
    const Ch<W> m0 = all<W>(-s[0] * a.inv_d), m1 = all<W>(-s[1] * a.inv_d), kk = all<W>(k);
#pragma unroll
    for (int i = 0; i < M; ++i) dxh[i] = mul(add(dxh[i], fma(xh[i], m0, m1)), kk);  // k last: what cancels is not scaled up first
    if (kind == LA_NORM_LAYER) clear<VEC>(dxh, in);
}

// BIAS: sums for the biases too.
template <typename T, typename R, int VEC, int NT, int NC, bool BIAS>
__global__ void __launch_bounds__(bn_block<NT, true>, bn_held<NT, NC>) bn_bwd_kernel(const BnArgs a)
{
    constexpr int BLOCK = bn_block<NT, true>;
    BN_ROWS(step)
    extern __shared__ __align__(16) uint8_t ring[];
    constexpr int BT = Ahead<T, VEC, NC, BLOCK>::BYTES, BR = Ahead<R, VEC, NC, BLOCK>::BYTES,
                  STAGE = 3 * BT + 2 * BR, PF = AHEAD<VEC, STAGE, BLOCK, bn_threads<NT, NC>>;
    Ch<W> total[BIAS ? 4 : 2][M];  // post_w, pre_w, post_b, pre_b
#pragma unroll
    for (int k = 0; k < (BIAS ? 4 : 2); ++k)
#pragma unroll
        for (int i = 0; i < M; ++i) total[k][i] = all<W>(0.f);
    Ahead<T, VEC, NC, BLOCK> ry, rg, rdn;
    Ahead<R, VEC, NC, BLOCK> rr, rdh;
    const uint32_t ring_at = ptx::smem_u32(ring);
    ry.place(ring_at, STAGE);
    rg.place(ring_at + BT, STAGE);
    rdn.place(ring_at + 2 * BT, STAGE);
    rr.place(ring_at + 3 * BT, STAGE);
    rdh.place(ring_at + 3 * BT + BR, STAGE);
    RowAt ahead(first, a.L), now(first, a.L);
    auto fetch = [&](long long row, int slot) {
        if (row < a.rows) {
            ry.fetch((const T *)a.y + row_of(a.vy, ahead.b, 0, ahead.t), slot, at, a.d);
            rr.fetch((const R *)a.r + row_of(a.vr, ahead.b, 0, ahead.t), slot, at, a.d);
            if (a.gate) rg.fetch((const T *)a.gate + row_of(a.vg, ahead.b, 0, ahead.t), slot, at, a.d);
            if (a.dh) rdh.fetch((const R *)a.dh + row_of(a.vdh, ahead.b, 0, ahead.t), slot, at, a.d);
            if (a.dn) rdn.fetch((const T *)a.dn + row_of(a.vdn, ahead.b, 0, ahead.t), slot, at, a.d);
        }
        ahead.next(step_b, step_t, a.L);
        row_issued<VEC>();
    };
#pragma unroll
    for (int i = 0; i < PF; ++i) fetch(first + i * step, i);
    int slot = 0;
    for (long long row = first; row < a.rows; row += step, slot = slot + 1 == PF ? 0 : slot + 1) {
        // what is needed late (dn and dh) stays in the ring until then: registers held over
        // the sums are what the kernel has least of
        Ch<W> u[M], h[M], slope[M], act[M], dh[M];
        row_arrived<VEC, PF>();
        {
            Ch<W> z[M];
#pragma unroll
            for (int i = 0; i < M; ++i) u[i] = h[i] = z[i] = dh[i] = all<W>(0.f);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (in[c]) {
                    ry.get(flat(u, c * VEC), slot, c);
                    rr.get(flat(h, c * VEC), slot, c);
                    if (a.gate) rg.get(flat(z, c * VEC), slot, c);
                }
            activate<T, true>(z, slope, act, a);
        }
        const float k1 = a.post == LA_NORM_NONE ? 1.f : statistics<VEC>(u, in, a.post, a, sum);
        const Ch<W> k1w = all<W>(k1), bs = all<W>(a.bs), rs = all<W>(a.rs);
        // x = w xh + b of the norm behind the block
        auto post = [&](int c, Ch<W> (&w)[VEC / W], Ch<W> (&x)[VEC / W]) {
            weights<VEC>(a.post_w, at[c], 1.f, w[0].v);
#pragma unroll
            for (int i = 0; i < VEC / W; ++i) x[i] = mul(u[c * VEC / W + i], w[i]);
            if (a.post_b) {
                Ch<W> bias[VEC / W];
                weights<VEC>(a.post_b, at[c], 0.f, bias[0].v);
#pragma unroll
                for (int i = 0; i < VEC / W; ++i) x[i] = add(x[i], bias[i]);
            }
        };
#pragma unroll
        for (int i = 0; i < M; ++i) {
            u[i] = mul(u[i], k1w);  // xh of y from here on
            act[i] = mul(act[i], bs);
        }
        if (a.dn) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (in[c]) {
                    Ch<W> w[VEC / W], x[VEC / W];
                    post(c, w, x);
#pragma unroll
                    for (int i = 0; i < VEC / W; ++i) {
                        const int m = c * VEC / W + i;
                        h[m] = fma(act[m], x[i], mul(rs, h[m]));
                    }
                }
            const float k2 = statistics<VEC>(h, in, a.pre, a, sum);
            const Ch<W> k2w = all<W>(k2);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (in[c]) {
                    Ch<W> w[VEC / W], dn[VEC / W];
                    rdn.get(dn[0].v, slot, c);
                    weights<VEC>(a.pre_w, at[c], 1.f, w[0].v);
#pragma unroll
                    for (int i = 0; i < VEC / W; ++i) {
                        const int m = c * VEC / W + i;
                        h[m] = mul(h[m], k2w);
                        total[1][m] = fma(dn[i], h[m], total[1][m]);
                        if (BIAS) total[BIAS ? 3 : 0][m] = add(total[BIAS ? 3 : 0][m], dn[i]);
                        dh[m] = mul(dn[i], w[i]);
                    }
                }
            norm_back<VEC>(dh, h, in, k2, a.pre, a, sum);
        }
        if (a.dh)
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (in[c]) {
                    Ch<W> x[VEC / W];
                    rdh.get(x[0].v, slot, c);
#pragma unroll
                    for (int i = 0; i < VEC / W; ++i) dh[c * VEC / W + i] = add(x[i], dh[c * VEC / W + i]);
                }
        // dh is the whole gradient of h
        R *const dr = (R *)a.dr + row_of(a.vdr, now.b, 0, now.t);
        T *const dg = (T *)a.dgate + row_of(a.vdg, now.b, 0, now.t);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (in[c]) {
                Ch<W> w[VEC / W], x[VEC / W], o[VEC / W];
#pragma unroll
                for (int i = 0; i < VEC / W; ++i) o[i] = mul(rs, dh[c * VEC / W + i]);
                put<VEC>(dr + at[c], o[0].v);
                post(c, w, x);
                if (a.gate) {
#pragma unroll
                    for (int i = 0; i < VEC / W; ++i) {
                        const int m = c * VEC / W + i;
                        o[i] = mul(mul(bs, dh[m]), x[i]);
                        if (a.act != LA_ACT_NONE) o[i] = mul(o[i], slope[m]);
                    }
                    put<VEC>(dg + at[c], o[0].v);
                }
#pragma unroll
                for (int i = 0; i < VEC / W; ++i) {
                    const int m = c * VEC / W + i;
                    const Ch<W> du = mul(dh[m], act[m]);
                    total[0][m] = fma(du, u[m], total[0][m]);
                    if (BIAS) total[BIAS ? 2 : 0][m] = add(total[BIAS ? 2 : 0][m], du);
                    dh[m] = mul(du, w[i]);
                }
            }
        if (a.post != LA_NORM_NONE) {
            clear<VEC>(dh, in);
            norm_back<VEC>(dh, u, in, k1, a.post, a, sum);
        }
        T *const dy = (T *)a.dy + row_of(a.vdy, now.b, 0, now.t);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (in[c]) put<VEC>(dy + at[c], flat(dh, c * VEC));
        fetch(row + PF * step, slot);
        now.next(step_b, step_t, a.L);
    }
    if (a.part) {
        // the block's row groups one after the other into shared memory, then the block's sums
        float *const acc = (float *)ring;  // [4][d], where the rows were
        if (VEC == 8) asm volatile("cp.async.wait_group 0;" ::: "memory");
        if constexpr (GROUPS > 1) {
            for (int g = 0; g < GROUPS; ++g) {
                __syncthreads();
                if (group == g)
#pragma unroll
                    for (int k = 0; k < (BIAS ? 4 : 2); ++k)
                        if (a.sums >> k & 1)
#pragma unroll
                            for (int i = 0; i < N; ++i)
                                if (in[i / VEC]) {
                                    float *const p = acc + k * a.d + at[i / VEC] + i % VEC;
                                    *p = g == 0 ? total[k][i / W].v[i % W] : *p + total[k][i / W].v[i % W];
                                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < 4 * a.d; i += BLOCK)
                if (a.sums >> (i / a.d) & 1) a.part[(long long)blockIdx.x * 4 * a.d + i] = acc[i];
        } else {
#pragma unroll
            for (int k = 0; k < (BIAS ? 4 : 2); ++k)
                if (a.sums >> k & 1)
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        if (in[c]) put<VEC>(a.part + ((long long)blockIdx.x * 4 + k) * a.d + at[c], flat(total[k], c * VEC));
        }
    }
}

struct BnJoin {
    const float *part;
    float *out[4];
    int blocks, d;
};
// 32 channels a block, the blocks' sums in 32 runs of every 32nd one, joined in order.
__global__ void __launch_bounds__(1024) bn_join_kernel(const BnJoin a)
{
    __shared__ float sm[32][33];
    const int k = blockIdx.y, x = threadIdx.x & 31, run = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    if (!a.out[k]) return;
    float s = 0.f;
    if (c < a.d)
#pragma unroll 8
        for (int g = run; g < a.blocks; g += 32) s += a.part[((long long)g * 4 + k) * a.d + c];
    sm[run][x] = s;
    __syncthreads();
    // 32 runs of a channel to the lanes of one warp
    s = sm[x][run];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (x == 0 && blockIdx.x * 32 + run < a.d) a.out[k][blockIdx.x * 32 + run] = s;
}

// ---- which kernel takes a row -----------------------------------------------------------------
// 8 channels a thread where every row can be read 16 bytes at a time; else one by one.
// Shared memory of a kernel: the ring, or where row groups share a block the sums that it is reused for.
template <typename T, typename R, int VEC, int NT, int NC, bool BWD> constexpr int ring_bytes(int d)
{
    constexpr int block = bn_block<NT, BWD>, bt = Ahead<T, VEC, NC, block>::BYTES, br = Ahead<R, VEC, NC, block>::BYTES,
                  stage = BWD ? 3 * bt + 2 * br : 2 * bt + br, ring = AHEAD<VEC, stage, block, BWD ? bn_threads<NT, NC> : 384> * stage;
    return BWD && NT < block ? std::max(ring, 16 * d) : ring;
}

// Blocks of a kernel that run at once on an SM, with its shared memory limit set; once a device and kernel.
template <auto KERN> int blocks_at_once(int block, int smem)
{
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if ((n = known[dev].load()) > 0) return n;
    if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERN, block, (size_t)smem) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    known[dev].store(n);
    return n;
}
constexpr int BN_MOST_BLOCKS = 8;  // of an SM

template <typename F> int by_shape(int d, bool wide, F &&f)
{
    std::integral_constant<int, 1> one;
    std::integral_constant<int, 2> two;
    std::integral_constant<int, 8> v;
    std::integral_constant<int, 32> t32;
    std::integral_constant<int, 64> t64;
    std::integral_constant<int, 128> t128;
    std::integral_constant<int, 256> t256;
    std::integral_constant<int, 512> t512;
    if (!wide) {
        // single channels, 8 a thread (16 for the longest rows): as few threads as hold the row, so that none idles
        // (B8 L4096 d500: 1850 us with 512 threads a row)
        if (d <= 256) return f(one, t32, v);
        if (d <= 512) return f(one, t64, v);
        if (d <= 1024) return f(one, t128, v);
        if (d <= 2048) return f(one, t256, v);
        if (d <= 4096) return f(one, t512, v);
        return f(one, t512, std::integral_constant<int, 16>());
    }
    // 8 channels a thread for rows up to 1536: their registers allow more rows at once (B2 L16384 d768 76 us and the
    // gradients 147, with all sums 169; 83, 158 and 222 with 16). 16 beyond: half the sums' and the rows' overhead (B8 L8192
    // d2048 228 and 480 us; 303 and 565 with 8).
    if (d <= 256) return f(v, t32, one);
    if (d <= 512) return f(v, t64, one);
    if (d <= 768) return f(v, std::integral_constant<int, 96>(), one);
    if (d <= 1024) return f(v, t128, one);
    if (d <= 1536) return f(v, std::integral_constant<int, 192>(), one);
    if (d <= 2048) return f(v, t128, two);
    if (d <= 4096) return f(v, t256, two);
    return f(v, t512, two);
}
template <typename F> int by_types(int dtype, int rtype, F &&f)
{
    if (dtype == LA_F32) return f(0.f, 0.f);
    if (rtype == LA_F32) return f(__nv_bfloat16(), 0.f);
    return f(__nv_bfloat16(), __nv_bfloat16());
}

View row_view(const la_strides *s, int L, int d)
{
    if (s) return View{s->b, 0, s->l};
    return View{(long long)L * d, 0, d};
}

bool bn_args_ok(int post, int pre, bool has_pre, int act, int d, int dtype, int rtype)
{
    if (post < LA_NORM_NONE || post > LA_NORM_LAYER || act < LA_ACT_NONE || act > BN_SIGMOID) return false;
    if (has_pre && pre != LA_NORM_RMS && pre != LA_NORM_LAYER) return false;
    if (!dtype_ok(dtype) || !dtype_ok(rtype) || (dtype == LA_F32 && rtype != LA_F32)) return false;
    return d <= BN_MAX_D;
}

}  // namespace

}  // namespace la

using namespace la;

extern "C" {

int la_block_norm_fwd(const void *y, const void *residual, const void *gate, const float *post_weight, const float *post_bias,
                      const float *pre_weight, const float *pre_bias, void *h, void *n, int B, int L, int d,
                      const la_strides *y_strides, const la_strides *residual_strides, const la_strides *gate_strides,
                      const la_strides *h_strides, const la_strides *n_strides, int post_norm, int pre_norm, int activation,
                      float residual_scale, float branch_scale, float eps, int dtype, int residual_dtype, void *stream)
{
    if (!y || !residual || !h) return LA_ERR_NULL;
    if (!sizes_ok(B, 1, L, d)) return LA_ERR_SHAPE;
    if (!bn_args_ok(post_norm, pre_norm, n != nullptr, activation, d, dtype, residual_dtype)) return LA_ERR_UNSUPPORTED;
    BnArgs a = {};
    a.y = y; a.r = residual; a.gate = gate; a.h = h; a.n = n;
    a.post_w = post_weight; a.post_b = post_bias; a.pre_w = pre_weight; a.pre_b = pre_bias;
    a.vy = row_view(y_strides, L, d);
    a.vr = row_view(residual_strides, L, d);
    a.vg = row_view(gate_strides, L, d);
    a.vh = row_view(h_strides, L, d);
    a.vn = row_view(n_strides, L, d);
    if (!input_view_ok(a.vy, B, 1, L) || !input_view_ok(a.vr, B, 1, L) || (gate && !input_view_ok(a.vg, B, 1, L)) ||
        !output_view_ok(a.vh, B, 1, L, d) || (n && !output_view_ok(a.vn, B, 1, L, d)) || !(eps > 0.f) || !isfinite(eps) ||
        !isfinite(residual_scale) || !isfinite(branch_scale))
        return LA_ERR_ARG;
    const size_t es = dtype_size(dtype), er = dtype_size(residual_dtype);
    if (!aligned(y, es) || !aligned(gate, es) || !aligned(n, es) || !aligned(residual, er) || !aligned(h, er) ||
        !aligned(post_weight, 4) || !aligned(post_bias, 4) || !aligned(pre_weight, 4) || !aligned(pre_bias, 4))
        return LA_ERR_ARG;
    a.rows = (long long)B * L;
    a.L = L; a.d = d; a.post = post_norm; a.pre = pre_norm; a.act = activation;
    a.rs = residual_scale; a.bs = branch_scale; a.eps = eps; a.inv_d = 1.f / (float)d;
    const int sms = device_sms();
    if (sms <= 0) return LA_ERR_CUDA;
    auto ok = [&](const void *p, const View &v, size_t e) { return !p || rows_aligned(p, v, B, 1, L, e, 16); };
    const bool wide = d % 8 == 0 && ok(y, a.vy, es) && ok(residual, a.vr, er) && ok(gate, a.vg, es) && ok(h, a.vh, er) &&
                      ok(n, a.vn, es) && aligned(post_weight, 16) && aligned(post_bias, 16) && aligned(pre_weight, 16) &&
                      aligned(pre_bias, 16);
    return by_types(dtype, residual_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        return by_shape(d, wide, [&](auto v, auto nt, auto nc) {
            constexpr int per_block = bn_block<nt, false> / nt, smem = ring_bytes<T, R, v, nt, nc, false>(0);
            const int at_once = blocks_at_once<bn_fwd_kernel<T, R, v, nt, nc>>(bn_block<nt, false>, smem);
            if (at_once <= 0) return (int)LA_ERR_CUDA;
            const long long grid = std::min<long long>((a.rows + per_block - 1) / per_block, (long long)sms * at_once);
            return launch(bn_fwd_kernel<T, R, v, nt, nc>, dim3((unsigned)grid), bn_block<nt, false>, smem, (cudaStream_t)stream, a);
        });
    });
}

size_t la_block_norm_bwd_workspace_bytes(int B, int L, int d)
{
    if (!sizes_ok(B, 1, L, d) || d > BN_MAX_D) return 0;
    // as many blocks as an SM may hold, each at most one for a row
    const int sms = device_sms() > 0 ? device_sms() : 152;
    const long long blocks = std::min<long long>((long long)B * L, (long long)sms * BN_MOST_BLOCKS);
    return (size_t)blocks * 4 * d * sizeof(float);
}

int la_block_norm_bwd(const void *y, const void *residual, const void *gate, const float *post_weight, const float *post_bias,
                      const float *pre_weight, const float *pre_bias, const void *dh, const void *dn, void *dresidual, void *dy,
                      void *dgate, float *dpost_weight, float *dpost_bias, float *dpre_weight, float *dpre_bias, int B, int L,
                      int d, const la_strides *y_strides, const la_strides *residual_strides, const la_strides *gate_strides,
                      const la_strides *dh_strides, const la_strides *dn_strides, const la_strides *dresidual_strides,
                      const la_strides *dy_strides, const la_strides *dgate_strides, int post_norm, int pre_norm, int activation,
                      float residual_scale, float branch_scale, float eps, int dtype, int residual_dtype, void *workspace,
                      size_t workspace_bytes, void *stream)
{
    if (!y || !residual || !dresidual || !dy || (!dh && !dn) || !gate != !dgate) return LA_ERR_NULL;
    if (!dn && (dpre_weight || dpre_bias)) return LA_ERR_NULL;
    if (!sizes_ok(B, 1, L, d)) return LA_ERR_SHAPE;
    if (!bn_args_ok(post_norm, pre_norm, dn != nullptr, activation, d, dtype, residual_dtype)) return LA_ERR_UNSUPPORTED;
    BnArgs a = {};
    a.y = y; a.r = residual; a.gate = gate; a.dh = dh; a.dn = dn;
    a.dr = dresidual; a.dy = dy; a.dgate = dgate;
    a.post_w = post_weight; a.post_b = post_bias; a.pre_w = pre_weight; a.pre_b = pre_bias;
    a.vy = row_view(y_strides, L, d);
    a.vr = row_view(residual_strides, L, d);
    a.vg = row_view(gate_strides, L, d);
    a.vdh = row_view(dh_strides, L, d);
    a.vdn = row_view(dn_strides, L, d);
    a.vdr = row_view(dresidual_strides, L, d);
    a.vdy = row_view(dy_strides, L, d);
    a.vdg = row_view(dgate_strides, L, d);
    if (!input_view_ok(a.vy, B, 1, L) || !input_view_ok(a.vr, B, 1, L) || (gate && !input_view_ok(a.vg, B, 1, L)) ||
        (dh && !input_view_ok(a.vdh, B, 1, L)) || (dn && !input_view_ok(a.vdn, B, 1, L)) || !output_view_ok(a.vdr, B, 1, L, d) ||
        !output_view_ok(a.vdy, B, 1, L, d) || (gate && !output_view_ok(a.vdg, B, 1, L, d)) || !(eps > 0.f) || !isfinite(eps) ||
        !isfinite(residual_scale) || !isfinite(branch_scale))
        return LA_ERR_ARG;
    const size_t es = dtype_size(dtype), er = dtype_size(residual_dtype);
    if (!aligned(y, es) || !aligned(gate, es) || !aligned(dn, es) || !aligned(dy, es) || !aligned(dgate, es) ||
        !aligned(residual, er) || !aligned(dh, er) || !aligned(dresidual, er) || !aligned(post_weight, 4) ||
        !aligned(post_bias, 4) || !aligned(pre_weight, 4) || !aligned(pre_bias, 4) || !aligned(dpost_weight, 4) ||
        !aligned(dpost_bias, 4) || !aligned(dpre_weight, 4) || !aligned(dpre_bias, 4) || !aligned(workspace, 16))
        return LA_ERR_ARG;
    a.rows = (long long)B * L;
    a.L = L; a.d = d; a.post = post_norm; a.pre = pre_norm; a.act = activation;
    a.rs = residual_scale; a.bs = branch_scale; a.eps = eps; a.inv_d = 1.f / (float)d;
    const int sms = device_sms();
    if (sms <= 0) return LA_ERR_CUDA;
    auto ok = [&](const void *p, const View &v, size_t e) { return !p || rows_aligned(p, v, B, 1, L, e, 16); };
    const bool wide = d % 8 == 0 && ok(y, a.vy, es) && ok(residual, a.vr, er) && ok(gate, a.vg, es) && ok(dh, a.vdh, er) &&
                      ok(dn, a.vdn, es) && ok(dresidual, a.vdr, er) && ok(dy, a.vdy, es) && ok(dgate, a.vdg, es) &&
                      aligned(post_weight, 16) && aligned(post_bias, 16) && aligned(pre_weight, 16) && aligned(pre_bias, 16);
    a.sums = (dpost_weight ? 1 : 0) | (dpre_weight ? 2 : 0) | (dpost_bias ? 4 : 0) | (dpre_bias ? 8 : 0);
    long long blocks = 0;
    const int rc = by_types(dtype, residual_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        return by_shape(d, wide, [&](auto v, auto nt, auto nc) {
            constexpr int per_block = bn_block<nt, true> / nt;
            const int most = v == 8 ? 8 * nt * nc : nt * nc, smem = ring_bytes<T, R, v, nt, nc, true>(most);  // for every d of it
            auto run = [&](auto bias) {
                const int at_once = blocks_at_once<bn_bwd_kernel<T, R, v, nt, nc, bias>>(bn_block<nt, true>, smem);
                if (at_once <= 0) return (int)LA_ERR_CUDA;
                blocks = std::min<long long>((a.rows + per_block - 1) / per_block, (long long)sms * std::min(at_once, BN_MOST_BLOCKS));
                if (a.sums) {
                    if (!workspace || workspace_bytes < (size_t)blocks * 4 * d * sizeof(float)) return (int)LA_ERR_WORKSPACE;
                    a.part = (float *)workspace;
                }
                return launch(bn_bwd_kernel<T, R, v, nt, nc, bias>, dim3((unsigned)blocks), bn_block<nt, true>, smem, (cudaStream_t)stream, a);
            };
            if constexpr (v == 8)
                if (!dpost_bias && !dpre_bias) return run(std::false_type());
            return run(std::true_type());
        });
    });
    if (rc != LA_OK || !a.sums) return rc;
    const BnJoin j{a.part, {dpost_weight, dpre_weight, dpost_bias, dpre_bias}, (int)blocks, d};
    return launch(bn_join_kernel, dim3((unsigned)((d + 31) / 32), 4), 1024, 0, (cudaStream_t)stream, j);
}

}  // extern "C"
