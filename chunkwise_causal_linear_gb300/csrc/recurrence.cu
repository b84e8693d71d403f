// recurrence.cu -- gated linear recurrence h_t = a_t h_{t-1} + w_t x_t, its gradients and its
// decoding step (sm_103a).
//
// A run of rows acts on the state before it as h -> P h + H (P the product of its gates, H what
// it adds from zero), and two runs in a row join to P = P2 P1, H = P2 H1 + H2.  So a run is
// folded on its own, and its rows are finished once the state before it is known.  Backwards,
// c_t = a_t e_t, e_t = dout_t + c_{t+1}: c -> P c + E with the same P.
//
// The rows of one head's block of 32 V channels go through one cluster of S blocks (S = 1: one
// block).  A step of the cluster covers S tiles, one per block; a tile is 8 warps of R rows (16
// or 32), a lane holds V channels of them in registers, as pairs for the packed fp32 instructions:
// two channels (V = 2), or one channel of rows i and i + R/2 (V = 1).  Per step: fold the R rows
// and put (P, H) into shared memory; one warp runs the carried state over the 8 folds while the
// others wait (when each did it for itself, that was a quarter of all instructions); every warp
// finishes its rows from its state.  With S > 1 that warp first sends the tile's (P, H) into the
// other blocks' shared memory (st.async, which counts on an mbarrier there) and so knows the
// state before the tile and after the step; the release of a cluster barrier in that place waited
// for the output rows still on their way (a quarter of the time).  Every input is read once and
// every output written once; nothing goes through global memory between the blocks, and the order
// of the sums depends on the sizes and the GPU alone.
//
// Measured (of the measured HBM rate): B1 H16 L65536 d64 fp32 (32 clusters of 8) forward 124 us,
// 97%, backward 209 us, 96%; B8 H16 L8192 d128 bf16 with sigmoid gates forward 129 us, 93%,
// backward 295 us, 68%: at 6 and 10 bytes an element and ~20 and ~50 instructions the bf16 cases
// are bound by instructions as much as by memory, and few heads of them (B1 H8 L65536 d128: 96 us,
// 62%, and 183 us, 55%; 24 and 50 instructions, issued 46% and 49% of the time) by the latency of a
// step besides.
//
// The inputs of the next steps are on the way while one is folded: each warp copies its own rows
// into its own ring in shared memory (cp.async, no barrier).
#include <stdlib.h>

#include <algorithm>
#include <atomic>

#include "layer.cuh"
#include "tc_ptx.cuh"

namespace la {

using namespace ptx;

namespace {

constexpr int RC = LA_RECURRENCE_CHUNK;  // rows between the states that the forward leaves
constexpr int REC_W = 8;                 // warps of a tile
constexpr int REC_THREADS = 32 * REC_W;
template <typename T> constexpr bool ACC = sizeof(T) == 4;  // see gate_of
constexpr int BWD_R = 16;                // rows of a warp, backward
constexpr int REC_MAX_SPLIT = 16;        // blocks of a cluster; above 8 asks for the larger size this GPU has

struct RecArgs {
    const void *x, *g, *dout;
    void *out, *dx, *dg;
    const float *h0, *dh_last, *chunks_in;
    float *h_last, *dh0, *chunks;
    const int *lengths;
    View vx, vg, vo, vdx, vdg;  // vo: out, or dout
    int B, H, L, d;
    int ncb;            // channel blocks of a head
    int split;          // blocks of a cluster
    int grx, grg, gro;  // bytes per copy of x, gate, dout: 16, 4 or 2 (their alignment)
    int *err;           // device error word
    unsigned long long timeout_ns;  // limit of a wait for another block
    int debug_stall;    // test knob: nothing is sent to the other blocks (forces a timeout)
};

// a and 1 - a from the gate input.  u = 2^-24.
//
// With bf16 activations both are off by at most (9 + 1.3 |g|) u relatively: the argument g log2(e) of
// the special function unit's 2^x is rounded (1.3 |g| u), 2^x 4 u, the sum 1 u, the reciprocal 2 u, a
// product or difference 1 u.  Next to 1, where a long memory adds the error of a up row by row, that
// is 2 u (measured): half a step of the bf16 output after 32768 rows.
//
// With fp32 activations (FINE) an a next to 1 is good to a rounding: it is 1 less 1 - a, which alone
// comes from the series or the exponential; and the exponential of a sigmoid has what its argument's
// rounding left out multiplied in, so that the smaller of a and 1 - a is off by at most 9 u.
constexpr float LOG2E = 1.44269504f;
template <int V> __device__ __forceinline__ Ch<V> pow2(Ch<V> t)
{
#pragma unroll
    for (int v = 0; v < V; ++v) t.v[v] = ex2(t.v[v]);
    return t;
}
template <int KIND, bool WANT_C, bool FINE, int V>
__device__ __forceinline__ void gate_of(const Ch<V> &g, Ch<V> &a, Ch<V> &c)
{
    if (KIND == LA_GATE_VALUE) {
        a = g;
        if (WANT_C) c = fma(g, all<V>(-1.f), all<V>(1.f));
    } else if (KIND == LA_GATE_LOG) {
        a = pow2(mul(g, all<V>(LOG2E)));
        if (FINE && !WANT_C) {
            // e^g by its series below 2^-4 (the first term left out is 2^-27); the error of the
            // power counts 1 / (1 - a) <= 17 times elsewhere
            Ch<V> p = fma(g, all<V>(1.f / 24), all<V>(1.f / 6));
            p = fma(g, p, all<V>(0.5f));
            p = fma(g, p, all<V>(1.f));
            const Ch<V> near = fma(g, p, all<V>(1.f));
#pragma unroll
            for (int v = 0; v < V; ++v) a.v[v] = fabsf(g.v[v]) < 0.0625f ? near.v[v] : a.v[v];
        }
        if (WANT_C) {
            // below log 2 from s = expm1(g / 2) by its series, expm1(g) = s (s + 2) (the first term
            // left out is 2e-8 of the sum)
            const Ch<V> y = mul(g, all<V>(0.5f));
            Ch<V> p = fma(y, all<V>(1.f / 5040), all<V>(1.f / 720));
            p = fma(y, p, all<V>(1.f / 120));
            p = fma(y, p, all<V>(1.f / 24));
            p = fma(y, p, all<V>(1.f / 6));
            p = fma(y, p, all<V>(0.5f));
            p = fma(y, p, all<V>(1.f));
            const Ch<V> s = mul(y, p), q = add(s, all<V>(2.f));
            const Ch<V> e = mul(mul(s, all<V>(-1.f)), q), f = fma(a, all<V>(-1.f), all<V>(1.f)),
                        near = fma(s, q, all<V>(1.f));
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool series = fabsf(g.v[v]) < 0.693f;
                c.v[v] = series ? e.v[v] : f.v[v];
                if (FINE && series) a.v[v] = near.v[v];
            }
        }
    } else if (FINE) {
        Ch<V> e;
#pragma unroll
        for (int v = 0; v < V; ++v) e.v[v] = max_nan(-fabsf(g.v[v]), -150.f);
        e = exp_fine(e);
        Ch<V> r = add(e, all<V>(1.f));
#pragma unroll
        for (int v = 0; v < V; ++v) r.v[v] = rcp(r.v[v]);
        const Ch<V> less = mul(e, r), more = fma(less, all<V>(-1.f), all<V>(1.f));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            a.v[v] = g.v[v] < 0.f ? less.v[v] : more.v[v];
            if (WANT_C) c.v[v] = g.v[v] < 0.f ? more.v[v] : less.v[v];
        }
    } else {
        // a = 1 / (1 + e), 1 - a = e a; where e is so large that a is 0, 1 - a is 1
        const Ch<V> e = pow2(mul(g, all<V>(-LOG2E))), d = add(e, all<V>(1.f));
#pragma unroll
        for (int v = 0; v < V; ++v) a.v[v] = rcp(d.v[v]);
        if (WANT_C) {
            c = mul(e, a);
#pragma unroll
            for (int v = 0; v < V; ++v) c.v[v] = a.v[v] == 0.f ? 1.f : c.v[v];
        }
    }
}

// The gate input of a = 1, 1 - a = 0.
template <int KIND> __device__ __forceinline__ float keep_gate()
{
    return KIND == LA_GATE_VALUE ? 1.f : KIND == LA_GATE_LOG ? 0.f : __int_as_float(0x7f800000);
}

// The gate input of a = 0.
template <int KIND> __device__ __forceinline__ bool forgets(float g)
{
    return KIND == LA_GATE_VALUE ? g == 0.f : g == __int_as_float(0xff800000);
}

// gate_of() flushes what is below the normal range.  Where something is not finite the difference
// counts: an a of 0 forgets it, a 1 - a of 0 makes it NaN.  There, and in the decoding step, such a
// gate is kept at the smallest number.
template <int KIND, bool WANT_C, bool FINE, int V>
__device__ __forceinline__ void gate_exact(const Ch<V> &g, Ch<V> &a, Ch<V> &c)
{
    gate_of<KIND, WANT_C, FINE, V>(g, a, c);
    if (KIND == LA_GATE_VALUE) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (a.v[v] == 0.f && !forgets<KIND>(g.v[v])) a.v[v] = __int_as_float(1);
        if (WANT_C && KIND == LA_GATE_SIGMOID && c.v[v] == 0.f && fabsf(g.v[v]) < __int_as_float(0x7f800000))
            c.v[v] = __int_as_float(1);
    }
}

// A product of gates P is 0 if and only if one of them is, so that P, too, forgets what a gate of 0
// forgets and nothing else.  One that fp32 rounds to 0 although no factor is 0 (gates of 0.44 over
// 128 rows) is kept at the smallest number of its sign: a finite state comes out no farther off than
// by a rounding of P, an infinity or NaN as itself.  An infinite or NaN gate does not outlive a 0.
__device__ __forceinline__ float least(float p) { return copysignf(__int_as_float(1), p); }
template <int V> __device__ __forceinline__ Ch<V> product(const Ch<V> &a, const Ch<V> &p)
{
    Ch<V> r = mul(a, p);
#pragma unroll
    for (int v = 0; v < V; ++v) r.v[v] = a.v[v] == 0.f || p.v[v] == 0.f ? 0.f : r.v[v] == 0.f ? least(r.v[v]) : r.v[v];
    return r;
}
// Not 0, infinite or NaN: then the plain product is the one above.
template <int V> __device__ __forceinline__ bool regular(const Ch<V> &p)
{
    bool ok = true;
#pragma unroll
    for (int v = 0; v < V; ++v) ok = ok && fabsf(p.v[v]) > 0.f && fabsf(p.v[v]) <= 3.402823466e38f;
    return ok;
}

// The state times a gate (or a product of gates), a gate of 0 forgetting infinities and NaN as
// well.
template <int V> __device__ __forceinline__ Ch<V> forget(const Ch<V> &a, const Ch<V> &h)
{
    Ch<V> r = mul(a, h);
#pragma unroll
    for (int v = 0; v < V; ++v) r.v[v] = a.v[v] == 0.f ? 0.f : r.v[v];
    return r;
}
template <int V> __device__ __forceinline__ Ch<V> step(const Ch<V> &a, const Ch<V> &h, const Ch<V> &b)
{
    Ch<V> r = fma(a, h, b);
#pragma unroll
    for (int v = 0; v < V; ++v) r.v[v] = a.v[v] == 0.f ? b.v[v] : r.v[v];
    return r;
}
// The common path leaves the forgetting of infinities and NaN out (a plain fma): they then stay to
// the last row, so whoever finds that one finite has the exact value, and the others start again
// with step().
template <int V> __device__ __forceinline__ bool finite(const Ch<V> &h)
{
    bool ok = true;
#pragma unroll
    for (int v = 0; v < V; ++v) ok = ok && fabsf(h.v[v]) <= 3.402823466e38f;
    return ok;
}

__device__ __forceinline__ int rows_of(const RecArgs &a, int b)
{
    return a.lengths ? max(0, min(a.lengths[b], a.L)) : a.L;
}

// ---- copies into the ring -----------------------------------------------------------------
template <int BYTES> __device__ __forceinline__ void cp_async(uint32_t dst, const void *src)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Rows [0, nrow) and channels [0, nch) of a warp's rows into its ring slot, CW channels a row, in
// copies of `gran` bytes: N copies make a row, a warp makes 32 / N rows at once.
template <typename T, int R, int CW, int BYTES>
__device__ __forceinline__ void copy_by(T *slot, const T *src, long long stride, int nrow, int nch, int lane)
{
    constexpr int E = BYTES / sizeof(T), N = CW / E, RP = 32 / N, M = R / RP;
    static_assert(32 % N == 0 && R % RP == 0, "whole rows per warp instruction");
    const int r0 = lane / N, c = lane % N * E;
    if (c >= nch) return;
    const T *p = src + r0 * stride + c;
    T *q = slot + r0 * CW + c;
    if constexpr (BYTES == 2) {
        if (nrow == R) {
            T v[M];
#pragma unroll
            for (int j = 0; j < M; ++j, p += RP * stride) v[j] = *p;
#pragma unroll
            for (int j = 0; j < M; ++j) q[j * RP * CW] = v[j];
        } else {
#pragma unroll 1
            for (int r = r0; r < nrow; r += RP, p += RP * stride, q += RP * CW) *q = *p;
        }
    } else {
        const uint32_t dst = smem_u32(q);
#pragma unroll
        for (int j = 0; j < M; ++j, p += RP * stride)
            if (r0 + j * RP < nrow) cp_async<BYTES>(dst + (uint32_t)sizeof(T) * j * RP * CW, p);
    }
}
// The rarer cases out of the way of the common one, which fits the instruction cache.  Rows that a
// sequence does not have are filled with what leaves the state alone.
template <typename T, int R, int CW>
__device__ __noinline__ void copy_odd(T *slot, const T *src, long long stride, int nrow, int nch, int gran, int lane,
                                      float fill)
{
    if (gran == 16) copy_by<T, R, CW, 16>(slot, src, stride, nrow, nch, lane);
    else if (gran == 4) copy_by<T, R, CW, 4>(slot, src, stride, nrow, nch, lane);
    else if constexpr (sizeof(T) == 2 && CW == 32) copy_by<T, R, CW, 2>(slot, src, stride, nrow, nch, lane);
    for (int r = nrow; r < R; ++r)
        for (int c = lane; c < CW; c += 32) slot[r * CW + c] = from_f32<T>(fill);
}
template <typename T, int R, int CW>
__device__ __forceinline__ void copy_rows(T *slot, const T *src, long long stride, int nrow, int nch, int gran,
                                          int lane, float fill = 0.f)
{
    if (nrow < R || gran != 16) {
        if (nrow > 0) copy_odd<T, R, CW>(slot, src, stride, nrow, nch, gran, lane, fill);
        return;
    }
    constexpr int E = 16 / sizeof(T), N = CW / E, RP = 32 / N;  // elements a copy, copies a row, rows at once
    const int r0 = lane / N, c = lane % N * E;
    const T *p = src + r0 * stride + c;
    const uint32_t dst = smem_u32(slot + r0 * CW + c);
    if (c < nch)
#pragma unroll
        for (int j = 0; j < R / RP; ++j, p += RP * stride)
            cp_async<16>(dst + (uint32_t)sizeof(T) * j * RP * CW, p);
}

// ---- V neighbouring channels (pairs, of bf16, are aligned and inside the channels together) -----
template <int V> __device__ __forceinline__ Ch<V> get(const float *p)
{
    static_assert(V == 1, "pairs are of bf16");
    return {{*p}};
}
template <int V> __device__ __forceinline__ Ch<V> get(const __nv_bfloat16 *p)
{
    if constexpr (V == 2) {
        const uint32_t t = *(const uint32_t *)p;
        return {{__uint_as_float(t << 16), __uint_as_float(t & 0xffff0000u)}};
    } else {
        return {{__bfloat162float(*p)}};
    }
}
template <int V> __device__ __forceinline__ void put(float *p, const Ch<V> &x)
{
    static_assert(V == 1, "pairs are of bf16");
    *p = x.v[0];
}
template <int V> __device__ __forceinline__ void put(__nv_bfloat16 *p, const Ch<V> &x)
{
    if constexpr (V == 2) *(__nv_bfloat162 *)p = __floats2bfloat162_rn(x.v[0], x.v[1]);
    else *p = __float2bfloat16_rn(x.v[0]);
}
// (P, H) of V channels, next to each other in shared memory
template <int V> struct __align__(8 * V) Fold {
    Ch<V> p, h;
};

// What a lane computes in pairs, for the packed instructions: two channels of every row (V = 2), or
// one channel of rows i and i + R/2 (V = 1), whose two runs are joined afterwards.
template <int V, int R> struct Pairs {
    static constexpr int N = V == 2 ? R : R / 2;  // pairs of a warp's rows
    static constexpr int CW = 32 * V;
    template <typename T> static __device__ __forceinline__ Ch<2> get(const T *p, int i)
    {
        if constexpr (V == 2) return la::get<2>(p + i * CW);
        else return {{la::get<1>(p + i * CW).v[0], la::get<1>(p + (i + N) * CW).v[0]}};
    }
    // row i at p, row i + N at q
    template <typename T> static __device__ __forceinline__ void put(T *p, T *q, const Ch<2> &x)
    {
        if constexpr (V == 2) {
            la::put<2>(p, x);
        } else {
            la::put<1>(p, Ch<1>{{x.v[0]}});
            la::put<1>(q, Ch<1>{{x.v[1]}});
        }
    }
    // the fold of all rows, the earlier run first
    static __device__ __forceinline__ Fold<V> join(const Ch<2> &p, const Ch<2> &h)
    {
        if constexpr (V == 2) return {p, h};
        else return {{{p.v[0] * p.v[1]}}, {{fmaf(p.v[1], h.v[0], h.v[1])}}};
    }
    // the states before the rows of a pair's runs
    static __device__ __forceinline__ Ch<2> spread(const Ch<V> &h, const Ch<2> &p, const Ch<2> &f)
    {
        if constexpr (V == 2) return h;
        else return {{h.v[0], fmaf(p.v[0], h.v[0], f.v[0])}};
    }
    // the same backwards: the later run comes first
    static __device__ __forceinline__ Ch<V> join_back(const Ch<2> &p, const Ch<2> &e)
    {
        if constexpr (V == 2) return e;
        else return {{fmaf(p.v[0], e.v[1], e.v[0])}};
    }
    static __device__ __forceinline__ Ch<2> spread_back(const Ch<V> &e, const Ch<2> &p, const Ch<2> &f)
    {
        if constexpr (V == 2) return e;
        else return {{fmaf(p.v[1], e.v[0], f.v[1]), e.v[0]}};
    }
};

// ---- rows one after the other -----------------------------------------------------------------
// Where a sequence ends among a warp's rows and where something is not finite: from the copies in
// shared memory, in a loop that stays small.
template <typename T, typename G, int KIND, bool COMP, int V>
__device__ __noinline__ Fold<V> fold_rows(const T *sx, const G *sg, int rows)
{
    Fold<V> f{all<V>(1.f), all<V>(0.f)};
#pragma unroll 1
    for (int i = 0; i < rows; ++i) {
        const Ch<V> x = get<V>(sx + i * 32 * V);
        Ch<V> a, c;
        gate_exact<KIND, COMP, ACC<T>, V>(get<V>(sg + i * 32 * V), a, c);
        f.h = step(a, f.h, COMP ? mul(c, x) : x);
        f.p = product(f.p, a);
    }
    return f;
}
// The product of a run's gates where the plain one is not regular.  Where every run has one (sigmoid
// gates of logits around -4, B1 H8 L65536 d128 bf16) the look at the gates takes 14 us of 103.
template <typename G, int KIND, int V, int R> __device__ __forceinline__ Ch<V> product_exact(const G *sg, Ch<V> p)
{
    bool zero[V] = {};
#pragma unroll 4
    for (int i = 0; i < R; ++i) {
        const Ch<V> g = get<V>(sg + i * 32 * V);
#pragma unroll
        for (int v = 0; v < V; ++v) zero[v] = zero[v] || forgets<KIND>(g.v[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) p.v[v] = zero[v] ? 0.f : p.v[v] == 0.f ? least(p.v[v]) : p.v[v];
    return p;
}
// out: this lane's channels of the first row; `present` rows of it exist
template <typename T, typename G, int KIND, bool COMP, int V>
__device__ __noinline__ void finish_rows(const T *sx, const G *sg, int rows, int present, Ch<V> h, T *out,
                                         long long stride)
{
#pragma unroll 1
    for (int i = 0; i < present; ++i, out += stride) {
        if (i < rows) {
            const Ch<V> x = get<V>(sx + i * 32 * V);
            Ch<V> a, c;
            gate_exact<KIND, COMP, ACC<T>, V>(get<V>(sg + i * 32 * V), a, c);
            h = step(a, h, COMP ? mul(c, x) : x);
        }
        put<V>(out, i < rows ? h : all<V>(0.f));
    }
}
// The folds f[0], f[stride], ... of n runs applied to h.
template <int V> __device__ __noinline__ Ch<V> apply_exact(const Fold<V> *f, int stride, int n, Ch<V> h)
{
#pragma unroll 1
    for (int i = 0; i < n; ++i) h = step(f[i * stride].p, h, f[i * stride].h);
    return h;
}
// The states before the warps of a tile, and the one after it, exactly; step -32 runs backwards.
template <int V> __device__ __noinline__ Ch<V> begin_exact(Ch<V> *begin, const Fold<V> *f, int stride, Ch<V> h)
{
#pragma unroll 1
    for (int i = 0; i < REC_W; ++i) {
        begin[i * stride] = h;
        h = step(f[i * stride].p, h, f[i * stride].h);
    }
    return h;
}
// n runs in a row as one.
template <int V> __device__ __noinline__ Fold<V> join_exact(const Fold<V> *f, int stride, int n)
{
    Fold<V> t{all<V>(1.f), all<V>(0.f)};
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        t.h = step(f[i * stride].p, t.h, f[i * stride].h);
        t.p = product(f[i * stride].p, t.p);
    }
    return t;
}

template <int V> struct BwdFold {
    Ch<V> p, h, e;
};
template <typename T, typename G, int KIND, bool COMP, int V>
__device__ __noinline__ BwdFold<V> fold_rows_bwd(const T *sx, const T *sd, const G *sg, int rows)
{
    const Fold<V> f = fold_rows<T, G, KIND, COMP, V>(sx, sg, rows);
    Ch<V> e = all<V>(0.f);
#pragma unroll 1
    for (int i = rows - 1; i >= 0; --i) {
        Ch<V> a, c;
        gate_exact<KIND, false, ACC<T>, V>(get<V>(sg + i * 32 * V), a, c);
        e = forget(a, add(e, get<V>(sd + i * 32 * V)));
    }
    return {f.p, f.h, e};
}
// h, e: the state before these rows and what comes back from those behind them
template <typename T, typename G, int KIND, bool COMP, int V>
__device__ __noinline__ void finish_rows_bwd(const T *sx, const T *sd, const G *sg, int rows, int present, Ch<V> h,
                                             Ch<V> e, T *dx, long long dx_stride, G *dg, long long dg_stride)
{
    Ch<V> before[BWD_R];  // the state before each row
#pragma unroll 1
    for (int i = 0; i < rows; ++i) {
        const Ch<V> x = get<V>(sx + i * 32 * V);
        Ch<V> a, c;
        gate_exact<KIND, COMP, ACC<T>, V>(get<V>(sg + i * 32 * V), a, c);
        before[i] = h;
        h = step(a, h, COMP ? mul(c, x) : x);
    }
#pragma unroll 1
    for (int i = present - 1; i >= 0; --i) {
        Ch<V> rx = all<V>(0.f), rg = rx;
        if (i < rows) {
            const Ch<V> hb = before[i], x = get<V>(sx + i * 32 * V);
            Ch<V> a, c;
            gate_exact<KIND, COMP || KIND == LA_GATE_SIGMOID, ACC<T>, V>(get<V>(sg + i * 32 * V), a, c);
            e = add(e, get<V>(sd + i * 32 * V));
            rx = COMP ? mul(c, e) : e;
            const Ch<V> f = COMP ? fma(x, all<V>(-1.f), hb) : hb, ae = forget(a, e);
            const Ch<V> slope = KIND == LA_GATE_VALUE ? all<V>(1.f) : KIND == LA_GATE_LOG ? a : mul(c, a);
            const Ch<V> se = KIND == LA_GATE_VALUE ? e : KIND == LA_GATE_LOG ? ae : mul(c, ae);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                // a small se is not to round an infinite f away
                const float r = fabsf(f.v[v]) <= 3.402823466e38f ? se.v[v] * f.v[v] : slope.v[v] * (e.v[v] * f.v[v]);
                rg.v[v] = slope.v[v] == 0.f ? 0.f : r;
            }
            e = ae;
        }
        put<V>(dx + i * dx_stride, rx);
        put<V>(dg + i * dg_stride, rg);
    }
}

// ---- between the blocks of a cluster -----------------------------------------------------------
// Sends a fold to `slot` in block `rank` of the cluster, counted there on `bar`.
__device__ __forceinline__ void send(const Fold<1> *slot, const uint64_t *bar, int rank, const Fold<1> &f)
{
    uint32_t to, sig;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(slot)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(sig) : "r"(smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to),
                 "f"(f.p.v[0]), "f"(f.h.v[0]), "r"(sig) : "memory");
}
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ bool arrived(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3; "
                 "selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(200000u) : "memory");
    return ok != 0;
}

// What the blocks of a cluster send one another, read and sent by warp 0 of each: two buffers, each
// with its mbarrier, used in turn.  A block sends for step k + 2 after it has what every block
// sent for step k + 1, and a block's warp 0 sends that when it has read step k.
constexpr int REC_BUFS = 2;
struct Peers {
    Fold<1> *slot;  // [REC_BUFS][split][32]
    uint64_t *bar;  // [REC_BUFS]
    int split, rank, *err;
    unsigned long long timeout_ns;
    bool dead, stall;  // a wait ran out: no more waiting; nothing is sent

    __device__ void init(void *mem, int rank_, const RecArgs &a)
    {
        bar = (uint64_t *)mem;
        slot = (Fold<1> *)((char *)mem + 16 * REC_BUFS);
        split = a.split;
        rank = rank_;
        err = a.err;
        timeout_ns = a.timeout_ns;
        dead = false;
        stall = a.debug_stall != 0;
        if (threadIdx.x == 0) {
            for (int i = 0; i < REC_BUFS; ++i) mbar_init(&bar[i], 1);
            mbar_init_fence();
        }
        cluster_barrier();  // every block is there, with its barriers, before anyone sends
    }
    __device__ __forceinline__ void publish(int buf, int lane, const Fold<1> &f)
    {
        // after a wait that ran out, a barrier's phase may not have ended: it takes no further
        // arrival.  The other blocks' waits run out too, before any block ends.
        dead = __any_sync(0xffffffffu, dead);
        if (dead) return;
        if (threadIdx.x == 0) mbar_arrive_expect_tx(&bar[buf], (uint32_t)(split * 32 * sizeof(Fold<1>)));
        for (int r = 0; r < split && !stall; ++r) send(slot + (buf * split + rank) * 32 + lane, &bar[buf], r, f);
    }
    // The carry over the tiles of a step, `carry = P carry + H`: returns the carry before this
    // block's tile and leaves the one after the step.
    __device__ __forceinline__ Ch<1> over(int buf, uint32_t parity, int lane, bool on, Ch<1> &carry)
    {
        if (!dead && !arrived(&bar[buf], parity)) {
            const uint64_t t0 = globaltimer();
            while (!arrived(&bar[buf], parity))
                if (globaltimer() - t0 > timeout_ns) {
                    record_error(err, LA_ERR_TIMEOUT);
                    dead = true;
                    break;
                }
        }
        const Fold<1> *f = slot + buf * split * 32 + lane;
        const Ch<1> start = carry;
        Ch<1> mine = carry;
#pragma unroll 4
        for (int r = 0; r < split; ++r) {
            if (r == rank) mine = carry;
            const Fold<1> q = f[r * 32];
            carry = fma(q.p, carry, q.h);
        }
        if (on && !finite(carry)) {
            carry = apply_exact<1>(f, 32, split, start);
            mine = apply_exact<1>(f, 32, rank, start);
        }
        return mine;
    }
    // Behind the last barrier of the cluster: where the wait of the last step ran out, a block that came
    // late has sent since then, and its folds may still be on their way into this block's memory.  They
    // take microseconds; a block that gave up earlier gets nothing any more (those behind it gave up
    // in the next step), and neither waits longer than this.
    __device__ __forceinline__ void settle(int buf, uint32_t parity)
    {
        if (!dead) return;
        const uint64_t t0 = globaltimer();
        while (!arrived(&bar[buf], parity) && globaltimer() - t0 < 1000000) {
        }
    }
    static constexpr size_t bytes(int split) { return 16 * REC_BUFS + sizeof(Fold<1>) * REC_BUFS * split * 32; }
};

// Shared memory: the folds of the warps of a tile and the states before each of them, the rings, and
// what the blocks of the cluster send.  One buffer of each is enough: folds are written before the
// first block barrier of a step and read, by the warps that run the states over them, before the
// second, after which the states are read.
// The rows of a warp are 16; in a cluster with bf16 activations 32 forward, where a step's fixed part
// weighs more than the registers (B1 H8 L65536 d128: 98 us and 114; backward would need 96 registers
// for three values a row).
template <typename T, typename G, int V, bool BWD, bool SPLIT> struct RecSmem {
    static constexpr int R = BWD ? BWD_R : SPLIT && sizeof(T) == 2 ? 32 : 16, TILE = R * REC_W;
    static_assert(TILE % RC == 0 && (RC % R == 0), "tiles, and chunks within them, start at a warp's first row");
    static constexpr size_t AGG = sizeof(Fold<V>) * REC_W * 32, START = sizeof(Ch<V>) * REC_W * 32;
    static constexpr size_t HEAD = BWD ? AGG + 3 * START : AGG + START;  // backward: H, and both states
    static constexpr size_t SLOT = (size_t)R * 32 * V * (sizeof(T) * (BWD ? 2 : 1) + sizeof(G));
    static constexpr size_t STAGE = REC_W * SLOT;
    // three stages where two blocks share an SM with them (227 KB, 1 KB taken a block), else two
    static constexpr int STAGES = HEAD + 3 * STAGE <= 112 * 1024 ? 3 : 2;
    static constexpr size_t PEERS = HEAD + STAGES * STAGE;
    static size_t bytes(int split) { return PEERS + (split > 1 ? Peers::bytes(split) : 0); }
};

// threadIdx.x / 32 as a value that the compiler knows to be the same in the whole warp
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0); }

// ---- forward ---------------------------------------------------------------------------------
// Blocks an SM that the registers are to leave room for.  The exact gates of fp32 activations take more
// than the 80 registers of three blocks (B1 H16 L65536 d64, log gates: 125 us and 144, with bf16 gates
// 120 and 127); gates that are values do not (124 us, with the bound of two 130).
template <typename T, int KIND, int V, int R> constexpr int fwd_blocks()
{
    return V == 1 && R == 16 && (sizeof(T) < 4 || KIND == LA_GATE_VALUE) ? 3 : 2;
}

template <typename T, typename G, int KIND, bool COMP, int V, bool SPLIT>
__global__ void __launch_bounds__(REC_THREADS, fwd_blocks<T, KIND, V, RecSmem<T, G, V, false, SPLIT>::R>())
    rec_fwd_kernel(const RecArgs a)
{
    using Sm = RecSmem<T, G, V, false, SPLIT>;
    constexpr int CW = 32 * V, ST = Sm::STAGES, R = Sm::R, TILE = Sm::TILE;
    extern __shared__ __align__(16) unsigned char smem[];
    Fold<V> *const agg = (Fold<V> *)smem;            // folds of the warps
    Ch<V> *const begin = (Ch<V> *)(smem + Sm::AGG);  // states before them
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int split = SPLIT ? a.split : 1, rank = SPLIT ? blockIdx.x % split : 0, blk = blockIdx.x / split;
    const int bh = blk / a.ncb, c0 = blk % a.ncb * CW, b = bh / a.H, hd = bh % a.H;
    const int c = c0 + lane * V;
    const bool on = c < a.d;  // lanes without a channel compute on what shared memory holds
    const T *x = (const T *)a.x + row_of(a.vx, b, hd, 0) + c0;
    const G *g = (const G *)a.g + row_of(a.vg, b, hd, 0) + c0;
    T *out = (T *)a.out + row_of(a.vo, b, hd, 0) + c0;
    const int n = rows_of(a, b), nc = (a.L + RC - 1) / RC;
    const int nt = (a.L + TILE - 1) / TILE, steps = (nt + split - 1) / split;
    unsigned char *const ring = smem + Sm::HEAD + warp * Sm::SLOT;
    auto first_row = [&](int k) { return (k * split + rank) * TILE + warp * R; };
    int in = 0, at = 0;  // ring slots of the next copy and the next step
    auto load = [&](int k) {
        if (k < steps) {
            const int t0 = first_row(k), rows = min(n - t0, R);
            T *sx = (T *)(ring + in * Sm::STAGE);
            copy_rows<T, R, CW>(sx, x + t0 * a.vx.l, a.vx.l, rows, a.d - c0, a.grx, lane);
            copy_rows<G, R, CW>((G *)(sx + R * CW), g + t0 * a.vg.l, a.vg.l, rows, a.d - c0, a.grg, lane,
                                keep_gate<KIND>());
        }
        cp_commit();
        in = in + 1 == ST ? 0 : in + 1;
    };
    Ch<V> carry = all<V>(0.f);
    if (a.h0 && on)
#pragma unroll
        for (int v = 0; v < V; ++v) carry.v[v] = a.h0[(size_t)bh * a.d + c + v];

    using Pr = Pairs<V, R>;
    static_assert(!SPLIT || V == 1, "clusters: one channel a lane");
    Peers peers;
#pragma unroll
    for (int k = 0; k < ST - 1; ++k) load(k);
    if constexpr (SPLIT) peers.init(smem + Sm::PEERS, rank, a);
    int buf = 0;
    uint32_t parity = 0;
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
        cp_wait<ST - 2>();
        __syncwarp();
        load(k + ST - 1);  // into the slot of step k - 1, which the whole warp has finished
        const T *const sx = (const T *)(ring + at * Sm::STAGE) + lane * V;
        const G *const sg = (const G *)(ring + at * Sm::STAGE + sizeof(T) * R * CW) + lane * V;
        at = at + 1 == ST ? 0 : at + 1;
        const int t0 = first_row(k), rows = min(n - t0, R);
        // gates and what joins the state; their fold goes to the warps of the tile
        Ch<2> ga[Pr::N], bx[Pr::N], p, f;
        Fold<V> own{all<V>(1.f), all<V>(0.f)};
        if (rows > 0) {
#pragma unroll
            for (int i = 0; i < Pr::N; ++i) {
                const Ch<2> xv = Pr::get(sx, i);
                Ch<2> w;
                gate_of<KIND, COMP, ACC<T>, 2>(Pr::get(sg, i), ga[i], w);
                bx[i] = COMP ? mul(w, xv) : xv;
            }
            p = ga[0];
            f = bx[0];
#pragma unroll
            for (int i = 1; i < Pr::N; ++i) {
                f = fma(ga[i], f, bx[i]);
                p = mul(p, ga[i]);
            }
            own = Pr::join(p, f);
            if (on && !finite(own.h)) own = fold_rows<T, G, KIND, COMP, V>(sx, sg, rows);
            else if (on && !regular(own.p)) own.p = product_exact<G, KIND, V, R>(sg, own.p);
        }
        agg[warp * 32 + lane] = own;
        __syncthreads();
        if (warp == 0) {
            const Fold<V> *const f8 = agg + lane;
            Ch<V> e = carry;
            if constexpr (SPLIT) {
                // the fold of the tile, for the other blocks
                Fold<V> t = f8[0];
                bool zero = t.p.v[0] == 0.f;
#pragma unroll
                for (int w = 1; w < REC_W; ++w) {
                    const Fold<V> q = f8[w * 32];
                    t.h = fma(q.p, t.h, q.h);
                    t.p = mul(q.p, t.p);
                    zero = zero || q.p.v[0] == 0.f;
                }
                if (on && !finite(t.h)) t = join_exact<V>(f8, 32, REC_W);
                else t.p.v[0] = zero ? 0.f : t.p.v[0] == 0.f ? least(t.p.v[0]) : t.p.v[0];
                peers.publish(buf, lane, t);
                e = peers.over(buf, parity, lane, on, carry);
            }
            const Ch<V> start = e;
#pragma unroll
            for (int w = 0; w < REC_W; ++w) {
                begin[w * 32 + lane] = e;
                const Fold<V> q = f8[w * 32];
                e = fma(q.p, e, q.h);
            }
            if (on && !finite(e)) e = begin_exact<V>(begin + lane, f8, 32, start);
            if constexpr (!SPLIT) carry = e;
        }
        __syncthreads();
        const Ch<V> h = begin[warp * 32 + lane];
        if (a.chunks && t0 % RC == 0 && t0 < a.L && on)
#pragma unroll
            for (int v = 0; v < V; ++v) a.chunks[((size_t)bh * nc + t0 / RC) * a.d + c + v] = h.v[v];
        T *const o = out + t0 * a.vo.l + lane * V;
        bool tame = rows == R;
        if (rows == R) {
            Ch<2> y = Pr::spread(h, p, f);
            T *q = o, *q2 = o + Pr::N * a.vo.l;
#pragma unroll
            for (int i = 0; i < Pr::N; ++i, q += a.vo.l, q2 += a.vo.l) {
                y = fma(ga[i], y, bx[i]);
                if (on) Pr::put(q, q2, y);
            }
            tame = finite(y);
        }
        if (!tame && on && t0 < a.L)
            finish_rows<T, G, KIND, COMP, V>(sx, sg, rows, min(a.L - t0, R), h, o, a.vo.l);
        if (++buf == REC_BUFS) {
            buf = 0;
            parity ^= 1;
        }
    }
    if constexpr (SPLIT) {
        cluster_barrier();  // nothing is sent to a block that has ended
        if (warp == 0) peers.settle(buf == 0 ? REC_BUFS - 1 : buf - 1, buf == 0 ? parity ^ 1 : parity);
    }
    if (a.h_last && rank == 0 && warp == 0 && on)
#pragma unroll
        for (int v = 0; v < V; ++v) a.h_last[(size_t)bh * a.d + c + v] = carry.v[v];
}

// ---- backward ----------------------------------------------------------------------------------
// The tiles from the last to the first.  h before each row is run forward again from the state
// that the forward left for the tile.
template <typename T, typename G, int KIND, bool COMP, bool SPLIT>
__global__ void __launch_bounds__(REC_THREADS, 2) rec_bwd_kernel(const RecArgs a)
{
    constexpr int V = 1;
    using Sm = RecSmem<T, G, V, true, SPLIT>;
    constexpr int CW = 32 * V, ST = Sm::STAGES, R = Sm::R, TILE = Sm::TILE;
    constexpr bool WANT_C = COMP || KIND == LA_GATE_SIGMOID;
    extern __shared__ __align__(16) unsigned char smem[];
    Fold<V> *const agg = (Fold<V> *)smem;            // (P, E) of the warps
    Ch<V> *const front = (Ch<V> *)(smem + Sm::AGG);  // their H
    Ch<V> *const begin = front + REC_W * 32, *const behind = begin + REC_W * 32;  // states before, e behind them
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int split = SPLIT ? a.split : 1, rank = SPLIT ? blockIdx.x % split : 0, blk = blockIdx.x / split;
    const int bh = blk / a.ncb, c0 = blk % a.ncb * CW, b = bh / a.H, hd = bh % a.H;
    const int c = c0 + lane * V;
    const bool on = c < a.d;  // lanes without a channel compute on what shared memory holds
    const T *x = (const T *)a.x + row_of(a.vx, b, hd, 0) + c0;
    const G *g = (const G *)a.g + row_of(a.vg, b, hd, 0) + c0;
    const T *dout = (const T *)a.dout + row_of(a.vo, b, hd, 0) + c0;
    T *dx = (T *)a.dx + row_of(a.vdx, b, hd, 0) + c0;
    G *dg = (G *)a.dg + row_of(a.vdg, b, hd, 0) + c0;
    const int n = rows_of(a, b), nc = (a.L + RC - 1) / RC;
    const int nt = (a.L + TILE - 1) / TILE, steps = (nt + split - 1) / split;
    unsigned char *const ring = smem + Sm::HEAD + warp * Sm::SLOT;
    // a step's tiles run backwards; before the first tile there are none (negative rows)
    auto first_row = [&](int k) { return (nt - 1 - (k * split + rank)) * TILE + warp * R; };
    int in = 0, at = 0;
    auto load = [&](int k) {
        if (k < steps && first_row(k) >= 0) {
            const int t0 = first_row(k), rows = min(n - t0, R);
            T *sx = (T *)(ring + in * Sm::STAGE), *sd = sx + R * CW;
            copy_rows<T, R, CW>(sx, x + t0 * a.vx.l, a.vx.l, rows, a.d - c0, a.grx, lane);
            copy_rows<T, R, CW>(sd, dout + t0 * a.vo.l, a.vo.l, rows, a.d - c0, a.gro, lane);
            copy_rows<G, R, CW>((G *)(sd + R * CW), g + t0 * a.vg.l, a.vg.l, rows, a.d - c0, a.grg, lane,
                                keep_gate<KIND>());
        }
        cp_commit();
        in = in + 1 == ST ? 0 : in + 1;
    };
    Ch<V> carry = all<V>(0.f);  // a_{t+1} e_{t+1}
    if (a.dh_last && on)
#pragma unroll
        for (int v = 0; v < V; ++v) carry.v[v] = a.dh_last[(size_t)bh * a.d + c + v];
#pragma unroll
    for (int k = 0; k < ST - 1; ++k) load(k);
    using Pr = Pairs<V, R>;
    Peers peers;
    if constexpr (SPLIT) peers.init(smem + Sm::PEERS, rank, a);
    int buf = 0;
    uint32_t parity = 0;
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
        const int tile = nt - 1 - (k * split + rank), t0 = first_row(k);
        const int rows = tile < 0 ? 0 : min(n - t0, R);
        Ch<V> before = all<V>(0.f);  // the state before the tile
        if (warp == 1 && on && tile >= 0)
#pragma unroll
            for (int v = 0; v < V; ++v)
                before.v[v] = a.chunks_in[((size_t)bh * nc + tile * (TILE / RC)) * a.d + c + v];
        cp_wait<ST - 2>();
        __syncwarp();
        load(k + ST - 1);  // into the slot of step k - 1, which the whole warp has finished
        const T *const sx = (const T *)(ring + at * Sm::STAGE) + lane * V, *const sd = sx + R * CW;
        const G *const sg = (const G *)(ring + at * Sm::STAGE + 2 * sizeof(T) * R * CW) + lane * V;
        at = at + 1 == ST ? 0 : at + 1;
        // hb: w x, then the state before the row; cc: 1 - a
        Ch<2> ga[Pr::N], hb[Pr::N], cc[Pr::N], p, f, g2;
        BwdFold<V> own{all<V>(1.f), all<V>(0.f), all<V>(0.f)};
        if (rows > 0) {
#pragma unroll
            for (int i = 0; i < Pr::N; ++i) {
                const Ch<2> xv = Pr::get(sx, i);
                gate_of<KIND, WANT_C, ACC<T>, 2>(Pr::get(sg, i), ga[i], cc[i]);
                hb[i] = COMP ? mul(cc[i], xv) : xv;
            }
            p = ga[0];
            f = hb[0];
#pragma unroll
            for (int i = 1; i < Pr::N; ++i) {
                f = fma(ga[i], f, hb[i]);
                p = mul(p, ga[i]);
            }
            g2 = mul(ga[Pr::N - 1], Pr::get(sd, Pr::N - 1));
#pragma unroll
            for (int i = Pr::N - 2; i >= 0; --i) g2 = mul(ga[i], add(g2, Pr::get(sd, i)));
            const Fold<V> o = Pr::join(p, f);
            own = {o.p, o.h, Pr::join_back(p, g2)};
            if (on && (!finite(own.h) || !finite(own.e))) own = fold_rows_bwd<T, G, KIND, COMP, V>(sx, sd, sg, rows);
            else if (on && !regular(own.p)) own.p = product_exact<G, KIND, V, R>(sg, own.p);
        }
        agg[warp * 32 + lane] = Fold<V>{own.p, own.e};
        front[warp * 32 + lane] = own.h;
        __syncthreads();
        const Fold<V> *const f8 = agg + lane;
        if (warp == 0) {  // e over the warps, the last one first
            Ch<V> e = carry;
            if constexpr (SPLIT) {
                Fold<V> t = f8[(REC_W - 1) * 32];
                bool zero = t.p.v[0] == 0.f;
#pragma unroll
                for (int w = REC_W - 2; w >= 0; --w) {
                    const Fold<V> q = f8[w * 32];
                    t.h = fma(q.p, t.h, q.h);
                    t.p = mul(q.p, t.p);
                    zero = zero || q.p.v[0] == 0.f;
                }
                if (on && !finite(t.h)) t = join_exact<V>(f8 + (REC_W - 1) * 32, -32, REC_W);
                else t.p.v[0] = zero ? 0.f : t.p.v[0] == 0.f ? least(t.p.v[0]) : t.p.v[0];
                peers.publish(buf, lane, t);
                e = peers.over(buf, parity, lane, on, carry);
            }
            const Ch<V> start = e;
#pragma unroll
            for (int w = REC_W - 1; w >= 0; --w) {
                behind[w * 32 + lane] = e;
                const Fold<V> q = f8[w * 32];
                e = fma(q.p, e, q.h);
            }
            if (on && !finite(e)) e = begin_exact<V>(behind + (REC_W - 1) * 32 + lane, f8 + (REC_W - 1) * 32, -32, start);
            if constexpr (!SPLIT) carry = e;
        } else if (warp == 1) {  // h over the warps
            Ch<V> h = before;
#pragma unroll
            for (int w = 0; w < REC_W; ++w) {
                begin[w * 32 + lane] = h;
                h = fma(f8[w * 32].p, h, front[w * 32 + lane]);
            }
            if (on && !finite(h)) {
                h = before;
#pragma unroll 1
                for (int w = 0; w < REC_W; ++w) {
                    begin[w * 32 + lane] = h;
                    h = step(f8[w * 32].p, h, front[w * 32 + lane]);
                }
            }
        }
        __syncthreads();
        const Ch<V> h = begin[warp * 32 + lane], e = behind[warp * 32 + lane];
        T *const ox = dx + t0 * a.vdx.l + lane * V;
        G *const og = dg + t0 * a.vdg.l + lane * V;
        bool tame = rows == R;
        if (rows == R) {
            Ch<2> y = Pr::spread(h, p, f), z = Pr::spread_back(e, p, g2);
#pragma unroll
            for (int i = 0; i < Pr::N; ++i) {
                const Ch<2> bx = hb[i];
                hb[i] = y;
                y = fma(ga[i], y, bx);
            }
            // while h and e are finite, a slope of 0 makes its product 0 by itself
            T *px = ox + (Pr::N - 1) * a.vdx.l, *px2 = px + Pr::N * a.vdx.l;
            G *pg = og + (Pr::N - 1) * a.vdg.l, *pg2 = pg + Pr::N * a.vdg.l;
#pragma unroll
            for (int i = Pr::N - 1; i >= 0; --i) {
                z = add(z, Pr::get(sd, i));  // e_t
                const Ch<2> rx = COMP ? mul(cc[i], z) : z, ae = mul(ga[i], z);
                Ch<2> q = hb[i];
                if (COMP) q = fma(Pr::get(sx, i), all<2>(-1.f), q);
                const Ch<2> se = KIND == LA_GATE_VALUE ? z : KIND == LA_GATE_LOG ? ae : mul(cc[i], ae);
                if (on) {
                    Pr::put(px, px2, rx);
                    Pr::put(pg, pg2, mul(se, q));
                }
                z = ae;
                px -= a.vdx.l;
                px2 -= a.vdx.l;
                pg -= a.vdg.l;
                pg2 -= a.vdg.l;
            }
            tame = finite(y) && finite(z);
        }
        if (!tame && on && tile >= 0 && t0 < a.L)
            finish_rows_bwd<T, G, KIND, COMP, V>(sx, sd, sg, rows, min(a.L - t0, R), h, e, ox, a.vdx.l, og, a.vdg.l);
        if (++buf == REC_BUFS) {
            buf = 0;
            parity ^= 1;
        }
    }
    if constexpr (SPLIT) {
        cluster_barrier();  // nothing is sent to a block that has ended
        if (warp == 0) peers.settle(buf == 0 ? REC_BUFS - 1 : buf - 1, buf == 0 ? parity ^ 1 : parity);
    }
    if (a.dh0 && rank == 0 && warp == 0 && on)
#pragma unroll
        for (int v = 0; v < V; ++v) a.dh0[(size_t)bh * a.d + c + v] = carry.v[v];
}

constexpr int STEP_THREADS = 128;

template <typename T, typename G, int KIND, bool COMP>
__global__ void __launch_bounds__(STEP_THREADS) rec_step_kernel(const T *x, const G *g, float *state, T *out,
                                                                long long n)
{
    const long long i = (long long)blockIdx.x * STEP_THREADS + threadIdx.x;
    if (i >= n) return;
    Ch<1> ga, c;
    gate_exact<KIND, COMP, ACC<T>, 1>({{to_f32(g[i])}}, ga, c);
    const Ch<1> xv{{to_f32(x[i])}}, h = step(ga, {{state[i]}}, COMP ? mul(c, xv) : xv);
    state[i] = h.v[0];
    out[i] = from_f32<T>(h.v[0]);
}

// ---- host side ---------------------------------------------------------------------------------
int granule(const void *p, const View &v, const RecArgs &a, size_t elem)
{
    for (size_t g : {(size_t)16, (size_t)4})
        if (g > elem ? rows_aligned(p, v, a.B, a.H, a.L, elem, g) && a.d * elem % g == 0 : g == elem) return (int)g;
    return 2;
}

// A kernel's launches: attributes set and cluster sizes looked up once per device.
struct RecKernel {
    const void *fn;
    size_t (*smem)(int split);
    std::atomic<bool> ready[64];
    std::atomic<int> fit[64][REC_MAX_SPLIT + 1];  // clusters of that size on the GPU at once, 0: not looked up

    void config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute &at, int split) const
    {
        cfg = {};
        cfg.blockDim = dim3(REC_THREADS);
        cfg.dynamicSmemBytes = smem(split);
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = (unsigned)split;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = split > 1 ? 1 : 0;
    }
    bool prepare(int dev, bool split)
    {
        if (ready[dev]) return true;
        const size_t most = smem(split ? REC_MAX_SPLIT : 1);
        if (status_of(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most)) != LA_OK ||
            (split && status_of(cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != LA_OK))
            return false;
        return ready[dev] = true;
    }
    // The largest cluster, and no more blocks of it than tiles, with which all blocks run at once:
    // a second wave of clusters costs as much as the first (48 blocks, 16384 rows, bf16: 54 us with
    // clusters of 5, 65 with 8, which take two waves, 63 with 4).
    int choose(int dev, long long blocks, long long tiles)
    {
        for (int s = (int)std::min(tiles, (long long)REC_MAX_SPLIT); s > 1; --s) {
            int n = fit[dev][s];
            if (!n) {
                cudaLaunchConfig_t cfg;
                cudaLaunchAttribute at;
                config(cfg, at, s);
                cfg.gridDim = dim3((unsigned)s);
                if (status_of(cudaOccupancyMaxActiveClusters(&n, fn, &cfg)) != LA_OK || n <= 0) n = -1;
                fit[dev][s] = n;
            }
            if (n >= blocks) return s;
        }
        return 1;
    }
    int launch(RecArgs &a, cudaStream_t stream) const
    {
        const long long blocks = (long long)a.B * a.H * a.ncb * a.split;
        if (blocks > INT_MAX) return LA_ERR_SHAPE;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute at;
        config(cfg, at, a.split);
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.stream = stream;
        void *args[] = {&a};
        return status_of(cudaLaunchKernelExC(&cfg, fn, args));
    }
};

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

template <bool BWD>
struct LaunchRec {
    RecArgs &a;
    int sms, dev;
    cudaStream_t s;

    template <typename T, typename G, int KIND, bool COMP, int V, bool SPLIT> static RecKernel &kernel()
    {
        const void *fn;
        if constexpr (BWD) fn = (const void *)rec_bwd_kernel<T, G, KIND, COMP, SPLIT>;
        else fn = (const void *)rec_fwd_kernel<T, G, KIND, COMP, V, SPLIT>;
        static RecKernel k{fn, &RecSmem<T, G, V, BWD, SPLIT>::bytes};
        return k;
    }
    bool pairs(const void *p, const View &v) const { return rows_aligned(p, v, a.B, a.H, a.L, 2, 4); }

    // Forward, two channels a lane for bf16 (fp32 would leave one block an SM) where they are aligned
    // together and the blocks of 64 channels alone give every SM one: half the instructions a row
    // (B8 H16 L8192 d128: 131 us and 174).  Else one channel a lane, for twice the blocks, and
    // clusters over the rows.
    template <typename T, typename G, int KIND, bool COMP> int operator()() const
    {
        const long long heads = (long long)a.B * a.H;
        a.split = 1;
        if constexpr (!BWD && sizeof(T) + sizeof(G) == 4) {
            a.ncb = (a.d + 63) / 64;
            if (a.d % 2 == 0 && a.d > 32 && heads * a.ncb >= sms && pairs(a.x, a.vx) && pairs(a.g, a.vg) &&
                pairs(a.out, a.vo)) {
                RecKernel &k = kernel<T, G, KIND, COMP, 2, false>();
                return k.prepare(dev, false) ? k.launch(a, s) : LA_ERR_CUDA;
            }
        }
        a.ncb = (a.d + 31) / 32;
        constexpr int TILE = RecSmem<T, G, 1, BWD, true>::TILE;
        const long long blocks = heads * a.ncb, tiles = ((long long)a.L + TILE - 1) / TILE;
        if (blocks <= sms && tiles > 1) {
            RecKernel &k = kernel<T, G, KIND, COMP, 1, true>();
            if (!k.prepare(dev, true)) return LA_ERR_CUDA;
            a.split = k.choose(dev, blocks, tiles);
            if (a.split > 1) return k.launch(a, s);
        }
        RecKernel &k = kernel<T, G, KIND, COMP, 1, false>();
        return k.prepare(dev, false) ? k.launch(a, s) : LA_ERR_CUDA;
    }
};

// The limit of a wait, and the test knob that makes it run out.
void set_limits(RecArgs &a)
{
    const char *e = getenv("LA_DEBUG_TIMEOUT_NS"), *st = getenv("LA_DEBUG_STALL");
    a.timeout_ns = e && *e ? strtoull(e, nullptr, 10) : 2000000000ull;
    a.debug_stall = st && *st && *st != '0';
}

struct LaunchStep {
    const void *x, *g;
    float *state;
    void *out;
    long long n;
    cudaStream_t s;
    template <typename T, typename G, int KIND, bool COMP> int operator()() const
    {
        const unsigned grid = (unsigned)((n + STEP_THREADS - 1) / STEP_THREADS);
        return la::launch(rec_step_kernel<T, G, KIND, COMP>, dim3(grid), STEP_THREADS, 0, s, (const T *)x, (const G *)g, state, (T *)out, n);
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
    a.grx = granule(x, a.vx, a, e);
    a.grg = granule(gate, a.vg, a, dtype_size(gate_dtype));
    const int sms = device_sms();
    int dev = 0;
    a.err = err_ptr();
    set_limits(a);
    if (sms <= 0 || !a.err || cudaGetDevice(&dev) != cudaSuccess) return LA_ERR_CUDA;
    return dispatch(dtype, gate_dtype, gate_kind, complement != 0, LaunchRec<false>{a, sms, dev, (cudaStream_t)stream});
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
    a.grx = granule(x, a.vx, a, e);
    a.grg = granule(gate, a.vg, a, eg);
    a.gro = granule(dout, a.vo, a, e);
    const int sms = device_sms();
    int dev = 0;
    a.err = err_ptr();
    set_limits(a);
    if (sms <= 0 || !a.err || cudaGetDevice(&dev) != cudaSuccess) return LA_ERR_CUDA;
    return dispatch(dtype, gate_dtype, gate_kind, complement != 0, LaunchRec<true>{a, sms, dev, (cudaStream_t)stream});
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
