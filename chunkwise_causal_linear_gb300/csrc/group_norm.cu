// group_norm.cu -- group norm over one head's channels of one token, with weight, bias and an
// activation or a gate, and its gradients (sm_103a).
//
// Bound by memory: x and gate read once, out written once.  A group is held in the registers of
// TPG threads (8 to 32 lanes of a warp, or the block for d above 1024), so mean, centred
// variance and the output come from one read, which is on its way some rows ahead.  A block stays with one head and walks over its
// tokens: weight and bias stay in registers, and so do the sums of their gradients, which leave
// the block once.  The blocks' sums are joined by a second, small kernel in a fixed order.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "layer.cuh"
#include "tc_common.cuh"

namespace la {

namespace {

constexpr int GN_THREADS = 256;
constexpr int GN_MAX_D = 8192;

struct GnArgs {
    const void *x, *gate, *dout;
    void *out, *dx, *dgate;
    const float *w, *b;
    float *dw, *db, *part;  // part: [nb][2][H d], the blocks' sums for dw and db
    View vx, vg, vo, vdx, vdg;
    int B, H, L, d, center, act;
    float eps, inv_d;
    int nb;  // blocks of a head
};

// ---- VEC neighbouring channels, in pairs -------------------------------------------------------
template <int VEC> constexpr int WIDTH = VEC > 1 ? 2 : 1;
template <int VEC> using Vec = Ch<WIDTH<VEC>>;  // [VEC / WIDTH] of them hold VEC channels

template <int VEC> __device__ __forceinline__ void load(const __nv_bfloat16 *p, Vec<VEC> *f)
{
    if constexpr (VEC == 8) {
        const uint4 t = *(const uint4 *)p;
        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = {{tcc::bf_lo(w[i]), tcc::bf_hi(w[i])}};
    } else if constexpr (VEC == 2) {
        const uint32_t w = *(const uint32_t *)p;
        f[0].v[0] = tcc::bf_lo(w);
        f[0].v[1] = tcc::bf_hi(w);
    } else {
        f[0].v[0] = __bfloat162float(*p);
    }
}
template <int VEC> __device__ __forceinline__ void load(const float *p, Vec<VEC> *f)
{
    if constexpr (VEC == 4) {
        const float4 w = *(const float4 *)p;
        f[0].v[0] = w.x;
        f[0].v[1] = w.y;
        f[1].v[0] = w.z;
        f[1].v[1] = w.w;
    } else {
        f[0].v[0] = *p;
    }
}
__device__ __forceinline__ uint32_t bf_pair(const Ch<2> &f)
{
    const __nv_bfloat162 t = __floats2bfloat162_rn(f.v[0], f.v[1]);
    return *(const uint32_t *)&t;
}
template <int VEC> __device__ __forceinline__ void store(__nv_bfloat16 *p, const Vec<VEC> *f)
{
    if constexpr (VEC == 8) *(uint4 *)p = make_uint4(bf_pair(f[0]), bf_pair(f[1]), bf_pair(f[2]), bf_pair(f[3]));
    else if constexpr (VEC == 2) *(uint32_t *)p = bf_pair(f[0]);
    else *p = __float2bfloat16_rn(f[0].v[0]);
}
template <int VEC> __device__ __forceinline__ void store(float *p, const Vec<VEC> *f)
{
    if constexpr (VEC == 4) *(float4 *)p = make_float4(f[0].v[0], f[0].v[1], f[1].v[0], f[1].v[1]);
    else *p = f[0].v[0];
}

// ---- sums over the threads of a group, the same in every one of them ---------------------------
template <int TPG, int N> __device__ __forceinline__ void group_sum(float (&v)[N], float *sm)
{
#pragma unroll
    for (int o = (TPG > 32 ? 32 : TPG) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (TPG > 32) {
        constexpr int W = TPG / 32;
        const int warp = threadIdx.x >> 5;
        __syncthreads();  // the sums before these have been read
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) sm[warp * N + i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += sm[w * N + i];
    }
}

// 1 / (1 + e^-z); 0 where it is below the normal range.  Off by at most (7 + 2.5 |z|) 2^-24 relatively,
// for bf16, whose outputs are rounded by up to 2^-8; by 9 2^-24 for fp32 (FINE: B8 H16 L4096 d128 with a
// gate 128 us and 218 backward, 127 and 214 without; with SiLU alone 97 and 146, 93 and 144).
template <bool FINE, int W> __device__ __forceinline__ Ch<W> sigmoid(const Ch<W> &z)
{
    Ch<W> e;
    if constexpr (FINE) {
        // from 88.5 on the reciprocal is 0
#pragma unroll
        for (int i = 0; i < W; ++i) e.v[i] = max_nan(min_nan(-z.v[i], 88.5f), -150.f);
        e = exp_fine(e);
    } else {
        e = mul(z, all<W>(-1.44269504f));
#pragma unroll
        for (int i = 0; i < W; ++i) e.v[i] = ex2(e.v[i]);
    }
    e = add(e, all<W>(1.f));
#pragma unroll
    for (int i = 0; i < W; ++i) e.v[i] = rcp(e.v[i]);
    return e;
}

// The tokens of a block's group of threads, r = first, first + step, ..., and where a tensor's rows
// of them are.
struct Walk {
    int b, t, sb, st, L;
    bool wrap;
    __device__ Walk(long long first, long long step, int L_) : L(L_), wrap(false)
    {
        b = (int)(first / L);
        t = (int)(first % L);
        sb = (int)(step / L);
        st = (int)(step % L);
    }
    __device__ __forceinline__ void next()
    {
        b += sb;
        t += st;
        wrap = t >= L;
        if (wrap) {
            t -= L;
            ++b;
        }
    }
};
template <typename T> struct Rows {
    T *p;
    long long by, back;  // a step, and what a step into the next sequence adds to it
    __device__ Rows(const void *base, const View &v, int h, const Walk &w)
        : p((T *)base + row_of(v, w.b, h, w.t)), by(w.sb * v.b + w.st * v.l), back(v.b - w.L * v.l)
    {
    }
    __device__ __forceinline__ void next(const Walk &w) { p += w.wrap ? by + back : by; }
};

template <int VEC, int NV> struct Group {
    static constexpr int W = WIDTH<VEC>, N = VEC / W;
    Vec<VEC> v[NV][N];
};
template <typename T, int VEC, int TPG, int NV>
__device__ __forceinline__ void write(const Group<VEC, NV> &g, T *p, int lane, int d)
{
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPG + lane) * VEC;
        if (c < d) store<VEC>(p + c, g.v[i]);
    }
}

// ---- the rows on their way ------------------------------------------------------------------------
// Each thread copies its own vectors of the next rows into its own places in shared memory, so
// nothing is synchronised and no register waits for memory.  Single bf16 values, which cp.async
// does not copy, are loaded when they are needed.
template <typename T, int VEC, int TPG, int NV, int ARRAYS, int BLOCKS> struct Ring {
    static constexpr int BYTES = VEC * (int)sizeof(T);  // of a vector
    static constexpr bool USED = BYTES >= 4;
    static constexpr int STAGE = ARRAYS * NV * BYTES * GN_THREADS;
    static constexpr int FIT = (160 * 1024) / (BLOCKS * STAGE);
    static constexpr int ST = !USED ? 1 : FIT > 6 ? 6 : FIT < 2 ? 2 : FIT;
    static constexpr int SMEM = USED ? ST * STAGE : 0;
    unsigned char *sm;
    int in = 0, at = 0;

    __device__ Ring(unsigned char *mem) : sm(mem + threadIdx.x * BYTES) {}
    __device__ __forceinline__ void copy(int array, const T *p, int lane, int d) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPG + lane) * VEC;
            const uint32_t to =
                (uint32_t)__cvta_generic_to_shared(sm + in * STAGE + (array * NV + i) * BYTES * GN_THREADS);
            if (c < d) {
                if constexpr (BYTES == 16)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p + c) : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(p + c) : "memory");
            }
        }
    }
    __device__ __forceinline__ void commit()
    {
        asm volatile("cp.async.commit_group;" ::: "memory");
        in = in + 1 == ST ? 0 : in + 1;
    }
    __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2 < 0 ? 0 : ST - 2) : "memory"); }
    __device__ __forceinline__ void take(int array, Group<VEC, NV> &g, int lane, int d, bool on) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const T *p = (const T *)(sm + at * STAGE + (array * NV + i) * BYTES * GN_THREADS);
            if (on && (i * TPG + lane) * VEC < d) {
                load<VEC>(p, g.v[i]);
            } else {
#pragma unroll
                for (int e = 0; e < Group<VEC, NV>::N; ++e) g.v[i][e] = all<WIDTH<VEC>>(0.f);
            }
        }
    }
    __device__ __forceinline__ void done() { at = at + 1 == ST ? 0 : at + 1; }
};
template <typename T, int VEC, int TPG, int NV>
__device__ __forceinline__ void read(Group<VEC, NV> &g, const T *p, int lane, int d, bool on)
{
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPG + lane) * VEC;
        if (on && c < d) {
            load<VEC>(p + c, g.v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < Group<VEC, NV>::N; ++e) g.v[i][e] = all<WIDTH<VEC>>(0.f);
        }
    }
}

// The inputs of a block's rows, one after the other.
template <typename T, int VEC, int TPG, int NV, int ARRAYS, int BLOCKS> struct Source {
    using R = Ring<T, VEC, TPG, NV, ARRAYS, BLOCKS>;
    R ring;
    Walk at;
    Rows<const T> p0, p1, p2;
    int lane, d, B;

    __device__ Source(unsigned char *mem, const Walk &w, const Rows<const T> &a0, const Rows<const T> &a1,
                      const Rows<const T> &a2, int lane_, const GnArgs &a)
        : ring(mem), at(w), p0(a0), p1(a1), p2(a2), lane(lane_), d(a.d), B(a.B)
    {
        if constexpr (R::USED)
#pragma unroll
            for (int i = 0; i < R::ST - 1; ++i) fetch();
    }
    __device__ __forceinline__ void step()
    {
        at.next();
        p0.next(at);
        if (ARRAYS > 1) p1.next(at);
        if (ARRAYS > 2) p2.next(at);
    }
    __device__ __forceinline__ void fetch()
    {
        if (at.b < B) {
            ring.copy(0, p0.p, lane, d);
            if (ARRAYS > 1) ring.copy(1, p1.p, lane, d);
            if (ARRAYS > 2) ring.copy(2, p2.p, lane, d);
        }
        ring.commit();
        step();
    }
    // the next row of each input, zeros where there is none
    __device__ __forceinline__ void next(Group<VEC, NV> *g, bool on)
    {
        if constexpr (R::USED) {
            ring.wait();
#pragma unroll
            for (int i = 0; i < ARRAYS; ++i) ring.take(i, g[i], lane, d, on);
            ring.done();
            fetch();
        } else {
            read<T, VEC, TPG, NV>(g[0], p0.p, lane, d, on);
            if (ARRAYS > 1) read<T, VEC, TPG, NV>(g[1], p1.p, lane, d, on);
            if (ARRAYS > 2) read<T, VEC, TPG, NV>(g[2], p2.p, lane, d, on);
            step();
        }
    }
};

template <int W> __device__ __forceinline__ float total(const Ch<W> &c)
{
    if constexpr (W == 2) return c.v[0] + c.v[1];
    else return c.v[0];
}

// x -> xh in place; returns rstd.  Channels past d count as nothing.
template <int VEC, int TPG, int NV>
__device__ __forceinline__ float normalise(Group<VEC, NV> &x, const GnArgs &a, int lane, float *sm)
{
    constexpr int W = Group<VEC, NV>::W, N = Group<VEC, NV>::N;
    if (a.center) {
        Ch<W> c = all<W>(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) c = add(c, x.v[i][e]);
        float s[1] = {total(c)};
        group_sum<TPG>(s, sm);
        const Ch<W> mean = all<W>(-s[0] * a.inv_d);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * TPG + lane) * VEC < a.d)
#pragma unroll
                for (int e = 0; e < N; ++e) x.v[i][e] = add(x.v[i][e], mean);
    }
    Ch<W> c = all<W>(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) c = fma(x.v[i][e], x.v[i][e], c);
    float q[1] = {total(c)};
    group_sum<TPG>(q, sm);
    const float rstd = rsqrtf(fmaf(q[0], a.inv_d, a.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) x.v[i][e] = mul(x.v[i][e], all<W>(rstd));
    return rstd;
}

// Weight and bias of the block's head: in registers where they are few, else read again.
template <int VEC, int TPG, int NV> struct Affine {
    static constexpr bool KEEP = NV * VEC <= 8;
    static constexpr int W = WIDTH<VEC>;
    Group<VEC, KEEP ? NV : 1> w_, b_;
    const float *w, *b;
    int lane, d;
    __device__ Affine(const GnArgs &a, int h, int lane_) : lane(lane_), d(a.d)
    {
        w = a.w ? a.w + (size_t)h * d : nullptr;
        b = a.b ? a.b + (size_t)h * d : nullptr;
        if constexpr (KEEP)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC / W; ++e) get(i, e, w_.v[i][e], b_.v[i][e]);
    }
    __device__ __forceinline__ void get(int i, int e, Ch<W> &wv, Ch<W> &bv) const
    {
        const int c = (i * TPG + lane) * VEC + e * W;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            wv.v[j] = w && c + j < d ? w[c + j] : 1.f;
            bv.v[j] = b && c + j < d ? b[c + j] : 0.f;
        }
    }
    __device__ __forceinline__ void at(int i, int e, Ch<W> &wv, Ch<W> &bv) const
    {
        if constexpr (KEEP) {
            wv = w_.v[i][e];
            bv = b_.v[i][e];
        } else {
            get(i, e, wv, bv);
        }
    }
};

// A group of a whole block holds up to GN_MAX_D channels; its vectors behind the last channel are left
// out of the activation (fp32, B4 H1 L4096 d2048: 203 us with them, 140 without).  Within a warp they
// are fewer, and the branch costs more (d1024: 66 us and 82).
template <int VEC, int TPG> __device__ __forceinline__ bool behind(int i, int d)
{
    return TPG > 32 && i > 0 && i * TPG * VEC >= d;
}

// Blocks an SM by the values a thread holds.
template <int VEC, int NV> __host__ __device__ constexpr int blocks_per_sm(bool bwd)
{
    return NV * VEC <= 8 ? (bwd ? 2 : 3) : NV * VEC <= 16 ? 2 : 1;
}
template <typename T, int VEC, int TPG, int NV, bool GATE, bool BWD>
using SourceOf = Source<T, VEC, TPG, NV, (BWD ? 2 : 1) + GATE, blocks_per_sm<VEC, NV>(BWD)>;

// What is asked for, known to the compiler: GATE and SILU.
template <typename T, int VEC, int TPG, int NV, bool GATE, bool SILU>
__global__ void __launch_bounds__(GN_THREADS, blocks_per_sm<VEC, NV>(false)) gn_fwd_kernel(const GnArgs a)
{
    constexpr int GPB = GN_THREADS / TPG, W = WIDTH<VEC>, N = VEC / W;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ float sm[GN_THREADS / 32];
    const int lane = threadIdx.x % TPG, group = threadIdx.x / TPG;
    const int h = blockIdx.x % a.H, part = blockIdx.x / a.H;
    const long long rows = (long long)a.B * a.L, first = (long long)part * GPB, step = (long long)a.nb * GPB;
    Walk at(first + group, step, a.L);
    const Rows<const T> px(a.x, a.vx, h, at), pz(a.gate, a.vg, h, at);
    Rows<T> po(a.out, a.vo, h, at);
    SourceOf<T, VEC, TPG, NV, GATE, false> src(dyn, at, px, pz, pz, lane, a);
    const Affine<VEC, TPG, NV> aff(a, h, lane);
    // every group of a warp (of the block, where the block is one) takes part in every turn's sums
    const int turns = (int)((rows - first + step - 1) / step);
    for (int k = 0; k < turns; ++k) {
        Group<VEC, NV> in[1 + GATE], &x = in[0], &z = in[GATE];
        const bool on = at.b < a.B;
        src.next(in, on);
        normalise<VEC, TPG, NV>(x, a, lane, sm);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (behind<VEC, TPG>(i, a.d)) continue;
                Ch<W> w, b;
                aff.at(i, e, w, b);
                const Ch<W> y = fma(x.v[i][e], w, b), g = GATE ? z.v[i][e] : y;
                const Ch<W> f = SILU ? mul(g, sigmoid<sizeof(T) == 4>(g)) : g;
                x.v[i][e] = GATE ? mul(y, f) : f;
            }
        if (on) write<T, VEC, TPG, NV>(x, po.p, lane, a.d);
        at.next();
        po.next(at);
    }
}

template <typename T, int VEC, int TPG, int NV, bool GATE, bool SILU>
__global__ void __launch_bounds__(GN_THREADS, blocks_per_sm<VEC, NV>(true)) gn_bwd_kernel(const GnArgs a)
{
    constexpr int GPB = GN_THREADS / TPG, W = WIDTH<VEC>, N = VEC / W;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ float sm[2 * GN_THREADS / 32];
    const int lane = threadIdx.x % TPG, group = threadIdx.x / TPG;
    const int h = blockIdx.x % a.H, part = blockIdx.x / a.H;
    const long long rows = (long long)a.B * a.L, first = (long long)part * GPB, step = (long long)a.nb * GPB;
    Walk at(first + group, step, a.L);
    const Rows<const T> px(a.x, a.vx, h, at), pz(a.gate, a.vg, h, at), pd(a.dout, a.vo, h, at);
    Rows<T> pdx(a.dx, a.vdx, h, at), pdz(a.dgate, a.vdg, h, at);
    SourceOf<T, VEC, TPG, NV, GATE, true> src(dyn, at, px, pd, pz, lane, a);
    const Affine<VEC, TPG, NV> aff(a, h, lane);
    Group<VEC, NV> dw = {}, db = {};
    const int turns = (int)((rows - first + step - 1) / step);
    for (int k = 0; k < turns; ++k) {
        Group<VEC, NV> in[2 + GATE], &x = in[0], &o = in[1], &z = in[1 + GATE];
        const bool on = at.b < a.B;
        src.next(in, on);
        const float rstd = normalise<VEC, TPG, NV>(x, a, lane, sm);
        Ch<W> s0 = all<W>(0.f), s1 = s0;  // sums of dy w and of dy w xh
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (behind<VEC, TPG>(i, a.d)) continue;
                Ch<W> w, b;
                aff.at(i, e, w, b);
                const Ch<W> xh = x.v[i][e], y = fma(xh, w, b), g = GATE ? z.v[i][e] : y;
                Ch<W> f = g, slope = all<W>(1.f);
                if (SILU) {
                    const Ch<W> sg = sigmoid<sizeof(T) == 4>(g);
                    f = mul(g, sg);
                    slope = fma(f, fma(sg, all<W>(-1.f), all<W>(1.f)), sg);  // sg (1 + g (1 - sg))
                }
                Ch<W> dy = o.v[i][e];
                if (GATE) {
                    z.v[i][e] = mul(mul(dy, y), slope);  // dgate
                    dy = mul(dy, f);
                } else {
                    dy = mul(dy, slope);
                }
                dw.v[i][e] = fma(dy, xh, dw.v[i][e]);
                db.v[i][e] = add(db.v[i][e], dy);
                dy = mul(dy, w);
                o.v[i][e] = dy;
                s0 = add(s0, dy);
                s1 = fma(dy, xh, s1);
            }
        float s[2] = {total(s0), total(s1)};
        group_sum<TPG>(s, sm);
        // dx = rstd (dy w - mean(dy w) - xh mean(dy w xh))
        const Ch<W> m1 = all<W>(a.center ? -s[0] * a.inv_d * rstd : 0.f), m2 = all<W>(-s[1] * a.inv_d * rstd),
                    r = all<W>(rstd);
        if (on) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < N; ++e) x.v[i][e] = fma(o.v[i][e], r, fma(x.v[i][e], m2, m1));
            write<T, VEC, TPG, NV>(x, pdx.p, lane, a.d);
            if (GATE) write<T, VEC, TPG, NV>(z, pdz.p, lane, a.d);
        }
        at.next();
        pdx.next(at);
        if (GATE) pdz.next(at);
    }
    if (!a.part) return;
    // the groups of the block joined, one after the other; the ring's memory is free now
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float *const sums = (float *)dyn;  // [2][GPB][d]
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPG + lane) * VEC;
        if (c < a.d)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                sums[group * a.d + c + e] = dw.v[i][e / W].v[e % W];
                sums[(GPB + group) * a.d + c + e] = db.v[i][e / W].v[e % W];
            }
    }
    __syncthreads();
    float *out = a.part + (size_t)part * 2 * a.H * a.d + (size_t)h * a.d;
    for (int c = threadIdx.x; c < 2 * a.d; c += GN_THREADS) {
        const int which = c >= a.d, cc = which ? c - a.d : c;
        const float *p = sums + (size_t)which * GPB * a.d + cc;
        float v = 0.f;
        for (int g = 0; g < GPB; ++g) v += p[g * a.d];
        out[(size_t)which * a.H * a.d + cc] = v;
    }
}

// dweight, dbias: the blocks' sums of 32 channels joined by 8 warps
__global__ void __launch_bounds__(GN_THREADS) gn_join_kernel(const GnArgs a)
{
    __shared__ float sm[2][8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long n = (long long)a.H * a.d, c = (long long)blockIdx.x * 32 + lane;
    tcc::pdl_wait();  // the blocks' sums are there
    float w = 0.f, b = 0.f;
    if (c < n)
        for (int p = warp; p < a.nb; p += 8) {
            w += a.part[(size_t)p * 2 * n + c];
            b += a.part[(size_t)p * 2 * n + n + c];
        }
    sm[0][warp][lane] = w;
    sm[1][warp][lane] = b;
    __syncthreads();
    if (warp < 2 && c < n) {
        float v = 0.f;
        for (int i = 0; i < 8; ++i) v += sm[warp][i][lane];
        float *out = warp ? a.db : a.dw;
        if (out) out[c] = v;
    }
}

// ---- host side -----------------------------------------------------------------------------------
// Blocks of a head: one wave of the GPU in all, because a block's ring takes some rows to fill;
// forward up to three where each still has 48 turns (B8 H16 L8192 d128: 126 us with three waves,
// 132 with one; B2 H12 L16384 d64: 31 with one, 34 with three).  The rows of a block's turn are taken
// from d alone; by_size() gives 32 (bf16, d <= 64) to 1 (single elements, d > 256), so that with few
// tokens some blocks have none and only write their sums of 0, and wide odd groups have more turns.
int blocks_of_head(int B, int H, int L, int d, int sms, bool bwd)
{
    const long long rows = (long long)B * L, gpb = d > 1024 ? 1 : d > 256 ? 8 : 16;
    long long want = std::max(1ll, (long long)sms * (bwd ? 2 : 3) / H);
    if (!bwd) want *= std::max(1ll, std::min(3ll, rows / (gpb * want * 48)));
    return (int)std::max(1ll, std::min(want, (rows + gpb - 1) / gpb));
}

template <auto KERN> using constant = std::integral_constant<decltype(KERN), KERN>;

// A kernel's limit of dynamic shared memory, set once per device.
template <auto KERN> bool raise_smem_limit(size_t bytes)
{
    static std::atomic<bool> done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (done[dev]) return true;
    if (status_of(cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)) != LA_OK) return false;
    return done[dev] = true;
}

template <typename T, int VEC, int TPG, int NV, bool BWD> int launch_gn(const GnArgs &a, cudaStream_t s)
{
    const long long blocks = (long long)a.nb * a.H;
    if (blocks > INT_MAX) return LA_ERR_SHAPE;
    auto go = [&](auto kernel, auto gate) {
        constexpr auto kern = decltype(kernel)::value;
        constexpr size_t ring = SourceOf<T, VEC, TPG, NV, decltype(gate)::value, BWD>::R::SMEM;
        // the limit is set once, to the most that any d asks for: two threads with different d must not
        // undercut each other between the attribute and the launch
        constexpr size_t most = std::max(ring, BWD ? sizeof(float) * 2 * GN_THREADS * VEC * NV : 0);
        if (most > 47 * 1024 && !raise_smem_limit<kern>(most)) return (int)LA_ERR_CUDA;
        size_t smem = ring;
        if (BWD && a.part) smem = std::max(smem, sizeof(float) * 2 * (GN_THREADS / TPG) * a.d);
        return launch(kern, dim3((unsigned)blocks), GN_THREADS, smem, s, a);
    };
    const bool silu = a.act == LA_ACT_SILU;
    const std::true_type yes;
    const std::false_type no;
    auto choose = [&](auto gate, auto silu) {
        constexpr bool GATE = decltype(gate)::value, SILU = decltype(silu)::value;
        if constexpr (BWD) return go(constant<gn_bwd_kernel<T, VEC, TPG, NV, GATE, SILU>>(), gate);
        else return go(constant<gn_fwd_kernel<T, VEC, TPG, NV, GATE, SILU>>(), gate);
    };
    if (a.gate) return silu ? choose(yes, yes) : choose(yes, no);
    return silu ? choose(no, yes) : choose(no, no);
}

// Threads and vectors of a group by its number of vectors: the fewest registers that hold it, a
// block once a warp would need more than 32 values a lane.
template <typename T, int VEC, bool BWD> int by_size(const GnArgs &a, cudaStream_t s)
{
    const int nv = (a.d + VEC - 1) / VEC;
    if constexpr (VEC == 8) {
        if (nv <= 8) return launch_gn<T, VEC, 8, 1, BWD>(a, s);
        if (nv <= 16) return launch_gn<T, VEC, 16, 1, BWD>(a, s);
        if (nv <= 32) return launch_gn<T, VEC, 32, 1, BWD>(a, s);
        if (nv <= 64) return launch_gn<T, VEC, 32, 2, BWD>(a, s);
        if (nv <= 128) return launch_gn<T, VEC, 32, 4, BWD>(a, s);
        if (nv <= 256) return launch_gn<T, VEC, 256, 1, BWD>(a, s);
        return launch_gn<T, VEC, 256, 4, BWD>(a, s);
    } else if constexpr (VEC == 4) {
        if (nv <= 8) return launch_gn<T, VEC, 8, 1, BWD>(a, s);
        if (nv <= 16) return launch_gn<T, VEC, 8, 2, BWD>(a, s);
        if (nv <= 32) return launch_gn<T, VEC, 16, 2, BWD>(a, s);
        if (nv <= 64) return launch_gn<T, VEC, 32, 2, BWD>(a, s);
        if (nv <= 128) return launch_gn<T, VEC, 32, 4, BWD>(a, s);
        if (nv <= 256) return launch_gn<T, VEC, 32, 8, BWD>(a, s);
        return launch_gn<T, VEC, 256, 8, BWD>(a, s);
    } else {
        if (nv <= 32) return launch_gn<T, VEC, 32, 1, BWD>(a, s);
        if (nv <= 64) return launch_gn<T, VEC, 32, 2, BWD>(a, s);
        if (nv <= 128) return launch_gn<T, VEC, 32, 4, BWD>(a, s);
        if (nv <= 256) return launch_gn<T, VEC, 32, 8, BWD>(a, s);
        if (nv <= 1024) return launch_gn<T, VEC, 256, 4, BWD>(a, s);
        return launch_gn<T, VEC, 256, 32 / VEC, BWD>(a, s);
    }
}

template <bool BWD> int by_type(const GnArgs &a, int dtype, cudaStream_t s)
{
    const size_t e = dtype_size(dtype);
    auto fits = [&](int vec) {
        auto ok = [&](const void *p, const View &v) { return !p || rows_aligned(p, v, a.B, a.H, a.L, e, vec * e); };
        return a.d % vec == 0 && ok(a.x, a.vx) && ok(a.gate, a.vg) && ok(a.out, a.vo) && ok(a.dout, a.vo) &&
               ok(a.dx, a.vdx) && ok(a.dgate, a.vdg);
    };
    if (dtype == LA_F32) return fits(4) ? by_size<float, 4, BWD>(a, s) : by_size<float, 1, BWD>(a, s);
    if (fits(8)) return by_size<__nv_bfloat16, 8, BWD>(a, s);
    return fits(2) ? by_size<__nv_bfloat16, 2, BWD>(a, s) : by_size<__nv_bfloat16, 1, BWD>(a, s);
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
    if (d > GN_MAX_D) return LA_ERR_UNSUPPORTED;
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
    const int sms = device_sms();
    if (sms <= 0) return LA_ERR_CUDA;
    a.inv_d = 1.f / (float)d;
    a.nb = blocks_of_head(B, H, L, d, sms, false);
    return by_type<false>(a, dtype, (cudaStream_t)stream);
}

size_t la_group_norm_bwd_workspace_bytes(int B, int H, int L, int d)
{
    if (!sizes_ok(B, H, L, d) || d > GN_MAX_D) return 0;
    const int sms = device_sms();
    return sizeof(float) * 2 * (size_t)blocks_of_head(B, H, L, d, sms > 0 ? sms : 152, true) * H * d;
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
    if (d > GN_MAX_D) return LA_ERR_UNSUPPORTED;
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
        a.part = (float *)workspace;
    }
    const int sms = device_sms();
    if (sms <= 0) return LA_ERR_CUDA;
    a.inv_d = 1.f / (float)d;
    a.nb = blocks_of_head(B, H, L, d, sms, true);
    cudaStream_t s = (cudaStream_t)stream;
    const int rc2 = by_type<true>(a, dtype, s);
    if (rc2 != LA_OK || !a.part) return rc2;
    const long long join = ((long long)H * d + 31) / 32;
    if (join > INT_MAX) return LA_ERR_SHAPE;
    return status_of(tcc::launch_dependent(gn_join_kernel, (int)join, GN_THREADS, 0, s, a));
}

}  // extern "C"
