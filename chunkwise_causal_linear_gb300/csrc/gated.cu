// gated.cu -- linear attention with a decay per head, or per token and head: entry points, the
// decoding step, and the path of every type and size (sm_103a).
//
//     S_t = a_t S_{t-1} + k_t v_t^T,      out_t = scale q_t^T S_t,      a_t = exp(g_t).
//
// The gradients are the same sweep with the roles changed, two of them from the last row on (D_t is
// the gradient of S_t, D_t = scale q_t dout_t^T + a_{t+1} D_{t+1}):
//
//     dq_t = scale S_t dout_t,    dk_t = D_t v_t,    dv_t = D_t^T k_t,    dg_t = <D_t, a_t S_{t-1}>.
//
// dg without a state per row: <D_t, a_t S_{t-1}> - <D_{t+1}, a_{t+1} S_t> = R_t - C_t with R_t = q_t . dq_t
// and C_t = k_t . dk_t, each without the row's own pair, which both hold.  It is summed from the end
// of a segment, where <D, S> is formed from the states, so that roundings gather over one segment only, and again
// from every row whose decay is 0, where it is 0.
//
// sweep_kernel runs the recurrence row by row in fp32: a thread holds 16 x 8 elements of the state, in
// pairs of rows for the packed instructions, and a row costs three of them per pair: decay, product
// with x, new pair (1.5 dk dv instructions of fp32 a row and head).  Bound by the latency of a row's steps, 0.5 to 0.63 us,
// short sequences and long ones: with one warp a scheduler, as B8 H16 d128 has, L1024 takes 642 us, of which the fp32
// pipes are busy 30%.  Rows of the operands reach shared memory by cp.async one tile ahead.  Few heads are cut into
// segments whose sums are formed first.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "gated.cuh"

namespace la {

namespace {

constexpr int SWEEP_ROWS = 16;   // rows of a tile
constexpr int SWEEP_COLS = 8;    // state columns of a thread
constexpr int SWEEP_WARPS = 4;

struct Sweep {
    const void *x, *y, *z, *w;  // S = a S + y z^T, out = x^T S; w: rows that the strict products meet
    View vx, vy, vz, vw, vo, vg;
    int sx, sy, sz, sw;  // heads of the operand per head of the state are H / s..: head h reads h / s
    const float *g;
    void *out;
    float *dot;  // [tiles * warps][heads][L]
    int out_f32;
    int B, H, L, dx, dz;
    float zscale, oscale;
    int reverse, totals;
    int seg_rows, nseg, tiles;
    const int *lengths, *slots;
    int n_slots;
    const float *init;  // state before the first row: [B or slots][H] (by_seg: [segment][B H])
    float *fin;         // state behind the last one, alike
    float *decay;       // totals: [segment][B H], the decay over the segment
    int by_seg;
    int rs, cs;  // element (row, column) of a stored state
    int vec;     // bit 0..2: x, y, z rows can be read 16 bytes at a time
    int *err;
};

__device__ __forceinline__ void copy16(float *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(float *dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// n rows of `len` channels into dst (row stride ld floats), row i of the tile at src + row(i)
template <typename Row>
__device__ __forceinline__ void stage(float *dst, int ld, const float *src, Row row, int n, int len, bool vec, float)
{
    if (vec) {
        const int c4 = len >> 2;
        for (int e = threadIdx.x; e < n * c4; e += blockDim.x) {
            const int i = e / c4, c = 4 * (e % c4);
            copy16(dst + i * ld + c, src + row(i) + c);
        }
    } else {
        for (int c = threadIdx.x; c < len; c += blockDim.x)
#pragma unroll 4
            for (int i = 0; i < n; ++i) copy4(dst + i * ld + c, src + row(i) + c);
    }
}
template <typename Row>
__device__ __forceinline__ void stage(float *dst, int ld, const __nv_bfloat16 *src, Row row, int n, int len, bool vec,
                                      float)
{
    if (vec) {
        const int c8 = len >> 3;
        for (int e = threadIdx.x; e < n * c8; e += blockDim.x) {
            const int i = e / c8, c = 8 * (e % c8);
            const uint4 t = *(const uint4 *)(src + row(i) + c);
            const uint32_t w[4] = {t.x, t.y, t.z, t.w};
            float4 *o = (float4 *)(dst + i * ld + c);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                o[k] = make_float4(__uint_as_float(w[2 * k] << 16), __uint_as_float(w[2 * k] & 0xFFFF0000u),
                                   __uint_as_float(w[2 * k + 1] << 16), __uint_as_float(w[2 * k + 1] & 0xFFFF0000u));
        }
    } else {
        // a channel of every row of the tile at once: the loads wait together, and no element costs a division
        for (int c = threadIdx.x; c < len; c += blockDim.x) {
            __nv_bfloat16 v[SWEEP_ROWS];
#pragma unroll
            for (int i = 0; i < SWEEP_ROWS; ++i)
                if (i < n) v[i] = src[row(i) + c];
#pragma unroll
            for (int i = 0; i < SWEEP_ROWS; ++i)
                if (i < n) dst[i * ld + c] = __bfloat162float(v[i]);
        }
    }
}

// RL lanes of a warp share a group of 8 columns, 16 rows each: up to 16 RL rows.
template <typename T, int RL, bool DOT>
__global__ void __launch_bounds__(32 * SWEEP_WARPS, 2) sweep_kernel(const Sweep a)
{
    constexpr int G = 32 / RL, CW = G * SWEEP_COLS, DX = 16 * RL, TR = SWEEP_ROWS;
    const int warps = blockDim.x >> 5, ZT = warps * CW, LD = 2 * DX + ZT;
    extern __shared__ __align__(16) float sm[];  // [2][TR][LD]: y, x, z; then the decays [2][TR][2]
    float *const gates = sm + 2 * TR * LD;
    const int tile = blockIdx.x % a.tiles, bs = blockIdx.x / a.tiles;
    const int seg = bs % a.nseg, bh = bs / a.nseg, b = bh / a.H, h = bh % a.H;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane % RL, grp = lane / RL;
    const int n_all = gated_rows(a.lengths, b, a.L);
    const int t0 = seg * a.seg_rows, t1 = min(t0 + a.seg_rows, a.L), te = max(t0, min(t1, n_all)), n = te - t0;
    const int col0 = tile * ZT + warp * CW;
    const T *px = (const T *)a.x, *py = (const T *)a.y, *pz = (const T *)a.z;
    const long long bx = b * a.vx.b + (h / a.sx) * a.vx.h, by = b * a.vy.b + (h / a.sy) * a.vy.h,
                    bz = b * a.vz.b + (h / a.sz) * a.vz.h + tile * ZT, bg = b * a.vg.b + h * a.vg.h;
    const int zn = min(ZT, a.dz - tile * ZT);
    const int slot = gated_slot(a.slots, b, a.n_slots, threadIdx.x == 0 ? a.err : nullptr);
    const long long at = (a.by_seg ? (long long)seg * a.B * a.H + bh : (long long)slot * a.H + h) * a.dx * a.dz;

    for (int i = threadIdx.x; i < 2 * TR * LD; i += blockDim.x) sm[i] = 0.f;
    // thread's columns: 4 (grp + G n) + e; rows: 4 (r + RL m) + 0..3
    Ch<2> S[8][SWEEP_COLS];
    const bool has_init = a.init && !a.totals && (a.by_seg || slot >= 0);
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
        for (int c = 0; c < SWEEP_COLS; ++c) {
            const int row = 4 * (r + RL * (p >> 1)) + 2 * (p & 1), col = col0 + 4 * (grp + G * (c >> 2)) + (c & 3);
            S[p][c] = all<2>(0.f);
            if (has_init && col < a.dz) {
                if (row < a.dx) S[p][c].v[0] = a.init[at + (long long)row * a.rs + (long long)col * a.cs];
                if (row + 1 < a.dx) S[p][c].v[1] = a.init[at + (long long)(row + 1) * a.rs + (long long)col * a.cs];
            }
        }
    __syncthreads();

    auto time_of = [&](int p) { return a.reverse ? te - 1 - p : t0 + p; };
    auto fill = [&](int p0, int buf) {
        const int m = min(TR, n - p0);
        float *d = sm + buf * TR * LD;
        stage(d, LD, py, [&](int i) { return by + (long long)time_of(p0 + i) * a.vy.l; }, m, a.dx, a.vec & 2, 0.f);
        if (!a.totals)
            stage(d + DX, LD, px, [&](int i) { return bx + (long long)time_of(p0 + i) * a.vx.l; }, m, a.dx, a.vec & 1, 0.f);
        stage(d + 2 * DX, LD, pz, [&](int i) { return bz + (long long)time_of(p0 + i) * a.vz.l; }, m, zn, a.vec & 4, 0.f);
        if (threadIdx.x < TR && (int)threadIdx.x < m) {
            // in reverse a row's state comes from the row behind it, by that row's decay
            const int p = p0 + threadIdx.x, t = time_of(p) + (a.reverse ? 1 : 0);
            const float g = a.reverse && p == 0 ? 0.f : a.g[bg + (long long)t * a.vg.l];
            gates[(buf * TR + threadIdx.x) * 2] = expf(g);
            gates[(buf * TR + threadIdx.x) * 2 + 1] = expm1f(g);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // the decay of the state, not by a product where a is next to 1: its rounding would be that of a
    // taken to the power of the rows
    auto decay = [&](float av, float em) {
        if (av > 0.5f) {
#pragma unroll
            for (int p = 0; p < 8; ++p)
#pragma unroll
                for (int c = 0; c < SWEEP_COLS; ++c) S[p][c] = fma(S[p][c], all<2>(em), S[p][c]);
        } else if (av > 0.f) {
#pragma unroll
            for (int p = 0; p < 8; ++p)
#pragma unroll
                for (int c = 0; c < SWEEP_COLS; ++c) S[p][c] = mul(S[p][c], all<2>(av));
        } else if (av == 0.f) {  // forgets infinities and NaN too
#pragma unroll
            for (int p = 0; p < 8; ++p)
#pragma unroll
                for (int c = 0; c < SWEEP_COLS; ++c) S[p][c] = all<2>(0.f);
        } else {  // NaN
#pragma unroll
            for (int p = 0; p < 8; ++p)
#pragma unroll
                for (int c = 0; c < SWEEP_COLS; ++c) S[p][c] = all<2>(av);
        }
    };

    if (n > 0) fill(0, 0);
    for (int p0 = 0; p0 < n; p0 += TR) {
        const int buf = (p0 / TR) & 1;
        if (p0 + TR < n) {
            fill(p0 + TR, buf ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const int m = min(TR, n - p0);
#pragma unroll 1
        for (int i = 0; i < m; ++i) {
            const float *d = sm + (buf * TR + i) * LD;
            const float2 gt = *(const float2 *)(gates + (buf * TR + i) * 2);
            if (gt.x != 1.f) decay(gt.x, gt.y);
            Ch<2> o2[SWEEP_COLS];
            Ch<2> xy = all<2>(0.f);
            const float4 z0 = *(const float4 *)(d + 2 * DX + warp * CW + 4 * grp),
                         z1 = *(const float4 *)(d + 2 * DX + warp * CW + 4 * (grp + G));
            float zv[SWEEP_COLS] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
            for (int c = 0; c < SWEEP_COLS; ++c) {
                zv[c] *= a.zscale;
                o2[c] = all<2>(0.f);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 y4 = *(const float4 *)(d + 4 * (r + RL * q));
                const Ch<2> ya{{y4.x, y4.y}}, yb{{y4.z, y4.w}};
                if (!a.totals) {
                    const float4 x4 = *(const float4 *)(d + DX + 4 * (r + RL * q));
                    const Ch<2> xa{{x4.x, x4.y}}, xb{{x4.z, x4.w}};
                    xy = fma(xa, ya, fma(xb, yb, xy));
#pragma unroll
                    for (int c = 0; c < SWEEP_COLS; ++c) o2[c] = fma(xa, S[2 * q][c], fma(xb, S[2 * q + 1][c], o2[c]));
                }
#pragma unroll
                for (int c = 0; c < SWEEP_COLS; ++c) {
                    S[2 * q][c] = fma(ya, all<2>(zv[c]), S[2 * q][c]);
                    S[2 * q + 1][c] = fma(yb, all<2>(zv[c]), S[2 * q + 1][c]);
                }
            }
            if (a.totals) continue;
            // sums over the RL lanes of the group, halving the columns that a lane goes on with
            float o[SWEEP_COLS], own = xy.v[0] + xy.v[1];
#pragma unroll
            for (int c = 0; c < SWEEP_COLS; ++c) o[c] = o2[c].v[0] + o2[c].v[1];
            int base = 0;
#pragma unroll
            for (int s = 1, cnt = SWEEP_COLS; s < RL; s <<= 1) {
                own += __shfl_xor_sync(0xffffffffu, own, s);
                if (cnt > 1) {
                    const bool up = r & s;
                    cnt >>= 1;
#pragma unroll
                    for (int c = 0; c < SWEEP_COLS / 2; ++c)
                        if (c < cnt) {
                            const float send = up ? o[c] : o[c + cnt], keep = up ? o[c + cnt] : o[c];
                            o[c] = keep + __shfl_xor_sync(0xffffffffu, send, s);
                        }
                    base += up ? cnt : 0;
                } else {
                    o[0] += __shfl_xor_sync(0xffffffffu, o[0], s);
                }
            }
            constexpr int LEFT = RL >= 8 ? 1 : SWEEP_COLS / RL;  // columns left to a lane
            const bool mine = RL <= 8 || r < 8;
            const int t = time_of(p0 + i);
            float dot = 0.f;
            if (mine)
#pragma unroll
                for (int c = 0; c < LEFT; ++c) {
                    const int ci = base + c, wc = 4 * (grp + G * (ci >> 2)) + (ci & 3), col = col0 + wc;
                    if (col < a.dz) {
                        const float strict = a.oscale * o[c];
                        if (a.out) {
                            const float val = fmaf(a.oscale * own, a.zscale * d[2 * DX + warp * CW + wc], strict);
                            const long long oi = row_of(a.vo, b, h, t) + col;
                            if (a.out_f32) ((float *)a.out)[oi] = val;
                            else ((T *)a.out)[oi] = from_f32<T>(val);
                        }
                        if (DOT) dot = fmaf(strict, to_f32(((const T *)a.w)[row_of(a.vw, b, h / a.sw, t) + col]), dot);
                    }
                }
            if (DOT) {
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
                if (lane == 0) a.dot[((long long)(tile * warps + warp) * a.B * a.H + bh) * a.L + t] = dot;
            }
        }
        __syncthreads();
    }
    if (a.reverse && n > 0) {  // over the first row
        const float g = a.g[bg + (long long)t0 * a.vg.l];
        decay(expf(g), expm1f(g));
    }
    if (a.fin && (a.by_seg || slot >= 0))
#pragma unroll
        for (int p = 0; p < 8; ++p)
#pragma unroll
            for (int c = 0; c < SWEEP_COLS; ++c) {
                const int row = 4 * (r + RL * (p >> 1)) + 2 * (p & 1), col = col0 + 4 * (grp + G * (c >> 2)) + (c & 3);
                if (col < a.dz) {
                    if (row < a.dx) a.fin[at + (long long)row * a.rs + (long long)col * a.cs] = S[p][c].v[0];
                    if (row + 1 < a.dx) a.fin[at + (long long)(row + 1) * a.rs + (long long)col * a.cs] = S[p][c].v[1];
                }
            }
    if (a.decay && tile == 0 && warp == 0) {
        double s = 0;
        for (int t = t0 + lane; t < te; t += 32) s += (double)a.g[bg + (long long)t * a.vg.l];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) a.decay[(long long)seg * a.B * a.H + bh] = (float)exp(s);
    }
    if (!a.totals && a.out)  // rows behind the sequence's end
        for (int t = te; t < t1; ++t)
            for (int c = threadIdx.x; c < zn; c += blockDim.x) {
                const long long oi = row_of(a.vo, b, h, t) + tile * ZT + c;
                if (a.out_f32) ((float *)a.out)[oi] = 0.f;
                else ((T *)a.out)[oi] = from_f32<T>(0.f);
            }
}

int lanes_of(int dx) { return dx <= 32 ? 2 : dx <= 64 ? 4 : dx <= 128 ? 8 : 16; }
int warps_of(int dx, int dz)
{
    const int cw = 32 / lanes_of(dx) * SWEEP_COLS;
    return std::min(SWEEP_WARPS, (dz + cw - 1) / cw);
}
int tiles_of(int dx, int dz)
{
    const int zt = warps_of(dx, dz) * (32 / lanes_of(dx) * SWEEP_COLS);
    return (dz + zt - 1) / zt;
}

template <typename T, int RL, bool DOT> int launch_sweep_rl(Sweep &s, cudaStream_t stream)
{
    const int warps = warps_of(s.dx, s.dz), zt = warps * (32 / RL) * SWEEP_COLS;
    const size_t smem = sizeof(float) * 2 * SWEEP_ROWS * (2 * 16 * RL + zt + 2);
    s.tiles = tiles_of(s.dx, s.dz);
    const double grid = (double)s.tiles * s.nseg * s.B * s.H;
    if (grid > INT_MAX) return LA_ERR_SHAPE;
    if (smem > 48 * 1024) {
        static std::atomic<uint64_t> done{0};  // devices whose limit is set
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return LA_ERR_CUDA;
        if (dev >= 64 || !(done.load() >> dev & 1)) {
            const size_t most = sizeof(float) * 2 * SWEEP_ROWS * (2 * 16 * RL + SWEEP_WARPS * (32 / RL) * SWEEP_COLS + 2);
            const int rc = status_of(cudaFuncSetAttribute(sweep_kernel<T, RL, DOT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most));
            if (rc != LA_OK) return rc;
            if (dev < 64) done |= 1ull << dev;
        }
    }
    return launch(sweep_kernel<T, RL, DOT>, dim3((unsigned)grid), 32 * warps, smem, stream, s);
}
template <typename T, bool DOT> int launch_sweep_t(Sweep &s, cudaStream_t stream)
{
    switch (lanes_of(s.dx)) {
    case 2: return launch_sweep_rl<T, 2, DOT>(s, stream);
    case 4: return launch_sweep_rl<T, 4, DOT>(s, stream);
    case 8: return launch_sweep_rl<T, 8, DOT>(s, stream);
    default: return launch_sweep_rl<T, 16, DOT>(s, stream);
    }
}
int launch_sweep(Sweep s, int dtype, int HX, int HY, int HZ, cudaStream_t stream)
{
    const size_t es = dtype_size(dtype);
    const int per = (int)(16 / es);  // elements of 16 bytes
    const int zt = warps_of(s.dx, s.dz) * (32 / lanes_of(s.dx)) * SWEEP_COLS;
    s.vec = 0;
    if (s.x && s.dx % per == 0 && rows_aligned(s.x, s.vx, s.B, HX, s.L, es, 16)) s.vec |= 1;
    if (s.dx % per == 0 && rows_aligned(s.y, s.vy, s.B, HY, s.L, es, 16)) s.vec |= 2;
    if (s.dz % per == 0 && zt % per == 0 && rows_aligned(s.z, s.vz, s.B, HZ, s.L, es, 16)) s.vec |= 4;
    if (dtype == LA_F32)
        return s.dot ? launch_sweep_t<float, true>(s, stream) : launch_sweep_t<float, false>(s, stream);
    return s.dot ? launch_sweep_t<__nv_bfloat16, true>(s, stream) : launch_sweep_t<__nv_bfloat16, false>(s, stream);
}

// ---- between the sweeps ------------------------------------------------------------------------
struct ScanArgs {
    float *T;
    const float *A, *first;
    float *last, *last_ws;
    const int *slots;
    int nseg, BH, H, n, n_slots, reverse;
    int *err;
};

// A thread an element, or four; the segments' sums eight at a time, so that their loads are on their way together.
template <int V> __global__ void __launch_bounds__(128) scan_kernel(const ScanArgs a)
{
    constexpr int AT_ONCE = 8;
    using F = Ch<V>;
    const int bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
    const int i = (blockIdx.x * 128 + threadIdx.x) * V;
    if (i >= a.n) return;
    const int slot = gated_slot(a.slots, b, a.n_slots, threadIdx.x == 0 ? a.err : nullptr);
    const long long at = ((long long)slot * a.H + h) * a.n + i;
    auto load = [](const float *p) {
        F f;
        if constexpr (V == 4) {
            const float4 t = *(const float4 *)p;
            f = {{t.x, t.y, t.z, t.w}};
        } else {
            f = {{*p}};
        }
        return f;
    };
    auto store = [](float *p, const F &f) {
        if constexpr (V == 4) *(float4 *)p = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
        else *p = f.v[0];
    };
    F s;
#pragma unroll
    for (int u = 0; u < V; ++u) s.v[u] = 0.f;
    if (a.first && slot >= 0) s = load(a.first + at);
    for (int j0 = 0; j0 < a.nseg; j0 += AT_ONCE) {
        F t[AT_ONCE];
        float w[AT_ONCE];
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
            if (j0 + j < a.nseg) {
                const long long seg = (a.reverse ? a.nseg - 1 - j0 - j : j0 + j) * (long long)a.BH + bh;
                t[j] = load(a.T + seg * a.n + i);
                w[j] = a.A[seg];
            }
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
            if (j0 + j < a.nseg) {
                const long long seg = (a.reverse ? a.nseg - 1 - j0 - j : j0 + j) * (long long)a.BH + bh;
                store(a.T + seg * a.n + i, s);
#pragma unroll
                for (int u = 0; u < V; ++u) s.v[u] = w[j] == 0.f ? t[j].v[u] : fmaf(w[j], s.v[u], t[j].v[u]);
            }
    }
    if (a.last && slot >= 0) store(a.last + at, s);
    if (a.last_ws) store(a.last_ws + (long long)bh * a.n + i, s);
}

struct ShareArgs {
    const float *x;
    void *out;
    View vo;
    int B, H, Hk, L, n;
};
// V channels of a row a thread; a block takes neighbouring rows of a sequence's key head.
template <typename T, int V> __global__ void __launch_bounds__(256) share_kernel(const ShareArgs a)
{
    const int group = a.H / a.Hk, per_row = a.n / V, rows = 256 / per_row > 0 ? 256 / per_row : 1;
    const int hk = blockIdx.y % a.Hk, b = blockIdx.y / a.Hk;
    const long long head = (long long)a.L * a.n;
    const float *const x = a.x + ((long long)b * a.H + (long long)hk * group) * head;
    for (int e = threadIdx.x; e < rows * per_row; e += 256) {
        const int t = blockIdx.x * rows + e / per_row, c = V * (e % per_row);
        if (t >= a.L) break;
        const float *const p = x + (long long)t * a.n + c;
        float s[V];
#pragma unroll
        for (int u = 0; u < V; ++u) s[u] = 0.f;
#pragma unroll 4
        for (int j = 0; j < group; ++j) {
            if constexpr (V == 4) {
                const float4 f = *(const float4 *)(p + j * head);
                s[0] += f.x; s[1] += f.y; s[2] += f.z; s[3] += f.w;
            } else {
                s[0] += p[j * head];
            }
        }
        T *const o = (T *)a.out + row_of(a.vo, b, hk, t) + c;
        if constexpr (V == 4 && sizeof(T) == 2) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(s[0], s[1]), hi = __floats2bfloat162_rn(s[2], s[3]);
            *(uint2 *)o = make_uint2(*(const uint32_t *)&lo, *(const uint32_t *)&hi);
        } else if constexpr (V == 4) {
            *(float4 *)o = make_float4(s[0], s[1], s[2], s[3]);
        } else {
            *o = from_f32<T>(s[0]);
        }
    }
}

struct ProductArgs {
    const float *D, *S;
    float *y;
    int n;
};
// Products summed by eights in fp32, those sums in 64 bits.
__global__ void __launch_bounds__(256) product_kernel(const ProductArgs a)
{
    __shared__ double part[8];
    const float *const D = a.D + (long long)blockIdx.x * a.n, *const S = a.S + (long long)blockIdx.x * a.n;
    double s = 0;
    for (int i0 = threadIdx.x; i0 < a.n; i0 += 256 * 8) {
        float d[8], v[8], f = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool in = i0 + 256 * u < a.n;
            d[u] = in ? D[i0 + 256 * u] : 0.f;
            v[u] = in ? S[i0 + 256 * u] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) f = fmaf(d[u], v[u], f);
        s += (double)f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i) s += part[i];
        a.y[blockIdx.x] = (float)s;
    }
}

struct LogDecayArgs {
    const float *r, *c, *g;
    float *y;  // [seg][heads]: <D, S> at the segments' ends; with `sums`, out: the segments' sums
    View vg;
    float *dg;
    const int *lengths;
    int sums;
    int nr, nc, B, H, L, seg_rows, nseg, initial;
};
// A block a segment, 1024 rows at a time from its end, four neighbouring ones a thread; a row's parts are summed in
// fp32, the rows in 64 bits, few operations of which a row leaves (the SM has two such lanes: a scan of every
// row took 45 us where this takes 13, B2 H12 L16384). The sums start again at every row whose decay is 0: its gradient is
// 0, every pair across it is, and what is behind it, infinities and NaN too, is not the rows' before it.
constexpr int LD_THREADS = 256, LD_ROWS = 4 * LD_THREADS;
__global__ void __launch_bounds__(LD_THREADS) log_decay_kernel(const LogDecayArgs a)
{
    __shared__ __align__(16) float diff[LD_ROWS];
    __shared__ __align__(4) uint8_t cut[LD_ROWS];
    __shared__ double sums[LD_THREADS / 32];
    __shared__ bool starts[LD_THREADS / 32];  // a reset among the warp's rows
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, BH = a.B * a.H;
    const int seg = blockIdx.x / BH, bh = blockIdx.x % BH, b = bh / a.H, h = bh % a.H;
    const int t0 = seg * a.seg_rows, t1 = min(t0 + a.seg_rows, a.L), te = max(t0, min(t1, gated_rows(a.lengths, b, a.L)));
    const long long at = (long long)bh * a.L, step = (long long)BH * a.L;
    if (a.dg)
        for (int t = te + (int)threadIdx.x; t < t1; t += LD_THREADS) a.dg[at + t] = 0.f;
    double all = 0;
    double carry = a.y[(long long)seg * BH + bh];
    for (int e = te; e > t0; e -= LD_ROWS) {  // place k is row e - 1 - k
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = threadIdx.x + LD_THREADS * u, t = e - 1 - k;
            float r = 0.f, c = 0.f;
            bool none = false;
            if (t >= t0) {
                none = a.g[row_of(a.vg, b, h, t)] < GATED_CUT;
#pragma unroll 8
                for (int i = 0; i < a.nr; ++i) r += a.r[i * step + at + t];
#pragma unroll 8
                for (int i = 0; i < a.nc; ++i) c += a.c[i * step + at + t];
            }
            diff[k] = none ? 0.f : r - c;
            cut[k] = none;
        }
        __syncthreads();
        const float4 f = *(const float4 *)(diff + 4 * threadIdx.x);
        const uint32_t at_cut = *(const uint32_t *)(cut + 4 * threadIdx.x);  // a byte a row
        double s[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int u = 1; u < 4; ++u)
            if (!(at_cut >> (8 * u) & 1)) s[u] += s[u - 1];
        // over the lanes behind the last one with a reset
        const uint32_t m = __ballot_sync(0xffffffffu, at_cut != 0), upto = m & (0xffffffffu >> (31 - lane));
        const int from = upto ? 31 - __clz(upto) : 0;
        double run = s[3];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double u = __shfl_up_sync(0xffffffffu, run, o);
            if (lane - o >= from) run += u;
        }
        if (lane == 31) {
            sums[warp] = run;
            starts[warp] = m != 0;
        }
        __syncthreads();
        double before = carry;
        for (int i = 0; i < LD_THREADS / 32; ++i) {
            if (i == warp) before = carry;
            carry = starts[i] ? sums[i] : carry + sums[i];
        }
        const double left = __shfl_up_sync(0xffffffffu, run, 1);  // of the lanes before this one
        const bool fresh = m & ((1u << lane) - 1u);
        before = lane == 0 ? before : fresh ? left : before + left;
        float4 x;
#pragma unroll
        for (int u = 0; u < 4; ++u)  // with no reset up to this row, what is before the thread's too
            (&x.x)[u] = (float)(at_cut & (0xffffffffu >> (24 - 8 * u)) ? s[u] : before + s[u]);
        *(float4 *)(diff + 4 * threadIdx.x) = x;
        __syncthreads();
        float four = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = threadIdx.x + LD_THREADS * u, t = e - 1 - k;
            // a first row with nothing before it has no gradient either
            const float x = t < t0 || cut[k] || (t == 0 && !a.initial) ? 0.f : diff[k];
            if (a.dg && t >= t0) a.dg[at + t] = x;
            four += x;
        }
        all += (double)four;
        __syncthreads();
    }
    if (!a.sums) return;
    // the segment's sum for the head's; fours in fp32 and the whole rounded once, as its terms are
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    __syncthreads();
    if (lane == 0) sums[warp] = all;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < LD_THREADS / 32; ++i) all += sums[i];
        a.y[(long long)seg * BH + bh] = (float)all;
    }
}

struct HeadSumArgs {
    const float *sums;  // [seg][B][H]
    float *out;
    int B, H, nseg;
};
// Over the segments and sequences of one head, in a fixed order.
__global__ void __launch_bounds__(256) head_sum_kernel(const HeadSumArgs a)
{
    __shared__ double part[8];
    const int h = blockIdx.x;
    const long long n = (long long)a.nseg * a.B;
    double s = 0;
    for (long long i = threadIdx.x; i < n; i += 256) s += (double)a.sums[i * a.H + h];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i) s += part[i];
        a.out[h] = (float)s;
    }
}

// ---- the decoding step ---------------------------------------------------------------------------
constexpr int STEP_THREADS = 128, STEP_AHEAD = 8;

struct StepArgs {
    const void *q, *k, *v;
    const float *g;
    float *state;
    const int *slots;
    void *out;
    View vq, vk, vv, vg, vo;
    int B, H, group, d, e, n_slots, tiles;
    float scale;
    int *err;
};

// Bound by the state, read and written once.  A block takes COLS columns of a head, and V columns of eight of a
// thread's rows are on their way at once.  With few heads 32 columns, so that they reach every SM (B8 H16 d128
// 6.3 us, 8.4 with 128); with many 128, rows of 512 bytes (B64 H32 d128, 268 MB: 52.9 us, 75% of measured copy
// bandwidth, 60 with 32).
template <typename T, int V, int COLS> __global__ void __launch_bounds__(STEP_THREADS, 6) step_kernel(const StepArgs a)
{
    static_assert(COLS / V <= 32, "each warp covers the columns");
    constexpr int LC = COLS / V, RG = STEP_THREADS / LC;  // lanes along the columns, row groups
    __shared__ float sums[STEP_THREADS / 32][COLS];
    const int tile = blockIdx.x % a.tiles, bh = blockIdx.x / a.tiles, b = bh / a.H, h = bh % a.H, hk = h / a.group;
    const int lc = threadIdx.x % LC, rg = threadIdx.x / LC, col = tile * COLS + V * lc;
    const int slot = gated_slot(a.slots, b, a.n_slots, threadIdx.x == 0 ? a.err : nullptr);
    const bool in = col < a.e;  // V divides e
    float *const S = a.state + ((long long)slot * a.H + h) * a.d * a.e + col;
    const T *const q = (const T *)a.q + row_of(a.vq, b, h, 0), *const k = (const T *)a.k + row_of(a.vk, b, hk, 0);
    const float g = a.g[row_of(a.vg, b, h, 0)], av = expf(g), em = expm1f(g);
    float v[V], o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        v[i] = in ? to_f32(((const T *)a.v)[row_of(a.vv, b, hk, 0) + col + i]) : 0.f;
        o[i] = 0.f;
    }
    for (int r0 = rg; r0 < a.d; r0 += RG * STEP_AHEAD) {
        float s[STEP_AHEAD][V], kk[STEP_AHEAD], qq[STEP_AHEAD];
#pragma unroll
        for (int m = 0; m < STEP_AHEAD; ++m) {
            const int row = r0 + m * RG;
#pragma unroll
            for (int i = 0; i < V; ++i) s[m][i] = 0.f;
            kk[m] = qq[m] = 0.f;
            if (row < a.d) {
                if (in && slot >= 0) {
                    if constexpr (V == 4) {
                        const float4 t = *(const float4 *)(S + (long long)row * a.e);
                        s[m][0] = t.x; s[m][1] = t.y; s[m][2] = t.z; s[m][3] = t.w;
                    } else {
                        s[m][0] = S[(long long)row * a.e];
                    }
                }
                kk[m] = to_f32(k[row]);
                qq[m] = to_f32(q[row]);
            }
        }
#pragma unroll
        for (int m = 0; m < STEP_AHEAD; ++m) {
            const int row = r0 + m * RG;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // as in the sweep: no product with a decay next to 1, and 0 forgets all
                const float old = av > 0.5f ? fmaf(s[m][i], em, s[m][i]) : av == 0.f ? 0.f : av * s[m][i];
                s[m][i] = fmaf(kk[m], v[i], old);
                o[i] = fmaf(qq[m], s[m][i], o[i]);
            }
            if (row < a.d && in && slot >= 0) {
                if constexpr (V == 4) *(float4 *)(S + (long long)row * a.e) = make_float4(s[m][0], s[m][1], s[m][2], s[m][3]);
                else S[(long long)row * a.e] = s[m][0];
            }
        }
    }
    // over the row groups: those of a warp, then the warps
#pragma unroll
    for (int w = LC; w < 32; w <<= 1)
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], w);
    if ((threadIdx.x & 31) < LC)
#pragma unroll
        for (int i = 0; i < V; ++i) sums[threadIdx.x >> 5][V * lc + i] = o[i];
    __syncthreads();
    const int c = threadIdx.x;
    if (c < COLS && tile * COLS + c < a.e) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < STEP_THREADS / 32; ++w) s += sums[w][c];
        ((T *)a.out)[row_of(a.vo, b, h, 0) + tile * COLS + c] = from_f32<T>(a.scale * s);
    }
}

constexpr int SEG_LEAST = 16;
int fwd_segments(int B, int H, int L, int d, int e, int sms)
{
    // eight warps an SM, as many as the state's registers allow, of 16 rows at least; the segments' sums cost two thirds
    // of a sweep, so that two segments would not pay. (A row takes a warp about half a microsecond however few there are.)
    const double warps = (double)B * H * tiles_of(d, e) * warps_of(d, e);
    const int want = (int)std::min(1024.0, std::floor(8.0 * sms / warps)), most = (L + SEG_LEAST - 1) / SEG_LEAST;
    const int n = std::min(want, most);
    return n < 3 ? 1 : n;
}
int rows_of_segments(int L, int n) { return (L + n - 1) / n; }

int bwd_segments(int B, int H, int L, int d, int e, int sms)
{
    const int anchors = (L + GATED_ANCHOR - 1) / GATED_ANCHOR;
    return std::max(anchors, fwd_segments(B, H, L, d, e, sms));
}

Sweep sweep_of(const GatedArgs &p, int seg_rows, int nseg)
{
    Sweep s = {};
    s.B = p.B; s.H = p.H; s.L = p.L;
    s.g = p.g; s.vg = p.vg;
    s.lengths = p.lengths;
    s.zscale = s.oscale = 1.f;
    s.sx = s.sy = s.sz = s.sw = 1;
    s.seg_rows = seg_rows;
    s.nseg = nseg;
    s.err = p.err;
    return s;
}

}  // namespace

// ---- the joins ------------------------------------------------------------------------------------
int gated_scan(const GatedArgs &p, float *T, const float *A, int nseg, int n, const float *first, const int *slots,
               float *last, float *last_ws, bool reverse)
{
    const ScanArgs a{T, A, first, last, last_ws, slots, nseg, p.B * p.H, p.H, n, p.n_slots, reverse, p.err};
    if (n % 4 == 0 && aligned(T, 16) && aligned(first, 16) && aligned(last, 16) && aligned(last_ws, 16))
        return launch(scan_kernel<4>, dim3((unsigned)((n / 4 + 127) / 128), (unsigned)a.BH), 128, 0, p.stream, a);
    return launch(scan_kernel<1>, dim3((unsigned)((n + 127) / 128), (unsigned)a.BH), 128, 0, p.stream, a);
}

int gated_share(const GatedArgs &p, const float *x, void *out, const View &vo, int n)
{
    const ShareArgs a{x, out, vo, p.B, p.H, p.Hk, p.L, n};
    const size_t es = dtype_size(p.dtype);
    const bool wide = n % 4 == 0 && aligned(x, 16) && rows_aligned(out, vo, p.B, p.Hk, p.L, es, 4 * es);
    const int per_row = wide ? n / 4 : n, rows = std::max(1, 256 / per_row);
    const dim3 grid((unsigned)((p.L + rows - 1) / rows), (unsigned)(p.B * p.Hk));
    auto run = [&](auto t) {
        using T = decltype(t);
        return wide ? launch(share_kernel<T, 4>, grid, 256, 0, p.stream, a) : launch(share_kernel<T, 1>, grid, 256, 0, p.stream, a);
    };
    return p.dtype == LA_F32 ? run(0.f) : run(__nv_bfloat16());
}

int gated_products(const GatedArgs &p, const float *D, const float *S, float *y, int nseg, int n)
{
    return launch(product_kernel, dim3((unsigned)(nseg * p.B * p.H)), 256, 0, p.stream, ProductArgs{D, S, y, n});
}

int gated_log_decay(const GatedArgs &p, const float *r, int nr, const float *c, int nc, float *y, int seg_rows, int nseg)
{
    const LogDecayArgs a{r, c, p.g, y, p.vg, p.dg, p.lengths, p.dg_head != nullptr, nr, nc, p.B, p.H, p.L, seg_rows, nseg, p.state0 != nullptr};
    int rc = launch(log_decay_kernel, dim3((unsigned)(p.B * p.H * nseg)), LD_THREADS, 0, p.stream, a);
    if (rc == LA_OK && p.dg_head) rc = launch(head_sum_kernel, dim3((unsigned)p.H), 256, 0, p.stream, HeadSumArgs{y, p.dg_head, p.B, p.H, nseg});
    return rc;
}

// ---- the path of every type and size -------------------------------------------------------------
size_t gated_simt_fwd_ws(int B, int H, int L, int d, int e, int sms)
{
    const int n = fwd_segments(B, H, L, d, e, sms);
    return n == 1 ? 0 : sizeof(float) * (size_t)n * B * H * ((size_t)d * e + 1);
}

int gated_simt_fwd(const GatedArgs &p)
{
    const int want = fwd_segments(p.B, p.H, p.L, p.d, p.e, p.sms), rows = rows_of_segments(p.L, want),
              nseg = (p.L + rows - 1) / rows, n = p.d * p.e;
    const size_t heads = (size_t)p.B * p.H;
    Sweep s = sweep_of(p, rows, nseg);
    s.y = p.k; s.vy = p.vk; s.sy = p.H / p.Hk;
    s.z = p.v; s.vz = p.vv; s.sz = p.H / p.Hk;
    s.dx = p.d; s.dz = p.e;
    s.rs = p.e; s.cs = 1;
    int rc;
    if (nseg > 1) {
        float *T = p.ws, *A = T + (size_t)want * heads * n;
        Sweep t = s;
        t.totals = t.by_seg = 1;
        t.fin = T;
        t.decay = A;
        if ((rc = launch_sweep(t, p.dtype, p.H, p.Hk, p.Hk, p.stream)) != LA_OK) return rc;
        if ((rc = gated_scan(p, T, A, nseg, n, p.state0, p.slots, p.state, nullptr, false)) != LA_OK) return rc;
        s.by_seg = 1;
        s.init = T;
    } else {
        s.slots = p.slots; s.n_slots = p.n_slots;
        s.init = p.state0;
        s.fin = p.state;
    }
    s.x = p.q; s.vx = p.vq;
    s.out = p.out; s.vo = p.vo;
    s.oscale = p.scale;
    return launch_sweep(s, p.dtype, p.H, p.Hk, p.Hk, p.stream);
}

namespace {
// Floats of the backward pass's workspace, part by part.
struct BwdSpace {
    size_t S, A, D, y, r, c, dk, dv, all;
    int nr, nc;
    BwdSpace(int B, int H, int Hk, int L, int d, int e, int nseg)
    {
        const size_t heads = (size_t)B * H, n = (size_t)d * e, rows = heads * L;
        nr = tiles_of(e, d) * warps_of(e, d);
        nc = tiles_of(e, d) * warps_of(e, d);
        size_t at = 0;
        auto take = [&](size_t k) { const size_t o = at; at += (k + 3) & ~(size_t)3; return o; };
        S = take((nseg + 1) * heads * n);
        A = take(nseg * heads);
        D = take(nseg * heads * n);
        y = take(nseg * heads);
        r = take(nr * rows);
        c = take(nc * rows);
        dk = take(H > Hk ? rows * d : 0);
        dv = take(H > Hk ? rows * e : 0);
        all = at;
    }
};
}  // namespace

size_t gated_simt_bwd_ws(int B, int H, int Hk, int L, int d, int e, int sms)
{
    return sizeof(float) * BwdSpace(B, H, Hk, L, d, e, bwd_segments(B, H, L, d, e, sms)).all;
}

int gated_simt_bwd(const GatedArgs &p)
{
    const int want = bwd_segments(p.B, p.H, p.L, p.d, p.e, p.sms), rows = rows_of_segments(p.L, want),
              nseg = (p.L + rows - 1) / rows, n = p.d * p.e, group = p.H / p.Hk;
    const size_t heads = (size_t)p.B * p.H;
    const BwdSpace w(p.B, p.H, p.Hk, p.L, p.d, p.e, want);
    float *const ws = p.ws;
    const bool dg = p.dg || p.dg_head;
    int rc;
    // states at the segments' starts, and behind the last one
    Sweep s = sweep_of(p, rows, nseg);
    s.by_seg = 1;
    s.totals = 1;
    s.y = p.k; s.vy = p.vk; s.sy = group;
    s.z = p.v; s.vz = p.vv; s.sz = group;
    s.dx = p.d; s.dz = p.e; s.rs = p.e; s.cs = 1;
    s.fin = ws + w.S;
    s.decay = ws + w.A;
    if ((rc = launch_sweep(s, p.dtype, p.H, p.Hk, p.Hk, p.stream)) != LA_OK) return rc;
    if ((rc = gated_scan(p, ws + w.S, ws + w.A, nseg, n, p.state0, nullptr, nullptr, ws + w.S + nseg * heads * n, false)) != LA_OK)
        return rc;
    // the states' gradients at the segments' ends, and that of the first state
    s = sweep_of(p, rows, nseg);
    s.by_seg = s.totals = s.reverse = 1;
    s.y = p.q; s.vy = p.vq;
    s.z = p.dout; s.vz = p.vo; s.zscale = p.scale;
    s.dx = p.d; s.dz = p.e; s.rs = p.e; s.cs = 1;
    s.fin = ws + w.D;
    if ((rc = launch_sweep(s, p.dtype, p.H, p.H, p.H, p.stream)) != LA_OK) return rc;
    if ((rc = gated_scan(p, ws + w.D, ws + w.A, nseg, n, p.dstate, nullptr, p.dstate0, nullptr, true)) != LA_OK) return rc;
    // dq = S dout
    s = sweep_of(p, rows, nseg);
    s.by_seg = 1;
    s.x = p.dout; s.vx = p.vo;
    s.y = p.v; s.vy = p.vv; s.sy = group;
    s.z = p.k; s.vz = p.vk; s.sz = group;
    s.dx = p.e; s.dz = p.d; s.rs = 1; s.cs = p.e;
    s.init = ws + w.S;
    s.out = p.dq; s.vo = p.vdq; s.oscale = p.scale;
    if (dg) {
        s.w = p.q; s.vw = p.vq;
        s.dot = ws + w.r;
    }
    if ((rc = launch_sweep(s, p.dtype, p.H, p.Hk, p.Hk, p.stream)) != LA_OK) return rc;
    // dk = D v
    auto per_head = [&](float *x, int c) { return View{(long long)p.H * p.L * c, (long long)p.L * c, c}; };
    s = sweep_of(p, rows, nseg);
    s.by_seg = s.reverse = 1;
    s.x = p.v; s.vx = p.vv; s.sx = group;
    s.y = p.dout; s.vy = p.vo;
    s.z = p.q; s.vz = p.vq; s.zscale = p.scale;
    s.dx = p.e; s.dz = p.d; s.rs = 1; s.cs = p.e;
    s.init = ws + w.D;
    s.out = p.dk; s.vo = p.vdk;
    if (group > 1) {
        s.out = ws + w.dk; s.vo = per_head(ws, p.d); s.out_f32 = 1;
    }
    if (dg) {
        s.w = p.k; s.vw = p.vk; s.sw = group;
        s.dot = ws + w.c;
    }
    if ((rc = launch_sweep(s, p.dtype, p.Hk, p.H, p.H, p.stream)) != LA_OK) return rc;
    // dv = D^T k
    s = sweep_of(p, rows, nseg);
    s.by_seg = s.reverse = 1;
    s.x = p.k; s.vx = p.vk; s.sx = group;
    s.y = p.q; s.vy = p.vq;
    s.z = p.dout; s.vz = p.vo; s.zscale = p.scale;
    s.dx = p.d; s.dz = p.e; s.rs = p.e; s.cs = 1;
    s.init = ws + w.D;
    s.out = p.dv; s.vo = p.vdv;
    if (group > 1) {
        s.out = ws + w.dv; s.vo = per_head(ws, p.e); s.out_f32 = 1;
    }
    if ((rc = launch_sweep(s, p.dtype, p.Hk, p.H, p.H, p.stream)) != LA_OK) return rc;
    if (group > 1) {
        if ((rc = gated_share(p, ws + w.dk, p.dk, p.vdk, p.d)) != LA_OK) return rc;
        if ((rc = gated_share(p, ws + w.dv, p.dv, p.vdv, p.e)) != LA_OK) return rc;
    }
    if (dg) {
        if ((rc = gated_products(p, ws + w.D, ws + w.S + heads * n, ws + w.y, nseg, n)) != LA_OK) return rc;
        if ((rc = gated_log_decay(p, ws + w.r, w.nr, ws + w.c, w.nc, ws + w.y, rows, nseg)) != LA_OK)
            return rc;
    }
    return LA_OK;
}

namespace {

View gate_view(const la_strides *s, int H, int L)
{
    if (s) return View{s->b, s->h, s->l};
    return View{(long long)H * L, L, 1};
}

bool gated_sizes_ok(int B, int H, int Hk, int L, int d, int e)
{
    if (!sizes_ok(B, H, L, d) || !sizes_ok(B, H, L, e) || Hk <= 0 || H % Hk != 0) return false;
    return (long long)B * H <= 65535;  // heads that one launch of the joins takes
}

}  // namespace

}  // namespace la

using namespace la;

extern "C" {

int la_gated_fwd(const void *q, const void *k, const void *v, const float *log_decay, const float *state0, float *state,
                 const int *slots, const int *lengths, void *out, int B, int H, int Hk, int L, int dk, int dv, int n_slots,
                 const la_strides *q_strides, const la_strides *k_strides, const la_strides *v_strides,
                 const la_strides *g_strides, const la_strides *out_strides, float scale, int dtype, void *workspace,
                 size_t workspace_bytes, void *stream, int path)
{
    if (!q || !k || !v || !log_decay || !out) return LA_ERR_NULL;
    if (!gated_sizes_ok(B, H, Hk, L, dk, dv) || (slots && n_slots <= 0)) return LA_ERR_SHAPE;
    if (!dtype_ok(dtype) || dk > 256 || dv > 256 || path < LA_PATH_AUTO || path > LA_PATH_TC) return LA_ERR_UNSUPPORTED;
    GatedArgs p = {};
    p.q = q; p.k = k; p.v = v; p.g = log_decay;
    p.state0 = state0; p.state = state; p.slots = slots; p.lengths = lengths;
    p.out = out;
    p.vq = make_view(q_strides, H, L, dk);
    p.vk = make_view(k_strides, Hk, L, dk);
    p.vv = make_view(v_strides, Hk, L, dv);
    p.vg = gate_view(g_strides, H, L);
    p.vo = make_view(out_strides, H, L, dv);
    if (!input_view_ok(p.vq, B, H, L) || !input_view_ok(p.vk, B, Hk, L) || !input_view_ok(p.vv, B, Hk, L) ||
        !input_view_ok(p.vg, B, H, L) || !output_view_ok(p.vo, B, H, L, dv) || !isfinite(scale))
        return LA_ERR_ARG;
    const size_t es = dtype_size(dtype);
    if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(out, es) || !aligned(log_decay, 4) ||
        !aligned(state0, 4) || !aligned(state, 4) || !aligned(slots, 4) || !aligned(lengths, 4) || !aligned(workspace, 16))
        return LA_ERR_ARG;
    p.B = B; p.H = H; p.Hk = Hk; p.L = L; p.d = dk; p.e = dv; p.n_slots = n_slots;
    p.scale = scale;
    p.dtype = dtype;
    p.ws = (float *)workspace;
    p.stream = (cudaStream_t)stream;
    const bool tc = path != LA_PATH_SIMT && gated_tc_fwd_ok(p);
    if (path == LA_PATH_TC && !tc) return LA_ERR_UNSUPPORTED;
    if ((p.sms = device_sms()) <= 0 || !(p.err = err_ptr())) return LA_ERR_CUDA;
    const size_t need = tc ? gated_tc_fwd_ws(B, H, L, dk, dv, p.sms) : gated_simt_fwd_ws(B, H, L, dk, dv, p.sms);
    if (need && (!workspace || workspace_bytes < need)) return LA_ERR_WORKSPACE;
    return tc ? gated_tc_fwd(p) : gated_simt_fwd(p);
}

size_t la_gated_workspace_bytes(int B, int H, int L, int dk, int dv, int dtype)
{
    if (!gated_sizes_ok(B, H, H, L, dk, dv) || dk > 256 || dv > 256 || !dtype_ok(dtype)) return 0;
    const int n = device_sms(), sms = n > 0 ? n : 152;
    const size_t simt = gated_simt_fwd_ws(B, H, L, dk, dv, sms);
    return dtype == LA_BF16 ? std::max(simt, gated_tc_fwd_ws(B, H, L, dk, dv, sms)) : simt;
}

int la_gated_bwd(const void *q, const void *k, const void *v, const float *log_decay, const float *state0,
                 const int *lengths, const void *dout, const float *dstate, void *grad_q, void *grad_k, void *grad_v, float *dlog_decay,
                 float *dlog_decay_head, float *dstate0, int B, int H, int Hk, int L, int dk, int dv,
                 const la_strides *q_strides, const la_strides *k_strides, const la_strides *v_strides,
                 const la_strides *g_strides, const la_strides *dout_strides, const la_strides *dq_strides,
                 const la_strides *dk_strides, const la_strides *dv_strides, float scale, int dtype, void *workspace,
                 size_t workspace_bytes, void *stream, int path)
{
    if (!q || !k || !v || !log_decay || !dout || !grad_q || !grad_k || !grad_v) return LA_ERR_NULL;
    if (!gated_sizes_ok(B, H, Hk, L, dk, dv)) return LA_ERR_SHAPE;
    if (!dtype_ok(dtype) || dk > 256 || dv > 256 || path < LA_PATH_AUTO || path > LA_PATH_TC) return LA_ERR_UNSUPPORTED;
    GatedArgs p = {};
    p.q = q; p.k = k; p.v = v; p.g = log_decay; p.dout = dout;
    p.state0 = state0; p.dstate = dstate; p.lengths = lengths;
    p.dq = grad_q; p.dk = grad_k; p.dv = grad_v; p.dg = dlog_decay; p.dg_head = dlog_decay_head; p.dstate0 = dstate0;
    p.vq = make_view(q_strides, H, L, dk);
    p.vk = make_view(k_strides, Hk, L, dk);
    p.vv = make_view(v_strides, Hk, L, dv);
    p.vg = gate_view(g_strides, H, L);
    p.vo = make_view(dout_strides, H, L, dv);
    p.vdq = make_view(dq_strides, H, L, dk);
    p.vdk = make_view(dk_strides, Hk, L, dk);
    p.vdv = make_view(dv_strides, Hk, L, dv);
    if (!input_view_ok(p.vq, B, H, L) || !input_view_ok(p.vk, B, Hk, L) || !input_view_ok(p.vv, B, Hk, L) ||
        !input_view_ok(p.vg, B, H, L) || !input_view_ok(p.vo, B, H, L) || !output_view_ok(p.vdq, B, H, L, dk) ||
        !output_view_ok(p.vdk, B, Hk, L, dk) || !output_view_ok(p.vdv, B, Hk, L, dv) || !isfinite(scale))
        return LA_ERR_ARG;
    const size_t es = dtype_size(dtype);
    if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(dout, es) || !aligned(grad_q, es) ||
        !aligned(grad_k, es) || !aligned(grad_v, es) || !aligned(log_decay, 4) || !aligned(state0, 4) || !aligned(dstate, 4) ||
        !aligned(dlog_decay, 4) || !aligned(dlog_decay_head, 4) || !aligned(dstate0, 4) || !aligned(lengths, 4) || !aligned(workspace, 16))
        return LA_ERR_ARG;
    p.B = B; p.H = H; p.Hk = Hk; p.L = L; p.d = dk; p.e = dv;
    p.scale = scale;
    p.dtype = dtype;
    p.ws = (float *)workspace;
    p.stream = (cudaStream_t)stream;
    const bool tc = path != LA_PATH_SIMT && gated_tc_bwd_ok(p);
    if (path == LA_PATH_TC && !tc) return LA_ERR_UNSUPPORTED;
    if ((p.sms = device_sms()) <= 0 || !(p.err = err_ptr())) return LA_ERR_CUDA;
    const size_t need = tc ? gated_tc_bwd_ws(B, H, Hk, L, dk, dv, p.sms) : gated_simt_bwd_ws(B, H, Hk, L, dk, dv, p.sms);
    if (!workspace || workspace_bytes < need) return LA_ERR_WORKSPACE;
    if ((double)B * H * bwd_segments(B, H, L, dk, dv, p.sms) > INT_MAX / 4) return LA_ERR_SHAPE;  // grids
    return tc ? gated_tc_bwd(p) : gated_simt_bwd(p);
}

size_t la_gated_bwd_workspace_bytes(int B, int H, int Hk, int L, int dk, int dv, int dtype)
{
    if (!gated_sizes_ok(B, H, Hk, L, dk, dv) || dk > 256 || dv > 256 || !dtype_ok(dtype)) return 0;
    const int n = device_sms(), sms = n > 0 ? n : 152;
    const size_t simt = gated_simt_bwd_ws(B, H, Hk, L, dk, dv, sms);
    return dtype == LA_BF16 ? std::max(simt, gated_tc_bwd_ws(B, H, Hk, L, dk, dv, sms)) : simt;
}

int la_gated_step(const void *q, const void *k, const void *v, const float *log_decay, float *state, const int *slots,
                  void *out, int B, int H, int Hk, int dk, int dv, int n_slots, const la_strides *q_strides,
                  const la_strides *k_strides, const la_strides *v_strides, const la_strides *g_strides, float scale,
                  int dtype, void *stream)
{
    if (!q || !k || !v || !log_decay || !state || !out) return LA_ERR_NULL;
    if (!gated_sizes_ok(B, H, Hk, 1, dk, dv) || (slots && n_slots <= 0)) return LA_ERR_SHAPE;
    if (!dtype_ok(dtype) || dk > 256 || dv > 256) return LA_ERR_UNSUPPORTED;
    StepArgs a = {};
    a.q = q; a.k = k; a.v = v; a.g = log_decay;
    a.state = state; a.slots = slots; a.out = out;
    a.vq = make_view(q_strides, H, 1, dk);
    a.vk = make_view(k_strides, Hk, 1, dk);
    a.vv = make_view(v_strides, Hk, 1, dv);
    a.vg = gate_view(g_strides, H, 1);
    a.vo = make_view(nullptr, H, 1, dv);
    if (!input_view_ok(a.vq, B, H, 1) || !input_view_ok(a.vk, B, Hk, 1) || !input_view_ok(a.vv, B, Hk, 1) ||
        !input_view_ok(a.vg, B, H, 1) || !isfinite(scale))
        return LA_ERR_ARG;
    const size_t es = dtype_size(dtype);
    if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(out, es) || !aligned(log_decay, 4) || !aligned(state, 4) ||
        !aligned(slots, 4))
        return LA_ERR_ARG;
    a.B = B; a.H = H; a.group = H / Hk; a.d = dk; a.e = dv; a.n_slots = n_slots;
    a.scale = scale;
    if (!(a.err = err_ptr())) return LA_ERR_CUDA;
    const bool wide = dv % 4 == 0 && aligned(state, 16), many = wide && dv > 64 && (long long)B * H >= 4ll * device_sms();
    const int cols = many ? 128 : 32;
    a.tiles = (dv + cols - 1) / cols;
    const dim3 grid((unsigned)((long long)B * H * a.tiles));
    cudaStream_t s = (cudaStream_t)stream;
    auto run = [&](auto t) {
        using T = decltype(t);
        if (many) return launch(step_kernel<T, 4, 128>, grid, STEP_THREADS, 0, s, a);
        return wide ? launch(step_kernel<T, 4, 32>, grid, STEP_THREADS, 0, s, a) : launch(step_kernel<T, 1, 32>, grid, STEP_THREADS, 0, s, a);
    };
    return dtype == LA_F32 ? run(0.f) : run(__nv_bfloat16());
}

}  // extern "C"
