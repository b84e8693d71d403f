// recurrence.cu -- gated linear recurrence h_t = a_t h_{t-1} + w_t x_t, its gradients and its
// decoding step (sm_103a).
//
// A run of rows acts on the state before it as h -> P h + H (P the product of its gates, H what
// it adds from zero), and two runs in a row join to P = P2 P1, H = P2 H1 + H2.  So a run is
// folded on its own, and its rows are finished once the state before it is known.  Backwards,
// c_t = a_t e_t, e_t = dout_t + c_{t+1}: c -> P c + E with the same P.
//
// The rows of one head's block of 32 V channels go through one cluster of S blocks (S = 1: one
// block).  A step of the cluster covers S tiles of 128 rows, one per block; a tile is 8 warps
// of 16 rows, a lane holds V channels of them in registers.  Per step: fold the 16 rows, put
// (P, H) into shared memory, one block barrier, fold the 8 warps; with S > 1 every block then
// writes its tile's (P, H) into the others' shared memory and one cluster barrier later every
// block knows the state before its tile and after the step.  Every input is read once and every
// output written once; nothing goes through global memory between the blocks, no flag is
// waited for, and the order of the sums depends on the sizes alone.
//
// The kernel is bound by memory (12 bytes and ~40 instructions an fp32 element), so the inputs
// of the next steps are on the way while one is folded: each warp copies its own rows into its
// own ring in shared memory (cp.async, no barrier).
#include <algorithm>

#include "layer.cuh"

namespace la {

namespace {

constexpr int RC = LA_RECURRENCE_CHUNK;
constexpr int REC_W = 8;             // warps of a tile
constexpr int REC_R = RC / REC_W;    // rows of a warp
constexpr int REC_THREADS = 32 * REC_W;
constexpr int REC_STAGES = 3;        // ring: one step in work, two on the way
constexpr int REC_MAX_SPLIT = 8;     // portable cluster size

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
};

// a, w and da/dg from the gate input.  1 - a comes from its own formula where a is close to 1.
// expf is good to 1 ulp and the approximate reciprocal of [1, 2] too, so a and 1 - a are off by
// at most 6 units of 2^-24.
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
        const float e = expf(-fabsf(g)), r = __fdividef(1.f, 1.f + e), s = e * r;
        a = g >= 0.f ? r : s;
        const float c = g >= 0.f ? s : r;
        w = COMP ? c : 1.f;
        slope = a * c;
    }
}

// The state times a gate (or a product of gates), a gate of 0 forgetting infinities and NaN as
// well.
__device__ __forceinline__ float forget(float a, float h) { return a == 0.f ? 0.f : a * h; }
__device__ __forceinline__ float step(float a, float h, float b) { return a == 0.f ? b : fmaf(a, h, b); }

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
template <typename T, int CW, int BYTES>
__device__ __forceinline__ void copy_by(T *slot, const T *src, long long stride, int nrow, int nch, int lane)
{
    constexpr int E = BYTES / sizeof(T), N = CW / E, RP = 32 / N;
    static_assert(32 % N == 0 && REC_R % RP == 0, "whole rows per warp instruction");
    const int r0 = lane / N, c = lane % N * E;
    if (c >= nch) return;
    const T *p = src + r0 * stride + c;
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(slot) + lane * BYTES;
    constexpr int M = REC_R / RP, BATCH = M < 8 ? M : 8;
    for (int j0 = 0; j0 < M; j0 += BATCH) {
        if constexpr (BYTES == 2) {
            T v[BATCH];
#pragma unroll
            for (int j = 0; j < BATCH; ++j, p += RP * stride)
                if (r0 + (j0 + j) * RP < nrow) v[j] = *p;
#pragma unroll
            for (int j = 0; j < BATCH; ++j) slot[lane + 32 * (j0 + j)] = v[j];
        } else {
#pragma unroll
            for (int j = 0; j < BATCH; ++j, p += RP * stride)
                if (r0 + (j0 + j) * RP < nrow) cp_async<BYTES>(dst + 32 * BYTES * (j0 + j), p);
        }
    }
}
template <typename T, int CW>
__device__ __forceinline__ void copy_rows(T *slot, const T *src, long long stride, int nrow, int nch, int gran,
                                          int lane)
{
    if (nrow <= 0) return;
    if (gran == 16) copy_by<T, CW, 16>(slot, src, stride, nrow, nch, lane);
    else if (gran == 4) copy_by<T, CW, 4>(slot, src, stride, nrow, nch, lane);
    else if constexpr (sizeof(T) == 2 && CW == 32) copy_by<T, CW, 2>(slot, src, stride, nrow, nch, lane);
}

// ---- V neighbouring channels ----------------------------------------------------------------
template <int V> __device__ __forceinline__ void get(const float *p, float (&v)[V])
{
    if constexpr (V == 2) {
        const float2 t = *(const float2 *)p;
        v[0] = t.x;
        v[1] = t.y;
    } else {
        v[0] = *p;
    }
}
template <int V> __device__ __forceinline__ void get(const __nv_bfloat16 *p, float (&v)[V])
{
    if constexpr (V == 2) {
        const float2 t = __bfloat1622float2(*(const __nv_bfloat162 *)p);
        v[0] = t.x;
        v[1] = t.y;
    } else {
        v[0] = __bfloat162float(*p);
    }
}
// V = 2 is launched only where pairs are aligned and inside the channels together
template <int V> __device__ __forceinline__ void put(float *p, const float (&v)[V])
{
    if constexpr (V == 2) *(float2 *)p = make_float2(v[0], v[1]);
    else *p = v[0];
}
template <int V> __device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&v)[V])
{
    if constexpr (V == 2) *(__nv_bfloat162 *)p = __floats2bfloat162_rn(v[0], v[1]);
    else *p = __float2bfloat16_rn(v[0]);
}

// ---- between the blocks of a cluster -----------------------------------------------------------
__device__ __forceinline__ void cluster_put(uint32_t addr, int rank, float p, float h)
{
    uint32_t far;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(addr), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(far), "f"(p), "f"(h) : "memory");
}
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The folds of a step: warps of the tile (agg, two buffers), tiles of the cluster (peer, two).
// Two buffers and one barrier a step are enough: a buffer is written again two steps later,
// after a barrier that every reader of it has reached.
template <int CW>
struct RecFolds {
    float2 agg[2][REC_W][CW];
    float2 peer[2][REC_MAX_SPLIT][CW];
};

// The carry through the tiles of a step in order `carry = P carry + H`: returns the carry before
// this block's tile and leaves the one after the step.  tot: this tile's fold.
template <int V, int CW>
__device__ __forceinline__ void across_tiles(RecFolds<CW> &f, int buf, int split, int rank, int warp, int lane,
                                             const float (&P)[V], const float (&H)[V], float (&carry)[V],
                                             float (&mine)[V])
{
    if (split == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            mine[v] = carry[v];
            carry[v] = step(P[v], carry[v], H[v]);
        }
        return;
    }
    if (warp < split) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            cluster_put((uint32_t)__cvta_generic_to_shared(&f.peer[buf][rank][lane * V + v]), warp, P[v], H[v]);
    }
    cluster_barrier();
    for (int r = 0; r < split; ++r) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (r == rank) mine[v] = carry[v];
            const float2 q = f.peer[buf][r][lane * V + v];
            carry[v] = step(q.x, carry[v], q.y);
        }
    }
}

template <typename T, typename G, int V>
__host__ __device__ constexpr size_t rec_slot_bytes(bool bwd) { return (size_t)REC_R * 32 * V * (sizeof(T) * (bwd ? 2 : 1) + sizeof(G)); }
template <typename T, typename G, int V>
constexpr size_t rec_smem(bool bwd)
{
    return sizeof(RecFolds<32 * V>) * (bwd ? 2 : 1) + REC_STAGES * REC_W * rec_slot_bytes<T, G, V>(bwd);
}

// ---- forward ---------------------------------------------------------------------------------
template <typename T, typename G, int KIND, bool COMP, int V>
__global__ void __launch_bounds__(REC_THREADS, 2) rec_fwd_kernel(const RecArgs a)
{
    constexpr int CW = 32 * V;
    extern __shared__ __align__(16) unsigned char smem[];
    RecFolds<CW> &folds = *(RecFolds<CW> *)smem;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = a.split, rank = blockIdx.x % split, blk = blockIdx.x / split;
    const int bh = blk / a.ncb, c0 = blk % a.ncb * CW, b = bh / a.H, hd = bh % a.H;
    const int c = c0 + lane * V;
    const bool on = c < a.d;
    const T *x = (const T *)a.x + row_of(a.vx, b, hd, 0) + c0;
    const G *g = (const G *)a.g + row_of(a.vg, b, hd, 0) + c0;
    T *out = (T *)a.out + row_of(a.vo, b, hd, 0) + c;
    const int n = rows_of(a, b), nt = (a.L + RC - 1) / RC, steps = (nt + split - 1) / split;
    unsigned char *ring = smem + sizeof(RecFolds<CW>) + warp * rec_slot_bytes<T, G, V>(false);
    auto slot = [&](int k) { return ring + (k % REC_STAGES) * (REC_W * rec_slot_bytes<T, G, V>(false)); };
    auto first_row = [&](int k) { return (k * split + rank) * RC + warp * REC_R; };
    auto load = [&](int k) {
        if (k < steps) {
            const int t0 = first_row(k), rows = min(n - t0, REC_R);
            T *sx = (T *)slot(k);
            copy_rows<T, CW>(sx, x + t0 * a.vx.l, a.vx.l, rows, a.d - c0, a.grx, lane);
            copy_rows<G, CW>((G *)(sx + REC_R * CW), g + t0 * a.vg.l, a.vg.l, rows, a.d - c0, a.grg, lane);
        }
        cp_commit();
    };
    float carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = a.h0 && on ? a.h0[(size_t)bh * a.d + c + v] : 0.f;
#pragma unroll
    for (int k = 0; k < REC_STAGES - 1; ++k) load(k);
    if (split > 1) cluster_barrier();  // every block of the cluster is there before it is written to
    for (int k = 0; k < steps; ++k) {
        cp_wait<REC_STAGES - 2>();
        __syncwarp();
        const T *sx = (const T *)slot(k);
        const G *sg = (const G *)(sx + REC_R * CW);
        const int t0 = first_row(k), rows = min(n - t0, REC_R);
        float ga[REC_R][V], bx[REC_R][V], P[V], H[V];
#pragma unroll
        for (int i = 0; i < REC_R; ++i) {
            float xv[V], gv[V];
            get<V>(sx + i * CW + lane * V, xv);
            get<V>(sg + i * CW + lane * V, gv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float w, sl;
                gate_of<KIND, COMP>(gv[v], ga[i][v], w, sl);
                bx[i][v] = COMP ? w * xv[v] : xv[v];
            }
        }
        load(k + REC_STAGES - 1);  // into the slot of step k - 1, which the whole warp has read
        if (rows < REC_R) {
#pragma unroll
            for (int i = 0; i < REC_R; ++i)
                if (i >= rows)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        ga[i][v] = 1.f;
                        bx[i][v] = 0.f;
                    }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = ga[0][v];
            H[v] = bx[0][v];
#pragma unroll
            for (int i = 1; i < REC_R; ++i) {
                H[v] = step(ga[i][v], H[v], bx[i][v]);
                P[v] *= ga[i][v];
            }
        }
        const int buf = k & 1;
#pragma unroll
        for (int v = 0; v < V; ++v) folds.agg[buf][warp][lane * V + v] = make_float2(P[v], H[v]);
        __syncthreads();
        // the rows of the warps before this one, and of the tile
        float Pw[V], Hw[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.f;
            H[v] = 0.f;
#pragma unroll
            for (int w = 0; w < REC_W; ++w) {
                if (w == warp) {
                    Pw[v] = P[v];
                    Hw[v] = H[v];
                }
                const float2 q = folds.agg[buf][w][lane * V + v];
                H[v] = step(q.x, H[v], q.y);
                P[v] *= q.x;
            }
        }
        float h[V];
        across_tiles<V, CW>(folds, buf, split, rank, warp, lane, P, H, carry, h);
        const int tile = k * split + rank;
        if (a.chunks && warp == 0 && on && tile < nt)
#pragma unroll
            for (int v = 0; v < V; ++v) a.chunks[((size_t)bh * nt + tile) * a.d + c + v] = h[v];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = step(Pw[v], h[v], Hw[v]);
        T *o = out + t0 * a.vo.l;
        if (rows == REC_R) {
#pragma unroll
            for (int i = 0; i < REC_R; ++i) {
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = step(ga[i][v], h[v], bx[i][v]);
                if (on) put<V>(o + i * a.vo.l, h);
            }
        } else {
#pragma unroll
            for (int i = 0; i < REC_R; ++i) {
                float z[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    h[v] = step(ga[i][v], h[v], bx[i][v]);
                    z[v] = i < rows ? h[v] : 0.f;
                }
                if (on && t0 + i < a.L) put<V>(o + i * a.vo.l, z);
            }
        }
    }
    if (a.h_last && rank == 0 && warp == 0 && on)
#pragma unroll
        for (int v = 0; v < V; ++v) a.h_last[(size_t)bh * a.d + c + v] = carry[v];
}

// ---- backward ----------------------------------------------------------------------------------
// The tiles from the last to the first.  h before each row is run forward again from the state
// that the forward left for the tile.
template <typename T, typename G, int KIND, bool COMP, int V>
__global__ void __launch_bounds__(REC_THREADS, 2) rec_bwd_kernel(const RecArgs a)
{
    constexpr int CW = 32 * V;
    extern __shared__ __align__(16) unsigned char smem[];
    RecFolds<CW> &back = *(RecFolds<CW> *)smem;                          // (P, E)
    RecFolds<CW> &ahead = *(RecFolds<CW> *)(smem + sizeof(RecFolds<CW>));  // (P, H); agg alone
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = a.split, rank = blockIdx.x % split, blk = blockIdx.x / split;
    const int bh = blk / a.ncb, c0 = blk % a.ncb * CW, b = bh / a.H, hd = bh % a.H;
    const int c = c0 + lane * V;
    const bool on = c < a.d;
    const T *x = (const T *)a.x + row_of(a.vx, b, hd, 0) + c0;
    const G *g = (const G *)a.g + row_of(a.vg, b, hd, 0) + c0;
    const T *dout = (const T *)a.dout + row_of(a.vo, b, hd, 0) + c0;
    T *dx = (T *)a.dx + row_of(a.vdx, b, hd, 0) + c;
    G *dg = (G *)a.dg + row_of(a.vdg, b, hd, 0) + c;
    const int n = rows_of(a, b), nt = (a.L + RC - 1) / RC, steps = (nt + split - 1) / split;
    unsigned char *ring = smem + 2 * sizeof(RecFolds<CW>) + warp * rec_slot_bytes<T, G, V>(true);
    auto slot = [&](int k) { return ring + (k % REC_STAGES) * (REC_W * rec_slot_bytes<T, G, V>(true)); };
    // a step's tiles run backwards; before the first tile there are none (negative rows)
    auto first_row = [&](int k) { return (nt - 1 - (k * split + rank)) * RC + warp * REC_R; };
    auto load = [&](int k) {
        if (k < steps && first_row(k) >= 0) {
            const int t0 = first_row(k), rows = min(n - t0, REC_R);
            T *sx = (T *)slot(k), *sd = sx + REC_R * CW;
            copy_rows<T, CW>(sx, x + t0 * a.vx.l, a.vx.l, rows, a.d - c0, a.grx, lane);
            copy_rows<T, CW>(sd, dout + t0 * a.vo.l, a.vo.l, rows, a.d - c0, a.gro, lane);
            copy_rows<G, CW>((G *)(sd + REC_R * CW), g + t0 * a.vg.l, a.vg.l, rows, a.d - c0, a.grg, lane);
        }
        cp_commit();
    };
    float carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = a.dh_last && on ? a.dh_last[(size_t)bh * a.d + c + v] : 0.f;
#pragma unroll
    for (int k = 0; k < REC_STAGES - 1; ++k) load(k);
    if (split > 1) cluster_barrier();
    for (int k = 0; k < steps; ++k) {
        cp_wait<REC_STAGES - 2>();
        __syncwarp();
        load(k + REC_STAGES - 1);  // into the slot of step k - 1, which the whole warp has read
        const T *sx = (const T *)slot(k), *sd = sx + REC_R * CW;
        const G *sg = (const G *)(sd + REC_R * CW);
        const int tile = nt - 1 - (k * split + rank), t0 = first_row(k);
        const int rows = tile < 0 ? 0 : min(n - t0, REC_R);
        float h[V];  // the state before the tile
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = on && tile >= 0 ? a.chunks_in[((size_t)bh * nt + tile) * a.d + c + v] : 0.f;
        float ga[REC_R][V], hb[REC_R][V], P[V], H[V], E[V];  // hb: w x, then the state before the row
#pragma unroll
        for (int i = 0; i < REC_R; ++i) {
            float xv[V], gv[V];
            get<V>(sx + i * CW + lane * V, xv);
            get<V>(sg + i * CW + lane * V, gv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float w, sl;
                gate_of<KIND, COMP>(gv[v], ga[i][v], w, sl);
                hb[i][v] = COMP ? w * xv[v] : xv[v];
                if (i >= rows) {
                    ga[i][v] = 1.f;
                    hb[i][v] = 0.f;
                }
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.f;
            H[v] = 0.f;
            E[v] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < REC_R; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                H[v] = step(ga[i][v], H[v], hb[i][v]);
                P[v] *= ga[i][v];
            }
#pragma unroll
        for (int i = REC_R - 1; i >= 0; --i) {
            float dv[V];
            get<V>(sd + i * CW + lane * V, dv);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (i < rows) E[v] = forget(ga[i][v], E[v] + dv[v]);
        }
        const int buf = k & 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            back.agg[buf][warp][lane * V + v] = make_float2(P[v], E[v]);
            ahead.agg[buf][warp][lane * V + v] = make_float2(P[v], H[v]);
        }
        __syncthreads();
        float Pw[V], Ew[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int w = 0; w < REC_W; ++w)
                if (w < warp) {
                    const float2 q = ahead.agg[buf][w][lane * V + v];
                    h[v] = step(q.x, h[v], q.y);
                }
            P[v] = 1.f;
            E[v] = 0.f;
#pragma unroll
            for (int w = REC_W - 1; w >= 0; --w) {
                if (w == warp) {
                    Pw[v] = P[v];
                    Ew[v] = E[v];
                }
                const float2 q = back.agg[buf][w][lane * V + v];
                E[v] = step(q.x, E[v], q.y);
                P[v] *= q.x;
            }
        }
        float e[V];
        across_tiles<V, CW>(back, buf, split, rank, warp, lane, P, E, carry, e);
#pragma unroll
        for (int v = 0; v < V; ++v) e[v] = step(Pw[v], e[v], Ew[v]);
#pragma unroll
        for (int i = 0; i < REC_R; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float bx = hb[i][v];
                hb[i][v] = h[v];
                h[v] = step(ga[i][v], h[v], bx);
            }
        if (tile >= 0) {
            T *ox = dx + t0 * a.vdx.l;
            G *og = dg + t0 * a.vdg.l;
#pragma unroll
            for (int i = REC_R - 1; i >= 0; --i) {
                float xv[V], gv[V], dv[V], rx[V], rg[V];
                get<V>(sx + i * CW + lane * V, xv);
                get<V>(sg + i * CW + lane * V, gv);
                get<V>(sd + i * CW + lane * V, dv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float ai, w, sl;
                    gate_of<KIND, COMP>(gv[v], ai, w, sl);
                    rx[v] = rg[v] = 0.f;
                    if (i < rows) {
                        e[v] += dv[v];  // e_t
                        rx[v] = COMP ? w * e[v] : e[v];
                        rg[v] = forget(sl, e[v] * (COMP ? hb[i][v] - xv[v] : hb[i][v]));
                        e[v] = forget(ga[i][v], e[v]);
                    }
                }
                if (on && t0 + i < a.L) {
                    put<V>(ox + i * a.vdx.l, rx);
                    put<V>(og + i * a.vdg.l, rg);
                }
            }
        }
    }
    if (a.dh0 && rank == 0 && warp == 0 && on)
#pragma unroll
        for (int v = 0; v < V; ++v) a.dh0[(size_t)bh * a.d + c + v] = carry[v];
}

constexpr int STEP_THREADS = 128;

template <typename T, typename G, int KIND, bool COMP>
__global__ void __launch_bounds__(STEP_THREADS) rec_step_kernel(const T *x, const G *g, float *state, T *out,
                                                                long long n)
{
    const long long i = (long long)blockIdx.x * STEP_THREADS + threadIdx.x;
    if (i >= n) return;
    float ga, w, sl;
    gate_of<KIND, COMP>(to_f32(g[i]), ga, w, sl);
    const float h = step(ga, state[i], COMP ? w * to_f32(x[i]) : to_f32(x[i]));
    state[i] = h;
    out[i] = from_f32<T>(h);
}

// ---- host side ---------------------------------------------------------------------------------
// Blocks of a cluster: as many as the sequence has tiles for and one wave of the GPU (two blocks
// an SM) holds.
int choose_split(long long blocks, int L, int sms)
{
    const long long tiles = ((long long)L + RC - 1) / RC, fit = 2ll * sms / blocks;
    return (int)std::max(1ll, std::min(std::min(tiles, fit), (long long)REC_MAX_SPLIT));
}

int granule(const void *p, const View &v, const RecArgs &a, size_t elem)
{
    for (size_t g : {(size_t)16, (size_t)4})
        if (g > elem ? rows_aligned(p, v, a.B, a.H, a.L, elem, g) && a.d * elem % g == 0 : g == elem) return (int)g;
    return 2;
}

template <typename Kern>
int launch_rec(Kern kern, const RecArgs &a, size_t smem, cudaStream_t s)
{
    const long long blocks = (long long)a.B * a.H * a.ncb * a.split;
    if (blocks > INT_MAX) return LA_ERR_SHAPE;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return LA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(REC_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
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

// Two channels a lane where both inputs are bf16 and pairs are whole and aligned: a row of a block
// is then 128 bytes, as it is with one channel a lane in fp32.
template <bool BWD>
struct LaunchRec {
    RecArgs &a;
    int sms;
    cudaStream_t s;
    template <typename T, typename G, int KIND, bool COMP, int V> int go() const
    {
        a.ncb = (a.d + 32 * V - 1) / (32 * V);
        a.split = choose_split((long long)a.B * a.H * a.ncb, a.L, sms);
        if constexpr (BWD) return launch_rec(rec_bwd_kernel<T, G, KIND, COMP, V>, a, rec_smem<T, G, V>(true), s);
        else return launch_rec(rec_fwd_kernel<T, G, KIND, COMP, V>, a, rec_smem<T, G, V>(false), s);
    }
    template <typename T, typename G, int KIND, bool COMP> int operator()() const
    {
        if constexpr (sizeof(T) == 2 && sizeof(G) == 2 && !BWD) {
            auto pairs = [&](const void *p, const View &v) { return rows_aligned(p, v, a.B, a.H, a.L, 2, 4); };
            if (a.d % 2 == 0 && a.d > 32 && pairs(a.x, a.vx) && pairs(a.g, a.vg) && pairs(a.out, a.vo))
                return go<T, G, KIND, COMP, 2>();
        }
        return go<T, G, KIND, COMP, 1>();
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
        const unsigned grid = (unsigned)((n + STEP_THREADS - 1) / STEP_THREADS);
        rec_step_kernel<T, G, KIND, COMP><<<grid, STEP_THREADS, 0, s>>>((const T *)x, (const G *)g, state, (T *)out, n);
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
    a.grx = granule(x, a.vx, a, e);
    a.grg = granule(gate, a.vg, a, dtype_size(gate_dtype));
    const int sms = device_sms();
    if (sms <= 0) return LA_ERR_CUDA;
    return dispatch(dtype, gate_dtype, gate_kind, complement != 0, LaunchRec<false>{a, sms, (cudaStream_t)stream});
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
    if (sms <= 0) return LA_ERR_CUDA;
    return dispatch(dtype, gate_dtype, gate_kind, complement != 0, LaunchRec<true>{a, sms, (cudaStream_t)stream});
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
