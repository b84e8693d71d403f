// gated_tc.cu -- the gated attention on the tensor cores (sm_103a): bf16, 64 or 128 channels.
//
// One sweep computes S <- a S + y z^T, out = x^T S over a head's rows, in chunks of 64. With G the sums of
// the chunk's log decays up to and with each row, S the state before the chunk:
//
//     out_i = e_i x_i^T S + sum_{j<=i} w_ij (x_i . y_j) z_j,     e_i = exp(G_i), w_ij = exp(G_i - G_j),
//     S    <- exp(G_63) S + sum_j f_j y_j z_j^T,                 f_j = exp(G_63 - G_j).
//
// No weight is above 1, and none is a quotient, so no decay is too fast; the log decays are data and differ
// by row, so no factor of theirs can be moved into an operand. A row whose decay is 0 cuts the chunk:
// pairs across it are 0. From the last row on (the gradients of k and v) e and f change places and
// the mask turns. The forward pass is the sweep of (q, k, v), dq that of (dout, v, k), dk that of (v, dout, q)
// and dv that of (k, q, dout), the last two from the end.
//
// Products per chunk (bf16 operands, fp32 sums; DX, DZ: 64 or 128 channels of x, y and of z):
//     scores  A     = X Y^T            M 64   N 64   K DX     both K-major
//     state   dS^T  = Z^T Y~           M DZ   N DX   K 64     both MN-major; Y~ = f Y in three bf16 parts
//     inter   Oi^T  = S^T X^T          M DZ   N 64   K DX     S^T from TMEM, in NS bf16 parts
//     intra   Oa^T  = Z^T P^T          M DZ   N 64   K 64     P = w A
//     inner   A2    = W Z^T            M 64   N 64   K DZ     backward only, see below
// What is rounded to bf16: P once, and S once where only a bf16 output reads it (NS = 1; the output's own
// rounding is as large). The state itself is fp32 in registers: dS is summed by itself and joins it by one
// rounding a chunk, and Y~'s three parts hold f Y to 2^-24, so that states are those of fp32 arithmetic. The
// decays' gradient reads the inter rows, there S too has three parts.
//
// Warps (640 threads, one block an SM): 0 loads tiles by TMA into a ring, 2 and 3 form the chunks' weights (64-bit
// sums), 1 issues the products. The 16 others all do the same, a part each: Y~, the rows of the chunk
// before, P, the state's update (S^T in registers: a lane of the warp's TMEM quadrant, a quarter of the columns) and
// its copy. The order hides each product behind a step that does not need it; and warps that run the
// same steps together share the instructions they fetch (with one group for Y~ and P and one for the state
// and the rows, fetching was the largest stall, and a chunk took 4,300 cycles).
//
// The decays' gradient (DOT) needs R_i = q_i . dq_i and C_j = k_j . dk_j without the rows' own pairs. Over
// earlier chunks they are the products of the inter rows with a fourth tile (q or k, W); inside the chunk
// R and C are the row and column sums of w_ij (dout_i . v_j) (q_i . k_j), which the dq sweep forms from both
// score blocks in fp32 (INNER). Every 1024 rows the sweeps store S and D for the anchors.
//
// Bound: at 128 channels a chunk reads and writes 64 KB, 2,500 cycles of an SM's share of the memory; it takes 4,100
// (B8 H16 L8192 262 us, 61% of the measured copy rate): the workers' instructions and the
// round of products and waits that one chunk's state makes. With DOT 6,000: three parts of the state are copied and
// multiplied.
#include <algorithm>
#include <atomic>
#include <stdlib.h>

#include "gated.cuh"
#include "tc_common.cuh"

namespace la {

using namespace ptx;
using namespace tcc;

namespace {

constexpr int GT_THREADS = 640;
constexpr int GT_C = 64;      // rows of a chunk
constexpr int GT_SLOTS = 8;   // ring of the chunks' weights
constexpr int GT_W0 = 4, GT_WORKERS = 16;  // the workers: warps 4 .. 19

struct GtArgs {
    CUtensorMap mx, my, mz, mw;
    const float *g;
    View vg, vo;
    void *out;
    int out_f32;
    int sx, sy, sz, sw;  // heads of the state to a head of the operand
    int B, H, L;
    float yscale, oscale;
    int reverse, totals;
    int seg_rows, nseg;
    const int *lengths, *slots;
    int n_slots;
    const float *init;
    float *fin, *decay;
    int by_seg;
    int rs, cs;          // element (x channel, z channel) of a stored state
    float *anchors;      // S at the anchors' starts (causal; one more behind the last) or D at their ends
    int anchor_chunks, n_anchors;
    float *dot;          // DOT: [4][B H][L] inter parts, then (inner) [4] row sums
    float *dotc;         // inner: [4][B H][L] column sums
    int *err;
    unsigned long long timeout_ns;
};

constexpr float GT_CUT = 16384.f;  // doublings that a decay of 0 counts for in G: no pair reaches across

struct Weights {          // of one chunk
    float hi[GT_C], lo[GT_C];  // G (-G in reverse) in doublings
    float kw[GT_C];       // of Y's rows (f, or e in reverse), times yscale
    float rw[GT_C];       // of the inter rows (e, or f in reverse), times oscale
    float a, em, pad[2];  // decay over the chunk, and that minus 1
};

// A log decay above -104 in units of 2^-44 doublings, to a unit: the product with log2 e in two parts.
constexpr int UNIT_BITS = 44;
constexpr float UNIT = 5.684341886080801e-14f, UNITS = 17592186044416.f;
__device__ __forceinline__ long long doublings(float g)
{
    constexpr float LOG2E = 1.44269502f, LOG2E_REST = 1.92596303e-8f;
    const float p = g * LOG2E, rest = fmaf(g, LOG2E_REST, fmaf(g, LOG2E, -p));
    return __float2ll_rn(p * UNITS) + __float2ll_rn(rest * UNITS);
}

template <int DX, int DZ, bool DOT> struct GtLayout {
    static constexpr int NS = DOT ? 3 : 1;  // bf16 parts of the state's copy
    static constexpr int X = GT_C * DX * 2, Z = GT_C * DZ * 2;
    static constexpr int STAGE = 2 * X + Z;
    static constexpr int WST = 3, WR = DOT ? WST * Z : 0;  // W's tiles are held longer: a ring of their own
    static constexpr int YT = 3 * X, P = GT_C * GT_C * 2;
    static constexpr int OUT = 16 * (DZ / 4) * 2;    // a worker's 16 rows of its quadrant's channels
    static constexpr int OUTS = GT_WORKERS * OUT;
    static constexpr int FIXED = WR + YT + P + OUTS + GT_SLOTS * (int)sizeof(Weights) + 256 + 1024;
    static constexpr int STAGES = (232448 - FIXED) / STAGE >= 4 ? 4 : (232448 - FIXED) / STAGE;
    static constexpr int OFF_WR = STAGES * STAGE, OFF_YT = OFF_WR + WR, OFF_P = OFF_YT + YT, OFF_O = OFF_P + P, OFF_W = OFF_O + OUTS,
                         OFF_BAR = OFF_W + GT_SLOTS * (int)sizeof(Weights), ALLOC = OFF_BAR + 256 + 1024;
    // TMEM columns
    // one part: two copies of the state in turn, so that the next one need not wait for the inter product
    static constexpr int COPIES = DOT ? 1 : 2;
    static constexpr uint32_t T_SC = 0, T_DS = NS * COPIES * (DX / 2), T_OI = T_DS + DX, T_OA = T_OI + 64, T_A = T_OA + 64;
    // the second score block has columns of its own where they are left, else those of Oi
    static constexpr bool A2_OWN = T_A + 128 <= 512;
    static constexpr uint32_t T_A2 = A2_OWN ? T_A + 64 : T_OI;
    static_assert(T_A + 64 <= 512 && ALLOC <= 232448 - 64 && STAGES >= (DOT ? 2 : 3), "fits");
    static_assert(STAGE % 1024 == 0 && YT % 1024 == 0, "swizzle atoms");
};

// Two values in three bf16 parts each: hi + mid + lo = x to 2^-24.
__device__ __forceinline__ Ch<2> less(const Ch<2> &x, uint32_t part)
{
    return fma(Ch<2>{{bf_lo(part), bf_hi(part)}}, all<2>(-1.f), x);
}
__device__ __forceinline__ void split3(Ch<2> x, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    hi = pack_bf16x2(x.v[0], x.v[1]);
    x = less(x, hi);
    mid = pack_bf16x2(x.v[0], x.v[1]);
    x = less(x, mid);
    lo = pack_bf16x2(x.v[0], x.v[1]);
}

// wait_phase with the clock read only once a wait was long (the timer is far from the SM), and its loop
// out of line: they are in the loop of every role.
__device__ __noinline__ bool wait_longer(uint64_t *bar, uint32_t parity, volatile int *abort, int *err, unsigned long long timeout_ns)
{
    return wait_phase(bar, parity, Ctl{abort, err, timeout_ns});
}
__device__ __forceinline__ bool wait_long(uint64_t *bar, uint32_t parity, const Ctl &ctl)
{
    if (mbar_try(bar, parity)) return true;
    return wait_longer(bar, parity, ctl.abort, ctl.err, ctl.timeout_ns);
}

// Chunks at a sweep's start whose rows' decays to its end are below the normal range of fp32: they add nothing to the
// sums of a segment. Called by the whole block; 0 where a log decay is positive. cs: scratch, a float a chunk.
__device__ __forceinline__ int far_chunks(const float *g, long long step, int t0, int te, int nch, bool rev, float *cs)
{
    __shared__ int found;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (nch > 8192) return 0;
    bool odd = false;
#pragma unroll 2
    for (int k = warp; k < nch; k += GT_THREADS / 32) {
        const int t = t0 + k * GT_C + lane;
        const float a = t < te ? g[(long long)t * step] : 0.f, b = t + 32 < te ? g[(long long)(t + 32) * step] : 0.f;
        odd |= !(a <= 0.f) || !(b <= 0.f);
        float s = a + b;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) cs[k] = s;
    }
    if (threadIdx.x == 0) found = 0;
    odd = __syncthreads_or(odd);
    if (warp == 0 && !odd) {
        float sum = 0.f;
        for (int k0 = 0; k0 < nch; k0 += 32) {  // from the sweep's end
            const int k = k0 + lane;
            float s = k < nch ? cs[rev ? k : nch - 1 - k] : 0.f;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += u;
            }
            const uint32_t below = __ballot_sync(0xffffffffu, k < nch && sum + s < -88.f);
            if (below) {
                if (lane == 0) found = nch - (k0 + __ffs(below));
                break;
            }
            sum += __shfl_sync(0xffffffffu, s, 31);
        }
    }
    __syncthreads();
    const int n = found;
    fence_async_smem();  // the tiles take the scratch's place
    __syncthreads();
    return n;
}

template <int DX, int DZ, bool DOT, bool INNER>
__global__ void __launch_bounds__(GT_THREADS, 1) gated_tc_kernel(const __grid_constant__ GtArgs a)
{
    using Lay = GtLayout<DX, DZ, DOT>;
    constexpr int C = GT_C, NST = Lay::STAGES, NS = Lay::NS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long sums[2], doubled[2];  // of the log decays, by the warps that form the weights: units, doublings
    __shared__ bool cuts_of[2];
    uint8_t *const sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Weights *const weights = (Weights *)(sm + Lay::OFF_W);
    uint64_t *const bars = (uint64_t *)(sm + Lay::OFF_BAR);
    uint64_t *const full = bars, *const stage_free = full + NST, *const yt_ready = stage_free + NST, *const state_done = yt_ready + 1,
             *const s_ready = state_done + 1, *const scores_done = s_ready + 1, *const sc_free = scores_done + 1,
             *const p_ready = sc_free + 1, *const o_done = p_ready + 1, *const o_free = o_done + 1,
             *const inter_done = o_free + 1, *const drain = inter_done + 1,
             *const w_free = drain + 1;
    uint32_t *const tmem_slot = (uint32_t *)(sm + Lay::OFF_BAR + 224);
    volatile int *const abort_flag = (volatile int *)(sm + Lay::OFF_BAR + 228);

    // The totals pass works on two chunks at a time: the second place of Y~ is the tiles of X, which it does not load,
    // that of dS the columns of Oi and after, the second barriers are ones that it does not need otherwise.
    uint64_t *const y_done[2] = {yt_ready, sc_free}, *const ds_done[2] = {state_done, scores_done}, *const ds_free[2] = {s_ready, p_ready};

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int BH = a.B * a.H, bh = blockIdx.x % BH, seg = blockIdx.x / BH, b = bh / a.H, h = bh % a.H;
    const int t0 = seg * a.seg_rows, t1 = min(t0 + a.seg_rows, a.L),
              te = max(t0, min(t1, gated_rows(a.lengths, b, a.L)));
    const bool totals = a.totals != 0, rev = INNER ? false : a.reverse != 0;
    const int slot = gated_slot(a.slots, b, a.n_slots, tid == 0 ? a.err : nullptr);
    const Ctl ctl{abort_flag, a.err, a.timeout_ns};
    auto tile_x = [&](int s) { return sm + s * Lay::STAGE; };
    auto tile_y = [&](int s) { return tile_x(s) + Lay::X; };
    auto tile_z = [&](int s) { return tile_y(s) + Lay::X; };
    auto tile_w = [&](int c) { return sm + Lay::OFF_WR + (c % Lay::WST) * Lay::Z; };  // of chunk c
    uint8_t *const yt = sm + Lay::OFF_YT, *const p_tile = sm + Lay::OFF_P;

    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 2);                       // the TMA's bytes, the weights
            mbar_init(&stage_free[i], 1);
        }
        for (int i = 0; i < Lay::WST; ++i) mbar_init(&w_free[i], GT_WORKERS);
        mbar_init(yt_ready, GT_WORKERS);
        mbar_init(state_done, 1);
        // No phase of a barrier completes before everyone has waited for the one before it, or a waiter could take
        // it for that one: the workers go round together, and each step of theirs needs the issuer's last one.
        mbar_init(s_ready, GT_WORKERS);
        mbar_init(scores_done, 1);
        mbar_init(sc_free, GT_WORKERS);
        mbar_init(p_ready, GT_WORKERS);
        mbar_init(o_done, 1);
        mbar_init(o_free, GT_WORKERS);
        mbar_init(inter_done, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    int nch = (te - t0 + C - 1) / C, skip = 0;
    if (!DOT && totals) {
        skip = far_chunks(a.g + b * a.vg.b + h * a.vg.h, a.vg.l, t0, te, nch, rev, (float *)sm);
        nch -= skip;
    }
    auto chunk_of = [&](int c) { return rev ? nch - 1 - c : c + skip; };  // c-th chunk of the sweep
    auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_long(bar, parity, ctl)) != 0; };
    auto arrive = [&](uint64_t *bar) {  // of a warp whose lanes have all done their part
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    // ---- a worker's place: quadrant q4 of TMEM, part `part` of four of the columns or rows
    const int q4 = warp & 3, part = (warp - GT_W0) >> 2, cpos = lane & 3;
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    const long long out0 = row_of(a.vo, b, h, 0);
    constexpr int HALVES = DZ / 64;  // blocks of 16 channels of a quadrant
    // block of 8 rows and 8 channels that this lane addresses for stmatrix and ldmatrix (of four, then the
    // next 8 rows), and its place in the worker's tile of 64- or 32-byte rows, free of bank conflicts
    const int at_row = (lane & 7) + (DZ == 64 ? 8 * (lane >> 4) : 0), at_ch = DZ == 64 ? (lane >> 3) & 1 : lane >> 3;
    uint8_t *const o_tile = sm + Lay::OFF_O + ((warp - GT_W0) & 15) * Lay::OUT;
    auto o_place = [](int row, int ch) { return row * (DZ / 2) + ((ch ^ (DZ == 64 ? (row >> 2) & 1 : (row >> 1) & 3)) << 4); };

    bool forgets = false;  // the decay over the chunk that the state has gone past last is 0
    // A quarter of the rows of the sweep's chunk c, the channels of the quadrant: the inter rows weighted, the intra
    // rows added, stored; with DOT the inter rows' products with W's. Lane l reads channel l / 4 of each block
    // of 8 and rows 2 (l % 4) and the next one of two blocks; stmatrix turns these pairs of rows into rows of
    // channels, which leave 16 bytes a lane. (Two-byte stores from a lane a channel took ten times the
    // instructions; TMA stores, 50 cycles of the unit each, were slower than these.)
    auto rows = [&](int c) {
        const int row0 = t0 + chunk_of(c) * C, nv = min(C, te - row0), first = 16 * part;
        const Weights &w = weights[c % GT_SLOTS];
        uint32_t oi[HALVES][8], oa[HALVES][8];
#pragma unroll
        for (int i = 0; i < HALVES; ++i) {
            tmem_ld16x256_x2(tmem + lanes + ((uint32_t)(16 * i) << 16) + Lay::T_OI + first, oi[i]);
            tmem_ld16x256_x2(tmem + lanes + ((uint32_t)(16 * i) << 16) + Lay::T_OA + first, oa[i]);
        }
        const float2 rw[2] = {*(const float2 *)&w.rw[first + 2 * cpos], *(const float2 *)&w.rw[first + 8 + 2 * cpos]};
        Ch<2> dot[2] = {all<2>(0.f), all<2>(0.f)};
        uint32_t wt[HALVES][4];
        if (DOT) {
            // W's blocks as O's: channels of the quadrant, rows first + 8 k
#pragma unroll
            for (int k = 0; k < HALVES; ++k) {
                const int t = first + 8 * k + at_row, cg = (DZ / 32) * q4 + at_ch;
                ldmatrix_t(smem_u32(tile_w(c)) + (cg >> 3) * C * 128 + t * 128 + (((cg & 7) ^ (t & 7)) << 4), wt[k]);
            }
        }
        tmem_wait_ld();
        tc_fence_before();
        arrive(o_free);
        // a row whose decay from the chunk's start is 0 has forgotten the state, whatever it held: 0 times an infinity or
        // NaN is not 0 (a branch on a register: 0.4% of a prompt without resets, 1.8% with one in eight chunks)
        if (forgets)
#pragma unroll
            for (int i = 0; i < HALVES; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (rw[e >> 1].x == 0.f) oi[i][2 * e] = 0;
                    if (rw[e >> 1].y == 0.f) oi[i][2 * e + 1] = 0;
                }
        Ch<2> y[HALVES][4];  // [][2 k + g]: rows 8 k .., channels 8 g ..
#pragma unroll
        for (int i = 0; i < HALVES; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Ch<2> r{{rw[e >> 1].x, rw[e >> 1].y}};
                const Ch<2> xi{{__uint_as_float(oi[i][2 * e]), __uint_as_float(oi[i][2 * e + 1])}},
                    xa{{__uint_as_float(oa[i][2 * e]), __uint_as_float(oa[i][2 * e + 1])}};
                y[i][e] = fma(r, xi, xa);
                if (DOT) {
                    const uint32_t u = DZ == 128 ? wt[e >> 1][2 * i + (e & 1)] : wt[0][e];
                    dot[e >> 1] = fma(mul(r, xi), Ch<2>{{bf_lo(u), bf_hi(u)}}, dot[e >> 1]);
                }
            }
        if (!a.out_f32) {
            uint32_t o[HALVES][4];
#pragma unroll
            for (int i = 0; i < HALVES; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] = pack_bf16x2(y[i][e].v[0], y[i][e].v[1]);
            const uint32_t tile = smem_u32(o_tile) + o_place(at_row, at_ch);
            __syncwarp();  // the tile's last rows have been read
            if constexpr (DZ == 128) {
                stmatrix_t(tile, o[0][0], o[0][1], o[1][0], o[1][1]);
                stmatrix_t(tile + 8 * (DZ / 2), o[0][2], o[0][3], o[1][2], o[1][3]);
            } else {
                stmatrix_t(tile, o[0][0], o[0][1], o[0][2], o[0][3]);
            }
            __syncwarp();
            constexpr int PIECES = DZ / 32;  // of 16 bytes in a row
            const int r = lane / PIECES, p = lane % PIECES;
            __nv_bfloat16 *const g = (__nv_bfloat16 *)a.out + out0 + (long long)(row0 + first + r) * a.vo.l + (DZ / 4) * q4 + 8 * p;
#pragma unroll
            for (int i = 0; i < 16 * PIECES / 32; ++i) {
                const int rr = r + i * (32 / PIECES);
                if (first + rr < nv) *(uint4 *)(g + (long long)(i * (32 / PIECES)) * a.vo.l) = *(const uint4 *)(o_tile + o_place(rr, p));
            }
        } else {
            float *const p = (float *)a.out + out0 + (DZ / 4) * q4 + (lane >> 2);
#pragma unroll
            for (int i = 0; i < HALVES; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int t = first + 8 * (e >> 1) + 2 * cpos + u;
                        if (t < nv) p[(long long)(row0 + t) * a.vo.l + 16 * i + 8 * (e & 1)] = y[i][e].v[u];
                    }
        }
        if (DOT) {
            // over the channels: lanes l / 4; a lane goes on with half of its four rows each time
            float v[4] = {dot[0].v[0], dot[0].v[1], dot[1].v[0], dot[1].v[1]};
            const bool up = lane & 4, up2 = lane & 8;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float send = up ? v[i] : v[i + 2], keep = up ? v[i + 2] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 4);
            }
            float d = up2 ? v[1] : v[0];
            d += __shfl_xor_sync(0xffffffffu, up2 ? v[0] : v[1], 8);
            d += __shfl_xor_sync(0xffffffffu, d, 16);
            const int t = first + (up ? 8 : 0) + 2 * cpos + (up2 ? 1 : 0);
            if (!(lane & 16) && t < nv) a.dot[((long long)q4 * BH + bh) * a.L + row0 + t] = d;
        }
    };

    if (warp == 0) {
        // ------------------------------------------------------------ tiles
        if (lane == 0) {
            int issued = 0;
            for (int c = 0; c < nch; ++c) {
                const int s = c % NST;
                if (c >= NST && !wait_long(&stage_free[s], ((c / NST) - 1) & 1, ctl)) break;
                if (DOT && c >= Lay::WST && !wait_long(&w_free[c % Lay::WST], ((c / Lay::WST) - 1) & 1, ctl)) break;
                const int row = t0 + chunk_of(c) * C;
                mbar_arrive_expect_tx(&full[s], totals ? Lay::X + Lay::Z : Lay::STAGE + (DOT ? Lay::Z : 0));
                for (int k = 0; k < DX / 64; ++k) {
                    if (!totals) tma_load_4d(tile_x(s) + k * C * 128, &a.mx, k * 64, row, h / a.sx, b, &full[s]);
                    tma_load_4d(tile_y(s) + k * C * 128, &a.my, k * 64, row, h / a.sy, b, &full[s]);
                }
                for (int k = 0; k < DZ / 64; ++k) {
                    tma_load_4d(tile_z(s) + k * C * 128, &a.mz, k * 64, row, h / a.sz, b, &full[s]);
                    if (DOT && !totals) tma_load_4d(tile_w(c) + k * C * 128, &a.mw, k * 64, row, h / a.sw, b, &full[s]);
                }
                issued = c + 1;
            }
            // never leave the CTA with loads in flight: wait for every issued stage to land
            for (int c = (issued > NST ? issued - NST : 0); c < issued; ++c) {
                const uint64_t begin = globaltimer();
                while (!mbar_try_sleep(&full[c % NST], (c / NST) & 1, 200000u))
                    if (globaltimer() - begin > ctl.timeout_ns) break;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        // The whole warp runs the loop and one lane of it issues, so that descriptors stay in uniform registers (a
        // product takes 35 cycles to issue instead of 100). In the order in which the workers get ready for them.
        const uint32_t one = elect_one(), tm = __reduce_or_sync(0xffffffffu, tmem);
        const int n = (int)__reduce_or_sync(0xffffffffu, (uint32_t)nch);
        constexpr uint32_t ID_SC = idesc_bf16_f32(C, C, 0, 0), ID_INTER = idesc_bf16_f32(DZ, C, 0, 0),
                           ID_STATE = idesc_bf16_f32(DZ, DX, 1, 1), ID_INTRA = idesc_bf16_f32(DZ, C, 1, 0);
        auto scores = [&](int c) {
            const int s = c % NST;
            if (!wait(&full[s], (c / NST) & 1)) return false;
            tc_fence_after();
            const uint64_t dx = smem_desc(smem_u32(tile_x(s)), 16, 1024), dy = smem_desc(smem_u32(tile_y(s)), 16, 1024);
#pragma unroll
            for (int k = 0; k < DX / 16; ++k) {
                const uint32_t o = (k >> 2) * C * 128 + (k & 3) * 32;
                mma_ss_if(tm + Lay::T_A, desc_add(dx, o), desc_add(dy, o), ID_SC, k > 0, one);
            }
            if (INNER) {
                const uint64_t dw = smem_desc(smem_u32(tile_w(c)), 16, 1024), dz = smem_desc(smem_u32(tile_z(s)), 16, 1024);
#pragma unroll
                for (int k = 0; k < DZ / 16; ++k) {
                    const uint32_t o = (k >> 2) * C * 128 + (k & 3) * 32;
                    mma_ss_if(tm + Lay::T_A2, desc_add(dw, o), desc_add(dz, o), ID_SC, k > 0, one);
                }
            }
            mma_commit_if(scores_done, one);
            return true;
        };
        // the second scores of the next chunk lie in Oi's columns: they wait for the rows' readers
        constexpr bool late = INNER && !Lay::A2_OWN;
        // Parts from the smallest on: the products' sums lose what is behind their 24 bits at every step, which
        // matters only while they are as large as the whole (the decays' gradients at 128 channels are off by 6.1e-7
        // in the mean, 1.1e-6 from the largest part on).
        auto sums_of = [&](int c, uint32_t y0, uint32_t y_step, uint32_t column) {  // dS of chunk c
            const uint64_t dz = smem_desc(smem_u32(tile_z(c % NST)), C * 128, 1024);
#pragma unroll
            for (int p = 2; p >= 0; --p) {
                const uint64_t dy = smem_desc(y0 + p * y_step, C * 128, 1024);
#pragma unroll
                for (int k = 0; k < C / 16; ++k)
                    mma_ss_if(tm + column, desc_add(dz, k * 2048), desc_add(dy, k * 2048), ID_STATE, p < 2 || k > 0, one);
            }
        };
        if (!DOT && totals)
            for (int c = 0; c < n; ++c) {
                const int i = c & 1;
                if (c >= 2 && !wait(ds_free[i], ((c >> 1) - 1) & 1)) break;
                if (!wait(y_done[i], (c >> 1) & 1)) break;
                tc_fence_after();
                if (i) sums_of(c, smem_u32(tile_x(0)), Lay::STAGE, Lay::T_OI);
                else sums_of(c, smem_u32(yt), Lay::X, Lay::T_DS);
                mma_commit_if(ds_done[i], one);
                mma_commit_if(&stage_free[c % NST], one);
            }
        bool ok = n > 0 && !totals && scores(0);
        for (int c = 0; ok && c < n; ++c) {
            const int s = c % NST;
            const uint64_t dz = smem_desc(smem_u32(tile_z(s)), C * 128, 1024);
            if (!(ok = wait(s_ready, c & 1))) break;  // the state's copy, and dS has been read
            if (!(ok = wait(yt_ready, c & 1))) break;
            tc_fence_after();
            sums_of(c, smem_u32(yt), Lay::X, Lay::T_DS);
            mma_commit_if(state_done, one);
            if (c > 0 && !(ok = wait(o_free, (c - 1) & 1))) break;
            if (late && !(ok = wait(sc_free, c & 1))) break;
            tc_fence_after();
            const uint64_t dx = smem_desc(smem_u32(tile_x(s)), 16, 1024);
            const uint32_t sc = tm + Lay::T_SC + (c % Lay::COPIES) * (DX / 2);
#pragma unroll
            for (int p = NS - 1; p >= 0; --p)
#pragma unroll
                for (int k = 0; k < DX / 16; ++k)
                    mma_ts_if(tm + Lay::T_OI, sc + p * (DX / 2) + k * 8, desc_add(dx, (k >> 2) * C * 128 + (k & 3) * 32), ID_INTER,
                              p < NS - 1 || k > 0, one);
            if (DOT) mma_commit_if(inter_done, one);
            if (!DOT) {
                if (!(ok = wait(sc_free, c & 1))) break;
                if (c + 1 < n && !(ok = scores(c + 1))) break;
            }
            if (!(ok = wait(p_ready, c & 1))) break;
            tc_fence_after();
            const uint64_t dp = smem_desc(smem_u32(p_tile), 16, 1024);
#pragma unroll
            for (int k = 0; k < C / 16; ++k)
                mma_ss_if(tm + Lay::T_OA, desc_add(dz, k * 2048), desc_add(dp, k * 32), ID_INTRA, k > 0, one);
            mma_commit_if(o_done, one);
            mma_commit_if(&stage_free[s], one);
            if (DOT && c + 1 < n) {  // after the rows' products, which the workers wait for in the same round
                if (!(ok = wait(sc_free, c & 1))) break;
                if (late && !(ok = wait(o_free, c & 1))) break;
                if (!(ok = scores(c + 1))) break;
            }
        }
        // every product issued above has completed before TMEM is released
        mma_commit_if(drain, one);
        const uint64_t begin = globaltimer();
        while (!mbar_try_sleep(drain, 0, 200000u))
            if (globaltimer() - begin > ctl.timeout_ns) break;
    } else if (warp < GT_W0) {
        // ------------------------------------------------------------ weights
        // Two warps take the chunks in turn: one alone needs 2,400 cycles a chunk, about what all the rest takes. Formed
        // and written a ring ahead of the tiles: place c % 8 was last read for chunk c - 8, and the tiles of chunk
        // c - 2 - NST are free, NST at most 4, so every reader has gone past chunk c - 7.
        const float *const gp = a.g + b * a.vg.b + h * a.vg.h;
        auto gate = [&](int c, int i) {  // log decay of row i of the sweep's chunk c; 0 behind the end
            const int t = t0 + chunk_of(c) * C + i;
            return c < nch && t < te ? gp[(long long)t * a.vg.l] : 0.f;
        };
        const int c0 = warp - 2;
        long long over = 0, whole_over = 0;  // the sum over this warp's chunks: units below a doubling, doublings
        bool cut = skip > 0;
        float g0 = gate(c0, 2 * lane), g1 = gate(c0, 2 * lane + 1);
        for (int c = c0; c < nch; c += 2) {
            const float n0 = gate(c + 2, 2 * lane), n1 = gate(c + 2, 2 * lane + 1);  // on its way meanwhile
            // sums of the rows 0 .. i in units of 2^-44 doublings; rows whose decay is 0 count as cuts
            // instead. (Sums in 64-bit floating point took 4,700 cycles a chunk, as long as all the rest.)
            const bool z0 = g0 < GATED_CUT, z1 = g1 < GATED_CUT;
            const bool odd = __any_sync(0xffffffffu, !(g0 < 88.f) || !(g1 < 88.f));  // NaN, or a decay past fp32
            const long long d0 = z0 || odd ? 0 : doublings(g0), d1 = z1 || odd ? 0 : doublings(g1);
            long long run = d0 + d1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += u;
            }
            const long long whole = __shfl_sync(0xffffffffu, run, 31);
            const uint32_t m0 = __ballot_sync(0xffffffffu, z0), m1 = __ballot_sync(0xffffffffu, z1);
            const uint32_t below = (1u << lane) - 1u;
            const int cuts = __popc(m0) + __popc(m1);
            const int r0 = __popc(m0 & (below | (1u << lane))) + __popc(m1 & below), r1 = r0 + (z1 ? 1 : 0);
            Weights &w = weights[c % GT_SLOTS];
            const float bad = odd ? __int_as_float(0x7fffffff) : 0.f;
            const float sign = rev ? -1.f : 1.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const long long G = i ? run : run - d1;
                const int id = i ? r1 : r0;
                // hi and lo together hold differences of rows to 2^-24 of what lies between two cuts
                const float g2 = (float)G * UNIT, rest = (float)(G - (long long)(float)G) * UNIT;
                const float cut = -GT_CUT * (float)id, hi = cut + g2, lo = (g2 - (hi - cut)) + rest;
                w.hi[2 * lane + i] = sign * hi + bad;
                w.lo[2 * lane + i] = sign * lo;
                const float start = id == 0 ? exp2f(g2) * fmaf(rest, 0.693147181f, 1.f) : 0.f;
                const float end = id == cuts ? exp2f((float)(whole - G) * UNIT) : 0.f;
                w.kw[2 * lane + i] = a.yscale * (rev ? start : end) + bad;
                w.rw[2 * lane + i] = a.oscale * (rev ? end : start) + bad;
            }
            over += whole;  // 64 bits of units hold 2^19 doublings, which a segment's rows may pass
            whole_over += over >> UNIT_BITS;
            over &= (1ll << UNIT_BITS) - 1;
            cut |= cuts > 0;
            if (lane == 0) {
                const float g2 = (float)whole * UNIT;
                w.a = (cuts ? 0.f : exp2f(g2)) + bad;
                w.em = (cuts ? -1.f : expm1f(g2 * 0.693147181f)) + bad;
            }
            g0 = n0;
            g1 = n1;
            const int s = c % NST;
            if (c >= NST && !wait(&stage_free[s], ((c / NST) - 1) & 1)) break;
            arrive(&full[s]);
        }
        if (lane == 0) {
            sums[c0] = over;
            doubled[c0] = whole_over;
            cuts_of[c0] = cut;
        }
    } else {
        // ------------------------------------------------------------ workers
        const int j = DZ == 128 ? 32 * q4 + lane : 16 * q4 + (lane & 15);  // z channel
        const bool live = DZ == 128 || lane < 16;
        constexpr int NX = DX / 4;  // x channels part * NX ..
        const long long n_state = (long long)DX * DZ;
        const long long at = (a.by_seg ? (long long)seg * BH + bh : (long long)slot * a.H + h) * n_state;
        Ch<2> S[NX / 2];
#pragma unroll
        for (int i = 0; i < NX / 2; ++i) S[i] = all<2>(0.f);
        auto place = [&](int i) { return (long long)(part * NX + i) * a.rs + (long long)j * a.cs; };
        if (a.init && !totals && live && (a.by_seg || slot >= 0)) {
            const float *p = a.init + at;
            if (a.rs == 1) {
#pragma unroll
                for (int i = 0; i < NX; i += 4) {
                    const float4 v = *(const float4 *)(p + place(i));
                    S[i / 2] = {{v.x, v.y}};
                    S[i / 2 + 1] = {{v.z, v.w}};
                }
            } else {
#pragma unroll
                for (int i = 0; i < NX; ++i) S[i / 2].v[i & 1] = p[place(i)];
            }
        }
        auto store = [&](float *p) {
            if (!live) return;
            if (a.rs == 1) {
#pragma unroll
                for (int i = 0; i < NX; i += 4)
                    *(float4 *)(p + place(i)) = make_float4(S[i / 2].v[0], S[i / 2].v[1], S[i / 2 + 1].v[0], S[i / 2 + 1].v[1]);
            } else {
#pragma unroll
                for (int i = 0; i < NX; ++i) p[place(i)] = S[i / 2].v[i & 1];
            }
        };
        // In a layout of their own, a warp's lanes next to one another: S and D are only multiplied element by element
        auto anchor = [&](int k) {
            float *const p = a.anchors + ((long long)k * BH + bh) * n_state + (long long)part * NX * DZ + j;
            if (live)
#pragma unroll
                for (int i = 0; i < NX; ++i) p[i * DZ] = S[i / 2].v[i & 1];
        };
        auto copy = [&](int c) {  // of the state before chunk c
#pragma unroll
            for (int i = 0; i < NX; i += 16) {
                uint32_t p[3][8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const Ch<2> &x = S[i / 2 + u];
                    if (NS == 1) p[0][u] = pack_bf16x2(x.v[0], x.v[1]);
                    else split3(x, p[0][u], p[1][u], p[2][u]);
                }
#pragma unroll
                for (int k = 0; k < NS; ++k)
                    tmem_st8(tmem + lanes + Lay::T_SC + (k + c % Lay::COPIES) * (DX / 2) + (part * NX + i) / 2, p[k]);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(s_ready);
        };
        const int first_anchor = a.anchors ? t0 / (a.anchor_chunks * C) : 0;
        const int anchors_here = a.anchors ? (t1 - t0 + a.anchor_chunks * C - 1) / (a.anchor_chunks * C) : 0;
        if (a.anchors && rev)  // those that end behind the sequence
            for (int k = (nch + a.anchor_chunks - 1) / a.anchor_chunks; k < anchors_here; ++k) anchor(first_anchor + k);
        if (!totals) copy(0);

        const int ft = 32 * (warp - GT_W0) + lane;
        constexpr int G = DX / 8, RG = 32 * GT_WORKERS / G, NR = C / RG;  // 16-byte pieces of a row; rows rg, rg + RG
        const int gi = ft % G, rg = ft / G, off = (gi >> 3) * C * 128 + (((gi & 7) ^ (rg & 7)) << 4) + rg * 128;
        const int ta = 16 * q4 + (lane >> 2), tb = ta + 8, col0 = 16 * part + 2 * cpos;
        const Ch<2> ps = all<2>(a.yscale * a.oscale), minus = all<2>(-1.f);
        if (rev ? part < q4 : part > q4)
            for (int k = 0; k < 2; ++k) {
                *(uint32_t *)(p_tile + ta * 128 + (((2 * part + k) ^ (ta & 7)) << 4) + 4 * cpos) = 0;
                *(uint32_t *)(p_tile + tb * 128 + (((2 * part + k) ^ (tb & 7)) << 4) + 4 * cpos) = 0;
            }
        auto form_y = [&](int c, uint8_t *y0, int y_step) {
            const int s = c % NST, row0 = t0 + chunk_of(c) * C, nv = min(C, te - row0);
            const Weights &w = weights[c % GT_SLOTS];
            const uint8_t *const src = tile_y(s) + off;
            uint8_t *const dst = y0 + off;
            uint4 v[NR];
#pragma unroll
            for (int m = 0; m < NR; ++m) v[m] = *(const uint4 *)(src + m * RG * 128);
#pragma unroll
            for (int m = 0; m < NR; ++m) {
                const int r = rg + m * RG;
                const Ch<2> kw = all<2>(w.kw[r]);
                uint32_t u[4] = {v[m].x, v[m].y, v[m].z, v[m].w}, hi[4], mid[4], lo[4];
                if (r >= nv) u[0] = u[1] = u[2] = u[3] = 0;  // behind the end: zeros, whatever is there
#pragma unroll
                for (int i = 0; i < 4; ++i) split3(mul(Ch<2>{{bf_lo(u[i]), bf_hi(u[i])}}, kw), hi[i], mid[i], lo[i]);
                uint8_t *const d = dst + m * RG * 128;
                *(uint4 *)d = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *(uint4 *)(d + y_step) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                *(uint4 *)(d + 2 * y_step) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            if (nv < C)
                for (int e = ft; e < (C - nv) * (DZ / 8); e += 32 * GT_WORKERS) {
                    const int r = nv + e / (DZ / 8), p = e % (DZ / 8);
                    *(uint4 *)(tile_z(s) + (p >> 3) * C * 128 + r * 128 + ((p & 7) << 4)) = make_uint4(0, 0, 0, 0);
                }
            fence_async_smem();
        };
        // The state over chunk c; next to 1 by the decay minus 1, whose rounding does not grow with the chunks.
        auto advance = [&](int c, uint32_t column, auto read) {
            uint32_t d[NX / 16][16];
#pragma unroll
            for (int i = 0; i < NX / 16; ++i) tmem_ld16(tmem + lanes + column + part * NX + 16 * i, d[i]);
            const Weights &w = weights[c % GT_SLOTS];
            const float da = w.a, em = w.em;
            forgets = da == 0.f;
            const bool near = da > 0.5f;
            const Ch<2> m = all<2>(near ? em : da), one = all<2>(near ? 1.f : 0.f);
            if (da == 0.f)  // forgets infinities and NaN too
#pragma unroll
                for (int i = 0; i < NX / 2; ++i) S[i] = all<2>(0.f);
            tmem_wait_ld();
            read();
#pragma unroll
            for (int i = 0; i < NX / 2; ++i) {
                const Ch<2> ds{{__uint_as_float(d[i / 8][2 * (i % 8)]), __uint_as_float(d[i / 8][2 * (i % 8) + 1])}};
                S[i] = fma(S[i], m, fma(S[i], one, ds));
            }
        };
        bool ok = true;
        if (!DOT && totals)
            for (int c = 0; c <= nch; ++c) {  // Y~ of one chunk, then the sum of the one before
                if (c < nch) {
                    if (!(ok = wait(&full[c % NST], (c / NST) & 1))) break;
                    if (c & 1) form_y(c, tile_x(0), Lay::STAGE);
                    else form_y(c, yt, Lay::X);
                    arrive(y_done[c & 1]);
                }
                if (c > 0) {
                    const int i = (c - 1) & 1;
                    if (!(ok = wait(ds_done[i], ((c - 1) >> 1) & 1))) break;
                    tc_fence_after();
                    advance(c - 1, i ? Lay::T_OI : Lay::T_DS, [&]() {
                        tc_fence_before();
                        arrive(ds_free[i]);
                    });
                }
            }
        for (int c = 0; !totals && c < nch; ++c) {
            const int s = c % NST, cc = chunk_of(c), row0 = t0 + cc * C, nv = min(C, te - row0);
            const Weights &w = weights[c % GT_SLOTS];
            if (a.anchors) {
                if (rev && (c == 0 || (cc + 1) % a.anchor_chunks == 0)) anchor(first_anchor + cc / a.anchor_chunks);
                if (!rev && cc % a.anchor_chunks == 0) anchor(first_anchor + cc / a.anchor_chunks);
            }
            // ---- Y~ (the one before has been read: dS of the chunk before was waited for)
            if (!(ok = wait(&full[s], (c / NST) & 1))) break;
            form_y(c, yt, Lay::X);
            arrive(yt_ready);
            // ---- the rows of the chunk before
            if (!DOT && c > 0) {
                if (!(ok = wait(o_done, (c - 1) & 1))) break;
                tc_fence_after();
                rows(c - 1);
            }
            // ---- P. Its one place has been read; with the intra product of the chunk before, this chunk's scores
            // are done too (not with DOT, whose issuer may take them up later).
            if ((DOT || c == 0) && !(ok = wait(scores_done, c & 1))) break;
            tc_fence_after();
            uint32_t r1[8], r2[8];
            tmem_ld16x256_x2(tmem + Lay::T_A + lanes + 16 * part, r1);
            if (INNER) tmem_ld16x256_x2(tmem + Lay::T_A2 + lanes + 16 * part, r2);
            // columns from <= col < to of a row count: up to the row itself, or in reverse from it on
            int from[2], to[2];
            Ch<2> ghi[2], glo[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = r ? tb : ta;
                from[r] = (rev ? row : 0) - col0;
                to[r] = (row >= nv ? 0 : rev ? nv : row + 1) - col0;
                ghi[r] = all<2>(w.hi[row]);
                glo[r] = all<2>(w.lo[row]);
            }
            float sum[2] = {0.f, 0.f}, sc[4] = {0.f, 0.f, 0.f, 0.f};
            tmem_wait_ld();
            tc_fence_before();
            arrive(sc_free);
            // (blocks behind the diagonal are 0: written once, before the loop)
            if (rev ? part >= q4 : part <= q4)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 h2 = *(const float2 *)&w.hi[col0 + 8 * k], l2 = *(const float2 *)&w.lo[col0 + 8 * k];
                const Ch<2> chi{{h2.x, h2.y}}, clo{{l2.x, l2.y}};
                uint32_t p[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int e = 4 * k + 2 * r;
                    const Ch<2> d = add(fma(chi, minus, ghi[r]), fma(clo, minus, glo[r])), wt{{ex2(d.v[0]), ex2(d.v[1])}};
                    Ch<2> x = mul(mul(Ch<2>{{__uint_as_float(r1[e]), __uint_as_float(r1[e + 1])}}, wt), ps);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const bool in = 8 * k + u >= from[r] && 8 * k + u < to[r];
                        if (INNER) {
                            const bool own = 8 * k + u == (r ? tb : ta) - col0;
                            const float y = in && !own ? x.v[u] * __uint_as_float(r2[e + u]) : 0.f;
                            sum[r] += y;
                            if (r == 0) sc[2 * k + u] = y;
                            else sc[2 * k + u] += y;
                        }
                        x.v[u] = in ? x.v[u] : 0.f;
                    }
                    p[r] = pack_bf16x2(x.v[0], x.v[1]);
                }
                const int ch = 2 * part + k;
                *(uint32_t *)(p_tile + ta * 128 + ((ch ^ (ta & 7)) << 4) + 4 * cpos) = p[0];
                *(uint32_t *)(p_tile + tb * 128 + ((ch ^ (tb & 7)) << 4) + 4 * cpos) = p[1];
            }
            fence_async_smem();
            arrive(p_ready);
            if (INNER) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
                    sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
                }
                float *const rp = a.dot + ((long long)(4 + part) * BH + bh) * a.L + row0;
                if (cpos == 0) {
                    if (ta < nv) rp[ta] = sum[0];
                    if (tb < nv) rp[tb] = sum[1];
                }
                int at_c = 0;
#pragma unroll
                for (int o = 4, n = 2; n > 0; o <<= 1, n >>= 1) {
                    const bool up = lane & o;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (i < n) {
                            const float send = up ? sc[i] : sc[i + n], keep = up ? sc[i + n] : sc[i];
                            sc[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                        }
                    at_c += up ? n : 0;
                }
                sc[0] += __shfl_xor_sync(0xffffffffu, sc[0], 16);
                const int col = col0 + 8 * (at_c >> 1) + (at_c & 1);
                if (!(lane & 16) && col < nv) a.dotc[((long long)q4 * BH + bh) * a.L + row0 + col] = sc[0];
            }
            // ---- the state
            if (!(ok = wait(state_done, c & 1))) break;
            tc_fence_after();
            advance(c, Lay::T_DS, []() {});
            if (DOT && !(ok = wait(inter_done, c & 1))) break;  // the copy has been read
            copy(c + 1);
            if (DOT) {
                if (!(ok = wait(o_done, c & 1))) break;
                tc_fence_after();
                rows(c);
                arrive(&w_free[c % Lay::WST]);
            }
        }
        if (!DOT && !totals && ok && nch > 0 && (ok = wait(o_done, (nch - 1) & 1))) {
            tc_fence_after();
            rows(nch - 1);
        }
        if (ok) {
            if (a.anchors && !rev) {
                for (int k = (nch + a.anchor_chunks - 1) / a.anchor_chunks; k < anchors_here; ++k) anchor(first_anchor + k);
                if (seg == a.nseg - 1) anchor(a.n_anchors);
            }
            if (a.fin && (a.by_seg || slot >= 0)) store(a.fin + at);
            // rows behind the sequence's end
            if (!totals && a.out)
                for (int t = te + (warp - GT_W0); t < t1; t += GT_WORKERS)
                    for (int i = lane; i < DZ; i += 32) {
                        const long long o = out0 + (long long)t * a.vo.l + i;
                        if (a.out_f32) ((float *)a.out)[o] = 0.f;
                        else ((__nv_bfloat16 *)a.out)[o] = __float2bfloat16_rn(0.f);
                    }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    if (tid == 0 && a.decay) {
        // past 2^17 doublings either way it is 0 or infinite all the same
        const long long over = min(max(doubled[0] + doubled[1], -(1ll << 17)), 1ll << 17);
        const long long units = (over << UNIT_BITS) + sums[0] + sums[1];
        a.decay[(long long)seg * BH + bh] = cuts_of[0] || cuts_of[1] ? 0.f : exp2f((float)units * UNIT);
    }
}

// ---- host side -----------------------------------------------------------------------------------
// [B, n, L, d] bf16 by strides; boxes of 64 channels x 64 rows of one head, 128-byte swizzle, rows past L
// zero.
bool map4(CUtensorMap *m, const void *ptr, const View &v, int B, int n, int L, int d)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)L, (cuuint64_t)n, (cuuint64_t)B};
    auto stride = [&](long long s, int len) { return (cuuint64_t)(len > 1 ? s * 2 : d * 2); };
    cuuint64_t strides[3] = {stride(v.l, L), stride(v.h, n), stride(v.b, B)};
    cuuint32_t box[4] = {64, GT_C, 1, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DX, int DZ, bool DOT, bool INNER> int launch_dims(const GtArgs &a, cudaStream_t stream)
{
    using Lay = GtLayout<DX, DZ, DOT>;
    static std::atomic<uint64_t> done{0};  // devices whose limit is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return LA_ERR_CUDA;
    if (dev >= 64 || !(done.load() >> dev & 1)) {
        const int rc = status_of(cudaFuncSetAttribute(gated_tc_kernel<DX, DZ, DOT, INNER>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::ALLOC));
        if (rc != LA_OK) return rc;
        if (dev < 64) done |= 1ull << dev;
    }
    return launch(gated_tc_kernel<DX, DZ, DOT, INNER>, dim3((unsigned)(a.B * a.H * a.nseg)), GT_THREADS, (size_t)Lay::ALLOC, stream, a);
}
template <bool DOT, bool INNER> int launch_dot(const GtArgs &a, int dx, int dz, cudaStream_t s)
{
    if (dx == 64) return dz == 64 ? launch_dims<64, 64, DOT, INNER>(a, s) : launch_dims<64, 128, DOT, INNER>(a, s);
    return dz == 64 ? launch_dims<128, 64, DOT, INNER>(a, s) : launch_dims<128, 128, DOT, INNER>(a, s);
}

struct Operand {
    const void *p = nullptr;
    View v = {};
    int n = 0, d = 0;  // heads, channels
};

struct Pass {
    Operand x, y, z, w;  // x.p NULL: totals; w.p NULL: no DOT
    bool inner = false;
    GtArgs a = {};
};

int launch_pass(const GatedArgs &p, Pass &s)
{
    GtArgs &a = s.a;
    a.B = p.B; a.H = p.H; a.L = p.L;
    a.g = p.g; a.vg = p.vg;
    a.lengths = p.lengths;
    a.err = p.err;
    a.totals = s.x.p == nullptr;
    a.timeout_ns = 2000000000ull;
    if (const char *e = getenv("LA_DEBUG_TIMEOUT_NS"); e && *e) a.timeout_ns = strtoull(e, nullptr, 10);
    a.sx = a.sw = 1;
    a.sy = p.H / s.y.n;
    a.sz = p.H / s.z.n;
    if (!map4(&a.my, s.y.p, s.y.v, p.B, s.y.n, p.L, s.y.d) || !map4(&a.mz, s.z.p, s.z.v, p.B, s.z.n, p.L, s.z.d)) return LA_ERR_CUDA;
    if (s.x.p) {
        a.sx = p.H / s.x.n;
        if (!map4(&a.mx, s.x.p, s.x.v, p.B, s.x.n, p.L, s.x.d)) return LA_ERR_CUDA;
    }
    if (!s.w.p) return launch_dot<false, false>(a, s.y.d, s.z.d, p.stream);
    a.sw = p.H / s.w.n;
    if (!map4(&a.mw, s.w.p, s.w.v, p.B, s.w.n, p.L, s.w.d)) return LA_ERR_CUDA;
    return s.inner ? launch_dot<true, true>(a, s.y.d, s.z.d, p.stream) : launch_dot<true, false>(a, s.y.d, s.z.d, p.stream);
}

bool tc_dim(int d) { return d == 64 || d == 128; }
bool tc_view(const void *p, const View &v, int B, int n, int L)
{
    auto ok = [&](long long s, int len) { return len == 1 || (s > 0 && s < (1ll << 38)); };
    return rows_aligned(p, v, B, n, L, 2, 16) && ok(v.b, B) && ok(v.h, n) && ok(v.l, L);
}

// Segments of a head's rows, one block each: where the heads alone leave half of the SMs idle or more, as many as
// run at once (two from a third to a half of the SMs), of 256 rows at least. The segments' sums are a pass over y and z,
// half of the sweep's bytes. More heads keep one each: further segments would wait for a second round of blocks.
int tc_segments(int BH, int L, int sms)
{
    const int want = std::min(sms / BH, (L + 255) / 256);
    return want < 2 ? 1 : want;
}
int chunk_rows(int L, int nseg) { return ((L + nseg - 1) / nseg + GT_C - 1) / GT_C * GT_C; }

struct TcBwdSpace {
    size_t T, A, U, S, D, y, r, c, dk, dv, all;
    int rows, nseg, anchor, n_anchors;
    TcBwdSpace(int B, int H, int Hk, int L, int d, int e, int sms)
    {
        const size_t heads = (size_t)B * H, n = (size_t)d * e;
        const int want = tc_segments(B * H, L, sms);
        rows = chunk_rows(L, want);
        // segments of more than one anchor are whole anchors
        if (want > 1 && rows > GATED_ANCHOR) rows = (rows + GATED_ANCHOR - 1) / GATED_ANCHOR * GATED_ANCHOR;
        nseg = (L + rows - 1) / rows;
        anchor = nseg > 1 && rows < GATED_ANCHOR ? rows : GATED_ANCHOR;
        n_anchors = (L + anchor - 1) / anchor;
        size_t at = 0;
        auto take = [&](size_t k) { const size_t o = at; at += (k + 3) & ~(size_t)3; return o; };
        T = take(nseg > 1 ? nseg * heads * n : 0);
        U = take(nseg > 1 ? nseg * heads * n : 0);
        A = take(nseg > 1 ? nseg * heads : 0);
        S = take((n_anchors + 1) * heads * n);
        D = take(n_anchors * heads * n);
        y = take(n_anchors * heads);
        r = take(8 * heads * L);
        c = take(8 * heads * L);
        dk = take(H > Hk ? heads * L * d : 0);
        dv = take(H > Hk ? heads * L * e : 0);
        all = at;
    }
};

}  // namespace

static bool inputs_ok(const GatedArgs &p)
{
    return p.dtype == LA_BF16 && tc_dim(p.d) && tc_dim(p.e) && tc_view(p.q, p.vq, p.B, p.H, p.L) &&
           tc_view(p.k, p.vk, p.B, p.Hk, p.L) && tc_view(p.v, p.vv, p.B, p.Hk, p.L);
}
bool gated_tc_fwd_ok(const GatedArgs &p) { return inputs_ok(p) && tc_view(p.out, p.vo, p.B, p.H, p.L); }
bool gated_tc_bwd_ok(const GatedArgs &p)
{
    return inputs_ok(p) && tc_view(p.dout, p.vo, p.B, p.H, p.L) && tc_view(p.dq, p.vdq, p.B, p.H, p.L) &&
           tc_view(p.dk, p.vdk, p.B, p.Hk, p.L) && tc_view(p.dv, p.vdv, p.B, p.Hk, p.L) &&
           aligned(p.state0, 16) && aligned(p.dstate, 16) && aligned(p.dstate0, 16);
}

size_t gated_tc_fwd_ws(int B, int H, int L, int d, int e, int sms)
{
    if (!tc_dim(d) || !tc_dim(e)) return 0;
    const int rows = chunk_rows(L, tc_segments(B * H, L, sms)), nseg = (L + rows - 1) / rows;
    return nseg == 1 ? 0 : sizeof(float) * (size_t)nseg * B * H * ((size_t)d * e + 1);
}
size_t gated_tc_bwd_ws(int B, int H, int Hk, int L, int d, int e, int sms)
{
    return tc_dim(d) && tc_dim(e) ? sizeof(float) * TcBwdSpace(B, H, Hk, L, d, e, sms).all : 0;
}

int gated_tc_fwd(const GatedArgs &p)
{
    const int rows = chunk_rows(p.L, tc_segments(p.B * p.H, p.L, p.sms)), nseg = (p.L + rows - 1) / rows, n = p.d * p.e;
    Pass s;
    s.y = {p.k, p.vk, p.Hk, p.d};
    s.z = {p.v, p.vv, p.Hk, p.e};
    s.a.seg_rows = rows; s.a.nseg = nseg;
    s.a.rs = p.e; s.a.cs = 1;
    s.a.yscale = 1.f; s.a.oscale = p.scale;
    int rc;
    if (nseg > 1) {
        float *T = p.ws, *A = T + (size_t)nseg * p.B * p.H * n;
        Pass t = s;
        t.a.by_seg = 1;
        t.a.fin = T;
        t.a.decay = A;
        if ((rc = launch_pass(p, t)) != LA_OK) return rc;
        if ((rc = gated_scan(p, T, A, nseg, n, p.state0, p.slots, p.state, nullptr, false)) != LA_OK) return rc;
        s.a.by_seg = 1;
        s.a.init = T;
    } else {
        s.a.slots = p.slots; s.a.n_slots = p.n_slots;
        s.a.init = p.state0;
        s.a.fin = p.state;
    }
    s.x = {p.q, p.vq, p.H, p.d};
    s.a.out = p.out; s.a.vo = p.vo;
    return launch_pass(p, s);
}

int gated_tc_bwd(const GatedArgs &p)
{
    const TcBwdSpace w(p.B, p.H, p.Hk, p.L, p.d, p.e, p.sms);
    const int n = p.d * p.e, group = p.H / p.Hk;
    const size_t heads = (size_t)p.B * p.H;
    float *const ws = p.ws;
    const bool dg = p.dg || p.dg_head;
    const Operand q{p.q, p.vq, p.H, p.d}, k{p.k, p.vk, p.Hk, p.d}, v{p.v, p.vv, p.Hk, p.e}, g{p.dout, p.vo, p.H, p.e};
    int rc;
    Pass base;
    base.a.seg_rows = w.rows; base.a.nseg = w.nseg;
    base.a.by_seg = w.nseg > 1;
    base.a.yscale = base.a.oscale = 1.f;
    base.a.anchor_chunks = w.anchor / GT_C; base.a.n_anchors = w.n_anchors;
    if (w.nseg > 1) {
        Pass s = base;  // states at the segments' starts
        s.y = k; s.z = v;
        s.a.rs = p.e; s.a.cs = 1;
        s.a.fin = ws + w.T; s.a.decay = ws + w.A;
        if ((rc = launch_pass(p, s)) != LA_OK) return rc;
        if ((rc = gated_scan(p, ws + w.T, ws + w.A, w.nseg, n, p.state0, nullptr, nullptr, nullptr, false)) != LA_OK) return rc;
        s = base;  // the states' gradients at their ends
        s.y = q; s.z = g;
        s.a.reverse = 1;
        s.a.rs = p.e; s.a.cs = 1;
        s.a.yscale = p.scale;
        s.a.fin = ws + w.U;
        if ((rc = launch_pass(p, s)) != LA_OK) return rc;
        if ((rc = gated_scan(p, ws + w.U, ws + w.A, w.nseg, n, p.dstate, nullptr, p.dstate0, nullptr, true)) != LA_OK) return rc;
    }
    Pass s = base;  // dq = S dout
    s.x = g; s.y = v; s.z = k;
    s.a.rs = 1; s.a.cs = p.e;
    s.a.init = w.nseg > 1 ? ws + w.T : p.state0;
    s.a.oscale = p.scale;
    s.a.out = p.dq; s.a.vo = p.vdq;
    if (dg) {
        s.w = q;
        s.inner = true;
        s.a.dot = ws + w.r; s.a.dotc = ws + w.c + 4 * heads * p.L;
        s.a.anchors = ws + w.S;
    }
    if ((rc = launch_pass(p, s)) != LA_OK) return rc;
    auto per_head = [&](int c) { return View{(long long)p.H * p.L * c, (long long)p.L * c, c}; };
    s = base;  // dk = D v
    s.x = v; s.y = g; s.z = q;
    s.a.reverse = 1;
    s.a.rs = 1; s.a.cs = p.e;
    s.a.init = w.nseg > 1 ? ws + w.U : p.dstate;
    s.a.yscale = p.scale;
    s.a.out = p.dk; s.a.vo = p.vdk;
    if (group > 1) {
        s.a.out = ws + w.dk; s.a.vo = per_head(p.d); s.a.out_f32 = 1;
    }
    if (dg) {
        s.w = k;
        s.a.dot = ws + w.c;
        s.a.anchors = ws + w.D;
    }
    if ((rc = launch_pass(p, s)) != LA_OK) return rc;
    s = base;  // dv = D^T k
    s.x = k; s.y = q; s.z = g;
    s.a.reverse = 1;
    s.a.rs = p.e; s.a.cs = 1;
    s.a.init = w.nseg > 1 ? ws + w.U : p.dstate;
    if (w.nseg == 1) s.a.fin = p.dstate0;  // the last reader of dstate
    s.a.yscale = p.scale;
    s.a.out = p.dv; s.a.vo = p.vdv;
    if (group > 1) {
        s.a.out = ws + w.dv; s.a.vo = per_head(p.e); s.a.out_f32 = 1;
    }
    if ((rc = launch_pass(p, s)) != LA_OK) return rc;
    if (group > 1) {
        if ((rc = gated_share(p, ws + w.dk, p.dk, p.vdk, p.d)) != LA_OK) return rc;
        if ((rc = gated_share(p, ws + w.dv, p.dv, p.vdv, p.e)) != LA_OK) return rc;
    }
    if (dg) {
        if ((rc = gated_products(p, ws + w.D, ws + w.S + heads * n, ws + w.y, w.n_anchors, n)) != LA_OK) return rc;
        if ((rc = gated_log_decay(p, ws + w.r, 8, ws + w.c, 8, ws + w.y, w.anchor, w.n_anchors)) != LA_OK)
            return rc;
    }
    return LA_OK;
}

}  // namespace la
