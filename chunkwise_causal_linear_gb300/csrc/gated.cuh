// gated.cuh -- what the two paths of the gated attention share: the problem as the entry points
// check it, where a sequence's state lies, and the launches.
#pragma once

#include "layer.cuh"

namespace la {

// Rows between two points at which the backward pass knows both the state and its gradient, and so
// the decays' gradient without the sums behind them.
constexpr int GATED_ANCHOR = 1024;

// A log decay below this counts as -inf: exp of it is 0 in fp32.
constexpr float GATED_CUT = -104.f;

struct GatedArgs {
    const void *q, *k, *v, *dout;
    void *out, *dq, *dk, *dv;
    const float *g, *state0, *dstate;
    float *state, *dg, *dg_head, *dstate0;
    const int *slots, *lengths;
    View vq, vk, vv, vg, vo, vdq, vdk, vdv;  // vo: out, or dout in the backward pass
    int B, H, Hk, L, d, e, n_slots;          // d: channels of q and k, e: of v
    float scale;
    int dtype;
    float *ws;
    int *err;
    cudaStream_t stream;
    int sms;
};

// Entry of sequence b's state in its array; -1 where it has none.  A slot past the pool counts as none
// and is reported.
__device__ __forceinline__ int gated_slot(const int *slots, int b, int n_slots, int *err)
{
    if (!slots) return b;
    const int s = slots[b];
    if (s >= n_slots) {
        record_error(err, LA_ERR_DEVICE);
        return -1;
    }
    return s < 0 ? -1 : s;
}

__device__ __forceinline__ int gated_rows(const int *lengths, int b, int L)
{
    return lengths ? min(max(lengths[b], 0), L) : L;
}

// States at the starts of the segments out of the segments' sums: T [nseg][heads][n] holds the sums
// and becomes the states, A [nseg][heads] the decays over the segments.
int gated_scan(const GatedArgs &p, float *T, const float *A, int nseg, int n, const float *first, const int *slots,
               float *last, float *last_ws, bool reverse);
// dk, dv of shared key heads: x [B][H][L][n] fp32, summed over the heads of each key head.
int gated_share(const GatedArgs &p, const float *x, void *out, const View &vo, int n);
// dg out of the rows' parts: r and c [parts][heads][L], the anchors' products y [nseg][heads], rows of
// a segment; then its sums over the rows of each head, where they are wanted.
int gated_log_decay(const GatedArgs &p, const float *r, int nr, const float *c, int nc, float *y, int seg_rows,
                    int nseg);
int gated_products(const GatedArgs &p, const float *D, const float *S, float *y, int nseg, int n);

size_t gated_simt_fwd_ws(int B, int H, int L, int d, int e, int sms);
size_t gated_simt_bwd_ws(int B, int H, int Hk, int L, int d, int e, int sms);
int gated_simt_fwd(const GatedArgs &p);
int gated_simt_bwd(const GatedArgs &p);

// The tensor cores' path: bf16, 64 or 128 channels, rows of 16-byte alignment, no broadcast.
bool gated_tc_fwd_ok(const GatedArgs &p);
bool gated_tc_bwd_ok(const GatedArgs &p);
size_t gated_tc_fwd_ws(int B, int H, int L, int d, int e, int sms);
size_t gated_tc_bwd_ws(int B, int H, int Hk, int L, int d, int e, int sms);
int gated_tc_fwd(const GatedArgs &p);
int gated_tc_bwd(const GatedArgs &p);

}  // namespace la
