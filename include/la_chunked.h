/*
 * la_chunked.h -- C ABI of the chunkwise-parallel causal linear attention forward pass
 * (GB300, sm_103a).  Library: chunkwise_causal_linear_gb300/liblachunked.so.
 *
 * What is computed (per (b, h) head, rows t = 0..L-1, phi applied row-wise):
 *
 *     num_t = sum_{s <= t} M[t,s] (phi(q_t) . phi(k_s)) v_s
 *     den_t = sum_{s <= t} M[t,s] (phi(q_t) . phi(k_s))
 *     out_t = normalize ? num_t / den_t : num_t
 *
 * with M[t,s] = 1 (causal linear attention), or M[t,s] = lambda_t^(l(t,s)),
 * l = 0 if s == t else 1 + floor(log2(t XOR s)) (Fenwick-level log-linear mask).
 *
 * Sources:
 *   "attention と線形の間" (sharin-2a1.pages.dev, parts/chunked.html), section 2:
 *       Chunked(q, k, v, c) -- chunks of c rows; inside a chunk the causally masked
 *       scores (diagonal kept), across chunks a d_k x d_v state carried forward;
 *       c <= 0 means 1; a partial last chunk is allowed.  Section 3: Shape cost model.
 *   "Linear Attention / Performerの理論と実装" (disassemble-channel.com): the ELU
 *       feature map, FAVOR+ positive random features, the normalised output y_t and the
 *       (S_t, z_t) recurrence.
 *   "論文紹介：Log Linear Attention" (docswell slides): Fenwick buckets (slides 15-21),
 *       level weights lambda (slide 17), chunkwise level-0 block plus per-level
 *       inter-chunk states (slides 34-35).
 *
 * Conventions for every entry point:
 *   - Layout: q, k [B, H, L, dk]; v, out [B, H, L, dv]; contiguous row-major.
 *   - All tensor pointers are DEVICE pointers unless the name says _host.  The caller
 *     owns every buffer; the library allocates no device memory.
 *   - Calls are asynchronous on `stream` (a cudaStream_t passed as void*; NULL = the
 *     legacy default stream) and return after the launches are queued.
 *   - Host-detectable errors return a negative la_status before anything is launched.
 *     Errors found on the device (a bounded wait that timed out, an index check) are
 *     recorded in a device error word that la_last_device_status() reads.
 *   - Concurrent calls on different streams are safe if they use different workspaces
 *     (the device error word is shared by all calls).
 */
#ifndef LA_CHUNKED_H
#define LA_CHUNKED_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------------------- */
enum la_status {
    LA_OK = 0,
    LA_ERR_NULL = -1,        /* a required pointer is NULL                               */
    LA_ERR_SHAPE = -2,       /* a dimension is <= 0, or sizes overflow                   */
    LA_ERR_UNSUPPORTED = -3, /* combination not supported (dtype, dims, feature map, C)  */
    LA_ERR_WORKSPACE = -4,   /* workspace missing or smaller than la_chunked_workspace_bytes */
    LA_ERR_CUDA = -5,        /* a CUDA runtime call failed (launch, copy, attribute)      */
    LA_ERR_TIMEOUT = -6,     /* device: a bounded wait gave up (read via la_last_device_status) */
    LA_ERR_DEVICE = -7,      /* device: an index or shape check failed inside a kernel    */
    LA_ERR_SCRATCH_LIMIT = -8, /* la_chunked_fwd_noalloc: the problem needs more scratch than
                                  its fixed buffer holds (8 MiB)                          */
    LA_ERR_ARG = -9            /* an argument value is out of range (gamma, eps, strides)  */
};

/* ---- feature maps phi -------------------------------------------------------------- */
enum la_fm_kind {
    LA_FM_IDENTITY = 0, /* phi(x) = x                                                     */
    LA_FM_ELU1 = 1,     /* phi(x) = elu(x) + 1 = (x >= 0 ? x + 1 : e^x)                   */
    LA_FM_FAVOR = 2     /* FAVOR+: x^ = x / dk^(1/4); phi(x) = exp(omega x^ - |x^|^2/2)/sqrt(m) */
};

typedef struct la_feature_map {
    int kind;            /* enum la_fm_kind                                              */
    int m;               /* FAVOR+: number of random features (the feature dimension);
                            other kinds: ignored (the feature dimension is dk)            */
    const float *omega;  /* FAVOR+: device [m, dk] fp32 row-major random matrix, owned by
                            the caller and read during the call; other kinds: ignored     */
} la_feature_map;

/* ---- storage dtypes of q, k, v, out ---------------------------------------------- */
enum la_dtype {
    LA_BF16 = 0,  /* bfloat16 storage; arithmetic in fp32 with bf16 tensor-core operands  */
    LA_F32 = 1    /* fp32 storage; arithmetic in fp32 (exact on small-integer inputs)     */
};

/* ---- execution paths ---------------------------------------------------------------- */
enum la_path {
    LA_PATH_AUTO = 0,    /* the library picks (see la_chunked_plan)                       */
    LA_PATH_SIMT = 1,    /* generic fp32 CUDA-core path: any C, any supported dims         */
    LA_PATH_TC = 2       /* tcgen05/TMEM tensor-core single-pass path (subset of shapes)   */
};

/*
 * la_chunked_fwd -- the forward pass.
 *
 *   q, k          device [B, H, L, dk], dtype `dtype`
 *   v             device [B, H, L, dv], dtype `dtype`
 *   out           device [B, H, L, dv], dtype `dtype`; fully overwritten
 *   C             chunk size: C <= 0 means 1, C >= L means one chunk ("attention and
 *                 linear order meet at the two ends", chunked page section 2)
 *   feature_map   NULL means identity
 *   normalize     0: out = num; 1: out = num / den
 *   level_weights NULL, or device [B, H, L, num_levels] fp32 lambda_t^(l) (log-linear).
 *                 num_levels must cover 1 + ceil(log2 L) levels, and with more than one
 *                 chunk C must be a power of two (chunk edges are then Fenwick edges).
 *   workspace     device scratch of at least la_chunked_workspace_bytes(...) bytes (may
 *                 be NULL when that is 0); contents on entry are ignored.
 *   stream        cudaStream_t as void*.
 * Returns LA_OK or a negative la_status (nothing launched on error).
 */
int la_chunked_fwd(const void *q, const void *k, const void *v, void *out,
                   int B, int H, int L, int dk, int dv, int C,
                   const la_feature_map *feature_map, int normalize,
                   const float *level_weights, int num_levels,
                   int dtype, void *workspace, size_t workspace_bytes, void *stream);

/* As la_chunked_fwd, with an explicit execution path (enum la_path).  LA_PATH_TC returns
 * LA_ERR_UNSUPPORTED for shapes the tensor-core path does not cover.  It covers bf16
 * storage, L >= 128, and:
 *   - identity / elu+1 features, with or without the normaliser, dk = D, (dk, dv) in
 *     {(64, 64), (64, 128), (128, 128)}, C in {16, 32, 64, 128, 256};
 *   - FAVOR+ features, dk = 64, m = 256, dv = 64, C = 64, with or without the normaliser;
 *   - the log-linear mask: identity features, no normaliser, dk = dv = 64, C = 64, at most
 *     4096 chunks, num_levels <= 32, L * num_levels a multiple of 4 and level_weights
 *     16-byte aligned (LA_PATH_AUTO falls back to LA_PATH_SIMT when it is not).
 * Few-head problems are split along the sequence into segments; their plan reports two
 * launches and a workspace for the segment totals. */
int la_chunked_fwd_path(const void *q, const void *k, const void *v, void *out,
                        int B, int H, int L, int dk, int dv, int C,
                        const la_feature_map *feature_map, int normalize,
                        const float *level_weights, int num_levels,
                        int dtype, void *workspace, size_t workspace_bytes, void *stream,
                        int path);

/*
 * la_chunked_fwd_host -- the same forward pass from HOST buffers: copies q, k, v (and
 * nothing else: omega and level_weights stay device pointers) from host memory into the
 * caller's device buffers q_dev, k_dev, v_dev, runs la_chunked_fwd on them into out_dev,
 * copies out_dev back into out_host.  Host buffers should be pinned (cudaHostAlloc /
 * page-locked) for the copies to be asynchronous; the host buffers must stay valid until
 * the stream reaches the end of the call.  Sizes and error behaviour as la_chunked_fwd.
 * When the plan is one unsplit launch and the step moves at least 64 MB, the call runs as a
 * pipeline over up to 8 groups of heads: copies in on one internal stream, the groups'
 * launches on `stream`, copies out on another internal stream, so the two copy directions
 * and the compute overlap.  Each head's arithmetic is that of la_chunked_fwd (identical
 * outputs).  Either way the work is ordered after what `stream` already holds, and `stream`
 * reaches the end of the call only after every copy.
 */
int la_chunked_fwd_host(const void *q_host, const void *k_host, const void *v_host,
                        void *out_host, void *q_dev, void *k_dev, void *v_dev, void *out_dev,
                        int B, int H, int L, int dk, int dv, int C,
                        const la_feature_map *feature_map, int normalize,
                        const float *level_weights, int num_levels,
                        int dtype, void *workspace, size_t workspace_bytes, void *stream);

/*
 * la_chunked_fwd_noalloc -- the same forward pass, for callers that cannot allocate device
 * memory (code running inside an allocator or a memory-pool callback, plugins whose host
 * application owns every device allocation, real-time loops that must never call
 * cudaMalloc / cudaFree).  No counterpart on the pages: it is a deployment variant.
 *
 * It allocates nothing.  Every problem whose la_chunked_workspace_bytes is nonzero takes
 * that scratch from a fixed 8 MiB array compiled into the library: the segment totals of a
 * sequence cut into segments (few heads, on the tensor-core paths), and the log-linear
 * mask's per-level chunk states.  Every GPU that loads the library holds those 8 MiB until
 * the process exits.  Problems that need more return LA_ERR_SCRATCH_LIMIT before anything
 * is launched (la_chunked_workspace_bytes tells how much a problem needs).
 *   - The first call on each device looks up the array's device address (with that device
 *     current); make that first call before any stream capture.  The address is kept for
 *     the life of the process: calls after cudaDeviceReset of that device are not
 *     supported.
 *   - All calls share the one array and it keeps the last call's contents; the kernel
 *     clears what it needs at the start of every call.  Calls that may overlap on the GPU
 *     (different streams, or different host threads) race on it: serialise them.
 * Arguments, layout and the other errors are those of la_chunked_fwd (no workspace).
 */
int la_chunked_fwd_noalloc(const void *q, const void *k, const void *v, void *out,
                           int B, int H, int L, int dk, int dv, int C,
                           const la_feature_map *feature_map, int normalize,
                           const float *level_weights, int num_levels,
                           int dtype, void *stream);

/* Bytes of device workspace la_chunked_fwd needs for this problem on the current device
 * (0 when none).  Returns 0 also for invalid arguments (la_chunked_fwd reports those). */
size_t la_chunked_workspace_bytes(int B, int H, int L, int dk, int dv, int C,
                                  const la_feature_map *feature_map, int normalize,
                                  int num_levels, int dtype);

/* ---- plan introspection (host only; no device call when num_sms > 0) --------------- */
typedef struct la_plan_info {
    int path;              /* enum la_path actually chosen                               */
    int chunk;             /* effective chunk size after clamping                         */
    int n_chunks;          /* ceil(L / chunk)                                             */
    int feature_dim;       /* D: dk, or m for FAVOR+                                      */
    int grid_x, grid_y;    /* main kernel grid                                            */
    int block;             /* threads per CTA of the main kernel                          */
    int smem_bytes;        /* dynamic shared memory per CTA of the main kernel            */
    int n_launches;        /* kernel launches per call                                    */
    size_t workspace_bytes;
} la_plan_info;

/* Fills *info with the plan for the problem as la_chunked_fwd_path(path) would run it.
 * num_sms: SM count to plan for (0 = query the current device).  Returns LA_OK or the
 * status la_chunked_fwd_path would return for these arguments (pointers are not
 * checked). */
int la_chunked_plan(int B, int H, int L, int dk, int dv, int C,
                    const la_feature_map *feature_map, int normalize, int loglinear,
                    int num_levels, int dtype, int path, int num_sms, la_plan_info *info);

/* Waits for `stream`, then returns and clears the device error word: LA_OK, or the
 * first device-side error (LA_ERR_TIMEOUT, LA_ERR_DEVICE) recorded since the last call,
 * or LA_ERR_CUDA if the stream itself reports an error. */
int la_last_device_status(void *stream);

/* Static description of a status code (never NULL). */
const char *la_status_string(int status);

/*
 * la_cost_model -- "attention と線形の間", section 3, Shape{L, D, C}: multiply-add counts
 * of the chunked order.  *state_macs = 2 L D^2 (writing and reading the D x D state, the
 * same for every C); *score_macs = 2 L C D (making the in-chunk scores and mixing the
 * values, proportional to C).  Either output pointer may be NULL.  Returns LA_OK, or
 * LA_ERR_SHAPE for negative sizes.
 */
int la_cost_model(long long L, long long D, long long C, long long *state_macs,
                  long long *score_macs);

/*
 * la_decode_step -- one step of the recurrent (decoding) form for every (b, h) head, the
 * inference counterpart of the chunked state ("Linear Attention / Performerの理論と実装",
 * "再帰的な状態更新"; "論文紹介：Log Linear Attention", slides 17-22 for the level weights).
 *
 *   q, k          device [B, H, dk] (this token), dtype `dtype`
 *   v, out        device [B, H, dv], dtype `dtype`; out is overwritten
 *   state         device fp32, read and updated in place.  Without level weights:
 *                 [B, H, D, dv] = S, the sum of phi(k_s) v_s^T over the tokens so far.
 *                 With level weights: [B, H, num_levels - 1, D, dv], the Fenwick level
 *                 states S^(1), S^(2), ... (zeros before the first token).
 *   zstate        device fp32 normaliser, [B, H, D] or [B, H, num_levels - 1, D]; may be
 *                 NULL when normalize is 0.  Updated in place like `state`.
 *   level_weights NULL, or device [B, H, num_levels] fp32 lambda_t^(l) of this token.
 *   t             this token's position (0-based); used by the level update only.
 * D is dk, or m for FAVOR+.  Plain: state += phi(k) v^T, z += phi(k), then
 * out = phi(q)^T state (/ phi(q)^T z).  Level weights: out = lambda^(0) (phi(q).phi(k)) v +
 * sum_{l>=1} lambda^(l) phi(q)^T S^(l) from the states before the update; then, with r =
 * trailing zeros of t+1, S^(r+1) = phi(k) v^T + sum_{l<=r} S^(l) and S^(1..r) = 0.  Stepping
 * t = 0..L-1 reproduces la_chunked_fwd's rows (the same function of the sequence).
 * Returns LA_OK, LA_ERR_NULL, LA_ERR_SHAPE (sizes, or num_levels too small for position
 * t+1: the update needs num_levels >= 2 + trailing zeros of t+1, one more level than the
 * forward pass over positions 0..t uses), LA_ERR_UNSUPPORTED, LA_ERR_CUDA.  Asynchronous on `stream`; the caller owns every
 * buffer and must not run two steps of the same state concurrently.
 */
int la_decode_step(const void *q, const void *k, const void *v, void *out, float *state,
                   float *zstate, int B, int H, int dk, int dv,
                   const la_feature_map *feature_map, int normalize,
                   const float *level_weights, int num_levels, long long t, int dtype,
                   void *stream);

/* Number of fp32 elements of la_decode_step's state and zstate for these sizes (0 on an
 * invalid combination).  num_levels = 0 means no level weights. */
long long la_decode_state_elems(int B, int H, int dk, int dv, const la_feature_map *feature_map,
                                int num_levels, long long *z_elems);

/*
 * la_noncausal_fwd -- bidirectional (non-causal) linear attention: every query sees every
 * key ("Linear Attention / Performerの理論と実装", the non-causal normalised form, and the
 * Performer's bidirectional FAVOR+ attention; "attention と線形の間" section 1, StateFirst):
 *     S = sum_s phi(k_s) v_s^T,  z = sum_s phi(k_s),  out_t = phi(q_t)^T S (/ phi(q_t)^T z).
 * Arguments as la_chunked_fwd (no chunk size, no level weights: the mask is all ones).
 * D (dk, or m for FAVOR+) must be at most 256.  The workspace holds the per-head state:
 * at least la_noncausal_workspace_bytes(...) bytes.  Returns LA_OK or a negative status
 * before any launch.
 */
int la_noncausal_fwd(const void *q, const void *k, const void *v, void *out, int B, int H, int L,
                     int dk, int dv, const la_feature_map *feature_map, int normalize, int dtype,
                     void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes la_noncausal_fwd needs (0 on an invalid or unsupported combination). */
size_t la_noncausal_workspace_bytes(int B, int H, int L, int dk, int dv,
                                    const la_feature_map *feature_map, int normalize, int dtype);

/*
 * la_decay_fwd -- causal linear attention with the Retention decay ("Linear Attention /
 * Performerの理論と実装", the section on the RNN without forgetting):
 *     S_t = gamma S_{t-1} + phi(k_t) v_t^T,        out_t = phi(q_t)^T S_t,
 * i.e. out_t = sum_{s<=t} gamma^(t-s) (phi(q_t).phi(k_s)) v_s.  With normalize the
 * normaliser decays alike, z_t = gamma z_{t-1} + phi(k_t), and out_t = phi(q_t)^T S_t /
 * phi(q_t)^T z_t (a weighted mean of the values; the page gives the update of S only).
 *   gamma   0 < gamma <= 1, one value for every head; gamma = 1 is la_chunked_fwd's result.
 *           Outside that range (or NaN): LA_ERR_ARG.
 *   path    enum la_path.  LA_PATH_TC covers bf16, identity / elu+1 features, dk = D,
 *           (dk, dv) in {(64, 64), (64, 128), (128, 128)}, C = 64, L >= 128 and
 *           gamma >= 0.5 (gamma^64 >= 2^-64); LA_PATH_AUTO takes it there and the generic
 *           fp32 path elsewhere (any C, dtype, feature map).
 * Other arguments, layouts and errors as la_chunked_fwd (no level weights).  The workspace
 * must hold la_decay_workspace_bytes(...) bytes (the few-head sequence split's totals).
 */
int la_decay_fwd(const void *q, const void *k, const void *v, void *out, int B, int H, int L,
                 int dk, int dv, int C, const la_feature_map *feature_map, int normalize,
                 float gamma, int dtype, void *workspace, size_t workspace_bytes, void *stream,
                 int path);

/* la_decode_step with the Retention decay: state = gamma state + phi(k) v^T, zstate =
 * gamma zstate + phi(k), then out = phi(q)^T state (/ phi(q)^T zstate).  Stepping t =
 * 0..L-1 from zero state reproduces la_decay_fwd's rows.  Buffers as la_decode_step without
 * level weights ([B, H, D, dv] and [B, H, D] fp32).  gamma as la_decay_fwd (LA_ERR_ARG
 * outside 0 < gamma <= 1). */
int la_decay_decode_step(const void *q, const void *k, const void *v, void *out, float *state,
                         float *zstate, int B, int H, int dk, int dv,
                         const la_feature_map *feature_map, int normalize, float gamma,
                         int dtype, void *stream);

/* Workspace bytes la_decay_fwd needs (0 when none, or on invalid arguments). */
size_t la_decay_workspace_bytes(int B, int H, int L, int dk, int dv, int C,
                                const la_feature_map *feature_map, int normalize, float gamma,
                                int dtype);

/* la_chunked_plan for la_decay_fwd: the plan la_decay_fwd(path) would run. */
int la_decay_plan(int B, int H, int L, int dk, int dv, int C, const la_feature_map *feature_map,
                  int normalize, float gamma, int dtype, int path, int num_sms, la_plan_info *info);

/*
 * la_chunked_bwd -- backward pass of the causal forward (la_chunked_fwd without level
 * weights, or la_decay_fwd): given dout = dL/dout, writes dq, dk, dv.  The pages give no
 * backward formulas; these follow from the chain rule on the causal definition (mask 1 or
 * gamma^(t-s), with or without the normaliser), then through the feature map.  They are
 * linear-attention passes with the roles swapped, two of them anti-causal:
 *   - LA_PATH_TC: bf16, L >= 128, 16-byte aligned q, k, v, dout and gradient buffers, and
 *     either identity / elu+1 features with (dk, dv) in {(64, 64), (128, 128)}, no decay or
 *     gamma >= 0.5 without the normaliser (the same gamma^|t-s| mask in every pass), or
 *     FAVOR+ with dk = dv = 64, m in {128, 256, 512} and no decay.  Every pass runs on the
 *     tensor-core forward with identity features (the anti-causal ones in its anti-causal
 *     mode, in place; FAVOR+ once per 128 features); the normaliser adds three passes and
 *     its feature-gradient passes keep fp32 rows;
 *   - LA_PATH_SIMT: every supported case, in fp32 on the generic kernel;
 *   - LA_PATH_AUTO picks the first that applies.
 *   q, k, v, dout   device, as la_chunked_fwd's q, k, v and out ([B, H, L, d], dtype).
 *                   The forward output is not an input: with the normaliser, dq is a small
 *                   difference of two large sums, so the pass recomputes the output in fp32
 *                   (a bf16-stored one would carry its rounding into dq about thirtyfold).
 *   grad_q, grad_k, grad_v  device outputs dq, dk, dv: same shapes and dtype as q, k, v;
 *                   fully overwritten
 *   gamma           1 for the plain mask, else the decay (0 < gamma < 1; LA_ERR_ARG outside)
 *   C               chunk size of the generic path's passes (any value; the result does
 *                   not depend on it beyond rounding); the tensor-core passes use 64
 *   workspace       at least la_chunked_bwd_workspace_bytes(...) bytes (intermediates:
 *                   about 4 (D + dv) floats per row on the generic route, at most about
 *                   6 (D + dv) on the tensor-core route, none there for identity features
 *                   without the normaliser)
 * D (dk, or m for FAVOR+) and dk must be at most 512 and dv below 512.  Returns LA_OK or a
 * negative status before any launch.
 */
int la_chunked_bwd(const void *q, const void *k, const void *v, const void *dout,
                   void *grad_q, void *grad_k, void *grad_v, int B, int H,
                   int L, int dk, int dv, int C, const la_feature_map *feature_map,
                   int normalize, float gamma, int dtype, void *workspace,
                   size_t workspace_bytes, void *stream, int path);

/* Workspace bytes la_chunked_bwd needs (0 on an invalid or unsupported combination). */
size_t la_chunked_bwd_workspace_bytes(int B, int H, int L, int dk, int dv, int C,
                                      const la_feature_map *feature_map, int normalize,
                                      int dtype);

/*
 * la_chunked_bwd_ll -- backward pass of the causal forward under the log-linear mask
 * (la_chunked_fwd with level_weights; "論文紹介：Log Linear Attention", slide 17, mask
 * M_ts = lambda_t^(l(t,s))): given dout, writes dq, dk, dv.  The level weights are treated as
 * data: their own gradient is not formed.  By the chain rule, with G_ts = M_ts (dout_t . v_s)
 * (normalised: M_ts (dout_t . v_s - dout_t . out_t) / den_t):
 *   dphi(q)_t = sum_{s<=t} G_ts phi(k_s)    -- a causal log-linear pass with the roles swapped;
 *   dphi(k)_s = sum_{t>=s} G_ts phi(q_t),   dv_s = sum_{t>=s} M_ts (phi(q_t).phi(k_s)) dout_t
 *                                            (/ den_t) -- anti-causal sums in which each pair is
 *                                            weighted by the LATER row's lambda; they are grouped
 *                                            by the aligned dyadic blocks of the level rule, one
 *                                            weighted state per block,
 * then through the feature map.  Generic fp32 route (path LA_PATH_AUTO or LA_PATH_SIMT;
 * LA_PATH_TC returns LA_ERR_UNSUPPORTED), any feature map, with or without the normaliser.
 *   level_weights  device [B, H, L, num_levels] fp32, as la_chunked_fwd's (1 + ceil(log2 L)
 *                  levels at least)
 *   C              ignored beyond la_chunked_fwd's checks (the passes use 64-row chunks)
 *   workspace      at least la_chunked_bwd_ll_workspace_bytes(...) bytes (fp32 rows of about
 *                  4 (D + dv) floats per row, level states, and one D x dv state per aligned
 *                  block of chunks per head)
 * Other arguments and errors as la_chunked_bwd (no decay).
 */
int la_chunked_bwd_ll(const void *q, const void *k, const void *v, const void *dout,
                      void *grad_q, void *grad_k, void *grad_v, int B, int H, int L, int dk,
                      int dv, int C, const la_feature_map *feature_map, int normalize,
                      const float *level_weights, int num_levels, int dtype, void *workspace,
                      size_t workspace_bytes, void *stream, int path);

/* Workspace bytes la_chunked_bwd_ll needs (0 on an invalid or unsupported combination). */
size_t la_chunked_bwd_ll_workspace_bytes(int B, int H, int L, int dk, int dv, int C,
                                         const la_feature_map *feature_map, int normalize,
                                         int num_levels, int dtype);

/*
 * Carried state.  The state a causal pass ends with seeds a decoding loop (prefill, then
 * la_decode_step / la_decay_decode_step) or the next segment of a sequence cut into
 * segments (one per stream, thread or rank): each segment's own final state T_r, an
 * exclusive prefix P_r = gamma^len_{r-1} P_{r-1} + T_{r-1} over the earlier segments (the
 * "attention と線形の間" section 2 chunk scan at segment granularity), and the segment's pass
 * started from P_r give the same rows as one pass over the whole sequence.
 *
 * la_chunked_state -- the final state of a causal pass over k, v ([B, H, L, dk], [B, H, L,
 * dv], dtype): state[b,h,i,j] = sum_t w_t phi(k_t)_i v_t,j and zstate[b,h,i] = sum_t w_t
 * phi(k_t)_i, with w_t = 1, or gamma^(L-1-t) for the Retention decay (gamma as
 * la_decay_fwd; 1 = none).  state: device fp32 [B, H, D, dv], zstate: device fp32 [B, H, D]
 * or NULL (not computed); both fully overwritten, the la_decode_step layout.  D (dk, or m
 * for FAVOR+) at most 256; no level weights.  Generic path (fp32 accumulation).
 */
int la_chunked_state(const void *k, const void *v, float *state, float *zstate, int B, int H, int L,
                     int dk, int dv, const la_feature_map *feature_map, float gamma, int dtype,
                     void *stream);

/* state = factor * state + seg_state, zstate likewise (both NULL or both given): one step of
 * the prefix above.  [B, H, D, dv] and [B, H, D] fp32 device arrays; factor in [0, 1] (the
 * decay over seg_state's segment, gamma^len, or 1), else LA_ERR_ARG. */
int la_state_combine(float *state, float *zstate, const float *seg_state, const float *seg_zstate,
                     int B, int H, int D, int dv, float factor, void *stream);

/*
 * la_chunked_fwd_init -- the causal forward (plain mask, or the decay when gamma != 1)
 * starting from a given state: row t also reads gamma^(t+1) phi(q_t)^T state0 (and
 * zstate0 in the normaliser), as if the rows that produced state0 preceded row 0.
 * state0, zstate0: device fp32 [B, H, D, dv] and [B, H, D] (la_chunked_state's layout), or
 * NULL for zero.  Other arguments as la_decay_fwd; no level weights.  The tensor-core path
 * covers it for identity / elu+1 with C <= 64 (decay: C = 64); FAVOR+ and C > 64 run on the
 * generic path.  The workspace is la_chunked_workspace_bytes (gamma = 1) or
 * la_decay_workspace_bytes.
 */
int la_chunked_fwd_init(const void *q, const void *k, const void *v, void *out, int B, int H, int L,
                        int dk, int dv, int C, const la_feature_map *feature_map, int normalize,
                        float gamma, const float *state0, const float *zstate0, int dtype,
                        void *workspace, size_t workspace_bytes, void *stream, int path);

/* ---- what stands around the attention: rotary positions, a gated recurrence, group norm ----
 *
 * None of the three is on the pages' hot path; they are what a layer built from it needs next
 * to it: the rotation of q and k that goes with the Retention decay, a recurrence whose decay
 * is data instead of one constant, and the per-head normalisation with a gate that replaces
 * the attention normaliser.  Layouts are [B, H, L, d] with adjacent channels; the strides of
 * the other three axes may be given, so that they work on views of a fused projection.
 * Every call runs on the current device; tensors must live there. */

/* Strides in elements: element (b, h, t, i) is at b*strides.b + h*strides.h + t*strides.l + i.
 * A NULL pointer means contiguous [B, H, L, d].  Strides of inputs must not be negative (0
 * broadcasts); those of outputs must keep all elements apart (LA_ERR_ARG otherwise). */
typedef struct la_strides {
    long long b, h, l;
} la_strides;

/* How the recurrence's gate a_t follows from the gate input g_t. */
enum la_gate_kind {
    LA_GATE_VALUE = 0,  /* a = g                                                          */
    LA_GATE_LOG = 1,    /* a = exp(g); g = -inf is a = 0                                  */
    LA_GATE_SIGMOID = 2 /* a = 1 / (1 + exp(-g))                                          */
};

/* Rows per stored state of la_recurrence_fwd. */
#define LA_RECURRENCE_CHUNK 64

/*
 * la_recurrence_fwd -- gated linear recurrence, one scalar state per channel:
 *     h_t = a_t h_{t-1} + w_t x_t,   out_t = h_t,   w = 1, or 1 - a with `complement`,
 * the elementwise counterpart of the decayed state S_t = gamma S_{t-1} + phi(k_t) v_t^T with
 * a decay per token and channel.  A gate of 0 forgets everything before its row (the first
 * row of a packed document).  States, gates and sums are fp32; out is rounded once.
 *   x, out        [B, H, L, d], dtype `dtype`
 *   gate          [B, H, L, d], dtype `gate_dtype`; gates are meant to be in [0, 1].  Others
 *                 are computed as the formula says, but rows are combined through products of
 *                 up to 256 gates in fp32: where those overflow, the result is not finite.
 *                 With u = 2^-24, a and 1 - a are evaluated in fp32 to (9 + 1.3 |g|) u
 *                 relatively, values below 2^-126 absolutely; for fp32 activations an a above 1/2
 *                 (log gates: above 15/16, or with complement) is off by u/2 and 9 u of 1 - a,
 *                 so that long memories keep their gain.
 *   h0            device fp32 [B, H, d], the state before row 0, or NULL for zero
 *   lengths       NULL, or device int [B]: sequence b ends after lengths[b] rows (clamped to
 *                 0..L).  Rows behind are not read; out is 0 there and the state stays.
 *   h_last        device fp32 [B, H, d], the state after the last row, or NULL; may be h0
 *   chunk_states  device fp32 [B, H, ceil(L / LA_RECURRENCE_CHUNK), d] or NULL: the states
 *                 before rows 0, 64, 128, ..., which la_recurrence_bwd reads
 * A gate of 0 (value 0, log or sigmoid of -inf) forgets infinities and NaN too, those of gates before
 * it among them; no other gate does, however small.  Outputs must not overlap inputs, but for
 * h_last.
 * Returns LA_OK, LA_ERR_NULL, LA_ERR_SHAPE, LA_ERR_UNSUPPORTED (dtype, gate kind), LA_ERR_ARG
 * (strides, alignment) or LA_ERR_CUDA.  Asynchronous on `stream`, no workspace; the sums' order
 * depends on the sizes and the GPU alone, so equal calls give equal bits.  Where few heads are
 * cut along L, the blocks of a cluster wait for one another, each wait with a limit:
 * LA_ERR_TIMEOUT from la_last_device_status.
 */
int la_recurrence_fwd(const void *x, const void *gate, const float *h0, const int *lengths,
                      void *out, float *h_last, float *chunk_states, int B, int H, int L, int d,
                      const la_strides *x_strides, const la_strides *gate_strides,
                      const la_strides *out_strides, int gate_kind, int complement, int dtype,
                      int gate_dtype, void *stream);

/*
 * la_recurrence_bwd -- its gradients.  With e_t = dout_t + a_{t+1} e_{t+1} (dh_last behind the
 * last row):
 *     dx_t = w_t e_t,  dgate_t = e_t (h_{t-1} - [complement] x_t) da/dg,  dh0 = a_0 e_0.
 * h_{t-1} is recomputed in fp32 from x, gate and the forward's chunk_states; the forward's
 * rounded output is not an input.
 *   dout          [B, H, L, d], dtype `dtype`
 *   dh_last       device fp32 [B, H, d], the gradient of h_last, or NULL for zero
 *   dx, dgate     [B, H, L, d], dtype `dtype` and `gate_dtype`; fully overwritten, 0 behind a
 *                 sequence's end
 *   dh0           device fp32 [B, H, d] or NULL; may be dh_last.  Otherwise outputs must not
 *                 overlap inputs.
 * Other arguments and errors as la_recurrence_fwd.
 */
int la_recurrence_bwd(const void *x, const void *gate, const float *chunk_states,
                      const int *lengths, const void *dout, const float *dh_last, void *dx,
                      void *dgate, float *dh0, int B, int H, int L, int d,
                      const la_strides *x_strides, const la_strides *gate_strides,
                      const la_strides *dout_strides, const la_strides *dx_strides,
                      const la_strides *dgate_strides, int gate_kind, int complement, int dtype,
                      int gate_dtype, void *stream);

/* One decoding step: state = a state + w x, out = state, for contiguous [B, H, d] x, gate, out
 * and fp32 state (updated in place, as la_decode_step's).  Stepping t = 0..L-1 reproduces
 * la_recurrence_fwd's rows. */
int la_recurrence_step(const void *x, const void *gate, float *state, void *out, int B, int H,
                       int d, int gate_kind, int complement, int dtype, int gate_dtype,
                       void *stream);

/* ---- rotary positions ---- */
enum la_rotary_layout {
    LA_ROTARY_HALF = 0,       /* channel j is turned with channel j + rot/2               */
    LA_ROTARY_INTERLEAVED = 1 /* channel 2j is turned with channel 2j + 1                 */
};

/* How the frequencies are scaled for contexts `factor` times the original length. */
enum la_rotary_scaling {
    LA_ROTARY_PLAIN = 0,  /* theta_j = base^(-2j/rot)                                       */
    LA_ROTARY_LINEAR = 1, /* theta_j / factor                                               */
    LA_ROTARY_PARTS = 2   /* by turns r over the original length: theta_j where r >= fast,
                             theta_j / factor where r <= slow, mixed linearly in r between  */
};

/*
 * la_rotary_table -- host only: fills turns[0..rot/2) with the frequencies as fractions of a
 * full turn per position, in units of 2^-64.  A position times that, modulo 2^64, is its
 * angle without a further rounding.  The caller copies the table to the device and keeps it.  fast, slow, original_length are read for LA_ROTARY_PARTS only (0 < slow
 * < fast).  LA_ERR_SHAPE for rot <= 0 or odd, LA_ERR_ARG for base <= 0, factor < 1, values
 * that are not finite, or more than 2^50 turns per position.
 */
int la_rotary_table(int rot, double base, int scaling, double factor, double original_length,
                    double fast, double slow, unsigned long long *turns);

/*
 * la_rotary -- turns the first `rot` channels of q and k by their positions: a pair (u, v) at
 * position p becomes amplitude (u cos - v sin, u sin + v cos) of the angle p theta_j; channels
 * from rot on are copied.  The gradient of a rotation is the rotation back: `inverse` turns
 * by -p theta_j (amplitude stays a factor).
 *   q, q_out      [B, H, L, d], k, k_out [B, Hk, L, d], dtype `dtype`; k and k_out may both be
 *                 NULL.  q_out may be q with the same strides (in place), k_out likewise;
 *                 other overlaps are not allowed.
 *   turns         device copy of la_rotary_table's array, rot/2 entries (rot = 0: may be NULL)
 *   positions     device int [B, L], or NULL: row t of every sequence is at offset + t
 *   rot           even, 0 <= rot <= d
 * Angles are position times the table's frequency to 2^-33 of a turn, sines and cosines fp32; each
 * output is rounded once.  The frequencies are those of 64-bit arithmetic, off by up to 2^-54 of a
 * turn, so the angle at position p is off by p times that (2^31: 2^-23 of a turn).
 * Returns LA_OK, LA_ERR_NULL, LA_ERR_SHAPE, LA_ERR_UNSUPPORTED, LA_ERR_ARG or LA_ERR_CUDA.
 */
int la_rotary(const void *q, const void *k, void *q_out, void *k_out,
              const unsigned long long *turns, const int *positions, long long offset, int B,
              int H, int Hk, int L, int d, int rot, const la_strides *q_strides,
              const la_strides *k_strides, const la_strides *q_out_strides,
              const la_strides *k_out_strides, int layout, int inverse, float amplitude,
              int dtype, void *stream);

/* ---- group norm with an activation, channels last ---- */
enum la_activation {
    LA_ACT_NONE = 0, /* act(y) = y                                                        */
    LA_ACT_SILU = 1, /* act(y) = y / (1 + exp(-y))                                        */
    LA_ACT_SIGMOID = 2 /* act(y) = 1 / (1 + exp(-y)); the gate of la_block_norm_fwd only   */
};

/*
 * la_group_norm_fwd -- the channels of each token normalised in H groups of d, as they leave
 * the attention, with the gate that follows it:
 *     xh = (x - mean) / sqrt(var + eps)  over the d channels of (b, h, t)
 *          (center = 0: x / sqrt(mean(x^2) + eps)),
 *     y = xh weight + bias,   out = y act(gate) with a gate, act(y) without.
 *   x             [B, H, L, d] (the attention's output layout), dtype `dtype`
 *   weight, bias  device fp32 [H, d] or NULL (1 and 0)
 *   gate, out     dtype `dtype`; their NULL strides mean contiguous [B, L, H, d], channels
 *                 last (gate itself may be NULL)
 *   eps           > 0 and finite, else LA_ERR_ARG
 *   d             at most 8192, else LA_ERR_UNSUPPORTED
 * Statistics are fp32 over values held in fp32, the variance from centred values.  SiLU's sigmoid
 * is off by 9 2^-24 relatively for fp32, (7 + 2.5 |z|) 2^-24 for bf16, and 0 where it is below
 * 2^-126.  Outputs must not overlap inputs.
 */
int la_group_norm_fwd(const void *x, const float *weight, const float *bias, const void *gate,
                      void *out, int B, int H, int L, int d, const la_strides *x_strides,
                      const la_strides *gate_strides, const la_strides *out_strides, int center,
                      int activation, float eps, int dtype, void *stream);

/*
 * la_group_norm_bwd -- its gradients from dout (as out, NULL strides: [B, L, H, d]): dx (as x),
 * dgate (as gate; NULL if and only if gate is), dweight and dbias (device fp32 [H, d], each
 * may be NULL).  Statistics are recomputed from x.  dweight and dbias are summed in a fixed
 * order through the workspace of la_group_norm_bwd_workspace_bytes(...) bytes (0 when neither
 * is asked for).  Outputs must not overlap inputs.
 */
int la_group_norm_bwd(const void *x, const float *weight, const float *bias, const void *gate,
                      const void *dout, void *dx, void *dgate, float *dweight, float *dbias,
                      int B, int H, int L, int d, const la_strides *x_strides,
                      const la_strides *gate_strides, const la_strides *dout_strides,
                      const la_strides *dx_strides, const la_strides *dgate_strides, int center,
                      int activation, float eps, int dtype, void *workspace,
                      size_t workspace_bytes, void *stream);

/* Workspace bytes la_group_norm_bwd needs for these sizes when weight gradients are asked for
 * (0 on invalid arguments). */
size_t la_group_norm_bwd_workspace_bytes(int B, int H, int L, int d);

/* ---- norms around a block, with its gate and the residual sum ---- */
enum la_norm_kind {
    LA_NORM_NONE = 0, /* x                                                                 */
    LA_NORM_RMS = 1,  /* x / sqrt(mean(x^2) + eps)                                          */
    LA_NORM_LAYER = 2 /* (x - mean) / sqrt(var + eps)                                       */
};

/*
 * la_block_norm_fwd -- behind a block, and before the next one:
 *     h = residual_scale r + branch_scale act(gate) (norm(y) post_weight + post_bias),
 *     n = norm(h) pre_weight + pre_bias,
 * over rows of d channels.  y is the block's output, r the residual stream before it, h behind it, n the
 * next block's input.  With post_norm LA_NORM_NONE post_weight is a layer scale.
 *   y, gate, n    [B, L, d], dtype `dtype`; gate may be NULL (act is 1), n may be NULL (only h is formed)
 *   residual, h   [B, L, d], dtype `residual_dtype`: `dtype`, or LA_F32
 *   strides       of the axes B and L (b and l; h is not read); NULL: contiguous.  0 broadcasts an input.
 *   *_weight, *_bias  device fp32 [d] or NULL (1 and 0)
 *   post_norm, pre_norm  enum la_norm_kind; pre_norm is not LA_NORM_NONE where n is given
 *   activation    enum la_activation, of the gate
 *   scales, eps   finite, eps > 0, else LA_ERR_ARG
 *   d             at most 8192, else LA_ERR_UNSUPPORTED
 * Statistics are fp32 over values held in fp32, n's over h before it is rounded; each output is rounded
 * once.  The sigmoid of a bf16 gate z is taken to (5 + |z|) 2^-23 of itself, and as 0 below -87.3.  h may be
 * residual, and n may be y, with the same strides; otherwise outputs must not overlap inputs.
 */
int la_block_norm_fwd(const void *y, const void *residual, const void *gate,
                      const float *post_weight, const float *post_bias, const float *pre_weight,
                      const float *pre_bias, void *h, void *n, int B, int L, int d,
                      const la_strides *y_strides, const la_strides *residual_strides,
                      const la_strides *gate_strides, const la_strides *h_strides,
                      const la_strides *n_strides, int post_norm, int pre_norm, int activation,
                      float residual_scale, float branch_scale, float eps, int dtype,
                      int residual_dtype, void *stream);

/*
 * la_block_norm_bwd -- its gradients from dh (as h; the gradient that reaches h by the residual stream, NULL
 * for zero) and dn (as n; NULL where n was not used): dresidual (as residual), dy (as y), dgate (as gate,
 * NULL if and only if gate is; a broadcast gate's is the whole [B, L, d]), and device fp32 [d] or NULL each
 * dpost_weight, dpost_bias, dpre_weight, dpre_bias (the last two with dn only).  Statistics and h are formed
 * again from y and r, so the forward's h may be gone.  The weights' sums are fp32, in a fixed order, through the
 * workspace of la_block_norm_bwd_workspace_bytes(...) bytes, 16-byte aligned (not needed without them).
 * dresidual may be dh, and dy may be dn, with the same strides; otherwise outputs must not overlap inputs.
 */
int la_block_norm_bwd(const void *y, const void *residual, const void *gate,
                      const float *post_weight, const float *post_bias, const float *pre_weight,
                      const float *pre_bias, const void *dh, const void *dn, void *dresidual,
                      void *dy, void *dgate, float *dpost_weight, float *dpost_bias,
                      float *dpre_weight, float *dpre_bias, int B, int L, int d,
                      const la_strides *y_strides, const la_strides *residual_strides,
                      const la_strides *gate_strides, const la_strides *dh_strides,
                      const la_strides *dn_strides, const la_strides *dresidual_strides,
                      const la_strides *dy_strides, const la_strides *dgate_strides, int post_norm,
                      int pre_norm, int activation, float residual_scale, float branch_scale,
                      float eps, int dtype, int residual_dtype, void *workspace,
                      size_t workspace_bytes, void *stream);

/* Workspace bytes la_block_norm_bwd needs for these sizes when weight gradients are asked for (0 on
 * invalid arguments). */
size_t la_block_norm_bwd_workspace_bytes(int B, int L, int d);

/* ---- gated attention: a decay for each head, or for each token and head ----
 *
 * la_gated_fwd -- causal linear attention whose state is decayed by data, for every head
 *     S_t = a_t S_{t-1} + k_t v_t^T,      out_t = scale q_t^T S_t,      a_t = exp(log_decay_t),
 * the chunked form for prompts and training; la_gated_step is its recurrent form for single tokens and
 * la_gated_bwd its gradients.  la_decay_fwd is the case of one constant for all heads.  Identity features,
 * no normaliser (la_group_norm_fwd follows instead).
 *   q             [B, H, L, dk], dtype `dtype`
 *   k, v          [B, Hk, L, dk] and [B, Hk, L, dv]; H a multiple of Hk: H / Hk neighbouring heads share a
 *                 key head, each with its own decay and state
 *   log_decay     device fp32 [B, H, L] by strides (NULL: contiguous); {0, 1, 0} takes a constant for each
 *                 head.  Meant to be at most 0; -inf forgets everything before its row (the first row of
 *                 a packed document).  Others are computed as the formula says where the products of a
 *                 chunk's decays stay finite.
 *   state0        device fp32 state before row 0, or NULL for zero; state: the state behind the last row,
 *                 or NULL; may be state0.  Without slots both are [B, H, dk, dv] (la_decode_step's layout).
 *   slots         NULL, or device int [B]: the states lie in pools [n_slots, H, dk, dv], sequence b's at
 *                 slots[b].  A negative slot is none: the sequence starts from zero and its last state is
 *                 not kept; so is one of n_slots or more, which la_last_device_status reports as
 *                 LA_ERR_DEVICE.  No two sequences may share a slot; the other slots keep their values.
 *   lengths       NULL, or device int [B]: sequence b ends after lengths[b] rows (clamped to 0..L).  Rows
 *                 behind are not used, whatever they hold; out is 0 there and the state stays.
 *   out           [B, H, L, dv], dtype `dtype`
 *   dk, dv        at most 256, B * H at most 65535
 *   scale         finite, else LA_ERR_ARG
 *   path          enum la_path.  LA_PATH_SIMT takes every case, in fp32 row by row.  LA_PATH_TC takes bf16 with
 *                 dk and dv of 64 or 128 each, rows of q, k, v and out on 16-byte boundaries and no stride of
 *                 0 (LA_ERR_UNSUPPORTED otherwise); LA_PATH_AUTO takes it there, for any length.  All else (fp32,
 *                 other widths, k expanded over heads) goes row by row, 10 to 20 times as long.
 *   workspace     device memory of la_gated_workspace_bytes(...) bytes, 16-byte aligned (NULL where that is 0)
 * States, decays and sums are fp32; out is rounded once.  LA_PATH_TC rounds two operands of its products to
 * bf16 (each off by 2^-8 of itself at most): a row's weighted scores, and the state where only out reads it; the
 * state itself is summed to fp32.  A log decay below -104, whose decay fp32 does not hold, counts as -inf, and a
 * product of decays below e^-88 may count as 0.  LA_PATH_SIMT decays the state once a row: there, as in
 * la_gated_step, log decays above -2^-25 leave it as it is, which L rows add up to L 2^-25 at most.
 * q, k, v and states are meant to be finite.  An infinity or NaN in a row may reach every row of its chunk
 * of 64 and those behind, up to the first log decay of -inf in a later chunk; one in state0 (a slot
 * that holds anything) up to the first -inf.  From that row on, out and the state are those of finite inputs.
 * (LA_PATH_SIMT: only rows from the bad one to the next -inf.)  Rows behind a sequence's end reach nothing.
 * The order of the sums depends on the sizes, the path, the GPU and the decays alone, so equal calls give
 * equal bits.  Outputs must not overlap inputs, but for state.
 * Every wait inside LA_PATH_TC has a limit: LA_ERR_TIMEOUT from la_last_device_status.
 * Returns LA_OK, LA_ERR_NULL, LA_ERR_SHAPE, LA_ERR_UNSUPPORTED, LA_ERR_ARG (strides, alignment, scale),
 * LA_ERR_WORKSPACE or LA_ERR_CUDA.  Asynchronous on `stream`.
 */
int la_gated_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                 const float *state0, float *state, const int *slots, const int *lengths, void *out,
                 int B, int H, int Hk, int L, int dk, int dv, int n_slots,
                 const la_strides *q_strides, const la_strides *k_strides,
                 const la_strides *v_strides, const la_strides *g_strides,
                 const la_strides *out_strides, float scale, int dtype, void *workspace,
                 size_t workspace_bytes, void *stream, int path);

/* Workspace bytes la_gated_fwd needs for these sizes on the current device, whatever the path (0 when
 * none, or on invalid arguments). */
size_t la_gated_workspace_bytes(int B, int H, int L, int dk, int dv, int dtype);

/*
 * la_gated_bwd -- its gradients.  With D_t = scale q_t dout_t^T + a_{t+1} D_{t+1} (dstate behind the last
 * row), the gradient of S_t:
 *     dq_t = scale S_t dout_t,    dk_t = D_t v_t,    dv_t = D_t^T k_t,
 *     dlog_decay_t = <D_t, a_t S_{t-1}>,    dstate0 = a_0 D_0.
 * The states are formed again from k, v and log_decay; nothing of the forward pass is kept.  What is not finite
 * reaches dq as it does out, and from its row back dk, dv and dstate0: up to the last -inf in an earlier
 * chunk, before whose row they are those of finite inputs; dlog_decay both ways.
 *   dout          [B, H, L, dv], dtype `dtype`
 *   dstate        device fp32 [B, H, dk, dv], the gradient of the state behind the last row, or NULL for zero
 *   dq, dk, dv    as q, k, v, fully overwritten, 0 behind a sequence's end; dk and dv of a shared key
 *                 head are the sums over its heads
 *   dlog_decay    device fp32 contiguous [B, H, L], or NULL
 *   dlog_decay_head  device fp32 [H]: its sums over sequences and rows, the gradient of a constant for
 *                 each head; or NULL.  Without both the decays' gradient is not formed.  It is summed
 *                 back over up to 1024 rows from products of states, so it is off by a few fp32
 *                 roundings of the largest values (and of <dstate, state>) among those rows, back to the last
 *                 row whose decay is 0, where the sum begins again.  It is 0 itself there, and for a first
 *                 row without state0.  Asking for it lets LA_PATH_TC read the state in three bf16 parts, so
 *                 dq and dk are nearer to fp32's than without.
 *   dstate0       device fp32 [B, H, dk, dv] or NULL; may be dstate.  Otherwise outputs must not overlap
 *                 inputs.
 *   workspace     la_gated_bwd_workspace_bytes(...) bytes, 16-byte aligned
 * Other arguments and errors as la_gated_fwd (no slots); LA_PATH_TC also wants dout, dq, dk, dv as q, and state0,
 * dstate and dstate0 on 16-byte boundaries.
 */
int la_gated_bwd(const void *q, const void *k, const void *v, const float *log_decay,
                 const float *state0, const int *lengths, const void *dout, const float *dstate,
                 void *grad_q, void *grad_k, void *grad_v, float *dlog_decay,
                 float *dlog_decay_head, float *dstate0, int B, int H, int Hk, int L, int dk, int dv,
                 const la_strides *q_strides, const la_strides *k_strides,
                 const la_strides *v_strides, const la_strides *g_strides,
                 const la_strides *dout_strides, const la_strides *dq_strides,
                 const la_strides *dk_strides, const la_strides *dv_strides, float scale, int dtype,
                 void *workspace, size_t workspace_bytes, void *stream, int path);

/* Workspace bytes la_gated_bwd needs (0 on invalid arguments). */
size_t la_gated_bwd_workspace_bytes(int B, int H, int Hk, int L, int dk, int dv, int dtype);

/* One decoding step: state = a state + k v^T, out = scale q^T state.  q [B, H, dk], k [B, Hk, dk], v
 * [B, Hk, dv], log_decay [B, H] by the strides' b and h (NULL: contiguous), out contiguous [B, H, dv];
 * state fp32, [B, H, dk, dv] or by slots a pool, updated in place.  A sequence without a slot starts
 * from zero and its state is not kept.  Stepping t = 0..L-1 reproduces la_gated_fwd's rows.  Other
 * arguments and errors as la_gated_fwd. */
int la_gated_step(const void *q, const void *k, const void *v, const float *log_decay, float *state,
                  const int *slots, void *out, int B, int H, int Hk, int dk, int dv, int n_slots,
                  const la_strides *q_strides, const la_strides *k_strides,
                  const la_strides *v_strides, const la_strides *g_strides, float scale, int dtype,
                  void *stream);

/* Library version string, e.g. "0.1.0". */
const char *la_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LA_CHUNKED_H */
