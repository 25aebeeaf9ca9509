/*
 * moe.h -- C ABI of libmoe: the MoE layer forward over a slot-addressed expert
 * cache, and the adaptive cache policy beside it, for one NVIDIA GB300
 * (sm_103a).
 *
 * Everything here follows the problem statement of the Strata expert-paths
 * page (hanayo.cn, "显存里缓存的是什么？", "路由以后，专家怎样分工？",
 * "哪些专家能长期留在显存？") and the FreeToken reading notes
 * (zhongzhuzhou.org, sections 3.3 and 4): experts are identified by
 * (layer, expert); a residency table maps that identity to a cache slot or to
 * a "not resident" sentinel; tokens that chose the same expert form one group
 * with input and output positions; the expert computes gate/up, SiLU(gate)*up
 * and the down projection on 4-bit block-scaled weights; outputs are merged
 * with the routing weights plus a gated shared expert; heat counters with
 * decay drive same-layer hot-in/cold-out swaps, and a swapped slot is
 * published only after its copy has landed.
 *
 * Conventions for every call
 *   - Pointers named *_dev / tensors are DEVICE memory owned by the caller,
 *     unless the argument says "host".  bf16 tensors are passed as raw 16-bit
 *     patterns (uint16_t).  All arrays are dense row-major.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *     compute call is asynchronous on that stream; it allocates nothing and
 *     does not synchronise.  The caller keeps the arguments alive until the
 *     stream has passed the call.
 *   - The return value reports errors the host can see at call time:
 *     MOE_OK, MOE_EINVAL (bad shape, k > E, NULL pointer, size limits),
 *     MOE_ENOMEM, MOE_ECUDA (a CUDA call or kernel launch failed).
 *     Conditions only the device can see (an expert neither resident nor
 *     staged, an index out of range, a NaN logit, a bounded wait that
 *     expired) are recorded in the workspace's device error word; the
 *     kernels never trap.  moe_sync_status() synchronises the stream, returns
 *     the first recorded device error and clears it.
 *   - Handles (moe_cache, moe_ws) are owned by the library and hold device
 *     memory allocated at creation.  They are not thread-safe; one stream
 *     should drive a workspace at a time.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* moe_stream_t; /* == cudaStream_t */

enum {
  MOE_OK = 0,
  MOE_EINVAL = 1,
  MOE_ENOMEM = 2,
  MOE_ECUDA = 3,
  MOE_EMISSING = 4, /* device: a routed expert is neither resident nor staged */
  MOE_ERANGE = 5,   /* device: an index (slot, expert id) is out of range     */
  MOE_ENAN = 6,     /* device: a router logit is NaN                          */
  MOE_ETIMEOUT = 7  /* device: a bounded wait gave up                          */
};

/* Source of a group's weights, as resolved by the residency lookup. */
enum { MOE_SRC_MISSING = -1, MOE_SRC_RESIDENT = 0, MOE_SRC_STAGED = 1, MOE_SRC_SKIPPED = 2 };

/* Forward modes. */
enum { MOE_MODE_AUTO = 0, MOE_MODE_DECODE = 1, MOE_MODE_PREFILL = 2 };

/* Decode paths (moe_ws_set_decode_path). */
enum { MOE_DECODE_FUSED = 0, MOE_DECODE_CHAIN = 1 };

typedef struct moe_cache moe_cache; /* residency + staging tables, slot pools, heats, backing store */
typedef struct moe_ws moe_ws;       /* per-call scratch: logits, ids, groups, h, o, error word */

/* ------------------------------------------------------------------ shapes */

/* One MoE layer.  H hidden, I routed intermediate, E experts, k per token,
 * I_shared shared-expert intermediate (0 = no shared expert).
 * Limits: H, I and a nonzero I_shared powers of two in [64, 4096];
 * 1 <= k <= min(E, 32); 1 <= E <= 1024.  Anything else is MOE_EINVAL. */
typedef struct {
  int H, I, E, k, I_shared;
} moe_layer_shape;

/* Per-layer weights that live outside the expert cache. */
typedef struct {
  const uint16_t* w_router;      /* bf16 [E, H]; NULL -> logits are an input (see moe_route) */
  const float* bias;             /* fp32 [E] added to the logits, or NULL                    */
  const uint16_t* w_shared_gate; /* bf16 [H] shared-expert gate vector, or NULL               */
  const void* shared_blob;       /* device blob of the shared expert (moe_pack_expert), or NULL */
  int layer;                     /* layer index in the cache's (layer, expert) space          */
  moe_layer_shape s;
} moe_layer_desc;

/* ------------------------------------------------------------- weight blobs
 * Canonical matrix format (the NVFP4 row layout of the Qwen3.8-Flash-Next
 * DGX Spark deployment notes, "一个 160 维向量在 packed 文件中占 90 字节" and
 * "NVFP4 code 和 scale 如何反量化"): rows x cols values, each row cols/2 code
 * bytes (two E2M1 codes per byte, low nibble = even column) followed by
 * cols/16 FP8-E4M3 block scales (one per 16 columns); one FP32 global scale
 * per matrix.  value = E2M1(code) * E4M3(scale) * global.
 *
 * An expert blob is the library's slot layout of one expert's three matrices
 * gate [I x H], up [I x H], down [H x I]: a 256-byte header, then code and
 * scale regions per matrix, each 256-byte aligned.  moe_blob_bytes() gives
 * its size; all slots of a cache have that stride. */
size_t moe_blob_bytes(int H, int I);

/* Repack one expert from canonical packed rows (HOST pointers: gate and up
 * [I][9H/16] bytes, down [H][9I/16] bytes) into a HOST blob buffer of
 * moe_blob_bytes(H, I) bytes.  Synchronous, host only. */
int moe_pack_expert(const uint8_t* gate_rows, const uint8_t* up_rows, const uint8_t* down_rows, int H, int I,
                    float gscale_gate, float gscale_up, float gscale_down, void* blob_out_host);

/* -------------------------------------------------------------- the cache */

/* Create a cache for L layers x E experts of shape (H, I): `nslots` cache
 * slots and `nstaging` staging slots in device memory, the residency and
 * staging tables (all -1), fp32 heat counters (0) and statistics.
 * `backing` holds the blobs of all L*E experts, expert (l, e) at offset
 * (l*E + e) * moe_blob_bytes(H, I); it is device memory when
 * backing_on_device != 0, else page-locked host memory (cudaHostAlloc'd or
 * cudaHostRegister'ed) that the device reads directly.  The caller owns it
 * and keeps it alive and unchanged while the cache exists (it is the source
 * of truth; evicted experts need no copy back).  Synchronous. */
int moe_cache_create(moe_cache** out, int L, int E, int H, int I, int nslots, int nstaging, const void* backing,
                     int backing_on_device);
int moe_cache_destroy(moe_cache* c);

/* Admit one expert into a free slot (the Strata page's admit(): only while a
 * free slot exists; otherwise *slot_out = -1 and the expert stays
 * non-resident).  Copies its blob from the backing store.  Synchronous. */
int moe_cache_admit(moe_cache* c, int layer, int expert, int32_t* slot_out);

/* Bulk set-up: make exactly the experts with mask_host[l*E+e] != 0 resident
 * (admitted in (layer, expert) order), or staged when `staging` != 0.
 * Synchronous.  Fails with MOE_ENOMEM when the pool is too small. */
int moe_cache_fill(moe_cache* c, const uint8_t* mask_host, int staging);

/* Device pointers to the cache's tables (valid for the cache's lifetime):
 * resid / stage int32 [L*E] (slot or -1), heat fp32 [L*E], slot_owner int32
 * [nslots] (l*E+e or -1), slot and staging pool bases; the global LRU's
 * lru_tick uint32 [nslots] (the LRU clock at each slot's last use, 0: never)
 * and lru_clock uint32 [1] (layer calls planned so far). */
typedef struct {
  int32_t* resid;
  int32_t* stage;
  float* heat;
  int32_t* slot_owner;
  void* slots;
  void* staging;
  size_t blob_bytes;
  int L, E, nslots, nstaging;
  uint32_t* lru_tick;
  uint32_t* lru_clock;
} moe_cache_view;
int moe_cache_get_view(const moe_cache* c, moe_cache_view* out);

/* Per-layer counters accumulated on the device: out_host receives
 * int64 [L][5] = {lookups, resident hits, staged, missing, skipped by the
 * tail skip}.  Synchronous. */
int moe_get_stats(const moe_cache* c, int64_t* out_host);

/* ---------------------------------------------------------- the workspace */

/* Scratch for layer calls of up to maxT tokens of shape s (device memory,
 * sized at creation).  Holds logits, top-k ids/weights, the expert groups,
 * the intermediate h, per-position expert outputs and the error word. */
int moe_ws_create(moe_ws** out, int maxT, moe_layer_shape s);
int moe_ws_destroy(moe_ws* ws);

/* Device pointers to the groups written by the last moe_group /
 * moe_layer_forward on this workspace (capacities maxT*k):
 *   num_groups int32[1]; grp_expert int32[G] ascending; grp_off int32[G+1];
 *   grp_slot int32[G] (slot or staging index, -1 missing);
 *   grp_src int32[G] (MOE_SRC_*); ent_tok int32[T*k]; ent_pos int32[T*k]
 *   (t*k + r), entries of group g at [grp_off[g], grp_off[g+1]) by token. */
typedef struct {
  int32_t* num_groups;
  int32_t* grp_expert;
  int32_t* grp_off;
  int32_t* grp_slot;
  int32_t* grp_src;
  int32_t* ent_tok;
  int32_t* ent_pos;
  float* logits;    /* fp32 [maxT, E] */
  int32_t* topk_ids; /* int32 [maxT, k] */
  float* topk_w;    /* fp32 [maxT, k] */
  int32_t* error;   /* int32[1] device error word (first error wins) */
} moe_ws_view;
int moe_ws_get_view(const moe_ws* ws, moe_ws_view* out);

/* Optional per-kernel timing.  When enabled, every hot-path call on this
 * workspace records a CUDA event pair around each kernel it launches, on the
 * call's stream.  moe_ws_kernel_times() synchronises on the last event and
 * writes, for the kernels of the most recent call in launch order, their
 * elapsed milliseconds (ms_out[i]) and static names (names_out[i], may be
 * NULL); *n_out receives the count (at most `max`).  Off by default. */
int moe_ws_set_profiling(moe_ws* ws, int enable);

/* Optional tail skip (Strata page, "还有一条会改变输出的路径：跳过尾部专家"):
 * with min_rank > 0, the grouping of later calls on this workspace drops a
 * group whose expert is not resident (staged or missing) when every entry has
 * a zero-based rank (its position r in the token's list) of at least
 * min_rank.  A dropped group keeps its place in the group arrays with source
 * MOE_SRC_SKIPPED, slot -1 and no blob; its entries' expert outputs are zero,
 * so the layer output moves by minus those entries' weighted outputs (the
 * other weights are not renormalised), and a dropped missing expert records
 * no MOE_EMISSING.  min_rank = 0 (the default) turns it off; min_rank >= k
 * drops nothing.  Applies where the grouping looks experts up (moe_group,
 * moe_layer_forward), not to moe_layer_forward_streamed.  MOE_EINVAL when
 * min_rank < 0.  Host-side setting, no stream work. */
int moe_ws_set_tail_skip(moe_ws* ws, int min_rank);

/* Heat update inside the grouping (Strata page, "哪些专家能长期留在显存？":
 * heat counts how often the router picks an expert).  With enable != 0, the
 * grouping of later moe_layer_forward and moe_group calls on this workspace
 * with a cache also adds the window's selection counts to the cache's heat
 * row of the call's layer, with the arithmetic of cache_heat_update
 * (heat = fl32(heat + (float)count), each selected expert once per call); the
 * caller then leaves cache_heat_update out.  Off by default.  Host-side
 * setting, no stream work. */
int moe_ws_set_fused_heat(moe_ws* ws, int enable);
int moe_ws_kernel_times(moe_ws* ws, int max, float* ms_out, const char** names_out, int* n_out);

/* Decode path of later moe_layer_forward calls on this workspace (the same
 * layer in either case: Strata page, "路由以后，专家怎样分工？").
 * MOE_DECODE_FUSED (the default) runs a decode call as ONE cooperative kernel
 * -- router, top-k, groups and lookup (with the heat update and the tail skip
 * when set), gate/up, down, combine, separated by grid barriers -- whenever the
 * shapes fit it: T <= 16, T*k <= 256, E <= 1024, H a power of two in
 * [512, 2048], I a power of two in [256, 1024], I_shared 0 or I, each CTA's
 * router rows (E + 1 over the SM count, rounded up) times H / 512 at most 32,
 * its shared-memory layout within 227 KB, x, y and w_router 16-byte aligned,
 * the shared blob 32-byte aligned; other calls run the chain.  MOE_DECODE_CHAIN always runs the chain of kernels (router,
 * top-k + groups, gate/up, down, combine).  The single kernel needs every
 * SM of the device for its CTAs (a cooperative launch: MOE_ECUDA if the device
 * cannot hold them at once).  Results agree within the layer's tolerance, not
 * bit for bit (the fp32 sums run in another order); ids, groups and lookups
 * are decided on each path's own logits.  MOE_EINVAL for another value.
 * Host-side setting, no stream work. */
int moe_ws_set_decode_path(moe_ws* ws, int path);

/* Fault-injection hook for tests of the bounded waits: the grid barriers of
 * the single-kernel decode give up after wait_ns nanoseconds (default one
 * second) and, with phantom_arrivals > 0, wait for that many arrivals beyond
 * the grid, which never come -- so the wait expires, MOE_ETIMEOUT is recorded
 * in the device error word, the CTAs skip the rest of the call (its outputs
 * are undefined) and the context stays usable.  moe_sync_status() resets the
 * barrier when it returns MOE_ETIMEOUT.  phantom_arrivals 0 restores normal
 * operation; wait_ns 0, phantom_arrivals < 0 or > 1024 is MOE_EINVAL.
 * Host-side setting, no stream work. */
int moe_ws_set_wait_test(moe_ws* ws, unsigned long long wait_ns, int phantom_arrivals);

/* Synchronise `stream`, return the device error word (MOE_OK if none) and
 * reset it to MOE_OK (after MOE_ETIMEOUT also the single-kernel decode's grid
 * barrier). */
int moe_sync_status(moe_ws* ws, moe_stream_t stream);
const char* moe_strerror(int code);

/* ------------------------------------------------------- the hot path calls */

/* Router logits and top-k with renormalised weights (Strata page, "显存里缓存
 * 的是什么？": the router picks each token's experts and their merge weights).
 *   x: bf16 [T, H]; w_router: bf16 [E, H] or NULL; bias: fp32 [E] or NULL;
 *   logits_io: fp32 [T, E] -- output l = x.W_r^T + bias (fp32 accumulate)
 *   when w_router != NULL, else an INPUT (same-logits mode);
 *   topk_ids: int32 [T, k] -- the k largest logits, weight descending, ties
 *   to the lower expert id; topk_w: fp32 [T, k] -- exp(l - l_max) / sum over
 *   the k chosen (= softmax over E renormalised over the k).
 * A NaN logit records MOE_ENAN in err_dev (int32[1], may be NULL). */
int moe_route(const uint16_t* x, const uint16_t* w_router, const float* bias, float* logits_io, int T, int H, int E,
              int k, int32_t* topk_ids, float* topk_w, int32_t* err_dev, moe_stream_t stream);

/* Dedupe one layer's selections into expert groups and look each group up
 * (Strata page, "路由以后，专家怎样分工？": repeated experts of a layer and
 * window form one group recording input and output positions; "哪些专家能长期
 * 留在显存？": (layer, expert) -> slot or sentinel).  topk_ids int32 [T, k]
 * (each row distinct ids in [0, E)).  Writes the workspace's group arrays
 * (moe_ws_view): groups by ascending expert id, entries by ascending token,
 * position t*k + r; slot from the residency table, else the staging table,
 * else MOE_SRC_MISSING (also recorded as MOE_EMISSING); with the workspace's
 * tail skip on, MOE_SRC_SKIPPED for the groups it drops (moe_ws_set_tail_skip).
 * Updates the cache's lookup counters.  Out-of-range ids record MOE_ERANGE.
 * MOE_EINVAL when T exceeds the workspace's maxT, k or E differ from the
 * workspace's shape, or E from the cache's. */
int moe_group(const int32_t* topk_ids, int T, int k, int E, int layer, moe_cache* c, moe_ws* ws,
              moe_stream_t stream);

/* The whole layer: router -> top-k -> groups -> lookup -> SwiGLU experts on
 * the slot blobs -> routing-weighted combine + sigmoid-gated shared expert:
 *   y[t] = sigmoid(x_t . w_sg) * S(x_t) + sum_r w[t,r] * E_{ids[t,r]}(x_t)
 * (Strata page, "路由以后，专家怎样分工？"; FreeToken notes section 3.2: the
 * merge is exact, no expert dropped unless the workspace's tail skip is on).  x: bf16 [T, H]; y: bf16 [T, H], or
 * fp32 [T, H] when y_is_fp32.  T <= the workspace's maxT.  mode selects the
 * decode kernels (the single-kernel decode or the chain: CUDA-core router,
 * mma.sync expert tiles) or the prefill kernels (router and grouped expert
 * GEMMs on the tensor cores); AUTO takes prefill from 32 tokens on where the
 * shape and the pointers allow it, else decode (from 32 tokens the grouped
 * GEMMs' 128-row weight tiles, reused across a group's tokens, are faster
 * than decode's 16-row units).  MOE_MODE_PREFILL needs H >= 128 and
 * 16-byte aligned x, y, w_router and w_shared_gate, else MOE_EINVAL; its y
 * accumulates in fp32 with atomic adds, so the order of the (at most k + 1)
 * terms per element may vary between runs. */
int moe_layer_forward(const moe_layer_desc* d, const uint16_t* x, void* y, int y_is_fp32, int T, moe_cache* c,
                      moe_ws* ws, int mode, moe_stream_t stream);

/* The prefill forward with the layer's routed experts streamed through the
 * staging pool (Strata expert paths, "PCIe 搬运怎样与计算重叠？": the copy stream
 * fills a staging slot and records `copied`, the compute stream waits on it,
 * computes and records `used`, and the copy stream waits on `used` before it
 * overwrites the slot).  The residency and staging tables are not consulted:
 * experts e in [u*U, u*U + U) form unit u; copy_stream copies their blobs
 * (one cudaMemcpyAsync of n*blob_bytes per unit, n <= U, from the cache's
 * backing pool, device or pinned host) into staging slots (u % 2)*U ..; stream
 * runs the grouped GEMMs of that unit's groups once they have landed.  The
 * shared expert runs with unit 0.  buffers = 2 double-buffers the units
 * (unit u + 1 copies while unit u computes); buffers = 1 keeps one half, so
 * each copy waits for the previous unit's GEMMs (the FreeToken notes'
 * "second buffer off" ablation, section 5.3).  Same arguments, layout and
 * result as moe_layer_forward in prefill mode, plus: U >= 1 with buffers*U <=
 * the cache's staging slots, buffers 1 or 2, a backing pool, and copy_stream
 * a stream other than stream, else MOE_EINVAL.  Both streams may be used again
 * as soon as the call returns; the staging slots' contents and table entries
 * are left undefined for lookups (the staging table itself is not changed). */
int moe_layer_forward_streamed(const moe_layer_desc* d, const uint16_t* x, void* y, int y_is_fp32, int T,
                               moe_cache* c, moe_ws* ws, int U, int buffers, moe_stream_t stream,
                               moe_stream_t copy_stream);

/* Activation rows as sums of NVFP4 terms, the B operands of the block-scaled
 * FP4 prefill GEMMs.  The format is the weights' (PLE offload page, "NVFP4 code
 * 和 scale 如何反量化": value = E2M1 code x FP8-E4M3 scale per 16 values x FP32
 * global scale); the pages give its decoding, and this quantiser is its plain
 * reading, applied R times to the remaining residual: term r of row i is
 * q = Q(v - q_1 - ... - q_{r-1}), Q with
 *   G: the smallest power of two with max|row| / (6 G) <= 448;
 *   s: per 16 values, the smallest non-negative E4M3 value with 6 s G >= max|block|;
 *   code: the E2M1 value nearest to v / (s G) (correctly rounded quotient), ties to even.
 *   src     rows x K activations, row i at src + i * ld elements: bf16 (src_is_fp32 = 0)
 *           or fp32; 16-byte aligned, ld a multiple of 8;
 *   codes   uint8 [rows * R][K / 2] out: term r of row i at row i * R + r, low nibble =
 *           even column; 8-byte aligned;
 *   scales  uint8 [rows * R][K / 16] out: the E4M3 block scales (sign bit clear);
 *   gscale  fp32 [rows * R] out: the global scales.
 * K a power of two in [64, 4096], 1 <= R <= 8, else MOE_EINVAL.  The residual is
 * kept in fp32: exact for bf16 rows, within one rounding per term for fp32 rows.
 * Asynchronous on `stream`. */
int moe_nvfp4_split(const void* src, int src_is_fp32, int rows, int K, int ld, int R, uint8_t* codes,
                    uint8_t* scales, float* gscale, moe_stream_t stream);

/* Several MoE layers of a prefill chunk, each layer's experts streamed whole
 * through the staging pool one layer ahead (FreeToken notes, section 3.1: layer
 * l + 1's experts copy into the second buffer while layer l computes with the
 * first; section 5.3: with the second buffer off, each copy waits until the
 * previous layer is done).  The layers sit on an fp32 residual stream as in
 * moe_residual_rmsnorm: for l = 0 .. L-1, x_res += y (l > 0), xn = bf16(RMSNorm
 * (x_res)), y = MoE_l(xn) in prefill mode; finally x_res += y.
 *   d       moe_layer_desc [L] (host), the same H, E and k, each with its layer;
 *   x_res   fp32 [T, H] device, the residual stream, updated in place (16-byte aligned);
 *   xn, y   bf16 [T, H] device scratch (16-byte aligned); on return xn holds the
 *           normalised final stream, y the last layer's output.
 * Layer l uses staging slots h * E .. h * E + E - 1 with h = l % buffers: the copy
 * stream waits on `used` of the layer that last read half h, copies the layer's E
 * blobs from the cache's backing pool (device or pinned host) in one
 * cudaMemcpyAsync and records `copied`; the compute stream waits on `copied` before
 * the layer's expert GEMMs and records `used` after them.  The residency and
 * staging tables are not consulted or changed.  buffers 1 or 2, buffers * E <= the
 * cache's staging slots, a backing pool, eps > 0, copy_stream distinct from
 * stream, and every layer valid for moe_layer_forward in prefill mode, else
 * MOE_EINVAL.  Both streams may be reused as soon as the call returns. */
int moe_layers_forward_streamed(const moe_layer_desc* d, int L, float* x_res, uint16_t* xn, uint16_t* y, int T,
                                moe_cache* c, moe_ws* ws, int buffers, float eps, moe_stream_t stream,
                                moe_stream_t copy_stream);

/* Heat update (Strata page, "哪些专家能长期留在显存？": accumulate how often
 * each expert is routed to): heat[layer*E+e] = fl32(heat + (float)count_e)
 * with count_e the number of (token, rank) selections of e in topk_ids
 * int32 [T, k].  Out-of-range ids record MOE_ERANGE in err_dev (may be NULL). */
int cache_heat_update(moe_cache* c, const int32_t* topk_ids, int T, int k, int layer, int32_t* err_dev,
                      moe_stream_t stream);

typedef struct {
  int layer, hot_expert, cold_expert, slot;
  float diff;
} moe_swap;

typedef struct {
  float threshold; /* 1.5f  */
  int max_swaps;   /* 96    */
  float decay;     /* 0.7f  */
} moe_policy_cfg;

/* One planning round (same section: pair hot non-resident with cold resident
 * experts of the same layer when the heat difference reaches the threshold,
 * sort by difference, cap per round, then decay all heats):
 *   per layer, non-resident experts by heat desc (id asc) are paired i-th with
 *   resident experts by heat asc (id asc) while fl32(h_hot - h_cold) >=
 *   threshold; candidates of all layers ordered by (diff desc, layer asc,
 *   hot id asc); the first max_swaps written to plan_dev (moe_swap[max_swaps],
 *   device) and their number to n_dev (int32[1], device); then every heat
 *   becomes fl32(heat * decay).  A NaN difference (a NaN heat, or infinite
 *   heats on both sides) fails the test, so it ends its layer's pairing there.
 *   Requires L*E <= 32768 and max_swaps <= 4096. */
int cache_plan_swaps(moe_cache* c, const moe_policy_cfg* p, moe_swap* plan_dev, int32_t* n_dev, moe_stream_t stream);

/* Residual stream and RMS normalisation between the layers of a decode stack.
 * The pages give the model as MoE layers in sequence but have no counterpart
 * to this step: it is the wrapper of the 48-layer decode workload,
 * x_{l+1} = x_l + MoE_l(RMSNorm(x_l)), with unit RMSNorm weight.
 *   x_res   float [T, H] device, the residual stream, updated in place:
 *           x_res += y_prev when y_prev != NULL (bf16 [T, H], the previous
 *           layer's output);
 *   xn_out  bf16 [T, H] device: bf16(x_res / sqrt(mean(x_res^2) + eps)),
 *           the next layer's input.
 * fp32 arithmetic (sum of squares in fp32, correctly rounded sqrt and
 * division).  H a multiple of 4 and at most 4096, eps > 0, x_res 16-byte and
 * the bf16 arrays 8-byte aligned, else MOE_EINVAL. */
int moe_residual_rmsnorm(float* x_res, const uint16_t* y_prev, uint16_t* xn_out, int T, int H, float eps,
                         moe_stream_t stream);

/* cache_plan_swaps on caller-owned tables, allocating nothing.  The pages
 * have no counterpart to this call: it exists for callers that cannot
 * allocate device memory where they plan -- a serving loop whose memory is
 * handed out by its own allocator under a fixed budget (a cudaMalloc would
 * step outside the budget or fail when it is spent), or one that keeps the
 * heat and residency tables in its own buffers without a moe_cache handle.
 *   heat_dev  float [L, E] device, read and then decayed in place (as the
 *             handle's heat table is by cache_plan_swaps);
 *   resid_dev int32 [L, E] device, slot of each resident expert, negative
 *             when not resident (the layout of moe_cache_view.resid).
 * The plan, its order, n_dev and the decayed heats are exactly those of
 * cache_plan_swaps on the same tables.  The planner's scratch is a 260 KB
 * static device array inside the library, so the sizes it takes are capped:
 * L <= 1024, E <= 1024, L*E <= 32768 and L*ceil(E/2) <= 16384; larger sizes
 * (and max_swaps outside 0..4096, threshold <= 0, NULL pointers) return
 * MOE_EINVAL before anything is launched.  Nothing in the scratch needs to
 * start at zero.  The scratch's address is looked up on the first call on
 * each device (with that device current); the lookup may load the module,
 * which a stream capture does not allow, so make the first call on each
 * device before any capture.  The looked-up address is kept for the life of
 * the process: after a cudaDeviceReset (or any teardown of the device's
 * primary context) it is stale, so do not call this function again in that
 * process.  All calls on one device share the scratch: calls that overlap in
 * time (other streams, other threads) race and must be serialised by the
 * caller.  Heats may be NaN or infinite: a layer's pairing stops at the first
 * pair whose difference fails the threshold test, as in cache_plan_swaps. */
int cache_plan_swaps_noalloc(float* heat_dev, const int32_t* resid_dev, int L, int E, const moe_policy_cfg* p,
                             moe_swap* plan_dev, int32_t* n_dev, moe_stream_t stream);

/* Execute a plan (same section: new weights are visible only after the copy
 * completes; a slot is reused only after earlier reads finished):
 *   on `compute`: unmap each cold expert (resid = -1), record event
 *   "unmapped";  on `copy`: wait "unmapped", copy each hot blob from the
 *   backing store into the slot, record "copied";  on `compute`: wait
 *   "copied", publish (resid[hot] = slot).  Kernels queued on `compute`
 *   before this call finish reading the old slots before the copy starts;
 *   kernels queued after it see either the old mapping (never) or the new one.
 *   No host synchronisation; n_dev is read on the device. */
int moe_cache_apply_swaps(moe_cache* c, const moe_swap* plan_dev, const int32_t* n_dev, moe_stream_t compute,
                          moe_stream_t copy);

/* Global LRU over the slots (FreeToken reading notes, section 3.3: one LRU for
 * every layer's (layer, expert) -- a hit refreshes its recency, a fill admits
 * the newly chosen expert, the least recently used is evicted; section 4: one
 * pass finds K victim candidates and the misses take the first q <= K).  Call
 * after a layer call's grouping on ws (moe_group, moe_layer_forward) for layer
 * `layer`: advances the cache's LRU clock, marks the slots of the call's
 * resident groups as used now, then writes into plan_dev (device moe_swap[K])
 * and *n_dev (device int32) the admissions: the call's i-th miss (a group that
 * is staged or missing, in group order) into the i-th victim, the victims
 * being the slots this call did not use, empty slots first, then least
 * recently used first, ties to the lower slot.  In an entry, `layer` and
 * hot_expert name the admitted expert, cold_expert the evicted one as
 * layer * E + expert (-1: the slot was empty), slot the slot, diff is 0; the
 * slots taken count as used now.  1 <= K <= 32 and a cache of 1 to 2^24 - 1
 * slots, else MOE_EINVAL.  The clock
 * is 32-bit: past 2^32 - 2 calls the device records MOE_ERANGE.  Async on
 * `stream`; execute the plan with moe_cache_apply_lru. */
int cache_lru_plan(moe_cache* c, const moe_ws* ws, int layer, int K, moe_swap* plan_dev, int32_t* n_dev,
                   moe_stream_t stream);

/* Executes an LRU plan with the publish-after-copy order of
 * moe_cache_apply_swaps (evicted entries cleared on `compute`; blobs copied
 * from the backing store on `copy` after that; admitted entries published on
 * `compute` after the copies), the evicted expert given by its flat id.  An
 * entry whose evicted expert does not own its slot (or whose slot is not
 * empty when no expert is named) is skipped, as moe_cache_apply_swaps skips
 * an inconsistent entry. */
int moe_cache_apply_lru(moe_cache* c, const moe_swap* plan_dev, const int32_t* n_dev, moe_stream_t compute,
                        moe_stream_t copy);

/* ------------------------------------------ the attention half of a layer
 * The pages keep a request's context beside the MoE path (Strata expert paths,
 * "KV" reuse and verify windows) without giving its kernels; the calls below
 * are this library's own: keys and values in a paged cache, the position
 * rotation on the way in, attention of the newest tokens over the pages, and
 * the norms around a block on the fp32 residual stream.
 *
 * A call serves B requests at once.  Request b's new tokens are rows
 * q_start[b] .. q_start[b+1] - 1 of the call's T token rows; kv_len[b] counts
 * its tokens in the cache with the new ones, so token i of the n_b new ones is
 * at position p = kv_len[b] - n_b + i.  Position p lives in page
 * page_table[b * table_stride + p / page], place p % page.  n_b = 0 is allowed;
 * q_start is non-decreasing with q_start[0] >= 0 and q_start[B] <= T; rows
 * outside [q_start[0], q_start[B]) may be read, change no result and are not
 * written. */

/* The page pools of one layer's keys and values (device memory of the caller).
 * Element (page, head, place, column) is at page * page_stride + head *
 * head_stride + place * tok_stride + column, in both pools.  The strides are
 * in elements, below 2^38, at least D and multiples of 16 bytes; the pools are
 * 16-byte aligned. */
typedef struct {
  void* k;
  void* v;
  int e4m3;              /* 0: bf16 elements; 1: FP8-E4M3 elements                     */
  int Hkv, D;            /* key heads 1..1024; columns 64, 128 or 256                  */
  int page, npages;      /* tokens in a page (a power of two, 1..65536; at least 2 for E4M3
                            with 64 columns), pages in a pool                          */
  long long page_stride, head_stride, tok_stride;
  const float* k_scale;  /* fp32 [Hkv] device: a stored code c stands for c * scale;   */
  const float* v_scale;  /*   NULL: 1.  Read only for E4M3 pools                       */
} moe_kv_pages;

typedef struct {
  const int32_t* q_start;    /* int32 [B + 1] device                                       */
  const int32_t* kv_len;     /* int32 [B] device                                           */
  const int32_t* page_table; /* int32 [B][table_stride] device                             */
  int B, T;                  /* requests; token rows                                       */
  int max_n;                 /* about the largest n_b: picks the kernel and its tiles, and with
                                them the order of sums: a result's last bits, no more   */
  int table_stride;          /* entries of a row: a request holds at most page times this  */
} moe_kv_batch;

typedef struct moe_rope moe_rope;       /* the rotation's frequencies */
typedef struct moe_attn_ws moe_attn_ws; /* scratch of the attention calls, error word */

/* Rotation of the first `rot` columns of a head by position p: pair i is columns
 * (i, i + rot/2), or (2i, 2i + 1) when interleaved, turned by the angle
 * p * f_i: (u, w) -> (u cos - w sin, w cos + u sin).  f_i = inv_freq_host[i]
 * (double [rot/2], finite) or, with NULL, theta^(-2i/rot).  The angle is kept
 * as a 64-bit fixed-point fraction of a turn: that of the double f_i, of a size
 * below 2^64, to 2^-33 turn at every 32-bit position.  rot a multiple of 16 in [16, 256]; theta > 0 and finite.
 * Synchronous (allocates the table). */
int moe_rope_create(moe_rope** out, int rot, int interleaved, double theta, const double* inv_freq_host);
int moe_rope_destroy(moe_rope* r);

/* Append the call's new keys and values to the cache, keys rotated by position,
 * and rotate the queries.  q bf16 [T][Hq][D] -> q_out (may be q), k and v bf16
 * [T][Hkv][D]; *_stride: elements between tokens (heads are D apart), multiples
 * of 8, at least heads * D (not checked for T <= 1); all pointers 16-byte
 * aligned.  q may be NULL (Hq 0), rope NULL (nothing
 * turns).  Rotation in fp32, one rounding to the stored type: bf16 to nearest
 * even; E4M3(x / scale), the quotient rounded in fp32, to nearest even,
 * saturating at 448, NaN kept.
 * A position outside [0, page * table_stride), or a page id outside
 * [0, npages), records MOE_ERANGE in err_dev (int32[1], may be NULL) and
 * nothing is stored for that token.  Two tokens must not share a place.
 * Asynchronous on `stream`. */
int moe_kv_append(const moe_kv_pages* kv, const moe_kv_batch* b, const moe_rope* rope, const uint16_t* q,
                  long long q_stride, uint16_t* q_out, long long q_out_stride, int Hq, const uint16_t* k,
                  long long k_stride, const uint16_t* v, long long v_stride, int32_t* err_dev, moe_stream_t stream);

/* Scratch for moe_paged_attention with Hq query heads on Hkv key heads of D
 * columns (Hq a multiple of Hkv, at most 64 times it): the parts of requests
 * split over their length, and the device error word.  Independent of batch
 * and lengths. */
int moe_attn_ws_create(moe_attn_ws** out, int Hq, int Hkv, int D);
int moe_attn_ws_destroy(moe_attn_ws* ws);
typedef struct {
  int32_t* error; /* int32[1] device error word (first error wins) */
} moe_attn_ws_view;
int moe_attn_ws_get_view(const moe_attn_ws* ws, moe_attn_ws_view* out);
/* Synchronise `stream`, return the workspace's device error word and reset it. */
int moe_attn_sync_status(moe_attn_ws* ws, moe_stream_t stream);

/* Fault-injection hook for tests of the attention kernels' bounded waits: with
 * stage 1 (the queries of a piece), 2 (the weights of a tile) or 3 (the slots of
 * keys and values) that stage's barriers wait for one arrival more, which never
 * comes.  Its waits give up after a second, MOE_ETIMEOUT is recorded in the
 * workspace's error word, the call's outputs are undefined (nothing else is
 * written) and the context stays usable.  Stage 0 restores normal operation; another
 * is MOE_EINVAL.  Host-side setting, no stream work. */
int moe_attn_ws_set_wait_test(moe_attn_ws* ws, int stage);

/* Attention of every new token over its request's pages.  With group
 * g = Hq / Hkv, token at position p, query head h reads key head h / g:
 *   s_j = scale * q . k_j over the keys j <= p (and j > p - window if window > 0),
 *   o = sum_j exp(s_j) v_j / sum_j exp(s_j).
 * A token that sees no key (p < 0) gets zeros, as does a row whose scores are
 * all -infinity.  Scores are of a size below 2^30: fp32 has steps of 64 there,
 * and a row past it may come out as zeros or NaN.  What lies in the pages
 * outside a request's kv_len keys is never used, whatever it holds, and pages
 * wholly before every window of a call need no valid table entry.
 *   q, o  bf16 [T][Hq][D]; strides between tokens as in moe_kv_append; o must not
 *         overlap q.
 * Scores, softmax sums and outputs accumulate in fp32; the weights exp(s - m)
 * are rounded to 16 bits for the product with v; over E4M3 pools a column of q
 * below 2^-14 of its row's largest is rounded to 2^-22 of that.  A key in a page whose id is
 * outside [0, npages) reads as zeros and records MOE_ERANGE in the workspace's
 * error word; so does kv_len beyond page * table_stride or 2^29, whose keys end
 * there, and q_start that decreases, with which nothing is computed.
 * max_n picks the kernel, whatever the requests hold.  The same arguments give the
 * same bits in every run; the rows of one request reach no other's.  scale
 * finite; window >= 0, 0 for none.  Calls with (T + B) * Hkv * (page *
 * table_stride / 128 + 4) < 2^31 are taken; larger ones may be MOE_EINVAL.
 * Asynchronous on `stream`; one stream drives a workspace at a time. */
int moe_paged_attention(const moe_kv_pages* kv, const moe_kv_batch* b, const uint16_t* q, long long q_stride, int Hq,
                        uint16_t* o, long long o_stride, float scale, int window, moe_attn_ws* ws,
                        moe_stream_t stream);

/* --------------------------------------------- a step of drafted token trees
 * Drafted tokens may branch: a request's new tokens are the nodes of a tree.
 * Node i is the request's i-th new row and follows its parent; node 0 is the
 * request's last token, whose successors were drafted.  The step: append and
 * attention of the nodes in every layer, moe_verify_drafts on the target's
 * probabilities, moe_kv_compact on the nodes it kept.  With base = kv_len - n,
 * node i lies in place base + i of the cache and is at position base + depth_i. */
typedef struct {
  const int32_t* parent; /* int32 [T] device: the parent's index among its request's nodes,
                            below the node's own; -1 for a root (depth 0)                */
  int32_t* depth;        /* int32 [T] device                                             */
  uint32_t* above;       /* uint32 [T][words] device: bit j of row i: node j is node i or above it */
  uint32_t* below;       /* uint32 [T][words] device: bit j of row i: node j is node i or below it */
  int words;             /* 1..8; a request has at most 32 * words nodes                 */
} moe_tree;

/* Fills depth, above and below from parent, once for all layers of a step.  A parent
 * that is not below its node's index is taken as -1; so are all nodes of a request
 * past 32 * words, whose masks are empty; both record MOE_ERANGE in err_dev
 * (int32[1], may be NULL), as does q_start that decreases.  Rows outside [q_start[0],
 * q_start[B]) are left as they are.  Asynchronous on `stream`. */
int moe_tree_prepare(const moe_kv_batch* b, const moe_tree* tree, int32_t* err_dev, moe_stream_t stream);

/* Norms of each head's query and key rows: w * x / sqrt(mean(x^2) + eps) over D columns. */
typedef struct {
  const uint16_t* w_q; /* bf16 [D] or NULL: ones; 16-byte aligned */
  const uint16_t* w_k;
  float eps;           /* > 0 and finite                          */
} moe_head_norm;

/* moe_kv_append with the heads of queries and keys normalised first (norm NULL:
 * not), and at a tree's positions (tree NULL: a request's tokens follow one
 * another; only tree->depth is read).  Norm and rotation in fp32, one rounding
 * to the stored type.  Everything else as in moe_kv_append. */
int moe_kv_append_norm(const moe_kv_pages* kv, const moe_kv_batch* b, const moe_tree* tree, const moe_rope* rope,
                       const moe_head_norm* norm, const uint16_t* q, long long q_stride, uint16_t* q_out,
                       long long q_out_stride, int Hq, const uint16_t* k, long long k_stride, const uint16_t* v,
                       long long v_stride, int32_t* err_dev, moe_stream_t stream);

/* moe_paged_attention of tree nodes: node i sees the keys of its request before
 * the tree (places below base), itself and the nodes above it, as tree->above and
 * tree->below say; with a window > 0, of those the ones at a position above its
 * own less the window.  What other nodes' places hold takes no part.  The masks
 * are moe_tree_prepare's for the same batch, each the other's transpose; with
 * others a row may see what either of them says.  Everything else as in
 * moe_paged_attention, with seven in the place of four in the size of a call. */
int moe_tree_attention(const moe_kv_pages* kv, const moe_kv_batch* b, const moe_tree* tree, const uint16_t* q,
                       long long q_stride, int Hq, uint16_t* o, long long o_stride, float scale, int window,
                       moe_attn_ws* ws, moe_stream_t stream);

/* What the target's probabilities keep of drafted trees, and the next token.  From
 * node 0 on, at node v with R = the target's row of v and s = 1, its children c in
 * the order of their indices, x their token:
 *   drafted by chance (draft given):  c is kept if u_c * s * q(x) < R(x), q the draft's
 *     row of v; else R = max(R - s * q, 0), s = sum R;
 *   picked (draft NULL):              c is kept if u_c * s < R(x); else s = s - R(x), R(x) = 0;
 * the walk goes on at a kept child.  Where none is kept, the request's next token is
 * the first j with sum_{i <= j} R(i) > u_last * sum R; where sum R is 0, of the
 * target's own row; -1 where that has none.  With u uniform and children drawn from
 * q independently of one another (or picked before u is known), kept tokens and next
 * token are distributed as the target's.
 * Rows are probabilities: an entry below 0 or NaN counts as 0, one above 1 as 1; sums
 * above 4 count as 4, s below 0 as 0.  Sums are kept in fixed point, 2^-60 a unit: no
 * order of sums changes a result.  A u below 0 or NaN counts as 0, from 1 on as the
 * largest below 1. */
typedef struct {
  const float* target;    /* fp32 [T][V] device, one row a node                           */
  long long target_stride; /* elements between rows, at least V (not checked for T <= 1)  */
  const float* draft;     /* fp32 [T][V] device: row v is what v's children were drawn from; or NULL */
  long long draft_stride;
  const int32_t* token;   /* int32 [T] device: the drafted tokens; node 0's is not used. One
                             outside [0, V) is never kept                                 */
  const int32_t* parent;  /* int32 [T] device, as in moe_tree; a node that node 0 is not above is
                             never reached, nor one whose parent is not below its own index */
  const float* u;         /* fp32 [T] device: a random number a node; node 0's is not used */
  const float* u_last;    /* fp32 [B] device                                              */
  int V;                  /* 1 .. 2^24                                                    */
} moe_verify_desc;

/* path int32 [B][path_stride]: the kept nodes in their order, node 0 first, then -1; at
 * most path_stride of them (the walk ends there as at a node without children).
 * count int32 [B]: how many; 0 for a request without nodes.  token int32 [B]: the
 * next token, -1 for a request without nodes.  The three lie apart, and from the
 * inputs.  Of b, q_start, B and T are used.
 * Nodes past 256 of a request are never reached and record MOE_ERANGE in err_dev
 * (int32[1], may be NULL), as does q_start that decreases.  path_stride >= 1, fp32
 * arrays 4-byte aligned.  Asynchronous on `stream`. */
int moe_verify_drafts(const moe_kv_batch* b, const moe_verify_desc* d, int32_t* path, int path_stride, int32_t* count,
                      int32_t* token, int32_t* err_dev, moe_stream_t stream);

/* The kept nodes' keys and values to the front of their tree, in the pools of L
 * layers (kv [L] host, of one geometry: all but the pointers and scales are the
 * same): place base + path[b][d] goes to place base + d for d < count[b].  path
 * int32 [B][path_stride] and count int32 [B] device, as moe_verify_drafts writes
 * them: indices rise and are below n_b, else MOE_ERANGE is recorded in err_dev
 * (int32[1], may be NULL), as does q_start that decreases, and the request's path ends
 * before the first that does not; count is cut to path_stride.  A place past the table
 * or in a page outside [0, npages) also records MOE_ERANGE and is neither read nor
 * written.  kv_len_out int32 [B] device or NULL: base + the kept nodes, the request's
 * tokens from here on; apart from path, count and the batch's arrays.  A pool that
 * several layers share, or a layer's keys and values, is moved once; others do not
 * overlap.  Two requests must not share a page of their trees.  L <= 4096.  Asynchronous on `stream`. */
int moe_kv_compact(const moe_kv_pages* kv, int L, const moe_kv_batch* b, const int32_t* path, int path_stride,
                   const int32_t* count, int32_t* kv_len_out, int32_t* err_dev, moe_stream_t stream);

/* Pages copied in the pools of L layers (kv as above): the first tokens[i] places of
 * page src[i], all where tokens is NULL, to page dst[i], i < n (int32 [n] device,
 * n <= 2^20).  A page may be a source several times; one that is a destination is
 * neither one again nor a source.  An id outside [0, npages) records MOE_ERANGE in
 * err_dev (int32[1], may be NULL) and nothing is copied for it; tokens outside
 * [0, page] count as the nearest.  Asynchronous on `stream`. */
int moe_kv_copy_pages(const moe_kv_pages* kv, int L, const int32_t* src, const int32_t* dst, const int32_t* tokens,
                      int n, int32_t* err_dev, moe_stream_t stream);

/* The norms around a block, its gate and its residual add in one pass:
 *   z  = post_norm ? w_post * y / sqrt(mean(y^2) + eps) : y
 *   x_out = x + res_scale * g * z,   g = gate, sigmoid(gate) or 1
 *   xn = w_pre * x_out / sqrt(mean(x_out^2) + eps).
 * moe_residual_rmsnorm is the case without weights, gate, scale and post-norm. */
typedef struct {
  const uint16_t* y;       /* bf16 [T][H] the block's output, or NULL: x_out = x       */
  long long y_stride;      /* elements between tokens                                  */
  int post_norm;           /* normalise y first                                        */
  const uint16_t* w_post;  /* bf16 [H] or NULL: ones; read only with post_norm         */
  const uint16_t* gate;    /* bf16 [T][H], or NULL: none                               */
  long long gate_stride;   /* elements between tokens; 0: one row for every token      */
  int gate_sigmoid;        /* the gate is sigmoid(gate)                                */
  float res_scale;
  const uint16_t* w_pre;   /* bf16 [H] or NULL: ones                                   */
  float eps;               /* > 0                                                      */
} moe_block_norm_desc;

/* x, x_out: fp32 [T][H] (x_out may be x, and may be NULL when x_out is not
 * wanted); xn: bf16 [T][H] or NULL; strides in elements between tokens, at least
 * H (not checked for T <= 1).  fp32 arithmetic, one rounding of xn.  1 <= H <=
 * 16384.  Natural alignment suffices; 16-byte aligned rows of a multiple of 8
 * columns take wider accesses.  Asynchronous on `stream`. */
int moe_block_norm(const moe_block_norm_desc* d, const float* x, long long x_stride, float* x_out,
                   long long x_out_stride, uint16_t* xn, long long xn_stride, int T, int H, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H */
