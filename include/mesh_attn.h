/*
 * mesh_attn.h -- C ABI of the single-GPU Mesh-Attention hot path (sm_103a).
 *
 * The operation.  Exact scaled-dot-product attention O = softmax(Q K^T * scale) V with the
 * natural-log row log-sum-exp LSE, computed the way Mesh-Attention decomposes it
 * ("Mesh-Attention: A New Communication-Efficient Distributed Attention with Improved Data
 * Locality", tutorial §"Mesh-Attention：从一维'环'到二维'网'" and the arXiv abstract):
 *   1. the sequence of S tokens is cut into P partitions of L = S/P tokens; the P x P
 *      Q-KV interaction matrix is assigned as 2D tiles to a sqrt(P) x sqrt(P) mesh of
 *      (virtual) devices, with KV Partition Rotation (KVR) and a greedy order
 *      (tutorial §"贪心算法：寻找最优的'流水线'");
 *   2. each tile computes, for every Q partition it holds, a partial output O_t and its
 *      LSE_t over the tile's KV partitions (the online m_i / l_i softmax of
 *      "环形注意力：突破长序列处理瓶颈的分布式计算范式", §"数值稳定性：Log-Sum-Exp技术的分布式应用");
 *   3. the partials of each Q partition are merged by LSE rescaling:
 *      lse = ln sum_t exp(lse_t), O = sum_t exp(lse_t - lse) O_t.
 * On one GPU the mesh devices are virtual: the plan fixes the tiles and the execution
 * order, and the receive volumes a real mesh would move are counted, not performed.
 *
 * Conventions shared by every call.
 *   - Tensors are dense, row-major, contiguous, in device memory owned by the caller:
 *     Q [B, Hq, S, d], K and V [B, Hkv, S, d], O [B, Hq, S, d], LSE [B, Hq, S].
 *     Query head h reads KV head h / (Hq / Hkv) (grouped-query attention).
 *   - Causal masking: key j is visible to query i iff j <= i (same token index space).
 *   - Partials are fp32: partial_o [B, Hq, n_slots, L, d] and partial_lse [B, Hq, n_slots, L],
 *     where the slots of partition p are [slot_off[p], slot_off[p+1]) (see
 *     mesh_attn_plan_slots).  O_t is normalised (acc / l) and lse_t = m + ln l.  A row with no
 *     visible key in a slot has O_t = 0 and lse_t = -inf; the merge gives it weight 0.
 *   - Every function returns a mesh_attn_status.  Nothing throws across the ABI.  All
 *     host-side checks run before anything is enqueued; on error nothing is enqueued.
 *     mesh_attn_last_error() gives a one-line description of the last error on the
 *     calling thread.
 *   - GPU calls are asynchronous on `stream` (a cudaStream_t passed as void*; NULL is the
 *     legacy default stream) and never synchronise, except mesh_attn_read_status.
 *   - Device-side failures (a bounded wait that gave up, a work-list index out of range)
 *     are recorded in the caller's status block d_status: MESH_ATTN_STATUS_WORDS int32 in
 *     device memory, zeroed by the caller before the first call; word 0 holds the first
 *     error code, word 1 the kernel role that raised it, word 2 the work unit.  Kernels
 *     skip their work while word 0 is non-zero.  No kernel traps or asserts.
 */
#ifndef MESH_ATTN_H
#define MESH_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MESH_ATTN_OK = 0,
  MESH_ATTN_ERR_INVALID_ARG = 1,    /* bad size, null pointer, P not a square, S % P != 0 */
  MESH_ATTN_ERR_UNSUPPORTED = 2,    /* a valid problem outside what the kernels implement */
  MESH_ATTN_ERR_MISALIGNED = 3,     /* a tensor pointer not 16-byte aligned */
  MESH_ATTN_ERR_CUDA = 4,           /* a CUDA runtime call failed (message in last_error) */
  MESH_ATTN_ERR_DEVICE_TIMEOUT = 5, /* a bounded device-side wait gave up (from d_status) */
  MESH_ATTN_ERR_OUT_OF_RANGE = 6,   /* a device-side index check failed (from d_status) */
  MESH_ATTN_ERR_INTERNAL = 7,       /* an internal invariant failed */
  MESH_ATTN_ERR_NO_MEMORY = 8,      /* a host allocation failed */
  MESH_ATTN_ERR_WORKSPACE = 9       /* the workspace passed is smaller than required */
} mesh_attn_status;

typedef enum { MESH_ATTN_F32 = 0, MESH_ATTN_BF16 = 1 } mesh_attn_dtype;

#define MESH_ATTN_STATUS_WORDS 4

/* Opaque plan: host memory only, immutable after creation, safe to share between threads
 * and streams.  Created and freed by the library. */
typedef struct mesh_attn_plan mesh_attn_plan;

typedef struct {
  int64_t S;              /* tokens */
  int64_t L;              /* tokens per partition, S / P */
  int32_t P;              /* partitions = virtual devices = tiles */
  int32_t R;              /* mesh side sqrt(P) (0 for a ring plan) */
  int32_t causal, kvr, greedy;
  int32_t n_slots;        /* partial slots = work items, (p, tile) pairs with a live block */
  int32_t n_steps;        /* steps of the slowest device (greedy or ring; 0 without greedy) */
  int32_t layout;         /* 0: sqrt(P) x sqrt(P) mesh tiles; 1: ring rows */
  int32_t tile_q;         /* Q partitions per tile: R (mesh) or 1 (ring) */
  int32_t tile_kv;        /* KV partitions per tile: R (mesh) or P (ring) */
  int64_t n_kv_entries;   /* sum over items of their KV partitions = live partition blocks */
  int64_t n_live_blocks;  /* live (p, k) partition blocks of the P x P matrix */
  int32_t n_kv_slots;     /* backward: (KV partition, tile) pairs with a live block */
  int32_t reserved;
} mesh_attn_plan_info;

/* Build the tile plan (tutorial §"Mesh-Attention：从一维'环'到二维'网'", items (b) and (c);
 * §"贪心算法"; abstract: 2D tiles, KVR, greedy scheduling).
 *   S >= 0 tokens, P >= 1 partitions with P a perfect square, P <= 4096, S % P == 0.
 *   causal, kvr, greedy: 0 or 1.
 *   Tile t = device v at mesh position (v / R, v % R) holds Q partitions {r R + j : j < R} and
 *   KV partitions {k R + c : k < R} with KVR (own mesh column; block (v, v) is local) or the
 *   contiguous {c R + k : k < R} without.  Causal: block (p, k) is live iff k <= p.
 *   Greedy: each virtual device repeatedly takes the Q or KV transfer that unlocks the most
 *   live blocks (ties: KV first, then the lower partition index); work items are ordered by
 *   the step that unlocks their last block, devices interleaved step by step; each item
 *   visits its KV partitions in arrival order.  Without greedy: (tile, p) order, KV ascending.
 *   S == 0 gives an empty plan (no slots, every GPU call is a no-op).
 * On success *out owns the plan; free it with mesh_attn_plan_destroy. */
int mesh_attn_plan_create(int64_t S, int32_t P, int32_t causal, int32_t kvr, int32_t greedy,
                          mesh_attn_plan** out);

/* Ring-Attention's work assignment as a plan of the same form, to compare against the mesh
 * through the same kernels (tutorial §"Ring-Attention 的'阿喀琉斯之踵'" and the 1D ring of
 * §"Mesh-Attention：从一维'环'到二维'网'", item (a)): device v owns Q partition v and
 * computes its whole row, visiting KV partitions in ring order v, v-1, ... (own first, one hop
 * per step); one partial slot per Q partition.  Receive counts: P - 1 KV partitions per device,
 * no Q and no partial output.  Any P >= 1 (P <= 4096), S >= 0 with S % P == 0. */
int mesh_attn_plan_create_ring(int64_t S, int32_t P, int32_t causal, mesh_attn_plan** out);

/* Free a plan (NULL is accepted).  The caller must not use it afterwards. */
int mesh_attn_plan_destroy(mesh_attn_plan* plan);

/* Scalar facts of the plan. */
int mesh_attn_plan_get_info(const mesh_attn_plan* plan, mesh_attn_plan_info* out);

/* Tile map: q_parts[t*tile_q + j], kv_parts[t*tile_kv + k] for t < P (caller arrays of
 * P*tile_q and P*tile_kv int32; tile_q = tile_kv = R for a mesh plan). */
int mesh_attn_plan_tiles(const mesh_attn_plan* plan, int32_t* q_parts, int32_t* kv_parts);

/* Partial-slot CSR: slot_off[P + 1] (caller array). */
int mesh_attn_plan_slots(const mesh_attn_plan* plan, int32_t* slot_off);

/* Execution order.  items[3 i + 0..2] = (Q partition p, tile t, slot) of the i-th item,
 * item_step[i] = greedy step that completes it (0 without greedy), the KV partitions of item
 * i in visiting order are kv_list[kv_off[i] .. kv_off[i+1]).  Caller arrays of n_slots*3,
 * n_slots, n_slots + 1 and n_kv_entries int32; any of them may be NULL to skip it. */
int mesh_attn_plan_order(const mesh_attn_plan* plan, int32_t* items, int32_t* item_step,
                         int32_t* kv_off, int32_t* kv_list);

/* The order in which the kernels take the work items: order[j] (n_slots int32, caller array) is
 * the index, in mesh_attn_plan_order's list, of the j-th item the kernels take.  The greedy pass
 * (tutorial §"贪心算法：寻找最优的'流水线'") fixes each virtual device's order of work; the
 * public list interleaves the devices step by step.  One GPU takes the devices' sequences tile
 * after tile (row-major over the mesh), each in its own greedy order, so that the work items
 * running together share a tile's KV partitions and its mesh row's Q partitions in L2.  A ring
 * plan is taken in its public order.  A permutation of 0 .. n_slots - 1. */
int mesh_attn_plan_launch_order(const mesh_attn_plan* plan, int32_t* order);

/* Receive volumes a real mesh would move, per device v (tutorial §"Mesh-Attention：从一维'环'
 * 到二维'网'": per-device traffic grows as O(sqrt(N)) rather than Ring's O(N); abstract: a
 * device gathers only some of the Q and KV partitions).
 *   counts[3 v + 0..2] = Q, KV and partial-O partitions device v receives (may be NULL);
 *   bytes[3 v + 0..2]  = the same in bytes: a Q partition is L*Hq*d elements of `dtype`, a KV
 *                        partition 2*L*Hkv*d elements, a partial L*Hq*(d + 1) fp32 (may be NULL);
 *   *ring_bytes = the KV bytes one device receives in plain Ring-Attention, (P - 1) KV
 *                 partitions (may be NULL). */
int mesh_attn_plan_volumes(const mesh_attn_plan* plan, int32_t Hq, int32_t Hkv, int32_t d,
                           mesh_attn_dtype dtype, int32_t* counts, int64_t* bytes,
                           int64_t* ring_bytes);

/* Element counts of partial_o and partial_lse for a batch of B sequences with Hq heads of
 * size d: B*Hq*n_slots*L*d and B*Hq*n_slots*L. */
int mesh_attn_partials_size(const mesh_attn_plan* plan, int32_t B, int32_t Hq, int32_t d,
                            size_t* o_elems, size_t* lse_elems);

/* Bytes of device workspace mesh_attn_tile_fwd with bf16 inputs, and mesh_attn_merge, need for
 * this plan (the plan's work list, slot offsets and a scheduling counter).  The caller allocates
 * it (16-byte aligned) and may reuse it across calls on one stream; calls that overlap on the GPU
 * need separate workspaces. */
int mesh_attn_workspace_size(const mesh_attn_plan* plan, size_t* bytes);

/* Bytes of device workspace mesh_attn_tile_fwd needs for inputs of `in_dtype` and these sizes:
 * the above for MESH_ATTN_BF16; for MESH_ATTN_F32 also room for the bf16 pieces the fp32 path
 * splits Q, K and V into, 6 * (B*Hq + 2*B*Hkv) * S * d bytes (see mesh_attn_tile_fwd).  Enough for
 * mesh_attn_merge as well. */
int mesh_attn_workspace_size_for(const mesh_attn_plan* plan, mesh_attn_dtype in_dtype, int32_t B,
                                 int32_t Hq, int32_t Hkv, int32_t d, size_t* bytes);

/* Tile attention forward: every (Q partition, tile) item of the plan, for every batch and
 * query head, writes its partial O_t and lse_t (step 2 above).
 *   in_dtype  MESH_ATTN_BF16 (tensor-core kernel: bf16 products, fp32 accumulation, fp32
 *             online softmax, P rounded to bf16 for the PV product) or MESH_ATTN_F32 (tensor-core
 *             kernel with fp32 accuracy: Q, K, V and P are each split exactly into three bf16
 *             pieces x = x1 + x2 + x3 and every product sums the six piece products of order
 *             >= 2^-16, x1y1 + x1y2 + x2y1 + x1y3 + x3y1 + x2y2, with fp32 accumulation; the
 *             pieces go into the workspace, which must then hold mesh_attn_workspace_size_for
 *             bytes).
 *   d         64 or 128.  B >= 0, Hq >= 0, Hkv >= 1, Hq % Hkv == 0.
 *   Q, K, V   device tensors of in_dtype, 16-byte aligned (layouts above).
 *   scale     softmax scale, finite and > 0 (1/sqrt(d) is the usual choice).
 *   partial_o, partial_lse  device fp32 outputs, sizes from mesh_attn_partials_size.
 *   workspace device buffer of at least mesh_attn_workspace_size bytes.
 *   d_status  device status block (see above).
 * Any L >= 1 works: query rows and keys past the end of a partition are masked, and what lies there
 * (another partition, head or batch) never reaches a result.  Inside a partition masked keys get
 * weight 0, and a weight of 0 still multiplies its value, so V (and for the backward calls every tensor)
 * must be finite in the 128-row block of a row's last visible key. */
int mesh_attn_tile_fwd(const mesh_attn_plan* plan, mesh_attn_dtype in_dtype, int32_t B,
                       int32_t Hq, int32_t Hkv, int32_t d, const void* Q, const void* K,
                       const void* V, float scale, float* partial_o, float* partial_lse,
                       void* workspace, size_t workspace_bytes, int32_t* d_status,
                       void* stream);

/* Maximum scratch of mesh_attn_tile_fwd_noalloc: device bytes every GPU that loads the
 * library reserves for it until the process exits. */
#define MESH_ATTN_NOALLOC_SCRATCH_BYTES (4u << 20)

/* Tile attention forward for callers that cannot allocate device memory.  The paper has no
 * counterpart: this is a service of this library.
 * Who needs it: code that runs where it may not call cudaMalloc -- under a framework whose
 * caching allocator already owns the device memory pool (a direct allocation would fail or
 * escape its accounting), inside an allocator or memory-pressure callback, or with a fixed,
 * pre-reserved memory budget -- and so cannot provide the workspace mesh_attn_tile_fwd asks
 * for.  It computes exactly what mesh_attn_tile_fwd computes, with the same arguments minus
 * the workspace; the caller still passes the inputs, the partial outputs and d_status.
 * The plan's work list (and, for fp32 inputs, the bf16 pieces of Q, K and V) goes into one fixed
 * array of MESH_ATTN_NOALLOC_SCRATCH_BYTES inside the library instead.  A call that needs more
 * (a work list of about 2.6 MB for P = 1024 causal; P = 4096 is too large; fp32 inputs above
 * about 4 MB of pieces) returns MESH_ATTN_ERR_WORKSPACE with the size in mesh_attn_last_error().
 * The first call on a device looks up that device's array address (cudaGetSymbolAddress with
 * the device current); make that first call before any stream capture.  No cudaMalloc, cudaFree
 * or other allocating call is made.  All calls on a device share the one array and each call
 * rewrites what the kernel reads from it, so calls that overlap on the GPU (other streams,
 * other host threads) race: serialise them. */
int mesh_attn_tile_fwd_noalloc(const mesh_attn_plan* plan, mesh_attn_dtype in_dtype, int32_t B,
                               int32_t Hq, int32_t Hkv, int32_t d, const void* Q, const void* K,
                               const void* V, float scale, float* partial_o, float* partial_lse,
                               int32_t* d_status, void* stream);

/* LSE merge (step 3): per (batch, head, row) over the slots of the row's partition,
 *   M = max_t lse_t, lse = M + ln sum_t exp(lse_t - M), O = sum_t exp(lse_t - lse) O_t;
 * a row whose slots are all -inf gets O = 0 and lse = -inf.
 *   out_dtype MESH_ATTN_BF16 (O rounded to nearest even) or MESH_ATTN_F32.
 *   partial_o, partial_lse  as written by mesh_attn_tile_fwd (or any values of that layout).
 *   O [B, Hq, S, d] of out_dtype, LSE [B, Hq, S] fp32: device outputs, 16-byte aligned.
 *   workspace, d_status, stream as for mesh_attn_tile_fwd. */
int mesh_attn_merge(const mesh_attn_plan* plan, mesh_attn_dtype out_dtype, int32_t B,
                    int32_t Hq, int32_t d, const float* partial_o, const float* partial_lse,
                    void* O, float* LSE, void* workspace, size_t workspace_bytes,
                    int32_t* d_status, void* stream);

/* ---------------------------------------------------------------- backward pass
 *
 * The pages describe the forward pass; Mesh-Attention is a training method (tutorial: end-to-end
 * training speedups; closing remarks on large-model training), so the backward pass keeps the
 * forward's tile structure.  With the forward's global LSE and an upstream gradient dO:
 *   P_ij = exp(scale q_i.k_j - LSE_i) over the visible keys,  dP_ij = dO_i . v_j,
 *   D_i = dO_i . O_i,  dS_ij = P_ij (dP_ij - D_i),
 *   dQ_i = scale sum_j dS_ij k_j,  dK_j = scale sum_i dS_ij q_i,  dV_j = sum_i P_ij dO_i,
 * a KV head's dK and dV summing over its query heads.  Tile t computes, for each of its work
 * items (p, t), the dQ sums over its KV partitions into the item's partial slot (the forward's
 * slots: summed along the mesh row), and for each of its KV partitions k with a live block, the
 * dK / dV sums over its Q partitions into a KV slot (summed along the mesh column back to k's
 * owner).  Partials are fp32:
 *   dq_partial [B, Hq, n_slots, L, d];  dk_partial, dv_partial [B, Hkv, n_kv_slots, L, d].
 * Call order: mesh_attn_bwd_prep (D), mesh_attn_tile_bwd, mesh_attn_bwd_reduce. */

/* KV slots: kv_slot_off[P + 1] (the slots of KV partition k are kv_slot_off[k] ..
 * kv_slot_off[k+1] - 1, grouped by k, tiles ascending); kv_items[3 i + 0..2] = (k, tile t,
 * kv slot i); the tile's Q partitions with a live block for k, ascending, are
 * q_list[q_off[i] .. q_off[i+1]).  Caller arrays of P + 1, n_kv_slots * 3, n_kv_slots + 1 and
 * n_live_blocks int32; any may be NULL to skip it. */
int mesh_attn_plan_kv_slots(const mesh_attn_plan* plan, int32_t* kv_slot_off, int32_t* kv_items,
                            int32_t* q_off, int32_t* q_list);

/* Element counts of the backward partials: *dq_elems = B*Hq*n_slots*L*d for dq_partial,
 * *dkv_elems = B*Hkv*n_kv_slots*L*d for each of dk_partial and dv_partial. */
int mesh_attn_bwd_partials_size(const mesh_attn_plan* plan, int32_t B, int32_t Hq, int32_t Hkv,
                                int32_t d, size_t* dq_elems, size_t* dkv_elems);

/* Bytes of device workspace mesh_attn_tile_bwd and mesh_attn_bwd_reduce need (both work lists,
 * both slot CSRs, two scheduling counters); caller-allocated, 16-byte aligned, reusable across
 * calls on one stream. */
int mesh_attn_bwd_workspace_size(const mesh_attn_plan* plan, size_t* bytes);

/* D[b, h, i] = sum_e dO[b, h, i, e] * O[b, h, i, e] in fp32 (the row term of dS).
 *   dtype of O and dO: MESH_ATTN_BF16 or MESH_ATTN_F32; O, dO [B, Hq, S, d] 16-byte aligned;
 *   D [B, Hq, S] fp32; d 64 or 128. */
int mesh_attn_bwd_prep(mesh_attn_dtype dtype, int32_t B, int32_t Hq, int64_t S, int32_t d,
                       const void* O, const void* dO, float* D, int32_t* d_status, void* stream);

/* Tile attention backward: the partial gradients above for every batch and head.
 *   in_dtype  MESH_ATTN_BF16 (tensor-core kernels: bf16 products with fp32 accumulation; P and
 *             dS rounded to bf16 for the products that take them) or MESH_ATTN_F32 (CUDA-core
 *             kernels, fp32 throughout).
 *   Q, K, V, dO of in_dtype (dO [B, Hq, S, d]), 16-byte aligned; LSE [B, Hq, S] fp32 as written by
 *   mesh_attn_merge; D from mesh_attn_bwd_prep; scale as in the forward call.
 *   dq_partial, dk_partial, dv_partial: fp32 outputs, sizes from mesh_attn_bwd_partials_size.
 *   Other arguments as for mesh_attn_tile_fwd.  Rows with LSE = -inf contribute nothing. */
int mesh_attn_tile_bwd(const mesh_attn_plan* plan, mesh_attn_dtype in_dtype, int32_t B, int32_t Hq,
                       int32_t Hkv, int32_t d, const void* Q, const void* K, const void* V,
                       const void* dO, const float* LSE, const float* D, float scale,
                       float* dq_partial, float* dk_partial, float* dv_partial, void* workspace,
                       size_t workspace_bytes, int32_t* d_status, void* stream);

/* Sum the backward partials: dQ [B, Hq, S, d] over the slots of each Q partition, dK and dV
 * [B, Hkv, S, d] over the KV slots of each KV partition, rounded to out_dtype (nearest even for
 * bf16).  Outputs 16-byte aligned; other arguments as for mesh_attn_merge. */
int mesh_attn_bwd_reduce(const mesh_attn_plan* plan, mesh_attn_dtype out_dtype, int32_t B,
                         int32_t Hq, int32_t Hkv, int32_t d, const float* dq_partial,
                         const float* dk_partial, const float* dv_partial, void* dQ, void* dK,
                         void* dV, void* workspace, size_t workspace_bytes, int32_t* d_status,
                         void* stream);

/* ---------------------------------------------------------------- rotary positions
 *
 * Rotary positions with several axes (time, height and width of a video, rows and columns of an
 * image, plain text with one), applied to q and k in one launch before the attention calls.
 * The pages leave positions to the model; long-context models rotate q and k.
 * The d columns of a head are `groups` equal groups rotated alike (1; 2 for the halves of a
 * differential head).  Pair i of a group turns by the angle
 *   phi = positions[pair_axis[i]][b][s] * freq[i]:   (x, y) -> (x cos phi - y sin phi,
 *                                                             y cos phi + x sin phi),
 * by -phi with inverse = 1, which is the backward pass (the gradient of q from the gradient of
 * the rotated q).  Pairs are columns (i, i + n_pairs) of the group, or (2 i, 2 i + 1) with
 * adjacent = 1; columns from 2 n_pairs on are copied.  Angles are products modulo a whole turn in
 * 64-bit fixed point: exact in the position, and off by |position| 2^-53 turns at most from the
 * rounding of freq / 2 pi (freq up to 2 pi; in proportion above).
 *   dtype       of q, k and both outputs; 2 <= d <= 1024, d % groups == 0,
 *               1 <= n_pairs <= 256, 2 n_pairs <= d / groups.
 *   q [B, Hq, S, d] with q_strides[3] = the batch, head and token strides in elements (the d
 *   columns are consecutive), and q_out with q_out_strides; k, Hk likewise.  Hq or Hk may be 0 (its
 *   pointers are then not used).  An output may be its input with the same strides; otherwise
 *   nothing may overlap.  Aligned to the element size; accesses are as wide as the addresses, the
 *   strides, the columns of a pair's members and the unrotated columns allow, 16 bytes at most.
 *   freq, pair_axis   HOST arrays of n_pairs: radians a position, finite; axis, 0 .. n_axes - 1
 *                     (n_axes 1 to 8).  Read before the call returns.
 *   positions   device integers of pos_bits 32 or 64, any sign; pos_strides[3] = axis, batch and token
 *               strides in elements (0 repeats, e.g. positions shared by a batch). */
int mesh_attn_rope(mesh_attn_dtype dtype, int32_t B, int64_t S, int32_t d, int32_t Hq, const void* q,
                   const int64_t* q_strides, void* q_out, const int64_t* q_out_strides, int32_t Hk,
                   const void* k, const int64_t* k_strides, void* k_out, const int64_t* k_out_strides,
                   int32_t groups, int32_t n_pairs, int32_t n_axes, const double* freq,
                   const int32_t* pair_axis, int32_t adjacent, int32_t inverse, const void* positions,
                   int32_t pos_bits, const int64_t* pos_strides, void* stream);

/* ---------------------------------------------------------------- differential attention
 *
 * The difference of two softmax maps over one V, with a learned weight lam per query head.  The
 * columns of a head's query and key are two halves, q = [q1 | q2], k = [k1 | k2], of d/2 each:
 *   P_m = softmax(scale q_m k_m^T) over the visible keys,  O_m = P_m V,
 *   O = O_1 - lam O_2,   LSE_m the natural-log row log-sum-exps.
 * The plan gives the sequence's length and the mask (its partitions, which share work between
 * devices, do not matter here); 1/sqrt(d/2) is the usual scale; LSE is [B, Hq, 2, S].  Backward, with D_m = dO . O_m and dP = dO V^T:
 *   dS_1 = P_1 (dP - D_1),  dS_2 = -lam P_2 (dP - D_2),  dV = (P_1 - lam P_2)^T dO,
 *   dq_m = scale dS_m k_m,  dk_m = scale dS_m^T q_m,  dlam_h = - sum over its rows of D_2.
 * lam: lam_n device values of the inputs' type, one per query head (lam_n = Hq) or one for all
 * (lam_n = 1); dlam has the same form, a shared lam's gradient being the sum over the heads.
 * Masked keys get weight 0 in both maps; a weight of 0 still multiplies its value, so V (and for the
 * backward call every tensor) must be finite in the 128-row block of a row's last visible key. */

/* A plan's constant tables for the device: the caller allocates mesh_attn_plan_tables_size bytes
 * of host memory, has mesh_attn_plan_tables_write fill them, and copies them once into a 16-byte
 * aligned device buffer that the differential calls then read (`tables`).  They depend on the
 * plan alone and are never written: any number of calls, streams and captured graphs may share them.
 * A call whose tables are of another plan records MESH_ATTN_ERR_INVALID_ARG in its status block
 * and does nothing else. */
int mesh_attn_plan_tables_size(const mesh_attn_plan* plan, size_t* bytes);
int mesh_attn_plan_tables_write(const mesh_attn_plan* plan, void* out, size_t out_bytes);

/* Bytes of device workspace the differential calls need: the forward's, or with backward = 1
 * enough for both directions.  Caller-allocated, 16-byte aligned, its contents do not matter; calls
 * that overlap on the GPU, captured graphs among them, need workspaces of their own. */
int mesh_attn_diff_workspace_size(const mesh_attn_plan* plan, mesh_attn_dtype dtype, int32_t B,
                                  int32_t Hq, int32_t Hkv, int32_t d, int32_t backward, size_t* bytes);

/* Forward: O [B, Hq, S, d] and LSE [B, Hq, 2, S] (fp32); O2 [B, Hq, S, d], the second map's
 * output, is what the backward call needs beside them and may be NULL.
 *   dtype  MESH_ATTN_BF16 or MESH_ATTN_F32, of Q, K, V, lam, O and O2; arithmetic as in
 *          mesh_attn_tile_fwd.  d 64 or 128, 2 B Hq S < 2^31 (fp32: 6 B Hq S < 2^31).
 *          Everything 16-byte aligned. */
int mesh_attn_diff_fwd(const mesh_attn_plan* plan, const void* tables, mesh_attn_dtype dtype, int32_t B,
                       int32_t Hq, int32_t Hkv, int32_t d, const void* Q, const void* K, const void* V,
                       const void* lam, int32_t lam_n, float scale, void* O, void* O2, float* LSE,
                       void* workspace, size_t workspace_bytes, int32_t* d_status, void* stream);

/* Backward: dQ [B, Hq, S, d], dK, dV [B, Hkv, S, d] and dlam [lam_n], all of dtype, from the
 * forward's O, O2 and LSE and the gradient dO [B, Hq, S, d].  With B, Hq or S of 0 the calls write
 * nothing: what is left of the gradients (dlam; dK and dV where Hq = 0) is the caller's to zero. */
int mesh_attn_diff_bwd(const mesh_attn_plan* plan, const void* tables, mesh_attn_dtype dtype, int32_t B,
                       int32_t Hq, int32_t Hkv, int32_t d, const void* Q, const void* K, const void* V,
                       const void* lam, int32_t lam_n, const void* O, const void* O2, const float* LSE,
                       const void* dO, float scale, void* dQ, void* dK, void* dV, void* dlam,
                       void* workspace, size_t workspace_bytes, int32_t* d_status, void* stream);

/* One new token a sequence over a cache: O [B, Hq, d] and LSE [B, Hq, 2] of q [B, Hq, d] (dense)
 * against the first lens[b] tokens of sequence b's cache, k_cache and v_cache [B, Hkv, T, d] with
 * strides[3] = batch, head and token strides in elements (multiples of 16 bytes; the d columns are
 * consecutive).  The new token's own key and value are in the cache, and counted, already.
 *   lens  device int32 [B], read on the device; 0 gives O = 0 and LSE = -inf.  A length outside
 *         [0, T] records MESH_ATTN_ERR_OUT_OF_RANGE and is taken as the nearer bound.
 * Tokens from lens[b] on are not read.  B <= 4096, T <= 2^30, d 64 or 128.
 *   workspace  mesh_attn_diff_decode_workspace_size bytes for these sizes or larger ones, 16-byte
 *              aligned, ZEROED once by the caller before its first call; every call leaves it ready
 *              for the next, of whatever sizes fit.  Calls that overlap on the GPU need their own.
 * This call does not skip its work on a non-zero status block. */
int mesh_attn_diff_decode_workspace_size(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int64_t T,
                                         size_t* bytes);
int mesh_attn_diff_decode(mesh_attn_dtype dtype, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int64_t T,
                          const void* q, const void* k_cache, const int64_t* k_strides, const void* v_cache,
                          const int64_t* v_strides, const int32_t* lens, const void* lam, int32_t lam_n,
                          float scale, void* O, float* LSE, void* workspace, size_t workspace_bytes,
                          int32_t* d_status, void* stream);

/* ---------------------------------------------------------------- a paged cache
 *
 * Keys and values of many sequences in pages of `page` tokens each: k_pages and v_pages [n_pages, Hkv, page, d] (strides[3] =
 * page, head and row strides in elements; the d columns are consecutive).  Sequence b's token i is row i % page of page
 * table[b * table_stride + i / page].  A call's new tokens stand one sequence after another: sequence b's are the rows
 * offsets[b] .. offsets[b + 1] - 1 (offsets ascend from 0), and they are the last of the lens[b] tokens it then has, so the first of
 * n has the place lens[b] - n.  table, offsets [B + 1] and lens [B] are int32 in device memory and are read there: a captured
 * graph replays with other lengths, tables and offsets.  Rows of the batch from offsets[B] on are left as they are.
 * A place, page or length that does not exist, or offsets that do not ascend, are recorded as MESH_ATTN_ERR_OUT_OF_RANGE. */

/* New tokens into their pages: k rotated (or copied, with n_pairs = 0), v copied, and q rotated into q_out, in one launch.
 *   q, k, v   [N, H, d] with strides[2] = token and head strides in elements, e.g. slices of one projection; q_out [N, Hq, d]
 *             likewise.  Hq may be 0 (q and q_out are then not used).  q_out may be q with the same strides; otherwise nothing may
 *             overlap.  Alignment and widths of accesses as in mesh_attn_rope.  page >= 1, 2 <= d <= 1024.
 *   groups, n_pairs, n_axes, freq, pair_axis, adjacent   as in mesh_attn_rope.
 *   positions  as there, pos_strides[2] = axis and token strides, [axes, N]; or NULL: each token's place in its sequence
 *              (one axis).
 * A token whose place or page does not exist is recorded and left out. */
int mesh_attn_paged_append(mesh_attn_dtype dtype, int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, const void* q,
                           const int64_t* q_strides, void* q_out, const int64_t* q_out_strides, const void* k,
                           const int64_t* k_strides, const void* v, const int64_t* v_strides, int32_t n_pages, int32_t page,
                           void* k_pages, const int64_t* k_page_strides, void* v_pages, const int64_t* v_page_strides,
                           const int32_t* table, int32_t max_pages, int64_t table_stride, const int32_t* offsets,
                           const int32_t* lens, int32_t groups, int32_t n_pairs, int32_t n_axes, const double* freq,
                           const int32_t* pair_axis, int32_t adjacent, const void* positions, int32_t pos_bits,
                           const int64_t* pos_strides, int32_t* d_status, void* stream);

/* Bytes of device workspace mesh_attn_paged_attn needs for at most N new tokens of B sequences, max_new of one of them, and these
 * heads.  Caller-allocated, 16-byte aligned, its first 2,048 bytes zeroed before its first call; calls leave it fit for the next,
 * whatever its sizes.  Calls that overlap on the GPU, captured graphs among them, need workspaces of their own. */
int mesh_attn_paged_workspace_size(mesh_attn_dtype dtype, int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d,
                                   int64_t max_new, size_t* bytes);

/* Attention of the new tokens over their sequences' pages, their own keys among them (append first): token i sees the keys
 * j <= i, with window > 0 those with i - j < window, by the score
 *   x = scale q.k, or cap tanh(scale q.k / cap) with cap > 0;   x -= slopes[h] (i - j) where slopes is not NULL.
 * O [N, Hq, d] and LSE [N, Hq] (natural log, fp32), dense.  q [N, Hq, d] with strides[2] = token and head strides.
 *   max_new   an upper bound of a sequence's new tokens, which picks the kernel; a sequence with more is recorded, and its tokens
 *             from max_new on are left out (those before have their places and results all the same).
 *   slopes    device fp32 [Hq], finite, or NULL.
 *   cap       0, or within 1e-18 and 1e18, as scale / cap is.
 *   dtype     MESH_ATTN_BF16 (P in bf16 for its product; two bf16 pieces with few rows) or MESH_ATTN_F32.  d 64 or 128; page a
 *             multiple of 16; B <= 4096; max_pages * page <= 2^30.  Tensors 16-byte aligned, strides multiples of 16 bytes.
 * Tokens of a page from the sequence's length on, and with a window those before all of its new tokens' windows, never reach a
 * result, NaN or not; values that some new token sees must be finite for all of its sequence's (a weight of 0 still multiplies them).
 * Pages wholly before all new tokens' windows (16 tokens of one, or a power of two that divides the page, at a time) are not read
 * and need not exist.
 * Another page that does not exist is recorded and read as zeros.  MESH_ATTN_ERR_OUT_OF_RANGE in the status block keeps
 * neither the other sequences nor later calls over pages from their work (range-masked and plain attention do nothing where their
 * block holds any error: they want another one).  Another error takes its place; outputs are then not to be used. */
int mesh_attn_paged_attn(mesh_attn_dtype dtype, int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, const void* q,
                         const int64_t* q_strides, int32_t n_pages, int32_t page, const void* k_pages, const int64_t* k_strides,
                         const void* v_pages, const int64_t* v_strides, const int32_t* table, int32_t max_pages,
                         int64_t table_stride, const int32_t* offsets, const int32_t* lens, int64_t max_new, float scale, float cap,
                         const float* slopes, int64_t window, void* O, float* LSE, void* workspace, size_t workspace_bytes,
                         int32_t* d_status, void* stream);

/* ---------------------------------------------------------------- range-masked attention
 *
 * Attention of a dense batch where query i of batch entry b sees the keys lo[b, i] <= j < hi[b, i]: causal attention
 * (0, i + 1), documents packed into one row (the document's start, i + 1), prefixes that see one another (a larger hi), windows (a
 * larger lo), padding (lo >= hi: no key; O = 0, LSE = -inf and no gradients).  Bounds outside 0 .. S are taken as the nearer
 * bound.  Scores are capped and biased by distance on request:
 *   x_ij = scale q_i.k_j, or cap tanh(scale q_i.k_j / cap) with cap > 0;   x_ij -= slopes[h] |i - j| where slopes is not NULL.
 * A cap, and scale / cap, is within 1e-18 and 1e18.
 * Backward, with P = exp(x - LSE), dP = dO V^T, D = dO . O and t = tanh(scale q.k / cap):
 *   dS = P (dP - D) (1 - t^2) (without a cap t = 0),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO;
 * slopes get no gradient.  Masked scores may be infinite or NaN, but a weight of 0 still multiplies its value: V (and for
 * the backward call every tensor, and the sums dO V^T in fp32) must be finite in all rows, those of padding too. */

/* Bytes of device workspace of the calls below: the forward's, or with backward = 1 enough for both directions.
 * Caller-allocated, 16-byte aligned, its contents do not matter; calls that overlap on the GPU, captured graphs among them, need
 * workspaces of their own. */
int mesh_attn_range_workspace_size(mesh_attn_dtype dtype, int32_t B, int32_t Hq, int32_t Hkv, int64_t S, int32_t d,
                                   int32_t backward, size_t* bytes);

/* Forward: O [B, Hq, S, d] and LSE [B, Hq, S] (fp32) of dense Q, K, V.
 *   lo, hi    device int32 [B, S], mask_stride elements from one batch entry to the next (0: one mask for all).
 *   slopes    device fp32 [Hq], finite, or NULL.
 *   dtype     MESH_ATTN_BF16 (tensor cores, P rounded to bf16 for its product) or MESH_ATTN_F32 (CUDA cores).  d 64 or 128;
 *             S <= 2^24, B * Hq * S < 2^30.  Tensors 16-byte aligned. */
int mesh_attn_range_fwd(mesh_attn_dtype dtype, int32_t B, int32_t Hq, int32_t Hkv, int64_t S, int32_t d, const void* Q,
                        const void* K, const void* V, const int32_t* lo, const int32_t* hi, int64_t mask_stride,
                        const float* slopes, float scale, float cap, void* O, float* LSE, void* workspace,
                        size_t workspace_bytes, int32_t* d_status, void* stream);

/* Backward: dQ [B, Hq, S, d], dK and dV [B, Hkv, S, d] of dtype, from the forward's O and LSE and the gradient dO
 * [B, Hq, S, d].  With B, Hq or S of 0 the call writes nothing (dK and dV where Hq = 0 are the caller's to zero). */
int mesh_attn_range_bwd(mesh_attn_dtype dtype, int32_t B, int32_t Hq, int32_t Hkv, int64_t S, int32_t d, const void* Q,
                        const void* K, const void* V, const int32_t* lo, const int32_t* hi, int64_t mask_stride,
                        const float* slopes, const void* O, const float* LSE, const void* dO, float scale, float cap, void* dQ,
                        void* dK, void* dV, void* workspace, size_t workspace_bytes, int32_t* d_status, void* stream);

/* Synchronise `stream`, copy word 0 of the device status block to *out (a mesh_attn_status).
 * Returns MESH_ATTN_ERR_CUDA if the copy or the synchronisation failed. */
int mesh_attn_read_status(const int32_t* d_status, void* stream, int32_t* out);

/* Static description of a status code. */
const char* mesh_attn_status_string(int status);

/* One-line description of the last error returned on the calling thread ("" if none). */
const char* mesh_attn_last_error(void);

/* Upper bound, in nanoseconds, on every device-side wait of later launches (process-wide;
 * default 2e9).  A wait that exceeds it records MESH_ATTN_ERR_DEVICE_TIMEOUT and the kernel
 * drains its copies in flight, frees its tensor memory and returns.  ns >= 0; 0 makes every
 * wait that is not already satisfied give up at once (used to test the error path). */
int mesh_attn_set_wait_limit_ns(int64_t ns);

#ifdef __cplusplus
}
#endif

#endif /* MESH_ATTN_H */
