// extern "C" entry points of differential attention over a plan (mesh_attn.h): the plan's device
// tables, argument checks, workspace layout and the sequence of launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>

#include "abi_util.h"
#include "internal.h"

namespace mesh {

static size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

TablesLayout tables_layout(const Plan& p) {
  TablesLayout t{};
  size_t at = 64;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = up(at + bytes, 16);
    return o;
  };
  t.flat_item = take(sizeof(DevItem));
  t.flat_list = take(4);
  t.total = at;
  return t;
}

uint64_t plan_tag(const Plan& p) {
  uint64_t h = 1469598103934665603ull;  // FNV-1a over what determines a plan
  for (uint64_t x : {(uint64_t)p.S, (uint64_t)p.P, (uint64_t)p.layout, (uint64_t)(p.causal * 4 + p.kvr * 2 + p.greedy)})
    for (int i = 0; i < 8; ++i) h = (h ^ ((x >> (8 * i)) & 255)) * 1099511628211ull;
  return h;
}

DiffWorkspace diff_workspace(const Plan& plan, mesh_attn_dtype dt, int32_t B, int32_t Hq, int32_t Hkv, int32_t d,
                             bool backward) {
  DiffWorkspace w{};
  size_t at = 512;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = up(at + bytes, 256);
    return o;
  };
  const size_t qrows = (size_t)B * Hq * plan.S;
  const bool f32 = dt == MESH_ATTN_F32;
  const int64_t nb = (plan.S + 127) / 128;
  if (!backward) {
    // fp32: both maps' outputs always go through the merge; bf16: those of tiles cut into parts
    if (const size_t rows = 2 * (f32 ? qrows * diff_fwd32_parts(plan.S, B, Hq)
                                     : (size_t)diff_fwd_max_parts(plan.S, B, Hq, plan.causal) * 128)) {
      w.part_o = take(rows * d * 4);
      w.part_lse = take(rows * 4);
    }
    if (f32) w.pieces = take(f32_pieces_layout(B, 2 * Hq, Hkv, plan.S, d).total);
  } else {
    w.dsum = take(2 * qrows * 4);
    const BwdParts parts = diff_bwd_parts(plan.S, B, Hq, Hkv, plan.causal);
    // per (batch, head): fp32 one sum per 64 rows; bf16 eight per part of a 128-row block
    w.dlam_part = take((size_t)B * Hq * 4 * (size_t)(f32 ? (plan.S + 63) / 64 : nb * 8 * parts.dq));
    const size_t kvrows = (size_t)B * Hkv * plan.S;
    if (f32) {  // partial sums of the splits, and of a KV head's query heads
      w.pieces = take(bwd32_pieces_layout(B, Hq, Hkv, plan.S, d).total);
      const size_t splits = (size_t)diff_bwd32_splits(plan.S, B, Hq, MAX_SMS);  // grows with the SM count
      if (splits > 1) w.dq_part = take(splits * qrows * d * 4);
      if (splits * (Hq / Hkv) > 1) {
        w.dk_part = take(splits * qrows * d * 4);
        w.dv_part = take(splits * qrows * d * 4);
      }
    } else {
      if (parts.dq > 1) w.dq_part = take(parts.dq * qrows * d * 4);
      if (parts.kv > 1) {
        w.dk_part = take(parts.kv * kvrows * d * 4);
        w.dv_part = take(parts.kv * kvrows * d * 4);
      }
    }
  }
  w.total = at;
  return w;
}

}  // namespace mesh

using mesh::DiffArgs;
using mesh::DiffWorkspace;
using mesh::is_aligned;
using mesh::launch_status;
using mesh::set_last_error;

namespace {

int check_sizes(const mesh_attn_plan* plan, mesh_attn_dtype dt, int32_t B, int32_t Hq, int32_t Hkv, int32_t d) {
  if (!plan) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "plan is NULL");
  if (dt != MESH_ATTN_F32 && dt != MESH_ATTN_BF16)
    return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "dtype must be MESH_ATTN_F32 or MESH_ATTN_BF16");
  if (B < 0 || Hq < 0) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "B and Hq must be >= 0");
  if (Hkv < 1 || Hq % Hkv != 0) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "need Hkv >= 1 and Hq % Hkv == 0");
  if (d != 64 && d != 128) return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "d must be 64 or 128");
  if ((int64_t)B * Hq > 0x3fffffff || 2 * (int64_t)B * Hq * plan->p.S >= (int64_t)1 << 31)
    return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "2 * B * Hq * S must be < 2^31");
  if (dt == MESH_ATTN_F32 && 6 * (int64_t)B * Hq * plan->p.S >= (int64_t)1 << 31)
    return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "fp32: 6 * B * Hq * S must be < 2^31");
  return MESH_ATTN_OK;
}

int check_common(const DiffArgs& a, mesh_attn_dtype dt, const void* workspace, size_t workspace_bytes, size_t need) {
  if (!(a.scale > 0.f) || !std::isfinite(a.scale))
    return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (a.lam_n != 1 && a.lam_n != a.Hq) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "lam_n must be 1 or Hq");
  if (!a.Q || !a.K || !a.V || !a.lam || !a.tables || !a.O || !a.LSE || !workspace || !a.status)
    return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "a tensor, tables, workspace or status pointer is NULL");
  for (const void* p : {a.Q, a.K, a.V, (const void*)a.O, (const void*)a.O2, a.tables, workspace})
    if (!is_aligned(p, 16))
      return set_last_error(MESH_ATTN_ERR_MISALIGNED, "tensors, tables and workspace must be 16-byte aligned");
  if (!is_aligned(a.LSE, 4) || !is_aligned(a.status, 4) || !is_aligned(a.lam, dt == MESH_ATTN_BF16 ? 2 : 4))
    return set_last_error(MESH_ATTN_ERR_MISALIGNED, "LSE, lam and status must be aligned to their element size");
  if (workspace_bytes < need)
    return set_last_error(MESH_ATTN_ERR_WORKSPACE, "workspace needs " + std::to_string(need) + " bytes");
  return MESH_ATTN_OK;
}

int sm_count(int* sms) {
  const cudaError_t e = mesh::current_sms(sms);
  if (e != cudaSuccess) return set_last_error(MESH_ATTN_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(e));
  *sms = std::min(*sms, mesh::MAX_SMS);
  return MESH_ATTN_OK;
}

DiffArgs make_args(const mesh_attn_plan* plan, const void* tables, int32_t B, int32_t Hq, int32_t Hkv, int32_t d,
                   const void* Q, const void* K, const void* V, const void* lam, int32_t lam_n, float scale, void* O,
                   void* O2, float* LSE, void* workspace, int32_t* status) {
  const mesh::Plan& pl = plan->p;
  DiffArgs a{};
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.lam = lam;
  a.lam_n = lam_n;
  a.tables = tables;
  a.tl = mesh::tables_layout(pl);
  a.tag = mesh::plan_tag(pl);
  a.status = status;
  a.O = O;
  a.O2 = O2;
  a.LSE = LSE;
  a.ws = static_cast<char*>(workspace);
  a.S = pl.S;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.causal = pl.causal ? 1 : 0;
  a.scale = scale;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.wait_limit_ns = mesh::current_wait_limit_ns();
  return a;
}

}  // namespace

extern "C" {

int mesh_attn_plan_tables_size(const mesh_attn_plan* plan, size_t* bytes) {
  return mesh::guarded_call([&]() -> int {
    if (!plan || !bytes) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "NULL argument");
    *bytes = mesh::tables_layout(plan->p).total;
    return (int)MESH_ATTN_OK;
  });
}

int mesh_attn_plan_tables_write(const mesh_attn_plan* plan, void* out, size_t out_bytes) {
  return mesh::guarded_call([&]() -> int {
    if (!plan || !out) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "NULL argument");
    const mesh::Plan& p = plan->p;
    const mesh::TablesLayout t = mesh::tables_layout(p);
    if (out_bytes < t.total)
      return set_last_error(MESH_ATTN_ERR_WORKSPACE, "tables need " + std::to_string(t.total) + " bytes");
    char* o = static_cast<char*>(out);
    std::memset(o, 0, t.total);
    const mesh::TablesHeader h{mesh::TABLES_MAGIC, mesh::plan_tag(p)};
    std::memcpy(o, &h, sizeof(h));
    auto put = [&](size_t off, const void* src, size_t bytes) {
      if (bytes) std::memcpy(o + off, src, bytes);
    };
    const mesh::DevItem flat{0, 0, 0, 1};
    const int32_t list = 0;  // its KV partition
    put(t.flat_item, &flat, sizeof(flat));
    put(t.flat_list, &list, sizeof(list));
    return (int)MESH_ATTN_OK;
  });
}

int mesh_attn_diff_workspace_size(const mesh_attn_plan* plan, mesh_attn_dtype dtype, int32_t B, int32_t Hq, int32_t Hkv,
                                  int32_t d, int32_t backward, size_t* bytes) {
  return mesh::guarded_call([&]() -> int {
    if (!bytes) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "bytes is NULL");
    if (backward != 0 && backward != 1) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "backward must be 0 or 1");
    const int rc = check_sizes(plan, dtype, B, Hq, Hkv, d);
    if (rc) return rc;
    *bytes = mesh::diff_workspace(plan->p, dtype, B, Hq, Hkv, d, false).total;
    if (backward) *bytes = std::max(*bytes, mesh::diff_workspace(plan->p, dtype, B, Hq, Hkv, d, true).total);
    return (int)MESH_ATTN_OK;
  });
}

int mesh_attn_diff_fwd(const mesh_attn_plan* plan, const void* tables, mesh_attn_dtype dtype, int32_t B, int32_t Hq,
                       int32_t Hkv, int32_t d, const void* Q, const void* K, const void* V, const void* lam,
                       int32_t lam_n, float scale, void* O, void* O2, float* LSE, void* workspace,
                       size_t workspace_bytes, int32_t* d_status, void* stream) {
  return mesh::guarded_call([&]() -> int {
    int rc = check_sizes(plan, dtype, B, Hq, Hkv, d);
    if (rc) return rc;
    if (plan->p.S == 0 || B == 0 || Hq == 0) return (int)MESH_ATTN_OK;
    const DiffArgs a = make_args(plan, tables, B, Hq, Hkv, d, Q, K, V, lam, lam_n, scale, O, O2, LSE, workspace, d_status);
    const DiffWorkspace w = mesh::diff_workspace(plan->p, dtype, B, Hq, Hkv, d, false);
    rc = check_common(a, dtype, workspace, workspace_bytes, w.total);
    if (rc) return rc;
    std::string err;
    if (dtype == MESH_ATTN_BF16) {
      int sms = 0;
      if ((rc = sm_count(&sms))) return rc;
      return launch_status(mesh::launch_diff_fwd_tc(a, w, sms, stream, &err), err);
    }
    // fp32: split into bf16 pieces, one map a head with the other half of its query's columns zero, so
    // that the plain fp32 tile kernel over 2 Hq heads gives both maps; then the merge
    const int32_t parts = mesh::diff_fwd32_parts(a.S, B, Hq);
    if ((rc = launch_status(mesh::launch_diff_split(a, w, stream, &err), err))) return rc;
    mesh::TileArgs t{};
    const char* tb = static_cast<const char*>(tables);
    t.part_o = reinterpret_cast<float*>(a.ws + w.part_o);
    t.part_lse = reinterpret_cast<float*>(a.ws + w.part_lse);
    t.items = reinterpret_cast<const mesh::DevItem*>(tb + a.tl.flat_item);
    t.kv_list = reinterpret_cast<const int32_t*>(tb + a.tl.flat_list);
    t.status = d_status;
    t.S = a.S;
    t.L = a.S;
    t.B = B;
    t.Hq = 2 * Hq;
    t.Hkv = Hkv;
    t.d = d;
    t.P = t.n_items = 1;
    t.n_slots = t.parts = parts;
    t.causal = a.causal;
    t.scale = scale;
    t.scale_log2 = a.scale_log2;
    t.wait_limit_ns = a.wait_limit_ns;
    t.pieces = a.ws + w.pieces;
    t.pieces_ready = true;
    if ((rc = launch_status(mesh::launch_tile_fwd_tc32(t, stream, &err), err))) return rc;
    return launch_status(mesh::launch_diff_merge(a, w, parts, stream, &err), err);
  });
}

int mesh_attn_diff_bwd(const mesh_attn_plan* plan, const void* tables, mesh_attn_dtype dtype, int32_t B, int32_t Hq,
                       int32_t Hkv, int32_t d, const void* Q, const void* K, const void* V, const void* lam,
                       int32_t lam_n, const void* O, const void* O2, const float* LSE, const void* dO, float scale,
                       void* dQ, void* dK, void* dV, void* dlam, void* workspace, size_t workspace_bytes,
                       int32_t* d_status, void* stream) {
  return mesh::guarded_call([&]() -> int {
    int rc = check_sizes(plan, dtype, B, Hq, Hkv, d);
    if (rc) return rc;
    if (plan->p.S == 0 || B == 0 || Hq == 0) return (int)MESH_ATTN_OK;
    DiffArgs a = make_args(plan, tables, B, Hq, Hkv, d, Q, K, V, lam, lam_n, scale, const_cast<void*>(O),
                           const_cast<void*>(O2), const_cast<float*>(LSE), workspace, d_status);
    a.dO = dO;
    a.dQ = dQ;
    a.dK = dK;
    a.dV = dV;
    a.dlam = dlam;
    const DiffWorkspace w = mesh::diff_workspace(plan->p, dtype, B, Hq, Hkv, d, true);
    rc = check_common(a, dtype, workspace, workspace_bytes, w.total);
    if (rc) return rc;
    if (!O2 || !dO || !dQ || !dK || !dV || !dlam)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "O2, dO or a gradient pointer is NULL");
    for (const void* p : {dO, (const void*)dQ, (const void*)dK, (const void*)dV})
      if (!is_aligned(p, 16)) return set_last_error(MESH_ATTN_ERR_MISALIGNED, "gradients must be 16-byte aligned");
    if (!is_aligned(dlam, dtype == MESH_ATTN_BF16 ? 2 : 4))
      return set_last_error(MESH_ATTN_ERR_MISALIGNED, "dlam must be aligned to its element size");
    std::string err;
    if (dtype == MESH_ATTN_BF16) {
      int sms = 0;
      if ((rc = sm_count(&sms))) return rc;
      const mesh::BwdParts parts = mesh::diff_bwd_parts(a.S, B, Hq, Hkv, a.causal != 0);
      if ((rc = launch_status(mesh::launch_diff_prep(a, w, dtype, stream, &err), err))) return rc;
      if ((rc = launch_status(mesh::launch_diff_bwd_tc(a, w, sms, parts, stream, &err), err))) return rc;
      return launch_status(mesh::launch_diff_dlam(a, w, dtype, (a.S + 127) / 128 * 8 * parts.dq, stream, &err), err);
    }
    if ((rc = launch_status(mesh::launch_diff_prep(a, w, dtype, stream, &err), err))) return rc;
    int sms = 0;
    if ((rc = sm_count(&sms))) return rc;
    if ((rc = launch_status(mesh::launch_diff_bwd_tc32(a, w, sms, stream, &err), err))) return rc;
    return launch_status(mesh::launch_diff_dlam(a, w, dtype, (a.S + 63) / 64, stream, &err), err);
  });
}

}  // extern "C"
