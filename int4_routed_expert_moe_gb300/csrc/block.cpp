// A whole MoE block in one call: norm, router's gate product, routing, experts
// and shared FFN, norm and residual sum. Host code alone: the parts' own calls
// in a row on one stream.
#include <initializer_list>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

// The workspace. The experts' part stays in one place for every T (its counters
// have to stay zero between calls); the shared FFN's moves with T, so its error
// word is set to 0 by the first norm.
struct BlockWs {
  size_t experts, experts_bytes, shared, shared_bytes, n, logits, ysh, y, total;
};
BlockWs block_ws(const moe_block* b, int T) {
  const size_t H = (size_t)b->shape.hidden;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  BlockWs w = {};
  size_t o = kWorkspaceHeader;
  w.experts = o;
  o += up(w.experts_bytes = moe_forward_workspace_bytes(&b->shape, T, b->top_k, b->experts, MOE_PATH_AUTO));
  w.shared = o;
  if (b->shared_inter) o += up(w.shared_bytes = moe_shared_workspace_bytes(T, b->shape.hidden, b->shared_inter));
  w.n = o; o += up((size_t)T * H * 2);
  w.logits = o; o += up((size_t)T * b->experts * 4);
  w.ysh = o;
  if (b->shared_inter) o += up((size_t)T * H * 2);
  w.y = o; o += up((size_t)T * H * 2);
  w.total = o;
  return w;
}

bool aligned(std::initializer_list<const void*> ps, uintptr_t to) {
  uintptr_t a = 0;
  for (const void* p : ps) a |= reinterpret_cast<uintptr_t>(p);
  return a % to == 0;
}

// Everything that does not depend on the call's buffers.
int check_block(const char* who, const moe_block* b, int stream_type, int T) {
  if (!b) return fail(MOE_ERR_ARG, "%s: NULL block", who);
  if (!valid_shape(&b->shape)) return fail(MOE_ERR_SHAPE, "%s: invalid expert shape", who);
  if (T < 0 || (long long)T * b->top_k > 65536)
    return fail(MOE_ERR_ARG, "%s: need 0 <= T, T * top_k <= 65536 (T=%d top_k=%d)", who, T, b->top_k);
  const int H = b->shape.hidden, Is = b->shared_inter;
  if (b->n_slots < 1) return fail(MOE_ERR_ARG, "%s: n_slots %d", who, b->n_slots);
  int rc = check_route_cfg(who, &b->route, b, MOE_F32, b->experts, 0, b->experts, b->top_k);
  if (rc != MOE_OK) return rc;
  // The parts' own checks, of an empty batch: nothing is enqueued.
  if ((rc = moe_norm(&b->norm, nullptr, stream_type, 0, H, nullptr, b->norm_b, nullptr, nullptr, nullptr, nullptr)) !=
          MOE_OK ||
      (rc = moe_norm_residual(&b->norm, nullptr, nullptr, stream_type, 0, H, nullptr, b->post_b, nullptr,
                              MOE_GATE_NONE, b->scale, b->residual_scale, nullptr, nullptr, nullptr, nullptr, nullptr,
                              nullptr, nullptr)) != MOE_OK)
    return rc;
  if (Is < 0 || (Is > 0 && (Is % 64 || Is > 65536)))
    return fail(MOE_ERR_ARG, "%s: shared_inter must be 0 or a multiple of 64 up to 65536 (%d)", who, Is);
  if (!b->norm_w || !b->gate_w || !b->pool || !b->slot_of || (b->post_b && !b->post_w) ||
      (Is ? !b->shared_g || !b->shared_u || !b->shared_d : b->shared_g || b->shared_u || b->shared_d))
    return fail(MOE_ERR_ARG, "%s: NULL pointer, or a shared weight without shared_inter", who);
  if (!aligned({b->norm_w, b->norm_b, b->post_w, b->post_b, b->gate_w, b->shared_g, b->shared_u, b->shared_d}, 16) ||
      !aligned({b->pool}, 256) || !aligned({b->gate_b, b->route_bias, b->slot_of}, 4))
    return fail(MOE_ERR_ARG, "%s: weights must be 16-byte, the pool 256-byte, biases and slot_of 4-byte aligned", who);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_block_workspace_bytes(const moe_block* b, int T) {
  if (!b || !moe::valid_shape(&b->shape) || T < 0 || b->top_k < 1 || b->top_k > 32 || b->experts < 1 ||
      b->experts > 1024 || b->shared_inter < 0 || b->shared_inter > 65536 || (long long)T * b->top_k > 65536)
    return 0;
  return moe::block_ws(b, T).total;
}

int moe_block_forward(const moe_block* b, void* h, int stream_type, int T, int32_t* ids, float* weights, float* logits,
                      void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "moe_block_forward";
  moe::NvtxRange nvtx_range(who);
  moe::clear_error();
  int rc = moe::check_block(who, b, stream_type, T);
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  if (!h || !ids || !weights || !workspace) return moe::fail(MOE_ERR_ARG, "%s: NULL pointer", who);
  if (!moe::aligned({h, logits}, 16) || !moe::aligned({ids, weights}, 4) || !moe::aligned({workspace}, 256))
    return moe::fail(MOE_ERR_ARG, "%s: h and logits must be 16-byte, ids and weights 4-byte, the workspace 256-byte "
                     "aligned", who);
  const moe::BlockWs w = moe::block_ws(b, T);
  if (workspace_bytes < w.total)
    return moe::fail(MOE_ERR_CAPACITY, "%s: workspace %zu < %zu bytes", who, workspace_bytes, w.total);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto flags = [&](size_t o) { return reinterpret_cast<int32_t*>(ws + o); };
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int H = b->shape.hidden, E = b->experts, Is = b->shared_inter;
  void *n = ws + w.n, *y = ws + w.y, *ysh = Is ? ws + w.ysh : nullptr;
  if (!logits) logits = reinterpret_cast<float*>(ws + w.logits);
  int32_t* shared_flags = Is ? flags(w.shared) : nullptr;
  auto layer = [&](bool check_only) {
    return moe::layer_scored(who, &b->shape, n, &b->route, logits, MOE_F32, E, T, E, b->top_k, b->route_bias, ids,
                             weights, b->pool, b->slot_of, b->n_slots, ysh, y, ws + w.experts, w.experts_bytes,
                             MOE_PATH_AUTO, stream, check_only);
  };
  if ((rc = layer(true)) != MOE_OK) return rc;  // the experts' path has limits of its own
  if ((rc = moe::block_norm_in(&b->norm, h, stream_type, T, H, b->norm_w, b->norm_b, n, shared_flags, st)) != MOE_OK)
    return rc;
  if ((rc = moe_linear(n, H, T, H, b->gate_w, E, b->gate_b, MOE_ACT_NONE, nullptr, 0, logits, MOE_F32, E, workspace,
                       moe::kWorkspaceHeader, stream)) != MOE_OK)
    return rc;
  if (Is && (rc = moe_shared_forward(n, T, H, Is, b->shared_g, b->shared_u, b->shared_d, ysh, ws + w.shared,
                                     w.shared_bytes, stream)) != MOE_OK)
    return rc;
  if ((rc = layer(false)) != MOE_OK) return rc;
  return moe::block_norm_out(&b->norm, y, h, stream_type, T, H, b->post_w, b->post_b, b->scale, b->residual_scale,
                             flags(0), flags(w.experts), shared_flags, st);
}

}  // extern "C"
