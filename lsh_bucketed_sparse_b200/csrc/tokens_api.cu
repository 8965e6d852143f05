// C ABI of the token table, the cross entropy and the expert moves (declared
// in include/lsh_attn.h): argument checks, then the launch.
#include <math.h>

#include "internal.h"
#include "lsh_attn.h"
#include "xent.cuh"

namespace lsh {
namespace {

#define CHECK(x)                 \
  do {                           \
    lsh_status _s = (x);         \
    if (_s != LSH_OK) return _s; \
  } while (0)

constexpr long long kMaxRows = 1ll << 30;
constexpr int kMaxVocab = 1 << 20, kMaxModel = 16384, kMaxExperts = 1023, kMaxTopK = 64;

lsh_status check_row(int d, int dtype, int index_type) {
  if (d < 8 || d > kMaxModel || d % 8)
    return fail(LSH_ERR_INVALID_ARG, "d_model=%d: must be a multiple of 8 in [8, %d]", d,
                kMaxModel);
  if (dtype != LSH_F32 && dtype != LSH_BF16)
    return fail(LSH_ERR_INVALID_ARG, "dtype=%d: must be LSH_F32 or LSH_BF16", dtype);
  if (index_type != LSH_I32 && index_type != LSH_I64)
    return fail(LSH_ERR_INVALID_ARG, "index_type=%d: must be LSH_I32 or LSH_I64", index_type);
  return LSH_OK;
}

lsh_status to_table(const lsh_table* s, TableProblem* p) {
  if (!s) return fail(LSH_ERR_INVALID_ARG, "shape is NULL");
  if (s->rows < 0 || s->rows > kMaxRows)
    return fail(LSH_ERR_INVALID_ARG, "rows=%lld: must be in [0, 2^30]", (long long)s->rows);
  if (s->vocab < 1 || s->vocab > kMaxVocab)
    return fail(LSH_ERR_INVALID_ARG, "vocab=%d: must be in [1, 2^20]", s->vocab);
  CHECK(check_row(s->d_model, s->dtype, s->index_type));
  if (!isfinite(s->scale)) return fail(LSH_ERR_INVALID_ARG, "scale is not finite");
  if (s->flags & ~LSH_FLAG_PORTABLE) return fail(LSH_ERR_INVALID_ARG, "unknown flag bits");
  p->rows = s->rows; p->vocab = s->vocab; p->d = s->d_model;
  p->bf16 = s->dtype == LSH_BF16; p->idx64 = s->index_type == LSH_I64;
  p->portable = (s->flags & LSH_FLAG_PORTABLE) != 0;
  p->scale = s->scale;
  return LSH_OK;
}

lsh_status to_route(const lsh_route* s, RouteProblem* p) {
  if (!s) return fail(LSH_ERR_INVALID_ARG, "shape is NULL");
  if (s->top_k < 1 || s->top_k > kMaxTopK)
    return fail(LSH_ERR_INVALID_ARG, "top_k=%d: must be in [1, %d]", s->top_k, kMaxTopK);
  if (s->tokens < 0 || s->tokens > kMaxRows / s->top_k)
    return fail(LSH_ERR_INVALID_ARG, "tokens=%lld: tokens * top_k must be in [0, 2^30]",
                (long long)s->tokens);
  if (s->n_experts < 1 || s->n_experts > kMaxExperts)
    return fail(LSH_ERR_INVALID_ARG, "n_experts=%d: must be in [1, %d]", s->n_experts,
                kMaxExperts);
  CHECK(check_row(s->d_model, s->dtype, s->index_type));
  if (s->flags) return fail(LSH_ERR_INVALID_ARG, "unknown flag bits");
  p->tokens = s->tokens; p->k = s->top_k; p->experts = s->n_experts; p->d = s->d_model;
  p->bf16 = s->dtype == LSH_BF16; p->idx64 = s->index_type == LSH_I64;
  return LSH_OK;
}

// A buffer of rows of D values: may be NULL with none.
lsh_status check_rows_ptr(const void* ptr, const char* name, long long rows) {
  return check_ptr(ptr, name, rows == 0);
}

// A vector with one value of `size` bytes per row or entry, read value by
// value, so that a slice of one (the targets, a token after the inputs) will do.
lsh_status check_vector(const void* ptr, const char* name, long long rows, size_t size) {
  if (!ptr) return rows == 0 ? LSH_OK : fail(LSH_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(ptr) % size)
    return fail(LSH_ERR_INVALID_ARG, "%s is not aligned to its %zu-byte values", name, size);
  return LSH_OK;
}

lsh_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return LSH_OK;
  CHECK(check_ptr(ws, "workspace"));
  if (reinterpret_cast<uintptr_t>(ws) % 256)
    return fail(LSH_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  if (have < need)
    return fail(LSH_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", have, need);
  return LSH_OK;
}

lsh_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? LSH_OK : cuda_fail(e, what);
}

template <typename Shape, typename Problem>
lsh_status size_query(const Shape* shape, size_t* bytes, lsh_status (*to)(const Shape*, Problem*),
                      size_t (*size)(const Problem&)) {
  Problem p;
  CHECK(to(shape, &p));
  if (!bytes) return fail(LSH_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = size(p);
  return LSH_OK;
}

size_t route_sort_workspace_bytes(const RouteProblem& p) {
  return p.tokens ? key_sort_scratch_bytes(p.entries(), p.experts) : 0;
}

lsh_status check_route_plan(const RouteProblem& p, const int32_t* undo, const int32_t* offsets) {
  CHECK(check_vector(undo, "undo", p.tokens, 4));
  return check_vector(offsets, "offsets", 1, 4);
}

}  // namespace
}  // namespace lsh

using namespace lsh;

extern "C" {

lsh_status lsh_attn_embed(const lsh_table* shape, const void* tokens, const void* table,
                          void* out, void* stream) {
  TableProblem p;
  CHECK(to_table(shape, &p));
  CHECK(check_vector(tokens, "tokens", p.rows, p.idx64 ? 8 : 4));
  CHECK(check_ptr(table, "table"));
  CHECK(check_rows_ptr(out, "out", p.rows));
  return launched(launch_embed(p, tokens, table, out, static_cast<cudaStream_t>(stream)),
                  "embed launch");
}

lsh_status lsh_attn_embed_backward_workspace_size(const lsh_table* shape, size_t* bytes) {
  return size_query(shape, bytes, to_table, embed_backward_workspace_bytes);
}

lsh_status lsh_attn_embed_backward(const lsh_table* shape, const void* tokens, const void* dout,
                                   const void* init, void* dtable, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  TableProblem p;
  CHECK(to_table(shape, &p));
  CHECK(check_vector(tokens, "tokens", p.rows, p.idx64 ? 8 : 4));
  CHECK(check_rows_ptr(dout, "dout", p.rows));
  CHECK(check_ptr(init, "init", true));
  CHECK(check_ptr(dtable, "dtable"));
  CHECK(check_workspace(workspace, workspace_bytes, embed_backward_workspace_bytes(p)));
  return launched(launch_embed_backward(p, tokens, dout, init, dtable, workspace,
                                        static_cast<cudaStream_t>(stream)),
                  "embed backward launch");
}

lsh_status lsh_attn_xent_workspace_size(const lsh_table* shape, size_t* bytes) {
  return size_query(shape, bytes, to_table, xent_workspace_bytes);
}

lsh_status lsh_attn_xent(const lsh_table* shape, const void* x, const void* table,
                         const void* targets, float* loss, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  TableProblem p;
  CHECK(to_table(shape, &p));
  CHECK(check_rows_ptr(x, "x", p.rows));
  CHECK(check_ptr(table, "table"));
  CHECK(check_vector(targets, "targets", p.rows, p.idx64 ? 8 : 4));
  CHECK(check_vector(loss, "loss", p.rows, 4));
  CHECK(check_vector(lse, "lse", p.rows, 4));
  CHECK(check_workspace(workspace, workspace_bytes, xent_workspace_bytes(p)));
  return launched(launch_xent(p, x, table, targets, loss, lse, workspace,
                              static_cast<cudaStream_t>(stream)),
                  "cross entropy launch");
}

lsh_status lsh_attn_xent_backward_workspace_size(const lsh_table* shape, size_t* bytes) {
  return size_query(shape, bytes, to_table, xent_backward_workspace_bytes);
}

lsh_status lsh_attn_xent_backward(const lsh_table* shape, const void* x, const void* table,
                                  const void* targets, const float* lse, const float* dloss,
                                  void* dx, void* dtable, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  TableProblem p;
  CHECK(to_table(shape, &p));
  CHECK(check_rows_ptr(x, "x", p.rows));
  CHECK(check_ptr(table, "table"));
  CHECK(check_vector(targets, "targets", p.rows, p.idx64 ? 8 : 4));
  CHECK(check_vector(lse, "lse", p.rows, 4));
  CHECK(check_vector(dloss, "dloss", p.rows, 4));
  CHECK(check_rows_ptr(dx, "dx", p.rows));
  CHECK(check_ptr(dtable, "dtable"));
  CHECK(check_workspace(workspace, workspace_bytes, xent_backward_workspace_bytes(p)));
  return launched(launch_xent_backward(p, x, table, targets, lse, dloss, dx, dtable, workspace,
                                       static_cast<cudaStream_t>(stream)),
                  "cross entropy backward launch");
}

lsh_status lsh_attn_route_sort_workspace_size(const lsh_route* shape, size_t* bytes) {
  return size_query(shape, bytes, to_route, route_sort_workspace_bytes);
}

lsh_status lsh_attn_route_sort(const lsh_route* shape, const void* experts, int32_t* perm,
                               int32_t* undo, int32_t* offsets, void* workspace,
                               size_t workspace_bytes, void* stream) {
  RouteProblem p;
  CHECK(to_route(shape, &p));
  CHECK(check_vector(experts, "experts", p.tokens, p.idx64 ? 8 : 4));
  CHECK(check_vector(perm, "perm", p.tokens, 4));
  CHECK(check_route_plan(p, undo, offsets));
  CHECK(check_workspace(workspace, workspace_bytes, route_sort_workspace_bytes(p)));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.tokens == 0)
    return launched(cudaMemsetAsync(offsets, 0, (size_t)(p.experts + 1) * sizeof(int32_t), st),
                    "clear offsets");
  KeyOrder o = {};
  o.perm = perm;
  o.undo = undo;
  o.offsets = offsets;
  return launched(launch_key_sort(p.entries(), p.experts, experts, p.idx64, o, workspace, st),
                  "route sort launch");
}

lsh_status lsh_attn_route_gather(const lsh_route* shape, const void* x, const int32_t* undo,
                                 const int32_t* offsets, void* xs, void* stream) {
  RouteProblem p;
  CHECK(to_route(shape, &p));
  CHECK(check_rows_ptr(x, "x", p.tokens));
  CHECK(check_route_plan(p, undo, offsets));
  CHECK(check_rows_ptr(xs, "xs", p.tokens));
  return launched(launch_route_gather(p, x, undo, offsets, xs, static_cast<cudaStream_t>(stream)),
                  "route gather launch");
}

lsh_status lsh_attn_route_gather_backward(const lsh_route* shape, const void* dxs,
                                          const int32_t* undo, const int32_t* offsets, void* dx,
                                          void* stream) {
  RouteProblem p;
  CHECK(to_route(shape, &p));
  CHECK(check_rows_ptr(dxs, "dxs", p.tokens));
  CHECK(check_route_plan(p, undo, offsets));
  CHECK(check_rows_ptr(dx, "dx", p.tokens));
  return launched(launch_route_combine(p, dxs, nullptr, undo, offsets, dx,
                                       static_cast<cudaStream_t>(stream)),
                  "route gather backward launch");
}

lsh_status lsh_attn_route_combine(const lsh_route* shape, const void* y, const float* weights,
                                  const int32_t* undo, const int32_t* offsets, void* out,
                                  void* stream) {
  RouteProblem p;
  CHECK(to_route(shape, &p));
  CHECK(check_rows_ptr(y, "y", p.tokens));
  CHECK(check_vector(weights, "weights", p.tokens, 4));
  CHECK(check_route_plan(p, undo, offsets));
  CHECK(check_rows_ptr(out, "out", p.tokens));
  return launched(launch_route_combine(p, y, weights, undo, offsets, out,
                                       static_cast<cudaStream_t>(stream)),
                  "route combine launch");
}

lsh_status lsh_attn_route_combine_backward(const lsh_route* shape, const void* dout,
                                           const void* y, const float* weights,
                                           const int32_t* undo, const int32_t* offsets, void* dy,
                                           float* dweights, void* stream) {
  RouteProblem p;
  CHECK(to_route(shape, &p));
  CHECK(check_rows_ptr(dout, "dout", p.tokens));
  CHECK(check_rows_ptr(y, "y", p.tokens));
  CHECK(check_vector(weights, "weights", p.tokens, 4));
  CHECK(check_route_plan(p, undo, offsets));
  CHECK(check_rows_ptr(dy, "dy", p.tokens));
  CHECK(check_vector(dweights, "dweights", p.tokens, 4));
  return launched(launch_route_combine_backward(p, dout, y, weights, undo, offsets, dy, dweights,
                                                static_cast<cudaStream_t>(stream)),
                  "route combine backward launch");
}

unsigned long long lsh_attn_test_xent_first_wait(unsigned long long ns) {
  return set_xent_first_wait_ns(ns);
}

unsigned long long lsh_attn_test_xent_piece_bytes(unsigned long long bytes) {
  return set_xent_piece_bytes(bytes);
}

}  // extern "C"
