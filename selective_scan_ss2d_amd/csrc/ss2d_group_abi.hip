// C entry points of the group norm: argument checks, partial sums.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ss2d.h"
#include "ss2d_group.h"
#include "ss2d_host.h"

namespace {

using ss2d::group::Args;
using ss2d::group::Plan;

struct Span {
  const void* p;
  int64_t bytes;
};

bool off(const void* p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int check(int64_t B, int64_t L, int64_t C, int64_t G, float eps, int dtype) {
  if (dtype != SS2D_F32 && dtype != SS2D_BF16) return SS2D_ERR_UNSUPPORTED;
  if (B < 0 || L < 0 || C < 1 || G < 1 || C % G != 0) return SS2D_ERR_SHAPE;
  if (!std::isfinite(eps) || eps < 0.0f) return SS2D_ERR_UNSUPPORTED;
  if (C > (1 << 20) || L >= (int64_t(1) << 31)) return SS2D_ERR_SHAPE;
  int64_t rows, n;
  if (!ss2d::host_mul_ok(B, L, &rows) || !ss2d::host_mul_ok(std::max(rows, B), C, &n) ||
      n > ss2d::kHostMaxElems / 64)
    return SS2D_ERR_SHAPE;
  // threads of one launch: a join's 64 per group of an image (more only where a thread then has four
  // channels of a chunk or more: below 2^26 in all), a block of 256 per image and 32 channels
  if (B > (int64_t(1) << 25) / G || B > (int64_t(1) << 23) / ((C + 31) / 32)) return SS2D_ERR_SHAPE;
  return SS2D_OK;
}

void set_shape(Args* a, int64_t B, int64_t L, int64_t C, int64_t G, int silu, float eps, int dtype) {
  a->B = B;
  a->L = L;
  a->C = static_cast<int>(C);
  a->G = static_cast<int>(G);
  a->cg = static_cast<int>(C / G);
  a->silu = silu;
  a->eps = eps;
  a->chunk = ss2d::group::chunk_positions(B, L, C, dtype);
  a->chunks = (L + a->chunk - 1) / a->chunk;
}

// Scratch of a plan: the channels' partial sums, statistics where none are given or kept, and the
// backward's group sums.
struct Layout {
  size_t stats, sums, bytes;
};
Layout layout(const Args& a, const Plan& p, bool backward, bool kept) {
  using ss2d::host_align256;
  const size_t pairs = host_align256(size_t(a.B) * a.G * 8);
  Layout w{0, 0, 0};
  const bool whole = p.rows > 0;
  if (!whole || backward) w.stats = host_align256(size_t(a.B) * (whole ? 1 : a.chunks) * 2 * a.C * 4);
  w.sums = w.stats + (whole || kept ? 0 : pairs);
  w.bytes = w.sums + (backward && !whole ? pairs : 0);
  return w;
}

bool pieces(int64_t C, int64_t e, const void* x, const void* y, const void* z) {
  return C % (16 / e) == 0 && !off(x, 16) && !off(y, 16) && !off(z, 16);
}

int overlap(const Span* outs, int n_out, const Span* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (ss2d::host_overlaps(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return SS2D_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (ss2d::host_overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return SS2D_ERR_ALIAS;
  }
  return SS2D_OK;
}

int take_scratch(char** ws, void* scratch, int64_t given, size_t bytes, hipStream_t st) {
  *ws = static_cast<char*>(scratch);
  if (bytes == 0) return SS2D_OK;
  if (!scratch) return ss2d::host_scratch_outside_graphs(ws, bytes, st);
  return given >= 0 && size_t(given) >= bytes ? SS2D_OK : SS2D_ERR_SCRATCH;
}

int finish(char* ws, void* scratch, size_t bytes, int err, hipStream_t st) {
  const hipError_t fe = scratch || bytes == 0 ? hipSuccess : hipFreeAsync(ws, st);
  if (err) return ss2d::host_hip_fail(static_cast<hipError_t>(err));
  return fe == hipSuccess ? SS2D_OK : ss2d::host_hip_fail(fe);
}

}  // namespace

extern "C" {

int64_t ss2d_group_norm_scratch_bytes(int backward, int kept, int64_t B, int64_t L, int64_t C, int64_t G, int dtype) {
  if (check(B, L, C, G, 0.0f, dtype) != SS2D_OK) return -1;
  Args a{};
  set_shape(&a, B, L, C, G, 0, 0.0f, dtype);
  size_t bytes = 0;  // of either width of a thread
  for (bool vec : {false, true}) {
    if (vec && C % (dtype == SS2D_F32 ? 4 : 8) != 0) continue;
    const Plan p = ss2d::group::plan(B, L, C, G, dtype, vec, backward != 0);
    bytes = std::max(bytes, layout(a, p, backward != 0, kept != 0).bytes);
  }
  return static_cast<int64_t>(bytes);
}

int ss2d_group_norm_forward(const void* x, const float* weight, const float* bias, void* y, float* stats,
                            void* scratch, int64_t scratch_bytes, int64_t B, int64_t L, int64_t C, int64_t G,
                            int silu, float eps, int dtype, void* stream) {
  int rc = check(B, L, C, G, eps, dtype);
  if (rc != SS2D_OK) return rc;
  if (B == 0 || (L == 0 && !stats)) return SS2D_OK;
  if (L > 0 && (!x || !y)) return SS2D_ERR_NULL;
  const int64_t e = dtype == SS2D_F32 ? 4 : 2, m = B * L * C;
  if (off(x, e) || off(y, e) || off(weight, 4) || off(bias, 4) || off(stats, 4) || off(scratch, 256))
    return SS2D_ERR_ALIGN;
  Args a{};
  set_shape(&a, B, L, C, G, silu, eps, dtype);
  const Plan p = ss2d::group::plan(B, L, C, G, dtype, pieces(C, e, x, y, nullptr), false);
  const Layout w = layout(a, p, false, stats != nullptr);
  const Span ins[] = {{x, m * e}, {weight, C * 4}, {bias, C * 4}};
  const Span outs[] = {{y, m * e}, {stats, B * G * 8}, {scratch, static_cast<int64_t>(w.bytes)}};
  rc = overlap(outs, 3, ins, 3);
  if (rc != SS2D_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws;
  rc = take_scratch(&ws, scratch, scratch_bytes, w.bytes, st);
  if (rc != SS2D_OK) return rc;
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.set = p.set;
  a.sets = p.rows > 0 ? a.C / p.set : 0;
  a.stats = stats;
  if (p.rows == 0) {
    a.parts = reinterpret_cast<float*>(ws);
    if (!stats) a.stats = reinterpret_cast<float*>(ws + w.stats);
  }
  return finish(ws, scratch, w.bytes, ss2d::group::launch_group(a, p, dtype, st), st);
}

int ss2d_group_norm_backward(const void* x, const float* weight, const float* bias, const float* stats,
                             const void* dy, void* dx, float* dweight, float* dbias, void* scratch,
                             int64_t scratch_bytes, int64_t B, int64_t L, int64_t C, int64_t G, int silu, float eps,
                             int dtype, void* stream) {
  int rc = check(B, L, C, G, eps, dtype);
  if (rc != SS2D_OK) return rc;
  const bool none = B == 0 || L == 0;  // the vectors' gradients are then 0
  if ((!none && (!x || !dy || !dx)) || (weight != nullptr) != (dweight != nullptr) ||
      (bias != nullptr) != (dbias != nullptr))
    return SS2D_ERR_NULL;
  const int64_t e = dtype == SS2D_F32 ? 4 : 2, m = B * L * C;
  for (const void* p : {x, dy, static_cast<const void*>(dx)})
    if (off(p, e)) return SS2D_ERR_ALIGN;
  for (const float* p : {weight, bias, stats, static_cast<const float*>(dweight), static_cast<const float*>(dbias)})
    if (off(p, 4)) return SS2D_ERR_ALIGN;
  if (off(scratch, 256)) return SS2D_ERR_ALIGN;
  Args a{};
  set_shape(&a, B, L, C, G, silu, eps, dtype);
  const Plan p = ss2d::group::plan(B, L, C, G, dtype, pieces(C, e, x, dy, dx), true);
  const Layout w = layout(a, p, true, stats != nullptr);
  const Span ins[] = {{x, m * e}, {weight, C * 4}, {bias, C * 4}, {stats, B * G * 8}, {dy, m * e}};
  const Span outs[] = {{dx, m * e}, {dweight, C * 4}, {dbias, C * 4}, {scratch, static_cast<int64_t>(w.bytes)}};
  rc = overlap(outs, 4, ins, 5);
  if (rc != SS2D_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws;
  rc = take_scratch(&ws, scratch, scratch_bytes, w.bytes, st);
  if (rc != SS2D_OK) return rc;
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.dy = dy;
  a.dx = dx;
  a.dw = dweight;
  a.db = dbias;
  a.given = stats != nullptr;
  a.set = p.set;
  a.sets = p.rows > 0 ? a.C / p.set : 0;
  a.parts = reinterpret_cast<float*>(ws);
  a.stats = stats ? const_cast<float*>(stats) : reinterpret_cast<float*>(ws + w.stats);
  a.sums = reinterpret_cast<float*>(ws + w.sums);
  return finish(ws, scratch, w.bytes, ss2d::group::launch_group_bwd(a, p, dtype, st), st);
}

}  // extern "C"
