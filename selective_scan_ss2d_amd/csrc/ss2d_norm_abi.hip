// C entry points of the block norm: argument checks, the backward's partial sums.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "ss2d.h"
#include "ss2d_host.h"
#include "ss2d_norm.h"

namespace {

using ss2d::norm::Args;

struct Span {
  const void* p;
  int64_t bytes;
};

int check(int64_t B, int64_t L, int64_t D, int64_t G, int first, float eps, int dtype, int ytype) {
  if (dtype != SS2D_F32 && dtype != SS2D_BF16) return SS2D_ERR_UNSUPPORTED;
  if (ytype != SS2D_F32 && ytype != dtype) return SS2D_ERR_UNSUPPORTED;
  if (B < 0 || L < 0 || D < 1 || G < 0) return SS2D_ERR_SHAPE;
  if (!std::isfinite(eps) || eps < 0.0f) return SS2D_ERR_UNSUPPORTED;
  if (D > (first ? ss2d::norm::kMaxDFirst : ss2d::norm::kMaxD)) return SS2D_ERR_UNSUPPORTED;
  if (first && L > ss2d::norm::kMaxLFirst) return SS2D_ERR_UNSUPPORTED;
  int64_t rows, n;
  if (!ss2d::host_mul_ok(B, L, &rows) || !ss2d::host_mul_ok(rows, D, &n) ||
      n > ss2d::kHostMaxElems / 64)
    return SS2D_ERR_SHAPE;
  // groups are runs of rows; channels first, of whole images
  if (G > 0 && ((first ? B : rows) % G != 0 || G >= (int64_t(1) << 31))) return SS2D_ERR_SHAPE;
  return SS2D_OK;
}

bool off(const void* p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

void set_shape(Args* a, int64_t B, int64_t L, int64_t D, int64_t G, int first, int layer,
               float eps) {
  a->B = B;
  a->L = L;
  a->D = static_cast<int>(D);
  a->G = G > 0 ? G : 1;
  a->group = (first ? B : B * L) / a->G;
  a->layer = layer;
  a->eps = eps;
}

// The backward's plan, and its scratch: the blocks' sums of the four vectors, and of res_scale's
// gradient where several blocks share a group.  Without rows there are no blocks, and the sums
// over them write zeros.
struct Scratch {
  int64_t blocks;
  size_t parts, bytes;
};
Scratch scratch_layout(Args* a, int first) {
  const bool none = a->B == 0 || a->L == 0;
  Scratch w;
  w.blocks = none ? 0 : ss2d::norm::plan_norm_bwd(a, first != 0);
  if (none) a->blocks_per_group = 0;
  w.parts = ss2d::host_align256(size_t(w.blocks) * ss2d::norm::kSums * a->D * 4);
  w.bytes = w.parts + (a->blocks_per_group > 1 ? size_t(a->G) * a->blocks_per_group * a->D * 4 : 0);
  return w;
}

int overlap(const Span* outs, int n_out, const Span* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (ss2d::host_overlaps(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes))
        return SS2D_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (ss2d::host_overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes))
        return SS2D_ERR_ALIAS;
  }
  return SS2D_OK;
}

}  // namespace

extern "C" {

int ss2d_norm_forward(const void* h, const void* z, const void* residual, const float* res_scale,
                      const float* w_post, const float* b_post, const float* w_pre,
                      const float* b_pre, void* y, void* n, int64_t B, int64_t L, int64_t D,
                      int64_t G, int channels_first, int layer, float eps, int dtype, int ytype,
                      void* stream) {
  int rc = check(B, L, D, G, channels_first, eps, dtype, ytype);
  if (rc != SS2D_OK) return rc;
  if (B == 0 || L == 0) return SS2D_OK;
  if (!h || (!y && !n) || (w_pre != nullptr) != (n != nullptr) || (G > 0) != (res_scale != nullptr) ||
      (b_post && !w_post) || (b_pre && !w_pre))
    return SS2D_ERR_NULL;
  const int64_t e = dtype == SS2D_F32 ? 4 : 2, ye = ytype == SS2D_F32 ? 4 : 2;
  for (const void* p : {h, z, static_cast<const void*>(n)})
    if (off(p, e)) return SS2D_ERR_ALIGN;
  for (const void* p : {residual, static_cast<const void*>(y)})
    if (off(p, ye)) return SS2D_ERR_ALIGN;
  for (const float* p : {res_scale, w_post, b_post, w_pre, b_pre})
    if (off(p, 4)) return SS2D_ERR_ALIGN;
  const int64_t m = B * L * D;
  const Span ins[] = {{h, m * e}, {z, m * e}, {residual, m * ye}, {res_scale, G * D * 4},
                      {w_post, D * 4}, {b_post, D * 4}, {w_pre, D * 4}, {b_pre, D * 4}};
  const Span outs[] = {{y, m * ye}, {n, m * e}};
  // y may replace the residual: every value is read by the thread that writes it, before
  const bool in_place = y && y == residual;
  if (overlap(outs, 2, ins, 2) != SS2D_OK || overlap(outs, 2, ins + 3, 5) != SS2D_OK ||
      overlap(outs + (in_place ? 1 : 0), in_place ? 1 : 2, ins + 2, 1) != SS2D_OK)
    return SS2D_ERR_ALIAS;
  Args a{};
  set_shape(&a, B, L, D, G, channels_first, layer, eps);
  a.h = h;
  a.z = z;
  a.residual = residual;
  a.scale = res_scale;
  a.w_post = w_post;
  a.b_post = b_post;
  a.w_pre = w_pre;
  a.b_pre = b_pre;
  a.y = y;
  a.n = n;
  bool vec = channels_first || D % 8 == 0;
  for (const void* p : {h, z, residual, static_cast<const void*>(y), static_cast<const void*>(n),
                        static_cast<const void*>(res_scale), static_cast<const void*>(w_post),
                        static_cast<const void*>(b_post), static_cast<const void*>(w_pre),
                        static_cast<const void*>(b_pre)})
    vec = vec && !off(p, 16);
  const int err = ss2d::norm::launch_norm(a, dtype, ytype, channels_first != 0, vec,
                                          static_cast<hipStream_t>(stream));
  return err ? ss2d::host_hip_fail(static_cast<hipError_t>(err)) : SS2D_OK;
}

int64_t ss2d_norm_scratch_bytes(int64_t B, int64_t L, int64_t D, int64_t G, int channels_first) {
  if (check(B, L, D, G, channels_first, 0.0f, SS2D_F32, SS2D_F32) != SS2D_OK) return -1;
  Args a{};
  set_shape(&a, B, L, D, G, channels_first, 0, 0.0f);
  return static_cast<int64_t>(scratch_layout(&a, channels_first).bytes);
}

int ss2d_norm_backward(const void* h, const void* z, const float* res_scale, const float* w_post,
                       const float* b_post, const float* w_pre, const void* y, const void* dy,
                       const void* dn, void* dh, void* dz, void* dresidual, float* dres_scale,
                       float* dw_post, float* db_post, float* dw_pre, float* db_pre, int64_t B,
                       int64_t L, int64_t D, int64_t G, int channels_first, int layer, float eps,
                       int dtype, int ytype, void* stream) {
  return ss2d_norm_backward_ws(h, z, res_scale, w_post, b_post, w_pre, y, dy, dn, dh, dz, dresidual, dres_scale,
                               dw_post, db_post, dw_pre, db_pre, nullptr, 0, B, L, D, G, channels_first, layer,
                               eps, dtype, ytype, stream);
}

int ss2d_norm_backward_ws(const void* h, const void* z, const float* res_scale, const float* w_post,
                          const float* b_post, const float* w_pre, const void* y, const void* dy,
                          const void* dn, void* dh, void* dz, void* dresidual, float* dres_scale,
                          float* dw_post, float* db_post, float* dw_pre, float* db_pre, void* scratch,
                          int64_t scratch_bytes, int64_t B, int64_t L, int64_t D, int64_t G,
                          int channels_first, int layer, float eps, int dtype, int ytype,
                          void* stream) {
  int rc = check(B, L, D, G, channels_first, eps, dtype, ytype);
  if (rc != SS2D_OK) return rc;
  const bool none = B == 0 || L == 0;  // the vectors' gradients are then 0
  if (!none && (!h || !dh || (!dy && !dn))) return SS2D_ERR_NULL;
  if ((w_pre != nullptr) != (dw_pre != nullptr) || (w_post != nullptr) != (dw_post != nullptr) ||
      (!none && (w_pre != nullptr) != (dn != nullptr)) || (!none && w_pre && !y) ||
      (!none && (z != nullptr) != (dz != nullptr)) || (G > 0) != (res_scale != nullptr) ||
      (res_scale != nullptr) != (dres_scale != nullptr) || (b_post && !w_post) ||
      (b_post != nullptr) != (db_post != nullptr) || (db_pre && !w_pre))
    return SS2D_ERR_NULL;
  const int64_t e = dtype == SS2D_F32 ? 4 : 2, ye = ytype == SS2D_F32 ? 4 : 2;
  for (const void* p : {h, z, dn, static_cast<const void*>(dh), static_cast<const void*>(dz)})
    if (off(p, e)) return SS2D_ERR_ALIGN;
  for (const void* p : {y, dy, static_cast<const void*>(dresidual)})
    if (off(p, ye)) return SS2D_ERR_ALIGN;
  for (const float* p : {res_scale, w_post, b_post, w_pre, static_cast<const float*>(dres_scale),
                         static_cast<const float*>(dw_post), static_cast<const float*>(db_post),
                         static_cast<const float*>(dw_pre), static_cast<const float*>(db_pre)})
    if (off(p, 4)) return SS2D_ERR_ALIGN;
  if (off(scratch, 256)) return SS2D_ERR_ALIGN;
  Args a{};
  set_shape(&a, B, L, D, G, channels_first, layer, eps);
  const Scratch w = scratch_layout(&a, channels_first);
  const int64_t m = B * L * D;
  const Span ins[] = {{h, m * e}, {z, m * e}, {res_scale, G * D * 4}, {w_post, D * 4},
                      {b_post, D * 4}, {w_pre, D * 4}, {y, m * ye}, {dy, m * ye}, {dn, m * e}};
  const Span outs[] = {{dh, m * e}, {dz, m * e}, {dresidual, m * ye}, {dres_scale, G * D * 4},
                       {dw_post, D * 4}, {db_post, D * 4}, {dw_pre, D * 4}, {db_pre, D * 4},
                       {scratch, static_cast<int64_t>(w.bytes)}};
  rc = overlap(outs, 9, ins, 9);
  if (rc != SS2D_OK) return rc;
  a.h = h;
  a.z = z;
  a.scale = res_scale;
  a.w_post = w_post;
  a.b_post = b_post;
  a.w_pre = w_pre;
  a.y = const_cast<void*>(y);
  a.dy = dy;
  a.dn = dn;
  a.dh = dh;
  a.dz = dz;
  a.dres = dresidual;
  a.dscale = dres_scale;
  a.dw_post = dw_post;
  a.db_post = db_post;
  a.dw_pre = dw_pre;
  a.db_pre = db_pre;
  bool vec = channels_first || D % 8 == 0;
  for (const void* p : {h, z, y, dy, dn, static_cast<const void*>(dh), static_cast<const void*>(dz),
                        static_cast<const void*>(dresidual), static_cast<const void*>(res_scale),
                        static_cast<const void*>(w_post), static_cast<const void*>(b_post),
                        static_cast<const void*>(w_pre)})
    vec = vec && !off(p, 16);
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(scratch);
  if (!scratch) rc = ss2d::host_scratch_outside_graphs(&ws, w.bytes, st);
  else if (scratch_bytes < 0 || size_t(scratch_bytes) < w.bytes) rc = SS2D_ERR_SCRATCH;
  if (rc != SS2D_OK) return rc;
  a.parts = reinterpret_cast<float*>(ws);
  a.scale_parts = a.blocks_per_group == 1 ? dres_scale : reinterpret_cast<float*>(ws + w.parts);
  int err = none ? 0 : ss2d::norm::launch_norm_bwd(a, dtype, ytype, channels_first != 0, vec, st);
  if (!err && (dw_post || dw_pre || dres_scale)) err = ss2d::norm::launch_norm_sums(a, w.blocks, st);
  const hipError_t fe = scratch ? hipSuccess : hipFreeAsync(ws, st);
  if (err) return ss2d::host_hip_fail(static_cast<hipError_t>(err));
  if (fe != hipSuccess) return ss2d::host_hip_fail(fe);
  return SS2D_OK;
}

}  // extern "C"
