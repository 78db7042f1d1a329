// C entry points of the short causal convolution: argument checks, the backward's partial sums.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "ss1d_conv.h"
#include "ss2d.h"
#include "ss2d_host.h"

namespace {

using ss2d::conv::Args;

constexpr int64_t kMaxTokens = int64_t(1) << 40;
constexpr int64_t kMaxWidth = int64_t(1) << 24;
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;  // of one launch

struct Span {
  const void* p;
  int64_t bytes;
};

bool off(const void* p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int check_sizes(int64_t B, int64_t L, int64_t S, int64_t D, int64_t KW, int dtype, bool packed) {
  if (dtype != SS2D_F32 && dtype != SS2D_BF16) return SS2D_ERR_UNSUPPORTED;
  if (B < 0 || L < 0 || S < 0 || D < 0 || KW < 1) return SS2D_ERR_SHAPE;
  if (packed ? B != 1 : S != B) return SS2D_ERR_SHAPE;
  if (KW > ss2d::conv::kMaxKW) return SS2D_ERR_UNSUPPORTED;
  if (B >= kMaxTokens || L >= kMaxTokens || S >= kMaxTokens || D > kMaxWidth) return SS2D_ERR_SHAPE;
  int64_t t, n;
  if (!ss2d::host_mul_ok(B, L, &t) || t >= kMaxTokens) return SS2D_ERR_SHAPE;
  if (!ss2d::host_mul_ok(t + S * 7, D, &n) || n > ss2d::kHostMaxElems / 4096) return SS2D_ERR_SHAPE;
  return SS2D_OK;
}

// x's strides and the bytes from its first to past its last element.
int set_rows(Args* a, int64_t* bytes, int64_t B, int64_t L, int64_t D, const int64_t* strides, int64_t e) {
  a->sx = {L * D, D};
  if (strides) a->sx = {strides[0], strides[1]};
  *bytes = 0;
  if (a->sx.b < 0 || a->sx.l < 0) return SS2D_ERR_SHAPE;
  if (B == 0 || L == 0 || D == 0) return SS2D_OK;
  int64_t tb, tl;
  if (!ss2d::host_mul_ok(B - 1, a->sx.b, &tb) || !ss2d::host_mul_ok(L - 1, a->sx.l, &tl) ||
      tb > ss2d::kHostMaxElems / 64 || tl > ss2d::kHostMaxElems / 64)
    return SS2D_ERR_SHAPE;
  *bytes = (tb + tl + D) * e;
  return SS2D_OK;
}

void set_sizes(Args* a, int64_t B, int64_t L, int64_t S, int64_t D, int64_t KW, int dtype, const int32_t* cu,
               bool packed, bool backward) {
  a->q = {cu, S, L, B * L};
  a->D = static_cast<int>(D);
  a->KW = static_cast<int>(KW);
  a->run = ss2d::conv::run_of(packed ? 0 : B, B * L, S, D, static_cast<int>(KW), dtype, backward);
  // a sequence without tokens still hands its state on: one unit of each
  a->units = S == 0 ? 0 : ss2d::unit_count(L, S, B * L, packed, a->run);
}

bool launchable(int64_t units, int64_t D) {
  return units + 8 <= (kMaxThreads - 256 * 4096) / (D + 256);
}

// Whether rows go in pieces of four channels.
bool pieces(const Args& a, int64_t e, std::initializer_list<const void*> data) {
  bool ok = a.D % 4 == 0 && a.sx.b % 4 == 0 && a.sx.l % 4 == 0;
  for (const void* p : data) ok = ok && !off(p, 4 * e);
  return ok;
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

// The states of dense rows without tokens are those before them, in units of the smaller data type.
__global__ __launch_bounds__(256) void k_copy(const uint16_t* from, uint16_t* to, int64_t count) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < count; i += int64_t(gridDim.x) * 256)
    to[i] = from ? from[i] : uint16_t(0);
}
int copy_states(const void* from, void* to, int64_t bytes, hipStream_t st) {
  if (!to || from == to || bytes == 0) return 0;
  const int64_t blocks = std::min<int64_t>((bytes + 511) / 512, 1 << 16);  // a launch's threads stay countable in 32 bits
  hipLaunchKernelGGL(k_copy, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, static_cast<const uint16_t*>(from),
                     static_cast<uint16_t*>(to), bytes / 2);
  return static_cast<int>(hipGetLastError());
}

// Bytes of partial sums, with the blocks along the units for either width of a thread.
int64_t part_bytes(const Args& a) {
  const int64_t blocks = std::max(ss2d::conv::unit_blocks(a, 1), ss2d::conv::unit_blocks(a, ss2d::conv::width_of(true)));
  return static_cast<int64_t>(ss2d::host_align256(size_t(blocks) * (a.KW + 1) * a.D * 4));
}

}  // namespace

extern "C" {

int ss1d_conv_forward(const void* x, const float* conv_w, const float* conv_b, const void* h0,
                      const int32_t* cu_seqlens, void* y, void* ht, int64_t B, int64_t L, int64_t S, int64_t D,
                      int64_t KW, const int64_t* strides, int silu, int dtype, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  int rc = check_sizes(B, L, S, D, KW, dtype, packed);
  if (rc != SS2D_OK) return rc;
  const int64_t e = dtype == SS2D_F32 ? 4 : 2, states = S * (KW - 1) * D * e;
  const bool none = B * L == 0;
  if (D == 0 || S == 0 || (none && !ht)) return SS2D_OK;
  if (!conv_w || (!none && (!x || !y))) return SS2D_ERR_NULL;
  Args a{};
  Span ins[5];
  ins[0].p = x;
  rc = set_rows(&a, &ins[0].bytes, B, L, D, strides, e);
  if (rc != SS2D_OK) return rc;
  for (const void* p : {x, h0, static_cast<const void*>(y), static_cast<const void*>(ht)})
    if (off(p, e)) return SS2D_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(conv_w), static_cast<const void*>(conv_b),
                        static_cast<const void*>(cu_seqlens)})
    if (off(p, 4)) return SS2D_ERR_ALIGN;
  set_sizes(&a, B, L, S, D, KW, dtype, cu_seqlens, packed, false);
  if (!launchable(a.units, D)) return SS2D_ERR_SHAPE;
  ins[1] = {conv_w, D * KW * 4};
  ins[2] = {conv_b, D * 4};
  ins[3] = {cu_seqlens, packed ? (S + 1) * 4 : 0};
  ins[4] = {h0, states};
  const Span outs[] = {{y, B * L * D * e}, {ht, states}};
  const bool in_place = ht && ht == h0;
  if (overlap(outs, 2, ins, in_place ? 4 : 5) != SS2D_OK || (in_place && overlap(outs, 1, ins + 4, 1) != SS2D_OK))
    return SS2D_ERR_ALIAS;
  a.x = x;
  a.w = conv_w;
  a.b = conv_b;
  a.h0 = h0;
  a.y = y;
  a.ht = ht;
  a.silu = silu;
  hipStream_t st = static_cast<hipStream_t>(stream);
  int err = 0;
  if (none && !packed) err = copy_states(h0, ht, states, st);
  else err = ss2d::conv::launch_conv(a, dtype, pieces(a, e, {x, h0, y, ht}), st);
  return err ? ss2d::host_hip_fail(static_cast<hipError_t>(err)) : SS2D_OK;
}

int64_t ss1d_conv_scratch_bytes(int64_t B, int64_t L, int64_t S, int64_t D, int64_t KW, int dtype, int packed) {
  if (check_sizes(B, L, S, D, KW, dtype, packed != 0) != SS2D_OK) return -1;
  Args a{};
  set_sizes(&a, B, L, S, D, KW, dtype, nullptr, packed != 0, true);
  return part_bytes(a);
}

int ss1d_conv_backward(const void* x, const float* conv_w, const float* conv_b, const void* h0,
                       const int32_t* cu_seqlens, const void* dy, const void* dht, void* dx, float* dconv_w,
                       float* dconv_b, void* dh0, void* scratch, int64_t scratch_bytes, int64_t B, int64_t L,
                       int64_t S, int64_t D, int64_t KW, const int64_t* strides, int silu, int dtype,
                       void* stream) {
  const bool packed = cu_seqlens != nullptr;
  int rc = check_sizes(B, L, S, D, KW, dtype, packed);
  if (rc != SS2D_OK) return rc;
  const int64_t e = dtype == SS2D_F32 ? 4 : 2, states = S * (KW - 1) * D * e, wide = B * L * D * e;
  const bool none = B * L == 0;
  if (D == 0) return SS2D_OK;
  if (!conv_w || !dconv_w || (conv_b != nullptr) != (dconv_b != nullptr) || (!none && (!x || !dy || !dx)))
    return SS2D_ERR_NULL;
  Args a{};
  Span ins[7];
  ins[0].p = x;
  rc = set_rows(&a, &ins[0].bytes, B, L, D, strides, e);
  if (rc != SS2D_OK) return rc;
  for (const void* p : {x, h0, dy, dht, static_cast<const void*>(dx), static_cast<const void*>(dh0)})
    if (off(p, e)) return SS2D_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(conv_w), static_cast<const void*>(conv_b),
                        static_cast<const void*>(cu_seqlens), static_cast<const void*>(dconv_w),
                        static_cast<const void*>(dconv_b)})
    if (off(p, 4)) return SS2D_ERR_ALIGN;
  if (off(scratch, 256)) return SS2D_ERR_ALIGN;
  set_sizes(&a, B, L, S, D, KW, dtype, cu_seqlens, packed, true);
  if (!launchable(a.units, D)) return SS2D_ERR_SHAPE;
  const int64_t bytes = part_bytes(a);
  ins[1] = {conv_w, D * KW * 4};
  ins[2] = {conv_b, D * 4};
  ins[3] = {cu_seqlens, packed ? (S + 1) * 4 : 0};
  ins[4] = {h0, states};
  ins[5] = {dy, wide};
  ins[6] = {dht, states};
  const Span outs[] = {{dx, wide}, {dconv_w, D * KW * 4}, {dconv_b, D * 4}, {dh0, states}, {scratch, bytes}};
  rc = overlap(outs, 5, ins, 7);
  if (rc != SS2D_OK) return rc;
  a.x = x;
  a.w = conv_w;
  a.b = conv_b;
  a.h0 = h0;
  a.dy = dy;
  a.dht = dht;
  a.dx = dx;
  a.dw = dconv_w;
  a.db = dconv_b;
  a.dh0 = dh0;
  a.silu = silu;
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(scratch);
  if (!scratch) rc = ss2d::host_scratch_outside_graphs(&ws, size_t(bytes), st);
  else if (scratch_bytes < bytes) rc = SS2D_ERR_SCRATCH;
  if (rc != SS2D_OK) return rc;
  a.parts = reinterpret_cast<float*>(ws);
  const bool vec = pieces(a, e, {x, h0, dy, dht, dx, dh0});
  int err = none && !packed ? copy_states(dht, dh0, states, st) : 0;
  if (!err && a.units > 0) err = ss2d::conv::launch_conv_bwd(a, dtype, vec, st);
  const int64_t blocks = a.units > 0 ? ss2d::conv::unit_blocks(a, ss2d::conv::width_of(vec)) : 0;
  if (!err) err = ss2d::conv::launch_conv_sums(a, blocks, st);
  const hipError_t fe = scratch ? hipSuccess : hipFreeAsync(ws, st);
  if (err) return ss2d::host_hip_fail(static_cast<hipError_t>(err));
  return fe == hipSuccess ? SS2D_OK : ss2d::host_hip_fail(fe);
}

int ss1d_conv_step(const void* x, const float* conv_w, const float* conv_b, void* state, const int32_t* slots,
                   void* y, int64_t B, int64_t T, int64_t S, int64_t D, int64_t KW, const int64_t* strides, int silu,
                   int dtype, void* stream) {
  int rc = check_sizes(B, T, B, D, KW, dtype, false);
  if (rc != SS2D_OK) return rc;
  int64_t n;
  if (S < 0 || S >= kMaxTokens || (!slots && S != B)) return SS2D_ERR_SHAPE;
  if (!ss2d::host_mul_ok(S, (KW - 1) * D, &n) || n > ss2d::kHostMaxElems / 4096) return SS2D_ERR_SHAPE;
  if (D > 0 && B > kMaxThreads / 64 / ((D + 63) / 64)) return SS2D_ERR_SHAPE;
  if (B == 0 || T == 0 || D == 0) return SS2D_OK;
  if (!x || !conv_w || !y || (KW > 1 && S > 0 && !state)) return SS2D_ERR_NULL;
  const int64_t e = dtype == SS2D_F32 ? 4 : 2;
  Args a{};
  Span ins[4];
  ins[0].p = x;
  rc = set_rows(&a, &ins[0].bytes, B, T, D, strides, e);
  if (rc != SS2D_OK) return rc;
  for (const void* p : {x, static_cast<const void*>(state), static_cast<const void*>(y)})
    if (off(p, e)) return SS2D_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(conv_w), static_cast<const void*>(conv_b),
                        static_cast<const void*>(slots)})
    if (off(p, 4)) return SS2D_ERR_ALIGN;
  ins[1] = {conv_w, D * KW * 4};
  ins[2] = {conv_b, D * 4};
  ins[3] = {slots, slots ? B * 4 : 0};
  const Span outs[] = {{y, B * T * D * e}, {state, n * e}};
  rc = overlap(outs, 2, ins, 4);
  if (rc != SS2D_OK) return rc;
  a.q = {nullptr, S, T, B * T};
  a.x = x;
  a.w = conv_w;
  a.b = conv_b;
  a.y = y;
  a.state = state;
  a.slots = {slots, static_cast<int>(B), S};
  a.D = static_cast<int>(D);
  a.KW = static_cast<int>(KW);
  a.silu = silu;
  const int err = ss2d::conv::launch_conv_step(a, dtype, pieces(a, e, {x, state, y}), static_cast<hipStream_t>(stream));
  return err ? ss2d::host_hip_fail(static_cast<hipError_t>(err)) : SS2D_OK;
}

}  // extern "C"
