// C entry points of the gated delta rule: argument checks, scratch and the kernel sequence.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ss1d_delta.h"
#include "ss1d_delta_step.h"
#include "ss2d.h"
#include "ss2d_host.h"

namespace {

using ss2d::delta::Args;
using ss2d::delta::Strides;

// Segment length that a test forces on its own thread (ss1d_delta_set_segment); -1: the rule's.
thread_local int64_t g_segment_override = -1;

constexpr int64_t kMaxTokens = int64_t(1) << 40;
constexpr int64_t kMaxLine = int64_t(1) << 24;    // elements from one token's row to the next
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;  // of one launch

struct Span {  // the memory of one argument
  const void* p;
  int64_t bytes;
};

// Bytes from the first to past the last element of a strided (B, L, H, D) tensor; -1 where
// the strides or the size are out of range.
int64_t strided_bytes(int64_t B, int64_t L, int64_t H, int64_t D, const Strides& s, int64_t e) {
  if (s.b < 0 || s.l < 0 || s.h < 0) return -1;
  if (B == 0 || L == 0 || H == 0 || D == 0) return 0;
  int64_t tb, tl, th;
  if (!ss2d::host_mul_ok(B - 1, s.b, &tb) || !ss2d::host_mul_ok(L - 1, s.l, &tl) ||
      !ss2d::host_mul_ok(H - 1, s.h, &th))
    return -1;
  const int64_t last = tb + tl + th + D;  // each term is below 2^62; so is what is allowed
  if (tb > ss2d::kHostMaxElems / 8 || tl > ss2d::kHostMaxElems / 8 ||
      th > ss2d::kHostMaxElems / 8)
    return -1;
  return last * e;
}

void default_strides(int64_t L, int64_t H, int64_t D, Strides* s) { *s = {L * H * D, H * D, D}; }

bool aligned_rows(const void* p, const Strides& s, int64_t D, int64_t e) {
  const int64_t unit = 16 / e;
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && s.b % unit == 0 && s.l % unit == 0 &&
         s.h % unit == 0 && D % 8 == 0;
}

int check_sizes(int64_t B, int64_t L, int64_t S, int64_t HK, int64_t H, int64_t DK, int64_t DV,
                int dtype, bool packed) {
  if (dtype != SS2D_F32 && dtype != SS2D_BF16) return SS2D_ERR_UNSUPPORTED;
  if (B < 0 || L < 0 || S < 0 || HK < 1 || H < 0 || DK < 1 || DV < 1) return SS2D_ERR_SHAPE;
  if (H % HK != 0) return SS2D_ERR_SHAPE;
  if (packed ? B != 1 : S != B) return SS2D_ERR_SHAPE;
  if (DK > ss2d::delta::kMaxDK) return SS2D_ERR_UNSUPPORTED;
  if (B >= kMaxTokens || L >= kMaxTokens || S >= kMaxTokens || H >= (1 << 20) ||
      DV >= (1 << 20))
    return SS2D_ERR_SHAPE;
  int64_t t, n;
  if (!ss2d::host_mul_ok(B, L, &t) || t >= kMaxTokens) return SS2D_ERR_SHAPE;
  if (!ss2d::host_mul_ok(t, H * DV, &n) || n > ss2d::kHostMaxElems / 64) return SS2D_ERR_SHAPE;
  if (!ss2d::host_mul_ok(S, H * DK * DV, &n) || n > ss2d::kHostMaxElems / 64)
    return SS2D_ERR_SHAPE;
  return SS2D_OK;
}

int64_t slot_count(int64_t L, int64_t S, int64_t T, bool packed, int64_t unit) {
  return packed ? T / unit + S : S * ((L + unit - 1) / unit);
}

// Chunks per segment, 0 for whole sequences.  A segmented forward does the state's recurrence
// about 2.5 times (M and Z, then the run), so it pays where most of the chip is idle otherwise.
// Dense sequences are cut below 320 waves, of the chip's 1024 SIMDs.  Forward and training step,
// time in segments over time whole, 29 shapes of 32 to 512 chunks, widths 32 to 128, both types:
//   144 to 256 waves   0.59 to 0.89   (8 x 1024 tokens of 16 heads of 64: 107 against 120 us)
//   288                0.92, 0.97
//   320 to 384         0.83 to 1.28, on average 1.04 (shorter ones lose, the longest win)
//   512                0.92 to 1.24, on average 1.06
// Packed sequences, the longest of which the others wait for, below 1024: 25 prompts of 12007
// tokens and 8 heads, 600 waves, take 441 us whole and 190 us in segments.  The segments are
// made long enough for about one wave per SIMD (1024), and no shorter than 8 chunks or
// sqrt(C / 4) of the C chunks of a row, because the join runs through them one by one.  4096
// tokens of 32 heads of 128: 304, 249, 253 and 221 us with 6, 8, 12 and 16 chunks (the rule
// gives 16); 2 x 65536 fp32 tokens of 3 heads of 64: 755, 617, 608 and 675 us with 12, 16, 24
// and 32 (24).  Even, so that blocks of 64 tokens do not straddle them.
int64_t segment_chunks(int64_t L, int64_t S, int64_t T, int64_t H, int64_t DV, bool packed) {
  using ss2d::delta::kC;
  if (T == 0) return 0;
  if (g_segment_override >= 0) return g_segment_override;
  const int64_t chunks = (L + kC - 1) / kC, tiles = (DV + 31) / 32;
  const int64_t waves = S * H * tiles, total = (T / kC + (packed ? S : 0)) * H * tiles;
  if (waves >= (packed ? 1024 : 320)) return 0;
  int64_t len = std::max<int64_t>(8, (total + 1023) / 1024);
  len = std::max<int64_t>(len, static_cast<int64_t>(std::ceil(std::sqrt(static_cast<double>(chunks) / 4))));
  len += len & 1;
  return 2 * len <= chunks ? len : 0;
}

int key_tiles(int64_t DK) { return DK <= 32 ? 1 : (DK <= 64 ? 2 : 4); }

// The state a training forward keeps: the marks, the end states, t and o in fp32, and the
// segments' transposed matrices.
struct Saved {
  int64_t marks, ends, rows, spans, bytes;
};
Saved saved_layout(int64_t L, int64_t S, int64_t T, int64_t H, int64_t DK, int64_t DV,
                   bool packed) {
  Saved s;
  s.marks = static_cast<int64_t>(ss2d::host_align256(
      size_t(slot_count(L, S, T, packed, ss2d::delta::kMark)) * H * DK * DV * 4));
  s.ends = static_cast<int64_t>(ss2d::host_align256(size_t(S) * H * DK * DV * 4));
  s.rows = static_cast<int64_t>(ss2d::host_align256(size_t(T) * H * DV * 4));
  const int64_t len = segment_chunks(L, S, T, H, DV, packed);
  s.spans = len ? static_cast<int64_t>(ss2d::host_align256(
                      size_t(slot_count(L, S, T, packed, len * ss2d::delta::kC)) * H *
                      ss2d::delta::matrix_bytes(key_tiles(DK))))
                : 0;
  s.bytes = s.marks + s.ends + 2 * s.rows + s.spans;
  return s;
}
void set_saved(Args* a, void* saved, const Saved& s) {
  char* at = static_cast<char*>(saved);
  a->marks = reinterpret_cast<float*>(at);
  a->ends = reinterpret_cast<float*>(at + s.marks);
  a->ts = reinterpret_cast<float*>(at + s.marks + s.ends);
  a->os = reinterpret_cast<float*>(at + s.marks + s.ends + s.rows);
  a->span_t = at + s.marks + s.ends + 2 * s.rows;
}

int check_pointers(const Span* ins, int n_in, const Span* outs, int n_out) {
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

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

struct Scratch {
  size_t keys, heads, z, starts, m, bytes;
};
Scratch scratch_layout(const Args& a, int dtype) {
  using namespace ss2d::delta;
  const int kt = key_tiles(a.DK);
  const bool f32 = dtype == SS2D_F32;
  Scratch s{};
  s.keys = 0;
  s.heads = size_t(a.slots) * a.HK * key_planes(f32, kt) * kPlane;
  s.z = ss2d::host_align256(s.heads + size_t(a.slots) * a.H * head_planes(f32, a.p_planes) * kPlane +
                            kReadPast);
  const size_t segments = size_t(a.seg_slots) * a.H * a.DK * 4;
  s.starts = s.z + ss2d::host_align256(segments * a.DV);
  s.m = s.starts + ss2d::host_align256(segments * a.DV);
  s.bytes = s.m + size_t(a.seg_slots) * a.H * matrix_bytes(kt);
  return s;
}

// What follows from the sizes alone.
void set_sizes(Args* a, int64_t B, int64_t L, int64_t S, int64_t HK, int64_t H, int64_t DK, int64_t DV,
               bool packed) {
  const int64_t T = B * L;
  a->S = S;
  a->L = L;
  a->T = T;
  a->H = static_cast<int>(H);
  a->HK = static_cast<int>(HK);
  a->rep = static_cast<int>(H / HK);
  a->DK = static_cast<int>(DK);
  a->DV = static_cast<int>(DV);
  a->slots = slot_count(L, S, T, packed, ss2d::delta::kC);
  a->marks_n = slot_count(L, S, T, packed, ss2d::delta::kMark);
  a->seglen = segment_chunks(L, S, T, H, DV, packed);
  a->seg_slots = a->seglen ? slot_count(L, S, T, packed, a->seglen * ss2d::delta::kC) : 0;
}

// The inputs of the forward and the backward: checks them and fills `a`; the spans of the
// inputs go to ins[0..5].
int set_inputs(Args* a, Span* ins, const void* q, const void* k, const void* v, const float* g,
               const float* beta, const float* h0, const int32_t* cu, int64_t B, int64_t L,
               int64_t S, int64_t HK, int64_t H, int64_t DK, int64_t DV, const int64_t* strides,
               float scale, int dtype) {
  const int64_t T = B * L, e = dtype == SS2D_F32 ? 4 : 2;
  set_sizes(a, B, L, S, HK, H, DK, DV, cu != nullptr);
  a->q = q;
  a->k = k;
  a->v = v;
  a->g = g;
  a->beta = beta;
  a->h0 = h0;
  a->cu = cu;
  default_strides(L, HK, DK, &a->sq);
  default_strides(L, HK, DK, &a->sk);
  default_strides(L, H, DV, &a->sv);
  if (strides) {
    a->sq = {strides[0], strides[1], strides[2]};
    a->sk = {strides[3], strides[4], strides[5]};
    a->sv = {strides[6], strides[7], strides[8]};
  }
  a->scale = scale;
  const int64_t qb = strided_bytes(B, L, HK, DK, a->sq, e),
                kb = strided_bytes(B, L, HK, DK, a->sk, e),
                vb = strided_bytes(B, L, H, DV, a->sv, e);
  if (qb < 0 || kb < 0 || vb < 0) return SS2D_ERR_SHAPE;
  // the kernels keep a chunk's row offsets in 32 bits
  if (a->sv.l > kMaxLine || H * DV > kMaxLine || HK * DK > kMaxLine) return SS2D_ERR_UNSUPPORTED;
  for (const void* p : {q, k, v})
    if (misaligned(p, static_cast<uintptr_t>(e))) return SS2D_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(g), static_cast<const void*>(beta),
                        static_cast<const void*>(h0), static_cast<const void*>(cu)})
    if (misaligned(p, 4)) return SS2D_ERR_ALIGN;
  ins[0] = {q, qb};
  ins[1] = {k, kb};
  ins[2] = {v, vb};
  ins[3] = {g, T * H * 4};
  ins[4] = {beta, T * H * 4};
  ins[5] = {cu, (S + 1) * 4};
  const int64_t tiles = (DV + 31) / 32;
  const int64_t units = a->seglen ? a->seg_slots : S;
  if ((a->slots * H / 4 + 1) * 256 > kMaxThreads ||
      std::max(units, S) * H > kMaxThreads / ((tiles + 8) * 64) ||
      a->marks_n * HK * 64 * ss2d::delta::kGradWaves > kMaxThreads || (a->marks_n * H / 4 + 1) * 256 > kMaxThreads)
    return SS2D_ERR_SHAPE;
  return SS2D_OK;
}

// The backward's: the chunk matrices (first the forward's where nothing was kept, then the
// backward's in their place), the states' gradients and dv in fp32, the gates' partial sums, and
// what a forward keeps where nothing was.
struct BackwardScratch {
  Scratch chunks;
  size_t dmarks, dvs, pbeta, pgate, pdots, keep, unused_o, bytes;
};
BackwardScratch backward_layout(const Args& a, int dtype, bool kept, bool packed) {
  using ss2d::host_align256;
  const int64_t tiles = (a.DV + 31) / 32, e = dtype == SS2D_F32 ? 4 : 2;
  const size_t rows = size_t(a.T) * a.H, marks = size_t(a.marks_n) * a.H;
  BackwardScratch w;
  w.chunks = scratch_layout(a, dtype);
  w.dmarks = host_align256(w.chunks.bytes);
  w.dvs = w.dmarks + host_align256(marks * a.DK * a.DV * 4);
  w.pbeta = w.dvs + (dtype == SS2D_F32 ? 0 : host_align256(rows * a.DV * 4));
  w.pgate = w.pbeta + host_align256(tiles * rows * 4);
  w.pdots = w.pgate + host_align256(tiles * rows * 4);
  w.keep = w.pdots + host_align256(marks * tiles * 4);
  w.unused_o = w.keep + (kept ? 0 : size_t(saved_layout(a.L, a.S, a.T, a.H, a.DK, a.DV, packed).bytes));
  w.bytes = w.unused_o + (kept ? 0 : host_align256(rows * a.DV * e));
  return w;
}

// The caller's scratch, or the library's (`own`), which hip records as nodes of their own in a
// captured graph: refused there.
struct Workspace {
  char* at = nullptr;
  bool own = false;
};
int take_scratch(Workspace* w, void* given, int64_t given_bytes, size_t bytes, hipStream_t st) {
  if (given) {
    w->at = static_cast<char*>(given);
    return given_bytes >= 0 && size_t(given_bytes) >= bytes ? SS2D_OK : SS2D_ERR_SCRATCH;
  }
  w->own = true;
  return ss2d::host_scratch_outside_graphs(&w->at, bytes, st);
}
int finish(const Workspace& w, int err, hipStream_t st) {
  const hipError_t fe = w.own ? hipFreeAsync(w.at, st) : hipSuccess;
  if (err) return ss2d::host_hip_fail(static_cast<hipError_t>(err));
  return fe == hipSuccess ? SS2D_OK : ss2d::host_hip_fail(fe);
}

bool aligned_keys(const Args& a, int64_t e) {
  return aligned_rows(a.q, a.sq, a.DK, e) && aligned_rows(a.k, a.sk, a.DK, e);
}

void set_scratch(Args* a, char* ws, const Scratch& w) {
  a->keys = ws + w.keys;
  a->heads = ws + w.heads;
  a->span_z = reinterpret_cast<float*>(ws + w.z);
  a->starts = reinterpret_cast<float*>(ws + w.starts);
  a->span_m = ws + w.m;
}

int run_forward(const Args& a, int dtype, bool save, hipStream_t st) {
  const bool al = aligned_keys(a, dtype == SS2D_F32 ? 4 : 2);
  int err = a.slots > 0 ? ss2d::delta::launch_prep(a, dtype, al, false, st) : 0;
  if (!err && a.seglen) err = ss2d::delta::launch_span(a, dtype, st);
  if (!err && a.seglen) err = ss2d::delta::launch_join(a, false, st);
  return err ? err : ss2d::delta::launch_scan(a, dtype, save, st);
}

}  // namespace

extern "C" {

int ss1d_delta_set_segment(int64_t chunks) {
  if (chunks < -1 || chunks > (1 << 20) || (chunks > 0 && chunks % 2 != 0)) return SS2D_ERR_SHAPE;
  g_segment_override = chunks;
  return SS2D_OK;
}

int64_t ss1d_delta_saved_bytes(int64_t B, int64_t L, int64_t S, int64_t H, int64_t DK, int64_t DV,
                               int packed) {
  if (check_sizes(B, L, S, 1, H, DK, DV, SS2D_BF16, packed != 0) != SS2D_OK) return -1;
  return saved_layout(L, S, B * L, H, DK, DV, packed != 0).bytes;
}

int64_t ss1d_delta_scratch_bytes(int backward, int kept, int64_t B, int64_t L, int64_t S, int64_t HK,
                                 int64_t H, int64_t DK, int64_t DV, int dtype, int packed) {
  if (check_sizes(B, L, S, HK, H, DK, DV, dtype, packed != 0) != SS2D_OK) return -1;
  Args a{};
  set_sizes(&a, B, L, S, HK, H, DK, DV, packed != 0);
  a.p_planes = backward || kept ? 3 : 2;
  const size_t bytes = backward ? backward_layout(a, dtype, kept != 0, packed != 0).bytes
                                : scratch_layout(a, dtype).bytes;
  return static_cast<int64_t>(bytes);
}

int ss1d_delta_forward(const void* q, const void* k, const void* v, const float* g,
                       const float* beta, const float* h0, const int32_t* cu_seqlens, void* o,
                       float* ht, void* saved, int64_t B, int64_t L, int64_t S, int64_t HK,
                       int64_t H, int64_t DK, int64_t DV, const int64_t* strides, float scale,
                       int dtype, void* stream) {
  return ss1d_delta_forward_ws(q, k, v, g, beta, h0, cu_seqlens, o, ht, saved, nullptr, 0, B, L, S, HK, H, DK,
                               DV, strides, scale, dtype, stream);
}

int ss1d_delta_forward_ws(const void* q, const void* k, const void* v, const float* g,
                          const float* beta, const float* h0, const int32_t* cu_seqlens, void* o,
                          float* ht, void* saved, void* scratch, int64_t scratch_bytes, int64_t B,
                          int64_t L, int64_t S, int64_t HK, int64_t H, int64_t DK, int64_t DV,
                          const int64_t* strides, float scale, int dtype, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  int rc = check_sizes(B, L, S, HK, H, DK, DV, dtype, packed);
  if (rc != SS2D_OK) return rc;
  if (!std::isfinite(scale)) return SS2D_ERR_UNSUPPORTED;
  if (S == 0 || H == 0) return SS2D_OK;
  const int64_t T = B * L, e = dtype == SS2D_F32 ? 4 : 2;
  if (T > 0 && (!q || !k || !v || !g || !beta || !o)) return SS2D_ERR_NULL;
  if (T == 0 && !ht) return SS2D_OK;
  Args a{};
  Span ins[6];
  rc = set_inputs(&a, ins, q, k, v, g, beta, h0, cu_seqlens, B, L, S, HK, H, DK, DV, strides, scale,
                  dtype);
  if (rc != SS2D_OK) return rc;
  a.o = o;
  a.ht = ht;
  if (misaligned(o, static_cast<uintptr_t>(e)) || misaligned(ht, 4) || misaligned(saved, 256) ||
      misaligned(scratch, 256))
    return SS2D_ERR_ALIGN;
  const int64_t state = S * H * DK * DV * 4;
  const Saved sv = saved_layout(L, S, T, H, DK, DV, packed);
  a.p_planes = saved ? 3 : 2;
  const Scratch w = scratch_layout(a, dtype);
  const Span outs[] = {{o, T * H * DV * e}, {ht, state}, {saved, sv.bytes},
                       {scratch, static_cast<int64_t>(w.bytes)}};
  rc = check_pointers(ins, 6, outs, 4);
  if (rc != SS2D_OK) return rc;
  // the end states may replace the initial ones: each wave reads its columns first, several
  // segments of a sequence read the join's copy
  const Span first[] = {{h0, state}};
  for (const Span& x : outs)
    if (!(x.p == ht && ht == h0) && check_pointers(first, 1, &x, 1) != SS2D_OK)
      return SS2D_ERR_ALIAS;

  hipStream_t st = static_cast<hipStream_t>(stream);
  Workspace ws;
  rc = take_scratch(&ws, scratch, scratch_bytes, w.bytes, st);
  if (rc != SS2D_OK) return rc;
  set_scratch(&a, ws.at, w);
  if (saved) set_saved(&a, saved, sv);
  return finish(ws, run_forward(a, dtype, saved != nullptr, st), st);
}

int ss1d_delta_backward(const void* q, const void* k, const void* v, const float* g,
                        const float* beta, const float* h0, const int32_t* cu_seqlens,
                        const void* saved, const void* dout, const float* dht, void* dq, void* dk,
                        void* dv, float* dg, float* dbeta, float* dh0, int64_t B, int64_t L,
                        int64_t S, int64_t HK, int64_t H, int64_t DK, int64_t DV,
                        const int64_t* strides, float scale, int dtype, void* stream) {
  return ss1d_delta_backward_ws(q, k, v, g, beta, h0, cu_seqlens, saved, dout, dht, dq, dk, dv, dg, dbeta, dh0,
                                nullptr, 0, B, L, S, HK, H, DK, DV, strides, scale, dtype, stream);
}

int ss1d_delta_backward_ws(const void* q, const void* k, const void* v, const float* g,
                           const float* beta, const float* h0, const int32_t* cu_seqlens,
                           const void* saved, const void* dout, const float* dht, void* dq, void* dk,
                           void* dv, float* dg, float* dbeta, float* dh0, void* scratch,
                           int64_t scratch_bytes, int64_t B, int64_t L, int64_t S, int64_t HK,
                           int64_t H, int64_t DK, int64_t DV, const int64_t* strides, float scale,
                           int dtype, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  int rc = check_sizes(B, L, S, HK, H, DK, DV, dtype, packed);
  if (rc != SS2D_OK) return rc;
  if (!std::isfinite(scale)) return SS2D_ERR_UNSUPPORTED;
  if (S == 0 || H == 0) return SS2D_OK;
  const int64_t T = B * L, e = dtype == SS2D_F32 ? 4 : 2;
  if (T == 0 && !dh0) return SS2D_OK;
  if (T > 0 && (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta))
    return SS2D_ERR_NULL;
  Args a{};
  Span ins[10];
  rc = set_inputs(&a, ins, q, k, v, g, beta, h0, cu_seqlens, B, L, S, HK, H, DK, DV, strides, scale,
                  dtype);
  if (rc != SS2D_OK) return rc;
  for (const void* p : {dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                        static_cast<const void*>(dv)})
    if (misaligned(p, static_cast<uintptr_t>(e))) return SS2D_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(dht), static_cast<const void*>(dg),
                        static_cast<const void*>(dbeta), static_cast<const void*>(dh0)})
    if (misaligned(p, 4)) return SS2D_ERR_ALIGN;
  if (misaligned(saved, 256) || misaligned(scratch, 256)) return SS2D_ERR_ALIGN;
  const int64_t state = S * H * DK * DV * 4;
  const Saved sv = saved_layout(L, S, T, H, DK, DV, packed);
  a.p_planes = 3;
  const BackwardScratch w = backward_layout(a, dtype, saved != nullptr, packed);
  ins[6] = {h0, state};
  ins[7] = {saved, sv.bytes};
  ins[8] = {dout, T * H * DV * e};
  ins[9] = {dht, state};
  const Span outs[] = {{dq, T * HK * DK * e}, {dk, T * HK * DK * e}, {dv, T * H * DV * e},
                       {dg, T * H * 4}, {dbeta, T * H * 4}, {dh0, state},
                       {scratch, static_cast<int64_t>(w.bytes)}};
  rc = check_pointers(ins, 10, outs, 7);
  if (rc != SS2D_OK) return rc;
  a.dout = dout;
  a.dht = dht;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dh0 = dh0;

  hipStream_t st = static_cast<hipStream_t>(stream);
  Workspace ws;
  rc = take_scratch(&ws, scratch, scratch_bytes, w.bytes, st);
  if (rc != SS2D_OK) return rc;
  set_scratch(&a, ws.at, w.chunks);
  a.dmarks = reinterpret_cast<float*>(ws.at + w.dmarks);
  a.dvs = dtype == SS2D_F32 ? static_cast<float*>(dv) : reinterpret_cast<float*>(ws.at + w.dvs);
  a.pbeta = reinterpret_cast<float*>(ws.at + w.pbeta);
  a.pgate = reinterpret_cast<float*>(ws.at + w.pgate);
  a.pdots = reinterpret_cast<float*>(ws.at + w.pdots);
  int err = 0;
  if (saved) {
    set_saved(&a, const_cast<void*>(saved), sv);
  } else {
    set_saved(&a, ws.at + w.keep, sv);
    a.o = ws.at + w.unused_o;
    err = run_forward(a, dtype, true, st);
  }
  const bool alk = aligned_keys(a, e);
  const Strides rows = {L * H * DV, H * DV, DV};
  const bool alv = aligned_rows(dout, rows, DV, e) && aligned_rows(dv, rows, DV, e);
  if (!err && a.slots > 0) err = ss2d::delta::launch_prep(a, dtype, alk, true, st);
  if (!err && a.seglen) err = ss2d::delta::launch_adjoint(a, dtype, true, st);
  if (!err && a.seglen) err = ss2d::delta::launch_join(a, true, st);
  if (!err) err = ss2d::delta::launch_adjoint(a, dtype, false, st);
  if (!err && a.marks_n > 0) err = ss2d::delta::launch_grads(a, dtype, alv, st);
  if (!err && a.marks_n > 0) err = ss2d::delta::launch_gate_grads(a, st);
  return finish(ws, err, st);
}

int ss1d_delta_step(const void* q, const void* k, const void* v, const float* g,
                    const float* beta, float* state, const int32_t* slots, void* o, int64_t B,
                    int64_t T, int64_t S, int64_t HK, int64_t H, int64_t DK, int64_t DV,
                    const int64_t* strides, float scale, int dtype, void* stream) {
  int rc = check_sizes(B, T, B, HK, H, DK, DV, dtype, false);
  if (rc != SS2D_OK) return rc;
  if (!std::isfinite(scale)) return SS2D_ERR_UNSUPPORTED;
  int64_t n;
  if (S < 0 || S >= kMaxTokens || !ss2d::host_mul_ok(S, H * DK * DV, &n) ||
      n > ss2d::kHostMaxElems / 64)
    return SS2D_ERR_SHAPE;
  if (!slots && S < B) return SS2D_ERR_SHAPE;
  if (B == 0 || T == 0 || H == 0 || S == 0) return SS2D_OK;
  if (!q || !k || !v || !g || !beta || !state || !o) return SS2D_ERR_NULL;
  const int64_t e = dtype == SS2D_F32 ? 4 : 2;
  ss2d::delta::StepArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.slots = slots;
  a.state = state;
  a.o = o;
  default_strides(T, HK, DK, &a.sq);
  default_strides(T, HK, DK, &a.sk);
  default_strides(T, H, DV, &a.sv);
  if (strides) {
    a.sq = {strides[0], strides[1], strides[2]};
    a.sk = {strides[3], strides[4], strides[5]};
    a.sv = {strides[6], strides[7], strides[8]};
  }
  a.B = B;
  a.T = T;
  a.S = S;
  a.H = static_cast<int>(H);
  a.HK = static_cast<int>(HK);
  a.rep = static_cast<int>(H / HK);
  a.DK = static_cast<int>(DK);
  a.DV = static_cast<int>(DV);
  a.scale = scale;
  const int64_t qb = strided_bytes(B, T, HK, DK, a.sq, e), kb = strided_bytes(B, T, HK, DK, a.sk, e),
                vb = strided_bytes(B, T, H, DV, a.sv, e);
  if (qb < 0 || kb < 0 || vb < 0) return SS2D_ERR_SHAPE;
  for (const void* p : {q, k, v, static_cast<const void*>(o)})
    if (misaligned(p, static_cast<uintptr_t>(e))) return SS2D_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(g), static_cast<const void*>(beta),
                        static_cast<const void*>(state), static_cast<const void*>(slots)})
    if (misaligned(p, 4)) return SS2D_ERR_ALIGN;
  const Span ins[] = {{q, qb}, {k, kb}, {v, vb}, {g, B * T * H * 4}, {beta, B * T * H * 4},
                      {slots, B * 4}};
  const Span outs[] = {{o, B * T * H * DV * e}, {state, S * H * DK * DV * 4}};
  rc = check_pointers(ins, 6, outs, 2);
  if (rc != SS2D_OK) return rc;
  if (B * H * ((DV + 15) / 16) * 64 > kMaxThreads) return SS2D_ERR_SHAPE;
  const bool vec = DV % 4 == 0 && !misaligned(state, 16);
  const int err = ss2d::delta::launch_step(a, dtype, vec, static_cast<hipStream_t>(stream));
  if (err) return ss2d::host_hip_fail(static_cast<hipError_t>(err));
  return SS2D_OK;
}

}  // extern "C"
