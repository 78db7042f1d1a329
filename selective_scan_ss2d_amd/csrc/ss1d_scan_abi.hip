// C entry points of the token-order selective scan: argument checks, scratch and the kernel sequence.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "ss1d_scan.h"
#include "ss1d_scan_step.h"
#include "ss2d.h"
#include "ss2d_host.h"

namespace {

using ss2d::RowStrides;
using ss2d::sscan::Args;
using ss2d::sscan::StepArgs;

// The plan that a test forces on its own thread (ss1d_scan_set_plan): lanes of a channel (0: the
// rule's) and tokens of a segment (-1: the rule's).
thread_local int g_lanes_override = 0;
thread_local int64_t g_segment_override = -1;

constexpr int64_t kMaxTokens = int64_t(1) << 40;
constexpr int64_t kMaxLine = int64_t(1) << 24;    // elements from one token's row to the next
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;  // of one launch

struct Span {  // the memory of one argument
  const void* p;
  int64_t bytes;
};

bool off(const void* p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int check_sizes(int64_t B, int64_t L, int64_t S, int64_t D, int64_t G, int64_t N, int dtype, bool packed) {
  if (dtype != SS2D_F32 && dtype != SS2D_BF16) return SS2D_ERR_UNSUPPORTED;
  if (B < 0 || L < 0 || S < 0 || D < 0 || G < 1 || N < 1) return SS2D_ERR_SHAPE;
  if (D % G != 0 || (packed ? B != 1 : S != B)) return SS2D_ERR_SHAPE;
  if (N > ss2d::sscan::kMaxN) return SS2D_ERR_UNSUPPORTED;
  if (B >= kMaxTokens || L >= kMaxTokens || S >= kMaxTokens || D > kMaxLine || G * N > kMaxLine)
    return SS2D_ERR_SHAPE;
  int64_t t, n;
  if (!ss2d::host_mul_ok(B, L, &t) || t >= kMaxTokens) return SS2D_ERR_SHAPE;
  if (!ss2d::host_mul_ok(t, D + 2 * G * N, &n) || n > ss2d::kHostMaxElems / 4096) return SS2D_ERR_SHAPE;
  if (!ss2d::host_mul_ok(S, D * N, &n) || n > ss2d::kHostMaxElems / 4096) return SS2D_ERR_SHAPE;
  return SS2D_OK;
}

// Bytes from the first to past the last element of a (B, L, width) tensor whose rows lie apart by
// its strides; -1 where they are out of range.
int64_t strided_bytes(int64_t B, int64_t L, int64_t width, const RowStrides& s, int64_t e) {
  if (s.b < 0 || s.l < 0 || s.l > kMaxLine) return -1;
  if (B == 0 || L == 0 || width == 0) return 0;
  int64_t tb, tl;
  if (!ss2d::host_mul_ok(B - 1, s.b, &tb) || !ss2d::host_mul_ok(L - 1, s.l, &tl) ||
      tb > ss2d::kHostMaxElems / 64 || tl > ss2d::kHostMaxElems / 64)
    return -1;
  return (tb + tl + width) * e;
}

// The data inputs u, dt_raw, z, Bs, Cs of a call, their strides and memory (ins[0..4]).
struct Data {
  RowStrides su, sd, sz, sb, sc;
  int64_t sbg, scg;
};
int set_data(Data* x, Span* ins, const void* u, const void* dt, const void* z, const void* Bs, const void* Cs,
             int64_t B, int64_t L, int64_t D, int64_t G, int64_t N, const int64_t* st, int64_t e) {
  x->su = x->sd = x->sz = {L * D, D};
  x->sb = x->sc = {L * G * N, G * N};
  x->sbg = x->scg = N;
  if (st) {
    x->su = {st[0], st[1]};
    x->sd = {st[2], st[3]};
    x->sz = {st[4], st[5]};
    x->sb = {st[6], st[7]};
    x->sbg = st[8];
    x->sc = {st[9], st[10]};
    x->scg = st[11];
  }
  // the strides of one token and of one group are not used, however wide
  if (L <= 1)
    for (RowStrides* s : {&x->su, &x->sd, &x->sz, &x->sb, &x->sc}) s->l = std::min(s->l, kMaxLine);
  if (G == 1)
    for (int64_t* s : {&x->sbg, &x->scg}) *s = std::min(*s, kMaxLine);
  if (x->sbg < 0 || x->scg < 0 || x->sbg > kMaxLine || x->scg > kMaxLine) return SS2D_ERR_SHAPE;
  if ((G - 1) * std::max(x->sbg, x->scg) > kMaxLine) return SS2D_ERR_SHAPE;
  const int64_t bytes[5] = {strided_bytes(B, L, D, x->su, e), strided_bytes(B, L, D, x->sd, e),
                            z ? strided_bytes(B, L, D, x->sz, e) : 0,
                            strided_bytes(B, L, (G - 1) * x->sbg + N, x->sb, e),
                            strided_bytes(B, L, (G - 1) * x->scg + N, x->sc, e)};
  const void* p[5] = {u, dt, z, Bs, Cs};
  for (int i = 0; i < 5; ++i) {
    if (bytes[i] < 0) return SS2D_ERR_SHAPE;
    if (off(p[i], e)) return SS2D_ERR_ALIGN;
    ins[i] = {p[i], bytes[i]};
  }
  return SS2D_OK;
}

int check_overlap(const Span* ins, int n_in, const Span* outs, int n_out) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (ss2d::host_overlaps(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return SS2D_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (ss2d::host_overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return SS2D_ERR_ALIAS;
  }
  return SS2D_OK;
}

// How a call is cut: the lanes of a channel, and the tokens of a segment (0: whole sequences).  The
// forward takes what these estimates of its time find shortest, in us, fitted to 60 shapes of 64 to
// 65536 tokens, 192 to 12288 channels, N 8 to 32 (`quads`: waves with four lanes per channel):
//   four lanes, whole       0.117 longest       (1024 tokens: 120; up to 1024 waves, 0.65 a wave more)
//   16 lanes, whole         (0.025 + 0.0275 waves / 1024) longest     (1024 x 4096 channels: 56)
//   four lanes, segments    14 + 1.2e-4 a token and wave   (1024 x 4096: 51; 4096 x 4096: 140, whole 475)
// each token's time by its states (kNS of a lane).  Segments are made for 4096 waves, four per SIMD,
// of 32 tokens at least: 4096 tokens x 4096 channels take 213, 158, 140 and 144 us in 4, 8, 16 and 32
// segments.  Of packed sequences the longest is not known here: four times their mean is assumed, and as
// many waves in the backward as for equal ones.  A long prompt among many short sequences is therefore
// not cut: 16,000 tokens and 39 sequences of 10, 4096 channels, take 2754 us (802 in segments of 256), a
// training step 10.5 ms (2.9); 4096 tokens and 255 single ones 684 (1142 in such segments).
// A forward that keeps states runs by four lanes.  The backward, whose waves fill a SIMD by twos, is
// cut below 2048 waves: 8 x 2048 tokens of 2048 channels take 758 us whole, 627 in segments.
void set_plan(Args* a, int64_t B, int64_t L, bool packed, bool saves, bool backward) {
  const int64_t S = a->q.S, T = a->q.T, Dg = a->D / a->G, tile = ss2d::sscan::tile_steps(a->N);
  a->lanes = 4;
  a->seglen = 0;
  a->units = S;
  if (T == 0 || a->D == 0 || S == 0) return;
  const int64_t per = a->G * ((Dg + 15) / 16), quads = S * per;  // waves of a sequence, of all
  // equal segments of the dense rows, as many as keep to 4096 waves
  const int64_t parts = std::max<int64_t>(2, 4096 / std::max<int64_t>(1, quads));
  const int64_t fair = packed ? T * per / 4096 : (L + parts - 1) / parts;
  const int64_t len = std::max<int64_t>(32, (fair + tile - 1) / tile * tile);
  const double longest = packed ? std::min<double>(T, 4.0 * T / S) : L;
  const double states = (ss2d::sscan::lane_states(a->N) + 3) / 7.0;
  const double rows = a->N > 16 ? 1.35 : 1.0, fill = std::max(1.0, quads * 4 / 1024.0);
  const double whole = 0.117 * longest * states * std::max(1.0, 0.35 + 0.65 * quads / 1024.0);
  const double by16 = (0.025 + 0.0275 * fill) * longest * rows;
  const double cut = 2 * len <= longest ? 14 + 1.2e-4 * T * per * states : 1e30;
  if (backward) {
    if (quads < 2048 && 2 * len <= longest) a->seglen = len;
  } else if (cut < whole && (saves || cut < by16)) {
    a->seglen = len;
  } else if (!saves && by16 < whole) {
    a->lanes = 16;
  }
  if (g_segment_override >= 0) a->seglen = (g_segment_override + tile - 1) / tile * tile;
  if (g_lanes_override) a->lanes = saves ? 4 : g_lanes_override;
  if (a->seglen) a->units = ss2d::unit_count(L, S, T, packed, a->seglen);
}

void set_sizes(Args* a, int64_t B, int64_t L, int64_t S, int64_t D, int64_t G, int64_t N, const int32_t* cu,
               bool packed, bool saves, bool backward) {
  a->q = {cu, S, L, B * L};
  a->D = static_cast<int>(D);
  a->G = static_cast<int>(G);
  a->N = static_cast<int>(N);
  a->cbg = static_cast<int>((D / G + ss2d::sscan::kBlockCh - 1) / ss2d::sscan::kBlockCh);
  set_plan(a, B, L, packed, saves, backward);
}

// Whether the threads of each launch that the call makes can be counted in 32 bits: the scan's blocks, of
// kThreads / lanes channels; a join's states; the backward's sums over channel blocks, of 16 tokens a
// block, and over units, of 64 columns.
bool launchable(const Args& a, bool packed, bool backward) {
  const int channels = ss2d::sscan::kThreads / (backward ? 4 : a.lanes);
  const int64_t blocks = a.G * ((a.D / a.G + channels - 1) / channels), per = int64_t(a.D) * a.N;
  if (a.units > kMaxThreads / ss2d::sscan::kThreads / std::max<int64_t>(1, blocks)) return false;
  if (a.seglen && a.q.S > (kMaxThreads - 256) / std::max<int64_t>(1, per)) return false;
  return !backward || (ss2d::unit_count(a.q.L, a.q.S, a.q.T, packed, 16) <= kMaxThreads / 256 &&
                       (int64_t(a.D) * (a.N + 2) + 63) / 64 <= kMaxThreads / 1024);
}

int64_t mark_bytes(int64_t L, int64_t S, int64_t T, int64_t D, int64_t N, bool packed) {
  return static_cast<int64_t>(ss2d::host_align256(
      size_t(ss2d::unit_count(L, S, T, packed, ss2d::sscan::tile_steps(N))) * D * N * 4));
}

// Scratch: the segments' states (again: of the forward that a backward without `saved` runs, cut as a
// saving forward is, so that its gradients are the same bit for bit), then the backward's.
struct Layout {
  size_t end, start, delta, bc, params, marks, y, bytes;
};
Layout layout(const Args& a, const Args& again, bool backward, bool kept, bool packed, int64_t e) {
  using ss2d::host_align256;
  size_t seg = a.seglen ? size_t(a.units) * a.D : 0;
  if (backward && !kept && again.seglen) seg = std::max(seg, size_t(again.units) * a.D);
  Layout w;
  w.end = 0;
  w.start = host_align256(seg * a.N * 4);
  w.delta = w.start + host_align256(seg * a.N * 4);
  w.bc = w.delta + host_align256(seg * 4);
  w.params = w.bc;
  w.marks = w.y = w.bytes = w.bc;
  if (!backward) return w;
  w.params = w.bc + host_align256(size_t(a.cbg) * a.q.T * a.G * 2 * a.N * 4);
  w.marks = w.params + host_align256(size_t(a.units) * a.D * (a.N + 2) * 4);
  w.y = w.marks + (kept ? 0 : size_t(mark_bytes(a.q.L, a.q.S, a.q.T, a.D, a.N, packed)));
  w.bytes = w.y + (kept ? 0 : host_align256(size_t(a.q.T) * a.D * e));
  return w;
}
void set_segments(Args* a, char* ws, const Layout& w) {
  a->seg_end = reinterpret_cast<float*>(ws + w.end);
  a->seg_start = reinterpret_cast<float*>(ws + w.start);
  a->seg_delta = reinterpret_cast<float*>(ws + w.delta);
}

int run_forward(const Args& a, int dtype, hipStream_t st) {
  if (a.units == 0) return 0;
  int err = a.seglen ? ss2d::sscan::launch_scan_segments(a, dtype, st) : 0;
  if (!err && a.seglen) err = ss2d::sscan::launch_scan_join(a, false, st);
  return err ? err : ss2d::sscan::launch_scan_tokens(a, dtype, st);
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
  if (bytes == 0) return SS2D_OK;
  w->own = true;
  return ss2d::host_scratch_outside_graphs(&w->at, bytes, st);
}
int finish(const Workspace& w, int err, hipStream_t st) {
  const hipError_t fe = w.own ? hipFreeAsync(w.at, st) : hipSuccess;
  if (err) return ss2d::host_hip_fail(static_cast<hipError_t>(err));
  return fe == hipSuccess ? SS2D_OK : ss2d::host_hip_fail(fe);
}

void set_inputs(Args* a, const Data& x, const void* u, const void* dt, const void* z, const void* Bs, const void* Cs,
                const float* A_log, const float* Ds, const float* bias, const float* h0) {
  a->u = u;
  a->dt = dt;
  a->z = z;
  a->Bs = Bs;
  a->Cs = Cs;
  a->A_log = A_log;
  a->Ds = Ds;
  a->bias = bias;
  a->h0 = h0;
  a->su = x.su;
  a->sd = x.sd;
  a->sz = x.sz;
  a->sb = x.sb;
  a->sc = x.sc;
  a->sbg = x.sbg;
  a->scg = x.scg;
}

}  // namespace

extern "C" {

int ss1d_scan_set_plan(int lanes, int64_t tokens) {
  if (lanes != 0 && lanes != 4 && lanes != 16) return SS2D_ERR_UNSUPPORTED;
  if (tokens < -1 || tokens > (int64_t(1) << 30)) return SS2D_ERR_SHAPE;
  g_lanes_override = lanes;
  g_segment_override = tokens;
  return SS2D_OK;
}

int64_t ss1d_scan_saved_bytes(int64_t B, int64_t L, int64_t S, int64_t D, int64_t N, int packed) {
  if (check_sizes(B, L, S, D, 1, N, SS2D_BF16, packed != 0) != SS2D_OK) return -1;
  return mark_bytes(L, S, B * L, D, N, packed != 0);
}

int64_t ss1d_scan_scratch_bytes(int backward, int kept, int64_t B, int64_t L, int64_t S, int64_t D, int64_t G,
                                int64_t N, int dtype, int packed) {
  if (check_sizes(B, L, S, D, G, N, dtype, packed != 0) != SS2D_OK) return -1;
  Args a{};
  set_sizes(&a, B, L, S, D, G, N, nullptr, packed != 0, backward || kept, backward != 0);
  Args again{};
  set_sizes(&again, B, L, S, D, G, N, nullptr, packed != 0, true, false);
  return static_cast<int64_t>(layout(a, again, backward != 0, kept != 0, packed != 0, dtype == SS2D_F32 ? 4 : 2).bytes);
}

int ss1d_scan_forward(const void* u, const void* dt_raw, const float* A_log, const void* Bs, const void* Cs,
                      const float* Ds, const float* dt_bias, const void* z, const float* h0,
                      const int32_t* cu_seqlens, void* y, float* ht, void* saved, void* scratch,
                      int64_t scratch_bytes, int64_t B, int64_t L, int64_t S, int64_t D, int64_t G, int64_t N,
                      const int64_t* strides, int dtype, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  int rc = check_sizes(B, L, S, D, G, N, dtype, packed);
  if (rc != SS2D_OK) return rc;
  if (D == 0 || S == 0 || (B * L == 0 && !ht)) return SS2D_OK;
  const bool none = B * L == 0;  // the end states are the initial ones
  if (!none && (!u || !dt_raw || !Bs || !Cs || !y)) return SS2D_ERR_NULL;
  if (!A_log || !Ds || !dt_bias) return SS2D_ERR_NULL;
  const int64_t e = dtype == SS2D_F32 ? 4 : 2;
  Data x;
  Span ins[10];
  rc = set_data(&x, ins, u, dt_raw, z, Bs, Cs, B, L, D, G, N, strides, e);
  if (rc != SS2D_OK) return rc;
  for (const void* p : {static_cast<const void*>(A_log), static_cast<const void*>(Ds),
                        static_cast<const void*>(dt_bias), static_cast<const void*>(h0),
                        static_cast<const void*>(cu_seqlens), static_cast<const void*>(ht)})
    if (off(p, 4)) return SS2D_ERR_ALIGN;
  if (off(y, e) || off(saved, 256) || off(scratch, 256)) return SS2D_ERR_ALIGN;
  Args a{};
  set_sizes(&a, B, L, S, D, G, N, cu_seqlens, packed, saved != nullptr, false);
  if (!launchable(a, packed, false)) return SS2D_ERR_SHAPE;
  const Layout w = layout(a, a, false, true, packed, e);
  const int64_t states = S * D * N * 4;
  ins[5] = {A_log, D * N * 4};
  ins[6] = {Ds, D * 4};
  ins[7] = {dt_bias, D * 4};
  ins[8] = {cu_seqlens, packed ? (S + 1) * 4 : 0};
  ins[9] = {h0, states};
  const Span outs[] = {{y, B * L * D * e}, {ht, states}, {saved, mark_bytes(L, S, B * L, D, N, packed)},
                       {scratch, static_cast<int64_t>(w.bytes)}};
  // ht may replace h0: a lane reads its states before it, or the join has taken them
  const bool in_place = ht && ht == h0;
  rc = check_overlap(ins, in_place ? 9 : 10, outs, 4);
  if (rc == SS2D_OK && in_place)
    for (int i : {0, 2, 3})
      if (ss2d::host_overlaps(outs[i].p, outs[i].bytes, h0, states)) rc = SS2D_ERR_ALIAS;
  if (rc != SS2D_OK) return rc;
  set_inputs(&a, x, u, dt_raw, z, Bs, Cs, A_log, Ds, dt_bias, h0);
  a.y = y;
  a.ht = ht;
  a.marks = static_cast<float*>(saved);
  hipStream_t st = static_cast<hipStream_t>(stream);
  Workspace ws;
  rc = take_scratch(&ws, scratch, scratch_bytes, w.bytes, st);
  if (rc != SS2D_OK) return rc;
  set_segments(&a, ws.at, w);
  return finish(ws, run_forward(a, dtype, st), st);
}

int ss1d_scan_backward(const void* u, const void* dt_raw, const float* A_log, const void* Bs, const void* Cs,
                       const float* Ds, const float* dt_bias, const void* z, const float* h0,
                       const int32_t* cu_seqlens, const void* saved, const void* dy, const float* dht, void* du,
                       void* ddt_raw, float* dA_log, void* dBs, void* dCs, float* dDs, float* ddt_bias, void* dz,
                       float* dh0, void* scratch, int64_t scratch_bytes, int64_t B, int64_t L, int64_t S, int64_t D,
                       int64_t G, int64_t N, const int64_t* strides, int dtype, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  int rc = check_sizes(B, L, S, D, G, N, dtype, packed);
  if (rc != SS2D_OK) return rc;
  const bool none = B * L == 0;
  if (D == 0 && none) return SS2D_OK;
  if (!none && (!dBs || !dCs)) return SS2D_ERR_NULL;
  if (!none && D > 0 && (!u || !dt_raw || !Bs || !Cs || !dy || !du || !ddt_raw || (z != nullptr) != (dz != nullptr)))
    return SS2D_ERR_NULL;
  if (D > 0 && (!A_log || !Ds || !dt_bias || !dA_log || !dDs || !ddt_bias)) return SS2D_ERR_NULL;
  const int64_t e = dtype == SS2D_F32 ? 4 : 2;
  Data x;
  Span ins[13];
  rc = set_data(&x, ins, u, dt_raw, z, Bs, Cs, B, L, D, G, N, strides, e);
  if (rc != SS2D_OK) return rc;
  for (const void* p : {static_cast<const void*>(A_log), static_cast<const void*>(Ds),
                        static_cast<const void*>(dt_bias), static_cast<const void*>(h0),
                        static_cast<const void*>(cu_seqlens), static_cast<const void*>(dht),
                        static_cast<const void*>(dA_log), static_cast<const void*>(dDs),
                        static_cast<const void*>(ddt_bias), static_cast<const void*>(dh0)})
    if (off(p, 4)) return SS2D_ERR_ALIGN;
  for (const void* p : {dy, static_cast<const void*>(du), static_cast<const void*>(ddt_raw),
                        static_cast<const void*>(dBs), static_cast<const void*>(dCs), static_cast<const void*>(dz)})
    if (off(p, e)) return SS2D_ERR_ALIGN;
  if (off(saved, 256) || off(scratch, 256)) return SS2D_ERR_ALIGN;
  Args a{};
  set_sizes(&a, B, L, S, D, G, N, cu_seqlens, packed, true, true);
  Args again{};
  set_sizes(&again, B, L, S, D, G, N, cu_seqlens, packed, true, false);
  if (!launchable(a, packed, true) || (!saved && !launchable(again, packed, false))) return SS2D_ERR_SHAPE;
  const Layout w = layout(a, again, true, saved != nullptr, packed, e);
  const int64_t states = S * D * N * 4, wide = B * L * D * e, bc = B * L * G * N * e;
  ins[5] = {A_log, D * N * 4};
  ins[6] = {Ds, D * 4};
  ins[7] = {dt_bias, D * 4};
  ins[8] = {cu_seqlens, packed ? (S + 1) * 4 : 0};
  ins[9] = {h0, states};
  ins[10] = {saved, mark_bytes(L, S, B * L, D, N, packed)};
  ins[11] = {dy, wide};
  ins[12] = {dht, states};
  const Span outs[] = {{du, wide}, {ddt_raw, wide}, {dz, wide}, {dBs, bc}, {dCs, bc}, {dA_log, D * N * 4},
                       {dDs, D * 4}, {ddt_bias, D * 4}, {dh0, states}, {scratch, static_cast<int64_t>(w.bytes)}};
  rc = check_overlap(ins, 13, outs, 10);
  if (rc != SS2D_OK) return rc;
  set_inputs(&a, x, u, dt_raw, z, Bs, Cs, A_log, Ds, dt_bias, h0);
  a.dy = dy;
  a.dht = dht;
  a.du = du;
  a.ddt = ddt_raw;
  a.dz = dz;
  a.dB = dBs;
  a.dC = dCs;
  a.dA = dA_log;
  a.dD = dDs;
  a.dbias = ddt_bias;
  a.dh0 = dh0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Workspace ws;
  rc = take_scratch(&ws, scratch, scratch_bytes, w.bytes, st);
  if (rc != SS2D_OK) return rc;
  set_segments(&a, ws.at, w);
  a.bc_parts = reinterpret_cast<float*>(ws.at + w.bc);
  a.par_parts = reinterpret_cast<float*>(ws.at + w.params);
  a.marks = const_cast<float*>(static_cast<const float*>(saved));
  int err = 0;
  if (!saved && D > 0) {  // the states before every tile, by the forward
    a.marks = reinterpret_cast<float*>(ws.at + w.marks);
    set_inputs(&again, x, u, dt_raw, z, Bs, Cs, A_log, Ds, dt_bias, h0);
    set_segments(&again, ws.at, w);
    again.marks = a.marks;
    again.y = ws.at + w.y;
    err = none ? 0 : run_forward(again, dtype, st);
  }
  if (!err && a.units > 0 && D > 0) {
    if (a.seglen) err = ss2d::sscan::launch_scan_adjoint_segments(a, dtype, st);
    if (!err && a.seglen) err = ss2d::sscan::launch_scan_join(a, true, st);
    if (!err) err = ss2d::sscan::launch_scan_adjoint(a, dtype, st);
  }
  if (!err) err = ss2d::sscan::launch_scan_sums(a, dtype, st);
  return finish(ws, err, st);
}

int ss1d_scan_step(const void* u, const void* dt_raw, const float* A_log, const void* Bs, const void* Cs,
                   const float* Ds, const float* dt_bias, const void* z, float* state, const int32_t* slots, void* y,
                   int64_t B, int64_t T, int64_t S, int64_t D, int64_t G, int64_t N, const int64_t* strides,
                   int dtype, void* stream) {
  int rc = check_sizes(B, T, B, D, G, N, dtype, false);
  if (rc != SS2D_OK) return rc;
  int64_t n;
  if (S < 0 || S >= kMaxTokens || (!slots && S != B)) return SS2D_ERR_SHAPE;
  if (!ss2d::host_mul_ok(S, D * N, &n) || n > ss2d::kHostMaxElems / 4096) return SS2D_ERR_SHAPE;
  if (D > 0 && (B > kMaxThreads / 256 / ((D + 63) / 64) || T >= (int64_t(1) << 31))) return SS2D_ERR_SHAPE;
  if (B == 0 || T == 0 || D == 0) return SS2D_OK;
  if (!u || !dt_raw || !A_log || !Bs || !Cs || !Ds || !dt_bias || (!state && S > 0) || !y) return SS2D_ERR_NULL;
  const int64_t e = dtype == SS2D_F32 ? 4 : 2;
  Data x;
  Span ins[9];
  rc = set_data(&x, ins, u, dt_raw, z, Bs, Cs, B, T, D, G, N, strides, e);
  if (rc != SS2D_OK) return rc;
  for (const void* p : {static_cast<const void*>(A_log), static_cast<const void*>(Ds),
                        static_cast<const void*>(dt_bias), static_cast<const void*>(state),
                        static_cast<const void*>(slots)})
    if (off(p, 4)) return SS2D_ERR_ALIGN;
  if (off(y, e)) return SS2D_ERR_ALIGN;
  ins[5] = {A_log, D * N * 4};
  ins[6] = {Ds, D * 4};
  ins[7] = {dt_bias, D * 4};
  ins[8] = {slots, slots ? B * 4 : 0};
  const Span outs[] = {{y, B * T * D * e}, {state, n * 4}};
  rc = check_overlap(ins, 9, outs, 2);
  if (rc != SS2D_OK) return rc;
  StepArgs a{u, dt_raw, z, Bs, Cs, A_log, Ds, dt_bias, {slots, static_cast<int>(B), S}, state, y,
             x.su, x.sd, x.sz, x.sb, x.sc, x.sbg, x.scg, static_cast<int>(T), static_cast<int>(D),
             static_cast<int>(G), static_cast<int>(N), false, 1};
  a.whole = (N == 16 || N == 32) && !off(state, 16) && !off(A_log, 16) && !off(Bs, 4 * e) && !off(Cs, 4 * e);
  for (int64_t v : {x.sb.b, x.sb.l, x.sbg, x.sc.b, x.sc.l, x.scg}) a.whole = a.whole && v % 4 == 0;
  // rows of a block: 8192 waves are enough to hide the loads (256 rows of 4096 channels: 45, 37, 32, 32
  // and 33 us with 65536, 32768, 16384, 8192 and 4096), and share what the channels' parameters cost
  a.rows = static_cast<int>(std::clamp<int64_t>(B * ((D + 15) / 16) / 8192, 1, 16));
  const int err = ss2d::sscan::launch_scan_step(a, dtype, static_cast<hipStream_t>(stream));
  return err ? ss2d::host_hip_fail(static_cast<hipError_t>(err)) : SS2D_OK;
}

}  // extern "C"
