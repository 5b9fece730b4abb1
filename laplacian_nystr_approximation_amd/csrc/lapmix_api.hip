// C ABI of the lapmix operators (declared in include/lapmix.h): validation,
// workspace sizes and the launches.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "lapmix.h"
#include "lapmix_internal.hpp"

using lapmix::Strides;

namespace {

bool ok(hipError_t e, const char* what) {
  if (e == hipSuccess) return true;
  const char* log = getenv("LAPNYS_LOG");
  if (log && *log && *log != '0')
    fprintf(stderr, "liblapnys: %s failed: %s (%d)\n", what, hipGetErrorString(e), (int)e);
  return false;
}

bool storage_type(int32_t t) { return t == LAPNYS_F32 || t == LAPNYS_BF16; }
int64_t element_size(int32_t t) { return t == LAPNYS_F32 ? 4 : t == LAPNYS_BF16 ? 2 : 1; }

// A tensor argument: `nd` dimensions of sizes n and element strides s, the
// channels (contiguous, `width` of them) counted apart.
struct View {
  uintptr_t base;
  int64_t esize, width;
  int nd;
  int64_t n[3], s[3];
};

View dense_view(const void* p, int64_t count, int64_t esize) { return {(uintptr_t)p, esize, count, 0, {}, {}}; }

View strided_view(const void* p, int32_t B, int32_t H, int32_t N, int32_t d, const Strides& st, int64_t esize) {
  View v = {(uintptr_t)p, esize, d, 0, {}, {}};
  const int64_t n[3] = {B, H, N}, s[3] = {st.b, st.h, st.n};
  // Dimensions of size 1 have no stride; the others go by rising stride.
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    int at = v.nd++;
    for (; at > 0 && v.s[at - 1] > s[i]; --at) v.n[at] = v.n[at - 1], v.s[at] = v.s[at - 1];
    v.n[at] = n[i], v.s[at] = s[i];
  }
  return v;
}

// Elements from the first to the last one of the view (inclusive).
int64_t extent(const View& v) {
  int64_t e = v.width;
  for (int i = 0; i < v.nd; ++i) e += (v.n[i] - 1) * v.s[i];
  return e;
}

// No two elements coincide when the innermost `level` dimensions span `inner` elements.
bool nests(const View& v, int level, int64_t inner) {
  for (int i = level; i < v.nd; ++i) {
    if (v.s[i] < inner) return false;
    inner += (v.n[i] - 1) * v.s[i];
  }
  return true;
}

bool distinct(const View& v) { return nests(v, 0, v.width); }

bool disjoint(const View& a, const View& b) {
  if (!a.base || !b.base) return true;
  const uintptr_t ea = a.base + (uintptr_t)(extent(a) * a.esize), eb = b.base + (uintptr_t)(extent(b) * b.esize);
  if (ea <= b.base || eb <= a.base) return true;
  // Two parts of one interleaved buffer: the same sizes and strides, apart by
  // at least what some inner dimensions span, with room for both in the next.
  if (a.esize != b.esize || a.width != b.width || a.nd != b.nd) return false;
  for (int i = 0; i < a.nd; ++i)
    if (a.n[i] != b.n[i] || a.s[i] != b.s[i]) return false;
  const uintptr_t gap = a.base < b.base ? b.base - a.base : a.base - b.base;
  if (gap % (uintptr_t)a.esize) return false;
  const int64_t delta = (int64_t)(gap / (uintptr_t)a.esize);
  int64_t inner = a.width;
  for (int i = 0; i < a.nd; ++i) {
    if (!nests(a, 0, a.width)) return false;
    if (delta >= inner && nests(a, i, delta + inner)) return true;
    inner += (a.n[i] - 1) * a.s[i];
  }
  return false;
}

// Every output is apart from every other tensor; empty views have base 0.
bool outputs_apart(const View* out, int nout, const View* in, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int j = i + 1; j < nout; ++j)
      if (!disjoint(out[i], out[j])) return false;
    for (int j = 0; j < nin; ++j)
      if (!disjoint(out[i], in[j])) return false;
  }
  return true;
}

// Strides of a [B, H, N, d] tensor: all zero mean dense, those of dimensions of
// size 1 do not matter.  Element offsets stay below 2^60, so byte offsets and
// the sums below fit 64 bits.
bool take_strides(const int64_t in[3], int32_t B, int32_t H, int32_t N, int32_t d, Strides* st) {
  const int64_t n[3] = {B, H, N};
  const bool dense = !in[0] && !in[1] && !in[2];
  int64_t s[3] = {(int64_t)H * N, N, 1};
  __int128 last = d;
  for (int i = 0; i < 3; ++i) {
    const __int128 v = dense ? (__int128)s[i] * d : n[i] == 1 ? 0 : in[i];
    if (v < 0) return false;
    last += v * (n[i] - 1);
    if (last > ((__int128)1 << 60)) return false;
    s[i] = n[i] == 1 ? 0 : (int64_t)v;
  }
  *st = {s[0], s[1], s[2]};
  return true;
}

bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// Width and the strides of dimensions that are stepped along are multiples of `per`
// elements, and the base of as many, or of 16 bytes.
bool vec_view(const View& v, int64_t per) {
  const uintptr_t bytes = (uintptr_t)(per * v.esize);
  if (v.base % (bytes < 16 ? bytes : 16) || v.width % per) return false;
  for (int i = 0; i < v.nd; ++i)
    if (v.s[i] % per) return false;
  return true;
}

int check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (!need) return LAPNYS_OK;
  return !ws || ((uintptr_t)ws & 255) || ws_bytes < need ? LAPNYS_ERR_WORKSPACE : LAPNYS_OK;
}

// ---- recurrence

constexpr int64_t kMaxScanColumns = (int64_t)1 << 28;
constexpr int32_t kMaxScanTokens = 1 << 30;

int scan_plan(const lapmix_scan_params* p, lapmix::ScanArgs* a) {
  *a = {};
  if (!p) return LAPNYS_ERR_INVALID_ARG;
  if (p->B <= 0 || p->H <= 0 || p->N <= 0 || p->d <= 0) return LAPNYS_ERR_INVALID_ARG;
  if (p->flags & ~(uint32_t)(LAPMIX_GATE_LOG | LAPMIX_COUPLED)) return LAPNYS_ERR_INVALID_ARG;
  if (!take_strides(p->x_stride, p->B, p->H, p->N, p->d, &a->xs) ||
      !take_strides(p->g_stride, p->B, p->H, p->N, p->d, &a->gs) ||
      !take_strides(p->y_stride, p->B, p->H, p->N, p->d, &a->ys))
    return LAPNYS_ERR_INVALID_ARG;
  if (!storage_type(p->dtype)) return LAPNYS_ERR_UNSUPPORTED;
  // Tokens and columns are counted in 32 bits, a launch's lanes too, elements in 64.
  if ((int64_t)p->B * p->H > kMaxScanColumns || (int64_t)p->B * p->H * p->d > kMaxScanColumns ||
      p->N > kMaxScanTokens)
    return LAPNYS_ERR_UNSUPPORTED;
  a->B = p->B, a->H = p->H, a->N = p->N, a->d = p->d;
  a->dtype = p->dtype;
  a->columns = (long long)p->B * p->H * p->d;
  a->ntiles = (int)(((int64_t)p->N + lapmix::kTile - 1) / lapmix::kTile);
  a->log_gate = (p->flags & LAPMIX_GATE_LOG) != 0;
  a->coupled = (p->flags & LAPMIX_COUPLED) != 0;
  if (a->columns * a->ntiles > ((int64_t)1 << 40)) return LAPNYS_ERR_UNSUPPORTED;
  return LAPNYS_OK;
}

// Rounded up to what workspaces are aligned to.
size_t workspace_bytes(const lapmix::ScanArgs& a) { return (lapmix::scan_workspace(a) + 255) & ~(size_t)255; }

bool element_aligned(const View& v) { return v.base % (uintptr_t)v.esize == 0; }

int scan_forward(const void* x, const void* g, const float* h0, const int32_t* lengths, void* y, float* hN,
                 float* states, const lapmix_scan_params* p, void* ws, size_t ws_bytes, hipStream_t s) {
  lapmix::ScanArgs a;
  int st = scan_plan(p, &a);
  if (st != LAPNYS_OK) return st;
  if (!x || !g || !y) return LAPNYS_ERR_INVALID_ARG;
  const int64_t e = element_size(a.dtype);
  const View vx = strided_view(x, a.B, a.H, a.N, a.d, a.xs, e), vg = strided_view(g, a.B, a.H, a.N, a.d, a.gs, e),
             vy = strided_view(y, a.B, a.H, a.N, a.d, a.ys, e), vh0 = dense_view(h0, a.columns, 4),
             vhN = dense_view(hN, a.columns, 4), vst = dense_view(states, a.columns * a.ntiles, 4),
             vlen = dense_view(lengths, a.B, 4);
  const View all[] = {vx, vg, vy, vh0, vhN, vst, vlen};
  for (const View& v : all)
    if (!element_aligned(v)) return LAPNYS_ERR_INVALID_ARG;
  if (!distinct(vy)) return LAPNYS_ERR_INVALID_ARG;
  const size_t need = workspace_bytes(a);
  const View vws = dense_view(need ? ws : nullptr, (int64_t)need, 1);
  const View out[] = {vy, vhN, vst, vws};
  const View in[] = {vx, vg, h0 == hN ? dense_view(nullptr, 0, 4) : vh0, vlen};
  if (!outputs_apart(out, 4, in, 4) || !disjoint(vh0, vy) || !disjoint(vh0, vst) || !disjoint(vh0, vws))
    return LAPNYS_ERR_INVALID_ARG;
  st = check_workspace(ws, ws_bytes, need);
  if (st != LAPNYS_OK) return st;
  a.vec = vec_view(vx, 4) && vec_view(vg, 4) && vec_view(vy, 4);
  a.x = x, a.g = g, a.h0 = h0, a.lengths = lengths, a.y = y, a.hN = hN, a.states = states;
  (void)hipGetLastError();
  return ok(lapmix::launch_scan_forward(a, ws, s), "recurrence launch") ? LAPNYS_OK : LAPNYS_ERR_HIP;
}

int scan_backward(const void* x, const void* g, const float* states, const int32_t* lengths, const void* dy,
                  const float* dhN, void* dx, void* dg, float* dh0, const lapmix_scan_params* p, void* ws,
                  size_t ws_bytes, hipStream_t s) {
  lapmix::ScanArgs a;
  int st = scan_plan(p, &a);
  if (st != LAPNYS_OK) return st;
  if (!x || !g || !states || !dy || !dx || !dg) return LAPNYS_ERR_INVALID_ARG;
  const int64_t e = element_size(a.dtype);
  const View vx = strided_view(x, a.B, a.H, a.N, a.d, a.xs, e), vg = strided_view(g, a.B, a.H, a.N, a.d, a.gs, e),
             vdy = strided_view(dy, a.B, a.H, a.N, a.d, a.ys, e), vdx = strided_view(dx, a.B, a.H, a.N, a.d, a.xs, e),
             vdg = strided_view(dg, a.B, a.H, a.N, a.d, a.gs, e), vst = dense_view(states, a.columns * a.ntiles, 4),
             vdhN = dense_view(dhN, a.columns, 4), vdh0 = dense_view(dh0, a.columns, 4),
             vlen = dense_view(lengths, a.B, 4);
  const View all[] = {vx, vg, vdy, vdx, vdg, vst, vdhN, vdh0, vlen};
  for (const View& v : all)
    if (!element_aligned(v)) return LAPNYS_ERR_INVALID_ARG;
  if (!distinct(vdx) || !distinct(vdg)) return LAPNYS_ERR_INVALID_ARG;
  const size_t need = workspace_bytes(a);
  const View vws = dense_view(need ? ws : nullptr, (int64_t)need, 1);
  const View out[] = {vdx, vdg, vdh0, vws};
  const View in[] = {vx, vg, vdy, vst, dhN == dh0 ? dense_view(nullptr, 0, 4) : vdhN, vlen};
  if (!outputs_apart(out, 4, in, 6) || !disjoint(vdhN, vdx) || !disjoint(vdhN, vdg) || !disjoint(vdhN, vws))
    return LAPNYS_ERR_INVALID_ARG;
  st = check_workspace(ws, ws_bytes, need);
  if (st != LAPNYS_OK) return st;
  a.vec = vec_view(vx, 4) && vec_view(vg, 4) && vec_view(vdy, 4) && vec_view(vdx, 4) && vec_view(vdg, 4);
  a.x = x, a.g = g, a.states = const_cast<float*>(states), a.lengths = lengths;
  a.dy = dy, a.dhN = dhN, a.dx = dx, a.dg = dg, a.dh0 = dh0;
  (void)hipGetLastError();
  return ok(lapmix::launch_scan_backward(a, ws, s), "recurrence backward launch") ? LAPNYS_OK : LAPNYS_ERR_HIP;
}

int scan_step(const void* x, const void* g, const int32_t* slots, const float* h_in, float* h_out, int32_t n_slots,
              void* y, const lapmix_scan_params* p, hipStream_t s) {
  lapmix::ScanArgs a;
  const int st = scan_plan(p, &a);
  if (st != LAPNYS_OK) return st;
  if (p->N != 1) return LAPNYS_ERR_SHAPE;
  if (!x || !g || !h_in || !h_out || !y || n_slots <= 0) return LAPNYS_ERR_INVALID_ARG;
  if (!slots && n_slots < p->B) return LAPNYS_ERR_SHAPE;
  // A wave takes columns of one sequence: as many sequences as a launch has waves.
  if ((int64_t)p->B * (((int64_t)p->H * p->d + 63) / 64) > (1 << 25)) return LAPNYS_ERR_UNSUPPORTED;
  const int64_t e = element_size(a.dtype), pool = (int64_t)n_slots * a.H * a.d;
  const View vx = strided_view(x, a.B, a.H, 1, a.d, a.xs, e), vg = strided_view(g, a.B, a.H, 1, a.d, a.gs, e),
             vy = strided_view(y, a.B, a.H, 1, a.d, a.ys, e), vin = dense_view(h_in, pool, 4),
             vout = dense_view(h_out, pool, 4), vslots = dense_view(slots, a.B, 4);
  const View all[] = {vx, vg, vy, vin, vout, vslots};
  for (const View& v : all)
    if (!element_aligned(v)) return LAPNYS_ERR_INVALID_ARG;
  if (!distinct(vy)) return LAPNYS_ERR_INVALID_ARG;
  const View out[] = {vy, vout};
  const View in[] = {vx, vg, h_in == h_out ? dense_view(nullptr, 0, 4) : vin, vslots};
  if (!outputs_apart(out, 2, in, 4)) return LAPNYS_ERR_INVALID_ARG;
  lapmix::StepArgs t = {};
  t.B = a.B, t.H = a.H, t.d = a.d, t.n_slots = n_slots;
  t.log_gate = a.log_gate, t.coupled = a.coupled, t.dtype = a.dtype;
  t.vec = vec_view(vx, 4) && vec_view(vg, 4) && vec_view(vy, 4) && aligned(h_in, 16) && aligned(h_out, 16);
  t.xs = a.xs, t.gs = a.gs, t.ys = a.ys;
  t.x = x, t.g = g, t.slots = slots, t.h_in = h_in, t.h_out = h_out, t.y = y;
  (void)hipGetLastError();
  return ok(lapmix::launch_scan_step(t, s), "recurrence step launch") ? LAPNYS_OK : LAPNYS_ERR_HIP;
}

// ---- norm

constexpr int kMaxColumns = 16384;

int norm_plan(const lapmix_norm_params* p, lapmix::NormArgs* a) {
  *a = {};
  if (!p) return LAPNYS_ERR_INVALID_ARG;
  if (p->B <= 0 || p->H <= 0 || p->N <= 0 || p->d <= 0 || p->reserved) return LAPNYS_ERR_INVALID_ARG;
  if (!(isfinite(p->eps) && p->eps > 0.f)) return LAPNYS_ERR_INVALID_ARG;
  if (!take_strides(p->x_stride, p->B, p->H, p->N, p->d, &a->xs)) return LAPNYS_ERR_INVALID_ARG;
  if (!storage_type(p->x_dtype) || !storage_type(p->r_dtype) ||
      !(storage_type(p->y_dtype) || p->y_dtype == LAPMIX_E4M3))
    return LAPNYS_ERR_UNSUPPORTED;
  const int64_t C = (int64_t)p->H * p->d, rows = (int64_t)p->B * p->N;
  if (C > kMaxColumns || rows > INT32_MAX) return LAPNYS_ERR_UNSUPPORTED;
  if (p->group) {
    if (p->y_dtype != LAPMIX_E4M3 || p->group < 16 || p->group > 512 || (p->group & (p->group - 1)))
      return LAPNYS_ERR_INVALID_ARG;
    if (C % p->group) return LAPNYS_ERR_SHAPE;
  }
  a->H = p->H, a->N = p->N, a->d = p->d, a->C = (int)C, a->rows = rows;
  a->x_dtype = p->x_dtype, a->r_dtype = p->r_dtype, a->y_dtype = p->y_dtype;
  a->group = p->group;
  a->eps = p->eps;
  return LAPNYS_OK;
}

int norm_forward(const void* x, const void* r, const float* w, void* s, void* y, float* scale,
                 const lapmix_norm_params* p, hipStream_t stream) {
  lapmix::NormArgs a;
  const int st = norm_plan(p, &a);
  if (st != LAPNYS_OK) return st;
  if (!x || !w || !y) return LAPNYS_ERR_INVALID_ARG;
  const bool e4m3 = a.y_dtype == LAPMIX_E4M3;
  if (e4m3 != (scale != nullptr)) return LAPNYS_ERR_INVALID_ARG;
  const int64_t n = a.rows * a.C;
  const View vx = strided_view(x, p->B, p->H, p->N, p->d, a.xs, element_size(a.x_dtype)),
             vr = dense_view(r, n, element_size(a.r_dtype)), vw = dense_view(w, a.C, 4),
             vs = dense_view(s, n, element_size(a.r_dtype)), vy = dense_view(y, n, element_size(a.y_dtype)),
             vsc = dense_view(scale, a.group ? n / a.group : a.rows, 4);
  const View all[] = {vx, vr, vw, vs, vy, vsc};
  for (const View& v : all)
    if (!element_aligned(v)) return LAPNYS_ERR_INVALID_ARG;
  const View out[] = {vs, vy, vsc};
  const View in[] = {vx, vw, r == s ? dense_view(nullptr, 0, 4) : vr};
  if (!outputs_apart(out, 3, in, 3)) return LAPNYS_ERR_INVALID_ARG;
  // Lanes hold 8 neighbouring columns: 16 bytes of bf16 or 32 of float32.
  a.vec = vec_view(vx, 8) && aligned(r, 16) && aligned(w, 16) && aligned(s, 16) &&
          aligned(y, e4m3 ? 8 : 16);
  if (a.group && !a.vec) return LAPNYS_ERR_UNSUPPORTED;
  a.x = x, a.r = r, a.w = w, a.s = s, a.y = y, a.scale = scale;
  (void)hipGetLastError();
  return ok(lapmix::launch_norm_forward(a, stream), "norm launch") ? LAPNYS_OK : LAPNYS_ERR_HIP;
}

int norm_workspace(const lapmix_norm_params* p, lapmix::NormArgs* a, size_t* bytes) {
  const int st = norm_plan(p, a);
  if (st != LAPNYS_OK) return st;
  if (a->y_dtype == LAPMIX_E4M3) return LAPNYS_ERR_UNSUPPORTED;
  *bytes = (lapmix::norm_part_count(*a) * a->C * sizeof(float) + 255) & ~(size_t)255;
  return LAPNYS_OK;
}

int norm_backward(const void* dy, const void* s, const float* w, const void* ds, void* dr, void* dx, float* dw,
                  const lapmix_norm_params* p, void* ws, size_t ws_bytes, hipStream_t stream) {
  lapmix::NormArgs a;
  size_t need = 0;
  int st = norm_workspace(p, &a, &need);
  if (st != LAPNYS_OK) return st;
  if (!dy || !s || !w || (!dr && !dx && !dw)) return LAPNYS_ERR_INVALID_ARG;
  const int64_t n = a.rows * a.C;
  const View vdy = dense_view(dy, n, element_size(a.y_dtype)), vs = dense_view(s, n, element_size(a.r_dtype)),
             vw = dense_view(w, a.C, 4), vds = dense_view(ds, n, element_size(a.r_dtype)),
             vdr = dense_view(dr, n, element_size(a.r_dtype)),
             vdx = strided_view(dx, p->B, p->H, p->N, p->d, a.xs, element_size(a.x_dtype)),
             vdw = dense_view(dw, a.C, 4);
  const View all[] = {vdy, vs, vw, vds, vdr, vdx, vdw};
  for (const View& v : all)
    if (!element_aligned(v)) return LAPNYS_ERR_INVALID_ARG;
  if (dx && !distinct(vdx)) return LAPNYS_ERR_INVALID_ARG;
  const View vws = dense_view(ws, (int64_t)need, 1);
  const View out[] = {vdr, vdx, vdw, vws};
  const View in[] = {vdy, vs, vw, ds == dr ? dense_view(nullptr, 0, 4) : vds};
  if (!outputs_apart(out, 4, in, 4)) return LAPNYS_ERR_INVALID_ARG;
  if (ds && ds == dr && (!disjoint(vds, vdx) || !disjoint(vds, vdw) || !disjoint(vds, vws)))
    return LAPNYS_ERR_INVALID_ARG;
  st = check_workspace(ws, ws_bytes, need);
  if (st != LAPNYS_OK) return st;
  a.vec = a.d % 8 == 0 && aligned(dy, 16) && aligned(s, 16) && aligned(w, 16) && aligned(ds, 16) && aligned(dr, 16) &&
          (!dx || vec_view(vdx, 8));
  a.dy = dy, a.s = const_cast<void*>(s), a.w = w, a.ds = ds, a.dr = dr, a.dx = dx, a.dw = dw, a.part = (float*)ws;
  (void)hipGetLastError();
  return ok(lapmix::launch_norm_backward(a, stream), "norm backward launch") ? LAPNYS_OK : LAPNYS_ERR_HIP;
}

}  // namespace

extern "C" {

int lapmix_scan_workspace_size(const lapmix_scan_params* p, size_t* bytes) {
  if (!bytes) return LAPNYS_ERR_INVALID_ARG;
  lapmix::ScanArgs a;
  const int st = scan_plan(p, &a);
  if (st != LAPNYS_OK) return st;
  *bytes = workspace_bytes(a);
  return LAPNYS_OK;
}

int lapmix_scan_states_size(const lapmix_scan_params* p, size_t* bytes) {
  if (!bytes) return LAPNYS_ERR_INVALID_ARG;
  lapmix::ScanArgs a;
  const int st = scan_plan(p, &a);
  if (st != LAPNYS_OK) return st;
  *bytes = (size_t)a.columns * a.ntiles * sizeof(float);
  return LAPNYS_OK;
}

int lapmix_scan_forward_ws(const void* x, const void* g, const float* h0, const int32_t* lengths, void* y, float* hN,
                           float* states, const lapmix_scan_params* p, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  return scan_forward(x, g, h0, lengths, y, hN, states, p, ws, ws_bytes, stream);
}

int lapmix_scan_backward_ws(const void* x, const void* g, const float* states, const int32_t* lengths,
                            const void* dy, const float* dhN, void* dx, void* dg, float* dh0,
                            const lapmix_scan_params* p, void* ws, size_t ws_bytes, hipStream_t stream) {
  return scan_backward(x, g, states, lengths, dy, dhN, dx, dg, dh0, p, ws, ws_bytes, stream);
}

int lapmix_scan_step(const void* x, const void* g, const int32_t* slots, const float* h_in, float* h_out,
                     int32_t n_slots, void* y, const lapmix_scan_params* p, hipStream_t stream) {
  return scan_step(x, g, slots, h_in, h_out, n_slots, y, p, stream);
}

int lapmix_norm_forward(const void* x, const void* r, const float* w, void* s, void* y, float* scale,
                        const lapmix_norm_params* p, hipStream_t stream) {
  return norm_forward(x, r, w, s, y, scale, p, stream);
}

int lapmix_norm_workspace_size(const lapmix_norm_params* p, size_t* bytes) {
  if (!bytes) return LAPNYS_ERR_INVALID_ARG;
  lapmix::NormArgs a;
  return norm_workspace(p, &a, bytes);
}

int lapmix_norm_backward_ws(const void* dy, const void* s, const float* w, const void* ds, void* dr, void* dx,
                            float* dw, const lapmix_norm_params* p, void* ws, size_t ws_bytes, hipStream_t stream) {
  return norm_backward(dy, s, w, ds, dr, dx, dw, p, ws, ws_bytes, stream);
}

}  // extern "C"
