// Gated linear recurrence (include/lapmix.h): h_t = f_t h_{t-1} + i_t x_t.
// One lane walks one column (batch, head, channel).
#include <type_traits>

#include "lapmix_internal.hpp"

namespace lapmix {

namespace {

// Forget gate f and 1 - f, each with a small relative error: one of them is
// formed by a quotient (or exp, expm1), the other as 1 minus it only where it is
// at least a half.
template <bool LOG>
__device__ __forceinline__ void gate(float g, float& f, float& rest) {
  if constexpr (LOG) {
    g = g > 0.f ? 0.f : g;  // keeps NaN
    f = __expf(g);
    rest = g > -0.5f ? -expm1f(g) : 1.f - f;
  } else {
    const float e = __expf(-fabsf(g));
    const float big = __frcp_rn(1.f + e), small = e * big;
    f = g < 0.f ? small : big;
    rest = g < 0.f ? big : small;
  }
}

struct Column {
  long long b, h;
  int c;
  int len;
  __device__ Column(const ScanArgs& a, long long col) {
    c = (int)(col % a.d);
    const long long bh = col / a.d;
    h = bh % a.H;
    b = bh / a.H;
    len = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
  }
  __device__ long long at(const Strides& s) const { return b * s.b + h * s.h + c; }
};

template <typename T, bool LOG, bool COUPLED>
__global__ __launch_bounds__(64) void forward_kernel(ScanArgs a) {
  const long long col = (long long)blockIdx.x * 64 + threadIdx.x;
  if (col >= a.columns) return;
  const Column k(a, col);
  const T* x = (const T*)a.x + k.at(a.xs);
  const T* g = (const T*)a.g + k.at(a.gs);
  T* y = (T*)a.y + k.at(a.ys);
  float h = a.h0 ? a.h0[col] : 0.f;
  float* st = a.states ? a.states + (col / a.d) * a.ntiles * a.d + k.c : nullptr;
  for (int n = 0; n < a.N; ++n) {
    if (st && n % kTile == 0) st[(long long)(n / kTile) * a.d] = h;
    float out = 0.f;
    if (n < k.len) {
      float f, rest;
      gate<LOG>(widen(g[n * a.gs.n]), f, rest);
      const float u = widen(x[n * a.xs.n]);
      h = f * h + (COUPLED ? rest * u : u);
      out = h;
    }
    narrow(out, y + n * a.ys.n);
  }
  if (a.hN) a.hN[col] = h;
}

template <typename T, bool LOG, bool COUPLED>
__global__ __launch_bounds__(64) void backward_kernel(ScanArgs a) {
  __shared__ float before[kTile][64];  // h_{t-1} of the tile's tokens
  const long long col = (long long)blockIdx.x * 64 + threadIdx.x;
  if (col >= a.columns) return;
  const int lane = threadIdx.x;
  const Column k(a, col);
  const T* x = (const T*)a.x + k.at(a.xs);
  const T* g = (const T*)a.g + k.at(a.gs);
  const T* dy = (const T*)a.dy + k.at(a.ys);
  T* dx = (T*)a.dx + k.at(a.xs);
  T* dg = (T*)a.dg + k.at(a.gs);
  const float* st = a.states + (col / a.d) * a.ntiles * a.d + k.c;
  float r = a.dhN ? a.dhN[col] : 0.f;  // f_{t+1} dh_{t+1}
  for (int t = a.ntiles - 1; t >= 0; --t) {
    const int n0 = t * kTile, n1 = min(n0 + kTile, a.N);
    float h = st[(long long)t * a.d];
    for (int n = n0; n < min(n1, k.len); ++n) {
      float f, rest;
      gate<LOG>(widen(g[n * a.gs.n]), f, rest);
      const float u = widen(x[n * a.xs.n]);
      before[n - n0][lane] = h;
      h = f * h + (COUPLED ? rest * u : u);
    }
    for (int n = n1 - 1; n >= n0; --n) {
      float gx = 0.f, gg = 0.f;
      if (n < k.len) {
        float f, rest;
        const float gn = widen(g[n * a.gs.n]);
        gate<LOG>(gn, f, rest);
        const float dh = widen(dy[n * a.ys.n]) + r;
        const float hp = before[n - n0][lane];
        gx = COUPLED ? dh * rest : dh;
        gg = dh * (COUPLED ? hp - widen(x[n * a.xs.n]) : hp) * (LOG ? (gn > 0.f ? 0.f : f) : f * rest);
        r = f * dh;
      }
      narrow(gx, dx + n * a.xs.n);
      narrow(gg, dg + n * a.gs.n);
    }
  }
  if (a.dh0) a.dh0[col] = r;
}

template <typename T, bool LOG, bool COUPLED>
__global__ __launch_bounds__(256) void step_kernel(StepArgs a) {
  const long long col = (long long)blockIdx.x * 256 + threadIdx.x;
  const int hd = a.H * a.d;
  if (col >= (long long)a.B * hd) return;
  const int b = (int)(col / hd), hc = (int)(col % hd);
  const int slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) return;
  const long long h = hc / a.d, c = hc % a.d;
  float f, rest;
  gate<LOG>(widen(((const T*)a.g)[b * a.gs.b + h * a.gs.h + c]), f, rest);
  const float u = widen(((const T*)a.x)[b * a.xs.b + h * a.xs.h + c]);
  const long long at = (long long)slot * hd + hc;
  const float v = f * a.h_in[at] + (COUPLED ? rest * u : u);
  a.h_out[at] = v;
  narrow(v, (T*)a.y + b * a.ys.b + h * a.ys.h + c);
}

// Calls f with the storage type, gate and coupling as compile-time values.
template <typename F>
void choose(int dtype, bool log_gate, bool coupled, F f) {
  auto flags = [&](auto t) {
    if (log_gate)
      coupled ? f(t, std::true_type(), std::true_type()) : f(t, std::true_type(), std::false_type());
    else
      coupled ? f(t, std::false_type(), std::true_type()) : f(t, std::false_type(), std::false_type());
  };
  if (dtype == 1)
    flags(uint16_t());
  else
    flags(float());
}

}  // namespace

hipError_t launch_scan_forward(const ScanArgs& a, hipStream_t s) {
  choose(a.dtype, a.log_gate, a.coupled, [&](auto t, auto lg, auto cp) {
    forward_kernel<decltype(t), decltype(lg)::value, decltype(cp)::value>
        <<<dim3((unsigned)((a.columns + 63) / 64)), dim3(64), 0, s>>>(a);
  });
  return hipGetLastError();
}

hipError_t launch_scan_backward(const ScanArgs& a, hipStream_t s) {
  choose(a.dtype, a.log_gate, a.coupled, [&](auto t, auto lg, auto cp) {
    backward_kernel<decltype(t), decltype(lg)::value, decltype(cp)::value>
        <<<dim3((unsigned)((a.columns + 63) / 64)), dim3(64), 0, s>>>(a);
  });
  return hipGetLastError();
}

hipError_t launch_scan_step(const StepArgs& a, hipStream_t s) {
  const long long n = (long long)a.B * a.H * a.d;
  choose(a.dtype, a.log_gate, a.coupled, [&](auto t, auto lg, auto cp) {
    step_kernel<decltype(t), decltype(lg)::value, decltype(cp)::value>
        <<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s>>>(a);
  });
  return hipGetLastError();
}

}  // namespace lapmix
