// Root-mean-square norm with the residual's addition (include/lapmix.h).
// One wave takes one row at a time, a column a lane.
#include <type_traits>

#include "lapmix_internal.hpp"

namespace lapmix {

namespace {

constexpr int kE4M3 = 2;

__device__ __forceinline__ float wave_sum(float v) {
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ float load(const void* p, int type, long long i) {
  return type == 1 ? widen(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}

__device__ __forceinline__ void store(void* p, int type, long long i, float v) {
  if (type == 1)
    narrow(v, (uint16_t*)p + i);
  else
    ((float*)p)[i] = v;
}

__device__ __forceinline__ float rounded(float v, int type) { return type == 1 ? (float)(__bf16)v : v; }

// e4m3 code of v, |v| <= 448 (NaN gives NaN).
__device__ __forceinline__ uint8_t e4m3(float v) {
  return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xff);
}

__device__ __forceinline__ float stored_sum(const NormArgs& a, long long row, int c) {
  const long long b = row / a.N, n = row % a.N;
  float v = load(a.x, a.x_dtype, b * a.xs.b + (c / a.d) * a.xs.h + n * a.xs.n + c % a.d);
  if (a.r) v += load(a.r, a.r_dtype, row * a.C + c);
  return rounded(v, a.r_dtype);
}

// The largest |y| of a group is never below this when it makes a scale: its
// reciprocal stays finite.
constexpr float kLeast = 0x1p-100f;

__global__ __launch_bounds__(64) void forward_kernel(NormArgs a) {
  const long long row = blockIdx.x;
  const int lane = threadIdx.x;
  float sum = 0.f;
  for (int c = lane; c < a.C; c += 64) {
    const float v = stored_sum(a, row, c);
    sum += v * v;
  }
  const float rstd = 1.f / sqrtf(wave_sum(sum) / (float)a.C + a.eps);
  const int group = a.group ? a.group : a.C;
  for (int g0 = 0; g0 < a.C; g0 += group) {
    float scale = 1.f, inv = 1.f;
    if (a.y_dtype == kE4M3) {
      float top = 0.f;
      for (int c = g0 + lane; c < g0 + group; c += 64) {
        const float v = fabsf(stored_sum(a, row, c) * rstd * a.w[c]);
        top = v > top || v != v ? v : top;
      }
      for (int m = 32; m; m >>= 1) {
        const float o = __shfl_xor(top, m);
        top = o > top || o != o ? o : top;
      }
      top = top < kLeast ? kLeast : top;
      scale = top / 448.f;
      inv = 448.f / top;
      if (lane == 0) a.scale[(row * a.C + g0) / group] = scale;
    }
    for (int c = g0 + lane; c < g0 + group; c += 64) {
      const float v = stored_sum(a, row, c), y = v * rstd * a.w[c];
      if (a.s) store(a.s, a.r_dtype, row * a.C + c, v);
      if (a.y_dtype == kE4M3)
        ((uint8_t*)a.y)[row * a.C + c] = e4m3(y * inv);
      else
        store(a.y, a.y_dtype, row * a.C + c, y);
    }
  }
}

__global__ __launch_bounds__(64) void backward_kernel(NormArgs a) {
  const int lane = threadIdx.x;
  const long long per = (a.rows + a.parts - 1) / a.parts;
  const long long r0 = blockIdx.x * per, r1 = min(a.rows, r0 + per);
  if (a.dw)
    for (int c = lane; c < a.C; c += 64) a.part[(long long)blockIdx.x * a.C + c] = 0.f;
  for (long long row = r0; row < r1; ++row) {
    const long long o = row * a.C;
    float ss = 0.f, dot = 0.f;
    for (int c = lane; c < a.C; c += 64) {
      const float v = load(a.s, a.r_dtype, o + c);
      ss += v * v;
      dot += load(a.dy, a.y_dtype, o + c) * a.w[c] * v;
    }
    const float rstd = 1.f / sqrtf(wave_sum(ss) / (float)a.C + a.eps);
    const float mean = wave_sum(dot) * rstd / (float)a.C;
    const long long b = row / a.N, n = row % a.N;
    for (int c = lane; c < a.C; c += 64) {
      const float u = load(a.s, a.r_dtype, o + c) * rstd, dy = load(a.dy, a.y_dtype, o + c);
      const float v = rstd * (dy * a.w[c] - u * mean) + (a.ds ? load(a.ds, a.r_dtype, o + c) : 0.f);
      if (a.dr) store(a.dr, a.r_dtype, o + c, v);
      if (a.dx) store(a.dx, a.x_dtype, b * a.xs.b + (c / a.d) * a.xs.h + n * a.xs.n + c % a.d, v);
      if (a.dw) a.part[(long long)blockIdx.x * a.C + c] += dy * u;
    }
  }
}

__global__ __launch_bounds__(64) void weight_kernel(NormArgs a) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= a.C) return;
  float sum = 0.f;
  for (int i = 0; i < a.parts; ++i) sum += a.part[(long long)i * a.C + c];
  a.dw[c] = sum;
}

}  // namespace

int norm_parts(long long rows, int) { return (int)(rows < 512 ? rows : 512); }

hipError_t launch_norm_forward(const NormArgs& a, hipStream_t s) {
  forward_kernel<<<dim3((unsigned)a.rows), dim3(64), 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s) {
  backward_kernel<<<dim3((unsigned)a.parts), dim3(64), 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.dw) return e;
  weight_kernel<<<dim3((unsigned)((a.C + 63) / 64)), dim3(64), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace lapmix
