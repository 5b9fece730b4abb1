// Internal declarations of the lapmix operators (include/lapmix.h): kernel
// arguments and launchers.  Not part of the public C ABI.
#pragma once

#include "lapnys_internal.hpp"

namespace lapmix {

using lapnys::f32x2;
using lapnys::f32x4;
using lapnys::u32x4;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
using lapnys::widen;

constexpr int kTile = 128;  // tokens of a tile (LAPMIX_SCAN_TILE)

// Element strides of a [B, H, N, d] tensor whose channels are contiguous.
struct Strides {
  int64_t b, h, n;
};

// Rounds a float32 to the storage type, to nearest even (NaN stays NaN).
__device__ __forceinline__ void narrow(float v, float* out) { *out = v; }
__device__ __forceinline__ void narrow(float v, uint16_t* out) { *out = __builtin_bit_cast(uint16_t, (__bf16)v); }

struct ScanArgs {
  int B, H, N, d;
  int ntiles;         // ceil(N / kTile)
  long long columns;  // B * H * d
  bool log_gate, coupled;
  int dtype;
  bool vec;           // every base and stride allows 16-byte accesses
  Strides xs, gs, ys;
  const void *x, *g;
  const int32_t* lengths;
  const float* h0;    // forward
  void* y;
  float* hN;
  float* states;
  const void* dy;     // backward
  const float* dhN;
  void *dx, *dg;
  float* dh0;
};

struct StepArgs {
  int B, H, d, n_slots;
  bool log_gate, coupled;
  int dtype;
  bool vec;
  Strides xs, gs, ys;
  const void *x, *g;
  const int32_t* slots;
  const float* h_in;
  float* h_out;
  void* y;
};

// Workspace bytes of a forward or backward call (0 where none is needed).
size_t scan_workspace(const ScanArgs& a);
hipError_t launch_scan_forward(const ScanArgs& a, void* ws, hipStream_t s);
hipError_t launch_scan_backward(const ScanArgs& a, void* ws, hipStream_t s);
hipError_t launch_scan_step(const StepArgs& a, hipStream_t s);

struct NormArgs {
  int H, N, d, C;
  long long rows;    // B * N
  long long first;   // the launch's first row (forward)
  int x_dtype, r_dtype, y_dtype, group;
  float eps;
  bool vec;
  Strides xs;
  const void *x, *r;
  const float* w;
  void *s, *y;
  float* scale;
  const void *dy, *ds;  // backward
  void *dr, *dx;
  float *dw, *part;     // part: [parts][C] partial sums of dw
  int parts;
};

// Partial sums of dw that a backward call may write.
size_t norm_part_count(const NormArgs& a);
hipError_t launch_norm_forward(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s);

}  // namespace lapmix
