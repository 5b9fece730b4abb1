// Root-mean-square norm with the residual's addition (include/lapmix.h).
//
// A row is held in registers by a part of a workgroup, or by all of it: lane i has
// the chunks i, i + TPR, ... of V neighbouring columns, so x and r are read once,
// the sum of squares and an e4m3 group's maximum are lane exchanges, and s and y
// are written from the registers.  The backward pass holds dy, s and ds the same
// way, the next row's already on their way while a row is worked on; each
// workgroup takes every gridDim-th row and keeps its part of dw in registers, and
// a second kernel adds the parts in a fixed order.  Both are bound by HBM.
//
// Measured (MI355X, a large copy runs at 5.2 TB/s): 32768 rows of 2048 in bf16 91 us
// forward (5.9 TB/s) and 128 us backward with dr, dx and dw (5.2); 16384 rows of 4096
// to e4m3 86 us with a scale every 128 columns (5.5) and 97 us with one a row, where
// all of the row's waves have to meet a second time; 16384 rows of 2560, forward and backward of a
// training step, 144 us.
#include <type_traits>

#include "lapmix_internal.hpp"

namespace lapmix {

namespace {

constexpr int kNarrow = 256;  // lanes of a workgroup that takes several rows side by side
constexpr int kWide = 1024;   // most lanes of one that takes a row

template <int N>
using Int = std::integral_constant<int, N>;

// V neighbouring elements as loaded.  V = 8 needs 16-byte alignment.
template <typename T, int V>
struct Raw;
template <typename T>
struct Raw<T, 1> {
  T e;
  __device__ __forceinline__ float operator[](int) const { return widen(e); }
};
template <>
struct Raw<float, 8> {
  f32x4 lo, hi;
  __device__ __forceinline__ float operator[](int i) const { return i < 4 ? lo[i] : hi[i - 4]; }
};
template <>
struct Raw<uint16_t, 8> {
  u32x4 e;
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(i % 2 ? e[i / 2] & 0xffff0000u : e[i / 2] << 16);
  }
};

template <int V, typename T>
__device__ __forceinline__ Raw<T, V> get(const T* p) {
  return *(const Raw<T, V>*)p;
}

struct E4M3 {};

// V floats rounded to T.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> pack(const float* v) {
  Raw<T, V> r;
  if constexpr (V == 1) {
    narrow(v[0], &r.e);
  } else if constexpr (sizeof(T) == 4) {
    r.lo = (f32x4){v[0], v[1], v[2], v[3]};
    r.hi = (f32x4){v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.e[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){v[2 * i], v[2 * i + 1]}, lapnys::bf16x2));
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void put(T* p, const float* v) {
  *(Raw<T, V>*)p = pack<T, V>(v);
}

struct Sum {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct Max {  // of what is not NaN
  __device__ double operator()(double a, double b) const { return fmax(a, b); }
};

// Over the lanes of a row (TPR of them, or with TPR = 0 the whole workgroup), in an
// order fixed by the lanes; every lane gets the results.  `shared` has N values for
// each wave; a call may use it again after another barrier.
template <int TPR, int N, typename T, typename F>
__device__ __forceinline__ void over_row(T (&v)[N], T* shared, F f) {
#pragma unroll
  for (int m = 1; m < (TPR ? TPR : 64); m *= 2)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = f(v[k], __shfl_xor(v[k], m));
  if constexpr (TPR == 0) {
    const int waves = blockDim.x / 64, wave = threadIdx.x / 64;
    if (threadIdx.x % 64 == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) shared[wave * N + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = shared[k];
    for (int i = 1; i < waves; ++i)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = f(v[k], shared[i * N + k]);
  }
}

// e4m3: the codes are those of 448 s w / max|s w|, from which the row's factor has
// cancelled, decided in 64 bits, where s w is exact: no value comes to lie on the
// other side of a border between two codes.  Nearly always 32 bits tell as much.

// The largest |y| that makes a scale is never below this.
constexpr double kLeast = 0x1p-100;

__device__ __forceinline__ float scale_of(double m, float rstd) {
  const double top = m * rstd;
  return (float)((top < kLeast ? kLeast : top) * (1. / 448.));
}

// Products of 32 bits in this range, and their remainders, neither overflow nor lose bits.
__device__ __forceinline__ bool ordinary(float z) { return z > 0x1p-90f && z < 0x1p100f; }

// The largest |s w| of a lane, exactly: the largest product rounded to 32 bits, and
// what rounding took from the products that come to it.
template <int V>
__device__ __forceinline__ double largest(const float (&s)[V], const Raw<float, V>& w) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(s[i] * w[i]));
  double t = 0.;
  if (ordinary(m)) {
    float rest = -m;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float r = fmaf(fabsf(s[i]), fabsf(w[i]), -m);
      rest = fabsf(s[i] * w[i]) == m ? fmaxf(rest, r) : rest;
    }
    t = (double)m + (double)rest;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) t = fmax(t, fabs((double)s[i] * (double)w[i]));
  }
  return t;
}

// Four codes, the first in the lowest byte.
__device__ __forceinline__ int codes4(float a, float b, float c, float d) {
  return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
}

// The codes by 32 bits (m: the largest |s w|, rounded); false if they are not certain.
template <int V>
__device__ __forceinline__ bool codes_of(int (&code)[2], const float (&s)[V], const Raw<float, V>& w, float m, float rstd) {
  // 32 bits are off by at most seven roundings, less than 2^-21 of the value: where a
  // little less and a little more than it have the same code, that is the code.
  const float near = __builtin_amdgcn_rcpf(m) * 448.f;
  const float less = near * (1.f - 0x1p-20f), more = near * (1.f + 0x1p-20f);
  auto four = [&](int i, float f) {
    if constexpr (V == 8)
      return codes4(s[i] * w[i] * f, s[i + 1] * w[i + 1] * f, s[i + 2] * w[i + 2] * f, s[i + 3] * w[i + 3] * f);
    else
      return codes4(s[0] * w[0] * f, 0.f, 0.f, 0.f);
  };
  bool sure = ordinary(m) && m * rstd > 2 * (float)kLeast;
#pragma unroll
  for (int k = 0; k < (V == 8 ? 2 : 1); ++k) {
    code[k] = four(4 * k, less);
    sure = sure && code[k] == four(4 * k, more);
  }
  return sure;
}

// The codes by 64 bits.
template <int V>
__device__ __forceinline__ void exact_codes(int (&code)[2], const float (&s)[V], const Raw<float, V>& w, double m,
                                            float rstd) {
  const double factor = m * rstd < kLeast ? rstd * (448. / kLeast) : 448. / m;
  float q[8] = {};
#pragma unroll
  for (int i = 0; i < V; ++i) q[i] = (float)((double)s[i] * (double)w[i] * factor);
#pragma unroll
  for (int k = 0; k < 2; ++k) code[k] = codes4(q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3]);
}

template <int V>
__device__ __forceinline__ void put_codes(uint8_t* p, const int (&code)[2]) {
  if constexpr (V == 8)
    *(int2*)p = make_int2(code[0], code[1]);
  else
    *p = (uint8_t)code[0];
}

// Where a lane works: TPR lanes to a row, or with TPR = 0 the whole workgroup.
template <int TPR>
struct Place {
  int lane, lanes, row, rows;  // of the row; rows side by side
  __device__ Place() {
    lanes = TPR ? TPR : blockDim.x;
    lane = TPR ? threadIdx.x % TPR : threadIdx.x;
    row = TPR ? threadIdx.x / TPR : 0;
    rows = TPR ? kNarrow / TPR : 1;
  }
};

// Offset of column c in a token of x or dx.
__device__ __forceinline__ int64_t in_heads(const NormArgs& a, int c) {
  if (a.H == 1) return c;
  const int h = c / a.d;
  return h * a.xs.h + (c - h * a.d);
}

// X, R, Y: types of x, r and s, and y.  CH chunks of V columns a lane.
template <typename X, typename R, typename Y, int V, int TPR, int CH>
__global__ __launch_bounds__(TPR ? kNarrow : kWide) void norm_forward_kernel(NormArgs a) {
  constexpr bool Q = std::is_same<Y, E4M3>::value;
  __shared__ struct {
    float f[kWide / 64];
    double d[kWide / 64];
  } shared;
  const Place<TPR> at;
  const long long row = a.first + (long long)blockIdx.x * at.rows + at.row;
  if (row >= a.rows) return;  // rows of part of a workgroup need no barrier
  const uint32_t b = (uint32_t)row / (uint32_t)a.N, n = (uint32_t)row % (uint32_t)a.N;
  const X* x = (const X*)a.x + b * a.xs.b + n * a.xs.n;
  Raw<X, V> xr[CH];
  Raw<R, V> rr[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (k * at.lanes + at.lane) * V;
    if (c < a.C) {
      xr[k] = get<V>(x + in_heads(a, c));
      if (a.r) rr[k] = get<V>((const R*)a.r + row * a.C + c);
    }
  }
  float v[CH][V], ss[1] = {0.f};
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (k * at.lanes + at.lane) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) v[k][i] = c < a.C ? (a.r ? xr[k][i] + rr[k][i] : xr[k][i]) : 0.f;
    rr[k] = pack<R, V>(v[k]);
    if (c < a.C && a.s) *(Raw<R, V>*)((R*)a.s + row * a.C + c) = rr[k];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[k][i] = rr[k][i];
      ss[0] += v[k][i] * v[k][i];
    }
  }
  over_row<TPR>(ss, shared.f, Sum());
  const float rstd = 1.f / sqrtf(ss[0] / (float)a.C + a.eps);
  Raw<float, V> w[CH];
  double top[1] = {0.};
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (k * at.lanes + at.lane) * V;
    if (c < a.C) {
      w[k] = get<V>(a.w + c);
      if constexpr (!Q) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] *= rstd * w[k][i];
        put<Y, V>((Y*)a.y + row * a.C + c, v[k]);
      }
    }
    if constexpr (Q) {
      if (a.group) {
        // A group lies in neighbouring lanes of one wave, within a chunk.
        float m = 0.f;
        if (c < a.C)
#pragma unroll
          for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(v[k][i] * w[k][i]));
        for (int o = 1; o < a.group / V; o *= 2) m = fmaxf(m, __shfl_xor(m, o));
        int code[2];
        const bool sure = c >= a.C || codes_of<V>(code, v[k], w[k], m, rstd);
        // The scale goes by what decides it in this group, not by what others in the wave
        // make of it: by 32 bits where they hold the maximum.
        double scaled = m;
        if (!__all(sure)) {
          double exact = c < a.C ? largest<V>(v[k], w[k]) : 0.;
          for (int o = 1; o < a.group / V; o *= 2) exact = fmax(exact, __shfl_xor(exact, o));
          if (!sure) exact_codes<V>(code, v[k], w[k], exact, rstd);
          if (!ordinary(m)) scaled = exact;
        }
        if (c < a.C) {
          if (c % a.group == 0) a.scale[(row * a.C + c) / a.group] = scale_of(scaled, rstd);
          put_codes<V>((uint8_t*)a.y + row * a.C + c, code);
        }
      } else if (c < a.C) {
        top[0] = fmax(top[0], largest<V>(v[k], w[k]));
      }
    }
  }
  if constexpr (Q) {
    if (a.group) return;
    over_row<TPR>(top, shared.d, Max());
    if (at.lane == 0) a.scale[row] = scale_of(top[0], rstd);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * at.lanes + at.lane) * V;
      int code[2];
      if (c >= a.C) continue;
      if (!codes_of<V>(code, v[k], w[k], (float)top[0], rstd)) exact_codes<V>(code, v[k], w[k], top[0], rstd);
      put_codes<V>((uint8_t*)a.y + row * a.C + c, code);
    }
  }
}

template <typename X, typename R, typename Y, int V, int TPR, int CH>
__global__ __launch_bounds__(TPR ? kNarrow : kWide) void norm_backward_kernel(NormArgs a) {
  __shared__ float shared[2][2 * kWide / 64];
  const Place<TPR> at;
  const long long step = (long long)gridDim.x * at.rows;
  Raw<float, V> w[CH];
  float dw[CH][V];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (k * at.lanes + at.lane) * V;
    if (c < a.C) w[k] = get<V>(a.w + c);
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = 0.f;
  }
  struct Row {
    Raw<R, V> s[CH], ds[CH];
    Raw<Y, V> dy[CH];
  };
  // With many chunks columns are worked out anew for each row: kept over the rows, the
  // addresses would not leave room for the row itself (8192 float32 rows of 8191 columns:
  // 433 us, anew 264; with four chunks it costs a tenth).
  int lane = at.lane;
  auto load = [&](long long row, Row& r) {
    if constexpr (CH > 4) asm volatile("" : "+v"(lane));
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * at.lanes + lane) * V;
      if (row < a.rows && c < a.C) {
        r.s[k] = get<V>((const R*)a.s + row * a.C + c);
        r.dy[k] = get<V>((const Y*)a.dy + row * a.C + c);
        if (a.ds) r.ds[k] = get<V>((const R*)a.ds + row * a.C + c);
      }
    }
  };
  // The next row's loads are under way during a row where registers allow.
  constexpr bool AHEAD = V * CH <= 8 && CH <= 4;
  Row next;
  long long row = (long long)blockIdx.x * at.rows + at.row;
  if (AHEAD) load(row, next);
  // Every lane makes the same number of turns: the whole workgroup meets in over_row.
  for (int turn = 0; row - at.row < a.rows; row += step, turn ^= 1) {
    if (!AHEAD) load(row, next);
    const Row r = next;
    if (AHEAD) load(row + step, next);
    const bool on = row < a.rows;
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < CH; ++k)
      if (on && (k * at.lanes + lane) * V < a.C)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sums[0] += r.s[k][i] * r.s[k][i];
          sums[1] += r.dy[k][i] * w[k][i] * r.s[k][i];
        }
    // Two slots in turn: a wave may still read one while another is a row further.
    over_row<TPR>(sums, shared[turn], Sum());
    const float rstd = 1.f / sqrtf(sums[0] / (float)a.C + a.eps);
    const float mean = sums[1] * rstd / (float)a.C;
    if (!on) continue;
    const uint32_t b = (uint32_t)row / (uint32_t)a.N, n = (uint32_t)row % (uint32_t)a.N;
    X* dx = (X*)a.dx + b * a.xs.b + n * a.xs.n;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * at.lanes + lane) * V;
      if (c >= a.C) continue;
      float g[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float u = r.s[k][i] * rstd;
        dw[k][i] += r.dy[k][i] * u;
        g[i] = rstd * (r.dy[k][i] * w[k][i] - u * mean) + (a.ds ? r.ds[k][i] : 0.f);
      }
      if (a.dr) put<R, V>((R*)a.dr + row * a.C + c, g);
      if (a.dx) {
        put<X, V>(dx + in_heads(a, c), g);
      }
    }
  }
  if (!a.dw) return;
  float* part = a.part + (long long)blockIdx.x * a.C;
  if constexpr (TPR != 0) {
    // The rows that the workgroup takes side by side make one part.
    constexpr int ROWS = kNarrow / TPR;
    __shared__ float sums[ROWS][TPR * CH * V];
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) sums[at.row][(k * TPR + at.lane) * V + i] = dw[k][i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.C; c += kNarrow) {
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) sum += sums[r][c];
      part[c] = sum;
    }
  } else {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * at.lanes + at.lane) * V;
      if (c < a.C)
#pragma unroll
        for (int i = 0; i < V; ++i) part[c + i] = dw[k][i];
    }
  }
}

// Adds the parts of dw: a workgroup takes 32 columns, its rows of 32 lanes every 32nd
// part each, kAtOnce of them under way at a time.
constexpr int kAtOnce = 8;

__global__ __launch_bounds__(kWide) void norm_weight_kernel(NormArgs a) {
  constexpr int ROWS = kWide / 32;
  __shared__ float sums[ROWS][33];
  const int lane = threadIdx.x % 32, row = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (c < a.C)
    for (int i = row; i < a.parts; i += ROWS * kAtOnce) {
      float v[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) v[k] = i + k * ROWS < a.parts ? a.part[(long long)(i + k * ROWS) * a.C + c] : 0.f;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) sum += v[k];
    }
  sums[row][lane] = sum;
  __syncthreads();
  // Rows of lanes now take a column each.
  float v[1] = {sums[lane][row]};
#pragma unroll
  for (int m = 1; m < 32; m *= 2) v[0] += __shfl_xor(v[0], m);
  const int out = blockIdx.x * 32 + row;
  if (lane == 0 && out < a.C) a.dw[out] = v[0];
}

// How rows of C columns are laid on lanes: TPR lanes of a workgroup of kNarrow, or
// (tpr = 0) a workgroup of `block` lanes.
struct Shape {
  int v, tpr, ch, block;
  int rows() const { return tpr ? kNarrow / tpr : 1; }
};

Shape shape_of(int C, bool vec) {
  const int v = vec ? 8 : 1, chunks = (C + v - 1) / v;
  auto wide = [&](int ch) { return Shape{v, 0, ch, ((chunks + ch - 1) / ch + 63) / 64 * 64}; };
  if (vec) {
    if (chunks <= 16) return {v, 16, 1, kNarrow};
    if (chunks <= 64) return {v, 64, 1, kNarrow};
    // Two chunks a lane beyond 1024 columns: fewer waves meet at the barriers.  (16384
    // rows of 4096 to e4m3: 99.0 us with one chunk, 86.9 with two; 32768 of 2048: 97.6
    // and 92.7; to bf16 92.7 and 90.9, backward 135 and 128.)
    return wide(chunks <= 128 ? 1 : 2);
  }
  if (chunks <= 64) return {v, 64, 1, kNarrow};
  return wide(chunks <= 4096 ? 4 : chunks <= 8192 ? 8 : 16);
}

template <typename F>
void with_shape(const Shape& s, F f) {
  if (s.v == 8) {
    if (s.tpr == 16) return f(Int<8>(), Int<16>(), Int<1>());
    if (s.tpr == 64) return f(Int<8>(), Int<64>(), Int<1>());
    return s.ch == 1 ? f(Int<8>(), Int<0>(), Int<1>()) : f(Int<8>(), Int<0>(), Int<2>());
  }
  if (s.tpr == 64) return f(Int<1>(), Int<64>(), Int<1>());
  if (s.ch == 4) return f(Int<1>(), Int<0>(), Int<4>());
  return s.ch == 8 ? f(Int<1>(), Int<0>(), Int<8>()) : f(Int<1>(), Int<0>(), Int<16>());
}

template <typename F>
void with_types(const NormArgs& a, F f) {
  auto y = [&](auto x, auto r) {
    if (a.y_dtype == 2) return f(x, r, E4M3());
    if (a.y_dtype == 1) return f(x, r, uint16_t());
    return f(x, r, float());
  };
  auto r = [&](auto x) { a.r_dtype == 1 ? y(x, uint16_t()) : y(x, float()); };
  a.x_dtype == 1 ? r(uint16_t()) : r(float());
}

}  // namespace

// Workgroups of the backward pass: about 16 waves to each of the 256 CUs, so that
// the parts of dw stay small beside the rows, and four rows or more for each.  (16384
// rows of 2560 bf16 columns, 5 waves a row: 114 us with 256 workgroups, 86 with 512,
// 88 with 1024, 97 with 2048; 4096 rows of 1024, 2 waves: 21.7, 16.1, 14.6, 17.3; 65536
// float32 rows of 67, 1 wave: 71 with 1024, 46 with 2048, 39 with 4096.)
static int norm_groups(long long rows, const Shape& shape) {
  const long long n = (rows + 4 * shape.rows() - 1) / (4 * shape.rows());
  const int waves = shape.block / 64, most = waves > 4 ? 512 : waves > 1 ? 1024 : 4096;
  return (int)(n < most ? n : most);
}

size_t norm_part_count(const NormArgs& a) {
  size_t most = 0;
  for (bool vec : {false, true}) {
    const Shape shape = shape_of(a.C, vec);
    const size_t n = (size_t)norm_groups(a.rows, shape);
    most = n > most ? n : most;
  }
  return most;
}

hipError_t launch_norm_forward(const NormArgs& args, hipStream_t s) {
  NormArgs a = args;
  const Shape shape = shape_of(a.C, a.vec);
  // A launch has at most 2^32 - 1 lanes: many rows go in several.
  const long long most = ((long long)1 << 31) / shape.block;
  hipError_t e = hipSuccess;
  for (a.first = 0; a.first < a.rows && e == hipSuccess; a.first += most * shape.rows()) {
    const long long groups = (a.rows - a.first + shape.rows() - 1) / shape.rows();
    const dim3 grid((unsigned)(groups < most ? groups : most)), block(shape.block);
    with_types(a, [&](auto x, auto r, auto y) {
      with_shape(shape, [&](auto v, auto tpr, auto ch) {
        norm_forward_kernel<decltype(x), decltype(r), decltype(y), decltype(v)::value, decltype(tpr)::value,
                            decltype(ch)::value><<<grid, block, 0, s>>>(a);
      });
    });
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_norm_backward(const NormArgs& args, hipStream_t s) {
  NormArgs a = args;
  const Shape shape = shape_of(a.C, a.vec);
  const int groups = norm_groups(a.rows, shape);
  a.parts = groups;
  with_types(a, [&](auto x, auto r, auto y) {
    if constexpr (!std::is_same<decltype(y), E4M3>::value)
      with_shape(shape, [&](auto v, auto tpr, auto ch) {
        norm_backward_kernel<decltype(x), decltype(r), decltype(y), decltype(v)::value, decltype(tpr)::value,
                             decltype(ch)::value><<<dim3(groups), dim3(shape.block), 0, s>>>(a);
      });
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.dw) return e;
  norm_weight_kernel<<<dim3((unsigned)((a.C + 31) / 32)), dim3(kWide), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace lapmix
