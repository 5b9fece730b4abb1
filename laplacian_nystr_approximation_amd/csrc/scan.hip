// Gated linear recurrence (include/lapmix.h): h_t = f_t h_{t-1} + i_t x_t.
//
// Any run of tokens maps the state before it to the state behind it by
// h -> A h + S (A the product of its gates, S its result from a zero state),
// and two runs compose to (A2 A1, A2 S1 + S2).  A workgroup takes a tile of
// kTile tokens by a few dozen columns (batch, head, channel): each lane holds a
// few consecutive tokens of 16 bytes' worth of neighbouring channels, walks them
// once for its (A, S), the lanes' pairs are composed over the wave by lane
// exchange and over the workgroup through LDS, and with the state before the tile
// known each lane walks its tokens a second time, in registers, and writes y.
// x and g are read once and y is written once: the kernel is bound by HBM.
//
// The state before a tile comes from one of two places.
//  - Loop form: the workgroup takes all tiles of its columns one after the other.
//  - Chain form, for few columns: every tile is a workgroup of its own.  Tiles
//    publish their (A, S), and every 16th tile the pair of its 16 tiles and every
//    256th that of its 256, so that a tile composes at most 15 + 15 pairs and
//    one for each 65536 tokens before it.  Which pairs are composed, and in which
//    order, depends on the tile's place alone: results repeat bit for bit.
//
// Waits end: a tile takes its place from a counter, in the order in which
// workgroups start, so it waits only for tiles of workgroups that have started
// before it, and the first unfinished one of those waits for nothing.
//
// The backward pass runs the tiles from the last to the first with r = f dh in
// the place of h (r_t = f_t (dy_t + r_{t+1})), and recomputes the tile's h from
// the state that the forward kept before it.
#include <type_traits>

#include "lapmix_internal.hpp"

namespace lapmix {

namespace {

constexpr int kFan = 16;  // tiles whose pairs are composed into one

struct Pair {
  float a, s;
};

__device__ __forceinline__ Pair compose(Pair first, Pair then) { return {then.a * first.a, then.a * first.s + then.s}; }

// A published pair.  The workspace is filled with kUnset before the launch; a
// published A is never that pattern (a NaN is stored as the canonical one), so
// the 64-bit word tells by itself whether it is there, and no fence is needed.
constexpr uint64_t kUnset = ~(uint64_t)0;
constexpr int kFillThreads = 256;

__global__ __launch_bounds__(kFillThreads) void scan_fill_kernel(uint64_t* words, long long n) {
  const long long i = (long long)blockIdx.x * kFillThreads + threadIdx.x;
  // Word 0 is the tile counter.
  if (i < n) words[i] = i == 0 ? 0 : kUnset;
}

__device__ __forceinline__ void publish(uint64_t* at, Pair p) {
  if (p.a != p.a) p.a = __builtin_nanf("");
  const uint64_t w = ((uint64_t)__float_as_uint(p.s) << 32) | __float_as_uint(p.a);
  __hip_atomic_store(at, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ uint64_t peek(const uint64_t* at) {
  return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ bool unset(uint64_t w) { return (uint32_t)w == (uint32_t)kUnset; }

__device__ __forceinline__ Pair pair_of(uint64_t w) {
  return {__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}

// Waits until a pair that was seen as `w` is there.  The bound on the polls only
// matters if a workspace is written from outside while the kernel runs: the
// results are then NaN.
__device__ __forceinline__ Pair wait_for(const uint64_t* at, uint64_t w) {
  for (int tries = 0; unset(w) && tries < (1 << 20); ++tries) {
    __builtin_amdgcn_s_sleep(1);
    w = peek(at);
  }
  return pair_of(w);
}

// The words of a launch's chain: the counter, then for each level [places][columns].
struct Chain {
  uint64_t* words;
  long long columns;
  long long level[3];  // first word of each level
};

__host__ __device__ inline long long chain_layout(int ntiles, long long columns, long long level[3]) {
  long long at = 32, n = ntiles;  // the counter has 256 bytes of its own
  for (int i = 0; i < 3; ++i) {
    level[i] = at;
    at += n * columns;
    n /= kFan;
  }
  return at;
}

// The pair of everything before place p for the columns of a workgroup of NT lanes,
// returned to the lanes tid < WIDTH, each with its own column's `own` pair.  The
// pairs to compose are spread over the workgroup (SLOTS lanes a column), so all
// of them are in flight at once.  All lanes call it.
template <int NT, int WIDTH>
__device__ __forceinline__ Pair chain_before(const Chain& c, int p, int last, uint32_t base, Pair own) {
  constexpr int SLOTS = NT / WIDTH < kFan ? NT / WIDTH : kFan, EACH = kFan / SLOTS;
  __shared__ Pair part[2][SLOTS][WIDTH];
  const int tid = threadIdx.x, slot = tid / WIDTH, lane = tid % WIDTH;
  const bool on = base + lane < (uint64_t)c.columns;
  uint64_t* w = c.words + (on ? base + lane : 0);
  const int p0 = p % kFan, q = p / kFan, q0 = q % kFan, t = q / kFan;
  if (slot == 0 && on && p < last) publish(w + c.level[0] + (long long)p * c.columns, own);
  const uint64_t* near = w + c.level[0] + (long long)(p - p0) * c.columns;
  const uint64_t* mid = w + c.level[1] + (long long)(q - q0) * c.columns;
  uint64_t wn[EACH], wm[EACH];
  const bool works = on && slot < SLOTS;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int k = slot * EACH + i;
    wn[i] = works && k < p0 ? peek(near + k * c.columns) : 0;
    wm[i] = works && k < q0 ? peek(mid + k * c.columns) : 0;
  }
  Pair sum = {1.f, 0.f};
#pragma unroll
  for (int i = 0; i < EACH; ++i)
    if (works && slot * EACH + i < p0) sum = compose(sum, wait_for(near + (slot * EACH + i) * c.columns, wn[i]));
  if (slot < SLOTS) part[0][slot][lane] = sum;
  __syncthreads();
  Pair before = {1.f, 0.f}, sixteen = {1.f, 0.f};
  if (slot == 0) {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) before = compose(before, part[0][i][lane]);
    // Published before anything else is waited for: the next tiles need it.
    if (p0 == kFan - 1) {
      sixteen = compose(before, own);
      if (on && p < last) publish(w + c.level[1] + (long long)q * c.columns, sixteen);
    }
  }
  if (q == 0) return before;
  sum = {1.f, 0.f};
#pragma unroll
  for (int i = 0; i < EACH; ++i)
    if (works && slot * EACH + i < q0) sum = compose(sum, wait_for(mid + (slot * EACH + i) * c.columns, wm[i]));
  if (slot < SLOTS) part[1][slot][lane] = sum;
  __syncthreads();
  if (slot == 0) {
    Pair m = {1.f, 0.f};
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) m = compose(m, part[1][i][lane]);
    if (p0 == kFan - 1 && q0 == kFan - 1 && on && p < last)
      publish(w + c.level[2] + (long long)t * c.columns, compose(m, sixteen));
    before = compose(m, before);
  }
  if (t == 0) return before;
  sum = {1.f, 0.f};
  const uint64_t* far = w + c.level[2];
  const int each = (t + SLOTS - 1) / SLOTS;
  for (int k = slot * each; works && k < min(t, slot * each + each); ++k)
    sum = compose(sum, wait_for(far + k * c.columns, peek(far + k * c.columns)));
  if (slot < SLOTS) part[0][slot][lane] = sum;
  __syncthreads();
  if (slot == 0) {
    Pair m = {1.f, 0.f};
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) m = compose(m, part[0][i][lane]);
    before = compose(m, before);
  }
  return before;
}

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
    const float big = __builtin_amdgcn_rcpf(1.f + e), small = e * big;
    f = g < 0.f ? small : big;
    rest = g < 0.f ? big : small;
  }
}

// A gate in one register, for a gate that is needed with both f and 1 - f again
// later: the smaller of them, with the sign bit where it is f.
__device__ __forceinline__ float pack_gate(float f, float rest) {
  return f < rest ? -f : fabsf(rest);
}

__device__ __forceinline__ void unpack_gate(float c, float& f, float& rest) {
  const float small = fabsf(c), big = 1.f - small;
  const bool is_f = __float_as_uint(c) >> 31;
  f = is_f ? small : big;
  rest = is_f ? big : small;
}

// Keeps a value in its register: what is derived from it again later is derived
// again, and does not stay alive in between.
__device__ __forceinline__ void keep(float& v) { asm volatile("" : "+v"(v)); }

// V neighbouring channels of a token, as loaded: 16 bytes, or one element.
template <typename T, int V>
struct Raw {
  using type = u32x4;
};
template <typename T>
struct Raw<T, 1> {
  using type = T;
};

template <typename T, int V>
__device__ __forceinline__ float element(const typename Raw<T, V>::type& raw, int v) {
  if constexpr (V == 1)
    return widen(raw);
  else if constexpr (sizeof(T) == 4)
    return __uint_as_float(raw[v]);
  else
    return __uint_as_float(v % 2 ? raw[v / 2] & 0xffff0000u : raw[v / 2] << 16);
}

template <typename T, int V>
__device__ __forceinline__ void put(T* at, const float* v) {
  if constexpr (V == 1) {
    narrow(v[0], at);
  } else if constexpr (sizeof(T) == 4) {
    *(f32x4*)at = (f32x4){v[0], v[1], v[2], v[3]};
  } else {
    u32x4 out;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      out[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){v[2 * i], v[2 * i + 1]}, lapnys::bf16x2));
    *(u32x4*)at = out;
  }
}

// Geometry of a workgroup of NT lanes with L tokens and V channels a lane.
template <int NT, int L, int V>
struct Tile {
  static constexpr int kCols = NT * L / kTile;  // lanes side by side
  static constexpr int kWidth = kCols * V;      // columns
  static constexpr int kWaves = NT / 64;
  static_assert(kCols >= 1 && kCols <= 32 && kWidth <= 64, "a wave holds whole rows of lanes");
};

// Exclusive scan of the lanes' pairs over the tile's rows, in the order of rising
// tokens (or falling ones).  Returns the pair of the rows before the lane's within
// its wave; `total` receives the waves' pairs.
template <int COLS, int V, bool REVERSE>
__device__ __forceinline__ void wave_scan(Pair p[V], Pair before[V]) {
  const int lane = threadIdx.x & 63;
  const int row = REVERSE ? (63 - lane) / COLS : lane / COLS;
  auto other = [&](float v, int rows) {
    return REVERSE ? __shfl_down(v, rows * COLS) : __shfl_up(v, rows * COLS);
  };
#pragma unroll
  for (int rows = 1; rows < 64 / COLS; rows *= 2)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Pair o = {other(p[v].a, rows), other(p[v].s, rows)};
      if (row >= rows) p[v] = compose(o, p[v]);
    }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    before[v] = {other(p[v].a, 1), other(p[v].s, 1)};
    if (row == 0) before[v] = {1.f, 0.f};
  }
}

// What a lane is in charge of.
struct Lane {
  uint32_t col;  // first column
  bool on;       // columns exist
  int len;       // tokens of the sequence
  int64_t x, g, y;
};

__device__ __forceinline__ Lane lane_of(const ScanArgs& a, uint32_t col) {
  Lane l;
  l.on = col < (uint32_t)a.columns;
  l.col = l.on ? col : 0;
  const uint32_t c = l.col % (uint32_t)a.d, bh = l.col / (uint32_t)a.d;
  const uint32_t h = bh % (uint32_t)a.H, b = bh / (uint32_t)a.H;
  l.len = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
  l.x = (int64_t)b * a.xs.b + (int64_t)h * a.xs.h + c;
  l.g = (int64_t)b * a.gs.b + (int64_t)h * a.gs.h + c;
  l.y = (int64_t)b * a.ys.b + (int64_t)h * a.ys.h + c;
  return l;
}

// The kept state before tile t of column col.
__device__ __forceinline__ float* state_at(const ScanArgs& a, uint32_t col, int t) {
  const uint32_t c = col % (uint32_t)a.d, bh = col / (uint32_t)a.d;
  return a.states + ((int64_t)bh * a.ntiles + t) * a.d + c;
}

template <typename T, int V, int NT, int L, bool LOG, bool COUPLED, bool CHAIN>
__global__ __launch_bounds__(NT) void scan_forward_kernel(ScanArgs a, Chain chain, int groups) {
  using G = Tile<NT, L, V>;
  using R = typename Raw<T, V>::type;
  __shared__ Pair totals[2][G::kWaves][G::kWidth];
  __shared__ float start[G::kWidth];
  __shared__ int place;
  const int tid = threadIdx.x, wave = tid / 64, cv = tid % G::kCols, row = tid / G::kCols;
  int group = blockIdx.x, tile = 0;
  if constexpr (CHAIN) {
    if (tid == 0) place = (int)atomicAdd((unsigned*)chain.words, 1u);
    __syncthreads();
    tile = place / groups;
    group = place % groups;
  }
  const uint32_t base = (uint32_t)group * G::kWidth;
  const Lane me = lane_of(a, base + cv * V);
  const T* x = (const T*)a.x + me.x;
  const T* g = (const T*)a.g + me.g;
  T* y = (T*)a.y + me.y;
  const int stored = me.on ? a.N : 0;
  // Lanes of the first wave also look after one column each: its carried state.
  const uint32_t mine = base + tid;
  const bool keeper = tid < G::kWidth && mine < (uint32_t)a.columns;
  float h_keep = keeper && a.h0 ? a.h0[mine] : 0.f;

  for (;; ++tile) {
    const int n0 = tile * kTile + row * L;
    R xr[L], gr[L];
    // Tokens behind the sequence's end read its last one and are masked below.
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int64_t n = max(min(n0 + j, me.len - 1), 0);
      gr[j] = *(const R*)(g + n * a.gs.n);
      xr[j] = *(const R*)(x + n * a.xs.n);
    }
    float f[L][V], u[L][V];
    Pair p[V], before[V];
    for (int v = 0; v < V; ++v) p[v] = {1.f, 0.f};
    const bool full = __all(tile * kTile + kTile <= me.len);
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float rest;
        gate<LOG>(element<T, V>(gr[j], v), f[j][v], rest);
        u[j][v] = element<T, V>(xr[j], v);
        if (COUPLED) u[j][v] *= rest;
        if (!full && n0 + j >= me.len) f[j][v] = 1.f, u[j][v] = 0.f;
        p[v] = compose(p[v], {f[j][v], u[j][v]});
      }
    wave_scan<G::kCols, V, false>(p, before);
    auto& tot = totals[tile & 1];
    if ((tid & 63) >= 64 - G::kCols)
#pragma unroll
      for (int v = 0; v < V; ++v) tot[wave][cv * V + v] = p[v];
    __syncthreads();
    Pair own = {1.f, 0.f};
    if (tid < G::kWidth) {
      own = tot[0][tid];
#pragma unroll
      for (int i = 1; i < G::kWaves; ++i) own = compose(own, tot[i][tid]);
    }
    float h = h_keep;
    if constexpr (CHAIN) {
      // The first tile's pair holds the initial state, which no other tile reads.
      if (tile == 0) own = {0.f, own.a * h + own.s};
      const Pair b = chain_before<NT, G::kWidth>(chain, tile, a.ntiles - 1, base, own);
      if (tile > 0) h = b.s;
      h_keep = tile == 0 ? own.s : own.a * h + own.s;
    } else {
      h_keep = own.a * h + own.s;
    }
    if (keeper) {
      start[tid] = h;
      if (a.states) *state_at(a, mine, tile) = h;
      if (a.hN && tile == a.ntiles - 1) a.hN[mine] = h_keep;
    }
    __syncthreads();
    float at[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      at[v] = start[cv * V + v];
      for (int i = 0; i < wave; ++i) at[v] = tot[i][cv * V + v].a * at[v] + tot[i][cv * V + v].s;
      at[v] = before[v].a * at[v] + before[v].s;
    }
#pragma unroll
    for (int j = 0; j < L; ++j) {
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        at[v] = f[j][v] * at[v] + u[j][v];
        out[v] = !full && n0 + j >= me.len ? 0.f : at[v];
      }
      if (n0 + j < stored) put<T, V>(y + (int64_t)(n0 + j) * a.ys.n, out);
    }
    if (CHAIN || tile == a.ntiles - 1) break;
  }
}

template <typename T, int V, int NT, int L, bool LOG, bool COUPLED, bool CHAIN>
__global__ __launch_bounds__(NT) void scan_backward_kernel(ScanArgs a, Chain chain, int groups) {
  using G = Tile<NT, L, V>;
  using R = typename Raw<T, V>::type;
  __shared__ Pair totals[2][2][G::kWaves][G::kWidth];  // forward and backward pairs
  __shared__ float start[2][G::kWidth];
  __shared__ int place;
  const int tid = threadIdx.x, wave = tid / 64, cv = tid % G::kCols, row = tid / G::kCols;
  int group = blockIdx.x, step = 0;
  if constexpr (CHAIN) {
    if (tid == 0) place = (int)atomicAdd((unsigned*)chain.words, 1u);
    __syncthreads();
    step = place / groups;
    group = place % groups;
  }
  const uint32_t base = (uint32_t)group * G::kWidth;
  const Lane me = lane_of(a, base + cv * V);
  const T* x = (const T*)a.x + me.x;
  const T* g = (const T*)a.g + me.g;
  const T* dy = (const T*)a.dy + me.y;
  T* dx = (T*)a.dx + me.x;
  T* dg = (T*)a.dg + me.g;
  const int stored = me.on ? a.N : 0;
  const uint32_t mine = base + tid;
  const bool keeper = tid < G::kWidth && mine < (uint32_t)a.columns;
  float r_keep = keeper && a.dhN ? a.dhN[mine] : 0.f;

  for (;; ++step) {
    const int tile = a.ntiles - 1 - step;
    const int n0 = tile * kTile + row * L;
    R xr[L], gr[L], yr[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int64_t n = max(min(n0 + j, me.len - 1), 0);
      gr[j] = *(const R*)(g + n * a.gs.n);
      yr[j] = *(const R*)(dy + n * a.ys.n);
      xr[j] = *(const R*)(x + n * a.xs.n);
    }
    const float h_keep = keeper ? *state_at(a, mine, tile) : 0.f;
    const bool full = __all(tile * kTile + kTile <= me.len);
    // Behind the sequence's end gates are 1 and x and dy are 0.
    constexpr bool BOTH = COUPLED || !LOG;  // 1 - f is needed too
    float c[L][V];
    auto decode = [&](int j, int v, float& f, float& rest) {
      if constexpr (BOTH)
        unpack_gate(c[j][v], f, rest);
      else
        f = c[j][v];
    };
    Pair p[V], hb[V], rb[V];
    for (int v = 0; v < V; ++v) p[v] = {1.f, 0.f};
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f, rest, u = element<T, V>(xr[j], v);
        gate<LOG>(element<T, V>(gr[j], v), f, rest);
        if (COUPLED) u *= rest;
        c[j][v] = BOTH ? pack_gate(f, rest) : f;
        if (!full && n0 + j >= me.len) f = 1.f, u = 0.f, c[j][v] = BOTH ? 0.f : 1.f;
        p[v] = compose(p[v], {f, u});
        keep(c[j][v]);
      }
    auto& tot = totals[step & 1];
    wave_scan<G::kCols, V, false>(p, hb);
    if ((tid & 63) >= 64 - G::kCols)
#pragma unroll
      for (int v = 0; v < V; ++v) tot[0][wave][cv * V + v] = p[v];
    for (int v = 0; v < V; ++v) p[v] = {1.f, 0.f};
#pragma unroll
    for (int j = L - 1; j >= 0; --j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f, rest, e = element<T, V>(yr[j], v);
        decode(j, v, f, rest);
        if (!full && n0 + j >= me.len) e = 0.f;
        p[v] = {p[v].a * f, f * (p[v].s + e)};
        keep(c[j][v]);
      }
    wave_scan<G::kCols, V, true>(p, rb);
    if ((tid & 63) < G::kCols)
#pragma unroll
      for (int v = 0; v < V; ++v) tot[1][wave][cv * V + v] = p[v];
    __syncthreads();
    Pair own = {1.f, 0.f};
    if (tid < G::kWidth) {
      own = tot[1][G::kWaves - 1][tid];
#pragma unroll
      for (int i = G::kWaves - 2; i >= 0; --i) own = compose(own, tot[1][i][tid]);
    }
    float r = r_keep;
    if constexpr (CHAIN) {
      if (step == 0) own = {0.f, own.a * r + own.s};
      const Pair b = chain_before<NT, G::kWidth>(chain, step, a.ntiles - 1, base, own);
      if (step > 0) r = b.s;
      r_keep = step == 0 ? own.s : own.a * r + own.s;
    } else {
      r_keep = own.a * r + own.s;
    }
    if (keeper) {
      start[0][tid] = h_keep;
      start[1][tid] = r;
      if (a.dh0 && tile == 0) a.dh0[mine] = r_keep;
    }
    __syncthreads();
    float at[V], dh[L][V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      at[v] = start[1][cv * V + v];
      for (int i = G::kWaves - 1; i > wave; --i) at[v] = tot[1][i][cv * V + v].a * at[v] + tot[1][i][cv * V + v].s;
      at[v] = rb[v].a * at[v] + rb[v].s;
    }
#pragma unroll
    for (int j = L - 1; j >= 0; --j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f, rest, e = element<T, V>(yr[j], v);
        decode(j, v, f, rest);
        if (!full && n0 + j >= me.len) e = 0.f;
        dh[j][v] = e + at[v];
        at[v] = f * dh[j][v];
        keep(c[j][v]);
      }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      at[v] = start[0][cv * V + v];
      for (int i = 0; i < wave; ++i) at[v] = tot[0][i][cv * V + v].a * at[v] + tot[0][i][cv * V + v].s;
      at[v] = hb[v].a * at[v] + hb[v].s;
    }
#pragma unroll
    for (int j = 0; j < L; ++j) {
      float gx[V], gg[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f, rest;
        decode(j, v, f, rest);
        const float u = element<T, V>(xr[j], v);
        gx[v] = COUPLED ? dh[j][v] * rest : dh[j][v];
        gg[v] = dh[j][v] * (COUPLED ? at[v] - u : at[v]);
        gg[v] *= LOG ? (element<T, V>(gr[j], v) > 0.f ? 0.f : f) : f * rest;
        at[v] = f * at[v] + (COUPLED ? rest * u : u);
        if (!full && n0 + j >= me.len) gx[v] = gg[v] = 0.f;
      }
      if (n0 + j < stored) {
        put<T, V>(dx + (int64_t)(n0 + j) * a.xs.n, gx);
        put<T, V>(dg + (int64_t)(n0 + j) * a.gs.n, gg);
      }
    }
    if (CHAIN || tile == 0) break;
  }
}

template <typename T, bool LOG, bool COUPLED>
__global__ __launch_bounds__(256) void scan_step_kernel(StepArgs a) {
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
hipError_t choose(int dtype, bool log_gate, bool coupled, F f) {
  auto flags = [&](auto t) {
    if (log_gate) return coupled ? f(t, std::true_type(), std::true_type()) : f(t, std::true_type(), std::false_type());
    return coupled ? f(t, std::false_type(), std::true_type()) : f(t, std::false_type(), std::false_type());
  };
  return dtype == 1 ? flags(uint16_t()) : flags(float());
}

// Few columns: a tile a workgroup.
bool chained(const ScanArgs& a) {
  return a.ntiles > 1 && a.columns < 65536 && a.columns * a.ntiles <= INT32_MAX;
}

// Zeroes the counter and unsets the words of a chain in the workspace.
hipError_t start_chain(const ScanArgs& a, void* ws, Chain* c, hipStream_t s) {
  c->words = (uint64_t*)ws;
  c->columns = a.columns;
  const long long n = chain_layout(a.ntiles, a.columns, c->level);
  scan_fill_kernel<<<dim3((unsigned)((n + kFillThreads - 1) / kFillThreads)), dim3(kFillThreads), 0, s>>>(c->words, n);
  return hipGetLastError();
}

template <bool BACKWARD, typename T, int V, int NT, int L, bool LOG, bool COUPLED>
hipError_t launch(const ScanArgs& a, void* ws, hipStream_t s) {
  const int groups = (int)((a.columns + Tile<NT, L, V>::kWidth - 1) / Tile<NT, L, V>::kWidth);
  Chain c = {};
  if (chained(a)) {
    const hipError_t e = start_chain(a, ws, &c, s);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((long long)groups * a.ntiles));
    if constexpr (BACKWARD)
      scan_backward_kernel<T, V, NT, L, LOG, COUPLED, true><<<grid, dim3(NT), 0, s>>>(a, c, groups);
    else
      scan_forward_kernel<T, V, NT, L, LOG, COUPLED, true><<<grid, dim3(NT), 0, s>>>(a, c, groups);
  } else {
    const dim3 grid((unsigned)groups);
    if constexpr (BACKWARD)
      scan_backward_kernel<T, V, NT, L, LOG, COUPLED, false><<<grid, dim3(NT), 0, s>>>(a, c, groups);
    else
      scan_forward_kernel<T, V, NT, L, LOG, COUPLED, false><<<grid, dim3(NT), 0, s>>>(a, c, groups);
  }
  return hipGetLastError();
}

template <bool BACKWARD>
hipError_t launch_scan(const ScanArgs& a, void* ws, hipStream_t s) {
  return choose(a.dtype, a.log_gate, a.coupled, [&](auto t, auto lg, auto cp) {
    using T = decltype(t);
    constexpr bool LOG = decltype(lg)::value, COUPLED = decltype(cp)::value;
    if (a.vec) return launch<BACKWARD, T, 16 / sizeof(T), 512, 4, LOG, COUPLED>(a, ws, s);
    return launch<BACKWARD, T, 1, 512, 16, LOG, COUPLED>(a, ws, s);
  });
}

}  // namespace

size_t scan_workspace(const ScanArgs& a) {
  if (!chained(a)) return 0;
  long long level[3];
  return (size_t)chain_layout(a.ntiles, a.columns, level) * sizeof(uint64_t);
}

hipError_t launch_scan_forward(const ScanArgs& a, void* ws, hipStream_t s) { return launch_scan<false>(a, ws, s); }

hipError_t launch_scan_backward(const ScanArgs& a, void* ws, hipStream_t s) { return launch_scan<true>(a, ws, s); }

hipError_t launch_scan_step(const StepArgs& a, hipStream_t s) {
  const long long n = (long long)a.B * a.H * a.d;
  return choose(a.dtype, a.log_gate, a.coupled, [&](auto t, auto lg, auto cp) {
    scan_step_kernel<decltype(t), decltype(lg)::value, decltype(cp)::value>
        <<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
  });
}

}  // namespace lapmix
