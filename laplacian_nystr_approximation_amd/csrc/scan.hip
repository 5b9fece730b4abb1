// Gated linear recurrence (include/lapmix.h): h_t = f_t h_{t-1} + i_t x_t.
//
// Any run of tokens maps the state before it to the state behind it by
// h -> A h + S (A the product of its gates, S its result from a zero state),
// and two runs compose to (A2 A1, A2 S1 + S2).  A workgroup takes a tile of
// kTile tokens by a few dozen columns (batch, head, channel): each lane holds a
// few consecutive tokens of V neighbouring channels, walks them once for its
// (A, S), the lanes' pairs are composed over the wave by lane exchange and over
// the workgroup through LDS, and with the state before the tile known each lane
// walks its tokens a second time, in registers, and writes y.  x and g are read
// once and y is written once: the kernel is bound by HBM.
//
// The state before a tile comes from one of two places.
//  - Loop form: a workgroup takes all tiles of its columns one after the other;
//    while it works on one, the loads of the next are under way.
//  - Chain form, for few columns: several workgroups share the tiles of a group of
//    columns and take them as they come.  A tile publishes its (A, S), every kFan-th
//    tile also the pair of the last kFan tiles, every kFan^2-th that of the last
//    kFan^2, and so on, so that a tile composes at most kFan - 1 pairs of each level.
//    Which pairs are composed, and in which order, depends on the tile's place
//    alone: results repeat bit for bit.
//
// Waits end: workgroups draw a group's tiles from the group's counter, in order, and
// finish one before they draw the next, so the lowest unfinished tile is being
// worked on and waits only for tiles below it, which are finished.
//
// Measured (MI355X, a large copy runs at 5.2 TB/s; forward and backward, the backward
// with dx and dg): 131072 columns of 1024 tokens in bf16, loop form, 164 us (4.9 TB/s)
// and 272 us (4.9); 65536 columns in float32 167 (4.8) and 270 (5.0); 4096 columns of
// 32768 tokens in bf16, chain form, 190 to 200 us (4.0 to 4.2) and 311 to 327 us (4.1
// to 4.3); 512 columns of 65536 tokens 52 and 94 us.
//
// A tile of the chain form takes 9.7 us of a forward workgroup's time: 3.1 until its
// loads are there, 1.4 for gates and pairs, 3.1 for publishing, waiting and composing
// (two trips to memory and back), 1.4 for y.  Three workgroups a CU (two in the
// backward) do not hide all of that, and one more does not fit the registers: where it
// was made to, it spilled (219 us and more forward, 376 and more backward).  What else
// was tried on the 4096 columns in bf16: one counter for all groups, 248 us forward (a
// draw at one address takes about 15 ns, whoever draws); drawing the next tile before
// this one's wait, with its loads under way during the wait, 250 (others then wait for
// a tile that is drawn but not begun); drawing it between the wait and y, 188 forward
// and 308 backward, but 305 instead of 285 where gates are logarithmic; tiles of 256
// tokens, 191; 512 lanes with 8 channels by 4 tokens each, 220 and 488; u, or h before each
// token, kept in LDS, 195 to 224 forward.
//
// The backward pass runs the tiles from the last to the first with r = f dh in
// the place of h (r_t = f_t (dy_t + r_{t+1})), and recomputes the tile's h from
// the state that the forward kept before it.
#include <type_traits>

#include "lapmix_internal.hpp"

namespace lapmix {

namespace {

// Pairs of a level that make one of the next.  (4096 columns of 32768 bf16 tokens, forward
// and backward: 8 pairs 204 and 318 us, 16 201 and 311, 32 201 and 311 to 319; 512 columns
// of 65536: 51.6 and 94.7, 52.8 and 94.1, 53.7 and 93.9.)
constexpr int kFan = 16;
constexpr int kLevels = 6;  // the highest level's pairs stand for kFan^5 tiles (2^27 tokens)
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct Pair {
  float a, s;
};

__device__ __forceinline__ Pair compose(Pair first, Pair then) { return {then.a * first.a, then.a * first.s + then.s}; }

// A published pair.  The workspace is filled with kUnset before the launch; a
// published A is never that pattern (a NaN is stored as the canonical one), so
// the 64-bit word tells by itself whether it is there, and no fence is needed.
constexpr uint64_t kUnset = ~(uint64_t)0;

// Words of a counter: each has 256 bytes of its own.
constexpr int kCounter = 32;

// A lane writes kFillEach pairs of words.
constexpr int kFillEach = 4;

__global__ __launch_bounds__(kThreads) void scan_fill_kernel(uint64_t* words, long long counters, long long n) {
  const long long first = (long long)blockIdx.x * (kThreads * kFillEach) + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kFillEach; ++k) {
    const long long i = 2 * (first + k * kThreads);
    const uint32_t v = i < counters ? 0 : (uint32_t)kUnset;
    if (i < n) *(u32x4*)(words + i) = (u32x4){v, v, v, v};
  }
}

__device__ __forceinline__ void publish(uint64_t* at, Pair p) {
  if (p.a != p.a) p.a = __builtin_nanf("");
  const uint64_t w = ((uint64_t)__float_as_uint(p.s) << 32) | __float_as_uint(p.a);
  __hip_atomic_store(at, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ uint64_t peek(const uint64_t* at) {
  return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Waits until a pair that was seen as `w` is there.  The bound on the polls only
// matters if a workspace is written from outside while the kernel runs: the
// results are then NaN.
__device__ __forceinline__ Pair wait_for(const uint64_t* at, uint64_t w) {
  for (int tries = 0; (uint32_t)w == (uint32_t)kUnset && tries < (1 << 18); ++tries) {
    __builtin_amdgcn_s_sleep(1);
    w = peek(at);
  }
  return {__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}

// The words of a launch's chain: the groups' counters, then for each level [places][columns].
struct Chain {
  uint64_t* words;
  long long columns;
  long long level[kLevels];  // first word of each level
};

long long chain_layout(int ntiles, long long columns, long long groups, long long level[kLevels]) {
  long long at = groups * kCounter, n = ntiles;
  for (int i = 0; i < kLevels; ++i) {
    level[i] = at;
    at += n * columns;
    n /= kFan;
  }
  return (at + 1) & ~1ll;  // filled two at a time
}

// The pair of everything before place p in the WIDTH columns from `base` on, for the
// lanes tid < WIDTH, which hand in their columns' own pairs.  All of a workgroup's
// lanes take part: each waits for a few of a column's pairs (SLOTS lanes a column).
template <int WIDTH>
__device__ __forceinline__ Pair chain_before(const Chain& c, int p, int last, uint32_t base, Pair own) {
  constexpr int SLOTS = kThreads / WIDTH, EACH = kFan / SLOTS, FIRST = 2;
  __shared__ Pair parts[kLevels][SLOTS][WIDTH];
  const int slot = threadIdx.x / WIDTH, lane = threadIdx.x % WIDTH;
  const bool on = base + lane < (uint64_t)c.columns;
  uint64_t* const words = c.words + (on ? base + lane : 0);
  auto at = [&](int level, int place) { return words + c.level[level] + place * c.columns; };
  const bool publishes = slot == 0 && on && p < last;
  if (publishes) publish(at(0, p), own);
  // The first levels' pairs are asked for together.
  uint64_t seen[FIRST][EACH];
  int q = p;
#pragma unroll
  for (int l = 0; l < FIRST; ++l, q /= kFan)
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int k = slot * EACH + i;
      seen[l][i] = on && k < q % kFan ? peek(at(l, q - q % kFan + k)) : 0;
    }
  bool full = true;  // the levels so far end with this place
  int levels = 0;
  q = p;
#pragma unroll
  for (int l = 0; l < kLevels; ++l, q /= kFan) {
    if (q == 0) break;
    const bool top = l == kLevels - 1;
    const int n = top ? q : q % kFan, first = q - n;
    Pair sum = {1.f, 0.f};
    if (l < FIRST) {
#pragma unroll
      for (int i = 0; i < EACH; ++i) {
        const int k = slot * EACH + i;
        if (on && k < n) sum = compose(sum, wait_for(at(l, first + k), seen[l][i]));
      }
    } else {
      const int each = (n + SLOTS - 1) / SLOTS;
      for (int k = slot * each; on && k < min(n, slot * each + each); ++k)
        sum = compose(sum, wait_for(at(l, first + k), peek(at(l, first + k))));
    }
    parts[l][slot][lane] = sum;
    levels = l + 1;
    // The next level's pair goes out before that level is waited for.
    full = full && !top && n == kFan - 1;
    if (full) {
      __syncthreads();
      if (slot == 0) {
        Pair all = {1.f, 0.f};
        for (int i = 0; i < SLOTS; ++i) all = compose(all, parts[l][i][lane]);
        own = compose(all, own);
        if (publishes) publish(at(l + 1, q / kFan), own);
      }
    }
  }
  __syncthreads();
  Pair before = {1.f, 0.f};
  if (slot == 0)
    for (int l = levels - 1; l >= 0; --l)
      for (int i = 0; i < SLOTS; ++i) before = compose(before, parts[l][i][lane]);
  return before;
}

// Forget gate f and 1 - f.  A gate close to 1 is passed on over many tokens, so it is
// formed as 1 minus its complement: then its only error is the last rounding, which
// has no drift, and the complement keeps its own relative accuracy.
template <bool LOG>
__device__ __forceinline__ void gate(float g, float& f, float& rest) {
  if constexpr (LOG) {
    g = g > 0.f ? 0.f : g;  // keeps NaN
    const float e = __expf(g);
    // exp(g) - 1 for g > -1/4 by its Taylor series: the first term left out is below
    // 2^-24 of the sum.
    float p = 1.f / 5040;
    p = fmaf(p, g, 1.f / 720);
    p = fmaf(p, g, 1.f / 120);
    p = fmaf(p, g, 1.f / 24);
    p = fmaf(p, g, 1.f / 6);
    p = fmaf(p, g, 0.5f);
    p = fmaf(p * g, g, g);
    const bool near = g > -0.25f;
    f = near ? 1.f + p : e;
    rest = near ? -p : 1.f - e;
  } else {
    const float e = __expf(-fabsf(g));
    const float small = e * __builtin_amdgcn_rcpf(1.f + e), big = 1.f - small;
    f = g < 0.f ? small : big;
    rest = g < 0.f ? big : small;
  }
}

// V neighbouring channels of a token, as loaded.
template <typename T, int V>
struct Raw;
template <typename T>
struct Raw<T, 1> {
  T e;
  __device__ __forceinline__ float operator[](int) const { return widen(e); }
};
template <>
struct Raw<float, 4> {
  f32x4 e;
  __device__ __forceinline__ float operator[](int v) const { return e[v]; }
};
template <>
struct Raw<uint16_t, 4> {
  u32x2 e;
  __device__ __forceinline__ float operator[](int v) const {
    return __uint_as_float(v % 2 ? e[v / 2] & 0xffff0000u : e[v / 2] << 16);
  }
};

// Keeps raw values in their registers: what is derived from them before is derived
// again behind, and takes no registers in between.
template <typename T, int V, int L>
__device__ __forceinline__ void keep(Raw<T, V> (&r)[L]) {
#pragma unroll
  for (int j = 0; j < L; ++j) asm volatile("" : "+v"(r[j].e));
}

template <int V, typename T>
__device__ __forceinline__ void put(T* at, const float* v) {
  if constexpr (V == 1) {
    narrow(v[0], at);
  } else if constexpr (sizeof(T) == 4) {
    *(f32x4*)at = (f32x4){v[0], v[1], v[2], v[3]};
  } else {
    u32x2 out;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      out[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){v[2 * i], v[2 * i + 1]}, lapnys::bf16x2));
    *(u32x2*)at = out;
  }
}

// A lane's share of a tile: L tokens of V channels; COLS lanes side by side span
// 128 bytes of a token (64 bytes or more in the form for unaligned tensors).
template <typename T, bool VEC>
struct Geometry {
  static constexpr int V = VEC ? 4 : 1;
  static constexpr int COLS = VEC ? 32 / sizeof(T) : 32;
  static constexpr int L = kTile * COLS / kThreads;
  static constexpr int WIDTH = COLS * V;  // columns of a workgroup
  static_assert(WIDTH >= 32 && WIDTH <= 64 && 64 % COLS == 0, "one wave looks after the columns' states");
};

// Composes the lanes' pairs over the wave's rows in the order of rising tokens (or
// falling ones).  p becomes the pair up to and with the lane's row, `before` that
// of the rows before it.
template <int COLS, int V, bool REVERSE>
__device__ __forceinline__ void wave_scan(Pair (&p)[V], Pair (&before)[V]) {
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
  bool on;          // its columns exist
  int len;          // tokens of the sequence
  int64_t x, g, y;  // offsets of token 0
  int64_t state;    // offset of the first kept state
};

__device__ __forceinline__ Lane lane_of(const ScanArgs& a, uint32_t col) {
  Lane l;
  l.on = col < (uint32_t)a.columns;
  if (!l.on) col = 0;
  const uint32_t bh = col / (uint32_t)a.d, c = col - bh * (uint32_t)a.d;
  const uint32_t b = bh / (uint32_t)a.H, h = bh - b * (uint32_t)a.H;
  l.len = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
  l.x = (int64_t)b * a.xs.b + (int64_t)h * a.xs.h + c;
  l.g = (int64_t)b * a.gs.b + (int64_t)h * a.gs.h + c;
  l.y = (int64_t)b * a.ys.b + (int64_t)h * a.ys.h + c;
  l.state = (int64_t)bh * a.ntiles * a.d + c;
  return l;
}

// L tokens' channels, `stride` elements apart.
template <typename T, int V, int L>
__device__ __forceinline__ void fetch(Raw<T, V> (&r)[L], const T* p, int64_t stride) {
#pragma unroll
  for (int j = 0; j < L; ++j, p += stride) r[j] = *(const Raw<T, V>*)p;
}

// The same from the tokens n0 .. n0 + L - 1 of a sequence that may end before: tokens
// behind its end read its last one (an empty one's first) and are masked by the caller.
template <typename T, int V, int L>
__device__ __forceinline__ void fetch_to(Raw<T, V> (&r)[L], const T* p, int64_t stride, int n0, int len) {
#pragma unroll
  for (int j = 0; j < L; ++j) r[j] = *(const Raw<T, V>*)(p + (int64_t)(max(min(n0 + j, len - 1), 0) - n0) * stride);
}

// Calls f with whether every token of a wave's lanes exists, as a compile-time value.
template <typename F>
__device__ __forceinline__ void when(bool full, F f) {
  if (full)
    f(std::true_type());
  else
    f(std::false_type());
}

// Where the waves enter a tile: the state before the first (or REVERSE: behind the
// last) wave's tokens and the waves' pairs give those of the others.  Returns the
// state that the tile passes on.
template <int WIDTH, bool REVERSE>
__device__ __forceinline__ float enter_waves(float (*start)[WIDTH], const Pair (*totals)[WIDTH], float h) {
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const int w = REVERSE ? kWaves - 1 - i : i;
    start[w][threadIdx.x] = h;
    h = totals[w][threadIdx.x].a * h + totals[w][threadIdx.x].s;
  }
  return h;
}

template <typename T, bool VEC, bool LOG, bool COUPLED, bool CHAIN>
__global__ __launch_bounds__(kThreads, CHAIN ? 3 : 2) void scan_forward_kernel(ScanArgs a, Chain chain, int groups) {
  using G = Geometry<T, VEC>;
  constexpr int V = G::V, L = G::L, WIDTH = G::WIDTH;
  __shared__ Pair totals[2][kWaves][WIDTH];
  __shared__ float start[kWaves][WIDTH];
  __shared__ int places[2];
  const int tid = threadIdx.x, wave = tid / 64, cv = tid % G::COLS * V, row = tid / G::COLS;
  const int last = a.ntiles - 1;
  const uint32_t group = blockIdx.x % groups, mine = group * WIDTH + tid;
  auto draw = [&] { return (int)atomicAdd((unsigned*)(chain.words + group * kCounter), 1u); };
  int tile = 0;
  if constexpr (CHAIN) {
    if (tid == 0) places[1] = draw();
    __syncthreads();
    tile = __builtin_amdgcn_readfirstlane(places[1]);
    if (tile > last) return;
  }
  const Lane me = lane_of(a, group * WIDTH + cv);
  const T* const x = (const T*)a.x + me.x + (int64_t)(row * L) * a.xs.n;
  const T* const g = (const T*)a.g + me.g + (int64_t)(row * L) * a.gs.n;
  T* const y = (T*)a.y + me.y + (int64_t)(row * L) * a.ys.n;
  Raw<T, V> xr[L], gr[L];
  auto is_full = [&](int t) { return __all(me.on && t * kTile + kTile <= me.len); };
  auto load = [&](int t) {
    const int64_t first = t * kTile;
    if (is_full(t)) {
      fetch(gr, g + first * a.gs.n, a.gs.n);
      fetch(xr, x + first * a.xs.n, a.xs.n);
    } else {
      fetch_to(gr, g + first * a.gs.n, a.gs.n, t * kTile + row * L, me.len);
      fetch_to(xr, x + first * a.xs.n, a.xs.n, t * kTile + row * L, me.len);
    }
  };
  load(tile);
  // Lanes of the first wave also look after one column each: its carried state.
  const bool keeper = tid < WIDTH && mine < (uint32_t)a.columns;
  float carried = tile == 0 && keeper && a.h0 ? a.h0[mine] : 0.f;

  for (int turn = 0;; turn ^= 1) {
    const int n0 = tile * kTile + row * L;
    const bool full = is_full(tile);
    keep(gr);
    keep(xr);
    float f[L][V], u[L][V];
    Pair p[V], before[V];
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = {1.f, 0.f};
    when(full, [&](auto all) {
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float rest;
          gate<LOG>(gr[j][v], f[j][v], rest);
          u[j][v] = COUPLED ? rest * xr[j][v] : xr[j][v];
          if (!all && n0 + j >= me.len) f[j][v] = 1.f, u[j][v] = 0.f;
          p[v] = compose(p[v], {f[j][v], u[j][v]});
        }
    });
    wave_scan<G::COLS, V, false>(p, before);
    auto& tot = totals[turn];
    if ((tid & 63) >= 64 - G::COLS)
#pragma unroll
      for (int v = 0; v < V; ++v) tot[wave][cv + v] = p[v];
    __syncthreads();
    if (!CHAIN && tile < last) load(tile + 1);
    if constexpr (CHAIN) {
      Pair own = {1.f, 0.f};
      if (keeper)
#pragma unroll
        for (int i = 0; i < kWaves; ++i) own = compose(own, tot[i][tid]);
      // The first tile's pair holds the initial state, which no other tile reads.
      if (tile == 0) own = {0.f, own.a * carried + own.s};
      const Pair b = chain_before<WIDTH>(chain, tile, last, group * WIDTH, own);
      if (tile > 0) carried = b.s;
    }
    if (keeper) {
      carried = enter_waves<WIDTH, false>(start, tot, carried);
      if (a.hN && tile == last) a.hN[mine] = carried;
    }
    __syncthreads();
    // Drawn only now that this tile waits for nothing any more.
    int drawn = 0;
    if (CHAIN && tid == 0) drawn = draw();
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = before[v].a * start[wave][cv + v] + before[v].s;
    if (a.states && row == 0 && me.on)
#pragma unroll
      for (int v = 0; v < V; ++v) a.states[me.state + (int64_t)tile * a.d + v] = h[v];
    when(full, [&](auto all) {
      T* at = y + (int64_t)(tile * kTile) * a.ys.n;
#pragma unroll
      for (int j = 0; j < L; ++j, at += a.ys.n) {
        float out[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          h[v] = f[j][v] * h[v] + u[j][v];
          out[v] = !all && n0 + j >= me.len ? 0.f : h[v];
        }
        if (all || (me.on && n0 + j < a.N)) put<V>(at, out);
      }
    });
    ++tile;
    if constexpr (CHAIN) {
      if (tid == 0) places[turn] = drawn;
      __syncthreads();
      tile = __builtin_amdgcn_readfirstlane(places[turn]);
    }
    if (tile > last) break;
    if (CHAIN) load(tile);
  }
}

template <typename T, bool VEC, bool LOG, bool COUPLED, bool CHAIN>
__global__ __launch_bounds__(kThreads, 2) void scan_backward_kernel(ScanArgs a, Chain chain, int groups) {
  using G = Geometry<T, VEC>;
  constexpr int V = G::V, L = G::L, WIDTH = G::WIDTH;
  __shared__ Pair totals[2][2][kWaves][WIDTH];   // of h and of r
  __shared__ float start[2][2][kWaves][WIDTH];
  __shared__ int places[2];
  const int tid = threadIdx.x, wave = tid / 64, cv = tid % G::COLS * V, row = tid / G::COLS;
  const int last = a.ntiles - 1;
  const uint32_t group = blockIdx.x % groups, mine = group * WIDTH + tid;
  auto draw = [&] { return (int)atomicAdd((unsigned*)(chain.words + group * kCounter), 1u); };
  int step = 0;  // tiles from the last one
  if constexpr (CHAIN) {
    if (tid == 0) places[1] = draw();
    __syncthreads();
    step = __builtin_amdgcn_readfirstlane(places[1]);
    if (step > last) return;
  }
  const Lane me = lane_of(a, group * WIDTH + cv);
  const int64_t rx = (int64_t)(row * L) * a.xs.n, rg = (int64_t)(row * L) * a.gs.n, ry = (int64_t)(row * L) * a.ys.n;
  const T* const x = (const T*)a.x + me.x + rx;
  const T* const g = (const T*)a.g + me.g + rg;
  const T* const dy = (const T*)a.dy + me.y + ry;
  T* const dx = (T*)a.dx + me.x + rx;
  T* const dg = (T*)a.dg + me.g + rg;
  Raw<T, V> xn[L], gr[L], yn[L];
  auto is_full = [&](int t) { return __all(me.on && t * kTile + kTile <= me.len); };
  auto load = [&](int t) {
    const int64_t first = t * kTile;
    if (is_full(t)) {
      fetch(gr, g + first * a.gs.n, a.gs.n);
      fetch(xn, x + first * a.xs.n, a.xs.n);
      fetch(yn, dy + first * a.ys.n, a.ys.n);
    } else {
      fetch_to(gr, g + first * a.gs.n, a.gs.n, t * kTile + row * L, me.len);
      fetch_to(xn, x + first * a.xs.n, a.xs.n, t * kTile + row * L, me.len);
      fetch_to(yn, dy + first * a.ys.n, a.ys.n, t * kTile + row * L, me.len);
    }
  };
  load(last - step);
  const bool keeper = tid < WIDTH && mine < (uint32_t)a.columns;
  const float* const kept = a.states + (keeper ? lane_of(a, mine).state : 0);
  float carried = step == 0 && keeper && a.dhN ? a.dhN[mine] : 0.f;

  for (int turn = 0;; turn ^= 1) {
    const int tile = last - step, n0 = tile * kTile + row * L;
    const float h_start = keeper ? kept[(int64_t)tile * a.d] : 0.f;
    const bool full = is_full(tile);
    keep(gr);
    keep(xn);
    keep(yn);
    // Behind the sequence's end gates are 1 and x and dy are 0.
    Raw<T, V> xr[L], yr[L];
    // A logarithmic gate that was cut off at 0, whose slope is 0, has its sign bit set.
    float f[L][V], rest[L][V];
    auto gate_at = [&](int j, int v) { return LOG ? fabsf(f[j][v]) : f[j][v]; };
    Pair p[V], q[V], hb[V], rb[V];
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = {1.f, 0.f};
    when(full, [&](auto all) {
#pragma unroll
      for (int j = 0; j < L; ++j) {
        xr[j] = xn[j];
        yr[j] = yn[j];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          gate<LOG>(gr[j][v], f[j][v], rest[j][v]);
          float u = COUPLED ? rest[j][v] * xr[j][v] : xr[j][v];
          if (LOG && gr[j][v] > 0.f) f[j][v] = -f[j][v];
          if (!all && n0 + j >= me.len) f[j][v] = 1.f, u = 0.f;
          p[v] = compose(p[v], {gate_at(j, v), u});
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) q[v] = {p[v].a, 0.f};
#pragma unroll
      for (int j = L - 1; j >= 0; --j)
#pragma unroll
        for (int v = 0; v < V; ++v)
          q[v].s = gate_at(j, v) * (q[v].s + (!all && n0 + j >= me.len ? 0.f : yr[j][v]));
    });
    keep(xr);
    keep(yr);
    auto& tot = totals[turn];
    wave_scan<G::COLS, V, false>(p, hb);
    if ((tid & 63) >= 64 - G::COLS)
#pragma unroll
      for (int v = 0; v < V; ++v) tot[0][wave][cv + v] = p[v];
    wave_scan<G::COLS, V, true>(q, rb);
    if ((tid & 63) < G::COLS)
#pragma unroll
      for (int v = 0; v < V; ++v) tot[1][wave][cv + v] = q[v];
    __syncthreads();
    if (!CHAIN && tile > 0) load(tile - 1);
    if (keeper) enter_waves<WIDTH, false>(start[turn][0], tot[0], h_start);
    if constexpr (CHAIN) {
      Pair own = {1.f, 0.f};
      if (keeper)
#pragma unroll
        for (int i = kWaves - 1; i >= 0; --i) own = compose(own, tot[1][i][tid]);
      if (step == 0) own = {0.f, own.a * carried + own.s};
      const Pair b = chain_before<WIDTH>(chain, step, last, group * WIDTH, own);
      if (step > 0) carried = b.s;
    }
    if (keeper) {
      carried = enter_waves<WIDTH, true>(start[turn][1], tot[1], carried);
      if (a.dh0 && tile == 0) a.dh0[mine] = carried;
    }
    __syncthreads();
    int drawn = 0;
    if (CHAIN && tid == 0) drawn = draw();
    float h[V], hp[L][V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = hb[v].a * start[turn][0][wave][cv + v] + hb[v].s;
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        hp[j][v] = h[v];
        h[v] = gate_at(j, v) * h[v] + (COUPLED ? rest[j][v] * xr[j][v] : xr[j][v]);
      }
    keep(xr);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = rb[v].a * start[turn][1][wave][cv + v] + rb[v].s;
    when(full, [&](auto all) {
      T* to_dx = dx + (int64_t)(tile * kTile + L - 1) * a.xs.n;
      T* to_dg = dg + (int64_t)(tile * kTile + L - 1) * a.gs.n;
#pragma unroll
      for (int j = L - 1; j >= 0; --j, to_dx -= a.xs.n, to_dg -= a.gs.n) {
        const bool dead = !all && n0 + j >= me.len;
        float gx[V], gg[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float dh = (dead ? 0.f : yr[j][v]) + h[v];
          h[v] = gate_at(j, v) * dh;
          gx[v] = COUPLED ? dh * rest[j][v] : dh;
          gg[v] = dh * (COUPLED ? hp[j][v] - xr[j][v] : hp[j][v]);
          gg[v] *= LOG ? (__float_as_uint(f[j][v]) >> 31 ? 0.f : f[j][v]) : f[j][v] * rest[j][v];
          if (dead) gx[v] = gg[v] = 0.f;
        }
        if (all || (me.on && n0 + j < a.N)) {
          put<V>(to_dx, gx);
          put<V>(to_dg, gg);
        }
      }
    });
    ++step;
    if constexpr (CHAIN) {
      if (tid == 0) places[turn] = drawn;
      __syncthreads();
      step = __builtin_amdgcn_readfirstlane(places[turn]);
    }
    if (step > last) break;
    if (CHAIN) load(last - step);
  }
}

// One token: a wave takes 64 times V columns of one sequence, so the slot is the
// same for all its lanes.  Bound by the launch, then by HBM (the states).
template <typename T, bool VEC, bool LOG, bool COUPLED>
__global__ __launch_bounds__(64) void scan_step_kernel(StepArgs a, int waves) {
  constexpr int V = VEC ? 4 : 1;
  const int b = blockIdx.x / waves, hd = a.H * a.d;
  const int hc = ((blockIdx.x - b * waves) * 64 + threadIdx.x) * V;
  const int slot = a.slots ? a.slots[b] : b;
  if (hc >= hd || slot < 0 || slot >= a.n_slots) return;
  const int h = hc / a.d, c = hc - h * a.d;
  const Raw<T, V> g = *(const Raw<T, V>*)((const T*)a.g + b * a.gs.b + h * a.gs.h + c);
  const Raw<T, V> x = *(const Raw<T, V>*)((const T*)a.x + b * a.xs.b + h * a.xs.h + c);
  const int64_t at = (int64_t)slot * hd + hc;
  const Raw<float, V> from = *(const Raw<float, V>*)(a.h_in + at);
  float to[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float f, rest;
    gate<LOG>(g[v], f, rest);
    to[v] = f * from[v] + (COUPLED ? rest * x[v] : x[v]);
  }
  put<V>(a.h_out + at, to);
  put<V>((T*)a.y + b * a.ys.b + h * a.ys.h + c, to);
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

// Chain form: from 5 tiles on, of fewer than 32768 columns.
//  - Columns (bf16, 134 M elements, forward / backward, chain against loop):
//    8192 columns 188 / 320 us against 371 / 558, 16384 174 / 283 against 208 / 314,
//    32768 180 / 285 against 169 / 274: there the loop form's 512 workgroups fill
//    the chip by themselves.
//  - Tiles (32 columns, float32, a call on its own, chain against loop): 4 tiles
//    13.8 / 15.2 us against 11.1 / 12.7, 5 tiles 13.4 / 14.9 against 11.4 / 15.4,
//    8 tiles 13.4 / 14.8 against 14.7 / 23.5: the chain costs a second launch.
bool chained(const ScanArgs& a) {
  return a.ntiles > 4 && a.columns < 32768 && a.columns * a.ntiles <= INT32_MAX / 2;
}

// Zeroes the counters and unsets the pairs of a chain in the workspace.
hipError_t start_chain(const ScanArgs& a, int groups, void* ws, Chain* c, hipStream_t s) {
  c->words = (uint64_t*)ws;
  c->columns = a.columns;
  const long long n = chain_layout(a.ntiles, a.columns, groups, c->level);
  const long long per = 2 * kThreads * kFillEach;
  scan_fill_kernel<<<dim3((unsigned)((n + per - 1) / per)), dim3(kThreads), 0, s>>>(
      c->words, (long long)groups * kCounter, n);
  return hipGetLastError();
}

// Workgroups of a chain launch: about what the chip's 256 CUs hold at once.
constexpr int kResident = 256 * 4;

int groups_of(const ScanArgs& a, int width) { return (int)((a.columns + width - 1) / width); }

template <bool BACKWARD, typename T, bool VEC, bool LOG, bool COUPLED>
hipError_t launch(const ScanArgs& a, void* ws, hipStream_t s) {
  constexpr int WIDTH = Geometry<T, VEC>::WIDTH;
  const int groups = groups_of(a, WIDTH);
  auto* const chain_form =
      BACKWARD ? scan_backward_kernel<T, VEC, LOG, COUPLED, true> : scan_forward_kernel<T, VEC, LOG, COUPLED, true>;
  auto* const loop_form =
      BACKWARD ? scan_backward_kernel<T, VEC, LOG, COUPLED, false> : scan_forward_kernel<T, VEC, LOG, COUPLED, false>;
  Chain c = {};
  if (!chained(a)) {
    loop_form<<<dim3(groups), dim3(kThreads), 0, s>>>(a, c, groups);
    return hipGetLastError();
  }
  const hipError_t e = start_chain(a, groups, ws, &c, s);
  if (e != hipSuccess) return e;
  const int share = (kResident + groups - 1) / groups;  // workgroups to a group
  chain_form<<<dim3((unsigned)(groups * (share < a.ntiles ? share : a.ntiles))), dim3(kThreads), 0, s>>>(a, c, groups);
  return hipGetLastError();
}

template <bool BACKWARD>
hipError_t launch_scan(const ScanArgs& a, void* ws, hipStream_t s) {
  return choose(a.dtype, a.log_gate, a.coupled, [&](auto t, auto lg, auto cp) {
    using T = decltype(t);
    constexpr bool LOG = decltype(lg)::value, COUPLED = decltype(cp)::value;
    return a.vec ? launch<BACKWARD, T, true, LOG, COUPLED>(a, ws, s) : launch<BACKWARD, T, false, LOG, COUPLED>(a, ws, s);
  });
}

}  // namespace

size_t scan_workspace(const ScanArgs& a) {
  if (!chained(a)) return 0;
  long long level[kLevels];
  // Groups are narrowest, and so most, at 32 columns.
  return (size_t)chain_layout(a.ntiles, a.columns, groups_of(a, 32), level) * sizeof(uint64_t);
}

hipError_t launch_scan_forward(const ScanArgs& a, void* ws, hipStream_t s) { return launch_scan<false>(a, ws, s); }

hipError_t launch_scan_backward(const ScanArgs& a, void* ws, hipStream_t s) { return launch_scan<true>(a, ws, s); }

hipError_t launch_scan_step(const StepArgs& a, hipStream_t s) {
  return choose(a.dtype, a.log_gate, a.coupled, [&](auto t, auto lg, auto cp) {
    using T = decltype(t);
    constexpr bool LOG = decltype(lg)::value, COUPLED = decltype(cp)::value;
    const int per = a.vec ? 256 : 64, waves = (a.H * a.d + per - 1) / per;
    const dim3 grid((unsigned)a.B * (unsigned)waves), block(64);
    if (a.vec)
      scan_step_kernel<T, true, LOG, COUPLED><<<grid, block, 0, s>>>(a, waves);
    else
      scan_step_kernel<T, false, LOG, COUPLED><<<grid, block, 0, s>>>(a, waves);
    return hipGetLastError();
  });
}

}  // namespace lapmix
