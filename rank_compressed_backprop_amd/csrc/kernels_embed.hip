// Rows of a table looked up by token and scaled, and the table's gradient (include/instant_ops.h):
//   y[m] = s W[t[m]]        gW[v] = s sum_{m: t[m] = v} gy[m]
//
// The gradient groups the places of equal tokens, in their order, and sums their rows in eights, the
// eights of a tile of 64 and the tiles of a run by its eighths, so it needs no float atomics and gives the same bits
// every time (the order is the tokens' alone, but not one row after the other):
//   split      segments of 1024 tokens, each ordered by class (token mod CLASSES, so that frequent
//              tokens, which often have low numbers, are spread)
//   group      a block a class collects its tokens from the segments and orders them by token; it
//              also knows which tokens of its class do not occur, and fills their rows with zeros
//   run_sum    tiles of the grouped places: runs of a token inside a tile are summed and written,
//              the ends of runs that cross its borders left as partial rows
//   run_join   sums the partial rows of a run, in order
#include <algorithm>

#include "ops.hpp"

namespace instant {

namespace {

constexpr int CLASS_BITS = 10, CLASSES = 1 << CLASS_BITS;
constexpr int WAVES = 4, HELD = 4;                       // of a block; runs of 64 tokens a wave
constexpr int SEG_BITS = 10, SEG = WAVES * HELD * WAVE;  // tokens of a segment
constexpr int MAX_ROWS = (1 << 18) / CLASSES, MAX_SEGS = EMBED_MAX_M / SEG;
static_assert(SEG == 1 << SEG_BITS && MAX_ROWS <= WAVES * WAVE, "a thread a row");
constexpr unsigned NO_TOKEN = 1u << 18;  // what takes no part

__device__ __forceinline__ int64_t token_at(const void* t, bool wide, size_t i) {
  return wide ? ((const int64_t*)t)[i] : (int64_t)((const int32_t*)t)[i];
}

template <class T> using vec8_t = typename MM<T>::vec8;

}  // namespace

// TPR threads a row, UNITS units of 8 columns a thread, 256 / TPR rows a block.
template <class T, int TPR, int UNITS>
__global__ __launch_bounds__(256) void embed_kernel(const void* __restrict__ tokens, bool wide, int M,
                                                    const T* __restrict__ w, int V, int C, float scale,
                                                    T* __restrict__ y) {
  constexpr int RPB = 256 / TPR;
  const int i = threadIdx.x % TPR;
  for (int m = blockIdx.x * RPB + (int)threadIdx.x / TPR; m < M; m += gridDim.x * RPB) {
    const int64_t t = token_at(tokens, wide, m);
    const bool in = t >= 0 && t < V;
    const T* row = w + (in ? (size_t)t * C : 0);
    T* out = y + (size_t)m * C;
    for (int n0 = 8 * i; n0 < C; n0 += 8 * TPR * UNITS) {
      vec8_t<T> v[UNITS];
#pragma unroll
      for (int k = 0; k < UNITS; ++k)
        v[k] = *reinterpret_cast<const vec8_t<T>*>(row + (n0 + 8 * TPR * k < C ? n0 + 8 * TPR * k : n0));
#pragma unroll
      for (int k = 0; k < UNITS; ++k) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = in ? (float)v[k][j] * scale : NAN;
        if (n0 + 8 * TPR * k < C) store_row<T, 8>(out + n0 + 8 * TPR * k, o);
      }
    }
  }
}

// The `used` tokens that take part and their places, grouped by token (in order of class, token,
// place).
struct Grouped {
  unsigned *token, *place;
  int* used;
};

namespace {

// Of the lanes in `in`, those whose value v of `bits` bits is this lane's (for lanes of `in`).
__device__ __forceinline__ uint64_t lanes_like(unsigned v, int bits, uint64_t in) {
  uint64_t m = in;
  for (int i = 0; i < bits; ++i) {
    const uint64_t one = __ballot(v >> i & 1);
    m &= v >> i & 1 ? one : ~one;
  }
  return m;
}

// What this lane has written to LDS is there for the wave's other lanes, and what it reads from here on
// is what they have written. (A wave's LDS operations run in order: no wait is needed, but neither the
// compiler nor the lanes' lock step promises the order without this.)
__device__ __forceinline__ void wave_settled() {
#ifdef __HIP_DEVICE_COMPILE__
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
#endif
}

// Adds the lanes of `in` (this one too if `is`) to counts[v]; returns this lane's number among
// those with its v, the wave's earlier ones first. Nothing is atomic: counts are the wave's own, and
// what one call's lanes have added is settled before the next call's (other) lanes read it.
__device__ __forceinline__ int number_in(int* counts, unsigned v, int bits, uint64_t in, bool is, int lane) {
  const uint64_t like = lanes_like(v, bits, in);
  const int before = __popcll(like & ((1ull << lane) - 1)), leader = __ffsll((unsigned long long)like) - 1;
  int base = 0;
  if (is && before == 0) {
    base = counts[v];
    counts[v] = base + __popcll(like);
  }
  wave_settled();
  return __shfl(base, leader < 0 ? 0 : leader) + before;
}

// The sum of v over the threads of a block of WAVES waves before this one; `all`: over all.
__device__ __forceinline__ int sum_before(int v, int* lds, int& all) {
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
  int upto = v;
#pragma unroll
  for (int d = 1; d < WAVE; d *= 2) {
    const int o = __shfl_up(upto, d);
    upto += lane >= d ? o : 0;
  }
  __syncthreads();  // the last sum's readers are done
  if (lane == WAVE - 1) lds[wave] = upto;
  __syncthreads();
  int before = upto - v;
  all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    before += w < wave ? lds[w] : 0;
    all += lds[w];
  }
  return before;
}

// The tokens at first, first + WAVE, ...: those that take part, and NO_TOKEN. (All are requested
// before one is looked at: behind the last the last again, so no branch is in the way.)
__device__ __forceinline__ void load_tokens(const void* tokens, bool wide, int M, int V, int64_t padding, int first,
                                            unsigned (&t)[HELD]) {
  int64_t v[HELD];
  if (wide) {
#pragma unroll
    for (int h = 0; h < HELD; ++h) v[h] = ((const int64_t*)tokens)[min(first + h * WAVE, M - 1)];
  } else {
#pragma unroll
    for (int h = 0; h < HELD; ++h) v[h] = ((const int32_t*)tokens)[min(first + h * WAVE, M - 1)];
  }
#pragma unroll
  for (int h = 0; h < HELD; ++h)
    t[h] = first + h * WAVE < M && v[h] >= 0 && v[h] < V && v[h] != padding ? (unsigned)v[h] : NO_TOKEN;
}

}  // namespace

// Segment blockIdx.x in order of class: list[SEG * segment + i] = row << SEG_BITS | place in the
// segment, starts[class * segments + segment] the class's first i (class CLASSES: the end).
__global__ __launch_bounds__(256) void split_kernel(const void* __restrict__ tokens, bool wide, int M, int V,
                                                    int64_t padding, unsigned* __restrict__ list,
                                                    int* __restrict__ starts) {
  __shared__ int counts[WAVES][CLASSES], sums[WAVES];
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE, seg = blockIdx.x, segs = gridDim.x;
  unsigned t[HELD];
  int number[HELD];
  load_tokens(tokens, wide, M, V, padding, seg * SEG + wave * HELD * WAVE + lane, t);
  for (int i = threadIdx.x; i < WAVES * CLASSES; i += 256) counts[0][i] = 0;
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HELD; ++h) {
    const bool is = t[h] != NO_TOKEN;
    number[h] = number_in(counts[wave], t[h] & (CLASSES - 1), CLASS_BITS, __ballot(is), is, lane);
  }
  __syncthreads();
  constexpr int PER = CLASSES / 256;
  int n[PER][WAVES], sum = 0, all;
#pragma unroll
  for (int k = 0; k < PER; ++k)
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      n[k][w] = counts[w][PER * threadIdx.x + k];
      sum += n[k][w];
    }
  int at = sum_before(sum, sums, all);
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    starts[(size_t)(PER * threadIdx.x + k) * segs + seg] = at;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      counts[w][PER * threadIdx.x + k] = at;
      at += n[k][w];
    }
  }
  if (threadIdx.x == 0) starts[(size_t)CLASSES * segs + seg] = all;
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HELD; ++h)
    if (t[h] != NO_TOKEN)
      list[(size_t)seg * SEG + counts[wave][t[h] & (CLASSES - 1)] + number[h]] =
          t[h] >> CLASS_BITS << SEG_BITS | (wave * HELD + h) * WAVE + lane;
}

// Class b = blockIdx.x of the tokens: out, from its tokens' first place in it on. rows: tokens of a
// class at most, 2^bits >= rows. DIRECT: from the tokens themselves, M <= SEG; else from the
// segments' lists. A round holds ROUND tokens of the class; with more than one, a first pass counts
// all of them. units: of 16 bytes in a row of `fill`, which the absent tokens' rows are cleared in
// (null: not).
// Every step is an integer's and in the order of the tokens, so the order is the same every time.
template <bool DIRECT>
__global__ __launch_bounds__(256) void group_kernel(const void* __restrict__ tokens, bool wide, int M, int V,
                                                    int64_t padding, const unsigned* __restrict__ list,
                                                    const int* __restrict__ starts, int segs, int rows, int bits,
                                                    Grouped out, uint4* __restrict__ fill, int units) {
  constexpr int RUNS = DIRECT ? HELD : 16, ROUND = WAVES * RUNS * WAVE;
  __shared__ int counts[WAVES][MAX_ROWS], sums[WAVES];
  // of the class's tokens: the first of a segment, and what to add to get its place in the list
  __shared__ int first[DIRECT ? 1 : MAX_SEGS], from[DIRECT ? 1 : MAX_SEGS];
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE, tid = threadIdx.x;
  const unsigned b = blockIdx.x;
  int n = M, below = 0;  // tokens of the class (DIRECT: of all), and of the classes before it
  if constexpr (!DIRECT) {
    n = 0;
    for (int s0 = 0; s0 < segs; s0 += 256) {
      int a = 0, e = 0, all;
      if (s0 + tid < segs) {
        a = starts[(size_t)b * segs + s0 + tid];
        e = starts[(size_t)(b + 1) * segs + s0 + tid];
      }
      below += a;
      const int before = sum_before(e - a, sums, all);
      if (s0 + tid < segs) {
        first[s0 + tid] = n + before;
        from[s0 + tid] = (s0 + tid) * SEG + a - (n + before);
      }
      n += all;
    }
    __syncthreads();
  }
  const int rounds = (n + ROUND - 1) / ROUND;
  unsigned row[RUNS], place[RUNS];  // row: NO_TOKEN where there is none
  int number[RUNS];
  auto none = [&](int h0) {
#pragma unroll
    for (int h = 0; h < RUNS; ++h)
      if (h >= h0) row[h] = NO_TOKEN;
  };
  // the first K runs from i0 on (steps of the searches and loads side by side)
  auto fetch = [&](auto K, int i0, int end) {
    int i[K], s[K];
#pragma unroll
    for (int h = 0; h < K; ++h) {
      i[h] = min(i0 + h * WAVE, n - 1);
      s[h] = 0;  // the last segment that begins up to i (one without tokens begins with the next)
    }
    for (int step = 1 << (31 - __clz(segs)); step > 0; step >>= 1)
#pragma unroll
      for (int h = 0; h < K; ++h)
        if (s[h] + step < segs && first[s[h] + step] <= i[h]) s[h] += step;
    unsigned e[K];
#pragma unroll
    for (int h = 0; h < K; ++h) e[h] = list[from[s[h]] + i[h]];
#pragma unroll
    for (int h = 0; h < K; ++h) {
      row[h] = i0 + h * WAVE < end ? e[h] >> SEG_BITS : NO_TOKEN;
      place[h] = (unsigned)s[h] * SEG + (e[h] & (SEG - 1));
    }
    none(K);
  };
  auto load = [&](int round) {
    if constexpr (DIRECT) {
      const int i0 = wave * RUNS * WAVE + lane;
      unsigned t[HELD];
      load_tokens(tokens, wide, M, V, padding, i0, t);
#pragma unroll
      for (int h = 0; h < HELD; ++h) {
        const unsigned c = t[h] & (CLASSES - 1);
        const bool is = t[h] != NO_TOKEN;
        below += is && c < b;
        row[h] = is && c == b ? t[h] >> CLASS_BITS : NO_TOKEN;
        place[h] = i0 + h * WAVE;
      }
    } else {
      const int begin = round * ROUND, left = min(n - begin, ROUND);
      const int runs = (left + WAVES * WAVE - 1) / (WAVES * WAVE);  // a wave, consecutive
      const int i0 = begin + wave * runs * WAVE + lane, end = min(begin + left, begin + (wave + 1) * runs * WAVE);
      if (runs == 1) fetch(std::integral_constant<int, 1>{}, i0, end);
      else if (runs <= 4) fetch(std::integral_constant<int, 4>{}, i0, end);
      else fetch(std::integral_constant<int, RUNS>{}, i0, end);
    }
  };
  auto clear = [&] {
    for (int i = tid; i < WAVES * MAX_ROWS; i += 256) counts[0][i] = 0;
    __syncthreads();
  };
  auto count = [&] {
#pragma unroll
    for (int h = 0; h < RUNS; ++h) {
      const bool is = row[h] != NO_TOKEN;
      const uint64_t in = __ballot(is);
      if (in) number[h] = number_in(counts[wave], row[h], bits, in, is, lane);
    }
  };
  clear();
  for (int r = 0; r < rounds; ++r) {
    load(r);
    count();
  }
  __syncthreads();
  // the tokens of row tid, and their first place
  int total = 0, next, all;
  if (tid < rows)
#pragma unroll
    for (int w = 0; w < WAVES; ++w) total += counts[w][tid];
  int before_class;
  sum_before(below, sums, before_class);
  next = before_class + sum_before(total, sums, all);
  if (b == gridDim.x - 1 && tid == 0) *out.used = before_class + all;  // (no class behind this)
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) {
      __syncthreads();
      clear();
      load(r);
      count();
      __syncthreads();
    }
    if (tid < rows)
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const int c = counts[w][tid];
        counts[w][tid] = next;
        next += c;
      }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < RUNS; ++h) {
      if (row[h] == NO_TOKEN) continue;
      const int at = counts[wave][row[h]] + number[h];
      out.token[at] = row[h] << CLASS_BITS | b;
      out.place[at] = place[h];
    }
  }
  if (!fill) return;
  // rows without a token, several at a time if they are short
  __syncthreads();
  if (tid < rows) counts[0][tid] = total;
  __syncthreads();
  int tpr = 16;
  while (tpr < units && tpr < 256) tpr *= 2;
  for (int r = tid / tpr; r < rows; r += 256 / tpr) {
    const size_t v = (size_t)r * CLASSES + b;
    if (v >= (size_t)V || counts[0][r]) continue;
    for (int k = tid % tpr; k < units; k += tpr) __builtin_nontemporal_store(zero4(), (f32x4*)fill + v * units + k);
  }
}

namespace {

// gw[n .. n+7] = scale * sum (+ what is there)
template <class T>
__device__ __forceinline__ void put(T* gw, bool add, float scale, float v[8]) {
  float o[8];
  if (add) load8(gw, o);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = add ? fmaf(v[j], scale, o[j]) : v[j] * scale;
  store_row<T, 8>(gw, v);
}

}  // namespace

// Tile blockIdx.x of TILE places, columns 512 blockIdx.y + 8 lane ..: each of 8 waves sums 8 places,
// all of whose rows are requested at once. What runs leave at the waves' borders goes through LDS,
// and what they leave at the tile's to memory: part[tile][0] the sum of a run that goes on from the
// tile before, part[tile][1] of one that begins here and goes on in the next. (A wave that went
// through 32 rows in batches of 8 took 57 us for 16384 x 4096 and 16 for 16384 x 768.)
constexpr int SUM_WAVES = 8, SUM_ROWS = 8, TILE = SUM_WAVES * SUM_ROWS;

template <class T>
__global__ __launch_bounds__(SUM_WAVES* WAVE) void run_sum_kernel(const T* __restrict__ gy, Grouped grouped, int C,
                                                                  float scale, bool add, T* __restrict__ gw,
                                                                  float* __restrict__ part) {
  // of each wave: its first run's sum if that began before, and its last run's if that begins here and goes on
  __shared__ __attribute__((aligned(32))) float ends[2][SUM_WAVES][8 * WAVE];
  const int M = *grouped.used, tile = blockIdx.x, i0 = tile * TILE;
  if (i0 >= M) return;
  const int count = min(TILE, M - i0), lane = threadIdx.x % WAVE, col = 8 * (WAVE * blockIdx.y + lane);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const bool in = col < C;
  unsigned token = 0, place = 0;
  if (lane < count) {
    token = grouped.token[i0 + lane];
    place = grouped.place[i0 + lane];
  }
  const unsigned none = ~0u;
  const unsigned prev = i0 ? grouped.token[i0 - 1] : none, behind = i0 + count < M ? grouped.token[i0 + count] : none;
  auto at = [&](int i) {
    return i < 0 ? prev : i >= count ? behind : (unsigned)__builtin_amdgcn_readlane(token, i);
  };
  const int s = wave * SUM_ROWS, e = min(s + SUM_ROWS, count);
  float acc[8];
  auto clear = [&] {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  };
  auto put_here = [&](unsigned t) {
    if (in) put(gw + (size_t)t * C + col, add, scale, acc);
  };
  clear();
  if (s < e) {
    vec8_t<T> v[SUM_ROWS];
    const T* from = gy + (in ? col : 0);
#pragma unroll
    for (int a = 0; a < SUM_ROWS; ++a)  // (behind the last row: the last again)
      v[a] = *reinterpret_cast<const vec8_t<T>*>(
          from + (size_t)(unsigned)__builtin_amdgcn_readlane(place, min(s + a, e - 1)) * C);
    bool began_before = at(s - 1) == at(s);
#pragma unroll
    for (int a = 0; a < SUM_ROWS; ++a) {
      const int i = s + a;
      if (i >= e) break;
      const unsigned t = at(i);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += (float)v[a][j];
      const bool goes_on = at(i + 1) == t;
      if (goes_on && i + 1 < e) continue;
      if (began_before || goes_on) store_row<float, 8>(&ends[began_before ? 0 : 1][wave][8 * lane], acc);
      else put_here(t);
      began_before = false;
      clear();
    }
  }
  __syncthreads();
  // the run of which this wave has the first part in this tile
  auto chain = [&](int which, unsigned t) {
    load8(&ends[which][wave][8 * lane], acc);
    int w = wave + 1;
    for (; w < SUM_WAVES && at(w * SUM_ROWS - 1) == t && at(w * SUM_ROWS) == t && w * SUM_ROWS < count; ++w) {
      float o[8];
      load8(&ends[0][w][8 * lane], o);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += o[j];
    }
    // it ends in this tile, unless every wave up to the end is its and the next tile begins with it
    const bool goes_on = at(min(w * SUM_ROWS, count) - 1) == t && min(w * SUM_ROWS, count) == count && behind == t;
    if (which == 1 && !goes_on) put_here(t);
    else if (in) store_row<float, 8>(part + ((size_t)2 * tile + which) * C + col, acc);
  };
  if (wave == 0 && prev == at(0)) chain(0, at(0));
  if (s < e) {
    const unsigned t = at(e - 1);
    int i = e - 1;
    while (i > s && at(i - 1) == t) --i;
    if (at(e) == t && !(i == s && at(s - 1) == t)) chain(1, t);
  }
}

// Tile blockIdx.x: if a run begins in it and goes on, its partial rows in order: each wave sums a
// part of them, and the waves' sums are added in order.
template <class T>
__global__ __launch_bounds__(SUM_WAVES* WAVE) void run_join_kernel(Grouped grouped, int C, float scale, bool add,
                                                                   const float* __restrict__ part,
                                                                   T* __restrict__ gw) {
  constexpr int AHEAD = 4;
  __shared__ __attribute__((aligned(32))) float sums[SUM_WAVES][8 * WAVE];
  const int M = *grouped.used, tile = blockIdx.x;
  const int64_t last = (int64_t)(tile + 1) * TILE - 1;
  if (last + 1 >= M) return;
  const unsigned t = grouped.token[last];
  if (grouped.token[last + 1] != t) return;
  if (tile > 0 && grouped.token[last - TILE] == t) return;  // it came from the tile before
  // tiles that go on with it: those that begin with it, looked up 64 at a time
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE, col = 8 * (WAVE * blockIdx.y + lane);
  int end = tile + 1;
  while (true) {
    const int64_t at = (int64_t)(end + lane) * TILE;
    const uint64_t other = __ballot(!(at < M && grouped.token[at] == t));
    if (other) {
      end += __ffsll((unsigned long long)other) - 1;
      break;
    }
    end += WAVE;
  }
  const bool in = col < C;
  const int64_t n = end - tile;  // partial rows
  const int u0 = tile + (int)(n * wave / SUM_WAVES), u1 = tile + (int)(n * (wave + 1) / SUM_WAVES);
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  for (int u = u0; u < u1; u += AHEAD) {
    float v[AHEAD][8];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int k = min(u + a, u1 - 1);
      load8(part + ((size_t)2 * k + (k == tile ? 1 : 0)) * C + (in ? col : 0), v[a]);
    }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += u + a < u1 ? v[a][j] : 0.0f;
  }
  store_row<float, 8>(&sums[wave][8 * lane], acc);
  __syncthreads();
  if (wave || !in) return;
  for (int w = 1; w < SUM_WAVES; ++w) {
    float o[8];
    load8(&sums[w][8 * lane], o);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += o[j];
  }
  put(gw + (size_t)t * C + col, add, scale, acc);
}

namespace {

// The workspace: offsets in bytes.
struct Layout {
  int segs;  // 0: the tokens are grouped directly
  size_t used, token, place, list, starts, part, end;
  Layout(int M, int C) {
    auto align256 = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t tiles = (M + TILE - 1) / TILE;
    segs = M <= SEG ? 0 : (M + SEG - 1) / SEG;
    used = 0;
    token = 256;
    place = token + align256((size_t)M * 4);
    list = place + align256((size_t)M * 4);
    starts = list + (size_t)segs * SEG * 4;
    part = starts + align256((size_t)segs * (CLASSES + 1) * 4);
    end = part + 2 * tiles * C * 4;
  }
};

template <class T>
hipError_t embed_bwd(const void* gy, const void* tokens, bool wide, int M, int V, int C, float scale, int64_t padding,
                     bool add, void* gw, void* ws, hipStream_t st) {
  if (!M) return add ? hipSuccess : launch_zero(gw, (size_t)V * C * sizeof(T), st);
  const Layout w(M, C);
  auto at = [&](size_t byte) { return (unsigned*)((char*)ws + byte); };
  const Grouped grouped{at(w.token), at(w.place), (int*)at(w.used)};
  float* part = (float*)at(w.part);
  const int classes = std::min(V, CLASSES), rows = (V + CLASSES - 1) / CLASSES;
  int bits = 0;
  while (1 << bits < rows) ++bits;
  uint4* fill = add ? nullptr : (uint4*)gw;
  const int units = (int)(C * sizeof(T) / 16);
  if (w.segs) {
    hipLaunchKernelGGL(split_kernel, dim3(w.segs), dim3(256), 0, st, tokens, wide, M, V, padding, at(w.list),
                       (int*)at(w.starts));
    hipLaunchKernelGGL(group_kernel<false>, dim3(classes), dim3(256), 0, st, tokens, wide, M, V, padding, at(w.list),
                       (const int*)at(w.starts), w.segs, rows, bits, grouped, fill, units);
  } else {
    hipLaunchKernelGGL(group_kernel<true>, dim3(classes), dim3(256), 0, st, tokens, wide, M, V, padding, nullptr,
                       nullptr, 0, rows, bits, grouped, fill, units);
  }
  const int tiles = (M + TILE - 1) / TILE, cols = (C + 8 * WAVE - 1) / (8 * WAVE);
  hipLaunchKernelGGL((run_sum_kernel<T>), dim3(tiles, cols), dim3(SUM_WAVES * WAVE), 0, st, (const T*)gy, grouped, C,
                     scale, add, (T*)gw, part);
  if (tiles > 1)
    hipLaunchKernelGGL((run_join_kernel<T>), dim3(tiles - 1, cols), dim3(SUM_WAVES * WAVE), 0, st, grouped, C, scale,
                       add, part, (T*)gw);
  return hipGetLastError();
}

template <class T>
hipError_t embed_fwd(const void* tokens, bool wide, int M, const void* w, int V, int C, float scale, void* y,
                     hipStream_t st) {
  const int u = C / 8;
#define FWD(TPR, UNITS)                                                                                              \
  hipLaunchKernelGGL((embed_kernel<T, TPR, UNITS>), dim3(std::min((M + 256 / TPR - 1) / (256 / TPR), 1 << 20)), \
                     dim3(256), 0, st, tokens, wide, M, (const T*)w, V, C, scale, (T*)y)
  if (u <= 16) FWD(16, 1);
  else if (u <= 64) FWD(64, 1);
  else if (u <= 128) FWD(64, 2);
  else if (u <= 256) FWD(64, 4);
  else FWD(128, 4);
#undef FWD
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_fwd(bool bf16_io, const void* tokens, bool wide, int M, const void* w, int V, int C,
                            float scale, void* y, hipStream_t st) {
  return bf16_io ? embed_fwd<bf16>(tokens, wide, M, w, V, C, scale, y, st)
                 : embed_fwd<float>(tokens, wide, M, w, V, C, scale, y, st);
}

size_t embed_bwd_bytes(int M, int C) { return M ? Layout(M, C).end : 0; }

hipError_t launch_embed_bwd(bool bf16_io, const void* gy, const void* tokens, bool wide, int M, int V, int C,
                            float scale, int64_t padding, bool add, void* gw, void* ws, hipStream_t st) {
  return bf16_io ? embed_bwd<bf16>(gy, tokens, wide, M, V, C, scale, padding, add, gw, ws, st)
                 : embed_bwd<float>(gy, tokens, wide, M, V, C, scale, padding, add, gw, ws, st);
}

}  // namespace instant
