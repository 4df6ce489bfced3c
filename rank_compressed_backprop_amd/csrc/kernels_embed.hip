// Rows of a table looked up by token and scaled, and the table's gradient (include/instant_ops.h):
//   y[m] = s W[t[m]]        gW[v] = s sum_{m: t[m] = v} gy[m], in the order of m
//
// The gradient sorts the tokens with their places and sums runs of equal tokens, so it needs no
// float atomics and gives the same bits every time:
//   chunk_sort   chunks of SORT_N tokens, each sorted in LDS by (token, place)
//   merge_rank   a token's place in the order of all: its place in its own chunk and, by binary
//                search, the tokens of the other chunks that come before it
//   run_sum      tiles of RUN_TILE sorted tokens: runs inside a tile are summed and written, the
//                ends of runs that cross its borders left as partial rows
//   run_join     sums the partial rows of a run, in order
#include <algorithm>

#include "ops.hpp"

namespace instant {

namespace {

constexpr int SORT_BITS = 12, SORT_N = 1 << SORT_BITS;  // tokens a chunk
constexpr unsigned NO_TOKEN = 1u << 18;                 // what takes no part: it sorts behind every token
constexpr int RUN_TILE = 32;

__device__ __forceinline__ int64_t token_at(const void* t, bool wide, size_t i) {
  return wide ? ((const int64_t*)t)[i] : (int64_t)((const int32_t*)t)[i];
}

template <class T> using vec8_t = typename MM<T>::vec8;

}  // namespace

// TPR threads a row of U units of 8 columns, 256 / TPR rows a block.
template <class T, int TPR>
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
    for (int n = 8 * i; n < C; n += 8 * TPR) {
      float v[8];
      load8(row + n, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = in ? v[j] * scale : NAN;
      store_row<T, 8>(out + n, v);
    }
  }
}

// keys[SORT_N * chunk + i]: (token, place in the chunk) of chunk blockIdx.x in order.
__global__ __launch_bounds__(1024) void chunk_sort_kernel(const void* __restrict__ tokens, bool wide, int M, int V,
                                                          int64_t padding, unsigned* __restrict__ keys) {
  __shared__ unsigned k[SORT_N];
  const int base = blockIdx.x * SORT_N;
  for (int i = threadIdx.x; i < SORT_N; i += 1024) {
    unsigned t = NO_TOKEN;
    if (base + i < M) {
      const int64_t v = token_at(tokens, wide, base + i);
      if (v >= 0 && v < V && v != padding) t = (unsigned)v;
    }
    k[i] = t << SORT_BITS | i;
  }
  for (int size = 2; size <= SORT_N; size *= 2)
    for (int d = size / 2; d > 0; d /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < SORT_N / 2; i += 1024) {
        const int a = (i & ~(d - 1)) * 2 + (i & (d - 1)), b = a + d;
        const unsigned x = k[a], y = k[b];
        if ((x > y) == ((a & size) == 0)) {
          k[a] = y;
          k[b] = x;
        }
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < SORT_N; i += 1024)
    if (base + i < M) keys[base + i] = k[i];
}

// sorted[i] = (token, place) of the i-th of the M tokens in order of (token, place). (A chunk's
// places behind M hold the last keys, which sort behind all that are stored.)
__global__ __launch_bounds__(256) void merge_rank_kernel(const unsigned* __restrict__ keys, int M,
                                                         uint2* __restrict__ sorted) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= M) return;
  const unsigned key = keys[i], t = key >> SORT_BITS;
  const int own = i >> SORT_BITS, chunks = (M + SORT_N - 1) >> SORT_BITS;
  int rank = i & (SORT_N - 1);
  for (int c = 0; c < chunks; ++c) {
    if (c == own) continue;
    // keys of chunk c below this: equal tokens come first from earlier chunks
    const unsigned limit = (c < own ? t + 1 : t) << SORT_BITS;
    int lo = 0, hi = min(SORT_N, M - (c << SORT_BITS));
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (keys[(c << SORT_BITS) + mid] < limit) lo = mid + 1;
      else hi = mid;
    }
    rank += lo;
  }
  sorted[rank] = uint2{t, (unsigned)(own << SORT_BITS) + (key & (SORT_N - 1))};
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

// Tile blockIdx.x, columns 8 (256 blockIdx.y + tid) ..: part[tile][0] the sum of a run that goes on
// from the tile before, part[tile][1] of one that begins here and goes on in the next.
template <class T>
__global__ __launch_bounds__(256) void run_sum_kernel(const T* __restrict__ gy, const uint2* __restrict__ sorted, int M,
                                                      int C, float scale, bool add, T* __restrict__ gw,
                                                      float* __restrict__ part) {
  const int tile = blockIdx.x, i0 = tile * RUN_TILE, i1 = min(i0 + RUN_TILE, M);
  const int n = 8 * (256 * blockIdx.y + threadIdx.x);
  if (n >= C) return;
  float acc[8];
  bool fresh = !(i0 > 0 && sorted[i0 - 1].x == sorted[i0].x);
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  for (int i = i0; i < i1; ++i) {
    const uint2 e = sorted[i];
    if (e.x == NO_TOKEN) break;
    float v[8];
    load8(gy + (size_t)e.y * C + n, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += v[j];
    const bool goes_on = i + 1 < M && sorted[i + 1].x == e.x;
    if (goes_on && i + 1 < i1) continue;
    if (fresh && !goes_on) put(gw + (size_t)e.x * C + n, add, scale, acc);
    else store_row<float, 8>(part + ((size_t)2 * tile + (fresh ? 1 : 0)) * C + n, acc);
    fresh = true;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  }
}

// Tile blockIdx.x: if a run begins in it and goes on, its partial rows in order.
template <class T>
__global__ __launch_bounds__(256) void run_join_kernel(const uint2* __restrict__ sorted, int M, int C, float scale,
                                                       bool add, const float* __restrict__ part, T* __restrict__ gw) {
  const int tile = blockIdx.x, last = (tile + 1) * RUN_TILE - 1;  // (the last tile has no block)
  const unsigned t = sorted[last].x;
  if (t == NO_TOKEN || sorted[last + 1].x != t) return;
  if (tile > 0 && sorted[tile * RUN_TILE - 1].x == t) return;  // it came from the tile before
  const int n = 8 * (256 * blockIdx.y + threadIdx.x);
  if (n >= C) return;
  float acc[8];
  load8(part + ((size_t)2 * tile + 1) * C + n, acc);
  for (int u = tile + 1; u * RUN_TILE < M && sorted[u * RUN_TILE].x == t; ++u) {
    float v[8];
    load8(part + (size_t)2 * u * C + n, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += v[j];
  }
  put(gw + (size_t)t * C + n, add, scale, acc);
}

namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <class T>
hipError_t embed_bwd(const void* gy, const void* tokens, bool wide, int M, int V, int C, float scale, int64_t padding,
                     bool add, void* gw, void* ws, hipStream_t st) {
  if (!add) {
    const hipError_t e = launch_zero(gw, (size_t)V * C * sizeof(T), st);
    if (e != hipSuccess) return e;
  }
  if (!M) return hipSuccess;
  unsigned* keys = (unsigned*)ws;
  uint2* sorted = (uint2*)((char*)ws + align256((size_t)M * 4));
  float* part = (float*)((char*)sorted + align256((size_t)M * 8));
  const int chunks = (M + SORT_N - 1) / SORT_N, tiles = (M + RUN_TILE - 1) / RUN_TILE;
  hipLaunchKernelGGL(chunk_sort_kernel, dim3(chunks), dim3(1024), 0, st, tokens, wide, M, V, padding, keys);
  hipLaunchKernelGGL(merge_rank_kernel, dim3((M + 255) / 256), dim3(256), 0, st, keys, M, sorted);
  const int cols = (C + 2047) / 2048;
  hipLaunchKernelGGL((run_sum_kernel<T>), dim3(tiles, cols), dim3(256), 0, st, (const T*)gy, sorted, M, C, scale, add,
                     (T*)gw, part);
  if (tiles > 1)
    hipLaunchKernelGGL((run_join_kernel<T>), dim3(tiles - 1, cols), dim3(256), 0, st, sorted, M, C, scale, add, part,
                       (T*)gw);
  return hipGetLastError();
}

template <class T>
hipError_t embed_fwd(const void* tokens, bool wide, int M, const void* w, int V, int C, float scale, void* y,
                     hipStream_t st) {
  const int u = C / 8;
#define FWD(TPR)                                                                                                   \
  hipLaunchKernelGGL((embed_kernel<T, TPR>), dim3(std::min((M + 256 / TPR - 1) / (256 / TPR), 1 << 20)), dim3(256), \
                     0, st, tokens, wide, M, (const T*)w, V, C, scale, (T*)y)
  if (u <= 16) FWD(16);
  else if (u <= 64) FWD(64);
  else FWD(256);
#undef FWD
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_fwd(bool bf16_io, const void* tokens, bool wide, int M, const void* w, int V, int C,
                            float scale, void* y, hipStream_t st) {
  return bf16_io ? embed_fwd<bf16>(tokens, wide, M, w, V, C, scale, y, st)
                 : embed_fwd<float>(tokens, wide, M, w, V, C, scale, y, st);
}

size_t embed_bwd_bytes(int M, int C) {
  if (!M) return 0;
  const size_t tiles = (M + RUN_TILE - 1) / RUN_TILE;
  return align256((size_t)M * 4) + align256((size_t)M * 8) + 2 * tiles * C * 4;
}

hipError_t launch_embed_bwd(bool bf16_io, const void* gy, const void* tokens, bool wide, int M, int V, int C,
                            float scale, int64_t padding, bool add, void* gw, void* ws, hipStream_t st) {
  return bf16_io ? embed_bwd<bf16>(gy, tokens, wide, M, V, C, scale, padding, add, gw, ws, st)
                 : embed_bwd<float>(gy, tokens, wide, M, V, C, scale, padding, add, gw, ws, st);
}

}  // namespace instant
