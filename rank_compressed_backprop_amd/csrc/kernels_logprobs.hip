// Log probabilities of given tokens from logits, the entropy and the most likely alternatives, and
// the logits' gradient (include/instant_ops.h):
//   m = max z, S = sum exp(z - m), E = sum exp(z - m) (z - m)
//   lse = m + log S;  logp = z_t - m - log S;  H = log S - E / S
//   gz_j = g_logp (1[j = t] - p_j) + g_lse p_j - g_H p_j (log p_j + H),  p_j = exp(z_j - m - log S)
#include <algorithm>

#include "ops.hpp"

namespace instant {

namespace {

constexpr float LOG2E = 1.44269504088896341f;
constexpr float LOWEST = -3.402823466e38f;  // the running maximum before any value: finite, so that
                                            // -inf - it is -inf (and its exponential 0), not NaN
constexpr float FAR = -1000.0f;  // exp of it and of all below is 0; finite, so that 0 * it is 0

// The values of a row in chunks of 16 bytes that are aligned in memory: chunk c holds elements
// first(c) .. first(c) + CE - 1, and the chunks at the ends may hang over the row.
template <class T> struct Row {
  static constexpr int CE = 16 / sizeof(T);
  const T* p;
  int n, off, chunks;
  __device__ Row(const T* base, size_t at, int n_) : p(base + at), n(n_) {
    off = (int)(((uintptr_t)p & 15) / sizeof(T));
    chunks = (off + n + CE - 1) / CE;
  }
  __device__ int first(int c) const { return c * CE - off; }
  // chunk c; places outside the row hold `none`
  __device__ void load(int c, float none, float v[CE]) const { load(p, true, c, none, v); }
  // the same elements of another row of n, whole chunks at once if its alignment is the same
  __device__ void load(const T* q, bool same, int c, float none, float v[CE]) const {
    const int j0 = first(c);
    if (same && j0 >= 0 && j0 + CE <= n) {
      typedef T vec __attribute__((ext_vector_type(CE)));
      const vec r = *reinterpret_cast<const vec*>(q + j0);
#pragma unroll
      for (int j = 0; j < CE; ++j) v[j] = (float)r[j];
    } else {
#pragma unroll
      for (int j = 0; j < CE; ++j) v[j] = j0 + j >= 0 && j0 + j < n ? (float)q[j0 + j] : none;
    }
  }
};

__device__ __forceinline__ float exp_of(float t) { return __builtin_amdgcn_exp2f(t * LOG2E); }

// Running maximum m, s = sum exp(z - m), e = sum exp(z - m) (z - m).
struct Sums {
  float m = LOWEST, s = 0.0f, e = 0.0f;
  // the sums as if m had been `to` >= m
  __device__ void rise(float to) {
    const float d = fmaxf(m - to, FAR), r = exp_of(d);
    e = r * fmaf(d, s, e);
    s *= r;
    m = to;
  }
  __device__ void add(float z) {  // z <= m, or NaN, which stays
    const float t = z - m, p = exp_of(t);
    s += p;
    e = fmaf(p, fmaxf(t, FAR), e);
  }
  __device__ void join(float om, float os, float oe) {
    const float to = fmaxf(m, om);
    rise(to);
    const float d = fmaxf(om - to, FAR), r = exp_of(d);
    s = fmaf(r, os, s);
    e = fmaf(r, fmaf(d, os, oe), e);
  }
};

// Order of the alternatives: larger values first, then lower places; -0 and 0 are equal, and a NaN
// ranks with -inf. The place may be an element's or a chunk's.
__device__ __forceinline__ unsigned order_of(float v) {
  const unsigned b = __builtin_bit_cast(unsigned, fmaxf(v, -INFINITY) + 0.0f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned o) {
  return __builtin_bit_cast(float, o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(float v, int place) { return (uint64_t)order_of(v) << 32 | ~(unsigned)place; }

__device__ __forceinline__ int64_t token_at(const void* t, bool wide, size_t i) {
  return wide ? ((const int64_t*)t)[i] : (int64_t)((const int32_t*)t)[i];
}

constexpr int CANDS = 1024;  // alternatives that are held for ranking

}  // namespace

// A block of TPB threads a row. One pass: each thread keeps the sums over its chunks (tid, tid +
// TPB, ...), which are joined in a fixed order.
//
// TOP: with it each thread keeps its largest value and the first of its chunks that holds it. Of
// the keys (value, chunk) of 64 groups of threads the k-th largest bounds the k-th alternative from
// below: k groups hold an element each that ranks before every element of a chunk that ranks below
// the bound. So only chunks of threads whose best reaches the bound are read again (about k of them
// in TPB, from the cache), and the few elements that reach it are ranked by counting. Should more
// reach it than are held, the k-th of those held is a higher bound, and the chunks are read again
// (each time at least CANDS - k elements fewer reach it).
template <class T, int TPB, bool TOP>
__global__ __launch_bounds__(TPB) void logprobs_kernel(const T* __restrict__ z, const void* __restrict__ targets,
                                                       bool wide, int M, int W, int V, int64_t ignore, int k,
                                                       float* __restrict__ logp, float* __restrict__ lse,
                                                       float* __restrict__ entropy, float* __restrict__ stats,
                                                       float* __restrict__ top_logp, int64_t* __restrict__ top_index) {
  typedef Row<T> R;
  constexpr int CE = R::CE, U = 32 / CE, WAVES = TPB / WAVE;
  __shared__ float sums[3][WAVES];
  __shared__ uint64_t groups[TOP ? 64 : 1], cand[TOP ? CANDS : 1], bound_;
  __shared__ int list[TOP ? TPB : 1], nlist, ncand;
  const int tid = threadIdx.x, lane = tid % WAVE, wave = tid / WAVE;
  for (int row = blockIdx.x; row < M; row += gridDim.x) {
    const R r(z, (size_t)row * W, V);
    int64_t t = -1;
    float zt = 0.0f;
    bool given = false, valid = false;
    if (tid == 0 && targets) {
      t = token_at(targets, wide, row);
      given = t != ignore;
      valid = t >= 0 && t < V;
      if (given && valid) zt = (float)r.p[t];
    }
    Sums a;
    float best = -INFINITY;
    int at = tid;
    for (int c0 = tid; c0 < r.chunks; c0 += U * TPB) {
      float v[U][CE], mx = a.m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c0 + u * TPB < r.chunks) {
          r.load(c0 + u * TPB, -INFINITY, v[u]);
        } else {
#pragma unroll
          for (int j = 0; j < CE; ++j) v[u][j] = -INFINITY;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float c = v[u][0];
#pragma unroll
        for (int j = 1; j < CE; ++j) c = fmaxf(c, v[u][j]);
        mx = fmaxf(mx, c);
        if (TOP && c > best) {
          best = c;
          at = c0 + u * TPB;
        }
      }
      a.rise(mx);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < CE; ++j) a.add(v[u][j]);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) a.join(__shfl_xor(a.m, d), __shfl_xor(a.s, d), __shfl_xor(a.e, d));
    const uint64_t mine = TOP && tid < r.chunks ? key_of(best, at) : 0;  // 0: no chunk
    __syncthreads();  // the last row's readers are done
    if (lane == 0) {
      sums[0][wave] = a.m;
      sums[1][wave] = a.s;
      sums[2][wave] = a.e;
    }
    if (TOP) {
      uint64_t g = mine;
#pragma unroll
      for (int d = 1; d < TPB / 64; d *= 2) {
        const uint64_t o = __shfl_xor(g, d);
        g = o > g ? o : g;
      }
      if (tid % (TPB / 64) == 0) groups[tid / (TPB / 64)] = g;
      if (tid == 0) {
        bound_ = 0;
        nlist = ncand = 0;
      }
    }
    __syncthreads();
    Sums all;
    all.m = sums[0][0];
    all.s = sums[1][0];
    all.e = sums[2][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) all.join(sums[0][w], sums[1][w], sums[2][w]);
    const bool empty = all.s == 0.0f;
    const float top = empty ? 0.0f : all.m, ls = logf(all.s);
    if (tid == 0) {
      if (logp)
        logp[row] = !given ? 0.0f : !valid ? NAN : empty ? -INFINITY : zt - top - ls;
      if (lse) lse[row] = top + ls;
      if (entropy) entropy[row] = empty ? 0.0f : ls - all.e / all.s;
      if (stats) {
        stats[2 * (size_t)row] = top;
        stats[2 * (size_t)row + 1] = ls;
      }
    }
    if constexpr (TOP) {
      if (wave == 0) {
        const uint64_t g = groups[lane];
        int rank = 0;
        for (int i = 0; i < 64; ++i) rank += groups[i] > g;
        if (rank == k - 1 && g) bound_ = g;
      }
      __syncthreads();
      // elements that reach the bound: of a larger value, or of its value and a chunk up to its
      uint64_t bound = bound_;
      if (mine && mine >= bound) list[atomicAdd(&nlist, 1)] = tid;
      __syncthreads();
      const int its = (r.chunks + TPB - 1) / TPB, nl = nlist;
      bool by_chunk = true;
      while (true) {
        for (int i = tid; i < its * nl; i += TPB) {
          const int c = (i / nl) * TPB + list[i % nl];
          if (c >= r.chunks) continue;
          float v[CE];
          r.load(c, -INFINITY, v);
#pragma unroll
          for (int j = 0; j < CE; ++j) {
            const int el = r.first(c) + j;
            if (el < 0 || el >= V) continue;
            if (key_of(v[j], by_chunk ? c : el) >= bound) {
              const int slot = atomicAdd(&ncand, 1);
              if (slot < CANDS) cand[slot] = key_of(v[j], el);
            }
          }
        }
        __syncthreads();
        const int n = min(ncand, CANDS);
        const bool more = ncand > CANDS;
        for (int i = tid; i < n; i += TPB) {
          const uint64_t g = cand[i];
          int rank = 0;
          for (int j = 0; j < n; ++j) rank += cand[j] > g;
          if (more) {
            if (rank == k - 1) bound_ = g;
          } else if (rank < k) {
            const float v = value_of((unsigned)(g >> 32));
            top_logp[(size_t)row * k + rank] = empty ? -INFINITY : v - top - ls;
            top_index[(size_t)row * k + rank] = (int64_t)(unsigned)~(unsigned)g;
          }
        }
        if (!more) break;
        __syncthreads();
        bound = bound_;
        by_chunk = false;
        if (tid == 0) ncand = 0;
        __syncthreads();
      }
    }
  }
}

// The logits' gradient, a piece of PIECE chunks of a row a block. gz may be z (a thread writes the
// chunks that it has read).
constexpr int BACK_CHUNKS = 1024;

template <class T>
__global__ __launch_bounds__(256) void logprobs_bwd_kernel(const T* z, const void* __restrict__ targets, bool wide,
                                                           int M, int W, int V, int64_t ignore,
                                                           const float* __restrict__ stats,
                                                           const float* __restrict__ entropy,
                                                           const float* __restrict__ g_logp,
                                                           const float* __restrict__ g_lse,
                                                           const float* __restrict__ g_ent, T* gz) {
  constexpr int CE = 16 / sizeof(T);
  // (a row of W values touches at most one chunk more than they fill)
  const int pieces = (W / CE + 2 + BACK_CHUNKS - 1) / BACK_CHUNKS;
  const size_t units = (size_t)M * pieces;
  for (size_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int row = (int)(u / pieces), piece = (int)(u % pieces);
    const Row<T> r(gz, (size_t)row * W, W);
    const T* in = z + (size_t)row * W;
    T* out = gz + (size_t)row * W;
    const bool same = (((uintptr_t)in ^ (uintptr_t)out) & 15) == 0;
    int64_t t = -1;
    float g = 0.0f;
    if (targets && g_logp) {
      t = token_at(targets, wide, row);
      if (t != ignore) g = t >= 0 && t < V ? g_logp[row] : NAN;
    }
    const float gl = g_lse ? g_lse[row] : 0.0f, gh = g_ent ? g_ent[row] : 0.0f;
    const float top = stats[2 * (size_t)row], ls = stats[2 * (size_t)row + 1];
    const bool none = g == 0.0f && gl == 0.0f && gh == 0.0f;  // zeros, whatever the row holds
    const bool empty = ls == -INFINITY;                         // p = 0
    const float c0 = gl - g - (gh != 0.0f ? gh * entropy[row] : 0.0f);
    const int c1 = min((piece + 1) * BACK_CHUNKS, r.chunks);
    for (int c = piece * BACK_CHUNKS + (int)threadIdx.x; c < c1; c += 256) {
      float v[CE], o[CE];
      const int j0 = r.first(c);
      r.load(in, same, c, 0.0f, v);
#pragma unroll
      for (int j = 0; j < CE; ++j) {
        const float lp = v[j] - top - ls;
        const float p = empty ? 0.0f : exp_of(lp);
        o[j] = p * fmaf(-gh, fmaxf(lp, FAR), c0);
        if (j0 + j == t) o[j] += g;
        if (none || j0 + j >= V) o[j] = 0.0f;
      }
      if (j0 >= 0 && j0 + CE <= W) {
        store_row<T, CE>(out + j0, o);
      } else {
#pragma unroll
        for (int j = 0; j < CE; ++j)
          if (j0 + j >= 0 && j0 + j < W) out[j0 + j] = from_f32<T>(o[j]);
      }
    }
  }
}

namespace {

template <class T, int TPB>
hipError_t run_fwd(const void* z, const void* targets, bool wide, int M, int W, int V, int64_t ignore, int k,
                   float* logp, float* lse, float* entropy, float* stats, float* top_logp, int64_t* top_index,
                   hipStream_t st) {
  const dim3 grid(std::min(M, 1 << 20));
  if (k)
    hipLaunchKernelGGL((logprobs_kernel<T, TPB, true>), grid, dim3(TPB), 0, st, (const T*)z, targets, wide, M, W, V,
                       ignore, k, logp, lse, entropy, stats, top_logp, top_index);
  else
    hipLaunchKernelGGL((logprobs_kernel<T, TPB, false>), grid, dim3(TPB), 0, st, (const T*)z, targets, wide, M, W, V,
                       ignore, k, logp, lse, entropy, stats, top_logp, top_index);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs_fwd(bool bf16_io, const void* z, const void* targets, bool wide, int M, int W, int V,
                               int64_t ignore, int k, float* logp, float* lse, float* entropy, float* stats,
                               float* top_logp, int64_t* top_index, hipStream_t st) {
  const int chunks = V / (bf16_io ? 8 : 4);
  // (TOP needs k <= 64 groups of threads with a chunk each, or few enough elements to hold)
  const int tpb = chunks <= 256 ? 64 : chunks >= 4096 && M <= 256 ? 1024 : 256;
#define FWD(T, TPB)                                                                                                 \
  return run_fwd<T, TPB>(z, targets, wide, M, W, V, ignore, k, logp, lse, entropy, stats, top_logp, top_index, st)
  if (bf16_io) {
    if (tpb == 64) FWD(bf16, 64);
    if (tpb == 256) FWD(bf16, 256);
    FWD(bf16, 1024);
  }
  if (tpb == 64) FWD(float, 64);
  if (tpb == 256) FWD(float, 256);
  FWD(float, 1024);
#undef FWD
}

hipError_t launch_logprobs_bwd(bool bf16_io, const void* z, const void* targets, bool wide, int M, int W, int V,
                               int64_t ignore, const float* stats, const float* entropy, const float* g_logp,
                               const float* g_lse, const float* g_ent, void* gz, hipStream_t st) {
  const int ce = bf16_io ? 8 : 4;
  const size_t pieces = (W / ce + 2 + BACK_CHUNKS - 1) / BACK_CHUNKS;
  const dim3 grid((unsigned)std::min<size_t>((size_t)M * pieces, 1 << 20));
  if (bf16_io)
    hipLaunchKernelGGL((logprobs_bwd_kernel<bf16>), grid, dim3(256), 0, st, (const bf16*)z, targets, wide, M, W, V,
                       ignore, stats, entropy, g_logp, g_lse, g_ent, (bf16*)gz);
  else
    hipLaunchKernelGGL((logprobs_bwd_kernel<float>), grid, dim3(256), 0, st, (const float*)z, targets, wide, M, W, V,
                       ignore, stats, entropy, g_logp, g_lse, g_ent, (float*)gz);
  return hipGetLastError();
}

}  // namespace instant
