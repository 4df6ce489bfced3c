// Log probabilities of given tokens from logits, the entropy and the most likely alternatives, and
// the logits' gradient (include/instant_ops.h):
//   m = max z, S = sum exp(z - m), E = sum exp(z - m) (z - m)
//   lse = m + log S;  logp = z_t - m - log S;  H = log S - E / S
//   gz_j = g_logp (1[j = t] - p_j) + g_lse p_j - g_H p_j (log p_j + H),  p_j = exp(z_j - m - log S)
#include <algorithm>

#include "ops.hpp"

namespace instant {

namespace {

constexpr float LOG2E = 1.44269504088896341f, LN2 = 0.693147180559945309f;
constexpr float LOWEST = -3.402823466e38f;  // the running maximum before any value: finite, so that
                                            // -inf - it is -inf (and its exponential 0), not NaN
constexpr float FAR = -1000.0f;  // 2^ or exp of it and of all below is 0; finite, so that 0 * it is 0

// The values of a row in chunks of 16 bytes that are aligned in memory: chunk c holds elements
// first(c) .. first(c) + CE - 1. Chunks [w0, w1) are whole; the ones at the ends may hang over the row.
template <class T> struct Row {
  static constexpr int CE = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(CE)));
  const T* p;
  int n, off, chunks, w0, w1;
  __device__ Row(const T* base, size_t at, int n_) : p(base + at), n(n_) {
    off = (int)(((uintptr_t)p & 15) / sizeof(T));
    chunks = (off + n + CE - 1) / CE;
    w0 = off ? 1 : 0;
    w1 = (off + n) / CE;
  }
  __device__ int first(int c) const { return c * CE - off; }
  __device__ vec whole(int c) const { return *reinterpret_cast<const vec*>(p + first(c)); }
  // any chunk, of this or another row of n; places outside it hold `none`
  __device__ void part(const T* q, int c, float none, float* v) const {
    const int j0 = first(c);
#pragma unroll
    for (int j = 0; j < CE; ++j) v[j] = j0 + j >= 0 && j0 + j < n ? (float)q[j0 + j] : none;
  }
  __device__ void load(int c, float none, float* v) const {
    if (c >= w0 && c < w1) {
      const vec r = whole(c);
#pragma unroll
      for (int j = 0; j < CE; ++j) v[j] = (float)r[j];
    } else {
      part(p, c, none, v);
    }
  }
};

__device__ __forceinline__ float exp_of(float t) { return __builtin_amdgcn_exp2f(t * LOG2E); }

// The exponent of two of a value z beside the running maximum m: log2(e) z - fl(log2(e) m), one
// operation and one rounding, where m is small enough that the rounding of log2(e) m is; it is made
// good where sums of different maxima meet, and at the end. Else log2(e) (z - m).
constexpr float NEAR = 1048576.0f;
__device__ __forceinline__ bool near(float m) { return fabsf(m) <= NEAR; }
__device__ __forceinline__ float rest(float m) { return near(m) ? fmaf(m, LOG2E, -(m * LOG2E)) : 0.0f; }

// Running maximum m, s = sum 2^t, e = sum 2^t t for the exponents t. (In base 2 and without a limit
// for t: 8.5 issue slots a value, of them 4 the exponential's; with a difference, a product and a
// limit 11, and 16384 x 30522 in bfloat16 was bound by them.)
struct Sums {
  float m = LOWEST, s = 0.0f, e = 0.0f;
  // the sums as if m had been `to` >= m
  __device__ void rise(float to) {
    const float d = fmaxf(fmaf(m - to, LOG2E, rest(to) - rest(m)), FAR), r = __builtin_amdgcn_exp2f(d);
    e = r * fmaf(d, s, e);
    s *= r;
    m = to;
  }
  // N values, none above m but NaN, which stays. An infinite one makes 0 * -inf of its product with
  // its exponent; the sum shows it, and they are added again with a limit: `limited` counts how often
  // in a row (after two times it is expected).
  // SMALL: with a limit at once, which is less code.
  template <int N, bool SMALL> __device__ void add(const float* z, int& limited) {
    float ps = 0.0f, pe = NAN;
    const float m2 = m * LOG2E;
    if (!SMALL && limited < 2 && near(m)) {
      pe = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float t = fmaf(z[j], LOG2E, -m2), p = __builtin_amdgcn_exp2f(t);
        ps += p;
        pe = fmaf(p, t, pe);
        if (j % 8 == 7) __builtin_amdgcn_sched_barrier(0);  // (all at once take 30 registers more)
      }
    }
    const bool again = pe != pe;
    limited = again ? limited + 1 : 0;
    if (again) {
      ps = pe = 0.0f;
      const bool n = near(m);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float t = n ? fmaf(z[j], LOG2E, -m2) : (z[j] - m) * LOG2E, p = __builtin_amdgcn_exp2f(t);
        ps += p;
        pe = fmaf(p, fmaxf(t, FAR), pe);
      }
    }
    s += ps;
    e += pe;
  }
  __device__ void join(float om, float os, float oe) {
    const float to = fmaxf(m, om);
    rise(to);
    Sums o;
    o.m = om;
    o.s = os;
    o.e = oe;
    o.rise(to);
    s += o.s;
    e += o.e;
  }
  __device__ bool empty() const { return s == 0.0f; }
  __device__ float top() const { return empty() ? 0.0f : m; }
  // log sum exp(z - top)
  __device__ float log_sum() const { return empty() ? -INFINITY : (log2f(s) - rest(m)) * LN2; }
  __device__ float entropy() const { return empty() ? 0.0f : (log2f(s) - e / s) * LN2; }
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

// ---- steps of a group of G threads that share a row (16: a quarter of a wave; 64; or a block)

template <int CTRL> __device__ __forceinline__ int moved(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, true);
}
// op over groups of G = 4, 16 or 64 lanes, all of them active; every lane receives it, and the order
// is fixed. (Lanes 1 and 2 apart, then mirrored in 8 and 16, then the wave's four rows of 16.)
template <int G, class F> __device__ __forceinline__ int over_lanes(int v, F op) {
  v = op(v, moved<0xB1>(v));
  v = op(v, moved<0x4E>(v));
  if constexpr (G >= 16) {
    v = op(v, moved<0x141>(v));
    v = op(v, moved<0x140>(v));
  }
  if constexpr (G == 64)
    v = op(op(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
           op(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
  return v;
}
__device__ __forceinline__ float f32(int v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ int bits(float v) { return __builtin_bit_cast(int, v); }
template <int G> __device__ __forceinline__ float max_over(float v) {
  return f32(over_lanes<G>(bits(v), [](int a, int b) { return bits(fmaxf(f32(a), f32(b))); }));
}
template <int G> __device__ __forceinline__ float sum_over(float v) {
  return f32(over_lanes<G>(bits(v), [](int a, int b) { return bits(f32(a) + f32(b)); }));
}
template <int G> __device__ __forceinline__ int min_over(int v) {
  return over_lanes<G>(v, [](int a, int b) { return a < b ? a : b; });
}

// What the threads of a row have written to LDS is there for the others. (Stores to memory are not
// waited for, as a plain barrier would.)
template <int TPR> __device__ __forceinline__ void settled() {
#ifdef __HIP_DEVICE_COMPILE__
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  if constexpr (TPR > WAVE) __builtin_amdgcn_s_barrier();
  else __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
#endif
}

// f(key, rank) for each of the n keys in LDS, which PAD zeros follow, by one of the four lanes that
// count the keys above it. TPR threads; t: this one's number.
constexpr int PAD = 32;
template <int TPR, class F> __device__ __forceinline__ void ranked(const uint64_t* keys, int n, int t, F&& f) {
  for (int i = t / 4; i < n; i += TPR / 4) {
    const uint64_t g = keys[i];
    int rank = 0;
    for (int j = t % 4; j < n; j += PAD) {
      uint64_t o[PAD / 4];
#pragma unroll
      for (int u = 0; u < PAD / 4; ++u) o[u] = keys[j + 4 * u];
#pragma unroll
      for (int u = 0; u < PAD / 4; ++u) rank += o[u] > g;
    }
    rank = over_lanes<4>(rank, [](int x, int y) { return x + y; });
    if (t % 4 == 0) f(g, rank);
  }
}

// Chunks of a step (1024 threads have 128 registers each; a wave with alternatives takes as few, so that four
// blocks fit a compute unit).
constexpr int step_chunks(int tpr, int ce, int top) { return (tpr == 1024 || (tpr == WAVE && top == 2) ? 16 : 32) / ce; }
// Alternatives that are held for ranking, for a row of a wave or of a block.
constexpr int cands_of(int tpr) { return tpr == 64 ? 512 : 1024; }
constexpr int MAX_SLICES = 16, JOIN_KEYS = 512;  // of a row, and their alternatives

// The results of the rows; null: not asked for.
struct Out {
  float *logp, *lse, *entropy, *stats, *top_logp;
  int64_t* top_index;
};

struct Target {
  float z;
  bool given, valid;
};

// One thread writes them.
__device__ __forceinline__ void write_row(const Out& o, int row, const Sums& a, const Target& t) {
  const float top = a.top(), ls = a.log_sum();
  if (o.logp) o.logp[row] = !t.given ? 0.0f : !t.valid ? NAN : a.empty() ? -INFINITY : t.z - top - ls;
  if (o.lse) o.lse[row] = top + ls;
  if (o.entropy) o.entropy[row] = a.entropy();
  if (o.stats) {
    o.stats[2 * (size_t)row] = top;
    o.stats[2 * (size_t)row + 1] = ls;
  }
}

// The alternative of rank `rank` of a row.
__device__ __forceinline__ void write_top(const Out& o, int row, int k, int rank, uint64_t key, const Sums& a) {
  o.top_logp[(size_t)row * k + rank] =
      a.empty() ? -INFINITY : value_of((unsigned)(key >> 32)) - a.top() - a.log_sum();
  o.top_index[(size_t)row * k + rank] = (int64_t)(unsigned)~(unsigned)key;
}

template <class T>
__device__ __forceinline__ Target target_of(const T* row, const void* targets, bool wide, int m, int V, int64_t ignore) {
  Target r{0.0f, false, false};
  if (targets) {
    const int64_t t = token_at(targets, wide, m);
    r.given = t != ignore;
    r.valid = t >= 0 && t < V;
    if (r.given && r.valid) r.z = (float)row[t];
  }
  return r;
}

}  // namespace

// TPR threads a row (a block of max(TPR, 256) threads), or (SPLIT) a block for each of `slices`
// slices of a row, whose sums and alternatives go to parts and keys for the join kernel. One pass
// over the logits: each thread keeps the sums over its chunks (tid, tid + TPR, ...), which are then
// added in a fixed order.
//
// TOP 1 (k = 1): each thread also keeps its largest value and the first of its chunks that holds it;
// the first chunk that holds the largest of all is read again by one thread.
// TOP 2: and the largest of each step of U chunks, in 16 bits of LDS (rounded up). Of the keys (value,
// chunk) of 64 groups of threads the k-th largest bounds the k-th alternative from below: k groups
// hold an element each that ranks before every element of a chunk that ranks below the bound. So only
// the chunks of steps that reach the bound are read again (a few more than k steps, from the
// cache), and the elements that reach it, a few more than k too, are ranked by counting.
// Should more reach it than are held, the k-th of those held is a higher bound, and they are looked up
// again (each time at least as many fewer reach it as are held, but k).
// (16384 x 30522, back to back, takes 196 to 204 us with k = 0, 218 with 1 and 243 to 251 with 20: what follows
// a row's pass keeps its registers from the next row. A block of 256 threads a row, with its barriers, took 310;
// reading again all chunks of the threads whose best reaches the bound 364, holding such chunks in LDS
// during the pass 360.)
template <class T, int TPR, int TOP, bool SPLIT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void logprobs_kernel(
    const T* __restrict__ z, const void* __restrict__ targets, bool wide, int M, int W, int V, int64_t ignore, int k,
    Out out, int slices, float* __restrict__ parts, uint64_t* __restrict__ keys, int most_steps) {
  typedef Row<T> R;
  constexpr int CE = R::CE, U = step_chunks(TPR, CE, TOP), RPB = TPR < 256 ? 256 / TPR : 1, WAVES = TPR < WAVE ? 1 : TPR / WAVE;
  constexpr int LANES = TPR < WAVE ? TPR : WAVE, CANDS = cands_of(TPR), PER = TPR / 64 ? TPR / 64 : 1;
  static_assert(TPR >= WAVE || TOP < 2, "ranking takes a wave");
  // Every chunk by the same short loop, not a step of U at a time. Few rows: a block goes through its code
  // once or twice, and much of its time is the code's way from memory. (64 x 128000 in float32: 14 us a
  // slice kernel, with steps 18.) For many rows it is slower (8192 x 128000, k = 20: 425 -> 546 us).
  constexpr bool SMALL = TPR == 1024;
  __shared__ float sums[RPB][3][WAVES];
  __shared__ uint64_t groups_[TOP == 2 ? RPB : 1][64], cand_[TOP == 2 ? RPB : 1][TOP == 2 ? CANDS + PAD : 1];
  __shared__ uint64_t bound_[RPB];
  constexpr int LIST = 256;  // steps of a wave that are looked up at a time
  extern __shared__ uint16_t largest_[];  // [row of the block][step][thread]
  __shared__ uint16_t list_[TOP == 2 ? RPB * WAVES : 1][TOP == 2 ? LIST : 1];
  __shared__ float best_[RPB][WAVES];
  __shared__ int at_[RPB][WAVES], ncand_[RPB];
  const int tid = threadIdx.x % TPR, lane = tid % LANES, wave = tid / LANES, slot = threadIdx.x / TPR;
  // (the trip count is the block's: a row of a block may have barriers)
  for (int first = SPLIT ? blockIdx.x / slices : blockIdx.x * RPB; first < M;
       first += SPLIT ? gridDim.x / slices : gridDim.x * RPB) {
    const int row = min(first + slot, M - 1);  // (rows behind the last: the last again, not written)
    const bool there = first + slot < M;
    const R r(z, (size_t)row * W, V);
    const int slice = SPLIT ? (int)(blockIdx.x % slices) : 0;
    const int begin = SPLIT ? (int)((int64_t)r.chunks * slice / slices) : 0;
    const int end = SPLIT ? (int)((int64_t)r.chunks * (slice + 1) / slices) : r.chunks;
    const int w0 = max(begin, r.w0), w1 = min(end, r.w1);  // whole chunks; and one before and behind, if any
    const bool head = begin < r.w0, tail = end > r.w1 && !(head && r.chunks == 1);
    Target target{0.0f, false, false};
    if (!SPLIT && tid == 0) target = target_of(r.p, targets, wide, row, V, ignore);
    Sums a;
    float best = -INFINITY;
    int at = 0x7fffffff;  // no chunk
    int limited = 0;
    const int steps = TOP == 2 ? max(w1 - w0, 0) / (U * TPR) + 1 : 0;  // (the last may be short)
    uint16_t* largest = largest_ + (size_t)slot * most_steps * TPR + tid;
    int step = 0;
    auto note = [&](float mx) {
      const unsigned b = __builtin_bit_cast(unsigned, mx);
      largest[step * TPR] = (uint16_t)((sizeof(T) == 2 || b >> 31 ? b : b + 0xffffu) >> 16);
    };
    auto end_chunk = [&](int c) {
        float v[CE], mx = -INFINITY;
        r.part(r.p, c, -INFINITY, v);
#pragma unroll
        for (int j = 0; j < CE; ++j) mx = fmaxf(mx, v[j]);
        if (TOP && (mx > best || at == 0x7fffffff)) {
          best = mx;
          at = c;
        }
        a.rise(fmaxf(a.m, mx));
        a.template add<CE, SMALL>(v, limited);
        limited = 0;
    };
    if (head && tid == 0) end_chunk(0);
    if (w0 < w1) {
      // The next chunks are requested before these are added (behind the last, the last again), and
      // no branch is between a request and the next.
      typename R::vec cur[U];
      int c = w0 + tid;
      if (TOP && c < w1 && at == 0x7fffffff) at = c;
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = r.whole(min(c + u * TPR, w1 - 1));
      auto add = [&](auto N) {  // the first N of the chunks in cur; their largest
        float v[N * CE], mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < N; ++u) {
          float cm = -INFINITY;
#pragma unroll
          for (int j = 0; j < CE; ++j) {
            v[u * CE + j] = (float)cur[u][j];
            cm = fmaxf(cm, v[u * CE + j]);
          }
          mx = fmaxf(mx, cm);
          if (TOP && cm > best) {
            best = cm;
            at = c + u * TPR;
          }
        }
        a.rise(fmaxf(a.m, mx));
        a.template add<N * CE, SMALL>(v, limited);
        return mx;
      };
      float mx = -INFINITY;
      if constexpr (SMALL) {
        for (int n = 1; c < w1; ++n) {
          mx = fmaxf(mx, add(std::integral_constant<int, 1>{}));
          if (TOP == 2 && (n % U == 0 || c + TPR >= w1)) {
            note(mx);
            ++step;
            mx = -INFINITY;
          }
          c += TPR;
#pragma unroll
          for (int u = 0; u + 1 < U; ++u) cur[u] = cur[u + 1];
          cur[U - 1] = r.whole(min(c + (U - 1) * TPR, w1 - 1));
        }
      } else {
        while (c + (U - 1) * TPR < w1) {
          typename R::vec next[U];
#pragma unroll
          for (int u = 0; u < U; ++u) next[u] = r.whole(min(c + (U + u) * TPR, w1 - 1));
          mx = add(std::integral_constant<int, U>{});
          if constexpr (TOP == 2) {
            note(mx);
            ++step;
          }
          c += U * TPR;
#pragma unroll
          for (int u = 0; u < U; ++u) cur[u] = next[u];
        }
        mx = -INFINITY;
        while (c < w1) {  // (at most U - 1 times)
          mx = fmaxf(mx, add(std::integral_constant<int, 1>{}));
          c += TPR;
#pragma unroll
          for (int u = 0; u + 1 < U; ++u) cur[u] = cur[u + 1];
        }
        if constexpr (TOP == 2)
          if (step < steps) note(mx);
      }
    }
    if (tail && tid == TPR - 1) end_chunk(r.chunks - 1);
    a.rise(max_over<LANES>(a.m));
    a.s = sum_over<LANES>(a.s);
    a.e = sum_over<LANES>(a.e);
    const bool has = at != 0x7fffffff;
    float wave_best = -INFINITY;
    int wave_at = 0x7fffffff;
    if constexpr (TOP == 1) {
      wave_best = max_over<LANES>(best);
      wave_at = min_over<LANES>(best == wave_best ? at : 0x7fffffff);
    }
    const uint64_t mine = TOP == 2 && has ? key_of(best, at) : 0;  // 0: no chunk
    if constexpr (TOP == 2) {
      uint64_t g = mine;
      if constexpr (PER > 1) {
        const float b = max_over<PER>(best);
        const int c = min_over<PER>(best == b ? at : 0x7fffffff);
        g = c == 0x7fffffff ? 0 : key_of(b, c);
      }
      if (tid % PER == 0) groups_[slot][tid / PER] = g;
      if (tid == 0) {
        ncand_[slot] = 0;
        bound_[slot] = 0;  // (fewer than k groups hold a chunk: everything reaches it)
      }
    }
    if constexpr (WAVES > 1) {
      if (lane == 0) {
        sums[slot][0][wave] = a.m;
        sums[slot][1][wave] = a.s;
        sums[slot][2][wave] = a.e;
        best_[slot][wave] = wave_best;
        at_[slot][wave] = wave_at;
      }
    }
    if constexpr (WAVES > 1 || TOP == 2) settled<TPR>();
    if constexpr (WAVES > 1) {
      a = Sums{};
      for (int w = 0; w < WAVES; ++w) {
        a.join(sums[slot][0][w], sums[slot][1][w], sums[slot][2][w]);
        if (TOP == 1) {
          const float b = best_[slot][w];
          const int c = at_[slot][w];
          if (w == 0 || b > wave_best || (b == wave_best && c < wave_at)) {
            wave_best = b;
            wave_at = c;
          }
        }
      }
    }
    const size_t part = (size_t)row * slices + slice;
    if (tid == 0 && there) {
      if constexpr (SPLIT) {
        parts[3 * part] = a.m;
        parts[3 * part + 1] = a.s;
        parts[3 * part + 2] = a.e;
      } else {
        write_row(out, row, a, target);
      }
      if constexpr (TOP == 1) {
        float v[CE];
        r.load(wave_at, -INFINITY, v);
        uint64_t key = 0;
#pragma unroll
        for (int j = 0; j < CE; ++j) {
          const int el = r.first(wave_at) + j;
          const uint64_t o = el >= 0 && el < V ? key_of(v[j], el) : 0;
          key = o > key ? o : key;
        }
        if constexpr (SPLIT) keys[part] = key;
        else write_top(out, row, 1, 0, key, a);
      }
    }
    if constexpr (TOP == 2) {
      uint64_t* cand = cand_[slot];
      // the k-th largest of the groups' keys (0: fewer hold a chunk), four lanes a key
      for (int i = wave * 16 + lane / 4; i < 64; i += WAVES * 16) {
        const uint64_t g = groups_[slot][i];
        int rank = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) rank += groups_[slot][4 * j + lane % 4] > g;
        rank = over_lanes<4>(rank, [](int x, int y) { return x + y; });
        if (rank == k - 1 && g && lane % 4 == 0) bound_[slot] = g;
      }
      settled<TPR>();
      uint64_t bound = bound_[slot];
      uint16_t* list = list_[slot * WAVES + wave];
      bool by_chunk = true;
      float bound_value = -INFINITY;
      int bound_place = 0x7fffffff;
      while (true) {
        if (bound) {
          bound_value = value_of((unsigned)(bound >> 32));
          bound_place = (int)~(unsigned)bound;
        }
        // elements that reach it: of a larger value, or of its value and a chunk (or place) up to its.
        // A lane looks at one (less code than a chunk a lane: what runs once in a small call is fetched
        // from memory first), N of them requested at a time.
        auto look = [&](auto N, const bool* is, const int* c, const int* j) {
          float v[N];
#pragma unroll
          for (int u = 0; u < N; ++u) {
            const int el = r.first(c[u]) + j[u];
            v[u] = (float)r.p[is[u] && el >= 0 && el < V ? el : 0];
          }
#pragma unroll
          for (int u = 0; u < N; ++u) {
            const int el = r.first(c[u]) + j[u];
            const float w = fmaxf(v[u], -INFINITY);
            if (is[u] && el >= 0 && el < V && (w > bound_value || (w == bound_value && (by_chunk ? c[u] : el) <= bound_place))) {
              const int n = atomicAdd(&ncand_[slot], 1);
              if (n < CANDS) cand[n] = key_of(w, el);
            }
          }
        };
        int n_list = 0;
        for (int s = 0; s <= steps; ++s) {
          if (s < steps && w0 < w1) {
            const int c = w0 + tid + s * U * TPR;  // of the step, the first
            const float most = __builtin_bit_cast(float, (unsigned)largest[s * TPR] << 16);
            const bool reach = c < w1 && (most > bound_value ||
                                          (most == bound_value && (by_chunk ? c : r.first(c)) <= bound_place));
            const uint64_t m = __ballot(reach);
            if (reach) list[n_list + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(s << 6 | lane);
            n_list += __popcll(m);
          }
          if (n_list <= LIST - WAVE && s < steps) continue;
          settled<WAVE>();
          const int elements = n_list * U * CE;
          for (int i0 = lane; i0 < elements; i0 += 4 * WAVE) {
            bool is[4];
            int c[4], j[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int i = min(i0 + u * WAVE, elements - 1), e = list[i / (U * CE)];
              c[u] = w0 + wave * WAVE + (e & 63) + ((e >> 6) * U + i / CE % U) * TPR;
              j[u] = i % CE;
              is[u] = i0 + u * WAVE < elements && c[u] < w1;
            }
            look(std::integral_constant<int, 4>{}, is, c, j);
          }
          n_list = 0;
          settled<WAVE>();
        }
        if (wave == 0 && (head || tail)) {
          const bool is = lane < CE ? head : tail && lane < 2 * CE;
          const int c = lane < CE ? 0 : r.chunks - 1, j = lane % CE;
          look(std::integral_constant<int, 1>{}, &is, &c, &j);
        }
        settled<TPR>();
        const int n = min(ncand_[slot], CANDS);
        const bool more = ncand_[slot] > CANDS;
        if (tid < PAD) cand[n + tid] = 0;
        settled<TPR>();
        ranked<TPR>(cand, n, tid, [&](uint64_t g, int rank) {
          if (more) {
            if (rank == k - 1) bound_[slot] = g;
          } else if (rank < k && there) {
            if constexpr (SPLIT) keys[part * k + rank] = g;
            else write_top(out, row, k, rank, g, a);
          }
        });
        if (!more) {
          if (SPLIT && there)  // a slice of fewer elements
            for (int i = n + tid; i < k; i += TPR) keys[part * k + i] = 0;
          break;
        }
        settled<TPR>();
        bound = bound_[slot];
        by_chunk = false;
        if (tid == 0) ncand_[slot] = 0;
        settled<TPR>();
      }
    }
    if constexpr (WAVES > 1 || TOP == 2) settled<TPR>();  // this row's readers are done
  }
}

// The slices of a row joined, a block a row.
template <class T, int TOP>
__global__ __launch_bounds__(256) void logprobs_join_kernel(const T* __restrict__ z, const void* __restrict__ targets,
                                                            bool wide, int W, int V, int64_t ignore, int k, Out out,
                                                            int slices, const float* __restrict__ parts,
                                                            const uint64_t* __restrict__ keys) {
  __shared__ uint64_t cand[TOP ? JOIN_KEYS + PAD : 1];
  const int row = blockIdx.x, n = slices * k;  // (n <= JOIN_KEYS)
  Target target{0.0f, false, false};
  if (threadIdx.x == 0) target = target_of(z + (size_t)row * W, targets, wide, row, V, ignore);
  if constexpr (TOP > 0)
    for (int i = threadIdx.x; i < n + PAD; i += 256) cand[i] = i < n ? keys[(size_t)row * n + i] : 0;
  Sums a;
  for (int w = 0; w < slices; ++w) {
    const float* p = parts + 3 * ((size_t)row * slices + w);
    a.join(p[0], p[1], p[2]);
  }
  if (threadIdx.x == 0) write_row(out, row, a, target);
  if constexpr (TOP > 0) {
    __syncthreads();
    ranked<256>(cand, n, threadIdx.x, [&](uint64_t g, int rank) {
      if (g && rank < k) write_top(out, row, k, rank, g, a);
    });
  }
}

// The logits' gradient. TPR threads a piece of BACK chunks a thread; a row of W values is `pieces`
// of them. A thread requests all its chunks before it stores one (gz may be z, so the compiler would
// not); it writes the chunks that it has read.
constexpr int BACK = 4;
// A gradient that the 256 MB cache cannot hold for its reader is stored past the caches (8192 x 128000 in
// bfloat16: calls on changing inputs 814 -> 808 us, back to back 817 -> 773 to 811; chunks two or eight at
// a time are no faster, nor is a grid that stays).
constexpr size_t CACHE = (size_t)256 << 20;

template <class T, int TPR>
__global__ __launch_bounds__(256) void logprobs_bwd_kernel(const T* z, const void* __restrict__ targets, bool wide,
                                                           int M, int W, int V, int64_t ignore, int pieces,
                                                           const float* __restrict__ stats,
                                                           const float* __restrict__ entropy,
                                                           const float* __restrict__ g_logp,
                                                           const float* __restrict__ g_lse,
                                                           const float* __restrict__ g_ent, T* gz, bool past) {
  constexpr int CE = 16 / sizeof(T), PPB = 256 / TPR;
  const size_t units = (size_t)M * pieces;
  for (size_t u = (size_t)blockIdx.x * PPB + threadIdx.x / TPR; u < units; u += (size_t)gridDim.x * PPB) {
    const int row = pieces == 1 ? (int)u : (int)(u / pieces), piece = pieces == 1 ? 0 : (int)(u - (size_t)row * pieces);
    const Row<T> r(gz, (size_t)row * W, W);
    const T* in = z + (size_t)row * W;
    T* out = gz + (size_t)row * W;
    const bool same = (((uintptr_t)in ^ (uintptr_t)out) & 15) == 0;
    const int c0 = piece * BACK * TPR + (int)threadIdx.x % TPR;
    typename Row<T>::vec raw[BACK];
    if (same && r.w0 < r.w1) {  // (chunks that are not whole are read below)
#pragma unroll
      for (int b = 0; b < BACK; ++b)
        raw[b] = *reinterpret_cast<const typename Row<T>::vec*>(in + r.first(min(max(c0 + b * TPR, r.w0), r.w1 - 1)));
    }
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
    const float base = gl - g - (gh != 0.0f ? gh * entropy[row] : 0.0f);
    const int tj = t >= 0 && t < V ? (int)t : -1;
    // Without an entropy gradient a value is p * base, with p's exponent of two in two operations. (Not in
    // one: log2(e) (top + ls) as one float32 is off by 2^-24 of itself, which for a top of 10^5 is more
    // than a bfloat16 result's own rounding.)
    const bool plain = gh == 0.0f && !empty && near(top);
    const float m2 = top * LOG2E, l2 = fmaf(ls, LOG2E, rest(top));
#pragma unroll
    for (int b = 0; b < BACK; ++b) {
      const int c = c0 + b * TPR, j0 = r.first(c);
      if (c >= r.chunks) break;
      const bool whole = c >= r.w0 && c < r.w1;
      float v[CE];
      if (whole && same) {
#pragma unroll
        for (int j = 0; j < CE; ++j) v[j] = (float)raw[b][j];
      } else {
        r.part(in, c, 0.0f, v);
      }
      if (plain) {
#pragma unroll
        for (int j = 0; j < CE; ++j) v[j] = base * __builtin_amdgcn_exp2f(fmaf(v[j], LOG2E, -m2) - l2);
      } else {
#pragma unroll
        for (int j = 0; j < CE; ++j) {
          const float lp = v[j] - top - ls;
          const float p = empty ? 0.0f : exp_of(lp);
          v[j] = p * fmaf(-gh, fmaxf(lp, FAR), base);
        }
      }
      if (tj >= j0 && tj < j0 + CE) {
#pragma unroll
        for (int j = 0; j < CE; ++j) v[j] += j0 + j == tj ? g : 0.0f;
      }
      if (none || j0 + CE > V) {
#pragma unroll
        for (int j = 0; j < CE; ++j) v[j] = none || j0 + j >= V ? 0.0f : v[j];
      }
      if (whole) {
        if (past) store_row_nt<T, CE>(out + j0, v);
        else store_row<T, CE>(out + j0, v);
      } else {
#pragma unroll
        for (int j = 0; j < CE; ++j)
          if (j0 + j >= 0 && j0 + j < W) out[j0 + j] = from_f32<T>(v[j]);
      }
    }
  }
}

namespace {

// Slices of a row (1: not split): for few rows of many chunks, a block of 1024 threads for each
// compute unit, with at most 80 alternatives of a row to join. (Both launches, us, whole rows and 2, 4, 8, 16
// slices; * the rule's. float32, 128000: 1 row, k = 0 16.9 12.1 9.0 8.1 8.1*, k = 20 24.0 17.3 13.4* 13.1 17.2;
// 64 rows 19.6 14.7 11.5* 12.4 15.8, k = 20 27.2 19.8 16.8* 23.6 37.3; 128 rows 20.0 15.7* 16.5, 28.2 21.0* 27.3;
// 256 rows 22.7* 25.4. bfloat16, 32000: 1 row 6.0* 6.9 6.4 6.7, k = 5 9.9* 9.8 9.5 9.5; 64 rows 6.6* 7.8, 10.6*
// 10.7. Between, whole rows are not the best: 1 row of 65528 8.8* 8.3 7.1 7.0, k = 5 13.5* 11.5 10.2 10.2.)
int slices_of(bool bf16_io, int M, int V, int k) {
  const int chunks = V / (bf16_io ? 8 : 4);
  if (M > 128 || chunks < 8192) return 1;
  return std::max(1, std::min({MAX_SLICES, 256 / std::max(M, 1), chunks / 1024, 80 / std::max(k, 1)}));
}

struct Call {
  const void *z, *targets;
  bool wide;
  int M, W, V;
  int64_t ignore;
  int k;
  Out out;
  hipStream_t st;
};

// Steps of a row of `chunks` chunks at most (logprobs_kernel, TOP 2), and their bytes of LDS a block.
template <class T, int TPR, int TOP> int most_steps(int chunks) { return chunks / (step_chunks(TPR, 16 / sizeof(T), TOP) * TPR) + 1; }
template <int TPR, int TOP> size_t lds_bytes(int steps) { return TOP == 2 ? (size_t)steps * std::max(TPR, 256) * 2 : 0; }

template <class T, int TPR, int TOP> hipError_t run_fwd(const Call& c) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  const int steps = most_steps<T, TPR, TOP>(c.V / (16 / (int)sizeof(T)) + 2);
  hipLaunchKernelGGL((logprobs_kernel<T, TPR, TOP, false>), dim3(std::min((c.M + RPB - 1) / RPB, 1 << 20)),
                     dim3(TPR < 256 ? 256 : TPR), (lds_bytes<TPR, TOP>(steps)), c.st, (const T*)c.z, c.targets, c.wide,
                     c.M, c.W, c.V, c.ignore, c.k, c.out, 1, nullptr, nullptr, steps);
  return hipGetLastError();
}

template <class T, int TOP> hipError_t run_top(const Call& c, void* ws) {
  const int slices = slices_of(sizeof(T) == 2, c.M, c.V, c.k), chunks = c.V / (16 / (int)sizeof(T));
  if (slices > 1) {
    uint64_t* keys = (uint64_t*)ws;
    float* parts = (float*)(keys + (size_t)c.M * slices * c.k);
    const int steps = most_steps<T, 1024, TOP>((chunks + 2) / slices + 1);
    hipLaunchKernelGGL((logprobs_kernel<T, 1024, TOP, true>), dim3(c.M * slices), dim3(1024), (lds_bytes<1024, TOP>(steps)),
                       c.st, (const T*)c.z, c.targets, c.wide, c.M, c.W, c.V, c.ignore, c.k, c.out, slices, parts, keys,
                       steps);
    hipLaunchKernelGGL((logprobs_join_kernel<T, TOP>), dim3(c.M), dim3(256), 0, c.st, (const T*)c.z, c.targets, c.wide,
                       c.W, c.V, c.ignore, c.k, c.out, slices, parts, keys);
    return hipGetLastError();
  }
  if constexpr (TOP < 2)
    if (chunks <= 128) return run_fwd<T, 16, TOP>(c);
  // A wave a row has no barriers, a block a row fewer rows at a time. (Calls, 256 threads and a wave: 16384 x
  // 8000 in bfloat16 66 and 51 us, with k = 5 127 and 71; 16384 x 16000 95 and 97, 156 and 118; 4096 x 30522
  // 51 and 50, 74 and 61; 4096 x 64000 91 and 94, 104 and 130. With 1024 rows of 30522 14 and 16, 23 and 26.)
  if (chunks <= (c.M < 2048 ? 512 : TOP == 2 ? 4096 : 1024)) return run_fwd<T, 64, TOP>(c);
  if (chunks < 1024 || c.M > 256) return run_fwd<T, 256, TOP>(c);
  return run_fwd<T, 1024, TOP>(c);
}

template <class T> hipError_t run_any(const Call& c, void* ws) {
  return c.k == 0 ? run_top<T, 0>(c, ws) : c.k == 1 ? run_top<T, 1>(c, ws) : run_top<T, 2>(c, ws);
}

template <class T, int TPR>
hipError_t run_bwd(const void* z, const void* targets, bool wide, int M, int W, int V, int64_t ignore,
                   const float* stats, const float* entropy, const float* g_logp, const float* g_lse,
                   const float* g_ent, void* gz, hipStream_t st) {
  // (a row touches at most one chunk more than it fills)
  const int chunks = W / (16 / (int)sizeof(T)) + 2, pieces = (chunks + BACK * TPR - 1) / (BACK * TPR);
  const size_t blocks = ((size_t)M * pieces + 256 / TPR - 1) / (256 / TPR);
  hipLaunchKernelGGL((logprobs_bwd_kernel<T, TPR>), dim3((unsigned)std::min<size_t>(blocks, 1 << 20)), dim3(256), 0, st,
                     (const T*)z, targets, wide, M, W, V, ignore, pieces, stats, entropy, g_logp, g_lse, g_ent, (T*)gz,
                     (size_t)M * W * sizeof(T) > CACHE);
  return hipGetLastError();
}

}  // namespace

size_t logprobs_fwd_bytes(bool bf16_io, int M, int V, int k) {
  const size_t s = slices_of(bf16_io, M, V, k);
  return s > 1 ? (size_t)M * s * (8 * k + 12) : 0;
}

hipError_t launch_logprobs_fwd(bool bf16_io, const void* z, const void* targets, bool wide, int M, int W, int V,
                               int64_t ignore, int k, float* logp, float* lse, float* entropy, float* stats,
                               float* top_logp, int64_t* top_index, void* ws, hipStream_t st) {
  const Call c{z, targets, wide, M, W, V, ignore, k, Out{logp, lse, entropy, stats, top_logp, top_index}, st};
  return bf16_io ? run_any<bf16>(c, ws) : run_any<float>(c, ws);
}

hipError_t launch_logprobs_bwd(bool bf16_io, const void* z, const void* targets, bool wide, int M, int W, int V,
                               int64_t ignore, const float* stats, const float* entropy, const float* g_logp,
                               const float* g_lse, const float* g_ent, void* gz, hipStream_t st) {
#define BWD(T, TPR) run_bwd<T, TPR>(z, targets, wide, M, W, V, ignore, stats, entropy, g_logp, g_lse, g_ent, gz, st)
  if (bf16_io) return W < 64 * BACK * 8 ? BWD(bf16, 64) : BWD(bf16, 256);
  return W < 64 * BACK * 4 ? BWD(float, 64) : BWD(float, 256);
#undef BWD
}

}  // namespace instant
