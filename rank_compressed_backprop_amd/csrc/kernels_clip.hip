// The norm over many tensors, and the tensors scaled by what it allows (include/instant_ops.h):
//   n = (sum_i sum_j g_ij^2)^(1/2);  out_ij = c g_ij, c = 1 if n + 1e-6 <= max, else max / (n + 1e-6)
//
// Squares are added in float64: a float32 square is out of range for values beyond 2^64 or below
// 2^-75, which bfloat16 gradients reach. Every block leaves one partial sum, and the partial sums
// are added in a fixed order, so the norm has the same bits every time.
//
// The tensors travel as the launch's arguments, TENSORS a launch: nothing is copied to the device,
// so a captured graph holds them and no buffer has to outlive the call.
#include <algorithm>
#include <cmath>

#include "ops.hpp"

namespace instant {

namespace {

constexpr int TENSORS = 120;      // a launch (of the 4 KB of arguments)
constexpr int PIECE = 1 << 15;    // elements that a block takes at a time
constexpr int GRID = 2048;        // blocks a launch at most
constexpr float EPS = 1e-6f;

struct Table {
  const void* src[TENSORS];
  void* dst[TENSORS];
  int64_t count[TENSORS];
  uint32_t end[TENSORS];    // pieces of the tensors up to and with this one
  uint8_t bf[TENSORS];      // bit 0: src is bfloat16, bit 1: dst is
  int n;
};

// The tensor of piece p, and the piece's first element.
__device__ __forceinline__ int find(const Table& t, uint32_t p, int64_t& first) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (p < t.end[mid]) hi = mid;
    else lo = mid + 1;
  }
  first = (int64_t)(p - (lo ? t.end[lo - 1] : 0)) * PIECE;
  return lo;
}

template <class T> __device__ __forceinline__ bool aligned8(const T* p) {
  return ((uintptr_t)p & 15) == 0;
}

// f(index, values, how many) over the elements [0, n) of p by the block's 256 threads: eight at a
// time where p + index lies on a 16-byte border, one at a time at the ends.
template <class T, class F> __device__ __forceinline__ void over(const T* p, int n, F&& f) {
  const int head = min(n, (int)((16 - ((uintptr_t)p & 15)) % 16 / sizeof(T)));
  const int whole = (n - head) / 8;
  for (int i = threadIdx.x; i < whole; i += 256) {
    float v[8];
    load8(p + head + 8 * i, v);
    f(head + 8 * i, v, std::integral_constant<int, 8>{});
  }
  const int tail = n - head - 8 * whole;
  const int i = (int)threadIdx.x < head ? (int)threadIdx.x : head + 8 * whole + ((int)threadIdx.x - head);
  if ((int)threadIdx.x < head + tail) {
    const float v[1] = {(float)p[i]};
    f(i, v, std::integral_constant<int, 1>{});
  }
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if (threadIdx.x % WAVE == 0) lds[threadIdx.x / WAVE] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < (int)blockDim.x / WAVE; ++i) v += lds[i];
  return v;
}

}  // namespace

__global__ __launch_bounds__(256) void square_sum_kernel(Table t, uint32_t pieces, double* __restrict__ part) {
  __shared__ double lds[4];
  double sum = 0.0;
  auto add = [&](int, const float* v, auto n) {
#pragma unroll
    for (int j = 0; j < decltype(n)::value; ++j) sum = fma((double)v[j], (double)v[j], sum);
  };
  for (uint32_t p = blockIdx.x; p < pieces; p += gridDim.x) {
    int64_t first;
    const int i = find(t, p, first);
    const int n = (int)min((int64_t)PIECE, t.count[i] - first);
    if (t.bf[i] & 1) over((const bf16*)t.src[i] + first, n, add);
    else over((const float*)t.src[i] + first, n, add);
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

namespace {

// The norm from the partial sums, by a block of 256 threads: every block's is the same.
__device__ __forceinline__ float norm_of(const double* part, int n) {
  __shared__ double lds[4];
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) sum += part[i];
  return (float)sqrt(block_sum(sum, lds));
}

// NaN stays NaN; an infinite norm gives 0.
__device__ __forceinline__ float factor_of(float norm, float max_norm) {
  return norm + EPS <= max_norm ? 1.0f : max_norm / (norm + EPS);
}

}  // namespace

__global__ __launch_bounds__(256) void norm_kernel(const double* __restrict__ part, int n, float* __restrict__ norm) {
  const float v = norm_of(part, n);
  if (threadIdx.x == 0) *norm = v;
}

namespace {

template <class S, class D>
__device__ __forceinline__ void scale_piece(const S* src, D* dst, int n, float c) {
  if (c == 1.0f && (const void*)src == (const void*)dst) return;
  const bool wide = [&] {  // where src lies on a border, so does dst
    const int head = (int)((16 - ((uintptr_t)src & 15)) % 16 / sizeof(S));
    return aligned8(dst + head);
  }();
  over(src, n, [&](int i, const float* v, auto k) {
    constexpr int K = decltype(k)::value;
    float o[K];
#pragma unroll
    for (int j = 0; j < K; ++j) o[j] = v[j] * c;
    if constexpr (K == 8) {
      if (wide) {
        store_row<D, 8>(dst + i, o);
        return;
      }
    }
#pragma unroll
    for (int j = 0; j < K; ++j) dst[i + j] = from_f32<D>(o[j]);
  });
}

}  // namespace

// parts > 0: the norm from the partial sums (which a launch of its own would take 7 us for), which block 0
// leaves at norm; else it is there. From the last piece to the first: the last ones' gradients are in the
// cache.
__global__ __launch_bounds__(256) void scale_kernel(Table t, uint32_t pieces, const double* __restrict__ part,
                                                    int parts, float max_norm, float* norm) {
  const float v = parts ? norm_of(part, parts) : *norm;
  if (parts && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  const float c = factor_of(v, max_norm);
  for (uint32_t k = blockIdx.x; k < pieces; k += gridDim.x) {
    int64_t first;
    const int i = find(t, pieces - 1 - k, first);
    const int n = (int)min((int64_t)PIECE, t.count[i] - first);
    const bf16* sb = (const bf16*)t.src[i] + first;
    const float* sf = (const float*)t.src[i] + first;
    bf16* db = (bf16*)t.dst[i] + first;
    float* df = (float*)t.dst[i] + first;
    switch (t.bf[i]) {
      case 0: scale_piece(sf, df, n, c); break;
      case 1: scale_piece(sb, df, n, c); break;
      case 2: scale_piece(sf, db, n, c); break;
      case 3: scale_piece(sb, db, n, c); break;
    }
  }
}

namespace {

int launches(int n) { return (n + TENSORS - 1) / TENSORS; }

// Tensors [first, ...) of a launch; its pieces (at most 2^40 / PIECE for each: 32 bits hold them).
uint32_t fill(Table& t, const void* const* src, void* const* dst, const int64_t* count, const int32_t* bf,
              const int32_t* dst_bf, int first, int n) {
  t.n = std::min(TENSORS, n - first);
  uint32_t pieces = 0;
  for (int i = 0; i < t.n; ++i) {
    const int k = first + i;
    t.src[i] = src[k];
    t.dst[i] = dst ? dst[k] : nullptr;
    t.count[i] = count[k];
    pieces += (uint32_t)((count[k] + PIECE - 1) / PIECE);
    t.end[i] = pieces;
    t.bf[i] = (uint8_t)((bf[k] ? 1 : 0) | (dst && dst_bf[k] ? 2 : 0));
  }
  return pieces;
}
static_assert((((int64_t)1 << 40) / PIECE) * TENSORS < (int64_t)1 << 32, "pieces");

// The partial sums of all tensors, and how many.
int square_sums(const void* const* src, const int64_t* count, const int32_t* bf, int n, double* part, hipStream_t st) {
  int parts = 0;
  for (int k = 0; k < n; k += TENSORS) {
    Table t;
    const uint32_t pieces = fill(t, src, nullptr, count, bf, nullptr, k, n);
    const int grid = (int)std::min<uint32_t>(pieces, GRID);
    if (!grid) continue;
    hipLaunchKernelGGL(square_sum_kernel, dim3(grid), dim3(256), 0, st, t, pieces, part + parts);
    parts += grid;
  }
  return parts;
}

}  // namespace

size_t grad_norm_bytes(int n) { return std::max<size_t>(1, launches(n)) * GRID * sizeof(double); }

hipError_t launch_grad_norm(const void* const* src, const int64_t* count, const int32_t* bf, int n, float* norm,
                            void* ws, hipStream_t st) {
  const int parts = square_sums(src, count, bf, n, (double*)ws, st);
  hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(256), 0, st, (const double*)ws, parts, norm);
  return hipGetLastError();
}

hipError_t launch_clip_grads(const void* const* src, const int64_t* count, const int32_t* bf, void* const* dst,
                             const int32_t* dst_bf, int n, float max_norm, float* norm, void* ws, hipStream_t st) {
  int parts = square_sums(src, count, bf, n, (double*)ws, st);
  if (n > TENSORS || !parts) {  // (several launches scale; or none)
    hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(256), 0, st, (const double*)ws, parts, norm);
    parts = 0;
  }
  for (int k = 0; k < n; k += TENSORS) {
    Table t;
    const uint32_t pieces = fill(t, src, dst, count, bf, dst_bf, k, n);
    if (!pieces) continue;
    hipLaunchKernelGGL(scale_kernel, dim3(std::min<uint32_t>(pieces, GRID)), dim3(256), 0, st, t, pieces,
                       (const double*)ws, parts, max_norm, norm);
  }
  return hipGetLastError();
}

}  // namespace instant
