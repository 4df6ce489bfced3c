// The three products of a linear layer in bfloat16 on the matrix cores (the layouts and the
// orientation are those of kernels_linear.hip; bf16 products are exact in the float32 sums).
//
// Four waves share a block tile of BM x BN, one to a SIMD, so a wave tile is up to 128 x 128:
// every operand byte read from LDS then feeds 128 products, and the LDS reads of a stage (64 k)
// take half the matrix cores' time (a wave tile of 64 x 64 would take all of it).
//
// A stage goes from memory straight to LDS (16 bytes a lane); two stages are held. A wave runs
// two half stages of 32 k by turns from two sets of operand registers:
//   multiply half 0 of stage s   while half 1 of s is read from LDS
//   wait for stage s + 1, barrier: every wave has read all of s
//   multiply half 1 of stage s   while half 0 of s + 1 is read and stage s + 2 is requested
//                                into the slot of s
// so the matrix cores always have operands in registers, and a request has the time of a whole
// stage to arrive. The reads and requests are dealt out between the products by hand.
//
// Rows (columns) of a tile that lie outside the operand are read from its last row (column
// chunk) instead: they only reach outputs that are not stored. Behind the contraction's end the
// last k is read again, and its place in LDS cleared by the lane that read it. Past the last
// stage the last one is requested again, so the loop has no branch around its products (with
// one, the compiler copies the 256 accumulators).
#include <algorithm>
#include <utility>

#include "dma.hpp"
#include "lds_tiles.hpp"
#include "ops.hpp"
#include "tile16.hpp"

namespace instant {

namespace {

constexpr int K16 = 64;  // k per stage

// f(0) .. f(N - 1) with constant arguments: register arrays are indexed by constants whatever
// the size of the body
template <int... I, class F> __device__ __forceinline__ void each(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F> __device__ __forceinline__ void each(F&& f) {
  each(std::make_integer_sequence<int, N>{}, f);
}

// 16 bytes per lane from base + off (base uniform) straight into LDS at lds_wave + 16 * lane.
__device__ __forceinline__ void lds_dma16_at(const void* base, unsigned off, void* lds_wave) {
  const unsigned lds = (unsigned)(uintptr_t)(__attribute__((address_space(3))) void*)lds_wave;
  __asm__ volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}

__device__ __forceinline__ void keep_in_agprs(f32x4& v) {
#ifdef __HIP_DEVICE_COMPILE__
  __asm__ volatile("" : "+a"(v));
#endif
}

// One operand of a block tile: W rows (columns of the k-major layout) of a stage in LDS.
//   k contiguous: W rows of 128 bytes; chunk c (16 bytes) of row r at c ^ (r & 7)
//   k-major     : 64 k rows of 2 W bytes; chunk c of row r at c ^ swizzle(r)
// PAIR: the operand of the first slot (columns n). In the k-contiguous layout LDS row
// 32 p + 16 hh + i holds operand row 32 p + 8 (i / 4) + 4 hh + i % 4, so its reads are those of
// the other operand; the k-major layout permutes as it is read (lds_tiles.hpp).
template <bool KMAJ, bool PAIR, int W>
struct Side {
  static constexpr int BYTES = W * K16 * 2;
  static constexpr int LOADS = BYTES / 4096;  // of 1024 bytes, for each of the four waves
  static constexpr int CPR = KMAJ ? W / 8 : 8;  // chunks a row
  // k contiguous: byte offsets of this lane's rows; k-major: of its column chunks
  unsigned off[LOADS];
  unsigned kb;  // bytes of one k row (k-major)
  int chunk;    // k contiguous: the logical chunk of all its loads (their rows differ by 32s)
  unsigned at;  // and its offset in the stage being requested

  __device__ static __forceinline__ int swz(int r) {
    if constexpr (!KMAJ) return r & 7;
    const int flip = W % 128 ? 7 : 15;  // (the flip of chunk bit 3 needs rows of whole 16 chunks)
    return (PAIR ? kswz_b(r) : kswz_a(r)) & flip;
  }
  // LDS row and logical chunk of this lane's load j
  __device__ static __forceinline__ void place(int j, int wave, int lane, int& r, int& c) {
    const int id = (j * 4 + wave) * 64 + lane;
    r = id / CPR;
    c = (id % CPR) ^ swz(r);
  }
  __device__ static __forceinline__ int row_of(int r) {
    if constexpr (!PAIR) return r;
    return (r & ~31) + 8 * ((r & 15) >> 2) + 4 * ((r >> 4) & 1) + (r & 3);
  }

  __device__ __forceinline__ void init(int first, int rows, int ld, int wave, int lane) {
    kb = 2u * (unsigned)ld;
    chunk = (lane & 7) ^ ((lane >> 3) & 7);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      int r, c;
      place(j, wave, lane, r, c);
      if constexpr (KMAJ) off[j] = 2u * (unsigned)min(8 * c, rows - 8 - first);  // rows % 8 == 0
      else off[j] = (unsigned)min(row_of(r), rows - 1 - first) * kb;
    }
  }
  // the tile's first element at stage k0
  __device__ static __forceinline__ const bf16* origin(const bf16* p, int first, int ld, int k0) {
    return KMAJ ? p + (size_t)k0 * ld + first : p + (size_t)first * ld + k0;
  }
  // a stage of which `left` >= 1 k are there (64 or more: all of it; k contiguous: a multiple of
  // 8) is requested next
  __device__ __forceinline__ void stage(int left) {
    if constexpr (!KMAJ) at = 16u * (unsigned)min(chunk, (left >> 3) - 1);
  }
  // load j of the stage at `base`
  __device__ __forceinline__ void issue(int j, const bf16* base, int left, unsigned char* lds, int wave, int lane) const {
    unsigned o = at + off[j];
    if constexpr (KMAJ) {
      int r, c;
      place(j, wave, lane, r, c);
      o = __umul24((unsigned)min(r, left - 1), kb) + off[j];  // (kb < 2^20)
    }
    lds_dma16_at(base, o, lds + 1024 * (j * 4 + wave));
  }
  // clears this lane's chunks behind the last of `left` k
  __device__ __forceinline__ void clear(int left, unsigned char* lds, int wave, int lane) const {
    each<LOADS>([&](auto j) {
      int r, c;
      place(j, wave, lane, r, c);
      if (KMAJ ? r >= left : 8 * chunk >= left)
        *reinterpret_cast<f32x4*>(lds + 1024 * (j * 4 + wave) + 16 * lane) = zero4();
    });
  }
  // the MFMA operand of 16-row tile `t` (first row 16 t of the tile) and k half h
  __device__ static __forceinline__ bf16x8 frag(const unsigned char* lds, int t, int h, int lane) {
    if constexpr (!KMAJ) {
      const int r = 16 * t + (lane & 15);
      return *reinterpret_cast<const bf16x8*>(lds + r * 128 + 16 * ((4 * h + (lane >> 4)) ^ (r & 7)));
    } else {
      const int q = lane >> 4, s = lane & 15, a = s & 3;
      const int col0 = PAIR ? 32 * (t >> 1) : 16 * t;
      const int col = PAIR ? col0 + 8 * a + 4 * ((t & 1) ^ (a & 1)) : col0 + 4 * a;
      const int r0 = 32 * h + 8 * q + (s >> 2);  // and row r0 + 4, which has the same swizzle
      const unsigned char* p = lds + r0 * (2 * W) + 16 * ((col >> 3) ^ swz(r0)) + (col & 7) * 2;
      const bf16x4 lo = tr_read(p), hi = tr_read(p + 8 * W);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

}  // namespace

// C(m, n) = sum_k A(m, k) B(n, k) over k slice blockIdx.z. WM x WN: 16-row tiles of a wave
// (WN even); the waves form a 2 x 2 grid. Grid (tiles, 1, S).
template <bool AKM, bool BKM, int WM, int WN, bool PART>
__global__ __launch_bounds__(256, 1) void tile16_kernel(const bf16* __restrict__ A, int lda, int M,
                                                        const bf16* __restrict__ B, int ldb, int N, int K, Epi ep,
                                                        float* __restrict__ part) {
  constexpr int BM = 32 * WM, BN = 32 * WN;
  typedef Side<AKM, false, BM> SA;
  typedef Side<BKM, true, BN> SB;
  constexpr int STAGE = SA::BYTES + SB::BYTES;
  __shared__ __attribute__((aligned(1024))) unsigned char ring[2][STAGE];
  const int lane = threadIdx.x & (WAVE - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int mt = (M + BM - 1) / BM, nt = (N + BN - 1) / BN;
  int tm, tn;
  tile_of(xcd_unit(blockIdx.x, mt * nt), mt, nt, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int nst = (K + K16 - 1) / K16, S = gridDim.z, z = blockIdx.z;
  const int s0 = (int)((long)nst * z / S), nq = (int)((long)nst * (z + 1) / S) - s0;
  const int wm = wave >> 1, wn = wave & 1;

  SA sa;
  SB sb;
  sa.init(m0, M, lda, wave, lane);
  sb.init(n0, N, ldb, wave, lane);
  // the next stage to request
  const bf16* pa = SA::origin(A, m0, lda, s0 * K16);
  const bf16* pb = SB::origin(B, n0, ldb, s0 * K16);
  const size_t da = AKM ? (size_t)K16 * lda : K16, db = BKM ? (size_t)K16 * ldb : K16;
  // k from that stage to the slice's end
  int left = min(K, (s0 + nq) * K16) - s0 * K16;
  const int tail = (left - 1) % K16 + 1;  // k of the slice's last stage
  sa.stage(left);
  sb.stage(left);
  constexpr int NDMA = SA::LOADS + SB::LOADS;
  auto request = [&](int j, unsigned char* st) {
    if (j < SA::LOADS) sa.issue(j, pa, left, st, wave, lane);
    else sb.issue(j - SA::LOADS, pb, left, st + SA::BYTES, wave, lane);
  };
  auto advance = [&] {  // (the last stage stays)
    const bool more = left > K16;
    pa += more ? da : 0;
    pb += more ? db : 0;
    left -= more ? K16 : 0;
    sa.stage(left);
    sb.stage(left);
  };

  f32x4 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j) acc[i][j] = zero4();
  bf16x8 fa[2][WM], fb[2][WN];
  constexpr int NREAD = WM + WN, NMMA = WM * WN;
  auto read = [&](auto r, auto set, const unsigned char* st) {  // operand r of half `set`
    if constexpr (r < WN) fb[set][r] = SB::frag(st + SA::BYTES, WN * wn + r, set, lane);
    else fa[set][r - WN] = SA::frag(st, WM * wm + r - WN, set, lane);
  };
  // The products of one half, with the reads of operand set `to` from st and (DMA) the requests
  // into slot dealt out over the first three quarters of them.
  auto half = [&](auto set, auto to, auto dma, const unsigned char* st, unsigned char* slot) {
    each<NMMA>([&](auto t) {
      acc[t / WN][t % WN] = MM<bf16>::mma(fb[set][t % WN], fa[set][t / WN], acc[t / WN][t % WN]);
      each<NREAD>([&](auto r) {
        if constexpr (r * (NMMA * 3 / 4) / NREAD == t) {
          read(r, to, st);
          __builtin_amdgcn_sched_barrier(0);
        }
      });
      if constexpr (decltype(dma)::value)
        each<NDMA>([&](auto j) {
          if constexpr (j * (NMMA * 3 / 4) / NDMA == t) {
            request(j, slot);
            __builtin_amdgcn_sched_barrier(0);
          }
        });
    });
  };
  // stage s has arrived for this wave: clear what lies behind the contraction's end
  auto arrived = [&](int s, unsigned char* st) {
    if (tail < K16 && s == nq - 1) {
      sa.clear(tail, st, wave, lane);
      sb.clear(tail, st + SA::BYTES, wave, lane);
      __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  };
  constexpr std::integral_constant<int, 0> h0{};
  constexpr std::integral_constant<int, 1> h1{};

#pragma unroll 1
  for (int q = 0; q < 2; ++q) {
    each<NDMA>([&](auto j) { request(j, ring[q]); });
    advance();
  }
  wait_vmcnt<NDMA>();
  arrived(0, ring[0]);
  bare_barrier();
  each<NREAD>([&](auto r) { read(r, h0, ring[0]); });

#pragma unroll 1
  for (int s = 0; s < nq; ++s) {
    unsigned char* cur = ring[s & 1];
    unsigned char* nxt = ring[(s & 1) ^ 1];
    half(h0, h1, std::false_type{}, cur, nullptr);
    wait_vmcnt<0>();  // stage s + 1 is here, and this wave's reads of s are done
    arrived(s + 1, nxt);
    bare_barrier();
    // (after the last stage what is read and requested goes unused)
    half(h1, h0, std::true_type{}, nxt, cur);
    advance();
  }
  wait_vmcnt<0>();  // nothing may land in LDS after this block's end
  // the sums stay in accumulation registers up to here (left to itself, the compiler moves them
  // to and fro inside the loop for the epilogue's sake: 1.6 times the loop's time)
  each<WM>([&](auto i) { each<WN>([&](auto j) { keep_in_agprs(acc[i][j]); }); });

  const int q4 = lane >> 4, l16 = lane & 15;
  each<WM>([&](auto i) {
    const int m = m0 + 16 * (WM * wm + i) + l16;
    each<WN / 2>([&](auto p) {
      const int n = n0 + 16 * WN * wn + 32 * p + 8 * q4;
      const bool in = m < M && n < N;
      // the k-major layout's halves alternate: this lane's first four columns are in tile
      // q4 % 2 of the pair (lds_tiles.hpp)
      const bool sw = BKM && (q4 & 1);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = acc[i][2 * p][j], b = acc[i][2 * p + 1][j];
        v[j] = sw ? b : a;
        v[4 + j] = sw ? a : b;
      }
      if constexpr (PART) {
        if (in) store_row<float, 8>(part + ((size_t)z * M + m) * N + n, v);
      } else {
        epilogue8<bf16, 16, 32>(ep, v, m, n, N, in);
      }
    });
  });
}

namespace {

template <bool AKM, bool BKM, int WM, int WN>
hipError_t go16(const bf16* A, int lda, int M, const bf16* B, int ldb, int N, int K, const Epi& ep, int S, float* part,
                hipStream_t st) {
  const unsigned tiles = (unsigned)((M + 32 * WM - 1) / (32 * WM)) * ((N + 32 * WN - 1) / (32 * WN));
  if (S > 1)
    hipLaunchKernelGGL((tile16_kernel<AKM, BKM, WM, WN, true>), dim3(tiles, 1, S), dim3(256), 0, st, A, lda, M, B, ldb,
                       N, K, ep, part);
  else
    hipLaunchKernelGGL((tile16_kernel<AKM, BKM, WM, WN, false>), dim3(tiles), dim3(256), 0, st, A, lda, M, B, ldb, N, K,
                       ep, part);
  return hipGetLastError();
}

}  // namespace

Plan16 plan16(int M, int N, int K) {
  // rounds of blocks over the 256 compute units times a block's time, which goes with its area
  // (and a floor for its operands' stages)
  static const int shapes[][2] = {{8, 8}, {8, 6}, {8, 4}, {4, 4}};
  Plan16 best{0, 0, 1};
  double least = 0;
  for (const auto& s : shapes) {
    const int bm = 32 * s[0], bn = 32 * s[1];
    const long tiles = (long)((M + bm - 1) / bm) * ((N + bn - 1) / bn);
    const int per_cu = s[0] == 4 ? 2 : 1;  // blocks that share a compute unit
    const double rounds = (double)((tiles + 256 * per_cu - 1) / (256 * per_cu)) * per_cu;
    const double cost = rounds * (bm * bn + 24.0 * (bm + bn));
    if (!best.wm || cost < least) {
      best = Plan16{s[0], s[1], 1};
      least = cost;
    }
  }
  const long tiles = (long)((M + 32 * best.wm - 1) / (32 * best.wm)) * ((N + 32 * best.wn - 1) / (32 * best.wn));
  const int nst = (K + K16 - 1) / K16;
  while (tiles * best.S * 2 <= 512 && best.S < 16 && nst / (2 * best.S) >= 4) best.S *= 2;
  return best;
}

hipError_t launch_tile16(bool akm, bool bkm, const void* A, int lda, int M, const void* B, int ldb, int N, int K,
                         const Epi& ep, float* part, hipStream_t st) {
  const Plan16 p = plan16(M, N, K);
#define GO(AK, BK, WM, WN) go16<AK, BK, WM, WN>((const bf16*)A, lda, M, (const bf16*)B, ldb, N, K, ep, p.S, part, st)
#define GO_SHAPE(AK, BK)                                                                                        \
  (p.wm == 4 ? GO(AK, BK, 4, 4) : p.wn == 8 ? GO(AK, BK, 8, 8) : p.wn == 6 ? GO(AK, BK, 8, 6) : GO(AK, BK, 8, 4))
  return akm ? GO_SHAPE(true, true) : bkm ? GO_SHAPE(false, true) : GO_SHAPE(false, false);
#undef GO_SHAPE
#undef GO
}

}  // namespace instant
