// The three products of a linear layer on the matrix cores, in bfloat16 (products exact, sums
// float32) or float32 (v_mfma_f32_16x16x4_f32):
//   fwd  y  [M][N]: A = x  [M][K] (k contiguous), B = w [N][K] (k contiguous)
//   gx   gx [M][K]: A = gz [M][N] (k contiguous), B = w [N][K] (k-major: the contraction is N)
//   gw   gw [N][K]: A = gz [M][N] (k-major: the contraction is M), B = x [M][K] (k-major)
//
// Orientation: the MFMA computes D[n][m] (the B operand takes the first slot). A lane receives
// D rows 4 q + v (q = lane / 16, v < 4) of column m = lane % 16.
//
// Four waves share a block tile of BM x BN, one to a SIMD, so a wave tile is up to 128 x 128:
// every operand byte read from LDS then feeds 128 products, and the LDS reads of a stage (128
// bytes of k: 64 bfloat16 or 32 float32)
// take half the matrix cores' time in bfloat16 (a wave tile of 64 x 64 would take all of it; in
// float32, at an eighth of the rate, LDS never matters).
//
// A stage goes from memory straight to LDS (16 bytes a lane); NS stages are held. A wave runs
// two half stages by turns from two sets of operand registers:
//   multiply half 0 of stage s   while half 1 of s is read from LDS
//   wait for stage s + 1, barrier: every wave has read all of s
//   multiply half 1 of stage s   while half 0 of s + 1 is read and stage s + NS is requested
//                                into the slot of s
// so the matrix cores always have operands in registers, and a request has the time of NS - 1
// stages to arrive. The reads and requests are dealt out between the products by hand.
//
// Rows (columns) of a tile that lie outside the operand are read from its last row (column
// chunk) instead: they only reach outputs that are not stored. Behind the contraction's end the
// last k is read again, and its place in LDS cleared by the lane that read it. Past the last
// stage the last one is requested again, so the loop has no branch around its products (with
// one, the compiler copies the 256 accumulators).
#pragma once

#include "dma.hpp"
#include "lds_tiles.hpp"
#include "ops.hpp"
#include "tile.hpp"

namespace instant {

namespace {

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

// One operand of a block tile: W rows (columns of the k-major layout) of a stage in LDS, in
// chunks of 16 bytes.
//   k contiguous: W rows of 128 bytes; chunk c of row r at c ^ (r & 7)
//   k-major     : KS k rows of W elements; chunk c of row r at c ^ swizzle(r)
// PAIR: the operand of the first slot (columns n): its 16-row tiles 2 p and 2 p + 1 hold the 32
// columns of pair p so that a lane receives 8 consecutive ones, row i of tile hh being column
// 8 (i / 4) + 4 hh + i % 4 of the pair. In the k-contiguous layout LDS row 32 p + 16 hh + i holds
// that operand row, so its reads are those of the other operand; the k-major layout permutes as
// it is read (bfloat16: lds_tiles.hpp, whose halves alternate).
template <class T, bool KMAJ, bool PAIR, int W>
struct Side {
  typedef typename MM<T>::frag frag;
  static constexpr int ES = sizeof(T), CE = 16 / ES;  // bytes of an element, elements of a chunk
  static constexpr int KS = 128 / ES;                 // k per stage
  static constexpr int BYTES = W * 128;
  static constexpr int LOADS = BYTES / 4096;  // of 1024 bytes, for each of the four waves
  static constexpr int CPR = KMAJ ? W / CE : 8;  // chunks a row
  static_assert(W % 32 == 0 && (!PAIR || W % 64 == 0), "the swizzles stay within a row");
  // k contiguous: byte offsets of this lane's rows; k-major: of its column chunks
  unsigned off[LOADS];
  unsigned kb;  // bytes between stored rows
  int chunk;    // k contiguous: the logical chunk of all its loads (their rows differ by 32s)
  unsigned at;  // and its offset in the stage being requested

  __device__ static __forceinline__ int swz(int r) {
    if constexpr (!KMAJ) {
      return r & 7;
    } else if constexpr (ES == 2) {
      // (a flip of a chunk bit needs rows of whole powers of two of chunks above it)
      constexpr int flip = W % 128 == 0 ? 15 : W % 64 == 0 ? 7 : 3;
      return (PAIR ? kswz_b(r) : kswz_a(r)) & flip;
    } else {
      // a read takes 16 columns of rows 4 q + g, q < 4: rows of odd q use the banks that those of
      // even q leave (PAIR: every other chunk of eight; else four chunks side by side)
      return ((r >> 2) & 1) * (PAIR ? 1 : 4);
    }
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
    kb = ES * (unsigned)ld;
    chunk = (lane & 7) ^ ((lane >> 3) & 7);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      int r, c;
      place(j, wave, lane, r, c);
      if constexpr (KMAJ) off[j] = ES * (unsigned)min(CE * c, rows - CE - first);  // rows % 8 == 0
      else off[j] = (unsigned)min(row_of(r), rows - 1 - first) * kb;
    }
  }
  // the tile's first element at stage k0
  __device__ static __forceinline__ const T* origin(const T* p, int first, int ld, int k0) {
    return KMAJ ? p + (size_t)k0 * ld + first : p + (size_t)first * ld + k0;
  }
  // a stage of which `left` >= 1 k are there (KS or more: all of it; k contiguous: a multiple of
  // 8) is requested next
  __device__ __forceinline__ void stage(int left) {
    if constexpr (!KMAJ) at = 16u * (unsigned)min(chunk, left / CE - 1);
  }
  // load j of the stage at `base`
  __device__ __forceinline__ void issue(int j, const T* base, int left, unsigned char* lds, int wave, int lane) const {
    unsigned o = at + off[j];
    if constexpr (KMAJ) {
      int r, c;
      place(j, wave, lane, r, c);
      o = __umul24((unsigned)min(r, left - 1), kb) + off[j];  // (kb <= 2^20)
    }
    lds_dma16_at(base, o, lds + 1024 * (j * 4 + wave));
  }
  // clears this lane's chunks behind the last of `left` k
  __device__ __forceinline__ void clear(int left, unsigned char* lds, int wave, int lane) const {
    each<LOADS>([&](auto j) {
      int r, c;
      place(j, wave, lane, r, c);
      if (KMAJ ? r >= left : CE * chunk >= left)
        *reinterpret_cast<f32x4*>(lds + 1024 * (j * 4 + wave) + 16 * lane) = zero4();
    });
  }
  // LDS reads that make one MFMA operand (16 bytes: the k of one k-step that the lane supplies),
  // and read `part` of the operand of 16-row tile `t` (first row 16 t of the tile), k half h
  static constexpr int PARTS = !KMAJ ? 1 : ES == 2 ? 2 : 4;
  __device__ static __forceinline__ void read(frag& f, int part, const unsigned char* lds, int t, int h, int lane) {
    const int q = lane >> 4, s = lane & 15;
    if constexpr (!KMAJ) {
      const int r = 16 * t + s;
      f = *reinterpret_cast<const frag*>(lds + r * 128 + 16 * ((4 * h + q) ^ (r & 7)));
    } else if constexpr (ES == 2) {
      const int a = s & 3;
      const int col0 = PAIR ? 32 * (t >> 1) : 16 * t;
      const int col = PAIR ? col0 + 8 * a + 4 * ((t & 1) ^ (a & 1)) : col0 + 4 * a;
      const int r0 = 32 * h + 8 * q + (s >> 2);  // and row r0 + 4, which has the same swizzle
      const bf16x4 v = tr_read(lds + (r0 + 4 * part) * (2 * W) + 16 * ((col >> 3) ^ swz(r0)) + (col & 7) * 2);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[4 * part + j] = v[j];
    } else {
      const int col = PAIR ? 32 * (t >> 1) + 8 * (s >> 2) + 4 * (t & 1) + (s & 3) : 16 * t + s;
      const int r = 16 * h + 4 * q + part;
      f[part] = *reinterpret_cast<const float*>(lds + r * (4 * W) + 16 * ((col >> 2) ^ swz(r)) + (col & 3) * 4);
    }
  }
};

}  // namespace

// C(m, n) = sum_k A(m, k) B(n, k) over k slice blockIdx.z. WM x WN: 16-row tiles of a wave
// (WN even); the waves form a 2 x 2 grid. Grid (tiles, 1, S).
template <class T, bool AKM, bool BKM, int WM, int WN, int NS, bool PART>
__global__ __launch_bounds__(256, 1) void tile_kernel(const T* __restrict__ A, int lda, int M, const T* __restrict__ B,
                                                      int ldb, int N, int K, Epi ep, float* __restrict__ part,
                                                      bool add) {
  typedef typename MM<T>::frag frag;
  typedef typename MM<T>::vec8 vec8;
  constexpr int BM = 32 * WM, BN = 32 * WN;
  typedef Side<T, AKM, false, BM> SA;
  typedef Side<T, BKM, true, BN> SB;
  constexpr int KS = SA::KS;
  constexpr int STAGE = SA::BYTES + SB::BYTES;
  // rows a wave turns at a time at the end, and the floats of one (4 more than its columns, for
  // the banks)
  constexpr int ROWS = WM == 8 ? 64 : WM == 1 ? 16 : 32, LDO = 16 * WN + 4;
  constexpr int TURN = 4 * ROWS * LDO * 4;
  __shared__ __attribute__((aligned(1024))) unsigned char ring[NS * STAGE > TURN ? NS * STAGE : TURN];
  const int lane = threadIdx.x & (WAVE - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int mt = (M + BM - 1) / BM, nt = (N + BN - 1) / BN;
  int tm, tn;
  tile_of(xcd_unit(blockIdx.x, mt * nt), mt, nt, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int nst = (K + KS - 1) / KS, S = gridDim.z, z = blockIdx.z;
  const int s0 = (int)((unsigned)nst * z / S), nq = (int)((unsigned)nst * (z + 1) / S) - s0;  // (nst <= 2^21)
  const int wm = wave >> 1, wn = wave & 1;

  SA sa;
  SB sb;
  sa.init(m0, M, lda, wave, lane);
  sb.init(n0, N, ldb, wave, lane);
  // the next stage to request
  const T* pa = SA::origin(A, m0, lda, s0 * KS);
  const T* pb = SB::origin(B, n0, ldb, s0 * KS);
  const size_t da = AKM ? (size_t)KS * lda : KS, db = BKM ? (size_t)KS * ldb : KS;
  // k from that stage to the slice's end
  int left = min(K, (s0 + nq) * KS) - s0 * KS;
  const int tail = (left - 1) % KS + 1;  // k of the slice's last stage
  sa.stage(left);
  sb.stage(left);
  constexpr int NDMA = SA::LOADS + SB::LOADS;
  auto request = [&](int j, unsigned char* st) {
    if (j < SA::LOADS) sa.issue(j, pa, left, st, wave, lane);
    else sb.issue(j - SA::LOADS, pb, left, st + SA::BYTES, wave, lane);
  };
  auto advance = [&] {  // (the last stage stays)
    const bool more = left > KS;
    pa += more ? da : 0;
    pb += more ? db : 0;
    left -= more ? KS : 0;
    sa.stage(left);
    sb.stage(left);
  };

  f32x4 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j) acc[i][j] = zero4();
  frag fa[2][WM], fb[2][WN];
  constexpr int NMMA = WM * WN, NRB = WN * SB::PARTS, NREAD = NRB + WM * SA::PARTS;
  auto read = [&](auto r, auto set, const unsigned char* st) {  // LDS read r of half `set`
    if constexpr (r < NRB) {
      constexpr int j = r / SB::PARTS;
      SB::read(fb[set][j], r % SB::PARTS, st + SA::BYTES, WN * wn + j, set, lane);
    } else {
      constexpr int i = (r - NRB) / SA::PARTS;
      SA::read(fa[set][i], (r - NRB) % SA::PARTS, st, WM * wm + i, set, lane);
    }
  };
  // The products of one half, with the reads of operand set `to` from st and (DMA) the requests
  // into slot dealt out evenly between them: a request holds the wave for the time of one
  // product, so two events in one place would leave the matrix cores idle.
  auto half = [&](auto set, auto to, auto dma, const unsigned char* st, unsigned char* slot) {
    constexpr int ND = decltype(dma)::value ? NDMA : 0, NE = NREAD + ND;
    each<NMMA>([&](auto t) {
      acc[t / WN][t % WN] = MM<T>::mma(fb[set][t % WN], fa[set][t / WN], acc[t / WN][t % WN]);
      each<NE>([&](auto e) {
        if constexpr (e * NMMA / NE == t) {
          constexpr int d = e * ND / NE;  // requests before event e
          if constexpr ((e + 1) * ND / NE > d) request(d, slot);
          else read(std::integral_constant<int, e - d>{}, to, st);
          __builtin_amdgcn_sched_barrier(0);
        }
      });
    });
  };
  // stage s has arrived for this wave: clear what lies behind the contraction's end
  auto arrived = [&](int s, unsigned char* st) {
    if (tail < KS && s == nq - 1) {
      sa.clear(tail, st, wave, lane);
      sb.clear(tail, st + SA::BYTES, wave, lane);
      __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  };
  constexpr std::integral_constant<int, 0> h0{};
  constexpr std::integral_constant<int, 1> h1{};

#pragma unroll 1
  for (int q = 0; q < NS; ++q) {
    each<NDMA>([&](auto j) { request(j, ring + q * STAGE); });
    advance();
  }
  wait_vmcnt<(NS - 1) * NDMA>();
  arrived(0, ring);
  bare_barrier();
  each<NREAD>([&](auto r) { read(r, h0, ring); });

  int slot = 0;
#pragma unroll 1
  for (int s = 0; s < nq; ++s) {
    // (left to itself, the scheduler mixes the loop's ends with the products, and up to 220 moves
    // between accumulation and vector registers a stage follow: 16384 x 4096 -> 11008 1550 us)
    __builtin_amdgcn_sched_barrier(0);
    unsigned char* cur = ring + slot * STAGE;
    slot = slot + 1 == NS ? 0 : slot + 1;
    unsigned char* nxt = ring + slot * STAGE;
    half(h0, h1, std::false_type{}, cur, nullptr);
    wait_vmcnt<(NS - 2) * NDMA>();  // stage s + 1 is here, and this wave's reads of s are done
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

  // Out through LDS: each wave turns ROWS rows of its tile at a time, so that the epilogue is one
  // small loop over 8 columns a lane with whole rows stored by neighbouring lanes. (Unrolled over
  // the accumulators it was 100 KB of code: 16384 x 768 -> 768 in 256 x 256 tiles 44.8 us, so 31.6.)
  bare_barrier();  // every wave is done with the ring
  float* mine = reinterpret_cast<float*>(ring) + wave * ROWS * LDO;
  const int q4 = lane >> 4, l16 = lane & 15;
  // the bfloat16 k-major layout's halves alternate: this lane's first four columns of a pair are in tile
  // q4 % 2 of it (lds_tiles.hpp)
  const int lo = BKM && sizeof(T) == 2 && (q4 & 1) ? 4 : 0;
  // lane -> row of a batch's RPI rows and 8 of its columns; four neighbouring lanes hold a group
  // of 32 columns. NB batches at a time, so that their loads, exponentials and stores overlap.
  constexpr int UPR = 2 * WN, RPI = WAVE / UPR, NB = ROWS / RPI < 4 ? ROWS / RPI : 4;
  const int row = lane / UPR, col = lane % UPR, n = n0 + 16 * WN * wn + 8 * col;
  // every lane has rows and columns in every batch, and they lie in the output
  const bool whole = ROWS % (RPI * NB) == 0 && WAVE % UPR == 0 && m0 + BM <= M && n0 + BN <= N;
  float bias[8];
  if constexpr (!PART) load_bias<T>(ep, n, N, bias);
  auto fetch_res = [&](vec8 (&r)[NB], int mr) {
    if (ep.res)
      each<NB>([&](auto k) {
        const int m = mr + k * RPI;
        if (m < M && n < N) r[k] = *reinterpret_cast<const vec8*>((const T*)ep.res + (size_t)m * N + n);
      });
  };
  each<WM * 16 / ROWS>([&](auto c) {
    const int mb = m0 + 16 * WM * wm + ROWS * c + row;
    vec8 r[NB];
    if constexpr (!PART) fetch_res(r, mb);  // (in flight while the rows are turned)
    each<ROWS / 16>([&](auto i) {
      each<WN>([&](auto j) {
        *reinterpret_cast<f32x4*>(mine + (16 * i + l16) * LDO + 32 * (j / 2) + 8 * q4 + ((j & 1) ? 4 - lo : lo)) =
            acc[c * (ROWS / 16) + i][j];
      });
    });
#pragma unroll 1
    for (int it = 0; it < ROWS; it += RPI * NB) {
      float v[NB][8];
      bool in[NB];
      each<NB>([&](auto k) {
        const int dr = it + k * RPI;
        in[k] = row < RPI && row + dr < ROWS && mb + dr < M && n < N;
        load8(mine + min(row + dr, ROWS - 1) * LDO + 8 * col, v[k]);
      });
      if constexpr (PART) {
        each<NB>([&](auto k) {
          if (!in[k]) return;
          float* p = part + ((size_t)z * M + mb + it + k * RPI) * N + n;
          if (add) {
            float o[8];
            load8(p, o);
            each<8>([&](auto j) { v[k][j] += o[j]; });
          }
          store_row<float, 8>(p, v[k]);
        });
      } else {
        vec8 rc[NB];
        each<NB>([&](auto k) { rc[k] = r[k]; });
        if (it + RPI * NB < ROWS) fetch_res(r, mb + it + RPI * NB);  // before this batch's stores
        epilogue<T, NB, 1, 2>(ep, bias, rc, v, mb + it, RPI, n, N, in, whole);
      }
    }
  });
}

namespace {

template <class T, bool AKM, bool BKM, int WM, int WN, int NS>
hipError_t run_tile(const Plan& p, const T* A, int lda, int M, const T* B, int ldb, int N, int K, const Epi& ep,
                    float* part, hipStream_t st) {
  const size_t all = (size_t)((M + 32 * WM - 1) / (32 * WM)) * ((N + 32 * WN - 1) / (32 * WN));
  if (all > 0xffffffu) return hipErrorInvalidValue;  // (a launch takes 2^32 threads: an output of 2^38 or more)
  const unsigned tiles = (unsigned)all;
  if (p.S < 1 || p.S > (K + 128 / (int)sizeof(T) - 1) / (128 / (int)sizeof(T))) return hipErrorInvalidValue;
  if (p.part)
    hipLaunchKernelGGL((tile_kernel<T, AKM, BKM, WM, WN, NS, true>), dim3(tiles, 1, p.S), dim3(256), 0, st, A, lda, M,
                       B, ldb, N, K, ep, part, p.add);
  else
    hipLaunchKernelGGL((tile_kernel<T, AKM, BKM, WM, WN, NS, false>), dim3(tiles), dim3(256), 0, st, A, lda, M, B, ldb,
                       N, K, ep, part, false);
  return hipGetLastError();
}

// The launch for one type and pair of layouts (each compiled in a file of its own).
template <class T, bool AKM, bool BKM>
hipError_t launch_planned(const Plan& p, const void* A, int lda, int M, const void* B, int ldb, int N, int K,
                          const Epi& ep, float* part, hipStream_t st) {
#define GO(WM, WN, NS)                        \
  if (p.wm == WM && p.wn == WN && p.ns == NS) \
    return run_tile<T, AKM, BKM, WM, WN, NS>(p, (const T*)A, lda, M, (const T*)B, ldb, N, K, ep, part, st)
  GO(8, 8, 2);
  GO(4, 4, 2);
  GO(2, 2, 2);
  GO(1, 2, 4);
  if constexpr (sizeof(T) == 2) {
    GO(8, 6, 2);
    GO(4, 4, 4);
    GO(2, 4, 3);
    GO(2, 2, 4);
  }
#undef GO
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace instant
