// Product of 8-bit activations and 8-bit weights with block scales:
//   out[t][n] = sum_b xs[t][b] * ws[n / 128][b] * sum_{k in b} x8[t][k] * w8[n][k]
// e4m3 codes, blocks b of 128 columns.
//
// Sums.  The 8-bit matrix instructions add eight neighbouring products with
// 13 bits below the largest of them (measured: truncated towards zero; the
// sums of eight then join with fp32's bits), a relative error of 1.5e-5 of a
// product of normal values.  That is far below bf16's rounding and far above
// fp32's.  So fp32 outputs, and all of up to 16 tokens, use the 16-bit
// matrix instructions on codes converted to fp16 (exact, as are the products
// in fp32; relative error 1e-8 per block), and bf16 outputs of more tokens
// the 8-bit ones, except where a workgroup has 16 of the tokens and the
// weights' way from HBM is what counts.
//
// Operand order: the weight rows are the instruction's rows and the tokens
// its columns, so a lane holds four consecutive n of one token: one scale
// product per 16 tokens and block (the weights' scale is uniform over a
// wave, whose rows lie in one block of 128), one fma per output and block,
// and 16-byte stores.  A lane's 32 bytes of a block are 16-byte chunks g and
// g + 4 of the row, g = lane / 16, for both operands: the order of k within
// a block does not matter as long as both sides agree, and a wave's load then
// covers 64 consecutive bytes of each row.
//
// direct_kernel: few outputs; operands straight into registers.  tile_kernel:
// the rest; tiles of both operands through LDS, in shapes from 32 x 16 to 256 x
// 256.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "kernels.h"

namespace moe {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

constexpr int kBlock = 128;
constexpr int kMaxLds = 160 * 1024;

__device__ __forceinline__ f32x4 mfma_block(i32x8 w, i32x8 x) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  // formats 0, 0: e4m3 both; no hardware scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, 0, 0, 0, 0, 0, 0);
}

// 16 codes (one 16-byte chunk) as two fp16 operands of 8.
struct Half16 {
  f16x8 lo, hi;
};
__device__ __forceinline__ Half16 to_f16(u32x4 c) {
  Half16 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, true);
    if (i < 2) {
      r.lo[4 * i] = a[0], r.lo[4 * i + 1] = a[1], r.lo[4 * i + 2] = b[0], r.lo[4 * i + 3] = b[1];
    } else {
      r.hi[4 * i - 8] = a[0], r.hi[4 * i - 7] = a[1], r.hi[4 * i - 6] = b[0], r.hi[4 * i - 5] = b[1];
    }
  }
  return r;
}

__device__ __forceinline__ f32x4 mfma_f16(f16x8 w, f16x8 x, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x, c, 0, 0, 0);
}

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi) {
  i32x8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = int(lo[i]), r[4 + i] = int(hi[i]);
  return r;
}

// One block of 16 rows as a matrix operand, in 8 and in 16 bits.
struct Frag8 {
  i32x8 v;
  __device__ Frag8() {}
  __device__ Frag8(u32x4 lo, u32x4 hi) : v(join(lo, hi)) {}
};
struct Frag16 {
  Half16 lo, hi;
  __device__ Frag16() {}
  __device__ Frag16(u32x4 l, u32x4 h) : lo(to_f16(l)), hi(to_f16(h)) {}
};
__device__ __forceinline__ f32x4 product(const Frag8& w, const Frag8& x) {
  return mfma_block(w.v, x.v);
}
__device__ __forceinline__ f32x4 product(const Frag16& w, const Frag16& x) {
  f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
  d = mfma_f16(w.lo.lo, x.lo.lo, d);
  d = mfma_f16(w.lo.hi, x.lo.hi, d);
  d = mfma_f16(w.hi.lo, x.hi.lo, d);
  return mfma_f16(w.hi.hi, x.hi.hi, d);
}

__device__ __forceinline__ u32x4 load16(const uint8_t* p) {
  return *reinterpret_cast<const u32x4*>(p);
}

// Four consecutive outputs of one token.
template <int OUT>
__device__ __forceinline__ void store4(const LinearArgs& a, int t, int n, f32x4 v) {
  if (t >= a.T || n >= a.N) return;
  const int64_t at = int64_t(t) * a.out_stride + n;
  if (a.wide_out >= (OUT == MOE_W_F32 ? 2 : 1) && n + 4 <= a.N) {
    if (OUT == MOE_W_F32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = v;
    } else {
      const f32x2 p = {v[0], v[1]}, q = {v[2], v[3]};
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
          make_uint2(__builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2_t)),
                     __builtin_bit_cast(uint32_t, __builtin_convertvector(q, bf16x2_t)));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < a.N) {
      if (OUT == MOE_W_F32) {
        static_cast<float*>(a.out)[at + i] = v[i];
      } else {
        const f32x2 p = {v[i], 0.0f};
        static_cast<uint16_t*>(a.out)[at + i] =
            uint16_t(__builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2_t)));
      }
    }
}

// ---- loads straight to LDS
//
// In assembly, because the compiler does not know which part of LDS a load
// fills and waits for all of them before the next read of any part: the loads
// of the blocks ahead then run in turn with the products (32,768 x 4096 x 2048:
// 330 us, 290 so).  Every wait for them is in this file (vmcnt counts the
// compiler's own loads and stores too, in the order of issue, so its waits are
// only ever longer than it thinks).  A load writes no register.  Reads of what
// they fill stay behind a wait that clobbers memory, and they stay behind the
// wait or barrier after the last reads of what they overwrite, as volatile
// assembly keeps its order.  M0: the LDS address, for the wave (nothing else here
// uses M0, which the compiler only sets next to its uses); the s_nop: 5 wait
// states between a vector write of a scalar operand and its use here.
#pragma clang diagnostic ignored "-Winline-asm"     // M0 among the clobbered registers

__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) {
  return __builtin_amdgcn_readfirstlane(
      uint32_t(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint8_t*)p)));
}

// A buffer of `bytes` bytes at p: what lies beyond reads as zero.
__device__ __forceinline__ u32x4 buffer_at(const uint8_t* p, uint32_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return u32x4{uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(a))),
               uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(a >> 32) & 0xFFFFu)),
               uint32_t(__builtin_amdgcn_readfirstlane(bytes)), 0x00027000u};
}

// 16 bytes per lane, lane l's to lds + 16 l: from offset at + base of a buffer.
// NT: read once.
template <bool NT>
__device__ __forceinline__ void buffer_to_lds(u32x4 src, uint32_t at, uint32_t base, uint32_t lds) {
  if (NT)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds" ::"s"(lds), "v"(at),
                 "s"(src), "s"(base)
                 : "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(at),
                 "s"(src), "s"(base)
                 : "m0");
}
// 4 bytes per lane, lane l's to lds + 4 l.
__device__ __forceinline__ void global_to_lds4(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "m0");
}

// ---- tiles through LDS

// Which of a wave's weight rows is operand row m of its i-th group of 16.
// A lane ends up with rows m = 4 (lane / 16) .. + 3 of every group: for fp32
// four consecutive outputs (16 bytes); for bf16 groups are taken in pairs of
// 32 rows so that a lane's four of both are eight consecutive ones.
template <int OUT>
__device__ __forceinline__ int weight_row(int i, int m) {
  return OUT == MOE_W_F32 ? i * 16 + m : (i >> 1) * 32 + (m >> 2) * 8 + (i & 1) * 4 + (m & 3);
}

// Eight consecutive outputs of one token as bf16.
__device__ __forceinline__ void store8(const LinearArgs& a, int t, int n, f32x4 u, f32x4 v) {
  if (t >= a.T || n >= a.N) return;
  if (a.wide_out == 2 && n + 8 <= a.N) {
    const f32x2 p[4] = {{u[0], u[1]}, {u[2], u[3]}, {v[0], v[1]}, {v[2], v[3]}};
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p[i], bf16x2_t));
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + int64_t(t) * a.out_stride + n) = q;
    return;
  }
  store4<MOE_W_BF16>(a, t, n, u);
  store4<MOE_W_BF16>(a, t, n + 4, v);
}

// Tiles of BN weight rows and BT tokens, WN x WT waves, NT: weights are read
// once (non-temporal), a ring of STAGES LDS buffers of one block of 128 columns
// each: STAGES - 1 blocks are on their way while one is multiplied, across tiles
// too (workgroups stay and walk over tiles, so that the first blocks of a tile
// arrive during the stores of the one before).  The loads are buffer loads
// straight to LDS: rows past the matrices' ends read as zero, and so do columns
// past K (their lanes' offset is moved out of range).  A row's 16-byte chunks are
// permuted in LDS by the row, so that the rows a fragment reads together meet
// no bank twice.  fp32 outputs, and those of 16 tokens, convert the codes to
// fp16 on their way from LDS.  Few tokens stream the weights (1 x 151,936 x 2048:
// 48 us, 6.5 TB/s; a bare read of the same bytes takes 45), many are bound by LDS,
// matrix instructions and the fma of the scales together (32,768 x 4096 x 2048:
// 281-300 us from card to card, 1.83-1.96 PFLOP/s).
//
// KS > 1, for few tiles: KS groups of WN x WT waves take every KS-th block each,
// with rings of their own, and their sums are joined in a fixed order at the
// end (one tile per workgroup then).
template <int BN, int BT, int WN, int WT, int STAGES, int KS, int OUT>
struct Tile {
  static constexpr int kWaves = WN * WT;                      // of one group
  static constexpr int NI = BN / WN / 16, TI = BT / WT / 16;
  static constexpr int kRows = BN + BT;                       // rows of one buffer, 128 bytes each
  static constexpr int kWLoads = BN / 8 / kWaves, kXLoads = BT / 8 / kWaves;
  static constexpr int kLoads = kWLoads + kXLoads;            // 1 KiB loads per wave and block
  static constexpr int kBuffer = kRows * kBlock + (BT > 64 ? BT : 64) * 4;   // and the tokens' scales,
                                                              // which whole waves load
  static constexpr int kStores = OUT == MOE_W_F32 ? NI * TI : NI * TI / 2;   // per wave and tile
  static_assert(BN % (8 * kWaves) == 0 && BT % (8 * kWaves) == 0 && kBlock % (BN / WN) == 0 &&
                    NI % 2 == 0 && BT <= 64 * kWaves,
                "tile shape");
};

template <int N>
__device__ __forceinline__ void wait_until() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N < 63 ? N : 63) : "memory");
}

// A barrier that leaves loads and stores under way (__syncthreads waits for
// them all); this wave's reads of LDS have ended.
__device__ __forceinline__ void barrier_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int BN, int BT, int WN, int WT, int STAGES, int KS, int OUT, bool NT>
__global__ __launch_bounds__(KS* WN* WT * 64) void tile_kernel(const LinearArgs a) {
  using S = Tile<BN, BT, WN, WT, STAGES, KS, OUT>;
  constexpr int NI = S::NI, TI = S::TI, LOADS = S::kLoads, BUFFER = S::kBuffer;
  extern __shared__ uint8_t all_lds[];
  const int lane = threadIdx.x & 63, all_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = all_wave / S::kWaves, wave = all_wave % S::kWaves;
  uint8_t* lds = all_lds + group * (STAGES * BUFFER);
  const int col = lane & 15, g = lane >> 4;
  const int wn = wave % WN, wt = wave / WN;
  const int KB = (a.K + kBlock - 1) / kBlock;

  // Tiles: XCD x (blockIdx mod 8) takes a contiguous run; along it, groups of
  // four token tiles walk over the weights together, so that what an XCD's
  // CUs read at a time fits its L2.
  const int tiles_n = (a.N + BN - 1) / BN, tiles_t = (a.T + BT - 1) / BT, tiles = tiles_n * tiles_t;
  const int run = (tiles + 7) / 8, first = int(blockIdx.x & 7) * run;
  const int last = min(first + run, tiles), step = int(gridDim.x >> 3);
  constexpr int kGroup = 4;
  auto place = [&](int id, int& n0, int& t0) {
    const int size = kGroup * tiles_n, gi = id / size, rem = id % size;
    const int rows = min(kGroup, tiles_t - gi * kGroup);
    t0 = (gi * kGroup + rem % rows) * BT;
    n0 = rem / rows * BN;
  };

  // the loads' side: every wave fills its share of the weight rows and of the
  // token rows, 8 rows per load, lane l the slot l % 8 of row l / 8
  constexpr int WL = S::kWLoads, XL = S::kXLoads;
  const int wrow0 = wave * (WL * 8), xrow0 = wave * (XL * 8);
  auto wswap = [](int r) { return OUT == MOE_W_F32 ? r & 7 : (r & 3) | ((r >> 1) & 4); };
  uint32_t off[3], off_last[3];      // weight rows' loads by parity, token rows'
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int r = wrow0 + i * 8 + (lane >> 3), chunk = (lane & 7) ^ (i < 2 ? wswap(r) : r & 7);
    off[i] = uint32_t(lane >> 3) * a.K + chunk * 16;
    off_last[i] = (KB - 1) * kBlock + chunk * 16 < a.K ? off[i] : 0x7FFFFFFFu;
  }
  int load_id = first + int(blockIdx.x >> 3), load_kb = group, load_buf = 0;
  int under_way = 0;     // blocks loaded and not yet multiplied
  if (load_id >= last) return;
  u32x4 wsrc, xsrc;
  const uint32_t lds_at = lds_address(lds);
  const float* scales;
  auto source = [&]() {
    int n0, t0;
    place(load_id, n0, t0);
    // (a load whose scalar offset passes the end reads zeros too)
    auto rows = [&](const uint8_t* p, int r0, int n) {
      const int64_t left = int64_t(n - r0) * a.K;
      return buffer_at(p + int64_t(r0) * a.K, uint32_t(left < 0x7FFFFFFF ? left : 0x7FFFFFFF));
    };
    wsrc = rows(a.w8, n0, a.N);
    xsrc = rows(a.x8, t0, a.T);
    scales = a.x_scale + int64_t(min(t0 + (wave * 64 + lane) % BT, a.T - 1)) * KB;
  };
  auto load = [&]() {
    if (load_id >= last || (KS > 1 && load_kb >= KB)) return;
    const uint32_t dst = lds_at + load_buf * BUFFER;
    const bool whole = load_kb + 1 < KB;
    const int k = load_kb * kBlock;
#pragma unroll
    for (int i = 0; i < WL; ++i)
      buffer_to_lds<NT>(wsrc, whole ? off[i & 1] : off_last[i & 1], (wrow0 + i * 8) * a.K + k,
                        dst + (wrow0 + i * 8) * kBlock);
#pragma unroll
    for (int i = 0; i < XL; ++i)
      buffer_to_lds<false>(xsrc, whole ? off[2] : off_last[2], (xrow0 + i * 8) * a.K + k,
                           dst + (BN + xrow0 + i * 8) * kBlock);
    if (wave * 64 < BT) global_to_lds4(scales + load_kb, dst + S::kRows * kBlock + wave * 256);
    load_buf = load_buf + 1 == STAGES ? 0 : load_buf + 1;
    ++under_way;
    load_kb += KS;
    if (KS == 1 && load_kb == KB) {
      load_kb = 0;
      load_id += step;
      if (load_id < last) source();
    }
  };
  source();
#pragma unroll
  for (int i = 0; i + 1 < STAGES; ++i) load();

  // the products' side
  using Frag = std::conditional_t<OUT == MOE_W_F32 || BT == 16, Frag16, Frag8>;
  auto frag = [&](const uint8_t* row, int swap) {
    return Frag(load16(row + ((g ^ swap) * 16)), load16(row + (((g + 4) ^ swap) * 16)));
  };
  const int x_at = (BN + wt * (BT / WT) + col) * kBlock, w_at = wn * (BN / WN) * kBlock;
  const int s_at = S::kRows * kBlock + (wt * (BT / WT) + col) * 4;
  int buf = 0;
  bool stored = false;
#pragma unroll 1
  for (int id = first + int(blockIdx.x >> 3); id < last; id += step) {
    int n0, t0;
    place(id, n0, t0);
    const int wave_n = n0 + wn * (BN / WN), wave_t = t0 + wt * (BT / WT);
    // (constant address space: scalar loads, which no count of vector loads waits for)
    const auto wsc = (const __attribute__((address_space(4))) float*)a.w_scale +
                     int64_t(min(wave_n, a.N - 1) / kBlock) * KB;
    f32x4 acc[NI][TI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < TI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float ws = wsc[min(group, KB - 1)];
#pragma unroll 1
    for (int kb = group; kb < KB + group; kb += KS) {   // (all groups take part in the barriers)
      // this block has arrived when no more than the later blocks' loads (and,
      // behind them, the last tile's stores) are outstanding
      if (under_way < STAGES - 1)
        wait_until<0>();
      else if (stored)
        wait_until<(STAGES - 2) * LOADS + S::kStores>();
      else
        wait_until<(STAGES - 2) * LOADS>();
      stored = false;
      --under_way;
      barrier_lds();
      if (KS > 1 && kb >= KB) break;
      const uint8_t* now = lds + buf * BUFFER;
      auto wfrag = [&](int i) {
        const int r = weight_row<OUT>(i, col);
        return frag(now + w_at + r * kBlock, wswap(r));
      };
      float sc[TI];
      Frag x[TI], w = wfrag(0);
#pragma unroll
      for (int j = 0; j < TI; ++j) {
        x[j] = frag(now + x_at + j * (16 * kBlock), col & 7);
        sc[j] = *reinterpret_cast<const float*>(now + s_at + j * 64) * ws;
      }
      load();      // into the buffer that every wave has left
      ws = wsc[min(kb + KS, KB - 1)];
      // the sums of group i - 1 join the accumulators while group i is multiplied
      f32x4 d[2][TI];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        Frag next;
        if (i + 1 < NI) next = wfrag(i + 1);
#pragma unroll
        for (int j = 0; j < TI; ++j) {
          d[i & 1][j] = product(w, x[j]);
          if (i > 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i - 1][j][e] = fmaf(d[(i - 1) & 1][j][e], sc[j], acc[i - 1][j][e]);
          }
          if (OUT == MOE_W_BF16) {
            // one matrix instruction, four fma, a fragment's read
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
            if (j < 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          }
        }
        w = next;
        if (OUT == MOE_W_BF16) __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int j = 0; j < TI; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[NI - 1][j][e] = fmaf(d[(NI - 1) & 1][j][e], sc[j], acc[NI - 1][j][e]);
      buf = buf + 1 == STAGES ? 0 : buf + 1;
    }
    if constexpr (KS > 1) {
      // groups 1 .. leave their sums in LDS, group 0 adds them in order
      static_assert(STAGES * KS * BUFFER >= (KS - 1) * BN * BT * 4, "room for the sums");
      f32x4* sums = reinterpret_cast<f32x4*>(all_lds);
      __syncthreads();
      if (group > 0) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < TI; ++j)
            sums[(((group - 1) * S::kWaves + wave) * NI * TI + i * TI + j) * 64 + lane] = acc[i][j];
      }
      __syncthreads();
      if (group > 0) return;
      for (int k = 0; k + 1 < KS; ++k)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < TI; ++j)
            acc[i][j] += sums[((k * S::kWaves + wave) * NI * TI + i * TI + j) * 64 + lane];
    }
#pragma unroll
    for (int j = 0; j < TI; ++j) {
      const int t = wave_t + j * 16 + col;
#pragma unroll
      for (int i = 0; i < NI; i += 2) {
        if (OUT == MOE_W_F32) {
          store4<OUT>(a, t, wave_n + i * 16 + g * 4, acc[i][j]);
          store4<OUT>(a, t, wave_n + i * 16 + 16 + g * 4, acc[i + 1][j]);
        } else {
          store8(a, t, wave_n + i * 16 + g * 8, acc[i][j], acc[i + 1][j]);
        }
      }
    }
    // with all of them issued as one store each, the next wait can leave them behind
    stored = a.wide_out == 2 && n0 + BN <= a.N && t0 + BT <= a.T;
  }
}

// ---- few outputs

// A workgroup owns NI x 16 weight rows and 16 tokens, and its KS waves split
// the blocks: each loads its own blocks straight into registers, the next while
// it multiplies one, and waits for nobody until the sums are joined, in a
// fixed order, through LDS.  Bound by latency (1 x 2048 x 2048: 3.6 us; 17 x 2048
// x 2048: 4.6) and by what one CU takes in: 16 waves instead of 8 change
// nothing, half the rows per workgroup almost halve the time while CUs are free.
template <int NI, int KS, int OUT>
__global__ __launch_bounds__(KS * 64) void direct_kernel(const LinearArgs a) {
  __shared__ f32x4 sums[KS][NI][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int KB = (a.K + kBlock - 1) / kBlock;
  const int tiles_n = (a.N + NI * 16 - 1) / (NI * 16);
  const int n0 = int(blockIdx.x) % tiles_n * (NI * 16), t0 = int(blockIdx.x) / tiles_n * 16;
  const uint8_t* wbase = a.w8 + int64_t(n0) * a.K;
  const float* wsc = a.w_scale + int64_t(n0 / kBlock) * KB;
  uint32_t woff[NI];     // rows past the ends repeat the last one
#pragma unroll
  for (int i = 0; i < NI; ++i)
    woff[i] = uint32_t(min(i * 16 + col, a.N - 1 - n0)) * a.K + g * 16;
  const int t = min(t0 + col, a.T - 1);
  const uint8_t* x = a.x8 + int64_t(t) * a.K + g * 16;
  const float* xsc = a.x_scale + int64_t(t) * KB;
  struct Raw {
    u32x4 w[NI][2], x[2];
    float scale;
  };
  auto load = [&](Raw& q, int kb) {
    const int k = kb * kBlock;
    if (k + kBlock <= a.K) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        q.w[i][0] = load16(wbase + k + woff[i]), q.w[i][1] = load16(wbase + k + 64 + woff[i]);
      q.x[0] = load16(x + k), q.x[1] = load16(x + k + 64);
    } else {
      // the last, shorter block: zeros past the row's end
      const u32x4 zero = {0u, 0u, 0u, 0u};
      const bool lo = k + g * 16 < a.K, hi = k + g * 16 + 64 < a.K;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        q.w[i][0] = q.w[i][1] = zero;
        if (lo) q.w[i][0] = load16(wbase + k + woff[i]);
        if (hi) q.w[i][1] = load16(wbase + k + 64 + woff[i]);
      }
      q.x[0] = q.x[1] = zero;
      if (lo) q.x[0] = load16(x + k);
      if (hi) q.x[1] = load16(x + k + 64);
    }
    q.scale = xsc[kb] * wsc[kb];
  };
  f32x4 acc[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](const Raw& q) {
    const Frag16 xf(q.x[0], q.x[1]);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const f32x4 d = product(Frag16(q.w[i][0], q.w[i][1]), xf);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(d[e], q.scale, acc[i][e]);
    }
  };
  Raw q[2];
  if (wave < KB) load(q[0], wave);
#pragma unroll 1
  for (int kb = wave; kb < KB; kb += 2 * KS) {
    if (kb + KS < KB) load(q[1], kb + KS);
    add(q[0]);
    if (kb + KS >= KB) break;
    if (kb + 2 * KS < KB) load(q[0], kb + 2 * KS);
    add(q[1]);
  }
  // wave i adds up the i-th 16 rows' sums, waves in order
#pragma unroll
  for (int i = 0; i < NI; ++i) sums[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave < NI) {
    f32x4 v = sums[0][wave][lane];
#pragma unroll
    for (int k = 1; k < KS; ++k) v += sums[k][wave][lane];
    store4<OUT>(a, t0 + col, n0 + wave * 16 + g * 4, v);
  }
}

// Dynamic LDS above 64 KiB has to be asked for.
template <class Kernel>
hipError_t allow_lds(Kernel kernel, int64_t bytes) {
  if (bytes <= 64 * 1024) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

template <int BN, int BT, int WN, int WT, int STAGES, int KS, int OUT, bool NT = false>
hipError_t launch_tile(const LinearArgs& a, hipStream_t st) {
  using S = Tile<BN, BT, WN, WT, STAGES, KS, OUT>;
  const auto kernel = tile_kernel<BN, BT, WN, WT, STAGES, KS, OUT, NT>;
  const int lds = KS * STAGES * S::kBuffer;
  static_assert(KS * STAGES * S::kBuffer <= kMaxLds, "LDS");
  const hipError_t e = allow_lds(kernel, lds);
  if (e != hipSuccess) return e;
  const int64_t tiles = int64_t((a.N + BN - 1) / BN) * ((a.T + BT - 1) / BT);
  if (tiles > 0x7FFFFFF) return hipErrorInvalidValue;
  // as many workgroups as fit at once (a multiple of the 8 XCDs); with several
  // groups of waves one for every tile
  const int64_t slots = 256 * (kMaxLds / lds);
  const int64_t grid = (KS > 1 || tiles < slots ? tiles + 7 : slots) / 8 * 8;
  kernel<<<dim3(uint32_t(grid)), KS * S::kWaves * 64, lds, st>>>(a);
  return hipGetLastError();
}

template <int NI, int OUT>
hipError_t launch_direct(const LinearArgs& a, hipStream_t st) {
  constexpr int KS = 8;
  const int tiles = ((a.N + NI * 16 - 1) / (NI * 16)) * ((a.T + 15) / 16);
  direct_kernel<NI, KS, OUT><<<tiles, KS * 64, 0, st>>>(a);
  return hipGetLastError();
}

// Which kernel.  Times are of T x N x K in us, weights from HBM.
template <int OUT>
hipError_t launch(const LinearArgs& a, hipStream_t st) {
  auto tiles = [&](int bn, int bt) {
    return int64_t((a.N + bn - 1) / bn) * ((a.T + bt - 1) / bt);
  };
  auto rounds = [](int64_t n, int slots) { return (n + slots - 1) / slots; };
  const int KB = (a.K + kBlock - 1) / kBlock;
  // Few tokens, many rows: every byte of the weights once, two workgroups of
  // two groups of waves per CU.
  if (a.T <= 16 && a.N >= 20000) return launch_tile<64, 16, 2, 1, 3, 2, OUT, true>(a, st);
  // A CU takes in no more than about 30 GB/s of what comes from HBM, however
  // many of its waves ask: the finest workgroups of which each CU gets at most
  // one.  32 x 1024 x 4096: 7.0 with 16 x 16, 11.5 with 32 x 32; 240 x 1000 x
  // 4096: 7.4-8.7 with 32 x 32 (12-14 with 64 x 64).  Short rows go straight
  // into registers (100 x 1000 x 2000: 4.7, through LDS 5.8), for long ones deeper
  // rings pay (16 x 8192 x 8192: 14, into registers 19).
  if (tiles(16, 16) <= 256) return launch_direct<1, OUT>(a, st);
  if (tiles(32, 16) <= 256) {
    if (KB >= 32) return launch_tile<32, 16, 1, 1, 4, 4, OUT, true>(a, st);
    return launch_direct<2, OUT>(a, st);
  }
  // 16 x 12,000 x 4096: 12 (15 into registers)
  if (a.T <= 16) return launch_tile<64, 16, 2, 1, 4, 2, OUT, true>(a, st);
  if (tiles(32, 32) <= 256) return launch_tile<32, 32, 1, 1, 4, 4, OUT>(a, st);
  // 64 x 8192 x 8192: 21-22 (34 with 64 x 64), 500 x 1000 x 2000: 6.9-7.9 (9.5-10)
  if (tiles(64, 32) <= 256) return launch_tile<64, 32, 2, 1, 3, 4, OUT>(a, st);
  // One tile of tokens: narrow tiles, several workgroups per CU.
  if (a.T <= 32) {
    // up to two per CU: two groups of waves each (20 x 25,000 x 4096: 23, 27-29
    // with one); 32 x 60,000 x 1024: 13-14 with 64 rows, 13-15 with 128, 32 x
    // 151,936 x 2048: 58-65 and 54-62
    if (tiles(64, 32) <= 512) return launch_tile<64, 32, 2, 1, 3, 2, OUT, true>(a, st);
    if (tiles(128, 64) <= 512) return launch_tile<64, 32, 2, 1, 3, 1, OUT, true>(a, st);
    return launch_tile<128, 64, 2, 2, 2, 1, OUT, true>(a, st);
  }
  if (a.T <= 64) {
    // 64 x 151,936 x 2048: 63-71 (75-81 with 64 rows), 64 x 40,000 x 4096: 46-49 (47-50)
    if (tiles(64, 64) > 512) return launch_tile<128, 64, 2, 2, 2, 1, OUT, true>(a, st);
  } else {
    if constexpr (OUT == MOE_W_BF16) {
      // a round of 256 tiles of 256 x 256 costs 1.6 of 512 of 128 x 128 (32,768
      // x 4096 x 2048: 293 and 379; 3000 x 4096 x 4096: 63 and 71, 300 x 40,000 x
      // 2048: 61 and 49)
      if (8 * rounds(tiles(256, 256), 256) <= 5 * rounds(tiles(128, 128), 512))
        return launch_tile<256, 256, 2, 4, 2, 1, OUT>(a, st);
    }
    // fp32 32,768 x 4096 x 2048: 566 and 603; bf16 300 x 40,000 x 2048: 44 and 49;
    // fp32 3000 x 4096 x 4096 (more to do for some CUs): 122 and 103
    if (2 * rounds(tiles(256, 128), 256) <= rounds(tiles(128, 128), 256))
      return launch_tile<256, 128, 4, 2, OUT == MOE_W_F32 ? 2 : 3, 1, OUT>(a, st);
    if (tiles(128, 128) > 256) return launch_tile<128, 128, 2, 2, 2, 1, OUT>(a, st);
    if (tiles(128, 128) > 128) return launch_tile<128, 128, 2, 2, 2, 2, OUT>(a, st);
  }
  // few tiles: groups of waves that share the blocks (777 x 1000 x 2000: fp32
  // 10.6 with four, 11.0 with two and deeper rings; bf16 10.0 and 8.8; 300 x 4096 x
  // 4096, 320 tiles: 18-25 with two, two workgroups per CU, 22-31 with one)
  if (tiles(64, 64) > 256) return launch_tile<64, 64, 2, 2, 2, 2, OUT>(a, st);
  if constexpr (OUT == MOE_W_F32)
    return launch_tile<64, 64, 2, 2, 2, 4, OUT>(a, st);
  else
    return launch_tile<64, 64, 2, 2, 4, 2, OUT>(a, st);
}

}  // namespace

hipError_t launch_scaled_linear(LinearArgs a, hipStream_t st) {
  // every row's start allows stores of 16 bytes: 2, of 8 bytes: 1 (bf16,
  // 30,000 x 300 x 496: 18 us; 30 with stores of one element and smaller tiles)
  const int64_t bytes = a.out_stride * (a.out_fmt == MOE_W_F32 ? 4 : 2);
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.out);
  a.wide_out = (at | bytes) % 16 == 0 ? 2 : (at | bytes) % 8 == 0 ? 1 : 0;
  return a.out_fmt == MOE_W_F32 ? launch<MOE_W_F32>(a, st) : launch<MOE_W_BF16>(a, st);
}

}  // namespace moe
