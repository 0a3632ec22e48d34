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
// ring_kernel: few tokens, many weight rows; every row is streamed once, the
// tokens stay in LDS.  direct_kernel: few outputs; operands straight into
// registers.  tile_kernel: the rest; tiles of both operands through LDS.

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

// ---- few tokens

__device__ __forceinline__ u32x4 load16(const uint8_t* p) {
  return *reinterpret_cast<const u32x4*>(p);
}

// The tokens into LDS as fp16, [T][row_blocks * 128], each row's 16-byte
// chunks permuted by the row (t & 7) so that 16 rows read at one column meet
// no bank twice; and their scales, [KB][16].
__device__ __forceinline__ void stage_tokens(const LinearArgs& a, int row_blocks, uint8_t* xl,
                                             float* xs) {
  const int KB = (a.K + kBlock - 1) / kBlock;
  const int chunks = KB * 8;                    // 16 codes each: two chunks of fp16
  const int all = a.T * chunks, step = int(blockDim.x);
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < all; i0 += 4 * step) {
    u32x4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * step, t = i / chunks, k = i % chunks * 16;
      v[j] = u32x4{0u, 0u, 0u, 0u};
      if (i < all && k < a.K) v[j] = load16(a.x8 + int64_t(t) * a.K + k);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * step, t = i / chunks, c = i % chunks;
      if (i >= all) break;
      const Half16 h = to_f16(v[j]);
      uint8_t* p = xl + int64_t(t) * row_blocks * (kBlock * 2);
      *reinterpret_cast<f16x8*>(p + ((2 * c) ^ (t & 7)) * 16) = h.lo;
      *reinterpret_cast<f16x8*>(p + ((2 * c + 1) ^ (t & 7)) * 16) = h.hi;
    }
  }
#pragma unroll 1
  for (int i = threadIdx.x; i < 16 * KB; i += step) {
    const int t = i / KB, b = i % KB;
    xs[b * 16 + t] = t < a.T ? a.x_scale[int64_t(t) * KB + b] : 0.0f;
  }
}

// One block of 16 weight rows (this lane's two chunks) times the staged tokens.
__device__ __forceinline__ void add_block(const LinearArgs& a, u32x4 wlo, u32x4 whi, float ws, int b,
                                          int row_blocks, const uint8_t* xl, const float* xs,
                                          f32x4& acc) {
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const Half16 lo = to_f16(wlo), hi = to_f16(whi);
  const int t = min(col, a.T - 1);     // columns past T are not stored
  const uint8_t* p = xl + int64_t(t) * row_blocks * (kBlock * 2);
  const int c = b * 16 + 2 * g;
  auto x = [&](int chunk) {
    return *reinterpret_cast<const f16x8*>(p + ((chunk ^ (t & 7)) * 16));
  };
  f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
  d = mfma_f16(lo.lo, x(c), d);
  d = mfma_f16(lo.hi, x(c + 1), d);
  d = mfma_f16(hi.lo, x(c + 8), d);
  d = mfma_f16(hi.hi, x(c + 9), d);
  const float sc = xs[b * 16 + col] * ws;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = fmaf(d[i], sc, acc[i]);
}

// Many weight rows: one workgroup per CU stays and its waves walk over tiles
// of 16 rows.  Each wave owns two LDS slots of two blocks (4 KiB) and loads
// one while it multiplies the other; nothing waits for another wave.  The
// loads go straight to LDS because a matrix operand's layout would split
// every row's line between two instructions: eight lanes fetch 128
// consecutive bytes of a row instead, non-temporal (each byte is used once).
// Measured on 151,936 x 2048 weights, 1 token: 47 us (6.6 TB/s; a bare
// read of the same bytes takes 45 us), against 55 us with loads into
// registers, and 51-57 us with more slots, more workgroups or ordinary loads.
constexpr int kRingWaves = 8;
constexpr int kRingBlocks = 2;                        // blocks per slot
constexpr int kRingSlot = kRingBlocks * 16 * kBlock;  // bytes
constexpr int kRingLoads = kRingSlot / 1024;
constexpr int kMaxLds = 160 * 1024;

// Every load of this wave has arrived, and its reads of LDS have ended (the
// next loads may overwrite what they read).
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}

// LDS of a workgroup: slots, two tiles' weight scales per wave, tokens, their scales.
inline int ring_scales(int KB) { return (KB + 63) / 64 * 64; }
inline int64_t ring_lds(int T, int KB) {
  const int row_blocks = (KB + kRingBlocks - 1) / kRingBlocks * kRingBlocks;
  return kRingWaves * (2 * kRingSlot + 2 * ring_scales(KB) * 4) +
         int64_t(T) * row_blocks * (kBlock * 2) + int64_t(row_blocks) * 16 * 4;
}

template <int OUT>
__global__ __launch_bounds__(kRingWaves * 64) void ring_kernel(const LinearArgs a) {
  extern __shared__ uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int KB = (a.K + kBlock - 1) / kBlock;
  const int steps = (KB + kRingBlocks - 1) / kRingBlocks, row_blocks = steps * kRingBlocks;
  const int tiles = (a.N + 15) / 16, stride = int(gridDim.x) * kRingWaves;
  const int scales = (KB + 63) / 64 * 64;
  uint8_t* slots = lds + wave * (2 * kRingSlot);
  float* wsl = reinterpret_cast<float*>(lds + kRingWaves * 2 * kRingSlot) + wave * 2 * scales;
  float* xs = reinterpret_cast<float*>(lds + kRingWaves * 2 * kRingSlot) + kRingWaves * 2 * scales;
  uint8_t* xl = reinterpret_cast<uint8_t*>(xs + row_blocks * 16);

  // load i of a slot fills rows 4i .. 4i + 3, 16 lanes (256 bytes) each; slot
  // s of a row holds the row's chunk s ^ (row & 7).  Chunks past the row's
  // end are read at its end and not used.
  constexpr int kLanes = kRingBlocks * 8, kRows = 64 / kLanes;
  const int lrow = lane / kLanes, lslot = lane % kLanes;
  int lt = int(blockIdx.x) * kRingWaves + wave, ls = 0, lslotno = 0, lbuf = 0;
  auto load = [&]() {
    if (lt >= tiles) return;
    if (ls == 0) {
      const float* src = a.w_scale + int64_t(lt * 16 / kBlock) * KB;
      for (int i = 0; i < scales; i += 64)
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)(src + min(i + lane, KB - 1)),
            (__attribute__((address_space(3))) void*)(wsl + lbuf * scales + i), 4, 0, 0);
      lbuf ^= 1;
    }
#pragma unroll
    for (int i = 0; i < kRingLoads; ++i) {
      const int r = i * kRows + lrow;
      const int k = min(ls * (kRingBlocks * kBlock) + ((lslot ^ (r & 7)) * 16), a.K - 16);
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(a.w8 + int64_t(min(lt * 16 + r, a.N - 1)) * a.K + k),
          (__attribute__((address_space(3))) void*)(slots + lslotno * kRingSlot + i * 1024), 16, 0,
          2 /* non-temporal */);
    }
    lslotno ^= 1;
    if (++ls == steps) ls = 0, lt += stride;
  };
  load();
  stage_tokens(a, row_blocks, xl, xs);
  __syncthreads();

  int slot = 0, buf = 0;
#pragma unroll 1
  for (int tile = int(blockIdx.x) * kRingWaves + wave; tile < tiles; tile += stride) {
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int st = 0; st < steps; ++st) {
      wait_loads();         // this slot has arrived, and the tile's scales before it
      load();
      const uint8_t* p = slots + slot * kRingSlot + col * (kRingBlocks * kBlock);
#pragma unroll
      for (int b = 0; b < kRingBlocks; ++b) {
        const int kb = st * kRingBlocks + b;
        if (kb >= KB) break;
        u32x4 lo = load16(p + ((b * 8 + g) ^ (col & 7)) * 16);
        u32x4 hi = load16(p + ((b * 8 + g + 4) ^ (col & 7)) * 16);
        if (kb * kBlock + kBlock > a.K) {
          if (kb * kBlock + g * 16 >= a.K) lo = u32x4{0u, 0u, 0u, 0u};
          if (kb * kBlock + g * 16 + 64 >= a.K) hi = u32x4{0u, 0u, 0u, 0u};
        }
        add_block(a, lo, hi, wsl[buf * scales + kb], kb, row_blocks, xl, xs, acc);
      }
      slot ^= 1;
    }
    buf ^= 1;
    store4<OUT>(a, col, tile * 16 + g * 4, acc);
  }
}

// ---- many tokens

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
// once (non-temporal), a ring of STAGES LDS
// buffers of one block of 128 columns each: STAGES - 1 blocks are on their way
// while one is multiplied, across tiles too (workgroups stay and walk over
// tiles, so that the first blocks of a tile arrive during the stores of the
// one before).  The loads are buffer loads straight to LDS: rows past the
// matrices' ends read as zero, and so do columns past K (their lanes' offset
// is moved out of range).  A row's 16-byte chunks are permuted in LDS by the
// row, so that the rows a fragment reads together meet no bank twice.
// fp32 outputs convert the codes to fp16 on their way from LDS.
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
  __amdgpu_buffer_rsrc_t wsrc, xsrc;
  const float* scales;
  auto source = [&]() {
    int n0, t0;
    place(load_id, n0, t0);
    // (a load whose scalar offset passes the end reads zeros too)
    auto rows = [&](const uint8_t* p, int r0, int n) {
      const int64_t left = int64_t(n - r0) * a.K;
      return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p + int64_t(r0) * a.K), 0,
                                               int(left < 0x7FFFFFFF ? left : 0x7FFFFFFF), 0x00027000);
    };
    wsrc = rows(a.w8, n0, a.N);
    xsrc = rows(a.x8, t0, a.T);
    scales = a.x_scale + int64_t(min(t0 + (wave * 64 + lane) % BT, a.T - 1)) * KB;
  };
  auto load = [&]() {
    if (load_id >= last || (KS > 1 && load_kb >= KB)) return;
    uint8_t* dst = lds + load_buf * BUFFER;
    const bool whole = load_kb + 1 < KB;
    const int k = load_kb * kBlock;
#pragma unroll
    for (int i = 0; i < WL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wsrc, (__attribute__((address_space(3))) void*)(dst + (wrow0 + i * 8) * kBlock), 16,
          whole ? off[i & 1] : off_last[i & 1], (wrow0 + i * 8) * a.K + k, 0, NT ? 2 : 0);
#pragma unroll
    for (int i = 0; i < XL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xsrc, (__attribute__((address_space(3))) void*)(dst + (BN + xrow0 + i * 8) * kBlock), 16,
          whole ? off[2] : off_last[2], (xrow0 + i * 8) * a.K + k, 0, 0);
    if (wave * 64 < BT)
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(scales + load_kb),
          (__attribute__((address_space(3))) void*)(dst + S::kRows * kBlock + wave * 256), 4, 0, 0);
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
  using Frag = std::conditional_t<OUT == MOE_W_F32, Frag16, Frag8>;
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
    const float* wsc = a.w_scale + int64_t(min(wave_n, a.N - 1) / kBlock) * KB;
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

// A workgroup owns NI x 16 weight rows and TI x 16 tokens, and its KS waves
// split the blocks: each loads its own blocks straight into registers, the
// next while it multiplies one, and waits for nobody until the sums are
// joined, in a fixed order, through LDS.  Bound by latency (1 x 2048 x 2048:
// 3.9 us; 17 x 2048 x 2048: 4.8) and by what one CU takes in: 16 waves instead
// of 8 change nothing, half the rows per workgroup almost halve the time
// while CUs are free.
template <int NI, int TI, int KS, int OUT>
__global__ __launch_bounds__(KS * 64) void direct_kernel(const LinearArgs a) {
  extern __shared__ uint8_t joined[];
  auto sums = reinterpret_cast<f32x4(*)[NI * TI][64]>(joined);      // [KS]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int KB = (a.K + kBlock - 1) / kBlock;
  const int tiles_n = (a.N + NI * 16 - 1) / (NI * 16);
  const int n0 = int(blockIdx.x) % tiles_n * (NI * 16), t0 = int(blockIdx.x) / tiles_n * (TI * 16);
  const uint8_t* wbase = a.w8 + int64_t(n0) * a.K;
  const uint8_t* xbase = a.x8 + int64_t(t0) * a.K;
  const float* sbase = a.x_scale + int64_t(t0) * KB;
  const float* wsc = a.w_scale + int64_t(n0 / kBlock) * KB;
  uint32_t woff[NI], xoff[TI], soff[TI];     // rows past the ends repeat the last one
#pragma unroll
  for (int i = 0; i < NI; ++i)
    woff[i] = uint32_t(min(i * 16 + col, a.N - 1 - n0)) * a.K + g * 16;
#pragma unroll
  for (int j = 0; j < TI; ++j) {
    const int r = min(j * 16 + col, a.T - 1 - t0);
    xoff[j] = uint32_t(r) * a.K + g * 16;
    soff[j] = uint32_t(r) * KB;
  }
  struct Raw {
    u32x4 w[NI][2], x[TI][2];
    float xs[TI], ws;
  };
  auto load = [&](Raw& q, int kb) {
    const int k = kb * kBlock;
    if (k + kBlock <= a.K) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        q.w[i][0] = load16(wbase + k + woff[i]), q.w[i][1] = load16(wbase + k + 64 + woff[i]);
#pragma unroll
      for (int j = 0; j < TI; ++j)
        q.x[j][0] = load16(xbase + k + xoff[j]), q.x[j][1] = load16(xbase + k + 64 + xoff[j]);
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
#pragma unroll
      for (int j = 0; j < TI; ++j) {
        q.x[j][0] = q.x[j][1] = zero;
        if (lo) q.x[j][0] = load16(xbase + k + xoff[j]);
        if (hi) q.x[j][1] = load16(xbase + k + 64 + xoff[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < TI; ++j) q.xs[j] = sbase[soff[j] + kb];
    q.ws = wsc[kb];
  };
  f32x4 acc[NI][TI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < TI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  using Frag = std::conditional_t<OUT == MOE_W_F32 || TI == 1, Frag16, Frag8>;
  auto add = [&](const Raw& q) {
    Frag x[TI];
    float sc[TI];
#pragma unroll
    for (int j = 0; j < TI; ++j) x[j] = Frag(q.x[j][0], q.x[j][1]), sc[j] = q.xs[j] * q.ws;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const Frag w(q.w[i][0], q.w[i][1]);
      f32x4 d[TI];
#pragma unroll
      for (int j = 0; j < TI; ++j) d[j] = product(w, x[j]);
#pragma unroll
      for (int j = 0; j < TI; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[j][e], sc[j], acc[i][j][e]);
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
  // every wave adds up its share of the groups of 16 x 16, waves in order
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < TI; ++j) sums[wave][i * TI + j][lane] = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int m = wave; m < NI * TI; m += KS) {
    f32x4 v = sums[0][m][lane];
#pragma unroll
    for (int k = 1; k < KS; ++k) v += sums[k][m][lane];
    store4<OUT>(a, t0 + m % TI * 16 + col, n0 + m / TI * 16 + g * 4, v);
  }
}

// Dynamic LDS above 64 KiB has to be asked for.
template <class Kernel>
hipError_t allow_lds(Kernel kernel, int64_t bytes) {
  if (bytes <= 64 * 1024) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

template <int OUT>
hipError_t launch_ring(const LinearArgs& a, hipStream_t st) {
  const int64_t lds = ring_lds(a.T, (a.K + kBlock - 1) / kBlock);
  const hipError_t e = allow_lds(ring_kernel<OUT>, lds);
  if (e != hipSuccess) return e;
  const int groups = ((a.N + 15) / 16 + kRingWaves - 1) / kRingWaves;
  ring_kernel<OUT><<<groups < 256 ? groups : 256, kRingWaves * 64, lds, st>>>(a);
  return hipGetLastError();
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

template <int NI, int TI, int KS, int OUT>
hipError_t launch_direct(const LinearArgs& a, hipStream_t st) {
  const int tiles = ((a.N + NI * 16 - 1) / (NI * 16)) * ((a.T + TI * 16 - 1) / (TI * 16));
  const int lds = KS * NI * TI * 1024;
  const hipError_t e = allow_lds(direct_kernel<NI, TI, KS, OUT>, lds);
  if (e != hipSuccess) return e;
  direct_kernel<NI, TI, KS, OUT><<<tiles, KS * 64, lds, st>>>(a);
  return hipGetLastError();
}

// Which kernel.  Times are of T x N x K in us, weights from HBM.
template <int OUT>
hipError_t launch(const LinearArgs& a, hipStream_t st) {
  auto tiles = [&](int bn, int bt) {
    return int64_t((a.N + bn - 1) / bn) * ((a.T + bt - 1) / bt);
  };
  auto rounds = [](int64_t n, int slots) { return (n + slots - 1) / slots; };
  // The ring needs tiles of 16 rows for more than half of its 2048 waves, and
  // tokens that fit LDS: 16 x 25,000 x 2048 takes 11.8 (16.6 direct), 1 x
  // 20,000 x 8192 37 (39), 1 x 16,384 x 4096 20 (16).
  if (a.T <= 16 && a.N >= 1250 * 16 && ring_lds(a.T, (a.K + kBlock - 1) / kBlock) <= kMaxLds)
    return launch_ring<OUT>(a, st);
  // A CU takes in no more than about 30 GB/s of what comes from HBM, however
  // many of its waves ask: the finest workgroups of which each CU gets at most
  // one.  32 x 1024 x 4096: 7.0 with 16 x 16, 11.5 with 32 x 32; 200 x 1000 x
  // 8000: 15 with 32 x 32 (27 as tiles of 64 x 64 through LDS); 500 x 1000 x
  // 2000: 7.3 with 64 x 32 (9.7); 777 x 1000 x 2000, 400 of them: 12.6 (10.1).
  if (tiles(16, 16) <= 256) return launch_direct<1, 1, 8, OUT>(a, st);
  if (tiles(32, 16) <= 256) return launch_direct<2, 1, 8, OUT>(a, st);
  if (a.T <= 16) {
    // 16 x 16,384 x 4096: 16.8 with 64 rows, 17.8 with 32; 1 x 20,000 x 8192
    // (the ring's without room): 46 with 64, 38 with 32
    if (tiles(64, 16) <= 256) return launch_direct<4, 1, 8, OUT>(a, st);
    return launch_direct<2, 1, 8, OUT>(a, st);
  }
  if (tiles(32, 32) <= 256) return launch_direct<2, 2, 8, OUT>(a, st);
  if (tiles(64, 32) <= 256) return launch_direct<4, 2, 8, OUT>(a, st);
  // Tiles through LDS.  One tile of tokens: narrow ones, three stages, several
  // workgroups per CU (32 x 151,936 x 2048: 61-66, as 64 x 64 88-95; 64 x
  // 151,936 x 2048: 76-79 with 128 rows, 83-88 with 64).  More rows per tile
  // only where that leaves no CU with more of them to do (64 x 40,000 x 4096:
  // 47-50 with 64 rows, 47-51 with 128).
  if (a.T <= 32) {
    // up to two per CU: two groups of waves each (25,000 rows, K 4096: 26 and 34)
    if (tiles(64, 32) <= 512) return launch_tile<64, 32, 2, 1, 3, 2, OUT, true>(a, st);
    return launch_tile<64, 32, 2, 1, 3, 1, OUT, true>(a, st);
  }
  if (a.T <= 64) {
    if (tiles(64, 64) > 512) {
      if (2 * rounds(tiles(128, 64), 256) <= rounds(tiles(64, 64), 256))
        return launch_tile<128, 64, 2, 2, 3, 1, OUT, true>(a, st);
      return launch_tile<64, 64, 2, 2, 3, 1, OUT, true>(a, st);
    }
  } else {
    if constexpr (OUT == MOE_W_BF16) {
      // a round of 256 tiles of 256 x 256 costs 1.6 of 512 of 128 x 128 (32,768
      // x 4096 x 2048: 330 and 413; 3000 x 4096 x 4096: 81 and 89, 500 x 40,000 x
      // 4096: 179 and 161)
      if (8 * rounds(tiles(256, 256), 256) <= 5 * rounds(tiles(128, 128), 512))
        return launch_tile<256, 256, 2, 4, 2, 1, OUT>(a, st);
    } else {
      // 4096 x 4096 x 4096: 146 and 157; 3000 x 4096 x 4096: 133 and 116
      if (2 * rounds(tiles(256, 128), 256) <= rounds(tiles(128, 128), 256))
        return launch_tile<256, 128, 4, 2, 3, 1, OUT>(a, st);
    }
    if (tiles(128, 128) > 256) return launch_tile<128, 128, 2, 2, 2, 1, OUT>(a, st);
    if (tiles(128, 128) > 128) return launch_tile<128, 128, 2, 2, 2, 2, OUT>(a, st);
  }
  // few tiles: groups of waves that share the blocks (100 x 4096 x 4096: 14 with
  // four, 17 with two; 300 x 4096 x 4096, 320 tiles: 22 with two)
  if (tiles(64, 64) > 256) return launch_tile<64, 64, 2, 2, 2, 2, OUT>(a, st);
  return launch_tile<64, 64, 2, 2, 2, 4, OUT>(a, st);
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
