// Attention of a step's new tokens over the paged cache of their sequences.
//
// Per new token and query head, over the positions p it sees:
//   out = sum_p exp(s_p - m) v_p / sum_p exp(s_p - m),   s_p = scale * q . k_p
// in one pass: a running m, sum and weighted sum of values.
//
// Rows and tiles.  The G = Hq / Hkv query heads that share a key head are
// rows of one tile with it: row r of a tile is token r / G, head r % G, so
// that keys and values are read once for all of them.  A tile has QT tokens
// (QT * G <= RB RW rows: RB = 16 or 32 per wave, RW waves), and walks over the
// positions in steps of KW * KS: KW groups of waves take KS each.  Up to 32
// rows four waves take positions of their own, with no barrier between them;
// taller tiles share what they load.
//
// Products.  Scores are formed as S^T = K Q^T (32 x 32 x 16 bf16 products, or
// 16 x 16 x 32: positions are the instruction's rows, query rows its columns),
// so a lane holds 16 (8) of 32 positions of one query row: the row's maximum
// is its own and one (two) exchanges between lanes, and the factors that
// rescale a row are the lane's own.  The weights' order is already that of
// the second product's operand (O^T = V^T P^T) if its position 8 h + j (h =
// lane / RB, of g = 64 / RB) is taken to be 4 g (j / 4) + 4 h + j % 4: the order
// of a sum's terms is free as long as both operands agree, and the transposing
// LDS reads of V take four (16 bits) or any eight (8 bits) positions at a time.
//
// Weights are rounded to bf16 for the second product (V is bf16 itself), off
// by 2^-8 of a weight at most, and the sum that divides them is that of the
// rounded ones: what is left is at most 2^-8 of the weighted mean of |v -
// out|, and much less over many positions, whose roundings go either way.
// For 8-bit outputs, whose scales are fp32, a weight is the sum of two bf16
// numbers (half as much again to multiply: a prompt of 16,384 tokens, 32 / 4 heads
// of 128, takes 2890 us in place of 2140), and for up to 32 rows, where HBM is what
// counts, of three.  With an 8-bit cache codes become bf16 (exact), a position's
// key scale multiplies its scores and its value scale its weights before their
// rounding.  In both cases the sum is that of the unrounded weights.
//
// The running maximum is raised when a row's largest score passes it by 2^8 (bf16:
// to 2^8 above that score, when it passes it at all): most steps leave the
// output's registers alone.  With a bf16 cache no weight passes 1, so that a
// weighted sum stays finite as far as the values' own sum does; with an 8-bit one
// weights are up to 2^8, as their products with small value scales would
// otherwise be subnormal bf16 numbers (scales of 2^-122: off by 11 %).  It is
// -infinity as long as a row has seen no position (then the row is zeros), and
// at least kLowest behind that: a row of NaN scores, or of -infinity alone, is
// NaN as its formula's 0 / 0 is, in whole tiles and in cut ones.
//
// Work.  All tiles' steps form one line (sequence, key head, pairs of the
// first and the last query tile, the second and the last but one ..., whose
// steps together are about the same whatever the mask), cut into equal runs,
// one per workgroup: a decode batch of any lengths, one long text and a
// prompt fill the GPU alike.  A workgroup finds its run from the lengths
// alone.  Tiles that are cut leave their parts (fp32, unnormalised) in the
// workspace and join_kernel adds them up in order.
//
// What bounds it (16 query and 2 key heads of 256): decode HBM (64 x 8192
// positions: 197 us, 5.4 TB/s; 5.18 is a copy's rate), a prompt the products and
// exponentials (16,384 tokens: 2050-2230 us, 990-1,070 TFLOP/s; an 8192^3
// library product 1,176), one token at 4097 a chain of loads and two launches
// (15.0 us).  Heads of 64 have as many exponentials, masks and roundings per
// score for a quarter of the products: vector instructions are issued in 54 % of
// a prompt's cycles, matrix instructions busy in 30 % (256: 43 and 48).

#include <hip/hip_runtime.h>

#include <type_traits>

#include "kernels.h"

namespace moe {
namespace {

typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(2))) int i32x2;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;
typedef uint32_t __attribute__((aligned(1))) u32_any;

#define MOE_LDS __attribute__((address_space(3)))

constexpr int kCus = 256;
constexpr int kMaxLds = 160 * 1024;
constexpr int kIds = 1024;                          // page numbers a workgroup holds at a time
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleFloor = 448.0f * 0x1p-126f;   // keeps every scale a normal number
constexpr float kRaise = 8.0f;                      // log2 of how far a row's maximum is let grow
constexpr float kLowest = -3.402823466e38f;         // maximum of a row that has seen no finite score
constexpr int kMaxGrid = 2 * kCus;

__device__ const u32x4 kZeros = {0u, 0u, 0u, 0u};   // what a position that is not there reads

// ---- loads straight to LDS, and waits for them
//
// In assembly, because the compiler waits for all of them before the next
// read of any part of LDS.  vmcnt counts in the order of issue, the
// compiler's own loads and stores among them, so the waits here are only
// ever longer than need be.  A load writes no register.  Reads of what they
// fill stay behind a wait that clobbers memory, and the loads stay behind
// the wait or barrier after the last reads of what they overwrite, as
// volatile assembly keeps its order.  The s_nop: 5 wait states between a
// vector write of a scalar operand and its use here.
#pragma clang diagnostic ignored "-Winline-asm"     // M0 among the clobbered registers

__device__ __forceinline__ void to_lds16(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "m0");
}
// From a scalar base and 32-bit offsets.
__device__ __forceinline__ void to_lds16(const uint8_t* base, uint32_t at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(at), "s"(base) : "m0");
}
__device__ __forceinline__ void to_lds4(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "m0");
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N <= 63, "vmcnt");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// This wave's reads of LDS have ended.
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// A barrier that leaves loads and stores under way.
__device__ __forceinline__ void barrier_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
__device__ __forceinline__ uint32_t lds_address(const MOE_LDS uint8_t* p) {
  return __builtin_amdgcn_readfirstlane(uint32_t(reinterpret_cast<uintptr_t>(p)));
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// Nothing is moved across by the compiler, which would read a product's
// operand right before it to save registers.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// The lane, computed anew: what a step derives from it is then not kept in
// registers from step to step (heads of 256 leave none).
__device__ __forceinline__ int lane_now() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
  return l;
}

// Eight e4m3 codes as bf16 (exact).
__device__ __forceinline__ bf16x8 from_codes(i32x2 c) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, false));
    r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, true));
  }
  return __builtin_bit_cast(bf16x8, r);
}

__device__ __forceinline__ bf16x8 operand(i32x2 c) { return from_codes(c); }
__device__ __forceinline__ bf16x8 operand(bf16x8 v) { return v; }

// The value of lane ^ 32 and the lane's own, in one order for both.
__device__ __forceinline__ f32x2 both_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f32x2{__uint_as_float(r[0]), __uint_as_float(r[1])};
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// ---- the line of work

// Quotient of two whole numbers, 0 <= a < 2^53, 0 < b < 2^53.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (__builtin_expect(((a | b) >> 32) == 0, 1)) return uint32_t(a) / uint32_t(b);
  int64_t q = int64_t(double(a) / double(b));
  const int64_t r = a - q * b;
  if (r < 0) --q;
  if (r >= b) ++q;
  return q;
}

struct Seq {
  int row0, n;          // its rows
  int off;              // position of its first new token
  int len;              // positions that may be there
  int nq;               // query tiles
  int most;             // steps of the longest
  int64_t pair, mid;    // steps set aside for a pair of tiles and for an unpaired one in the middle
  int64_t head;         // for a key head
};

template <int STEP>
__device__ __forceinline__ int tile_steps(const AttnArgs& a, const Seq& s, int qt, int* k0) {
  const int t0 = qt * a.QT, t1 = min(s.n, t0 + a.QT);
  const int end = min(max(s.off + t1, 0), s.len);
  const int start = a.window ? max(s.off + t0 - (a.window - 1), 0) : 0;
  *k0 = start / STEP;
  return max(1, (end + STEP - 1) / STEP - *k0);
}

template <int STEP>
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  Seq s;
  s.row0 = min(max(a.kv.q_off[b], 0), a.T);
  s.n = min(max(a.kv.q_off[b + 1], s.row0), a.T) - s.row0;
  const int len = min(max(a.kv.kv_len[b], 0), 1 << 30);
  s.off = len - s.n;
  s.len = min(len, a.kv.max_pages << a.kv.page_shift);
  s.nq = s.n <= a.QT ? (s.n > 0 ? 1 : 0) : (s.n + a.QT - 1) / a.QT;
  s.pair = s.mid = s.head = 0;
  s.most = 0;
  if (!s.n) return s;
  int64_t most = (s.len + STEP - 1) / STEP;
  if (a.window) most = min(most, (int64_t(a.window) + a.QT) / STEP + 2);
  s.most = int(max(most, int64_t(1)));
  if (s.nq > 1) {
    s.pair = 2 * int64_t(s.most);
    // tiles qt and nq - 1 - qt end at positions that add up to the same
    if (s.off >= 0) s.pair = min(s.pair, (2 * int64_t(s.off) + int64_t(s.nq + 1) * a.QT) / STEP + 2);
  }
  int k0;
  if (s.nq & 1) s.mid = tile_steps<STEP>(a, s, s.nq / 2, &k0);
  s.head = (s.nq / 2) * s.pair + s.mid;
  return s;
}

__device__ __forceinline__ int64_t lane_of(int64_t v, int lane) {
  return (int64_t(__builtin_amdgcn_readlane(int(v >> 32), lane)) << 32) |
         uint32_t(__builtin_amdgcn_readlane(int(v), lane));
}
__device__ __forceinline__ Seq lane_of(const Seq& s, int lane) {
  Seq r;
  r.row0 = __builtin_amdgcn_readlane(s.row0, lane);
  r.n = __builtin_amdgcn_readlane(s.n, lane);
  r.off = __builtin_amdgcn_readlane(s.off, lane);
  r.len = __builtin_amdgcn_readlane(s.len, lane);
  r.nq = __builtin_amdgcn_readlane(s.nq, lane);
  r.most = __builtin_amdgcn_readlane(s.most, lane);
  r.pair = lane_of(s.pair, lane);
  r.mid = lane_of(s.mid, lane);
  r.head = lane_of(s.head, lane);
  return r;
}

// Where a workgroup's run begins and ends.
struct Run {
  int64_t total;        // steps of the line
  int64_t length;       // of every run
  bool whole;           // tiles are not cut: a run has those that begin in it
  int b;                // sequence of the first step
  int64_t r;            // its place in the sequence's part of the line
  Seq s;
};

// By every wave for itself (no barrier, no LDS): a lane has neighbouring
// sequences.
template <class S>
__device__ __forceinline__ Run find_run(const AttnArgs& a, int me) {
  const int lane = threadIdx.x & (kWave - 1);
  const int each = (a.kv.B + kWave - 1) / kWave;
  Run run;
  Seq mine;
  int64_t c = 0;
  int n = 0, most = 0;
  for (int i = 0; i < each; ++i) {
    const int b = lane * each + i;
    mine = seq_of<S::kStep>(a, min(b, a.kv.B - 1));
    if (b < a.kv.B) {
      c += a.kv.Hkv * mine.head;
      n += mine.nq;
      most = max(most, mine.most);
    }
  }
  int64_t upto = c;
  for (int d = 1; d < kWave && d < a.kv.B; d <<= 1) {
    const int64_t y = __shfl_up(upto, d, kWave);
    if (lane >= d) upto += y;
    n += __shfl_down(n, d, kWave);       // (lane 0 gets them all)
    most = max(most, __shfl_down(most, d, kWave));
  }
  run.total = lane_of(upto, min(a.kv.B, kWave) - 1);
  const int64_t tiles = int64_t(__builtin_amdgcn_readlane(n, 0)) * a.kv.Hkv;
  most = __builtin_amdgcn_readlane(most, 0);
  run.length = quotient(run.total + a.grid - 1, a.grid);
  // A cut tile's parts cost about kCut steps each to leave and to join.  Cut
  // if the longest tile, or as many average ones as a workgroup gets, takes
  // longer than equal runs and two cuts.
  const int64_t rounds = quotient(tiles + a.grid - 1, a.grid);
  run.whole = most <= run.length + 2 * S::kCut &&
              rounds * run.total <= (run.length + 2 * S::kCut) * max(tiles, int64_t(1));
  if (!run.whole) run.length = max(run.length, int64_t(S::kLeast));
  const int64_t x = me * run.length;
  run.b = 0, run.r = 0;
  if (x >= run.total) return run;
  const int at = __builtin_ctzll(__ballot(x < upto));
  run.b = at * each;
  run.r = x - lane_of(upto, at) + lane_of(c, at);
  if (each == 1)
    run.s = lane_of(mine, at);
  else
    run.s = seq_of<S::kStep>(a, run.b);
  return run;
}

// What join_kernel needs of the tile that runs through the start of a
// workgroup's run, at the first such start of a tile.
struct Joint {
  int32_t first;        // the workgroup with the first part (its second slot; the others': their first)
  int32_t row0, tokens, head;
};
// The number of its parts, 0: nothing to join here; then the Joints.
__device__ __forceinline__ int32_t* joint_parts(const AttnArgs& a) { return static_cast<int32_t*>(a.joints); }
__device__ __forceinline__ Joint* joint_at(const AttnArgs& a, int i) {
  return reinterpret_cast<Joint*>(joint_parts(a) + kMaxGrid) + i;
}

// A token's output, four columns per lane (D / 4 lanes a row).
__device__ __forceinline__ void store_row4(const AttnArgs& a, int64_t row, int head, int D, int col, f32x4 v) {
  if (a.out) {
    const u32x2 p = {pack2(v[0], v[1]), pack2(v[2], v[3])};
    *reinterpret_cast<u32x2_any*>(a.out + row * a.out_stride + int64_t(head) * D + col) = p;
  }
  if (a.x8) {
    // 128 columns share a scale: 32 lanes
    float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
    m = fmaxf(m, dpp_f32<0xB1>(m));
    m = fmaxf(m, dpp_f32<0x4E>(m));
    m = fmaxf(m, dpp_f32<0x141>(m));
    m = fmaxf(m, dpp_f32<0x140>(m));
    m = fmaxf(m, __shfl_xor(m, 16, kWave));
    const float s = fmaxf(m, kScaleFloor) / kE4m3Max;
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] / s, v[1] / s, 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] / s, v[3] / s, c, true);
    const int64_t at = (row * a.Hq + head) * D + col;
    *reinterpret_cast<u32_any*>(a.x8 + at) = uint32_t(c);
    if (col % 128 == 0) a.x8_scale[at / 128] = s;
  }
}

// ---- the kernel

// PARTS: bf16 numbers that a weight is the sum of.
template <int D_, bool F8_, int RB_, int RW_, int KW_, int KS_, int NS_, int PARTS_>
struct Shape {
  static constexpr int D = D_, RB = RB_, RW = RW_, KW = KW_, KS = KS_, NS = NS_;
  static constexpr int kParts = PARTS_;
  static constexpr bool F8 = F8_;
  static constexpr int kWaves = RW * KW, kThreads = kWaves * kWave;
  static constexpr int kRows = RB * RW;
  static constexpr int kGroups = 64 / RB;                   // lanes of a row
  static constexpr int kStep = KW * KS;
  static constexpr int kPitch = D * (F8 ? 1 : 2);           // bytes of a position's row
  static constexpr int kChunks = kPitch / 16;
  static constexpr int kArea = KS * kPitch;                 // keys (or values) of a group's step
  static constexpr int kLoads = kArea / 1024;               // 1 KiB loads for it
  static constexpr int kRing = KW * NS * 2 * kArea;
  static constexpr int kScales = F8 ? KW * (NS + 1) * 2 * KS * 4 : 0;
  // columns of an epilogue's round (a wave's rows go through LDS)
  static constexpr int kCols = D < 128 || RW == 1 ? D : 128;
  static constexpr int kOutPitch = kCols + 4;               // (rows 4 banks apart)
  static constexpr int kOut = kWaves * RB * kOutPitch * 4;
  static constexpr int kData = kRing + kScales > kOut ? kRing + kScales : kOut;
  static constexpr int kLds = kData + kIds * 4 + kWaves * RB * 8;
  static constexpr int kPerCu = kMaxLds / (kLds + 256) >= 2 && kThreads <= 256 ? 2 : 1;
  static constexpr int kRowsAt = 64 / kChunks;              // positions of a 1 KiB load
  static constexpr int kAhead = 4;                          // operand reads ahead of their products
  // In steps: what a cut costs each side (the tile's rows in fp32 out and in),
  // and the shortest run if tiles are cut.
  static constexpr int kCut = RW, kLeast = RW;
  static_assert(kLds + 256 <= kMaxLds && (RW == 1 || NS >= 2) && (KS == 32 || KS == 64), "shape");
  static_assert(RW == 1 || 2 * kLoads % RW == 0, "loads");

  // Permutations of a row's 16-byte chunks in LDS (row parts of 256 bytes),
  // so that what is read together meets no bank twice: keys, 16 rows of one
  // chunk; values, with r0, r1 ... the bits of a row: in 16 bits 4 rows of 4
  // chunks (32 query rows) or 8 of 2 (16), told apart by r0 r1 and r0 r1 r2; in
  // 8 bits 8 rows of 2 chunks, by r0 r1 r3, or 16 of one, by r0 r1 r2 r4.  All
  // are sums of bits: of a row's parts, the sum of theirs.
  static __device__ __forceinline__ int key_swizzle(int row) {
    return kPitch >= 256 ? row & 15 : kPitch == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
  }
  static __device__ __forceinline__ int value_swizzle(int row) {
    const int r2 = (row >> 2) & 1;
    if (!F8) return kPitch >= 256 ? (row & 3) << 2 | r2 << 1 : (row & 2) << 1 | r2 << 1;
    const int r34 = ((row >> 3) ^ (row >> 4)) & 1;
    if (kPitch == 256) return r34 << 3 | (row & 3) << 1 | r2;
    if (kPitch == 128) return r34 << 2 | (row & 2) | r2;
    return r34 << 1 | r2;
  }
};

// One product of 16 or 32 rows, and what a lane holds of its result.
template <int RB>
struct Product;
template <>
struct Product<32> {
  typedef f32x16 Acc;
  static __device__ __forceinline__ Acc add(bf16x8 x, bf16x8 y, Acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, c, 0, 0, 0);
  }
  // Maximum (sum) over the lanes of a row.
  static __device__ __forceinline__ float row_max(float v) {
    const f32x2 h = both_halves(v);
    return fmaxf(h[0], h[1]);
  }
  static __device__ __forceinline__ float row_sum(float v) {
    const f32x2 h = both_halves(v);
    return h[0] + h[1];
  }
};
template <>
struct Product<16> {
  typedef f32x4 Acc;
  static __device__ __forceinline__ Acc add(bf16x8 x, bf16x8 y, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
  }
  static __device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, kWave));
    return Product<32>::row_max(v);
  }
  static __device__ __forceinline__ float row_sum(float v) {
    v += __shfl_xor(v, 16, kWave);
    return Product<32>::row_sum(v);
  }
};

template <class S>
__global__ __launch_bounds__(S::kThreads, S::kPerCu * S::kThreads / 256) void attention_kernel(const AttnArgs a) {
  constexpr int D = S::D, RB = S::RB, RW = S::RW, KW = S::KW, KS = S::KS, NS = S::NS, STEP = S::kStep;
  // A product's inner length is KK: 16 columns of 32 rows or 32 of 16.  A lane's
  // EACH results of a product are rows (positions, columns) place(e) of its RB.
  constexpr int GROUPS = S::kGroups, KK = 8 * GROUPS, EACH = RB * RB / 64;
  constexpr int NB = KS / RB, NP = KS / KK;       // products for a step's positions: scores, values
  using P = Product<RB>;
  auto place = [](int e) { return e / 4 * (4 * GROUPS) + e % 4; };     // (and 4 times the lane's group)
  constexpr int PARTS = S::kParts;
  constexpr bool F8 = S::F8;
  constexpr int AHEAD = S::kAhead;
  // Operands as they lie in LDS: 16 bytes of a key row (8-bit: two products'),
  // 8 positions of a value column.
  using KeyPart = std::conditional_t<F8, i32x4, bf16x8>;
  using ValuePart = std::conditional_t<F8, i32x2, bf16x8>;
  constexpr int PITCH = S::kPitch, BANKS = PITCH < 256 ? PITCH : 256;   // (a row's part that chunks are permuted in)
  extern __shared__ __align__(256) uint8_t smem[];
  MOE_LDS uint8_t* const lds = (MOE_LDS uint8_t*)smem;
  int32_t* const ids = reinterpret_cast<int32_t*>(smem + S::kData);
  f32x2* const stats = reinterpret_cast<f32x2*>(smem + S::kData + kIds * 4);   // [waves][RB]: maximum, sum

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = wave / RW, rw = wave % RW;
  const int col = lane % RB, part_of_row = lane / RB;
  // (heads of 256 leave no registers for what a step derives from it)
  auto lane_at = [&] { return D == 256 ? lane_now() : lane; };
  // neighbouring runs on one XCD (workgroups go to the 8 in turn): they share keys and values
  const int me = int(blockIdx.x & 7) * (a.grid >> 3) + int(blockIdx.x >> 3);

  const Run run = find_run<S>(a, me);
  const int64_t x0 = me * run.length, x1 = min(run.total, x0 + run.length);
  if (x0 >= x1) {
    if (threadIdx.x == 0) joint_parts(a)[me] = 0;
    return;
  }
  int64_t x = x0, r = run.r;
  int b = run.b;
  Seq s = run.s;

  while (x < x1) {
    if (r >= a.kv.Hkv * s.head) {
      r -= a.kv.Hkv * s.head;
      s = seq_of<STEP>(a, ++b);
      continue;
    }
    // which tile, and from which of its steps
    const int h = a.kv.Hkv == 1 ? 0 : int(quotient(r, s.head));
    const int64_t in_head = r - h * s.head;
    const int pairs = s.nq / 2;
    int qt, tile0, steps;           // query tile; its first step; its number of steps
    int from;                       // steps done by the workgroups before
    if (in_head >= pairs * s.pair) {
      qt = pairs;
      steps = tile_steps<STEP>(a, s, qt, &tile0);
      from = int(in_head - pairs * s.pair);
    } else {
      qt = int(quotient(in_head, s.pair));
      from = int(in_head - qt * s.pair);
      steps = tile_steps<STEP>(a, s, qt, &tile0);
      if (from >= steps) {
        from -= steps;
        qt = s.nq - 1 - qt;
        steps = tile_steps<STEP>(a, s, qt, &tile0);
        if (__builtin_expect(from >= steps, 0)) {      // what the pair does not need
          if (threadIdx.x == 0 && x == x0) joint_parts(a)[me] = 0;
          const int64_t skip = s.pair - (in_head - int64_t(s.nq - 1 - qt) * s.pair);
          x += skip, r += skip;
          continue;
        }
      }
    }
    const int t0 = qt * a.QT, nt = min(s.n - t0, a.QT);
    if (x == x0 && threadIdx.x == 0) {
      int parts = 0;
      // (the tile's first cut is this one)
      if (!run.whole && from > 0 && x - from >= x0 - run.length) {
        parts = int(quotient(x - from + steps - 1, run.length)) - (me - 1) + 1;
        Joint j;
        j.first = me - 1;
        j.row0 = s.row0 + t0;
        j.tokens = nt;
        j.head = h;
        *joint_at(a, me) = j;
      }
      joint_parts(a)[me] = parts;
    }
    int take = steps - from;
    if (run.whole) {
      if (from > 0) {               // the run before has it
        x += take, r += take;
        continue;
      }
    } else if (take > x1 - x) {
      take = int(x1 - x);
    }
    const bool whole = take == steps;
    const int slot = me * 2 + (from == 0 ? 1 : 0);
    x += take, r += take;

    // ---- the tile's queries: this wave's rows, as the products' right operand
    const int lr = rw * RB + col;                       // this lane's row of the tile
    const int token = a.token_of(lr);
    const bool live = token < nt;
    const int rpos = live ? s.off + t0 + token : -1;    // the last position it sees
    const int rfirst = a.window ? max(rpos - (a.window - 1), 0) : 0;
    bf16x8 q[D / KK];
    {
      const uint16_t* qp = a.q + int64_t(s.row0 + t0 + (live ? token : 0)) * a.q_stride +
                           int64_t(h * a.G + (lr - token * a.G)) * D + part_of_row * (F8 ? 16 : 8);
      // (8-bit keys: a lane's 16 columns are two products')
#pragma unroll
      for (int i = 0; i < D / KK; ++i) {
        u32x4 v = {0u, 0u, 0u, 0u};
        const int c = F8 ? i / 2 * (2 * KK) + i % 2 * 8 : i * KK;
        if (live) v = *reinterpret_cast<const u32x4_any*>(qp + c);
        q[i] = __builtin_bit_cast(bf16x8, v);
      }
    }
    // what every row of this wave sees, and what any does
    const int wave_t1 = min(nt - 1, a.token_of(rw * RB + RB - 1)), wave_t0 = min(a.token_of(rw * RB), nt - 1);
    const bool wave_live = a.token_of(rw * RB) < nt;
    const int sees_all = s.off + t0 + wave_t0;                                    // up to here
    const int sees_any = wave_live ? s.off + t0 + wave_t1 : -1;
    const int from_all = a.window ? s.off + t0 + wave_t1 - (a.window - 1) : 0;     // from here
    const int from_any = a.window ? s.off + t0 + wave_t0 - (a.window - 1) : 0;

    typename P::Acc o[D / RB];
#pragma unroll
    for (int i = 0; i < D / RB; ++i)
#pragma unroll
      for (int j = 0; j < EACH; ++j) o[i][j] = 0.0f;
    float mref = -INFINITY, sum = 0.0f, lost = 0.0f;     // (what the sum's roundings lost)

    // ---- the positions, as far as the page numbers held in LDS reach
    constexpr int ELEM = F8 ? 1 : 2;
    const uint8_t* const kbase = a.kv.k + int64_t(h) * a.kv.head_stride * ELEM;
    const uint8_t* const vbase = a.kv.v + int64_t(h) * a.kv.head_stride * ELEM;
    const uint32_t page_bytes = uint32_t(a.kv.page_stride) * ELEM, slot_bytes = uint32_t(a.kv.slot_stride) * ELEM;
    const int shift = a.kv.page_shift;
    const bool one_page = (1 << shift) >= (RW == 1 ? 16 : S::kRowsAt) && slot_bytes <= 1u << 26;
    const int span = max(1, int(min(int64_t(kIds - 1) << shift, int64_t(1) << 30)) / STEP);
    for (int s0 = 0; s0 < take; s0 += span) {
      const int count = min(span, take - s0);
      const int step0 = tile0 + from + s0;
      const int page0 = int((int64_t(step0) * STEP) >> shift);
      const int pages = int(((int64_t(step0 + count) * STEP - 1) >> shift) - page0) + 1;
      barrier_lds();          // the ids, and all of LDS, have been used up
      for (int i = threadIdx.x; i < pages; i += S::kThreads) {
        int id = -1;
        if (page0 + i < a.kv.max_pages) id = a.kv.page_table[b * a.kv.table_stride + page0 + i];
        ids[i] = id >= 0 && id < a.kv.num_pages ? id : -1;
      }
      __syncthreads();

      // page of a position, or -1 if the position is not there
      auto page_of = [&](int pos) -> int { return pos < s.len ? ids[(pos >> shift) - page0] : -1; };
      auto slot_lds = [&](int st, bool value) -> MOE_LDS uint8_t* {
        return lds + ((kw * NS + st) * 2 + (value ? 1 : 0)) * S::kArea;
      };
      auto scales_of = [&](int i, bool value) -> MOE_LDS uint8_t* {
        return lds + S::kRing + ((kw * (NS + 1) + i % (NS + 1)) * 2 + (value ? 1 : 0)) * KS * 4;
      };
      // the lane's position (KS of them) of a step: its page, or -1
      auto pages_of = [&](int i) -> int { return page_of((step0 + i) * STEP + kw * KS + (lane_at() & (KS - 1))); };
      // Load j of step i's keys or values.  Where all positions are there and a
      // load's lie in one page, its base is the wave's (`even`).
      auto load = [&](int i, int j, bool value, bool even, int id_here, int l) {
        const int row0 = j * S::kRowsAt, pos0 = (step0 + i) * STEP + kw * KS + row0;
        const uint32_t to = lds_address(slot_lds(i % NS, value) + j * 1024);
        const int swz0 = value ? S::value_swizzle(row0) : S::key_swizzle(row0);
        // (row0's bits and those of the lane's row are apart, and so are their swizzles')
        const int lrow = l / S::kChunks;
        const int chunk = ((l % S::kChunks) ^ (value ? S::value_swizzle(lrow) : S::key_swizzle(lrow))) * 16;
        if (even) {
          const uint32_t id = __builtin_amdgcn_readlane(id_here, row0);
          const uint8_t* base = (value ? vbase : kbase) + uint64_t(id) * page_bytes +
                                uint64_t(uint32_t(pos0 & ((1 << shift) - 1))) * slot_bytes;
          to_lds16(base, (chunk ^ (swz0 * 16)) + uint32_t(lrow) * slot_bytes, to);
        } else {
          const int pos = pos0 + lrow, id = page_of(pos);
          const uint8_t* p = (value ? vbase : kbase) + uint64_t(uint32_t(id)) * page_bytes +
                             uint64_t(uint32_t(pos & ((1 << shift) - 1))) * slot_bytes + (chunk ^ (swz0 * 16));
          if (id < 0) p = reinterpret_cast<const uint8_t*>(&kZeros);
          to_lds16(p, to);
        }
      };
      auto load_scales = [&](int i, bool value) {
        // (32 positions: the lower half of the wave keys', the upper values')
        const int l = lane_at();
        const bool up = KS == 32 ? l >= 32 : value;
        const int row = l & (KS - 1);
        const int pos = (step0 + i) * STEP + kw * KS + row;
        const int id = page_of(pos);
        const float* p = (up ? a.kv.v_scale : a.kv.k_scale) +
                         ((int64_t(id) << shift) + (pos & ((1 << shift) - 1))) * a.kv.Hkv + h;
        if (id < 0) p = reinterpret_cast<const float*>(&kZeros);
        to_lds4(p, lds_address(scales_of(i, KS == 32 ? false : value)));
      };
      constexpr int kScaleLoads = F8 ? 1 : 0;      // with the keys of a wave's own step
      auto load_own = [&](int i, bool value) {
        const int id = pages_of(i), l = lane_at();
        if (one_page && __ballot(id < 0) == 0) {
          // 16 positions from one base (a page lookup for every load: one token
          // 15.9 us instead of 15.0, four 29.2 instead of 27.8)
          const int lrow = l / S::kChunks;
          const int chunk = ((l % S::kChunks) ^ (value ? S::value_swizzle(lrow) : S::key_swizzle(lrow))) * 16;
          const uint32_t from = uint32_t(lrow) * slot_bytes;
          const uint32_t to = lds_address(slot_lds(i % NS, value));
#pragma unroll
          for (int g = 0; g < KS / 16; ++g) {
            const int pos0 = (step0 + i) * STEP + kw * KS + g * 16;
            const uint8_t* base = (value ? vbase : kbase) +
                                  uint64_t(uint32_t(__builtin_amdgcn_readlane(id, g * 16))) * page_bytes +
                                  uint64_t(uint32_t(pos0 & ((1 << shift) - 1))) * slot_bytes;
#pragma unroll
            for (int j = 0; j < 16 / S::kRowsAt; ++j) {
              const int row0 = g * 16 + j * S::kRowsAt;
              const int swz0 = value ? S::value_swizzle(row0) : S::key_swizzle(row0);
              to_lds16(base, (chunk ^ (swz0 * 16)) + from, to + row0 * PITCH);
              base += uint32_t(S::kRowsAt) * slot_bytes;
            }
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < S::kLoads; ++j) load(i, j, value, false, id, l);
        }
        if (F8 && !value) load_scales(i, false);
      };
      // RW waves share a step's loads
      constexpr int kShare = 2 * S::kLoads / RW;
      auto load_shared = [&](int i) {
        const int id = pages_of(i), l = lane_at();
        if (one_page && __ballot(id < 0) == 0) {
#pragma unroll
          for (int j = 0; j < kShare; ++j) {
            const int g = rw * kShare + j;
            load(i, g % S::kLoads, g >= S::kLoads, true, id, l);
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < kShare; ++j) {
            const int g = rw * kShare + j;
            load(i, g % S::kLoads, g >= S::kLoads, false, id, l);
          }
        }
        if (F8) load_scales(i, KS == 64 && (rw & 1));      // (by every wave: one count of loads for all)
      };

      if constexpr (RW == 1) {
        for (int i = 0; i < NS && i < count; ++i) {
          load_own(i, false);
          load_own(i, true);
        }
      } else {
        for (int i = 0; i < NS - 1 && i < count; ++i) load_shared(i);
      }

      for (int i = 0; i < count; ++i) {
        if constexpr (RW == 1) {
          // behind these keys: NS values and NS - 1 keys, if the end is not near
          if (i + NS <= count)
            wait_loads<(2 * NS - 1) * S::kLoads + (NS - 1) * kScaleLoads>();
          else
            wait_loads<0>();
        } else {
          // behind this step's loads: those of NS - 2 steps, if the end is not near
          if (i + NS - 2 < count)
            wait_loads<(NS - 2) * (kShare + kScaleLoads)>();
          else
            wait_loads<0>();
          barrier_lds();
        }
        const int pos0 = (step0 + i) * STEP + kw * KS;      // this group's positions
        MOE_LDS uint8_t* const kl = slot_lds(i % NS, false);
        MOE_LDS uint8_t* const vl = slot_lds(i % NS, true);

        // which of the positions are there
        const int l = lane_at(), col = l % RB, group = l / RB;
        uint32_t there[KS / 32];
        bool all = true;
#pragma unroll
        for (int n = 0; n < KS / 32; ++n) {
          there[n] = uint32_t(__ballot(page_of(pos0 + n * 32 + (l & 31)) >= 0));
          all = all && there[n] == 0xFFFFFFFFu;
        }
        const bool any = pos0 <= sees_any && pos0 + KS > from_any;
        typename P::Acc sc[NB];
        float least = kLowest;      // -infinity: this lane's row sees none of the positions
        if (any) {
          // chunk c of a row lies at c ^ key_swizzle(row): with the lane's part
          // of c in the address, the rest of it is an exclusive or (below 256
          // bytes) and an offset; RB rows further the permutation is the same
          // or differs by key_swizzle(RB)
          const uint32_t at = uint32_t(reinterpret_cast<uintptr_t>(kl)) + col * PITCH +
                              (S::key_swizzle(col) ^ group) * 16;
          constexpr int ROW = D / KK / (F8 ? 2 : 1), COUNT = NB * ROW;      // reads
          __builtin_amdgcn_s_setprio(1);
          auto read = [&](int u) {
            const int n = u / ROW, k = u % ROW;
            const uint32_t x = k * 16 * GROUPS ^ (S::key_swizzle(n * RB) * 16);
            return *(MOE_LDS KeyPart*)(uintptr_t)((at ^ (x % BANKS)) + x / BANKS * BANKS + n * RB * PITCH);
          };
          KeyPart part[AHEAD];
#pragma unroll
          for (int u = 0; u < AHEAD && u < COUNT; ++u) part[u] = read(u);
          if constexpr (F8) {
            bf16x8 lo = from_codes(i32x2{part[0][0], part[0][1]}), hi;
            in_order();
#pragma unroll
            for (int u = 0; u < COUNT; ++u) {
              const int n = u / ROW, k = u % ROW * 2;
              if (k == 0) {
#pragma unroll
                for (int j = 0; j < EACH; ++j) sc[n][j] = 0.0f;
              }
              const KeyPart now = part[u % AHEAD];
              if (u + AHEAD < COUNT) part[u % AHEAD] = read(u + AHEAD);
              sc[n] = P::add(lo, q[k], sc[n]);
              hi = from_codes(i32x2{now[2], now[3]});
              in_order();
              sc[n] = P::add(hi, q[k + 1], sc[n]);
              if (u + 1 < COUNT) lo = from_codes(i32x2{part[(u + 1) % AHEAD][0], part[(u + 1) % AHEAD][1]});
              in_order();
            }
          } else {
            in_order();
#pragma unroll
            for (int u = 0; u < COUNT; ++u) {
              const int n = u / ROW, k = u % ROW;
              if (k == 0) {
#pragma unroll
                for (int j = 0; j < EACH; ++j) sc[n][j] = 0.0f;
              }
              const KeyPart now = part[u % AHEAD];
              if (u + AHEAD < COUNT) part[u % AHEAD] = read(u + AHEAD);
              sc[n] = P::add(now, q[k], sc[n]);
              in_order();
            }
          }
          if (F8) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
              for (int g = 0; g < EACH / 4; ++g) {
                const f32x4 w = *(MOE_LDS f32x4*)(scales_of(i, false) + (n * RB + place(4 * g) + 4 * group) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[n][4 * g + e] *= w[e];
              }
          }
          if (!all || pos0 + KS - 1 > sees_all || pos0 < from_all) {
            uint32_t some = 0;
#pragma unroll
            for (int n = 0; n < KS / 32; ++n) {
              // a bit for each of the 32 positions that this lane's row sees
              const int last = rpos - pos0 - n * 32, first = rfirst - pos0 - n * 32;
              uint32_t sees = last >= 31 ? ~0u : last < 0 ? 0u : (2u << last) - 1u;
              sees &= first <= 0 ? ~0u : first > 31 ? 0u : ~0u << first;
              sees &= there[n];
              some |= sees;
              sees >>= 4 * group;
#pragma unroll
              for (int m = 0; m < 32 / RB; ++m)
#pragma unroll
                for (int j = 0; j < EACH; ++j) {
                  const int k = n * (32 / RB) + m;
                  sc[k][j] = sees & (1u << (m * RB + place(j))) ? sc[k][j] : -INFINITY;
                }
            }
            least = some ? kLowest : -INFINITY;
          }
        }
        if constexpr (RW == 1) {
          wait_reads();
          if (i + NS < count) load_own(i + NS, false);
        } else if (i + NS - 1 < count) {
          load_shared(i + NS - 1);      // (not where all waves leave the barrier together)
        }
        bf16x8 p[PARTS][NP];
        if (any) {
          __builtin_amdgcn_s_setprio(0);
          float top = sc[0][0];
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int j = 0; j < EACH; ++j) top = fmaxf(top, sc[n][j]);
          top = fmaxf(P::row_max(top) * a.scale2, least);     // (NaN is no maximum)
          constexpr float ABOVE = F8 ? 0.0f : kRaise;
          if (__ballot(top > mref + (kRaise - ABOVE))) {
            // (a row by its own scores alone, whatever the rows beside it do)
            const float m = top > mref + (kRaise - ABOVE) ? top + ABOVE : mref;
            const float f = m == -INFINITY ? 1.0f : exp2_fast(mref - m);
            sum *= f, lost *= f;
#pragma unroll
            for (int n = 0; n < D / RB; ++n)
#pragma unroll
              for (int j = 0; j < EACH; ++j) o[n][j] *= f;
            mref = m;
          }
          const float m = mref == -INFINITY ? 0.0f : mref;
          float add = 0.0f;
          // eight weights at a time: a product's operand
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int e = n * 8 + j;
              w[j] = exp2_fast(fmaf(sc[e / EACH][e % EACH], a.scale2, -m));
            }
            if (F8 || PARTS > 1) add += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
            if (F8) {
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const f32x4 v = *(MOE_LDS f32x4*)(scales_of(i, KS != 32) +
                                                  ((KS == 32 ? 32 : 0) + n * KK + place(4 * g) + 4 * group) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[4 * g + e] *= v[e];
              }
            }
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
              u32x4 c;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float* const x = w + 2 * e;
                c[e] = pack2(x[0], x[1]);
                if (!F8 && PARTS == 1) add = dot2_bf16(c[e], 0x3F803F80u, add);
                x[0] -= __uint_as_float(c[e] << 16), x[1] -= __uint_as_float(c[e] & 0xFFFF0000u);
              }
              p[k][n] = __builtin_bit_cast(bf16x8, c);
            }
          }
          // a sum over a long text keeps what is small next to it
          const float y = add - lost, s = sum + y;
          lost = (s - sum) - y;
          sum = s;
        }
        if constexpr (RW == 1) {
          // behind these values: NS keys and NS - 1 values
          if (i + NS < count)
            wait_loads<(2 * NS - 1) * S::kLoads + NS * kScaleLoads>();
          else
            wait_loads<0>();
        }
        if (any) {
          // 16 lanes give the rows that the transposing read takes: 4 rows of 16
          // columns (16 bits), 8 of 16 (8 bits); the permutation as for keys
          const int li = l & 15, cols16 = RB == 32 ? (l >> 4) & 1 : 0;
          const int row = 4 * group + (F8 ? (li >> 3) * (4 * GROUPS) + ((li >> 1) & 3) : li >> 2);
          const int chunk = F8 ? cols16 : 2 * cols16 + ((li & 3) >> 1);
          const uint32_t at = uint32_t(reinterpret_cast<uintptr_t>(vl)) + row * PITCH +
                              (chunk ^ S::value_swizzle(row)) * 16 + (li & 1) * 8;
          constexpr int COLS = D / RB, COUNT = NP * COLS;
          __builtin_amdgcn_s_setprio(1);
          auto read = [&](int u) {
            constexpr int UNIT = F8 ? RB : 2 * RB;
            const int n = u / COLS;
            const uint32_t x = u % COLS * UNIT;
            auto from = [&](int r) {       // r rows further
              const uint32_t y = x ^ (S::value_swizzle(r) * 16);
              return (at ^ (y % BANKS)) + y / BANKS * BANKS + r * PITCH;
            };
            ValuePart v;
            if constexpr (F8) {
              v = __builtin_amdgcn_ds_read_tr8_b64_v2i32((MOE_LDS i32x2*)(uintptr_t)from(n * KK));
            } else {
              const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(uintptr_t)from(n * KK));
              const s16x4 hi =
                  __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(uintptr_t)from(n * KK + 4 * GROUPS));
              v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
            return v;
          };
          ValuePart part[AHEAD];
#pragma unroll
          for (int u = 0; u < AHEAD && u < COUNT; ++u) part[u] = read(u);
          bf16x8 vf = operand(part[0]);
          in_order();
#pragma unroll
          for (int u = 0; u < COUNT; ++u) {
            const int n = u / COLS, d = u % COLS;
            const bf16x8 now = vf;
            if (u + AHEAD < COUNT) part[u % AHEAD] = read(u + AHEAD);
#pragma unroll
            for (int k = PARTS - 1; k >= 0; --k) o[d] = P::add(now, p[k][n], o[d]);
            if (u + 1 < COUNT) vf = operand(part[(u + 1) % AHEAD]);
            in_order();
          }
        }
        if constexpr (RW == 1) {
          wait_reads();
          if (i + NS < count) load_own(i + NS, true);
        }
      }
    }

    // ---- the tile's end: rows through LDS, 128 columns at a time
    sum = P::row_sum(sum);
    barrier_lds();         // the steps' LDS has been used up
    float m = mref;
    float f = 1.0f;
    if constexpr (KW > 1) {
      if (part_of_row == 0) stats[wave * RB + col] = f32x2{mref, sum};
      barrier_lds();
      f32x2 st[KW];
#pragma unroll
      for (int k = 0; k < KW; ++k) st[k] = stats[(k * RW + rw) * RB + col], m = fmaxf(m, st[k][0]);
      sum = 0.0f;
#pragma unroll
      for (int k = 0; k < KW; ++k) sum += m == -INFINITY ? 0.0f : st[k][1] * exp2_fast(st[k][0] - m);
      f = m == -INFINITY ? 0.0f : exp2_fast(mref - m);
    }
    float* const part = a.parts + int64_t(slot) * S::kRows * (D + 2);
    if (whole)
      f = m == -INFINITY ? 0.0f : f / sum;
    else if (kw == 0 && part_of_row == 0)
      *reinterpret_cast<f32x2*>(part + S::kRows * D + lr * 2) = f32x2{m, sum};
    float* const mine_out = reinterpret_cast<float*>(smem) + wave * RB * S::kOutPitch;
    constexpr int kLanes = S::kCols / 4, kRowsAt = 64 / kLanes;     // lanes of a row, rows at a time
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += S::kCols) {
#pragma unroll
      for (int d = 0; d < S::kCols / RB; ++d)
#pragma unroll
        for (int g = 0; g < EACH / 4; ++g) {
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = o[c0 / RB + d][4 * g + e] * f;
          *reinterpret_cast<f32x4*>(mine_out + col * S::kOutPitch + d * RB + place(4 * g) + 4 * part_of_row) = v;
        }
      barrier_lds();
      // the KW waves of these rows take RB / KW of them each
#pragma unroll 1
      for (int i = 0; i < RB / KW; i += kRowsAt) {
        const int row = kw * (RB / KW) + i + lane / kLanes, c = (lane % kLanes) * 4;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KW; ++k)
          v += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(smem) +
                                               ((k * RW + rw) * RB + row) * S::kOutPitch + c);
        const int tr = rw * RB + row, tk = a.token_of(tr);
        if (whole) {
          if (tk < nt) store_row4(a, s.row0 + t0 + tk, h * a.G + tr - tk * a.G, D, c0 + c, v);
        } else {
          *reinterpret_cast<f32x4*>(part + tr * D + c0 + c) = v;
        }
      }
      barrier_lds();
    }
  }
}

// The parts of a cut tile, in order: out = sum_i exp2(m_i - m) o_i / sum_i
// exp2(m_i - m) l_i.  Every workgroup counts the cut tiles' rows and takes its
// share.  D / 4 lanes hold a row, four columns each: where there are many rows,
// they go through a row's parts by themselves; where there are few, all
// groups of lanes of a workgroup share a row's parts.
constexpr int kJoinThreads = 512;

template <int D>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const AttnArgs a, int rows) {
  constexpr int LANES = D / 4, GROUPS = kJoinThreads / LANES, AHEAD = 8;
  static_assert(kMaxGrid == kJoinThreads, "a thread per run");
  __shared__ int32_t upto[kMaxGrid];       // rows of the cut tiles up to this one
  __shared__ int32_t parts_of[kMaxGrid];
  __shared__ Joint joints[kMaxGrid];
  __shared__ int32_t waves[kJoinThreads / kWave];
  __shared__ f32x4 acc[kJoinThreads];
  __shared__ f32x2 stat[GROUPS];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  {
    int n = 0;
    if (int(threadIdx.x) < a.grid) {
      const int parts = joint_parts(a)[threadIdx.x];
      const Joint j = *joint_at(a, threadIdx.x);
      parts_of[threadIdx.x] = parts;
      joints[threadIdx.x] = j;
      if (parts > 0) n = min(j.tokens * a.G, rows);
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int y = __shfl_up(n, d, kWave);
      if (lane >= d) n += y;
    }
    if (lane == kWave - 1) waves[wave] = n;
    __syncthreads();
    for (int w = 0; w < wave; ++w) n += waves[w];
    upto[threadIdx.x] = n;
    __syncthreads();
  }
  const int total = upto[kMaxGrid - 1];
  const int sub = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const bool many = total > int(gridDim.x) * 2;
  const int split = many ? 1 : GROUPS;             // groups that share a row
  const int stride = many ? int(gridDim.x) * GROUPS : int(gridDim.x);
  for (int base = many ? int(blockIdx.x) * GROUPS : int(blockIdx.x); base < total; base += stride) {
    const int item = many ? base + group : base;
    const bool live = item < total;
    int at = 0;
    for (int d = kMaxGrid / 2; d; d >>= 1)
      if (upto[at + d - 1] <= item) at += d;
    at = min(at, kMaxGrid - 1);
    const Joint j = joints[at];
    const int parts = live ? parts_of[at] : 0;
    const int row = item - (at ? upto[at - 1] : 0);
    float m = -INFINITY, l = 0.0f;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = many ? 0 : group; p < parts; p += split * AHEAD) {
      f32x2 st[AHEAD];
      f32x4 w[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        st[k] = f32x2{-INFINITY, 0.0f};
        const int pk = p + k * split;
        if (pk < parts) {
          const int slot = (j.first + pk) * 2 + (pk == 0 ? 1 : 0);
          const float* part = a.parts + int64_t(slot) * rows * (D + 2);
          st[k] = *reinterpret_cast<const f32x2*>(part + rows * D + row * 2);
          w[k] = *reinterpret_cast<const f32x4*>(part + row * D + sub * 4);
        }
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const float top = fmaxf(m, st[k][0]);
        if (st[k][0] == -INFINITY) continue;
        const float f = exp2_fast(m - top), g = exp2_fast(st[k][0] - top);
        l = l * f + st[k][1] * g;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = v[e] * f + w[k][e] * g;
        m = top;
      }
    }
    if (!many) {
      __syncthreads();
      acc[threadIdx.x] = v;
      if (sub == 0) stat[group] = f32x2{m, l};
      __syncthreads();
      if (group == 0) {
        float top = -INFINITY;
#pragma unroll
        for (int p = 0; p < GROUPS; ++p) top = fmaxf(top, stat[p][0]);
        m = top, l = 0.0f;
        v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (top > -INFINITY) {
#pragma unroll
          for (int p = 0; p < GROUPS; ++p) {
            const float f = exp2_fast(stat[p][0] - top);
            l += stat[p][1] * f;
            const f32x4 w = acc[p * LANES + sub];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += w[e] * f;
          }
        }
      }
    }
    if (live && (many || group == 0)) {
      const float f = m == -INFINITY ? 0.0f : 1.0f / l;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= f;
      const int tk = a.token_of(row);
      store_row4(a, j.row0 + tk, j.head * a.G + row - tk * a.G, D, sub * 4, v);
    }
  }
}

// Dynamic LDS above 64 KiB has to be asked for.
template <class Kernel>
hipError_t allow_lds(Kernel kernel, int64_t bytes) {
  if (bytes <= 64 * 1024) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

// Rows of a tile for so many rows per sequence.
int rows_for(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256; }

constexpr size_t kJointBytes = kMaxGrid * (sizeof(int32_t) + sizeof(Joint));

size_t parts_bytes(int rows, int D) {
  return size_t(rows <= 128 ? kMaxGrid : kCus) * 2 * rows * (D + 2) * 4;
}

template <class S>
hipError_t launch_shape(AttnArgs a, hipStream_t st) {
  static_assert((S::kRows <= 128 ? kMaxGrid : kCus) >= kCus * S::kPerCu, "workspace");
  a.QT = S::kRows / a.G;
  a.joints = a.ws;
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + kJointBytes);
  a.inv_g = (65536 + a.G - 1) / a.G;
  // no more workgroups than steps there can be (a multiple of the 8 XCDs)
  const int64_t tiles = int64_t(a.T) / a.QT + a.kv.B;
  const int64_t steps = ((int64_t(a.kv.max_pages) << a.kv.page_shift) + S::kStep - 1) / S::kStep;
  const int64_t most = tiles * a.kv.Hkv * (steps + 2);
  const int64_t full = kCus * S::kPerCu;
  a.grid = int((most < full ? most + 7 : full) / 8 * 8);
  const auto kernel = attention_kernel<S>;
  const hipError_t e = allow_lds(kernel, S::kLds);
  if (e != hipSuccess) return e;
  kernel<<<a.grid, S::kThreads, S::kLds, st>>>(a);
  join_kernel<S::D><<<2 * kCus, kJoinThreads, 0, st>>>(a, S::kRows);
  return hipGetLastError();
}

template <int D, bool F8, int PARTS>
hipError_t launch(const AttnArgs& a, hipStream_t st) {
  // (an 8-bit cache needs half the LDS)
  constexpr int NS = D == 256 && !F8 ? 1 : 2, KS = D == 256 ? 32 : 64;
  const int64_t tokens = (int64_t(a.T) + a.kv.B - 1) / a.kv.B;
  // Tall tiles multiply at twice the rate of those of 64 rows, but cutting them
  // moves rows * D * 4 bytes per workgroup out and in again: only for steps of
  // many products (as far as the host can tell: the tables may be wider than
  // the texts are long).  In us with 64, 128 and 256 rows at the products in
  // brackets: 16 / 2 heads of 256, 512 tokens at 512 (1.1e9) 35, 61, 75, at 1024
  // (2.1e9) 43, 55, 59, at 2048 (4.3e9) 60, 65, 65, at 4096 (8.6e9) 92, 80, 81, 64 at
  // 32,000 (8.4e9) 100, 88, 82; 32 / 4 of 128, 512 at 1024 (2.1e9) 34, 34, 43, at 2048
  // (4.3e9) 43, 42, 42, 64 at 32,000 (8.4e9) 88, 64, 61; 15 / 5 of 64, 512 at 4096 (2e9)
  // 32, 32, 34.
  const int64_t cap = int64_t(a.kv.max_pages) << a.kv.page_shift;
  const int64_t seen = a.window && a.window < cap ? a.window : cap;
  const double work = double(a.T) * a.Hq * double(seen) * D;
  const int64_t tallest = work < 2.5e9 ? 64 : work < 5e9 ? 128 : 256;
  const int64_t rows = tokens * a.G < tallest ? tokens * a.G : tallest > a.G ? tallest : a.G;
  switch (rows_for(rows)) {
    case 16:
      return launch_shape<Shape<D, F8, 16, 1, 4, 32, NS, 3>>(a, st);
    case 32:
      return launch_shape<Shape<D, F8, 32, 1, 4, 32, NS, 3>>(a, st);
    case 64:
      return launch_shape<Shape<D, F8, 32, 2, 2, 32, 2, PARTS>>(a, st);
    case 128:
      return launch_shape<Shape<D, F8, 32, 4, 1, KS, 2, PARTS>>(a, st);
    default:
      return launch_shape<Shape<D, F8, 32, 8, 1, KS, 2, PARTS>>(a, st);
  }
}

}  // namespace

size_t attention_ws(int T, int Hq, int Hkv, int D) {
  // (whatever B is: the tiles are no larger than one sequence's rows need)
  const int rows = rows_for(int64_t(T > 0 ? T : 1) * (Hq / Hkv));
  size_t most = 0;
  for (int r = 16; r <= rows; r *= 2)
    if (parts_bytes(r, D) > most) most = parts_bytes(r, D);
  return kJointBytes + most;
}

hipError_t launch_paged_attention(const AttnArgs& a, hipStream_t st) {
  const bool f8 = a.kv.f8, fine = a.x8 != nullptr;
  if (a.kv.D == 64) return f8 ? launch<64, true, 1>(a, st) : launch<64, false, 1>(a, st);
  if (a.kv.D == 128)
    return f8 ? fine ? launch<128, true, 2>(a, st) : launch<128, true, 1>(a, st)
              : fine ? launch<128, false, 2>(a, st) : launch<128, false, 1>(a, st);
  return f8 ? fine ? launch<256, true, 2>(a, st) : launch<256, true, 1>(a, st)
            : fine ? launch<256, false, 2>(a, st) : launch<256, false, 1>(a, st);
}

}  // namespace moe
