// Sampling with temperature, min-p, top-k and top-p from given uniform
// numbers, one token per row of logits.
//
// Tokens are ordered by logit, descending, the lower index first among equal
// ones.  With w = exp((logit - largest) / temperature), every filter keeps a
// prefix of that order: min-p the w >= min_p, top-k the first k, top-p the
// shortest prefix that holds the share p of what is left.  The token drawn
// is the first whose running sum exceeds u times the kept sum.  So each of
// top-k, top-p and the draw asks one question: at which token of the order
// does a running sum (of ones, or of w) reach a target?  No sort is needed:
//
//  1. the largest logit of the row;
//  2. how many tokens, and which sum of w, fall into each of 4096 bins of
//     (largest - logit) / temperature, 96 bins per unit.  Prefix sums over the
//     bins bound the bins in which the three targets can fall (the sums that
//     top-p and the draw refer to are known up to one bin of the question
//     before);
//  3. the tokens of those few bins are listed, and the three questions are
//     answered exactly among them: by 8 key bits at a time, then among at most
//     64 tokens within one wave.
//
// Sums.  Within bin b, w = e^(-b/96) (1 - v) with 0 <= v < 0.0105.  v is
// evaluated in 64 bits and held as an integer q (27 bits for 151,936 tokens:
// w to 2^-34 of itself), and a token adds (1, q) to its bin as one 64-bit
// integer, the count in the high bits: one LDS atomic per token, no
// exponential, and no order of the additions to depend on.  A bin's mass is an
// integer too, rint(e^(-b/96) (count - sum q / S) 2^s), s chosen so that a
// row's sum stays below 2^62.  So a row's answer does not depend on how it
// was split nor on which atomic came first, and the steps agree on every sum
// to the last bit.  (A draw next to the border between two tokens of a flat
// row needs such sums: with fp32 ones about one in 10,000 would differ.)
// A lone token below 2^-(s + 1) of the largest has mass 0, so the last kept
// token (u >= 1) is found by count.  Tokens more than 42 units below the
// largest (w < 6e-19) are never drawn.
//
// Many rows, or short ones: sample_row_kernel, one workgroup per row and one
// launch.  Few long rows: three launches with a slice of a row per workgroup;
// the last workgroup of a row to arrive does what needs the whole row.

#include <hip/hip_runtime.h>

#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 512;           // of the kernels over slices
constexpr int kRowThreads = 1024;       // of the kernel over rows
constexpr int kBins = 4096;
constexpr double kBinsPerUnit = 96.0;
constexpr double kToInt = 0x1.8p52;     // added: the low 32 bits are the nearest integer
constexpr double kCutoff = 42.0;        // units below the largest logit from which on nothing is drawn
constexpr int kMaxParts = 256;
constexpr int kSlice = 4096;            // logits of a row per workgroup
constexpr int kListCap = 16384;         // listed candidates of a row
constexpr int kLdsList = 3200;          // of which this many are searched in LDS
constexpr int kRowList = 12288;         // listed candidates in LDS with a workgroup per row

struct RowCtl {
  uint32_t pick_done, listed, drawn;   // drawn: rows finished (row 0's only)
};

// The workspace, from SampleArgs.ws (256-byte aligned).
struct Ws {
  uint64_t* part;    // [T][kMaxParts] largest keys of the slices
  RowCtl* ctl;       // [T]
  uint64_t* bins;    // [T][kBins] packed sums per bin
  uint64_t* list;    // [T][kListCap] candidates' keys
};

__host__ __device__ inline size_t align256(size_t v) { return (v + 255) / 256 * 256; }

__host__ __device__ inline size_t ws_layout(int T, uint8_t* base, Ws* w) {
  size_t o = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = base + o;
    o += align256(bytes);
    return p;
  };
  w->part = reinterpret_cast<uint64_t*>(take(size_t(T) * kMaxParts * 8));
  w->ctl = reinterpret_cast<RowCtl*>(take(size_t(T) * sizeof(RowCtl)));
  w->bins = reinterpret_cast<uint64_t*>(take(size_t(T) * kBins * 8));
  w->list = reinterpret_cast<uint64_t*>(take(size_t(T) * kListCap * 8));
  return o;
}

// ---- logits

// Elements of one 16-byte load.
template <int FMT>
constexpr int kVec = FMT == MOE_W_F32 ? 4 : 8;

// Row `row` as a range of 16-byte vectors: vector i holds elements
// [i * kVec - lead, ...); the first and the last may lie partly outside.
template <int FMT>
struct RowView {
  typedef const __attribute__((address_space(1))) uint8_t* Bytes;
  typedef const __attribute__((address_space(1))) float* Floats;
  typedef const __attribute__((address_space(1))) uint16_t* Halves;
  typedef const __attribute__((address_space(1))) u32x4* Vectors;
  Bytes base;            // address of vector 0 (16-byte aligned; not read before the row)
  int lead;              // elements of vector 0 in front of the row
  int V;
  int vecs;
  int inner0, inner1;    // vectors wholly inside: [inner0, inner1]
  __device__ RowView(const void* logits, int64_t stride, int row, int v) {
    constexpr int size = FMT == MOE_W_F32 ? 4 : 2;
    const uintptr_t a = reinterpret_cast<uintptr_t>(logits) + uintptr_t(row) * stride * size;
    base = (Bytes)(a & ~uintptr_t(15));
    lead = int(a & 15) / size;
    V = v;
    vecs = (V + lead + kVec<FMT> - 1) / kVec<FMT>;
    inner0 = lead ? 1 : 0;
    inner1 = (V + lead) / kVec<FMT> - 1;
  }
  __device__ float at(int i) const {
    if (FMT == MOE_W_F32) return ((Floats)base)[lead + int64_t(i)];
    return bf16_to_f32(((Halves)base)[lead + int64_t(i)]);
  }
  // vector i's 16 bytes, elements outside the row as -infinity
  __device__ __forceinline__ u32x4 load(int i) const {
    u32x4 q;
    if (inner1 >= inner0) q = ((Vectors)base)[int64_t(max(inner0, min(i, inner1)))];
    if (i < inner0 || i > inner1) {
      const int e = i * kVec<FMT> - lead;
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        uint32_t w;
        if (FMT == MOE_W_F32) {
          w = __float_as_uint(e + j >= 0 && e + j < V ? at(e + j) : -__builtin_inff());
        } else {
          const int k = e + 2 * j;
          const float lo = k >= 0 && k < V ? at(k) : -__builtin_inff();
          const float hi = k + 1 >= 0 && k + 1 < V ? at(k + 1) : -__builtin_inff();
          w = (__float_as_uint(lo) >> 16) | __float_as_uint(hi);
        }
        if (j == 0) q[0] = w;
        else if (j == 1) q[1] = w;
        else if (j == 2) q[2] = w;
        else q[3] = w;
      }
    }
    return q;
  }
};

// Vectors [begin, end) of a row, four logits at a time: f(x, first index, in),
// whole waves at once (in: this lane's logits exist).  U vectors per thread
// are on their way while U are worked on.
template <int FMT, int U, class F>
__device__ __forceinline__ void for_slice(const RowView<FMT>& v, int begin, int end, const F& f) {
  const int step = int(blockDim.x), lane = threadIdx.x & 63;
  const int wave0 = begin + int(threadIdx.x) - lane;
  u32x4 next[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (wave0 + u * step + lane < end) next[u] = v.load(wave0 + u * step + lane);
#pragma unroll 1
  for (int i0 = wave0; i0 < end; i0 += U * step) {
    u32x4 now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      now[u] = next[u];
      const int i = i0 + (U + u) * step + lane;
      if (i < end) next[u] = v.load(i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * step + lane, at = i * kVec<FMT> - v.lead;
      const u32x4 q = now[u];
      if (FMT == MOE_W_F32) {
        const float x[4] = {__uint_as_float(q[0]), __uint_as_float(q[1]), __uint_as_float(q[2]),
                            __uint_as_float(q[3])};
        f(x, at, i < end);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x[4] = {__uint_as_float(q[2 * h] << 16), __uint_as_float(q[2 * h] & 0xFFFF0000u),
                              __uint_as_float(q[2 * h + 1] << 16),
                              __uint_as_float(q[2 * h + 1] & 0xFFFF0000u)};
          f(x, at + 4 * h, i < end);
        }
      }
    }
  }
}

// Unique key of a token: a larger key comes earlier in the order.
__device__ __forceinline__ uint64_t key_of(float x, int idx) {
  return (uint64_t(ordered_bits(x)) << 32) | uint64_t(~uint32_t(idx));
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t o = uint32_t(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ int index_of(uint64_t key) { return int(~uint32_t(key)); }

// ---- across lanes and workgroups

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint64_t shfl_u64(uint64_t v, int lane) {
  const uint32_t lo = __shfl(uint32_t(v), lane, kWave), hi = __shfl(uint32_t(v >> 32), lane, kWave);
  return (uint64_t(hi) << 32) | lo;
}

// The value of one lane, the same in all.
__device__ __forceinline__ uint64_t lane_u64(uint64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(v), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(uint32_t(v >> 32), lane);
  return (uint64_t(hi) << 32) | lo;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or_zero(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xF, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ void scan_step(uint64_t& v) {
  const uint64_t lo = dpp_or_zero<CTRL, ROWS>(uint32_t(v)), hi = dpp_or_zero<CTRL, ROWS>(uint32_t(v >> 32));
  v += (hi << 32) | lo;
}
// Inclusive prefix sum over the wave's lanes (DPP: row shifts, then broadcasts
// of the rows' last lanes).
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {
  scan_step<0x111, 0xF>(v);
  scan_step<0x112, 0xF>(v);
  scan_step<0x114, 0xF>(v);
  scan_step<0x118, 0xF>(v);
  scan_step<0x142, 0xA>(v);
  scan_step<0x143, 0xC>(v);
  return v;
}

// red: one word per wave.
__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t* red) {
  v = wave_max_u64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  const int lane = threadIdx.x & 63;
  return wave_max_u64(lane < int(blockDim.x) / kWave ? red[lane] : 0);
}

// Inclusive prefixes of a and b over the workgroup; red: two words per wave.
__device__ __forceinline__ void block_scan(uint64_t& a, uint64_t& b, uint64_t* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  a = wave_scan(a);
  b = wave_scan(b);
  __syncthreads();
  if (lane == 63) red[2 * wave] = a, red[2 * wave + 1] = b;
  __syncthreads();
  // every wave scans the waves' sums
  const bool in = lane < int(blockDim.x) / kWave;
  uint64_t xa = wave_scan(in ? red[2 * lane] : 0), xb = wave_scan(in ? red[2 * lane + 1] : 0);
  const int before = __builtin_amdgcn_readfirstlane(wave) - 1;
  xa = before < 0 ? 0 : lane_u64(xa, before);
  xb = before < 0 ? 0 : lane_u64(xb, before);
  a += xa;
  b += xb;
}

// What workgroups of one launch hand to each other goes through relaxed
// device-scope atomics, which act on memory that every XCD sees, and the
// arrival is counted once they have completed.  A device-scope fence would
// write back the XCD's whole L2 instead (measured: the sums of 64 rows took
// 53 us with one per wave, 29 us without).
template <class Tp>
__device__ __forceinline__ void put(Tp* p, Tp v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class Tp>
__device__ __forceinline__ Tp get(const Tp* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether this workgroup is the last of `n` to arrive at `counter`; what the
// others put or added before arriving is what it gets afterwards.
__device__ bool arrive_last(uint32_t* counter, uint32_t n, uint32_t* flag) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    *flag = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const bool last = *flag == n - 1;
  asm volatile("" ::: "memory");
  return last;
}

// ---- one row's parameters, bins and weights

struct Row {
  bool greedy;
  int top_k;          // <= 0: all
  double top_p;       // >= 1: all
  double u;
  double inv_tau;
  double top64;       // the largest logit, 0 if that is infinite
  double bins;        // bins per logit
  double limit;       // place beyond which nothing is drawn (min-p, kCutoff)
  double v0, v1, v2, v3;      // S v as a polynomial of the place's distance from the bin's middle
  double inv_s;       // 1 / S
  double unit;        // 2^s
  uint64_t q_mask;
  int q_bits;         // the count begins at this bit, 32 or higher
  float top;          // the largest logit
  bool top_inf;       // it is infinite: only its equals can be drawn
  uint64_t top_key;   // 0: no usable logit
};

// exp(-d), 0 <= d <= 700: d = n ln2 + r, |r| <= ln2 / 2 (ln2 as its nearest
// double and the rest), then the power series to r^12 (remainder below 2e-16).
__device__ __forceinline__ double exp_minus(double d) {
  const double n = rint(d * 1.4426950408889634);
  double r = fma(n, 0.6931471805599453, -d);
  r = fma(n, 2.3190468138462996e-17, r);
  double p = 1.0 / 479001600.0;
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return p * __longlong_as_double((int64_t)(1023 - int(n)) << 52);
}

// The row's parameters from its largest key.
struct Given {
  float tau, min_p, top_p, u;
  int top_k;
};
__device__ __forceinline__ Given load_given(const SampleArgs& a, int row) {
  Given g;
  g.tau = a.temperature ? a.temperature[row] : 1.0f;
  g.min_p = a.min_p ? a.min_p[row] : 0.0f;
  g.top_p = a.top_p ? a.top_p[row] : 1.0f;
  g.top_k = a.top_k ? a.top_k[row] : 0;
  g.u = a.u[row];
  return g;
}
__device__ Row make_row(const SampleArgs& a, const Given& g, uint64_t top_key) {
  Row r;
  r.top_key = top_key;
  r.top = logit_of(top_key);
  r.top_inf = r.top == __builtin_inff();
  r.top64 = r.top_inf ? 0.0 : double(r.top);
  r.top_k = g.top_k;
  r.top_p = g.top_p < 1.0f ? fmax(double(g.top_p), 0.0) : 1.0;     // NaN: no cut
  r.u = g.u > 0.0f ? fmin(double(g.u), 1.0) : 0.0;
  r.greedy = !(g.tau > 0.0f) || g.min_p > 1.0f || g.top_k == 1 || top_key == 0;
  r.inv_tau = r.greedy ? 1.0 : 1.0 / double(g.tau);
  r.bins = r.inv_tau * kBinsPerUnit;
  r.limit = kCutoff * kBinsPerUnit;
  if (g.min_p > 0.0f && g.min_p <= 1.0f) {
    // -ln(min_p): fp32's logarithm, and one Newton step in 64 bits
    const double m = double(g.min_p), d = fmax(double(-logf(g.min_p)), 0.0);
    r.limit = fmin(r.limit, (d - (m / exp_minus(d) - 1.0)) * kBinsPerUnit);
  }
  r.limit -= 0.5;
  // v = 1 - exp(-(f + 1/2) / 96), |f| <= 1/2, to f^3, and S; f^4 as f^2 / 4 -
  // 1 / 128, which is within 1 / 128 of it there (4e-12 of v's unit)
  const double s = __longlong_as_double((int64_t)(1023 + a.frac_bits + 6) << 52);   // v < 2^-6 * 0.67
  const double middle = 0x1.fd571ba7c4ef1p-1;                                        // exp(-1 / 192)
  r.inv_s = 1.0 / s;
  r.v0 = s * (1.0 - middle);
  r.v1 = s * middle / kBinsPerUnit;
  r.v2 = r.v1 / (-2.0 * kBinsPerUnit);
  r.v3 = r.v2 / (-3.0 * kBinsPerUnit);
  const double v4 = r.v3 / (-4.0 * kBinsPerUnit);
  r.v2 += 0.25 * v4;
  r.v0 -= v4 / 128.0;
  r.unit = __longlong_as_double((int64_t)(1023 + a.shift) << 52);
  r.q_bits = a.q_bits;
  r.q_mask = (uint64_t(1) << a.q_bits) - 1;
  return r;
}

// A row whose largest logit is infinite draws among its equals alone: these
// as 0, the others as -infinity.
__device__ __forceinline__ float seen(const Row& r, float x) {
  return !r.top_inf ? x : x == r.top ? 0.0f : -__builtin_inff();
}
// Place of a logit: (largest - logit) in bins, less 1/2; monotone in x, NaN
// where x is one.  The nearest integer is its bin (0 .. kBins - 1 if the
// place is at most r.limit).
__device__ __forceinline__ double place_of(const Row& r, float x) {
  return fma(r.top64 - double(x), r.bins, -0.5);
}
__device__ __forceinline__ int bin_at(double place) {
  return int(uint32_t(__double_as_longlong(place + kToInt)));
}
// Position within the bin, 0 to 1.
__device__ __forceinline__ double within(double place) { return place - ((place + kToInt) - kToInt) + 0.5; }
// A bound of the logits that are at most (side -1) or at least (side 1) t
// bins below the largest: below, or above, all of them, by a little.
__device__ __forceinline__ float logit_bound(const Row& r, double t, double side) {
  const double x = r.top64 - t / r.bins;
  const double b = x + side * (fabs(x) + fabs(r.top64)) * 0x1p-20;
  return !r.top_inf && fabs(b) < 3.0e38 ? float(b) : float(side) * __builtin_inff();
}
// A token adds this to its bin: a count of one, and q.
__device__ __forceinline__ uint64_t packed_of(const Row& r, double place) {
  const double f = place - ((place + kToInt) - kToInt);
  double q = fma(r.v3, f, r.v2);
  q = fma(q, f, r.v1);
  q = fma(q, f, r.v0);
  return (uint64_t(1u << (r.q_bits - 32)) << 32) | uint64_t(uint32_t(__double_as_longlong(q + kToInt)));
}
// Mass of tokens of one bin (scale = e^(-bin/96) 2^s) from their packed sum.
__device__ __forceinline__ double bin_step(int j) {   // e^(-j/96), 0 <= j < 8
  const double e = 0x1.fab1c0ce7a11bp-1, e2 = e * e, e4 = e2 * e2;   // e = e^(-1/96)
  return (j & 1 ? e : 1.0) * (j & 2 ? e2 : 1.0) * (j & 4 ? e4 : 1.0);
}
__device__ __forceinline__ double bin_scale8(const Row& r, int bin) {   // of bin's run of eight
  return exp_minus(double(bin & ~7) / kBinsPerUnit) * r.unit;
}
__device__ __forceinline__ double bin_scale(const Row& r, int bin) {
  return bin_scale8(r, bin) * bin_step(bin & 7);
}
__device__ __forceinline__ uint64_t mass_of(const Row& r, double scale, uint64_t packed) {
  const double n = double(packed >> r.q_bits) - double(packed & r.q_mask) * r.inv_s;
  return uint64_t(rint(n * scale));
}

// Targets: the running sum (count, or mass) that the boundary token reaches first.
__device__ __forceinline__ uint64_t top_p_target(double p, uint64_t zk) {
  const uint64_t t = uint64_t(ceil(p * double(zk)));
  return t < 1 ? 1 : t > zk ? zk : t;
}
__device__ __forceinline__ uint64_t draw_target(double u, uint64_t zn) {
  const uint64_t t = uint64_t(floor(u * double(zn))) + 1;   // the sum exceeds u * zn
  return t > zn ? zn : t;
}
// u >= 1 takes the last kept token.  Behind top-p that is the one that reaches
// the whole kept sum; without, a token whose mass rounds to 0 may be the last,
// and the draw goes by the count of the kept ones.
__device__ __forceinline__ bool draws_last(const Row& r) { return r.u >= 1.0 && r.top_p >= 1.0; }
__device__ __forceinline__ uint32_t kept_count(const Row& r, uint32_t all) {
  return r.top_k > 0 && uint32_t(r.top_k) < all ? uint32_t(r.top_k) : all;
}

// ---- the steps

// Largest key of vectors [begin, end) of a row, over the workgroup.
template <int FMT>
__device__ __forceinline__ uint64_t largest_key(const RowView<FMT>& v, int begin, int end, uint64_t* red) {
  float best = -__builtin_inff();
  int at = 0;
  for_slice<FMT, 4>(v, begin, end, [&](const float (&x)[4], int first, bool in) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (in && x[j] > best) best = x[j], at = first + j;   // the first of equal ones
  });
  return block_max(best > -__builtin_inff() ? key_of(best, at) : 0, red);
}

// Adds the tokens of vectors [begin, end) to the bins in LDS.  Bound by the
// LDS atomics, which meet in the dense bins (151,936 tokens: 27 us of one CU,
// 14 where min-p leaves few; without branches, four tokens at a time, the same).
template <int FMT>
__device__ __forceinline__ void fill_bins(const Row& r, const RowView<FMT>& v, int begin, int end,
                                          uint64_t* bins) {
  const float low = logit_bound(r, r.limit + 0.5, -1.0);
  for_slice<FMT, 2>(v, begin, end, [&](const float (&x)[4], int, bool in) {
    // (NaN and -infinity fail the comparisons)
    const bool any = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= low;
    if (__ballot(in && any) == 0) return;
    float y[4] = {x[0], x[1], x[2], x[3]};
    if (__builtin_expect(r.top_inf, 0)) {
      asm volatile("");      // a branch, not four selections
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = seen(r, x[j]);
    }
    double place[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) place[j] = place_of(r, y[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (in && place[j] <= r.limit)
        atomicAdd(reinterpret_cast<unsigned long long*>(&bins[bin_at(place[j])]),
                  (unsigned long long)packed_of(r, place[j]));
  });
}

// First bin whose inclusive prefix reaches target (the last one if none does), found
// by one wave: 64 ends of 64 bins each, then those 64 bins.
template <class Tp>
__device__ __forceinline__ int first_reaching(const Tp* prefix, Tp target) {
  static_assert(kBins == 64 * 64, "two steps");
  const int lane = threadIdx.x & 63;
  const int run = __popcll(__ballot(prefix[lane * 64 + 63] < target));
  if (run == 64) return kBins - 1;
  return run * 64 + __popcll(__ballot(prefix[run * 64 + lane] < target));
}

// The bins [lo, hi] in which each target can fall, from the inclusive prefixes
// of masses and counts; one wave.
__device__ __forceinline__ void find_targets(const Row& r, const uint64_t* mass, const uint32_t* count,
                                             int* lo, int* hi) {
  uint64_t z0 = mass[kBins - 1], z1 = z0;      // bounds of the sum kept so far
#pragma unroll
  for (int q = 0; q < 3; ++q) lo[q] = 0, hi[q] = -1;
  if (r.top_k > 0 && uint32_t(r.top_k) < count[kBins - 1]) {
    const int b = first_reaching(count, uint32_t(r.top_k));
    lo[0] = hi[0] = b;
    z0 = max_u64(b ? mass[b - 1] : 0, 1);
    z1 = max_u64(mass[b], 1);
  }
  if (r.top_p < 1.0) {
    lo[1] = first_reaching(mass, top_p_target(r.top_p, z0));
    hi[1] = first_reaching(mass, top_p_target(r.top_p, z1));
    z0 = max_u64(lo[1] ? mass[lo[1] - 1] : 0, 1);
    z1 = mass[hi[1]];
  }
  if (draws_last(r)) {
    lo[2] = hi[2] = first_reaching(count, kept_count(r, count[kBins - 1]));
  } else {
    lo[2] = first_reaching(mass, draw_target(r.u, z0));
    hi[2] = first_reaching(mass, draw_target(r.u, z1));
  }
}

// From the bins' packed sums (PER per thread, from bin threadIdx.x * PER) the
// inclusive prefixes of masses and counts in LDS, and the bins [lo, hi] in
// which each target can fall: the same in every thread.
template <int PER>
__device__ __forceinline__ void bound_targets(const Row& r, const uint64_t* packed, uint64_t* mass,
                                              uint32_t* count, uint64_t* red, int* lo, int* hi) {
  const int b0 = int(threadIdx.x) * PER;
  static_assert(8 % PER == 0, "a thread's bins lie in one run of eight");
  uint64_t m[PER], mp = 0, cp = 0;
  const double scale = bin_scale8(r, b0);
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    m[j] = mass_of(r, scale * bin_step((b0 + j) & 7), packed[j]);
    mp += m[j];
    cp += packed[j] >> r.q_bits;
  }
  block_scan(mp, cp, red);
#pragma unroll
  for (int j = PER - 1; j >= 0; --j) {
    mass[b0 + j] = mp;
    count[b0 + j] = uint32_t(cp);
    mp -= m[j];
    cp -= packed[j] >> r.q_bits;
  }
  __syncthreads();
  // one wave finds the bins for all (issue slots that the others leave to it)
  int* found = reinterpret_cast<int*>(red);
  if (threadIdx.x < kWave) {
    find_targets(r, mass, count, lo, hi);
    if (threadIdx.x == 0) {
#pragma unroll
      for (int q = 0; q < 3; ++q) found[2 * q] = lo[q], found[2 * q + 1] = hi[q];
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    lo[q] = __builtin_amdgcn_readfirstlane(found[2 * q]);
    hi[q] = __builtin_amdgcn_readfirstlane(found[2 * q + 1]);
  }
}

// Which tokens matter: those of the bins [lo, hi], and few others.
struct Wanted {
  // every logit x of the bins of question q has |x scale - middle| <= kNear
  // (and few others do): the half width is 2^-18 of the logits there at
  // least, so that scale, middle and the fma are off by 2^-6 each at most
  static constexpr float kNear = 1.0625f;
  float scale[3], middle[3];
  float lowest;              // and is at or above this
  bool asked[2];             // questions 0 and 1
  bool open;                 // a range has no end: infinities could pass
  __device__ Wanted(const Row& r, const int* lo, const int* hi) {
    open = false;
    lowest = __builtin_inff();
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      if (q < 2) asked[q] = hi[q] >= lo[q];
      scale[q] = middle[q] = 0.0f;
      if (hi[q] < lo[q]) continue;
      // (the largest logit is an end too: a bound past fp32's range would leave no middle)
      const float from = logit_bound(r, double(hi[q] + 1), -1.0);
      const float to = fminf(logit_bound(r, double(lo[q]), 1.0), r.top);
      const float c = 0.5f * from + 0.5f * to;
      const float half = fmaxf(0.5f * to - 0.5f * from, fmaxf(fabsf(c) * 0x1p-18f, 0x1p-100f));
      scale[q] = 1.0f / half;
      middle[q] = c / half;
      lowest = fminf(lowest, from);
      open |= from == -__builtin_inff();
    }
  }
  // at most kNear: x is wanted (NaN is not)
  __device__ __forceinline__ float away(int q, float x) const { return fabsf(fmaf(x, scale[q], -middle[q])); }
  __device__ __forceinline__ bool operator()(const Row& r, float x) const {
    if (open) return place_of(r, seen(r, x)) <= r.limit;
    return away(2, x) <= kNear || (asked[1] && away(1, x) <= kNear) || (asked[0] && away(0, x) <= kNear);
  }
};

// Lists the wanted tokens of vectors [begin, end): each wave fills its own
// segment (LDS, room keys) and calls full(n) before it would overflow, which
// returns how many it still holds.  Returns the number in the segment.
// Tokens of bins next to the wanted ones may be listed, in part, and tokens
// beyond the limit: the sums through the former miss every target, and the
// latter are left out where candidates are used.  (A row of 151,936 with 1000
// candidates: 25 us; 36 with the exact bins, in 64 bits, here.)
template <int FMT, class Full>
__device__ __forceinline__ uint32_t list_wanted(const Row& r, const Wanted& wanted, const RowView<FMT>& v,
                                                int begin, int end, uint64_t* segment, uint32_t room,
                                                const Full& full) {
  const uint64_t self = uint64_t(1) << (threadIdx.x & 63), below = self - 1;
  uint32_t n = 0;
  for_slice<FMT, 2>(v, begin, end, [&](const float (&x)[4], int first, bool in) {
    // (NaN and -infinity fail the comparison, where the ranges have ends)
    const bool high = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= wanted.lowest;
    if (__ballot(in && high) == 0) return;
    float off[4];
    if (__builtin_expect(wanted.open, 0)) {
      asm volatile("");      // a branch, not four selections
#pragma unroll
      for (int j = 0; j < 4; ++j) off[j] = wanted(r, x[j]) ? 0.0f : 2.0f;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) off[j] = wanted.away(2, x[j]);
      if (wanted.asked[1]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) off[j] = fminf(off[j], wanted.away(1, x[j]));
      }
      if (wanted.asked[0]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) off[j] = fminf(off[j], wanted.away(0, x[j]));
      }
    }
    const float least = fminf(fminf(off[0], off[1]), fminf(off[2], off[3]));
    if (__ballot(in && least <= Wanted::kNear) == 0) return;
    uint64_t mask[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) mask[j] = __ballot(in && off[j] <= Wanted::kNear);
    if (n + 4 * kWave > room) n = full(n);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (mask[j] == 0) continue;
      const uint32_t at = n + uint32_t(__popcll(mask[j] & below));
      if ((mask[j] & self) && at < room) segment[at] = key_of(x[j], first + j);
      n += uint32_t(__popcll(mask[j]));
    }
  });
  return n;
}

struct PickLds {
  uint64_t hsum[256];
  uint64_t few[64];
  uint64_t all_or, all_and, key, sum, prefix, base;
  uint32_t n, left;
  int32_t bin;
};

// The three questions of one row among its candidates (for_each(f) calls
// f(key, have) for each, whole waves at once): the drawn token's key, and the
// kept sum.  mass_before(b) and count_before(b): sums of the bins in front of
// b; total: the row's.
template <class Mass, class Count, class ForEach>
__device__ __forceinline__ uint64_t draw_token(const Row& r, const int* lo, const int* hi, uint64_t total,
                                               const Mass& mass_before, const Count& count_before,
                                               PickLds& s, uint64_t* kept, const ForEach& for_each) {
  uint64_t z = total;
#pragma unroll 1
  for (int q = 0; q < 3; ++q) {
    const bool by_count = q == 0 || (q == 2 && draws_last(r));
    if (hi[q] < lo[q]) continue;
    const uint64_t target = by_count ? uint64_t(kept_count(r, count_before(kBins)))
                            : q == 1 ? top_p_target(r.top_p, z)
                                     : draw_target(r.u, z);
    __syncthreads();
    if (threadIdx.x == 0) s.all_or = 0, s.all_and = ~0ull, s.n = 0, s.bin = lo[q], s.base = 0;
    if (threadIdx.x < 256) s.hsum[threadIdx.x] = 0;
    __syncthreads();
    // the bin, and the sum in front of it
#pragma unroll 1
    for (int b = lo[q] + int(threadIdx.x); b <= hi[q]; b += int(blockDim.x)) {
      const uint64_t before = by_count ? uint64_t(count_before(b)) : mass_before(b);
      const uint64_t after = by_count ? uint64_t(count_before(b + 1)) : mass_before(b + 1);
      if (before < target && after >= target) s.bin = b, s.base = before;
    }
    __syncthreads();
    const int bin = s.bin;
    const uint64_t base = s.base;
    const double scale = bin_scale(r, bin);
    // the sum through tokens whose packed sum from the bin's front is p
    auto sum_of = [&](uint64_t p) { return base + (by_count ? p >> r.q_bits : mass_of(r, scale, p)); };
    // Narrow the bin to at most 64 tokens: first by the position within the
    // bin, in 256 parts, then (equal logits) by the key, 8 bits at a time
    // from the highest bit in which the keys differ.
    uint32_t left = count_before(bin + 1) - count_before(bin);
    uint64_t front = 0;      // packed sum of the bin's tokens ahead of the range
    int part = -1;           // the part, -1: all
    int sh = 64;             // the keys' bits from sh up are prefix, 64: any
    uint64_t prefix = 0;
    auto part_of = [](double place) { return min(int(within(place) * 256.0), 255); };
    auto active = [&](uint64_t key, double* place) {
      *place = place_of(r, seen(r, logit_of(key)));
      return *place <= r.limit && bin_at(*place) == bin && (part < 0 || part_of(*place) == part) &&
             (sh == 64 || (key >> sh) == prefix);
    };
#pragma unroll 1
    while (left > 64 && sh > 0) {
      const bool by_part = part < 0;
      int next = 0;
      if (!by_part) {
        if (sh == 64) {
          uint64_t o = 0, n = ~0ull;
          for_each([&](uint64_t key, bool have) {
            double t;
            if (have && active(key, &t)) o |= key, n &= key;
          });
          if (n != ~0ull) {
            atomicOr(reinterpret_cast<unsigned long long*>(&s.all_or), (unsigned long long)o);
            atomicAnd(reinterpret_cast<unsigned long long*>(&s.all_and), (unsigned long long)n);
          }
          __syncthreads();
          const uint64_t differ = s.all_or & ~s.all_and;   // not 0: keys are unique
          sh = 64 - __clzll((long long)differ);
          prefix = sh == 64 ? 0 : s.all_or >> sh;
        }
        next = sh > 8 ? sh - 8 : 0;
        if (threadIdx.x < 256) s.hsum[threadIdx.x] = 0;
        __syncthreads();
      }
      const uint64_t digits = (uint64_t(1) << (sh - next)) - 1;
      for_each([&](uint64_t key, bool have) {
        double t;
        if (!have || !active(key, &t)) return;
        const int d = by_part ? 255 - part_of(t) : int((key >> next) & digits);
        atomicAdd(reinterpret_cast<unsigned long long*>(&s.hsum[d]), (unsigned long long)packed_of(r, t));
      });
      __syncthreads();
      if (threadIdx.x < 64) {
        // lane i holds digits 255 - 4i .. 252 - 4i: descending
        uint64_t v[4], sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += v[j] = s.hsum[255 - 4 * int(threadIdx.x) - j];
        uint64_t before = front + wave_scan(sum) - sum;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          const uint64_t vj = j == 0 ? v[0] : j == 1 ? v[1] : j == 2 ? v[2] : v[3];
          if (vj && sum_of(before) < target && sum_of(before + vj) >= target) {
            s.prefix = uint64_t(255 - 4 * int(threadIdx.x) - j);
            s.sum = before;
            s.left = uint32_t(vj >> r.q_bits);
          }
          before += vj;
        }
      }
      __syncthreads();
      front = s.sum;
      left = s.left;
      if (by_part) {
        part = 255 - int(s.prefix);
      } else {
        prefix = ((sh == 64 ? 0 : prefix) << (sh - next)) | s.prefix;
        sh = next;
      }
    }
    for_each([&](uint64_t key, bool have) {
      double t;
      const bool take = have && active(key, &t);
      const uint64_t mask = __ballot(take);
      if (mask == 0) return;
      const int lane = threadIdx.x & 63;
      uint32_t at = 0;
      if (lane == 0) at = atomicAdd(&s.n, uint32_t(__popcll(mask)));
      at = __shfl(at, 0, kWave) + uint32_t(__popcll(mask & ((uint64_t(1) << lane) - 1)));
      if (take && at < 64) s.few[at] = key;
    });
    __syncthreads();
    if (threadIdx.x < 64) {
      const uint32_t n = min(s.n, 64u);
      const bool have = threadIdx.x < n;
      const uint64_t key = have ? s.few[threadIdx.x] : 0;
      const uint64_t mine = have ? packed_of(r, place_of(r, seen(r, logit_of(key)))) : 0;
      uint64_t ahead = front;
#pragma unroll 1
      for (uint32_t j = 0; j < n; ++j) {
        const uint64_t ok = shfl_u64(key, int(j)), op = shfl_u64(mine, int(j));
        if (ok > key) ahead += op;
      }
      if (have && sum_of(ahead) < target && sum_of(ahead + mine) >= target) {
        s.key = key;
        s.sum = ahead + mine;
      }
    }
    __syncthreads();
    if (q == 2) break;
    z = max_u64(mass_before(bin) + mass_of(r, scale, s.sum), 1);
  }
  *kept = z;
  return s.key;
}

// The same by one wave, for up to 64 candidates: lane i holds the i-th (key 0:
// none).
template <class Mass, class Count>
__device__ __forceinline__ uint64_t draw_token_wave(const Row& r, const int* lo, const int* hi,
                                                    uint64_t total, const Mass& mass_before,
                                                    const Count& count_before, uint32_t n, uint64_t key,
                                                    uint64_t* kept) {
  const double place = place_of(r, seen(r, logit_of(key)));
  if (!(place <= r.limit)) key = 0;
  const int my_bin = key ? bin_at(place) : -1;
  const uint64_t mine = key ? packed_of(r, place) : 0;
  // packed sum of the candidates of this one's bin in front of it
  uint64_t ahead = 0;
#pragma unroll 1
  for (uint32_t j = 0; j < n; ++j) {
    const uint64_t ok = shfl_u64(key, int(j)), op = shfl_u64(mine, int(j));
    const int ob = __shfl(my_bin, int(j), kWave);
    if (ok > key && ob == my_bin) ahead += op;
  }
  const double scale = bin_scale(r, max(my_bin, 0));
  const uint64_t m0 = mass_before(max(my_bin, 0)), c0 = count_before(max(my_bin, 0));
  const uint64_t mass_to = m0 + mass_of(r, scale, ahead), mass_thru = m0 + mass_of(r, scale, ahead + mine);
  const uint64_t count_to = c0 + (ahead >> r.q_bits);
  uint64_t z = total;
  if (hi[0] >= lo[0]) {
    const uint64_t hit = __ballot(key && count_to + 1 == uint64_t(r.top_k));
    z = max_u64(shfl_u64(mass_thru, __ffsll((long long)hit) - 1), 1);
  }
  if (hi[1] >= lo[1]) {
    const uint64_t target = top_p_target(r.top_p, z);
    const uint64_t hit = __ballot(key && mass_to < target && mass_thru >= target);
    z = max_u64(shfl_u64(mass_thru, __ffsll((long long)hit) - 1), 1);
  }
  const bool last = draws_last(r);
  const uint64_t target = last ? uint64_t(kept_count(r, count_before(kBins))) : draw_target(r.u, z);
  const uint64_t hit = __ballot(key && (last ? count_to + 1 == target : mass_to < target && mass_thru >= target));
  *kept = z;
  return shfl_u64(key, __ffsll((long long)hit) - 1);
}

// The drawn token's probability.
__device__ __forceinline__ float prob_of(const Row& r, uint64_t key, uint64_t kept) {
  const double t = place_of(r, seen(r, logit_of(key))) + 0.5;
  return float(exp_minus(fmax(0.0, fmin(t / kBinsPerUnit, kCutoff))) * r.unit / double(kept));
}

// ---- one workgroup per row

template <int FMT>
__global__ __launch_bounds__(kRowThreads) void sample_row_kernel(const SampleArgs a) {
  constexpr int PER = kBins / kRowThreads;
  __shared__ uint64_t mass[kBins];
  __shared__ uint32_t count[kBins];
  __shared__ uint64_t list[kRowList];
  __shared__ uint64_t red[2 * kRowThreads / kWave];
  __shared__ PickLds s;
  __shared__ uint32_t listed[kRowThreads / kWave];
  const int row = blockIdx.x;
  const Given given = load_given(a, row);
  const RowView<FMT> v(a.logits, a.stride, row, a.V);
#pragma unroll
  for (int j = 0; j < PER; ++j) mass[j * kRowThreads + threadIdx.x] = 0;
  const uint64_t top = largest_key<FMT>(v, 0, v.vecs, red);
  const Row r = make_row(a, given, top);
  if (r.greedy) {
    if (threadIdx.x == 0) {
      a.tokens[row] = top ? index_of(top) : -1;
      if (a.prob) a.prob[row] = top ? 1.0f : 0.0f;
    }
    return;
  }
  fill_bins<FMT>(r, v, 0, v.vecs, mass);
  __syncthreads();
  uint64_t packed[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) packed[j] = mass[threadIdx.x * PER + j];
  int lo[3], hi[3];
  bound_targets<PER>(r, packed, mass, count, red, lo, hi);
  const Wanted wanted(r, lo, hi);
  // the wanted tokens, every wave's in its own segment
  constexpr int kWaves = kRowThreads / kWave, kRoom = kRowList / kWaves;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint64_t* segment = list + wave * kRoom;
  const uint32_t mine = list_wanted<FMT>(r, wanted, v, 0, v.vecs, segment, kRoom,
                                         [](uint32_t n) { return n; });
  if (lane == 0) listed[wave] = mine;
  __syncthreads();
  uint32_t n = 0, before = 0, most = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? listed[w] : 0;
    n += listed[w];
    most = max(most, listed[w]);
  }
  auto mass_before = [&](int b) { return b ? mass[b - 1] : uint64_t(0); };
  auto count_before = [&](int b) { return b ? count[b - 1] : 0u; };
  uint64_t key, kept;
  if (n <= uint32_t(kWave)) {
    if (uint32_t(lane) < mine) s.few[before + lane] = segment[lane];
    __syncthreads();
    if (wave > 0) return;
    key = draw_token_wave(r, lo, hi, mass[kBins - 1], mass_before, count_before, n,
                          uint32_t(lane) < n ? s.few[lane] : 0, &kept);
  } else if (most <= uint32_t(kRoom)) {
    key = draw_token(r, lo, hi, mass[kBins - 1], mass_before, count_before, s, &kept, [&](auto&& f) {
#pragma unroll 1
      for (uint32_t k = 0; k < mine; k += kWave)
        f(k + lane < mine ? segment[k + lane] : 0, k + lane < mine);
    });
  } else {
    // more candidates than the list holds (long runs of equal logits): the row itself
    key = draw_token(r, lo, hi, mass[kBins - 1], mass_before, count_before, s, &kept, [&](auto&& f) {
#pragma unroll 1
      for (int i = threadIdx.x; i - lane < a.V; i += kRowThreads) {
        const float x = i < a.V ? v.at(i) : -__builtin_inff();
        f(key_of(x, i), i < a.V && wanted(r, x));
      }
    });
  }
  if (threadIdx.x == 0) {
    a.tokens[row] = index_of(key);
    if (a.prob) a.prob[row] = prob_of(r, key, kept);
  }
}

// Drafts that the rows' tokens agree with, from the front.
__global__ __launch_bounds__(kWave) void sample_accept_kernel(const SampleArgs a) {
  const int i = threadIdx.x;                    // T <= 64
  const bool agree = i < a.T - 1 && a.draft[i] == a.tokens[i];
  const uint64_t mask = __ballot(agree);
  if (i == 0) *a.n_out = (mask == ~0ull ? kWave : __ffsll((long long)~mask) - 1) + 1;
}

// ---- a slice of a row per workgroup

__device__ __forceinline__ Row read_row(const SampleArgs& a, const Ws& w, int row, uint64_t* red) {
  uint64_t k = 0;
  if (int(threadIdx.x) < a.parts) k = w.part[int64_t(row) * kMaxParts + threadIdx.x];
  const Given g = load_given(a, row);      // under way before the first wait
  return make_row(a, g, block_max(k, red));
}

// 1. Largest logit of every slice; clears the row's sums.
template <int FMT>
__global__ __launch_bounds__(kThreads) void sample_max_kernel(const SampleArgs a) {
  __shared__ uint64_t red[2 * kThreads / kWave];
  Ws w;
  ws_layout(a.T, static_cast<uint8_t*>(a.ws), &w);
  const int p = blockIdx.x, row = blockIdx.y;
  const int per_bins = (kBins + a.parts - 1) / a.parts;
  const int b1 = min(kBins, (p + 1) * per_bins);
  for (int b = p * per_bins + threadIdx.x; b < b1; b += kThreads) w.bins[int64_t(row) * kBins + b] = 0;
  if (p == 0 && threadIdx.x < sizeof(RowCtl) / 4)
    reinterpret_cast<uint32_t*>(&w.ctl[row])[threadIdx.x] = 0;
  const RowView<FMT> v(a.logits, a.stride, row, a.V);
  const int per = (v.vecs + a.parts - 1) / a.parts;
  const uint64_t k = largest_key<FMT>(v, p * per, min(v.vecs, (p + 1) * per), red);
  if (threadIdx.x == 0) w.part[int64_t(row) * kMaxParts + p] = k;
}

// 2. Sums per bin.
template <int FMT>
__global__ __launch_bounds__(kThreads) void sample_hist_kernel(const SampleArgs a) {
  constexpr int PER = kBins / kThreads;
  __shared__ uint64_t bins[kBins];
  __shared__ uint64_t red[2 * kThreads / kWave];
  Ws w;
  ws_layout(a.T, static_cast<uint8_t*>(a.ws), &w);
  const int row = blockIdx.y;
#pragma unroll
  for (int j = 0; j < PER; ++j) bins[j * kThreads + threadIdx.x] = 0;
  const Row r = read_row(a, w, row, red);
  if (r.greedy) return;
  const RowView<FMT> v(a.logits, a.stride, row, a.V);
  const int per = (v.vecs + a.parts - 1) / a.parts;
  fill_bins<FMT>(r, v, int(blockIdx.x) * per, min(v.vecs, (int(blockIdx.x) + 1) * per), bins);
  __syncthreads();
  uint64_t* sums = w.bins + int64_t(row) * kBins;
#pragma unroll 1
  for (int b = threadIdx.x; b < kBins; b += kThreads)
    if (bins[b]) __hip_atomic_fetch_add(&sums[b], bins[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A finished row: its token; with drafts, the last row to finish counts the
// drafts that the tokens agree with.
__device__ void finish_row(const SampleArgs& a, const Ws& w, int row, int token, float prob,
                           uint32_t* flag) {
  if (threadIdx.x == 0) {
    put(&a.tokens[row], token);
    if (a.prob) a.prob[row] = prob;
  }
  if (!a.n_out) return;
  if (!arrive_last(&w.ctl[0].drawn, a.T, flag)) return;
  if (threadIdx.x == 0) {
    int kept = 0;
    while (kept < a.T - 1 && a.draft[kept] == get(&a.tokens[kept])) ++kept;
    *a.n_out = kept + 1;
  }
}

// 3. The bins that matter (every workgroup finds them for itself: one hand-over
// less), their tokens, and the three answers.
template <int FMT>
__global__ __launch_bounds__(kThreads) void sample_pick_kernel(const SampleArgs a) {
  constexpr int PER = kBins / kThreads;
  __shared__ uint64_t mass[kBins];
  __shared__ uint32_t count[kBins];
  __shared__ uint64_t space[kLdsList];
  __shared__ uint64_t red[2 * kThreads / kWave];
  __shared__ PickLds s;
  __shared__ uint32_t flag;
  Ws w;
  ws_layout(a.T, static_cast<uint8_t*>(a.ws), &w);
  const int row = blockIdx.y;
  RowCtl& ctl = w.ctl[row];
  uint64_t packed[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) packed[j] = w.bins[int64_t(row) * kBins + threadIdx.x * PER + j];
  const Row r = read_row(a, w, row, red);
  if (r.greedy) {
    if (blockIdx.x == 0)
      finish_row(a, w, row, r.top_key ? index_of(r.top_key) : -1, r.top_key ? 1.0f : 0.0f, &flag);
    return;
  }
  int lo[3], hi[3];
  bound_targets<PER>(r, packed, mass, count, red, lo, hi);
  const Wanted wanted(r, lo, hi);
  uint64_t* list = w.list + int64_t(row) * kListCap;
  const RowView<FMT> v(a.logits, a.stride, row, a.V);
  const int per = (v.vecs + a.parts - 1) / a.parts;
  const int begin = int(blockIdx.x) * per, end = min(v.vecs, begin + per);
  {
    constexpr uint32_t kRoom = kLdsList / (kThreads / kWave);
    const int lane = threadIdx.x & 63;
    uint64_t* segment = space + (threadIdx.x >> 6) * kRoom;
    auto empty = [&](uint32_t n) {
      uint32_t at = 0;
      if (lane == 0)
        at = __hip_atomic_fetch_add(&ctl.listed, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      at = __shfl(at, 0, kWave);
      __builtin_amdgcn_wave_barrier();   // the segment's writes stay in front of its reads
#pragma unroll 1
      for (uint32_t k = lane; k < n; k += kWave)
        if (at + k < uint32_t(kListCap)) put(&list[at + k], segment[k]);
      __builtin_amdgcn_wave_barrier();
      return 0u;
    };
    const uint32_t n = list_wanted<FMT>(r, wanted, v, begin, end, segment, kRoom, empty);
    if (n) empty(n);
  }
  if (!arrive_last(&ctl.pick_done, a.parts, &flag)) return;

  const uint32_t n = get(&ctl.listed);
  auto mass_before = [&](int b) { return b ? mass[b - 1] : uint64_t(0); };
  auto count_before = [&](int b) { return b ? count[b - 1] : 0u; };
  uint64_t key, kept;
  if (n <= uint32_t(kWave)) {
    const uint32_t i = threadIdx.x & 63;      // (every wave finds the same)
    key = draw_token_wave(r, lo, hi, mass[kBins - 1], mass_before, count_before, n,
                          i < n ? get(&list[i]) : 0, &kept);
  } else if (n <= uint32_t(kListCap)) {
    const bool in_lds = n <= uint32_t(kLdsList);
    if (in_lds)
      for (uint32_t k = threadIdx.x; k < n; k += kThreads) space[k] = get(&list[k]);
    key = draw_token(r, lo, hi, mass[kBins - 1], mass_before, count_before, s, &kept, [&](auto&& f) {
#pragma unroll 1
      for (uint32_t k = threadIdx.x; k - (threadIdx.x & 63) < n; k += kThreads)
        f(k >= n ? 0 : in_lds ? space[k] : get(&list[k]), k < n);
    });
  } else {
    // more candidates than the list holds (long runs of equal logits): the row itself
    key = draw_token(r, lo, hi, mass[kBins - 1], mass_before, count_before, s, &kept, [&](auto&& f) {
#pragma unroll 1
      for (int i = threadIdx.x; i - int(threadIdx.x & 63) < a.V; i += kThreads) {
        const float x = i < a.V ? v.at(i) : -__builtin_inff();
        f(key_of(x, i), i < a.V && wanted(r, x));
      }
    });
  }
  __syncthreads();
  finish_row(a, w, row, index_of(key), prob_of(r, key, kept), &flag);
}

// Up to how many rows of V logits go in slices.  A workgroup per row has one
// launch but one CU's speed: 16 x 32,000 takes 24 us (25 us in slices), 16 x
// 151,936 61 us (29 us), 64 x 48,000 34 us (34 us), 128 x 64,000 44 us (46 us), 128
// and 256 x 151,936 75 and 94 us (64 and 108 us).
int sliced_rows(int V) { return V <= 36000 ? 0 : V / 650 - 1; }

template <int FMT>
hipError_t launch(SampleArgs a, hipStream_t st) {
  if (a.T > sliced_rows(a.V)) {
    sample_row_kernel<FMT><<<a.T, kRowThreads, 0, st>>>(a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.n_out) {
      sample_accept_kernel<<<1, kWave, 0, st>>>(a);
      e = hipGetLastError();
    }
    return e;
  }
  // a slice per workgroup for few rows; else one workgroup per CU or two, as
  // many as the bins' LDS lets in (16, 32, 64 x 151,936: 29, 32, 46 us with one,
  // 32, 34, 44 with two; three, in turns, 42, 48, 59)
  const int slices = (a.V + kSlice - 1) / kSlice;
  a.parts = max(1, min(min(slices, kMaxParts), max(1, (a.T <= 40 ? 256 : 512) / a.T)));
  const dim3 grid(a.parts, a.T);
  sample_max_kernel<FMT><<<grid, kThreads, 0, st>>>(a);
  sample_hist_kernel<FMT><<<grid, kThreads, 0, st>>>(a);
  sample_pick_kernel<FMT><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

// What the slices use; more rows, which use none, ask for no more than the
// most rows in slices, so that a workspace serves smaller calls too.  One row's
// at least.
size_t sample_ws(int T, int V) {
  Ws w;
  return ws_layout(min(T, max(1, sliced_rows(V))), nullptr, &w);
}

hipError_t launch_sample(SampleArgs a, hipStream_t st) {
  int bits = 0;      // V <= 2^bits
  while ((int64_t(1) << bits) < a.V) ++bits;
  // a row's masses sum to less than 2^62; a bin's packed sum holds a count up
  // to 2^bits above 2^bits values of frac_bits bits
  a.shift = min(52, 61 - bits);
  a.frac_bits = min(28, 63 - 2 * bits);
  a.q_bits = max(32, bits + a.frac_bits);
  return a.fmt == MOE_W_F32 ? launch<MOE_W_F32>(a, st) : launch<MOE_W_BF16>(a, st);
}

}  // namespace moe
