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
//  1. sample_max_kernel: the largest logit of every slice of a row;
//  2. sample_hist_kernel: sums over 4096 bins of (largest - logit) /
//     temperature, 96 bins per unit: of w, or, for a top_k up to 2048, of
//     ones (no exponential then: the at most 2048 tokens in front of top-k's
//     bin are all listed below).  The last workgroup of a row takes prefix
//     sums over the bins and bounds the bins in which the targets can fall
//     (the sums that top-p and the draw refer to are known up to one bin of
//     the question before);
//  3. sample_pick_kernel: lists the tokens of those bins; the last workgroup
//     of a row answers the three questions exactly among them, by 8 key bits
//     at a time, then among at most 64 tokens within one wave.
//
// w is an integer: rint(exp(.) * 2^s), s chosen so that a row's sum stays
// below 2^62 (s = 43 for 151,936 tokens).  Integer sums have no order, so a
// row's answer does not depend on how it was split, nor on which atomic came
// first, and the steps agree on every sum to the last bit.  exp is evaluated
// in 64 bits (relative error below 1e-14): a draw next to the border between
// two tokens of a flat row needs it, and 64-bit fma runs at the fp32 rate
// here.  Weights that round to zero (below 2^-s / 2 of the largest) are never
// drawn.
//
// Bound: step 1 reads the logits from HBM, the others from the caches as far
// as these hold them; few rows are bound by the three launches' latency.
// The last-workgroup hand-overs wait for nothing: whoever arrives last goes
// on.

#include <hip/hip_runtime.h>

#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kBins = 4096;
constexpr float kBinsPerUnit = 96.0f;   // 42.6 units in all
constexpr double kCutoff = -42.0;       // no weight below: exp(-42) * 2^52 < 0.003
constexpr int kMaxParts = 256;
constexpr int kSlice = 4096;            // logits of a row per workgroup, with few rows
constexpr int kListCap = 16384;         // listed candidates of a row
constexpr int kLdsList = 4096;          // of which this many are searched in LDS
constexpr int kSmallK = 2048;           // top_k up to which every token in front is listed
constexpr int kBinsPerThread = kBins / kThreads;
constexpr int kWaves = kThreads / kWave;
constexpr int kSegment = kLdsList / kWaves;   // a wave's share of the list in LDS

struct RowCtl {
  uint32_t hist_done, pick_done, listed, drawn;   // drawn: rows finished (row 0's only)
  int32_t lo[3], hi[3];       // bins in which the three targets can fall (hi < lo: not asked)
};

// The workspace, from SampleArgs.ws (256-byte aligned).
struct Ws {
  uint64_t* part;    // [T][kMaxParts] largest keys of the slices
  RowCtl* ctl;       // [T]
  uint64_t* mass;    // [T][kBins + 1] sums of w per bin, later their exclusive prefix
  uint32_t* count;   // [T][kBins + 1] the same for counts
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
  w->mass = reinterpret_cast<uint64_t*>(take(size_t(T) * (kBins + 1) * 8));
  w->count = reinterpret_cast<uint32_t*>(take(size_t(T) * (kBins + 1) * 4));
  w->list = reinterpret_cast<uint64_t*>(take(size_t(T) * kListCap * 8));
  return o;
}

// ---- logits

// Elements of one 16-byte load.
template <int FMT>
constexpr int kVec = FMT == MOE_W_F32 ? 4 : 8;

// Row `row` as a range of 16-byte vectors: vector i holds elements
// [i * kVec - lead, ...).
template <int FMT>
struct RowView {
  const uint8_t* base;   // address of vector 0 (16-byte aligned; not read before the row)
  int lead;              // elements of vector 0 in front of the row
  int V;
  int vecs;
  __device__ RowView(const void* logits, int64_t stride, int row, int v) {
    constexpr int size = FMT == MOE_W_F32 ? 4 : 2;
    const uintptr_t a = reinterpret_cast<uintptr_t>(logits) + uintptr_t(row) * stride * size;
    base = reinterpret_cast<const uint8_t*>(a & ~uintptr_t(15));
    lead = int(a & 15) / size;
    V = v;
    vecs = (V + lead + kVec<FMT> - 1) / kVec<FMT>;
  }
  __device__ float at(int i) const {
    if (FMT == MOE_W_F32) return reinterpret_cast<const float*>(base)[lead + int64_t(i)];
    return bf16_to_f32(reinterpret_cast<const uint16_t*>(base)[lead + int64_t(i)]);
  }
  // vector i's logits into x, those outside the row as -infinity
  __device__ void load(int i, float* x) const {
    const int e = i * kVec<FMT> - lead;
    if (e >= 0 && e + kVec<FMT> <= V) {
      const u32x4 q = *reinterpret_cast<const u32x4*>(base + int64_t(i) * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (FMT == MOE_W_F32) {
          x[j] = __uint_as_float(q[j]);
        } else {
          x[2 * j] = __uint_as_float(q[j] << 16);
          x[2 * j + 1] = __uint_as_float(q[j] & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kVec<FMT>; ++j)
        x[j] = e + j >= 0 && e + j < V ? at(e + j) : -__builtin_inff();
    }
  }
};

// Unique key of a token: a larger key comes earlier in the order.
__device__ __forceinline__ uint64_t key_of(float x, int idx) {
  return (uint64_t(ordered_bits(x)) << 32) | uint64_t(~uint32_t(idx));
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t o = uint32_t(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ int index_of(uint64_t key) { return int(~uint32_t(key)); }
// A logit that can be drawn at all: not NaN, not -infinity.
__device__ __forceinline__ bool usable(float x) { return x > -__builtin_inff(); }

// ---- one row's parameters and the weight of a logit

struct Row {
  bool greedy;
  bool small_k;       // the bins hold counts, and every token in front of top-k's bin is listed
  int top_k;          // <= 0: all
  double top_p;       // >= 1: all
  double min_p;
  double u;
  double inv_tau;
  float bin_scale;    // bins per logit
  float bin_limit;    // bins from here on hold no weight
  float top;          // the largest logit
  uint64_t top_key;   // 0: no usable logit
};

__device__ __forceinline__ double exp64(double d, int s, double* scaled) {
  // exp(d), kCutoff <= d <= 0: d = n ln2 + r, |r| <= ln2 / 2 (ln2 as its
  // nearest double and the rest), then the power series to r^12 (remainder
  // below 2e-16).  *scaled = exp(d) * 2^s + 2^52, rounded once: its mantissa
  // is the integer weight.
  const double n = rint(d * 1.4426950408889634);
  double r = fma(n, -0.6931471805599453, d);
  r = fma(n, -2.3190468138462996e-17, r);
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
  const int e = int(n);
  *scaled = fma(p, __longlong_as_double((int64_t)(e + s + 1023) << 52), 0x1p52);
  return p * __longlong_as_double((int64_t)(e + 1023) << 52);
}

// Integer weight of a usable logit (0: never drawn).
__device__ __forceinline__ uint64_t weight_of(const Row& r, float x, int s) {
  const double d = x == r.top ? 0.0 : (double(x) - double(r.top)) * r.inv_tau;
  if (!(d >= kCutoff)) return 0;
  double scaled;
  const double w = exp64(d, s, &scaled);
  if (w < r.min_p) return 0;
  return uint64_t(__double_as_longlong(scaled)) - uint64_t(__double_as_longlong(0x1p52));
}

// (largest - logit) in bins, not below 0; monotone in x.
__device__ __forceinline__ float bins_below(const Row& r, float x) {
  return x == r.top ? 0.0f : (r.top - x) * r.bin_scale;
}
__device__ __forceinline__ int bin_of(const Row& r, float x) {
  return int(fminf(bins_below(r, x), float(kBins - 1)));
}

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint64_t shfl_u64(uint64_t v, int lane) {
  const uint32_t lo = __shfl(uint32_t(v), lane, kWave), hi = __shfl(uint32_t(v >> 32), lane, kWave);
  return (uint64_t(hi) << 32) | lo;
}

__device__ uint64_t block_max(uint64_t v, uint64_t* red) {
  v = wave_max_u64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  uint64_t m = 0;
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) m = max_u64(m, red[w]);
  return m;
}

// The row's parameters; ends with every thread holding them.
__device__ Row read_row(const SampleArgs& a, const Ws& w, int row, uint64_t* red) {
  Row r;
  // every load is under way before the first wait
  uint64_t k = 0;
  if (int(threadIdx.x) < a.parts) k = w.part[int64_t(row) * kMaxParts + threadIdx.x];
  const float tau = a.temperature ? a.temperature[row] : 1.0f;
  const float mp = a.min_p ? a.min_p[row] : 0.0f;
  const float tp = a.top_p ? a.top_p[row] : 1.0f;
  const float u = a.u[row];
  r.top_k = a.top_k ? a.top_k[row] : 0;
  r.top_key = block_max(k, red);
  r.top = logit_of(r.top_key);
  r.top_p = tp < 1.0f ? fmax(double(tp), 0.0) : 1.0;     // NaN: no cut
  r.min_p = mp > 0.0f ? double(mp) : 0.0;
  r.u = u > 0.0f ? fmin(double(u), 1.0) : 0.0;
  r.greedy = !(tau > 0.0f) || mp > 1.0f || r.top_k == 1 || r.top_key == 0;
  r.small_k = r.top_k > 0 && r.top_k <= kSmallK;
  r.inv_tau = r.greedy ? 1.0 : 1.0 / double(tau);
  r.bin_scale = float(fmin(r.inv_tau * double(kBinsPerUnit), 3.0e38));
  // no weight beyond min_p, nor beyond kCutoff (a bin more for the roundings
  // of this logarithm and of the bins)
  const float units = mp > 0.0f ? fminf(-__logf(fminf(mp, 1.0f)), float(-kCutoff)) : float(-kCutoff);
  r.bin_limit = fminf(units * kBinsPerUnit + 2.0f, float(kBins - 1));
  return r;
}

// Inclusive prefix over the workgroup of one (count, mass) pair per thread.
__device__ void block_scan2(uint32_t& c, uint64_t& m, uint64_t* red, uint32_t* redc) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll 1
  for (int d = 1; d < kWave; d <<= 1) {
    const uint32_t oc = __shfl_up(c, d, kWave);
    const uint32_t ol = __shfl_up(uint32_t(m), d, kWave), oh = __shfl_up(uint32_t(m >> 32), d, kWave);
    if (lane >= d) {
      c += oc;
      m += (uint64_t(oh) << 32) | ol;
    }
  }
  __syncthreads();
  if (lane == 63) red[wave] = m, redc[wave] = c;
  __syncthreads();
#pragma unroll 1
  for (int w = 0; w < wave; ++w) c += redc[w], m += red[w];
}

// First bin whose inclusive prefix reaches target (kBins - 1 if none does).
template <class Tp>
__device__ __forceinline__ int first_reaching(const Tp* prefix, Tp target) {
  int b = -1;
#pragma unroll 1
  for (int step = kBins / 2; step; step >>= 1)
    if (prefix[b + step] < target) b += step;
  return b + 1;
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

// What workgroups of one launch hand to each other goes through relaxed
// device-scope atomics, which act on memory that every XCD sees, and the
// arrival is counted once they have completed.  A device-scope fence would
// write back the XCD's whole L2 instead (measured: the sums of 64 rows took
// 53 us with one per wave).
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

// A slice's 16-byte vectors, two at a time per thread: f(x, first index).
template <int FMT, class F>
__device__ __forceinline__ void for_slice(const RowView<FMT>& v, int begin, int end, const F& f) {
#pragma unroll 1
  for (int i = begin + int(threadIdx.x); i < end; i += 2 * kThreads) {
    float x[2][kVec<FMT>];
    v.load(i, x[0]);
    const bool two = i + kThreads < end;
    if (two) v.load(i + kThreads, x[1]);
    f(x[0], i * kVec<FMT> - v.lead);
    if (two) f(x[1], (i + kThreads) * kVec<FMT> - v.lead);
  }
}

// ---- 1. largest logit of every slice; clears the row's sums

template <int FMT>
__global__ __launch_bounds__(kThreads) void sample_max_kernel(const SampleArgs a) {
  __shared__ uint64_t red[kWaves];
  Ws w;
  ws_layout(a.T, static_cast<uint8_t*>(a.ws), &w);
  const int p = blockIdx.x, row = blockIdx.y;
  // this slice's share of the bins, and the row's counters
  const int per_bins = (kBins + 1 + a.parts - 1) / a.parts;
  const int b1 = min(kBins + 1, (p + 1) * per_bins);
  for (int b = p * per_bins + threadIdx.x; b < b1; b += kThreads) {
    w.mass[int64_t(row) * (kBins + 1) + b] = 0;
    w.count[int64_t(row) * (kBins + 1) + b] = 0;
  }
  if (p == 0 && threadIdx.x < sizeof(RowCtl) / 4)
    reinterpret_cast<uint32_t*>(&w.ctl[row])[threadIdx.x] = 0;

  const RowView<FMT> v(a.logits, a.stride, row, a.V);
  const int per = (v.vecs + a.parts - 1) / a.parts;
  float best = -__builtin_inff();
  int at = 0;
  for_slice<FMT>(v, p * per, min(v.vecs, (p + 1) * per), [&](const float* x, int first) {
#pragma unroll
    for (int j = 0; j < kVec<FMT>; ++j)
      if (x[j] > best) best = x[j], at = first + j;   // the first of equal ones
  });
  const uint64_t k = block_max(usable(best) ? key_of(best, at) : 0, red);
  if (threadIdx.x == 0) w.part[int64_t(row) * kMaxParts + p] = k;
}

// ---- 2. sums per bin, then the bins that matter

template <int FMT>
__global__ __launch_bounds__(kThreads) void sample_hist_kernel(const SampleArgs a) {
  __shared__ uint64_t mass[kBins];
  __shared__ uint32_t count[kBins];
  __shared__ uint64_t red[kWaves];
  __shared__ uint32_t redc[kWaves];
  __shared__ uint32_t flag;
  Ws w;
  ws_layout(a.T, static_cast<uint8_t*>(a.ws), &w);
  const int row = blockIdx.y;
  const Row r = read_row(a, w, row, red);
  if (r.greedy) return;
  const bool want_mass = !r.small_k, want_count = r.top_k > 0;
#pragma unroll 1
  for (int b = threadIdx.x; b < kBins; b += kThreads) mass[b] = 0, count[b] = 0;
  __syncthreads();
  const RowView<FMT> v(a.logits, a.stride, row, a.V);
  const int per = (v.vecs + a.parts - 1) / a.parts;
  for_slice<FMT>(v, int(blockIdx.x) * per, min(v.vecs, (int(blockIdx.x) + 1) * per),
                 [&](const float* x, int) {
#pragma unroll
    for (int j = 0; j < kVec<FMT>; ++j) {
      const float bins = bins_below(r, x[j]);
      if (!usable(x[j]) || !(bins < r.bin_limit)) continue;
      const int b = int(bins);
      if (want_mass) {
        const uint64_t m = weight_of(r, x[j], a.shift);
        if (m == 0) continue;
        atomicAdd(reinterpret_cast<unsigned long long*>(&mass[b]), (unsigned long long)m);
      }
      if (want_count) atomicAdd(&count[b], 1u);
    }
  });
  __syncthreads();
  uint64_t* gm = w.mass + int64_t(row) * (kBins + 1);
  uint32_t* gc = w.count + int64_t(row) * (kBins + 1);
#pragma unroll 1
  for (int b = threadIdx.x; b < kBins; b += kThreads) {
    if (mass[b]) __hip_atomic_fetch_add(&gm[b], mass[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (count[b]) __hip_atomic_fetch_add(&gc[b], count[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (!arrive_last(&w.ctl[row].hist_done, a.parts, &flag)) return;

  // inclusive prefix sums over the bins, in LDS and in place
  uint64_t m[kBinsPerThread], mp = 0;
  uint32_t c[kBinsPerThread], cp = 0;
  const int b0 = int(threadIdx.x) * kBinsPerThread;
#pragma unroll
  for (int j = 0; j < kBinsPerThread; ++j) {
    m[j] = get(&gm[b0 + j]);
    c[j] = get(&gc[b0 + j]);
  }
#pragma unroll
  for (int j = 0; j < kBinsPerThread; ++j) mp += m[j], cp += c[j];
  block_scan2(cp, mp, red, redc);
#pragma unroll
  for (int j = kBinsPerThread - 1; j >= 0; --j) {
    mass[b0 + j] = mp;
    count[b0 + j] = cp;
    mp -= m[j];
    cp -= c[j];
  }
  __syncthreads();
#pragma unroll 1
  for (int b = threadIdx.x; b < kBins; b += kThreads) gm[b + 1] = mass[b], gc[b + 1] = count[b];
  if (threadIdx.x == 0) gm[0] = 0, gc[0] = 0;
  // bins [lo, hi] where each target can fall; every thread finds the same
  const uint64_t mtot = mass[kBins - 1];
  const uint32_t ctot = count[kBins - 1];
  int lo[3] = {0, 0, 0}, hi[3] = {-1, -1, -1};
  uint64_t z0 = mtot, z1 = mtot;      // bounds of the sum kept so far
  if (want_count && uint32_t(r.top_k) < ctot) {
    const int b = first_reaching(count, uint32_t(r.top_k));
    lo[0] = hi[0] = b;
    z0 = (b ? mass[b - 1] : 0) + 1;   // at least one of the bin's tokens is kept
    z1 = mass[b];
  }
  if (want_mass) {
    if (r.top_p < 1.0) {
      lo[1] = first_reaching(mass, top_p_target(r.top_p, z0));
      hi[1] = first_reaching(mass, top_p_target(r.top_p, z1));
      z0 = (lo[1] ? mass[lo[1] - 1] : 0) + 1;
      z1 = mass[hi[1]];
    }
    lo[2] = first_reaching(mass, draw_target(r.u, z0));
    hi[2] = first_reaching(mass, draw_target(r.u, z1));
  } else {
    // counts only: every token up to top-k's bin is listed
    lo[1] = 0;
    hi[1] = hi[0] >= 0 ? hi[0] : kBins - 1;
  }
  if (threadIdx.x == 0) {
#pragma unroll
    for (int q = 0; q < 3; ++q) w.ctl[row].lo[q] = lo[q], w.ctl[row].hi[q] = hi[q];
  }
}

// ---- 3. the tokens of those bins, and the three answers

struct PickLds {
  uint64_t list[kLdsList];
  uint64_t hmass[256];
  uint32_t hcount[256];
  uint64_t few[64];
  uint64_t red[kWaves];
  uint64_t all_or, all_and, key, sum, prefix;
  uint32_t n, flag, last;
  int32_t bin;
};

// The three questions of one row among its candidates (for_each(f) calls
// f(key) for each): the drawn token's key, and the kept sum.
template <class ForEach>
__device__ uint64_t draw_token(const Row& r, const uint64_t* gm, const uint32_t* gc, int shift,
                               const int* lo, const int* hi, PickLds& s, uint64_t* kept,
                               const ForEach& for_each) {
  uint64_t z = gm[kBins];     // (with small_k: set by the first question)
  uint64_t last_key = 0;      // tokens behind this key are cut off (small_k)
#pragma unroll 1
  for (int q = 0; q < 3; ++q) {
    const bool by_count = q == 0;
    if (q < 2 && hi[q] < lo[q]) {
      if (!(q == 0 && r.small_k)) continue;
    }
    if (q == 1 && !(r.top_p < 1.0)) continue;
    __syncthreads();
    if (threadIdx.x == 0) s.all_or = 0, s.all_and = ~0ull, s.n = 0, s.bin = -1, s.sum = 0, s.key = 0;
    __syncthreads();
    uint64_t target = by_count ? uint64_t(r.top_k) : q == 1 ? top_p_target(r.top_p, z)
                                                           : draw_target(r.u, z);
    const bool ask = !by_count || hi[0] >= lo[0];   // (small_k without a cut: the sum alone)
    uint64_t base = 0;
    int bin = -1;
    if (!r.small_k || by_count) {
      // the bin, and the sum in front of it
#pragma unroll 1
      for (int b = lo[q] + int(threadIdx.x); b <= hi[q]; b += kThreads) {
        const uint64_t before = by_count ? uint64_t(gc[b]) : gm[b];
        const uint64_t after = by_count ? uint64_t(gc[b + 1]) : gm[b + 1];
        if (before < target && after >= target) s.bin = b, s.sum = before;
      }
      __syncthreads();
      bin = s.bin;
      base = s.sum;
    }
    // narrow the key range to at most 64 tokens, 8 bits at a time from the
    // highest bit in which the keys differ
    int sh = 64;
    uint64_t prefix = 0;
    auto active = [&](uint64_t key) {
      return (sh == 64 || (key >> sh) == prefix) && key >= last_key &&
             (bin < 0 || bin_of(r, logit_of(key)) == bin);
    };
    if (ask) {
      uint32_t left = 0;
#pragma unroll 1
      for (;;) {
        // the active tokens, if there are few
        uint64_t o = 0, n = ~0ull;
        for_each([&](uint64_t key) {
          if (active(key)) {
            o |= key, n &= key;
            const uint32_t i = atomicAdd(&s.n, 1u);
            if (i < 64) s.few[i] = key;
          }
        });
        if (sh == 64 && n != ~0ull) {
          atomicOr(reinterpret_cast<unsigned long long*>(&s.all_or), (unsigned long long)o);
          atomicAnd(reinterpret_cast<unsigned long long*>(&s.all_and), (unsigned long long)n);
        }
        __syncthreads();
        left = s.n;
        if (left <= 64 || sh == 0) break;
        int from = sh;
        if (sh == 64) {
          const uint64_t differ = s.all_or & ~s.all_and;   // not 0: keys are unique
          from = 64 - __clzll((long long)differ);
          prefix = from == 64 ? 0 : s.all_or >> from;
        }
        sh = from;
        const int next = sh > 8 ? sh - 8 : 0;
        const uint64_t digits = (uint64_t(1) << (sh - next)) - 1;
        __syncthreads();
        if (threadIdx.x < 256) s.hmass[threadIdx.x] = 0, s.hcount[threadIdx.x] = 0;
        if (threadIdx.x == 0) s.n = 0;
        __syncthreads();
        for_each([&](uint64_t key) {
          if (!active(key)) return;
          const int d = int((key >> next) & digits);
          if (by_count)
            atomicAdd(&s.hcount[d], 1u);
          else
            atomicAdd(reinterpret_cast<unsigned long long*>(&s.hmass[d]),
                      (unsigned long long)weight_of(r, logit_of(key), shift));
        });
        __syncthreads();
        if (threadIdx.x < 64) {
          // lane i holds digits 255 - 4i .. 252 - 4i: descending
          uint64_t v[4], sum = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = 255 - 4 * int(threadIdx.x) - j;
            v[j] = by_count ? uint64_t(s.hcount[d]) : s.hmass[d];
            sum += v[j];
          }
          uint64_t inc = sum;
#pragma unroll 1
          for (int d = 1; d < kWave; d <<= 1) {
            const uint64_t before = shfl_u64(inc, max(0, int(threadIdx.x) - d));
            if (int(threadIdx.x) >= d) inc += before;
          }
          uint64_t before = base + inc - sum;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (before < target && before + v[j] >= target) {
              s.prefix = ((sh == 64 ? 0 : prefix) << (sh - next)) |
                         uint64_t(255 - 4 * int(threadIdx.x) - j);
              s.sum = before;
            }
            before += v[j];
          }
        }
        __syncthreads();
        prefix = s.prefix;
        base = s.sum;
        sh = next;
      }
      if (threadIdx.x < 64) {
        const uint32_t n = min(left, 64u);
        const bool have = threadIdx.x < n;
        const uint64_t key = have ? s.few[threadIdx.x] : 0;
        const uint64_t mine = !have ? 0 : by_count ? 1 : weight_of(r, logit_of(key), shift);
        uint64_t front = base;     // the sum in front of this token
#pragma unroll 1
        for (uint32_t j = 0; j < n; ++j) {
          const uint64_t ok = shfl_u64(key, int(j)), om = shfl_u64(mine, int(j));
          if (ok > key) front += om;
        }
        if (have && front < target && front + mine >= target) {
          s.key = key;
          s.sum = front + mine;    // through this token
        }
      }
      __syncthreads();
    }
    const uint64_t key = s.key;
    if (q == 2) {
      *kept = z;
      return key;
    }
    z = s.sum;
    if (by_count) {
      // the mass through top-k's token: of its bin's tokens up to it, or of all listed ones
      __syncthreads();
      if (threadIdx.x == 0) s.sum = 0;
      __syncthreads();
      uint64_t part = 0;
      for_each([&](uint64_t k2) {
        if (k2 >= key && (r.small_k || bin_of(r, logit_of(k2)) == bin))
          part += weight_of(r, logit_of(k2), shift);
      });
      if (part) atomicAdd(reinterpret_cast<unsigned long long*>(&s.sum), (unsigned long long)part);
      __syncthreads();
      z = s.sum + (r.small_k ? 0 : gm[bin]);
      if (r.small_k) last_key = key;
    }
  }
  return 0;   // not reached: the third question returns
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

template <int FMT>
__global__ __launch_bounds__(kThreads) void sample_pick_kernel(const SampleArgs a) {
  __shared__ PickLds s;
  Ws w;
  ws_layout(a.T, static_cast<uint8_t*>(a.ws), &w);
  const int row = blockIdx.y;
  RowCtl& ctl = w.ctl[row];
  int lo[3], hi[3];
#pragma unroll
  for (int q = 0; q < 3; ++q) lo[q] = ctl.lo[q], hi[q] = ctl.hi[q];
  const Row r = read_row(a, w, row, s.red);
  if (r.greedy) {
    if (blockIdx.x == 0)
      finish_row(a, w, row, r.top_key ? index_of(r.top_key) : -1, r.top_key ? 1.0f : 0.0f, &s.flag);
    return;
  }
  // no candidate lies beyond `deepest` (a bin past the last, or the limit)
  const float deepest = fminf(float(max(max(hi[0], hi[1]), hi[2]) + 1), r.bin_limit);
  auto wanted = [&](float x) {
    const float bins = bins_below(r, x);
    if (!(bins < deepest) || !usable(x)) return false;
    const int b = int(bins);
    return (b >= lo[0] && b <= hi[0]) || (b >= lo[1] && b <= hi[1]) || (b >= lo[2] && b <= hi[2]);
  };
  uint64_t* list = w.list + int64_t(row) * kListCap;
  const RowView<FMT> v(a.logits, a.stride, row, a.V);
  const int per = (v.vecs + a.parts - 1) / a.parts;
  const int begin = int(blockIdx.x) * per, end = min(v.vecs, begin + per);
  {
    // each wave fills its own segment in LDS and empties it into the list
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t* seg = s.list + wave * kSegment;
    uint32_t n = 0;
    auto empty = [&]() {
      uint32_t at = 0;
      if (lane == 0)
        at = __hip_atomic_fetch_add(&ctl.listed, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      at = __shfl(at, 0, kWave);
      __builtin_amdgcn_wave_barrier();   // the segment's writes stay in front of its reads
#pragma unroll 1
      for (uint32_t k = lane; k < n; k += kWave)
        if (at + k < uint32_t(kListCap)) put(&list[at + k], seg[k]);
      __builtin_amdgcn_wave_barrier();
      n = 0;
    };
    auto take = [&](const float* x, int first, bool in) {
      bool want[kVec<FMT>], any = false;
#pragma unroll
      for (int j = 0; j < kVec<FMT>; ++j) {
        want[j] = in && wanted(x[j]);
        any |= want[j];
      }
      if (__ballot(any) == 0) return;
      if (n + 64 * kVec<FMT> > uint32_t(kSegment)) empty();
#pragma unroll
      for (int j = 0; j < kVec<FMT>; ++j) {
        const uint64_t mask = __ballot(want[j]);
        if (want[j])
          seg[n + __popcll(mask & ((uint64_t(1) << lane) - 1))] = key_of(x[j], first + j);
        n += uint32_t(__popcll(mask));
      }
    };
    // whole waves take part in every step
#pragma unroll 1
    for (int i0 = begin + wave * kWave; i0 < end; i0 += 2 * kThreads) {
      float x[2][kVec<FMT>];
      const int i = i0 + lane, i2 = i + kThreads;
      if (i < end) v.load(i, x[0]);
      if (i2 < end) v.load(i2, x[1]);
      take(x[0], i * kVec<FMT> - v.lead, i < end);
      take(x[1], i2 * kVec<FMT> - v.lead, i2 < end);
    }
    if (n) empty();
  }
  if (!arrive_last(&ctl.pick_done, a.parts, &s.last)) return;

  const uint64_t* gm = w.mass + int64_t(row) * (kBins + 1);
  const uint32_t* gc = w.count + int64_t(row) * (kBins + 1);
  const uint32_t n = get(&ctl.listed);
  uint64_t key, kept = 1;
  if (n <= uint32_t(kListCap)) {
    const bool in_lds = n <= uint32_t(kLdsList);
    if (in_lds)
      for (uint32_t k = threadIdx.x; k < n; k += kThreads) s.list[k] = get(&list[k]);
    __syncthreads();
    key = draw_token(r, gm, gc, a.shift, lo, hi, s, &kept, [&](auto&& f) {
#pragma unroll 1
      for (uint32_t k = threadIdx.x; k < n; k += kThreads) f(in_lds ? s.list[k] : get(&list[k]));
    });
  } else {
    // more candidates than the list holds (long runs of equal logits): the row itself
    key = draw_token(r, gm, gc, a.shift, lo, hi, s, &kept, [&](auto&& f) {
#pragma unroll 1
      for (int i = threadIdx.x; i < a.V; i += kThreads) {
        const float x = v.at(i);
        if (wanted(x)) f(key_of(x, i));
      }
    });
  }
  const float x = logit_of(key);
  const double d = x == r.top ? 0.0 : (double(x) - double(r.top)) * r.inv_tau;
  double scaled;
  const double weight = exp64(fmax(d, kCutoff), a.shift, &scaled);
  const double prob = weight * __longlong_as_double((int64_t)(a.shift + 1023) << 52) / double(kept);
  __syncthreads();
  finish_row(a, w, row, index_of(key), float(prob), &s.flag);
}

template <int FMT>
hipError_t launch(const SampleArgs& a, hipStream_t st) {
  const dim3 grid(a.parts, a.T);
  sample_max_kernel<FMT><<<grid, kThreads, 0, st>>>(a);
  sample_hist_kernel<FMT><<<grid, kThreads, 0, st>>>(a);
  sample_pick_kernel<FMT><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t sample_ws(int T) {
  Ws w;
  return ws_layout(T, nullptr, &w);
}

hipError_t launch_sample(SampleArgs a, hipStream_t st) {
  // a slice per workgroup for few rows; for many, as many workgroups as the
  // 256 CUs hold at once (three each, by the bins' LDS)
  const int slices = (a.V + kSlice - 1) / kSlice;
  a.parts = max(1, min(min(slices, kMaxParts), max(1, 768 / a.T)));
  // a row's weights sum to less than 2^62 and convert exactly from a double
  int bits = 0;
  while ((int64_t(1) << bits) < a.V) ++bits;
  a.shift = min(52, 61 - bits);
  return a.fmt == MOE_W_F32 ? launch<MOE_W_F32>(a, st) : launch<MOE_W_BF16>(a, st);
}

}  // namespace moe
