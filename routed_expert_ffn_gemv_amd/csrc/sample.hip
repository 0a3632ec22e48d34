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
//  2. sample_hist_kernel: count and sum of w over 4096 bins of (largest -
//     logit) / temperature, 96 bins per unit.  The last workgroup of a row
//     takes prefix sums over the bins and bounds the bins in which the
//     three targets can fall (the sums that top-p and the draw refer to are
//     known up to one bin of the question before);
//  3. sample_pick_kernel: collects the tokens of those few bins; the last
//     workgroup of a row answers the three questions exactly among them, by
//     8 key bits at a time, then among at most 64 tokens within one wave.
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
constexpr int kTile = 4096;             // logits a workgroup takes at a time: 8 per thread
constexpr int kPerThread = kTile / kThreads;
constexpr int kListCap = 16384;         // listed candidates of a row
constexpr int kLdsList = 4096;          // of which this many are searched in LDS
constexpr int kBinsPerThread = kBins / kThreads;

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
  int top_k;          // <= 0: all
  double top_p;       // >= 1: all
  double min_p;
  double u;
  double inv_tau;
  float bin_scale;    // bins per logit
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

__device__ __forceinline__ int bin_of(const Row& r, float x) {
  if (x == r.top) return 0;
  const float b = (r.top - x) * r.bin_scale;   // monotone in x
  return b < float(kBins - 1) ? int(b) : kBins - 1;
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
  uint64_t k = 0;
  if (int(threadIdx.x) < a.parts) k = w.part[int64_t(row) * kMaxParts + threadIdx.x];
  r.top_key = block_max(k, red);
  r.top = logit_of(r.top_key);
  const float tau = a.temperature ? a.temperature[row] : 1.0f;
  const float mp = a.min_p ? a.min_p[row] : 0.0f;
  const float tp = a.top_p ? a.top_p[row] : 1.0f;
  const float u = a.u[row];
  r.top_k = a.top_k ? a.top_k[row] : 0;
  r.top_p = tp < 1.0f ? fmax(double(tp), 0.0) : 1.0;     // NaN: no cut
  r.min_p = mp > 0.0f ? double(mp) : 0.0;
  r.u = u > 0.0f ? fmin(double(u), 1.0) : 0.0;
  r.greedy = !(tau > 0.0f) || mp > 1.0f || r.top_k == 1 || r.top_key == 0;
  r.inv_tau = r.greedy ? 1.0 : 1.0 / double(tau);
  r.bin_scale = float(fmin(r.inv_tau * double(kBinsPerUnit), 3.0e38));
  return r;
}

// Exclusive prefix over the workgroup of (count, mass) pairs; tot_* receive the totals.
__device__ void block_scan2(uint32_t& c, uint64_t& m, uint64_t* red, uint32_t* redc,
                            uint32_t* tot_c, uint64_t* tot_m) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t ic = c;
  uint64_t im = m;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const uint32_t oc = __shfl_up(ic, d, kWave);
    const uint32_t ol = __shfl_up(uint32_t(im), d, kWave), oh = __shfl_up(uint32_t(im >> 32), d, kWave);
    if (lane >= d) {
      ic += oc;
      im += (uint64_t(oh) << 32) | ol;
    }
  }
  __syncthreads();
  if (lane == 63) red[wave] = im, redc[wave] = ic;
  __syncthreads();
  uint32_t bc = 0, sc = 0;
  uint64_t bm = 0, sm = 0;
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) {
    if (w < wave) bc += redc[w], bm += red[w];
    sc += redc[w];
    sm += red[w];
  }
  c = bc + ic - c;
  m = bm + im - m;
  *tot_c = sc;
  *tot_m = sm;
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

// Whether this workgroup is the last of `n` to arrive at `counter`; what the
// others wrote before arriving is visible to it afterwards.
__device__ bool arrive_last(uint32_t* counter, uint32_t n, uint32_t* flag) {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
  __syncthreads();
  if (threadIdx.x == 0)
    *flag = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const bool last = *flag == n - 1;
  if (last) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  return last;
}

// ---- 1. largest logit of every slice; clears the row's sums

template <int FMT>
__global__ __launch_bounds__(kThreads) void sample_max_kernel(const SampleArgs a) {
  __shared__ uint64_t red[kThreads / kWave];
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
  const int end = min(v.vecs, (p + 1) * per);
  float best = -__builtin_inff();
  int at = 0;
  for (int i = p * per + threadIdx.x; i < end; i += kThreads) {
    float x[kVec<FMT>];
    v.load(i, x);
#pragma unroll
    for (int j = 0; j < kVec<FMT>; ++j)
      if (x[j] > best) best = x[j], at = i * kVec<FMT> - v.lead + j;   // the first of equal ones
  }
  const uint64_t k = block_max(usable(best) ? key_of(best, at) : 0, red);
  if (threadIdx.x == 0) w.part[int64_t(row) * kMaxParts + p] = k;
}

// ---- 2. sums per bin, then the bins that matter

template <int FMT>
__global__ __launch_bounds__(kThreads) void sample_hist_kernel(const SampleArgs a) {
  __shared__ uint64_t mass[kBins];
  __shared__ uint32_t count[kBins];
  __shared__ uint64_t red[kThreads / kWave];
  __shared__ uint32_t redc[kThreads / kWave];
  __shared__ uint32_t flag;
  __shared__ int bound[6];
  __shared__ uint64_t at_k[2];   // mass in front of the top-k bin, and through it
  __shared__ uint64_t at_n[2];
  Ws w;
  ws_layout(a.T, static_cast<uint8_t*>(a.ws), &w);
  const int row = blockIdx.y;
  const Row r = read_row(a, w, row, red);
  if (r.greedy) return;
  for (int b = threadIdx.x; b < kBins; b += kThreads) mass[b] = 0, count[b] = 0;
  __syncthreads();
  const RowView<FMT> v(a.logits, a.stride, row, a.V);
  const int per = (v.vecs + a.parts - 1) / a.parts;
  const int end = min(v.vecs, (int(blockIdx.x) + 1) * per);
  for (int i = int(blockIdx.x) * per + threadIdx.x; i < end; i += kThreads) {
    float x[kVec<FMT>];
    v.load(i, x);
#pragma unroll
    for (int j = 0; j < kVec<FMT>; ++j) {
      if (!usable(x[j])) continue;
      const uint64_t m = weight_of(r, x[j], a.shift);
      if (m == 0) continue;
      const int b = bin_of(r, x[j]);
      atomicAdd(reinterpret_cast<unsigned long long*>(&mass[b]), (unsigned long long)m);
      atomicAdd(&count[b], 1u);
    }
  }
  __syncthreads();
  uint64_t* gm = w.mass + int64_t(row) * (kBins + 1);
  uint32_t* gc = w.count + int64_t(row) * (kBins + 1);
  for (int b = threadIdx.x; b < kBins; b += kThreads)
    if (count[b]) {
      __hip_atomic_fetch_add(&gm[b], mass[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_fetch_add(&gc[b], count[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  if (!arrive_last(&w.ctl[row].hist_done, a.parts, &flag)) return;

  // exclusive prefix sums over the bins, in place
  uint64_t m[kBinsPerThread], msum = 0, mtot;
  uint32_t c[kBinsPerThread], csum = 0, ctot;
#pragma unroll
  for (int j = 0; j < kBinsPerThread; ++j) {
    m[j] = gm[threadIdx.x * kBinsPerThread + j];
    c[j] = gc[threadIdx.x * kBinsPerThread + j];
    msum += m[j];
    csum += c[j];
  }
  uint64_t mpre = msum;
  uint32_t cpre = csum;
  block_scan2(cpre, mpre, red, redc, &ctot, &mtot);
  // bins where each target can fall: [lo, hi] per question
  if (threadIdx.x < 6) bound[threadIdx.x] = (threadIdx.x & 1) ? -1 : 0;
  if (threadIdx.x == 0) at_k[0] = at_k[1] = mtot, at_n[0] = at_n[1] = mtot;
  __syncthreads();
  const bool ask_k = r.top_k > 0 && uint32_t(r.top_k) < ctot;
  uint64_t mb = mpre;
  uint32_t cb = cpre;
#pragma unroll
  for (int j = 0; j < kBinsPerThread; ++j) {
    const int b = threadIdx.x * kBinsPerThread + j;
    gm[b] = mb;
    gc[b] = cb;
    if (ask_k && cb < uint32_t(r.top_k) && cb + c[j] >= uint32_t(r.top_k)) {
      bound[0] = bound[1] = b;
      at_k[0] = mb + 1;        // at least one of the bin's tokens is kept
      at_k[1] = mb + m[j];
    }
    mb += m[j];
    cb += c[j];
  }
  if (threadIdx.x == kThreads - 1) gm[kBins] = mb, gc[kBins] = cb;
  __syncthreads();
  const bool ask_p = r.top_p < 1.0;
  // question q's bins between the targets lo_t and hi_t; the mass in front of
  // the first, and through the last, bound the next question's sum
  auto bins_of = [&](int q, uint64_t lo_t, uint64_t hi_t, uint64_t* edge) {
    uint64_t before = mpre;
#pragma unroll
    for (int j = 0; j < kBinsPerThread; ++j) {
      const int b = threadIdx.x * kBinsPerThread + j;
      const uint64_t after = before + m[j];
      if (before < lo_t && after >= lo_t) bound[2 * q] = b, edge[0] = before + 1;
      if (before < hi_t && after >= hi_t) bound[2 * q + 1] = b, edge[1] = after;
      before = after;
    }
    __syncthreads();
  };
  if (ask_p) {
    bins_of(1, top_p_target(r.top_p, at_k[0]), top_p_target(r.top_p, at_k[1]), at_n);
  } else if (threadIdx.x == 0) {
    at_n[0] = at_k[0];
    at_n[1] = at_k[1];
  }
  __syncthreads();
  const uint64_t lo_t = draw_target(r.u, at_n[0]), hi_t = draw_target(r.u, at_n[1]);
  __syncthreads();
  bins_of(2, lo_t, hi_t, at_k);
  if (threadIdx.x < 3) {
    w.ctl[row].lo[threadIdx.x] = bound[2 * threadIdx.x];
    w.ctl[row].hi[threadIdx.x] = bound[2 * threadIdx.x + 1];
  }
}

// ---- 3. the tokens of those bins, and the three answers

struct PickLds {
  uint64_t list[kLdsList];
  uint64_t hmass[256];
  uint32_t hcount[256];
  uint64_t few[64];
  uint64_t red[kThreads / kWave];
  uint64_t all_or, all_and, key, base, prefix;
  uint32_t n, flag, left, last;
  int32_t bin;
};

// The boundary token of one question among a row's candidates.
template <int FMT, class ForEach>
__device__ uint64_t find_token(const Row& r, const Ws& w, int row, int shift, bool by_count,
                               uint64_t target, int lo, int hi, PickLds& s, uint64_t* upto,
                               const ForEach& for_each) {
  const uint64_t* gm = w.mass + int64_t(row) * (kBins + 1);
  const uint32_t* gc = w.count + int64_t(row) * (kBins + 1);
  // the bin, and the sum in front of it
  __syncthreads();
  if (threadIdx.x == 0) s.all_or = 0, s.all_and = ~0ull, s.n = 0, s.bin = lo, s.base = 0, s.left = 0;
  __syncthreads();
  for (int b = lo + int(threadIdx.x); b <= hi; b += kThreads) {
    const uint64_t before = by_count ? uint64_t(gc[b]) : gm[b];
    const uint64_t after = by_count ? uint64_t(gc[b + 1]) : gm[b + 1];
    if (before < target && after >= target) s.bin = b, s.base = before, s.left = gc[b + 1] - gc[b];
  }
  __syncthreads();
  const int bin = s.bin;
  uint64_t base = s.base;
  uint32_t left = s.left;
  // narrow the key range to at most 64 tokens, 8 bits at a time from the
  // highest bit in which the bin's keys differ
  int sh = 64;
  uint64_t prefix = 0;
  auto active = [&](uint64_t key) {
    return (sh == 64 || (key >> sh) == prefix) && bin_of(r, logit_of(key)) == bin;
  };
  if (left > 64) {
    uint64_t o = 0, n = ~0ull;
    for_each([&](uint64_t key) {
      if (active(key)) o |= key, n &= key;
    });
    atomicOr(reinterpret_cast<unsigned long long*>(&s.all_or), (unsigned long long)o);
    atomicAnd(reinterpret_cast<unsigned long long*>(&s.all_and), (unsigned long long)n);
    __syncthreads();
    const uint64_t differ = s.all_or & ~s.all_and;
    sh = 64 - __clzll((long long)differ);     // more than one key: differ != 0
    prefix = sh == 64 ? 0 : s.all_or >> sh;
  }
  while (left > 64 && sh > 0) {
    const int next = sh > 8 ? sh - 8 : 0;
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += kThreads) s.hmass[i] = 0, s.hcount[i] = 0;
    __syncthreads();
    const uint64_t digits = (uint64_t(1) << (sh - next)) - 1;
    for_each([&](uint64_t key) {
      if (!active(key)) return;
      const int d = int((key >> next) & digits);
      if (!by_count)
        atomicAdd(reinterpret_cast<unsigned long long*>(&s.hmass[d]),
                  (unsigned long long)weight_of(r, logit_of(key), shift));
      atomicAdd(&s.hcount[d], 1u);
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
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const uint64_t o = shfl_u64(inc, max(0, int(threadIdx.x) - d));
        if (int(threadIdx.x) >= d) inc += o;
      }
      uint64_t before = base + inc - sum;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (before < target && before + v[j] >= target) {
          const int d = 255 - 4 * int(threadIdx.x) - j;
          s.prefix = ((sh == 64 ? 0 : prefix) << (sh - next)) | uint64_t(d);
          s.base = before;
          s.left = s.hcount[d];
        }
        before += v[j];
      }
    }
    __syncthreads();
    prefix = s.prefix;
    base = s.base;
    left = s.left;
    sh = next;
  }
  for_each([&](uint64_t key) {
    if (active(key)) {
      const uint32_t i = atomicAdd(&s.n, 1u);
      if (i < 64) s.few[i] = key;
    }
  });
  __syncthreads();
  if (threadIdx.x < 64) {
    const uint32_t n = min(s.n, 64u);
    const bool have = threadIdx.x < n;
    const uint64_t key = have ? s.few[threadIdx.x] : 0;
    const uint64_t mass = have ? weight_of(r, logit_of(key), shift) : 0;
    const uint64_t mine = by_count ? (have ? 1 : 0) : mass;
    uint64_t front = 0, front_mass = 0;     // of the tokens ahead of this one
    for (uint32_t j = 0; j < n; ++j) {
      const uint64_t ok = shfl_u64(key, int(j)), om = shfl_u64(mass, int(j));
      if (ok > key) front_mass += om, front += by_count ? 1 : om;
    }
    if (have && base + front < target && base + front + mine >= target) {
      s.key = key;
      s.all_or = front_mass + mass;      // of these few, through this token
    }
  }
  __syncthreads();
  const uint64_t key = s.key;
  if (upto) {
    // mass through the boundary token
    if (!by_count) {
      *upto = base + s.all_or;
    } else {
      // the bin's tokens ahead of the few are not among them: sum again
      __syncthreads();
      if (threadIdx.x == 0) s.base = 0;
      __syncthreads();
      uint64_t part = 0;
      for_each([&](uint64_t k2) {
        if (k2 >= key && bin_of(r, logit_of(k2)) == bin) part += weight_of(r, logit_of(k2), shift);
      });
      if (part)
        atomicAdd(reinterpret_cast<unsigned long long*>(&s.base), (unsigned long long)part);
      __syncthreads();
      *upto = gm[bin] + s.base;
    }
  }
  return key;
}

template <int FMT, class ForEach>
__device__ uint64_t draw_token(const SampleArgs& a, const Row& r, const Ws& w, int row, PickLds& s,
                               double* prob, const ForEach& for_each) {
  const RowCtl& ctl = w.ctl[row];
  uint64_t z = w.mass[int64_t(row) * (kBins + 1) + kBins];
  const int lo0 = ctl.lo[0], hi0 = ctl.hi[0], lo1 = ctl.lo[1], hi1 = ctl.hi[1];
  if (hi0 >= lo0)
    find_token<FMT>(r, w, row, a.shift, true, uint64_t(r.top_k), lo0, hi0, s, &z, for_each);
  if (hi1 >= lo1)
    find_token<FMT>(r, w, row, a.shift, false, top_p_target(r.top_p, z), lo1, hi1, s, &z, for_each);
  const uint64_t key = find_token<FMT>(r, w, row, a.shift, false, draw_target(r.u, z), ctl.lo[2],
                                       ctl.hi[2], s, nullptr, for_each);
  const float x = logit_of(key);
  double scaled;
  const double d = x == r.top ? 0.0 : (double(x) - double(r.top)) * r.inv_tau;
  *prob = exp64(d, a.shift, &scaled) * __longlong_as_double((int64_t)(a.shift + 1023) << 52) / double(z);
  return key;
}

// A finished row: its token; with drafts, the last row to finish counts the
// drafts that the tokens agree with.
__device__ void finish_row(const SampleArgs& a, const Ws& w, int row, int token, float prob,
                           uint32_t* flag) {
  if (threadIdx.x == 0) {
    a.tokens[row] = token;
    if (a.prob) a.prob[row] = prob;
  }
  if (!a.n_out) return;
  if (!arrive_last(&w.ctl[0].drawn, a.T, flag)) return;
  if (threadIdx.x == 0) {
    int kept = 0;
    while (kept < a.T - 1 && a.draft[kept] == a.tokens[kept]) ++kept;
    *a.n_out = kept + 1;
  }
}

template <int FMT>
__global__ __launch_bounds__(kThreads) void sample_pick_kernel(const SampleArgs a) {
  __shared__ PickLds s;
  Ws w;
  ws_layout(a.T, static_cast<uint8_t*>(a.ws), &w);
  const int row = blockIdx.y;
  const Row r = read_row(a, w, row, s.red);
  if (r.greedy) {
    if (blockIdx.x == 0)
      finish_row(a, w, row, r.top_key ? index_of(r.top_key) : -1, r.top_key ? 1.0f : 0.0f, &s.flag);
    return;
  }
  RowCtl& ctl = w.ctl[row];
  const int lo0 = ctl.lo[0], hi0 = ctl.hi[0], lo1 = ctl.lo[1], hi1 = ctl.hi[1], lo2 = ctl.lo[2],
            hi2 = ctl.hi[2];
  auto wanted = [&](float x) {
    if (!usable(x)) return false;
    const int b = bin_of(r, x);
    if (!((b >= lo0 && b <= hi0) || (b >= lo1 && b <= hi1) || (b >= lo2 && b <= hi2))) return false;
    return weight_of(r, x, a.shift) != 0;
  };
  uint64_t* list = w.list + int64_t(row) * kListCap;
  const RowView<FMT> v(a.logits, a.stride, row, a.V);
  const int per = (v.vecs + a.parts - 1) / a.parts;
  const int begin = int(blockIdx.x) * per, end = min(v.vecs, begin + per);
  constexpr int kVecs = kTile / kVec<FMT>;
  for (int i0 = begin; i0 < end; i0 += kVecs) {
    __syncthreads();
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    for (int i = i0 + threadIdx.x; i < min(end, i0 + kVecs); i += kThreads) {
      float x[kVec<FMT>];
      v.load(i, x);
#pragma unroll
      for (int j = 0; j < kVec<FMT>; ++j)
        if (wanted(x[j])) s.list[atomicAdd(&s.n, 1u)] = key_of(x[j], i * kVec<FMT> - v.lead + j);
    }
    __syncthreads();
    const uint32_t n = s.n;
    if (n == 0) continue;
    if (threadIdx.x == 0)
      s.flag = __hip_atomic_fetch_add(&ctl.listed, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const uint32_t at = s.flag;
    for (uint32_t k = threadIdx.x; k < n; k += kThreads)
      if (at + k < uint32_t(kListCap)) list[at + k] = s.list[k];
  }
  if (!arrive_last(&ctl.pick_done, a.parts, &s.last)) return;

  const uint32_t n = __hip_atomic_load(&ctl.listed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  double prob;
  uint64_t key;
  if (n <= uint32_t(kLdsList)) {
    for (uint32_t k = threadIdx.x; k < n; k += kThreads) s.list[k] = list[k];
    __syncthreads();
    key = draw_token<FMT>(a, r, w, row, s, &prob, [&](auto&& f) {
      for (uint32_t k = threadIdx.x; k < n; k += kThreads) f(s.list[k]);
    });
  } else if (n <= uint32_t(kListCap)) {
    key = draw_token<FMT>(a, r, w, row, s, &prob, [&](auto&& f) {
      for (uint32_t k = threadIdx.x; k < n; k += kThreads) f(list[k]);
    });
  } else {
    // more candidates than the list holds (long runs of equal logits): the row itself
    key = draw_token<FMT>(a, r, w, row, s, &prob, [&](auto&& f) {
      for (int i = threadIdx.x; i < v.vecs; i += kThreads) {
        float x[kVec<FMT>];
        v.load(i, x);
#pragma unroll
        for (int j = 0; j < kVec<FMT>; ++j)
          if (wanted(x[j])) f(key_of(x[j], i * kVec<FMT> - v.lead + j));
      }
    });
  }
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
  // one tile per workgroup for few rows, about 4 workgroups per CU for many
  const int tiles = (a.V + kTile - 1) / kTile;
  a.parts = max(1, min(min(tiles, kMaxParts), max(1, 1024 / a.T)));
  // a row's weights sum to less than 2^62 and convert exactly from a double
  int bits = 0;
  while ((int64_t(1) << bits) < a.V) ++bits;
  a.shift = min(52, 61 - bits);
  return a.fmt == MOE_W_F32 ? launch<MOE_W_F32>(a, st) : launch<MOE_W_BF16>(a, st);
}

}  // namespace moe
