// Norm and rotation of the new tokens' query and key heads; keys and values
// into their positions' places in the paged cache.
//
// Per head row a of D columns (queries and keys; values are copied):
//   a = a * (1 / sqrt(mean(a^2) + eps)) * weight          (fp32)
//   (a1, a2) -> (a1 c - a2 s, a2 c + a1 s) for the R / 2 pairs
// then one rounding, to bf16 or (keys and values of an 8-bit cache) to e4m3
// with the row's scale max(amax, 448 * 2^-126) / 448.
//
// Angles: position * freq in 64 bits, less its whole turns, so that a far
// position loses nothing; the rest of a turn goes to fp32 sines.
//
// One workgroup per token (for few tokens per part of a token's rows): a lane
// holds 8 columns, D / 8 lanes a row, 256 threads 8 to 32 rows at a time.  The
// token's cosines and sines are computed once, by one thread per pair, and
// kept in registers for all rows, as a lane's columns are always the same.
// A column's partner is read from LDS, where column c lies at (c % 8) * lanes
// + c / 8: neighbouring lanes then read neighbouring words whatever R is.

#include <hip/hip_runtime.h>

#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleFloor = 448.0f * 0x1p-126f;   // keeps every scale a normal number

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
// 16 bytes at any element's address
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

__device__ __forceinline__ void load8(const void* p, int fmt, int64_t i, float* v) {
  if (fmt == MOE_W_F32) {
    const f32x4_any* q = reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + i);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(a[j] << 16);
      v[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ u32x4 pack8(const float* v) {
  u32x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x2 p = {v[2 * j], v[2 * j + 1]};
    r[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2_t));
  }
  return r;
}

template <int G>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  if constexpr (G >= 16) v = fmaxf(v, dpp_f32<0x140>(v));
  if constexpr (G >= 32) v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return v;
}

// The number of q_off[1 .. B] that are <= t: token t's sequence.  A wave
// probes 64 entries at a time.
__device__ __forceinline__ int sequence_of(const int32_t* q_off, int B, int t) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, len = B;
  while (len > 0) {
    const int step = (len + kWave - 1) / kWave;
    const int e = (lane + 1) * step;
    const bool before = e <= len && q_off[lo + e] <= t;
    const int c = __popcll(__ballot(before));
    lo += c * step;
    len = min(step - 1, len - c * step);
  }
  return lo;
}

template <int D>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, ROWS = kThreads / LPR;
  __shared__ f32x2 turn[D / 2];
  __shared__ float part[kThreads * 8];
  const int t = blockIdx.x;
  const int sub = threadIdx.x % LPR, row0 = blockIdx.y * ROWS + threadIdx.x / LPR;
  const int step = gridDim.y * ROWS;
  const int rows = a.Hq + 2 * a.kv.Hkv;
  const int64_t base = int64_t(t) * a.stride + sub * 8;

  float next[8];
  if (row0 < rows) load8(a.qkv, a.fmt, base + int64_t(row0) * D, next);

  const int b = __builtin_amdgcn_readfirstlane(sequence_of(a.kv.q_off, a.kv.B, t));
  if (b >= a.kv.B) return;
  const int first = a.kv.q_off[b], end = a.kv.q_off[b + 1];
  if (t < first || t >= end) return;
  // (64 bits: the three numbers are the caller's)
  const int64_t pos = int64_t(a.kv.kv_len[b]) - end + t;
  int64_t place = -1;                    // the position's index among all pages' slots
  int page = -1;
  if (pos >= 0 && pos < (int64_t(a.kv.max_pages) << a.kv.page_shift)) {
    page = a.kv.page_table[b * a.kv.table_stride + (pos >> a.kv.page_shift)];
    if (page < 0 || page >= a.kv.num_pages) page = -1;
  }
  const int slot = int(pos & ((1 << a.kv.page_shift) - 1));
  if (page >= 0) place = (int64_t(page) << a.kv.page_shift) + slot;

  const int half = a.R / 2;
  if (threadIdx.x < half) {
    const double turns = double(pos) * a.freq[threadIdx.x] * 0.15915494309189533577;   // 1 / (2 pi)
    float s, c;
    sincospif(2.0f * float(turns - rint(turns)), &s, &c);
    turn[threadIdx.x] = f32x2{c * a.rot_scale, s * a.rot_scale};
  }
  __syncthreads();
  // column sub * 8 + j becomes v * co + partner * si
  float co[8], si[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = sub * 8 + j;
    co[j] = 1.0f, si[j] = 0.0f;
    if (c < a.R) {
      const int p = a.interleaved ? c >> 1 : c < half ? c : c - half;
      const bool one = a.interleaved ? !(c & 1) : c < half;
      co[j] = turn[p][0];
      si[j] = one ? -turn[p][1] : turn[p][1];
    }
  }
  float* mine = part + threadIdx.x / LPR * D;

  for (int r = row0; r < rows; r += step) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = next[j];
    if (r + step < rows) load8(a.qkv, a.fmt, base + int64_t(r + step) * D, next);
    const bool key = r >= a.Hq, value = r >= a.Hq + a.kv.Hkv;
    if (!value) {
      const void* weight = key ? a.k_weight : a.q_weight;
      if (weight) {
        float w[8], ss = 0.0f;
        load8(weight, a.weight_fmt, sub * 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
        ss = group_sum<LPR>(ss);
        const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * inv * w[j];
      }
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float x = v[j], y = v[j + 1];
          v[j] = x * co[j] + y * si[j];
          v[j + 1] = y * co[j + 1] + x * si[j + 1];
        }
      } else if (a.R) {
        // (a row's lanes are of one wave, whose LDS accesses stay in order)
#pragma unroll
        for (int j = 0; j < 8; ++j) mine[j * LPR + sub] = v[j];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = sub * 8 + j, o = c < half ? c + half : c - half;
          if (c < a.R) v[j] = v[j] * co[j] + mine[(o & 7) * LPR + (o >> 3)] * si[j];
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
    }
    if (!key) {
      *reinterpret_cast<u32x4_any*>(a.q + int64_t(t) * a.q_stride + r * D + sub * 8) = pack8(v);
      continue;
    }
    if (place < 0) continue;
    const int h = r - a.Hq - (value ? a.kv.Hkv : 0);
    const int64_t at = page * a.kv.page_stride + slot * a.kv.slot_stride + h * a.kv.head_stride + sub * 8;
    uint8_t* to = value ? a.kv.v : a.kv.k;
    if (!a.kv.f8) {
      *reinterpret_cast<u32x4*>(to + at * 2) = pack8(v);
      continue;
    }
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
    m = group_max<LPR>(m);
    const float s = fmaxf(m, kScaleFloor) / kE4m3Max;
    u32x2 q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] / s, v[4 * i + 1] / s, 0, false);
      q[i] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] / s, v[4 * i + 3] / s, p, true));
    }
    *reinterpret_cast<u32x2*>(to + at) = q;
    if (sub == 0) (value ? a.kv.v_scale : a.kv.k_scale)[place * a.kv.Hkv + h] = s;
  }
}

template <int D>
hipError_t launch(const RopeArgs& a, hipStream_t st) {
  constexpr int ROWS = kThreads / (D / 8);
  const int parts = (a.Hq + 2 * a.kv.Hkv + ROWS - 1) / ROWS;
  const dim3 grid(a.T, a.T < 1024 ? parts : 1);
  rope_kernel<D><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st) {
  if (a.kv.D == 64) return launch<64>(a, st);
  if (a.kv.D == 128) return launch<128>(a, st);
  return launch<256>(a, st);
}

}  // namespace moe
