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
// position loses nothing; cosine, sine and their product with rot_scale in 64
// bits too, rounded once (with fp32 sines of the rest of a turn, off by up to 2^-23
// radians, the same times: 149 us for the prompt below, 4.2 for one token).
//
// A lane holds 8 columns, D / 8 lanes a row, 256 threads 8 to 32 rows at a
// time, and a thread has its next three rows under way.  For many tokens a
// workgroup takes four, whose sequences, positions and sines its four waves
// find side by side (a chain of loads as long as a token's rows take); for few
// tokens a workgroup takes a part of one's rows.  A token's cosines and sines
// stay in registers for all its rows, as a lane's columns are always the same.
// A column's partner is read from LDS, where column c lies at (c % 8) * lanes +
// c / 8: neighbouring lanes then read neighbouring words whatever R is.
//
// HBM-bound for many tokens (32,768 of 16 + 2 x 2 heads of 256, bf16: 149 us,
// 4.5 TB/s of 5.2 that a copy reaches), latency for few (1: 4.2 us on the GPU).

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

// Eight columns as they lie in memory.
template <int FMT>
struct Raw {
  u32x4 words[FMT == MOE_W_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if (FMT == MOE_W_F32) {
      const f32x4_any* q = reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + i);
      words[0] = __builtin_bit_cast(u32x4, f32x4(q[0]));
      words[FMT == MOE_W_F32] = __builtin_bit_cast(u32x4, f32x4(q[1]));
    } else {
      words[0] = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(p) + i);
    }
  }
  __device__ __forceinline__ void values(float* v) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (FMT == MOE_W_F32) {
        v[j] = __uint_as_float(words[0][j]);
        v[4 + j] = __uint_as_float(words[FMT == MOE_W_F32][j]);
      } else {
        v[2 * j] = __uint_as_float(words[0][j] << 16);
        v[2 * j + 1] = __uint_as_float(words[0][j] & 0xFFFF0000u);
      }
    }
  }
};

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

// Where a token's keys and values go.
struct Place {
  int page;            // -1: nowhere
  int slot;
  bool live;           // of some sequence
};

// TOKENS: 1 (all waves look it up) or one per wave.
template <int D, int TOKENS, int FMT>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, ROWS = kThreads / LPR, AHEAD = TOKENS == 1 ? 1 : 3;
  __shared__ f32x2 turn[TOKENS][D / 2];
  __shared__ Place places[TOKENS];
  __shared__ float part[kThreads * 8];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int t0 = blockIdx.x * TOKENS, tokens = min(TOKENS, a.T - t0);
  const int sub = threadIdx.x % LPR, row0 = blockIdx.y * ROWS + threadIdx.x / LPR;
  const int step = gridDim.y * ROWS;
  const int rows = a.Hq + 2 * a.kv.Hkv;
  const int half = a.R / 2;

  // a thread's next rows, as they are (one workgroup per token: one, for more of them at once)
  Raw<FMT> now[AHEAD], next[AHEAD];
  auto fetch = [&](int tok, int r, Raw<FMT>* to) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (tok < tokens && r + k * step < rows)
        to[k].load(a.qkv, int64_t(t0 + tok) * a.stride + (r + k * step) * D + sub * 8);
  };
  fetch(0, row0, next);

  {
    const int tok = TOKENS == 1 ? 0 : wave, t = t0 + tok;
    const int b = tok < tokens ? __builtin_amdgcn_readfirstlane(sequence_of(a.kv.q_off, a.kv.B, t)) : a.kv.B;
    Place p = {-1, 0, false};
    if (b < a.kv.B) {
      const int first = a.kv.q_off[b], end = a.kv.q_off[b + 1];
      p.live = t >= first && t < end;
      // (64 bits: the three numbers are the caller's)
      const int64_t pos = int64_t(a.kv.kv_len[b]) - end + t;
      if (pos >= 0 && pos < (int64_t(a.kv.max_pages) << a.kv.page_shift)) {
        p.page = a.kv.page_table[b * a.kv.table_stride + (pos >> a.kv.page_shift)];
        if (p.page < 0 || p.page >= a.kv.num_pages) p.page = -1;
      }
      p.slot = int(pos & ((1 << a.kv.page_shift) - 1));
      for (int j = TOKENS == 1 ? int(threadIdx.x) : lane; j < half; j += TOKENS == 1 ? kThreads : kWave) {
        const double turns = double(pos) * a.freq[j] * 0.15915494309189533577;   // 1 / (2 pi)
        double s, c;
        sincospi(2.0 * (turns - rint(turns)), &s, &c);
        turn[tok][j] = f32x2{float(c * a.rot_scale), float(s * a.rot_scale)};
      }
    }
    if (lane == 0) places[tok] = p;
  }
  float weights[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k ? a.k_weight : a.q_weight) load8(k ? a.k_weight : a.q_weight, a.weight_fmt, sub * 8, weights[k]);
  __syncthreads();
  if (row0 >= rows) return;

  // lanes whose columns all stay as they are take no part in the rotation; one
  // that holds column R rotates those before it and keeps the others' values (a
  // product with a cosine of 1 and a sine of 0 would make NaN of an infinity).
  // Only where R is not a multiple of 8: looked at for every row, 32,768 tokens
  // of 20 heads of 256 took 166 us in place of 147.
  const bool turns = sub * 8 < a.R, mixed = a.R % 8 != 0;
  const int turning = a.R - sub * 8;     // the lane's first so many columns
  int partner[8];      // where each column's lies in LDS
  if (turns) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = sub * 8 + j, o = j >= turning ? c : c < half ? c + half : c - half;
      partner[j] = (o & 7) * LPR + (o >> 3);
    }
  }
  float* mine = part + threadIdx.x / LPR * D;

#pragma unroll 1
  for (int tok = 0; tok < tokens; ++tok) {
    const Place place = places[tok];
    // column sub * 8 + j becomes v * co + partner * si
    float co[8], si[8];
    if (turns && place.live) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = sub * 8 + j;
        const bool one = a.interleaved ? !(j & 1) : c < half;
        const f32x2 w = turn[tok][j >= turning ? 0 : a.interleaved ? c >> 1 : one ? c : c - half];
        co[j] = w[0];
        si[j] = one ? -w[1] : w[1];
      }
    }
    const int64_t t = t0 + tok;
#pragma unroll 1
    for (int r0 = row0; r0 < rows; r0 += AHEAD * step) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) now[k] = next[k];
      if (r0 + AHEAD * step < rows)
        fetch(tok, r0 + AHEAD * step, next);
      else
        fetch(tok + 1, row0, next);
      if (!place.live) continue;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int r = r0 + k * step;
        if (r >= rows) break;
        float v[8];
        now[k].values(v);
        const bool key = r >= a.Hq, value = r >= a.Hq + a.kv.Hkv;
        if (!value) {
          if (key ? a.k_weight : a.q_weight) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
            ss = group_sum<LPR>(ss);
            float mean = ss * (1.0f / D) + a.eps;
            // A row whose squares leave fp32's range is multiplied by a power of two
            // first: sums of them then end within 2^120, and begin at 2^-106.
            const bool out = !(mean >= 0x1p-80f && mean <= 0x1.fffffep127f);
            if (__builtin_expect(__ballot(out) != 0, 0)) {
              const float k = !out ? 1.0f : ss > 1.0f ? 0x1p-72f : 0x1p96f;
              ss = 0.0f;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                v[j] *= k;
                ss = fmaf(v[j], v[j], ss);
              }
              mean = group_sum<LPR>(ss) * (1.0f / D) + a.eps * k * k;
            }
            const float inv = rsqrtf(mean);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = v[j] * inv * (key ? weights[1][j] : weights[0][j]);
          }
          if (turns) {
            if (a.interleaved) {
#pragma unroll
              for (int j = 0; j < 8; j += 2) {
                if (mixed && j >= turning) continue;
                const float x = v[j], y = v[j + 1];
                v[j] = x * co[j] + y * si[j];
                v[j + 1] = y * co[j + 1] + x * si[j + 1];
              }
            } else {
              // (a row's lanes are of one wave, whose LDS accesses stay in order)
#pragma unroll
              for (int j = 0; j < 8; ++j) mine[j * LPR + sub] = v[j];
              __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
              __builtin_amdgcn_wave_barrier();
              __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] = v[j] * co[j] + mine[partner[j]] * si[j];
              if (mixed) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (j >= turning) v[j] = mine[j * LPR + sub];
              }
              __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
              __builtin_amdgcn_wave_barrier();
            }
          }
        }
        if (!key) {
          *reinterpret_cast<u32x4_any*>(a.q + t * a.q_stride + r * D + sub * 8) = pack8(v);
          continue;
        }
        if (place.page < 0) continue;
        const int h = r - a.Hq - (value ? a.kv.Hkv : 0);
        const int64_t at = place.page * a.kv.page_stride + place.slot * a.kv.slot_stride +
                         h * a.kv.head_stride + sub * 8;
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
        // (the division itself, not a product with the scale's inverse: one rounding
        // less before the code is chosen)
        u32x2 q;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] / s, v[4 * i + 1] / s, 0, false);
          q[i] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] / s, v[4 * i + 3] / s, p, true));
        }
        *reinterpret_cast<u32x2*>(to + at) = q;
        if (sub == 0)
          (value ? a.kv.v_scale : a.kv.k_scale)[((int64_t(place.page) << a.kv.page_shift) + place.slot) * a.kv.Hkv + h] = s;
      }
    }
  }
}

template <int D, int FMT>
hipError_t launch(const RopeArgs& a, hipStream_t st) {
  constexpr int ROWS = kThreads / (D / 8), TOKENS = kThreads / kWave;
  // Four tokens per workgroup from 8 workgroups per CU on: of 20 heads of 256,
  // 32,768 tokens take 149 us (one each: 188), 16,384 79 (89), 8192 36 (36), 4096 20
  // (21), 2048 16 (13), as half of the CUs get two; of 15 heads of 64 in fp32, 32,768
  // 68 (65), 8192 21 (20), 2196 8.9 (8.0).
  if (a.T >= 8192) {
    rope_kernel<D, TOKENS, FMT><<<(a.T + TOKENS - 1) / TOKENS, kThreads, 0, st>>>(a);
  } else {
    const int parts = (a.Hq + 2 * a.kv.Hkv + ROWS - 1) / ROWS;
    rope_kernel<D, 1, FMT><<<dim3(a.T, a.T < 1024 ? parts : 1), kThreads, 0, st>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st) {
  const bool f32 = a.fmt == MOE_W_F32;
  if (a.kv.D == 64) return f32 ? launch<64, MOE_W_F32>(a, st) : launch<64, MOE_W_BF16>(a, st);
  if (a.kv.D == 128) return f32 ? launch<128, MOE_W_F32>(a, st) : launch<128, MOE_W_BF16>(a, st);
  return f32 ? launch<256, MOE_W_F32>(a, st) : launch<256, MOE_W_BF16>(a, st);
}

}  // namespace moe
