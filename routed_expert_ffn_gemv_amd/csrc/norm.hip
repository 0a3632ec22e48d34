// Residual addition and root-mean-square norm between two layers, with an
// 8-bit output beside (or in place of) the bf16 one.
//
// Per row, with v = the new residual as it is stored:
//   inv  = 1 / sqrt(mean(v^2) + eps)
//   n    = v * inv * weight                       (fp32, in this order)
//   x    = bf16(n)
//   s_b  = max(amax |n| over the 128 columns of block b, 448 * 2^-126) / 448
//   x8   = e4m3(n / s_b)
// The mean square is summed in 64 bits and rounded once: every value of n is
// then the same whatever the split of the row over lanes, so that a value
// next to a border between two 8-bit codes falls on the same side for every
// shape of launch (64-bit fma runs at the fp32 rate here, two instructions
// per element, far below the memory time).
//
// One pass: a row stays in registers between the sums and the outputs.  Each
// lane holds chunks of 8 consecutive columns, so the 128 columns that share
// a scale are 16 neighbouring lanes of one chunk and their maximum is four
// DPP steps.  HBM-bound for many rows (32,768 x 2048, fp32 y, bf16 residual,
// both outputs: 129 us, 5.7 TB/s; a copy of 1 GiB runs at 5.15), latency-bound
// for few (1 x 2048, bf16 output: 2.8 us in a row of launches, 2.3 by itself).

#include <hip/hip_runtime.h>

#include "kernels.h"

namespace moe {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;

constexpr int kMaxGrid = 1 << 20;
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleFloor = 448.0f * 0x1p-126f;   // keeps every scale a normal number

// Maximum over aligned groups of 16 lanes (one 128-column block).
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  v = fmaxf(v, dpp_f32<0x140>(v));
  return v;
}

// Sum over aligned groups of LANES lanes.
template <int LANES>
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
  for (int m = 1; m < LANES; m <<= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

// Two floats to a pair of bf16 bits, nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

__device__ __forceinline__ float round_bf16(float a) {
  return bf16_to_f32(pack_bf16(a, 0.0f) & 0xFFFFu);
}

// 16 and 8 bytes at any element's address: rows of odd length take the same
// accesses, which the hardware splits (32,768 x 2047: 181 us, element by element
// 409; 2048 columns: 129).
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef u32x2 __attribute__((aligned(1))) u32x2_any;

// 8 consecutive elements from p + i, of which n exist (1 .. 8; WHOLE: 8).
template <bool WHOLE>
__device__ __forceinline__ void load8(const void* p, int fmt, int64_t i, int n, float* v) {
  if (WHOLE || n == 8) {
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
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.0f;
    if (j < n)
      v[j] = fmt == MOE_W_F32 ? static_cast<const float*>(p)[i + j]
                              : bf16_to_f32(static_cast<const uint16_t*>(p)[i + j]);
  }
}

template <bool WHOLE>
__device__ __forceinline__ void store8(void* p, int fmt, int64_t i, int n, const float* v) {
  if (WHOLE || n == 8) {
    if (fmt == MOE_W_F32) {
      f32x4_any* q = reinterpret_cast<f32x4_any*>(static_cast<float*>(p) + i);
      q[0] = f32x4{v[0], v[1], v[2], v[3]};
      q[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      *reinterpret_cast<u32x4_any*>(static_cast<uint16_t*>(p) + i) =
          u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                pack_bf16(v[6], v[7])};
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) {
      if (fmt == MOE_W_F32)
        static_cast<float*>(p)[i + j] = v[j];
      else
        static_cast<uint16_t*>(p)[i + j] = uint16_t(pack_bf16(v[j], 0.0f));
    }
}

// LPR lanes per row (a wave's half, a wave or several), ROWS rows per
// workgroup, NCH chunks of 8 columns per lane; WHOLE: H is a multiple of 8.
template <int LPR, int ROWS, int NCH, bool WHOLE>
__global__ __launch_bounds__(LPR* ROWS) void norm_kernel(const NormArgs a) {
  constexpr int WPR = LPR / kWave;      // waves per row
  __shared__ double part[LPR * ROWS / kWave];
  const int wave = threadIdx.x / kWave;
  const int sub = threadIdx.x % LPR;       // lane within the row's
  const int64_t t = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * ROWS + threadIdx.x / LPR;
  const bool live = t < a.T;

  float v[NCH][8];
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int col = (c * LPR + sub) * 8;
    const int n = live ? min(8, a.H - col) : 0;
    if (n > 0) {
      load8<WHOLE>(a.resid, a.resid_fmt, t * a.resid_stride + col, n, v[c]);
      if (a.y) {
        float y[8];
        load8<WHOLE>(a.y, a.y_fmt, t * a.y_stride + col, n, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[c][j] += y[j];
          if (a.resid_fmt == MOE_W_BF16) v[c][j] = round_bf16(v[c][j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fma(double(v[c][j]), double(v[c][j]), ss);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = 0.0f;
    }
  }
  ss = lanes_sum<(LPR < kWave ? LPR : kWave)>(ss);
  if (WPR > 1) {
    if ((threadIdx.x & (kWave - 1)) == 0) part[wave] = ss;
    __syncthreads();
    ss = 0.0;
    const int first = wave / (WPR > 1 ? WPR : 1) * WPR;
#pragma unroll
    for (int w = 0; w < WPR; ++w) ss += part[first + w];
  }
  const float inv = float(1.0 / sqrt(ss / double(a.H) + double(a.eps)));

#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int col = (c * LPR + sub) * 8;
    const int n = live ? min(8, a.H - col) : 0;
    if (n > 0 && a.resid_out) store8<WHOLE>(a.resid_out, a.resid_fmt, t * a.resid_out_stride + col, n, v[c]);
    float o[8];
    if (n > 0) {
      load8<WHOLE>(a.weight, a.weight_fmt, col, n, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = v[c][j] * inv * o[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = 0.0f;
    }
    if (n > 0 && a.x) store8<WHOLE>(a.x, MOE_W_BF16, t * a.x_stride + col, n, o);
    if (a.x8) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(o[j]));
      m = row16_max(m);                               // every lane of the wave takes part
      const float s = fmaxf(m, kScaleFloor) / kE4m3Max;
      if (n > 0) {
        uint32_t q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int p = __builtin_amdgcn_cvt_pk_fp8_f32(o[4 * h] / s, o[4 * h + 1] / s, 0, false);
          p = __builtin_amdgcn_cvt_pk_fp8_f32(o[4 * h + 2] / s, o[4 * h + 3] / s, p, true);
          q[h] = uint32_t(p);
        }
        uint8_t* dst = a.x8 + t * a.H + col;
        if (WHOLE || n == 8) {
          *reinterpret_cast<u32x2_any*>(dst) = u32x2{q[0], q[1]};
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < n) dst[j] = uint8_t(q[j / 4] >> (8 * (j % 4)));
        }
        if (col % 128 == 0) a.x8_scale[t * ((a.H + 127) / 128) + col / 128] = s;
      }
    }
  }
}

template <int LPR, int ROWS, int NCH>
hipError_t launch(const NormArgs& a, hipStream_t st) {
  // two dimensions: one holds less than 2^32 threads
  const int groups = (a.T + ROWS - 1) / ROWS, wide = groups < kMaxGrid ? groups : kMaxGrid;
  const dim3 grid(wide, (groups + wide - 1) / wide);
  if (a.H % 8 == 0)
    norm_kernel<LPR, ROWS, NCH, true><<<grid, LPR * ROWS, 0, st>>>(a);
  else
    norm_kernel<LPR, ROWS, NCH, false><<<grid, LPR * ROWS, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t st) {
  // One chunk of 8 columns per lane as long as a workgroup holds the row: few
  // idle lanes, and all loads of a row under way together.  32,768 x 2048: 129 us
  // with four waves per row, 135 with two, 148 with one (1 x 2048: 3.2, 4.0, 5.9);
  // 8000 x 8192: 133 with 16, 143 with four; 300,000 x 200: 119 with half a wave,
  // 182 with one.
  if (a.H <= 256) return launch<32, 8, 1>(a, st);
  if (a.H <= 512) return launch<64, 4, 1>(a, st);
  if (a.H <= 1024) return launch<128, 2, 1>(a, st);
  if (a.H <= 2048) return launch<256, 1, 1>(a, st);
  if (a.H <= 4096) return launch<512, 1, 1>(a, st);
  if (a.H <= 8192) return launch<1024, 1, 1>(a, st);
  if (a.H <= 16384) return launch<1024, 1, 2>(a, st);
  return launch<1024, 1, 4>(a, st);
}

}  // namespace moe
