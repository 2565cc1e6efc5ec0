// Residual addition + root-mean-square norm + quantize, in one pass.
//
//   r = bf16(x + residual)                       (r = x without a residual)
//   y = r * rsqrt(mean(r^2) + eps) * weight      fp32, not rounded to bf16
//   out = y in NVFP4 (static global scale, as nvfp4_quantize), or
//   out = E4M3(y * (1 / s)), s = amax / 448 over the row or over 128 elements
//
// HBM-bound: 6 bytes an element for x, residual and r, 0.56 or 1 for out.  A
// row is read once and stays in registers: a thread owns blocks of 16
// elements (its NVFP4 scale block), the row's sum of squares goes through
// shuffles and, for rows wider than a warp, shared memory.
//
// Measured: [8192, 7168] to E4M3 with a scale per 128: 72.5 us for 413 MB (5.7
// TB/s, 84 % of the copy rate); [777, 5120] to NVFP4: 6.0 us; one row of 5120:
// 2.6 us.  A persistent kernel with the next row on its way took 92 us, five
// CTAs an SM 81; 32-byte accesses would give 71 on rows that lie on 32 bytes.
#include "common.cuh"
#include "internal.h"

namespace nvfp4 {
namespace {

enum NormOut { NORM_NVFP4 = 0, NORM_FP8 = 1 };

// Four floats -> four E4M3 bytes, round to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n"
      ".reg .b16 lo, hi;\n"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      "mov.b32 %0, {lo, hi};\n"
      "}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Sum (or maximum) over the threads of one row: the warp for rows of one
// warp, the CTA otherwise (a power of two of warps is not needed).
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int warps, float *s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  // every warp reduces the warps' values for itself (32 at most), in the same order
  const int lane = threadIdx.x & 31;
  v = lane < warps ? s[lane] : 0.0f;   // (the maxima are of magnitudes)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  return v;
}

struct NormArgs {
  const uint16_t *x, *residual, *weight;
  const float *eps, *gs;
  uint16_t *r_out;
  uint8_t *out, *sf;      // codes or E4M3 values; NVFP4 block scales
  float *scale;           // E4M3: fp32 scales
  int64_t m, k;
  int tpr;                // threads of a row (a multiple of 32)
  int group;              // E4M3: 0 = one scale a row, else 128
  bool swizzled;
};

// 1 / sqrt(sum / k + eps) as the sum of two floats: the roundings of the mean,
// of the root and of the first product with it then stay below y's own one,
// and a value moves to another code only within an fp32 ulp of a boundary.
__device__ __forceinline__ float2 inverse_root(float sum, float k, float eps) {
  const float q = __fdiv_rn(sum, k), s = q + eps, bb = s - q;
  const float s_lo = (q - (s - bb)) + (eps - bb) + __fdividef(fmaf(-q, k, sum), k);
  const float r = __frsqrt_rn(s), h = s * r;
  const float e = fmaf(-h, r, 1.0f) - (fmaf(s, r, -h) + s_lo * r) * r;
  const float r_lo = 0.5f * r * e;
  return make_float2(r, fabsf(r_lo) < r ? r_lo : 0.0f);       // (not of infinities)
}

// y of one block: r (bf16 pairs) * rstd * weight, rounded once to fp32.
__device__ __forceinline__ void norm16(const uint32_t (&r)[8], const uint16_t *weight, float2 rstd, float (&y)[16]) {
  const uint4 *q = reinterpret_cast<const uint4 *>(weight);
  const uint4 v0 = __ldg(q), v1 = __ldg(q + 1);
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float f = i & 1 ? bf16_hi(r[i / 2]) : bf16_lo(r[i / 2]), g = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    const float t = f * rstd.x, e = fmaf(f, rstd.y, fmaf(f, rstd.x, -t));
    y[i] = fmaf(t, g, e * g);
  }
}

// Largest magnitude of a block, NaN where one is: it makes the block's scale
// E4M3's NaN (fmaxf would drop it, and make zeros of a row that holds one).
__device__ __forceinline__ float amax16_nan(const float (&y)[16]) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(fabsf(y[i])));
  return amax;
}

__device__ __forceinline__ float amax16(const float (&y)[16]) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(y[i]));
  return amax;
}

// Block j of the row belongs to thread j % tpr; CH blocks a thread, held as
// the bf16 pairs of r.
template <NormOut OUT, int CH, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) rms_norm_kernel(const NormArgs a) {
  __shared__ float s_sum[32], s_max[32];
  pdl_trigger();
  pdl_wait();
  const int cols = (int)(a.k >> 4), warps = a.tpr >> 5;
  const int t = warps == 1 ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const int64_t row = warps == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const int cp4 = (cols + 3) >> 2;
  if (row >= a.m) {        // padding rows of the swizzled scale layout (a whole warp or CTA)
    if (OUT == NORM_NVFP4 && a.swizzled && row < ((a.m + 127) & ~(int64_t)127))
      for (int j = t; j < cp4 * 4; j += a.tpr) a.sf[sf_swizzled_offset(row, j, cp4)] = 0;
    return;
  }
  uint32_t r[CH][8] = {};
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int j = t + c * a.tpr;
    if (j < cols) {
      const int64_t at = row * a.k + (int64_t)j * 16;
      const uint4 *q = reinterpret_cast<const uint4 *>(a.x + at);
      const uint4 v0 = __ldcs(q), v1 = __ldcs(q + 1);
      r[c][0] = v0.x, r[c][1] = v0.y, r[c][2] = v0.z, r[c][3] = v0.w;
      r[c][4] = v1.x, r[c][5] = v1.y, r[c][6] = v1.z, r[c][7] = v1.w;
      if (a.residual) {
        const uint4 *p = reinterpret_cast<const uint4 *>(a.residual + at);
        const uint4 u0 = __ldcs(p), u1 = __ldcs(p + 1);
        const uint32_t u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __nv_bfloat162 b =
              __floats2bfloat162_rn(bf16_lo(r[c][i]) + bf16_lo(u[i]), bf16_hi(r[c][i]) + bf16_hi(u[i]));
          r[c][i] = *reinterpret_cast<const uint32_t *>(&b);
        }
      }
      if (a.r_out) {
        uint4 *o = reinterpret_cast<uint4 *>(a.r_out + at);
        __stcs(o, make_uint4(r[c][0], r[c][1], r[c][2], r[c][3]));          // (read again only after the next products)
        __stcs(o + 1, make_uint4(r[c][4], r[c][5], r[c][6], r[c][7]));
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum = fmaf(bf16_lo(r[c][i]), bf16_lo(r[c][i]), sum);
      sum = fmaf(bf16_hi(r[c][i]), bf16_hi(r[c][i]), sum);
    }
  }
  sum = row_reduce<false>(sum, warps, s_sum);
  const float2 rstd = inverse_root(sum, (float)a.k, __ldg(a.eps));
  if (OUT == NORM_NVFP4) {
    const float gs = __ldg(a.gs);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int j = t + c * a.tpr;
      uint32_t sf = 0;
      if (j < cols) {
        float y[16];
        norm16(r[c], a.weight + (int64_t)j * 16, rstd, y);
        uint32_t lo, hi;
        sf = quantize_block16(y, amax16_nan(y), gs, lo, hi);
        *reinterpret_cast<uint2 *>(a.out + row * (a.k >> 1) + (int64_t)j * 8) = make_uint2(lo, hi);
      }
      if (a.swizzled) {
        if (j < cp4 * 4) a.sf[sf_swizzled_offset(row, j, cp4)] = (uint8_t)sf;
      } else if (j < cols) {
        a.sf[row * cols + j] = (uint8_t)sf;
      }
    }
    return;
  }
  float amax_row = 0.0f;
  if (a.group == 0) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int j = t + c * a.tpr;
      if (j >= cols) continue;
      float y[16];
      norm16(r[c], a.weight + (int64_t)j * 16, rstd, y);
      amax_row = fmaxf(amax_row, amax16(y));
    }
    amax_row = row_reduce<true>(amax_row, warps, s_max);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int j = t + c * a.tpr;
    float y[16] = {};
    if (j < cols) norm16(r[c], a.weight + (int64_t)j * 16, rstd, y);
    float amax = amax_row;
    if (a.group) {   // 128 elements: 8 neighbouring lanes (tpr % 8 == 0, whole groups in the row)
      amax = amax16(y);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    if (j >= cols) continue;
    // (not below the smallest normal number: 1 / s would be infinite, and a zero times it NaN)
    const float s = amax > 0.0f ? fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f) : 1.0f, inv = __fdiv_rn(1.0f, s);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = e4m3_pack4(y[4 * i] * inv, y[4 * i + 1] * inv, y[4 * i + 2] * inv, y[4 * i + 3] * inv);
    *reinterpret_cast<uint4 *>(a.out + row * a.k + (int64_t)j * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    if (a.group) {
      if ((j & 7) == 0) a.scale[row * (a.k >> 7) + (j >> 3)] = s;
    } else if (j == 0) {
      a.scale[row] = s;
    }
  }
}

template <NormOut OUT>
cudaError_t launch_norm(NormArgs a, int64_t rows, cudaStream_t st) {
  // Rows of up to 8192 elements: two blocks a thread, so that four small CTAs
  // an SM load, reduce and store out of step ([8192, 7168] to E4M3: 72 us; one
  // block a thread 77 us, four 84 us) -- unless the rows are too few to fill
  // the SMs and a row's own latency counts ([1, 5120]: 2.6 us with one block a
  // thread, 3.3 us with two).  Wider rows: up to 512 threads.
  const int cols = (int)(a.k / 16);
  const int ch = cols <= 512 ? (cols <= 32 || rows <= num_sms() ? 1 : 2) : cols <= 1024 ? 2 : cols <= 2048 ? 4 : 8;
  a.tpr = ((cols + ch - 1) / ch + 31) / 32 * 32;
  const int threads = a.tpr == 32 ? 256 : a.tpr;     // narrow rows: a warp each, eight to a CTA
  const int64_t grid = a.tpr == 32 ? (rows + 7) / 8 : rows;
  auto kernel = ch == 1     ? rms_norm_kernel<OUT, 1, 512, 2>
                : ch == 2   ? (threads <= 256 ? rms_norm_kernel<OUT, 2, 256, 4> : rms_norm_kernel<OUT, 2, 512, 1>)
                : ch == 4   ? rms_norm_kernel<OUT, 4, 512, 1>
                            : rms_norm_kernel<OUT, 8, 512, 1>;
  return launch_pdl(kernel, dim3((unsigned)grid), dim3(threads), 0, st, a);
}

}  // namespace

cudaError_t launch_rms_norm_nvfp4(const uint16_t *x, const uint16_t *residual, const uint16_t *weight,
                                  const float *eps, const float *gs, uint16_t *r_out, uint8_t *out_fp4,
                                  uint8_t *out_sf, bool swizzled, int64_t m, int64_t k, cudaStream_t st) {
  NormArgs a{};
  a.x = x, a.residual = residual, a.weight = weight, a.eps = eps, a.gs = gs, a.r_out = r_out;
  a.out = out_fp4, a.sf = out_sf, a.m = m, a.k = k, a.swizzled = swizzled;
  return launch_norm<NORM_NVFP4>(a, swizzled ? (m + 127) / 128 * 128 : m, st);
}

cudaError_t launch_rms_norm_fp8(const uint16_t *x, const uint16_t *residual, const uint16_t *weight,
                                const float *eps, uint16_t *r_out, uint8_t *out, float *scale, int group, int64_t m,
                                int64_t k, cudaStream_t st) {
  NormArgs a{};
  a.x = x, a.residual = residual, a.weight = weight, a.eps = eps, a.r_out = r_out;
  a.out = out, a.scale = scale, a.m = m, a.k = k, a.group = group;
  return launch_norm<NORM_FP8>(a, m, st);
}

}  // namespace nvfp4
