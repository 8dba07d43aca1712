// Residual addition, RMSNorm and MXFP8 quantization of a row in one pass:
//   h = x + res,  y = h * gamma / sqrt(mean(h^2) + eps),
//   e = floor(log2 max|y|) - 8 per 32 channels,  q = e4m3(y * 2^-e).
//
// The row stays in registers between the sum of squares and the quantization, so each input is
// read once and each output written once: 2 (x) + 2 (res) bytes in, 2 (h) + 1 (q) + 1/32 (scale)
// bytes out per element, and 2 more for the normed row on request. HBM bounds it; there is no
// product.
//
// Rounding: h, the squares, their sum and y are fp32. h enters the norm unrounded and y enters
// both of its outputs unrounded, so H (bf16), Y (bf16) and the E4M3 codes are each rounded once.
//
// Work split: 8 consecutive channels per thread and step (one 16-byte load of each input, one
// 8-byte store of codes), four neighbouring threads to a 32-channel block, whole warps to a
// row, so that the block maximum and the four scale bytes of a layout word meet by shuffles.
#include "osc_device.cuh"
#include "osc_internal.h"

namespace osc {

namespace {

__device__ __forceinline__ uint4 load_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

}  // namespace

// C: steps of 8 channels per thread. A CTA holds p.rows_per_cta rows of `tpr` threads each.
// Rows M .. (next multiple of 128) only write zero scales.
template <int C>
__global__ void __launch_bounds__(1024) add_rmsnorm_fp8_kernel(AddNormParams p, int tpr) {
  __shared__ float part[32];
  const int sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * p.rows_per_cta + sub;
  const int nchunk = p.K >> 3, nslot4 = p.K >> 7;
  const bool live = row < p.M;
  const size_t base = (size_t)row * p.K;
  // the scale word of four blocks: 512-byte atoms of 128 rows x 4 slots
  uint8_t* const srow = p.S + (size_t)(row >> 7) * nslot4 * 512 + (size_t)((row & 31) * 16 + ((row >> 5) & 3) * 4);

  grid_dep_wait();
  grid_dep_launch();
  float h[C][8];
  float ss = 0.f;
  if (live) {
    uint4 a[C], b[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = c * tpr + t;
      if (ch < nchunk) {
        a[c] = load_stream(p.X + base + (size_t)ch * 8);
        if (p.res) b[c] = load_stream(p.res + base + (size_t)ch * 8);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int ch = c * tpr + t;
      if (ch < nchunk) {
        unpack8(a[c], h[c]);
        if (p.res) {
          float r[8];
          unpack8(b[c], r);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[c][i] += r[i];
        }
        if (p.H) *reinterpret_cast<uint4*>(p.H + base + (size_t)ch * 8) = pack8(h[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[c][i], h[c][i], ss);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const int wpr = tpr >> 5;
  if (wpr > 1) {
    if (lane == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < wpr; ++w) ss += part[sub * wpr + w];   // every thread in the same order
  }
  if (!live) {
    if (row < ((p.M + 127) & ~127))
      for (int s = t; s < nslot4; s += tpr) *reinterpret_cast<uint32_t*>(srow + (size_t)s * 512) = 0u;
    return;
  }
  const float ms = ss / (float)p.K + p.eps;
  const float inv = ms > 0.f ? 1.0f / sqrtf(ms) : 0.f;   // an all-zero row with eps = 0 stays zero
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int ch = c * tpr + t;
    if (ch >= nchunk) break;                             // the same for a whole warp
    float g[8], y[8];
    unpack8(*reinterpret_cast<const uint4*>(p.gamma + (size_t)ch * 8), g);
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = (h[c][i] * inv) * g[i];
      am = fmaxf(am, fabsf(y[i]));
    }
    if (p.Y) *reinterpret_cast<uint4*>(p.Y + base + (size_t)ch * 8) = pack8(y);
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
    // floor(log2 amax) - 8 from the exponent field, at least -127 (also for a zero or subnormal block)
    const int e = max((int)(__float_as_uint(am) >> 23) - 127 - 8, -127);
    const float f = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e: the product is exact
    const uint2 q = make_uint2(e4m3x4(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                               e4m3x4(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
    *reinterpret_cast<uint2*>(p.Q + base + (size_t)ch * 8) = q;
    uint32_t s = (uint32_t)(e + 127) << (((lane >> 2) & 3) * 8);
    s |= __shfl_xor_sync(0xffffffffu, s, 4);
    s |= __shfl_xor_sync(0xffffffffu, s, 8);
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(srow + (size_t)(ch >> 4) * 512) = s;
  }
}

template <int C>
static cudaError_t launch_c(AddNormParams p, int tpr, cudaStream_t s) {
  p.rows_per_cta = std::max(1, 128 / tpr);
  cudaLaunchConfig_t cfg = {};
  const int mpad = (p.M + 127) / 128 * 128;
  cfg.gridDim = dim3((mpad + p.rows_per_cta - 1) / p.rows_per_cta, 1, 1);
  cfg.blockDim = dim3(tpr * p.rows_per_cta, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, add_rmsnorm_fp8_kernel<C>, p, tpr);
}

cudaError_t launch_add_rmsnorm_fp8(const AddNormParams& p, int num_sms, cudaStream_t s) {
  const int nchunk = p.K / 8;
  auto tpr = [&](int c) { return ((nchunk + c - 1) / c + 31) / 32 * 32; };
  int c = p.M >= 4 * num_sms ? 4 : 1;
  while (tpr(c) > 1024) c *= 2;
  switch (c) {
    case 1: return launch_c<1>(p, tpr(1), s);
    case 2: return launch_c<2>(p, tpr(2), s);
    case 4: return launch_c<4>(p, tpr(4), s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace osc
