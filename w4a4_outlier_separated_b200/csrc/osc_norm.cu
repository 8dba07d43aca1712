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
// row, so that the block maximum meets by shuffles. One CTA per row (or a few short rows): a row's sum
// needs all of it, so what keeps the memory busy is the other rows' CTAs on the SM.
//
// Measured (B200, launches back to back in a graph, inputs cold): 16384 x 4096 with a residual 73.8 us, 6.4 TB/s, 97 % of
// the copy bandwidth. 2048 x 4096: 11.7 us against 9.0 (the fill and the drain of 14 rows per SM). 4001 x 6144
// without a residual: 19.6 us against 11.4; neither the issue (63 % of its slots) nor the memory (58 %) is the bound
// there: 64 registers leave 30 of 64 warps on an SM, whose rows load, reduce and quantize in step and do not hide the
// loads' latency. One row: 1.9 us, the launch. Measured slower: persistent CTAs with the next row's loads in registers
// (4001 x 6144: 23.7 us) or with a ring of rows in shared memory (31 us): fewer rows are worked on at once.
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

// Two fp32 values in one 64-bit register: the packed operations round each half as the scalar ones do.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2f(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4& v, f2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t bf16x2(f2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint4 pack8(const f2 (&f)[4]) {
  return make_uint4(bf16x2(f[0]), bf16x2(f[1]), bf16x2(f[2]), bf16x2(f[3]));
}

// Four E4M3 codes, low byte first.
__device__ __forceinline__ uint32_t e4m3x4(f2 a, f2 b) {
  float x, y, z, w;
  unpack2(a, x, y);
  unpack2(b, z, w);
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r) : "f"(x), "f"(y), "f"(z), "f"(w));
  return r;
}

// What follows the sum of squares of a row, for 8 channels of the calling thread: the normed values (at yp, where
// wanted), their block's exponent, the codes (at q) and (one lane in four) the scale. A warp's lanes hold consecutive
// channels.
__device__ __forceinline__ void norm_quant8(const f2 (&h)[4], f2 inv2, const uint4& gamma, uint16_t* yp, uint8_t* qp,
                                            uint8_t* sp) {
  const int lane = threadIdx.x & 31;
  f2 g[4], y[4];
  unpack8(gamma, g);
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = mul2f(mul2f(h[i], inv2), g[i]);
    float lo, hi;
    unpack2(y[i], lo, hi);
    am = fmaxf(am, fmaxf(fabsf(lo), fabsf(hi)));
  }
  if (yp) *reinterpret_cast<uint4*>(yp) = pack8(y);
  am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
  am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
  // the exponent e = floor(log2 amax) - 8, at least -127 (also for a zero or subnormal block), as its byte e + 127
  const int byte = max((int)(__float_as_uint(am) >> 23) - 8, 0);
  const float f = __uint_as_float((uint32_t)(254 - byte) << 23);   // 2^-e: the product is exact
  const f2 ff = pack2(f, f);
  const uint2 q = make_uint2(e4m3x4(mul2f(y[0], ff), mul2f(y[1], ff)), e4m3x4(mul2f(y[2], ff), mul2f(y[3], ff)));
  *reinterpret_cast<uint2*>(qp) = q;
  // one byte of each four lanes; a layout word's four bytes meet in one write of the warp
  if ((lane & 3) == 0) *sp = (uint8_t)byte;
}

// The first scale word of a row (the next ones 512 bytes apart): atoms of 128 rows x 4 slots.
__device__ __forceinline__ uint8_t* scale_row(const AddNormParams& p, int row) {
  return p.S + (size_t)(row >> 7) * (p.K >> 7) * 512 + (size_t)((row & 31) * 16 + ((row >> 5) & 3) * 4);
}

// 1 / sqrt(ss / K + eps), within 2^-22 of it (the root's own error); an all-zero row with eps = 0 stays zero, and a NaN
// in the row makes all of it NaN.
__device__ __forceinline__ f2 inverse2(const AddNormParams& p, float ss) {
  const float ms = ss * __frcp_rn((float)p.K) + p.eps;
  const float inv = ms == 0.f ? 0.f : rsqrtf(ms);
  return pack2(inv, inv);
}

}  // namespace

// C: steps of 8 channels per thread; RES: there is a residual; WHOLE: every thread has all its steps. A CTA holds
// p.rows_per_cta rows of `tpr` threads each. Rows M .. (next multiple of 128) only write zero scales.
template <int C, bool RES, bool WHOLE>
__global__ void __launch_bounds__(1024) add_rmsnorm_fp8_kernel(AddNormParams p, int tpr) {
  __shared__ float part[32];
  const int sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * p.rows_per_cta + sub;
  const int nchunk = p.K >> 3;
  const bool live = row < p.M;
  const size_t first = (size_t)row * p.K + t * 8;        // the thread's first channel; its steps are tpr * 8 apart
  uint8_t* srow = scale_row(p, row) + (size_t)(t >> 4) * 512 + ((t >> 2) & 3);

  grid_dep_wait();
  grid_dep_launch();
  f2 h[C][4];
  f2 ss2 = pack2(0.f, 0.f);
  if (live) {
    uint4 a[C], b[C];
    const uint16_t *x = p.X + first, *r = p.res + first;
#pragma unroll
    for (int c = 0; c < C; ++c, x += tpr * 8, r += tpr * 8) {
      if (WHOLE || c * tpr + t < nchunk) {
        a[c] = load_stream(x);
        if (RES) b[c] = load_stream(r);
      }
    }
    uint16_t* hp = p.H + first;
#pragma unroll
    for (int c = 0; c < C; ++c, hp += tpr * 8) {
      if (WHOLE || c * tpr + t < nchunk) {
        unpack8(a[c], h[c]);
        if (RES) {
          f2 v[4];
          unpack8(b[c], v);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[c][i] = add2(h[c][i], v[i]);
        }
        if (p.H) *reinterpret_cast<uint4*>(hp) = pack8(h[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss2 = fma2(h[c][i], h[c][i], ss2);
      }
    }
  }
  float ss, odd;
  unpack2(ss2, ss, odd);
  ss += odd;
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
      for (int s = t; s < (p.K >> 7); s += tpr) *reinterpret_cast<uint32_t*>(scale_row(p, row) + (size_t)s * 512) = 0u;
    return;
  }
  const f2 inv2 = inverse2(p, ss);
  const uint16_t* gp = p.gamma + t * 8;
  uint8_t* q = p.Q + first;
  uint16_t* y = p.Y ? p.Y + first : nullptr;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (!WHOLE && c * tpr + t >= nchunk) break;          // the same for a whole warp
    norm_quant8(h[c], inv2, *reinterpret_cast<const uint4*>(gp), y, q, srow);
    gp += tpr * 8;
    q += tpr * 8;
    srow += (size_t)(tpr >> 4) * 512;
    if (y) y += tpr * 8;
  }
}

template <int C, bool RES, bool WHOLE>
static cudaError_t launch_w(AddNormParams p, int tpr, cudaStream_t s) {
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
  return cudaLaunchKernelEx(&cfg, add_rmsnorm_fp8_kernel<C, RES, WHOLE>, p, tpr);
}

template <int C>
static cudaError_t launch_c(const AddNormParams& p, int tpr, cudaStream_t s) {
  if (C == 1 || C * tpr * 8 == p.K)                        // one step of K % 256 = 0 channels is always whole
    return p.res ? launch_w<C, true, true>(p, tpr, s) : launch_w<C, false, true>(p, tpr, s);
  if constexpr (C > 1) return p.res ? launch_w<C, true, false>(p, tpr, s) : launch_w<C, false, false>(p, tpr, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_add_rmsnorm_fp8(const AddNormParams& p, int num_sms, cudaStream_t s) {
  // steps per thread: one where rows are few, so that a row has the most threads (one row of 4096: 2.0 against 2.6 us with
  // four steps), four where they fill the SMs (2048 rows: 12 against 13 us, 16384 rows: 74 against 90 us)
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
