// Few bf16 token rows times a prepared 4-bit weight (decoding with unquantized activations):
//   Y[m][n] = sum_{k not in the table} x[m][k] q[n][k] 2^e[n][k/V]  +  sum_i x[m][ch_i] W_L[n][i].
// The weight is what has to be read (N K / 2 bytes of codes, N K / V of scales, 2 N K_L of W_L);
// everything else is small, so the kernel is built around keeping those bytes in flight.
//
// Unit: 32 weight rows, the four octets {q*32 + j*8 .. +7} (q = 0..3) of a 128-row block, because
// the scale layout keeps exactly those rows' words together: 128 contiguous bytes per 512-byte
// atom. A CTA (or a cluster of S CTAs that split K) owns a unit. Its warps take chunks of 128
// channels in turn; a warp copies a chunk's codes, scales and token rows into its own stages of
// shared memory with cp.async and computes without waiting for any other warp. The warps' sums
// meet once, in shared memory (across the cluster in distributed shared memory), in a fixed order.
//
// Arithmetic: mma.m16n8k16 on f16 operands with fp32 accumulators, the weight rows as the
// 16-row side and the tokens as the 8-wide side. E2M1 codes become f16 exactly (one conversion
// per two codes). The bf16 tokens become f16 after scaling each token's 128 channels by the power
// of two that puts their largest magnitude in [2^14, 2^15): a value keeps all its bits down to
// 2^-31 of that maximum, and below that errs by at most 2^-39 of it, far under the fp32 sum's own
// rounding. A scale block's products are summed in fp32, then multiplied by the weight's and the
// token's powers of two (exact) and added in fp32. Y is rounded once.
// The protected channels are zeroed in the staged tokens; their products run as bf16 mma of the
// gathered tokens with W_L into the same sums.
#include <cuda_fp16.h>

#include "osc_device.cuh"
#include "osc_internal.h"

namespace osc {

namespace {

constexpr int GV_WARPS = 8;
constexpr int GV_ROWS = 32;                       // weight rows of a unit
constexpr int GV_CHUNK = 128;                     // channels of a chunk
constexpr int GV_WBYTES = GV_ROWS * GV_CHUNK / 2; // codes of a stage

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
  const int n = full ? 16 : 0;                    // 0: the 16 bytes are filled with zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts64(uint32_t a, uint2 v) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" :: "r"(a), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ void sts32f(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" :: "r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ float lds32f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds32f_cluster(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

// Eight E2M1 codes (low nibble first) as four f16 pairs, exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^(byte - 127) (0 stands for 2^-127, a subnormal).
__device__ __forceinline__ float e8m0(uint32_t byte) { return __uint_as_float(max(byte << 23, 0x00400000u)); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ uint32_t redux_max(uint32_t v) {
  uint32_t r;
  asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(r) : "r"(v));
  return r;
}

// Shared memory of a CTA, in bytes from its start.
struct GvSmem {
  int stage, warp, chan, ids, flag, total;
};
__host__ __device__ inline GvSmem gv_smem(int V, int mt, int stages, int n_list, int rows, int E) {
  GvSmem m;
  m.stage = GV_WBYTES + GV_ROWS * 4 * (32 / V) + mt * 256 + 64;   // codes, scales, tokens, token scales
  m.warp = stages * m.stage;
  m.chan = GV_WARPS * m.warp;                                      // channel of each W_L column
  m.ids = m.chan + (n_list + 31) / 32 * 32 * 4;                    // grouped: expert ids
  m.flag = m.ids + (rows + 3) / 4 * 16;                            // grouped: experts with rows
  m.total = m.flag + (E + 3) / 4 * 16;
  return m;
}

}  // namespace

// V: channels of a scale slot; NT: token tiles of 8; ST: stages per warp.
template <int V, int NT, int ST, bool GROUPED>
__global__ void __launch_bounds__(GV_WARPS * 32, 2) gemv_kernel(GemvParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_scan[2][GV_WARPS];
  __shared__ int s_list[16];
  __shared__ int s_slot[3];   // rows of this pass, where the next one starts, the expert
  __shared__ float s_sum[GV_ROWS * 16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int S = p.S;
  const int unit = blockIdx.x / S, rank = blockIdx.x - unit * S;
  const int N = p.N, K = p.K, nslot4 = K / V / 4;
  const int n_table = p.L ? K / p.G * p.R : 0;
  const GvSmem sm = gv_smem(V, p.mt, p.stages, min(n_table, p.K_L), GROUPED ? p.M : 0, GROUPED ? p.E : 0);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t swarp = sbase + warp * sm.warp;
  const int row0 = (unit >> 2) * 128 + (unit & 3) * 8;   // first row of octet 0; octet q is 32 q further

  grid_dep_wait();
  grid_dep_launch();

  // ---- which expert and which rows (grouped), which tokens (dense)
  int e = 0, n_rows = p.M;
  int* const ids = reinterpret_cast<int*>(smem + sm.ids);
  if constexpr (GROUPED) {
    int* const flag = reinterpret_cast<int*>(smem + sm.flag);
    for (int i = tid; i < p.E; i += GV_WARPS * 32) flag[i] = 0;
    __syncthreads();
    for (int r = tid; r < p.M; r += GV_WARPS * 32) {
      const int id = p.expert[r];
      ids[r] = id;
      if (id >= 0 && id < p.E) flag[id] = 1;
      else if (id >= p.E && blockIdx.x == 0 && blockIdx.y == 0) record_status(p.status, DEV_BAD_TABLE);
    }
    __syncthreads();
    if (blockIdx.y == 0) {
      // rows without an expert come out as zeros
      for (int r = warp * S + rank; r < p.M; r += GV_WARPS * S) {
        if (ids[r] >= 0 && ids[r] < p.E) continue;
        const int n = row0 + (lane >> 3) * 32 + (lane & 7);
        if (n < N) {
          p.Y[(size_t)r * N + n] = 0;
          if (p.Yf32) p.Yf32[(size_t)r * N + n] = 0.f;
        }
      }
    }
    if (warp == 0) {
      // the blockIdx.y-th expert (ascending) that has rows
      int left = blockIdx.y, found = -1;
      for (int b = 0; b < p.E; b += 32) {
        const unsigned m = __ballot_sync(0xffffffffu, b + lane < p.E && flag[b + lane] != 0);
        const int c = __popc(m);
        if (left < c) {
          found = b + (int)__fns(m, 0, left + 1);
          break;
        }
        left -= c;
      }
      if (lane == 0) s_slot[2] = found;
    }
    __syncthreads();
    e = s_slot[2];
    if (e < 0) return;                                   // the same for the whole cluster
  }
  const uint8_t* const QW = p.QW + (size_t)e * N * (K / 2);
  const uint8_t* const SW = p.SW + (size_t)e * ((N + 127) / 128) * nslot4 * 512;
  const uint16_t* const WL = p.WL + (size_t)e * N * p.K_L;
  const int8_t* const L = p.L + (size_t)e * n_table;

  // ---- the channel of each W_L column (-1: a pad column, or a channel already taken)
  int n_col = 0;
  int* const chan = reinterpret_cast<int*>(smem + sm.chan);
  if (n_table) {
    int it = 0;
    for (int b = 0; b < n_table; b += GV_WARPS * 32, it ^= 1) {
      const int i = b + tid;
      int v = i < n_table ? (int)L[i] : -1;
      if (v >= p.G) {
        if (unit == 0 && rank == 0) record_status(p.status, DEV_BAD_TABLE);
        v = -1;
      }
      const unsigned m = __ballot_sync(0xffffffffu, v >= 0);
      if (lane == 0) s_scan[it][warp] = __popc(m);
      __syncthreads();
      int col = n_col + __popc(m & ((1u << lane) - 1u));
      for (int w = 0; w < GV_WARPS; ++w) {
        if (w < warp) col += s_scan[it][w];
        n_col += s_scan[it][w];
      }
      if (v >= 0) {
        if (col >= p.K_L) {
          if (unit == 0 && rank == 0) record_status(p.status, DEV_BAD_TABLE);
        } else {
          bool again = false;
          for (int r = 1; r <= i % p.R; ++r) again |= (int)L[i - r] == v;
          chan[col] = again ? -1 : (i / p.R) * p.G + v;
        }
      }
    }
    n_col = min(n_col, p.K_L);
    for (int i = n_col + tid; i < (n_col + 31) / 32 * 32; i += GV_WARPS * 32) chan[i] = -1;
    __syncthreads();
  }

  const int c_end = (int)((long long)(K / GV_CHUNK) * (rank + 1) / S);
  const int c_beg = (int)((long long)(K / GV_CHUNK) * rank / S) + warp;

  for (int tile0 = GROUPED ? 0 : blockIdx.y * p.mt;;) {
    // ---- this pass's tokens: at most mt rows
    int nt_rows;
    if constexpr (GROUPED) {
      if (warp == 0) {
        // the next mt rows of expert e, in ascending order
        int have = 0, r = tile0;
        for (; r < p.M && have < p.mt; r += 32) {
          const bool hit = r + lane < p.M && ids[r + lane] == e;
          const unsigned m = __ballot_sync(0xffffffffu, hit);
          const int at = have + __popc(m & ((1u << lane) - 1u));
          if (hit && at < p.mt) s_list[at] = r + lane;
          const int c = __popc(m);
          if (have + c > p.mt) {                          // go on behind the last row taken
            r += (int)__fns(m, 0, p.mt - have + 1);
            have = p.mt;
            break;
          }
          have += c;
        }
        if (lane == 0) {
          s_slot[0] = have;
          s_slot[1] = min(r, p.M);
        }
      }
      __syncthreads();
      nt_rows = s_slot[0];
      tile0 = s_slot[1];
      if (nt_rows == 0) break;
    } else {
      nt_rows = min(p.mt, n_rows - tile0);
    }
    auto xrow = [&](int m) -> const uint16_t* {
      if constexpr (GROUPED) return p.X + (size_t)(s_list[m] / p.fan) * K;
      else return p.X + (size_t)(tile0 + m) * K;
    };

    auto load = [&](int c, int stage) {
      const uint32_t sw = swarp + stage * sm.stage;
#pragma unroll
      for (int i = 0; i < GV_WBYTES / 512; ++i) {
        const int lr = i * 8 + g;                         // row of the unit; its 16-byte piece t
        const int n = row0 + i * 32 + g;
        const bool ok = n < N;
        cp_async16(sw + lr * 64 + ((t ^ ((lr >> 1) & 3)) << 4),
                   QW + (size_t)(ok ? n : 0) * (K / 2) + (size_t)c * (GV_CHUNK / 2) + t * 16, ok);
      }
      constexpr int ATOMS = 32 / V;
      if (lane < 8 * ATOMS)
        cp_async16(sw + GV_WBYTES + lane * 16,
                   SW + ((size_t)(unit >> 2) * nslot4 + (size_t)c * ATOMS + (lane >> 3)) * 512 + (unit & 3) * 128 +
                       (lane & 7) * 16, true);
      const uint32_t sx = sw + GV_WBYTES + GV_ROWS * 4 * ATOMS;
      for (int i = lane; i < nt_rows * 16; i += 32) {
        const int m = i >> 4, q = i & 15;
        cp_async16(sx + m * 256 + ((q ^ ((m & 1) << 2)) << 4), xrow(m) + (size_t)c * GV_CHUNK + q * 8, true);
      }
    };

#pragma unroll
    for (int i = 0; i < ST; ++i) {
      if (c_beg + i * GV_WARPS < c_end) load(c_beg + i * GV_WARPS, i);
      cp_async_commit();
    }

    float acc[2][NT][4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[a][b][i] = 0.f;

    // ---- protected channels: 32 columns of W_L at a time
    for (int cc = rank * GV_WARPS + warp; cc * 32 < n_col; cc += S * GV_WARPS) {
      const int i0 = cc * 32 + t * 8;
      uint4 wl[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = row0 + q * 32 + g;
        wl[q] = n < N && i0 < p.K_L ? __ldg(reinterpret_cast<const uint4*>(WL + (size_t)n * p.K_L + i0)) : make_uint4(0, 0, 0, 0);
      }
      uint32_t xb[NT][4];
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        const int m = b * 8 + g;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t lo = 0, hi = 0;
          const int k0 = chan[i0 + 2 * i], k1 = chan[i0 + 2 * i + 1];
          if (m < nt_rows) {
            const uint16_t* x = xrow(m);
            if (k0 >= 0) lo = x[k0];
            if (k1 >= 0) hi = x[k1];
          }
          xb[b][i] = lo | (hi << 16);
        }
      }
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          mma_bf16(acc[a][b], wl[2 * a].x, wl[2 * a + 1].x, wl[2 * a].y, wl[2 * a + 1].y, xb[b][0], xb[b][1]);
          mma_bf16(acc[a][b], wl[2 * a].z, wl[2 * a + 1].z, wl[2 * a].w, wl[2 * a + 1].w, xb[b][2], xb[b][3]);
        }
    }

    // ---- the 4-bit part
    int stage = 0;
    for (int c = c_beg; c < c_end; c += GV_WARPS) {
      // the lane's four channels of the chunk, without the protected ones
      uint2 keep = make_uint2(0xFFFFFFFFu, 0xFFFFFFFFu);
      if (n_table) {
        const int k = c * GV_CHUNK + lane * 4;
        const int grp = k / p.G, local = k - grp * p.G;
        for (int r = 0; r < p.R; ++r) {
          const int at = (int)L[grp * p.R + r] - local;
          if (at == 0) keep.x &= 0xFFFF0000u;
          if (at == 1) keep.x &= 0x0000FFFFu;
          if (at == 2) keep.y &= 0xFFFF0000u;
          if (at == 3) keep.y &= 0x0000FFFFu;
        }
      }
      cp_async_wait<ST - 1>();
      __syncwarp();
      const uint32_t sw = swarp + stage * sm.stage;
      const uint32_t ss = sw + GV_WBYTES;
      const uint32_t sx = ss + GV_ROWS * 4 * (32 / V);
      const uint32_t sf = sx + p.mt * 256;
      // tokens to f16, in place
      for (int m = 0; m < nt_rows; ++m) {
        const uint32_t a = sx + m * 256 + (((lane >> 1) ^ ((m & 1) << 2)) << 4) + (lane & 1) * 8;
        uint2 v = lds64(a);
        v.x &= keep.x;
        v.y &= keep.y;
        const uint32_t am = max(max(v.x & 0x7FFFu, (v.x >> 16) & 0x7FFFu), max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu));
        const uint32_t ex = max(redux_max(am) >> 7, 15u);
        const float f = __uint_as_float((268u - ex) << 23);    // the maximum comes to [2^14, 2^15)
        v.x = pack_f16x2(__uint_as_float(v.x << 16) * f, __uint_as_float(v.x & 0xFFFF0000u) * f);
        v.y = pack_f16x2(__uint_as_float(v.y << 16) * f, __uint_as_float(v.y & 0xFFFF0000u) * f);
        sts64(a, v);
        if (lane == 0) sts32f(sf + m * 4, __uint_as_float((ex - 14u) << 23));
      }
      __syncwarp();
      float cs[2][NT][4];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) cs[a][b][i] = 0.f;
      uint4 sc[32 / V];                                        // this row's scale words, octets 0..3
#pragma unroll
      for (int i = 0; i < 32 / V; ++i) sc[i] = lds128(ss + i * 128 + g * 16);
#pragma unroll
      for (int blk = 0; blk < 4; ++blk) {
        uint32_t xb[NT][4];
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          const int m = b * 8 + g;
          const uint32_t a = sx + m * 256;
          const int sz = (m & 1) << 2;
          if (m < nt_rows) {
            if constexpr (V == 32) {
              const uint4 v = lds128(a + (((blk * 4 + t) ^ sz) << 4));
              xb[b][0] = v.x; xb[b][1] = v.y; xb[b][2] = v.z; xb[b][3] = v.w;
            } else {
              const uint2 u = lds64(a + (((blk * 4 + (t >> 1)) ^ sz) << 4) + (t & 1) * 8);
              const uint2 v = lds64(a + (((blk * 4 + 2 + (t >> 1)) ^ sz) << 4) + (t & 1) * 8);
              xb[b][0] = u.x; xb[b][1] = u.y; xb[b][2] = v.x; xb[b][3] = v.y;
            }
          } else {
            xb[b][0] = xb[b][1] = xb[b][2] = xb[b][3] = 0u;
          }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const int lo = a * 16 + g, hi = lo + 8;
          const uint32_t al = sw + lo * 64 + ((blk ^ ((lo >> 1) & 3)) << 4), ah = sw + hi * 64 + ((blk ^ ((hi >> 1) & 3)) << 4);
          uint32_t wl, wh;
          if constexpr (V == 32) {
            wl = lds32(al + t * 4);
            wh = lds32(ah + t * 4);
          } else {
            wl = lds16(al + t * 2) | (lds16(al + 8 + t * 2) << 16);
            wh = lds16(ah + t * 2) | (lds16(ah + 8 + t * 2) << 16);
          }
          uint32_t fl[4], fh[4];
          e2m1x8_to_f16(wl, fl);
          e2m1x8_to_f16(wh, fh);
          if constexpr (V == 32) {
            const uint32_t wdl = a == 0 ? sc[0].x : sc[0].z, wdh = a == 0 ? sc[0].y : sc[0].w;
            const float s0 = e8m0((wdl >> (8 * blk)) & 255u), s1 = e8m0((wdh >> (8 * blk)) & 255u);
#pragma unroll
            for (int b = 0; b < NT; ++b) {
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(d, fl[0], fh[0], fl[1], fh[1], xb[b][0], xb[b][1]);
              mma_f16(d, fl[2], fh[2], fl[3], fh[3], xb[b][2], xb[b][3]);
              cs[a][b][0] = fmaf(d[0], s0, cs[a][b][0]);
              cs[a][b][1] = fmaf(d[1], s0, cs[a][b][1]);
              cs[a][b][2] = fmaf(d[2], s1, cs[a][b][2]);
              cs[a][b][3] = fmaf(d[3], s1, cs[a][b][3]);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int slot = blk * 2 + h;
              const uint4 w4 = sc[slot >> 2];
              const uint32_t wdl = a == 0 ? w4.x : w4.z, wdh = a == 0 ? w4.y : w4.w;
              const float s0 = e8m0((wdl >> (8 * (slot & 3))) & 255u), s1 = e8m0((wdh >> (8 * (slot & 3))) & 255u);
#pragma unroll
              for (int b = 0; b < NT; ++b) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(d, fl[2 * h], fh[2 * h], fl[2 * h + 1], fh[2 * h + 1], xb[b][2 * h], xb[b][2 * h + 1]);
                cs[a][b][0] = fmaf(d[0], s0, cs[a][b][0]);
                cs[a][b][1] = fmaf(d[1], s0, cs[a][b][1]);
                cs[a][b][2] = fmaf(d[2], s1, cs[a][b][2]);
                cs[a][b][3] = fmaf(d[3], s1, cs[a][b][3]);
              }
            }
          }
        }
      }
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        const int m = b * 8 + 2 * t;
        const float f0 = m < nt_rows ? lds32f(sf + m * 4) : 0.f, f1 = m + 1 < nt_rows ? lds32f(sf + m * 4 + 4) : 0.f;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          acc[a][b][0] = fmaf(cs[a][b][0], f0, acc[a][b][0]);
          acc[a][b][1] = fmaf(cs[a][b][1], f1, acc[a][b][1]);
          acc[a][b][2] = fmaf(cs[a][b][2], f0, acc[a][b][2]);
          acc[a][b][3] = fmaf(cs[a][b][3], f1, acc[a][b][3]);
        }
      }
      __syncwarp();
      if (c + ST * GV_WARPS < c_end) load(c + ST * GV_WARPS, stage);
      cp_async_commit();
      stage = stage + 1 == ST ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- join the warps' sums (each in its own first stage), then the cluster's, in rank order
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int lr = a * 16 + g + (i >> 1) * 8, m = b * 8 + 2 * t + (i & 1);
          sts32f(swarp + (m * GV_ROWS + lr) * 4, acc[a][b][i]);
        }
    __syncthreads();
    const int n_out = nt_rows * GV_ROWS;
    auto store = [&](int o, float v) {
      const int m = o / GV_ROWS, lr = o % GV_ROWS;
      const int n = row0 + (lr >> 3) * 32 + (lr & 7);
      if (n >= N) return;
      size_t r;
      if constexpr (GROUPED) r = (size_t)s_list[m];
      else r = (size_t)(tile0 + m);
      __nv_bfloat16 h = __float2bfloat16_rn(v);
      p.Y[r * N + n] = *reinterpret_cast<uint16_t*>(&h);
      if (p.Yf32) p.Yf32[r * N + n] = v;
    };
    for (int o = tid; o < n_out; o += GV_WARPS * 32) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < GV_WARPS; ++w) v += lds32f(sbase + w * sm.warp + o * 4);
      if (S == 1) store(o, v);
      else s_sum[o] = v;
    }
    if (S > 1) {
      cluster_sync();
      const uint32_t su = smem_u32(s_sum);
      for (int o = tid * S + rank; o < n_out; o += GV_WARPS * 32 * S) {
        float v = 0.f;
        for (int r = 0; r < S; ++r) v += lds32f_cluster(mapa_shared(su + o * 4, r));
        store(o, v);
      }
      cluster_sync();                                      // the others have read this CTA's sums
    }
    if constexpr (!GROUPED) break;
    __syncthreads();                                       // the list and the stages are free again
  }
}

namespace {

template <int V, int NT, int ST, bool GROUPED>
cudaError_t launch_t(GemvParams p, int slots, cudaStream_t s) {
  static PerDeviceOnce attr_once;
  const cudaError_t ae = attr_once.run([] {
    cudaError_t e = cudaFuncSetAttribute(gemv_kernel<V, NT, ST, GROUPED>, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    return e;
  });
  if (ae != cudaSuccess) return ae;
  const int n_table = p.L ? p.K / p.G * p.R : 0;
  const int per_cta = (p.K / GV_CHUNK + p.S - 1) / p.S;
  p.stages = std::min(ST, (per_cta + GV_WARPS - 1) / GV_WARPS);
  const GvSmem sm = gv_smem(V, p.mt, p.stages, std::min(n_table, p.K_L), GROUPED ? p.M : 0, GROUPED ? p.E : 0);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_units * p.S, slots, 1);
  cfg.blockDim = dim3(GV_WARPS * 32, 1, 1);
  cfg.dynamicSmemBytes = sm.total;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, gemv_kernel<V, NT, ST, GROUPED>, p);
}

template <int NT, int ST, bool GROUPED>
cudaError_t launch_v(const GemvParams& p, int slots, cudaStream_t s) {
  return p.G == 16 ? launch_t<16, NT, ST, GROUPED>(p, slots, s) : launch_t<32, NT, ST, GROUPED>(p, slots, s);
}

}  // namespace

cudaError_t launch_gemv(const GemvParams& q, int num_sms, cudaStream_t s) {
  (void)num_sms;
  GemvParams p = q;
  p.n_units = p.N / 128 * 4 + std::min(4, p.N % 128 / 8);
  const int chunks = p.K / GV_CHUNK;
  // the K range of a CTA: at most 4 chunks per warp
  p.S = std::max(1, std::min(8, (chunks + 4 * GV_WARPS - 1) / (4 * GV_WARPS)));
  if (p.expert) {
    const int slots = std::min(p.M, p.E);
    if (p.M <= 64) {
      p.mt = std::min(p.M, 8);
      return launch_v<1, 4, true>(p, slots, s);
    }
    p.mt = 16;
    return launch_v<2, 2, true>(p, slots, s);
  }
  if (p.M <= 8) {
    p.mt = p.M;
    return launch_v<1, 4, false>(p, 1, s);
  }
  p.mt = std::min(p.M, 16);
  return launch_v<2, 2, false>(p, (p.M + 15) / 16, s);
}

}  // namespace osc
