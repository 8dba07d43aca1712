// Few bf16 token rows times a prepared 4-bit weight (decoding with unquantized activations):
//   Y[m][n] = sum_{k not in the table} x[m][k] q[n][k] 2^e[n][k/V]  +  sum_i x[m][ch_i] W_L[n][i].
// The weight is what has to be read (N K / 2 bytes of codes, N K / V of scales, 2 N K_L of W_L);
// everything else is small, so the kernel is built around keeping those bytes in flight.
//
// Unit: 32 weight rows, the four octets {q*32 + j*8 .. +7} (q = 0..3) of a 128-row block, because
// the scale layout keeps exactly those rows' words together: 128 contiguous bytes per 512-byte
// atom. Item: a unit's codes and scales of 256 channels, or its W_L of 64 columns (both 128 bytes a
// row). The work is the units of every pass (an expert's rows, mt at a time; the dense form is one
// expert), in one line, each pass after some empty places that stand for its start; each CTA, one
// per SM, takes an equal run of the line, whose parts of one pass are its segments. A segment
// stages its tokens once; teams of warps share its units, a team's warps a unit's items. Each warp
// copies its items by TMA into its own ring of stages, running ahead over the ends of units, and
// computes without waiting for another warp; a unit's sums meet in shared memory in a fixed order.
// Where units are few, or one CTA cannot hold the tokens, a cluster of S CTAs splits K and adds its
// sums through distributed shared memory.
//
// Arithmetic: mma.m16n8k16 on f16 operands with fp32 accumulators, the weight rows as the
// 16-row side and the tokens as the 8-wide side. E2M1 codes become f16 exactly (one conversion
// per two codes). The bf16 tokens become f16 after scaling each token's 256 channels by the power
// of two that puts their largest magnitude in [2^14, 2^15): a value keeps all its bits down to
// 2^-31 of that maximum. Where a value lies below (against weights that are zero at the large channels the
// small ones are all there is), the segment's tokens are staged once more, as bf16 and 2^112 times larger, and
// its weights become bf16 2^-112 times theirs (the f16 exponent in bf16's place): the products are the same
// numbers, and a value keeps its bits down to 2^-130 of the maximum. Such a call takes 1.5 to 2 times as long (K = 4096,
// N = 24576, one row: 25.3 against 13.8 us; 16 rows: 40.2 against 22.2), which is why the others stay in f16. Looking
// for such values costs three minima for each eight values, 0 to 0.5 us of a call; a zero among them takes a second look
// by the lanes that have met one (one zero: 0.9 us at one row, 2.2 us at 16).
// A scale block's products are summed in fp32, then multiplied by the weight's and the token's powers of two (exact) and
// added in fp32. Y is rounded once.
// With one or two tokens an mma takes four scale blocks at once, each in columns of its own (two with up to
// four tokens): a quarter of the scalings and of the shared-memory reads.
// The protected channels are zeroed in the staged tokens and kept apart in bf16; their products
// with W_L run as bf16 mma into the same sums.
//
// Measured (B200, launches back to back in a graph on three sets of inputs in turn): K = 4096, one token, N = 98304
// (codes and scales of 214 MB, no table): 36.4 us, 5.9 TB/s, 90 % of the copy bandwidth (39.7 us on some runs). N = 24576:
// 13.7 us against a floor of 8.5; N = 6144: 7.1 us against 2.2 (three sets of it stay in L2; with weights that do not, 7.0
// too). What is left there is the start, about 5000 cycles before the first item is multiplied (the tokens' and the
// table's round trip, their conversion by every CTA), and 1.3 or 5.2 units to an SM. In the stream itself the ALU pipe (two
// cycles a conversion) and the memory are about even: 460 cycles per item and SM sub-partition, by clock stamps in a
// copy of the kernel. With 9 to 16 tokens the conversion of the tokens takes 5 of 26 us (N = 24576), and after it the
// two warps of a scheduler do not cover the latencies between dependent instructions (issue 46 %, ALU 38 %, DRAM 24 %).
// Measured slower: one warp's ring filled with cp.async instead of TMA (FFN 19 against 17 us at the time), one team of 16
// warps per unit (20 against 16.4 us), sums handed over through mbarriers without any team barrier (QKV 7.7 against
// 7.0 us), two CTAs of 8 warps per SM (same time, 4 rows 19.1 against 16.5 us).
#include <cuda_fp16.h>
#include <type_traits>

#include "osc_device.cuh"
#include "osc_internal.h"

namespace osc {

namespace {

constexpr int GV_ROWS = 32;                       // weight rows of a unit
constexpr int CH = 256;                           // channels of an item: 128 bytes of codes a row

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
// Arrive on an mbarrier when this thread's earlier cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ float4 lds128f_cluster(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

// Eight E2M1 codes (low nibble first) as four f16 pairs, exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t& h0, uint32_t& h1, uint32_t& h2, uint32_t& h3) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3) : "r"(w));
}

// LB bytes of codes as f16 pairs; with LB = 2 also the two 8 bytes further, the next step's.
template <int LB>
__device__ __forceinline__ void load_codes(const uint8_t* from, uint32_t (&h)[LB == 2 ? 4 : LB]) {
  if constexpr (LB == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(from);
    e2m1x8_to_f16(v.x, h[0], h[1], h[2], h[3]);
    e2m1x8_to_f16(v.y, h[4], h[5], h[6], h[7]);
    e2m1x8_to_f16(v.z, h[8], h[9], h[10], h[11]);
    e2m1x8_to_f16(v.w, h[12], h[13], h[14], h[15]);
  } else if constexpr (LB == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(from);
    e2m1x8_to_f16(v.x, h[0], h[1], h[2], h[3]);
    e2m1x8_to_f16(v.y, h[4], h[5], h[6], h[7]);
  } else if constexpr (LB == 4) {
    e2m1x8_to_f16(*reinterpret_cast<const uint32_t*>(from), h[0], h[1], h[2], h[3]);
  } else {
    const uint32_t lo = *reinterpret_cast<const uint16_t*>(from), hi = *reinterpret_cast<const uint16_t*>(from + 8);
    e2m1x8_to_f16(lo | hi << 16, h[0], h[1], h[2], h[3]);
  }
}

// An E2M1 value as f16 (a pair of them) to the bf16 that is 2^-112 of it: the exponent of 5 bits in the place of 8.
__device__ __forceinline__ uint32_t f16_to_bf16_2m112(uint32_t h) { return (h >> 3 & 0x0FFF0FFFu) | (h & 0x80008000u); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same onto zero
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The two scales 2^(byte - 127) of the low bytes, through bf16 (exact, 2^-127 as its subnormal).
__device__ __forceinline__ void e8m0x2(uint32_t w, float& f0, float& f1) {
  uint32_t b;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %1;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, l;\n\t}"
      : "=r"(b) : "r"(w));
  f0 = __uint_as_float(b << 16);
  f1 = __uint_as_float(b & 0xFFFF0000u);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// max(|a|, |b|) per bf16 half; the sign bits of the result are junk.
__device__ __forceinline__ uint32_t maxabs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// min(|a|, |b|) per bf16 half; the sign bits of the result are junk.
__device__ __forceinline__ uint32_t minabs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Whether one of eight bf16 values is not zero and has an exponent below am - 31. A magnitude less 1, with the top bit
// turned, is in the order of signed 16-bit numbers, zero the largest.
__device__ __forceinline__ bool below(const uint4& q, uint32_t am) {
  auto key = [](uint32_t w) { return (w & 0x7FFF7FFFu) + 0x7FFF7FFFu; };
  auto least = [](uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.s16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  };
  const uint32_t m = least(least(key(q.x), key(q.y)), least(key(q.z), key(q.w)));
  return min((int)(short)m, (int)m >> 16) < (int)(max(am, 31u) - 31u) * 128 - 32769;
}

// Rows lr .. lr + 3 of unit u (in one octet), row r of Y.
__device__ __forceinline__ void store4(const GemvParams& p, int r, int u, int lr, const float4& v) {
  const int n = (u >> 2) * 128 + (u & 3) * 8 + (lr >> 3) * 32 + (lr & 7);
  if (n >= p.N) return;
  const size_t o = (size_t)r * p.N + n;
  *reinterpret_cast<uint2*>(p.Y + o) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  if (p.Yf32) *reinterpret_cast<float4*>(p.Yf32 + o) = v;
}

__device__ __forceinline__ int cluster_id() {
  uint32_t r;
  asm("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return (int)r;
}

// Shared memory of a CTA, in bytes from its start. kc: channels of this CTA's K range (at most); cols: W_L
// columns.
struct GvSmem {
  int stage, warp, sc, x, zero, red, xs, b, bcols, ent, ids, cnt, at, total;
};
// A warp's sums: row r of token m at m * 32 + (r ^ (m / 2 % 4) * 8), so that the mma fragments' stores
// (tokens 2t, rows g) and the reads (4 rows a lane) meet different banks.
__host__ __device__ constexpr int gv_sums(int NT, bool two) { return (two ? 2 : 8 * NT) * GV_ROWS * 4; }
__host__ __device__ inline GvSmem gv_smem(int V, int NT, int NW, int ST, bool two, int mt, int kc, int cols,
                                          int n_table, int rows, int E) {
  GvSmem m;
  m.stage = GV_ROWS * CH / 2;                                      // codes, or W_L columns
  m.warp = ST * m.stage;
  m.sc = NW * m.warp;                                              // the stages' scales
  m.x = m.sc + NW * ST * GV_ROWS * CH / V;                         // tokens in f16
  m.zero = m.x + mt * kc * 2;                                      // 64 bytes of zeros
  m.red = m.zero + 64;                                             // two sets of the warps' sums (NT = 1)
  m.xs = m.red + (NT == 1 ? 2 * NW * gv_sums(1, two) : 0);             // the tokens' powers of two, per item
  m.b = (m.xs + kc / CH * NT * 32 + 127) / 128 * 128;              // protected channels' values
  m.bcols = ((cols < n_table ? cols : n_table) + 63) / 64 * 64;
  m.ent = m.b + mt * m.bcols * 2;                                  // table entries with their columns
  m.ids = m.ent + (n_table + 3) / 4 * 16;                          // grouped: expert ids
  m.cnt = m.ids + (rows + 3) / 4 * 16;                             // grouped: rows of each expert
  m.at = m.cnt + (E + 3) / 4 * 16;                                 // where a warp's sums lie (NT = 2)
  m.total = m.at + NW * 4 + 1024;                                  // and room to start at a multiple of 1024
  return m;
}

// The team's warps meet at a barrier of their own (at most 8 teams of two warps or more need one).
__device__ __forceinline__ void team_sync(int id, int threads) {
  if (threads == 32) __syncwarp();
  else asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// A look at the tokens of a segment as they came (rows of X by `list`, or from tile0 on), and where one has a value that
// f16 has cut, all of them anew as bf16: the return value. x, xs: the staged tokens and their powers of two; ent: the table's
// entries or nullptr; the CTA's items c0 .. c0 + nc - 1; low: the warp's items at which the lane looks. A function of its
// own, and the bf16 units behind the others, so that the calls that never come here do not fetch their instructions (cold
// caches, 16 rows of K = 4096, N = 24576: 27.6 against 34.4 us with both on the way, one token through 8 experts 9.0
// against 12.0).
template <int NT, int NW, bool GROUPED>
__device__ __noinline__ bool restage_bf16(const GemvParams& p, uint8_t* x, const uint32_t* xs, const int* ent, const int* list,
                                          int tile0, int nt_rows, int c0, int nc, unsigned low) {
  constexpr int MB = NT * 4;                               // tokens at a time, for their latencies' sake
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool wide = true;
  for (int turn = 0; turn < 2 && wide; ++turn) {
    bool cut = turn > 0;
    for (int c = warp; c < nc; c += NW) {
      if (turn == 0 && !(low >> (c / NW & 31) & 1)) continue;
      const int k = (c0 + c) * CH + lane * (CH / 32), grp = (k >> p.g_shift) * p.R, local = k & (p.G - 1);
      for (int m0 = 0; m0 < nt_rows; m0 += MB) {
        uint4 q[MB];
#pragma unroll
        for (int y = 0; y < MB; ++y) {
          const int m = min(m0 + y, nt_rows - 1);
          const int row = !GROUPED ? tile0 + m : p.fan_inv ? __umulhi(list[m], p.fan_inv) : list[m];
          q[y] = *reinterpret_cast<const uint4*>(p.X + (size_t)row * p.K + k);
        }
        for (int r = 0; ent && r < p.R; ++r) {
          const int w = ent[grp + r], at = (w & 255) - local;
          if (w < 0 || at < 0 || at >= CH / 32) continue;
          const uint32_t keep = ~(0xFFFFu << (at & 1) * 16);
#pragma unroll
          for (int y = 0; y < MB; ++y) {
            if (at >> 1 == 0) q[y].x &= keep;
            if (at >> 1 == 1) q[y].y &= keep;
            if (at >> 1 == 2) q[y].z &= keep;
            if (at >> 1 == 3) q[y].w &= keep;
          }
        }
#pragma unroll
        for (int y = 0; y < MB; ++y) {
          const int m = m0 + y;
          if (m >= nt_rows) continue;
          const uint32_t two_e = xs[c * 8 * NT + m];
          if (turn == 0) {
            const uint32_t am = (two_e >> 23) + 14;
            cut |= am < 255 && below(q[y], am);            // beside infinities and NaN there is no sum to keep
            continue;
          }
          // the power of two before and 2^112: the maximum comes to [2^126, 2^127)
          const float f = __uint_as_float((254u << 23) - two_e);
          auto two = [&](uint32_t w) {
            return pack_bf16x2(__uint_as_float(w << 16) * f * 0x1p112f, __uint_as_float(w & 0xFFFF0000u) * f * 0x1p112f);
          };
          *reinterpret_cast<uint4*>(x + c * CH * 2 + m * p.kc * 2 + ((lane * (CH / 16)) ^ ((m & 1) << 6))) =
              make_uint4(two(q[y].x), two(q[y].y), two(q[y].z), two(q[y].w));
        }
      }
    }
    wide = __syncthreads_or(cut);
  }
  return wide;
}

}  // namespace

// V: channels of a scale slot; NT: token tiles of 8; NW: warps; ST: stages per warp; TWO: the
// passes have one or two tokens.
template <int V, int NT, int NW, int ST, bool GROUPED, bool TWO>
__global__ void __launch_bounds__(NW * 32, 1) gemv_kernel(const __grid_constant__ GemvMaps maps,
                                                           const __grid_constant__ GemvParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  __shared__ uint64_t s_full[NW][ST];   // a stage's data has arrived
  __shared__ uint64_t s_xbar;           // the tokens have arrived
  __shared__ int s_abort;
  __shared__ bool s_wide;               // the segment's tokens are staged as bf16
  __shared__ int s_scan[2][NW];
  __shared__ int s_cols[2];             // first W_L column of this CTA's K range, one past the last
  __shared__ int s_list[16];            // the segment's rows of Y (grouped)
  __shared__ int s_row[3][32];          // up to 32 rows: a row's expert, the rows of that, passes up to and with them
  __shared__ int s_seg[3];              // the segment's expert, rows, first row of its pass (grouped)
  __shared__ __align__(16) float s_sum[GV_ROWS * 8 * NT];
  constexpr int THREADS = NW * 32;
  constexpr int SLOT = 32 / V;                             // scale slots of 32 channels
  constexpr int RB = CH / 2;                               // bytes of an item's row: codes, or CH / 4 W_L columns
  constexpr int COLS = CH / 4;
  constexpr int SBYTES = GV_ROWS * CH / V;                 // scales of an item
  constexpr int XB = CH / 16;                              // bytes of a lane of an item of a token
  static_assert(NT == 1 || gv_sums(NT, TWO) <= GV_ROWS * RB, "a stage takes a warp's sums");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int S = p.S;
  const int cta = S == 1 ? blockIdx.x : cluster_id(), rank = S == 1 ? 0 : cluster_ctarank();
  const int N = p.N, K = p.K;
  const int n_table = p.L ? (K >> p.g_shift) * p.R : 0;
  const GvSmem sm = gv_smem(V, NT, NW, ST, TWO, p.mt, p.kc, p.K_L, n_table, GROUPED ? p.M : 0, GROUPED ? p.E : 0);
  const uint32_t sbase = smem_u32(smem);
  const int swarp = warp * sm.warp, sscale = sm.sc + warp * (ST * SBYTES);
  auto ld32 = [&](int off) { return *reinterpret_cast<const uint32_t*>(smem + off); };
  auto ld64 = [&](int off) { return *reinterpret_cast<const uint2*>(smem + off); };
  auto ld128 = [&](int off) { return *reinterpret_cast<const uint4*>(smem + off); };
  // this CTA's part of K, in items
  const int c0 = rank * p.nc_base + min(rank, p.nc_more), nc = p.nc_base + (rank < p.nc_more ? 1 : 0);

  // a warp's stages and their barriers are its own
  const uint32_t bars = smem_u32(&s_full[warp][0]);
  if (tid < 16) reinterpret_cast<uint32_t*>(smem + sm.zero)[tid] = 0u;
  if (lane == 0) {
    s_abort = 0;
    s_wide = false;
    for (int i = 0; i < ST; ++i) mbar_init(bars + i * 8, 33);   // the copying lane, and each lane's scales
    if (warp == 0) mbar_init(smem_u32(&s_xbar), NW);
    fence_barrier_init();
    if (warp == 0) {
      tma_prefetch_desc(&maps.w);
      if (n_table && p.K_L) tma_prefetch_desc(&maps.wl);   // without columns there is no map
    }
  }
  __syncthreads();

  grid_dep_wait();
  grid_dep_launch();

  // ---- the rows of each expert (grouped); up to 32 rows every warp finds them by itself, lane r for row r
  int* const ids = reinterpret_cast<int*>(smem + sm.ids);
  int* const cnt = reinterpret_cast<int*>(smem + sm.cnt);
  const bool small = GROUPED && p.M <= 32;
  unsigned w_each = p.w_each, w_more = p.w_more;
  if constexpr (GROUPED) {
    int passes;
    if (small) {
      int my_id = -1;
      if (lane < p.M) my_id = p.expert[lane];
      if (my_id >= p.E) {
        if (cta == 0 && warp == 0) record_status(p.status, DEV_BAD_TABLE);
        my_id = -1;
      }
      const unsigned same = __match_any_sync(0xffffffffu, max(my_id, -1));
      int my_pass = my_id >= 0 && __ffs(same) - 1 == lane ? (__popc(same) + p.mt - 1) >> p.mt_shift : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, my_pass, o);
        if (lane >= o) my_pass += x;
      }
      passes = __shfl_sync(0xffffffffu, my_pass, 31);
      // the same from every warp
      s_row[0][lane] = my_id;
      s_row[1][lane] = same;
      s_row[2][lane] = my_pass;
      __syncwarp();
    } else {
      const int first_id = tid < p.M ? p.expert[tid] : -1;
      for (int i = tid; i < p.E; i += THREADS) cnt[i] = 0;
      __syncthreads();
      for (int r = tid; r < p.M; r += THREADS) {
        const int id = r == tid ? first_id : p.expert[r];
        ids[r] = id;
        if (id >= 0 && id < p.E) atomicAdd(&cnt[id], 1);
        else if (id >= p.E && cta == 0) record_status(p.status, DEV_BAD_TABLE);
      }
      __syncthreads();
      int n = 0;
      for (int i = tid; i < p.E; i += THREADS) n += (cnt[i] + p.mt - 1) >> p.mt_shift;
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) s_scan[0][warp] = n;
      __syncthreads();
      passes = __reduce_add_sync(0xffffffffu, lane < NW ? s_scan[0][lane] : 0);
    }
    // rows without an expert come out as zeros
    for (int r = blockIdx.x + warp * gridDim.x; r < p.M; r += gridDim.x * NW) {
      const int id = small ? s_row[0][r] : ids[r];
      if (id >= 0 && id < p.E) continue;
      for (int n = lane * 4; n < N; n += 128) {
        *reinterpret_cast<uint2*>(p.Y + (size_t)r * N + n) = make_uint2(0, 0);
        if (p.Yf32) *reinterpret_cast<float4*>(p.Yf32 + (size_t)r * N + n) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    const unsigned total = passes ? (unsigned)passes * (p.n_units + p.gap) - p.gap : 0u;
    w_each = total / (unsigned)p.n_cta;
    w_more = total - w_each * p.n_cta;
  }
  // this CTA's run of the line, on which each pass is gap empty places and then its units (the line starts at the
  // first pass's units)
  const unsigned pitch = p.n_units + p.gap;
  unsigned wa = cta * w_each + min((unsigned)cta, w_more) + p.gap;
  const unsigned wb = wa + w_each + (cta < w_more ? 1 : 0);

  int stage = 0;                                           // of the next item to use
  uint32_t parity = 0, xparity = 0;                        // of its barrier, of the tokens'
  bool dead = false;                                       // a wait ran out
  while (wa < wb) {
    // ---- the segment: units u0 .. u1 - 1 of one pass over expert e
    int e = 0, tile0 = 0, nt_rows;
    const int pass = wa >= pitch ? wa / pitch : 0;
    const unsigned at0 = pass * pitch + p.gap;             // the place of the pass's first unit
    const int u0 = max(0, (int)(wa - at0)), u1 = min(p.n_units, (int)(wb - at0));
    wa = at0 + p.n_units;
    if (u1 <= u0) break;                                   // the run ends before the pass's units
    if constexpr (!GROUPED) {
      tile0 = pass * p.mt;
      nt_rows = min(p.mt, p.M - tile0);
    } else if (small) {
      const int l = __ffs(__ballot_sync(0xffffffffu, pass < s_row[2][lane])) - 1;
      const unsigned rows = s_row[1][l];
      e = s_row[0][l];
      const int n = __popc(rows), before = s_row[2][l] - ((n + p.mt - 1) >> p.mt_shift);
      const int first = (pass - before) * p.mt, i = __popc(rows & ((1u << lane) - 1u)) - first;
      nt_rows = min(n - first, p.mt);
      if (rows >> lane & 1 && i >= 0 && i < p.mt) s_list[i] = lane;   // the same from every warp
      __syncwarp();
    } else {
      // the expert that has pass number `pass`: 32 experts a warp at a time
      int before = 0;
      for (int b = 0;; b += THREADS) {
        const int c = b + tid < p.E ? (cnt[b + tid] + p.mt - 1) >> p.mt_shift : 0;
        const int sum = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) s_scan[1][warp] = sum;
        __syncthreads();
        const int x = lane < NW ? s_scan[1][lane] : 0;
        const int low = before + __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
        if (pass >= low && pass < low + sum) {
          int up = c;                                      // inclusive over the lanes
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += y;
          }
          if (pass >= low + up - c && pass < low + up) {
            s_seg[0] = b + tid;
            s_seg[1] = min(cnt[b + tid] - (pass - low - up + c) * p.mt, p.mt);
            s_seg[2] = (pass - low - up + c) * p.mt;
          }
        }
        before += __reduce_add_sync(0xffffffffu, x);
        __syncthreads();
        if (pass < before) break;
      }
      e = s_seg[0];
      nt_rows = s_seg[1];
      // its rows first .. first + nt_rows - 1, in ascending order
      const int first = s_seg[2];
      int have = -first;
      for (int r = 0, it = 0; r < p.M && have < nt_rows; r += THREADS, it ^= 1) {
        const bool hit = r + tid < p.M && ids[r + tid] == e;
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        if (lane == 0) s_scan[it][warp] = __popc(m);
        __syncthreads();
        const int x = lane < NW ? s_scan[it][lane] : 0;
        const int i = have + __reduce_add_sync(0xffffffffu, lane < warp ? x : 0) + __popc(m & ((1u << lane) - 1u));
        if (hit && i >= 0 && i < nt_rows) s_list[i] = r + tid;
        have += __reduce_add_sync(0xffffffffu, x);
      }
      __syncthreads();
    }
    // teams of tw warps: the fewest rounds over the teams, a round costing a warp's items and about OV / 4 more for
    // their sums; every warp of a team has items of every unit, and a cluster's CTAs are one team each
    constexpr int LOG_NW = NW == 16 ? 4 : 3, OV = 2;
    static_assert(NW == 1 << LOG_NW, "warps");
    int tw_shift = LOG_NW;
    if (S == 1) {                                          // lane i looks at teams of 2^i, the larger of two equal ones wins
      const int nu = u1 - u0, n = nc + (n_table ? (min(p.K_L, n_table) + COLS - 1) / COLS : 0), i = min(lane, LOG_NW);
      const int cost = ((nu + (NW >> i) - 1) >> (LOG_NW - i)) * (4 * ((n + (1 << i) - 1) >> i) + OV);
      tw_shift = 7 - (__reduce_min_sync(0xffffffffu, 1 << i <= nc ? cost * 8 + 7 - i : 0x7FFFFFFF) & 7);
    }
    const int tw = 1 << tw_shift, teams = NW >> tw_shift, team = warp >> tw_shift, twarp = warp & (tw - 1);
    const int8_t* const L = p.L + (size_t)e * n_table;
    const int wrow0 = GROUPED ? e * N : 0;                 // the expert's first row of QW and W_L
    // the lane's 16 bytes of an item's scales: atom lane / 8 of it, row lane % 8 of each octet
    const int satoms = K / V / 4;
    const uint8_t* const sfrom = p.SW + ((size_t)(GROUPED ? e * ((N + 127) / 128) : 0) * satoms +
                                         (size_t)c0 * (CH / V / 4) + (lane >> 3)) * 512 + (lane & 7) * 16;
    auto xrow = [&](int m) -> const uint16_t* {
      if constexpr (GROUPED) return p.X + (size_t)(p.fan_inv ? __umulhi(s_list[m], p.fan_inv) : s_list[m]) * K;
      else return p.X + (size_t)(tile0 + m) * K;
    };

    // ---- what the rest waits for first: the table, and the tokens as they are (one copy each)
    const int8_t l_first = tid < n_table ? L[tid] : -1;
    if (lane == 0) {
      const uint32_t xbar = smem_u32(&s_xbar), bytes = nc * CH * 2;
      mbar_arrive_expect_tx(xbar, max(0, (nt_rows - warp + NW - 1) / NW) * bytes);
      for (int m = warp; m < nt_rows; m += NW) bulk_load(sbase + sm.x + m * p.kc * 2, xrow(m) + (size_t)c0 * CH, bytes, xbar);
    }

    // ---- start the weight stream: the next item to load is pj of unit pu. Items 0 .. nc - 1 of a
    // unit are codes; the W_L columns' items follow, known only after the table has been read. The
    // first item of a unit goes to the next warp of the team in each unit.
    int items = 0x7FFFFFFF, w0 = 0;
    int pu = dead ? u1 : u0 + team, poff = 0, pj = twarp;
    auto settle = [&] {                                    // past the end of a unit: to the next one
      while (pj >= items && pu < u1) {
        pu += teams;
        poff += items;
        pj = (twarp - poff) & (tw - 1);
      }
    };
    auto load_next = [&](int to) {
      if (pu >= u1) return;
      if (lane == 0) {
        const uint32_t sw = sbase + swarp + to * sm.stage, bar = bars + to * 8;
        const bool main = pj < nc;
        const CUtensorMap* const m = main ? &maps.w : &maps.wl;
        const int x = main ? (c0 + pj) * RB : (w0 + pj - nc) * COLS;
        mbar_arrive_expect_tx(bar, GV_ROWS * RB);
        // octet q: rows 32 q + 8 (pu % 4) .. + 7 of the 128-row block
        if (p.rows32) {
          tma_load_3d(sw, m, x, (pu & 3) * 8, (wrow0 >> 5) + (pu >> 2) * 4, bar);
        } else {
#pragma unroll 1
          for (int q = 0; q < 4; ++q)
            tma_load_3d(sw + q * 8 * RB, m, x, wrow0 + (pu >> 2) * 128 + q * 32 + (pu & 3) * 8, 0, bar);
        }
      }
      if (pj < nc && lane * 16 < SBYTES)
        cp_async16(sbase + sscale + to * SBYTES + lane * 16,
                     sfrom + ((size_t)(pu >> 2) * satoms + (size_t)pj * (CH / V / 4)) * 512 + (pu & 3) * 128);
      cp_async_arrive(bars + to * 8);
      pj += tw;
      if (pj >= items) settle();
    };
    // one item now, the others when the tokens are staged, so that these do not queue behind them
    int pre = 0, pstage = stage;
    if (pj < nc) {
      load_next(pstage);
      pstage = pstage + 1 == ST ? 0 : pstage + 1;
      pre = 1;
    }

    // ---- the table: each entry with its W_L column (-1: none)
    int* const ent = reinterpret_cast<int*>(smem + sm.ent);
    int cols = 0;
    if (n_table) {
      const int e0 = (c0 * CH >> p.g_shift) * p.R, e1 = ((c0 + nc) * CH >> p.g_shift) * p.R;
      int n_col = 0, it = 0;
      for (int i = tid; i < p.mt * sm.bcols / 8; i += THREADS) reinterpret_cast<uint4*>(smem + sm.b)[i] = make_uint4(0, 0, 0, 0);
      for (int b = 0; b < n_table; b += THREADS, it ^= 1) {
        const int i = b + tid;
        int v = b == 0 ? (int)l_first : i < n_table ? (int)L[i] : -1;
        if (v >= p.G) {
          if (u0 == 0) record_status(p.status, DEV_BAD_TABLE);
          v = -1;
        }
        const unsigned m = __ballot_sync(0xffffffffu, v >= 0);
        if (lane == 0) s_scan[it][warp] = __popc(m);
        __syncthreads();
        const int c = lane < NW ? s_scan[it][lane] : 0;
        const int col = n_col + __reduce_add_sync(0xffffffffu, lane < warp ? c : 0) + __popc(m & ((1u << lane) - 1u));
        n_col += __reduce_add_sync(0xffffffffu, c);
        if (i == e0) s_cols[0] = col;
        if (i == e1) s_cols[1] = col;
        if (v >= 0 && col >= p.K_L) {
          if (u0 == 0) record_status(p.status, DEV_BAD_TABLE);
          v = -1;
        }
        if (i < n_table) ent[i] = v >= 0 ? col << 8 | v : -1;
      }
      if (tid == 0 && e1 == n_table) s_cols[1] = n_col;
      __syncthreads();
      w0 = min(s_cols[0], p.K_L) / COLS;
      cols = max(0, (min(s_cols[1], p.K_L) + COLS - 1) / COLS - w0);
    }
    items = nc + cols;
    if (pj >= items) settle();

    // ---- stage the tokens: protected channels apart, the rest as f16 with a power of two per token and item,
    // in place (16-byte pieces of odd tokens trade places in fours, so that two tokens' 64 bytes will meet
    // different banks)
    mbar_wait(smem_u32(&s_xbar), xparity, &s_abort, p.status);
    xparity ^= 1;
    unsigned low = 0;                                      // items where the lane has met a value that f16 has cut, or a zero
    auto convert = [&](auto mb) {
      constexpr int MB = decltype(mb)::value;              // tokens at a time, for their latencies' sake
      for (int c = warp; c < nc; c += NW) {
        const int k = (c0 + c) * CH + lane * (CH / 32);
        const int grp = (k >> p.g_shift) * p.R, local = k & (p.G - 1);
        uint8_t* const xc = smem + sm.x + c * CH * 2;
        for (int m0 = 0; m0 < nt_rows; m0 += MB) {
          uint32_t v[MB][XB / 4], am[MB], mn[MB];          // mn: least magnitudes, protected ones among them
#pragma unroll
          for (int y = 0; y < MB; ++y) {
            const int m = MB == 1 ? m0 : min(m0 + y, nt_rows - 1);
            const uint8_t* const x = xc + m * p.kc * 2 + lane * XB;
            const uint4 q = *reinterpret_cast<const uint4*>(x);
            v[y][0] = q.x; v[y][1] = q.y; v[y][2] = q.z; v[y][3] = q.w;
            mn[y] = minabs2(minabs2(q.x, q.y), minabs2(q.z, q.w));
          }
          if (n_table)
            for (int r = 0; r < p.R; ++r) {
              const int w = ent[grp + r], at = (w & 255) - local, col = w >> 8;
              if (w < 0 || at < 0 || at >= CH / 32) continue;
#pragma unroll
              for (int y = 0; y < MB; ++y) {
                // in table order: a channel named twice gives its value once and then 0
                const int m = m0 + y;
                uint32_t x = 0;
#pragma unroll
                for (int i = 0; i < XB / 4; ++i) {
                  const uint32_t hit = i == at >> 1 ? 0xFFFFu << (at & 1) * 16 : 0u;
                  x |= v[y][i] & hit;
                  v[y][i] &= ~hit;
                }
                if (MB == 1 || m < nt_rows)
                  *reinterpret_cast<uint16_t*>(smem + sm.b + m * sm.bcols * 2 + (((col >> 3) ^ ((m & 1) << 2)) << 4) +
                                               (col & 7) * 2) = (uint16_t)(x >> (at & 1) * 16);
              }
            }
          __syncwarp();
#pragma unroll
          for (int y = 0; y < MB; ++y) {
            const uint32_t a = maxabs2(maxabs2(v[y][0], v[y][1]), maxabs2(v[y][2], v[y][3]));
            am[y] = max(a & 0x7FFFu, (a >> 16) & 0x7FFFu);
          }
#pragma unroll
          for (int y = 0; y < MB; ++y) am[y] = max(__reduce_max_sync(0xffffffffu, am[y]) >> 7, 15u);
#pragma unroll
          for (int y = 0; y < MB; ++y) {
            const int m = m0 + y;
            if (MB > 1 && m >= nt_rows) continue;
            const float f = __uint_as_float((268u - am[y]) << 23);   // the maximum comes to [2^14, 2^15)
#pragma unroll
            for (int i = 0; i < XB / 4; ++i)
              v[y][i] = pack_f16x2(__uint_as_float(v[y][i] << 16) * f, __uint_as_float(v[y][i] & 0xFFFF0000u) * f);
            uint8_t* const x = xc + m * p.kc * 2 + ((lane * XB) ^ ((m & 1) << 6));
            *reinterpret_cast<uint4*>(x) = make_uint4(v[y][0], v[y][1], v[y][2], v[y][3]);
            if (lane == 0) *reinterpret_cast<float*>(smem + sm.xs + (c * 8 * NT + m) * 4) = __uint_as_float((am[y] - 14u) << 23);
          }
          // a half keeps its top bit where its magnitude is 2^-31 of the maximum or more
          uint32_t high = 0x80008000u;
#pragma unroll
          for (int y = 0; y < MB; ++y) high &= (mn[y] | 0x80008000u) - (max(am[y], 31u) - 31u) * 0x00800080u;
          if (high != 0x80008000u) low |= 1u << (c / NW & 31);
        }
      }
    };
    if (TWO || nt_rows <= 2) convert(std::integral_constant<int, 1>{});
    else convert(std::integral_constant<int, 4>{});
#pragma unroll 1
    for (; pre < ST; ++pre) {
      load_next(pstage);
      pstage = pstage + 1 == ST ? 0 : pstage + 1;
    }
    // rare: a lane has met a value that f16 has cut, or a zero (the answer in shared memory: a register more spills)
    if (__builtin_expect(__syncthreads_or(low != 0), 0))
      s_wide = restage_bf16<NT, NW, GROUPED>(p, smem + sm.x, reinterpret_cast<const uint32_t*>(smem + sm.xs),
                                             n_table ? ent : nullptr, GROUPED ? s_list : nullptr, tile0, nt_rows, c0, nc, low);

    // ---- the units. P: scale blocks of an mma. An mma's 16 k-slots are four of each lane t; a lane's slots
    // lie in one scale block, 4 / P lanes to a block. Column n of a tile is token n / P against block n % P
    // of the step alone: the B operand of lane (g, t) is zero where its block is not g % P, so that the P
    // blocks' sums stay apart and one scale each is enough for a step of P blocks. Rows: lane g takes
    // row rg of each octet, the bit reversal of g, so that neighbours' equal pieces meet different banks.
    // WIDE: the tokens are staged as bf16.
    auto run = [&](auto pc, auto wc) {
      constexpr int P = decltype(pc)::value;
      constexpr bool WIDE = decltype(wc)::value;
      constexpr int STEP = V * P;                          // channels of a step
      constexpr int LB = STEP / 8;                         // a lane's code bytes of a step and row
      const int rg = (g & 1) << 2 | (g & 2) | g >> 2;
      const int rd = rg * RB + (((t * LB >> 4) ^ rg) << 4) + (t * LB & 15), rw = rg * RB + ((t ^ rg) << 4);   // codes, W_L
      int xa[NT], ba[NT];
      bool live[NT];
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        const int m = b * 8 + g / P, mw = min(b * 8 + g, nt_rows - 1);
        live[b] = m < nt_rows && t / (4 / P) == g % P;
        // lanes past the last token: zeros, or with P = 1 its repetition (those columns are never stored)
        const int mx = P == 1 ? mw : m;
        xa[b] = sm.x + mx * p.kc * 2 + (((mx & 1) << 6) ^ (t * STEP / 2));
        ba[b] = sm.b + mw * sm.bcols * 2 + ((mw & 1) << 6) + t * 16;
      }
      auto next_stage = [&] {
        if (++stage == ST) {
          stage = 0;
          parity ^= 1;
        }
      };
      int off = 0;
      int red = sm.red;                                    // this unit's set of sums (NT = 1)
      for (int u = u0 + team; u < u1; u += teams) {
        float acc[2][NT][4], accw[2][NT][4];               // codes' sums by column; W_L's by token
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[a][b][i] = accw[a][b][i] = 0.f;
        const int j0 = (twarp - off) & (tw - 1);
        for (int j = j0; j < items; j += tw) {
          // a wait that ran out is recorded: nothing more is loaded, every loop ends, the sums are undefined
          if (!mbar_wait(bars + stage * 8, parity, &s_abort, p.status)) {
            dead = true;
            pu = u1;
          }
          const int sw = swarp + stage * sm.stage;
          if (j >= nc) {
            // protected channels: COLS columns of W_L
#pragma unroll
            for (int h = 0; h < CH / 128; ++h) {
              uint4 wl[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) wl[q] = ld128(((sw + rw) ^ (h * 64)) + q * 8 * RB);
#pragma unroll
              for (int b = 0; b < NT; ++b) {
                const int c = (w0 + j - nc) * (COLS / 32) + h;
                const uint4 x = ld128((ba[b] + (c >> 1) * 128) ^ ((c & 1) * 64));
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                  mma_bf16(accw[a][b], wl[2 * a].x, wl[2 * a + 1].x, wl[2 * a].y, wl[2 * a + 1].y, x.x, x.y);
                  mma_bf16(accw[a][b], wl[2 * a].z, wl[2 * a + 1].z, wl[2 * a].w, wl[2 * a + 1].w, x.z, x.w);
                }
              }
            }
          } else {
            float cs[2][NT][4];
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
              for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) cs[a][b][i] = 0.f;
            const int ssc = sscale + stage * SBYTES + rg * 16;
#pragma unroll
            for (int h = 0; h < CH / 128; ++h) {
              // the scales of the lane's columns 2t, 2t + 1 of each step, for its row in octets 0..3
              constexpr int STEPS = 128 / STEP, NS = P == 1 ? 1 : 2;
              float sc[4][STEPS][NS];
#pragma unroll
              for (int i = 0; i < SLOT; ++i) {
                const uint4 w4 = ld128(ssc + (h * SLOT + i) * 128);
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if constexpr (P == 4) {
                    e8m0x2(w[q] >> ((t & 1) * 16), sc[q][i][0], sc[q][i][NS - 1]);
                  } else if constexpr (P == 2) {
                    e8m0x2(w[q], sc[q][2 * i][0], sc[q][2 * i][NS - 1]);
                    e8m0x2(w[q] >> 16, sc[q][2 * i + 1][0], sc[q][2 * i + 1][NS - 1]);
                  } else {
                    e8m0x2(w[q], sc[q][4 * i][0], sc[q][4 * i + 1][0]);
                    e8m0x2(w[q] >> 16, sc[q][4 * i + 2][0], sc[q][4 * i + 3][0]);
                  }
                }
              }
              constexpr int PAIR = LB == 2 ? 2 : 1, LN = STEP / 8 * PAIR;
              uint32_t fl[2][LN], fh[2][LN];               // f16 pairs of rows rg and rg + octet, by tile
#pragma unroll
              for (int st = 0; st < STEPS; ++st) {
                constexpr int XN = STEP / 8;               // a lane's words of a step: tokens
                constexpr int CO = STEP / 2, XO = STEP * 2;   // a row's code bytes, a token's bytes of a step
                uint32_t xb[NT][XN];
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                  const int x = xa[b] + j * (CH * 2) + h * 256;
#pragma unroll
                  for (int i = 0; i < XN; i += 4) {
                    const int at = P == 1 || live[b] ? (x ^ (st * XO & 255)) + i * 4 : sm.zero + i * 4;
                    if constexpr (XN >= 4) {
                      const uint4 v = ld128(at);
                      xb[b][i] = v.x; xb[b][i + 1] = v.y; xb[b][i + 2] = v.z; xb[b][i + 3] = v.w;
                    } else {
                      const uint2 v = ld64(at);
                      xb[b][0] = v.x; xb[b][1] = v.y;
                    }
                  }
                }
                const int w0b = (sw + rd) ^ (h * 64 + st * CO);
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                  if (st % PAIR == 0) {
                    load_codes<LB>(smem + w0b + a * 16 * RB, fl[a]);
                    load_codes<LB>(smem + w0b + (a * 16 + 8) * RB, fh[a]);
#pragma unroll
                    for (int i = 0; WIDE && i < LN; ++i) {
                      fl[a][i] = f16_to_bf16_2m112(fl[a][i]);
                      fh[a][i] = f16_to_bf16_2m112(fh[a][i]);
                    }
                  }
                  const uint32_t* const l = fl[a] + st % PAIR * 2, *const h8 = fh[a] + st % PAIR * 2;
                  const float s0 = sc[2 * a][st][0], s1 = sc[2 * a][st][NS - 1];
                  const float s2 = sc[2 * a + 1][st][0], s3 = sc[2 * a + 1][st][NS - 1];
#pragma unroll
                  for (int b = 0; b < NT; ++b) {
                    float d[4];
                    if constexpr (WIDE) {
                      d[0] = d[1] = d[2] = d[3] = 0.f;
#pragma unroll
                      for (int i = 0; i < STEP / 8; i += 2) mma_bf16(d, l[i], h8[i], l[i + 1], h8[i + 1], xb[b][i], xb[b][i + 1]);
                    } else {
                      mma_f16_first(d, l[0], h8[0], l[1], h8[1], xb[b][0], xb[b][1]);
#pragma unroll
                      for (int i = 2; i < STEP / 8; i += 2) mma_f16(d, l[i], h8[i], l[i + 1], h8[i + 1], xb[b][i], xb[b][i + 1]);
                    }
                    cs[a][b][0] = fmaf(d[0], s0, cs[a][b][0]);
                    cs[a][b][1] = fmaf(d[1], s1, cs[a][b][1]);
                    cs[a][b][2] = fmaf(d[2], s2, cs[a][b][2]);
                    cs[a][b][3] = fmaf(d[3], s3, cs[a][b][3]);
                  }
                }
              }
            }
#pragma unroll
            for (int b = 0; b < NT; ++b) {
              const int f = sm.xs + (j * 8 * NT + b * 8 + 2 * t / P) * 4;
              const float f0 = __uint_as_float(ld32(f)), f1 = P == 1 ? __uint_as_float(ld32(f + 4)) : f0;
#pragma unroll
              for (int a = 0; a < 2; ++a) {
                acc[a][b][0] = fmaf(cs[a][b][0], f0, acc[a][b][0]);
                acc[a][b][1] = fmaf(cs[a][b][1], f1, acc[a][b][1]);
                acc[a][b][2] = fmaf(cs[a][b][2], f0, acc[a][b][2]);
                acc[a][b][3] = fmaf(cs[a][b][3], f1, acc[a][b][3]);
              }
            }
          }
          if (NT == 1 || j + tw < items) {                 // NT = 2: the last stage takes the sums first
            __syncwarp();
            load_next(stage);
            next_stage();
          }
        }

        // ---- join the team's sums (every warp has had an item): in one of two sets (the other may still
        // be being read), or where these do not fit (NT = 2) in the stage just consumed
        int* const at = reinterpret_cast<int*>(smem + sm.at);
        int to = red + warp * gv_sums(NT, TWO);
        if constexpr (NT == 2) {
          __syncwarp();
          to = swarp + stage * sm.stage;
          if (lane == 0) at[warp] = to;
        }
        // the blocks' columns of a token add up to its sum, which then takes its place among the tokens' columns
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              float v0 = acc[a][b][i], v1 = acc[a][b][i + 1];
              if constexpr (P > 1) {
                v0 += v1;                                  // P = 2: lane t has token t
                if constexpr (P == 4) v0 += __shfl_xor_sync(0xffffffffu, v0, 1);   // lanes 2m, 2m + 1 have token m
                v1 = __shfl_sync(0xffffffffu, v0, (lane & ~3) | (P == 4 ? 2 : min(2 * t + 1, 3)));
                v0 = __shfl_sync(0xffffffffu, v0, (lane & ~3) | (P == 4 ? 0 : min(2 * t, 3)));
              }
              acc[a][b][i] = v0 + accw[a][b][i];
              acc[a][b][i + 1] = v1 + accw[a][b][i + 1];
            }
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int m = b * 8 + 2 * t + i;
            if (m >= nt_rows) continue;
            float* const x = reinterpret_cast<float*>(smem + to) + m * GV_ROWS + rg;
            x[0 ^ t * 8] = acc[0][b][i];
            x[8 ^ t * 8] = acc[0][b][2 + i];
            x[16 ^ t * 8] = acc[1][b][i];
            x[24 ^ t * 8] = acc[1][b][2 + i];
          }
        if (NT == 2) fence_proxy_async_smem();             // the next copy into this stage comes after
        team_sync(1 + team, tw * 32);
        // a lane sums 4 rows of a token over the team's warps (P = 4: over half of them, and two lanes meet);
        // another warp's turn first in each unit
        constexpr int HALVES = P == 4 ? 2 : 1, TOK = 4 / HALVES;
        const int lr = (lane & 7) * 4, half = HALVES == 2 ? (lane >> 3) & 1 : 0;
        for (int mb = j0 * TOK; mb < nt_rows; mb += tw * TOK) {
          const int m = mb + (lane >> 3) / HALVES;
          const int o = (m * GV_ROWS + (lr ^ (m >> 1 & 3) * 8)) * 4;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (m < nt_rows) {
#pragma unroll 4
            for (int w = team * tw + half; w < team * tw + tw; w += HALVES) {
              const float4 x = *reinterpret_cast<const float4*>(smem + (NT == 1 ? red + w * gv_sums(NT, TWO) : at[w]) + o);
              v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
            }
          }
          if constexpr (HALVES == 2) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, 8);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, 8);
            v.z += __shfl_xor_sync(0xffffffffu, v.z, 8);
            v.w += __shfl_xor_sync(0xffffffffu, v.w, 8);
          }
          if (m < nt_rows && half == 0) {
            if (S == 1) store4(p, GROUPED ? s_list[m] : tile0 + m, u, lr, v);
            else *reinterpret_cast<float4*>(s_sum + m * GV_ROWS + lr) = v;
          }
        }
        if (S > 1) {                                       // one team per CTA
          cluster_sync();
          const uint32_t su = smem_u32(s_sum);
          for (int o = tid * S + rank; o < nt_rows * (GV_ROWS / 4); o += THREADS * S) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < S; ++r) {
              const float4 x = lds128f_cluster(mapa_shared(su + o * 16, r));
              v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
            }
            store4(p, tile0 + o / (GV_ROWS / 4), u, o % (GV_ROWS / 4) * 4, v);
          }
          cluster_sync();                                  // the others have read this CTA's sums
        } else if (NT == 2) {
          team_sync(1 + team, tw * 32);                    // the sums have been read
        }
        if (NT == 2) {
          load_next(stage);
          next_stage();
        }
        if (NT == 1) red = 2 * sm.red + NW * gv_sums(NT, TWO) - red;
        off += items;
      }
    };
    const std::false_type plain{};
    if (__builtin_expect(!s_wide, 1)) {
      if (NT == 2) run(std::integral_constant<int, 1>{}, plain);
      else if (TWO || nt_rows <= 2) run(std::integral_constant<int, 4>{}, plain);
      else if (nt_rows <= 4) run(std::integral_constant<int, 2>{}, plain);
      else run(std::integral_constant<int, 1>{}, plain);
    } else {
      run(std::integral_constant<int, TWO ? 4 : 1>{}, std::true_type{});
      __syncthreads();
      s_wide = false;
    }
    if (wa < wb) {
      fence_proxy_async_smem();                            // the next tokens' copies come after
      __syncthreads();                                     // the list, the table and the tokens are free again
    }
  }
  // after a timeout, copies still in flight get a moment to land before the shared memory is given up
  if (*reinterpret_cast<volatile int*>(&s_abort)) {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 10000000ull) {}
  }
}

namespace {

// Tensor maps of the codes and of W_L, one copy of an item each. Rows as (32 rows) x (blocks of 32), so
// that one box {a row's bytes, 8 rows, 4 blocks} is a unit's four octets; where N is not a multiple of
// 32 as one run of rows, a box of 8. Swizzled by the 128-byte row, so that 8 rows' equal pieces meet
// different banks.
cudaError_t encode_gemv_maps(GemvMaps* m, const GemvParams& p, int E) {
  const uint64_t rows = (uint64_t)E * p.N;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  auto operand = [&](CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t width, uint64_t pitch, uint32_t box) {
    const uint64_t d3[3] = {width, 32, rows / 32}, s3[2] = {pitch, pitch * 32};
    const uint64_t d1[3] = {width, rows, 1}, s1[2] = {pitch, pitch * rows};
    const uint32_t b3[3] = {box, 8, 4}, b1[3] = {box, 8, 1};
    return p.rows32 ? encode_map(map, dt, 3, base, d3, s3, b3, sw) : encode_map(map, dt, 3, base, d1, s1, b1, sw);
  };
  cudaError_t e = operand(&m->w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.QW, (uint64_t)p.K / 2, (uint64_t)p.K / 2, CH / 2);
  if (e == cudaSuccess && p.L && p.K_L)
    e = operand(&m->wl, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.WL, (uint64_t)p.K_L, (uint64_t)p.K_L * 2, CH / 4);
  return e;
}

// Items that the start of a pass counts for in the cut of the work: a CTA whose run crosses into another pass drains its
// ring and stages anew, 6000 cycles in which it would multiply some 45 items (16 tokens by 8 experts, K = 768: 19.6 us
// against 22.3 us cut by units alone; 33 tokens, K = 2048: 39.7 against 40.6). One number for all variants: over eleven
// calls, grouped and in dense passes, G = 16 to 64, it is the best of 1, 20, 45, 90 and 180 or within 7 % of it.
constexpr int GV_GAP = 45;
constexpr int GV_SMEM_MAX = 232448 - 4096;                 // 227 KB less the static part (3 KB at most)

template <int V, int NT, int NW, int ST, bool GROUPED, bool TWO>
cudaError_t launch_t(const GemvMaps& maps, const GemvParams& p, int smem, cudaStream_t s) {
  static PerDeviceOnce attr_once;
  const cudaError_t ae = attr_once.run([] {
    return cudaFuncSetAttribute(gemv_kernel<V, NT, NW, ST, GROUPED, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                GV_SMEM_MAX);
  });
  if (ae != cudaSuccess) return ae;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_cta * p.S, 1, 1);
  cfg.blockDim = dim3(NW * 32, 1, 1);
  cfg.dynamicSmemBytes = smem;
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
  return cudaLaunchKernelEx(&cfg, gemv_kernel<V, NT, NW, ST, GROUPED, TWO>, maps, p);
}

// How many clusters of S = 1 .. 8 CTAs that fill an SM each are resident at once, at (*n)[S]. Clusters of three CTAs
// and more do not tile the GPCs (45 of three on 148 SMs), and a launch of more runs in two waves: one row, K = 12288, S = 3:
// 44 clusters 6.5 us, 48 clusters 11.9 us.
cudaError_t resident_clusters(int num_sms, const int** n) {
  static PerDeviceOnce once;
  static int count[PerDeviceOnce::kMaxDevices][9];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = once.run([=] {
    count[dev][1] = num_sms;
    const auto kernel = gemv_kernel<32, 1, 16, 2, false, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GV_SMEM_MAX);
    for (int s = 2; s <= 8 && e == cudaSuccess; ++s) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = s;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(s, 1, 1);
      cfg.blockDim = dim3(16 * 32, 1, 1);
      cfg.dynamicSmemBytes = GV_SMEM_MAX;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int c = 0;
      e = cudaOccupancyMaxActiveClusters(&c, kernel, &cfg);
      count[dev][s] = std::max(1, c);
    }
    return e;
  });
  *n = e == cudaSuccess ? count[dev] : nullptr;
  return e;
}

// S parts of K, one per CTA of a cluster, and what a call with NW warps will take with them, in 10 ns and less what all
// calls take. A CTA's unit costs 0.12 us an item with 16 warps and 0.16 with 8, which in turn start 0.4 us sooner; the
// join over the cluster costs a unit 1.5 us, the last one 1.0: figures of one row. With more rows, or G = 16, an item and
// the join both cost more, so the same choice comes out well: forced to every other number of parts, calls of 1 to 16
// rows, G = 16 to 64, K = 4096 to 16384 were at most 3 % faster, but for 16 rows of K = 12288, N = 1536 (three parts 14.0
// us, four 12.4). One row, K = 12288, N = 4096: whole 8.3 us, two parts 11.2; 16 rows, N = 2048, K = 4096: two parts 6.8
// us, whole 8.7; 16 rows, K = 16384, N = 512, G = 16: eight parts 9.4 us, six 9.4, seven (in two waves) 13.2.
struct GvSplit {
  int S;
  long long cost;
};
GvSplit gv_split(int NW, int max_s, int chunks, long long work, const int* clusters) {
  GvSplit r{1, 0x7FFFFFFFFFFFFFFFll};
  for (int S = 1; S <= max_s && (S == 1 || chunks / S >= NW); ++S) {
    const long long n = (work + clusters[S] - 1) / clusters[S];   // a CTA's units
    const long long cost = (NW == 16 ? 40 : 0) + n * ((chunks + S - 1) / S) * (NW == 16 ? 12 : 16) + (S > 1 ? 150 * n - 50 : 0);
    if (cost < r.cost) r = GvSplit{S, cost};
  }
  return r;
}

// The split of one call. NT, NW and ST are the kernel's, p.mt the most tokens of a pass. Where `try_only` and
// the tokens of a pass would not fit one CTA it returns cudaErrorInvalidValue and launches nothing; else it
// splits K further, then takes fewer tokens a pass (one always fits within the limits of the entry points).
template <int NT, int NW, int ST, bool GROUPED, bool TWO = false>
cudaError_t launch_v(GemvParams p, bool try_only, const int* clusters, cudaStream_t s) {
  const int V = p.G == 16 ? 16 : 32;
  const int chunks = p.K / CH;
  const int n_table = p.L ? p.K / p.G * p.R : 0;
  auto smem_of = [&](int S) {
    p.kc = (chunks + S - 1) / S * CH;
    return gv_smem(V, NT, NW, ST, TWO, p.mt, p.kc, p.K_L, n_table, GROUPED ? p.M : 0, GROUPED ? p.E : 0).total;
  };
  const int max_s = GROUPED ? 1 : 8;
  p.gap = std::max(1, GV_GAP / chunks);
  auto work_of = [&] { return (long long)(p.n_units + p.gap) * ((p.M + p.mt - 1) / p.mt) - p.gap; };
  p.S = gv_split(NW, max_s, chunks, work_of(), clusters).S;
  while (smem_of(p.S) > GV_SMEM_MAX) {
    if (try_only) return cudaErrorInvalidValue;
    if (p.S < max_s && chunks / (p.S + 1) >= NW) ++p.S;
    else if (p.mt > 1) p.mt = (p.mt + 1) / 2;
    else return cudaErrorInvalidValue;
  }
  const int smem = smem_of(p.S);
  while (1 << p.mt_shift < p.mt) ++p.mt_shift;
  p.nc_base = chunks / p.S;
  p.nc_more = chunks % p.S;
  const long long work = work_of();
  if (work > 0x7FFFFFFF) return cudaErrorInvalidValue;
  // grouped: at most one pass per row
  p.n_cta = (int)std::min<long long>(clusters[p.S], GROUPED ? (long long)p.n_units * p.M : work);
  p.w_each = (unsigned)(work / p.n_cta);
  p.w_more = (unsigned)(work % p.n_cta);
  GemvMaps maps;
  const cudaError_t e = encode_gemv_maps(&maps, p, GROUPED ? p.E : 1);
  if (e != cudaSuccess) return e;
  return V == 16 ? launch_t<16, NT, NW, ST, GROUPED, TWO>(maps, p, smem, s)
                 : launch_t<32, NT, NW, ST, GROUPED, TWO>(maps, p, smem, s);
}

}  // namespace

// The variant by the rows, by the time that gv_split expects, and by what fits:
//   1 .. 8 rows: one token tile, 16 warps with two stages each, or 8 with three where a CTA has few items (one row, N = 544:
//   K = 2048 4.4 against 4.7 us, K = 6144 in three parts 5.1 against 6.4; N = 6144, K = 4096: 7.5 against 7.1) or the tokens
//   and tables leave too little room for the first ring (5 rows, K = 12288, N = 4096, G = 16: 14.6 us in two parts, against
//   16.4 us for 16 warps on K in three parts). One or two rows have kernels of their own, without the code for more and with room for two rows' sums
//   alone (N = 6144: 7.1 against 7.4 us; two rows of K = 12288, G = 16: 11.1 against 12.9).
//   Routed rows: 16 warps, or 8 where these do not fit (33 tokens by 8 experts: 41.7 against 44.8 us).
//   9 rows and more: two token tiles, 16 rows a pass, 8 warps with the registers of 16 (16 rows, N = 24576: 25.9 us,
//   against 30.2 us in passes of 8 rows and 31.5 us with 16 warps on items of 128 channels).
cudaError_t launch_gemv(const GemvParams& q, int num_sms, cudaStream_t s) {
  GemvParams p = q;
  p.n_units = p.N / 128 * 4 + std::min(4, p.N % 128 / 8);
  p.g_shift = p.G == 16 ? 4 : p.G == 32 ? 5 : 6;
  p.rows32 = p.N % 32 == 0;
  p.fan_inv = (unsigned)(((1LL << 32) + p.fan - 1) / p.fan);   // exact for rows up to GEMV_MAX_ROWS; 0 for a fan of 1
  const int* clusters;
  const cudaError_t e = resident_clusters(num_sms, &clusters);
  if (e != cudaSuccess) return e;
  if (p.expert) {
    p.mt = p.M > 4 ? 8 : p.M > 2 ? 4 : p.M;
    const cudaError_t e = launch_v<1, 16, 2, true>(p, true, clusters, s);
    return e != cudaErrorInvalidValue ? e : launch_v<1, 8, 2, true>(p, false, clusters, s);
  }
  if (p.M <= 8) {
    p.mt = p.M;
    if (gv_split(16, 8, p.K / CH, p.n_units, clusters).cost <= gv_split(8, 8, p.K / CH, p.n_units, clusters).cost) {
      const cudaError_t e = p.M <= 2 ? launch_v<1, 16, 2, false, true>(p, true, clusters, s)
                                     : launch_v<1, 16, 2, false>(p, true, clusters, s);
      if (e != cudaErrorInvalidValue) return e;
    }
    return p.M <= 2 ? launch_v<1, 8, 3, false, true>(p, false, clusters, s)
                    : launch_v<1, 8, 3, false>(p, false, clusters, s);
  }
  p.mt = std::min(p.M, 16);
  return launch_v<2, 8, 2, false>(p, false, clusters, s);
}

}  // namespace osc
