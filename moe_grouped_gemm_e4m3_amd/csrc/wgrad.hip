// wgrad.hip - the FP8 weight gradient: the cast of activations per channel over blocks of 128
// tokens, and the grouped product that sums over an expert's tokens.
//
//   dW[g][n][k] = sum over the blocks j of 128 rows of expert g of
//                 (sum over the rows m of j of qa[n][m] qb[k][m]) * sfa[j][n] * sfb[j][k]
//
// Both operands are scaled per 1x128 along the rows they are summed over, so the scale of a
// partial product is a factor per output row times one per output column.
#include <math.h>

#include "dg_device.h"
#include "dg_launch.h"

namespace dg {
namespace {

// ---------------------------------------------------------------------------------
// per-channel cast
// ---------------------------------------------------------------------------------
// One workgroup per 128 rows x 64 channels: thread t reads 4 consecutive rows of 8 channels, the
// maxima of a channel meet in LDS, and the codes leave through LDS as runs of 128 rows of one
// channel (16-byte chunks XOR-swizzled by the channel's run of 8, which spreads the banks). Rows that
// hold no token (row_pair < 0) and rows past the input are zero; blocks past the rows in use are left
// alone. Bound by HBM: 2 or 4 bytes in, one out per element. In a call on 9088 rows of 7168 in bf16: 46 us,
// on 4001 of 18432: 53 us, 4.2 TB/s.
template <bool kBf16, bool kPow2>
__global__ __launch_bounds__(256) void cast_per_channel_kernel(ChannelCastProblem p, int64_t wg0) {
  __shared__ __attribute__((aligned(16))) float wave_amax[4][64], scale[64], reciprocal[64];
  __shared__ __attribute__((aligned(16))) uint8_t tile[64 * kQ];
  const uint32_t per_block = (uint32_t)(p.K / 64);  // workgroups per 128 rows
  const uint32_t wg = (uint32_t)wg0 + blockIdx.x;
  const int64_t blk = wg / per_block;
  const int64_t m0 = blk * kQ, k0 = (int64_t)(wg % per_block) * 64;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int c8 = t & 7, r4 = t >> 3;
  int64_t src[4];
  if (p.row_pair != nullptr) {
    const v4i pair = *reinterpret_cast<const v4i*>(p.row_pair + m0 + 4 * r4);
#pragma unroll
    for (int i = 0; i < 4; ++i) src[i] = pair[i] < 0 ? p.M : (int64_t)((uint32_t)pair[i] / (uint32_t)p.topk);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) src[i] = m0 + 4 * r4 + i;
  }
  if (p.used != nullptr && m0 >= *p.used) return;
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i][k] = 0.0f;
    if (src[i] < p.M) {
      load4<kBf16>(p.x, src[i] * p.K + k0 + 8 * c8, &v[i][0]);
      load4<kBf16>(p.x, src[i] * p.K + k0 + 8 * c8 + 4, &v[i][4]);
    }
  }
  float amax[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    amax[k] = fmaxf(fmaxf(fabsf(v[0][k]), fabsf(v[1][k])), fmaxf(fabsf(v[2][k]), fabsf(v[3][k])));
#pragma unroll
    for (int o = 8; o <= 32; o <<= 1) amax[k] = fmaxf(amax[k], __shfl_xor(amax[k], o, 64));
  }
  if (lane < 8) {
    *reinterpret_cast<float4*>(&wave_amax[w][8 * c8]) = make_float4(amax[0], amax[1], amax[2], amax[3]);
    *reinterpret_cast<float4*>(&wave_amax[w][8 * c8 + 4]) = make_float4(amax[4], amax[5], amax[6], amax[7]);
  }
  __syncthreads();
  if (t < 64) {
    const float a = fmaxf(fmaxf(wave_amax[0][t], wave_amax[1][t]), fmaxf(wave_amax[2][t], wave_amax[3][t]));
    const float s = kPow2 ? pow2_ceil(a / 448.0f) : a / 448.0f;
    scale[t] = s;
    reciprocal[t] = 1.0f / s;
    p.sf[blk * p.K + k0 + t] = s;
  }
  __syncthreads();
  float s[8], r[8];
  bool fast = true;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    s[k] = scale[8 * c8 + k];
    r[k] = reciprocal[8 * c8 + k];
    fast = fast && by_reciprocal<kPow2>(s[k]);
  }
  fast = __all(fast);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float col[4] = {v[0][k], v[1][k], v[2][k], v[3][k]};
    uint32_t codes;
    if (fast) {
      float q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = kPow2 ? col[i] * r[k] : divide_by(col[i], s[k], r[k]);
      codes = e4m3_hw_pack4(q[0], q[1], q[2], q[3]);
    } else {
      codes = quant4_hw(col, s[k]);
    }
    *reinterpret_cast<uint32_t*>(tile + (8 * c8 + k) * kQ + (((r4 >> 2) ^ c8) << 4) + (r4 & 3) * 4) = codes;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int piece = i * 256 + t, c = piece >> 3, part = piece & 7;
    *reinterpret_cast<v4i*>(p.q + (k0 + c) * p.M_out + m0 + part * 16) =
        *reinterpret_cast<const v4i*>(tile + c * kQ + ((part ^ (c >> 3)) << 4));
  }
}

// ---------------------------------------------------------------------------------
// grouped product
// ---------------------------------------------------------------------------------
// The offsets do not change while the kernel runs: scalar loads, which the waits for vector memory do
// not hold up.
__device__ __forceinline__ int group_block(const WgradProblem& p, int i) {
  typedef const __attribute__((address_space(4))) int32_t* constant_ptr;
  const int rows = ((constant_ptr)(uintptr_t)p.offsets)[__builtin_amdgcn_readfirstlane(i)];
  return __builtin_amdgcn_readfirstlane((rows < 0 ? 0 : rows > (int)p.M ? (int)p.M : rows) / kQ);
}

// BK x BN tiles of d^T (rows: channels k of b, columns: channels n of a), WM x WN waves of
// (BK / WM) x (BN / WN). The rows are the output's contiguous axis: a lane's four results of an
// MFMA are four neighbours in memory. Each block of 128 tokens of both operands and both scale
// vectors goes straight from global memory into one of two LDS stages (16-byte chunks XOR-swizzled
// by row). Per block a wave runs TM strips of 16 rows against its TN column fragments, which stay in
// registers; strips are read one (fp32) or two ahead of their MFMAs. Once the last strip is in registers
// the stage is free: its refill goes out one load to an MFMA over the strips left, as the loads of
// all waves at once keep the load path, and so the MFMAs behind them, busy for some 1000 cycles of a
// block's 3500 (bf16 results, 4096 x 7168 x 18432: 446 -> 421 us with power-of-two scales, 554 -> 528 with
// fp32, in a row of products alone).
//   kFp8 (bf16 results, fp32 scales): each MFMA starts from zero and its result is folded in with
//   acc = fma(P, sk * sn, acc): a product and an FMA per element and block, one strip behind the MFMAs.
//   kFp8Pow2 (bf16 results, power-of-two scales): the matrix unit applies them (lane l: row l & 15 of the
//   strip, column l & 15 of the fragment) and accumulates in its own fp32 registers.
//   kBf16 (fp32 results, both kinds of scales): the FP8 MFMAs align 8 neighbouring products and cut them 13
//   bits below the largest, some 1e-5 of a result, which bf16 (4e-3) hides and fp32 does not. e4m3 codes are
//   exact in bf16, and so is a product of two in fp32: the codes are widened in registers (two to an
//   instruction) and four bf16 MFMAs of 32 rows sum a block in fp32. Folded in as above, P * sk first: the
//   product of two scales may be past fp32 where the term is not.
// An expert has few blocks (1024 rows: 8), so a tile's start and end count as much as its loop. The
// workgroups are therefore persistent: each takes tiles slot, slot + grid, ..., and its loads run
// ahead from one tile into the next, so that the next tile's first blocks arrive while this one's
// results are written.
// Measured behind their casts, fp32 results: 8 experts of 1024 rows, 7168 x 2048, 332 us (470 MB of results);
// 32 of 256 rows, 4096 x 2048, added to c 588 us (4.5 TB/s: bound by c and d); one matrix of 4001 rows, 7168 x
// 18432, 1067 us (1.0 PFLOP/s; vector ALU 59 %, MFMA 44 % busy: two conversions and two operations of the fold
// to an MFMA). bf16 results: 137 us with power-of-two scales (1.8 PFLOP/s); 280 us; 564 us (1.9 PFLOP/s) and 443
// (2.4) with power-of-two scales, where the same instructions on zeros take a sixth less: the chip lowers its
// clock under the operands' switching.
// Two fp32 values as two bf16, round to nearest even (one instruction on gfx950).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// Strips x and y hold runs of channels 4 g and 16 + 4 g in the lanes of group g = lane >> 4. Afterwards
// group g holds the runs 8 g (x) and 8 g + 4 (y): the halves of the wave change places, then its rows
// of 16 lanes.
__device__ __forceinline__ uint2 swap_runs(uint32_t x, uint32_t y) {
  const auto half = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  const auto row = __builtin_amdgcn_permlane16_swap(half[0], half[1], false, false);
  return make_uint2(row[0], row[1]);
}

// A row's 32 codes of one lane group, widened: 8 of each of the four MFMAs that sum a block.
struct Wide {
  v8bf part[4];
};
template <bool kHigh>
__device__ __forceinline__ v2bf widen2(int codes) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, kHigh);
}
__device__ __forceinline__ Wide widen(const v8i& codes) {
  Wide r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const v2bf x = widen2<false>(codes[2 * i]), y = widen2<true>(codes[2 * i]);
    const v2bf z = widen2<false>(codes[2 * i + 1]), w = widen2<true>(codes[2 * i + 1]);
    r.part[i] = v8bf{x[0], x[1], y[0], y[1], z[0], z[1], w[0], w[1]};
  }
  return r;
}
// The sum over a block of 128 rows: of codes as they are, or widened.
__device__ __forceinline__ v4f block_product(const v8i& a, const v8i& b) { return mfma_f8_16x16x128(a, b); }
__device__ __forceinline__ v4f block_product(const Wide& a, const Wide& b) {
  v4f sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[i], b.part[i], sum, 0, 0, 0);
  return sum;
}

enum : int { kOutBf16, kOutBf16Add, kOutF32, kOutF32Add };  // type of d; with c added
enum : int { kFp8, kFp8Pow2, kBf16 };                       // products

template <int BK, int BN, int WM, int WN, int kProducts, int kOut, bool kSplit = false>
__global__ __launch_bounds__(64 * WM * WN) void wgrad_kernel(WgradProblem p) {
  constexpr bool kPow2 = kProducts == kFp8Pow2;
  constexpr int NW = WM * WN;
  constexpr int WTM = BK / WM, WTN = BN / WN, TM = WTM / 16, TN = WTN / 16;
  constexpr int ADMA = BK * 8 / (64 * NW), BDMA = BN * 8 / (64 * NW);  // 1 KB direct loads per wave and block
  constexpr int PER_STAGE = ADMA + BDMA + 1;                           // and 64 scales
  constexpr int STAGE_BYTES = (BK + BN) * (kQ + 4);
  constexpr int STORES16 = TM / 2 * TN;  // store instructions of a whole bf16 tile per wave
  static_assert(ADMA * 64 * NW == BK * 8 && BDMA * 64 * NW == BN * 8 && BK + BN == 64 * NW, "direct-load split");
  static_assert(TM >= 2 && TM % 2 == 0, "strip slots alternate and repeat every block");
  static_assert(2 * STAGE_BYTES <= 160 * 1024 && STORES16 < 64, "LDS ring, vmcnt");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * STAGE_BYTES];

  const int t = threadIdx.x, l = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = w % WM, wn = w / WM;
  const int fr = l & 15, g4 = l >> 4;

  // groups in order; in a group, bands of 8 column tiles walked row tile by row tile: the workgroups
  // of one XCD take neighbouring tiles
  const int tiles_k = (int)((p.K + BK - 1) / BK), tiles_n = (int)((p.N + BN - 1) / BN);
  const int per_group = tiles_k * tiles_n;
  const int64_t tiles = (int64_t)per_group * p.G * (kSplit ? p.splits : 1);
  const int64_t slot = xcd_remap(blockIdx.x, gridDim.x);
  struct Tile {
    int g, first, blocks;
    int64_t n0, k0;
  };
  auto tile_at = [&](int64_t at) {
    Tile q;
    q.g = (int)(at / per_group);
    const int rem = (int)(at % per_group);
    constexpr int GM = 8;
    const int band = rem / (GM * tiles_k), in = rem % (GM * tiles_k);
    const int gm = min(tiles_n - band * GM, GM);
    q.n0 = (int64_t)(band * GM + in % gm) * BN;
    q.k0 = (int64_t)(in / gm) * BK;
    const int g = kSplit ? q.g / p.splits : q.g;  // split: every part of a group is an output of its own
    q.first = p.offsets ? group_block(p, g) : 0;
    q.blocks = (p.offsets ? group_block(p, g + 1) : (int)(p.M / kQ)) - q.first;
    if constexpr (kSplit) {
      const int part = q.g % p.splits, all = max(q.blocks, 0);
      const int lo = (int)((int64_t)all * part / p.splits);
      q.blocks = (int)((int64_t)all * (part + 1) / p.splits) - lo;
      q.first += lo;
    }
    return q;
  };

  // ---- the stream of loads: every block of this workgroup's tiles in order ----
  // A wave's direct load u covers 8 rows, 64 rows (NW = 8; 32 for NW = 4) after load u - 1; lanes
  // differ by one offset. Loads past the last channel (a tile over the edge, K or N an odd multiple of
  // 128) repeat the tile's first rows.
  constexpr int URUN = NW * 8;
  int64_t next_tile = slot;
  int ahead_blk = 0, ahead_blocks = 0;
  const uint8_t *A = nullptr, *B = nullptr;
  const float* S = nullptr;
  const int64_t urun = URUN * p.M;
  int64_t ka[ADMA], na[BDMA];  // bytes from the tile's first row to load u's
  const uint32_t voff = (uint32_t)((w * 8 + (l >> 3)) * p.M) + (uint32_t)(((l & 7) ^ ((l >> 3) & 7)) << 4);
  const uint32_t soff = (uint32_t)l * 4;
  const bool row_scales = w * 64 < BK;  // wave w carries the scales of 64 channels, the rows' first
  const int64_t sstep = row_scales ? p.K : p.N;
  const uint32_t base = (uint32_t)(uintptr_t)smem;
  // the next block of the stream; false past the last one, where the latest block stays
  auto advance = [&] {
    if (ahead_blk < ahead_blocks) {
      A += kQ;
      B += kQ;
      S += sstep;
      ++ahead_blk;
      return true;
    }
    while (true) {
      if (next_tile >= tiles) return false;
      const Tile q = tile_at(next_tile);
      next_tile += gridDim.x;
      if (q.blocks <= 0) continue;
      ahead_blk = 1;
      ahead_blocks = q.blocks;
      A = p.b + q.k0 * p.M + (int64_t)q.first * kQ;
      B = p.a + q.n0 * p.M + (int64_t)q.first * kQ;
      const int rows_k = (int)(p.K - q.k0 < BK ? p.K - q.k0 : BK), rows_n = (int)(p.N - q.n0 < BN ? p.N - q.n0 : BN);
#pragma unroll
      for (int u = 0; u < ADMA; ++u) ka[u] = u * URUN < rows_k ? u * urun : 0;
#pragma unroll
      for (int u = 0; u < BDMA; ++u) na[u] = u * URUN < rows_n ? u * urun : 0;
      const int ch = w * 64 - (row_scales ? 0 : BK), most = row_scales ? rows_k : rows_n;
      S = (row_scales ? p.sfb + (int64_t)q.first * p.K + q.k0 : p.sfa + (int64_t)q.first * p.N + q.n0) + (ch < most ? ch : 0);
      return true;
    }
  };
  auto load = [&](int stage, int u) {
    const uint32_t sbase = base + (uint32_t)(stage * STAGE_BYTES);
    if (u < ADMA) lds_dma16(voff, A + ka[u < ADMA ? u : 0], sbase + (uint32_t)((u * NW + w) * 1024));
    else if (u < ADMA + BDMA)
      lds_dma16(voff, B + na[u < ADMA + BDMA && u >= ADMA ? u - ADMA : 0], sbase + (uint32_t)(BK * kQ + ((u - ADMA) * NW + w) * 1024));
    else lds_dma4(soff, S, sbase + (uint32_t)((BK + BN) * kQ + w * 256));
  };
  auto issue = [&](int stage) {
    if (!advance()) return false;
#pragma unroll
    for (int u = 0; u < PER_STAGE; ++u) load(stage, u);
    return true;
  };
  // Before a block's last strips: the next block's loads have landed, and this block's stage is read.
  // The store instructions issued since those loads may stay in flight (the counter falls in order).
  // After results with c added there is nothing to wait for: c was loaded after those loads, and used.
  enum { kWaitAll, kWaitBehindStores, kLanded };
  int state = kWaitAll;
  auto landed = [&] {
    if (state == kWaitAll) wait_vmcnt<0>();
    else if (state == kWaitBehindStores) wait_vmcnt<STORES16>();
    state = kWaitAll;
    // the reads of the stage to be refilled are done: the barrier alone does not wait for them, and loads
    // that hit the L1 could overtake them
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    lds_barrier();
  };

  const uint32_t sw0 = (uint32_t)((g4 ^ (fr & 7)) << 4), sw1 = (uint32_t)(((g4 + 4) ^ (fr & 7)) << 4);
  const uint32_t a_lane = (uint32_t)((wm * WTM + fr) * kQ);
  const uint32_t b_lane = (uint32_t)(BK * kQ + (wn * WTN + fr) * kQ);
  const uint32_t sk_lane = (uint32_t)((BK + BN) * kQ + (wm * WTM + (kPow2 ? fr : 4 * g4)) * 4);
  const uint32_t sn_lane = (uint32_t)((BK + BN) * kQ + (BK + wn * WTN + fr) * 4);
  auto read_b = [&](v8i& bf, float& sn, int stage, int j) {
    const uint8_t* st = smem + stage * STAGE_BYTES;
    bf = cat8(*reinterpret_cast<const v4i*>(st + b_lane + j * 16 * kQ + sw0),
              *reinterpret_cast<const v4i*>(st + b_lane + j * 16 * kQ + sw1));
    sn = *reinterpret_cast<const float*>(st + sn_lane + 64 * j);
  };
  auto read_a = [&](v8i& af, int stage, int i) {
    const uint8_t* st = smem + stage * STAGE_BYTES;
    af = cat8(*reinterpret_cast<const v4i*>(st + a_lane + i * 16 * kQ + sw0),
              *reinterpret_cast<const v4i*>(st + a_lane + i * 16 * kQ + sw1));
  };
  // fp32: the scales of this lane's four result rows of a strip
  auto read_s = [&](float4& sk, int stage, int i) {
    sk = *reinterpret_cast<const float4*>(smem + stage * STAGE_BYTES + sk_lane + 64 * i);
  };

  if (issue(0)) {
    if (issue(1)) wait_vmcnt<PER_STAGE>();
    else wait_vmcnt<0>();
    lds_barrier();
  }
  int st = 0;
  for (int64_t at = slot; at < tiles; at += gridDim.x) {
    const Tile q = tile_at(at);
    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    // the first block's fragments (read here, not with the block before: they would hold registers
    // while the results are written)
    v8i bf[TN], a0;
    float sn[TN];
    float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (q.blocks > 0) {
#pragma unroll
      for (int j = 0; j < TN; ++j) read_b(bf[j], sn[j], st, j);
      read_a(a0, st, 0);
      if constexpr (!kPow2) read_s(s0, st, 0);
    }
    if constexpr (kPow2) {
      float sk[TM];  // scales of this lane's row of every strip
      auto read_sk = [&](int stage) {
#pragma unroll
        for (int i = 0; i < TM; ++i) sk[i] = *reinterpret_cast<const float*>(smem + stage * STAGE_BYTES + sk_lane + 64 * i);
      };
      if (q.blocks > 0) read_sk(st);
      for (int blk = 0; blk < q.blocks; ++blk) {
        v8i af[3] = {a0, a0, a0};
        int ek[TM], en[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) ek[i] = (int)(__float_as_uint(sk[i]) >> 23);
#pragma unroll
        for (int j = 0; j < TN; ++j) en[j] = (int)(__float_as_uint(sn[j]) >> 23);
        auto strip = [&](int i) {
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = mfma_f8_16x16x128_scaled(af[i % 3], bf[j], acc[i][j], ek[i], en[j]);
        };
        read_a(af[1], st, 1);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
        for (int i = 0; i < TM - 3; ++i) {
          if (i + 2 < TM) read_a(af[(i + 2) % 3], st, i + 2);  // two strips ahead
          strip(i);
          // the reads between the MFMAs that they are written beside: the compiler would put each right
          // before its use
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (i + 2 < TM && j < 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          }
        }
        read_a(af[(TM - 1) % 3], st, TM - 1);
        // keep the strips' MFMAs before the refill: the compiler would sink them behind its branches,
        // with every strip's fragments in registers until then
#pragma unroll
        for (int i = 0; i < TM - 3; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(acc[i][j]));
        __builtin_amdgcn_sched_barrier(0);
        (void)advance();
        landed();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 2 * TN; ++m) {
          const int i = TM - 3 + m / TN, j = m % TN;
          if (m < PER_STAGE) load(st, m);
          acc[i][j] = mfma_f8_16x16x128_scaled(af[i % 3], bf[j], acc[i][j], ek[i], en[j]);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int u = 2 * TN; u < PER_STAGE; ++u) load(st, u);
        read_a(a0, st ^ 1, 0);  // after a tile's last block: not used
        strip(TM - 1);
#pragma unroll
        for (int j = 0; j < TN; ++j) read_b(bf[j], sn[j], st ^ 1, j);
        read_sk(st ^ 1);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
        }
        st ^= 1;
      }
    } else {
      // products and factors of the two latest strips; the first promotion adds 0 * 0
      v4f pp[2][TN];
      float4 tk[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
      float tn[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        pp[0][j] = pp[1][j] = v4f{0.f, 0.f, 0.f, 0.f};
        tn[j] = 0.0f;
      }
      auto promote1 = [&](int s, int i, int j) {
        const float4 s4 = tk[s];
        if constexpr (kProducts == kBf16) {
          acc[i][j][0] = fmaf(pp[s][j][0] * s4.x, tn[j], acc[i][j][0]);
          acc[i][j][1] = fmaf(pp[s][j][1] * s4.y, tn[j], acc[i][j][1]);
          acc[i][j][2] = fmaf(pp[s][j][2] * s4.z, tn[j], acc[i][j][2]);
          acc[i][j][3] = fmaf(pp[s][j][3] * s4.w, tn[j], acc[i][j][3]);
        } else {
          acc[i][j][0] = fmaf(pp[s][j][0], s4.x * tn[j], acc[i][j][0]);
          acc[i][j][1] = fmaf(pp[s][j][1], s4.y * tn[j], acc[i][j][1]);
          acc[i][j][2] = fmaf(pp[s][j][2], s4.z * tn[j], acc[i][j][2]);
          acc[i][j][3] = fmaf(pp[s][j][3], s4.w * tn[j], acc[i][j][3]);
        }
      };
      auto operand = [&](const v8i& codes) {
        if constexpr (kProducts == kBf16) return widen(codes);
        else return codes;
      };
      auto promote = [&](int s, int i) {
#pragma unroll
        for (int j = 0; j < TN; ++j) promote1(s, i, j);
        // keep the promotion between the MFMAs that it was written between
#pragma unroll
        for (int j = 0; j < TN; ++j) asm volatile("" ::"v"(acc[i][j]));
      };
      for (int blk = 0; blk < q.blocks; ++blk) {
        v8i af[2] = {a0, a0};
        float4 sk[2] = {s0, s0};
        decltype(operand(a0)) wb[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) wb[j] = operand(bf[j]);
#pragma unroll
        for (int i = 0; i < TM - 2; ++i) {
          const int c = i & 1;
          read_a(af[c ^ 1], st, i + 1);
          read_s(sk[c ^ 1], st, i + 1);
          const auto wa = operand(af[c]);
#pragma unroll
          for (int j = 0; j < TN; ++j) pp[c][j] = block_product(wa, wb[j]);
          promote(c ^ 1, i == 0 ? TM - 1 : i - 1);  // strip 0: the previous block's last
          tk[c] = sk[c];
          if (i == 0)
#pragma unroll
            for (int j = 0; j < TN; ++j) tn[j] = sn[j];
          if constexpr (kProducts == kBf16) {
            // 16 MFMAs beside 16 conversions and 32 operations of a promotion; the first strip's with b's 64
#pragma unroll
            for (int m = 0; m < 4 * TN; ++m) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              if (i == 0) __builtin_amdgcn_sched_group_barrier(0x002, 7, 0);
              else __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
            }
          } else {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
            }
          }
        }
        read_a(af[1], st, TM - 1);
        read_s(sk[1], st, TM - 1);
        const auto w0 = operand(af[0]);
        __builtin_amdgcn_sched_barrier(0);
        (void)advance();
        landed();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          load(st, j);
          pp[0][j] = block_product(w0, wb[j]);
          promote1(1, TM - 3, j);
          __builtin_amdgcn_sched_barrier(0);
        }
        tk[0] = sk[0];
        read_a(a0, st ^ 1, 0);
        read_s(s0, st ^ 1, 0);
        const auto w1 = operand(af[1]);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          load(st, TN + j);
          pp[1][j] = block_product(w1, wb[j]);
          promote1(0, TM - 2, j);
          read_b(bf[j], sn[j], st ^ 1, j);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int u = 2 * TN; u < PER_STAGE; ++u) load(st, u);
        tk[1] = sk[1];
        st ^= 1;
      }
      promote(1, TM - 1);
    }

    // Results: lane (g4, fr) holds 4 neighbouring channels k, 16 i + 4 g4, of channel n = fr of its
    // fragment. For bf16, two lane swaps over a pair of strips give it 8 neighbours, 32 (i / 2) + 8 g4,
    // so that an instruction moves 16 bytes a lane and 64 contiguous ones a channel (32-byte pieces
    // straight from the MFMA layout took 1.7 times as long per byte).
    // One offset per lane; the rest of an address is the same throughout the wave. K and N are
    // multiples of 128, so a wave's part of a tile over the edge is inside the matrix or outside.
    static_assert(128 % WTM == 0 && 128 % WTN == 0, "a wave's part of a tile is whole or empty");
    const int64_t kw = q.k0 + wm * WTM, nw = q.n0 + wn * WTN;
    if (kw >= p.K || nw >= p.N) continue;
    const int64_t at0 = ((int64_t)q.g * p.N + nw) * p.K + kw;
    const int64_t step = 16 * p.K;
    if constexpr (kOut == kOutF32) {
      const uint32_t lane_at = (uint32_t)(fr * p.K) + 4 * g4;
      float* d = static_cast<float*>(p.d) + at0;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int i = 0; i < TM; ++i) *reinterpret_cast<v4f*>(d + 16 * i + lane_at) = acc[i][j];
        d += step;
      }
    } else if constexpr (kOut == kOutF32Add) {
      const uint32_t lane_at = (uint32_t)(fr * p.K) + 4 * g4;
      float* d = static_cast<float*>(p.d) + at0;
      const float* c = static_cast<const float*>(p.c) + at0;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        v4f cr[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) cr[i] = *reinterpret_cast<const v4f*>(c + 16 * i + lane_at);
#pragma unroll
        for (int i = 0; i < TM; ++i) *reinterpret_cast<v4f*>(d + 16 * i + lane_at) = acc[i][j] + cr[i];
        d += step;
        c += step;
      }
    } else {
      const uint32_t lane_at = (uint32_t)(fr * p.K) + 8 * g4;
      uint16_t* d = static_cast<uint16_t*>(p.d) + at0;
      const uint16_t* c = static_cast<const uint16_t*>(p.c) + at0;
      // c two column fragments ahead, in the registers that the operands' fragments no longer need
      v4i cr[2][TM / 2];
      auto load_c = [&](int j) {
        if constexpr (kOut == kOutBf16Add) {
#pragma unroll
          for (int i2 = 0; i2 < TM / 2; ++i2) cr[j & 1][i2] = *reinterpret_cast<const v4i*>(c + 32 * i2 + lane_at);
          c += step;
        }
      };
      load_c(0);
      load_c(1);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        v4i cj[TM / 2];
#pragma unroll
        for (int i2 = 0; i2 < TM / 2; ++i2) cj[i2] = cr[j & 1][i2];
        if (j + 2 < TN) load_c(j + 2);
#pragma unroll
        for (int i2 = 0; i2 < TM / 2; ++i2) {
          v4i o;
          if constexpr (kOut == kOutBf16Add) {
            float v[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint2 run = swap_runs(__float_as_uint(acc[2 * i2][j][r]), __float_as_uint(acc[2 * i2 + 1][j][r]));
              v[r] = __uint_as_float(run.x);
              v[4 + r] = __uint_as_float(run.y);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
              o[r] = (int)pack_bf16(v[2 * r] + bf16_to_f32((uint32_t)cj[i2][r] & 0xFFFFu),
                                    v[2 * r + 1] + bf16_to_f32((uint32_t)cj[i2][r] >> 16));
          } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint2 run = swap_runs(pack_bf16(acc[2 * i2][j][2 * r], acc[2 * i2][j][2 * r + 1]),
                                          pack_bf16(acc[2 * i2 + 1][j][2 * r], acc[2 * i2 + 1][j][2 * r + 1]));
              o[r] = (int)run.x;
              o[2 + r] = (int)run.y;
            }
          }
          *reinterpret_cast<v4i*>(d + 32 * i2 + lane_at) = o;
        }
        d += step;
      }
    }
    if constexpr (kOut == kOutBf16Add || kOut == kOutF32Add) state = kLanded;
    // exactly STORES16 store instructions, and nothing else, since the latest loads?
    if constexpr (kOut == kOutBf16) state = q.blocks > 0 ? kWaitBehindStores : kWaitAll;
  }
  wait_vmcnt<0>();  // past the last block the latest one was loaded again
}

// The launch of persistent workgroups, at most `grid` of them.
template <int BK, int BN, int WM, int WN>
dim3 wgrad_grid(const WgradProblem& p, int64_t grid) {
  const int64_t tiles = ((p.K + BK - 1) / BK) * ((p.N + BN - 1) / BN) * p.G;
  return dim3((unsigned)(tiles < grid ? tiles : grid));
}

template <int BK, int BN, int WM, int WN>
hipError_t run_wgrad_bf16(const WgradProblem& p, int64_t grid, hipStream_t stream) {
  const dim3 wgs = wgrad_grid<BK, BN, WM, WN>(p, grid), block(64 * WM * WN);
  switch ((p.c != nullptr ? 1 : 0) + (p.pow2 ? 2 : 0)) {
    case 0: wgrad_kernel<BK, BN, WM, WN, kFp8, kOutBf16><<<wgs, block, 0, stream>>>(p); break;
    case 1: wgrad_kernel<BK, BN, WM, WN, kFp8, kOutBf16Add><<<wgs, block, 0, stream>>>(p); break;
    case 2: wgrad_kernel<BK, BN, WM, WN, kFp8Pow2, kOutBf16><<<wgs, block, 0, stream>>>(p); break;
    default: wgrad_kernel<BK, BN, WM, WN, kFp8Pow2, kOutBf16Add><<<wgs, block, 0, stream>>>(p); break;
  }
  return hipGetLastError();
}

// 128 x 128 tiles alone: a wave of a 256 x 256 one would need some 40 registers more than it has, for the
// widened fragments beside 128 sums.
hipError_t run_wgrad_f32(const WgradProblem& p, int64_t grid, hipStream_t stream) {
  const dim3 wgs = wgrad_grid<128, 128, 2, 2>(p, grid), block(256);
  if (p.c != nullptr) wgrad_kernel<128, 128, 2, 2, kBf16, kOutF32Add><<<wgs, block, 0, stream>>>(p);
  else wgrad_kernel<128, 128, 2, 2, kBf16, kOutF32><<<wgs, block, 0, stream>>>(p);
  return hipGetLastError();
}

// d = c + the parts of a split sum, in their order; 4 values a thread.
template <bool kBf16>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ parts, WgradProblem p) {
  const int64_t per = p.N * p.K, all = per * p.G;
  for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; e < all; e += (int64_t)gridDim.x * 1024) {
    const int64_t g = e / per;
    const float* src = parts + g * p.splits * per + (e - g * per);
    v4f v = *reinterpret_cast<const v4f*>(src);
    for (int s = 1; s < p.splits; ++s) v += *reinterpret_cast<const v4f*>(src + s * per);
    if (p.c != nullptr) {
      float c[4];
      load4<kBf16>(p.c, e, c);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += c[i];
    }
    if constexpr (kBf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.d) + e) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    else
      *reinterpret_cast<v4f*>(static_cast<float*>(p.d) + e) = v;
  }
}

// Parts that a group's blocks are split into where the 128 x 128 tiles do not fill the chip. A block of a
// tile takes about 0.75 us (FP8 products; widened ones 1.2); a part writes its sums in fp32 and the join reads them, at about 3 TB/s, and
// the join's launch costs some 4 us: the number of parts that makes the sum of these least, if that
// is a tenth less than no parts. Measured, parts against none, fp32 (bf16) results: 256 x 256 over 8192 rows 17.1
// against 76.6 us (15.1, 47.7), 1024 x 1024 33.3 against 78.0 (25.3, 48.3), 512 x 512 over 2048 rows 14.6 against
// 23.2 (12.6, 15.3); no parts are taken for 1024 x 1024 over 2048 rows (23.7 us; bf16 15.5, and 20.2 in 4 parts).
int wgrad_splits(int64_t G, int64_t M, int64_t N, int64_t K) {
  if (G < 1) return 1;
  const int64_t slots = 2 * (int64_t)cu_count(), tiles = (N / 128) * (K / 128) * G, blocks = M / kQ / G;
  if (tiles < 1 || 2 * tiles > slots) return 1;
  const double product = 0.75 * (double)blocks, part = (double)(G * N * K) * 8 / 3e6;  // us
  int64_t s = (int64_t)(sqrt(product / part) + 0.5);
  for (const int64_t most : {slots / tiles, blocks / 4, (int64_t)16})
    if (s > most) s = most;
  if (s < 2 || product / (double)s + part * (double)s + 4 > 0.9 * product) return 1;
  return (int)s;
}

hipError_t run_wgrad_split(const WgradProblem& p, hipStream_t stream) {
  const int64_t tiles = (p.K / 128) * (p.N / 128) * p.G * p.splits, most = 2 * (int64_t)cu_count();
  const dim3 wgs((unsigned)(tiles < most ? tiles : most)), block(256);
  if (!p.bf16) wgrad_kernel<128, 128, 2, 2, kBf16, kOutF32, true><<<wgs, block, 0, stream>>>(p);
  else if (p.pow2) wgrad_kernel<128, 128, 2, 2, kFp8Pow2, kOutF32, true><<<wgs, block, 0, stream>>>(p);
  else wgrad_kernel<128, 128, 2, 2, kFp8, kOutF32, true><<<wgs, block, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

int64_t wgrad_workspace(int64_t G, int64_t M, int64_t N, int64_t K) {
  const int s = wgrad_splits(G, M, N, K);
  return s > 1 ? s * G * N * K * 4 : 0;
}

hipError_t launch_cast_per_channel(const ChannelCastProblem& p, int bf16, int pow2, hipStream_t stream) {
  const int64_t wgs = (p.K / 64) * (p.M_out / kQ);
  if (wgs > 0x7FFFFFFF) return hipErrorInvalidValue;  // 16 TB of codes
  return launch_in_pieces(wgs, [&](dim3 grid, int64_t wg0) {
    const dim3 block(256);
    if (bf16 && pow2) cast_per_channel_kernel<true, true><<<grid, block, 0, stream>>>(p, wg0);
    else if (bf16) cast_per_channel_kernel<true, false><<<grid, block, 0, stream>>>(p, wg0);
    else if (pow2) cast_per_channel_kernel<false, true><<<grid, block, 0, stream>>>(p, wg0);
    else cast_per_channel_kernel<false, false><<<grid, block, 0, stream>>>(p, wg0);
  });
}

hipError_t launch_wgrad(const WgradProblem& problem, float* workspace, hipStream_t stream, const char** chosen) {
  WgradProblem p = problem;
  p.splits = workspace != nullptr ? wgrad_splits(p.G, p.M, p.N, p.K) : 1;
  if (p.splits > 1) {
    *chosen = p.bf16 ? "wgrad_128x128_split" : "wgrad_f32_128x128_split";
    WgradProblem part = p;
    part.c = nullptr;
    part.d = workspace;
    const hipError_t e = run_wgrad_split(part, stream);
    if (e != hipSuccess) return e;
    int64_t wgs = (p.N * p.K * p.G / 4 + 255) / 256;
    if (wgs > 2048) wgs = 2048;
    if (p.bf16) join_kernel<true><<<dim3((unsigned)wgs), dim3(256), 0, stream>>>(workspace, p);
    else join_kernel<false><<<dim3((unsigned)wgs), dim3(256), 0, stream>>>(workspace, p);
    return hipGetLastError();
  }
  const int64_t cus = cu_count();
  if (!p.bf16) {
    *chosen = "wgrad_f32_128x128";
    return run_wgrad_f32(p, 2 * cus, stream);
  }
  // 256 x 256 tiles, one workgroup per CU, or 128 x 128 ones, two: whichever takes less time in
  // rounds, a round of two small tiles worth 0.59 of a large one's (half the products at 0.82 to 0.86 of
  // the rate, measured on 4096 x 7168 x 18432: 528 against 644 us, and on 32 experts of 256 rows, 4096 x 2048
  // added to c: 276 against 319 us). Few tiles go to more CUs as small ones (4 experts, 256 x 384,
  // 301 x 2 rows: 7.7 against 14.2 us).
  const int64_t large = ((p.K + 255) / 256) * ((p.N + 255) / 256) * p.G, small = (p.K / 128) * (p.N / 128) * p.G;
  if (100 * ((large + cus - 1) / cus) <= 59 * ((small + 2 * cus - 1) / (2 * cus))) {
    *chosen = "wgrad_256x256";
    return run_wgrad_bf16<256, 256, 2, 4>(p, cus, stream);
  }
  *chosen = "wgrad_128x128";
  return run_wgrad_bf16<128, 128, 2, 2>(p, 2 * cus, stream);
}

}  // namespace dg
