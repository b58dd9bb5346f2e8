// dg_device.h - device helpers for the gfx950 kernels: e4m3 encoding, bf16 rounding,
// FP8 MFMA wrappers and operand vector types.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kQ = 128;  // scale granularity along K, and the weight block edge

// ---------------------------------------------------------------------------------
// fp32 -> OCP E4M3FN, round to nearest even, saturating at +-448, sign of zero kept.
// The format (bias 7, 3 mantissa bits, subnormals below 2^-6, max finite 448) is OCP
// E4M3FN, fixed by the 448 bound the DeepSeek-V3 repo review quotes ("Risks" 6).
// Normal range: round the fp32 pattern at mantissa bit 20 and rebias the exponent.
// Subnormal range (|y| < 2^-6): |y| * 512 is exact, and rint() rounds half to even.
// ---------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t e4m3_encode(float y) {
  uint32_t bits = __float_as_uint(y);
  uint32_t sign = (bits >> 24) & 0x80u;
  uint32_t mag = bits & 0x7FFFFFFFu;
  uint32_t code;
  if (mag >= 0x43E00000u) {          // |y| >= 448 (and inf): saturate
    code = 0x7Eu;
  } else if (mag < 0x3C800000u) {    // |y| < 2^-6
    code = (uint32_t)__builtin_rintf(__uint_as_float(mag) * 512.0f);
  } else {
    uint32_t r = (mag + 0x7FFFFu + ((mag >> 20) & 1u)) >> 20;
    code = r - (120u << 3);            // exponent bias 127 -> 7
    code = code > 0x7Eu ? 0x7Eu : code;
  }
  return sign | code;
}

// Four fp32 values -> four e4m3 codes (byte i = code of value i) with gfx950's conversion
// instruction (v_cvt_pk_fp8_f32: OCP E4M3FN, round to nearest even). It does not saturate:
// it agrees with e4m3_encode for |y| <= 464 (below the midpoint between 448 and 480 every
// value rounds to at most 448), which callers must guarantee.
__device__ __forceinline__ uint32_t e4m3_hw_pack4(float y0, float y1, float y2, float y3) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y0, y1, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y2, y3, (int)lo, true);
}

// The smallest power of two >= v (v >= 0), and >= 2^-126, from the fp32 bits: a normal v
// with a zero mantissa is a power of two already; otherwise the exponent goes up by one.
// This is the UE8M0 (power-of-two) scale of the casts. NaN, the largest value of a chunk of NaN alone, stays
// NaN, and so do the chunk's codes.
__device__ __forceinline__ float pow2_ceil(float v) {
  const uint32_t b = __float_as_uint(v);
  if (b > 0x7F800000u) return v;
  if (b < 0x00800000u) return __uint_as_float(0x00800000u);  // 0 and subnormals
  const uint32_t e = (b >> 23) + ((b & 0x007FFFFFu) ? 1u : 0u);
  return __uint_as_float(e << 23);
}

// fp32 -> bf16 bits, round to nearest even (inputs here are finite or NaN).
__device__ __forceinline__ uint32_t bf16_rne(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0u;
  u += 0x7FFFu + ((u >> 16) & 1u);
  return u >> 16;
}

__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }

// One 16x16x128 FP8 (e4m3 x e4m3) MFMA into a fresh fp32 partial. Operand lane layout:
// lane l supplies row (l & 15) of its 16-row strip and 32 K-bytes (group l >> 4); A and
// B pair byte-for-byte within a lane group, so any fixed split of the 128 K bytes over
// (group, byte) works if A and B use the same one. Output: lane l, element r holds row
// 4 * (l >> 4) + r, column l & 15.
__device__ __forceinline__ v4f mfma_f8_16x16x128(const v8i& a, const v8i& b) {
  v4f z = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}

// c + 2^(ea-127) * 2^(eb-127) * (A . B) on the matrix unit (block-scaled form): ea is the
// E8M0 scale this lane supplies for its A row (l & 15), eb the one for its B column; both
// in byte 0 of the operand. The scale covers the 32 K values of the lane's group, so a
// scale shared by a whole 128-K block is the same in every lane group.
__device__ __forceinline__ v4f mfma_f8_16x16x128_scaled(const v8i& a, const v8i& b, const v4f& c, int ea, int eb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, ea, 0, eb);
}

__device__ __forceinline__ v8i cat8(const v4i& lo, const v4i& hi) {
  v8i r;
  r[0] = lo[0]; r[1] = lo[1]; r[2] = lo[2]; r[3] = lo[3];
  r[4] = hi[0]; r[5] = hi[1]; r[6] = hi[2]; r[7] = hi[3];
  return r;
}

// Work-group index remap so that consecutively numbered logical tiles run on the same
// XCD (workgroups are dealt to the 8 XCDs round-robin; each XCD has its own L2).
__device__ __forceinline__ uint32_t xcd_remap(uint32_t hw_id, uint32_t nwg) {
  constexpr uint32_t kXcd = 8;
  uint32_t q = nwg / kXcd, r = nwg % kXcd;
  uint32_t x = hw_id % kXcd, i = hw_id / kXcd;
  return x * q + (x < r ? x : r) + i;
}

// Four consecutive values of an fp32 or bf16 tensor, from element `elem` (a multiple of 4).
template <bool kBf16>
__device__ __forceinline__ void load4(const void* base, int64_t elem, float v[4]) {
  if constexpr (kBf16) {
    uint2 raw = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + elem);
    v[0] = bf16_to_f32(raw.x & 0xFFFFu);
    v[1] = bf16_to_f32(raw.x >> 16);
    v[2] = bf16_to_f32(raw.y & 0xFFFFu);
    v[3] = bf16_to_f32(raw.y >> 16);
  } else {
    float4 raw = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
    v[0] = raw.x; v[1] = raw.y; v[2] = raw.z; v[3] = raw.w;
  }
}

// The codes of one chunk from its scale: q = e4m3(x / s) with the division correctly rounded
// and the hardware conversion, which equals the saturating encoder for every |x / s| <= 464
// (checked on every fp32 value). With s = fp32(amax / 448) >= amax / 448 * (1 - 2^-24), every
// quotient is at most 448.00003; power-of-two scales are >= amax / 448. s == 0 (an all-zero
// chunk, or amax / 448 underflowing) gives signed zeros.
__device__ __forceinline__ uint32_t quant4_hw(const float v[4], float s) {
  const uint32_t signs = ((__float_as_uint(v[0]) >> 31) << 7) | ((__float_as_uint(v[1]) >> 31) << 15) |
                         ((__float_as_uint(v[2]) >> 31) << 23) | ((__float_as_uint(v[3]) >> 31) << 31);
  const uint32_t codes = e4m3_hw_pack4(v[0] / s, v[1] / s, v[2] / s, v[3] / s);
  return s == 0.0f ? signs : codes;
}

// The quotient v / s correctly rounded, from r = RN(1 / s) by one correction step: q0 = RN(v r), the
// remainder v - s q0 is exact in an FMA, and q0 plus the remainder times r rounds to v / s unless the
// remainder underflows, which takes s < 2^-80, or s is not finite. Three operations where a division
// takes about ten. The remainder is taken as s q0 - v and subtracted: where it vanishes that adds -0, and the
// quotient -0 stays -0.
__device__ __forceinline__ float divide_by(float v, float s, float r) {
  const float q0 = v * r;
  return fmaf(-fmaf(q0, s, -v), r, q0);
}

// v / s may be taken from RN(1 / s): by divide_by, or (power-of-two scales) as the exact product. Not
// for the scales of chunks with an infinity, of NaN alone or of zeros.
template <bool kPow2>
__device__ __forceinline__ bool by_reciprocal(float s) {
  return s >= (kPow2 ? 0x1p-126f : 0x1p-80f) && s <= 0x1p120f;
}

// Sixteen codes of one chunk from its scale, as quant4_hw.
template <bool kPow2>
__device__ __forceinline__ v4i quant16(const float (&v)[16], float s) {
  v4i o;
  const float r = 1.0f / s;
  if (__all(by_reciprocal<kPow2>(s))) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = kPow2 ? v[4 * i + k] * r : divide_by(v[4 * i + k], s, r);
      o[i] = (int)e4m3_hw_pack4(q[0], q[1], q[2], q[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (int)quant4_hw(&v[4 * i], s);
  }
  return o;
}

// Workgroup barrier that orders LDS only: outstanding global loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Direct global->LDS loads (global_load_lds_dwordx4 / _dword: lane i of a wave writes
// bytes [16i, 16i+16) (or [4i, 4i+4)) after the LDS base held in M0). They are issued from
// inline assembly: they write only LDS and have no output registers; an address is a
// wave-uniform 64-bit base plus a per-lane 32-bit offset. Waits for them are explicit.
// M0 is listed as clobbered (the compiler warns that it cannot preserve a reserved register
// across the statement): in these kernels nothing else uses M0, every M0 write in the
// generated code being one of these, so there is nothing to preserve.
// Wave-uniform values in scalar registers; a no-op for values already there. The operands
// below must be uniform, and the compiler cannot always prove that they are.
__device__ __forceinline__ const void* uniform_ptr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const void*>(((uint64_t)hi << 32) | lo);
}
// kStream adds the non-temporal hint, for bytes that no other workgroup of the launch reads
// (the masked layout's expert weights: one tile streams each group's columns).
template <bool kStream = false>
__device__ __forceinline__ void lds_dma16(uint32_t voff, const void* sbase, uint32_t lds_base) {
  if constexpr (kStream)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(__builtin_amdgcn_readfirstlane(lds_base)),
                 "v"(voff), "s"(uniform_ptr(sbase))
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(lds_base)),
                 "v"(voff), "s"(uniform_ptr(sbase))
                 : "memory", "m0");
}
__device__ __forceinline__ void lds_dma4(uint32_t voff, const void* sbase, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(lds_base)),
               "v"(voff), "s"(uniform_ptr(sbase))
               : "memory", "m0");
}
// s_waitcnt with only the vector-memory counter constrained (gfx9 encoding)
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// Wait until at most n groups of P vector-memory loads are outstanding, for a runtime
// n (clamped to [0, MAXN]): s_waitcnt takes an immediate, so this unrolls to a chain.
template <int P, int MAXN>
__device__ __forceinline__ void wait_groups(int n) {
  if constexpr (MAXN <= 0) {
    wait_vmcnt<0>();
  } else {
    if (n >= MAXN) wait_vmcnt<MAXN * P>();
    else wait_groups<P, MAXN - 1>(n);
  }
}

}  // namespace dg
