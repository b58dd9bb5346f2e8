// dg_launch.h - internal interface between the C-ABI layer (api.hip) and the kernel
// translation units. Host-side only; no HIP types beyond hipStream_t / hipError_t.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

// Which operand layout a GEMM launch serves.
enum class Layout : int { Dense = 0, Contiguous = 1, Masked = 2 };

// One GEMM problem as the kernels see it. For Dense, G = 1. For Contiguous, rows of a/d
// are M_total = M and b/sfb are [G,N,K] / [G,N/128,K/128]. For Masked, a/sfa/d hold G
// groups of M rows each (M = M_max).
struct GemmProblem {
  const uint8_t* a;
  const float* sfa;
  const uint8_t* b;
  const float* sfb;
  uint16_t* d;
  const int32_t* m_indices;  // Contiguous only
  const int32_t* masked_m;   // Masked only
  int64_t M, N, K;
  int32_t G;
  Layout layout;
  bool pow2;  // every sfa / sfb value is a power of two (UE8M0 scales)
};

// Kernel schedules. Decode: 64-row M blocks, K split across the waves of a workgroup,
// operands streamed straight into registers. Tile: LDS-staged, double-buffered tiles.
// Tile64 (chosen internally for dense M <= 64, never passed in through the C ABI): 64x128
// direct-load tiles.
enum class Schedule : int { Auto = 0, Decode = 1, Tile128 = 2, Tile256 = 3, Tile64 = 4 };

hipError_t launch_gemm(const GemmProblem& p, Schedule s, int64_t expected_m, hipStream_t stream,
                       const char** chosen);

// Gate/up GEMM with the SwiGLU + per-token FP8 cast epilogue: p.b holds 2I = p.N rows per
// group (gate rows, then up rows); writes hq [rows, I] e4m3 and sh [I/128][rows] (per group
// for the masked layout). hipErrorNotSupported (before any launch) when the shape is out of
// the kernel's range.
hipError_t launch_gemm_swiglu(const GemmProblem& p, uint8_t* hq, float* sh, int64_t expected_m, hipStream_t stream,
                              const char** chosen);

// Per-token cast of G groups of M rows; masked_m (or nullptr): only rows r < masked_m[g] of
// group g are cast, the others left unwritten.
hipError_t launch_cast_per_token(const void* x, int bf16, int pow2, int64_t G, int64_t M, int64_t K,
                                 const int32_t* masked_m, uint8_t* q, float* sf, hipStream_t stream);
// x [n] fp32 -> q [n] e4m3 with the hardware conversion (n % 4 == 0, n > 0).
hipError_t launch_convert_e4m3(const float* x, uint8_t* q, int64_t n, hipStream_t stream);
hipError_t launch_cast_per_block(const void* w, int bf16, int pow2, int64_t N, int64_t K, uint8_t* q, float* sf,
                                 hipStream_t stream);

// Compute units of the current device (cached per device; 256 on MI355X).
int cu_count();

// A launch holds fewer than 2^32 threads: workgroups of 256 past that go to further launches, each told
// the number of its first. Every piece but the last is a multiple of the 8 XCDs, so that a workgroup's
// number says which XCD it runs on as in one launch.
constexpr int64_t kPieceWorkgroups = (1 << 24) - 8;
template <typename Launch>
hipError_t launch_in_pieces(int64_t wgs, Launch launch) {
  for (int64_t wg0 = 0; wg0 < wgs; wg0 += kPieceWorkgroups) {
    launch(dim3((unsigned)(wgs - wg0 < kPieceWorkgroups ? wgs - wg0 : kPieceWorkgroups)), wg0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---- mixture-of-experts operators (moe.hip) ----
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 64;

struct RouteProblem {
  const void* logits;  // [T, E]
  const float* bias;   // [E] or nullptr (forward)
  int32_t* ids;        // [T, topk]: written forward, read backward
  float* weights;      // [T, topk] (forward)
  const float* dweights;  // [T, topk] (backward)
  void* dlogits;          // [T, E] (backward)
  int64_t T;
  int E, topk, groups, topk_groups, group_top;
  float scale;
  bool bf16, sigmoid, renormalise;
};
hipError_t launch_route(const RouteProblem& p, hipStream_t stream);
hipError_t launch_route_backward(const RouteProblem& p, hipStream_t stream);

struct LayoutProblem {
  const int32_t* ids;  // [pairs] expert of each (token, choice)
  int64_t pairs;
  int64_t rows;  // contiguous: M_total; masked: M_max
  int32_t G;
  bool masked;
  int32_t* pos;        // [pairs] row of each pair, or -1
  int32_t* row_pair;   // [rows] (masked [G, rows]) pair of each row, or -1
  int32_t* m_indices;  // [rows] (contiguous)
  int32_t* offsets;    // [G + 1] (contiguous)
  int32_t* masked_m;   // [G] (masked)
};
hipError_t launch_layout(const LayoutProblem& p, hipStream_t stream);

struct DispatchProblem {
  const void* x;  // [T, kblocks * 128]
  const int32_t* pos;       // [T, topk]
  const int32_t* row_pair;  // [groups, rows]
  uint8_t* q;
  float* sf;  // [groups, kblocks, rows]
  int64_t T, rows, groups;
  int topk, kblocks;
  bool masked;
};
hipError_t launch_dispatch(const DispatchProblem& p, int bf16, int pow2, hipStream_t stream);

struct CombineProblem {
  const uint16_t* y;  // [rows, H] bf16
  const int32_t* pos;  // [T, topk]
  const int32_t* row_pair;  // [rows] or nullptr (backward, contiguous layout)
  const float* weights;  // [T, topk] or nullptr: ones (forward)
  uint16_t* out;         // [T, H] (forward)
  const uint16_t* dout;  // [T, H] (backward)
  uint16_t* dy;          // [rows, H] (backward)
  float* dweights;       // [T, topk] (backward)
  int64_t T, rows, H;
  int topk;
};
hipError_t launch_combine(const CombineProblem& p, hipStream_t stream);
hipError_t launch_combine_backward(const CombineProblem& p, hipStream_t stream);

// ---- weight gradient (wgrad.hip) ----
struct ChannelCastProblem {
  const void* x;  // [M, K]
  const int32_t* row_pair;  // [M_out] or nullptr: row r of x itself
  const int32_t* used;      // device: rows in use (the layout's last offset), or nullptr: all
  uint8_t* q;  // [K, M_out]
  float* sf;   // [M_out / 128, K]
  int64_t M, K, M_out;
  int topk;
};
hipError_t launch_cast_per_channel(const ChannelCastProblem& p, int bf16, int pow2, hipStream_t stream);

struct WgradProblem {
  const uint8_t* a;  // [N, M]
  const float* sfa;  // [M / 128, N]
  const uint8_t* b;  // [K, M]
  const float* sfb;  // [M / 128, K]
  const int32_t* offsets;  // [G + 1] rows, multiples of 128, or nullptr: one group of all rows
  const void* c;  // [G, N, K] or nullptr
  void* d;        // [G, N, K]
  int64_t M, N, K;
  int32_t G;
  bool pow2;
  bool bf16;  // c and d are bf16, else fp32
  int splits;  // parts of every group's sum (set by the launcher)
};
// workspace: wgrad_workspace bytes for a split sum, or nullptr for none.
hipError_t launch_wgrad(const WgradProblem& p, float* workspace, hipStream_t stream, const char** chosen);
int64_t wgrad_workspace(int64_t G, int64_t M, int64_t N, int64_t K);

// The DG_* tuning switches (DG_TILE, DG_DECODE, DG_DECODE2, DG_DECODE3, DG_LOG) are read
// from the environment once per process; this reads them again.
void reload_tuning_switches();
// DG_LOG is set: every call names its chosen kernel on stderr.
bool log_switch();

}  // namespace dg
