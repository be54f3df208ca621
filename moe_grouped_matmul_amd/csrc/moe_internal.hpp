// Internal declarations of the mixture-of-experts operators: launchers that
// api_moe.cpp calls.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

// ---- products of microscaled 4-bit operands (mxfp4_gemm.hip)

// One launch: A [rows][K/2] (masked: [G][rows][K/2]) and B [G][N][K/2] e2m1
// codes, two to a byte; scale words [K/128][rows] and [K/128][N] (per group).
struct MxGemmParams {
  const uint8_t* A;
  const int32_t* sfa;
  const uint8_t* B;
  const int32_t* sfb;
  uint16_t* D;
  void* ws;              // dense, splits > 1: counters then fp32 partials
  const int32_t* index;  // m_indices (contiguous) or masked_m (masked)
  int64_t rows;          // M, M_total or max_m (of one launch)
  int64_t sfa_ld;        // words between consecutive 128s of A's scales: the caller's row count
  int N;
  int K;
  int G;
  int m_tiles;
  int n_tiles;
  int splits;
  int steps_per_split;  // K steps of 256
  bool stream_weights;  // weight loads carry the non-temporal policy
};

enum MxForm { kMxDense = 0, kMxContiguous = 1, kMxMasked = 2 };
// Tile shapes compiled (rows x columns).
enum MxTile { kMx64x64 = 0, kMx128x256 = 1, kMx256x256 = 2 };
constexpr int mx_bm(int tile) { return tile == kMx64x64 ? 64 : tile == kMx128x256 ? 128 : 256; }
constexpr int mx_bn(int tile) { return tile == kMx64x64 ? 64 : 256; }
constexpr int kMxMaxCounters = 1024;
constexpr size_t kMxCounterBytes = 4 * kMxMaxCounters;
// Workspace of a dense launch with splits > 1: one counter per tile, then the partials.
size_t mx_workspace_bytes(int tile, int m_tiles, int n_tiles, int splits);
// The persistent kernel of 256 x 256 and 128 x 256 tiles (mxfp4_wide.hip),
// dense or contiguous, over p.n_tiles column tiles with `grid` workgroups.  One
// contiguous launch has at most kMxWideMaxBlocks 128-row blocks.
constexpr int kMxWideMaxBlocks = 2048;
hipError_t launch_mxfp4_wide(int form, int grid, const MxGemmParams& p, hipStream_t stream);
hipError_t launch_mxfp4_gemm(int form, int tile, const MxGemmParams& p, hipStream_t stream);

// ---- quantiser (mxfp4_quant.hip)
hipError_t launch_quant_mxfp4(const void* x, bool bf16, uint8_t* q, int32_t* sf, const int32_t* row_token, int64_t G,
                              int64_t T, int64_t R, int64_t K, hipStream_t stream);
hipError_t launch_dequant_mxfp4(const uint8_t* q, const int32_t* sf, void* y, bool bf16, int64_t G, int64_t R,
                                int64_t K, hipStream_t stream);

// ---- gate (moe_gate.hip)
struct GateParams {
  const void* logits;    // [T][E]
  const uint8_t* valid;  // [T] or null
  int32_t* idx;          // [T][k]
  float* w;              // [T][k]
  int32_t* counts;       // [E + 1]
  float* prob_sum;       // [E]
  float* loss;           // [1]
  void* ws;
  int64_t T;
  int E;
  int k;
  int renorm;
  float w_scale;
  float coef;
};
struct GateBwdParams {
  const void* logits;
  const int32_t* idx;
  const float* w;
  const int32_t* counts;
  const float* dw;     // [T][k] or null
  const float* dloss;  // [1] or null
  void* dlogits;
  int64_t T;
  int E;
  int k;
  int renorm;
  float w_scale;
  float coef;
};
size_t gate_workspace_bytes(int64_t T, int64_t E);
hipError_t launch_gate(const GateParams& p, bool bf16, hipStream_t stream);
hipError_t launch_gate_bwd(const GateBwdParams& p, bool bf16, hipStream_t stream);

// ---- layout (moe_layout.hip)
struct LayoutParams {
  const int32_t* idx;  // [n] = [T][k]
  int32_t* counts;     // [G]
  int32_t* m_indices;  // [rows], contiguous only
  int32_t* row_token;  // [rows]
  int32_t* row_of;     // [n]
  void* ws;
  int64_t n;
  int k;
  int first;
  int G;
  int64_t max_m;  // 0: contiguous
  int64_t rows;
};
size_t layout_workspace_needed(int64_t n, int64_t G);
size_t layout_workspace_bytes(int64_t n, int64_t G);  // asked for: enough for up to n choices
hipError_t launch_layout(const LayoutParams& p, hipStream_t stream);

// ---- combine (moe_combine.hip)
hipError_t launch_combine(const uint16_t* rows, const int32_t* row_of, const float* w, void* y, bool bf16_y, int64_t T,
                          int64_t k, int64_t N, int64_t R, hipStream_t stream);
hipError_t launch_combine_bwd(const void* dy, bool bf16_y, const uint16_t* rows, const int32_t* row_of, const float* w,
                              uint16_t* drows, float* dw, int64_t T, int64_t k, int64_t N, int64_t R,
                              hipStream_t stream);

}  // namespace dg
