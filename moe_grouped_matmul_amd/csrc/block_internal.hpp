// Internal declarations of the operators that join the products of a block
// (norm, gradient of an epilogue, experts for a few tokens): launchers that
// api_block.cpp calls.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

constexpr size_t kBlockWsCounterBytes = 4096;  // a workspace's counters, zero between calls

// ---- root-mean-square norm (rms_norm.hip)
constexpr int kNormMaxK = 16384;
enum ScaleKind { kNoQuant = 0, kScaleF32 = 1, kScaleUe8m0 = 2 };
struct NormParams {
  const void* x;         // [M][K]
  const void* residual;  // [M][K] or null
  const void* weight;    // [K], of x's type or fp32
  void* h;               // [M][K] or null
  void* y;               // [M][K] or null
  uint8_t* q;            // [M][K] or null
  void* sf;
  float* rstd;           // [M] or null
  int64_t M;
  int K;
  bool weight_bf16;
  float eps;
};
struct NormBwdParams {
  const void* dy;
  const void* h;
  const void* weight;
  const float* rstd;
  const void* dh;   // or null
  void* dx;
  float* dw;        // [K]
  float* partials;  // [norm_bwd_grid()][K]
  int64_t M;
  int K;
  bool weight_bf16;
};
hipError_t launch_rms_norm(const NormParams& p, bool bf16, int kind, int cus, hipStream_t stream);
int norm_bwd_grid(int64_t M, int64_t K, int cus);
hipError_t launch_rms_norm_bwd(const NormBwdParams& p, bool bf16, int cus, hipStream_t stream);
// out[c] = sum over r of partials[r][c] (rows in order within each of 16 slices, then the slices)
hipError_t launch_column_sum(const float* partials, float* out, int64_t rows, int N, hipStream_t stream);


// ---- gradient of a product's epilogue (epilogue_bwd.hip)
struct EpilogueBwdParams {
  const uint16_t* dy;   // [M][N]
  const uint16_t* pre;  // [M][N], unused without an activation
  uint16_t* dz;         // [M][N] or null
  uint8_t* q;           // [M][N] or null
  float* sf;            // [N/128][M]
  float* dbias;         // [N]
  float* partials;      // [ceil(M / rows_per_wg)][N], null without dbias
  int64_t M;
  int64_t rows_per_wg;  // epilogue_bwd_rows()
  int N;
};
int64_t epilogue_bwd_rows(int64_t M, int64_t N, int cus);
int64_t epilogue_bwd_partials(int64_t M, int64_t N, int cus);  // rows of partials that serve up to M rows
hipError_t launch_epilogue_bwd(const EpilogueBwdParams& p, int act, hipStream_t stream);


// ---- experts of a mixture-of-experts layer for a few tokens (moe_experts.hip)
constexpr int kExpertsMaxTokens = 64;
constexpr int kExpertsMaxTopK = 16;
constexpr int kExpertsMaxChoices = kExpertsMaxTokens * kExpertsMaxTopK;
constexpr int kExpertsMaxGroups = 1024;
constexpr int kExpertsMaxDim = 32768;  // H and I: a wave's quarter of a row is at most 64 steps of 128
// The choices by expert, as the first kernel leaves them for the second in the workspace
struct ExpertsTable {
  int n;                                // chosen experts
  uint32_t run[kExpertsMaxChoices];     // of each: number, tokens and first entry
  uint32_t entry[kExpertsMaxChoices];   // token << 16 | choice whose row of h is the token's
  float weight[kExpertsMaxChoices];
};
struct ExpertsParams {
  const uint16_t* x;     // [T][H] bf16
  const int32_t* idx;    // [T][k]
  const float* w;        // [T][k]
  const uint8_t* w1;     // [G][2 I][H], gate rows first
  const void* s1;
  const uint8_t* w2;     // [G][H][I]
  const void* s2;
  uint16_t* y;           // [T][H] bf16
  uint16_t* h;           // [T k][I] bf16
  ExpertsTable* table;
  float* partials;       // [H / 16][splits][T][16], splits > 1
  unsigned int* counters;
  int T, k, first, G, H, I;
  int splits;
};
int experts_splits(int64_t T, int64_t choices, int64_t H, int64_t I, int64_t G, int cus);
size_t experts_h_bytes(int64_t choices, int64_t I);
hipError_t launch_moe_experts(const ExpertsParams& p, bool fp4, bool stream_weights, int cus, hipStream_t stream);

}  // namespace dg
