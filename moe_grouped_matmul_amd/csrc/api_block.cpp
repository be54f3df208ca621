// C ABI of the operators that join the products of a block: the root-mean-square
// norm, the gradient of a product's epilogue, and the experts of a layer for a
// few tokens.  As in api.cpp, no call allocates, synchronises or reads device
// data on the host, and no call throws.

#include <cmath>

#include "block_internal.hpp"
#include "dg.h"
#include "host.hpp"

namespace {

using namespace dg;

constexpr int64_t kIntMax = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxNormRows = ((int64_t)1 << 23) - 1;  // workgroups of up to 512 threads in a launch: thread counts are 32 bits

hipStream_t hs(void* stream) { return static_cast<hipStream_t>(stream); }

int launched(hipError_t e) {
  return e == hipSuccess ? ok() : fail(DG_ERR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
}

int check_norm(int dtype, int weight_dtype, int64_t M, int64_t K) {
  if ((dtype != DG_F32 && dtype != DG_BF16) || (weight_dtype != DG_F32 && weight_dtype != DG_BF16))
    return fail(DG_ERR_INVALID_ARG, "dtypes must be DG_F32 or DG_BF16 (got %d and %d)", dtype, weight_dtype);
  if (K <= 0 || K % 8 || K > kNormMaxK)
    return fail(DG_ERR_SHAPE, "K must be a positive multiple of 8 up to %d (got %lld)", kNormMaxK, (long long)K);
  if (M < 0) return fail(DG_ERR_SHAPE, "M must be >= 0");
  if (M > kMaxNormRows) return fail(DG_ERR_SHAPE, "M must be below 2^23 (got %lld)", (long long)M);
  return DG_OK;
}

// bytes of the rows of partial sums past a workspace's counters
size_t partials_bytes(int64_t rows, int64_t N) { return kBlockWsCounterBytes + (size_t)rows * (size_t)N * 4; }

int check_partials(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws || !aligned(ws, 16) || ws_bytes < need)
    return fail(DG_ERR_WORKSPACE, "a 16-byte aligned workspace of at least %zu bytes is needed", need);
  return DG_OK;
}

constexpr size_t kTableBytes = (sizeof(ExpertsTable) + 255) / 256 * 256;

size_t experts_bytes(int64_t choices, int64_t T, int64_t H, int64_t I, int splits) {
  // (more than 8 tokens may be summed by twice as many workgroups to twice as many columns)
  const int most = T > 8 ? 2 * splits : splits;
  return kBlockWsCounterBytes + kTableBytes + experts_h_bytes(choices, I) + (most > 1 ? (size_t)most * (size_t)H * (size_t)T * 4 : 0);
}

bool experts_dim(int64_t d) { return d > 0 && d % 128 == 0 && d <= kExpertsMaxDim; }

int run_experts(bool fp4, const uint16_t* x, const int32_t* topk_idx, const float* topk_w, const uint8_t* w1, const void* s1,
                const uint8_t* w2, const void* s2, uint16_t* y, int64_t T, int64_t k, int64_t first_expert, int64_t G, int64_t H,
                int64_t I, void* ws, size_t ws_bytes, void* stream) {
  if (T < 0 || T > kExpertsMaxTokens) return fail(DG_ERR_SHAPE, "T must be in [0, %d] (got %lld)", kExpertsMaxTokens, (long long)T);
  if (k < 1 || k > kExpertsMaxTopK) return fail(DG_ERR_SHAPE, "k must be in [1, %d] (got %lld)", kExpertsMaxTopK, (long long)k);
  if (G < 1 || G > kExpertsMaxGroups) return fail(DG_ERR_SHAPE, "G must be in [1, %d] (got %lld)", kExpertsMaxGroups, (long long)G);
  if (first_expert < 0 || first_expert > kIntMax - G) return fail(DG_ERR_SHAPE, "first_expert out of range");
  if (!experts_dim(H) || !experts_dim(I))
    return fail(DG_ERR_SHAPE, "H and I must be positive multiples of 128 up to %d (got %lld and %lld)", kExpertsMaxDim, (long long)H, (long long)I);
  if (T == 0) return ok();
  if (!x || !topk_idx || !topk_w || !w1 || !s1 || !w2 || !s2 || !y) return fail(DG_ERR_INVALID_ARG, "null pointer");
  if (!aligned(x, 16) || !aligned(w1, 16) || !aligned(w2, 16) || !aligned(y, 16))
    return fail(DG_ERR_ALIGN, "x, w1, w2 and y must be 16-byte aligned");
  if (!aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(s1, 4) || !aligned(s2, 4))
    return fail(DG_ERR_ALIGN, "topk_idx, topk_w and scales must be 4-byte aligned");
  int cus = 0, rc = check_device(&cus);
  if (rc) return rc;
  const int splits = experts_splits(T, T * k, H, I, G, effective_cus(cus));
  const size_t need = experts_bytes(T * k, T, H, I, splits);
  if (!ws || !aligned(ws, 16) || ws_bytes < need)
    return fail(DG_ERR_WORKSPACE, "a 16-byte aligned workspace of at least %zu bytes is needed", need);
  uint8_t* base = static_cast<uint8_t*>(ws) + kBlockWsCounterBytes;
  ExpertsParams p{};
  p.x = x;
  p.idx = topk_idx;
  p.w = topk_w;
  p.w1 = w1;
  p.s1 = s1;
  p.w2 = w2;
  p.s2 = s2;
  p.y = y;
  p.table = reinterpret_cast<ExpertsTable*>(base);
  p.h = reinterpret_cast<uint16_t*>(base + kTableBytes);
  p.partials = reinterpret_cast<float*>(base + kTableBytes + experts_h_bytes(T * k, I));
  p.counters = static_cast<unsigned int*>(ws);
  p.T = (int)T;
  p.k = (int)k;
  p.first = (int)first_expert;
  p.G = (int)G;
  p.H = (int)H;
  p.I = (int)I;
  p.splits = splits;
  // Weights that the L2 caches cannot hold, nor the 256 MB Infinity Cache beside those of other layers, are streamed past both:
  // of layers in turn 96 MiB take 28 -> 26.5 us (one token) and 38.5 -> 38 (64), 192 MiB 43 -> 39.5 and 57 -> 54, while 24 MiB
  // would take 19 -> 20 (64).  One layer again and again would come from the cache: 192 MiB, 64 tokens 44 us, streamed 52.
  const bool stream_weights = G * 3 * H * I / (fp4 ? 2 : 1) >= (int64_t)64 << 20;
  return launched(launch_moe_experts(p, fp4, stream_weights, effective_cus(cus), hs(stream)));
}

float* partials_of(void* ws) { return reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kBlockWsCounterBytes); }

}  // namespace

namespace dg {

int check_activation(int act) {
  return act >= DG_ACT_NONE && act <= DG_ACT_GELU_TANH ? DG_OK : fail(DG_ERR_INVALID_ARG, "unknown activation %d", act);
}

size_t block_workspace_size(int op, int64_t rows, int64_t N, int64_t K, int cus) {
  if (rows < 0 || rows > kIntMax) return 0;
  size_t need = 0;
  if (op == DG_OP_RMS_NORM_BWD) {
    if (K <= 0 || K % 8 || K > kNormMaxK) return 0;
    need = partials_bytes(norm_bwd_grid(rows, K, cus), K);
  } else if (op == DG_OP_EPILOGUE_BWD) {
    if (N <= 0 || N % 16 || N > (int64_t)1 << 30) return 0;
    need = partials_bytes(epilogue_bwd_partials(rows, N, cus), N);
  } else if (op == DG_OP_MOE_EXPERTS) {
    if (rows > kExpertsMaxChoices || !experts_dim(N) || !experts_dim(K)) return 0;
    const int64_t tokens = rows < kExpertsMaxTokens ? rows : kExpertsMaxTokens;  // k may be 1
    // (as many tokens as choices, whose workgroups are the smaller and so the more)
    need = experts_bytes(rows, tokens, N, K, experts_splits(kExpertsMaxTokens, rows, N, K, kExpertsMaxGroups, cus));
  }
  return (need + 15) / 16 * 16;
}

}  // namespace dg

extern "C" {

int dg_rms_norm(const void* x, const void* residual, const void* weight, int dtype, int weight_dtype, void* h, void* y,
                uint8_t* q, void* sf, int scale_kind, float* rstd, int64_t M, int64_t K, float eps, void* stream) {
  int rc = check_norm(dtype, weight_dtype, M, K);
  if (rc) return rc;
  if (!(eps > 0.f) || std::isinf(eps)) return fail(DG_ERR_INVALID_ARG, "eps must be positive and finite");
  if (scale_kind != DG_SCALE_F32 && scale_kind != DG_SCALE_UE8M0)
    return fail(DG_ERR_INVALID_ARG, "scale_kind must be DG_SCALE_F32 or DG_SCALE_UE8M0 (got %d)", scale_kind);
  if (M == 0) return ok();
  if (!x || !weight || (!y && !q) || (residual && !h) || (!q != !sf)) return fail(DG_ERR_INVALID_ARG, "null pointer");
  if (q && K % 128) return fail(DG_ERR_SHAPE, "K must be a multiple of 128 for the quantised output (got %lld)", (long long)K);
  if (h && h == y) return fail(DG_ERR_INVALID_ARG, "h and y must be different arrays");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(h, 16) || !aligned(y, 16) || !aligned(q, 16))
    return fail(DG_ERR_ALIGN, "x, residual, weight, h, y and q must be 16-byte aligned");
  if (!aligned(sf, 4) || !aligned(rstd, 4)) return fail(DG_ERR_ALIGN, "sf and rstd must be 4-byte aligned");
  int cus = 0;
  if ((rc = check_device(&cus))) return rc;
  const NormParams p{x, residual, weight, h, y, q, sf, rstd, M, (int)K, weight_dtype == DG_BF16, eps};
  const int kind = !q ? kNoQuant : scale_kind == DG_SCALE_F32 ? kScaleF32 : kScaleUe8m0;
  return launched(launch_rms_norm(p, dtype == DG_BF16, kind, effective_cus(cus), hs(stream)));
}

int dg_rms_norm_bwd(const void* dy, const void* h, const void* weight, const float* rstd, int dtype, int weight_dtype,
                    const void* dh, void* dx, float* dw, int64_t M, int64_t K, void* workspace, size_t workspace_bytes,
                    void* stream) {
  int rc = check_norm(dtype, weight_dtype, M, K);
  if (rc) return rc;
  if (!weight || !dw || (M > 0 && (!dy || !h || !rstd || !dx))) return fail(DG_ERR_INVALID_ARG, "null pointer");
  if (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(dh, 16) || !aligned(dx, 16))
    return fail(DG_ERR_ALIGN, "dy, h, weight, dh and dx must be 16-byte aligned");
  if (!aligned(rstd, 4) || !aligned(dw, 4)) return fail(DG_ERR_ALIGN, "rstd and dw must be 4-byte aligned");
  int cus = 0;
  if ((rc = check_device(&cus))) return rc;
  cus = effective_cus(cus);
  if ((rc = check_partials(workspace, workspace_bytes, partials_bytes(norm_bwd_grid(M, K, cus), K)))) return rc;
  const NormBwdParams p{dy, h, weight, rstd, dh, dx, dw, partials_of(workspace), M, (int)K, weight_dtype == DG_BF16};
  return launched(launch_rms_norm_bwd(p, dtype == DG_BF16, cus, hs(stream)));
}

int dg_epilogue_bwd(const uint16_t* dy, const uint16_t* pre, int act, uint16_t* dz, uint8_t* q, float* sf, float* dbias,
                    int64_t M, int64_t N, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_activation(act);
  if (rc) return rc;
  if (N <= 0 || N % 16 || N > (int64_t)1 << 30) return fail(DG_ERR_SHAPE, "N must be a positive multiple of 16 (got %lld)", (long long)N);
  if (M < 0 || M > kIntMax) return fail(DG_ERR_SHAPE, "M out of range");
  if ((!dz && !q && !dbias) || (!q != !sf) || (M > 0 && (!dy || (!pre && act != DG_ACT_NONE))))
    return fail(DG_ERR_INVALID_ARG, "null pointer");
  if (q && N % 128) return fail(DG_ERR_SHAPE, "N must be a multiple of 128 for the quantised output (got %lld)", (long long)N);
  if (!aligned(dy, 16) || !aligned(pre, 16) || !aligned(dz, 16) || !aligned(q, 16))
    return fail(DG_ERR_ALIGN, "dy, pre, dz and q must be 16-byte aligned");
  if (!aligned(sf, 4) || !aligned(dbias, 4)) return fail(DG_ERR_ALIGN, "sf and dbias must be 4-byte aligned");
  if (M == 0 && !dbias) return ok();
  int cus = 0;
  if ((rc = check_device(&cus))) return rc;
  const int64_t rows = M == 0 ? 8 : epilogue_bwd_rows(M, N, effective_cus(cus));
  if (dbias && (rc = check_partials(workspace, workspace_bytes, partials_bytes(ceil_div(M, rows), N)))) return rc;
  const EpilogueBwdParams p{dy, pre, dz, q, sf, dbias, dbias ? partials_of(workspace) : nullptr, M, rows, (int)N};
  return launched(launch_epilogue_bwd(p, act, hs(stream)));
}

int dg_moe_experts_fp8(const uint16_t* x, const int32_t* topk_idx, const float* topk_w, const uint8_t* w1, const float* s1,
                       const uint8_t* w2, const float* s2, uint16_t* y, int64_t T, int64_t k, int64_t first_expert, int64_t G,
                       int64_t H, int64_t I, void* workspace, size_t workspace_bytes, void* stream) {
  return run_experts(false, x, topk_idx, topk_w, w1, s1, w2, s2, y, T, k, first_expert, G, H, I, workspace, workspace_bytes, stream);
}

int dg_moe_experts_mxfp4(const uint16_t* x, const int32_t* topk_idx, const float* topk_w, const uint8_t* w1, const int32_t* s1,
                         const uint8_t* w2, const int32_t* s2, uint16_t* y, int64_t T, int64_t k, int64_t first_expert, int64_t G,
                         int64_t H, int64_t I, void* workspace, size_t workspace_bytes, void* stream) {
  return run_experts(true, x, topk_idx, topk_w, w1, s1, w2, s2, y, T, k, first_expert, G, H, I, workspace, workspace_bytes, stream);
}

}  // extern "C"
