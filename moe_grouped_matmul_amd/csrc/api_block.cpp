// C ABI of the operators that join the products of a block: the root-mean-square
// norm and the gradient of a product's epilogue.  As in api.cpp, no call
// allocates, synchronises or reads device data on the host, and no call throws.

#include <cmath>

#include "block_internal.hpp"
#include "dg.h"
#include "host.hpp"

namespace {

using namespace dg;

constexpr int64_t kIntMax = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxWorkgroups = ((int64_t)1 << 24) - 1;  // of 256 threads in a launch: thread counts are 32 bits

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
  if (M > kMaxWorkgroups) return fail(DG_ERR_SHAPE, "M too large");
  return DG_OK;
}

// bytes of the rows of partial sums past a workspace's counters
size_t partials_bytes(int64_t rows, int64_t N) { return kBlockWsCounterBytes + (size_t)rows * (size_t)N * 4; }

int check_partials(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws || !aligned(ws, 16) || ws_bytes < need)
    return fail(DG_ERR_WORKSPACE, "a 16-byte aligned workspace of at least %zu bytes is needed", need);
  return DG_OK;
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
  const int64_t rows = M == 0 ? 16 : epilogue_bwd_rows(M, N, effective_cus(cus));
  if (dbias && (rc = check_partials(workspace, workspace_bytes, partials_bytes(ceil_div(M, rows), N)))) return rc;
  const EpilogueBwdParams p{dy, pre, dz, q, sf, dbias, dbias ? partials_of(workspace) : nullptr, M, rows, (int)N};
  return launched(launch_epilogue_bwd(p, act, hs(stream)));
}

}  // extern "C"
