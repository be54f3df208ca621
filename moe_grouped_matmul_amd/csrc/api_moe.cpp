// C ABI of the mixture-of-experts operators and the microscaled 4-bit
// products: argument validation, plans and launches on the caller's stream.
// As in api.cpp, no call allocates, synchronises or reads device data on the
// host, and no call throws.

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "dg.h"
#include "host.hpp"
#include "moe_internal.hpp"

namespace {

using namespace dg;

constexpr int64_t kIntMax = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxWorkgroups = ((int64_t)1 << 24) - 1;  // of 256 threads in a launch: thread counts are 32 bits
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTopK = 16;

hipStream_t hs(void* stream) { return static_cast<hipStream_t>(stream); }

int launched(hipError_t e) {
  return e == hipSuccess ? ok() : fail(DG_ERR_LAUNCH, "launch failed: %s", hipGetErrorString(e));
}

int check_dtype(int dtype) {
  if (dtype != DG_F32 && dtype != DG_BF16) return fail(DG_ERR_INVALID_ARG, "dtype must be DG_F32 or DG_BF16 (got %d)", dtype);
  return DG_OK;
}

// ---- microscaled 4-bit products

// DG_FORCE_CONFIG's "mxfp4=<bm>x<bn>[x<splits>]": the tile shape wherever the form has it, -1 without one.
int mx_forced_tile(int* splits = nullptr) {
  const char* e = std::getenv("DG_FORCE_CONFIG");
  const char* at = e ? std::strstr(e, "mxfp4=") : nullptr;
  int bm = 0, bn = 0, sp = 0;
  if (!at || std::sscanf(at + 6, "%dx%dx%d", &bm, &bn, &sp) < 2) return -1;
  if (splits) *splits = sp;
  for (int t : {kMx64x64, kMx128x256, kMx256x256})
    if (bm == mx_bm(t) && bn == mx_bn(t)) return t;
  return -1;
}

struct MxPlan {
  int tile = kMx64x64;
  int m_tiles = 0;
  int n_tiles = 0;
  int splits = 1;
  int steps_per_split = 0;
};

// Estimated times (us) of a call. 64 x 64 and 128 x 256 tiles: rounds of tiles over the CUs (two 64 x 64 workgroups to a
// CU), a step of 256 K elements costing 0.45 and 1.05 us a round, and the start, epilogue and last write-back.
double mx_cost_us(int tile, int64_t tiles, int64_t K, int cus) {
  const double steps = (double)ceil_div(K, 256);
  if (tile == kMx64x64) return (double)ceil_div(tiles, 2 * cus) * (0.45 * steps + 1.5) + 3.0;
  return (double)ceil_div(tiles, cus) * (1.05 * steps + 3.0) + 5.0;
}
// The persistent kernel's: whole rounds of 256 x 256 tiles, then as it distributes the rest (the same rules). A step of
// a large tile costs 0.66 us and 0.9 more as all CUs run one (the clock), of a 128 x 256 tile 1.0, of a 128 x 128
// quarter 0.5; steps run in twos, a quarter's in fours. Fitted, with the above, to 28 dense shapes of 200-4352 rows with
// every tile shape forced: the tile of least estimate was the fastest or within 10% of it on each (1024 x 4096 x 4096:
// 20, 22 and 16 us; 1024 x 2048 x 7168: 16, 31 and 20; 2048 x 4096 x 2048: 24, 16 and 17; 2500 x 4096 x 7168: 66, 66 and
// 45; 4000 x 4096 x 512: 33, 18 and 15).
double mx_wide_us(int64_t large, int64_t small, int64_t K, int cus) {
  const int64_t rounds = large / cus;
  const int64_t rest = large % cus;
  const bool cut = rest > 0 && 2 * rest + small <= cus;
  const bool spread = rest > 0 && !cut;
  const int64_t halves = std::max<int64_t>(0, small + (cut ? 2 * rest : 0) - (spread ? 2 * (cus - rest) : 0));
  const bool quarters = halves % cus > 0 && 2 * (halves % cus) <= cus;
  const int64_t half_rounds = quarters ? halves / cus : ceil_div(halves, cus);
  double step = 1.56 * (double)rounds + 1.0 * (double)half_rounds;
  if (spread) step += 0.66 + 0.9 * (rounds ? 1.0 : (double)rest / (double)cus);
  return step * 2.0 * (double)ceil_div(K, 512) + (quarters ? 2.0 * (double)ceil_div(K, 1024) : 0.0) +
         (rounds || spread ? 11.0 : half_rounds ? 9.0 : 6.0);
}

// Dense: the tile shape of least estimated time; 64 x 64 tiles that leave CUs idle split K where that is estimated to
// pay (64 x 2112 x 7168: 11.7 us whole, 8.6 in four parts; 64 x 7168 x 2048: 6.2 whole, 7.4 in two; more parts than CUs
// were slower everywhere).
MxPlan plan_mx_dense(int64_t M, int64_t N, int64_t K, int cus, size_t ws_bytes) {
  MxPlan pl;
  const int64_t steps = ceil_div(K, 256);
  double best = -1.0;
  for (int t : {kMx64x64, kMx128x256, kMx256x256}) {
    const int64_t n_tiles = ceil_div(N, mx_bn(t));
    const bool odd = M % 256 >= 1 && M % 256 <= 128;  // the last row tile has up to 128 rows
    const double c = t == kMx256x256 ? mx_wide_us((M + 127) / 256 * n_tiles, odd ? n_tiles : 0, K, cus)
                                     : mx_cost_us(t, ceil_div(M, mx_bm(t)) * n_tiles, K, cus);
    if (best < 0 || c < best) {
      best = c;
      pl.tile = t;
    }
  }
  int forced_splits = 0;
  if (const int f = mx_forced_tile(&forced_splits); f >= 0) pl.tile = f;
  pl.m_tiles = (int)ceil_div(M, mx_bm(pl.tile));
  pl.n_tiles = (int)ceil_div(N, mx_bn(pl.tile));
  int64_t s = 1;
  if (pl.tile == kMx64x64) {
    const int64_t tiles = (int64_t)pl.m_tiles * pl.n_tiles;
    // a step costs 0.27 us, splitting 2 us and 0.3 us a part; at most one workgroup a CU
    double least = 0.27 * (double)steps;
    for (int64_t c = 2; c <= 8 && c * tiles <= cus && c <= steps; ++c) {
      const double t = 0.27 * (double)ceil_div(steps, c) + 2.0 + 0.3 * (double)c;
      if (t < least) {
        least = t;
        s = c;
      }
    }
    if (forced_splits > 0) s = std::min<int64_t>(forced_splits, steps);
    if (s < 1 || tiles > kMxMaxCounters) s = 1;
    while (s > 1 && mx_workspace_bytes(pl.tile, pl.m_tiles, pl.n_tiles, (int)s) > ws_bytes) --s;
  }
  pl.steps_per_split = (int)ceil_div(steps, s);
  pl.splits = (int)ceil_div(steps, pl.steps_per_split);  // every split non-empty
  return pl;
}

// Contiguous: the tile shape of least estimated time. Every other expert's number of 128-row blocks is taken to be odd,
// the persistent kernel is charged 4 us for reading m_indices first, and the weights of all experts and the output pass
// at 2.8, 3.5 or 4.3 TB/s at most (experts of few rows, whose weights no other row tile repeats: 64 experts, 256 rows,
// 4096 x 7168 in 314, 220 and 214 us). Of 18 layouts of 8-8192 rows and 2-64 experts the choice was the fastest of the
// three or within 3% of it on 16 (2000 rows of 16 experts, 512 x 7168, 16, 31 and 24 us; 1000 of 4, 4096 x 2048, 20, 16
// and 19; 8192 of 16, 4096 x 1024, 96, 58 and 47), and slower on two: 1500 of 8, 4096 x 1024, 25, 22 (chosen) and 18;
// 8192 of 64, 512 x 2048, 26, 17 and 23 (chosen).
int mx_contiguous_tile(int64_t rows, int64_t N, int64_t K, int64_t G, int cus) {
  const int64_t blocks = ceil_div(rows, 128);
  const int64_t odd = std::min(blocks, (G + 1) / 2);
  const double mb = 1e-6 * ((double)G * (double)N * (double)K / 2 + 2.0 * (double)rows * (double)N);
  int tile = kMx64x64;
  double best = -1.0;
  for (int t : {kMx64x64, kMx128x256, kMx256x256}) {
    const int64_t n_tiles = ceil_div(N, mx_bn(t));
    const double c = t == kMx256x256   ? std::max(mx_wide_us((blocks - odd + 1) / 2 * n_tiles, odd * n_tiles, K, cus) + 4.0, mb / 4.3 + 10.5)
                     : t == kMx128x256 ? std::max(mx_cost_us(t, blocks * n_tiles, K, cus), mb / 3.5 + 8.0)
                                       : std::max(mx_cost_us(t, 2 * blocks * n_tiles, K, cus), mb / 2.8 + 3.0);
    if (best < 0 || c < best) {
      best = c;
      tile = t;
    }
  }
  return tile;
}

int check_mx_shape(int64_t N, int64_t K) {
  if (K <= 0 || K % 128 != 0) return fail(DG_ERR_SHAPE, "K must be a positive multiple of 128 (got %lld)", (long long)K);
  if (N <= 0 || N % 16 != 0) return fail(DG_ERR_SHAPE, "N must be a positive multiple of 16 (got %lld)", (long long)N);
  // a tile's rows (256 of K / 2 bytes) are addressed with 32-bit offsets
  if (K > (int64_t)1 << 24 || N > (int64_t)1 << 30) return fail(DG_ERR_SHAPE, "N or K too large");
  return DG_OK;
}

int check_mx_operands(const void* A, const void* sfa, const void* B, const void* sfb, const void* D) {
  if (!A || !sfa || !B || !sfb || !D) return fail(DG_ERR_INVALID_ARG, "null operand pointer");
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(D, 16))
    return fail(DG_ERR_ALIGN, "A, B and D must be 16-byte aligned");
  if (!aligned(sfa, 4) || !aligned(sfb, 4)) return fail(DG_ERR_ALIGN, "scale arrays must be 4-byte aligned");
  return DG_OK;
}

int run_mx(int form, const uint8_t* A, const int32_t* sfa, const uint8_t* B, const int32_t* sfb, uint16_t* D,
           const int32_t* index, int64_t rows, int64_t N, int64_t K, int64_t G, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_mx_shape(N, K);
  if (rc) return rc;
  if (G < 1 || G > kMaxGroups) return fail(DG_ERR_SHAPE, "G must be in [1, 1024] (got %lld)", (long long)G);
  if (rows < 0) return fail(DG_ERR_SHAPE, "row counts must be >= 0");
  if (rows > kIntMax) return fail(DG_ERR_SHAPE, "too many rows (%lld)", (long long)rows);
  if (rows == 0) return ok();
  if ((rc = check_mx_operands(A, sfa, B, sfb, D))) return rc;
  if (form != kMxDense && !index) return fail(DG_ERR_INVALID_ARG, form == kMxMasked ? "null masked_m" : "null m_indices");
  if (form != kMxDense && !aligned(index, 4)) return fail(DG_ERR_ALIGN, "index arrays must be 4-byte aligned");
  if (ws && (!aligned(ws, 16) || ws_bytes % 4))
    return fail(DG_ERR_WORKSPACE, "workspace must be 16-byte aligned with a size that is a multiple of 4");
  // scale words of an operand (masked: of one expert) are addressed with 32-bit offsets, up to three rows of them past K
  if (rows * (K / 128 + 8) * 4 >= kOffLim || N * (K / 128 + 8) * 4 >= kOffLim) return fail(DG_ERR_SHAPE, "scale arrays exceed 4 GiB");
  int cus = 0;
  if ((rc = check_device(&cus))) return rc;
  if (form == kMxContiguous && (rc = check_contiguous_layout(index, rows, G, stream))) return rc;
  cus = effective_cus(cus);
  MxPlan pl;
  if (form == kMxDense) {
    pl = plan_mx_dense(rows, N, K, cus, ws ? ws_bytes : 0);
  } else {
    // masked: by the estimates at full experts (32 experts x 128 rows, 4096 x 7168, in 64 x 64 and 128 x 256 tiles: 144 and
    // 94 us; 8 x 256, 3584 x 1536: 22 and 13; 8 x 256, 1024 x 2048: 8.5 and 12.5)
    const auto cost = [&](int t) { return mx_cost_us(t, G * ceil_div(rows, mx_bm(t)) * ceil_div(N, mx_bn(t)), K, cus); };
    pl.tile = form == kMxContiguous ? mx_contiguous_tile(rows, N, K, G, cus) : cost(kMx64x64) < cost(kMx128x256) ? kMx64x64 : kMx128x256;
    const int f = mx_forced_tile();
    if (f >= 0 && (form == kMxContiguous || f != kMx256x256)) pl.tile = f;
    pl.m_tiles = (int)ceil_div(rows, mx_bm(pl.tile));
    pl.n_tiles = (int)ceil_div(N, mx_bn(pl.tile));
    pl.steps_per_split = (int)ceil_div(K, 256);
  }
  const int64_t units = (int64_t)pl.n_tiles * (form == kMxMasked ? G : pl.splits);
  if (pl.tile != kMx256x256 && (ceil_div(units, 8) * 8) * pl.m_tiles > kMaxWorkgroups / 2) return fail(DG_ERR_SHAPE, "too many tiles");
  MxGemmParams p{};
  p.A = A;
  p.sfa = sfa;
  p.sfa_ld = rows;
  p.B = B;
  p.sfb = sfb;
  p.D = D;
  p.ws = ws;
  p.index = index;
  p.rows = rows;
  p.N = (int)N;
  p.K = (int)K;
  p.G = (int)G;
  p.m_tiles = pl.m_tiles;
  p.n_tiles = pl.n_tiles;
  p.splits = pl.splits;
  p.steps_per_split = pl.steps_per_split;
  // one row tile reads each weight once; weights that the 256 MB Infinity Cache cannot hold from one call to the next
  // are streamed past it (32 experts of 4096 x 7168: 103 -> 94 us; 7168 x 16384, which it holds: 16 -> 19 us, so not there)
  p.stream_weights = pl.m_tiles == 1 && G * N * (K / 2) >= (int64_t)256 << 20;
  if (print_configs())
    std::fprintf(stderr, "[dg] mxfp4%s rows=%lld N=%lld K=%lld G=%lld tile=%dx%d tiles=%lld splits=%d\n",
                 form == kMxDense ? "" : form == kMxMasked ? "_masked" : "_contiguous", (long long)rows, (long long)N,
                 (long long)K, (long long)G, mx_bm(pl.tile), mx_bn(pl.tile), (long long)pl.m_tiles * pl.n_tiles, pl.splits);
  if (pl.tile != kMx256x256) return launched(launch_mxfp4_gemm(form, pl.tile, p, hs(stream)));
  // persistent tiles; the contiguous form lists a launch's 128-row blocks in LDS, so longer calls run in chunks of rows
  const int64_t chunk = form == kMxContiguous ? (int64_t)kMxWideMaxBlocks * 128 : rows;
  for (int64_t r0 = 0; r0 < rows; r0 += chunk) {
    p.rows = std::min(chunk, rows - r0);
    p.A = A + r0 * (K / 2);
    p.sfa = sfa + r0;
    p.D = D + r0 * N;
    p.index = index ? index + r0 : nullptr;
    const int64_t quarters = ceil_div(p.rows, 128) * 2 * pl.n_tiles;  // the smallest pieces a tile is cut into
    const hipError_t e = launch_mxfp4_wide(form, (int)std::min<int64_t>(quarters, cus), p, hs(stream));
    if (e != hipSuccess) return launched(e);
  }
  return ok();
}

int check_quant(int dtype, int64_t G, int64_t R, int64_t K) {
  int rc = check_dtype(dtype);
  if (rc) return rc;
  if (K <= 0 || K % 128) return fail(DG_ERR_SHAPE, "K must be a positive multiple of 128 (got %lld)", (long long)K);
  if (G < 0 || R < 0) return fail(DG_ERR_SHAPE, "G and row counts must be >= 0");
  // one launch, 4 rows x 512 columns a workgroup
  if (K > kIntMax || R > kIntMax || G > 65535 || ceil_div(R, 4) * ceil_div(K, 512) > kMaxWorkgroups)
    return fail(DG_ERR_SHAPE, "problem too large");
  return DG_OK;
}

int check_topk(int64_t T, int64_t k) {
  if (T < 0) return fail(DG_ERR_SHAPE, "T must be >= 0");
  if (k < 1 || k > kMaxTopK) return fail(DG_ERR_SHAPE, "k must be in [1, 16] (got %lld)", (long long)k);
  if (T * k > kIntMax) return fail(DG_ERR_SHAPE, "T * k too large");
  return DG_OK;
}

int check_gate(int dtype, int64_t T, int64_t E, int64_t k, float w_scale) {
  int rc = check_dtype(dtype);
  if (rc) return rc;
  if (T > kIntMax) return fail(DG_ERR_SHAPE, "T too large");
  if ((rc = check_topk(T, k))) return rc;
  if (E < 1 || E > kMaxExperts) return fail(DG_ERR_SHAPE, "E must be in [1, 1024] (got %lld)", (long long)E);
  if (k > E) return fail(DG_ERR_SHAPE, "k must be at most E (got %lld of %lld)", (long long)k, (long long)E);
  if (!(std::fabs(w_scale) > 0.f) || std::isinf(w_scale)) return fail(DG_ERR_INVALID_ARG, "w_scale must be finite and not 0");
  return DG_OK;
}

int run_layout(const int32_t* topk_idx, int32_t* counts, int32_t* m_indices, int32_t* row_token, int32_t* row_of, int64_t T,
               int64_t k, int64_t first_expert, int64_t G, int64_t max_m, int64_t rows, void* ws, size_t ws_bytes,
               void* stream) {
  if (T > kIntMax) return fail(DG_ERR_SHAPE, "T too large");
  int rc = check_topk(T, k);
  if (rc) return rc;
  if (G < 1 || G > kMaxGroups) return fail(DG_ERR_SHAPE, "G must be in [1, 1024] (got %lld)", (long long)G);
  if (first_expert < 0 || first_expert > kIntMax - G) return fail(DG_ERR_SHAPE, "first_expert out of range");
  if (rows < 0 || rows > kIntMax || T * k + 128 * G > kIntMax) return fail(DG_ERR_SHAPE, "row numbers must fit 32 bits");
  const bool masked = max_m > 0;
  if (!counts || (rows > 0 && (!row_token || (!masked && !m_indices))) || (T > 0 && (!topk_idx || !row_of)))
    return fail(DG_ERR_INVALID_ARG, "null pointer");
  if (!aligned(topk_idx, 4) || !aligned(counts, 4) || !aligned(row_token, 4) || !aligned(row_of, 4) || !aligned(m_indices, 4))
    return fail(DG_ERR_ALIGN, "index arrays must be 4-byte aligned");
  const size_t need = layout_workspace_needed(T * k, G);
  if (!ws || !aligned(ws, 16) || ws_bytes < need)
    return fail(DG_ERR_WORKSPACE, "a 16-byte aligned workspace of at least %zu bytes is needed", need);
  int cus = 0;
  if ((rc = check_device(&cus))) return rc;
  LayoutParams p{};
  p.idx = topk_idx;
  p.counts = counts;
  p.m_indices = masked ? nullptr : m_indices;
  p.row_token = row_token;
  p.row_of = row_of;
  p.ws = ws;
  p.n = T * k;
  p.k = (int)k;
  p.first = (int)first_expert;
  p.G = (int)G;
  p.max_m = max_m;
  p.rows = rows;
  return launched(launch_layout(p, hs(stream)));
}

int check_combine(int dtype, int64_t T, int64_t k, int64_t N, int64_t R) {
  int rc = check_dtype(dtype);
  if (rc) return rc;
  if (T > kIntMax) return fail(DG_ERR_SHAPE, "T too large");
  if ((rc = check_topk(T, k))) return rc;
  if (N <= 0 || N % 16) return fail(DG_ERR_SHAPE, "N must be a positive multiple of 16 (got %lld)", (long long)N);
  if (N > (int64_t)1 << 30 || R < 0 || R > kIntMax)
    return fail(DG_ERR_SHAPE, "N or row count out of range");
  return DG_OK;
}

}  // namespace

namespace dg {

size_t moe_workspace_size(int op, int64_t rows, int64_t N, int64_t K, int64_t G, int cus) {
  size_t need = 0;
  if (op == DG_OP_MXFP4_GEMM_NT) {
    if (rows <= 0 || rows > kIntMax || N <= 0 || N > (int64_t)1 << 30 || K <= 0 || K % 128) return 0;
    const MxPlan pl = plan_mx_dense(rows, N, K, cus, (size_t)-1);
    need = mx_workspace_bytes(pl.tile, pl.m_tiles, pl.n_tiles, pl.splits);
  } else if (op == DG_OP_MOE_GATE) {
    if (rows < 0 || rows > kIntMax || N < 1 || N > kMaxExperts) return 0;
    need = gate_workspace_bytes(rows, N);
  } else if (op == DG_OP_MOE_LAYOUT) {
    if (rows < 0 || rows > kIntMax || K < 1 || K > kMaxTopK || G < 1 || G > kMaxGroups) return 0;
    need = layout_workspace_bytes(rows * K, G);
  }
  return (need + 15) / 16 * 16;
}

int moe_describe_plan(int op, int64_t rows, int64_t N, int64_t K, int64_t G, int cus, char* buf, size_t n) {
  if (op != DG_OP_MXFP4_GEMM_NT || rows <= 0 || rows > kIntMax || N <= 0 || N % 16 || N > (int64_t)1 << 30 || K <= 0 || K % 128 ||
      K > (int64_t)1 << 24)
    return 0;
  (void)G;
  const MxPlan pl = plan_mx_dense(rows, N, K, cus, (size_t)-1);
  std::snprintf(buf, n, "kernel=mxfp4 tile=%dx%d tiles=%lld splits=%d", mx_bm(pl.tile), mx_bn(pl.tile),
                (long long)pl.m_tiles * pl.n_tiles, pl.splits);
  return 1;
}

}  // namespace dg

extern "C" {

int dg_quant_mxfp4(const void* x, int dtype, uint8_t* q, int32_t* sf, const int32_t* row_token, int64_t G, int64_t T,
                   int64_t R, int64_t K, void* stream) {
  int rc = check_quant(dtype, G, R, K);
  if (rc) return rc;
  if (T < 0 || T > kIntMax) return fail(DG_ERR_SHAPE, "T out of range");
  if (G == 0 || R == 0) return ok();
  if (!q || !sf || (!x && (T > 0 || !row_token))) return fail(DG_ERR_INVALID_ARG, "null pointer");
  if (!aligned(x, 16) || !aligned(q, 16)) return fail(DG_ERR_ALIGN, "x and q must be 16-byte aligned");
  if (!aligned(sf, 4) || !aligned(row_token, 4)) return fail(DG_ERR_ALIGN, "sf and row_token must be 4-byte aligned");
  int cus = 0;
  if ((rc = check_device(&cus))) return rc;
  return launched(launch_quant_mxfp4(x, dtype == DG_BF16, q, sf, row_token, G, T, R, K, hs(stream)));
}

int dg_dequant_mxfp4(const uint8_t* q, const int32_t* sf, void* y, int dtype, int64_t G, int64_t R, int64_t K, void* stream) {
  int rc = check_quant(dtype, G, R, K);
  if (rc) return rc;
  if (G == 0 || R == 0) return ok();
  if (!q || !sf || !y) return fail(DG_ERR_INVALID_ARG, "null pointer");
  if (!aligned(y, 16) || !aligned(q, 16)) return fail(DG_ERR_ALIGN, "q and y must be 16-byte aligned");
  if (!aligned(sf, 4)) return fail(DG_ERR_ALIGN, "sf must be 4-byte aligned");
  int cus = 0;
  if ((rc = check_device(&cus))) return rc;
  return launched(launch_dequant_mxfp4(q, sf, y, dtype == DG_BF16, G, R, K, hs(stream)));
}

int dg_mxfp4_gemm_nt(const uint8_t* A, const int32_t* sfa, const uint8_t* B, const int32_t* sfb, uint16_t* D, int64_t M,
                     int64_t N, int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  return run_mx(kMxDense, A, sfa, B, sfb, D, nullptr, M, N, K, 1, workspace, workspace_bytes, stream);
}

int dg_m_grouped_mxfp4_gemm_nt_contiguous(const uint8_t* A, const int32_t* sfa, const uint8_t* B, const int32_t* sfb,
                                          uint16_t* D, const int32_t* m_indices, int64_t M_total, int64_t N, int64_t K,
                                          int64_t G, void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  return run_mx(kMxContiguous, A, sfa, B, sfb, D, m_indices, M_total, N, K, G, nullptr, 0, stream);
}

int dg_m_grouped_mxfp4_gemm_nt_masked(const uint8_t* A, const int32_t* sfa, const uint8_t* B, const int32_t* sfb, uint16_t* D,
                                      const int32_t* masked_m, int64_t G, int64_t max_m, int64_t N, int64_t K,
                                      int64_t expected_m, void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  (void)expected_m;
  return run_mx(kMxMasked, A, sfa, B, sfb, D, masked_m, max_m, N, K, G, nullptr, 0, stream);
}

int dg_moe_gate(const void* logits, int dtype, const uint8_t* valid, int32_t* topk_idx, float* topk_w, int32_t* counts,
                float* prob_sum, float* loss, int64_t T, int64_t E, int64_t k, int renorm, float w_scale, float loss_coef,
                void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_gate(dtype, T, E, k, w_scale);
  if (rc) return rc;
  if (!counts || !prob_sum || !loss || (T > 0 && (!logits || !topk_idx || !topk_w)))
    return fail(DG_ERR_INVALID_ARG, "null pointer");
  if (!aligned(logits, 16)) return fail(DG_ERR_ALIGN, "logits must be 16-byte aligned");
  if (!aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(counts, 4) || !aligned(prob_sum, 4) || !aligned(loss, 4))
    return fail(DG_ERR_ALIGN, "outputs must be 4-byte aligned");
  const size_t need = gate_workspace_bytes(T, E);
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < need)
    return fail(DG_ERR_WORKSPACE, "a 16-byte aligned workspace of at least %zu bytes is needed", need);
  int cus = 0;
  if ((rc = check_device(&cus))) return rc;
  GateParams p{logits, valid, topk_idx, topk_w, counts, prob_sum, loss, workspace, T, (int)E, (int)k, renorm, w_scale, loss_coef};
  return launched(launch_gate(p, dtype == DG_BF16, hs(stream)));
}

int dg_moe_gate_bwd(const void* logits, int dtype, const int32_t* topk_idx, const float* topk_w, const int32_t* counts,
                    const float* dw, const float* dloss, void* dlogits, int64_t T, int64_t E, int64_t k, int renorm,
                    float w_scale, float loss_coef, void* stream) {
  int rc = check_gate(dtype, T, E, k, w_scale);
  if (rc) return rc;
  if (T == 0) return ok();
  if (!logits || !topk_idx || !topk_w || !counts || !dlogits) return fail(DG_ERR_INVALID_ARG, "null pointer");
  if (!aligned(logits, 16) || !aligned(dlogits, 16)) return fail(DG_ERR_ALIGN, "logits and dlogits must be 16-byte aligned");
  if (!aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(counts, 4) || !aligned(dw, 4) || !aligned(dloss, 4))
    return fail(DG_ERR_ALIGN, "index and gradient arrays must be 4-byte aligned");
  int cus = 0;
  if ((rc = check_device(&cus))) return rc;
  GateBwdParams p{logits, topk_idx, topk_w, counts, dw, dloss, dlogits, T, (int)E, (int)k, renorm, w_scale, loss_coef};
  return launched(launch_gate_bwd(p, dtype == DG_BF16, hs(stream)));
}

int dg_moe_layout_contiguous(const int32_t* topk_idx, int32_t* counts, int32_t* m_indices, int32_t* row_token, int32_t* row_of,
                             int64_t T, int64_t k, int64_t first_expert, int64_t G, int64_t M_total, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return run_layout(topk_idx, counts, m_indices, row_token, row_of, T, k, first_expert, G, 0, M_total, workspace,
                    workspace_bytes, stream);
}

int dg_moe_layout_masked(const int32_t* topk_idx, int32_t* masked_m, int32_t* row_token, int32_t* row_of, int64_t T, int64_t k,
                         int64_t first_expert, int64_t G, int64_t max_m, void* workspace, size_t workspace_bytes,
                         void* stream) {
  if (max_m < 1 || max_m > kIntMax || G > kMaxGroups) return fail(DG_ERR_SHAPE, "max_m must be >= 1 and G at most 1024");
  return run_layout(topk_idx, masked_m, nullptr, row_token, row_of, T, k, first_expert, G, max_m, G * max_m, workspace,
                    workspace_bytes, stream);
}

int dg_moe_combine(const uint16_t* rows, const int32_t* row_of, const float* w, void* y, int dtype, int64_t T, int64_t k,
                   int64_t N, int64_t R, void* stream) {
  int rc = check_combine(dtype, T, k, N, R);
  if (rc) return rc;
  if (T == 0) return ok();
  if ((!rows && R > 0) || !row_of || !w || !y) return fail(DG_ERR_INVALID_ARG, "null pointer");
  if (!aligned(rows, 16) || !aligned(y, 16)) return fail(DG_ERR_ALIGN, "rows and y must be 16-byte aligned");
  if (!aligned(row_of, 4) || !aligned(w, 4)) return fail(DG_ERR_ALIGN, "row_of and w must be 4-byte aligned");
  int cus = 0;
  if ((rc = check_device(&cus))) return rc;
  return launched(launch_combine(rows, row_of, w, y, dtype == DG_BF16, T, k, N, R, hs(stream)));
}

int dg_moe_combine_bwd(const void* dy, int dtype, const uint16_t* rows, const int32_t* row_of, const float* w, uint16_t* drows,
                       float* dw, int64_t T, int64_t k, int64_t N, int64_t R, void* stream) {
  int rc = check_combine(dtype, T, k, N, R);
  if (rc) return rc;
  if (T == 0) return ok();
  if (!dy || (R > 0 && (!rows || !drows)) || !row_of || !w || !dw) return fail(DG_ERR_INVALID_ARG, "null pointer");
  if (!aligned(rows, 16) || !aligned(dy, 16) || !aligned(drows, 16))
    return fail(DG_ERR_ALIGN, "dy, rows and drows must be 16-byte aligned");
  if (!aligned(row_of, 4) || !aligned(w, 4) || !aligned(dw, 4)) return fail(DG_ERR_ALIGN, "row_of, w and dw must be 4-byte aligned");
  int cus = 0;
  if ((rc = check_device(&cus))) return rc;
  return launched(launch_combine_bwd(dy, dtype == DG_BF16, rows, row_of, w, drows, dw, T, k, N, R, hs(stream)));
}

}  // extern "C"
