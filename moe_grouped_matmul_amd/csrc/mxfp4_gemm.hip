// Products of microscaled 4-bit operands for gfx950: D = A . B^T in bf16,
//   D[i, j] = sum_b 2^(ea[i, b] + eb[j, b] - 254) sum_{k < 32} a[i, 32 b + k] * w[j, 32 b + k]
// with e2m1 elements (two to a byte, the lower nibble first) and one
// power-of-two exponent byte per 32 elements of a row, four to a 32-bit word.
// Dense, M-grouped contiguous (one expert per aligned 128-row block) and
// M-grouped masked (masked_m[g] rows of each expert) forms.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes 32 elements (16 bytes) of one row
// from each lane and that block's exponent byte beside them, so a lane's
// operand is one aligned 16-byte chunk and its scale one byte, and products
// are accumulated in fp32 over the whole K range.  A product of two e2m1 values
// has at most 6 significant bits, so a block's 32 products add without loss.
// Where blocks of different scale meet, and with the accumulator, 24 bits are
// kept: a 1 beside 2^23 survives, inside one instruction and across two, a 1
// beside 2^24 does not, so sums that fit 24 bits are exact in any order.
//
// Organisation: a workgroup computes one BM x BN tile.  K advances in steps
// of 256 elements, 128 bytes per operand row, through a ring of P LDS slots
// that buffer-to-LDS loads fill P - 1 steps ahead; one barrier a step
// publishes slot j and frees slot j - 1.  A slot holds BM rows of A, BN rows
// of B (16-byte chunk c of a row at position c ^ (row % 8), so the 16 rows of
// one operand read lie on distinct banks) and their scale words of the step's
// two 128-element halves.  The weights are the row operand of the MFMA and
// their rows are permuted inside a wave's columns, so a lane ends with up to
// 16 consecutive output columns of one row.
//
// Two tiles.  128 x 256 (8 waves, 3 slots, one workgroup a CU) reads each
// weight once where an expert has up to 128 rows: 32 experts x 128 rows, 2048
// in all, 4096 x 7168, 94 us, 5.5 TB/s of weights, rows and output, which is
// above the card's large copy.  64 x 64 (4 waves, 4 slots, two workgroups a
// CU) occupies the CUs where large tiles are few; it is bound by the latency of
// its few steps: 64 x 7168 x 2048 6.2 us (7.8 MB of weights, which stay in the
// Infinity Cache between calls; an empty launch takes 2.5), 512 x 4096 x 4096
// 11.4 us.  K is split where that leaves CUs idle and the sum of the parts, by
// the last workgroup of a tile, costs less than it saves.  Large dense and
// contiguous products run on the persistent tiles of mxfp4_wide.hip.

#include "dg_internal.hpp"
#include "gemm_common.hpp"
#include "moe_internal.hpp"

namespace dg {
namespace {

constexpr int kMxRsrcWord3 = 0x00020000;  // raw (untyped) buffer
constexpr uint32_t kMxOOB = 0xFFFFFF00u;  // an offset past every buffer range used here
constexpr int kMxCoherent = 16;           // sc1: split-K partials, coherent across the XCDs
constexpr int kMxStream = 2;              // nt: weights that one workgroup reads once

typedef unsigned int mxu32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, kMxRsrcWord3);
}

template <int V>
struct Const {
  static constexpr int value = V;
};

template <int BM, int BN, int WM, int WN, int P, int FORM, bool NT>
__global__ void __launch_bounds__(64 * WM * WN) mxfp4_gemm_kernel(MxGemmParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM / 16;          // 16-row tiles of a wave
  constexpr int TN = BN / WN / 16;          // 16-column tiles of a wave
  constexpr int TG = TN < 4 ? TN : 4;       // column tiles whose outputs are one run of 4 TG columns
  constexpr int A_INS = BM / 8 / NW;        // 1 KB (8-row) loads per wave and step
  constexpr int B_INS = BN / 8 / NW;
  constexpr int SROWS = BM + BN;            // scale words per 128-element half
  constexpr int S_INS = (2 * SROWS / 64 + NW - 1) / NW;  // 64-word loads per wave and step
  constexpr int L_STEP = A_INS + B_INS + S_INS;
  static_assert(A_INS >= 1 && B_INS >= 1 && BM % 64 == 0 && BN % 64 == 0, "tile shape");
  static_assert((P - 1) * L_STEP < 64, "vmcnt range");
  constexpr int SLOT_S = SROWS * 128;  // scale words after the operand rows
  constexpr int SLOT = SLOT_S + S_INS * NW * 256;

  __shared__ __attribute__((aligned(1024))) uint8_t slot0[SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t slot1[SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t slot2[P > 2 ? SLOT : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t slot3[P > 3 ? SLOT : 16];
  __shared__ int last_split;
  auto slot = [&](auto st) -> uint8_t* {
    constexpr int i = decltype(st)::value;
    if constexpr (i == 0) return slot0;
    else if constexpr (i == 1) return slot1;
    else if constexpr (i == 2) return slot2;
    else return slot3;
  };

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN;
  const int wn = wave % WN;
  const int q = lane >> 4;
  const int q16 = lane & 15;
  const int bid = (int)blockIdx.x;

  // workgroup -> (row tile, column tile, split or expert)
  int mt, nt, split = 0, e = 0;
  if constexpr (FORM == kMxContiguous) {
    grouped_mn(xcd_tile(bid, p.m_tiles * p.n_tiles), p.m_tiles, p.n_tiles, 8, &mt, &nt);
  } else if (FORM == kMxDense && p.m_tiles > 1 && p.splits == 1) {
    grouped_mn(xcd_tile(bid, p.m_tiles * p.n_tiles), p.m_tiles, p.n_tiles, 4, &mt, &nt);
  } else {
    // the row tiles of one (column tile, split | expert) unit are 8 ids apart:
    // the same XCD under round-robin dispatch, sharing the unit's weights
    const int r8 = bid >> 3;
    mt = r8 % p.m_tiles;
    const int unit = (r8 / p.m_tiles) * 8 + (bid & 7);
    const int per = FORM == kMxMasked ? p.G : p.splits;
    if (unit >= p.n_tiles * per) return;  // padding of the grid to 8 units
    if (FORM == kMxMasked) {
      e = unit / p.n_tiles;
      nt = unit - e * p.n_tiles;
    } else {
      split = unit % p.splits;
      nt = unit / p.splits;
    }
  }

  const int N = p.N;
  const int kbytes = p.K >> 1;  // bytes per operand row
  const int KB = p.K >> 7;      // scale words per row
  const int64_t ld = p.rows;    // rows of A (of one expert)
  int rows = (int)(p.rows - (int64_t)mt * BM < BM ? p.rows - (int64_t)mt * BM : BM);
  int64_t row0 = (int64_t)mt * BM;
  const uint8_t* A = p.A;
  const int32_t* sfa = p.sfa;
  uint16_t* D = p.D;
  unsigned long long tag[2] = {~0ull, ~0ull};  // contiguous: rows of the block's expert
  if constexpr (FORM == kMxMasked) {
    int m = p.index[e];
    m = m < 0 ? 0 : (m > (int)p.rows ? (int)p.rows : m);
    if (m <= mt * BM) return;
    rows = m - mt * BM < BM ? m - mt * BM : BM;
    A += (int64_t)e * ld * kbytes;
    sfa += (int64_t)e * ld * KB;
    D += (int64_t)e * ld * N;
  }
  if constexpr (FORM == kMxContiguous) {
    static_assert(128 % BM == 0, "a contiguous tile lies in one aligned block");
    const int64_t block = row0 & ~(int64_t)127;
    int x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = block + 64 * h + lane;
      x[h] = r < p.rows ? p.index[r] : -1;
      if (x[h] >= p.G) x[h] = -1;
    }
    int top = x[0] > x[1] ? x[0] : x[1];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const int y = __shfl_xor(top, o);
      top = y > top ? y : top;
    }
    e = __builtin_amdgcn_readfirstlane(top);
    if (e < 0) return;  // only padding: nothing to write
    tag[0] = __ballot(x[0] == e);
    tag[1] = __ballot(x[1] == e);
    if (BM == 64) {
      tag[0] = tag[(row0 >> 6) & 1];
      if (tag[0] == 0ull) return;  // this half is padding
    }
  }
  const int n0 = nt * BN;
  const int cols = N - n0 < BN ? N - n0 : BN;
  const int steps = (KB + 1) >> 1;
  const int s_lo = FORM == kMxDense ? split * p.steps_per_split : 0;
  const int s_hi = FORM == kMxDense && s_lo + p.steps_per_split < steps ? s_lo + p.steps_per_split : steps;
  const int nsteps = s_hi - s_lo;

  const uint8_t* Bt = p.B + ((int64_t)e * N + n0) * kbytes;
  const int32_t* sbt = p.sfb + (int64_t)e * N * KB + n0;
  const int32_t* sat = sfa + row0;
  const uint8_t* At = A + row0 * kbytes;
  const uint32_t a_bytes = (uint32_t)rows * (uint32_t)kbytes;
  const uint32_t b_bytes = (uint32_t)cols * (uint32_t)kbytes;

  // Loads.  Every 1 KB operand load fills 8 LDS rows: lane l writes row l / 8,
  // position l % 8, from K chunk (l % 8) ^ (l / 8).  Rows past the tile's end
  // lie past the buffer range and read as zeros.
  const int chunk = (lane & 7) ^ (lane >> 3);
  uint32_t a_off[A_INS], b_off[B_INS], s_off[S_INS];
#pragma unroll
  for (int i = 0; i < A_INS; ++i) {
    const int r = 8 * (i * NW + wave) + (lane >> 3);
    a_off[i] = r < rows ? (uint32_t)r * (uint32_t)kbytes + 16u * chunk : kMxOOB;
  }
#pragma unroll
  for (int i = 0; i < B_INS; ++i) {
    // LDS row r of B holds the weight row that makes a lane's outputs consecutive
    const int r = 8 * (i * NW + wave) + (lane >> 3);
    const int in = r % (16 * TN), j = in / 16, ii = in % 16;
    const int c = r - in + (j / TG) * (16 * TG) + (ii >> 2) * 4 * TG + 4 * (j % TG) + (ii & 3);
    b_off[i] = c < cols ? (uint32_t)c * (uint32_t)kbytes + 16u * chunk : kMxOOB;
  }
  // scale words: 64-word group s of a step is half s / (SROWS / 64), rows
  // 64 (s % (SROWS / 64)) + lane of A then B (B in LDS row order)
#pragma unroll
  for (int i = 0; i < S_INS; ++i) {
    const int s = i * NW + wave;
    const int r = 64 * (s % (SROWS / 64)) + lane;
    if (r < BM) {
      s_off[i] = r < rows ? 4u * r : kMxOOB;
    } else {
      const int rb = r - BM;
      const int in = rb % (16 * TN), j = in / 16, ii = in % 16;
      const int c = rb - in + (j / TG) * (16 * TG) + (ii >> 2) * 4 * TG + 4 * (j % TG) + (ii & 3);
      s_off[i] = c < cols ? 4u * c : kMxOOB;
    }
    if (s >= 2 * SROWS / 64) s_off[i] = kMxOOB;
  }
  // the second half of the last step lies past K where K is an odd number of halves
  const bool odd = KB & 1;

  auto issue = [&](auto st, int j) {
    uint8_t* sl = slot(st);
    const bool in = j < nsteps;
    const int step = s_lo + j;
    const bool half = odd && step == steps - 1;
    const uint32_t past = half && chunk >= 4 ? kMxOOB : 0u;  // chunks past K: out of range, zeros
    const __amdgpu_buffer_rsrc_t ra = mx_rsrc(At, in ? a_bytes : 0u);
    const __amdgpu_buffer_rsrc_t rb = mx_rsrc(Bt, in ? b_bytes : 0u);
    const int ks = in ? step << 7 : 0;
#pragma unroll
    for (int i = 0; i < A_INS; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (DG_LDS void*)(sl + (i * NW + wave) * 1024), 16, a_off[i] | past, ks, 0, 0);
#pragma unroll
    for (int i = 0; i < B_INS; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (DG_LDS void*)(sl + BM * 128 + (i * NW + wave) * 1024), 16, b_off[i] | past, ks,
                                               0, NT ? kMxStream : 0);
#pragma unroll
    for (int i = 0; i < S_INS; ++i) {
      const int s = i * NW + wave;  // uniform
      const int h = s / (SROWS / 64);
      const bool isb = 64 * (s % (SROWS / 64)) >= BM;
      const bool live = in && !(half && h == 1) && h < 2;
      // the word row of this half as a buffer of its own, so no offset passes 32 bits
      const int64_t kb = live ? 2 * (int64_t)step + h : 0;
      const __amdgpu_buffer_rsrc_t rs = isb ? mx_rsrc(sbt + kb * N, live ? (uint32_t)cols * 4u : 0u)
                                            : mx_rsrc(sat + kb * ld, live ? (uint32_t)rows * 4u : 0u);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (DG_LDS void*)(sl + SLOT_S + s * 256), 4, s_off[i], 0, 0, 0);
    }
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // operand reads: row 16 t + lane % 16, chunk 4 h + q; scale byte q of the row's word
  const uint32_t fr[2] = {(uint32_t)(q16 * 128 + ((q ^ (lane & 7)) << 4)), (uint32_t)(q16 * 128 + (((q + 4) ^ (lane & 7)) << 4))};
  const uint32_t a_row = (uint32_t)(wm * TM * 16);
  const uint32_t b_row = (uint32_t)(wn * TN * 16);

  auto compute = [&](auto st) {
    const uint8_t* sl = slot(st);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x8 af[TM], bf[TN];
      int sa[TM], sb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(sl + a_row * 128 + i * 2048 + fr[h]);
        af[i] = i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
        sa[i] = sl[SLOT_S + h * SROWS * 4 + (a_row + 16 * i + q16) * 4 + q];
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const uint4 v = *reinterpret_cast<const uint4*>(sl + BM * 128 + b_row * 128 + j * 2048 + fr[h]);
        bf[j] = i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
        sb[j] = sl[SLOT_S + h * SROWS * 4 + (BM + b_row + 16 * j + q16) * 4 + q];
      }
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[j], af[i], acc[i][j], 4, 4, 0, sb[j], 0, sa[i]);
    }
  };

  auto step = [&](auto st, int j) {
    constexpr int nx = (decltype(st)::value + P - 1) % P;
    wait_vmcnt<(P - 2) * L_STEP>();  // this wave's loads of step j have landed
    wait_lgkmcnt0();                 // and its reads of step j - 1 returned
    __builtin_amdgcn_s_barrier();
    issue(Const<nx>{}, j + P - 1);
    compute(st);
  };

  issue(Const<0>{}, 0);
  if constexpr (P > 2) issue(Const<1>{}, 1);
  if constexpr (P > 3) issue(Const<2>{}, 2);
  // the step count is padded to whole ring cycles; padding steps load zeros and add nothing
  for (int j = 0; j < nsteps; j += P) {
    step(Const<0>{}, j);
    step(Const<1>{}, j + 1);
    if constexpr (P > 2) step(Const<2>{}, j + 2);
    if constexpr (P > 3) step(Const<3>{}, j + 3);
  }
  wait_vmcnt<0>();  // no LDS writes in flight past this point

  if constexpr (FORM == kMxDense) {
    if (p.splits > 1) {
      // Partials in fragment order, written and read with sc1 (coherent at
      // agent scope); every wave waits until its stores are acknowledged
      // before the barrier that precedes the counter's increment, and the
      // last split reads only after its increment returned.  The splits are
      // added in the order 0, 1, 2, ..., whichever ends last.
      const int tiles = p.m_tiles * p.n_tiles;
      const int tile = mt * p.n_tiles + nt;
      constexpr uint32_t FB = TM * TN * 1024u;  // one wave's fragments
      uint8_t* base = reinterpret_cast<uint8_t*>(p.ws) + kMxCounterBytes;
      const int64_t split_bytes = (int64_t)tiles * NW * FB;
      const int64_t own = ((int64_t)tile * NW + wave) * FB;
      {
        const __amdgpu_buffer_rsrc_t rw = mx_rsrc(base + split * split_bytes + own, FB);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(mxu32x4, acc[i][j]), rw,
                                                   (uint32_t)((i * TN + j) * 1024 + lane * 16), 0, kMxCoherent);
      }
      wait_vmcnt<0>();
      __syncthreads();
      unsigned int* counters = reinterpret_cast<unsigned int*>(p.ws);
      if (tid == 0)
        last_split = __hip_atomic_fetch_add(&counters[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                     (unsigned int)(p.splits - 1);
      __syncthreads();
      if (!last_split) return;
      for (int s = 0; s < p.splits; ++s) {
        const __amdgpu_buffer_rsrc_t rw = mx_rsrc(base + s * split_bytes + own, FB);
        f32x4 t[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            t[i][j] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                    rw, (uint32_t)((i * TN + j) * 1024 + lane * 16), 0, kMxCoherent));
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = s == 0 ? t[i][j] : acc[i][j] + t[i][j];
      }
      if (tid == 0)  // ready for the next call on this workspace
        __hip_atomic_store(&counters[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }

  // bf16 store: lane l holds row 16 i + l % 16 and columns 4 TG q + [0, 4 TG)
  // of each run of 16 TG columns
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = (int)a_row + 16 * i + q16;
    bool ok = r < rows;
    if constexpr (FORM == kMxContiguous) ok = ok && ((tag[r >> 6] >> (r & 63)) & 1ull);
    if (!ok) continue;
    uint16_t* dst = D + (row0 + r) * (int64_t)N + n0;
#pragma unroll
    for (int g = 0; g < TN / TG; ++g) {
      const int c = (int)b_row + g * 16 * TG + q * 4 * TG;
      if (c >= cols) continue;  // N and n0 are multiples of 16, so a run of 4 TG columns is inside or outside
#pragma unroll
      for (int j = 0; j < TG; ++j) {
        uint2 o;
        o.x = pack_bf16x2(acc[i][g * TG + j][0], acc[i][g * TG + j][1]);
        o.y = pack_bf16x2(acc[i][g * TG + j][2], acc[i][g * TG + j][3]);
        *reinterpret_cast<uint2*>(dst + c + 4 * j) = o;
      }
    }
  }
#endif
}

template <int BM, int BN, int WM, int WN, int P, int FORM>
hipError_t launch_mx(const MxGemmParams& p, hipStream_t stream) {
  int64_t grid;
  if (FORM == kMxContiguous || (FORM == kMxDense && p.m_tiles > 1 && p.splits == 1)) {
    grid = (int64_t)p.m_tiles * p.n_tiles;
  } else {
    const int64_t units = (int64_t)p.n_tiles * (FORM == kMxMasked ? p.G : p.splits);
    grid = (units + 7) / 8 * 8 * p.m_tiles;
  }
  if (FORM != kMxContiguous && p.stream_weights)
    hipLaunchKernelGGL((mxfp4_gemm_kernel<BM, BN, WM, WN, P, FORM, FORM != kMxContiguous>), dim3((unsigned)grid),
                       dim3(64 * WM * WN), 0, stream, p);
  else
    hipLaunchKernelGGL((mxfp4_gemm_kernel<BM, BN, WM, WN, P, FORM, false>), dim3((unsigned)grid), dim3(64 * WM * WN), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

size_t mx_workspace_bytes(int tile, int m_tiles, int n_tiles, int splits) {
  if (splits <= 1) return 0;
  return kMxCounterBytes + (size_t)splits * m_tiles * n_tiles * mx_bm(tile) * mx_bn(tile) * 4;
}

hipError_t launch_mxfp4_gemm(int form, int tile, const MxGemmParams& p, hipStream_t stream) {
  if (form == kMxContiguous)
    return tile == kMx64x64 ? launch_mx<64, 64, 1, 4, 4, kMxContiguous>(p, stream)
                            : launch_mx<128, 256, 2, 4, 3, kMxContiguous>(p, stream);
  if (form == kMxMasked)
    return tile == kMx64x64 ? launch_mx<64, 64, 1, 4, 4, kMxMasked>(p, stream)
                            : launch_mx<128, 256, 2, 4, 3, kMxMasked>(p, stream);
  return tile == kMx64x64 ? launch_mx<64, 64, 1, 4, 4, kMxDense>(p, stream)
                          : launch_mx<128, 256, 2, 4, 3, kMxDense>(p, stream);
}

}  // namespace dg
