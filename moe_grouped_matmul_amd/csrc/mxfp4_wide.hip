// Large products of microscaled 4-bit operands for gfx950 (the operation of
// mxfp4_gemm.hip), dense and contiguous: a persistent workgroup of four waves,
// one per SIMD, walks output tiles of 256 x 256 and then of 128 x 256.
//
// A wave holds 128 rows of the tile and 128 of its columns (256 x 256) or 64
// (128 x 256): 8 x 8 or 8 x 4 accumulators of v_mfma_scale_f32_16x16x128_f8f6f4
// in the accumulation registers.  For the large tile a step of 256 K elements
// reads (128 + 128) x 128 bytes of LDS per 128 matrix instructions.  With one
// wave per SIMD nothing hides a wait, so the operands of a half step (128 K
// elements) are read during the half step before it, a few instructions after
// each matrix instruction:
//
//   matrix instructions   first half of j | second half of j | first half of j + 1
//   LDS reads             second half of j | first half of j + 1
//   barrier                              ^
//
// At the barrier every wave has step j's operands in registers and its loads
// of step j + 1 have landed, so the slot of step j is free for step j + 2 and
// two slots (136 KB) keep a whole step of loads in flight.
//
// Measured (4096 x 4096 x 7168): 3050 cycles a step, of which the matrix cores
// are busy 2048 and the waves wait 130, at a clock of 1.9 GHz.  32 x 32 x 64
// instructions take 2850 cycles a step at 1.7 GHz and the same time: the clock
// follows the power, and that is what bounds the kernel.
//
// Tiles.  Contiguous: only aligned 128-row blocks hold rows of one expert (of
// several in a block the largest is computed, as in every other tile shape), so
// every workgroup reads m_indices at its start and pairs the blocks of each run
// of one expert from the run's first block on; an odd one is a tile of 128
// rows.  Dense: a last tile of up to 128 rows.  The large tiles are walked in
// rounds of one per workgroup; the tiles of a last, partial round and the small
// ones go to the workgroups with the least work, the former cut in two where
// everything left then fits one round of small tiles, and small ones that fill
// half a round or less are cut once more, into 128 x 128 quarters.  A quarter's
// step is short against the latency of its loads, so its slots hold two steps
// (rows 128 on are the same rows further along K) and it meets a barrier every
// other one.  Measured, 8 experts x 16384 rows, 4096 x 7168: 276 us without
// quarters, 270 with quarters of one step a slot, 267 us (3.6 PFLOP/s); 8192
// rows 163, 156, 148; one expert of 4352 rows 78, 74.5, 67.  Reading all of
// m_indices with half a wave a block against a thread's first row of each and a
// wave for the rest: 16384 rows 251 -> 248 us in even segments, 262144 rows of
// 8 experts, 512 x 256, 214 -> 141.
#include <utility>

#include "dg_internal.hpp"
#include "gemm_common.hpp"
#include "moe_internal.hpp"

namespace dg {
namespace {

constexpr int kMwRsrcWord3 = 0x00020000;  // raw (untyped) buffer

typedef int mwi32x4 __attribute__((ext_vector_type(4)));
typedef int mwi32x4u __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mw_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, kMwRsrcWord3);
}

// the loop bodies below are inlined whole, so that their arrays stay in registers
#define MW_INLINE __attribute__((always_inline))

template <int V>
struct Const {
  static constexpr int value = V;
};

template <class F, int... I>
__device__ __forceinline__ void each(F&& f, std::integer_sequence<int, I...>) {
  (f(Const<I>{}), ...);
}
// f(0), ..., f(N - 1) with constant arguments
template <int N, class F>
__device__ __forceinline__ void unrolled(F&& f) {
  each(f, std::make_integer_sequence<int, N>{});
}

// operands of one half step: 16 bytes per lane and 16-row tile
struct Half {
  uint4 a[8], b[8];
};
// scales of one step: the lane's two blocks of each row, first half in byte 0, second in byte 1
struct Scales {
  int a[8], b[8];
};

constexpr int kNone = 0xFFFF;

// maximum with the lane that DPP control C exchanges with
template <int C>
__device__ __forceinline__ uint32_t dpp_max(uint32_t u) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, C, 0xf, 0xf, true);
  return o > u ? o : u;
}

template <int FORM>
__global__ void __launch_bounds__(256, 1) mxfp4_wide_kernel(MxGemmParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool CONTIG = FORM == kMxContiguous;
  constexpr int BM = 256, BN = 256, NW = 4;
  constexpr int INS = BM / 8 / NW;  // 1 KB (8-row) loads per wave, step and operand
  constexpr int S_INS = 2 * (BM + BN) / 64 / NW;
  constexpr int SLOT_S = (BM + BN) * 128;
  constexpr int SLOT = SLOT_S + 2 * (BM + BN) * 4;
  constexpr int MAXB = CONTIG ? kMxWideMaxBlocks : 1;
  __shared__ __attribute__((aligned(1024))) uint8_t slot0[SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t slot1[SLOT];
  __shared__ uint16_t expert_of[MAXB];  // contiguous: of each 128-row block
  __shared__ uint16_t large_at[MAXB], small_at[MAXB];  // first blocks of the tiles
  __shared__ int listed[2];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4;
  const int q16 = lane & 15;
  const int N = p.N;
  const int kbytes = p.K >> 1;
  const int KB = p.K >> 7;
  const int steps = (KB + 3) >> 2 << 1;  // of 256 elements, even: a last one past K is zeros
  const int64_t M = p.rows;
  const uint32_t ld = (uint32_t)p.sfa_ld;
  const int n_tiles = p.n_tiles;
  const int G = (int)gridDim.x;
  const int bid = (int)blockIdx.x;

  // row tiles: large ones and small ones
  int n_large, n_small;
  if constexpr (CONTIG) {
    const int nb = (int)((M + 127) >> 7);
    // a block's expert is the largest index in [0, G) among its rows; half a wave reads a block, 16 blocks of a wave in flight
    const int sub = lane & 31;
    for (int b1 = 2 * wave; b1 < nb; b1 += 16 * NW) {
      const int b0 = b1 + (lane >> 5);
      mwi32x4u x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t r = (int64_t)(b0 + 2 * NW * i) * 128 + 4 * sub;
        x[i] = mwi32x4u{-1, -1, -1, -1};
        if (r + 3 < M) x[i] = *reinterpret_cast<const mwi32x4u*>(p.index + r);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int b = b0 + 2 * NW * i;
        uint32_t top = 0;  // the index + 1
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t v = (uint32_t)x[i][k] < (uint32_t)p.G ? (uint32_t)x[i][k] + 1u : 0u;
          top = v > top ? v : top;
        }
        top = dpp_max<0xB1>(top);   // pairs of lanes
        top = dpp_max<0x4E>(top);   // pairs of pairs
        top = dpp_max<0x141>(top);  // the quads of eight
        top = dpp_max<0x140>(top);  // the eights of sixteen
        const auto both = __builtin_amdgcn_permlane16_swap(top, top, false, false);
        top = both[0] > both[1] ? both[0] : both[1];
        if (sub == 0 && b < nb) expert_of[b] = (uint16_t)(top ? top - 1u : kNone);
      }
    }
    __syncthreads();
    if (tid == 0) {  // the rows past the last four whole ones
      int e = expert_of[nb - 1] == kNone ? -1 : (int)expert_of[nb - 1];
      for (int64_t r = M & ~(int64_t)3; r < M; ++r) {
        const int v = p.index[r];
        if (v < p.G && v > e) e = v;
      }
      expert_of[nb - 1] = (uint16_t)(e < 0 ? kNone : e);
    }
    __syncthreads();
    if (wave == 0) {
      int run = 0, nl = 0, ns = 0;  // first block of the current run, tiles so far
      for (int b0 = 0; b0 < nb; b0 += 64) {
        const int b = b0 + lane;
        const int e = b < nb ? expert_of[b] : kNone;
        const int before = b > 0 && b < nb ? expert_of[b - 1] : kNone;
        const int after = b + 1 < nb ? expert_of[b + 1] : kNone;
        int first = e != before || b == 0 ? b : -1;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int u = __shfl_up(first, o);
          if (lane >= o && u > first) first = u;
        }
        if (first < 0) first = run;  // the run began in an earlier group of blocks
        run = __shfl(first, 63);
        const bool heads = e != kNone && ((b - first) & 1) == 0;
        const unsigned long long below = (1ull << lane) - 1ull;
        const unsigned long long ml = __ballot(heads && after == e);
        const unsigned long long ms = __ballot(heads && after != e);
        if ((ml >> lane) & 1ull) large_at[nl + __popcll(ml & below)] = (uint16_t)b;
        if ((ms >> lane) & 1ull) small_at[ns + __popcll(ms & below)] = (uint16_t)b;
        nl += __popcll(ml);
        ns += __popcll(ms);
      }
      if (lane == 0) {
        listed[0] = nl;
        listed[1] = ns;
      }
    }
    __syncthreads();
    n_large = __builtin_amdgcn_readfirstlane(listed[0]);
    n_small = __builtin_amdgcn_readfirstlane(listed[1]);
  } else {
    n_large = (int)((M + 127) >> 8);  // a rest of up to 128 rows is a small tile
    n_small = (M & 255) >= 1 && (M & 255) <= 128 ? 1 : 0;
  }

  // tiles of this workgroup: whole rounds of large ones, then what is left
  const int T = n_large * n_tiles;
  const int rounds = T / G;
  const int rest = T - rounds * G;
  const bool cut = rest > 0 && 2 * rest + n_small * n_tiles <= G;
  const int S = n_small * n_tiles + (cut ? 2 * rest : 0);  // small tiles, the halves of the cut ones last
  const int own_large = rounds + (!cut && bid < rest ? 1 : 0);
  const bool spread = rest > 0 && !cut;  // workgroups without a tile of the last round take two small ones first
  auto small_id = [&](int i) MW_INLINE {
    if (!spread) return bid + i * G;
    if (bid < rest) return 2 * (G - rest) + bid + i * G;
    return i < 2 ? bid - rest + i * (G - rest) : 2 * (G - rest) + bid + (i - 2) * G;
  };
  // of the small tiles that do not fill a round, 128 x 128 quarters where those fit one
  const int free = spread ? 2 * (G - rest) : 0;
  const int last = S > free ? (S - free) % G : 0;
  const int whole_small = 2 * last <= G ? S - last : S;
  int own_small = 0;
  while (small_id(own_small) < whole_small) ++own_small;
  const int pieces = own_large + own_small;
  const int units = pieces + (bid < 2 * (S - whole_small) ? 1 : 0);
  if (units == 0) return;
  // unit u: first row, rows, first column, columns, expert
  auto unit = [&](int u, int64_t* row0, int* rows, int* n0, int* cols, int* e) MW_INLINE {
    const bool quarter = u >= pieces;
    int b, blocks = 2, tile;
    int* nt = &tile;
    if (u < own_large) {
      int mt;
      grouped_mn(round_tile(bid, u, G, T), n_large, n_tiles, 4, &mt, nt);
      b = CONTIG ? (int)large_at[CONTIG ? mt : 0] : 2 * mt;
    } else {
      const int i = quarter ? whole_small + (bid >> 1) : small_id(u - own_large);
      blocks = 1;
      if (i < n_small * n_tiles) {
        const int st = i / n_tiles;
        *nt = i - st * n_tiles;
        b = CONTIG ? (int)small_at[CONTIG ? st : 0] : 2 * n_large;
      } else {
        const int c = i - n_small * n_tiles;
        int mt;
        grouped_mn(rounds * G + (c >> 1), n_large, n_tiles, 4, &mt, nt);
        b = (CONTIG ? (int)large_at[CONTIG ? mt : 0] : 2 * mt) + (c & 1);
      }
    }
    b = __builtin_amdgcn_readfirstlane(b);
    *row0 = (int64_t)b * 128;
    const int64_t left = M - *row0;
    *rows = left < blocks * 128 ? (left < 0 ? 0 : (int)left) : blocks * 128;
    *n0 = tile * BN + (quarter ? 128 * (bid & 1) : 0);
    const int width = quarter ? 128 : BN;
    *cols = N - *n0 < width ? N - *n0 : width;
    *e = CONTIG ? __builtin_amdgcn_readfirstlane((int)expert_of[CONTIG ? b : 0]) : 0;
  };

  // ---- loads.  A 1 KB load fills 8 LDS rows: lane l writes row l / 8, position l % 8, from K chunk 2 p % 8 + p / 4 with
  // p = (l % 8) ^ (l / 8): even chunks, one per lane group of a read, lie in one half of a row's positions and odd ones in
  // the other, without which a read takes twice its cycles (two lanes to a bank).
  // Wave w fills rows 64 w + 8 i of A and of B in load i; B's row 64 w + in holds the column that makes a lane's
  // outputs consecutive.  A lane's offset is fixed for the whole kernel and everything else is in the scalar offset,
  // which the range check includes: rows past the tile's end read as zeros.  Past K a row runs into the next one
  // (or the end, zeros), but its scale words there are past their range and read as 2^-127: against another 2^-127
  // no product is left in fp32, so neither a half step nor a whole one past K adds anything.
  const int l8 = lane >> 3;
  const int pos = (lane & 7) ^ l8;
  const int chunk = (pos & 3) << 1 | pos >> 2;
  // Of a quarter the waves 2 and 3 fill rows 128 on with the same rows' next step: two steps to a slot.
  uint32_t a_off, b_off, sa_off, sb_off;
  int stride = 1;  // steps in a slot, of the unit at the issue pointer
  auto lane_offsets = [&](int w, int ahead) MW_INLINE {
    a_off = (uint32_t)(64 * w + l8) * (uint32_t)kbytes + 16u * chunk + 128u * ahead;
    b_off = (uint32_t)(64 * w + 16 * (l8 >> 2) + (l8 & 3)) * (uint32_t)kbytes + 16u * chunk + 128u * ahead;
    // scale words of rows 64 w + lane, B's in LDS row order
    sa_off = 4u * (uint32_t)(64 * w + lane) + 8u * ahead * ld;
    sb_off = 4u * (uint32_t)(64 * w + 16 * (q16 >> 2) + 4 * q + (q16 & 3)) + 8u * ahead * (uint32_t)N;
  };
  lane_offsets(wave, 0);
  __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
  int is_seg = 0;
  int64_t row0 = 0;  // of the unit at the issue pointer
  int rows = 0, n0 = 0, e = 0;
  auto is_setup = [&]() MW_INLINE {
    int cols;
    unit(is_seg, &row0, &rows, &n0, &cols, &e);
    if (is_seg >= pieces) {
      stride = 2;
      lane_offsets(wave & 1, wave >> 1);
    }
    ra = mw_rsrc(p.A + row0 * kbytes, (uint32_t)rows * (uint32_t)kbytes);
    if (cols < 0) cols = 0;  // the second quarter of a narrow last tile
    rb = mw_rsrc(p.B + ((int64_t)e * N + n0) * kbytes, (uint32_t)cols * (uint32_t)kbytes);
    rsa = mw_rsrc(p.sfa + row0, ((uint32_t)(KB - 1) * ld + (uint32_t)rows) * 4u);
    rsb = mw_rsrc(p.sfb + (int64_t)e * N * KB + n0, cols ? ((uint32_t)(KB - 1) * (uint32_t)N + (uint32_t)cols) * 4u : 0u);
  };
  is_setup();

  auto slot = [&](auto st) MW_INLINE -> uint8_t* {
    if constexpr (decltype(st)::value == 0) return slot0;
    else return slot1;
  };
  constexpr int LOADS = 2 * INS + S_INS;
  // load n of step k of the tile at the issue pointer into slot st
  auto issue = [&](auto st, int k, auto nc) MW_INLINE {
    constexpr int n = decltype(nc)::value;
    uint8_t* sl = slot(st);
    if constexpr (n < INS) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (DG_LDS void*)(sl + wave * 8192 + n * 1024), 16, a_off,
                                               (k << 7) + 8 * n * kbytes, 0, 0);
    } else if constexpr (n < 2 * INS) {
      constexpr int i = n - INS;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (DG_LDS void*)(sl + BM * 128 + wave * 8192 + i * 1024), 16, b_off,
                                               (k << 7) + (32 * (i & 1) + 4 * (i >> 1)) * kbytes, 0, 0);
    } else {
      constexpr int i = n - 2 * INS;  // half i / 2 of A (even i) or B
      constexpr int at = SLOT_S + (i >> 1) * (BM + BN) * 4 + (i & 1) * BM * 4;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(i & 1 ? rsb : rsa, (DG_LDS void*)(sl + at + wave * 256), 4, i & 1 ? sb_off : sa_off,
                                               (int)((uint32_t)(2 * k + (i >> 1)) * 4u * (i & 1 ? (uint32_t)N : ld)), 0, 0);
    }
  };

  // ---- LDS reads.  Lane group q = lane / 16 holds blocks 2 q (first half) and 2 q + 1 (second half) of a step's eight:
  // their scale bytes are neighbours and one 2-byte read serves both halves.
  const uint32_t fr0 = (uint32_t)(q16 * 128 + ((q ^ (lane & 7)) << 4));
  const uint32_t fr1 = (uint32_t)(q16 * 128 + (((q + 4) ^ (lane & 7)) << 4));
  // the wave's first LDS row of A and of B: (128 rows, 128 columns) of a large tile, (all 128 rows, 64
  // columns) of a small one, (all 128 rows, 32 columns) of a quarter
  const uint32_t s_base = (uint32_t)(SLOT_S + (q >> 1) * (BM + BN) * 4 + q16 * 4 + 2 * (q & 1));
  auto a_row = [&](auto tn) MW_INLINE -> int { return decltype(tn)::value == 8 ? (wave >> 1) * 128 : 0; };
  auto b_row = [&](auto tn) MW_INLINE -> int { return decltype(tn)::value == 8 ? (wave & 1) * 128 : wave * 8 * decltype(tn)::value * 2; };
  // operands of TN column tiles in the order the matrix instructions need them (A's tiles within the first eight, B's one
  // per eight): b 0, a 0-7, b 1-
  auto read = [&](auto tn, const uint8_t* sl, uint32_t fr, int n, Half& f, int row = 0) MW_INLINE {
    const uint8_t* a = sl + (row + a_row(tn)) * 128 + fr;
    const uint8_t* b = sl + (row + BM + b_row(tn)) * 128 + fr;
    if (n == 0) f.b[0] = *reinterpret_cast<const uint4*>(b);
    else if (n < 9) f.a[n - 1] = *reinterpret_cast<const uint4*>(a + (n - 1) * 2048);
    else f.b[n - 8] = *reinterpret_cast<const uint4*>(b + (n - 8) * 2048);
  };
  // scale n < TN of B, then of A
  auto read_scale = [&](auto tn, const uint8_t* sl, int n, Scales& s, int row = 0) MW_INLINE {
    constexpr int TN = decltype(tn)::value;
    if (n < TN) s.b[n] = *reinterpret_cast<const uint16_t*>(sl + s_base + (row + BM + b_row(tn)) * 4 + n * 64);
    else s.a[n - TN] = *reinterpret_cast<const uint16_t*>(sl + s_base + (row + a_row(tn)) * 4 + (n - TN) * 64);
  };

  f32x4 acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // In place on the accumulation registers (left to the compiler, part of the accumulators ends in vector registers
  // and is copied back and forth every step).  An accumulator is used again 64 matrix instructions later, past every
  // wait state; settle() stands between matrix instructions and other accesses of the accumulators.
  auto mfma = [&](auto hc, const Half& f, const Scales& s, int i, int j) MW_INLINE {
    const uint4 a = f.a[i], b = f.b[j];
    const mwi32x4 av{(int)a.x, (int)a.y, (int)a.z, (int)a.w}, bv{(int)b.x, (int)b.y, (int)b.z, (int)b.w};
    f32x4& c = acc[i][j];
    const int ws = s.b[j], xs = s.a[i];
    if constexpr (decltype(hc)::value == 0)  // scales in byte 0
      asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                   : "+a"(c) : "v"(bv), "v"(av), "v"(ws), "v"(xs));
    else  // in byte 1
      asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                   : "+a"(c) : "v"(bv), "v"(av), "v"(ws), "v"(xs));
  };
  auto settle = []() MW_INLINE {
    asm volatile("s_nop 15\n\ts_nop 15");
    __builtin_amdgcn_sched_barrier(0);
  };

  int cp = 0;  // unit being computed
  Half f0, f1;    // first and second half of a step
  Scales sc[2];   // of the steps in the two slots

  // the lane's rows to store (bit i: row 16 i + l % 16 of the wave's) and where; taken while the tile is still at the
  // issue pointer, before its last steps
  uint32_t st_rows = 0;
  int64_t st_row = 0;
  int st_col = 0;
  auto place = [&](auto tn) MW_INLINE {
    const int r0 = a_row(tn) + q16;
    st_rows = 0;
    st_row = row0 + r0;
    // a quarter's wave has two of the four column tiles whose outputs are consecutive
    st_col = n0 + q * 16 + (decltype(tn)::value == 2 ? (wave >> 1) * 64 + (wave & 1) * 8 : b_row(tn));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bool ok = r0 + 16 * i < rows;
      // contiguous: only the rows tagged with the tile's expert
      if constexpr (CONTIG) ok = ok && p.index[ok ? st_row + 16 * i : 0] == e;
      st_rows |= ok ? 1u << i : 0u;
    }
  };
  auto store = [&](auto tn) MW_INLINE {
    constexpr int TN = decltype(tn)::value;
    settle();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint16_t* dst = p.D + (st_row + 16 * i) * (int64_t)N;
#pragma unroll
      for (int g = 0; g < TN / 4; ++g) {
        const int c = st_col + 64 * g;
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 v = acc[i][4 * g + j];
          w[2 * j] = pack_bf16x2(v[0], v[1]);
          w[2 * j + 1] = pack_bf16x2(v[2], v[3]);
          acc[i][4 * g + j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        if (((st_rows >> i) & 1u) && c < N) {  // N is a multiple of 16
          *reinterpret_cast<uint4*>(dst + c) = uint4{w[0], w[1], w[2], w[3]};
          *reinterpret_cast<uint4*>(dst + c + 8) = uint4{w[4], w[5], w[6], w[7]};
        }
      }
      if constexpr (TN == 2) {
        const f32x4 u = acc[i][0], v = acc[i][1];
        if (((st_rows >> i) & 1u) && st_col < N)
          *reinterpret_cast<uint4*>(dst + st_col) = uint4{pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
    }
    settle();
  };

  // one step in slot st over TN column tiles; the loads of step k at the issue pointer follow into it
  auto step = [&](auto tn, auto st, int k) MW_INLINE {
    constexpr int TN = decltype(tn)::value;
    constexpr int own = decltype(st)::value;
    constexpr int other = 1 - own;
    constexpr int NM = 8 * TN;   // matrix instructions of a half step
    constexpr int NR = 8 + TN;   // operand reads of a half step, and scale reads of a step
    const uint8_t* slo = slot(st);
    const uint8_t* sln = slot(Const<other>{});
    unrolled<NM>([&](auto c) MW_INLINE {
      constexpr int n = decltype(c)::value;
      mfma(Const<0>{}, f0, sc[own], n & 7, n >> 3);
      constexpr int every = TN == 8 ? 3 : 2;
      if constexpr (n < every * NR && n % every == 0) read(tn, slo, fr1, n / every, f1);
      __builtin_amdgcn_sched_barrier(0);
    });
    wait_vmcnt<0>();   // this wave's loads of the next step have landed
    wait_lgkmcnt0();   // and its reads of this one returned
    __builtin_amdgcn_s_barrier();
    unrolled<NM>([&](auto c) MW_INLINE {
      constexpr int n = decltype(c)::value;
      mfma(Const<1>{}, f1, sc[own], n & 7, n >> 3);
      if constexpr (n < NR) read_scale(tn, sln, n, sc[other]);
      if constexpr (TN == 8) {
        if constexpr (n >= 16 && n < 48 && n % 2 == 0) read(tn, sln, fr0, (n - 16) / 2, f0);
        if constexpr ((n & 1) && n / 2 < LOADS) issue(st, k, Const<n / 2>{});
      } else {
        if constexpr (n >= NR && n < 2 * NR) read(tn, sln, fr0, n - NR, f0);
        if constexpr (n < LOADS) issue(st, k, c);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // the two steps in slot st of a quarter
  auto quarter_step = [&](auto st, int k) MW_INLINE {
    constexpr Const<2> tn;
    constexpr int own = decltype(st)::value;
    constexpr int other = 1 - own;
    constexpr int NM = 16, NR = 10;
    const uint8_t* slo = slot(st);
    const uint8_t* sln = slot(Const<other>{});
    Scales s2;
    unrolled<NM>([&](auto c) MW_INLINE {
      constexpr int n = decltype(c)::value;
      mfma(Const<0>{}, f0, sc[own], n & 7, n >> 3);
      if constexpr (n < NR) {
        read(tn, slo, fr1, n, f1);
        read_scale(tn, slo, n, s2, 128);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    unrolled<NM>([&](auto c) MW_INLINE {
      constexpr int n = decltype(c)::value;
      mfma(Const<1>{}, f1, sc[own], n & 7, n >> 3);
      if constexpr (n < NR) read(tn, slo, fr0, n, f0, 128);
      __builtin_amdgcn_sched_barrier(0);
    });
    unrolled<NM>([&](auto c) MW_INLINE {
      constexpr int n = decltype(c)::value;
      mfma(Const<0>{}, f0, s2, n & 7, n >> 3);
      if constexpr (n < NR) read(tn, slo, fr1, n, f1, 128);
      __builtin_amdgcn_sched_barrier(0);
    });
    wait_vmcnt<0>();
    wait_lgkmcnt0();
    __builtin_amdgcn_s_barrier();
    unrolled<NM>([&](auto c) MW_INLINE {
      constexpr int n = decltype(c)::value;
      mfma(Const<1>{}, f1, s2, n & 7, n >> 3);
      issue(st, k, c);
      if constexpr (n + NM < LOADS) issue(st, k, Const<n + NM>{});
      if constexpr (n < NR) {
        read_scale(tn, sln, n, sc[other]);
        read(tn, sln, fr0, n, f0);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // first operands of a unit whose step 0 is in slot 0
  auto begin = [&](auto tn) MW_INLINE {
    constexpr int NR = 8 + decltype(tn)::value;
    unrolled<NR>([&](auto c) MW_INLINE { read_scale(tn, slot0, decltype(c)::value, sc[0]); });
    unrolled<NR>([&](auto c) MW_INLINE { read(tn, slot0, fr0, decltype(c)::value, f0); });
  };
  auto walk = [&](auto tn, int end) MW_INLINE {
    for (; cp < end; ++cp) {
      constexpr int per = decltype(tn)::value == 2 ? 4 : 2;  // steps in the two slots
      int k = per;  // steps issued of the tile at the issue pointer
      for (int j = 0; j < steps; j += per) {
        if (j + per >= steps) {  // the next loads are the next tile's (after the last tile: its own again, read by none)
          k = 0;
          place(tn);
          if (++is_seg < units) is_setup();
        }
        if constexpr (per == 4) {
          quarter_step(Const<0>{}, k);
          quarter_step(Const<1>{}, k + stride);
        } else {
          step(tn, Const<0>{}, k);
          step(tn, Const<1>{}, k + stride);
        }
        k += 2 * stride;
      }
      store(tn);
    }
  };

  settle();
  unrolled<LOADS>([&](auto c) MW_INLINE { issue(Const<0>{}, 0, c); });
  unrolled<LOADS>([&](auto c) MW_INLINE { issue(Const<1>{}, stride, c); });
  wait_vmcnt<LOADS>();
  __builtin_amdgcn_s_barrier();
  if (own_large > 0) {
    begin(Const<8>{});
    walk(Const<8>{}, own_large);
  }
  if (own_small > 0) {  // step 0 of the first small tile landed before the last barrier
    begin(Const<4>{});
    walk(Const<4>{}, pieces);
  }
  if (units > pieces) {
    begin(Const<2>{});
    walk(Const<2>{}, units);
  }
  wait_vmcnt<0>();  // no LDS writes in flight past this point
#endif
}

}  // namespace

hipError_t launch_mxfp4_wide(int form, int grid, const MxGemmParams& p, hipStream_t stream) {
  if (form == kMxContiguous)
    hipLaunchKernelGGL(mxfp4_wide_kernel<kMxContiguous>, dim3((unsigned)grid), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(mxfp4_wide_kernel<kMxDense>, dim3((unsigned)grid), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dg
