// Large products of microscaled 4-bit operands for gfx950 (the operation of
// mxfp4_gemm.hip): a persistent workgroup of four waves, one per SIMD, walks
// 256 x 256 output tiles.
//
// Each wave holds 128 x 128 of the tile: 8 x 8 accumulators of
// v_mfma_scale_f32_16x16x128_f8f6f4 in the 256 accumulation registers, so a
// step of 256 K elements reads (128 + 128) x 128 bytes of LDS for 128 matrix
// instructions.  Eight waves of 64 x 128 would read half as much again, and
// LDS reads plus the writes of the loads would then take as many cycles as the
// matrix instructions do.  With one wave per SIMD nothing hides a wait, so the
// operands of a half step (128 K elements, 64 matrix instructions) are read
// during the half step before it, a few instructions after each
// matrix instruction:
//
//   matrix instructions   first half of j | second half of j | first half of j + 1
//   LDS reads             second half of j | first half of j + 1
//   barrier                              ^
//
// At the barrier every wave has step j's operands in registers and its loads
// of step j + 1 have landed, so the slot of step j is free for step j + 2 and
// two slots (136 KB) keep a whole step of loads in flight.
//
// Contiguous form: only aligned 128-row blocks hold rows of one expert, so a
// tile whose two blocks belong to different experts is two passes.  Every
// workgroup lists its passes (tile, expert, rows tagged with it) in LDS first.

#include <utility>

#include "dg_internal.hpp"
#include "gemm_common.hpp"
#include "moe_internal.hpp"

namespace dg {
namespace {

constexpr int kMwRsrcWord3 = 0x00020000;  // raw (untyped) buffer
constexpr uint32_t kMwOOB = 0xFFFFFF00u;  // an offset past every buffer range used here

typedef int mwi32x4 __attribute__((ext_vector_type(4)));

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

template <int FORM>
__global__ void __launch_bounds__(256, 1) mxfp4_wide_kernel(MxGemmParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool CONTIG = FORM == kMxContiguous;
  constexpr int BM = 256, BN = 256, NW = 4;
  constexpr int INS = BM / 8 / NW;  // 1 KB (8-row) loads per wave, step and operand
  constexpr int S_INS = 2 * (BM + BN) / 64 / NW;
  constexpr int SLOT_S = (BM + BN) * 128;
  constexpr int SLOT = SLOT_S + 2 * (BM + BN) * 4;
  constexpr int MAXT = kMxWideMaxTiles;
  __shared__ __attribute__((aligned(1024))) uint8_t slot0[SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t slot1[SLOT];
  __shared__ int pass_tile[CONTIG ? 2 * MAXT : 1];
  __shared__ int pass_exp[CONTIG ? 2 * MAXT : 1];
  __shared__ unsigned long long pass_mask[CONTIG ? 2 * MAXT : 1][4];  // tagged rows, 64 a word
  __shared__ int tile_np[CONTIG ? MAXT + 1 : 1];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1;
  const int wn = wave & 1;
  const int q = lane >> 4;
  const int q16 = lane & 15;
  const int N = p.N;
  const int kbytes = p.K >> 1;
  const int KB = p.K >> 7;
  const int steps = (KB + 3) >> 2 << 1;  // of 256 elements, even: a last one past K is zeros
  const int64_t M = p.rows;
  const int T = p.m_tiles * p.n_tiles;
  const int G = (int)gridDim.x;
  const int bid = (int)blockIdx.x;
  const int n_tiles = bid < T ? (T - bid + G - 1) / G : 0;  // tiles of this workgroup
  if (n_tiles == 0) return;
  auto tile_mn = [&](int s, int* mt, int* nt) { grouped_mn(round_tile(bid, s, G, T), p.m_tiles, p.n_tiles, 4, mt, nt); };

  int nseg = n_tiles;
  if constexpr (CONTIG) {
    // experts of the tile's two 128-row blocks (-1: no tagged row) and the lane's four rows
    auto experts = [&](int s, int* x, int* e) {
      int mt, nt;
      tile_mn(s, &mt, &nt);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t r = (int64_t)mt * BM + 64 * k + lane;
        const int v = r < M ? p.index[r] : -1;
        x[k] = v >= 0 && v < p.G ? v : -1;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int v = x[2 * h] > x[2 * h + 1] ? x[2 * h] : x[2 * h + 1];
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
          const int u = __shfl_xor(v, o);
          v = u > v ? u : v;
        }
        e[h] = v;
      }
      return (e[0] >= 0 ? 1 : 0) + (e[1] >= 0 && e[1] != e[0] ? 1 : 0);
    };
    for (int s = wave; s < n_tiles; s += NW) {
      int x[4], e[2];
      const int n = experts(s, x, e);
      if (lane == 0) tile_np[s] = n;
    }
    __syncthreads();
    if (wave == 0) {  // exclusive prefix (n_tiles <= MAXT = 64)
      const int own = lane < n_tiles ? tile_np[lane] : 0;
      int c = own;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(c, o);
        if (lane >= o) c += u;
      }
      if (lane < n_tiles) tile_np[lane] = c - own;
      if (lane == 63) tile_np[MAXT] = c;
    }
    __syncthreads();
    for (int s = wave; s < n_tiles; s += NW) {
      int x[4], e[2];
      const int n = experts(s, x, e);
      const int first = tile_np[s];
      for (int i = 0; i < n; ++i) {
        const int ex = i == 0 && e[0] >= 0 ? e[0] : e[1];
        unsigned long long m[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = __ballot(x[k] == ex);
        if (lane == 0) {
          pass_tile[first + i] = s;
          pass_exp[first + i] = ex;
#pragma unroll
          for (int k = 0; k < 4; ++k) pass_mask[first + i][k] = m[k];
        }
      }
    }
    __syncthreads();
    nseg = __builtin_amdgcn_readfirstlane(tile_np[MAXT]);
    if (nseg == 0) return;  // only padding
  }

  // ---- loads.  A 1 KB load fills 8 LDS rows: lane l writes row l / 8, position l % 8, from K chunk (l % 8) ^ (l / 8).
  // Wave w fills rows 64 w + 8 i of A and of B in load i; B's row 64 w + in holds the column that makes a lane's
  // outputs consecutive.  A lane's offset is fixed for the whole kernel and everything else is in the scalar offset,
  // which the range check includes: rows past the tile's end read as zeros.  Past K a row runs into the next one
  // (or the end, zeros), but its scale words there are past their range and read as 2^-127: against another 2^-127
  // no product is left in fp32, so neither a half step nor a whole one past K adds anything.
  const int l8 = lane >> 3;
  const int chunk = (lane & 7) ^ l8;
  const uint32_t a_off = (uint32_t)(64 * wave + l8) * (uint32_t)kbytes + 16u * chunk;
  const uint32_t b_off = (uint32_t)(64 * wave + 16 * (l8 >> 2) + (l8 & 3)) * (uint32_t)kbytes + 16u * chunk;
  // scale words of rows 64 w + lane, B's in LDS row order
  const uint32_t sa_off = 4u * (uint32_t)tid;
  const uint32_t sb_off = 4u * (uint32_t)(64 * wave + 16 * (q16 >> 2) + 4 * q + (q16 & 3));
  __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
  int is_seg = 0;
  auto is_setup = [&]() MW_INLINE {
    int mt, nt, e = 0;
    if constexpr (CONTIG) {
      tile_mn(__builtin_amdgcn_readfirstlane(pass_tile[is_seg]), &mt, &nt);
      e = __builtin_amdgcn_readfirstlane(pass_exp[is_seg]);
    } else {
      tile_mn(is_seg, &mt, &nt);
    }
    const int64_t row0 = (int64_t)mt * BM;
    const int rows = M - row0 < BM ? (int)(M - row0) : BM;
    const int n0 = nt * BN;
    const int cols = N - n0 < BN ? N - n0 : BN;
    ra = mw_rsrc(p.A + row0 * kbytes, (uint32_t)rows * (uint32_t)kbytes);
    rb = mw_rsrc(p.B + ((int64_t)e * N + n0) * kbytes, (uint32_t)cols * (uint32_t)kbytes);
    rsa = mw_rsrc(p.sfa + row0, ((uint32_t)(KB - 1) * (uint32_t)M + (uint32_t)rows) * 4u);
    rsb = mw_rsrc(p.sfb + (int64_t)e * N * KB + n0, ((uint32_t)(KB - 1) * (uint32_t)N + (uint32_t)cols) * 4u);
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
                                               (int)((uint32_t)(2 * k + (i >> 1)) * 4u * (uint32_t)(i & 1 ? (int64_t)N : M)), 0, 0);
    }
  };

  // ---- LDS reads.  Lane group q = lane / 16 holds blocks 2 q (first half) and 2 q + 1 (second half) of a step's eight:
  // their scale bytes are neighbours and one 2-byte read serves both halves.
  const uint32_t fr0 = (uint32_t)(q16 * 128 + (((2 * q) ^ (lane & 7)) << 4));
  const uint32_t fr1 = (uint32_t)(q16 * 128 + (((2 * q + 1) ^ (lane & 7)) << 4));
  const uint32_t a_base = (uint32_t)(wm * 128 * 128);
  const uint32_t b_base = (uint32_t)(BM * 128 + wn * 128 * 128);
  const uint32_t s_base = (uint32_t)(SLOT_S + (q >> 1) * (BM + BN) * 4 + q16 * 4 + 2 * (q & 1));
  const uint32_t sa_base = s_base + (uint32_t)(wm * 128 * 4);
  const uint32_t sb_base = s_base + (uint32_t)((BM + wn * 128) * 4);
  // operands in the order the matrix instructions need them (A's tiles within the first eight, B's one per eight):
  // b 0, a 0-7, b 1-7
  auto read = [&](const uint8_t* sl, uint32_t fr, int n, Half& f) MW_INLINE {
    if (n == 0) f.b[0] = *reinterpret_cast<const uint4*>(sl + b_base + fr);
    else if (n < 9) f.a[n - 1] = *reinterpret_cast<const uint4*>(sl + a_base + fr + (n - 1) * 2048);
    else f.b[n - 8] = *reinterpret_cast<const uint4*>(sl + b_base + fr + (n - 8) * 2048);
  };
  auto read_scale = [&](const uint8_t* sl, int n, Scales& s) MW_INLINE {
    if (n & 1) s.a[n >> 1] = *reinterpret_cast<const uint16_t*>(sl + sa_base + (n >> 1) * 64);
    else s.b[n >> 1] = *reinterpret_cast<const uint16_t*>(sl + sb_base + (n >> 1) * 64);
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

  int cp_seg = 0;
  Half f0, f1;    // first and second half
  Scales sc[2];   // of the steps in the two slots

  auto store = [&]() MW_INLINE {
    settle();
    int mt, nt;
    unsigned long long tag[2] = {~0ull, ~0ull};
    if constexpr (CONTIG) {
      tile_mn(__builtin_amdgcn_readfirstlane(pass_tile[cp_seg]), &mt, &nt);
      tag[0] = pass_mask[cp_seg][2 * wm];
      tag[1] = pass_mask[cp_seg][2 * wm + 1];
    } else {
      tile_mn(cp_seg, &mt, &nt);
    }
    const int64_t row0 = (int64_t)mt * BM + wm * 128;
    const int col0 = nt * BN + wn * 128 + q * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 16 * i + q16;
      bool ok = row0 + r < M;
      if constexpr (CONTIG) ok = ok && ((tag[i >> 2] >> (r & 63)) & 1ull);
      uint16_t* dst = p.D + (row0 + r) * (int64_t)N;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int c = col0 + 64 * g;
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 v = acc[i][4 * g + j];
          w[2 * j] = pack_bf16x2(v[0], v[1]);
          w[2 * j + 1] = pack_bf16x2(v[2], v[3]);
          acc[i][4 * g + j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        if (ok && c < N) {  // N is a multiple of 16
          *reinterpret_cast<uint4*>(dst + c) = uint4{w[0], w[1], w[2], w[3]};
          *reinterpret_cast<uint4*>(dst + c + 8) = uint4{w[4], w[5], w[6], w[7]};
        }
      }
    }
    settle();
  };

  // one step in slot st; the loads of step k at the issue pointer follow into it
  auto step = [&](auto st, int k) MW_INLINE {
    constexpr int own = decltype(st)::value;
    constexpr int other = 1 - own;
    const uint8_t* slo = slot(st);
    const uint8_t* sln = slot(Const<other>{});
    unrolled<64>([&](auto c) MW_INLINE {
      constexpr int n = decltype(c)::value;
      mfma(Const<0>{}, f0, sc[own], n & 7, n >> 3);
      if constexpr (n < 48 && n % 3 == 0) read(slo, fr1, n / 3, f1);
      __builtin_amdgcn_sched_barrier(0);
    });
    wait_vmcnt<0>();   // this wave's loads of the next step have landed
    wait_lgkmcnt0();   // and its reads of this one returned
    __builtin_amdgcn_s_barrier();
    unrolled<64>([&](auto c) MW_INLINE {
      constexpr int n = decltype(c)::value;
      mfma(Const<1>{}, f1, sc[own], n & 7, n >> 3);
      if constexpr (n < 16) read_scale(sln, n, sc[other]);
      else if constexpr (n < 48 && n % 2 == 0) read(sln, fr0, (n - 16) / 2, f0);
      if constexpr ((n & 1) && n / 2 < LOADS) issue(st, k, Const<n / 2>{});
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  settle();
  unrolled<LOADS>([&](auto c) MW_INLINE { issue(Const<0>{}, 0, c); });
  unrolled<LOADS>([&](auto c) MW_INLINE { issue(Const<1>{}, 1, c); });
  wait_vmcnt<LOADS>();
  __builtin_amdgcn_s_barrier();
  unrolled<16>([&](auto c) MW_INLINE { read_scale(slot0, decltype(c)::value, sc[0]); });
  unrolled<16>([&](auto c) MW_INLINE { read(slot0, fr0, decltype(c)::value, f0); });
  for (; cp_seg < nseg; ++cp_seg) {
    int k = 2;  // steps issued of the tile at the issue pointer
    for (int j = 0; j < steps; j += 2) {
      if (j + 2 == steps) {  // the next loads are the next tile's (after the last tile: its own again, read by none)
        k = 0;
        if (++is_seg < nseg) is_setup();
      }
      step(Const<0>{}, k);
      step(Const<1>{}, k + 1);
      k += 2;
    }
    store();
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
