// mx_tile.h -- the MXFP4 tile product of the 4-bit expert GEMMs.
//
// A tile computes D[n][t] = sum_k Wt[n][k] * X[t][k] for BW weight rows n and
// BT token rows t, both operands MXFP4, fp32 accumulation.  K is walked in
// ascending steps of 128, one v_mfma_scale_f32_16x16x128_f8f6f4 per 16 x 16
// block and step, never split, so an element's bits depend on its own weight
// row and token row only (the library's batch invariance), whichever of the
// tiles below computes it.
//
// A 16-row fragment of a 128-wide K step is 1 KiB, as a bf16 fragment of a
// 32-wide step is, and one matrix instruction takes as long: direct-to-LDS
// loads of 16 bytes a lane and conflict-free 16-byte reads, as in gemm_tile.h,
// with every byte carrying four times the elements.  What is new are the
// scales.  They travel through LDS with the data, because vmcnt counts in
// order: a scale loaded to registers one step ahead would wait for every
// later stage of the prefetch as well.
//
// MxWide (many rows an expert, matrix bound): BW = 256 or 128 by 128 tokens,
//   8 wavefronts, all operands in 3 stages of one K step, two workgroups a
//   CU.  Both operands are read in fragment layout: the token rows are
//   gathered once in sorted order before the first product (and the first
//   product writes the second's operand that way), because at this rate a K
//   step of a CU is 0.43 us and token lines of two steps, as the bf16 tile
//   gathers them, do not fit LDS far enough ahead.  A 256 x 256 tile with one
//   workgroup a CU moves a third fewer bytes, but a CU had nothing to
//   multiply while it started or ended a tile, and 2.25 such tiles a CU (16
//   experts of about 1024 rows, 2048 weight rows) take the time of three
//   (that layer's two products: 165 and 90 us with token lines, 129 and 82
//   with fragments, 95 and 73 with this tile; 4 wavefronts of 128 x 64 in its
//   place 105 and 74; 81 and 73 with a step's LDS reads all under way before
//   its products).  What binds it: the matrix units are busy 39% and 19% of
//   the time, LDS 24% and 17%; loads and barriers without reads and products
//   take 61 and 67 us, and the two parts overlap only in part.  Storing y
//   costs the second product 25 us.  The next tile's loads issued before the
//   epilogue, y stored without the LDS stage: no gain.
// MxStream (a few rows an expert, bound by the weights' bytes): 128 x 64, 4
//   wavefronts of 64 x 32, token rows gathered by the tile, all operands in 4
//   stages of one K step; three workgroups a CU, so that some load while
//   another starts or ends a tile (128 tokens on 32 experts of d = 7168, I =
//   2048: two workgroups with 5 stages took 115 and 56 us for the two
//   products, three with 4 stages 111 and 51; tiles of 128 rows, which read
//   the weights of an expert of more than 64 rows once, 112 and 83).
#pragma once

#include "gemm_tile.h"
#include "mxfp4.h"

namespace moe {

// The thread's index, opaque to the compiler: what an epilogue derives from
// it is then computed there.  Hoisted out of the tile loop, those addresses
// stay live across the K loop, whose registers are all in use (measured: 372
// bytes a lane of scratch, the second product 363 instead of 80 us).
__device__ __forceinline__ int opaque_tid() {
  int v = static_cast<int>(threadIdx.x);
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ void lds_dma4(const void* g, void* l) { __builtin_amdgcn_global_load_lds(g, l, 4, 0, 0); }

template <int BW_>
struct MxWide {
  static constexpr bool STREAM = false;
  static constexpr int PER_CU = 2;  // workgroups
  static constexpr int BW = BW_, BT = 128, WR = BW / 64, WT = 8 / WR, NW = 8, NTHREADS = 512;
  static constexpr int AW = BW / WR / 16, AT = BT / WT / 16;
  static constexpr int NST = 3, LW = BW / 16 / NW, LT = BT / 16 / NW, LS = 1;
  static constexpr int NQ = BW / 64, NQT = BT / 64;  // 64-row groups of weight and token scales
  static constexpr int T0 = BW * 64, S0 = T0 + BT * 64, STAGE = S0 + (NQ + NQT) * 256;
  static constexpr size_t LDS_BYTES = static_cast<size_t>(NST) * STAGE;
  static_assert(AW == 4 && (AT == 4 || AT == 2) && LW >= 1 && LT >= 1 && NQ + NQT <= NW, "wave tile, loads");
  static_assert(PER_CU * (LDS_BYTES + 2304) <= 160 * 1024, "two workgroups a CU, with their tables");
};

struct MxStream {
  static constexpr bool STREAM = true;
  static constexpr int PER_CU = 3;
  static constexpr int BW = 128, BT = 64, WR = 2, WT = 2, NW = 4, NTHREADS = 256;
  static constexpr int AW = BW / WR / 16, AT = BT / WT / 16;
  static constexpr int NST = 4, LW = BW / 16 / NW, LT = BT / 16 / NW;
  static constexpr int NQ = BW / 64;
  static constexpr int LS = 1;
  static constexpr int T0 = BW * 64, S0 = T0 + BT * 64, STAGE = S0 + NQ * 256 + BT * 4;
  static constexpr size_t LDS_BYTES = static_cast<size_t>(NST) * STAGE;
  static_assert(NQ == 2 && BT == 64 && NW == 4, "one scale load a wavefront and step");
  static_assert((NST - 2) * (LW + LT + LS) <= 63, "vmcnt");
  static_assert(PER_CU * (LDS_BYTES + 1280) <= 160 * 1024, "three workgroups a CU, with their tables");
};

// wave-uniform, kept in scalar registers
__device__ __forceinline__ int mx_wave() { return uniform(wave_id()); }
template <class C>
__device__ __forceinline__ int mx_wr() { return mx_wave() % C::WR; }
template <class C>
__device__ __forceinline__ int mx_wt() { return mx_wave() / C::WR; }

template <class C>
struct MxAcc {
  f32x4 v[C::AW][C::AT];
};

// Global addresses of a tile's operands: wave-uniform, but for the gathered
// token rows of MxStream.
struct MxWideSrc {
  const uint8_t* w;      // first weight fragment of the tile
  const uint8_t* t;      // first token fragment
  const uint8_t* scale;  // scale words this wavefront loads (weights or tokens)
  int KB;                // K steps
};
template <class C>
struct MxStreamSrc {
  const uint8_t* w;
  const uint8_t* tok[C::LT];
  const uint8_t* scale;
  int KB;
};

// MxWide: wcodes, wscales: the matrix's codes and scales, nt: tile along its
// rows; tcodes, tscales: the token matrix in the same layout, row0: the
// tile's first row in it (a multiple of 64).
template <class C>
__device__ __forceinline__ MxWideSrc mx_wide_src(const uint8_t* wcodes, const uint8_t* wscales, int K, int nt,
                                                 const uint8_t* tcodes, const uint8_t* tscales, int row0) {
  MxWideSrc s;
  s.KB = K / 128;
  const size_t fstep = static_cast<size_t>(s.KB) * 1024, qstep = static_cast<size_t>(mx_kq(K)) * 1024;
  s.w = wcodes + static_cast<size_t>(nt) * (C::BW / 16) * fstep;
  s.t = tcodes + static_cast<size_t>(row0 / 16) * fstep;
  // scale groups: the weights', the tokens', and again from the first for the
  // wavefronts left over
  const int g = mx_wave() % (C::NQ + C::NQT);
  s.scale = g < C::NQ ? wscales + static_cast<size_t>(nt * C::NQ + g) * qstep
                       : tscales + static_cast<size_t>(row0 / 64 + g - C::NQ) * qstep;
  return s;
}

// MxStream: row(r): index of tile row r in the token matrix (valid for r <
// count); tcodes, tscales: token codes and scales with row strides.
template <class C, class Row>
__device__ __forceinline__ void mx_stream_src(MxStreamSrc<C>& s, const uint8_t* wcodes, const uint8_t* wscales, int K,
                                              int nt, const uint8_t* tcodes, const uint8_t* tscales, int count,
                                              Row row) {
  s.KB = K / 128;
  s.w = wcodes + static_cast<size_t>(nt) * (C::BW / 16) * s.KB * 1024;
  const size_t cs = mx_codes_stride(K), ss = mx_scales_stride(K);
#pragma unroll
  for (int i = 0; i < C::LT; ++i)
    s.tok[i] = tcodes + static_cast<size_t>(row(min((C::NW * i + wave_id()) * 16 + (lane_id() & 15), count - 1))) * cs;
  if (wave_id() >= 2)
    s.scale = tscales + static_cast<size_t>(row(min(lane_id(), count - 1))) * ss;
  else
    s.scale = wscales + static_cast<size_t>(nt * C::NQ + wave_id()) * mx_kq(K) * 1024 + lane_id() * 4;
}

template <class C>
struct MxFrags {
  u32x4 a[C::AW];
  u32x4 b[C::AT];
  uint32_t sa;
  uint32_t sb[C::STREAM ? C::AT : 1];
};

// Block (A, B) and the ones after it, column by column; the byte selects are
// part of the instruction.
template <class C, int A, int B>
__device__ __forceinline__ void mx_mfma_from(const MxFrags<C>& f, MxAcc<C>& acc, int nbv) {
  if constexpr (B < C::AT) {
    if constexpr (A < C::AW) {
      if (!C::STREAM || B < nbv)
        acc.v[A][B] = mfma_mx<A, C::STREAM ? 0 : B>(f.a[A], f.b[B], acc.v[A][B], f.sa, f.sb[C::STREAM ? B : 0]);
      mx_mfma_from<C, A + 1, B>(f, acc, nbv);
    } else {
      mx_mfma_from<C, 0, B + 1>(f, acc, nbv);
    }
  }
}
template <class C>
__device__ __forceinline__ void mx_mfma(const MxFrags<C>& f, MxAcc<C>& acc, int nbv) {
  mx_mfma_from<C, 0, 0>(f, acc, nbv);
}

// ------------------------------------------------------------------ loads and reads of a K step

template <class C>
__device__ __forceinline__ void mx_issue(const MxStreamSrc<C>& s, uint8_t* lds, int kt) {
  uint8_t* st = lds + (kt % C::NST) * C::STAGE;
  const int wave = mx_wave(), lane = lane_id();
#pragma unroll
  for (int i = 0; i < C::LW; ++i) {
    const int f = C::NW * i + wave;
    lds_dma16_nt(s.w + (static_cast<size_t>(f) * s.KB + kt) * 1024 + lane * 16, st + f * 1024);
  }
#pragma unroll
  for (int i = 0; i < C::LT; ++i)
    lds_dma16(s.tok[i] + kt * 64 + (lane >> 4) * 16, st + C::T0 + (C::NW * i + wave) * 1024);
  if (wave >= 2)  // both load the same 256 bytes
    lds_dma4(s.scale + kt * 4, st + C::S0 + C::NQ * 256);
  else
    lds_dma4(s.scale + static_cast<size_t>(kt) * 256, st + C::S0 + wave * 256);
}

template <class C>
__device__ __forceinline__ void mx_read(const uint8_t* st, MxFrags<C>& f, int nbv) {
  const int lane = lane_id(), wr = mx_wr<C>(), wt = mx_wt<C>();
  f.sa = *reinterpret_cast<const uint32_t*>(st + C::S0 + wr * 256 + lane * 4);
#pragma unroll
  for (int a = 0; a < C::AW; ++a) f.a[a] = ld16(st + (wr * C::AW + a) * 1024 + lane * 16);
#pragma unroll
  for (int b = 0; b < C::AT; ++b)
    if (b < nbv) {
      f.sb[b] = *reinterpret_cast<const uint32_t*>(st + C::S0 + C::NQ * 256 + ((wt * C::AT + b) * 16 + (lane & 15)) * 4) >>
                (8 * (lane >> 4));
      f.b[b] = ld16(st + C::T0 + (wt * C::AT + b) * 1024 + lane * 16);
    }
}

template <class C, int N>
__device__ __forceinline__ void mx_wait_from(int later) {
  if constexpr (N <= C::NST - 2) {
    if (later == N) wait_vmcnt<N * (C::LW + C::LT + C::LS)>();
    else mx_wait_from<C, N + 1>(later);
  }
}

// The K loop.  ACT false: no row of the wavefront is valid; it loads and waits
// with the others.
template <class C, bool ACT>
__device__ __forceinline__ void mx_run(const MxStreamSrc<C>& s, uint8_t* lds, MxAcc<C>& acc, int nbv) {
  const int nk = s.KB;
#pragma unroll
  for (int k = 0; k < C::NST - 1; ++k)
    if (k < nk) mx_issue<C>(s, lds, k);
  for (int kt = 0; kt < nk; ++kt) {
    const int later = min(C::NST - 2, nk - 1 - kt);
    if (later <= 0) wait_vmcnt<0>();
    else mx_wait_from<C, 1>(later);
    raw_barrier();  // step kt is in LDS, and every wavefront has read step kt - 1
    if (kt + C::NST - 1 < nk) mx_issue<C>(s, lds, kt + C::NST - 1);
    if constexpr (ACT) {
      MxFrags<C> f;
      mx_read<C>(lds + (kt % C::NST) * C::STAGE, f, nbv);
      mx_mfma<C>(f, acc, nbv);
    }
    // the reads of this stage are complete before the next barrier frees it
    wait_lgkm0();
  }
  raw_barrier();
}

// A wave-uniform pointer in scalar registers.
__device__ __forceinline__ const uint8_t* mx_uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(static_cast<uint32_t>(uniform(static_cast<int>(v)))) |
                                          static_cast<uint64_t>(static_cast<uint32_t>(uniform(static_cast<int>(v >> 32)))) << 32);
}

template <class C, bool ACT>
__device__ __forceinline__ void mx_run(const MxWideSrc& s, uint8_t* lds, MxAcc<C>& acc, int) {
  const int nk = s.KB, wave = mx_wave(), wr = mx_wr<C>(), wt = mx_wt<C>();
  const size_t fstep = static_cast<size_t>(nk) * 1024;
  const uint32_t lane = lane_id();
  const uint8_t *gw[C::LW], *gt[C::LT], *gs = mx_uniform(s.scale);
#pragma unroll
  for (int i = 0; i < C::LW; ++i) gw[i] = mx_uniform(s.w + (C::NW * i + wave) * fstep);
#pragma unroll
  for (int i = 0; i < C::LT; ++i) gt[i] = mx_uniform(s.t + (C::NW * i + wave) * fstep);
  uint8_t *in = lds + wave * 1024, *ins = lds + C::S0 + wave % (C::NQ + C::NQT) * 256;
  int fill = 0, use = 0;  // stage offsets
  const auto wrap = [](int o) { return o == (C::NST - 1) * C::STAGE ? 0 : o + C::STAGE; };
  const auto issue = [&]() {
#pragma unroll
    for (int i = 0; i < C::LW; ++i) {
      lds_dma16(gw[i] + lane * 16u, in + fill + C::NW * i * 1024);
      gw[i] += 1024;
    }
#pragma unroll
    for (int i = 0; i < C::LT; ++i) {
      lds_dma16(gt[i] + lane * 16u, in + fill + C::T0 + C::NW * i * 1024);
      gt[i] += 1024;
    }
    lds_dma4(gs + lane * 4u, ins + fill);
    gs += 256;
    fill = wrap(fill);
  };
#pragma unroll
  for (int k = 0; k < C::NST - 1; ++k)
    if (k < nk) issue();
  const uint8_t *la = lds + wr * C::AW * 1024 + lane * 16, *lb = lds + C::T0 + wt * C::AT * 1024 + lane * 16;
  const uint8_t *lsa = lds + C::S0 + wr * 256 + lane * 4;
  const uint8_t *lsb = lds + C::S0 + (C::NQ + wt * C::AT / 4) * 256 + lane * 4;
  for (int kt = 0; kt < nk; ++kt) {
    const int later = min(C::NST - 2, nk - 1 - kt);
    if (later <= 0) wait_vmcnt<0>();
    else mx_wait_from<C, 1>(later);
    raw_barrier();  // step kt is in LDS, and every wavefront has read step kt - 1
    MxFrags<C> f;
    if constexpr (ACT) {
      f.sa = *reinterpret_cast<const uint32_t*>(lsa + use);
      f.sb[0] = *reinterpret_cast<const uint32_t*>(lsb + use);
      f.b[0] = ld16(lb + use);
#pragma unroll
      for (int a = 0; a < C::AW; ++a) f.a[a] = ld16(la + use + a * 1024);
#pragma unroll
      for (int b = 1; b < C::AT; ++b) f.b[b] = ld16(lb + use + b * 1024);
      use = wrap(use);
      // all reads are under way before the first product: left alone, the
      // compiler reads a token block once the products of the one before are
      // issued, and the wavefront waits out LDS three times a step
      __builtin_amdgcn_sched_barrier(0);
    }
    if (kt + C::NST - 1 < nk) issue();
    if constexpr (ACT) {
      // the wavefront's token blocks are bytes AT * wt % 4 .. of their group's word
      f.sb[0] >>= 8 * (wt * C::AT % 4);
      mx_mfma<C>(f, acc, C::AT);
      __builtin_amdgcn_sched_barrier(0);
    }
    // the reads of this stage are complete before the next barrier frees it
    wait_lgkm0();
  }
  raw_barrier();
}

// Computes one tile.  count: valid token rows (>= 1); the accumulators of
// rows past them hold no meaningful values.  All threads must call it; on
// entry no direct-to-LDS load of the workgroup is in flight, on exit none is
// and a barrier has passed.
template <class C, class Src>
__device__ __forceinline__ void mx_tile(const Src& s, uint8_t* lds, MxAcc<C>& acc, int count) {
#pragma unroll
  for (int a = 0; a < C::AW; ++a)
#pragma unroll
    for (int b = 0; b < C::AT; ++b) acc.v[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int first = uniform(mx_wt<C>() * C::AT * 16);
  if (first < count) mx_run<C, true>(s, lds, acc, min(C::AT, (count - first + 15) / 16));
  else mx_run<C, false>(s, lds, acc, 0);
}

}  // namespace moe
