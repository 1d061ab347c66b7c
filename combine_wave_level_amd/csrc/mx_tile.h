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
// 32-wide step is, and one matrix instruction takes as long: the data
// movement of gemm_tile.h fits unchanged (direct-to-LDS loads of 16 bytes a
// lane, whole 128-byte token lines swizzled by row, conflict-free 16-byte
// reads) and every byte of it carries four times the elements.  What is new
// are the scales.  They travel through LDS with the data, because vmcnt
// counts in order: a scale loaded to registers one step ahead would wait for
// every later stage of the prefetch as well.
//
// MxWide (many rows an expert, matrix bound): BW = 256 or 128 by 256 tokens,
//   8 wavefronts of BW/2 x 64, the two of a SIMD one phase apart (see
//   gemm_tile.h); weights in 4 stages of one K step, token lines in 2 slots
//   of two, scales in 2 slots of four K steps (one load a wavefront per four
//   steps).
// MxStream (a few rows an expert, bound by the weights' bytes): 128 x 64, 4
//   wavefronts of 64 x 32, all operands in 5 stages of one K step; two
//   workgroups a CU, so that one loads while the other starts or ends a tile.
#pragma once

#include "gemm_tile.h"
#include "mxfp4.h"

namespace moe {

__device__ __forceinline__ void lds_dma4(const void* g, void* l) { __builtin_amdgcn_global_load_lds(g, l, 4, 0, 0); }

template <int BW_>
struct MxWide {
  static constexpr bool STREAM = false;
  static constexpr int BW = BW_, BT = 256, WR = 2, WT = 4, NW = 8, NTHREADS = 512;
  static constexpr int AW = BW / WR / 16, AT = BT / WT / 16;
  static constexpr int NST = 4, LW = BW / 16 / NW, LT = BT / 8 / NW;
  static constexpr int NQ = BW / 64;               // 64-row groups of weight scales
  static constexpr int WSTAGE = BW * 64, TSLOT = BT * 128, SSLOT = NQ * 1024 + BT * 16;
  static constexpr int T0 = NST * WSTAGE, S0 = T0 + 2 * TSLOT;
  static constexpr size_t LDS_BYTES = S0 + 2 * SSLOT;
  static_assert(AW % 4 == 0 && LW >= 1 && NQ <= 4, "wave tile holds whole scale words");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
};

struct MxStream {
  static constexpr bool STREAM = true;
  static constexpr int BW = 128, BT = 64, WR = 2, WT = 2, NW = 4, NTHREADS = 256;
  static constexpr int AW = BW / WR / 16, AT = BT / WT / 16;
  static constexpr int NST = 5, LW = BW / 16 / NW, LT = BT / 16 / NW;
  static constexpr int NQ = BW / 64;
  static constexpr int LS = 1;
  static constexpr int T0 = BW * 64, S0 = T0 + BT * 64, STAGE = S0 + NQ * 256 + BT * 4;
  static constexpr size_t LDS_BYTES = static_cast<size_t>(NST) * STAGE;
  static_assert(NQ == 2 && BT == 64 && NW == 4, "one scale load a wavefront and step");
  static_assert((NST - 2) * (LW + LT + LS) <= 63, "vmcnt");
};

template <class C>
__device__ __forceinline__ int mx_wr() { return wave_id() % C::WR; }
template <class C>
__device__ __forceinline__ int mx_wt() { return wave_id() / C::WR; }

template <class C>
struct MxAcc {
  f32x4 v[C::AW][C::AT];
};

// This lane's global addresses: the token rows it loads (as trow_index of the
// bf16 tile: 8 rows of whole lines a load, or 16 rows of 64 bytes) and the
// scales its wavefront loads.
template <class C>
struct MxSrc {
  const uint8_t* w;         // packed codes, first fragment of the tile's rows
  const uint8_t* tok[C::LT];
  const uint8_t* scale;
  int KB;                   // K steps of the matrix
};

// Tile row (0 .. BT-1) that token load i of this lane covers.
template <class C>
__device__ __forceinline__ int mx_trow(int i) {
  if constexpr (C::STREAM) return (C::NW * i + wave_id()) * 16 + (lane_id() & 15);
  return (C::NW * i + wave_id()) * 8 + (lane_id() >> 3);
}
// Whether this wavefront loads token scales, and for which tile row.
template <class C>
__device__ __forceinline__ bool mx_loads_tscale() { return C::STREAM ? wave_id() >= 2 : wave_id() >= 4; }
template <class C>
__device__ __forceinline__ int mx_srow() { return C::STREAM ? lane_id() : (wave_id() - 4) * 64 + lane_id(); }
// The 64-row group of weight scales it loads otherwise (MxWide<128> has two
// groups for four wavefronts: the second pair repeats the first's loads).
template <class C>
__device__ __forceinline__ int mx_squad() { return wave_id() % C::NQ; }

// Fills MxSrc.  wcodes, wscales: the matrix's codes and scales; nt: tile along
// the weight rows; row(r): index of tile row r in the token matrix (valid for
// r < count); tcodes, tscales: token codes and scales with row strides.
template <class C, class Row>
__device__ __forceinline__ void mx_src(MxSrc<C>& s, const uint8_t* wcodes, const uint8_t* wscales, int K, int nt,
                                       const uint8_t* tcodes, const uint8_t* tscales, int count, Row row) {
  s.KB = K / 128;
  s.w = wcodes + static_cast<size_t>(nt) * (C::BW / 16) * s.KB * 1024;
  const size_t cs = mx_codes_stride(K), ss = mx_scales_stride(K);
#pragma unroll
  for (int i = 0; i < C::LT; ++i) s.tok[i] = tcodes + static_cast<size_t>(row(min(mx_trow<C>(i), count - 1))) * cs;
  if (mx_loads_tscale<C>())
    s.scale = tscales + static_cast<size_t>(row(min(mx_srow<C>(), count - 1))) * ss;
  else
    s.scale = wscales + static_cast<size_t>(nt * C::NQ + mx_squad<C>()) * mx_kq(K) * 1024 +
              lane_id() * (C::STREAM ? 4 : 16);
}

template <class C>
struct MxFrags {
  u32x4 a[C::AW];
  u32x4 b[C::AT];
  uint32_t sa[C::AW / 4];
  uint32_t sb[C::AT];
};

template <class C, int A>
__device__ __forceinline__ void mx_mfma_col(const MxFrags<C>& f, MxAcc<C>& acc, int b) {
  if constexpr (A < C::AW) {
    acc.v[A][b] = mfma_mx<A % 4, 0>(f.a[A], f.b[b], acc.v[A][b], f.sa[A / 4], f.sb[b]);
    mx_mfma_col<C, A + 1>(f, acc, b);
  }
}

template <class C>
__device__ __forceinline__ void mx_mfma(const MxFrags<C>& f, MxAcc<C>& acc, int nbv) {
#pragma unroll
  for (int b = 0; b < C::AT; ++b)
    if (!C::STREAM || b < nbv) mx_mfma_col<C, 0>(f, acc, b);
}

// ------------------------------------------------------------------ MxWide

template <class C>
__device__ __forceinline__ void mxw_issue_w(const MxSrc<C>& s, uint8_t* lds, int kt) {
  uint8_t* st = lds + (kt % C::NST) * C::WSTAGE;
#pragma unroll
  for (int i = 0; i < C::LW; ++i) {
    const int f = C::NW * i + wave_id();
    lds_dma16(s.w + (static_cast<size_t>(f) * s.KB + kt) * 1024 + lane_id() * 16, st + f * 1024);
  }
}

template <class C>
__device__ __forceinline__ void mxw_issue_t(const MxSrc<C>& s, uint8_t* lds, int j) {
  uint8_t* ts = lds + C::T0 + (j & 1) * C::TSLOT;
  const int chunk = (lane_id() & 7) ^ (lane_id() >> 3);
#pragma unroll
  for (int i = 0; i < C::LT; ++i) lds_dma16(s.tok[i] + j * 128 + chunk * 16, ts + (C::NW * i + wave_id()) * 1024);
}

// Scales of K steps 4q .. 4q+3: weight words [group][step][lane], token bytes
// [row][step][block].
template <class C>
__device__ __forceinline__ void mxw_issue_s(const MxSrc<C>& s, uint8_t* lds, int q) {
  uint8_t* ss = lds + C::S0 + (q & 1) * C::SSLOT;
  if (mx_loads_tscale<C>())
    lds_dma16(s.scale + q * 16, ss + C::NQ * 1024 + (wave_id() - 4) * 1024);
  else
    lds_dma16(s.scale + static_cast<size_t>(q) * 1024, ss + mx_squad<C>() * 1024);
}

template <class C>
__device__ __forceinline__ void mxw_read(const uint8_t* lds, int kt, MxFrags<C>& f) {
  const int lane = lane_id(), wr = mx_wr<C>(), wt = mx_wt<C>();
  const uint8_t* st = lds + (kt % C::NST) * C::WSTAGE;
  const uint8_t* ts = lds + C::T0 + ((kt >> 1) & 1) * C::TSLOT;
  const uint8_t* ss = lds + C::S0 + ((kt >> 2) & 1) * C::SSLOT;
#pragma unroll
  for (int q = 0; q < C::AW / 4; ++q)
    f.sa[q] = *reinterpret_cast<const uint32_t*>(ss + (wr * (C::AW / 4) + q) * 1024 + (kt & 3) * 256 + lane * 4);
#pragma unroll
  for (int b = 0; b < C::AT; ++b)
    f.sb[b] = *reinterpret_cast<const uint32_t*>(ss + C::NQ * 1024 + ((wt * C::AT + b) * 16 + (lane & 15)) * 16 +
                                                 (kt & 3) * 4) >> (8 * (lane >> 4));
#pragma unroll
  for (int a = 0; a < C::AW; ++a) f.a[a] = ld16(st + (wr * C::AW + a) * 1024 + lane * 16);
  const int hb = (lane >> 3) & 1, rr = lane & 7, pos = (4 * (kt & 1) + (lane >> 4)) ^ rr;
  const uint8_t* tl = ts + hb * 1024 + rr * 128 + pos * 16;
#pragma unroll
  for (int b = 0; b < C::AT; ++b) f.b[b] = ld16(tl + (wt * C::AT + b) * 2048);
}

// After iteration i's issues, wait for the loads of step i + 1.  In issue
// order: S(0), T(0), W(0..2); iteration i issues S(i/4 + 1) when i % 4 == 0,
// W(i+3), and T(i/2 + 1) when i is even, each where it exists.  Issued after
// the last load that step i + 1 needs: odd i (T((i+1)/2), iteration i - 1):
// W(i+3); even i (T(i/2), iteration i - 2): W(i+2), W(i+3), T(i/2 + 1), and
// scales that only allow more.
template <class C>
__device__ __forceinline__ void mxw_wait_next(int i, int nk) {
  if (i + 1 >= nk) return;
  if (i & 1) {
    if (i + 3 < nk) wait_vmcnt<C::LW>(); else wait_vmcnt<0>();
  } else {
    if (i + 3 < nk) wait_vmcnt<2 * C::LW + C::LT>();
    else if (i + 2 < nk) wait_vmcnt<C::LW + C::LT>();
    else wait_vmcnt<0>();
  }
}

template <class C, bool ACT>
__device__ __forceinline__ void mxw_run(const MxSrc<C>& s, uint8_t* lds, MxAcc<C>& acc) {
  const int nk = s.KB;
  const bool late = uniform(wave_id()) >= C::NW / 2;
  MxFrags<C> f;
  mxw_issue_s<C>(s, lds, 0);
  mxw_issue_t<C>(s, lds, 0);
#pragma unroll
  for (int k = 0; k < C::NST - 1; ++k)
    if (k < nk) mxw_issue_w<C>(s, lds, k);
  if (nk > 2) wait_vmcnt<2 * C::LW>();
  else if (nk > 1) wait_vmcnt<C::LW>();
  else wait_vmcnt<0>();
  raw_barrier();
  if (late) raw_barrier();
  for (int i = 0; i < nk; ++i) {
    if (!(i & 3) && i + 4 < nk) mxw_issue_s<C>(s, lds, i / 4 + 1);
    if (i + 3 < nk) mxw_issue_w<C>(s, lds, i + 3);
    if (!(i & 1) && i + 2 < nk) mxw_issue_t<C>(s, lds, i / 2 + 1);
    if constexpr (ACT) mxw_read<C>(lds, i, f);
    mxw_wait_next<C>(i, nk);
    wait_lgkm0();
    raw_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (ACT) mx_mfma<C>(f, acc, C::AT);
    __builtin_amdgcn_sched_barrier(0);
    mxw_wait_next<C>(i, nk);
    raw_barrier();
  }
  if (!late) raw_barrier();
  wait_vmcnt<0>();
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  raw_barrier();
}

// ------------------------------------------------------------------ MxStream

template <class C>
__device__ __forceinline__ void mxs_issue(const MxSrc<C>& s, uint8_t* lds, int kt) {
  uint8_t* st = lds + (kt % C::NST) * C::STAGE;
#pragma unroll
  for (int i = 0; i < C::LW; ++i) {
    const int f = C::NW * i + wave_id();
    lds_dma16_nt(s.w + (static_cast<size_t>(f) * s.KB + kt) * 1024 + lane_id() * 16, st + f * 1024);
  }
#pragma unroll
  for (int i = 0; i < C::LT; ++i)
    lds_dma16(s.tok[i] + kt * 64 + (lane_id() >> 4) * 16, st + C::T0 + (C::NW * i + wave_id()) * 1024);
  if (mx_loads_tscale<C>())  // wavefronts 2 and 3 load the same 256 bytes
    lds_dma4(s.scale + kt * 4, st + C::S0 + C::NQ * 256);
  else
    lds_dma4(s.scale + static_cast<size_t>(kt) * 256, st + C::S0 + mx_squad<C>() * 256);
}

template <class C>
__device__ __forceinline__ void mxs_read(const uint8_t* st, MxFrags<C>& f, int nbv) {
  const int lane = lane_id(), wr = mx_wr<C>(), wt = mx_wt<C>();
  f.sa[0] = *reinterpret_cast<const uint32_t*>(st + C::S0 + wr * 256 + lane * 4);
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
__device__ __forceinline__ void mxs_wait_from(int later) {
  if constexpr (N <= C::NST - 2) {
    if (later == N) wait_vmcnt<N * (C::LW + C::LT + C::LS)>();
    else mxs_wait_from<C, N + 1>(later);
  }
}

template <class C>
__device__ __forceinline__ void mxs_run(const MxSrc<C>& s, uint8_t* lds, MxAcc<C>& acc, int nbv) {
  const int nk = s.KB;
#pragma unroll
  for (int k = 0; k < C::NST - 1; ++k)
    if (k < nk) mxs_issue<C>(s, lds, k);
  for (int kt = 0; kt < nk; ++kt) {
    const int later = min(C::NST - 2, nk - 1 - kt);
    if (later <= 0) wait_vmcnt<0>();
    else mxs_wait_from<C, 1>(later);
    raw_barrier();  // step kt is in LDS, and every wavefront is past step kt - 1
    if (kt + C::NST - 1 < nk) mxs_issue<C>(s, lds, kt + C::NST - 1);
    if (nbv > 0) {
      MxFrags<C> f;
      mxs_read<C>(lds + (kt % C::NST) * C::STAGE, f, nbv);
      mx_mfma<C>(f, acc, nbv);
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
template <class C>
__device__ __forceinline__ void mx_tile(const MxSrc<C>& s, uint8_t* lds, MxAcc<C>& acc, int count) {
#pragma unroll
  for (int a = 0; a < C::AW; ++a)
#pragma unroll
    for (int b = 0; b < C::AT; ++b) acc.v[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int first = uniform(mx_wt<C>() * C::AT * 16);
  if constexpr (C::STREAM) {
    mxs_run<C>(s, lds, acc, max(0, min(C::AT, (count - first + 15) / 16)));
  } else {
    if (first < count) mxw_run<C, true>(s, lds, acc);
    else mxw_run<C, false>(s, lds, acc);
  }
}

}  // namespace moe
