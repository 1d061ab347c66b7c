// ffn_mxfp4.hip -- the expert FFN with both operands of both products in
// MXFP4: per routed pair h1 = xq W1q, h3 = xq W3q, a = silu(h1) * h3 (or
// max(h1, 0)^2) in fp32, aq = MXFP4(a), y = aq W2q rounded to bf16, then the
// combine.  The same phases, tile order and combine as the bf16 FFN
// (ffn.hip) around the tiles of mx_tile.h.
#include "ffn_parts.h"
#include "moe_internal.h"
#include "mx_tile.h"
#include "wave_sched.h"

namespace moe {
namespace {

// The GEMM1 epilogue: activation, block scale and codes in registers.  The
// 32 intermediate indices of a block are four row blocks of one wavefront
// (gate, up, gate, up; two when ungated), spread over the four lanes of a
// token column, so the block's largest magnitude takes two lane exchanges.
// `a` is quantised from fp32, without a rounding to bf16 in between.  Codes
// (two bytes a lane and row block pair) and scales are staged in LDS and
// leave as whole 16-byte pieces of the rows.
template <class C, bool GATED>
__device__ __forceinline__ void mx_store_act(const MxAcc<C>& acc, uint8_t* lds, uint8_t* __restrict__ codes,
                                             uint8_t* __restrict__ scales, int row0, int count, int nt, int I) {
  constexpr int RB = GATED ? 4 : 2;             // row blocks per 32 intermediate indices
  constexpr int NB = C::BW / (16 * RB);         // MX blocks per tile row
  constexpr int CB = NB * 16;                   // code bytes per tile row
  constexpr int CH = CB / 16;                   // 16-byte pieces
  static_assert(static_cast<size_t>(C::BT) * (CB + NB) <= C::LDS_BYTES, "stage fits");
  uint8_t* sst = lds + C::BT * CB;
  const int lane = lane_id(), g = lane >> 4, wr = mx_wr<C>(), wt = mx_wt<C>();
#pragma unroll
  for (int b = 0; b < C::AT; ++b) {
    if ((wt * C::AT + b) * 16 >= count) continue;  // wave-uniform
    const int t = (wt * C::AT + b) * 16 + (lane & 15);
#pragma unroll
    for (int q = 0; q < C::AW / RB; ++q) {
      float v[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (GATED) {
          v[r] = mx_silu_mul(acc.v[q * 4][b][r], acc.v[q * 4 + 1][b][r]);
          v[4 + r] = mx_silu_mul(acc.v[q * 4 + 2][b][r], acc.v[q * 4 + 3][b][r]);
        } else {
          v[r] = relu_sq(acc.v[q * 2][b][r]);
          v[4 + r] = relu_sq(acc.v[q * 2 + 1][b][r]);
        }
      }
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16, kWave)));
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32, kWave)));
      const uint32_t sb = mx_scale_byte(m);
      const float inv = mx_inv_scale(sb);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = mx_scaled(v[j], inv, sb);
      const uint32_t c = mx_codes8(v);
      const int blk = wr * (C::AW / RB) + q;
      // elements 4g .. 4g+3 and 16 + 4g .. 16 + 4g + 3 of the block
      uint8_t* cr = lds + (t * CH + (blk ^ (t % CH))) * 16 + 2 * g;
      *reinterpret_cast<uint16_t*>(cr) = static_cast<uint16_t>(c);
      *reinterpret_cast<uint16_t*>(cr + 8) = static_cast<uint16_t>(c >> 16);
      if (g == 0) sst[t * NB + blk] = static_cast<uint8_t>(sb);
    }
  }
  __syncthreads();
  const size_t cs = mx_codes_stride(I), ss = mx_scales_stride(I);
  for (int i = threadIdx.x; i < count * CH; i += C::NTHREADS) {
    const int t = i / CH, c = i % CH;
    st16(codes + static_cast<size_t>(row0 + t) * cs + nt * CB + c * 16, ld16(lds + (t * CH + (c ^ (t % CH))) * 16));
  }
  for (int i = threadIdx.x; i < count * (NB / 2); i += C::NTHREADS) {
    const int t = i / (NB / 2), c = i % (NB / 2);
    *reinterpret_cast<uint16_t*>(scales + static_cast<size_t>(row0 + t) * ss + nt * NB + c * 2) =
        *reinterpret_cast<const uint16_t*>(sst + t * NB + c * 2);
  }
  __syncthreads();
}

struct MxArgs {
  const uint8_t* xc;      // token codes and scales
  const uint8_t* xs;
  const uint8_t* w;       // first expert's codes and scales
  const uint8_t* ws;
  const int32_t* offsets;
  const int32_t* sorted_token;
  uint8_t* ac;            // activation codes and scales, sorted rows
  uint8_t* as;
  uint16_t* y;
  int E_local, d, I;
};

// build_mtile_prefix by the first wavefront: its one-thread loop waits out
// E_local loads in turn, several microseconds before the first tile.
__device__ __forceinline__ void mx_mtile_prefix(const int32_t* __restrict__ offsets, int E_local, int BT,
                                                int32_t* mt_pre) {
  if (wave_id() != 0) return;
  const int lane = lane_id();
  int32_t n[kMaxLocalExperts / kWave];
#pragma unroll
  for (int c = 0; c < kMaxLocalExperts / kWave; ++c) {
    const int e = c * kWave + lane;
    n[c] = e < E_local ? (offsets[e + 1] - offsets[e] + BT - 1) / BT : 0;
  }
  int run = 0;
#pragma unroll
  for (int c = 0; c < kMaxLocalExperts / kWave; ++c) {
    if (c * kWave >= E_local) break;
    int incl = n[c];
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int o = __shfl_up(incl, off, kWave);
      incl += lane >= off ? o : 0;
    }
    if (c * kWave + lane < E_local) mt_pre[c * kWave + lane] = run + incl - n[c];
    run += __shfl(incl, kWave - 1, kWave);
  }
  if (lane == 0) mt_pre[E_local] = run;
}

// Tile loop of a phase: f(expert, first row, rows, n-tile).
template <class C, class F>
__device__ __forceinline__ void mx_tiles(const MxArgs& A, int NT, F f) {
  __shared__ int32_t mt_pre[kMaxLocalExperts + 1];
  __shared__ int32_t xcd_order;
  mx_mtile_prefix(A.offsets, A.E_local, C::BT, mt_pre);
  __syncthreads();
  if (threadIdx.x == 0) xcd_order = !C::STREAM && phase_xcd_order(mt_pre, A.E_local);
  __syncthreads();
  const bool xo = uniform(xcd_order) != 0;
  const PhaseTiles r = phase_tiles(uniform(mt_pre[A.E_local] * NT), xo, static_cast<int>(blockIdx.x),
                                   static_cast<int>(gridDim.x));
  for (int g = r.begin + r.first; g < r.end; g += r.stride) {
    int e, mt, nt;
    phase_tile(mt_pre, A.E_local, NT, g, xo, e, mt, nt);
    e = uniform(e);
    mt = uniform(mt);
    nt = uniform(nt);
    const int row0 = uniform(A.offsets[e] + (mt - mt_pre[e]) * C::BT);
    f(e, row0, uniform(min(C::BT, A.offsets[e + 1] - row0)), nt);
  }
}

template <class C, bool GATED>
__global__ __launch_bounds__(C::NTHREADS) void gemm1_mx_kernel(MxArgs A) {
  extern __shared__ __align__(16) uint8_t mx_lds[];
  const int N = (GATED ? 2 : 1) * A.I;
  mx_tiles<C>(A, N / C::BW, [&](int e, int row0, int count, int nt) {
    MxSrc<C> s;
    mx_src<C>(s, A.w + e * mx_mat_codes(N, A.d), A.ws + e * mx_mat_scales(N, A.d), A.d, nt, A.xc, A.xs, count,
              [&](int r) { return A.sorted_token[row0 + r]; });
    MxAcc<C> acc;
    mx_tile<C>(s, mx_lds, acc, count);
    mx_store_act<C, GATED>(acc, mx_lds, A.ac, A.as, row0, count, nt, A.I);
  });
}

template <class C>
__global__ __launch_bounds__(C::NTHREADS) void gemm2_mx_kernel(MxArgs A) {
  extern __shared__ __align__(16) uint8_t mx_lds[];
  static_assert(static_cast<size_t>(C::BT) * C::BW * 2 <= C::LDS_BYTES, "output stage fits the tile's LDS");
  mx_tiles<C>(A, A.d / C::BW, [&](int e, int row0, int count, int nt) {
    MxSrc<C> s;
    mx_src<C>(s, A.w + e * mx_mat_codes(A.d, A.I), A.ws + e * mx_mat_scales(A.d, A.I), A.I, nt, A.ac, A.as, count,
              [&](int r) { return row0 + r; });
    MxAcc<C> acc;
    mx_tile<C>(s, mx_lds, acc, count);
    uint16_t* lds = reinterpret_cast<uint16_t*>(mx_lds);
    const int lane = lane_id(), wr = mx_wr<C>(), wt = mx_wt<C>();
#pragma unroll
    for (int b = 0; b < C::AT; ++b) {
      if ((wt * C::AT + b) * 16 >= count) continue;  // wave-uniform
      const int t = (wt * C::AT + b) * 16 + (lane & 15);
#pragma unroll
      for (int a = 0; a < C::AW; ++a) {
        const f32x4 v = acc.v[a][b];
        const u32x2 pk{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        out_put<C::BW>(lds, t, (wr * C::AW + a) * 16 + 4 * (lane / 16), pk);
      }
    }
    out_flush<C::BW, C::NW>(lds, A.y + static_cast<size_t>(row0) * A.d + nt * C::BW, A.d, count);
  });
}

template <class K>
hipError_t launch_phase(K kern, int threads, size_t lds, const MxArgs& A, hipStream_t s) {
  int dev = 0, cus = 0, per_cu = 0;
  hipError_t e;
  if ((e = hipGetDevice(&dev)) != hipSuccess) return e;
  if ((e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev)) != hipSuccess) return e;
  if ((e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, kern, threads, lds)) != hipSuccess) return e;
  kern<<<max(1, per_cu) * cus, threads, lds, s>>>(A);
  return hipGetLastError();
}

template <class C>
hipError_t launch_g1(bool gated, const MxArgs& A, hipStream_t s) {
  return launch_phase(gated ? gemm1_mx_kernel<C, true> : gemm1_mx_kernel<C, false>, C::NTHREADS, C::LDS_BYTES, A, s);
}
template <class C>
hipError_t launch_g2(const MxArgs& A, hipStream_t s) {
  return launch_phase(gemm2_mx_kernel<C>, C::NTHREADS, C::LDS_BYTES, A, s);
}

}  // namespace

hipError_t launch_ffn_mxfp4(const moe_problem_t& p, const WsLayout& L, const uint8_t* xc, const uint8_t* xs,
                            const void* packed, const int32_t* offsets, const int32_t* sorted_token,
                            const int32_t* pair_pos, const float* topk_w, void* y, void* out, char* ws,
                            hipStream_t s) {
  if (p.T == 0) return hipSuccess;
  const int gr = gate_rows(p);
  const PackedMxLayout PL = packed_mx_layout(p.d, p.I, p.E_global, p.E_local, p.x_dtype == MOE_BF16, gr);
  const uint8_t* base = static_cast<const uint8_t*>(packed);
  // the activations in 4 bits take the place of the bf16 ones: a row of
  // codes and scales has at most I / 2 + 64 + I / 32 + 12 of the region's 2 I
  // bytes a row
  uint8_t* ac = reinterpret_cast<uint8_t*>(ws + L.act);
  MxArgs A{xc, xs, base + PL.w13, base + PL.w13s, offsets, sorted_token, ac,
           ac + static_cast<size_t>(L.P_max) * mx_codes_stride(p.I), static_cast<uint16_t*>(y), p.E_local, p.d, p.I};
  const double rows = static_cast<double>(p.T) * p.k / p.E_global;
  const bool wide = rows >= 96.0;
  hipError_t e;
  if (!wide) e = launch_g1<MxStream>(gr == 2, A, s);
  else if (gr * p.I % 256 == 0) e = launch_g1<MxWide<256>>(gr == 2, A, s);
  else e = launch_g1<MxWide<128>>(gr == 2, A, s);
  if (e != hipSuccess) return e;
  A.w = base + PL.w2;
  A.ws = base + PL.w2s;
  if (!wide) e = launch_g2<MxStream>(A, s);
  else if (p.d % 256 == 0) e = launch_g2<MxWide<256>>(A, s);
  else e = launch_g2<MxWide<128>>(A, s);
  if (e != hipSuccess || !out) return e;
  return launch_combine(p, y, pair_pos, topk_w, out, s);
}

}  // namespace moe
