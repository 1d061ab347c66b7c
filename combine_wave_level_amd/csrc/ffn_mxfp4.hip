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
// (two bytes a lane and row block pair) and scales are staged in LDS.
// code(t, blk) and scale(t, blk) give the staged places of tile row t, block
// blk of the tile: 16 bytes of codes, and the scale byte.
template <class C, bool GATED, class Code, class Scale>
__device__ __forceinline__ void mx_quantize_act(const MxAcc<C>& acc, int count, Code code, Scale scale) {
  constexpr int RB = GATED ? 4 : 2;             // row blocks per 32 intermediate indices
  const int lane = opaque_tid() & (kWave - 1), g = lane >> 4, wr = mx_wr<C>(), wt = mx_wt<C>();
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
      uint8_t* cr = code(t, blk) + 2 * g;
      *reinterpret_cast<uint16_t*>(cr) = static_cast<uint16_t>(c);
      *reinterpret_cast<uint16_t*>(cr + 8) = static_cast<uint16_t>(c >> 16);
      if (g == 0) *scale(t, blk) = static_cast<uint8_t>(sb);
    }
  }
}

// Rows (MxStream): whole 16-byte pieces of sorted rows row0 .. + count.
template <class C, bool GATED>
__device__ __forceinline__ void mx_store_act_rows(const MxAcc<C>& acc, uint8_t* lds, uint8_t* __restrict__ codes,
                                                  uint8_t* __restrict__ scales, int row0, int count, int nt, int I) {
  constexpr int NB = C::BW / (GATED ? 64 : 32);  // MX blocks per tile row
  static_assert(static_cast<size_t>(C::BT) * NB * 17 <= C::LDS_BYTES, "stage fits");
  uint8_t* sst = lds + C::BT * NB * 16;
  mx_quantize_act<C, GATED>(acc, count, [&](int t, int blk) { return lds + (t * NB + (blk ^ (t % NB))) * 16; },
                            [&](int t, int blk) { return sst + t * NB + blk; });
  __syncthreads();
  const size_t cs = mx_codes_stride(I), ss = mx_scales_stride(I);
  for (int i = opaque_tid(); i < count * NB; i += C::NTHREADS) {
    const int t = i / NB, c = i % NB;
    st16(codes + static_cast<size_t>(row0 + t) * cs + (nt * NB + c) * 16, ld16(lds + (t * NB + (c ^ (t % NB))) * 16));
  }
  for (int i = opaque_tid(); i < count * (NB / 2); i += C::NTHREADS) {
    const int t = i / (NB / 2), c = i % (NB / 2);
    *reinterpret_cast<uint16_t*>(scales + static_cast<size_t>(row0 + t) * ss + nt * NB + c * 2) =
        *reinterpret_cast<const uint16_t*>(sst + t * NB + c * 2);
  }
  __syncthreads();
}

// Fragments (MxWide): the second product's token operand, padded rows prow0
// .. (a multiple of 64).  A tile's blocks of a row block and K step are
// consecutive 256-byte runs of one fragment.  Rows past count hold whatever
// was there; their columns are never used.
template <class C, bool GATED>
__device__ __forceinline__ void mx_store_act_frags(const MxAcc<C>& acc, uint8_t* lds, uint8_t* __restrict__ codes,
                                                   uint8_t* __restrict__ scales, int prow0, int count, int nt, int I) {
  constexpr int NB = C::BW / (GATED ? 64 : 32);
  static_assert(static_cast<size_t>(C::BT) * NB * 17 <= C::LDS_BYTES, "stage fits");
  uint8_t* sst = lds + C::BT * NB * 16;  // [row quad][block][row] words, byte = row block of the quad
  mx_quantize_act<C, GATED>(acc, count, [&](int t, int blk) { return lds + ((t / 16 * NB + blk) * 16 + t % 16) * 16; },
                            [&](int t, int blk) { return sst + ((t / 64 * NB + blk) * 16 + t % 16) * 4 + t / 16 % 4; });
  __syncthreads();
  const int KB = I / 128, nrb = (count + 15) / 16;
  for (int i = opaque_tid(); i < nrb * NB * 16; i += C::NTHREADS) {
    const int rb = i / (NB * 16), j = i % (NB * 16);  // j: 16-byte piece of the row block's run
    const int blk = nt * NB + j / 16;
    st16(codes + (static_cast<size_t>(prow0 / 16 + rb) * KB + blk / 4) * 1024 + (blk % 4) * 256 + (j % 16) * 16,
         ld16(lds + i * 16));
  }
  const int kq = mx_kq(I), nq = (count + 63) / 64;
  for (int i = opaque_tid(); i < nq * NB * 16; i += C::NTHREADS) {
    const int q = i / (NB * 16), j = i % (NB * 16), blk = nt * NB + j / 16, ks = blk / 4;
    *reinterpret_cast<uint32_t*>(scales + (static_cast<size_t>(prow0 / 64 + q) * kq * 4 + ks) * 256 +
                                 ((blk % 4) * 16 + j % 16) * 4) = *reinterpret_cast<const uint32_t*>(sst + i * 4);
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
  uint8_t* ac;            // activation codes and scales
  uint8_t* as;            // (MxStream: sorted rows; MxWide: fragments of padded rows, as are xc and xs)
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

// First row of each expert in the padded row space of the fragment layouts
// (its rows rounded up to 64), from the m-tile prefix's wavefront.
__device__ __forceinline__ void mx_seg_prefix(const int32_t* __restrict__ offsets, int E_local, int32_t* seg) {
  mx_mtile_prefix(offsets, E_local, 64, seg);  // in units of 64 rows
}

// Tile loop of a phase: f(expert, first row, rows, n-tile, first padded row).
template <class C, class F>
__device__ __forceinline__ void mx_tiles(const MxArgs& A, int NT, F f) {
  __shared__ int32_t mt_pre[kMaxLocalExperts + 1];
  __shared__ int32_t seg[kMaxLocalExperts + 1];
  __shared__ int32_t xcd_order;
  mx_mtile_prefix(A.offsets, A.E_local, C::BT, mt_pre);
  if (!C::STREAM) mx_seg_prefix(A.offsets, A.E_local, seg);
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
    const int prow0 = C::STREAM ? 0 : uniform(seg[e]) * 64 + (mt - uniform(mt_pre[e])) * C::BT;
    f(e, row0, uniform(min(C::BT, A.offsets[e + 1] - row0)), nt, prow0);
  }
}

// MxWide's token operand: the codes and scales of the routed rows in sorted
// order, in fragment layout over the padded rows (rows that pad an expert
// repeat its last one).  A workgroup takes 64 rows and a range of four-step
// groups of K: a wavefront copies a row block's pieces of a fragment (16 rows
// of 64 bytes, from the caches; 1 KiB written), and the scales pass through
// LDS, 16 bytes of a row at a time, on their way into words (fetched word by
// word they touched as many lines again as the codes).
__global__ __launch_bounds__(256) void mx_gather_kernel(const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                                                        const int32_t* __restrict__ offsets,
                                                        const int32_t* __restrict__ sorted_token, int E_local, int K,
                                                        uint8_t* __restrict__ fc, uint8_t* __restrict__ fs) {
  __shared__ int32_t seg[kMaxLocalExperts + 1];
  __shared__ int32_t tok[64];
  __shared__ __align__(16) uint8_t sc[64 * 16];
  mx_seg_prefix(offsets, E_local, seg);
  __syncthreads();
  const int nquads = uniform(seg[E_local]), KB = K / 128, kq = mx_kq(K);
  const size_t cs = mx_codes_stride(K), ss = mx_scales_stride(K);
  const int g0 = kq * static_cast<int>(blockIdx.y) / static_cast<int>(gridDim.y);
  const int g1 = kq * (static_cast<int>(blockIdx.y) + 1) / static_cast<int>(gridDim.y);
  const int l = lane_id(), rb = wave_id();
  for (int q = blockIdx.x; q < nquads; q += gridDim.x) {
    const int e = uniform(sched_expert_of(seg, 0, E_local, q));
    __syncthreads();  // tok free
    if (threadIdx.x < 64) {
      const int r = offsets[e] + (q - seg[e]) * 64 + static_cast<int>(threadIdx.x);
      tok[threadIdx.x] = sorted_token[min(r, offsets[e + 1] - 1)];
    }
    __syncthreads();
    const uint8_t* src = xc + static_cast<size_t>(tok[rb * 16 + l % 16]) * cs + (l / 16) * 16;
    uint8_t* dst = fc + static_cast<size_t>(q * 4 + rb) * KB * 1024 + l * 16;
    for (int g = g0; g < g1; ++g) {
      u32x4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (g * 4 + k < KB) v[k] = ld16(src + (g * 4 + k) * 64);
      if (threadIdx.x < 64)
        st16(sc + threadIdx.x * 16, ld16(xs + static_cast<size_t>(tok[threadIdx.x]) * ss + g * 16));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (g * 4 + k < KB) st16(dst + static_cast<size_t>(g * 4 + k) * 1024, v[k]);
      __syncthreads();
      // word (step rb of the group, lane l); steps past K are never read
      uint32_t w = 0;
#pragma unroll
      for (int a = 0; a < 4; ++a) w |= static_cast<uint32_t>(sc[(a * 16 + l % 16) * 16 + rb * 4 + l / 16]) << (8 * a);
      *reinterpret_cast<uint32_t*>(fs + (static_cast<size_t>(q) * kq + g) * 1024 + rb * 256 + l * 4) = w;
      __syncthreads();
    }
  }
}

template <class C, bool GATED>
__global__ __launch_bounds__(C::NTHREADS, C::PER_CU * C::NW / 4) void gemm1_mx_kernel(MxArgs A) {
  extern __shared__ __align__(16) uint8_t mx_lds[];
  const int N = (GATED ? 2 : 1) * A.I;
  mx_tiles<C>(A, N / C::BW, [&](int e, int row0, int count, int nt, int prow0) {
    const uint8_t *wc = A.w + e * mx_mat_codes(N, A.d), *wsc = A.ws + e * mx_mat_scales(N, A.d);
    MxAcc<C> acc;
    if constexpr (C::STREAM) {
      MxStreamSrc<C> s;
      mx_stream_src<C>(s, wc, wsc, A.d, nt, A.xc, A.xs, count, [&](int r) { return A.sorted_token[row0 + r]; });
      mx_tile<C>(s, mx_lds, acc, count);
      mx_store_act_rows<C, GATED>(acc, mx_lds, A.ac, A.as, row0, count, nt, A.I);
    } else {
      mx_tile<C>(mx_wide_src<C>(wc, wsc, A.d, nt, A.xc, A.xs, prow0), mx_lds, acc, count);
      mx_store_act_frags<C, GATED>(acc, mx_lds, A.ac, A.as, prow0, count, nt, A.I);
    }
  });
}

template <class C>
__global__ __launch_bounds__(C::NTHREADS, C::PER_CU * C::NW / 4) void gemm2_mx_kernel(MxArgs A) {
  extern __shared__ __align__(16) uint8_t mx_lds[];
  static_assert(static_cast<size_t>(C::BT) * C::BW * 2 <= C::LDS_BYTES, "output stage fits the tile's LDS");
  mx_tiles<C>(A, A.d / C::BW, [&](int e, int row0, int count, int nt, int prow0) {
    const uint8_t *wc = A.w + e * mx_mat_codes(A.d, A.I), *wsc = A.ws + e * mx_mat_scales(A.d, A.I);
    MxAcc<C> acc;
    if constexpr (C::STREAM) {
      MxStreamSrc<C> s;
      mx_stream_src<C>(s, wc, wsc, A.I, nt, A.ac, A.as, count, [&](int r) { return row0 + r; });
      mx_tile<C>(s, mx_lds, acc, count);
    } else {
      mx_tile<C>(mx_wide_src<C>(wc, wsc, A.I, nt, A.ac, A.as, prow0), mx_lds, acc, count);
    }
    // y rounded to bf16, staged as [row][16-byte piece] (pieces swizzled by
    // row, as out_put does) and stored as whole rows
    uint16_t* lds = reinterpret_cast<uint16_t*>(mx_lds);
    const int tid = opaque_tid(), lane = tid & (kWave - 1), wr = mx_wr<C>(), wt = mx_wt<C>();
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
    __syncthreads();
    constexpr int CH = C::BW / 8;
    uint16_t* dst = A.y + static_cast<size_t>(row0) * A.d + nt * C::BW;
    for (int i = tid; i < count * CH; i += C::NTHREADS)
      st16(dst + static_cast<size_t>(i / CH) * A.d + i % CH * 8, ld16(lds + OutStage<C::BW>::slot(i / CH, i % CH) * 8));
    __syncthreads();
  });
}

// The grid is what the device holds at once (LDS and registers of both
// products' kernels fit C::PER_CU workgroups a CU by their bounds).
template <class C, class K>
hipError_t launch_phase(K kern, const MxArgs& A, hipStream_t s) {
  int dev = 0, cus = 0;
  hipError_t e;
  if ((e = hipGetDevice(&dev)) != hipSuccess) return e;
  if ((e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev)) != hipSuccess) return e;
  kern<<<C::PER_CU * cus, C::NTHREADS, C::LDS_BYTES, s>>>(A);
  return hipGetLastError();
}

template <class C>
hipError_t launch_g1(bool gated, const MxArgs& A, hipStream_t s) {
  return launch_phase<C>(gated ? gemm1_mx_kernel<C, true> : gemm1_mx_kernel<C, false>, A, s);
}
template <class C>
hipError_t launch_g2(const MxArgs& A, hipStream_t s) {
  return launch_phase<C>(gemm2_mx_kernel<C>, A, s);
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
  // The matrix-bound tiles from 64 rows an expert on the average.  Measured,
  // quantisation to combine, MxWide against MxStream: d = 4096, I = 1024, 16
  // experts: 48 against 40 us at 48 rows, 51 against 55 at 64, 55 against 61
  // at 96; d = 7168, I = 2048, 32 experts: 183 against 171, 191 against 253,
  // 206 against 339; d = 2048, I = 768, 64 experts: 61 against 54, 66 against
  // 74, 73 against 91.  And where their operands fit: the activations
  // in 4 bits take the place of the bf16 ones (2 I bytes a row of P_max).
  // MxStream: rows of at most I / 2 + 64 code and I / 32 + 12 scale bytes.
  // MxWide: fragments over the padded rows (and the up to 64 rows that the
  // last tile may read past them), and the gathered token operand likewise in
  // the place of y (2 d bytes a row), which the second product then writes:
  // with P_max >= 64 E_local that takes a little over half of either, and
  // only layers a few hundred wide with one or two experts fall short.
  const size_t pad = static_cast<size_t>(L.P_pad), pmax = static_cast<size_t>(L.P_max);
  const auto frag_bytes = [&](int K) { return (pad + 64) * (static_cast<size_t>(K) / 2 + 16 * static_cast<size_t>(mx_kq(K))); };
  const bool wide = static_cast<double>(p.T) * p.k / p.E_global >= 64.0 && frag_bytes(p.d) <= pmax * p.d * 2 &&
                    frag_bytes(p.I) <= pmax * p.I * 2;
  uint8_t* ac = reinterpret_cast<uint8_t*>(ws + L.act);
  MxArgs A{xc, xs, base + PL.w13, base + PL.w13s, offsets, sorted_token, ac,
           ac + (wide ? (pad + 64) * (p.I / 2) : pmax * mx_codes_stride(p.I)), static_cast<uint16_t*>(y), p.E_local,
           p.d, p.I};
  hipError_t e;
  if (!wide) {
    e = launch_g1<MxStream>(gr == 2, A, s);
  } else {
    uint8_t* fc = static_cast<uint8_t*>(y);
    uint8_t* fs = fc + (pad + 64) * (p.d / 2);
    const dim3 ggrid(static_cast<unsigned>(min(pad / 64, static_cast<size_t>(2048))), min(mx_kq(p.d), 8));
    mx_gather_kernel<<<ggrid, 256, 0, s>>>(
        xc, xs, offsets, sorted_token, p.E_local, p.d, fc, fs);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    A.xc = fc;
    A.xs = fs;
    if (gr * p.I % 256 == 0) e = launch_g1<MxWide<256>>(gr == 2, A, s);
    else e = launch_g1<MxWide<128>>(gr == 2, A, s);
  }
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
