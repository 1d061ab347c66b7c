// mxfp4.hip -- MXFP4 conversions: token rows to codes and scales and back,
// and the one-time quantisation and re-layout of the expert weights for the
// 4-bit products (and its inverse).  The format is described in mxfp4.h.
#include "moe_internal.h"
#include "mxfp4.h"

namespace moe {
namespace {

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

template <bool BF16>
__device__ __forceinline__ void load8(const void* __restrict__ x, size_t chunk, float (&v)[8]) {
  if constexpr (BF16) {
    const u32x4 q = ld16(static_cast<const uint16_t*>(x) + chunk * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  } else {
    const float* p = static_cast<const float*>(x) + chunk * 8;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

// Rows to codes and scales.  Four lanes share a block, eight elements each,
// so a wavefront reads 512 consecutive elements with 16-byte loads and
// writes their 256 bytes of codes in one store; the block's largest
// magnitude comes from two lane exchanges.  Bound by memory: x read once (8192
// x 4096 bf16 there and back: 32.5 us, 5.2 TB/s).
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(const void* __restrict__ x, size_t nchunks, int cpr,
                                                             size_t cs, size_t ss, uint8_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales) {
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= nchunks) return;  // nchunks % 4 == 0: the lanes of a block leave together
  const size_t t = i / cpr;
  const int c = static_cast<int>(i - t * cpr);
  float v[8];
  load8<BF16>(x, i, v);
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 1, kWave)));
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 2, kWave)));
  const uint32_t sb = mx_scale_byte(m);
  const float inv = mx_inv_scale(sb);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = mx_scaled(v[j], inv, sb);
  uint8_t* cr = codes + t * cs;
  uint8_t* sr = scales + t * ss;
  *reinterpret_cast<uint32_t*>(cr + c * 4) = mx_codes8(v);
  if ((c & 3) == 0) sr[c / 4] = static_cast<uint8_t>(sb);
  // padding (rows that are no multiple of 256, 512 elements)
  if (static_cast<size_t>(cpr) * 4 + c * 4 < cs) *reinterpret_cast<uint32_t*>(cr + cpr * 4 + c * 4) = 0;
  if (static_cast<size_t>(cpr) / 4 + c * 4 < ss) *reinterpret_cast<uint32_t*>(sr + cpr / 4 + c * 4) = 0;
}

// Codes and scales back to values, eight a lane.
template <bool BF16>
__global__ __launch_bounds__(256) void dequantize_mxfp4_kernel(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, size_t nchunks,
                                                               int cpr, size_t cs, size_t ss, void* __restrict__ x) {
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= nchunks) return;
  const size_t t = i / cpr;
  const int c = static_cast<int>(i - t * cpr);
  float v[8];
  mx_values8(*reinterpret_cast<const uint32_t*>(codes + t * cs + c * 4), mx_scale(scales[t * ss + c / 4]), v);
  if constexpr (BF16) {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = mx_bf16x2(v[2 * j], v[2 * j + 1]);
    st16(static_cast<uint16_t*>(x) + i * 8, o);
  } else {
    float* p = static_cast<float*>(x) + i * 8;
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
  }
}

// ------------------------------------------------------------------ weights

// Where column n, 32-element block kb of a math-layout matrix S[K][n_src]
// sits in its packed matrix: packed row, then code slot and scale byte.
struct MxPlace {
  size_t code, scale;  // byte offsets in the matrix's codes and scales
};
// ROWS 1: packed row = n.  ROWS 2: the interleave of W1 (sel = 0) and W3
// (sel = 1) by 16 columns.
template <int ROWS>
__device__ __forceinline__ MxPlace mx_place(int n, int sel, int kb, int K) {
  const int row = ROWS == 1 ? n : ((n / 16) * 2 + sel) * 16 + n % 16;
  const int nb = row / 16, r = row % 16, ks = kb / 4, g = kb % 4;
  MxPlace p;
  p.code = (static_cast<size_t>(nb) * (K / 128) + ks) * 1024 + (g * 16 + r) * 16;
  p.scale = ((static_cast<size_t>(nb / 4) * mx_kq(K) + ks / 4) * 4 + ks % 4) * 256 + (g * 16 + r) * 4 + nb % 4;
  return p;
}

// One thread quantises one block of one column: its 32 reads are strided,
// and the 64 lanes of a wavefront take consecutive columns, so every read
// instruction is contiguous.  blockIdx.y = 32-element block, z = expert and
// (ROWS 2) matrix.  Bound by memory (16 experts of d = 4096, I = 1024 in bf16
// there and back: 206 us, 4.9 TB/s).
template <bool BF16, int ROWS>
__global__ __launch_bounds__(256) void pack_mxfp4_kernel(const void* __restrict__ S, const void* __restrict__ S2, int K,
                                                         int N, uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  const int e = blockIdx.z / ROWS, sel = blockIdx.z % ROWS, kb = blockIdx.y;
  const MxPlace p = mx_place<ROWS>(n, sel, kb, K);
  uint8_t* sc = scales + static_cast<size_t>(e) * mx_mat_scales(ROWS * N, K) + p.scale;
  if (kb * kMxBlock >= K) {  // the scale words past K, so that the buffer is written entirely
    *sc = 0;
    return;
  }
  const void* src = sel ? S2 : S;
  const size_t at = (static_cast<size_t>(e) * K + static_cast<size_t>(kb) * kMxBlock) * N + n;
  float v[kMxBlock];
#pragma unroll
  for (int j = 0; j < kMxBlock; ++j) {
    if constexpr (BF16)
      v[j] = bf16_to_f32(static_cast<const uint16_t*>(src)[at + static_cast<size_t>(j) * N]);
    else
      v[j] = static_cast<const float*>(src)[at + static_cast<size_t>(j) * N];
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kMxBlock; ++j) m = max(m, abs_bits(v[j]));
  const uint32_t sb = mx_scale_byte(m);
  const float inv = mx_inv_scale(sb);
  u32x4 o;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = mx_scaled(v[q * 8 + j], inv, sb);
    o[q] = mx_codes8(w);
  }
  st16(codes + static_cast<size_t>(e) * mx_mat_codes(ROWS * N, K) + p.code, o);
  *sc = static_cast<uint8_t>(sb);
}

template <bool BF16, int ROWS>
__global__ __launch_bounds__(256) void unpack_mxfp4_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int K, int N,
                                                           void* __restrict__ S, void* __restrict__ S2) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  const int e = blockIdx.z / ROWS, sel = blockIdx.z % ROWS, kb = blockIdx.y;
  const MxPlace p = mx_place<ROWS>(n, sel, kb, K);
  const u32x4 q = ld16(codes + static_cast<size_t>(e) * mx_mat_codes(ROWS * N, K) + p.code);
  const float sc = mx_scale(scales[static_cast<size_t>(e) * mx_mat_scales(ROWS * N, K) + p.scale]);
  void* dst = sel ? S2 : S;
  const size_t at = (static_cast<size_t>(e) * K + static_cast<size_t>(kb) * kMxBlock) * N + n;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float v[8];
    mx_values8(q[c], sc, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const size_t i = at + static_cast<size_t>(c * 8 + j) * N;
      if constexpr (BF16)
        static_cast<uint16_t*>(dst)[i] = static_cast<uint16_t>(__float_as_uint(v[j]) >> 16);
      else
        static_cast<float*>(dst)[i] = v[j];
    }
  }
}

template <int ROWS>
hipError_t pack_mat(bool bf16, const void* S, const void* S2, int E, int K, int N, uint8_t* codes, uint8_t* scales,
                    hipStream_t s) {
  const dim3 grid((N + 255) / 256, mx_kq(K) * 16, E * ROWS);
  if (bf16)
    pack_mxfp4_kernel<true, ROWS><<<grid, 256, 0, s>>>(S, S2, K, N, codes, scales);
  else
    pack_mxfp4_kernel<false, ROWS><<<grid, 256, 0, s>>>(S, S2, K, N, codes, scales);
  return hipGetLastError();
}

template <int ROWS>
hipError_t unpack_mat(bool bf16, const uint8_t* codes, const uint8_t* scales, int E, int K, int N, void* S, void* S2,
                      hipStream_t s) {
  const dim3 grid((N + 255) / 256, K / kMxBlock, E * ROWS);
  if (bf16)
    unpack_mxfp4_kernel<true, ROWS><<<grid, 256, 0, s>>>(codes, scales, K, N, S, S2);
  else
    unpack_mxfp4_kernel<false, ROWS><<<grid, 256, 0, s>>>(codes, scales, K, N, S, S2);
  return hipGetLastError();
}

PackedMxLayout layout_of(const moe_problem_t& p) {
  return packed_mx_layout(p.d, p.I, p.E_global, p.E_local, p.x_dtype == MOE_BF16, gate_rows(p));
}

// f(first row, chunks of eight elements, workgroups) for the rows of a launch:
// all of them, but for more than 2^34 elements (a launch has fewer than 2^32
// threads).
template <class F>
hipError_t by_rows(int T, int cpr, F f) {
  const int rows = static_cast<int>(min(size_t{1} << 24, (size_t{1} << 31) / cpr));
  for (int t = 0; t < T; t += rows) {
    const size_t n = static_cast<size_t>(min(rows, T - t)) * cpr;
    f(static_cast<size_t>(t), n, static_cast<unsigned>((n + 255) / 256));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_quantize_mxfp4(const moe_problem_t& p, const void* x, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s) {
  const int cpr = p.d / 8;
  const size_t cs = mx_codes_stride(p.d), ss = mx_scales_stride(p.d);
  const size_t row = static_cast<size_t>(p.d) * (p.x_dtype == MOE_BF16 ? 2 : 4);
  return by_rows(p.T, cpr, [&](size_t t0, size_t n, unsigned blocks) {
    const void* xr = static_cast<const uint8_t*>(x) + t0 * row;
    if (p.x_dtype == MOE_BF16)
      quantize_mxfp4_kernel<true><<<blocks, 256, 0, s>>>(xr, n, cpr, cs, ss, codes + t0 * cs, scales + t0 * ss);
    else
      quantize_mxfp4_kernel<false><<<blocks, 256, 0, s>>>(xr, n, cpr, cs, ss, codes + t0 * cs, scales + t0 * ss);
  });
}

hipError_t launch_dequantize_mxfp4(const moe_problem_t& p, const uint8_t* codes, const uint8_t* scales, void* x,
                                   hipStream_t s) {
  const int cpr = p.d / 8;
  const size_t cs = mx_codes_stride(p.d), ss = mx_scales_stride(p.d);
  const size_t row = static_cast<size_t>(p.d) * (p.x_dtype == MOE_BF16 ? 2 : 4);
  return by_rows(p.T, cpr, [&](size_t t0, size_t n, unsigned blocks) {
    void* xr = static_cast<uint8_t*>(x) + t0 * row;
    if (p.x_dtype == MOE_BF16)
      dequantize_mxfp4_kernel<true><<<blocks, 256, 0, s>>>(codes + t0 * cs, scales + t0 * ss, n, cpr, cs, ss, xr);
    else
      dequantize_mxfp4_kernel<false><<<blocks, 256, 0, s>>>(codes + t0 * cs, scales + t0 * ss, n, cpr, cs, ss, xr);
  });
}

hipError_t launch_pack_mxfp4(const moe_problem_t& p, const void* Wg, const void* W1, const void* W3, const void* W2,
                             void* packed, hipStream_t s) {
  const PackedMxLayout L = layout_of(p);
  uint8_t* base = static_cast<uint8_t*>(packed);
  const bool bf = p.w_dtype == MOE_BF16;
  hipError_t e = launch_pack_router(p, Wg, base + L.router, s);
  if (e != hipSuccess) return e;
  e = gate_rows(p) == 2 ? pack_mat<2>(bf, W1, W3, p.E_local, p.d, p.I, base + L.w13, base + L.w13s, s)
                        : pack_mat<1>(bf, W1, nullptr, p.E_local, p.d, p.I, base + L.w13, base + L.w13s, s);
  if (e != hipSuccess) return e;
  return pack_mat<1>(bf, W2, nullptr, p.E_local, p.I, p.d, base + L.w2, base + L.w2s, s);
}

hipError_t launch_unpack_mxfp4(const moe_problem_t& p, const void* packed, void* W1, void* W3, void* W2,
                               hipStream_t s) {
  const PackedMxLayout L = layout_of(p);
  const uint8_t* base = static_cast<const uint8_t*>(packed);
  const bool bf = p.w_dtype == MOE_BF16;
  const hipError_t e =
      gate_rows(p) == 2 ? unpack_mat<2>(bf, base + L.w13, base + L.w13s, p.E_local, p.d, p.I, W1, W3, s)
                        : unpack_mat<1>(bf, base + L.w13, base + L.w13s, p.E_local, p.d, p.I, W1, nullptr, s);
  if (e != hipSuccess) return e;
  return unpack_mat<1>(bf, base + L.w2, base + L.w2s, p.E_local, p.I, p.d, W2, nullptr, s);
}

}  // namespace moe
