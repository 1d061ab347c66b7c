// mxfp4.h -- the 4-bit microscaled format (MXFP4): device-side conversions
// and the layouts shared by the quantiser, the weight packing and the
// products.
//
// A block is 32 consecutive elements along the reduction index with one
// power-of-two scale 2^k, stored as the byte k + 127 (E8M0), and 32 E2M1
// codes (values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a
// byte, the even element in the low half.  k is the smallest integer >= -127
// with max |x| <= 6 * 2^k, so no element saturates (the rule the FP8 rows of
// quant.hip use with 448 in the place of 6); each element is x / 2^k rounded
// to the nearest E2M1 value, ties to the even code.  The largest fp32 gives
// k = 126, so the division is one exact product with 2^-k inside fp32's
// normal range (a quotient that leaves that range is far below half the
// smallest E2M1 step).  A block that holds an infinity or a NaN has scale
// byte 255 (NaN) and codes 0: all of it reads as NaN.
#pragma once

#include "moe_common.h"

namespace moe {

constexpr int kMxBlock = 32;
constexpr uint32_t kMxNan = 255;

// Bytes per row of the codes and of the scales of `cols` elements.  Codes are
// padded to whole 128-byte lines (the products fetch token rows by lines) and
// scales to 16 bytes (one load covers 512 elements); the padding is zero.
__host__ __device__ constexpr size_t mx_codes_stride(int cols) { return (static_cast<size_t>(cols) / 2 + 127) / 128 * 128; }
__host__ __device__ constexpr size_t mx_scales_stride(int cols) {
  return (static_cast<size_t>(cols) / kMxBlock + 15) / 16 * 16;
}

// Scale byte of a block from the largest magnitude's fp32 bits (sign
// cleared; compared as integers, which orders NaN above everything).  With
// |x| = 1.m * 2^e: |x| <= 6 * 2^k = 1.5 * 2^(k + 2) holds first at k = e - 2
// when 1.m <= 1.5, else at k = e - 1.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return kMxNan;
  const int e = static_cast<int>(amax_bits >> 23) - 2 + ((amax_bits & 0x7fffffu) > 0x400000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 0));
}
// 2^-k (0 for a NaN block: its codes are 0 whatever the elements).
__device__ __forceinline__ float mx_inv_scale(uint32_t sb) {
  return sb == kMxNan ? 0.0f : __uint_as_float((254u - sb) << 23);
}
// 2^k; 2^-127 is subnormal; NaN for byte 255.
__device__ __forceinline__ float mx_scale(uint32_t sb) {
  if (sb == 0) return __uint_as_float(0x00400000u);
  return __uint_as_float(sb == kMxNan ? 0x7fc00000u : sb << 23);
}

// An element times 2^-k; a NaN block's elements become 0.
__device__ __forceinline__ float mx_scaled(float v, float inv, uint32_t sb) { return sb == kMxNan ? 0.0f : v * inv; }

// Eight codes (element 0 in the lowest four bits) of values already divided
// by the block scale: gfx950's conversion rounds to nearest even, scale 1.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8]) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], 1.0f, 3);
  return r;
}

// The eight values of a word of codes, times the block scale.  An E2M1 value
// times a power of two is exact in fp32 and in bf16 down to scale 2^-127.
__device__ __forceinline__ void mx_values8(uint32_t codes, float scale, float (&v)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
  v[0] = a.x * scale; v[1] = a.y * scale; v[2] = b.x * scale; v[3] = b.y * scale;
  v[4] = c.x * scale; v[5] = c.y * scale; v[6] = d.x * scale; v[7] = d.y * scale;
}

// Two such values as bf16: they have at most three significant bits, so the
// upper halves are the exact values, also below bf16's normal range, which
// the conversion instruction was seen to flush to zero.
__device__ __forceinline__ uint32_t mx_bf16x2(float lo, float hi) {
  return (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xffff0000u);
}

// ------------------------------------------------------------------ weights
//
// A packed matrix M[N][K] (N output rows, K the reduction index, N % 64 == 0,
// K % 128 == 0):
//   codes : 16 x 128 fragments of 1 KiB, slot s (16 bytes) = row s % 16,
//           block s / 16 of the fragment: lane s's operand of
//           v_mfma_scale_f32_16x16x128_f8f6f4.  Fragments of a row block are
//           consecutive along K (frag_offset with KB = K / 128).
//   scales: per 64 rows (four row blocks) and 128 k, 64 words: word l, byte a
//           = scale of row block a, row l % 16, block l / 16.  So one word a
//           lane holds the scales of four of its operands, picked by the
//           instruction's byte select.  The words of four K steps are
//           consecutive (1 KiB); K is padded to whole 512 with zero words.
__host__ __device__ constexpr int mx_kq(int K) { return (K + 511) / 512; }
__host__ __device__ constexpr size_t mx_mat_codes(int N, int K) { return static_cast<size_t>(N) * K / 2; }
__host__ __device__ constexpr size_t mx_mat_scales(int N, int K) { return static_cast<size_t>(N / 64) * mx_kq(K) * 1024; }

// The packed buffer of moe_pack_weights_mxfp4: the router weights (as in
// packed_layout, at offset 0), then per local expert W13 ([gr I][d], rows
// interleaved as in the bf16 layout) and W2^T ([d][I]), codes and scales.
struct PackedMxLayout {
  size_t router, w13, w13s, w2, w2s, total;
  int Epad;
};
__host__ __device__ inline PackedMxLayout packed_mx_layout(int d, int I, int E_global, int E_local, int x_is_bf16,
                                                           int gate_rows) {
  PackedMxLayout L;
  L.Epad = static_cast<int>(align_up(static_cast<size_t>(E_global), 128));
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 1024);
    return at;
  };
  L.router = take(static_cast<size_t>(L.Epad) * d * (x_is_bf16 ? 2 : 4));
  L.w13 = take(static_cast<size_t>(E_local) * mx_mat_codes(gate_rows * I, d));
  L.w13s = take(static_cast<size_t>(E_local) * mx_mat_scales(gate_rows * I, d));
  L.w2 = take(static_cast<size_t>(E_local) * mx_mat_codes(d, I));
  L.w2s = take(static_cast<size_t>(E_local) * mx_mat_scales(d, I));
  L.total = off;
  return L;
}

// silu(h1) * h3 for a result that goes to 4 bits: the exponential and the
// reciprocal are the hardware's (each within about an ulp; the exponent's
// product adds |h1| 2^-24), far inside a code step, where the library expf
// and the IEEE division of the bf16 path took a third of the first product's
// time.  The limits are those of h / (1 + exp(-h)): exp2 overflows to
// infinity, whose reciprocal is 0.
__device__ __forceinline__ float mx_silu_mul(float h1, float h3) {
  return h1 * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(h1 * -1.44269504f)) * h3;
}

// ------------------------------------------------------------------ product
//
// v_mfma_scale_f32_16x16x128_f8f6f4 on two MXFP4 operands: lane l holds the
// 32 codes of row (or column) l % 16, block l / 16 (checked on the device
// against a host sum: exact), each operand's scale in byte `sel` of a word.
typedef int i32x8 __attribute__((ext_vector_type(8)));

template <int SA, int SB>
__device__ __forceinline__ f32x4 mfma_mx(const u32x4& a, const u32x4& b, const f32x4& c, uint32_t sa, uint32_t sb) {
  const i32x8 av = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w), 0, 0, 0, 0};
  const i32x8 bv = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, SA, static_cast<int>(sa), SB,
                                                          static_cast<int>(sb));
}

}  // namespace moe
