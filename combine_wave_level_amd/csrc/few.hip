// few.hip -- the whole layer for a few tokens (T <= 16): router, top-k, both
// expert products and the combine, without dispatch tables.
//
// At most 16 tokens means at most 16 rows an expert: one 16-column block of
// the matrix instruction.  The layer is then a stream of the touched
// experts' weights, each fragment used once, so it goes from memory straight
// into the operand registers of the wavefront that multiplies it (no LDS
// stage: nothing would be shared), with the loads of the next fragments in
// flight.  The tokens' operands are laid out k-major (16-byte pieces of one
// k-group of all rows side by side), so that one matrix instruction's operand
// is at most 1 KiB of consecutive memory, from the caches.
//
// The routing is that of moe_route bit for bit (the same chains of matrix
// instructions, partial sums and selection order), and the expert products
// that of the composed path: the same instruction over the same unsplit
// ascending K for every element.  The one difference is that the pairs' y
// never leave the chip here, so they are not rounded to bf16 before the
// combine.
#include "ffn_parts.h"
#include "moe_internal.h"
#include "mxfp4.h"

namespace moe {
namespace {

constexpr int kFew = MOE_FEW_MAX_TOKENS;
static_assert(kFew == 16, "one column block of the matrix instruction");
constexpr int kMaxE = 256, kMaxK = 64;

struct FewArgs {
  const void* x;
  const void* wg;          // router weights (packed buffer, offset 0)
  const float* bias;
  const uint8_t* w13;      // codes (bf16 or MXFP4 fragments) and MXFP4 scales
  const uint8_t* w13s;
  const uint8_t* w2;
  const uint8_t* w2s;
  float* partial;          // [splits][T][E]
  uint8_t* xs;             // staged token operand, k-major; MXFP4: codes, then scales
  uint8_t* act;            // activations, per slot k-major; MXFP4: codes, then scales
  int32_t* topk_idx;
  float* topk_w;
  float* logits;
  void* out;
  int T, d, I, E, k, e_begin, E_local, splits;
};

// ------------------------------------------------------------------ the stream

// One wavefront: 16 rows of router weights times the tokens over n K steps of
// 32.  w, b: the rows' fragments and the tokens for this lane, 1 KiB and 64
// bytes apart.  U fragments are in flight.
template <int U>
__device__ __forceinline__ f32x4 few_stream(const uint8_t* __restrict__ w, const uint8_t* __restrict__ b, int n) {
  u32x4 ra[U], rb[U];
  auto load = [&](int u, int i) {
    i = min(i, n - 1);
    ra[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + static_cast<size_t>(i) * 1024));
    rb[u] = ld16(b + static_cast<size_t>(i) * 64);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, u);
  f32x4 acc{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < n; i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u < n) acc = mfma16x16x32(ra[u], rb[u], acc);
      load(u, i + u + U);
    }
  }
  return acc;
}

// U K steps of operands in flight for RB row blocks.
template <bool MX, int RB, int U>
struct FewRing {
  u32x4 a[U][RB], b[U];
  uint32_t sa[U], sb[U];
  // w, w + w1: the row blocks' fragments; ws: their scale words, bs: scale byte
  __device__ __forceinline__ void load(int u, const uint8_t* w, size_t w1, const uint8_t* t, const uint8_t* ws,
                                       const uint8_t* bs) {
    a[u][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w));
    if constexpr (RB == 2) a[u][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + w1));
    b[u] = ld16(t);
    if constexpr (MX) {
      sa[u] = *reinterpret_cast<const uint32_t*>(ws);
      sb[u] = *bs;
    }
  }
  // shift: to the first row block's byte of the scale word
  __device__ __forceinline__ void multiply(int u, f32x4 (&acc)[RB], int shift) const {
    if constexpr (MX) {
      const uint32_t s = sa[u] >> shift;
      acc[0] = mfma_mx<0, 0>(a[u][0], b[u], acc[0], s, sb[u]);
      if constexpr (RB == 2) acc[1] = mfma_mx<1, 0>(a[u][1], b[u], acc[1], s, sb[u]);
    } else {
      acc[0] = mfma16x16x32(a[u][0], b[u], acc[0]);
      if constexpr (RB == 2) acc[1] = mfma16x16x32(a[u][1], b[u], acc[1]);
    }
  }
};

// ------------------------------------------------------------------ kernel 1

// Partial logits of 16 experts over one range of d by one wavefront: the
// chain of matrix instructions of router_logits_mfma_kernel.
__device__ __forceinline__ void few_logits_bf16(const FewArgs& A, int job) {
  const int lane = lane_id(), r = lane & 15, g = lane >> 4;
  const int neb = (A.E + 15) / 16, eb = job % neb, sp = job / neb;
  const int ks = A.d / A.splits / 32, kb0 = sp * ks;
  const uint16_t* w = static_cast<const uint16_t*>(A.wg) + frag_offset(eb, kb0, A.d / 32) + lane * 8;
  const uint16_t* xr = static_cast<const uint16_t*>(A.x) + static_cast<size_t>(min(r, A.T - 1)) * A.d + kb0 * 32 + g * 8;
  const f32x4 acc = few_stream<16>(reinterpret_cast<const uint8_t*>(w), reinterpret_cast<const uint8_t*>(xr), ks);
  if (r < A.T) {
    float* o = A.partial + (static_cast<size_t>(sp) * A.T + r) * A.E;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (eb * 16 + 4 * g + i < A.E) o[eb * 16 + 4 * g + i] = acc[i];
  }
}

// fp32 logits of 16 experts for all tokens by one workgroup: thread (t, e)
// runs router_logits_f32_kernel's chain of fused multiply-adds over the
// hidden index, both operands staged through LDS 128 indices at a time.
__device__ __forceinline__ void few_logits_f32(const FewArgs& A, int eb, float* lds) {
  const int Epad = static_cast<int>(align_up(static_cast<size_t>(A.E), 128));
  const float *x = static_cast<const float*>(A.x), *wg = static_cast<const float*>(A.wg);
  const int t = threadIdx.x / 16, e = threadIdx.x % 16;
  float* sx = lds;              // [16][128]
  float* sw = lds + 16 * 128;   // [128][16]
  float nx[8], nw[8], acc = 0.f;
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = i * 256 + threadIdx.x;
      nx[i] = j / 128 < A.T ? x[static_cast<size_t>(j / 128) * A.d + k0 + j % 128] : 0.f;
      nw[i] = wg[static_cast<size_t>(k0 + j / 16) * Epad + eb * 16 + j % 16];
    }
  };
  fetch(0);
  for (int k0 = 0; k0 < A.d; k0 += 128) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sx[i * 256 + threadIdx.x] = nx[i];
      sw[i * 256 + threadIdx.x] = nw[i];
    }
    __syncthreads();
    if (k0 + 128 < A.d) fetch(k0 + 128);
#pragma unroll 16
    for (int i = 0; i < 128; ++i) acc = fmaf(sx[t * 128 + i], sw[i * 16 + e], acc);
  }
  if (t < A.T && eb * 16 + e < A.E) A.partial[static_cast<size_t>(t) * A.E + eb * 16 + e] = acc;
}

// Stages eight elements of a token's row: bf16 (rounded from fp32), or codes
// and scale (the quantiser's arithmetic; four lanes share a block).
template <bool XBF, bool MX>
__device__ __forceinline__ void few_stage(const FewArgs& A, int i) {
  const int cpr = A.d / 8;
  if (i >= A.T * cpr) return;  // cpr % 4 == 0: the lanes of a block leave together
  const int t = i / cpr, c = i % cpr;
  float v[8];
  u32x4 raw{};
  if constexpr (XBF) {
    raw = ld16(static_cast<const uint16_t*>(A.x) + static_cast<size_t>(i) * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(raw[j] << 16);
      v[2 * j + 1] = __uint_as_float(raw[j] & 0xffff0000u);
    }
  } else {
    const float* p = static_cast<const float*>(A.x) + static_cast<size_t>(i) * 8;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  }
  if constexpr (!MX) {
    if constexpr (!XBF) raw = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    st16(A.xs + (static_cast<size_t>(c) * A.T + t) * 16, raw);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 1, kWave)));
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 2, kWave)));
    const uint32_t sb = mx_scale_byte(m);
    const float inv = mx_inv_scale(sb);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = mx_scaled(v[j], inv, sb);
    const int blk = c / 4;
    *reinterpret_cast<uint32_t*>(A.xs + (static_cast<size_t>(blk) * A.T + t) * 16 + (c % 4) * 4) = mx_codes8(v);
    if (c % 4 == 0) A.xs[static_cast<size_t>(A.T) * A.d / 2 + static_cast<size_t>(blk) * A.T + t] = static_cast<uint8_t>(sb);
  }
}

// Logits and staged rows.  Workgroups [0, nlog): logits; the rest stage.
template <bool XBF, bool MX>
__global__ __launch_bounds__(256) void few_front_kernel(FewArgs A, int nlog) {
  __shared__ float lds[XBF ? 1 : 4096];
  const int b = blockIdx.x;
  if (b < nlog) {
    if constexpr (XBF) {
      const int job = b * 4 + wave_id();
      if (job < (A.E + 15) / 16 * A.splits) few_logits_bf16(A, job);
    } else {
      few_logits_f32(A, b, lds);
    }
    return;
  }
  few_stage<XBF, MX>(A, (b - nlog) * 256 + static_cast<int>(threadIdx.x));
}

// ------------------------------------------------------------------ routing in LDS

// What every workgroup of the expert kernels derives for itself: the picks,
// their weights, and the touched local experts ("slots") with their rows.
struct FewRoute {
  int32_t idx[kFew * kMaxK];
  float val[kFew * kMaxK];     // weights
  int16_t row[kFew * kMaxK];   // pair -> pair row, -1: expert not local
  uint32_t mask[kMaxE];        // per local expert: the tokens that pick it
  int16_t slot_of[kMaxE];
  int16_t slot_e[kMaxE];       // slot -> local expert
  int16_t base[kMaxE + 1];     // slot -> first pair row
  int nslots;
};

// Largest value over the wavefront, by the lane shifts of the vector ALU.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define MOE_STEP(ctrl) v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), ctrl, 0xf, 0xf, true)))
  MOE_STEP(0x111);  // row_shr 1, 2, 4, 8
  MOE_STEP(0x112);
  MOE_STEP(0x114);
  MOE_STEP(0x118);
  MOE_STEP(0x142);  // row_bcast 15, 31
  MOE_STEP(0x143);
#undef MOE_STEP
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

// Order-preserving integer of a logit; 0 for NaN (never picked), -0 as +0
// (they tie).
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return v == v ? b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
}

// All tokens' logits into LDS: the partial sums of every element are in
// flight together (a loop over them waited out a memory round trip for each
// of up to eight, most of this kernel's time on a small layer), then added in
// ascending order, then the bias.
template <int NT>
__device__ __forceinline__ void few_logits(const FewArgs& A, float* __restrict__ lg, bool write) {
  const int TE = A.T * A.E;
  for (int i0 = threadIdx.x; i0 < TE; i0 += 4 * NT) {
    float p[4][8], bias[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = min(i0 + u * NT, TE - 1);
#pragma unroll
      for (int sp = 0; sp < 8; ++sp) p[u][sp] = sp < A.splits ? A.partial[static_cast<size_t>(sp) * TE + i] : 0.f;
      bias[u] = A.bias ? A.bias[i % A.E] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * NT;
      if (i >= TE) break;
      float acc = p[u][0];
#pragma unroll
      for (int sp = 1; sp < 8; ++sp)
        if (sp < A.splits) acc += p[u][sp];
      if (A.bias) acc += bias[u];
      lg[i] = acc;
      if (write && A.logits) A.logits[i] = acc;
    }
  }
}

// topk_token's selection for token t by one wavefront, with the same picks
// and the same weights: k rounds of the largest value, ties to the lower
// expert, NaN never; a token without enough comparable logits is left
// 0x7fffffff and its weights come out NaN as there.  Every workgroup waits for
// this chain, so a round is kept short: integer keys and lane shifts take
// 0.1 us, topk_token's lane exchanges of (value, index) pairs several times
// that.
__device__ __forceinline__ void few_topk(const FewArgs& A, FewRoute& R, const float* __restrict__ lg, int t, bool write) {
  const int lane = lane_id(), nq = (A.E + kWave - 1) / kWave;
  uint32_t key[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = lane + 64 * q;
    key[q] = e < A.E ? logit_key(lg[t * A.E + e]) : 0u;
  }
  float my_v = -__builtin_inff();
  int my_i = 0x7fffffff;
  for (int j = 0; j < A.k; ++j) {
    uint32_t mine = key[0];
    if (nq > 1) mine = max(mine, key[1]);
    if (nq > 2) mine = max(mine, max(key[2], key[3]));
    const uint32_t best = wave_max(mine);
    if (best == 0) break;  // no comparable logit left
    int win = 0;
#pragma unroll
    for (int q = 3; q >= 0; --q)
      if (q < nq) {
        const unsigned long long m = __ballot(key[q] == best);
        if (m) win = 64 * q + __ffsll(m) - 1;
      }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < nq && lane + 64 * q == win) key[q] = 0;
    if (lane == j) {
      my_v = key_logit(best);
      my_i = win;
    }
  }
  const float vmax = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_v), 0));
  const float ex = lane < A.k ? expf(my_v - vmax) : 0.f;
  float sum = 0.f;
  for (int j = 0; j < A.k; ++j) sum += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ex), j));  // ascending
  if (lane < A.k) {
    const float w = ex / sum;
    R.idx[t * A.k + lane] = my_i;
    R.val[t * A.k + lane] = w;
    if (write) {
      A.topk_idx[t * A.k + lane] = my_i;
      A.topk_w[t * A.k + lane] = w;
    }
  }
}

// FROM_LOGITS: selects from the partial logits; else takes the picks and
// weights that the first expert kernel wrote.
template <int NT, bool FROM_LOGITS>
__device__ __forceinline__ void few_route(const FewArgs& A, FewRoute& R, float* __restrict__ lg, bool write) {
  const int tid = threadIdx.x, TK = A.T * A.k;
  for (int i = tid; i < kMaxE; i += NT) R.mask[i] = 0;
  if constexpr (FROM_LOGITS) {
    few_logits<NT>(A, lg, write);
    __syncthreads();
    for (int t = uniform(wave_id()); t < A.T; t += NT / kWave) few_topk(A, R, lg, t, write);
  } else {
    for (int i = tid; i < TK; i += NT) {
      R.idx[i] = A.topk_idx[i];
      R.val[i] = A.topk_w[i];
    }
  }
  __syncthreads();
  for (int i = tid; i < TK; i += NT) {
    const int le = R.idx[i] - A.e_begin;
    if (le >= 0 && le < A.E_local) atomicOr(&R.mask[le], 1u << (i / A.k));
  }
  __syncthreads();
  if (wave_id() == 0) {
    const int lane = lane_id();
    int slots = 0, rows = 0;
    for (int c = 0; c * kWave < A.E_local; ++c) {
      const int e = c * kWave + lane, n = __popc(R.mask[e]);
      int incl = n;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const int o = __shfl_up(incl, off, kWave);
        incl += lane >= off ? o : 0;
      }
      const unsigned long long any = __ballot(n > 0);
      const int s = slots + __popcll(any & ((1ull << lane) - 1));
      if (n > 0) {
        R.slot_e[s] = static_cast<int16_t>(e);
        R.slot_of[e] = static_cast<int16_t>(s);
        R.base[s] = static_cast<int16_t>(rows + incl - n);
      }
      slots += __popcll(any);
      rows += __shfl(incl, kWave - 1, kWave);
    }
    if (lane == 0) {
      R.base[slots] = static_cast<int16_t>(rows);
      R.nslots = slots;
    }
  }
  __syncthreads();
  if constexpr (FROM_LOGITS) return;  // the pairs' rows are the combine's
  for (int i = tid; i < TK; i += NT) {
    const int t = i / A.k, le = R.idx[i] - A.e_begin;
    R.row[i] = le >= 0 && le < A.E_local
                   ? static_cast<int16_t>(R.base[R.slot_of[le]] + __popc(R.mask[le] & ((1u << t) - 1)))
                   : static_cast<int16_t>(-1);
  }
  __syncthreads();
}

// Token of row r of a slot's mask (r < popcount).
__device__ __forceinline__ int nth_bit(uint32_t mask, int r) {
  for (int i = 0; i < r; ++i) mask &= mask - 1;
  return __ffs(mask) - 1;
}

constexpr int kHStride = 17;  // floats per row of the h exchange

// LDS-only barrier: the loads in flight stay in flight.
__device__ __forceinline__ void few_lds_barrier() {
  wait_lgkm0();
  raw_barrier();
}

// Activation of a GEMM1 task (64 RB packed rows: 32 RB intermediate indices
// gated, 64 RB ungated) from the four wavefronts' accumulators: gate and up meet in
// LDS, and 16 consecutive lanes hold one token's block of 32 for the scale.
template <bool MX, bool GATED, int RB>
__device__ __forceinline__ void few_act(const FewArgs& A, const FewRoute& R, float* h, int slot, int nq, const f32x4 (&acc)[RB]) {
  const int lane = lane_id(), r = lane & 15, g = lane >> 4;
  const int base = R.base[slot], m = R.base[slot + 1] - base;
  few_lds_barrier();  // h free
#pragma unroll
  for (int a = 0; a < RB; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) h[((wave_id() * RB + a) * 16 + 4 * g + i) * kHStride + r] = acc[a][i];
  few_lds_barrier();
  const int t = threadIdx.x / 16, p = threadIdx.x % 16;  // row of the slot, element pair of a block
  constexpr int NBLK = RB * (GATED ? 1 : 2);  // blocks of 32 along I
#pragma unroll
  for (int blk = 0; blk < NBLK; ++blk) {
    float v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = 2 * p + i;  // element of the block
      if constexpr (GATED) {
        const int hr = blk * 64 + (q / 16) * 32 + q % 16;
        const float h1 = h[hr * kHStride + t], h3 = h[(hr + 16) * kHStride + t];
        v[i] = MX ? mx_silu_mul(h1, h3) : silu_mul(h1, h3);
      } else {
        v[i] = relu_sq(h[(blk * 32 + q) * kHStride + t]);
      }
    }
    const int kb = nq * NBLK + blk;  // block of 32 along I
    if constexpr (MX) {
      uint32_t mb = max(__float_as_uint(v[0]) & 0x7fffffffu, __float_as_uint(v[1]) & 0x7fffffffu);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) mb = max(mb, static_cast<uint32_t>(__shfl_xor(static_cast<int>(mb), o, kWave)));
      const uint32_t sb = mx_scale_byte(mb);
      const float inv = mx_inv_scale(sb);
      uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, mx_scaled(v[0], inv, sb), mx_scaled(v[1], inv, sb), 1.0f, 0) & 0xffu;
      c |= static_cast<uint32_t>(__shfl_xor(static_cast<int>(c), 1, kWave)) << 8;   // even lanes: two bytes
      c |= static_cast<uint32_t>(__shfl_xor(static_cast<int>(c), 2, kWave)) << 16;  // lanes 0 mod 4: four
      if (t < m) {
        const size_t P = R.base[R.nslots];
        uint8_t* ac = A.act + static_cast<size_t>(base) * A.I / 2 + (static_cast<size_t>(kb) * m + t) * 16;
        if (p % 4 == 0) *reinterpret_cast<uint32_t*>(ac + p) = c;
        if (p == 0) A.act[P * A.I / 2 + static_cast<size_t>(base) * (A.I / 32) + static_cast<size_t>(kb) * m + t] = static_cast<uint8_t>(sb);
      }
    } else if (t < m) {
      const int q = 2 * p;
      uint8_t* ac = A.act + static_cast<size_t>(base) * A.I * 2 + ((static_cast<size_t>(kb) * 4 + q / 8) * m + t) * 16 + (q % 8) * 2;
      *reinterpret_cast<uint32_t*>(ac) = pack_bf16x2(v[0], v[1]);
    }
  }
}

// The GEMM1 tasks blockIdx.x, + gridDim.x, ... of n (slot i / per, 64 RB packed
// rows i % per), RB row blocks a wavefront (few_row_blocks).  The loads run on
// from one task into the next, as in few_gemm2.
template <bool MX, bool GATED, int RB, int U>
__device__ __forceinline__ void few_gemm1(const FewArgs& A, const FewRoute& R, float* h, int n, int per) {
  const int lane = lane_id(), r = lane & 15, g = lane >> 4, wave = uniform(wave_id());
  const int N = (GATED ? 2 : 1) * A.I, KB = MX ? A.d / 128 : A.d / 32, step = static_cast<int>(gridDim.x);
  const uint8_t *w = nullptr, *b = nullptr, *ws = nullptr, *bs = nullptr;
  const uint32_t bstep = 64 * A.T;
  uint32_t on = 1;  // 0 behind the last task: the same address again
  int li = static_cast<int>(blockIdx.x) - step, left = 0;
  if (li + step >= n) return;
  auto next = [&]() {
    li += step;
    if (li >= n) {
      on = 0;
      w -= 1024, b -= bstep;
      if (MX) ws -= 256, bs -= bstep / 16;
      left = 1 << 30;
      return;
    }
    const int slot = uniform(li / per), nb = (uniform(li % per) * 4 + wave) * RB;
    const int e = uniform(R.slot_e[slot]), m = uniform(R.base[slot + 1] - R.base[slot]);
    const int tok = nth_bit(R.mask[e], min(r, m - 1));
    left = KB;
    b = A.xs + (static_cast<size_t>(g) * A.T + tok) * 16;
    if constexpr (MX) {
      w = A.w13 + e * mx_mat_codes(N, A.d) + static_cast<size_t>(nb) * KB * 1024 + lane * 16;
      ws = A.w13s + e * mx_mat_scales(N, A.d) + static_cast<size_t>(nb / 4) * mx_kq(A.d) * 1024 + lane * 4;
      bs = A.xs + static_cast<size_t>(A.T) * A.d / 2 + static_cast<size_t>(g) * A.T + tok;
    } else {
      w = A.w13 + (static_cast<size_t>(e) * N * A.d + frag_offset(nb, 0, KB)) * 2 + lane * 16;
    }
  };
  const size_t w1 = static_cast<size_t>(KB) * 1024;  // to the second row block
  const int shift = 8 * (wave * RB % 4);             // the wavefront's bytes of a scale word
  FewRing<MX, RB, U> ring;
  auto load = [&](int u) {
    ring.load(u, w, w1, b, ws, bs);
    w += on * 1024;
    b += on * bstep;
    if (MX) ws += on * 256, bs += on * (bstep / 16);
    if (--left == 0) next();
  };
  next();
#pragma unroll
  for (int u = 0; u < U; ++u) load(u);
  f32x4 acc[RB] = {};
  int ci = static_cast<int>(blockIdx.x), todo = KB;
  while (ci < n) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (ci < n) {
        ring.multiply(u, acc, shift);
        if (--todo == 0) {
          few_act<MX, GATED, RB>(A, R, h, uniform(ci / per), uniform(ci % per), acc);
#pragma unroll
          for (int a = 0; a < RB; ++a) acc[a] = f32x4{0.f, 0.f, 0.f, 0.f};
          ci += step;
          todo = KB;
        }
      }
      load(u);
    }
  }
}

// GEMM2 and combine of 16 RB nrb output columns for all slots, by NW
// wavefronts.  A wavefront takes (slot, 16 RB columns) jobs; its loads run on
// from one job into the next, so the short reductions of a narrow layer do
// not drain the stream.  The pairs' y meet in LDS in fp32, and each output
// is combine_token's rank-ordered sum.
template <bool MX, bool OUT_BF16, int RB, int NW, int U>
__device__ __forceinline__ void few_gemm2(const FewArgs& A, const FewRoute& R, float* __restrict__ y, int task, int nrb) {
  const int lane = lane_id(), r = lane & 15, g = lane >> 4, cols = 16 * RB * nrb;
  const size_t P = R.base[R.nslots];
  const int KB = MX ? A.I / 128 : A.I / 32, njobs = R.nslots * nrb;
  const uint8_t *w = nullptr, *b = nullptr, *ws = nullptr, *bs = nullptr;
  uint32_t bstep = 0, wstep = 0;
  int ljob = uniform(wave_id()) - NW, left = 0;
  auto next = [&]() {  // addresses of the next job's first fragment; after the last job, the same one again
    ljob += NW;
    if (ljob >= njobs) {
      if (w) w -= wstep, b -= bstep;
      if (MX && w) ws -= wstep / 4, bs -= bstep / 16;
      wstep = bstep = 0;
      left = 1 << 30;
      return;
    }
    const int slot = uniform(ljob / nrb), nb = (task * nrb + uniform(ljob % nrb)) * RB;
    const int e = uniform(R.slot_e[slot]), base = uniform(R.base[slot]), m = uniform(R.base[slot + 1]) - base;
    const int rr = min(r, m - 1);
    wstep = 1024;
    bstep = 64 * m;
    left = KB;
    if constexpr (MX) {
      w = A.w2 + e * mx_mat_codes(A.d, A.I) + static_cast<size_t>(nb) * KB * 1024 + lane * 16;
      ws = A.w2s + e * mx_mat_scales(A.d, A.I) + static_cast<size_t>(nb / 4) * mx_kq(A.I) * 1024 + lane * 4;
      b = A.act + static_cast<size_t>(base) * A.I / 2 + (static_cast<size_t>(g) * m + rr) * 16;
      bs = A.act + P * A.I / 2 + static_cast<size_t>(base) * (A.I / 32) + static_cast<size_t>(g) * m + rr;
    } else {
      w = A.w2 + (static_cast<size_t>(e) * A.d * A.I + frag_offset(nb, 0, KB)) * 2 + lane * 16;
      b = A.act + static_cast<size_t>(base) * A.I * 2 + (static_cast<size_t>(g) * m + rr) * 16;
    }
  };
  __syncthreads();  // y free
  if (uniform(wave_id()) < njobs) {
    const size_t w1 = static_cast<size_t>(KB) * 1024;  // to the second row block
    FewRing<MX, RB, U> ring;
    auto load = [&](int u) {
      ring.load(u, w, w1, b, ws, bs);
      if (MX) ws += wstep / 4, bs += bstep / 16;
      w += wstep;
      b += bstep;
      if (--left == 0) next();
    };
    next();
#pragma unroll
    for (int u = 0; u < U; ++u) load(u);
    f32x4 acc[RB] = {};
    int job = uniform(wave_id()), todo = KB;
    while (job < njobs) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (job < njobs) {
          const int rb = uniform(job % nrb);
          ring.multiply(u, acc, 8 * ((task * nrb + rb) * RB % 4));
          if (--todo == 0) {
            const int slot = uniform(job / nrb), base = uniform(R.base[slot]), m = uniform(R.base[slot + 1]) - base;
            if (r < m) {
              float* yr = y + (base + r) * cols + rb * 16 * RB + 4 * g;
#pragma unroll
              for (int a = 0; a < RB; ++a) *reinterpret_cast<f32x4*>(yr + 16 * a) = acc[a];
            }
#pragma unroll
            for (int a = 0; a < RB; ++a) acc[a] = f32x4{0.f, 0.f, 0.f, 0.f};
            job += NW;
            todo = KB;
          }
        }
        load(u);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < A.T * cols / 2; i += 64 * NW) {
    const int t = i / (cols / 2), c = i % (cols / 2) * 2;
    float a0 = 0.f, a1 = 0.f;
    for (int j = 0; j < A.k; ++j) {
      const int row = R.row[t * A.k + j];
      if (row < 0) continue;
      const f32x2 v = *reinterpret_cast<const f32x2*>(y + row * cols + c);
      const float wj = R.val[t * A.k + j];
      a0 = fmaf(wj, v.x, a0);
      a1 = fmaf(wj, v.y, a1);
    }
    const size_t at = static_cast<size_t>(t) * A.d + static_cast<size_t>(task) * cols + c;
    if constexpr (OUT_BF16) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(A.out) + at) = pack_bf16x2(a0, a1);
    else *reinterpret_cast<f32x2*>(static_cast<float*>(A.out) + at) = f32x2{a0, a1};
  }
}

template <bool MX, bool GATED, int RB>
__global__ __launch_bounds__(256, RB == 2 ? 3 : 4) void few_gemm1_kernel(FewArgs A) {
  extern __shared__ __align__(16) float few_h[];  // the logits, then h
  __shared__ FewRoute R;
  few_route<256, true>(A, R, few_h, blockIdx.x == 0);  // ends with a barrier: the logits are free
  const int per = (GATED ? 2 : 1) * A.I / (64 * RB), n = uniform(R.nslots) * per;
  few_gemm1<MX, GATED, RB, 8>(A, R, few_h, n, per);
}

constexpr int kFewWaves2 = 8;

// y in LDS: 16 RB nrb columns a pair.  nrb is 1 from 8 slots up; with fewer
// there are at most 16 pairs a slot: 7 * 16 pairs of 32 RB columns, 3 * 16 of
// 64 RB, or 16 of 128 (RB = 1).
constexpr size_t few_y_bytes(int pairs, int rb) { return static_cast<size_t>(pairs * 16 > 3584 ? pairs * 16 : 3584) * 4 * rb; }

template <bool MX, bool OUT_BF16, int RB>
__global__ __launch_bounds__(64 * kFewWaves2, RB == 2 ? 2 : 4) void few_gemm2_kernel(FewArgs A) {
  extern __shared__ __align__(16) float few_y[];
  __shared__ FewRoute R;
  few_route<64 * kFewWaves2, false>(A, R, nullptr, false);
  // enough jobs for the wavefronts
  const int ns = uniform(R.nslots), nrb = ns >= 8 ? 1 : (ns >= 4 ? 2 : (ns >= 2 || RB == 2 ? 4 : 8));
  const int n = A.d / (16 * RB * nrb);
  // Workgroups go to the XCDs in turn.  The G tasks that share an MXFP4 scale
  // word are given to one XCD, one after the other, so that it is fetched
  // once; in plain order several XCDs fetched it, a fifth of the bytes more.
  constexpr int G = 4 / RB;
  const int shared = nrb == 1 ? n / (8 * G) * (8 * G) : 0;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int j = i / 8;
    const int task = i < shared ? (j / G * 8 + i % 8) * G + j % G : i;
    few_gemm2<MX, OUT_BF16, RB, kFewWaves2, 8>(A, R, few_y, task, nrb);
  }
}

// Row blocks a wavefront multiplies with one token operand (and, in MXFP4,
// one scale word).  Two where the layer streams: with one, the number of
// loads bound the 4-bit stream (eight tokens of d = 7168, I = 2048 on 26
// experts: 85 and 41 us for the two products, with two 74 and 35; the same
// traffic).  One where a wavefront's latency counts (13 tokens, d = 2048, I =
// 512: 17.2 and 7.7 us, with two 17.7 and 8.8) and for bf16, which has no
// scales to load (one token, d = 7168: 75 and 39 us with either; d = 2048, I =
// 768: 14.8 and 9.6 us, with two 16.9 and 13.7).  The border lies between
// 35 and 125 MB of first-product weights that the batch can touch.
int few_row_blocks(const moe_problem_t& p, bool mx, int slots) {  // 2: mx only
  return mx && static_cast<double>(slots) * gate_rows(p) * p.I * p.d / 2 >= 64e6 ? 2 : 1;
}

template <int RB>
hipError_t few_experts(const FewArgs& A, const moe_problem_t& p, bool mx, int slots, hipStream_t s) {
  const bool gated = gate_rows(p) == 2, obf = p.out_dtype == MOE_BF16;
  int dev = 0, cus = 0;
  hipError_t e;
  if ((e = hipGetDevice(&dev)) != hipSuccess) return e;
  if ((e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev)) != hipSuccess) return e;
  const int n1 = slots * (gate_rows(p) * p.I / (64 * RB)), n2 = p.d / (16 * RB);
  auto g1 = gated ? few_gemm1_kernel<true, true, RB> : few_gemm1_kernel<true, false, RB>;
  if constexpr (RB == 1)
    if (!mx) g1 = gated ? few_gemm1_kernel<false, true, RB> : few_gemm1_kernel<false, false, RB>;
  g1<<<min(n1, (RB == 2 ? 3 : 4) * cus), 256, max(64 * RB * kHStride, p.T * p.E_global) * sizeof(float), s>>>(A);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  auto g2 = obf ? few_gemm2_kernel<true, true, RB> : few_gemm2_kernel<true, false, RB>;
  if constexpr (RB == 1)
    if (!mx) g2 = obf ? few_gemm2_kernel<false, true, RB> : few_gemm2_kernel<false, false, RB>;
  g2<<<min(n2, 2 * cus), 64 * kFewWaves2, few_y_bytes(p.T * min(p.k, p.E_local), RB), s>>>(A);
  return hipGetLastError();
}

template <bool XBF, bool MX>
hipError_t front(const FewArgs& A, hipStream_t s) {
  const int jobs = (A.E + 15) / 16 * A.splits, nlog = XBF ? (jobs + 3) / 4 : (A.E + 15) / 16;
  const int stage = (A.T * (A.d / 8) + 255) / 256;
  few_front_kernel<XBF, MX><<<nlog + stage, 256, 0, s>>>(A, nlog);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_forward_few(const moe_problem_t& p, const WsLayout& L, const void* x, const void* packed, bool mx,
                              const float* bias, int32_t* topk_idx, float* topk_w, float* logits, void* out, char* ws,
                              hipStream_t s) {
  if (p.T == 0) return hipSuccess;
  const bool xbf = p.x_dtype == MOE_BF16;
  const uint8_t* base = static_cast<const uint8_t*>(packed);
  FewArgs A{};
  A.x = x;
  A.wg = packed;
  A.bias = bias;
  if (mx) {
    const PackedMxLayout PL = packed_mx_layout(p.d, p.I, p.E_global, p.E_local, xbf, gate_rows(p));
    A.w13 = base + PL.w13;
    A.w13s = base + PL.w13s;
    A.w2 = base + PL.w2;
    A.w2s = base + PL.w2s;
  } else {
    const PackedLayout PL = packed_layout(p.d, p.I, p.E_global, p.E_local, xbf, gate_rows(p));
    A.w13 = base + PL.w13;
    A.w2 = base + PL.w2;
  }
  A.partial = reinterpret_cast<float*>(ws + L.logits);
  A.xs = reinterpret_cast<uint8_t*>(ws + L.xbf);
  A.act = reinterpret_cast<uint8_t*>(ws + L.act);
  A.topk_idx = topk_idx;
  A.topk_w = topk_w;
  A.logits = logits;
  A.out = out;
  A.T = p.T;
  A.d = p.d;
  A.I = p.I;
  A.E = p.E_global;
  A.k = p.k;
  A.e_begin = p.e_begin;
  A.E_local = p.E_local;
  A.splits = router_splits(p.d, p.E_global, xbf);
  hipError_t e = xbf ? (mx ? front<true, true>(A, s) : front<true, false>(A, s))
                     : (mx ? front<false, true>(A, s) : front<false, false>(A, s));
  if (e != hipSuccess) return e;
  const int slots = min(p.E_local, p.T * p.k);  // most experts the batch can touch
  return few_row_blocks(p, mx, slots) == 2 ? few_experts<2>(A, p, mx, slots, s) : few_experts<1>(A, p, mx, slots, s);
}

}  // namespace moe
