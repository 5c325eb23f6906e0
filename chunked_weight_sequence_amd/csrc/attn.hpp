// Device pieces shared by the attention kernels (attention.hip, decode.hip).
//
// A wave works on 32-row blocks of keys against 32 queries per block of columns:
//     S^T = K Q^T    v_mfma_f32_32x32x16_bf16, keys as the A operand (from LDS), queries as B
//                    (registers): lane l then holds query l % 32 and keys 8 (j / 4) + 4 (l / 32) + j % 4
//     O^T += V^T P^T the same instruction: the exponentials of a lane, rounded to bf16 in pairs,
//                    are the B operand as they stand if the 16 keys of a product are taken in the
//                    order 8 (e / 4) + 4 (l / 32) + e % 4, e = 0..7; the V^T fragments are formed
//                    in that order by transposing LDS reads. P never leaves the registers.
// The weights are rounded to bf16 for that product because the instruction takes both operands in one type
// and the values are bf16 (fp16 would not hold them): off by half a step, 2^-8 of each weight at most, the
// sum that divides them taken before. The result's distance from the 64-bit one is 1.2 to 1.4 times that of
// a result whose only rounding is its own. A second product with what the rounding left would take that
// away at half as much matrix work again: where the matrix pipe has room, in the one-token kernel, it cost 0
// to 4% (1 sequence of 4096 8.23 -> 8.41 us, 33 ragged ones 22.3 -> 23.2), the prompt kernel has none.
//
// The softmax statistics of a query are in lanes l and l + 32, its output column in the same
// lanes: a maximum needs one exchange between the halves, a rescale is a per-lane factor.
//
// LDS tiles are rows of dh bf16 in 16-byte chunks, filled by direct copies (64 lanes x 16 bytes in
// a row), so rows are not padded; chunk c of row r sits at slot c ^ ksw(r) (K) or c ^ vsw(r) (V),
// which spreads the 8 lanes of a 16-byte read pass, and the 32 lanes of a transposing one, over
// all banks.
#pragma once
#include "common.hpp"
#include "dma_row.hpp"

namespace ttt {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kMaxBf16 = 0x1.FEp127f;

template <int DH>
__device__ __forceinline__ constexpr int ksw(int r) { return r & 7; }
template <int DH>
__device__ __forceinline__ constexpr int vsw(int r) { return DH == 128 ? 4 * (r & 3) : 4 * ((r >> 1) & 1); }

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

__device__ __forceinline__ uint2 tr_read(const char* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p));
}

// One direct copy with a 64-bit address per lane, M0 written a wait state ahead.
__device__ __forceinline__ void dma16_far(const void* p, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(m0));
}

__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// For sums of values that pass fp32 before they are divided by the sum of the weights, whose inverse is inv:
// the exponent of a power of two, 2 to 4 times that sum, that the weights are divided by first; of a power of
// two, so that equal weights of 1 still are held exactly.
__device__ __forceinline__ float headroom(float inv) { return float(2 - __builtin_amdgcn_frexp_expf(inv)); }
// Such a mean, which weights that were rounded up may carry past the largest bf16; infinities stay.
__device__ __forceinline__ float in_range(float x) {
  return fabsf(x) < INFINITY ? fminf(fmaxf(x, -kMaxBf16), kMaxBf16) : x;
}

// 1 / l and m * scale + ln l of a row with the largest logit m (before the scale) and the sum of weights l: 0
// and -inf for a row that sees nothing. Without weights below a finite maximum, the logits times log2(e)
// passed fp32: NaN.
__device__ __forceinline__ float inverse_sum(float l, float m) {
  return l == 0.f ? (m == -INFINITY ? 0.f : NAN) : 1.f / l;
}
__device__ __forceinline__ float log_sum(float l, float m, float scale) {
  return l == 0.f ? (m == -INFINITY ? -INFINITY : NAN) : m * scale + __logf(l);
}

// Byte offsets, inside a tile, of a lane's K and V^T fragments.
template <int DH>
struct FragOff {
  static constexpr int kN = 4, vN = DH / 32;
  uint32_t k[kN], v[vN];
  __device__ __forceinline__ explicit FragOff(int lane) {
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      k[i] = uint32_t(r * DH * 2 + (((2 * i + h) ^ ksw<DH>(r)) << 4));
#pragma unroll
    for (int i = 0; i < vN; ++i) v[i] = channels(lane, i);
  }
  // a lane's place of channels 32 dt ..
  __device__ __forceinline__ static uint32_t channels(int lane, int dt) {
    const int vr = 4 * (lane >> 5) + ((lane & 15) >> 2);
    const int c = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    return uint32_t(vr * DH * 2 + (((4 * dt + c) ^ vsw<DH>(vr)) << 4) + 8 * (lane & 1));
  }
  // K fragment of 32-row block kb, contraction step ks (channels 16 ks ..)
  __device__ __forceinline__ uint4 key(const char* tile, int kb, int ks) const {
    return *reinterpret_cast<const uint4*>(tile + k[ks & 3] + kb * 32 * DH * 2 + (ks >> 2) * 128);
  }
  // V^T fragment of channels 32 dt .., the 16 keys 16 s ..
  __device__ __forceinline__ uint4 value(const char* tile, int s, int dt) const {
    return value_at(tile + v[dt], s);
  }
  // the same from the lane's place of the channels
  __device__ __forceinline__ static uint4 value_at(const char* place, int s) {
    const uint2 lo = tr_read(place + s * 16 * DH * 2);
    const uint2 hi = tr_read(place + (s * 16 + 8) * DH * 2);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
};

}  // namespace ttt
