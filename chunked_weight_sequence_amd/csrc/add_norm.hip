// RMS norm of a residual stream with the residual's addition, in one pass, to the input's type or to 8
// bits with scales.
//
// For row n of D channels:
//     h = x + r                                        (h = x without a residual), written as S
//     y = h * rsqrt(mean(h^2) + eps) * w               (w = 1 where none is given)
// Y holds y in the input's type, or, for an output in 8 bits, e4m3(y / scale) with
//     scale = max(max |y| / 448, 2^-126)               of the row, or of each group of channels.
// fp32 arithmetic on the unrounded sum h, each output rounded once (448 is e4m3's largest value, so nothing
// saturates; 2^-126 keeps scales normal numbers, and rows of zeros from dividing by zero).
//
// Bound by HBM: each input is read once and each output written once. A row is held in registers by one
// wave, or by a workgroup's four, 8 channels of a lane side by side; rows are taken by new workgroups, not in a
// loop, with which fewer are under way at once. The largest |h w| of a scale is found together with the sum of
// squares, since the factor between h w and y is one of the whole row. With a residual: 32768 x 2560 bf16 to e4m3 by
// 128, 587 MB, 110 us (5.3 TB/s; in a loop, with the next row read ahead and the weights kept, 165), to bf16, 671 MB,
// 125 us; 4099 x 1000 fp32, 66 MB, 14 us; 512 x 2560 bf16 6 us.
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace ttt {
namespace {

// 8 channels as they lie in memory.
template <typename T>
struct Eight {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(v[i].x);
        x[4 * i + 1] = __uint_as_float(v[i].y);
        x[4 * i + 2] = __uint_as_float(v[i].z);
        x[4 * i + 3] = __uint_as_float(v[i].w);
      }
    }
  }
  __device__ __forceinline__ void pack(const float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
      v[0] = make_uint4(pack2bf(x[0], x[1]), pack2bf(x[2], x[3]), pack2bf(x[4], x[5]), pack2bf(x[6], x[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                          __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
    }
  }
};

// 8 values in e4m3, rounded to nearest even.
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8]) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
  return make_uint2(uint32_t(lo), uint32_t(hi));
}

// y / scale, rounded to nearest: the product with the rounded reciprocal and a correction by its remainder, which fp32
// holds exactly where the quotient is not below every code and the scale not near fp32's ends (Markstein 1990). Rows
// with other scales divide. By 128, 32768 x 2560: 110 us, with divisions 113, with the product alone, whose two roundings put
// values beside a tie on the other code, 108.
struct Quotient {
  float scale, inv;
  bool plain;
  __device__ __forceinline__ explicit Quotient(float s) : scale(s), inv(1.f / s), plain(s > 0x1p-80f && s < 0x1p100f) {}
  __device__ __forceinline__ float operator()(float y) const {
    const float q = y * inv;
    return fmaf(fmaf(-q, scale, y), inv, q);
  }
};

// W waves to a row, CH times 8 channels to a lane.
template <typename T, bool E4M3, int W, int CH>
__global__ __launch_bounds__(256) void k_add_norm(AddNormArgs a) {
  __shared__ float2 part[2][4];  // of the sums, and of those that are taken again
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int li = W == 1 ? lane : tid, D = a.D, n8 = D >> 3;
  const long n = (long(blockIdx.y) * gridDim.x + blockIdx.x) * (4 / W) + (W == 1 ? wave : 0);
  if (n >= a.N) return;  // the same for all waves of a row
  const T *X = static_cast<const T*>(a.X) + n * a.xs, *R = static_cast<const T*>(a.R) + n * a.rs;
  const bool with_r = a.R != nullptr;

  bool on[CH];
  Eight<T> x[CH], r[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    on[i] = i * 64 * W + li < n8;
    if (on[i]) {
      x[i].load(X + 8 * (i * 64 * W + li));
      if (with_r) r[i].load(R + 8 * (i * 64 * W + li));
    }
  }
  float w[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[i][e] = 1.f;
    if (a.w && on[i]) {
      const float4* p = reinterpret_cast<const float4*>(a.w + 8 * (i * 64 * W + li));
      const float4 u = p[0], v = p[1];
      w[i][0] = u.x, w[i][1] = u.y, w[i][2] = u.z, w[i][3] = u.w;
      w[i][4] = v.x, w[i][5] = v.y, w[i][6] = v.z, w[i][7] = v.w;
    }
  }
  // sum of squares and largest |h w| of the row
  int turn = 0;
  const auto reduce = [&](float& ss, float& top) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      ss += __shfl_xor(ss, d);
      if (E4M3) top = fmaxf(top, __shfl_xor(top, d));
    }
    if constexpr (W > 1) {
      if (lane == 0) part[turn][wave] = make_float2(ss, top);
      __syncthreads();
      ss = part[turn][0].x;
      top = part[turn][0].y;
#pragma unroll
      for (int i = 1; i < W; ++i) {
        ss += part[turn][i].x;
        top = fmaxf(top, part[turn][i].y);
      }
      turn ^= 1;
    }
  };
  float h[CH][8], ss = 0.f, top = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = 0.f;
    if (!on[i]) continue;
    x[i].unpack(h[i]);
    if (with_r) {
      float b[8];
      r[i].unpack(b);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] += b[e];
    }
    if (a.S) {
      Eight<T> s;
      s.pack(h[i]);
      s.store(static_cast<T*>(a.S) + n * a.ss + 8 * (i * 64 * W + li));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ss = fmaf(h[i][e], h[i][e], ss);
      if (E4M3) top = fmaxf(top, fabsf(h[i][e] * w[i][e]));
    }
  }
  reduce(ss, top);
  float eps = a.eps;
  // Squares that leave fp32 (values past 2^63, or all below 2^-40 where eps does not hide them): the row is
  // scaled by a power of two first. All lanes of a row decide alike.
  const bool large = !(ss < 0x1p126f), small = ss < 0x1p-80f && eps < 0x1p-80f;
  if (__builtin_expect(large || small, 0)) {
    const float s = large ? 0x1p-72f : 0x1p96f;
    ss = top = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[i][e] *= s;
        ss = fmaf(h[i][e], h[i][e], ss);
        if (E4M3) top = fmaxf(top, fabsf(h[i][e] * w[i][e]));
      }
    reduce(ss, top);
    eps = eps * s * s;
  }
  const float rs = rsqrtf(ss / float(D) + eps);
  if constexpr (E4M3) {
    const int per = a.group >> 3;  // lanes to a group, a power of two
    const long sn = a.group ? n * (D / a.group) : n;
    float most = top * rs;  // |y|
    if (!a.group && __builtin_expect(!(top > 0x1p-100f && top < 0x1p126f), 0)) {
      // a weight far from 1: h w leaves fp32 where y need not
      float none = 0.f;
      most = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(h[i][e] * rs * w[i][e]));
      reduce(none, most);
    }
    Quotient by(fmaxf(most / 448.f, 0x1p-126f));
    if (!a.group && li == 0) a.scales[sn] = by.scale;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float y[8], g = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = h[i][e] * rs * w[i][e];
        g = fmaxf(g, fabsf(y[e]));
      }
      if (a.group) {  // a group's lanes are all on or all off
        for (int d = 1; d < per; d *= 2) g = fmaxf(g, __shfl_xor(g, d));
        by = Quotient(fmaxf(g / 448.f, 0x1p-126f));
        const int c = i * 64 * W + li;
        if (on[i] && (c & (per - 1)) == 0) a.scales[sn + c / per] = by.scale;
      }
      if (__builtin_expect(by.plain, 1)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = by(y[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] /= by.scale;
      }
      if (on[i])
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.Y) + n * a.ys + 8 * (i * 64 * W + li)) = pack8_e4m3(y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = h[i][e] * rs * w[i][e];
      Eight<T> o;
      o.pack(y);
      if (on[i]) o.store(static_cast<T*>(a.Y) + n * a.ys + 8 * (i * 64 * W + li));
    }
  }
}

template <typename T, bool E4M3, int W, int CH>
void launch(const AddNormArgs& a) {
  const long rows = 4 / W, n = (a.N + rows - 1) / rows, most = 1 << 23;  // a launch counts its threads along x in 32 bits
  const dim3 grid(unsigned(n < most ? n : most), unsigned((n + most - 1) / most));
  hipLaunchKernelGGL((k_add_norm<T, E4M3, W, CH>), grid, dim3(256), 0, a.stream, a);
}
template <typename T, bool E4M3>
void launch(const AddNormArgs& a) {
  // Four waves to a row from 2048 channels on, and past 512 where rows are few. One wave / four, with a residual: bf16
  // 32768 x 2560 124 / 126 us, 4096 x 4096 23.6 / 23.2, 16384 x 4096 108 / 100, 16384 x 1024 22.9 / 26.6, 4096 x 512
  // 6.5 / 8.0, but 512 x 1536 6.3 / 5.6; fp32 16384 x 2048 107 / 103, 65536 x 128 29 / 50.
  const int n8 = a.D / 8;
  if (n8 >= 256 || (a.N < 2048 && n8 > 64)) {
    const int ch = (n8 + 255) / 256;
    if (ch <= 1) launch<T, E4M3, 4, 1>(a);
    else if (ch <= 2) launch<T, E4M3, 4, 2>(a);
    else if (ch <= 3) launch<T, E4M3, 4, 3>(a);
    else if (ch <= 5) launch<T, E4M3, 4, 5>(a);
    else launch<T, E4M3, 4, 8>(a);
  } else {
    const int ch = (n8 + 63) / 64;
    if (ch <= 1) launch<T, E4M3, 1, 1>(a);
    else if (ch <= 2) launch<T, E4M3, 1, 2>(a);
    else if (ch <= 3) launch<T, E4M3, 1, 3>(a);
    else launch<T, E4M3, 1, 4>(a);
  }
}

}  // namespace

hipError_t add_norm(const AddNormArgs& a) {
  if (a.bf16) a.e4m3 ? launch<uint16_t, true>(a) : launch<uint16_t, false>(a);
  else a.e4m3 ? launch<float, true>(a) : launch<float, false>(a);
  return hipGetLastError();
}

}  // namespace ttt
