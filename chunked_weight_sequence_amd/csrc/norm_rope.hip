// Per-head RMS norm and rotation of queries and keys in one pass, with the cache write.
//
// For token t and head x [dh] of Q or K (norm only where a weight w is given):
//     y = x * rsqrt(mean(x^2) + eps) * w
//     (a, b) -> rope_scale * (a cos - b sin, a sin + b cos)   at angle pos[t] * inv_freq[j]
// for the rot / 2 pairs of the head's first `rot` channels: (j, j + rot/2) in the half layout,
// (2j, 2j + 1) in the interleaved one. Channels past rot keep y. Everything is fp32 and rounded
// once; the angle is reduced to a fraction of a turn in fp64, since a position of 2^20 times a
// frequency of 1 leaves fp32 only four bits of the angle's fraction.
//
// A lane holds 16 channels of one head: one group of 16 channels holds 8 whole pairs in either
// layout (8 channels j.. and 8 channels j + rot/2.. in the half layout), so rotation needs no
// exchange between lanes and every load and store is 16 bytes. L = dh / 16 lanes (rounded up to a
// power of two) share a head and sum its squares by lane exchange; a wave walks the heads of its
// token 64 / L at a time, the next heads' loads in flight while these are worked on. The sines
// and cosines are computed once per token (one angle per thread) and shared through LDS.
// Bound by HBM: each input is read once and each output written once.
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace ttt {
namespace {

constexpr int NR_MAX_HALF = 128;  // rot / 2 at most

template <typename T>
struct Raw {
  static constexpr int n = sizeof(T) == 2 ? 2 : 4;
  uint4 v[n];
};

template <typename T>
__device__ __forceinline__ Raw<T> raw_load(const T* p, int e0, int e1) {
  Raw<T> r;
  if constexpr (sizeof(T) == 2) {
    r.v[0] = *reinterpret_cast<const uint4*>(p + e0);
    r.v[1] = *reinterpret_cast<const uint4*>(p + e1);
  } else {
    r.v[0] = *reinterpret_cast<const uint4*>(p + e0);
    r.v[1] = *reinterpret_cast<const uint4*>(p + e0 + 4);
    r.v[2] = *reinterpret_cast<const uint4*>(p + e1);
    r.v[3] = *reinterpret_cast<const uint4*>(p + e1 + 4);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void raw_store(T* p, int e0, int e1, const Raw<T>& r) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p + e0) = r.v[0];
    *reinterpret_cast<uint4*>(p + e1) = r.v[1];
  } else {
    *reinterpret_cast<uint4*>(p + e0) = r.v[0];
    *reinterpret_cast<uint4*>(p + e0 + 4) = r.v[1];
    *reinterpret_cast<uint4*>(p + e1) = r.v[2];
    *reinterpret_cast<uint4*>(p + e1 + 4) = r.v[3];
  }
}
template <typename T>
__device__ __forceinline__ void raw_unpack(const Raw<T>& r, float (&x)[16]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t w[4] = {r.v[q].x, r.v[q].y, r.v[q].z, r.v[q].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[8 * q + 2 * i] = __uint_as_float(w[i] << 16);
        x[8 * q + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[4 * q] = __uint_as_float(r.v[q].x);
      x[4 * q + 1] = __uint_as_float(r.v[q].y);
      x[4 * q + 2] = __uint_as_float(r.v[q].z);
      x[4 * q + 3] = __uint_as_float(r.v[q].w);
    }
  }
}
template <typename T>
__device__ __forceinline__ Raw<T> raw_pack(const float (&x)[16]) {
  Raw<T> r;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      r.v[q] = make_uint4(pack2bf(x[8 * q], x[8 * q + 1]), pack2bf(x[8 * q + 2], x[8 * q + 3]),
                          pack2bf(x[8 * q + 4], x[8 * q + 5]), pack2bf(x[8 * q + 6], x[8 * q + 7]));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      r.v[q] = make_uint4(__float_as_uint(x[4 * q]), __float_as_uint(x[4 * q + 1]),
                          __float_as_uint(x[4 * q + 2]), __float_as_uint(x[4 * q + 3]));
  }
  return r;
}

// lsh: log2 of the lanes per head; wpt: waves per token (1: four tokens per workgroup, 4: one)
template <typename T, bool INTER>
__global__ __launch_bounds__(256) void k_norm_rope(NormRopeArgs a, int lsh, int wpt) {
  __shared__ float2 cs[4][NR_MAX_HALF];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int tpb = 4 / wpt, half = a.rot >> 1;
  const long t0 = long(blockIdx.x) * tpb;
  const long t = t0 + wave / wpt;
  const bool on = t < a.N;  // wave-uniform

  const int L = 1 << lsh, c = lane & (L - 1), step = wpt << (6 - lsh);
  const bool live = c < (a.dh >> 4), rotates = c < (a.rot >> 4);
  const int e0 = (INTER || !rotates) ? 16 * c : 8 * c;
  const int e1 = (INTER || !rotates) ? e0 + 8 : half + e0;
  const int Hq = a.Hq, Hqk = a.Hq + a.Hkv, dh = a.dh;
  const int heads = Hqk + (a.Vc ? a.Hkv : 0);
  const T* q = static_cast<const T*>(a.Q) + t * a.qs;
  const T* k = static_cast<const T*>(a.K) + t * a.ks - long(Hq) * dh;
  const T* v = static_cast<const T*>(a.V) + t * a.vs - long(Hqk) * dh;
  auto src = [=](int i) { return (i < Hq ? q : i < Hqk ? k : v) + long(i) * dh; };
  int h = (wave % wpt) * (64 >> lsh) + (lane >> lsh);
  Raw<T> cur{};
  if (on && live && h < heads) cur = raw_load(src(h), e0, e1);
  const int slot = (on && a.slots) ? a.slots[t] : -1;

  for (int i = tid; i < tpb * half; i += 256) {
    const int tt = i / half, f = i - tt * half;
    if (t0 + tt < a.N) {
      const double turns = double(a.pos[t0 + tt]) * a.inv_freq[f] * 0.15915494309189533577;
      float s, co;
      sincospif(2.f * float(turns - rint(turns)), &s, &co);
      cs[tt][f] = make_float2(co * a.rope_scale, s * a.rope_scale);
    }
  }
  __syncthreads();
  if (!on) return;
  float2 turn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) turn[i] = rotates ? cs[wave / wpt][8 * c + i] : make_float2(1.f, 0.f);
  const float *qwp = a.qw, *kwp = a.kw;
  const bool qn = qwp != nullptr, kn = kwp != nullptr;
  float qw[16], kw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int e = i < 8 ? e0 + i : e1 + i - 8;
    qw[i] = qn && live ? qwp[e] : 1.f;
    kw[i] = kn && live ? kwp[e] : 1.f;
  }
  const float inv_dh = 1.f / float(a.dh);
  const bool cached = a.slots && slot >= 0 && slot < a.n_slots;
  T* qo = static_cast<T*>(a.Qo) + t * a.qos;
  T* ko = static_cast<T*>(a.Ko) + t * a.kos;
  T* kc = static_cast<T*>(a.Kc) + long(slot) * a.Hkv * a.dh;
  T* vc = static_cast<T*>(a.Vc) + long(slot) * a.Hkv * a.dh;
  // every lane of a wave makes the same number of rounds: the lanes of a head exchange sums
  const int rounds = (heads - (wave % wpt) * (64 >> lsh) + step - 1) / step;
  for (int r = 0; r < rounds; ++r, h += step) {
    const bool here = live && h < heads;
    Raw<T> next{};
    if (live && h + step < heads) next = raw_load(src(h + step), e0, e1);
    float x[16];
    raw_unpack<T>(cur, x);
    const bool isq = h < Hq;
    if (isq ? qn : kn) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
      for (int d = 1; d < L; d *= 2) ss += __shfl_xor(ss, d);
      const float rs = rsqrtf(ss * inv_dh + a.eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = x[i] * rs * (isq ? qw[i] : kw[i]);
    }
    if (rotates) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + 8;
        const float xa = x[ia], xb = x[ib];
        x[ia] = xa * turn[i].x - xb * turn[i].y;
        x[ib] = xa * turn[i].y + xb * turn[i].x;
      }
    }
    const Raw<T> out = raw_pack<T>(x);
    if (here) {
      if (isq) {
        raw_store(qo + long(h) * dh, e0, e1, out);
      } else if (h < Hqk) {
        const long o = long(h - Hq) * dh;
        if (a.Ko) raw_store(ko + o, e0, e1, out);
        if (cached) raw_store(kc + o, e0, e1, out);
      } else if (cached) {
        raw_store(vc + long(h - Hqk) * dh, e0, e1, cur);
      }
    }
    cur = next;
  }
}

}  // namespace

hipError_t norm_rope(const NormRopeArgs& a) {
  int lsh = 0;
  while ((16 << lsh) < a.dh) ++lsh;
  // Four waves on a token while that still leaves the chip short of waves (N tokens on 1024
  // SIMDs); one wave per token past that, so that the angles of four tokens are one per thread.
  const int wpt = a.N <= 2048 ? 4 : 1, tpb = 4 / wpt;
  const dim3 grid(unsigned((a.N + tpb - 1) / tpb)), block(256);
  if (a.bf16 && a.interleaved)
    hipLaunchKernelGGL((k_norm_rope<uint16_t, true>), grid, block, 0, a.stream, a, lsh, wpt);
  else if (a.bf16)
    hipLaunchKernelGGL((k_norm_rope<uint16_t, false>), grid, block, 0, a.stream, a, lsh, wpt);
  else if (a.interleaved)
    hipLaunchKernelGGL((k_norm_rope<float, true>), grid, block, 0, a.stream, a, lsh, wpt);
  else
    hipLaunchKernelGGL((k_norm_rope<float, false>), grid, block, 0, a.stream, a, lsh, wpt);
  return hipGetLastError();
}

}  // namespace ttt
