// Per-head RMS norm and rotation of queries and keys in one pass, with the cache write.
//
// For token t and head x [dh] of Q or K (norm only where a weight w is given):
//     y = x * rsqrt(mean(x^2) + eps) * w
//     (a, b) -> rope_scale * (a cos - b sin, a sin + b cos)   at angle pos[t] * inv_freq[j]
// for the rot / 2 pairs of the head's first `rot` channels: (j, j + rot/2) in the half layout,
// (2j, 2j + 1) in the interleaved one. Channels past rot keep y. Everything is fp32 and rounded
// once; the angle is reduced to a fraction of a turn in fp64, since a position of 2^20 times a
// frequency of 1 leaves fp32 only four bits of the angle's fraction. Its sine and cosine are taken in
// fp64 too for fp32 results; for bf16 ones, whose half step is 2^15 times as large, in fp32.
//
// A lane holds 16 channels of one head: one group of 16 channels holds 8 whole pairs in either
// layout (8 channels j.. and 8 channels j + rot/2.. in the half layout), so rotation needs no
// exchange between lanes and every load and store is 16 bytes. L = dh / 16 lanes (rounded up to a
// power of two) share a head and sum its squares by lane exchange; a wave walks the heads of its
// token 64 / L at a time, the next heads' loads in flight while these are worked on. The sines
// and cosines are computed once per token (one angle per thread) and shared through LDS.
// Bound by HBM: each input is read once and each output written once. 32768 tokens of 32/8 heads of 128
// bf16 with the cache write, 872 MB: 166 us, 5.25 TB/s (a copy of 2 GiB: 4.9); 1023 tokens of 16/16 heads
// of 64 in fp32, 17 MB: 6.4 us; 1 token 3.9 us, of which an empty launch is 2.
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

// A 16-byte read from global memory (head_at's pointer does not tell the compiler which memory).
__device__ __forceinline__ uint4 ld16(const void* p) {
  typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
  const u32x4_t v = *(const __attribute__((address_space(1))) u32x4_t*)reinterpret_cast<uintptr_t>(p);
  return make_uint4(v.x, v.y, v.z, v.w);
}
template <typename T>
__device__ __forceinline__ Raw<T> raw_load(const T* p, int e0, int e1) {
  Raw<T> r;
  if constexpr (sizeof(T) == 2) {
    r.v[0] = ld16(p + e0);
    r.v[1] = ld16(p + e1);
  } else {
    r.v[0] = ld16(p + e0);
    r.v[1] = ld16(p + e0 + 4);
    r.v[2] = ld16(p + e1);
    r.v[3] = ld16(p + e1 + 4);
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

// Where head h of a token lies: queries, then keys, then values. Selected by value, no array or
// closure of pointers: the compiler would put one into LDS and read the workgroup's size from the
// dispatch packet, which lies in host memory (15 us for the last of the chip's XCDs).
template <typename T>
__device__ __forceinline__ const T* head_at(const T* q, const T* k, const T* v, int h, int Hq, int Hqk,
                                            int dh) {
  const uintptr_t p = h < Hq ? uintptr_t(q) : h < Hqk ? uintptr_t(k) : uintptr_t(v);
  const int i = h < Hq ? h : h < Hqk ? h - Hq : h - Hqk;
  return reinterpret_cast<const T*>(p) + long(i) * dh;
}

// A lane's 16 weights of the norm.
struct Weights {
  float4 v[4];
  __device__ __forceinline__ void load(const float* p, int e0, int e1) {
    if (!p) return;  // no norm: not read
    v[0] = *reinterpret_cast<const float4*>(p + e0);
    v[1] = *reinterpret_cast<const float4*>(p + e0 + 4);
    v[2] = *reinterpret_cast<const float4*>(p + e1);
    v[3] = *reinterpret_cast<const float4*>(p + e1 + 4);
  }
  __device__ __forceinline__ float at(int i) const {
    const float4& q = v[i >> 2];
    return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
  }
};

// lsh: log2 of the lanes per head; wsh: log2 of the waves per token (a workgroup of 4 waves takes
// 4 >> wsh tokens)
template <typename T, bool INTER>
__global__ __launch_bounds__(256) void k_norm_rope(NormRopeArgs a, int lsh, int wsh) {
  __shared__ float2 cs[4][NR_MAX_HALF];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int tpb = 4 >> wsh, half = a.rot >> 1;
  const long t0 = long(blockIdx.x) * tpb;
  const long t = t0 + (wave >> wsh);
  const bool on = t < a.N;  // wave-uniform

  const int L = 1 << lsh, c = lane & (L - 1), hpw = 64 >> lsh, step = hpw << wsh;
  const bool live = c < (a.dh >> 4), rotates = c < (a.rot >> 4);
  const int e0 = (INTER || !rotates) ? 16 * c : 8 * c;
  const int e1 = (INTER || !rotates) ? e0 + 8 : half + e0;
  const int Hq = a.Hq, Hqk = a.Hq + a.Hkv, dh = a.dh;
  const int heads = Hqk + (a.Vc ? a.Hkv : 0);
  const T* q = static_cast<const T*>(a.Q) + t * a.qs;
  const T* k = static_cast<const T*>(a.K) + t * a.ks;
  const T* v = static_cast<const T*>(a.V) + t * a.vs;
  const float *qwp = a.qw, *kwp = a.kw;
  const bool qn = qwp != nullptr, kn = kwp != nullptr;
  const int h0 = (wave & ((1 << wsh) - 1)) * hpw;
  int h = h0 + (lane >> lsh);

  // everything that comes from memory is asked for before the angles are worked out
  Raw<T> cur{};
  if (on && live && h < heads) cur = raw_load(head_at(q, k, v, h, Hq, Hqk, dh), e0, e1);
  const int slot = (on && a.slots) ? a.slots[t] : -1;
  bool isq = h < Hq;
  Weights w;
  if (live) w.load(isq ? qwp : kwp, e0, e1);

  for (int i = tid; i < tpb * half; i += 256) {
    const int tt = i / half, f = i - tt * half;
    if (t0 + tt < a.N) {
      const double turns = double(a.pos[t0 + tt]) * a.inv_freq[f] * 0.15915494309189533577;
      if constexpr (sizeof(T) == 4) {  // fp32 results show what sines in fp32 lose (1 token: 0.1 us more)
        double s, co;
        sincospi(2. * (turns - rint(turns)), &s, &co);
        cs[tt][f] = make_float2(float(co * a.rope_scale), float(s * a.rope_scale));
      } else {
        float s, co;
        sincospif(2.f * float(turns - rint(turns)), &s, &co);
        cs[tt][f] = make_float2(co * a.rope_scale, s * a.rope_scale);
      }
    }
  }
  __syncthreads();
  if (!on) return;
  float2 turn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) turn[i] = rotates ? cs[wave >> wsh][8 * c + i] : make_float2(1.f, 0.f);
  const float inv_dh = 1.f / float(dh);
  const bool cached = a.slots && slot >= 0 && slot < a.n_slots;
  T* qo = static_cast<T*>(a.Qo) + t * a.qos;
  T* ko = static_cast<T*>(a.Ko) + t * a.kos;
  T* kc = static_cast<T*>(a.Kc) + long(slot) * a.Hkv * dh;
  T* vc = static_cast<T*>(a.Vc) + long(slot) * a.Hkv * dh;
  // every lane of a wave makes the same number of rounds: the lanes of a head exchange sums
  for (int r = h0; r < heads; r += step, h += step) {
    const bool here = live && h < heads;
    Raw<T> next{};
    if (live && h + step < heads) next = raw_load(head_at(q, k, v, h + step, Hq, Hqk, dh), e0, e1);
    if (isq && h >= Hq) {  // the lane's heads have moved on to the keys
      isq = false;
      if (live) w.load(kwp, e0, e1);
    }
    float x[16];
    raw_unpack<T>(cur, x);
    if (isq ? qn : kn) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
      for (int d = 1; d < L; d *= 2) ss += __shfl_xor(ss, d);
      float eps = a.eps;
      // Squares that leave fp32 (values past 2^63, or all below 2^-40 where eps does not hide them): the head
      // is scaled by a power of two first. All lanes of a head decide alike.
      const bool large = !(ss < 0x1p126f), small = ss < 0x1p-80f && eps < 0x1p-80f;
      if (__builtin_expect(__any(large || small), 0)) {
        const float s = large ? 0x1p-72f : small ? 0x1p96f : 1.f;
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] *= s;
          ss = fmaf(x[i], x[i], ss);
        }
        for (int d = 1; d < L; d *= 2) ss += __shfl_xor(ss, d);
        eps = eps * s * s;
      }
      const float rs = rsqrtf(ss * inv_dh + eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = x[i] * rs * w.at(i);
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
  // Up to four waves on a token, as many as its heads fill, while all waves of the launch are on the chip at
  // once (4 on each of 1024 SIMDs): past that they only repeat each other's start. 4 / 2 / 1 waves a token
  // in a graph, 32/8 heads of 128 with the cache write: 1024 tokens 7.1 / 7.2 / 9.5 us, 1280 9.4 / 8.3 / 10.1,
  // 2048 12.3 / 10.3 / 11.6, 2560 14.6 / 13.4 / 13.3, 8192 35.2 / 33.9 / 35.0; fp32 1024 tokens 12.2 / 11.6 /
  // 12.1; 32/32 heads 1024 10.5 / 12.1 / 15.4, 2048 19.0 / 19.5 / 20.7; 8/8 of 256 without it 1024 5.3 / 5.8 /
  // 7.6, 2048 8.9 / 8.1 / 8.8, 4096 15.2 / 13.9 / 12.9. 2 / 1 of 16/4 heads of 64: 2048 5.1 / 5.7,
  // 2560 6.6 / 6.2.
  const int waves = (((a.Hq + a.Hkv + (a.Vc ? a.Hkv : 0)) << lsh) + 63) / 64;
  int wsh = waves < 2 ? 0 : waves < 4 ? 1 : 2;
  while (wsh > 0 && long(a.N) << wsh > 4096) --wsh;
  const int tpb = 4 >> wsh;
  const dim3 grid(unsigned((a.N + tpb - 1) / tpb)), block(256);
  if (a.bf16 && a.interleaved)
    hipLaunchKernelGGL((k_norm_rope<uint16_t, true>), grid, block, 0, a.stream, a, lsh, wsh);
  else if (a.bf16)
    hipLaunchKernelGGL((k_norm_rope<uint16_t, false>), grid, block, 0, a.stream, a, lsh, wsh);
  else if (a.interleaved)
    hipLaunchKernelGGL((k_norm_rope<float, true>), grid, block, 0, a.stream, a, lsh, wsh);
  else
    hipLaunchKernelGGL((k_norm_rope<float, false>), grid, block, 0, a.stream, a, lsh, wsh);
  return hipGetLastError();
}

}  // namespace ttt
