// The gated delta rule, one token per sequence: for sequence s and value head h, with the state S [dk, dv],
//     keep = exp(g),  u = beta (v - keep S^T k),  S' = keep S + k u^T,  o = scale S'^T q
// q and k divided by their norm where asked. Value head h reads key head h / (Hv / Hk). fp32 throughout, o
// rounded once.
//
// Bound by HBM: a head's state (64 KB at 128 x 128) is read once and written once. A workgroup takes some
// columns of one head's state into registers, all of its loads asked for at once; the sums over the rows for
// S^T k and S^T q are taken together, since o = scale (keep S^T q + (k . q) u), so the workgroup
// meets once. 2048 heads of 128 x 128 (64 sequences of 32): 54 us, 5.0 TB/s, as much as a copy reaches (4.95); 46 where
// the same pool is taken again and again, of which a part stays in the last cache. 32 heads: 3.7 us, of which an empty
// kernel takes 2.
#include "common.hpp"
#include "launch.hpp"

namespace ttt {
namespace {

template <int DK, int DVT>
__global__ __launch_bounds__(256) void k_delta_step(DeltaArgs a) {
  constexpr int LP = DVT / 4, RP = 256 / LP, IT = DK / RP;  // lanes to a row, rows at once, rows of a thread
  constexpr int PER = DK / 64;                              // channels of q and k to a lane
  __shared__ float qk_s[4][2][DK];
  __shared__ float4 sum_s[4][2][LP];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int tiles = a.dv / DVT;
  int id = blockIdx.x;
  const int tile = id % tiles;
  id /= tiles;
  const int h = id % a.Hv, s = id / a.Hv, hk = h / (a.Hv / a.Hk);
  const long slot = a.slots ? a.slots[s] : s;
  const bool kept = slot >= 0 && slot < a.n_slots;
  const int r0 = tid / LP, c = 4 * (tid % LP);
  const long at = ((kept ? slot : 0) * a.Hv + h) * long(DK) * a.dv + long(r0) * a.dv + tile * DVT + c;
  float4 st[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    st[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (kept && a.state_in) st[i] = *reinterpret_cast<const float4*>(a.state_in + at + long(i) * RP * a.dv);
  }
  const uint16_t* q = static_cast<const uint16_t*>(a.Q) + s * a.qs + hk * DK + PER * lane;
  const uint16_t* k = static_cast<const uint16_t*>(a.K) + s * a.ks + hk * DK + PER * lane;
  const uint2 vr = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.V) + s * a.vs + h * a.dv +
                                                   tile * DVT + c);
  const float keep = expf(a.g[long(s) * a.Hv + h]), beta = a.beta[long(s) * a.Hv + h];
  float x[PER], y[PER], qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    x[i] = bf2f(q[i]);
    y[i] = bf2f(k[i]);
    qq = fmaf(x[i], x[i], qq);
    kk = fmaf(y[i], y[i], kk);
    qk = fmaf(x[i], y[i], qk);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    qq += __shfl_xor(qq, d);
    kk += __shfl_xor(kk, d);
    qk += __shfl_xor(qk, d);
  }
  float rq = a.scale, rk = 1.f;
  if (a.norm) {
    rq *= rsqrtf(qq + a.eps);
    rk = rsqrtf(kk + a.eps);
  }
  qk *= rq * rk;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    qk_s[wave][0][PER * lane + i] = x[i] * rq;
    qk_s[wave][1][PER * lane + i] = y[i] * rk;
  }
  __builtin_amdgcn_wave_barrier();
  float4 p = make_float4(0.f, 0.f, 0.f, 0.f), o = p;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const float qr = qk_s[wave][0][r0 + i * RP], kr = qk_s[wave][1][r0 + i * RP];
    p.x = fmaf(kr, st[i].x, p.x);
    p.y = fmaf(kr, st[i].y, p.y);
    p.z = fmaf(kr, st[i].z, p.z);
    p.w = fmaf(kr, st[i].w, p.w);
    o.x = fmaf(qr, st[i].x, o.x);
    o.y = fmaf(qr, st[i].y, o.y);
    o.z = fmaf(qr, st[i].z, o.z);
    o.w = fmaf(qr, st[i].w, o.w);
  }
#pragma unroll
  for (int d = LP; d < 64; d *= 2) {
    p.x += __shfl_xor(p.x, d);
    p.y += __shfl_xor(p.y, d);
    p.z += __shfl_xor(p.z, d);
    p.w += __shfl_xor(p.w, d);
    o.x += __shfl_xor(o.x, d);
    o.y += __shfl_xor(o.y, d);
    o.z += __shfl_xor(o.z, d);
    o.w += __shfl_xor(o.w, d);
  }
  if (lane < LP) {
    sum_s[wave][0][lane] = p;
    sum_s[wave][1][lane] = o;
  }
  __syncthreads();
  p = sum_s[0][0][tid % LP];
  o = sum_s[0][1][tid % LP];
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    const float4 pw = sum_s[w][0][tid % LP], ow = sum_s[w][1][tid % LP];
    p = make_float4(p.x + pw.x, p.y + pw.y, p.z + pw.z, p.w + pw.w);
    o = make_float4(o.x + ow.x, o.y + ow.y, o.z + ow.z, o.w + ow.w);
  }
  const float4 u = make_float4(beta * (__uint_as_float(vr.x << 16) - keep * p.x),
                               beta * (__uint_as_float(vr.x & 0xFFFF0000u) - keep * p.y),
                               beta * (__uint_as_float(vr.y << 16) - keep * p.z),
                               beta * (__uint_as_float(vr.y & 0xFFFF0000u) - keep * p.w));
  if (kept && a.state_out) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const float kr = qk_s[wave][1][r0 + i * RP];
      *reinterpret_cast<float4*>(a.state_out + at + long(i) * RP * a.dv) =
          make_float4(fmaf(kr, u.x, keep * st[i].x), fmaf(kr, u.y, keep * st[i].y),
                      fmaf(kr, u.z, keep * st[i].z), fmaf(kr, u.w, keep * st[i].w));
    }
  }
  if (r0 == 0)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.O) + s * a.os + h * a.dv + tile * DVT + c) =
        make_uint2(pack2bf(fmaf(qk, u.x, keep * o.x), fmaf(qk, u.y, keep * o.y)),
                   pack2bf(fmaf(qk, u.z, keep * o.z), fmaf(qk, u.w, keep * o.w)));
}

template <int DK>
void launch(const DeltaArgs& a, int tile) {
  const dim3 grid(unsigned(long(a.n_seq) * a.Hv * (a.dv / tile))), block(256);
  if (tile == 32) hipLaunchKernelGGL((k_delta_step<DK, 32>), grid, block, 0, a.stream, a);
  else hipLaunchKernelGGL((k_delta_step<DK, 64>), grid, block, 0, a.stream, a);
}

}  // namespace

hipError_t delta_step(const DeltaArgs& a) {
  const long heads = long(a.n_seq) * a.Hv;
  // Columns of a workgroup: 32 while those are at most the card's 256 units, else 64. States of 128 x 128, tiles of 32
  // and of 64 columns: 8 heads 3.4 and 3.6 us, 64 heads 3.9 and 4.1, 128 heads 6.1 and 5.9, 1024 heads 28.8 and 28.5,
  // 4096 heads 104 and 98.6. (128 columns: 4.2, 5.1, 6.1, 30.2, 104.)
  const int tile = heads * a.dv <= 256 * 32 ? 32 : 64;
  a.dk == 128 ? launch<128>(a, tile) : launch<64>(a, tile);
  return hipGetLastError();
}

}  // namespace ttt
