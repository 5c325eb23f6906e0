// Causal attention over packed sequences with grouped heads, bf16.
//
// Sequence s has queries [cu_q[s], cu_q[s+1]) and keys [cu_k[s], cu_k[s+1]) (lq and lk of them);
// its last query stands at its last key. Query i, head h, sees key j of head h / G (G = Hq / Hkv)
// when i + lk - lq - window < j <= i + lk - lq (no lower limit without a window):
//     o = sum_j softmax_j(scale q . k_j) v_j,   lse = log sum_j exp(scale q . k_j)
// and o = 0, lse = -inf where nothing is visible.
//
// The G query heads that share a key head are rows of one problem: row r of a sequence is query
// r / G, head r % G, so one pass over the keys serves them all and a tile's causal edge spans
// 1 / G as many queries. A workgroup of 4 waves owns BM = 128 * QT consecutive rows (32 * QT per
// wave, as the columns of S^T) and walks the visible keys in tiles of 64 with the running maximum
// and sum of a softmax in fp32.
#include "attn.hpp"
#include "launch.hpp"

namespace ttt {
namespace {

constexpr int AP_BN = 64;

struct PackedDev {
  const uint16_t *Q, *K, *V;
  long qs, ks, vs;
  uint16_t* O;
  long os;
  float* lse;
  const int *cu_q, *cu_k;
  int n_seq, Nq, Nk, Hq, Hkv, G;
  float scale;
  int window;
  int tiles, splits;
  float* part;  // splits > 1: [splits][Nq * Hq][dh] sums, then [splits][Nq * Hq] (m, l)
};

// Sequence that holds row tile `tile`: sequence s owns the ids [base(s), base(s + 1)) with
// base(s) = cu_q[s] * G / BM + s, at least as many as it has tiles. A 64-way search over the
// wave's lanes; -1 if no sequence starts at or below `tile`.
__device__ __forceinline__ long ap_base(const PackedDev& a, int s, int BM) {
  const int c = min(max(a.cu_q[s], 0), a.Nq);
  return long(c) * a.G / BM + s;
}
__device__ __forceinline__ int ap_find(const PackedDev& a, int tile, int BM, int lane) {
  int lo = 0, len = a.n_seq;
  while (true) {
    const int step = (len + 63) / 64;
    const int s = lo + lane * step;
    const bool below = lane * step < len && ap_base(a, s, BM) <= tile;
    const int n = __popcll(__ballot(below));
    if (n == 0) return -1;
    const int at = (n - 1) * step;
    if (step == 1) return lo + at;
    len = min(step, len - at);
    lo += at;
  }
}

template <int DH, int QT>
__global__ __launch_bounds__(256, QT == 1 ? 2 : 1) void k_attention_packed(PackedDev a) {
  constexpr int BM = 128 * QT, TILE = AP_BN * DH * 2, KS = DH / 16, DT = DH / 32;
  __shared__ __align__(1024) char sm[2][2][TILE];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int h = lane >> 5;
  const int kvh = blockIdx.x % a.Hkv;
  const int rest = blockIdx.x / a.Hkv;
  const int split = rest % a.splits;
  const int tile = a.tiles - 1 - rest / a.splits;

  const int seq = __builtin_amdgcn_readfirstlane(ap_find(a, tile, BM, lane));
  if (seq < 0) return;
  const int q0 = min(max(a.cu_q[seq], 0), a.Nq), q1 = min(max(a.cu_q[seq + 1], q0), a.Nq);
  const int k0 = min(max(a.cu_k[seq], 0), a.Nk), k1 = min(max(a.cu_k[seq + 1], k0), a.Nk);
  const int rows = (q1 - q0) * a.G, lk = k1 - k0, off = lk - (q1 - q0);
  const long row0l = (tile - (long(q0) * a.G / BM + seq)) * BM;
  if (row0l < 0 || row0l >= rows) return;
  const int row0 = int(row0l);

  // the lane's query column of each block: its row, its last and first visible keys
  int row[QT], hi[QT], lo[QT];
  uint4 qf[QT][KS];
#pragma unroll
  for (int b = 0; b < QT; ++b) {
    row[b] = row0 + (wave * QT + b) * 32 + (lane & 31);
    const int r = min(row[b], rows - 1), qi = r / a.G, g = r - qi * a.G;
    hi[b] = qi + off;
    lo[b] = a.window > 0 ? qi + off - a.window + 1 : 0;
    const uint16_t* p = a.Q + long(q0 + qi) * a.qs + (kvh * a.G + g) * DH + 8 * h;
#pragma unroll
    for (int s = 0; s < KS; ++s) qf[b][s] = *reinterpret_cast<const uint4*>(p + 16 * s);
  }
  // key tiles of the workgroup, and the wave's own limits
  const int qa = row0 / a.G, qb = (min(row0 + BM, rows) - 1) / a.G;
  const int kend = min(lk, qb + off + 1);
  const int kbeg = a.window > 0 ? max(0, qa + off - a.window + 1) : 0;
  int t0 = kbeg / AP_BN, t1 = kend > kbeg ? (kend + AP_BN - 1) / AP_BN : t0;
  if (a.splits > 1) {
    const int per = (t1 - t0 + a.splits - 1) / a.splits;
    t0 = min(t0 + split * per, t1);
    t1 = min(t0 + per, t1);
  }
  const int wr = row0 + wave * 32 * QT;
  const int wlo = min(wr, rows - 1), whi = min(wr + 32 * QT, rows) - 1;
  const bool wave_on = wr < rows;
  const int hi_min = wlo / a.G + off, hi_max = (whi < wlo ? wlo : whi) / a.G + off;
  const int lo_max = a.window > 0 ? hi_max - a.window + 1 : 0;
  const int lo_min = a.window > 0 ? hi_min - a.window + 1 : 0;

  using CK = TileCopy<DH, AP_BN, 4, false>;
  using CV = TileCopy<DH, AP_BN, 4, true>;
  const char* Kb = reinterpret_cast<const char*>(a.K + long(k0) * a.ks + kvh * DH);
  const char* Vb = reinterpret_cast<const char*>(a.V + long(k0) * a.vs + kvh * DH);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_u32(&sm[0][0][0]));
  auto issue = [&](int t, int buf) {
    const int first = t * AP_BN, last = lk - 1 - first;
    const char* kb = Kb + long(first) * a.ks * 2;
    const char* vb = Vb + long(first) * a.vs * 2;
    const uint32_t kd = lds0 + buf * 2 * TILE + wave * 1024, vd = kd + TILE;
#pragma unroll
    for (int i = 0; i < CK::N; ++i)
      dma16(uint32_t(min(CK::row(i, wave, lane), last)) * uint32_t(a.ks * 2) +
                CK::chunk(i, wave, lane), kb, kd + i * 4096);
#pragma unroll
    for (int i = 0; i < CV::N; ++i)
      dma16(uint32_t(min(CV::row(i, wave, lane), last)) * uint32_t(a.vs * 2) +
                CV::chunk(i, wave, lane), vb, vd + i * 4096);
  };

  const FragOff<DH> fo(lane);
  f32x16 o[DT][QT];
  float m[QT], l[QT];
#pragma unroll
  for (int b = 0; b < QT; ++b) {
    m[b] = -INFINITY;
    l[b] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][b][i] = 0.f;
  }
  const float c = a.scale * kLog2e;

  if (t0 < t1) issue(t0, 0);
  for (int t = t0; t < t1; ++t) {
    const int buf = (t - t0) & 1;
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (t + 1 < t1) issue(t + 1, buf ^ 1);
    const int kv0 = t * AP_BN;
    if (!wave_on || kv0 > hi_max || kv0 + AP_BN - 1 < lo_min) continue;
    const char* kt = &sm[buf][0][0];
    const char* vt = &sm[buf][1][0];
    f32x16 s[2][QT];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int b = 0; b < QT; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kb][b][i] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const uint4 kf = fo.key(kt, kb, ks);
#pragma unroll
        for (int b = 0; b < QT; ++b) s[kb][b] = mfma32x32x16(kf, qf[b][ks], s[kb][b]);
      }
    if (kv0 + AP_BN - 1 > hi_min || kv0 < lo_max) {
#pragma unroll
      for (int b = 0; b < QT; ++b)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = kv0 + 32 * kb + 8 * (i / 4) + 4 * h + (i & 3);
            if (j > hi[b] || j < lo[b]) s[kb][b][i] = -INFINITY;
          }
    }
    uint4 pf[QT][4];
#pragma unroll
    for (int b = 0; b < QT; ++b) {
      float mx = m[b];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[kb][b][i]);
      mx = max_halves(mx);
      const float base = mx == -INFINITY ? 0.f : mx * c;
      const float al = exp2_fast(fmaf(m[b], c, -base));
      float sum = 0.f;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        float p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          p[i] = exp2_fast(fmaf(s[kb][b][i], c, -base));
          sum += p[i];
        }
        pf[b][2 * kb] = make_uint4(pack2bf(p[0], p[1]), pack2bf(p[2], p[3]), pack2bf(p[4], p[5]),
                                   pack2bf(p[6], p[7]));
        pf[b][2 * kb + 1] = make_uint4(pack2bf(p[8], p[9]), pack2bf(p[10], p[11]),
                                       pack2bf(p[12], p[13]), pack2bf(p[14], p[15]));
      }
      l[b] = l[b] * al + sum;
      if (__any(mx != m[b])) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][b][i] *= al;
      }
      m[b] = mx;
    }
#pragma unroll
    for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const uint4 vf = fo.value(vt, s4, d);
#pragma unroll
        for (int b = 0; b < QT; ++b) o[d][b] = mfma32x32x16(vf, pf[b][s4], o[d][b]);
      }
  }

  if (!wave_on) return;
#pragma unroll
  for (int b = 0; b < QT; ++b) {
    const float lt = sum_halves(l[b]);
    if (row[b] >= rows) continue;
    const int qi = row[b] / a.G, hq = kvh * a.G + row[b] - qi * a.G;
    const long rr = long(q0 + qi) * a.Hq + hq;
    if (a.splits > 1) {
      const long n = long(a.Nq) * a.Hq;
      float* po = a.part + (long(split) * n + rr) * DH + 4 * h;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4*>(po + 32 * d + 2 * i) =
              make_float4(o[d][b][i], o[d][b][i + 1], o[d][b][i + 2], o[d][b][i + 3]);
      if (h == 0) {
        float* ml = a.part + long(a.splits) * n * DH + (long(split) * n + rr) * 2;
        *reinterpret_cast<float2*>(ml) = make_float2(m[b], lt);
      }
      continue;
    }
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
    uint16_t* po = a.O + long(q0 + qi) * a.os + hq * DH + 4 * h;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<uint2*>(po + 32 * d + 2 * i) =
            make_uint2(pack2bf(o[d][b][i] * inv, o[d][b][i + 1] * inv),
                       pack2bf(o[d][b][i + 2] * inv, o[d][b][i + 3] * inv));
    if (a.lse && h == 0) a.lse[rr] = lt == 0.f ? -INFINITY : m[b] * a.scale + __logf(lt);
  }
}

}  // namespace

size_t attention_packed_workspace(int, int, int, int, int, int) { return 0; }

hipError_t attention_packed(const PackedArgs& a) {
  PackedDev d{static_cast<const uint16_t*>(a.Q), static_cast<const uint16_t*>(a.K),
              static_cast<const uint16_t*>(a.V), a.qs, a.ks, a.vs, static_cast<uint16_t*>(a.O),
              a.os, a.lse, a.cu_q, a.cu_k, a.n_seq, a.Nq, a.Nk, a.Hq, a.Hkv, a.Hq / a.Hkv,
              a.scale, a.window, 0, 1, nullptr};
  const int BM = 256;
  d.tiles = int(long(a.Nq) * d.G / BM) + a.n_seq;
  const dim3 grid(unsigned(d.tiles) * a.Hkv);
  if (a.dh == 128)
    hipLaunchKernelGGL((k_attention_packed<128, 2>), grid, dim3(256), 0, a.stream, d);
  else
    hipLaunchKernelGGL((k_attention_packed<64, 2>), grid, dim3(256), 0, a.stream, d);
  return hipGetLastError();
}

}  // namespace ttt
