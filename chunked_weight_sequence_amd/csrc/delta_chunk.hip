// The gated delta rule over packed sequences, 64 tokens at a time, bf16 inputs, fp32 state.
//
// Per value head, with a_t = exp(g_t):  u_t = beta_t (v_t - a_t S^T k_t),  S <- a_t S + k_t u_t^T,
// o_t = scale S^T q_t. Inside a chunk with G_i = g_1 + .. + g_i, and S the state before it:
//     u = T (V - diag(e^G) K S)          T = (1 + L)^-1 diag(beta),  L_ij = beta_i e^(G_i - G_j) k_i.k_j, i > j
//     O = scale (diag(e^G) Q S + A u)    A_ij = e^(G_i - G_j) q_i.k_j, i >= j
//     S <- e^(G_C) S + K^T diag(e^(G_C - G)) u
// so only S goes from chunk to chunk. q and k are divided by their norm by factors of the rows of these
// products (K and Q enter them as the bf16 they are).
//
// Two launches. k_delta_prepare, one workgroup per chunk and head: T and A, and the factors of the rows.
// k_delta_scan, one workgroup per sequence, head and some columns of the state: the recurrence over the
// chunks. A wave keeps 16 NB columns of S in accumulators from the first chunk to the last and needs
// nothing of the other waves, which only share the tiles in LDS: a product's result [rows, columns] has the lane
// layout of the next product's operand [contraction, columns] if the 32 rows of a contraction are taken in the
// order 16 (e / 4) + 4 (l / 16) + e % 4, e = 0..7, in both operands.
//
// Precision: what is not bf16 enters a product as a sum of bf16 planes, S as two, T, V - e^G K S and u as three
// (of the nine products of planes of T and V - .., the six above 2^-24). One plane less for any of the three
// leaves 3 .. 6e-6 of the state's size after 2048 tokens, this 3 .. 7e-7 (an fp32 computation 2e-7); S
// itself is never rounded to fewer bits, and its error in S^T k enters a chunk's u only. O, which is rounded to
// bf16, takes one plane of S and u, and A in bf16.
#include <type_traits>

#include "common.hpp"
#include "dma.hpp"
#include "launch.hpp"

namespace ttt {
namespace {

#define DL_INLINE __attribute__((always_inline))

constexpr int DL_C = 64;             // tokens of a chunk
constexpr int DL_FRAGS = 6;          // 16 x 32 blocks of a lower triangle: (row block, contraction step) with
                                     // step <= row block / 2, numbered row block + (row block > 1) * (row block - 2) + step
constexpr int DL_TOK = 4 * DL_FRAGS * 1024;  // byte offset of the rows' factors behind 3 planes of T, then A
constexpr int DL_UNIT = DL_TOK + 1024;       // bytes of a chunk and head in the workspace
// the rows' factors: e^G and the norm of k [64], e^(G_C - G) and the norm of k [64], scale e^G and the norm of
// q [64], e^(G_C)
constexpr int DL_FROM = 0, DL_LEFT = 64, DL_OUT = 128, DL_WHOLE = 192;

__device__ __forceinline__ constexpr int dl_frag(int rb, int ks) { return rb + (rb > 1 ? rb - 2 : 0) + ks; }

struct DeltaChunk {
  int q0, n;       // first token and tokens of the sequence
  int base, seq;   // its first chunk's number
};
__device__ __forceinline__ DeltaChunk dl_sequence(const DeltaPackedArgs& a, int s) {
  DeltaChunk c;
  c.seq = s;
  c.q0 = min(max(a.cu[s], 0), a.N);
  c.n = max(min(max(a.cu[s + 1], 0), a.N) - c.q0, 0);
  c.base = c.q0 / DL_C + s;
  return c;
}
// The sequence that owns chunk number `id`: s has the numbers from cu[s] / 64 + s on, at least as many as it has
// chunks. By all lanes of a wave.
__device__ __forceinline__ int dl_find(const DeltaPackedArgs& a, int id, int lane) {
  int lo = 0, len = a.d.n_seq;
  while (true) {
    const int step = (len + 63) / 64, s = lo + lane * step;
    const bool in = lane * step < len;
    const bool le = in && min(max(a.cu[in ? s : lo], 0), a.N) / DL_C + s <= id;
    const int n = max(__popcll(__ballot(le)), 1);
    lo += (n - 1) * step;
    if (step == 1) return __builtin_amdgcn_readfirstlane(lo);
    len = min(step, len - (n - 1) * step);
  }
}

// Tiles of rows of W bf16 in LDS, in units of 32 bytes (16 channels); unit u of row r at slot u ^ turn(r), so that
// 16 rows' reads of one unit, whole rows' worth of lanes, fall on all banks.
template <int W>
__device__ __forceinline__ int dl_turn(int r) {
  return W >= 128 ? r & 7 : W == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
}
template <int W>
__device__ __forceinline__ int dl_at(int r, int unit) { return r * W * 2 + ((unit ^ dl_turn<W>(r)) << 5); }

// The 1 KB number i of a 64-row tile: rows of a sequence from `src` on, `left` of which exist (the last one stands
// for those behind it), by one wave.
template <int W>
__device__ __forceinline__ void dl_copy_rows(int i, const void* src, long stride, int left, uint32_t lds, int lane) {
  constexpr int CH = W / 8, RPI = 64 / CH;  // 16-byte pieces of a row, rows of a copy
  const int r = i * RPI + lane / CH, p = lane % CH;
  const uint32_t off = uint32_t(min(r, left - 1)) * uint32_t(stride * 2) + ((p ^ (dl_turn<W>(r) << 1)) << 4);
  dma16(off, static_cast<const char*>(src), __builtin_amdgcn_readfirstlane(lds + i * 1024));
}

typedef short dl_s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) dl_s16x4 dl_lds_s16x4;
// 4 rows' values of a lane's column out of a row-major tile: 16 lanes read 4 rows x 16 channels.
__device__ __forceinline__ uint2 dl_transposed(const char* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((dl_lds_s16x4*)p));
}
// The 4 rows 4 (l / 16) .. of row block rb, column 16 unit + l % 16.
template <int W>
__device__ __forceinline__ uint2 dl_column(const char* tile, int rb, int unit, int lane) {
  const int r = 16 * rb + 4 * (lane >> 4) + ((lane & 15) >> 2);
  return dl_transposed(tile + dl_at<W>(r, unit) + 8 * (lane & 3));
}
// Row 16 rb + l % 16 with the channels of contraction step ks in the order of the products' results.
template <int W>
__device__ __forceinline__ uint4 dl_row(const char* tile, int rb, int ks, int lane) {
  const int r = 16 * rb + (lane & 15), g = lane >> 4;
  const uint2 lo = *reinterpret_cast<const uint2*>(tile + dl_at<W>(r, 2 * ks) + 8 * g);
  const uint2 hi = *reinterpret_cast<const uint2*>(tile + dl_at<W>(r, 2 * ks + 1) + 8 * g);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// Rounds 8 values to a plane of bf16 and leaves what the rounding lost.
__device__ __forceinline__ uint4 dl_plane(float (&x)[8], bool last = false) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = pack2bf(x[2 * i], x[2 * i + 1]);
    if (!last) {
      x[2 * i] -= __uint_as_float(w[i] << 16);
      x[2 * i + 1] -= __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Operands of a contraction step out of its two row blocks of a product's result, in P planes.
template <int P>
__device__ __forceinline__ void dl_planes(const f32x4& a, const f32x4& b, uint4 (&out)[P]) {
  float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
  for (int p = 0; p < P; ++p) out[p] = dl_plane(x, p == P - 1);
}

__device__ __forceinline__ f32x4 dl_mma_f32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// --------------------------------------------------------------------------------------------
template <int DK>
__global__ __launch_bounds__(256) void k_delta_prepare(DeltaPackedArgs a) {
  constexpr int TILE = DL_C * DK * 2, LW = 68;  // row of L and T in floats
  __shared__ __align__(1024) char kq[2 * TILE > DL_C * LW * 4 ? 2 * TILE : DL_C * LW * 4];  // K, Q; then T
  __shared__ __align__(16) float ls[DL_C][LW];
  __shared__ double gs[DL_C];
  __shared__ float bs[DL_C], rk_s[DL_C], rq_s[DL_C];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int h = blockIdx.x % a.d.Hv, id = blockIdx.x / a.d.Hv;
  const DeltaChunk sq = dl_sequence(a, dl_find(a, id, lane));
  const int t0 = (id - sq.base) * DL_C, left = min(sq.n - t0, DL_C);
  if (id < sq.base || left <= 0) return;
  const int hk = h / (a.d.Hv / a.d.Hk);
  const long tok = sq.q0 + t0;
  char* const ks = kq;
  char* const qs = kq + TILE;
  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_u32(kq));
#pragma unroll
  for (int i = 0; i < TILE / 4096; ++i) {
    dl_copy_rows<DK>(4 * i + wave, static_cast<const uint16_t*>(a.d.K) + tok * a.d.ks + hk * DK, a.d.ks, left, lds, lane);
    dl_copy_rows<DK>(4 * i + wave, static_cast<const uint16_t*>(a.d.Q) + tok * a.d.qs + hk * DK, a.d.qs, left, lds + TILE, lane);
  }
  if (wave == 0) {
    // sums of the gates in fp64: their differences count, also behind a gate that forgets everything (-inf:
    // e^-1000 is 0 as well, and sums of it stay finite)
    const long at = (tok + min(lane, left - 1)) * a.d.Hv + h;
    float g = a.d.g[at];
    g = lane < left ? (g < -1000.f ? -1000.f : g) : 0.f;
    double G = g;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double up = __shfl_up(G, d);
      if (lane >= d) G += up;
    }
    gs[lane] = G;
    bs[lane] = lane < left ? a.d.beta[at] : 0.f;
  }
  wait_vm<0>();
  __syncthreads();
  {
    // the norms: four threads to a row
    const int r = tid >> 2, part = tid & 3;
    float kk = 0.f, qq = 0.f;
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) {  // 8 channels: any order, each once
      const uint4 kv = *reinterpret_cast<const uint4*>(ks + r * DK * 2 + 16 * (4 * i + part));
      const uint4 qv = *reinterpret_cast<const uint4*>(qs + r * DK * 2 + 16 * (4 * i + part));
      const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w}, qw[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float k0 = __uint_as_float(kw[e] << 16), k1 = __uint_as_float(kw[e] & 0xFFFF0000u);
        const float q0 = __uint_as_float(qw[e] << 16), q1 = __uint_as_float(qw[e] & 0xFFFF0000u);
        kk = fmaf(k0, k0, fmaf(k1, k1, kk));
        qq = fmaf(q0, q0, fmaf(q1, q1, qq));
      }
    }
    kk += __shfl_xor(kk, 1);
    qq += __shfl_xor(qq, 1);
    kk += __shfl_xor(kk, 2);
    qq += __shfl_xor(qq, 2);
    if (part == 0) {
      rk_s[r] = a.d.norm ? rsqrtf(kk + a.d.eps) : 1.f;
      rq_s[r] = a.d.scale * (a.d.norm ? rsqrtf(qq + a.d.eps) : 1.f);
    }
  }
  __syncthreads();

  // Row block `wave` of L and A, as blocks [j, i] of products K K^T and K Q^T: lane l has row i = l % 16 of the
  // block and its columns j = 4 (l / 16) ..
  char* const unit = static_cast<char*>(a.ws) + (size_t(id) * a.d.Hv + h) * DL_UNIT;
  const int g4 = 4 * (lane >> 4), i0 = 16 * wave + (lane & 15);
  {
    const double gi = gs[i0];
    const float bi = bs[i0] * rk_s[i0], qi = i0 < left ? rq_s[i0] : 0.f;
    uint4 kf[DK / 32], qf[DK / 32];
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      kf[s] = dl_row<DK>(ks, wave, s, lane);
      qf[s] = dl_row<DK>(qs, wave, s, lane);
    }
    uint2 aw[4];
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      aw[jb] = make_uint2(0, 0);
      if (jb > wave) continue;
      f32x4 kk = {0.f, 0.f, 0.f, 0.f}, kq2 = kk;
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) {
        const uint4 f = dl_row<DK>(ks, jb, s, lane);
        kk = mfma16x16x32(f, kf[s], kk);
        kq2 = mfma16x16x32(f, qf[s], kq2);
      }
      float lv[4], av[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * jb + g4 + r;
        const float decay = expf(float(gi - gs[j])) * rk_s[j];
        lv[r] = j < i0 && i0 < left ? bi * decay * kk[r] : 0.f;
        av[r] = j <= i0 && i0 < left ? qi * decay * kq2[r] : 0.f;
      }
      *reinterpret_cast<float4*>(&ls[i0][16 * jb + g4]) = make_float4(lv[0], lv[1], lv[2], lv[3]);
      aw[jb] = make_uint2(pack2bf(av[0], av[1]), pack2bf(av[2], av[3]));
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s <= wave / 2)
        *reinterpret_cast<uint4*>(unit + (18 + dl_frag(wave, s)) * 1024 + 16 * lane) =
            make_uint4(aw[2 * s].x, aw[2 * s].y, aw[2 * s + 1].x, aw[2 * s + 1].y);
  }
  if (wave == 3) {
    float* f = reinterpret_cast<float*>(unit + DL_TOK);
    const double G = gs[lane], all = gs[DL_C - 1];
    f[DL_FROM + lane] = expf(float(G)) * rk_s[lane];
    f[DL_LEFT + lane] = expf(float(all - G)) * rk_s[lane];
    f[DL_OUT + lane] = expf(float(G)) * rq_s[lane];
    f[DL_WHOLE + lane] = expf(float(all));
  }
  __syncthreads();  // L is there; K and Q have been read

  // The inverse of 1 + L: the four diagonal blocks by forward substitution, a column to a lane, then block
  // column `wave` from the top: T_ij = -T_ii sum_k L_ik T_kj.
  float(*const ts)[LW] = reinterpret_cast<float(*)[LW]>(kq);
  {
    const int c = lane & 15, b = wave;  // lanes 16 .. 63 repeat the first 16
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = i == c ? 1.f : 0.f;
#pragma unroll
      for (int k = 0; k < i; ++k) x = fmaf(-ls[16 * b + i][16 * b + k], t[k], x);
      t[i] = x;
    }
    if (lane < 16)
#pragma unroll
      for (int i = 0; i < 16; ++i) ts[16 * b + i][16 * b + c] = t[i];
  }
  __syncthreads();
  {
    f32x4 col[4];  // T_kj, j = wave, as operands: column l % 16, rows 4 (l / 16) ..
#pragma unroll
    for (int r = 0; r < 4; ++r) col[0][r] = ts[16 * wave + g4 + r][16 * wave + (lane & 15)];
#pragma unroll
    for (int n = 1; n < 4; ++n) {
      const int ib = wave + n;
      if (ib > 3) break;
      f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < n; ++k) {
        const float4 l = *reinterpret_cast<const float4*>(&ls[16 * ib + (lane & 15)][16 * (wave + k) + g4]);
        y = dl_mma_f32(l.x, col[k][0], y);
        y = dl_mma_f32(l.y, col[k][1], y);
        y = dl_mma_f32(l.z, col[k][2], y);
        y = dl_mma_f32(l.w, col[k][3], y);
      }
      const float4 d = *reinterpret_cast<const float4*>(&ts[16 * ib + (lane & 15)][16 * ib + g4]);
      f32x4 z = {0.f, 0.f, 0.f, 0.f};
      z = dl_mma_f32(d.x, -y[0], z);
      z = dl_mma_f32(d.y, -y[1], z);
      z = dl_mma_f32(d.z, -y[2], z);
      z = dl_mma_f32(d.w, -y[3], z);
      col[n] = z;
#pragma unroll
      for (int r = 0; r < 4; ++r) ts[16 * ib + g4 + r][16 * wave + (lane & 15)] = z[r];
    }
  }
  __syncthreads();
  // row block `wave` of T, its columns times beta, in three planes
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s > wave / 2) break;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int jb = 2 * s + e / 4, j = 16 * jb + g4 + e % 4;
      x[e] = jb <= wave ? ts[i0][j] * bs[j] : 0.f;
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<uint4*>(unit + (6 * p + dl_frag(wave, s)) * 1024 + 16 * lane) = dl_plane(x, p == 2);
  }
}

// --------------------------------------------------------------------------------------------
// W waves of 16 NB columns each.
template <int DK, int W, int NB>
__global__ __launch_bounds__(64 * W) void k_delta_scan(DeltaPackedArgs a) {
  constexpr int COLS = 16 * NB * W, KT = DL_C * DK * 2, VT = DL_C * COLS * 2;
  constexpr int DB = DK / 16, KS = DK / 32;  // row blocks of the state, contraction steps over them
  // K, Q, the workspace's unit, V
  constexpr int AT_Q = KT, AT_U = 2 * KT, AT_V = AT_U + DL_UNIT, STAGE = AT_V + VT;
  __shared__ __align__(1024) char sm[2][STAGE];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  // the tiles of a head on one XCD: they read the same K, Q, T and A
  const int heads = a.d.n_seq * a.d.Hv, hd = blockIdx.x % heads, tile = blockIdx.x / heads;
  const int h = hd % a.d.Hv, s = hd / a.d.Hv, hk = h / (a.d.Hv / a.d.Hk);
  const DeltaChunk sq = dl_sequence(a, s);
  const long slot = a.d.slots ? a.d.slots[s] : s;
  const bool kept = slot >= 0 && slot < a.d.n_slots;
  const int col = tile * COLS + wave * 16 * NB, g4 = 4 * (lane >> 4), c16 = lane & 15;
  const int chunks = (sq.n + DL_C - 1) / DL_C;
  const long state = ((kept ? slot : 0) * a.d.Hv + h) * long(DK) * a.d.dv + col + c16;

  f32x4 S[DB][NB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        S[d][b][r] = kept && a.d.state_in ? a.d.state_in[state + long(16 * d + g4 + r) * a.d.dv + 16 * b] : 0.f;

  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_u32(sm));
  const uint16_t* kp = static_cast<const uint16_t*>(a.d.K) + long(sq.q0) * a.d.ks + hk * DK;
  const uint16_t* qp = static_cast<const uint16_t*>(a.d.Q) + long(sq.q0) * a.d.qs + hk * DK;
  const uint16_t* vp = static_cast<const uint16_t*>(a.d.V) + long(sq.q0) * a.d.vs + h * a.d.dv + tile * COLS;
  const char* up = static_cast<const char*>(a.ws) + (size_t(sq.base) * a.d.Hv + h) * DL_UNIT;
  const auto copy = [&](int c) DL_INLINE {  // of chunk c into its stage
    const uint32_t to = lds + (c & 1) * STAGE;
    const int left = sq.n - c * DL_C;
    const char* u = up + size_t(c) * a.d.Hv * DL_UNIT;
#pragma unroll
    for (int i = 0; i < KT / 1024 / W; ++i) {
      dl_copy_rows<DK>(W * i + wave, kp + long(c) * DL_C * a.d.ks, a.d.ks, left, to, lane);
      dl_copy_rows<DK>(W * i + wave, qp + long(c) * DL_C * a.d.qs, a.d.qs, left, to + AT_Q, lane);
    }
#pragma unroll
    for (int i = 0; i < (DL_UNIT / 1024 + W - 1) / W; ++i)
      if (W * i + wave < DL_UNIT / 1024)
        dma16(uint32_t((W * i + wave) * 1024 + lane * 16), u,
              __builtin_amdgcn_readfirstlane(to + AT_U + (W * i + wave) * 1024));
#pragma unroll
    for (int i = 0; i < VT / 1024 / W; ++i)
      dl_copy_rows<COLS>(W * i + wave, vp + long(c) * DL_C * a.d.vs, a.d.vs, left, to + AT_V, lane);
  };
  if (chunks > 0) copy(0);
  for (int c = 0; c < chunks; ++c) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (c + 1 < chunks) copy(c + 1);
    const char* const kt = sm[c & 1];
    const char* const qt = kt + AT_Q;
    const char* const ut = kt + AT_U;
    const char* const vt = kt + AT_V;
    const float* const f = reinterpret_cast<const float*>(ut + DL_TOK);
    const int left = sq.n - c * DL_C;
    const auto T = [&](int p, int rb, int ks) DL_INLINE {
      return *reinterpret_cast<const uint4*>(ut + (6 * p + dl_frag(rb, ks)) * 1024 + 16 * lane);
    };

    // S in two planes; P = K S
    uint4 sp[KS][NB][2];
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int b = 0; b < NB; ++b) dl_planes<2>(S[2 * k][b], S[2 * k + 1][b], sp[k][b]);
    f32x4 x[4][NB];
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
#pragma unroll
      for (int b = 0; b < NB; ++b) x[rb][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint4 kf = dl_row<DK>(kt, rb, k, lane);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int p = 0; p < 2; ++p) x[rb][b] = mfma16x16x32(kf, sp[k][b][p], x[rb][b]);
      }
    }
    // V - e^G P
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
      const float4 from = *reinterpret_cast<const float4*>(f + DL_FROM + 16 * rb + g4);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint2 v = dl_column<COLS>(vt, rb, wave * NB + b, lane);
        x[rb][b] = f32x4{fmaf(-from.x, x[rb][b][0], __uint_as_float(v.x << 16)),
                         fmaf(-from.y, x[rb][b][1], __uint_as_float(v.x & 0xFFFF0000u)),
                         fmaf(-from.z, x[rb][b][2], __uint_as_float(v.y << 16)),
                         fmaf(-from.w, x[rb][b][3], __uint_as_float(v.y & 0xFFFF0000u))};
      }
    }
    uint4 xp[2][NB][3];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int b = 0; b < NB; ++b) dl_planes<3>(x[2 * k][b], x[2 * k + 1][b], xp[k][b]);
    // u = T (..): the planes' products from the smallest on
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
#pragma unroll
      for (int b = 0; b < NB; ++b) x[rb][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k <= rb / 2; ++k) {
        const uint4 t[3] = {T(0, rb, k), T(1, rb, k), T(2, rb, k)};
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          x[rb][b] = mfma16x16x32(t[2], xp[k][b][0], x[rb][b]);
          x[rb][b] = mfma16x16x32(t[1], xp[k][b][1], x[rb][b]);
          x[rb][b] = mfma16x16x32(t[0], xp[k][b][2], x[rb][b]);
          x[rb][b] = mfma16x16x32(t[1], xp[k][b][0], x[rb][b]);
          x[rb][b] = mfma16x16x32(t[0], xp[k][b][1], x[rb][b]);
          x[rb][b] = mfma16x16x32(t[0], xp[k][b][0], x[rb][b]);
        }
      }
    }
    // one plane of u for O, and what the state takes in three
    uint4 uh[2][NB];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint4 one[1];
        dl_planes<1>(x[2 * k][b], x[2 * k + 1][b], one);
        uh[k][b] = one[0];
      }
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
      const float4 keep = *reinterpret_cast<const float4*>(f + DL_LEFT + 16 * rb + g4);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        x[rb][b] = f32x4{x[rb][b][0] * keep.x, x[rb][b][1] * keep.y, x[rb][b][2] * keep.z, x[rb][b][3] * keep.w};
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int b = 0; b < NB; ++b) dl_planes<3>(x[2 * k][b], x[2 * k + 1][b], xp[k][b]);
    const float whole = f[DL_WHOLE];
#pragma unroll
    for (int d = 0; d < DB; ++d) {
#pragma unroll
      for (int b = 0; b < NB; ++b) S[d][b] *= whole;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint2 lo = dl_column<DK>(kt, 2 * k, d, lane), hi = dl_column<DK>(kt, 2 * k + 1, d, lane);
        const uint4 kf = make_uint4(lo.x, lo.y, hi.x, hi.y);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int p = 2; p >= 0; --p) S[d][b] = mfma16x16x32(kf, xp[k][b][p], S[d][b]);
      }
    }
    // O^T = S^T Q^T e^G + u^T A^T: a lane has 4 neighbouring columns of a token
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      const float out = f[DL_OUT + 16 * tb + c16];
      const int t = 16 * tb + c16;
      f32x4 o[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) o[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint4 qf = dl_row<DK>(qt, tb, k, lane);
#pragma unroll
        for (int b = 0; b < NB; ++b) o[b] = mfma16x16x32(sp[k][b][0], qf, o[b]);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) o[b] *= out;
#pragma unroll
      for (int k = 0; k <= tb / 2; ++k) {
        const uint4 af = *reinterpret_cast<const uint4*>(ut + (18 + dl_frag(tb, k)) * 1024 + 16 * lane);
#pragma unroll
        for (int b = 0; b < NB; ++b) o[b] = mfma16x16x32(uh[k][b], af, o[b]);
      }
      if (t < left) {
        uint16_t* p = static_cast<uint16_t*>(a.d.O) + (sq.q0 + long(c) * DL_C + t) * a.d.os + h * a.d.dv + col + g4;
#pragma unroll
        for (int b = 0; b < NB; ++b)
          *reinterpret_cast<uint2*>(p + 16 * b) = make_uint2(pack2bf(o[b][0], o[b][1]), pack2bf(o[b][2], o[b][3]));
      }
    }
  }
  if (kept && a.d.state_out)
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) a.d.state_out[state + long(16 * d + g4 + r) * a.d.dv + 16 * b] = S[d][b][r];
}

long units(int n_seq, int N) { return N / DL_C + n_seq; }  // numbers of chunks

template <int DK>
hipError_t launch(const DeltaPackedArgs& a) {
  const DeltaArgs& d = a.d;
  hipLaunchKernelGGL((k_delta_prepare<DK>), dim3(unsigned(units(d.n_seq, a.N) * d.Hv)), dim3(256), 0, d.stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const long heads = long(d.n_seq) * d.Hv;
  if (d.dv % 128 == 0 && heads * d.dv / 64 > 512)
    hipLaunchKernelGGL((k_delta_scan<DK, 4, 2>), dim3(unsigned(heads * (d.dv / 128))), dim3(256), 0, d.stream, a);
  else if (heads * d.dv / 32 > 256)
    hipLaunchKernelGGL((k_delta_scan<DK, 4, 1>), dim3(unsigned(heads * (d.dv / 64))), dim3(256), 0, d.stream, a);
  else
    hipLaunchKernelGGL((k_delta_scan<DK, 2, 1>), dim3(unsigned(heads * (d.dv / 32))), dim3(128), 0, d.stream, a);
  return hipGetLastError();
}

}  // namespace

size_t delta_packed_workspace(int n_seq, int N, int Hv) { return size_t(units(n_seq, N)) * Hv * DL_UNIT; }

hipError_t delta_packed(const DeltaPackedArgs& a) { return a.d.dk == 128 ? launch<128>(a) : launch<64>(a); }

}  // namespace ttt
