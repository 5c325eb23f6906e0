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
// chunks. S stays in accumulators from the first chunk to the last: a product's result [rows, columns] has the lane
// layout of the next product's operand [contraction, columns] if the 32 rows of a contraction are taken in the
// order 16 (e / 4) + 4 (l / 16) + e % 4, e = 0..7, in both operands. Rows of S are channels in such an order
// (dl_channel) that K and Q need none: a lane's 8 channels lie side by side.
//
// Precision: what is not bf16 enters a product as a sum of bf16 planes, S, T, V - e^G K S and u as three each (of the
// nine products of planes of T and V - .., the six above 2^-24). The state is then off by 2e-7 of its size after 2048
// tokens, as an fp32 computation is; with two planes of S it was 1.2e-6, with two of the others as well 3 .. 6e-6. O,
// which is rounded to bf16 (1.66e-3 of its size, root of the mean square), takes two planes of S and u, which do not show
// in it, and A in bf16: 2.0e-3 with it. A second plane of A would be 6 KB more for each chunk and head to write and read, and
// 18 KB more of LDS, which two tiles of 128 x 16 leave no room for.
//
// What bounds it. k_delta_prepare: memory, for the most part its own 25 KB per 64 tokens and head of T, A and factors
// beside K and Q (32768 tokens of 32 heads: 419 MB out, 604 in, 203 .. 212 us, 5 TB/s, as much as a copy reaches; three
// planes of T in the order in which the scan's operands lie are more bytes than L would be, but the inverse is computed
// once for a head and not in each of its column tiles). k_delta_scan: the chain through S, whose 512 chunks follow each
// other here: 790 .. 870 us, 3450 clocks a chunk at 2.0 GHz; of that 72 matrix instructions of the wave that
// has most, 17 clocks each, and between them splits into planes and three meetings. 8192 tokens in 11 sequences of 32
// heads: 52 + 161 us.
#include <type_traits>

#include "common.hpp"
#include "dma_row.hpp"
#include "launch.hpp"

namespace ttt {
namespace {

#define DL_INLINE __attribute__((always_inline))

constexpr int DL_C = 64;             // tokens of a chunk
constexpr int DL_FRAGS = 6;          // 16 x 32 blocks of a lower triangle: (row block, contraction step) with
                                     // step <= row block / 2, numbered row block + (row block > 1) * (row block - 2) + step
constexpr int DL_TOK = 4 * DL_FRAGS * 1024;  // byte offset of the rows' factors behind 3 planes of T, then A
constexpr int DL_UNIT = DL_TOK + 1024;       // bytes of a chunk and head in the workspace
constexpr int DL_A = 3 * DL_FRAGS * 1024;    // where A begins
// the rows' factors: e^G and the norm of k [64], e^(G_C - G) and the norm of k [64], scale e^G and the norm of
// q [64], e^(G_C)
constexpr int DL_FROM = 0, DL_LEFT = 64, DL_OUT = 128, DL_WHOLE = 192;

__device__ __forceinline__ constexpr int dl_frag(int rb, int ks) { return rb + (rb > 1 ? rb - 2 : 0) + ks; }

// Up to 1024 sequences are scanned in the order of their lengths, the longest first, so that none starts late:
// k_delta_prepare leaves that order behind the units. (11 documents in 8192 tokens, 32 heads: 213 us in their own
// order, 168 by length.) A place in it takes a pass over all lengths, so that more of them are taken as they lie.
__host__ __device__ __forceinline__ constexpr bool dl_ranked(int n_seq) { return n_seq > 1 && n_seq <= 1024; }

struct DeltaChunk {
  int q0, n;  // first token and tokens of the sequence
  int base;   // its first chunk's number
};
__device__ __forceinline__ DeltaChunk dl_sequence(const DeltaPackedArgs& a, int s) {
  DeltaChunk c;
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

long units(int n_seq, int N) { return N / DL_C + n_seq; }  // numbers of chunks
__device__ __forceinline__ int* dl_order(const DeltaPackedArgs& a) {
  return reinterpret_cast<int*>(static_cast<char*>(a.ws) + size_t(a.N / DL_C + a.d.n_seq) * a.d.Hv * DL_UNIT);
}
// The place of sequence s among all by length. By all lanes of a wave.
__device__ __forceinline__ int dl_rank(const DeltaPackedArgs& a, int s, int lane) {
  const int n = dl_sequence(a, s).n;
  int rank = 0;
  for (int j0 = 0; j0 < a.d.n_seq; j0 += 64) {
    const int j = j0 + lane, nj = dl_sequence(a, min(j, a.d.n_seq - 1)).n;
    rank += __popcll(__ballot(j < a.d.n_seq && (nj > n || (nj == n && j < s))));
  }
  return rank;
}

// Tiles of rows of W bf16 in LDS, in pieces of 16 bytes; piece p of row r at slot p ^ turn(r). Reads of 8 bytes go by
// 32 lanes: 16 rows of one piece each, or (transposed) 8 rows of two neighbouring ones; either way the turns put
// them on all banks.
template <int W>
__device__ __forceinline__ int dl_turn(int r) {
  return W == 128 ? (r & 7) << 1 | (r >> 3 & 1) : W == 64 ? (r >> 1 & 3) << 1 | (r >> 3 & 1) : W == 32 ? (r >> 2 & 1) << 1 : 0;
}
template <int W>
__device__ __forceinline__ int dl_at(int r, int piece) { return r * W * 2 + ((piece ^ dl_turn<W>(r)) << 4); }

// The 1 KB number i of a 64-row tile: rows of a sequence from `src` on, `left` of which exist (the last one stands
// for those behind it), by one wave.
template <int W>
__device__ __forceinline__ void dl_copy_rows(int i, const void* src, long stride, int left, uint32_t lds, int lane) {
  constexpr int CH = W / 8, RPI = 64 / CH;  // pieces of a row, rows of a copy
  const int r = i * RPI + lane / CH, p = lane % CH;
  const uint32_t off = uint32_t(min(r, left - 1)) * uint32_t(stride * 2) + ((p ^ dl_turn<W>(r)) << 4);
  dma16(off, static_cast<const char*>(src), __builtin_amdgcn_readfirstlane(lds + i * 1024));
}

typedef short dl_s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) dl_s16x4 dl_lds_s16x4;
// 4 rows' values of a lane's column out of a row-major tile: 16 lanes read 4 rows x 16 channels.
__device__ __forceinline__ uint2 dl_transposed(const char* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((dl_lds_s16x4*)p));
}
// The 4 rows 4 (l / 16) .. of row block rb, column 16 cb + l % 16.
template <int W>
__device__ __forceinline__ uint2 dl_column(const char* tile, int rb, int cb, int lane) {
  const int r = 16 * rb + 4 * (lane >> 4) + ((lane & 15) >> 2);
  return dl_transposed(tile + dl_at<W>(r, 2 * cb + (lane >> 1 & 1)) + 8 * (lane & 1));
}
// Row 16 rb + l % 16, channels 32 ks + 8 (l / 16) ..
template <int W>
__device__ __forceinline__ uint4 dl_row(const char* tile, int rb, int ks, int lane) {
  return *reinterpret_cast<const uint4*>(tile + dl_at<W>(16 * rb + (lane & 15), 4 * ks + (lane >> 4)));
}
// The 4 rows 4 (l / 16) .. of row block rb, channel dl_channel(d, l % 16).
__device__ __forceinline__ constexpr int dl_channel(int d, int m) { return 32 * (d / 2) + 8 * (m / 4) + 4 * (d % 2) + m % 4; }
template <int W>
__device__ __forceinline__ uint2 dl_channels(const char* tile, int rb, int d, int lane) {
  const int r = 16 * rb + 4 * (lane >> 4) + ((lane & 15) >> 2);
  return dl_transposed(tile + dl_at<W>(r, 4 * (d / 2) + (lane & 3)) + 8 * (d % 2));
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
  constexpr int KS = DK / 32, LW = 68, DW = 20;  // contraction steps; rows of L, then T, and of the diagonal blocks, in floats
  __shared__ __align__(16) float ls[DL_C][LW];
  __shared__ __align__(16) float ds[4][16][DW];
  __shared__ double gs[DL_C];  // log2 of the decays, summed up
  __shared__ __align__(16) float bs[DL_C], rk_s[DL_C], rq_s[DL_C];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int h = blockIdx.x % a.d.Hv, id = blockIdx.x / a.d.Hv;
  const DeltaChunk sq = dl_sequence(a, dl_find(a, id, lane));
  const int t0 = (id - sq.base) * DL_C, left = min(sq.n - t0, DL_C);
  if (wave == 2 && dl_ranked(a.d.n_seq) && int(blockIdx.x) < a.d.n_seq) {  // there are as many workgroups and more
    const int rank = dl_rank(a, blockIdx.x, lane);
    if (lane == 0) dl_order(a)[rank] = blockIdx.x;
  }
  if (id < sq.base || left <= 0) return;
  const int hk = h / (a.d.Hv / a.d.Hk);
  const long tok = sq.q0 + t0;
  const int g4 = 4 * (lane >> 4), i0 = 16 * wave + (lane & 15);  // a lane's row of K and Q, and of L and A
  // rows of K and Q as operands: lane l has row l % 16, channels 32 s + 8 (l / 16) ..; row blocks up to the wave's own
  const auto load = [&](const void* x, long stride, int rb, uint4 (&f)[KS]) DL_INLINE {
    const uint16_t* p = static_cast<const uint16_t*>(x) + (tok + min(16 * rb + (lane & 15), left - 1)) * stride + hk * DK + 2 * g4;
#pragma unroll
    for (int s = 0; s < KS; ++s) f[s] = *reinterpret_cast<const uint4*>(p + 32 * s);
  };
  uint4 kf[4][KS], qf[KS];
  load(a.d.K, a.d.ks, wave, kf[3]);
  load(a.d.Q, a.d.qs, wave, qf);
#pragma unroll
  for (int jb = 0; jb < 3; ++jb)
    if (jb < wave) load(a.d.K, a.d.ks, jb, kf[jb]);
  if (wave == 0) {
    // sums of the gates in fp64: their differences count, also behind a gate that forgets everything (-inf:
    // e^-1000 is 0 as well, and sums of it stay finite)
    const long at = (tok + min(lane, left - 1)) * a.d.Hv + h;
    float g = a.d.g[at];
    const float beta = a.d.beta[at];
    g = lane < left ? (g < -1000.f ? -1000.f : g) : 0.f;
    double G = g * 1.4426950408889634074;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double up = __shfl_up(G, d);
      if (lane >= d) G += up;
    }
    gs[lane] = G;
    bs[lane] = lane < left ? beta : 0.f;
  }
  // Row block `wave` of K K^T and Q K^T, as blocks [j, i] of products K K^T and K Q^T: lane l has row i = l % 16 of
  // the block and its columns j = 4 (l / 16) .. The squares of the norms are the diagonals of K K^T and Q Q^T.
  f32x4 kk[4], kq[4], qq = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < KS; ++s) qq = mfma16x16x32(qf[s], qf[s], qq);
#pragma unroll
  for (int jb = 3; jb >= 0; --jb) {
    kk[jb] = kq[jb] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (jb > wave) continue;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint4 f = jb < 3 && jb < wave ? kf[jb][s] : kf[3][s];
      kk[jb] = mfma16x16x32(f, kf[3][s], kk[jb]);
      kq[jb] = mfma16x16x32(f, qf[s], kq[jb]);
    }
  }
  if ((lane & 15) / 4 == lane / 16) {  // has the diagonal's i = j
    const f32x4 d = wave == 0 ? kk[0] : wave == 1 ? kk[1] : wave == 2 ? kk[2] : kk[3];
    const int r = lane & 3;
    const float k2 = r == 0 ? d[0] : r == 1 ? d[1] : r == 2 ? d[2] : d[3];
    const float q2 = r == 0 ? qq[0] : r == 1 ? qq[1] : r == 2 ? qq[2] : qq[3];
    rk_s[i0] = a.d.norm ? rsqrtf(k2 + a.d.eps) : 1.f;
    rq_s[i0] = a.d.scale * (a.d.norm ? rsqrtf(q2 + a.d.eps) : 1.f);
  }
  __syncthreads();

  // the same of L and A
  char* const unit = static_cast<char*>(a.ws) + (size_t(id) * a.d.Hv + h) * DL_UNIT;
  {
    const double gi = gs[i0];
    const float bi = bs[i0] * rk_s[i0], qi = i0 < left ? rq_s[i0] : 0.f;
    uint2 aw[4];
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      aw[jb] = make_uint2(0, 0);
      if (jb > wave) continue;
      const float4 rk = *reinterpret_cast<const float4*>(&rk_s[16 * jb + g4]);
      float lv[4], av[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * jb + g4 + r;
        const float decay = __builtin_amdgcn_exp2f(float(gi - gs[j])) * (r == 0 ? rk.x : r == 1 ? rk.y : r == 2 ? rk.z : rk.w);
        lv[r] = j < i0 && i0 < left ? bi * decay * kk[jb][r] : 0.f;
        av[r] = j <= i0 && i0 < left ? qi * decay * kq[jb][r] : 0.f;
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
  if (wave == 0) {
    float* f = reinterpret_cast<float*>(unit + DL_TOK);
    const double G = gs[lane], all = gs[DL_C - 1];
    const float from = __builtin_amdgcn_exp2f(float(G));
    f[DL_FROM + lane] = from * rk_s[lane];
    f[DL_LEFT + lane] = __builtin_amdgcn_exp2f(float(all - G)) * rk_s[lane];
    f[DL_OUT + lane] = from * rq_s[lane];
    f[DL_WHOLE + lane] = __builtin_amdgcn_exp2f(float(all));
  }
  __syncthreads();
  // The inverse of 1 + L: the four diagonal blocks by forward substitution, a column to each lane of one wave
  if (wave == 3) {
    const int c = lane & 15, b = lane >> 4;
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x[4] = {i == c ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < i; k += 4) {
        const float4 l = *reinterpret_cast<const float4*>(&ls[16 * b + i][16 * b + k]);
        x[0] = fmaf(-l.x, t[k], x[0]);
        if (k + 1 < i) x[1] = fmaf(-l.y, t[k + 1], x[1]);
        if (k + 2 < i) x[2] = fmaf(-l.z, t[k + 2], x[2]);
        if (k + 3 < i) x[3] = fmaf(-l.w, t[k + 3], x[3]);
      }
      t[i] = (x[0] + x[1]) + (x[2] + x[3]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) ds[b][i][c] = t[i];
  }
  __syncthreads();
  // then block column `wave` from the top: T_ij = -T_ii sum_k L_ik T_kj
  f32x4 col[4];  // T_kj, j = wave, as operands: column l % 16, rows 4 (l / 16) ..
#pragma unroll
  for (int r = 0; r < 4; ++r) col[0][r] = ds[wave][g4 + r][lane & 15];
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
    const float4 d = *reinterpret_cast<const float4*>(&ds[ib][lane & 15][g4]);
    f32x4 z = {0.f, 0.f, 0.f, 0.f};
    z = dl_mma_f32(d.x, -y[0], z);
    z = dl_mma_f32(d.y, -y[1], z);
    z = dl_mma_f32(d.z, -y[2], z);
    z = dl_mma_f32(d.w, -y[3], z);
    col[n] = z;
  }
  __syncthreads();  // L has been read: T takes its place
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    if (wave + n > 3) break;
#pragma unroll
    for (int r = 0; r < 4; ++r) ls[16 * (wave + n) + g4 + r][16 * wave + (lane & 15)] = col[n][r];
  }
  __syncthreads();
  // row block `wave` of T, its columns times beta, in three planes
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s > wave / 2) break;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const int jb = 2 * s + e / 4, j = 16 * jb + g4;
      const float4 t = jb <= wave ? *reinterpret_cast<const float4*>(&ls[i0][j]) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 b = *reinterpret_cast<const float4*>(&bs[j]);
      x[e] = t.x * b.x, x[e + 1] = t.y * b.y, x[e + 2] = t.z * b.z, x[e + 3] = t.w * b.w;
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<uint4*>(unit + (6 * p + dl_frag(wave, s)) * 1024 + 16 * lane) = dl_plane(x, p == 2);
  }
}

// --------------------------------------------------------------------------------------------
// A split of 8 values into three planes of bf16 in 20 small steps, which stand between products.
struct DlSplit {
  float x[8];
  uint32_t w[3][4];
  __device__ __forceinline__ void step(int n) {
    if (n < 16) {
      const int p = n / 8, i = n % 8 / 2;
      if (n % 2 == 0) {
        w[p][i] = pack2bf(x[2 * i], x[2 * i + 1]);
        x[2 * i] -= __uint_as_float(w[p][i] << 16);
      } else {
        x[2 * i + 1] -= __uint_as_float(w[p][i] & 0xFFFF0000u);
      }
    } else {
      w[2][n - 16] = pack2bf(x[2 * (n - 16)], x[2 * (n - 16) + 1]);
    }
  }
  __device__ __forceinline__ void set(int i, float v) { x[i] = v; }
  __device__ __forceinline__ uint4 plane(int p) const { return make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]); }
};
__device__ __forceinline__ void dl_fence() { __builtin_amdgcn_sched_barrier(0); }
// All waves; LDS written before is seen behind it. (The vector-memory counter is left alone.)
__device__ __forceinline__ void dl_meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Where the waves meet. LDS written before is seen behind it; the vector-memory counter is left alone.
template <int MOST>
__device__ __forceinline__ void dl_meet_copied() {  // and at most MOST of the wave's copies and stores are under way
  wait_vm<MOST>();
  dl_meet();
}

// One workgroup: 16 or 32 columns of a state, in TILES tiles of 16. A tile has two waves that carry it from chunk to chunk,
// each on a SIMD of its own, and two that do the rest beside them. Of the carrying waves the first has the state's
// first half of rows and the chunk's first 32 tokens, the second the others: each multiplies its rows of S by all of
// K, hands the sums for the other's tokens over, solves for its tokens' u (the second with what the first hands on)
// and adds all u to its rows. Their vector work is dealt out between the products. The others copy tiles
// into LDS and compute the outputs, 32 tokens each, from the planes of S and the u that are left in LDS. All
// meet three times a chunk; what is there behind a meeting:
//   1  the sums for the other's tokens; the planes of S
//   2  the first half's V - e^G K S, in planes; Q of chunk c; K, V and A of chunk c + 1
//   3  u, and what of it the state takes, in planes
// K, V and A are copied two chunks ahead: one ahead, the copies were late where the inputs come from HBM (32768 tokens of
// 32 heads, both launches 1046 us, this 984; 8192 tokens 260 and 255).
// What u adds to the outputs is added behind 3, while the carrying waves finish the state and begin the next chunk.
template <int DK, int TILES>
__global__ __launch_bounds__(256 * TILES, 1) void k_delta_scan(DeltaPackedArgs a) {
  constexpr int CARRY = 2 * TILES, CW = 16 * TILES, KT = DL_C * DK * 2, VT = DL_C * CW * 2;
  constexpr int DB = DK / 16, KS = DK / 32;  // row blocks of the state, contraction steps over them
  constexpr int DH = DB / 2, KH = KS / 2;    // a wave's share of them
  constexpr int REST = DL_UNIT - DL_A;                             // A and the rows' factors
  constexpr int AT_U = KT, AT_V = AT_U + REST, STAGE = AT_V + VT;  // K, these, V
  struct Hand {
    char s[2 * KS * 1024];  // two planes of S
    char u[4 * 1024];       // u, row blocks in fp32
    char r[3 * 1024];       // planes of the first half's V - e^G K S
    char sum[4 * 1024];     // sums for the tokens of the first, of the second wave
    char x[6 * 1024];       // planes of what the state takes of u
  };
  __shared__ __align__(1024) char sm[3][STAGE];
  __shared__ __align__(1024) char q_s[KT];
  __shared__ __align__(1024) Hand hand[TILES];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  // the column tiles of a head follow each other on one XCD where there are 8 heads: they read the same K, Q, T and A
  const int wide = a.d.Hv * (a.d.dv / CW), nth = blockIdx.x / wide;
  const int h = blockIdx.x % wide % a.d.Hv, col0 = blockIdx.x % wide / a.d.Hv * CW, hk = h / (a.d.Hv / a.d.Hk);
  const int s = dl_ranked(a.d.n_seq) ? __builtin_amdgcn_readfirstlane(dl_order(a)[nth]) : nth;
  const DeltaChunk sq = dl_sequence(a, s);
  const int me = wave & 1, tile = TILES == 2 ? wave >> 1 & 1 : 0, col = col0 + 16 * tile;
  const int g4 = 4 * (lane >> 4), c16 = lane & 15, l16 = 16 * lane;
  const int chunks = (sq.n + DL_C - 1) / DL_C;
  char *const s_s = hand[tile].s, *const u_s = hand[tile].u, *const r_s = hand[tile].r, *const x_s = hand[tile].x,
       *const sum_s = hand[tile].sum;

  if (wave >= CARRY) {
    constexpr int NK = KT / 1024 / CARRY, NU = (REST / 1024 + CARRY - 1) / CARRY, BACK = 3 * 1024;  // copies of a wave; NU: some are repetitions
    const int w = wave - CARRY;
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_u32(sm)), lds_q = __builtin_amdgcn_readfirstlane(lds_u32(q_s));
    const uint16_t* kp = static_cast<const uint16_t*>(a.d.K) + long(sq.q0) * a.d.ks + hk * DK;
    const uint16_t* qp = static_cast<const uint16_t*>(a.d.Q) + long(sq.q0) * a.d.qs + hk * DK;
    const uint16_t* vp = static_cast<const uint16_t*>(a.d.V) + long(sq.q0) * a.d.vs + h * a.d.dv + col0;
    const char* up = static_cast<const char*>(a.ws) + (size_t(sq.base) * a.d.Hv + h) * DL_UNIT;
    // A lane's offsets in the copies of 16 rows of K or Q; the instruction counts 1024 i for the i-th itself, and
    // 3 KB the base lacks, so that no offset is negative.
    constexpr int CH = DK / 8, RPI = 64 / CH;
    constexpr int N16 = 16 / RPI;
    static_assert(N16 <= 4 && NK % N16 == 0, "a wave copies 16 rows at a time");
    const auto offsets = [&](long stride, uint32_t (&off)[N16]) DL_INLINE {
#pragma unroll
      for (int i = 0; i < N16; ++i) {
        const int r = i * RPI + lane / CH;
        off[i] = uint32_t(r) * uint32_t(stride * 2) + ((lane % CH ^ dl_turn<DK>(r)) << 4) + BACK - 1024 * i;
      }
    };
    uint32_t ko[N16], qo[N16];
    offsets(a.d.ks, ko);
    offsets(a.d.qs, qo);
    const auto rows = [&](const uint16_t* src, long stride, const uint32_t (&off)[N16], int left, uint32_t to) DL_INLINE {
      if (left >= DL_C) {
#pragma unroll
        for (int n = 0; n < NK / N16; ++n) {
          const char* base = reinterpret_cast<const char*>(src + long(16 * (NK / N16 * w + n)) * stride) - BACK;
          dma16_at<0>(off[0], base, to + (NK * w + N16 * n) * 1024);
          dma16_at<1>(off[1], base, to);
          if constexpr (N16 == 4) {
            dma16_at<2>(off[2], base, to);
            dma16_at<3>(off[3], base, to);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < NK; ++i) dl_copy_rows<DK>(NK * w + i, src, stride, left, to, lane);
      }
    };
    // The copies of chunk c, in three parts: they are waited for one after the other, so their numbers count, and
    // stores that follow stay behind them. K, V and A go to one of three stages.
    const auto part = [&](int which, int c, int stage = 0) DL_INLINE {
      const uint32_t to = lds + stage * STAGE;
      const int left = sq.n - c * DL_C;
      if (which == 0) rows(kp + long(c) * DL_C * a.d.ks, a.d.ks, ko, left, to);
      if (which == 2) rows(qp + long(c) * DL_C * a.d.qs, a.d.qs, qo, left, lds_q);
      if (which == 1) {
        dl_copy_rows<CW>(w, vp + long(c) * DL_C * a.d.vs, a.d.vs, left, to + AT_V, lane);
        const char* u = up + size_t(c) * a.d.Hv * DL_UNIT + DL_A;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          const int n = min(NU * w + i, REST / 1024 - 1);
          dma16(l16, u + n * 1024, to + AT_U + n * 1024);
        }
      }
      asm volatile("" ::: "memory");
      dl_fence();
    };
    constexpr int NVU = 1 + NU, STORES = 2;
    f32x4 o[2];
    uint4 af[2][2];  // (those of the first half's second step are not used)
    // the outputs of a chunk: what S gave, + u^T A^T
    const auto finish = [&](int c) DL_INLINE {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k > me) break;
        uint4 u[2];
        dl_planes<2>(*reinterpret_cast<const f32x4*>(u_s + 2 * k * 1024 + l16),
                     *reinterpret_cast<const f32x4*>(u_s + (2 * k + 1) * 1024 + l16), u);
#pragma unroll
        for (int p = 1; p >= 0; --p)
#pragma unroll
          for (int t = 0; t < 2; ++t) o[t] = mfma16x16x32(u[p], af[t][k], o[t]);
      }
      const int left = sq.n - c * DL_C;
      uint16_t* p = static_cast<uint16_t*>(a.d.O) + (sq.q0 + long(c) * DL_C) * a.d.os + h * a.d.dv + col + g4;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tok = 16 * (2 * me + t) + c16;
        if (tok < left)
          *reinterpret_cast<uint2*>(p + long(tok) * a.d.os) = make_uint2(pack2bf(o[t][0], o[t][1]), pack2bf(o[t][2], o[t][3]));
      }
    };
    if (chunks > 0) {
      part(0, 0);
      part(1, 0);
      part(2, 0);
    }
    if (chunks > 1) {
      part(0, 1, 1);
      part(1, 1, 1);
    }
    dl_meet_copied<0>();
    int at = 0, to = 2;  // c and c + 2 modulo 3
    for (int c = 0; c < chunks; ++c) {
      const bool next = c + 2 < chunks;
      if (next) part(0, c + 2, to);
      if (c > 0) finish(c - 1);
      asm volatile("" ::: "memory");  // its stores stay between the copies: they are counted together
      dl_fence();
      const char* const ut = sm[at] + AT_U;
      const float* const f = reinterpret_cast<const float*>(ut + DL_TOK - DL_A);
      dl_meet();  // 1
      if (next) part(1, c + 2, to);
      uint4 sp[KS][2];
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int p = 0; p < 2; ++p) sp[k][p] = *reinterpret_cast<const uint4*>(s_s + (2 * k + p) * 1024 + l16);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          af[t][k] = *reinterpret_cast<const uint4*>(ut + (me ? dl_frag(2 + t, k) : t) * 1024 + l16);
      // 2: behind K, V and A of the next chunk and Q of this one come K of the one after, the last outputs, its V and A
      if (next) dl_meet_copied<NK + STORES + NVU>();
      else dl_meet_copied<STORES>();
      // O^T = S^T Q^T e^G: a lane has 4 neighbouring columns of a token
#pragma unroll
      for (int t = 0; t < 2; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint4 q[2] = {dl_row<DK>(q_s, 2 * me, k, lane), dl_row<DK>(q_s, 2 * me + 1, k, lane)};
#pragma unroll
        for (int p = 1; p >= 0; --p)
#pragma unroll
          for (int t = 0; t < 2; ++t) o[t] = mfma16x16x32(sp[k][p], q[t], o[t]);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) o[t] *= f[DL_OUT + 16 * (2 * me + t) + c16];
      dl_meet();  // 3
      if (c + 1 < chunks) part(2, c + 1);
      to = at;
      at = at == 2 ? 0 : at + 1;
    }
    dl_meet();  // the last u
    if (chunks > 0) finish(chunks - 1);
    return;
  }

  __builtin_amdgcn_s_setprio(3);
  const long slot = a.d.slots ? a.d.slots[s] : s;
  const bool kept = slot >= 0 && slot < a.d.n_slots;
  const long state = ((kept ? slot : 0) * a.d.Hv + h) * long(DK) * a.d.dv + col + c16;
  const auto row = [&](int d, int r) DL_INLINE { return state + long(dl_channel(DH * me + d, g4) + r) * a.d.dv; };
  f32x4 S[DH];
#pragma unroll
  for (int d = 0; d < DH; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) S[d][r] = kept && a.d.state_in ? a.d.state_in[row(d, r)] : 0.f;
  uint4 sp[KH][3];
  DlSplit cut;
  const auto cut_state = [&](int k, int n) DL_INLINE {  // step n of the split of the wave's rows 32 k ..
    if (n == 0)
#pragma unroll
      for (int i = 0; i < 8; ++i) cut.set(i, S[2 * k + i / 4][i % 4]);
    cut.step(n);
    if (n == 19)
#pragma unroll
      for (int p = 0; p < 3; ++p) sp[k][p] = cut.plane(p);
  };
  const auto leave = [&](int k) DL_INLINE {  // two planes of the state for the outputs
#pragma unroll
    for (int p = 0; p < 2; ++p) *reinterpret_cast<uint4*>(s_s + (2 * (KH * me + k) + p) * 1024 + l16) = sp[k][p];
  };
  // steps of `op`, `total` in all, in proportion to the slots of a phase, the first `wait` of them without
  const auto deal = [&](int at, int slots, int wait, int total, auto&& op) DL_INLINE {
    if (at < wait) return;
    const int n0 = (at - wait) * total / (slots - wait), n1 = (at + 1 - wait) * total / (slots - wait);
#pragma unroll
    for (int n = n0; n < n1; ++n) op(n);
  };
#pragma unroll
  for (int k = 0; k < KH - 1; ++k)
#pragma unroll
    for (int n = 0; n < 20; ++n) cut_state(k, n);

  // Products of planes, the largest last but for the order in which the planes get ready.
  constexpr int TP[6] = {2, 1, 0, 1, 0, 0}, XP[6] = {0, 0, 0, 1, 1, 2};
  uint4 kf[KH][4];  // K: blocks 0, 1 the other wave's tokens, 2, 3 its own
  const auto read_k = [&](const char* kt, int i) DL_INLINE {
    const int b = i % 4;
    kf[i / 4][b] = dl_row<DK>(kt, 2 * (b < 2 ? 1 - me : me) + b % 2, KH * me + i / 4, lane);
  };
  // T of the wave's tokens by its own (t) and, for the second, by the first's (t0): straight from the workspace, a chunk
  // ahead (of the last one's: again)
  uint4 t[2][3], t0[2][3];
  const char* const up = static_cast<const char*>(a.ws) + (size_t(sq.base) * a.d.Hv + h) * DL_UNIT;
  const auto T = [&](int c, int p, int frag) DL_INLINE {
    return *reinterpret_cast<const uint4*>(up + size_t(min(c, chunks - 1)) * a.d.Hv * DL_UNIT + (6 * p + frag) * 1024 + l16);
  };
  const auto read_own = [&](int c) DL_INLINE {
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int b = 0; b < 2; ++b) t[b][p] = T(c, p, me ? dl_frag(2 + b, 1) : b);
  };
  const auto read_first = [&](int c) DL_INLINE {
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int b = 0; b < 2; ++b) t0[b][p] = T(c, p, dl_frag(2 + b, 0));
  };
  if (chunks > 0) {
    read_own(0);
    if (me) read_first(0);
  }
  dl_meet();
  if (chunks > 0)
#pragma unroll
    for (int i = 0; i < 4 * KH; ++i) read_k(sm[0], i);
  for (int c = 0, at = 0; c < chunks; ++c) {
    if (KH == 1)
#pragma unroll
      for (int n = 0; n < 20; ++n) cut_state(0, n);
    const char* const kt = sm[at];
    at = at == 2 ? 0 : at + 1;
    const char* const ut = kt + AT_U;
    const char* const vt = kt + AT_V;
    const float* const f = reinterpret_cast<const float*>(ut + DL_TOK - DL_A);
    // P = K S over the wave's rows of S, whose last ones are split meanwhile; what the next steps take is read
    f32x4 x[4];
    uint4 kc[2][DH];
    uint2 v[2];
    float4 from[2], keep[2];
    const auto read_kc = [&](int k, int d) DL_INLINE {  // K^T of tokens 32 k .., the wave's row block d
      const uint2 lo = dl_channels<DK>(kt, 2 * k, DH * me + d, lane), hi = dl_channels<DK>(kt, 2 * k + 1, DH * me + d, lane);
      return make_uint4(lo.x, lo.y, hi.x, hi.y);
    };
#pragma unroll
    for (int k = 0; k < 12 * KH; ++k) {
      const int st = k / 12, p = 2 - k % 6 / 2, b = 2 * (k / 6 % 2) + k % 2;
      if (k < 12 && k % 6 < 2) x[b] = f32x4{0.f, 0.f, 0.f, 0.f};
      x[b] = mfma16x16x32(kf[st][b], sp[st][p], x[b]);
      if (KH == 2 && k < 12) deal(k, 12, 0, 20, [&](int n) DL_INLINE { cut_state(KH - 1, n); });
      if (k == 1) leave(0);
      if (KH == 2 && k == 14) leave(1);
      if (k >= 2 && k < 4) {
        v[k - 2] = dl_column<CW>(vt, 2 * me + k - 2, tile, lane);
        from[k - 2] = *reinterpret_cast<const float4*>(f + DL_FROM + 16 * (2 * me + k - 2) + g4);
      } else if (k >= 15 && k < 17) {
        keep[k - 15] = *reinterpret_cast<const float4*>(f + DL_LEFT + 16 * (2 * me + k - 15) + g4);
      }
      if (k == 12 * KH - 2) {
        *reinterpret_cast<f32x4*>(sum_s + (1 - me) * 2048 + l16) = x[0];
        *reinterpret_cast<f32x4*>(sum_s + (1 - me) * 2048 + 1024 + l16) = x[1];
      }
      dl_fence();
    }
    dl_meet();  // 1
    f32x4 other[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) other[b] = *reinterpret_cast<const f32x4*>(sum_s + me * 2048 + b * 1024 + l16);
    if (KH == 1)
#pragma unroll
      for (int b = 0; b < 2; ++b) keep[b] = *reinterpret_cast<const float4*>(f + DL_LEFT + 16 * (2 * me + b) + g4);
    const float whole = f[DL_WHOLE];
    // V - e^G P of the wave's tokens, in planes, and u = T (..) of those
    f32x4 u[2];
    uint4 xp[3];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const f32x4 y = x[2 + b] + other[b];
      cut.set(4 * b, fmaf(-from[b].x, y[0], __uint_as_float(v[b].x << 16)));
      cut.set(4 * b + 1, fmaf(-from[b].y, y[1], __uint_as_float(v[b].x & 0xFFFF0000u)));
      cut.set(4 * b + 2, fmaf(-from[b].z, y[2], __uint_as_float(v[b].y << 16)));
      cut.set(4 * b + 3, fmaf(-from[b].w, y[3], __uint_as_float(v[b].y & 0xFFFF0000u)));
    }
#pragma unroll
    for (int n = 0; n < 8; ++n) cut.step(n);
    xp[0] = cut.plane(0);
    u[0] = u[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 12; ++k) {
      const int n = k / 2, b = k % 2;
      if (k == 6) xp[1] = cut.plane(1);
      if (k == 10) xp[2] = cut.plane(2);
      if (me == 0 && k == 10) {
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4*>(r_s + p * 1024 + l16) = xp[p];
      }
      u[b] = mfma16x16x32(t[b][TP[n]], xp[XP[n]], u[b]);
      if (k < 8) deal(k, 8, 0, 12, [&](int i) DL_INLINE { cut.step(8 + i); });
      if (k < DH) kc[0][k] = read_kc(me, k);  // own tokens
      dl_fence();
    }
    read_own(c + 1);
    dl_meet();  // 2
#pragma unroll
    for (int d = 0; d < DH; ++d) S[d] *= whole;
    if (me) {
      uint4 r[3];
#pragma unroll
      for (int p = 0; p < 3; ++p) r[p] = *reinterpret_cast<const uint4*>(r_s + p * 1024 + l16);
      dl_fence();
#pragma unroll
      for (int n = 0; n < 6; ++n)
#pragma unroll
        for (int b = 0; b < 2; ++b) u[b] = mfma16x16x32(t0[b][TP[n]], r[XP[n]], u[b]);
      read_first(c + 1);
    }
    uint4 xu[3], xo[3];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      cut.set(4 * b, u[b][0] * keep[b].x);
      cut.set(4 * b + 1, u[b][1] * keep[b].y);
      cut.set(4 * b + 2, u[b][2] * keep[b].z);
      cut.set(4 * b + 3, u[b][3] * keep[b].w);
      *reinterpret_cast<f32x4*>(u_s + (2 * me + b) * 1024 + l16) = u[b];
    }
#pragma unroll
    for (int n = 0; n < 20; ++n) {
      cut.step(n);
      if (n % 8 == 7 || n == 19) {
        xu[n / 8] = cut.plane(n / 8);
        *reinterpret_cast<uint4*>(x_s + me * 3072 + n / 8 * 1024 + l16) = xu[n / 8];
      }
    }
#pragma unroll
    for (int d = 0; d < DH; ++d) kc[1][d] = read_kc(1 - me, d);
    dl_fence();
    if (me == 0) {
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int d = 0; d < DH; ++d) S[d] = mfma16x16x32(kc[0][d], xu[p], S[d]);
    }
    dl_meet();  // 3
#pragma unroll
    for (int p = 0; p < 3; ++p) xo[p] = *reinterpret_cast<const uint4*>(x_s + (1 - me) * 3072 + p * 1024 + l16);
    dl_fence();
    if (me) {
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int d = 0; d < DH; ++d) S[d] = mfma16x16x32(kc[0][d], xu[p], S[d]);
    }
    dl_fence();
    // with the split of the rows that are done, and the next chunk's K (of the last one's: not used)
#pragma unroll
    for (int k = 0; k < 3 * DH; ++k) {
      const int d = 2 * (k / 6) + k % 2, p = 2 - k % 6 / 2;
      S[d] = mfma16x16x32(kc[1][d], xo[p], S[d]);
      if (k < 4 * KH) read_k(sm[at], k);
      if (KH > 1) deal(k, 3 * DH, 7, 20 * (KH - 1), [&](int i) DL_INLINE { cut_state(i / 20, i % 20); });
      dl_fence();
    }
  }
  dl_meet();  // the last u
  if (kept && a.d.state_out)
#pragma unroll
    for (int d = 0; d < DH; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) a.d.state_out[row(d, r)] = S[d][r];
}

template <int DK>
hipError_t launch(const DeltaPackedArgs& a) {
  const DeltaArgs& d = a.d;
  hipLaunchKernelGGL((k_delta_prepare<DK>), dim3(unsigned(units(d.n_seq, a.N) * d.Hv)), dim3(256), 0, d.stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const long heads = long(d.n_seq) * d.Hv;
  // 16 columns of a workgroup where each then has one of the card's 256 units to itself, and its carrying waves a SIMD:
  // 32 where there are more (one fits a unit). 8192 tokens, both launches with 16 and with 32 columns: 128 x 128, 4 heads 193
  // and 229 us, 32 heads 254 and 280, 40 heads 500 and 314, 128 heads 1366 and 803; 64 x 128, 8 heads 173 and 202, 32 heads 205
  // and 230, 40 heads 268 and 262, 64 heads 370 and 298; 128 x 64, 64 heads 325 and 357, 96 heads 648 and 419; 11 sequences in
  // 8192 tokens, 32 heads of 128 x 128, 282 and 200.
  if (heads * (d.dv / 16) <= 256)
    hipLaunchKernelGGL((k_delta_scan<DK, 1>), dim3(unsigned(heads * (d.dv / 16))), dim3(256), 0, d.stream, a);
  else
    hipLaunchKernelGGL((k_delta_scan<DK, 2>), dim3(unsigned(heads * (d.dv / 32))), dim3(512), 0, d.stream, a);
  return hipGetLastError();
}

}  // namespace

size_t delta_packed_workspace(int n_seq, int N, int Hv) {
  return size_t(units(n_seq, N)) * Hv * DL_UNIT + (dl_ranked(n_seq) ? (n_seq * 4 + 255) / 256 * 256 : 0);
}

hipError_t delta_packed(const DeltaPackedArgs& a) { return a.d.dk == 128 ? launch<128>(a) : launch<64>(a); }

}  // namespace ttt
