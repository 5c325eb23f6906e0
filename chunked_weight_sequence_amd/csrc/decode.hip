// One-token attention over a paged cache, grouped heads, bf16, and the joining of partial
// results that a split over the keys leaves (also used by attention.hip).
//
// Sequence s holds n = lengths[s] tokens; token j is row table[s][j / page] * page + j % page of
// the caches [n_pages * page][Hkv][dh]. Its query sees the last `window` of them (all without a
// window): o = sum_j softmax_j(scale q . k_j) v_j, lse = log sum_j exp(scale q . k_j); o = 0 and
// lse = -inf where nothing is visible. Tokens of a page outside [0, n_pages) are left out.
//
// Bound by HBM: every visible K and V row is read once. A workgroup takes a piece of one
// sequence and one key head, with up to 32 of the query heads that share it as the columns of
// S^T (attn.hpp); its 2 or 4 waves walk 32-key tiles independently, each through its own two-stage LDS
// ring of direct copies (no barrier in the loop), and join their sums through LDS at the end.
// Copies are whole rows, so each instruction reads 1 KB in full lines. Rows that are masked
// (behind the last token, before the window) are replaced by a visible row of the tile in the
// copy itself: what lies in them, NaN included, never enters a product. 32/8 heads of 128: 16 sequences
// of 32768 tokens, 2.1 GB, 365 .. 378 us (5.7 TB/s; a copy reaches 4.9), 1 of 4096 8.2 us in two launches; 33 of
// up to 5000, 16/4 heads of 64, 86 MB, 22 .. 25 us.
#include <type_traits>

#include "attn.hpp"
#include "attn_plan.hpp"
#include "launch.hpp"

namespace ttt {
namespace {

constexpr int DC_BN = 32;

// a row of zeros: what stands for the tokens of a page that does not exist
__device__ const uint4 dc_zeros[16] = {};

struct DecodeDev {
  const uint16_t* Q;
  long qs;
  const char *Kc, *Vc;
  uint16_t* O;
  long os;
  float* lse;
  const int *table, *lengths;
  int max_pages, psh, n_pages;
  int n_seq, Hq, Hkv, G;
  float scale;
  int window;
  int splits;
  float* part;
};

// The page table through the scalar cache: a vector load in the key loop would make the compiler
// wait for every copy in flight, since the vector-memory counter counts them together.
typedef const __attribute__((address_space(4))) int const_int;

template <int DH, int W>
__global__ __launch_bounds__(64 * W) void k_attention_decode(DecodeDev a) {
  constexpr int TILE = DC_BN * DH * 2, KS = DH / 16, DT = DH / 32, RPI = 1024 / (DH * 2);
  constexpr int NI = 16 / RPI;  // copies per 16-token half of a tile
  __shared__ __align__(1024) char sm[W][2][2][TILE];  // wave, stage, K / V
  __shared__ float2 ml_s[W][32];
  __shared__ bool odd_s;  // a result is not finite, although its weights are
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int h = lane >> 5, col = lane & 31;
  int id = blockIdx.x;
  const int kvh = id % a.Hkv;
  id /= a.Hkv;
  const int split = id % a.splits;
  id /= a.splits;
  const int seq = id % a.n_seq, g0 = (id / a.n_seq) * 32;
  const int gn = min(a.G - g0, 32);

  const int psh = a.psh;
  const long cap = long(a.max_pages) << psh;
  const int n = int(min(long(max(a.lengths[seq], 0)), cap));
  const int first = a.window > 0 ? max(0, n - a.window) : 0;
  int t0 = first / DC_BN, t1 = n > first ? (n + DC_BN - 1) / DC_BN : t0;
  {
    const int per = (t1 - t0 + a.splits - 1) / a.splits;
    t0 = min(t0 + split * per, t1);
    t1 = min(t0 + per, t1);
  }
  uint4 qf[KS];
  {
    const uint16_t* p = a.Q + long(seq) * a.qs + (kvh * a.G + g0 + min(col, gn - 1)) * DH + 8 * h;
#pragma unroll
    for (int s = 0; s < KS; ++s) qf[s] = *reinterpret_cast<const uint4*>(p + 16 * s);
  }
  const_int* table =
      (const_int*)(reinterpret_cast<uintptr_t>(a.table) + size_t(seq) * a.max_pages * 4);
  const uint32_t rowb = uint32_t(a.Hkv) * DH * 2;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_u32(&sm[wave][0][0][0]));
  const int lrow = lane / (64 / RPI), lchunk = lane % (64 / RPI);
  // Copies tile t into a stage; returns which 16-token halves exist (bit 0, bit 1).
  auto issue = [&](int t, int stage) __attribute__((always_inline)) {
    int good = 0;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int f = t * DC_BN + 16 * hf;
      int lo = max(f, first), hi = min(f + 15, n - 1);
      if (lo > hi) lo = hi = min(max(f, first), n - 1);
      const int page = table[__builtin_amdgcn_readfirstlane(lo >> psh)];
      const bool ok = page >= 0 && page < a.n_pages;
      good |= int(ok) << hf;
      // row of token `lo`; page size is a power of two of at least 16, so a half is in one page
      const long row = ok ? (long(page) << psh) + (lo & ((1 << psh) - 1)) : 0;
      const long at = row * rowb + kvh * DH * 2;
      const char* kb = ok ? a.Kc + at : reinterpret_cast<const char*>(dc_zeros);
      const char* vb = ok ? a.Vc + at : reinterpret_cast<const char*>(dc_zeros);
      const uint32_t rb = ok ? rowb : 0;
      const uint32_t dst = lds0 + stage * 2 * TILE + hf * (TILE / 2);
      // the instruction adds 1024 i to both addresses: that much less here, and 3 KB more, which the
      // bases lack, so that no offset is negative
      constexpr uint32_t BACK = 3 * 1024;
      const auto copies = [&](const char* base, uint32_t m0, auto swizzle) __attribute__((always_inline)) {
        const auto one = [&](auto i) __attribute__((always_inline)) {
          constexpr int I = decltype(i)::value;
          const int r = 16 * hf + I * RPI + lrow;  // row of the tile
          const uint32_t o = uint32_t(min(max(t * DC_BN + r, lo), hi) - lo) * rb;
          dma16_at<I>(o + uint32_t((lchunk ^ swizzle(r)) << 4) + (BACK - 1024 * I), base - BACK, m0);
        };
        one(std::integral_constant<int, 0>());
        one(std::integral_constant<int, 1>());
        if constexpr (NI == 4) {
          one(std::integral_constant<int, 2>());
          one(std::integral_constant<int, 3>());
        }
      };
      copies(kb, dst, [](int r) { return ksw<DH>(r); });
      copies(vb, dst + TILE, [](int r) { return vsw<DH>(r); });
    }
    return good;
  };

  const FragOff<DH> fo(lane);
  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;
  const float c = a.scale * kLog2e;

  // The weights are relative to the running maximum and divided by their sum at the end, so sums of finite
  // values can pass fp32 on the way although their mean does not. Where that shows in the results, they are
  // taken a second time, with the weights lower by a power of two, 2^-add, above the sum of the first.
  float* js = reinterpret_cast<float*>(&sm[0][0][0][0]);
  const long nrows = long(a.n_seq) * a.Hq;
  float add = 0.f, whole = 0.f;
  bool again = false;
  if (tid == 0) odd_s = false;  // seen by all behind the first barrier
  while (true) {
    int good = 0, t = t0 + wave, stage = 0;
    if (t < t1) good = issue(t, 0);
    for (; t < t1; t += W, stage ^= 1) {
      int good_next = 0;
      // this tile's stage was read two rounds ago: those reads are done before it is refilled
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (t + W < t1) {
        good_next = issue(t + W, stage ^ 1);
        wait_vm<4 * NI>();
      } else {
        wait_vm<0>();
      }
      const char* kt = &sm[wave][stage][0][0];
      const char* vt = &sm[wave][stage][1][0];
      f32x16 s;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) s = mfma32x32x16(fo.key(kt, 0, ks), qf[ks], s);
      const int j0 = t * DC_BN;
      if (good != 3 || j0 < first || j0 + DC_BN > n) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = j0 + 8 * (i / 4) + 4 * h + (i & 3);
          if (j < first || j >= n || !((good >> (i / 8)) & 1)) s[i] = -INFINITY;
        }
      }
      float mx = m;
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[i]);
      mx = max_halves(mx);
      const float top = mx == -INFINITY ? 0.f : mx * c, base = top + add;
      // exactly 1 where the maximum stays: m c - top, the rounding of top, would change the sums tile by tile
      const float al = mx == m ? 1.f : exp2_fast(fmaf(m, c, -top));
      float p[16], sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p[i] = exp2_fast(fmaf(s[i], c, -base));
        sum += p[i];
      }
      l = l * al + sum;
      m = mx;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= al;
#pragma unroll
      for (int s2 = 0; s2 < 2; ++s2) {  // the weights as bf16 (attn.hpp: why)
        const uint4 pf = make_uint4(pack2bf(p[8 * s2], p[8 * s2 + 1]), pack2bf(p[8 * s2 + 2], p[8 * s2 + 3]),
                                    pack2bf(p[8 * s2 + 4], p[8 * s2 + 5]), pack2bf(p[8 * s2 + 6], p[8 * s2 + 7]));
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = mfma32x32x16(fo.value(vt, s2, d), pf, o[d]);
      }
      good = good_next;
    }
    l = again ? whole : sum_halves(l);

    // join the waves: [wave][column][channel] fp32 in the ring that no copy fills any more
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __syncthreads();
    if (col < gn) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4*>(js + (wave * 32 + col) * DH + 32 * d + 2 * i + 4 * h) =
              make_float4(o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]);
      if (h == 0) ml_s[wave][col] = make_float2(m, l);
    }
    __syncthreads();
    for (int e = tid; e < gn * (DH / 4); e += 64 * W) {
      const int g = e / (DH / 4), d4 = e % (DH / 4) * 4;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) mx = fmaxf(mx, ml_s[w][g].x);
      const float base = mx == -INFINITY ? 0.f : mx * c;
      float lt = 0.f, part[W];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 x = ml_s[w][g];
        part[w] = exp2_fast(fmaf(x.x, c, -base));
        lt = fmaf(part[w], x.y, lt);
      }
      const float inv = inverse_sum(lt, mx);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {  // the wave's weight in the mean before its values: finite stays finite
        float f = part[w] * inv;
        if (again) f *= exp2_fast(headroom(inverse_sum(ml_s[w][g].y, ml_s[w][g].x)));
        const float4 v = *reinterpret_cast<const float4*>(js + (w * 32 + g) * DH + d4);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      if (again) acc = make_float4(in_range(acc.x), in_range(acc.y), in_range(acc.z), in_range(acc.w));
      if (lt < INFINITY && acc.x * 0.f + acc.y * 0.f + acc.z * 0.f + acc.w * 0.f != 0.f) odd_s = true;
      const int hq = kvh * a.G + g0 + g;
      const long rr = long(seq) * a.Hq + hq;
      if (a.splits > 1) {
        *reinterpret_cast<float4*>(a.part + (split * nrows + rr) * DH + d4) = acc;
        if (d4 == 0)
          *reinterpret_cast<float2*>(a.part + a.splits * nrows * DH + (split * nrows + rr) * 2) =
              make_float2(mx, lt);
      } else {
        *reinterpret_cast<uint2*>(a.O + long(seq) * a.os + hq * DH + d4) =
            make_uint2(pack2bf(acc.x, acc.y), pack2bf(acc.z, acc.w));
        if (a.lse && d4 == 0) a.lse[rr] = log_sum(lt, mx, a.scale);
      }
    }
    if (again) break;
    __syncthreads();
    if (!__builtin_amdgcn_readfirstlane(odd_s)) break;
    again = true;
    whole = l;
    add = headroom(inverse_sum(l, m));
    l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  }
}

// Row of the partial results that the i-th of R rows of workgroup `block` takes, -1 past the last: the
// key head is the fastest index, as in the kernels that wrote them, so that the sums are read on the
// XCD whose L2 they were written through (150 tokens of 32/8 heads after 4000, the whole call:
// 22.6 us, in the order of the tokens 27.0).
template <int R>
__device__ __forceinline__ long join_row(int block, int i, long nrows, int Hq, int Hkv) {
  const uint32_t G = uint32_t(Hq) / uint32_t(Hkv), kvh = uint32_t(block) % uint32_t(Hkv);
  const uint32_t x = uint32_t(block) / uint32_t(Hkv) * R + i, t = x / G;
  const long rr = long(t) * Hq + kvh * G + (x - t * G);
  return rr < nrows ? rr : -1;
}

// Joins the `splits` partial means of each row (token, head), weighted by their share of the row's sum of
// weights, so that no sum of finite values passes fp32; one wave per row, four channels per
// lane, so that a wave has 2 (dh 128) or 4 splits side by side. What it waits for is one round of
// memory: the statistics and the first 8 loads of sums per lane are asked for together (64 splits of 32
// rows: 3.5 us, 15 us with the sums asked for one after the other once the weights are known). Fixed order,
// so the same inputs give the same bits.
template <int DH, int W>
__global__ __launch_bounds__(64 * W) void k_attention_join(const float* part, int splits,
                                                        const int* cu_q, int n_seq, long nrows,
                                                        int Hq, int Hkv, uint16_t* O, long os,
                                                        float* lse, float scale) {
  constexpr int LP = DH / 4, SP = 64 / LP, U = 8;  // lanes per split, splits side by side, loads at once
  const int lane = threadIdx.x & 63, sub = lane / LP, ch = 4 * (lane % LP);
  const long rr = join_row<W>(blockIdx.x, threadIdx.x >> 6, nrows, Hq, Hkv);
  if (rr < 0) return;
  const float* p = part + rr * DH + ch;
  const long step = nrows * DH;
  float2 x = make_float2(-INFINITY, 0.f);
  if (lane < splits)
    x = *reinterpret_cast<const float2*>(part + splits * step + (lane * nrows + rr) * 2);
  float4 v[U];
  const auto load = [&](int s0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int s = s0 + u * SP + sub;
      if (s < splits) v[u] = *reinterpret_cast<const float4*>(p + s * step);
    }
  };
  load(0);
  if (cu_q) {  // a row of no sequence
    const int t = int(rr / Hq);
    if (t < cu_q[0] || t >= cu_q[n_seq]) return;
  }
  const float c = scale * kLog2e;
  float mx = x.x;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) mx = fmaxf(mx, __shfl_xor(mx, d));
  const float base = mx == -INFINITY ? 0.f : mx * c;
  float f = exp2_fast(fmaf(x.x, c, -base)) * x.y, lt = f;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) lt += __shfl_xor(lt, d);
  f *= inverse_sum(lt, mx);
  float acc[4] = {};
  for (int s0 = 0; s0 < splits; s0 += U * SP) {
    if (s0) load(s0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = __shfl(f, (s0 + u * SP + sub) & 63);
      acc[0] = fmaf(w, v[u].x, acc[0]);
      acc[1] = fmaf(w, v[u].y, acc[1]);
      acc[2] = fmaf(w, v[u].z, acc[2]);
      acc[3] = fmaf(w, v[u].w, acc[3]);
    }
  }
#pragma unroll
  for (int d = LP; d < 64; d *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], d);
  if (sub == 0)
    *reinterpret_cast<uint2*>(O + (rr / Hq) * os + (rr % Hq) * DH + ch) =
        make_uint2(pack2bf(acc[0], acc[1]), pack2bf(acc[2], acc[3]));
  if (lse && lane == 0) lse[rr] = log_sum(lt, mx, scale);
}

// The same for up to 8 splits, which is where there are many rows: a row per 32 (dh 128) or 16 lanes, four
// channels each, every lane with all of the row's statistics, so that nothing is exchanged. Against the
// form above, whole calls: 512 tokens after 15872 (16384 rows, 4 splits) 127.5 -> 125.4 us, 1024 after 15360
// 236 -> 231, 300 after 4000 35.4 -> 33.4.
template <int DH>
__global__ __launch_bounds__(256) void k_attention_join_few(const float* part, int splits,
                                                            const int* cu_q, int n_seq, long nrows,
                                                            int Hq, int Hkv, uint16_t* O, long os,
                                                            float* lse, float scale) {
  constexpr int LP = DH / 4, U = 8;
  const int ch = 4 * (threadIdx.x % LP);
  const long rr = join_row<256 / LP>(blockIdx.x, threadIdx.x / LP, nrows, Hq, Hkv);
  if (rr < 0) return;
  const float* p = part + rr * DH + ch;
  const float* ml = part + splits * nrows * DH + rr * 2;
  float2 x[U];
  float4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < splits) x[u] = *reinterpret_cast<const float2*>(ml + u * nrows * 2);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < splits) v[u] = *reinterpret_cast<const float4*>(p + u * nrows * DH);
  if (cu_q) {  // a row of no sequence
    const int t = int(rr / Hq);
    if (t < cu_q[0] || t >= cu_q[n_seq]) return;
  }
  const float c = scale * kLog2e;
  float mx = -INFINITY;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < splits) mx = fmaxf(mx, x[u].x);
  const float base = mx == -INFINITY ? 0.f : mx * c;
  float lt = 0.f, acc[4] = {};
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < splits) {
      x[u].y *= exp2_fast(fmaf(x[u].x, c, -base));
      lt += x[u].y;
    }
  const float inv = inverse_sum(lt, mx);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < splits) {
      const float w = x[u].y * inv;
      acc[0] = fmaf(w, v[u].x, acc[0]);
      acc[1] = fmaf(w, v[u].y, acc[1]);
      acc[2] = fmaf(w, v[u].z, acc[2]);
      acc[3] = fmaf(w, v[u].w, acc[3]);
    }
  *reinterpret_cast<uint2*>(O + (rr / Hq) * os + (rr % Hq) * DH + ch) =
      make_uint2(pack2bf(acc[0], acc[1]), pack2bf(acc[2], acc[3]));
  if (lse && ch == 0) lse[rr] = log_sum(lt, mx, scale);
}

}  // namespace

hipError_t attention_join(const float* part, int splits, const int* cu_q, int n_seq, long nrows,
                          int Hq, int Hkv, int dh, void* O, long os, float* lse, float scale,
                          hipStream_t stream) {
  const int rows = join_rows(splits, nrows, dh);  // per workgroup
  const long per_head = nrows / Hkv;
  const dim3 grid(unsigned((per_head + rows - 1) / rows * Hkv)), block(splits <= 8 ? 256 : 64 * rows);
  const auto k = splits <= 8 ? (dh == 128 ? k_attention_join_few<128> : k_attention_join_few<64>)
                 : rows == 1 ? (dh == 128 ? k_attention_join<128, 1> : k_attention_join<64, 1>)
                             : (dh == 128 ? k_attention_join<128, 4> : k_attention_join<64, 4>);
  hipLaunchKernelGGL(k, grid, block, 0, stream, part, splits, cu_q, n_seq, nrows, Hq, Hkv,
                     static_cast<uint16_t*>(O), os, lse, scale);
  return hipGetLastError();
}

size_t attention_decode_workspace(int n_seq, int max_pages, int page, int Hq, int Hkv, int dh) {
  return decode_workspace(n_seq, max_pages, page, Hq, Hkv, dh);
}

hipError_t attention_decode(const DecodeArgs& a) {
  const int G = a.Hq / a.Hkv;
  const DecodePlan p = decode_plan(a.n_seq, a.max_pages, a.page, a.Hkv, G, a.dh, a.window);
  const DecodeDev d{static_cast<const uint16_t*>(a.Q), a.qs, static_cast<const char*>(a.Kc),
              static_cast<const char*>(a.Vc), static_cast<uint16_t*>(a.O), a.os, a.lse, a.table,
              a.lengths, a.max_pages, __builtin_ctz(unsigned(a.page)), a.n_pages, a.n_seq, a.Hq,
              a.Hkv, G, a.scale, a.window,
              p.splits, static_cast<float*>(a.ws)};
  const dim3 grid(unsigned(a.Hkv) * d.splits * a.n_seq * ((G + 31) / 32));
  if (a.dh == 64)
    hipLaunchKernelGGL((k_attention_decode<64, 4>), grid, dim3(256), 0, a.stream, d);
  else if (p.waves == 4)
    hipLaunchKernelGGL((k_attention_decode<128, 4>), grid, dim3(256), 0, a.stream, d);
  else
    hipLaunchKernelGGL((k_attention_decode<128, 2>), grid, dim3(128), 0, a.stream, d);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || d.splits == 1) return e;
  return attention_join(d.part, d.splits, nullptr, 0, long(a.n_seq) * a.Hq, a.Hq, a.Hkv, a.dh, a.O, a.os, a.lse,
                        a.scale, a.stream);
}

}  // namespace ttt
