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
// and sum of a softmax in fp32. While the exponentials of one tile are taken (the vector unit: 760
// clocks per tile and 32 rows), the matrix pipe works on the scores of the next and the values of this
// one (33 clocks per 32x32x16 product: 1056 with heads of 128, 528 with 64). So heads of 128 are bound by
// the matrix pipe, and by power where rows are long (the clock falls to 1.6 .. 2.0 GHz), heads of 64 by
// the vector unit. 32/8 heads of 128: 16384 tokens 1.69 .. 1.88 ms (1170 .. 1300 TFLOP/s over the visible
// pairs; a large matrix product 1350 .. 1550), 11 documents in 8192 tokens 90 .. 118 us by their lengths, 512
// tokens after 15872 122 .. 127 us with the join; 32/32 heads of 64, 8191 tokens, window 2048: 139 .. 154 us.
// A workgroup takes 4 us to its first round (its sequence 0.6, set up 0.6, copies 1.5, queries to registers
// 0.5, first scores 0.9), 1.2 .. 1.5 per tile of 128 rows with two on a unit, and 2 to write its rows.
//
// The paged form is the same kernel with other copies: a wave's 16 rows of a tile lie in one page (a page has at least 16),
// so a tile takes four page numbers, read through the scalar cache a tile ahead. It costs little: 512 tokens after
// 15872, 32/8 heads of 128, 122 .. 132 us with the join (1026 TFLOP/s), 4 pieces of 2000 tokens, 32/32 heads of 64,
// window 2048, 169 .. 186 us. Few rows per key are bound by HBM instead: 16 x 5 tokens on up to 8000, 16/4 heads
// of 64, 21 .. 25 us by the lengths (72 MB, 3.3 TB/s; without the join 4.2); a piece of 512 tokens and 14 single ones on up
// to 12000 take both in turn, 138 .. 172 us by the lengths.
#include <type_traits>

#include "attn.hpp"
#include "attn_plan.hpp"
#include "launch.hpp"

namespace ttt {
namespace {

#define AP_INLINE __attribute__((always_inline))

constexpr int AP_BN = PLAN_TILE;
constexpr float AP_SLACK = 8.f;  // log2

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
  int half;     // pieces of work from here on are taken from the other end (packed_plan)
  bool longest;  // sequences in the order of their keys (packed_plan)
  // paged: K and V are caches [n_pages << psh][Hkv][DH], a sequence has lengths[s] keys
  const int *table, *lengths;
  int max_pages, psh, n_pages;
  float* part;  // splits > 1: [splits][Nq * Hq][dh] means, then [splits][Nq * Hq] (m, l)
};

// The w-th piece of work: a sequence's offsets (clamped to the buffers) and which of its row tiles, its
// last one first.
struct Work {
  int q0, q1, k0, k1, r;  // r < 0: there is no such tile; paged: k0 is 0
  int s;                  // paged: the sequence
};
template <bool PAGED>
__device__ __forceinline__ Work ap_find(const PackedDev& a, int w, int BM, int lane) {
  // of sequences one after the other: s owns the ids [base(s), base(s + 1)), at least as many as it has
  // tiles
  const auto base = [&](int cu, int s) { return int(uint32_t(cu) * uint32_t(a.G) / uint32_t(BM)) + s; };
  const auto clampq = [&](int s) { return min(max(a.cu_q[s], 0), a.Nq); };
  const auto clampk = [&](int s) { return min(max(a.cu_k[s], 0), a.Nk); };
  const auto cached = [&](int s) { return min(max(a.lengths[s], 0), a.max_pages << a.psh); };
  const int tile = a.tiles - 1 - w;
  Work p;
  p.r = -1;
  int at = 0;
  const auto tiles = [&](int lq) {
    return int((uint32_t(max(lq, 0)) * uint32_t(a.G) + uint32_t(BM - 1)) / uint32_t(BM));
  };
  if (a.n_seq == 1) {
    p.q0 = clampq(0);
    p.q1 = clampq(1);
    p.k0 = PAGED ? 0 : clampk(0);
    p.k1 = PAGED ? cached(0) : clampk(1);
    p.r = tiles(p.q1 - p.q0) - 1 - w;
  } else if (a.n_seq < 64) {  // one load for everything: lane s has sequence s
    const int s = min(lane, a.n_seq);
    const int cq = clampq(s), ck = PAGED ? cached(min(lane, a.n_seq - 1)) : clampk(s);
    if (a.longest) {
      // the sequence with most keys first, so that what starts last is short (otherwise the last one first)
      const int cq1 = __builtin_amdgcn_update_dpp(0, cq, 0x130, 0xF, 0xF, true);  // of the lane above
      const int ck1 = __builtin_amdgcn_update_dpp(0, ck, 0x130, 0xF, 0xF, true);
      const int lk = PAGED ? ck : max(ck1 - ck, 0);
      const int n = tiles(cq1 - cq);
      int before = 0;  // row tiles of the sequences that come first
      for (int j = 0; j < a.n_seq; ++j) {
        const int kj = __builtin_amdgcn_readlane(lk, j), nj = __builtin_amdgcn_readlane(n, j);
        before += kj > lk || (kj == lk && j < lane) ? nj : 0;
      }
      const uint64_t on = __ballot(lane < a.n_seq && w >= before && w - before < n);
      if (on) {
        at = __builtin_ctzll(on);
        p.r = __builtin_amdgcn_readlane(n, at) - 1 - (w - __builtin_amdgcn_readlane(before, at));
      }
    } else {
      at = __popcll(__ballot(lane < a.n_seq && base(cq, s) <= tile)) - 1;
      if (at >= 0) p.r = tile - base(__builtin_amdgcn_readlane(cq, at), at);
      else at = 0;
    }
    p.q0 = __builtin_amdgcn_readlane(cq, at);
    p.q1 = __builtin_amdgcn_readlane(cq, at + 1);
    p.k0 = PAGED ? 0 : __builtin_amdgcn_readlane(ck, at);
    p.k1 = __builtin_amdgcn_readlane(ck, PAGED ? at : at + 1);
  } else {  // 64-way search
    int lo = 0, len = a.n_seq;
    bool some = true;
    while (true) {
      const int step = (len + 63) / 64, s = lo + lane * step;
      const bool in = lane * step < len;
      const int n = __popcll(__ballot(in && base(clampq(in ? s : lo), s) <= tile));
      some = n > 0;
      if (some) at = lo + (n - 1) * step;
      if (!some || step == 1) break;
      len = min(step, len - (n - 1) * step);
      lo = at;
    }
    at = __builtin_amdgcn_readfirstlane(at);
    p.q0 = clampq(at);
    p.q1 = clampq(at + 1);
    p.k0 = PAGED ? 0 : clampk(at);
    p.k1 = PAGED ? cached(at) : clampk(at + 1);
    if (some) p.r = tile - base(p.q0, at);
  }
  p.q1 = max(p.q1, p.q0);
  p.k1 = max(p.k1, p.k0);
  p.s = at;
  return p;
}

// S^T tile of 32 keys by 32 queries into ordinary registers, where the exponentials are taken; the
// queries sit in accumulator registers. Inline assembly, because the compiler would put every
// product's result into accumulator registers and copy 64 values a tile. The result may be read a
// whole phase later only (ap_settle).
__device__ __forceinline__ void ap_mma0(f32x16& d, const uint4& k, const bf16x8& q) {
  asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, 0"
      : "=&v"(d) : "v"(__builtin_bit_cast(bf16x8, k)), "a"(q));
}
__device__ __forceinline__ void ap_mma(f32x16& d, const uint4& k, const bf16x8& q) {
  asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0"
      : "+v"(d) : "v"(__builtin_bit_cast(bf16x8, k)), "a"(q));
}
// What follows reads these results of ap_mma: either at least three phases' quarters of products lie
// between (NOPS false), or 16 + 16 wait states, where an 8-pass product needs 11, are put there.
template <bool NOPS, int QT>
__device__ __forceinline__ void ap_settle(f32x16 (&s)[2][QT]) {
  if (NOPS) asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
  for (int b = 0; b < QT; ++b) asm volatile("" : "+v"(s[0][b]), "+v"(s[1][b]));
}
// o *= f in the accumulator registers where the products keep it, behind a branch. Assembly: as an
// ordinary product the compiler copies the accumulator out in every round, before it knows whether it
// has to be scaled.
__device__ __forceinline__ void ap_rescale(f32x16& o, float f) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x = o[i], t;
    asm volatile("v_accvgpr_read_b32 %1, %0\n\tv_mul_f32 %1, %1, %2\n\tv_accvgpr_write_b32 %0, %1"
                 : "+a"(x), "=&v"(t) : "v"(f));
    o[i] = x;
  }
}
// A copy that the compiler leaves where it stands (see ap_hide).
__device__ __forceinline__ void ap_move(f32x16& to, const f32x16& from) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x;
    asm volatile("v_mov_b32 %0, %1" : "=v"(x) : "v"(from[i]));
    to[i] = x;
  }
}
// x = -inf where j > last (or j < first), in place: as an ordinary selection the result would be
// another register, and every tile, masked or not, would be copied to where the masked ones end.
__device__ __forceinline__ void ap_hide_after(float& x, int j, int last) {
  asm volatile("v_cmp_gt_i32 vcc, %1, %2\n\ts_nop 1\n\tv_cndmask_b32 %0, %0, %3, vcc"
               : "+v"(x) : "n"(j), "v"(last), "v"(-INFINITY) : "vcc");
}
__device__ __forceinline__ void ap_hide_before(float& x, int j, int first) {
  asm volatile("v_cmp_lt_i32 vcc, %1, %2\n\ts_nop 1\n\tv_cndmask_b32 %0, %0, %3, vcc"
               : "+v"(x) : "n"(j), "v"(first), "v"(-INFINITY) : "vcc");
}
// Waits until at most N of the wave's LDS reads are under way (they return in order).
template <int N>
__device__ __forceinline__ void ap_wait() { __builtin_amdgcn_s_waitcnt(0xC07F | (N << 8)); }
__device__ __forceinline__ void ap_fence() { __builtin_amdgcn_sched_barrier(0); }

// How the 48 QT steps of a tile's exponentials (14 clocks each) are dealt out over the slots of a
// round: in proportion to what a slot's product (33 clocks) leaves free beside its own issue, operand
// reads and copies. at[k] .. at[k + 1]: slot k's steps (phase A, then the first three quarters of
// phase B); at[0] of them come before the first product, while its operands are on their way from LDS.
template <int KS, int DT, int NI, int QT>
struct ApPlan {
  static constexpr int SA = 2 * QT * KS, SB = 4 * QT * DT, OPS = 48 * QT, FIRST = 3 * QT;
  int at[SA + 3 * SB / 4 + 1];
  // slot of the i-th copy (V, then K)
  static constexpr int copy_slot(int i) { return 4 * (i / 3) + i % 3 + 1; }
  static constexpr int room(int k) {
    const bool reads = k % (2 * QT) == 0;
    int r = k < SA ? (reads ? 14 : 28) : (reads ? 6 : 28);
    for (int i = 0; i < 2 * NI; ++i)
      if (k == copy_slot(i)) r = 8;
    return r;
  }
  constexpr ApPlan() : at() {
    int total = 0, sum = 0;
    for (int k = 0; k < SA + 3 * SB / 4; ++k) total += room(k);
    for (int k = 0; k < SA + 3 * SB / 4; ++k) {
      at[k] = FIRST + (sum * (OPS - FIRST) + total / 2) / total;
      sum += room(k);
    }
    at[SA + 3 * SB / 4] = OPS;
  }
  // the weights of the 16 keys that a quarter of phase B multiplies are ready when it begins
  constexpr bool in_time() const {
    for (int s = 0; s < 4; ++s)
      if (at[SA + s * SB / 4] < 12 * QT * (s + 1)) return false;
    return true;
  }
};

// The sums of 32 channels (32 d ..) of one block of 32 rows again, with care for infinities and NaN: the tiles
// multiply a value that a row does not see by a weight of 0, and 0 times an infinity or a NaN is a NaN. Here
// such values are multiplied as 0, and what the rows that see them get is found by products of 1 and 0:
// which of +inf, -inf and NaN a row sees at all. The maxima and sums of the first pass are right and stay;
// the weights are lower by a power of two (headroom), so that sums of finite values, whose mean is finite, do
// not pass fp32 on the way. By the wave alone, 32 keys [j, j + 32) of [j0, j1) at a
// time: K straight into registers, V by way of its own 32 rows of LDS. 16384 tokens of 32/8 heads of 128
// take 1.7 .. 2.3 ms; with one infinity in the last token 2.9 ms, in the first, which every row of a head sees,
// 9.6 ms, with nothing but NaN in V 44 ms.
// row(j): the row of key j; there(j): whether the 16 keys j .. exist (j a multiple of 16).
template <int DH, int KS, class Row, class There>
__device__ __forceinline__ f32x16 ap_again(int d, const bf16x8 (&qf)[KS], const char* tile,
                                           const uint16_t* K, long ks, const uint16_t* V, long vs, Row row,
                                           There there, int j0, int j1, int lo, int hi, float c, float base,
                                           float inv, int lane) {
  constexpr int RPI = 1024 / (DH * 2);
  asm volatile("" : "+v"(lane));  // nothing of this is worked out before
  const char* const place = tile + FragOff<DH>::channels(lane, d);
  const uint32_t lds = lds_u32(tile);
  const int h = lane >> 5;
  f32x16 o;
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  for (int j = j0; j < j1; j += 32) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the last tile has been read
#pragma unroll 1
    for (int i = 0; i < 32 / RPI; ++i) {
      const int r = i * RPI + lane / (64 / RPI), ch = (lane % (64 / RPI)) ^ vsw<DH>(r);
      dma16_far(V + row(min(j + r, j1 - 1)) * vs + 8 * ch, __builtin_amdgcn_readfirstlane(lds + i * 1024));
    }
    const uint16_t* kp = K + row(min(j + (lane & 31), j1 - 1)) * ks + 8 * h;
    const bool good[2] = {there(j), there(min(j + 16, j1 - 1) & ~15)};
    f32x16 s;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const uint4 kf = *reinterpret_cast<const uint4*>(kp + 16 * k);
      if (k == 0) ap_mma0(s, kf, qf[0]);
      else ap_mma(s, kf, qf[k]);
      if (k % 4 == 3) ap_fence();  // not all loads at once: the registers are the main loop's
    }
    asm volatile("s_nop 15\n\ts_nop 15" : "+v"(s));
    uint32_t pw[8], seen = 0;  // weights as bf16 pairs, as in the main loop; bit i: the row sees its i-th key
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      float p[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = j + 8 * (i / 4) + 4 * h + (i & 3) + e;
        const bool in = key >= lo && key <= hi && key < j1 && good[i / 8];
        p[e] = in ? exp2_fast(fmaf(s[i + e], c, -base) - headroom(inv)) : 0.f;
        seen |= uint32_t(in) << (i + e);
      }
      pw[i / 2] = pack2bf(p[0], p[1]);
    }
    wait_vm<0>();
    ap_fence();
    // +inf, -inf and NaN as 1, 2^8 and 2^16: their sum over 32 keys, exact in fp32, tells which a row sees
    uint32_t code[2][4];
    bool odd = false;
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const uint4 v = FragOff<DH>::value_at(place, st);
      uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        code[st][e] = 0;
#pragma unroll
        for (int half = 0; half < 32; half += 16) {
          const uint32_t y = x[e] >> half & 0xFFFF;
          if ((y & 0x7F80) != 0x7F80) continue;
          odd = true;
          code[st][e] |= uint32_t(y == 0x7F80 ? 0x3F80 : y == 0xFF80 ? 0x4380 : 0x4780) << half;
          x[e] &= 0xFFFF0000u >> half;
        }
      }
      o = mfma32x32x16(make_uint4(x[0], x[1], x[2], x[3]),
                       make_uint4(pw[4 * st], pw[4 * st + 1], pw[4 * st + 2], pw[4 * st + 3]), o);
      ap_fence();
    }
    if (!__any(odd)) continue;
    f32x16 n;
#pragma unroll
    for (int i = 0; i < 16; ++i) n[i] = 0.f;
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      uint32_t one[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t two = seen >> (8 * st + 2 * e) & 3;
        one[e] = ((two & 1) | (two & 2) << 15) * 0x3F80;
      }
      n = mfma32x32x16(make_uint4(code[st][0], code[st][1], code[st][2], code[st][3]),
                       make_uint4(one[0], one[1], one[2], one[3]), n);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = int(n[i]);
      if (k & 0xFF) o[i] += INFINITY;
      if (k & 0xFF00) o[i] -= INFINITY;
      if (k >> 16) o[i] = NAN;
    }
  }
  return o;
}

// The page table through the scalar cache: a vector load would count with the copies in flight.
typedef const __attribute__((address_space(4))) int const_int;

// PAGED: the keys and values of a sequence lie in pages of a cache. The 16 rows of a tile that a wave copies are
// in one page, since pages hold 2^psh >= 16 tokens: what differs is where a copy's base comes from.
template <int DH, int QT, bool PAGED>
__global__ __launch_bounds__(256, QT == 2 ? 1 : 2) void k_attention_packed(PackedDev a) {
  constexpr int BM = 128 * QT, TILE = AP_BN * DH * 2, KS = DH / 16, DT = DH / 32;
  // [stage][K / V]; then, with 256 rows, one region per wave that holds its queries at the start and its
  // results at the end (otherwise they pass through a stage that is not in use)
  constexpr bool OWN = QT == 2;
  __shared__ __align__(1024) char smem[4 * TILE + (OWN ? BM * DH * 2 : 0)];
  char(&sm)[2][2][TILE] = *reinterpret_cast<char(*)[2][2][TILE]>(smem);
  const int kvh = blockIdx.x % a.Hkv;
  const int rest = blockIdx.x / a.Hkv;
  const int split = rest % a.splits;
  const int turn = rest / a.splits;
  // PAGED: the first rows, all there are of a single token, on another SIMD from one piece of work to the next
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(PAGED ? ((tid >> 6) + rest) & 3 : tid >> 6);
  const int h = lane >> 5;

  const Work wk = ap_find<PAGED>(a, turn < a.half ? turn : a.tiles - 1 - (turn - a.half), BM, lane);
  if (wk.r < 0) return;
  const int q0 = wk.q0, k0 = wk.k0, G = a.G;
  const int rows = (wk.q1 - q0) * G, lk = wk.k1 - k0, off = lk - (wk.q1 - q0);
  const int row0 = wk.r * BM;
  if (row0 >= rows) return;
  // Row x of the workgroup is query qa + v / G, head v % G, v = first + x. The quotient in fp32: v is
  // below 2^17, so its error, 2^-22 v / G, is less than the 1 / (2 G) to the next whole number.
  const int qa = row0 / G, first = row0 - qa * G, rows_here = min(BM, rows - row0);
  const float inv_g = 1.f / float(G);
  const auto query = [&](int x) { return int((float(first + x) + 0.5f) * inv_g); };  // less qa
  // element offset of row x from head kvh * G of query qa (one 32 x 32 bit product)
  const auto element = [&](int x, uint32_t stride) {
    return uint64_t(uint32_t(query(x))) * (stride - uint32_t(G * DH)) + uint32_t((first + x) * DH);
  };

  const FragOff<DH> fo(lane);
  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_u32(smem));
  constexpr int WROWS = 32 * QT;                      // rows of a wave
  const int wrow = wave * WROWS;
  char* const mine = smem + (OWN ? 4 * TILE : 2 * TILE) + wrow * DH * 2;  // for the queries
  // the lane's query column of each block: its last and first visible keys
  int hi[QT], lo[QT];
#pragma unroll
  for (int b = 0; b < QT; ++b) {
    const int qi = qa + query(min(wrow + 32 * b + (lane & 31), rows_here - 1));
    hi[b] = qi + off;
    lo[b] = a.window > 0 ? qi + off - a.window + 1 : 0;
  }
  // key tiles of the workgroup, and the wave's own limits
  const int qb = qa + query(rows_here - 1);
  const int kend = min(lk, qb + off + 1);
  const int kbeg = a.window > 0 ? max(0, qa + off - a.window + 1) : 0;
  int t0 = kbeg / AP_BN, t1 = kend > kbeg ? (kend + AP_BN - 1) / AP_BN : t0;
  if (a.splits > 1) {
    const int per = (t1 - t0 + a.splits - 1) / a.splits;
    t0 = min(t0 + split * per, t1);
    t1 = min(t0 + per, t1);
  }
  const int hi_min = qa + query(min(wrow, rows_here - 1)) + off;
  const int lo_max =
      a.window > 0 ? qa + query(min(wrow + WROWS, rows_here) - 1) + off - a.window + 1 : 0;

  // Copies: wave w fills tile rows 64 / 4 w .. in NI instructions of RPI rows. A row past the
  // sequence's last is replaced by that one (and masked). Offsets are 3 KB up, the bases 3 KB down,
  // so that no offset is negative when dma16_at adds its 1024 i.
  constexpr int RPI = 1024 / (DH * 2), NI = AP_BN / RPI / 4, BACK = 3 * 1024;
  const int crow = wave * (AP_BN / 4) + lane / (64 / RPI), cp = lane % (64 / RPI);
  const uint32_t kstep = uint32_t(a.ks) * 2, vstep = uint32_t(a.vs) * 2;
  uint32_t koff[NI], voff[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = crow + i * RPI, from = PAGED ? r - wave * (AP_BN / 4) : r;
    koff[i] = from * kstep + ((cp ^ ksw<DH>(r)) << 4) + (BACK - 1024 * i);
    voff[i] = from * vstep + ((cp ^ vsw<DH>(r)) << 4) + (BACK - 1024 * i);
  }
  const int tlast = t1 - 1, over = (tlast + 1) * AP_BN - lk;  // rows of the last tile that are not there
  auto cut = [&](uint32_t (&off)[NI], uint32_t step) AP_INLINE {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      // PAGED: the wave's rows are counted from the 16 that hold the sequence's last key, if they lie behind it
      const int r = crow + i * RPI - wave * (AP_BN / 4), g = tlast * AP_BN + wave * (AP_BN / 4);
      const uint32_t d = PAGED ? uint32_t(r - (min(g + r, lk - 1) - min(g, (lk - 1) & ~15))) * step
                               : uint32_t(max(crow + i * RPI - (AP_BN - 1 - over), 0)) * step;
      asm volatile("v_sub_u32 %0, %0, %1" : "+v"(off[i]) : "v"(d));
    }
  };
  const uint32_t lds0 = lds + wave * (TILE / 4);
  // the next tiles to copy; K stays at the last one, which is then copied again and not read
  const char* kp = reinterpret_cast<const char*>(a.K + (PAGED ? 0 : (long(k0) + t0 * AP_BN) * a.ks) + kvh * DH) - BACK;
  const char* vp = reinterpret_cast<const char*>(a.V + (PAGED ? 0 : (long(k0) + t0 * AP_BN) * a.vs) + kvh * DH) - BACK;
  const size_t ktile = size_t(AP_BN) * kstep, vtile = size_t(AP_BN) * vstep;
  // PAGED: the pages of a tile's four groups of 16 keys, and from them the wave's base and which groups exist.
  // What a group that does not exist is copied from, the first page, is masked.
  const char *const kc = kp, *const vc = vp;
  const_int* const table =
      (const_int*)(reinterpret_cast<uintptr_t>(a.table) + size_t(PAGED ? wk.s : 0) * a.max_pages * 4);
  struct Pages {
    int p[4], t;
  };
  const auto pages = [&](int t) AP_INLINE {
    Pages x;
    x.t = min(t, t1 - 1);
#pragma unroll
    for (int g = 0; g < 4; ++g)
      x.p[g] = table[__builtin_amdgcn_readfirstlane(min(x.t * AP_BN + 16 * g, (lk - 1) & ~15) >> a.psh)];
    return x;
  };
  const auto exists = [&](int page) AP_INLINE { return uint32_t(page) < uint32_t(a.n_pages); };
  const auto groups = [&](const Pages& x) AP_INLINE {  // bit g: group g exists
    int good = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) good |= int(exists(x.p[g])) << g;
    return good;
  };
  const auto first_row = [&](const Pages& x) AP_INLINE {  // of the wave's group
    const int page = wave == 0 ? x.p[0] : wave == 1 ? x.p[1] : wave == 2 ? x.p[2] : x.p[3];
    const int j = min(x.t * AP_BN + wave * (AP_BN / 4), (lk - 1) & ~15) & ((1 << a.psh) - 1);
    return (long(exists(page) ? page : 0) << a.psh) + j;
  };
  Pages ahead = {};      // of the tile after the one whose K is copied next
  long krow = 0;         // the wave's first row of that tile
  int good0 = 15, good1 = 15;  // groups that exist of the tile whose scores come next, and of the one after it
  auto copy_k = [&](auto i, int buf) AP_INLINE {
    constexpr int I = decltype(i)::value;
    dma16_at<I>(koff[I], kp, lds0 + buf * 2 * TILE);
  };
  auto copy_v = [&](auto i, int buf) AP_INLINE {
    constexpr int I = decltype(i)::value;
    dma16_at<I>(voff[I], vp, lds0 + buf * 2 * TILE + TILE);
  };
  auto each = [&](auto&& f) AP_INLINE {
    f(std::integral_constant<int, 0>());
    f(std::integral_constant<int, 1>());
    if constexpr (NI == 4) {
      f(std::integral_constant<int, 2>());
      f(std::integral_constant<int, 3>());
    }
  };

  // K of tile t + 1 and V of tile t are in LDS when round t begins; what a wave copies for the next one, and from
  // where
  const auto advance = [&](int t) AP_INLINE {
    if (PAGED) {  // K of tile t + 2 (the last one again where there is none) and V of tile t + 1
      vp = vc + krow * vstep;
      krow = first_row(ahead);
      kp = kc + krow * kstep;
      good0 = good1;
      good1 = groups(ahead);
      ahead = pages(t + 3);
    } else {
      vp += vtile;
      if (t + 2 < t1) kp += ktile;
    }
    if (t + 2 >= tlast) {
      if (t + 2 == tlast) cut(koff, kstep);
      if (t + 1 == tlast) cut(voff, vstep);
    }
  };
  const auto begin = [&]() AP_INLINE {
    if (PAGED) {
      const Pages x = pages(t0), y = pages(t0 + 1);
      ahead = pages(t0 + 2);
      good0 = groups(x);
      good1 = groups(y);
      const long row = first_row(x);
      krow = first_row(y);
      kp = kc + row * kstep;
      vp = vc + row * vstep;
    }
    if (t0 == tlast) {
      cut(koff, kstep);
      cut(voff, vstep);
    }
    each([&](auto i) AP_INLINE { copy_k(i, 0); });
  };
  const auto second_k = [&]() AP_INLINE {
    kp = PAGED ? kc + krow * kstep : kp + ktile;
    if (t0 + 1 == tlast) cut(koff, kstep);
    each([&](auto i) AP_INLINE { copy_k(i, 1); });
  };
  // PAGED: a wave without rows copies its part of the tiles and does nothing else, which leaves the matrix pipe
  // to others where workgroups have few rows (in 2 pieces, 512 tokens and 14 single ones on up to 12000 tokens, 32/8
  // heads of 128, 177 -> 164 us; 16 x 5 tokens on up to 8000, 16/4 heads of 64, 59 -> 56).
  if (PAGED && wrow >= rows_here) {
    if (t0 >= t1) return;
    begin();
    each([&](auto i) AP_INLINE { copy_v(i, 0); });
    if (OWN && t0 < tlast) second_k();
    wait_vm<0>();
    asm volatile("s_barrier" ::: "memory");
    if (!OWN && t0 < tlast) second_k();
    for (int t = t0; t + 1 < t1; ++t) {
      asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
      advance(t);
      const int buf = (t - t0) & 1;
      each([&](auto i) AP_INLINE { copy_v(i, buf ^ 1); });
      each([&](auto i) AP_INLINE { copy_k(i, buf); });
    }
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    return;
  }

  f32x16 o[DT][QT];
  // reference maximum, the largest logit that it serves, its exponent, the sum of the weights
  float m[QT], most[QT], base[QT], l[QT][2];
#pragma unroll
  for (int b = 0; b < QT; ++b) {
    m[b] = most[b] = -INFINITY;
    base[b] = 0.f;
    l[b][0] = l[b][1] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][b][i] = 0.f;
  }
  // finite for every scale: a row that has seen nothing yet has most = -inf + slack
  const float c = a.scale * kLog2e, slack = fminf(AP_SLACK / c, 3.4e38f);

  // Masks tile t where an edge crosses the wave's rows, and takes its maxima again.
  auto maxima = [&](const f32x16 (&s)[2][QT], float (&mx)[QT]) AP_INLINE {
#pragma unroll
    for (int b = 0; b < QT; ++b) {
      mx[b] = -INFINITY;
#pragma unroll
      for (int e = 0; e < 32; e += 2)
        mx[b] = fmaxf(fmaxf(mx[b], s[e >> 4][b][e & 15]), s[e >> 4][b][(e & 15) + 1]);
    }
  };
  auto mask = [&](int t, f32x16 (&s)[2][QT], float (&mx)[QT]) AP_INLINE {
    const int kv0 = t * AP_BN;
    const bool after = kv0 + AP_BN - 1 > hi_min, before = kv0 < lo_max, holes = PAGED && good0 != 15;
    if (after || before || holes) {
      if (holes) {
#pragma unroll
        for (int b = 0; b < QT; ++b)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x = s[e >> 4][b][e & 15];
            ap_hide_before(x, 0, good0 >> (2 * (e >> 4) + (e & 15) / 8) & 1 ? 0 : 1);
            s[e >> 4][b][e & 15] = x;
          }
      }
      if (after) {
#pragma unroll
        for (int b = 0; b < QT; ++b)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x = s[e >> 4][b][e & 15];
            ap_hide_after(x, 32 * (e >> 4) + 8 * ((e & 15) / 4) + (e & 3), hi[b] - kv0 - 4 * h);
            s[e >> 4][b][e & 15] = x;
          }
      }
      if (before) {
#pragma unroll
        for (int b = 0; b < QT; ++b)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x = s[e >> 4][b][e & 15];
            ap_hide_before(x, 32 * (e >> 4) + 8 * ((e & 15) / 4) + (e & 3), lo[b] - kv0 - 4 * h);
            s[e >> 4][b][e & 15] = x;
          }
      }
      maxima(s, mx);
    }
  };
  // Moves the reference maximum where a logit exceeds it by 2^AP_SLACK: until then exponentials of
  // up to 2^AP_SLACK are summed as they are, and nothing has to be rescaled.
  auto move = [&](const float (&mx)[QT], int b) AP_INLINE {  // returns the factor of the sums
    const float old = m[b], mn = fmaxf(max_halves(mx[b]), old);
    base[b] = mn == -INFINITY ? 0.f : mn * c;
    m[b] = mn;
    most[b] = mn + slack;
    return exp2_fast(fmaf(old, c, -base[b]));
  };
  auto rebase = [&](const float (&mx)[QT]) AP_INLINE {
    bool grow = false;  // each half of a query's lanes looks at its own keys
#pragma unroll
    for (int b = 0; b < QT; ++b) grow = grow || mx[b] > most[b];
    if (__any(grow)) {
      asm volatile("s_nop 15\n\ts_nop 15");  // the last products have written the accumulator
#pragma unroll
      for (int b = 0; b < QT; ++b) {
        const float al = move(mx, b);
        l[b][0] *= al;
        l[b][1] *= al;
#pragma unroll
        for (int d = 0; d < DT; ++d) ap_rescale(o[d][b], al);
      }
      asm volatile("s_nop 7");  // written before a product reads it
    }
  };

  // the first copies: K of the first tile, the wave's queries (rows as K's: chunk c of row r at slot
  // c ^ ksw(r)), V of the first tile
  bf16x8 qf[QT][KS];
  if (t0 < t1) {
    begin();
    const uint16_t* Qh = a.Q + long(q0 + qa) * a.qs + long(kvh) * G * DH;
    const uint32_t qdst = lds + uint32_t(mine - smem);
#pragma unroll
    for (int i = 0; i < WROWS / RPI; ++i) {
      const int r = i * RPI + lane / (64 / RPI);
      dma16_far(Qh + element(min(wrow + r, rows_here - 1), uint32_t(a.qs)) + 8 * (cp ^ ksw<DH>(r)),
                __builtin_amdgcn_readfirstlane(qdst + i * 1024));
    }
    each([&](auto i) AP_INLINE { copy_v(i, 0); });
    if (OWN && t0 < tlast) {
      second_k();
      wait_vm<2 * NI>();
    } else {
      wait_vm<NI>();
    }
  }
#pragma unroll
  for (int b = 0; b < QT; ++b)
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qf[b][k] = __builtin_bit_cast(bf16x8, fo.key(mine, b, k));
      asm volatile("" : "+a"(qf[b][k]));
    }
  asm volatile("s_nop 7");  // in accumulator registers some wait states before the first product
  ap_fence();
  auto scores = [&](const char* kt, f32x16 (&s)[2][QT]) AP_INLINE {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const uint4 kf[2] = {fo.key(kt, 0, ks), fo.key(kt, 1, ks)};
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int b = 0; b < QT; ++b) {
          if (ks == 0) ap_mma0(s[kb][b], kf[kb], qf[b][0]);
          else ap_mma(s[kb][b], kf[kb], qf[b][ks]);
        }
    }
    ap_fence();
    ap_settle<true>(s);
    ap_fence();
  };
  float mx[QT];
  f32x16 s0[2][QT];
  using B0 = std::integral_constant<int, 0>;
  using B1 = std::integral_constant<int, 1>;
  // One round: the scores of the next tile (phase A) and the products with this tile's values
  // (phase B) keep the matrix pipe busy while the exponentials of this tile, then the maxima of the
  // next, are taken in the gaps. A slot is one product and its share of the other work, held
  // together by fences; operands are read four products ahead. NEXT: there is a next tile, and
  // phase A also copies K of the one after it and V of the next.
  using Plan = ApPlan<KS, DT, NI, QT>;
  static_assert(Plan().in_time(), "a product before its operand");
  constexpr int SA = Plan::SA, SB = Plan::SB;
  auto round = [&](auto next, auto buf, const char* kt, const char* vt, f32x16 (&s)[2][QT],
                   f32x16 (&sn)[2][QT], float (&mx)[QT]) AP_INLINE {
    constexpr bool NEXT = decltype(next)::value;
    constexpr int BUF = decltype(buf)::value;
    constexpr Plan plan{};
    uint32_t pw[2][QT][8];  // the weights as bf16 pairs (attn.hpp: why bf16): [key block][query block]
    float p0 = 0.f, p1 = 0.f;
    // the tile's own sums, added to the row's once: 2^20 equal weights one by one lose 0.4%, and no time is won
    float lt[QT][2] = {};
    auto op = [&](int n) AP_INLINE {  // unit n / 3: two neighbouring weights, in the order phase B takes them
      const int u = n / 3, st = u / (4 * QT), kb = st >> 1, b = (u >> 2) % QT, i = 8 * (st & 1) + 2 * (u & 3);
      if (n % 3 == 0) p0 = exp2_fast(fmaf(s[kb][b][i], c, -base[b]));
      if (n % 3 == 1) p1 = exp2_fast(fmaf(s[kb][b][i + 1], c, -base[b]));
      if (n % 3 == 2) {
        pw[kb][b][i / 2] = pack2bf(p0, p1);
        lt[b][0] += p0;
        lt[b][1] += p1;
        asm volatile("" : "+v"(lt[b][0]), "+v"(lt[b][1]));  // here, not behind the round
        if (st == 3 && (u & 3) == 3) {
          l[b][0] += lt[b][0];
          l[b][1] += lt[b][1];
        }
      }
    };
    uint4 kf[2][2], vf[2][2];
    if (NEXT) {
      kf[0][0] = fo.key(kt, 0, 0);
      kf[0][1] = fo.key(kt, 1, 0);
      ap_fence();
    } else {
      vf[0][0] = fo.value(vt, 0, 0);
      vf[0][1] = fo.value(vt, 0, 1);
    }
#pragma unroll
    for (int n = 0; n < (NEXT ? plan.at[0] : plan.at[SA]); ++n) op(n);
    if (NEXT) {
#pragma unroll
      for (int k = 0; k < SA; ++k) {
        const int ks = k / (2 * QT), kb = (k / QT) & 1, b = k % QT;
        ap_fence();
        if (k % (2 * QT) == 0) {
          if (ks + 1 < KS) {
            kf[(ks + 1) & 1][0] = fo.key(kt, 0, ks + 1);
            kf[(ks + 1) & 1][1] = fo.key(kt, 1, ks + 1);
            ap_wait<2>();
          } else {
            vf[0][0] = fo.value(vt, 0, 0);
            vf[0][1] = fo.value(vt, 0, 1);
            ap_wait<4>();
          }
          ap_fence();
        }
        if (ks == 0) ap_mma0(sn[kb][b], kf[0][kb], qf[b][0]);
        else ap_mma(sn[kb][b], kf[ks & 1][kb], qf[b][ks]);
        each([&](auto i) AP_INLINE {
          if (k == Plan::copy_slot(decltype(i)::value)) copy_v(i, BUF ^ 1);
          if (k == Plan::copy_slot(NI + decltype(i)::value)) copy_k(i, BUF);
        });
#pragma unroll
        for (int n = plan.at[k]; n < plan.at[k + 1]; ++n) op(n);
      }
    }
    float m2[QT];
#pragma unroll
    for (int b = 0; b < QT; ++b) m2[b] = -INFINITY;
#pragma unroll
    for (int k = 0; k < SB; ++k) {
      constexpr int PW = SB / 4, SE = 3 * PW;  // slots per 16 keys; slots with exponentials
      const int st = k / PW, d = (k % PW) / QT, b = k % QT, pr = k / (2 * QT);
      ap_fence();
      if (k % (2 * QT) == 0) {
        if (pr + 1 < SB / (2 * QT)) {
          const int st1 = (k + 2 * QT) / PW, d1 = ((k + 2 * QT) % PW) / QT;
          vf[(pr + 1) & 1][0] = fo.value(vt, st1, d1);
          vf[(pr + 1) & 1][1] = fo.value(vt, st1, d1 + 1);
          ap_wait<4>();
        } else {
          ap_wait<0>();
        }
        ap_fence();
      }
      if (NEXT && k == SE) {
        ap_settle<false>(sn);
        ap_fence();
      }
      const uint32_t* w = &pw[st >> 1][b][4 * (st & 1)];
      o[d][b] = mfma32x32x16(vf[pr & 1][d & 1], make_uint4(w[0], w[1], w[2], w[3]), o[d][b]);
      if (k < SE) {
#pragma unroll
        for (int n = plan.at[SA + k]; n < plan.at[SA + k + 1]; ++n) op(n);
      } else if (NEXT) {
        constexpr int PER = 32 * QT / PW;  // values of the next scores per slot
        const int e0 = (k - SE) * PER, q = e0 >> 5;
#pragma unroll
        for (int e = e0; e < e0 + PER; e += 2)
          m2[q] = fmaxf(fmaxf(m2[q], sn[(e >> 4) & 1][q][e & 15]), sn[(e >> 4) & 1][q][(e & 15) + 1]);
        asm volatile("" : "+v"(m2[q]));  // here, not behind the phase
      }
    }
    ap_fence();
#pragma unroll
    for (int b = 0; b < QT; ++b) mx[b] = m2[b];
  };

  f32x16 s1[2][QT];
  auto step = [&](int t, auto buf, f32x16 (&s)[2][QT], f32x16 (&sn)[2][QT]) AP_INLINE {
    constexpr int B = decltype(buf)::value;
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    advance(t);
    round(std::true_type(), buf, &sm[B ^ 1][0][0], &sm[B][1][0], s, sn, mx);
    mask(t + 1, sn, mx);
    rebase(mx);
  };
  if (t0 < t1) {
    // every wave's part of the first K tile is there, every wave has its queries
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (!OWN && t0 < tlast) second_k();
    scores(&sm[0][0][0], s0);
    maxima(s0, mx);
    mask(t0, s0, mx);
#pragma unroll
    for (int b = 0; b < QT; ++b) move(mx, b);
  }
  for (int t = t0; t + 1 < t1; t += 2) {
    step(t, B0(), s0, s1);
    if (t + 2 < t1) {
      step(t + 1, B1(), s1, s0);
    } else {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int b = 0; b < QT; ++b) ap_move(s0[kb][b], s1[kb][b]);
    }
  }
  if (t0 < t1) {  // the last tile
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const char* vt = &sm[(t1 - 1 - t0) & 1][1][0];
    round(std::false_type(), B0(), vt, vt, s0, s1, mx);
  }

  // Results. Partial ones go out as they are; others by way of LDS, in whole rows: chunk c (16 bytes)
  // of a row at slot c ^ (row % (chunks of a row)).
  constexpr int CH = DH / 8;
  int ln = threadIdx.x & 63;
  asm volatile("" : "+v"(ln));  // what follows from it is computed here, not kept through the loop
  char* const out = OWN ? mine : smem + (((t1 - t0) & 1) ? 2 * TILE : 0) + wrow * DH * 2;
#pragma unroll
  for (int b = 0; b < QT; ++b) {
    const float lt = sum_halves(l[b][0] + l[b][1]);
    float inv = inverse_sum(lt, m[b]), zero = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) zero = fmaf(o[d][b][i], 0.f, zero);
    if (__any(zero != 0.f && lt == lt)) {  // not finite, although the weights are
      // Channels by 32, and only those with such a sum: an infinity or NaN in a tile reaches the sums of its
      // channel in all 32 rows, and weights rounded at another maximum change the last bits of the other 31.
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 16; ++i) odd = odd || !(fabsf(o[d][b][i]) < INFINITY);
        float f = inv;
        if (__any(odd && lt == lt)) {
          const auto row = [&](int j) AP_INLINE {
            if (!PAGED) return long(j);
            const int page = a.table[size_t(wk.s) * a.max_pages + (j >> a.psh)];
            return (long(exists(page) ? page : 0) << a.psh) + (j & ((1 << a.psh) - 1));
          };
          const auto there = [&](int j) AP_INLINE {
            return !PAGED || exists(a.table[size_t(wk.s) * a.max_pages + (j >> a.psh)]);
          };
          o[d][b] = ap_again<DH>(d, qf[b], out + 32 * b * DH * 2, a.K + long(k0) * a.ks + kvh * DH, a.ks,
                                 a.V + long(k0) * a.vs + kvh * DH, a.vs, row, there, t0 * AP_BN,
                                 min(t1 * AP_BN, lk), lo[b], hi[b], c, base[b], inv, ln);
          f *= exp2_fast(headroom(inv));
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][b][i] = in_range(o[d][b][i] * f);
      }
      inv = 1.f;
    }
    const int r = 32 * b + (ln & 31), x = wrow + r, qi = query(x);
    const bool on = x < rows_here;
    const long rr = long(q0 + qa + qi) * a.Hq + kvh * G + first + x - qi * G;
    if (a.splits > 1) {
      if (!on) continue;
      const long n = long(a.Nq) * a.Hq;
      float* po = a.part + (long(split) * n + rr) * DH + 4 * (ln >> 5);
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4*>(po + 32 * d + 2 * i) =
              make_float4(o[d][b][i] * inv, o[d][b][i + 1] * inv, o[d][b][i + 2] * inv,
                          o[d][b][i + 3] * inv);
      if (ln < 32) {
        float* ml = a.part + long(a.splits) * n * DH + (long(split) * n + rr) * 2;
        *reinterpret_cast<float2*>(ml) = make_float2(m[b], lt);
      }
      continue;
    }
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<uint2*>(out + r * DH * 2 + (((4 * d + i / 4) ^ (r % CH)) << 4) + 8 * (ln >> 5)) =
            make_uint2(pack2bf(o[d][b][i] * inv, o[d][b][i + 1] * inv),
                       pack2bf(o[d][b][i + 2] * inv, o[d][b][i + 3] * inv));
    if (a.lse && ln < 32 && on) a.lse[rr] = log_sum(lt, m[b], a.scale);
  }
  if (a.splits == 1) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    uint16_t* Oh = a.O + long(q0 + qa) * a.os + long(kvh) * G * DH;
#pragma unroll
    for (int i = 0; i < WROWS / RPI; ++i) {
      const int r = i * RPI + ln / (64 / RPI), x = wrow + r;
      const uint4 v = *reinterpret_cast<const uint4*>(out + r * DH * 2 + ((ln % CH ^ (r % CH)) << 4));
      if (x < rows_here) *reinterpret_cast<uint4*>(Oh + element(x, uint32_t(a.os)) + 8 * (ln % CH)) = v;
    }
  }
}

}  // namespace

size_t attention_packed_workspace(int n_seq, int Nq, int Nk, int Hq, int Hkv, int dh) {
  return packed_workspace(n_seq, Nq, Nk, Hq, Hkv, dh);
}

namespace {

template <bool PAGED>
hipError_t ap_launch(const PackedArgs& a, const PackedPlan& p, const PackedDev& d) {
  const dim3 grid(unsigned(p.tiles) * a.Hkv * p.splits);
  if (p.qt == 2)
    hipLaunchKernelGGL((k_attention_packed<128, 2, PAGED>), grid, dim3(256), 0, a.stream, d);
  else if (a.dh == 128)
    hipLaunchKernelGGL((k_attention_packed<128, 1, PAGED>), grid, dim3(256), 0, a.stream, d);
  else
    hipLaunchKernelGGL((k_attention_packed<64, 1, PAGED>), grid, dim3(256), 0, a.stream, d);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  return attention_join(d.part, p.splits, a.cu_q, a.n_seq, long(a.Nq) * a.Hq, a.Hq, a.Hkv, a.dh, a.O, a.os,
                        a.lse, a.scale, a.stream);
}

PackedDev ap_device(const PackedArgs& a, const PackedPlan& p) {
  return {static_cast<const uint16_t*>(a.Q), static_cast<const uint16_t*>(a.K), static_cast<const uint16_t*>(a.V),
          a.qs, a.ks, a.vs, static_cast<uint16_t*>(a.O), a.os, a.lse, a.cu_q, a.cu_k, a.n_seq, a.Nq, a.Nk, a.Hq,
          a.Hkv, a.Hq / a.Hkv, a.scale, a.window, p.tiles, p.splits, p.half, p.longest, nullptr, nullptr, 0, 0, 0,
          static_cast<float*>(a.ws)};
}

}  // namespace

hipError_t attention_packed(const PackedArgs& a) {
  const PackedPlan p = packed_plan(a.n_seq, a.Nq, a.Nk, a.Hq, a.Hkv, a.dh, a.window);
  return ap_launch<false>(a, p, ap_device(a, p));
}

size_t attention_paged_workspace(int n_seq, int Nq, int max_pages, int page, int Hq, int Hkv, int dh) {
  return paged_workspace(n_seq, Nq, max_pages, page, Hq, Hkv, dh);
}

hipError_t attention_paged(const PackedArgs& a, const Paged& g) {
  const PackedPlan p = paged_plan(a.n_seq, a.Nq, g.max_pages, g.page, a.Hq, a.Hkv, a.dh, a.window);
  PackedDev d = ap_device(a, p);
  d.table = g.table;
  d.lengths = g.lengths;
  d.max_pages = g.max_pages;
  d.psh = __builtin_ctz(unsigned(g.page));
  d.n_pages = g.n_pages;
  return ap_launch<true>(a, p, d);
}

}  // namespace ttt
