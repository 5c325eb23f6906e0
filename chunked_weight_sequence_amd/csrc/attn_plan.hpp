// What the attention calls launch: rules on sizes only, for the host, with both sides measured. No device
// code, so that a host program can ask them too.
#pragma once
#include <cstddef>

namespace ttt {

constexpr int PLAN_TILE = 64, PLAN_MAX_SPLITS = 64;

// What a call launches: rows per workgroup (128 QT) and pieces of the key axis.
struct PackedPlan {
  int qt, tiles, splits, half;
  bool longest;
};
// Keys that an average row sees.
inline long packed_seen(int n_seq, int Nq, long Nk, int window) {
  const long seen = (Nk > Nq / 2 ? Nk - Nq / 2 : Nk) / n_seq;
  return window > 0 && window < seen ? window : seen;
}
// Keys that the last row sees.
inline long packed_keys(int n_seq, long Nk, int window) {
  const long keys = Nk / n_seq;
  return window > 0 && window < keys ? window : keys;
}
// Workgroups that have rows, if the sequences are alike.
inline long packed_wgs(int qt, int n_seq, int Nq, int Hq, int Hkv) {
  const long rows = long(Nq) * (Hq / Hkv), BM = 128 * qt;
  return ((rows + BM - 1) / BM + n_seq - 1) * Hkv;
}
// Pieces that the keys of a row are split into, if row tiles alone leave compute units free: the number that
// makes the longest row's tiles (0.75 us each, 1.5 with 256 rows, 0.5 for heads of 64) and the joining
// (5 us, and the partial sums written and read at 4 TB/s) cost least, each piece at least 256 keys.
// Measured, 32/8 heads of 128: 512 tokens after 15872, 323 us whole, 125 us in 4; 64 tokens after 16000,
// 35 us in 32 pieces, 31 us in 16; 1024 tokens 20 us whole, 35 us in 2; 2048 tokens of 8/4 heads of 64
// 24 us whole, 28 us in 2.
inline int packed_splits(int qt, int n_seq, int Nq, long Nk, int Hq, int Hkv, int dh, int window) {
  const long keys = packed_keys(n_seq, Nk, window);
  // a compute unit each, where a workgroup counts for as much as an average row has of the longest
  const long seen = packed_seen(n_seq, Nq, Nk, window);
  long most = 256 * keys / (packed_wgs(qt, n_seq, Nq, Hq, Hkv) * (seen < 1 ? 1 : seen));
  if (most > keys / 256) most = keys / 256;
  if (most > 64) most = 64;
  const double tiles = keys / 64 * (qt == 2 ? 1.5 : dh == 64 ? 0.5 : 0.75);
  const double join = double(Nq) * Hq * dh * 8 / 4e6;
  int best = 1;
  double cost = tiles;
  for (int n = 2; n <= most; ++n) {
    const double t = tiles / n + 5 + n * join;
    if (t < cost) cost = t, best = n;
  }
  return best;
}
// The form, judged with the pieces that are launched: pieces(qt) of rows by 128 qt, of which 256 only where `wide`.
template <class Pieces>
inline PackedPlan plan_rows(int n_seq, int Nq, long Nk, int Hq, int Hkv, int dh, int window, bool wide, Pieces pieces) {
  // 256 rows share each tile read from LDS, which costs least power (long rows are bound by that), but
  // leave the chip's 256 places unevenly filled and nothing to run while a workgroup starts and ends
  // (14000 clocks; a tile takes 2900). So: rows of at least 2048 keys whose workgroups fill at least 9
  // of 10 places, in pieces of at least 1024, and that are many if their rows differ in length.
  // Measured, 256 rows against 128, 32/8 heads of 128: 16384 tokens 1.76 / 1.87 ms, 512 after 15872 126
  // / 138 us, 256 after 16000 75 / 80 us; but 64 after 16000 37 / 31 us, 200 after 4000 31 / 28 us,
  // 4096 tokens of 16/4 heads 98 / 74 us, 2048 tokens 52 / 44 us, 11 documents in 8192 tokens 110 / 105
  // us, 12000 tokens of 4/1 heads in 2 documents 205 / 153 us. Heads of 64, which the vector unit
  // bounds: 8191 tokens, window 2048, 188 / 145 us.
  PackedPlan p{1, 0, 1, 0, false};
  if (wide && dh == 128 && packed_seen(n_seq, Nq, Nk, window) >= 2048) {
    const long many = pieces(2), wgs = packed_wgs(2, n_seq, Nq, Hq, Hkv), n = wgs * many;
    const long seen = packed_seen(n_seq, Nq, Nk, window);
    if (seen >= 1024 * many && 10 * n >= 9 * 256 * ((n + 255) / 256) &&
        (wgs >= 384 || 4 * packed_keys(n_seq, Nk, window) <= 5 * seen))
      p.qt = 2;
  }
  const long rows = long(Nq) * (Hq / Hkv);
  p.tiles = n_seq == 1 ? int((rows + 128 * p.qt - 1) / (128 * p.qt)) : int(rows / (128 * p.qt)) + n_seq;
  p.splits = pieces(p.qt);
  // Row tiles are taken from the last on, so that the longest rows start first. Where all workgroups
  // start at once, two on a compute unit (three of heads of 64), those past the first 256 come in the
  // opposite order, so that each unit has long and short ones: 2048 tokens of 32/8 heads of 128 44 ->
  // 42 us, 1800 38 -> 35.6, 4000 of 8/4 heads of 64 46 -> 44 us.
  const long wgs = packed_wgs(p.qt, n_seq, Nq, Hq, Hkv) * p.splits;
  // Sequences with most keys first, where workgroups go more than once around the chip and so few times
  // that the last to start counts, and finding the order (30 clocks a sequence in each) is little beside
  // a row's tiles. Ordered / not, means over six draws of lengths: 16/8 heads of 128, 8 .. 14 sequences in
  // 8800 tokens (1100 workgroups) 0.92 .. 0.94, in 16000 (2000) 0.95 .. 0.98; 32/8 heads, 5 .. 14 in 3200 ..
  // 8000 tokens (800 .. 2000) 0.96 .. 1.005, 16 in 4096 0.99; 16/4 of 64 in 12000 (1500) 0.87 .. 0.96. But
  // 5 .. 16 in 512 tokens (under 300) 1.02 .. 1.15, 24 in 4400 tokens (3 tiles a row) 1.10, 16 in 16384 with
  // a window of 512 (4600) 1.06.
  p.longest = n_seq > 1 && n_seq <= 16 && n_seq <= 4 * (packed_keys(n_seq, Nk, window) / PLAN_TILE) &&
              wgs > 512 && wgs <= 3200;
  p.half = p.qt == 1 && wgs > 256 && wgs <= (dh == 64 ? 768 : 512) ? 256 / (Hkv * p.splits) : p.tiles;
  return p;
}
inline PackedPlan packed_plan(int n_seq, int Nq, long Nk, int Hq, int Hkv, int dh, int window) {
  return plan_rows(n_seq, Nq, Nk, Hq, Hkv, dh, window, true,
                   [&](int qt) { return packed_splits(qt, n_seq, Nq, Nk, Hq, Hkv, dh, window); });
}

inline size_t packed_workspace(int n_seq, int Nq, long Nk, int Hq, int Hkv, int dh) {
  // the window is not known here; with one there are no more pieces than without
  const int a = packed_splits(1, n_seq, Nq, Nk, Hq, Hkv, dh, 0);
  const int b = packed_splits(2, n_seq, Nq, Nk, Hq, Hkv, dh, 0);
  const int n = a > b ? a : b;
  return n > 1 ? size_t(n) * Nq * Hq * (dh + 2) * 4 : 0;
}

// New tokens over a paged cache: the rules above with as many keys as the page tables can hold, since only the
// device knows the lengths.
inline long paged_keys(int n_seq, int max_pages, int page) { return long(n_seq) * max_pages * page; }
// Pieces that the keys are split into where there are several sequences: lengths and numbers of rows differ then, so
// a quarter more workgroups than the chip holds at once, twice as many where a sequence has one wave's rows, which HBM
// bounds, and the joining weighs half as much again. Means over three draws of lengths, what is taken (in brackets) and others:
//   few rows, 32/8 heads of 128: 15 single tokens on up to 12000 (8) 75, 5 84, 10 78 us; 16 on up to 30000 (8) 203, 4 236;
//   32 x 2 on up to 8000 (4) 129, 2 138, 6 124. 16/4 heads of 64: 16 x 5 on up to 8000 (18) 25, 12 24, 14 26, 8 25; 16 single
//   on up to 30000 (24) 54, 12 57, 8 62; 15 on up to 12000 (26) 27, 8 29; 4 x 6 on up to 16000 (49) 16.5, 24 18, 12 25
//   more rows, 32/8 heads of 128: 512 tokens and 14 single ones on up to 12000 (3) 162, 2 157, 4 181, whole 243, and of the same sizes to
//   the host 16 x up to 64 on up to 8000 (3) 83, 2 101, 4 78, whole 156; 4 x up to 500 on up to 6000 (whole) 143, 2 137, but
//   4 x 500 on 6000 each (whole) 180, 2 197; 8 x 16 on 4000 (6) 34, 2 41; 2000 tokens and 30 single ones on up to 8000, 16/4 heads
//   of 64, (3) 95, 4 94, whole 115
inline int paged_splits(int qt, int n_seq, int Nq, long Nk, int Hq, int Hkv, int dh, int window) {
  if (n_seq == 1) return packed_splits(qt, n_seq, Nq, Nk, Hq, Hkv, dh, window);
  const long keys = packed_keys(n_seq, Nk, window), wgs = packed_wgs(qt, n_seq, Nq, Hq, Hkv);
  const long places = qt == 2 ? 256 : dh == 64 ? 768 : 512;
  const bool few = long(Nq) * (Hq / Hkv) <= 32L * n_seq;
  long most = ((few ? 2 * places : 5 * places / 4) + wgs / 2) / wgs;
  if (most > keys / 256) most = keys / 256;
  if (most > PLAN_MAX_SPLITS) most = PLAN_MAX_SPLITS;
  const double tiles = keys / 64 * (qt == 2 ? 1.5 : dh == 64 ? 0.5 : 0.75);
  const double join = 1.5 * double(Nq) * Hq * dh * 8 / 4e6;
  int best = 1;
  double cost = tiles;
  for (int n = 2; n <= most; ++n) {
    const double t = tiles / n + 5 + n * join;
    if (t < cost) cost = t, best = n;
  }
  return best;
}
inline PackedPlan paged_plan(int n_seq, int Nq, int max_pages, int page, int Hq, int Hkv, int dh, int window) {
  const long Nk = paged_keys(n_seq, max_pages, page);
  // 256 rows only for sequences that fill several such tiles, and where plan_rows finds that what is launched fills the
  // chip. 256 / 128, each in its best number of pieces, sequences alike and of unlike lengths, 32/8 heads of 128: 2 x 1024
  // tokens on 16000 keys 469 / 477 and 276 / 286 us, 2 x 512 on 12000 192 / 201 and 120 / 123, 4 x 256 on 15744 247 / 267
  // and 141 / 125, 8 x 500 on 15500 934 / 930 and 426 / 401, 4 x 1000 on 8000 462 / 454 and 199 / 182; 2 x 260 on 8000 in the 4
  // pieces that are launched, which 256 rows do not fill, 118 / 103 and 69 / 65. With fewer rows 8 x 200 after 7800 225 / 216,
  // 16 x 60 172 / 156, 15 single tokens on up to 12000 101 / 78, 32 x 2 on up to 8000 160 / 129.
  // One sequence takes them where its rows do not fit in 128, as the sequence's key tiles are then copied once: 40 tokens on
  // 65536 keys 76 / 87 us, 64 86 / 110; but 1 token 58 / 51, 5 on 32768 37 / 31, 32 (128 rows) 44 / 37, on 131072 127 / 126.
  const long rows = long(Nq) * (Hq / Hkv);
  const bool wide = n_seq == 1 ? rows > 128 : rows >= 1024L * n_seq;
  PackedPlan p = plan_rows(n_seq, Nq, Nk, Hq, Hkv, dh, window, wide,
                           [&](int qt) { return paged_splits(qt, n_seq, Nq, Nk, Hq, Hkv, dh, window); });
  if (n_seq > 1) {
    p.half = p.tiles;
    // In pieces, sequences are ordered where a piece has a tile for each of them. Ordered / not, means over three draws of
    // lengths: 16 x up to 64 tokens on up to 8000 85 / 98 us, 16 x up to 16 on 16000 117 / 141, 12 x up to 200 on 9000 127 / 152,
    // 15 single tokens on 12000 76 / 87, a piece of 512 beside 14 single tokens 164 / 166; but 16 x up to 5 on 8000, 16/4
    // heads of 64 (7 tiles a piece), 26.6 / 25.4.
    if (p.splits > 1) p.longest = p.longest && n_seq <= packed_keys(n_seq, Nk, window) / PLAN_TILE / p.splits;
  }
  return p;
}
inline size_t paged_workspace(int n_seq, int Nq, int max_pages, int page, int Hq, int Hkv, int dh) {
  // the window is not known here; with one there are no more pieces than without
  const long Nk = paged_keys(n_seq, max_pages, page);
  const int a = paged_splits(1, n_seq, Nq, Nk, Hq, Hkv, dh, 0), b = paged_splits(2, n_seq, Nq, Nk, Hq, Hkv, dh, 0);
  const int n = a > b ? a : b;
  return n > 1 ? size_t(n) * Nq * Hq * (dh + 2) * 4 : 0;
}

// What a call launches: waves per workgroup and pieces per sequence, from the most that the page
// table can hold, since only the device knows the lengths.
struct DecodePlan {
  int waves, splits;
};
inline DecodePlan decode_plan(int n_seq, int max_pages, int page, int Hkv, int G, int dh, int window) {
  const long wgs = long(n_seq) * Hkv * ((G + 31) / 32);
  long keys = long(max_pages) * page;
  if (window > 0 && window < keys) keys = window;
  // The ring of 4 waves of heads of 128 takes a compute unit's LDS; with 2 waves, one workgroup starts
  // or ends while the other streams, which counts when each unit has several: from 1536 tokens per
  // unit on. 4 / 2 waves, 32/8 heads of 128: 100 x 512 tokens 47 / 39 us, 200 x 500 96 / 91, 64 x
  // 1000 45 / 43, but 1 x 32768 28 / 29, 1 x 4096 8.3 / 9.8.
  const int waves = dh == 128 && wgs * keys >= 256 * 1536 ? 2 : 4;
  // As many pieces as fill the chip, of at least 128 tokens (a tile per wave), and up to four times
  // as many, since lengths differ and the last to end counts, where a piece still has 1024 (heads of
  // 64, whose tiles are half as large: 512). Measured in pieces for four times the chip's workgroups
  // of 4 waves / for once, without the second limit: 16 x 32768 tokens 365 / 374 us, 33 of up to 5000,
  // 16/4 heads of 64, 21 / 33 us, but 64 x 1000 52 / 45 us, 4 x 2000 11.8 / 9.6 us.
  const auto pieces = [&](long want, long least) {
    const long n = (want + wgs - 1) / wgs, most = keys / least;
    return n < most ? n : most;
  };
  const long chip = 1024 / waves;
  const long a = pieces(chip, 128), b = pieces(4 * chip, dh == 128 ? 1024 : 512), n = a > b ? a : b;
  return {waves, int(n < 1 ? 1 : n > PLAN_MAX_SPLITS ? PLAN_MAX_SPLITS : n)};
}

inline size_t decode_workspace(int n_seq, int max_pages, int page, int Hq, int Hkv, int dh) {
  // the window is not known here: without one there are no fewer pieces than with it
  const int ns = decode_plan(n_seq, max_pages, page, Hkv, Hq / Hkv, dh, 0).splits;
  return ns > 1 ? size_t(ns) * n_seq * Hq * (dh + 2) * 4 : 0;
}

// Rows of a workgroup that joins pieces: up to 8 of them by the form without exchanges (1024 / dh); else a
// wave a row, and with few rows one row a workgroup, on as many compute units.
inline int join_rows(int splits, long nrows, int dh) {
  return splits <= 8 ? 1024 / dh : nrows < 1024 ? 1 : 4;
}

}  // namespace ttt
