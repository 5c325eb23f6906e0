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
inline long packed_seen(int n_seq, int Nq, int Nk, int window) {
  const long seen = (Nk > Nq / 2 ? Nk - Nq / 2 : Nk) / n_seq;
  return window > 0 && window < seen ? window : seen;
}
// Keys that the last row sees.
inline long packed_keys(int n_seq, int Nk, int window) {
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
inline int packed_splits(int qt, int n_seq, int Nq, int Nk, int Hq, int Hkv, int dh, int window) {
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
inline PackedPlan packed_plan(int n_seq, int Nq, int Nk, int Hq, int Hkv, int dh, int window) {
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
  if (dh == 128 && packed_seen(n_seq, Nq, Nk, window) >= 2048) {
    const int pieces = packed_splits(2, n_seq, Nq, Nk, Hq, Hkv, dh, window);
    const long wgs = packed_wgs(2, n_seq, Nq, Hq, Hkv), n = wgs * pieces;
    const long seen = packed_seen(n_seq, Nq, Nk, window);
    if (seen >= 1024 * pieces && 10 * n >= 9 * 256 * ((n + 255) / 256) &&
        (wgs >= 384 || 4 * packed_keys(n_seq, Nk, window) <= 5 * seen))
      p.qt = 2;
  }
  const long rows = long(Nq) * (Hq / Hkv);
  p.tiles = n_seq == 1 ? int((rows + 128 * p.qt - 1) / (128 * p.qt)) : int(rows / (128 * p.qt)) + n_seq;
  p.splits = packed_splits(p.qt, n_seq, Nq, Nk, Hq, Hkv, dh, window);
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

inline size_t packed_workspace(int n_seq, int Nq, int Nk, int Hq, int Hkv, int dh) {
  // the window is not known here; with one there are no more pieces than without
  const int a = packed_splits(1, n_seq, Nq, Nk, Hq, Hkv, dh, 0);
  const int b = packed_splits(2, n_seq, Nq, Nk, Hq, Hkv, dh, 0);
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
