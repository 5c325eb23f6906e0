// C ABI of libttt_mi355x: host-side validation, kernel selection and launch on the caller's
// stream. Every check runs before anything is enqueued, so a rejected call touches neither the
// device nor any output. The library never allocates device memory and never synchronises
// (except ttt_chunk_scan_profile, which is documented to).
#include <cmath>
#include <math.h>
#include <stdint.h>

#include "../../include/ttt_mi355x.h"
#include "launch.hpp"

#define TTT_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
  const void* p;
  size_t bytes;
};

bool overlap(Range a, Range b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

bool valid_dtype(int d) { return d == TTT_F32 || d == TTT_BF16; }
size_t dsize(int d) { return d == TTT_BF16 ? 2 : 4; }

// `segments`: a bf16 workspace smaller than the full need is accepted here (the caller then
// runs the scan in segments, see scan_run); the range checked for overlaps is the one given.
ttt_status scan_check(const void* Z, const void* Vhat, ttt_dtype in_dtype, const float* W0,
                      int w0_shared, void* O, ttt_dtype out_dtype, float* W_final, int B, int T,
                      int d_ff, int d_model, int chunk, float eta, void* ws, size_t ws_bytes,
                      size_t* need, bool segments = false) {
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype)) return TTT_E_DTYPE;
  if (!Z || !Vhat || !W0 || !O) return TTT_E_NULL;
  if (B < 1 || T < 1 || chunk < 1 || d_ff < 16 || d_model < 16) return TTT_E_SHAPE;
  if (d_ff % 16 || d_model % 16) return TTT_E_SHAPE;
  if (T > (1 << 26) || d_ff > (1 << 20) || d_model > (1 << 20) || B > 65535) return TTT_E_SHAPE;
  if (!isfinite(eta)) return TTT_E_SHAPE;
  // The bf16 path carries the state as W / eta in the matrix-core accumulator, so a nonzero eta
  // must keep that quotient in fp32 range.
  if (in_dtype == TTT_BF16 && eta != 0.f && !(fabsf(eta) >= 1e-18f && fabsf(eta) <= 1e18f))
    return TTT_E_UNSUPPORTED;
  if (!aligned16(Z) || !aligned16(Vhat) || !aligned16(W0) || !aligned16(O) ||
      !aligned16(W_final) || !aligned16(ws))
    return TTT_E_ALIGN;
  const size_t isz = dsize(in_dtype), osz = dsize(out_dtype);
  const size_t DF = size_t(d_model) * d_ff;
  const Range rz{Z, size_t(B) * T * d_ff * isz}, rv{Vhat, size_t(B) * T * d_model * isz};
  const Range rw0{W0, (w0_shared ? 1 : size_t(B)) * DF * 4};
  const Range ro{O, size_t(B) * T * d_model * osz};
  const Range rwf{W_final, W_final ? size_t(B) * DF * 4 : 0};
  *need = in_dtype == TTT_BF16 ? ttt::scan_mfma_workspace(B, T, d_ff, d_model, chunk)
                               : ttt::scan_simt_workspace(B, T, d_ff, d_model, chunk);
  const bool seg = segments && in_dtype == TTT_BF16 && ws_bytes < *need;
  const Range rws{ws, seg ? ws_bytes : *need};
  if (overlap(ro, rz) || overlap(ro, rv) || overlap(ro, rw0) || overlap(ro, rwf))
    return TTT_E_ALIAS;
  if (overlap(rwf, rz) || overlap(rwf, rv)) return TTT_E_ALIAS;
  if (W_final && overlap(rwf, rw0)) {
    const bool inplace = static_cast<const void*>(W_final) == static_cast<const void*>(W0) &&
                         (!w0_shared || B == 1);
    if (!inplace) return TTT_E_ALIAS;
  }
  if (*need > 0) {
    if (!ws || (!seg && ws_bytes < *need)) return TTT_E_WORKSPACE;
    if (overlap(rws, rz) || overlap(rws, rv) || overlap(rws, rw0) || overlap(rws, ro) ||
        overlap(rws, rwf))
      return TTT_E_ALIAS;
  }
  return TTT_OK;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Segments of the bf16 scan for a workspace smaller than the whole sequence needs: the longest
// run of whole groups (Ts tokens) whose own workspace, plus an fp32 state buffer of
// B x d_model x d_ff when the caller gives no W_final to carry the state in, fits.
struct SegPlan {
  int Ts = 0;
  size_t seg_bytes = 0, state_off = 0;
};
bool seg_plan(int B, int T, int F, int D, int C, bool need_state, size_t ws_bytes, SegPlan* sp) {
  const int G = ttt::scan_mfma_group(B, T, F, D, C);
  const int n_g = (T + G - 1) / G;
  const size_t state = need_state ? align256(size_t(B) * D * F * 4) : 0;
  for (int m = n_g - 1; m >= 1; --m) {
    const size_t wsb = align256(ttt::scan_mfma_workspace(B, m * G, F, D, C));
    if (wsb + state <= ws_bytes) {
      sp->Ts = m * G;
      sp->seg_bytes = wsb;
      sp->state_off = wsb;
      return true;
    }
  }
  return false;
}

size_t scan_min_workspace(int B, int T, int F, int D, int C) {
  const int G = ttt::scan_mfma_group(B, T, F, D, C);
  const size_t full = ttt::scan_mfma_workspace(B, T, F, D, C);
  if (G >= T) return full;
  const size_t one = align256(ttt::scan_mfma_workspace(B, G, F, D, C)) +
                     align256(size_t(B) * D * F * 4);
  return one < full ? one : full;
}

ttt_status scan_run(const void* Z, const void* Vhat, ttt_dtype in_dtype, const float* W0,
                    int w0_shared, void* O, ttt_dtype out_dtype, float* W_final, int B, int T,
                    int d_ff, int d_model, int chunk, float eta, void* ws, size_t ws_bytes,
                    hipStream_t stream, ttt::PhaseClock* clk) {
  size_t need = 0;
  const ttt_status st = scan_check(Z, Vhat, in_dtype, W0, w0_shared, O, out_dtype, W_final, B, T,
                                   d_ff, d_model, chunk, eta, ws, ws_bytes, &need, true);
  if (st != TTT_OK) return st;
  if (in_dtype == TTT_BF16 && ws_bytes < need) {
    // Workspace below the whole sequence's need: the scan runs over segments of whole groups,
    // each resuming from the state the previous one ended with (W0 of segment s + 1 = W_final
    // of segment s; with C dividing every segment start this is the same scan, up to the
    // rounding of the state handed across).
    SegPlan sp;
    if (!seg_plan(B, T, d_ff, d_model, chunk, W_final == nullptr, ws_bytes, &sp))
      return TTT_E_WORKSPACE;
    float* state = W_final ? W_final : reinterpret_cast<float*>(static_cast<char*>(ws) + sp.state_off);
    const size_t isz = dsize(in_dtype), osz = dsize(out_dtype);
    (void)hipGetLastError();
    for (int t0 = 0; t0 < T; t0 += sp.Ts) {
      const int Tn = T - t0 < sp.Ts ? T - t0 : sp.Ts;
      const bool first = t0 == 0, last = t0 + Tn >= T;
      ttt::ScanArgs a{static_cast<const char*>(Z) + size_t(t0) * d_ff * isz,
                      static_cast<const char*>(Vhat) + size_t(t0) * d_model * isz, true,
                      first ? W0 : state, first ? (w0_shared != 0 || B == 1) : B == 1,
                      static_cast<char*>(O) + size_t(t0) * d_model * osz, out_dtype == TTT_BF16,
                      last ? W_final : state, B, Tn, d_ff, d_model, chunk, eta, ws, sp.seg_bytes,
                      stream};
      a.T_stride = T;
      if (ttt::scan_mfma(a, clk) != hipSuccess) return TTT_E_LAUNCH;
    }
    return TTT_OK;
  }
  ttt::ScanArgs a{Z, Vhat, in_dtype == TTT_BF16, W0, w0_shared != 0 || B == 1, O,
                  out_dtype == TTT_BF16, W_final, B, T, d_ff, d_model, chunk, eta, ws,
                  ws_bytes, stream};
  (void)hipGetLastError();  // clear any stale error so it is not attributed to this call
  const hipError_t e = a.in_bf16 ? ttt::scan_mfma(a, clk) : ttt::scan_simt(a, clk);
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

}  // namespace

TTT_EXPORT ttt_status ttt_chunk_scan(const void* Z, const void* Vhat, ttt_dtype in_dtype,
                                     const float* W0, int w0_shared, void* O,
                                     ttt_dtype out_dtype, float* W_final, int B, int T, int d_ff,
                                     int d_model, int chunk, float eta, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
  return scan_run(Z, Vhat, in_dtype, W0, w0_shared, O, out_dtype, W_final, B, T, d_ff, d_model,
                  chunk, eta, workspace, workspace_bytes, stream, nullptr);
}

TTT_EXPORT ttt_status ttt_chunk_scan_noalloc(const void* Z, const void* Vhat, ttt_dtype in_dtype,
                                             const float* W0, int w0_shared, void* O,
                                             ttt_dtype out_dtype, float* W_final, int B, int T,
                                             int d_ff, int d_model, int chunk, float eta,
                                             hipStream_t stream) {
  // host-only checks first (a size beyond the static scratch is refused before any HIP call)
  size_t need = 0;
  const ttt_status st = scan_check(Z, Vhat, in_dtype, W0, w0_shared, O, out_dtype, W_final, B, T,
                                   d_ff, d_model, chunk, eta, nullptr, 0, &need);
  if (st != TTT_OK && st != TTT_E_WORKSPACE) return st;
  if (need > TTT_SCAN_SCRATCH_BYTES) {
    // too large for one pass in the scratch: segments of whole groups, if one fits
    SegPlan sp;
    if (in_dtype != TTT_BF16 || !seg_plan(B, T, d_ff, d_model, chunk, W_final == nullptr,
                                          TTT_SCAN_SCRATCH_BYTES, &sp))
      return TTT_E_WORKSPACE;
  }
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return TTT_E_LAUNCH;
  if (stream) {
    int sdev = -1;
    if (hipStreamGetDevice(stream, &sdev) != hipSuccess) return TTT_E_LAUNCH;
    if (sdev != dev) return TTT_E_UNSUPPORTED;
  }
  void* ws = nullptr;
  if (need > 0 && ttt::scan_scratch(dev, &ws) != hipSuccess) return TTT_E_LAUNCH;
  return scan_run(Z, Vhat, in_dtype, W0, w0_shared, O, out_dtype, W_final, B, T, d_ff, d_model,
                  chunk, eta, ws, need > 0 ? size_t(TTT_SCAN_SCRATCH_BYTES) : 0, stream, nullptr);
}

TTT_EXPORT size_t ttt_chunk_scan_workspace(int B, int T, int d_ff, int d_model, int chunk,
                                           ttt_dtype in_dtype) {
  if (!valid_dtype(in_dtype) || B < 1 || T < 1 || chunk < 1 || d_ff < 16 || d_model < 16 ||
      d_ff % 16 || d_model % 16 || T > (1 << 26) || d_ff > (1 << 20) || d_model > (1 << 20) ||
      B > 65535)
    return 0;
  return in_dtype == TTT_BF16 ? ttt::scan_mfma_workspace(B, T, d_ff, d_model, chunk)
                              : ttt::scan_simt_workspace(B, T, d_ff, d_model, chunk);
}

TTT_EXPORT ttt_status ttt_chunk_scan_profile(const void* Z, const void* Vhat, ttt_dtype in_dtype,
                                             const float* W0, int w0_shared, void* O,
                                             ttt_dtype out_dtype, float* W_final, int B, int T,
                                             int d_ff, int d_model, int chunk, float eta,
                                             void* workspace, size_t workspace_bytes,
                                             hipStream_t stream, float* phase_ms,
                                             int* phase_launches) {
  ttt::PhaseClock clk;
  clk.stream = stream;
  const ttt_status st = scan_run(Z, Vhat, in_dtype, W0, w0_shared, O, out_dtype, W_final, B, T,
                                 d_ff, d_model, chunk, eta, workspace, workspace_bytes, stream,
                                 &clk);
  const hipError_t e = clk.finish(phase_ms, phase_launches);
  if (st != TTT_OK) return st;
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

TTT_EXPORT size_t ttt_chunk_scan_workspace_min(int B, int T, int d_ff, int d_model, int chunk,
                                               ttt_dtype in_dtype) {
  const size_t full = ttt_chunk_scan_workspace(B, T, d_ff, d_model, chunk, in_dtype);
  if (full == 0 || in_dtype != TTT_BF16) return full;
  return scan_min_workspace(B, T, d_ff, d_model, chunk);
}

TTT_EXPORT ttt_status ttt_chunk_scan_handover_timeouts(int B, int T, int d_ff, int d_model,
                                                       int chunk, ttt_dtype in_dtype,
                                                       const void* workspace,
                                                       size_t workspace_bytes, unsigned* count,
                                                       hipStream_t stream) {
  if (!valid_dtype(in_dtype)) return TTT_E_DTYPE;
  if (!count) return TTT_E_NULL;
  const size_t need = ttt_chunk_scan_workspace(B, T, d_ff, d_model, chunk, in_dtype);
  if (need == 0 && in_dtype == TTT_BF16) return TTT_E_SHAPE;
  if (!aligned16(count) || !aligned16(workspace)) return TTT_E_ALIGN;
  const void* src = nullptr;
  if (in_dtype == TTT_BF16) {
    if (!workspace || workspace_bytes < need) return TTT_E_WORKSPACE;
    src = static_cast<const char*>(workspace) +
          ttt::scan_mfma_timeout_word(B, T, d_ff, d_model, chunk);
  }
  if (overlap(Range{count, 4}, Range{workspace, need})) return TTT_E_ALIAS;
  (void)hipGetLastError();
  return ttt::scan_mfma_copy_word(src, count, stream) == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

TTT_EXPORT ttt_status ttt_scan_test_overrides(int group_tokens, int token_split,
                                              int spin_limit) {
  ttt::scan_mfma_test_overrides(group_tokens, token_split, spin_limit);
  return TTT_OK;
}

namespace {
bool clip_on(float tau) { return tau > 0.f && std::isfinite(tau); }

// Workspace of ttt_chunk_scan_docs: the scan's own, then (clipping) the scaled targets, the norm
// slots and the factors.
size_t docs_workspace(int B, int T, int d_ff, int d_model, int chunk, ttt_dtype in_dtype,
                      float tau, size_t* scan_part) {
  const size_t sc = in_dtype == TTT_BF16 ? ttt::scan_mfma_workspace(B, T, d_ff, d_model, chunk)
                                         : ttt::scan_simt_workspace(B, T, d_ff, d_model, chunk);
  *scan_part = (sc + 255) & ~size_t(255);
  return *scan_part +
         (clip_on(tau) ? ttt::clip_workspace(B, T, d_model, chunk, in_dtype == TTT_BF16) : 0);
}
}  // namespace

TTT_EXPORT size_t ttt_chunk_scan_docs_workspace(int B, int T, int d_ff, int d_model, int chunk,
                                                ttt_dtype in_dtype, float clip_tau) {
  if (!valid_dtype(in_dtype) || B < 1 || T < 1 || chunk < 1 || d_ff < 16 || d_model < 16 ||
      d_ff % 16 || d_model % 16 || T > (1 << 26) || d_ff > (1 << 20) || d_model > (1 << 20) ||
      B > 65535 || std::isnan(clip_tau))
    return 0;
  size_t part = 0;
  return docs_workspace(B, T, d_ff, d_model, chunk, in_dtype, clip_tau, &part);
}

TTT_EXPORT ttt_status ttt_chunk_scan_docs(const void* Z, const void* Vhat, ttt_dtype in_dtype,
                                          const float* W0, int w0_shared, void* O,
                                          ttt_dtype out_dtype, float* W_final, int B, int T,
                                          int d_ff, int d_model, int chunk, float eta,
                                          const int* doc_starts, const int* doc_counts,
                                          float clip_tau, void* workspace,
                                          size_t workspace_bytes, hipStream_t stream) {
  size_t scan_need = 0;
  const ttt_status st = scan_check(Z, Vhat, in_dtype, W0, w0_shared, O, out_dtype, W_final, B, T,
                                   d_ff, d_model, chunk, eta, workspace, workspace_bytes,
                                   &scan_need);
  if (st != TTT_OK) return st;
  if (std::isnan(clip_tau)) return TTT_E_SHAPE;
  // document starts: per sequence, strictly increasing multiples of chunk inside (0, T)
  if (doc_counts) {
    if (!doc_starts) {
      for (int b = 0; b < B; ++b)
        if (doc_counts[b] != 0) return TTT_E_NULL;
    }
    long k = 0;
    for (int b = 0; b < B; ++b) {
      if (doc_counts[b] < 0 || doc_counts[b] > T) return TTT_E_SHAPE;
      int prev = 0;
      for (int i = 0; i < doc_counts[b]; ++i, ++k) {
        const int s = doc_starts[k];
        if (s <= prev || s >= T || s % chunk) return TTT_E_SHAPE;
        prev = s;
      }
    }
  }
  size_t scan_part = 0;
  const size_t need =
      docs_workspace(B, T, d_ff, d_model, chunk, in_dtype, clip_tau, &scan_part);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return TTT_E_WORKSPACE;
    const size_t isz = dsize(in_dtype), DF = size_t(d_model) * d_ff;
    const Range rws{workspace, need}, rz{Z, size_t(B) * T * d_ff * isz},
        rv{Vhat, size_t(B) * T * d_model * isz}, rw0{W0, (w0_shared ? 1 : size_t(B)) * DF * 4},
        ro{O, size_t(B) * T * d_model * dsize(out_dtype)},
        rwf{W_final, W_final ? size_t(B) * DF * 4 : 0};
    for (Range r : {rz, rv, rw0, ro, rwf})
      if (overlap(rws, r)) return TTT_E_ALIAS;
  }
  const bool bf = in_dtype == TTT_BF16;
  (void)hipGetLastError();
  const void* Vsrc = Vhat;
  if (clip_on(clip_tau) && eta != 0.f) {
    ttt::ClipArgs c{Z, Vhat, bf, B, T, d_ff, d_model, chunk, eta, clip_tau,
                    static_cast<char*>(workspace) + scan_part, stream};
    if (ttt::clip_targets(c) != hipSuccess) return TTT_E_LAUNCH;
    Vsrc = static_cast<char*>(workspace) + scan_part;  // the scaled targets
  }
  auto launch = [&](const ttt::ScanArgs& a) {
    return bf ? ttt::scan_mfma(a, nullptr) : ttt::scan_simt(a, nullptr);
  };
  bool any_doc = false;
  if (doc_counts)
    for (int b = 0; b < B; ++b) any_doc = any_doc || doc_counts[b] > 0;
  if (!any_doc) {
    ttt::ScanArgs a{Z, Vsrc, bf, W0, w0_shared != 0 || B == 1, O, out_dtype == TTT_BF16,
                    W_final, B, T, d_ff, d_model, chunk, eta, workspace, scan_part, stream};
    return launch(a) == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
  }
  // Documents that start on the bf16 scan's group boundaries, or inside a group on an edge of
  // the apply's token tiles: one batched scan whose state chain goes back to W0 at each start.
  // Starts on group boundaries give the bits of separate scans of the documents; a start inside
  // a group gives the document other group edges than a separate scan would (results within
  // rounding of it).
  if (bf) {
    bool inside = false;
    int tile = 0, unit = 1;
    const int G = ttt::scan_mfma_reset_group(B, T, d_ff, d_model, chunk, &inside, &tile, &unit);
    bool aligned = G > 0;
    long k = 0;
    for (int b = 0; b < B && aligned; ++b) {
      for (int i = 0; i < doc_counts[b]; ++i) {
        const int off = doc_starts[k + i] % G;
        aligned = aligned && (off == 0 || (inside && off % tile == 0));
      }
      k += doc_counts[b];
    }
    if (aligned) {
      const int n_units = (T + unit - 1) / unit;
      ttt::ResetMask mask{};
      k = 0;
      for (int b = 0; b < B; ++b) {
        for (int i = 0; i < doc_counts[b]; ++i) {
          const int bit = b * n_units + doc_starts[k + i] / unit;
          mask.bits[bit >> 5] |= 1u << (bit & 31);
        }
        k += doc_counts[b];
      }
      ttt::ScanArgs a{Z, Vsrc, bf, W0, w0_shared != 0 || B == 1, O, out_dtype == TTT_BF16,
                      W_final, B, T, d_ff, d_model, chunk, eta, workspace, scan_part, stream,
                      &mask};
      return launch(a) == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
    }
  }
  // otherwise every document is an independent scan from W0; only a sequence's last one sets
  // W_final
  const size_t isz = dsize(in_dtype), osz = dsize(out_dtype);
  const size_t DF = size_t(d_model) * d_ff;
  long k = 0;
  for (int b = 0; b < B; ++b) {
    const int n = doc_counts[b];
    for (int i = 0; i <= n; ++i) {
      const int s = i == 0 ? 0 : doc_starts[k + i - 1];
      const int e = i == n ? T : doc_starts[k + i];
      const size_t row = size_t(b) * T + s;
      ttt::ScanArgs a{static_cast<const char*>(Z) + row * d_ff * isz,
                      static_cast<const char*>(Vsrc) + row * d_model * isz, bf,
                      W0 + (w0_shared ? 0 : size_t(b) * DF), true,
                      static_cast<char*>(O) + row * d_model * osz, out_dtype == TTT_BF16,
                      i == n && W_final ? W_final + size_t(b) * DF : nullptr, 1, e - s, d_ff,
                      d_model, chunk, eta, workspace, scan_part, stream};
      if (launch(a) != hipSuccess) return TTT_E_LAUNCH;
    }
    k += n;
  }
  return TTT_OK;
}

TTT_EXPORT ttt_status ttt_linear_minibatch(const void* Q, const void* K, const void* V,
                                           ttt_dtype in_dtype, const float* W0, void* O,
                                           ttt_dtype out_dtype, float* W_final, float* loss,
                                           int B, int T, int H, int dh, int minibatch, float eta,
                                           hipStream_t stream) {
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype)) return TTT_E_DTYPE;
  if (!Q || !K || !V || !O) return TTT_E_NULL;
  if (B < 1 || T < 1 || H < 1 || dh < 1 || minibatch < 1 || T % minibatch) return TTT_E_SHAPE;
  if (T > (1 << 26) || B > 65535 || H > 4096 || size_t(B) * H > 65535u * 1024u)
    return TTT_E_SHAPE;
  if (!isfinite(eta)) return TTT_E_SHAPE;
  if (dh != 64) return TTT_E_UNSUPPORTED;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned16(W0) ||
      !aligned16(W_final) || !aligned16(loss))
    return TTT_E_ALIGN;
  const size_t n = size_t(B) * T * H * dh, isz = dsize(in_dtype);
  const Range rq{Q, n * isz}, rk{K, n * isz}, rv{V, n * isz}, ro{O, n * dsize(out_dtype)};
  const size_t wbytes = size_t(B) * H * dh * dh * 4;
  const Range rw0{W0, W0 ? wbytes : 0}, rwf{W_final, W_final ? wbytes : 0};
  const Range rl{loss, loss ? size_t(B) * T * H * 4 : 0};
  for (Range r : {rq, rk, rv, rw0})
    if (overlap(ro, r) || overlap(rwf, r.p == W0 ? Range{nullptr, 0} : r) || overlap(rl, r))
      return TTT_E_ALIAS;
  if (W_final && W0 && overlap(rwf, rw0) && W_final != W0) return TTT_E_ALIAS;
  if (overlap(ro, rwf) || overlap(ro, rl) || overlap(rwf, rl)) return TTT_E_ALIAS;
  ttt::LinearArgs a{Q, K, V, in_dtype == TTT_BF16, W0, O, out_dtype == TTT_BF16, W_final, loss,
                    B, T, H, dh, minibatch, eta, stream};
  (void)hipGetLastError();
  const hipError_t e = ttt::linear_chunk_supported(a)  ? ttt::linear_chunk(a)
                       : ttt::linear_mfma_supported(a) ? ttt::linear_mfma(a)
                                                       : ttt::linear_simt(a);
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

TTT_EXPORT ttt_status ttt_surprisal_route(const float* loss, const void* K, const void* V,
                                          ttt_dtype kv_dtype, int B, int T, int H, int dh,
                                          int chunk, float pct, float ema, float chunk_ratio,
                                          int capacity, float* tau, unsigned char* routed_mask,
                                          int* cache_idx, void* cache_k, void* cache_v,
                                          int* cache_count, int* routed_total,
                                          hipStream_t stream) {
  if (!valid_dtype(kv_dtype)) return TTT_E_DTYPE;
  if (!loss || !cache_idx || !cache_count || !routed_total) return TTT_E_NULL;
  if ((cache_k && !K) || (cache_v && !V)) return TTT_E_NULL;
  if (B < 1 || T < 1 || H < 1 || dh < 1 || chunk < 1 || capacity < 1) return TTT_E_SHAPE;
  if (T % chunk || chunk > 1024 || T > (1 << 22) || capacity > 4096 ||
      B > 65535)
    return TTT_E_SHAPE;
  if (!(pct > 0.f && pct <= 1.f) || !(ema >= 0.f && ema <= 1.f) || !isfinite(chunk_ratio))
    return TTT_E_SHAPE;
  const size_t esz = dsize(kv_dtype);
  if ((size_t(H) * dh * esz) % 16) return TTT_E_SHAPE;
  if (!aligned16(loss) || !aligned16(K) || !aligned16(V) || !aligned16(tau) ||
      !aligned16(routed_mask) || !aligned16(cache_idx) || !aligned16(cache_k) ||
      !aligned16(cache_v) || !aligned16(cache_count) || !aligned16(routed_total))
    return TTT_E_ALIGN;
  const size_t row = size_t(H) * dh * esz;
  const Range ins[] = {{loss, size_t(B) * T * H * 4}, {K, cache_k ? size_t(B) * T * row : 0},
                       {V, cache_v ? size_t(B) * T * row : 0}};
  const Range outs[] = {{tau, tau ? size_t(B) * (T / chunk) * 4 : 0},
                        {routed_mask, routed_mask ? size_t(B) * T : 0},
                        {cache_idx, size_t(B) * capacity * 4},
                        {cache_k, cache_k ? size_t(B) * capacity * row : 0},
                        {cache_v, cache_v ? size_t(B) * capacity * row : 0},
                        {cache_count, size_t(B) * 4},
                        {routed_total, size_t(B) * 4}};
  for (const Range& o : outs) {
    for (const Range& i : ins)
      if (overlap(o, i)) return TTT_E_ALIAS;
    for (const Range& o2 : outs)
      if (&o2 != &o && overlap(o, o2)) return TTT_E_ALIAS;
  }
  ttt::RouteArgs a{loss, K, V, int(esz), B, T, H, dh, chunk, pct, ema, chunk_ratio, capacity,
                   tau, routed_mask, cache_idx, cache_k, cache_v, cache_count, routed_total,
                   stream};
  (void)hipGetLastError();
  const hipError_t e = ttt::route(a);
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

namespace {
bool target_shape_ok(int B, int T, int d_in, int d_out, int chunk, int width) {
  return B >= 1 && T >= 1 && chunk >= 1 && width >= 1 && width <= 16 && d_in >= 64 &&
         d_out >= 16 && d_in % 64 == 0 && d_out % 16 == 0 && T <= (1 << 26) &&
         d_in <= (1 << 16) && d_out <= (1 << 16) && B <= 65535 &&
         size_t(T) * (d_in / 8) / 256 < (1u << 31);
}
}  // namespace

TTT_EXPORT size_t ttt_lm_target_workspace(int B, int T, int d_in, int d_out) {
  if (!target_shape_ok(B, T, d_in, d_out, 1, 1)) return 0;
  return ttt::lm_target_workspace(B, T, d_in, d_out);
}

TTT_EXPORT ttt_status ttt_lm_target(const void* X0, ttt_dtype in_dtype, const float* conv_w,
                                    int width, const void* W_target, void* V_hat,
                                    ttt_dtype out_dtype, int B, int T, int d_in, int d_out,
                                    int chunk, void* workspace, size_t workspace_bytes,
                                    hipStream_t stream) {
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype)) return TTT_E_DTYPE;
  if (!X0 || !conv_w || !W_target || !V_hat) return TTT_E_NULL;
  if (!target_shape_ok(B, T, d_in, d_out, chunk, width)) return TTT_E_SHAPE;
  if (in_dtype != TTT_BF16) return TTT_E_UNSUPPORTED;
  if (!aligned16(X0) || !aligned16(conv_w) || !aligned16(W_target) || !aligned16(V_hat) ||
      !aligned16(workspace))
    return TTT_E_ALIGN;
  const size_t need = ttt_lm_target_workspace(B, T, d_in, d_out);
  if (!workspace || workspace_bytes < need) return TTT_E_WORKSPACE;
  const Range rx{X0, size_t(B) * T * d_in * 2}, rc{conv_w, size_t(width) * d_in * 4},
      rw{W_target, size_t(d_in) * d_out * 2}, rv{V_hat, size_t(B) * T * d_out * dsize(out_dtype)},
      rs{workspace, need};
  for (Range r : {rx, rc, rw})
    if (overlap(rv, r) || overlap(rs, r)) return TTT_E_ALIAS;
  if (overlap(rv, rs)) return TTT_E_ALIAS;
  ttt::TargetArgs a{X0, conv_w, width, W_target, V_hat, out_dtype == TTT_BF16, B, T, d_in,
                    d_out, chunk, workspace, stream};
  (void)hipGetLastError();
  const hipError_t e = ttt::lm_target(a);
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

namespace {
bool gated_z_shape_ok(int B, int T, int d_model, int d_ff) {
  return B >= 1 && B <= 65535 && T >= 1 && T <= (1 << 26) && d_model >= 64 &&
         d_model % 64 == 0 && d_model <= (1 << 16) && d_ff >= 8 && d_ff % 8 == 0 &&
         d_ff <= (1 << 20) && size_t((d_ff + 127) / 128) * ((T + 127) / 128) < (1u << 31) &&
         (size_t(d_ff) + 128) * d_model * 2 < (size_t(1) << 32);
}
}  // namespace

TTT_EXPORT ttt_status ttt_gated_z(const void* X, ttt_dtype in_dtype, const void* W_gu, void* Z,
                                  ttt_dtype out_dtype, int B, int T, int d_model, int d_ff,
                                  hipStream_t stream) {
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype)) return TTT_E_DTYPE;
  if (!X || !W_gu || !Z) return TTT_E_NULL;
  if (!gated_z_shape_ok(B, T, d_model, d_ff)) return TTT_E_SHAPE;
  if (in_dtype != TTT_BF16) return TTT_E_UNSUPPORTED;
  if (!aligned16(X) || !aligned16(W_gu) || !aligned16(Z)) return TTT_E_ALIGN;
  const Range rx{X, size_t(B) * T * d_model * 2}, rw{W_gu, size_t(d_model) * d_ff * 4},
      rz{Z, size_t(B) * T * d_ff * dsize(out_dtype)};
  if (overlap(rz, rx) || overlap(rz, rw)) return TTT_E_ALIAS;
  ttt::GatedZArgs a{X, W_gu, Z, out_dtype == TTT_BF16, B, T, d_model, d_ff, stream};
  (void)hipGetLastError();
  const hipError_t e = ttt::gated_z(a);
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

TTT_EXPORT ttt_status ttt_cache_readout(const void* Q, const void* K, const void* V,
                                        ttt_dtype qkv_dtype, const unsigned char* routed_mask,
                                        const void* ttt_out, void* out, ttt_dtype out_dtype,
                                        const float* alpha, int B, int T, int H, int dh,
                                        int chunk, int capacity, float scale,
                                        hipStream_t stream) {
  if (!valid_dtype(qkv_dtype) || !valid_dtype(out_dtype)) return TTT_E_DTYPE;
  if (!Q || !K || !V || !routed_mask || !ttt_out || !out || !alpha) return TTT_E_NULL;
  if (B < 1 || B > 65535 || T < 1 || T > (1 << 24) || H < 1 || H > 65535 || dh < 1 ||
      chunk < 1 || T % chunk || capacity < 1 || !std::isfinite(scale))
    return TTT_E_SHAPE;
  if (qkv_dtype != TTT_BF16 || dh != 64 || chunk % 64 || capacity > 256) return TTT_E_UNSUPPORTED;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(ttt_out) ||
      !aligned16(out) || !aligned16(alpha) || !aligned16(routed_mask))
    return TTT_E_ALIGN;
  const size_t n = size_t(B) * T * H * dh;
  const Range rq{Q, n * 2}, rk{K, n * 2}, rv{V, n * 2}, rm{routed_mask, size_t(B) * T},
      ra{alpha, size_t(H) * dh * 4}, rt{ttt_out, n * dsize(out_dtype)},
      ro{out, n * dsize(out_dtype)};
  for (Range r : {rq, rk, rv, rm, ra})
    if (overlap(ro, r)) return TTT_E_ALIAS;
  if (out != ttt_out && overlap(ro, rt)) return TTT_E_ALIAS;  // in place is allowed
  ttt::ReadoutArgs a{Q, K, V, routed_mask, ttt_out, out, alpha, out_dtype == TTT_BF16,
                     B, T, H, chunk, capacity, scale, stream};
  (void)hipGetLastError();
  const hipError_t e = ttt::cache_readout(a);
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

namespace {
// Rows of `len` bytes, one every `stride` bytes.
struct Rows {
  const void* p;
  size_t n, stride, len;
};
Range span(Rows r) { return {r.p, r.p && r.n ? (r.n - 1) * r.stride + r.len : 0}; }
// Whether two sets of rows share a byte. Rows with one stride, such as column slices of one buffer, are
// compared within a row; rows with different strides count as overlapping if their spans do.
bool overlap(Rows a, Rows b) {
  if (!overlap(span(a), span(b))) return false;
  if (a.stride != b.stride || a.n == 1 || b.n == 1) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const size_t s = a.stride, d = y >= x ? (y - x) % s : (s - (x - y) % s) % s;
  return !(d >= a.len && d + b.len <= s);  // b's rows start d bytes into a's period
}
Rows whole(const void* p, size_t bytes) { return {p, size_t(p ? 1 : 0), bytes, bytes}; }

bool stride_ok(long long s, long long heads_dh, size_t esz, long long most) {
  return s >= heads_dh && s <= most && (size_t(s) * esz) % 16 == 0;
}
}  // namespace

TTT_EXPORT ttt_status ttt_rope_frequencies(double* inv_freq, int rot, double base,
                                           ttt_rope_scaling scaling, double factor,
                                           int original_length, double beta_fast,
                                           double beta_slow, float* rope_scale) {
  if (!inv_freq) return TTT_E_NULL;
  const int kind = int(scaling);
  if (kind < TTT_ROPE_PLAIN || kind > TTT_ROPE_YARN) return TTT_E_SHAPE;
  if (rot < 2 || rot > 256 || rot % 2 || !(base > 1.) || !std::isfinite(base) || !(factor >= 1.) ||
      !std::isfinite(factor))
    return TTT_E_SHAPE;
  if (kind == TTT_ROPE_NTK && rot < 4) return TTT_E_SHAPE;
  if (kind == TTT_ROPE_YARN && (original_length < 1 || !(beta_slow > 0.) ||
                                !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
    return TTT_E_SHAPE;
  if (kind == TTT_ROPE_NTK) base *= std::pow(factor, double(rot) / (rot - 2));
  // the (fractional) pair that turns n times in original_length positions
  auto pair_of = [&](double n) {
    return rot * std::log(original_length / (n * 6.283185307179586)) / (2. * std::log(base));
  };
  double low = 0., high = 0.;
  if (kind == TTT_ROPE_YARN) {
    low = std::fmax(std::floor(pair_of(beta_fast)), 0.);
    high = std::fmin(std::ceil(pair_of(beta_slow)), rot - 1.);
    if (high <= low) high = low + 1e-3;
  }
  for (int j = 0; j < rot / 2; ++j) {
    const double f = std::pow(base, -2. * j / rot);
    double share = kind == TTT_ROPE_LINEAR ? 1. : 0.;  // of the interpolated frequency
    if (kind == TTT_ROPE_YARN) share = std::fmin(std::fmax((j - low) / (high - low), 0.), 1.);
    inv_freq[j] = f * (1. - share) + f / factor * share;
  }
  if (rope_scale)
    *rope_scale = kind == TTT_ROPE_YARN && factor > 1. ? float(0.1 * std::log(factor) + 1.) : 1.f;
  return TTT_OK;
}

TTT_EXPORT ttt_status ttt_qk_norm_rope(const void* Q, long long q_stride, const void* K,
                                       long long k_stride, const void* V, long long v_stride,
                                       ttt_dtype dtype, const float* q_weight,
                                       const float* k_weight, float eps, const int* pos,
                                       const double* inv_freq, int rot, ttt_rope_layout layout,
                                       float rope_scale, void* Q_out, long long qo_stride,
                                       void* K_out, long long ko_stride, void* K_cache,
                                       void* V_cache, const int* slots, long long n_slots, int N,
                                       int Hq, int Hkv, int dh, hipStream_t stream) {
  if (!valid_dtype(dtype)) return TTT_E_DTYPE;
  if (!Q || !K || !pos || !Q_out || (rot > 0 && !inv_freq)) return TTT_E_NULL;
  if (slots ? !V || !K_cache || !V_cache : !K_out) return TTT_E_NULL;
  if (!slots && (V || K_cache || V_cache)) return TTT_E_NULL;
  // N: a launch counts its threads in 32 bits (64 a token)
  if (N < 1 || N > (1 << 25) || Hq < 1 || Hkv < 1 || Hq > (1 << 16) || Hkv > (1 << 16) ||
      dh < 16 || dh > 256 || dh % 16 || rot < 0 || rot > dh || rot % 16 ||
      (Hq + 2ll * Hkv) * dh > (1 << 20))
    return TTT_E_SHAPE;
  if ((layout != TTT_ROPE_HALF && layout != TTT_ROPE_INTERLEAVED) || !(eps >= 0.f) ||
      !std::isfinite(eps) || !std::isfinite(rope_scale))
    return TTT_E_SHAPE;
  const size_t esz = dsize(dtype);
  const long long most = 1ll << 31, wq = (long long)Hq * dh, wk = (long long)Hkv * dh;
  if (!stride_ok(q_stride, wq, esz, most) || !stride_ok(k_stride, wk, esz, most) ||
      !stride_ok(qo_stride, wq, esz, most) || (K_out && !stride_ok(ko_stride, wk, esz, most)) ||
      (slots && !stride_ok(v_stride, wk, esz, most)))
    return TTT_E_SHAPE;
  if (slots && (n_slots < 1 || n_slots > 0x7FFFFFFFll)) return TTT_E_SHAPE;
  for (const void* p : {Q, K, V, (const void*)q_weight, (const void*)k_weight, (const void*)pos,
                        (const void*)inv_freq, (const void*)Q_out, (const void*)K_out,
                        (const void*)K_cache, (const void*)V_cache, (const void*)slots})
    if (!aligned16(p)) return TTT_E_ALIGN;
  const size_t n = size_t(N);
  const Rows rq{Q, n, size_t(q_stride) * esz, size_t(wq) * esz},
      rk{K, n, size_t(k_stride) * esz, size_t(wk) * esz},
      rv{V, slots ? n : 0, size_t(v_stride) * esz, size_t(wk) * esz},
      oq{Q_out, n, size_t(qo_stride) * esz, size_t(wq) * esz},
      ok{K_out, K_out ? n : 0, size_t(ko_stride) * esz, size_t(wk) * esz},
      ck = whole(K_cache, slots ? size_t(n_slots) * wk * esz : 0),
      cv = whole(V_cache, slots ? size_t(n_slots) * wk * esz : 0);
  const Rows ins[] = {rq, rk, rv, whole(q_weight, size_t(dh) * 4), whole(k_weight, size_t(dh) * 4),
                      whole(pos, n * 4), whole(inv_freq, size_t(rot) * 4),
                      whole(slots, n * 4)};
  const Rows outs[] = {oq, ok, ck, cv};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 8; ++i) {
      // in place: the same rows, each head read by the lanes that write it
      if (i == o && o < 2 && outs[o].p == ins[i].p && outs[o].stride == ins[i].stride) continue;
      if (overlap(outs[o], ins[i])) return TTT_E_ALIAS;
    }
    for (int p = 0; p < o; ++p)
      if (overlap(outs[o], outs[p])) return TTT_E_ALIAS;
  }
  ttt::NormRopeArgs a{Q, K, V, long(q_stride), long(k_stride), long(v_stride), dtype == TTT_BF16,
                      q_weight, k_weight, eps, pos, inv_freq, rot, layout == TTT_ROPE_INTERLEAVED,
                      rope_scale, Q_out, K_out, long(qo_stride), long(ko_stride), K_cache, V_cache,
                      slots, long(n_slots), N, Hq, Hkv, dh, stream};
  (void)hipGetLastError();
  const hipError_t e = ttt::norm_rope(a);
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

namespace {
bool heads_ok(int Hq, int Hkv, int dh) {
  return Hq >= 1 && Hkv >= 1 && Hq <= (1 << 16) && Hq % Hkv == 0 && dh >= 1 &&
         (long long)Hq * dh <= (1 << 22);
}
bool packed_ok(int n_seq, int Nq, int Nk, int Hq, int Hkv, int dh) {
  return heads_ok(Hq, Hkv, dh) && n_seq >= 1 && n_seq <= (1 << 20) && Nq >= 1 && Nk >= 1 &&
         Nq <= (1 << 26) && Nk <= (1 << 26) &&
         // a launch counts its threads in 32 bits: 256 per 128 rows, and per sequence and key head
         (long long)Nq * Hq + 128ll * n_seq * Hkv < (1ll << 31);
}
bool decode_ok(int n_seq, int max_pages, int page, int Hq, int Hkv, int dh) {
  return heads_ok(Hq, Hkv, dh) && n_seq >= 1 && n_seq <= (1 << 20) && max_pages >= 1 && page >= 1 &&
         (long long)max_pages * page <= (1 << 30) &&
         (long long)n_seq * Hq < (1 << 24);  // 256 threads each at most, counted in 32 bits
}
bool page_ok(int page) { return page >= 16 && page <= 65536 && (page & (page - 1)) == 0; }
bool scale_ok(float s) { return s > 0.f && std::isfinite(s); }
}  // namespace

TTT_EXPORT size_t ttt_attention_packed_workspace(int n_seq, int Nq, int Nk, int Hq, int Hkv, int dh) {
  if (!packed_ok(n_seq, Nq, Nk, Hq, Hkv, dh) || (dh != 64 && dh != 128)) return 0;
  return ttt::attention_packed_workspace(n_seq, Nq, Nk, Hq, Hkv, dh);
}

TTT_EXPORT ttt_status ttt_attention_packed(const void* Q, long long q_stride, const void* K,
                                           long long k_stride, const void* V, long long v_stride,
                                           ttt_dtype dtype, void* O, long long o_stride,
                                           float* lse, const int* cu_q, const int* cu_k, int n_seq,
                                           int Nq, int Nk, int Hq, int Hkv, int dh, float scale,
                                           int window, void* workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
  if (!valid_dtype(dtype)) return TTT_E_DTYPE;
  if (!Q || !K || !V || !O || !cu_q || !cu_k) return TTT_E_NULL;
  if (!packed_ok(n_seq, Nq, Nk, Hq, Hkv, dh) || window < 0 || window > (1 << 30) || !scale_ok(scale))
    return TTT_E_SHAPE;
  if (dtype != TTT_BF16 || (dh != 64 && dh != 128)) return TTT_E_UNSUPPORTED;
  const long long most = 1 << 23, wq = (long long)Hq * dh, wk = (long long)Hkv * dh;
  if (!stride_ok(q_stride, wq, 2, most) || !stride_ok(k_stride, wk, 2, most) ||
      !stride_ok(v_stride, wk, 2, most) || !stride_ok(o_stride, wq, 2, most))
    return TTT_E_SHAPE;
  for (const void* p : {Q, K, V, (const void*)O, (const void*)lse, (const void*)cu_q,
                        (const void*)cu_k, (const void*)workspace})
    if (!aligned16(p)) return TTT_E_ALIGN;
  const size_t need = ttt::attention_packed_workspace(n_seq, Nq, Nk, Hq, Hkv, dh);
  if (need && (!workspace || workspace_bytes < need)) return TTT_E_WORKSPACE;
  const size_t nq = size_t(Nq), nk = size_t(Nk);
  const Rows ins[] = {{Q, nq, size_t(q_stride) * 2, size_t(wq) * 2},
                      {K, nk, size_t(k_stride) * 2, size_t(wk) * 2},
                      {V, nk, size_t(v_stride) * 2, size_t(wk) * 2},
                      whole(cu_q, size_t(n_seq + 1) * 4), whole(cu_k, size_t(n_seq + 1) * 4)};
  const Rows outs[] = {{O, nq, size_t(o_stride) * 2, size_t(wq) * 2},
                       whole(lse, nq * Hq * 4), whole(need ? workspace : nullptr, need)};
  for (int o = 0; o < 3; ++o) {
    for (const Rows& i : ins)
      if (overlap(outs[o], i)) return TTT_E_ALIAS;
    for (int p = 0; p < o; ++p)
      if (overlap(outs[o], outs[p])) return TTT_E_ALIAS;
  }
  ttt::PackedArgs a{Q, K, V, long(q_stride), long(k_stride), long(v_stride), O, long(o_stride), lse,
                    cu_q, cu_k, n_seq, Nq, Nk, Hq, Hkv, dh, scale, window, workspace, stream};
  (void)hipGetLastError();
  const hipError_t e = ttt::attention_packed(a);
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

TTT_EXPORT size_t ttt_attention_decode_workspace(int n_seq, int max_pages, int page_size, int Hq,
                                                 int Hkv, int dh) {
  if (!decode_ok(n_seq, max_pages, page_size, Hq, Hkv, dh) || !page_ok(page_size) ||
      (dh != 64 && dh != 128))
    return 0;
  return ttt::attention_decode_workspace(n_seq, max_pages, page_size, Hq, Hkv, dh);
}

TTT_EXPORT ttt_status ttt_attention_decode(const void* Q, long long q_stride, const void* K_cache,
                                           const void* V_cache, ttt_dtype dtype, void* O,
                                           long long o_stride, float* lse, const int* page_table,
                                           int max_pages, int page_size, int n_pages,
                                           const int* lengths, int n_seq, int Hq, int Hkv, int dh,
                                           float scale, int window, void* workspace,
                                           size_t workspace_bytes, hipStream_t stream) {
  if (!valid_dtype(dtype)) return TTT_E_DTYPE;
  if (!Q || !K_cache || !V_cache || !O || !page_table || !lengths) return TTT_E_NULL;
  if (!decode_ok(n_seq, max_pages, page_size, Hq, Hkv, dh) || n_pages < 1 ||
      (long long)n_pages * page_size > (1ll << 36) || window < 0 || window > (1 << 30) || !scale_ok(scale))
    return TTT_E_SHAPE;
  if (dtype != TTT_BF16 || (dh != 64 && dh != 128) || !page_ok(page_size)) return TTT_E_UNSUPPORTED;
  const long long most = 1 << 23, wq = (long long)Hq * dh;
  if (!stride_ok(q_stride, wq, 2, most) || !stride_ok(o_stride, wq, 2, most)) return TTT_E_SHAPE;
  for (const void* p : {Q, K_cache, V_cache, (const void*)O, (const void*)lse,
                        (const void*)page_table, (const void*)lengths, (const void*)workspace})
    if (!aligned16(p)) return TTT_E_ALIGN;
  const size_t need =
      ttt::attention_decode_workspace(n_seq, max_pages, page_size, Hq, Hkv, dh);
  if (need && (!workspace || workspace_bytes < need)) return TTT_E_WORKSPACE;
  const size_t ns = size_t(n_seq), cache = size_t(n_pages) * page_size * Hkv * dh * 2;
  const Rows ins[] = {{Q, ns, size_t(q_stride) * 2, size_t(wq) * 2}, whole(K_cache, cache),
                      whole(V_cache, cache), whole(page_table, ns * max_pages * 4),
                      whole(lengths, ns * 4)};
  const Rows outs[] = {{O, ns, size_t(o_stride) * 2, size_t(wq) * 2},
                       whole(lse, ns * Hq * 4), whole(need ? workspace : nullptr, need)};
  for (int o = 0; o < 3; ++o) {
    for (const Rows& i : ins)
      if (overlap(outs[o], i)) return TTT_E_ALIAS;
    for (int p = 0; p < o; ++p)
      if (overlap(outs[o], outs[p])) return TTT_E_ALIAS;
  }
  ttt::DecodeArgs a{Q, long(q_stride), K_cache, V_cache, O, long(o_stride), lse, page_table,
                    lengths, max_pages, page_size, n_pages, n_seq, Hq, Hkv, dh, scale, window,
                    workspace, stream};
  (void)hipGetLastError();
  const hipError_t e = ttt::attention_decode(a);
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

namespace {
bool paged_ok(int n_seq, int Nq, int max_pages, int page, int Hq, int Hkv, int dh) {
  return packed_ok(n_seq, Nq, 1, Hq, Hkv, dh) && max_pages >= 1 && page >= 1 &&
         (long long)max_pages * page <= (1 << 30);
}
}  // namespace

TTT_EXPORT size_t ttt_attention_paged_workspace(int n_seq, int Nq, int max_pages, int page_size, int Hq,
                                                int Hkv, int dh) {
  if (!paged_ok(n_seq, Nq, max_pages, page_size, Hq, Hkv, dh) || !page_ok(page_size) || (dh != 64 && dh != 128))
    return 0;
  return ttt::attention_paged_workspace(n_seq, Nq, max_pages, page_size, Hq, Hkv, dh);
}

TTT_EXPORT ttt_status ttt_attention_paged(const void* Q, long long q_stride, const void* K_cache,
                                          const void* V_cache, ttt_dtype dtype, void* O, long long o_stride,
                                          float* lse, const int* cu_q, const int* page_table, int max_pages,
                                          int page_size, int n_pages, const int* lengths, int n_seq, int Nq,
                                          int Hq, int Hkv, int dh, float scale, int window, void* workspace,
                                          size_t workspace_bytes, hipStream_t stream) {
  if (!valid_dtype(dtype)) return TTT_E_DTYPE;
  if (!Q || !K_cache || !V_cache || !O || !cu_q || !page_table || !lengths) return TTT_E_NULL;
  if (!paged_ok(n_seq, Nq, max_pages, page_size, Hq, Hkv, dh) || n_pages < 1 ||
      (long long)n_pages * page_size > (1ll << 36) || window < 0 || window > (1 << 30) || !scale_ok(scale))
    return TTT_E_SHAPE;
  if (dtype != TTT_BF16 || (dh != 64 && dh != 128) || !page_ok(page_size)) return TTT_E_UNSUPPORTED;
  const long long most = 1 << 23, wq = (long long)Hq * dh, wk = (long long)Hkv * dh;
  if (!stride_ok(q_stride, wq, 2, most) || !stride_ok(o_stride, wq, 2, most)) return TTT_E_SHAPE;
  for (const void* p : {Q, K_cache, V_cache, (const void*)O, (const void*)lse, (const void*)cu_q,
                        (const void*)page_table, (const void*)lengths, (const void*)workspace})
    if (!aligned16(p)) return TTT_E_ALIGN;
  const size_t need = ttt::attention_paged_workspace(n_seq, Nq, max_pages, page_size, Hq, Hkv, dh);
  if (need && (!workspace || workspace_bytes < need)) return TTT_E_WORKSPACE;
  const size_t nq = size_t(Nq), ns = size_t(n_seq), cache = size_t(n_pages) * page_size * wk * 2;
  const Rows ins[] = {{Q, nq, size_t(q_stride) * 2, size_t(wq) * 2}, whole(K_cache, cache),
                      whole(V_cache, cache), whole(cu_q, (ns + 1) * 4), whole(page_table, ns * max_pages * 4),
                      whole(lengths, ns * 4)};
  const Rows outs[] = {{O, nq, size_t(o_stride) * 2, size_t(wq) * 2},
                       whole(lse, nq * Hq * 4), whole(need ? workspace : nullptr, need)};
  for (int o = 0; o < 3; ++o) {
    for (const Rows& i : ins)
      if (overlap(outs[o], i)) return TTT_E_ALIAS;
    for (int p = 0; p < o; ++p)
      if (overlap(outs[o], outs[p])) return TTT_E_ALIAS;
  }
  const ttt::PackedArgs a{Q, K_cache, V_cache, long(q_stride), long(wk), long(wk), O, long(o_stride), lse,
                          cu_q, nullptr, n_seq, Nq, 0, Hq, Hkv, dh, scale, window, workspace, stream};
  (void)hipGetLastError();
  const hipError_t e = ttt::attention_paged(a, {page_table, lengths, max_pages, page_size, n_pages});
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

TTT_EXPORT ttt_status ttt_add_rms_norm(const void* X, long long x_stride, const void* R, long long r_stride,
                                       ttt_dtype dtype, const float* weight, float eps, void* S,
                                       long long s_stride, void* Y, long long y_stride, float* scales,
                                       int group, int N, int D, hipStream_t stream) {
  if (!valid_dtype(dtype)) return TTT_E_DTYPE;
  if (!X || !Y) return TTT_E_NULL;
  if (N < 1 || N > (1 << 30) || D < 8 || D > 16384 || D % 8 || !(eps >= 0.f) || !std::isfinite(eps))
    return TTT_E_SHAPE;
  if (group && (!scales || group < 16 || group > 512 || (group & (group - 1)) || D % group)) return TTT_E_SHAPE;
  const size_t esz = dsize(dtype), ysz = scales ? 1 : esz;
  const long long most = 1ll << 31;
  if (!stride_ok(x_stride, D, esz, most) || (R && !stride_ok(r_stride, D, esz, most)) ||
      (S && !stride_ok(s_stride, D, esz, most)) || y_stride < D || y_stride > most ||
      (size_t(y_stride) * ysz) % (scales ? 8 : 16))
    return TTT_E_SHAPE;
  for (const void* p : {X, R, (const void*)weight, (const void*)S, (const void*)Y, (const void*)scales})
    if (!aligned16(p)) return TTT_E_ALIGN;
  const size_t n = size_t(N), row = size_t(D) * esz;
  const Rows rx{X, n, size_t(x_stride) * esz, row}, rr{R, R ? n : 0, size_t(r_stride) * esz, row},
      rs{S, S ? n : 0, size_t(s_stride) * esz, row}, ry{Y, n, size_t(y_stride) * ysz, size_t(D) * ysz};
  const Rows ins[] = {rx, rr, whole(weight, size_t(D) * 4)};
  const Rows outs[] = {rs, ry, whole(scales, n * (group ? D / group : 1) * 4)};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 3; ++i) {
      // in place: the same rows, each channel read by the lane that writes it
      const bool same = outs[o].p == ins[i].p && outs[o].stride == ins[i].stride;
      if (same && i < 2 && (o == 0 || (o == 1 && !scales))) continue;
      if (overlap(outs[o], ins[i])) return TTT_E_ALIAS;
    }
    for (int p = 0; p < o; ++p)
      if (overlap(outs[o], outs[p])) return TTT_E_ALIAS;
  }
  ttt::AddNormArgs a{X, R, long(x_stride), long(r_stride), weight, eps, S, Y, long(s_stride), long(y_stride),
                     scales, group, N, D, dtype == TTT_BF16, scales != nullptr, stream};
  (void)hipGetLastError();
  const hipError_t e = ttt::add_norm(a);
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

namespace {
// What a call of the gated delta rule gets, and what it asks of that.
struct DeltaCall {
  const void *Q, *K, *V;
  long long q_stride, k_stride, v_stride;
  ttt_dtype dtype;
  const float *g, *beta;
  void* O;
  long long o_stride;
  const float* state_in;
  float* state_out;
  const int* slots;
  long long n_slots;
  int tokens, n_seq, Hk, Hv, dk, dv;
  float scale, eps;
  long long most;  // tokens * Hv * dv, exclusive: a launch counts its threads in 32 bits
};
bool delta_shape_ok(int tokens, int n_seq, int Hk, int Hv, int dk, int dv) {
  return tokens >= 1 && n_seq >= 1 && n_seq <= (1 << 20) && Hk >= 1 && Hv >= 1 && Hv <= (1 << 16) &&
         Hv % Hk == 0 && dk >= 1 && dv >= 1 && dk <= 65536 && dv <= 65536 &&
         (long long)Hk * dk <= (1 << 22) && (long long)Hv * dv <= (1 << 22);
}
bool delta_supported(int dk, int dv) { return (dk == 64 || dk == 128) && dv % 64 == 0 && dv <= 512; }
ttt_status delta_check(const DeltaCall& c, Rows cu, Rows ws) {
  if (!valid_dtype(c.dtype)) return TTT_E_DTYPE;
  if (!c.Q || !c.K || !c.V || !c.g || !c.beta || !c.O) return TTT_E_NULL;
  if (!delta_shape_ok(c.tokens, c.n_seq, c.Hk, c.Hv, c.dk, c.dv) ||
      (long long)c.tokens * c.Hv * c.dv >= c.most || !std::isfinite(c.scale) || !(c.eps >= 0.f) ||
      !std::isfinite(c.eps))
    return TTT_E_SHAPE;
  if (c.dtype != TTT_BF16 || !delta_supported(c.dk, c.dv)) return TTT_E_UNSUPPORTED;
  const long long most = 1ll << 31, wk = (long long)c.Hk * c.dk, wv = (long long)c.Hv * c.dv;
  if (!stride_ok(c.q_stride, wk, 2, most) || !stride_ok(c.k_stride, wk, 2, most) ||
      !stride_ok(c.v_stride, wv, 2, most) || !stride_ok(c.o_stride, wv, 2, most))
    return TTT_E_SHAPE;
  const bool pool = c.state_in || c.state_out;
  if (pool && (c.n_slots < (c.slots ? 1 : c.n_seq) || c.n_slots > 0x7FFFFFFFll)) return TTT_E_SHAPE;
  for (const void* p : {c.Q, c.K, c.V, (const void*)c.g, (const void*)c.beta, (const void*)c.O,
                        (const void*)c.state_in, (const void*)c.state_out, (const void*)c.slots, cu.p, ws.p})
    if (!aligned16(p)) return TTT_E_ALIGN;
  const size_t n = size_t(c.tokens), states = pool ? size_t(c.n_slots) * wv * c.dk * 4 : 0;
  const Rows ins[] = {whole(c.state_in, states),
                      {c.Q, n, size_t(c.q_stride) * 2, size_t(wk) * 2},
                      {c.K, n, size_t(c.k_stride) * 2, size_t(wk) * 2},
                      {c.V, n, size_t(c.v_stride) * 2, size_t(wv) * 2},
                      whole(c.g, n * c.Hv * 4), whole(c.beta, n * c.Hv * 4),
                      whole(c.slots, size_t(c.n_seq) * 4), cu};
  const Rows outs[] = {whole(c.state_out, states), {c.O, n, size_t(c.o_stride) * 2, size_t(wv) * 2}, ws};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 8; ++i) {
      if (i == 0 && o == 0 && c.state_in == c.state_out) continue;  // in place
      if (overlap(outs[o], ins[i])) return TTT_E_ALIAS;
    }
    for (int p = 0; p < o; ++p)
      if (overlap(outs[o], outs[p])) return TTT_E_ALIAS;
  }
  return TTT_OK;
}
ttt::DeltaArgs delta_args(const DeltaCall& c, int normalize, hipStream_t stream) {
  return {c.Q, c.K, c.V, long(c.q_stride), long(c.k_stride), long(c.v_stride), c.g, c.beta, c.O,
          long(c.o_stride), c.state_in, c.state_out, c.slots, long(c.n_slots), c.n_seq, c.Hk, c.Hv, c.dk,
          c.dv, c.scale, normalize != 0, c.eps, stream};
}
}  // namespace

TTT_EXPORT ttt_status ttt_gated_delta_decode(const void* Q, long long q_stride, const void* K,
                                             long long k_stride, const void* V, long long v_stride,
                                             ttt_dtype dtype, const float* g, const float* beta, void* O,
                                             long long o_stride, const float* state_in, float* state_out,
                                             const int* slots, long long n_slots, int n_seq, int Hk, int Hv,
                                             int dk, int dv, float scale, int normalize, float eps,
                                             hipStream_t stream) {
  const DeltaCall c{Q, K, V, q_stride, k_stride, v_stride, dtype, g, beta, O, o_stride, state_in, state_out,
                    slots, n_slots, n_seq, n_seq, Hk, Hv, dk, dv, scale, eps, 1ll << 30};
  const ttt_status s = delta_check(c, whole(nullptr, 0), whole(nullptr, 0));
  if (s != TTT_OK) return s;
  (void)hipGetLastError();
  const hipError_t e = ttt::delta_step(delta_args(c, normalize, stream));
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

namespace {
bool delta_packed_ok(int n_seq, int N, int Hk, int Hv, int dk, int dv) {
  return delta_shape_ok(N, n_seq, Hk, Hv, dk, dv) && N <= (1 << 26) &&
         // a launch counts its threads in 32 bits: 256 per 64 tokens and head, 512 per 32 columns
         ((long long)N / 64 + n_seq) * Hv < (1 << 24) && (long long)n_seq * Hv * dv < (1 << 28);
}
}  // namespace

TTT_EXPORT size_t ttt_gated_delta_packed_workspace(int n_seq, int N, int Hk, int Hv, int dk, int dv) {
  if (!delta_packed_ok(n_seq, N, Hk, Hv, dk, dv) || !delta_supported(dk, dv)) return 0;
  return ttt::delta_packed_workspace(n_seq, N, Hv);
}

TTT_EXPORT ttt_status ttt_gated_delta_packed(const void* Q, long long q_stride, const void* K,
                                             long long k_stride, const void* V, long long v_stride,
                                             ttt_dtype dtype, const float* g, const float* beta, void* O,
                                             long long o_stride, const float* state_in, float* state_out,
                                             const int* slots, long long n_slots, const int* cu, int n_seq,
                                             int N, int Hk, int Hv, int dk, int dv, float scale,
                                             int normalize, float eps, void* workspace,
                                             size_t workspace_bytes, hipStream_t stream) {
  if (!valid_dtype(dtype)) return TTT_E_DTYPE;
  if (!cu) return TTT_E_NULL;
  if (!delta_packed_ok(n_seq, N, Hk, Hv, dk, dv)) return TTT_E_SHAPE;
  const long long most = 1 << 23;  // 64 rows' offsets in 32 bits
  if (q_stride > most || k_stride > most || v_stride > most || o_stride > most) return TTT_E_SHAPE;
  const size_t need = delta_supported(dk, dv) ? ttt::delta_packed_workspace(n_seq, N, Hv) : 0;
  const DeltaCall c{Q, K, V, q_stride, k_stride, v_stride, dtype, g, beta, O, o_stride, state_in, state_out,
                    slots, n_slots, N, n_seq, Hk, Hv, dk, dv, scale, eps, 1ll << 62};
  const ttt_status s = delta_check(c, whole(cu, size_t(n_seq + 1) * 4), whole(workspace, need));
  if (s != TTT_OK) return s;
  if (!workspace || workspace_bytes < need) return TTT_E_WORKSPACE;
  (void)hipGetLastError();
  const hipError_t e = ttt::delta_packed({delta_args(c, normalize, stream), cu, N, workspace});
  return e == hipSuccess ? TTT_OK : TTT_E_LAUNCH;
}

TTT_EXPORT const char* ttt_status_string(ttt_status s) {
  switch (s) {
    case TTT_OK: return "TTT_OK: success";
    case TTT_E_NULL: return "TTT_E_NULL: a required pointer is NULL";
    case TTT_E_SHAPE: return "TTT_E_SHAPE: a size or parameter is out of range";
    case TTT_E_DTYPE: return "TTT_E_DTYPE: unknown dtype code";
    case TTT_E_ALIGN: return "TTT_E_ALIGN: a pointer is not 16-byte aligned";
    case TTT_E_WORKSPACE: return "TTT_E_WORKSPACE: workspace missing or too small";
    case TTT_E_UNSUPPORTED: return "TTT_E_UNSUPPORTED: valid request this library does not implement";
    case TTT_E_LAUNCH: return "TTT_E_LAUNCH: the HIP runtime rejected a launch";
    case TTT_E_ALIAS: return "TTT_E_ALIAS: an output overlaps an input";
  }
  return "unknown ttt_status";
}

TTT_EXPORT int ttt_abi_version(void) { return TTT_ABI_VERSION; }
