// C ABI of the GBLA library (include/gbla.h): argument validation, workspace
// layout, tiling choices and the launch sequence of every entry point.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <string>
#include <vector>

#include "../../include/gbla.h"
#include "kernels.h"
#include "mbarrier.cuh"

using namespace gbla;

namespace {

thread_local std::string g_last_error;
thread_local int g_policy = GBLA_POLICY_AUTO;  // gbla_set_kernel_policy

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
int cdiv(int a, int b) { return (a + b - 1) / b; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Per-launch profiler names of the GEMMs, by Variant: the projection, dx~ and dW GEMMs.
const char* const kGemmNames[3][3] = {
    {"projection gemm[tc]", "projection gemm[mma]", "projection gemm[f32]"},
    {"dx~ gemm[tc]", "dx~ gemm[mma]", "dx~ gemm[f32]"},
    {"dW gemm[tc]", "dW gemm[mma]", "dW gemm[f32]"},
};

// Everything derived from a shape: sequence form, tilings, buffer sizes.
struct Plan {
  bool f32;
  int B, L, d, H, dh, T, n_seq, mode;
  int HD, N1, NP;        // H*dh, 4*H*dh + H, N1 padded to 64
  int chunk, chunk_per_seq, n_chunks;  // state-reduction chunks (grid.x)
  int tile, tile_per_seq, n_tiles;     // readout / key-side tiles (grid.x)
  int wsplit, n_wsplit;                // dW split over rows
  int conv_blocks;
  int sms;               // SMs of the current device
  int max_grid;          // CTAs of a range-split kernel the workspace provides for (>= 2 x SMs)
  size_t io;             // bytes per io element
};

gbla_status make_plan(const gbla_shape* s, Plan& p) {
  if (!s) return GBLA_ERR_INVALID_ARG;
  if (s->io_dtype != GBLA_F32 && s->io_dtype != GBLA_BF16) return GBLA_ERR_INVALID_ARG;
  if (s->gate != GBLA_GATE_SIGMOID && s->gate != GBLA_GATE_SOFTMAX) return GBLA_ERR_INVALID_ARG;
  if (s->B < 1 || s->L < 1 || s->d < 1 || s->H < 1 || s->d_h < 1) return GBLA_ERR_INVALID_ARG;
  if (!(s->rms_eps >= 0.f)) return GBLA_ERR_INVALID_ARG;
  if (s->cu_seqlens && s->seq_lens) return GBLA_ERR_INVALID_ARG;
  if (s->cu_seqlens && (s->B != 1 || s->num_seqs < 1)) return GBLA_ERR_INVALID_ARG;
  p.f32 = s->io_dtype == GBLA_F32;
  p.io = p.f32 ? 4 : 2;
  p.B = s->B; p.L = s->L; p.d = s->d; p.H = s->H; p.dh = s->d_h;
  p.sms = sm_count();
  p.max_grid = std::max(512, 2 * p.sms);
  const int kSMs = p.sms;
  if (p.f32) {
    if (p.dh % 4 != 0 || p.dh > 128) return GBLA_ERR_UNSUPPORTED;
  } else {
    if (p.dh != 32 && p.dh != 64 && p.dh != 128) return GBLA_ERR_UNSUPPORTED;
  }
  const long long T = s->cu_seqlens ? (long long)s->L : (long long)s->B * s->L;
  if (T > (8LL << 20)) return GBLA_ERR_UNSUPPORTED;  // grid rows of the GEMMs
  if ((long long)s->H * s->d_h > 65536) return GBLA_ERR_UNSUPPORTED;
  p.T = (int)T;
  p.mode = s->cu_seqlens ? SEQ_VARLEN : (s->seq_lens ? SEQ_PADDED : SEQ_DENSE);
  p.n_seq = s->cu_seqlens ? s->num_seqs : s->B;
  p.HD = p.H * p.dh;
  p.N1 = 4 * p.HD + p.H;
  p.NP = (p.N1 + 63) / 64 * 64;
  const int pairs = p.n_seq * p.H;
  const int cg = p.f32 ? 64 : 128;  // chunk granule: the row tile of the query-side backward
  if (p.mode == SEQ_VARLEN) {
    const long long want = ((long long)p.T * p.H + kSMs - 1) / kSMs;
    p.chunk = (int)std::min<long long>(2048, std::max<long long>(256, (want + cg - 1) / cg * cg));
    p.chunk_per_seq = 0;
    p.n_chunks = cdiv(p.T, p.chunk) + p.n_seq;
  } else {
    // Chunks per sequence: one CTA per (chunk, head) of the state reduction
    // and the query-side backward, two resident per SM.  Take the split with
    // the least work on the busiest SM: its CTAs x (tiles per CTA + one tile
    // for start-up and the combine), at 3.7 time units a tile when two CTAs
    // share the SM and 4.5 when one runs alone (measured per-tile times of the
    // query-side backward).
    const int tiles = cdiv(p.L, cg);
    long long best_cost = -1;
    int best_tpc = tiles;
    for (int per = 1; per <= std::min(tiles, 64); ++per) {
      const int tpc = cdiv(tiles, per);
      const long long ctas = (long long)pairs * cdiv(tiles, tpc);
      const long long per_sm = (ctas + kSMs - 1) / kSMs;
      const long long cost = per_sm >= 2 ? per_sm * (tpc + 1) * 37 : (long long)(tpc + 1) * 45;
      if (best_cost < 0 || cost < best_cost) {
        best_cost = cost;
        best_tpc = tpc;
      }
    }
    p.chunk = best_tpc * cg;
    p.chunk_per_seq = cdiv(p.L, p.chunk);
    p.n_chunks = p.chunk_per_seq * p.n_seq;
  }
  p.tile = p.f32 ? 64 : (p.dh == 128 ? 128 : 256);
  if (p.mode == SEQ_VARLEN) {
    p.tile_per_seq = 0;
    p.n_tiles = cdiv(p.T, p.tile) + p.n_seq;
  } else {
    p.tile_per_seq = cdiv(p.L, p.tile);
    p.n_tiles = p.tile_per_seq * p.n_seq;
  }
  // dW = x~^T dP: split the T rows so that output tiles x splits fill whole
  // waves of the GPU (tiles of the bf16 tensor-core GEMM: 128 x 256; of the
  // fp32 GEMM: 64 x 64), each split at least 1024 rows.
  const int tiles = p.f32 ? cdiv(p.d, 64) * cdiv(p.NP, 64) : cdiv(p.d, 128) * cdiv(p.NP, 256);
  const int max_split = std::max(1, std::min(16, p.T / 1024));
  int want_split = 1;
  double best = -1.0;
  for (int sp = 1; sp <= max_split; ++sp) {
    const int units = tiles * sp;
    const double eff = (double)units / ((double)cdiv(units, kSMs) * kSMs);
    if (eff > best + 0.02) { best = eff; want_split = sp; }  // the smallest split within 2% of the best
  }
  p.wsplit = cdiv(cdiv(p.T, want_split), 64) * 64;
  p.n_wsplit = cdiv(p.T, p.wsplit);
  p.conv_blocks = conv_bwd_parts_max(p.T);
  return GBLA_OK;
}

gbla_status check_layer_shape(const Plan& p) {
  if (p.d % (p.f32 ? 4 : 64) != 0) return GBLA_ERR_UNSUPPORTED;
  return GBLA_OK;
}

// Byte layout of a workspace (or of the saved buffer), in order.
struct Layout {
  size_t err, cnt_f, cnt_b, pre_c, pre_t;
  size_t partial, partial_m, state, state_bf, state_m, center;
  size_t xt, P, gate, Wt;
  size_t Wp, dP, dxt, dW, dstate, dstate_bf, gamma_part, bg_part, conv_part;
  size_t pre_d, LF, LB, lamc, HF, HB;  // the decay core: its chunks' prefix, chunk and scan states
  size_t total;
};

// 256-query blocks (per sequence) of the softmax attention.
constexpr int kSaBlock = 256;
int sa_blocks(const Plan& p) {
  return p.mode == SEQ_VARLEN ? cdiv(p.T, kSaBlock) + p.n_seq : cdiv(p.L, kSaBlock) * p.n_seq;
}

// Chunks (128 rows, per sequence) of the decay core.
int decay_chunks(const Plan& p) {
  return p.mode == SEQ_VARLEN ? cdiv(p.T, kDecayChunk) + p.n_seq : cdiv(p.L, kDecayChunk) * p.n_seq;
}

struct Cursor {
  size_t off = 0;
  size_t take(size_t bytes) { const size_t o = off; off = align_up(off + bytes); return o; }
};


size_t state_bytes(const Plan& p) { return (size_t)p.n_seq * p.H * p.dh * state_ld(p.dh) * 4; }
size_t state_bf_bytes(const Plan& p) { return (size_t)p.n_seq * p.H * p.dh * state_bf_ld(p.dh) * 2; }

// Saved activations of a training forward: x~, P = [q|k|v|r], gate, state.
struct SavedLayout { size_t xt, P, gate, state, state_bf, state_m, center, rsinv, total; };
size_t center_bytes(const Plan& p) { return (size_t)p.n_seq * p.H * p.dh * 4; }
SavedLayout saved_layout(const Plan& p) {
  Cursor c;
  SavedLayout s;
  s.xt = c.take((size_t)p.T * p.d * p.io);
  s.P = c.take((size_t)p.T * 4 * p.HD * p.io);
  s.gate = c.take((size_t)p.T * p.H * 4);
  s.state = c.take(state_bytes(p));
  s.state_bf = c.take(state_bf_bytes(p));
  s.state_m = c.take((size_t)p.n_seq * p.H * 4);
  s.center = c.take(center_bytes(p));
  s.rsinv = c.take((size_t)p.T * p.H * 8);  // per row and head: RMSNorm rs and 1/den of the readout
  s.total = c.off;
  return s;
}

// Partial-state slots: one per (chunk, head) for the split-L kernels; the
// tcgen05 query-side backward takes one per (sequence, head) plus one per CTA
// (a CTA boundary inside a (sequence, head)).
int partial_slots(const Plan& p) { return std::max(p.n_chunks * p.H, p.n_seq * p.H + p.max_grid); }

Layout ws_layout(const Plan& p, int op) {
  Cursor c;
  Layout l;
  std::memset(&l, 0xff, sizeof(l));
  const size_t cnt = (size_t)p.n_seq * p.H * 4;
  l.err = c.take(16 + 2 * cnt);  // err word, then forward and backward counters
  l.cnt_f = l.err + 16;
  l.cnt_b = l.cnt_f + cnt;
  if (p.mode == SEQ_VARLEN) {
    l.pre_c = c.take((size_t)(p.n_seq + 1) * 4);
    l.pre_t = c.take((size_t)(p.n_seq + 1) * 4);
  }
  if (op != GBLA_OP_SA_FORWARD) {  // split-L partial states (every kernel but the softmax attention)
    l.partial = c.take((size_t)partial_slots(p) * p.dh * state_ld(p.dh) * 4);
    l.partial_m = c.take((size_t)p.n_chunks * p.H * 4);
  }
  if (op == GBLA_OP_FORWARD) {  // inference forward keeps its activations here
    l.state = c.take(state_bytes(p));
    l.state_bf = c.take(state_bf_bytes(p));
    l.state_m = c.take((size_t)p.n_seq * p.H * 4);
    l.center = c.take(center_bytes(p));
    l.xt = c.take((size_t)p.T * p.d * p.io);
    l.P = c.take((size_t)p.T * 4 * p.HD * p.io);
    l.gate = c.take((size_t)p.T * p.H * 4);
    l.Wt = c.take((size_t)p.d * p.NP * p.io);  // packed W_all [d][NP]
  } else if (op == GBLA_OP_BACKWARD) {
    l.Wp = c.take((size_t)p.d * p.NP * p.io);
    l.dP = c.take((size_t)p.T * p.NP * p.io);
    l.dxt = c.take((size_t)p.T * p.d * p.io);
    l.dW = c.take((size_t)p.n_wsplit * p.d * p.NP * 4);
    l.dstate = c.take(state_bytes(p));
    l.dstate_bf = c.take(state_bf_bytes(p));
    l.gamma_part = c.take((size_t)std::max(p.n_chunks * p.H, p.max_grid) * p.dh * 4);
    // db_g partial rows: two per tile (tcgen05 kernel) or one per chunk
    l.bg_part = c.take((size_t)std::max(2 * p.n_tiles, p.n_chunks) * p.H * 4);
    l.conv_part = c.take((size_t)p.conv_blocks * p.d * 5 * 4);
  } else if (op == GBLA_OP_SA_FORWARD) {
    if (p.mode == SEQ_VARLEN) l.pre_d = c.take((size_t)(p.n_seq + 1) * 4);
  } else if (op == GBLA_OP_DECAY_FORWARD) {
    const size_t ch = (size_t)decay_chunks(p) * p.H;
    if (p.mode == SEQ_VARLEN) l.pre_d = c.take((size_t)(p.n_seq + 1) * 4);
    l.LF = c.take(ch * p.dh * state_ld(p.dh) * 2);
    l.LB = c.take(ch * p.dh * state_ld(p.dh) * 2);
    l.lamc = c.take(ch * 4);
    l.HF = c.take(ch * p.dh * state_bf_ld(p.dh) * 2);
    l.HB = c.take(ch * p.dh * state_bf_ld(p.dh) * 2);
  } else {  // core forward / backward
    l.state = c.take(state_bytes(p));
    l.state_bf = c.take(state_bf_bytes(p));
    l.state_m = c.take((size_t)p.n_seq * p.H * 4);
    l.center = c.take(center_bytes(p));
    if (op == GBLA_OP_CORE_BACKWARD) {
      l.dstate = c.take(state_bytes(p));
      l.dstate_bf = c.take(state_bf_bytes(p));
    }
  }
  l.total = c.off;
  return l;
}

template <typename T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(base) + off);
}

gbla_status cuda_fail(cudaError_t e, const char* what) {
  g_last_error = std::string(what) + ": " + cudaGetErrorString(e);
  return GBLA_ERR_CUDA;
}

// Per-launch timing (gbla_profiling_*): when on, every launch of this thread
// is bracketed by two CUDA events recorded on the call's stream.
struct ProfRecord { const char* name; cudaEvent_t t0, t1; };
struct Profiler {
  bool on = false;
  std::vector<ProfRecord> rec;
  std::vector<cudaEvent_t> pool;
  cudaEvent_t event() {
    if (!pool.empty()) { cudaEvent_t e = pool.back(); pool.pop_back(); return e; }
    cudaEvent_t e = nullptr;
    cudaEventCreate(&e);
    return e;
  }
};
thread_local Profiler g_prof;

#define GBLA_CHECK(call, what)                                         \
  do {                                                                 \
    cudaEvent_t t0_ = nullptr;                                         \
    if (g_prof.on) { t0_ = g_prof.event(); cudaEventRecord(t0_, c.st); } \
    cudaError_t e_ = (call);                                           \
    if (g_prof.on) {                                                   \
      cudaEvent_t t1_ = g_prof.event();                                \
      cudaEventRecord(t1_, c.st);                                      \
      g_prof.rec.push_back({what, t0_, t1_});                          \
    }                                                                  \
    if (e_ != cudaSuccess) return cuda_fail(e_, what);                 \
  } while (0)

struct Ctx {
  Plan p;
  Layout l;
  SeqDesc seq;
  Tiling chunks, tiles;
  int* err;          // workspace error word (always valid)
  const int* kerr;   // what the state / conv kernels read: err, or null in the dense form
  cudaStream_t st;
  int pre = 0;       // P holds [phi(q) | phi(k) | v | r] (the bf16 layer)
  // The error word and counters to clear, when the call's first kernel (the
  // weight pack) clears them instead of a memset; null once cleared.
  void* zero = nullptr;
  size_t zero_bytes = 0;
};

// The bf16 layer applies the feature map phi = elu + 1 to q and k in the
// projection epilogue, so the state kernels read phi(q) and phi(k) directly.
bool layer_pre(const Plan& p, const gbla_shape*) { return !p.f32; }

// zero_in_pack: the caller's first kernel is the weight pack, which then
// clears the error word and counters (dense batches: no sequence-data check
// runs before it).
gbla_status begin(const gbla_shape* s, int op, void* ws, size_t ws_bytes, void* stream, Ctx& c,
                  bool zero_in_pack = false) {
  gbla_status r = make_plan(s, c.p);
  if (r != GBLA_OK) return r;
  c.l = ws_layout(c.p, op);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0 || ws_bytes < c.l.total) return GBLA_ERR_WORKSPACE;
  c.st = static_cast<cudaStream_t>(stream);
  const Plan& p = c.p;
  c.seq.mode = p.mode;
  c.seq.n_seq = p.n_seq;
  c.seq.L = p.mode == SEQ_VARLEN ? p.T : p.L;
  c.seq.T = p.T;
  c.seq.lens = s->seq_lens;
  c.seq.cu = s->cu_seqlens;
  c.chunks.tile = p.chunk;
  c.chunks.per_seq = p.chunk_per_seq;
  c.chunks.prefix = p.mode == SEQ_VARLEN ? at<int32_t>(ws, c.l.pre_c) : nullptr;
  c.tiles.tile = p.tile;
  c.tiles.per_seq = p.tile_per_seq;
  c.tiles.prefix = p.mode == SEQ_VARLEN ? at<int32_t>(ws, c.l.pre_t) : nullptr;
  c.err = at<int>(ws, c.l.err);
  // Only the varlen and padded forms have sequence data to check on the
  // device; in the dense form the kernels skip the error-word read.
  c.kerr = p.mode == SEQ_DENSE ? nullptr : c.err;
  const size_t zero_bytes = c.l.cnt_b + (size_t)p.n_seq * p.H * 4 - c.l.err;
  if (zero_in_pack && p.mode == SEQ_DENSE) {
    c.zero = at<char>(ws, c.l.err);
    c.zero_bytes = zero_bytes;
  } else {
    GBLA_CHECK(cudaMemsetAsync(at<char>(ws, c.l.err), 0, zero_bytes, c.st), "memset");
  }
  if (p.mode != SEQ_DENSE) {
    const int ts[2] = {p.chunk, p.tile};
    int32_t* pre[2] = {const_cast<int32_t*>(c.chunks.prefix), const_cast<int32_t*>(c.tiles.prefix)};
    GBLA_CHECK(launch_plan(c.seq, p.mode == SEQ_VARLEN ? 2 : 0, ts, pre, c.err, c.st), "plan");
  }
  return GBLA_OK;
}

// ------------------------------------------------------ gated linear recurrence
// Sizes and workspace of glr_forward / glr_backward (their shape needs no heads).
struct GlrPlan {
  bool f32;
  int T, L, d, n_seq, mode, cut;
  int64_t pieces;  // saved states
};

gbla_status make_glr_plan(const gbla_shape* s, GlrPlan& p) {
  if (!s) return GBLA_ERR_INVALID_ARG;
  if (s->io_dtype != GBLA_F32 && s->io_dtype != GBLA_BF16) return GBLA_ERR_INVALID_ARG;
  if (s->B < 1 || s->L < 1 || s->d < 1) return GBLA_ERR_INVALID_ARG;
  if (s->cu_seqlens && (s->seq_lens || s->B != 1 || s->num_seqs < 1)) return GBLA_ERR_INVALID_ARG;
  const long long T = s->cu_seqlens ? (long long)s->L : (long long)s->B * s->L;
  if (T > (1LL << 30) || s->d > (1 << 20)) return GBLA_ERR_UNSUPPORTED;
  p.f32 = s->io_dtype == GBLA_F32;
  p.T = (int)T; p.L = s->L; p.d = s->d;
  p.mode = s->cu_seqlens ? SEQ_VARLEN : (s->seq_lens ? SEQ_PADDED : SEQ_DENSE);
  p.n_seq = s->cu_seqlens ? s->num_seqs : s->B;
  if ((long long)p.n_seq * p.d > (1LL << 38) || p.n_seq > (1 << 30)) return GBLA_ERR_UNSUPPORTED;
  // Slots, or packed sequences, one by one, or all rows as one stream, whose tiles of one round are neighbours and wait for one
  // another.  The stream is the faster one in few rounds, and where sequences fill too little of their tiles.  Measured, us
  // forward / backward as a stream against one by one, d = 512, bf16, rounds of tiles in brackets:
  //   dense   L = 64 [6] 65 / 106, 95 / 99;  L = 65 [6] 97 / 194, 95 / 179;  L = 100 [0] 22 / 34, 24 / 36, [6] 95 / 179, 69 / 122,
  //           [53] 1054 / 2228, 413 / 763;  L = 256 [6] 83 / 175, 52 / 99, [53] 908 / 2928, 280 / 544;  L = 512 [0] 19 / 35, 19 / 35
  //   padded  L = 200 [13] 176 / 371, 124 / 239
  //   packed  of 16 .. 128 rows (53 on the mean) [6] 104 / 192, 122 / 157, [13, d = 1024] 235 / 398, 214 / 274, [107] 2426 / 4755, 1541 / 1992;
  //           of 1 .. 64 (15) [107] 2691 / 6239, 5293 / 5508;  of 64 .. 256 (137) [1] 32 / 54, 42 / 61, [6] 87 / 176, 89 / 141,
  //           [26] 421 / 808, 257 / 421;  of 512 .. 2048 [3, d = 1024] 42 / 77, 48 / 77, [6] 69 / 132, 65 / 106, [27] 254 / 568, 171 / 289
  const long long rounds = T / kGlrRowsFwd * cdiv(p.d, 64) / (2LL * sm_count()), mean = T / p.n_seq;
  if (p.mode != SEQ_VARLEN)
    p.cut = p.L >= kGlrSlot || (p.L > kGlrRowsBwd && rounds >= 3) ? GLR_SLOTS : GLR_STREAM;
  else  // (the order of the chunks is made for calls of up to 8 M rows)
    p.cut = p.n_seq > 1 && T <= (8LL << 20) && ((mean >= 128 && rounds >= 6) || (mean >= 48 && rounds >= 13)) ? GLR_SEQS : GLR_STREAM;
  p.pieces = p.cut == GLR_SLOTS ? (int64_t)p.n_seq * cdiv(p.L, kGlrPiece)
             : p.cut == GLR_SEQS ? p.T / kGlrPiece + p.n_seq : cdiv(p.T, kGlrPiece);
  if (((long long)p.T / kGlrRowsBwd + p.n_seq + 1) * cdiv(p.d, 64) > 0x7fffffffLL) return GBLA_ERR_UNSUPPORTED;  // tiles are counted in 31 bits
  return GBLA_OK;
}

size_t glr_dp(const GlrPlan& p) { return (size_t)cdiv(p.d, 64) * 64; }
// n / d as (t + (n - t) / 2) >> s with t = the high word of n m (Granlund and Montgomery); s = -1: d = 1.
GlrDiv glr_div(uint32_t d) {
  int l = 0;
  while ((1ull << l) < d) ++l;
  return GlrDiv{(uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1), l - 1};
}
GlrTiles glr_tiles(const GlrPlan& p, int rows) {
  GlrTiles t{};
  t.cut = p.cut;
  t.rows = rows;
  t.by_cg = glr_div((uint32_t)cdiv(p.d, 64));
  t.by_seq = glr_div((uint32_t)p.n_seq);
  t.per_seq = p.cut == GLR_SLOTS ? cdiv(p.L, rows) : 0;
  t.n_chunks = p.cut == GLR_SLOTS ? t.per_seq * p.n_seq : p.cut == GLR_SEQS ? p.T / rows + p.n_seq : cdiv(p.T, rows);
  // word c of a slot or sequence whose rows begin at r, the s-th: r / rows + s + c; groups and larger groups alike
  // (none where no slot has a chunk behind one, a group, a larger group)
  const int s = p.cut == GLR_STREAM ? 1 : p.n_seq;
  auto words = [&](int chunks) { return p.cut == GLR_SLOTS && t.per_seq <= chunks ? 0 : p.T / (chunks * rows) + s; };
  t.n_words = words(1);
  t.n_groups = words(16);
  t.n_large = words(256);
  t.levels = p.cut == GLR_SEQS ? cdiv(p.T, rows) : 0;
  return t;
}
struct GlrLayout { size_t err, ticket, count, level, marks, zero_bytes, kd, order, words, n_words, part, n_part, part2, total; };
GlrLayout glr_layout(const GlrPlan& p, int op) {
  Cursor c;
  GlrLayout l{};
  const GlrTiles t = glr_tiles(p, op == GBLA_OP_GLR_FORWARD ? kGlrRowsFwd : kGlrRowsBwd);
  l.err = c.take(32);  // the error word, then the tile counter, then the number of ordered chunks
  l.ticket = l.err + 16;
  l.count = l.err + 24;
  if (p.cut == GLR_SEQS) l.level = c.take((size_t)t.levels * 4);
  else if (p.mode == SEQ_VARLEN) l.marks = c.take((size_t)cdiv(p.T, 64) * 8);
  l.zero_bytes = c.off;
  l.kd = c.take(glr_dp(p) * 4);
  if (p.cut == GLR_SEQS) l.order = c.take((size_t)t.n_chunks * 16);
  l.n_words = ((size_t)t.n_words + t.n_groups + t.n_large) * glr_dp(p);
  l.words = c.take(l.n_words * 8);
  if (op == GBLA_OP_GLR_BACKWARD) {
    l.n_part = (size_t)t.n_chunks * p.d;
    l.part = c.take(l.n_part * 4);
    l.part2 = c.take((size_t)kDlamRows * p.d * 4);
  }
  l.total = c.off;
  return l;
}

struct GlrCtx {
  GlrPlan p;
  GlrLayout l;
  GlrTiles t;
  int* level;
  GlrArgs a;
  int* err;
  cudaStream_t st;
};

// The arguments that both directions share; checks them and the sequence data.
gbla_status glr_begin(const gbla_shape* shape, int op, const void* x, const void* r, const void* i, int64_t ld,
                      const float* lam, float cc, int reverse, const float* h0, void* ws, size_t ws_bytes, void* stream,
                      GlrCtx& c) {
  gbla_status s = make_glr_plan(shape, c.p);
  if (s != GBLA_OK) return s;
  const GlrPlan& p = c.p;
  const size_t es = p.f32 ? 4 : 2;
  for (const void* q : {x, r, i})
    if (!q || reinterpret_cast<uintptr_t>(q) % es) return GBLA_ERR_INVALID_ARG;
  if (!lam || !aligned4(lam) || !aligned4(h0) || ld < p.d || !(cc > 0.f) || cc > 3e38f) return GBLA_ERR_INVALID_ARG;
  if (reverse != 0 && reverse != 1) return GBLA_ERR_INVALID_ARG;
  c.l = glr_layout(p, op);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0 || ws_bytes < c.l.total) return GBLA_ERR_WORKSPACE;
  c.st = static_cast<cudaStream_t>(stream);
  c.err = at<int>(ws, c.l.err);
  GlrArgs& a = c.a;
  a = GlrArgs{};
  a.x = x; a.r = r; a.i = i; a.ld = ld;
  a.lam = lam; a.c = cc; a.reverse = reverse; a.h0 = h0;
  a.d = p.d; a.pieces = p.cut == GLR_SLOTS ? cdiv(p.L, kGlrPiece) : 0;
  a.seq.mode = p.mode; a.seq.n_seq = p.n_seq; a.seq.L = p.mode == SEQ_VARLEN ? p.T : p.L; a.seq.T = p.T;
  a.seq.lens = shape->seq_lens; a.seq.cu = shape->cu_seqlens;
  a.err = p.mode == SEQ_DENSE ? nullptr : c.err;
  a.err_out = c.err;
  a.ticket = at<unsigned long long>(ws, c.l.ticket);
  a.marks = p.mode == SEQ_VARLEN && p.cut == GLR_STREAM ? at<uint64_t>(ws, c.l.marks) : nullptr;
  c.t = glr_tiles(p, op == GBLA_OP_GLR_FORWARD ? kGlrRowsFwd : kGlrRowsBwd);
  c.level = nullptr;
  if (p.cut == GLR_SEQS) {
    c.t.order = at<int4>(ws, c.l.order);
    c.t.n_order = at<int>(ws, c.l.count);
    c.level = at<int>(ws, c.l.level);
  }
  a.words = at<uint64_t>(ws, c.l.words);
  a.kd = at<float>(ws, c.l.kd);
  a.dp = (int64_t)glr_dp(p);
  return GBLA_OK;
}

// Clears the error word, the tile counter, the marks and the scan's words, forms c softplus(lam), checks the sequence data on
// the device, and orders the chunks of packed sequences.
gbla_status glr_prepare(GlrCtx& c) {
  if (c.p.mode != SEQ_DENSE) GBLA_CHECK(cudaMemsetAsync(c.err, 0, c.l.zero_bytes, c.st), "memset");
  GBLA_CHECK(launch_glr_prep(c.a, c.t, (int64_t)c.l.n_words, c.a.dlam_part ? (int64_t)c.l.n_part : 0, c.level, c.err, c.st), "glr prep");
  if (c.p.cut == GLR_SEQS) GBLA_CHECK(launch_glr_order(c.a, c.t, c.level, c.st), "glr order");
  return GBLA_OK;
}

// Dense rows without saved states: a thread for two channels of a sequence, row by row (true), or tiles.  The first takes a
// row's latency (0.28 us where the inputs are still in L2, 0.69 from memory: 0.55 for calls that read 8 MB at most, which may be
// either) or its bytes at 4.7 TB/s, the tiles 10 us and their values (slots padded to tiles, channels to 64) at a rate that goes by
// the cut, a million a us: 0.53 for slots (at most 6.6 TB/s), as one stream 0.33 where slots begin at tiles' borders and 0.3
// elsewhere, 0.1 where rows are not copied by TMA.  Measured on the device, us of this one against the tiles', d = 512, bf16:
// B = 16, L = 16 (in L2) 5.6 / 10.2, L = 40 26 / 10; B = 128, L = 32 23 / 12; B = 300, L = 40 32 / 34, L = 128 95 / 64, L = 2048
// 1453 / 555; B = 512, L = 64 52 / 60, L = 256 198 / 154; B = 1024, L = 300 283 / 463; B = 4096, L = 64 231 / 373, L = 256 899 / 1131;
// fp32: B = 150, L = 1024 679 / 198, B = 1024, L = 64 117 / 124, L = 256 455 / 362; d = 33: B = 300, L = 200 137 / 39, B = 4800
// 159 / 463.  Of 518 shapes five lose more than 1.3 times by it, 1.6 at most, none of them more than 6 us.
bool glr_step_is_faster(const GlrCtx& c) {
  const GlrPlan& p = c.p;
  const GlrArgs& a = c.a;
  const size_t es = p.f32 ? 4 : 2;
  uintptr_t bits = (uintptr_t)(a.ld * es) | (uintptr_t)(p.d * es);
  for (const void* q : {a.x, a.r, a.i}) bits |= reinterpret_cast<uintptr_t>(q);
  const double row = 4. * es * p.n_seq * p.d, latency = 0.75 * row * p.L <= 8e6 ? 0.55 : 0.69;
  const double rate = bits % 16 ? 0.1e6
                      : p.cut == GLR_SLOTS ? std::min(0.53e6, 6.6e6 / (4. * es))
                      : kGlrRowsFwd % p.L == 0 ? 0.33e6 : 0.3e6;
  const double rows = (double)p.n_seq * (p.cut == GLR_SLOTS ? (double)c.t.per_seq * kGlrRowsFwd : p.L);
  return 1.2 + p.L * std::max(latency, row / 4.7e6) <= 10. + rows * glr_dp(p) / rate;
}

// ------------------------------------------------------------ AdamW
// Arguments of one tensor; norm_only: what gbla_grad_norm reads.
bool adam_tensor_ok(const gbla_adamw_tensor& t, bool norm_only) {
  if (t.n < 0 || t.n > (1LL << 40)) return false;
  if (t.grad_dtype != GBLA_F32 && t.grad_dtype != GBLA_BF16) return false;
  if (t.n == 0) return true;
  auto ok = [](const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; };
  if (!ok(t.grad, t.grad_dtype == GBLA_F32 ? 4 : 2)) return false;
  if (norm_only) return true;
  if (t.param_dtype != GBLA_F32 && t.param_dtype != GBLA_BF16) return false;
  if (!ok(t.param, t.param_dtype == GBLA_F32 ? 4 : 2)) return false;
  if (t.master && (t.param_dtype == GBLA_F32 || !aligned4(t.master))) return false;
  if (!t.m_scale != !t.v_scale || !aligned4(t.m_scale) || !aligned4(t.v_scale)) return false;
  const size_t a = t.m_scale ? 1 : 4;
  return ok(t.m, a) && ok(t.v, a) && t.weight_decay >= 0. && t.weight_decay <= 1e30;
}

// Units of all tensors.
int64_t adam_units(const gbla_adamw_tensor* t, int n) {
  int64_t u = 0;
  for (int k = 0; k < n; ++k) u += (t[k].n + kAdamUnit - 1) / kAdamUnit;
  return u;
}
// The size of the launches' tables of tensors with values.
int adam_cap(const gbla_adamw_tensor* t, int n) {
  int live = 0;
  for (int k = 0; k < n; ++k) live += t[k].n > 0;
  return live <= kAdamFew ? kAdamFew : kAdamMany;
}

// The workspace: the error word (0: these calls find no error on the device), the step's scalars, the norm's partials.
constexpr size_t kAdamScalars = 64, kAdamParts = 256;
static_assert(kAdamScalars + sizeof(AdamScalars) <= kAdamParts, "");
// One fp64 partial for each CTA of each launch.
size_t adam_parts(const gbla_adamw_tensor* t, int n) {
  const int cap = adam_cap(t, n);
  return (size_t)(n / cap + 1) * adamw_ctas(std::max<int64_t>(1, adam_units(t, n)));
}

gbla_status adam_check(const gbla_adamw_tensor* t, int n, bool norm_only, void* ws, size_t ws_bytes) {
  if (n < 0 || (n > 0 && !t)) return GBLA_ERR_INVALID_ARG;
  for (int k = 0; k < n; ++k)
    if (!adam_tensor_ok(t[k], norm_only)) return GBLA_ERR_INVALID_ARG;
  if (adam_units(t, n) > (1LL << 30)) return GBLA_ERR_UNSUPPORTED;  // units are counted in 32 bits
  if (!ws || reinterpret_cast<uintptr_t>(ws) % kAlign || ws_bytes < kAdamParts + 8 * adam_parts(t, n))
    return GBLA_ERR_WORKSPACE;
  return GBLA_OK;
}

// fn(table) for each launch's table of at most N tensors.  The tensors without values are left out; norm_only: of each grad,
// grad_dtype and n alone.
template <int N, typename F>
gbla_status adam_tables(const gbla_adamw_tensor* t, int n, bool norm_only, double lr, F&& fn) {
  AdamTable<N> tab;
  tab.n = tab.units = 0;
  int64_t place = 0;
  for (int k = 0; k < n; ++k) {
    if (t[k].n > 0) {
      AdamTensor& o = tab.t[tab.n++];
      o = AdamTensor{};
      o.grad = t[k].grad; o.gb = t[k].grad_dtype == GBLA_BF16;
      o.n = t[k].n; o.place = place; o.first = tab.units;
      uintptr_t bits = reinterpret_cast<uintptr_t>(o.grad);
      if (!norm_only) {
        o.param = t[k].param; o.master = t[k].master; o.m = t[k].m; o.v = t[k].v;
        o.ms = t[k].m_scale; o.vs = t[k].v_scale;
        o.keep = (float)(1. - lr * t[k].weight_decay);
        o.pb = t[k].param_dtype == GBLA_BF16;
        for (const void* q : {(const void*)o.param, (const void*)o.master, (const void*)o.m, (const void*)o.v})
          bits |= reinterpret_cast<uintptr_t>(q);
      }
      o.vec = bits % 16 == 0;
      tab.units += (int)((t[k].n + kAdamUnit - 1) / kAdamUnit);
      place += (t[k].n + kAdamBlock - 1) / kAdamBlock * kAdamBlock;
    }
    if (tab.n == N || (k == n - 1 && tab.n > 0)) {
      const gbla_status r = fn(tab);
      if (r != GBLA_OK) return r;
      tab.n = tab.units = 0;
    }
  }
  return GBLA_OK;
}

struct AdamCtx { cudaStream_t st; };

template <int N>
gbla_status run_grad_norm(const gbla_adamw_tensor* t, int n, float* norm, void* ws, AdamCtx c) {
  double* part = at<double>(ws, kAdamParts);
  int parts = 0;
  const gbla_status r = adam_tables<N>(t, n, true, 0., [&](const AdamTable<N>& tab) {
    GBLA_CHECK(launch_sumsq<N>(tab, part + parts, c.st), "grad sumsq");
    parts += adamw_ctas(tab.units);
    return GBLA_OK;
  });
  if (r != GBLA_OK) return r;
  GBLA_CHECK(launch_norm(part, parts, norm, at<int>(ws, 0), c.st), "grad norm");
  return GBLA_OK;
}

template <int N>
gbla_status run_adamw(const gbla_adamw_tensor* t, int n, double lr, const AdamScalars* s, AdamCtx c) {
  return adam_tables<N>(t, n, false, lr, [&](const AdamTable<N>& tab) {
    GBLA_CHECK(launch_adamw<N>(tab, s, c.st), "adamw");
    return GBLA_OK;
  });
}

// State reduction + combine.  The bf16 path centres the state on the
// k~-weighted mean of v (center); the fp32 path keeps it uncentred.
// The layer's bf16 readout: the tcgen05 kernel where it applies.
// The mma.sync readout loads a (sequence, head) state per CTA: it takes a
// chunk of rows (up to 2048) per CTA, not a tile, so that the load is spread
// over more rows.  Every row is written by its own index, whatever the tiling.
cudaError_t launch_readout_chunks_bf16(const ReadoutArgs& ra, bool norm, const Tiling& chunks, int n_chunks,
                                       cudaStream_t st) {
  ReadoutArgs rc = ra;
  rc.tiles = chunks;
  return launch_readout_bf16(rc, norm, n_chunks, st);
}

// The core readout: tcgen05 where it applies (unless the policy asks for
// mma.sync), else the mma.sync kernel over the chunks.
cudaError_t launch_readout_core_bf16(const ReadoutArgs& ra, int n_tiles, const Tiling& chunks, int n_chunks,
                                     cudaStream_t st, const char** name) {
  if (g_policy != GBLA_POLICY_MMA) {
    const cudaError_t e = launch_readout_core_tc(ra, n_tiles, st);
    if (e != cudaErrorNotSupported) {
      *name = "readout[tc]";
      return e;
    }
    (void)cudaGetLastError();
  }
  *name = "readout[mma]";
  return launch_readout_chunks_bf16(ra, false, chunks, n_chunks, st);
}

cudaError_t launch_readout_layer_bf16(const ReadoutArgs& ra, int n_tiles, const Tiling& chunks, int n_chunks,
                                      cudaStream_t st, const char** nm) {
  if (g_policy != GBLA_POLICY_MMA) {
    *nm = "readout[tc]";
    const cudaError_t e = launch_readout_tc(ra, n_tiles, st);
    if (e != cudaErrorNotSupported) return e;
    (void)cudaGetLastError();
  }
  *nm = "readout[mma]";
  return launch_readout_chunks_bf16(ra, true, chunks, n_chunks, st);
}

// The layer's bf16 key-side backward: the tcgen05 kernel where it applies;
// *bg_rows = the rows of db_g partials written.
// The mma.sync key-side backward, like the readout, takes a chunk of rows per
// CTA (one load of [dS | dz] for up to 2048 rows).  Its db_g partials are one
// row per CTA: n_chunks <= 2 n_tiles rows, which the partial buffer holds.
cudaError_t launch_bwd_kv_chunks_bf16(const BwdKVArgs& kv, const Tiling& chunks, int n_chunks, cudaStream_t st) {
  BwdKVArgs kc = kv;
  kc.tiles = chunks;
  return launch_bwd_kv_bf16(kc, n_chunks, st);
}

// The core's query-side backward: tcgen05 where it applies (d_h = 64; unless
// the policy asks for mma.sync), else the mma.sync kernel.
cudaError_t launch_bwd_q_core_bf16(const BwdQArgs& q, int hd, int n_tiles, const Ctx& c, const char** nm) {
  if (g_policy != GBLA_POLICY_MMA) {
    int parts = 0;
    const cudaError_t e = launch_bwd_q_tc(q, hd, n_tiles, &parts, c.st);
    if (e != cudaErrorNotSupported) {
      *nm = "bwd_q[tc]";
      return e;
    }
    (void)cudaGetLastError();
  }
  *nm = "bwd_q[mma]";
  return launch_bwd_q_bf16(q, false, c.p.n_chunks, c.st);
}

// The core's key-side backward: tcgen05 where it applies (unless the policy
// asks for mma.sync), else the mma.sync kernel over the chunks.
cudaError_t launch_bwd_kv_core_bf16(const BwdKVArgs& kv, int n_tiles, const Ctx& c, const char** nm) {
  if (g_policy != GBLA_POLICY_MMA) {
    int parts = 0;
    const cudaError_t e = launch_bwd_kv_tc(kv, n_tiles, &parts, c.st);
    if (e != cudaErrorNotSupported) {
      *nm = "bwd_kv[tc]";
      return e;
    }
    (void)cudaGetLastError();
  }
  *nm = "bwd_kv[mma]";
  return launch_bwd_kv_chunks_bf16(kv, c.chunks, c.p.n_chunks, c.st);
}

cudaError_t launch_bwd_kv_layer_bf16(const BwdKVArgs& kv, int n_tiles, const Tiling& chunks, int n_chunks,
                                     int* bg_rows, cudaStream_t st, const char** nm) {
  if (g_policy != GBLA_POLICY_MMA) {
    *nm = "bwd_kv[tc]";
    const cudaError_t e = launch_bwd_kv_tc(kv, n_tiles, bg_rows, st);
    if (e != cudaErrorNotSupported) return e;
    (void)cudaGetLastError();
  }
  *nm = "bwd_kv[mma]";
  *bg_rows = n_chunks;
  return launch_bwd_kv_chunks_bf16(kv, chunks, n_chunks, st);
}

// The layer's bf16 query-side backward: the tcgen05 kernel where it applies.
// *gamma_rows = the rows of dgamma partials written.
cudaError_t launch_bwd_q_layer_bf16(const BwdQArgs& q, int hd, int n_chunks, int n_tiles, int* gamma_rows,
                                    cudaStream_t st, const char** nm) {
  if (g_policy != GBLA_POLICY_MMA) {
    *nm = "bwd_q[tc]";
    cudaError_t e = launch_bwd_q_tc(q, hd, n_tiles, gamma_rows, st);
    if (e != cudaErrorNotSupported) return e;
    (void)cudaGetLastError();
    e = launch_bwd_q_tc128(q, hd, n_tiles, gamma_rows, st);
    if (e != cudaErrorNotSupported) return e;
    (void)cudaGetLastError();
  }
  *nm = "bwd_q[mma]";
  *gamma_rows = n_chunks * q.H;
  return launch_bwd_q_bf16(q, true, n_chunks, st);
}

// The bf16 state reduction: the tcgen05 kernel where it applies (gate values,
// d_h = 64) and either each SM streams at least 20 of its 256-row tiles or
// phi(k) is not stored (the core entry points: the mma.sync kernel then
// applies phi in registers, 65 against 61 us at 13 tiles an SM), else the
// mma.sync kernel (softmax logits, other d_h; and shorter batches of the
// layer, where the tcgen05 kernel's fixed start and final drain outweigh its
// faster stream: measured 51 against 47 us at 13 tiles an SM, 80 against 81
// at 27, 129 against 132 at 54).
cudaError_t launch_reduce_layer_bf16(const ReduceArgs& a, int n_chunks, int n_tiles, int sms, cudaStream_t st,
                                     const char** nm) {
  const long long units = (long long)a.seq.T * a.H / 256;
  if (((units >= 20LL * sms || !a.pre) && g_policy != GBLA_POLICY_MMA) || g_policy == GBLA_POLICY_TC) {
    *nm = "reduce[tc]";
    const cudaError_t e = launch_reduce_tc(a, n_tiles, st);
    if (e != cudaErrorNotSupported) return e;
    (void)cudaGetLastError();
  }
  *nm = "reduce[mma]";
  return launch_reduce_bf16(a, n_chunks, st);
}

gbla_status run_reduce(Ctx& c, const void* k, const void* v, int64_t ld, const float* g, int gate_kind, float* state,
                       bf16* state_bf, float* state_m, float* pub_state, float* center, void* ws) {
  const Plan& p = c.p;
  ReduceArgs a{};
  a.k = k; a.v = v; a.ldk = ld; a.ldv = ld;
  a.g = g; a.ldg = p.H; a.gate_kind = gate_kind;
  a.H = p.H; a.dh = p.dh;
  a.seq = c.seq; a.chunks = c.chunks;
  a.partial = at<float>(ws, c.l.partial);
  a.partial_m = at<float>(ws, c.l.partial_m);
  a.counters = at<int>(ws, c.l.cnt_f);
  a.state = state; a.state_bf = state_bf; a.state_m = state_m; a.pub_state = pub_state;
  a.pre = c.pre;
  a.center = p.f32 ? nullptr : center;
  a.err = c.kerr;
  a.tiles = c.tiles;
  a.partial_slots = partial_slots(p);
  a.err_out = c.err;
  const char* nm = "reduce[f32]";
  GBLA_CHECK(p.f32 ? launch_reduce_f32(a, p.n_chunks, c.st) : launch_reduce_layer_bf16(a, p.n_chunks, p.n_tiles, p.sms, c.st, &nm),
             nm);
  return GBLA_OK;
}

}  // namespace

extern "C" {

gbla_status gbla_validate_shape(const gbla_shape* shape) {
  Plan p;
  return make_plan(shape, p);
}

size_t gbla_workspace_size(const gbla_shape* shape, int op) {
  if (op == GBLA_OP_GLR_FORWARD || op == GBLA_OP_GLR_BACKWARD) {
    GlrPlan g;
    return make_glr_plan(shape, g) == GBLA_OK ? glr_layout(g, op).total : 0;
  }
  Plan p;
  if (make_plan(shape, p) != GBLA_OK) return 0;
  if (op < GBLA_OP_FORWARD || op > GBLA_OP_SA_FORWARD) return 0;
  return ws_layout(p, op).total;
}

size_t gbla_saved_size(const gbla_shape* shape) {
  Plan p;
  if (make_plan(shape, p) != GBLA_OK) return 0;
  return saved_layout(p).total;
}

gbla_status gbla_forward(const gbla_shape* shape, const void* x, const void* conv_w, const void* conv_b,
                         const void* W_q, const void* W_k, const void* W_v, const void* W_r, const void* w_g,
                         const void* b_g, const void* rms_w, void* y, void* saved, void* ws, size_t ws_bytes,
                         void* stream) {
  Plan p0;
  gbla_status r = make_plan(shape, p0);
  if (r != GBLA_OK) return r;
  if ((r = check_layer_shape(p0)) != GBLA_OK) return r;
  const void* req[] = {x, conv_w, W_q, W_k, W_v, W_r, w_g, y};
  for (const void* q : req)
    if (!q || !aligned16(q)) return GBLA_ERR_INVALID_ARG;
  for (const void* q : {conv_b, b_g, rms_w})
    if (q && !aligned16(q)) return GBLA_ERR_INVALID_ARG;
  if (saved && (reinterpret_cast<uintptr_t>(saved) % kAlign) != 0) return GBLA_ERR_INVALID_ARG;
  Ctx c;
  if ((r = begin(shape, GBLA_OP_FORWARD, ws, ws_bytes, stream, c, true)) != GBLA_OK) return r;
  const Plan& p = c.p;
  const Layout& l = c.l;
  void *xt, *P;
  float *gate, *state, *state_m, *center;
  bf16* state_bf;
  if (saved) {
    const SavedLayout s = saved_layout(p);
    xt = at<char>(saved, s.xt); P = at<char>(saved, s.P); gate = at<float>(saved, s.gate);
    state = at<float>(saved, s.state); state_bf = at<bf16>(saved, s.state_bf); state_m = at<float>(saved, s.state_m);
    center = at<float>(saved, s.center);
  } else {
    xt = at<char>(ws, l.xt); P = at<char>(ws, l.P); gate = at<float>(ws, l.gate);
    state = at<float>(ws, l.state); state_bf = at<bf16>(ws, l.state_bf); state_m = at<float>(ws, l.state_m);
    center = at<float>(ws, l.center);
  }
  if (p.f32) center = nullptr;
  // packed weights first: the pack also clears the error word and counters (dense batches)
  const void* W[4] = {W_q, W_k, W_v, W_r};
  void* Wt = at<char>(ws, l.Wt);
  GBLA_CHECK(launch_pack_weights(W, w_g, p.d, p.H, p.dh, p.f32, Wt, p.NP, c.zero, c.zero_bytes, c.st), "pack");
  // Eq. 4: conv
  ConvArgs ca{};
  ca.x = x; ca.w = conv_w; ca.b = conv_b; ca.xt = xt; ca.T = p.T; ca.d = p.d; ca.seq = c.seq; ca.err = c.kerr; ca.err_out = c.err;
  int tiled = 0;
  GBLA_CHECK(launch_conv_fwd(ca, p.f32, c.st, &tiled), tiled ? "conv[bulk]" : "conv[plain]");
  c.pre = layer_pre(p, shape) ? 1 : 0;
  // Eq. 4, 5, 7: projections and gate
  GemmArgs ga{};
  ga.A = xt; ga.lda = p.d; ga.a_kmajor = 1;
  ga.B = Wt; ga.ldb = p.NP; ga.b_kmajor = 0;  // B(n, k) = W_all[k][n]: N-major
  ga.C = P; ga.ldc = 4 * p.HD;
  ga.M = p.T; ga.N = p.N1; ga.K = p.d; ga.k_split = (p.d + 31) / 32 * 32;
  ga.epi = c.pre ? EPI_PROJ_PRE : EPI_PROJ; ga.n_main = 4 * p.HD; ga.hd = p.HD; ga.dh = p.dh;
  ga.bias_g = shape->gate == GBLA_GATE_SIGMOID ? b_g : nullptr;
  ga.gate_mode = shape->gate == GBLA_GATE_SIGMOID ? 0 : 1; ga.gate = gate; ga.ldgate = p.H; ga.io_f32 = p.f32;
  ga.err = c.err;
  ga.pair = 1;  // CTA pairs: each CTA loads half of B, a third less operand traffic per SM
  int var = VAR_TC;
  GBLA_CHECK(launch_gemm(ga, c.st, &var), kGemmNames[0][var]);
  // Eq. 5/6: state
  const size_t es = p.io;
  const char* Pc = static_cast<const char*>(P);
  r = run_reduce(c, Pc + p.HD * es, Pc + 2 * p.HD * es, 4 * p.HD, gate,
                 shape->gate == GBLA_GATE_SIGMOID ? GATE_VALUES : GATE_LOGITS, state, state_bf, state_m, nullptr,
                 center, ws);
  if (r != GBLA_OK) return r;
  // Eq. 5/6 readout fused with Eq. 7
  ReadoutArgs ra{};
  ra.q = P; ra.ldq = 4 * p.HD;
  ra.r = Pc + 3 * p.HD * es; ra.ldr = 4 * p.HD;
  ra.rms_w = rms_w; ra.eps = shape->rms_eps;
  ra.state = state; ra.state_bf = state_bf; ra.center = center; ra.pre = c.pre;
  ra.out = y; ra.ldo = p.HD; ra.den = nullptr;
  ra.rsinv = (saved && !p.f32) ? at<float>(saved, saved_layout(p).rsinv) : nullptr;
  ra.H = p.H; ra.dh = p.dh; ra.seq = c.seq; ra.tiles = c.tiles; ra.err = c.kerr; ra.err_out = c.err;
  const char* nm = "readout[f32]";
  GBLA_CHECK(p.f32 ? launch_readout_f32(ra, true, p.n_tiles, c.st)
                   : launch_readout_layer_bf16(ra, p.n_tiles, c.chunks, p.n_chunks, c.st, &nm),
             nm);
  return GBLA_OK;
}

gbla_status gbla_backward(const gbla_shape* shape, const void* x, const void* conv_w, const void* conv_b,
                          const void* W_q, const void* W_k, const void* W_v, const void* W_r, const void* w_g,
                          const void* b_g, const void* rms_w, const void* saved, const void* dy, void* dx,
                          float* dconv_w, float* dconv_b, float* dW_q, float* dW_k, float* dW_v, float* dW_r,
                          float* dw_g, float* db_g, float* drms_w, void* ws, size_t ws_bytes, void* stream) {
  (void)conv_b; (void)b_g;
  Plan p0;
  gbla_status r = make_plan(shape, p0);
  if (r != GBLA_OK) return r;
  if ((r = check_layer_shape(p0)) != GBLA_OK) return r;
  const void* req[] = {x, conv_w, W_q, W_k, W_v, W_r, w_g, saved, dy, dx};
  for (const void* q : req)
    if (!q || !aligned16(q)) return GBLA_ERR_INVALID_ARG;
  if (rms_w && !aligned16(rms_w)) return GBLA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(saved) % kAlign) != 0) return GBLA_ERR_INVALID_ARG;
  Ctx c;
  if ((r = begin(shape, GBLA_OP_BACKWARD, ws, ws_bytes, stream, c, true)) != GBLA_OK) return r;
  const Plan& p = c.p;
  const Layout& l = c.l;
  const SavedLayout s = saved_layout(p);
  const size_t es = p.io;
  const char* P = at<const char>(const_cast<void*>(saved), s.P);
  const void* xt = at<const char>(const_cast<void*>(saved), s.xt);
  const float* gate = at<const float>(const_cast<void*>(saved), s.gate);
  char* dP = at<char>(ws, l.dP);
  const bool sig = shape->gate == GBLA_GATE_SIGMOID;
  const int pre = layer_pre(p, shape) ? 1 : 0;
  // gamma_part and bg_part: every CTA of bwd_q / bwd_kv writes its row (zeros when it has no rows)
  const void* W[4] = {W_q, W_k, W_v, W_r};
  GBLA_CHECK(launch_pack_weights(W, w_g, p.d, p.H, p.dh, p.f32, at<char>(ws, l.Wp), p.NP, c.zero, c.zero_bytes, c.st),
             "pack");
  // Eq. 7 + Eq. 5/6 query side: dr, dq, [dS | dz]
  BwdQArgs q{};
  q.q = P; q.ldq = 4 * p.HD;
  q.r = P + 3 * p.HD * es; q.ldr = 4 * p.HD;
  q.dy = dy; q.lddy = p.HD;
  q.rms_w = rms_w; q.eps = shape->rms_eps;
  q.state = at<const float>(const_cast<void*>(saved), s.state);
  q.state_bf = at<const bf16>(const_cast<void*>(saved), s.state_bf);
  const float* center = p.f32 ? nullptr : at<const float>(const_cast<void*>(saved), s.center);
  q.center = center;
  q.pre = pre;
  q.dq = dP; q.lddq = p.NP;
  q.dr = dP + 3 * p.HD * es; q.lddr = p.NP;
  q.gamma_part = at<float>(ws, l.gamma_part);
  q.partial = at<float>(ws, l.partial); q.counters = at<int>(ws, l.cnt_b);
  q.dstate = at<float>(ws, l.dstate); q.dstate_bf = at<bf16>(ws, l.dstate_bf);
  q.rsinv = at<const float>(const_cast<void*>(saved), s.rsinv);
  q.H = p.H; q.dh = p.dh; q.seq = c.seq; q.chunks = c.chunks; q.tiles = c.tiles; q.err = c.kerr; q.err_out = c.err;
  q.partial_slots = partial_slots(p);
  int gamma_rows = p.n_chunks * p.H;
  const char* nm = "bwd_q[f32]";
  GBLA_CHECK(p.f32 ? launch_bwd_q_f32(q, true, p.n_chunks, c.st)
                   : launch_bwd_q_layer_bf16(q, p.HD, p.n_chunks, p.n_tiles, &gamma_rows, c.st, &nm),
             nm);
  // key side: dk, dv, ds
  BwdKVArgs kv{};
  kv.k = P + p.HD * es; kv.ldk = 4 * p.HD;
  kv.v = P + 2 * p.HD * es; kv.ldv = 4 * p.HD;
  kv.g = gate; kv.ldg = p.H; kv.gate_kind = sig ? GATE_VALUES : GATE_LOGITS;
  kv.state_m = at<const float>(const_cast<void*>(saved), s.state_m);
  kv.dstate = at<float>(ws, l.dstate); kv.dstate_bf = at<bf16>(ws, l.dstate_bf);
  kv.center = center;
  kv.pre = pre;
  kv.dk = dP + p.HD * es; kv.lddk = p.NP;
  kv.dv = dP + 2 * p.HD * es; kv.lddv = p.NP;
  kv.ds = dP; kv.ldds = p.NP; kv.gate_grad = sig ? GG_SIGMOID : GG_SOFTMAX;
  // ds of head h lands in column 4*H*dh + h: offset the pointer, keep the stride
  kv.ds = dP + (size_t)4 * p.HD * es;
  kv.zero_cols_from = kv.zero_cols_to = 0;  // the pad columns of dP are never read
  kv.bg_part = at<float>(ws, l.bg_part);
  kv.H = p.H; kv.dh = p.dh; kv.seq = c.seq; kv.tiles = c.tiles; kv.err = c.kerr; kv.err_out = c.err;
  int bg_rows = p.n_tiles;
  nm = "bwd_kv[f32]";
  GBLA_CHECK(p.f32 ? launch_bwd_kv_f32(kv, p.n_tiles, c.st)
                   : launch_bwd_kv_layer_bf16(kv, p.n_tiles, c.chunks, p.n_chunks, &bg_rows, c.st, &nm),
             nm);
  // Eq. 4 projections backward: dx~ = dP W_all^T, dW_all = x~^T dP
  GemmArgs g1{};
  g1.A = dP; g1.lda = p.NP; g1.a_kmajor = 1;
  g1.B = at<char>(ws, l.Wp); g1.ldb = p.NP; g1.b_kmajor = 1;
  g1.C = at<char>(ws, l.dxt); g1.ldc = p.d;  // dx~ in the io dtype
  // K = N1, not the padded NP: the pad columns of dP and W_all are never read (the
  // tensor-core GEMM's loads zero-fill past N1), so nothing needs to clear them
  g1.M = p.T; g1.N = p.d; g1.K = p.N1; g1.k_split = p.N1; g1.epi = p.f32 ? EPI_F32 : EPI_BF16; g1.io_f32 = p.f32;
  g1.err = c.err;
  g1.pair = 1;  // long K: the operand feed limits, CTA pairs halve it per SM
  int var = VAR_TC;
  GBLA_CHECK(launch_gemm(g1, c.st, &var), kGemmNames[1][var]);
  GemmArgs g2{};
  g2.A = xt; g2.lda = p.d; g2.a_kmajor = 0;
  g2.B = dP; g2.ldb = p.NP; g2.b_kmajor = 0;
  g2.C = at<float>(ws, l.dW); g2.ldc = p.NP;
  g2.M = p.d; g2.N = p.N1; g2.K = p.T; g2.k_split = p.wsplit; g2.epi = EPI_SPLITK; g2.io_f32 = p.f32; g2.err = c.err;
  g2.pair = 1;  // long K: the operand feed limits, CTA pairs halve it per SM
  GBLA_CHECK(launch_gemm(g2, c.st, &var), kGemmNames[2][var]);

  // Eq. 4 conv backward
  ConvArgs ca{};
  ca.x = x; ca.w = conv_w; ca.dxt = at<char>(ws, l.dxt); ca.dx = dx; ca.part = at<float>(ws, l.conv_part);
  ca.T = p.T; ca.d = p.d; ca.seq = c.seq; ca.err = c.kerr; ca.err_out = c.err;
  int nparts = 0, tiled = 0;
  GBLA_CHECK(launch_conv_bwd(ca, p.f32, &nparts, c.st, &tiled), tiled ? "conv bwd[bulk]" : "conv bwd[plain]");
  // the parameter gradients from their partials, one launch: W_all, conv taps and bias, gamma, b_g
  ColsumJobs js{};
  js.sc.part = at<float>(ws, l.dW);  // and the split-K sum of the weight gradient
  js.sc.S = p.n_wsplit; js.sc.d = p.d; js.sc.np = p.NP; js.sc.H = p.H; js.sc.dh = p.dh;
  js.sc.out[0] = dW_q; js.sc.out[1] = dW_k; js.sc.out[2] = dW_v; js.sc.out[3] = dW_r; js.sc.out[4] = dw_g;
  if (dconv_w || dconv_b)
    js.j[js.n++] = ColsumJob{ca.part, nparts, (int64_t)p.d * 5, (int64_t)p.d * 5, (float*)dconv_w, (float*)dconv_b, 1};
  if (drms_w) js.j[js.n++] = ColsumJob{q.gamma_part, gamma_rows, p.dh, p.dh, (float*)drms_w, nullptr, 0};
  if (db_g) js.j[js.n++] = ColsumJob{kv.bg_part, bg_rows, p.H, p.H, (float*)db_g, nullptr, 0};
  GBLA_CHECK(launch_colsums(js, c.st), "param grads");
  return GBLA_OK;
}

gbla_status bla_core_forward(const gbla_shape* shape, const void* q, const void* k, const void* v, const float* g,
                             void* o, float* den, float* state, void* ws, size_t ws_bytes, void* stream) {
  for (const void* ptr : {q, k, v, (const void*)g, (const void*)o})
    if (!ptr || !aligned16(ptr)) return GBLA_ERR_INVALID_ARG;
  for (const void* ptr : {(const void*)den, (const void*)state})
    if (ptr && !aligned16(ptr)) return GBLA_ERR_INVALID_ARG;
  Ctx c;
  gbla_status r = begin(shape, GBLA_OP_CORE_FORWARD, ws, ws_bytes, stream, c);
  if (r != GBLA_OK) return r;
  const Plan& p = c.p;
  float* st = at<float>(ws, c.l.state);
  bf16* sbf = at<bf16>(ws, c.l.state_bf);
  float* center = p.f32 ? nullptr : at<float>(ws, c.l.center);
  r = run_reduce(c, k, v, p.HD, g, GATE_VALUES, st, sbf, at<float>(ws, c.l.state_m), state, center, ws);
  if (r != GBLA_OK) return r;
  ReadoutArgs ra{};
  ra.q = q; ra.ldq = p.HD;
  ra.state = st; ra.state_bf = sbf; ra.center = center;
  ra.out = o; ra.ldo = p.HD; ra.den = den;
  ra.H = p.H; ra.dh = p.dh; ra.seq = c.seq; ra.tiles = c.tiles; ra.err = c.kerr;
  const char* nm = "readout[f32]";
  GBLA_CHECK(p.f32 ? launch_readout_f32(ra, false, p.n_tiles, c.st)
                   : launch_readout_core_bf16(ra, p.n_tiles, c.chunks, p.n_chunks, c.st, &nm),
             nm);
  return GBLA_OK;
}

gbla_status bla_core_backward(const gbla_shape* shape, const void* q, const void* k, const void* v, const float* g,
                              const void* d_o, void* dq, void* dk, void* dv, float* dg, void* ws, size_t ws_bytes,
                              void* stream) {
  for (const void* ptr : {q, k, v, (const void*)g, d_o, (const void*)dq, (const void*)dk, (const void*)dv, (const void*)dg})
    if (!ptr || !aligned16(ptr)) return GBLA_ERR_INVALID_ARG;
  Ctx c;
  gbla_status r = begin(shape, GBLA_OP_CORE_BACKWARD, ws, ws_bytes, stream, c);
  if (r != GBLA_OK) return r;
  const Plan& p = c.p;
  float* st = at<float>(ws, c.l.state);
  bf16* sbf = at<bf16>(ws, c.l.state_bf);
  float* center = p.f32 ? nullptr : at<float>(ws, c.l.center);
  r = run_reduce(c, k, v, p.HD, g, GATE_VALUES, st, sbf, at<float>(ws, c.l.state_m), nullptr, center, ws);
  if (r != GBLA_OK) return r;
  BwdQArgs a{};
  a.q = q; a.ldq = p.HD; a.dy = d_o; a.lddy = p.HD;
  a.state = st; a.state_bf = sbf; a.center = center;
  a.dq = dq; a.lddq = p.HD;
  a.partial = at<float>(ws, c.l.partial); a.counters = at<int>(ws, c.l.cnt_b);
  a.dstate = at<float>(ws, c.l.dstate); a.dstate_bf = at<bf16>(ws, c.l.dstate_bf);
  a.H = p.H; a.dh = p.dh; a.seq = c.seq; a.chunks = c.chunks; a.tiles = c.tiles; a.err = c.kerr; a.err_out = c.err;
  a.partial_slots = partial_slots(p);
  const char* nmq = "bwd_q[f32]";
  GBLA_CHECK(p.f32 ? launch_bwd_q_f32(a, false, p.n_chunks, c.st) : launch_bwd_q_core_bf16(a, p.HD, p.n_tiles, c, &nmq),
             nmq);
  BwdKVArgs kv{};
  kv.k = k; kv.ldk = p.HD; kv.v = v; kv.ldv = p.HD;
  kv.g = g; kv.ldg = p.H; kv.gate_kind = GATE_VALUES;
  kv.dstate = a.dstate; kv.dstate_bf = a.dstate_bf; kv.center = center;
  kv.dk = dk; kv.lddk = p.HD; kv.dv = dv; kv.lddv = p.HD;
  kv.ds = dg; kv.ldds = p.H; kv.gate_grad = GG_DG;
  kv.H = p.H; kv.dh = p.dh; kv.seq = c.seq; kv.tiles = c.tiles; kv.err = c.kerr;
  const char* nm = "bwd_kv[f32]";
  GBLA_CHECK(p.f32 ? launch_bwd_kv_f32(kv, p.n_tiles, c.st) : launch_bwd_kv_core_bf16(kv, p.n_tiles, c, &nm), nm);
  return GBLA_OK;
}

gbla_status bla_decay_core_forward(const gbla_shape* shape, const void* q, const void* k, const void* v,
                                   const float* g, const float* lam, void* o, float* den, void* ws, size_t ws_bytes,
                                   void* stream) {
  for (const void* ptr : {q, k, v, (const void*)g, (const void*)lam, (const void*)o})
    if (!ptr || !aligned16(ptr)) return GBLA_ERR_INVALID_ARG;
  if (den && !aligned16(den)) return GBLA_ERR_INVALID_ARG;
  Plan p0;
  gbla_status r = make_plan(shape, p0);
  if (r != GBLA_OK) return r;
  if (p0.f32 || p0.dh != 64) return GBLA_ERR_UNSUPPORTED;
  Ctx c;
  if ((r = begin(shape, GBLA_OP_DECAY_FORWARD, ws, ws_bytes, stream, c)) != GBLA_OK) return r;
  const Plan& p = c.p;
  DecayArgs a{};
  a.q = q; a.k = k; a.v = v; a.ld = p.HD;
  a.g = g; a.lam = lam; a.ldg = p.H;
  a.o = o; a.den = den;
  a.LF = at<bf16>(ws, c.l.LF); a.LB = at<bf16>(ws, c.l.LB); a.Lam = at<float>(ws, c.l.lamc);
  a.HF = at<bf16>(ws, c.l.HF); a.HB = at<bf16>(ws, c.l.HB);
  a.H = p.H; a.dh = p.dh; a.seq = c.seq; a.err = c.kerr;
  a.tiles.tile = kDecayChunk;
  a.tiles.per_seq = p.mode == SEQ_VARLEN ? 0 : cdiv(p.L, kDecayChunk);
  a.tiles.prefix = p.mode == SEQ_VARLEN ? at<int32_t>(ws, c.l.pre_d) : nullptr;
  if (p.mode == SEQ_VARLEN) {
    const int ts[1] = {kDecayChunk};
    int32_t* pre[1] = {at<int32_t>(ws, c.l.pre_d)};
    GBLA_CHECK(launch_plan(c.seq, 1, ts, pre, c.err, c.st), "plan");
  }
  GBLA_CHECK(launch_decay_states(a, decay_chunks(p), c.st), "decay states[mma]");
  GBLA_CHECK(launch_decay_scan(a, p.n_seq, c.st), "decay scan");
  GBLA_CHECK(launch_decay_out(a, decay_chunks(p), c.st), "decay out[mma]");
  return GBLA_OK;
}

gbla_status sa_core_forward(const gbla_shape* shape, const void* q, const void* k, const void* v, void* o, void* ws,
                            size_t ws_bytes, void* stream) {
  for (const void* ptr : {q, k, v, (const void*)o})
    if (!ptr || !aligned16(ptr)) return GBLA_ERR_INVALID_ARG;
  Plan p0;
  gbla_status r = make_plan(shape, p0);
  if (r != GBLA_OK) return r;
  if (p0.f32 || p0.dh != 64) return GBLA_ERR_UNSUPPORTED;
  Ctx c;
  if ((r = begin(shape, GBLA_OP_SA_FORWARD, ws, ws_bytes, stream, c)) != GBLA_OK) return r;
  const Plan& p = c.p;
  SaArgs a{};
  a.q = q; a.k = k; a.v = v; a.o = o; a.ld = p.HD;
  a.H = p.H; a.dh = p.dh; a.seq = c.seq; a.err = c.kerr; a.err_out = c.err;
  a.tiles.tile = kSaBlock;
  a.tiles.per_seq = p.mode == SEQ_VARLEN ? 0 : cdiv(p.L, kSaBlock);
  a.tiles.prefix = p.mode == SEQ_VARLEN ? at<int32_t>(ws, c.l.pre_d) : nullptr;
  if (p.mode == SEQ_VARLEN) {
    const int ts[1] = {kSaBlock};
    int32_t* pre[1] = {at<int32_t>(ws, c.l.pre_d)};
    GBLA_CHECK(launch_plan(c.seq, 1, ts, pre, c.err, c.st), "plan");
  }
  GBLA_CHECK(launch_sa_fwd_tc(a, sa_blocks(p), c.st), "sa[tc]");
  return GBLA_OK;
}

size_t glr_saved_size(const gbla_shape* shape) {
  GlrPlan p;
  return make_glr_plan(shape, p) == GBLA_OK ? align_up((size_t)p.pieces * p.d * 4) : 0;
}

gbla_status glr_forward(const gbla_shape* shape, const void* x, const void* r, const void* i, int64_t ld,
                        const float* lam, float c_decay, int reverse, const float* h0, void* y, float* hT, void* saved,
                        void* ws, size_t ws_bytes, void* stream) {
  GlrCtx c;
  gbla_status s = glr_begin(shape, GBLA_OP_GLR_FORWARD, x, r, i, ld, lam, c_decay, reverse, h0, ws, ws_bytes, stream, c);
  if (s != GBLA_OK) return s;
  const size_t es = c.p.f32 ? 4 : 2;
  if (!y || reinterpret_cast<uintptr_t>(y) % es || !aligned4(hT)) return GBLA_ERR_INVALID_ARG;
  if (saved && reinterpret_cast<uintptr_t>(saved) % kAlign) return GBLA_ERR_INVALID_ARG;
  c.a.y = y; c.a.hT = hT; c.a.saved = static_cast<float*>(saved);
  if (c.p.mode == SEQ_DENSE && !saved && glr_step_is_faster(c)) {
    GBLA_CHECK(launch_glr_step(c.a, c.p.f32, c.err, c.st), "glr step");
    return GBLA_OK;
  }
  if ((s = glr_prepare(c)) != GBLA_OK) return s;
  GBLA_CHECK(launch_glr_fwd(c.a, c.t, c.p.f32, c.st), "glr fwd");
  if (hT && c.p.mode != SEQ_DENSE) GBLA_CHECK(launch_glr_empty(c.a, h0, hT, c.st), "glr empty");
  return GBLA_OK;
}

gbla_status glr_backward(const gbla_shape* shape, const void* x, const void* r, const void* i, int64_t ld,
                         const float* lam, float c_decay, int reverse, const float* h0, const void* saved,
                         const void* dy, const float* dhT, void* dx, void* dr, void* di, int64_t ldd, float* dlam,
                         float* dh0, void* ws, size_t ws_bytes, void* stream) {
  GlrCtx c;
  gbla_status s = glr_begin(shape, GBLA_OP_GLR_BACKWARD, x, r, i, ld, lam, c_decay, reverse, h0, ws, ws_bytes, stream, c);
  if (s != GBLA_OK) return s;
  const size_t es = c.p.f32 ? 4 : 2;
  for (const void* q : {dy, (const void*)dx, (const void*)dr, (const void*)di})
    if (!q || reinterpret_cast<uintptr_t>(q) % es) return GBLA_ERR_INVALID_ARG;
  if (!saved || reinterpret_cast<uintptr_t>(saved) % kAlign) return GBLA_ERR_INVALID_ARG;
  if (!aligned4(dhT) || !aligned4(dlam) || !aligned4(dh0) || ldd < c.p.d) return GBLA_ERR_INVALID_ARG;
  GlrArgs& a = c.a;
  a.saved = static_cast<float*>(const_cast<void*>(saved));
  a.dy = dy; a.dhT = dhT; a.dx = dx; a.dr = dr; a.di = di; a.ldd = ldd; a.dh0 = dh0;
  a.dlam_part = dlam ? at<float>(ws, c.l.part) : nullptr;
  if ((s = glr_prepare(c)) != GBLA_OK) return s;
  const GlrTiles& t = c.t;
  GBLA_CHECK(launch_glr_bwd(a, t, c.p.f32, c.st), "glr bwd");
  if (dlam) GBLA_CHECK(launch_glr_dlam(a, t.n_chunks, at<float>(ws, c.l.part2), dlam, c.st), "glr dlam");
  if (dh0 && c.p.mode != SEQ_DENSE) GBLA_CHECK(launch_glr_empty(a, dhT, dh0, c.st), "glr empty");
  return GBLA_OK;
}

size_t gbla_adamw_workspace_size(const gbla_adamw_tensor* tensors, int n_tensors) {
  if (n_tensors < 0 || (n_tensors > 0 && !tensors)) return 0;
  for (int k = 0; k < n_tensors; ++k)
    if (tensors[k].n < 0 || tensors[k].n > (1LL << 40)) return 0;
  return align_up(kAdamParts + 8 * adam_parts(tensors, n_tensors));
}

gbla_status gbla_grad_norm(const gbla_adamw_tensor* tensors, int n_tensors, float* norm, void* ws, size_t ws_bytes,
                           void* stream) {
  const gbla_status r = adam_check(tensors, n_tensors, true, ws, ws_bytes);
  if (r != GBLA_OK) return r;
  if (!norm || !aligned4(norm)) return GBLA_ERR_INVALID_ARG;
  const AdamCtx c{static_cast<cudaStream_t>(stream)};
  return adam_cap(tensors, n_tensors) == kAdamFew ? run_grad_norm<kAdamFew>(tensors, n_tensors, norm, ws, c)
                                                  : run_grad_norm<kAdamMany>(tensors, n_tensors, norm, ws, c);
}

gbla_status gbla_adamw_step(const gbla_adamw_tensor* tensors, int n_tensors, const gbla_adamw_config* config,
                            int64_t* step, const float* norm, void* ws, size_t ws_bytes, void* stream) {
  const gbla_status r = adam_check(tensors, n_tensors, false, ws, ws_bytes);
  if (r != GBLA_OK) return r;
  if (!config || !step || reinterpret_cast<uintptr_t>(step) % 8 || !aligned4(norm)) return GBLA_ERR_INVALID_ARG;
  const gbla_adamw_config& g = *config;
  auto in = [](double v, double lo, double hi) { return v >= lo && v <= hi; };  // false for NaN
  if (!in(g.lr, 0., 1e30) || !in(g.beta1, 0., 0.9999999) || !in(g.beta2, 0., 0.9999999) || !in(g.eps, 1e-30, 1e30) ||
      !in(g.max_norm, 0., 1e30) || (g.max_norm > 0. && !norm))
    return GBLA_ERR_INVALID_ARG;
  const AdamCtx c{static_cast<cudaStream_t>(stream)};
  AdamScalars* s = at<AdamScalars>(ws, kAdamScalars);
  AdamStep a{g.lr, g.beta1, g.beta2, g.eps, g.max_norm, std::log(g.beta1), std::log(g.beta2), g.seed};  // beta = 0: -inf
  GBLA_CHECK(launch_adamw_begin(a, step, norm, s, at<int>(ws, 0), c.st), "adamw begin");
  return adam_cap(tensors, n_tensors) == kAdamFew ? run_adamw<kAdamFew>(tensors, n_tensors, g.lr, s, c)
                                                  : run_adamw<kAdamMany>(tensors, n_tensors, g.lr, s, c);
}

gbla_status gbla_check_device_status(const void* ws, void* stream) {
  if (!ws) return GBLA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int err = 0;
  cudaError_t e = cudaMemcpyAsync(&err, ws, sizeof(int), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "check_device_status");
  if (err & 1) return GBLA_ERR_DEVICE_CHECK;
  if (err & kErrTimeout) return GBLA_ERR_DEVICE_TIMEOUT;
  return err ? GBLA_ERR_DEVICE_CHECK : GBLA_OK;
}

gbla_status gbla_diag_bounded_wait(void* ws, size_t ws_bytes, unsigned polls, void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0 || ws_bytes < 16) return GBLA_ERR_WORKSPACE;
  if (polls < 1 || polls > (1u << 20)) return GBLA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int), st);
  if (e == cudaSuccess) e = launch_diag_wait(static_cast<int*>(ws), polls, st);
  if (e != cudaSuccess) return cuda_fail(e, "diag_bounded_wait");
  return GBLA_OK;
}

const char* gbla_status_string(int status) {
  switch (status) {
    case GBLA_OK: return "GBLA_OK";
    case GBLA_ERR_INVALID_ARG: return "GBLA_ERR_INVALID_ARG: null or misaligned pointer, or bad dimension";
    case GBLA_ERR_UNSUPPORTED: return "GBLA_ERR_UNSUPPORTED: no kernel for this shape (d_h, d alignment or size)";
    case GBLA_ERR_WORKSPACE: return "GBLA_ERR_WORKSPACE: workspace NULL, not 256-byte aligned, or too small";
    case GBLA_ERR_CUDA: return "GBLA_ERR_CUDA: a CUDA call failed (see gbla_last_error)";
    case GBLA_ERR_DEVICE_CHECK: return "GBLA_ERR_DEVICE_CHECK: bad cu_seqlens / seq_lens detected on the device";
    case GBLA_ERR_DEVICE_TIMEOUT:
      return "GBLA_ERR_DEVICE_TIMEOUT: a kernel's bounded wait for its copies or MMAs gave up; results are invalid";
    default: return "unknown gbla_status";
  }
}

const char* gbla_last_error(void) { return g_last_error.c_str(); }

void gbla_profiling_enable(int on) { g_prof.on = on != 0; }

gbla_status gbla_set_kernel_policy(int policy) {
  if (policy != GBLA_POLICY_AUTO && policy != GBLA_POLICY_TC && policy != GBLA_POLICY_MMA) return GBLA_ERR_INVALID_ARG;
  g_policy = policy;
  return GBLA_OK;
}

int gbla_profiling_read(const char** names, float* ms, int cap) {
  const int n = (int)g_prof.rec.size();
  if (n > 0) cudaEventSynchronize(g_prof.rec.back().t1);
  for (int i = 0; i < n; ++i) {
    ProfRecord& r = g_prof.rec[i];
    if (i < cap) {
      float t = -1.f;
      if (cudaEventElapsedTime(&t, r.t0, r.t1) != cudaSuccess) t = -1.f;
      if (names) names[i] = r.name;
      if (ms) ms[i] = t;
    }
    g_prof.pool.push_back(r.t0);
    g_prof.pool.push_back(r.t1);
  }
  g_prof.rec.clear();
  return n;
}

int gbla_version(void) { return 100; }

}  // extern "C"
