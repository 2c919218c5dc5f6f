// Internal interface between the C-ABI front end of the operators around the
// recurrence (kda_layer_api.cpp, plain C++) and the HIP translation units
// that hold their kernels: the short convolution, the selective scan and the
// norm of queries and keys.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace kda {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A launch has less than 2^32 threads along its first dimension.
inline bool grid_fits(int64_t groups, int64_t threads) { return groups <= (int64_t)UINT32_MAX / threads; }

// ---- short convolution ---------------------------------------------------
// One wave owns 64 vectors of channels and `tile` tokens, one workgroup
// kConvWaves such tiles in a row.
constexpr int kConvWaves = 4;
constexpr int kConvBatch = 8;  // token rows a wave loads before it uses them (forward 21.5 us; 22.6 with 4)

struct ConvArgs {
  const void* x;
  int64_t ld;
  const float* w;
  const float* bias;
  const void* init;
  const int32_t* cu;  // null: rows of T tokens
  int n_seqs;
  int64_t T, tokens;
  int D;
  int tile;
  int64_t n_part;  // workgroups along the tokens
};

// Tokens per wave: the longest tile (less of the window is read twice, and
// backward fewer partial sums are left) that still leaves `waves` waves.
// Forward over 4096 tokens of 6144 channels in bf16: 21.5 us with tiles of at
// most 16 tokens, 24.5 with 8, 21.6 with 32; backward over 2 x 4096 tokens of
// 4096 channels: 49 us with 64, 57 with 32, 49 with 128 (half the partial
// sums but no more time won, and short batches lose waves).  1024 waves in
// place of 2048 measure the same, 4096 cost 24.5 and 56.6 us.
inline int conv_tile(int64_t tokens, int64_t channel_waves, int longest, int64_t waves) {
  int tile = longest;
  while (tile > kConvBatch && channel_waves * ceil_div(tokens, tile) < waves) tile /= 2;
  return tile;
}

int launch_conv_forward(int is_bf16, int width, int silu, const ConvArgs& a, void* y, void* fin, void* stream);
int launch_conv_step(int is_bf16, int width, int silu, const ConvArgs& a, void* state, void* y, void* stream);
int launch_conv_backward(int is_bf16, int width, int silu, const ConvArgs& a, const void* dy, const void* dfin,
                         void* dx, float* dw, float* db, void* dinit, float* part, void* stream);

// Channels of one vector in the forward and in the backward pass.
constexpr int conv_vec(bool bf16, bool backward) { return bf16 && !backward ? 8 : 4; }
inline int64_t conv_channel_waves(int D, int vec) { return ceil_div(D < vec ? D : ceil_div(D, vec), 64); }
inline int conv_forward_tile(int is_bf16, int64_t tokens, int D) {
  return conv_tile(tokens, conv_channel_waves(D, conv_vec(is_bf16, false)), 16, 2048);
}
inline int conv_backward_tile(int64_t tokens, int D) {
  return conv_tile(tokens, conv_channel_waves(D, conv_vec(false, true)), 64, 2048);
}
// Partial sums of dweight and dbias: one row of (width + 1) * D floats per
// workgroup along the tokens.
inline int64_t conv_parts(int64_t tokens, int tile) { return ceil_div(ceil_div(tokens, tile), kConvWaves); }

// ---- selective scan --------------------------------------------------------
// A call cuts the tokens of the whole batch into slots of `slot` tokens (a
// multiple of kScanTile, unless rows are the slots); each workgroup scans one
// slot of its channels.  The forward scans give a wave 16
// channels, the backward scan 4 (whose lanes hold scan_ns(N) states each).
constexpr int kScanMaxStates = 64;
constexpr int kScanTile = 64;  // tokens of B and C staged at once (forward)
inline int scan_ns(int N) { return N <= 16 ? 1 : N <= 32 ? 2 : 4; }

struct ScanArgs {
  const void *x, *dt, *z, *Bm, *Cm;
  int64_t ld_x, ld_dt, ld_z, ld_b, ld_c;
  const float *A, *skip, *bias, *h0;
  const int32_t* cu;  // null: rows of T tokens
  int n_seqs;
  int64_t T, tokens;
  int D, N, G, softplus;
  int has_z;  // 0: z is x again, loaded and not used
  int64_t slot, n_slots;
  int blocks_per_group;  // workgroups over the channels of one group
};

// Workspace of a forward call: the state that every slot hands on, its sum of
// delta, and a word that says what passes through it.
struct ScanPlan {
  int64_t slot, n_slots;
  bool carry;  // some sequence may pass from one slot to the next
  size_t hend_off, sum_off, kind_off, ws_bytes;
};
constexpr int kScanWaves = 4;  // waves per workgroup (forward)

inline ScanPlan plan_scan(int64_t tokens, int rows, int64_t T, bool packed, int D, int N, int G, int n_cu) {
  ScanPlan p{};
  const int64_t cus = n_cu > 0 ? n_cu : 256;
  const int64_t waves = (int64_t)G * ceil_div(D / G, 16);  // of one slot
  if (tokens == 0) {
    p.slot = 1;
    p.n_slots = 1;
  } else if (!packed && waves * rows >= 4 * cus) {
    // The rows alone put a wave on every SIMD: no slots to chain, a token is
    // scanned once.  Rows of 2048 tokens of 2048 channels, bf16, as slots and
    // cut: 6 of them (3 waves a compute unit) 226 and 191 us, 8 (4) 226 and 237,
    // 16 332 and 428; rows of 1000 tokens of 4096: 3 of them (3) 111 and 105, 6
    // (6) 167 and 193.
    p.slot = T;
    p.n_slots = rows;
  } else {
    // waves for 32 a compute unit, twice what it holds at once.  1 x 4096
    // tokens of 4096 channels, bf16: 135 us; with 16, 138; 8, 155; 64, 142
    // (packed 20011 tokens of 771 channels, fp32: 169, 171, 208, 169 us)
    int64_t n = 32 * cus / waves;
    if (n > tokens / 64) n = tokens / 64;
    if (n > 512) n = 512;
    if (n < 1) n = 1;
    p.slot = ceil_div(ceil_div(tokens, n), kScanTile) * kScanTile;
    p.n_slots = ceil_div(tokens, p.slot);
  }
  p.carry = p.n_slots > 1 && (packed || p.slot % T != 0);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  const size_t slots = p.carry ? (size_t)p.n_slots : 0;
  p.hend_off = take(slots * D * N * 4);
  p.sum_off = take(slots * D * 4);
  p.kind_off = take(slots * 4);
  p.ws_bytes = off;
  return p;
}

int launch_scan_forward(int is_bf16, const ScanArgs& a, const ScanPlan& p, void* o, float* ht, void* ws, void* stream);
int launch_scan_step(int is_bf16, const ScanArgs& a, float* state, void* o, void* stream);

// One token: lanes of a channel, four states each, and sequences a lane:
// several, whose rates are then loaded once, where that leaves 16 waves a
// compute unit (256 sequences, 4096 channels, 16 states: 22.5 us with three
// sequences a lane, 23.4 with two, 25.7 with four, 25.4 with one).
constexpr int kScanStepSeqs = 3;
inline int scan_step_lanes(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
inline int scan_step_seqs(int64_t tokens, int D, int N) {
  return tokens * D * scan_step_lanes(N) >= (int64_t)kScanStepSeqs * 256 * 16 * 64 ? kScanStepSeqs : 1;
}

// Waves per workgroup of the backward scan; each workgroup leaves dB and dC of
// its 16 channels as one row of partial sums.  (8 waves leave half the rows,
// but measured 13 % slower: the barrier of every 16 tokens then holds up
// twice as many, and three waves a SIMD no longer divide evenly.)
constexpr int kScanBwdWaves = 4;

struct ScanBwdPlan {
  int64_t slot, n_slots;
  bool carry;
  int blocks_per_group;
  // byte offsets: state at the slots' ends and gradient at their starts, sum
  // of delta, what passes through; state before every group of 16 tokens and
  // sum of delta up to it; per-slot sums of dA, dskip and ddt_bias;
  // per-workgroup sums of dB and dC
  size_t hend_off, adj_off, sum_off, kind_off, group_off, group_sum_off, da_off, dskip_off, dbias_off, db_off, dc_off,
      ws_bytes;
};

inline ScanBwdPlan plan_scan_backward(int64_t tokens, int rows, int D, int N, int G) {
  ScanBwdPlan p{};
  // Slots for about 4096 waves of 16 channels, and 64 tokens at least.  2 x
  // 2048 tokens of 2048 channels: 240 us, with 2048 waves 240, with 8192 258; of
  // 1024 channels 137 and, with 2048, 130; packed 8192 tokens of 1024 channels
  // in fp32: 267, 257, 291; 2 x 2048 tokens of 4096 channels with 4 states: 380
  // and, with 2048, 390.
  const int64_t waves = (int64_t)G * ceil_div(D / G, 16);
  int64_t n = 4096 / waves;
  if (n > tokens / kScanTile) n = tokens / kScanTile;
  if (n < 1) n = 1;
  p.slot = tokens > 0 ? ceil_div(ceil_div(tokens, n), kScanTile) * kScanTile : kScanTile;
  p.n_slots = tokens > 0 ? ceil_div(tokens, p.slot) : 1;
  p.carry = p.n_slots > 1;
  p.blocks_per_group = (int)ceil_div(D / G, 4 * kScanBwdWaves);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  const size_t slots = (size_t)p.n_slots, dn = (size_t)D * N * 4, between = p.carry ? slots : 0;
  // every range of tokens starts a group: at most one range per sequence and slot
  const size_t groups = tokens > 0 ? (size_t)(tokens / 16 + rows + p.n_slots + 1) : 0;
  p.hend_off = take(between * dn);
  p.adj_off = take(between * dn);
  p.sum_off = take(between * D * 4);
  p.kind_off = take(between * 4);
  p.group_off = take(groups * dn);
  p.group_sum_off = take(groups * D * 4);
  p.da_off = take(slots * dn);
  p.dskip_off = take(slots * D * 4);
  p.dbias_off = take(slots * D * 4);
  p.db_off = take((size_t)p.blocks_per_group * tokens * G * N * 4);
  p.dc_off = take((size_t)p.blocks_per_group * tokens * G * N * 4);
  p.ws_bytes = off;
  return p;
}

// Workgroups of a scan's launches: the forward scans and the backward pass's
// states, 16 channels a wave; the backward pass's own.
inline int64_t scan_groups(int64_t n_slots, int D, int G) {
  return n_slots * G * ceil_div(D / G, 16 * kScanWaves);
}
inline bool scan_fits(const ScanPlan& p, int D, int G) {
  return grid_fits(scan_groups(p.n_slots, D, G) + 7, 64 * kScanWaves);
}
inline bool scan_backward_fits(const ScanBwdPlan& p, int64_t tokens, int D, int N, int G) {
  return grid_fits(scan_groups(p.n_slots, D, G) + 7, 64 * kScanWaves) &&
         grid_fits(p.n_slots * G * p.blocks_per_group + 7, 64 * kScanBwdWaves) &&
         grid_fits(ceil_div((int64_t)D * N + 2 * (int64_t)D, 64), 1024) &&  // sums over the slots
         grid_fits(ceil_div(tokens * G * N, 256), 256);                     // and over the channels
}

struct ScanGrads {
  const void* dout;
  const float* dht;
  void *dx, *ddt, *dz, *dB, *dC;
  float *dA, *dskip, *dbias, *dh0;
};

int launch_scan_backward(int is_bf16, const ScanArgs& a, const ScanBwdPlan& p, const ScanGrads& g, void* ws,
                         void* stream);

// ---- norm of queries and keys ----------------------------------------------
struct NormArgs {
  const void *q, *k;
  int64_t ld_q, ld_k;
  const float *wq, *wk;
  const int32_t* pos;
  const float* freq;
  int n_tokens, Hq, Hk, d, rot;
  int interleaved;
  float sum_factor;  // 1 (unit) or 1 / d (rms)
  float eps, q_scale;
};

// Four pairs a lane when neither the head nor its rotated part ends inside
// such a group, else single pairs (8192 tokens of 32 + 8 heads of 128, half
// rotated, bf16: 32 us, with single pairs 54; backward of 16 + 4 heads of 64
// the same 34 us in fp32, 27 in bf16, either way); lanes per head the power of two that
// covers the head (64 at most: single pairs of wide heads then come in chunks).
inline bool norm_four_pairs(int d, int rot) { return d % 8 == 0 && rot % 8 == 0; }
inline int norm_head_lanes(int d, int rot) {
  const int wanted = norm_four_pairs(d, rot) ? d / 8 : d / 2;
  int lanes = norm_four_pairs(d, rot) ? 4 : 16;
  while (lanes < 64 && lanes < wanted) lanes *= 2;
  return lanes;
}
// groups of heads, a wave each at a time, that a token has: those of q, then those of k
inline int norm_groups(int Hq, int Hk, int head_lanes) {
  const int per = 64 / head_lanes;
  return (Hq + per - 1) / per + (Hk + per - 1) / per;
}
// Groups of heads a wave takes of a token: up to 16 (its angles serve them
// all: rotated forward 33.0 us with 16, 38.9 with 8, 41.1 with 4), while
// `waves` waves are left.
inline int norm_steps(int n_tokens, int groups, int64_t waves) {
  int steps = groups < 16 ? groups : 16;
  while (steps > 1 && n_tokens * ceil_div(groups, steps) < waves) steps = (steps + 1) / 2;
  return steps;
}
constexpr int kNormMinWaves = 4096;
constexpr int kNormForwardWaves = 4;  // waves per workgroup (forward)
inline bool norm_forward_fits(const NormArgs& a) {
  const int groups = norm_groups(a.Hq, a.Hk, norm_head_lanes(a.d, a.rot));
  const int64_t per_token = ceil_div(groups, norm_steps(a.n_tokens, groups, kNormMinWaves));
  return grid_fits(ceil_div(a.n_tokens * per_token, kNormForwardWaves), 64 * kNormForwardWaves);
}

// Workgroups of the backward pass at most (a power of two); each leaves a row
// of d floats of partial sums for each of the weights' gradients.  One on
// every compute unit: twice as many measured 40 us against 34 (8192 tokens of
// 16 + 4 heads of 64, fp32).
constexpr int kNormParts = 256;

int launch_norm_forward(int is_bf16, const NormArgs& a, void* qo, void* ko, void* stream);
int launch_norm_backward(int is_bf16, const NormArgs& a, const void* dqo, const void* dko, void* dq, void* dk,
                         float* dwq, float* dwk, float* part, void* stream);

}  // namespace kda
