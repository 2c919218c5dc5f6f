// Internal interface between the C-ABI front end (kda_block_api.cpp, plain
// C++) and the HIP translation unit of linear attention with a decay for each
// head (kda_linear_attn.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kda_layer.h"

namespace kda {

constexpr int kLinearMaxDim = 128;  // channels of a head, d_k and d_v
constexpr int kLinearChunk = 64;    // tokens that one matrix product takes at most

struct LinearArgs {
  const void *q, *k, *v, *g;  // g: log decays [tokens, H], null without
  const float* decay;         // log decays [H], null without
  int64_t ld_q, ld_k, ld_v, ld_g;
  const float* h0;
  const int32_t* cu;  // null: rows of T tokens
  int n_seqs;
  int64_t T, tokens;
  int Hq, H, dk, dv;
  float scale;
  int64_t slot;
  int n_slots;
};

// A call cuts the tokens of the whole batch into slots; a workgroup scans one
// slot of one head.  `carry`: a sequence may pass from one slot to the next,
// so the state that every slot hands on is composed first.
struct LinearPlan {
  int64_t slot, n_slots;
  bool carry;
  // byte offsets.  Per slot and head: the state at its end, the gradient of
  // the state at its start, the sum of its log decays; per slot what passes
  // through; backward, per token and head, what the decays' gradients are
  // suffix sums of (a query's and a key's part), per slot and head and per
  // sequence and head what they start from; the gradients of shared queries
  // and keys by head.
  size_t end_off, adj_off, sum_off, kind_off, dot_q_off, dot_k_off, slot_dot_off, seq_dot_off, dq_off, dk_off, ws_bytes;
};

// The kernels' tiles hold 64 or 128 channels of either kind; so do the states
// in the workspace.
constexpr int linear_pad(int d) { return d <= 64 ? 64 : 128; }
// Workgroups that a compute unit holds, by the tiles' channels.
constexpr int linear_groups_of_unit(int dk, int dv) { return dk <= 64 && dv <= 64 ? 3 : 2; }
constexpr size_t linear_record(int dk, int dv) { return (size_t)linear_pad(dk) * linear_pad(dv); }

inline LinearPlan plan_linear(int64_t tokens, int rows, int64_t T, bool packed, int H, int n_cu, int dk, int dv,
                              bool backward) {
  LinearPlan p{};
  const int64_t cus = n_cu > 0 ? n_cu : 256;
  dk = linear_pad(dk);
  dv = linear_pad(dv);
  const size_t record = (size_t)dk * dv;
  if (tokens == 0) {
    p.slot = 1;
    p.n_slots = 1;
  } else if (!packed && (int64_t)rows * H >= cus) {
    // Rows of their own from one workgroup a compute unit on, without a pass for
    // states: 8 rows of 4096 tokens of 32 heads of 128 359 us, with slots for
    // two workgroups a unit 431 (gradients 1091 and 1200); 16 rows of 1024 tokens
    // of 16 heads 95 and 126 (285 and 358; 64 channels 64 and 78, fp32 224 and 303).
    p.slot = T;
    p.n_slots = rows;
  } else {
    // As many workgroups as every compute unit holds, unless their states, one
    // for every slot and head, then cost more than the others hide: at least
    // the tokens whose keys and values are half a state (256 with 128 channels
    // of both; half of that took 61.5 us against 55.4 for 4096 tokens of 16
    // heads, and their gradients 153 against 139).  Where that leaves more than
    // one each, as for 16384 tokens, two take 147 us and one 163.  Shorter slots
    // only where not even one each would be left.  Rows and sequences shorter
    // than a slot go one after the other in its workgroup (255 rows of one token
    // of one head 479 us, 256 of them, each a slot, 14; 256 packed tokens that
    // are sequences of 16 heads 547).
    auto slots_of = [&](int64_t groups) {
      const int64_t n = groups / H < 1 ? 1 : groups / H;
      return ceil_div(ceil_div(tokens, n), kLinearChunk) * kLinearChunk;
    };
    const int64_t full = slots_of(linear_groups_of_unit(dk, dv) * cus), one = slots_of(cus);
    const int64_t least = ceil_div(4 * dk * dv / (dk + dv), kLinearChunk) * kLinearChunk;
    p.slot = full >= least ? full : one < least ? one : least;
    p.n_slots = ceil_div(tokens, p.slot);
  }
  p.carry = p.n_slots > 1 && (packed || p.slot % T != 0);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  const size_t slots = p.carry ? (size_t)p.n_slots : 0, heads = (size_t)H;
  p.end_off = take(slots * heads * record * 4);
  p.adj_off = backward ? take(slots * heads * record * 4) : 0;
  p.sum_off = take(slots * heads * 8);
  p.kind_off = take(slots * 4);
  if (backward) {
    p.dot_q_off = take((size_t)tokens * heads * 4);
    p.dot_k_off = take((size_t)tokens * heads * 4);
    p.slot_dot_off = take((size_t)p.n_slots * heads * 4);
    p.seq_dot_off = take((size_t)rows * heads * 4);
  }
  p.ws_bytes = off;
  return p;
}

// Shared queries and keys get their gradients by head first, in fp32.
inline void plan_linear_shared(LinearPlan* p, int64_t tokens, int H, int Hq, int dk) {
  if (H == Hq) return;
  const size_t each = ((size_t)tokens * H * dk * 4 + 255) / 256 * 256;
  p->dq_off = p->ws_bytes;
  p->dk_off = p->dq_off + each;
  p->ws_bytes = p->dk_off + each;
}

inline int64_t linear_groups(const LinearPlan& p, int H) { return p.n_slots * (int64_t)H; }
// The launches' grids: sweeps of 512 threads at most a slot and head (three
// roles of them backward), the chain's states, the shared heads' sums.
inline bool linear_fits(const LinearPlan& p, int64_t tokens, int H, size_t record, int Hq, int dk) {
  return grid_fits(3 * linear_groups(p, H), 512) && grid_fits(H * (int64_t)record / 1024, 256) &&
         grid_fits(ceil_div(tokens * Hq * dk, 256), 256);
}

inline bool linear_step_fits(const LinearArgs& a) {
  return grid_fits(a.tokens * a.H, a.dk <= 64 ? a.dv <= 64 ? 256 : 512 : a.dv <= 64 ? 512 : 1024);
}

struct LinearGrads {
  const void* dout;
  const float* dht;
  void *dq, *dk, *dv, *dg;
  float* dh0;
};

int launch_linear_forward(int is_bf16, const LinearArgs& a, const LinearPlan& p, void* o, float* ht, void* ws,
                          void* stream);
int launch_linear_step(int is_bf16, const LinearArgs& a, float* state, void* o, void* stream);
int launch_linear_backward(int is_bf16, const LinearArgs& a, const LinearPlan& p, const LinearGrads& g, void* ws,
                           void* stream);

}  // namespace kda
