// Selective state space scan for gfx950: forward, one-token step, backward.
//
// Per channel c and state n, with delta = softplus(dt + bias):
//   a_t = exp(delta_t A),  h_t = a_t h_{t-1} + delta_t x_t B_t,
//   y_t = sum_n C_t h_t + skip x_t,  o_t = y_t z_t sigmoid(z_t).
// Backward, with dy = dout z sigmoid(z) and dh the gradient of h_t (all that
// follows token t included):
//   dh_t = C_t dy_t + a_{t+1} dh_{t+1},  m_t = dh_t a_t h_{t-1}
//   dx = skip dy + delta sum_n dh B,     ddelta = sum_n m A + x sum_n dh B
//   dB = sum_c dh delta x,  dC = sum_c h dy,  dA = sum_t m delta
//   dskip = sum dy x,  dz = dout y (z sigmoid(z))',  dh0 = a_1 dh_1.
//
// Every (token, channel, state) costs an exponential of its own, so no
// matrix product stands for the scan, and at 16 states it is the vector unit
// that bounds it: per element an exponential, its argument, the update (two)
// and the sum's product.  The exponential alone takes the unit as long as
// two to four of the others.
//
// Measured in bf16 at 16 states.  1 x 4096 tokens of 4096 channels: 135 us,
// of which (under the profiler, which adds a sixth) the states of the slots 62,
// the chain 9 and the outputs 86; 28 us would move the bytes (135 MB), and the
// two scans issue vector instructions in 76 and 82 % of their cycles.  8 x 2048
// tokens of the same, whose rows need no slots: 334 us.  Backward 2 x 2048
// tokens of 2048 channels: 239 us, of which (likewise) states 67 (65 % vector
// issue), chain 9, main 180 (84 %), sums 15; 24 us would move the bytes.
//
// Layout of the forward scans ("quads").  A wave holds 16 channels, lane l
// channel l / 4 and the quarter l % 4 of its states (NS of them), so four
// neighbour lanes share a channel.  Tokens come in groups of 16; the four
// lanes of a channel each prepare four of them (delta, delta x, the gate),
// which makes that work once per token and channel, and read each other's
// results as an operand modifier.  A token's sum over the states is the
// lane's own products and a sum over the four quarters; those of four tokens
// are taken together (fold_quad) and come out in the lanes that prepared the
// tokens.
// B and C of 64 tokens are staged in LDS as fp32, [token][state]; a lane
// reads its quarter, the same address for all 16 channels.
//
// The time axis is cut into slots when the channels alone do not fill the
// device.  A first launch scans every slot that a sequence leaves
// unfinished, from a zero state if the sequence entered it from an earlier
// slot, and keeps the state it hands on and the slot's sum of delta; the
// second goes over the slots in order and makes true states of those,
//   h <- exp(A sum delta) h + h_slot;
// the third scans every slot for good.  Slots are ranges of the batch's
// tokens, whatever its sequences are: a workgroup walks the sequences of its
// slot, and a token range that ends inside a group leaves the state alone
// (delta = 0).
#include "kda_layer_device.h"

namespace kda {

namespace {

// exp(delta A) = exp2(delta A2).  Finite, so that the tokens past a range's
// end (delta = 0) keep the state whatever A is; NaN stays NaN.
__device__ __forceinline__ float log2_rate(float a) {
  const float v = a * kLog2e;
  return v < -3.4e38f ? -3.4e38f : v > 3.4e38f ? 3.4e38f : v;
}

// A lane's channel: its group and number (a real one also where the lane has
// none of its own), and the states it holds, first + i * step.
struct Channel {
  int g, c;
  bool active;
  int first, step;
};
__device__ __forceinline__ Channel channel_of(const ScanArgs& a, int block, int in_block, int per_block, int first,
                                              int step) {
  const int per_group = a.D / a.G, g = block / a.blocks_per_group;
  const int at = (block - g * a.blocks_per_group) * per_block + in_block;
  return Channel{g, g * per_group + (at < per_group ? at : per_group - 1), at < per_group, first, step};
}

// Workgroup -> (slot, channel block), consecutive channel blocks of a slot on
// one XCD (workgroups are dealt to the 8 XCDs in turn): their rows share
// cache lines.  False past the end.
__device__ __forceinline__ bool work_of(const ScanArgs& a, int* slot, int* block) {
  const int n_blocks = a.G * a.blocks_per_group, total = (int)a.n_slots * n_blocks, per = (total + 7) / 8;
  const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  *slot = uniform(id / n_blocks);
  *block = uniform(id - *slot * n_blocks);
  return id < total;
}
inline dim3 work_grid(const ScanArgs& a) {
  const int64_t total = a.n_slots * a.G * a.blocks_per_group;
  return dim3((unsigned)((total + 7) / 8 * 8));
}

// A slot's tokens.
struct Slot {
  int lo, hi;
  bool last;
};
__device__ __forceinline__ Slot slot_of(const ScanArgs& a, int slot) {
  const int64_t lo = slot * a.slot, hi = lo + a.slot;
  return Slot{(int)lo, (int)(hi < a.tokens ? hi : a.tokens), slot + 1 >= a.n_slots};
}

// Per-channel constants of a lane.
template <int NS>
struct Rates {
  float A2[NS];  // log2 e times A, 0 for states past N
  float skip, bias;
  __device__ __forceinline__ void load(const ScanArgs& a, const Channel& ch) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int n = ch.first + i * ch.step;
      A2[i] = n < a.N ? log2_rate(a.A[(int64_t)ch.c * a.N + n]) : 0.f;
    }
    skip = a.skip ? a.skip[ch.c] : 0.f;
    bias = a.bias ? a.bias[ch.c] : 0.f;
  }
};

// A decay of the wave's channels may be above 1: not when delta is a softplus
// and no rate is above zero, and the products of decays then need no care.
template <int NS>
__device__ __forceinline__ bool may_grow(const ScanArgs& a, const Rates<NS>& r) {
  bool above = !a.softplus;
#pragma unroll
  for (int i = 0; i < NS; ++i) above = above || r.A2[i] > 0.f;
  return __any(above);
}

// One row [D, N] of states (zeros where p is null and past N).
template <int NS>
__device__ __forceinline__ void load_state(const float* __restrict__ p, int64_t row, const ScanArgs& a,
                                           const Channel& ch, float (&h)[NS]) {
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = ch.first + i * ch.step;
    h[i] = p && n < a.N ? p[(row * a.D + ch.c) * a.N + n] : 0.f;
  }
}
template <int NS>
__device__ __forceinline__ void store_state(float* __restrict__ p, int64_t row, const ScanArgs& a, const Channel& ch,
                                            const float (&h)[NS]) {
  if (!ch.active) return;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = ch.first + i * ch.step;
    if (n < a.N) p[(row * a.D + ch.c) * a.N + n] = h[i];
  }
}

// 2^x v: a decay over many tokens times what it carries.  Where steps of
// either sign or rates above zero make states grow and shrink again, the decay
// of a whole range can pass fp32 although no token's result does, so its whole
// part is added to v's exponent.  (The rest is above 1/2 and at most 1: the
// product stays in range before that.)
__device__ __forceinline__ float scaled(float x, float v) {
  const float t = __builtin_amdgcn_fmed3f(x, -1e9f, 1e9f), whole = __builtin_ceilf(t);
  return __builtin_amdgcn_ldexpf(v * exp2_fast(t - whole), (int)whole);
}

__device__ __forceinline__ float delta_of(const ScanArgs& a, float v) {
  const float sp = softplus(v);
  return a.softplus ? sp : v;
}

// ---- forward scans ("quads") ---------------------------------------------------

// Loads are issued ahead of their use and stay as they come from memory
// until then: what is converted, or merged after a branch, is waited for.

// Tiles of B and C: TOK tokens from t0 of group g as [token][NP states],
// zero past the range's end and past N.  A thread holds element
// threadIdx.x + k THREADS of the tile.  A scan of the state alone has no use
// for C.
template <typename T, int NP, int TOK, int THREADS, bool WITH_C>
struct TileRows {
  static constexpr int PER = TOK * NP / THREADS;
  T b[PER], c[PER];
  __device__ __forceinline__ void load(const ScanArgs& a, int g, int t0, int end) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int el = threadIdx.x + k * THREADS, n = el % NP;
      const int t = t0 + el / NP;
      const int64_t tok = t < end ? t : end - 1;
      const int at = g * a.N + (n < a.N ? n : a.N - 1);
      b[k] = ((const T*)a.Bm)[tok * a.ld_b + at];
      if (WITH_C) c[k] = ((const T*)a.Cm)[tok * a.ld_c + at];
    }
  }
  __device__ __forceinline__ void store(const ScanArgs& a, float* s, int t0, int end) const {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int el = threadIdx.x + k * THREADS;
      const bool there = el % NP < a.N && t0 + el / NP < end;
      s[el] = there ? Elem<T>::to_f32(b[k]) : 0.f;
      if (WITH_C) s[TOK * NP + el] = there ? Elem<T>::to_f32(c[k]) : 0.f;
    }
  }
};

// What a scan does: the state only, the outputs, or the state and the
// gradient sent to the state before the range (adj).
enum Mode { kState, kOutput, kAdjoint };

// Offsets in bytes of a lane's first token of a group, from the group's row.
struct LaneOffsets {
  uint32_t x, dt, z, o;
};

// A lane's four tokens of a group: q, q + 4, q + 8 and q + 12.
template <typename T, Mode M>
struct Four {
  T x_[4], dt_[4], z_[4], g_[4];
  // whole group: one scalar address and one lane offset per array
  __device__ __forceinline__ void load(const ScanArgs& a, const T* __restrict__ dout, const LaneOffsets& l, int t) {
    auto row = [&](const void* p, int64_t ld, int m, uint32_t off) {
      return *(const T*)((const char*)((const T*)p + (t + 4 * (int64_t)m) * ld) + off);
    };
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      x_[m] = row(a.x, a.ld_x, m, l.x);
      dt_[m] = row(a.dt, a.ld_dt, m, l.dt);
      if (M != kState) z_[m] = row(a.z, a.ld_z, m, l.z);
      if (M == kAdjoint) g_[m] = row(dout, a.D, m, l.o);
    }
  }
  // a group cut short at `end`: the last token for those past it
  __device__ __forceinline__ void load(const ScanArgs& a, const T* __restrict__ dout, const Channel& ch, int t, int q,
                                       int end) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int64_t tok = t + 4 * m + q < end ? t + 4 * m + q : end - 1;
      x_[m] = ((const T*)a.x)[tok * a.ld_x + ch.c];
      dt_[m] = ((const T*)a.dt)[tok * a.ld_dt + ch.c];
      if (M != kState) z_[m] = ((const T*)a.z)[tok * a.ld_z + ch.c];
      if (M == kAdjoint) g_[m] = dout[tok * a.D + ch.c];
    }
  }
};

// lane K's value in all four lanes of a quad
template <int K>
__device__ __forceinline__ float quad_bcast(float v) {
  return dpp<K * 0x55>(v);
}
// sum over the quad, in all four lanes
__device__ __forceinline__ float quad_sum(float v) {
  v += dpp<kPairSwap>(v);
  return v + dpp<kQuadSwap>(v);
}
// Four sums over the quad, lane k's result that of p[k].  Each fold halves
// the values a lane answers for and adds its neighbour's share of them.
__device__ __forceinline__ float fold_quad(const float (&p)[4], int q) {
  const bool odd = q & 1, upper = q & 2;
  const float a = (odd ? p[1] : p[0]) + dpp<kPairSwap>(odd ? p[0] : p[1]);
  const float b = (odd ? p[3] : p[2]) + dpp<kPairSwap>(odd ? p[2] : p[3]);
  return (upper ? b : a) + dpp<kQuadSwap>(upper ? a : b);
}

template <int NS>
__device__ __forceinline__ void load_lds(const float* p, float (&v)[NS]) {
  if constexpr (NS >= 4) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
      const f32x4 x = *(const f32x4*)(p + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i + e] = x[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = p[i];
  }
}

// State of one scan: the state itself, and for kAdjoint the gradient sent
// back.
template <int NS>
struct Scanned {
  float h[NS], adj[NS];
};

// One group of 16 tokens from token t.  WHOLE: all of them are before `end`.
// s: this lane's quarter of the group's first token of B; C is `c_off` floats
// further.  kAdjoint sums what the group's tokens send to the state before it,
// with the product of the decays so far, and sends that back through the
// range's tokens before the group, whose sum of delta is `before`.  GROWS: a
// decay may be above 1; the product then keeps its exponent apart.  WILD:
// states past N are kept zero whatever comes.  Returns this lane's sum of delta.
template <typename T, int NS, Mode M, bool WHOLE, bool GROWS = false, bool WILD = false>
__device__ __forceinline__ float scan_group(const ScanArgs& a, const Channel& ch, const Rates<NS>& r, int q,
                                            const Four<T, M>& in, const LaneOffsets& l, int t, int end,
                                            const float* s, int c_off, float before, Scanned<NS>& st,
                                            T* __restrict__ o) {
  constexpr int NP = 4 * NS;
  float y[4], sum = 0.f, adj[NS], run[NS];
  int exponent[NS];
  if (M == kAdjoint) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      adj[i] = 0.f;
      run[i] = 1.f;
      exponent[i] = 0;
    }
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const bool there = WHOLE || t + 4 * m + q < end;
    float d = delta_of(a, Elem<T>::to_f32(in.dt_[m]) + r.bias), v = d * Elem<T>::to_f32(in.x_[m]);
    if (!WHOLE) {
      d = there ? d : 0.f;
      v = there ? v : 0.f;
    }
    sum += d;
    float g = 0.f, part[4];
    if (M == kAdjoint) {
      const float z = Elem<T>::to_f32(in.z_[m]), gate = z * sigmoid(z);
      g = Elem<T>::to_f32(in.g_[m]) * (a.has_z ? gate : 1.f);
      g = there ? g : 0.f;
    }
    static_for<4>([&](auto lane) {
      constexpr int k = decltype(lane)::value;
      float B[NS], C[NS];
      load_lds<NS>(s + (4 * m + k) * NP, B);
      if (M != kState) load_lds<NS>(s + c_off + (4 * m + k) * NP, C);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float e = exp2_fast(quad_bcast<k>(d) * r.A2[i]);
        const float put = quad_bcast<k>(v) * B[i];
        st.h[i] = __builtin_fmaf(e, st.h[i], put);
        if (WILD) st.h[i] = ch.first + i < a.N ? st.h[i] : 0.f;
        if (M == kOutput) part[k] = i ? part[k] + C[i] * st.h[i] : C[i] * st.h[i];
        if (M == kAdjoint) {
          run[i] *= e;
          const float back = quad_bcast<k>(g) * C[i];
          if (GROWS) {
            exponent[i] += __builtin_amdgcn_frexp_expf(run[i]);
            run[i] = __builtin_amdgcn_frexp_mantf(run[i]);
            adj[i] += __builtin_amdgcn_ldexpf(run[i] * back, exponent[i]);
          } else {
            adj[i] += run[i] * back;
          }
        }
      }
    });
    if (M == kOutput) y[m] = fold_quad(part, q);
  }
  if (M == kAdjoint) {
#pragma unroll
    for (int i = 0; i < NS; ++i) st.adj[i] += scaled(before * r.A2[i], adj[i]);
  }
  if (M == kOutput && ch.active) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float x = Elem<T>::to_f32(in.x_[m]), z = Elem<T>::to_f32(in.z_[m]), gate = z * sigmoid(z);
      const float v = (y[m] + r.skip * x) * (a.has_z ? gate : 1.f);
      T* at = (T*)((char*)(o + (t + 4 * (int64_t)m) * a.D) + l.o);
      if (WHOLE || t + 4 * m + q < end) *at = Elem<T>::from_f32(v);
    }
  }
  return sum;
}

// What the backward pass keeps of every group of 16 tokens: the state before
// it, scanned from what the range started from, and the range's sum of delta
// before it.  Groups are numbered by groups_at(): ranges follow one another,
// each starts a group of its own.
struct GroupStates {
  float *h, *sum;
};
__device__ __forceinline__ int groups_at(int t0, int seq, int slot) { return t0 / 16 + seq + slot; }

template <int NS>
__device__ __forceinline__ void keep_group(const ScanArgs& a, const Channel& ch, const GroupStates& k, int group,
                                           const float (&h)[NS], float before) {
  store_state<NS>(k.h, group, a, ch, h);
  if (ch.active && ch.first == 0) k.sum[(int64_t)group * a.D + ch.c] = before;
}

// Scans tokens [t0, end) of one sequence.  Returns the lane's sum of delta.
// KEEP: leaves what GroupStates says from group `group` on.
// PADS: some lanes hold states past N, the last state of a channel's last lane
// among them.  They read zeros for B and C and stay zero, unless an infinite
// delta x makes NaN of them.  A tile of tokens that ends so is scanned again
// with them kept zero (20011 tokens of 771 channels, 12 states, fp32: 169 us; a
// look at every group's inputs beforehand 175).
template <typename T, int NS, Mode M, bool KEEP = false, bool PADS = false>
__device__ __forceinline__ float scan_range(const ScanArgs& a, const Channel& ch, const Rates<NS>& r, int q,
                                            const LaneOffsets& l, int t0, int end, float* s, Scanned<NS>& st,
                                            T* __restrict__ o, const T* __restrict__ dout, GroupStates keep = {},
                                            int group = 0) {
  constexpr int THREADS = 64 * kScanWaves, NP = 4 * NS, C_OFF = kScanTile * NP, BUF = 2 * C_OFF;
  TileRows<T, NP, kScanTile, THREADS, M != kState> tile;
  Four<T, M> next;
  float sum = 0.f;
  const bool grows = M == kAdjoint && may_grow(a, r);
  auto group_of = [&](const Four<T, M>& in, int u, const float* at, auto whole) {
    const float before = KEEP ? quad_sum(sum) : 0.f;
    if (KEEP) keep_group<NS>(a, ch, keep, group++, st.h, before);
    if (M == kAdjoint && grows)
      return scan_group<T, NS, M, whole.value, true>(a, ch, r, q, in, l, u, end, at, C_OFF, before, st, o);
    return scan_group<T, NS, M, whole.value>(a, ch, r, q, in, l, u, end, at, C_OFF, before, st, o);
  };
  __shared__ float entered[PADS ? NS : 1][THREADS];  // the states that entered the tile
  if (t0 + 16 <= end) next.load(a, dout, l, t0);
  tile.load(a, ch.g, t0, end);
  __syncthreads();  // the range before may still be reading
  tile.store(a, s, t0, end);
  __syncthreads();
  int buf = 0;
  for (int t = t0; t < end; t += kScanTile) {
    const bool more = end - t > kScanTile;
    if (more) tile.load(a, ch.g, t + kScanTile, end);
    const float* sq = s + buf * BUF + q * NS;
    int u = t;
    if (PADS) {
#pragma unroll
      for (int i = 0; i < NS; ++i) entered[i][threadIdx.x] = st.h[i];
    }
    for (; u + 16 <= end && u < t + kScanTile; u += 16) {
      const Four<T, M> cur = next;
      if (u + 32 <= end) next.load(a, dout, l, u + 16);
      sum += group_of(cur, u, sq + (u - t) * NP, std::true_type{});
    }
    if (u < end && u < t + kScanTile) {
      Four<T, M> cur;
      cur.load(a, dout, ch, u, q, end);
      sum += group_of(cur, u, sq + (u - t) * NP, std::false_type{});
    }
    if (PADS && __any(q == 3 && st.h[NS - 1] != 0.f)) {
#pragma unroll
      for (int i = 0; i < NS; ++i) st.h[i] = ch.first + i < a.N ? entered[i][threadIdx.x] : 0.f;
      for (u = t; u < end && u < t + kScanTile; u += 16) {
        Four<T, M> cur;
        cur.load(a, dout, ch, u, q, end);
        scan_group<T, NS, M, false, false, true>(a, ch, r, q, cur, l, u, end, sq + (u - t) * NP, C_OFF, 0.f, st, o);
      }
    }
    if (more) {
      buf ^= 1;
      tile.store(a, s + buf * BUF, t + kScanTile, end);
      __syncthreads();
    }
  }
  return sum;
}

// A workgroup's place in the forward scans.
template <int NS>
struct QuadWork {
  int slot, q;
  Slot tok;
  Channel ch;
  Rates<NS> r;
  LaneOffsets l;
  __device__ __forceinline__ bool init(const ScanArgs& a, size_t esz) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    int block;
    if (!work_of(a, &slot, &block)) return false;
    q = lane & 3;
    ch = channel_of(a, block, wave * 16 + (lane >> 2), 16 * kScanWaves, q * NS, 1);
    r.load(a, ch);
    tok = slot_of(a, slot);
    const uint32_t e = (uint32_t)esz;
    l = LaneOffsets{e * (uint32_t)(q * a.ld_x + ch.c), e * (uint32_t)(q * a.ld_dt + ch.c),
                    e * (uint32_t)(q * a.ld_z + ch.c), e * (uint32_t)(q * (int64_t)a.D + ch.c)};
    return true;
  }
};

// What the first launch found of a slot (one word per slot): whether a
// sequence goes on past its end, and whether that one entered it from an
// earlier slot; and, for the backward pass, whether one entered it.
enum SlotKind { kNothing = 0, kStarted = 1, kPassed = 2, kEntered = 4 };

// Forward.  M = kState: the first launch, over what a slot leaves unfinished;
// kOutput: the last one, hend then holding the states at the slots' ends.
template <typename T, int NS, Mode M, bool PADS>
__global__ void __launch_bounds__(64 * kScanWaves, 2)
scan_forward(const ScanArgs a, float* __restrict__ hend, float* __restrict__ sum, int* __restrict__ kind,
             T* __restrict__ o, float* __restrict__ ht) {
  __shared__ __align__(16) float s[2 * 2 * kScanTile * 4 * NS];
  QuadWork<NS> w;
  if (!w.init(a, sizeof(T))) return;
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  const int lo = w.tok.lo, hi = w.tok.hi;
  Scanned<NS> st;
  if (M == kState) {
    const int n = uniform(seqs.from(hi)) - 1;  // the last sequence that starts in the slot or before
    const bool on = !w.tok.last && n >= 0 && uniform((int)seqs.end(n)) > hi;
    const int start = on ? uniform((int)seqs.start(n)) : 0;
    const bool own = start >= lo;
    if (threadIdx.x == 0) kind[w.slot] = !on ? kNothing : own ? kStarted : kPassed;
    if (!on) return;
    load_state<NS>(own ? a.h0 : nullptr, n, a, w.ch, st.h);
    const float d = scan_range<T, NS, M>(a, w.ch, w.r, w.q, w.l, own ? start : lo, hi, s, st, (T*)nullptr,
                                         (const T*)nullptr);
    store_state<NS>(hend, w.slot, a, w.ch, st.h);
    const float total = quad_sum(d);
    if (!own && w.ch.active && w.q == 0) sum[(int64_t)w.slot * a.D + w.ch.c] = total;
    return;
  }
  int n = uniform(seqs.from(lo)), at = lo;
  if (n > 0) {
    const int end = uniform((int)seqs.end(n - 1));
    if (end > lo) {  // a sequence that entered from an earlier slot
      at = end;
      load_state<NS>(hend, w.slot - 1, a, w.ch, st.h);
      scan_range<T, NS, M, false, PADS>(a, w.ch, w.r, w.q, w.l, lo, end < hi ? end : hi, s, st, o, (const T*)nullptr);
      if (ht && end <= hi) store_state<NS>(ht, n - 1, a, w.ch, st.h);
    }
  }
  // those that start here; the last slot also has the empty ones behind the last token
  for (; n < a.n_seqs; ++n) {
    const Span range = seqs.next(n, &at);
    const int start = uniform(range.start), end = uniform(range.end);
    if (!w.tok.last && start >= hi) break;
    load_state<NS>(a.h0, n, a, w.ch, st.h);
    if (start < end)
      scan_range<T, NS, M, false, PADS>(a, w.ch, w.r, w.q, w.l, start, end < hi ? end : hi, s, st, o,
                                        (const T*)nullptr);
    if (ht && end <= hi) store_state<NS>(ht, n, a, w.ch, st.h);
  }
}

// The second launch: true states at the slots' ends out of what each slot
// made of a zero state, in place, and (blockIdx.y = 1) likewise the gradients
// of the states at the slots' starts, from the last slot to the first:
//   h_i <- h_i + exp(A sum_i) h_{i-1},   g_i <- g_i + exp(A sum_i) g_{i+1}
// for the slots that a sequence passes through.  A lane takes one state of
// one channel; the 8 waves of a workgroup take an eighth of the slots each,
// first composing it to (exponent of the decays, state), then again from the
// state that the waves before hand on, so that the chain is an eighth as
// long.  Loads go ahead of it in batches.
constexpr int kChainWaves = 8;
template <int BATCH>
__global__ void __launch_bounds__(64 * kChainWaves)
scan_chain(const float* __restrict__ A, int64_t dn, int N, int D, int n_slots, float* __restrict__ hend,
           float* __restrict__ adj, const float* __restrict__ sum, const int* __restrict__ kind) {
  __shared__ float decay[kChainWaves][64], state[kChainWaves][64];
  __shared__ int through[kChainWaves];  // one sequence passes all of a wave's slots
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const bool back = blockIdx.y != 0;
  float* __restrict__ v = back ? adj : hend;
  int64_t el = (int64_t)blockIdx.x * 64 + lane;
  const bool there = el < dn;
  el = there ? el : dn - 1;
  const int64_t c = el / N;
  const float A2 = log2_rate(A[el]);
  const int per = (n_slots + kChainWaves - 1) / kChainWaves;
  // positions along the chain: slot i, or n_slots - 1 - i going back
  const int first = wave * per, last = first + per < n_slots ? first + per : n_slots;
  int unbroken = 1;
  auto walk = [&](float& x, float& h, bool write) {
    for (int i0 = first; i0 < last; i0 += BATCH) {
      float s[BATCH], made[BATCH];
      int kd[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int i = i0 + k < last ? i0 + k : last - 1, slot = back ? n_slots - 1 - i : i;
        s[k] = sum[(int64_t)slot * D + c];
        made[k] = v[(int64_t)slot * dn + el];
        kd[k] = kind[slot];
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        if (i0 + k >= last) break;
        // what the slot holds counts only where a sequence leaves it (back: enters it)
        const bool passed = kd[k] & kPassed, holds = back ? kd[k] & kEntered : kd[k] & (kStarted | kPassed);
        const float by = __builtin_amdgcn_fmed3f(s[k] * A2, -1e30f, 1e30f);
        h = (passed ? scaled(by, h) : 0.f) + (holds ? made[k] : 0.f);
        x += by;  // of use where all of the wave's slots are passed
        unbroken = passed ? unbroken : 0;
        if (write && there) v[(int64_t)(back ? n_slots - 1 - i0 - k : i0 + k) * dn + el] = h;
      }
    }
  };
  float x = 0.f, h = 0.f;
  walk(x, h, false);
  decay[wave][lane] = x;
  state[wave][lane] = h;
  through[wave] = unbroken;
  __syncthreads();
  h = 0.f;
  for (int w = 0; w < wave; ++w) h = (through[w] ? scaled(decay[w][lane], h) : 0.f) + state[w][lane];
  walk(x, h, true);
}

// ---- one token ---------------------------------------------------------------
// The state is read once and written once, which is all the step costs: a
// lane owns 4 consecutive states (16 bytes) of a channel in SEQS sequences,
// n_far apart, LPC lanes a channel, so that the rates are loaded once for the
// sequences and the loads of all are under way together (256 sequences, 4096
// channels, 16 states: 22.0 us, 142.9 MB; loads and stores that bypass the
// caches cost 8 % more).  Without VEC (N no multiple of 4) the same states are
// loaded one by one, which takes the same call 52 us.
template <typename T, int LPC, bool VEC, int SEQS>
__global__ void __launch_bounds__(256)
scan_step(const ScanArgs a, float* __restrict__ state, T* __restrict__ o, int n_far) {
  const int sub = threadIdx.x % LPC;
  const uint32_t channel = (blockIdx.x * 256u + threadIdx.x) / LPC, row = channel / (uint32_t)a.D;
  const int c = (int)(channel - row * (uint32_t)a.D);
  if (row >= (uint32_t)n_far) return;
  const int g = c / (a.D / a.G), n0 = sub * 4;
  auto there = [&](int i) { return VEC ? n0 < a.N : n0 + i < a.N; };
  const int at = n0 < a.N ? n0 : 0;  // a real state also for the lanes past the last
  typedef float quad __attribute__((ext_vector_type(4), aligned(4)));
  quad h[SEQS];
  float B[SEQS][4], C[SEQS][4];
  T x[SEQS], dt[SEQS], z[SEQS];
#pragma unroll
  for (int q = 0; q < SEQS; ++q) {
    const int64_t s = (int64_t)row + (int64_t)q * n_far, seq = s < a.tokens ? s : row;
    const float* st = state + (seq * a.D + c) * a.N;
    const T* __restrict__ Bm = (const T*)a.Bm + seq * a.ld_b + (int64_t)g * a.N;
    const T* __restrict__ Cm = (const T*)a.Cm + seq * a.ld_c + (int64_t)g * a.N;
    if (VEC) {
      h[q] = *(const quad*)(st + at);
      load_vec<T, 4>(Bm + at, B[q]);
      load_vec<T, 4>(Cm + at, C[q]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[q][i] = st[there(i) ? n0 + i : 0];
        B[q][i] = load_f32(Bm + (there(i) ? n0 + i : 0));
        C[q][i] = load_f32(Cm + (there(i) ? n0 + i : 0));
      }
    }
    x[q] = ((const T*)a.x)[seq * a.ld_x + c];
    dt[q] = ((const T*)a.dt)[seq * a.ld_dt + c];
    z[q] = ((const T*)a.z)[seq * a.ld_z + c];
  }
  float rate[4];
  if (VEC) {
    load_vec<float, 4>(a.A + (int64_t)c * a.N + at, rate);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) rate[i] = a.A[(int64_t)c * a.N + (there(i) ? n0 + i : 0)];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) rate[i] = log2_rate(rate[i]);
  const float skip = a.skip ? a.skip[c] : 0.f, bias = a.bias ? a.bias[c] : 0.f;
#pragma unroll
  for (int q = 0; q < SEQS; ++q) {
    const int64_t seq = (int64_t)row + (int64_t)q * n_far;
    if (seq >= a.tokens) break;
    const float xs = Elem<T>::to_f32(x[q]), delta = delta_of(a, Elem<T>::to_f32(dt[q]) + bias), dx = delta * xs;
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[q][i] = exp2_fast(delta * rate[i]) * h[q][i] + dx * B[q][i];
      y += there(i) ? C[q][i] * h[q][i] : 0.f;
    }
    float* st = state + (seq * a.D + c) * a.N;
    if (VEC) {
      if (n0 < a.N) *(quad*)(st + n0) = h[q];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (there(i)) st[n0 + i] = h[q][i];
    }
    if constexpr (LPC >= 2) y += dpp<kPairSwap>(y);
    if constexpr (LPC >= 4) y += dpp<kQuadMirror>(y);
    if constexpr (LPC >= 8) y += dpp<kHalfMirror>(y);
    if constexpr (LPC >= 16) y += dpp<kRowMirror>(y);
    if (sub == 0) {
      const float zs = Elem<T>::to_f32(z[q]), gate = zs * sigmoid(zs);
      o[seq * a.D + c] = Elem<T>::from_f32((y + skip * xs) * (a.has_z ? gate : 1.f));
    }
  }
}

// ---- backward ------------------------------------------------------------------
// The first launch walks every slot forward once and leaves the state before
// every group of 16 tokens, the state that the slot hands on, and the
// gradient it hands back (the part of the state gradient at its start that
// its own tokens make, summed forward in time with the running product of
// the decays).  A range that continues an earlier slot's sequence starts from
// zero there; what the state that truly enters adds to a group's state is
// exp(A sum delta) times it.  scan_chain, when sequences pass from slot to
// slot, composes the states and gradients between them.  The next launch
// walks the groups of every slot back, redoing each group's recurrence in
// registers.  The last two add the partial sums.
template <typename T, int NS>
__global__ void __launch_bounds__(64 * kScanWaves, NS <= 4 ? 3 : 2)
scan_backward_states(const ScanArgs a, const T* __restrict__ dout, const float* __restrict__ dht,
                     float* __restrict__ hend, float* __restrict__ adj, float* __restrict__ sum,
                     int* __restrict__ kind, const GroupStates keep) {
  __shared__ __align__(16) float s[2 * 2 * kScanTile * 4 * NS];
  QuadWork<NS> w;
  if (!w.init(a, sizeof(T))) return;
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  const int lo = w.tok.lo, hi = w.tok.hi;
  Scanned<NS> st;
  int n = uniform(seqs.from(lo));
  const int before = n > 0 ? uniform((int)seqs.end(n - 1)) : lo;
  int found = kNothing, at = before > lo ? before : lo;
  if (before > lo) {  // entered from an earlier slot
    found = kEntered | (before > hi ? kPassed : 0);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      st.h[i] = st.adj[i] = 0.f;
    }
    const float d = scan_range<T, NS, kAdjoint, true>(a, w.ch, w.r, w.q, w.l, lo, before < hi ? before : hi, s, st,
                                                      (T*)nullptr, dout, keep, groups_at(lo, n - 1, w.slot));
    const float all = quad_sum(d);
    if (before <= hi) {
      float last[NS];
      load_state<NS>(dht, n - 1, a, w.ch, last);
#pragma unroll
      for (int i = 0; i < NS; ++i) st.adj[i] += scaled(all * w.r.A2[i], last[i]);
    } else {
      store_state<NS>(hend, w.slot, a, w.ch, st.h);
      if (w.ch.active && w.q == 0) sum[(int64_t)w.slot * a.D + w.ch.c] = all;
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {  // a NaN decay reaches back through any gradient
      const float x = all * w.r.A2[i];
      st.adj[i] = x != x ? x : st.adj[i];
    }
    store_state<NS>(adj, w.slot, a, w.ch, st.adj);
  }
  for (; n < a.n_seqs; ++n) {
    const Span range = seqs.next(n, &at);
    const int start = uniform(range.start), end = uniform(range.end);
    if (start >= hi) break;
    if (start >= end) continue;
    load_state<NS>(a.h0, n, a, w.ch, st.h);
    scan_range<T, NS, kState, true>(a, w.ch, w.r, w.q, w.l, start, end < hi ? end : hi, s, st, (T*)nullptr, dout, keep,
                                    groups_at(start, n, w.slot));
    if (end > hi) {  // goes on past the slot
      found |= kStarted;
      store_state<NS>(hend, w.slot, a, w.ch, st.h);
    }
  }
  if (kind && threadIdx.x == 0) kind[w.slot] = found;
}

// Layout of the backward scan ("rows").  A row of 16 lanes holds one channel,
// lane j the states j, j + 16, ... and, of a group of 16 tokens, the inputs
// of token j; a wave has 4 channels.  In the recurrence token k's values are
// lane k's, broadcast over the row as an operand modifier; the sums over the
// states of a group's tokens are folded lane by lane (RowSums) as the tokens
// come.  Sums over channels, of which the backward pass has two per element,
// begin with the wave's 4 rows: four tokens' values are added across the rows
// by three swaps and three additions (fold_rows), which leaves token k's sum
// in row k, so a group becomes one [16 tokens][16 states] tile in four
// registers.  (v_mfma_f32_16x16x4f32 with a one-hot left operand does the
// same, 32 cycles of the matrix pipe each, and was slower.)  The tiles of the
// waves are added in LDS, those of the workgroups by a later launch.  B and C
// of 64 tokens are staged as [state][token] with rows of 68 words: four
// tokens are one 16-byte read, free of bank conflicts.
constexpr int kColLd = kScanTile + 4;

// Tiles of B and C as [state][token]; a thread holds one state of every
// (THREADS / 16)-th token.
template <typename T, int NS, int THREADS>
struct TileCols {
  static constexpr int PER = kScanTile * 16 / THREADS;  // tokens a thread
  T b[NS][PER], c[NS][PER];
  __device__ __forceinline__ void load(const ScanArgs& a, int g, int t0, int end) {
    const int n = threadIdx.x & 15, t = threadIdx.x >> 4;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int tk = t0 + t + k * (THREADS / 16);
      const int64_t tok = tk < end ? tk : end - 1;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int at = g * a.N + (n + 16 * i < a.N ? n + 16 * i : a.N - 1);
        b[i][k] = ((const T*)a.Bm)[tok * a.ld_b + at];
        c[i][k] = ((const T*)a.Cm)[tok * a.ld_c + at];
      }
    }
  }
  // s: [2][NS * 16][kColLd], B first
  __device__ __forceinline__ void store(const ScanArgs& a, float* s, int t0, int end) const {
    const int n = threadIdx.x & 15, t = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int tok = t + k * (THREADS / 16);
        const bool there = n + 16 * i < a.N && t0 + tok < end;
        s[(n + 16 * i) * kColLd + tok] = there ? Elem<T>::to_f32(b[i][k]) : 0.f;
        s[(NS * 16 + n + 16 * i) * kColLd + tok] = there ? Elem<T>::to_f32(c[i][k]) : 0.f;
      }
  }
};

// Sixteen sums over a row of 16 lanes, lane j's result that of token j.  The
// tokens come in order, from either end; each fold halves the tokens a lane
// answers for and adds the share of the lane 1, 2, 4 or 8 off, which answers
// for the other half and for the same of the halvings before, so 16 sums take
// 15 additions in place of 64.
struct RowSums {
  float v[16], v2[8], v4[4], v8[2], total;
  template <int CTRL>
  __device__ __forceinline__ static float fold(float lo, float hi, bool up) {
    return (up ? hi : lo) + dpp<CTRL>(up ? lo : hi);
  }
  // after v[K] has been set; DOWN: the tokens come from the last to the first
  template <int K, bool DOWN>
  __device__ __forceinline__ void done(int j) {
    constexpr int at = DOWN ? 0 : 1;
    if constexpr (K % 2 == at) v2[K / 2] = fold<kPairSwap>(v[K & ~1], v[K | 1], j & 1);
    if constexpr (K % 4 == 3 * at) v4[K / 4] = fold<kQuadSwap>(v2[K / 2 & ~1], v2[K / 2 | 1], j & 2);
    if constexpr (K % 8 == 7 * at) v8[K / 8] = fold<kRotate4>(v4[K / 4 & ~1], v4[K / 4 | 1], j & 4);
    if constexpr (K == 15 * at) total = fold<kRotate8>(v8[0], v8[1], j & 8);
  }
};

// Sums over the wave's four rows of 16 lanes: row k of the result is the sum
// of p[k]'s rows.  Each swap pairs two values' halves, so that one addition
// serves both.
__device__ __forceinline__ float fold_rows(const float (&p)[4]) {
  auto fold = [](float x, float y, auto swap) {
    const auto s = swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y));
    return __builtin_bit_cast(float, (uint32_t)s[0]) + __builtin_bit_cast(float, (uint32_t)s[1]);
  };
  auto halves = [](uint32_t x, uint32_t y) { return __builtin_amdgcn_permlane32_swap(x, y, false, false); };
  auto rows = [](uint32_t x, uint32_t y) { return __builtin_amdgcn_permlane16_swap(x, y, false, false); };
  return fold(fold(p[0], p[2], halves), fold(p[1], p[3], halves), rows);
}

// What the backward scan reads and writes beside the inputs.
struct ScanBwdBuffers {
  const float *hend, *adj;    // at every slot's end and start; null without carry
  GroupStates groups;
  float *da, *dskip, *dbias;  // per slot
  float *db, *dc;             // per workgroup of channels
};

// Lane j's token of a group, and the lane's states before the group.
template <typename T, int NS>
struct Token {
  T x_, dt_, z_, dout_;
  float h_[NS], sum_;
  __device__ __forceinline__ void load(const ScanArgs& a, const T* __restrict__ dout, const GroupStates& k,
                                       const Channel& ch, const LaneOffsets& l, int t, int group) {
    auto at = [&](const void* p, int64_t ld, uint32_t off) {
      return *(const T*)((const char*)((const T*)p + t * ld) + off);
    };
    x_ = at(a.x, a.ld_x, l.x);
    dt_ = at(a.dt, a.ld_dt, l.dt);
    z_ = at(a.z, a.ld_z, l.z);
    dout_ = at(dout, a.D, l.o);
    const float* row = k.sum + (int64_t)group * a.D;
    sum_ = *(const float*)((const char*)row + 4u * (uint32_t)ch.c);
    const float* states = k.h + (int64_t)group * a.D * a.N;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int n = ch.first + 16 * i;
      h_[i] = *(const float*)((const char*)states + 4u * (uint32_t)(ch.c * a.N + (n < a.N ? n : a.N - 1)));
    }
  }
  __device__ __forceinline__ float x() const { return Elem<T>::to_f32(x_); }
  __device__ __forceinline__ float dt() const { return Elem<T>::to_f32(dt_); }
  __device__ __forceinline__ float z() const { return Elem<T>::to_f32(z_); }
  __device__ __forceinline__ float dout() const { return Elem<T>::to_f32(dout_); }
};
__device__ __forceinline__ LaneOffsets lane_offsets(const ScanArgs& a, int token, int c, size_t esz) {
  const uint32_t e = (uint32_t)esz;
  return LaneOffsets{e * (uint32_t)(token * a.ld_x + c), e * (uint32_t)(token * a.ld_dt + c),
                     e * (uint32_t)(token * a.ld_z + c), e * (uint32_t)(token * (int64_t)a.D + c)};
}

// CARE: some lanes have no state or no channel, or a range's end may cut a
// group short.  Such lanes read zeros for B and C, or have zeros for delta,
// delta x and dy, and stay zero; tokens past the end have a delta of zero.  Only
// an infinity (of an input, or of a product) makes NaN of a lane's zeros or of
// dA's products with such a delta; a group that ends so is walked again with
// both left out (a call over 4096 tokens of 2048 channels in 40 sequences, bf16,
// 16 states: 277 us, 271 without care; 24 states 236 and 221).
template <typename T, int NS, bool CARE>
__global__ void __launch_bounds__(64 * kScanBwdWaves, NS == 1 ? 3 : 1)
scan_backward(const ScanArgs a, const ScanGrads g, const ScanBwdBuffers w) {
  constexpr int WV = kScanBwdWaves, THREADS = 64 * WV;
  __shared__ __align__(16) float bc[2 * NS * 16 * kColLd];  // B, C of a tile
  __shared__ float tiles[2][WV][2][NS][256];                // dB, dC of a group, per wave
  __shared__ float before[3][CARE ? NS : 1][THREADS];       // a lane's states, gradients and dA before a group
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), j = lane & 15;
  int slot, block;
  if (!work_of(a, &slot, &block)) return;
  const Channel ch = channel_of(a, block, wave * 4 + (lane >> 4), 4 * WV, j, 16);
  const int group = uniform(ch.g), in_group = block - group * a.blocks_per_group;
  Rates<NS> r;
  r.load(a, ch);
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  const Slot own = slot_of(a, slot);
  const int lo = own.lo, hi = own.hi;
  const T* __restrict__ dout = (const T*)g.dout;
  const LaneOffsets l = lane_offsets(a, j, ch.c, sizeof(T));
  float dA[NS], dskip = 0.f, dbias = 0.f;
#pragma unroll
  for (int i = 0; i < NS; ++i) dA[i] = 0.f;
  int buf = 0;
  bool real[NS];  // a state, and a channel, that there is
#pragma unroll
  for (int i = 0; i < NS; ++i) real[i] = ch.active && j + 16 * i < a.N;

  // tokens [t0, end) of one sequence, whose groups are `at`, at + 1, ...: h
  // the state that entered the range (zero when the groups' states have it),
  // gr the gradient of the state after it; leaves the gradient of the state
  // before it in gr
  auto range = [&](int t0, int end, int at, const float(&h)[NS], float(&gr)[NS]) {
    int q = (end - t0 - 1) / 16;
    TileCols<T, NS, THREADS> tile;
    tile.load(a, group, t0 + (q & ~3) * 16, end);
    Token<T, NS> next;
    int tokens = end - t0 - 16 * q;  // of the last group, then 16
    next.load(a, dout, w.groups, ch, lane_offsets(a, j < tokens ? j : tokens - 1, ch.c, sizeof(T)), t0 + 16 * q, at + q);
    __syncthreads();  // the range before may still be reading
    tile.store(a, bc, t0 + (q & ~3) * 16, end);
    __syncthreads();
    bool there = ch.active && j < tokens;
    for (; q >= 0; --q) {
      const Token<T, NS> cur = next;
      const int t = t0 + 16 * q;
      if (q > 0) next.load(a, dout, w.groups, ch, l, t - 16, at + q - 1);
      if ((q & 3) == 0 && q > 0) tile.load(a, group, t - kScanTile, end);
      const float* sb = bc + j * kColLd + (q & 3) * 16;
      const float* sc = sb + NS * 16 * kColLd;
      const float v = cur.dt() + r.bias, x = cur.x();
      const float delta = there ? delta_of(a, v) : 0.f;
      const float dx = there ? delta * x : 0.f;
      float first[NS], hh[16][NS], dd[16][NS];
#pragma unroll
      for (int i = 0; i < NS; ++i) first[i] = cur.h_[i] + scaled(cur.sum_ * r.A2[i], h[i]);
      RowSums ys, s1, s2;
      float dy, dz;
      float tb[NS][4], tc[NS][4];  // dB and dC of tokens 4 e + row
      // the group's tokens forward, then back
      auto walk = [&](auto care) {
        static_for<4>([&](auto k4) {
          f32x4 B[NS], C[NS];
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            B[i] = *(const f32x4*)(sb + i * 16 * kColLd + 4 * k4);
            C[i] = *(const f32x4*)(sc + i * 16 * kColLd + 4 * k4);
          }
          static_for<4>([&](auto e) {
            constexpr int k = 4 * decltype(k4)::value + decltype(e)::value;
            const float dk = row_bcast<k>(delta), xk = row_bcast<k>(dx);
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
              dd[k][i] = exp2_fast(dk * r.A2[i]);
              const float put = xk * B[i][decltype(e)::value];
              hh[k][i] = __builtin_fmaf(dd[k][i], k ? hh[k ? k - 1 : 0][i] : first[i], put);
              if (care) hh[k][i] = real[i] ? hh[k][i] : 0.f;
              y = i ? y + C[i][decltype(e)::value] * hh[k][i] : C[i][decltype(e)::value] * hh[k][i];
            }
            ys.v[k] = y;
            ys.template done<k, false>(j);
          });
          __builtin_amdgcn_sched_barrier(0);
        });
        const float z = cur.z(), dout_j = cur.dout(), sg = sigmoid(z), y = ys.total + r.skip * x;
        dz = dout_j * y * (sg * (1.f + z * (1.f - sg)));
        dy = dout_j * (a.has_z ? z * sg : 1.f);
        dy = there ? dy : 0.f;
        // other registers to the compiler, which would else keep the 32 values
        // broadcast above for the loop below
        float delta_b = delta, dx_b = dx;
        asm volatile("" : "+v"(delta_b), "+v"(dx_b));
        static_for<4>([&](auto k4r) {
          constexpr int k4 = 3 - decltype(k4r)::value;
          f32x4 B[NS], C[NS];
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            B[i] = *(const f32x4*)(sb + i * 16 * kColLd + 4 * k4);
            C[i] = *(const f32x4*)(sc + i * 16 * kColLd + 4 * k4);
          }
          float vb[NS][4], vc[NS][4];
          static_for<4>([&](auto er) {
            constexpr int e = 3 - decltype(er)::value, k = 4 * k4 + e;
            const float dk = row_bcast<k>(delta_b), gk = row_bcast<k>(dy), xk = row_bcast<k>(dx_b);
            float p1 = 0.f, p2 = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
              float dh = __builtin_fmaf(gk, C[i][e], gr[i]);
              if (care) dh = real[i] ? dh : 0.f;
              vc[i][e] = gk * hh[k][i];
              vb[i][e] = xk * dh;
              gr[i] = dh * dd[k][i];
              if (care) gr[i] = real[i] ? gr[i] : 0.f;
              const float m = gr[i] * (k ? hh[k ? k - 1 : 0][i] : first[i]);
              p1 = i ? p1 + m * r.A2[i] : m * r.A2[i];
              p2 = i ? p2 + dh * B[i][e] : dh * B[i][e];
              if (!care || k < tokens) dA[i] = __builtin_fmaf(dk, m, dA[i]);
            }
            s1.v[k] = p1;
            s2.v[k] = p2;
            s1.template done<k, true>(j);
            s2.template done<k, true>(j);
          });
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            tb[i][k4] = fold_rows(vb[i]);
            tc[i][k4] = fold_rows(vc[i]);
          }
          __builtin_amdgcn_sched_barrier(0);
        });
      };
      if (CARE) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          first[i] = real[i] ? first[i] : 0.f;
          before[0][i][threadIdx.x] = first[i];
          before[1][i][threadIdx.x] = gr[i];
          before[2][i][threadIdx.x] = dA[i];
        }
      }
      walk(std::false_type{});
      if (CARE) {
        bool again = false;
#pragma unroll
        for (int i = 0; i < NS; ++i)
          again = again || (!real[i] && (hh[15][i] != 0.f || gr[i] != 0.f)) || (tokens < 16 && dA[i] != dA[i]);
        if (__any(again)) {
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            first[i] = before[0][i][threadIdx.x];
            gr[i] = before[1][i][threadIdx.x];
            dA[i] = before[2][i][threadIdx.x];
          }
          walk(std::true_type{});
        }
      }
      const float slope = a.softplus ? sigmoid(v) : 1.f;
      const float ddt = (kLn2 * s1.total + x * s2.total) * slope;
      if (there) {
        auto to = [&](void* p) { return (T*)((char*)((T*)p + (int64_t)t * a.D) + l.o); };
        *to(g.dx) = Elem<T>::from_f32(r.skip * dy + delta * s2.total);
        *to(g.ddt) = Elem<T>::from_f32(ddt);
        if (a.has_z) *to(g.dz) = Elem<T>::from_f32(dz);
        dskip += dy * x;
        dbias += ddt;
      }
      // the workgroup's dB and dC of these tokens, waves in order
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          tiles[buf][wave][0][i][(4 * e + (lane >> 4)) * 16 + j] = tb[i][e];
          tiles[buf][wave][1][i][(4 * e + (lane >> 4)) * 16 + j] = tc[i][e];
        }
      __syncthreads();
      const int64_t row = ((int64_t)in_group * a.tokens + t) * a.G + group;
#pragma unroll
      for (int el = threadIdx.x; el < 2 * NS * 256; el += THREADS) {
        const int which = el / (NS * 256), i = el / 256 % NS, tk = el / 16 % 16, n = el % 16 + 16 * i;
        float sum = 0.f;
#pragma unroll
        for (int wv = 0; wv < WV; ++wv) sum += tiles[buf][wv][which][i][el % 256];
        if (n < a.N && t + tk < end) ((which ? w.dc : w.db) + row * a.N)[(uint32_t)(tk * a.G * a.N + n)] = sum;
      }
      buf ^= 1;
      if ((q & 3) == 0 && q > 0) {
        // every wave has read its last of this tile before the barrier above
        tile.store(a, bc, t - kScanTile, end);
        __syncthreads();
      }
      there = ch.active;
      tokens = 16;
    }
  };

  float h[NS], gr[NS];
  // gradient of the state of sequence n at `end`, or at the slot's end
  auto leaving = [&](int n, int end) {
    load_state<NS>(end <= hi ? g.dht : w.adj, end <= hi ? n : slot + 1, a, ch, gr);
  };
  int n = uniform(seqs.from(lo)), at = lo;
  if (n > 0) {
    const int end = uniform((int)seqs.end(n - 1));
    if (end > lo) {  // entered from an earlier slot
      at = end;
      load_state<NS>(w.hend, slot - 1, a, ch, h);
      leaving(n - 1, end);
      range(lo, end < hi ? end : hi, groups_at(lo, n - 1, slot), h, gr);
    }
  }
#pragma unroll
  for (int i = 0; i < NS; ++i) h[i] = 0.f;
  for (; n < a.n_seqs; ++n) {
    const Span tok = seqs.next(n, &at);
    const int start = uniform(tok.start), end = uniform(tok.end);
    if (!own.last && start >= hi) break;
    leaving(n, end);
    if (start < end) range(start, end < hi ? end : hi, groups_at(start, n, slot), h, gr);
    if (g.dh0) store_state<NS>(g.dh0, n, a, ch, gr);
  }
  store_state<NS>(w.da, slot, a, ch, dA);
  dskip = row_sum(dskip);
  dbias = row_sum(dbias);
  if (ch.active && j == 0) {
    w.dskip[(int64_t)slot * a.D + ch.c] = dskip;
    w.dbias[(int64_t)slot * a.D + ch.c] = dbias;
  }
}

// The sums of dA, dskip and dbias over the slots: 64
// columns a workgroup, rows dealt to 16 waves whose sums are added in order.
__global__ void __launch_bounds__(1024)
scan_sum_slots(const float* __restrict__ da, const float* __restrict__ ds, const float* __restrict__ db, int n_rows,
               int64_t dn, int D, float* __restrict__ dA, float* __restrict__ dskip, float* __restrict__ dbias) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t col = (int64_t)blockIdx.x * 64 + lane, cols = dn;
  const float* __restrict__ rows = da;
  float* out = dA;
  if (col >= dn) {
    col -= dn;
    cols = D;
    rows = col < D ? ds : db;
    out = col < D ? dskip : dbias;
    if (col >= D) col -= D;
    if (col >= D) out = nullptr;
  }
  float v = 0.f;
  if (out)
    for (int r = wave; r < n_rows; r += 16) v += rows[r * cols + col];
  sums[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || !out) return;
  v = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) v += sums[w][lane];
  out[col] = v;
}

// dB and dC: the channel workgroups' sums added.
template <typename T>
__global__ void __launch_bounds__(256)
scan_sum_channels(const float* __restrict__ db, const float* __restrict__ dc, int n_rows, int64_t cols,
                  const int32_t* __restrict__ cu, int n_seqs, int64_t per_token, T* __restrict__ dB,
                  T* __restrict__ dC) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= cols) return;
  if (cu && at / per_token >= cu[n_seqs]) return;  // behind the last sequence
  const float* __restrict__ rows = blockIdx.y ? dc : db;
  float v = 0.f;
#pragma unroll 8
  for (int r = 0; r < n_rows; ++r) v += rows[r * cols + at];
  (blockIdx.y ? dC : dB)[at] = Elem<T>::from_f32(v);
}

// ---- launches ------------------------------------------------------------------
template <typename F>
int launch_chain(const ScanArgs& a, F* hend, F* adj, const F* sum, const int* kind, hipStream_t st) {
  const int64_t dn = (int64_t)a.D * a.N;
  // loads ahead: four slots while a wave has no more, else sixteen (32 slots: 138.5 us for the whole call with 4,
  // 141 with 16; 512 slots: 64.0 and 63.3)
  return (int)launch_kernel(a.n_slots <= 4 * kChainWaves ? scan_chain<4> : scan_chain<16>,
                            dim3((unsigned)ceil_div(dn, 64), adj ? 2 : 1), dim3(64 * kChainWaves), st, a.A, dn, a.N,
                            a.D, (int)a.n_slots, hend, adj, sum, kind);
}

template <typename T, int NS>
int forward_t(ScanArgs a, const ScanPlan& p, void* o, float* ht, void* ws, hipStream_t st) {
  a.slot = p.slot;
  a.n_slots = p.n_slots;
  a.blocks_per_group = (int)ceil_div(a.D / a.G, 16 * kScanWaves);
  float *hend = nullptr, *sum = nullptr;
  int* kind = nullptr;
  if (p.carry) {
    hend = (float*)((char*)ws + p.hend_off);
    sum = (float*)((char*)ws + p.sum_off);
    kind = (int*)((char*)ws + p.kind_off);
    const hipError_t e = launch_kernel(scan_forward<T, NS, kState, false>, work_grid(a), dim3(64 * kScanWaves), st, a,
                                       hend, sum, kind, (T*)nullptr, (float*)nullptr);
    if (e != hipSuccess) return (int)e;
    const int err = launch_chain(a, hend, (float*)nullptr, sum, kind, st);
    if (err != 0) return err;
  }
  return (int)launch_kernel(a.N < 4 * NS ? scan_forward<T, NS, kOutput, true> : scan_forward<T, NS, kOutput, false>,
                            work_grid(a), dim3(64 * kScanWaves), st, a, hend, sum, kind, (T*)o, ht);
}

template <typename T>
int step_t(const ScanArgs& a, float* state, void* o, hipStream_t st) {
  auto go = [&](auto lpc, auto vec, auto seqs) {
    const int64_t n_far = ceil_div(a.tokens, seqs.value), blocks = ceil_div(n_far * a.D * lpc.value, 256);
    return (int)launch_kernel(scan_step<T, lpc.value, vec.value, seqs.value>, dim3((unsigned)blocks), dim3(256), st, a,
                              state, (T*)o, (int)n_far);
  };
  const int per_channel = scan_step_lanes(a.N);
  auto shape = [&](auto lpc, auto vec) {
    return scan_step_seqs(a.tokens, a.D, a.N) > 1 ? go(lpc, vec, std::integral_constant<int, kScanStepSeqs>{})
                                                  : go(lpc, vec, std::integral_constant<int, 1>{});
  };
  auto lanes = [&](auto vec) {
    if (per_channel == 1) return shape(std::integral_constant<int, 1>{}, vec);
    if (per_channel == 2) return shape(std::integral_constant<int, 2>{}, vec);
    if (per_channel == 4) return shape(std::integral_constant<int, 4>{}, vec);
    if (per_channel == 8) return shape(std::integral_constant<int, 8>{}, vec);
    return shape(std::integral_constant<int, 16>{}, vec);
  };
  return a.N % 4 == 0 ? lanes(std::true_type{}) : lanes(std::false_type{});
}

// f(element type, states per lane) for the forward scans, which share a
// channel's states among 4 lanes, and for the backward scan (16 lanes)
template <typename F>
int dispatch_quads(int is_bf16, int N, F&& f) {
  auto states = [&](auto t) {
    return N <= 4    ? f(t, std::integral_constant<int, 1>{})
           : N <= 8  ? f(t, std::integral_constant<int, 2>{})
           : N <= 16 ? f(t, std::integral_constant<int, 4>{})
           : N <= 32 ? f(t, std::integral_constant<int, 8>{})
                     : f(t, std::integral_constant<int, 16>{});
  };
  return is_bf16 ? states(bf16_t{}) : states(float{});
}
template <typename F>
int dispatch_rows(int is_bf16, int N, F&& f) {
  auto states = [&](auto t) {
    const int ns = scan_ns(N);
    return ns == 1   ? f(t, std::integral_constant<int, 1>{})
           : ns == 2 ? f(t, std::integral_constant<int, 2>{})
                     : f(t, std::integral_constant<int, 4>{});
  };
  return is_bf16 ? states(bf16_t{}) : states(float{});
}

template <typename T, int NS>
int backward_t(ScanArgs a, const ScanBwdPlan& p, const ScanGrads& g, void* ws, hipStream_t st) {
  char* base = (char*)ws;
  auto at = [&](size_t off) { return (float*)(base + off); };
  a.slot = p.slot;
  a.n_slots = p.n_slots;
  float *hend = at(p.hend_off), *adj = at(p.adj_off), *sum = at(p.sum_off);
  int* kind = p.carry ? (int*)(base + p.kind_off) : nullptr;
  const GroupStates groups{at(p.group_off), at(p.group_sum_off)};
  if (a.tokens > 0) {
    a.blocks_per_group = (int)ceil_div(a.D / a.G, 16 * kScanWaves);
    const int err = dispatch_quads(sizeof(T) == 2, a.N, [&](auto t, auto ns) {
      typedef decltype(t) U;
      return (int)launch_kernel(scan_backward_states<U, ns.value>, work_grid(a), dim3(64 * kScanWaves), st, a,
                                (const U*)g.dout, g.dht, hend, adj, sum, kind, groups);
    });
    if (err != 0) return err;
  }
  if (p.carry) {
    const int err = launch_chain(a, hend, adj, sum, kind, st);
    if (err != 0) return err;
  }
  a.blocks_per_group = p.blocks_per_group;
  const ScanBwdBuffers w{hend, adj, groups, at(p.da_off), at(p.dskip_off), at(p.dbias_off), at(p.db_off),
                         at(p.dc_off)};
  const bool whole = a.N == 16 * NS && a.D / a.G % 16 == 0 && !a.cu && a.T % 16 == 0;
  auto* kernel = whole ? scan_backward<T, NS, false> : scan_backward<T, NS, true>;
  hipError_t e = launch_kernel(kernel, work_grid(a), dim3(64 * kScanBwdWaves), st, a, g, w);
  if (e != hipSuccess) return (int)e;
  const int64_t dn = (int64_t)a.D * a.N, cols = a.tokens * a.G * a.N;
  e = launch_kernel(scan_sum_slots, dim3((unsigned)ceil_div(dn + 2 * (int64_t)a.D, 64)), dim3(1024), st, w.da,
                    w.dskip, w.dbias, (int)p.n_slots, dn, a.D, g.dA, g.dskip, g.dbias);
  if (e != hipSuccess || cols == 0) return (int)e;
  return (int)launch_kernel(scan_sum_channels<T>, dim3((unsigned)ceil_div(cols, 256), 2), dim3(256), st, w.db, w.dc,
                            p.blocks_per_group, cols, a.cu, a.n_seqs, (int64_t)a.G * a.N, (T*)g.dB, (T*)g.dC);
}

}  // namespace

int launch_scan_forward(int is_bf16, const ScanArgs& a, const ScanPlan& p, void* o, float* ht, void* ws,
                        void* stream) {
  return dispatch_quads(is_bf16, a.N, [&](auto t, auto ns) {
    return forward_t<decltype(t), ns.value>(a, p, o, ht, ws, (hipStream_t)stream);
  });
}

int launch_scan_backward(int is_bf16, const ScanArgs& a, const ScanBwdPlan& p, const ScanGrads& g, void* ws,
                         void* stream) {
  return dispatch_rows(is_bf16, a.N, [&](auto t, auto ns) {
    return backward_t<decltype(t), ns.value>(a, p, g, ws, (hipStream_t)stream);
  });
}

int launch_scan_step(int is_bf16, const ScanArgs& a, float* state, void* o, void* stream) {
  return is_bf16 ? step_t<bf16_t>(a, state, o, (hipStream_t)stream) : step_t<float>(a, state, o, (hipStream_t)stream);
}

}  // namespace kda
