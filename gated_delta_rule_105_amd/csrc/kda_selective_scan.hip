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
// that bounds it: per element one exponential (four issue slots), the
// argument, the update (two) and the sum's product.
//
// Layout.  A row of 16 lanes holds one channel, lane j the states j, j + 16,
// ...: a wave has 4 channels, a workgroup of 4 waves 16.  Tokens come in
// groups of 16, and lane j also prepares token j of the group (delta,
// delta x, the gates), so that this work is done once per token and channel;
// inside the recurrence token k's values are lane k's, broadcast over the
// row as an operand modifier.  The 16 sums over the states of a group are
// taken together (row_sums), after which lane j holds token j's output.  B
// and C of 64 tokens are staged in LDS as fp32, [state][token] with rows of
// 68 words: four tokens are one 16-byte read, free of bank conflicts.
//
// The time axis is cut into slots when the channels alone do not fill the
// device.  A first launch scans every slot that a sequence leaves
// unfinished, from a zero state if the sequence entered it from an earlier
// slot, and keeps the state it hands on and the slot's sum of delta; the
// second composes the state entering each slot from those,
//   h <- exp(A sum delta) h + h_slot,
// and scans it for good.  Slots are ranges of the batch's tokens, whatever
// its sequences are: a workgroup walks the sequences of its slot, and a
// token range that ends inside a group leaves the state alone (delta = 0).
#include "kda_layer_device.h"

namespace kda {

namespace {

constexpr int kTileLd = kScanTile + 4;  // words per state of a staged tile

// exp(delta A) = exp2(delta A2).  Finite, so that the tokens past a range's
// end (delta = 0) keep the state whatever A is; NaN stays NaN.
__device__ __forceinline__ float log2_rate(float a) {
  const float v = a * kLog2e;
  return v < -3.4e38f ? -3.4e38f : v > 3.4e38f ? 3.4e38f : v;
}

// The channel of a row of 16 lanes.
struct Channel {
  int g, c;      // group, channel (a real one also where the lanes are idle)
  bool active;
};
__device__ __forceinline__ Channel channel_of(const ScanArgs& a, int block, int in_block, int per_block) {
  const int per_group = a.D / a.G, g = block / a.blocks_per_group;
  const int at = (block - g * a.blocks_per_group) * per_block + in_block;
  return Channel{g, g * per_group + (at < per_group ? at : per_group - 1), at < per_group};
}

// Workgroup -> (slot, channel block), consecutive channel blocks of a slot on
// one XCD (workgroups are dealt to the 8 XCDs in turn): their rows share
// cache lines.  False past the end.
__device__ __forceinline__ bool work_of(const ScanArgs& a, int64_t* slot, int* block) {
  const int64_t n_blocks = (int64_t)a.G * a.blocks_per_group, total = a.n_slots * n_blocks;
  const int64_t id = (int64_t)(blockIdx.x & 7) * ((total + 7) / 8) + (blockIdx.x >> 3);
  *slot = id / n_blocks;
  *block = (int)(id - *slot * n_blocks);
  return id < total && (int64_t)(blockIdx.x >> 3) < (total + 7) / 8;
}
inline dim3 work_grid(const ScanArgs& a) {
  const int64_t total = a.n_slots * a.G * a.blocks_per_group;
  return dim3((unsigned)((total + 7) / 8 * 8));
}

// Per-channel constants of a lane.
template <int NS>
struct Rates {
  float A2[NS];  // log2 e times A, 0 for states past N
  float skip, bias;
  __device__ __forceinline__ void load(const ScanArgs& a, int c, int j) {
#pragma unroll
    for (int i = 0; i < NS; ++i) A2[i] = j + 16 * i < a.N ? log2_rate(a.A[(int64_t)c * a.N + j + 16 * i]) : 0.f;
    skip = a.skip ? a.skip[c] : 0.f;
    bias = a.bias ? a.bias[c] : 0.f;
  }
};

template <int NS>
__device__ __forceinline__ void load_state(const float* __restrict__ p, int64_t row, const ScanArgs& a, int c, int j,
                                           float (&h)[NS]) {
#pragma unroll
  for (int i = 0; i < NS; ++i)
    h[i] = p && j + 16 * i < a.N ? p[(row * a.D + c) * a.N + j + 16 * i] : 0.f;
}
template <int NS>
__device__ __forceinline__ void store_state(float* __restrict__ p, int64_t row, const ScanArgs& a, const Channel& ch,
                                            int j, const float (&h)[NS]) {
  if (!ch.active) return;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (j + 16 * i < a.N) p[(row * a.D + ch.c) * a.N + j + 16 * i] = h[i];
}

// The state entering slot `slot` of a sequence that started at token lo.
template <int NS>
__device__ __forceinline__ void incoming(const ScanArgs& a, const float* __restrict__ hend,
                                         const float* __restrict__ sum, int64_t lo, int64_t slot, int c, int j,
                                         const Rates<NS>& r, float (&h)[NS]) {
  int64_t i = lo / a.slot;
  load_state<NS>(hend, i, a, c, j, h);
  for (++i; i < slot; ++i) {
    float e[NS];
    load_state<NS>(hend, i, a, c, j, e);
    const float sd = sum[i * a.D + c];
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = exp2_fast(sd * r.A2[n]) * h[n] + e[n];
  }
}

// Tiles of B and C: element (n, t) of tokens [t0, t0 + TOK) of group g,
// zero past the range's end and past N.  A thread holds one state of every
// (THREADS / 16)-th token.
template <typename T, int NS, int TOK, int THREADS>
struct TileLoad {
  static constexpr int PER = TOK * 16 / THREADS;  // tokens a thread
  float b[NS][PER], c[NS][PER];
  __device__ __forceinline__ void load(const ScanArgs& a, int g, int64_t t0, int64_t end) {
    const int n = threadIdx.x & 15, t = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int64_t tok = t0 + t + k * (THREADS / 16);
        const bool there = n + 16 * i < a.N && tok < end;
        const int at = g * a.N + n + 16 * i;
        b[i][k] = there ? load_f32((const T*)a.Bm + tok * a.ld_b + at) : 0.f;
        c[i][k] = there ? load_f32((const T*)a.Cm + tok * a.ld_c + at) : 0.f;
      }
  }
  // s: [2][NS * 16][LD], B first
  template <int LD>
  __device__ __forceinline__ void store(float* s, int at = 0) const {
    const int n = threadIdx.x & 15, t = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        s[(n + 16 * i) * LD + at + t + k * (THREADS / 16)] = b[i][k];
        s[(NS * 16 + n + 16 * i) * LD + at + t + k * (THREADS / 16)] = c[i][k];
      }
  }
};

// Lane j's token of a group: its inputs, and what the recurrence takes of it.
template <typename T>
struct Token {
  float x, dt, z;
  __device__ __forceinline__ void load(const ScanArgs& a, const Channel& ch, int64_t t, int64_t end) {
    x = dt = z = 0.f;
    if (t >= end || !ch.active) return;
    x = load_f32((const T*)a.x + t * a.ld_x + ch.c);
    dt = load_f32((const T*)a.dt + t * a.ld_dt + ch.c);
    if (a.z) z = load_f32((const T*)a.z + t * a.ld_z + ch.c);
  }
};

// Scans tokens [t0, end) of one sequence from h.  OUT: writes o; else only
// the state, and returns the sum of delta (this lane's tokens of it).
template <typename T, int NS, bool OUT>
__device__ __forceinline__ float scan_range(const ScanArgs& a, const Channel& ch, const Rates<NS>& r, int j,
                                            int64_t t0, int64_t end, float* s, float (&h)[NS], T* __restrict__ o) {
  constexpr int THREADS = 64 * kScanWaves, BUF = 2 * NS * 16 * kTileLd;
  TileLoad<T, NS, kScanTile, THREADS> tile;
  Token<T> next;
  float sum = 0.f;
  tile.load(a, ch.g, t0, end);
  next.load(a, ch, t0 + j, end);
  __syncthreads();  // the range before may still be reading
  tile.template store<kTileLd>(s);
  __syncthreads();
  int buf = 0;
  for (int64_t t = t0; t < end; t += kScanTile) {
    const bool more = t + kScanTile < end;
    if (more) tile.load(a, ch.g, t + kScanTile, end);
    const float* sb = s + buf * BUF + j * kTileLd;
    const float* sc = sb + NS * 16 * kTileLd;
    for (int q = 0; q < kScanTile && t + q < end; q += 16) {
      const Token<T> cur = next;
      const int64_t tok = t + q + j;
      next.load(a, ch, tok + 16, end);
      const float v = cur.dt + r.bias;
      const bool there = tok < end && ch.active;
      const float delta = there ? (a.softplus ? softplus(v) : v) : 0.f;
      const float dx = there ? delta * cur.x : 0.f;
      if (!OUT) sum += delta;
      float p[16];
      static_for<4>([&](auto k4) {
        f32x4 B[NS], C[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          B[i] = *(const f32x4*)(sb + i * 16 * kTileLd + q + 4 * k4);
          if (OUT) C[i] = *(const f32x4*)(sc + i * 16 * kTileLd + q + 4 * k4);
        }
        static_for<4>([&](auto e) {
          constexpr int k = 4 * decltype(k4)::value + decltype(e)::value;
          const float dk = row_bcast<k>(delta), xk = row_bcast<k>(dx);
          float y = 0.f;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            h[i] = exp2_fast(dk * r.A2[i]) * h[i] + xk * B[i][decltype(e)::value];
            if (OUT) y += C[i][decltype(e)::value] * h[i];
          }
          p[k] = y;
        });
      });
      if (OUT) {
        float y = row_sums(p, j) + r.skip * cur.x;
        if (a.z) y *= cur.z * sigmoid(cur.z);
        if (there) o[tok * a.D + ch.c] = Elem<T>::from_f32(y);
      }
    }
    if (more) {
      buf ^= 1;
      tile.template store<kTileLd>(s + buf * BUF);
      __syncthreads();
    }
  }
  return sum;
}

// Forward.  OUT = false: the first launch, over what a slot leaves unfinished.
template <typename T, int NS, bool OUT>
__global__ void __launch_bounds__(64 * kScanWaves)
scan_forward(const ScanArgs a, float* __restrict__ hend, float* __restrict__ sum, T* __restrict__ o,
             float* __restrict__ ht) {
  __shared__ __align__(16) float s[2 * 2 * NS * 16 * kTileLd];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), j = lane & 15;
  int64_t slot;
  int block;
  if (!work_of(a, &slot, &block)) return;
  const Channel ch = channel_of(a, block, wave * 4 + (lane >> 4), 4 * kScanWaves);
  Rates<NS> r;
  r.load(a, ch.c, j);
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  const int64_t lo = slot * a.slot, hi = lo + a.slot < a.tokens ? lo + a.slot : a.tokens;
  float h[NS];
  if (!OUT) {
    const int n = seqs.from(hi) - 1;  // the last sequence that starts in the slot or before
    if (slot + 1 >= a.n_slots || n < 0 || seqs.end(n) <= hi) return;
    const int64_t start = seqs.start(n);
    const bool own = start >= lo;
    load_state<NS>(own ? a.h0 : nullptr, n, a, ch.c, j, h);
    const float d = scan_range<T, NS, false>(a, ch, r, j, own ? start : lo, hi, s, h, (T*)nullptr);
    store_state<NS>(hend, slot, a, ch, j, h);
    const float total = row_sum(d);
    if (!own && ch.active && j == 0) sum[slot * a.D + ch.c] = total;
    return;
  }
  int n = seqs.from(lo);
  if (n > 0 && seqs.end(n - 1) > lo) {  // a sequence that entered from an earlier slot
    const int64_t end = seqs.end(n - 1);
    incoming<NS>(a, hend, sum, seqs.start(n - 1), slot, ch.c, j, r, h);
    scan_range<T, NS, true>(a, ch, r, j, lo, end < hi ? end : hi, s, h, o);
    if (ht && end <= hi) store_state<NS>(ht, n - 1, a, ch, j, h);
  }
  // those that start here; the last slot also has the empty ones behind the last token
  for (; n < a.n_seqs && (slot + 1 >= a.n_slots || seqs.start(n) < hi); ++n) {
    const int64_t start = seqs.start(n), end = seqs.end(n);
    load_state<NS>(a.h0, n, a, ch.c, j, h);
    if (start < end) scan_range<T, NS, true>(a, ch, r, j, start, end < hi ? end : hi, s, h, o);
    if (ht && end <= hi) store_state<NS>(ht, n, a, ch, j, h);
  }
}

// ---- one token ---------------------------------------------------------------
// The state is read once and written once, which is all the step costs: a
// lane owns 4 consecutive states (16 bytes), LPC lanes a channel.  Without
// VEC (N no multiple of 4) the same states are loaded one by one.
template <typename T, int LPC, bool VEC>
__global__ void __launch_bounds__(256) scan_step(const ScanArgs a, float* __restrict__ state, T* __restrict__ o) {
  const int sub = threadIdx.x % LPC;
  const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPC;
  const int64_t seq = id / a.D;
  const int c = (int)(id - seq * a.D);
  if (seq >= a.tokens) return;
  const int g = c / (a.D / a.G), n0 = sub * 4;
  float* __restrict__ st = state + id * a.N;
  const float* __restrict__ A = a.A + (int64_t)c * a.N;
  const T* __restrict__ Bm = (const T*)a.Bm + seq * a.ld_b + (int64_t)g * a.N;
  const T* __restrict__ Cm = (const T*)a.Cm + seq * a.ld_c + (int64_t)g * a.N;
  float h[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f}, B[4] = {0.f, 0.f, 0.f, 0.f},
        C[4] = {0.f, 0.f, 0.f, 0.f};
  if (VEC) {
    if (n0 < a.N) {
      load_vec<float, 4>(st + n0, h);
      load_vec<float, 4>(A + n0, r);
      load_vec<T, 4>(Bm + n0, B);
      load_vec<T, 4>(Cm + n0, C);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < a.N) {
        h[i] = st[n0 + i];
        r[i] = A[n0 + i];
        B[i] = load_f32(Bm + n0 + i);
        C[i] = load_f32(Cm + n0 + i);
      }
  }
  const float x = load_f32((const T*)a.x + seq * a.ld_x + c);
  const float v = load_f32((const T*)a.dt + seq * a.ld_dt + c) + (a.bias ? a.bias[c] : 0.f);
  const float z = a.z ? load_f32((const T*)a.z + seq * a.ld_z + c) : 0.f;
  const float delta = a.softplus ? softplus(v) : v;
  float y = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = exp2_fast(delta * log2_rate(r[i])) * h[i] + delta * x * B[i];
    y += C[i] * h[i];
  }
  if (VEC) {
    if (n0 < a.N) store_vec<float, 4>(st + n0, h);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < a.N) st[n0 + i] = h[i];
  }
  if constexpr (LPC >= 2) y += dpp<kPairSwap>(y);
  if constexpr (LPC >= 4) y += dpp<kQuadMirror>(y);
  if constexpr (LPC >= 8) y += dpp<kHalfMirror>(y);
  if constexpr (LPC >= 16) y += dpp<kRowMirror>(y);
  if (sub == 0) {
    y += (a.skip ? a.skip[c] : 0.f) * x;
    if (a.z) y *= z * sigmoid(z);
    o[id] = Elem<T>::from_f32(y);
  }
}

// ---- backward ------------------------------------------------------------------
// Three launches.  The first, only when sequences pass from slot to slot,
// walks every slot once and leaves what its neighbours need: the state it
// hands on (as forward), the gradient it hands back (the part of the state
// gradient at its start that its own tokens make, summed forward in time
// with the running product of the decays), and its sum of delta.  The second
// takes a slot with the state entering it and the gradient of the state
// leaving it composed from those: it runs forward leaving the state before
// every group of 16 tokens in LDS, then walks the groups back, redoing each
// group's recurrence in registers.  The third adds the partial sums.
//
// Sums over channels (dB, dC) of one token are products of the 4 rows of a
// wave: v_mfma_f32_16x16x4f32 with the token's dy (delta x) in row k of the
// left operand, zeros in the others, and h (dh) as it lies in the registers,
// so a group's 16 products accumulate into one [16 tokens][16 states] tile.
// The matrix pipe does them beside the vector unit.  The tiles of the waves
// are added in LDS, those of the workgroups by the third launch.
template <typename T>
struct TokenGrad : Token<T> {
  float dout;
  __device__ __forceinline__ void load(const ScanArgs& a, const T* __restrict__ g, const Channel& ch, int64_t t,
                                       int64_t end) {
    Token<T>::load(a, ch, t, end);
    dout = t < end && ch.active ? load_f32(g + t * a.D + ch.c) : 0.f;
  }
};

// Tokens [t0, end) from state h: the state after them, and in adj the sum of
// the gradients they send to the state before them, times `run` (the product
// of their decays when it starts at 1).  Returns this lane's part of the sum
// of delta.
template <typename T, int NS>
__device__ __forceinline__ float carry_range(const ScanArgs& a, const T* __restrict__ dout, const Channel& ch,
                                             const Rates<NS>& r, int j, int64_t t0, int64_t end, float* s,
                                             float (&h)[NS], float (&adj)[NS], float (&run)[NS]) {
  constexpr int THREADS = 64 * kScanWaves;
  TileLoad<T, NS, kScanTile, THREADS> tile;
  TokenGrad<T> next;
  float sum = 0.f;
  next.load(a, dout, ch, t0 + j, end);
  for (int64_t t = t0; t < end; t += kScanTile) {
    tile.load(a, ch.g, t, end);
    __syncthreads();
    tile.template store<kTileLd>(s);
    __syncthreads();
    const float* sb = s + j * kTileLd;
    const float* sc = sb + NS * 16 * kTileLd;
    for (int q = 0; q < kScanTile && t + q < end; q += 16) {
      const TokenGrad<T> cur = next;
      const int64_t tok = t + q + j;
      next.load(a, dout, ch, tok + 16, end);
      const float v = cur.dt + r.bias;
      const bool there = tok < end && ch.active;
      const float delta = there ? (a.softplus ? softplus(v) : v) : 0.f;
      const float dx = there ? delta * cur.x : 0.f;
      const float dy = there ? (a.z ? cur.dout * (cur.z * sigmoid(cur.z)) : cur.dout) : 0.f;
      sum += delta;
      static_for<4>([&](auto k4) {
        f32x4 B[NS], C[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          B[i] = *(const f32x4*)(sb + i * 16 * kTileLd + q + 4 * k4);
          C[i] = *(const f32x4*)(sc + i * 16 * kTileLd + q + 4 * k4);
        }
        static_for<4>([&](auto e) {
          constexpr int k = 4 * decltype(k4)::value + decltype(e)::value;
          const float dk = row_bcast<k>(delta), xk = row_bcast<k>(dx), gk = row_bcast<k>(dy);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const float d = exp2_fast(dk * r.A2[i]);
            h[i] = d * h[i] + xk * B[i][decltype(e)::value];
            run[i] *= d;
            adj[i] += run[i] * (C[i][decltype(e)::value] * gk);
          }
        });
      });
    }
  }
  return sum;
}

template <typename T, int NS>
__global__ void __launch_bounds__(64 * kScanWaves)
scan_backward_carry(const ScanArgs a, const T* __restrict__ dout, const float* __restrict__ dht,
                    float* __restrict__ hend, float* __restrict__ adj, float* __restrict__ sum) {
  __shared__ __align__(16) float s[2 * NS * 16 * kTileLd];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), j = lane & 15;
  int64_t slot;
  int block;
  if (!work_of(a, &slot, &block)) return;
  const Channel ch = channel_of(a, block, wave * 4 + (lane >> 4), 4 * kScanWaves);
  Rates<NS> r;
  r.load(a, ch.c, j);
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  const int64_t lo = slot * a.slot, hi = lo + a.slot < a.tokens ? lo + a.slot : a.tokens;
  float h[NS], g[NS], run[NS];
  int n = seqs.from(lo);
  if (n > 0 && seqs.end(n - 1) > lo) {  // entered from an earlier slot
    const int64_t end = seqs.end(n - 1);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      h[i] = g[i] = 0.f;
      run[i] = 1.f;
    }
    const float d = carry_range<T, NS>(a, dout, ch, r, j, lo, end < hi ? end : hi, s, h, g, run);
    if (end <= hi) {
      float last[NS];
      load_state<NS>(dht, n - 1, a, ch.c, j, last);
#pragma unroll
      for (int i = 0; i < NS; ++i) g[i] += run[i] * last[i];
    } else {
      store_state<NS>(hend, slot, a, ch, j, h);
      const float total = row_sum(d);
      if (ch.active && j == 0) sum[slot * a.D + ch.c] = total;
    }
    store_state<NS>(adj, slot, a, ch, j, g);
  }
  n = seqs.from(hi) - 1;
  if (n >= 0 && seqs.start(n) >= lo && seqs.end(n) > hi) {  // starts here and goes on
    load_state<NS>(a.h0, n, a, ch.c, j, h);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      g[i] = 0.f;
      run[i] = 1.f;
    }
    carry_range<T, NS>(a, dout, ch, r, j, seqs.start(n), hi, s, h, g, run);
    store_state<NS>(hend, slot, a, ch, j, h);
  }
}

// What the second launch reads and writes beside the inputs.
struct ScanBwdBuffers {
  const float *hend, *adj, *sum;  // of every slot; null without carry
  float *da, *dskip, *dbias;      // per slot
  float *db, *dc;                 // per workgroup of channels
};

template <typename T, int NS>
struct BwdLds {
  static constexpr int WV = scan_bwd_waves(NS), SLOT = scan_bwd_slot(NS), LD = SLOT + 4;
  __align__(16) float bc[2 * NS * 16 * LD];     // B, C of the slot
  float before[WV][SLOT / 16][NS][64];          // state before every group
  float tiles[2][WV][2][NS][256];               // dB, dC of a group, per wave
};

template <typename T, int NS>
__global__ void __launch_bounds__(64 * scan_bwd_waves(NS))
scan_backward(const ScanArgs a, const ScanGrads g, const ScanBwdBuffers w) {
  typedef BwdLds<T, NS> Lds;
  constexpr int WV = Lds::WV, LD = Lds::LD, THREADS = 64 * WV;
  __shared__ Lds s;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), j = lane & 15;
  int64_t slot;
  int block;
  if (!work_of(a, &slot, &block)) return;
  const Channel ch = channel_of(a, block, wave * 4 + (lane >> 4), 4 * WV);
  const int in_group = block - ch.g * a.blocks_per_group;
  Rates<NS> r;
  r.load(a, ch.c, j);
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  const int64_t lo = slot * a.slot, hi = lo + a.slot < a.tokens ? lo + a.slot : a.tokens;
  const T* __restrict__ dout = (const T*)g.dout;
  float dA[NS], dskip = 0.f, dbias = 0.f;
#pragma unroll
  for (int i = 0; i < NS; ++i) dA[i] = 0.f;
  int buf = 0;

  // tokens [t0, end) of one sequence: h the state before them, gr the
  // gradient of the state after them; leaves the gradient of h in gr
  auto range = [&](int64_t t0, int64_t end, float(&h)[NS], float(&gr)[NS]) {
    const int groups = (int)((end - t0 + 15) / 16);
    __syncthreads();  // the range before may still be reading
    for (int t = 0; t < groups * 16; t += kScanTile) {
      TileLoad<T, NS, kScanTile, THREADS> tile;
      tile.load(a, ch.g, t0 + t, end);
      tile.template store<LD>(s.bc, t);
    }
    __syncthreads();
    const float* sb = s.bc + j * LD;
    const float* sc = sb + NS * 16 * LD;
    for (int q = 0; q < groups; ++q) {
#pragma unroll
      for (int i = 0; i < NS; ++i) s.before[wave][q][i][lane] = h[i];
      if (q + 1 == groups) break;
      Token<T> cur;
      cur.load(a, ch, t0 + q * 16 + j, end);
      const float v = cur.dt + r.bias;
      const float delta = ch.active ? (a.softplus ? softplus(v) : v) : 0.f;
      const float dx = delta * cur.x;
      static_for<4>([&](auto k4) {
        f32x4 B[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) B[i] = *(const f32x4*)(sb + i * 16 * LD + q * 16 + 4 * k4);
        static_for<4>([&](auto e) {
          constexpr int k = 4 * decltype(k4)::value + decltype(e)::value;
          const float dk = row_bcast<k>(delta), xk = row_bcast<k>(dx);
#pragma unroll
          for (int i = 0; i < NS; ++i)
            h[i] = exp2_fast(dk * r.A2[i]) * h[i] + xk * B[i][decltype(e)::value];
        });
      });
    }
    TokenGrad<T> next;
    next.load(a, dout, ch, t0 + (groups - 1) * 16 + j, end);
    for (int q = groups - 1; q >= 0; --q) {
      const TokenGrad<T> cur = next;
      const int64_t tok = t0 + q * 16 + j;
      if (q > 0) next.load(a, dout, ch, tok - 16, end);
      const float v = cur.dt + r.bias;
      const bool there = tok < end && ch.active;
      const float delta = there ? (a.softplus ? softplus(v) : v) : 0.f;
      const float dx = there ? delta * cur.x : 0.f;
      float first[NS], hh[16][NS], dd[16][NS], p[16];
#pragma unroll
      for (int i = 0; i < NS; ++i) first[i] = s.before[wave][q][i][lane];
      static_for<4>([&](auto k4) {
        f32x4 B[NS], C[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          B[i] = *(const f32x4*)(sb + i * 16 * LD + q * 16 + 4 * k4);
          C[i] = *(const f32x4*)(sc + i * 16 * LD + q * 16 + 4 * k4);
        }
        static_for<4>([&](auto e) {
          constexpr int k = 4 * decltype(k4)::value + decltype(e)::value;
          const float dk = row_bcast<k>(delta), xk = row_bcast<k>(dx);
          float y = 0.f;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            dd[k][i] = exp2_fast(dk * r.A2[i]);
            hh[k][i] = dd[k][i] * (k ? hh[k ? k - 1 : 0][i] : first[i]) + xk * B[i][decltype(e)::value];
            y += C[i][decltype(e)::value] * hh[k][i];
          }
          p[k] = y;
        });
      });
      float dy = cur.dout;
      if (a.z) {
        const float y = row_sums(p, j) + r.skip * cur.x, sg = sigmoid(cur.z);
        const float dz = cur.dout * y * (sg * (1.f + cur.z * (1.f - sg)));
        dy = cur.dout * (cur.z * sg);
        if (there) ((T*)g.dz)[tok * a.D + ch.c] = Elem<T>::from_f32(dz);
      }
      dy = there ? dy : 0.f;
      f32x4 tb[NS], tc[NS];
#pragma unroll
      for (int i = 0; i < NS; ++i) tb[i] = tc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
      float p1[16], p2[16];
      static_for<4>([&](auto k4r) {
        constexpr int k4 = 3 - decltype(k4r)::value;
        f32x4 B[NS], C[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          B[i] = *(const f32x4*)(sb + i * 16 * LD + q * 16 + 4 * k4);
          C[i] = *(const f32x4*)(sc + i * 16 * LD + q * 16 + 4 * k4);
        }
        static_for<4>([&](auto er) {
          constexpr int e = 3 - decltype(er)::value, k = 4 * k4 + e;
          const float dk = row_bcast<k>(delta), gk = row_bcast<k>(dy);
          const float of_dy = j == k ? dy : 0.f, of_dx = j == k ? dx : 0.f;
          p1[k] = p2[k] = 0.f;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const float dh = C[i][e] * gk + gr[i];
            tc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(of_dy, hh[k][i], tc[i], 0, 0, 0);
            tb[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(of_dx, dh, tb[i], 0, 0, 0);
            gr[i] = dh * dd[k][i];
            const float m = gr[i] * (k ? hh[k ? k - 1 : 0][i] : first[i]);
            p1[k] += m * r.A2[i];
            p2[k] += dh * B[i][e];
            dA[i] += m * dk;
          }
        });
      });
      const float s1 = kLn2 * row_sums(p1, j), s2 = row_sums(p2, j);
      const float ddt = (s1 + cur.x * s2) * (a.softplus ? sigmoid(v) : 1.f);
      if (there) {
        ((T*)g.dx)[tok * a.D + ch.c] = Elem<T>::from_f32(r.skip * dy + delta * s2);
        ((T*)g.ddt)[tok * a.D + ch.c] = Elem<T>::from_f32(ddt);
        dskip += dy * cur.x;
        dbias += ddt;
      }
      // the workgroup's dB and dC of these tokens, waves in order
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = (4 * (lane >> 4) + e) * 16 + j;
          s.tiles[buf][wave][0][i][at] = tb[i][e];
          s.tiles[buf][wave][1][i][at] = tc[i][e];
        }
      __syncthreads();
#pragma unroll
      for (int at = threadIdx.x; at < 2 * NS * 256; at += THREADS) {
        const int which = at / (NS * 256), i = at / 256 % NS, el = at % 256, n = (el & 15) + 16 * i;
        const int64_t t = t0 + q * 16 + (el >> 4);
        float sum = 0.f;
#pragma unroll
        for (int wv = 0; wv < WV; ++wv) sum += s.tiles[buf][wv][which][i][el];
        if (n < a.N && t < end)
          (which ? w.dc : w.db)[((in_group * a.tokens + t) * a.G + ch.g) * a.N + n] = sum;
      }
      buf ^= 1;
    }
  };

  float h[NS], gr[NS];
  // gradient of the state of sequence n at `end`, or at the slot's end
  auto leaving = [&](int n, int64_t end) {
    if (end <= hi) {
      load_state<NS>(g.dht, n, a, ch.c, j, gr);
      return;
    }
    int64_t i = (end - 1) / a.slot;
    load_state<NS>(w.adj, i, a, ch.c, j, gr);
    for (--i; i > slot; --i) {
      float e[NS];
      load_state<NS>(w.adj, i, a, ch.c, j, e);
      const float sd = w.sum[i * a.D + ch.c];
#pragma unroll
      for (int k = 0; k < NS; ++k) gr[k] = exp2_fast(sd * r.A2[k]) * gr[k] + e[k];
    }
  };
  int n = seqs.from(lo);
  if (n > 0 && seqs.end(n - 1) > lo) {
    const int64_t end = seqs.end(n - 1);
    incoming<NS>(a, w.hend, w.sum, seqs.start(n - 1), slot, ch.c, j, r, h);
    leaving(n - 1, end);
    range(lo, end < hi ? end : hi, h, gr);
  }
  for (; n < a.n_seqs && (slot + 1 >= a.n_slots || seqs.start(n) < hi); ++n) {
    const int64_t start = seqs.start(n), end = seqs.end(n);
    load_state<NS>(a.h0, n, a, ch.c, j, h);
    leaving(n, end);
    if (start < end) range(start, end < hi ? end : hi, h, gr);
    if (g.dh0) store_state<NS>(g.dh0, n, a, ch, j, gr);
  }
  store_state<NS>(w.da, slot, a, ch, j, dA);
  dskip = row_sum(dskip);
  dbias = row_sum(dbias);
  if (ch.active && j == 0) {
    w.dskip[slot * a.D + ch.c] = dskip;
    w.dbias[slot * a.D + ch.c] = dbias;
  }
}

// Third launch, part one: dA, dskip and dbias, the slots' rows added: 64
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

// Part two: dB and dC, the channel workgroups' sums added.
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
template <typename T, int NS>
int forward_t(ScanArgs a, const ScanPlan& p, void* o, float* ht, void* ws, hipStream_t st) {
  a.slot = p.slot;
  a.n_slots = p.n_slots;
  a.blocks_per_group = (int)ceil_div(a.D / a.G, 4 * kScanWaves);
  float* hend = p.carry ? (float*)((char*)ws + p.hend_off) : nullptr;
  float* sum = p.carry ? (float*)((char*)ws + p.sum_off) : nullptr;
  if (p.carry) {
    const hipError_t e = launch_kernel(scan_forward<T, NS, false>, work_grid(a), dim3(64 * kScanWaves), st, a, hend,
                                       sum, (T*)nullptr, (float*)nullptr);
    if (e != hipSuccess) return (int)e;
  }
  return (int)launch_kernel(scan_forward<T, NS, true>, work_grid(a), dim3(64 * kScanWaves), st, a, hend, sum, (T*)o,
                            ht);
}

template <typename T>
int step_t(const ScanArgs& a, float* state, void* o, hipStream_t st) {
  auto go = [&](auto lpc, auto vec) {
    const int64_t blocks = ceil_div(a.tokens * a.D * lpc.value, 256);
    if (blocks > INT32_MAX) return (int)hipErrorInvalidValue;
    return (int)launch_kernel(scan_step<T, lpc.value, vec.value>, dim3((unsigned)blocks), dim3(256), st, a, state,
                              (T*)o);
  };
  auto lanes = [&](auto vec) {
    if (a.N <= 4) return go(std::integral_constant<int, 1>{}, vec);
    if (a.N <= 8) return go(std::integral_constant<int, 2>{}, vec);
    if (a.N <= 16) return go(std::integral_constant<int, 4>{}, vec);
    if (a.N <= 32) return go(std::integral_constant<int, 8>{}, vec);
    return go(std::integral_constant<int, 16>{}, vec);
  };
  return a.N % 4 == 0 ? lanes(std::true_type{}) : lanes(std::false_type{});
}

template <typename T, int NS>
int backward_t(ScanArgs a, const ScanBwdPlan& p, const ScanGrads& g, void* ws, hipStream_t st) {
  char* base = (char*)ws;
  auto at = [&](size_t off) { return (float*)(base + off); };
  a.slot = p.slot;
  a.n_slots = p.n_slots;
  float *hend = at(p.hend_off), *adj = at(p.adj_off), *sum = at(p.sum_off);
  hipError_t e;
  if (p.carry) {
    a.blocks_per_group = (int)ceil_div(a.D / a.G, 4 * kScanWaves);
    e = launch_kernel(scan_backward_carry<T, NS>, work_grid(a), dim3(64 * kScanWaves), st, a, (const T*)g.dout,
                      g.dht, hend, adj, sum);
    if (e != hipSuccess) return (int)e;
  }
  a.blocks_per_group = p.blocks_per_group;
  const ScanBwdBuffers w{hend, adj, sum, at(p.da_off), at(p.dskip_off), at(p.dbias_off), at(p.db_off), at(p.dc_off)};
  e = launch_kernel(scan_backward<T, NS>, work_grid(a), dim3(64 * scan_bwd_waves(NS)), st, a, g, w);
  if (e != hipSuccess) return (int)e;
  const int64_t dn = (int64_t)a.D * a.N, cols = a.tokens * a.G * a.N;
  e = launch_kernel(scan_sum_slots, dim3((unsigned)ceil_div(dn + 2 * (int64_t)a.D, 64)), dim3(1024), st, w.da,
                    w.dskip, w.dbias, (int)p.n_slots, dn, a.D, g.dA, g.dskip, g.dbias);
  if (e != hipSuccess || cols == 0) return (int)e;
  return (int)launch_kernel(scan_sum_channels<T>, dim3((unsigned)ceil_div(cols, 256), 2), dim3(256), st, w.db, w.dc,
                            p.blocks_per_group, cols, a.cu, a.n_seqs, (int64_t)a.G * a.N, (T*)g.dB, (T*)g.dC);
}

// f(element type, states per lane) for a call's type and number of states
template <typename F>
int dispatch(int is_bf16, int N, F&& f) {
  auto states = [&](auto t) {
    const int ns = scan_ns(N);
    return ns == 1   ? f(t, std::integral_constant<int, 1>{})
           : ns == 2 ? f(t, std::integral_constant<int, 2>{})
                     : f(t, std::integral_constant<int, 4>{});
  };
  return is_bf16 ? states(bf16_t{}) : states(float{});
}

}  // namespace

int launch_scan_forward(int is_bf16, const ScanArgs& a, const ScanPlan& p, void* o, float* ht, void* ws,
                        void* stream) {
  return dispatch(is_bf16, a.N, [&](auto t, auto ns) {
    return forward_t<decltype(t), ns.value>(a, p, o, ht, ws, (hipStream_t)stream);
  });
}

int launch_scan_backward(int is_bf16, const ScanArgs& a, const ScanBwdPlan& p, const ScanGrads& g, void* ws,
                         void* stream) {
  return dispatch(is_bf16, a.N, [&](auto t, auto ns) {
    return backward_t<decltype(t), ns.value>(a, p, g, ws, (hipStream_t)stream);
  });
}

int launch_scan_step(int is_bf16, const ScanArgs& a, float* state, void* o, void* stream) {
  return is_bf16 ? step_t<bf16_t>(a, state, o, (hipStream_t)stream) : step_t<float>(a, state, o, (hipStream_t)stream);
}

}  // namespace kda
