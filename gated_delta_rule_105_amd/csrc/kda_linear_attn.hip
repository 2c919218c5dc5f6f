// Linear attention with a decay for each head, for gfx950: whole sequences,
// one token, and gradients.
//
// Per sequence and head, with a_t = exp(min(g_t, 0)):
//   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// A chunk of C tokens, G the running sum of the log decays over it, S the
// state before it:
//   P = scale (Q K^T) o D,  D_ij = e^{G_i - G_j} for j <= i and 0 above,
//   O = P V + scale e^{G} Q S,   S <- e^{G_C} S + K^T (e^{G_C - G} V).
// No factor is above 1, so nothing overflows that the recurrence would not
// make overflow.  The running sums are kept in 64 bits: a decay between two
// tokens is the difference of two of them, which a strongly decaying token
// before both would take digits from in 32.
//
// The gradients are the same computation three times over.  dq is the forward
// form with (dout, v, k) for (q, k, v) and the transposed state; dv and dk are
// the form going back in time with (k, q, dout) and (v, dout, q):
//   dV = P^T dO + e^{G_C - G} K dS,   dS <- e^{G_C} dS + scale (e^G Q)^T dO,
// dS the gradient of the state after the chunk.  A decay stands in every
// product of a query at its token or later with a key before it, so with M =
// (Q K^T) o D o scale (dO V^T) below the diagonal
//   dg_t = sum_{i >= t > j} M_ij + sum_{s >= t} x_s + sum_{s < t} y_s + e^{G_C} <S, dS>,
// x_s = q_s . (the state's part of dq_s), y_s = k_s . (dS's part of dk_s),
// and because <S_end, dS> = e^{G_C} <S, dS> + sum y, all of it is the suffix
// sum of (row sum of M - column sum of M + x - y) plus <S_end, dS> of the end
// of the sequence or slot.
#include "kda_layer_device.h"
#include "kda_linear.h"

namespace kda {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kThreads = 256, kWaves = 4;

// Tokens of a chunk: both types then fill LDS alike.
template <typename T> constexpr int kTokens = sizeof(T) == 2 ? 64 : 32;

// Orders LDS accesses only: the next chunk's loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ---- LDS arrays ----------------------------------------------------------------
// [tokens][W], rows of W + 16 elements, in units of 4 elements; unit u of row
// t is at u ^ ((t >> 2) & 3).  16 rows at one unit (row fragments) and 4 rows
// by 4 units (transpose reads) are then in banks of their own, and for tiles
// that start at multiples of 16 a lane's offset is one register plus an
// immediate.
template <int W> constexpr int kLd = W + 16;
template <typename T, int W> constexpr int kTileBytes = kTokens<T> * kLd<W> * (int)sizeof(T);

// a lane's place in row fragments and in column pieces
template <typename T, int W> struct Lane {
  int row, col;
  __device__ __forceinline__ explicit Lane(int lane) {
    const int g = lane >> 4, i = lane & 15;
    row = i * kLd<W> + ((g ^ ((i >> 2) & 3)) << 2);
    if constexpr (sizeof(T) == 2) col = (4 * g + (i >> 2)) * kLd<W> + (((i & 3) ^ g) << 2);
    else col = 4 * g * kLd<W> + (((i >> 2) ^ g) << 2) + (i & 3);
  }
};

// Operand whose k runs along row r0 + i, from element k0.
template <int W>
__device__ __forceinline__ bf16x8 row_frag(const bf16_t* X, const Lane<bf16_t, W>& l, int r0, int k0) {
  const bf16_t* p = X + l.row + r0 * kLd<W> + k0;
  const bf16x4 lo = *(const bf16x4*)p, hi = *(const bf16x4*)(p + 16);
  return (bf16x8){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}
template <int W>
__device__ __forceinline__ f32x4 row_frag(const float* X, const Lane<float, W>& l, int r0, int k0) {
  return *(const f32x4*)(X + l.row + r0 * kLd<W> + k0);
}
// Operand whose k runs down column c0 + i, from row r0 (bf16: two transpose reads).
template <int W>
__device__ __forceinline__ bf16x8 col_frag(const bf16_t* X, const Lane<bf16_t, W>& l, int r0, int c0) {
  const bf16_t* p = X + l.col + r0 * kLd<W> + c0;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * kLd<W>));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int W>
__device__ __forceinline__ f32x4 col_frag(const float* X, const Lane<float, W>& l, int r0, int c0) {
  f32x4 x;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = X[l.col + (r0 + e) * kLd<W> + c0];
  return x;
}

// ---- operands rounded from fp32 ---------------------------------------------------
// bf16 operands that are not inputs are sums of pieces of 8 bits each: two
// (2^-17 of the value) where they only go into bf16 results, which rounds
// those a hundred times more coarsely; three (2^-25) for the state, which is
// handed out in fp32.  One piece for the products with P and S would double
// the outputs' mean square error.
template <typename T> struct Pieces;
template <> struct Pieces<float> {
  static constexpr int OUT = 1, STATE = 1;
  template <int N>
  __device__ static __forceinline__ void cut(const f32x4 (&x)[1], f32x4 (&f)[N]) {
    f[0] = x[0];
  }
};
__device__ __forceinline__ bf16x8 round8(const f32x4& a, const f32x4& b) { return frag_from_acc(a, b); }
__device__ __forceinline__ f32x4 low4(const bf16x8& f, int half) {
  const uint4 w = __builtin_bit_cast(uint4, f);
  const uint32_t a = half ? w.z : w.x, b = half ? w.w : w.y;
  return (f32x4){__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u), __uint_as_float(b << 16),
                 __uint_as_float(b & 0xffff0000u)};
}
template <> struct Pieces<bf16_t> {
  static constexpr int OUT = 2, STATE = 3;
  template <int N>
  __device__ static __forceinline__ void cut(const f32x4 (&x)[2], bf16x8 (&f)[N]) {
    f32x4 a = x[0], b = x[1];
#pragma unroll
    for (int p = 0; p < N; ++p) {
      f[p] = round8(a, b);
      a -= low4(f[p], 0);
      b -= low4(f[p], 1);
    }
  }
};
// accumulator tiles that make one operand
template <typename T> constexpr int kAccs = sizeof(T) == 2 ? 2 : 1;

// an input operand as fp32, element by element
__device__ __forceinline__ void widen(const bf16x8& f, f32x4 (&x)[2]) {
  x[0] = low4(f, 0);
  x[1] = low4(f, 1);
}
__device__ __forceinline__ void widen(const f32x4& f, f32x4 (&x)[1]) { x[0] = f; }

// ---- rows of an input -----------------------------------------------------------
// One head of an input: its first element, the distance between tokens, its channels.
struct View {
  const void* p;
  int64_t ld;
  int d;
};

// C tokens of W channels on the way from memory to LDS: 16 bytes a lane,
// rows and channels that are not there read some that are, and become zeros
// on the way to LDS.
template <typename T, int W> struct Stage {
  static constexpr int VE = 16 / (int)sizeof(T), VPR = W / VE, RPP = kThreads / VPR, N = kTokens<T> / RPP;
  typedef typename Pack<T, VE>::type vec;
  vec v[N];
  __device__ __forceinline__ void load(const View& x, int tok, int n) {
    const int c = (int)(threadIdx.x % VPR) * VE, r = (int)(threadIdx.x / VPR);
    const T* p = (const T*)x.p;
    if (x.d % VE == 0) {
      p += c < x.d ? c : 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = r + i * RPP;
        v[i] = *(const vec*)(p + (int64_t)(tok + (row < n ? row : n - 1)) * x.ld);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = r + i * RPP;
        const T* at = p + (int64_t)(tok + (row < n ? row : n - 1)) * x.ld;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const T y = at[c + e < x.d ? c + e : 0];
          v[i][e] = c + e < x.d ? y : (T)0;
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* X, int d, int n) const {
    const int c = (int)(threadIdx.x % VPR) * VE, r = (int)(threadIdx.x / VPR);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = r + i * RPP, s = (row >> 2) & 3;
      const bool there = c < d && row < n;
      uint4 w = __builtin_bit_cast(uint4, v[i]);
      w = there ? w : make_uint4(0, 0, 0, 0);
      if constexpr (sizeof(T) == 2) {
        // two units, the swizzle's low bit swaps them
        const bool swap = s & 1;
        const uint4 y = swap ? make_uint4(w.z, w.w, w.x, w.y) : w;
        *(uint4*)(X + row * kLd<W> + (((c >> 2) ^ (s & 2)) << 2)) = y;
      } else {
        *(uint4*)(X + row * kLd<W> + (((c >> 2) ^ s) << 2)) = w;
      }
    }
  }
  // whether some row that is there holds an infinity or a NaN
  __device__ __forceinline__ bool wild(int d, int n) const {
    const int c = (int)(threadIdx.x % VPR) * VE, r = (int)(threadIdx.x / VPR);
    bool found = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      bool any = false;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        if constexpr (sizeof(T) == 2) any |= (v[i][e] & 0x7f80) == 0x7f80;
        else any |= (__float_as_uint(v[i][e]) & 0x7f800000u) == 0x7f800000u;
      }
      found |= any && c < d && r + i * RPP < n;
    }
    return found;
  }
};

// four channels from c on of one token, zeros past the last
template <typename T>
__device__ __forceinline__ f32x4 load4(const View& x, int64_t tok, int c) {
  const T* p = (const T*)x.p + tok * x.ld;
  float v[4];
  if (x.d % 4 == 0) {
    load_vec<T, 4>(p + (c < x.d ? c : 0), v);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = c < x.d ? v[e] : 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float y = Elem<T>::to_f32(p[c + e < x.d ? c + e : 0]);
      v[e] = c + e < x.d ? y : 0.f;
    }
  }
  return (f32x4){v[0], v[1], v[2], v[3]};
}
template <typename T>
__device__ __forceinline__ void store4(T* p, int c, int d, const f32x4& x) {
  if (d % 4 == 0) {
    const float v[4] = {x[0], x[1], x[2], x[3]};
    if (c < d) store_vec<T, 4>(p + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < d) p[c + e] = Elem<T>::from_f32(x[e]);
  }
}

// ---- decays ------------------------------------------------------------------------
// Inclusive sums over the wave's lanes, in 64 bits.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp64(double v) {
  const uint64_t w = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)w, CTRL, ROWS, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(w >> 32), CTRL, ROWS, 0xf, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sums(double v) {
  v += dpp64<0x111, 0xf>(v);
  v += dpp64<0x112, 0xf>(v);
  v += dpp64<0x114, 0xf>(v);
  v += dpp64<0x118, 0xf>(v);
  v += dpp64<0x142, 0xa>(v);  // lane 15 of the row before
  v += dpp64<0x143, 0xc>(v);  // lane 31
  return v;
}
// 2^x of a difference of sums of log decays: 0 below what fp32 holds
__device__ __forceinline__ float decay_of(double x) { return exp2_fast((float)x); }

// A token's log decay in units of a factor 2.  Values above 0 count as 0, and
// those below -10000 (infinities) as that, whose factor is 0 in fp32 and in
// 64 bits: differences of their sums stay finite.  A NaN stays.
__device__ __forceinline__ double log2_decay(float g) {
  g = g > 0.f ? 0.f : g;
  g = g < -1e4f ? -1e4f : g;
  return (double)g * 1.4426950408889634;
}

template <typename T>
__device__ __forceinline__ float raw_decay(const LinearArgs& a, int h, int tok, int n, int lane) {
  if (a.g) return Elem<T>::to_f32(((const T*)a.g)[(int64_t)(tok + (lane < n ? lane : n - 1)) * a.ld_g + h]);
  return a.decay ? a.decay[h] : 0.f;
}

// Decays of a chunk's tokens in LDS.
template <typename T> struct Decays {
  double sum[kTokens<T>];               // running sums
  float row[kTokens<T>], col[kTokens<T>];  // factors of the state's part of an output, and of a token's part in the state
  float whole;
  int wild;
  __device__ __forceinline__ void fill(float g, int n, bool back, float row_scale, float col_scale, int lane) {
    const double s = wave_sums(lane < n ? log2_decay(g) : 0.0);
    const uint64_t w = __builtin_bit_cast(uint64_t, s);
    const double all = __builtin_bit_cast(
        double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(w >> 32), 63) << 32 |
                    (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)w, 63));
    const float since = decay_of(s), until = decay_of(all - s);
    if (lane < kTokens<T>) {
      sum[lane] = s;
      row[lane] = (back ? until : since) * row_scale;
      col[lane] = (back ? since : until) * col_scale;
    }
    if (lane == 0) whole = decay_of(all);
  }
};

// ---- states in registers ----------------------------------------------------------
// State tiles: rows the channels that a product sums over (16 m + 4 g + r in
// lane 16 g + i), columns a wave's own (c0 + 16 nt + i).  In memory states are
// [d_k][d_v]; TR: rows are d_v.
template <int M, int NT>
struct State {
  f32x4 s[M][NT];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) s[m][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
  }
  // element (row, col), f(pointer offset, its four values)
  template <bool TR>
  __device__ __forceinline__ void load(const float* p, int rows, int cols, int c0, int lane) {
    if (!p) return zero();
    const int g = lane >> 4, i = lane & 15;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int col = c0 + 16 * t + i;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * m + 4 * g + r;
          const bool there = row < rows && col < cols;
          const float x = p[there ? TR ? col * rows + row : row * cols + col : 0];
          s[m][t][r] = there ? x : 0.f;
        }
      }
  }
  template <bool TR>
  __device__ __forceinline__ void store(float* p, int rows, int cols, int c0, int lane) const {
    const int g = lane >> 4, i = lane & 15;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int col = c0 + 16 * t + i;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * m + 4 * g + r;
          if (row < rows && col < cols) p[TR ? col * rows + row : row * cols + col] = s[m][t][r];
        }
      }
  }
  // this lane's part of the inner product with a state in memory
  template <bool TR>
  __device__ __forceinline__ float dot(const float* p, int rows, int cols, int c0, int lane) const {
    const int g = lane >> 4, i = lane & 15;
    float sum = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int col = c0 + 16 * t + i;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * m + 4 * g + r;
          const bool there = row < rows && col < cols;
          const float x = p[there ? TR ? col * rows + row : row * cols + col : 0];
          sum += there ? s[m][t][r] * x : 0.f;
        }
      }
    return sum;
  }
};

// ---- a chunk's step of the state ------------------------------------------------------
// S <- whole S + K^T (col V): V's fragments are this wave's own columns,
// scaled and cut to pieces; K's are read from LDS as they are.
template <typename T, int DK, int NT, int PIECES>
__device__ __forceinline__ void step_state(const T* K, const Lane<T, DK>& lk, const typename Frag<T>::type (&vf)[2][NT],
                                           const Decays<T>& d, int lane, State<DK / 16, NT>& st) {
  constexpr int KB = Elem<T>::KB;
  const int g = lane >> 4;
  typename Frag<T>::type f[2][NT][PIECES];
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    f32x4 by[kAccs<T>];
#pragma unroll
    for (int h = 0; h < kAccs<T>; ++h) by[h] = *(const f32x4*)(d.col + KB * kb + 16 * h + 4 * g);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 x[kAccs<T>];
      widen(vf[kb][t], x);
#pragma unroll
      for (int h = 0; h < kAccs<T>; ++h) x[h] *= by[h];
      Pieces<T>::template cut<PIECES>(x, f[kb][t]);
    }
  }
  const float whole = d.whole;
#pragma unroll
  for (int m = 0; m < DK / 16; ++m) {
#pragma unroll
    for (int t = 0; t < NT; ++t) st.s[m][t] *= whole;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const auto kf = col_frag<DK>(K, lk, KB * kb, 16 * m);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int p = PIECES - 1; p >= 0; --p) st.s[m][t] = mma(kf, f[kb][t][p], st.s[m][t]);
    }
  }
}

template <typename T, int DV, int NT>
__device__ __forceinline__ void own_columns(const T* V, const Lane<T, DV>& lv, int c0,
                                            typename Frag<T>::type (&vf)[2][NT]) {
#pragma unroll
  for (int kb = 0; kb < 2; ++kb)
#pragma unroll
    for (int t = 0; t < NT; ++t) vf[kb][t] = col_frag<DV>(V, lv, Elem<T>::KB * kb, c0 + 16 * t);
}

// Slots, and what of a sequence passes through one.
enum Kind { kNothing = 0, kStarted = 1, kPassed = 2, kEntered = 4 };
struct Slot {
  int slot, lo, hi;
  bool last;
  __device__ __forceinline__ Slot(const LinearArgs& a, int s) : slot(s) {
    lo = (int)(s * a.slot);
    const int64_t end = (s + 1) * a.slot;
    hi = (int)(end < a.tokens ? end : a.tokens);
    last = s == a.n_slots - 1;
  }
};

// ---- states of the slots ---------------------------------------------------------------
// What a slot hands on: forward the state at its end, of the sequence that
// goes on past it, from zero where that sequence entered; backward
// (blockIdx.y = 1) the gradient of the state at its start, of the sequence
// that entered.  rows of K, columns of V: k and v, backward q and dout.
template <typename T, int DK, int NT, bool BACK>
__device__ __forceinline__ void states_range(const LinearArgs& a, const View& k, const View& v, int h, int t0, int end,
                                             char* smem, State<DK / 16, NT>& st, double* total) {
  constexpr int C = kTokens<T>, DV = 64 * NT;
  T* K = (T*)smem;
  T* V = (T*)(smem + kTileBytes<T, DK>);
  Decays<T>* d = (Decays<T>*)(smem + kTileBytes<T, DK> + kTileBytes<T, DV>);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c0 = wave * 16 * NT;
  const Lane<T, DK> lk(lane);
  const Lane<T, DV> lv(lane);
  const int chunks = (end - t0 + C - 1) / C;
  Stage<T, DK> sk;
  Stage<T, DV> sv;
  float g = 0.f;
  auto load = [&](int i) {
    const int t = t0 + (BACK ? chunks - 1 - i : i) * C, n = end - t < C ? end - t : C;
    sk.load(k, t, n);
    sv.load(v, t, n);
    g = raw_decay<T>(a, h, t, n, lane);
  };
  load(0);
  for (int i = 0; i < chunks; ++i) {
    const int t = t0 + (BACK ? chunks - 1 - i : i) * C, n = end - t < C ? end - t : C;
    sk.store(K, k.d, n);
    sv.store(V, v.d, n);
    if (wave == 0) d->fill(g, n, BACK, 1.f, BACK ? a.scale : 1.f, lane);
    lds_barrier();
    if (i + 1 < chunks) load(i + 1);
    if (total) *total += d->sum[C - 1];
    typename Frag<T>::type vf[2][NT];
    own_columns<T, DV, NT>(V, lv, c0, vf);
    step_state<T, DK, NT, Pieces<T>::STATE>(K, lk, vf, *d, lane, st);
    lds_barrier();
  }
}

template <typename T, int DK, int NT>
constexpr int kStatesLds = kTileBytes<T, DK> + kTileBytes<T, 64 * NT> + (int)sizeof(Decays<T>);

template <typename T, int DK, int NT>
__global__ void __launch_bounds__(kThreads, 2)
linear_states(const LinearArgs a, const T* __restrict__ dout, const float* __restrict__ dht, float* __restrict__ ends,
              float* __restrict__ adj, double* __restrict__ sums, int* __restrict__ kinds) {
  __shared__ __align__(16) char smem[kStatesLds<T, DK, NT>];
  const int h = (int)(blockIdx.x % (unsigned)a.H), hq = h / (a.H / a.Hq);
  const Slot w(a, (int)(blockIdx.x / (unsigned)a.H));
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  const int lane = threadIdx.x & 63, c0 = uniform(threadIdx.x >> 6) * 16 * NT;
  const int64_t floats = (int64_t)a.dk * a.dv, at = ((int64_t)w.slot * a.H + h) * floats;
  State<DK / 16, NT> st;
  const int first = uniform(seqs.from(w.lo)), before = first > 0 ? uniform((int)seqs.end(first - 1)) : w.lo;
  const bool entered = before > w.lo;
  double total = 0.0;
  if (blockIdx.y == 0) {
    const int n = uniform(seqs.from(w.hi)) - 1;  // the last sequence that starts in the slot or before
    const bool on = !w.last && n >= 0 && uniform((int)seqs.end(n)) > w.hi;
    const int start = on ? uniform((int)seqs.start(n)) : 0;
    const bool own = start >= w.lo;
    if (h == 0 && threadIdx.x == 0)
      kinds[w.slot] = (!on ? kNothing : own ? kStarted : kPassed) | (entered ? kEntered : 0);
    if (!on) return;
    st.template load<false>(own && a.h0 ? a.h0 + ((int64_t)n * a.H + h) * floats : nullptr, a.dk, a.dv, c0, lane);
    const View k{(const T*)a.k + hq * a.dk, a.ld_k, a.dk}, v{(const T*)a.v + h * a.dv, a.ld_v, a.dv};
    states_range<T, DK, NT, false>(a, k, v, h, own ? start : w.lo, w.hi, smem, st, &total);
    st.template store<false>(ends + at, a.dk, a.dv, c0, lane);
    if (!own && threadIdx.x == 0) sums[(int64_t)w.slot * a.H + h] = total;
  } else {
    if (!entered) return;
    const bool ends_here = before <= w.hi;
    st.template load<false>(ends_here && dht ? dht + ((int64_t)(first - 1) * a.H + h) * floats : nullptr, a.dk, a.dv, c0,
                            lane);
    const View q{(const T*)a.q + hq * a.dk, a.ld_q, a.dk}, d{dout + h * a.dv, (int64_t)a.H * a.dv, a.dv};
    states_range<T, DK, NT, true>(a, q, d, h, w.lo, ends_here ? before : w.hi, smem, st, nullptr);
    st.template store<false>(adj + at, a.dk, a.dv, c0, lane);
  }
}

// True states at the slots' ends out of what each slot made of a zero state,
// in place: S_i <- S_i + decay_i S_{i-1} where a sequence passes through slot
// i; likewise (blockIdx.y = 1) the gradients from the last slot to the first.
// A lane takes one element; loads go ahead of the chain in batches.
__global__ void __launch_bounds__(256)
linear_chain(int H, int64_t floats, int n_slots, float* __restrict__ ends, float* __restrict__ adj,
             const double* __restrict__ sums, const int* __restrict__ kinds) {
  constexpr int BATCH = 8;
  const bool back = blockIdx.y != 0;
  const int64_t per = (floats + 255) / 256;
  const int h = (int)(blockIdx.x / per);
  int64_t el = (blockIdx.x % per) * 256 + threadIdx.x;
  if (el >= floats) return;
  float* __restrict__ v = (back ? adj : ends) + h * floats + el;
  const int64_t step = (int64_t)H * floats;
  float s = 0.f;
  for (int i0 = 0; i0 < n_slots; i0 += BATCH) {
    float made[BATCH], by[BATCH];
    int kd[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const int i = i0 + j < n_slots ? i0 + j : n_slots - 1, slot = back ? n_slots - 1 - i : i;
      kd[j] = kinds[slot];
      made[j] = v[slot * step];
      by[j] = decay_of(sums[(int64_t)slot * H + h]);
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      if (i0 + j >= n_slots) break;
      const int slot = back ? n_slots - 1 - i0 - j : i0 + j;
      const bool holds = back ? kd[j] & kEntered : kd[j] & (kStarted | kPassed);
      s = (kd[j] & kPassed ? by[j] * s : 0.f) + (holds ? made[j] : 0.f);
      if (kd[j] & kPassed) v[slot * step] = s;
    }
  }
}

// ---- outputs -------------------------------------------------------------------------------
// One form for the outputs and the three gradients ("sweep"): rows of Q meet
// rows of K, whose weights sum rows of V.
enum Role { kForward, kDq, kDk, kDv };

struct Sweep {
  View q, k, v;
  View other;       // the rows that an output's state part is multiplied with for the decays' gradients
  void* out;        // [tokens, H, v.d], this head's first element; fp32 with `wide`
  bool wide;
  float p_scale, row_scale, col_scale;
  float* dots;      // [H, tokens], this head's row (null: none)
};

template <typename T, int DK, int NT>
struct SweepLds {
  T q[kTokens<T> * kLd<DK>], k[kTokens<T> * kLd<DK>], v[kTokens<T> * kLd<64 * NT>];
  T p[Pieces<T>::OUT][kTokens<T> * kLd<kTokens<T>>];
  Decays<T> d;
  float dot[kWaves][kTokens<T>];
  float sums[10][2][16];  // row and column sums of M's tiles
};

// the tiles on and beside the diagonal, in the order that waves take them
__device__ __forceinline__ void tile_of(int t, int* a, int* b) {
  *a = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
  *b = t - *a * (*a + 1) / 2;
}

// Tokens [t0, end) of one sequence; the state before them (BACK: the gradient
// of the state after them) in, that after (before) them out.
template <typename T, int DK, int NT, Role R>
__device__ __forceinline__ void sweep_range(const LinearArgs& a, const Sweep& w, int h, int t0, int end, bool keep,
                                            SweepLds<T, DK, NT>& m, State<DK / 16, NT>& st) {
  constexpr bool BACK = R == kDk || R == kDv, M_SUMS = R == kDq;
  constexpr int C = kTokens<T>, DV = 64 * NT, KB = Elem<T>::KB, RT = C / 16, TILES = RT * (RT + 1) / 2;
  constexpr int OUT = Pieces<T>::OUT;
  typedef typename Frag<T>::type frag;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c0 = wave * 16 * NT;
  const int g = lane >> 4, i16 = lane & 15;
  const Lane<T, DK> lk(lane);
  const Lane<T, DV> lv(lane);
  const Lane<T, C> lp(lane);
  const int chunks = (end - t0 + C - 1) / C;
  Stage<T, DK> sq, sk;
  Stage<T, DV> sv;
  float gd = 0.f;
  auto load = [&](int t, int n) {
    sq.load(w.q, t, n);
    sk.load(w.k, t, n);
    sv.load(w.v, t, n);
    gd = raw_decay<T>(a, h, t, n, lane);
  };
  // chunk i is [t, t + n); one that holds an infinity or a NaN among V is
  // walked token by token (one < n), so that a weight of zero never meets it
  int i = 0, one = 0;
  auto start_of = [&](int c) { return t0 + (BACK ? chunks - 1 - c : c) * C; };
  auto size_of = [&](int t) { return end - t < C ? end - t : C; };
  int t = start_of(0), n = size_of(t), whole_n = n;
  bool single = false;
  load(t, n);
  while (true) {
    sq.store(m.q, w.q.d, n);
    sk.store(m.k, w.k.d, n);
    sv.store(m.v, w.v.d, n);
    if (wave == 0) m.d.fill(gd, n, BACK, w.row_scale, w.col_scale, lane);
    if (!single && n > 1 && __ballot(sv.wild(w.v.d, n)) != 0 && lane == 0) m.d.wild = 1;
    lds_barrier();
    if (!single && uniform(m.d.wild)) {
      lds_barrier();  // all have read it
      if (threadIdx.x == 0) m.d.wild = 0;
      single = true;
      one = 0;
      whole_n = n;
      n = 1;
      t = start_of(i) + (BACK ? whole_n - 1 : 0);
      load(t, n);
      lds_barrier();
      continue;
    }
    // what comes next
    int t_next = -1, n_next = 0;
    if (single && one + 1 < whole_n) {
      t_next = BACK ? t - 1 : t + 1;
      n_next = 1;
    } else if (i + 1 < chunks) {
      t_next = start_of(i + 1);
      n_next = size_of(t_next);
    }
    if (t_next >= 0) load(t_next, n_next);

    // P, shared out by tiles
#pragma unroll
    for (int u = 0; u < (TILES + kWaves - 1) / kWaves; ++u) {
      const int tile = wave + u * kWaves;
      if (tile >= TILES) break;
      int ra, rb;
      tile_of(tile, &ra, &rb);
      const int rt = BACK ? rb : ra, ct = BACK ? ra : rb;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < DK / KB; ++kb)
        acc = mma(row_frag<DK>(m.k, lk, 16 * ct, KB * kb), row_frag<DK>(m.q, lk, 16 * rt, KB * kb), acc);
      const double gi = m.d.sum[16 * rt + i16];
      f32x4 p;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const double gj = m.d.sum[16 * ct + 4 * g + r];
        const int di = 16 * (rt - ct) + i16 - 4 * g - r;  // row minus column
        const bool on = BACK ? di <= 0 : di >= 0;
        p[r] = on ? acc[r] * decay_of(BACK ? gj - gi : gi - gj) * w.p_scale : 0.f;
      }
      if (M_SUMS && w.dots) {
        // M = (Q K^T) o P, this role's V being the keys
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < DV / KB; ++kb) {
          const int row = 16 * rt + i16;
          const int64_t tok = t + (row < n ? row : n - 1);
          frag qf;
          if constexpr (sizeof(T) == 2)
            qf = round8(load4<T>(w.other, tok, KB * kb + 4 * g), load4<T>(w.other, tok, KB * kb + 16 + 4 * g));
          else
            qf = load4<T>(w.other, tok, KB * kb + 4 * g);
          s = mma(row_frag<DV>(m.v, lv, 16 * ct, KB * kb), qf, s);
        }
        float across = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int di = 16 * (rt - ct) + i16 - 4 * g - r;
          s[r] = di > 0 ? s[r] * p[r] : 0.f;
          across += s[r];
          s[r] = row_sum(s[r]);
        }
        across += __shfl_xor(across, 16, 64);
        across += __shfl_xor(across, 32, 64);
        if (g == 0) m.sums[tile][0][i16] = across;
        if (i16 == 0) *(f32x4*)&m.sums[tile][1][4 * g] = s;
      }
      f32x4 x = p;
#pragma unroll
      for (int c = 0; c < OUT; ++c) {
        T* at = m.p[c] + lp.row + 16 * rt * kLd<C> + 16 * ct;
        if constexpr (sizeof(T) == 2) {
          const uint2 b = make_uint2(__builtin_bit_cast(uint32_t, f32x2_to_bf16x2(x[0], x[1])),
                                     __builtin_bit_cast(uint32_t, f32x2_to_bf16x2(x[2], x[3])));
          *(uint2*)at = b;
          x -= (f32x4){__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u), __uint_as_float(b.y << 16),
                       __uint_as_float(b.y & 0xffff0000u)};
        } else {
          *(f32x4*)at = x;
        }
      }
    }
    lds_barrier();

    // the state's part of the outputs, transposed: rows are channels of V, columns tokens
    f32x4 acc[RT][NT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int x = 0; x < NT; ++x) acc[rt][x] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < DK / KB; ++kb) {
      frag sf[NT][OUT];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        f32x4 s[kAccs<T>];
#pragma unroll
        for (int e = 0; e < kAccs<T>; ++e) s[e] = st.s[kAccs<T> * kb + e][x];
        Pieces<T>::template cut<OUT>(s, sf[x]);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const frag qf = row_frag<DK>(m.q, lk, 16 * rt, KB * kb);
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int c = OUT - 1; c >= 0; --c) acc[rt][x] = mma(sf[x][c], qf, acc[rt][x]);
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float by = m.d.row[16 * rt + i16];
#pragma unroll
      for (int x = 0; x < NT; ++x) acc[rt][x] *= by;
    }
    if ((R == kDq || R == kDk) && w.dots) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int row = 16 * rt + i16;
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          const f32x4 y = load4<T>(w.other, t + (row < n ? row : n - 1), c0 + 16 * x + 4 * g);
#pragma unroll
          for (int r = 0; r < 4; ++r) s += acc[rt][x][r] * y[r];
        }
        s += __shfl_xor(s, 16, 64);
        s += __shfl_xor(s, 32, 64);
        if (g == 0) m.dot[wave][row] = s;
      }
    }
    // the chunk's own part
    frag vf[2][NT];
    own_columns<T, DV, NT>(m.v, lv, c0, vf);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if (BACK ? KB * (kb + 1) <= 16 * rt : KB * kb > 16 * rt) continue;
#pragma unroll
        for (int c = OUT - 1; c >= 0; --c) {
          const frag pf = row_frag<C>(m.p[c], lp, 16 * rt, KB * kb);
#pragma unroll
          for (int x = 0; x < NT; ++x) acc[rt][x] = mma(vf[kb][x], pf, acc[rt][x]);
        }
      }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = 16 * rt + i16;
      if (row < n) {
        const int64_t at = (int64_t)(t + row) * a.H * w.v.d;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          if (w.wide) store4<float>((float*)w.out + at, c0 + 16 * x + 4 * g, w.v.d, acc[rt][x]);
          else store4<T>((T*)w.out + at, c0 + 16 * x + 4 * g, w.v.d, acc[rt][x]);
        }
      }
    }
    if (keep) step_state<T, DK, NT, Pieces<T>::STATE>(m.k, lk, vf, m.d, lane, st);
    else step_state<T, DK, NT, OUT>(m.k, lk, vf, m.d, lane, st);
    lds_barrier();
    if ((R == kDq || R == kDk) && w.dots && (int)threadIdx.x < n) {
      const int row = threadIdx.x;
      float s = m.dot[0][row] + m.dot[1][row] + m.dot[2][row] + m.dot[3][row];
      if (M_SUMS) {
        const int mt = row / 16;
        for (int b = 0; b <= mt; ++b) s += m.sums[mt * (mt + 1) / 2 + b][0][row % 16];
        for (int b = mt; b < RT; ++b) s -= m.sums[b * (b + 1) / 2 + mt][1][row % 16];
      }
      w.dots[t + row] = s;
    }
    if (t_next < 0) break;
    if (single && one + 1 < whole_n) {
      ++one;
    } else {
      single = false;
      ++i;
    }
    t = t_next;
    n = n_next;
  }
  if (w.dots) lds_barrier();  // dot and sums are read
}

// One slot of one head.  dS: what a sequence's last state's inner product with its gradient is wanted of.
template <typename T, int DK, int NT, Role R>
__device__ __forceinline__ void sweep_slot(const LinearArgs& a, const Sweep& w, int h, const Slot& s, const float* enter,
                                           const float* seq_state, float* leave, const float* dht, const float* adj,
                                           float* seq_dot, float* slot_dot, SweepLds<T, DK, NT>& m) {
  constexpr bool BACK = R == kDk || R == kDv, TR = R == kDq || R == kDk;
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  const int lane = threadIdx.x & 63, c0 = uniform(threadIdx.x >> 6) * 16 * NT;
  const int64_t floats = (int64_t)a.dk * a.dv;
  const int rows = w.q.d, cols = w.v.d;
  State<DK / 16, NT> st;
  // all of P beside the tiles that are written stays zero
  for (int x = threadIdx.x; x < (int)(sizeof(m.p) / 16); x += kThreads) ((uint4*)m.p)[x] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) m.d.wild = 0;
  lds_barrier();
  auto of_slot = [&](int i) { return enter + ((int64_t)i * a.H + h) * floats; };
  auto of_seq = [&](const float* p, int n) { return p ? p + ((int64_t)n * a.H + h) * floats : nullptr; };
  // <S, dS> at the end of a range
  auto inner = [&](const float* p, float* out) {
    float x = p ? st.template dot<TR>(p, rows, cols, c0, lane) : 0.f;
    x = row_sum(x);
    x += __shfl_xor(x, 16, 64);
    x += __shfl_xor(x, 32, 64);
    if (lane == 0) m.dot[threadIdx.x >> 6][0] = x;
    lds_barrier();
    if (threadIdx.x == 0) *out = m.dot[0][0] + m.dot[1][0] + m.dot[2][0] + m.dot[3][0];
    lds_barrier();
  };
  auto piece = [&](int n, int start, int end, bool entered) {
    const bool done = end <= s.hi;
    const int stop = done ? end : s.hi;
    if (BACK) st.template load<TR>(done ? of_seq(seq_state, n) : of_slot(s.slot + 1), rows, cols, c0, lane);
    else st.template load<TR>(entered ? of_slot(s.slot - 1) : of_seq(seq_state, n), rows, cols, c0, lane);
    const bool out = leave && (BACK ? !entered : done);
    if (start < stop) sweep_range<T, DK, NT, R>(a, w, h, start, stop, out, m, st);
    if (R == kDq && w.dots) {
      if (done) inner(of_seq(dht, n), seq_dot + (int64_t)n * a.H + h);
      else inner(adj + ((int64_t)(s.slot + 1) * a.H + h) * floats, slot_dot + (int64_t)s.slot * a.H + h);
    }
    if (out) st.template store<TR>(leave + ((int64_t)n * a.H + h) * floats, rows, cols, c0, lane);
  };
  int n = uniform(seqs.from(s.lo)), at = s.lo;
  if (n > 0) {
    const int end = uniform((int)seqs.end(n - 1));
    if (end > s.lo) {
      at = end;
      piece(n - 1, s.lo, end, true);
    }
  }
  // those that start here; the last slot also has the empty ones behind the last token
  for (; n < a.n_seqs; ++n) {
    const Span range = seqs.next(n, &at);
    const int start = uniform(range.start), end = uniform(range.end);
    if (!s.last && start >= s.hi) break;
    piece(n, start, end, false);
  }
}

template <typename T, int DK, int NT>
__global__ void __launch_bounds__(kThreads, 2)
linear_forward(const LinearArgs a, const float* __restrict__ ends, T* __restrict__ o, float* __restrict__ ht) {
  __shared__ __align__(16) SweepLds<T, DK, NT> m;
  const int h = (int)(blockIdx.x % (unsigned)a.H), hq = h / (a.H / a.Hq);
  const Slot s(a, (int)(blockIdx.x / (unsigned)a.H));
  Sweep w{};
  w.q = View{(const T*)a.q + hq * a.dk, a.ld_q, a.dk};
  w.k = View{(const T*)a.k + hq * a.dk, a.ld_k, a.dk};
  w.v = View{(const T*)a.v + h * a.dv, a.ld_v, a.dv};
  w.out = o + h * a.dv;
  w.p_scale = w.row_scale = a.scale;
  w.col_scale = 1.f;
  sweep_slot<T, DK, NT, kForward>(a, w, h, s, ends, a.h0, ht, nullptr, nullptr, nullptr, nullptr, m);
}

// Where the backward pass's launches leave what others read.
struct LinearWork {
  const float *ends, *adj;
  float *dot_q, *dot_k, *slot_dot, *seq_dot, *dq, *dk;
};

// The three gradients, a third of the workgroups each.
template <typename T, int DK, int DV, Role R>
__device__ __forceinline__ void gradient(const LinearArgs& a, const LinearGrads& g, const LinearWork& x, int h,
                                         const Slot& s, void* smem) {
  const int hq = h / (a.H / a.Hq);
  const bool shared = a.H != a.Hq;
  const View q{(const T*)a.q + hq * a.dk, a.ld_q, a.dk}, k{(const T*)a.k + hq * a.dk, a.ld_k, a.dk},
      v{(const T*)a.v + h * a.dv, a.ld_v, a.dv}, d{(const T*)g.dout + h * a.dv, (int64_t)a.H * a.dv, a.dv};
  Sweep w{};
  const float* enter = R == kDq ? x.ends : x.adj;
  if (R == kDq) {
    w.q = d, w.k = v, w.v = k, w.other = q;
    w.p_scale = w.row_scale = a.scale;
    w.col_scale = 1.f;
    w.dots = g.dg ? x.dot_q + (int64_t)h * a.tokens : nullptr;
  } else {
    w.q = R == kDk ? v : k, w.k = R == kDk ? d : q, w.v = R == kDk ? q : d;
    w.other = k;
    w.p_scale = w.col_scale = a.scale;
    w.row_scale = 1.f;
    w.dots = R == kDk && g.dg ? x.dot_k + (int64_t)h * a.tokens : nullptr;
  }
  if (R == kDv) {
    w.out = (T*)g.dv + h * a.dv;
  } else {
    w.wide = shared;
    if (shared) w.out = (R == kDq ? x.dq : x.dk) + h * a.dk;
    else w.out = (T*)(R == kDq ? g.dq : g.dk) + h * a.dk;
  }
  sweep_slot<T, R == kDv ? DK : DV, (R == kDv ? DV : DK) / 64, R>(
      a, w, h, s, enter, R == kDq ? a.h0 : g.dht, R == kDv ? g.dh0 : nullptr, g.dht, x.adj, x.seq_dot, x.slot_dot,
      *(SweepLds<T, R == kDv ? DK : DV, (R == kDv ? DV : DK) / 64>*)smem);
}

template <typename T, int DK, int DV>
constexpr int kBackwardLds = sizeof(SweepLds<T, DK, DV / 64>) > sizeof(SweepLds<T, DV, DK / 64>)
                                 ? sizeof(SweepLds<T, DK, DV / 64>)
                                 : sizeof(SweepLds<T, DV, DK / 64>);

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kThreads, 2)
linear_backward(const LinearArgs a, const LinearGrads g, const LinearWork x) {
  __shared__ __align__(16) char smem[kBackwardLds<T, DK, DV>];
  const unsigned role = blockIdx.x % 3, id = blockIdx.x / 3;
  const int h = (int)(id % (unsigned)a.H);
  const Slot s(a, (int)(id / (unsigned)a.H));
  if (role == 0) gradient<T, DK, DV, kDq>(a, g, x, h, s, smem);
  else if (role == 1) gradient<T, DK, DV, kDk>(a, g, x, h, s, smem);
  else gradient<T, DK, DV, kDv>(a, g, x, h, s, smem);
}

// The decays' gradients: a wave takes one slot of one head, 64 tokens at a
// time from each sequence's end, as suffix sums in 64 bits.
template <typename T>
__global__ void __launch_bounds__(64)
linear_decay_grad(const LinearArgs a, const LinearWork x, T* __restrict__ dg) {
  const int h = (int)(blockIdx.x % (unsigned)a.H), lane = threadIdx.x;
  const Slot s(a, (int)(blockIdx.x / (unsigned)a.H));
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  const float* __restrict__ dq = x.dot_q + (int64_t)h * a.tokens;
  const float* __restrict__ dk = x.dot_k + (int64_t)h * a.tokens;
  auto piece = [&](int n, int start, int end) {
    const bool done = end <= s.hi;
    const int stop = done ? end : s.hi;
    if (start >= stop) return;
    double carry = done ? x.seq_dot[(int64_t)n * a.H + h] : x.slot_dot[(int64_t)s.slot * a.H + h];
    for (int e = stop; e > start; e -= 64) {
      const int t = e - 1 - lane;  // lane 0 is the last token
      const bool there = t >= start;
      const double v = wave_sums(there ? (double)dq[t] - (double)dk[t] : 0.0) + carry;
      if (there) {
        const float g = Elem<T>::to_f32(((const T*)a.g)[(int64_t)t * a.ld_g + h]);
        dg[(int64_t)t * a.H + h] = Elem<T>::from_f32(g > 0.f ? 0.f : (float)v);
      }
      carry = __shfl(v, 63, 64);
    }
  };
  int n = uniform(seqs.from(s.lo)), at = s.lo;
  if (n > 0) {
    const int end = uniform((int)seqs.end(n - 1));
    if (end > s.lo) {
      at = end;
      piece(n - 1, s.lo, end);
    }
  }
  for (; n < a.n_seqs; ++n) {
    const Span range = seqs.next(n, &at);
    const int start = uniform(range.start), end = uniform(range.end);
    if (start >= s.hi) break;
    piece(n, start, end);
  }
}

// Gradients of shared queries and keys: the sum over the heads that share.
// Tokens behind the last sequence have none.
template <typename T>
__global__ void __launch_bounds__(256)
linear_shared(const LinearArgs a, const float* __restrict__ pq, const float* __restrict__ pk, T* __restrict__ dq,
              T* __restrict__ dkk) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, row = at / a.dk, c = at - row * a.dk;
  if (row >= Seqs{a.cu, a.n_seqs, a.T, a.tokens}.end(a.n_seqs - 1) * a.Hq) return;
  const int dk = a.dk, share = a.H / a.Hq;
  const float* __restrict__ p = (blockIdx.y ? pk : pq) + row * share * dk + c;
  float s = 0.f;
  for (int u = 0; u < share; ++u) s += p[(int64_t)u * dk];
  (blockIdx.y ? dkk : dq)[at] = Elem<T>::from_f32(s);
}

// ---- one token ------------------------------------------------------------------------------
// The state is read once and written once.  A workgroup owns one (sequence,
// head); a thread 4 columns of every (threads / LC)-th row.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(DK * DV / 16)
linear_step(const LinearArgs a, float* __restrict__ state, T* __restrict__ o) {
  constexpr int NTH = DK * DV / 16, LC = DV / 4, RP = NTH / LC, NI = DK / RP, NW = NTH / 64;
  __shared__ float sk[DK], sq[DK];
  __shared__ f32x4 part[NW][LC];
  const int64_t nh = blockIdx.x;
  const int h = (int)(nh % a.H), hq = h / (a.H / a.Hq);
  const int64_t seq = nh / a.H;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, c = tid % LC * 4, r0 = tid / LC;
  float* __restrict__ S = state + nh * a.dk * a.dv;
  const bool quads = a.dv % 4 == 0;
  typedef float quad __attribute__((ext_vector_type(4), aligned(4)));
  f32x4 s[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int row = r0 + i * RP;
    const float* p = S + (row < a.dk ? row : 0) * a.dv;
    if (quads) {
      const quad x = *(const quad*)(p + (c < a.dv ? c : 0));
      s[i] = (f32x4){x[0], x[1], x[2], x[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = p[c + e < a.dv ? c + e : 0];
    }
  }
  for (int x = tid; x < DK; x += NTH) {
    sk[x] = x < a.dk ? load_f32((const T*)a.k + seq * a.ld_k + hq * a.dk + x) : 0.f;
    sq[x] = x < a.dk ? load_f32((const T*)a.q + seq * a.ld_q + hq * a.dk + x) * a.scale : 0.f;
  }
  const f32x4 v = load4<T>(View{(const T*)a.v + h * a.dv, a.ld_v, a.dv}, seq, c);
  float g = a.g ? load_f32((const T*)a.g + seq * a.ld_g + h) : a.decay ? a.decay[h] : 0.f;
  const float by = decay_of(log2_decay(g));
  __syncthreads();
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int row = r0 + i * RP;
    const bool there = row < a.dk;
    const float k = sk[row], q = sq[row];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[i][e] = s[i][e] * by + k * v[e];
      y[e] += there ? q * s[i][e] : 0.f;
    }
    if (!there) continue;
    float* p = S + row * a.dv;
    if (quads) {
      if (c < a.dv) *(quad*)(p + c) = (quad){s[i][0], s[i][1], s[i][2], s[i][3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.dv) p[c + e] = s[i][e];
    }
  }
#pragma unroll
  for (int off = LC; off < 64; off <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += __shfl_xor(y[e], off, 64);
  if (lane < LC) part[wave][lane] = y;
  __syncthreads();
  if (tid >= LC) return;
  y = part[0][tid];
#pragma unroll
  for (int w = 1; w < NW; ++w) y += part[w][tid];
  store4<T>(o + nh * a.dv, c, a.dv, y);
}

// ---- launches ---------------------------------------------------------------------------------
template <int DK_, int DV_> struct Dims {
  static constexpr int DK = DK_, DV = DV_;
};
template <typename F>
int dispatch(int is_bf16, const LinearArgs& a, F&& f) {
  auto dims = [&](auto t) {
    if (a.dk <= 64) return a.dv <= 64 ? f(t, Dims<64, 64>{}) : f(t, Dims<64, 128>{});
    return a.dv <= 64 ? f(t, Dims<128, 64>{}) : f(t, Dims<128, 128>{});
  };
  return is_bf16 ? dims(bf16_t{}) : dims(float{});
}

// the states that the slots hand on, and (backward) the gradients
template <typename T, int DK, int DV>
int states(const LinearArgs& a, const LinearPlan& p, const void* dout, const float* dht, char* ws, bool back,
           hipStream_t st) {
  float *ends = (float*)(ws + p.end_off), *adj = (float*)(ws + p.adj_off);
  double* sums = (double*)(ws + p.sum_off);
  int* kinds = (int*)(ws + p.kind_off);
  const unsigned sides = back ? 2 : 1;
  hipError_t e = launch_kernel(linear_states<T, DK, DV / 64>, dim3((unsigned)linear_groups(p, a.H), sides),
                               dim3(kThreads), st, a, (const T*)dout, dht, ends, adj, sums, kinds);
  if (e != hipSuccess) return (int)e;
  const int64_t floats = (int64_t)a.dk * a.dv;
  return (int)launch_kernel(linear_chain, dim3((unsigned)(a.H * ceil_div(floats, 256)), sides), dim3(256), st, a.H,
                            floats, (int)p.n_slots, ends, adj, sums, kinds);
}

}  // namespace

int launch_linear_forward(int is_bf16, const LinearArgs& a, const LinearPlan& p, void* o, float* ht, void* ws,
                          void* stream) {
  const hipStream_t st = (hipStream_t)stream;
  return dispatch(is_bf16, a, [&](auto t, auto dims) {
    typedef decltype(t) T;
    if (p.carry) {
      const int e = states<T, dims.DK, dims.DV>(a, p, nullptr, nullptr, (char*)ws, false, st);
      if (e != 0) return e;
    }
    return (int)launch_kernel(linear_forward<T, dims.DK, dims.DV / 64>, dim3((unsigned)linear_groups(p, a.H)),
                              dim3(kThreads), st, a, (const float*)((char*)ws + p.end_off), (T*)o, ht);
  });
}

int launch_linear_step(int is_bf16, const LinearArgs& a, float* state, void* o, void* stream) {
  return dispatch(is_bf16, a, [&](auto t, auto dims) {
    typedef decltype(t) T;
    return (int)launch_kernel(linear_step<T, dims.DK, dims.DV>, dim3((unsigned)(a.tokens * a.H)),
                              dim3(dims.DK * dims.DV / 16), (hipStream_t)stream, a, state, (T*)o);
  });
}

int launch_linear_backward(int is_bf16, const LinearArgs& a, const LinearPlan& p, const LinearGrads& g, void* ws,
                           void* stream) {
  const hipStream_t st = (hipStream_t)stream;
  return dispatch(is_bf16, a, [&](auto t, auto dims) {
    typedef decltype(t) T;
    char* w = (char*)ws;
    if (p.carry) {
      const int e = states<T, dims.DK, dims.DV>(a, p, g.dout, g.dht, w, true, st);
      if (e != 0) return e;
    }
    const LinearWork x{(float*)(w + p.end_off),    (float*)(w + p.adj_off),     (float*)(w + p.dot_q_off),
                       (float*)(w + p.dot_k_off),  (float*)(w + p.slot_dot_off), (float*)(w + p.seq_dot_off),
                       (float*)(w + p.dq_off),     (float*)(w + p.dk_off)};
    const unsigned groups = (unsigned)linear_groups(p, a.H);
    hipError_t e = launch_kernel(linear_backward<T, dims.DK, dims.DV>, dim3(3 * groups), dim3(kThreads), st, a, g, x);
    if (e != hipSuccess) return (int)e;
    if (a.H != a.Hq && a.tokens > 0) {
      const int64_t n = a.tokens * a.Hq * a.dk;
      e = launch_kernel(linear_shared<T>, dim3((unsigned)ceil_div(n, 256), 2), dim3(256), st, a,
                        (const float*)x.dq, (const float*)x.dk, (T*)g.dq, (T*)g.dk);
      if (e != hipSuccess) return (int)e;
    }
    if (!g.dg || a.tokens == 0) return 0;
    return (int)launch_kernel(linear_decay_grad<T>, dim3(groups), dim3(64), st, a, x, (T*)g.dg);
  });
}

}  // namespace kda
