// Linear attention with a decay for each head, for gfx950: whole sequences,
// one token, and gradients.
//
// Per sequence and head, with a_t = exp(min(g_t, 0)):
//   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// A chunk of C tokens, G the running sum of the log decays over it, S the
// state before it:
//   P = scale (Q K^T) o D,  D_ij = e^{G_i - G_j} for j <= i and 0 above,
//   O = P V + scale e^{G} Q S,   S <- e^{G_C} S + K^T (e^{G_C - G} V).
// No decay is above 1, so none overflows.  (Q K^T is a product that the
// recurrence does not form: it has to stay inside fp32.)  The running sums are
// kept in 64 bits: a decay between two tokens is the difference of two of them,
// which a strongly decaying token before both would take digits from in 32.
//
// The gradients are the same computation three times over.  dq is the forward
// form with (dout, v, k) for (q, k, v) and the transposed state; dv and dk are
// the form going back in time with (k, q, dout) and (v, dout, q):
//   dV = P^T dO + e^{G_C - G} K dS,   dS <- e^{G_C} dS + scale (e^G Q)^T dO,
// dS the gradient of the state after the chunk.  A decay stands in every
// product of a query at its token or later with a key before it.  With P below
// the diagonal only, x_s = q_s . (dq_s without its own token's key) and y_s =
// k_s . (dk_s without its own token's query), the products between tokens
// before t or tokens from t on stand in both, and
//   dg_t = sum_{s >= t} (x_s - y_s) + <S_end, dS>
// of the end of the sequence or slot.  A token's product with itself, which
// has no decay, would be the largest of either sum and is left out of both.
//
// A prompt goes in three launches, so that a few rows fill the device: the
// state that every slot of tokens hands on (linear_states), the true states
// from those (linear_chain), the outputs (linear_forward); the gradients in
// five at most.  Necessary bytes are few (a large copy would take 13.5 us for
// 4096 tokens of 16 heads of 128 in bf16, the matrix products 4.4): what
// bounds it is the length of a chunk's chain of phases, products of 16-row
// tiles with waits for LDS between them.  That case takes 52.5 us a call; its two
// rows of 2048 tokens backward 123 to 130; 16384 tokens of 32 heads of 128 keys
// and 64 values that share one query and key 149 to 155; 5003 tokens of 6 fp32
// heads 97.  In a kernel trace, whose calls are up to 17 percent longer, the
// launches take 16 + 8.7 + 33, 26 + 11.6 + 85 + 5.8, 50 + 9 + 122 and 21 + 12 + 66.
#include "kda_layer_device.h"
#include "kda_linear.h"
#include "kda_rows.h"

namespace kda {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// A workgroup has a wave for every 16 columns of the state (channels of V):
// waves of 32 columns read half of LDS for the same products, but a chunk's
// phases then wait longer (the prompt of 4096 tokens took 78 us against 66).
template <int DV> constexpr int kWaves = DV / 16;
template <int DV> constexpr int kThreads = 64 * kWaves<DV>;
// the waves of a SIMD that registers are left for
template <int DK, int DV> constexpr int kWavesOfSimd = linear_groups_of_unit(DK, DV) * kWaves<DV> / 4;

// Tokens of a chunk: both types then fill LDS alike, and two workgroups of
// the widest heads share a compute unit (80 KB each).
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
  typedef const __attribute__((address_space(3))) bf16_t lds_bf16;
  lds_bf16* p = (lds_bf16*)X + l.col + (r0 * kLd<W> + c0);
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

// x, formed anew (a move that the compiler takes for an exchange between
// lanes): what follows from it, addresses and masks, is computed where it is
// used and not kept in registers across the chunks.  Inline assembly would do
// the same, but the wait states behind matrix instructions are counted by
// what the compiler knows of the instructions between.
__device__ __forceinline__ int here(int x) { return __builtin_amdgcn_update_dpp(x, x, 0xe4, 0xf, 0xf, false); }

// Likewise: x is formed here, not where it is used next (an addition behind a
// product would move behind the chunk's barrier, its operands kept until then).
__device__ __forceinline__ f32x4 formed(f32x4 x) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = __uint_as_float((uint32_t)here((int)__float_as_uint(x[e])));
  return x;
}

// The sum of neighbouring groups of N lanes: of x in the even ones, of y in the odd ones.
template <int N>
__device__ __forceinline__ float swap_sum(float x, float y) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  if constexpr (N == 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
  } else {
    const auto p = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
}

// Nothing is moved across: operands' loads stay together ahead of their first use.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// ---- operands rounded from fp32 ---------------------------------------------------
// bf16 operands that are not inputs (weights, states, decayed values) are sums
// of three pieces of 8 bits each, which is all of an fp32 number.  Two pieces
// would leave ten times as many outputs off the rounding of their value (2e-3
// of them against 2e-4), and a sum that cancels without its last bits.
template <typename T> struct Pieces;
template <> struct Pieces<float> {
  static constexpr int COUNT = 1;
  __device__ static __forceinline__ f32x4 next(f32x4 (&x)[1]) { return x[0]; }
};
__device__ __forceinline__ bf16x8 round8(const f32x4& a, const f32x4& b) { return frag_from_acc(a, b); }
__device__ __forceinline__ f32x4 low4(const bf16x8& f, int half) {
  const uint4 w = __builtin_bit_cast(uint4, f);
  const uint32_t a = half ? w.z : w.x, b = half ? w.w : w.y;
  return (f32x4){__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u), __uint_as_float(b << 16),
                 __uint_as_float(b & 0xffff0000u)};
}
template <> struct Pieces<bf16_t> {
  static constexpr int COUNT = 3;
  // the largest piece of what is left of x, and the rest
  __device__ static __forceinline__ bf16x8 next(f32x4 (&x)[2]) {
    const bf16x8 f = round8(x[0], x[1]);
    x[0] -= low4(f, 0);
    x[1] -= low4(f, 1);
    return f;
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

// Rows of one head as a buffer resource that ends with row n - 1: rows behind
// read as zeros and are not written.  kNowhere is an offset past its end.
// With n = 0 nothing is read: loads ahead need no branch (what is merged
// behind one is waited for there).
constexpr uint32_t kNowhere = 0x80000000u;
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const View& x, int64_t tok, int n) {
  return rsrc((const T*)x.p + tok * x.ld, n > 0 ? (uint32_t)(((n - 1) * (int)x.ld + x.d) * (int)sizeof(T)) : 0u);
}

// C tokens of W channels on the way from memory to LDS, 16 bytes a lane;
// zeros for rows and channels that are not there.  A row's last vector, where
// the row ends inside it, is read from further ahead and moved down.
template <typename T, int W, int THREADS> struct Stage {
  static constexpr int VE = 16 / (int)sizeof(T), VPR = W / VE, RPP = THREADS / VPR, N = kTokens<T> / RPP;
  uint4 v[N];
  __device__ __forceinline__ void load(const View& x, int tok, int n) {
    const int thread = here((int)threadIdx.x), c = thread % VPR * VE, r = thread / VPR, step = (int)x.ld * (int)sizeof(T);
    const __amdgpu_buffer_rsrc_t rows = rows_of<T>(x, tok, n);
    const int at = c + VE <= x.d ? c : x.d - VE;
    const uint32_t off = c < x.d && x.d >= VE ? (uint32_t)(r * step + at * (int)sizeof(T)) : kNowhere;
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rows, off, i * RPP * step, 0));
  }
  // Whether a row of fewer channels than a vector has holds an infinity or a NaN.
  __device__ __forceinline__ bool store(T* X, const View& x, int tok, int n) {
    const int thread = here((int)threadIdx.x), c = thread % VPR * VE, r = thread / VPR;
    if (x.d % VE != 0 && x.d >= VE) {
      const bool tail = c < x.d && c + VE > x.d;
      const int bits = (VE - x.d % VE) * 8 * (int)sizeof(T);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint64_t lo = (uint64_t)v[i].y << 32 | v[i].x, hi = (uint64_t)v[i].w << 32 | v[i].z;
        const uint64_t a = bits < 64 ? lo >> bits | hi << (64 - bits) : hi >> (bits - 64), b = bits < 64 ? hi >> bits : 0;
        v[i] = tail ? make_uint4((uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)) : v[i];
      }
    }
    // RPP is a multiple of 8: the rows' swizzles differ in the upper bit at most
    const int swizzle = (r >> 2) & 3, other = swizzle & 1 ? -4 : 4;
    T* const row = X + r * kLd<W>;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      T* at = row + (((c >> 2) ^ swizzle ^ ((i * RPP >> 2) & 3)) << 2) + i * RPP * kLd<W>;
      if constexpr (sizeof(T) == 2) {
        *(uint2*)at = make_uint2(v[i].x, v[i].y);
        *(uint2*)(at + other) = make_uint2(v[i].z, v[i].w);
      } else {
        *(uint4*)at = v[i];
      }
    }
    // rows of fewer channels than a vector has, over the zeros that the same lane wrote
    bool narrow_wild = false;
    if (x.d < VE && c == 0)
#pragma unroll 1
      for (int k = r; k < n; k += RPP)
#pragma unroll 1
        for (int e = 0; e < x.d; ++e) {
          const T y = ((const T*)x.p)[(int64_t)(tok + k) * x.ld + e];
          X[k * kLd<W> + (((e >> 2) ^ ((k >> 2) & 3)) << 2) + (e & 3)] = y;
          narrow_wild |= (__float_as_uint(Elem<T>::to_f32(y)) & 0x7f800000u) == 0x7f800000u;
        }
    return narrow_wild;
  }
  // Back to memory, from the places that store() gives a lane, so that it may
  // write them anew without a barrier.  Whole vectors only.
  __device__ __forceinline__ static void write(const T* X, const View& y, int tok, int n) {
    const int thread = here((int)threadIdx.x), c = thread % VPR * VE, r = thread / VPR, step = (int)y.ld * (int)sizeof(T);
    const __amdgpu_buffer_rsrc_t rows = rows_of<T>(y, tok, n);
    const uint32_t off = c < y.d ? (uint32_t)(r * step + c * (int)sizeof(T)) : kNowhere;
    const int swizzle = (r >> 2) & 3, other = swizzle & 1 ? -4 : 4;
    const T* const row = X + r * kLd<W>;
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const T* at = row + (((c >> 2) ^ swizzle ^ ((i * RPP >> 2) & 3)) << 2) + i * RPP * kLd<W>;
      if constexpr (sizeof(T) == 2) {
        const uint2 a = *(const uint2*)at, b = *(const uint2*)(at + other);
        x[i] = (u32x4){a.x, a.y, b.x, b.y};
      } else {
        x[i] = *(const u32x4*)at;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) __builtin_amdgcn_raw_buffer_store_b128(x[i], rows, off + (uint32_t)(i * RPP * step), 0, 0);
  }
  // Whether some row may hold an infinity or a NaN: the largest magnitude of
  // all that was read, so that zeros for what is not there need no care.
  // Narrow rows are not in the registers: store() tells of them.
  __device__ __forceinline__ bool wild() const {
    if constexpr (sizeof(T) == 2) {
      typedef uint16_t pair __attribute__((ext_vector_type(2)));
      pair most = {0, 0};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint4 w = v[i];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          most = __builtin_elementwise_max(most, __builtin_bit_cast(pair, (&w.x)[e] & 0x7fff7fffu));
      }
      return most[0] >= 0x7f80 || most[1] >= 0x7f80;
    } else {
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint4 w = v[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) most = max(most, (&w.x)[e] & 0x7fffffffu);
      }
      return most >= 0x7f800000u;
    }
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
// Four channels of a lane's row of a resource: row i + r0 (r0 the same for the
// wave), channels c + c1 (c1 a constant).  d is a multiple of 4 with QUADS.
struct Lanes4 {
  __amdgpu_buffer_rsrc_t rows;
  int step, off, c, d;  // bytes between rows, the lane's offset, its first channel, channels
  __device__ __forceinline__ Lanes4(__amdgpu_buffer_rsrc_t rows, int64_t ld, int esz, int d, int i, int c)
      : rows(rows), step((int)ld * esz), off(i * step + c * esz), c(c), d(d) {}
};
template <typename T> struct Four {
  typedef uint32_t words __attribute__((ext_vector_type(sizeof(T))));  // 4 elements
  words w;
  template <bool QUADS>
  __device__ __forceinline__ void load(const Lanes4& l, int r0, int c1) {
    constexpr int E = (int)sizeof(T);
    const int row = r0 * l.step;
    if constexpr (QUADS) {
      const uint32_t off = l.c + c1 < l.d ? (uint32_t)(l.off + c1 * E) : kNowhere;
      if constexpr (E == 2) w = __builtin_bit_cast(words, __builtin_amdgcn_raw_buffer_load_b64(l.rows, off, row, 0));
      else w = __builtin_bit_cast(words, __builtin_amdgcn_raw_buffer_load_b128(l.rows, off, row, 0));
    } else {
      w = (words)0u;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (l.c + c1 + e < l.d) {
          if constexpr (E == 2)
            w[e / 2] |= ((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(l.rows, l.off + (c1 + e) * E, row, 0) & 0xffffu)
                        << e % 2 * 16;
          else w[e] = __builtin_amdgcn_raw_buffer_load_b32(l.rows, l.off + (c1 + e) * E, row, 0);
        }
    }
  }
  __device__ __forceinline__ void load(const Lanes4& l, int r0, int c1) {
    if (l.d % 4 == 0) load<true>(l, r0, c1);
    else load<false>(l, r0, c1);
  }
  __device__ __forceinline__ f32x4 get() const {
    if constexpr (sizeof(T) == 2)
      return (f32x4){__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                     __uint_as_float(w[1] & 0xffff0000u)};
    else return __builtin_bit_cast(f32x4, w);
  }
};
template <typename T, bool QUADS>
__device__ __forceinline__ void store4(const Lanes4& l, int r0, int c1, const f32x4& x) {
  constexpr int E = (int)sizeof(T);
  const int row = r0 * l.step;
  if constexpr (QUADS) {
    const uint32_t off = l.c + c1 < l.d ? (uint32_t)(l.off + c1 * E) : kNowhere;
    if constexpr (E == 2) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const bf16x2 a = f32x2_to_bf16x2(x[0], x[1]), b = f32x2_to_bf16x2(x[2], x[3]);
      __builtin_amdgcn_raw_buffer_store_b64((u32x2){__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)},
                                            l.rows, off, row, 0);
    } else {
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      // the row in the lanes' offset: a store of 16 bytes with a scalar one read registers that the next instruction had
      // written already (the compiler leaves a wait state only without it)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), l.rows, off + (uint32_t)row, 0, 0);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (l.c + c1 + e < l.d) {
        if constexpr (E == 2) __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(x[e]), l.rows, l.off + (c1 + e) * E, row, 0);
        else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[e]), l.rows, l.off + (c1 + e) * E, row, 0);
      }
  }
}

// four elements in LDS
__device__ __forceinline__ void put4(float* at, const f32x4& x) { *(f32x4*)at = x; }
__device__ __forceinline__ void put4(bf16_t* at, const f32x4& x) {
  *(uint2*)at = make_uint2(__builtin_bit_cast(uint32_t, f32x2_to_bf16x2(x[0], x[1])),
                           __builtin_bit_cast(uint32_t, f32x2_to_bf16x2(x[2], x[3])));
}

__device__ __forceinline__ f32x4 get4(const float* at) { return *(const f32x4*)at; }
__device__ __forceinline__ f32x4 get4(const bf16_t* at) {
  const uint2 w = *(const uint2*)at;
  return (f32x4){__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                 __uint_as_float(w.y & 0xffff0000u)};
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

// The same for a single token's decay, which a state is multiplied with at
// every step: the exponential instruction's errors lie to one side beside 1
// (0.12 times 2^-24 low on average) and would add up.  x = n + f with |f| <=
// 1/2, taken apart in 64 bits, 2^f = 1 + f (sum of ln2^k f^(k-1) / k!): less
// than 1.3 times 2^-24 off, to either side, and exactly 1 at 0.
__device__ __forceinline__ float step_decay(double x) {
  const float n = __builtin_rintf((float)x), f = (float)(x - (double)n);
  float p = 1.5252734e-5f;
  p = __builtin_fmaf(p, f, 1.5403530e-4f);
  p = __builtin_fmaf(p, f, 1.3333558e-3f);
  p = __builtin_fmaf(p, f, 9.6181291e-3f);
  p = __builtin_fmaf(p, f, 5.5504109e-2f);
  p = __builtin_fmaf(p, f, 2.4022651e-1f);
  p = __builtin_fmaf(p, f, 6.9314718e-1f);
  const float y = __builtin_ldexpf(__builtin_fmaf(p, f, 1.f), n > -200.f ? (int)n : -200);
  return y < 0x1p-126f ? 0.f : y;
}

// A token's log decay in units of a factor 2.  Values above 0 count as 0, and
// those below -10000 (infinities) as that, whose factor is 0 in fp32 and in
// 64 bits: differences of their sums stay finite.  A NaN stays.
__device__ __forceinline__ double log2_decay(float g) {
  g = g > 0.f ? 0.f : g;
  g = g < -1e4f ? -1e4f : g;
  return (double)g * 1.4426950408889634;
}

// A chunk's log decays, a lane each, on their way from memory.
template <typename T> struct LogDecays {
  View g;       // by token (none: an empty range)
  float fixed;  // by head
  float raw;
  __device__ __forceinline__ LogDecays(const LinearArgs& a, int h)
      : g{(const T*)a.g + h, a.g ? a.ld_g : 0, a.g ? 1 : 0}, fixed(a.decay ? a.decay[h] : 0.f), raw(0.f) {}
  __device__ __forceinline__ void load(int tok, int n, int lane) {
    const __amdgpu_buffer_rsrc_t rows = rows_of<T>(g, tok, n);
    const int off = lane * (int)g.ld * (int)sizeof(T);
    if constexpr (sizeof(T) == 2) raw = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(rows, off, 0, 0));
    else raw = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rows, off, 0, 0));
  }
  __device__ __forceinline__ float get() const {
    const float x = sizeof(T) == 2 ? __uint_as_float(__float_as_uint(raw) << 16) : raw;
    return g.d ? x : fixed;
  }
};

// Decays of a chunk's tokens in LDS, read four at a time.
template <typename T> struct alignas(16) Decays {
  double sum[kTokens<T>];               // running sums
  float row[kTokens<T>], col[kTokens<T>];  // factors of the state's part of an output, and of a token's part in the state
  float whole;
  int undefined;  // a NaN is among them
  // `lone`: a single token is none away from itself, also where its decay is a NaN
  __device__ __forceinline__ void fill(float g, int n, bool back, bool lone, float row_scale, float col_scale, int lane) {
    const double s = wave_sums(lane < n ? log2_decay(g) : 0.0);
    const uint64_t w = __builtin_bit_cast(uint64_t, s);
    const double all = __builtin_bit_cast(
        double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(w >> 32), 63) << 32 |
                    (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)w, 63));
    const float since = decay_of(s), until = decay_of(lone ? 0.0 : all - s);
    if (lane < kTokens<T>) {
      sum[lane] = lone ? 0.0 : s;
      row[lane] = (back ? until : since) * row_scale;
      col[lane] = (back ? since : until) * col_scale;
    }
    const bool nan = __ballot(lane < n && g != g) != 0;
    if (lane == 0) whole = decay_of(all), undefined = nan;
  }
};

// rows and columns of the second of two lie where 16-byte reads want them
static_assert(sizeof(Decays<bf16_t>) % 16 == 0 && sizeof(Decays<float>) % 16 == 0, "");

// ---- states in registers ----------------------------------------------------------
// State tiles: rows the channels that a product sums over (16 m + 4 g + r in
// lane 16 g + i), columns a wave's own (16 wave + i).  Records in the
// workspace hold whole tiles, padding included, in the order of the lanes:
// tile (row tile, column tile) is 256 floats, a lane's four side by side.  A
// role whose state is the transposed one (TR) reads them across.  The
// caller's states are [d_k][d_v].
template <int DK, int DV>
struct State {
  static constexpr int M = DK / 16;
  f32x4 s[M];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int m = 0; m < M; ++m) s[m] = (f32x4){0.f, 0.f, 0.f, 0.f};
  }
  // f(tile's four values, record's four values)
  template <bool TR, typename F>
  __device__ __forceinline__ void with_record(const float* p, int lane, int wave, F&& f) const {
    const __amdgpu_buffer_rsrc_t rec = rsrc(p, DK * DV * 4);
    const int g = lane >> 4, i = lane & 15, off = 4 * (TR ? 64 * (i >> 2) + 16 * g + (i & 3) : 4 * lane);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      f32x4 x;
      if (TR) {
        // row tile `wave`, column tile m of a record of DV rows and DK columns
#pragma unroll
        for (int r = 0; r < 4; ++r)
          x[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rec, off + 16 * r, (wave * M + m) * 1024, 0));
      } else {
        x = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rec, off, (m * (DV / 16) + wave) * 1024, 0));
      }
      f(m, x);
    }
  }
  template <bool TR>
  __device__ __forceinline__ void load(const float* p, int lane, int wave) {
    with_record<TR>(p, lane, wave, [&](int m, const f32x4& x) { s[m] = x; });
  }
  __device__ __forceinline__ void store(float* p, int lane, int wave) const {
#pragma unroll
    for (int m = 0; m < M; ++m) *(f32x4*)(p + (m * (DV / 16) + wave) * 256 + 4 * lane) = s[m];
  }
  __device__ __forceinline__ float dot(const float* p, int lane, int wave) const {
    float sum = 0.f;
    with_record<false>(p, lane, wave, [&](int m, const f32x4& x) {
#pragma unroll
      for (int r = 0; r < 4; ++r) sum += s[m][r] * x[r];
    });
    return sum;
  }

  // A caller's state, rows by cols of it (TR: held cols by rows).  Straight to
  // the lanes: through LDS, where every load and store would be of whole
  // lines, a workgroup with a state to read started 5 us later.
  // f(tile, its place r: offset of the lane, offset of the wave)
  template <bool TR, typename F>
  __device__ __forceinline__ static void places(int rows, int cols, int lane, int wave, F&& f) {
    const int g = lane >> 4, col = 16 * wave + (lane & 15);
    const uint32_t off = col < cols ? (uint32_t)(TR ? col * rows + 4 * g : 4 * g * cols + col) * 4 : kNowhere;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // not transposed, rows past the last are past the end
        if (TR) f(m, r, (16 * m + 4 * g + r < rows ? off : kNowhere) + (16 * m + r) * 4, 0);
        else f(m, r, off, (16 * m + r) * cols * 4);
      }
  }
  template <bool TR, typename F>
  __device__ __forceinline__ static void with_caller(const float* p, int rows, int cols, int lane, int wave, F&& f) {
    const __amdgpu_buffer_rsrc_t mem = rsrc(p, (uint32_t)(rows * cols * 4));
    places<TR>(rows, cols, here(lane), wave, [&](int m, int r, uint32_t off, int at) {
      f(m, r, __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(mem, off, at, 0)));
    });
  }
  template <bool TR>
  __device__ __forceinline__ void load_caller(const float* p, int rows, int cols, int lane, int wave) {
    if (!p) return zero();
    with_caller<TR>(p, rows, cols, lane, wave, [&](int m, int r, float x) { s[m][r] = x; });
  }
  template <bool TR>
  __device__ __forceinline__ float dot_caller(const float* p, int rows, int cols, int lane, int wave) const {
    float sum = 0.f;
    with_caller<TR>(p, rows, cols, lane, wave, [&](int m, int r, float x) { sum += s[m][r] * x; });
    return sum;
  }
  template <bool TR>
  __device__ __forceinline__ void store_caller(float* p, int rows, int cols, int lane, int wave) const {
    const __amdgpu_buffer_rsrc_t mem = rsrc(p, (uint32_t)(rows * cols * 4));
    places<TR>(rows, cols, here(lane), wave, [&](int m, int r, uint32_t off, int at) {
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s[m][r]), mem, off, at, 0);
    });
  }
};

// ---- a chunk's step of the state ------------------------------------------------------
// S <- whole S + K^T (col V): V's fragments are this wave's own columns,
// scaled and cut to pieces; K's are read from LDS as they are.
template <typename T, int DK, int DV, int ROWS = 4>
__device__ __forceinline__ void step_state(const T* K, const Lane<T, DK>& lk, const typename Frag<T>::type (&vf)[2],
                                           const Decays<T>& d, int lane, State<DK, DV>& st) {
  constexpr int KB = Elem<T>::KB, PIECES = Pieces<T>::COUNT;
  const int g = lane >> 4;
  const float whole = d.whole;
  auto scaled = [&](int kb, f32x4 (&x)[kAccs<T>]) {
    widen(vf[kb], x);
#pragma unroll
    for (int h = 0; h < kAccs<T>; ++h) x[h] *= *(const f32x4*)(d.col + KB * kb + 16 * h + 4 * g);
  };
  if constexpr (PIECES == 1) {
    // fp32: the chunk's sum is formed by itself and added to the state once.
    // Added product by product, a state of many chunks took a rounding of its
    // own size with each of eight (outputs of rows of 1024 tokens 3.7e-7 off,
    // with one of them 2.2e-7; 94.1 against 97.1 us for 5003 packed tokens).
    // bf16 makes six products of a chunk of twice the tokens; there the sums
    // cost 128 by 128 channels registers (training step 125 against 136 us).
    f32x4 f[2][1];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) scaled(kb, f[kb]);
#pragma unroll
    for (int m = 0; m < DK / 16; m += 2) {
      f32x4 sum[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) sum[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 2; ++i) sum[i] = mma(col_frag<DK>(K, lk, KB * kb, 16 * (m + i)), f[kb][0], sum[i]);
#pragma unroll
      for (int i = 0; i < 2; ++i) st.s[m + i] = formed(st.s[m + i] * whole + sum[i]);
    }
  } else {
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) st.s[m] *= whole;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      typename Frag<T>::type f[PIECES];
      f32x4 x[kAccs<T>];
      scaled(kb, x);
#pragma unroll
      for (int p = 0; p < PIECES; ++p) f[p] = Pieces<T>::next(x);
      // ROWS row tiles at a time: a product's result is not wanted by the next
#pragma unroll
      for (int m = 0; m < DK / 16; m += ROWS) {
        typename Frag<T>::type kf[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) kf[i] = col_frag<DK>(K, lk, KB * kb, 16 * (m + i));
#pragma unroll
        for (int p = PIECES - 1; p >= 0; --p)
#pragma unroll
          for (int i = 0; i < ROWS; ++i) st.s[m + i] = mma(kf[i], f[p], st.s[m + i]);
      }
    }
  }
}

template <typename T, int DV>
__device__ __forceinline__ void own_columns(const T* V, const Lane<T, DV>& lv, int c0, typename Frag<T>::type (&vf)[2]) {
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) vf[kb] = col_frag<DV>(V, lv, Elem<T>::KB * kb, c0);
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
// that entered.  Rows and columns: k and v.  In the backward pass (TR) the
// transposed states are wanted: v and k, and for the gradients dout and q.
// 16 us for 4096 tokens of 16 bf16 heads, 256 workgroups of four chunks: 5300
// cycles a chunk, of them 1540 of matrix instructions (three pieces of V) and
// 1850 with their operands' reads; the first chunk waits 2800 for memory.  A
// second set of tiles in LDS, one barrier a chunk, and the decays of four
// chunks at once measured the same (57.1 and 58.4 us for the three launches).
template <typename T, int DK, int DV, bool BACK, typename F>
__device__ __forceinline__ void states_range(const LinearArgs& a, const View& k, const View& v, int h, int t0, int end,
                                             char* smem, State<DK, DV>& st, double* total, F&& enter) {
  constexpr int C = kTokens<T>, THREADS = kThreads<DV>;
  T* K = (T*)smem;
  T* V = (T*)(smem + kTileBytes<T, DK>);
  Decays<T>* const both = (Decays<T>*)(smem + kTileBytes<T, DK> + kTileBytes<T, DV>);  // of this chunk and the next
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c0 = wave * 16;
  const Lane<T, DK> lk(lane);
  const Lane<T, DV> lv(lane);
  const int chunks = (end - t0 + C - 1) / C;
  // Chunks are loaded two ahead: one chunk's products are shorter than memory
  // takes with a workgroup or two on a compute unit.
  Stage<T, DK, THREADS> sk[2];
  Stage<T, DV, THREADS> sv[2];
  LogDecays<T> g(a, h);
  auto start_of = [&](int i) { return i < chunks ? t0 + (BACK ? chunks - 1 - i : i) * C : t0; };
  auto size_of = [&](int i) {
    const int left = end - start_of(i), n = left < C ? left : C;
    return i < chunks ? n : 0;
  };
  auto load = [&](auto set, int i) {
    sk[set.value].load(k, start_of(i), size_of(i));
    sv[set.value].load(v, start_of(i), size_of(i));
  };
  auto decays = [&](int i) {
    if (wave == 0) both[i & 1].fill(g.get(), size_of(i), BACK, false, 1.f, BACK ? a.scale : 1.f, lane);
  };
  auto chunk = [&](auto set, int i) {
    sk[set.value].store(K, k, start_of(i), size_of(i));
    sv[set.value].store(V, v, start_of(i), size_of(i));
    lds_barrier();
    const Decays<T>* d = both + (i & 1);
    load(set, i + 2);
    g.load(start_of(i + 1), size_of(i + 1), lane);
    if (total) *total += d->sum[C - 1];
    typename Frag<T>::type vf[2];
    own_columns<T, DV>(V, lv, c0, vf);
    step_state<T, DK, DV>(K, lk, vf, *d, lane, st);
    decays(i + 1);
    lds_barrier();
  };
  constexpr std::integral_constant<int, 0> even;
  constexpr std::integral_constant<int, 1> odd;
  g.load(start_of(0), size_of(0), lane);
  load(even, 0);
  load(odd, 1);
  enter();
  decays(0);
  for (int i = 0; i < chunks; i += 2) {
    chunk(even, i);
    if (i + 1 < chunks) chunk(odd, i + 1);
  }
}

template <typename T, int DK, int DV>
constexpr int kStatesLds = kTileBytes<T, DK> + kTileBytes<T, DV> + 2 * (int)sizeof(Decays<T>);
template <typename T, int DK, int DV, bool TR>
__global__ void __launch_bounds__(kThreads<DV>, (kWavesOfSimd<DK, DV>))
linear_states(const LinearArgs a, const T* __restrict__ dout, const float* __restrict__ dht, float* __restrict__ ends,
              float* __restrict__ adj, double* __restrict__ sums, int* __restrict__ kinds) {
  __shared__ __align__(16) char smem[kStatesLds<T, DK, DV>];
  const int h = (int)(blockIdx.x % (unsigned)a.H), hq = h / (a.H / a.Hq);
  const Slot w(a, (int)(blockIdx.x / (unsigned)a.H));
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int64_t floats = (int64_t)a.dk * a.dv, at = ((int64_t)w.slot * a.H + h) * DK * DV;
  State<DK, DV> st;
  const int first = uniform(seqs.from(w.lo)), before = first > 0 ? uniform((int)seqs.end(first - 1)) : w.lo;
  const bool entered = before > w.lo;
  double total = 0.0;
  if (!TR || blockIdx.y == 0) {
    const int n = uniform(seqs.from(w.hi)) - 1;  // the last sequence that starts in the slot or before
    const bool on = !w.last && n >= 0 && uniform((int)seqs.end(n)) > w.hi;
    const int start = on ? uniform((int)seqs.start(n)) : 0;
    const bool own = start >= w.lo;
    if (h == 0 && threadIdx.x == 0)
      kinds[w.slot] = (!on ? kNothing : own ? kStarted : kPassed) | (entered ? kEntered : 0);
    if (!on) return;
    auto enter = [&] {
      st.template load_caller<TR>(own && a.h0 ? a.h0 + ((int64_t)n * a.H + h) * floats : nullptr, TR ? a.dv : a.dk,
                                  TR ? a.dk : a.dv, lane, wave);
    };
    const View k{(const T*)a.k + hq * a.dk, a.ld_k, a.dk}, v{(const T*)a.v + h * a.dv, a.ld_v, a.dv};
    states_range<T, DK, DV, false>(a, TR ? v : k, TR ? k : v, h, own ? start : w.lo, w.hi, smem, st, &total, enter);
    st.store(ends + at, lane, wave);
    if (!own && threadIdx.x == 0) sums[(int64_t)w.slot * a.H + h] = total;
  } else if constexpr (TR) {
    if (!entered) return;
    const bool ends_here = before <= w.hi;
    auto enter = [&] {
      st.template load_caller<TR>(ends_here && dht ? dht + ((int64_t)(first - 1) * a.H + h) * floats : nullptr, a.dv,
                                  a.dk, lane, wave);
    };
    const View q{(const T*)a.q + hq * a.dk, a.ld_q, a.dk}, d{dout + h * a.dv, (int64_t)a.H * a.dv, a.dv};
    states_range<T, DK, DV, true>(a, d, q, h, w.lo, ends_here ? before : w.hi, smem, st, nullptr, enter);
    st.store(adj + at, lane, wave);
  }
}

// True states at the slots' ends out of what each slot made of a zero state,
// in place: S_i <- S_i + decay_i S_{i-1} where a sequence passes through slot
// i; likewise (blockIdx.y = 1) the gradients from the last slot to the first.
// A lane takes four elements; a batch of eight slots is loaded while the one
// before is passed through (without: 2 to 5 us more; batches of 16 6 us more).
// 8.4 us for 16 slots of 16 heads of 128 by 128, 33.5 MB read and written (4.0
// TB/s, with hits in the caches).
__global__ void __launch_bounds__(256)
linear_chain(int H, int64_t quads, int n_slots, float* __restrict__ ends, float* __restrict__ adj,
             const double* __restrict__ sums, const int* __restrict__ kinds) {
  constexpr int BATCH = 8;
  const bool back = blockIdx.y != 0;
  const int64_t per = quads / 256;
  const int h = (int)(blockIdx.x / per);
  const int64_t el = (blockIdx.x % per) * 256 + threadIdx.x;
  f32x4* __restrict__ v = (f32x4*)(back ? adj : ends) + h * quads + el;
  const int64_t step = (int64_t)H * quads;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  struct Batch {
    f32x4 made[BATCH];
    double by[BATCH];
    int kd[BATCH];
  } x, y;
  auto load = [&](Batch& b, int i0) {
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const int i = i0 + j < n_slots ? i0 + j : n_slots - 1, slot = back ? n_slots - 1 - i : i;
      b.kd[j] = kinds[slot];
      b.made[j] = v[slot * step];
      b.by[j] = sums[(int64_t)slot * H + h];
    }
  };
  auto pass = [&](const Batch& b, int i0) {
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      if (i0 + j >= n_slots) break;
      const int slot = back ? n_slots - 1 - i0 - j : i0 + j;
      const bool holds = back ? b.kd[j] & kEntered : b.kd[j] & (kStarted | kPassed), passed = b.kd[j] & kPassed;
      const float by = decay_of(b.by[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = (passed ? by * s[e] : 0.f) + (holds ? b.made[j][e] : 0.f);
      if (passed) v[slot * step] = s;
    }
  };
  load(x, 0);
  for (int i0 = 0; i0 < n_slots; i0 += 2 * BATCH) {
    load(y, i0 + BATCH);
    pass(x, i0);
    load(x, i0 + 2 * BATCH);
    pass(y, i0 + BATCH);
  }
}

// ---- outputs -------------------------------------------------------------------------------
// One form for the outputs and the three gradients ("sweep"): rows of Q meet
// rows of K, whose weights sum rows of V.
// A chunk of 64 bf16 tokens of 128 by 128 channels takes a workgroup 13,600
// cycles, and two beside each other on a compute unit 26,000: 3900 each are of
// matrix instructions, 5200 of the vector unit (rounding to pieces, decays),
// the rest waits, for LDS (510 KB read a chunk) and at three barriers.  Where
// one workgroup a unit is left, two that share a slot, the second after a pass
// over the first half for its state, took the same time as one (30.3 and 32.4
// us for the prompt's sweep): the second pass's start costs what it hides.
enum Role { kForward, kDq, kDk, kDv };

struct Sweep {
  View q, k, v;
  View other;       // the rows that outputs are multiplied with for the decays' gradients
  void* out;        // [tokens, H, v.d], this head's first element; fp32 with `wide`
  bool wide;
  float p_scale, row_scale, col_scale;
  float* dots;      // [H, tokens], this head's row (null: none)
};

// P's tiles on and beside the diagonal, in the order that waves take them.
__device__ __forceinline__ void tile_of(int t, int* a, int* b) {
  *a = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
  *b = t - *a * (*a + 1) / 2;
}
template <typename T> constexpr int kRowTiles = kTokens<T> / 16;
template <typename T> constexpr int kPTiles = kRowTiles<T> * (kRowTiles<T> + 1) / 2;

// Tiles of P in LDS are in the order of the lanes, four elements of a row
// each: what a lane of one wave forms, the same lane of every wave reads.
// P's operand of row tile rt for the tokens from KB kb on; the other side of
// the diagonal (BACK: before rt) is zeros.
template <bool BACK, int KB>
__device__ __forceinline__ bf16x8 p_frag(const bf16_t* P, int rt, int kb, int lane) {
  bf16x4 x[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int ct = 2 * kb + half, hi = ct > rt ? ct : rt, lo = ct > rt ? rt : ct;
    x[half] = (BACK ? ct >= rt : ct <= rt) ? *(const bf16x4*)(P + (hi * (hi + 1) / 2 + lo) * 256 + 4 * lane)
                                           : __builtin_bit_cast(bf16x4, (uint64_t)0);
  }
  return (bf16x8){x[0][0], x[0][1], x[0][2], x[0][3], x[1][0], x[1][1], x[1][2], x[1][3]};
}
template <bool BACK, int KB>
__device__ __forceinline__ f32x4 p_frag(const float* P, int rt, int ct, int lane) {
  const int hi = ct > rt ? ct : rt, lo = ct > rt ? rt : ct;
  return *(const f32x4*)(P + (hi * (hi + 1) / 2 + lo) * 256 + 4 * lane);
}

template <typename T, int DK, int DV>
struct SweepLds {
  T q[kTokens<T> * kLd<DK>], k[kTokens<T> * kLd<DK>], v[kTokens<T> * kLd<DV>];
  T p[Pieces<T>::COUNT][kPTiles<T> * 256];
  Decays<T> d[2];  // of this chunk and the next
  int wild;
  float dot[kWaves<DV>][kTokens<T>];
  float diagonal[kTokens<T>];  // of P, where it is kept apart
};

// Tokens [t0, end) of one sequence; the state before them (BACK: the gradient
// of the state after them) comes from `enter`, called when the first loads are
// under way, and that after (before) them is left in st.
template <typename T, int DK, int DV, Role R, typename F>
__device__ __forceinline__ void sweep_range(const LinearArgs& a, const Sweep& w, int h, int t0, int end,
                                            SweepLds<T, DK, DV>& m, State<DK, DV>& st, F&& enter) {
  constexpr bool BACK = R == kDk || R == kDv;
  constexpr int C = kTokens<T>, KB = Elem<T>::KB, RT = kRowTiles<T>, TILES = kPTiles<T>;
  constexpr int PIECES = Pieces<T>::COUNT, WAVES = kWaves<DV>, THREADS = kThreads<DV>;
  typedef typename Frag<T>::type frag;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c0 = wave * 16;
  const int chunks = (end - t0 + C - 1) / C;
  // For the decays' gradients a token's own product is added to the output
  // behind the inner product that they take, which is to hold other tokens' only.
  const bool strict = (R == kDq || R == kDk) && w.dots;
  Stage<T, DK, THREADS> sq, sk;
  Stage<T, DV, THREADS> sv;
  LogDecays<T> gd(a, h);
  auto load = [&](int t, int n) {
    sq.load(w.q, t, n);
    sk.load(w.k, t, n);
    sv.load(w.v, t, n);
  };
  // chunk i is [t, t + n); one that holds an infinity or a NaN among V is
  // walked token by token (one < n), so that a weight of zero never meets it,
  // and one with a NaN among its decays, back in time
  int i = 0, one = 0;
  auto start_of = [&](int c) { return t0 + (BACK ? chunks - 1 - c : c) * C; };
  auto size_of = [&](int t) { return end - t < C ? end - t : C; };
  int t = start_of(0), n = size_of(t), whole_n = n, buf = 0;
  bool single = false;
  // one wave does the decays of a chunk, ahead of it
  auto decays = [&](int b, int n) {
    if (wave != WAVES - 1) return;
    m.d[b].fill(gd.get(), n, BACK, n == 1, w.row_scale, w.col_scale, lane);
  };
  gd.load(t, n, lane);
  load(t, n);
  enter();
  decays(0, n);
  while (true) {
    sq.store(m.q, w.q, t, n);
    sk.store(m.k, w.k, t, n);
    const bool narrow_wild = sv.store(m.v, w.v, t, n);
    if (!single && n > 1 && __ballot(narrow_wild || sv.wild()) != 0 && lane == 0) m.wild = 1;
    lds_barrier();
    // Back in time a NaN among the decays does not concern the tokens behind
    // it, but it is in all the running sums there.  (It lies with the chunk's
    // decays: the next chunk's are written while others may still read here.)
    if (!single && n > 1 && uniform(m.wild | (BACK ? m.d[buf].undefined : 0))) {
      lds_barrier();  // all have read it
      if (threadIdx.x == 0) m.wild = 0;
      single = true;
      one = 0;
      whole_n = n;
      n = 1;
      t = start_of(i) + (BACK ? whole_n - 1 : 0);
      gd.load(t, n, lane);
      load(t, n);
      decays(buf, n);
      lds_barrier();
      continue;
    }
    // what comes next
    int t_next = t, n_next = 0;
    if (single && one + 1 < whole_n) {
      t_next = BACK ? t - 1 : t + 1;
      n_next = 1;
    } else if (i + 1 < chunks) {
      t_next = start_of(i + 1);
      n_next = size_of(t_next);
    }
    gd.load(t_next, n_next, lane);
    const Decays<T>& d = m.d[buf];

    // P, shared out by tiles
    auto p_tile = [&](int tile) {
      const int ln = here(lane), g = ln >> 4, i16 = ln & 15;
      const Lane<T, DK> lk(ln);
      int ra, rb;
      tile_of(tile, &ra, &rb);
      const int rt = BACK ? rb : ra, ct = BACK ? ra : rb;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      // four steps' operands at a time, so that one wait serves them
#pragma unroll
      for (int kb = 0; kb < DK / KB; kb += 4) {
        constexpr int U = DK / KB < 4 ? DK / KB : 4;
        frag x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          x[u] = row_frag<DK>(m.k, lk, 16 * ct, KB * (kb + u));
          y[u] = row_frag<DK>(m.q, lk, 16 * rt, KB * (kb + u));
        }
        fence();
#pragma unroll
        for (int u = 0; u < U; ++u) acc = mma(x[u], y[u], acc);
      }
      const double gi = d.sum[16 * rt + i16];
      const int at = i16 - 4 * g + 16 * (rt - ct);  // row minus column, of r = 0
      f32x4 p;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const double gj = d.sum[16 * ct + 4 * g + r];
        const float x = acc[r] * (decay_of(BACK ? gj - gi : gi - gj) * w.p_scale);
        p[r] = (BACK ? at <= r : at >= r) ? x : 0.f;
      }
      if (strict && rt == ct) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (at == r) m.diagonal[16 * rt + i16] = p[r];
          p[r] = at == r ? 0.f : p[r];
        }
      }
      f32x4 x = p;
#pragma unroll
      for (int c = 0; c < PIECES; ++c) {
        T* at = m.p[c] + tile * 256 + 4 * ln;
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
    };
#pragma unroll 1
    for (int tile = wave; tile < TILES; tile += WAVES) p_tile(tile);

    // the state's part of the outputs, transposed: rows are channels of V, columns tokens
    const int ln = here(lane), g = ln >> 4, i16 = ln & 15;
    const Lane<T, DK> lk(ln);
    // the rows that outputs are multiplied with arrive under the products
    Four<T> other[RT];
    if (strict) {
      const Lanes4 rows(rows_of<T>(w.other, t, n), w.other.ld, sizeof(T), w.other.d, i16, c0 + 4 * g);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) other[rt].load(rows, 16 * rt, 0);
    }
    f32x4 acc[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[rt] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < DK / KB; ++kb) {
      f32x4 s[kAccs<T>];
#pragma unroll
      for (int e = 0; e < kAccs<T>; ++e) s[e] = st.s[kAccs<T> * kb + e];
      frag qf[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) qf[rt] = row_frag<DK>(m.q, lk, 16 * rt, KB * kb);
      // a piece at a time: three together would cost registers
#pragma unroll
      for (int c = 0; c < PIECES; ++c) {
        const frag sf = Pieces<T>::next(s);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[rt] = mma(sf, qf[rt], acc[rt]);
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[rt] *= d.row[16 * rt + i16];
    // the next chunk's loads have the products below to arrive in (ahead of those above they would cost registers)
    load(t_next, n_next);
    decays(buf ^ 1, n_next);
    lds_barrier();
    // the chunk's own part
    frag vf[2];
    own_columns<T, DV>(m.v, Lane<T, DV>(ln), c0, vf);
    if (!strict || n > 1)  // the one token may hold an infinity, which a zero is not multiplied with
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int c = PIECES - 1; c >= 0; --c)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            if (BACK ? KB * (kb + 1) <= 16 * rt : KB * kb > 16 * rt) continue;  // zeros of P
            acc[rt] = mma(vf[kb], p_frag<BACK, KB>(m.p[c], rt, kb, ln), acc[rt]);
          }
    if (strict) {
      float s[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const f32x4 z = other[rt].get(), v = get4(m.v + Lane<T, DV>(ln).row + 16 * rt * kLd<DV> + c0);
        const float own = m.diagonal[16 * rt + i16];
        s[rt] = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          s[rt] += acc[rt][r] * z[r];
          acc[rt][r] += own * v[r];
        }
      }
      // over the four rows of lanes; row g is left with the sum of tokens 16 g + i
      float all = swap_sum<16>(s[0], s[1]);
      if constexpr (RT == 4) all = swap_sum<32>(all, swap_sum<16>(s[2], s[3]));
      else all = swap_sum<32>(all, all);
      if (lane < C) m.dot[wave][lane] = all;
    }
    // The outputs go to memory in whole vectors, by way of this wave's own
    // columns of V, which nothing else reads any more; or as they are.
    const View y{w.out, (int64_t)a.H * w.v.d, w.v.d};
    const bool by_rows = !((R == kDq || R == kDk) && w.wide) && y.d % (16 / (int)sizeof(T)) == 0;
    auto out = [&](auto type, auto quads) {
      typedef decltype(type) E;
      const Lanes4 to(rows_of<E>(y, t, n), y.ld, sizeof(E), y.d, i16, c0 + 4 * g);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) store4<E, quads.value>(to, 16 * rt, 0, acc[rt]);
    };
    auto out_as = [&](auto type) {
      if (y.d % 4 == 0) out(type, std::true_type{});
      else out(type, std::false_type{});
    };
    if (by_rows) {
      const Lane<T, DV> lv(ln);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) put4(m.v + lv.row + 16 * rt * kLd<DV> + c0, acc[rt]);
    } else if ((R == kDq || R == kDk) && w.wide) {
      out_as(float{});
    } else {
      out_as(T{});
    }
    // The widest gradients leave fewer registers for it (2x2048 tokens of 16
    // heads of 128 127 us with four row tiles at a time, 123 with two; other
    // sizes within 1 percent).
    constexpr int ROWS = R != kForward && DK == 128 && DV == 128 ? 2 : 4;
    if (ROWS == 2) fence();
    step_state<T, DK, DV, ROWS>(m.k, Lane<T, DK>(here(lane)), vf, d, lane, st);
    lds_barrier();
    if (by_rows) Stage<T, DV, THREADS>::write(m.v, y, t, n);
    if (strict && (int)threadIdx.x < n) {
      const int row = threadIdx.x;
      float s = 0.f;
#pragma unroll
      for (int x = 0; x < WAVES; ++x) s += m.dot[x][row];
      w.dots[t + row] = s;
    }
    if (n_next == 0) break;
    if (single && one + 1 < whole_n) {
      ++one;
    } else {
      single = false;
      ++i;
    }
    t = t_next;
    n = n_next;
    buf ^= 1;
  }
  if (strict) lds_barrier();  // the dots are read
}

// One slot of one head.  dS: what a sequence's last state's inner product with its gradient is wanted of.
template <typename T, int DK, int DV, Role R>
__device__ __forceinline__ void sweep_slot(const LinearArgs& a, const Sweep& w, int h, const Slot& s, const float* enter,
                                           const float* seq_state, float* leave, const float* dht, const float* adj,
                                           float* seq_dot, float* slot_dot, SweepLds<T, DK, DV>& m) {
  constexpr bool BACK = R == kDk || R == kDv, TR = R == kDq || R == kDk;
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int64_t floats = (int64_t)a.dk * a.dv, record = DK * DV;
  const int rows = w.q.d, cols = w.v.d;
  State<DK, DV> st;
  if (threadIdx.x == 0) m.wild = 0;
  lds_barrier();
  auto of_slot = [&](int i) { return enter + ((int64_t)i * a.H + h) * record; };
  auto of_seq = [&](const float* p, int n) { return p ? p + ((int64_t)n * a.H + h) * floats : nullptr; };
  // <S, dS> at the end of a range
  auto inner = [&](float x, float* out) {
    x = row_sum(x);
    x += __shfl_xor(x, 16, 64);
    x += __shfl_xor(x, 32, 64);
    if (lane == 0) m.dot[threadIdx.x >> 6][0] = x;
    lds_barrier();
    if (threadIdx.x == 0) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves<DV>; ++w) sum += m.dot[w][0];
      *out = sum;
    }
    lds_barrier();
  };
  auto piece = [&](int n, int start, int end, bool entered) {
    const bool done = end <= s.hi;
    const int stop = done ? end : s.hi;
    auto enter_state = [&] {
      // records: the state's own orientation forward, the transposed one backward
      if (BACK ? !done : entered) st.template load<R == kDv>(of_slot(BACK ? s.slot + 1 : s.slot - 1), lane, wave);
      else st.template load_caller<TR>(of_seq(seq_state, n), rows, cols, lane, wave);
    };
    const bool out = leave && (BACK ? !entered : done);
    if (start < stop) sweep_range<T, DK, DV, R>(a, w, h, start, stop, m, st, enter_state);
    else enter_state();
    if (R == kDq && w.dots) {
      float x = 0.f;
      if (!done) x = st.dot(adj + ((int64_t)(s.slot + 1) * a.H + h) * record, lane, wave);
      else if (dht) x = st.template dot_caller<TR>(of_seq(dht, n), rows, cols, lane, wave);
      inner(x, (done ? seq_dot + (int64_t)n * a.H : slot_dot + (int64_t)s.slot * a.H) + h);
    }
    if (out) st.template store_caller<TR>(leave + ((int64_t)n * a.H + h) * floats, rows, cols, lane, wave);
  };
  // the sequence that entered, then those that start here; the last slot also has the empty ones behind the last token
  int n = uniform(seqs.from(s.lo)), at = s.lo;
  bool entered = n > 0 && uniform((int)seqs.end(n - 1)) > s.lo;
  if (entered) --n;
  for (; n < a.n_seqs; ++n) {
    const Span range = seqs.next(n, &at);
    const int start = uniform(range.start), end = uniform(range.end);
    if (!s.last && start >= s.hi) break;
    piece(n, start, end, entered);
    entered = false;
  }
}

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kThreads<DV>, (kWavesOfSimd<DK, DV>))
linear_forward(const LinearArgs a, const float* __restrict__ ends, T* __restrict__ o, float* __restrict__ ht) {
  __shared__ __align__(16) SweepLds<T, DK, DV> m;
  const int h = (int)(blockIdx.x % (unsigned)a.H), hq = h / (a.H / a.Hq);
  const Slot s(a, (int)(blockIdx.x / (unsigned)a.H));
  Sweep w{};
  w.q = View{(const T*)a.q + hq * a.dk, a.ld_q, a.dk};
  w.k = View{(const T*)a.k + hq * a.dk, a.ld_k, a.dk};
  w.v = View{(const T*)a.v + h * a.dv, a.ld_v, a.dv};
  w.out = o + h * a.dv;
  w.p_scale = w.row_scale = a.scale;
  w.col_scale = 1.f;
  sweep_slot<T, DK, DV, kForward>(a, w, h, s, ends, a.h0, ht, nullptr, nullptr, nullptr, nullptr, m);
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
  sweep_slot<T, R == kDv ? DK : DV, R == kDv ? DV : DK, R>(
      a, w, h, s, enter, R == kDq ? a.h0 : g.dht, R == kDv ? g.dh0 : nullptr, g.dht, x.adj, x.seq_dot, x.slot_dot,
      *(SweepLds<T, R == kDv ? DK : DV, R == kDv ? DV : DK>*)smem);
}

// The workgroups of a launch take its roles in turn: all three where their
// workgroups are of one size, else those with columns of d_k, and dv alone.
template <typename T, int DK, int DV, Role FIRST, int COUNT>
__global__ void __launch_bounds__(kThreads<(FIRST == kDv ? DV : DK)>,
                                  (kWavesOfSimd<(FIRST == kDv ? DK : DV), (FIRST == kDv ? DV : DK)>))
linear_backward(const LinearArgs a, const LinearGrads g, const LinearWork x) {
  typedef SweepLds<T, DV, DK> OfKeys;
  typedef SweepLds<T, DK, DV> OfValues;
  constexpr size_t keys = FIRST == kDv ? 0 : sizeof(OfKeys), values = FIRST == kDv || COUNT == 3 ? sizeof(OfValues) : 0;
  __shared__ __align__(16) char smem[keys > values ? keys : values];
  const unsigned role = blockIdx.x % COUNT, id = blockIdx.x / COUNT;
  const int h = (int)(id % (unsigned)a.H);
  const Slot s(a, (int)(id / (unsigned)a.H));
  if constexpr (FIRST == kDv) {
    gradient<T, DK, DV, kDv>(a, g, x, h, s, smem);
  } else {
    if (role == 0) gradient<T, DK, DV, kDq>(a, g, x, h, s, smem);
    else if (role == 1) gradient<T, DK, DV, kDk>(a, g, x, h, s, smem);
    else if constexpr (COUNT == 3) gradient<T, DK, DV, kDv>(a, g, x, h, s, smem);
  }
}

// The decays' gradients: a wave takes one slot of one head, 64 tokens at a
// time from each sequence's end, as suffix sums in 64 bits.  A token whose
// factor is 0 lets nothing through: its own gradient is 0, and the sums begin
// anew before it, without what the roundings of later tokens have left.  5.5
// us for 4096 tokens of 16 heads: four dependent rounds of 64 tokens a wave.
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
      double v = wave_sums(there ? (double)dq[t] - (double)dk[t] : 0.0) + carry;
      const float g = there ? Elem<T>::to_f32(((const T*)a.g)[(int64_t)t * a.ld_g + h]) : 0.f;
      const uint64_t cuts = __ballot(decay_of(log2_decay(g)) == 0.f);
      if (cuts != 0) {
        const uint64_t later = cuts & ~0ull >> (63 - lane);  // this token's and those of later ones
        const int at = later != 0 ? 63 - __builtin_clzll(later) : 0;
        const double upto = __shfl(v, at, 64);
        v = later != 0 ? v - upto : v;
      }
      if (there) dg[(int64_t)t * a.H + h] = Elem<T>::from_f32(g > 0.f ? 0.f : (float)v);
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

// Gradients of shared queries and keys: the sum over the heads that share, in
// the order of the heads (atomics would change with the order of workgroups).
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
// The state is read once and written once, which is all that counts: 256
// sequences of 32 heads of 128 by 128, 1.08 GB, 211 us, the rate of a large
// copy (5.1 TB/s).  A workgroup owns one (sequence, head); a thread 4 columns of
// every (threads / LC)-th row, with all its loads issued before the first use.
// 4 sequences of 8 heads of 64 by 64 take 3.7 us, a launch and one round trip.
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
  const float by = step_decay(log2_decay(g));
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
  const View out{o + h * a.dv, (int64_t)a.H * a.dv, a.dv};
  const Lanes4 to(rows_of<T>(out, seq, 1), 0, sizeof(T), a.dv, 0, c);
  if (quads) store4<T, true>(to, 0, 0, y);
  else store4<T, false>(to, 0, 0, y);
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

// the states that the slots hand on, and (BACK) the gradients
template <typename T, int DK, int DV, bool BACK>
int states(const LinearArgs& a, const LinearPlan& p, const void* dout, const float* dht, char* ws, hipStream_t st) {
  float *ends = (float*)(ws + p.end_off), *adj = (float*)(ws + p.adj_off);
  double* sums = (double*)(ws + p.sum_off);
  int* kinds = (int*)(ws + p.kind_off);
  const unsigned sides = BACK ? 2 : 1;
  constexpr int ROWS = BACK ? DV : DK, COLS = BACK ? DK : DV;
  const hipError_t e = launch_kernel(linear_states<T, ROWS, COLS, BACK>, dim3((unsigned)linear_groups(p, a.H), sides),
                                     dim3(kThreads<COLS>), st, a, (const T*)dout, dht, ends, adj, sums, kinds);
  if (e != hipSuccess) return (int)e;
  const int64_t quads = DK * DV / 4;
  return (int)launch_kernel(linear_chain, dim3((unsigned)(a.H * quads / 256), sides), dim3(256), st, a.H, quads,
                            (int)p.n_slots, ends, adj, sums, kinds);
}

}  // namespace

int launch_linear_forward(int is_bf16, const LinearArgs& a, const LinearPlan& p, void* o, float* ht, void* ws,
                          void* stream) {
  const hipStream_t st = (hipStream_t)stream;
  return dispatch(is_bf16, a, [&](auto t, auto dims) {
    typedef decltype(t) T;
    if (p.carry) {
      const int e = states<T, dims.DK, dims.DV, false>(a, p, nullptr, nullptr, (char*)ws, st);
      if (e != 0) return e;
    }
    return (int)launch_kernel(linear_forward<T, dims.DK, dims.DV>, dim3((unsigned)linear_groups(p, a.H)),
                              dim3(kThreads<dims.DV>), st, a, (const float*)((char*)ws + p.end_off), (T*)o, ht);
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
      const int e = states<T, dims.DK, dims.DV, true>(a, p, g.dout, g.dht, w, st);
      if (e != 0) return e;
    }
    const LinearWork x{(float*)(w + p.end_off),    (float*)(w + p.adj_off),     (float*)(w + p.dot_q_off),
                       (float*)(w + p.dot_k_off),  (float*)(w + p.slot_dot_off), (float*)(w + p.seq_dot_off),
                       (float*)(w + p.dq_off),     (float*)(w + p.dk_off)};
    const unsigned groups = (unsigned)linear_groups(p, a.H);
    hipError_t e;
    if constexpr (dims.DK == dims.DV) {
      e = launch_kernel(linear_backward<T, dims.DK, dims.DV, kDq, 3>, dim3(3 * groups), dim3(kThreads<dims.DK>), st, a, g,
                        x);
    } else {
      e = launch_kernel(linear_backward<T, dims.DK, dims.DV, kDq, 2>, dim3(2 * groups), dim3(kThreads<dims.DK>), st, a, g,
                        x);
      if (e == hipSuccess)
        e = launch_kernel(linear_backward<T, dims.DK, dims.DV, kDv, 1>, dim3(groups), dim3(kThreads<dims.DV>), st, a, g,
                          x);
    }
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
