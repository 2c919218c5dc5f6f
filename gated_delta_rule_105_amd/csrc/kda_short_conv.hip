// Short causal convolution for gfx950: forward, one-token step and backward.
//
// With xe a sequence preceded by its initial state's W - 1 inputs and w[j]
// the taps of a channel (the last one meets the token itself):
//   u_t = bias + sum_j w[j] xe[t + j],    y = u  or  u sigmoid(u)
// and backward, with du = dy act'(u) (zero outside the sequence):
//   dx_s = sum_j w[j] du[s + W - 1 - j],  dw[j] = sum_t du_t xe[t + j],
//   dbias = sum_t du_t.
// All of it is bound by memory: a token-channel is read once and written
// once (two reads in the backward pass) for some 2 W + 8 operations.
// Measured: forward 4096 tokens of 6144 channels, bf16, 20.5 us (100.8 MB,
// 4.9 TB/s, what a large copy reaches); 5003 packed tokens of 1011 channels,
// fp32, 10.2 us (4.0 TB/s: some 1300 waves, one batch each); one token for
// 256 sequences of 6144 channels 6.4 us (3.9 TB/s, one load's latency and the
// launch; 8.5 between calls that follow one another, which is the host's);
// backward 2 x 4096 tokens of 4096 channels, bf16, 46 us and 4.6 for
// the parameters' sums (201.5 MB necessary, 224 moved: batches that run past
// a tile are read twice).
//
// A lane owns one vector of channels (16 bytes forward, 4 channels backward)
// and walks a tile of tokens with the last W - 1 inputs in registers, so an
// input is loaded once per tile and the window costs W - 1 extra rows a
// tile.  Rows come kConvBatch at a time, the next batch's loads issued before
// this one is used.  Every wave's token range is uniform: where its sequences
// begin and end is scalar control flow.  A last vector that would pass the end
// of the row is moved back to end with it; its channels overlap the
// neighbour's and both write the same values.  The step, which updates in
// place, takes single channels.
#include "kda_layer_device.h"

namespace kda {

namespace {

// first channel of a lane's vector
template <int V>
__device__ __forceinline__ int channel_of(int vec, int D, bool* active) {
  const int c = vec * V;
  *active = c < D;
  return c + V <= D ? c : D - V;
}

template <int V, int W>
__device__ __forceinline__ void load_taps(const float* __restrict__ w, const float* __restrict__ bias, int c,
                                          float (&taps)[W][V], float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    b[i] = bias ? bias[c + i] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) taps[j][i] = w[(int64_t)(c + i) * W + j];
  }
}

// row r of a sequence that starts at token lo, preceded by its initial state (r < 0: the state)
template <typename T, int V, int W>
__device__ __forceinline__ void load_row(const T* __restrict__ x, int64_t ld, const T* __restrict__ init, int D, int s,
                                         int lo, int r, int c, float (&v)[V]) {
  if (r >= 0) {
    load_vec<T, V>(x + (int64_t)(lo + r) * ld + c, v);
  } else if (init) {
    load_vec<T, V>(init + ((int64_t)s * (W - 1) + (W - 1) + r) * D + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.f;
  }
}

// Rows t .. t + kConvBatch - 1 of an array as they come from memory (row
// `last` for those past it): one scalar address each, and the lane's offset.
template <typename T, int V>
struct Batch {
  typename Pack<T, V>::type r[kConvBatch];
  __device__ __forceinline__ void load(const T* __restrict__ x, int64_t ld, int c, int t, int last) {
#pragma unroll
    for (int k = 0; k < kConvBatch; ++k) {
      const T* row = x + (int64_t)(t + k < last ? t + k : last) * ld;
      r[k] = *(const typename Pack<T, V>::type*)((const char*)row + (uint32_t)c * (uint32_t)sizeof(T));
    }
  }
  __device__ __forceinline__ float get(int k, int i) const {
    if constexpr (V == 1) return Elem<T>::to_f32(r[k]);
    else return Elem<T>::to_f32(r[k][i]);
  }
};

template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(256) conv_forward(const ConvArgs a, T* __restrict__ y, T* __restrict__ fin) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  bool active;
  const int c = channel_of<V>(blockIdx.y * 64 + lane, a.D, &active);
  if (!active) return;
  const T* __restrict__ x = (const T*)a.x;
  const T* __restrict__ init = (const T*)a.init;
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  if (blockIdx.x >= a.n_part) {  // one row of one sequence's final state per wave
    const int64_t item = (blockIdx.x - a.n_part) * kConvWaves + wave;
    if (item >= (int64_t)a.n_seqs * (W - 1)) return;
    const int s = (int)(item / (W - 1)), p = (int)(item % (W - 1));
    const int lo = (int)seqs.start(s), len = (int)seqs.end(s) - lo;
    float v[V];
    load_row<T, V, W>(x, a.ld, init, a.D, s, lo, len - (W - 1) + p, c, v);
    store_vec<T, V>(fin + item * a.D + c, v);
    return;
  }
  const int64_t begin = ((int64_t)blockIdx.x * kConvWaves + wave) * a.tile;
  if (begin >= a.tokens) return;
  int t = (int)begin;
  const int t1 = (int)(begin + a.tile < a.tokens ? begin + a.tile : a.tokens);
  float taps[W][V], b[V];
  load_taps<V, W>(a.w, a.bias, c, taps, b);
  int s = uniform(seqs.from(begin + 1)) - 1;  // the last sequence that starts at t or before
  if (s < 0) s = 0;
  for (; s < a.n_seqs && t < t1; ++s) {
    const int lo = uniform((int)seqs.start(s)), hi = uniform((int)seqs.end(s));
    if (hi <= t) continue;
    if (t < lo) t = lo;
    const int e = hi < t1 ? hi : t1;
    Batch<T, V> next;
    next.load(x, a.ld, c, t, e - 1);
    float win[W - 1][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<T, V, W>(x, a.ld, init, a.D, s, lo, t - lo - (W - 1) + j, c, win[j]);
    for (; t < e; t += kConvBatch) {
      const Batch<T, V> r = next;
      if (t + kConvBatch < e) next.load(x, a.ld, c, t + kConvBatch, e - 1);
#pragma unroll
      for (int k = 0; k < kConvBatch; ++k) {
        float u[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float v = r.get(k, i);
          u[i] = b[i];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) u[i] += taps[j][i] * win[j][i];
          u[i] += taps[W - 1][i] * v;
          if (SILU) u[i] *= sigmoid(u[i]);
#pragma unroll
          for (int j = 0; j + 1 < W - 1; ++j) win[j][i] = win[j + 1][i];
          win[W - 2][i] = v;
        }
        if (t + k < e) store_vec<T, V>(y + (int64_t)(t + k) * a.D + c, u);
      }
    }
    t = e;
  }
}

// One token: a lane owns a channel of kStepSeqs sequences, n_far apart, so that
// the taps are loaded once for all of them and the rows of all are under way
// together (4096 sequences of 6144 channels, 4 taps: bf16 77 us with two, 91 with
// one, 77 with four; fp32 142, 136, 149).  Vectors of channels, 16 bytes a lane,
// measured 105 and 148 us there, 16.5 against 17.6 with 2 taps in fp32 for 1024
// sequences, and 8.6 against 6.4 for 256 sequences in bf16.
constexpr int kStepSeqs = 2;
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(256) conv_step(const ConvArgs a, T* __restrict__ state, T* __restrict__ y, int n_far) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  const int n0 = (int)(id / (uint32_t)a.D), c = (int)(id - (uint32_t)n0 * (uint32_t)a.D);
  if (n0 >= n_far) return;
  const T* __restrict__ x = (const T*)a.x;
  T rows[kStepSeqs][W];
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q) {
    const int64_t n = n0 + q * n_far < a.tokens ? n0 + q * n_far : n0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) rows[q][j] = state[(n * (W - 1) + j) * a.D + c];
    rows[q][W - 1] = x[n * a.ld + c];
  }
  float taps[W][1], b[1];
  load_taps<1, W>(a.w, a.bias, c, taps, b);
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q) {
    const int64_t n = n0 + q * n_far;
    if (n >= a.tokens) break;
    float u = b[0];
#pragma unroll
    for (int j = 0; j < W; ++j) u += taps[j][0] * Elem<T>::to_f32(rows[q][j]);
    if (SILU) u *= sigmoid(u);
    // the inputs move up a row as they are
#pragma unroll
    for (int j = 0; j < W - 1; ++j) state[(n * (W - 1) + j) * a.D + c] = rows[q][j + 1];
    y[n * a.D + c] = Elem<T>::from_f32(u);
  }
}

// du from dy and the pre-activation
template <bool SILU>
__device__ __forceinline__ float act_grad(float dy, float u) {
  if (!SILU) return dy;
  const float g = sigmoid(u);
  return dy * (g * (1.f + u * (1.f - g)));
}

template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(256)
conv_backward(const ConvArgs a, const T* __restrict__ dy, const T* __restrict__ dfin, T* __restrict__ dx,
              T* __restrict__ dinit, float* __restrict__ part) {
  __shared__ float sums[kConvWaves][W + 1][V][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  bool active;
  const int c = channel_of<V>(blockIdx.y * 64 + lane, a.D, &active);
  const T* __restrict__ x = (const T*)a.x;
  const T* __restrict__ init = (const T*)a.init;
  const Seqs seqs{a.cu, a.n_seqs, a.T, a.tokens};
  float taps[W][V], b[V];
  if (blockIdx.x >= a.n_part) {  // one row of one initial state's gradient per wave
    const int64_t item = (blockIdx.x - a.n_part) * kConvWaves + wave;
    if (!active || item >= (int64_t)a.n_seqs * (W - 1)) return;
    const int s = (int)(item / (W - 1)), p = (int)(item % (W - 1));
    const int lo = (int)seqs.start(s), len = (int)seqs.end(s) - lo;
    load_taps<V, W>(a.w, a.bias, c, taps, b);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    if (dfin && p >= len) load_vec<T, V>(dfin + ((int64_t)s * (W - 1) + p - len) * a.D + c, acc);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {  // row p is tap j of token p - j
      if (p - j < 0 || p - j >= len) continue;
      float u[V], g[V];
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] = b[i];
#pragma unroll
      for (int m = 0; m < W; ++m) {
        float v[V];
        load_row<T, V, W>(x, a.ld, init, a.D, s, lo, p - j - (W - 1) + m, c, v);
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] += taps[m][i] * v[i];
      }
      load_vec<T, V>(dy + (int64_t)(lo + p - j) * a.D + c, g);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += taps[j][i] * act_grad<SILU>(g[i], u[i]);
    }
    store_vec<T, V>(dinit + item * a.D + c, acc);
    return;
  }
  float dw[W][V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
  }
  const int64_t begin = ((int64_t)blockIdx.x * kConvWaves + wave) * a.tile;
  if (active && begin < a.tokens) {
    int t = (int)begin;
    const int t1 = (int)(begin + a.tile < a.tokens ? begin + a.tile : a.tokens);
    load_taps<V, W>(a.w, a.bias, c, taps, b);
    int s = uniform(seqs.from(begin + 1)) - 1;
    if (s < 0) s = 0;
    for (; s < a.n_seqs && t < t1; ++s) {
      const int lo = uniform((int)seqs.start(s)), hi = uniform((int)seqs.end(s));
      if (hi <= t) continue;
      if (t < lo) t = lo;
      // tokens [t, e) of this sequence: their dx needs du up to W - 1 tokens further
      const int first = t, e = hi < t1 ? hi : t1, last = e + W - 1;
      Batch<T, V> nx, ng;
      nx.load(x, a.ld, c, t, hi - 1);
      ng.load(dy, a.D, c, t, hi - 1);
      float win[W - 1][V], du[W - 1][V];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        load_row<T, V, W>(x, a.ld, init, a.D, s, lo, t - lo - (W - 1) + j, c, win[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) du[j][i] = 0.f;
      }
      // one batch; INSIDE: all of its tokens, and those whose dx they complete, are this wave's own
      auto batch = [&](const Batch<T, V>& rx, const Batch<T, V>& rg, auto inside) {
        constexpr bool INSIDE = decltype(inside)::value;
#pragma unroll
        for (int k = 0; k < kConvBatch; ++k) {
          const bool in_seq = INSIDE || t + k < hi, own = INSIDE || t + k < e;
          float out[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float v = rx.get(k, i);
            float u = b[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) u += taps[j][i] * win[j][i];
            u += taps[W - 1][i] * v;
            const float d = in_seq ? act_grad<SILU>(rg.get(k, i), u) : 0.f;
            if (own) {
              db[i] += d;
#pragma unroll
              for (int j = 0; j < W - 1; ++j) dw[j][i] += d * win[j][i];
              dw[W - 1][i] += d * v;
            }
            // dx of token t + k - (W - 1)
            out[i] = taps[0][i] * d;
#pragma unroll
            for (int j = 1; j < W; ++j) out[i] += taps[j][i] * du[W - 1 - j][i];
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) {
              win[j][i] = win[j + 1][i];
              du[j][i] = du[j + 1][i];
            }
            win[W - 2][i] = v;
            du[W - 2][i] = d;
          }
          const int at = t + k - (W - 1);
          if (INSIDE || (at >= first && at < e)) {
            if (!INSIDE && dfin && at >= hi - (W - 1)) {
              float f[V];
              load_vec<T, V>(dfin + ((int64_t)s * (W - 1) + at - (hi - (W - 1))) * a.D + c, f);
#pragma unroll
              for (int i = 0; i < V; ++i) out[i] += f[i];
            }
            store_vec<T, V>((T*)((char*)(dx + (int64_t)at * a.D) + (uint32_t)c * (uint32_t)sizeof(T)), out);
          }
        }
      };
      for (; t < last; t += kConvBatch) {
        const Batch<T, V> rx = nx, rg = ng;
        if (t + kConvBatch < last) {
          nx.load(x, a.ld, c, t + kConvBatch, hi - 1);
          ng.load(dy, a.D, c, t + kConvBatch, hi - 1);
        }
        if (t - (W - 1) >= first && t + kConvBatch <= e)
          batch(rx, rg, std::true_type{});
        else
          batch(rx, rg, std::false_type{});
      }
      t = e;
    }
  }
  // the workgroup's partial sums, waves in order
#pragma unroll
  for (int i = 0; i < V; ++i) {
    sums[wave][W][i][lane] = db[i];
#pragma unroll
    for (int j = 0; j < W; ++j) sums[wave][j][i][lane] = dw[j][i];
  }
  __syncthreads();
  if (!active) return;
  float* __restrict__ row = part + (int64_t)blockIdx.x * (W + 1) * a.D;
  for (int q = wave; q < (W + 1) * V; q += kConvWaves) {
    const int j = q / V, i = q % V;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kConvWaves; ++w) v += sums[w][j][i][lane];
    row[(int64_t)j * a.D + c + i] = v;
  }
}

// dweight [D, W] and dbias [D] from the rows of partial sums: 64 columns a
// workgroup, the rows dealt to its 16 waves and their sums added in order.
__global__ void __launch_bounds__(1024) conv_params(const float* __restrict__ part, int64_t n_part, int D, int W,
                                                    float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t cols = (int64_t)(W + 1) * D, col = (int64_t)blockIdx.x * 64 + lane;
  float v = 0.f;
  if (col < cols)
    for (int64_t r = wave; r < n_part; r += 16) v += part[r * cols + col];
  sums[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || col >= cols) return;
  v = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) v += sums[w][lane];
  const int j = (int)(col / D), c = (int)(col % D);
  if (j < W)
    dw[(int64_t)c * W + j] = v;
  else if (db)
    db[c] = v;
}

template <typename T, int V, int W, bool SILU>
int forward_t(const ConvArgs& a, void* y, void* fin, hipStream_t st) {
  const int64_t states = fin ? ceil_div((int64_t)a.n_seqs * (W - 1), kConvWaves) : 0;
  const dim3 grid((unsigned)(a.n_part + states), (unsigned)ceil_div(ceil_div(a.D, V), 64));
  return (int)launch_kernel(conv_forward<T, V, W, SILU>, grid, dim3(256), st, a, (T*)y, (T*)fin);
}
template <typename T, int W, bool SILU>
int step_t(const ConvArgs& a, void* state, void* y, hipStream_t st) {
  const int64_t n_far = ceil_div(a.tokens, kStepSeqs), groups = ceil_div(n_far * a.D, 256);
  return (int)launch_kernel(conv_step<T, W, SILU>, dim3((unsigned)groups), dim3(256), st, a, (T*)state, (T*)y,
                            (int)n_far);
}
template <typename T, int V, int W, bool SILU>
int backward_t(const ConvArgs& a, const void* dy, const void* dfin, void* dx, float* dw, float* db, void* dinit,
               float* part, hipStream_t st) {
  const int64_t states = dinit ? ceil_div((int64_t)a.n_seqs * (W - 1), kConvWaves) : 0;
  const dim3 grid((unsigned)(a.n_part + states), (unsigned)ceil_div(ceil_div(a.D, V), 64));
  if (grid.x > 0) {
    const hipError_t e = launch_kernel(conv_backward<T, V, W, SILU>, grid, dim3(256), st, a, (const T*)dy,
                                       (const T*)dfin, (T*)dx, (T*)dinit, part);
    if (e != hipSuccess) return (int)e;
  }
  return (int)launch_kernel(conv_params, dim3((unsigned)ceil_div((int64_t)(W + 1) * a.D, 64)), dim3(1024), st, part,
                            a.n_part, a.D, W, dw, db);
}

// Chooses the instance: type, taps, activation, and vectors of VEC channels
// or single ones when a row has fewer than VEC.
template <typename T, int VEC, typename F>
int dispatch_t(int width, int silu, int D, F&& f) {
  auto w = [&](auto vec) {
    auto act = [&](auto taps) {
      return silu ? f(T{}, vec, taps, std::true_type{}) : f(T{}, vec, taps, std::false_type{});
    };
    return width == 2   ? act(std::integral_constant<int, 2>{})
           : width == 3 ? act(std::integral_constant<int, 3>{})
                        : act(std::integral_constant<int, 4>{});
  };
  return D < VEC ? w(std::integral_constant<int, 1>{}) : w(std::integral_constant<int, VEC>{});
}
template <int VEC_BF16, int VEC_F32, typename F>
int dispatch(int is_bf16, int width, int silu, int D, F&& f) {
  return is_bf16 ? dispatch_t<bf16_t, VEC_BF16>(width, silu, D, f) : dispatch_t<float, VEC_F32>(width, silu, D, f);
}

}  // namespace

int launch_conv_forward(int is_bf16, int width, int silu, const ConvArgs& a, void* y, void* fin, void* stream) {
  return dispatch<conv_vec(true, false), conv_vec(false, false)>(is_bf16, width, silu, a.D, [&](auto t, auto vec, auto taps, auto act) {
    return forward_t<decltype(t), vec.value, taps.value, act.value>(a, y, fin, (hipStream_t)stream);
  });
}
int launch_conv_step(int is_bf16, int width, int silu, const ConvArgs& a, void* state, void* y, void* stream) {
  return dispatch<1, 1>(is_bf16, width, silu, a.D, [&](auto t, auto, auto taps, auto act) {
    return step_t<decltype(t), taps.value, act.value>(a, state, y, (hipStream_t)stream);
  });
}
int launch_conv_backward(int is_bf16, int width, int silu, const ConvArgs& a, const void* dy, const void* dfin,
                         void* dx, float* dw, float* db, void* dinit, float* part, void* stream) {
  return dispatch<conv_vec(true, true), conv_vec(false, true)>(is_bf16, width, silu, a.D, [&](auto t, auto vec, auto taps, auto act) {
    return backward_t<decltype(t), vec.value, taps.value, act.value>(a, dy, dfin, dx, dw, db, dinit, part,
                                                                     (hipStream_t)stream);
  });
}

}  // namespace kda
