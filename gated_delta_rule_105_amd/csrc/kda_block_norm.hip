// The norms at a block's end and their gradients, for gfx950: the heads' norm
// with the output gate, and the residual sum with the norm before the next
// block.
//
//   gated:     y = n w a(z),  n = x r,  r = (mean x^2 + eps)^-1/2,  a = sigmoid or SiLU
//              dn = dy w a,  dx = r (dn - n mean(n dn)),  dz = dy n w a'(z),  dw = sum dy n a
//   residual:  t = res + scale c x,  y = n w with n the same of t
//              dt = dtotal + r (dn - n mean(n dn)),  dn = dy w,  dx = scale c dt,
//              dw = sum dy n,  dc = sum scale dt x
// with mean(n dn) = r mean(x dn), so that both sums of a row are taken of its
// inputs at once.  All of it is bound by memory: every element is read once
// and written once, a row stays in registers between its sums and its outputs.
// Measured, bf16, on inputs that change from call to call (a large copy reaches
// 5.13 TB/s): forward 65536 heads of 128, gated, 50.3 MB, 10.0 us (with hits in
// the last-level cache); 4096 tokens of 4096 channels, residual, 134 MB, 23.0 us
// (5.8 TB/s, part of it from the cache); backward 131072 heads of 128, gated, 168
// MB, 37.9 us (4.4 TB/s); 8192 tokens of 2048 channels, residual, 201 MB, 45 us
// (4.5 TB/s); on the same inputs again 32 and 37 us.
#include "kda_block.h"
#include "kda_layer_device.h"

namespace kda {
namespace {

constexpr int kThreads = kBlockNormThreads, kWaves = kThreads / 64;

// V channels of each of N loads, LANES lanes apart.
template <int V, int N>
struct Row {
  float v[N][V];
};
template <typename T, int V, int N>
struct RawRow {
  typename Pack<T, V>::type v[N];
  template <int LANES>
  __device__ __forceinline__ void load(const T* __restrict__ p, int sub, int D) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * LANES + sub) * V;
      v[i] = *(const typename Pack<T, V>::type*)(p + (c < D ? c : 0));
    }
  }
  template <int LANES>
  __device__ __forceinline__ Row<V, N> get(int sub, int D) const {
    Row<V, N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool there = (i * LANES + sub) * V < D;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float x;
        if constexpr (V == 1) x = Elem<T>::to_f32(v[i]);
        else x = Elem<T>::to_f32(v[i][e]);
        r.v[i][e] = there ? x : 0.f;
      }
    }
    return r;
  }
};
template <typename T, int LANES, int V, int N>
__device__ __forceinline__ void store_row(T* __restrict__ p, int sub, int D, const Row<V, N>& r) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * LANES + sub) * V;
    if (c < D) store_vec<T, V>(p + c, r.v[i]);
  }
}
// a parameter's row; ones without
template <int LANES, int V, int N>
__device__ __forceinline__ Row<V, N> param_row(const float* __restrict__ p, int sub, int D) {
  Row<V, N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * LANES + sub) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) r.v[i][e] = 1.f;
    if (p && c < D) load_vec<float, V>(p + c, r.v[i]);
  }
  return r;
}

// sums of a row's lanes, in each of them
template <int LANES, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float (*lds)[kWaves]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = row_sum(v[k]);
    if constexpr (LANES >= 32) v[k] += __shfl_xor(v[k], 16, 64);
    if constexpr (LANES >= 64) v[k] += __shfl_xor(v[k], 32, 64);
  }
  if constexpr (LANES == kThreads) {
    __syncthreads();  // the row before is read
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) lds[k][threadIdx.x >> 6] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = (lds[k][0] + lds[k][1]) + (lds[k][2] + lds[k][3]);
  }
}

__device__ __forceinline__ float inv_norm(float ss, int D, float eps) { return 1.f / sqrtf(ss / (float)D + eps); }

// e^x.  x in units of a factor 2 is a rounded product; without what it left
// out the result is |x| roundings off (3.7e-6 of a gate at -86).  For fp32 that
// is a factor of its own, and the result within 3 times 2^-24.  bf16 rounds
// outputs a thousand times more coarsely: no more of them are off the rounding
// of their value either way (9e-6), and the factor's instructions took 10.6
// against 10.1 us for 65536 heads of 128 channels, 34.1 against 32.3 backward.
template <typename T>
__device__ __forceinline__ float exp_of(float x) {
  constexpr float kLn2Rest = -1.9046542e-9f;  // ln 2 - kLn2
  const float hi = x * kLog2e, e = exp2_fast(hi);
  if constexpr (sizeof(T) == 2) return e;
  const float rest = __builtin_fmaf(-hi, kLn2Rest, __builtin_fmaf(-hi, kLn2, x));
  // past what fp32 holds there is no rest, only 0 or an infinity
  return __builtin_fabsf(x) < 87.f ? __builtin_fmaf(e, rest, e) : e;
}

// a(z) and a'(z).  Of the sigmoid and its complement the smaller is e^-|z|
// times the larger, so neither is a difference.
template <typename T> struct Gate {
  float a, slope;
  __device__ __forceinline__ Gate(float z, int silu) {
    const float e = exp_of<T>(-__builtin_fabsf(z)), big = __builtin_amdgcn_rcpf(1.f + e), small = e * big;
    const float s = z < 0.f ? small : big, c = z < 0.f ? big : small;
    a = silu ? z * s : s;
    slope = silu ? s * (1.f + z * c) : s * c;
  }
  // a(z) alone: below -88 the sigmoid is 0, within what fp32 holds as a normal number
  __device__ __forceinline__ static float value(float z, int silu) {
    const float s = __builtin_amdgcn_rcpf(1.f + exp_of<T>(-z));
    return silu ? z * s : s;
  }
};

__device__ __forceinline__ int64_t row_at(int row, int H, int D, int64_t ld) {
  if (H == 1) return row * ld;
  const int tok = row / H;
  return tok * ld + (int64_t)(row - tok * H) * D;
}

// Forward.  A group of LANES lanes takes a row (four, with their loads
// together, took 82 us against 71 for 524288 heads of 128 channels in bf16).
template <typename T, int V, int LANES, int N, bool GATED>
__global__ void __launch_bounds__(kThreads)
block_forward(const BlockNormArgs a, T* __restrict__ y, T* __restrict__ total) {
  constexpr int G = kThreads / LANES;
  __shared__ float lds[1][kWaves];
  const int sub = threadIdx.x % LANES, last = (int)a.rows - 1;
  const int64_t at = (int64_t)blockIdx.x * G + threadIdx.x / LANES, flat = at * a.D;
  const int row = at < last ? (int)at : last;
  RawRow<T, V, N> rx, rz;
  rx.template load<LANES>((const T*)a.x + row_at(row, a.H, a.D, a.ld_x), sub, a.D);
  rz.template load<LANES>((const T*)a.z + row_at(row, a.H, a.D, a.ld_z), sub, a.D);
  const Row<V, N> w = param_row<LANES, V, N>(a.w, sub, a.D);
  const Row<V, N> c = param_row<LANES, V, N>(GATED ? nullptr : a.channels, sub, a.D);
  Row<V, N> x = rx.template get<LANES>(sub, a.D);
  const Row<V, N> z = rz.template get<LANES>(sub, a.D);
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (!GATED) x.v[i][e] = z.v[i][e] + a.scale * c.v[i][e] * x.v[i][e];
      ss[0] += x.v[i][e] * x.v[i][e];
    }
  row_sums<LANES>(ss, lds);
  const float r = inv_norm(ss[0], a.D, a.eps);
  Row<V, N> o;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float n = x.v[i][e] * r * w.v[i][e];
      o.v[i][e] = GATED ? n * Gate<T>::value(z.v[i][e], a.act) : n;
    }
  if (at > last) return;
  store_row<T, LANES>(y + flat, sub, a.D, o);
  if (!GATED) store_row<T, LANES>(total + flat, sub, a.D, x);
}

// Backward.  Each group of lanes takes every (gridDim.x G)-th row and keeps
// the parameters' sums of its channels; the workgroup leaves one row of
// partial sums for each parameter.
template <typename T, int V, int LANES, int N, bool GATED>
__global__ void __launch_bounds__(kThreads)
block_backward(const BlockNormArgs a, const T* __restrict__ dy, const T* __restrict__ dtotal, T* __restrict__ dx,
               T* __restrict__ dz, float* __restrict__ part, int want_w, int want_c) {
  constexpr int G = kThreads / LANES;
  __shared__ float lds[2][kWaves];
  __shared__ float sums[G > 1 ? G : 1][LANES * V + 1];
  const int sub = threadIdx.x % LANES, group = threadIdx.x / LANES, rows = (int)a.rows;
  const Row<V, N> w = param_row<LANES, V, N>(a.w, sub, a.D);
  const Row<V, N> c = param_row<LANES, V, N>(GATED ? nullptr : a.channels, sub, a.D);
  Row<V, N> dw, dc;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) dw.v[i][e] = dc.v[i][e] = 0.f;
  const bool with_x = GATED || want_c;
  struct Rows {
    RawRow<T, V, N> x, z, y, t;
  };
  auto load = [&](Rows& r, int64_t at) {
    const int row = at < rows ? (int)at : rows - 1;
    const int64_t flat = (int64_t)row * a.D;
    r.z.template load<LANES>((const T*)a.z + row_at(row, a.H, a.D, a.ld_z), sub, a.D);
    r.y.template load<LANES>(dy + flat, sub, a.D);
    if (with_x) r.x.template load<LANES>((const T*)a.x + row_at(row, a.H, a.D, a.ld_x), sub, a.D);
    if (!GATED && dtotal) r.t.template load<LANES>(dtotal + flat, sub, a.D);
  };
  // Rows of one load a lane are loaded one ahead: 41.2 against 43.4 us for the
  // gated norm of 131072 heads of 128 channels; of two loads and more, 4096
  // channels took 87.1 us with it and 84.6 without.
  constexpr bool AHEAD = N == 1;
  Rows next;
  if (AHEAD) load(next, (int64_t)blockIdx.x * G + group);
  // every group goes round as often as the first, so that all meet at the sums' barriers
  for (int64_t base = (int64_t)blockIdx.x * G; base < rows; base += (int64_t)gridDim.x * G) {
    const bool there = base + group < rows;
    const int64_t flat = (there ? base + group : rows - 1) * a.D;
    if (!AHEAD) load(next, base + group);
    const auto [rx, rz, ry, rt] = next;
    if (AHEAD) load(next, base + (int64_t)gridDim.x * G + group);
    const Row<V, N> z = rz.template get<LANES>(sub, a.D), g = ry.template get<LANES>(sub, a.D);
    Row<V, N> x, dn;
    if (GATED) x = rx.template get<LANES>(sub, a.D);
    else x = z;  // the sum itself
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        dn.v[i][e] = g.v[i][e] * w.v[i][e];
        if (GATED) dn.v[i][e] *= Gate<T>(z.v[i][e], a.act).a;
        s[0] += x.v[i][e] * x.v[i][e];
        s[1] += x.v[i][e] * dn.v[i][e];
      }
    row_sums<LANES>(s, lds);
    const float r = inv_norm(s[0], a.D, a.eps), back = s[1] / (float)a.D * r;
    Row<V, N> ox, oz;
    Row<V, N> t, xs;
    if (!GATED && dtotal) t = rt.template get<LANES>(sub, a.D);
    if (!GATED && want_c) xs = rx.template get<LANES>(sub, a.D);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float n = x.v[i][e] * r;
        float d = r * (dn.v[i][e] - n * back);
        float of_w = g.v[i][e] * n;
        if (GATED) {
          const Gate<T> gate(z.v[i][e], a.act);
          ox.v[i][e] = d;
          oz.v[i][e] = of_w * w.v[i][e] * gate.slope;
          of_w *= gate.a;
        } else {
          if (dtotal) d += t.v[i][e];
          oz.v[i][e] = d;
          ox.v[i][e] = a.scale * d * c.v[i][e];
          if (want_c) dc.v[i][e] += there ? a.scale * d * xs.v[i][e] : 0.f;
        }
        dw.v[i][e] += there ? of_w : 0.f;
      }
    if (!there) continue;
    if (dx) store_row<T, LANES>(dx + flat, sub, a.D, ox);
    store_row<T, LANES>(dz + flat, sub, a.D, oz);
  }
  // rows of partial sums
  auto leave = [&](const Row<V, N>& d, float* __restrict__ row) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (G == 1) {
        const int ch = (i * LANES + sub) * V;
        if (ch < a.D) store_vec<float, V>(row + ch, d.v[i]);
      } else {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) sums[group][sub * V + e] = d.v[i][e];
        __syncthreads();
        for (int x = threadIdx.x; x < LANES * V; x += kThreads) {
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < G; ++k) s += sums[k][x];
          if (i * LANES * V + x < a.D) row[i * LANES * V + x] = s;
        }
      }
    }
  };
  if (want_w) leave(dw, part + (int64_t)blockIdx.x * a.D);
  if (!GATED && want_c) leave(dc, part + (int64_t)(gridDim.x + blockIdx.x) * a.D);
}

// The parameters' gradients from the workgroups' rows: 64 channels a
// workgroup, rows dealt to 16 waves whose sums are added in order.
__global__ void __launch_bounds__(1024)
block_params(const float* __restrict__ part, int n_part, int D, float* __restrict__ dw, float* __restrict__ dc) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  float* out = blockIdx.y ? dc : dw;
  if (!out) return;
  const float* __restrict__ rows = part + (int64_t)blockIdx.y * n_part * D;
  float v = 0.f;
  if (c < D)
#pragma unroll 8
    for (int r = wave; r < n_part; r += 16) v += rows[(int64_t)r * D + c];
  sums[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || c >= D) return;
  v = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) v += sums[w][lane];
  out[c] = v;
}

template <int V_, int LANES_, int N_> struct Shape {
  static constexpr int V = V_, LANES = LANES_, N = N_;
};
// the shape that block_norm_shape chooses
template <typename F>
int dispatch(int is_bf16, int D, F&& f) {
  const RowShape s = block_norm_shape(D, is_bf16 ? 2 : 4);
  auto shape = [&](auto t, auto v) {
    constexpr int V = decltype(v)::value;
    if (s.lanes == 16) return f(t, Shape<V, 16, 1>{});
    if (s.lanes == 32) return f(t, Shape<V, 32, 1>{});
    if (s.lanes == 64) {
      return s.loads == 1 ? f(t, Shape<V, 64, 1>{}) : f(t, Shape<V, 64, 2>{});
    }
    if (s.loads == 1) return f(t, Shape<V, 256, 1>{});
    if (s.loads == 2) return f(t, Shape<V, 256, 2>{});
    if constexpr (V == 8) {
      return f(t, Shape<V, 256, 4>{});
    } else {
      if (s.loads == 4) return f(t, Shape<V, 256, 4>{});
      if constexpr (V == 4) return f(t, Shape<V, 256, 8>{});
      else return s.loads == 8 ? f(t, Shape<V, 256, 8>{}) : f(t, Shape<V, 256, 32>{});
    }
  };
  if (is_bf16) return s.vec > 1 ? shape(bf16_t{}, std::integral_constant<int, 8>{})
                                : shape(bf16_t{}, std::integral_constant<int, 1>{});
  return s.vec > 1 ? shape(float{}, std::integral_constant<int, 4>{}) : shape(float{}, std::integral_constant<int, 1>{});
}

template <bool GATED>
int forward(int is_bf16, const BlockNormArgs& a, void* y, void* total, hipStream_t st) {
  return dispatch(is_bf16, a.D, [&](auto t, auto s) {
    typedef decltype(t) T;
    return (int)launch_kernel(block_forward<T, s.V, s.LANES, s.N, GATED>,
                              dim3((unsigned)ceil_div(a.rows, kThreads / s.LANES)), dim3(kThreads), st, a, (T*)y,
                              (T*)total);
  });
}

template <bool GATED>
int backward(int is_bf16, const BlockNormArgs& a, const void* dy, const void* dtotal, void* dx, void* dz, float* dw,
             float* dc, float* part, hipStream_t st) {
  const int n_part = (int)block_norm_parts(a.rows, a.D, is_bf16 ? 2 : 4);
  if (n_part > 0) {
    const int e = dispatch(is_bf16, a.D, [&](auto t, auto s) {
      typedef decltype(t) T;
      return (int)launch_kernel(block_backward<T, s.V, s.LANES, s.N, GATED>, dim3((unsigned)n_part), dim3(kThreads), st,
                                a, (const T*)dy, (const T*)dtotal, (T*)dx, (T*)dz, part, dw != nullptr, dc != nullptr);
    });
    if (e != 0) return e;
  }
  if (!dw && !dc) return 0;
  return (int)launch_kernel(block_params, dim3((unsigned)ceil_div(a.D, 64), 2), dim3(1024), st, part, n_part, a.D, dw,
                            dc);
}

}  // namespace

int launch_gated_norm_forward(int is_bf16, const BlockNormArgs& a, void* y, void* stream) {
  return forward<true>(is_bf16, a, y, nullptr, (hipStream_t)stream);
}
int launch_gated_norm_backward(int is_bf16, const BlockNormArgs& a, const void* dy, void* dx, void* dz, float* dw,
                               float* part, void* stream) {
  return backward<true>(is_bf16, a, dy, nullptr, dx, dz, dw, nullptr, part, (hipStream_t)stream);
}
int launch_residual_norm_forward(int is_bf16, const BlockNormArgs& a, void* y, void* total, void* stream) {
  return forward<false>(is_bf16, a, y, total, (hipStream_t)stream);
}
int launch_residual_norm_backward(int is_bf16, const BlockNormArgs& a, const void* dy, const void* dtotal, void* dx,
                                  void* dres, float* dw, float* dchannels, float* part, void* stream) {
  return backward<false>(is_bf16, a, dy, dtotal, dx, dres, dw, dchannels, part, (hipStream_t)stream);
}

}  // namespace kda
