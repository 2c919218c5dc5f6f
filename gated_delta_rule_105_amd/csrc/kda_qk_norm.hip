// Norm of every query and key head with the position rotation in the same
// pass, and its gradient, for gfx950.
//
//   r = (f sum x^2 + eps)^-1/2   (f = 1: unit vectors, f = 1 / d: rms)
//   v = x r w,  pair i of v turned by the angle pos * inv_freq[i],  out = s v
// and backward, with g the upstream gradient times s turned back:
//   dw = sum g x r,  dx = r (g w - f x r sum(g w x r)).
// Both directions are bound by memory: every element is read once (twice
// backward) and written once.
//
// A head's d / 2 pairs are spread over LPH lanes, PV consecutive pairs a
// lane (16 bytes of bf16 when PV = 4), so one wave holds 64 / LPH heads and a
// sum over a head is a few exchanges between lanes.  The two channels of a
// rotated pair sit side by side or rot / 2 apart; either way a lane loads
// both, so the rotation needs no exchange.  A wave keeps the cosines and
// sines of a token while it goes through the token's heads: they are taken
// in revolutions, reduced in 64 bits, because fp32 would lose the angle of a
// far position (2^-24 of a million is 0.06 revolutions).
#include "kda_layer_device.h"

namespace kda {

namespace {

// Pairs a head has per lane: chunks of PV pairs, NC of them LPH lanes apart.
template <int PV, int NC>
struct HeadPairs {
  float a[NC][PV], b[NC][PV];
};

// Channel of pair p's first element, and the distance to its second.
struct PairMap {
  int half;  // rot / 2 when the rotated pairs are rot / 2 apart, else 0
  __device__ __forceinline__ int first(int p) const { return p < half ? p : 2 * p; }
  __device__ __forceinline__ int gap(int p) const { return p < half ? half : 1; }
};

template <typename T, int PV, int NC, int LPH>
__device__ __forceinline__ void load_pairs(const T* __restrict__ x, int sub, int n_pairs, const PairMap& m,
                                           HeadPairs<PV, NC>& v) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int p = (i * LPH + sub) * PV;
#pragma unroll
    for (int e = 0; e < PV; ++e) v.a[i][e] = v.b[i][e] = 0.f;
    if (p >= n_pairs) continue;
    if (p < m.half) {
      load_vec<T, PV>(x + p, v.a[i]);
      load_vec<T, PV>(x + p + m.half, v.b[i]);
    } else {
      float t[2 * PV];
      load_vec<T, 2 * PV>(x + 2 * p, t);
#pragma unroll
      for (int e = 0; e < PV; ++e) {
        v.a[i][e] = t[2 * e];
        v.b[i][e] = t[2 * e + 1];
      }
    }
  }
}

template <typename T, int PV, int NC, int LPH>
__device__ __forceinline__ void store_pairs(T* __restrict__ x, int sub, int n_pairs, const PairMap& m,
                                            const HeadPairs<PV, NC>& v) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int p = (i * LPH + sub) * PV;
    if (p >= n_pairs) continue;
    if (p < m.half) {
      store_vec<T, PV>(x + p, v.a[i]);
      store_vec<T, PV>(x + p + m.half, v.b[i]);
    } else {
      float t[2 * PV];
#pragma unroll
      for (int e = 0; e < PV; ++e) {
        t[2 * e] = v.a[i][e];
        t[2 * e + 1] = v.b[i][e];
      }
      store_vec<T, 2 * PV>(x + 2 * p, t);
    }
  }
}

// sum over the LPH lanes of a head, in each of them
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
  if constexpr (LPH >= 2) v += dpp<kPairSwap>(v);
  if constexpr (LPH >= 4) v += dpp<kQuadMirror>(v);
  if constexpr (LPH >= 8) v += dpp<kHalfMirror>(v);
  if constexpr (LPH >= 16) v += dpp<kRowMirror>(v);
  if constexpr (LPH >= 32) v += __shfl_xor(v, 16, 64);
  if constexpr (LPH >= 64) v += __shfl_xor(v, 32, 64);
  return v;
}

// cosines and sines of a token's pairs; 1 and 0 past the rotated ones
template <int PV, int NC, int LPH>
__device__ __forceinline__ void load_turns(int pos, const float* __restrict__ freq, int sub, int n_rot,
                                           HeadPairs<PV, NC>& cs) {
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < PV; ++e) {
      const int p = (i * LPH + sub) * PV + e;
      cs.a[i][e] = 1.f;
      cs.b[i][e] = 0.f;
      if (p < n_rot) {
        const double turns = (double)pos * (double)freq[p] * 0.15915494309189535;
        const float half_turns = (float)(2.0 * (turns - __builtin_rint(turns)));
        sincospif(half_turns, &cs.b[i][e], &cs.a[i][e]);
      }
    }
}

template <int PV, int NC>
__device__ __forceinline__ void load_weight(const float* __restrict__ w, int sub, int lph, int n_pairs,
                                            const PairMap& m, HeadPairs<PV, NC>& v) {
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < PV; ++e) {
      const int p = (i * lph + sub) * PV + e;
      const bool there = w && p < n_pairs;
      v.a[i][e] = there ? w[m.first(p)] : 1.f;
      v.b[i][e] = there ? w[m.first(p) + m.gap(p)] : 1.f;
    }
}

// 1 / sqrt, rounded as the division and the square root are (the hardware's
// approximation is a unit in the last place off)
__device__ __forceinline__ float inv_norm(float ss, float f, float eps) { return 1.f / sqrtf(f * ss + eps); }

// Forward: a wave takes `steps` groups of 64 / LPH heads of one token; the
// heads of q come first, then those of k.
template <typename T, int PV, int NC, int LPH>
__global__ void __launch_bounds__(256)
norm_forward(const NormArgs a, T* __restrict__ qo, T* __restrict__ ko, int steps, int waves_per_token) {
  constexpr int HPW = 64 / LPH;
  const int lane = threadIdx.x & 63, sub = lane % LPH, head_in = lane / LPH;
  const int64_t id = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
  const int64_t tok = id / waves_per_token;
  if (tok >= a.n_tokens) return;
  const int part = (int)(id - tok * waves_per_token);
  const int n_pairs = a.d / 2, n_heads = a.Hq + a.Hk, n_rot = a.rot / 2;
  const PairMap m{a.interleaved ? 0 : n_rot};
  HeadPairs<PV, NC> cs;
  if (n_rot) load_turns<PV, NC, LPH>(a.pos[tok], a.freq, sub, n_rot, cs);
  for (int st = 0; st < steps; ++st) {
    const int h = (part * steps + st) * HPW + head_in;
    const bool there = h < n_heads, is_q = h < a.Hq;
    if (!there) continue;  // whole heads; the exchanges stay inside one
    const T* __restrict__ x = is_q ? (const T*)a.q + tok * a.ld_q + (int64_t)h * a.d
                                   : (const T*)a.k + tok * a.ld_k + (int64_t)(h - a.Hq) * a.d;
    T* __restrict__ out = is_q ? qo + (tok * a.Hq + h) * a.d : ko + (tok * a.Hk + (h - a.Hq)) * a.d;
    HeadPairs<PV, NC> v, w;
    load_pairs<T, PV, NC, LPH>(x, sub, n_pairs, m, v);
    load_weight<PV, NC>(is_q ? a.wq : a.wk, sub, LPH, n_pairs, m, w);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < PV; ++e) ss += v.a[i][e] * v.a[i][e] + v.b[i][e] * v.b[i][e];
    const float r = inv_norm(head_sum<LPH>(ss), a.sum_factor, a.eps) * (is_q ? a.q_scale : 1.f);
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < PV; ++e) {
        const float va = v.a[i][e] * r * w.a[i][e], vb = v.b[i][e] * r * w.b[i][e];
        v.a[i][e] = n_rot ? va * cs.a[i][e] - vb * cs.b[i][e] : va;
        v.b[i][e] = n_rot ? va * cs.b[i][e] + vb * cs.a[i][e] : vb;
      }
    store_pairs<T, PV, NC, LPH>(out, sub, n_pairs, m, v);
  }
}

// Backward over one of q (blockIdx.y = 0) and k (1): the workgroup's waves
// go through tokens blockIdx.x * 4 + wave, + 4 * gridDim.x, ..., all heads
// of each, with the weight's gradient in registers.
template <typename T, int PV, int NC, int LPH>
__global__ void __launch_bounds__(256)
norm_backward(const NormArgs a, const T* __restrict__ dqo, const T* __restrict__ dko, T* __restrict__ dq,
              T* __restrict__ dk, float* __restrict__ part, int want_q, int want_k) {
  constexpr int HPW = 64 / LPH;
  __shared__ float sums[4][2][NC * PV][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), sub = lane % LPH, head_in = lane / LPH;
  const bool is_q = blockIdx.y == 0;
  const int H = is_q ? a.Hq : a.Hk;
  const int64_t ld = is_q ? a.ld_q : a.ld_k;
  const T* __restrict__ x0 = (const T*)(is_q ? a.q : a.k);
  const T* __restrict__ g0 = is_q ? dqo : dko;
  T* __restrict__ out0 = is_q ? dq : dk;
  const float scale = is_q ? a.q_scale : 1.f;
  const int n_pairs = a.d / 2, n_rot = a.rot / 2;
  const PairMap m{a.interleaved ? 0 : n_rot};
  HeadPairs<PV, NC> cs, w, dw;
  load_weight<PV, NC>(is_q ? a.wq : a.wk, sub, LPH, n_pairs, m, w);
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < PV; ++e) dw.a[i][e] = dw.b[i][e] = 0.f;
  for (int64_t tok = (int64_t)blockIdx.x * 4 + wave; tok < a.n_tokens; tok += (int64_t)gridDim.x * 4) {
    if (n_rot) load_turns<PV, NC, LPH>(a.pos[tok], a.freq, sub, n_rot, cs);
    for (int h = head_in; h < H; h += HPW) {
      HeadPairs<PV, NC> v, g;
      load_pairs<T, PV, NC, LPH>(x0 + tok * ld + (int64_t)h * a.d, sub, n_pairs, m, v);
      load_pairs<T, PV, NC, LPH>(g0 + (tok * H + h) * a.d, sub, n_pairs, m, g);
      float ss = 0.f, along = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < PV; ++e) {
          const float ga = g.a[i][e] * scale, gb = g.b[i][e] * scale;
          g.a[i][e] = n_rot ? ga * cs.a[i][e] + gb * cs.b[i][e] : ga;
          g.b[i][e] = n_rot ? gb * cs.a[i][e] - ga * cs.b[i][e] : gb;
          ss += v.a[i][e] * v.a[i][e] + v.b[i][e] * v.b[i][e];
          along += g.a[i][e] * w.a[i][e] * v.a[i][e] + g.b[i][e] * w.b[i][e] * v.b[i][e];
        }
      const float r = inv_norm(head_sum<LPH>(ss), a.sum_factor, a.eps);
      const float back = head_sum<LPH>(along) * a.sum_factor * r;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < PV; ++e) {
          const float ha = v.a[i][e] * r, hb = v.b[i][e] * r;
          dw.a[i][e] += g.a[i][e] * ha;
          dw.b[i][e] += g.b[i][e] * hb;
          v.a[i][e] = r * (g.a[i][e] * w.a[i][e] - ha * back);
          v.b[i][e] = r * (g.b[i][e] * w.b[i][e] - hb * back);
        }
      store_pairs<T, PV, NC, LPH>(out0 + (tok * H + h) * a.d, sub, n_pairs, m, v);
    }
  }
  if (!(is_q ? want_q : want_k)) return;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < PV; ++e) {
      sums[wave][0][i * PV + e][lane] = dw.a[i][e];
      sums[wave][1][i * PV + e][lane] = dw.b[i][e];
    }
  __syncthreads();
  float* __restrict__ row = part + ((int64_t)blockIdx.y * kNormParts + blockIdx.x) * a.d;
  for (int c = threadIdx.x; c < 2 * NC * PV * LPH; c += 256) {
    const int which = c % 2, s = c / 2 % LPH, ie = c / 2 / LPH;
    const int p = (ie / PV * LPH + s) * PV + ie % PV;
    if (p >= n_pairs) continue;
    float v = 0.f;
    for (int wv = 0; wv < 4; ++wv)
#pragma unroll
      for (int h = 0; h < HPW; ++h) v += sums[wv][which][ie][h * LPH + s];
    row[m.first(p) + (which ? m.gap(p) : 0)] = v;
  }
}

// dq_weight (blockIdx.y = 0) and dk_weight (1) from the workgroups' rows
__global__ void __launch_bounds__(1024)
norm_params(const float* __restrict__ part, int n_part, int d, float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  float* out = blockIdx.y ? dwk : dwq;
  if (!out) return;
  const float* __restrict__ rows = part + (int64_t)blockIdx.y * kNormParts * d;
  float v = 0.f;
  if (c < d)
    for (int r = wave; r < n_part; r += 16) v += rows[(int64_t)r * d + c];
  sums[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || c >= d) return;
  v = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) v += sums[w][lane];
  out[c] = v;
}

template <typename T, int PV, int NC, int LPH>
int forward_t(const NormArgs& a, void* qo, void* ko, hipStream_t st) {
  const int groups = (int)ceil_div(a.Hq + a.Hk, 64 / LPH);
  // heads of one token a wave goes through: up to 8 groups, while 4096 waves are left
  int steps = 8;
  while (steps > 1 && (steps > groups || a.n_tokens * ceil_div(groups, steps) < 4096)) steps /= 2;
  const int per_token = (int)ceil_div(groups, steps);
  const int64_t blocks = ceil_div((int64_t)a.n_tokens * per_token, 4);
  if (blocks > INT32_MAX) return (int)hipErrorInvalidValue;
  return (int)launch_kernel(norm_forward<T, PV, NC, LPH>, dim3((unsigned)blocks), dim3(256), st, a, (T*)qo, (T*)ko,
                            steps, per_token);
}
template <typename T, int PV, int NC, int LPH>
int backward_t(const NormArgs& a, const void* dqo, const void* dko, void* dq, void* dk, float* dwq, float* dwk,
               float* part, hipStream_t st) {
  const int64_t want = ceil_div(a.n_tokens, 4);
  const int blocks = want < kNormParts ? (int)want : kNormParts;
  if (blocks > 0) {
    const hipError_t e = launch_kernel(norm_backward<T, PV, NC, LPH>, dim3(blocks, 2), dim3(256), st, a,
                                       (const T*)dqo, (const T*)dko, (T*)dq, (T*)dk, part, dwq != nullptr,
                                       dwk != nullptr);
    if (e != hipSuccess) return (int)e;
  }
  if (!dwq && !dwk) return 0;
  return (int)launch_kernel(norm_params, dim3((unsigned)ceil_div(a.d, 64), 2), dim3(1024), st, part, blocks, a.d,
                            dwq, dwk);
}

template <int PV_, int NC_, int LPH_> struct Shape {
  static constexpr int PV = PV_, NC = NC_, LPH = LPH_;
};

// Four pairs a lane when neither the head nor its rotated part ends inside
// such a group, else single pairs; lanes per head the power of two that
// covers the head.
template <typename T, typename F>
int dispatch_t(int d, int rot, F&& f) {
  const int pairs = d / 2;
  if (d % 8 == 0 && rot % 8 == 0) {
    if (pairs <= 16) return f(T{}, Shape<4, 1, 4>{});
    if (pairs <= 32) return f(T{}, Shape<4, 1, 8>{});
    if (pairs <= 64) return f(T{}, Shape<4, 1, 16>{});
    if (pairs <= 128) return f(T{}, Shape<4, 1, 32>{});
    return f(T{}, Shape<4, 1, 64>{});
  }
  if (pairs <= 16) return f(T{}, Shape<1, 1, 16>{});
  if (pairs <= 32) return f(T{}, Shape<1, 1, 32>{});
  if (pairs <= 64) return f(T{}, Shape<1, 1, 64>{});
  if (pairs <= 128) return f(T{}, Shape<1, 2, 64>{});
  return f(T{}, Shape<1, 4, 64>{});
}
template <typename F>
int dispatch(int is_bf16, int d, int rot, F&& f) {
  return is_bf16 ? dispatch_t<bf16_t>(d, rot, f) : dispatch_t<float>(d, rot, f);
}

}  // namespace

int launch_norm_forward(int is_bf16, const NormArgs& a, void* qo, void* ko, void* stream) {
  return dispatch(is_bf16, a.d, a.rot, [&](auto t, auto s) {
    return forward_t<decltype(t), s.PV, s.NC, s.LPH>(a, qo, ko, (hipStream_t)stream);
  });
}
int launch_norm_backward(int is_bf16, const NormArgs& a, const void* dqo, const void* dko, void* dq, void* dk,
                         float* dwq, float* dwk, float* part, void* stream) {
  return dispatch(is_bf16, a.d, a.rot, [&](auto t, auto s) {
    return backward_t<decltype(t), s.PV, s.NC, s.LPH>(a, dqo, dko, dq, dk, dwq, dwk, part, (hipStream_t)stream);
  });
}

}  // namespace kda
