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
// rotated pair sit side by side (WIDE: one load of 2 PV channels) or rot / 2
// apart (two loads of PV); either way a lane loads both, so the rotation
// needs no exchange.  Channels that are not rotated are paired as they come.
// A wave keeps the cosines and sines of a token while it goes through the
// token's heads: they are taken in quarter turns, reduced in 64 bits, because
// fp32 would lose the angle of a far position (2^-24 of a million is 0.06
// revolutions); the rest, an eighth of a turn at most, is rounded to fp32
// once, 2^-24 of itself.  Heads are loaded kNormBatch groups at a time before
// the first is used.
//
// Measured: unit vectors of 4096 tokens, 16 + 16 heads of 128, bf16, 12.8 us
// (67.1 MB, 5.2 TB/s); 8192 tokens of 32 + 8 heads of 128, half rotated, 31 us
// (167.8 MB, 5.4 TB/s; a large copy reaches 4.9 beyond the last-level cache);
// 8 tokens 4.8 us, which is the launch and one token's chain of loads, angles
// and sums; backward 8192 tokens of 16 + 4 heads of 64, 32 us in fp32 (125.8
// MB) and 23.6 in bf16 (62.9), which waits for its loads (34 and 48 % vector
// issue), and 4 for the weights' sums.
#include "kda_layer_device.h"

namespace kda {

namespace {

// groups of heads (forward; half backward) a wave loads at a time: rotated
// forward 33.0 us with 4, 34.9 with 2, 38.3 with 8 (registers)
constexpr int kNormBatch = 4;

// PV pairs (a, b) in each of NC chunks, LPH lanes apart.
template <int PV, int NC>
struct Pairs {
  float a[NC][PV], b[NC][PV];
};

// Where a lane's pairs are in a head.
template <int PV, int NC, int LPH, bool WIDE>
struct Place {
  int first[NC], second[NC];  // channels of the first pair's a and b
  bool there[NC];
  __device__ __forceinline__ Place(int sub, int d, int n_rot) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = (i * LPH + sub) * PV;
      there[i] = p < d / 2;
      first[i] = !there[i] ? 0 : !WIDE && p < n_rot ? p : 2 * p;
      second[i] = WIDE ? first[i] + 1 : p < n_rot ? first[i] + n_rot : first[i] + PV;
    }
  }
  // channel of pair e's a (b: from second) relative to the head
  __device__ __forceinline__ static int step(int e) { return WIDE ? 2 * e : e; }
};

// A head's pairs as they come from memory.
template <typename T, int PV, int NC, bool WIDE>
struct Raw {
  typename Pack<T, WIDE ? 2 * PV : PV>::type lo[NC];
  typename Pack<T, PV>::type hi[NC];
  template <int LPH>
  __device__ __forceinline__ void load(const T* __restrict__ x, const Place<PV, NC, LPH, WIDE>& at) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      lo[i] = *(const typename Pack<T, WIDE ? 2 * PV : PV>::type*)(x + at.first[i]);
      if (!WIDE) hi[i] = *(const typename Pack<T, PV>::type*)(x + at.second[i]);
    }
  }
  template <int LPH>
  __device__ __forceinline__ void get(const Place<PV, NC, LPH, WIDE>& at, bool head, Pairs<PV, NC>& v) const {
    auto el = [](auto r, int e) {
      if constexpr (std::is_arithmetic_v<decltype(r)>) return Elem<T>::to_f32(r);
      else return Elem<T>::to_f32(r[e]);
    };
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < PV; ++e) {
        const float a = el(lo[i], WIDE ? 2 * e : e), b = WIDE ? el(lo[i], 2 * e + 1) : el(hi[i], e);
        v.a[i][e] = head && at.there[i] ? a : 0.f;
        v.b[i][e] = head && at.there[i] ? b : 0.f;
      }
  }
};

template <typename T, int PV, int NC, int LPH, bool WIDE>
__device__ __forceinline__ void store_pairs(T* __restrict__ x, const Place<PV, NC, LPH, WIDE>& at,
                                            const Pairs<PV, NC>& v) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (!at.there[i]) continue;
    if constexpr (WIDE) {
      float t[2 * PV];
#pragma unroll
      for (int e = 0; e < PV; ++e) {
        t[2 * e] = v.a[i][e];
        t[2 * e + 1] = v.b[i][e];
      }
      store_vec<T, 2 * PV>(x + at.first[i], t);
    } else {
      store_vec<T, PV>(x + at.first[i], v.a[i]);
      store_vec<T, PV>(x + at.second[i], v.b[i]);
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
                                           Pairs<PV, NC>& cs) {
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < PV; ++e) {
      const int p = (i * LPH + sub) * PV + e;
      cs.a[i][e] = 1.f;
      cs.b[i][e] = 0.f;
      if (p < n_rot) {
        // the rest beside the nearest quarter turn, which fp32 holds to 2^-24 of itself
        const double quarters = (double)pos * (double)freq[p] * 0.6366197723675814, whole = __builtin_rint(quarters);
        const int k = (int)(whole - 4.0 * __builtin_rint(0.25 * whole));
        float s, c;
        sincospif(0.5f * (float)(quarters - whole), &s, &c);
        const float a = k & 1 ? s : c, b = k & 1 ? c : s;
        cs.a[i][e] = (k + 1) & 2 ? -a : a;
        cs.b[i][e] = k & 2 ? -b : b;
      }
    }
}

template <int PV, int NC, int LPH, bool WIDE>
__device__ __forceinline__ void load_weight(const float* __restrict__ w, const Place<PV, NC, LPH, WIDE>& at,
                                            Pairs<PV, NC>& v) {
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < PV; ++e) {
      const bool there = w && at.there[i];
      v.a[i][e] = there ? w[at.first[i] + at.step(e)] : 1.f;
      v.b[i][e] = there ? w[at.second[i] + at.step(e)] : 1.f;
    }
}

// 1 / sqrt, rounded as the division and the square root are (the hardware's
// approximation is a unit in the last place off)
__device__ __forceinline__ float inv_norm(float ss, float f, float eps) { return 1.f / sqrtf(f * ss + eps); }

// A token's heads in groups of HPW: those of q, then those of k.
template <int HPW>
struct Groups {
  int q, all;
  __device__ explicit Groups(const NormArgs& a) : q((a.Hq + HPW - 1) / HPW), all(q + (a.Hk + HPW - 1) / HPW) {}
};

// Forward: a wave takes `steps` groups of heads of one token.
template <typename T, int PV, int NC, int LPH, bool WIDE>
__global__ void __launch_bounds__(64 * kNormForwardWaves)
norm_forward(const NormArgs a, T* __restrict__ qo, T* __restrict__ ko, int steps, int waves_per_token) {
  constexpr int HPW = 64 / LPH, U = kNormBatch / NC > 0 ? kNormBatch / NC : 1;
  const int lane = threadIdx.x & 63, sub = lane % LPH, head_in = lane / LPH;
  const int id = (int)blockIdx.x * kNormForwardWaves + uniform(threadIdx.x >> 6);
  const int tok = id / waves_per_token;
  if (tok >= a.n_tokens) return;
  const Groups<HPW> groups(a);
  int g = (id - tok * waves_per_token) * steps;
  const int last = g + steps < groups.all ? g + steps : groups.all;
  const int n_rot = a.rot / 2;
  const Place<PV, NC, LPH, WIDE> at(sub, a.d, n_rot);
  // a group's heads; lanes past the last head read it again
  auto head_of = [&](int group, bool* q, bool* there) {
    *q = group < groups.q;
    const int h = (*q ? group : group - groups.q) * HPW + head_in, H = *q ? a.Hq : a.Hk;
    *there = h < H;
    return h < H ? h : H - 1;
  };
  Raw<T, PV, NC, WIDE> raw[U];
  auto load = [&](int from) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bool q, there;
      const int h = head_of(from + u < last ? from + u : last - 1, &q, &there);
      raw[u].load((q ? (const T*)a.q + tok * a.ld_q : (const T*)a.k + tok * a.ld_k) + h * a.d, at);
    }
  };
  load(g);
  Pairs<PV, NC> cs, wq, wk;
  load_weight(a.wq, at, wq);
  load_weight(a.wk, at, wk);
  if (n_rot) load_turns<PV, NC, LPH>(a.pos[tok], a.freq, sub, n_rot, cs);
  for (; g < last; g += U) {
    if (g != (id - tok * waves_per_token) * steps) load(g);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (g + u >= last) break;
      bool q, there;
      const int h = head_of(g + u, &q, &there);
      Pairs<PV, NC> v;
      raw[u].get(at, there, v);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < PV; ++e) ss += v.a[i][e] * v.a[i][e] + v.b[i][e] * v.b[i][e];
      const float r = inv_norm(head_sum<LPH>(ss), a.sum_factor, a.eps) * (q ? a.q_scale : 1.f);
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < PV; ++e) {
          const float va = v.a[i][e] * r * (q ? wq.a[i][e] : wk.a[i][e]),
                      vb = v.b[i][e] * r * (q ? wq.b[i][e] : wk.b[i][e]);
          v.a[i][e] = n_rot ? va * cs.a[i][e] - vb * cs.b[i][e] : va;
          v.b[i][e] = n_rot ? va * cs.b[i][e] + vb * cs.a[i][e] : vb;
        }
      if (there) store_pairs((q ? qo + (int64_t)tok * a.Hq * a.d : ko + (int64_t)tok * a.Hk * a.d) + h * a.d, at, v);
    }
  }
}

// Backward: a wave takes `steps` groups of heads of every token that is
// its, gridDim.x * kNormWaves / waves_per_token tokens apart, and sums the
// weights' gradients in registers; the workgroup leaves one row of partial
// sums for each of q and k.
constexpr int kNormWaves = 16;
template <typename T, int PV, int NC, int LPH, bool WIDE>
__global__ void __launch_bounds__(64 * kNormWaves)
norm_backward(const NormArgs a, const T* __restrict__ dqo, const T* __restrict__ dko, T* __restrict__ dq,
              T* __restrict__ dk, float* __restrict__ part, int want_q, int want_k, int steps, int waves_per_token) {
  constexpr int HPW = 64 / LPH, U = kNormBatch / 2 / NC > 0 ? kNormBatch / 2 / NC : 1;
  __shared__ float sums[kNormWaves][2][NC * PV][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), sub = lane % LPH, head_in = lane / LPH;
  const Groups<HPW> groups(a);
  const int id = (int)blockIdx.x * kNormWaves + wave, stride = (int)gridDim.x * kNormWaves / waves_per_token;
  const int first = id % waves_per_token * steps, last = first + steps < groups.all ? first + steps : groups.all;
  const int n_rot = a.rot / 2;
  const Place<PV, NC, LPH, WIDE> at(sub, a.d, n_rot);
  Pairs<PV, NC> cs, wq, wk, dwq, dwk;
  load_weight(a.wq, at, wq);
  load_weight(a.wk, at, wk);
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < PV; ++e) dwq.a[i][e] = dwq.b[i][e] = dwk.a[i][e] = dwk.b[i][e] = 0.f;
  auto head_of = [&](int group, bool* q, bool* there) {
    *q = group < groups.q;
    const int h = (*q ? group : group - groups.q) * HPW + head_in, H = *q ? a.Hq : a.Hk;
    *there = h < H;
    return h < H ? h : H - 1;
  };
  for (int tok = id / waves_per_token; tok < a.n_tokens; tok += stride) {
    if (n_rot) load_turns<PV, NC, LPH>(a.pos[tok], a.freq, sub, n_rot, cs);
    for (int g = first; g < last; g += U) {
      Raw<T, PV, NC, WIDE> rx[U], rg[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        bool q, there;
        const int h = head_of(g + u < last ? g + u : last - 1, &q, &there);
        rx[u].load((q ? (const T*)a.q + tok * a.ld_q : (const T*)a.k + tok * a.ld_k) + h * a.d, at);
        rg[u].load((q ? dqo + (int64_t)tok * a.Hq * a.d : dko + (int64_t)tok * a.Hk * a.d) + h * a.d, at);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (g + u >= last) break;
        bool q, there;
        const int h = head_of(g + u, &q, &there);
        const float scale = q ? a.q_scale : 1.f;
        Pairs<PV, NC> v, gr;
        rx[u].get(at, there, v);
        rg[u].get(at, there, gr);
        float ss = 0.f, along = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int e = 0; e < PV; ++e) {
            const float ga = gr.a[i][e] * scale, gb = gr.b[i][e] * scale;
            gr.a[i][e] = n_rot ? ga * cs.a[i][e] + gb * cs.b[i][e] : ga;
            gr.b[i][e] = n_rot ? gb * cs.a[i][e] - ga * cs.b[i][e] : gb;
            ss += v.a[i][e] * v.a[i][e] + v.b[i][e] * v.b[i][e];
            along += gr.a[i][e] * (q ? wq.a[i][e] : wk.a[i][e]) * v.a[i][e] +
                     gr.b[i][e] * (q ? wq.b[i][e] : wk.b[i][e]) * v.b[i][e];
          }
        // lanes beyond the last head hold zeros, whose norm without an epsilon is none
        const float norm = inv_norm(head_sum<LPH>(ss), a.sum_factor, a.eps), r = there ? norm : 0.f;
        const float back = head_sum<LPH>(along) * a.sum_factor * r;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int e = 0; e < PV; ++e) {
            const float ha = v.a[i][e] * r, hb = v.b[i][e] * r;
            const float da = gr.a[i][e] * ha, db = gr.b[i][e] * hb;
            if (q) {
              dwq.a[i][e] += da;
              dwq.b[i][e] += db;
            } else {
              dwk.a[i][e] += da;
              dwk.b[i][e] += db;
            }
            v.a[i][e] = r * (gr.a[i][e] * (q ? wq.a[i][e] : wk.a[i][e]) - ha * back);
            v.b[i][e] = r * (gr.b[i][e] * (q ? wq.b[i][e] : wk.b[i][e]) - hb * back);
          }
        if (there) store_pairs((q ? dq + (int64_t)tok * a.Hq * a.d : dk + (int64_t)tok * a.Hk * a.d) + h * a.d, at, v);
      }
    }
  }
  auto reduce = [&](const Pairs<PV, NC>& dw, float* row) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < PV; ++e) {
        sums[wave][0][i * PV + e][lane] = dw.a[i][e];
        sums[wave][1][i * PV + e][lane] = dw.b[i][e];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * NC * PV * LPH; c += 64 * kNormWaves) {
      const int which = c % 2, s = c / 2 % LPH, ie = c / 2 / LPH;
      const Place<PV, NC, LPH, WIDE> of(s, a.d, n_rot);
      float v = 0.f;
      for (int wv = 0; wv < kNormWaves; ++wv)
#pragma unroll
        for (int h = 0; h < HPW; ++h) v += sums[wv][which][ie][h * LPH + s];
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (i == ie / PV && of.there[i]) row[(which ? of.second[i] : of.first[i]) + of.step(ie % PV)] = v;
    }
  };
  if (want_q) reduce(dwq, part + (int64_t)blockIdx.x * a.d);
  if (want_k) reduce(dwk, part + (int64_t)(kNormParts + blockIdx.x) * a.d);
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
#pragma unroll 16
    for (int r = wave; r < n_part; r += 16) v += rows[(int64_t)r * d + c];
  sums[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || c >= d) return;
  v = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) v += sums[w][lane];
  out[c] = v;
}

template <typename T, int PV, int NC, int LPH, bool WIDE>
int forward_t(const NormArgs& a, void* qo, void* ko, hipStream_t st) {
  const int groups = norm_groups(a.Hq, a.Hk, LPH), steps = norm_steps(a.n_tokens, groups, kNormMinWaves);
  const int per_token = (int)ceil_div(groups, steps);
  const int64_t blocks = ceil_div((int64_t)a.n_tokens * per_token, kNormForwardWaves);
  return (int)launch_kernel(norm_forward<T, PV, NC, LPH, WIDE>, dim3((unsigned)blocks), dim3(64 * kNormForwardWaves),
                            st, a, (T*)qo, (T*)ko, steps, per_token);
}
template <typename T, int PV, int NC, int LPH, bool WIDE>
int backward_t(const NormArgs& a, const void* dqo, const void* dko, void* dq, void* dk, float* dwq, float* dwk,
               float* part, hipStream_t st) {
  const int groups = norm_groups(a.Hq, a.Hk, LPH);
  int steps = norm_steps(a.n_tokens, groups, kNormMinWaves), per_token = (int)ceil_div(groups, steps);
  // a token's waves divide the grid's, so that a wave keeps its place in the token
  while (per_token & (per_token - 1)) ++per_token;
  if (per_token > kNormParts * kNormWaves) per_token = kNormParts * kNormWaves;
  steps = (int)ceil_div(groups, per_token);
  int64_t blocks = ceil_div((int64_t)a.n_tokens * per_token, kNormWaves);
  if (blocks > kNormParts) blocks = kNormParts;
  while (blocks & (blocks - 1)) ++blocks;
  if (blocks > 0) {
    const hipError_t e = launch_kernel(norm_backward<T, PV, NC, LPH, WIDE>, dim3((unsigned)blocks),
                                       dim3(64 * kNormWaves), st, a, (const T*)dqo, (const T*)dko, (T*)dq, (T*)dk,
                                       part, dwq != nullptr, dwk != nullptr, steps, per_token);
    if (e != hipSuccess) return (int)e;
  }
  if (!dwq && !dwk) return 0;
  return (int)launch_kernel(norm_params, dim3((unsigned)ceil_div(a.d, 64), 2), dim3(1024), st, part, (int)blocks, a.d,
                            dwq, dwk);
}

template <int PV_, int NC_, int LPH_> struct Shape {
  static constexpr int PV = PV_, NC = NC_, LPH = LPH_;
};

// the shape that norm_four_pairs and norm_head_lanes choose
template <typename T, typename F>
int dispatch_t(int d, int rot, F&& f) {
  const int lanes = norm_head_lanes(d, rot);
  if (norm_four_pairs(d, rot)) {
    if (lanes == 4) return f(T{}, Shape<4, 1, 4>{});
    if (lanes == 8) return f(T{}, Shape<4, 1, 8>{});
    if (lanes == 16) return f(T{}, Shape<4, 1, 16>{});
    if (lanes == 32) return f(T{}, Shape<4, 1, 32>{});
    return f(T{}, Shape<4, 1, 64>{});
  }
  if (lanes == 16) return f(T{}, Shape<1, 1, 16>{});
  if (lanes == 32) return f(T{}, Shape<1, 1, 32>{});
  if (d <= 128) return f(T{}, Shape<1, 1, 64>{});
  if (d <= 256) return f(T{}, Shape<1, 2, 64>{});
  return f(T{}, Shape<1, 4, 64>{});
}
template <typename F>
int dispatch(int is_bf16, const NormArgs& a, F&& f) {
  const bool wide = a.interleaved || a.rot == 0;
  auto go = [&](auto t, auto s) { return wide ? f(t, s, std::true_type{}) : f(t, s, std::false_type{}); };
  return is_bf16 ? dispatch_t<bf16_t>(a.d, a.rot, go) : dispatch_t<float>(a.d, a.rot, go);
}

}  // namespace

int launch_norm_forward(int is_bf16, const NormArgs& a, void* qo, void* ko, void* stream) {
  return dispatch(is_bf16, a, [&](auto t, auto s, auto wide) {
    return forward_t<decltype(t), s.PV, s.NC, s.LPH, wide.value>(a, qo, ko, (hipStream_t)stream);
  });
}
int launch_norm_backward(int is_bf16, const NormArgs& a, const void* dqo, const void* dko, void* dq, void* dk,
                         float* dwq, float* dwk, float* part, void* stream) {
  return dispatch(is_bf16, a, [&](auto t, auto s, auto wide) {
    return backward_t<decltype(t), s.PV, s.NC, s.LPH, wide.value>(a, dqo, dko, dq, dk, dwq, dwk, part,
                                                                  (hipStream_t)stream);
  });
}

}  // namespace kda
