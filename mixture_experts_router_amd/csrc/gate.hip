// The routing gate (softmax or sigmoid scores, a balancing bias, groups,
// top-k, renormalised weights) and its gradient.
//
//   s_e   = softmax(l)_e  or  1 / (1 + exp(-l_e))
//   key_e = s_e + b_e                       (no bias: the order of l itself)
//   a group of gs consecutive experts is worth the sum of its best one or two
//   keys; the group_k best groups stay; the k best keys among them are chosen,
//   the lower index first among equal keys
//   l_e = -inf masks e: s_e = 0 and key_e = -inf, whatever the bias; a key of
//   -inf adds nothing as a group's second best
//   w_j   = c s_j,  or renormalised  c s_j / sum_r s_r   (sigmoid: + 1e-20)
//
// Which of two experts is chosen is decided as keys formed in 64 bits decide
// it, whatever the rounding of a 32-bit score: the selection runs on fp32
// keys, whose error is bounded below, and a round in which another live key
// lies within that bound of the best is decided again among those candidates
// with keys in fp64.  Without a bias, and with groups ranked by their best
// expert, the logits give the order exactly and no score is formed for it.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// ------------------------------------------------------- ordered keys ---
//
// fp32 values as unsigned integers of the same order, so a maximum is one
// v_max_u32 a step: -0 counts as +0, NaN is the lowest live key (1), and 0
// stands for "not a candidate".
__device__ __forceinline__ uint32_t key_of(float v) {
  v = v + 0.0f;
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  u ^= (uint32_t)((int32_t)u >> 31) | 0x80000000u;
  return v != v ? 1u : u;
}

__device__ __forceinline__ float value_of(uint32_t key) {
  return __builtin_bit_cast(float, (key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

__device__ __forceinline__ uint64_t key_of64(double v) {
  v = v + 0.0;
  uint64_t u = __builtin_bit_cast(uint64_t, v);
  u ^= (uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull;
  return v != v ? 1u : u;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROWS, 0xF, false);
}

constexpr int DPP_BCAST15 = 0x142;  // lane 15 of a row to the next row
constexpr int DPP_BCAST31 = 0x143;  // lane 31 to lanes 32-63

// maximum over the 64 lanes, in a scalar register
__device__ __forceinline__ uint32_t wave_max_key(uint32_t v) {
  v = max(v, dpp_u<DPP_QUAD_1032, 0xF>(v));
  v = max(v, dpp_u<DPP_QUAD_2301, 0xF>(v));
  v = max(v, dpp_u<DPP_ROW_HALF_MIRROR, 0xF>(v));
  v = max(v, dpp_u<DPP_ROW_MIRROR, 0xF>(v));
  v = max(v, dpp_u<DPP_BCAST15, 0xA>(v));
  v = max(v, dpp_u<DPP_BCAST31, 0xC>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// 64-bit maximum, then the lowest index that holds it (slow path only)
__device__ __forceinline__ int wave_best64(uint64_t key, int index) {
#pragma unroll 1
  for (int off = 1; off < WAVE; off <<= 1) {
    const uint64_t ok = __shfl_xor(key, off);
    const int oi = __shfl_xor(index, off);
    const bool take = ok > key || (ok == key && oi < index);
    key = take ? ok : key;
    index = take ? oi : index;
  }
  return __builtin_amdgcn_readfirstlane(index);
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll 1
  for (int off = 1; off < WAVE; off <<= 1) v += __shfl_xor(v, off);
  return v;
}

// orders LDS accesses of one wave (its LDS instructions execute in order)
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ------------------------------------------------------- logits -------
template <int LT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (LT == GATE_F32) return ((const float*)p)[i];
  else return act_to_f32(((const uint16_t*)p)[i], LT);
}

// N = 1, 2 or 4 consecutive logits, aligned to their size
template <int LT, int N>
__device__ __forceinline__ void load_logits(const void* p, int64_t i, float* v) {
  if constexpr (N == 1) {
    v[0] = load_logit<LT>(p, i);
  } else if constexpr (LT == GATE_F32) {
    typedef float vec __attribute__((ext_vector_type(N)));
    const vec r = *(const vec*)((const float*)p + i);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = r[j];
  } else {
    typedef uint16_t vec __attribute__((ext_vector_type(N)));
    const vec r = *(const vec*)((const uint16_t*)p + i);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = act_to_f32(r[j], LT);
  }
}

// sum over the eight lanes of a half row; every lane of it gets the same bits
__device__ __forceinline__ float sum8(float v) {
  v += dpp_f<DPP_QUAD_1032>(v);
  v += dpp_f<DPP_QUAD_2301>(v);
  v += dpp_f<DPP_ROW_HALF_MIRROR>(v);
  return v;
}

__device__ __forceinline__ float max8(float v) {
  v = fmaxf(v, dpp_f<DPP_QUAD_1032>(v));
  v = fmaxf(v, dpp_f<DPP_QUAD_2301>(v));
  v = fmaxf(v, dpp_f<DPP_ROW_HALF_MIRROR>(v));
  return v;
}

__device__ __forceinline__ float sigmoid_f32(float l) { return 1.0f / (1.0f + expf(-l)); }

constexpr float SIGMOID_EPS = 1e-20f;  // added to the selected scores' sum

}  // namespace

// ----------------------------------------------------------- the gate ---
//
// One wave per token; lane i holds the VPL consecutive experts i*VPL ...
// (VPL = 1, 2, 4 for up to 64, 128, 256 experts), so a row is one coalesced
// load and each of the k rounds is six DPP maxima and a few ballots.
//
// Error bounds of the fp32 keys (u = 2^-24, products and sums rounded once,
// v_exp_f32 and v_rcp_f32 within one ulp):
//   sigmoid: the exponential is off by (2|l| + 2) u relative, which reaches s
//     times s (1 - s), and s (1 - s) |l| <= 0.224; the sum 1 + e adds u s, the
//     reciprocal 2 u s: less than 4 u = 2^-22 in all.
//   softmax: p is off by less than 40 u p_max: (3|d| + 2) u on each term
//     (p |d| <= 0.37 p_max), and in the sum the same weighted by p, at most
//     3 u (ln 256) + 2 u, and ten roundings.
//   the bias adds u |key|.
// Two keys further apart than twice that keep their order; the windows below
// (2^-20, or 2^-17 p_max, plus 2^-22 |key|) hold that with a margin.
template <int VPL, int LT>
__global__ __launch_bounds__(256) void gate_kernel(const void* __restrict__ logits, int64_t ld, int vec, int T, int E,
                                                   int k, GateDev g, int32_t* __restrict__ idx,
                                                   float* __restrict__ w, int32_t* __restrict__ k_used,
                                                   float* __restrict__ entropy, int32_t* __restrict__ clear_word) {
  __shared__ uint32_t keys[4][64 * VPL];
  __shared__ double lds[4][64 * VPL];
  const int lane = lane_id(), wave = wave_id();
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (k_used) *k_used = k;
    if (entropy) *entropy = 0.0f;
    if (clear_word) *clear_word = 0;
  }
  if (t >= T) return;
  const int e0 = lane * VPL;
  float l[VPL], b[VPL];
  const int64_t at = t * ld + e0;
#pragma unroll
  for (int j = 0; j < VPL; ++j) l[j] = b[j] = 0.0f;
  if (vec) {  // E is a multiple of VPL: a lane's experts are all there or all missing
    if (e0 < E) load_logits<LT, VPL>(logits, at, l);
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j < E) l[j] = load_logit<LT>(logits, at + j);
  }
  if (g.bias) {
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j < E) b[j] = g.bias[e0 + j];
  }

  // ---- keys
  const bool by_score = g.bias != nullptr || (g.groups > 1 && g.group_best == 2);
  const bool softmax = g.score == GATE_SOFTMAX;
  float m_all = 0.0f, z_all = 1.0f;  // softmax over all experts
  float ex[VPL];
  if (softmax && (by_score || !g.renorm)) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j < E) m = fmaxf(m, l[j]);
    m_all = wave_max(m);
    if (m_all == -INFINITY) m_all = 0.0f;  // every expert masked: all terms are 0
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      ex[j] = e0 + j < E ? expf(l[j] - m_all) : 0.0f;
      z += ex[j];
    }
    z_all = wave_sum(z);
    if (z_all == 0.0f) z_all = 1.0f;
  }
  uint32_t key[VPL];
  float window = 0.0f;
  if (by_score) {
    const float rz = softmax ? __builtin_amdgcn_rcpf(z_all) : 1.0f;
    window = softmax ? ldexp_f(rz, -17) : 0x1p-20f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const float s = softmax ? ex[j] * rz : __builtin_amdgcn_rcpf(1.0f + __expf(-l[j]));
      key[j] = key_of(l[j] == -INFINITY ? -INFINITY : s + b[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = key_of(l[j]);
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    if (e0 + j >= E) key[j] = 0u;

  // the keys in 64 bits (taken only where 32 bits do not decide)
  auto keys64 = [&](double* d) __attribute__((always_inline)) {
    if (softmax) {
      double z = 0.0;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        d[j] = e0 + j < E ? exp((double)l[j] - (double)m_all) : 0.0;
        z += d[j];
      }
      z = wave_sum64(z);
#pragma unroll
      for (int j = 0; j < VPL; ++j) d[j] = d[j] / z + (double)b[j];  // z = 0 only where all are masked
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) d[j] = 1.0 / (1.0 + exp(-(double)l[j])) + (double)b[j];
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (l[j] == -INFINITY) d[j] = -INFINITY;
  };

  // ---- groups: lane i < G ranks group i, G <= 64
  if (g.groups > 1) {
    const int G = g.groups, gs = E / G;
    uint32_t* row = keys[wave];
#pragma unroll
    for (int j = 0; j < VPL; ++j) row[e0 + j] = key[j];
    wave_lds_fence();
    uint32_t best = 0u, next = 0u;
    if (lane < G) {
      for (int i = 0; i < gs; ++i) {
        const uint32_t u = row[lane * gs + i];
        next = max(next, min(best, u));
        best = max(best, u);
      }
    }
    float value = value_of(best), err = 0.0f;
    if (g.group_best == 2) {
      const float second = value_of(next), v2 = second == -INFINITY ? 0.0f : second;
      err = 2.0f * window + 0x1p-22f * (fabsf(value) + fabsf(v2));
      value = value + v2;
    } else if (by_score) {
      err = window + 0x1p-22f * fabsf(value);
    }
    // two sums whose ranges value +- err do not meet keep their order
    const uint32_t top = lane < G ? key_of(value + err) : 0u;
    const float low = value - err;
    uint32_t gkey = lane < G ? key_of(value) : 0u;
    uint64_t kept = 0;
#pragma unroll 1
    for (int s = 0; s < g.group_k; ++s) {
      const uint32_t m = wave_max_key(gkey);
      int win = (int)__builtin_ctzll(__ballot(gkey == m && gkey != 0u));
      if (by_score) {
        const uint32_t bar = key_of(readlane_f(low, win));
        const uint64_t near = __ballot(gkey != 0u && max(top, gkey) >= bar);
        if ((near & (near - 1)) != 0) {
          double d[VPL];
          keys64(d);
          wave_lds_fence();
#pragma unroll
          for (int j = 0; j < VPL; ++j) lds[wave][e0 + j] = d[j];
          wave_lds_fence();
          double v = 0.0;
          if (near >> lane & 1) {
            uint64_t b1 = 0, b2 = 0;
            int i1 = 0, i2 = 0;
            for (int i = 0; i < gs; ++i) {
              const uint64_t u = key_of64(lds[wave][lane * gs + i]);
              if (u > b1) {
                b2 = b1, i2 = i1;
                b1 = u, i1 = i;
              } else if (u > b2) {
                b2 = u, i2 = i;
              }
            }
            v = lds[wave][lane * gs + i1];
            const double second = lds[wave][lane * gs + i2];
            if (g.group_best == 2 && second != -INFINITY) v = v + second;
          }
          win = wave_best64(near >> lane & 1 ? key_of64(v) : 0ull, lane);
        }
      }
      kept |= 1ull << win;
      if (lane == win) gkey = 0u;
    }
    // e / gs for e < 256: ceil(2^16 / gs) is exact enough for gs <= 256
    const uint32_t inv = (65536u + gs - 1) / gs;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j < E && !(kept >> (((uint32_t)(e0 + j) * inv) >> 16) & 1)) key[j] = 0u;
  }

  // ---- the k best keys; lane s keeps the expert of slot s
  int mine = 0;
#pragma unroll 1
  for (int s = 0; s < k; ++s) {
    uint32_t lm = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) lm = max(lm, key[j]);
    const uint32_t m = wave_max_key(lm);
    int e = 64 * VPL;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const uint64_t hit = __ballot(key[j] == m);
      const int c = hit ? (int)__builtin_ctzll(hit) * VPL + j : 64 * VPL;
      e = min(e, c);
    }
    if (by_score) {
      const float v = value_of(m);
      const uint32_t bar = key_of(v - (window + 0x1p-22f * fabsf(v)));
      int near = 0;
#pragma unroll
      for (int j = 0; j < VPL; ++j) near += (int)__popcll(__ballot(key[j] != 0u && key[j] >= bar));
      if (near != 1) {
        double d[VPL];
        keys64(d);
        uint64_t bk = 0;
        int bi = 64 * VPL;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const uint64_t u = key[j] != 0u && key[j] >= bar ? key_of64(d[j]) : 0ull;
          if (u > bk) bk = u, bi = e0 + j;
        }
        e = wave_best64(bk, bi);
      }
    }
    if (lane == s) mine = e;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j == e) key[j] = 0u;
  }

  // ---- weights, slot s in lane s (lanes k..7 add nothing)
  float ls = 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const float v = lane_read_f(l[j], mine / VPL);
    if (mine % VPL == j) ls = v;
  }
  const bool on = lane < k;
  const bool masked = ls == -INFINITY;  // a masked expert has weight 0, also where all are masked
  float wt;
  if (softmax) {
    if (g.renorm) {
      const float lm = max8(on ? ls : -INFINITY);
      const float p = on && !masked ? expf(ls - lm) : 0.0f;
      wt = p / sum8(p);
    } else {
      wt = expf(ls - m_all) / z_all;
    }
    wt = masked ? 0.0f : wt;
  } else {
    const float s1 = on ? sigmoid_f32(ls) : 0.0f;
    wt = g.renorm ? s1 / (sum8(s1) + SIGMOID_EPS) : s1;
  }
  if (on) {
    idx[t * k + lane] = mine;
    w[t * k + lane] = g.scale * wt;
  }
}

// -------------------------------------------------------- its gradient ---
//
// Sixteen lanes a token, four tokens a wave: lane i of a row holds slot i % 8
// and the experts 4 i .. 4 i + 3 of every 64.  With g_j = c dw_j at the
// selected experts and S the sum of their scores,
//   renormalised  ds_j = (g_j - sum_r g_r s_r / S) / S
//   sigmoid       dl_j = ds_j s_j (1 - s_j),  0 elsewhere
//   softmax       dl_j = p_j (g_j - sum_r g_r p_r), p over the selected when
//                 renormalised (0 elsewhere), else over all experts
// The selected gradients are scattered into an LDS row that is written out
// whole, so the kernel is bound by the [T, E] gradient's bytes.  Only the
// dense form reads every logit.  1 - s is formed as 1 / (1 + exp(l)).
template <int LT>
__global__ __launch_bounds__(256) void gate_backward_kernel(const void* __restrict__ logits, int64_t ld, int T, int E,
                                                            int k, int score, int renorm, float scale,
                                                            const int32_t* __restrict__ idx,
                                                            const float* __restrict__ dw, void* __restrict__ out,
                                                            int64_t ldo, int vec) {
  __shared__ f32x4 lds[16][64];
  const int lane = lane_id(), i16 = lane % 16, slot = i16 % 8;
  const int row = threadIdx.x / 16;
  const int64_t t = (int64_t)blockIdx.x * 16 + row;
  const bool tv = t < T;
  const bool dense = score == GATE_SOFTMAX && !renorm;
  float* r = (float*)lds[row];
  const int nv = (E + 63) / 64;
  for (int c = 0; c < nv; ++c) lds[row][i16 + 16 * c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  int e = -1;
  float gv = 0.0f, ls = -INFINITY;
  if (tv && slot < k) {
    e = idx[t * k + slot];
    if (e < 0 || e >= E) e = -1;  // no expert: no part in any sum
    if (e >= 0) {
      gv = scale * dw[t * k + slot];
      ls = load_logit<LT>(logits, t * ld + e);
    }
  }
  // a masked expert's score is 0: neither its gradient nor the incoming one counts
  float val;
  float dot = 0.0f, m = -INFINITY, z = 0.0f;
  if (score == GATE_SIGMOID) {
    const float s = e >= 0 ? sigmoid_f32(ls) : 0.0f;
    const float ds = 1.0f / (1.0f + expf(ls));
    if (renorm) {
      const float total = sum8(s) + SIGMOID_EPS;
      const float mean = sum8(s != 0.0f ? gv * s : 0.0f) / total;
      gv = (gv - mean) / total;
    }
    val = s != 0.0f ? gv * (s * ds) : 0.0f;
  } else if (renorm) {
    m = max8(ls);
    const float p0 = ls == -INFINITY ? 0.0f : expf(ls - m);
    const float sum = sum8(p0);
    const float p = p0 != 0.0f ? p0 / sum : 0.0f;
    const float mean = sum8(p != 0.0f ? gv * p : 0.0f);
    val = p != 0.0f ? p * (gv - mean) : 0.0f;
  } else {
    if (tv) {
      for (int x = i16; x < E; x += 16) m = fmaxf(m, load_logit<LT>(logits, t * ld + x));
    }
    m = fmaxf(m, dpp_f<DPP_QUAD_1032>(m));
    m = fmaxf(m, dpp_f<DPP_QUAD_2301>(m));
    m = fmaxf(m, dpp_f<DPP_ROW_HALF_MIRROR>(m));
    m = fmaxf(m, dpp_f<DPP_ROW_MIRROR>(m));
    if (tv) {
      for (int x = i16; x < E; x += 16) {
        const float v = load_logit<LT>(logits, t * ld + x);
        z += v == -INFINITY ? 0.0f : expf(v - m);
      }
    }
    z = sum8(z);
    z += dpp_f<DPP_ROW_MIRROR>(z);
    const float p = ls == -INFINITY ? 0.0f : expf(ls - m) / z;
    dot = sum8(p != 0.0f ? gv * p : 0.0f);
    val = gv;
  }

  // equal indices in a row: the first of them holds the sum, the others write nothing
  bool first = e >= 0;
  float total = val;
  auto merge = [&](int n, int oe, float ov) __attribute__((always_inline)) {
    if (oe == e) {
      total += ov;
      if (n <= slot) first = false;  // an earlier slot
    }
  };
  merge(1, dpp_i<0x121>(e), dpp_f<0x121>(val));
  merge(2, dpp_i<0x122>(e), dpp_f<0x122>(val));
  merge(3, dpp_i<0x123>(e), dpp_f<0x123>(val));
  merge(4, dpp_i<0x124>(e), dpp_f<0x124>(val));
  merge(5, dpp_i<0x125>(e), dpp_f<0x125>(val));
  merge(6, dpp_i<0x126>(e), dpp_f<0x126>(val));
  merge(7, dpp_i<0x127>(e), dpp_f<0x127>(val));
  wave_lds_fence();
  if (first && i16 < 8) r[e] = total;
  wave_lds_fence();
  if (!tv) return;

  auto grad = [&](float gsel, int x) __attribute__((always_inline)) {
    if (!dense) return gsel;
    const float v = load_logit<LT>(logits, t * ld + x);
    const float p = v == -INFINITY ? 0.0f : expf(v - m) / z;
    return p != 0.0f ? p * (gsel - dot) : 0.0f;
  };
  if (vec) {
    for (int c = 0; c < nv; ++c) {
      const int x = 4 * (i16 + 16 * c);
      if (x >= E) break;
      f32x4 v = lds[row][i16 + 16 * c];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = grad(v[j], x + j);
      if constexpr (LT == GATE_F32) {
        *(f32x4*)((float*)out + t * ldo + x) = v;
      } else {
        u32x2 o;
        o.x = (uint32_t)f32_to_act_bits(v.x, LT) | (uint32_t)f32_to_act_bits(v.y, LT) << 16;
        o.y = (uint32_t)f32_to_act_bits(v.z, LT) | (uint32_t)f32_to_act_bits(v.w, LT) << 16;
        *(u32x2*)((uint16_t*)out + t * ldo + x) = o;
      }
    }
  } else {
    for (int x = i16; x < E; x += 16) {
      const float v = grad(r[x], x);
      if constexpr (LT == GATE_F32) ((float*)out)[t * ldo + x] = v;
      else ((uint16_t*)out)[t * ldo + x] = f32_to_act_bits(v, LT);
    }
  }
}

// ------------------------------------------------------------- launchers --

namespace {
int lt_bytes(int lt) { return lt == GATE_F32 ? 4 : 2; }
}  // namespace

hipError_t launch_gate(const void* logits, int lt, int64_t ld, int T, int E, int k, const GateDev& g, int32_t* idx,
                       float* w, hipStream_t st, int32_t* k_used, float* entropy, int32_t* clear_word) {
  const int vpl = E <= 64 ? 1 : E <= 128 ? 2 : 4;
  // one load per lane where a row starts aligned to a lane's piece
  const int vec = E % vpl == 0 && ld % vpl == 0 && (reinterpret_cast<uintptr_t>(logits) % (vpl * lt_bytes(lt))) == 0;
  const unsigned grid = (unsigned)(((int64_t)T + 3) / 4);
  auto go = [&](auto kern) {
    return launch_kernel(kern, grid, 256, 0, st, logits, ld, vec, T, E, k, g, idx, w, k_used, entropy, clear_word);
  };
  auto pick = [&](auto lc) {
    constexpr int LT = decltype(lc)::value;
    return vpl == 1 ? go(gate_kernel<1, LT>) : vpl == 2 ? go(gate_kernel<2, LT>) : go(gate_kernel<4, LT>);
  };
  if (lt == GATE_F32) return pick(std::integral_constant<int, GATE_F32>{});
  if (lt == ACT_BF16) return pick(std::integral_constant<int, ACT_BF16>{});
  return pick(std::integral_constant<int, ACT_F16>{});
}

hipError_t launch_gate_backward(const void* logits, int lt, int64_t ld, int T, int E, int k, const GateDev& g,
                                const int32_t* idx, const float* dw, void* out, int64_t ldo, hipStream_t st) {
  const int vec = E % 4 == 0 && ldo % 4 == 0 && (reinterpret_cast<uintptr_t>(out) % (4 * lt_bytes(lt))) == 0;
  const unsigned grid = (unsigned)(((int64_t)T + 15) / 16);
  auto go = [&](auto kern) {
    return launch_kernel(kern, grid, 256, 0, st, logits, ld, T, E, k, g.score, g.renorm, g.scale, idx, dw, out, ldo,
                         vec);
  };
  if (lt == GATE_F32) return go(gate_backward_kernel<GATE_F32>);
  if (lt == ACT_BF16) return go(gate_backward_kernel<ACT_BF16>);
  return go(gate_backward_kernel<ACT_F16>);
}

}  // namespace moe
