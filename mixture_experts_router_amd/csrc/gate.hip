// The routing gate (softmax or sigmoid scores, a balancing bias, groups,
// top-k, renormalised weights) and its gradient.
//
//   s_e   = softmax(l)_e  or  1 / (1 + exp(-l_e))
//   key_e = s_e + b_e                       (no bias: the order of l itself)
//   a group of gs consecutive experts is worth the sum of its best one or two
//   keys; the group_k best groups stay; the k best keys among them are chosen,
//   the lower index first among equal keys
//   l_e = -inf masks e: s_e = 0 and key_e = -inf, whatever the bias; a key of
//   -inf or NaN adds nothing as a group's second best
//   for the order, a softmax leaves NaN logits out of its maximum and sum, and
//   takes its limit where there are logits of +inf
//   w_j   = c s_j,  or renormalised  c s_j / sum_r s_r   (sigmoid: + 1e-20)
//
// Which of two experts is chosen is decided as keys formed in 64 bits decide
// it, whatever the rounding of a 32-bit score: the selection runs on fp32
// keys, whose error is bounded below, and a token in which two keys that matter
// lie within that bound of each other is selected again with keys in fp64.
// Without a bias, and with groups ranked by their best expert, the logits give
// the order exactly and no score is formed for it.
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

__device__ __forceinline__ double value_of64(uint64_t key) {
  return __builtin_bit_cast(double, (key >> 63) != 0 ? key ^ 0x8000000000000000ull : ~key);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, true);
}

// maximum over the 16 lanes of a row, in every lane of it
__device__ __forceinline__ uint32_t max16_u(uint32_t v) {
  v = max(v, dpp_u<DPP_QUAD_1032, 0xF>(v));
  v = max(v, dpp_u<DPP_QUAD_2301, 0xF>(v));
  v = max(v, dpp_u<DPP_ROW_HALF_MIRROR, 0xF>(v));
  v = max(v, dpp_u<DPP_ROW_MIRROR, 0xF>(v));
  return v;
}

__device__ __forceinline__ void or16(uint32_t& v) {
  v |= dpp_u<DPP_QUAD_1032, 0xF>(v);
  v |= dpp_u<DPP_QUAD_2301, 0xF>(v);
  v |= dpp_u<DPP_ROW_HALF_MIRROR, 0xF>(v);
  v |= dpp_u<DPP_ROW_MIRROR, 0xF>(v);
}

// the next lane's value (0 past the row)
__device__ __forceinline__ uint32_t dpp_next(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x101, 0xF, 0xF, true);
}

__device__ __forceinline__ uint64_t lane_read64(uint64_t v, int src) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(src << 2, (int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute(src << 2, (int)(uint32_t)(v >> 32));
  return (uint64_t)hi << 32 | lo;
}

// maximum over the 64 lanes, in a scalar register
__device__ __forceinline__ uint32_t wave_max_key(uint32_t v) {
  v = max16_u(v);
  const uint32_t r0 = __builtin_amdgcn_readlane(v, 0), r1 = __builtin_amdgcn_readlane(v, 16);
  const uint32_t r2 = __builtin_amdgcn_readlane(v, 32), r3 = __builtin_amdgcn_readlane(v, 48);
  return max(max(r0, r1), max(r2, r3));
}

// the index of the largest 64-bit key, of equal ones the first lane's (indices
// grow with the lane): the high words' maximum, then the low words' among those
__device__ __forceinline__ int wave_best64(uint64_t key, int index) {
  const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
  const uint32_t m1 = wave_max_key(hi);
  const uint32_t m0 = wave_max_key(hi == m1 ? lo : 0u);
  return __builtin_amdgcn_readlane(index, (int)__builtin_ctzll(__ballot(hi == m1 && lo == m0)));
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll 1
  for (int off = 1; off < WAVE; off <<= 1)
    v += __builtin_bit_cast(double, lane_read64(__builtin_bit_cast(uint64_t, v), lane_id() ^ off));
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

__device__ __forceinline__ float sum16(float v) {
  v = sum8(v);
  return v + dpp_f<DPP_ROW_MIRROR>(v);
}

__device__ __forceinline__ float max16(float v) {
  v = max8(v);
  return fmaxf(v, dpp_f<DPP_ROW_MIRROR>(v));
}

__device__ __forceinline__ float sigmoid_f32(float l) { return 1.0f / (1.0f + expf(-l)); }

constexpr float SIGMOID_EPS = 1e-20f;  // added to the selected scores' sum

}  // namespace

// ------------------------------------------------------ the exact order --
//
// One wave, one token: the k experts by keys in fp64, lane s returning slot
// s's.  Taken only for tokens whose fp32 keys do not decide.  lds: one key per
// expert.
template <int VPL, int LT>
__device__ __forceinline__ int exact_experts(const void* __restrict__ logits, int64_t ld, int64_t t, int E, int k,
                                             const GateDev& g, uint64_t* __restrict__ lds) {
  const int lane = lane_id(), e0 = lane * VPL;
  // +inf lies far beyond every other logit, which makes the scores their limits
  auto finite = [](float l) { return l == INFINITY ? 1e300 : (double)l; };
  double d[VPL];
  float l[VPL], m = -__FLT_MAX__;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    l[j] = e0 + j < E ? load_logit<LT>(logits, t * ld + e0 + j) : -INFINITY;
    m = fmaxf(m, l[j]);  // passes over NaN
  }
  if (g.score == GATE_SOFTMAX) {
    const double top = finite(wave_max(m));
    double z = 0.0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      d[j] = exp(finite(l[j]) - top);
      z += __builtin_fmax(d[j], 0.0);  // NaN adds nothing
    }
    z = wave_sum64(z);
#pragma unroll
    for (int j = 0; j < VPL; ++j) d[j] = d[j] / z;  // z = 0 only where all are masked or NaN
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) d[j] = 1.0 / (1.0 + exp(-(double)l[j]));
  }
  uint64_t key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    if (g.bias && e0 + j < E) d[j] = d[j] + (double)g.bias[e0 + j];
    if (l[j] == -INFINITY) d[j] = -INFINITY;
    key[j] = e0 + j < E ? key_of64(d[j]) : 0ull;
  }
  if (g.groups > 1) {
    const int G = g.groups, gs = E / G;
    wave_lds_fence();
#pragma unroll
    for (int j = 0; j < VPL; ++j) lds[e0 + j] = key[j];
    wave_lds_fence();
    // `per` lanes a group (G <= 64) find its best two keys together
    int shift = 0;
    while (G << (shift + 1) <= WAVE) ++shift;
    const int per = 1 << shift, group = lane >> shift, part = lane & (per - 1);
    uint64_t b1 = 0, b2 = 0;
    if (group < G) {
#pragma unroll 4
      for (int i = part; i < gs; i += per) {
        const uint64_t u = lds[group * gs + i];
        b2 = max(b2, min(b1, u));
        b1 = max(b1, u);
      }
    }
#pragma unroll 1
    for (int off = 1; off < per; off <<= 1) {
      const uint64_t o1 = lane_read64(b1, lane ^ off), o2 = lane_read64(b2, lane ^ off);
      b2 = max(max(b2, o2), min(b1, o1));
      b1 = max(b1, o1);
    }
    double v = value_of64(b1);
    const double second = value_of64(b2);
    if (g.group_best == 2 && second > -INFINITY) v = v + second;
    uint64_t worth = group < G && part == 0 ? key_of64(v) : 0ull;
    uint64_t kept = 0;
#pragma unroll 1
    for (int s = 0; s < g.group_k; ++s) {
      const int win = wave_best64(worth, group);
      kept |= 1ull << win;
      if (group == win) worth = 0ull;
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j < E && !(kept >> ((e0 + j) / gs) & 1)) key[j] = 0ull;
  }
  int mine = 0;
#pragma unroll 1
  for (int s = 0; s < k; ++s) {
    uint64_t bk = 0;
    int bi = 64 * VPL;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (key[j] > bk) bk = key[j], bi = e0 + j;
    const int e = wave_best64(bk, bi);
    if (lane == s) mine = e;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j == e) key[j] = 0ull;
  }
  return mine;
}

// ------------------------------------------------------ sorting networks --
//
// A key and its place j < 16 in the lane as one double in [1, 2): the 32 key
// bits, then 15 - j, in the mantissa.  Larger key first, lower index first
// among equal keys is then the order of the doubles, and a comparator is
// v_max_f64 + v_min_f64 (full rate, like fp32).
__device__ __forceinline__ double pack_key(uint32_t key, int j) {
  const uint32_t hi = __builtin_amdgcn_alignbit(0x3FFu, key, 12), lo = (key << 20) | (uint32_t)(15 - j);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ void order2(double& a, double& b) {
  const double hi = __builtin_fmax(a, b), lo = __builtin_fmin(a, b);
  a = hi;
  b = lo;
}

// descending; 5 and 19 comparators
__device__ __forceinline__ void sort4(double* v) {
  order2(v[0], v[1]), order2(v[2], v[3]), order2(v[0], v[2]), order2(v[1], v[3]), order2(v[1], v[2]);
}

__device__ __forceinline__ void sort8(double* v) {
  sort4(v), sort4(v + 4);  // odd-even merge of the two halves
  order2(v[0], v[4]), order2(v[1], v[5]), order2(v[2], v[6]), order2(v[3], v[7]);
  order2(v[2], v[4]), order2(v[3], v[5]);
  order2(v[1], v[2]), order2(v[3], v[4]), order2(v[5], v[6]);
}

// ----------------------------------------------------------- the gate ---
//
// Sixteen lanes a token, four tokens a wave; lane i of a row holds the EPL
// consecutive experts i*EPL ... (EPL = 4, 8, 16 for up to 64, 128, 256
// experts).  Each lane sorts its keys once and keeps the best eight in LDS, so
// each of the k rounds compares sixteen list heads (eight DPP steps for the key
// and the lowest index) and one lane moves to its next, which is in registers
// already while the one after it is read.
//
// Bound by vector instructions: 850 a wave for 256 experts in groups with a
// bias (16 exponentials and reciprocals a lane; 110 for the sort; 300 for nine
// rounds), counted as 890 issue slots of four cycles, 24 us at 2.4 GHz of the
// 30.3 that 65536 tokens take (67 MB of logits: 10 us at the rate of a fill of
// that size).  A wave a token with 64-bit keys took 158 us.
//   65536 x 256, sigmoid, bias, 8 groups of two's worth  30.3 us  (2.3 TB/s); bf16, fp16 30.8, 30.2
//   65536 x 256, softmax, nothing else                   19.3 us  (3.7 TB/s); bf16, fp16 19.3, 19.4
//   65536 x 64, sigmoid, bias                            11.3 us
//   4096 x 64, sigmoid, bias  3.8 us;   64 x 256 in groups  4.8;   1 x 64  2.9
// (an empty kernel: 2.3 us).  A workgroup is one wave: groups of four run
// 0.4 us slower at 65536 tokens and 0.3 at 64, and 0.3 faster at 16384 x 64.  At
// least five waves a SIMD: six spill (8192 x 256 in groups 0.3 us slower), eight
// spill more (4 us slower at 65536).
//
// Where scores order the experts, the fp32 keys decide unless two that matter
// lie within the window of their error: two slots next to each other, the
// last slot and the best key left out, or the border of the kept groups.  Such
// a token is selected again by exact_experts, some 3 us of latency for its wave.
// Of fp32 logits around 0 with ordinary biases that are 0.1% or less at 256
// experts: 1.5 us of 4096 x 256 in groups, and of 65536.  An exact tie (equal
// logits, equal biases) between two slots needs no second look, nor does a group
// masked whole, whose worth is -inf; an exact tie at the last slot does, and so
// do the many close keys where sigmoids saturate, as the window is absolute.
// 65536 x 256, sigmoid, top-8:
//   fp32, 8 groups, bias                               30.3 us, a group masked 28.9
//   bf16, 8 groups, bias 30.8; bias 0 (many ties at the last slot)      43.6
//   bf16, no groups, bias 0                                             38.8
//   fp32, no groups, bias 0, logits around 0: 25.9; around -12: 49.8; around +8: 97.8
//
// Error bounds of the fp32 keys (u = 2^-24, products and sums rounded once,
// v_exp_f32 and v_rcp_f32 within one ulp, 2 u):
//   sigmoid: exp(-l) is off by (1.33 |l| + 2) u relative (the rounded product
//     with the rounded log2 e, then the exponential), which reaches s times
//     s (1 - s), and s (1 - s) |l| <= 0.224: 0.8 u; the sum 1 + e adds u s, the
//     reciprocal 2 u s: less than 4 u in all.
//   softmax: a term is off by (2.33 |d| + 2) u (the difference d is rounded
//     too), and p |d| <= 0.37 p_max; the sum by the same weighted with p, at
//     most 2.33 u ln 256 + 2 u, and 19 roundings; the reciprocal and the product
//     3 u: less than 40 u p_max.
//   the bias adds u |key|.
// KEY_ERR, SOFTMAX_ERR p_max and KEY_ROUND |key| are these with a margin.  Two
// keys further apart than the sum of their errors keep their order.
constexpr float KEY_ERR = 0x1.1p-22f, SOFTMAX_ERR = 0x1.48p-19f, KEY_ROUND = 0x1.1p-24f;
constexpr int GATE_PITCH = 260;         // LDS words a token holds its keys in
constexpr int GATE_WORDS = 9 * 64 * 2;  // LDS words: nine list entries a lane (the last is the end), four tokens' keys,
                                        // or one 64-bit key per expert of one token
static_assert(GATE_WORDS >= 4 * GATE_PITCH && GATE_WORDS >= 2 * 256, "LDS of a wave");

template <int EPL, int LT, bool by_score>
__global__ __launch_bounds__(64, 5) void gate_kernel(const void* __restrict__ logits, int64_t ld, int vec, int T, int E,
                                                   int k, GateDev g, int32_t* __restrict__ idx,
                                                   float* __restrict__ w, int32_t* __restrict__ k_used,
                                                   float* __restrict__ entropy, int32_t* __restrict__ clear_word) {
  __shared__ __attribute__((aligned(16))) uint32_t wlds[GATE_WORDS];
  constexpr int LL = EPL < 8 ? EPL : 8;  // a lane's list: at most MOE_MAX_K of its experts are chosen
  const int lane = lane_id(), i16 = lane % 16, r = lane / 16;
  const int64_t t0 = (int64_t)blockIdx.x * 4;
  const int64_t t = t0 + r;
  const bool tv = t < T;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (k_used) *k_used = k;
    if (entropy) *entropy = 0.0f;
    if (clear_word) *clear_word = 0;
  }
  const int e0 = i16 * EPL;
  float l[EPL], b[EPL];
  const int64_t at = (tv ? t : 0) * ld + e0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    l[j] = -INFINITY;
    b[j] = 0.0f;
  }
  if (vec) {  // E is a multiple of four
#pragma unroll
    for (int j = 0; j < EPL; j += 4)
      if (e0 + j < E) load_logits<LT, 4>(logits, at + j, l + j);
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e0 + j < E) l[j] = load_logit<LT>(logits, at + j);
  }
  if (g.bias) {
    if (E % 4 == 0 && (reinterpret_cast<uintptr_t>(g.bias) & 15u) == 0) {
#pragma unroll
      for (int j = 0; j < EPL; j += 4)
        if (e0 + j < E) load_logits<GATE_F32, 4>(g.bias, e0 + j, b + j);
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (e0 + j < E) b[j] = g.bias[e0 + j];
    }
  }

  // ---- keys
  const bool softmax = g.score == GATE_SOFTMAX;
  float m_all = 0.0f, z_all = 1.0f, key_err = KEY_ERR;  // softmax over all experts; sigmoid's error
  bool unsure = false;
  uint32_t key[EPL];
  if (softmax && (by_score || !g.renorm)) {
    float m = l[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) m = fmaxf(m, l[j]);
    m_all = max16(m);
    if (m_all == -INFINITY) m_all = 0.0f;  // every expert masked: all terms are 0
    float z = 0.0f, ex[EPL];
    if (g.renorm) {  // the probabilities only order the experts
#pragma unroll
      for (int j = 0; j < EPL; ++j) z += ex[j] = __expf(l[j] - m_all);
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) z += ex[j] = expf(l[j] - m_all);
    }
    z_all = sum16(z);
    if (z_all == 0.0f) z_all = 1.0f;
    const float rz = __builtin_amdgcn_rcpf(z_all);
    key_err = SOFTMAX_ERR * rz;
#pragma unroll
    for (int j = 0; j < EPL; ++j) b[j] = ex[j] * rz + b[j];
  } else if (by_score) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) b[j] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[j])) + b[j];
  }
  if (by_score) {
    // the score's sum is never -0 and its NaNs are left to the exact order, so
    // these keys need no canonical form
    float low = l[0], any = b[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) {
      low = fminf(low, l[j]);
      any += b[j];
    }
    unsure = any != any;
    if (__ballot(low == -INFINITY)) {  // masked experts (or lanes without any)
#pragma unroll
      for (int j = 0; j < EPL; ++j) b[j] = l[j] == -INFINITY ? -INFINITY : b[j];
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const uint32_t u = __builtin_bit_cast(uint32_t, b[j]);
      key[j] = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = key_of(l[j]);
  }
  if (E != 16 * EPL || t0 + 4 > T) {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e0 + j >= E || !tv) key[j] = 0u;
  }

  // ---- groups: a group's worth as a range [low, high] of keys, of which only
  // the order counts: kept if fewer than group_k others can be above it,
  // dropped if group_k others are
  auto range = [&](uint32_t best, uint32_t next, uint32_t& low, uint32_t& high) __attribute__((always_inline)) {
    low = high = best;
    if (!by_score || best == 0u) return;
    if (value_of(best) == -INFINITY) return;  // every expert masked (or its bias -inf): worth -inf, exactly
    float v = value_of(best), err = key_err + KEY_ROUND * fabsf(v);
    if (g.group_best == 2) {
      const float v2 = value_of(next);
      if (v2 != -INFINITY) {
        err = err + (key_err + KEY_ROUND * fabsf(v2));
        v = v + v2;
        err = err + KEY_ROUND * fabsf(v);
      }
    }
    err = err + 4.0f * KEY_ROUND * fabsf(v);  // the roundings of the range's own ends
    const float lo = v - err, hi = v + err;
    const bool sure = lo <= hi;  // NaN: anything is possible
    low = sure ? key_of(lo) : 1u;
    high = sure ? key_of(hi) : 0xFFFFFFFFu;
  };
  const int G = g.groups, gs = G > 1 ? E / G : 1;
  const int lanes = gs / EPL;  // lanes a group, where a group is whole lanes
  const bool whole = G > 1 && gs % EPL == 0 && (lanes & (lanes - 1)) == 0;
  if (G > 1 && !whole) {
    // any size: lanes take groups i16, i16 + 16, ... from LDS
    uint32_t* const row = wlds + r * GATE_PITCH;
#pragma unroll
    for (int j = 0; j < EPL; ++j) row[e0 + j] = key[j];
    wave_lds_fence();
    uint32_t low[4], high[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int gg = i16 + 16 * q;
      low[q] = high[q] = 0u;
      if (gg < G) {
        uint32_t best = 0u, next = 0u;
        for (int i = 0; i < gs; ++i) {
          const uint32_t u = row[gg * gs + i];
          next = max(next, min(best, u));
          best = max(best, u);
        }
        range(best, next, low[q], high[q]);
      }
    }
    wave_lds_fence();
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i16 + 16 * q < G) {
        row[2 * (i16 + 16 * q)] = low[q];
        row[2 * (i16 + 16 * q) + 1] = high[q];
      }
    wave_lds_fence();
    uint64_t kept = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int gg = i16 + 16 * q;
      if (gg < G) {
        int may = 0, must = 0;
        for (int h = 0; h < G; ++h) {
          const uint32_t hl = row[2 * h], hh = row[2 * h + 1];
          may += by_score ? (int)(hh >= low[q]) & (int)(h != gg)
                          : (int)(hh > low[q]) | ((int)(hh == low[q]) & (int)(h < gg));
          must += by_score ? (int)(hl > high[q]) : 0;
        }
        if (may < g.group_k) kept |= 1ull << gg;
        else if (by_score && must < g.group_k) unsure = true;
      }
    }
    uint32_t k0 = (uint32_t)kept, k1 = (uint32_t)(kept >> 32);
    or16(k0);
    or16(k1);
    kept = (uint64_t)k1 << 32 | k0;
    // e / gs for e < 256 and gs <= 128
    const uint32_t inv = (65536u + gs - 1) / gs;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (!(kept >> (((uint32_t)(e0 + j) * inv) >> 16 & 63u) & 1)) key[j] = 0u;
  }

  // ---- each lane's experts in order
  double list[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) list[j] = pack_key(key[j], j);
  if constexpr (EPL == 4) {
    sort4(list);
  } else {
    sort8(list);
    if constexpr (EPL == 16) {  // the best eight of two sorted eights
      sort8(list + 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) list[j] = __builtin_fmax(list[j], list[15 - j]);
#pragma unroll
      for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((j & d) == 0) order2(list[j], list[j + d]);
    }
  }
  auto key_in = [](double d) { return (uint32_t)(__builtin_bit_cast(uint64_t, d) >> 20); };
  auto expert_in = [e0](double d) {  // 256 - e = 256 - e0 - j
    return ((uint32_t)__builtin_bit_cast(uint64_t, d) & 15u) + (uint32_t)(241 - e0);
  };

  bool dropped = false;
  if (whole) {
    uint32_t best = key_in(list[0]), next = key_in(list[1]);
    auto join = [&](uint32_t ob, uint32_t on) __attribute__((always_inline)) {
      next = max(min(best, ob), max(next, on));
      best = max(best, ob);
    };
    if (lanes > 1) join(dpp_u<DPP_QUAD_1032, 0xF>(best), dpp_u<DPP_QUAD_1032, 0xF>(next));
    if (lanes > 2) join(dpp_u<DPP_QUAD_2301, 0xF>(best), dpp_u<DPP_QUAD_2301, 0xF>(next));
    if (lanes > 4) join(dpp_u<DPP_ROW_HALF_MIRROR, 0xF>(best), dpp_u<DPP_ROW_HALF_MIRROR, 0xF>(next));
    uint32_t low, high;
    range(best, next, low, high);
    int may = 0, must = 0;
    auto rival = [&](int n, uint32_t hl, uint32_t hh) __attribute__((always_inline)) {
      // without ranges the lower group wins a tie: n lanes back is lower unless it wrapped
      may += by_score ? (int)(hh >= low) : (int)(hh > low) | ((int)(hh == low) & (int)(n <= i16));
      must += by_score ? (int)(hl > high) : 0;
    };
    // the other groups of the row, one turn of `lanes` at a time (lanes without
    // experts hold 0, below every key)
#define MOE_GATE_TURN(n) \
  if (((n) & (lanes - 1)) == 0) rival(n, dpp_u<0x120 + (n), 0xF>(low), dpp_u<0x120 + (n), 0xF>(high))
    MOE_GATE_TURN(1);
    MOE_GATE_TURN(2);
    MOE_GATE_TURN(3);
    MOE_GATE_TURN(4);
    MOE_GATE_TURN(5);
    MOE_GATE_TURN(6);
    MOE_GATE_TURN(7);
    MOE_GATE_TURN(8);
    MOE_GATE_TURN(9);
    MOE_GATE_TURN(10);
    MOE_GATE_TURN(11);
    MOE_GATE_TURN(12);
    MOE_GATE_TURN(13);
    MOE_GATE_TURN(14);
    MOE_GATE_TURN(15);
#undef MOE_GATE_TURN
    unsure |= by_score && may >= g.group_k && must < g.group_k && best != 0u;
    dropped = may >= g.group_k;
  }

  // ---- the k best keys, and with scores the best one left out: lane s keeps slot s
  uint32_t mine = 0u;
  int me = 0;
  const int last = by_score ? k : k - 1;
  u32x2* const entry = (u32x2*)wlds + lane;  // entry j of this lane at entry[64 * j]
  wave_lds_fence();
#pragma unroll
  for (int j = 1; j < LL; ++j) entry[64 * j] = u32x2{dropped ? 0u : key_in(list[j]), expert_in(list[j])};
  entry[64 * LL] = u32x2{0u, 0u};
  wave_lds_fence();
  uint32_t hk = dropped ? 0u : key_in(list[0]), hc = expert_in(list[0]);
  const bool more = EPL > LL && !dropped && key_in(list[LL - 1]) != 0u;  // the lane may hold more keys than its list
  int next = 64;
#pragma unroll 1
  for (int s = 0; s <= last; ++s) {
    const u32x2 after = entry[next];
    const uint32_t m = max16_u(hk);
    const uint32_t c = max16_u(hk == m ? hc : 0u);  // the lowest index: the largest 256 - e
    if (i16 == s) {
      mine = m;
      me = 256 - (int)c;
    }
    const bool taken = hc == c;  // an expert is in one list
    hk = taken ? after.x : hk;
    hc = taken ? after.y : hc;
    next = min(next + (taken ? 64 : 0), 64 * LL);
  }
  unsure |= more && hk == 0u;  // eight chosen from one lane: its ninth was not looked at

  const bool held = tv && i16 <= last && mine != 0u;
  float ls = held ? load_logit<LT>(logits, t * ld + me) : 0.0f;
  if (by_score) {
    const float bs = held && g.bias ? g.bias[me] : 0.0f;
    // read from the next lane by every lane of the row: never behind a condition,
    // which would switch the lane that is read off
    const uint32_t after = dpp_next(mine);
    const float v = value_of(mine), nv = value_of(after);
    const float nl = __builtin_bit_cast(float, dpp_next(__builtin_bit_cast(uint32_t, ls)));
    const float nb = __builtin_bit_cast(float, dpp_next(__builtin_bit_cast(uint32_t, bs)));
    const bool rival = i16 < k && after != 0u;
    const bool apart = v - nv > 2.0f * (key_err + KEY_ROUND * fabsf(v));  // false for NaN and infinities
    const bool tie = i16 + 1 < k && ls == nl && (bs == nb || ls == -INFINITY);
    uint64_t again = __ballot(tv && ((rival && !apart && !tie) || unsure));
    while (again) {
      const int rr = (int)__builtin_ctzll(again) / 16;
      again &= ~(0xFFFFull << (16 * rr));
      const int e = exact_experts<EPL / 4, LT>(logits, ld, t0 + rr, E, k, g, (uint64_t*)wlds);
      const int mv = __builtin_amdgcn_ds_bpermute(i16 << 2, e);
      if (r == rr && i16 < k) {
        me = mv;
        ls = load_logit<LT>(logits, t * ld + me);
      }
    }
  }

  // ---- weights of slot i16 (lanes k..15 add nothing)
  const bool on = tv && i16 < k;
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
  } else {
    const float s1 = on ? sigmoid_f32(ls) : 0.0f;
    wt = g.renorm ? s1 / (sum8(s1) + SIGMOID_EPS) : s1;
  }
  wt = masked ? 0.0f : wt;  // also beside a NaN
  if (on) {
    idx[t * k + i16] = me;
    w[t * k + i16] = g.scale * wt;
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
// whole, so the kernel is bound by the [T, E] gradient's bytes (65536 x 256
// fp32, 67 MB: 18 us, 3.7 TB/s written beside the selected logits' lines; 25 us
// with stores that stay in the caches; bf16 12.7, fp16 11.9).  Only the dense
// form reads every logit, three times and one a load, and forms each exponential
// twice: 65536 x 256 in 47 us (fp32; 27 by its bytes), 40 (bf16), 39 (fp16).
// 1 - s is formed as 1 / (1 + exp(l)).
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
    m = max16(m);
    if (tv) {
      for (int x = i16; x < E; x += 16) {
        const float v = load_logit<LT>(logits, t * ld + x);
        z += v == -INFINITY ? 0.0f : expf(v - m);
      }
    }
    z = sum16(z);
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
        __builtin_nontemporal_store(v, (f32x4*)((float*)out + t * ldo + x));
      } else {
        u32x2 o;
        o.x = (uint32_t)f32_to_act_bits(v.x, LT) | (uint32_t)f32_to_act_bits(v.y, LT) << 16;
        o.y = (uint32_t)f32_to_act_bits(v.z, LT) | (uint32_t)f32_to_act_bits(v.w, LT) << 16;
        __builtin_nontemporal_store(o, (u32x2*)((uint16_t*)out + t * ldo + x));
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
  // four logits a load where rows start aligned to that
  const int vec = E % 4 == 0 && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) % (4 * lt_bytes(lt))) == 0;
  const unsigned grid = (unsigned)(((int64_t)T + 3) / 4);
  auto go = [&](auto kern) {
    return launch_kernel(kern, grid, 64, 0, st, logits, ld, vec, T, E, k, g, idx, w, k_used, entropy, clear_word);
  };
  // a bias, or groups ranked by two experts, order by scores; else the logits do
  // (65536 x 256: 30 against 20 us)
  const bool by_score = g.bias != nullptr || (g.groups > 1 && g.group_best == 2);
  auto size = [&](auto lc, auto sc) {
    constexpr int LT = decltype(lc)::value;
    constexpr bool S = decltype(sc)::value;
    return E <= 64 ? go(gate_kernel<4, LT, S>) : E <= 128 ? go(gate_kernel<8, LT, S>) : go(gate_kernel<16, LT, S>);
  };
  auto pick = [&](auto lc) { return by_score ? size(lc, std::true_type{}) : size(lc, std::false_type{}); };
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
