// Balance loss of the routing, the experts' counts, and the gradient (gfx950).
//
//   p_te   = softmax(l_t)_e  or  s_te / (sum_j s_tj + 1e-20), s = 1 / (1 + exp(-l))
//   over the n live tokens of a sequence:
//   counts_e = pairs (t, slot) routed to e,  prob_e = mean p_te
//   loss     = E / (k n) sum_e counts_e prob_e
//   z        = mean (log sum_e exp l_te)^2                    (softmax)
//   d loss / d l_tj = p_j (g_j - sum_e g_e p_e),  g_e = E / (k n^2) counts_e   (sigmoid: times 1 - s_j)
//   d z / d l_tj    = 2 / n lse_t p_j
//
// A logit of -inf has probability 0 and no gradient, also in a row that holds
// nothing else, which adds nothing to prob and z.  Sums are fp32 per workgroup
// and joined in a fixed order; the last sums of a sequence are 64 bits.
//
// Sixteen lanes a token as in the gate, so a row is read once in whole lines and
// its maximum and sum are DPP steps.  65536 x 256 fp32 logits are 67 MB: 17.2 us
// (3.9 TB/s) and 4.5 us for the join of 512 chunks; the gradient reads and writes
// them, 134 MB in 30 us (4.5 TB/s; a copy reaches 5.1).  Short batches are a
// chain of latencies.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr float SCORE_EPS = 1e-20f;

// Sums of one chunk and sequence: prob sums, counts (each E rounded up to 4), z sum, tokens
__host__ __device__ constexpr int slot_words(int E) { return 2 * ((E + 3) / 4 * 4) + 4; }

// tokens of a chunk: at most 512 chunks, two workgroups a CU
int chunk_tokens(int T) {
  const int64_t c = ((int64_t)T + 511) / 512;
  return (int)((c + 31) / 32 * 32);
}

// One launch, a workgroup a sequence, for few tokens: 512 x 32 in 7.2 us of
// kernels and 9.2 us a call, against 3.6 and 3.8 us and 13.1 us a call in two.
// More tokens need more CUs (1237 x 160 in nine sequences: 17.1 us against 12.3
// and 4.0).
bool whole_sequences(int T) { return T <= 512; }

constexpr float LOG2E = 1.44269504088896341f, LN2 = 0.69314718055994531f;

template <int LT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (LT == GATE_F32) return ((const float*)p)[i];
  else return act_to_f32(((const uint16_t*)p)[i], LT);
}

template <int LT>
__device__ __forceinline__ f32x4 load_logits4(const void* p, int64_t i) {
  if constexpr (LT == GATE_F32) {
    return *(const f32x4*)((const float*)p + i);
  } else {
    const u32x2 v = *(const u32x2*)((const uint16_t*)p + i);
    return f32x4{act_to_f32(v.x & 0xFFFFu, LT), act_to_f32(v.x >> 16, LT), act_to_f32(v.y & 0xFFFFu, LT),
                 act_to_f32(v.y >> 16, LT)};
  }
}

// over the 16 lanes of a row, in every lane of it
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, dpp_f<DPP_QUAD_1032>(v));
  v = fmaxf(v, dpp_f<DPP_QUAD_2301>(v));
  v = fmaxf(v, dpp_f<DPP_ROW_HALF_MIRROR>(v));
  return fmaxf(v, dpp_f<DPP_ROW_MIRROR>(v));
}

__device__ __forceinline__ float sum16(float v) {
  v += dpp_f<DPP_QUAD_1032>(v);
  v += dpp_f<DPP_QUAD_2301>(v);
  v += dpp_f<DPP_ROW_HALF_MIRROR>(v);
  return v + dpp_f<DPP_ROW_MIRROR>(v);
}

// Expert of element j of register block c of lane i: 64 c + 4 i + j.  Lanes
// past E, and rows that are not live, hold -inf.
template <int LT, int NB>
__device__ __forceinline__ void load_row(const void* logits, int64_t at, int E, int vec, bool live, int i16,
                                         f32x4 (&l)[NB]) {
#pragma unroll
  for (int c = 0; c < NB; ++c) {
    const int x = 64 * c + 4 * i16;
    l[c] = f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (!live || x >= E) continue;
    if (vec) {
      l[c] = load_logits4<LT>(logits, at + x);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (x + j < E) l[c][j] = load_logit<LT>(logits, at + x + j);
    }
  }
}

// Scores of a row in place of its logits, without their sum's division: the
// exponentials over their maximum, or the sigmoids (GRAD: 1 - s in q).  inv:
// what makes them probabilities, by mul0: a masked expert's are 0 also beside
// NaN.  Returns the softmax's lse (0 for a row that masks everything).
//
// The hardware's exponential and logarithm to base 2, after the maximum is taken
// off (l may be any float): (l - m) log2(e) is off by about |l - m| 2^-23.
template <int NB, bool SOFTMAX, bool GRAD>
__device__ __forceinline__ float scores(f32x4 (&l)[NB], f32x4 (&q)[NB], float& inv) {
  float sum = 0.0f;
  if constexpr (SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int c = 0; c < NB; ++c) m = fmaxf(m, fmaxf(fmaxf(l[c].x, l[c].y), fmaxf(l[c].z, l[c].w)));
    m = max16(m);
    m = m == -INFINITY ? 0.0f : m;  // nothing but masked experts, or NaN (fmaxf passes it over)
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        l[c][j] = __builtin_amdgcn_exp2f((l[c][j] - m) * LOG2E);
        sum += l[c][j];
      }
    sum = sum16(sum);
    inv = __builtin_amdgcn_rcpf(sum);
    return sum == 0.0f ? 0.0f : m + __builtin_amdgcn_logf(sum) * LN2;  // a NaN's sum is NaN
  } else {
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = l[c][j] * LOG2E;
        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v));  // exactly 0 at -inf
        if constexpr (GRAD) q[c][j] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v));
        l[c][j] = s;
        sum += s;
      }
    sum = sum16(sum) + SCORE_EPS;
    inv = __builtin_amdgcn_rcpf(sum);
    return 0.0f;
  }
}

// A row whose sum is NaN (a NaN or +inf logit): NaN for every expert that is not
// masked, also where its exponential had vanished
template <int LT, int NB>
__device__ __forceinline__ void spread_nan(const void* logits, int64_t at, int E, int vec, int i16, f32x4 (&p)[NB]) {
  load_row<LT, NB>(logits, at, E, vec, true, i16, p);
#pragma unroll
  for (int c = 0; c < NB; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) p[c][j] = p[c][j] == -INFINITY ? 0.0f : NAN;
}

// first sequence that ends after token t: offsets[s] <= t < offsets[s + 1] if the token is in one
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int64_t t) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (int)(((unsigned)lo + (unsigned)hi) / 2u);
    if (offsets[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// The same for a token that the whole wave asks for: 64 probes at a time
__device__ __forceinline__ int sequence_of_wave(const int32_t* offsets, int S, int64_t t) {
  int lo = 0, span = S;
  while (span > 0) {
    const int step = (span + 63) / 64;
    const int at = lo + lane_id() * step;
    const int before = (int)__builtin_popcountll(__ballot(at < lo + span && offsets[min(at, S - 1) + 1] <= t));
    if (before == 0) break;
    const int end = lo + span;
    lo += (before - 1) * step + 1;
    span = min(step - 1, end - lo);
  }
  return lo;
}

// What a workgroup sums of consecutive tokens
template <int WAVES>
struct Sums {
  float prob[WAVES][256];
  int hist[256];
  float z[WAVES];
  int n[WAVES];
};

// The tokens [from, to): sums of the probabilities by wave, counts, z and live
// tokens.  Sixteen lanes a token, the next token's logits loaded before the
// present one's are used.  Ends with a barrier.
template <int NB, int LT, bool SOFTMAX, int WAVES>
__device__ __forceinline__ void sum_tokens(const void* logits, int64_t ld, int vec, int E, int k, const int32_t* idx,
                                           const uint8_t* mask, int64_t from, int64_t to, Sums<WAVES>& out) {
  constexpr int THREADS = 64 * WAVES, ROWS = 4 * WAVES;
  const int tid = threadIdx.x, lane = lane_id(), wave = wave_id(), i16 = lane % 16;
  if (tid < 256) out.hist[tid] = 0;
  int64_t t = from + tid / 16;
  bool live = t < to && (!mask || mask[t] != 0);
  f32x4 p[NB], q[NB], next[NB];
  load_row<LT, NB>(logits, t * ld, E, vec, live, i16, next);
  __syncthreads();
  for (int64_t i = from * k + tid; i < to * k; i += THREADS) {
    const int e = idx[i];
    if (e >= 0 && e < E && (!mask || mask[i / k] != 0)) atomicAdd(&out.hist[e], 1);
  }
  f32x4 acc[NB];
#pragma unroll
  for (int c = 0; c < NB; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float za = 0.0f;
  int n = 0;
  for (int64_t t0 = from; t0 < to; t0 += ROWS) {
    n += live;
#pragma unroll
    for (int c = 0; c < NB; ++c) p[c] = next[c];
    const int64_t at = t * ld;
    t += ROWS;
    live = t < to && (!mask || mask[t] != 0);
    load_row<LT, NB>(logits, t * ld, E, vec, live, i16, next);
    float inv;
    const float lse = scores<NB, SOFTMAX, false>(p, q, inv);
    if (inv != inv) spread_nan<LT, NB>(logits, at, E, vec, i16, p);
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[c][j] += mul0(p[c][j], inv);
    za += lse * lse;
  }
  // the four rows of a wave
#pragma unroll
  for (int c = 0; c < NB; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v = acc[c][j];
      v += lane_read_f(v, lane ^ 16);
      v += lane_read_f(v, lane ^ 32);
      if (lane < 16) out.prob[wave][64 * c + 4 * i16 + j] = v;
    }
  za += lane_read_f(za, lane ^ 16);
  za += lane_read_f(za, lane ^ 32);
  n += __shfl_xor(n, 16, WAVE);
  n += __shfl_xor(n, 32, WAVE);
  if (lane == 0) {
    out.z[wave] = za;
    out.n[wave] = n;
  }
  __syncthreads();
}

struct BalanceOut {
  float* loss;
  float* z;
  float* prob;
  int32_t* counts;
  int32_t* tokens;
};

// Results of sequence s from its sums: thread e has expert e's (0 past E).
// Every thread calls it; means and the loss's sum in 64 bits.
__device__ __forceinline__ void finish_sequence(const BalanceOut& o, int s, int E, int k, float prob, int count,
                                                double z, int n, double (&part)[4]) {
  const int tid = threadIdx.x;
  if (tid < 256) {
    double d = 0.0;
    if (tid < E) {
      const double mean = n ? (double)prob / n : 0.0;
      if (o.prob) o.prob[(int64_t)s * E + tid] = (float)mean;
      o.counts[(int64_t)s * E + tid] = count;
      d = count ? (double)count * mean : 0.0;
    }
    for (int i = 1; i < 64; i <<= 1) d += __shfl_xor(d, i, WAVE);
    if (tid % 64 == 0) part[tid / 64] = d;
  }
  __syncthreads();
  if (tid == 0) {
    o.loss[s] = n ? (float)((((part[0] + part[1]) + part[2]) + part[3]) * E / ((double)k * n)) : 0.0f;
    if (o.z) o.z[s] = n ? (float)(z / n) : 0.0f;
    o.tokens[s] = n;
  }
}

// A workgroup a sequence
template <int NB, int LT, bool SOFTMAX>
__global__ __launch_bounds__(1024) void balance_whole_kernel(const void* __restrict__ logits, int64_t ld, int vec,
                                                             int T, int E, int k, const int32_t* __restrict__ idx,
                                                             BalanceDev b, BalanceOut o) {
  __shared__ Sums<16> sums;
  __shared__ double part[4];
  const int s = blockIdx.x, tid = threadIdx.x;
  int64_t from = 0, to = T;
  if (b.offsets) {
    from = max((int64_t)0, (int64_t)b.offsets[s]);
    to = min((int64_t)T, (int64_t)b.offsets[s + 1]);
  }
  sum_tokens<NB, LT, SOFTMAX, 16>(logits, ld, vec, E, k, idx, b.mask, from, to, sums);
  float prob = 0.0f;
  double z = 0.0;
  int n = 0;
  if (tid < E)
    for (int w = 0; w < 16; ++w) prob += sums.prob[w][tid];
  for (int w = 0; w < 16; ++w) {
    z += sums.z[w];
    n += sums.n[w];
  }
  finish_sequence(o, s, E, k, prob, tid < E ? sums.hist[tid] : 0, z, n, part);
}

// A workgroup sums the chunk [lo, hi) of tokens, each sequence in it into a
// slot of its own: chunk c and sequence s meet at most once on the way
// through both, so c + s names the slot.  The gridDim.y workgroups of a chunk
// take its sequences by turns (a sequence is a chain of latencies, some 4 us).
template <int NB, int LT, bool SOFTMAX>
__global__ __launch_bounds__(512) void balance_part_kernel(const void* __restrict__ logits, int64_t ld, int vec, int T,
                                                           int E, int k, const int32_t* __restrict__ idx, BalanceDev b,
                                                           int chunk, float* __restrict__ slots) {
  __shared__ Sums<8> sums;
  const int tid = threadIdx.x;
  const int64_t lo = (int64_t)blockIdx.x * chunk, hi = min((int64_t)T, lo + chunk);
  const int words = slot_words(E), padded = (E + 3) / 4 * 4;
  int s = b.offsets ? sequence_of_wave(b.offsets, b.S, lo) : 0;
  for (s += blockIdx.y; s < b.S; s += gridDim.y) {
    const int64_t from = b.offsets ? max(lo, (int64_t)b.offsets[s]) : lo;
    const int64_t to = b.offsets ? min(hi, (int64_t)b.offsets[s + 1]) : hi;
    if (from >= hi) break;
    if (from >= to) continue;
    sum_tokens<NB, LT, SOFTMAX, 8>(logits, ld, vec, E, k, idx, b.mask, from, to, sums);
    float* slot = slots + ((int64_t)blockIdx.x + s) * words;
    if (tid < padded) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) v += sums.prob[w][tid];
      slot[tid] = v;
      ((int*)slot)[padded + tid] = sums.hist[tid];
    }
    if (tid == 0) {
      float v = 0.0f;
      int m = 0;
      for (int w = 0; w < 8; ++w) {
        v += sums.z[w];
        m += sums.n[w];
      }
      slot[2 * padded] = v;
      ((int*)slot)[2 * padded + 1] = m;
    }
    __syncthreads();
  }
}

// A workgroup a sequence: its slots in order of the sixteen waves' shares, four
// experts a lane
__global__ __launch_bounds__(1024) void balance_join_kernel(const float* __restrict__ slots, int T, int E, int k,
                                                            BalanceDev b, int chunk, BalanceOut o) {
  __shared__ f32x4 psum[16][64];
  __shared__ int csum[16][256];
  __shared__ double zsum[16];
  __shared__ int nsum[16];
  __shared__ double part[4];
  const int s = blockIdx.x, tid = threadIdx.x, lane = lane_id(), wave = wave_id();
  const int words = slot_words(E), padded = (E + 3) / 4 * 4;
  int64_t from = 0, to = T;
  if (b.offsets) {
    from = max((int64_t)0, (int64_t)b.offsets[s]);
    to = min((int64_t)T, (int64_t)b.offsets[s + 1]);
  }
  const int64_t c0 = from / chunk, c1 = from < to ? (to - 1) / chunk + 1 : c0;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  int c[4] = {0, 0, 0, 0};
  if (4 * lane < E) {
#pragma unroll 8
    for (int64_t i = c0 + wave; i < c1; i += 16) {
      const float* slot = slots + (i + s) * words + 4 * lane;
      const f32x4 a = *(const f32x4*)slot;
      const u32x4 h = *(const u32x4*)(slot + padded);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] += a[j];
        c[j] += (int)h[j];
      }
    }
  }
  psum[wave][lane] = v;
#pragma unroll
  for (int j = 0; j < 4; ++j) csum[wave][4 * lane + j] = c[j];
  double zs = 0.0;
  int n = 0;
  for (int64_t i = c0 + tid; i < c1; i += 1024) {
    const float* slot = slots + (i + s) * words + 2 * padded;
    zs += slot[0];
    n += ((const int*)slot)[1];
  }
  for (int i = 1; i < 64; i <<= 1) {
    zs += __shfl_xor(zs, i, WAVE);
    n += __shfl_xor(n, i, WAVE);
  }
  if (lane == 0) {
    zsum[wave] = zs;
    nsum[wave] = n;
  }
  __syncthreads();
  float prob = 0.0f;
  int count = 0;
  zs = 0.0;
  n = 0;
  if (tid < E)
    for (int w = 0; w < 16; ++w) {
      prob += ((const float*)psum[w])[tid];
      count += csum[w][tid];
    }
  for (int w = 0; w < 16; ++w) {
    zs += zsum[w];
    n += nsum[w];
  }
  finish_sequence(o, s, E, k, prob, count, zs, n, part);
}

// The gradient.  A workgroup takes `rows` tokens, sixteen at a time and the next
// ones' logits loaded before; a row of lanes keeps its sequence's slopes while
// its tokens stay in it.  Bound by the logits read and the gradient written.
template <int NB, int LT, bool SOFTMAX>
__global__ __launch_bounds__(256) void balance_backward_kernel(const void* __restrict__ logits, int64_t ld, int vec,
                                                               int T, int E, int k, BalanceDev b, int rows,
                                                               const int32_t* __restrict__ counts,
                                                               const int32_t* __restrict__ tokens,
                                                               const float* __restrict__ grad_loss,
                                                               const float* __restrict__ grad_z,
                                                               void* __restrict__ out, int64_t ldo, int vec_out) {
  const int lane = lane_id(), i16 = lane % 16;
  int64_t t = (int64_t)blockIdx.x * rows + threadIdx.x / 16;
  const int64_t end = min((int64_t)T, (int64_t)(blockIdx.x + 1) * rows);
  f32x4 p[NB], q[NB], g[NB], next[NB];
  bool on = t < end && (!b.mask || b.mask[t] != 0);
  load_row<LT, NB>(logits, t * ld, E, vec, on, i16, next);
  int s = -1;
  int64_t s_from = 0, s_to = b.offsets ? 0 : T;  // tokens of the sequence whose slopes are held
  float slope = 0.0f, zslope = 0.0f;
  if (!b.offsets) s = 0;
  bool fresh = !b.offsets;
  for (; t < end; t += 16) {
    const bool was = on;
#pragma unroll
    for (int c = 0; c < NB; ++c) p[c] = next[c];
    const int64_t t2 = t + 16;
    on = t2 < end && (!b.mask || b.mask[t2] != 0);
    load_row<LT, NB>(logits, t2 * ld, E, vec, on, i16, next);
    if (b.offsets && (t >= s_to || s < 0)) {
      s = sequence_of(b.offsets, b.S, t);
      s_from = s < b.S ? b.offsets[s] : (int64_t)T;
      s_to = s < b.S ? b.offsets[s + 1] : (int64_t)T;
      fresh = true;
    }
    if (fresh) {
      const int n = s < b.S ? tokens[s] : 0;
      const float nf = (float)n;
      slope = n > 0 && grad_loss ? grad_loss[s] * ((float)E / ((float)k * nf * nf)) : 0.0f;
      zslope = SOFTMAX && n > 0 && grad_z ? grad_z[s] * (2.0f / nf) : 0.0f;
#pragma unroll
      for (int c = 0; c < NB; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int x = 64 * c + 4 * i16 + j;
          g[c][j] = n > 0 && x < E ? slope * (float)counts[(int64_t)s * E + x] : 0.0f;
        }
      fresh = false;
    }
    const bool live = was && t >= s_from && t < s_to;
    float inv;
    const float lse = scores<NB, SOFTMAX, true>(p, q, inv);
    if (inv != inv) spread_nan<LT, NB>(logits, t * ld, E, vec, i16, p);
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[c][j] = mul0(p[c][j], inv);
        dot = __builtin_fmaf(g[c][j], p[c][j], dot);
      }
    dot = sum16(dot);
    const float add = zslope * lse - dot;
#pragma unroll
    for (int c = 0; c < NB; ++c) {
      const int x = 64 * c + 4 * i16;
      if (x >= E) continue;
      f32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float d = mul0(p[c][j], g[c][j] + add);
        if (!SOFTMAX) d *= q[c][j];
        v[j] = live ? d : 0.0f;
      }
      if (vec_out) {
        if constexpr (LT == GATE_F32) {
          __builtin_nontemporal_store(v, (f32x4*)((float*)out + t * ldo + x));
        } else {
          u32x2 o;
          o.x = (uint32_t)f32_to_act_bits(v.x, LT) | (uint32_t)f32_to_act_bits(v.y, LT) << 16;
          o.y = (uint32_t)f32_to_act_bits(v.z, LT) | (uint32_t)f32_to_act_bits(v.w, LT) << 16;
          __builtin_nontemporal_store(o, (u32x2*)((uint16_t*)out + t * ldo + x));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (x + j < E) {
            if constexpr (LT == GATE_F32) ((float*)out)[t * ldo + x + j] = v[j];
            else ((uint16_t*)out)[t * ldo + x + j] = f32_to_act_bits(v[j], LT);
          }
      }
    }
  }
}

// ------------------------------------------------------------- launchers --

int rows_vec(const void* p, int lt, int E, int64_t ld) {
  const int bytes = lt == GATE_F32 ? 4 : 2;
  return E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * bytes) == 0;
}

// go(IC<register blocks>, IC<logit type>, softmax) for the call's experts, type and score
template <typename F>
hipError_t dispatch(int E, int lt, int score, F&& go) {
  auto by_score = [&](auto nb, auto l) {
    return score == GATE_SOFTMAX ? go(nb, l, std::true_type{}) : go(nb, l, std::false_type{});
  };
  auto by_type = [&](auto nb) {
    if (lt == GATE_F32) return by_score(nb, std::integral_constant<int, GATE_F32>{});
    if (lt == ACT_BF16) return by_score(nb, std::integral_constant<int, ACT_BF16>{});
    return by_score(nb, std::integral_constant<int, ACT_F16>{});
  };
  return E <= 64    ? by_type(std::integral_constant<int, 1>{})
         : E <= 128 ? by_type(std::integral_constant<int, 2>{})
                    : by_type(std::integral_constant<int, 4>{});
}

}  // namespace

int64_t balance_ws_bytes(int T, int E, int S) {
  if (whole_sequences(T)) return 0;
  const int chunk = chunk_tokens(T);
  return (((int64_t)T + chunk - 1) / chunk + S) * slot_words(E) * 4;
}

hipError_t launch_balance(const void* logits, int lt, int64_t ld, int T, int E, int k, const int32_t* idx,
                          const BalanceDev& b, float* loss, float* z, float* prob, int32_t* counts, int32_t* tokens,
                          void* ws, hipStream_t st) {
  const int vec = rows_vec(logits, lt, E, ld);
  const BalanceOut o{loss, z, prob, counts, tokens};
  const bool whole = whole_sequences(T);
  const int chunk = whole ? 1 : chunk_tokens(T);
  const unsigned chunks = (unsigned)((T + (int64_t)chunk - 1) / chunk);
  const unsigned turns = whole ? 1u : std::max(1u, std::min({512u / chunks, (unsigned)b.S, 8u}));
  note_launch(whole ? "balance_whole" : "balance_part");
  const hipError_t r = dispatch(E, lt, b.score, [&](auto nb, auto l, auto softmax) {
    constexpr int NB = decltype(nb)::value, LT = decltype(l)::value;
    constexpr bool SM = decltype(softmax)::value;
    if (whole)
      return launch_kernel(balance_whole_kernel<NB, LT, SM>, (unsigned)b.S, 1024, 0, st, logits, ld, vec, T, E, k, idx,
                           b, o);
    return launch_kernel(balance_part_kernel<NB, LT, SM>, dim3(chunks, turns), 512, 0, st, logits, ld, vec, T, E, k,
                         idx, b, chunk, (float*)ws);
  });
  if (r != hipSuccess || whole) return r;
  note_launch("balance_join");
  return launch_kernel(balance_join_kernel, (unsigned)b.S, 1024, 0, st, (const float*)ws, T, E, k, b, chunk, o);
}

hipError_t launch_balance_backward(const void* logits, int lt, int64_t ld, int T, int E, int k, const BalanceDev& b,
                                   const int32_t* counts, const int32_t* tokens, const float* grad_loss,
                                   const float* grad_z, void* out, int64_t ldo, hipStream_t st) {
  const int vec = rows_vec(logits, lt, E, ld), vec_out = rows_vec(out, lt, E, ldo);
  // 16 tokens a workgroup until there are four workgroups a CU, then up to 64
  const int rows = (int)std::min<int64_t>(64, std::max<int64_t>(16, ((int64_t)T / 1024 + 15) / 16 * 16));
  note_launch("balance_backward");
  return dispatch(E, lt, b.score, [&](auto nb, auto l, auto softmax) {
    constexpr int NB = decltype(nb)::value, LT = decltype(l)::value;
    constexpr bool SM = decltype(softmax)::value;
    return launch_kernel(balance_backward_kernel<NB, LT, SM>, (unsigned)(((int64_t)T + rows - 1) / rows), 256, 0, st,
                         logits, ld, vec, T, E, k, b, rows, counts, tokens, grad_loss, grad_z, out, ldo, vec_out);
  });
}

}  // namespace moe
