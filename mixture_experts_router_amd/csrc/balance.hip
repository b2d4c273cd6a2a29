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
// and joined in a fixed order.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr float SCORE_EPS = 1e-20f;
constexpr int PART_THREADS = 512;  // 32 tokens at a time, sixteen lanes a token
constexpr int JOIN_THREADS = 1024;

// Sums of one chunk and sequence: prob sums, counts (each E rounded up to 4), z sum, tokens
__host__ __device__ constexpr int slot_words(int E) { return 2 * ((E + 3) / 4 * 4) + 4; }

// tokens of a chunk: at most 1024 chunks
int chunk_tokens(int T) {
  const int64_t c = ((int64_t)T + 1023) / 1024;
  return (int)((c + 31) / 32 * 32);
}

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

// Probabilities of a row in place of its logits; the softmax's lse (0 for a
// row that masks everything), or with sigmoid scores 1 - s in q
template <int NB, bool SOFTMAX>
__device__ __forceinline__ float probabilities(f32x4 (&l)[NB], f32x4 (&q)[NB]) {
  float sum = 0.0f;
  if constexpr (SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int c = 0; c < NB; ++c) m = fmaxf(m, fmaxf(fmaxf(l[c].x, l[c].y), fmaxf(l[c].z, l[c].w)));
    m = max16(m);
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = l[c][j] == -INFINITY ? 0.0f : expf(l[c][j] - m);
        l[c][j] = e;
        sum += e;
      }
    sum = sum16(sum);
    const float inv = 1.0f / sum;
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) l[c][j] = l[c][j] != 0.0f ? l[c][j] * inv : 0.0f;
    return sum == 0.0f ? 0.0f : m + logf(sum);
  } else {
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = l[c][j];
        const float s = 1.0f / (1.0f + expf(-v));
        q[c][j] = 1.0f / (1.0f + expf(v));
        l[c][j] = s;
        sum += s;
      }
    sum = sum16(sum) + SCORE_EPS;
    const float inv = 1.0f / sum;
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) l[c][j] = l[c][j] != 0.0f ? l[c][j] * inv : 0.0f;
    return 0.0f;
  }
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

// A workgroup sums the chunk [lo, hi) of tokens, each sequence in it into a
// slot of its own: chunk c and sequence s meet at most once on the way
// through both, so c + s names the slot.
template <int NB, int LT, bool SOFTMAX>
__global__ __launch_bounds__(PART_THREADS) void balance_part_kernel(const void* __restrict__ logits, int64_t ld,
                                                                    int vec, int T, int E, int k,
                                                                    const int32_t* __restrict__ idx, BalanceDev b,
                                                                    int chunk, float* __restrict__ slots) {
  __shared__ float psum[PART_THREADS / 64][256];
  __shared__ int hist[256];
  __shared__ float zsum[PART_THREADS / 64];
  __shared__ int nsum[PART_THREADS / 64];
  const int tid = threadIdx.x, lane = lane_id(), wave = wave_id(), i16 = lane % 16;
  const int64_t lo = (int64_t)blockIdx.x * chunk, hi = min((int64_t)T, lo + chunk);
  const int words = slot_words(E), padded = (E + 3) / 4 * 4;

  int s = b.offsets ? sequence_of(b.offsets, b.S, lo) : 0;
  for (; s < b.S; ++s) {
    const int64_t from = b.offsets ? max(lo, (int64_t)b.offsets[s]) : lo;
    const int64_t to = b.offsets ? min(hi, (int64_t)b.offsets[s + 1]) : hi;
    if (from >= hi) break;
    if (from >= to) continue;
    if (tid < 256) hist[tid] = 0;
    __syncthreads();

    f32x4 acc[NB];
#pragma unroll
    for (int c = 0; c < NB; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float za = 0.0f;
    int n = 0;
    for (int64_t t0 = from; t0 < to; t0 += PART_THREADS / 16) {
      const int64_t t = t0 + tid / 16;
      const bool live = t < to && (!b.mask || b.mask[t] != 0);
      f32x4 p[NB], q[NB];
      load_row<LT, NB>(logits, t * ld, E, vec, live, i16, p);
      const float lse = probabilities<NB, SOFTMAX>(p, q);
#pragma unroll
      for (int c = 0; c < NB; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[c][j] += p[c][j];
      za += lse * lse;
      n += live;
    }
    for (int64_t i = from * k + tid; i < to * k; i += PART_THREADS) {
      const int e = idx[i];
      if (e >= 0 && e < E && (!b.mask || b.mask[i / k] != 0)) atomicAdd(&hist[e], 1);
    }

    // the four rows of a wave, then the waves in order
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v = acc[c][j];
        v += lane_read_f(v, lane ^ 16);
        v += lane_read_f(v, lane ^ 32);
        if (lane < 16) psum[wave][64 * c + 4 * i16 + j] = v;
      }
    za += lane_read_f(za, lane ^ 16);
    za += lane_read_f(za, lane ^ 32);
    n += __shfl_xor(n, 16, WAVE);
    n += __shfl_xor(n, 32, WAVE);
    if (lane == 0) {
      zsum[wave] = za;
      nsum[wave] = n;
    }
    __syncthreads();
    float* slot = slots + ((int64_t)blockIdx.x + s) * words;
    if (tid < E) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < PART_THREADS / 64; ++w) v += psum[w][tid];
      slot[tid] = v;
      ((int*)slot)[padded + tid] = hist[tid];
    }
    if (tid == 0) {
      float v = 0.0f;
      int m = 0;
      for (int w = 0; w < PART_THREADS / 64; ++w) {
        v += zsum[w];
        m += nsum[w];
      }
      slot[2 * padded] = v;
      ((int*)slot)[2 * padded + 1] = m;
    }
    __syncthreads();
  }
}

// A workgroup a sequence: its slots in order, then the loss
__global__ __launch_bounds__(JOIN_THREADS) void balance_join_kernel(const float* __restrict__ slots, int T, int E,
                                                                    int k, BalanceDev b, int chunk,
                                                                    float* __restrict__ loss, float* __restrict__ z,
                                                                    float* __restrict__ prob,
                                                                    int32_t* __restrict__ counts,
                                                                    int32_t* __restrict__ tokens) {
  __shared__ float psum[4][256];
  __shared__ int csum[4][256];
  __shared__ double dsum[4];
  __shared__ int n_all;
  const int s = blockIdx.x, tid = threadIdx.x, e = tid % 256, g = tid / 256;
  const int words = slot_words(E), padded = (E + 3) / 4 * 4;
  int64_t from = 0, to = T;
  if (b.offsets) {
    from = max((int64_t)0, (int64_t)b.offsets[s]);
    to = min((int64_t)T, (int64_t)b.offsets[s + 1]);
  }
  const int64_t c0 = from / chunk, c1 = from < to ? (to - 1) / chunk + 1 : c0;
  float v = 0.0f;
  int c = 0;
  if (e < E)
    for (int64_t i = c0 + g; i < c1; i += 4) {
      const float* slot = slots + (i + s) * words;
      v += slot[e];
      c += ((const int*)slot)[padded + e];
    }
  psum[g][e] = v;
  csum[g][e] = c;
  double zs = 0.0;
  int n = 0;
  if (tid < 64) {
    for (int64_t i = c0 + tid; i < c1; i += 64) {
      const float* slot = slots + (i + s) * words;
      zs += slot[2 * padded];
      n += ((const int*)slot)[2 * padded + 1];
    }
    for (int o = 1; o < 64; o <<= 1) {
      zs += __shfl_xor(zs, o, WAVE);
      n += __shfl_xor(n, o, WAVE);
    }
    if (tid == 0) {
      tokens[s] = n;
      if (z) z[s] = n ? (float)(zs / n) : 0.0f;
    }
  }
  if (tid == 0) n_all = n;
  __syncthreads();
  n = n_all;
  double d = 0.0;
  if (tid < 256) {
    const float total = ((psum[0][tid] + psum[1][tid]) + psum[2][tid]) + psum[3][tid];
    const int cnt = csum[0][tid] + csum[1][tid] + csum[2][tid] + csum[3][tid];
    if (tid < E) {
      const double mean = n ? (double)total / n : 0.0;
      if (prob) prob[(int64_t)s * E + tid] = (float)mean;
      counts[(int64_t)s * E + tid] = cnt;
      d = cnt ? (double)cnt * mean : 0.0;
    }
    for (int o = 1; o < 64; o <<= 1) d += __shfl_xor(d, o, WAVE);
    if (tid % 64 == 0) dsum[tid / 64] = d;
  }
  __syncthreads();
  if (tid == 0) loss[s] = n ? (float)((((dsum[0] + dsum[1]) + dsum[2]) + dsum[3]) * E / ((double)k * n)) : 0.0f;
}

template <int NB, int LT, bool SOFTMAX>
__global__ __launch_bounds__(256) void balance_backward_kernel(const void* __restrict__ logits, int64_t ld, int vec,
                                                               int T, int E, int k, BalanceDev b,
                                                               const int32_t* __restrict__ counts,
                                                               const int32_t* __restrict__ tokens,
                                                               const float* __restrict__ grad_loss,
                                                               const float* __restrict__ grad_z,
                                                               void* __restrict__ out, int64_t ldo, int vec_out) {
  const int lane = lane_id(), i16 = lane % 16;
  const int64_t t = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
  if (t >= T) return;
  int s = 0;
  bool live = !b.mask || b.mask[t] != 0;
  if (b.offsets && live) {
    s = sequence_of(b.offsets, b.S, t);
    live = s < b.S && b.offsets[s] <= t;
  }
  int n = 0;
  if (live) n = tokens[s];
  live = live && n > 0;
  f32x4 p[NB], q[NB], g[NB];
  load_row<LT, NB>(logits, t * ld, E, vec, live, i16, p);
  const float nf = (float)n;
  const float slope = live && grad_loss ? grad_loss[s] * ((float)E / ((float)k * nf * nf)) : 0.0f;
#pragma unroll
  for (int c = 0; c < NB; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int x = 64 * c + 4 * i16 + j;
      g[c][j] = live && x < E ? slope * (float)counts[(int64_t)s * E + x] : 0.0f;
    }
  const float lse = probabilities<NB, SOFTMAX>(p, q);
  float dot = 0.0f;
#pragma unroll
  for (int c = 0; c < NB; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) dot += g[c][j] * p[c][j];
  dot = sum16(dot);
  const float add = SOFTMAX && live && grad_z ? grad_z[s] * (2.0f / nf) * lse - dot : -dot;
#pragma unroll
  for (int c = 0; c < NB; ++c) {
    const int x = 64 * c + 4 * i16;
    if (x >= E) continue;
    f32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float d = p[c][j] * (g[c][j] + add);
      if (!SOFTMAX) d *= q[c][j];
      v[j] = live && p[c][j] != 0.0f ? d : 0.0f;
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
  if (T == 0) return 0;
  const int chunk = chunk_tokens(T);
  return (((int64_t)T + chunk - 1) / chunk + S) * slot_words(E) * 4;
}

hipError_t launch_balance(const void* logits, int lt, int64_t ld, int T, int E, int k, const int32_t* idx,
                          const BalanceDev& b, float* loss, float* z, float* prob, int32_t* counts, int32_t* tokens,
                          void* ws, hipStream_t st) {
  const int chunk = T ? chunk_tokens(T) : 1;
  if (T) {
    const int vec = rows_vec(logits, lt, E, ld);
    const hipError_t r = dispatch(E, lt, b.score, [&](auto nb, auto l, auto softmax) {
      constexpr int NB = decltype(nb)::value, LT = decltype(l)::value;
      constexpr bool SM = decltype(softmax)::value;
      return launch_kernel(balance_part_kernel<NB, LT, SM>, (unsigned)((T + chunk - 1) / chunk), PART_THREADS, 0, st,
                           logits, ld, vec, T, E, k, idx, b, chunk, (float*)ws);
    });
    if (r != hipSuccess) return r;
  }
  return launch_kernel(balance_join_kernel, (unsigned)b.S, JOIN_THREADS, 0, st, (const float*)ws, T, E, k, b, chunk,
                       loss, z, prob, counts, tokens);
}

hipError_t launch_balance_backward(const void* logits, int lt, int64_t ld, int T, int E, int k, const BalanceDev& b,
                                   const int32_t* counts, const int32_t* tokens, const float* grad_loss,
                                   const float* grad_z, void* out, int64_t ldo, hipStream_t st) {
  const int vec = rows_vec(logits, lt, E, ld), vec_out = rows_vec(out, lt, E, ldo);
  return dispatch(E, lt, b.score, [&](auto nb, auto l, auto softmax) {
    constexpr int NB = decltype(nb)::value, LT = decltype(l)::value;
    constexpr bool SM = decltype(softmax)::value;
    return launch_kernel(balance_backward_kernel<NB, LT, SM>, (unsigned)(((int64_t)T + 15) / 16), 256, 0, st, logits,
                         ld, vec, T, E, k, b, counts, tokens, grad_loss, grad_z, out, ldo, vec_out);
  });
}

}  // namespace moe
