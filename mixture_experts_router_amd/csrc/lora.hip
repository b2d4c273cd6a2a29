// Low-rank adapters of many requests beside a projection that they share:
//
//   out[t] = base[t] + scale_a * (x[t] A_a^T) B_a^T,   a = ids[t]
//
// with A_a [R, K] and B_a [N, R] of adapter a.  Two launches: v = x A^T into
// fp32 partial sums, then base + scale v B^T.  Both look at chunks of 64
// consecutive tokens: every wave reads the chunk's 64 ids (one a lane), walks
// its distinct adapters with ballots and works on the tokens of one adapter
// at a time on the matrix cores, so neither sorted ids nor a sorting launch
// are needed, each adapter is read once a chunk, and runs of one request fill
// the tiles.  Workgroup (chunk, j, s) takes the j-th, (j + J)-th ... distinct
// adapter and the s-th part of the reduced (or written) columns.
//
// Rounding: x A^T has exact products and fp32 sums, which stay in fp32.  For
// the second product v goes to the matrix cores as two 16-bit parts (hi + lo:
// 2^-18 relative for bf16, 2^-22 for fp16), three for a bf16 adapter with an
// fp32 output, so the only rounding that shows is the output's.  fp16 parts are
// taken of v * 2^-e_t, the token's largest |v| brought to 2^13 .. 2^14, which
// keeps fp32's range.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int CHUNK = 64;  // tokens a workgroup looks at: one id a lane

template <int ACT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (ACT == ACT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// the chunk's adapter of this lane's token: -1 none (also for ids outside
// [0, L)), -2 past the last token
__device__ __forceinline__ int chunk_id(const int32_t* __restrict__ ids, int64_t t0, int T, int L) {
  const int64_t t = t0 + lane_id();
  if (t >= T) return -2;
  const int a = ids[t];
  return a >= 0 && a < L ? a : -1;
}

// lane p receives the lane of the p-th set bit of `set` (p < popcount)
__device__ __forceinline__ int nth_lane(uint64_t set) {
  const int lane = lane_id();
  const uint64_t lt = lanemask_lt();
  const int to = set >> lane & 1 ? (int)__popcll(set & lt) : (int)__popcll(set) + (int)__popcll(~set & lt);
  return __builtin_amdgcn_ds_permute(to << 2, lane);
}

__device__ __forceinline__ int adapter_rank(const int32_t* __restrict__ ranks, int a, int R) {
  return ranks ? min(max(ranks[a], 0), R) : R;
}

// ------------------------------------------------------------- x A^T ----
//
// D = A x^T: rows are ranks, columns tokens, so a lane ends with four
// consecutive ranks of one token.  The four waves take consecutive parts of
// the workgroup's columns and are added through LDS in wave order; lane group
// g = lane / 16 of a 64-column block reads columns 16 g .. 16 g + 15 (32
// contiguous bytes) of its row, the same order in both operands.
template <int ACT, int RT>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                          const uint16_t* __restrict__ am,
                                                          const int32_t* __restrict__ ids,
                                                          const int32_t* __restrict__ ranks, float* __restrict__ part,
                                                          int T, int L, int R, int K) {
  constexpr int NT = RT == 8 ? 2 : 4;  // token tiles a pass
  constexpr int UB = RT <= 2 ? 2 : 1;  // 64-column blocks in flight
  __shared__ f32x4 red[2][RT * NT][WAVE];
  const int lane = lane_id(), wave = wave_id();
  const int l16 = lane % 16, g = lane / 16;
  const int64_t t0 = (int64_t)blockIdx.x * CHUNK;
  const int id = chunk_id(ids, t0, T, L);
  const int nb = (K + 63) / 64, W = gridDim.z * 4, slot = blockIdx.z * 4 + wave;
  const int b0 = (int)((int64_t)nb * slot / W), b1 = (int)((int64_t)nb * (slot + 1) / W);
  uint64_t left = __ballot(id >= 0);
  for (int n = 0; left != 0; ++n) {
    const int a = __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(left));
    const uint64_t mine = __ballot(id == a);
    left &= ~mine;
    if (n % (int)gridDim.y != (int)blockIdx.y) continue;
    const int m = (int)__popcll(mine);
    const int nth = nth_lane(mine);
    const int rank = adapter_rank(ranks, a, R);
    const uint16_t* arow = am + ((int64_t)a * R + l16) * K + 16 * g;
    for (int i0 = 0; i0 * 16 < m; i0 += NT) {
      f32x4 acc[RT][NT];
      const uint16_t* xrow[NT];
      int tok[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int p = (i0 + i) * 16 + l16;
        tok[i] = __builtin_amdgcn_ds_bpermute((p < m ? p : 0) << 2, nth);
        if (p >= m) tok[i] = -1;
        xrow[i] = x + (t0 + max(tok[i], 0)) * ldx + 16 * g;
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
      const int nt = min(NT, (m - i0 * 16 + 15) / 16);
      for (int b = b0; b < b1; b += UB) {
        u32x4 av[UB][2][RT], xv[UB][2][NT];
#pragma unroll
        for (int u = 0; u < UB; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = (b + u) * 64 + 8 * h;
            const bool in = b + u < b1 && c + 16 * g < K;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              xv[u][h][i] = u32x4{0u, 0u, 0u, 0u};
              if (i < nt && in && tok[i] >= 0) xv[u][h][i] = load16(xrow[i] + c);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              av[u][h][r] = u32x4{0u, 0u, 0u, 0u};
              if (in && r * 16 + l16 < rank) av[u][h][r] = load16(arow + (int64_t)r * 16 * K + c);
            }
          }
#pragma unroll
        for (int u = 0; u < UB; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < NT; ++i)
              if (i < nt) {
#pragma unroll
                for (int r = 0; r < RT; ++r) acc[r][i] = mfma16<ACT>(av[u][h][r], xv[u][h][i], acc[r][i]);
              }
      }
      // (w0 + w2) + (w1 + w3)
      __syncthreads();
      if (wave >= 2) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (i < nt) {
#pragma unroll
            for (int r = 0; r < RT; ++r) red[wave - 2][r * NT + i][lane] = acc[r][i];
          }
      }
      __syncthreads();
      if (wave < 2) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (i < nt) {
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[r][i] = acc[r][i] + red[wave][r * NT + i][lane];
          }
      }
      __syncthreads();
      if (wave == 1) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (i < nt) {
#pragma unroll
            for (int r = 0; r < RT; ++r) red[0][r * NT + i][lane] = acc[r][i];
          }
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (i < nt && tok[i] >= 0) {
            float* to = part + ((int64_t)blockIdx.z * T + t0 + tok[i]) * R;
#pragma unroll
            for (int r = 0; r < RT; ++r)
              if (r * 16 + 4 * g < R) *(f32x4*)(to + r * 16 + 4 * g) = acc[r][i] + red[0][r * NT + i][lane];
          }
      }
    }
  }
}

// ------------------------------------------------- base + scale v B^T ---

// splits v (finite or not) into NP 16-bit parts, each the rounding of what
// the earlier ones leave
template <int ACT, int NP>
__device__ __forceinline__ void split_parts(float v, uint16_t* o) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    o[i] = f32_to_act_bits(v, ACT);
    const float f = act_to_f32(o[i], ACT);
    v = fabsf(f) < INFINITY ? v - f : 0.0f;  // inf and NaN are the first part alone
  }
}

// RS: 32-rank steps of the reduction; 0 stands for up to 16 ranks, where one
// matrix instruction takes the first two parts side by side
template <int ACT, bool F32, int RS>
__global__ __launch_bounds__(256) void lora_expand_kernel(const float* __restrict__ part, int S,
                                                          const uint16_t* __restrict__ bm,
                                                          const float* __restrict__ scale,
                                                          const int32_t* __restrict__ ids,
                                                          const int32_t* __restrict__ ranks, const void* base,
                                                          int64_t ldb, void* out, int64_t ldo, int T, int L, int R,
                                                          int N, int vec) {
  constexpr int NP = F32 && ACT == ACT_BF16 ? 3 : 2;
  constexpr int RP = RS == 0 ? 16 : RS * 32;
  constexpr int STEPS = RS == 0 ? 1 : RS;
  __shared__ __attribute__((aligned(16))) uint16_t vs[NP][CHUNK][RP + 8];
  __shared__ int exps[CHUNK];
  const int lane = lane_id(), wave = wave_id();
  const int l16 = lane % 16, g = lane / 16;
  const int64_t t0 = (int64_t)blockIdx.x * CHUNK;
  const int id = chunk_id(ids, t0, T, L);
  const int nb = (N + 31) / 32;
  const int b0 = (int)((int64_t)nb * blockIdx.z / gridDim.z), b1 = (int)((int64_t)nb * (blockIdx.z + 1) / gridDim.z);
  uint64_t left = __ballot(id >= -1);
  for (int n = 0; left != 0; ++n) {
    const int a = __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(left));
    const uint64_t mine = __ballot(id == a);
    left &= ~mine;
    if (n % (int)gridDim.y != (int)blockIdx.y) continue;
    const int m = (int)__popcll(mine);
    const int nth = nth_lane(mine);
    if (a < 0) {
      // no adapter: out is base, moved only if the two are not one buffer
      if (out == base) continue;
      const int c0 = b0 * 32, c1 = min(N, b1 * 32);
      for (int p = wave; p < m; p += 4) {
        const int64_t t = t0 + __builtin_amdgcn_readlane(nth, p);
        for (int c = c0 + lane; c < c1; c += WAVE) {
          if constexpr (F32) ((float*)out)[t * ldo + c] = ((const float*)base)[t * ldb + c];
          else ((uint16_t*)out)[t * ldo + c] = ((const uint16_t*)base)[t * ldb + c];
        }
      }
      continue;
    }
    const int rank = adapter_rank(ranks, a, R);
    __syncthreads();  // the previous adapter's parts are read
    {
      const float sc = scale ? scale[a] : 1.0f;
      const int row = threadIdx.x / 16, i16 = threadIdx.x % 16;
      for (int p0 = 0; p0 < m; p0 += 16) {
        const int p = p0 + row;
        const int tok = __builtin_amdgcn_ds_bpermute((p < m ? p : 0) << 2, nth);
        const float* from = part + (t0 + tok) * R;
        float v[RP / 16];
        float top = 0.0f;
#pragma unroll
        for (int q = 0; q < RP / 16; ++q) {
          const int r = i16 + 16 * q;
          v[q] = 0.0f;
          if (r < rank) {
            for (int s = 0; s < S; ++s) v[q] += from[(int64_t)s * T * R + r];
            v[q] *= sc;
          }
          top = fmaxf(top, fabsf(v[q]));
        }
        int e = 0;
        if constexpr (ACT == ACT_F16) {
          top = fmaxf(top, dpp_f<DPP_QUAD_1032>(top));
          top = fmaxf(top, dpp_f<DPP_QUAD_2301>(top));
          top = fmaxf(top, dpp_f<DPP_ROW_HALF_MIRROR>(top));
          top = fmaxf(top, dpp_f<DPP_ROW_MIRROR>(top));
          if (top > 0.0f && top < INFINITY) e = __builtin_amdgcn_frexp_expf(top) - 14;
        }
        if (p < m) {
          if (i16 == 0) exps[p] = e;
#pragma unroll
          for (int q = 0; q < RP / 16; ++q) {
            uint16_t o[NP];
            split_parts<ACT, NP>(ACT == ACT_F16 ? ldexp_f(v[q], -e) : v[q], o);
#pragma unroll
            for (int i = 0; i < NP; ++i) vs[i][p][i16 + 16 * q] = o[i];
          }
        }
      }
    }
    __syncthreads();
    const int nt = (m + 15) / 16;
    for (int b = b0 + wave; b < b1; b += 4) {
      // D = B v^T: tile u's row i is column 8 (i / 4) + 4 u + i % 4 of the 32,
      // so a lane ends with eight consecutive columns of one token
      const int n0 = b * 32;
      u32x4 bv[STEPS][2];
#pragma unroll
      for (int q = 0; q < STEPS; ++q)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int nr = n0 + l16 / 4 * 8 + 4 * u + l16 % 4;
          const int r0 = RS == 0 ? g % 2 * 8 : 32 * q + 8 * g;
          u32x4 w = u32x4{0u, 0u, 0u, 0u};
          if (nr < N && r0 < rank) {
            w = load16(bm + ((int64_t)a * N + nr) * R + r0);
            if (r0 + 8 > rank) {  // columns past the rank may hold anything
#pragma unroll
              for (int h = 0; h < 4; ++h)
                w[h] &= (r0 + 2 * h < rank ? 0xFFFFu : 0u) | (r0 + 2 * h + 1 < rank ? 0xFFFF0000u : 0u);
            }
          }
          bv[q][u] = w;
        }
      for (int i = 0; i < nt; ++i) {
        const int p = min(i * 16 + l16, m - 1);
        const int64_t t = t0 + __builtin_amdgcn_ds_bpermute(p << 2, nth);
        const int c = n0 + 8 * g;
        const bool live = i * 16 + l16 < m;
        const bool whole = vec && c + 8 <= N;
        u32x4 o0 = u32x4{0u, 0u, 0u, 0u}, o1 = o0;
        if (live && whole) {
          if constexpr (F32) {
            o0 = load16((const float*)base + t * ldb + c);
            o1 = load16((const float*)base + t * ldb + c + 4);
          } else {
            o0 = load16((const uint16_t*)base + t * ldb + c);
          }
        }
        f32x4 acc[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int q = 0; q < STEPS; ++q) {
          if constexpr (RS == 0) {
            const u32x4 v01 = *(const u32x4*)&vs[g / 2][p][g % 2 * 8];
#pragma unroll
            for (int u = 0; u < 2; ++u) acc[u] = mfma16<ACT>(bv[0][u], v01, acc[u]);
            if constexpr (NP == 3) {
              const u32x4 v2 = g < 2 ? *(const u32x4*)&vs[NP - 1][p][g * 8] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
              for (int u = 0; u < 2; ++u) acc[u] = mfma16<ACT>(bv[0][u], v2, acc[u]);
            }
          } else {
#pragma unroll
            for (int h = NP - 1; h >= 0; --h) {  // small parts first
              const u32x4 v = *(const u32x4*)&vs[h][p][32 * q + 8 * g];
#pragma unroll
              for (int u = 0; u < 2; ++u) acc[u] = mfma16<ACT>(bv[q][u], v, acc[u]);
            }
          }
        }
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = acc[j / 4][j % 4];
        if constexpr (ACT == ACT_F16) {
          const int e = exps[p];
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = ldexp_f(d[j], e);
        }
        if (live) {
          if (whole) {
            if constexpr (F32) {
              f32x4 y0 = __builtin_bit_cast(f32x4, o0), y1 = __builtin_bit_cast(f32x4, o1);
  #pragma unroll
              for (int j = 0; j < 4; ++j) {
                y0[j] = y0[j] + d[j];
                y1[j] = y1[j] + d[j + 4];
              }
              *(f32x4*)((float*)out + t * ldo + c) = y0;
              *(f32x4*)((float*)out + t * ldo + c + 4) = y1;
            } else {
              u32x4 y;
  #pragma unroll
              for (int j = 0; j < 4; ++j)
                y[j] = (uint32_t)f32_to_act_bits(act_to_f32(o0[j] & 0xFFFFu, ACT) + d[2 * j], ACT) |
                       (uint32_t)f32_to_act_bits(act_to_f32(o0[j] >> 16, ACT) + d[2 * j + 1], ACT) << 16;
              *(u32x4*)((uint16_t*)out + t * ldo + c) = y;
            }
          } else {
  #pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c + j < N) {
                if constexpr (F32)
                  ((float*)out)[t * ldo + c + j] = ((const float*)base)[t * ldb + c + j] + d[j];
                else
                  ((uint16_t*)out)[t * ldo + c + j] =
                      f32_to_act_bits(act_to_f32(((const uint16_t*)base)[t * ldb + c + j], ACT) + d[j], ACT);
              }
          }
        }
      }
    }
  }
}

struct LoraGrid {
  int chunks, J, S, NS;
};

// Adapters walked side by side (J) and splits of the reduced (S) and written
// (NS) columns, from the sizes alone: the ids are on the device.
LoraGrid lora_grid(int T, int K, int N, int L, int R) {
  LoraGrid r;
  r.chunks = (int)(((int64_t)T + CHUNK - 1) / CHUNK);
  r.J = std::max(1, std::min(std::min(T, CHUNK), std::min(L, 512 / r.chunks)));
  const int nbk = (K + 63) / 64, nbn = (N + 31) / 32;
  const int work = r.chunks * std::min(r.J, 16);
  r.S = std::max(1, std::min(std::min(16, nbk / 4), 1024 / work));
  r.NS = std::max(1, std::min(std::min(32, nbn / 4), 2048 / work));
  return r;
}

}  // namespace

int64_t lora_partial_floats(int T, int K, int N, int L, int R) {
  return (int64_t)lora_grid(T, K, N, L, R).S * T * R;
}

hipError_t launch_lora(const void* x, int act, int64_t ldx, int T, const LoraDev& ad, const int32_t* ids,
                       const void* base, int64_t ldb, void* out, int64_t ldo, bool out_f32, float* part,
                       hipStream_t st) {
  const LoraGrid lg = lora_grid(T, ad.K, ad.N, ad.L, ad.R);
  const int per = out_f32 ? 4 : 8;  // elements of 16 bytes
  const int vec = ldb % per == 0 && ldo % per == 0 &&
                  ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const dim3 gs(lg.chunks, lg.J, lg.S), ge(lg.chunks, lg.J, lg.NS);
  auto shrink = [&](auto kern) {
    return launch_kernel(kern, gs, 256, 0, st, (const uint16_t*)x, ldx, (const uint16_t*)ad.a, ids, ad.ranks, part, T,
                         ad.L, ad.R, ad.K);
  };
  auto expand = [&](auto kern) {
    return launch_kernel(kern, ge, 256, 0, st, (const float*)part, lg.S, (const uint16_t*)ad.b, ad.scale, ids,
                         ad.ranks, base, ldb, out, ldo, T, ad.L, ad.R, ad.N, vec);
  };
  auto run = [&](auto ac) {
    constexpr int A = decltype(ac)::value;
    hipError_t e = ad.R <= 16   ? shrink(lora_shrink_kernel<A, 1>)
                   : ad.R <= 32 ? shrink(lora_shrink_kernel<A, 2>)
                   : ad.R <= 64 ? shrink(lora_shrink_kernel<A, 4>)
                                : shrink(lora_shrink_kernel<A, 8>);
    if (e != hipSuccess) return e;
    auto go = [&](auto fc) {
      constexpr bool F = decltype(fc)::value;
      return ad.R <= 16   ? expand(lora_expand_kernel<A, F, 0>)
             : ad.R <= 32 ? expand(lora_expand_kernel<A, F, 1>)
             : ad.R <= 64 ? expand(lora_expand_kernel<A, F, 2>)
                          : expand(lora_expand_kernel<A, F, 4>);
    };
    return out_f32 ? go(std::true_type{}) : go(std::false_type{});
  };
  return act == ACT_BF16 ? run(std::integral_constant<int, ACT_BF16>{}) : run(std::integral_constant<int, ACT_F16>{});
}

}  // namespace moe
