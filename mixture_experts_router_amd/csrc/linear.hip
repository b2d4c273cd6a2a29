// Dense products with a fused epilogue, and their gradients (gfx950):
//
//   z = x W^T + bias,   out = residual + row_scale * act(z)
//   dz = row_scale * g * act'(z),  dx = dz W,  dW = dz^T x,  dbias = sum dz,  drow_scale = sum g act(z)
//
// All three products are C[m, n] = sum_k A(m, k) B(n, k) with fp16 or bf16
// operands and fp32 sums; what differs is which index is contiguous in memory.
#include "common.hpp"
#include "kernels.hpp"

#include <algorithm>

namespace moe {
namespace {

typedef __bf16 bf16;
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int NUM_XCD = 8;  // workgroups go round-robin over 8 XCDs, each with its own L2
constexpr uint32_t OUT_OF_RANGE = 0x80000000u;  // a byte offset past every descriptor: the load gives zeros

template <int DT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == ACT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// 16 bytes per lane from buffer r at voff + soff into LDS (lane i at lds + 16 i).
// In assembly because the compiler waits for every such load before a transposed
// LDS read (its builtin carries no alias information): 132 against 114 us for the
// gradient of W of 2816 x 4096 from 4096 tokens.  It has no register outputs;
// the kernel itself waits for it (wait_vmcnt) before the barrier that hands the
// stage over.  s_nop: M0, and scalars that come from vector instructions, must
// be written five cycles before the load reads them.
__device__ __forceinline__ void dma16(u32x4 r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(r), "s"(soff)
               : "memory", "m0");
}

__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) { return (uint32_t)(uintptr_t)(lds_void*)p; }

__device__ __forceinline__ u32x4 buffer_of(const void* base, uint32_t bytes) {
  const uint64_t p = (uint64_t)(uintptr_t)base;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)p),
               (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(p >> 32)) & 0xFFFFu, bytes, (uint32_t)RSRC_WORD3};
}

// wait until at most N vector memory instructions of this wave are pending
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N <= 63, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

template <int V>
struct IC {
  static constexpr int value = V;
};

// f(IC<S>), f(IC<S + 1>), ... f(IC<N - 1>) while f returns true
template <int S, int N, typename F>
__device__ __forceinline__ void for_each(F&& f) {
  if constexpr (S < N) {
    if (f(IC<S>{})) for_each<S + 1, N>(f);
  }
}

// ------------------------------------------------------------ activations --
//
// The hardware's exponential (base 2) and reciprocal: exp is off by |z| 2^-24
// beside two units in the last place, where the value or its complement has
// shrunk by as much, so no activation is off by more than a few 2^-24.

constexpr float LOG2E = 1.44269504088896341f;

__device__ __forceinline__ float sigmoid_(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-LOG2E * v));
}

// The normal distribution Phi(z) = erfc(-z / sqrt 2) / 2, and exp(-z^2 / 2).
// erfc(x) = exp(-x^2) F(t) / (1 + 2 x) for x >= 0 with t = (x - 3.75) / (x + 3.75)
// (Shepherd and Laframboise, "Chebyshev approximation of (1 + 2x) exp(x^2) erfc x
// in 0 <= x < infinity", 1981); F here a polynomial, off by at most 4.4e-8.  Phi is off
// by 3 2^-24 at most (erfcf: the epilogue of 777 x 2816 4 us longer).
__device__ __forceinline__ float normal_(float z, float& e) {
  constexpr float F[] = {1.23751259f, -0.140240654f, 0.00358627038f, 0.082278423f, -0.108814269f, 0.0922907665f, -0.0586468577f, 0.0284092519f, -0.00984449498f, 0.00167591218f, 0.000396307616f, -0.000224116753f};
  const float x = 0.70710678118654752f * fabsf(z);
  e = __builtin_amdgcn_exp2f(-LOG2E * (x * x));
  const float y = fminf(x, 40.0f);  // e is 0 there (or NaN, as z)
  const float t = (y - 3.75f) * __builtin_amdgcn_rcpf(y + 3.75f);
  float f = F[11];
#pragma unroll
  for (int i = 10; i >= 0; --i) f = __builtin_fmaf(f, t, F[i]);
  const float tail = 0.5f * (e * f) * __builtin_amdgcn_rcpf(__builtin_fmaf(2.0f, y, 1.0f));
  return z > 0.0f ? 1.0f - tail : tail;
}

// act(z) and its slope; at infinities (products beyond fp16's range) their limits
__device__ __forceinline__ float activate_slope(int act, float z, float& slope) {
  switch (act) {
    case LIN_RELU:
      slope = z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
      return z > 0.0f ? z : (z != z ? z : 0.0f);
    case LIN_SILU: {
      const float s = sigmoid_(z);
      slope = mul0(s, 1.0f + mul0(z, sigmoid_(-z)));
      return mul0(z, s);
    }
    case LIN_GELU: {
      float e;
      const float c = normal_(z, e);
      slope = c + mul0(z, 0.39894228040143268f * e);
      return mul0(z, c);
    }
    case LIN_SIGMOID: {
      const float s = sigmoid_(z);
      slope = s * sigmoid_(-z);
      return s;
    }
    default:
      slope = 1.0f;
      return z;
  }
}

// ------------------------------------------------------------------ rows --

template <int DT>
__device__ __forceinline__ float half_to_f32(uint32_t bits) {
  return act_to_f32(bits, DT);
}

// W = 8 or 1 values from `at` of a row of 16-bit (f32: 32-bit) values, of which
// `left` exist (the others are 0); vec: all of them, 16-byte aligned
template <int DT, int W>
__device__ __forceinline__ void load_n(const void* p, bool f32, int64_t at, int left, bool vec, float (&v)[W]) {
  if (f32) {
    const float* q = (const float*)p + at;
    if (W == 8 && vec) {
#pragma unroll
      for (int h = 0; h < W / 4; ++h) {
        const f32x4 a = *(const f32x4*)(q + 4 * h);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * h + j] = a[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = j < left ? q[j] : 0.0f;
    }
  } else {
    const uint16_t* q = (const uint16_t*)p + at;
    if (W == 8 && vec) {
      const u32x4 a = load16(q);
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = half_to_f32<DT>(j % 2 ? a[j / 2] >> 16 : a[j / 2] & 0xFFFFu);
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = j < left ? half_to_f32<DT>(q[j]) : 0.0f;
    }
  }
}

// two values rounded to 16 bits (to nearest even; NaN stays NaN)
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == ACT_BF16) {
    typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(bf16)a, (bf16)b});
  } else {
    return __builtin_bit_cast(uint32_t, f16x2{(f16)a, (f16)b});
  }
}

template <int DT, int W>
__device__ __forceinline__ void store_n(void* p, bool f32, int64_t at, int left, bool vec, const float (&v)[W]) {
  if (f32) {
    float* q = (float*)p + at;
    if (W == 8 && vec) {
#pragma unroll
      for (int h = 0; h < W / 4; ++h) *(f32x4*)(q + 4 * h) = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (j < left) q[j] = v[j];
    }
  } else {
    uint16_t* q = (uint16_t*)p + at;
    if (W == 8 && vec) {
      u32x4 a = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < W / 2; ++j) a[j] = pack2<DT>(v[2 * j], v[2 * j + 1]);
      *(u32x4*)q = a;
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (j < left) q[j] = (uint16_t)pack2<DT>(v[j], 0.0f);
    }
  }
}

// An fp32 gradient's dz in two 16-bit parts of its sign, so that the products keep
// what its 32 bits hold: rounded once, fp16 loses all that is below 2^-25 (a balance
// loss's gradient is 1e-8 and less) or above 65504, and a router's gradients in bf16
// are off by 2.4e-3 where their own rounding is 1.7e-3.  The matrix instructions are
// twice as many: 36 to 45 us for 4096 x 4096 to 64, at most 30% more up to 256
// columns; 185 to 320 us for 2816, where bf16 takes one (moe_linear_backward).
// The first is dz without its low bits, the second what is left.  fp16: the first
// holds dz 2^-SHIFT_DZ, the second what is left of that times 2^SHIFT_LOW, together
// 2^-37 up to 2^24; where what is left has no room (dz above 2^13), the first is
// rounded instead.  A second part of 0 beside a first is replaced by a tiny one, and
// both have dz's sign, so that an infinite weight or input gives dz's infinity, not
// NaN.
constexpr int SHIFT_DZ = 8, SHIFT_LOW = 20;

template <int DT>
__device__ __forceinline__ void two_parts(float v, uint32_t& first, uint32_t& second) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, v), sign = bits >> 16 & 0x8000u;
  if (!(fabsf(v) < INFINITY)) {
    first = second = pack2<DT>(v, 0.0f) & 0xFFFFu;
    return;
  }
  if constexpr (DT == ACT_BF16) {
    first = bits >> 16;
    second = pack2<DT>(v - half_to_f32<DT>(first), 0.0f) & 0xFFFFu;
    if ((first & 0x7FFFu) && !(second & 0x7FFFu)) second = sign | 0x0080u;
  } else {
    const float a = v * (1.0f / (1 << SHIFT_DZ));
    first = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, 0.0f)) & 0xFFFFu;
    const float left = (a - half_to_f32<DT>(first)) * (float)(1 << SHIFT_LOW);
    second = pack2<DT>(left, 0.0f) & 0xFFFFu;
    if (fabsf(left) > 65504.0f) {
      first = pack2<DT>(a, 0.0f) & 0xFFFFu;
      second = sign;
    }
    if ((first & 0x7FFFu) && !(second & 0x7FFFu)) second = sign | 1u;
  }
}

// eight values in both parts
template <int DT>
__device__ __forceinline__ void store_parts(uint16_t* p, int64_t low, int left, bool vec, const float (&v)[8]) {
  uint32_t a[8], b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) two_parts<DT>(v[j], a[j], b[j]);
  if (vec) {
    *(u32x4*)p = u32x4{a[0] | a[1] << 16, a[2] | a[3] << 16, a[4] | a[5] << 16, a[6] | a[7] << 16};
    *(u32x4*)(p + low) = u32x4{b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) {
        p[j] = (uint16_t)a[j];
        p[low + j] = (uint16_t)b[j];
      }
  }
}

// W = 8 or 1 columns from n of output row t from their fp32 sums (gated: u the
// sums of the up columns).  Everything is fp32 up to the one rounding that gives
// `out`; the kept z is rounded on its own.  The choices are made once for the
// columns: made for each, they took 25 us of a 4096 x 4096 output.
template <int DT, bool GATED, int W>
__device__ __forceinline__ void finish(const LinearEpi& e, int64_t t, int n, float (&z)[W], float (&u)[W]) {
  const int left = e.C - n;
  const bool vec = e.vec && left >= W;
  if (e.bias) {
    const bool bvec = e.bias_vec && left >= W;
    float b[W];
    load_n<DT, W>(e.bias, e.bias_f32, n, left, bvec, b);
#pragma unroll
    for (int j = 0; j < W; ++j) z[j] += b[j];
    if (GATED) {
      load_n<DT, W>(e.bias, e.bias_f32, (int64_t)e.C + n, left, bvec, b);
#pragma unroll
      for (int j = 0; j < W; ++j) u[j] += b[j];
    }
  }
  if (e.pre) {
    store_n<DT, W>(e.pre, false, t * e.ldp + n, left, vec, z);
    if (GATED) store_n<DT, W>(e.pre, false, t * e.ldp + e.C + n, left, vec, u);
  }
  if constexpr (GATED) {
#pragma unroll
    for (int j = 0; j < W; ++j) z[j] = z[j] * sigmoid_(z[j]) * u[j];
  } else if (e.act != LIN_NONE) {
    auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < W; ++j) z[j] = f(z[j]);
    };
    switch (e.act) {
      case LIN_RELU: each([](float v) { return v > 0.0f ? v : (v != v ? v : 0.0f); }); break;
      case LIN_SILU: each([](float v) { return v * sigmoid_(v); }); break;
      case LIN_GELU: each([](float v) { float e; return v * normal_(v, e); }); break;
      default: each([](float v) { return sigmoid_(v); }); break;
    }
  }
  if (e.row_scale) {
    const float rs = e.row_scale[t];
#pragma unroll
    for (int j = 0; j < W; ++j) z[j] *= rs;
  }
  if (e.res) {
    float r[W];
    load_n<DT, W>(e.res, e.out_f32, t * e.ldr + n, left, vec, r);
#pragma unroll
    for (int j = 0; j < W; ++j) z[j] += r[j];
  }
  store_n<DT, W>(e.out, e.out_f32, t * e.ldo + n, left, vec, z);
}

// ------------------------------------------------------------ tile kernel --
//
// One workgroup computes BM x BN of C with WM x WN waves; k advances 64 a
// step through NS stages in LDS that global_load_lds fills (16 bytes a lane, no
// registers).  An operand whose k is contiguous stages rows of 64 k (128 bytes,
// 16-byte pieces XORed with the row so that a wave's 16-byte reads meet no bank
// twice); one whose m (n) is contiguous stages 64 rows of BM (BN) values and is
// read with ds_read_b64_tr_b16, which transposes 4 x 16 blocks on the way into
// the registers.
//
// A wave of the 256 x 256 tile (eight waves of 128 x 64) reads 12 KB of LDS for
// 512 cycles of MFMAs, so LDS keeps up; the MFMAs run 58% of the cycles, at about
// 1.9 GHz under the card's power limit (operands of zeros took 205 us where
// others took 258).  8192^3 in 745 us, 1475 TFLOP/s; 4096 x 11008 to 4096 in 258
// us from the caches, 1431 TFLOP/s (282 to 292 us, by the box, with a residual and
// other operands each time); smaller tiles wait for LDS: 128 x 128 needs it for 768
// cycles a step of 512 cycles of MFMAs (777 x 4096 to 2816 28 us).
//
// Offsets: a descriptor starts at the tile's first element (64-bit), so that
// offsets within it stay below 2^31; rows, columns and k past the operand's end
// point past every descriptor and read zeros.
struct Operand {
  const uint16_t* p;
  int64_t ld;  // elements between rows (of k, or of m)
  int n;       // extent in m (or n)
  int64_t low = 0;  // elements from p to its second part (0: there is none)
};

template <bool TR, int R, int NI>
struct Loader {
  uint32_t off[NI];  // byte offsets of this wave's NI load instructions
  int kc[NI];        // first k (TR: the k row) of the lane's piece
  const uint16_t* base;
  const uint16_t* base2;  // GATED: the up rows
  int64_t ld;
  u32x4 buf, buf2;
  uint32_t soff;
  int left;

  // Piece p of k row kr lies at place p ^ swizzle(kr).  32 lanes of a transposed
  // read take 32 bytes of eight rows, kr .. kr + 3 and kr + 8 .. kr + 11, which
  // must lie in different eighths of the 256 bytes of banks (rows of 192 values
  // are 384 bytes, so every other row is half way round already).
  static __device__ __forceinline__ int swizzle(int kr) {
    return (R % 128 == 0 ? (kr & 3) << 2 : ((kr >> 1) & 1) << 2) ^ (((kr >> 3) & 1) << 1);
  }
  // GATED: tile rows run over 32 gate rows from m0 and the 32 up rows `up` further, by turns
  template <bool GATED>
  __device__ __forceinline__ void init(const Operand& o, int m0, int up, int q0, int lane) {
    ld = o.ld;
    const int wide = (GATED ? up : o.n) - m0;
    if constexpr (!TR) {
      base = o.p + (int64_t)m0 * ld;
      base2 = o.p + ((int64_t)m0 + up) * ld;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = 8 * (q0 + i) + lane / 8;
        const int piece = (lane & 7) ^ ((r / 2) & 7);
        const int row = GATED ? 32 * (r / 64) + r % 32 : r;
        kc[i] = 8 * piece;
        off[i] = row < wide ? (uint32_t)((int64_t)row * ld * 2) + (uint32_t)piece * 16u : OUT_OF_RANGE;
      }
    } else {
      base = o.p + m0;
      constexpr int PPR = R / 8;  // pieces a row
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int at = 64 * (q0 + i) + lane;
        const int kr = at / PPR;
        const int piece = (at % PPR) ^ swizzle(kr);
        kc[i] = kr;
        off[i] = 8 * piece < wide ? (uint32_t)((int64_t)kr * ld * 2) + (uint32_t)piece * 16u : OUT_OF_RANGE;
      }
    }
  }
  // The loads of the step k0 .. k0 + 63, of which `end` exist (none of it: zeros,
  // without memory traffic), `part` elements from the operand's start: their
  // buffers, then load instruction i
  template <bool GATED>
  __device__ __forceinline__ void begin(int k0, int end, int64_t part = 0) {
    left = end;
    const uint32_t range = left > 0 ? OUT_OF_RANGE : 0u;
    soff = TR ? 0u : (uint32_t)k0 * 2u;
    buf = buffer_of((TR ? base + (int64_t)k0 * ld : base) + part, range);
    buf2 = buffer_of(GATED ? base2 : base, range);
  }
  template <bool GATED>
  __device__ __forceinline__ void issue(int i, int q0, uint32_t lds) const {
    dma16(GATED && ((q0 + i) / 4) % 2 ? buf2 : buf, kc[i] < left ? off[i] : OUT_OF_RANGE, soff, lds + (q0 + i) * 1024);
  }
  // fragment of 16 m (from m) and 32 k (half j of the stage): lane l holds m + l % 16, k = 32 j + 8 (l / 16) + 0..7
  static __device__ __forceinline__ u32x4 read(const uint8_t* lds, int m, int j, int lane) {
    if constexpr (!TR) {
      const int row = m + lane % 16;
      const int piece = (4 * j + lane / 16) ^ ((row / 2) & 7);
      return *(const u32x4*)(lds + (row * 128 + (piece << 4)));
    } else {
      // Lane i of a 16-lane group reads 4 values of row i / 4 and gets column i of
      // the group's 4 x 16 block.  The swizzle is the same for all of a lane's
      // rows, so a fragment's address is one exclusive or and one sum.
      const int kr = 8 * (lane / 16) + ((lane & 15) >> 2);
      const int at = kr * (R * 2) + (lane & 3) * 8 + ((m * 2) ^ (swizzle(kr) << 4));
      auto half = [&](int off) __attribute__((always_inline)) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + (at + off)));
      };
      const int k = j * (32 * R * 2);
      const s16x4 a = half(k), b = half(k + 4 * R * 2);
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// elements between the rows of partial sums
__host__ __device__ constexpr int64_t part_row(int64_t n) { return (n + 7) / 8 * 8; }

struct TileParams {
  Operand a, b;
  int K;         // k of one part
  int k_all;     // the same, or of both parts, each rounded up to whole steps
  int m_tiles, n_tiles, splits, group_m, per_xcd;
  int k_split;   // k of one split, a multiple of 64
  float* part;   // splits > 1: fp32 sums [splits][M][part_row(N)]
  LinearEpi e;
};

// GATED: the wave's second column block holds the up columns of its first.
// KS 2: two waves share a block of C, each half of every stage's k-steps, and
// add up at the end (a second wave on the SIMD where the tile has only four
// blocks).
// PARTS 2: A is the sum of two 16-bit parts, one after the other along k, and B is
// read twice; the second part first (see two_parts).
template <int DT, bool TA, bool TB, bool GATED, int BM, int BN, int WM, int WN, int KS, int NS, int PARTS = 1>
__global__ __launch_bounds__(64 * WM * WN * KS, 1) void linear_tile_kernel(TileParams prm) {
  constexpr int WAVES = WM * WN * KS;
  constexpr int JW = 2 / KS;  // MFMA k-steps of a stage and wave
  constexpr int MS = BM / WM / 32, NSUB = BN / WN / 32;  // blocks of 32 rows and columns of a wave
  constexpr int MB = 2 * MS, NB = 2 * NSUB, MH = MB / 2;  // fragments of 16
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
  constexpr int NIA = BM / 8 / WAVES, NIB = BN / 8 / WAVES, LOADS = NIA + NIB;
  static_assert(NIA >= 1 && NIB >= 1, "every wave loads");
  static_assert(!GATED || NSUB == 2, "one gate and one up block a wave");
  static_assert(NS >= 2 && NS <= 4 && NS * STAGE <= 160 * 1024, "LDS");
  // epilogue: each wave passes 32 rows of its columns through its own part of the stages
  constexpr int ROWF = 32 * NSUB + 4;  // floats a row, with padding
  constexpr int ROWS_BYTES = 32 * ROWF * 4;
  constexpr int PER_STAGE = STAGE / ROWS_BYTES;  // waves that fit in a stage
  static_assert(PER_STAGE * NS >= WAVES, "epilogue rows");
  // one array per stage: distinct objects let the compiler see that reading a
  // stage does not wait on loads still landing in the others
  __shared__ __attribute__((aligned(16))) uint8_t st0[STAGE], st1[STAGE], st2[NS > 2 ? STAGE : 16],
      st3[NS > 3 ? STAGE : 16];
  auto stage = [&](auto S_) __attribute__((always_inline)) -> uint8_t* {
    constexpr int S = decltype(S_)::value;
    if constexpr (S == 0) return st0;
    else if constexpr (S == 1) return st1;
    else if constexpr (S == 2) return st2;
    else return st3;
  };
  typedef Loader<TA, BM, NIA> LA;
  typedef Loader<TB, BN, NIB> LB;

  const int lane = lane_id(), wave = wave_id();
  const int wm = wave / WN % WM, wn = wave % WN, kh = wave / (WM * WN);

  // ---- the tile: XCD x takes a contiguous range of the tiles, which run over
  // the row tiles of a group, then column tiles, then groups, then splits
  const int logical = ((int)blockIdx.x % NUM_XCD) * prm.per_xcd + (int)blockIdx.x / NUM_XCD;
  const int tiles = prm.m_tiles * prm.n_tiles;
  const int split = logical / tiles;
  if (split >= prm.splits) return;
  const int in = logical - split * tiles;
  const int per_group = prm.group_m * prm.n_tiles;
  const int mg = in / per_group;
  const int gm = min(prm.group_m, prm.m_tiles - mg * prm.group_m);
  const int rem = in - mg * per_group;
  const int mt = mg * prm.group_m + rem % gm, nt = rem / gm;
  const int m0 = mt * BM;
  const int c0 = nt * (GATED ? BN / 2 : BN);  // first output column

  const int k_lo = split * prm.k_split, k_hi = min(prm.k_all, k_lo + prm.k_split);
  const int steps = (k_hi - k_lo + 63) / 64;  // not positive: all sums 0
  const int k_part = PARTS == 2 ? prm.k_all / 2 : 0;  // where the first part begins

  LA la;
  LB lb;
  la.template init<false>(prm.a, m0, 0, wave * NIA, lane);
  lb.template init<GATED>(prm.b, c0, prm.e.C, wave * NIB, lane);

  f32x4 acc[MB][NB];
#pragma unroll
  for (int mi = 0; mi < MB; ++mi)
#pragma unroll
    for (int ni = 0; ni < NB; ++ni) acc[mi][ni] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  auto begin = [&](int step) __attribute__((always_inline)) {
    int k0 = k_lo + 64 * step, end = k_hi - k0;
    if constexpr (PARTS == 2) {
      const bool second = k0 < k_part;
      k0 -= second ? 0 : k_part;
      end = min(end, prm.K - k0);
      la.template begin<false>(k0, end, second ? prm.a.low : 0);
    } else {
      la.template begin<false>(k0, end);
    }
    lb.template begin<GATED>(k0, end);
  };
  // fp16's second part is 2^SHIFT times its value: the sums so far, where the first begins
  auto scale = [&](float by) __attribute__((always_inline)) {
#pragma unroll
    for (int mi = 0; mi < MB; ++mi)
#pragma unroll
      for (int ni = 0; ni < NB; ++ni) acc[mi][ni] *= by;
  };
  const int turn = PARTS == 2 ? (k_part - k_lo) / 64 : 0;
  auto issue = [&](auto S_, int i) __attribute__((always_inline)) {  // load i of the step, into stage S
    const uint32_t st = lds_address(stage(S_));
    if (i < NIA) la.template issue<false>(i, wave * NIA, st);
    else lb.template issue<GATED>(i - NIA, wave * NIB, st + A_BYTES);
  };
  // fragment i of half h of the wave's rows, and of its columns, at k-step j
  auto read_a = [&](const uint8_t* st, int j, int h, int i, u32x4 (&af)[MH]) __attribute__((always_inline)) {
    af[i] = LA::read(st, (wm * MB + h * MH + i) * 16, kh * JW + j, lane);
  };
  auto read_b = [&](const uint8_t* st, int j, int i, u32x4 (&bf)[NB]) __attribute__((always_inline)) {
    bf[i] = LB::read(st + A_BYTES, (wn * NB + i) * 16, kh * JW + j, lane);
  };

  // A k-step's MFMAs run in two halves of the wave's rows; the next half's
  // fragments are read behind the first of them.  Before the last half of a stage
  // its reads are complete: one wait for the next stage's loads and one barrier,
  // after which the next stage's first fragments are read, and the loads that
  // refill this stage NS steps ahead go out, behind one MFMA each.  (All reads
  // before a half's MFMAs: 777 x 4096 to 2816 30.3 against 27.8 us, 4096 x 11008
  // 267 against 255.)  16 x 16 x 32 products: 8% faster than 32 x 32 x 16 at
  // 8192^3, where the card's power sets the clock; four waves of 128 x 128 spill.
  if (steps > 0) {
    u32x4 af[2][MH], bf[2][NB];
    for_each<0, NS>([&](auto S_) __attribute__((always_inline)) {
      begin(decltype(S_)::value);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) issue(S_, i);
      __builtin_amdgcn_sched_barrier(0);
      return true;
    });
    wait_vmcnt<(NS - 1) * LOADS>();
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int n = 0; n < NB; ++n) read_b(st0, 0, n, bf[0]);
#pragma unroll
    for (int n = 0; n < MH; ++n) read_a(st0, 0, 0, n, af[0]);
    auto step = [&](auto S_, int i) __attribute__((always_inline)) {
      constexpr int S = decltype(S_)::value, N = (S + 1) % NS;
      if constexpr (PARTS == 2 && DT == ACT_F16) {
        if (i == turn) scale(1.0f / (1 << SHIFT_LOW));
      }
      constexpr int B0 = KS == 1 ? 0 : S & 1;  // the columns' registers of the first k-step
      static_assert(KS == 1 || NS % 2 == 0, "registers by turns");
      const uint8_t* st = stage(S_);
      constexpr int HALVES = 2 * JW;
      for_each<0, HALVES>([&](auto H_) __attribute__((always_inline)) {
        constexpr int hf = decltype(H_)::value, j = hf / 2, B = (B0 + j) & 1;
        constexpr bool last = hf == HALVES - 1;
        if constexpr (last) {
          wait_vmcnt<(NS - 2) * LOADS>();      // this wave's loads of the next step have landed
          __builtin_amdgcn_s_waitcnt(0xC07F);  // and its reads of this stage (lgkmcnt 0)
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_sched_barrier(0);
          begin(i + NS);
        }
        const uint8_t* from = last ? stage(IC<N>{}) : st;
        constexpr int jn = last ? 0 : (hf + 1) / 2, hn = last ? 0 : (hf + 1) % 2;
        constexpr int NRB = last || hf % 2 == 1 ? NB : 0, READS = NRB + MH;
        constexpr int MMAS = MH * NB;
        for_each<0, MMAS>([&](auto M_) __attribute__((always_inline)) {
          constexpr int m = decltype(M_)::value;
          f32x4& c = acc[(hf % 2) * MH + m / NB][m % NB];
          c = mfma16<DT>(af[hf & 1][m / NB], bf[B][m % NB], c);
          __builtin_amdgcn_sched_barrier(0);
          constexpr int r0 = 2 * m * READS / MMAS, r1 = 2 * (m + 1) * READS / MMAS;
          for_each<(r0 < READS ? r0 : READS), (r1 < READS ? r1 : READS)>([&](auto R_) __attribute__((always_inline)) {
            constexpr int r = decltype(R_)::value;
            if constexpr (r < NRB) read_b(from, jn, r, bf[B ^ 1]);
            else read_a(from, jn, hn, r - NRB, af[last ? 0 : (hf + 1) & 1]);
            return true;
          });
          if constexpr (last) {
#pragma unroll
            for (int l = m * LOADS / MMAS; l < (m + 1) * LOADS / MMAS; ++l) issue(S_, l);
          }
          __builtin_amdgcn_sched_barrier(0);
          return true;
        });
        __builtin_amdgcn_sched_barrier(0);
        return true;
      });
    };
    int i = 0;
    for (; i + NS <= steps; i += NS)
      for_each<0, NS>([&](auto S_) __attribute__((always_inline)) {
        step(S_, i + decltype(S_)::value);
        return true;
      });
    for_each<0, NS - 1>([&](auto S_) __attribute__((always_inline)) {
      if (i + decltype(S_)::value >= steps) return false;
      step(S_, i + decltype(S_)::value);
      return true;
    });
  }
  if constexpr (PARTS == 2 && DT == ACT_F16)
    scale(k_hi > k_part ? (float)(1 << SHIFT_DZ) : (float)(1 << SHIFT_DZ) / (1 << SHIFT_LOW));
  wait_vmcnt<0>();  // no load into LDS lands after this
  __syncthreads();

  // ---- KS 2: each wave of a pair passes the row blocks that the other finishes
  constexpr int MO = MS / KS;  // row blocks that a wave finishes: kh MO ..
  static_assert(MS % KS == 0, "whole row blocks");
  if constexpr (KS == 2) {
    constexpr int TILE = NSUB * 4096;  // bytes of a 32-row block's accumulators
    constexpr int FIT = STAGE / TILE;
    static_assert(FIT * NS >= WAVES * MO, "accumulators");
    auto at = [&](int w, int mo) __attribute__((always_inline)) {
      const int i = w * MO + mo, p = i / FIT;
      return (f32x4*)((p == 0 ? st0 : p == 1 ? st1 : p == 2 ? st2 : st3) + i % FIT * TILE);
    };
    constexpr int FRAGS = 2 * NB;  // fragments of a 32-row block
#pragma unroll
    for (int mo = 0; mo < MO; ++mo)
#pragma unroll
      for (int q = 0; q < FRAGS; ++q)
        at(wave, mo)[q * 64 + lane] = kh == 0 ? acc[2 * (MO + mo) + q / NB][q % NB] : acc[2 * mo + q / NB][q % NB];
    __syncthreads();
#pragma unroll
    for (int mo = 0; mo < MO; ++mo)
#pragma unroll
      for (int q = 0; q < FRAGS; ++q) {
        const f32x4 v = at(wave ^ (WM * WN), mo)[q * 64 + lane];
        f32x4& c = acc[2 * mo + q / NB][q % NB];
        c = kh == 0 ? c + v : v + acc[2 * (MO + mo) + q / NB][q % NB];  // the first half of k, then the second
      }
    __syncthreads();
  }

  // ---- epilogue: register r of lane l holds row 4 (l / 16) + r, column l % 16 of a fragment
  const int M = prm.a.n;
  const int place = wave / PER_STAGE;
  float* rows = (float*)((place == 0 ? st0 : place == 1 ? st1 : place == 2 ? st2 : st3) +
                         wave % PER_STAGE * ROWS_BYTES);
  constexpr int LPR = GATED ? 4 : 4 * NSUB;  // lanes a row, eight columns each
  constexpr int IT = LPR / 2;                // turns of 64 / LPR rows
  const int w0 = c0 + wn * (GATED ? 32 : 32 * NSUB);  // the wave's first output column
  const int row0 = m0 + (wm * MS + kh * MO) * 32;     // and row
  auto eight = [](const float* q, float (&v)[8]) __attribute__((always_inline)) {
    const f32x4 a = *(const f32x4*)q, b = *(const f32x4*)(q + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  };
  // Nothing but a scale and a residual: short enough to unroll, so that the
  // residual is loaded early and stores follow each other (a product of one step,
  // 4096 x 64 to 4096: 16.5 to 15.2 us; 4096 x 11008 to 4096 with a residual: 294
  // to 292.5)
  const bool simple =
      !GATED && prm.splits == 1 && prm.e.vec && prm.e.act == LIN_NONE && !prm.e.bias && !prm.e.pre;
  struct Residual {
    u32x4 v[IT][2];
  };
  auto residual = [&](int mi, Residual& q) __attribute__((always_inline)) {
    if (!prm.e.res) return;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int64_t t = row0 + mi * 32 + lane / LPR + it * (64 / LPR);
      const int n = w0 + 8 * (lane % LPR);
      if (t >= M || n + 8 > prm.e.C) continue;
      const int64_t at = t * prm.e.ldr + n;
      if (prm.e.out_f32) {
        q.v[it][0] = load16((const float*)prm.e.res + at);
        q.v[it][1] = load16((const float*)prm.e.res + at + 4);
      } else {
        q.v[it][0] = load16((const uint16_t*)prm.e.res + at);
      }
    }
  };
  Residual here;
  if (simple) residual(0, here);
#pragma unroll
  for (int mi = 0; mi < MO; ++mi) {
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int ni = 0; ni < NB; ++ni)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          rows[(16 * a + 4 * (lane / 16) + r) * ROWF + ni * 16 + lane % 16] = acc[2 * mi + a][ni][r];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int64_t t0 = row0 + mi * 32;
    if (simple) {
      // the next rows' residual is under way while these are written
      Residual next;
      if (mi + 1 < MO) residual(mi + 1, next);
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const int r = lane / LPR + it * (64 / LPR), c = 8 * (lane % LPR);
        if (t0 + r >= M || w0 + c >= prm.e.C) continue;
        float z[8], u[8];
        eight(rows + r * ROWF + c, z);
        if (w0 + c + 8 > prm.e.C) {
          finish<DT, false, 8>(prm.e, t0 + r, w0 + c, z, u);
          continue;
        }
        if (prm.e.row_scale) {
          const float rs = prm.e.row_scale[t0 + r];
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] *= rs;
        }
        if (prm.e.res) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            // (a bit cast of a vector's element itself gives element 0)
            const uint32_t h = here.v[it][0][j / 2], f = here.v[it][j / 4][j % 4];
            z[j] += prm.e.out_f32 ? __builtin_bit_cast(float, f) : half_to_f32<DT>(j % 2 ? h >> 16 : h & 0xFFFFu);
          }
        }
        store_n<DT, 8>(prm.e.out, prm.e.out_f32, (t0 + r) * prm.e.ldo + w0 + c, 8, true, z);
      }
      here = next;
    } else if (prm.splits > 1 || prm.e.vec) {
#pragma unroll 1
      for (int r = lane / LPR; r < 32; r += 64 / LPR) {
        const int c = 8 * (lane % LPR);
        const float* src = rows + r * ROWF + c;
        float z[8], u[8];
        eight(src, z);
        if constexpr (GATED) eight(src + 32, u);
        if (t0 + r < M && w0 + c < prm.e.C) {
          if (prm.splits > 1)  // whole eights: the rows of `part` are padded
            store_n<DT, 8>(prm.part, true, ((int64_t)split * M + t0 + r) * part_row(prm.e.C) + w0 + c, 8, true, z);
          else
            finish<DT, GATED, 8>(prm.e, t0 + r, w0 + c, z, u);
        }
      }
    } else {
      // rows that do not start aligned: a lane a column, so that a store still covers whole lines
      constexpr int CW = GATED ? 32 : 32 * NSUB;
#pragma unroll 1
      for (int r = lane / CW; r < 32; r += 64 / CW) {
        const int c = lane % CW;
        float z[1] = {rows[r * ROWF + c]}, u[1] = {0.0f};
        if constexpr (GATED) u[0] = rows[r * ROWF + 32 + c];
        if (t0 + r < M && w0 + c < prm.e.C) finish<DT, GATED, 1>(prm.e, t0 + r, w0 + c, z, u);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------- stream kernel --
//
// Few tokens or few columns: a workgroup computes 16 G columns of 16 H tokens,
// its eight waves taking every eighth 64 of k (a wave's operands are used by no
// other, so they go from memory to registers; no barrier before the end).  W is
// the MFMA's row operand, so a lane ends with four consecutive columns of one
// token.  A load takes 64 bytes of sixteen rows; a unit of 64 k is two of them a
// row group and two MFMAs a block, and the next unit's loads are under way while
// one is multiplied.  The waves' sums go through LDS.
//
// One token is bound by the bytes of W: 22016 rows of 4096 in 34.7 us, 5.2 TB/s
// (a copy reaches 5.1).  More are bound by what the L2s give, about 9 TB/s in
// this pattern for 16 (G + H) rows a workgroup, which is why larger G and H
// (tried up to 4 and 4) lose to the tile kernel where they read less.
// Non-temporal loads of W were slower (8.9 against 8.1 us for 4096 x 4096).
// GATED: groups G / 2 .. G - 1 are the up columns of the first G / 2.
struct StreamParams {
  const uint16_t* x;
  const uint16_t* w;
  int64_t ldx, ldw;
  int T, N, K, t_tiles;
  LinearEpi e;
};

template <int DT, bool GATED, int G, int H>
__global__ __launch_bounds__(512, 4) void linear_stream_kernel(StreamParams prm) {
  constexpr int WAVES = 8;
  constexpr int OG = GATED ? G / 2 : G;  // groups of output columns
  __shared__ f32x4 sums[WAVES][G * H][64];
  const int lane = lane_id(), wave = wave_id(), r = lane % 16, g = lane / 16;
  // tokens fastest: the workgroups that run at a time share their rows of W
  const int tt = (int)blockIdx.x % prm.t_tiles, ct = (int)blockIdx.x / prm.t_tiles;
  const int t0 = tt * 16 * H, c0 = ct * 16 * OG;
  const rsrc_t rx = make_rsrc(prm.x + (int64_t)t0 * prm.ldx, OUT_OF_RANGE);
  const rsrc_t rw = make_rsrc(prm.w + (int64_t)c0 * prm.ldw, OUT_OF_RANGE);
  const rsrc_t ru = make_rsrc(prm.w + ((int64_t)prm.e.C + c0) * prm.ldw, OUT_OF_RANGE);
  uint32_t xo[H], wo[G];
#pragma unroll
  for (int h = 0; h < H; ++h)
    xo[h] = t0 + 16 * h + r < prm.T ? (uint32_t)((16 * h + r) * prm.ldx * 2) + (uint32_t)g * 16u : OUT_OF_RANGE;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int c = 16 * (i % OG) + r;
    wo[i] = c0 + c < prm.e.C ? (uint32_t)(c * prm.ldw * 2) + (uint32_t)g * 16u : OUT_OF_RANGE;
  }
  struct Unit {
    u32x4 w[G][2], x[H][2];
  };
  auto load = [&](Unit& v, int u) __attribute__((always_inline)) {
    const int k = 64 * u + 8 * g;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const bool in = k + 32 * b < prm.K;
      const int at = 128 * u + 64 * b;
#pragma unroll
      for (int i = 0; i < G; ++i)
        v.w[i][b] = __builtin_amdgcn_raw_buffer_load_b128(GATED && i >= OG ? ru : rw,
                                                          (int)(in ? wo[i] + at : OUT_OF_RANGE), 0, 0);
#pragma unroll
      for (int h = 0; h < H; ++h)
        v.x[h][b] = __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(in ? xo[h] + at : OUT_OF_RANGE), 0, 0);
    }
  };
  f32x4 acc[G][H];
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int h = 0; h < H; ++h) acc[i][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](const Unit& v) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int h = 0; h < H; ++h) acc[i][h] = mfma16<DT>(v.w[i][b], v.x[h][b], acc[i][h]);
  };
  // units past the last are zeros without memory traffic
  const int units = (prm.K + 63) / 64;
  Unit a, b;
  load(a, wave);
  for (int u = wave; u < units; u += 2 * WAVES) {
    load(b, u + WAVES);
    __builtin_amdgcn_sched_barrier(0);
    multiply(a);
    load(a, u + 2 * WAVES);
    __builtin_amdgcn_sched_barrier(0);
    multiply(b);
  }
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int h = 0; h < H; ++h) sums[wave][i * H + h][lane] = acc[i][h];
  __syncthreads();
  // a thread eight columns of a token: lanes 32 q + t and 32 q + 16 + t of a group hold columns 8 q .. 8 q + 7
  for (int o = threadIdx.x; o < OG * 2 * 16 * H; o += 512) {
    const int q = o % (2 * OG), t = o / (2 * OG);
    const int i = q / 2, at = 32 * (q % 2) + t % 16, h = t / 16;
    auto total = [&](int grp, float (&v)[8]) __attribute__((always_inline)) {
      f32x4 lo = sums[0][grp * H + h][at], hi = sums[0][grp * H + h][at + 16];
#pragma unroll
      for (int wv = 1; wv < WAVES; ++wv) {
        lo += sums[wv][grp * H + h][at];
        hi += sums[wv][grp * H + h][at + 16];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = lo[j];
        v[4 + j] = hi[j];
      }
    };
    const int n = c0 + 16 * i + 8 * (q % 2);
    if (t0 + t < prm.T && n < prm.e.C) {
      float z[8], u[8];
      total(i, z);
      if constexpr (GATED) total(OG + i, u);
      finish<DT, GATED, 8>(prm.e, t0 + t, n, z, u);
    }
  }
}

// The sums of the splits in order, and the epilogue: a thread W columns of a row
// (one where the rows it writes do not start aligned).  A launch and the sums'
// bytes: 2.9 us for five shares of 64 x 4096.
template <int DT, int W>
__global__ __launch_bounds__(256) void linear_join_kernel(const float* __restrict__ part, int splits, int M, int N,
                                                          LinearEpi e) {
  const int chunks = (e.C + W - 1) / W;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)M * chunks) return;
  const int64_t t = i / chunks;
  const int n = (int)(i - t * chunks) * W;
  const bool gated = e.act == LIN_SWIGLU;
  const bool up_vec = e.C % 4 == 0 && n + W <= e.C;
  float z[W], u[W];
#pragma unroll
  for (int j = 0; j < W; ++j) z[j] = u[j] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const int64_t row = ((int64_t)s * M + t) * part_row(N) + n;
    float v[W];
    load_n<DT, W>(part, true, row, W, true, v);  // past the end: the padding, or another half's
#pragma unroll
    for (int j = 0; j < W; ++j) z[j] += v[j];
    if (gated) {
      load_n<DT, W>(part, true, row + e.C, e.C - n, up_vec, v);
#pragma unroll
      for (int j = 0; j < W; ++j) u[j] += v[j];
    }
  }
  if (gated) finish<DT, true, W>(e, t, n, z, u);
  else finish<DT, false, W>(e, t, n, z, u);
}

// ------------------------------------------------------- gradient of z ----
//
// A workgroup takes g.rows rows and 8 g.across columns (gated: of each half), a
// thread eight columns of every (256 / g.across)-th row.  dz is the operand of both
// products: rounded to their 16 bits, which is what the gradient that came in was
// rounded by, or in two parts where that has more (g.low).  The sums of bias and
// row_scale use it unrounded and go to part[row block][N] and row_part[column
// block][T], joined in order (one block's are the result).  The
// last column block writes zeros up to ldz.  Bound by its bytes: 58 MB of 4096 x 2 x
// 1408 in 16 to 17.5 us, 3.5 TB/s (one column block a workgroup of 16 rows: 60 us).
template <int DT>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinearGrad g) {
  __shared__ float sums[256][17];
  __shared__ float row_sum[LINEAR_DZ_ROWS];
  const int tid = threadIdx.x, across = g.across;
  const bool gated = g.act == LIN_SWIGLU;
  const int64_t t0 = (int64_t)blockIdx.x * g.rows;
  const int rows = (int)min((int64_t)g.rows, g.T - t0);
  const int n = 8 * ((int)blockIdx.y * across + tid % across);
  const int left = g.C - n;
  const bool vec = g.vec && left >= 8;
  float cs[8], cu[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cs[j] = cu[j] = 0.0f;
#pragma unroll 2
  for (int r = tid / across; r < rows; r += 256 / across) {
    const int64_t t = t0 + r;
    float dot = 0.0f;
    if (left > 0) {
      float d[8], d2[8], z[8], u[8];  // columns past the end: all 0
      load_n<DT, 8>(g.g, g.g_f32, t * g.ldg + n, left, vec, d);
      if (g.z) load_n<DT, 8>(g.z, false, t * g.ldz_in + n, left, vec, z);
      if (gated) load_n<DT, 8>(g.z, false, t * g.ldz_in + g.C + n, left, vec, u);
      const float rs = g.rs ? g.rs[t] : 1.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gv = g.rs ? d[j] * rs : d[j];
        float a = 0.0f, slope = 1.0f;
        if (g.z) a = activate_slope(gated ? LIN_SILU : g.act, z[j], slope);
        d2[j] = 0.0f;
        if (gated) {
          dot += d[j] * (a * u[j]);
          d2[j] = gv * a;
          slope *= u[j];
        } else {
          dot += d[j] * a;
        }
        d[j] = gv * slope;
        cs[j] += d[j];
        cu[j] += d2[j];
      }
      if (g.dz && g.low) {
        store_parts<DT>(g.dz + t * g.ldz + n, g.low, left, vec, d);
        if (gated) store_parts<DT>(g.dz + t * g.ldz + g.C + n, g.low, left, vec, d2);
      } else if (g.dz) {
        store_n<DT, 8>(g.dz, false, t * g.ldz + n, left, vec, d);
        if (gated) store_n<DT, 8>(g.dz, false, t * g.ldz + g.C + n, left, vec, d2);
      }
    }
    if (g.row_part) {  // the threads of a row are of one wave
      for (int o = 1; o < across; o <<= 1) dot += lane_read_f(dot, lane_id() ^ o);
      if (tid % across == 0) row_sum[r] = dot;
    }
  }
  if (g.dz && blockIdx.y + 1 == gridDim.y) {
    const int pad = (int)(g.ldz - g.N);
    for (int i = tid; i < rows * pad; i += 256) {
      uint16_t* z = g.dz + (t0 + i / pad) * g.ldz + g.N + i % pad;
      z[0] = 0;
      if (g.low) z[g.low] = 0;
    }
  }
  if (g.part) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sums[tid][j] = cs[j];
      sums[tid][8 + j] = cu[j];
    }
  }
  __syncthreads();
  if (g.part) {
    float* p = g.part + (int64_t)blockIdx.x * g.N;
    for (int i = tid; i < across * 16; i += 256) {
      const int c = i / 16, j = i % 16;
      const int m = 8 * ((int)blockIdx.y * across + c) + j % 8;
      float v = 0.0f;
      for (int q = c; q < 256; q += across) v += sums[q][j];
      if (m < g.C && (j < 8 || gated)) p[j < 8 ? m : g.C + m] = v;
    }
  }
  if (g.row_part)
    for (int r = tid; r < rows; r += 256) g.row_part[(int64_t)blockIdx.y * g.T + t0 + r] = row_sum[r];
}

// out[i] = sum over b of part[b][i]: 16 groups of every 16th b, then the groups.
// A workgroup 64 of the n; 256 blocks of 64 columns in 2.3 us (one thread a column:
// 60 us).
__global__ __launch_bounds__(1024) void linear_sums_kernel(const float* __restrict__ part, int blocks, int64_t n,
                                                           float* __restrict__ out) {
  __shared__ float sums[16][64];
  const int group = threadIdx.x / 64, lane = lane_id();
  const int64_t i = (int64_t)blockIdx.x * 64 + lane;
  float v = 0.0f;
  if (i < n) {
#pragma unroll 8
    for (int b = group; b < blocks; b += 16) v += part[(int64_t)b * n + i];
  }
  sums[group][lane] = v;
  __syncthreads();
  if (group == 0 && i < n) {
#pragma unroll
    for (int q = 1; q < 16; ++q) v += sums[q][lane];
    out[i] = v;
  }
}

// -------------------------------------------------------------- launchers --

constexpr int CUS = 256;
constexpr int64_t MAX_GRID = 1 << 22;  // workgroups of up to 512 threads: a launch has fewer than 2^32 threads

// the summed index, of both parts (each rounded up to whole steps)
constexpr int64_t k_of_parts(int64_t K, int parts) { return parts == 2 ? 2 * ((K + 63) / 64 * 64) : K; }

struct Plan {
  int bm, bn;  // rows and columns of a tile
  int splits;
  double us;  // what the product is expected to take
};

// The tile and the split of k of a product M x N over K: the least of what the
// forms are expected to take, rounds of workgroups times (steps of a share times
// us a step, or the operands' bytes at 5 TB/s, and us to begin and to finish),
// and the join of the shares.  Measured us a step of 64 k: 256 x 256 1.52, 192 x
// 256 1.25, 128 x 256 0.9, 192 x 128 0.66, 128 x 128 0.45 (154 workgroups) to 0.5
// (256); 64 x 64 0.25 to 0.45 (512, two a CU).  Gated, the waves' 32 gate and 32 up
// columns leave four waves for 192 x 128, too few (1237 x 4096 to 2 x 2048 55 us
// against 52 with 128 x 256).  Results against a fixed tile of 128 in brackets, us:
// 64 x 2816 to 4096 11.6 (15.1), 2048 x 4096 to 4096 63 (77), 4096 x 11008 to 4096
// 255 (450); against 128 x 256 1237 x 4096 to 4096 48 (54), 8192 x 4096 to 1408 97
// (112 with 128 x 128).
// Two parts: 256 x 256 leaves too few registers (up to 38 spilled; where none is, the
// router's gradients take as long with it).
Plan plan_of(int64_t M, int64_t N, int64_t K, bool gated = false, int parts = 1) {
  Plan p{128, 128, 1, 0.0};
  if (M < 1 || N < 1) return p;
  const int64_t steps = (K + 63) / 64;
  const double bytes_us = (double)((M + N) * K) * 2.0 / 5.0e6;
  auto offer = [&](int bm, int bn, int64_t at_once, double step, double ends, int64_t splits) {
    const int64_t work = ((M + bm - 1) / bm) * ((N + bn - 1) / bn) * splits;
    if (work > MAX_GRID && bm * bn < (parts == 1 ? 256 : 192) * 256) return;  // but for the largest tile
    const int64_t share = (steps + splits - 1) / splits;
    double us = std::max((double)((work + at_once - 1) / at_once) * ((double)share * step + ends), bytes_us + ends);
    if (splits > 1) us += 3.5 + (double)(splits * M * N) * 4.0 / 2.5e6;
    if (p.us == 0.0 || us < p.us) p = Plan{bm, bn, (int)splits, us};
  };
  if (parts == 1) offer(256, 256, CUS, 1.52, 8.0, 1);
  offer(192, 256, CUS, 1.25, 7.5, 1);
  offer(128, 256, CUS, 0.9, 6.0, 1);
  if (!gated) offer(192, 128, CUS, 0.66, 6.0, 1);
  const int64_t wide = ((M + 127) / 128) * ((N + 127) / 128), small = ((M + 63) / 64) * ((N + 63) / 64);
  auto filled = [](int64_t work, int64_t at_once) { return (double)std::min(work, at_once) / (double)at_once; };
  for (int64_t s : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32}) {
    if (s > 1 && 2 * s > steps) break;  // shares of two steps or more
    offer(128, 128, CUS, 0.38 + 0.12 * filled(wide * s, CUS), 4.5, s);
    offer(64, 64, 2 * CUS, 0.2 + 0.25 * filled(small * s, 2 * CUS), 4.0, s);
  }
  return p;
}

template <int DT, bool TA, bool TB, bool GATED, int PARTS = 1>
hipError_t launch_tile(const Operand& a, const Operand& b, int N, int K, const LinearEpi& e, float* part,
                       hipStream_t st) {
  TileParams prm;
  prm.a = a;
  prm.b = b;
  prm.K = K;
  prm.k_all = (int)k_of_parts(K, PARTS);
  prm.e = e;
  prm.part = part;
  const Plan p = plan_of(a.n, N, prm.k_all, GATED, PARTS);
  const bool split = p.splits > 1;
  if (split && !part) return hipErrorInvalidValue;
  const int64_t steps = (prm.k_all + 63) / 64;
  prm.splits = p.splits;
  prm.k_split = (int)((steps + p.splits - 1) / p.splits) * 64;
  prm.m_tiles = (a.n + p.bm - 1) / p.bm;
  const int C = split ? N : e.C;
  prm.e.C = C;
  // gated: half of the tile's columns, but for the 64-row tile, which is 64 x 128 then
  const int cols = GATED && !split && p.bm != 64 ? p.bn / 2 : p.bn;
  prm.n_tiles = (C + cols - 1) / cols;
  prm.group_m = std::min(prm.m_tiles, 8);
  const int64_t total = (int64_t)prm.m_tiles * prm.n_tiles * prm.splits;
  prm.per_xcd = (int)((total + NUM_XCD - 1) / NUM_XCD);
  const dim3 grid((unsigned)(prm.per_xcd * NUM_XCD));
  auto go = [&](const char* name, auto kern, unsigned threads) {
    note_launch(name);
    return launch_kernel(kern, grid, threads, 0, st, prm);
  };
  if constexpr (PARTS == 1) {
    if (p.bm == 256) return go("linear_256x256", linear_tile_kernel<DT, TA, TB, GATED, 256, 256, 2, 4, 1, 2>, 512);
  }
  if constexpr (!GATED) {
    if (p.bm == 192 && p.bn == 128)
      return go("linear_192x128", linear_tile_kernel<DT, TA, TB, false, 192, 128, 2, 4, 1, 4, PARTS>, 512);
  }
  if (p.bm == 192) return go("linear_192x256", linear_tile_kernel<DT, TA, TB, GATED, 192, 256, 2, 4, 1, 2, PARTS>, 512);
  if (p.bn == 256) return go("linear_128x256", linear_tile_kernel<DT, TA, TB, GATED, 128, 256, 2, 4, 1, 3, PARTS>, 512);
  if (!split && p.bm == 128) return go("linear_128x128", linear_tile_kernel<DT, TA, TB, GATED, 128, 128, 2, 2, 2, 4, PARTS>, 512);
  if constexpr (GATED) {  // 64 columns of each half
    if (!split) return go("linear_64x128", linear_tile_kernel<DT, TA, TB, true, 64, 128, 2, 2, 1, 3, PARTS>, 256);
  }
  const hipError_t r = p.bm == 64
                           ? go("linear_64x64", linear_tile_kernel<DT, TA, TB, false, 64, 64, 2, 2, 1, 4, PARTS>, 256)
                           : go("linear_128x128", linear_tile_kernel<DT, TA, TB, false, 128, 128, 2, 2, 2, 4, PARTS>, 512);
  if (r != hipSuccess || !split) return r;
  const int w = e.vec ? 8 : 1;
  const int64_t threads = (int64_t)a.n * ((e.C + w - 1) / w);
  note_launch("linear_join");
  return launch_kernel(e.vec ? linear_join_kernel<DT, 8> : linear_join_kernel<DT, 1>, (unsigned)((threads + 255) / 256),
                       256, 0, st, part, p.splits, a.n, N, e);
}

// Groups of 16 columns and 16 tokens of a workgroup of the stream kernel
struct StreamPlan {
  int g, h;  // g 0: the tile kernel instead
};

// Where it is expected to take less than the tile kernel: a workgroup loads
// 16 G rows of W and up to 16 H tokens, which the L2s give at about 9 TB/s in
// this pattern, and a wave's units take 0.5 us each.  (16 x 4096 to 4096 10.4
// against 14.8 us, 777 x 4096 to 64 9.9 against 13.4; 64 x 2816 to 4096 18.0
// against 11.5.)
StreamPlan stream_plan(int64_t T, int64_t N, int64_t K, bool gated) {
  const int g = gated ? 2 : 1;
  auto bytes = [&](int h) {
    return ((T + 16 * h - 1) / (16 * h)) * ((N + 16 * g - 1) / (16 * g)) * (16 * g + std::min<int64_t>(T, 16 * h)) * 2 * K;
  };
  const int h = T > 16 && bytes(2) < bytes(1) && ((T + 31) / 32) * ((N + 16 * g - 1) / (16 * g)) >= CUS ? 2 : 1;
  const double us = 2.5 + std::max((double)bytes(h) / 9.0e6, 0.5 * (double)((K + 511) / 512));
  if (((T + 16 * h - 1) / (16 * h)) * ((N + 16 * g - 1) / (16 * g)) > MAX_GRID) return StreamPlan{0, 0};
  return us <= plan_of(T, N, K, gated).us ? StreamPlan{g, h} : StreamPlan{0, 0};
}

template <int DT, bool GATED>
hipError_t launch_stream(const StreamPlan& p, const void* x, int64_t ldx, int T, const void* w, int64_t ldw, int N,
                         int K, const LinearEpi& e, hipStream_t st) {
  StreamParams prm{(const uint16_t*)x, (const uint16_t*)w, ldx, ldw, T, N, K, (T + 16 * p.h - 1) / (16 * p.h), e};
  const int cols = GATED ? 8 * p.g : 16 * p.g;
  const unsigned grid = (unsigned)((int64_t)prm.t_tiles * ((e.C + cols - 1) / cols));
  auto go = [&](auto kern) {
    note_launch(p.h == 2 ? "linear_stream_2" : "linear_stream_1");
    return launch_kernel(kern, grid, 512, 0, st, prm);
  };
  return p.h == 2 ? go(linear_stream_kernel<DT, GATED, GATED ? 2 : 1, 2>)
                  : go(linear_stream_kernel<DT, GATED, GATED ? 2 : 1, 1>);
}

template <int DT>
hipError_t forward(const void* x, int64_t ldx, int T, const void* w, int64_t ldw, int N, int K, const LinearEpi& e,
                   float* part, hipStream_t st) {
  const bool gated = e.act == LIN_SWIGLU;
  const StreamPlan p = stream_plan(T, N, K, gated);
  if (p.g)
    return gated ? launch_stream<DT, true>(p, x, ldx, T, w, ldw, N, K, e, st)
                 : launch_stream<DT, false>(p, x, ldx, T, w, ldw, N, K, e, st);
  const Operand a{(const uint16_t*)x, ldx, T}, b{(const uint16_t*)w, ldw, N};
  if (gated) return launch_tile<DT, false, false, true>(a, b, N, K, e, part, st);
  return launch_tile<DT, false, false, false>(a, b, N, K, e, part, st);
}

LinearEpi plain_out(void* out, int64_t ld, int C) {
  LinearEpi e{};
  e.out = out;
  e.ldo = ld;
  e.C = C;
  e.act = LIN_NONE;
  e.vec = ld % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
  return e;
}

template <int DT>
hipError_t backward(const LinearGrad& g, const void* x, int64_t ldx, const void* w, int64_t ldw, int K, void* dx,
                    int64_t ldx_out, void* dw, int64_t ldw_out, float* dbias, float* drs, const uint16_t* dz,
                    int64_t ldz, float* part, hipStream_t st) {
  if (g.T && (g.dz || g.part || g.row_part)) {
    note_launch("linear_dz");
    const hipError_t r = launch_kernel(linear_dz_kernel<DT>, dim3((unsigned)g.blocks, (unsigned)g.column_blocks), 256, 0,
                                       st, g);
    if (r != hipSuccess) return r;
  }
  auto sums = [&](const float* p, int blocks, int64_t n, float* out) {
    note_launch("linear_sums");
    return launch_kernel(linear_sums_kernel, (unsigned)((n + 63) / 64), 1024, 0, st, p, blocks, n, out);
  };
  if (dbias && g.part != dbias) {
    const hipError_t r = sums(g.part, g.blocks, g.N, dbias);
    if (r != hipSuccess) return r;
  }
  if (g.T && drs && g.row_part != drs) {
    const hipError_t r = sums(g.row_part, g.column_blocks, g.T, drs);
    if (r != hipSuccess) return r;
  }
  if (dx) {
    const Operand a{dz, ldz, (int)g.T, g.low}, b{(const uint16_t*)w, ldw, K};
    const LinearEpi e = plain_out(dx, ldx_out, K);
    const hipError_t r = g.low ? launch_tile<DT, false, true, false, 2>(a, b, K, g.N, e, part, st)
                               : launch_tile<DT, false, true, false>(a, b, K, g.N, e, part, st);
    if (r != hipSuccess) return r;
  }
  if (dw) {
    const Operand a{dz, ldz, g.N, g.low}, b{(const uint16_t*)x, ldx, K};
    const LinearEpi e = plain_out(dw, ldw_out, K);
    return g.low ? launch_tile<DT, true, true, false, 2>(a, b, K, (int)g.T, e, part, st)
                 : launch_tile<DT, true, true, false>(a, b, K, (int)g.T, e, part, st);
  }
  return hipSuccess;
}

}  // namespace

static int64_t part_bytes(const Plan& p, int64_t M, int64_t N) {
  return p.splits > 1 ? (int64_t)p.splits * M * part_row(N) * 4 : 0;
}

int64_t linear_forward_bytes(int64_t T, int64_t N, int64_t K) {
  int64_t bytes = 0;  // gated and not: the larger
  for (bool gated : {false, true})
    if (!stream_plan(T, N, K, gated).g) bytes = std::max(bytes, part_bytes(plan_of(T, N, K, gated), T, N));
  return bytes;
}

int64_t linear_part_bytes(int64_t M, int64_t N, int64_t K, int parts) {
  return part_bytes(plan_of(M, N, k_of_parts(K, parts), false, parts), M, N);
}

hipError_t launch_linear(const void* x, int dt, int64_t ldx, int T, const void* w, int64_t ldw, int N, int K,
                         const LinearEpi& e, float* part, hipStream_t st) {
  return dt == ACT_BF16 ? forward<ACT_BF16>(x, ldx, T, w, ldw, N, K, e, part, st)
                        : forward<ACT_F16>(x, ldx, T, w, ldw, N, K, e, part, st);
}

hipError_t launch_linear_backward(const LinearGrad& g, int dt, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                  int K, void* dx, int64_t ldx_out, void* dw, int64_t ldw_out, float* dbias, float* drs,
                                  const uint16_t* dz, int64_t ldz, float* part, hipStream_t st) {
  return dt == ACT_BF16
             ? backward<ACT_BF16>(g, x, ldx, w, ldw, K, dx, ldx_out, dw, ldw_out, dbias, drs, dz, ldz, part, st)
             : backward<ACT_F16>(g, x, ldx, w, ldw, K, dx, ldx_out, dw, ldw_out, dbias, drs, dz, ldz, part, st);
}

}  // namespace moe
