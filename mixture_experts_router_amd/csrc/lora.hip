// Low-rank adapters of many requests beside a projection that they share:
//
//   out[t] = base[t] + scale_a * (x[t] A_a^T) B_a^T,   a = ids[t]
//
// with A_a [R, K] and B_a [N, R] of adapter a, in one launch.  Every wave of a
// workgroup reads the 64 ids of its chunk of consecutive tokens (one a lane)
// and finds the chunk's tiles with ballots: up to 16 tokens of one adapter on
// the matrix cores.  So ids come in any order, without a sorting launch, and
// runs of one request fill the tiles.
//
// Rounding: x A^T has exact products and fp32 sums, which stay in fp32.  For
// the second product v goes to the matrix cores as two 16-bit parts (hi + lo:
// 2^-18 relative for bf16, 2^-22 for fp16), three for a bf16 adapter with an
// fp32 output.  Of a 16-bit output only its own rounding shows; of an fp32 one
// the 2^-22 of fp16 adapters is less than the fp32 sums over K and the ranks
// round, and a third part would take it below 2^-24.  fp16 parts are
// taken of v * 2^-e_t, the token's largest finite |v| brought to 2^13 .. 2^14,
// which keeps fp32's range.
//
// Time, and what bounds it (K = N = 4096 unless said; a card that copies 1 GB
// at 5.1 TB/s and launches an empty kernel in 2.3 us):
//   1 token, rank 16, fp16                    7.6 us   0.3 MB: a chain of dependent
//       loads (ids, A, the sums through LDS, B and base), each 0.5 .. 1 us, and
//       some thousand instructions a wave in a row
//   64 tokens of 48 adapters, rank 32, bf16  12.3 us  12 MB (34 adapters in use):
//       the same chain with A's and B's rows in it (1.0 TB/s over the whole call).
//       They come from the Infinity Cache, which holds the three sets of inputs
//       taken in turn; over forty sets, which it does not, 14.4
//   777 tokens, N = 64, rank 8, fp32 out     10.2 us   7.6 MB: likewise
//   4096 tokens in runs of 6, rank 64, bf16  48.5 us   105 MB, 2.2 TB/s: some 20 us for
//       each product, which do not overlap (one workgroup a CU).  Neither is
//       bound by one thing: without the loads of A 38 us, of B 45, of x 46, of
//       base 45, without the stores 42.5, without base and stores 40.  Eight
//       waves hide the latencies of loads, LDS and matrix instructions only in
//       part, and sixteen do not fit the registers of 64 ranks
//   4096 tokens of 48 adapters in no order, K = N = 1024, rank 16, bf16  36.5 us, 28 MB;
//       N = 256, fp32 out 52 us (fp16 55), 49 MB; 512 tokens, rank 32, 34.7 us, 38 MB:
//       among 64 tokens an adapter has one or two, so a tile is a tenth full, and
//       A and B of most adapters are read again for each 64 tokens
//   rank 128, bf16: 1 token 25 us, 64 tokens of 48 adapters 32 .. 47 (77 MB), 4096
//       tokens in runs 82 (113 MB): eight waves take two rank tiles at a time
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int CHUNK = 64;  // tokens a workgroup looks at: one id a lane

// Loads whose place may not exist go through a descriptor's range check, which
// gives zeros: no branch, and 32-bit offsets.  FAR lies beyond every
// descriptor here (the sizes stay below 2^31 bytes) and still does with any
// offset within one added.
constexpr uint32_t FAR = 0x80000000u;

__device__ __forceinline__ u32x4 buf_load16(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
}

template <int ACT>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (ACT == ACT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// up to 16 ranks: half the columns an instruction
template <int ACT>
__device__ __forceinline__ f32x4 mfma16(u32x2 a, u32x2 b, f32x4 c) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef f16 f16x4 __attribute__((ext_vector_type(4)));
  if constexpr (ACT == ACT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, a), __builtin_bit_cast(s16x4, b), c, 0,
                                                     0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(f16x4, a), __builtin_bit_cast(f16x4, b), c, 0, 0,
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

// The tiles of a chunk: runs of up to 16 of the lanes with one id, each known
// by its first lane.  Lanes of equal ids are found bit by bit of the id.
struct Tiles {
  uint64_t same, first;  // lanes of this lane's id; the tiles' first lanes
  int at, count;         // this lane's place among them; the tiles

  __device__ __forceinline__ Tiles(int id, int L) {
    same = ~0ull;
    uint32_t key = (uint32_t)(id + 2);
#pragma unroll 1
    for (uint32_t top = (uint32_t)L + 1; top != 0; top >>= 1, key >>= 1) {
      const bool on = key & 1;
      same &= __ballot(on) ^ (on ? 0ull : ~0ull);
    }
    at = (int)__popcll(same & lanemask_lt());
    first = __ballot(id >= -1 && at % 16 == 0);
    count = (int)__popcll(first);
  }
  // the j-th tile's first lane (j < count)
  __device__ __forceinline__ int leader(int j) const {
    return (int)__builtin_ctzll(__ballot((first >> lane_id() & 1) && (int)__popcll(first & lanemask_lt()) == j));
  }
  __device__ __forceinline__ uint64_t of(int lane) const {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(same >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)same, lane);
  }
  __device__ __forceinline__ int place(int lane) const { return __builtin_amdgcn_readlane(at, lane); }
};

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

// ------------------------------------------------- base + scale v B^T ---

// two fp32 as two 16-bit values, round to nearest even (the hardware's conversions)
template <int ACT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (ACT == ACT_BF16) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
  } else {
    return __builtin_bit_cast(uint32_t, f16x2{(f16)a, (f16)b});
  }
}

// splits v (finite or not) into NP 16-bit parts, each the rounding of what
// the earlier ones leave; a number between bf16's largest and fp32's has the
// largest as its first part
template <int ACT, int NP>
__device__ __forceinline__ void split_parts(float v, uint16_t* o) {
  constexpr float MOST = 0x1.fefffep127f;  // rounds to bf16's largest
  const bool finite = fabsf(v) < INFINITY;  // inf and NaN are the first part alone
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    o[i] = (uint16_t)pack2<ACT>(ACT == ACT_BF16 && i == 0 && finite ? __builtin_amdgcn_fmed3f(v, -MOST, MOST) : v, 0.0f);
    // scaled fp16: never 0 for a number that is not, which an infinity in B would show
    if (ACT == ACT_F16 && i == 0 && v != 0.0f && (o[i] & 0x7FFFu) == 0) o[i] |= 1u;
    v = finite ? v - act_to_f32(o[i], ACT) : 0.0f;
  }
}

// order of one wave's LDS accesses (its LDS instructions execute in order)
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 4 x 4 transpose of 16-byte pieces between the four lanes of a quad and four
// registers: lane q's piece j becomes lane j's piece q.  A tile's rows are
// loaded with four consecutive lanes on 64 contiguous bytes of a row (load j:
// row 4 (lane / 4 % 4) + j), which the L1 serves more than twice as fast as
// sixteen rows a sixteen lanes (16.0 against 7.3 TB/s from L2), and this makes
// lane l hold row l % 16 as the matrix instructions want it.
// Two exchanges, of lane bit 0 with register bit 0 and of bit 1 with bit 1: each
// register is one v_cndmask whose other operand comes through a quad
// permutation (the compiler makes two instructions of it).  a, b, c, d are the
// words of v[0] .. v[3].  s_nop 1 at both ends: a DPP operand and a matrix
// instruction's may be read two wait states after the vector instruction that
// wrote them; inside, at least two instructions lie between.
__device__ __forceinline__ void quad_transpose(u32x4 (&v)[4]) {
  uint32_t a0 = v[0][0], a1 = v[0][1], a2 = v[0][2], a3 = v[0][3], b0 = v[1][0], b1 = v[1][1], b2 = v[1][2],
           b3 = v[1][3], c0 = v[2][0], c1 = v[2][1], c2 = v[2][2], c3 = v[2][3], d0 = v[3][0], d1 = v[3][1],
           d2 = v[3][2], d3 = v[3][3], t0, t1, t2, t3, u0, u1, u2, u3;
  asm("s_nop 1\n\t"
      "s_mov_b32 vcc_lo, 0x55555555\n\ts_mov_b32 vcc_hi, 0x55555555\n\t"
      "v_cndmask_b32_dpp %[t0], %[b0], %[a0], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[u0], %[d0], %[c0], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[t1], %[b1], %[a1], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[u1], %[d1], %[c1], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[t2], %[b2], %[a2], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[u2], %[d2], %[c2], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[t3], %[b3], %[a3], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[u3], %[d3], %[c3], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "s_mov_b32 vcc_lo, 0xaaaaaaaa\n\ts_mov_b32 vcc_hi, 0xaaaaaaaa\n\t"
      "v_cndmask_b32_dpp %[b0], %[a0], %[b0], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[d0], %[c0], %[d0], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[b1], %[a1], %[b1], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[d1], %[c1], %[d1], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[b2], %[a2], %[b2], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[d2], %[c2], %[d2], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[b3], %[a3], %[b3], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[d3], %[c3], %[d3], vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "s_mov_b32 vcc_lo, 0x33333333\n\ts_mov_b32 vcc_hi, 0x33333333\n\t"
      "v_cndmask_b32_dpp %[a0], %[u0], %[t0], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[a1], %[u1], %[t1], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[a2], %[u2], %[t2], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[a3], %[u3], %[t3], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "s_mov_b32 vcc_lo, 0xcccccccc\n\ts_mov_b32 vcc_hi, 0xcccccccc\n\t"
      "v_cndmask_b32_dpp %[c0], %[t0], %[u0], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[c1], %[t1], %[u1], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[c2], %[t2], %[u2], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[c3], %[t3], %[u3], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "s_mov_b32 vcc_lo, 0x33333333\n\ts_mov_b32 vcc_hi, 0x33333333\n\t"
      "v_cndmask_b32_dpp %[t0], %[d0], %[b0], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[t1], %[d1], %[b1], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[t2], %[d2], %[b2], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[t3], %[d3], %[b3], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "s_mov_b32 vcc_lo, 0xcccccccc\n\ts_mov_b32 vcc_hi, 0xcccccccc\n\t"
      "v_cndmask_b32_dpp %[d0], %[b0], %[d0], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[d1], %[b1], %[d1], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[d2], %[b2], %[d2], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %[d3], %[b3], %[d3], vcc quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "s_nop 1"
      : [a0] "+&v"(a0), [a1] "+&v"(a1), [a2] "+&v"(a2), [a3] "+&v"(a3),
        [b0] "+&v"(b0), [b1] "+&v"(b1), [b2] "+&v"(b2), [b3] "+&v"(b3),
        [c0] "+&v"(c0), [c1] "+&v"(c1), [c2] "+&v"(c2), [c3] "+&v"(c3),
        [d0] "+&v"(d0), [d1] "+&v"(d1), [d2] "+&v"(d2), [d3] "+&v"(d3),
        [t0] "=&v"(t0), [t1] "=&v"(t1), [t2] "=&v"(t2), [t3] "=&v"(t3), [u0] "=&v"(u0), [u1] "=&v"(u1), [u2] "=&v"(u2), [u3] "=&v"(u3)
      :
      : "vcc");
  v[0] = u32x4{a0, a1, a2, a3};
  v[1] = u32x4{t0, t1, t2, t3};
  v[2] = u32x4{c0, c1, c2, c3};
  v[3] = u32x4{d0, d1, d2, d3};
}

// columns c0 .. c1 - 1 of the chunk's tokens nth[p0 .. p0 + cnt): out = base, a row a wave
template <bool F32>
__device__ __forceinline__ void copy_rows(const void* base, int64_t ldb, void* out, int64_t ldo, int64_t t0, int nth,
                                          int p0, int cnt, int c0, int c1, int vec) {
  constexpr int PER = F32 ? 4 : 8;
  const int lane = lane_id();
  for (int p = wave_id(); p < cnt; p += (int)blockDim.x / WAVE) {
    const int64_t t = t0 + __builtin_amdgcn_readlane(nth, p0 + p);
    int c = c0;
    if (vec) {
      for (c += lane * PER; c + PER <= c1; c += WAVE * PER) {
        if constexpr (F32) *(u32x4*)((float*)out + t * ldo + c) = load16((const float*)base + t * ldb + c);
        else *(u32x4*)((uint16_t*)out + t * ldo + c) = load16((const uint16_t*)base + t * ldb + c);
      }
      c = c0 + max(c1 - c0, 0) / PER * PER;
    }
    for (c += lane; c < c1; c += WAVE) {
      if constexpr (F32) ((float*)out)[t * ldo + c] = ((const float*)base)[t * ldb + c];
      else ((uint16_t*)out)[t * ldo + c] = ((const uint16_t*)base)[t * ldb + c];
    }
  }
}

// the chunk's rows of a matrix of n columns of es bytes
__device__ __forceinline__ rsrc_t chunk_rows(const void* p, int es, int64_t t0, int64_t ld, int T, int n) {
  const int rows = (int)min((int64_t)CHUNK, T - t0);
  return make_rsrc((const uint8_t*)p + t0 * ld * es, (uint32_t)(((rows - 1) * ld + n) * es));
}

// what a lane holds of a rank step: eight of 32 ranks, four of 16
template <int RT>
using Piece = std::conditional_t<RT == 1, u32x2, u32x4>;

// the parts of token p's v as operands
template <int RT, int NP, int STEPS, int ROWS, int PITCH>
__device__ __forceinline__ void load_parts(const uint16_t (&vs)[NP][ROWS][PITCH], int p, Piece<RT> (&vv)[NP][STEPS]) {
  constexpr int N = sizeof(Piece<RT>) / 2;
  const int g = lane_id() / 16;
#pragma unroll
  for (int h = 0; h < NP; ++h)
#pragma unroll
    for (int q = 0; q < STEPS; ++q) vv[h][q] = *(const Piece<RT>*)&vs[h][p][(4 * q + g) * N];
}

// Columns n0 .. n0 + 31 of 16 tokens (token l16 of lane group g): D = B v^T,
// where tile u's row i is column 8 (i / 4) + 4 u + i % 4 of the 32, so a lane
// ends with eight consecutive columns of one token.  Loads and use are apart, so
// a wave has the next blocks' loads in flight.
template <int RT>
struct BRows {  // this lane's 16-byte pieces of 32 rows of B: RT of them, 32 / RT rows apart
  static constexpr int PR = 2 * RT, STEP = WAVE / PR;  // pieces a row, rows a load
  static constexpr int BP = RT * 32 + 16;  // bytes between rows in LDS: 16 consecutive rows start in different banks
  rsrc_t b;
  uint32_t from, row_bytes;
  int to;
  bool ragged;

  __device__ __forceinline__ BRows(const uint16_t* bm, int a, int N, int R, int rank) {
    const int row = lane_id() / PR, piece = lane_id() % PR;
    b = make_rsrc(bm + (int64_t)a * N * R, (uint32_t)N * R * 2);
    row_bytes = R * 2;
    from = piece * 8 < rank ? row * row_bytes + piece * 16 : FAR;
    to = row * BP + piece * 16;
    ragged = rank % 8 != 0;
  }
  // the rows of columns 32 blk ...; from b1 on zeros that read nothing (2^30
  // lies beyond B, and past FAR)
  __device__ __forceinline__ void load(u32x4 (&raw)[RT], int blk, int b1) const {
    const uint32_t off = from + (blk < b1 ? (uint32_t)(blk * 32) * row_bytes : 0x40000000u);
#pragma unroll
    for (int i = 0; i < RT; ++i) raw[i] = buf_load16(b, off + (uint32_t)(i * STEP) * row_bytes);
  }
};

// the loaded rows through LDS, from which every lane takes its own row's pieces
template <int RT, int STEPS = RT == 1 ? 1 : RT / 2>
__device__ __forceinline__ void take_rows(const u32x4 (&raw)[RT], const BRows<RT>& rows, int rank, uint8_t* lds,
                                          Piece<RT> (&bv)[STEPS][2]) {
  constexpr int N = sizeof(Piece<RT>) / 2;  // ranks a lane holds
  const int l16 = lane_id() % 16, g = lane_id() / 16;
  wave_order();  // the block before is read
#pragma unroll
  for (int i = 0; i < RT; ++i) *(u32x4*)(lds + rows.to + i * BRows<RT>::STEP * BRows<RT>::BP) = raw[i];
  wave_order();
#pragma unroll
  for (int q = 0; q < STEPS; ++q)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      bv[q][u] =
          *(const Piece<RT>*)(lds + (l16 / 4 * 8 + 4 * u + l16 % 4) * BRows<RT>::BP + (4 * q + g) * N * 2);
  if (rows.ragged) {
    // columns past the rank may hold anything (whole pieces of them are zeros)
    asm volatile("");  // a branch: these masks are not worth computing otherwise
#pragma unroll
    for (int q = 0; q < STEPS; ++q)
#pragma unroll
      for (int h = 0; h < N / 2; ++h) {
        const int r = (4 * q + g) * N + 2 * h;
        const uint32_t mask = (r < rank ? 0xFFFFu : 0u) | (r + 1 < rank ? 0xFFFF0000u : 0u);
        bv[q][0][h] &= mask;
        bv[q][1][h] &= mask;
      }
  }
}

// v B^T of the block's 32 columns: this lane's eight columns of its token.  The
// low parts go first.  With an infinity in B their sum is infinite, or NaN by a
// low part of 0, whatever v is; brought back to a number, it leaves the result
// to the first part, which has v's sign and is 0 only where v is.
template <int ACT, int RT, int NP, int STEPS = RT == 1 ? 1 : RT / 2>
__device__ __forceinline__ void block_product(const Piece<RT> (&bv)[STEPS][2], const Piece<RT> (&vv)[NP][STEPS], int e,
                                              float (&d)[8]) {
  f32x4 acc[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
  for (int h = NP - 1; h >= 0; --h) {
#pragma unroll
    for (int q = 0; q < STEPS; ++q)
#pragma unroll
      for (int u = 0; u < 2; ++u) acc[u] = mfma16<ACT>(bv[q][u], vv[h][q], acc[u]);
    if (h == 1) {
      // one scalar, with its sign and without: two constants would hold a vector
      // register too, over the whole kernel (64 tokens of 48 adapters: 12.6 against 12.3 us)
      float most = __FLT_MAX__;
      asm("" : "+s"(most));
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j / 4][j % 4] = __builtin_amdgcn_fmed3f(acc[j / 4][j % 4], -most, most);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) d[j] = ACT == ACT_F16 ? ldexp_f(acc[j / 4][j % 4], e) : acc[j / 4][j % 4];
}

// out = base + d for eight whole columns.  Non-temporal: in a long batch the
// written rows otherwise push out the ones still to be read (4096 tokens, 4096
// columns, rank 64: 51 against 67 us; rank 16: 34 against 46).
template <int ACT, bool F32>
__device__ __forceinline__ void add_store(const u32x4 (&o)[F32 ? 2 : 1], const float (&d)[8], void* out, int64_t io) {
  if constexpr (F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 y = __builtin_bit_cast(f32x4, o[h]);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = y[j] + d[4 * h + j];
      __builtin_nontemporal_store(y, (f32x4*)((float*)out + io + 4 * h));
    }
  } else {
    u32x4 y;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      y[j] = pack2<ACT>(act_to_f32(o[0][j] & 0xFFFFu, ACT) + d[2 * j], act_to_f32(o[0][j] >> 16, ACT) + d[2 * j + 1]);
    __builtin_nontemporal_store(y, (u32x4*)((uint16_t*)out + io));
  }
}

// ----------------------------------------------------------- the kernel --
//
// Both products of a tile (up to 16 tokens of one adapter) in one workgroup
// of eight or sixteen waves: the waves take consecutive parts of K and are added through
// LDS in wave order, the tokens' sums are split into the parts the matrix
// cores take, and the waves share the output's columns.
//
// The chunk's work comes in units of one tile and one of 2^cut parts of the
// columns (the first product is repeated for each part), which its gridDim.y
// workgroups take in turn.  `cut` grows while the chunk's units fit its share
// of the CUs side by side, so a few tiles still fill the chip: the
// number of tiles is known only here, from the ids.  Against parts chosen by T
// alone: 1024 tokens in runs, rank 64, 22.0 against 27.3 us; 300 tokens, rank
// 16, 12.5 against 17.8; 64 tokens of 48 adapters, rank 32, 13.0 against 14.4; 8
// tokens, rank 64, 15.9 against 14.8.  The result does not depend on it.

// Waves by the ranks: sixteen of 128 registers where their operands fit, up to
// 32 ranks (against eight: 64 tokens of 48 adapters, rank 32, 12.3 and 13.1 us; 4096
// tokens of 48 adapters, K = N = 1024, rank 16, 38 and 50; one token, rank 16, 7.8 and
// 8.1; the same within 0.3 us for runs of one adapter), eight above (rank 64, 4096
// tokens: 48.5 us, 62 with sixteen).
template <int RT>
constexpr int WAVES = RT <= 2 ? 16 : 8;
constexpr int MOST_CUT = 3;  // at most 2^3 parts of the columns

template <int ACT, bool F32, int RT>
__global__ __launch_bounds__(64 * WAVES<RT>) void lora_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                       const uint16_t* __restrict__ am,
                                                       const uint16_t* __restrict__ bm,
                                                       const float* __restrict__ scale,
                                                       const int32_t* __restrict__ ids,
                                                       const int32_t* __restrict__ ranks, const void* base,
                                                       int64_t ldb, void* out, int64_t ldo, int T, int L, int R, int K,
                                                       int N, int vec, int share, int most) {
  constexpr int FW = WAVES<RT>, NP = F32 && ACT == ACT_BF16 ? 3 : 2;
  constexpr int STEPS = RT == 1 ? 1 : RT / 2;  // 32-rank steps of the second product
  constexpr int RP = RT * 16, TILE = 16;
  constexpr int RB = RT < 4 ? RT : RT == 8 ? 2 : 4;  // rank tiles loaded, and summed over the waves, together
  constexpr int H = RT / RB;
  // Loads in flight a wave: items of the first product, and of the second
  // base's blocks (from HBM) and B's (from L2).  With sixteen waves one of each;
  // two items spill (one token: 9.9 against 7.8 us).  RT = 4: two items spill, two
  // of base's blocks give 51 us for 4096 tokens against 48.7, and four of B's 50.4.
  constexpr int DEEP = RT <= 4 ? 1 : 2;
  constexpr int TURN = DEEP < H ? H : DEEP;
  constexpr int AHEAD = RT <= 2 ? 1 : F32 ? 2 : 4, BAHEAD = RT == 4 ? 2 : 1;
  constexpr int OV = F32 ? 2 : 1;
  constexpr int VR = (RP + WAVE - 1) / WAVE;
  union Shared {
    f32x4 red[FW][RB][WAVE];
    uint8_t b[FW][32 * BRows<RT>::BP];
  };
  __shared__ __attribute__((aligned(16))) Shared sh;
  __shared__ float vsum[TILE][RP + 4];
  __shared__ __attribute__((aligned(16))) uint16_t vs[NP][TILE][RP + 8];
  __shared__ int exps[TILE];
  const int lane = lane_id(), wave = wave_id();
  const int l16 = lane % 16, g = lane / 16;
  const int64_t t0 = (int64_t)blockIdx.x * CHUNK;
  const int id = chunk_id(ids, t0, T, L);
  const int kb = (K + 127) / 128, k0 = kb * wave / FW, k1 = kb * (wave + 1) / FW;
  const int nb = (N + 31) / 32;
  const rsrc_t rx = chunk_rows(x, 2, t0, ldx, T, K);
  const rsrc_t rb = chunk_rows(base, F32 ? 4 : 2, t0, ldb, T, N);
  const Tiles tiles(id, L);
  int cut = 0;  // the output's columns in 2^cut parts
  while (tiles.count << (cut + 1) <= share && cut < most) ++cut;
  const int per = (nb + (1 << cut) - 1) >> cut;
  for (int unit = blockIdx.y; unit < tiles.count << cut; unit += gridDim.y) {
    const int z = unit & ((1 << cut) - 1), tile = unit >> cut;
    const int b0 = min(nb, z * per), b1 = min(nb, b0 + per);
    const int first = tiles.leader(tile);
    const int a = __builtin_amdgcn_readlane(id, first);
    const uint64_t mine = tiles.of(first);
    const int p0 = tiles.place(first), cnt = min(TILE, (int)__popcll(mine) - p0);
    const int nth = nth_lane(mine);
    if (a < 0) {
      // no adapter: out is base, moved only if the two are not one buffer
      if (out != base) copy_rows<F32>(base, ldb, out, ldo, t0, nth, p0, cnt, b0 * 32, min(N, b1 * 32), vec);
      continue;
    }
    const int rank = adapter_rank(ranks, a, R);
    // sizes the compiler must not know from here on: it would keep every
    // product of them in registers over the loop, and spill
    asm volatile("" : "+s"(K), "+s"(N), "+s"(R));

    // ---- x A^T over this wave's columns.  A: load j is this lane's piece of
    // row lrow + j of a 16-row tile, eight columns from lcol of a 128-column
    // block, and the quad transpose makes it columns 32 g + 8 j of row l16.
    // x, read once, comes in that place.
    const bool have = l16 < cnt;
    const int tok = __builtin_amdgcn_ds_bpermute((p0 + (have ? l16 : 0)) << 2, nth);
    const int64_t t = t0 + tok;
    const uint32_t xoff = have ? (uint32_t)tok * (uint32_t)ldx * 2 + g * 64 : FAR;
    const uint32_t at = have && vec ? (uint32_t)tok * (uint32_t)ldb * (F32 ? 4 : 2) + g * (F32 ? 32 : 16) : FAR;
    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const rsrc_t ra = make_rsrc(am + (int64_t)a * R * K, (uint32_t)rank * K * 2);  // rows up to the rank
    const int lrow = lane / 4 % 4 * 4, lcol = g * 32 + lane % 4 * 8;
    const uint32_t aoff = (uint32_t)(lrow * K + lcol) * 2;
    struct Item {
      u32x4 x[4], a[RB][4];
    } it[DEEP];
    const int items = (k1 - k0) * H;
    auto load_x = [&](u32x4 (&v)[4], int i) __attribute__((always_inline)) {
      const int c = (k0 + i / H) * 128;
      const int end = i < items ? K : 0;  // past the last item: zeros, unread
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = buf_load16(rx, c + g * 32 + 8 * j < end ? xoff + (c + 8 * j) * 2 : FAR);
    };
    auto load_a = [&](u32x4 (&v)[4], int i, int r) __attribute__((always_inline)) {  // rank tile r
      const int c = (k0 + i / H) * 128;
      const uint32_t off = c + lcol < (i < items ? K : 0) ? aoff + c * 2 : FAR;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = buf_load16(ra, off + (uint32_t)((r * 16 + j) * K) * 2);
    };
    u32x4 xn[4];
#pragma unroll
    for (int h = 0; h < DEEP; ++h) {
      load_x(it[h].x, h);
#pragma unroll
      for (int r = 0; r < RB; ++r) load_a(it[h].a[r], h, h % H * RB + r);
    }
#pragma unroll 1
    for (int i = 0; i < items; i += TURN) {
#pragma unroll
      for (int h = 0; h < TURN; ++h) {
        Item& now = it[h % DEEP];
        if (DEEP == 1) load_x(xn, i + h + 1);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          quad_transpose(now.a[r]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[h % H * RB + r] = mfma16<ACT>(now.a[r][j], now.x[j], acc[h % H * RB + r]);
          if (DEEP > 1 && r == RB - 1) load_x(now.x, i + h + DEEP);
          load_a(now.a[r], i + h + DEEP, (h + DEEP) % H * RB + r);
        }
        if (DEEP == 1) {
#pragma unroll
          for (int j = 0; j < 4; ++j) now.x[j] = xn[j];
        }
      }
    }

    // ---- the second product's first loads, which do not wait for the sums
    const BRows<RT> rows(bm, a, N, R, rank);
    u32x4 braw[BAHEAD][RT], o[AHEAD][OV];
    auto load_o = [&](u32x4 (&v)[OV], int blk) __attribute__((always_inline)) {
      const uint32_t off = blk < b1 && blk * 32 + 8 * g + 8 <= N ? at + (uint32_t)(blk * 32) * (F32 ? 4 : 2) : FAR;
#pragma unroll
      for (int h = 0; h < OV; ++h) v[h] = buf_load16(rb, off + 16 * h);
    };
#pragma unroll
    for (int h = 0; h < BAHEAD; ++h) rows.load(braw[h], b0 + wave + FW * h, b1);
#pragma unroll
    for (int h = 0; h < AHEAD; ++h) load_o(o[h], b0 + wave + FW * h);

    // ---- the waves' sums, token by token as 16-bit parts
#pragma unroll
    for (int r0 = 0; r0 < RT; r0 += RB) {
      __syncthreads();  // the last tile's B rows, or the sums before these, are read
#pragma unroll
      for (int r = 0; r < RB; ++r) sh.red[wave][r][lane] = acc[r0 + r];
      __syncthreads();
      for (int i = threadIdx.x; i < RB * 256; i += 64 * FW) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < FW; ++w) v += ((const float*)sh.red[w])[i];
        vsum[i / 4 % 16][(r0 + i / 256) * 16 + i % 256 / 64 * 4 + i % 4] = v;
      }
    }
    __syncthreads();
    const float sc = scale ? scale[a] : 1.0f;
    for (int p = wave; p < TILE; p += FW) {
      float v[VR], top = 0.0f;
#pragma unroll
      for (int q = 0; q < VR; ++q) {
        const int r = lane + WAVE * q;
        v[q] = r < rank ? vsum[p][r] * sc : 0.0f;  // past the rank zero, also where x is not finite
        const float size = fabsf(v[q]);
        top = fmaxf(top, size < INFINITY ? size : 0.0f);  // an infinite or NaN rank leaves the others their scale
      }
      int e = 0;
      if constexpr (ACT == ACT_F16) {
        top = wave_max(top);
        if (top > 0.0f) e = __builtin_amdgcn_frexp_expf(top) - 14;
        if (lane == 0) exps[p] = e;
      }
#pragma unroll
      for (int q = 0; q < VR; ++q) {
        const int r = lane + WAVE * q;
        uint16_t parts[NP];
        split_parts<ACT, NP>(ACT == ACT_F16 ? ldexp_f(v[q], -e) : v[q], parts);
        if (r < RP) {
#pragma unroll
          for (int h = 0; h < NP; ++h) vs[h][p][r] = parts[h];
        }
      }
    }
    __syncthreads();

    // ---- base + v B^T: this wave's every FW-th block of 32 columns
    Piece<RT> vv[NP][STEPS];
    load_parts<RT>(vs, l16, vv);
    const int e = ACT == ACT_F16 ? exps[l16] : 0;
    const int whole = vec ? min(b1, N / 32) : b0;  // blocks of 32 columns that can be moved in 16 bytes
    int b = b0 + wave;
#pragma unroll 1
    for (; b < whole; b += FW * AHEAD) {
#pragma unroll
      for (int h = 0; h < AHEAD; ++h) {
        const int now = b + FW * h;
        if (now < whole) {
          Piece<RT> bv[STEPS][2];
          take_rows<RT>(braw[h % BAHEAD], rows, rank, sh.b[wave], bv);
          rows.load(braw[h % BAHEAD], now + FW * BAHEAD, b1);
          float d[8];
          block_product<ACT, RT, NP>(bv, vv, e, d);
          if (have) add_store<ACT, F32>(o[h], d, out, t * ldo + now * 32 + 8 * g);
          load_o(o[h], now + FW * AHEAD);
        }
      }
    }
    // the others, element by element
    b = b0 + wave + (max(whole - b0 - wave, 0) + FW - 1) / FW * FW;
#pragma unroll 1
    for (; b < b1; b += FW) {
      Piece<RT> bv[STEPS][2];
      rows.load(braw[0], b, b1);
      take_rows<RT>(braw[0], rows, rank, sh.b[wave], bv);
      float d[8];
      block_product<ACT, RT, NP>(bv, vv, e, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = b * 32 + 8 * g + j;
        if (have && c < N) {
          if constexpr (F32)
            ((float*)out)[t * ldo + c] = ((const float*)base)[t * ldb + c] + d[j];
          else
            ((uint16_t*)out)[t * ldo + c] =
                (uint16_t)pack2<ACT>(act_to_f32(((const uint16_t*)base)[t * ldb + c], ACT) + d[j], 0.0f);
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_lora(const void* x, int act, int64_t ldx, int T, const LoraDev& ad, const int32_t* ids,
                       const void* base, int64_t ldb, void* out, int64_t ldo, bool out_f32, int num_cu,
                       hipStream_t st) {
  const int per = out_f32 ? 4 : 8;  // elements of 16 bytes
  const int vec = ldb % per == 0 && ldo % per == 0 &&
                  ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const int chunks = (int)(((int64_t)T + CHUNK - 1) / CHUNK);
  // A CU holds one workgroup: a chunk's share of the CUs (twice as many: 51.7
  // against 48.8 us for 4096 tokens, 20.5 against 14.0 for 64 tokens of 48 adapters).
  // At most eight parts, each of eight blocks of 32 columns or more (one token,
  // rank 16: 8 us in eight parts, 12.7 in one; sixteen: no faster).
  const int share = std::max(1, num_cu / chunks);
  int most = 0;
  while (most < MOST_CUT && 16 << most <= (ad.N + 31) / 32) ++most;
  const int W = std::min(std::min(T, CHUNK) << most, share);
  const dim3 grid(chunks, W);
  auto go = [&](auto kern, int threads) {
    return launch_kernel(kern, grid, threads, 0, st, (const uint16_t*)x, ldx, (const uint16_t*)ad.a,
                         (const uint16_t*)ad.b, ad.scale, ids, ad.ranks, base, ldb, out, ldo, T, ad.L, ad.R, ad.K, ad.N,
                         vec, share, most);
  };
  auto rank = [&](auto ac, auto fc) {
    constexpr int A = decltype(ac)::value;
    constexpr bool F = decltype(fc)::value;
    return ad.R <= 16   ? go(lora_kernel<A, F, 1>, 64 * WAVES<1>)
           : ad.R <= 32 ? go(lora_kernel<A, F, 2>, 64 * WAVES<2>)
           : ad.R <= 64 ? go(lora_kernel<A, F, 4>, 64 * WAVES<4>)
                        : go(lora_kernel<A, F, 8>, 64 * WAVES<8>);
  };
  auto type = [&](auto ac) { return out_f32 ? rank(ac, std::true_type{}) : rank(ac, std::false_type{}); };
  return act == ACT_BF16 ? type(std::integral_constant<int, ACT_BF16>{}) : type(std::integral_constant<int, ACT_F16>{});
}

}  // namespace moe
