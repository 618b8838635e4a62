// Device helpers and launch interfaces shared by the packed products for many
// tokens (packed_linear.hip, packed_backward.hip) and the low-rank adapters
// beside them (adapter.hip).
#pragma once
#include "common.hpp"

namespace gptq {

// 16-bit element types: 1 bf16, 2 fp16 (the values of gptq_dtype).
constexpr int kBF16 = 1, kF16 = 2;

// Low-rank adapters of several requests: A [m][rank][d_in], B [m][d_out][rank],
// both dense and of the activations' 16-bit type; token t uses adapter
// index[t] (index null: 0), none when that lies outside 0 .. m-1.
struct Adapters {
  const uint16_t* A;
  const uint16_t* B;
  const float* alpha;     // null: 1
  const int32_t* index;   // null: adapter 0 for every token
  int m, rank;
  const int32_t* order;   // null, or all tokens in the order of their adapters

  // Token at a place of a tile; the places past the last token have none (-1).
  GPTQ_DEV int64_t token(int64_t place, int64_t n) const { return place >= n ? -1 : (order ? (int64_t)order[place] : place); }
};

// A packed layer as gptq_pack / gptq_quantize_layer write it.
struct PackedLayer {
  const uint32_t* words;
  int64_t ldw;
  const float* scales;
  const int32_t* zeros;
  int64_t ldg;
  const int32_t* perm;    // null: packed column j is input j
  int bits;
  int r, c;
  int cpg;                // 32-column chunks per group (all of them: one ruler per row)
  int shift;              // log2 of cpg, 31 for one group, -1 where it is neither

  // Group of a chunk (a division by a variable is some twenty instructions).
  GPTQ_DEV int group(int chunk) const { return shift >= 0 ? chunk >> shift : chunk / cpg; }
};

// ---------------------------------------------------------------- 16-bit values
template <int DT>
GPTQ_DEV float f16_to_f32(uint32_t bits) {
  if constexpr (DT == kBF16) return __uint_as_float(bits << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// Round to nearest even; bf16 keeps NaN.
template <int DT>
GPTQ_DEV uint16_t f32_to_16(float v) {
  if constexpr (DT == kBF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return __builtin_bit_cast(uint16_t, (_Float16)v);
}

template <int DT>
GPTQ_DEV uint32_t pack2(float lo, float hi) {
  return (uint32_t)f32_to_16<DT>(lo) | ((uint32_t)f32_to_16<DT>(hi) << 16);
}

// One output value to a matrix of type yt (0 fp32, 1 bf16, 2 fp16).
template <int YT>
GPTQ_DEV void store_out(void* Y, int64_t at, float v) {
  if constexpr (YT == 0) static_cast<float*>(Y)[at] = v;
  else static_cast<uint16_t*>(Y)[at] = f32_to_16<YT>(v);
}

// Eight consecutive 16-bit values of which the first `valid` exist (the rest
// read as 0).  vec: the address is 16-byte aligned.
GPTQ_DEV u32x4 load8(const uint16_t* p, int valid, bool vec) {
  if (vec && valid >= 8) return *reinterpret_cast<const u32x4*>(p);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < valid) v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
  return v;
}

// 16 x 16 x 32 matrix product: lane l holds A[l & 15][8 (l >> 4) + e] and
// B[8 (l >> 4) + e][l & 15], and C[4 (l >> 4) + i][l & 15] in component i.
template <int DT>
GPTQ_DEV floatx4 mfma16(u32x4 a, u32x4 b, floatx4 c) {
  if constexpr (DT == kBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// 32 x 32 x 16: lane l holds A[l & 31][8 (l >> 5) + e] and B[8 (l >> 5) + e][l & 31],
// and C[8 (i >> 2) + 4 (l >> 5) + (i & 3)][l & 31] in component i.
template <int DT>
GPTQ_DEV floatx16 mfma32(u32x4 a, u32x4 b, floatx16 c) {
  if constexpr (DT == kBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Tile shapes of the two: E x E outputs, K of the contraction, the lane's
// position in an operand (row l % E, K offset 8 (l / E)) and the row of
// accumulator component i.
template <class Acc>
struct TileShape;
template <>
struct TileShape<floatx4> {
  static constexpr int E = 16, K = 32, C = 4;
  static GPTQ_DEV int acc_row(int lane, int i) { return 4 * (lane >> 4) + i; }
};
template <>
struct TileShape<floatx16> {
  static constexpr int E = 32, K = 16, C = 16;
  static GPTQ_DEV int acc_row(int lane, int i) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }
};

// ---------------------------------------------------------------- adapters
// Adapter of token t, or -1.
GPTQ_DEV int adapter_of(const Adapters& ad, int64_t t, int64_t n) {
  if (t < 0 || t >= n) return -1;
  const int a = ad.index ? ad.index[t] : 0;
  return (uint32_t)a < (uint32_t)ad.m ? a : -1;
}

// An fp32 operand of a bf16 matrix product as TERMS of them, v = v1 + v2 (+ v3):
// each term holds 8 more significant bits, so the rest is below 2^-17 |v| with
// two terms and 2^-25 |v| with three.
template <int TERMS>
GPTQ_DEV void split8(const float (&v)[8], u32x4 (&t)[TERMS]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
  for (int k = 0; k < TERMS; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = pack2<kBF16>(r[2 * i], r[2 * i + 1]);
      t[k][i] = w;
      r[2 * i] -= __uint_as_float(w << 16);
      r[2 * i + 1] -= __uint_as_float(w & 0xFFFF0000u);
    }
}

// A 16-bit operand in bf16: itself, or two terms for fp16 (exact: 11
// significant bits against 8 + 8).
template <int DT>
struct Terms16 {
  static constexpr int N = DT == kBF16 ? 1 : 2;
  u32x4 t[N];
  GPTQ_DEV explicit Terms16(u32x4 v) {
    if constexpr (DT == kBF16) {
      t[0] = v;
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = f16_to_f32<kF16>(v[i] & 0xFFFFu);
        f[2 * i + 1] = f16_to_f32<kF16>(v[i] >> 16);
      }
      split8<2>(f, t);
    }
  }
};

// c + V Z of an fp32 operand in TERMS terms and a 16-bit one, smallest products
// first.  The product of both last terms is left out: 2^-16 of two terms (16-bit
// results), 2^-25 of three, with fp16 Z; with bf16 Z, which is one term, nothing is.
template <int DT, int TERMS>
GPTQ_DEV floatx4 mfma_terms(const u32x4 (&v)[TERMS], const Terms16<DT>& z, floatx4 c) {
  if constexpr (TERMS == 3) {
    c = mfma16<kBF16>(v[2], z.t[0], c);
    if constexpr (DT == kF16) c = mfma16<kBF16>(v[1], z.t[1], c);
  }
  c = mfma16<kBF16>(v[1], z.t[0], c);
  if constexpr (DT == kF16) c = mfma16<kBF16>(v[0], z.t[1], c);
  return mfma16<kBF16>(v[0], z.t[0], c);
}
template <int DT, int TERMS>
GPTQ_DEV floatx16 mfma_terms(const u32x4 (&v)[TERMS], const Terms16<DT>& z, floatx16 c) {
  if constexpr (TERMS == 3) {
    c = mfma32<kBF16>(v[2], z.t[0], c);
    if constexpr (DT == kF16) c = mfma32<kBF16>(v[1], z.t[1], c);
  }
  c = mfma32<kBF16>(v[1], z.t[0], c);
  if constexpr (DT == kF16) c = mfma32<kBF16>(v[0], z.t[1], c);
  return mfma32<kBF16>(v[0], z.t[0], c);
}

// Eight fp32 values (16-byte aligned).
GPTQ_DEV void load8f(const float* p, float (&v)[8]) {
  const floatx4 a = *reinterpret_cast<const floatx4*>(p), b = *reinterpret_cast<const floatx4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

// sum_p S[p] b[p] of one output: its row b of 16-bit values.
template <int DT>
GPTQ_DEV float rank_dot(const float* S, const uint16_t* b, int rank) {
  float sum = 0.f;
  for (int p = 0; p < rank; p += 8) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(b + p);
    float v[8];
    load8f(S + p, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum = __builtin_fmaf(v[2 * e], f16_to_f32<DT>(w[e] & 0xFFFFu), sum);
      sum = __builtin_fmaf(v[2 * e + 1], f16_to_f32<DT>(w[e] >> 16), sum);
    }
  }
  return sum;
}

// out[q] += S B_a^T of one adapter's tokens among the Tile::E of a tile (accumulator
// layout, row = place): a product over all of them, of which only the members'
// rows are kept.  It goes on from out, so that a token's sum does not depend on
// whether it shares its tile.  t: the token of the lane's place, or -1.
template <int DT, int TERMS, int NT, class Acc>
GPTQ_DEV void expand_shared(const Adapters& ad, int a, uint32_t members, const uint16_t* B, int64_t rows, const float* S, int64_t t,
                            const int64_t (&row)[NT], Acc (&out)[NT]) {
  using Tile = TileShape<Acc>;
  const int lane = threadIdx.x & 63, kq = lane / Tile::E;
  Acc acc[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) acc[q] = out[q];
  for (int k0 = 0; k0 < ad.rank; k0 += Tile::K) {
    const int k = k0 + 8 * kq;
    float v[8] = {};
    if (k < ad.rank && t >= 0) load8f(S + t * ad.rank + k, v);
    u32x4 s[TERMS];
    split8<TERMS>(v, s);
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      u32x4 b = {0u, 0u, 0u, 0u};
      if (k < ad.rank && row[q] >= 0)
        b = *reinterpret_cast<const u32x4*>(B + ((int64_t)a * rows + row[q]) * ad.rank + k);
      acc[q] = mfma_terms<DT, TERMS>(s, Terms16<DT>(b), acc[q]);
    }
  }
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int i = 0; i < Tile::C; ++i)
      out[q][i] = (members >> Tile::acc_row(lane, i)) & 1 ? acc[q][i] : out[q][i];
}

// out[q] += (S B_a^T) of the tokens at places t0 .. and NT sets of a tile's outputs, in
// the accumulator layout (row = place): the low-rank product beside a tile.
// S [n][rank] fp32 already holds alpha; row[q] is this lane's output row
// (column of the tile) in B [m][rows][rank], or -1.  The adapters that occur
// among the tokens are taken one after the other, each as a product over all of
// them, of which only its own tokens' rows are kept: a value that is not finite
// in one request's adapter or tokens stays in that request's rows.  Places in the
// order of adapters leave one or two of them to a tile.
// fp32 results take S in three terms, 16-bit ones in two.
template <int DT, int TERMS, int NT, class Acc>
GPTQ_DEV void expand_add(const Adapters& ad, const uint16_t* B, int64_t rows, const float* S, int64_t t0, int64_t n,
                         const int64_t (&row)[NT], Acc (&out)[NT]) {
  using Tile = TileShape<Acc>;
  const int64_t t = ad.token(t0 + (threadIdx.x & 63) % Tile::E, n);
  const int mine = adapter_of(ad, t, n);
  uint32_t rest = (uint32_t)(__ballot(mine >= 0) & ((1ull << Tile::E) - 1));
  while (rest) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(rest));
    const uint32_t members = (uint32_t)(__ballot(mine == a) & ((1ull << Tile::E) - 1));
    rest &= ~members;
    expand_shared<DT, TERMS, NT>(ad, a, members, B, rows, S, t, row, out);
  }
}

// The first k of eight outputs from `at`.  vec: eight start on 16 bytes there.
template <int OT>
GPTQ_DEV void store8(void* out, int64_t at, const float (&v)[8], int k, bool vec) {
  if (vec && k == 8) {
    if constexpr (OT == 0) {
      float* o = static_cast<float*>(out) + at;
      *reinterpret_cast<floatx4*>(o) = floatx4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<floatx4*>(o + 4) = floatx4{v[4], v[5], v[6], v[7]};
    } else {
      const u32x4 o = {pack2<OT>(v[0], v[1]), pack2<OT>(v[2], v[3]), pack2<OT>(v[4], v[5]), pack2<OT>(v[6], v[7])};
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + at) = o;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < k) store_out<OT>(out, at + e, v[e]);
  }
}

// ---------------------------------------------------------------- tile results
// A wave's 32 x 32 NT accumulators into its own 32 x (32 NT + 4) floats of LDS, rows
// of places.
template <int NT>
GPTQ_DEV void turn_tile(float* lds, const floatx16 (&acc)[NT]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int e = 0; e < 16; ++e) lds[TileShape<floatx16>::acc_row(lane, e) * (32 * NT + 4) + 32 * q + (lane & 31)] = acc[q][e];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Stores the 32 tokens at places t0 .. x 32 NT outputs of a wave (accumulators of
// mfma32) to out, turned through LDS so that a row leaves in whole runs of eight
// outputs per lane (single stores of two bytes took a tenth of a 256 x 256
// tile's time at 4096 columns).  vec: rows of out start on 16 bytes.
template <int OT, int NT>
GPTQ_DEV void store_tile(float* lds, const floatx16 (&acc)[NT], const Adapters& ad, void* out, int64_t t0, int64_t n, int64_t j0,
                         int64_t cols, int64_t ldo, bool vec) {
  constexpr int W = 32 * NT, RUNS = W / 8;   // of a row
  const int lane = threadIdx.x & 63;
  turn_tile<NT>(lds, acc);
#pragma unroll
  for (int k = 0; k < RUNS / 2; ++k) {
    const int run = 64 * k + lane, r = run / RUNS, c = 8 * (run % RUNS);
    const int64_t t = ad.token(t0 + r, n), j = j0 + c;
    if (t < 0 || j >= cols) continue;
    float v[8];
    load8f(lds + r * (W + 4) + c, v);
    store8<OT>(out, t * ldo + j, v, (int)min((int64_t)8, cols - j), vec);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Whether rows of a result of type ot (0 fp32) start on 16 bytes.
inline bool rows_on_16(const void* p, int64_t ld, int ot) {
  const int64_t e = ot == 0 ? 4 : 2;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * e % 16 == 0;
}

// ---------------------------------------------------------------- tile order
// Tile of workgroup b.  Panels of 8 token tiles are walked row tile by row
// tile; the dispatcher deals workgroups round robin to the 8 XCDs, so within
// 256 workgroups XCD x is given 32 consecutive places of that walk: 8 token
// tiles x 4 row tiles, whose activations and words its L2 shares.
GPTQ_DEV void tile_of(int64_t b, int tok_tiles, int row_tiles, int& tok, int& row) {
  const int64_t all = (int64_t)tok_tiles * row_tiles;
  if (b < (all & ~(int64_t)255)) b = (b & ~(int64_t)255) | ((b & 7) << 5) | ((b & 255) >> 3);
  const int64_t per = (int64_t)8 * row_tiles;
  const int panel = (int)(b / per), in = (int)(b - panel * per);
  const int h = min(8, tok_tiles - 8 * panel);
  row = in / h;
  tok = 8 * panel + in - row * h;
}

// ---------------------------------------------------------------- packed words
// Eight consecutive codes of a row as one 32-bit block: the word itself (4
// bits), or bits 24m .. 24m+23 of a chunk's 96 (3 bits).
template <int BITS>
GPTQ_DEV uint32_t code_block(const uint32_t* chunk, int m) {
  if constexpr (BITS == 4) return chunk[m];
  const int bit = 24 * m, w = bit >> 5;
  return (__builtin_amdgcn_alignbit(chunk[w < 2 ? w + 1 : 2], chunk[w], bit & 31)) & 0xFFFFFFu;
}

// Block b of a 3-bit row (its bits 24 .. 31 are not the block's).
GPTQ_DEV uint32_t straddling_block(const uint32_t* words, int b) {
  const uint32_t* c = words + 3 * (int64_t)(b >> 2);
  const int bit = 24 * (b & 3), at = bit >> 5;
  return __builtin_amdgcn_alignbit(c[at < 2 ? at + 1 : 2], c[at], bit & 31);
}

// A weight in fp32, as quantize_layer's w_hat holds it, to be rounded to type DT.  The
// product is kept apart from that rounding: in one instruction with it, fp16 values
// come out rounded once from the exact product, and 2 in 100000 differ from the
// rounded w_hat.
template <int DT>
GPTQ_DEV float weight32(uint32_t code, float zero, float scale) {
  float w = ((float)code - zero) * scale;
  if constexpr (DT == kF16) asm("" : "+v"(w));
  return w;
}

// 32 consecutive codes of a row.
template <int BITS>
struct Chunk {
  uint32_t w[BITS];
};

template <int BITS>
GPTQ_DEV Chunk<BITS> load_chunk(const uint32_t* words, int ch) {
  Chunk<BITS> c;
  const uint32_t* p = words + (int64_t)BITS * ch;
  if constexpr (BITS == 4) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) c.w[i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) c.w[i] = p[i];
  }
  return c;
}

// Codes t and t + 4 of a block of eight, t = 0 .. 3, as pairs of 16-bit floats
// 2^BITS + q.
// exponent: code_exponent() in a vector register, so that mask and exponent are
// one instruction (its other constant, the mask, takes the one scalar operand).
template <int BITS, int DT>
GPTQ_DEV uint32_t code_exponent() {
  uint32_t v = (DT == kBF16 ? 0x3F80u + (BITS << 7) : 0x3C00u + (BITS << 10)) * 0x10001u;
  asm volatile("" : "+v"(v));
  return v;
}
template <int BITS, int DT>
GPTQ_DEV u32x4 code_pairs(uint32_t blk, uint32_t exponent) {
  constexpr int P = (DT == kBF16 ? 7 : 10) - BITS;   // lowest bit of the code in the mantissa
  constexpr uint32_t mask = (((1u << BITS) - 1) << P) * 0x10001u;
  if constexpr (BITS == 3) blk = (blk & 0xFFFu) | ((blk & 0xFFF000u) << 4);   // codes 4 .. 7 to the high half
  u32x4 v;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    constexpr int B = BITS;
    const int sh = P - B * t;
    v[t] = ((sh >= 0 ? blk << sh : blk >> -sh) & mask) | exponent;
  }
  return v;
}

// Eight consecutive activations in the order of code_pairs.
GPTQ_DEV u32x4 pair_order(u32x4 v) {
  u32x4 p;
  p[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
  p[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
  p[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
  p[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
  return p;
}

// ---------------------------------------------------------------- launches
// xt / dt: 1 bf16, 2 fp16; yt: 0 fp32, 1 bf16, 2 fp16.

// Whether the dispatcher takes a grid: its threads are counted in 32 bits.  Each
// file's *_fits below says so of its launches at a call's sizes, for the host's
// checks before any of them is enqueued.
inline bool grid_fits(int64_t groups, int64_t threads) { return groups <= 0xFFFFFFFFll / threads; }

// S[t][p] = alpha sum_k X[t][k] A_a[p][k]: X [n][ldx] (d columns), A [m][rank][lda]
// on 16 bytes, lda a multiple of 8 and zero past d.  S: n x rank results in
// adapter_down_floats() of workspace, in which the parts of a split contraction
// follow the results.  Up to two such problems in one launch (p[1].X null: one);
// X as adapter_rows_direct says.  join: the one problem's parts are joined (else
// the reader joins them).  Returns the parts of p[0], 1 once joined.
inline __host__ __device__ int64_t down_values(int64_t n, int64_t rank) { return (n * rank + 63) / 64 * 64; }
struct DownProblem {
  const uint16_t* X;
  int64_t d, ldx;
  const uint16_t* A;
  int64_t lda;
  float* S;
  bool vec;        // set by the launch, as splits
  int splits;
};
struct DownArgs {
  Adapters ad;
  int64_t n;
  DownProblem p[2];
  int64_t blocks0; // set by the launch
};
int64_t adapter_down_floats(int64_t n, int64_t d, int64_t rank);
bool adapter_down_fits(int64_t n, int m, int64_t rank, int problems);
int launch_adapter_down(const DownArgs& g, int xt, bool join, hipStream_t s);
// The parts that a launch leaves of a problem.
int adapter_down_parts(int64_t n, int m, int64_t d);
// Whether rows can be a down problem's X as they are (else padded, see below).
bool adapter_rows_direct(const void* X, int64_t n, int64_t d, int64_t ldx, int m);

// What is laid out before the products, each piece where its pointer is set:
// order: all n tokens by adapter (adapters_want_order);
// list: tokens by adapter: list[start[a]] .. are the count[a] tokens of adapter a,
//   ascending, then -1 up to start[a + 1]; starts are multiples of 32;
// turn: dst[a][j][i] = src[a][i][j] of m matrices, src [rows][cols] dense, dst row
//   stride ldd >= rows, zero in columns rows .. ldd-1;
// pad: dst[t][0 .. gemm16_depth(d)) = src[t][0 .. d) and zeros.
bool adapters_want_order(int64_t n, int m, const int32_t* index);
inline int64_t list_places(int64_t n, int64_t m) { return (n + 31) / 32 * 32 + 32 * m; }
struct TransposeArgs {
  const uint16_t* src;
  int64_t rows, cols;
  uint16_t* dst;
  int64_t ldd;        // a multiple of 8; dst on 16 bytes
  int64_t tiles, blocks;   // set by the launch, as vec
  bool vec;
};
struct PadArgs {
  const uint16_t* src;
  int64_t d, lds;
  uint16_t* dst;
  int64_t kp, blocks;
};
struct PrepareArgs {
  Adapters ad;
  int64_t n;
  int32_t *order, *list, *start, *count;
  int order_blocks, list_blocks;   // set by the launch, as blocks and kp
  TransposeArgs turn[2];
  PadArgs pad[2];
};
void launch_prepare_adapters(const PrepareArgs& g, hipStream_t s);
// With everything that a call may lay out: A and B transposed (their rows r and c, or
// 0), and rows of `padded` columns in all copied.
bool prepare_adapters_fits(int64_t n, int64_t m, int64_t rank, int64_t r, int64_t c, int64_t padded);

// out = base + S B^T, of type yt.  base: of the same type (null: 0), or the sum of
// `splits` parts [n][ldp] fp32 times 2^ex[t] (ex null: 1), ldp = part_width(rows).
// S null: no adapters, and parts to join.
inline int64_t part_width(int64_t rows) { return (rows + 7) / 8 * 8; }
struct UpArgs {
  const float* S;
  int64_t n, rows;
  Adapters ad;
  const uint16_t* B;      // [m][rows][rank] of type xt
  const void* base;
  int64_t ldb;
  const float* part;
  int64_t ldp;
  int splits;
  const int32_t* ex;
  void* out;
  int64_t ldo;
  int64_t col_tiles;      // set by the launch
  bool vec_base, vec_out;
};
void launch_adapter_up(const UpArgs& u, int xt, int yt, hipStream_t s);
bool adapter_up_fits(int64_t n, int m, int64_t rows);
bool join_rows_fits(int64_t n, int64_t rows);
// gA[a][p][k] = sum over a's tokens of T[t][p] X[t][k] and gB[a][i][p] = ... S[t][p]
// dY[t][i], from the rank values S[0] = T and S[1] = S in list order: terms[w] holds the
// three bf16 terms of S[w][list[i]][p] (0 where list[i] is -1), rank rows and places in
// blocks of 16 x 32.
struct TermsArgs {
  Adapters ad;
  int64_t n, places;
  const int32_t *list, *start;
  float* S[2];
  int splits[2];       // parts that down left
  bool keep[2];        // joined values are written to S
  uint16_t* terms[2];
};
struct GradProblem {
  const uint16_t* terms;
  const uint16_t* Z;   // rows on 16 bytes
  int64_t cols, ldz, width;   // width: columns that can be read, a multiple of 8
  int up;              // 0: G[a][p][j], 1: G[a][j][p]
  float* G;            // set by the launch, as what follows
  int splits;
  int64_t col_blocks, items;
};
struct GradArgs {
  Adapters ad;
  const int32_t *list, *start, *count;
  int rank_blocks;     // set by the launch
  GradProblem p[2];    // gA, gB
};
int64_t adapter_grad_floats(int64_t n, int m, int64_t r, int64_t c, int rank);
bool adapter_grads_fits(int64_t n, int m, int64_t r, int64_t c, int rank);
void launch_adapter_grads(const TermsArgs& terms, const GradArgs& g, int zt, float* gA, float* gB, float* part, hipStream_t s);

// out = X W^T (+ S B^T): gemm16.hip.  The contraction has kp columns, a
// multiple of its step, with zeros in W past the last one (and finite values
// in X).
constexpr int kGemm16Step = 64;
inline int64_t gemm16_depth(int64_t k) { return (k + kGemm16Step - 1) / kGemm16Step * kGemm16Step; }
struct Gemm16 {
  const uint16_t* X;      // [n][ldx], rows on 16 bytes, ldx < 2^22
  const uint16_t* W;      // [terms][cols][kp], kp < 2^22
  int64_t n, ldx, kp;
  int cols, tok_tiles, col_tiles;
  Adapters ad;
  const uint16_t* B;      // [m][cols][rank]
  const float* S;         // null: no adapters
  void* out;
  int64_t ldo;
  bool vec;               // set by launch_gemm16, as splits
  int splits;
  float* part;            // gemm16_part_floats() of workspace (null where that is 0)
};
// dt: type of X, W and B; ot: of out.  fp32 results take W in as many terms of
// its type as fp32 has bits.
constexpr int gemm16_terms(int dt, int ot) { return ot != 0 ? 1 : (dt == kBF16 ? 3 : 2); }
void launch_gemm16(const Gemm16& a, int dt, int ot, hipStream_t s);
int64_t gemm16_part_floats(int64_t n, int64_t cols, int64_t kp, int dt, int ot);
// With the copy of rows of kp columns that it may need.
bool gemm16_fits(int64_t n, int64_t cols, int64_t kp);
// Whether rows of d values can be its X as they are, and a copy (n x
// gemm16_depth(d)) that can.
bool gemm16_takes(const void* X, int64_t d, int64_t ldx);
void launch_pad_rows(const void* X, int64_t n, int64_t d, int64_t ldx, const int32_t* perm, uint16_t* dst, hipStream_t s);

// Y = X W_hat^T (+ S B^T): packed_linear.hip.
void launch_packed_linear(const void* X, int xt, int64_t n, int64_t ldx, const PackedLayer& w, const Adapters& ad,
                          const float* S, void* Y, int yt, int64_t ldy, hipStream_t s);
// dst[t][j] = X[t][perm[j]] (entries outside 0 .. c-1 clamped), dst dense.
void launch_gather_columns(const void* X, int64_t n, int64_t c, int64_t ldx, const int32_t* perm, void* dst, hipStream_t s);
bool packed_rows_fits(int64_t n, int64_t r, int64_t c);
// The same for many tokens: packed_tiles.hip.  ws: packed_tiles_bytes().
bool packed_tiles(int64_t n, int64_t r, int64_t c);
double packed_rows_us(int64_t n, int64_t r, int64_t c);   // launch_packed_linear's time, as its model has it
int64_t packed_tiles_bytes(int64_t n, int64_t r, int64_t c, int yt);
bool packed_tiles_copies(int64_t n, int yt);   // whether through a dequantized copy
bool packed_tiles_fits(int64_t n, int64_t r, int64_t c, int yt);
void launch_packed_tiles(const void* X, int xt, int64_t n, int64_t ldx, const PackedLayer& w, const Adapters& ad, const float* S,
                         void* Y, int yt, int64_t ldy, void* ws, hipStream_t s);
// dX = dY W_hat (+ T A): packed_backward.hip.  At: A transposed to [m][c][rank];
// Wt: gemm16_terms x c x gemm16_depth(r) values, rows: n x gemm16_depth(r), part: as
// Gemm16's.
void launch_packed_backward(const void* dY, int xt, int64_t n, int64_t ldy, const PackedLayer& w, const Adapters& ad,
                            const uint16_t* At, const float* T, void* dX, int ot, int64_t ldx, uint16_t* Wt, uint16_t* rows,
                            float* part, hipStream_t s);
bool packed_backward_fits(int64_t n, int64_t r, int64_t c);

}  // namespace gptq
