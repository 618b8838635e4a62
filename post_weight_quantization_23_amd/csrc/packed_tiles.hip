// Product of many tokens (prompts, batches) with a packed layer on tiles of the
// matrix cores, with the low-rank adapters beside it.
//
// Codes become fp16 values q - z exactly, in about nine operations for eight
// codes (centered).  Activations become fp16 once per call (prepare_tokens): bf16
// ones are scaled by a power of two per token, its largest value to 2^14 .. 2^15,
// which keeps every value within 2^-31 of the largest exactly and the others to
// 2^-39 of it (half of fp16's smallest step, 2^-25).  A
// group's products are then whole-number weights times activations with fp32
// sums, and its scale multiplies the sum: the weights are never rounded.
//
// Work split: 4 waves of 32 MT tokens x 32 NT rows over the same tokens, so a
// workgroup is 32 MT x 128 NT.  Activations of 128 columns come into LDS by
// loads that write it (double buffered; 16-byte chunks permuted by the row, so
// that operand reads spread over the banks); words go straight into the
// registers of the one wave that needs them, which dequantizes them once and
// uses them for all MT token tiles.  517 tokens of 4096 x 4096 at 3 bits take 35 us (0.5
// PFLOP/s), 7 of preparing and 7 of joining before and after; LDS reads and the
// dequantizing share the issue with the matrix cores.
#include "adapter.hpp"

namespace gptq {

namespace {

typedef __attribute__((address_space(3))) unsigned char lds_u8;
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));

constexpr int STEP = 128, ROWB = STEP * 2;   // columns of a step, bytes of an LDS row
constexpr int64_t kCopyTokens = 1024;         // see packed_tiles_copies

struct TileArgs {
  const uint16_t* X;   // prepared activations [n][ldx]
  const int32_t* ex;   // their exponents
  int64_t n;
  int ldx, row_tiles, tok_tiles;
  PackedLayer w;
  int splits;          // parts of the contraction
  float* out;          // parts [splits][n][r], to be summed and times 2^ex; or the
  int64_t ldo;         //   results themselves (one part, rows of ldo)
  bool direct, vec;    // results; rows of out start on 16 bytes
};

// What turns a block's codes into fp16 values q - z, a pair at a time: a field
// at bit p of each half, under the exponent of 1024, reads as 1024 + 2^p q;
// times 2^-p, minus 2^(10-p) + z, it is q - z, every step exact.  The fields
// that a half's ten mantissa bits hold need no shift (two of four at 4 bits,
// three at 3 bits).
template <int BITS>
struct Center {
  static constexpr int FIT = BITS == 4 ? 2 : 3;   // fields read in place
  half2_t off[FIT];                               // 2^(10 - BITS f) + z
  GPTQ_DEV void set(int zero) {
#pragma unroll
    for (int f = 0; f < FIT; ++f) {
      const _Float16 o = (_Float16)(float)((1 << (10 - BITS * f)) + zero);
      off[f] = half2_t{o, o};
    }
  }
};

// Codes (t, t + 4) of a block as fp16 pairs q - z.  magic is 0x64006400 in a
// vector register, so that mask and exponent are one instruction (its other
// constant, the mask, takes the one scalar operand).
template <int BITS>
GPTQ_DEV u32x4 centered(uint32_t blk, const Center<BITS>& c, uint32_t magic) {
  if constexpr (BITS == 3) blk = (blk & 0xFFFu) | ((blk & 0xFFF000u) << 4);   // codes 4 .. 7 to the high half
  u32x4 v;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    constexpr int FIT = Center<BITS>::FIT;
    const int f = t % FIT;
    const uint32_t w = t < FIT ? blk : blk >> (BITS * FIT);
    const uint32_t pair = (w & ((((1u << BITS) - 1) << (BITS * f)) * 0x10001u)) | magic;
    const _Float16 k = (_Float16)(1.0f / (float)(1 << (BITS * f)));
    const half2_t h = __builtin_bit_cast(half2_t, pair);
    const half2_t d = f == 0 ? h - c.off[0] : h * half2_t{k, k} - c.off[f];
    v[t] = __builtin_bit_cast(uint32_t, d);
  }
  return v;
}

// CPS: chunks of 32 columns that share a ruler within a step (4, 2 or 1).
template <int BITS, int MT, int CPS>
GPTQ_DEV void tiles_body(const TileArgs& a, unsigned char* xs) {
  constexpr int NT = 1;   // 32-row tiles per wave (two need more registers than two waves a SIMD have: 1.09 against 0.89 ms)
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 31, h = lane >> 5;
  int tt, rt;
  const int64_t tile = blockIdx.x / a.splits;
  const int split = (int)(blockIdx.x - tile * a.splits);
  tile_of(tile, a.tok_tiles, a.row_tiles, tt, rt);
  const int64_t t0 = (int64_t)tt * 32 * MT;
  const int row0 = rt * 128 * NT + wave * 32 * NT;
  const int nch = a.w.c >> 5, all = (nch + 3) >> 2, each = (all + a.splits - 1) / a.splits;
  const int s0 = split * each, steps = min(all, s0 + each);

  const uint32_t* words[NT];
  const float* srow[NT];
  const int32_t* zrow[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int row = min(row0 + 32 * q + m, a.w.r - 1);
    words[q] = a.w.words + (int64_t)row * a.w.ldw;
    srow[q] = a.w.scales + (int64_t)row * a.w.ldg;
    zrow[q] = a.w.zeros + (int64_t)row * a.w.ldg;
  }

  // activations: an instruction of a wave moves 4 rows of 256 bytes; rows past
  // the last token lie outside the descriptor's records and read as zero
  int off[2 * MT];
#pragma unroll
  for (int q = 0; q < 2 * MT; ++q) {
    const int row = 4 * (wave * 2 * MT + q) + (lane >> 4);
    off[q] = (row * a.ldx + 8 * ((lane & 15) ^ (row & 15))) * 2;
  }
  const int records = (int)(min(a.n - t0, (int64_t)32 * MT) * a.ldx * 2);
  lds_u8* lbase = (lds_u8*)xs;
  auto load_x = [&](int s) {
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc((void*)(a.X + t0 * a.ldx + s * STEP), (short)0,
                                                                        records - s * ROWB, 0x00020000);
#pragma unroll
    for (int q = 0; q < 2 * MT; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, lbase + (s & 1) * (32 * MT * ROWB) + (wave * 2 * MT + q) * 1024, 16, off[q], 0,
                                               0, 0);
  };

  constexpr int RU = 4 / CPS;   // rulers per step
  Chunk<BITS> cw[NT][2];
  float sc[NT][RU];
  int ze[NT][RU];
  auto load_w = [&](int s) {
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      cw[q][0] = load_chunk<BITS>(words[q], min(4 * s + 2 * h, nch - 1));
      cw[q][1] = load_chunk<BITS>(words[q], min(4 * s + 2 * h + 1, nch - 1));
#pragma unroll
      for (int u = 0; u < RU; ++u) {
        const int g = a.w.group(min(4 * s + CPS * u, nch - 1));
        sc[q][u] = srow[q][g];
        ze[q][u] = zrow[q][g];
      }
    }
  };

  floatx16 tot[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int q = 0; q < NT; ++q) tot[i][q] = floatx16{};

  uint32_t magic = 0x64006400u;
  asm volatile("" : "+v"(magic));
  load_x(s0);
  load_w(s0);
  for (int s = s0; s < steps; ++s) {
    // this step's operands.  CPS == 4: product j takes words j of the lane's
    // two chunks, columns 64 h + 8 j.  Otherwise the halves exchange words, so
    // that products 2 ch and 2 ch + 1 are chunk ch alone, columns 32 ch + 8 h
    // and + 16.
    u32x4 wf[NT][8];
    float scale[NT][RU];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      Center<BITS> o[RU];
#pragma unroll
      for (int u = 0; u < RU; ++u) {
        scale[q][u] = sc[q][u];
        o[u].set(ze[q][u]);
      }
      uint32_t blk[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) blk[j] = code_block<BITS>(cw[q][j >> 2].w, j & 3);
      if constexpr (CPS < 4) {
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const auto r = __builtin_amdgcn_permlane32_swap(blk[j], blk[j + 1], false, false);
          const int c = j >> 2, u = (j >> 1) & 1;   // chunk of the half's two, product of the chunk
          x[2 * c + u] = r[0];                      // chunk c (held by half 0)
          x[2 * (2 + c) + u] = r[1];                // chunk 2 + c (held by half 1)
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) blk[j] = x[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) wf[q][j] = centered<BITS>(blk[j], o[CPS == 4 ? 0 : (j >> 1) / CPS], magic);
    }
    // own loads have landed; with every wave here, the other buffer is free
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (s + 1 < steps) {
      load_x(s + 1);
      load_w(s + 1);
    }
    const unsigned char* xb = xs + (s & 1) * (32 * MT * ROWB);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      u32x4 x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int chunk = CPS == 4 ? 8 * h + j : 4 * (j >> 1) + 2 * (j & 1) + h;
        x[j] = *reinterpret_cast<const u32x4*>(xb + (32 * i + m) * ROWB + ((chunk ^ (m & 15)) << 4));
      }
#pragma unroll
      for (int u = 0; u < RU; ++u)
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          floatx16 p = floatx16{};
#pragma unroll
          for (int j = 2 * CPS * u; j < 2 * CPS * (u + 1); ++j) p = mfma32<kF16>(x[j], wf[q][j], p);
#pragma unroll
          for (int e = 0; e < 16; ++e) tot[i][q][e] = __builtin_fmaf(scale[q][u], p[e], tot[i][q][e]);
        }
    }
  }

  float* own = reinterpret_cast<float*>(xs) + wave * 32 * (32 * NT + 4);
  __syncthreads();   // the last step's operands have been read
  const int64_t width = a.direct ? a.w.r : a.ldo;   // the columns between r and a part's width are sums of the last row
  float* out = a.out + (int64_t)split * a.n * a.ldo;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t ti = t0 + 32 * i;
    if (a.direct) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int ex = a.ex[min(ti + TileShape<floatx16>::acc_row(lane, e), a.n - 1)];
#pragma unroll
        for (int q = 0; q < NT; ++q) tot[i][q][e] = __builtin_ldexpf(tot[i][q][e], ex);
      }
    }
    store_tile<0, NT>(own, tot[i], Adapters{}, out, ti, a.n, row0, width, a.ldo, a.vec);
  }
}

template <int BITS, int MT, int CPS>
__global__ __launch_bounds__(256, 2) void tiles_kernel(TileArgs a) {
  // the operands of two steps, and then four waves' results
  __shared__ __align__(16) unsigned char xs[2 * 32 * MT * ROWB > 4 * 32 * 36 * 4 ? 2 * 32 * MT * ROWB : 4 * 32 * 36 * 4];
  tiles_body<BITS, MT, CPS>(a, xs);
}

// Activations for tiles_kernel: fp16 in the order of code_pairs, columns
// gathered through perm, zero up to whole steps, and the token's exponent
// (the value is X' 2^ex).  One workgroup per token.
template <int DT>
__global__ __launch_bounds__(256) void prepare_tokens_kernel(const uint16_t* __restrict__ X, int64_t ldx, bool vec, int c,
                                                             const int32_t* __restrict__ perm, uint16_t* __restrict__ dst,
                                                             int ldd, int32_t* __restrict__ exps) {
  __shared__ float wave_max[4];
  const int64_t t = blockIdx.x;
  const uint16_t* x = X + t * ldx;
  auto load = [&](int j) {
    if (!perm) return load8(x + j, 8, vec);
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p0 = min(max(perm[j + 2 * e], 0), c - 1), p1 = min(max(perm[j + 2 * e + 1], 0), c - 1);
      v[e] = (uint32_t)x[p0] | ((uint32_t)x[p1] << 16);
    }
    return v;
  };
  int shift = 0;
  if constexpr (DT == kBF16) {
    float top = 0.f;
    for (int j = 8 * threadIdx.x; j < c; j += 2048) {
      const u32x4 v = load8(x + j, 8, vec);   // any order will do
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        top = fmaxf(top, fabsf(__uint_as_float(v[e] << 16)));
        top = fmaxf(top, fabsf(__uint_as_float(v[e] & 0xFFFF0000u)));
      }
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) top = fmaxf(top, __shfl_xor(top, s));
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wave_max[0], wave_max[1]), fmaxf(wave_max[2], wave_max[3]));
    shift = top > 0.f && top < __builtin_inff() ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
  }
  if (threadIdx.x == 0) exps[t] = -shift;
  for (int j = 8 * threadIdx.x; j < ldd; j += 2048) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (j < c) v = load(j);
    if constexpr (DT == kBF16) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = pack2<kF16>(__builtin_ldexpf(__uint_as_float(v[e] << 16), shift),
                           __builtin_ldexpf(__uint_as_float(v[e] & 0xFFFF0000u), shift));
    }
    *reinterpret_cast<u32x4*>(dst + t * ldd + j) = pair_order(v);
  }
}

// Chunks of a step that share a ruler (CPS of tiles_kernel).
int chunks_per_ruler(const PackedLayer& w) { return w.cpg % 4 == 0 || w.shift == 31 ? 4 : (w.cpg % 2 == 0 ? 2 : 1); }

template <int BITS, int MT>
void launch_tiles(const TileArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.tok_tiles * a.row_tiles * a.splits)), block(256);
  const int chunks = chunks_per_ruler(a.w);
  if (chunks == 4) hipLaunchKernelGGL((tiles_kernel<BITS, MT, 4>), grid, block, 0, s, a);
  else if (chunks == 2) hipLaunchKernelGGL((tiles_kernel<BITS, MT, 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((tiles_kernel<BITS, MT, 1>), grid, block, 0, s, a);
}

// The layer as 16-bit rows in packed column order, zero from column c to kp.
// One wave per row, a block of eight columns per lane.
template <int BITS, int DT>
__global__ __launch_bounds__(256) void dequant_rows_kernel(PackedLayer w, uint16_t* __restrict__ W, int kp) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= w.r) return;
  const float* srow = w.scales + row * w.ldg;
  const int32_t* zrow = w.zeros + row * w.ldg;
  const uint32_t* words = w.words + row * w.ldw;
  for (int b = threadIdx.x & 63; 8 * b < kp; b += 64) {
    u32x4 o = {0u, 0u, 0u, 0u};
    if (8 * b < w.c) {
      const int g = w.group(b >> 2);
      const float z = (float)zrow[g], sc = srow[g];
      const uint32_t blk = BITS == 4 ? words[b] : straddling_block(words, b);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w0 = weight32<DT>((blk >> (2 * BITS * e)) & ((1u << BITS) - 1), z, sc);
        const float w1 = weight32<DT>((blk >> (2 * BITS * e + BITS)) & ((1u << BITS) - 1), z, sc);
        o[e] = pack2<DT>(w0, w1);
      }
    }
    *reinterpret_cast<u32x4*>(W + row * kp + 8 * b) = o;
  }
}

// Tiles of 32 mt tokens x 128 rows, the contraction in `splits` parts, as a model of
// the measured times has it: microseconds of a step for one workgroup alone on
// a CU and for two, by the chunks that share a ruler (a scale for every 32
// columns takes four times the multiplications), and parts written and read
// back at 8 TB/s (they stay in the caches).  On 30 sizes (65 to 1000 tokens, six
// layers) the choice was within 19 % of the best of 24, half of them within 4 %.
struct TilePlan {
  int mt, splits;
  double us;
};

TilePlan plan_tiles(int64_t n, int64_t r, int64_t c, int chunks) {
  const double alone0 = chunks == 4 ? 0.85 : (chunks == 2 ? 1.1 : 1.45), alone1 = chunks == 4 ? 0.14 : (chunks == 2 ? 0.17 : 0.21);
  const double two0 = chunks == 4 ? 0.66 : (chunks == 2 ? 1.0 : 1.9), two1 = chunks == 4 ? 0.48 : (chunks == 2 ? 0.55 : 0.7);
  const int64_t steps = (c + STEP - 1) / STEP, row_tiles = (r + 127) / 128;
  TilePlan best{4, 1, 1e30};
  for (int mt = 1; mt <= 4; mt *= 2)
    for (int64_t splits = 1; splits <= 16 && (splits == 1 || 2 * splits <= steps); ++splits) {
      const int64_t groups = (n + 32 * mt - 1) / (32 * mt) * row_tiles * splits, each = (steps + splits - 1) / splits;
      const int64_t per_cu = (groups + 255) / 256;
      const double us = each * (per_cu / 2 * (two0 + two1 * mt) + per_cu % 2 * (alone0 + alone1 * mt)) + splits * n * r * 8 / 8e6;
      if (us < best.us) best = {mt, (int)splits, us};
    }
  return best;
}

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }
int64_t tiles_width(int64_t c) { return (c + STEP - 1) / STEP * STEP; }

}  // namespace

// 16-bit results of many tokens: the layer is dequantized once into 16-bit rows
// (each weight rounded to the activations' type, as gptq_linear_forward does)
// and multiplied by gemm16.  Its product runs at 1.25 PFLOP/s where the tiles
// here, which also multiply scales and dequantize for every 128 tokens, reach
// 0.83, and the copy costs 34 us for 45 million weights: 655 against 950 us for
// 8192 tokens of 11008 x 4096 in groups of 128 (of 32: 654 and 1271), 109 and 139
// for 1024.  The two meet at some 600 tokens (4096 x 4096: 512 tokens 44 and 42,
// 768 54 and 57, 1024 57 and 69) and later in layers of few rows (1024 x 4096: 1024
// tokens 35 and 31, 1536 35 and 39).  From 1024 tokens on the speed is taken for
// the rounding; below, and for fp32 results of any number, the weights stay
// unrounded.
bool packed_tiles_copies(int64_t n, int yt) { return yt != 0 && n >= kCopyTokens; }

// Below the tokens of a copy, the kernel for few tokens as long as the models of both
// say so; tiles take three launches, with what these leave between them in memory
// (10 us).  By that kernel and in tiles: 512 tokens of 1024 x 4096 16 and 28 us, 128 of
// 4096 x 4096 16 and 27, 512 of them 54 and 42, 65 tokens of 12288 x 8192 55 and 46.
bool packed_tiles(int64_t n, int64_t r, int64_t c) {
  if (n <= 64 || c >= (int64_t(1) << 22) - STEP) return false;
  return n >= kCopyTokens || packed_rows_us(n, r, c) > 10 + plan_tiles(n, r, c, 4).us;
}

int64_t packed_tiles_bytes(int64_t n, int64_t r, int64_t c, int yt) {
  if (packed_tiles_copies(n, yt))
    return align256(n * gemm16_depth(c) * 2) + align256(r * gemm16_depth(c) * 2) + 4 * gemm16_part_floats(n, r, gemm16_depth(c), yt, yt);
  int64_t splits = yt == 0 ? 0 : 1;   // one part of fp32 results is the results
  for (const int chunks : {4, 2, 1}) {
    const int k = plan_tiles(n, r, c, chunks).splits;
    splits = k > 1 && k > splits ? k : splits;
  }
  return align256(n * tiles_width(c) * 2) + align256(n * 4) + align256(splits * n * part_width(r) * 4);
}

bool packed_tiles_fits(int64_t n, int64_t r, int64_t c, int yt) {
  if (packed_tiles_copies(n, yt)) return grid_fits((r + 3) / 4, 256) && gemm16_fits(n, r, gemm16_depth(c));
  const int64_t row_tiles = (r + 127) / 128;
  // a workgroup for each token to prepare; the largest tiles, as a bound that plan_tiles needs
  if (!grid_fits(n, 256) || !grid_fits((n + 127) / 128 * row_tiles, 256)) return false;
  for (const int chunks : {4, 2, 1}) {
    const TilePlan p = plan_tiles(n, r, c, chunks);
    if (!grid_fits((n + 32 * p.mt - 1) / (32 * p.mt) * row_tiles * p.splits, 256)) return false;
    if ((yt != 0 || p.splits > 1) && !join_rows_fits(n, r)) return false;
  }
  return true;
}

void launch_packed_tiles(const void* X, int xt, int64_t n, int64_t ldx, const PackedLayer& w, const Adapters& ad, const float* S,
                         void* Y, int yt, int64_t ldy, void* ws, hipStream_t s) {
  auto* xp = static_cast<uint16_t*>(ws);
  const dim3 block(256);
  if (packed_tiles_copies(n, yt)) {
    Gemm16 g{};
    g.kp = gemm16_depth(w.c);
    g.X = static_cast<const uint16_t*>(X);
    g.ldx = ldx;
    if (w.perm || !gemm16_takes(X, w.c, ldx)) {
      launch_pad_rows(X, n, w.c, ldx, w.perm, xp, s);
      g.X = xp;
      g.ldx = g.kp;
    }
    uint16_t* W = xp + align256(n * g.kp * 2) / 2;
    const dim3 dgrid((unsigned)((w.r + 3) / 4));
#define GPTQ_DEQ(B_, D_) hipLaunchKernelGGL((dequant_rows_kernel<B_, D_>), dgrid, block, 0, s, w, W, (int)g.kp)
    if (w.bits == 4) { if (xt == kBF16) GPTQ_DEQ(4, kBF16); else GPTQ_DEQ(4, kF16); }
    else { if (xt == kBF16) GPTQ_DEQ(3, kBF16); else GPTQ_DEQ(3, kF16); }
#undef GPTQ_DEQ
    g.W = W;
    g.part = reinterpret_cast<float*>(W + align256((int64_t)w.r * g.kp * 2) / 2);
    g.n = n;
    g.cols = w.r;
    g.ad = ad;
    g.B = ad.B;
    g.S = S;
    g.out = Y;
    g.ldo = ldy;
    launch_gemm16(g, xt, yt, s);
    return;
  }
  const int ldp = (int)tiles_width(w.c);
  auto* ex = reinterpret_cast<int32_t*>(xp + align256(n * ldp * 2) / 2);
  const auto* x = static_cast<const uint16_t*>(X);
  const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0;
  if (xt == kBF16) hipLaunchKernelGGL((prepare_tokens_kernel<kBF16>), dim3((unsigned)n), block, 0, s, x, ldx, vec, w.c, w.perm, xp, ldp, ex);
  else hipLaunchKernelGGL((prepare_tokens_kernel<kF16>), dim3((unsigned)n), block, 0, s, x, ldx, vec, w.c, w.perm, xp, ldp, ex);
  const TilePlan p = plan_tiles(n, w.r, w.c, chunks_per_ruler(w));
  TileArgs a{};
  a.X = xp;
  a.ex = ex;
  a.n = n;
  a.ldx = ldp;
  a.w = w;
  a.tok_tiles = (int)((n + 32 * p.mt - 1) / (32 * p.mt));
  a.row_tiles = (w.r + 127) / 128;
  a.splits = p.splits;
  a.direct = yt == 0 && p.splits == 1;
  a.out = a.direct ? static_cast<float*>(Y) : reinterpret_cast<float*>(ex + align256(n * 4) / 4);
  a.ldo = a.direct ? ldy : part_width(w.r);
  a.vec = rows_on_16(a.out, a.ldo, 0);
#define GPTQ_TILES(B_) (p.mt == 4 ? launch_tiles<B_, 4>(a, s) : p.mt == 2 ? launch_tiles<B_, 2>(a, s) : launch_tiles<B_, 1>(a, s))
  if (w.bits == 4) GPTQ_TILES(4);
  else GPTQ_TILES(3);
#undef GPTQ_TILES
  if (a.direct && !S) return;
  // the parts joined, the adapters added, one rounding
  UpArgs u{};
  u.S = S;
  u.n = n;
  u.rows = w.r;
  u.ad = ad;
  u.B = ad.B;
  if (a.direct) {
    u.base = Y;
    u.ldb = ldy;
  } else {
    u.part = a.out;
    u.ldp = a.ldo;
    u.splits = p.splits;
    u.ex = ex;
  }
  u.out = Y;
  u.ldo = ldy;
  launch_adapter_up(u, xt, yt, s);
}

}  // namespace gptq
