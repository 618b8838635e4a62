// out = X W^T (+ S B^T) with 16-bit operands that are both contiguous along the
// contraction, on tiles of the matrix cores: the product behind the input
// gradient (packed_backward.hip) and behind the packed product of many tokens
// (packed_tiles.hip), each of which prepares its operands first.  A 256 x 256 tile
// runs at 1.17 to 1.26 PFLOP/s (4096 to 8192 tokens of 11008 x 4096) with the matrix
// cores busy 58 % of the time, at the clock that the power limit leaves; waves
// of 128 x 128 (four instead of eight), raised wave priority and operands fetched
// a step ahead were no faster.
#include "adapter.hpp"

namespace gptq {

namespace {

typedef __attribute__((address_space(3))) unsigned char lds_u8;

// ---------------------------------------------------------------- product
constexpr int LK = kGemm16Step, ROWB = LK * 2;   // contraction step, bytes of an LDS row

// Chunk c (16 bytes) of LDS row f lies at place c ^ swz(f).
GPTQ_DEV int swz(int f) { return (f ^ (f >> 3)) & 7; }

// What the adapters' part of a tile keeps in LDS behind the operands: token and
// adapter of each place.
template <int TM>
struct Places {
  int tok[TM], who[TM];
};

// acc[i][q] += S B_a^T for the tile's adapters (S in TERMS bf16 terms).  S and, for one
// adapter after the other, the tile's rows of B come into the operands' LDS in
// whole runs, 64 ranks at a time: operands loaded straight into registers would
// touch 32 rows per instruction, at a place a cycle (2085 tokens of 4096 x 4096
// with rank 64 on tiles of 96 x 128: 110 us, 116 so).  Sets of 32 places that one adapter has to itself take
// its products onto their sums; the others follow by expand_shared, so that a
// value that is not finite in one request stays there.
template <int DT, int TERMS, int MT, int NT, int WM, int WN>
GPTQ_DEV void expand_staged(const Gemm16& a, const Places<32 * MT * WM>* pl, unsigned char* smem, int j0, int wm, int wn,
                            const int64_t (&col)[NT], floatx16 (&acc)[MT][NT]) {
  constexpr int TM = 32 * MT * WM, TN = 32 * NT * WN, RANKS = 64;
  constexpr int QS = TM / 4 / (WM * WN), QB = TN / 8 / WN;   // load instructions per wave: 4 rows of S, 8 of B
  static_assert(QS * 4 * WM * WN == TM && QB * 8 * WN == TN, "rows divide over the waves");
  static_assert(TM * 256 + WM * TN * 128 <= 2 * (TM + TN) * ROWB, "S and each wave row's B fit the operands' LDS");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), m = lane & 31, h = lane >> 5;
  const int rank = a.ad.rank;
  unsigned char* bs = smem + TM * 256 + (wave / WN) * TN * 128;   // B of the waves with these tokens
  lds_u8 *ls = (lds_u8*)smem, *lb = (lds_u8*)bs;
  for (int k0 = 0; k0 < rank; k0 += RANKS) {
    const int ranks = min(RANKS, rank - k0);
#pragma unroll 2
    for (int q = 0; q < QS; ++q) {
      const int row = 4 * (wave * QS + q) + (lane >> 4), piece = (lane & 15) ^ (row & 15);
      const float* from = a.S + (int64_t)max(pl->tok[row], 0) * rank + k0 + (4 * piece < ranks ? 4 * piece : 0);
      __builtin_amdgcn_global_load_lds((const void __attribute__((address_space(1)))*)from,
                                       (void __attribute__((address_space(3)))*)(ls + (wave * QS + q) * 1024), 16, 0, 0);
    }
    int held = -1;   // the adapter whose B lies in bs
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int at = wm + 32 * i + m, tok = pl->tok[at], mine = pl->who[at], first = __builtin_amdgcn_readfirstlane(mine);
      const bool whole = first >= 0 && (uint32_t)__ballot(mine == first) == (uint32_t)__ballot(tok >= 0);
      if (whole && first != held) {
        held = first;
#pragma unroll 2
        for (int q = 0; q < QB; ++q) {
          const int row = 8 * ((wave % WN) * QB + q) + (lane >> 3), piece = (lane & 7) ^ (row & 7);
          const uint16_t* from = a.B + ((int64_t)first * a.cols + min(j0 + row, a.cols - 1)) * rank + k0 + (8 * piece < ranks ? 8 * piece : 0);
          __builtin_amdgcn_global_load_lds((const void __attribute__((address_space(1)))*)from,
                                           (void __attribute__((address_space(3)))*)(lb + ((wave % WN) * QB + q) * 1024), 16, 0, 0);
        }
      }
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if (whole) {
        for (int k1 = 0; k1 < ranks; k1 += 16) {
          const int k = k1 + 8 * h;
          const bool in = k < ranks;
          const floatx4 lo = *reinterpret_cast<const floatx4*>(smem + at * 256 + (((k >> 2) ^ (at & 15)) << 4));
          const floatx4 hi = *reinterpret_cast<const floatx4*>(smem + at * 256 + ((((k >> 2) + 1) ^ (at & 15)) << 4));
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = in ? lo[e] : 0.f;
            v[4 + e] = in ? hi[e] : 0.f;
          }
          u32x4 s[TERMS];
          split8<TERMS>(v, s);
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            const int f = wn + 32 * q + m;
            u32x4 b = *reinterpret_cast<const u32x4*>(bs + f * 128 + (((k >> 3) ^ (f & 7)) << 4));
            if (!in) b = u32x4{0u, 0u, 0u, 0u};
            acc[i][q] = mfma_terms<DT, TERMS>(s, Terms16<DT>(b), acc[i][q]);
          }
        }
      } else if (k0 == 0) {
        uint32_t rest = (uint32_t)__ballot(mine >= 0);
        while (rest) {
          const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctz(rest));
          const uint32_t members = (uint32_t)__ballot(mine == ad);
          rest &= ~members;
          expand_shared<DT, TERMS, NT>(a.ad, ad, members, a.B, a.cols, a.S, tok, col, acc[i]);
        }
      }
      __syncthreads();   // before B, or S, is replaced
    }
  }
}

// WM x WN waves of 32 MT tokens x 32 NT columns.  Both operands come from
// memory straight into LDS (double buffered, one barrier per step), each lane
// fetching the chunk that belongs at its place; tokens and columns past the end
// lie outside the descriptors' records and read as zero, except that tokens by
// adapter, which are fetched by address, repeat the last one.  LOW: adapters beside the product (1), tokens by adapter too (2: ad.order;
// without either a 256 x 256 tile keeps all its registers).  PARTS: the workgroup takes one of
// `splits` parts of the contraction and writes its fp32 sums to part.
template <int DT, int OT, int TERMS, int LOW, bool PARTS, int MT, int NT, int WM, int WN>
GPTQ_DEV void gemm_body(const Gemm16& a, unsigned char* smem) {
  constexpr int TM = 32 * MT * WM, TN = 32 * NT * WN, NW = WM * WN, BUF = (TM + TN) * ROWB;
  constexpr int QX = TM / 8 / NW, QW = TN / 8 / NW;   // load instructions per wave: 8 rows each
  static_assert(QX * 8 * NW == TM && QW * 8 * NW == TN, "tiles divide over the waves");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 31, h = lane >> 5;
  int tt, ct;
  const int64_t tile = PARTS ? blockIdx.x / a.splits : blockIdx.x;
  const int split = PARTS ? (int)(blockIdx.x - tile * a.splits) : 0;
  tile_of(tile, a.tok_tiles, a.col_tiles, tt, ct);
  const int64_t t0 = (int64_t)tt * TM;
  const int j0 = ct * TN;
  const int wm = (wave / WN) * 32 * MT, wn = (wave % WN) * 32 * NT;
  lds_u8* lbase = (lds_u8*)smem;

  int offx[QX], offw[QW];
  const uint16_t* fromx[QX];
#pragma unroll
  for (int q = 0; q < QX; ++q) {
    const int row = 8 * (wave * QX + q) + (lane >> 3), piece = 8 * ((lane & 7) ^ swz(row));
    if constexpr (LOW == 2) fromx[q] = a.X + (int64_t)a.ad.order[min(t0 + row, a.n - 1)] * a.ldx + piece;
    else offx[q] = (row * (int)a.ldx + piece) * 2;
  }
#pragma unroll
  for (int q = 0; q < QW; ++q) {
    const int row = 8 * (wave * QW + q) + (lane >> 3);
    offw[q] = (row * (int)a.kp + 8 * ((lane & 7) ^ swz(row))) * 2;
  }
  const int xrec = (int)(min(a.n - t0, (int64_t)TM) * a.ldx * 2), wrec = (int)(min(a.cols - j0, TN) * a.kp * 2);
  const int steps = (int)(a.kp / LK), total = TERMS * steps, each = PARTS ? (total + a.splits - 1) / a.splits : total;
  const int first = split * each, all = min(total, first + each);
  auto load = [&](int s) {
    const int term = TERMS == 1 ? 0 : s / steps, k0 = (s - term * steps) * LK;
    const __amdgpu_buffer_rsrc_t rx =
        __builtin_amdgcn_make_buffer_rsrc((void*)(a.X + t0 * a.ldx + k0), (short)0, xrec - 2 * k0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(a.W + ((int64_t)term * a.cols + j0) * a.kp + k0), (short)0, wrec - 2 * k0, 0x00020000);
    lds_u8* to = lbase + (s & 1) * BUF;
#pragma unroll
    for (int q = 0; q < QX; ++q) {
      if constexpr (LOW == 2)
        __builtin_amdgcn_global_load_lds((const void __attribute__((address_space(1)))*)(fromx[q] + k0),
                                         (void __attribute__((address_space(3)))*)(to + (wave * QX + q) * 1024), 16, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, to + (wave * QX + q) * 1024, 16, offx[q], 0, 0, 0);
    }
#pragma unroll
    for (int q = 0; q < QW; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, to + TM * ROWB + (wave * QW + q) * 1024, 16, offw[q], 0, 0, 0);
  };

  floatx16 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int q = 0; q < NT; ++q) acc[i][q] = floatx16{};

  Places<TM>* pl = reinterpret_cast<Places<TM>*>(smem + 2 * BUF);
  if (LOW && tid < TM) {
    const int64_t t = a.ad.token(t0 + tid, a.n);
    pl->tok[tid] = (int)t;
    pl->who[tid] = adapter_of(a.ad, t, a.n);
  }
  if (first < all) load(first);   // past the end there are no records to bound it
  for (int s = first; s < all; ++s) {
    // own loads have landed; with every wave here, the other buffer is free
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (s + 1 < all) load(s + 1);
    const unsigned char* xb = smem + (s & 1) * BUF;
    const unsigned char* wb = xb + TM * ROWB;
#pragma unroll
    for (int k = 0; k < LK / 16; ++k) {
      u32x4 x[MT], w[NT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int f = wm + 32 * i + m;
        x[i] = *reinterpret_cast<const u32x4*>(xb + f * ROWB + (((2 * k + h) ^ swz(f)) << 4));
      }
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const int f = wn + 32 * q + m;
        w[q] = *reinterpret_cast<const u32x4*>(wb + f * ROWB + (((2 * k + h) ^ swz(f)) << 4));
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[i][q] = mfma32<DT>(x[i], w[q], acc[i][q]);
    }
  }

  static_assert(NW * 32 * (32 * NT + 4) * 4 <= 2 * BUF, "tile results fit the operands' LDS");
  float* own = reinterpret_cast<float*>(smem) + wave * 32 * (32 * NT + 4);
  __syncthreads();   // the last step's operands have been read
  if constexpr (PARTS) {
    const int64_t ldp = (a.cols + 7) & ~7;
    float* part = a.part + (int64_t)split * a.n * ldp;
#pragma unroll
    for (int i = 0; i < MT; ++i)
      store_tile<0, NT>(own, acc[i], a.ad, part, t0 + wm + 32 * i, a.n, j0 + wn, ldp, ldp, true);
    return;
  }
  int64_t col[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int at = j0 + wn + 32 * q + m;
    col[q] = at < a.cols ? at : -1;
  }
  if constexpr (LOW != 0) {
    expand_staged<DT, OT == 0 ? 3 : 2, MT, NT, WM, WN>(a, pl, smem, j0, wm, wn, col, acc);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
    store_tile<OT, NT>(own, acc[i], a.ad, a.out, t0 + wm + 32 * i, a.n, j0 + wn, a.cols, a.ldo, a.vec);
}

// LDS of a workgroup, and the waves per SIMD that it leaves room for (the smallest
// tile three: with registers for two 512 tokens of 4096 x 11008 took 84 us, so 64).
template <int LOW, int TM, int TN>
constexpr int gemm_lds() { return 2 * (TM + TN) * ROWB + (LOW ? (int)sizeof(Places<TM>) : 0); }
template <int LOW, int MT, int NT, int WM, int WN>
constexpr int gemm_waves() { return WM * WN == 4 && 3 * gemm_lds<LOW, 32 * MT * WM, 32 * NT * WN>() <= 160 * 1024 ? 3 : 2; }

template <int DT, int OT, int TERMS, int LOW, bool PARTS, int MT, int NT, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, (gemm_waves<LOW, MT, NT, WM, WN>())) void gemm_kernel(Gemm16 a) {
  extern __shared__ __align__(16) unsigned char gsm[];
  gemm_body<DT, OT, TERMS, LOW, PARTS, MT, NT, WM, WN>(a, gsm);
}

template <int DT, int OT, int TERMS, int LOW, bool PARTS, int MT, int NT, int WM, int WN>
void launch_gemm(Gemm16 a, hipStream_t s) {
  constexpr int TM = 32 * MT * WM, TN = 32 * NT * WN, LDS = gemm_lds<LOW, TM, TN>();
  static const bool set = [] {   // once, thread-safe
    (void)hipFuncSetAttribute((const void*)gemm_kernel<DT, OT, TERMS, LOW, PARTS, MT, NT, WM, WN>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    return true;
  }();
  (void)set;
  a.tok_tiles = (int)((a.n + TM - 1) / TM);
  a.col_tiles = (a.cols + TN - 1) / TN;
  hipLaunchKernelGGL((gemm_kernel<DT, OT, TERMS, LOW, PARTS, MT, NT, WM, WN>),
                     dim3((unsigned)((int64_t)a.tok_tiles * a.col_tiles * a.splits)), dim3(64 * WM * WN), LDS, s, a);
}

// Tiles: 256 x 256 (8 waves of 128 x 64), 256 x 192 and 192 x 256 (8 of 64 x 96 and 96 x 64),
// 128 x 128 (4 of 64 x 64), 96 and 64 x 128 (4 of 96 or 64 x 32).  A launch takes as
// long as its fullest CU, ceil(tiles / 256) of them, and a large tile reads less of
// LDS for each product.  The input gradient of 2085 tokens of 4096 x 4096 took 107, 95, 96,
// 114, 107 and 110 us in this order, of 6000 tokens of 11008 x 4096 577, 644, 527, 636, 705
// and 837, of 1024 tokens of 1024 x 4096 38, 35, 34, 23, 26 and 22; the choice was within
// 9 % of the best on 84 sizes (300 to 8192 tokens, six layers), 1 % on average.
enum Shape { k256, k256x192, k192x256, k128, k96, k64, kShapes };

Shape choose_shape(int64_t n, int64_t cols, bool low) {
  constexpr int64_t tm[kShapes] = {256, 256, 192, 128, 96, 64}, tn[kShapes] = {256, 192, 256, 128, 128, 128};
  constexpr double cost[kShapes] = {0.83, 0.84, 0.84, 1.0, 1.12, 1.15};
  Shape best = k256;
  double least = 1e30;
  for (int i = 0; i < kShapes; ++i) {
    if (low && i == k256x192) continue;   // four wave rows, each with an adapter's B, are more than its LDS holds
    const int64_t tiles = (n + tm[i] - 1) / tm[i] * ((cols + tn[i] - 1) / tn[i]);
    const double us = cost[i] * tm[i] * tn[i] * (double)((tiles + 255) / 256);
    if (us < least) least = us, best = (Shape)i;
  }
  return best;
}

// Parts of the contraction, while the tiles are too few for the chip (128 x 128
// then).  Each takes ceil(steps / splits) steps, so the last of them could start past
// the end (13 parts of 9 in 108 steps): as many as hold steps are left.
int gemm16_splits(int64_t n, int64_t cols, int64_t steps) {
  if (n == 0 || cols == 0) return 1;
  const int64_t tiles = (n + 127) / 128 * ((cols + 127) / 128);
  int64_t splits = 384 / tiles;
  splits = splits < steps / 8 ? splits : steps / 8;
  if (splits < 3) return 1;
  splits = splits < 16 ? splits : 16;
  const int64_t each = (steps + splits - 1) / splits;
  return (int)((steps + each - 1) / each);
}

template <int DT, int OT, int TERMS, int LOW>
void launch_shape(const Gemm16& a, hipStream_t s) {
  switch (choose_shape(a.n, a.cols, LOW != 0)) {
    case k256: return launch_gemm<DT, OT, TERMS, LOW, false, 4, 2, 2, 4>(a, s);
    case k256x192:
      if constexpr (LOW == 0) launch_gemm<DT, OT, TERMS, 0, false, 2, 3, 4, 2>(a, s);
      return;
    case k192x256: return launch_gemm<DT, OT, TERMS, LOW, false, 3, 2, 2, 4>(a, s);
    case k128: return launch_gemm<DT, OT, TERMS, LOW, false, 2, 2, 2, 2>(a, s);
    case k96: return launch_gemm<DT, OT, TERMS, LOW, false, 3, 1, 1, 4>(a, s);
    case k64: return launch_gemm<DT, OT, TERMS, LOW, false, 2, 1, 1, 4>(a, s);
    case kShapes: return;
  }
}

template <int DT, int OT, int TERMS>
void choose_gemm(const Gemm16& a, hipStream_t s) {
  if (a.splits > 1) launch_gemm<DT, 0, TERMS, 0, true, 2, 2, 2, 2>(a, s);
  else if (!a.S) launch_shape<DT, OT, TERMS, 0>(a, s);
  else if (a.ad.order) launch_shape<DT, OT, TERMS, 2>(a, s);
  else launch_shape<DT, OT, TERMS, 1>(a, s);
}

// dst[t][0 .. kp) = src[t][0 .. d) (through perm, entries outside 0 .. d-1
// clamped) and zeros: rows for the product where the given ones do not start on
// 16 bytes, do not end on a whole step, or lie in another order.
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* __restrict__ src, int64_t n, int64_t d, int64_t lds, bool vec,
                                                       const int32_t* __restrict__ perm, uint16_t* __restrict__ dst, int64_t kp) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = kp >> 3, t = i / per, k = (i - t * per) * 8;
  if (t >= n) return;
  u32x4 v = {0u, 0u, 0u, 0u};
  if (k < d && perm) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e < d) v[e >> 1] |= (uint32_t)src[t * lds + min(max((int64_t)perm[k + e], (int64_t)0), d - 1)] << (16 * (e & 1));
  } else if (k < d) {
    v = load8(src + t * lds + k, (int)min((int64_t)8, d - k), vec);
  }
  *reinterpret_cast<u32x4*>(dst + t * kp + k) = v;
}

}  // namespace

void launch_gemm16(const Gemm16& g, int dt, int ot, hipStream_t s) {
  Gemm16 a = g;
  a.splits = gemm16_splits(a.n, a.cols, gemm16_terms(dt, ot) * (a.kp / LK));
  a.vec = rows_on_16(a.out, a.ldo, ot);
  if (a.splits > 1) a.ad.order = nullptr;   // the adapters follow where the parts are joined
  if (dt == kBF16) { if (ot == 0) choose_gemm<kBF16, 0, gemm16_terms(kBF16, 0)>(a, s); else choose_gemm<kBF16, kBF16, 1>(a, s); }
  else { if (ot == 0) choose_gemm<kF16, 0, gemm16_terms(kF16, 0)>(a, s); else choose_gemm<kF16, kF16, 1>(a, s); }
  if (a.splits == 1) return;
  UpArgs u{};
  u.S = g.S;
  u.n = g.n;
  u.rows = g.cols;
  u.ad = g.ad;
  u.B = g.B;
  u.part = a.part;
  u.ldp = part_width(g.cols);
  u.splits = a.splits;
  u.out = g.out;
  u.ldo = g.ldo;
  launch_adapter_up(u, dt, ot, s);
}

int64_t gemm16_part_floats(int64_t n, int64_t cols, int64_t kp, int dt, int ot) {
  const int splits = gemm16_splits(n, cols, gemm16_terms(dt, ot) * (kp / LK));
  return splits > 1 ? splits * n * part_width(cols) : 0;
}

// In tiles of 64 x 128 at the smallest; parts are for fewer tiles than the chip takes at once.
bool gemm16_fits(int64_t n, int64_t cols, int64_t kp) {
  return grid_fits((n + 63) / 64 * ((cols + 127) / 128), 256) && grid_fits((n * (kp / 8) + 255) / 256, 256);
}

bool gemm16_takes(const void* X, int64_t d, int64_t ldx) {
  return reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0 && ldx < (int64_t(1) << 22) && d % LK == 0;
}

void launch_pad_rows(const void* X, int64_t n, int64_t d, int64_t ldx, const int32_t* perm, uint16_t* dst, hipStream_t s) {
  const int64_t kp = gemm16_depth(d);
  const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0;
  hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)((n * (kp / 8) + 255) / 256)), dim3(256), 0, s, static_cast<const uint16_t*>(X), n,
                     d, ldx, vec, perm, dst, kp);
}

}  // namespace gptq
