// Product of many tokens with a packed layer, with the low-rank adapters of
// their requests beside it:
//     Y[t, i] = sum_j s[i, g(j)] (q[i, j] - z[i, g(j)]) X[t, perm[j]] + (S B_a^T)[t, i].
//
// Codes enter the matrix cores as whole numbers: a b-bit code shifted to the
// top of a 16-bit float's mantissa under the exponent of 2^b reads as 2^b + q
// exactly, one shift and one and-or for two codes.  With P = sum (2^b + q) x and
// X_g = sum x over a group (a product with ones, on the matrix cores too), the
// group's part is s (P - (2^b + z) X_g): the weights are never rounded, and
// every sum is fp32.  While zeros lie among the codes (0 .. 2^b - 1), the subtraction
// costs a factor below 8 in the error of the fp32 sums, three bits of 24; zeros
// far from them, up to 1000, cost as much more as they are larger.
#include <type_traits>

#include "adapter.hpp"

namespace gptq {

namespace {

typedef __attribute__((address_space(3))) unsigned char lds_u8;

struct FwdArgs {
  const uint16_t* X;
  int64_t ldx, n;
  PackedLayer w;
  Adapters ad;
  const float* S;    // null: no adapters
  void* Y;
  int64_t ldy;
  bool y32;
  int row_tiles;
  int quads;         // tokens of a workgroup in fours
};

// Register j of lane (m, kq) <-> register kq of lane (m, j), lane = m + 16 kq.
GPTQ_DEV void transpose4(uint32_t (&v)[4]) {
  auto swap16 = [](uint32_t& x, uint32_t& y) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    x = r[0];
    y = r[1];
  };
  auto swap32 = [](uint32_t& x, uint32_t& y) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    x = r[0];
    y = r[1];
  };
  swap16(v[0], v[1]);
  swap16(v[2], v[3]);
  swap32(v[0], v[2]);
  swap32(v[1], v[3]);
}

// Token groups (of 16) and row tiles of a workgroup, steps of a run, waves: what a
// workgroup reads for one token group or row tile serves the others too, as long
// as enough workgroups are left (rows_shape).  Four waves and 12 were slower than
// eight at every size tried, two steps ahead faster than one up to 16 tokens.
constexpr int MAX_TG = 4, MAX_NT = 3, WAVES = 8;
constexpr int steps_ahead(int tg) { return tg == 1 ? 2 : 1; }

// LDS bytes of a step of one wave: 16 NT rows of words, then tokens of 256 bytes.
constexpr int step_bytes(int bits, int nt, int quads) { return 256 * bits * nt + 1024 * quads; }

// 16 TG tokens x 16 NT rows per workgroup.  The waves split the columns in runs of
// AHEAD steps of 128 and are joined through LDS in wave order.
//
// What a run reads comes through the wave's own part of LDS, by loads that write
// it.  The operand layout gives consecutive lanes consecutive rows, so loading
// operands straight into registers touches 64 places of 16 bytes per
// instruction, and the L1 cache takes them one a cycle: that, not memory, set the
// pace (16 tokens of 11008 x 4096 at 3 bits: 22 us, and 40 thousand accesses
// per CU; 14 us now).  The loads into LDS give 4 (words) or 16 (activations)
// consecutive lanes one row.  What bounds it now are the waits for a run and about
// 140 instructions per step of 128 columns, not memory (1.3 TB/s of words).
//
// A lane then holds chunk kq of row m (lane = m + 16 kq); the blocks of codes are
// transposed, so that product j takes chunk j alone.  Steps, tokens and rows past
// the end repeat the last ones, under a scale of zero or with results that are
// dropped.  WIDE: groups hold whole steps, so that rulers apply per step;
// otherwise each lane reads its own chunk's ruler, and the transpose spreads
// them as well.
template <int BITS, int DT, bool WIDE, int TG, int NT>
GPTQ_DEV void rows16_body(const FwdArgs& a, unsigned char* smem) {
  constexpr int AHEAD = steps_ahead(TG);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, kq = lane >> 4;
  const int64_t tile = blockIdx.x / a.row_tiles;
  const int64_t t0 = tile * 16 * TG;
  const int row0 = (int)(blockIdx.x - tile * a.row_tiles) * 16 * NT;
  const int nch = a.w.c >> 5, steps = (nch + 3) >> 2;
  int64_t ruler[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) ruler[q] = (int64_t)min(row0 + 16 * q + m, a.w.r - 1) * a.w.ldg;
  const uint32_t one = DT == kBF16 ? 0x3F803F80u : 0x3C003C00u;
  const u32x4 ones = {one, one, one, one};
  const uint32_t exponent = code_exponent<BITS, DT>();
  const floatx4 zero4 = {0.f, 0.f, 0.f, 0.f};

  const int sb = step_bytes(BITS, NT, a.quads);
  unsigned char* own = smem + wave * AHEAD * sb;
  lds_u8* lown = (lds_u8*)own;

  // Global sources of this lane: words (4 bits: piece lane & 3 of row lane >> 2;
  // 3 bits: dwords lane, lane + 64, lane + 128 of the step's 16 x 12), tokens
  // (piece lane & 15 of tokens lane >> 4, + 4, ...).  Pieces are permuted by the
  // row, so that operand reads spread over the banks.
  constexpr int WL = BITS == 4 ? 1 : 3;
  const uint32_t* wsrc[NT][WL];
  int wcol[WL];    // chunk of the step (4 bits), dword of the step (3 bits)
#pragma unroll
  for (int i = 0; i < WL; ++i) {
    const int at = lane + 64 * i, rr = BITS == 4 ? at >> 2 : at / 12;
#pragma unroll
    for (int q = 0; q < NT; ++q) wsrc[q][i] = a.w.words + (int64_t)min(row0 + 16 * q + rr, a.w.r - 1) * a.w.ldw;
    wcol[i] = BITS == 4 ? (at & 3) ^ ((rr >> 2) & 3) : at - 12 * rr;
  }
  const uint16_t* xsrc[4 * TG];
  int xpiece[4];
#pragma unroll
  for (int i = 0; i < 4 * TG; ++i) {
    const int rr = 4 * i + (lane >> 4);
    xsrc[i] = a.X + min(t0 + rr, a.n - 1) * a.ldx;
    xpiece[i & 3] = (lane & 15) ^ (rr & 15);
  }

  int xrow[TG];    // the lane's token of each group; the last one in place of those that are not there
  floatx4 tot[TG][NT];
#pragma unroll
  for (int u = 0; u < TG; ++u) {
    xrow[u] = min(16 * u + m, 4 * a.quads - 1);
#pragma unroll
    for (int q = 0; q < NT; ++q) tot[u][q] = zero4;
  }
  auto run = [&](int s0, auto tail) __attribute__((always_inline)) {
    constexpr bool TAIL = decltype(tail)::value;   // the run may pass the last chunk
    float sc[AHEAD][NT];
    int ze[AHEAD][NT];
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      const int s = s0 + d;
      lds_u8* to = lown + d * sb;
      const int g = a.w.group(TAIL ? min(4 * s + (WIDE ? 0 : kq), nch - 1) : 4 * s + (WIDE ? 0 : kq));
#pragma unroll
      for (int q = 0; q < NT; ++q) {
#pragma unroll
        for (int i = 0; i < WL; ++i) {
          const int col = (BITS == 4 ? 4 : 12) * s + wcol[i], last = (BITS == 4 ? nch : 3 * nch) - 1;
          const uint32_t* from = wsrc[q][i] + (BITS == 4 ? 4 : 1) * (int64_t)(TAIL ? min(col, last) : col);
          auto* src = (const void __attribute__((address_space(1)))*)from;
          auto* dst = (void __attribute__((address_space(3)))*)(to + 256 * BITS * q + 256 * i);
          if constexpr (BITS == 4) __builtin_amdgcn_global_load_lds(src, dst, 16, 0, 0);
          else __builtin_amdgcn_global_load_lds(src, dst, 4, 0, 0);
        }
        sc[d][q] = a.w.scales[ruler[q] + g];
        ze[d][q] = a.w.zeros[ruler[q] + g];
      }
#pragma unroll
      for (int i = 0; i < 4 * TG; ++i)
        if (i < a.quads) {
          const int piece = 16 * s + xpiece[i & 3];
          __builtin_amdgcn_global_load_lds((const void __attribute__((address_space(1)))*)(xsrc[i] + 8 * (int64_t)(TAIL ? min(piece, 4 * nch - 1) : piece)),
                                           (void __attribute__((address_space(3)))*)(to + 256 * BITS * NT + 1024 * i), 16, 0, 0);
        }
    }
    __builtin_amdgcn_s_waitcnt(0);   // the wave reads only what it has loaded itself
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      const int s = s0 + d;
      const unsigned char* from = own + d * sb;
      uint32_t blk[NT][4], scs[NT][4], zes[NT][4];
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        uint32_t chunk[BITS];
        if constexpr (BITS == 4) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(from + 1024 * q + m * 64 + ((kq ^ ((m >> 2) & 3)) << 4));
#pragma unroll
          for (int i = 0; i < 4; ++i) chunk[i] = v[i];
        } else {
#pragma unroll
          for (int i = 0; i < 3; ++i) chunk[i] = *reinterpret_cast<const uint32_t*>(from + 768 * q + m * 48 + kq * 12 + 4 * i);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          blk[q][j] = code_block<BITS>(chunk, j);
          scs[q][j] = __float_as_uint(sc[d][q]);
          zes[q][j] = (uint32_t)ze[d][q];
        }
        transpose4(blk[q]);
        if constexpr (!WIDE) {
          transpose4(scs[q]);
          transpose4(zes[q]);
        }
      }
      floatx4 p[TG][NT], xs[TG];
#pragma unroll
      for (int u = 0; u < TG; ++u) {
        xs[u] = zero4;
#pragma unroll
        for (int q = 0; q < NT; ++q) p[u][q] = zero4;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = !TAIL || 4 * s + j < nch;
        u32x4 w[NT];
#pragma unroll
        for (int q = 0; q < NT; ++q) w[q] = code_pairs<BITS, DT>(blk[q][j], exponent);
#pragma unroll
        for (int u = 0; u < TG; ++u) {
          u32x4 x = *reinterpret_cast<const u32x4*>(from + 256 * BITS * NT + xrow[u] * 256 + (((4 * j + kq) ^ (xrow[u] & 15)) << 4));
          if (WIDE && !in) x = u32x4{0u, 0u, 0u, 0u};   // a step's last chunks
          x = pair_order(x);
          xs[u] = mfma16<DT>(x, ones, xs[u]);
#pragma unroll
          for (int q = 0; q < NT; ++q) p[u][q] = mfma16<DT>(x, w[q], p[u][q]);
        }
        if (!WIDE || j == 3) {
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            const float scale = (!TAIL || (WIDE ? 4 * s < nch : in)) ? __uint_as_float(scs[q][j]) : 0.f;
            const float off = (float)(1 << BITS) + (float)(int)zes[q][j];
#pragma unroll
            for (int u = 0; u < TG; ++u) {
#pragma unroll
              for (int e = 0; e < 4; ++e) tot[u][q][e] = __builtin_fmaf(scale, __builtin_fmaf(-off, xs[u][e], p[u][q][e]), tot[u][q][e]);
              p[u][q] = zero4;
            }
          }
#pragma unroll
          for (int u = 0; u < TG; ++u) xs[u] = zero4;
        }
      }
    }
  };
  int s0 = AHEAD * wave;
  for (; 4 * (s0 + AHEAD) <= nch; s0 += WAVES * AHEAD) run(s0, std::false_type{});
  if (s0 < steps) run(s0, std::true_type{});

  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);   // [wave][u][q][e][lane]
#pragma unroll
  for (int u = 0; u < TG; ++u)
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[(((wave * TG + u) * NT + q) * 4 + e) * 64 + lane] = tot[u][q][e];
  __syncthreads();
  // 16 TG tokens x 16 NT rows of the accumulators' layout
  for (int o = threadIdx.x; o < 256 * TG * NT; o += 64 * WAVES) {
    const int tok = o / (16 * NT), at = o % (16 * NT);
    const int l = (((tok >> 4) * NT + (at >> 4)) * 4 + (tok & 3)) * 64 + ((tok >> 2) & 3) * 16 + (at & 15);
    const int64_t t = t0 + tok;
    const int out = row0 + at;
    if (t >= a.n || out >= a.w.r) continue;
    float v = red[l];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += red[w * TG * NT * 256 + l];
    const int ad = a.S ? adapter_of(a.ad, t, a.n) : -1;
    if (ad >= 0) v += rank_dot<DT>(a.S + t * a.ad.rank, a.ad.B + ((int64_t)ad * a.w.r + out) * a.ad.rank, a.ad.rank);
    if (a.y32) store_out<0>(a.Y, t * a.ldy + out, v);
    else store_out<DT>(a.Y, t * a.ldy + out, v);
  }
}

template <int BITS, int DT, bool WIDE, int TG, int NT>
__global__ __launch_bounds__(64 * WAVES) void rows16_kernel(FwdArgs a) {
  extern __shared__ __align__(16) unsigned char rsm[];
  rows16_body<BITS, DT, WIDE, TG, NT>(a, rsm);
}

__global__ __launch_bounds__(256) void gather_columns_kernel(const uint16_t* __restrict__ X, int64_t c, int64_t ldx,
                                                             const int32_t* __restrict__ perm, uint16_t* __restrict__ dst,
                                                             int64_t items) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // eight columns of one token
  if (i >= items) return;
  const int64_t per = c >> 3, t = i / per, j = (i - t * per) * 8;
  const uint16_t* x = X + t * ldx;
  u32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int p0 = min(max(perm[j + 2 * e], 0), (int)c - 1), p1 = min(max(perm[j + 2 * e + 1], 0), (int)c - 1);
    v[e] = (uint32_t)x[p0] | ((uint32_t)x[p1] << 16);
  }
  *reinterpret_cast<u32x4*>(dst + t * c + j) = v;
}

template <int BITS, int DT, bool WIDE, int TG, int NT>
void launch_rows16(FwdArgs a, hipStream_t s) {
  constexpr int RUN = WAVES * steps_ahead(TG), JOIN = WAVES * TG * NT * 1024;   // bytes of the waves' results
  static const bool set = [] {   // once, thread-safe
    constexpr int LDS = RUN * step_bytes(BITS, NT, 4 * TG);
    (void)hipFuncSetAttribute((const void*)rows16_kernel<BITS, DT, WIDE, TG, NT>, hipFuncAttributeMaxDynamicSharedMemorySize,
                              LDS > JOIN ? LDS : JOIN);
    return true;
  }();
  (void)set;
  a.row_tiles = (a.w.r + 16 * NT - 1) / (16 * NT);
  a.quads = a.n >= 16 * TG ? 4 * TG : (int)((a.n + 3) / 4);
  const int lds = RUN * step_bytes(BITS, NT, a.quads);
  hipLaunchKernelGGL((rows16_kernel<BITS, DT, WIDE, TG, NT>), dim3((unsigned)((a.n + 16 * TG - 1) / (16 * TG) * a.row_tiles)),
                     dim3(64 * WAVES), lds > JOIN ? lds : JOIN, s, a);
}

// A workgroup at a time per CU (its LDS allows no second): as many turns as the 256
// CUs need, each of a length that grows with the workgroup's share.  Microseconds
// per 4096 columns; 48 tokens of 4096 x 4096 measured 9.6 with (3, 1), 12.9 with
// (1, 1), of 12288 x 8192 29 with (3, 3), 44 with (3, 1) and 61 with (1, 1), of
// 1024 x 4096 8.1 with (3, 1) and 5.9 with (1, 1).  (4, 3) runs out of registers, (4, 1)
// never beat (2, 2), which needs as many workgroups, nor (1, 2) and (1, 3) these.
struct RowsShape {
  int tg, nt;
  double turns;
};

RowsShape rows_shape(int64_t n, int64_t r) {
  constexpr double turn[MAX_TG][MAX_NT] = {{4.3}, {5.7, 8.4, 11.0}, {7.5, 10.2, 13.3}, {0, 12.5}};   // 0: not built
  RowsShape best{1, 1, 1e30};
  for (int tg = 1; tg <= MAX_TG; ++tg)
    for (int nt = 1; nt <= MAX_NT; ++nt) {
      if (turn[tg - 1][nt - 1] == 0) continue;
      const int64_t groups = (n + 16 * tg - 1) / (16 * tg) * ((r + 16 * nt - 1) / (16 * nt));
      const double us = turn[tg - 1][nt - 1] * (double)((groups + 255) / 256);
      if (us < best.turns) best = {tg, nt, us};
    }
  return best;
}

template <int BITS, int DT, bool WIDE>
void launch_shape(const FwdArgs& a, hipStream_t s) {
  const RowsShape p = rows_shape(a.n, a.w.r);
  switch (4 * p.tg + p.nt) {
    case 4 * 1 + 1: return launch_rows16<BITS, DT, WIDE, 1, 1>(a, s);
    case 4 * 2 + 1: return launch_rows16<BITS, DT, WIDE, 2, 1>(a, s);
    case 4 * 2 + 2: return launch_rows16<BITS, DT, WIDE, 2, 2>(a, s);
    case 4 * 2 + 3: return launch_rows16<BITS, DT, WIDE, 2, 3>(a, s);
    case 4 * 3 + 1: return launch_rows16<BITS, DT, WIDE, 3, 1>(a, s);
    case 4 * 3 + 2: return launch_rows16<BITS, DT, WIDE, 3, 2>(a, s);
    case 4 * 3 + 3: return launch_rows16<BITS, DT, WIDE, 3, 3>(a, s);
    case 4 * 4 + 2: return launch_rows16<BITS, DT, WIDE, 4, 2>(a, s);
  }
}

template <int BITS, int DT>
void launch_forward(const FwdArgs& a, hipStream_t s) {
  if (a.w.cpg % 4 == 0 || a.w.shift == 31) launch_shape<BITS, DT, true>(a, s);
  else launch_shape<BITS, DT, false>(a, s);
}

}  // namespace

bool packed_rows_fits(int64_t n, int64_t r, int64_t c) {
  const RowsShape p = rows_shape(n, r);
  return grid_fits((n + 16 * p.tg - 1) / (16 * p.tg) * ((r + 16 * p.nt - 1) / (16 * p.nt)), 64 * WAVES) &&
         grid_fits((n * (c / 8) + 255) / 256, 256);
}

double packed_rows_us(int64_t n, int64_t r, int64_t c) { return 2 + rows_shape(n, r).turns * (double)c / 4096; }

void launch_gather_columns(const void* X, int64_t n, int64_t c, int64_t ldx, const int32_t* perm, void* dst, hipStream_t s) {
  const int64_t items = n * (c >> 3);
  hipLaunchKernelGGL(gather_columns_kernel, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, s,
                     static_cast<const uint16_t*>(X), c, ldx, perm, static_cast<uint16_t*>(dst), items);
}

void launch_packed_linear(const void* X, int xt, int64_t n, int64_t ldx, const PackedLayer& w, const Adapters& ad,
                          const float* S, void* Y, int yt, int64_t ldy, hipStream_t s) {
  FwdArgs a;
  a.X = static_cast<const uint16_t*>(X);
  a.ldx = ldx;
  a.n = n;
  a.w = w;
  a.ad = ad;
  a.S = S;
  a.Y = Y;
  a.ldy = ldy;
  a.y32 = yt == 0;
#define GPTQ_FWD(B_) (xt == kBF16 ? launch_forward<B_, kBF16>(a, s) : launch_forward<B_, kF16>(a, s))
  if (w.bits == 4) GPTQ_FWD(4);
  else GPTQ_FWD(3);
#undef GPTQ_FWD
}

}  // namespace gptq
