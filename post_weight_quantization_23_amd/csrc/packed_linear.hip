// Product of many tokens with a packed layer, with the low-rank adapters of
// their requests beside it:
//     Y[t, i] = sum_j s[i, g(j)] (q[i, j] - z[i, g(j)]) X[t, perm[j]] + (S B_a^T)[t, i].
//
// Codes enter the matrix cores as whole numbers: a b-bit code shifted to the
// top of a 16-bit float's mantissa under the exponent of 2^b reads as 2^b + q
// exactly, one shift and one and-or for two codes.  With P = sum (2^b + q) x and
// X_g = sum x over a group (a product with ones, on the matrix cores too), the
// group's part is s (P - (2^b + z) X_g): the weights are never rounded, and
// every sum is fp32.  The subtraction costs a factor below 8 in the error of
// the fp32 sums, three bits of 24.
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
  int row_tiles;
  int quads;         // tokens of a workgroup in fours, at most four
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

// Row tiles of a workgroup, steps of a run, waves.  Two row tiles (the activations
// read once for both) leave half the CUs without work at 4096 rows (8.2 against
// 6.3 us for 16 tokens of 4096 x 4096) and gain nothing at 11008 (15.5 against
// 14.2); four waves: 8.1 and 14.9.
constexpr int NT = 1, AHEAD = 2, WAVES = 8;

// LDS bytes of a step of one wave: 16 NT rows of words, then 4 ceil(n / 4) tokens of
// 256 bytes.
constexpr int step_bytes(int bits, int nt, int quads) { return 256 * bits * nt + 1024 * quads; }

// 16 tokens x 16 NT rows per workgroup.  The waves split the columns in runs of
// AHEAD steps of 128 and are joined through LDS in wave order.
//
// What a run reads comes through the wave's own part of LDS, by loads that write
// it.  The operand layout gives consecutive lanes consecutive rows, so loading
// operands straight into registers touches 64 places of 16 bytes per
// instruction, and the L1 cache takes them one a cycle: that, not memory, set the
// pace (16 tokens of 11008 x 4096 at 3 bits: 22 us, and 40 thousand accesses
// per CU).  The loads into LDS give 4 (words) or 16 (activations) consecutive
// lanes one row.
//
// A lane then holds chunk kq of row m (lane = m + 16 kq); the blocks of codes are
// transposed, so that product j takes chunk j alone.  Steps, tokens and rows past
// the end repeat the last ones, under a scale of zero or with results that are
// dropped.  WIDE: groups hold whole steps, so that rulers apply per step;
// otherwise each lane reads its own chunk's ruler, and the transpose spreads
// them as well.
template <int BITS, int DT, int YT, bool WIDE>
GPTQ_DEV void rows16_body(const FwdArgs& a, unsigned char* smem) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, kq = lane >> 4;
  const int64_t tile = blockIdx.x / a.row_tiles;
  const int64_t t0 = tile * 16;
  const int row0 = (int)(blockIdx.x - tile * a.row_tiles) * 16 * NT;
  const int nch = a.w.c >> 5, steps = (nch + 3) >> 2;
  const float* srow[NT];
  const int32_t* zrow[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int row = min(row0 + 16 * q + m, a.w.r - 1);
    srow[q] = a.w.scales + (int64_t)row * a.w.ldg;
    zrow[q] = a.w.zeros + (int64_t)row * a.w.ldg;
  }
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
  const uint16_t* xsrc[4];
  int xpiece[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rr = 4 * i + (lane >> 4);
    xsrc[i] = a.X + min(t0 + rr, a.n - 1) * a.ldx;
    xpiece[i] = (lane & 15) ^ (rr & 15);
  }

  floatx4 tot[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) tot[q] = zero4;
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
        sc[d][q] = srow[q][g];
        ze[d][q] = zrow[q][g];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < a.quads) {
          const int piece = 16 * s + xpiece[i];
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
      floatx4 p[NT], xs = zero4;
#pragma unroll
      for (int q = 0; q < NT; ++q) p[q] = zero4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = !TAIL || 4 * s + j < nch;
        u32x4 x = *reinterpret_cast<const u32x4*>(from + 256 * BITS * NT + m * 256 + (((4 * j + kq) ^ m) << 4));
        if (WIDE && !in) x = u32x4{0u, 0u, 0u, 0u};   // a step's last chunks
        x = pair_order(x);
        xs = mfma16<DT>(x, ones, xs);
#pragma unroll
        for (int q = 0; q < NT; ++q) p[q] = mfma16<DT>(x, code_pairs<BITS, DT>(blk[q][j], exponent), p[q]);
        if (!WIDE || j == 3) {
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            const float scale = (!TAIL || (WIDE ? 4 * s < nch : in)) ? __uint_as_float(scs[q][j]) : 0.f;
            const float off = (float)(1 << BITS) + (float)(int)zes[q][j];
#pragma unroll
            for (int e = 0; e < 4; ++e) tot[q][e] = __builtin_fmaf(scale, __builtin_fmaf(-off, xs[e], p[q][e]), tot[q][e]);
            p[q] = zero4;
          }
          xs = zero4;
        }
      }
    }
  };
  int s0 = AHEAD * wave;
  for (; 4 * (s0 + AHEAD) <= nch; s0 += WAVES * AHEAD) run(s0, std::false_type{});
  if (s0 < steps) run(s0, std::true_type{});

  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);   // [wave][q][e][lane]
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[((wave * NT + q) * 4 + e) * 64 + lane] = tot[q][e];
  __syncthreads();
  // 16 tokens x 16 NT rows of the accumulators' layout
  for (int o = threadIdx.x; o < 256 * NT; o += 64 * WAVES) {
    const int tok = o / (16 * NT), at = o % (16 * NT), l = (((at >> 4) * 4) + (tok & 3)) * 64 + (tok >> 2) * 16 + (at & 15);
    const int64_t t = t0 + tok;
    const int out = row0 + at;
    if (t >= a.n || out >= a.w.r) continue;
    float v = red[l];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += red[w * NT * 256 + l];
    const int ad = a.S ? adapter_of(a.ad, t, a.n) : -1;
    if (ad >= 0) v += rank_dot<DT>(a.S + t * a.ad.rank, a.ad.B + ((int64_t)ad * a.w.r + out) * a.ad.rank, a.ad.rank);
    store_out<YT>(a.Y, t * a.ldy + out, v);
  }
}

template <int BITS, int DT, int YT, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void rows16_kernel(FwdArgs a) {
  extern __shared__ __align__(16) unsigned char rsm[];
  rows16_body<BITS, DT, YT, WIDE>(a, rsm);
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

template <int BITS, int DT, int YT, bool WIDE>
void launch_rows16(FwdArgs a, hipStream_t s) {
  constexpr int JOIN = WAVES * NT * 1024;   // bytes of the waves' results
  static const bool set = [] {   // once, thread-safe
    constexpr int LDS = WAVES * AHEAD * step_bytes(BITS, NT, 4);
    (void)hipFuncSetAttribute((const void*)rows16_kernel<BITS, DT, YT, WIDE>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, LDS > JOIN ? LDS : JOIN);
    return true;
  }();
  (void)set;
  a.row_tiles = (a.w.r + 16 * NT - 1) / (16 * NT);
  const int lds = WAVES * AHEAD * step_bytes(BITS, NT, a.quads);
  hipLaunchKernelGGL((rows16_kernel<BITS, DT, YT, WIDE>), dim3((unsigned)((a.n + 15) / 16 * a.row_tiles)),
                     dim3(64 * WAVES), lds > JOIN ? lds : JOIN, s, a);
}

template <int BITS, int DT, int YT>
void launch_forward(const FwdArgs& a, hipStream_t s) {
  if (a.w.cpg % 4 == 0 || a.w.shift == 31) launch_rows16<BITS, DT, YT, true>(a, s);
  else launch_rows16<BITS, DT, YT, false>(a, s);
}

}  // namespace

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
  a.quads = n >= 16 ? 4 : (int)((n + 3) / 4);
#define GPTQ_FWD(B_)                                                                          \
  do {                                                                                        \
    if (xt == kBF16) { if (yt == 0) launch_forward<B_, kBF16, 0>(a, s); else launch_forward<B_, kBF16, kBF16>(a, s); } \
    else { if (yt == 0) launch_forward<B_, kF16, 0>(a, s); else launch_forward<B_, kF16, kF16>(a, s); }                \
  } while (0)
  if (w.bits == 4) GPTQ_FWD(4);
  else GPTQ_FWD(3);
#undef GPTQ_FWD
}

}  // namespace gptq
