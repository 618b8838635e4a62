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
#include "adapter.hpp"

namespace gptq {

namespace {

struct FwdArgs {
  const uint16_t* X;
  int64_t ldx, n;
  PackedLayer w;
  Adapters ad;
  const float* S;    // null: no adapters
  void* Y;
  int64_t ldy;
  int row_tiles;
};

constexpr int kWaves = 8;
constexpr int kAhead = 4;   // steps of a wave whose words are requested together

// 16 MT tokens x 16 rows per workgroup.  The waves split the columns in steps
// of 128 (lane (m, kq): row m, chunk kq of the step's four) and are joined
// through LDS in wave order; each wave requests the words and rulers of four
// of its steps before it uses the first.  The lanes' blocks of codes are then
// transposed, so that product j holds chunk j alone and a row's activations are
// read in runs of 64 bytes.  There are no branches on the way: steps, tokens and
// rows past the end repeat the last ones, under a scale of zero or with results
// that are dropped (conditional loads waited for memory one after the other).
// WIDE: groups hold whole steps, so that rulers apply per step, else per chunk.
template <int BITS, int DT, int YT, int MT, bool WIDE>
__global__ __launch_bounds__(64 * kWaves) void rows16_kernel(FwdArgs a) {
  __shared__ float red[kWaves][MT][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, kq = lane >> 4;
  const int64_t tile = blockIdx.x / a.row_tiles;
  const int64_t t0 = tile * 16 * MT;
  const int row0 = (int)(blockIdx.x - tile * a.row_tiles) * 16;
  const int row = min(row0 + m, a.w.r - 1);
  const int nch = a.w.c >> 5, steps = (nch + 3) >> 2;
  const uint32_t* words = a.w.words + (int64_t)row * a.w.ldw;
  const float* srow = a.w.scales + (int64_t)row * a.w.ldg;
  const int32_t* zrow = a.w.zeros + (int64_t)row * a.w.ldg;
  const uint32_t one = DT == kBF16 ? 0x3F803F80u : 0x3C003C00u;
  const u32x4 ones = {one, one, one, one};
  const floatx4 zero4 = {0.f, 0.f, 0.f, 0.f};
  constexpr int RU = WIDE ? 1 : 4;   // rulers per step

  const uint16_t* xrow[MT];
  floatx4 tot[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    xrow[i] = a.X + min(t0 + 16 * i + m, a.n - 1) * a.ldx;
    tot[i] = zero4;
  }

  for (int s0 = wave; s0 < steps; s0 += kWaves * kAhead) {
    Chunk<BITS> cw[kAhead];
    float sc[kAhead][RU];
    int ze[kAhead][RU];
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const int s = s0 + d * kWaves;
      cw[d] = load_chunk<BITS>(words, min(4 * s + kq, nch - 1));
#pragma unroll
      for (int u = 0; u < RU; ++u) {
        const int g = min(4 * s + u, nch - 1) / a.w.cpg;
        const bool in = 4 * s + u < nch;
        const float v = srow[g];
        sc[d][u] = in ? v : 0.f;
        ze[d][u] = zrow[g];
      }
    }
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const int s = s0 + d * kWaves;
      uint32_t blk[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) blk[j] = code_block<BITS>(cw[d].w, j);
      // register j of lane (m, kq) <-> register kq of lane (m, j)
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
      swap16(blk[0], blk[1]);
      swap16(blk[2], blk[3]);
      swap32(blk[0], blk[2]);
      swap32(blk[1], blk[3]);
      floatx4 p[MT], xs[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) p[i] = xs[i] = zero4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 w = code_pairs<BITS, DT>(blk[j]);
        const bool in = 4 * s + j < nch;
        const int64_t col = 32 * (int64_t)min(4 * s + j, nch - 1) + 8 * kq;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          u32x4 x = *reinterpret_cast<const u32x4*>(xrow[i] + col);
          if (WIDE && !in) x = u32x4{0u, 0u, 0u, 0u};   // a step's last chunks (wave-uniform)
          x = pair_order(x);
          p[i] = mfma16<DT>(x, w, p[i]);
          xs[i] = mfma16<DT>(x, ones, xs[i]);
        }
        if (!WIDE || j == 3) {
          const float scale = sc[d][WIDE ? 0 : j], off = (float)(1 << BITS) + (float)ze[d][WIDE ? 0 : j];
#pragma unroll
          for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) tot[i][e] = __builtin_fmaf(scale, __builtin_fmaf(-off, xs[i][e], p[i][e]), tot[i][e]);
            p[i] = xs[i] = zero4;
          }
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][i][e][lane] = tot[i][e];
  __syncthreads();
  // an output per thread: 16 tokens x 16 rows of the accumulators' layout
#pragma unroll
  for (int o = threadIdx.x; o < 256 * MT; o += 64 * kWaves) {
    const int tok = o >> 4, i = tok >> 4, e = tok & 3, l = ((tok >> 2) & 3) * 16 + (o & 15);
    const int64_t t = t0 + tok;
    const int out = row0 + (o & 15);
    if (t >= a.n || out >= a.w.r) continue;
    float v = red[0][i][e][l];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += red[w][i][e][l];
    const int ad = a.S ? adapter_of(a.ad, t, a.n) : -1;
    if (ad >= 0) v += rank_dot<DT>(a.S + t * a.ad.rank, a.ad.B + ((int64_t)ad * a.w.r + out) * a.ad.rank, a.ad.rank);
    store_out<YT>(a.Y, t * a.ldy + out, v);
  }
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

template <int BITS, int DT, int YT, int MT>
void launch_rows16(const FwdArgs& a, hipStream_t s) {
  const int64_t tiles = (a.n + 16 * MT - 1) / (16 * MT);
  const dim3 grid((unsigned)(tiles * a.row_tiles)), block(64 * kWaves);
  if (a.w.cpg % 4 == 0 || a.w.cpg >= (a.w.c >> 5)) hipLaunchKernelGGL((rows16_kernel<BITS, DT, YT, MT, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((rows16_kernel<BITS, DT, YT, MT, false>), grid, block, 0, s, a);
}

template <int BITS, int DT, int YT>
void launch_forward(const FwdArgs& a, hipStream_t s) {
  if (a.n <= 16) launch_rows16<BITS, DT, YT, 1>(a, s);
  else if (a.n <= 32) launch_rows16<BITS, DT, YT, 2>(a, s);
  else launch_rows16<BITS, DT, YT, 4>(a, s);
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
  a.row_tiles = (w.r + 15) / 16;
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
