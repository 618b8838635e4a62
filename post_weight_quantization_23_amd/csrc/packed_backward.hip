// Gradient of the packed product with respect to its input, with the adapters'
// part beside it:
//     dX[t, k] = sum_i dY[t, i] W_hat[i, k] + (T A_a)[t, k].
//
// The contraction runs over the layer's rows, along which the words are not
// contiguous and the rulers change.  So the weights are dequantized once per
// call into a transposed 16-bit copy (rows of the input columns, in original
// order), and the product runs on that: writing 2 r c bytes costs about a tenth
// of the product at 4096 tokens, and dequantizing inside the product instead
// costs more vector instructions per weight (a separate scale for each) than
// the matrix cores hide below some 256 tokens per dequantized tile.  Each
// weight is rounded once to dY's 16-bit type, as gptq_linear_forward does; for
// fp32 results it is held in as many 16-bit terms as fp32 has bits (three bf16,
// two fp16), each multiplied in turn.
#include "adapter.hpp"

namespace gptq {

namespace {

// ---------------------------------------------------------------- dequantized copy
// Wt[term][src(j)][i] = 16-bit terms of W_hat[i, j], zero for i >= r.  A thread
// takes one block of eight columns in eight consecutive rows: 256 threads are
// 64 rows x 32 blocks, whole 128-byte lines of words in and of values out (11008 x
// 4096 at 4 bits: 31 us for 113 MB, 3.6 TB/s).
template <int BITS, int DT, int TERMS>
__global__ __launch_bounds__(256) void dequant_t_kernel(PackedLayer w, uint16_t* __restrict__ Wt, int64_t kp, int64_t row_tiles) {
  const int64_t ct = blockIdx.x / row_tiles, rt = blockIdx.x - ct * row_tiles;
  const int64_t i0 = rt * 64 + 8 * (threadIdx.x & 7);
  const int gb = (int)ct * 32 + (threadIdx.x >> 3);      // block of eight columns
  if (gb * 8 >= w.c) return;
  const int g = w.group(gb >> 2);
  uint32_t blk[8];
  float sc[8], ze[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t row = i0 + e;
    blk[e] = 0u;
    sc[e] = ze[e] = 0.f;
    if (row < w.r) {
      const uint32_t* p = w.words + row * w.ldw;
      blk[e] = BITS == 4 ? p[gb] : straddling_block(p, gb);
      sc[e] = w.scales[row * w.ldg + g];
      ze[e] = (float)w.zeros[row * w.ldg + g];
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int j = 8 * gb + k;
    const int64_t col = w.perm ? min(max(w.perm[j], 0), w.c - 1) : j;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = weight32<DT>((blk[e] >> (BITS * k)) & ((1u << BITS) - 1), ze[e], sc[e]);
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[e] = pack2<DT>(v[2 * e], v[2 * e + 1]);
        if (t + 1 < TERMS) {
          v[2 * e] -= f16_to_f32<DT>(o[e] & 0xFFFFu);
          v[2 * e + 1] -= f16_to_f32<DT>(o[e] >> 16);
        }
      }
      *reinterpret_cast<u32x4*>(Wt + ((int64_t)t * w.c + col) * kp + i0) = o;
    }
  }
}

}  // namespace

bool packed_backward_fits(int64_t n, int64_t r, int64_t c) {
  const int64_t kp = gemm16_depth(r);
  return grid_fits(kp / 64 * ((c + 255) / 256), 256) && gemm16_fits(n, c, kp);
}

void launch_packed_backward(const void* dY, int xt, int64_t n, int64_t ldy, const PackedLayer& w, const Adapters& ad,
                            const uint16_t* At, const float* T, void* dX, int ot, int64_t ldx, uint16_t* Wt, uint16_t* rows,
                            float* part, hipStream_t s) {
  const int64_t kp = gemm16_depth(w.r);
  const int64_t rt = kp / 64;
  const dim3 dgrid((unsigned)(rt * ((w.c + 255) / 256)));
#define GPTQ_DEQ(B_)                                                                                                              \
  do {                                                                                                                            \
    if (xt == kBF16) {                                                                                                            \
      if (ot == 0) hipLaunchKernelGGL((dequant_t_kernel<B_, kBF16, gemm16_terms(kBF16, 0)>), dgrid, dim3(256), 0, s, w, Wt, kp, rt);                    \
      else hipLaunchKernelGGL((dequant_t_kernel<B_, kBF16, 1>), dgrid, dim3(256), 0, s, w, Wt, kp, rt);                            \
    } else {                                                                                                                      \
      if (ot == 0) hipLaunchKernelGGL((dequant_t_kernel<B_, kF16, gemm16_terms(kF16, 0)>), dgrid, dim3(256), 0, s, w, Wt, kp, rt);                     \
      else hipLaunchKernelGGL((dequant_t_kernel<B_, kF16, 1>), dgrid, dim3(256), 0, s, w, Wt, kp, rt);                             \
    }                                                                                                                             \
  } while (0)
  if (w.bits == 4) GPTQ_DEQ(4);
  else GPTQ_DEQ(3);
#undef GPTQ_DEQ
  Gemm16 a{};
  a.X = static_cast<const uint16_t*>(dY);
  a.ldx = ldy;
  a.n = n;
  if (!gemm16_takes(dY, w.r, ldy)) {
    launch_pad_rows(dY, n, w.r, ldy, nullptr, rows, s);
    a.X = rows;
    a.ldx = kp;
  }
  a.W = Wt;
  a.part = part;
  a.kp = kp;
  a.cols = w.c;
  a.ad = ad;
  a.B = At;
  a.S = T;
  a.out = dX;
  a.ldo = ldx;
  launch_gemm16(a, xt, ot, s);
}

}  // namespace gptq
