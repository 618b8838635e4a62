// Gradient of the packed product with respect to its input, with the adapters'
// part beside it:
//     dX[t, perm[j]] = sum_i dY[t, i] s[i, g(j)] (q[i, j] - z[i, g(j)]) + (T A_a)[t, perm[j]].
//
// The contraction runs over the layer's rows, along which the words are not
// contiguous and the rulers change, so the weights are dequantized on the way
// into LDS: a thread reads one block of eight codes in several consecutive
// rows and writes each column's values of those rows side by side, which is
// the transpose.  Each weight is rounded once to dY's 16-bit type, as
// gptq_linear_forward does; for fp32 results it enters as two 16-bit terms.
// Sums are fp32.  Workgroup: 64 MW tokens x 128 packed columns, 64 rows a
// step; 2 MW waves of 64 x 64.
#include "adapter.hpp"

namespace gptq {

namespace {

constexpr int TN = 128, TK = 64, ROWB = TK * 2;   // columns, contraction step, bytes of an LDS row

struct BwdArgs {
  const uint16_t* dY;
  int64_t ldy, n;
  bool vec;
  PackedLayer w;
  Adapters ad;
  const uint16_t* At;   // [m][c][rank]
  const float* T;       // null: no adapters
  void* dX;
  int64_t ldx;
  int col_tiles;
};

// 16-byte chunks of an LDS row are permuted by the row, so that 16 rows read
// at one position spread over the banks.
GPTQ_DEV int lds_at(int row, int k) { return row * ROWB + ((((k >> 3) ^ row ^ (row >> 3)) & 7) << 4) + (k & 7) * 2; }

template <int BITS, int DT, int OT, int MW>
__global__ __launch_bounds__(128 * MW) void backward_kernel(BwdArgs a) {
  constexpr int TM = 64 * MW, THREADS = 128 * MW;
  constexpr bool SPLIT = OT == 0;
  constexpr int RP = TK * (TN / 8) / THREADS;    // rows of one block per thread
  constexpr int AP = TM * (TK / 8) / THREADS;    // 16-byte chunks of dY per thread
  __shared__ __align__(16) unsigned char As[TM * ROWB];
  __shared__ __align__(16) unsigned char Ws[(SPLIT ? 2 : 1) * TN * ROWB];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, kq = lane >> 4;
  const int64_t tile = blockIdx.x / a.col_tiles;
  const int64_t t0 = tile * TM;
  const int j0 = (int)(blockIdx.x - tile * a.col_tiles) * TN;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  const int r = a.w.r;

  // this thread's block of eight codes, and its rows within a step
  const int b = tid & 15, i0 = (tid >> 4) * RP;
  const int gb = (j0 >> 3) + b;
  const bool in = gb * 8 < a.w.c;
  const int group = in ? (gb >> 2) / a.w.cpg : 0;

  u32x4 av[AP];
  uint32_t blk[RP];
  float sc[RP], ze[RP];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int c = 0; c < AP; ++c) {
      const int at = tid + c * THREADS;
      const int64_t t = t0 + (at >> 3);
      const int k = k0 + (at & 7) * 8;
      av[c] = t < a.n ? load8(a.dY + t * a.ldy + k, r - k, a.vec) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < RP; ++i) {
      const int row = k0 + i0 + i;
      blk[i] = 0u;
      sc[i] = ze[i] = 0.f;
      if (in && row < r) {
        const uint32_t* w = a.w.words + (int64_t)row * a.w.ldw;
        if constexpr (BITS == 4) {
          blk[i] = w[gb];
        } else {
          const uint32_t* c = w + 3 * (int64_t)(gb >> 2);
          const int bit = 24 * (gb & 3), at = bit >> 5;
          blk[i] = __builtin_amdgcn_alignbit(c[min(at + 1, 2)], c[at], bit & 31);
        }
        sc[i] = a.w.scales[(int64_t)row * a.w.ldg + group];
        ze[i] = (float)a.w.zeros[(int64_t)row * a.w.ldg + group];
      }
    }
  };
  auto stage = [&]() {
#pragma unroll
    for (int c = 0; c < AP; ++c) {
      const int at = tid + c * THREADS;
      *reinterpret_cast<u32x4*>(As + lds_at(at >> 3, (at & 7) * 8)) = av[c];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t hi[RP / 2], lo[RP / 2];
#pragma unroll
      for (int i = 0; i < RP / 2; ++i) {
        const float w0 = ((float)((blk[2 * i] >> (BITS * e)) & ((1u << BITS) - 1)) - ze[2 * i]) * sc[2 * i];
        const float w1 = ((float)((blk[2 * i + 1] >> (BITS * e)) & ((1u << BITS) - 1)) - ze[2 * i + 1]) * sc[2 * i + 1];
        hi[i] = pack2<DT>(w0, w1);
        if constexpr (SPLIT) lo[i] = pack2<DT>(w0 - f16_to_f32<DT>(hi[i] & 0xFFFFu), w1 - f16_to_f32<DT>(hi[i] >> 16));
      }
      unsigned char* at = Ws + lds_at(8 * b + e, i0);
      if constexpr (RP == 2) {
        *reinterpret_cast<uint32_t*>(at) = hi[0];
        if constexpr (SPLIT) *reinterpret_cast<uint32_t*>(at + TN * ROWB) = lo[0];
      } else {
        *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
        if constexpr (SPLIT) *reinterpret_cast<uint2*>(at + TN * ROWB) = make_uint2(lo[0], lo[1]);
      }
    }
  };

  floatx4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  fetch(0);
  for (int k0 = 0; k0 < r; k0 += TK) {
    __syncthreads();
    stage();
    __syncthreads();
    if (k0 + TK < r) fetch(k0 + TK);
#pragma unroll
    for (int k = 0; k < TK; k += 32) {
      u32x4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const u32x4*>(As + lds_at(wm + 16 * i + m, k + 8 * kq));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned char* at = Ws + lds_at(wn + 16 * j + m, k + 8 * kq);
        const u32x4 w = *reinterpret_cast<const u32x4*>(at);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = mfma16<DT>(x[i], w, acc[i][j]);
        if constexpr (SPLIT) {
          const u32x4 wl = *reinterpret_cast<const u32x4*>(at + TN * ROWB);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i][j] = mfma16<DT>(x[i], wl, acc[i][j]);
        }
      }
    }
  }

  int64_t col[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int p = j0 + wn + 16 * j + m;
    col[j] = p >= a.w.c ? -1 : (a.w.perm ? min(max(a.w.perm[p], 0), a.w.c - 1) : p);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t ti = t0 + wm + 16 * i;
    if (a.T) expand_add<DT, OT == 0 ? 3 : 2, 4>(a.ad, a.At, a.w.c, a.T, ti, a.n, col, acc[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t t = ti + 4 * kq + e;
        if (t < a.n && col[j] >= 0) store_out<OT>(a.dX, t * a.ldx + col[j], acc[i][j][e]);
      }
  }
}

}  // namespace

void launch_packed_backward(const void* dY, int xt, int64_t n, int64_t ldy, const PackedLayer& w, const Adapters& ad,
                            const uint16_t* At, const float* T, void* dX, int ot, int64_t ldx, hipStream_t s) {
  BwdArgs a;
  a.dY = static_cast<const uint16_t*>(dY);
  a.ldy = ldy;
  a.n = n;
  a.vec = reinterpret_cast<uintptr_t>(dY) % 16 == 0 && ldy % 8 == 0;
  a.w = w;
  a.ad = ad;
  a.At = At;
  a.T = T;
  a.dX = dX;
  a.ldx = ldx;
  a.col_tiles = (w.c + TN - 1) / TN;
  const dim3 grid((unsigned)((n + 127) / 128 * a.col_tiles)), block(256);
#define GPTQ_BWD(B_, D_)                                                                   \
  do {                                                                                     \
    if (ot == 0) hipLaunchKernelGGL((backward_kernel<B_, D_, 0, 2>), grid, block, 0, s, a); \
    else hipLaunchKernelGGL((backward_kernel<B_, D_, D_, 2>), grid, block, 0, s, a);       \
  } while (0)
  if (w.bits == 4) { if (xt == kBF16) GPTQ_BWD(4, kBF16); else GPTQ_BWD(4, kF16); }
  else { if (xt == kBF16) GPTQ_BWD(3, kBF16); else GPTQ_BWD(3, kF16); }
#undef GPTQ_BWD
}

}  // namespace gptq
