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

typedef __attribute__((address_space(3))) unsigned char lds_u8;

// ---------------------------------------------------------------- dequantized copy
// Wt[term][src(j)][i] = 16-bit terms of W_hat[i, j], zero for i >= r.  A thread
// takes one block of eight columns in eight consecutive rows: 256 threads are
// 64 rows x 32 blocks, whole 128-byte lines of words in and of values out.
template <int BITS, int DT, int TERMS>
__global__ __launch_bounds__(256) void dequant_t_kernel(PackedLayer w, uint16_t* __restrict__ Wt, int64_t kp, int64_t row_tiles) {
  const int64_t ct = blockIdx.x / row_tiles, rt = blockIdx.x - ct * row_tiles;
  const int64_t i0 = rt * 64 + 8 * (threadIdx.x & 7);
  const int gb = (int)ct * 32 + (threadIdx.x >> 3);      // block of eight columns
  if (gb * 8 >= w.c) return;
  const int g = (gb >> 2) / w.cpg;
  uint32_t blk[8];
  float sc[8], ze[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t row = i0 + e;
    blk[e] = 0u;
    sc[e] = ze[e] = 0.f;
    if (row < w.r) {
      const uint32_t* p = w.words + row * w.ldw;
      if constexpr (BITS == 4) {
        blk[e] = p[gb];
      } else {
        const uint32_t* c = p + 3 * (int64_t)(gb >> 2);
        const int bit = 24 * (gb & 3), at = bit >> 5;
        blk[e] = __builtin_amdgcn_alignbit(c[min(at + 1, 2)], c[at], bit & 31);
      }
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
    for (int e = 0; e < 8; ++e) v[e] = ((float)((blk[e] >> (BITS * k)) & ((1u << BITS) - 1)) - ze[e]) * sc[e];
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

// dst[t][0 .. kp) = src[t][0 .. d) and zeros: rows for the product where the
// given ones do not start on 16 bytes or do not end on a whole step.
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* __restrict__ src, int64_t n, int64_t d, int64_t lds, bool vec,
                                                       uint16_t* __restrict__ dst, int64_t kp) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = kp >> 3, t = i / per, k = (i - t * per) * 8;
  if (t >= n) return;
  u32x4 v = {0u, 0u, 0u, 0u};
  if (k < d) v = load8(src + t * lds + k, (int)min((int64_t)8, d - k), vec);
  *reinterpret_cast<u32x4*>(dst + t * kp + k) = v;
}

// ---------------------------------------------------------------- product
constexpr int LK = 64, ROWB = LK * 2;   // contraction step, bytes of an LDS row

struct GemmArgs16 {
  const uint16_t* X;    // [n][ldx], kp columns
  const uint16_t* W;    // [terms][cols][kp]
  int64_t n, ldx, kp;
  int cols, tok_tiles, col_tiles;
  Adapters ad;
  const uint16_t* At;   // [m][cols][rank]
  const float* T;       // null: no adapters
  void* out;
  int64_t ldo;
};

// Chunk c (16 bytes) of LDS row f lies at place c ^ swz(f).
GPTQ_DEV int swz(int f) { return (f ^ (f >> 3)) & 7; }

// WM x WN waves of 32 MT tokens x 32 NT columns.  Both operands come from
// memory straight into LDS (double buffered, one barrier per step), each lane
// fetching the chunk that belongs at its place; rows past the end lie outside
// the descriptors' records and read as zero.
template <int DT, int OT, int TERMS, int MT, int NT, int WM, int WN>
GPTQ_DEV void gemm_body(const GemmArgs16& a, unsigned char* smem) {
  constexpr int TM = 32 * MT * WM, TN = 32 * NT * WN, NW = WM * WN, BUF = (TM + TN) * ROWB;
  constexpr int QX = TM / 8 / NW, QW = TN / 8 / NW;   // load instructions per wave: 8 rows each
  static_assert(QX * 8 * NW == TM && QW * 8 * NW == TN, "tiles divide over the waves");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 31, h = lane >> 5;
  int tt, ct;
  tile_of(blockIdx.x, a.tok_tiles, a.col_tiles, tt, ct);
  const int64_t t0 = (int64_t)tt * TM;
  const int j0 = ct * TN;
  const int wm = (wave / WN) * 32 * MT, wn = (wave % WN) * 32 * NT;
  lds_u8* lbase = (lds_u8*)smem;

  int offx[QX], offw[QW];
#pragma unroll
  for (int q = 0; q < QX; ++q) {
    const int row = 8 * (wave * QX + q) + (lane >> 3);
    offx[q] = (row * (int)a.ldx + 8 * ((lane & 7) ^ swz(row))) * 2;
  }
#pragma unroll
  for (int q = 0; q < QW; ++q) {
    const int row = 8 * (wave * QW + q) + (lane >> 3);
    offw[q] = (row * (int)a.kp + 8 * ((lane & 7) ^ swz(row))) * 2;
  }
  const int xrec = (int)(min(a.n - t0, (int64_t)TM) * a.ldx * 2), wrec = (int)(min(a.cols - j0, TN) * a.kp * 2);
  const int steps = (int)(a.kp / LK), all = TERMS * steps;
  auto load = [&](int s) {
    const int term = TERMS == 1 ? 0 : s / steps, k0 = (s - term * steps) * LK;
    const __amdgpu_buffer_rsrc_t rx =
        __builtin_amdgcn_make_buffer_rsrc((void*)(a.X + t0 * a.ldx + k0), (short)0, xrec - 2 * k0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(a.W + ((int64_t)term * a.cols + j0) * a.kp + k0), (short)0, wrec - 2 * k0, 0x00020000);
    lds_u8* to = lbase + (s & 1) * BUF;
#pragma unroll
    for (int q = 0; q < QX; ++q) __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, to + (wave * QX + q) * 1024, 16, offx[q], 0, 0, 0);
#pragma unroll
    for (int q = 0; q < QW; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, to + TM * ROWB + (wave * QW + q) * 1024, 16, offw[q], 0, 0, 0);
  };

  floatx16 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int q = 0; q < NT; ++q) acc[i][q] = floatx16{};

  load(0);
  for (int s = 0; s < all; ++s) {
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

  int64_t col[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int at = j0 + wn + 32 * q + m;
    col[q] = at < a.cols ? at : -1;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t ti = t0 + wm + 32 * i;
    if (a.T) expand_add<DT, OT == 0 ? 3 : 2, NT>(a.ad, a.At, a.cols, a.T, ti, a.n, col, acc[i]);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int64_t t = ti + TileShape<floatx16>::acc_row(lane, e);
#pragma unroll
      for (int q = 0; q < NT; ++q)
        if (t < a.n && col[q] >= 0) store_out<OT>(a.out, t * a.ldo + col[q], acc[i][q][e]);
    }
  }
}

template <int DT, int OT, int TERMS, int MT, int NT, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void gemm_kernel(GemmArgs16 a) {
  extern __shared__ __align__(16) unsigned char gsm[];
  gemm_body<DT, OT, TERMS, MT, NT, WM, WN>(a, gsm);
}

template <int DT, int OT, int TERMS, int MT, int NT, int WM, int WN>
void launch_gemm(GemmArgs16 a, hipStream_t s) {
  constexpr int TM = 32 * MT * WM, TN = 32 * NT * WN, LDS = 2 * (TM + TN) * ROWB;
  static const bool set = [] {   // once, thread-safe
    (void)hipFuncSetAttribute((const void*)gemm_kernel<DT, OT, TERMS, MT, NT, WM, WN>, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    return true;
  }();
  (void)set;
  a.tok_tiles = (int)((a.n + TM - 1) / TM);
  a.col_tiles = (a.cols + TN - 1) / TN;
  hipLaunchKernelGGL((gemm_kernel<DT, OT, TERMS, MT, NT, WM, WN>), dim3((unsigned)((int64_t)a.tok_tiles * a.col_tiles)),
                     dim3(64 * WM * WN), LDS, s, a);
}

template <int DT, int OT>
void choose_gemm(const GemmArgs16& a, hipStream_t s) {
  constexpr int TERMS = backward_terms(DT, OT);
#ifdef PROBE_G
  if (PROBE_G == 0) launch_gemm<DT, OT, TERMS, 4, 2, 2, 4>(a, s);
  else if (PROBE_G == 1) launch_gemm<DT, OT, TERMS, 2, 2, 2, 2>(a, s);
  else launch_gemm<DT, OT, TERMS, 2, 1, 1, 4>(a, s);
#else
  const int64_t big = (a.n + 255) / 256 * ((a.cols + 255) / 256);
  if (big >= 192) launch_gemm<DT, OT, TERMS, 4, 2, 2, 4>(a, s);
  else launch_gemm<DT, OT, TERMS, 2, 2, 2, 2>(a, s);
#endif
}

}  // namespace

int64_t backward_depth(int64_t r) { return (r + LK - 1) / LK * LK; }

void launch_packed_backward(const void* dY, int xt, int64_t n, int64_t ldy, const PackedLayer& w, const Adapters& ad,
                            const uint16_t* At, const float* T, void* dX, int ot, int64_t ldx, uint16_t* Wt, uint16_t* rows,
                            hipStream_t s) {
  const int64_t kp = backward_depth(w.r);
  const int64_t rt = kp / 64;
  const dim3 dgrid((unsigned)(rt * ((w.c + 255) / 256)));
#define GPTQ_DEQ(B_)                                                                                                              \
  do {                                                                                                                            \
    if (xt == kBF16) {                                                                                                            \
      if (ot == 0) hipLaunchKernelGGL((dequant_t_kernel<B_, kBF16, 3>), dgrid, dim3(256), 0, s, w, Wt, kp, rt);                    \
      else hipLaunchKernelGGL((dequant_t_kernel<B_, kBF16, 1>), dgrid, dim3(256), 0, s, w, Wt, kp, rt);                            \
    } else {                                                                                                                      \
      if (ot == 0) hipLaunchKernelGGL((dequant_t_kernel<B_, kF16, 2>), dgrid, dim3(256), 0, s, w, Wt, kp, rt);                     \
      else hipLaunchKernelGGL((dequant_t_kernel<B_, kF16, 1>), dgrid, dim3(256), 0, s, w, Wt, kp, rt);                             \
    }                                                                                                                             \
  } while (0)
  if (w.bits == 4) GPTQ_DEQ(4);
  else GPTQ_DEQ(3);
#undef GPTQ_DEQ
  GemmArgs16 a{};
  a.X = static_cast<const uint16_t*>(dY);
  a.ldx = ldy;
  a.n = n;
  const bool vec = reinterpret_cast<uintptr_t>(dY) % 16 == 0 && ldy % 8 == 0;
  if (!vec || w.r % LK != 0 || ldy >= (int64_t(1) << 22)) {
    hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)((n * (kp / 8) + 255) / 256)), dim3(256), 0, s, a.X, n, (int64_t)w.r, ldy, vec,
                       rows, kp);
    a.X = rows;
    a.ldx = kp;
  }
  a.W = Wt;
  a.kp = kp;
  a.cols = w.c;
  a.ad = ad;
  a.At = At;
  a.T = T;
  a.out = dX;
  a.ldo = ldx;
  if (xt == kBF16) { if (ot == 0) choose_gemm<kBF16, 0>(a, s); else choose_gemm<kBF16, kBF16>(a, s); }
  else { if (ot == 0) choose_gemm<kF16, 0>(a, s); else choose_gemm<kF16, kF16>(a, s); }
}

}  // namespace gptq
