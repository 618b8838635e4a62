// Orthogonalised updates of low-rank factors by Newton-Schulz products.
//
// M_{k+1} = q(S_k) M_k with S_k = M_k M_k^T and q(S) = a + b S + c S^2.  All S_k and
// q(S_k) are polynomials of S_0 and so commute: S_{k+1} = S_k q(S_k)^2, and the
// long side of M is read twice only, for S_0 and for the result
// q(S_{n-1}) .. q(S_0) M_0.  An error d in S_0 grows by a^2 (11.9 for the usual
// coefficients) a step and moves singular values s near 1e-3 by 1e7 s d: 32 bits
// would leave 1e-3 there, so S_0 and the iteration are held in 64.
// Three launches: parts of S_0 over the long side, the iteration (a workgroup
// for each matrix), the result.
#include "orthogonal.hpp"

namespace gptq {

namespace {

typedef double doublex4 __attribute__((ext_vector_type(4)));

GPTQ_DEV float load_value(const void* p, int64_t at, int type) {
  if (type == 0) return static_cast<const float*>(p)[at];
  const uint16_t v = static_cast<const uint16_t*>(p)[at];
  return type == kBF16 ? f16_to_f32<kBF16>(v) : f16_to_f32<kF16>(v);
}

// Tile (i, j), i <= j, of a symmetric matrix of B x B tiles.
GPTQ_DEV int tile_index(int i, int j, int B) { return i * B - i * (i - 1) / 2 + j - i; }
GPTQ_DEV void tile_of_index(int t, int B, int& i, int& j) {
  i = 0;
  while (t >= B - i) t -= B - i++;
  j = i + t;
}

// C[4 e + (lane >> 4)][lane & 15] in component e; A[lane & 15][lane >> 4], B[lane >> 4][lane & 15].
GPTQ_DEV doublex4 mfma64(double a, double b, doublex4 c) { return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0); }

// ---------------------------------------------------------------- S_0
// A workgroup takes a run of the long side, 64 values at a time through LDS (fp32,
// the shorter side contiguous), and writes its part of every tile of G G^T.
constexpr int KS = 64, LDG = kOrthoRank + 4;

GPTQ_DEV void stage(const OrthoProblem& o, int type, int64_t mat, int64_t k0, int width, float* lds, int threads) {
  // lds[k][i] = G[i][k0 + k], zero past the matrix
  const int pp = ortho_blocks(o.p) * 16;
  for (int e = threadIdx.x; e < width * pp; e += threads) {
    int i, k;
    if (o.tall) i = e % pp, k = e / pp;
    else k = e % width, i = e / width;
    float v = 0.f;
    if (i < o.p && k0 + k < o.q)
      v = load_value(o.G, mat * o.rows * o.cols + (o.tall ? (k0 + k) * o.p + i : i * o.q + k0 + k), type);
    lds[k * LDG + i] = v;
  }
}

__global__ __launch_bounds__(256) void gram_kernel(OrthoArgs a, int type, int64_t blocks0) {
  __shared__ __align__(16) float g[KS * LDG];
  const int which = blockIdx.x >= blocks0;
  const OrthoProblem& o = a.p[which];
  const int64_t b = blockIdx.x - (which ? blocks0 : 0), mat = b / o.splits;
  const int split = (int)(b - mat * o.splits), B = ortho_blocks(o.p), tiles = ortho_tiles(o.p);
  const int64_t each = ((o.q + o.splits - 1) / o.splits + KS - 1) / KS * KS, first = split * each, last = min(o.q, first + each);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, h = lane >> 4;
  constexpr int MOST = 9;   // tiles of a wave: 36 / 4
  doublex4 acc[MOST];
  int ti[MOST], tj[MOST];
#pragma unroll
  for (int e = 0; e < MOST; ++e) {
    acc[e] = doublex4{0, 0, 0, 0};
    const int t = min(wave + 4 * e, tiles - 1);
    tile_of_index(t, B, ti[e], tj[e]);
  }
  for (int64_t k0 = first; k0 < last; k0 += KS) {
    __syncthreads();
    stage(o, type, mat, k0, KS, g, 256);
    __syncthreads();
    for (int k = 0; k < KS; k += 4) {
#pragma unroll
      for (int e = 0; e < MOST; ++e)
        if (wave + 4 * e < tiles) {
          const float* row = g + (k + h) * LDG + r;
          acc[e] = mfma64((double)row[16 * ti[e]], (double)row[16 * tj[e]], acc[e]);
        }
    }
  }
  double* part = o.part + (mat * o.splits + split) * tiles * 256;
#pragma unroll
  for (int e = 0; e < MOST; ++e)
    if (wave + 4 * e < tiles)
#pragma unroll
      for (int f = 0; f < 4; ++f) part[(wave + 4 * e) * 256 + (4 * f + h) * 16 + r] = acc[e][f];
}

// ---------------------------------------------------------------- the iteration
// Symmetric matrices as the tiles of their upper half, rows of 17 values (banks).
constexpr int TROW = 17, TSIZE = 16 * TROW;

template <int B>
GPTQ_DEV double element(const double* S, int ti, int tj, int i, int j) {
  return ti <= tj ? S[tile_index(ti, tj, B) * TSIZE + i * TROW + j] : S[tile_index(tj, ti, B) * TSIZE + j * TROW + i];
}

template <int B>
struct Chain {
  static constexpr int TILES = B * (B + 1) / 2, WAVES = TILES < 16 ? TILES : 16, MOST = (TILES + WAVES - 1) / WAVES;
  int lane, wave, r, h;
  int ti[MOST], tj[MOST];

  GPTQ_DEV void set() {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    r = lane & 15;
    h = lane >> 4;
    for (int e = 0; e < MOST; ++e) tile_of_index(min(wave + WAVES * e, TILES - 1), B, ti[e], tj[e]);
  }
  GPTQ_DEV bool has(int e) const { return wave + WAVES * e < TILES; }

  // acc = this wave's tiles of X Y (commuting, symmetric).
  GPTQ_DEV void product(const double* X, const double* Y, doublex4 (&acc)[MOST]) const {
#pragma unroll
    for (int e = 0; e < MOST; ++e) {
      acc[e] = doublex4{0, 0, 0, 0};
      if (!has(e)) continue;
      for (int tk = 0; tk < B; ++tk)
#pragma unroll
        for (int k = 0; k < 16; k += 4)
          acc[e] = mfma64(element<B>(X, ti[e], tk, r, k + h), element<B>(Y, tk, tj[e], k + h, r), acc[e]);
    }
  }
  template <class F>
  GPTQ_DEV void each(F&& f) const {
#pragma unroll
    for (int e = 0; e < MOST; ++e)
      if (has(e))
#pragma unroll
        for (int g = 0; g < 4; ++g) f(e, g, wave + WAVES * e, 4 * g + h, r);
  }
  GPTQ_DEV void write(double* X, const doublex4 (&acc)[MOST]) const {
    each([&](int e, int g, int t, int i, int j) { X[t * TSIZE + i * TROW + j] = acc[e][g]; });
  }
};

template <int B>
GPTQ_DEV void iterate(const OrthoArgs& a, const OrthoProblem& o, int64_t mat, double* lds) {
  using C = Chain<B>;
  C c;
  c.set();
  double *S = lds, *T = lds + C::TILES * TSIZE;
  __shared__ double norm;
  doublex4 acc[C::MOST], q[C::MOST];
  const double* part = o.part + mat * o.splits * C::TILES * 256;
  c.each([&](int e, int g, int t, int i, int j) {
    double v = 0;
    for (int s = 0; s < o.splits; ++s) v += part[((int64_t)s * C::TILES + t) * 256 + i * 16 + j];
    acc[e][g] = v;
  });
  c.write(S, acc);
  __syncthreads();
  if (c.wave == 0) {
    double v = 0;
    for (int i = c.lane; i < 16 * B; i += 64) v += S[tile_index(i / 16, i / 16, B) * TSIZE + (i % 16) * (TROW + 1)];
    for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
    if (c.lane == 0) {
      norm = sqrt(v) + a.eps;
      o.inv[mat] = 1.0 / norm;
    }
  }
  __syncthreads();
  const double by = 1.0 / norm;
  c.each([&](int e, int g, int t, int i, int j) { S[t * TSIZE + i * TROW + j] = acc[e][g] * by * by; });
  __syncthreads();
  double* steps = o.steps + mat * a.steps * C::TILES * 256;
  for (int k = 0; k < a.steps; ++k) {
    c.product(S, S, acc);
    // q(S) to T and to memory
    c.each([&](int e, int g, int t, int i, int j) {
      const double v = a.c * acc[e][g] + a.b * S[t * TSIZE + i * TROW + j] + (c.ti[e] == c.tj[e] && i == j ? a.a : 0.0);
      q[e][g] = v;
      T[t * TSIZE + i * TROW + j] = v;
      if (k + 1 < a.steps) steps[((int64_t)k * C::TILES + t) * 256 + i * 16 + j] = v;
    });
    __syncthreads();
    if (k + 1 == a.steps) break;
    c.product(S, T, acc);
    __syncthreads();
    c.write(S, acc);
    __syncthreads();
    c.product(S, T, acc);
    __syncthreads();
    c.write(S, acc);
    __syncthreads();
  }
  // T holds the last step's q: the earlier ones follow
  for (int k = a.steps - 2; k >= 0; --k) {
    c.each([&](int e, int g, int t, int i, int j) { S[t * TSIZE + i * TROW + j] = steps[((int64_t)k * C::TILES + t) * 256 + i * 16 + j]; });
    __syncthreads();
    c.product(T, S, acc);
    __syncthreads();
    c.write(T, acc);
    __syncthreads();
  }
  float* R = o.R + mat * (16 * B) * (16 * B);
  for (int e = threadIdx.x; e < 256 * B * B; e += 64 * C::WAVES) {
    const int i = e / (16 * B), j = e % (16 * B);
    R[e] = (float)element<B>(T, i / 16, j / 16, i % 16, j % 16);
  }
}

template <int B>
__global__ __launch_bounds__(64 * Chain<B>::WAVES) void chain_kernel(OrthoArgs a, int which) {
  extern __shared__ __align__(16) double cs[];
  iterate<B>(a, a.p[which], blockIdx.x, cs);
}

// ---------------------------------------------------------------- result
// out = R M_0 for a run of 64 values of the long side, each wave 16 of them.  The
// lanes run along the side that is contiguous in memory; R is symmetric, so either operand order
// holds it.
GPTQ_DEV floatx4 mfma_f32(float a, float b, floatx4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

GPTQ_DEV void store_value(void* p, int64_t at, float v, int type) {
  if (type == 0) static_cast<float*>(p)[at] = v;
  else static_cast<uint16_t*>(p)[at] = type == kBF16 ? f32_to_16<kBF16>(v) : f32_to_16<kF16>(v);
}

__global__ __launch_bounds__(256) void apply_kernel(OrthoArgs a, int gt, int ot, int64_t blocks0) {
  extern __shared__ __align__(16) float as[];
  const int which = blockIdx.x >= blocks0;
  const OrthoProblem& o = a.p[which];
  const int64_t runs = (o.q + KS - 1) / KS, b = blockIdx.x - (which ? blocks0 : 0), mat = b / runs, k0 = (b - mat * runs) * KS;
  const int B = ortho_blocks(o.p), pp = 16 * B, ldr = pp + 4;
  float *R = as, *g = as + pp * ldr;
  for (int e = threadIdx.x; e < pp * pp; e += 256) R[e / pp * ldr + e % pp] = o.R[mat * pp * pp + e];
  stage(o, gt, mat, k0, KS, g, 256);
  __syncthreads();
  const double inv = o.inv[mat];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, h = lane >> 4, at = 16 * wave;
  floatx4 acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < pp; k += 4) {
    const float m0 = (float)((double)g[(at + r) * LDG + k + h] * inv);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < B) {
        const float w = R[(16 * i + r) * ldr + k + h];
        acc[i] = o.tall ? mfma_f32(m0, w, acc[i]) : mfma_f32(w, m0, acc[i]);
      }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < B)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int s = o.tall ? 16 * i + r : 16 * i + 4 * h + e;          // place on the shorter side
        const int64_t l = k0 + at + (o.tall ? 4 * h + e : r);            // on the longer one
        if (s < o.p && l < o.q) store_value(o.out, mat * o.rows * o.cols + (o.tall ? l * o.p + s : s * o.q + l), acc[i][e], ot);
      }
}

template <int B>
void chain(const OrthoArgs& a, int which, hipStream_t s) {
  constexpr int LDS = 2 * Chain<B>::TILES * TSIZE * 8;
  static const bool set = [] {
    (void)hipFuncSetAttribute((const void*)chain_kernel<B>, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    return true;
  }();
  (void)set;
  hipLaunchKernelGGL(chain_kernel<B>, dim3((unsigned)a.m), dim3(64 * Chain<B>::WAVES), LDS, s, a, which);
}

}  // namespace

void launch_orthogonalize(const OrthoArgs& a, int gt, int ot, hipStream_t s) {
  int64_t gram[2] = {0, 0}, apply[2] = {0, 0};
  int most = 0;
  for (int w = 0; w < 2; ++w)
    if (a.p[w].G) {
      gram[w] = a.m * a.p[w].splits;
      apply[w] = a.m * ((a.p[w].q + KS - 1) / KS);
      most = most > a.p[w].p ? most : a.p[w].p;
    }
  hipLaunchKernelGGL(gram_kernel, dim3((unsigned)(gram[0] + gram[1])), dim3(256), 0, s, a, gt, gram[0]);
  for (int w = 0; w < 2; ++w)
    if (a.p[w].G) switch (ortho_blocks(a.p[w].p)) {
      case 1: chain<1>(a, w, s); break;
      case 2: chain<2>(a, w, s); break;
      case 3: chain<3>(a, w, s); break;
      case 4: chain<4>(a, w, s); break;
      case 5: chain<5>(a, w, s); break;
      case 6: chain<6>(a, w, s); break;
      case 7: chain<7>(a, w, s); break;
      default: chain<8>(a, w, s); break;
    }
  const int pp = 16 * ortho_blocks(most), lds = (pp * (pp + 4) + KS * LDG) * 4;
  static const bool set = [] {
    (void)hipFuncSetAttribute((const void*)apply_kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                              (kOrthoRank * (kOrthoRank + 4) + KS * LDG) * 4);
    return true;
  }();
  (void)set;
  hipLaunchKernelGGL(apply_kernel, dim3((unsigned)(apply[0] + apply[1])), dim3(256), lds, s, a, gt, ot, apply[0]);
}

int ortho_splits(int64_t m, int64_t q) {
  const int64_t runs = (q + KS - 1) / KS, want = 256 / (2 * (m > 0 ? m : 1));
  int64_t splits = want < 8 ? 8 : want;
  splits = splits < runs ? splits : runs;
  splits = splits < 64 ? splits : 64;
  return (int)(splits > 0 ? splits : 1);
}

bool ortho_fits(int64_t m, int64_t q) {
  return grid_fits(2 * m * ((q + KS - 1) / KS), 256) && grid_fits(m, 1024) && grid_fits(2 * m * 64, 256);
}

}  // namespace gptq
