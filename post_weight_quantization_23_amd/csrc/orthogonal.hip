// Orthogonalised updates of low-rank factors by Newton-Schulz products.
//
// M_{k+1} = q(S_k) M_k with S_k = M_k M_k^T and q(S) = a + b S + c S^2.  All S_k and
// q(S_k) are polynomials of S_0 and so commute: S_{k+1} = S_k q(S_k)^2, and the
// long side of M is read twice only, for S_0 and for the result
// q(S_{n-1}) .. q(S_0) M_0.  An error d in S_0 grows by a^2 (11.9 for the usual
// coefficients) a step and moves singular values s near 1e-3 by 1e7 s d: 32 bits
// would leave 1e-3 there, so S_0 and the iteration are held in 64.  So are R = q .. q, which is
// a^n where M has no part, and its product with M_0, where those parts have to cancel
// (five steps of a row repeated 128 times: off by 4e-4 with R and the product in 32 bits).
// Rounding leaves eigenvalues of S_0 near -1e-17 where they are zero, and below zero
// nothing bounds s q(s)^2 (16 steps of such a matrix: values of 1e7).  After as many steps as
// a^2 may multiply up to 2^16 (five) S is therefore formed again, from M = R M_0, run by
// run of the long side, and is positive again but for rounding of its own.
// Launches: parts of S_0 over the long side, the iteration, the result.  Up to 64 rows a
// workgroup iterates a matrix by itself; above that (more 64-bit products than one
// CU is quick at) a launch takes a step of all matrices on many.  An adapter of rank
// 16 beside 4096 x 4096 takes 19 us, five of rank 64 beside 11008 x 4096 87 us (S_0
// 18, iteration 45, result 24), eight of rank 128 262 us (62, 108 in six launches, 94).
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

// ---------------------------------------------------------------- a run of the long side in LDS
// KS values of the long side in fp32, zeros past the matrix: rows of the shorter side
// (KS values and padding), or of the longer one where that is how they lie in memory.
// The paddings keep the lanes of a read, which run along one side and
// four values of the other, in different banks.
constexpr int KS = 64;

template <int B, bool TALL>
struct Run {
  static constexpr int PP = 16 * B;
  // gram: lanes along the shorter side; apply: along the longer one
  static constexpr int GRAM = TALL ? 16 * (B | 1) : KS + 4, APPLY = TALL ? PP + 4 : KS + 16;
  static constexpr int ROWS = TALL ? KS : PP;
  static constexpr int FLOATS = ROWS * (GRAM > APPLY ? GRAM : APPLY);
  static constexpr int PER = PP * KS / 4;   // fours of values

  // Four values of thread's place v of a run: of short row s from long k, or the reverse.
  static GPTQ_DEV floatx4 fetch(const OrthoProblem& o, int type, int64_t mat, int64_t k0, int v) {
    const int row = TALL ? v / (PP / 4) : v / (KS / 4), col = 4 * (TALL ? v % (PP / 4) : v % (KS / 4));
    const int64_t r = TALL ? k0 + row : row, c = TALL ? col : k0 + col;
    floatx4 x = {0.f, 0.f, 0.f, 0.f};
    if (r >= o.rows || c >= o.cols) return x;
    const int64_t at = mat * o.rows * o.cols + r * o.cols + c;
    if (o.vec) {
      if (type == 0) return *reinterpret_cast<const floatx4*>(static_cast<const float*>(o.G) + at);
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(o.G) + at);
      const uint32_t u[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = type == kBF16 ? f16_to_f32<kBF16>(u[e]) : f16_to_f32<kF16>(u[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < o.cols) x[e] = load_value(o.G, at + e, type);
    }
    return x;
  }
  static GPTQ_DEV void put(float* lds, int stride, int v, floatx4 x) {
    const int row = TALL ? v / (PP / 4) : v / (KS / 4), col = 4 * (TALL ? v % (PP / 4) : v % (KS / 4));
    *reinterpret_cast<floatx4*>(lds + row * stride + col) = x;
  }
  static GPTQ_DEV float get(const float* lds, int stride, int s, int l) { return TALL ? lds[l * stride + s] : lds[s * stride + l]; }
};

// ---------------------------------------------------------------- S_0
// Parts of G G^T over the long side; 64-bit products bound it (rank 128: its operations take 33 us
// at 67 TFLOP/s, the kernel 62).  A wave holds tile rows i and B-1-i of the upper
// half, B+1 tiles whatever i is, so a fragment of the run serves several products;
// the waves with the same rows share the run's values out among them and
// are added up through LDS in their order.
// AGAIN: of R G / |G| instead, of which each run is made in LDS first.
constexpr int GRAM_THREADS = 512;
constexpr int MADE = KS + 4;   // values of a row of it (banks)

template <int B, bool TALL, bool AGAIN>
GPTQ_DEV void gram(const OrthoProblem& o, int type, int64_t mat, int split, float* lds) {
  using R = Run<B, TALL>;
  constexpr int PAIRS = (B + 1) / 2, SHARE = GRAM_THREADS / 64 / PAIRS, TILES = ortho_tiles(16 * B);
  constexpr int LD = (R::PER + GRAM_THREADS - 1) / GRAM_THREADS;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, h = lane >> 4;
  const int pair = wave % PAIRS, share = wave / PAIRS, i0 = pair, i1 = B - 1 - pair;
  const int64_t run = ((o.q + KS - 1) / KS + o.splits - 1) / o.splits * KS, first = split * run, last = min(o.q, first + run);
  doublex4 up[B], low[B];
#pragma unroll
  for (int t = 0; t < B; ++t) up[t] = low[t] = doublex4{0, 0, 0, 0};
  floatx4 next[LD];
  double* made = reinterpret_cast<double*>(lds + R::FLOATS);   // [16 B][MADE]
  static_assert(R::FLOATS % 2 == 0, "64-bit values behind the run");
  auto value = [&](int s, int l) { return AGAIN ? made[s * MADE + l] : (double)R::get(lds, R::GRAM, s, l); };
  auto fetch = [&](int64_t k0) {
#pragma unroll
    for (int e = 0; e < LD; ++e)
      if (threadIdx.x + GRAM_THREADS * e < R::PER) next[e] = R::fetch(o, type, mat, k0, threadIdx.x + GRAM_THREADS * e);
  };
  if (first < last) fetch(first);
  for (int64_t k0 = first; k0 < last; k0 += KS) {
    __syncthreads();   // the last run has been read
#pragma unroll
    for (int e = 0; e < LD; ++e)
      if (threadIdx.x + GRAM_THREADS * e < R::PER) R::put(lds, R::GRAM, threadIdx.x + GRAM_THREADS * e, next[e]);
    __syncthreads();
    if (k0 + KS < last) fetch(k0 + KS);
    if constexpr (AGAIN) {
      const double *by = o.R + mat * o.apart, inv = o.inv[mat];
      for (int t = wave; t < B * (KS / 16); t += GRAM_THREADS / 64) {
        const int i = 16 * (t / (KS / 16)), j = 16 * (t % (KS / 16));
        doublex4 v = {0, 0, 0, 0};
        for (int k = 0; k < 16 * B; k += 4) v = mfma64(by[(k + h) * 16 * B + i + r], (double)R::get(lds, R::GRAM, k + h, j + r), v);
#pragma unroll
        for (int e = 0; e < 4; ++e) made[(i + 4 * e + h) * MADE + j + r] = v[e] * inv;
      }
      __syncthreads();
    }
    if (share >= SHARE) continue;
    for (int k1 = 0; k1 < KS; k1 += 4 * SHARE) {
      const int k = k1 + 4 * share;
      const double a0 = value(16 * i0 + r, k + h), a1 = value(16 * i1 + r, k + h);
#pragma unroll
      for (int t = 0; t < B; ++t)
        if (t >= i0) {
          const double b = value(16 * t + r, k + h);
          up[t] = mfma64(a0, b, up[t]);
          if (t >= i1 && i1 != i0) low[t] = mfma64(a1, b, low[t]);
        }
    }
  }
  double* sum = reinterpret_cast<double*>(lds);
  auto each = [&](auto&& f) {
#pragma unroll
    for (int t = 0; t < B; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (t >= i0) up[t][e] = f(up[t][e], tile_index(i0, t, B) * 256 + (4 * e + h) * 16 + r);
        if (t >= i1 && i1 != i0) low[t][e] = f(low[t][e], tile_index(i1, t, B) * 256 + (4 * e + h) * 16 + r);
      }
  };
  for (int w = 1; w < SHARE; ++w) {
    __syncthreads();
    if (share == w) each([&](double v, int at) { return sum[at] = v; });
    __syncthreads();
    if (share == 0) each([&](double v, int at) { return v + sum[at]; });
  }
  double* part = o.part + (mat * o.splits + split) * TILES * 256;
  if (share == 0) each([&](double v, int at) { return part[at] = v; });
}

template <int B, bool AGAIN>
__global__ __launch_bounds__(GRAM_THREADS) void gram_kernel(OrthoArgs a, int which, int type, int64_t blocks0) {
  constexpr int RUN = (Run<B, true>::FLOATS > Run<B, false>::FLOATS ? Run<B, true>::FLOATS : Run<B, false>::FLOATS) + (AGAIN ? 2 * 16 * B * MADE : 0);
  constexpr int SUM = 512 * ortho_tiles(16 * B);
  __shared__ __align__(16) float lds[RUN > SUM ? RUN : SUM];
  int64_t b = blockIdx.x;
  if (b >= blocks0) b -= blocks0, which = 1;
  const OrthoProblem& o = a.p[which];
  const int64_t mat = b / o.splits;
  const int split = (int)(b - mat * o.splits);
  if (o.tall) gram<B, true, AGAIN>(o, type, mat, split, lds);
  else gram<B, false, AGAIN>(o, type, mat, split, lds);
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
  static constexpr int THREADS = WAVES < 8 ? 512 : 64 * WAVES;   // all of them read the parts of S_0
  int lane, wave, r, h;
  int ti[MOST], tj[MOST];

  GPTQ_DEV void set() {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    r = lane & 15;
    h = lane >> 4;
#pragma unroll
    for (int e = 0; e < MOST; ++e) tile_of_index(min(wave + WAVES * e, TILES - 1), B, ti[e], tj[e]);
  }
  GPTQ_DEV bool has(int e) const { return wave < WAVES && wave + WAVES * e < TILES; }

  // acc = this wave's tiles of X Y (commuting, symmetric).
  GPTQ_DEV void product(const double* X, const double* Y, doublex4 (&acc)[MOST]) const {
#pragma unroll
    for (int e = 0; e < MOST; ++e) acc[e] = doublex4{0, 0, 0, 0};
    if (wave >= WAVES) return;
    for (int tk = 0; tk < B; ++tk) {
      double x[MOST][4], y[MOST][4];
#pragma unroll
      for (int e = 0; e < MOST; ++e) {
        const bool xu = ti[e] <= tk, yu = tk <= tj[e];   // which half holds the tile
        const double* xt = X + (xu ? tile_index(ti[e], tk, B) : tile_index(tk, ti[e], B)) * TSIZE + r * (xu ? TROW : 1) + h * (xu ? 1 : TROW);
        const double* yt = Y + (yu ? tile_index(tk, tj[e], B) : tile_index(tj[e], tk, B)) * TSIZE + r * (yu ? 1 : TROW) + h * (yu ? TROW : 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[e][k] = xt[4 * k * (xu ? 1 : TROW)];
          y[e][k] = yt[4 * k * (yu ? TROW : 1)];
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < MOST; ++e)
          if (has(e)) acc[e] = mfma64(x[e][k], y[e][k], acc[e]);
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
  constexpr int N = C::TILES * 256, GROUPS = C::THREADS / N > 0 ? C::THREADS / N : 1;
  C c;
  c.set();
  double *S = lds, *T = S + C::TILES * TSIZE, *R = T + C::TILES * TSIZE;   // R: the product of the steps so far
  __shared__ double norm, sums[GROUPS > 1 ? GROUPS * N : 1];
  // the parts of S_0, in their order
  const int parts = o.splits;
  const double* part = o.part + mat * parts * N;
  for (int e = threadIdx.x; e < N * GROUPS; e += C::THREADS) {
    const int at = e % N, group = e / N, each = (parts + GROUPS - 1) / GROUPS, last = min(parts, (group + 1) * each);
    double v = 0;
#pragma unroll 8
    for (int s = group * each; s < last; ++s) v += part[(int64_t)s * N + at];
    if constexpr (GROUPS > 1) sums[e] = v;
    else S[at / 256 * TSIZE + at % 256 / 16 * TROW + at % 16] = v;
  }
  __syncthreads();
  if constexpr (GROUPS > 1) {
    for (int e = threadIdx.x; e < N; e += C::THREADS) {
      double v = 0;
      for (int g = 0; g < GROUPS; ++g) v += sums[g * N + e];
      S[e / 256 * TSIZE + e % 256 / 16 * TROW + e % 16] = v;
    }
    __syncthreads();
  }
  if (c.wave == 0) {
    double v = 0;
    for (int i = c.lane; i < 16 * B; i += 64) v += S[tile_index(i / 16, i / 16, B) * TSIZE + (i % 16) * (TROW + 1)];
    for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
    if (c.lane == 0) {
      norm = a.first ? 1.0 / (sqrt(v) + a.eps) : 1.0;
      if (a.first) o.inv[mat] = norm;
    }
  }
  __syncthreads();
  const double by = norm;
  for (int e = threadIdx.x; e < C::TILES * TSIZE; e += C::THREADS) S[e] = S[e] * by * by;
  __syncthreads();
  doublex4 acc[C::MOST], more[C::MOST];
  for (int k = 0; k < a.steps; ++k) {
    c.product(S, S, acc);
    // q(S)
    c.each([&](int e, int g, int t, int i, int j) {
      const double v = a.c * acc[e][g] + a.b * S[t * TSIZE + i * TROW + j] + (c.ti[e] == c.tj[e] && i == j ? a.a : 0.0);
      T[t * TSIZE + i * TROW + j] = v;
      if (k == 0) R[t * TSIZE + i * TROW + j] = v;
    });
    __syncthreads();
    const bool on = k + 1 < a.steps;
    if (on) c.product(S, T, acc);
    if (k > 0) c.product(T, R, more);
    __syncthreads();
    if (on) c.write(S, acc);
    if (k > 0) c.write(R, more);
    __syncthreads();
    if (!on) break;
    c.product(S, T, acc);
    __syncthreads();
    c.write(S, acc);
    __syncthreads();
  }
  double* all = o.R + mat * o.apart;
  if (a.first) {
    for (int e = threadIdx.x; e < 256 * B * B; e += C::THREADS) {
      const int i = e / (16 * B), j = e % (16 * B);
      all[e] = element<B>(R, i / 16, j / 16, i % 16, j % 16);
    }
    return;
  }
  // times the product of the steps before, which was formed of another S and so does not commute
  constexpr int MORE = (B * B + C::THREADS / 64 - 1) / (C::THREADS / 64);
  doublex4 total[MORE];
#pragma unroll
  for (int e = 0; e < MORE; ++e) {
    const int t = min(c.wave + C::THREADS / 64 * e, B * B - 1), i = t / B, j = t % B;
    total[e] = doublex4{0, 0, 0, 0};
    for (int k = 0; k < 16 * B; k += 4)
      total[e] = mfma64(element<B>(R, i, k / 16, c.r, k % 16 + c.h), all[(16 * j + c.r) * 16 * B + k + c.h], total[e]);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < MORE; ++e) {
    const int t = c.wave + C::THREADS / 64 * e, i = t / B, j = t % B;
    if (t < B * B)
#pragma unroll
      for (int g = 0; g < 4; ++g) all[(16 * j + c.r) * 16 * B + 16 * i + 4 * g + c.h] = total[e][g];
  }
}

template <int B>
__global__ __launch_bounds__(Chain<B>::THREADS) void chain_kernel(OrthoArgs a, int which) {
  __shared__ __align__(16) double cs[3 * Chain<B>::TILES * TSIZE];
  int64_t mat = blockIdx.x;
  if (mat >= a.m) mat -= a.m, which = 1;
  iterate<B>(a, a.p[which], mat, cs);
}

// ---------------------------------------------------------------- the iteration, over many CUs
// Matrices of more than 64 rows: a launch for each step, a workgroup for 16 rows of S_k
// and a wave for each of its tiles.  With all polynomials of S commuting, rows of
// what a step needs come from the same rows and S alone:
//   U = S S, Q = a + b S + c U, T = Q S, V = T S, S' = T Q = a T + b V + c V S, R' = Q R
// so a wave keeps its 16 columns of S (rows, S being symmetric) and R (held transposed) in registers and
// only rows pass through LDS.  (One workgroup with the matrix in LDS: 254 us for 16 matrices
// of 128, these six launches 108.  A launch for each of 14 products made the call of eight adapters
// 17 us longer.)
struct WideArgs {
  double a, b, c;
  int64_t m;               // matrices of the first problem
  int64_t size;            // values of a matrix's buffers
  double* base[2];         // of either problem
  int s, s1, r, r1;        // buffers: S, S', R, R'
  bool first, last;        // R is the identity; no S' is wanted
  bool again;              // R holds steps of an S formed before, and does not commute with this one
};
enum { kS0, kS1, kR0, kR1, kWideBuffers };   // ortho_wide's four

template <int B>
__global__ __launch_bounds__(64 * B) void wide_kernel(WideArgs a) {
  constexpr int PP = 16 * B, LD = PP + 2;
  __shared__ __align__(16) double rows[16 * LD];
  const int lane = threadIdx.x & 63, tj = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, h = lane >> 4, ti = blockIdx.y;
  int64_t mat = blockIdx.x;
  const int side = mat >= a.m;
  if (side) mat -= a.m;
  double* own = a.base[side] + mat * a.size;
  const double *S = own + a.s * PP * PP, *R = own + a.r * PP * PP;
  // of eight values of the contraction a lane has two
  double2 s[2 * B], rr[2 * B];
#pragma unroll
  for (int k = 0; k < 2 * B; ++k) s[k] = *reinterpret_cast<const double2*>(S + (16 * tj + r) * PP + 8 * k + 2 * h);
  if (!a.first)
#pragma unroll
    for (int k = 0; k < 2 * B; ++k) rr[k] = *reinterpret_cast<const double2*>(R + (16 * tj + r) * PP + 8 * k + 2 * h);
  auto put = [&](const doublex4& v) {
    __syncthreads();   // the rows before have been read
#pragma unroll
    for (int e = 0; e < 4; ++e) rows[(4 * e + h) * LD + 16 * tj + r] = v[e];
    __syncthreads();
  };
  auto product = [&](const double2 (&y)[2 * B]) {
    doublex4 acc[2] = {};
#pragma unroll
    for (int k = 0; k < 2 * B; ++k) {
      const double2 x = *reinterpret_cast<const double2*>(rows + r * LD + 8 * k + 2 * h);
      acc[0] = mfma64(x.x, y[k].x, acc[0]);
      acc[1] = mfma64(x.y, y[k].y, acc[1]);
    }
    return acc[0] + acc[1];
  };
  auto write = [&](int buffer, const doublex4& v) {
    double* to = own + buffer * PP * PP;
#pragma unroll
    for (int e = 0; e < 4; ++e) to[(16 * ti + 4 * e + h) * PP + 16 * tj + r] = v[e];
  };
  doublex4 q;
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = S[(16 * ti + 4 * e + h) * PP + 16 * tj + r];
  put(q);
  q = a.b * q + a.c * product(s);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (ti == tj && 4 * e + h == r) q[e] += a.a;
  if (!a.first || !a.last) put(q);
  const doublex4 next = a.first ? q : product(rr);
  if (a.again) {
    double* to = own + a.r1 * PP * PP;
#pragma unroll
    for (int e = 0; e < 4; ++e) to[(16 * tj + r) * PP + 16 * ti + 4 * e + h] = next[e];
  } else {
    write(a.r1, next);
  }
  if (a.last) return;
  const doublex4 t = product(s);
  put(t);
  const doublex4 v = product(s);
  put(v);
  write(a.s1, a.a * t + a.b * v + a.c * product(s));
}

// S_0 / |G|^2 from its parts: a workgroup for each tile, each with the trace of all of them.
template <int B>
__global__ __launch_bounds__(256) void wide_start_kernel(OrthoArgs a, int which, WideArgs w) {
  constexpr int PP = 16 * B, N = ortho_tiles(PP) * 256;
  __shared__ double sums[4];
  int64_t mat = blockIdx.x;
  const int side = mat >= w.m;
  if (side) mat -= w.m, which = 1;
  const OrthoProblem& o = a.p[which];
  const double* part = o.part + mat * o.splits * N;
  const int tid = threadIdx.x, t = blockIdx.y;
  auto sum = [&](int at) {
    double v = 0;
#pragma unroll 8
    for (int s = 0; s < o.splits; ++s) v += part[(int64_t)s * N + at];
    return v;
  };
  double v = tid < PP ? sum(tile_index(tid / 16, tid / 16, B) * 256 + tid % 16 * 17) : 0;
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  if ((tid & 63) == 0) sums[tid >> 6] = v;
  const double mine = sum(t * 256 + tid);
  __syncthreads();
  const double by = a.first ? 1.0 / (sqrt(sums[0] + sums[1] + sums[2] + sums[3]) + a.eps) : 1.0;
  if (a.first && t == 0 && tid == 0) o.inv[mat] = by;
  int ti, tj;
  tile_of_index(t, B, ti, tj);
  double* S = w.base[side] + mat * w.size + (int64_t)kS0 * PP * PP;
  const int i = 16 * ti + tid / 16, j = 16 * tj + tid % 16;
  if (ti < tj || i <= j) S[i * PP + j] = S[j * PP + i] = mine * by * by;
}

// a.steps steps; R of the problems is in buffer `held`, before and after.
template <int B>
void wide(OrthoArgs& a, int which, bool both, int& held, hipStream_t s) {
  constexpr int PP = 16 * B, TILES = ortho_tiles(PP);
  WideArgs w{};
  w.a = a.a;
  w.b = a.b;
  w.c = a.c;
  w.m = a.m;
  w.size = (int64_t)kWideBuffers * PP * PP;
  for (int k = 0; k <= (both ? 1 : 0); ++k) w.base[k] = a.p[which + k].wide;
  const int64_t mats = both ? 2 * a.m : a.m;
  hipLaunchKernelGGL(wide_start_kernel<B>, dim3((unsigned)mats, TILES), dim3(256), 0, s, a, which, w);
  for (int k = 0; k < a.steps; ++k) {
    w.first = a.first && k == 0;
    w.again = !a.first;
    w.last = k + 1 == a.steps;
    w.s = k % 2 ? kS1 : kS0;
    w.s1 = k % 2 ? kS0 : kS1;
    w.r = held;
    w.r1 = held = held == kR0 ? kR1 : kR0;
    hipLaunchKernelGGL(wide_kernel<B>, dim3((unsigned)mats, B), dim3(64 * B), 0, s, w);
  }
  for (int k = 0; k <= (both ? 1 : 0); ++k) a.p[which + k].R = w.base[k] + held * PP * PP;
}

// ---------------------------------------------------------------- result
// out = R G / |G| for runs of the long side, with 64-bit products of G as it is (divided and rounded first,
// its parts would no longer cancel).  For eight adapters of rank 128 59 us of operations at 67 TFLOP/s and
// 26 us of memory, which take 94 (rounded to 32 bits 56).  Wave w holds rows 16 (w % B) .. of R / |G| in
// registers and takes every (waves / B)th set of 16 long values of a run.  The lanes
// run along the side that is contiguous in memory.
// Steps from one S formed of M to the next: its error, of which the last of them sees a^2
// for each step before it, is multiplied by 2^16 at most.
int steps_at_once(double a, int steps) {
  int n = 1;
  for (double by = a * a; n < steps && by <= 65536.0; by *= a * a) ++n;
  return n;
}

template <int B>
struct Apply {
  static constexpr int SETS = B >= 5 ? 1 : 2, THREADS = 64 * B * SETS;
};

template <int B, bool TALL, int OT>
GPTQ_DEV void apply(const OrthoProblem& o, int gt, int64_t mat, int64_t first, int64_t last, float* lds) {
  using R = Run<B, TALL>;
  constexpr int SETS = Apply<B>::SETS, THREADS = Apply<B>::THREADS, LD = (R::PER + THREADS - 1) / THREADS, PP = 16 * B;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, h = lane >> 4;
  const int row = wave % B, set = wave / B;
  floatx4 next[LD];
  auto fetch = [&](int64_t k0) {
#pragma unroll
    for (int e = 0; e < LD; ++e)
      if (threadIdx.x + THREADS * e < R::PER) next[e] = R::fetch(o, gt, mat, k0, threadIdx.x + THREADS * e);
  };
  fetch(first);
  double w[4 * B];
  const double *by = o.R + mat * o.apart, inv = o.inv[mat];
#pragma unroll
  for (int k = 0; k < 4 * B; ++k) w[k] = by[(4 * k + h) * PP + 16 * row + r] * inv;
  for (int64_t k0 = first; k0 < last; k0 += KS) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < LD; ++e)
      if (threadIdx.x + THREADS * e < R::PER) R::put(lds, R::APPLY, threadIdx.x + THREADS * e, next[e]);
    __syncthreads();
    if (k0 + KS < last) fetch(k0 + KS);
    for (int at = 32 * set; at < KS; at += 32 * SETS) {   // two sets of 16 at a time
      doublex4 acc[2] = {};
#pragma unroll
      for (int k = 0; k < 4 * B; ++k)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const double g = R::get(lds, R::APPLY, 4 * k + h, at + 16 * q + r);
          acc[q] = TALL ? mfma64(g, w[k], acc[q]) : mfma64(w[k], g, acc[q]);
        }
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int s = 16 * row + (TALL ? r : 4 * e + h);                        // place on the shorter side
          const int64_t l = k0 + at + 16 * q + (TALL ? 4 * e + h : r);            // on the longer one
          if (s < o.p && l < o.q) store_out<OT>(o.out, mat * o.rows * o.cols + (TALL ? l * o.p + s : s * o.q + l), (float)acc[q][e]);
        }
    }
  }
}

template <int B, int OT>
__global__ __launch_bounds__(Apply<B>::THREADS) void apply_kernel(OrthoArgs a, int which, int gt, int64_t blocks0, int runs) {
  __shared__ __align__(16) float lds[Run<B, true>::FLOATS > Run<B, false>::FLOATS ? Run<B, true>::FLOATS : Run<B, false>::FLOATS];
  int64_t b = blockIdx.x;
  if (b >= blocks0) b -= blocks0, which = 1;
  const OrthoProblem& o = a.p[which];
  const int64_t per = (o.q + (int64_t)KS * runs - 1) / ((int64_t)KS * runs), mat = b / per, first = (b - mat * per) * KS * runs;
  const int64_t last = min(o.q, first + KS * runs);
  if (o.tall) apply<B, true, OT>(o, gt, mat, first, last, lds);
  else apply<B, false, OT>(o, gt, mat, first, last, lds);
}

// One launch of each kernel for the problems of B tile rows: `which` and, if both, the other;
// and of S and its steps again while steps are left.
template <int B>
void orthogonalize(OrthoArgs a, int which, bool both, int gt, int ot, hipStream_t s) {
  // runs of a workgroup: the places of two or three workgroups on each CU filled once
  int64_t all = 0;
  for (int w = which; w <= (both ? 1 : which); ++w) all += a.m * ((a.p[w].q + KS - 1) / KS);
  const int64_t slots = B > kOrthoNarrow ? 512 : 768;
  const int runs = (int)(all <= slots ? 1 : (all + slots - 1) / slots < 16 ? (all + slots - 1) / slots : 16);
  int64_t gram[2] = {0, 0}, apply[2] = {0, 0};
  for (int w = which; w <= (both ? 1 : which); ++w) {
    gram[w - which] = a.m * a.p[w].splits;
    apply[w - which] = a.m * ((a.p[w].q + (int64_t)KS * runs - 1) / ((int64_t)KS * runs));
  }
  const int steps = a.steps, most = steps_at_once(a.a, steps);
  [[maybe_unused]] int held = kR1;
  for (int done = 0; done < steps; done += most) {
    a.first = done == 0;
    a.steps = steps - done < most ? steps - done : most;
    const dim3 parts((unsigned)(gram[0] + gram[1])), by(GRAM_THREADS);
    if (a.first) hipLaunchKernelGGL((gram_kernel<B, false>), parts, by, 0, s, a, which, gt, gram[0]);
    else hipLaunchKernelGGL((gram_kernel<B, true>), parts, by, 0, s, a, which, gt, gram[0]);
    if constexpr (B > kOrthoNarrow) wide<B>(a, which, both, held, s);
    else hipLaunchKernelGGL(chain_kernel<B>, dim3((unsigned)(both ? 2 * a.m : a.m)), dim3(Chain<B>::THREADS), 0, s, a, which);
  }
  const dim3 grid((unsigned)(apply[0] + apply[1])), block(Apply<B>::THREADS);
  if (ot == 0) hipLaunchKernelGGL((apply_kernel<B, 0>), grid, block, 0, s, a, which, gt, apply[0], runs);
  else if (ot == kBF16) hipLaunchKernelGGL((apply_kernel<B, kBF16>), grid, block, 0, s, a, which, gt, apply[0], runs);
  else hipLaunchKernelGGL((apply_kernel<B, kF16>), grid, block, 0, s, a, which, gt, apply[0], runs);
}

void choose(const OrthoArgs& a, int which, bool both, int gt, int ot, hipStream_t s) {
  switch (ortho_blocks(a.p[which].p)) {
    case 1: return orthogonalize<1>(a, which, both, gt, ot, s);
    case 2: return orthogonalize<2>(a, which, both, gt, ot, s);
    case 3: return orthogonalize<3>(a, which, both, gt, ot, s);
    case 4: return orthogonalize<4>(a, which, both, gt, ot, s);
    case 5: return orthogonalize<5>(a, which, both, gt, ot, s);
    case 6: return orthogonalize<6>(a, which, both, gt, ot, s);
    case 7: return orthogonalize<7>(a, which, both, gt, ot, s);
    default: return orthogonalize<8>(a, which, both, gt, ot, s);
  }
}

}  // namespace

void launch_orthogonalize(const OrthoArgs& args, int gt, int ot, hipStream_t s) {
  OrthoArgs a = args;
  const int64_t e = gt == 0 ? 4 : 2;
  for (OrthoProblem& o : a.p) o.vec = o.G && reinterpret_cast<uintptr_t>(o.G) % (4 * e) == 0 && o.cols % 4 == 0;
  const bool two = a.p[1].G != nullptr, same = two && ortho_blocks(a.p[0].p) == ortho_blocks(a.p[1].p);
  choose(a, 0, same, gt, ot, s);
  if (two && !same) choose(a, 1, false, gt, ot, s);
}

// Parts of S_0: of as many runs each, for both factors together, as one workgroup on every CU
// takes; a matrix's iteration reads them all.
int ortho_splits(int64_t m, int64_t q, int64_t both) {
  const int64_t runs = (q + KS - 1) / KS, all = (m > 0 ? m : 1) * ((both + KS - 1) / KS);
  int64_t each = (all + 255) / 256;
  each = each > runs / 32 ? each : (runs + 31) / 32;
  return (int)((runs + each - 1) / each);
}

bool ortho_fits(int64_t m, int64_t q) { return grid_fits(2 * m * ((q + KS - 1) / KS), 512) && grid_fits(2 * m, 1024) && grid_fits(2 * m * 32, 512); }

}  // namespace gptq
