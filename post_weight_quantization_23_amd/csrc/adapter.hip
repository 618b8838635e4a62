// Low-rank adapters of many requests beside a shared projection:
//     delta[t, i] = alpha_a sum_p B_a[i, p] sum_k A_a[p, k] X[t, k],  a = index[t]
// and their gradients
//     gA_a[p, k] = alpha_a sum_t (dY B_a)[t, p] X[t, k]
//     gB_a[i, p] = alpha_a sum_t dY[t, i] (A_a X)[t, p]     (t over a's tokens).
// The product through the rank is two products: down (X to rank values per
// token, fp32, alpha multiplied in) and up (rank values to the outputs).
#include "adapter.hpp"

namespace gptq {

namespace {

// ---------------------------------------------------------------- down
// A few tokens: one wave per (token, rank row), 64 lanes x 8 elements a load, four
// loads of each operand in flight (a chain of single ones waits for memory once
// per 512 elements).  fp32 sums, folded over the wave in a fixed order.
template <int DT>
__global__ __launch_bounds__(256) void down_kernel(const uint16_t* __restrict__ X, int64_t n, int64_t d, int64_t ldx,
                                                   Adapters ad, const uint16_t* __restrict__ A, int64_t lda, bool vec,
                                                   float* __restrict__ S) {
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = item / ad.rank;
  const int p = (int)(item - t * ad.rank);
  if (t >= n) return;
  const int a = adapter_of(ad, t, n);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  if (a >= 0) {
    const uint16_t* x = X + t * ldx;
    const uint16_t* w = A + ((int64_t)a * ad.rank + p) * lda;
    for (int64_t k0 = 8 * lane; k0 < d; k0 += 2048) {
      u32x4 xv[4], wv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t k = k0 + 512 * u;
        xv[u] = wv[u] = u32x4{0u, 0u, 0u, 0u};
        if (k < d) {
          xv[u] = load8(x + k, (int)min((int64_t)8, d - k), vec);
          wv[u] = *reinterpret_cast<const u32x4*>(w + k);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[u] = __builtin_fmaf(f16_to_f32<DT>(xv[u][i] & 0xFFFFu), f16_to_f32<DT>(wv[u][i] & 0xFFFFu), sum[u]);
          sum[u] = __builtin_fmaf(f16_to_f32<DT>(xv[u][i] >> 16), f16_to_f32<DT>(wv[u][i] >> 16), sum[u]);
        }
    }
  }
  float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) all += __shfl_xor(all, m);
  if (lane == 0) S[item] = a >= 0 && ad.alpha ? all * ad.alpha[a] : all;
}

// Many tokens: a workgroup takes 64 tokens and one of `splits` parts of the
// contraction, its four waves every fourth step of 64 of that part (a whole
// line of memory per row), all 16 RT
// rank rows (operands come from memory in the layout of the product, which
// reads X once).  The adapters that occur among the tokens are taken in turn;
// each writes its own tokens' rows.  Waves are joined through LDS in wave
// order (each has a slot there: adding them up in one, wave after wave, took
// longer than the product), parts by scale_join_kernel.
// FAST: rows of X start on 16 bytes and hold whole steps; then every load is
// unconditional (tokens and rank rows past the end repeat the last one, whose
// results are dropped), so that several steps' loads are in flight.
template <int DT, int RT, bool FAST>
__global__ __launch_bounds__(256) void down_tiles_kernel(const uint16_t* __restrict__ X, int64_t n, int64_t d, int64_t ldx, Adapters ad,
                                                         const uint16_t* __restrict__ A, int64_t lda, bool vec, float* __restrict__ S,
                                                         int splits) {
  constexpr int LD = 16 * RT + 4;   // floats of a token's row in a slot
  extern __shared__ __align__(16) float slots[];   // [4][64][LD]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, kq = lane >> 4;
  const int64_t tile = blockIdx.x / splits;
  const int split = (int)(blockIdx.x - tile * splits);
  const int64_t t0 = tile * 64;
  const int64_t steps = (d + 63) / 64, per = (steps + splits - 1) / splits;
  const int64_t s1 = min(steps, (split + 1) * per);
  float* out = S + (int64_t)split * n * ad.rank;
  const int64_t lane_token = ad.token(t0 + lane, n);
  const int mine = adapter_of(ad, lane_token, n);
  uint64_t rest = __ballot(mine >= 0);
  // this thread's four rank values of every (64 / RT)-th token
  const int col = 4 * (threadIdx.x % (4 * RT)), tok0 = threadIdx.x / (4 * RT);
#pragma unroll
  for (int tok = tok0; tok < 64; tok += 64 / RT)
    if (!((rest >> tok) & 1) && t0 + tok < n && col < ad.rank)
      *reinterpret_cast<floatx4*>(out + ad.token(t0 + tok, n) * ad.rank + col) = floatx4{0.f, 0.f, 0.f, 0.f};
  const uint16_t* xrow[4];   // tokens past the end repeat the last one
#pragma unroll
  for (int i = 0; i < 4; ++i) xrow[i] = X + ad.token(min(t0 + 16 * i + m, n - 1), n) * ldx;
  while (rest) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(rest));
    const uint64_t members = __ballot(mine == a);
    rest &= ~members;
    const uint16_t* w = A + (int64_t)a * ad.rank * lda;
    floatx4 acc[4][RT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int p = 0; p < RT; ++p) acc[i][p] = floatx4{0.f, 0.f, 0.f, 0.f};
    auto step = [&](int64_t k) __attribute__((always_inline)) {
      u32x4 x[4], b[RT];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = u32x4{0u, 0u, 0u, 0u};
        if constexpr (FAST) x[i] = *reinterpret_cast<const u32x4*>(xrow[i] + k);
        else if (k < d) x[i] = load8(xrow[i] + k, (int)min((int64_t)8, d - k), vec);
      }
#pragma unroll
      for (int p = 0; p < RT; ++p) {
        b[p] = u32x4{0u, 0u, 0u, 0u};
        if constexpr (FAST) b[p] = *reinterpret_cast<const u32x4*>(w + (int64_t)min(16 * p + m, ad.rank - 1) * lda + k);
        else if (16 * p + m < ad.rank && k < d) b[p] = *reinterpret_cast<const u32x4*>(w + (int64_t)(16 * p + m) * lda + k);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < RT; ++p) acc[i][p] = mfma16<DT>(x[i], b[p], acc[i][p]);
    };
#pragma unroll FAST && RT <= 4 ? 2 : 1
    for (int64_t s = split * per + wave; s < s1; s += 4) {
      step(64 * s + 8 * kq);
      step(64 * s + 32 + 8 * kq);
    }
    float* slot = slots + wave * 64 * LD;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int p = 0; p < RT; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) slot[(16 * i + 4 * kq + e) * LD + 16 * p + m] = acc[i][p][e];
    __syncthreads();
    const float f = splits == 1 && ad.alpha ? ad.alpha[a] : 1.f;
#pragma unroll
    for (int tok = tok0; tok < 64; tok += 64 / RT) {
      const float* at = slots + tok * LD + col;
      floatx4 v = *reinterpret_cast<const floatx4*>(at);
#pragma unroll
      for (int u = 1; u < 4; ++u) v += *reinterpret_cast<const floatx4*>(at + u * 64 * LD);
      if (((members >> tok) & 1) && col < ad.rank) *reinterpret_cast<floatx4*>(out + ad.token(t0 + tok, n) * ad.rank + col) = f * v;
    }
    __syncthreads();
  }
}

// S[t][p] = alpha_a (sum of the parts), four values per thread.
__global__ __launch_bounds__(256) void scale_join_kernel(const float* __restrict__ part, int64_t n, Adapters ad, int splits,
                                                         float* __restrict__ S) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, all = n * ad.rank;
  if (i >= all) return;
  floatx4 v = *reinterpret_cast<const floatx4*>(part + i);
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const floatx4*>(part + s * all + i);
  const int a = adapter_of(ad, i / ad.rank, n);
  if (a >= 0 && ad.alpha) v *= ad.alpha[a];
  *reinterpret_cast<floatx4*>(S + i) = v;
}

// ---------------------------------------------------------------- up
// What the low-rank product is added to, k <= 8 outputs from column j of token t.
template <int YT>
GPTQ_DEV void add_base(const UpArgs& u, float (&v)[8], int64_t t, int64_t j, int k) {
  if (u.part) {
    float sum[8] = {};
    const int64_t at = t * u.rows + j;
    for (int s = 0; s < u.splits; ++s) {
      const float* p = u.part + s * u.n * u.rows + at;
      if (k == 8 && u.vec_base) {
        float w[8];
        load8f(p, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += w[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < k) sum[e] += p[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += u.ex ? __builtin_ldexpf(sum[e], u.ex[t]) : sum[e];
  } else if (u.base) {
    if constexpr (YT == 0) {
      const float* p = static_cast<const float*>(u.base) + t * u.ldb + j;
      if (k == 8 && u.vec_base) {
        float w[8];
        load8f(p, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += w[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < k) v[e] += p[e];
      }
    } else {
      const u32x4 w = load8(static_cast<const uint16_t*>(u.base) + t * u.ldb + j, k, u.vec_base);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] += f16_to_f32<YT>(w[e] & 0xFFFFu);
        v[2 * e + 1] += f16_to_f32<YT>(w[e] >> 16);
      }
    }
  }
}

// Many tokens: a wave takes 32 tokens x 64 outputs on the matrix cores.
template <int DT, int YT>
__global__ __launch_bounds__(256) void up_tiles_kernel(UpArgs u) {
  __shared__ float turn[4][32 * 68];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t tile = blockIdx.x / u.col_tiles, ct = blockIdx.x - tile * u.col_tiles;
  const int64_t t0 = tile * 32, j0 = ct * 256 + 64 * wave;
  int64_t row[2];
  floatx16 acc[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t j = j0 + 32 * q + (lane & 31);
    row[q] = j < u.rows ? j : -1;
    acc[q] = floatx16{};
  }
  if (u.S) expand_add<DT, YT == 0 ? 3 : 2, 2>(u.ad, u.B, u.rows, u.S, t0, u.n, row, acc);
  store_tile<YT, 2>(turn[wave], acc, u.ad, u.out, t0, u.n, j0, u.rows, u.ldo, u.vec_out,
                    [&](float (&v)[8], int64_t t, int64_t j, int k) { add_base<YT>(u, v, t, j, k); });
}

// A few tokens: a thread takes one output of one token, and its row of that
// token's adapter (a tile of 32 tokens would take 32 adapters in turn).
template <int DT, int YT>
__global__ __launch_bounds__(256) void up_kernel(UpArgs u) {
  const int64_t t = blockIdx.x / u.col_tiles, ct = blockIdx.x - t * u.col_tiles;
  const int64_t j = ct * 256 + threadIdx.x;
  if (j >= u.rows) return;
  float v[8] = {};
  const int a = u.S ? adapter_of(u.ad, t, u.n) : -1;
  if (a >= 0) v[0] = rank_dot<DT>(u.S + t * u.ad.rank, u.B + ((int64_t)a * u.rows + j) * u.ad.rank, u.ad.rank);
  add_base<YT>(u, v, t, j, 1);
  store_out<YT>(u.out, t * u.ldo + j, v[0]);
}

// ---------------------------------------------------------------- transpose
__global__ __launch_bounds__(256) void transpose16_kernel(const uint16_t* __restrict__ src, int64_t rows, int64_t cols,
                                                          uint16_t* __restrict__ dst, int64_t ldd, int64_t row_tiles) {
  __shared__ uint16_t tile[64][66];
  const int64_t bt = blockIdx.x / row_tiles, rt = blockIdx.x - bt * row_tiles;
  const int64_t ct_n = (cols + 63) / 64;
  const int64_t a = bt / ct_n, ct = bt - a * ct_n;
  const int64_t i0 = rt * 64, j0 = ct * 64;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int r = w; r < 64; r += 4) {
    const int64_t i = i0 + r, j = j0 + lane;
    tile[r][lane] = (i < rows && j < cols) ? src[(a * rows + i) * cols + j] : (uint16_t)0;
  }
  __syncthreads();
  for (int r = w; r < 64; r += 4) {
    const int64_t j = j0 + r, i = i0 + lane;
    if (j < cols && i < ldd) dst[(a * cols + j) * ldd + i] = tile[lane][r];
  }
}

// ---------------------------------------------------------------- token lists
// Workgroup a lists its adapter's tokens in ascending order.  It counts the
// tokens of the adapters before it (c) and starts at 32 (ceil(c / 32) + a): the
// next one starts at least count + 1 places further and on a multiple of 32.
// No atomics, so the order is fixed.
__global__ __launch_bounds__(1024) void token_lists_kernel(Adapters ad, int64_t n, int32_t* __restrict__ order,
                                                           int32_t* __restrict__ start, int32_t* __restrict__ counts) {
  __shared__ int below[16];
  __shared__ int count[16];
  const int a = blockIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int less = 0;
  for (int64_t t = threadIdx.x; t < n; t += 1024) {
    const int v = adapter_of(ad, t, n);
    less += v >= 0 && v < a;
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) less += __shfl_xor(less, m);
  if (lane == 0) below[w] = less;
  __syncthreads();
  int before_all = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) before_all += below[i];
  const int64_t first = 32 * ((int64_t)(before_all + 31) / 32 + a);
  int64_t at = first;
  for (int64_t t0 = 0; t0 < n; t0 += 1024) {
    const int64_t t = t0 + threadIdx.x;
    const bool in = adapter_of(ad, t, n) == a;
    const uint64_t mask = __ballot(in);
    if (lane == 0) count[w] = __popcll(mask);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      before += i < w ? count[i] : 0;
      all += count[i];
    }
    if (in) order[at + before + __popcll(mask & ((1ull << lane) - 1))] = (int32_t)t;
    at += all;
    __syncthreads();
  }
  const int mine = (int)(at - first);
  const int64_t next = 32 * ((int64_t)(before_all + mine + 31) / 32 + a + 1);
  for (int64_t i = at + threadIdx.x; i < next; i += 1024) order[i] = -1;
  if (threadIdx.x == 0) {
    start[a] = (int32_t)first;
    counts[a] = mine;
    if (a == ad.m - 1) start[a + 1] = (int32_t)next;
  }
}

// All tokens by adapter, ascending, those without one last: workgroup a places the
// tokens of adapter a (a == m: without) after those of the adapters before it.
__global__ __launch_bounds__(1024) void token_order_kernel(Adapters ad, int64_t n, int32_t* __restrict__ order) {
  __shared__ int below[16];
  __shared__ int count[16];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint32_t a = blockIdx.x;   // as the unsigned adapter of a token, none being m
  auto key = [&](int64_t t) { return min((uint32_t)adapter_of(ad, t, n), (uint32_t)ad.m); };
  int less = 0;
  for (int64_t t = threadIdx.x; t < n; t += 1024) less += key(t) < a;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) less += __shfl_xor(less, m);
  if (lane == 0) below[w] = less;
  __syncthreads();
  int64_t at = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) at += below[i];
  for (int64_t t0 = 0; t0 < n; t0 += 1024) {
    const int64_t t = t0 + threadIdx.x;
    const bool in = t < n && key(t) == a;
    const uint64_t mask = __ballot(in);
    if (lane == 0) count[w] = __popcll(mask);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      before += i < w ? count[i] : 0;
      all += count[i];
    }
    if (in) order[at + before + __popcll(mask & ((1ull << lane) - 1))] = (int32_t)t;
    at += all;
    __syncthreads();
  }
}

// The rank values in list order, transposed and split into three bf16 terms: the
// gradients' operand as it is loaded.  One thread per rank row and eight places.
__global__ __launch_bounds__(256) void sorted_terms_kernel(const float* __restrict__ V, int rank, const int32_t* __restrict__ order,
                                                           const int32_t* __restrict__ used, int64_t places,
                                                           uint16_t* __restrict__ terms) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t p8 = i / rank * 8;
  const int p = (int)(i % rank);
  if (p8 >= *used) return;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int t = order[p8 + e];
    v[e] = t >= 0 ? V[(int64_t)t * rank + p] : 0.f;
  }
  u32x4 k[3];
  split8<3>(v, k);
#pragma unroll
  for (int u = 0; u < 3; ++u) *reinterpret_cast<u32x4*>(terms + ((int64_t)u * rank + p) * places + p8) = k[u];
}

// ---------------------------------------------------------------- gradients
// G[p, j] = sum over the adapter's tokens of V[t, p] Z[t, j].  The contraction
// runs over tokens, along which Z is not contiguous.  A lane loads 8 columns of
// 8 tokens of Z; column u of them is its operand of the u-th of eight products,
// whose 16 columns are j0 + 8 (lane & 15) + u: the transpose happens in
// registers.  Tokens come through the adapter's list, so they may lie in any
// order; places past its end repeat its first token and multiply zeros.  V
// comes in three bf16 terms (24 significant bits) and fp16 Z is split in two,
// so the gradient keeps fp32's range and precision.
// A wave takes 128 columns x 16 RT rank rows and one of `splits` parts of the
// adapter's tokens, by itself (four waves joined through LDS spent more time
// there than on their five blocks of tokens); parts are added in order by
// join_kernel.
template <int DT, int RT>
__global__ __launch_bounds__(256) void grad_kernel(const uint16_t* __restrict__ terms, int64_t places, const uint16_t* __restrict__ Z,
                                                   int64_t cols, int64_t ldz, bool vec, int rank, const int32_t* __restrict__ order,
                                                   const int32_t* __restrict__ start, const int32_t* __restrict__ counts, int up,
                                                   float* __restrict__ G, int64_t items, int64_t col_blocks, int rank_blocks, int splits) {
  const int lane = threadIdx.x & 63, m = lane & 15, kq = lane >> 4;
  int64_t b = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (b >= items) return;
  const int64_t cb = b % col_blocks;
  b /= col_blocks;
  const int rb = (int)(b % rank_blocks);
  b /= rank_blocks;
  const int split = (int)(b % splits);
  const int a = (int)(b / splits);
  const int64_t first = start[a];
  const int count = counts[a];
  // whole 16-byte loads where rows allow them: columns past the end repeat the
  // last eight, whose results are dropped
  const int64_t jv = cb * 128 + 8 * m;
  const bool whole = vec && cols % 8 == 0;
  const int64_t j0 = whole ? min(jv, cols - 8) : jv;
  const int valid = (int)max((int64_t)0, min((int64_t)8, cols - j0));
  const int p0 = rb * 16 * RT;

  floatx4 acc[RT][8];
#pragma unroll
  for (int p = 0; p < RT; ++p)
#pragma unroll
    for (int u = 0; u < 8; ++u) acc[p][u] = floatx4{0.f, 0.f, 0.f, 0.f};

  const int blocks = (count + 31) / 32;
  const int each = (blocks + splits - 1) / splits;
  const int b0 = split * each, b1 = min(blocks, (split + 1) * each);
  // tokens two blocks ahead, their rows of Z and the terms one block ahead
  struct Operands {
    u32x4 z[8], v[RT][3];
  } f0, f1;
  typedef int int4_t __attribute__((ext_vector_type(4)));
  int4_t tok[2];
  const int spare = b0 < b1 ? order[first] : 0;
  auto load_tokens = [&](int blk) __attribute__((always_inline)) {
    const int4_t* p = reinterpret_cast<const int4_t*>(order + first + 32 * (int64_t)blk + 8 * kq);   // 32-byte aligned
    tok[0] = p[0];
    tok[1] = p[1];
  };
  auto load = [&](Operands& f, int blk) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      int t = tok[e >> 2][e & 3];
      if (t < 0) t = spare;
      if (whole) f.z[e] = *reinterpret_cast<const u32x4*>(Z + (int64_t)t * ldz + j0);
      else f.z[e] = load8(Z + (int64_t)t * ldz + j0, valid, vec);
    }
#pragma unroll
    for (int p = 0; p < RT; ++p)
#pragma unroll
      for (int k = 0; k < 3; ++k)
        f.v[p][k] = *reinterpret_cast<const u32x4*>(terms + ((int64_t)k * rank + min(p0 + 16 * p + m, rank - 1)) * places + first +
                                                    32 * (int64_t)blk + 8 * kq);
    if (blk + 1 < b1) load_tokens(blk + 1);
  };
  auto use = [&](const Operands& f) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      u32x4 c;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c[e] = __builtin_amdgcn_perm(f.z[2 * e + 1][u >> 1], f.z[2 * e][u >> 1], (u & 1) ? 0x07060302u : 0x05040100u);
      const Terms16<DT> zt(c);
#pragma unroll
      for (int p = 0; p < RT; ++p) acc[p][u] = mfma_terms<DT, 3>(f.v[p], zt, acc[p][u]);
    }
  };
  int blk = b0;
  if (blk < b1) {
    load_tokens(blk);
    load(f0, blk);
  }
  while (blk < b1) {
    if (blk + 1 < b1) load(f1, blk + 1);
    use(f0);
    if (++blk >= b1) break;
    if (blk + 1 < b1) load(f0, blk + 1);
    use(f1);
    ++blk;
  }

  // row of the accumulator = rank, column = 8 (lane & 15) + u
  const int64_t m_all = items / (col_blocks * rank_blocks * splits);
  float* g = G + ((int64_t)split * m_all + a) * rank * cols;
#pragma unroll
  for (int p = 0; p < RT; ++p) {
    const int pr = p0 + 16 * p + 4 * kq;
    if (up) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (jv + u < cols && pr < rank) *reinterpret_cast<floatx4*>(g + (jv + u) * rank + pr) = acc[p][u];   // rank % 8 == 0
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (pr + i >= rank) continue;
        float* o = g + (int64_t)(pr + i) * cols + jv;
        if (jv + 8 <= cols && cols % 4 == 0) {
          *reinterpret_cast<floatx4*>(o) = floatx4{acc[p][0][i], acc[p][1][i], acc[p][2][i], acc[p][3][i]};
          *reinterpret_cast<floatx4*>(o + 4) = floatx4{acc[p][4][i], acc[p][5][i], acc[p][6][i], acc[p][7][i]};
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (jv + u < cols) o[u] = acc[p][u][i];
        }
      }
    }
  }
}

__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ part, int64_t n, int splits,
                                                   float* __restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  floatx4 v = *reinterpret_cast<const floatx4*>(part + i);
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const floatx4*>(part + s * n + i);
  *reinterpret_cast<floatx4*>(out + i) = v;
}

// Parts of the contraction of down_tiles_kernel: enough workgroups for the
// chip, each wave left with two steps at least.
int down_splits(int64_t n, int64_t d) {
  const int64_t tiles = (n + 63) / 64, steps = (d + 63) / 64;
  int64_t splits = 512 / tiles;
  splits = splits < steps / 8 ? splits : steps / 8;
  return splits < 1 ? 1 : (splits > 16 ? 16 : (int)splits);
}

// Whether each token is taken by itself: a few of them, or so many adapters that a
// tile would hold ten and more.
bool by_token(int64_t n, int m) { return n <= 64 || n <= 4 * (int64_t)m; }

}  // namespace

template <int DT, int RT, bool FAST, class... Args>
static void launch_down_tiles(dim3 grid, hipStream_t s, Args... args) {
  constexpr int LDS = 4 * 64 * (16 * RT + 4) * 4;
  static const bool set = [] {   // once, thread-safe
    (void)hipFuncSetAttribute((const void*)down_tiles_kernel<DT, RT, FAST>, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    return true;
  }();
  (void)set;
  hipLaunchKernelGGL((down_tiles_kernel<DT, RT, FAST>), grid, dim3(256), LDS, s, args...);
}

int64_t adapter_down_floats(int64_t n, int64_t d, int64_t rank) {
  const int64_t one = (n * rank + 63) / 64 * 64;
  const int splits = n <= 64 ? 1 : down_splits(n, d);
  return splits == 1 ? one : one + splits * n * rank;
}

void launch_adapter_down(const void* X, int xt, int64_t n, int64_t d, int64_t ldx, const Adapters& ad, const uint16_t* A,
                         int64_t lda, float* S, hipStream_t s) {
  const dim3 block(256);
  const bool vec = rows_on_16(X, ldx, xt);
  const auto* x = static_cast<const uint16_t*>(X);
  if (by_token(n, ad.m)) {
    const dim3 grid((unsigned)((n * ad.rank + 3) / 4));
    if (xt == kBF16) hipLaunchKernelGGL((down_kernel<kBF16>), grid, block, 0, s, x, n, d, ldx, ad, A, lda, vec, S);
    else hipLaunchKernelGGL((down_kernel<kF16>), grid, block, 0, s, x, n, d, ldx, ad, A, lda, vec, S);
    return;
  }
  const int splits = down_splits(n, d);
  float* out = splits == 1 ? S : S + (n * ad.rank + 63) / 64 * 64;
  const dim3 grid((unsigned)((n + 63) / 64 * splits));
#define GPTQ_DOWN(D_, R_)                                                                                                    \
  (vec && d % 64 == 0 ? launch_down_tiles<D_, R_, true>(grid, s, x, n, d, ldx, ad, A, lda, vec, out, splits)                 \
                      : launch_down_tiles<D_, R_, false>(grid, s, x, n, d, ldx, ad, A, lda, vec, out, splits))
#define GPTQ_DOWN_R(D_)                     \
  do {                                      \
    if (ad.rank <= 16) GPTQ_DOWN(D_, 1);    \
    else if (ad.rank <= 32) GPTQ_DOWN(D_, 2); \
    else if (ad.rank <= 64) GPTQ_DOWN(D_, 4); \
    else GPTQ_DOWN(D_, 8);                  \
  } while (0)
  if (xt == kBF16) GPTQ_DOWN_R(kBF16);
  else GPTQ_DOWN_R(kF16);
#undef GPTQ_DOWN_R
#undef GPTQ_DOWN
  if (splits > 1)
    hipLaunchKernelGGL(scale_join_kernel, dim3((unsigned)((n * ad.rank / 4 + 255) / 256)), block, 0, s, out, n, ad, splits, S);
}

void launch_adapter_up(const UpArgs& given, int xt, int yt, hipStream_t s) {
  UpArgs u = given;
  u.col_tiles = (u.rows + 255) / 256;
  u.vec_base = u.part ? rows_on_16(u.part, u.rows, 0) : rows_on_16(u.base, u.ldb, yt);
  u.vec_out = rows_on_16(u.out, u.ldo, yt);
  const bool few = u.n <= 64 || (u.S && by_token(u.n, u.ad.m));
  const dim3 grid((unsigned)((few ? u.n : (u.n + 31) / 32) * u.col_tiles)), block(256);
#define GPTQ_UP(D_, Y_)                                                                \
  do {                                                                                 \
    if (few) hipLaunchKernelGGL((up_kernel<D_, Y_>), grid, block, 0, s, u);            \
    else hipLaunchKernelGGL((up_tiles_kernel<D_, Y_>), grid, block, 0, s, u);          \
  } while (0)
  if (xt == kBF16) { if (yt == 0) GPTQ_UP(kBF16, 0); else GPTQ_UP(kBF16, kBF16); }
  else { if (yt == 0) GPTQ_UP(kF16, 0); else GPTQ_UP(kF16, kF16); }
#undef GPTQ_UP
}

void launch_transpose16(const uint16_t* src, int m, int64_t rows, int64_t cols, uint16_t* dst, int64_t ldd, hipStream_t s) {
  const int64_t rt = (ldd + 63) / 64;
  hipLaunchKernelGGL(transpose16_kernel, dim3((unsigned)(rt * ((cols + 63) / 64) * m)), dim3(256), 0, s, src, rows, cols, dst,
                     ldd, rt);
}

bool adapters_want_order(int64_t n, int m, const int32_t* index) { return index && m > 1 && !by_token(n, m); }

void launch_token_order(const Adapters& ad, int64_t n, int32_t* order, hipStream_t s) {
  hipLaunchKernelGGL(token_order_kernel, dim3((unsigned)ad.m + 1), dim3(1024), 0, s, ad, n, order);
}

void launch_token_lists(const Adapters& ad, int64_t n, int32_t* order, int32_t* start, int32_t* count, hipStream_t s) {
  hipLaunchKernelGGL(token_lists_kernel, dim3((unsigned)ad.m), dim3(1024), 0, s, ad, n, order, start, count);
}

void launch_sorted_terms(const float* V, int rank, const int32_t* order, const int32_t* used, int64_t places, uint16_t* terms,
                         hipStream_t s) {
  hipLaunchKernelGGL(sorted_terms_kernel, dim3((unsigned)((places / 8 * rank + 255) / 256)), dim3(256), 0, s, V, rank, order, used, places,
                     terms);
}

// Rank rows of a gradient wave: 32 (64 would leave one wave per SIMD).
int grad_rows(int rank) { return rank <= 16 ? 16 : 32; }

int adapter_grad_splits(int64_t n, int m, int64_t cols, int rank) {
  if (n == 0 || cols == 0) return 1;
  const int64_t waves = (cols + 127) / 128 * m * ((rank + grad_rows(rank) - 1) / grad_rows(rank));
  int64_t splits = (2048 + waves - 1) / waves;
  const int64_t most = (n + m - 1) / m / 64;   // two blocks of tokens each
  splits = splits < most ? splits : most;
  return splits < 1 ? 1 : (splits > 16 ? 16 : (int)splits);
}

void launch_adapter_grad(const uint16_t* terms, int64_t places, const void* Z, int zt, int64_t n, int64_t cols, int64_t ldz,
                         const Adapters& ad, const int32_t* order, const int32_t* start, const int32_t* count, int up, float* G,
                         float* part, int splits, hipStream_t s) {
  const bool vec = rows_on_16(Z, ldz, zt);
  const int rt = grad_rows(ad.rank);
  const int rb = (ad.rank + rt - 1) / rt;
  const int64_t cb = (cols + 127) / 128, items = cb * rb * splits * ad.m;
  const dim3 grid((unsigned)((items + 3) / 4)), block(256);
  float* dst = splits > 1 ? part : G;
  const auto* z = static_cast<const uint16_t*>(Z);
#define GPTQ_GRAD(D_, R_)                                                                                                       \
  hipLaunchKernelGGL((grad_kernel<D_, R_>), grid, block, 0, s, terms, places, z, cols, ldz, vec, ad.rank, order, start, count, up, dst, \
                     items, cb, rb, splits)
  if (zt == kBF16) { if (rt == 16) GPTQ_GRAD(kBF16, 1); else GPTQ_GRAD(kBF16, 2); }
  else { if (rt == 16) GPTQ_GRAD(kF16, 1); else GPTQ_GRAD(kF16, 2); }
#undef GPTQ_GRAD
  if (splits > 1) {
    const int64_t all = (int64_t)ad.m * ad.rank * cols;   // rank is a multiple of 8: whole vectors
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)((all / 4 + 255) / 256)), dim3(256), 0, s, part, all, splits, G);
  }
}

}  // namespace gptq
