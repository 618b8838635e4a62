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

typedef __attribute__((address_space(3))) unsigned char lds_u8;

// fp32 sums of split gradients: out = parts added in order, for up to two of them.
struct JoinArgs {
  const float* part[2];
  float* out[2];
  int64_t n[2];
  int splits[2];
};

// ---------------------------------------------------------------- down
// A few tokens: one wave per (token, rank row), 64 lanes x 8 elements a load, four
// loads of each operand in flight (a chain of single ones waits for memory once
// per 512 elements).  fp32 sums, folded over the wave in a fixed order.
template <int DT>
__global__ __launch_bounds__(256) void down_kernel(DownArgs g) {
  const int lane = threadIdx.x & 63;
  int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t per = g.n * g.ad.rank;
  const DownProblem& q = g.p[item < per ? 0 : 1];
  if (item >= per) item -= per;
  const int64_t t = item / g.ad.rank;
  const int p = (int)(item - t * g.ad.rank);
  if (t >= g.n || !q.X) return;
  const int a = adapter_of(g.ad, t, g.n);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  if (a >= 0) {
    const uint16_t* x = q.X + t * q.ldx;
    const uint16_t* w = q.A + ((int64_t)a * g.ad.rank + p) * q.lda;
    for (int64_t k0 = 8 * lane; k0 < q.d; k0 += 2048) {
      u32x4 xv[4], wv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t k = k0 + 512 * u;
        xv[u] = wv[u] = u32x4{0u, 0u, 0u, 0u};
        if (k < q.d) {
          xv[u] = load8(x + k, (int)min((int64_t)8, q.d - k), q.vec);
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
  if (lane == 0) q.S[item] = a >= 0 && g.ad.alpha ? all * g.ad.alpha[a] : all;
}

// Many tokens: a workgroup takes the 64 tokens at 64 places and one of `splits`
// parts of the contraction, each wave 16 of the tokens and all 16 RT rank rows.
// Steps of 64 come into LDS by loads that write it (double buffered): loading
// operands straight into registers touches 64 places of 16 bytes per
// instruction, which the L1 cache takes one a cycle, against 16 here (4096
// tokens of 11008, rank 64: 37 us, memory's share is 18; with 4096 columns beside
// them 41 us now, 3 TB/s).  The adapters that
// occur among the tokens are taken in turn; each writes its own tokens' rows.
// Parts are added by the kernels that read them.
template <int DT, int RT>
GPTQ_DEV void down_tiles_body(const DownArgs& g, unsigned char* smem) {
  constexpr int ROWB = 128, XB = 64 * ROWB, BUF = XB + 16 * RT * ROWB;
  constexpr int QW = 16 * RT / 8;   // load instructions of a step for the rank rows (8 rows each); the tokens take 8
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, kq = lane >> 4;
  const Adapters& ad = g.ad;
  int64_t b = blockIdx.x;
  const bool second = b >= g.blocks0;
  const DownProblem& q = g.p[second ? 1 : 0];
  if (second) b -= g.blocks0;
  const int64_t tile = b / q.splits;
  const int split = (int)(b - tile * q.splits);
  const int64_t t0 = tile * 64;
  const int64_t steps = (q.d + 63) / 64, per = (steps + q.splits - 1) / q.splits;
  const int64_t sa = split * per, s1 = min(steps, sa + per);
  float* out = q.splits == 1 ? q.S : q.S + down_values(g.n, ad.rank) + (int64_t)split * g.n * ad.rank;
  const int mine = adapter_of(ad, ad.token(t0 + lane, g.n), g.n);
  uint64_t rest = __ballot(mine >= 0);
  // rows of tokens without an adapter: this thread's four rank values of every (64 / RT)-th token
  const int col = 4 * (threadIdx.x % (4 * RT)), tok0 = threadIdx.x / (4 * RT);
#pragma unroll
  for (int tok = tok0; tok < 64; tok += 64 / RT)
    if (!((rest >> tok) & 1) && t0 + tok < g.n && col < ad.rank)
      *reinterpret_cast<floatx4*>(out + ad.token(t0 + tok, g.n) * ad.rank + col) = floatx4{0.f, 0.f, 0.f, 0.f};

  // sources of this lane: piece (16 bytes) lane & 7 of row lane >> 3, permuted by
  // the row; tokens past the end repeat the last one, pieces past the end of a
  // row its last one
  lds_u8* lbase = (lds_u8*)smem;
  const uint16_t* xsrc[2];
  int xpiece[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 8 * (2 * wave + i) + (lane >> 3);
    xsrc[i] = q.X + ad.token(min(t0 + row, g.n - 1), g.n) * q.ldx;
    xpiece[i] = (lane & 7) ^ (row & 7);
  }
  const int64_t xlast = q.d / 8 - 1, wlast = q.lda / 8 - 1;
  while (rest) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(rest));
    const uint64_t members = __ballot(mine == a);
    rest &= ~members;
    const uint16_t* w = q.A + (int64_t)a * ad.rank * q.lda;
    auto load = [&](int64_t s) __attribute__((always_inline)) {
      lds_u8* to = lbase + ((s - sa) & 1) * BUF;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        __builtin_amdgcn_global_load_lds((const void __attribute__((address_space(1)))*)(xsrc[i] + 8 * min(8 * s + xpiece[i], xlast)),
                                         (void __attribute__((address_space(3)))*)(to + (2 * wave + i) * 1024), 16, 0, 0);
#pragma unroll
      for (int i = wave; i < QW; i += 4) {
        const int row = 8 * i + (lane >> 3);
        __builtin_amdgcn_global_load_lds(
            (const void __attribute__((address_space(1)))*)(w + (int64_t)min(row, ad.rank - 1) * q.lda + 8 * min(8 * s + ((lane & 7) ^ (row & 7)), wlast)),
            (void __attribute__((address_space(3)))*)(to + XB + i * 1024), 16, 0, 0);
      }
    };
    floatx4 acc[RT];
#pragma unroll
    for (int p = 0; p < RT; ++p) acc[p] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (sa < s1) load(sa);
    for (int64_t s = sa; s < s1; ++s) {
      __builtin_amdgcn_s_waitcnt(0);   // own loads have landed; with every wave here, the other buffer is free
      unsigned char* at = smem + ((s - sa) & 1) * BUF;
      if (8 * s + 8 > q.d / 8) {       // the last step's places past the end, of the tokens that this wave loaded
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (8 * s + xpiece[i] > xlast) *reinterpret_cast<u32x4*>(at + (2 * wave + i) * 1024 + lane * 16) = u32x4{0u, 0u, 0u, 0u};
      }
      __syncthreads();
      if (s + 1 < s1) load(s + 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int xr = 16 * wave + m;
        const u32x4 x = *reinterpret_cast<const u32x4*>(at + xr * ROWB + (((4 * h + kq) ^ (xr & 7)) << 4));
#pragma unroll
        for (int p = 0; p < RT; ++p) {
          const int wr = 16 * p + m;
          const u32x4 v = *reinterpret_cast<const u32x4*>(at + XB + wr * ROWB + (((4 * h + kq) ^ (wr & 7)) << 4));
          acc[p] = mfma16<DT>(x, v, acc[p]);
        }
      }
    }
    const float f = q.splits == 1 && ad.alpha ? ad.alpha[a] : 1.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int tok = 16 * wave + 4 * kq + e;
      if (!((members >> tok) & 1)) continue;
      float* o = out + ad.token(t0 + tok, g.n) * ad.rank;
#pragma unroll
      for (int p = 0; p < RT; ++p)
        if (16 * p + m < ad.rank) o[16 * p + m] = f * acc[p][e];
    }
    __syncthreads();   // every wave has read the last step
  }
}

template <int DT, int RT>
__global__ __launch_bounds__(256) void down_tiles_kernel(DownArgs g) {
  __shared__ __align__(16) unsigned char smem[2 * (64 + 16 * RT) * 128];
  down_tiles_body<DT, RT>(g, smem);
}

// S[t][p] = alpha_a (sum of the parts), four values per thread.
__global__ __launch_bounds__(256) void scale_join_kernel(float* __restrict__ S, int64_t n, Adapters ad, int splits) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, all = n * ad.rank;
  if (i >= all) return;
  const float* part = S + down_values(n, ad.rank);
  floatx4 v = *reinterpret_cast<const floatx4*>(part + i);
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const floatx4*>(part + s * all + i);
  const int a = adapter_of(ad, i / ad.rank, n);
  if (a >= 0 && ad.alpha) v *= ad.alpha[a];
  *reinterpret_cast<floatx4*>(S + i) = v;
}

// ---------------------------------------------------------------- up
// Sum of the parts of eight outputs (their rows are padded to whole eights), two
// chains of adds so that four loads are in flight.
GPTQ_DEV void join_parts(const UpArgs& u, int64_t t, int64_t j, float (&v)[8]) {
  const float* p = u.part + t * u.ldp + j;
  const int64_t step = u.n * u.ldp;
  float a[8], b[8] = {};
  load8f(p, a);
  int s = 1;
  for (; s + 1 < u.splits; s += 2) {
    float x[8], y[8];
    load8f(p + s * step, x);
    load8f(p + (s + 1) * step, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] += x[e];
      b[e] += y[e];
    }
  }
  if (s < u.splits) {
    float x[8];
    load8f(p + s * step, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] += x[e];
  }
  const int ex = u.ex ? u.ex[t] : 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += __builtin_ldexpf(a[e] + b[e], ex);
}

// What the low-rank product is added to, k <= 8 outputs from column j (a multiple of 8) of token t.
template <int YT>
GPTQ_DEV void add_base(const UpArgs& u, float (&v)[8], int64_t t, int64_t j, int k) {
  if (u.part) {
    join_parts(u, t, j, v);
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

// Many tokens: a wave takes 32 tokens x 64 outputs on the matrix cores.  Memory
// bounds it (180 MB for 4099 tokens of 11008 outputs).  PLAIN: added to rows on 16
// bytes, of whole eights; these are asked for first, so that their way from
// memory runs beside the rank values' (48 us, 60 without; a wave of 32 outputs, with
// more waves in a SIMD: 54).
template <int DT, int YT, bool PLAIN>
__global__ __launch_bounds__(256) void up_tiles_kernel(UpArgs u) {
  constexpr int PIECES = YT == 0 ? 2 : 1;   // of 16 bytes in eight outputs
  __shared__ float turn[4][32 * 36];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t tile = blockIdx.x / u.col_tiles, ct = blockIdx.x - tile * u.col_tiles;
  const int64_t t0 = tile * 32, j0 = ct * 256 + 64 * wave;
  // this lane's eight outputs of four places: 32 q + 8 (lane & 3) of place 16 k + lane / 4
  int64_t tok[2];
  u32x4 base[2][2][PIECES];
#pragma unroll
  for (int k = 0; k < 2; ++k) tok[k] = u.ad.token(t0 + 16 * k + (lane >> 2), u.n);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t j = j0 + 32 * q + 8 * (lane & 3);
    if (!PLAIN || j >= u.rows) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int p = 0; p < PIECES; ++p)
        base[q][k][p] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(u.base) +
                                                        (max(tok[k], (int64_t)0) * u.ldb + j) * (YT == 0 ? 4 : 2) + 16 * p);
  }
  int64_t row[2];
  floatx16 acc[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t i = j0 + 32 * q + (lane & 31);
    row[q] = i < u.rows ? i : -1;
    acc[q] = floatx16{};
  }
  expand_add<DT, YT == 0 ? 3 : 2, 2>(u.ad, u.B, u.rows, u.S, t0, u.n, row, acc);
  float* own = turn[wave];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t j = j0 + 32 * q + 8 * (lane & 3);
    const floatx16 half[1] = {acc[q]};
    turn_tile<1>(own, half);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (tok[k] < 0 || j >= u.rows) continue;
      float v[8];
      load8f(own + (16 * k + (lane >> 2)) * 36 + 8 * (lane & 3), v);
      if constexpr (PLAIN) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if constexpr (YT == 0) {
            const uint32_t w = base[q][k][e >> 2][e & 3];
            v[e] += __builtin_bit_cast(float, w);
          } else {
            v[e] += f16_to_f32<YT>((base[q][k][0][e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
          }
        }
        store8<YT>(u.out, tok[k] * u.ldo + j, v, 8, true);
      } else {
        const int count = (int)min((int64_t)8, u.rows - j);
        add_base<YT>(u, v, tok[k], j, count);
        store8<YT>(u.out, tok[k] * u.ldo + j, v, count, u.vec_out);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // read before the other half replaces it
  }
}

// A few tokens: SHARE threads take one output of one token, and its row of that
// token's adapter (a tile of 32 tokens would take 32 adapters in turn).  Rows of
// more than 16 ranks go to four threads, eight ranks each in turn, so that a load
// touches 16 places instead of 64 (39 tokens, 11008 outputs of rank 88: 18 us,
// 78 with one); one thread does for shorter ones (32 tokens, 4096 outputs of rank
// 16: 2.9 us).
template <int DT, int YT, int SHARE>
__global__ __launch_bounds__(256) void up_kernel(UpArgs u) {
  const int64_t t = blockIdx.x / u.col_tiles, ct = blockIdx.x - t * u.col_tiles;
  const int part = threadIdx.x % SHARE, rank = u.ad.rank;
  const int a = adapter_of(u.ad, t, u.n);
#pragma unroll
  for (int i = 0; i < SHARE; ++i) {
    const int64_t j = ct * 256 + (256 * i + (int)threadIdx.x) / SHARE;
    float v[8] = {};
    if (a >= 0 && j < u.rows) {
      const float* S = u.S + t * rank;
      const uint16_t* row = u.B + ((int64_t)a * u.rows + j) * rank;
      for (int p = 8 * part; p < rank; p += 8 * SHARE) v[0] += rank_dot<DT>(S + p, row + p, 8);
    }
#pragma unroll
    for (int m = 1; m < SHARE; m <<= 1) v[0] += __shfl_xor(v[0], m);
    if (part || j >= u.rows) continue;
    if (u.part) {
      float w[8] = {};
      join_parts(u, t, j & ~(int64_t)7, w);
      float mine = w[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) mine = (j & 7) == e ? w[e] : mine;
      v[0] += mine;
    } else {
      add_base<YT>(u, v, t, j, 1);
    }
    store_out<YT>(u.out, t * u.ldo + j, v[0]);
  }
}

// Parts joined without adapters: a thread takes eight outputs of one token.
template <int YT>
__global__ __launch_bounds__(256) void join_rows_kernel(UpArgs u) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = u.ldp >> 3, t = i / per, j = (i - t * per) * 8;
  if (t >= u.n) return;
  float v[8] = {};
  join_parts(u, t, j, v);
  store8<YT>(u.out, t * u.ldo + j, v, (int)min((int64_t)8, u.rows - j), u.vec_out);
}


// ---------------------------------------------------------------- preparation
// Everything that has to be laid out before the products, in one launch of
// workgroups that each do one piece: they are small, and a launch each took
// longer than the work.

// Two tiles of 64 x 64, by 512 threads each: 16 bytes a load and a store.
GPTQ_DEV void transpose_piece(const TransposeArgs& v, int64_t b, uint16_t (&tiles)[2][64][72]) {
  uint16_t (&tile)[64][72] = tiles[threadIdx.x >> 9];
  const int64_t row_tiles = (v.ldd + 63) / 64, ct_n = (v.cols + 63) / 64;
  b = 2 * b + (threadIdx.x >> 9);
  const int64_t bt = b / row_tiles, rt = b - bt * row_tiles, a = bt / ct_n, ct = bt - a * ct_n;
  const int64_t i0 = rt * 64, j0 = ct * 64;
  const int r = (threadIdx.x & 511) >> 3, k = 8 * (threadIdx.x & 7);
  u32x4 x = {0u, 0u, 0u, 0u};
  if (b < v.tiles && i0 + r < v.rows && j0 + k < v.cols)
    x = load8(v.src + (a * v.rows + i0 + r) * v.cols + j0 + k, (int)min((int64_t)8, v.cols - j0 - k), v.vec);
  *reinterpret_cast<u32x4*>(&tile[r][k]) = x;
  __syncthreads();
  if (b < v.tiles && j0 + r < v.cols && i0 + k < v.ldd) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (uint32_t)tile[k + 2 * e][r] | ((uint32_t)tile[k + 2 * e + 1][r] << 16);
    *reinterpret_cast<u32x4*>(v.dst + (a * v.cols + j0 + r) * v.ldd + i0 + k) = x;
  }
}

GPTQ_DEV void pad_piece(const PadArgs& v, int64_t n, int64_t b) {
  const int64_t i = b * 1024 + threadIdx.x, per = v.kp >> 3, t = i / per, k = (i - t * per) * 8;
  if (t >= n) return;
  u32x4 x = {0u, 0u, 0u, 0u};
  if (k < v.d) x = load8(v.src + t * v.lds + k, (int)min((int64_t)8, v.d - k), false);
  *reinterpret_cast<u32x4*>(v.dst + t * v.kp + k) = x;
}

// Tokens of one adapter placed in ascending order from `at` on; `in` says whose.
// Returns the place after the last.  No atomics, so the order is fixed.
template <class In>
GPTQ_DEV int64_t place_tokens(int64_t n, int64_t at, int32_t* order, int (&count)[16], const In& in) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int64_t t0 = 0; t0 < n; t0 += 1024) {
    const int64_t t = t0 + threadIdx.x;
    const bool mine = t < n && in(t);
    const uint64_t mask = __ballot(mine);
    if (lane == 0) count[w] = __popcll(mask);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      before += i < w ? count[i] : 0;
      all += count[i];
    }
    if (mine) order[at + before + __popcll(mask & ((1ull << lane) - 1))] = (int32_t)t;
    at += all;
    __syncthreads();
  }
  return at;
}

// Tokens for which `in` holds, counted by the workgroup.
template <class In>
GPTQ_DEV int64_t count_tokens(int64_t n, int (&count)[16], const In& in) {
  int c = 0;
  for (int64_t t = threadIdx.x; t < n; t += 1024) c += in(t);
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) c += __shfl_xor(c, m);
  if ((threadIdx.x & 63) == 0) count[threadIdx.x >> 6] = c;
  __syncthreads();
  int64_t all = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) all += count[i];
  __syncthreads();
  return all;
}

__global__ __launch_bounds__(1024) void prepare_adapters_kernel(PrepareArgs g) {
  __shared__ __align__(16) uint16_t tile[2][64][72];
  __shared__ int count[16];
  const Adapters& ad = g.ad;
  const int64_t n = g.n;
  // an adapter as an unsigned number, m where a token has none
  auto key = [&](int64_t t) { return min((uint32_t)adapter_of(ad, t, n), (uint32_t)ad.m); };
  int64_t b = blockIdx.x;
  if (b < g.order_blocks) {
    // all tokens by adapter, ascending, those without one last
    const uint32_t a = (uint32_t)b;
    const int64_t at = count_tokens(n, count, [&](int64_t t) { return key(t) < a; });
    place_tokens(n, at, g.order, count, [&](int64_t t) { return key(t) == a; });
    return;
  }
  b -= g.order_blocks;
  if (b < g.list_blocks) {
    // an adapter's tokens from a multiple of 32 on: with c tokens of the adapters
    // before it, list a starts at 32 (ceil(c / 32) + a), and the next one starts
    // at least count + 1 places further
    const uint32_t a = (uint32_t)b;
    const int64_t c = count_tokens(n, count, [&](int64_t t) { return key(t) < a; });
    const int64_t first = 32 * ((c + 31) / 32 + a);
    const int64_t at = place_tokens(n, first, g.list, count, [&](int64_t t) { return key(t) == a; });
    const int64_t next = 32 * ((c + at - first + 31) / 32 + a + 1);
    for (int64_t i = at + threadIdx.x; i < next; i += 1024) g.list[i] = -1;
    if (threadIdx.x == 0) {
      g.start[a] = (int32_t)first;
      g.count[a] = (int32_t)(at - first);
      if ((int)a == ad.m - 1) g.start[a + 1] = (int32_t)next;
    }
    return;
  }
  b -= g.list_blocks;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (b < g.turn[i].blocks) return transpose_piece(g.turn[i], b, tile);
    b -= g.turn[i].blocks;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (b < g.pad[i].blocks) return pad_piece(g.pad[i], n, b);
    b -= g.pad[i].blocks;
  }
}

// Place of the k-th term of 16 rank rows and 32 places in the list: a block of 64
// lanes' operands, each of eight places of one row (lane = row + 16 (place / 8)), so
// that a wave loads it in one run (rows of whole lists touched 64 places per load).
GPTQ_DEV int64_t terms_at(int64_t block, int rows, int k, int rank) {
  return ((block * ((rank + 15) >> 4) + rows) * 3 + k) * 512;
}

// The rank values in list order, transposed and split into three bf16 terms: the
// gradients' operand as it is loaded; the rows that fill the last 16 stay as they
// are, their sums are dropped.  One thread per rank row and eight places;
// it joins the parts that down_tiles_kernel left, and keeps the joined values
// where `keep` says so.
__global__ __launch_bounds__(256) void sorted_terms_kernel(TermsArgs g) {
  const int rank = g.ad.rank;
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t one = g.places / 8 * rank;
  const int which = i < one ? 0 : 1;
  if (which) i -= one;
  const int64_t p8 = i / rank * 8;
  const int p = (int)(i % rank);
  if (p8 >= g.start[g.ad.m]) return;
  float* S = g.S[which];
  const int splits = g.splits[which];
  const float* part = S + down_values(g.n, rank);
  // every load unconditional (places without a token read token 0)
  int tok[8];
  float v[8], f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) tok[e] = g.list[p8 + e];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t t = max(tok[e], 0);
    v[e] = splits == 1 ? S[t * rank + p] : part[t * rank + p];
    const int a = splits == 1 || !g.ad.alpha ? -1 : adapter_of(g.ad, t, g.n);
    f[e] = a >= 0 ? g.ad.alpha[a] : 1.f;
  }
  for (int s = 1; s < splits; ++s)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += part[((int64_t)s * g.n + max(tok[e], 0)) * rank + p];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = tok[e] >= 0 ? v[e] * f[e] : 0.f;
    if (splits > 1 && g.keep[which] && tok[e] >= 0) S[(int64_t)tok[e] * rank + p] = v[e];
  }
  u32x4 k[3];
  split8<3>(v, k);
#pragma unroll
  for (int u = 0; u < 3; ++u)
    *reinterpret_cast<u32x4*>(g.terms[which] + terms_at(p8 >> 5, p >> 4, u, rank) + ((p & 15) + 16 * ((p8 >> 3) & 3)) * 8) = k[u];
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
// join_kernel.  4096 tokens of 11008 and 4096 columns, rank 64, take 57 us, 2.2 TB/s of
// rows.
template <int DT, int RT>
__global__ __launch_bounds__(256) void grad_kernel(GradArgs g) {
  const int lane = threadIdx.x & 63, m = lane & 15, kq = lane >> 4;
  int64_t b = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const GradProblem& q = g.p[b < g.p[0].items ? 0 : 1];
  if (b >= g.p[0].items) b -= g.p[0].items;
  if (b >= q.items) return;
  const int rank = g.ad.rank, splits = q.splits;
  const int64_t cols = q.cols, ldz = q.ldz;
  const uint16_t* terms = q.terms;
  const uint16_t* Z = q.Z;
  const int32_t* order = g.list;
  const int rb = (int)(b % g.rank_blocks);   // neighbours: they read the same rows of Z
  b /= g.rank_blocks;
  const int64_t cb = b % q.col_blocks;
  b /= q.col_blocks;
  const int split = (int)(b % splits);
  const int a = (int)(b / splits);
  const int64_t first = g.start[a];
  const int count = g.count[a];
  // columns past the end of Z's rows (a multiple of 8) repeat the last eight, whose
  // results are dropped
  const int64_t jv = cb * 128 + 8 * m;
  const int64_t j0 = min(jv, q.width - 8);
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
      f.z[e] = *reinterpret_cast<const u32x4*>(Z + (int64_t)t * ldz + j0);
    }
#pragma unroll
    for (int p = 0; p < RT; ++p)
#pragma unroll
      for (int k = 0; k < 3; ++k)
        f.v[p][k] = *reinterpret_cast<const u32x4*>(terms + terms_at((first >> 5) + blk, min(p0 + 16 * p, rank - 1) >> 4, k, rank) + 8 * lane);
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
  float* to = q.G + ((int64_t)split * g.ad.m + a) * rank * cols;
#pragma unroll
  for (int p = 0; p < RT; ++p) {
    const int pr = p0 + 16 * p + 4 * kq;
    if (q.up) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (jv + u < cols && pr < rank) *reinterpret_cast<floatx4*>(to + (jv + u) * rank + pr) = acc[p][u];   // rank % 8 == 0
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (pr + i >= rank) continue;
        float* o = to + (int64_t)(pr + i) * cols + jv;
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

__global__ __launch_bounds__(256) void join_kernel(JoinArgs g) {
  int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int which = i < g.n[0] ? 0 : 1;
  if (which) i -= g.n[0];
  const int64_t n = g.n[which];
  if (i >= n) return;
  const float* part = g.part[which];
  floatx4 v = *reinterpret_cast<const floatx4*>(part + i);
  for (int s = 1; s < g.splits[which]; ++s) v += *reinterpret_cast<const floatx4*>(part + s * n + i);
  *reinterpret_cast<floatx4*>(g.out[which] + i) = v;
}

// Parts of the contraction of down_tiles_kernel: enough workgroups for the
// chip, two steps of 64 at least in each.
int down_splits(int64_t n, int64_t d) {
  const int64_t tiles = (n + 63) / 64, steps = (d + 63) / 64;
  int64_t splits = 512 / tiles;
  splits = splits < steps / 2 ? splits : steps / 2;
  return splits < 1 ? 1 : (splits > 8 ? 8 : (int)splits);
}

// Whether each token is taken by itself: a few of them, or at least one stored adapter
// for every four of them, so that a tile of 32 places would hold eight and more if all
// are in use.  Adapters added to 1024 tokens of 4096 x 4096 with rank 64, by token and
// in tiles: 201 and 621 us with one for each token, 160 and 190 with one for four, 158
// and 89 with one for eight; 256 tokens with rank 16 16 and 66, 16 and 40 in the last two.
// How many are in use only the index says, which is on the device: a large bank of
// which a batch uses few is taken token by token too (one of 256: 94 us, 27 in tiles).
bool by_token(int64_t n, int m) { return n <= 64 || n <= 4 * (int64_t)m; }

// Rank rows of a gradient wave: 32 (more do not fit its registers).
int grad_rows(int rank) { return rank <= 16 ? 16 : 32; }

// Parts of an adapter's tokens, up to 512 waves: more of them write and read more sums
// than they gain (4096 tokens, five adapters of rank 64 on 11008 x 4096: 113 us with
// 512 waves, 122 with 1024, 136 with 2048; eight of rank 32 on 8192 x 8192: 53, 69, 81).
int grad_splits(int64_t n, int m, int64_t cols, int rank) {
  if (n == 0 || cols == 0) return 1;
  const int64_t waves = (cols + 127) / 128 * m * ((rank + grad_rows(rank) - 1) / grad_rows(rank));
  int64_t splits = (512 + waves - 1) / waves;
  const int64_t most = (n + m - 1) / m / 64;   // two blocks of tokens each
  splits = splits < most ? splits : most;
  return splits < 1 ? 1 : (splits > 16 ? 16 : (int)splits);
}

int64_t align64(int64_t floats) { return (floats + 63) / 64 * 64; }

}  // namespace

// ---------------------------------------------------------------- launches
int64_t adapter_down_floats(int64_t n, int64_t d, int64_t rank) {
  const int splits = n <= 64 ? 1 : down_splits(n, d);
  return splits == 1 ? down_values(n, rank) : down_values(n, rank) + splits * n * rank;
}

int adapter_down_parts(int64_t n, int m, int64_t d) { return by_token(n, m) ? 1 : down_splits(n, d); }

bool adapter_down_fits(int64_t n, int m, int64_t rank, int problems) {
  if (by_token(n, m)) return grid_fits((problems * n * rank + 3) / 4, 256);
  return grid_fits(problems * ((n + 63) / 64) * 8, 256) && grid_fits((n * rank / 4 + 255) / 256, 256);
}

bool adapter_rows_direct(const void* X, int64_t n, int64_t d, int64_t ldx, int m) {
  return (reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0 && d % 8 == 0) || by_token(n, m);
}

bool prepare_adapters_fits(int64_t n, int64_t m, int64_t rank, int64_t r, int64_t c, int64_t padded) {
  const int64_t tiles = m * ((rank + 63) / 64) * ((r + 63) / 64 + (c + 63) / 64);
  return grid_fits(2 * m + 1 + (tiles + 2) / 2 + n * (padded / 8) / 1024 + 2, 1024);
}

void launch_prepare_adapters(const PrepareArgs& given, hipStream_t s) {
  PrepareArgs g = given;
  g.order_blocks = g.order ? g.ad.m + 1 : 0;
  g.list_blocks = g.list ? g.ad.m : 0;
  int64_t blocks = (int64_t)g.order_blocks + g.list_blocks;
  for (auto& v : g.turn) {
    v.tiles = v.src ? (v.ldd + 63) / 64 * ((v.cols + 63) / 64) * g.ad.m : 0;
    v.blocks = (v.tiles + 1) / 2;
    v.vec = v.src && reinterpret_cast<uintptr_t>(v.src) % 16 == 0 && v.cols % 8 == 0;
    blocks += v.blocks;
  }
  for (auto& v : g.pad) {
    v.kp = gemm16_depth(v.d);
    v.blocks = v.src ? (g.n * (v.kp / 8) + 1023) / 1024 : 0;
    blocks += v.blocks;
  }
  if (blocks) hipLaunchKernelGGL(prepare_adapters_kernel, dim3((unsigned)blocks), dim3(1024), 0, s, g);
}

bool adapters_want_order(int64_t n, int m, const int32_t* index) { return index && m > 1 && !by_token(n, m); }

int launch_adapter_down(const DownArgs& given, int xt, bool join, hipStream_t s) {
  DownArgs g = given;
  const dim3 block(256);
  const int problems = g.p[1].X ? 2 : 1;
  for (auto& q : g.p) {
    q.splits = 1;
    q.vec = rows_on_16(q.X, q.ldx, kBF16);
  }
  if (by_token(g.n, g.ad.m)) {
    const dim3 grid((unsigned)((problems * g.n * g.ad.rank + 3) / 4));
    if (xt == kBF16) hipLaunchKernelGGL((down_kernel<kBF16>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((down_kernel<kF16>), grid, block, 0, s, g);
    return 1;
  }
  int64_t blocks = 0;
  for (int i = 0; i < problems; ++i) {
    g.p[i].splits = down_splits(g.n, g.p[i].d);
    blocks += (g.n + 63) / 64 * g.p[i].splits;
    if (i == 0) g.blocks0 = blocks;
  }
  const dim3 grid((unsigned)blocks);
#define GPTQ_DOWN(D_)                                                                              \
  do {                                                                                             \
    if (g.ad.rank <= 16) hipLaunchKernelGGL((down_tiles_kernel<D_, 1>), grid, block, 0, s, g);     \
    else if (g.ad.rank <= 32) hipLaunchKernelGGL((down_tiles_kernel<D_, 2>), grid, block, 0, s, g); \
    else if (g.ad.rank <= 64) hipLaunchKernelGGL((down_tiles_kernel<D_, 4>), grid, block, 0, s, g); \
    else hipLaunchKernelGGL((down_tiles_kernel<D_, 8>), grid, block, 0, s, g);                     \
  } while (0)
  if (xt == kBF16) GPTQ_DOWN(kBF16);
  else GPTQ_DOWN(kF16);
#undef GPTQ_DOWN
  if (join && g.p[0].splits > 1) {
    hipLaunchKernelGGL(scale_join_kernel, dim3((unsigned)((g.n * g.ad.rank / 4 + 255) / 256)), block, 0, s, g.p[0].S, g.n, g.ad,
                       g.p[0].splits);
    return 1;
  }
  return g.p[0].splits;
}

bool adapter_up_fits(int64_t n, int m, int64_t rows) {
  return grid_fits((by_token(n, m) ? n : (n + 31) / 32) * ((rows + 255) / 256), 256);
}

bool join_rows_fits(int64_t n, int64_t rows) { return grid_fits((n * (part_width(rows) / 8) + 255) / 256, 256); }

void launch_adapter_up(const UpArgs& given, int xt, int yt, hipStream_t s) {
  UpArgs u = given;
  u.col_tiles = (u.rows + 255) / 256;
  u.vec_base = rows_on_16(u.base, u.ldb, yt);
  u.vec_out = rows_on_16(u.out, u.ldo, yt);
  if (!u.S) {
    const dim3 flat((unsigned)((u.n * (u.ldp / 8) + 255) / 256));
    if (yt == 0) hipLaunchKernelGGL((join_rows_kernel<0>), flat, dim3(256), 0, s, u);
    else if (yt == kBF16) hipLaunchKernelGGL((join_rows_kernel<kBF16>), flat, dim3(256), 0, s, u);
    else hipLaunchKernelGGL((join_rows_kernel<kF16>), flat, dim3(256), 0, s, u);
    return;
  }
  const bool few = by_token(u.n, u.ad.m), plain = u.base && !u.part && u.vec_base && u.vec_out && u.rows % 8 == 0;
  const dim3 grid((unsigned)((few ? u.n : (u.n + 31) / 32) * u.col_tiles)), block(256);
#define GPTQ_UP(D_, Y_)                                                                \
  do {                                                                                 \
    if (few && u.ad.rank <= 16) hipLaunchKernelGGL((up_kernel<D_, Y_, 1>), grid, block, 0, s, u); \
    else if (few) hipLaunchKernelGGL((up_kernel<D_, Y_, 4>), grid, block, 0, s, u);    \
    else if (plain) hipLaunchKernelGGL((up_tiles_kernel<D_, Y_, true>), grid, block, 0, s, u); \
    else hipLaunchKernelGGL((up_tiles_kernel<D_, Y_, false>), grid, block, 0, s, u);   \
  } while (0)
  if (xt == kBF16) { if (yt == 0) GPTQ_UP(kBF16, 0); else GPTQ_UP(kBF16, kBF16); }
  else { if (yt == 0) GPTQ_UP(kF16, 0); else GPTQ_UP(kF16, kF16); }
#undef GPTQ_UP
}

int64_t adapter_grad_floats(int64_t n, int m, int64_t r, int64_t c, int rank) {
  int64_t floats = 0;
  for (const int64_t cols : {c, r}) {
    const int splits = grad_splits(n, m, cols, rank);
    if (splits > 1) floats += align64(splits * m * rank * cols);
  }
  return floats;
}

bool adapter_grads_fits(int64_t n, int m, int64_t r, int64_t c, int rank) {
  const int64_t rank_blocks = (rank + grad_rows(rank) - 1) / grad_rows(rank);
  int64_t items = 0;
  for (const int64_t cols : {c, r}) items += (cols + 127) / 128 * rank_blocks * grad_splits(n, m, cols, rank) * m;
  const int64_t places = list_places(n, m);
  return places < INT32_MAX && grid_fits((2 * (places / 8) * rank + 255) / 256, 256) && grid_fits((items + 3) / 4, 256) &&
         grid_fits(((r + c) * rank * m / 4 + 255) / 256, 256);
}

void launch_adapter_grads(const TermsArgs& terms, const GradArgs& given, int zt, float* gA, float* gB, float* part, hipStream_t s) {
  const dim3 block(256);
  if (terms.n > 0)
    hipLaunchKernelGGL(sorted_terms_kernel, dim3((unsigned)((2 * (terms.places / 8) * terms.ad.rank + 255) / 256)), block, 0, s, terms);
  GradArgs g = given;
  const int rt = grad_rows(g.ad.rank);
  g.rank_blocks = (g.ad.rank + rt - 1) / rt;
  JoinArgs j{};
  for (int i = 0; i < 2; ++i) {
    GradProblem& q = g.p[i];
    float* out = i == 0 ? gA : gB;
    q.splits = grad_splits(terms.n, g.ad.m, q.cols, g.ad.rank);
    q.col_blocks = (q.cols + 127) / 128;
    q.items = q.col_blocks * g.rank_blocks * q.splits * g.ad.m;
    q.G = out;
    if (q.splits > 1) {
      const int64_t all = (int64_t)g.ad.m * g.ad.rank * q.cols;   // rank is a multiple of 8: whole vectors
      const int k = j.n[0] ? 1 : 0;
      q.G = part;
      j.part[k] = part;
      j.out[k] = out;
      j.n[k] = all;
      j.splits[k] = q.splits;
      part += align64(q.splits * all);
    }
  }
  const dim3 grid((unsigned)((g.p[0].items + g.p[1].items + 3) / 4));
  if (zt == kBF16) {
    if (rt == 16) hipLaunchKernelGGL((grad_kernel<kBF16, 1>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((grad_kernel<kBF16, 2>), grid, block, 0, s, g);
  } else {
    if (rt == 16) hipLaunchKernelGGL((grad_kernel<kF16, 1>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((grad_kernel<kF16, 2>), grid, block, 0, s, g);
  }
  if (j.n[0]) hipLaunchKernelGGL(join_kernel, dim3((unsigned)(((j.n[0] + j.n[1]) / 4 + 255) / 256)), block, 0, s, j);
}

}  // namespace gptq
