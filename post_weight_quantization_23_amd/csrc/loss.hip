// The loss over a vocabulary, around its matrix products: which tokens have a target
// and their rows, the join of the tiles' softmax statistics, and the join of the
// input gradient's parts.
#include "loss.hpp"

namespace gptq {

namespace {

// Places of the tokens that have a target, by one workgroup: 4096 tokens a turn as
// four sets of 1024, whose waves' counts are summed up by every wave for itself.
// For fp16 gradients the largest finite |dloss| is brought to 2^14 .. 2^15 by a power
// of two, so that entries of D down to 2^-28 of it are normal numbers.
__global__ __launch_bounds__(1024) void keep_kernel(KeepArgs a) {
  constexpr int SETS = 4, WAVES = 16;
  __shared__ int counts[SETS * WAVES];
  __shared__ float tops[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t before = 0;
  float top = 0.f;
  for (int64_t base = 0; base < a.n; base += SETS * 1024) {
    int64_t y[SETS];
    uint64_t has[SETS];
#pragma unroll
    for (int k = 0; k < SETS; ++k) {
      const int64_t t = base + k * 1024 + tid;
      y[k] = t < a.n ? a.target[t] : -1;
    }
#pragma unroll
    for (int k = 0; k < SETS; ++k) {
      has[k] = __ballot((uint64_t)y[k] < (uint64_t)a.vocab);
      if (lane == 0) counts[k * WAVES + wave] = __popcll(has[k]);
    }
    __syncthreads();
    int sum = counts[lane];   // inclusive over the 64 (set, wave) pairs
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int v = __shfl_up(sum, o);
      sum += lane >= o ? v : 0;
    }
#pragma unroll
    for (int k = 0; k < SETS; ++k) {
      const int64_t t = base + k * 1024 + tid;
      const int at = k * WAVES + wave, upto = at ? __shfl(sum, at - 1) : 0;
      if (t >= a.n) continue;
      const bool mine = (has[k] >> lane) & 1;
      const int64_t p = before + upto + __popcll(has[k] & ((1ull << lane) - 1));
      a.k.place_of[t] = mine ? (int32_t)p : -1;
      if (mine) {
        a.k.token[p] = (int32_t)t;
        a.k.col[p] = (int32_t)y[k];
        if (a.grad) {
          const float g = a.dloss ? a.dloss[t] : 1.f;
          a.k.lse[p] = a.lse_in[t];
          a.k.grad[p] = g;
          if (fabsf(g) < INFINITY) top = fmaxf(top, fabsf(g));
        }
      } else if (a.loss) {
        a.loss[t] = 0.f;
        a.lse[t] = 0.f;
      }
    }
    before += __shfl(sum, 63);
    __syncthreads();   // before the counts are replaced
  }
  if (tid == 0) *a.k.count = (int32_t)before;
  if (!a.grad) return;
  int e = 0;   // grad = dloss 2^e
  if (a.half) {
#pragma unroll
    for (int o = 1; o < 64; o *= 2) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    for (int i = 0; i < WAVES; ++i) top = fmaxf(top, tops[i]);
    e = top > 0.f ? min(15 - ilogbf(top) - 1, 120) : 0;
    for (int64_t p = tid; p < before; p += 1024) a.k.grad[p] = ldexpf(a.k.grad[p], e);
  }
  if (tid == 0) *a.k.down = ldexpf(1.f, -e);
  if (tid < 64 && a.d > 0) {
    // Parts of dX's contraction, a lane for each number of them: rounds of tiles over the
    // CUs (two of the smaller tiles each), at 1.75 us for 64 entries of the vocabulary, against
    // writing and reading the parts, 5 ns for 1000 values (1536 tokens of 32000 x 4096:
    // two parts and five both take 451 us).
    const int64_t tile = a.large ? 256 : 128;
    const float slots = a.large ? 256.f : 512.f, parts = lane + 1;
    const int64_t tiles = (before + tile - 1) / tile * ((a.d + tile - 1) / tile), steps = (a.width + 63) / 64;
    const bool can = lane == 0 || (lane < kMostSplits && tiles * (lane + 1) <= kMostParts && steps >= 8 * (lane + 1));
    const float us = steps * (a.large ? 1.75f : 1.f) * ceilf(tiles * parts / slots) / parts + (lane ? before * a.d * 5e-6f * parts : 0.f);
    float least = can ? us : INFINITY;
    int best = lane + 1;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const float other = __shfl_xor(least, o);
      const int of = __shfl_xor(best, o);
      if (other < least || (other == least && of < best)) least = other, best = of;
    }
    const int64_t each = (steps + best - 1) / best;   // of equal length, none empty
    if (lane == 0) *a.k.splits = steps > 0 ? (int)((steps + each - 1) / each) : 1;
  }
}

// One thread per eight columns of a token (8192 tokens of 4096: 24 us, 5.6 TB/s in and out).
template <bool DX>
__global__ __launch_bounds__(256) void gather_kernel(GatherArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = a.kp >> 3, t = i / per, k = (i - t * per) * 8;
  if (t >= a.n) return;
  const int p = a.k.place_of[t];
  if (p >= 0) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k < a.d) v = load8(a.X + t * a.ldx + k, 8, a.vec);
    *reinterpret_cast<u32x4*>(a.rows + p * a.kp + k) = v;
  } else if (DX && k < a.d) {
    const float zero[8] = {};
    store8<kBF16>(a.dX, t * a.ldd + k, zero, 8, a.vec_dx);
  }
}

// ---------------------------------------------------------------- statistics
// TOKENS tokens by 256 / TOKENS threads each, which join every so many of its tiles: kJoinTokens
// where there are enough of them, else one wave for each.
template <int TOKENS>
__global__ __launch_bounds__(256) void loss_join_kernel(LossArgs a, int tiles, float* __restrict__ loss, float* __restrict__ lse) {
  constexpr int PARTS = 256 / TOKENS;
  __shared__ float2 sums[PARTS][TOKENS + 1];
  const int tok = TOKENS == kJoinTokens ? threadIdx.x % TOKENS : threadIdx.x / PARTS, part = TOKENS == kJoinTokens ? threadIdx.x / TOKENS : threadIdx.x % PARTS;
  const int64_t p = (int64_t)blockIdx.x * TOKENS + tok, count = a.target ? a.n : *a.k.count;
  float2 v = {-INFINITY, 0.f};
  if (p < count)
    for (int i = part; i < tiles; i += 4 * PARTS) {   // four loads at once
      float2 u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = i + e * PARTS < tiles ? a.part[(int64_t)(i + e * PARTS) * a.n + p] : float2{-INFINITY, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) v = join_sums(v, u[e]);
    }
  if constexpr (PARTS == 64) {
#pragma unroll
    for (int o = 1; o < 64; o *= 2) v = join_sums(v, float2{__shfl_xor(v.x, o), __shfl_xor(v.y, o)});
    if (part != 0 || p >= count) return;
  } else {
    sums[part][tok] = v;
    __syncthreads();
    if (part != 0 || p >= count) return;
    for (int i = 1; i < PARTS; ++i) v = join_sums(v, sums[i][tok]);
  }
  const bool none = a.target && (uint64_t)a.target[p] >= (uint64_t)a.vocab;
  const int64_t t = a.target ? p : a.k.token[p];
  lse[t] = none ? 0.f : v.x + logf(v.y);
  loss[t] = none ? 0.f : (v.x - a.at_target[p]) + logf(v.y);   // not lse - z: lse is rounded at its size
}

// ---------------------------------------------------------------- input gradient
template <int DT>
__global__ __launch_bounds__(256) void join_x_kernel(GradXArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = a.d >> 3, p = i / per, j = (i - p * per) * 8;
  const int64_t count = *a.k.count;
  const int splits = *a.k.splits;
  if (p >= count || (splits == 1 && !a.pieces)) return;
  float v[8] = {};
  for (int s = 0; s < splits; ++s) {
    float u[8];
    load8f(a.part + ((int64_t)s * count + p) * a.d + j, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += u[e];
  }
  add_row<DT>(a.W0 + a.k.col[p] * a.ldw + j, a.k.rest[p], v);
  const float down = *a.k.down;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= down;
  store8<DT>(a.dX, (int64_t)a.k.token[p] * a.ldd + j, v, 8, a.vec);
}

}  // namespace

void launch_keep(const KeepArgs& a, hipStream_t s) { hipLaunchKernelGGL(keep_kernel, dim3(1), dim3(1024), 0, s, a); }

void launch_gather_kept(GatherArgs a, hipStream_t s) {
  a.vec = rows_on_16(a.X, a.ldx, kBF16);
  a.vec_dx = a.dX && rows_on_16(a.dX, a.ldd, kBF16);
  const dim3 grid((unsigned)((a.n * (a.kp / 8) + 255) / 256));
  if (a.dX) hipLaunchKernelGGL(gather_kernel<true>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(gather_kernel<false>, grid, dim3(256), 0, s, a);
}

void launch_loss_join(const LossArgs& a, float* loss, float* lse, hipStream_t s) {
  const int tiles = (int)loss_tiles(a.n, a.vocab);
  if (a.n > 1024) hipLaunchKernelGGL(loss_join_kernel<kJoinTokens>, dim3((unsigned)((a.n + kJoinTokens - 1) / kJoinTokens)), dim3(256), 0, s, a, tiles, loss, lse);
  else hipLaunchKernelGGL(loss_join_kernel<4>, dim3((unsigned)((a.n + 3) / 4)), dim3(256), 0, s, a, tiles, loss, lse);
}

void launch_join_x(const GradXArgs& a, int dt, hipStream_t s) {
  const dim3 grid((unsigned)((a.n * (a.d / 8) + 255) / 256));
  if (dt == kBF16) hipLaunchKernelGGL(join_x_kernel<kBF16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(join_x_kernel<kF16>, grid, dim3(256), 0, s, a);
}

}  // namespace gptq
