// The matrix products of the loss over a vocabulary: logits, whose tiles leave as
// softmax statistics or as gradients, and the two products of those gradients.
// One main loop: 16-bit operands through LDS (double buffered, asynchronous
// loads, one barrier a step), each either contiguous along the contraction or
// across it.  Operands across it are read from LDS transposed (ds_read_b64_tr), so
// that neither W, the rows nor the gradients are ever laid out a second time.
// Tiles of 256 x 256 run at 1.26 PFLOP/s for statistics (8192 tokens of 128000 x 4096, matrix
// cores busy 67 % at the 1.75 GHz that the power limit leaves), and of 4096 tokens
// of 32000 x 4096 at 1.17 for D (its 262 MB written), 1.28 for dX and 1.10 for dW.
#include "loss.hpp"

namespace gptq {

namespace {

typedef __attribute__((address_space(3))) unsigned char lds_u8;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

constexpr int LK = 64;   // contraction step
constexpr int kOutside = 0x7FFFFFFF;   // an offset past every record

// An operand: E entries (rows of A, columns of B) of a tile and LK values of the
// contraction.  Along: entry f's LK values are 128 bytes, chunk c (16 bytes)
// at place c ^ swz(f).  Across: the entries of one k are 2 E bytes, granule g (16
// entries) at place g ^ turn(k): the eight pieces of 32 bytes that a transposed read
// of 32 lanes touches (4 k, 2 granules) lie in different banks.
GPTQ_DEV int swz(int f) { return (f ^ (f >> 3)) & 7; }
template <int E>
GPTQ_DEV int turn(int k) { return ((2 * (k & 3)) ^ ((k >> 3) & 1)) & (E / 16 - 1); }

struct Source {
  const uint16_t* p;
  int64_t ld;
  int64_t entries;   // rows of an operand along the contraction, columns of one across it
  int64_t depth;     // values of the contraction; along it a multiple of 8
};

template <bool ACROSS, int E, int NW>
struct Operand {
  static constexpr int BYTES = E * LK * 2, Q = BYTES / 1024 / NW;   // load instructions per wave
  static_assert(Q * 1024 * NW == BYTES, "operand divides over the waves");
  const uint16_t* base;
  int64_t ld, depth;
  int left;          // entries of the tile that exist
  int off[Q];

  GPTQ_DEV void set(const Source& s, int64_t e0, int wave, int lane) {
    base = ACROSS ? s.p + e0 : s.p + e0 * s.ld;
    ld = s.ld;
    depth = s.depth;
    left = (int)min(s.entries - e0, (int64_t)(ACROSS ? (int64_t)1 << 30 : E));
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if constexpr (ACROSS) {
        constexpr int CH = E / 8, KR = 64 / CH;   // chunks of a k, k of an instruction
        const int k = (wave * Q + q) * KR + lane / CH, c = lane % CH;
        off[q] = (int)((k * ld + 8 * (2 * ((c >> 1) ^ turn<E>(k)) + (c & 1))) * 2);
      } else {
        const int row = 8 * (wave * Q + q) + (lane >> 3);
        off[q] = (int)((row * ld + 8 * ((lane & 7) ^ swz(row))) * 2);
      }
    }
  }

  // Values k0 .. k0 + LK - 1 to LDS; what does not exist reads as zero.
  GPTQ_DEV void load(lds_u8* to, int64_t k0, int wave, int lane) const {
    const int ks = (int)max((int64_t)0, min(depth - k0, (int64_t)LK));   // none past the end
    if constexpr (ACROSS) {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(base + k0 * ld), (short)0, ks > 0 ? (int)(((ks - 1) * ld + min(left, (int)ld)) * 2) : 0, 0x00020000);
#pragma unroll
      for (int q = 0; q < Q; ++q) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to + (wave * Q + q) * 1024, 16, off[q], 0, 0, 0);
    } else {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(base + k0), (short)0, ks > 0 ? (int)(((left - 1) * ld + ks) * 2) : 0, 0x00020000);
      if (ks == LK) {
#pragma unroll
        for (int q = 0; q < Q; ++q) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to + (wave * Q + q) * 1024, 16, off[q], 0, 0, 0);
      } else {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int row = 8 * (wave * Q + q) + (lane >> 3);
          const int at = 8 * ((lane & 7) ^ swz(row)) < ks ? off[q] : kOutside;
          __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to + (wave * Q + q) * 1024, 16, at, 0, 0, 0);
        }
      }
    }
  }

  // Addresses of the fragments of 32 entries each from f0 on (a multiple of 32; of 32 COUNT
  // where COUNT is a power of two).  Both places are exclusive ors of
  // bits of their own, so what changes with the step's values k and
  // the set i is a constant offset beside few registers:
  //   along   f * 128 + ((2 k + h) ^ swz(f)) * 16: one for each k, 32 entries 4096 bytes apart
  //           (their odd sets exclusive or 64, which is another k's)
  //   across  one for each set, k values 32 E bytes apart
  template <int COUNT>
  struct Fragments {
    static constexpr int REGS = ACROSS ? COUNT : LK / 16, READS = ACROSS ? 2 * COUNT : COUNT;
    uint32_t at[REGS];

    GPTQ_DEV void set(const lds_u8* from, int f0, int lane) {
      const uint32_t base = (uint32_t)(uintptr_t)from;
      const int h = lane >> 5;
#pragma unroll
      for (int r = 0; r < REGS; ++r) {
        if constexpr (ACROSS) {
          const int i = lane & 15, g = ((f0 + 32 * r) >> 4) + ((lane >> 4) & 1), k = 8 * h + (i >> 2);
          at[r] = base + k * (2 * E) + ((g ^ turn<E>(k)) << 5) + (i & 3) * 8;
        } else {
          const int f = f0 + (lane & 31);
          at[r] = base + f * (2 * LK) + (((2 * r + h) ^ swz(f)) << 4);
        }
      }
    }
    GPTQ_DEV void move(int by) {
#pragma unroll
      for (int r = 0; r < REGS; ++r) at[r] += by;
    }
    // Values 16 K + 8 h .. + 7 of entry f0 + 32 i + (lane & 31), of an operand along the contraction.
    template <int K>
    GPTQ_DEV void read(u32x4 (&v)[COUNT]) const {
#pragma unroll
      for (int i = 0; i < COUNT; ++i) v[i] = *(const lds_u32x4*)(uintptr_t)(at[K ^ (2 * (i & 1))] + 32 * 2 * LK * i);
    }
  };
};

// The same of operands across it, at the addresses `at`: a lane of 16 gives the address of four
// values of one k and gets four k of its own entry.  The builtin of this
// instruction waits for every asynchronous load to LDS in flight, whichever buffer it
// writes (gradients of 2048 tokens of 32000 x 4096: 907 us); these blocks wait for reads
// alone, and hold the wait themselves.
#define GPTQ_TR(out, from, off) "ds_read_b64_tr_b16 %" #out ", %" #from " offset:%" #off "\n\t"
typedef uint2 Half;   // four values
GPTQ_DEV u32x4 whole(Half lo, Half hi) { return u32x4{lo.x, lo.y, hi.x, hi.y}; }

template <int E, int K>
GPTQ_DEV void read_across(const uint32_t (&at)[2], u32x4 (&v)[2]) {
  Half a, b, c, d;
  asm volatile(GPTQ_TR(0, 4, 6) GPTQ_TR(1, 4, 7) GPTQ_TR(2, 5, 6) GPTQ_TR(3, 5, 7) "s_waitcnt lgkmcnt(0)"
               : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)
               : "v"(at[0]), "v"(at[1]), "n"(32 * E * K), "n"(32 * E * K + 8 * E)
               : "memory");
  v[0] = whole(a, b);
  v[1] = whole(c, d);
}

// Both operands: four fragments of E entries and two of F.
template <int E, int F, int K>
GPTQ_DEV void read_across(const uint32_t (&at)[4], u32x4 (&v)[4], const uint32_t (&bt)[2], u32x4 (&w)[2]) {
  Half a[8], b[4];
  asm volatile(GPTQ_TR(0, 12, 18) GPTQ_TR(1, 12, 19) GPTQ_TR(8, 16, 20) GPTQ_TR(9, 16, 21) GPTQ_TR(10, 17, 20) GPTQ_TR(11, 17, 21)
               GPTQ_TR(2, 13, 18) GPTQ_TR(3, 13, 19) GPTQ_TR(4, 14, 18) GPTQ_TR(5, 14, 19) GPTQ_TR(6, 15, 18) GPTQ_TR(7, 15, 19)
               "s_waitcnt lgkmcnt(0)"
               : "=&v"(a[0]), "=&v"(a[1]), "=&v"(a[2]), "=&v"(a[3]), "=&v"(a[4]), "=&v"(a[5]), "=&v"(a[6]), "=&v"(a[7]),
                 "=&v"(b[0]), "=&v"(b[1]), "=&v"(b[2]), "=&v"(b[3])
               : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(bt[0]), "v"(bt[1]),
                 "n"(32 * E * K), "n"(32 * E * K + 8 * E), "n"(32 * F * K), "n"(32 * F * K + 8 * F)
               : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = whole(a[2 * i], a[2 * i + 1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = whole(b[2 * i], b[2 * i + 1]);
}
#undef GPTQ_TR

// The order of READS reads of LDS and PRODUCTS matrix products: ONCE reads, a product, and so on,
// then the products that are left.
template <int READS, int PRODUCTS, int ONCE>
GPTQ_DEV void spread() {
  if constexpr (READS > 0) {
    __builtin_amdgcn_sched_group_barrier(0x100, READS < ONCE ? READS : ONCE, 0);
    if constexpr (PRODUCTS > 0) __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    spread<(READS > ONCE ? READS - ONCE : 0), (PRODUCTS > 0 ? PRODUCTS - 1 : 0), ONCE>();
  } else if constexpr (PRODUCTS > 0) {
    __builtin_amdgcn_sched_group_barrier(0x8, PRODUCTS, 0);
  }
}

template <int K>
struct At {
  static constexpr int value = K;
};

// acc = A B^T of steps first .. last - 1.  Fragments are read from LDS 16 values of
// the contraction ahead of their products, also over the end of a step: the barrier stands before
// the last 16 values' products, when their fragments are in registers, so that the
// step's buffer takes the step after the next while they run.
template <int DT, bool TA, bool TB, int MT, int NT, int WM, int WN>
struct Product {
  static constexpr int TM = 32 * MT * WM, TN = 32 * NT * WN, NW = WM * WN, BUF = (TM + TN) * LK * 2;
  typedef Operand<TA, TM, NW> OpA;
  typedef Operand<TB, TN, NW> OpB;
  typedef typename OpA::template Fragments<MT> FragA;
  typedef typename OpB::template Fragments<NT> FragB;
  // Operands along the contraction are read four fragments ahead of each product (loss of 8192
  // tokens of 128000 x 4096: 6.90 ms, one ahead 7.08).
  static constexpr int READS = FragA::READS + FragB::READS, ONCE = 4;
  static_assert(!TA || TB, "reads of operands across the contraction: of B, or of both");

  static GPTQ_DEV void run(const Source& a, const Source& b, int64_t a0, int64_t b0, int64_t first, int64_t last,
                           unsigned char* smem, floatx16 (&acc)[MT][NT]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = (wave / WN) * 32 * MT, wn = (wave % WN) * 32 * NT;
    lds_u8* lbase = (lds_u8*)smem;
    OpA oa;
    OpB ob;
    oa.set(a, a0, wave, lane);
    ob.set(b, b0, wave, lane);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int q = 0; q < NT; ++q) acc[i][q] = floatx16{};
    if (first >= last) return;
    auto load = [&](int64_t s) {
      lds_u8* to = lbase + (s & 1) * BUF;
      oa.load(to, s * LK, wave, lane);
      ob.load(to + OpA::BYTES, s * LK, wave, lane);
    };
    FragA fa;
    FragB fb;
    fa.set(lbase + (first & 1) * BUF, wm, lane);
    fb.set(lbase + (first & 1) * BUF + OpA::BYTES, wn, lane);
    u32x4 x[2][MT], y[2][NT];
    auto read = [&](auto value, int set) {
      constexpr int K = decltype(value)::value;
      if constexpr (TA) {
        read_across<TM, TN, K>(fa.at, x[set], fb.at, y[set]);
      } else {
        fa.template read<K>(x[set]);
        if constexpr (TB) read_across<TN, K>(fb.at, y[set]);
        else fb.template read<K>(y[set]);
      }
    };
    auto multiply = [&](int set) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[i][q] = mfma32<DT>(x[set][i], y[set][q], acc[i][q]);
    };
    load(first);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    load(first + 1);
    read(At<0>(), 0);
    auto quarter = [&](auto value) {   // reads values 16 K .., multiplies the ones before them
      constexpr int K = decltype(value)::value;
      read(value, K & 1);
      multiply((K & 1) ^ 1);
      if constexpr (!TB) spread<READS, MT * NT, ONCE>();
    };
    auto most = [&]() {   // a step but for its last 16 values
      quarter(At<1>());
      quarter(At<2>());
      quarter(At<3>());
    };
    for (int64_t s = first; s + 1 < last; ++s) {
      most();
      // the next step's loads have landed and this one's buffer has been read, by every wave
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      load(s + 2);
      const int by = s & 1 ? -BUF : BUF;
      fa.move(by);
      fb.move(by);
      quarter(At<0>());
    }
    most();
    multiply(1);
    __builtin_amdgcn_s_waitcnt(0);   // what was loaded past the last step
    __syncthreads();   // the last step's operands have been read
  }
};
static_assert(LK == 64, "a step is four times 16 values, the last of them in set 1");

// ---------------------------------------------------------------- tile order
// Place b of the walk over `all` tiles: of 256 workgroups, which the dispatcher deals round
// robin to the 8 XCDs, each XCD gets 32 consecutive places.  Tiles past the kept
// tokens' are not among them, so that they leave no XCD with less to do.
GPTQ_DEV int64_t place_of(int64_t b, int64_t all) {
  return b < (all & ~(int64_t)255) ? (b & ~(int64_t)255) | ((b & 7) << 5) | ((b & 255) >> 3) : b;
}
// Tile of a place: panels of 8 tiles of tokens, walked column by column.
GPTQ_DEV void tile_at(int64_t place, int tok_tiles, int col_tiles, int& tok, int& col) {
  const int64_t per = (int64_t)8 * col_tiles;
  const int panel = (int)(place / per), in = (int)(place - panel * per), h = min(8, tok_tiles - 8 * panel);
  col = in / h;
  tok = 8 * panel + in - col * h;
}

// ---------------------------------------------------------------- logits
// What becomes of a tile of WM x WN waves of 32 MT vocabulary entries (rows of the
// accumulators) x 32 NT tokens (columns): a lane holds most of a token's entries
// itself, so the largest and the sum cost one exchange between lanes.  A wave's tile starts
// at entry wm and token wn; lds is free.  Entry of a lane's value: wm + 4 (lane >> 5) + 32 i + within(e).
GPTQ_DEV constexpr int within(int e) { return 8 * (e >> 2) + (e & 3); }

// Statistics of entries v0 .. of tile vt, and the targets' logits.  Every wave of the
// workgroup calls it unless WM is 1.
template <int MT, int NT, int WM, int WN>
GPTQ_DEV void finish_loss(const LossArgs& a, floatx16 (&acc)[MT][NT], unsigned char* lds, int64_t count, int64_t t0, int64_t v0, int vt,
                          int wave) {
  constexpr int TM = 32 * MT * WM, TN = 32 * NT * WN;
  const int lane = threadIdx.x & 63, m = lane & 31, wm = (wave / WN) * 32 * MT, wn = (wave % WN) * 32 * NT;
  const int lowest = wm + 4 * (lane >> 5), last = (int)min(a.width - v0, (int64_t)TM);   // entries of this tile
  float2* part = reinterpret_cast<float2*>(lds);   // [WM][TN]
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int64_t p = t0 + wn + 32 * q + m;
    int64_t y = p < count ? (a.target ? a.target[p] : (int64_t)a.k.col[p]) : -1;
    y = (uint64_t)y < (uint64_t)a.vocab ? y - v0 : -1;   // entry of the tile
    if (last < TM) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (32 * i + within(e) >= last - lowest) acc[i][q][e] = -INFINITY;
    }
    if (__any(y >= wm && y < wm + 32 * MT)) {
      const int own = (int)y - lowest;   // in range where it counts
      float z = 0.f;
      bool mine = false;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (32 * i + within(e) == own) z = acc[i][q][e], mine = true;
      if (mine && y >= 0 && y < last) a.at_target[p] = z;
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, acc[i][q][e]);
    top = fmaxf(top, __shfl_xor(top, 32));
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) sum += __builtin_amdgcn_exp2f((acc[i][q][e] - ref) * kLog2e);
    sum += __shfl_xor(sum, 32);
    if (lane >= 32) continue;
    if constexpr (WM > 1) part[(wave / WN) * TN + wn + 32 * q + m] = float2{top, sum};
    else if (p < count) a.part[(int64_t)vt * a.n + p] = float2{top, sum};
  }
  if constexpr (WM > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < TN; c += 64 * WM * WN) {
      float2 v = part[c];
#pragma unroll
      for (int i = 1; i < WM; ++i) v = join_sums(v, part[i * TN + c]);
      if (t0 + c < count) a.part[(int64_t)vt * a.n + t0 + c] = v;
    }
  }
}

// Rows of D, rounded, a wave's tokens 32 at a time as rows of its `own` LDS (32 x
// (32 MT + 8) values), so that they leave in whole runs.
template <int DT, int MT, int NT, int WM, int WN>
GPTQ_DEV void finish_grad(const LossArgs& a, const floatx16 (&acc)[MT][NT], uint16_t* own, int64_t count, int64_t t0, int64_t v0, int wave) {
  constexpr int TM = 32 * MT * WM, W = 32 * MT, LD = W + 8, RUNS = W / 8;
  const int lane = threadIdx.x & 63, m = lane & 31, wm = (wave / WN) * 32 * MT, wn = (wave % WN) * 32 * NT;
  const int lowest = wm + 4 * (lane >> 5), last = (int)min(a.width - v0, (int64_t)TM);
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int64_t p = t0 + wn + 32 * q + m;
    const int64_t y = p < count ? (int64_t)a.k.col[p] - a.v0 - v0 : -1;
    const int own_row = (int)y - lowest;
    const float lse = p < count ? a.k.lse[p] : 0.f, g = p < count ? a.k.grad[p] : 0.f;
    float target = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        float v[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int at = 32 * i + within(e + f);
          v[f] = __builtin_amdgcn_exp2f((acc[i][q][e + f] - lse) * kLog2e);
          if (at == own_row) v[f] -= 1.f;
          v[f] = at < last - lowest ? v[f] * g : 0.f;
          target = at == own_row ? v[f] : target;
        }
        *reinterpret_cast<uint2*>(own + m * LD + 32 * i + within(e) + 4 * (lane >> 5)) = uint2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
      }
    // the lane that holds the target's entry
    if (y >= wm && y < wm + 32 * MT && ((int)y >> 2 & 1) == lane >> 5)
      a.k.rest[p] = target - f16_to_f32<DT>(f32_to_16<DT>(target));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int k = 0; k < RUNS / 2; ++k) {
      const int run = 64 * k + lane, r = run / RUNS, c = 8 * (run % RUNS);
      const int64_t at = t0 + wn + 32 * q + r;
      if (at < count && v0 + wm + c < a.ldp)
        *reinterpret_cast<u32x4*>(a.P + at * a.ldp + v0 + wm + c) = *reinterpret_cast<const u32x4*>(own + r * LD + c);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

template <int DT, bool GRAD, int MT, int NT, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void logits_kernel(LossArgs a, int voc_tiles) {
  using P = Product<DT, false, false, MT, NT, WM, WN>;
  extern __shared__ __align__(16) unsigned char lsm[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t count = !GRAD && a.target ? a.n : *a.k.count;
  const int tok_tiles = (int)((count + P::TN - 1) / P::TN);
  const int64_t all = (int64_t)tok_tiles * voc_tiles;
  if (blockIdx.x >= all) return;
  int tt, vt;
  tile_at(place_of(blockIdx.x, all), tok_tiles, voc_tiles, tt, vt);
  const int64_t t0 = (int64_t)tt * P::TN, v0 = (int64_t)vt * P::TM;
  const Source w{a.W + a.v0 * a.ldw, a.ldw, a.width, a.d}, x{a.rows, a.ldr, count, a.d};
  floatx16 acc[MT][NT];
  P::run(w, x, v0, t0, 0, (a.d + LK - 1) / LK, lsm, acc);
  if constexpr (GRAD) {
    static_assert(WM * WN * 32 * (32 * MT + 8) * 2 <= 2 * P::BUF, "results fit the operands' LDS");
    finish_grad<DT, MT, NT, WM, WN>(a, acc, reinterpret_cast<uint16_t*>(lsm) + wave * 32 * (32 * MT + 8), count, t0, v0, wave);
  } else {
    finish_loss<MT, NT, WM, WN>(a, acc, lsm, count, t0, v0, vt, wave);
  }
}

// Up to 64 tokens of a vocabulary whose tiles of 128 entries would leave most CUs idle: what
// bounds those is how long a workgroup walks along the contraction.  Here one takes 32
// entries, its eight waves share the contraction out among them, straight from memory to
// registers and without a barrier, and are added up in LDS at the end.  A token of
// 4000 x 8192 takes 26 us instead of 60, both gradients of 6 tokens of 2553 x 6376 52
// instead of 98; but pieces of 32 bytes of each row are poorer loads than LDS tiles' once there
// are enough of those.  A call on 1 and 64 tokens of 8000 x 4096 takes 19 and 36 us here, 36 and
// 41 in tiles; of 12000 x 4096 34 and 60 against 37 and 44.
constexpr int64_t kFewVocab = 8192;
constexpr int FEW_WAVES = 8;

template <int DT, bool GRAD, int NT>
__global__ __launch_bounds__(64 * FEW_WAVES) void few_kernel(LossArgs a) {
  constexpr int AHEAD = 8 / NT;   // sets of 16 values of the contraction in flight
  __shared__ __align__(16) float sums[FEW_WAVES - 1][NT][16 * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), m = lane & 31, h = lane >> 5;
  const int64_t count = !GRAD && a.target ? a.n : *a.k.count, v0 = (int64_t)blockIdx.x * 32;
  const int d = (int)a.d;
  const bool row = v0 + m < a.width;
  const uint16_t* w = a.W + (a.v0 + min(v0 + m, a.width - 1)) * a.ldw + 8 * h;
  const uint16_t* x[NT];
  bool there[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    there[q] = 32 * q + m < count;
    x[q] = a.rows + (there[q] ? 32 * q + m : 0) * a.ldr + 8 * h;
  }
  floatx16 acc[1][NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) acc[0][q] = floatx16{};
  for (int k0 = 16 * AHEAD * wave; k0 < d; k0 += 16 * AHEAD * FEW_WAVES) {
    u32x4 u[AHEAD], v[NT][AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const bool in = k0 + 16 * j + 8 * h < d;
      u[j] = u32x4{0u, 0u, 0u, 0u};
      if (row && in) u[j] = *reinterpret_cast<const u32x4*>(w + k0 + 16 * j);
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        v[q][j] = u32x4{0u, 0u, 0u, 0u};
        if (there[q] && in) v[q][j] = *reinterpret_cast<const u32x4*>(x[q] + k0 + 16 * j);
      }
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
#pragma unroll
      for (int q = 0; q < NT; ++q) acc[0][q] = mfma32<DT>(u[j], v[q][j], acc[0][q]);
  }
  if (wave > 0)
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int e = 0; e < 16; ++e) sums[wave - 1][q][64 * e + lane] = acc[0][q][e];
  __syncthreads();
  if (wave > 0) return;
#pragma unroll 1
  for (int i = 0; i < FEW_WAVES - 1; ++i)
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[0][q][e] += sums[i][q][64 * e + lane];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if constexpr (GRAD) finish_grad<DT, 1, NT, 1, 1>(a, acc, reinterpret_cast<uint16_t*>(&sums[0][0][0]), count, 0, v0, 0);
  else finish_loss<1, NT, 1, 1>(a, acc, nullptr, count, 0, v0, (int)blockIdx.x, 0);
}

// ---------------------------------------------------------------- gradients
// Stores of a wave's 32 rows x 32 NT columns times `by`, turned through its LDS.  row_at(r, also, much):
// the row's place, and optionally a row of 16-bit values `also` of which `much` is added first.
template <int OT, int NT, class F>
GPTQ_DEV void store_rows(float* lds, const floatx16 (&acc)[NT], int64_t j0, int64_t cols, bool vec, float by, F&& row_at) {
  constexpr int W = 32 * NT, RUNS = W / 8;
  const int lane = threadIdx.x & 63;
  turn_tile<NT>(lds, acc);
#pragma unroll
  for (int k = 0; k < RUNS / 2; ++k) {
    const int run = 64 * k + lane, r = run / RUNS, c = 8 * (run % RUNS);
    const uint16_t* also = nullptr;
    float much = 0.f;
    uint16_t* to = row_at(r, also, much);
    if (!to || j0 + c >= cols) continue;
    float v[8];
    load8f(lds + r * (W + 4) + c, v);
    if (also) add_row<OT>(also + j0 + c, much, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= by;
    store8<OT>(to, j0 + c, v, (int)min((int64_t)8, cols - j0 - c), vec);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// dX: tiles of TM kept tokens x TN columns, contracted over the piece's entries.
template <int DT, int MT, int NT, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void grad_x_kernel(GradXArgs a, int col_tiles) {
  using P = Product<DT, false, true, MT, NT, WM, WN>;
  extern __shared__ __align__(16) unsigned char lsm[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave / WN) * 32 * MT, wn = (wave % WN) * 32 * NT;
  const int64_t count = *a.k.count;
  const int splits = *a.k.splits, tok_tiles = (int)((count + P::TM - 1) / P::TM);
  const int64_t tiles = (int64_t)tok_tiles * col_tiles;
  if (blockIdx.x >= tiles * splits) return;
  const int64_t place = place_of(blockIdx.x, tiles * splits);
  const int split = (int)(place / tiles);
  int tt, ct;
  tile_at(place - split * tiles, tok_tiles, col_tiles, tt, ct);
  const int64_t t0 = (int64_t)tt * P::TM, j0 = (int64_t)ct * P::TN;
  const int64_t steps = (a.width + LK - 1) / LK, each = (steps + splits - 1) / splits;
  const int64_t first = min(steps, split * each), last = min(steps, first + each);
  floatx16 acc[MT][NT];
  P::run(Source{a.P, a.ldp, count, a.ldp}, Source{a.W, a.ldw, a.d, a.width}, t0, j0, first, last, lsm, acc);
  static_assert(WM * WN * 32 * (32 * NT + 4) * 4 <= 2 * P::BUF, "results fit the operands' LDS");
  float* own = reinterpret_cast<float*>(lsm) + wave * 32 * (32 * NT + 4);
  if (splits > 1 || a.pieces) {
    constexpr int W = 32 * NT, RUNS = W / 4;
    const int lane = threadIdx.x & 63;
    float* part = a.part + (int64_t)split * count * a.d;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      turn_tile<NT>(own, acc[i]);
#pragma unroll
      for (int k = 0; k < RUNS / 2; ++k) {
        const int run = 64 * k + lane, r = run / RUNS, c = 4 * (run % RUNS);
        const int64_t p = t0 + wm + 32 * i + r, j = j0 + wn + c;
        if (p >= count || j >= a.d) continue;
        floatx4 v = *reinterpret_cast<const floatx4*>(own + r * (W + 4) + c);
        floatx4* to = reinterpret_cast<floatx4*>(part + p * a.d + j);
        if (a.add) v += *to;
        *to = v;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  } else {
    const float down = *a.k.down;
#pragma unroll
    for (int i = 0; i < MT; ++i)
      store_rows<DT, NT>(own, acc[i], j0 + wn, a.d, a.vec, down, [&](int r, const uint16_t*& also, float& much) -> uint16_t* {
        const int64_t p = t0 + wm + 32 * i + r;
        if (p >= count) return nullptr;
        also = a.W0 + a.k.col[p] * a.ldw;
        much = a.k.rest[p];
        return a.dX + (int64_t)a.k.token[p] * a.ldd;
      });
  }
}

// What rounding took from the targets' entries of D, for a wave's 32 MT entries from v0 of the vocabulary on x
// 32 NT columns from j0: a product over the tokens whose targets are among them, 16 at a time in
// their order, one entry of a column of its left operand each.  A target's entry is most of a
// token's row of D, so this is most of what dW would be off by (4096 tokens of 32000 x 4096: 2.4e-3, with
// it 1.7e-3, that of its own rounding).  The wave looks through all tokens for them: both gradients take
// 2772 us there instead of 2760; dW of 8192 tokens of 1000 x 4096, eight to an entry, 390 instead of 295.
// lds: the wave's own.
template <int DT, int MT, int NT>
GPTQ_DEV void add_rest(const GradWArgs& a, floatx16 (&acc)[MT][NT], void* lds, int64_t count, int64_t v0, int64_t j0) {
  constexpr int SETS = 16, ONCE = 16, ROOM = 64 * SETS + ONCE;   // tokens looked at at once: 64 SETS
  const int lane = threadIdx.x & 63, m = lane & 31, h = lane >> 5;
  int32_t *place = static_cast<int32_t*>(lds), *entry = place + ROOM;
  static_assert(2 * ROOM <= 32 * (32 * NT + 4), "a wave's LDS");
  int have = 0;
#pragma unroll 1
  for (int64_t base = 0; base < count; base += 64 * SETS) {
    int at[SETS];
#pragma unroll
    for (int k = 0; k < SETS; ++k) {
      at[k] = a.k.col[min(base + 64 * k + lane, count - 1)] - (int)v0;
    }
#pragma unroll
    for (int k = 0; k < SETS; ++k) {
      const bool mine = base + 64 * k + lane < count && (uint32_t)at[k] < 32u * MT;
      const uint64_t all = __ballot(mine);
      if (mine) {
        const int to = have + __popcll(all & ((1ull << lane) - 1));
        place[to] = (int32_t)(base + 64 * k + lane);
        entry[to] = at[k];
      }
      have += __popcll(all);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const bool end = base + 64 * SETS >= count;
    int from = 0;
#pragma unroll 1
    for (; end ? from < have : have - from >= ONCE; from += ONCE) {
      // all loads before the first use: what does not exist is read from the last that does, and meets a
      // left operand of zero, or columns that are not stored
      u32x4 left[MT], right[NT];
      int own[8];
      float r[8];
      uint32_t x[NT][8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int of = from + 8 * h + e, p = place[min(of, have - 1)];
        own[e] = of < have ? entry[min(of, have - 1)] : -1;
        r[e] = a.k.rest[p];
#pragma unroll
        for (int q = 0; q < NT; ++q) x[q][e] = a.rows[p * a.kp + min(j0 + 32 * q + m, a.kp - 1)];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
          left[i][e] = (own[2 * e] == 32 * i + m ? f32_to_16<DT>(r[2 * e]) : 0u) | (own[2 * e + 1] == 32 * i + m ? (uint32_t)f32_to_16<DT>(r[2 * e + 1]) << 16 : 0u);
#pragma unroll
        for (int q = 0; q < NT; ++q) right[q][e] = x[q][2 * e] | x[q][2 * e + 1] << 16;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[i][q] = mfma32<DT>(left[i], right[q], acc[i][q]);
    }
    if (end) break;
    have -= from;   // fewer than 16 go first next time
    const int32_t p = place[from + (lane & 15)], e = entry[from + (lane & 15)];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (lane < have) place[lane] = p, entry[lane] = e;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// dW: tiles of TM vocabulary entries x TN columns, contracted over the kept tokens.
template <int DT, int MT, int NT, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void grad_w_kernel(GradWArgs a, int voc_tiles, int col_tiles) {
  using P = Product<DT, true, true, MT, NT, WM, WN>;
  extern __shared__ __align__(16) unsigned char lsm[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave / WN) * 32 * MT, wn = (wave % WN) * 32 * NT;
  const int64_t count = *a.k.count;
  int vt, ct;
  tile_at(place_of(blockIdx.x, (int64_t)voc_tiles * col_tiles), voc_tiles, col_tiles, vt, ct);
  const int64_t v0 = (int64_t)vt * P::TM, j0 = (int64_t)ct * P::TN;
  floatx16 acc[MT][NT];
  P::run(Source{a.P, a.ldp, a.ldp, count}, Source{a.rows, a.kp, a.kp, count}, v0, j0, 0, (count + LK - 1) / LK, lsm, acc);
  static_assert(WM * WN * 32 * (32 * NT + 4) * 4 <= 2 * P::BUF, "results fit the operands' LDS");
  float* own = reinterpret_cast<float*>(lsm) + wave * 32 * (32 * NT + 4);
  add_rest<DT, MT, NT>(a, acc, own, count, a.v0 + v0 + wm, j0 + wn);
  const float down = *a.k.down;
#pragma unroll
  for (int i = 0; i < MT; ++i)
    store_rows<DT, NT>(own, acc[i], j0 + wn, a.d, a.vec, down, [&](int r, const uint16_t*&, float&) -> uint16_t* {
      const int64_t v = v0 + wm + 32 * i + r;
      return v < a.width ? a.dW + v * a.ldd : nullptr;
    });
}

// Dynamic LDS of a kernel, set once (thread-safe).
template <class K>
void allow_lds(K kernel, int bytes) {
  (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

template <int DT, bool GRAD, int MT, int NT, int WM, int WN>   // a tile of 32 MT WM entries x 32 NT WN tokens
void logits(const LossArgs& a, hipStream_t s) {
  using P = Product<DT, false, false, MT, NT, WM, WN>;
  static const bool set = (allow_lds(logits_kernel<DT, GRAD, MT, NT, WM, WN>, 2 * P::BUF), true);
  (void)set;
  const int tt = (int)tiles_of(a.n, P::TN), vt = (int)tiles_of(a.width, P::TM);
  hipLaunchKernelGGL((logits_kernel<DT, GRAD, MT, NT, WM, WN>), dim3((unsigned)((int64_t)tt * vt)), dim3(64 * WM * WN), 2 * P::BUF, s,
                     a, vt);
}

template <int DT, bool GRAD>
void logits_shape(const LossArgs& a, hipStream_t s) {
  switch (loss_shape(a.n, a.vocab)) {
    case k256x256: return logits<DT, GRAD, 4, 2, 2, 4>(a, s);
    case k128x128: return logits<DT, GRAD, 2, 2, 2, 2>(a, s);
    case k128x64: return logits<DT, GRAD, 1, 2, 4, 1>(a, s);
    case k128x32: return logits<DT, GRAD, 1, 1, 4, 1>(a, s);
    case kFew:
      const dim3 grid((unsigned)tiles_of(GRAD ? a.ldp : a.width, 32));   // D is read up to its row stride
      if (a.n > 32) hipLaunchKernelGGL((few_kernel<DT, GRAD, 2>), grid, dim3(64 * FEW_WAVES), 0, s, a);
      else hipLaunchKernelGGL((few_kernel<DT, GRAD, 1>), grid, dim3(64 * FEW_WAVES), 0, s, a);
  }
}

template <int DT, int MT, int NT, int WM, int WN>
void grad_x(const GradXArgs& a, hipStream_t s) {
  using P = Product<DT, false, true, MT, NT, WM, WN>;
  static const bool set = (allow_lds(grad_x_kernel<DT, MT, NT, WM, WN>, 2 * P::BUF), true);
  (void)set;
  const int64_t tiles = tiles_of(a.n, P::TM) * tiles_of(a.d, P::TN);
  hipLaunchKernelGGL((grad_x_kernel<DT, MT, NT, WM, WN>), dim3((unsigned)(tiles > kMostParts ? tiles : kMostParts)), dim3(64 * WM * WN),
                     2 * P::BUF, s, a, (int)tiles_of(a.d, P::TN));
}

template <int DT, int MT, int NT, int WM, int WN>
void grad_w(const GradWArgs& a, hipStream_t s) {
  using P = Product<DT, true, true, MT, NT, WM, WN>;
  static const bool set = (allow_lds(grad_w_kernel<DT, MT, NT, WM, WN>, 2 * P::BUF), true);
  (void)set;
  const int vt = (int)tiles_of(a.width, P::TM), ct = (int)tiles_of(a.d, P::TN);
  hipLaunchKernelGGL((grad_w_kernel<DT, MT, NT, WM, WN>), dim3((unsigned)((int64_t)vt * ct)), dim3(64 * WM * WN), 2 * P::BUF, s, a, vt, ct);
}

}  // namespace

void launch_logits(const LossArgs& a, int dt, bool grad, hipStream_t s) {
  if (dt == kBF16) grad ? logits_shape<kBF16, true>(a, s) : logits_shape<kBF16, false>(a, s);
  else grad ? logits_shape<kF16, true>(a, s) : logits_shape<kF16, false>(a, s);
}

void launch_grad_x(const GradXArgs& a, int dt, hipStream_t s) {
  if (dt == kBF16) grad_x_large(a.n) ? grad_x<kBF16, 4, 2, 2, 4>(a, s) : grad_x<kBF16, 2, 2, 2, 2>(a, s);
  else grad_x_large(a.n) ? grad_x<kF16, 4, 2, 2, 4>(a, s) : grad_x<kF16, 2, 2, 2, 2>(a, s);
}

void launch_grad_w(const GradWArgs& a, int dt, hipStream_t s) {
  if (dt == kBF16) grad_w<kBF16, 4, 2, 2, 4>(a, s);
  else grad_w<kF16, 4, 2, 2, 4>(a, s);
}

// dX of 300 tokens (150 of them kept) of 32000 x 4096: 65 us in tiles of 256 x 256, 80 of 128 x 128.
bool grad_x_large(int64_t n) { return n > 128; }

// Several parts are of at most kMostParts tiles in all, one part is of all tokens.
int64_t grad_x_part_floats(int64_t n, int64_t d, bool pieces) {
  const int64_t tile = grad_x_large(n) ? 256 : 128, all = kMostSplits * n * d, parts = kMostParts * tile * tile;
  const int64_t several = all < parts ? all : parts;
  return pieces && several < n * d ? n * d : several;
}

// Of 128 x 128 tiles a CU holds two, and few tokens leave fewer of its places empty; a
// 256 x 256 tile reads half as much of LDS for a product.  Logits of 300, 517 and 1000
// tokens (50, 30 and 10 % of them without a target; 32000 x 4096, 50021 x 4096, 50021
// x 1024) took 76, 216 and 158 us in the former, 111, 225 and 174 in the latter; of
// 2048 tokens of 32000 x 4096 645 and 570.  (256 x 128: 91, 268, 170 and 680.)
LossShape loss_shape(int64_t n, int64_t vocab) {
  if (n <= 64 && vocab <= kFewVocab) return kFew;
  if (n <= 32) return k128x32;
  if (n <= 64) return k128x64;
  return n <= 1024 ? k128x128 : k256x256;
}

// Gradients of a piece are n x width 16-bit values: 512 MB.
int64_t loss_piece(int64_t n, int64_t vocab) {
  const int64_t tile = 256, least = (int64_t(1) << 28) / (n > 0 ? n : 1) / tile * tile;
  const int64_t most = least < tile ? tile : (least < (1 << 21) ? least : 1 << 21);   // rows of it are below 2^22
  return vocab <= most ? vocab : most;
}

bool loss_takes(const void* X, int64_t n, int64_t d, int64_t ldx) {
  return n <= kFewTokens && reinterpret_cast<uintptr_t>(X) % 16 == 0 && ldx % 8 == 0 && ldx < (int64_t(1) << 22);
}

bool loss_fits(int64_t n, int64_t vocab, int64_t d, bool grad) {
  constexpr int64_t tokens[] = {256, 128, 64, 32, 64};
  if (!grid_fits(tiles_of(n, tokens[loss_shape(n, vocab)]) * loss_tiles(n, vocab), 512)) return false;
  if (!grid_fits(tiles_of(n * (gemm16_depth(d) / 8), 256), 256)) return false;
  if (!grad) return grid_fits(tiles_of(n, kJoinTokens), 256);
  const int64_t tile = grad_x_large(n) ? 256 : 128;
  return grid_fits(tiles_of(n, tile) * tiles_of(d, tile), 512) && grid_fits(tiles_of(vocab, 256) * tiles_of(d, 256), 512);
}

}  // namespace gptq
