// Launch interface of the orthogonalised adapter updates (orthogonal.hip; internal
// to the library).
#pragma once
#include "adapter.hpp"

namespace gptq {

// One factor of every adapter: m matrices of rows x cols.  p: the shorter side
// (1 .. 128), q: the longer one; tall: rows > cols.
struct OrthoProblem {
  const void* G;
  void* out;
  int64_t rows, cols;
  int64_t q;
  int p;
  bool tall;
  int splits;            // parts of q in S_0
  bool vec;              // set by the launch: four values of a row start on their multiple
  double* part;          // [m][splits][tiles][256]
  double* inv;           // [m]: 1 / (|G|_F + eps)
  double* wide;          // [m][ortho_wide]
  double* R;             // the products q .. q transposed, pp x pp of each matrix, pp: p rounded up to 16 (in
  int64_t apart;         // wide where that is used: set by the launch), this many values apart
};
struct OrthoArgs {
  int64_t m;
  int steps;
  bool first;            // S is formed from G, not from R G (set by the launch)
  double a, b, c, eps;
  OrthoProblem p[2];     // p[1].G null: one
};
constexpr int kOrthoRank = 128;
constexpr int ortho_blocks(int p) { return (p + 15) / 16; }
constexpr int ortho_tiles(int p) { return ortho_blocks(p) * (ortho_blocks(p) + 1) / 2; }
// Tile rows up to which a workgroup iterates on its own.  Calls of 1, 5 and 32 adapters beside 11008 x 4096 so and
// with a launch for each step: rank 48 49, 67 and 192 us against 56, 73 and 195; rank 64 68, 87 and 236 against
// 65, 84 and 238.
constexpr int kOrthoNarrow = 4;
// fp64 values of a matrix's buffers in memory, for the iteration over many CUs.
inline int64_t ortho_wide(int p) {
  const int64_t pp = 16 * ortho_blocks(p);
  return ortho_blocks(p) > kOrthoNarrow ? 4 * pp * pp : 0;
}
int ortho_splits(int64_t m, int64_t q, int64_t both);
bool ortho_fits(int64_t m, int64_t q);
// gt / ot: 0 fp32, 1 bf16, 2 fp16.
void launch_orthogonalize(const OrthoArgs& a, int gt, int ot, hipStream_t s);

}  // namespace gptq
