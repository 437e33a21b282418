// i8_choice.hip -- test-only host library: which tiles a product in 8-bit
// integers takes for a call (csrc/i8/i8_choice.hpp), so that tests can say that
// their cases reach each of them.  Runs no kernel.
#include "../../nvfp4_block_scaled_group_amd/csrc/i8/i8_choice.hpp"
#include "../../nvfp4_block_scaled_group_amd/csrc/i8/i8_token.hpp"

using namespace i8;

// kind: 0 fp32 out, 1 bf16 out, 2 gated block.  routing: 0 one projection, 1 by
// h_splits, 2 by device offsets.  Returns the shape (0 Big, 1 Mid, 2 Mid4) plus
// 3 where it runs in parts of the contraction, 6 for the kernel of few rows.
extern "C" int i8_choice(int kind, int routing, int64_t rows, int64_t n, int64_t k, int32_t E, const int64_t* h_splits) {
  if (routing == 0 && few(rows, k)) return 6;
  Routing R;
  R.num_experts = E;
  R.m_capacity = (int32_t)rows;
  R.d_offs = nullptr;
  R.d_status = nullptr;
  if (routing == 1 && host_routing(h_splits, rows, E, &R)) return -1;
  static const int32_t device = 0;  // only asked whether there is one
  if (routing == 2) R.d_offs = &device;
  const int64_t ws = routing == 0 ? kMaxWorkspace : 0;
  const Choice c = kind == 0   ? choose<kOutF32>(rows, n, k, R, routing == 0, ws)
                   : kind == 1 ? choose<kOutBf16>(rows, n, k, R, routing == 0, ws)
                               : choose<kGluSilu>(rows, n, k, R, routing == 0, ws);
  return c.shape + (c.parts > 1 ? 3 : 0);
}
