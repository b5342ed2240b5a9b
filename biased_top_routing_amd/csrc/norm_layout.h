// Shapes and workspace of the norm's kernels.
#pragma once

#include <algorithm>

#include "common.h"

namespace moe {

// moe_norm_backward: a workgroup of 256 lanes x 4 chunks of 16 bytes holds a row, or a panel of a longer one, or a
// wavefront of it a row of up to 256 chunks (16384 x 2048 59 -> 46 us, 16384 x 512 47 -> 18); each of at most
// kNormBwdBlocks workgroups (a panel) leaves a partial sum of dweight.  16384 x 7168: 180 us, 191 with 512 lanes x 2
// chunks, 190 with 1024 workgroups; 16384 x 2048: 46, and 48 with 1024.
constexpr int kNormBwdThreads = 256, kNormBwdChunks = 4, kNormBwdBlocks = 512;

struct NormBwdLayout {
  int blocks, panels, rows;   // rows: that a workgroup works on at a time
  size_t off_rm, off_part, total;

  explicit NormBwdLayout(const moe_cfg* c) {
    const int64_t chunks = (int64_t)c->H * (int64_t)act_bytes(c) / 16, panel = kNormBwdThreads * kNormBwdChunks;
    panels = (int)((chunks + panel - 1) / panel);
    rows = chunks <= panel / 4 ? 4 : 1;
    blocks = std::max(1, std::min((int)(((int64_t)c->T + rows - 1) / rows), kNormBwdBlocks));
    size_t o = 0;
    auto take = [&](size_t bytes) { const size_t at = o; o = align_up(o + bytes, 256); return at; };
    off_rm = take(panels > 1 ? (size_t)c->T * 8 : 0);
    off_part = take((size_t)blocks * c->H * 4);
    total = o;
  }
};

}  // namespace moe
