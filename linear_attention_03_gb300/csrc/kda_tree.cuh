// kda_tree.cuh -- the tree of drafted tokens shared by the tree kernels.
// Node m of a sequence hangs below node parent[m] < m, or directly below the
// tokens that came before it (-1).  Any other value means that m is no node,
// and then nothing below m is one.
#pragma once

#include <stdint.h>

#include "kda.h"

namespace kda {

constexpr int kMaxTreeNodes = KDA_MAX_TREE_NODES;   // one bit each in a 64-bit set

// m and the nodes above it, one bit each; 0 when m is no node.  The walk goes
// to ever smaller indices, so it ends after at most m + 1 steps.
__device__ __forceinline__ uint64_t tree_line(const int32_t *parent, int m) {
    uint64_t line = 0;
    for (int at = m;;) {
        line |= uint64_t{1} << at;
        const int p = parent[at];
        if (p == -1) return line;
        if (p < 0 || p >= at) return 0;
        at = p;
    }
}

}  // namespace kda
