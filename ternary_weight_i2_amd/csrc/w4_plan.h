// w4_plan.h -- which launch a product with 4-bit weights takes (w4.hip: the kernels).  Host
// arithmetic on the call's sizes, without HIP.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace bitnet {

// tt: tiles of 16 tokens to a workgroup (1: the kernel of up to 16 tokens); for more tokens
// rt: tiles of 16 rows to each of its eight waves, the workgroups over rows and tokens, and
// the shares of the blocks of 128 channels that are summed afterwards.
struct W4Plan {
    int tt, rt;
    int64_t rows, tokens;
    int shares;
};
inline W4Plan w4_plan(int64_t N, int64_t M, int64_t K) {
    if (N <= 16) return W4Plan{1, 1, 0, 1, 1};
    W4Plan p;
    p.tt = N <= 32 ? 2 : 4;
    const int64_t tiles = (M + 15) / 16, blocks = K / 128, units = 256;
    p.tokens = (N + 16 * p.tt - 1) / (16 * p.tt);
    // two tiles to a wave halve what is read of the operands in LDS, if they leave enough workgroups
    // with shares of eight blocks
    p.rt = (tiles + 15) / 16 * p.tokens * std::max<int64_t>(blocks / 8, 1) >= units ? 2 : 1;
    p.rows = (tiles + 8 * p.rt - 1) / (8 * p.rt);
    const int64_t most = std::max<int64_t>(blocks / 4, 1);
    p.shares = (int)std::max<int64_t>(std::min({units / (p.rows * p.tokens), most, (int64_t)32}), 1);
    return p;
}

}  // namespace bitnet
