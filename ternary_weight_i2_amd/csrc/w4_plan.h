// w4_plan.h -- which launch a product with 4-bit weights takes (w4.hip: the kernels).  Host
// arithmetic on the call's sizes, without HIP.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace bitnet {

// tt: tiles of 16 tokens to a workgroup of eight waves, rt: tiles of 16 rows to a wave, wk: the
// waves that share a tile's blocks of 128 channels; the workgroups over rows and tokens, and
// the shares of the blocks that are summed afterwards.
struct W4Plan {
    int tt, rt, wk;
    int64_t rows, tokens;
    int shares;
};
// Measured in graphs, bf16 (the shares' sums are a second launch of about 2 us).
inline W4Plan w4_plan(int64_t N, int64_t M, int64_t K) {
    const int64_t tiles = (M + 15) / 16, blocks = K / 128, units = 256;   // compute units
    W4Plan p;
    p.tt = N <= 16 ? 1 : N <= 32 ? 2 : 4;
    p.rt = p.wk = p.shares = 1;
    p.tokens = (N + 16 * p.tt - 1) / (16 * p.tt);
    if (p.tt == 1) {
        // Four waves to a unit at least, first by sharing tiles (a token times 2560 x 2560: 11.0 us with
        // one wave to a tile, 9.2 with two, 7.5 with four), then, of many blocks, by shares of
        // at least 16 for up to 16 waves (8192 x 8192: 14.0 us with two waves and four shares, 19.7
        // with four waves, 26 with two; 28672 x 8192: 32 us with two shares, 36 to 40 with
        // more waves to a tile).
        while (p.wk < 4 && 2 * p.wk <= blocks && tiles * p.wk < 4 * units) p.wk *= 2;
        p.rows = (tiles * p.wk + 7) / 8;
        p.shares = (int)std::max<int64_t>(std::min(blocks / 16, 16 * units / (tiles * p.wk)), 1);
        return p;
    }
    // Two tiles to a wave halve what is read of the operands in LDS, if they leave a workgroup to
    // each unit with shares of eight blocks.
    p.rt = (tiles + 15) / 16 * p.tokens * std::max<int64_t>(blocks / 8, 1) >= units ? 2 : 1;
    p.rows = (tiles + 8 * p.rt - 1) / (8 * p.rt);
    p.shares = (int)std::max<int64_t>(
        std::min({units / (p.rows * p.tokens), blocks / 4, (int64_t)32}), 1);
    return p;
}

}  // namespace bitnet
