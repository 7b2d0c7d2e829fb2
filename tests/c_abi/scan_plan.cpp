// Reads selective scans (B T D N G, and 1 for a packed batch), a line each, and prints how each is run: lanes for a
// channel, state values in a lane, tokens of a tile, segments, tokens of a segment.
#include <cstdio>

#include "scan_plan.h"

int main() {
    long long B, T, D, N, G, packed;
    while (std::scanf("%lld %lld %lld %lld %lld %lld", &B, &T, &D, &N, &G, &packed) == 6) {
        const gdr::ScanCut cut = gdr::scan_cut(B, T, D, G, N, packed != 0);
        const gdr::ScanTile tile = gdr::scan_tile(B, D, N, G, packed != 0, cut.segs);
        std::printf("%d %d %d %d %d\n", tile.lanes, tile.states, gdr::scan_tile_tokens(tile.lanes, tile.states), cut.segs, cut.seg_len);
    }
    return 0;
}
