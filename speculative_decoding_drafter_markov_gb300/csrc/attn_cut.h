// attn_cut.h -- arithmetic of the attention's work that needs no GPU: any C++
// compiler takes it, so that the CPU can walk it to the ends of its ranges.
#pragma once

#ifdef __CUDACC__
#define DSPARK_CUT __device__ __forceinline__
#else
#define DSPARK_CUT inline
#endif

namespace dspark {
namespace attn {

DSPARK_CUT int least(int a, int b) { return a < b ? a : b; }

// The token by which a copying lane finds its page: the first of box b (of `box`
// tokens) of tile t.  There are lanes for more boxes than a tile has: those look where
// its last box does, so that no token number passes the end of the tile, the only one
// that is known to fit 32 bits; nor does any pass the unit's last token.
DSPARK_CUT int lookup_token(int t, int tile_log2, int b, int box, int last) {
    return least((t << tile_log2) + least(b * box, (1 << tile_log2) - box), last);
}

}  // namespace attn
}  // namespace dspark
