// sink_bwd.cuh -- how the windowed backward's work is cut into items, shared by
// the main and the finishing kernel.
//
// Per (batch, key/value head) row, key tile t has a list of G * range(t) query
// tiles: the heads of its group, one after another, each over the query tiles
// [t, t + range(t)) that see it -- the window's, or all of them for tile 0 when
// there are sinks.  A list is cut into pieces of plan.piece tiles; a tile with
// one piece writes its dK and dV itself, the pieces of the others write
// partial sums (fp32, dK with the scale) to slabs, which the finishing kernel
// adds up in order: dK and dV have the same bits on every call.
//
// Items are (piece, row) with the row fastest.  In a large problem only tile 0
// is cut, and the pieces' order is arithmetic; a problem too small to fill the
// SMs has every list cut, with a table of the tiles' first pieces (a kernel
// parameter).  A CTA with few items looks them up once, into shared memory.
#pragma once

#include "internal.h"

namespace dfa {

struct SinkItem {
    int t, row, off, n;    // key tile; row; first tile of its list and how many
    bool whole;            // the list's only piece
};

__host__ __device__ inline int sink_range(const SinkBwdPlan& p, int t) {
    if (t == 0 && p.n_sink > 0) return p.n_q;
    return p.window_tiles < p.n_q - t ? p.window_tiles : p.n_q - t;
}

__host__ __device__ inline SinkItem sink_item(const SinkBwdPlan& p, int it) {
    SinkItem x;
    const int piece = it / p.rows;
    int first;
    x.row = it % p.rows;
    if (p.cut_all) {
        int lo = 0, hi = p.n_q - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (p.first[mid] <= piece) lo = mid;
            else hi = mid - 1;
        }
        x.t = lo;
        first = p.first[lo];
    } else {
        x.t = piece < p.pieces0 ? 0 : piece - p.pieces0 + 1;
        first = x.t == 0 ? 0 : piece;
    }
    const int len = p.G * sink_range(p, x.t);
    const int size = p.cut_all || x.t == 0 ? p.piece : len;
    x.off = (piece - first) * size;
    x.n = len - x.off < size ? len - x.off : size;
    x.whole = len <= size;
    return x;
}

}  // namespace dfa
