// Query rows of a ragged batch held on the device (sm_103a): which sequence a
// row belongs to, its position, and the pages that it sees.
#pragma once
#include <cstdint>

namespace kvp {
namespace {

// Rows of sequence s: start[s] .. start[s + 1] - 1 (start null: row s), its
// last cached tokens.  A length above MB * bs counts as that.
struct QueryRows {
    const int32_t *start, *tables, *lens;
    int32_t S, T, MB, bs;

    __device__ __forceinline__ int begin(int s) const { return start ? start[s] : s; }
    __device__ __forceinline__ int len(int s) const {
        return (int)min((int64_t)max(lens[s], 0), (int64_t)MB * bs);
    }
    // The last sequence s for which below(s) holds, 0 if it does for none; it
    // holds up to some sequence.  By whole warps, 32 places at a time: each turn
    // is a load's latency, and one finds a sequence of 32, two of 1024.
    template <class Below>
    __device__ __forceinline__ int last(Below below) const {
        int lo = 0, n = S;
        while (n > 1) {
            const int step = (n + 31) >> 5, at = (threadIdx.x & 31) * step;
            const uint32_t m = __ballot_sync(0xffffffffu, at < n && below(lo + at));
            const int k = m ? 31 - __clz(m) : 0;
            lo += k * step;
            n = min(step, n - k * step);
        }
        return lo;
    }
    // The sequence of row r, or -1: a row behind the last sequence's.  (Of empty
    // sequences and the one behind them the last.)  By whole warps.
    __device__ __forceinline__ int sequence(int r) const {
        if (!start) return r;
        if (r < start[0] || r >= start[S]) return -1;
        return last([&](int s) { return start[s] <= r; });
    }
    // Position of row r of sequence s; negative for a query without a token.
    __device__ __forceinline__ int position(int s, int r) const {
        const int n = len(s);
        return min(n - begin(s + 1) + r, n - 1);
    }
    // Pages that it sees.
    __device__ __forceinline__ int pages(int s, int r) const {
        const int p = position(s, r);
        return p < 0 ? 0 : p / bs + 1;
    }
    // Tile x of at most qt consecutive rows of one sequence: tiles start anew
    // at every sequence's first row.  The tiles of sequence s begin at index
    // start[s] / qt + s, so at most T / qt + S of them have rows.  By whole warps.
    __device__ __forceinline__ bool tile(int qt, int x, int &r0, int &nr, int &s) const {
        if (qt == 1 || !start) {
            r0 = x;
            nr = 1;
            s = sequence(x);
            return s >= 0;
        }
        s = last([&](int i) { return start[i] / qt + i <= x; });
        r0 = start[s] + (x - (start[s] / qt + s)) * qt;
        const int end = min(start[s + 1], T);
        nr = min(qt, end - r0);
        return r0 >= 0 && nr > 0;
    }
    static int64_t tiles(int64_t rows, int64_t seqs, int qt) { return rows / qt + seqs; }
};

}  // namespace
}  // namespace kvp
