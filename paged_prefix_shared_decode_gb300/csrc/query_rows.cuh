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
    // The sequence of row r, or -1: a row behind the last sequence's.
    __device__ __forceinline__ int sequence(int r) const {
        if (!start) return r;
        if (r < start[0] || r >= start[S]) return -1;
        int lo = 0, hi = S - 1;       // the last s with start[s] <= r (empty sequences lie before it)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start[mid] <= r) lo = mid; else hi = mid - 1;
        }
        return lo;
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
    // start[s] / qt + s, so at most T / qt + S of them have rows.
    __device__ __forceinline__ bool tile(int qt, int x, int &r0, int &nr, int &s) const {
        if (qt == 1 || !start) {
            r0 = x;
            nr = 1;
            s = sequence(x);
            return s >= 0;
        }
        int lo = 0, hi = S - 1;       // the last s whose tiles begin at or before x
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start[mid] / qt + mid <= x) lo = mid; else hi = mid - 1;
        }
        s = lo;
        r0 = start[s] + (x - (start[s] / qt + s)) * qt;
        const int end = min(start[s + 1], T);
        nr = min(qt, end - r0);
        return r0 >= 0 && nr > 0;
    }
    static int64_t tiles(int64_t rows, int64_t seqs, int qt) { return rows / qt + seqs; }
};

}  // namespace
}  // namespace kvp
