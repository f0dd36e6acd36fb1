// Row index arithmetic of the RMS norm's kernels: which elements each thread of
// a team has, and which of its vectors may be read whole.  Host code too, so
// that it can be checked without a GPU.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace gb {

// A row's elements start at any element, and the buffers at 16 bytes.  Row
// tensors of one shape share their offsets, so a team of threads covers a row
// from the vector boundary at or before its first element, `skew` elements
// ahead: vector v of thread i has elements p - skew .. p - skew + 7 of the
// row, p = 8 (i + v team).  A team is a power of two of a warp's lanes for
// short rows, else whole warps, one team a block (in the forward kernel), and
// its rows lie a multiple of 8 apart: the skew, and with it what each thread
// has, stays the same from row to row.
constexpr int kMaxTeam = 512;

template <int V> struct Mine {
    int skew, lo, hi;    // its end vectors' own parts: [lo, 8) of the first, [0, hi) of the last
    uint32_t has;        // bit v: some of vector v is the row's
    uint32_t head, tail; // bit v: but not all of it, at the row's start / end
};
template <int V>
__host__ __device__ __forceinline__ Mine<V> mine_of(uint64_t row, uint32_t cols, int i, int team) {
    Mine<V> m{(int)(row * cols & 7), 0, 8, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int pos = 8 * (i + v * team), lo = m.skew - pos, hi = m.skew + (int)cols - pos;
        if (hi <= 0) continue;
        m.has |= 1u << v;
        if (lo > 0) {
            m.head |= 1u << v;
            m.lo = lo;
        }
        if (hi < 8) {
            m.tail |= 1u << v;
            m.hi = hi;
        }
    }
    return m;
}

// Rows below this one may be read in whole vectors: row r's last vector ends
// at element round_up((r + 1) cols, 8), within the tensor's rows * cols
// elements exactly when r + 1 <= floor(floor(rows * cols / 8) * 8 / cols).
// Narrow rows are why it is no matter of the last row alone: the last vector
// of every row that ends within 7 elements of the tensor's end is cut by it.
__host__ __device__ __forceinline__ uint64_t whole_rows(uint64_t rows, uint32_t cols) {
    return (rows * cols & ~(uint64_t)7) / cols;
}
// The vectors that a thread reads whole of a row (bit v); of its others, the
// tail's if it has one, it reads its own elements.
template <int V>
__host__ __device__ __forceinline__ uint32_t whole_vectors(const Mine<V> &m, bool cut) {
    return m.has & ~(cut ? m.tail : 0u);
}

// Threads of a team with V vectors each that hold a row of cols elements (and
// its skew); 0 if that is more than kMaxTeam.
inline int team_of(uint32_t cols, int V) {
    const uint64_t need = ((uint64_t)cols + (cols % 8 ? 7 : 0) + 8 * V - 1) / (8 * V);
    if (need > kMaxTeam) return 0;
    if (V > 1 || need > 32) return (int)(need + 31) / 32 * 32;
    int t = 1;
    while ((uint64_t)t < need) t *= 2;
    return t;
}

}  // namespace gb
