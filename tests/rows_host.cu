// The RMS norm kernels' row index arithmetic on the host: for every small
// shape, team and vector count, which elements each thread of each row's team
// would read, and whether a row's own elements are each one thread's.
// Prints "ok <rows checked>", or the first access out of range.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "gb_rows.cuh"

static uint64_t n_checked = 0;

// Rows of one team, `per` teams a block: it has rows first, first + stride, ..
// and, as the kernels, its threads' vectors from the first of them.
template <int V> static void check(uint64_t rows, uint32_t cols, int team, uint64_t stride) {
    const uint64_t n = rows * cols, whole_to = gb::whole_rows(rows, cols);
    std::vector<int> owners(cols);
    for (uint64_t first = 0; first < stride && first < rows; ++first)
        for (uint64_t row = first; row < rows; row += stride, ++n_checked) {
            owners.assign(cols, 0);
            const bool cut = row >= whole_to;
            for (int i = 0; i < team; ++i) {
                const gb::Mine<V> m = gb::mine_of<V>(first, cols, i, team);
                const uint64_t at = row * cols - m.skew;  // a vector boundary within the tensor
                const uint32_t whole = gb::whole_vectors<V>(m, cut);
                bool bad = at % 8 != 0 || m.skew < 0 || (uint64_t)m.skew > row * cols;
                for (int v = 0; v < V; ++v) {
                    if (!(m.has >> v & 1)) continue;
                    const uint64_t p = at + 8 * (uint64_t)(i + v * team);
                    const int lo = m.head >> v & 1 ? m.lo : 0, hi = m.tail >> v & 1 ? m.hi : 8;
                    if (whole >> v & 1) bad |= p + 8 > n;
                    else bad |= !(m.tail >> v & 1) || p + hi > n;
                    for (int k = lo; k < hi && !bad; ++k) {
                        const uint64_t e = p + k;
                        if (e < row * cols || e >= (row + 1) * cols) bad = true;
                        else ++owners[e - row * cols];
                    }
                }
                if (bad) {
                    printf("%llu x %u, V %d, team %d, row %llu, thread %d\n", (unsigned long long)rows, cols, V, team,
                           (unsigned long long)row, i);
                    exit(1);
                }
            }
            for (uint32_t c = 0; c < cols; ++c)
                if (owners[c] != 1) {
                    printf("%llu x %u, V %d, team %d: column %u has %d threads\n", (unsigned long long)rows, cols, V, team, c,
                           owners[c]);
                    exit(1);
                }
        }
}

template <int V> static void shapes(uint64_t rows, uint32_t cols) {
    const int team = gb::team_of(cols, V);
    if (team == 0) return;
    check<V>(rows, cols, team, 8);       // a team walks over several rows, a multiple of 8 apart
    check<V>(rows, cols, team, 1 << 20); // one row a team
}

int main() {
    for (uint32_t cols = 1; cols <= 330; cols += cols < 40 ? 1 : 7)
        for (uint64_t rows = 1; rows <= (cols < 40 ? 70 : 19); ++rows) {
            shapes<1>(rows, cols);
            shapes<2>(rows, cols);
            shapes<3>(rows, cols);
            shapes<4>(rows, cols);
        }
    const uint32_t wide[] = {2047, 4089, 4096, 8191, 8192, 16377, 16384, 16385};
    for (uint32_t cols : wide)
        for (uint64_t rows = 1; rows <= 9; ++rows) {
            shapes<1>(rows, cols);
            shapes<2>(rows, cols);
            shapes<4>(rows, cols);
        }
    printf("ok %llu\n", (unsigned long long)n_checked);
    return 0;
}
