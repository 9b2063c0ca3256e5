// Which rows the quantization of the 8-bit products takes (i8_first_row and
// i8_rows_at of gg_int8.h, the kernel's own), for every small [lo, hi):
// each row of it, and no other, from any number of waves.  Built and run under sanitizers by
// tests/test_int8_rows.py.  Exit status 0 when every check holds.
#include <cstdio>
#include <vector>

#include "gg_int8.h"

static int g_failed = 0, g_checked = 0;

template <int Y>
static void check(int M, int lo, int hi, int waves) {
    std::vector<int> taken(M, 0);
    int outside = 0;
    for (int w = 0; w < waves; ++w)
        for (int64_t r0 = gg::i8_first_row<Y>(lo, hi) + Y * w; r0 < hi; r0 += Y * waves) {
            int64_t row[Y];
            gg::i8_rows_at<Y>(r0, lo, hi, row);
            for (int64_t r : row) {
                if (r < lo || r >= hi) ++outside;
                else ++taken[r];
            }
            if (Y == 2 && row[0] != row[Y - 1] && (row[0] % 2 != 0 || row[Y - 1] != row[0] + 1)) ++outside;   // a pair shares its lines
        }
    bool ok = outside == 0;
    for (int r = 0; r < M; ++r) ok &= (taken[r] > 0) == (r >= lo && r < hi) && taken[r] <= Y;
    ++g_checked;
    if (!ok) {
        ++g_failed;
        std::fprintf(stderr, "%d rows at a time, %d waves, rows [%d, %d) of %d: wrong rows\n", Y, waves, lo, hi, M);
    }
}

int main() {
    const int M = 13;
    for (int lo = 0; lo <= M; ++lo)
        for (int hi = 0; hi <= M; ++hi)      // also hi < lo: offsets that decrease
            for (int waves : {1, 3, 8}) {
                check<1>(M, lo, hi, waves);
                check<2>(M, lo, hi, waves);
            }
    std::printf("%d of %d checks failed\n", g_failed, g_checked);
    return g_failed ? 1 : 0;
}
