// The launches of the 8-bit products (i8_plan of gg_int8.h) on 256 CUs.  Built
// and run under sanitizers by tests/test_int8_plan.py.  Exit status 0 when
// every check holds.
#include <cstdio>

#include "gg_int8.h"

static int g_failed = 0, g_checked = 0;

static void check(const char* what, int M, int E, int N, int K, int tile, int group) {
    const gg::Int8Plan p = gg::i8_plan(M, E, N, static_cast<int>(gg::i8_cont_p(K)), 256);
    ++g_checked;
    if (p.tile == tile && p.group == group) return;
    ++g_failed;
    std::fprintf(stderr, "%s (M %d, E %d, N %d, K %d): tile %d, group %d, not %d, %d\n", what, M, E, N, K, p.tile, p.group,
                 tile, group);
}

int main() {
    check("one token", 8, 128, 4096, 4096, 0, 0);
    check("a small batch", 2880, 128, 3712, 2688, 128, 32);
    check("few experts", 777, 5, 2056, 1048, 128, 96);
    check("few experts, a wide sum", 777, 5, 2056, 8192, 128, 0);
    check("36 rows an expert, wide", 128 * 36, 128, 3712, 2688, 256, 0);
    check("96 rows an expert, wide", 128 * 96, 128, 3712, 2688, 128, 32);
    check("86 rows an expert", 128 * 86, 128, 1536, 2048, 128, 64);
    check("80 rows an expert", 128 * 80, 128, 4096, 4096, 128, 32);
    check("119 rows an expert", 128 * 119, 128, 2048, 768, 128, 96);
    check("120 rows an expert", 128 * 120, 128, 2048, 768, 256, 96);
    check("200 rows an expert", 128 * 200, 128, 1536, 2048, 256, 64);
    check("a training batch", 131072, 128, 2048, 768, 256, 96);
    check("the largest count", 2147483647, 1024, 131072, 131072, 256, 0);
    std::printf("%d of %d checks failed\n", g_failed, g_checked);
    return g_failed ? 1 : 0;
}
