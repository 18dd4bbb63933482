// model_ops_probe.cc -- prints the library's choices for gemm_xent and
// embed_rows_grad, compiled with a plain C++ compiler against the library's own
// policy header (tests/test_model_ops_policy.py drives it).
//
//   xent  M N sm_count forward     -> "cta_group tile_n"
//   panel M N tile_n               -> "rows"
//   piece rows N                   -> "columns"
//   sum   M K n sm_count last      -> "cta_group tile_n splits used each used_of_last"
//   chunk M                        -> "tokens"
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "policy.h"

int main(int argc, char** argv) {
    using namespace libgemm;
    auto arg = [&](int i) { return i < argc ? std::atoll(argv[i]) : 0ll; };
    if (argc < 3) return 1;
    if (std::strcmp(argv[1], "xent") == 0) {
        const XentShape s = plan_xent(arg(2), arg(3), (int)arg(4), arg(5) != 0);
        std::printf("%d %d\n", s.cta_group, s.tile_n);
    } else if (std::strcmp(argv[1], "panel") == 0) {
        std::printf("%lld\n", (long long)xent_panel_rows(arg(2), arg(3), (int)arg(4)));
    } else if (std::strcmp(argv[1], "piece") == 0) {
        std::printf("%lld\n", (long long)xent_piece_cols(arg(2), arg(3)));
    } else if (std::strcmp(argv[1], "sum") == 0) {
        const XentSumPlan p = plan_xent_sum(arg(2), arg(3), arg(4), (int)arg(5));
        const long long each = p.each(arg(4)), kb = (arg(6) + 63) / 64;
        std::printf("%d %d %d %d %lld %lld\n", p.shape.cta_group, p.shape.tile_n, p.splits,
                    p.used(arg(4)), each, (kb + each - 1) / each);
    } else if (std::strcmp(argv[1], "chunk") == 0) {
        std::printf("%d\n", embed_chunk(arg(2)));
    } else {
        return 1;
    }
    return 0;
}
