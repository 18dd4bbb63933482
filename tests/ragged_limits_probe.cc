// ragged_limits_probe.cc -- prints the round-ups that the ragged kernels share
// with the host, compiled with a plain C++ compiler and its overflow checks
// against the library's own policy header (tests/test_ragged_limits.py drives
// it).
//
//   units ROWS TILE_W            -> units of a group of ROWS rows
//   width ROWS STEP MOST         -> rows that a unit of ROWS rows left spans
//   blocks K0 K_END              -> 64-deep blocks of a depth group
//   rows G M N NUM_KB SMS OUT    -> CTAs per unit of gemm_grouped (OUT: RaggedOut)
//   depth G M N SMS OUT AVG      -> CTAs per unit of gemm_grouped_k (OUT: RaggedOut)
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "policy.h"

int main(int argc, char** argv) {
    using namespace libgemm;
    auto arg = [&](int i) { return i < argc ? std::atoi(argv[i]) : 0; };
    if (argc == 4 && std::strcmp(argv[1], "units") == 0)
        std::printf("%d\n", ragged_units(arg(2), arg(3)));
    else if (argc == 5 && std::strcmp(argv[1], "width") == 0)
        std::printf("%d\n", ragged_width(arg(2), arg(3), arg(4)));
    else if (argc == 4 && std::strcmp(argv[1], "blocks") == 0)
        std::printf("%d\n", ragged_blocks(arg(2), arg(3)));
    else if (argc == 8 && std::strcmp(argv[1], "rows") == 0)
        std::printf("%d\n", plan_grouped(arg(2), arg(3), arg(4), arg(5), arg(6),
                                         (RaggedOut)arg(7)).cta_group);
    else if (argc == 8 && std::strcmp(argv[1], "depth") == 0)
        std::printf("%d\n", plan_grouped_k(arg(2), arg(3), arg(4), arg(5), (RaggedOut)arg(6),
                                           arg(7)).cta_group);
    else
        return 2;
    return 0;
}
