// ragged_probe.cc -- prints the host-side choices of the grouped products and
// of the adapters, compiled with a plain C++ compiler against the library's
// own policy header (tests/test_ragged_policy.py drives it).
//
//   grouped   G M N num_kb sm_count    -> "cta_group tile_w split"
//   ticket G M N num_kb sm_count       -> "0" or "1"
//   grouped_k G M N sm_count           -> "cta_group tile_w split"
//   lora M N num_kb listed slot sm_count
//       -> "cta_group tile_w split rows_blocks scan_blocks lanes shrink_w shrink_split chains"
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "policy.h"

int main(int argc, char** argv) {
    using namespace libgemm;
    auto arg = [&](int i) { return i < argc ? std::atoll(argv[i]) : 0; };
    if (argc == 7 && std::strcmp(argv[1], "grouped") == 0) {
        const RaggedShape s = plan_grouped(arg(2), arg(3), arg(4), arg(5), (int)arg(6));
        std::printf("%d %d %d\n", s.cta_group, s.tile_w, s.split);
        return 0;
    }
    if (argc == 7 && std::strcmp(argv[1], "ticket") == 0) {
        const RaggedShape s = plan_grouped(arg(2), arg(3), arg(4), arg(5), (int)arg(6));
        std::printf("%d\n", plan_grouped_ticket(s, arg(3), arg(4), arg(5), (int)arg(6)) ? 1 : 0);
        return 0;
    }
    if (argc == 6 && std::strcmp(argv[1], "grouped_k") == 0) {
        const RaggedShape s = plan_grouped_k(arg(2), arg(3), arg(4), (int)arg(5));
        std::printf("%d %d %d\n", s.cta_group, s.tile_w, s.split);
        return 0;
    }
    if (argc == 8 && std::strcmp(argv[1], "lora") == 0) {
        const LoraShape s =
            plan_lora(arg(2), arg(3), arg(4), arg(5), (int)arg(6), (int)arg(7));
        std::printf("%d %d %d %d %d %d %d %d %d\n", s.expand.cta_group, s.expand.tile_w,
                    s.expand.split, s.rows_blocks, s.scan_blocks, s.lanes, s.shrink_w, s.shrink_split, s.chains);
        return 0;
    }
    return 2;
}
