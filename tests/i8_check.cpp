// Host program for the rules of schedule.hpp that the int8 product and the operators over rows and gradients go
// by. Reads one query per line from stdin and prints one answer per line:
//   i8 M N K cus        -> kernel, reads B past the caches, tile rows, tile columns
//   back T              -> workgroups of the norm's gradient
//   grads units         -> workgroups of a launch over gradients
//   past bytes          -> whether a call's gradients go past the caches
#include <cstdint>
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>

#include "schedule.hpp"

int main() {
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string kind;
        in >> kind;
        if (kind == "i8") {
            int64_t M, N, K;
            int cus;
            in >> M >> N >> K >> cus;
            const bsfp8::sched::I8Kernel k = bsfp8::sched::i8_kernel(M, N, K, cus);
            const bsfp8::sched::I8Tile t = bsfp8::sched::kI8Tiles[k];
            std::printf("%d %d %d %d\n", k, bsfp8::sched::i8_reads_once(M, N, k, cus) ? 1 : 0, t.bm, t.bn);
        } else if (kind == "back") {
            int64_t T;
            in >> T;
            std::printf("%lld\n", (long long)bsfp8::sched::norm_backward_blocks(T));
        } else if (kind == "grads") {
            int64_t units;
            in >> units;
            std::printf("%lld\n", (long long)bsfp8::sched::grad_blocks(units));
        } else if (kind == "past") {
            double bytes;
            in >> bytes;
            std::printf("%d\n", bsfp8::sched::grads_past_caches(bytes) ? 1 : 0);
        } else {
            return 1;
        }
    }
    return 0;
}
