// Prints sort_split's answer for every number of slots given.
#include <cstdio>
#include <cstdlib>

#include "sort_split.h"

int main(int argc, char **argv) {
    for (int i = 1; i < argc; ++i) {
        const nsq::SortSplit s = nsq::sort_split(std::atoll(argv[i]));
        std::printf("%d %d\n", s.per, s.blocks);
    }
    return 0;
}
