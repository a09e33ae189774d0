// How ns_moe_sort deals its slots to workgroups. Plain C++, so that a program
// without a GPU can check it over the whole range of slots.
#pragma once

#include <cstdint>

namespace nsq {

constexpr int kSortThreads = 512;
constexpr int kMaxSortBlocks = 256;
constexpr int kOneRounds = 4;   // most rounds of one workgroup by itself

struct SortSplit {
    int32_t per;      // slots of a workgroup: a multiple of kSortThreads
    int32_t blocks;   // one: a single launch
};

// One workgroup up to 4 rounds of 512 slots (2048 slots: 4.9 us; 4096: 9.3, two launches 6.4), past that two
// launches over up to 256 workgroups (524288 slots of 256 experts: 128 workgroups 15.5 us, 512 25). `slots` is
// below 2^31, but a sum that rounds it up is not: 64 bits throughout.
inline SortSplit sort_split(int64_t slots) {
    const int64_t rounds = (slots + kSortThreads - 1) / kSortThreads;
    const int64_t per = rounds == 0 ? 1 : rounds <= kOneRounds ? rounds : (rounds + kMaxSortBlocks - 1) / kMaxSortBlocks;
    return {(int32_t)(per * kSortThreads), rounds == 0 ? 1 : (int32_t)((rounds + per - 1) / per)};
}

}  // namespace nsq
