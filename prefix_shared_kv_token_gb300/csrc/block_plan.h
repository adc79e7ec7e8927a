// What the planner and the kernels over block-scaled pools agree on.
#pragma once

#include <cstddef>
#include <cstdint>

namespace pkv {

// Batches of more units than this (decode: streams; extend: requests) have the tiles before each
// written down: adding them up in every CTA of the second kernel would grow with the square of the
// batch (decode of 65,536 requests of 100 keys: 9.6 ms, with the list 2.9).
constexpr int kManyUnits = 512;

// The list of an extend call of few tokens a request, behind its workspace's header.
inline size_t block_list_bytes(int32_t batch) {
    return batch > kManyUnits ? (((size_t)batch + 1) * sizeof(int32_t) + 255) & ~size_t(255) : 0;
}

}  // namespace pkv
