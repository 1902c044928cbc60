// kvq_plan.cuh -- how packed prompts are cut into items (prompts.cu): arithmetic that the host can run too.
#pragma once

#include <stdint.h>

namespace kvq {
namespace plan {

constexpr int kTile = 128;                       // rows of a row tile, keys of a key tile

// Two row tiles of a prompt: tokens tok0 .. of the prompt at [begin, begin + len).
struct Item { int begin, len, tok0, keys; };     // keys: key tiles that its last row sees

struct Plan { int count, pad[63]; };             // and the items behind it

// prompt s, whatever starts holds; its items, and the i-th of them
__host__ __device__ __forceinline__ void prompt_range(const int32_t* starts, int64_t s, int64_t total, int& begin, int& len) {
    const int n = (int)total, a = starts[s], z = starts[s + 1];
    begin = a < 0 ? 0 : a < n ? a : n;
    len = (z < begin ? begin : z < n ? z : n) - begin;
}
__host__ __device__ __forceinline__ int items_of(int len, int tpt) { return (int)(((int64_t)len + 2 * tpt - 1) / (2 * tpt)); }
__host__ __device__ __forceinline__ Item item_at(int begin, int len, int i, int tpt) {
    const int tok0 = i * 2 * tpt, end = tok0 + 2 * tpt;
    return Item{begin, len, tok0, ((end < len ? end : len) + kTile - 1) / kTile};
}

// Items of prompts that do not overlap, at most.
inline int64_t most_items(int64_t prompts, int64_t total, int64_t group) {
    return total / (2 * (kTile / group)) + (prompts < total ? prompts : total);
}

// How many of a prompt's n items are made where those before it have `before`: prompts that overlap ask
// for more than `most` in all (16383 of 2^20 tokens each for more than 2^31).
__host__ __device__ __forceinline__ int items_left(int64_t before, int n, int64_t most) {
    const int64_t left = most - before;
    return left <= 0 ? 0 : left < n ? (int)left : n;
}

}  // namespace plan
}  // namespace kvq
