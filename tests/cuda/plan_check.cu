// How packed prompts are cut into items (kvq_plan.cuh), on the host: prompts in order lose none, whatever they are, and
// overlapping ones make no more than the most that prompts in order can have.  Prints one line per failure.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "kvq_plan.cuh"

using namespace kvq::plan;

// items asked for and made, with every item made inside its prompt
static bool count(const std::vector<int32_t>& starts, int64_t total, int group, int64_t& asked, int64_t& made)
{
    const int64_t prompts = (int64_t)starts.size() - 1, most = most_items(prompts, total, group);
    const int tpt = kTile / group;
    asked = made = 0;
    for (int64_t s = 0; s < prompts; ++s) {
        int begin, len;
        prompt_range(starts.data(), s, total, begin, len);
        if (begin < 0 || len < 0 || begin + (int64_t)len > total) return false;
        const int n = items_of(len, tpt), m = items_left(asked, n, most);
        if (m < 0 || m > n) return false;
        if (m > 0) {
            const Item x = item_at(begin, len, m - 1, tpt);
            if (x.tok0 < 0 || x.tok0 >= len || x.keys < 1 || (x.keys - 1) * (int64_t)kTile >= len) return false;
        }
        asked += n;
        made += m;
    }
    return made <= most && most <= 0x7FFFFFFF;
}

int main()
{
    int bad = 0;
    int64_t asked, made;
    // 16384 starts that alternate between 0 and 2^20: more items than 32 bits count
    std::vector<int32_t> wild(16385);
    for (size_t i = 0; i < wild.size(); ++i) wild[i] = i % 2 ? 1 << 20 : 0;
    if (!count(wild, 1 << 20, 64, asked, made)) bad += printf("overlapping prompts: more items than the workspace holds\n");
    if (asked <= 0x7FFFFFFF) bad += printf("overlapping prompts: the case asks for %lld only\n", (long long)asked);
    const int32_t odd[][4] = {{-5, 40, 1000, 7}, {30, 10, 60, 0}, {0, 0x7FFFFFFF, 5, 0}, {-0x7FFFFFFF - 1, 0x7FFFFFFF, 0, 60}, {60, 0, 60, 0}};
    for (const auto& o : odd)
        for (int group : {1, 3, 64})
            if (!count(std::vector<int32_t>(o, o + 4), 60, group, asked, made)) bad += printf("starts %d %d ..\n", o[0], o[1]);
    srand(1);
    for (int i = 0; i < 2000; ++i) {             // in order, starts before 0 and behind the end among them
        const int group = 1 + rand() % 64, prompts = 1 + rand() % 50, span = 1 + rand() % (i % 3 ? 400 : 5);
        std::vector<int32_t> st{rand() % 20 - 10};
        for (int s = 0; s < prompts; ++s) st.push_back(st.back() + rand() % span);
        const int64_t total = 1 + rand() % (st.back() > 0 ? 2 * st.back() : 5);
        if (!count(st, total, group, asked, made) || made != asked)
            bad += printf("in order: %lld of %lld items, group %d, %d prompts\n", (long long)made, (long long)asked, group, prompts);
    }
    if (!count({0, 0x7FFFFEFF}, 0x7FFFFEFF, 64, asked, made) || made != asked) bad += printf("the longest prompt\n");
    return bad != 0;
}
