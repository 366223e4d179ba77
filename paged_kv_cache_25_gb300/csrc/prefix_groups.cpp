// Host: which sequences of a batch share leading blocks, as the shared-prefix decode
// takes it.
//
// Sequences are sorted by their rows of block ids; neighbours' common leading runs
// then give the tree of shared prefixes (an interval of sorted sequences for every
// branching point, built with one stack).  A group at an interval of n sequences with a
// common run of r blocks saves (n - 1) * r block reads; bottom up, an interval becomes a
// group when that is at least what the groups inside it would save.  A call takes
// PA_MAX_PREFIX_GROUPS of them: beyond that, those that save the least are let go.
#include <algorithm>
#include <cstdint>
#include <vector>

#include "../../include/pa.h"

extern "C" int pa_shared_prefix_groups(const int32_t* tables, int max_blocks, const int32_t* lens,
                                       int num_seqs, int block_size, int min_prefix_tokens,
                                       int32_t* group_of_seq, int32_t* prefix_lens)
{
    if (num_seqs < 0 || max_blocks <= 0 || block_size <= 0) return -1;
    if (num_seqs == 0) return 0;
    if (!tables || !lens || !group_of_seq || !prefix_lens) return -1;
    const int64_t need = min_prefix_tokens > block_size ? (static_cast<int64_t>(min_prefix_tokens) + block_size - 1) / block_size : 1;
    try {
        // full blocks of each sequence, up to the first unused entry
        std::vector<int> full(num_seqs), order(num_seqs);
        auto row = [&](int s) { return tables + static_cast<int64_t>(s) * max_blocks; };
        for (int s = 0; s < num_seqs; ++s) {
            const int n = std::min(std::max(lens[s], 0) / block_size, max_blocks);
            int i = 0;
            while (i < n && row(s)[i] >= 0) ++i;
            full[s] = i;
            order[s] = s;
            group_of_seq[s] = -1;
        }
        std::sort(order.begin(), order.end(), [&](int a, int b) {
            const int32_t *x = row(a), *y = row(b);
            const int n = std::min(full[a], full[b]);
            for (int i = 0; i < n; ++i)
                if (x[i] != y[i]) return x[i] < y[i];
            return full[a] != full[b] ? full[a] < full[b] : a < b;
        });
        auto common = [&](int a, int b) {
            const int32_t *x = row(a), *y = row(b);
            const int n = std::min(full[a], full[b]);
            int i = 0;
            while (i < n && x[i] == y[i]) ++i;
            return i;
        };
        struct Node {
            int run, lo, hi;              // common blocks of sorted sequences lo..hi
            int64_t saved;                // of the best choice in it
            bool group;                   // that choice is the node itself
            std::vector<int> inside;
        };
        std::vector<Node> nodes;
        std::vector<int> stack, done;     // open intervals; closed ones without a parent
        auto close = [&](int hi) {
            const int id = stack.back();
            stack.pop_back();
            Node& n = nodes[id];
            n.hi = hi;
            int64_t below = 0;
            for (int c : n.inside) below += nodes[c].saved;
            const int64_t own = n.run >= need ? static_cast<int64_t>(n.hi - n.lo) * n.run : 0;
            n.group = own > 0 && own >= below;
            n.saved = n.group ? own : below;
            return id;
        };
        for (int i = 1; i <= num_seqs; ++i) {
            const int run = i < num_seqs ? common(order[i - 1], order[i]) : 0;
            int lo = i - 1, child = -1;
            while (!stack.empty() && nodes[stack.back()].run > run) {
                if (child >= 0) nodes[stack.back()].inside.push_back(child);
                child = close(i - 1);
                lo = nodes[child].lo;
            }
            if (run > 0 && (stack.empty() || nodes[stack.back()].run < run)) {
                nodes.push_back(Node{run, lo, lo, 0, false, {}});
                stack.push_back(static_cast<int>(nodes.size()) - 1);
            }
            if (child >= 0) {
                if (stack.empty()) done.push_back(child);
                else nodes[stack.back()].inside.push_back(child);
            }
        }
        // the chosen intervals, from the outermost in
        std::vector<int> chosen;
        std::vector<int> todo(done.rbegin(), done.rend());
        while (!todo.empty()) {
            const int id = todo.back();
            const Node& n = nodes[id];
            todo.pop_back();
            if (n.group) chosen.push_back(id);
            else todo.insert(todo.end(), n.inside.rbegin(), n.inside.rend());
        }
        if (chosen.size() > PA_MAX_PREFIX_GROUPS) {
            std::stable_sort(chosen.begin(), chosen.end(),
                             [&](int a, int b) { return nodes[a].saved > nodes[b].saved; });
            chosen.resize(PA_MAX_PREFIX_GROUPS);
        }
        int groups = 0;
        for (const int id : chosen) {
            const Node& n = nodes[id];
            for (int i = n.lo; i <= n.hi; ++i) group_of_seq[order[i]] = groups;
            prefix_lens[groups++] = n.run * block_size;
        }
        return groups;
    } catch (...) {
        return -1;
    }
}
