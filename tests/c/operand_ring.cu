/* A model of the product's ring of operand stages on the CPU: the warp that loads, as
 * the kernels do it, leaves by leave_ring (csrc/operand_ring.cuh); loads, matrix
 * instructions and their commits run beside it in an order drawn from a seed.  Built
 * as a host-only shared library by tests/test_operand_ring.py. */
#include "operand_ring.cuh"

#include <cstdint>
#include <deque>
#include <random>
#include <vector>

namespace {

template <int STAGES>
struct Model {
    std::mt19937 rng;
    int64_t gives_up_at;                       // the block that the instructions do not take any more
    int64_t full[STAGES] = {}, empty[STAGES] = {};  // completed phases
    int64_t issued = 0;                        // blocks whose instructions have been issued
    std::vector<int> loads;                    // stages with a load in flight
    std::deque<int> commits;                   // stages with a commit in flight, in order

    // One thing that happens by itself; false if nothing can.
    bool step() {
        const bool can_land = !loads.empty(), can_commit = !commits.empty();
        const bool can_issue = issued < gives_up_at && full[issued % STAGES] > issued / STAGES;
        const int choices = int(can_land) + int(can_commit) + int(can_issue);
        if (!choices) return false;
        int pick = int(rng() % unsigned(choices));
        if (can_land && pick-- == 0) {
            const size_t i = rng() % loads.size();
            ++full[loads[i]];
            loads.erase(loads.begin() + long(i));
        } else if (can_commit && pick-- == 0) {
            ++empty[commits.front()];
            commits.pop_front();
        } else {
            commits.push_back(int(issued++ % STAGES));
        }
        return true;
    }
    // A bounded wait: runs out when nothing can happen any more.
    bool wait(const int64_t &completed, uint32_t parity) {
        while (uint32_t(completed & 1) == parity)
            if (!step()) return false;
        return true;
    }
    int64_t run(int64_t blocks, bool *ok) {
        int64_t filled = 0;
        *ok = true;
        for (; filled < blocks; ++filled) {
            const int s = int(filled % STAGES);
            if (filled >= STAGES && !wait(empty[s], uint32_t(filled / STAGES - 1) & 1u)) {
                *ok = false;
                break;
            }
            loads.push_back(s);
            for (unsigned k = rng() % 3; k && step(); --k) {
            }
        }
        const bool left = tr::leave_ring<STAGES>(
            filled, [&](int s, uint32_t p) { return wait(empty[s], p); }, [&](int s, uint32_t p) { wait(full[s], p); });
        *ok = *ok && left;
        // What would arrive after the block has left.
        return int64_t(loads.size() + commits.size());
    }
};

template <int STAGES>
long long walk(long long blocks, long long gives_up_at, unsigned seed, int *ok) {
    Model<STAGES> m;
    m.rng.seed(seed);
    m.gives_up_at = gives_up_at;
    bool good;
    const int64_t n = m.run(blocks, &good);
    *ok = good;
    return n;
}

}  // namespace

extern "C" long long ring_leftovers(int stages, long long blocks, long long gives_up_at, unsigned seed, int *ok) {
    switch (stages) {
        case 2: return walk<2>(blocks, gives_up_at, seed, ok);
        case 3: return walk<3>(blocks, gives_up_at, seed, ok);
        case 4: return walk<4>(blocks, gives_up_at, seed, ok);
        case 5: return walk<5>(blocks, gives_up_at, seed, ok);
    }
    return -1;
}
