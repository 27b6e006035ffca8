// Runs csrc/mbar_wait.cuh on the host: four warps of 32 threads, the votes and
// the group's barrier by std::barrier, and mbarriers whose phase completes when
// each lane's own script says so, as it does for the lanes of a GPU when the time
// of a wait runs out at about the moment the phase completes.  Prints a line
// per scenario: how many of the 128 threads got "true".  argv[1]: the scenario.
#include <atomic>
#include <barrier>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>

#define __device__
#define __forceinline__ inline

namespace {

constexpr int kThreads = 128;
std::barrier<> group(kThreads);
std::barrier<>* warps[4];
std::atomic<int> votes[4], group_votes;
std::atomic<long long> now{0};              // the clock, moved by the scenario
int dead_word;                              // looked at through a volatile pointer, as on the GPU
thread_local int tid, looks;
int scenario;

int __all_sync(unsigned, int p)
{
    const int w = tid / 32;
    if (!p) votes[w] = 1;
    warps[w]->arrive_and_wait();
    const int r = votes[w] == 0;
    warps[w]->arrive_and_wait();
    votes[w] = 0;
    warps[w]->arrive_and_wait();
    return r;
}
bool group_all(bool ok)
{
    if (!ok) group_votes = 1;
    group.arrive_and_wait();
    const bool r = group_votes == 0;
    group.arrive_and_wait();
    if (tid == 0) group_votes = 0;
    group.arrive_and_wait();
    return r;
}
long long clock64() { return now; }
void __nanosleep(unsigned) {}

}  // namespace

namespace fp4q {

// One look.  0: the phase is complete for all.  1: never, and time runs out.
// 2: for the odd lanes from the first look on, for the even ones never.  3: for
// warp 2 never, for the others at once.  4: late, but in time.
inline bool mbar_try(uint32_t, uint32_t)
{
    ++looks;
    if (scenario != 0 && scenario != 4) now += 1ll << 24;
    switch (scenario) {
    case 0: return true;
    case 1: return false;
    case 2: return tid % 2 == 1;
    case 3: return tid / 32 != 2;
    default: return looks > 70 + tid % 3;
    }
}

}  // namespace fp4q

#include "mbar_wait.cuh"

int main(int argc, char** argv)
{
    if (argc < 2) return 2;
    scenario = std::atoi(argv[1]);
    for (auto& w : warps) w = new std::barrier<>(32);
    std::atomic<int> in_warp[4]{}, in_group{0};
    std::vector<std::thread> threads;
    for (int i = 0; i < kThreads; ++i)
        threads.emplace_back([&, i] {
            tid = i;
            if (fp4q::mbar_wait(0, 0, &dead_word)) ++in_warp[i / 32];
            group.arrive_and_wait();
            if (i == 0) dead_word = 0, now = 0;
            group.arrive_and_wait();
            looks = 0;
            if (group_all(fp4q::mbar_wait_long(0, 0, &dead_word))) ++in_group;
        });
    for (auto& t : threads) t.join();
    std::printf("warps %d %d %d %d group %d dead %d\n", (int)in_warp[0], (int)in_warp[1], (int)in_warp[2], (int)in_warp[3],
                (int)in_group, dead_word);
    std::fflush(stdout);
    std::_Exit(0);
}
