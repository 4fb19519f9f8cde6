// Test-only: several host threads call rowops_expert_plan in tight loops.
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <thread>
#include <vector>

struct PlanCall {
    const float *indices, *values;
    int32_t *offsets, *order, *slot;
    int64_t rows, k, experts;
    void* workspace;
    size_t workspace_bytes;
    void* stream;
};
using PlanFn = int (*)(const float*, const float*, int32_t*, int32_t*, int32_t*, int64_t, int64_t, int64_t, void*,
                       size_t, void*);

// Each call is made `turns` times by a thread of its own; the first status that is not 0.
extern "C" int plan_threads(void* fn, const PlanCall* calls, int n, int turns) {
    const PlanFn plan = reinterpret_cast<PlanFn>(fn);
    std::atomic<int> status{0}, ready{0};
    std::vector<std::thread> threads;
    for (int i = 0; i < n; ++i)
        threads.emplace_back([&, i] {
            const PlanCall& c = calls[i];
            ++ready;
            while (ready.load() < n) {
            }
            for (int t = 0; t < turns && status.load() == 0; ++t) {
                const int s = plan(c.indices, c.values, c.offsets, c.order, c.slot, c.rows, c.k, c.experts, c.workspace,
                                   c.workspace_bytes, c.stream);
                int none = 0;
                if (s != 0) status.compare_exchange_strong(none, s);
            }
        });
    for (auto& t : threads) t.join();
    return status.load();
}
