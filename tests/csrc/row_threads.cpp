// Test-only: several host threads call rowops_softmax_fwd or rowops_softmax_bwd in
// tight loops, each on rows of a length of its own.
#include <atomic>
#include <cstdint>
#include <thread>
#include <vector>

struct RowCall {
    const float *a, *b;  // x; or y and dy
    float* out;
    int64_t rows, cols;
    void* stream;
};
using Fwd = int (*)(const float*, float*, int64_t, int64_t, void*);
using Bwd = int (*)(const float*, const float*, float*, int64_t, int64_t, void*);

// The first status that is not 0.
extern "C" int row_threads(void* fn, int backward, const RowCall* calls, int n, int turns) {
    std::atomic<int> status{0}, ready{0};
    std::vector<std::thread> threads;
    for (int i = 0; i < n; ++i)
        threads.emplace_back([&, i] {
            const RowCall& c = calls[i];
            ++ready;
            while (ready.load() < n) {
            }
            for (int t = 0; t < turns && status.load() == 0; ++t) {
                const int s = backward ? reinterpret_cast<Bwd>(fn)(c.a, c.b, c.out, c.rows, c.cols, c.stream)
                                       : reinterpret_cast<Fwd>(fn)(c.a, c.out, c.rows, c.cols, c.stream);
                int none = 0;
                if (s != 0) status.compare_exchange_strong(none, s);
            }
        });
    for (auto& t : threads) t.join();
    return status.load();
}
