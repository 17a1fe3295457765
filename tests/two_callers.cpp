// two_callers.cpp -- two host threads that make 4-bit cache attention calls of their own
// at the same time, as fast as they can, through the C entry.
#include <atomic>
#include <thread>

#include "fa.h"

using Entry = decltype(&fa_fwd_kvcache4);
struct Call {
    const void *q;
    const fa_kv_cache4 *cache;
    const int *len;
    void *o;
    float *lse;
    int B, Hq;
    void *workspace;
    size_t bytes;
    void *stream;
};

// times calls of each; the number that did not return FA_OK
extern "C" int two_callers(Entry entry, const Call *calls, int device, int times) {
    std::atomic<int> failed{0}, ready{0};
    auto run = [&](const Call &c) {
        cudaSetDevice(device);
        for (++ready; ready.load() < 2;) {}
        for (int i = 0; i < times; ++i)
            if (entry(c.q, c.cache, c.len, c.o, c.lse, c.B, 1, c.Hq, 0.125f, 0.f, -1, FA_BF16, c.workspace, c.bytes,
                      static_cast<cudaStream_t>(c.stream)) != FA_OK)
                ++failed;
    };
    std::thread a([&] { run(calls[0]); }), b([&] { run(calls[1]); });
    a.join();
    b.join();
    return failed.load();
}
