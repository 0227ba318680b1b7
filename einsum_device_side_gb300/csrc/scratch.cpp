// scratch.cpp -- small workspace that a stream keeps.
//
// A pool block costs its call an event and a look at every block still retiring (several us of host
// time when calls follow one another closely).  Calls that need a few MB take them here instead: one
// block per (device, stream, host thread), used by one call after the other in stream order, so that
// nothing has to be retired.  The thread is part of the key because two threads may enqueue on one
// stream at once, and their calls' launches then interleave.  A larger request replaces the block;
// the old one, which earlier launches may still use, is kept until tropical_release_pool.
#include <cuda_runtime.h>

#include <atomic>
#include <map>
#include <mutex>
#include <tuple>
#include <vector>

#include "internal.h"

namespace trop {
namespace {

struct Kept {
    void* p;
    size_t bytes;
};
using Key = std::tuple<int, cudaStream_t, uint64_t>;
struct Scratch {
    std::mutex mu;
    std::map<Key, Kept> blocks;
    std::vector<std::pair<int, void*>> replaced;
};
Scratch& scratch()
{
    static Scratch* s = new Scratch();
    return *s;
}
uint64_t thread_number()
{
    static std::atomic<uint64_t> next{0};
    static thread_local const uint64_t mine = next.fetch_add(1);
    return mine;
}

}  // namespace

bool stream_scratch(size_t bytes, cudaStream_t s, void** out)
{
    if (bytes > SCRATCH_MOST || capture_arena()) return false;
    // a captured launch outlives the call, and is replayed on other streams: its workspace is its own
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone) {
        cudaGetLastError();
        return false;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    Scratch& S = scratch();
    std::lock_guard<std::mutex> lk(S.mu);
    Kept& k = S.blocks[Key(dev, s, thread_number())];
    if (k.bytes < bytes) {
        size_t want = 65536;
        while (want < bytes) want *= 2;
        void* p = nullptr;
        if (cudaMalloc(&p, want) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        if (k.p) S.replaced.emplace_back(dev, k.p);
        k = Kept{p, want};
    }
    *out = k.p;
    return true;
}

void release_scratch()
{
    Scratch& S = scratch();
    std::lock_guard<std::mutex> lk(S.mu);
    for (auto& b : S.blocks)
        if (b.second.p) {
            cudaSetDevice(std::get<0>(b.first));
            cudaFree(b.second.p);
        }
    for (auto& r : S.replaced) {
        cudaSetDevice(r.first);
        cudaFree(r.second);
    }
    S.blocks.clear();
    S.replaced.clear();
}

}  // namespace trop
