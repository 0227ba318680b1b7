// scratch.cpp -- the workspace of a call of the training operators.
//
// A pool block costs its call an event and a look at every block still retiring (several us of host
// time when calls follow one another closely).  Calls that need a few MB take them here instead: one
// block per (device, stream, host thread), used by one call after the other in stream order, so that
// nothing has to be retired.  The thread is part of the key because two threads may enqueue on one
// stream at once, and their calls' launches then interleave.  A thread that ends leaves its blocks to the
// next thread on their streams.  Streams are told apart by their id, which, unlike a handle, never comes
// back after the stream was destroyed with launches still on their way.  A larger request replaces the
// block; the old one, which earlier launches may still use, is kept until tropical_release_pool.
// Behind each block lies an arrival ticket, zeroed once in stream order; a call without a kept block has its
// ticket in its workspace, zeroed before its launches.
//
// Launches that the caller captures into a graph outlive the call and are replayed in any order with
// other calls: their workspace is allocated and freed by nodes of that graph, and so is its ticket.
#include <cuda_runtime.h>

#include <atomic>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

#include "internal.h"

namespace trop {
namespace {

constexpr uint64_t NOBODY = ~0ull;  // a block whose thread has ended
constexpr size_t TICKET = 256;      // bytes behind a block
constexpr size_t MOST_BLOCKS = 64;  // kept in all; calls on further streams and threads use the pool
struct Kept {
    void* p;
    size_t bytes;
    uint64_t thread;
};
using Key = std::pair<int, unsigned long long>;  // device, stream id
struct Scratch {
    std::mutex mu;
    std::map<Key, std::vector<Kept>> streams;
    size_t blocks = 0;
    std::vector<std::pair<int, void*>> replaced;
};
Scratch& scratch()
{
    static Scratch* s = new Scratch();
    return *s;
}
struct Thread {
    uint64_t number;
    Thread()
    {
        static std::atomic<uint64_t> next{0};
        number = next.fetch_add(1);
    }
    ~Thread()
    {
        Scratch& S = scratch();
        std::lock_guard<std::mutex> lk(S.mu);
        for (auto& s : S.streams)
            for (Kept& k : s.second)
                if (k.thread == number) k.thread = NOBODY;
    }
};

// A block of at most SCRATCH_MOST bytes that stays the stream's and the thread's, and its ticket; false where the pool has
// to serve.
bool stream_scratch(size_t bytes, cudaStream_t s, void** out, uint32_t** ticket)
{
    if (bytes > SCRATCH_MOST || capture_arena()) return false;
    int dev = 0;
    unsigned long long id = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaStreamGetId(s, &id) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    static thread_local const Thread me;
    Scratch& S = scratch();
    std::lock_guard<std::mutex> lk(S.mu);
    try {
        std::vector<Kept>& kept = S.streams[Key(dev, id)];
        Kept* k = nullptr;
        for (Kept& q : kept)
            if (q.thread == me.number) k = &q;
        if (!k)  // (all its launches are ahead of this call's on the stream)
            for (Kept& q : kept)
                if (q.thread == NOBODY) k = &q;
        if (!k || k->bytes < bytes) {
            if (!k && S.blocks >= MOST_BLOCKS) return false;
            size_t want = 65536;
            while (want < bytes) want *= 2;
            if (!k) kept.reserve(kept.size() + 1);  // (k points into it)
            S.replaced.reserve(S.replaced.size() + 1);
            void* p = nullptr;
            if (cudaMalloc(&p, want + TICKET) != cudaSuccess) {
                cudaGetLastError();
                return false;
            }
            if (cudaMemsetAsync((char*)p + want, 0, TICKET, s) != cudaSuccess) {
                cudaGetLastError();
                cudaFree(p);
                return false;
            }
            if (k) {
                S.replaced.emplace_back(dev, k->p);
                k->p = p;
                k->bytes = want;
            } else {
                kept.push_back(Kept{p, want, me.number});
                k = &kept.back();
                ++S.blocks;
            }
        }
        k->thread = me.number;
        *out = k->p;
        *ticket = (uint32_t*)((char*)k->p + k->bytes);
        return true;
    } catch (...) {  // no host memory for the table
        return false;
    }
}

}  // namespace

Workspace::~Workspace()
{
    if (!own) return;
    if (captured) {
        if (cudaFreeAsync(own, s) != cudaSuccess) cudaGetLastError();  // (the capture has failed: its end says so)
    } else {
        pool_retire(own, s);
    }
}

int Workspace::take()
{
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    if (!capture_arena()) {
        const cudaError_t e = cudaStreamIsCapturing(s, &status);
        if (e != cudaSuccess) return cuda_error(e, "cudaStreamIsCapturing");
    }
    captured = status != cudaStreamCaptureStatusNone;
    void* p = nullptr;
    if (captured) {
        at_ticket = add(sizeof(uint32_t));
        const cudaError_t e = cudaMallocAsync(&p, bytes, s);
        if (e != cudaSuccess) return cuda_error(e, "cudaMallocAsync (captured workspace)");
        own = p;
    } else if (!stream_scratch(bytes, s, &p, &kept_ticket)) {
        if (bytes > SCRATCH_MOST) (void)stream_scratch(0, s, &p, &kept_ticket);
        at_ticket = add(sizeof(uint32_t));  // (used where no block is kept)
        TROP_TRY(pool_alloc(bytes, s, &p));
        own = p;
    }
    base = (char*)p;
    return TROP_OK;
}

int Workspace::ticket(uint32_t** out)
{
    if (capture_arena()) return stream_tickets(s, 1, out);
    if (kept_ticket) {
        *out = kept_ticket;
        return TROP_OK;
    }
    *out = (uint32_t*)(base + at_ticket);
    const cudaError_t e = cudaMemsetAsync(*out, 0, sizeof(uint32_t), s);
    return e == cudaSuccess ? (int)TROP_OK : cuda_error(e, "cudaMemsetAsync (ticket)");
}

void release_scratch()
{
    Scratch& S = scratch();
    std::lock_guard<std::mutex> lk(S.mu);
    for (auto& s : S.streams)
        for (Kept& k : s.second) {
            cudaSetDevice(s.first.first);
            cudaFree(k.p);
        }
    for (auto& r : S.replaced) {
        cudaSetDevice(r.first);
        cudaFree(r.second);
    }
    S.streams.clear();
    S.replaced.clear();
    S.blocks = 0;
}

}  // namespace trop
