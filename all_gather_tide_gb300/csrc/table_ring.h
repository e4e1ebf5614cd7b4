// Ring of per-call pointer tables: pinned host copy, device copy, reused while the contents and the
// stream stay the same.  Shared by the group object and the tensor list.
#pragma once

#include <cstdint>
#include <cstring>
#include <vector>

#include <cuda_runtime.h>

namespace tide {

constexpr int kSlots = 4;  // pointer-table ring depth

// One entry of the ring of pointer tables.  The host copy is pinned so the upload is a true
// asynchronous copy on the caller's stream; `done` is recorded after the kernel that reads the
// device copy, so the slot is only rewritten once that kernel has finished.
struct Slot {
    std::vector<const void*> content;
    const void** host = nullptr;
    void** dev = nullptr;
    cudaEvent_t done = nullptr;
    unsigned long long stream = 0;  // its id: a handle may mean another stream later, or in another thread
    uint64_t last_use = 0;
    bool valid = false;
    bool pending = false;
};

struct TableRing {
    Slot slots[kSlots];
    uint64_t use_clock = 0;

    // Slots of `words` 8-byte entries each, in one pinned and one device block.
    cudaError_t create(size_t words) {
        const size_t bytes = kSlots * words * sizeof(void*);
        cudaError_t e = cudaHostAlloc(reinterpret_cast<void**>(&slots[0].host), bytes, cudaHostAllocDefault);
        if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&slots[0].dev), bytes);
        for (int k = 0; k < kSlots && e == cudaSuccess; ++k) {
            slots[k].host = slots[0].host + k * words;
            slots[k].dev = slots[0].dev + k * words;
            e = cudaEventCreateWithFlags(&slots[k].done, cudaEventDisableTiming);
        }
        return e;
    }

    // Waits for the work that reads the slots, then frees them.
    void release() {
        for (Slot& s : slots) {
            if (!s.done) continue;
            cudaEventSynchronize(s.done);
            cudaEventDestroy(s.done);
        }
        if (slots[0].host) cudaFreeHost(slots[0].host);
        if (slots[0].dev) cudaFree(slots[0].dev);
        for (Slot& s : slots) s = Slot{};
    }

    // A table given in parts, one after the other, each of whole 8-byte entries.
    struct Part {
        const void* data;
        size_t words;
    };

    // The index of a slot that already holds this table for this stream, or -1.
    int find(const Part* parts, int count, cudaStream_t stream) {
        unsigned long long id;
        if (cudaStreamGetId(stream, &id) != cudaSuccess) return -1;  // put() reports it
        for (int k = 0; k < kSlots; ++k) {
            Slot& s = slots[k];
            if (!s.valid || s.stream != id) continue;
            size_t at = 0;
            bool same = true;
            for (int i = 0; i < count && same; ++i) {
                same = at + parts[i].words <= s.content.size() &&
                       std::memcmp(s.content.data() + at, parts[i].data, parts[i].words * sizeof(void*)) == 0;
                at += parts[i].words;
            }
            if (!same || at != s.content.size()) continue;
            s.last_use = ++use_clock;
            return k;
        }
        return -1;
    }

    // Uploads a table that find() did not find and returns its slot's index.  The caller calls
    // finish(k) after its launch.
    cudaError_t put(const Part* parts, int count, cudaStream_t stream, int* slot) {
        unsigned long long id;
        if (const cudaError_t e = cudaStreamGetId(stream, &id); e != cudaSuccess) return e;
        // victim: an unused slot, else the least recently used one
        int k = -1;
        for (int i = 0; i < kSlots && k < 0; ++i)
            if (!slots[i].valid) k = i;
        if (k < 0) {
            k = 0;
            for (int i = 1; i < kSlots; ++i)
                if (slots[i].last_use < slots[k].last_use) k = i;
        }
        Slot& s = slots[k];
        if (s.pending) {
            const cudaError_t e = cudaEventSynchronize(s.done);
            if (e != cudaSuccess) return e;
        }
        s.valid = false;
        s.content.clear();
        for (int i = 0; i < count; ++i) {
            const auto* from = static_cast<const void* const*>(parts[i].data);
            s.content.insert(s.content.end(), from, from + parts[i].words);
        }
        const size_t bytes = s.content.size() * sizeof(void*);
        std::memcpy(s.host, s.content.data(), bytes);
        const cudaError_t e = cudaMemcpyAsync(s.dev, s.host, bytes, cudaMemcpyHostToDevice, stream);
        if (e != cudaSuccess) return e;
        s.stream = id;
        s.valid = true;
        s.last_use = ++use_clock;
        *slot = k;
        return cudaSuccess;
    }

    // Uploads `ptrs` into a ring slot, or finds a slot already holding the same table for the same
    // stream, and returns its index.
    cudaError_t upload(const std::vector<const void*>& ptrs, cudaStream_t stream, int* slot) {
        const Part part{ptrs.data(), ptrs.size()};
        *slot = find(&part, 1, stream);
        return *slot >= 0 ? cudaSuccess : put(&part, 1, stream, slot);
    }

    cudaError_t finish(int k, cudaStream_t stream) {
        Slot& s = slots[k];
        const cudaError_t e = cudaEventRecord(s.done, stream);
        if (e == cudaSuccess) s.pending = true;
        return e;
    }
};

}  // namespace tide
