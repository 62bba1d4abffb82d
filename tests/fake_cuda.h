/* Put in front of the library's sources in a test build (nvcc -include): the CUDA runtime's memory
 * and stream calls work on host memory, without a GPU, in the order that the runtime promises and
 * no sooner. A memset or an asynchronous copy waits in its stream's queue until something waits
 * for that stream; cudaMemset is asynchronous and goes to the default stream, which streams made
 * without blocking (as torch's are) do not wait for. */
#pragma once
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <map>
#include <vector>

#define FAKE_API extern "C" __attribute__((visibility("default"), used))

namespace fake_cuda {

inline std::map<cudaStream_t, std::vector<std::function<void()>>> queues;
struct Block {
    void* at;
    size_t bytes;
};
inline std::vector<Block> blocks;  // in the order of their allocation; never handed out again
inline int fail_allocation = -1;   // this one (counted from 0) fails

inline void run(cudaStream_t s) {
    std::vector<std::function<void()>> ops;
    ops.swap(queues[s]);
    for (auto& op : ops) op();
}
inline cudaError_t get_device(int* d) {
    *d = 0;
    return cudaSuccess;
}
inline cudaError_t set_device(int) { return cudaSuccess; }
inline cudaError_t get_properties(cudaDeviceProp* p, int) {
    std::memset(p, 0, sizeof(*p));
    p->major = 10;
    p->minor = 3;
    p->multiProcessorCount = 152;
    return cudaSuccess;
}
template <typename T>
cudaError_t allocate(T** p, size_t bytes) {
    if (static_cast<int>(blocks.size()) == fail_allocation) {
        fail_allocation = -1;
        return cudaErrorMemoryAllocation;
    }
    void* const at = std::malloc(bytes);
    if (bytes <= (1u << 20)) std::memset(at, 0xAB, bytes);  // (large ones stay untouched pages)
    blocks.push_back({at, bytes});
    *p = static_cast<T*>(at);
    return cudaSuccess;
}
inline cudaError_t release(void*) { return cudaSuccess; }
inline cudaError_t set_async(void* p, int v, size_t n, cudaStream_t s) {
    queues[s].push_back([=] { std::memset(p, v, n); });
    return cudaSuccess;
}
inline cudaError_t set(void* p, int v, size_t n) { return set_async(p, v, n, nullptr); }
inline cudaError_t copy_async(void* to, const void* from, size_t n, cudaMemcpyKind kind, cudaStream_t s) {
    if (kind == cudaMemcpyDeviceToDevice) {
        queues[s].push_back([=] { std::memcpy(to, from, n); });
        return cudaSuccess;
    }
    // Pageable host memory: the stream is waited for, then the copy made; one to the device may end
    // after the call, from a buffer of the runtime's.
    run(s);
    if (kind == cudaMemcpyDeviceToHost) {
        std::memcpy(to, from, n);
    } else {
        const auto* const bytes = static_cast<const uint8_t*>(from);
        queues[s].push_back([to, staged = std::vector<uint8_t>(bytes, bytes + n)] {
            std::memcpy(to, staged.data(), staged.size());
        });
    }
    return cudaSuccess;
}
inline cudaError_t copy(void* to, const void* from, size_t n, cudaMemcpyKind kind) {
    return copy_async(to, from, n, kind, nullptr);
}
inline cudaError_t sync_stream(cudaStream_t s) {
    run(s);
    return cudaSuccess;
}
inline cudaError_t sync_device() {
    for (auto& q : queues) run(q.first);
    return cudaSuccess;
}

}  // namespace fake_cuda

// What is still queued runs now (the device catches up).
FAKE_API inline void fake_catch_up() { fake_cuda::sync_device(); }
FAKE_API inline int fake_blocks() { return static_cast<int>(fake_cuda::blocks.size()); }
FAKE_API inline void* fake_block(int i) { return fake_cuda::blocks[i].at; }
FAKE_API inline int64_t fake_block_bytes(int i) { return static_cast<int64_t>(fake_cuda::blocks[i].bytes); }
FAKE_API inline void fake_fail_allocation(int i) { fake_cuda::fail_allocation = i; }

#undef cudaGetDeviceProperties
#define cudaGetDevice fake_cuda::get_device
#define cudaSetDevice fake_cuda::set_device
#define cudaGetDeviceProperties fake_cuda::get_properties
#define cudaMalloc fake_cuda::allocate
#define cudaFree fake_cuda::release
#define cudaMemset fake_cuda::set
#define cudaMemsetAsync fake_cuda::set_async
#define cudaMemcpy fake_cuda::copy
#define cudaMemcpyAsync fake_cuda::copy_async
#define cudaStreamSynchronize fake_cuda::sync_stream
#define cudaDeviceSynchronize fake_cuda::sync_device
