// launch.cuh -- the host side of a launch: a kernel's shared memory limit and
// the blocks of it that fit an SM, asked of the driver once per device, the
// number of SMs, and tensor maps.
#pragma once
#include <mutex>

#include "common.cuh"

namespace gdr {

// Every kernel is launched with one dynamic shared memory size and block size of its own, so that no call lowers a limit that
// another thread is about to launch under.  Past the table's end the driver is asked every time (a microsecond of the
// host's time).
inline cudaError_t prepare_kernel(const void *kernel, size_t smem, int threads = 0, int *blocks = nullptr) {
    constexpr int kMost = 1024;
    struct Entry {
        const void *kernel;
        int device, blocks;
    };
    static std::mutex mu;
    static Entry table[kMost];
    static int count = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < count; ++i)
        if (table[i].kernel == kernel && table[i].device == dev) {
            if (blocks) *blocks = table[i].blocks;
            return cudaSuccess;
        }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    int fit = 0, sms = 0;
    if (e == cudaSuccess && blocks) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, threads, smem);
    if (e == cudaSuccess && blocks) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (blocks) *blocks = fit * sms;
    if (count < kMost) table[count++] = Entry{kernel, dev, fit * sms};
    return cudaSuccess;
}

// SMs of the device of the first call (148 where there is none: workspace sizes are asked for on hosts too).
inline int sm_count() {
    static std::atomic<int> known{0};
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 148;
        known.store(n, std::memory_order_relaxed);
    }
    return n;
}

// A tensor map by the driver's encoder, which needs the device's context current in this thread.  The runtime makes it so at
// a thread's first call that needs it, which may be behind this one (an autograd thread, for instance).
template <typename F, typename... A>
bool encode_map(F encode, A... a) {
    if (encode(a...) == 0) return true;
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode(a...) == 0;
}

}  // namespace gdr
