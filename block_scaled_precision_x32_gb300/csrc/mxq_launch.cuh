// mxq_launch.cuh -- launches that overlap with the end of the kernel in front
// of them in the stream.  On a GB300 about 2.5 us pass between two dependent
// kernels of a stream, as long as the smallest ones here run; launched this
// way a kernel's blocks start, and set themselves up, while the last blocks of
// the one in front are still running.  (8192x8192 weight, one token, calls
// back to back: 18.1 -> 15.6 us.)
//
// A kernel launched so calls wait_for_stream() before it touches memory.  One
// that allocates tensor memory calls let_next_start() after that: a block of
// a kernel behind it that took the columns first, and then waited for this
// one to end, would keep it from ever ending.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace mxq {

// The next kernel of the stream may start its blocks where this one's leave
// room, once all of this one's have called this ...
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// ... and here waits until everything in front of it in the stream is done and visible.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Allows `kernel` up to `most` bytes of dynamic shared memory, once a device.
// The limit belongs to the kernel on the device, whichever host thread sets
// it: `most` is what the largest of all calls takes, so that no thread lowers
// it between another one's setting and launch.
constexpr int kDevices = 64;
template <typename... Params>
cudaError_t allow_shared_memory(void (*kernel)(Params...), size_t most, std::atomic<bool> (&allowed)[kDevices]) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess || (device < kDevices && allowed[device].load(std::memory_order_relaxed))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e == cudaSuccess && device < kDevices) allowed[device].store(true, std::memory_order_relaxed);
    return e;
}

// cluster: 0 for a launch without clusters.
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                              cudaStream_t stream, Args&&... args) {
    cudaLaunchAttribute attrs[2]{};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace mxq
