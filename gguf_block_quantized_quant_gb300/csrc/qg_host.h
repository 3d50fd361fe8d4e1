// qg_host.h -- host helpers shared by the translation units that hold C entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <set>
#include <utility>

namespace qg {

// SM count of the current device, or a negative status (qg_abi.cu).
int device_sms();
// SM count for planning when no device is usable: 152 then (qg_abi.cu).
int device_sms_planning();

// Asks once per kernel and device for `bytes` of dynamic shared memory (qg_attn.cu).
bool allow_smem(const void *kern, uint32_t bytes);

// Runs ask(kern) once per kernel and device and says whether it held; a failure is not remembered.  Nothing is thrown: the
// callers stand below C entry points.
template <class Ask>
bool once_per_device(std::set<std::pair<const void *, int>> &done, std::mutex &mu, const void *kern, Ask &&ask) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    try {
        const std::lock_guard<std::mutex> lock(mu);
        if (done.count({kern, dev})) return true;
        if (!ask()) return false;
        done.insert({kern, dev});
        return true;
    } catch (...) {
        return false;
    }
}

inline bool host_aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Launch with programmatic stream serialization: the kernel may start while the previous
// kernel in the stream is still running (it must griddep_wait() before touching its data).
template <class... KArgs, class... Args>
bool launch_programmatic(void (*kern)(KArgs...), dim3 grid, int block, size_t smem, cudaStream_t s, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return cudaGetLastError() == cudaSuccess;
}

}  // namespace qg
