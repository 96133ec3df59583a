// host.h -- what the translation units of the C ABI share on the host: the
// per-device state, the checks and the tensor-map cache (defined in
// bsfp8_api.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bsfp8.h"

namespace bsfp8 {

struct DeviceState {
    bool ready = false;
    int error = 0;               // FP8_OK, or a sticky set-up failure (e.g. wrong architecture)
    int sm_count = 0;
    uint32_t *status = nullptr;  // 256-byte device allocation, word 0 used
};

// One-time set-up of the current device.  Returns FP8_OK and fills *out.
int device_setup(DeviceState **out);

// SM cycles a device-side wait may spin (FP8_DEBUG_WAIT_LIMIT_CYCLES).
long long wait_limit();

// The pipeline stage CTA 0 never loads (FP8_DEBUG_WITHHOLD_STAGE), -1: none.
int withheld_stage();

// C (elems bf16 values, 16-byte multiples) = 0.
int zero_fill(void *C, int64_t elems, cudaStream_t stream);

// Cached tensor map of a K-major byte matrix [rows, K] with a box of 128 K
// bytes x box_rows rows, 128-byte swizzle; K and rows past the end read as 0.
int encode_kmajor(CUtensorMap *m, const void *base, int64_t rows, int64_t K, int box_rows);

// Cached tensor map of experts' gate and up rows [E, 2 I, K] for boxes of 128 columns: 16 gate
// rows and 16 up rows in turn, 128 K bytes, 128-byte swizzle; past the ends reads as 0.
int encode_gate_up(CUtensorMap *m, const void *base, int64_t E, int64_t I, int64_t K);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Kernel attributes and other one-time work of the 128-granular entry points
// (block128_api.cu); called by device_setup.
int block128_setup();

// The same of the mixture-of-experts entry points (moe_api.cu).
int moe_setup();

constexpr int64_t kLim = int64_t(1) << 30;   // 32-bit indices in the kernels keep room for a tile past the end

// Launches with programmatic stream serialization: the kernel's start overlaps the end of
// the previous one of these kernels on the stream (each waits before it touches memory).
template <typename Args>
int launch(void (*kernel)(Args), dim3 grid, int threads, int smem, int cluster, const Args &args, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess) return FP8_OK;
    (void)cudaGetLastError();   // reported here: not left for a later call
    return FP8_ERR_CUDA;
}

// The tensor-map cache may fail to allocate: no exception leaves a C entry point.
template <typename F>
int guarded(F body) {
    try {
        return body();
    } catch (...) {
        return FP8_ERR_CUDA;
    }
}

}  // namespace bsfp8
