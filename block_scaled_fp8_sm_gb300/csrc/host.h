// host.h -- what the translation units of the C ABI share on the host: the
// per-device state, the checks and the tensor-map cache (defined in
// bsfp8_api.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

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

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Kernel attributes and other one-time work of the 128-granular entry points
// (block128_api.cu); called by device_setup.
int block128_setup();

}  // namespace bsfp8
