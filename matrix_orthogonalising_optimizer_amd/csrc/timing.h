// Launches of the host-side translation units, timed when the diagnostics
// are on (dmuon_timing_enable).
#pragma once

#include <hip/hip_runtime.h>

#include <functional>

namespace dmuon {
// Run `launch`, recorded under `name` with its algorithmic work.
hipError_t timed_launch(const char* name, double flops, double bytes, hipStream_t st,
                        const std::function<hipError_t()>& launch);
}  // namespace dmuon
