// Internal interface of the operators on a language model's selections
// (tokens by expert, attention over a cache and its eviction, sampling): the
// host checks fill in the public argument structs, the launchers take them as
// checked.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/topk.h"

namespace tk {

// Experts of one call: one digit of the counting sort, whose counters fit LDS.
constexpr int64_t EXPERTS_MAX = 8192;

size_t dispatch_workspace(int64_t tokens, int64_t k, int64_t experts);
hipError_t launch_dispatch(const topk_dispatch_args& a, void* ws, hipStream_t s);

hipError_t launch_combine(const topk_combine_args& a, hipStream_t s);

size_t combine_grad_workspace(const topk_combine_grad_args& a);
hipError_t launch_combine_grad(const topk_combine_grad_args& a, void* ws, hipStream_t s);

// Widest head of attend: its accumulators stay in registers.
constexpr int64_t HEAD_MAX = 256;

// Entries of attend's caches lie less than this many elements apart: a step's
// rows are then within the range of a 32-bit offset in bytes.
constexpr int64_t STEP_MAX = int64_t(1) << 24;

size_t attend_workspace(const topk_attend_args& a, int cus);
hipError_t launch_attend(const topk_attend_args& a, void* ws, int cus, hipStream_t s);

size_t evict_workspace(const topk_evict_args& a);
hipError_t launch_evict(const topk_evict_args& a, void* ws, hipStream_t s);

// Longest row of sample: its weights keep 38 bits or more, and a row has at most 1024 chunks.
constexpr int64_t VOCABULARY_MAX = int64_t(1) << 24;

size_t sample_workspace(const topk_sample_args& a);
hipError_t launch_sample(const topk_sample_args& a, void* ws, hipStream_t s);

}  // namespace tk
