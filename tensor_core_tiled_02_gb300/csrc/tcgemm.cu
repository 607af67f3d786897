// The library's one translation unit: the GEMM and the blocked add, and the
// layer operators, which share its device facts, tuning config and status word.
#include <algorithm>
#include <initializer_list>
#include <utility>

#include "gemm_f16.cu"

#include "layer_ops.cuh"
