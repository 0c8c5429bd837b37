// int8_gemm.hpp -- registry of the kernels of the 8-bit integer product.
#pragma once
#include "instances.hpp"

namespace igc {

struct Int8Instance {
    Instance tile;     // the configuration; its K tile of bk counts pairs of values
    const void* fn;    // whole products
    const void* lean;  // those without activation and kept pre-activation
    const void* part;  // one part of a K split, for the epilogue to follow
};

// Each compiled object (one configuration) registers its kernels when the library is loaded.
void register_int8(const Int8Instance& instance);

}  // namespace igc
