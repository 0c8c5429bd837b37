// instances.hpp -- registry of compiled kernel instances (host side).
#pragma once
#include <stdint.h>

#include "igc.h"
#include "tile_configs.hpp"

namespace igc {

struct Instance {
    int bm, bn, bk, d, waves, mfma, half, loaders, sync;
    int op;              // OpKind: 0 GEMM, 1 forward conv, 2 data gradient, 3 filter gradient
    bool fp16, a_kc, b_kc;
    bool full;           // every loop variant compiled (else only K % 8 == 0 GEMMs and whole-tap convolutions)
    // kernels by loop variant (PLAIN, UNIFORM_TAP, RAGGED, CONV_GENERIC), nullptr where not built:
    const void* fn[4];     // __global__ gemm_kernel<Cfg<...>, V>: data-parallel grid and split-K
    const void* fn_sk[4];  // __global__ gemm_sk_kernel<Cfg<...>, V>: stream-K
    int64_t lds_bytes;   // static LDS of one workgroup
};

// The same configuration's kernels with the fused epilogue (epilogue.hpp).
struct EpiInstance {
    int bm, bn, bk, d, waves, mfma, half, loaders, sync;
    int op;
    bool fp16, a_kc, b_kc;
    // forward and backward, by loop variant; nullptr where not built (RAGGED: PLAIN, whose epilogue adds the K tail)
    const void* fn[2][4];
    const void* part[4];   // one part of a K split, for the epilogue to follow
};

// Each compiled object (one configuration, one operation family) registers
// its table when the library is loaded.
void register_instances(const Instance* table, int count);

const Instance* find_instance(const igc_tune_t& t, bool fp16, bool a_kc, bool b_kc, int op);
void register_epilogues(const EpiInstance* table, int count);
const EpiInstance* find_epilogue(const Instance& inst);
igc_tune_t default_tune(int64_t M, int64_t N, int64_t K, int op);
// The built-in choice for a call with an epilogue: no stream-K.
igc_tune_t epilogue_tune(int64_t M, int64_t N, int64_t K, int op, bool a_kc);
int num_tunes();
igc_tune_t tune_at(int i);
int tune_scope(int i);

}  // namespace igc
