// few_rows.hpp -- host side of the product of a few rows (few_rows.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace igc {

struct Epi;
struct EpiInt8;

constexpr int64_t kFewRows = 32;  // most rows the kernel takes

// Whether it is the faster one for M <= kFewRows rows.
bool few_rows_faster(int64_t M, int64_t N, int64_t K, bool b_kc);

// How a product of M <= kFewRows rows is cut: NB operands of 16 columns a wave,
// `cols` workgroups across N, `splits` along K (each `per` of K).
struct FewRowsPlan {
    int nb;
    int64_t cols;
    int splits;
    int64_t per;
};
FewRowsPlan few_rows_plan(int64_t M, int64_t N, int64_t K, bool b_kc);
// The same of 8-bit operands, B column-major.
bool few_rows_int8_faster(int64_t M, int64_t N, int64_t K);
FewRowsPlan few_rows_int8_plan(int64_t M, int64_t N, int64_t K);

struct FewRowsArgs {
    const void* A;
    const void* B;
    void* C;
    float* ws;  // splits > 1: fp32 partials (int32 of 8-bit operands), split s at s * M * ldws, row pitch ldws
    int64_t N, K, lda, ldb, ldc, ldws, per;
    int M, cols, splits, out_kind;
};
hipError_t launch_few_rows(const FewRowsArgs& a, const Epi& e, bool fp16, bool b_kc, int nb, hipStream_t stream);
// 8-bit operands, B column-major.
hipError_t launch_few_rows_int8(const FewRowsArgs& a, const EpiInt8& e, hipStream_t stream);

}  // namespace igc
