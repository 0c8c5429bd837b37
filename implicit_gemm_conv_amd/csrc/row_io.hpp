// row_io.hpp -- eight consecutive values of a row, or of the vector of its
// columns' parameters, between storage and fp32 registers.
#pragma once
#include "activation.hpp"

namespace igc {

// Eight consecutive values of row storage, element `off` first.  vec: whole
// 16-byte pieces may be read as long as they hold one value below `left` (how
// many of the eight lie inside the row); rows are then 16-byte multiples, so
// the rest of such a piece is the row's own padding.
__device__ __forceinline__ u32x4s_t raw8(const void* base, int64_t off) {
    return *(const u32x4s_t*)((const char*)base + off * 2);
}
__device__ __forceinline__ void decode8(u32x4s_t w, int kind, float (&v)[8]) {
    if (kind == KIND_BF16)
        unpack8<false>(w, v);
    else
        unpack8<true>(w, v);
}
__device__ __forceinline__ void load8(const void* base, int64_t off, int kind, int left, bool vec, float (&v)[8]) {
    if (!vec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? load_kind(base, off + i, kind) : 0.0f;
    } else if (kind == KIND_F32) {
        const f32x4s_t lo = *(const f32x4s_t*)((const float*)base + off);
        f32x4s_t hi{0, 0, 0, 0};
        if (left > 4) hi = *(const f32x4s_t*)((const float*)base + off + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
    } else {
        decode8(raw8(base, off), kind, v);
    }
}
__device__ __forceinline__ void store8(void* base, int64_t off, int kind, int left, bool vec, const float (&v)[8]) {
    if (vec && left >= 8) {
        if (kind == KIND_F32) {
            *(f32x4s_t*)((float*)base + off) = f32x4s_t{v[0], v[1], v[2], v[3]};
            *(f32x4s_t*)((float*)base + off + 4) = f32x4s_t{v[4], v[5], v[6], v[7]};
        } else {
            *(u32x4s_t*)((char*)base + off * 2) = kind == KIND_BF16 ? pack8<false>(v) : pack8<true>(v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) store_kind(base, off + i, kind, v[i]);
    }
}

// gamma of the eight columns from c on, of C: zeros past their end, ones without a gamma.  A vector's memory ends with
// its last value, unlike a matrix row's, and it need not begin at a 16-byte multiple.  The last C % 8 values are read as
// the eight that end with the last one and moved down, so that every lane waits for one load (norm of 1 x 1001 with a
// gamma in 16 bits 2.86 us, in fp32 2.96; 3.05 with a branch for the lane that has the end and reads each value).
// SHORT: C may be below 8.
typedef u32x4s_t __attribute__((aligned(2))) u32x4v_t;
typedef f32x4s_t __attribute__((aligned(4))) f32x4v_t;
typedef __attribute__((ext_vector_type(2))) uint64_t u64x2_t;
template <bool SHORT>
__device__ __forceinline__ void load_gamma(const void* gamma, int kind, int c, int C, float (&g)[8]) {
    const int left = C - c;
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = gamma ? 0.0f : 1.0f;
    if (!gamma || left <= 0) return;
    if constexpr (SHORT)
        if (C < 8) {
            load8(gamma, c, kind, left, false, g);
            return;
        }
    const int at = left < 8 ? C - 8 : c, past = left < 8 ? 8 - left : 0;
    if (kind == KIND_F32) {
        const f32x4v_t* p = (const f32x4v_t*)((const float*)gamma + at);
        const f32x4s_t lo = p[0], hi = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = lo[i], g[4 + i] = hi[i];
        if (past > 0) {
#pragma unroll
            for (int by = 4; by >= 1; by >>= 1)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float next = i + by < 8 ? g[i + by] : 0.0f;
                    g[i] = past & by ? next : g[i];
                }
        }
    } else {
        u64x2_t w = __builtin_bit_cast(u64x2_t, *(const u32x4v_t*)((const unsigned short*)gamma + at));
        if (past > 0) {
            const uint64_t lo = past >= 4 ? w[1] : w[0], hi = past >= 4 ? 0 : w[1];
            const int bits = 16 * (past & 3);
            w[0] = lo >> bits | (hi << 1) << (63 - bits);
            w[1] = hi >> bits;
        }
        decode8(__builtin_bit_cast(u32x4s_t, w), kind, g);
    }
}

}  // namespace igc
