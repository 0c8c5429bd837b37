// activation.hpp -- the activations of the fused operators and their
// derivatives, in fp32, and the conversions between fp32 and the stored types.
//
//   none       z
//   relu       max(z, 0)
//   gelu       z Phi(z), Phi the normal distribution function
//   gelu_tanh  z/2 (1 + tanh u), u = sqrt(2/pi) (z + 0.044715 z^3); the same
//              as z sigmoid(2u), which needs one exponential and one
//              reciprocal
//   silu       z sigmoid(z)
// A NaN stays a NaN through every one of them and its derivative.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace igc {

enum ActKind : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };
// The storage types of include/igc.h's igc_out_t.
enum StoreKind : int { KIND_F32 = 0, KIND_BF16 = 1, KIND_F16 = 2 };

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

constexpr float kLog2e = 1.44269504088896340736f;

// 1 / (1 + exp(-x)).  exp overflows to infinity for x < -88, whose reciprocal
// is the 0 it should be.
__device__ __forceinline__ float sigmoid(float x) { return fast_rcp(1.0f + fast_exp2(-kLog2e * x)); }

// Phi(z) and, through `e`, exp(-z^2/2).  With x = |z|/sqrt(2) the tail
// Phi(-|z|) = erfc(x)/2 = exp(-x^2) t P(t), t = 1/(1 + 0.51 x): P is a
// polynomial fitted to exp(x^2) erfc(x) / (2 t) over 0 <= x <= 10 for the
// smallest largest relative error, 8.6e-7.  Working with the tail keeps the
// relative accuracy of z Phi(z) for negative z, where 1 + erf would cancel.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float x = 0.70710678118654752f * __builtin_fabsf(z);
    const float t = fast_rcp(__builtin_fmaf(0.51f, x, 1.0f));
    float q = 0.04724987743198132f;
    q = __builtin_fmaf(q, t, -0.1795670659452422f);
    q = __builtin_fmaf(q, t, 0.17922234320949498f);
    q = __builtin_fmaf(q, t, 0.027526746511527864f);
    q = __builtin_fmaf(q, t, 0.13953295481185748f);
    q = __builtin_fmaf(q, t, 0.1420761754948425f);
    q = __builtin_fmaf(q, t, 0.14395875013190326f);
    e = fast_exp2(-0.5f * kLog2e * z * z);
    const float tail = q * t * e;
    return z < 0.0f ? tail : 1.0f - tail;
}

constexpr float kGeluTanh1 = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGeluTanh3 = 0.07135481282712062f;  // 2 sqrt(2/pi) * 0.044715

template <int ACT>
__device__ __forceinline__ float act_of(float z) {
    if constexpr (ACT == ACT_RELU) {
        return z <= 0.0f ? 0.0f : z;  // a NaN compares false and passes
    } else if constexpr (ACT == ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    } else if constexpr (ACT == ACT_GELU_TANH) {
        return z * sigmoid(z * __builtin_fmaf(kGeluTanh3, z * z, kGeluTanh1));
    } else if constexpr (ACT == ACT_SILU) {
        return z * sigmoid(z);
    } else {
        return z;
    }
}

// act'(z); the derivative of relu at 0 is 0.
template <int ACT>
__device__ __forceinline__ float act_grad_of(float z) {
    if constexpr (ACT == ACT_RELU) {
        return z <= 0.0f ? 0.0f : (z > 0.0f ? 1.0f : z);
    } else if constexpr (ACT == ACT_GELU) {
        float e;
        const float c = normal_cdf(z, e);
        return __builtin_fmaf(z, 0.3989422804014327f * e, c);
    } else if constexpr (ACT == ACT_GELU_TANH) {
        // s + z s (1 - s) (2u)'.  Past |z| = 20 the sigmoid is 0 or 1 to the last bit; the bound keeps z^2 finite
        const float b = z > 20.0f ? 20.0f : (z < -20.0f ? -20.0f : z);
        const float s = sigmoid(b * __builtin_fmaf(kGeluTanh3, b * b, kGeluTanh1));
        return __builtin_fmaf(b * s * (1.0f - s), __builtin_fmaf(3.0f * kGeluTanh3, b * b, kGeluTanh1), s);
    } else if constexpr (ACT == ACT_SILU) {
        const float s = sigmoid(z);
        return s * __builtin_fmaf(z, 1.0f - s, 1.0f);
    } else {
        return 1.0f;
    }
}

// f(ACT constant) for the runtime `act`: one uniform branch around a whole
// block of elements.
template <int A>
struct ActC {
    static constexpr int value = A;
};
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case ACT_RELU: f(ActC<ACT_RELU>{}); break;
        case ACT_GELU: f(ActC<ACT_GELU>{}); break;
        case ACT_GELU_TANH: f(ActC<ACT_GELU_TANH>{}); break;
        case ACT_SILU: f(ActC<ACT_SILU>{}); break;
        default: f(ActC<ACT_NONE>{}); break;
    }
}

// ---- stored values --------------------------------------------------------
typedef __attribute__((ext_vector_type(4))) unsigned u32x4s_t;
typedef __attribute__((ext_vector_type(4))) float f32x4s_t;

__device__ __forceinline__ float bf16_bits(unsigned hi16) { return __builtin_bit_cast(float, hi16 << 16); }
__device__ __forceinline__ float f16_bits(unsigned lo16) {
    return (float)__builtin_bit_cast(_Float16, (unsigned short)lo16);
}
// The two values of one 32-bit word of 16-bit storage.
template <bool F16>
__device__ __forceinline__ void unpack2(unsigned w, float& a, float& b) {
    if constexpr (F16) {
        a = f16_bits(w & 0xffffu);
        b = f16_bits(w >> 16);
    } else {
        a = bf16_bits(w & 0xffffu);
        b = __builtin_bit_cast(float, w & 0xffff0000u);
    }
}
template <bool F16>
__device__ __forceinline__ unsigned pack2(float a, float b) {  // round to nearest even
    if constexpr (F16) {
        typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;
        return __builtin_bit_cast(unsigned, f16x2_t{(_Float16)a, (_Float16)b});
    } else {
        typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
        return __builtin_bit_cast(unsigned, bf16x2_t{(__bf16)a, (__bf16)b});
    }
}
template <bool F16>
__device__ __forceinline__ void unpack8(u32x4s_t w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2<F16>(w[i], v[2 * i], v[2 * i + 1]);
}
template <bool F16>
__device__ __forceinline__ u32x4s_t pack8(const float (&v)[8]) {
    return u32x4s_t{pack2<F16>(v[0], v[1]), pack2<F16>(v[2], v[3]), pack2<F16>(v[4], v[5]), pack2<F16>(v[6], v[7])};
}

// Element i of an array of a runtime storage type.
__device__ __forceinline__ float load_kind(const void* base, int64_t i, int kind) {
    if (kind == KIND_F32) return ((const float*)base)[i];
    const unsigned w = ((const unsigned short*)base)[i];
    return kind == KIND_BF16 ? bf16_bits(w) : f16_bits(w);
}
__device__ __forceinline__ void store_kind(void* base, int64_t i, int kind, float v) {
    if (kind == KIND_F32)
        ((float*)base)[i] = v;
    else if (kind == KIND_BF16)
        ((__bf16*)base)[i] = (__bf16)v;
    else
        ((_Float16*)base)[i] = (_Float16)v;
}

}  // namespace igc
