// rms_norm.hip -- rows: the root-mean-square norm with the residual's addition,
// to 16 bits or to 8 bits with a scale a row, its gradient, and the rounding of
// an activation's rows to 8 bits.
//
//   norm      h = x + residual (rounded to its type, as it is kept)
//             rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd gamma
//   8 bits    scale = max |v| / 127,  q = nearest(v / scale), v a row's values.
//             In the norm rstd is common to a row and cancels in q, so one
//             reduction, of sum h^2 and max |h gamma|, does for both.
//   gradient  g = dy gamma, xh = h rstd:  dx = rstd (g - xh mean(g xh)) + dh,
//             dgamma = sum over the rows of dy xh
//   rows      v = act(x) gate, to 8 bits
//
// Memory bounds all of them: every value is read once and written once.  T
// threads hold a row in registers, V vectors of eight values (16 bytes) each,
// between the reduction and the output; a workgroup holds several rows where
// they are short.  Rows of more than 8 * 1024 * 4 values (the gradient: half
// as many, as it keeps its sums beside them) are read twice.  All sums are fp32
// and taken in a fixed order.
//
// 8192 rows of 4096 in bf16, residual read, h kept, calls of one graph, launches
// included (a copy reaches 4.9 TB/s; what the cache still holds of the call
// before helps):
//   norm 49 us, 268 MB at 5.5 TB/s; to 8 bits 50, 235 MB at 4.7; gated rows to
//   8 bits 34, 168 MB at 5.0; gradient with dh and dgamma 57, 268 MB at 4.7.
// A kernel trace has 43 us of the first and 48 + 5 of the last.
// One row of 4096: 3.0, 3.3, 3.1 and 4.8 us, a launch (the gradient: two) and
// one trip to memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "column_sum.hpp"
#include "epilogue.hpp"
#include "host.hpp"
#include "igc.h"

namespace igc {

typedef __attribute__((ext_vector_type(2))) unsigned u32x2n_t;

struct RowArgs {
    const void* x;      // rows read: x, or h of the backward pass
    const void* res;    // norm: residual; rows to 8 bits: gate; backward: dh
    const void* dy;
    const void* gamma;
    void* h;
    void* y;            // norm: y; backward: dx
    int8_t* q;
    float* scale;
    float* rstd;        // written by the norm, read by the backward pass
    void* dgamma;
    float* part;        // backward: the workgroups' sums for dgamma, C each
    int64_t M, ldx, ldr, lddy, ldh, ldy, ldq;
    int C;
    float eps;
    int param_kind, act;
};

// 16 bytes of a row from column c: zeros where the row has ended.  A piece with one value inside is read whole (rows
// are 16-byte multiples) and what lies past the end is cleared.
__device__ __forceinline__ u32x4s_t load_piece(const void* base, int64_t off, int left) {
    u32x4s_t w{0, 0, 0, 0};
    if (left > 0) w = raw8(base, off);
    if (left < 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] &= left >= 2 * i + 2 ? 0xffffffffu : (left == 2 * i + 1 ? 0xffffu : 0u);
    }
    return w;
}
template <bool F16>
__device__ __forceinline__ void store_piece(void* base, int64_t off, int left, const float (&v)[8]) {
    if (left > 0) store8(base, off, F16 ? KIND_F16 : KIND_BF16, left, true, v);
}

template <bool F16>
__device__ __forceinline__ u32x4s_t add_rounded(u32x4s_t a, u32x4s_t b) {
    float x[8], y[8];
    unpack8<F16>(a, x);
    unpack8<F16>(b, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] += y[i];
    return pack8<F16>(x);
}

// of a row that T threads hold (short ones, 16)
template <int T>
__device__ __forceinline__ void load_gamma(const RowArgs& a, int c, float (&g)[8]) {
    load_gamma<T == 16>(a.gamma, a.param_kind, c, a.C, g);
}

// The magnitude as an integer, whose order puts infinity above every number and NaN above infinity.
__device__ __forceinline__ unsigned magnitude(float v) { return __builtin_bit_cast(unsigned, v) & 0x7fffffffu; }

// Sum and largest magnitude over the T threads of a row, in every one of them.  T > 64: through LDS, `red` holds a
// pair for each wave of the workgroup; every thread of it takes part.
template <int T>
__device__ __forceinline__ void row_reduce(float& s, unsigned& m, float (*red)[2]) {
    constexpr int L = T < 64 ? T : 64;
#pragma unroll
    for (int d = L >> 1; d >= 1; d >>= 1) {
        s += __shfl_xor(s, d);
        const unsigned o = (unsigned)__shfl_xor((int)m, d);
        m = o > m ? o : m;
    }
    if constexpr (T > 64) {
        const int wave = (int)threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            red[wave][0] = s;
            red[wave][1] = __builtin_bit_cast(float, m);
        }
        __syncthreads();
        const int first = wave / (T / 64) * (T / 64);
        s = 0.0f;
        m = 0;
#pragma unroll
        for (int w = 0; w < T / 64; ++w) {
            s += red[first + w][0];
            const unsigned o = __builtin_bit_cast(unsigned, red[first + w][1]);
            m = o > m ? o : m;
        }
    }
}

// Sum over a row's threads as row_reduce takes it, in loops: for a path that is seldom taken, it needs few registers.
template <int T>
__device__ __forceinline__ float row_sum(float s, float* red) {
    constexpr int L = T < 64 ? T : 64;
#pragma unroll 1
    for (int d = L >> 1; d >= 1; d >>= 1) s += __shfl_xor(s, d);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
        __syncthreads();
        s = 0.0f;
#pragma unroll 1
        for (int w = 0; w < T / 64; ++w) s += red[w];
    }
    return s;
}

// 1 / sqrt(mean + eps) of a row whose sum of squares is s.  In bf16 the squares may leave fp32's range where their root
// does not: above it rstd comes out as 0, and below it as more than 2^45, which needs an eps near 0.  Such a row is
// summed once more, its values times a power of two that brings them back, for which `squares(by)` gives a thread's sum
// of (by h)^2.  The branch is one of whole waves, its code behind the kernel's end, and ordinary rows pay its test (8192 x
// 1024 13.3 -> 13.5 us, 1 x 4096 and 4096 x 8192 nothing).  Every thread that shares row_reduce<T>'s barriers calls this
// after it with the same s.  Unrolled as row_reduce is, the second sum took the kernels' occupancy from 8 waves to 7 (300
// x 6000 to 8 bits 6.5 -> 7.5 us).
template <bool F16, int T, int W, class Squares>
__device__ __forceinline__ float row_rstd(const RowArgs& a, float s, float (&red)[W], Squares&& squares) {
    static_assert(T <= 64 || W == T / 64, "one row to the waves that share barriers");
    float rstd = 1.0f / __builtin_sqrtf(s / (float)a.C + a.eps);
    if constexpr (!F16) {
        const bool far = !(rstd > 0.0f && rstd < 0x1p45f);
        if (__builtin_expect(__ballot(far) != 0, 0)) {
            const float by = s > 1.0f ? 0x1p-80f : 0x1p70f;
            const float again = row_sum<T>(squares(by), red);
            if (far) rstd = by / __builtin_sqrtf(again / (float)a.C + a.eps * by * by);
        }
    }
    return rstd;
}

// How a row of largest magnitude `top` goes to 8 bits: q = nearest(127 v / top), ties to even, scale = top / 127.
// `pre` keeps 127 / top and 127 top finite.  A row of zeros has scale 0; one with an infinity or a NaN has that for its
// scale, and zeros.
//
// 127 / top is kept as two numbers, `inv` and what its rounding lost, and a product of both is rounded to fp32 before it
// is to a whole number, so that a tie (one value in 5000 to 100000 in rows of 16-bit values times a 16-bit gamma) is met
// exactly: with `inv` alone half of them went the wrong way.  Looking again at values near a tie instead is a branch that
// is seldom taken, whose code is then fetched: 512 rows of 8192, gated, 6.6 -> 7.7 us.
//
// LOW: a NaN among the values may have low bits (gamma's may; a 16-bit type's are 0), which are not to be taken for one.
template <bool LOW>
struct ToInt8 {
    float pre, inv, rest;
    unsigned keep;  // (LOW) the bytes of a row that has a largest magnitude
    __device__ __forceinline__ explicit ToInt8(float t) {
        keep = t < __builtin_inff() ? 0xffffffffu : 0u;
        pre = t < 0x1p-100f ? 0x1p100f : (t > 0x1p100f ? 0x1p-100f : 1.0f);
        const float top = t * pre;
        inv = t > 0.0f ? 127.0f / top : 0.0f;
        rest = inv > 0.0f ? __builtin_fmaf(-inv, top, 127.0f) * inv * (1.0f / 127.0f) : 0.0f;
    }
    // Eight values as bytes: 1.5 * 2^23 added puts the nearest whole number (ties to even) into the low bits.
    __device__ __forceinline__ u32x2n_t operator()(const float (&v)[8]) const {
#pragma clang fp contract(off)  // p is the rounded product
        unsigned b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = v[i] * pre, p = x * inv, e = __builtin_fmaf(x, rest, __builtin_fmaf(x, inv, -p));
            b[i] = __builtin_bit_cast(unsigned, (p + e) + 12582912.0f);
        }
        u32x2n_t w;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const unsigned lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0c0c0400u);
            const unsigned hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x0c0c0400u);
            w[i] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
            if constexpr (LOW) w[i] &= keep;
        }
        return w;
    }
};
__device__ __forceinline__ void store_int8(int8_t* q, int64_t off, int left, u32x2n_t w) {
    if (left >= 8) {
        *(u32x2n_t*)(q + off) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) q[off + i] = (int8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}

// Threads of a workgroup.  The norm's has one row to the waves that share barriers.
template <int T>
constexpr int kRowThreads = T < 256 ? 256 : T;
template <int T>
constexpr int kNormThreads = T < 128 ? 256 : T;

// A row's scale in the norm, whose largest |h gamma| is `top`: without one (an infinity or a NaN, or a product past
// fp32, though h rstd gamma might fit), NaN.
__device__ __forceinline__ float norm_scale(float top, float rstd) {
    return top < __builtin_inff() ? top * rstd / 127.0f : __builtin_nanf("");
}

// ---- norm ----------------------------------------------------------------------------------------------------------

template <bool F16, bool INT8, int T, int V>
__global__ __launch_bounds__(kNormThreads<T>) void rms_norm_kernel(const RowArgs a) {
    constexpr int R = kNormThreads<T> / T;
    __shared__ float red[kNormThreads<T> / 64][2], again[kNormThreads<T> / 64];
    const int t = (int)threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * R + (int)threadIdx.x / T;
    const bool in = row < a.M;
    u32x4s_t h[V], r[V];
    float g[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * 8, left = in ? a.C - c : 0;
        h[v] = load_piece(a.x, row * a.ldx + c, left);
        if (a.res) r[v] = load_piece(a.res, row * a.ldr + c, left);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * 8;
        load_gamma<T>(a, c, g[v]);
    }
    float s = 0.0f;
    unsigned m = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (a.res) h[v] = add_rounded<F16>(h[v], r[v]);
        float f[8];
        unpack8<F16>(h[v], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s = __builtin_fmaf(f[i], f[i], s);
            if constexpr (INT8) {
                const unsigned o = magnitude(f[i] * g[v][i]);
                m = o > m ? o : m;
            }
        }
    }
    row_reduce<T>(s, m, red);
    const float rstd = row_rstd<F16, T>(a, s, again, [&](float by) __attribute__((always_inline)) {
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f[8];
            unpack8<F16>(h[v], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(f[i] * by, f[i] * by, sum);
        }
        return sum;
    });
    if (!in) return;
    if (t == 0 && a.rstd) a.rstd[row] = rstd;
    const float top = __builtin_bit_cast(float, m);
    [[maybe_unused]] const ToInt8<true> to(top);
    if constexpr (INT8)
        if (t == 0) a.scale[row] = norm_scale(top, rstd);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * 8, left = a.C - c;
        float f[8];
        unpack8<F16>(h[v], f);
        if (a.h) store_piece<F16>(a.h, row * a.ldh + c, left, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = INT8 ? f[i] * g[v][i] : f[i] * rstd * g[v][i];
        if constexpr (INT8)
            store_int8(a.q, row * a.ldq + c, left, to(f));
        else
            store_piece<F16>(a.y, row * a.ldy + c, left, f);
    }
}

// Rows that registers do not hold: one workgroup of 1024 threads, x and residual read twice.
template <bool F16, bool INT8>
__global__ __launch_bounds__(1024) void rms_norm_long_kernel(const RowArgs a) {
    __shared__ float red[16][2], again[16];
    const int64_t row = blockIdx.x;
    float s = 0.0f;
    unsigned m = 0;
    for (int c = (int)threadIdx.x * 8; c < a.C; c += 8192) {
        u32x4s_t h = load_piece(a.x, row * a.ldx + c, a.C - c);
        if (a.res) h = add_rounded<F16>(h, load_piece(a.res, row * a.ldr + c, a.C - c));
        float f[8], g[8];
        unpack8<F16>(h, f);
        if constexpr (INT8) load_gamma<1024>(a, c, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s = __builtin_fmaf(f[i], f[i], s);
            if constexpr (INT8) {
                const unsigned o = magnitude(f[i] * g[i]);
                m = o > m ? o : m;
            }
        }
    }
    row_reduce<1024>(s, m, red);
    const float rstd = row_rstd<F16, 1024>(a, s, again, [&](float by) __attribute__((always_inline)) {
        float sum = 0.0f;
        for (int c = (int)threadIdx.x * 8; c < a.C; c += 8192) {
            u32x4s_t h = load_piece(a.x, row * a.ldx + c, a.C - c);
            if (a.res) h = add_rounded<F16>(h, load_piece(a.res, row * a.ldr + c, a.C - c));
            float f[8];
            unpack8<F16>(h, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(f[i] * by, f[i] * by, sum);
        }
        return sum;
    });
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
    const float top = __builtin_bit_cast(float, m);
    [[maybe_unused]] const ToInt8<true> to(top);
    if constexpr (INT8)
        if (threadIdx.x == 0) a.scale[row] = norm_scale(top, rstd);
    for (int c = (int)threadIdx.x * 8; c < a.C; c += 8192) {
        const int left = a.C - c;
        u32x4s_t h = load_piece(a.x, row * a.ldx + c, left);
        if (a.res) h = add_rounded<F16>(h, load_piece(a.res, row * a.ldr + c, left));
        float f[8], g[8];
        unpack8<F16>(h, f);
        load_gamma<1024>(a, c, g);
        if (a.h) store_piece<F16>(a.h, row * a.ldh + c, left, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = INT8 ? f[i] * g[i] : f[i] * rstd * g[i];
        if constexpr (INT8)
            store_int8(a.q, row * a.ldq + c, left, to(f));
        else
            store_piece<F16>(a.y, row * a.ldy + c, left, f);
    }
}

// ---- rows to 8 bits ------------------------------------------------------------------------------------------------

// act(x) * gate of eight columns.
template <bool F16>
__device__ __forceinline__ void activated(const RowArgs& a, u32x4s_t x, u32x4s_t gate, float (&f)[8]) {
    unpack8<F16>(x, f);
    with_act(a.act, [&](auto A) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = act_of<decltype(A)::value>(f[i]);
    });
    if (a.res) {
        float g[8];
        unpack8<F16>(gate, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= g[i];
    }
}

template <bool F16, int T, int V>
__global__ __launch_bounds__(kRowThreads<T>) void quantize_rows_kernel(const RowArgs a) {
    constexpr int R = kRowThreads<T> / T;
    __shared__ float red[kRowThreads<T> / 64][2];
    const int t = (int)threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * R + (int)threadIdx.x / T;
    const bool in = row < a.M;
    u32x4s_t x[V], r[V];
    float f[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * 8, left = in ? a.C - c : 0;
        x[v] = load_piece(a.x, row * a.ldx + c, left);
        if (a.res) r[v] = load_piece(a.res, row * a.ldr + c, left);
    }
    float s = 0.0f;
    unsigned m = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        activated<F16>(a, x[v], r[v], f[v]);  // (0 past the row's end: every activation is 0 there)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned o = magnitude(f[v][i]);
            m = o > m ? o : m;
        }
    }
    row_reduce<T>(s, m, red);
    if (!in) return;
    const float top = __builtin_bit_cast(float, m);
    const ToInt8<false> to(top);
    if (t == 0) a.scale[row] = top / 127.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * 8;
        store_int8(a.q, row * a.ldq + c, a.C - c, to(f[v]));
    }
}

template <bool F16>
__global__ __launch_bounds__(1024) void quantize_rows_long_kernel(const RowArgs a) {
    __shared__ float red[16][2];
    const int64_t row = blockIdx.x;
    const auto values = [&](int c, float (&f)[8]) __attribute__((always_inline)) {
        u32x4s_t gate{0, 0, 0, 0};
        if (a.res) gate = load_piece(a.res, row * a.ldr + c, a.C - c);
        activated<F16>(a, load_piece(a.x, row * a.ldx + c, a.C - c), gate, f);
    };
    float s = 0.0f;
    unsigned m = 0;
    for (int c = (int)threadIdx.x * 8; c < a.C; c += 8192) {
        float f[8];
        values(c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned o = magnitude(f[i]);
            m = o > m ? o : m;
        }
    }
    row_reduce<1024>(s, m, red);
    const float top = __builtin_bit_cast(float, m);
    const ToInt8<false> to(top);
    if (threadIdx.x == 0) a.scale[row] = top / 127.0f;
    for (int c = (int)threadIdx.x * 8; c < a.C; c += 8192) {
        float f[8];
        values(c, f);
        store_int8(a.q, row * a.ldq + c, a.C - c, to(f));
    }
}

// ---- gradient of the norm ------------------------------------------------------------------------------------------

// gamma of a workgroup's columns, which every row needs: in registers, or, of rows so wide that it would spill beside
// their values and sums, in LDS (2048 x 16384: 90 and 67 us).
template <int T, int V>
struct RowGamma {
    static constexpr bool kLds = T * V > 1024;
    float reg[kLds ? 1 : V][8];
    IGC_LDS f32x4s_t* lds;
    // one row a workgroup (kLds): a thread writes what it reads, so nothing waits for another
    __device__ __forceinline__ void load(const RowArgs& a, int t) {
        if constexpr (kLds) {
            __shared__ f32x4s_t store[2 * V * T];
            lds = (IGC_LDS f32x4s_t*)store + t;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * 8;
            if constexpr (kLds) {
                float g[8];
                load_gamma<T>(a, c, g);
                lds[2 * v * T] = f32x4s_t{g[0], g[1], g[2], g[3]};
                lds[(2 * v + 1) * T] = f32x4s_t{g[4], g[5], g[6], g[7]};
            } else {
                load_gamma<T>(a, c, reg[v]);
            }
        }
    }
    __device__ __forceinline__ void get(int v, float (&g)[8]) const {
        if constexpr (kLds) {
            const f32x4s_t lo = lds[2 * v * T], hi = lds[(2 * v + 1) * T];
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = lo[i], g[4 + i] = hi[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = reg[v][i];
        }
    }
};

// The workgroups take rows in turn and keep their sums for dgamma in registers; at the end each writes them out, and
// column_sum adds the workgroups' (or, of a single workgroup, they are dgamma).  Other workgroups of the CU, not loads of
// a next row, cover a row's loads (asking for it ahead measured the same).
template <bool F16, int T, int V>
__global__ __launch_bounds__(kRowThreads<T>) void rms_norm_backward_kernel(const RowArgs a) {
    constexpr int BT = kRowThreads<T>, R = BT / T;
    static_assert(R == 1 || !RowGamma<T, V>::kLds, "wide rows are one to a workgroup");
    __shared__ float red[2][BT / 64][2];
    __shared__ float cols[R > 1 ? R : 1][R > 1 ? T * V * 8 : 1];
    const int t = (int)threadIdx.x % T, rl = (int)threadIdx.x / T;
    const int64_t step = (int64_t)gridDim.x * R;
    RowGamma<T, V> gamma;
    gamma.load(a, t);
    float dg[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[v][i] = 0.0f;
    int odd = 0;
    for (int64_t base = (int64_t)blockIdx.x * R; base < a.M; base += step) {
        const int64_t row = base + rl;
        const bool in = row < a.M;
        const float rs = in ? a.rstd[row] : 0.0f;
        u32x4s_t h[V], dy[V], dh[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * 8, left = in ? a.C - c : 0;
            h[v] = load_piece(a.x, row * a.ldx + c, left);
            dy[v] = load_piece(a.dy, row * a.lddy + c, left);
            if (a.res) dh[v] = load_piece(a.res, row * a.ldr + c, left);
        }
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float fh[8], fd[8], g[8];
            gamma.get(v, g);
            unpack8<F16>(h[v], fh);
            unpack8<F16>(dy[v], fd);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s = __builtin_fmaf(fd[i] * g[i], fh[i], s);
                dg[v][i] = __builtin_fmaf(fd[i], fh[i] * rs, dg[v][i]);
            }
        }
        unsigned none = 0;
        row_reduce<T>(s, none, red[odd]);  // (two sets of sums in turn: one barrier a row)
        odd ^= 1;
        const float k = s / (float)a.C * rs * rs;  // xh mean(g xh) = h k
        if (!in) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * 8;
            float fh[8], fd[8], g[8];
            gamma.get(v, g);
            unpack8<F16>(h[v], fh);
            unpack8<F16>(dy[v], fd);
#pragma unroll
            for (int i = 0; i < 8; ++i) fd[i] = rs * __builtin_fmaf(-k, fh[i], fd[i] * g[i]);
            if (a.res) {
                unpack8<F16>(dh[v], fh);
#pragma unroll
                for (int i = 0; i < 8; ++i) fd[i] += fh[i];
            }
            store_piece<F16>(a.y, row * a.ldy + c, a.C - c, fd);
        }
    }
    if (!a.dgamma) return;
    if constexpr (R > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) cols[rl][(v * T + t) * 8 + i] = dg[v][i];
        __syncthreads();
        if (rl > 0) return;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                for (int k = 1; k < R; ++k) dg[v][i] += cols[k][(v * T + t) * 8 + i];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c + i >= a.C) continue;
            if (gridDim.x == 1)
                store_kind(a.dgamma, c + i, a.param_kind, dg[v][i]);
            else
                a.part[(int64_t)blockIdx.x * a.C + c + i] = dg[v][i];
        }
    }
}

// Long rows: each read twice.  The sums for dgamma, of which a thread adds to its own columns alone, are in LDS where
// 128 KB hold them (SUMS: C <= 32768), otherwise in the workgroup's part of the workspace, which takes them at the end.
template <bool F16, bool SUMS>
__global__ __launch_bounds__(1024) void rms_norm_backward_long_kernel(const RowArgs a) {
    __shared__ float red[2][16][2];
    __shared__ f32x4s_t sums[SUMS ? 8192 : 1];
    float* part = a.part ? a.part + (int64_t)blockIdx.x * a.C : nullptr;
    if constexpr (SUMS) {
        for (int k = 0; k < 8; ++k) sums[k * 1024 + (int)threadIdx.x] = f32x4s_t{0, 0, 0, 0};
    }
    int odd = 0;
    bool first = true;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const float rs = a.rstd[row];
        float s = 0.0f;
        int k = (int)threadIdx.x;
        for (int c = (int)threadIdx.x * 8; c < a.C; c += 8192, k += 2048) {
            float fh[8], fd[8], g[8];
            unpack8<F16>(load_piece(a.x, row * a.ldx + c, a.C - c), fh);
            unpack8<F16>(load_piece(a.dy, row * a.lddy + c, a.C - c), fd);
            load_gamma<1024>(a, c, g);
            if constexpr (SUMS) {
                f32x4s_t lo = sums[k], hi = sums[k + 1024];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo[i] = __builtin_fmaf(fd[i], fh[i] * rs, lo[i]);
                    hi[i] = __builtin_fmaf(fd[4 + i], fh[4 + i] * rs, hi[i]);
                }
                sums[k] = lo;
                sums[k + 1024] = hi;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) s = __builtin_fmaf(fd[i] * g[i], fh[i], s);
        }
        unsigned none = 0;
        row_reduce<1024>(s, none, red[odd]);
        odd ^= 1;
        const float m = s / (float)a.C * rs * rs;
        for (int c = (int)threadIdx.x * 8; c < a.C; c += 8192) {
            const int left = a.C - c;
            float fh[8], fd[8], g[8], dx[8];
            unpack8<F16>(load_piece(a.x, row * a.ldx + c, left), fh);
            unpack8<F16>(load_piece(a.dy, row * a.lddy + c, left), fd);
            load_gamma<1024>(a, c, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) dx[i] = rs * __builtin_fmaf(-m, fh[i], fd[i] * g[i]);
            if (a.res) {
                float f[8];
                unpack8<F16>(load_piece(a.res, row * a.ldr + c, left), f);
#pragma unroll
                for (int i = 0; i < 8; ++i) dx[i] += f[i];
            }
            store_piece<F16>(a.y, row * a.ldy + c, left, dx);
            if (!SUMS && part) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < left) part[c + i] = __builtin_fmaf(fd[i], fh[i] * rs, first ? 0.0f : part[c + i]);
            }
        }
        first = false;
    }
    if constexpr (SUMS) {
        if (!part) return;
        int k = (int)threadIdx.x;
        for (int c = (int)threadIdx.x * 8; c < a.C; c += 8192, k += 2048) {
            const f32x4s_t lo = sums[k], hi = sums[k + 1024];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < a.C) part[c + i] = i < 4 ? lo[i & 3] : hi[i & 3];
        }
    }
}

// ---- host ----------------------------------------------------------------------------------------------------------

enum RowOp : int { ROW_NORM = 0, ROW_QUANTIZE = 1, ROW_BACKWARD = 2 };
// Threads and vectors of a row; T == 0: rows that registers do not hold.
struct RowShape {
    int T, V;
    int least = 256;  // threads of a workgroup with rows of fewer are 256
    constexpr int threads() const { return T == 0 ? 1024 : (T < least ? 256 : T); }
    constexpr int rows() const { return T == 0 ? 1 : threads() / T; }
};
// Measured (many rows; us): norm 8192 x 4096 (512, 1) 48 and (256, 2) 52, to 8 bits 45 and 47, rows to 8 bits 32.2 and
// 31.0; norm 4096 x 8192 (512, 2) 54, to 8 bits 48.5, (1024, 1) 52 and 50; gradient 8192 x 4096 (512, 1) 57, (256, 2) 60,
// 4096 x 8192 (512, 2) 59, (1024, 1) 62.  A single row is fastest with one vector a thread: norm of 8192 values (1024, 1)
// 4.0, (512, 2) 4.3, of 4096 (512, 1) 3.6, (256, 2) 4.0.
static constexpr RowShape row_shape(int64_t M, int64_t C, RowOp op) {
    const int64_t n = (C + 7) / 8;
    if (n <= 16) return {16, 1};
    if (n <= 64) return {64, 1};
    if (n <= 128) return {128, 1, op == ROW_NORM ? 128 : 256};
    if (n <= 256) return {256, 1};
    if (n <= 512) return op == ROW_QUANTIZE && M >= 512 ? RowShape{256, 2} : RowShape{512, 1};
    if (n <= 1024) return op != ROW_BACKWARD && M < 512 ? RowShape{1024, 1} : RowShape{512, 2};
    if (n <= 2048) return {1024, 2};
    if (n <= 4096 && op != ROW_BACKWARD) return {1024, 4};  // (the backward pass has no registers for it)
    return {0, 0};
}

// The kernels of each operator: the shapes that row_shape gives it, all of them and no others.
#define IGC_NORM_SHAPES(X) \
    X(16, 1) X(64, 1) X(128, 1) X(256, 1) X(512, 1) X(1024, 1) X(512, 2) X(1024, 2) X(1024, 4)
#define IGC_QUANTIZE_SHAPES(X) \
    X(16, 1) X(64, 1) X(128, 1) X(256, 1) X(512, 1) X(256, 2) X(1024, 1) X(512, 2) X(1024, 2) X(1024, 4)
#define IGC_BACKWARD_SHAPES(X) X(16, 1) X(64, 1) X(128, 1) X(256, 1) X(512, 1) X(512, 2) X(1024, 2)
#define IGC_SHAPE(TT, VV) RowShape{TT, VV},
constexpr RowShape kNormShapes[] = {IGC_NORM_SHAPES(IGC_SHAPE)}, kQuantizeShapes[] = {IGC_QUANTIZE_SHAPES(IGC_SHAPE)},
                   kBackwardShapes[] = {IGC_BACKWARD_SHAPES(IGC_SHAPE)};
#undef IGC_SHAPE
template <int N>
constexpr bool are_those_of(const RowShape (&list)[N], RowOp op) {
    bool given[N] = {};
    for (int64_t n = 1; n <= 4097; ++n)
        for (const int64_t M : {1, 511, 512}) {
            const RowShape s = row_shape(M, 8 * n, op);
            int at = 0;
            while (at < N && (list[at].T != s.T || list[at].V != s.V)) ++at;
            if (at == N && s.T != 0) return false;
            if (at < N) given[at] = true;
        }
    for (const bool g : given)
        if (!g) return false;
    return true;
}
static_assert(are_those_of(kNormShapes, ROW_NORM));
static_assert(are_those_of(kQuantizeShapes, ROW_QUANTIZE));
static_assert(are_those_of(kBackwardShapes, ROW_BACKWARD));

// The kernel of shape s, or (T == 0) that of long rows.
template <bool F16, bool INT8>
static auto norm_kernel(RowShape s) {
#define IGC_ROW_CASE(TT, VV) \
    if (s.T == TT && s.V == VV) return &rms_norm_kernel<F16, INT8, TT, VV>;
    IGC_NORM_SHAPES(IGC_ROW_CASE)
#undef IGC_ROW_CASE
    return &rms_norm_long_kernel<F16, INT8>;
}
template <bool F16>
static auto quantize_kernel(RowShape s) {
#define IGC_ROW_CASE(TT, VV) \
    if (s.T == TT && s.V == VV) return &quantize_rows_kernel<F16, TT, VV>;
    IGC_QUANTIZE_SHAPES(IGC_ROW_CASE)
#undef IGC_ROW_CASE
    return &quantize_rows_long_kernel<F16>;
}
template <bool F16>
static auto backward_kernel(RowShape s, int64_t C) {
#define IGC_ROW_CASE(TT, VV) \
    if (s.T == TT && s.V == VV) return &rms_norm_backward_kernel<F16, TT, VV>;
    IGC_BACKWARD_SHAPES(IGC_ROW_CASE)
#undef IGC_ROW_CASE
    return C <= 32768 ? &rms_norm_backward_long_kernel<F16, true> : &rms_norm_backward_long_kernel<F16, false>;
}

// Rows of `bytes` a value: INVALID without a pointer or with rows that overlap, MISALIGNED by the 16-byte rule.
static igc_status_t check_rows(const void* ptr, int64_t ld, int64_t C, int bytes) {
    if (!ptr || ld < C) return IGC_ERR_INVALID_VALUE;
    return !aligned16(ptr) || ld * bytes % 16 != 0 ? IGC_ERR_MISALIGNED : IGC_OK;
}
static bool misplaced(const void* ptr, igc_out_t type) { return reinterpret_cast<uintptr_t>(ptr) % out_size(type) != 0; }
// Sizes beyond these are refused, as are leading dimensions whose offsets pass 64 bits (and, for the gradient, a dgamma
// of more columns than column_sum's grid takes).
static bool rows_too_large(int64_t M, int64_t C) { return M >= (1ll << 30) || C >= (1ll << 30); }
static bool sums_too_large(int64_t C) { return !launchable((C + 31) / 32, 1024); }
static bool strides_too_large(std::initializer_list<int64_t> lds) {
    for (const int64_t ld : lds)
        if (ld >= (1ll << 32)) return true;
    return false;
}

static igc_status_t norm_any(bool fp16, bool int8, int64_t M, int64_t C, const void* x, int64_t ldx, const void* res,
                             int64_t ldr, void* h, int64_t ldh, const void* gamma, igc_out_t pt, float eps, void* y,
                             int64_t ldy, float* scale, float* rstd, hipStream_t stream) {
    if (M < 0 || C < 1 || !valid_type(pt) || !(eps >= 0.0f)) return IGC_ERR_INVALID_VALUE;
    if (M == 0) return IGC_OK;
    if (const igc_status_t st = check_rows(x, ldx, C, 2)) return st;
    if (res)
        if (const igc_status_t st = check_rows(res, ldr, C, 2)) return st;
    if (h)
        if (const igc_status_t st = check_rows(h, ldh, C, 2)) return st;
    if (const igc_status_t st = check_rows(y, ldy, C, int8 ? 1 : 2)) return st;
    if (int8 && !scale) return IGC_ERR_INVALID_VALUE;
    if (misplaced(gamma, pt) || misplaced(scale, IGC_OUT_F32) || misplaced(rstd, IGC_OUT_F32)) return IGC_ERR_MISALIGNED;
    if (rows_too_large(M, C) || strides_too_large({ldx, res ? ldr : 0, h ? ldh : 0, ldy})) return IGC_ERR_UNSUPPORTED;
    const RowShape s = row_shape(M, C, ROW_NORM);
    const int64_t blocks = (M + s.rows() - 1) / s.rows();
    if (!launchable(blocks, s.threads())) return IGC_ERR_UNSUPPORTED;
    RowArgs a{};
    a.x = x;
    a.res = res;
    a.h = h;
    a.gamma = gamma;
    a.y = int8 ? nullptr : y;
    a.q = int8 ? (int8_t*)y : nullptr;
    a.scale = scale;
    a.rstd = rstd;
    a.M = M;
    a.C = (int)C;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldy = a.ldq = ldy;
    a.eps = eps;
    a.param_kind = (int)pt;
    (void)hipGetLastError();
    const auto kernel = int8 ? (fp16 ? norm_kernel<true, true>(s) : norm_kernel<false, true>(s))
                             : (fp16 ? norm_kernel<true, false>(s) : norm_kernel<false, false>(s));
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(s.threads()), 0, stream, a);
    return hipGetLastError() == hipSuccess ? IGC_OK : IGC_ERR_HIP;
}

static igc_status_t quantize_any(bool fp16, int64_t M, int64_t C, igc_act_t act, const void* x, int64_t ldx,
                                 const void* gate, int64_t ldg, int8_t* q, int64_t ldq, float* scale, hipStream_t stream) {
    if (M < 0 || C < 1 || (int)act < IGC_ACT_NONE || (int)act > IGC_ACT_SILU) return IGC_ERR_INVALID_VALUE;
    if (M == 0) return IGC_OK;
    if (const igc_status_t st = check_rows(x, ldx, C, 2)) return st;
    if (gate)
        if (const igc_status_t st = check_rows(gate, ldg, C, 2)) return st;
    if (const igc_status_t st = check_rows(q, ldq, C, 1)) return st;
    if (!scale) return IGC_ERR_INVALID_VALUE;
    if (misplaced(scale, IGC_OUT_F32)) return IGC_ERR_MISALIGNED;
    if (rows_too_large(M, C) || strides_too_large({ldx, gate ? ldg : 0, ldq})) return IGC_ERR_UNSUPPORTED;
    const RowShape s = row_shape(M, C, ROW_QUANTIZE);
    const int64_t blocks = (M + s.rows() - 1) / s.rows();
    if (!launchable(blocks, s.threads())) return IGC_ERR_UNSUPPORTED;
    RowArgs a{};
    a.x = x;
    a.res = gate;
    a.q = q;
    a.scale = scale;
    a.M = M;
    a.C = (int)C;
    a.ldx = ldx;
    a.ldr = ldg;
    a.ldq = ldq;
    a.act = (int)act;
    (void)hipGetLastError();
    hipLaunchKernelGGL(fp16 ? quantize_kernel<true>(s) : quantize_kernel<false>(s), dim3((unsigned)blocks),
                       dim3(s.threads()), 0, stream, a);
    return hipGetLastError() == hipSuccess ? IGC_OK : IGC_ERR_HIP;
}

// Workgroups of the backward pass, which take rows in turn: as many as the CUs hold and no more, at four rows' time
// each or more where that leaves one for every CU, so that the sums for dgamma that they leave stay small beside the
// rows (777 x 1001: 256 of them 9.0 us, 389 9.9; 512 x 2048: 256 8.9, 512 9.5; 8192 x 2048: 768 32.4, 512 34.6).
static int64_t backward_groups(RowShape s, int64_t M) {
    const int64_t blocks = (M + s.rows() - 1) / s.rows();
    const int64_t most = s.threads() >= 1024 || s.T * s.V > 512 ? 256 : (s.T == 512 ? 384 : (s.T == 256 ? 768 : 512));
    const int64_t want = blocks / 4 < 256 ? 256 : (blocks / 4 < most ? blocks / 4 : most);
    return blocks < want ? blocks : want;
}
static int64_t backward_bytes(RowShape s, int64_t M, int64_t C) {
    const int64_t g = backward_groups(s, M);
    return g > 1 || s.T == 0 ? round_up(g * C * 4, 256) : 0;
}

static igc_status_t backward_any(bool fp16, int64_t M, int64_t C, const void* h, int64_t ldh, const void* gamma,
                                 igc_out_t pt, const float* rstd, const void* dy, int64_t lddy, const void* dh,
                                 int64_t lddh, void* dx, int64_t lddx, void* dgamma, void* user_ws, int64_t user_ws_bytes,
                                 hipStream_t stream) {
    if (M < 0 || C < 1 || !valid_type(pt)) return IGC_ERR_INVALID_VALUE;
    if (M == 0 && !dgamma) return IGC_OK;
    if (M > 0) {
        if (const igc_status_t st = check_rows(h, ldh, C, 2)) return st;
        if (const igc_status_t st = check_rows(dy, lddy, C, 2)) return st;
        if (dh)
            if (const igc_status_t st = check_rows(dh, lddh, C, 2)) return st;
        if (const igc_status_t st = check_rows(dx, lddx, C, 2)) return st;
        if (!rstd) return IGC_ERR_INVALID_VALUE;
    }
    if (misplaced(gamma, pt) || misplaced(dgamma, pt) || misplaced(rstd, IGC_OUT_F32)) return IGC_ERR_MISALIGNED;
    if (rows_too_large(M, C) || (dgamma && sums_too_large(C)) ||
        (M > 0 && strides_too_large({ldh, lddy, dh ? lddh : 0, lddx})))
        return IGC_ERR_UNSUPPORTED;
    const RowShape s = row_shape(M, C, ROW_BACKWARD);
    const int64_t groups = backward_groups(s, M);
    Workspace ws;
    if (const igc_status_t st = ws.take(dgamma && M > 0 ? backward_bytes(s, M, C) : 0, user_ws, user_ws_bytes, stream))
        return st;
    RowArgs a{};
    a.x = h;
    a.res = dh;
    a.dy = dy;
    a.gamma = gamma;
    a.y = dx;
    a.rstd = const_cast<float*>(rstd);
    a.dgamma = dgamma;
    a.part = dgamma ? (float*)ws.ptr : nullptr;
    a.M = M;
    a.C = (int)C;
    a.ldx = ldh;
    a.ldr = lddh;
    a.lddy = lddy;
    a.ldy = lddx;
    a.param_kind = (int)pt;
    (void)hipGetLastError();
    if (M > 0) {
        hipLaunchKernelGGL(fp16 ? backward_kernel<true>(s, C) : backward_kernel<false>(s, C), dim3((unsigned)groups),
                           dim3(s.threads()), 0, stream, a);
        if (hipGetLastError() != hipSuccess) return IGC_ERR_HIP;
    }
    // (one workgroup wrote dgamma itself, but of long rows)
    if (dgamma && (M == 0 || groups > 1 || s.T == 0))
        if (launch_column_sum((const float*)ws.ptr, C, (int)groups, dgamma, (int)pt, stream) != hipSuccess) return IGC_ERR_HIP;
    return IGC_OK;
}

}  // namespace igc

using namespace igc;

extern "C" {

#define IGC_NORM(T, FP16)                                                                                               \
    igc_status_t rms_norm_##T(int64_t M, int64_t C, const void* x, int64_t ldx, const void* residual, int64_t ldr,      \
                              void* h, int64_t ldh, const void* gamma, igc_out_t param_type, float eps, void* y,        \
                              int64_t ldy, float* rstd, igc_stream_t stream) {                                          \
        return norm_any(FP16, false, M, C, x, ldx, residual, ldr, h, ldh, gamma, param_type, eps, y, ldy, nullptr,      \
                        rstd, (hipStream_t)stream);                                                                     \
    }                                                                                                                   \
    igc_status_t rms_norm_int8_##T(int64_t M, int64_t C, const void* x, int64_t ldx, const void* residual, int64_t ldr, \
                                   void* h, int64_t ldh, const void* gamma, igc_out_t param_type, float eps, int8_t* q, \
                                   int64_t ldq, float* scale, igc_stream_t stream) {                                    \
        return norm_any(FP16, true, M, C, x, ldx, residual, ldr, h, ldh, gamma, param_type, eps, q, ldq, scale,         \
                        nullptr, (hipStream_t)stream);                                                                  \
    }                                                                                                                   \
    igc_status_t rms_norm_backward_##T(int64_t M, int64_t C, const void* h, int64_t ldh, const void* gamma,             \
                                       igc_out_t param_type, const float* rstd, const void* dy, int64_t lddy,           \
                                       const void* dh, int64_t lddh, void* dx, int64_t lddx, void* dgamma,              \
                                       igc_stream_t stream) {                                                           \
        return backward_any(FP16, M, C, h, ldh, gamma, param_type, rstd, dy, lddy, dh, lddh, dx, lddx, dgamma, nullptr, \
                            0, (hipStream_t)stream);                                                                    \
    }                                                                                                                   \
    igc_status_t rms_norm_backward_##T##_ex(int64_t M, int64_t C, const void* h, int64_t ldh, const void* gamma,        \
                                            igc_out_t param_type, const float* rstd, const void* dy, int64_t lddy,      \
                                            const void* dh, int64_t lddh, void* dx, int64_t lddx, void* dgamma,         \
                                            void* workspace, int64_t workspace_bytes, igc_stream_t stream) {            \
        return backward_any(FP16, M, C, h, ldh, gamma, param_type, rstd, dy, lddy, dh, lddh, dx, lddx, dgamma,          \
                            workspace, workspace_bytes, (hipStream_t)stream);                                           \
    }                                                                                                                   \
    igc_status_t quantize_rows_int8_##T(int64_t M, int64_t C, igc_act_t act, const void* x, int64_t ldx,                \
                                        const void* gate, int64_t ldg, int8_t* q, int64_t ldq, float* scale,            \
                                        igc_stream_t stream) {                                                          \
        return quantize_any(FP16, M, C, act, x, ldx, gate, ldg, q, ldq, scale, (hipStream_t)stream);                    \
    }
IGC_NORM(bf16, false)
IGC_NORM(fp16, true)

int64_t igc_rms_norm_backward_workspace_bytes(int64_t M, int64_t C) {
    if (M < 0 || C < 1 || rows_too_large(M, C) || sums_too_large(C)) return -1;
    return M == 0 ? 0 : backward_bytes(row_shape(M, C, ROW_BACKWARD), M, C);
}

}  // extern "C"
