// group_norm.hip -- group norm with an activation over channels-last images:
//   mu, var over the H*W*(C/G) values of an image's group; rstd = 1/sqrt(var + eps)
//   z = gamma (x - mu) rstd + beta;   y = act(z)
// and its gradient, with xh = (x - mu) rstd and dz = dy act'(z):
//   dbeta = sum dz;  dgamma = sum dz xh;
//   dx = rstd (gamma dz - mean(gamma dz) - xh mean(gamma dz xh))   (means over the group)
//
// Bound by memory: x in and y out, 4 bytes a value (backward: x, dy, dx, 6).
// The pixels of an image are cut into chunks.  A first kernel reduces every
// chunk per channel, a second joins the chunks (and a group's channels) in
// order, a third reads the image again and writes the result.  A thread keeps
// eight channels (16 bytes of a pixel) and walks over pixels, whatever the
// group size: groups of any width, also those that no vector fits, differ only
// in how the joined statistics are looked up.
//
// Variance: a thread sums d = x - x0 and d^2 with its own first value x0 of
// each channel as the shift, which loses nothing to a large mean and is never
// worse than the thread's count times the rounding (x0 is one of the values);
// the per-thread means and squared deviations are then joined by
//   mean = sum n_i mean_i / n,  M2 = sum M2_i + n_i (mean_i - mean)^2.
// All of it is fp32.  No atomics: results do not depend on timing.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epilogue.hpp"
#include "host.hpp"

namespace igc {

struct GnArgs {
    const void* x;
    const void* dy;        // backward
    void* out;             // y or dx
    const void* gamma;     // nullptr: 1
    const void* beta;      // nullptr: 0
    float *mean, *rstd;    // N x G
    float* part;           // N x chunks x C pairs: (mean, M2), or (sum dz, sum dz xh)
    float* joined;         // backward: N x G pairs (mean of gamma dz, mean of gamma dz xh)
    void *dgamma, *dbeta;  // nullptr: not wanted
    int64_t ldx, lddy, ldo;
    int64_t HW;
    int N, C, G, cpg, param_kind, act;
    int chunks, pixels;    // chunks of an image and pixels per chunk
    int sv, pl, slabs;     // vectors (8 channels) a workgroup covers, its pixel lanes, slabs of an image's channels
    float eps;
};

constexpr int kGnThreads = 256;  // at most

// Where a thread of a chunk works: its vector of channels and its pixel lane.
struct GnSpot {
    int n, chunk, v, p, c;  // c: first channel
    int64_t p0, p1;         // the chunk's pixels
    bool on;
    __device__ __forceinline__ explicit GnSpot(const GnArgs& a) {
        const int b = (int)blockIdx.x;
        const int slab = b % a.slabs, q = b / a.slabs;
        chunk = q % a.chunks;
        n = q / a.chunks;
        v = (int)threadIdx.x % a.sv;
        p = (int)threadIdx.x / a.sv;
        c = (slab * a.sv + v) * 8;
        on = p < a.pl && c < a.C;
        p0 = (int64_t)chunk * a.pixels;
        p1 = p0 + a.pixels < a.HW ? p0 + a.pixels : a.HW;
    }
};

// Per-channel means and squared deviations of a chunk.
template <bool FP16>
__global__ __launch_bounds__(kGnThreads) void gn_partial_kernel(const GnArgs a) {
    __shared__ float smean[kGnThreads * 8], sm2[kGnThreads * 8];
    const GnSpot s(a);
    if (s.on) {
        float x0[8], sum[8], sq[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x0[i] = sum[i] = sq[i] = 0.0f;
        const char* img = (const char*)a.x + ((int64_t)s.n * a.HW * a.ldx + s.c) * 2;
        const int64_t first = s.p0 + s.p;
        if (first < s.p1) unpack8<FP16>(*(const u32x4s_t*)(img + first * a.ldx * 2), x0);
        constexpr int U = 4;
        for (int64_t p = first; p < s.p1; p += U * a.pl) {
            u32x4s_t w[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * a.pl < s.p1) w[u] = *(const u32x4s_t*)(img + (p + u * a.pl) * a.ldx * 2);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p + u * a.pl >= s.p1) break;
                float v[8];
                unpack8<FP16>(w[u], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = v[i] - x0[i];
                    sum[i] += d;
                    sq[i] = __builtin_fmaf(d, d, sq[i]);
                }
            }
        }
        const int cnt = first < s.p1 ? (int)((s.p1 - first + a.pl - 1) / a.pl) : 0;
        const float rn = cnt > 0 ? 1.0f / (float)cnt : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float m = sum[i] * rn;
            smean[(s.p * a.sv + s.v) * 8 + i] = x0[i] + m;
            const float m2 = sq[i] - sum[i] * m;
            sm2[(s.p * a.sv + s.v) * 8 + i] = m2 < 0.0f ? 0.0f : m2;  // (a NaN stays one)
        }
    }
    __syncthreads();
    const int nch = a.sv * 8, total = (int)(s.p1 - s.p0);
    const int slab = (int)blockIdx.x % a.slabs;
    for (int ch = (int)threadIdx.x; ch < nch; ch += (int)blockDim.x) {
        const int c = slab * nch + ch;
        if (c >= a.C) break;
        float mean = 0.0f;
        for (int p = 0; p < a.pl && p < total; ++p) {
            const int cnt = (total - p + a.pl - 1) / a.pl;
            mean = __builtin_fmaf((float)cnt, smean[p * nch + ch], mean);
        }
        mean /= (float)total;
        float m2 = 0.0f;
        for (int p = 0; p < a.pl && p < total; ++p) {
            const int cnt = (total - p + a.pl - 1) / a.pl;
            const float d = smean[p * nch + ch] - mean;
            m2 += sm2[p * nch + ch] + (float)cnt * d * d;
        }
        float* dst = a.part + (((int64_t)s.n * a.chunks + s.chunk) * a.C + c) * 2;
        dst[0] = mean;
        dst[1] = m2;
    }
}

// Sum over a workgroup of 256 threads, in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    __syncthreads();  // an earlier sum has been read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// Joins the chunks and channels of one group of one image into its statistics.
__global__ __launch_bounds__(256) void gn_finish_kernel(const GnArgs a) {
    __shared__ float red[4];
    const int n = (int)blockIdx.x / a.G, g = (int)blockIdx.x % a.G;
    const float* part = a.part + ((int64_t)n * a.chunks * a.C + (int64_t)g * a.cpg) * 2;
    const int items = a.chunks * a.cpg;
    const float total = (float)a.HW * (float)a.cpg;
    float s = 0.0f;
    for (int i = (int)threadIdx.x; i < items; i += 256) {
        const int k = i / a.cpg, c = i - k * a.cpg;
        const int64_t cnt = a.HW - (int64_t)k * a.pixels < a.pixels ? a.HW - (int64_t)k * a.pixels : a.pixels;
        s = __builtin_fmaf((float)cnt, part[((int64_t)k * a.C + c) * 2], s);
    }
    const float mean = block_sum(s, red) / total;
    s = 0.0f;
    for (int i = (int)threadIdx.x; i < items; i += 256) {
        const int k = i / a.cpg, c = i - k * a.cpg;
        const int64_t cnt = a.HW - (int64_t)k * a.pixels < a.pixels ? a.HW - (int64_t)k * a.pixels : a.pixels;
        const float d = part[((int64_t)k * a.C + c) * 2] - mean;
        s += part[((int64_t)k * a.C + c) * 2 + 1] + (float)cnt * d * d;
    }
    const float var = block_sum(s, red) / total;
    if (threadIdx.x == 0) {
        a.mean[blockIdx.x] = mean;
        a.rstd[blockIdx.x] = 1.0f / __builtin_sqrtf(var + a.eps);
    }
}

// A thread's channels: mean, rstd * gamma (or rstd and gamma apart) and beta.
struct GnChannels {
    float mu[8], rs[8], ga[8], be[8];
    __device__ __forceinline__ GnChannels(const GnArgs& a, int n, int c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int g = n * a.G + (c + i) / a.cpg;
            mu[i] = a.mean[g];
            rs[i] = a.rstd[g];
            ga[i] = a.gamma ? load_kind(a.gamma, c + i, a.param_kind) : 1.0f;
            be[i] = a.beta ? load_kind(a.beta, c + i, a.param_kind) : 0.0f;
        }
    }
};

template <bool FP16>
__global__ __launch_bounds__(kGnThreads) void gn_apply_kernel(const GnArgs a) {
    const GnSpot s(a);
    if (!s.on) return;
    const GnChannels k(a, s.n, s.c);
    const char* img = (const char*)a.x + ((int64_t)s.n * a.HW * a.ldx + s.c) * 2;
    char* out = (char*)a.out + ((int64_t)s.n * a.HW * a.ldo + s.c) * 2;
    with_act(a.act, [&](auto A) __attribute__((always_inline)) {
        constexpr int ACT = decltype(A)::value;
        constexpr int U = 4;
        for (int64_t p = s.p0 + s.p; p < s.p1; p += U * a.pl) {
            u32x4s_t w[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * a.pl < s.p1) w[u] = *(const u32x4s_t*)(img + (p + u * a.pl) * a.ldx * 2);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p + u * a.pl >= s.p1) break;
                float v[8];
                unpack8<FP16>(w[u], v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = act_of<ACT>(__builtin_fmaf((v[i] - k.mu[i]) * k.rs[i], k.ga[i], k.be[i]));
                *(u32x4s_t*)(out + (p + u * a.pl) * a.ldo * 2) = pack8<FP16>(v);
            }
        }
    });
}

// Per-channel sums of dz and dz xh of a chunk.
template <bool FP16>
__global__ __launch_bounds__(kGnThreads) void gn_backward_partial_kernel(const GnArgs a) {
    __shared__ float s1[kGnThreads * 8], s2[kGnThreads * 8];
    const GnSpot s(a);
    if (s.on) {
        const GnChannels k(a, s.n, s.c);
        float sz[8], sx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sz[i] = sx[i] = 0.0f;
        const char* img = (const char*)a.x + ((int64_t)s.n * a.HW * a.ldx + s.c) * 2;
        const char* grad = (const char*)a.dy + ((int64_t)s.n * a.HW * a.lddy + s.c) * 2;
        with_act(a.act, [&](auto A) __attribute__((always_inline)) {
            constexpr int ACT = decltype(A)::value;
            constexpr int U = 2;
            for (int64_t p = s.p0 + s.p; p < s.p1; p += U * a.pl) {
                u32x4s_t w[U], d[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (p + u * a.pl < s.p1) {
                        w[u] = *(const u32x4s_t*)(img + (p + u * a.pl) * a.ldx * 2);
                        d[u] = *(const u32x4s_t*)(grad + (p + u * a.pl) * a.lddy * 2);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (p + u * a.pl >= s.p1) break;
                    float v[8], e[8];
                    unpack8<FP16>(w[u], v);
                    unpack8<FP16>(d[u], e);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float xh = (v[i] - k.mu[i]) * k.rs[i];
                        const float dz = e[i] * act_grad_of<ACT>(__builtin_fmaf(xh, k.ga[i], k.be[i]));
                        sz[i] += dz;
                        sx[i] = __builtin_fmaf(dz, xh, sx[i]);
                    }
                }
            }
        });
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s1[(s.p * a.sv + s.v) * 8 + i] = sz[i];
            s2[(s.p * a.sv + s.v) * 8 + i] = sx[i];
        }
    }
    __syncthreads();
    const int nch = a.sv * 8, slab = (int)blockIdx.x % a.slabs;
    for (int ch = (int)threadIdx.x; ch < nch; ch += (int)blockDim.x) {
        const int c = slab * nch + ch;
        if (c >= a.C) break;
        float t1 = 0.0f, t2 = 0.0f;
        for (int p = 0; p < a.pl; ++p) {
            t1 += s1[p * nch + ch];
            t2 += s2[p * nch + ch];
        }
        float* dst = a.part + (((int64_t)s.n * a.chunks + s.chunk) * a.C + c) * 2;
        dst[0] = t1;
        dst[1] = t2;
    }
}

// The first N*G workgroups: a group's two means.  The others: 32 channels'
// dgamma and dbeta each, summed over the images' chunks by 8 lanes a channel.
__global__ __launch_bounds__(256) void gn_backward_finish_kernel(const GnArgs a) {
    __shared__ float red[2 * 8 * 32];
    const int groups = a.N * a.G;
    if ((int)blockIdx.x < groups) {
        const int n = (int)blockIdx.x / a.G, g = (int)blockIdx.x % a.G;
        const float* part = a.part + ((int64_t)n * a.chunks * a.C + (int64_t)g * a.cpg) * 2;
        const int items = a.chunks * a.cpg;
        float t1 = 0.0f, t2 = 0.0f;
        for (int i = (int)threadIdx.x; i < items; i += 256) {
            const int k = i / a.cpg, c = i - k * a.cpg;
            const float ga = a.gamma ? load_kind(a.gamma, (int64_t)g * a.cpg + c, a.param_kind) : 1.0f;
            t1 = __builtin_fmaf(ga, part[((int64_t)k * a.C + c) * 2], t1);
            t2 = __builtin_fmaf(ga, part[((int64_t)k * a.C + c) * 2 + 1], t2);
        }
        const float total = (float)a.HW * (float)a.cpg;
        t1 = block_sum(t1, red) / total;
        t2 = block_sum(t2, red) / total;
        if (threadIdx.x == 0) {
            a.joined[blockIdx.x * 2] = t1;
            a.joined[blockIdx.x * 2 + 1] = t2;
        }
        return;
    }
    const int c = ((int)blockIdx.x - groups) * 32 + ((int)threadIdx.x & 31), l = (int)threadIdx.x >> 5;
    float t1 = 0.0f, t2 = 0.0f;
    if (c < a.C) {
        const int64_t items = (int64_t)a.N * a.chunks;
        for (int64_t i = l; i < items; i += 8) {
            t1 += a.part[(i * a.C + c) * 2];
            t2 += a.part[(i * a.C + c) * 2 + 1];
        }
    }
    red[threadIdx.x] = t1;
    red[256 + threadIdx.x] = t2;
    __syncthreads();
    if (l == 0 && c < a.C) {
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            t1 += red[k * 32 + threadIdx.x];
            t2 += red[256 + k * 32 + threadIdx.x];
        }
        if (a.dbeta) store_kind(a.dbeta, c, a.param_kind, t1);
        if (a.dgamma) store_kind(a.dgamma, c, a.param_kind, t2);
    }
}

template <bool FP16>
__global__ __launch_bounds__(kGnThreads) void gn_backward_apply_kernel(const GnArgs a) {
    const GnSpot s(a);
    if (!s.on) return;
    const GnChannels k(a, s.n, s.c);
    float c1[8], c2[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int g = s.n * a.G + (s.c + i) / a.cpg;
        c1[i] = a.joined[g * 2];
        c2[i] = a.joined[g * 2 + 1];
    }
    const char* img = (const char*)a.x + ((int64_t)s.n * a.HW * a.ldx + s.c) * 2;
    const char* grad = (const char*)a.dy + ((int64_t)s.n * a.HW * a.lddy + s.c) * 2;
    char* out = (char*)a.out + ((int64_t)s.n * a.HW * a.ldo + s.c) * 2;
    with_act(a.act, [&](auto A) __attribute__((always_inline)) {
        constexpr int ACT = decltype(A)::value;
        constexpr int U = 2;
        for (int64_t p = s.p0 + s.p; p < s.p1; p += U * a.pl) {
            u32x4s_t w[U], d[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * a.pl < s.p1) {
                    w[u] = *(const u32x4s_t*)(img + (p + u * a.pl) * a.ldx * 2);
                    d[u] = *(const u32x4s_t*)(grad + (p + u * a.pl) * a.lddy * 2);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p + u * a.pl >= s.p1) break;
                float v[8], e[8];
                unpack8<FP16>(w[u], v);
                unpack8<FP16>(d[u], e);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = (v[i] - k.mu[i]) * k.rs[i];
                    const float dz = e[i] * act_grad_of<ACT>(__builtin_fmaf(xh, k.ga[i], k.be[i]));
                    v[i] = k.rs[i] * (__builtin_fmaf(k.ga[i], dz, -c1[i]) - xh * c2[i]);
                }
                *(u32x4s_t*)(out + (p + u * a.pl) * a.ldo * 2) = pack8<FP16>(v);
            }
        }
    });
}

// ---- host -----------------------------------------------------------------

struct GnPlan {
    int sv, pl, slabs, threads, chunks, pixels;
    int64_t part_bytes, stat_bytes, bytes;
};

static GnPlan gn_plan(int64_t N, int64_t HW, int64_t C, int64_t G) {
    GnPlan p{};
    const int64_t vecs = C / 8;
    p.sv = (int)(vecs < kGnThreads ? vecs : kGnThreads);
    p.slabs = (int)((vecs + p.sv - 1) / p.sv);
    p.pl = kGnThreads / p.sv;
    if (p.pl > HW) p.pl = (int)HW;
    p.threads = (p.pl * p.sv + 63) / 64 * 64;
    // about eight workgroups a CU, each with at least four pixels a lane
    int64_t chunks = N > 0 ? (2048 + N * p.slabs - 1) / (N * p.slabs) : 1;
    const int64_t most = (HW + 4 * p.pl - 1) / (4 * p.pl);
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    p.pixels = (int)((HW + chunks - 1) / chunks);
    p.chunks = (int)((HW + p.pixels - 1) / p.pixels);
    p.part_bytes = round_up(N * p.chunks * C * 8, 256);
    p.stat_bytes = round_up(N * G * 8, 256);  // mean and rstd, or the two means of the backward pass
    p.bytes = p.part_bytes + p.stat_bytes;
    return p;
}

// What every entry point checks of an image tensor; 0 pixels never come here.
static igc_status_t check_image(const void* ptr, int64_t ld, int64_t C) {
    if (!ptr || ld < C) return IGC_ERR_INVALID_VALUE;
    return aligned16(ptr) && ld % 8 == 0 ? IGC_OK : IGC_ERR_MISALIGNED;
}
static igc_status_t check_shape(int N, int H, int W, int C, int G, igc_out_t pt, igc_act_t act) {
    if (N < 0 || H < 1 || W < 1 || C < 1 || G < 1 || C % G != 0) return IGC_ERR_INVALID_VALUE;
    if (!valid_type(pt) || (int)act < IGC_ACT_NONE || (int)act > IGC_ACT_SILU) return IGC_ERR_INVALID_VALUE;
    if (C % 8 != 0) return IGC_ERR_MISALIGNED;
    const int64_t hw = (int64_t)H * W;
    if (hw > 0x7fffffff || (int64_t)N * G > 0x3fffffff || (int64_t)N * C > 0x3fffffff) return IGC_ERR_UNSUPPORTED;
    return IGC_OK;
}
static bool aligned_params(const void* p, igc_out_t t) { return reinterpret_cast<uintptr_t>(p) % out_size(t) == 0; }

static GnArgs gn_args(const GnPlan& pl, int N, int64_t HW, int C, int G, const void* gamma, const void* beta,
                      igc_out_t pt, igc_act_t act, const Workspace& ws) {
    GnArgs a{};
    a.gamma = gamma;
    a.beta = beta;
    a.part = (float*)ws.ptr;
    a.HW = HW;
    a.N = N;
    a.C = C;
    a.G = G;
    a.cpg = C / G;
    a.param_kind = (int)pt;
    a.act = (int)act;
    a.chunks = pl.chunks;
    a.pixels = pl.pixels;
    a.sv = pl.sv;
    a.pl = pl.pl;
    a.slabs = pl.slabs;
    return a;
}

template <bool FP16>
static igc_status_t gn_forward(int N, int H, int W, int C, int G, const void* x, int64_t ldx, const void* gamma,
                               const void* beta, igc_out_t pt, float eps, igc_act_t act, void* y, int64_t ldy,
                               float* mean, float* rstd, void* user_ws, int64_t user_ws_bytes, hipStream_t stream) {
    if (const igc_status_t st = check_shape(N, H, W, C, G, pt, act)) return st;
    if (!(eps >= 0.0f)) return IGC_ERR_INVALID_VALUE;
    if (N == 0) return IGC_OK;
    if (const igc_status_t st = check_image(x, ldx, C)) return st;
    if (const igc_status_t st = check_image(y, ldy, C)) return st;
    if (!aligned_params(gamma, pt) || !aligned_params(beta, pt) || !aligned_params(mean, IGC_OUT_F32) ||
        !aligned_params(rstd, IGC_OUT_F32))
        return IGC_ERR_MISALIGNED;
    const int64_t HW = (int64_t)H * W;
    const GnPlan pl = gn_plan(N, HW, C, G);
    const int64_t grid = (int64_t)N * pl.chunks * pl.slabs;
    if (grid > 0x7fffffff) return IGC_ERR_UNSUPPORTED;
    Workspace ws;
    if (const igc_status_t st = ws.take(pl.bytes, user_ws, user_ws_bytes, stream)) return st;
    (void)hipGetLastError();
    GnArgs a = gn_args(pl, N, HW, C, G, gamma, beta, pt, act, ws);
    float* stats = (float*)((char*)ws.ptr + pl.part_bytes);
    a.x = x;
    a.out = y;
    a.ldx = ldx;
    a.ldo = ldy;
    a.mean = mean ? mean : stats;
    a.rstd = rstd ? rstd : stats + (int64_t)N * G;
    a.eps = eps;
    hipLaunchKernelGGL(gn_partial_kernel<FP16>, dim3((unsigned)grid), dim3(pl.threads), 0, stream, a);
    hipLaunchKernelGGL(gn_finish_kernel, dim3((unsigned)(N * G)), dim3(256), 0, stream, a);
    hipLaunchKernelGGL(gn_apply_kernel<FP16>, dim3((unsigned)grid), dim3(pl.threads), 0, stream, a);
    return hipGetLastError() == hipSuccess ? IGC_OK : IGC_ERR_HIP;
}

template <bool FP16>
static igc_status_t gn_backward(int N, int H, int W, int C, int G, const void* x, int64_t ldx, const void* gamma,
                                const void* beta, igc_out_t pt, const float* mean, const float* rstd, igc_act_t act,
                                const void* dy, int64_t lddy, void* dx, int64_t lddx, void* dgamma, void* dbeta,
                                void* user_ws, int64_t user_ws_bytes, hipStream_t stream) {
    if (const igc_status_t st = check_shape(N, H, W, C, G, pt, act)) return st;
    if (!aligned_params(gamma, pt) || !aligned_params(beta, pt) || !aligned_params(dgamma, pt) ||
        !aligned_params(dbeta, pt) || !aligned_params(mean, IGC_OUT_F32) || !aligned_params(rstd, IGC_OUT_F32))
        return IGC_ERR_MISALIGNED;
    if (N == 0 && !dgamma && !dbeta) return IGC_OK;
    if (N > 0) {
        if (const igc_status_t st = check_image(x, ldx, C)) return st;
        if (const igc_status_t st = check_image(dy, lddy, C)) return st;
        if (const igc_status_t st = check_image(dx, lddx, C)) return st;
        if (!mean || !rstd) return IGC_ERR_INVALID_VALUE;
    }
    const int64_t HW = (int64_t)H * W;
    const GnPlan pl = gn_plan(N, HW, C, G);
    const int64_t grid = (int64_t)N * pl.chunks * pl.slabs;
    if (grid > 0x7fffffff) return IGC_ERR_UNSUPPORTED;
    Workspace ws;
    if (const igc_status_t st = ws.take(N > 0 ? pl.bytes : 0, user_ws, user_ws_bytes, stream)) return st;
    (void)hipGetLastError();
    GnArgs a = gn_args(pl, N, HW, C, G, gamma, beta, pt, act, ws);
    a.x = x;
    a.dy = dy;
    a.out = dx;
    a.ldx = ldx;
    a.lddy = lddy;
    a.ldo = lddx;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.joined = (float*)((char*)ws.ptr + pl.part_bytes);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    if (grid > 0) hipLaunchKernelGGL(gn_backward_partial_kernel<FP16>, dim3((unsigned)grid), dim3(pl.threads), 0, stream, a);
    const unsigned params = dgamma || dbeta ? (unsigned)((C + 31) / 32) : 0;
    hipLaunchKernelGGL(gn_backward_finish_kernel, dim3((unsigned)(N * G) + params), dim3(256), 0, stream, a);
    if (grid > 0) hipLaunchKernelGGL(gn_backward_apply_kernel<FP16>, dim3((unsigned)grid), dim3(pl.threads), 0, stream, a);
    return hipGetLastError() == hipSuccess ? IGC_OK : IGC_ERR_HIP;
}

}  // namespace igc

using namespace igc;

extern "C" {

#define IGC_GN_FORWARD(NAME, FP16)                                                                                     \
    igc_status_t NAME(int N, int H, int W, int C, int G, const void* x, int64_t ldx, const void* gamma,                \
                      const void* beta, igc_out_t param_type, float eps, igc_act_t act, void* y, int64_t ldy,          \
                      float* mean, float* rstd, igc_stream_t stream) {                                                 \
        return gn_forward<FP16>(N, H, W, C, G, x, ldx, gamma, beta, param_type, eps, act, y, ldy, mean, rstd, nullptr, \
                                0, (hipStream_t)stream);                                                               \
    }                                                                                                                  \
    igc_status_t NAME##_ex(int N, int H, int W, int C, int G, const void* x, int64_t ldx, const void* gamma,           \
                           const void* beta, igc_out_t param_type, float eps, igc_act_t act, void* y, int64_t ldy,     \
                           float* mean, float* rstd, void* workspace, int64_t workspace_bytes, igc_stream_t stream) {  \
        return gn_forward<FP16>(N, H, W, C, G, x, ldx, gamma, beta, param_type, eps, act, y, ldy, mean, rstd,          \
                                workspace, workspace_bytes, (hipStream_t)stream);                                      \
    }
IGC_GN_FORWARD(group_norm_nhwc_bf16, false)
IGC_GN_FORWARD(group_norm_nhwc_fp16, true)

#define IGC_GN_BACKWARD(NAME, FP16)                                                                                    \
    igc_status_t NAME(int N, int H, int W, int C, int G, const void* x, int64_t ldx, const void* gamma,                \
                      const void* beta, igc_out_t param_type, const float* mean, const float* rstd, igc_act_t act,     \
                      const void* dy, int64_t lddy, void* dx, int64_t lddx, void* dgamma, void* dbeta,                 \
                      igc_stream_t stream) {                                                                           \
        return gn_backward<FP16>(N, H, W, C, G, x, ldx, gamma, beta, param_type, mean, rstd, act, dy, lddy, dx, lddx,  \
                                 dgamma, dbeta, nullptr, 0, (hipStream_t)stream);                                      \
    }                                                                                                                  \
    igc_status_t NAME##_ex(int N, int H, int W, int C, int G, const void* x, int64_t ldx, const void* gamma,           \
                           const void* beta, igc_out_t param_type, const float* mean, const float* rstd,               \
                           igc_act_t act, const void* dy, int64_t lddy, void* dx, int64_t lddx, void* dgamma,          \
                           void* dbeta, void* workspace, int64_t workspace_bytes, igc_stream_t stream) {               \
        return gn_backward<FP16>(N, H, W, C, G, x, ldx, gamma, beta, param_type, mean, rstd, act, dy, lddy, dx, lddx,  \
                                 dgamma, dbeta, workspace, workspace_bytes, (hipStream_t)stream);                      \
    }
IGC_GN_BACKWARD(group_norm_nhwc_backward_bf16, false)
IGC_GN_BACKWARD(group_norm_nhwc_backward_fp16, true)

int64_t igc_group_norm_workspace_bytes(int N, int H, int W, int C, int G) {
    if (check_shape(N, H, W, C, G, IGC_OUT_F32, IGC_ACT_NONE) != IGC_OK) return -1;
    return N == 0 ? 0 : gn_plan(N, (int64_t)H * W, C, G).bytes;
}

}  // extern "C"
