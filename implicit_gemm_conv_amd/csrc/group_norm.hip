// group_norm.hip -- group norm with an activation over channels-last images:
//   mu, var over the H*W*(C/G) values of an image's group; rstd = 1/sqrt(var + eps)
//   z = gamma (x - mu) rstd + beta;   y = act(z)
// and its gradient, with xh = (x - mu) rstd and dz = dy act'(z):
//   dbeta = sum dz;  dgamma = sum dz xh;
//   dx = rstd (gamma dz - mean(gamma dz) - xh mean(gamma dz xh))   (means over the group)
//
// Bound by memory: x in and y out, 4 bytes a value (backward: x, dy, dx, 6);
// small ones by the latency of a launch and of a few dependent loads.  Two forms:
//   - one workgroup for an image's slab of whole groups, in one launch: forward
//     x stays in registers from the statistics to the output, backward x and dy
//     do, or are read twice (gn_resident_kernel, gn_backward_slab_kernel);
//   - chunks of an image's pixels, in two launches: the first reduces every
//     chunk by group, the second joins the chunks, each workgroup for itself
//     while its first pixels arrive, reads the image again and writes.
// A thread keeps eight channels (16 bytes of a pixel) and walks over pixels,
// whatever the group size: groups of any width, also those that no vector fits,
// differ only in how the joined statistics are looked up.
// Measured (bf16, silu; forward, backward with gamma and beta's gradients):
// 32 of 56 x 56 x 256 in 32 groups 27.6 and 51.5 us (3.7 and 3.0 TB/s; backward
// has 38 operations a value, 27 us), 16 of 27 x 27 x 320 12.4 and 18.5, 32 of
// 48 x 48 x 640 in one 55 and 92, 2 of 8 x 8 x 1280 5.3 and 8.8.
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
#include "fastdiv.hpp"
#include "host.hpp"

namespace igc {

struct GnArgs {
    const void* x;
    const void* dy;        // backward
    void* out;             // y or dx
    const void* gamma;     // nullptr: 1
    const void* beta;      // nullptr: 0
    float *mean, *rstd;    // N x G
    float* part;           // pairs of every unit of channels and chunk, N x C/uw x chunks: (mean, M2); backward
                           // (sum gamma dz, sum gamma dz xh)
    float* sums;           // backward: pairs (sum dz, sum dz xh) of every channel, `rows` of them (images or chunks)
    void *dgamma, *dbeta;  // nullptr: not wanted
    int64_t ldx, lddy, ldo;
    int64_t HW;
    int N, C, G, cpg, param_kind, act;
    uint32_t cpg_magic;    // fastdiv multiplier of cpg
    int chunks, pixels;    // chunks of an image and pixels per chunk
    int uw;                // channels of a unit: a group, or what of it lies in one slab
    int rows;              // of `sums`
    int grid;              // workgroups over the images
    int sv, pl, slabs;     // vectors (8 channels) a workgroup covers, its pixel lanes, slabs of an image's channels
    float eps;
};

__device__ __forceinline__ int group_of(const GnArgs& a, int channel) {
    return (int)fastdiv((uint32_t)channel, (uint32_t)a.cpg, a.cpg_magic);
}

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

// Lanes of a workgroup for `items` sums of one length: as many neighbours an
// item as there are, a power of two and at most a wave.
struct GnLanes {
    int lanes, lane, item, step;
    __device__ __forceinline__ explicit GnLanes(int items) {
        lanes = 64;
        while (lanes > 1 && lanes * items > (int)blockDim.x) lanes >>= 1;
        lane = (int)threadIdx.x & (lanes - 1);
        item = (int)threadIdx.x / lanes;
        step = (int)blockDim.x / lanes;
    }
    // over the item's lanes, in a fixed order; every one of them gets it
    __device__ __forceinline__ float sum(float v) const {
        for (int d = lanes >> 1; d >= 1; d >>= 1) v += __shfl_xor(v, d);
        return v;
    }
};

// Threads for each of `items` sums that lie side by side in LDS rows, so that
// neighbouring threads take neighbouring items.
__device__ __forceinline__ int lanes_share(int items) {
    const int share = (int)blockDim.x / items;
    return share < 1 ? 1 : (share > 16 ? 16 : share);
}

__device__ __forceinline__ float* unit_pair(const GnArgs& a, int n, int unit, int chunk) {
    return a.part + (((int64_t)n * (a.C / a.uw) + unit) * a.chunks + chunk) * 2;
}

// Means and squared deviations of a chunk, by unit of channels.
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
    const int nch = a.sv * 8, total = (int)(s.p1 - s.p0), slab = (int)blockIdx.x % a.slabs;
    const int here = a.C - slab * nch < nch ? a.C - slab * nch : nch;  // channels of this slab
    // The pixel lanes of a channel, into lane 0's: several threads a channel, taking the lanes' means about lane 0's.
    const int q0 = total / a.pl, extra = total - q0 * a.pl;  // pixels of a lane, and lanes with one more
    const int share = lanes_share(here);
    for (int ch = (int)threadIdx.x % (share > 1 ? here : (int)blockDim.x); ch < here; ch += (int)blockDim.x) {
        const int q = share > 1 ? (int)threadIdx.x / here : 0;
        const float m0 = smean[ch];
        float t1 = 0.0f, t2 = 0.0f;
        if (q < share) {
#pragma unroll 4
            for (int p = q; p < a.pl; p += share) {
                const float n = (float)(q0 + (p < extra)), d = smean[p * nch + ch] - m0;
                if (n > 0.0f) {
                    t1 = __builtin_fmaf(n, d, t1);
                    t2 += sm2[p * nch + ch] + n * d * d;
                }
            }
        }
        if (share > 1) {
            __syncthreads();
            if (q < share) smean[q * here + ch] = t1, sm2[q * here + ch] = t2;
            __syncthreads();
            if (q == 0)
                for (int k = 1; k < share; ++k) t1 += smean[k * here + ch], t2 += sm2[k * here + ch];
        }
        if (q == 0) {
            const float dm = t1 / (float)total, m2 = t2 - t1 * dm;
            smean[ch] = m0 + dm;
            sm2[ch] = m2 < 0.0f ? 0.0f : m2;
        }
    }
    __syncthreads();
    const GnLanes j(nch / a.uw);  // (of a full slab: the order of a unit's sum is the same in every slab)
    for (int u = j.item; u < here / a.uw; u += j.step) {  // the channels of a unit, equal in number of pixels
        float mean = 0.0f, m2 = 0.0f;
        for (int c = j.lane; c < a.uw; c += j.lanes) mean += smean[u * a.uw + c];
        mean = j.sum(mean) / (float)a.uw;
        for (int c = j.lane; c < a.uw; c += j.lanes) {
            const float d = smean[u * a.uw + c] - mean;
            m2 += sm2[u * a.uw + c] + (float)total * d * d;
        }
        m2 = j.sum(m2);
        if (j.lane == 0) {
            float* dst = unit_pair(a, s.n, slab * nch / a.uw + u, s.chunk);
            dst[0] = mean;
            dst[1] = m2;
        }
    }
}

// The groups that the channels of a slab belong to.  A group may lie across
// slabs, whose workgroups each join it for themselves: `shared` groups are what
// the join's lanes are dealt for, the same number in every slab, so that all of
// them add in one order and get the same bits.
struct GnGroups {
    int c0, g0, count, shared;
    __device__ __forceinline__ explicit GnGroups(const GnArgs& a) {
        c0 = (int)blockIdx.x % a.slabs * a.sv * 8;
        const int c1 = (c0 + a.sv * 8 < a.C ? c0 + a.sv * 8 : a.C) - 1;
        g0 = group_of(a, c0);
        count = group_of(a, c1) - g0 + 1;
        shared = a.slabs > 1 ? group_of(a, a.sv * 8) + 1 : a.G;
    }
};

constexpr int kGnThreadsChannels = kGnThreads * 8;  // channels of a slab at most, so its groups

// Joins the chunks of the slab's groups into their statistics, to sm and sr by
// group of the slab; of the first chunk's workgroups the one whose slab holds a
// group's first channel writes them out.  The chunks'
// means are taken about the first one's, one pass over the pairs: what that
// loses is at most the number of chunks times a rounding, since the first chunk
// is part of the variance.
__device__ __forceinline__ void join_chunks(const GnArgs& a, int n, int chunk, float* sm, float* sr) {
    const GnGroups gs(a);
    const GnLanes j(gs.shared);
    const int upg = a.cpg / a.uw, pairs = upg * a.chunks;
    const float total = (float)a.HW * (float)a.cpg;
    const float full = (float)a.pixels * (float)a.uw;
    const float last = (float)(int)(a.HW - (int64_t)(a.chunks - 1) * a.pixels) * (float)a.uw;
    for (int g = j.item; g < gs.count; g += j.step) {
        const float* src = unit_pair(a, n, (gs.g0 + g) * upg, 0);
        const float m0 = src[0];
        float s1 = 0.0f, s2 = 0.0f;
        int at = j.lane % a.chunks;  // the pair's chunk
        const int ahead = j.lanes % a.chunks;
        constexpr int U = 8;
        for (int k = j.lane; k < pairs; k += U * j.lanes) {
            float m[U], q[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k + u * j.lanes < pairs) m[u] = src[2 * (k + u * j.lanes)], q[u] = src[2 * (k + u * j.lanes) + 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (k + u * j.lanes >= pairs) break;
                const float d = m[u] - m0, w = at + 1 < a.chunks ? full : last;
                s1 = __builtin_fmaf(w, d, s1);
                s2 += q[u] + w * d * d;
                at += ahead;
                if (at >= a.chunks) at -= a.chunks;
            }
        }
        s1 = j.sum(s1);
        s2 = j.sum(s2);
        const float dm = s1 / total, m2 = s2 - s1 * dm;
        if (j.lane == 0) {
            const float mean = m0 + dm, rstd = 1.0f / __builtin_sqrtf((m2 < 0.0f ? 0.0f : m2) / total + a.eps);
            sm[g] = mean;
            sr[g] = rstd;
            const bool first = chunk == 0 && (gs.g0 + g) * a.cpg >= gs.c0;
            if (first && a.mean) a.mean[n * a.G + gs.g0 + g] = mean;
            if (first && a.rstd) a.rstd[n * a.G + gs.g0 + g] = rstd;
        }
    }
    __syncthreads();
}

template <bool FP16>
__global__ __launch_bounds__(kGnThreads) void gn_apply_kernel(const GnArgs a) {
    __shared__ float sm[kGnThreadsChannels], sr[kGnThreadsChannels];
    const GnSpot s(a);
    constexpr int U = 4;
    const char* img = (const char*)a.x + ((int64_t)s.n * a.HW * a.ldx + s.c) * 2;
    char* out = (char*)a.out + ((int64_t)s.n * a.HW * a.ldo + s.c) * 2;
    u32x4s_t w[U];
    auto load = [&](int64_t p) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s.on && p + u * a.pl < s.p1) w[u] = *(const u32x4s_t*)(img + (p + u * a.pl) * a.ldx * 2);
    };
    load(s.p0 + s.p);  // on its way during the join
    join_chunks(a, s.n, s.chunk, sm, sr);
    if (!s.on) return;
    const int g0 = GnGroups(a).g0;
    float mu[8], ga[8], be[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int g = group_of(a, s.c + i) - g0;
        mu[i] = sm[g];
        ga[i] = sr[g] * (a.gamma ? load_kind(a.gamma, s.c + i, a.param_kind) : 1.0f);
        be[i] = a.beta ? load_kind(a.beta, s.c + i, a.param_kind) : 0.0f;
    }
    with_act(a.act, [&](auto A) __attribute__((always_inline)) {
        constexpr int ACT = decltype(A)::value;
        for (int64_t p = s.p0 + s.p; p < s.p1; p += U * a.pl) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p + u * a.pl >= s.p1) break;
                float v[8];
                unpack8<FP16>(w[u], v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = act_of<ACT>(__builtin_fmaf(v[i] - mu[i], ga[i], be[i]));
                *(u32x4s_t*)(out + (p + u * a.pl) * a.ldo * 2) = pack8<FP16>(v);
            }
            load(p + U * a.pl);
        }
    });
}

// Sums of dz and dz xh of a chunk, by channel and, weighted with gamma, by unit.
template <bool FP16>
__global__ __launch_bounds__(kGnThreads) void gn_backward_partial_kernel(const GnArgs a) {
    __shared__ float s1[kGnThreads * 8], s2[kGnThreads * 8];
    const GnSpot s(a);
    if (s.on) {
        float mu[8], rs[8], ga[8], be[8], sz[8], sx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int g = s.n * a.G + group_of(a, s.c + i);
            mu[i] = a.mean[g];
            rs[i] = a.rstd[g];
            ga[i] = rs[i] * (a.gamma ? load_kind(a.gamma, s.c + i, a.param_kind) : 1.0f);
            be[i] = a.beta ? load_kind(a.beta, s.c + i, a.param_kind) : 0.0f;
            sz[i] = sx[i] = 0.0f;
        }
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
                        const float c = v[i] - mu[i];
                        const float dz = e[i] * act_grad_of<ACT>(__builtin_fmaf(c, ga[i], be[i]));
                        sz[i] += dz;
                        sx[i] = __builtin_fmaf(dz, c, sx[i]);
                    }
                }
            }
        });
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s1[(s.p * a.sv + s.v) * 8 + i] = sz[i];
            s2[(s.p * a.sv + s.v) * 8 + i] = sx[i] * rs[i];
        }
    }
    __syncthreads();
    const int nch = a.sv * 8, slab = (int)blockIdx.x % a.slabs;
    const int here = a.C - slab * nch < nch ? a.C - slab * nch : nch;
    const int share = lanes_share(here);
    for (int ch = (int)threadIdx.x % (share > 1 ? here : (int)blockDim.x); ch < here; ch += (int)blockDim.x) {
        const int c = slab * nch + ch, q = share > 1 ? (int)threadIdx.x / here : 0;
        float t1 = 0.0f, t2 = 0.0f;
        if (q < share) {
#pragma unroll 4
            for (int p = q; p < a.pl; p += share) {
                t1 += s1[p * nch + ch];
                t2 += s2[p * nch + ch];
            }
        }
        if (share > 1) {
            __syncthreads();
            if (q < share) s1[q * here + ch] = t1, s2[q * here + ch] = t2;
            __syncthreads();
            if (q == 0)
                for (int k = 1; k < share; ++k) t1 += s1[k * here + ch], t2 += s2[k * here + ch];
        }
        if (q > 0) continue;
        if (a.dgamma || a.dbeta) {
            float* dst = a.sums + (((int64_t)s.n * a.chunks + s.chunk) * a.C + c) * 2;
            dst[0] = t1;
            dst[1] = t2;
        }
        const float ga = a.gamma ? load_kind(a.gamma, c, a.param_kind) : 1.0f;
        s1[ch] = ga * t1;
        s2[ch] = ga * t2;
    }
    __syncthreads();
    const GnLanes j(nch / a.uw);
    for (int u = j.item; u < here / a.uw; u += j.step) {
        float t1 = 0.0f, t2 = 0.0f;
        for (int c = j.lane; c < a.uw; c += j.lanes) {
            t1 += s1[u * a.uw + c];
            t2 += s2[u * a.uw + c];
        }
        t1 = j.sum(t1);
        t2 = j.sum(t2);
        if (j.lane == 0) {
            float* dst = unit_pair(a, s.n, slab * nch / a.uw + u, s.chunk);
            dst[0] = t1;
            dst[1] = t2;
        }
    }
}

// dgamma and dbeta of COLS channels: the rows of `sums`, added in order by the workgroup's lanes of each channel.
template <int COLS>
__device__ __forceinline__ void gn_param_sums(const GnArgs& a, int block, int threads, float* red) {
    const int t = (int)threadIdx.x, lanes = threads / COLS;
    const int c = block * COLS + t % COLS, l = t / COLS;
    float t1 = 0.0f, t2 = 0.0f;
    if (c < a.C) {
#pragma unroll 8
        for (int n = l; n < a.rows; n += lanes) {
            t1 += a.sums[((int64_t)n * a.C + c) * 2];
            t2 += a.sums[((int64_t)n * a.C + c) * 2 + 1];
        }
    }
    red[t] = t1;
    red[threads + t] = t2;
    __syncthreads();
    if (l == 0 && c < a.C) {
        for (int k = 1; k < lanes; ++k) {
            t1 += red[k * COLS + t];
            t2 += red[threads + k * COLS + t];
        }
        if (a.dbeta) store_kind(a.dbeta, c, a.param_kind, t1);
        if (a.dgamma) store_kind(a.dgamma, c, a.param_kind, t2);
    }
}
constexpr int kGnJoinThreads = 512;
__global__ __launch_bounds__(kGnJoinThreads) void gn_param_kernel(const GnArgs a) {
    __shared__ float red[2 * kGnJoinThreads];
    gn_param_sums<32>(a, (int)blockIdx.x, kGnJoinThreads, red);
}

template <bool FP16>
__global__ __launch_bounds__(kGnThreads) void gn_backward_apply_kernel(const GnArgs a) {
    __shared__ float s1[kGnThreadsChannels], s2[kGnThreadsChannels];  // the two means of the slab's groups
    if ((int)blockIdx.x >= a.grid) {  // the workgroups past the images': dgamma and dbeta
        gn_param_sums<8>(a, (int)blockIdx.x - a.grid, (int)blockDim.x, s1);
        return;
    }
    const GnSpot s(a);
    constexpr int U = 2;
    const char* img = (const char*)a.x + ((int64_t)s.n * a.HW * a.ldx + s.c) * 2;
    const char* grad = (const char*)a.dy + ((int64_t)s.n * a.HW * a.lddy + s.c) * 2;
    char* out = (char*)a.out + ((int64_t)s.n * a.HW * a.ldo + s.c) * 2;
    u32x4s_t w[U], d[U];
    auto load = [&](int64_t p) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s.on && p + u * a.pl < s.p1) {
                w[u] = *(const u32x4s_t*)(img + (p + u * a.pl) * a.ldx * 2);
                d[u] = *(const u32x4s_t*)(grad + (p + u * a.pl) * a.lddy * 2);
            }
    };
    load(s.p0 + s.p);  // on its way during the join
    const GnGroups gs(a);
    {
        const GnLanes j(gs.shared);
        const int upg = a.cpg / a.uw, pairs = upg * a.chunks;
        const float rn = 1.0f / ((float)a.HW * (float)a.cpg);
        for (int g = j.item; g < gs.count; g += j.step) {
            const float* src = unit_pair(a, s.n, (gs.g0 + g) * upg, 0);
            float t1 = 0.0f, t2 = 0.0f;
#pragma unroll 8
            for (int k = j.lane; k < pairs; k += j.lanes) {
                t1 += src[2 * k];
                t2 += src[2 * k + 1];
            }
            t1 = j.sum(t1);
            t2 = j.sum(t2);
            if (j.lane == 0) {
                s1[g] = t1 * rn;
                s2[g] = t2 * rn;
            }
        }
    }
    __syncthreads();
    if (!s.on) return;
    // dx = ga dz - (x - mu) rs^2 c2 - rs c1
    float mu[8], ga[8], be[8], c2[8], c1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int g = group_of(a, s.c + i);
        const float rs = a.rstd[s.n * a.G + g];
        mu[i] = a.mean[s.n * a.G + g];
        ga[i] = rs * (a.gamma ? load_kind(a.gamma, s.c + i, a.param_kind) : 1.0f);
        be[i] = a.beta ? load_kind(a.beta, s.c + i, a.param_kind) : 0.0f;
        c2[i] = -rs * rs * s2[g - gs.g0];
        c1[i] = -rs * s1[g - gs.g0];
    }
    with_act(a.act, [&](auto A) __attribute__((always_inline)) {
        constexpr int ACT = decltype(A)::value;
        for (int64_t p = s.p0 + s.p; p < s.p1; p += U * a.pl) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p + u * a.pl >= s.p1) break;
                float v[8], e[8];
                unpack8<FP16>(w[u], v);
                unpack8<FP16>(d[u], e);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float c = v[i] - mu[i];
                    const float dz = e[i] * act_grad_of<ACT>(__builtin_fmaf(c, ga[i], be[i]));
                    v[i] = __builtin_fmaf(ga[i], dz, __builtin_fmaf(c, c2[i], c1[i]));
                }
                *(u32x4s_t*)(out + (p + u * a.pl) * a.ldo * 2) = pack8<FP16>(v);
            }
            load(p + U * a.pl);
        }
    });
}

// ---- images held on chip ----------------------------------------------------
// Where a workgroup's registers hold all of an image's pixels for a slab of
// whole groups, one kernel reads x once, reduces, and writes y: 4 bytes a value
// and one launch.  A thread keeps NV vectors; sums of a group go through LDS in
// a fixed order.  The mean comes first and then the squared deviations from it,
// from the registers, so the variance needs no shift.  The sum times
// the rounded reciprocal of the count is corrected by its remainder, so that the
// mean of a constant group is the constant wherever the sum is exact: with eps =
// 1e-5 a mean of 1000 that is off by one step moves xh by 0.02.  (A division in
// each thread instead: 16 of 27 x 27 x 320 13.4 us, 12.8 without.)
__device__ __forceinline__ void one_at_a_time() { __builtin_amdgcn_sched_barrier(0); }  // one vector unpacked at once

// The packed values are what stays in registers from one phase to the next:
// without this the compiler keeps their unpacked form, twice the size.
template <int NV>
__device__ __forceinline__ void keep_packed(u32x4s_t (&x)[NV]) {
#pragma unroll
    for (int k = 0; k < NV; ++k) asm volatile("" : "+v"(x[k]));
}

struct GnSlab {
    int n, v, p, c, sv;  // image, vector, pixel lane, first channel, vectors of this slab
    int groups, g0;      // of this slab, and the first
    bool on;
    __device__ __forceinline__ explicit GnSlab(const GnArgs& a) {
        const int id = xcd_order((int)blockIdx.x, a.grid);  // an image's slabs share lines: keep them on one XCD
        n = id / a.slabs;
        const int slab = id - n * a.slabs;
        sv = a.C / 8 - slab * a.sv < a.sv ? a.C / 8 - slab * a.sv : a.sv;
        v = (int)threadIdx.x % a.sv;
        p = (int)threadIdx.x / a.sv;
        c = (slab * a.sv + v) * 8;
        groups = sv * 8 / a.cpg;
        g0 = slab * a.sv * 8 / a.cpg;
        on = p < a.pl && v < sv;
    }
};

// Sum of each of the slab's channels over the workgroup's pixel lanes, to
// chan[channel]: up to 16 threads a channel, whose lanes lie along the channels
// (consecutive LDS words), then one.  `red` holds 8 floats a thread.  Every
// thread calls it.
__device__ __forceinline__ void channel_sums(const GnArgs& a, const GnSlab& s, const float (&val)[8], float* red,
                                             float* chan) {
    const int t = (int)threadIdx.x, row = a.sv * 8;  // channels of a full slab: a row of `red`
    __syncthreads();                                 // `red` and `chan` of an earlier call have been read
    if (s.on) {
        float* dst = red + s.p * row + s.v * 8;
        *(f32x4s_t*)dst = f32x4s_t{val[0], val[1], val[2], val[3]};
        *(f32x4s_t*)(dst + 4) = f32x4s_t{val[4], val[5], val[6], val[7]};
    }
    __syncthreads();
    const int nch = s.sv * 8, turn = (int)blockDim.x < nch ? (int)blockDim.x : nch;
    int per = (int)blockDim.x / turn;  // threads a channel
    per = per > 16 ? 16 : per;
    if (per > 1) {  // one turn covers every channel
        const int q = t / nch, c = t - q * nch;
        float sum = 0.0f;
        if (q < per)
            for (int p = q; p < a.pl; p += per) sum += red[p * row + c];
        __syncthreads();
        if (q < per) red[q * nch + c] = sum;
        __syncthreads();
        if (t < nch) {
            sum = red[t];
            for (int k = 1; k < per; ++k) sum += red[k * nch + t];
            chan[t] = sum;
        }
    } else {
        for (int c = t; c < nch; c += turn) {
            float sum = 0.0f;
            for (int p = 0; p < a.pl; ++p) sum += red[p * row + c];
            chan[c] = sum;
        }
    }
    __syncthreads();
}

// Sums over the slab's groups, to out[group]: W values a thread, one (all its
// channels being of one group) or its eight channels apart.  `red` holds W
// floats a thread, `chan` the slab's channels (W == 1: a value a wave).  Every thread calls it.
template <int W>
__device__ __forceinline__ void group_sums(const GnArgs& a, const GnSlab& s, const float (&val)[W], float* red,
                                           float* chan, float* out) {
    const int lane = (int)threadIdx.x & 63, waves = (int)(blockDim.x >> 6);
    if constexpr (W == 1) {
        __syncthreads();  // `red` and `out` of an earlier call have been read
        if (s.on) red[s.p * a.sv + s.v] = val[0];
        __syncthreads();
    } else {
        channel_sums(a, s, val, red, chan);
    }
    if constexpr (W == 1) {
        // The values of a group, per of every pixel lane, by as many waves as there are for a group.
        const int per = a.cpg / 8, share = waves / s.groups > 1 ? waves / s.groups : 1;
        const int wave = (int)threadIdx.x >> 6, part = wave % share, len = per * a.pl;
        for (int g = wave / share; g < s.groups; g += waves / share) {
            float t = 0.0f;
            for (int i = part * 64 + lane; i < len; i += 64 * share) {
                const int p = i / per;
                t += red[p * a.sv + g * per + i - p * per];
            }
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) t += __shfl_xor(t, d);
            if (lane == 0) (share > 1 ? chan[wave] : out[g]) = t;
        }
        if (share > 1) {
            __syncthreads();
            if ((int)threadIdx.x < s.groups) {
                float t = chan[threadIdx.x * share];
                for (int k = 1; k < share; ++k) t += chan[threadIdx.x * share + k];
                out[threadIdx.x] = t;
            }
        }
    } else {
        for (int g = (int)(threadIdx.x >> 6); g < s.groups; g += waves) {  // a wave a group
            float t = 0.0f;
            for (int c = lane; c < a.cpg; c += 64) t += chan[g * a.cpg + c];
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) t += __shfl_xor(t, d);
            if (lane == 0) out[g] = t;
        }
    }
    __syncthreads();
}

constexpr int kGnMaxThreads = 1024, kGnMaxVecs = 256;  // of a workgroup of the resident kernels

template <bool FP16, int NV, bool SINGLE>
__global__ __launch_bounds__(kGnMaxThreads) void gn_resident_kernel(const GnArgs a) {
    constexpr int W = SINGLE ? 1 : 8;
    __shared__ __attribute__((aligned(16))) float red[kGnMaxThreads * W];
    __shared__ float sums[kGnMaxVecs * W];  // by group of the slab
    __shared__ float chan[SINGLE ? kGnMaxThreads / 64 : kGnMaxVecs * 8];
    const GnSlab s(a);
    const char* img = (const char*)a.x + ((int64_t)s.n * a.HW * a.ldx + s.c) * 2;
    u32x4s_t x[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int p = s.p + k * a.pl;
        x[k] = u32x4s_t{0, 0, 0, 0};
        if (s.on && p < a.HW) x[k] = *(const u32x4s_t*)(img + p * a.ldx * 2);
    }
    float ga[8], be[8];
    int gi[W];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        ga[i] = s.on && a.gamma ? load_kind(a.gamma, s.c + i, a.param_kind) : 1.0f;
        be[i] = s.on && a.beta ? load_kind(a.beta, s.c + i, a.param_kind) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) gi[i] = s.on ? group_of(a, s.c + i) - s.g0 : 0;
    const float count = (float)a.HW * (float)a.cpg, rn = 1.0f / count;
    float acc[W], mu[W], rs[W];
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {  // absent pixels are zeros
        float v[8];
        unpack8<FP16>(x[k], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i % W] += v[i];
        one_at_a_time();
    }
    group_sums<W>(a, s, acc, red, chan, sums);
    keep_packed(x);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float sum = sums[gi[i]], m = sum * rn, rest = __builtin_fmaf(-m, count, sum);
        mu[i] = rest == rest ? __builtin_fmaf(rest, rn, m) : m;  // (an infinite sum has none)
        acc[i] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (s.p + k * a.pl >= a.HW) break;
        float v[8];
        unpack8<FP16>(x[k], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = v[i] - mu[i % W];
            acc[i % W] = __builtin_fmaf(d, d, acc[i % W]);
        }
        one_at_a_time();
    }
    group_sums<W>(a, s, acc, red, chan, sums);
    keep_packed(x);
#pragma unroll
    for (int i = 0; i < W; ++i) rs[i] = 1.0f / __builtin_sqrtf(sums[gi[i]] * rn + a.eps);
    if (s.on && s.p == 0 && a.mean) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (s.c + i == (s.g0 + gi[i]) * a.cpg) a.mean[s.n * a.G + s.g0 + gi[i]] = mu[i];
    }
    if (s.on && s.p == 0 && a.rstd) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (s.c + i == (s.g0 + gi[i]) * a.cpg) a.rstd[s.n * a.G + s.g0 + gi[i]] = rs[i];
    }
    if (!s.on) return;
    char* out = (char*)a.out + ((int64_t)s.n * a.HW * a.ldo + s.c) * 2;
    with_act(a.act, [&](auto A) __attribute__((always_inline)) {
        constexpr int ACT = decltype(A)::value;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int p = s.p + k * a.pl;
            if (p >= a.HW) break;
            float v[8];
            unpack8<FP16>(x[k], v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = act_of<ACT>(__builtin_fmaf((v[i] - mu[i % W]) * rs[i % W], ga[i], be[i]));
            *(u32x4s_t*)(out + p * a.ldo * 2) = pack8<FP16>(v);
            one_at_a_time();
        }
    });
}

// The gradient, one workgroup for an image's slab of whole groups.  The sums of
// each channel go to `sums` for dgamma and dbeta, a group's to its two means.
// NV > 0: x and dy stay in registers between the two passes (8 bytes read, 4
// written a pair); NV == 0: both are read again, from the caches as far as they
// go, any number of pixels.  Work per value (two exponentials and reciprocals
// among about 35 operations) is as long as the memory's: with registers full one
// workgroup has the CU to itself and the two add up, so beyond four vectors a
// thread the second form, which overlaps them, is the faster one.
template <bool FP16, int NV, bool SINGLE>
__global__ __launch_bounds__(kGnMaxThreads) void gn_backward_slab_kernel(const GnArgs a) {
    constexpr int W = SINGLE ? 1 : 8;
    constexpr int U = NV > 0 ? NV : 2;  // pixels in flight
    __shared__ __attribute__((aligned(16))) float red[kGnMaxThreads * 8];
    __shared__ float chan[2 * 8 * kGnMaxVecs];  // the slab's channels, both sums
    const GnSlab s(a);
    const char* img = (const char*)a.x + ((int64_t)s.n * a.HW * a.ldx + s.c) * 2;
    const char* grad = (const char*)a.dy + ((int64_t)s.n * a.HW * a.lddy + s.c) * 2;
    u32x4s_t x[U], d[U];
    auto load = [&](int p0) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int p = p0 + k * a.pl;
            x[k] = d[k] = u32x4s_t{0, 0, 0, 0};
            if (s.on && p < a.HW) {
                x[k] = *(const u32x4s_t*)(img + p * a.ldx * 2);
                d[k] = *(const u32x4s_t*)(grad + p * a.lddy * 2);
            }
        }
    };
    load(s.p);
    float mu[W], rs[W], ga[8], be[8], s1[8], s2[8];  // ga: rstd gamma, so z = (x - mu) ga + beta
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const int g = s.on ? s.n * a.G + group_of(a, s.c + i) : 0;
        mu[i] = a.mean[g];
        rs[i] = a.rstd[g];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        ga[i] = rs[i % W] * (s.on && a.gamma ? load_kind(a.gamma, s.c + i, a.param_kind) : 1.0f);
        be[i] = s.on && a.beta ? load_kind(a.beta, s.c + i, a.param_kind) : 0.0f;
        s1[i] = s2[i] = 0.0f;
    }
    with_act(a.act, [&](auto A) __attribute__((always_inline)) {
        constexpr int ACT = decltype(A)::value;
        for (int p0 = s.p; p0 < a.HW; p0 += U * a.pl) {
            if (NV == 0 && p0 != s.p) load(p0);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (p0 + k * a.pl >= a.HW) break;
                float v[8], e[8];
                unpack8<FP16>(x[k], v);
                unpack8<FP16>(d[k], e);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float c = v[i] - mu[i % W];
                    const float dz = e[i] * act_grad_of<ACT>(__builtin_fmaf(c, ga[i], be[i]));
                    s1[i] += dz;
                    s2[i] = __builtin_fmaf(dz, c, s2[i]);
                }
                one_at_a_time();
            }
            if (NV > 0) break;
        }
    });
#pragma unroll
    for (int i = 0; i < 8; ++i) s2[i] *= rs[i % W];
    const int lane = (int)threadIdx.x & 63, waves = (int)(blockDim.x >> 6), nch = s.sv * 8;
    channel_sums(a, s, s1, red, chan);
    channel_sums(a, s, s2, red, chan + nch);
    if (NV == 0) load(s.p);  // on its way during the rest of the join
    const int c0 = s.g0 * a.cpg;  // the slab's first channel
    if (a.dgamma || a.dbeta)
        for (int i = (int)threadIdx.x; i < nch; i += (int)blockDim.x) {
            float* dst = a.sums + ((int64_t)s.n * a.C + c0 + i) * 2;
            dst[0] = chan[i];
            dst[1] = chan[nch + i];
        }
    // a wave a group: its two means, into `red`
    const float rn = 1.0f / ((float)a.HW * (float)a.cpg);
    for (int g = (int)(threadIdx.x >> 6); g < s.groups; g += waves) {
        float t1 = 0.0f, t2 = 0.0f;
        for (int c = g * a.cpg + lane; c < (g + 1) * a.cpg; c += 64) {
            const float w = a.gamma ? load_kind(a.gamma, c0 + c, a.param_kind) : 1.0f;
            t1 = __builtin_fmaf(w, chan[c], t1);
            t2 = __builtin_fmaf(w, chan[nch + c], t2);
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) {
            t1 += __shfl_xor(t1, m);
            t2 += __shfl_xor(t2, m);
        }
        if (lane == 0) {
            red[2 * g] = t1 * rn;
            red[2 * g + 1] = t2 * rn;
        }
    }
    __syncthreads();
    if (!s.on) return;
    keep_packed(x);
    keep_packed(d);
    // dx = ga dz - (x - mu) rs^2 c2 - rs c1
    float c1[W], c2[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const int g = group_of(a, s.c + i) - s.g0;
        c1[i] = -rs[i] * red[2 * g];
        c2[i] = -rs[i] * rs[i] * red[2 * g + 1];
    }
    char* out = (char*)a.out + ((int64_t)s.n * a.HW * a.ldo + s.c) * 2;
    with_act(a.act, [&](auto A) __attribute__((always_inline)) {
        constexpr int ACT = decltype(A)::value;
        for (int p0 = s.p; p0 < a.HW; p0 += U * a.pl) {
            if (NV == 0 && p0 != s.p) load(p0);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int p = p0 + k * a.pl;
                if (p >= a.HW) break;
                float v[8], e[8];
                unpack8<FP16>(x[k], v);
                unpack8<FP16>(d[k], e);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float c = v[i] - mu[i % W];
                    const float dz = e[i] * act_grad_of<ACT>(__builtin_fmaf(c, ga[i], be[i]));
                    v[i] = __builtin_fmaf(ga[i], dz, __builtin_fmaf(c, c2[i % W], c1[i % W]));
                }
                *(u32x4s_t*)(out + p * a.ldo * 2) = pack8<FP16>(v);
                one_at_a_time();
            }
            if (NV > 0) break;
        }
    });
}

// ---- host -----------------------------------------------------------------

// Most vectors a thread of the resident kernels holds (of each tensor): forward
// what 128 registers leave room for; backward a larger slab is faster read twice.
constexpr int kGnMostForward = 16, kGnMostBackward = 4;
constexpr int64_t kGnSlabs = 128;

struct GnPlan {
    bool slab;      // one workgroup for an image's slab of groups; otherwise chunks of pixels
    bool resident;  // the slab stays in registers
    int nv;         // vectors a thread holds; 0: not resident
    int sv, pl, slabs, threads, chunks, pixels, uw;
    int64_t part_bytes, sum_bytes, bytes;
};

// One workgroup of up to 1024 threads for an image's slab of sv vectors (whole
// groups).  Resident where the threads can hold it; backward also read twice.
static bool slab_plan(GnPlan& p, int64_t N, int64_t HW, int64_t C, int64_t G, bool backward) {
    const int64_t vecs = C / 8, cpg = C / G, most = backward ? kGnMostBackward : kGnMostForward;
    int64_t base = cpg;  // lcm(cpg, 8) / 8 vectors: the narrowest slab of whole vectors and groups
    while (base % 8 != 0) base *= 2;
    base /= 8;
    if (base > kGnMaxVecs) return false;
    auto slabs = [&](int64_t v) { return N * ((vecs + v - 1) / v); };
    auto fits = [&](int64_t sv) { return HW <= most * (kGnMaxThreads / sv); };
    // Wider slabs read and write longer pieces of a pixel, as long as every CU
    // keeps one; read twice, they have 64-byte pieces at least.
    int64_t sv = base;
    if (!fits(base)) {
        while (backward && sv < 4 && 2 * sv <= vecs) sv *= 2;
        if (!backward) return false;
    }
    while (2 * sv <= vecs && 2 * sv <= kGnMaxVecs && slabs(2 * sv) >= 256 && (backward || fits(2 * sv))) sv *= 2;
    // A large slab takes its workgroup longer than the chunks' second launch
    // takes, unless half the CUs have one and its pieces fill half a line.
    // Forward: 1 of 64 x 64 x 128 in 32 groups (4096 vectors) 14.3 us, in chunks
    // 13.6; 9 of 24 x 24 x 40 in one (2880) 9.0 and 12.1; backward: 9 of 24 x 24 x 40
    // 15.4 and 13.8, 1 of 16 x 16 x 1280 in 32 (1280) 12.0 and 16.5.  With the CUs
    // full: forward of 32 of 56 x 56 x 256 in 32, 64-byte pieces, 26 and 53; of 8 of
    // 128 x 128 x 128, 16-byte pieces, 66 and 30.
    if (HW * sv > (backward ? 2048 : 3584) && (sv < 4 || slabs(sv) < kGnSlabs)) return false;
    p.resident = fits(sv);
    p.slab = true;
    p.sv = (int)sv;
    p.slabs = (int)((vecs + sv - 1) / sv);
    // Several vectors a thread: what a thread does once (indexes, parameters,
    // its part of the joins) costs as much as four vectors.  Eight forward and
    // four backward, down to 256 threads (forward of 16 of 27 x 27 x 320 12.5
    // us, 15.3 with 1024 threads; of 2 of 16 x 16 x 1280 7.2 and 9.9; backward
    // of 16 of 16 x 16 x 512 13.2 and 15.2).
    const int64_t held = HW * sv, least = backward ? (held < 256 ? held : 256) : (held < 512 ? held / 2 : 256);
    int64_t threads = held / (backward ? 4 : 8);
    threads = threads < least ? least : threads;
    // room for four (eight) pixels a thread where it holds them
    if (p.resident && threads < sv * ((HW + (backward ? 3 : 7)) / (backward ? 4 : 8)))
        threads = sv * ((HW + (backward ? 3 : 7)) / (backward ? 4 : 8));
    threads = threads < sv ? sv : threads;
    threads = (threads + 63) / 64 * 64;
    p.threads = (int)(threads < kGnMaxThreads ? threads : kGnMaxThreads);
    p.pl = (int)(p.threads / sv);
    if (p.pl > HW) p.pl = (int)HW;
    p.nv = 1;
    while (p.resident && p.nv * (int64_t)p.pl < HW) p.nv *= 2;
    if (!p.resident) p.nv = 0;
    return true;
}

static GnPlan gn_plan(int64_t N, int64_t HW, int64_t C, int64_t G, bool backward) {
    GnPlan p{};
    if (slab_plan(p, N, HW, C, G, backward)) {
        p.sum_bytes = round_up(N * C * 8, 256);
        p.bytes = p.sum_bytes;
        return p;
    }
    p = GnPlan{};
    const int64_t vecs = C / 8;
    p.sv = (int)(vecs < kGnThreads ? vecs : kGnThreads);
    p.slabs = (int)((vecs + p.sv - 1) / p.sv);
    p.pl = kGnThreads / p.sv;
    if (p.pl > HW) p.pl = (int)HW;
    p.threads = (p.pl * p.sv + 63) / 64 * 64;
    // a unit of channels lies in one group and one slab
    int64_t uw = C / G;
    for (int64_t q = p.slabs > 1 ? 8 * p.sv : 0; q != 0;) {
        const int64_t r = uw % q;
        uw = q;
        q = r;
    }
    p.uw = (int)uw;
    // A workgroup a CU, two from 16 MB on (4 of 64 x 64 x 320 forward and backward
    // 17.6 and 21.4 us, 21.0 and 24.7 with two, 26.5 and 29.6 with four; 12 of 42 x 30
    // x 1136 47.6 and 85.9, 34.4 and 55.1 with two), of at least two pixels a lane.
    // Every workgroup joins units x chunks pairs after a stream of pixels x
    // vectors / chunks: no more chunks than balance the two, the square root of
    // pixels x vectors / units (1 of 64 x 64 x 320 in 32 groups, 71: 85 chunks 17.3 us,
    // 171 20.1; 1 of 32 x 32 x 640, 50: 43 chunks 15.5 us, 171 19.7).
    const int64_t wanted = N * HW * vecs < (1 << 20) ? 256 : 512;
    int64_t chunks = N > 0 ? (wanted + N * p.slabs - 1) / (N * p.slabs) : 1;
    const int64_t top = (HW + 2 * p.pl - 1) / (2 * p.pl);
    int64_t join = 1;
    while ((join + 1) * (join + 1) <= HW * uw / 8 && join < chunks) ++join;
    if (chunks > top) chunks = top;
    if (chunks > join) chunks = join;
    if (chunks < 1) chunks = 1;
    p.pixels = (int)((HW + chunks - 1) / chunks);
    p.chunks = (int)((HW + p.pixels - 1) / p.pixels);
    p.part_bytes = round_up(N * p.chunks * (C / uw) * 8, 256);
    p.sum_bytes = backward ? round_up(N * p.chunks * C * 8, 256) : 0;
    p.bytes = p.part_bytes + p.sum_bytes;
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

template <bool FP16, bool SINGLE>
static void launch_resident(const GnArgs& a, const GnPlan& pl, hipStream_t stream) {
    const dim3 grid((unsigned)a.grid), block(pl.threads);
    switch (pl.nv) {
        case 1: hipLaunchKernelGGL((gn_resident_kernel<FP16, 1, SINGLE>), grid, block, 0, stream, a); break;
        case 2: hipLaunchKernelGGL((gn_resident_kernel<FP16, 2, SINGLE>), grid, block, 0, stream, a); break;
        case 4: hipLaunchKernelGGL((gn_resident_kernel<FP16, 4, SINGLE>), grid, block, 0, stream, a); break;
        case 8: hipLaunchKernelGGL((gn_resident_kernel<FP16, 8, SINGLE>), grid, block, 0, stream, a); break;
        default: hipLaunchKernelGGL((gn_resident_kernel<FP16, 16, SINGLE>), grid, block, 0, stream, a); break;
    }
}
template <bool FP16, bool SINGLE>
static void launch_backward_slab(const GnArgs& a, const GnPlan& pl, hipStream_t stream) {
    const dim3 grid((unsigned)a.grid), block(pl.threads);
    switch (pl.nv) {
        case 1: hipLaunchKernelGGL((gn_backward_slab_kernel<FP16, 1, SINGLE>), grid, block, 0, stream, a); break;
        case 2: hipLaunchKernelGGL((gn_backward_slab_kernel<FP16, 2, SINGLE>), grid, block, 0, stream, a); break;
        case 4: hipLaunchKernelGGL((gn_backward_slab_kernel<FP16, 4, SINGLE>), grid, block, 0, stream, a); break;
        default: hipLaunchKernelGGL((gn_backward_slab_kernel<FP16, 0, SINGLE>), grid, block, 0, stream, a); break;
    }
}

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
    a.cpg_magic = fastdiv_magic((uint32_t)a.cpg);
    a.param_kind = (int)pt;
    a.act = (int)act;
    a.chunks = pl.chunks;
    a.pixels = pl.pixels;
    a.uw = pl.uw;
    a.rows = pl.slab ? N : N * pl.chunks;
    a.grid = (int)((int64_t)N * (pl.slab ? 1 : pl.chunks) * pl.slabs);
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
    const GnPlan pl = gn_plan(N, HW, C, G, false);
    if (!launchable((int64_t)N * (pl.slab ? 1 : pl.chunks) * pl.slabs, pl.threads)) return IGC_ERR_UNSUPPORTED;
    Workspace ws;
    if (const igc_status_t st = ws.take(pl.slab ? 0 : pl.bytes, user_ws, user_ws_bytes, stream)) return st;
    (void)hipGetLastError();
    GnArgs a = gn_args(pl, N, HW, C, G, gamma, beta, pt, act, ws);
    a.x = x;
    a.out = y;
    a.ldx = ldx;
    a.ldo = ldy;
    if (pl.slab) {
        a.mean = mean;
        a.rstd = rstd;
        a.eps = eps;
        if (a.cpg % 8 == 0)
            launch_resident<FP16, true>(a, pl, stream);
        else
            launch_resident<FP16, false>(a, pl, stream);
        return hipGetLastError() == hipSuccess ? IGC_OK : IGC_ERR_HIP;
    }
    const unsigned grid = (unsigned)a.grid;
    a.mean = mean;
    a.rstd = rstd;
    a.eps = eps;
    hipLaunchKernelGGL(gn_partial_kernel<FP16>, dim3(grid), dim3(pl.threads), 0, stream, a);
    hipLaunchKernelGGL(gn_apply_kernel<FP16>, dim3(grid), dim3(pl.threads), 0, stream, a);
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
    const GnPlan pl = gn_plan(N, HW, C, G, true);
    const unsigned cols = pl.slab || N == 0 ? 32 : 8;  // channels of a workgroup that sums for dgamma and dbeta
    const unsigned params = dgamma || dbeta ? ((unsigned)C + cols - 1) / cols : 0;
    const int64_t images = (int64_t)N * (pl.slab ? 1 : pl.chunks) * pl.slabs;  // workgroups over them
    if (cols == 8 ? !launchable(images + params, pl.threads)
                  : !launchable(images, pl.threads) || !launchable(params, kGnJoinThreads))
        return IGC_ERR_UNSUPPORTED;
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
    a.sums = (float*)((char*)ws.ptr + pl.part_bytes);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    if (N > 0 && !pl.slab) {
        hipLaunchKernelGGL(gn_backward_partial_kernel<FP16>, dim3((unsigned)a.grid), dim3(pl.threads), 0, stream, a);
        hipLaunchKernelGGL(gn_backward_apply_kernel<FP16>, dim3((unsigned)a.grid + params), dim3(pl.threads), 0, stream,
                           a);
    } else {
        if (N > 0 && a.cpg % 8 == 0)
            launch_backward_slab<FP16, true>(a, pl, stream);
        else if (N > 0)
            launch_backward_slab<FP16, false>(a, pl, stream);
        if (params) hipLaunchKernelGGL(gn_param_kernel, dim3(params), dim3(kGnJoinThreads), 0, stream, a);
    }
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
    if (N == 0) return 0;
    const int64_t forward = gn_plan(N, (int64_t)H * W, C, G, false).bytes;
    const int64_t backward = gn_plan(N, (int64_t)H * W, C, G, true).bytes;
    return forward > backward ? forward : backward;
}

}  // extern "C"
