// int8_gemm.hip -- C ABI of the 8-bit integer product: argument checks, choice
// of kernel and launch.  The kernels are in int8_instances.hip (tiles) and
// few_rows.hip (up to 32 rows).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epilogue.hpp"
#include "few_rows.hpp"
#include "host.hpp"
#include "igc.h"
#include "int8_gemm.hpp"
#include "ring.hpp"
#include "split_reduce.hpp"

namespace igc {

constexpr int kMaxInt8 = 16;
static Int8Instance g_int8[kMaxInt8];
static int g_nint8 = 0;

void register_int8(const Int8Instance& instance) {
    if (g_nint8 < kMaxInt8) g_int8[g_nint8++] = instance;
}

static const Int8Instance* find_int8(const igc_tune_t& q) {
    const int loaders = q.loader_waves == 0 ? q.waves : q.loader_waves;
    for (int i = 0; i < g_nint8; ++i) {
        const Instance& e = g_int8[i].tile;
        if (e.bm == q.bm && e.bn == q.bn && e.bk == q.bk && e.d == q.pipe_depth && e.waves == q.waves &&
            e.mfma == (q.mfma == 0 ? 32 : q.mfma) && e.half == q.half_stage && e.loaders == loaders &&
            e.sync == q.ring_sync)
            return &g_int8[i];
    }
    return nullptr;
}

// A K loop over `pairs` of values in at most s parts, each a whole number of ring periods of K tiles of bk pairs.
struct Int8Parts {
    int count;
    int64_t per;
};
static Int8Parts parts_of(int64_t pairs, int64_t s, int bk, int depth, int half) {
    const int64_t unit = (int64_t)bk * Ring::period(Ring::units(depth, half)), per = round_up((pairs + s - 1) / s, unit);
    return {(int)((pairs + per - 1) / per), per};
}

// |A[m][k] B[n][k]| <= 2^14: a sum of fewer than 2^17 of them stays inside 32 bits.
constexpr int64_t kMaxK = (1ll << 17) - 1;

// The cheapest tile and K split by what they cost, in us: launch, first loads
// and epilogue; a K tile of 128 values, whose time grows with what all busy CUs
// load for it, and by a third where rows of K values do not begin on whole
// cache lines; a further round; for a split a second launch and the partials
// twice through memory.  Fitted to 287 shapes, 140 of them with K a multiple of
// 128, with every tile and up to 16 parts: the choice takes 0.5% more than the
// best of them all (geometric mean; 13% at most), and 0.4% on 130 others (9%).
// A split is priced as K / s, which the constants were fitted with, and told as
// the parts that run, which whole ring periods may make fewer.  Priced by those
// parts, 245 of 7695 sizes take another schedule, 0.3% slower (geometric mean;
// 0.84 to 1.28).
//
// Two tiles are this product's own.  32 x 64 is for grids that leave CUs idle,
// where a K tile takes what one CU needs to load it: 64 x 4096 x 4096 8.3 us (64 x
// 64: 9.7), 256 x 2048 x 8192 12.8 (15.8), but 512 x 4096 x 4096 21.9 (16.7).  64 x 64
// in a ring of 5 stages, of which two workgroups still share a CU, takes 16.2 us
// for 512 x 2048 x 8192 (4 stages: 18.3; 8: 16.8) and 0.15 more in the smallest calls.
static igc_tune_t int8_tune(int64_t M, int64_t N, int64_t K) {
    constexpr struct {
        int bm, bn, depth, waves, loaders, half;
        double fixed, round, least, step, load;  // load: for each KB of a K tile with every CU busy
    } kinds[] = {{32, 64, 5, 4, 0, 0, 4.0, 0.67, 0.0, 0.107, 0.0032},
                 {64, 64, 5, 8, 4, 0, 4.3, 1.0, 0.0, 0.122, 0.0051},
                 {64, 128, 4, 8, 4, 0, 4.75, 2.6, 0.0, 0.183, 0.0051},
                 {128, 128, 4, 8, 4, 0, 5.9, 3.9, 0.0, 0.233, 0.0068},
                 {256, 128, 3, 8, 4, 0, 7.8, 6.1, 0.26, 0.353, 0.0084},
                 {256, 256, 2, 8, 4, 1, 12.4, 9.1, 0.84, 0.474, 0.0136}};
    igc_tune_t t = {};
    double best = -1;
    for (const auto& q : kinds) {
        const int64_t tiles = ((M + q.bm - 1) / q.bm) * ((N + q.bn - 1) / q.bn), steps = (K + 127) / 128;
        const double kb = ((double)(M < q.bm ? M : q.bm) + (double)(N < q.bn ? N : q.bn)) * 128.0 / 1024.0;
        const auto step = [&](double busy) {
            const double us = (q.step + kb * q.load * busy) * (K % 128 ? 1.35 : 1.0);
            return us > q.least ? us : q.least;
        };
        for (int64_t s = 1; s <= 16 && (s == 1 || (K / s >= 512 && tiles * s <= 256 && q.bm * q.bn <= 256 * 128)); ++s) {
            const double join = s > 1 ? 3.4 + (double)s * (double)M * (double)N * 8.0 / 5.2e6 : 0.0;
            if (s > 1 && q.fixed + join >= best) break;  // (the join grows with the parts)
            const int64_t work = tiles * s, rounds = (work + 255) / 256;
            const double last = (double)(work - (rounds - 1) * 256) / 256.0;  // of the CUs
            const double cost = q.fixed + (double)(rounds - 1) * q.round +
                          (double)((steps + s - 1) / s) * ((double)(rounds - 1) * step(1.0) + step(last)) + join;
            if (best < 0 || cost < best) {
                best = cost;
                t = igc_tune_t{q.bm, q.bn, 64, q.depth, q.waves, 16, q.half, q.loaders, s > 1 ? (int)s : 0, 0, 0, 0};
            }
        }
    }
    if (t.k_splits > 1) {
        const int count = parts_of(K / 16 * 8, t.k_splits, t.bk, t.pipe_depth, t.half_stage).count;
        t.k_splits = count > 1 ? count : 0;
    }
    return t;
}

struct Int8Plan {
    igc_tune_t tune = {};
    const Int8Instance* inst = nullptr;
    bool valid = true, few = false;
    bool fits = true;         // a schedule that is compiled, in a grid that can be launched
    FewRowsPlan rows = {};
    int S = 1;                // K parts
    int64_t per = 0;          // pairs of K a part
    int64_t ldws = 0, bytes = 0;
};

// Sizes beyond these are refused before a schedule is looked for.
static bool sizes_too_large(int64_t M, int64_t N, int64_t K) { return K > kMaxK || M >= (1ll << 31) || N >= (1ll << 31); }

static Int8Plan plan_of(const igc_tune_t* tune, int64_t M, int64_t N, int64_t K) {
    Int8Plan pl;
    const int64_t pairs = K / 16 * 8;  // what the K loop runs to; the last K % 16 are added after it
    if (!tune && M >= 1 && M <= kFewRows && few_rows_int8_faster(M, N, K)) {
        pl.few = true;
        pl.rows = few_rows_int8_plan(M, N, K);
        pl.fits = N < (1ll << 30) && launchable(pl.rows.cols * pl.rows.splits, 512);
        pl.ldws = round_up(N, 4);
        pl.bytes = pl.rows.splits > 1 ? round_up(pl.rows.splits * M * pl.ldws * 4, 256) : 0;
        return pl;
    }
    pl.tune = tune ? *tune : int8_tune(M, N, K);
    pl.inst = find_int8(pl.tune);
    pl.valid = pl.tune.stream_k >= 0 && pl.tune.sk_hybrid == 0 && !(pl.tune.k_splits > 1 && pl.tune.stream_k > 0);
    pl.fits = pl.inst && pl.tune.stream_k <= 0;
    if (!pl.fits) return pl;
    const Instance& t = pl.inst->tile;
    if (pl.tune.k_splits > 1 && pairs > 0) {
        const Int8Parts parts = parts_of(pairs, pl.tune.k_splits, t.bk, t.d, t.half);
        pl.per = parts.per;
        pl.S = parts.count;
    }
    const int64_t tiles = ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
    pl.fits = tiles <= 0x7fffffff && launchable(tiles * pl.S, 64 * t.waves);
    if (pl.fits && pl.S > 1) {
        pl.fits = pl.inst->part && launchable((M * ((N + 7) / 8) + 255) / 256, 256);
        pl.ldws = round_up(N, 4);
        pl.bytes = round_up((int64_t)pl.S * M * pl.ldws * 4, 256);
    }
    return pl;
}

static igc_status_t check_epilogue(const igc_epilogue_t* q, int64_t N, EpiInt8& e) {
    e = EpiInt8{};
    if (!q) return IGC_OK;
    if ((int)q->act < IGC_ACT_NONE || (int)q->act > IGC_ACT_SILU || (q->backward != 0 && q->backward != 1))
        return IGC_ERR_INVALID_VALUE;
    if (q->backward) return IGC_ERR_UNSUPPORTED;
    e.act = (int)q->act;
    if (q->bias) {
        if (!valid_type(q->bias_type)) return IGC_ERR_INVALID_VALUE;
        if (reinterpret_cast<uintptr_t>(q->bias) % out_size(q->bias_type)) return IGC_ERR_MISALIGNED;
        e.bias = q->bias;
        e.bias_kind = (int)q->bias_type;
    }
    const auto matrix = [&](const void* ptr, int64_t ld, igc_out_t type) {
        if (!valid_type(type) || ld < N) return IGC_ERR_INVALID_VALUE;
        return !aligned16(ptr) || ld * out_size(type) % 16 != 0 ? IGC_ERR_MISALIGNED : IGC_OK;
    };
    if (q->residual) {
        if (const igc_status_t st = matrix(q->residual, q->ldr, q->residual_type)) return st;
        e.res = q->residual;
        e.ldr = q->ldr;
        e.res_kind = (int)q->residual_type;
    }
    if (q->pre) {
        if (const igc_status_t st = matrix(q->pre, q->ldp, q->pre_type)) return st;
        e.pre = q->pre;
        e.ldp = q->ldp;
        e.pre_kind = (int)q->pre_type;
    }
    return IGC_OK;
}

static igc_status_t int8_any(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* sa,
                             const int8_t* B, int64_t ldb, const float* sb, void* D, int64_t ldd, igc_out_t dt,
                             const igc_epilogue_t* epi, const igc_tune_t* tune, void* user_ws, int64_t user_ws_bytes,
                             hipStream_t stream) {
    if (M < 0 || N < 0 || K < 0 || !valid_type(dt)) return IGC_ERR_INVALID_VALUE;
    EpiInt8 e;
    if (const igc_status_t st = check_epilogue(epi, N, e)) return st;
    e.sa = sa;
    e.sb = sb;
    if (sizes_too_large(M, N, K)) return IGC_ERR_UNSUPPORTED;
    const Int8Plan pl = plan_of(tune, M, N, K);
    if (!pl.valid) return IGC_ERR_INVALID_VALUE;
    if (!pl.fits) return IGC_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return IGC_OK;
    if (!D || ldd < N) return IGC_ERR_INVALID_VALUE;
    if (K > 0) {
        if (!A || !B || lda < K || ldb < K) return IGC_ERR_INVALID_VALUE;
        if (!aligned16(A) || !aligned16(B) || lda % 16 != 0 || ldb % 16 != 0) return IGC_ERR_MISALIGNED;
    }
    if (!aligned16(D) || ldd * out_size(dt) % 16 != 0 || (reinterpret_cast<uintptr_t>(sa) & 3u) ||
        (reinterpret_cast<uintptr_t>(sb) & 3u))
        return IGC_ERR_MISALIGNED;

    // per-tile buffer offsets are 32-bit: one tile's rows span less than 2^31 bytes
    constexpr int64_t kSpan = 0x7fff0000ll;
    if (lda > kSpan || ldb > kSpan || ldd > kSpan || e.ldr > kSpan || e.ldp > kSpan) return IGC_ERR_UNSUPPORTED;
    if (pl.few) {
        if (M * lda >= kSpan || 64 * ldb + 256 >= kSpan) return IGC_ERR_UNSUPPORTED;
        Workspace ws;
        if (const igc_status_t st = ws.take(pl.bytes, user_ws, user_ws_bytes, stream)) return st;
        (void)hipGetLastError();
        FewRowsArgs a{};
        a.A = A;
        a.B = B;
        a.C = D;
        a.ws = (float*)ws.ptr;
        a.N = N;
        a.K = K;
        a.lda = lda;
        a.ldb = ldb;
        a.ldc = ldd;
        a.ldws = pl.ldws;
        a.per = pl.rows.per;
        a.M = (int)M;
        a.cols = (int)pl.rows.cols;
        a.splits = pl.rows.splits;
        a.out_kind = (int)dt;
        hipError_t err = launch_few_rows_int8(a, e, stream);
        if (err == hipSuccess && pl.rows.splits > 1)
            err = launch_split_epilogue((const int*)a.ws, pl.rows.splits, M * a.ldws, M, N, a.ldws, D, ldd, (int)dt, e,
                                        stream);
        return err == hipSuccess ? IGC_OK : IGC_ERR_HIP;
    }

    const Instance& t = pl.inst->tile;
    const int64_t tiles_m = (M + t.bm - 1) / t.bm, tiles_n = (N + t.bn - 1) / t.bn;
    const auto span = [&](int64_t ld, int kind) { return t.bm * ld * (kind == OUT_F32 ? 4 : 2) >= kSpan; };
    const bool split = pl.S > 1;
    if (t.bm * lda + 2 * t.bk >= kSpan || t.bn * ldb + 2 * t.bk >= kSpan || (split && t.bm * pl.ldws * 4 >= kSpan) ||
        (!split && (span(ldd, (int)dt) || (e.res && span(e.ldr, e.res_kind)) || (e.pre && span(e.ldp, e.pre_kind)))))
        return IGC_ERR_UNSUPPORTED;
    const void* fn = split ? pl.inst->part : (e.act == ACT_NONE && !e.pre ? pl.inst->lean : pl.inst->fn);
    Workspace ws;
    if (const igc_status_t st = ws.take(pl.bytes, user_ws, user_ws_bytes, stream)) return st;
    (void)hipGetLastError();  // launch errors below are ours alone
    Params p = {};
    p.A = A;
    p.B = B;
    p.C = D;
    p.M = M;
    p.N = N;
    p.K = K / 16 * 8;
    p.lda = lda / 2;
    p.ldb = ldb / 2;
    p.ldc = ldd;
    p.tiles_m = (int)tiles_m;
    p.tiles_n = (int)tiles_n;
    p.out_kind = (int)dt;
    p.group_m = 8;
    p.k_ragged8 = (int)(K % 16);
    p.vec_ok = 1;
    p.k_splits = pl.S;
    p.k_per_split = split ? pl.per : (p.K > 0 ? p.K : 1);
    p.ws = (float*)ws.ptr;
    p.ldws = pl.ldws;
    p.ws_stride = M * pl.ldws;
    void* args[] = {&p, &e};  // (the kernel of a part takes the first alone)
    hipError_t err = hipLaunchKernel(fn, dim3((unsigned)(tiles_m * tiles_n * pl.S)), dim3(64 * t.waves), args, 0, stream);
    if (err == hipSuccess && split)
        err = launch_split_epilogue((const int*)p.ws, pl.S, p.ws_stride, M, N, p.ldws, D, ldd, (int)dt, e, stream);
    if (err != hipSuccess) return IGC_ERR_HIP;
    return hipGetLastError() == hipSuccess ? IGC_OK : IGC_ERR_HIP;
}

}  // namespace igc

using namespace igc;

extern "C" {

igc_status_t gemm_int8(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* scale_a,
                       const int8_t* B, int64_t ldb, const float* scale_b, void* D, int64_t ldd, igc_out_t d_type,
                       const igc_epilogue_t* epilogue, igc_stream_t stream) {
    return int8_any(M, N, K, A, lda, scale_a, B, ldb, scale_b, D, ldd, d_type, epilogue, nullptr, nullptr, 0,
                    (hipStream_t)stream);
}

igc_status_t gemm_int8_ex(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* scale_a,
                          const int8_t* B, int64_t ldb, const float* scale_b, void* D, int64_t ldd, igc_out_t d_type,
                          const igc_epilogue_t* epilogue, const igc_tune_t* tune, void* workspace,
                          int64_t workspace_bytes, igc_stream_t stream) {
    return int8_any(M, N, K, A, lda, scale_a, B, ldb, scale_b, D, ldd, d_type, epilogue, tune, workspace,
                    workspace_bytes, (hipStream_t)stream);
}

int64_t igc_gemm_int8_workspace_bytes(int64_t M, int64_t N, int64_t K, const igc_tune_t* tune) {
    if (M < 0 || N < 0 || K < 0 || sizes_too_large(M, N, K)) return -1;
    const Int8Plan pl = plan_of(tune, M, N, K);
    if (!pl.valid || !pl.fits) return -1;
    return M == 0 || N == 0 ? 0 : pl.bytes;
}

int igc_gemm_int8_default_tune(int64_t M, int64_t N, int64_t K, igc_tune_t* out) {
    if (!out || M < 0 || N < 0 || K < 0 || sizes_too_large(M, N, K)) return 0;
    const Int8Plan pl = plan_of(nullptr, M, N, K);
    if (!pl.fits) return 0;
    if (pl.few) {
        *out = igc_tune_t{};
        out->bn = 16 * pl.rows.nb;
        out->k_splits = pl.rows.splits;
        return 1;
    }
    *out = pl.tune;
    return 1;
}

}  // extern "C"
