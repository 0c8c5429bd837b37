// few_rows.hip -- D = epilogue(A * B) for at most 32 rows of A, the products
// of single tokens and small batches.  B, the weights, is read once and is all
// that counts: every workgroup streams its own columns of B from memory
// straight into MFMA operands in registers, with no LDS on the way, and A,
// small enough to stay in the caches, is read beside it.
//
// A workgroup's waves cut its K range among them in turns of UK and add their
// fp32 sums through LDS; where N alone gives too few workgroups K is cut across
// workgroups too (splits), and the split epilogue adds those partials.
//
// A workgroup covers 16*NB columns.  B column-major (K contiguous): NB blocks
// of 16; a lane loads eight consecutive k of one column, which is an operand of
// the 16x16x32 MFMA as it lies.  B row-major (N contiguous): a lane loads NB
// consecutive columns of eight k rows and turns them into NB operands with one
// byte permute per register (two k of one column from two rows), so the MFMA's
// column index is every NB-th column.
//
// Measured, calls of one graph one after the other, weights from memory (in
// brackets: the same weights again, from the last-level cache): 1 x 4096 x 4096
// column-major 8.8 us (7.2; 33.6 MB, 3.8 TB/s), 1 x 16384 x 4096 32.2 (23.2) and
// row-major 28.2 (23.0; 4.8 TB/s), 17 x 8192 x 2048 row-major 13.6 (9.3; 2.5 TB/s:
// two row blocks have operand blocks of 32 columns, 64-byte pieces of a row),
// 1 x 1024 x 1024 column-major 4.0 (3.0).  What is left at 4096 is a launch, a
// first load and the join: 2 us beyond the bytes.  A through LDS instead of
// straight from the caches measured no faster.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epilogue.hpp"
#include "few_rows.hpp"

namespace igc {

typedef __attribute__((ext_vector_type(2))) unsigned u32x2f_t;

// Of a 16-byte piece of a row starting at element k: the elements below `end`, zeros past it.
__device__ __forceinline__ u32x4s_t keep_below(u32x4s_t w, int64_t k, int64_t end) {
    const int n = end - k >= 8 ? 8 : (int)(end - k);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = n >= 2 * i + 2 ? w[i] : (n == 2 * i + 1 ? (w[i] & 0xffffu) : 0u);
    return w;
}

// Eight k of a row, the first of them k: `base` is the row's address of the
// turn's first k (uniform) and `off` the lane's offset from it, so a load needs
// one 32-bit register a lane.  MASKED: zeros at and past `end`, where nothing is read.
template <bool MASKED>
__device__ __forceinline__ u32x4s_t load_k8(const char* base, uint32_t off, int64_t k, int64_t end) {
    if constexpr (MASKED) {
        if (k >= end) return u32x4s_t{0, 0, 0, 0};
        return keep_below(*(const u32x4s_t*)(base + off), k, end);
    } else {
        return *(const u32x4s_t*)(base + off);
    }
}

// One 32-deep step of B for a wave: NB operands of 8 k per lane.  B_KC: NB
// blocks of 16 columns; else the NB neighbouring columns of one load.
template <bool B_KC, int NB>
struct BStep {
    unsigned w[4 * NB];

    // `base`: the step's first k in column n0; off[j]: the lane's eight k and its column of block j (B_KC), off[0]:
    // its eight k and first column.  k: the lane's first k
    template <bool MASKED>
    __device__ __forceinline__ void load(const char* base, const uint32_t (&off)[B_KC ? NB : 1], int64_t ldb, int64_t k,
                                         int64_t end) {
        if constexpr (B_KC) {
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const u32x4s_t v = load_k8<MASKED>(base, off[j], k, end);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[4 * j + i] = v[i];
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const bool in = !MASKED || k + kk < end;
                const char* r = base + kk * ldb * 2 + off[0];
                if constexpr (NB == 8) {
                    u32x4s_t v{0, 0, 0, 0};
                    if (in) v = *(const u32x4s_t*)r;
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[kk * 4 + i] = v[i];
                } else if constexpr (NB == 4) {
                    u32x2f_t v{0, 0};
                    if (in) v = *(const u32x2f_t*)r;
                    w[kk * 2] = v[0], w[kk * 2 + 1] = v[1];
                } else {
                    w[kk] = in ? *(const unsigned*)r : 0u;
                }
            }
        }
    }
    // operand j: the eight k of the lane's column j
    __device__ __forceinline__ i16x8_t operand(int j) const {
        u32x4s_t v;
        if constexpr (B_KC) {
            v = u32x4s_t{w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]};
        } else {
            const unsigned sel = j & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = __builtin_amdgcn_perm(w[(2 * i + 1) * (NB / 2) + j / 2], w[2 * i * (NB / 2) + j / 2], sel);
        }
        return __builtin_bit_cast(i16x8_t, v);
    }
};

// MT: 16-row blocks of A; WAVES; U: 32-deep steps a turn.
template <bool FP16, bool B_KC, int MT, int NB, int WAVES, int U>
__global__ __launch_bounds__(64 * WAVES) void few_rows_kernel(const FewRowsArgs a, const Epi e) {
    using Step = BStep<B_KC, NB>;
    constexpr int COLS = 16 * NB;            // columns of the workgroup
    constexpr int UK = 32 * U;
    constexpr int E = MT * 16 * COLS;        // elements of the workgroup
    constexpr int EPT = (E + 64 * WAVES - 1) / (64 * WAVES);
    __shared__ __attribute__((aligned(16))) float red[WAVES * E];  // [wave][operand block][lane][4]

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int id = xcd_order((int)blockIdx.x, a.cols * a.splits);
    const int split = id / a.cols;
    const int64_t n0 = (int64_t)(id - split * a.cols) * COLS;
    const int64_t kbase = (int64_t)split * a.per;
    const int64_t kend = kbase + a.per < a.K ? kbase + a.per : a.K;

    // columns past N and rows past M repeat the last one: their sums are never stored
    const char* bbase = (const char*)a.B + (B_KC ? n0 * a.ldb : n0) * 2;
    const int64_t bstep = B_KC ? 2 : a.ldb * 2;  // bytes from one k to the next
    const int left = a.N - n0 < COLS ? (int)(a.N - n0) : COLS;
    uint32_t boff[B_KC ? NB : 1];
    if constexpr (B_KC) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
            boff[j] = (uint32_t)((16 * j + r < left ? 16 * j + r : left - 1) * a.ldb + 8 * g) * 2;
    } else {
        boff[0] = (uint32_t)(8 * g * a.ldb + (NB * r < left ? NB * r : (left - 1) / NB * NB)) * 2;
    }
    uint32_t aoff[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) aoff[i] = (uint32_t)((16 * i + r < a.M ? 16 * i + r : a.M - 1) * a.lda + 8 * g) * 2;

    // element x = thread + 64 WAVES t of the workgroup is (x / COLS, x % COLS): what its epilogue reads comes first
    EpiElement el[EPT];
    if (a.splits == 1) {
#pragma unroll
        for (int t = 0; t < EPT; ++t) {
            const int x = (int)threadIdx.x + t * 64 * WAVES, m = x / COLS, c = x % COLS;
            if (x < E && m < a.M && c < left) el[t].fetch(e, m, n0 + c);
        }
    }

    f32x4_t acc[MT][NB];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};

    // B of two turns in flight
    Step cur[U], nxt[U];
    auto load_b = [&](Step (&s)[U], int64_t k) __attribute__((always_inline)) {
        const char* base = bbase + k * bstep;
        if (k + UK <= kend) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                s[u].template load<false>(base + 32 * u * bstep, boff, a.ldb, k + 32 * u + 8 * g, kend);
        } else if (k < kend) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                s[u].template load<true>(base + 32 * u * bstep, boff, a.ldb, k + 32 * u + 8 * g, kend);
        }
    };
    int64_t k = kbase + (int64_t)wave * UK;
    load_b(cur, k);
    for (; k < kend; k += WAVES * UK) {
        u32x4s_t fa[U][MT];
        const char* base = (const char*)a.A + k * 2;
        if (k + UK <= kend) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < MT; ++i) fa[u][i] = load_k8<false>(base + 64 * u, aoff[i], 0, 0);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < MT; ++i) fa[u][i] = load_k8<true>(base + 64 * u, aoff[i], k + 32 * u + 8 * g, kend);
        }
        load_b(nxt, k + WAVES * UK);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const i16x8_t fb = cur[u].operand(j);
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[i][j] = mfma<FP16>(fb, __builtin_bit_cast(i16x8_t, fa[u][i]), acc[i][j]);
            }
#pragma unroll
        for (int u = 0; u < U; ++u) cur[u] = nxt[u];
    }

#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) *(f32x4_t*)&red[((wave * MT + i) * NB + j) * 256 + lane * 4] = acc[i][j];
    __syncthreads();
    // element (m, c) of the workgroup: block (m/16, j), lane 16*(q/4) + m%16, word q%4, where column c is number q of
    // operand j: c = 16*j + q (B_KC) or NB*q + j
#pragma unroll
    for (int t = 0; t < EPT; ++t) {
        const int x = (int)threadIdx.x + t * 64 * WAVES;
        const int m = x / COLS, c = x % COLS;
        if (m >= a.M || c >= left || x >= E) continue;
        const int j = B_KC ? c / 16 : c % NB, q = B_KC ? c % 16 : c / NB;
        const float* src = &red[((m >> 4) * NB + j) * 256 + ((q >> 2) * 16 + (m & 15)) * 4 + (q & 3)];
        float s = src[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += src[w * E];
        if (a.splits > 1)
            a.ws[((int64_t)split * a.M + m) * a.ldws + n0 + c] = s;
        else
            el[t].finish(e, a.C, a.ldc, a.out_kind, m, n0 + c, s);
    }
}

// Against the 64-row tiles of the fused epilogue, whose waves share a tile of A
// and of B and which split K further (time here / time there, geometric means
// over weights in and out of the caches):
//   K <= 2048, N <= 8192, 12 shapes: column-major 0.58 with one row, 0.64 with
//   16, 0.76 with 32; row-major 0.77, 0.89, 1.01 with 24 and 1.08 with 32;
//   larger: column-major with K >= 2048 0.85 with one row, 0.92 with 8, 1.04
//   with 16 (with a smaller K up to 1.28); row-major 0.99 and 1.04, but 0.90 and
//   0.96 for N >= 16384, where a workgroup reads longer pieces of its rows.
bool few_rows_faster(int64_t M, int64_t N, int64_t K, bool b_kc) {
    if (K <= 2048 && N <= 8192) return M <= (b_kc ? kFewRows : 20);
    return M <= 8 && (b_kc ? K >= 2048 : N >= 16384);
}

FewRowsPlan few_rows_plan(int64_t M, int64_t N, int64_t K, bool b_kc) {
    constexpr int64_t kCUs = 256;
    FewRowsPlan pl{};
    const auto cols = [&](int64_t nb) { return (N + 16 * nb - 1) / (16 * nb); };
    // B row-major: the widest operand blocks that still give every CU a
    // workgroup (1 x 16384 x 4096: 28 us with four, 40 with two; 1 x 65536 x 1024:
    // 28.5 with eight, 30.4 with four).  Column-major gains nothing from more.
    pl.nb = b_kc ? 1 : (M <= 16 && cols(8) >= kCUs ? 8 : (M <= 16 && cols(4) >= kCUs ? 4 : 2));
    pl.cols = cols(pl.nb);
    // K is cut across workgroups while CUs are idle and the parts save more than
    // the second launch costs (column-major 1 x 512 x 16000: 9.8 us in six or eight,
    // 12.0 in three; 1 x 1000 x 4096 7.3 whole, 8.2 in two).
    int64_t s = 1;
    if (b_kc && K >= 6144 && pl.cols > 0) {
        s = kCUs / pl.cols < K / 2048 ? kCUs / pl.cols : K / 2048;
        if (s < 1) s = 1;
    }
    const int64_t per = (K + s - 1) / s;
    pl.per = (per + 127) / 128 * 128;
    pl.splits = K > 0 ? (int)((K + pl.per - 1) / pl.per) : 1;
    if (pl.per <= 0) pl.per = 128;
    return pl;
}

template <bool FP16, bool B_KC, int MT, int NB>
static hipError_t go(const FewRowsArgs& a, const Epi& e, hipStream_t stream) {
    // Eight waves; sixteen for B row-major where 128 registers hold their operands, whose smaller turns spread
    // better (17 x 8192 x 2048 12.3 -> 11.1 us).  A turn holds 32 KB of B a workgroup (column-major) or 64 KB.
    constexpr int W = !B_KC && NB <= 4 ? 16 : 8;
    constexpr int U = B_KC ? 4 : (W == 16 ? 4 / NB : 8 / NB);
    hipLaunchKernelGGL((few_rows_kernel<FP16, B_KC, MT, NB, W, U>), dim3((unsigned)(a.cols * a.splits)), dim3(64 * W), 0,
                       stream, a, e);
    return hipGetLastError();
}

template <bool FP16, bool B_KC>
static hipError_t pick_few(const FewRowsArgs& a, const Epi& e, int nb, hipStream_t st) {
    if constexpr (B_KC) {
        return a.M <= 16 ? go<FP16, true, 1, 1>(a, e, st) : go<FP16, true, 2, 1>(a, e, st);
    } else {
        if (a.M > 16) return go<FP16, false, 2, 2>(a, e, st);
        if (nb == 8) return go<FP16, false, 1, 8>(a, e, st);
        return nb == 4 ? go<FP16, false, 1, 4>(a, e, st) : go<FP16, false, 1, 2>(a, e, st);
    }
}

hipError_t launch_few_rows(const FewRowsArgs& a, const Epi& e, bool fp16, bool b_kc, int nb, hipStream_t stream) {
    if (fp16) return b_kc ? pick_few<true, true>(a, e, nb, stream) : pick_few<true, false>(a, e, nb, stream);
    return b_kc ? pick_few<false, true>(a, e, nb, stream) : pick_few<false, false>(a, e, nb, stream);
}

}  // namespace igc
