// few_rows.hip -- D = epilogue(A * B) for at most 64 rows of A, the products
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
// Measured (weights from memory, not the caches): 1 x 4096 x 4096 8.0 us
// column-major and 12.0 row-major (33.6 MB), 1 x 16384 x 4096 21.5 and 22.3 (6.2
// TB/s); the 128 x 128 tiles take 36, 35, 24 and 24.  What is left at 4096 is a
// launch, a first load and the join: 2 us beyond the bytes.  A through LDS
// instead of straight from the caches measured no faster.
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

    // element x = thread + 512 t of the workgroup is (x / COLS, x % COLS): what its epilogue reads comes first
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

FewRowsPlan few_rows_plan(int64_t M, int64_t N, int64_t K, bool b_kc) {
    constexpr int64_t kCUs = 256;
    const int64_t mt = (M + 15) / 16;
    FewRowsPlan pl{};
    // The widest operand blocks that still give every CU a workgroup: B
    // row-major reads longer pieces of its rows, and with several blocks of A
    // each is read for more columns (64 x 16384 x 4096: 55 us with two blocks,
    // 82 with one).  One block of A gains nothing from more columns of B.
    pl.nb = b_kc ? (mt == 1 ? 1 : (mt == 2 ? 4 : 2)) : (mt == 1 ? 8 : (mt == 2 ? 4 : 2));
    while (pl.nb > (b_kc ? 1 : 2) && (N + 16 * pl.nb - 1) / (16 * pl.nb) < kCUs) pl.nb /= 2;
    pl.cols = (N + 16 * pl.nb - 1) / (16 * pl.nb);
    // K is cut across workgroups while CUs are idle and every part is long
    // enough to pay for the second launch (1 x 1024 x 4096: column-major 7.0 us
    // whole, 7.7 in four; row-major, whose workgroups are twice as wide, 11.3
    // whole, 9.4 in four; 64 x 1024 x 16384 93 whole, 23 in eight).
    int64_t s = pl.cols > 0 ? kCUs / pl.cols : 1;
    const int64_t part = b_kc ? 4096 : 1024;
    if (s > K / part) s = K / part;
    if (s < 1) s = 1;
    const int64_t per = (K + s - 1) / s;
    pl.per = (per + 127) / 128 * 128;
    pl.splits = K > 0 ? (int)((K + pl.per - 1) / pl.per) : 1;
    if (pl.per <= 0) pl.per = 128;
    return pl;
}

template <bool FP16, bool B_KC, int MT, int NB>
static hipError_t go(const FewRowsArgs& a, const Epi& e, hipStream_t stream) {
    // Eight waves; sixteen for B row-major where 128 registers hold their operands, whose smaller turns spread
    // better (17 x 8192 x 2048 12.3 -> 11.1 us).  A turn holds 16 to 32 KB of B a workgroup.
    constexpr int W = !B_KC && MT <= 2 && NB <= 4 ? 16 : 8;
    constexpr int U = B_KC ? 4 / NB : (W == 16 ? 4 / NB : 8 / NB);
    hipLaunchKernelGGL((few_rows_kernel<FP16, B_KC, MT, NB, W, U>), dim3((unsigned)(a.cols * a.splits)), dim3(64 * W), 0,
                       stream, a, e);
    return hipGetLastError();
}

template <bool FP16, bool B_KC>
static hipError_t pick_few(const FewRowsArgs& a, const Epi& e, int nb, hipStream_t st) {
    const int mt = (a.M + 15) / 16;
    if constexpr (B_KC) {
        if (mt == 1) return go<FP16, true, 1, 1>(a, e, st);
        if (nb == 1) {
            if (mt == 2) return go<FP16, true, 2, 1>(a, e, st);
            if (mt == 3) return go<FP16, true, 3, 1>(a, e, st);
            return go<FP16, true, 4, 1>(a, e, st);
        }
    } else if (mt == 1) {
        if (nb == 8) return go<FP16, false, 1, 8>(a, e, st);
        if (nb == 4) return go<FP16, false, 1, 4>(a, e, st);
        return go<FP16, false, 1, 2>(a, e, st);
    }
    if (mt == 2) return nb == 4 ? go<FP16, B_KC, 2, 4>(a, e, st) : go<FP16, B_KC, 2, 2>(a, e, st);
    if (mt == 3) return go<FP16, B_KC, 3, 2>(a, e, st);
    return go<FP16, B_KC, 4, 2>(a, e, st);
}

hipError_t launch_few_rows(const FewRowsArgs& a, const Epi& e, bool fp16, bool b_kc, int nb, hipStream_t stream) {
    if (fp16) return b_kc ? pick_few<true, true>(a, e, nb, stream) : pick_few<true, false>(a, e, nb, stream);
    return b_kc ? pick_few<false, true>(a, e, nb, stream) : pick_few<false, false>(a, e, nb, stream);
}

}  // namespace igc
