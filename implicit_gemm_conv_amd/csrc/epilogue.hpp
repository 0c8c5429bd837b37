// epilogue.hpp -- bias, activation and residual applied to the accumulators of
// the mainloop (mainloop.hpp) before they are rounded, once, to the output:
//   forward:   z = (A*B)[m][n] + bias[n];  pre = round(z) if kept;
//              D = round(act(z) + residual[m][n])
//   backward:  D = round(z * act'(pre[m][n]) + residual[m][n])
#pragma once
#include "activation.hpp"
#include "mainloop.hpp"

namespace igc {

// Plain values only: passed to the kernels by value.
struct Epi {
    const void* bias;  // N values, or nullptr
    const void* res;   // M x N, rows ldr apart, or nullptr
    void* pre;         // M x N, rows ldp apart: written (forward) or read (backward); nullptr: none
    int64_t ldr, ldp;
    int bias_kind, res_kind, pre_kind;
    int act;
    int backward;
};

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

// Epilogue of one element: what it reads, then the rest.
struct EpiElement {
    float bias = 0.0f, res = 0.0f, pre = 0.0f;
    __device__ __forceinline__ void fetch(const Epi& e, int64_t m, int64_t n) {
        if (e.bias) bias = load_kind(e.bias, n, e.bias_kind);
        if (e.res) res = load_kind(e.res, m * e.ldr + n, e.res_kind);
        if (e.backward && e.pre) pre = load_kind(e.pre, m * e.ldp + n, e.pre_kind);
    }
    __device__ __forceinline__ void finish(const Epi& e, void* out, int64_t ldc, int out_kind, int64_t m, int64_t n,
                                           float acc) const {
        const float z = acc + bias;
        float y = z;
        if (e.backward) {
            if (e.pre)
                with_act(e.act, [&](auto A) __attribute__((always_inline)) {
                    y = z * act_grad_of<decltype(A)::value>(pre);
                });
        } else {
            if (e.pre) store_kind(e.pre, m * e.ldp + n, e.pre_kind, z);
            with_act(e.act, [&](auto A) __attribute__((always_inline)) { y = act_of<decltype(A)::value>(z); });
        }
        store_kind(out, m * ldc + n, out_kind, e.res ? y + res : y);
    }
};

// Epilogue of a tile.  Each wave passes its sub-tile through a private piece
// of the drained ring as fp32, NI block rows at a time (16 KB a wave for the
// largest tile), and reads it back eight consecutive columns a lane, so that
// the residual is read and the output written as 16-byte pieces of whole row
// segments, and everything up to the one rounding happens in fp32.  The
// activation needs the accumulators out of their statically indexed registers
// anyway: it runs in a loop over the staged rows, UQ row groups a turn, and so
// is compiled once per pass instead of once per register.  What bounds it: one
// workgroup holds a CU, so nothing covers the tile's output and residual but
// the other waves of the same tile.  Rows and columns outside are left out by
// buffer offsets past the end, not by branches: loads and stores retire in one
// order, and with a known number of stores between, the wait for the next
// turn's residual, requested before them, leaves them in flight.
//
// Measured, 4096 x 4096 x 1024 on 256 x 256 tiles: 31.0 us without an epilogue, 33.4
// through this one with nothing to do, bias 34.1, gelu_tanh 36.5, gelu 42.0,
// residual 37.0, pre kept 37.1, the backward form 41.8.
//
// Chunk c (16 bytes, four columns) of staged row r lies at c ^ (r & (CPR-1)):
// the 16 rows of an accumulator block are written to distinct banks, and the
// two chunks a lane reads back stay distinct over the lanes of a phase.
typedef __attribute__((ext_vector_type(4))) int i32x4e_t;
typedef __attribute__((ext_vector_type(2))) unsigned u32x2e_t;

// One of the matrices beside the product: a buffer at the wave's sub-tile and
// the byte distance of its rows and of eight columns.
struct EpiMatrix {
    __amdgpu_buffer_rsrc_t rs;
    uint32_t first, step;  // the lane's offset in row group 0, and from one group to the next
    int kind;
    __device__ __forceinline__ EpiMatrix(const void* base, int64_t ld, int kind_, int64_t m, int64_t n, int row, int col,
                                         int rpi)
        : kind(kind_) {
        const int esz = kind == KIND_F32 ? 4 : 2;
        rs = make_rsrc_u((const char*)base + (m * ld + n) * esz);
        first = (uint32_t)((row * ld + col) * esz);
        step = (uint32_t)(rpi * ld * esz);
    }
    __device__ __forceinline__ u32x4s_t load(int q, bool in, int half) const {
        return __builtin_bit_cast(u32x4s_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                rs, in ? first + q * step + 16 * half : kOob, 0, 0));
    }
    __device__ __forceinline__ void store(int q, bool in, int half, u32x4s_t w) const {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4e_t, w), rs,
                                               in ? first + q * step + 16 * half : kOob, 0, 0);
    }
    // eight values of row group q; `left` of them lie in the row
    __device__ __forceinline__ void load8(int q, bool in, int left, float (&v)[8]) const {
        if (kind == KIND_F32) {
            const f32x4s_t lo = __builtin_bit_cast(f32x4s_t, load(q, in, 0));
            const f32x4s_t hi = __builtin_bit_cast(f32x4s_t, load(q, in && left > 4, 1));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
        } else {
            decode8(load(q, in, 0), kind, v);
        }
    }
    // The same, written.  tail: N % 8, what `left` is where it is less than eight: that piece goes out as its four,
    // two and one values, behind a branch that only waves at the end of the rows take (with a loop over its values
    // 1894 x 5071 x 88 took 27.9 us on 256 x 256 tiles, against 17.7 for 5072 columns; now 17.1).
    __device__ __forceinline__ void store8(int q, bool in, int left, int tail, const float (&v)[8]) const {
        const bool whole = in && left >= 8, part = in && left < 8;
        if (kind == KIND_F32) {
            store(q, whole, 0, __builtin_bit_cast(u32x4s_t, f32x4s_t{v[0], v[1], v[2], v[3]}));
            store(q, whole, 1, __builtin_bit_cast(u32x4s_t, f32x4s_t{v[4], v[5], v[6], v[7]}));
            if (tail && __builtin_amdgcn_ballot_w64(part)) {
                const int at = part ? (int)(first + q * step) : (int)kOob;
                const auto rest = [&](float x, float y, float z, int o) __attribute__((always_inline)) {
                    if (tail & 2) {
                        __builtin_amdgcn_raw_buffer_store_b64(
                            u32x2e_t{__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y)}, rs, o, 0, 0);
                        if (tail & 1)
                            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, z), rs, part ? o + 8 : o, 0, 0);
                    } else if (tail & 1) {
                        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, x), rs, o, 0, 0);
                    }
                };
                if (tail & 4) {
                    store(q, part, 0, __builtin_bit_cast(u32x4s_t, f32x4s_t{v[0], v[1], v[2], v[3]}));
                    rest(v[4], v[5], v[6], part ? at + 16 : at);
                } else {
                    rest(v[0], v[1], v[2], at);
                }
            }
        } else {
            const u32x4s_t w = kind == KIND_BF16 ? pack8<false>(v) : pack8<true>(v);
            store(q, whole, 0, w);
            if (tail && __builtin_amdgcn_ballot_w64(part)) {
                const int at = part ? (int)(first + q * step) : (int)kOob;
                // (branches, not selects: those between two elements of a register array go through scratch)
                const auto rest = [&](unsigned x, unsigned y, int o) __attribute__((always_inline)) {
                    if (tail & 2) {
                        __builtin_amdgcn_raw_buffer_store_b32(x, rs, o, 0, 0);
                        if (tail & 1) __builtin_amdgcn_raw_buffer_store_b16((unsigned short)y, rs, part ? o + 4 : o, 0, 0);
                    } else if (tail & 1) {
                        __builtin_amdgcn_raw_buffer_store_b16((unsigned short)x, rs, o, 0, 0);
                    }
                };
                if (tail & 4) {
                    __builtin_amdgcn_raw_buffer_store_b64(u32x2e_t{w[0], w[1]}, rs, at, 0, 0);
                    rest(w[2], w[3], part ? at + 8 : at);
                } else {
                    rest(w[0], w[1], at);
                }
            }
        }
    }
};

template <class C, int I0, int NI, bool BWD, class ML>
__device__ __forceinline__ void epi_rows(ML& ml, const typename C::Acc (&acc)[C::FM][C::FN], IGC_LDS char* reg,
                                         const Params& p, const Epi& e, const float (&bias)[8], int lane) {
    constexpr int RB = C::WTN * 4, CPR = RB / 16;
    constexpr int LPR = C::WTN / 8;  // lanes per row
    constexpr int RPI = 64 / LPR;    // rows per group
    constexpr int NQ = NI * 16 / RPI;
    constexpr int UQ = NQ % 4 == 0 && !BWD ? 4 : (NQ % 2 == 0 ? 2 : 1);  // (four spill in the backward form)
    static_assert(NQ >= 1 && NI * 16 % RPI == 0, "whole row groups");
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            const int row = 16 * i + (lane & 15), c = 4 * j + (lane >> 4);
            *(IGC_LDS f32x4_t*)(reg + row * RB + ((c ^ (row & (CPR - 1))) << 4)) = acc[I0 + i][j];
        }
    const int row0 = lane / LPR, col = (lane % LPR) * 8;
    const int64_t m0 = ml.m0 + ml.wm * C::WTM + 16 * I0, n0 = ml.n0 + ml.wn * C::WTN;
    const int left = p.N - (n0 + col) >= 8 ? 8 : (int)(p.N - (n0 + col));
    // row group q of this lane is inside while q * RPI < rows
    const int rows = left > 0 ? (p.M - (m0 + row0) < 4096 ? (int)(p.M - (m0 + row0)) : 4096) : 0;
    const EpiMatrix out(p.C, p.ldc, p.out_kind, m0, n0, row0, col, RPI);
    const EpiMatrix res(e.res ? e.res : p.C, e.ldr, e.res_kind, m0, n0, row0, col, RPI);
    const EpiMatrix pre(e.pre ? e.pre : p.C, e.ldp, e.pre_kind, m0, n0, row0, col, RPI);
    const bool res_raw = e.res && e.res_kind != KIND_F32;
    const bool pre_raw = BWD && e.pre && e.pre_kind != KIND_F32;
    u32x4s_t rv[UQ], gv[UQ];
    auto fetch = [&](int q) __attribute__((always_inline)) {
        if (res_raw) {
#pragma unroll
            for (int u = 0; u < UQ; ++u) rv[u] = res.load(q + u, (q + u) * RPI < rows, 0);
        }
        if (pre_raw) {
#pragma unroll
            for (int u = 0; u < UQ; ++u) gv[u] = pre.load(q + u, (q + u) * RPI < rows, 0);
        }
    };
#pragma unroll
    for (int u = 0; u < UQ; ++u) rv[u] = gv[u] = u32x4s_t{0, 0, 0, 0};
    fetch(0);
    // the wave's own writes, read back by other lanes of the same wave
    wait_lgkmcnt0();
    compiler_fence();
#pragma unroll 1
    for (int q0 = 0; q0 < NQ; q0 += UQ) {
        float v[UQ][8];
#pragma unroll
        for (int u = 0; u < UQ; ++u) {
            const int row = (q0 + u) * RPI + row0, c = col / 4, x = row & (CPR - 1);
            const f32x4_t lo = *(const IGC_LDS f32x4_t*)(reg + row * RB + ((c ^ x) << 4));
            const f32x4_t hi = *(const IGC_LDS f32x4_t*)(reg + row * RB + (((c + 1) ^ x) << 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[u][i] = lo[i] + bias[i], v[u][4 + i] = hi[i] + bias[4 + i];
        }
        if constexpr (BWD) {
            if (e.pre) {
                float g[UQ][8];
#pragma unroll
                for (int u = 0; u < UQ; ++u) {
                    if (pre_raw)
                        decode8(gv[u], e.pre_kind, g[u]);
                    else
                        pre.load8(q0 + u, (q0 + u) * RPI < rows, left, g[u]);
                }
                with_act(e.act, [&](auto A) __attribute__((always_inline)) {
#pragma unroll
                    for (int u = 0; u < UQ; ++u)
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[u][i] *= act_grad_of<decltype(A)::value>(g[u][i]);
                });
            }
        } else {
            if (e.pre) {
#pragma unroll
                for (int u = 0; u < UQ; ++u)
                    pre.store8(q0 + u, (q0 + u) * RPI < rows, left, (int)(p.N & 7), v[u]);
            }
            with_act(e.act, [&](auto A) __attribute__((always_inline)) {
#pragma unroll
                for (int u = 0; u < UQ; ++u)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[u][i] = act_of<decltype(A)::value>(v[u][i]);
            });
        }
        if (e.res) {
#pragma unroll
            for (int u = 0; u < UQ; ++u) {
                float r[8];
                if (res_raw)
                    decode8(rv[u], e.res_kind, r);
                else
                    res.load8(q0 + u, (q0 + u) * RPI < rows, left, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] += r[i];
            }
        }
        if (q0 + UQ < NQ) fetch(q0 + UQ);
#pragma unroll
        for (int u = 0; u < UQ; ++u)
            out.store8(q0 + u, (q0 + u) * RPI < rows, left, (int)(p.N & 7), v[u]);
    }
    // reads done before the piece is written again
    wait_lgkmcnt0();
    compiler_fence();
}

// Every pass of a wave's sub-tile, at most four block rows each.
template <class C, int I0, bool BWD, class ML>
__device__ __forceinline__ void epi_passes(ML& ml, const typename C::Acc (&acc)[C::FM][C::FN], IGC_LDS char* reg,
                                           const Params& p, const Epi& e, const float (&bias)[8], int lane) {
    if constexpr (I0 < C::FM) {
        constexpr int NI = C::FM - I0 < 4 ? C::FM - I0 : 4;
        epi_rows<C, I0, NI, BWD>(ml, acc, reg, p, e, bias, lane);
        epi_passes<C, I0 + NI, BWD>(ml, acc, reg, p, e, bias, lane);
    }
}

// The last K % 8 (p.k_ragged8) of K, past the p.K that the loop ran to: one more
// MFMA a block, its operands straight from memory, zeros for the k that are not
// there and in place of what lies past a row's end.  The loop stays the one for
// whole chunks; the one that mends straddling chunks in LDS needs registers that
// 256 x 256 tiles do not have (4096 x 4096 x 1001: 84 us with it, 41 with this).
template <class C, class ML>
__device__ __forceinline__ void add_k_tail(const Params& p, const ML& ml, typename C::Acc (&acc)[C::FM][C::FN], int lane) {
    auto piece = [&](const void* base, int64_t ld, bool k_contiguous, int64_t row) __attribute__((always_inline)) {
        u32x4s_t w{0, 0, 0, 0};
        if (lane < 16) {  // the lanes of an operand's first eight k
            if (k_contiguous) {
                w = raw8(base, row * ld + p.K);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = p.k_ragged8 >= 2 * i + 2 ? w[i] : (p.k_ragged8 == 2 * i + 1 ? (w[i] & 0xffffu) : 0u);
            } else {
#pragma unroll
                for (int k = 0; k < 7; ++k)
                    if (k < p.k_ragged8)
                        w[k / 2] |= (unsigned)((const unsigned short*)base)[(p.K + k) * ld + row] << (16 * (k & 1));
            }
        }
        return __builtin_bit_cast(i16x8_t, w);
    };
    const int r = lane & 15;
    i16x8_t fb[C::FN];
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        const int64_t n = ml.n0 + ml.wn * C::WTN + 16 * j + r;
        fb[j] = piece(p.B, p.ldb, C::B_KC, n < p.N ? n : p.N - 1);
    }
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
        const int64_t m = ml.m0 + ml.wm * C::WTM + 16 * i + r;
        const i16x8_t fa = piece(p.A, p.lda, C::A_KC, m < p.M ? m : p.M - 1);
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = mfma<C::FP16>(fb[j], fa, acc[i][j]);
    }
}

// The data-parallel kernel of mainloop.hpp with the epilogue above.  (A K
// split writes fp32 partials and applies the epilogue to their sum.)
template <class C, int V, bool BWD>
__global__ __launch_bounds__(C::NT) void gemm_epi_kernel(const Params p, const Epi e) {
    static_assert(variant_applies<C, V>(), "loop variant of another operation");
    static_assert(C::MI == 16 && C::SYNC == 0, "epilogue of the 16x16x32 barrier rings");
    constexpr int PIECE = 4 * 16 * C::WTN * 4;  // a wave's staging area
    static_assert(stage_pieces<C, PIECE>() >= C::NW, "the ring holds every wave's staged rows");
    const int id = xcd_order((int)blockIdx.x, p.tiles_m * p.tiles_n);
    int tm, tn;
    group_coords(id, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    float bias[8];
    const auto load_bias = [&](int64_t n0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) bias[i] = e.bias && n0 + i < p.N ? load_kind(e.bias, n0 + i, e.bias_kind) : 0.0f;
    };
    // The bias of tiles of up to 128 x 128 waits for nothing if it is asked for before the K loop (1000 x 500 x 250
    // 5.96 and 5.80 us, 1024 x 1024 x 1024 7.53 and 7.38); larger ones have no registers to keep it in.
    constexpr bool EARLY = C::BM * C::BN <= 128 * 128;
    if constexpr (EARLY)
        load_bias((int64_t)tn * C::BN + (int)(threadIdx.x >> 6) % C::WN * C::WTN + ((int)threadIdx.x & 63) % (C::WTN / 8) * 8);
    run_tile<C, V>(p, tm, tn, 0, p.K, [&](auto& ml, auto& acc) __attribute__((always_inline)) {
        // opaque copy of the lane: nothing derived from it is computed before, and kept through, the K loop
        int lane = ml.lane;
        asm volatile("" : "+v"(lane));
        if constexpr (!EARLY) load_bias(ml.n0 + ml.wn * C::WTN + (lane % (C::WTN / 8)) * 8);
        if constexpr (C::OPK == OP_GEMM)
            if (p.k_ragged8) add_k_tail<C>(p, ml, acc, lane);
        ring_barrier();  // every wave has finished reading the ring
        epi_passes<C, 0, BWD>(ml, acc, stage_piece<C, PIECE>(ml.wave), p, e, bias, lane);
    });
}

// One split of a K split: the fp32 partial tile to the workspace, staged like
// the epilogue so that it is written as whole row segments whatever M and N
// (the plain kernel's stores fall back to single elements in edge tiles: 100 x
// 200 x 8192 in 16 parts 16.5 us with them, 11.4 staged; 1000 x 512 x 8192 in
// 4 parts 24.4 and 20.1).  Columns up to ldws, N rounded up to 4, are the
// workspace's own.  A kernel of its own: with the split's indexes in
// gemm_epi_kernel the 256 x 256 tiles lost 1 us of 35.
template <class C, int V>
__global__ __launch_bounds__(C::NT) void gemm_part_kernel(const Params p) {
    constexpr int PIECE = 4 * 16 * C::WTN * 4, RB = C::WTN * 4, CPR = RB / 16;
    constexpr int RPI = 64 / CPR;  // rows a group: a lane holds one chunk
    static_assert(stage_pieces<C, PIECE>() >= C::NW, "the ring holds every wave's staged rows");
    const int T = p.tiles_m * p.tiles_n;
    const int id = xcd_order((int)blockIdx.x, T * p.k_splits);
    const int split = id / T;
    int tm, tn;
    group_coords(id - split * T, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    const int64_t kbase = (int64_t)split * p.k_per_split;
    const int64_t kend = kbase + p.k_per_split < p.K ? kbase + p.k_per_split : p.K;
    run_tile<C, V>(p, tm, tn, kbase, kend, [&](auto& ml, auto& acc) __attribute__((always_inline)) {
        int lane = ml.lane;
        asm volatile("" : "+v"(lane));
        IGC_LDS char* reg = stage_piece<C, PIECE>(ml.wave);
        if constexpr (C::OPK == OP_GEMM)
            if (p.k_ragged8 && split == p.k_splits - 1) add_k_tail<C>(p, ml, acc, lane);
        ring_barrier();  // every wave has finished reading the ring
        static_for<0, (C::FM + 3) / 4>([&](auto PASS) __attribute__((always_inline)) {
            constexpr int I0 = 4 * PASS, NI = C::FM - I0 < 4 ? C::FM - I0 : 4;
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < C::FN; ++j) {
                    const int row = 16 * i + (lane & 15), c = 4 * j + (lane >> 4);
                    *(IGC_LDS f32x4_t*)(reg + row * RB + ((c ^ (row & (CPR - 1))) << 4)) = acc[I0 + i][j];
                }
            const int row0 = lane / CPR, c = lane % CPR;
            const int64_t m0 = ml.m0 + ml.wm * C::WTM + 16 * I0, n0 = ml.n0 + ml.wn * C::WTN;
            const int rows = n0 + 4 * c < p.ldws ? (p.M - (m0 + row0) < 4096 ? (int)(p.M - (m0 + row0)) : 4096) : 0;
            const EpiMatrix out(p.ws + (int64_t)split * p.ws_stride, p.ldws, KIND_F32, m0, n0, row0, 4 * c, RPI);
            wait_lgkmcnt0();
            compiler_fence();
#pragma unroll
            for (int q = 0; q < NI * 16 / RPI; ++q) {
                const int row = q * RPI + row0;
                const u32x4s_t v = *(const IGC_LDS u32x4s_t*)(reg + row * RB + ((c ^ (row & (CPR - 1))) << 4));
                out.store(q, q * RPI < rows, 0, v);
            }
            wait_lgkmcnt0();
            compiler_fence();
        });
    });
}

}  // namespace igc
