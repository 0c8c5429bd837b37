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

// Epilogue of one element whose product is `acc`.
__device__ __forceinline__ void epi_element(const Epi& e, void* out, int64_t ldc, int out_kind, int64_t m, int64_t n,
                                            float acc) {
    float z = acc + (e.bias ? load_kind(e.bias, n, e.bias_kind) : 0.0f);
    const float r = e.res ? load_kind(e.res, m * e.ldr + n, e.res_kind) : 0.0f;
    float y = z;
    if (e.backward) {
        if (e.pre) {
            const float g = load_kind(e.pre, m * e.ldp + n, e.pre_kind);
            with_act(e.act, [&](auto A) __attribute__((always_inline)) { y = z * act_grad_of<decltype(A)::value>(g); });
        }
    } else {
        if (e.pre) store_kind(e.pre, m * e.ldp + n, e.pre_kind, z);
        with_act(e.act, [&](auto A) __attribute__((always_inline)) { y = act_of<decltype(A)::value>(z); });
    }
    store_kind(out, m * ldc + n, out_kind, e.res ? y + r : y);
}

// Epilogue of a tile.  Each wave passes its sub-tile through a private piece
// of the drained ring as fp32, NI block rows at a time (16 KB a wave for the
// largest tile), and reads it back eight consecutive columns a lane, so that
// the residual is read and the output written as 16-byte pieces of whole row
// segments, and everything up to the one rounding happens in fp32.  The
// activation needs the accumulators out of their statically indexed registers
// anyway: it runs in a loop over the staged rows, UQ row groups a turn, and so
// is compiled once per kernel half instead of once per register.  What bounds
// it: one workgroup holds a CU, so nothing covers the tile's 128 KB of output
// and of residual but the other waves' activations; the residual of the next
// UQ row groups is in flight while a turn computes.
//
// Chunk c (16 bytes, four columns) of staged row r lies at c ^ (r & (CPR-1)):
// the 16 rows of an accumulator block are written to distinct banks, and the
// two chunks a lane reads back stay distinct over the lanes of a phase.
template <class C, int I0, int NI, bool BWD, class ML>
__device__ __forceinline__ void epi_rows(ML& ml, const typename C::Acc (&acc)[C::FM][C::FN], IGC_LDS char* reg,
                                         const Params& p, const Epi& e, const float (&bias)[8], int lane, bool vec) {
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
    const int col = (lane % LPR) * 8;
    const int64_t m0 = ml.m0 + ml.wm * C::WTM + 16 * I0 + lane / LPR, n0 = ml.n0 + ml.wn * C::WTN + col;
    const int64_t rows = p.M - m0;  // row group q of this lane is inside while q * RPI < rows
    const int left = p.N - n0 >= 8 ? 8 : (int)(p.N - n0);
    const bool res_raw = e.res && vec && e.res_kind != KIND_F32;
    const bool pre_raw = BWD && e.pre && vec && e.pre_kind != KIND_F32;
    u32x4s_t rv[UQ], gv[UQ];
    auto fetch = [&](int q, int u) __attribute__((always_inline)) {
        const bool in = left > 0 && q * RPI < rows;
        if (res_raw && in) rv[u] = raw8(e.res, (m0 + q * RPI) * e.ldr + n0);
        if (pre_raw && in) gv[u] = raw8(e.pre, (m0 + q * RPI) * e.ldp + n0);
    };
#pragma unroll
    for (int u = 0; u < UQ; ++u) {
        rv[u] = u32x4s_t{0, 0, 0, 0};
        gv[u] = u32x4s_t{0, 0, 0, 0};
        fetch(u, u);
    }
    // the wave's own writes, read back by other lanes of the same wave
    wait_lgkmcnt0();
    compiler_fence();
#pragma unroll 1
    for (int q0 = 0; q0 < NQ; q0 += UQ) {
        float v[UQ][8];
#pragma unroll
        for (int u = 0; u < UQ; ++u) {
            const int row = (q0 + u) * RPI + lane / LPR, c = col / 4, x = row & (CPR - 1);
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
                    if (pre_raw) {
                        decode8(gv[u], e.pre_kind, g[u]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) g[u][i] = 0.0f;
                        if (left > 0 && (q0 + u) * RPI < rows)
                            load8(e.pre, (m0 + (q0 + u) * RPI) * e.ldp + n0, e.pre_kind, left, vec, g[u]);
                    }
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
                    if (left > 0 && (q0 + u) * RPI < rows)
                        store8(e.pre, (m0 + (q0 + u) * RPI) * e.ldp + n0, e.pre_kind, left, vec, v[u]);
            }
            with_act(e.act, [&](auto A) __attribute__((always_inline)) {
#pragma unroll
                for (int u = 0; u < UQ; ++u)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[u][i] = act_of<decltype(A)::value>(v[u][i]);
            });
        }
#pragma unroll
        for (int u = 0; u < UQ; ++u) {
            const bool in = left > 0 && (q0 + u) * RPI < rows;
            if (e.res) {
                float r[8];
                if (res_raw) {
                    decode8(rv[u], e.res_kind, r);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) r[i] = 0.0f;
                    if (in) load8(e.res, (m0 + (q0 + u) * RPI) * e.ldr + n0, e.res_kind, left, vec, r);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] += r[i];
            }
            if (in) store8(p.C, (m0 + (q0 + u) * RPI) * p.ldc + n0, p.out_kind, left, vec, v[u]);
        }
#pragma unroll
        for (int u = 0; u < UQ; ++u)
            if (q0 + UQ + u < NQ) fetch(q0 + UQ + u, u);
    }
    // reads done before the piece is written again
    wait_lgkmcnt0();
    compiler_fence();
}

// Every pass of a wave's sub-tile, at most four block rows each.
template <class C, int I0, bool BWD, class ML>
__device__ __forceinline__ void epi_passes(ML& ml, const typename C::Acc (&acc)[C::FM][C::FN], IGC_LDS char* reg,
                                           const Params& p, const Epi& e, const float (&bias)[8], int lane, bool vec) {
    if constexpr (I0 < C::FM) {
        constexpr int NI = C::FM - I0 < 4 ? C::FM - I0 : 4;
        epi_rows<C, I0, NI, BWD>(ml, acc, reg, p, e, bias, lane, vec);
        epi_passes<C, I0 + NI, BWD>(ml, acc, reg, p, e, bias, lane, vec);
    }
}

// The data-parallel kernel of mainloop.hpp with the epilogue above.  (A K
// split runs the plain kernel and applies the epilogue to the summed partials.)
template <class C, int V, bool BWD>
__global__ __launch_bounds__(C::NT) void gemm_epi_kernel(const Params p, const Epi e) {
    static_assert(variant_applies<C, V>(), "loop variant of another operation");
    static_assert(C::MI == 16 && C::SYNC == 0, "epilogue of the 16x16x32 barrier rings");
    constexpr int PIECE = 4 * 16 * C::WTN * 4;  // a wave's staging area
    static_assert(stage_pieces<C, PIECE>() >= C::NW, "the ring holds every wave's staged rows");
    const int id = xcd_order((int)blockIdx.x, p.tiles_m * p.tiles_n);
    int tm, tn;
    group_coords(id, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    run_tile<C, V>(p, tm, tn, 0, p.K, [&](auto& ml, auto& acc) __attribute__((always_inline)) {
        // opaque copy of the lane: nothing derived from it is computed before, and kept through, the K loop
        int lane = ml.lane;
        asm volatile("" : "+v"(lane));
        const bool vec = p.vec_ok;
        float bias[8];
        const int64_t n0 = ml.n0 + ml.wn * C::WTN + (lane % (C::WTN / 8)) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) bias[i] = e.bias && n0 + i < p.N ? load_kind(e.bias, n0 + i, e.bias_kind) : 0.0f;
        ring_barrier();  // every wave has finished reading the ring
        epi_passes<C, 0, BWD>(ml, acc, stage_piece<C, PIECE>(ml.wave), p, e, bias, lane, vec);
    });
}

}  // namespace igc
