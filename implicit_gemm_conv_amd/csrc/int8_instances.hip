// int8_instances.hip -- the product of 8-bit integers on the mainloop of
// mainloop.hpp, for one tile configuration (IGC_BM .. IGC_SYNC given on the
// command line, as instances.hip).
//
// D = act(sa[m] sb[n] sum_k A[m][k] B[n][k] + bias[n]) + residual.  With K
// together in both operands a 16-byte chunk of 8-bit values lies in LDS and in
// registers as one of 16-bit values does, so the K loop is that of a bf16
// product of K/2 with another instruction (16x16x64 on integers, twice the
// operations in the same time) and integer accumulators: the sum is exact,
// whatever order, tile or split it is taken in.  The epilogue turns it into
// fp32, times the row's scale, as it stages rows, and applies the column's and
// the bias in one step as it reads them back.
//
// 8192 x 8192 x 8192 393 us, 2800 TOP/s (a loop of the instruction alone: 4150);
// 512 x 16384 x 2048 in 256 x 128 tiles 21.8, one round of them.  Smaller tiles
// are bound by the path from memory to LDS: 2048 x 1024 x 16384 in 64 x 128
// tiles 39.5 us, 35 of the 42 bytes a clock that a CU reaches when it does
// nothing but load.  Operands straight to registers (64-byte pieces of rows) took
// 1.5 to 2.5 times as long, counters in place of the barrier 1.4 times; K cut
// among the waves of a workgroup, fragments read a K tile ahead, and more or
// fewer loading waves measured the same.
#include "epilogue.hpp"
#include "int8_gemm.hpp"

namespace igc {

// (a type of its own for every configuration, as the kernels' names are made of it)
template <int BM, int BN, int BK, int D, int NW, int MI, int HALF, int NL, int SYNC>
struct Int8Cfg : Cfg<false, BM, BN, BK, D, NW, MI, HALF, NL, SYNC, true, true, OP_GEMM> {
    using Acc = i32x4_t;
};
using Here = Int8Cfg<IGC_BM, IGC_BN, IGC_BK, IGC_D, IGC_W, IGC_MI, IGC_HALF, IGC_LW, IGC_SYNC>;
static_assert(kInt8<Here> && Here::MI == 16, "the integer instruction is 16x16x64");

template <class C, int PATH>
__global__ __launch_bounds__(C::NT) void gemm_int8_kernel(const Params p, const EpiInt8 e) {
    epi_tile<C, PLAIN, false, PATH>(p, e);
}

template <class C>
constexpr const void* part_of() {
    if constexpr (C::BM * C::BN > 256 * 128)
        return nullptr;
    else
        return reinterpret_cast<const void*>(&gemm_part_kernel<C, PLAIN>);
}

namespace {
struct Registrar {
    Registrar() {
        register_int8(Int8Instance{Instance{IGC_BM, IGC_BN, IGC_BK, IGC_D, IGC_W, IGC_MI, IGC_HALF, Here::NL, IGC_SYNC,
                                            OP_GEMM, false, true, true, true, {}, {}, Here::LDS_BYTES},
                                   reinterpret_cast<const void*>(&gemm_int8_kernel<Here, EPI_ALL>),
                                   reinterpret_cast<const void*>(&gemm_int8_kernel<Here, EPI_LEAN>), part_of<Here>()});
    }
};
const Registrar registrar;
}  // namespace

}  // namespace igc
