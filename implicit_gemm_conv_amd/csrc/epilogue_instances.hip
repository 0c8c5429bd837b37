// epilogue_instances.hip -- instantiates gemm_epi_kernel for one tile
// configuration (IGC_BM .. IGC_SYNC given on the command line, as
// instances.hip) and one operation family IGC_FAMILY:
//   0: bf16 GEMM, 1: fp16 GEMM (every operand layout, both directions)
//   2: forward convolution (bf16 and fp16, forward direction)
// and registers the table when the library is loaded.
#include "epilogue.hpp"
#include "instances.hpp"

namespace igc {

template <bool FP16, bool AKC, bool BKC, int OPK>
using Here = Cfg<FP16, IGC_BM, IGC_BN, IGC_BK, IGC_D, IGC_W, IGC_MI, IGC_HALF, IGC_LW, IGC_SYNC, AKC, BKC, OPK>;

template <class C, int V, bool BWD>
constexpr const void* kernel_of() {
    if constexpr (!variant_applies<C, V>() || V == RAGGED || (BWD && C::OPK != OP_GEMM))
        return nullptr;
    else
        return reinterpret_cast<const void*>(&gemm_epi_kernel<C, V, BWD>);
}

// The built-in choice splits K on tiles of up to 256 x 128; larger ones, split
// only by request, keep the plain kernel.
template <class C, int V>
constexpr const void* part_of() {
    if constexpr (!variant_applies<C, V>() || V == RAGGED || C::BM * C::BN > 256 * 128)
        return nullptr;
    else
        return reinterpret_cast<const void*>(&gemm_part_kernel<C, V>);
}

template <bool FP16, bool AKC, bool BKC, int OPK>
EpiInstance entry() {
    using C = Here<FP16, AKC, BKC, OPK>;
    return EpiInstance{IGC_BM, IGC_BN, IGC_BK, IGC_D, IGC_W, IGC_MI, IGC_HALF, C::NL, IGC_SYNC, OPK, FP16, AKC, BKC,
                       {{kernel_of<C, PLAIN, false>(), kernel_of<C, UNIFORM_TAP, false>(),
                         kernel_of<C, RAGGED, false>(), kernel_of<C, CONV_GENERIC, false>()},
                        {kernel_of<C, PLAIN, true>(), kernel_of<C, UNIFORM_TAP, true>(), kernel_of<C, RAGGED, true>(),
                         kernel_of<C, CONV_GENERIC, true>()}},
                       {part_of<C, PLAIN>(), part_of<C, UNIFORM_TAP>(), part_of<C, RAGGED>(),
                        part_of<C, CONV_GENERIC>()}};
}

static const EpiInstance kTable[] = {
#if IGC_FAMILY == 0
    entry<false, true, true, OP_GEMM>(), entry<false, true, false, OP_GEMM>(), entry<false, false, true, OP_GEMM>(),
    entry<false, false, false, OP_GEMM>(),
#elif IGC_FAMILY == 1
    entry<true, true, true, OP_GEMM>(), entry<true, true, false, OP_GEMM>(), entry<true, false, true, OP_GEMM>(),
    entry<true, false, false, OP_GEMM>(),
#elif IGC_FAMILY == 2
    entry<false, true, true, OP_FPROP>(), entry<true, true, true, OP_FPROP>(),
#else
#error "IGC_FAMILY must be 0..2"
#endif
};

namespace {
struct Registrar {
    Registrar() { register_epilogues(kTable, (int)(sizeof(kTable) / sizeof(kTable[0]))); }
};
const Registrar registrar;
}  // namespace

}  // namespace igc
