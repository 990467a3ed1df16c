// kernels_ffn_linear_2sm_l0.cu -- instantiations of the CTA-pair kernel with the
// epilogue of a linear layer, RRR operand layout: every tile width and output format.
#include "gemm_sm103_2sm.cuh"
#include "kernels.h"

namespace tsg {

namespace {
template <int BN>
const void* pick(int out) {
    switch (out) {
        case kOutF16: return reinterpret_cast<const void*>(&gemm_sm103_2sm<BN, kOutF16, 0, false, kEpiLinear>);
        case kOutBF16: return reinterpret_cast<const void*>(&gemm_sm103_2sm<BN, kOutBF16, 0, false, kEpiLinear>);
        case kOutF32: return reinterpret_cast<const void*>(&gemm_sm103_2sm<BN, kOutF32, 0, false, kEpiLinear>);
        default: return nullptr;
    }
}
}  // namespace

const void* kernel_linear_2sm_layout0(int block_n, int out_kind) {
    switch (block_n) {
        case 128: return pick<128>(out_kind);
        case 256: return pick<256>(out_kind);
        case 512: return pick<512>(out_kind);
        default: return nullptr;
    }
}

}  // namespace tsg
