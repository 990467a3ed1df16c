// ffn_backward.cu -- the elementwise halves of the feed-forward backward
// passes: the gradient at the activation, which the two products of each
// backward pass then read as a 16-bit operand.
//
//   linear:  dZ = dC act'(Z),  db = column sums of dZ
//   gated:   dG = dH U act'(G),  dU = dH act(G)
//
// Both stream: 2 (dC) + 4 (Z) + 2 (dZ) bytes a value for the linear layer,
// 2 + 8 + 4 for the gated one, against a few dozen flops, so HBM bounds
// them.  A thread holds 8 neighbouring columns (16 bytes of a 16-bit row, a
// warp 512 contiguous bytes) and walks down rows.
#include <algorithm>

#include "ffn_epilogue.cuh"
#include "ffn_kernels.h"

namespace tsg {

namespace {

constexpr int kStripCols = 256;  // columns of a thread block: 32 threads of 8
constexpr int kRowLanes = 8;     // rows in flight per block
constexpr int kLinearPerSM = 4, kGatedPerSM = 3;  // resident blocks

// 8 fp32 values to the 16-bit row at p, columns [i, i + 8) of n.
template <bool kBF16>
__device__ __forceinline__ void store8_16(void* p, int64_t i, int64_t n, const float (&v)[8]) {
    if (i + 8 <= n) {
        uint4 w;
        w.x = pack16<kBF16>(v[0], v[1]);
        w.y = pack16<kBF16>(v[2], v[3]);
        w.z = pack16<kBF16>(v[4], v[5]);
        w.w = pack16<kBF16>(v[6], v[7]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) store16<kBF16>(p, i + j, v[j]);
    }
}

// Row chunk y covers rows [y M / Y, (y + 1) M / Y).
__device__ __forceinline__ int64_t chunk_begin(int64_t M, int64_t y, int64_t Y) { return y * M / Y; }

// Column sums: each block sums its rows (thread partials in row order, the
// 8 row lanes in lane order), the strip's blocks leave their sums in
// `partials`, and the last of them to arrive adds them in chunk order, so
// the bits do not depend on which block that is.
//
// Four blocks an SM (their 64 registers a thread just hold one row's
// vectors): 4096 x 16384 bf16, gelu, sums alone, 85 us; with 3 blocks 110,
// with 5 91, and with two rows in flight a thread 114 to 129, whatever the
// vector's width.
template <bool kBF16, int kAct>
__global__ void __launch_bounds__(256, kLinearPerSM) linear_grad_sm103(const LinearGradArgs a, const ColumnSums sums) {
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kStripCols + tx * 8;
    const int64_t r1 = chunk_begin(a.M, blockIdx.y + 1, gridDim.y);
    griddep_launch();
    griddep_wait();
    float acc[8] = {};
    if (col < a.N) {
        for (int64_t r = chunk_begin(a.M, blockIdx.y, gridDim.y) + ty; r < r1; r += kRowLanes) {
            float d[8];
            load8_16<kBF16>(static_cast<const uint16_t*>(a.dC) + r * a.lddc, col, a.N, d);
            if constexpr (kAct != kActNone) {
                float z[8];
                load8_f32(a.saved + r * a.lds, col, a.N, z);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    float2 v, dv;
                    act_both<kAct>({z[j], z[j + 1]}, v, dv);
                    d[j] *= dv.x;
                    d[j + 1] *= dv.y;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += d[j];
            if (a.dZ) store8_16<kBF16>(static_cast<uint16_t*>(a.dZ) + r * a.ldz, col, a.N, d);
        }
    }
    if (!a.dbias) return;

    __shared__ float part[kRowLanes][kStripCols];
    __shared__ int is_last;
#pragma unroll
    for (int j = 0; j < 8; ++j) part[ty][tx * 8 + j] = acc[j];
    __syncthreads();
    float total = 0.0f;
#pragma unroll
    for (int k = 0; k < kRowLanes; ++k) total += part[k][threadIdx.x];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kStripCols + threadIdx.x;
    if (gridDim.y > 1) {
        if (c < a.N) sums.partials[static_cast<int64_t>(blockIdx.y) * a.N + c] = total;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0)
            is_last = atom_acq_rel_gpu_add(sums.counters + blockIdx.x, 1) == static_cast<int>(gridDim.y) - 1;
        __syncthreads();
        if (!is_last) return;
        __threadfence();
        total = 0.0f;
        if (c < a.N) {
            // (8 loads in flight; the sum is in chunk order all the same)
            const float* p = sums.partials + c;
            for (int64_t y = 0; y < gridDim.y; y += 8) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = y + k < gridDim.y ? __ldcg(p + (y + k) * a.N) : 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) total += v[k];
            }
        }
        if (threadIdx.x == 0) sums.counters[blockIdx.x] = 0;  // ready for the next launch
    }
    if (c < a.N) {
        if (a.dbias_f32)
            static_cast<float*>(a.dbias)[c] = total;
        else
            store16<kBF16>(a.dbias, c, total);
    }
}

template <bool kBF16, int kAct>
__global__ void __launch_bounds__(256, kGatedPerSM) gated_grad_sm103(const GatedGradArgs a) {
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kStripCols + tx * 8;
    griddep_launch();
    if (col >= a.F) return;
    griddep_wait();
    const int64_t r1 = chunk_begin(a.M, blockIdx.y + 1, gridDim.y);
    for (int64_t r = chunk_begin(a.M, blockIdx.y, gridDim.y) + ty; r < r1; r += kRowLanes) {
        float d[8], g[8], u[8];
        load8_16<kBF16>(static_cast<const uint16_t*>(a.dH) + r * a.lddh, col, a.F, d);
        const float* z = a.saved + r * 2 * a.F;
        load8_f32(z, col, a.F, g);
        load8_f32(z + a.F, col, a.F, u);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float2 dh = {d[j], d[j + 1]};
            float2 v, dv;
            act_both<kAct>({g[j], g[j + 1]}, v, dv);
            const float2 dg = mul2(mul2(dh, {u[j], u[j + 1]}), dv), du = mul2(dh, v);
            g[j] = dg.x, g[j + 1] = dg.y;
            u[j] = du.x, u[j + 1] = du.y;
        }
        uint16_t* out = static_cast<uint16_t*>(a.dGU) + r * 2 * a.F;
        store8_16<kBF16>(out, col, a.F, g);
        store8_16<kBF16>(out + a.F, col, a.F, u);
    }
}

// Calls launch(bf16, activation) with both as compile-time values.
template <class Launch>
cudaError_t by_act(bool bf16, int act, Launch&& launch) {
    auto with = [&](auto b) {
        switch (act) {
            case kActRelu: return launch(b, std::integral_constant<int, kActRelu>{});
            case kActGelu: return launch(b, std::integral_constant<int, kActGelu>{});
            case kActGeluTanh: return launch(b, std::integral_constant<int, kActGeluTanh>{});
            case kActSilu: return launch(b, std::integral_constant<int, kActSilu>{});
            case kActSigmoid: return launch(b, std::integral_constant<int, kActSigmoid>{});
            default: return launch(b, std::integral_constant<int, kActNone>{});
        }
    };
    return bf16 ? with(std::true_type{}) : with(std::false_type{});
}

template <class... Args>
cudaError_t launch_grid(void (*kernel)(Args...), int64_t strips, int64_t chunks, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(strips), static_cast<unsigned>(chunks), 1);
    lc.blockDim = dim3(256, 1, 1);
    lc.stream = stream;
    // The products before and after take most of an SM's shared memory: the
    // same split of it between shared memory and cache spares every SM a
    // change of it at both ends.
    cudaLaunchAttribute attr[2] = {dependent_launch(), {}};
    attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
    attr[1].val.sharedMemCarveout = 100;
    lc.attrs = attr;
    lc.numAttrs = 2;
    return cudaLaunchKernelEx(&lc, kernel, args...);
}

// Row chunks: as many as fill the `slots` blocks that can be resident in
// `rounds` whole rounds or a few more (the fewest that fill nine tenths of
// them, or else those that fill most), of 16 rows at least.  Several rounds
// keep the rows being read at any time close together: gated 4096 x 14336,
// one round 183 us, three 140; the linear layer, whose chunks cost
// partial sums, is as fast with two as with one.
int64_t row_chunks(int64_t M, int64_t strips, int64_t slots, int64_t rounds) {
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>((M + 15) / 16, 65535));
    int64_t best = std::min(most, std::max<int64_t>(1, (rounds - 1) * slots / strips));
    double fill = 0.0;
    for (int64_t y = best; y <= most && strips * y <= (rounds + 3) * slots; ++y) {
        const int64_t blocks = strips * y, full = (blocks + slots - 1) / slots * slots;
        const double f = static_cast<double>(blocks) / static_cast<double>(full);
        if (f > fill) {
            fill = f;
            best = y;
        }
        if (f >= 0.9) break;
    }
    return best;
}

}  // namespace

cudaError_t launch_linear_grad(const LinearGradArgs& a, const ColumnSums& sums, int num_sms, cudaStream_t stream) {
    const int64_t strips = (a.N + kStripCols - 1) / kStripCols;
    int64_t y = row_chunks(a.M, strips, static_cast<int64_t>(num_sms) * kLinearPerSM, 2);
    if (a.dbias) {
        // the partials and counters have to fit; one chunk needs neither
        if (y * a.N > sums.partial_floats) y = sums.partial_floats / a.N;
        if (strips > sums.num_counters || y < 1) y = 1;
    }
    return by_act(a.bf16, a.act, [&](auto b, auto act) {
        return launch_grid(&linear_grad_sm103<decltype(b)::value, decltype(act)::value>, strips, y, stream, a, sums);
    });
}

cudaError_t launch_gated_grad(const GatedGradArgs& a, int num_sms, cudaStream_t stream) {
    const int64_t strips = (a.F + kStripCols - 1) / kStripCols;
    const int64_t y = row_chunks(a.M, strips, static_cast<int64_t>(num_sms) * kGatedPerSM, 3);
    return by_act(a.bf16, a.act, [&](auto b, auto act) {
        return launch_grid(&gated_grad_sm103<decltype(b)::value, decltype(act)::value>, strips, y, stream, a);
    });
}

}  // namespace tsg
