// ffn_rows.cu -- the linear and gated layers for a few rows of X (decoding:
// one token of each of a few sequences), where the weights' bytes are the
// work: every weight is read once and meets at most 16 rows.
//
// A thread block owns strips of output columns; its 8 warps split K, hold
// fp32 sums in registers (tensor-core fragments: mma.sync m16n8k16 with 16
// weight columns as its rows and 8 rows of X as its columns, so that one
// instruction meets 256 weights with 8 rows and arithmetic never limits
// the loads) and add them up in shared memory.  Where there are fewer strips
// than the SMs need, 2, 4 or 8 blocks of a cluster split K further and
// exchange their sums through distributed shared memory.  All sums are added
// in a fixed order.
//
// HBM bounds it, so what counts is bytes in flight: one block an SM, and
// each thread keeps a ring of 16-byte asynchronous copies of the weights it
// will use itself (no barrier guards a slot) that runs ahead across strips,
// over 100 KiB an SM in all.  The copies take a length, so the last partial
// vectors of K and of the columns read as zeros past their end.
//
// The order of k within a fragment is free as long as W and X agree, so a
// thread takes whole 16-byte vectors of W as they lie in memory:
//   W stored N x K: 8 neighbouring k of one column, two fragments' worth;
//   W stored K x N: 8 neighbouring columns at 4 neighbouring k, whose pairs
//     are put together with byte permutations (one for two weights).
#include "ffn_epilogue.cuh"
#include "ffn_kernels.h"
#include "tsgemm.h"

namespace tsg {

namespace {

constexpr int kWarps = 8;

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8).
template <bool kBF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    if constexpr (kBF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Asynchronous copy of the first `bytes` (0 to 16) of 16 bytes to shared
// memory; zeros follow them.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
                 : "memory");
    return v;
}
// Bytes of the 8 values from i on that are below n: 0 to 16.
__device__ __forceinline__ int bytes_in(int64_t i, int64_t n) {
    const int64_t left = n - i;
    return left >= 8 ? 16 : (left > 0 ? static_cast<int>(left) * 2 : 0);
}

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <bool kRCR, int MT>
struct RowsShape {
    static constexpr int kGroup = kRCR ? 16 : 64;  // columns of a group; a strip is two groups
    static constexpr int kStrip = 2 * kGroup;
    static constexpr int kStepK = kRCR ? 32 : 16;  // K of a step
    static constexpr int kFrags = kRCR ? 1 : 4;    // 16-column fragments of a group
    static constexpr int kWVecs = kRCR ? 4 : 8;    // 16-byte vectors of W that a thread takes in a step
    static constexpr int kVecs = kWVecs + MT;      // and of X
    static constexpr int kDepth = kRCR ? 8 : 4;    // steps in flight
    static constexpr int kLd = kStrip + 4;         // row of sums (m) in shared memory, padded against conflicts
    static constexpr uint32_t kStepBytes = kVecs * 32 * 16;  // of a warp's ring
    static constexpr uint32_t kRingBytes = kWarps * kDepth * kStepBytes;
    static constexpr uint32_t kSmemBytes = kRingBytes + (kWarps * 8 + 8 * MT) * kLd * 4u;
};

// kRCR: W stored N x K.  MT: groups of 8 rows of X.  A block's strip is two
// groups of columns: neighbours, or for the gated layer the same columns of
// the gate and of the up half.
template <bool kBF16, bool kRCR, bool kGated, int MT>
__global__ void __launch_bounds__(32 * kWarps, 1) few_rows_sm103(const FewRowsArgs a) {
    using S = RowsShape<kRCR, MT>;
    constexpr int kGroup = S::kGroup, kStrip = S::kStrip, kFrags = S::kFrags, kLd = S::kLd, kDepth = S::kDepth;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    using Row = float[kLd];
    Row* sums = reinterpret_cast<Row*>(smem_raw + S::kRingBytes);  // [8 MT][kLd]
    Row* part = sums + 8 * MT;                                      // [kWarps][8][kLd], one group of 8 rows at a time

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t parts = static_cast<uint32_t>(a.kparts), rank = parts > 1 ? cluster_ctarank() : 0u;
    const int64_t strips = (a.N + (kGated ? kGroup : kStrip) - 1) / (kGated ? kGroup : kStrip);
    const int64_t strip0 = blockIdx.x / parts, strip_step = gridDim.x / parts;

    const uint16_t* W = static_cast<const uint16_t*>(a.W);
    const uint16_t* X = static_cast<const uint16_t*>(a.X);
    // First weight column of group j of a strip, and one past the last it may use.
    auto col0 = [&](int64_t strip, int j) {
        return kGated ? strip * kGroup + j * a.N : strip * kStrip + j * kGroup;
    };
    auto col1 = [&](int j) { return kGated ? a.N + j * a.N : a.N; };

    // This warp's steps of a strip: blocks of kStepK among [k0, k1), every
    // kWarps-th.
    const int64_t blocks = (a.K + S::kStepK - 1) / S::kStepK;
    const int64_t k0 = blocks * rank / parts + warp, k1 = blocks * (rank + 1) / parts;
    const uint32_t ring = smem_u32(smem_raw) + static_cast<uint32_t>(warp) * (kDepth * S::kStepBytes) + lane * 16u;

    // The copies of one step: of the cursor's strip and block, which moves on.
    int64_t cs = k0 < k1 ? strip0 : strips, cb = k0;
    auto issue = [&](uint32_t slot) {
        if (cs < strips) {
            const uint32_t dst = ring + slot * S::kStepBytes;
            const int64_t k = cb * S::kStepK;
            if constexpr (kRCR) {
                // columns g and g + 8 of each group, 8 k
                const int bytes = bytes_in(k + t * 8, a.K);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int64_t n = col0(cs, v >> 1) + g + 8 * (v & 1);
                    const bool in = n < col1(v >> 1) && bytes > 0;
                    cp_async16(dst + v * 512u, in ? W + n * a.ldw + k + t * 8 : W, in ? bytes : 0);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const bool in = g + 8 * i < a.M && bytes > 0;
                    cp_async16(dst + (4 + i) * 512u, in ? X + (g + 8 * i) * a.ldx + k + t * 8 : X, in ? bytes : 0);
                }
            } else {
                // columns 8 g .. + 7 of each group at k + 4 t .. + 3
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    const int64_t n = col0(cs, v >> 2) + 8 * g, row = k + 4 * t + (v & 3);
                    const int bytes = row < a.K ? bytes_in(n, col1(v >> 2)) : 0;
                    cp_async16(dst + v * 512u, bytes ? W + row * a.ldw + n : W, bytes);
                }
                // (8 bytes of X are needed: the 8 values from 4 t - 4 (t % 2) on hold them)
                const int64_t kx = k + 8 * (t >> 1);
                const int bytes = bytes_in(kx, a.K);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const bool in = g + 8 * i < a.M && bytes > 0;
                    cp_async16(dst + (8 + i) * 512u, in ? X + (g + 8 * i) * a.ldx + kx : X, in ? bytes : 0);
                }
            }
            cb += kWarps;
            if (cb >= k1) {
                cb = k0;
                cs += strip_step;
            }
        }
        cp_async_commit();  // (an empty group past the end keeps the count)
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i) issue(i);

    uint32_t slot = 0;
    for (int64_t strip = strip0; strip < strips; strip += strip_step) {
        float d[2][kFrags][MT][4] = {};
        for (int64_t b = k0; b < k1; b += kWarps) {
            cp_async_wait<kDepth - 1>();  // this thread's oldest step has landed
            const uint32_t src = ring + slot * S::kStepBytes;
            uint4 w[S::kWVecs], x[MT];
#pragma unroll
            for (int v = 0; v < S::kWVecs; ++v) w[v] = ld_shared_u4(src + v * 512u);
#pragma unroll
            for (int i = 0; i < MT; ++i) x[i] = ld_shared_u4(src + (S::kWVecs + i) * 512u);
            if constexpr (kRCR) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const uint4 p = w[2 * j], q = w[2 * j + 1];
                        mma_16816<kBF16>(d[j][0][i], p.x, q.x, p.y, q.y, x[i].x, x[i].y);
                        mma_16816<kBF16>(d[j][0][i], p.z, q.z, p.w, q.w, x[i].z, x[i].w);
                    }
            } else {
                // fragment f of a group: its row r is column 8 (r % 8) + 2 f + r / 8
                auto frag = [&](int j, int f, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
                    const uint32_t a0 = __byte_perm(r0, r1, 0x5410), a1 = __byte_perm(r0, r1, 0x7632);
                    const uint32_t a2 = __byte_perm(r2, r3, 0x5410), a3 = __byte_perm(r2, r3, 0x7632);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const uint32_t b0 = t & 1 ? x[i].z : x[i].x, b1 = t & 1 ? x[i].w : x[i].y;
                        mma_16816<kBF16>(d[j][f][i], a0, a1, a2, a3, b0, b1);
                    }
                };
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    frag(j, 0, w[4 * j].x, w[4 * j + 1].x, w[4 * j + 2].x, w[4 * j + 3].x);
                    frag(j, 1, w[4 * j].y, w[4 * j + 1].y, w[4 * j + 2].y, w[4 * j + 3].y);
                    frag(j, 2, w[4 * j].z, w[4 * j + 1].z, w[4 * j + 2].z, w[4 * j + 3].z);
                    frag(j, 3, w[4 * j].w, w[4 * j + 1].w, w[4 * j + 2].w, w[4 * j + 3].w);
                }
            }
            issue(slot);  // the slot's vectors are in registers
            slot = slot + 1 == kDepth ? 0 : slot + 1;
        }

        // A fragment's (row r, column m): thread (g, t) holds rows g and g + 8,
        // columns 2 t and 2 t + 1.  (The strip before has been read: its sums
        // are finished between the same two barriers.)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if (i > 0) __syncthreads();
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int f = 0; f < kFrags; ++f)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int h = v >> 1;
                        const int n = j * kGroup + (kRCR ? g + 8 * h : 8 * g + 2 * f + h);
                        part[warp * 8 + 2 * t + (v & 1)][n] = d[j][f][i][v];
                    }
            __syncthreads();
            for (int x = threadIdx.x; x < 8 * kStrip; x += 32 * kWarps) {
                const int m = x / kStrip, n = x % kStrip;
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += part[w * 8 + m][n];
                sums[8 * i + m][n] = s;
            }
        }
        if (parts > 1)
            cluster_sync();
        else
            __syncthreads();

        // Each block of the cluster finishes its share of the strip's outputs.
        const uint32_t base = smem_u32(&sums[0][0]);
        auto total = [&](int m, int n) {
            if (parts == 1) return sums[m][n];
            float s = 0.0f;
            for (uint32_t r = 0; r < parts; ++r)
                s += ld_shared_cluster_f32(mapa_shared(base + static_cast<uint32_t>(m * kLd + n) * 4u, r));
            return s;
        };
        constexpr int kOutCols = kGated ? kGroup : kStrip;
        const int64_t out0 = strip * kOutCols;
        const FfnEpilogue& e = a.epi;
        for (int i = static_cast<int>(rank) * 32 * kWarps + threadIdx.x; i < 8 * MT * kOutCols;
             i += static_cast<int>(parts) * 32 * kWarps) {
            const int m = i / kOutCols, n = i % kOutCols;
            const int64_t col = out0 + n;
            if (m >= a.M || col >= a.N) continue;
            float z = total(m, n), v;
            if constexpr (kGated) {
                const float u = total(m, n + kGroup);
                if (e.saved) {
                    e.saved[m * e.lds + col] = z;
                    e.saved[m * e.lds + a.N + col] = u;
                }
                with_act(e.act, [&](auto act) { v = act_value<decltype(act)::value>(z); });
                v *= u;
            } else {
                if (e.bias_kind == kElemF32)
                    z += static_cast<const float*>(e.bias)[col];
                else if (e.bias_kind != kElemNone)
                    z += load16<kBF16>(e.bias, col);
                if (e.saved) e.saved[m * e.lds + col] = z;
                with_act(e.act, [&](auto act) { v = act_value<decltype(act)::value>(z); });
                if (e.residual)
                    v += a.out_f32 ? static_cast<const float*>(e.residual)[m * e.ldr + col]
                                   : load16<kBF16>(e.residual, m * e.ldr + col);
            }
            if (a.out_f32)
                static_cast<float*>(a.C)[m * e.ldc + col] = v;
            else
                store16<kBF16>(a.C, m * e.ldc + col, v);
        }
        if (parts > 1) cluster_sync();  // no block leaves or goes on while another reads its sums
    }
}

struct RowsKernel {
    const void* kernel;
    uint32_t smem;
};
// By (bf16, W stored N x K, gated, more than 8 rows).
template <bool kBF16, bool kRCR, bool kGated, int MT>
RowsKernel entry() {
    return {reinterpret_cast<const void*>(&few_rows_sm103<kBF16, kRCR, kGated, MT>), RowsShape<kRCR, MT>::kSmemBytes};
}
RowsKernel rows_kernel(int i) {
    switch (i) {
        case 0: return entry<false, false, false, 1>();
        case 1: return entry<false, false, false, 2>();
        case 2: return entry<false, false, true, 1>();
        case 3: return entry<false, false, true, 2>();
        case 4: return entry<false, true, false, 1>();
        case 5: return entry<false, true, false, 2>();
        case 6: return entry<false, true, true, 1>();
        case 7: return entry<false, true, true, 2>();
        case 8: return entry<true, false, false, 1>();
        case 9: return entry<true, false, false, 2>();
        case 10: return entry<true, false, true, 1>();
        case 11: return entry<true, false, true, 2>();
        case 12: return entry<true, true, false, 1>();
        case 13: return entry<true, true, false, 2>();
        case 14: return entry<true, true, true, 1>();
        default: return entry<true, true, true, 2>();
    }
}

}  // namespace

cudaError_t init_few_rows() {
    for (int i = 0; i < 16; ++i) {
        const RowsKernel k = rows_kernel(i);
        const cudaError_t st =
            cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(k.smem));
        if (st != cudaSuccess) return st;
    }
    return cudaSuccess;
}

cudaError_t launch_few_rows(const FewRowsArgs& args, bool bf16, bool rcr, bool gated, int num_sms, cudaStream_t stream) {
    FewRowsArgs a = args;
    const RowsKernel k = rows_kernel((bf16 ? 8 : 0) + (rcr ? 4 : 0) + (gated ? 2 : 0) + (a.M > 8 ? 1 : 0));
    const int64_t group = rcr ? 16 : 64, cols = gated ? group : 2 * group;
    const int64_t strips = (a.N + cols - 1) / cols;
    // split K until most SMs have a block, as long as every warp keeps two
    // steps
    const int64_t steps = a.K / (rcr ? 32 : 16);
    int parts = 1;
    while (parts < 8 && strips * parts < 100 && steps >= 2 * kWarps * (2 * parts)) parts *= 2;
    a.kparts = parts;
    cudaLaunchConfig_t lc{};
    const int64_t clusters = strips < num_sms / parts ? strips : num_sms / parts;
    lc.gridDim = dim3(static_cast<unsigned>(clusters * parts), 1, 1);
    lc.blockDim = dim3(32 * kWarps, 1, 1);
    lc.dynamicSmemBytes = k.smem;
    lc.stream = stream;
    cudaLaunchAttribute attr{};
    if (parts > 1) {
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = static_cast<unsigned>(parts);
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        lc.attrs = &attr;
        lc.numAttrs = 1;
    }
    void* params[1] = {&a};
    return cudaLaunchKernelExC(&lc, k.kernel, params);
}

}  // namespace tsg
