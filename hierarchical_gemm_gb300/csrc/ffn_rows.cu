// ffn_rows.cu -- the linear and gated layers for a few rows of X (decoding:
// one token of each of a few sequences), where the weights' bytes are the
// work: every weight is read once and meets at most 32 rows.
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
// each warp keeps a ring of 16-byte asynchronous copies of its own (no
// block-wide barrier guards a slot) that runs ahead across strips, over
// 100 KiB an SM in all.  The copies take a length, so the last partial
// vectors of K and of the columns read as zeros past their end.  Measured, one
// row, bf16, in a chain: 28672 x 4096 (N x K) 36 us, 6.5 TB/s, 0.96 of the
// copy rate; 14336 x 8192 (K x N) 39; 4096 x 4096 7.2, where the launch is a
// third (registers in place of the rings: 41, 50 and 12.6).
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
    // Blocks an SM, and steps in flight of each, as many as shared memory
    // holds.  W stored N x K with more than 8 rows of X has two shallower
    // blocks, whose arithmetic overlaps (8192 x 8192: 16 rows 28.8 -> 27.9 us,
    // 32 rows 38.4 -> 33.8); the other forms are faster with one.
    static constexpr int kPerSM = kRCR && MT > 1 ? 2 : 1;
    static constexpr int kDepth = kRCR ? (MT == 1 ? 8 : (MT == 2 ? 4 : 3)) : (MT > 2 ? 3 : 4);
    static constexpr int kLd = kStrip + 4;         // row of sums (m) in shared memory, padded against conflicts
    static constexpr uint32_t kStepBytes = kVecs * 32 * 16;  // of a warp's ring
    static constexpr uint32_t kRingBytes = kWarps * kDepth * kStepBytes;
    static constexpr uint32_t kSmemBytes = kRingBytes + (kWarps * 8 + 8 * MT) * kLd * 4u;
};

// kRCR: W stored N x K.  MT: groups of 8 rows of X.  A block's strip is two
// groups of columns: neighbours, or for the gated layer the same columns of
// the gate and of the up half.
template <bool kBF16, bool kRCR, bool kGated, int MT>
__global__ void __launch_bounds__(32 * kWarps, (RowsShape<kRCR, MT>::kPerSM)) few_rows_sm103(const FewRowsArgs a) {
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
    //
    // Who copies what: W stored N x K, each thread its own vectors.  Stored
    // K x N, 8 neighbouring threads copy 128 bytes of a row (thread (g, t)
    // copying its own would touch 4 rows at a time in 16-byte pieces, and
    // ask L2 for every 32-byte sector twice), so thread l copies the vectors
    // of thread (gl, tl) = (l mod 8, l / 8); both sides address a vector by
    // (g, t) in an order free of bank conflicts.
    const uint32_t warp_ring = smem_u32(smem_raw) + static_cast<uint32_t>(warp) * (kDepth * S::kStepBytes);
    auto place = [](int vg, int vt) { return static_cast<uint32_t>(vt * 8 + (vg ^ (2 * vt))) * 16u; };
    const int gl = lane & 7, tl = lane >> 3;
    const uint32_t ring_wr = warp_ring + (kRCR ? lane * 16u : place(gl, tl));
    const uint32_t ring_rd = warp_ring + (kRCR ? lane * 16u : place(g, t));
    // (X for W stored K x N: 16-byte vectors of 8 k, two a row)
    const uint32_t ring_rdx = warp_ring + (kRCR ? lane * 16u : place(g, t >> 1));

    // The copies of one step: of the cursor's strip and block, which moves on.
    // Addresses are kept and moved along (pw: this thread's first vector of W
    // in the step; its others lie `vec_off` further on), and what may be read
    // of each is worked out once a strip; the last, partial block of K looks
    // at every vector again.
    const int vg = kRCR ? g : gl, vt = kRCR ? t : tl;         // the vectors' place in a step
    const int64_t vec_k = kRCR ? 8 * vt : 4 * vt;             // first k of them, of the step
    const int64_t step_elems = kRCR ? S::kStepK * kWarps : S::kStepK * kWarps * a.ldw;
    const int64_t group_off = kRCR ? (kGated ? a.N : kGroup) * a.ldw : (kGated ? a.N : kGroup);
    auto vec_off = [&](int v) {
        return kRCR ? (v >> 1) * group_off + (v & 1) * 8 * a.ldw : (v >> 2) * group_off + (v & 3) * a.ldw;
    };
    constexpr int kColSets = kRCR ? 4 : 2;  // vectors of W that can differ in their columns
    int64_t cs = k0 < k1 ? strip0 : strips, cb = k0;
    const uint16_t* pw = W;
    const uint16_t* px = X;
    int wbytes[kColSets];
    auto enter_strip = [&] {
        if (cs >= strips) return;
        if constexpr (kRCR) {
            pw = W + (col0(cs, 0) + vg) * a.ldw + cb * S::kStepK + vec_k;
            px = X + vg * a.ldx + cb * S::kStepK + vec_k;
#pragma unroll
            for (int v = 0; v < 4; ++v) wbytes[v] = col0(cs, v >> 1) + vg + 8 * (v & 1) < col1(v >> 1) ? 16 : 0;
        } else {
            pw = W + (cb * S::kStepK + vec_k) * a.ldw + col0(cs, 0) + 8 * vg;
            px = X + vg * a.ldx + cb * S::kStepK + 8 * vt;
#pragma unroll
            for (int j = 0; j < 2; ++j) wbytes[j] = bytes_in(col0(cs, j) + 8 * vg, col1(j));
        }
    };
    enter_strip();
    // (with two blocks an SM the next kernel's would move in beside these,
    // unevenly: 4096 x 4096, 32 rows, 14.9 us against 11.8)
    if constexpr (S::kPerSM == 1) griddep_launch();
    griddep_wait();
    auto issue = [&](uint32_t slot) {
        if (cs < strips) {
            const uint32_t dst = ring_wr + slot * S::kStepBytes;
            const bool whole = (cb + 1) * S::kStepK <= a.K;
            const int64_t k = cb * S::kStepK + vec_k;
#pragma unroll
            for (int v = 0; v < S::kWVecs; ++v) {
                int bytes = wbytes[kRCR ? v : v >> 2];
                if (!whole) {
                    if constexpr (kRCR)
                        bytes = bytes ? bytes_in(k, a.K) : 0;
                    else
                        bytes = k + (v & 3) < a.K ? bytes : 0;
                }
                cp_async16(dst + v * 512u, bytes ? pw + vec_off(v) : W, bytes);
            }
            if (kRCR || vt < 2) {  // (W stored K x N: a row of X has two vectors in a step)
                const int xbytes = whole ? 16 : bytes_in(cb * S::kStepK + 8 * vt, a.K);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int bytes = vg + 8 * i < a.M ? xbytes : 0;
                    cp_async16(dst + (S::kWVecs + i) * 512u, bytes ? px + 8 * i * a.ldx : X, bytes);
                }
            }
            cb += kWarps;
            pw += step_elems;
            px += S::kStepK * kWarps;
            if (cb >= k1) {
                cb = k0;
                cs += strip_step;
                enter_strip();
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
            if constexpr (!kRCR) __syncwarp();  // and so have the other threads'
            const uint32_t src = ring_rd + slot * S::kStepBytes, srcx = ring_rdx + slot * S::kStepBytes;
            uint4 w[S::kWVecs], x[MT];
#pragma unroll
            for (int v = 0; v < S::kWVecs; ++v) w[v] = ld_shared_v4(src + v * 512u);
#pragma unroll
            for (int i = 0; i < MT; ++i) x[i] = ld_shared_v4(srcx + (S::kWVecs + i) * 512u);
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
            if constexpr (!kRCR) __syncwarp();  // every thread has its vectors in registers
            issue(slot);
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
                with_act(e.act, [&](auto act) { v = act_value<decltype(act)::value>(splat(z)).x; });
                v *= u;
            } else {
                if (e.bias_kind == kElemF32)
                    z += static_cast<const float*>(e.bias)[col];
                else if (e.bias_kind != kElemNone)
                    z += load16<kBF16>(e.bias, col);
                if (e.saved) e.saved[m * e.lds + col] = z;
                with_act(e.act, [&](auto act) { v = act_value<decltype(act)::value>(splat(z)).x; });
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
    int per_sm;
};
template <bool kBF16, bool kRCR, bool kGated, int MT>
RowsKernel entry() {
    using S = RowsShape<kRCR, MT>;
    static_assert(S::kPerSM * (S::kSmemBytes + 1024) <= 233472, "shared memory of an SM");
    return {reinterpret_cast<const void*>(&few_rows_sm103<kBF16, kRCR, kGated, MT>), S::kSmemBytes, S::kPerSM};
}
template <bool kBF16, bool kRCR, bool kGated>
RowsKernel by_rows(int groups) {
    return groups == 1 ? entry<kBF16, kRCR, kGated, 1>()
                       : (groups == 2 ? entry<kBF16, kRCR, kGated, 2>() : entry<kBF16, kRCR, kGated, 4>());
}
// groups of 8 rows: 1, 2 or 4
RowsKernel rows_kernel(bool bf16, bool rcr, bool gated, int groups) {
    if (bf16) {
        if (rcr) return gated ? by_rows<true, true, true>(groups) : by_rows<true, true, false>(groups);
        return gated ? by_rows<true, false, true>(groups) : by_rows<true, false, false>(groups);
    }
    if (rcr) return gated ? by_rows<false, true, true>(groups) : by_rows<false, true, false>(groups);
    return gated ? by_rows<false, false, true>(groups) : by_rows<false, false, false>(groups);
}

}  // namespace

cudaError_t init_few_rows() {
    for (int i = 0; i < 24; ++i) {
        const RowsKernel k = rows_kernel(i & 1, i & 2, i & 4, 1 << (i >> 3));
        const cudaError_t st =
            cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(k.smem));
        if (st != cudaSuccess) return st;
    }
    return cudaSuccess;
}

bool few_rows_fit(int64_t M, int64_t N, int64_t K, bool rcr, bool gated, int num_sms) {
    if (M <= 8) return true;
    if (M > kFewRows) return false;
    if (M > 16 && (gated ? 2 * N : N) * K > (int64_t{1} << 26)) return false;
    const int64_t cols = gated ? 64 : 128;
    return rcr || (N + cols - 1) / cols <= num_sms;
}

cudaError_t launch_few_rows(const FewRowsArgs& args, bool bf16, bool rcr, bool gated, int num_sms, cudaStream_t stream) {
    FewRowsArgs a = args;
    const RowsKernel k = rows_kernel(bf16, rcr, gated, a.M <= 8 ? 1 : (a.M <= 16 ? 2 : 4));
    const int64_t group = rcr ? 16 : 64, cols = gated ? group : 2 * group;
    const int64_t strips = (a.N + cols - 1) / cols;
    // Fewer strips than SMs: split K as many ways as most of the SMs can hold
    // at once (of clusters of 8 fewer fit: they do not fill a GPC), as long as
    // every warp keeps a step.  (Clusters that walk
    // over several strips lose more in their barriers than the evener load
    // gives: 8192 x 14336, 256 strips, 74 us against 40.)
    const int64_t steps = a.K / (rcr ? 32 : 16);
    int parts = 1;
    while (parts < 8 && strips * 2 * parts <= (parts == 4 ? num_sms * 2 / 3 : num_sms * 7 / 8) &&
           steps >= kWarps * 2 * parts)
        parts *= 2;
    a.kparts = parts;
    cudaLaunchConfig_t lc{};
    const int64_t room = static_cast<int64_t>(num_sms) * k.per_sm / parts;
    const int64_t clusters = strips < room ? strips : room;
    lc.gridDim = dim3(static_cast<unsigned>(clusters * parts), 1, 1);
    lc.blockDim = dim3(32 * kWarps, 1, 1);
    lc.dynamicSmemBytes = k.smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[2] = {dependent_launch(), {}};
    if (parts > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(parts);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
    }
    lc.attrs = attr;
    lc.numAttrs = parts > 1 ? 2 : 1;
    void* params[1] = {&a};
    return cudaLaunchKernelExC(&lc, k.kernel, params);
}

}  // namespace tsg
