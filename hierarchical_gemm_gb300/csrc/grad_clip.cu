// grad_clip.cu -- the global norm of many tensors, and their clipping by it.
//
//   n = sqrt(sum g^2);   out = g min(1, max_norm / (n + 1e-6))
//
// Two launches: the first reads every value and sums its square, the last
// thread block of it to finish adds the blocks' partials in block order and
// leaves the norm and the coefficient; the second reads again, scales and
// writes.  HBM bounds both (a multiply-add a value).  The tensors' addresses
// and sizes travel in the kernel's parameters, so a call copies nothing to
// the device beforehand.
//
// Squares are summed in fp32 over 32 values and in fp64 from there on.  A
// group of 8 whose fp32 sum could have overflowed or lost its small squares
// is summed again in fp64.
#include <cmath>

#include "ffn_epilogue.cuh"
#include "ffn_kernels.h"
#include "tsgemm.h"

namespace tsg {

namespace {

constexpr int kClipThreads = 256;
constexpr int kVecsPerThread = 4;                                       // 16-byte vectors of 8 16-bit values
constexpr int64_t kChunk = int64_t{kClipThreads} * kVecsPerThread * 8;  // values of a chunk: 8192
constexpr int kMaxTensors = 512;                                        // per launch (the parameters' size)

struct ClipTable {
    const void* in[kMaxTensors];
    void* out[kMaxTensors];
    int64_t numel[kMaxTensors];
    int64_t first[kMaxTensors];  // chunks of the tensors before this one
    uint8_t kind[kMaxTensors];   // ElemKind; bit 7: both addresses 16-byte aligned
    int32_t count;
    int64_t chunks;
};
static_assert(sizeof(ClipTable) + 128 <= 32764, "kernel parameters");

// The tensor that chunk c belongs to.
__device__ __forceinline__ int tensor_of(const ClipTable& t, int64_t c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Values [i, i + 8) of n at p.
__device__ __forceinline__ void load8_any(int kind, bool aligned, const void* p, int64_t i, int64_t n, float (&v)[8]) {
    if (aligned) {
        load8(kind, p, i, n, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = 0.0f;
        if (i + j < n)
            v[j] = kind == kElemF32 ? static_cast<const float*>(p)[i + j]
                                    : (kind == kElemBF16 ? load16<true>(p, i + j) : load16<false>(p, i + j));
    }
}
__device__ __forceinline__ void store8_any(int kind, bool aligned, void* p, int64_t i, int64_t n, const float (&v)[8]) {
    if (aligned && i + 8 <= n) {
        if (kind == kElemF32) {
            float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
            d[0] = make_float4(v[0], v[1], v[2], v[3]);
            d[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint4 w;
            uint32_t* x = &w.x;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = kind == kElemBF16 ? pack16<true>(v[2 * j], v[2 * j + 1]) : pack16<false>(v[2 * j], v[2 * j + 1]);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = w;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (i + j >= n) break;
        if (kind == kElemF32)
            static_cast<float*>(p)[i + j] = v[j];
        else if (kind == kElemBF16)
            store16<true>(p, i + j, v[j]);
        else
            store16<false>(p, i + j, v[j]);
    }
}

__device__ __forceinline__ double block_sum(double x) {
    __shared__ double part[kClipThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kClipThreads / 32; ++w) s += part[w];
    return s;
}

// Chunks blockIdx.x, blockIdx.x + gridDim.x, ...; this launch's partials
// start at `base`, `total` of them come from all launches, and the last
// launch (`final`) makes the norm.
__global__ void __launch_bounds__(kClipThreads) clip_norm_sm103(const __grid_constant__ ClipTable t, double* partials,
                                                                int base, int total, int final, int* counter,
                                                                float max_norm, float* norm, float* coef) {
    double acc = 0.0;
    for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const int k = tensor_of(t, c);
        const int kind = t.kind[k] & 0x7f;
        const bool aligned = t.kind[k] & 0x80;
        const int64_t n = t.numel[k], at = (c - t.first[k]) * kChunk + threadIdx.x * 8;
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < kVecsPerThread; ++v) {
            const int64_t i = at + v * (kClipThreads * 8);
            if (i >= n) break;
            float x[8], q = 0.0f;
            load8_any(kind, aligned, t.in[k], i, n, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) q = fmaf(x[j], x[j], q);
            if (q > 1e37f || q < 1e-30f) {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
                if (top > 0.0f) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc += static_cast<double>(x[j]) * static_cast<double>(x[j]);
                }
            } else {
                s += q;  // (a NaN comes through here)
            }
        }
        acc += static_cast<double>(s);
    }
    const double mine = block_sum(acc);
    __shared__ int is_last;
    if (threadIdx.x == 0) {
        partials[base + blockIdx.x] = mine;
        is_last = 0;
        if (final) is_last = atom_acq_rel_gpu_add(counter, 1) == static_cast<int>(gridDim.x) - 1;
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    double x = 0.0;
    for (int i = threadIdx.x; i < total; i += kClipThreads) x += __ldcg(partials + i);
    x = block_sum(x);
    if (threadIdx.x == 0) {
        const double n = sqrt(x);
        *norm = static_cast<float>(n);
        double f = static_cast<double>(max_norm) / (n + 1e-6);
        if (f > 1.0) f = 1.0;  // (a NaN stays one)
        *coef = static_cast<float>(f);
        *counter = 0;  // ready for the next launch
    }
}

__global__ void __launch_bounds__(kClipThreads) clip_scale_sm103(const __grid_constant__ ClipTable t,
                                                                 const float* coef, int in_place) {
    const float f = *coef;
    if (in_place && f == 1.0f) return;  // nothing to change
    for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const int k = tensor_of(t, c);
        const int kind = t.kind[k] & 0x7f;
        const bool aligned = t.kind[k] & 0x80;
        const int64_t n = t.numel[k], at = (c - t.first[k]) * kChunk + threadIdx.x * 8;
#pragma unroll
        for (int v = 0; v < kVecsPerThread; ++v) {
            const int64_t i = at + v * (kClipThreads * 8);
            if (i >= n) break;
            float x[8];
            load8_any(kind, aligned, t.in[k], i, n, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= f;
            store8_any(kind, aligned, t.out[k], i, n, x);
        }
    }
}

}  // namespace

cudaError_t launch_clip(int64_t count, const void* const* grads, void* const* out, const int64_t* numel,
                        const int32_t* dtype, float max_norm, float* norm, const ClipScratch& scratch, int num_sms,
                        cudaStream_t stream) {
    ClipTable t;
    const int64_t most_blocks = static_cast<int64_t>(num_sms) * 8;
    auto fill = [&](int64_t from, bool* in_place) {
        t.count = 0;
        t.chunks = 0;
        *in_place = true;
        int64_t i = from;
        for (; i < count && t.count < kMaxTensors; ++i) {
            if (numel[i] == 0) continue;
            const int k = t.count++;
            t.in[k] = grads[i];
            t.out[k] = out[i];
            t.numel[k] = numel[i];
            t.first[k] = t.chunks;
            t.chunks += (numel[i] + kChunk - 1) / kChunk;
            const bool aligned =
                ((reinterpret_cast<uintptr_t>(grads[i]) | reinterpret_cast<uintptr_t>(out[i])) & 15u) == 0;
            const int kind = dtype[i] == TSGEMM_F32 ? kElemF32 : (dtype[i] == TSGEMM_BF16 ? kElemBF16 : kElemF16);
            t.kind[k] = static_cast<uint8_t>(kind | (aligned ? 0x80 : 0));
            if (grads[i] != out[i]) *in_place = false;
        }
        return i;
    };
    auto blocks = [&](int64_t limit) {
        const int64_t b = t.chunks < limit ? t.chunks : limit;
        return static_cast<int>(b < 1 ? 1 : b);
    };
    // launches of kMaxTensors non-empty tensors each; their partials share
    // the scratch
    int64_t tables = 0;
    bool same = true;
    for (int64_t i = 0; i < count || tables == 0; ++tables) i = fill(i, &same);
    int64_t per = scratch.max_partials / tables;
    if (per < 1) return cudaErrorInvalidValue;
    if (per > most_blocks) per = most_blocks;
    int base = 0;
    int64_t i = 0;
    for (int64_t k = 0; k < tables; ++k) {
        i = fill(i, &same);
        const int b = blocks(per);
        clip_norm_sm103<<<b, kClipThreads, 0, stream>>>(t, scratch.partials, base, base + b, k == tables - 1,
                                                        scratch.counter, max_norm, norm, scratch.coef);
        base += b;
    }
    i = 0;
    for (int64_t k = 0; k < tables; ++k) {
        i = fill(i, &same);
        if (t.chunks) clip_scale_sm103<<<blocks(most_blocks), kClipThreads, 0, stream>>>(t, scratch.coef, same ? 1 : 0);
    }
    return cudaGetLastError();
}

}  // namespace tsg
