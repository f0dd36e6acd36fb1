// Kernel argument blocks and launchers of the training-step operators
// (gradient norm, AdamW, RMS norm and its gradient), shared by their kernels
// and gb_train_api.cu.
#pragma once

#include <cuda_fp16.h>
#include <type_traits>

#include "gb_device.cuh"
#include "gb_kernels.cuh"

namespace gb {

// ------------------------------------------------------- many-tensor tables
// A many-tensor call walks warp tiles of kTile elements over all its tensors.
// The table of pointers travels in the kernel's parameters (at most 32,764
// bytes of them), so a call copies nothing to the device, allocates nothing
// and may be captured; calls with more tensors than a table holds are split.
// Copying a large table costs the host 1.5 us a call, so few tensors have a
// small one.
constexpr int kNormTensors = 1024;
constexpr int kAdamwTensors = 512;
constexpr int kFewTensors = 32;

// The place in the table of a warp's piece of work `at`: the first tensor
// whose pieces end beyond it.  A warp's pieces ascend, so it searches only
// when it leaves a tensor.
__device__ __forceinline__ int find_tensor(const uint32_t *end, int n, uint32_t at) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (at < end[mid]) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Elements between the 32-byte boundary at or before p and p: with tiles laid
// from that boundary all but a tensor's first and last tile are whole
// vectors.  `eb` bytes an element; 8 elements are one lane's vector.
inline uint32_t vector_shift(const void *p, size_t eb) { return (uint32_t)(((uintptr_t)p / eb) & 7u); }

// Tiles of a tensor whose first tile starts `shift` elements before element 0.
inline uint64_t tiles_of(uint64_t n, uint32_t shift, uint32_t tile) { return (n + shift + tile - 1) / tile; }

// Device workspace of a context, for the calls that join partial sums: ticket
// counters (the eager calls' one, then one for each captured call, in turn),
// then float64 or float32 partials of the eager calls and of the captured
// ones.  One fixed allocation, made by the first such call and kept: a
// captured call's pointers stay good.
constexpr size_t kWorkHead = 64u << 10;
constexpr size_t kWorkFloats = 8u << 20;

template <int N> struct NormArgs {
    double *partials;    // one per block of every launch of the call
    uint32_t *ticket;    // blocks of the last launch that have finished; 0 between calls
    float *out;          // [2]: norm, factor
    float max_norm;
    uint32_t first_partial;  // of this launch
    int last;                // the call's last launch: its last block joins the partials
    int n_tensors;
    uint32_t tiles;
    const void *grad[N];
    uint64_t numel[N];
    uint32_t tile_end[N];
    unsigned char shift[N];
};
constexpr int kNormPartials = 4096;  // partials of one launch, at most
constexpr int kNormTile = 4 * kTile;

// A tensor whose arrays do not lie alike to a vector: element-wise accesses.
constexpr unsigned short kScattered = 8;

template <int N> struct AdamwArgs {
    float beta1, gain1, beta2, gain2;  // gain = 1 - beta
    float keep;                        // 1 - lr * weight_decay
    float rate;                        // lr / (1 - beta1^step)
    float unroot;                      // 1 / sqrt(1 - beta2^step)
    float eps;
    const float *grad_scale;
    int n_tensors;
    uint32_t span;   // tiles of a span: 1, a warp's; with 8-bit states a block's
    uint32_t spans;  // of all tensors
    unsigned short layout[N];  // vector_shift, or kScattered
    uint32_t key[N];           // of the random numbers
    float *param[N];
    const void *grad[N];
    void *m[N];
    void *v[N];
    void *copy[N];
    uint64_t numel[N];
    uint32_t span_end[N];
};
static_assert(sizeof(NormArgs<kNormTensors>) <= 32764 && sizeof(AdamwArgs<kAdamwTensors>) <= 32764, "kernel parameters");

// ------------------------------------------------------------------- rows
struct RmsArgs {
    const void *x, *residual, *weight;
    void *sum, *out;
    float *rstd;
    uint64_t rows, whole_rows;
    uint32_t cols;
    float eps, inv_cols;
    uint64_t scales_off;  // 8-bit output: byte offset of the scales
    int team;             // threads per row, set by the launcher
};
struct RmsGradArgs {
    const void *dy, *h, *weight, *dsum;
    const float *rstd;
    void *dx, *dweight;
    float *partials;  // [n_partials, cols]
    int n_partials;  // set by the launcher
    uint64_t rows, whole_rows;
    uint32_t cols;
    float inv_cols;
    int team;  // threads per row, set by the launcher
};

// Eight elements of a lane, in a vector's registers.
template <typename T> struct Raw8;
template <> struct Raw8<float> { U8x32 w; };
template <> struct Raw8<__nv_bfloat16> { uint4 w; };
template <> struct Raw8<__half> { uint4 w; };
__device__ __forceinline__ uint4 ld_rw_u4(const void *p) {
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ uint2 ld_rw_u2(const void *p) {
    uint2 r;
    asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float v[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r.w.w[k]);
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16> &r, float v[8]) {
    const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack8(const Raw8<__half> &r, float v[8]) {
    const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*(const __half2 *)&w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
// 32-bit mixing of the random numbers' counters: two multiplications by odd
// constants (hexadecimal digits of pi) between xor-shifts, a bijection.
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t z) {
    z ^= z >> 16;
    z *= 0x85A308D3u;
    z ^= z >> 15;
    z *= 0xEC4E6C89u;
    return z ^ (z >> 16);
}

// Of kFewTensors and kNormTensors, of kFewTensors and kAdamwTensors.
template <int N> cudaError_t launch_grad_norm(const NormArgs<N> &a, int dtype, uint32_t blocks, cudaStream_t s);
uint32_t grad_norm_blocks(uint32_t tiles);
// Tiles a block takes at once with 8-bit states: 32, whose scales fill whole
// sectors and whose two barriers cost little, where that leaves each of an
// SM's 4 blocks two spans or more (64 Mi elements: 176 us; 8 tiles 199 us, 16
// tiles 183 us, 64 tiles 177 us); else 8, one a warp.
inline uint32_t adamw_span(uint64_t elems) { return elems >= (uint64_t)sm_count() * 4 * 2 * 32 * kTile ? 32 : 8; }
template <int N> cudaError_t launch_adamw(const AdamwArgs<N> &a, int dtype, int state_block, bool copies, cudaStream_t s);
cudaError_t launch_rms_norm(RmsArgs &a, int dtype, int codec, int block, cudaStream_t s);
cudaError_t launch_rms_norm_backward(RmsGradArgs &a, int dtype, cudaStream_t s);

// A programmatic dependent launch, as launch_grid's, of any shape.
template <typename Args>
cudaError_t launch_pdl(void (*kern)(Args), dim3 grid, unsigned threads, size_t smem, const Args &a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    count_launch();
    if (e != cudaSuccess) {
        cudaGetLastError();  // clear it: the caller reports e
        return e;
    }
    return cudaGetLastError();
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (sizeof(T) == 4) {
        return 0;
    } else if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *(const uint32_t *)&h;
    } else {
        return cvt_bf16x2(lo, hi);
    }
}
template <typename T>
__device__ __forceinline__ void st8(T *p, const float v[8]) {
    if constexpr (sizeof(T) == 4) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(v[k]);
        st_v8(p, w);
    } else {
        st_u4(p, make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])));
    }
}

// Element types of the operators.
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

}  // namespace gb
