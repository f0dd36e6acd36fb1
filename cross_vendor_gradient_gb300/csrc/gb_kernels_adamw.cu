// The global gradient norm and the AdamW step over many tensors (sm_103a).
//
// Norm.  norm = sqrt(sum of g^2 over every element of every tensor); factor =
// what clipping to max_norm multiplies gradients with.  Each lane adds the
// squares of 32 elements at a time to a compensated float32 sum, and goes over
// its elements once more where they are too small or too large for that;
// lanes and blocks are joined in float64 and in a fixed order, so the result
// does not change from run to run.
//
// AdamW (decoupled weight decay), float32:
//   g = grad * grad_scale
//   m = beta1 m + (1 - beta1) g;   v = beta2 v + (1 - beta2) g^2
//   p = p (1 - lr wd) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
// The products and sums of m and v are rounded one by one, without
// contraction, so that any IEEE arithmetic gives their bits.
// Both are pure streaming: a few operations for 2 .. 28 bytes an element.
#include "gb_train.cuh"

namespace gb {

// ------------------------------------------------------------------- norm
// Read once, so the lines are evicted first.
template <typename T>
__device__ __forceinline__ Raw8<T> ld_grad8(const T *p) {
    if constexpr (sizeof(T) == 4) return {ld_stream_v8(p)};
    else return {ld_stream_u4(p)};
}

// What tells whether any of a lane's elements is not zero, signs aside.
template <typename T>
__device__ __forceinline__ void gather_bits(const Raw8<T> &r, uint32_t &bits) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k) bits |= r.w.w[k];
    } else {
        bits |= r.w.x | r.w.y | r.w.z | r.w.w;
    }
}

// A lane's sum of squares where float32 cannot take it.  Gradients times 2^96
// for a lane whose squares are small (all others have vanished next to the
// least sum that is taken as it is), times 2^-4 for one whose sum has
// overflowed: infinite only if a single square is, NaN only if a gradient is.
template <typename T, int N>
__device__ __forceinline__ double rescaled_squares(const NormArgs<N> &a, bool small) {
    const int lane = threadIdx.x & 31;
    const float scale = small ? 0x1p96f : 0x1p-4f;
    double sum = 0.0;
    for (uint32_t tile = blockIdx.x * 8 + (threadIdx.x >> 5); tile < a.tiles; tile += gridDim.x * 8) {
        const int t = find_tensor(a.tile_end, a.n_tensors, tile);
        const uint64_t shift = a.shift[t], n = a.numel[t] + shift, base = (uint64_t)(tile - (t ? a.tile_end[t - 1] : 0)) * kNormTile;
        const T *g = (const T *)a.grad[t] - shift;
        const bool whole = base >= shift && base + kNormTile <= n;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            float s = 0.0f, top = 0.0f;
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
                const uint64_t j = whole ? base + i * kTile + 8 * lane + k : base + 128 * k + 32 * i + lane;
                const float x = j >= shift && j < n ? to_f32(g[j]) : 0.0f;
                top = fmaxf(top, __fmul_rn(x, x));
                s = fmaf(x * scale, x * scale, s);
            }
            sum += (double)(isinf(top) && !isnan(s) ? top : s);
        }
    }
    return sum * (small ? 0x1p-192 : 0x1p8);
}

// Blocks of an SM, and of the grid for each SM: all that 40 registers leave
// room for, so that every block runs from the start (1.1 G bf16 elements: 303
// us, 7.3 TB/s; with 8 for each SM 354 us).
constexpr int kNormBlocks = 6;

template <typename T, int N>
__global__ void __launch_bounds__(256, kNormBlocks) k_grad_norm(const __grid_constant__ NormArgs<N> a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t stride = gridDim.x * 8;
    // float16 squares and their sums neither vanish nor overflow
    constexpr bool kRange = !std::is_same<T, __half>::value;
    float acc = 0.0f, lost = 0.0f;
    uint32_t bits = 0;
    uint32_t first = 0, end = 0, shift = 0;
    const T *g = nullptr;
    uint64_t n = 0;
    for (uint32_t tile = blockIdx.x * 8 + warp + wait_prior_grid(); tile < a.tiles; tile += stride) {
        if (tile >= end) {
            const int t = find_tensor(a.tile_end, a.n_tensors, tile);
            first = t ? a.tile_end[t - 1] : 0;
            end = a.tile_end[t];
            shift = a.shift[t];
            g = (const T *)a.grad[t] - shift;  // a vector boundary; elements [shift, n) are the tensor's
            n = a.numel[t] + shift;
        }
        const uint64_t base = (uint64_t)(tile - first) * kNormTile;
        float s[8] = {};
        if (base >= shift && base + kNormTile <= n) {
            Raw8<T> r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = ld_grad8(g + base + i * kTile + 8 * lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v[8];
                unpack8(r[i], v);
                if (kRange) gather_bits(r[i], bits);
#pragma unroll
                for (int k = 0; k < 8; ++k) s[k] = fmaf(v[k], v[k], s[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t j = base + 128 * k + 32 * i + lane;
                    const float x = j >= shift && j < n ? to_f32(g[j]) : 0.0f;
                    if (kRange) bits |= __float_as_uint(x);
                    s[k] = fmaf(x, x, s[k]);
                }
        }
        // compensated: acc + s = now + lost
        const float add = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])) - lost;
        const float now = acc + add;
        lost = (now - acc) - add;
        acc = now;
    }
    __shared__ double part[8];
    __shared__ bool join;
    double sum = (double)acc - (double)lost;
    // Below 2^-100 what vanishes of up to 2^22 squares, 2^-150 of each, may count.
    const bool small = kRange && acc < 0x1p-100f && (bits & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu));
    if (small || !(acc <= 0x1.fffffep127f)) sum = rescaled_squares<T>(a, small);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += part[w];
        a.partials[a.first_partial + blockIdx.x] = sum;
        __threadfence();
        join = a.last && atomicInc(a.ticket, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!join) return;
    // the last block to finish adds every partial, in order
    __threadfence();
    sum = 0.0;
    for (uint32_t i = threadIdx.x; i < a.first_partial + gridDim.x; i += 256) sum += __ldcg(a.partials + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += part[w];
        const float norm = (float)sqrt(sum);
        float factor = 1.0f;
        if (a.max_norm > 0.0f) factor = fminf(1.0f, a.max_norm / (norm + 1e-6f));
        if (!isfinite(norm)) factor = __int_as_float(0x7FC00000);  // NaN: the step is refused
        a.out[0] = norm;
        a.out[1] = factor;
    }
}

uint32_t grad_norm_blocks(uint32_t tiles) {
    const uint32_t want = (tiles + 7) / 8, cap = (uint32_t)sm_count() * kNormBlocks;
    const uint32_t most = cap < (uint32_t)kNormPartials ? cap : (uint32_t)kNormPartials;
    return want < 1 ? 1 : want < most ? want : most;
}

template <int N>
cudaError_t launch_grad_norm(const NormArgs<N> &a, int dtype, uint32_t blocks, cudaStream_t s) {
    switch (dtype) {
    case GB_F32: return launch_pdl(k_grad_norm<float, N>, dim3(blocks), 256, 0, a, s);
    case GB_BF16: return launch_pdl(k_grad_norm<__nv_bfloat16, N>, dim3(blocks), 256, 0, a, s);
    default: return launch_pdl(k_grad_norm<__half, N>, dim3(blocks), 256, 0, a, s);
    }
}
template cudaError_t launch_grad_norm<kFewTensors>(const NormArgs<kFewTensors> &, int, uint32_t, cudaStream_t);
template cudaError_t launch_grad_norm<kNormTensors>(const NormArgs<kNormTensors> &, int, uint32_t, cudaStream_t);

// ------------------------------------------------------------------ AdamW
// 8-bit states.  m and v each lie in an E4M3 payload (codes, then one
// power-of-two scale per block), decoded at the start of the step and encoded
// at its end; p is computed from the float32 m and v.  The code of y =
// value / scale is floor(|y| / q + r), q the distance of E4M3's values around
// y and r a random number of 16 bits: rounded to nearest, a moving average
// that moves by less than half of q a step would stand still.  A second
// moment above zero (2^-129 at least) never gets code 0, which would divide by
// eps alone.
//
// Random numbers: z = mix32(key + q_lo * 0x9E3779B1 + q_hi * 0x85A308D3) for
// each group q of 8 elements, key of the seed, the step and the tensor; over
// the group's elements z runs through z = z * 2891336453 + 0x9E3779B9.  Its
// high half rounds m, its low half v.
__device__ __forceinline__ uint32_t group_random(uint32_t key, uint64_t q) {
    return mix32(key + (uint32_t)q * 0x9E3779B1u + (uint32_t)(q >> 32) * 0x85A308D3u);
}
__device__ __forceinline__ uint32_t next_random(uint32_t z) { return z * 2891336453u + 0x9E3779B9u; }
__device__ __forceinline__ uint32_t random_m(uint32_t z) { return (z >> 16) << 4; }
__device__ __forceinline__ uint32_t random_v(uint32_t z) { return (z & 0xFFFFu) << 4; }

// E4M3 codes by float32's bits.  x / scale times 2^-120 has E4M3's exponent
// field in float32's, E4M3's subnormals lie on float32's, and the code is the
// float's bits cut at bit 20.  Adding r20 = r / 2^16 * 2^20 before the cut
// carries into the code with the wanted probability.  e4m3_bits: the code in
// bits 20 .. 26, the sign in bit 31, what is cut off below.  1 / scale is
// multiplied first: the product of both factors would underflow.
__device__ __forceinline__ uint32_t e4m3_bits(float x, float inv, uint32_t r20) {
    return __float_as_uint(__fmul_rn(__fmul_rn(x, inv), 0x1p-120f)) + r20;
}
// ... of a second moment: at least code 1 where it is above zero.
__device__ __forceinline__ uint32_t above_zero(uint32_t bits, float x) {
    return max(bits, min(__float_as_uint(x), 1u << 20));
}
// One code, of any value: infinities and NaN are coded as NaN.
__device__ __forceinline__ unsigned char e4m3_code(float x, float inv, uint32_t r20, bool above) {
    const uint32_t sign = __float_as_uint(x) >> 24 & 0x80u;
    if (!isfinite(x)) return (unsigned char)(sign | 0x7Fu);
    const uint32_t c = e4m3_bits(x, inv, r20);
    return (unsigned char)(sign | ((above ? above_zero(c, x) : c) >> 20 & 0x7Fu));
}
// A block's largest finite magnitude sets its scale: what is coded as NaN
// must not push the other elements' scale up.
__device__ __forceinline__ float finite_mag(float x) { return isfinite(x) ? fabsf(x) : 0.0f; }

// The largest of magnitudes; a NaN among them stays.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_nan8(const float v[8]) {
    return max_nan(max_nan(max_nan(fabsf(v[0]), fabsf(v[1]), fabsf(v[2])), fabsf(v[3]), fabsf(v[4])),
                   max_nan(fabsf(v[5]), fabsf(v[6]), fabsf(v[7])));
}
// The largest of a codec block's lanes' magnitudes: the warp's, or its half's.
__device__ __forceinline__ float warp_max_nan(float m) {
    float r;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
    return r;
}
template <int B>
__device__ __forceinline__ float block_max_nan(float m, int lane) {
    if constexpr (B == 256) return warp_max_nan(m);
    const float lo = warp_max_nan(lane < 16 ? m : 0.0f), hi = warp_max_nan(lane < 16 ? 0.0f : m);
    return lane < 16 ? lo : hi;
}

// Square root and reciprocal to 2^-23 of the value, one instruction each;
// next to p's own rounding their error is nothing.  Subnormal v counts as
// zero; eps is at least 2^-63 (gb_adamw_step), the root of the least normal.
__device__ __forceinline__ float sqrt_fast(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int N>
__device__ __forceinline__ void adamw_update(const AdamwArgs<N> &a, float g, float &p, float &m, float &v) {
    m = __fadd_rn(__fmul_rn(m, a.beta1), __fmul_rn(g, a.gain1));
    v = __fadd_rn(__fmul_rn(v, a.beta2), __fmul_rn(__fmul_rn(g, g), a.gain2));
    const float u = m * rcp_fast(fmaf(sqrt_fast(v), a.unroot, a.eps));
    p = fmaf(-a.rate, u, p * a.keep);
}

// A warp's place in the table: tensor t's spans are [first, end).  The
// tensor's addresses are read from the kernel's parameters where they are
// used: kept in registers they would cost a third of the warps.
struct Place {
    int t;
    uint32_t first, end;
};
template <int N>
__device__ __forceinline__ void find_place(const AdamwArgs<N> &a, uint32_t span, Place &q) {
    if (span < q.end) return;
    q.t = find_tensor(a.span_end, a.n_tensors, span);
    q.first = q.t ? a.span_end[q.t - 1] : 0;
    q.end = a.span_end[q.t];
}
// Byte offset of the scale of element j's block in a payload of n elements.
template <int B>
__device__ __forceinline__ uint64_t scale_offset(uint64_t n, int64_t j) {
    return round_up(n, 16) + 4 * ((uint64_t)j / B);
}

// A tile element by element: the tensor's first and last tiles, and every
// tile of tensors whose arrays have no common vector boundary.  Lane l owns
// elements base + 32 k + l, k = 0 .. 7, so each access of the warp is one
// contiguous piece.
// Not inlined, so that its registers do not add to the vectors' path.
template <typename T, int B, bool COPY, int N>
__device__ __noinline__ void adamw_tile_elements(const AdamwArgs<N> &a, int t, int64_t base, float scale) {
    const int lane = threadIdx.x & 31;
    const uint64_t n = a.numel[t];
    float *const ps = a.param[t];
    const T *const gs = (const T *)a.grad[t];
    void *const mp = a.m[t], *const vp = a.v[t];
    float *const ms = (float *)((unsigned char *)mp + round_up(n, 16));
    float *const vs = (float *)((unsigned char *)vp + round_up(n, 16));
    float p[8], m[8], v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint64_t j = (uint64_t)(base + 32 * k + lane);  // before element 0: beyond n
        p[k] = m[k] = v[k] = 0.0f;
        if (j >= n) continue;
        p[k] = ps[j];
        if constexpr (B > 0) {
            float unused;
            fp8x2_to_f32<GB_CODEC_E4M3>(((const unsigned char *)mp)[j], m[k], unused);
            fp8x2_to_f32<GB_CODEC_E4M3>(((const unsigned char *)vp)[j], v[k], unused);
            m[k] *= ms[j / B];
            v[k] *= vs[j / B];
        } else {
            m[k] = ((const float *)mp)[j];
            v[k] = ((const float *)vp)[j];
        }
        const float g = __fmul_rn(to_f32(gs[j]), scale);
        adamw_update(a, g, p[k], m[k], v[k]);
    }
    float minv[2] = {}, vinv[2] = {};
    if constexpr (B > 0) {
#pragma unroll
        for (int b = 0; b < 256 / B; ++b) {
            float mm = 0.0f, vm = 0.0f;
#pragma unroll
            for (int k = 0; k < B / 32; ++k) {
                mm = fmaxf(mm, finite_mag(m[b * 4 + k]));
                vm = fmaxf(vm, finite_mag(v[b * 4 + k]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
                vm = fmaxf(vm, __shfl_xor_sync(0xFFFFFFFFu, vm, o));
            }
            const int mk = block_scale_exp<GB_CODEC_E4M3>(mm), vk = block_scale_exp<GB_CODEC_E4M3>(vm);
            minv[b] = pow2f(-mk);
            vinv[b] = pow2f(-vk);
            if (lane == 0 && (uint64_t)base + b * B < n) {
                ms[base / B + b] = pow2f(mk);
                vs[base / B + b] = pow2f(vk);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint64_t j = (uint64_t)(base + 32 * k + lane);
        if (j >= n) continue;
        ps[j] = p[k];
        if constexpr (COPY) ((T *)a.copy[t])[j] = from_f32<T>(p[k]);
        if constexpr (B > 0) {
            const int b = B == 128 ? k >> 2 : 0;
            uint32_t z = group_random(a.key[t], j >> 3);
            for (int i = 0; i < (lane & 7); ++i) z = next_random(z);
            ((unsigned char *)mp)[j] = e4m3_code(m[k], minv[b], random_m(z), false);
            ((unsigned char *)vp)[j] = e4m3_code(v[k], vinv[b], random_v(z), true);
        } else {
            ((float *)mp)[j] = m[k];
            ((float *)vp)[j] = v[k];
        }
    }
}

// What a lane has of a whole tile: elements 8 lane .. 8 lane + 7.
template <bool EIGHT> struct StateLoads {  // float32 states
    U8x32 m, v;
};
template <> struct StateLoads<true> {  // codes
    uint2 m, v;
};
template <typename T, int B> struct TileLoads : StateLoads<(B > 0)> {
    U8x32 p;
    Raw8<T> g;
};

template <typename T, int N>
__device__ __forceinline__ TileLoads<T, 0> adamw_load(const AdamwArgs<N> &a, int t, int64_t j) {
    return {{ld_rw_v8((const float *)a.m[t] + j), ld_rw_v8((const float *)a.v[t] + j)}, ld_rw_v8(a.param[t] + j),
            ld_grad8((const T *)a.grad[t] + j)};
}

// Eight values of a state from their E4M3 codes.
__device__ __forceinline__ void decode8(uint2 c, float scale, float v[8]) {
    fp8x2_to_f32<GB_CODEC_E4M3>(c.x & 0xFFFFu, v[0], v[1]);
    fp8x2_to_f32<GB_CODEC_E4M3>(c.x >> 16, v[2], v[3]);
    fp8x2_to_f32<GB_CODEC_E4M3>(c.y & 0xFFFFu, v[4], v[5]);
    fp8x2_to_f32<GB_CODEC_E4M3>(c.y >> 16, v[6], v[7]);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __fmul_rn(v[k], scale);
}
// Four codes of e4m3_bits' form to the bytes of one word, without signs and
// with them.
__device__ __forceinline__ uint32_t gather4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t lo = __byte_perm(a, b, 0x7632) >> 4, hi = __byte_perm(c, d, 0x7632) >> 4;
    return __byte_perm(lo, hi, 0x6420);
}
__device__ __forceinline__ uint32_t gather2_signed(uint32_t a, uint32_t b) {  // to bytes 0 and 2
    const uint32_t u = __byte_perm(a, b, 0x7632);
    return (u >> 4 & 0x007F007Fu) | (u >> 8 & ~0x007F007Fu);
}
__device__ __forceinline__ uint32_t gather4_signed(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(gather2_signed(a, b), gather2_signed(c, d), 0x6420);
}

// One lane's elements of a whole tile: p and its copy are written, m and v
// (8-bit states: given decoded) left in registers.
template <typename T, int B, bool COPY, int N>
__device__ __forceinline__ void adamw_vectors(const AdamwArgs<N> &a, float *to, T *copy, float scale, const TileLoads<T, B> &r,
                                              float m[8], float v[8]) {
    float p[8], g[8];
    unpack8(r.g, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        p[k] = __uint_as_float(r.p.w[k]);
        if constexpr (B == 0) {
            m[k] = __uint_as_float(r.m.w[k]);
            v[k] = __uint_as_float(r.v.w[k]);
        }
        adamw_update(a, __fmul_rn(g[k], scale), p[k], m[k], v[k]);
    }
    st8(to, p);
    if constexpr (COPY) st8(copy, p);
}

// The codes of a lane's m and v, and its block's scales; z is the group's
// random number.
template <int B>
__device__ __forceinline__ void encode_states(uint32_t z, int lane, const float m[8], const float v[8], uint2 &mc,
                                              uint2 &vc, float &mscale, float &vscale) {
    float mm = block_max_nan<B>(max_nan8(m), lane), vm = block_max_nan<B>(max_nan8(v), lane);
    const bool odd = __any_sync(0xFFFFFFFFu, !isfinite(mm) || !isfinite(vm));
    if (odd) {  // the largest finite ones instead
        mm = vm = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            mm = fmaxf(mm, finite_mag(m[k]));
            vm = fmaxf(vm, finite_mag(v[k]));
        }
        mm = block_max_nan<B>(mm, lane);
        vm = block_max_nan<B>(vm, lane);
    }
    const int mk = block_scale_exp<GB_CODEC_E4M3>(mm), vk = block_scale_exp<GB_CODEC_E4M3>(vm);
    const float minv = pow2f(-mk), vinv = pow2f(-vk);
    mscale = pow2f(mk);
    vscale = pow2f(vk);
    if (odd) {
        unsigned char cm[8], cv[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            cm[k] = e4m3_code(m[k], minv, random_m(z), false);
            cv[k] = e4m3_code(v[k], vinv, random_v(z), true);
            z = next_random(z);
        }
        mc = make_uint2(cm[0] | cm[1] << 8 | cm[2] << 16 | (uint32_t)cm[3] << 24,
                        cm[4] | cm[5] << 8 | cm[6] << 16 | (uint32_t)cm[7] << 24);
        vc = make_uint2(cv[0] | cv[1] << 8 | cv[2] << 16 | (uint32_t)cv[3] << 24,
                        cv[4] | cv[5] << 8 | cv[6] << 16 | (uint32_t)cv[7] << 24);
    } else {
        uint32_t cm[8], cv[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            cm[k] = e4m3_bits(m[k], minv, random_m(z));
            cv[k] = above_zero(e4m3_bits(v[k], vinv, random_v(z)), v[k]);
            z = next_random(z);
        }
        mc = make_uint2(gather4_signed(cm[0], cm[1], cm[2], cm[3]), gather4_signed(cm[4], cm[5], cm[6], cm[7]));
        vc = make_uint2(gather4(cv[0], cv[1], cv[2], cv[3]), gather4(cv[4], cv[5], cv[6], cv[7]));
    }
}

// 8-bit states of tensors that do not start on vectors (packed into a flat
// buffer without gaps): codes lie on vectors of the tensor, p, g and the copy
// `shift` elements beside their own.  A lane reads the vector at or before its
// elements and takes the rest from the next lane (64 Mi elements, bf16 with
// copies: 283 us against 585 element by element and 173 on vectors).  What it
// reads of the tiles beside its own, which other warps may be writing, is not
// used.
__device__ __forceinline__ uint32_t shift_of(const void *p, uint32_t eb) { return (uint32_t)((uintptr_t)p / eb) & 7u; }

// Elements base + 8 lane .. of a tensor; elements base - 7 .. base + 263 are
// all the tensor's.
template <typename T>
__device__ __forceinline__ void load_shifted(const T *tensor, int64_t base, int lane, float out[8]) {
    const uint32_t shift = shift_of(tensor, sizeof(T));
    const T *const p = tensor + base - shift + 8 * lane;
    constexpr int kWords = 2 * sizeof(T);
    auto load = [](const T *q) {
        Raw8<T> r;
        if constexpr (sizeof(T) == 4) r.w = ld_rw_v8(q);
        else r.w = ld_rw_u4(q);
        return r;
    };
    const Raw8<T> own = load(p);
    Raw8<T> next = own;
    if (lane == 31) next = load(p + 8);
    float a[16];
    unpack8(own, a);
    const uint32_t *const o = (const uint32_t *)&own;
    uint32_t *const n = (uint32_t *)&next;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const uint32_t w = __shfl_down_sync(0xFFFFFFFFu, o[i], 1);
        if (lane != 31) n[i] = w;
    }
    unpack8(next, a + 8);
#pragma unroll
    for (int step = 4; step > 0; step >>= 1)
#pragma unroll
        for (int k = 0; k < 8 + step; ++k)
            if (k + step < 16) a[k] = shift & step ? a[k + step] : a[k];
#pragma unroll
    for (int k = 0; k < 8; ++k) out[k] = a[k];
}
// ... and back: lane 0 and lane 31 write the tile's two cut vectors by element.
template <typename T>
__device__ __forceinline__ void store_shifted(T *tensor, int64_t base, int lane, const float v[8]) {
    const uint32_t shift = shift_of(tensor, sizeof(T));
    float a[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        a[k] = __shfl_up_sync(0xFFFFFFFFu, v[k], 1);
        a[8 + k] = v[k];
    }
#pragma unroll
    for (int step = 4; step > 0; step >>= 1)
#pragma unroll
        for (int k = 15; k >= 8 - (step - 1); --k)
            if (k >= step) a[k] = shift & step ? a[k - step] : a[k];
    T *const p = tensor + base - shift + 8 * lane;
    if (lane > 0 || shift == 0) st8(p, a + 8);
    if (shift == 0) return;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k + shift < 8) tensor[base + k] = from_f32<T>(v[k]);
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k + shift >= 8) tensor[base + 8 * 31 + k] = from_f32<T>(v[k]);
}

// Float32 states: one warp per tile of 256 elements, and a grid of as many
// warps, so that finished blocks are replaced (64 Mi elements, 28 bytes each
// with a bf16 gradient and copy: 273 us, 6.9 TB/s; in 4 blocks an SM that loop
// 304 us).
template <typename T, bool COPY, int N>
__global__ void __launch_bounds__(256) k_adamw(const __grid_constant__ AdamwArgs<N> a) {
    const int lane = threadIdx.x & 31;
    const uint32_t stride = gridDim.x * 8, zero = wait_prior_grid();
    uint32_t tile = blockIdx.x * 8 + (threadIdx.x >> 5) + zero;
    const float scale = a.grad_scale ? a.grad_scale[zero] : 1.0f;  // the kernel before this one may write it
    if (!isfinite(scale)) return;  // the step is refused: nothing changes
    Place q;
    q.end = 0;
    for (; tile < a.spans; tile += stride) {
        find_place(a, tile, q);
        const uint32_t layout = a.layout[q.t];
        const int64_t base = (int64_t)(tile - q.first) * kTile - (layout & 7u), j = base + 8 * lane;
        if (layout == kScattered || base < 0 || (uint64_t)base + kTile > a.numel[q.t]) {
            adamw_tile_elements<T, 0, COPY>(a, q.t, base, scale);
            continue;
        }
        float m[8], v[8];
        adamw_vectors<T, 0, COPY>(a, a.param[q.t] + j, COPY ? (T *)a.copy[q.t] + j : nullptr, scale, adamw_load<T>(a, q.t, j), m, v);
        st8((float *)a.m[q.t] + j, m);
        st8((float *)a.v[q.t] + j, v);
    }
}

// 8-bit states in blocks of B.  A block takes a span of 8 or 32 tiles of one
// tensor, 8 neighbours at a time, one a warp.  The span's scales pass through
// shared memory, so that they are read and written as whole sectors: written
// by each warp, 4 bytes at a time, they cost more than all the arithmetic
// (64 Mi elements, 12 bytes of bf16 gradient, copy and parameter: 195 us,
// and 169 us without those stores).  Now 176 us, 6.1 TB/s of 6.7 copied.
// What does not help: more loads ahead of a warp, in registers (207 .. 217
// us) or by asynchronous copies into shared memory (212 .. 218 us) -- both
// take warps away.
constexpr uint32_t kSpanTiles = 32;

// SHIFTED: some tensor of the launch starts off its vectors (in a kernel of
// its own: the code costs the others registers, and with them a block an SM).
// 64 tensors of 1 Mi elements, bf16 with copies: 172 us; one of them off its
// vectors 193 us, half of them 234 us, all 284 us.
template <typename T, int B, bool COPY, bool SHIFTED, int N>
__global__ void __launch_bounds__(256, SHIFTED ? 3 : 4) k_adamw8(const __grid_constant__ AdamwArgs<N> a) {
    constexpr int kPer = kTile / B;  // scales of a tile
    __shared__ float ms[kSpanTiles * kPer], vs[kSpanTiles * kPer];
    const uint32_t zero = wait_prior_grid(), lane = (threadIdx.x & 31) + zero;
    const int warp = threadIdx.x >> 5;
    const float scale = a.grad_scale ? a.grad_scale[zero] : 1.0f;
    if (!isfinite(scale)) return;  // the step is refused: nothing changes
    Place q;
    q.end = 0;
    for (uint32_t span = blockIdx.x; span < a.spans; span += gridDim.x) {
        find_place(a, span, q);
        const int t = q.t;
        const uint64_t n = a.numel[t], base = (uint64_t)(span - q.first) * a.span * kTile, rest = n - base;
        const uint32_t mine = rest < a.span * kTile ? (uint32_t)rest : a.span * kTile;  // elements of the span
        const int tiles = (int)((mine + kTile - 1) / kTile);
        // tiles [lo, hi) go in vectors, the rest element by element; a shifted tile's vectors reach beyond it
        const bool shifted = SHIFTED && a.layout[t] == kScattered;
        const int lo = shifted && base == 0 ? 1 : 0;
        const int hi = !shifted ? (int)(mine / kTile) : rest >= mine + 8ull ? tiles : rest >= kTile + 8 ? (int)((rest - 8) / kTile) : 0;
        unsigned char *const mc = (unsigned char *)a.m[t] + base, *const vc = (unsigned char *)a.v[t] + base;
        float *const mscale = (float *)((unsigned char *)a.m[t] + round_up(n, 16)) + base / B + zero;
        float *const vscale = (float *)((unsigned char *)a.v[t] + round_up(n, 16)) + base / B + zero;
        const bool mover = (int)threadIdx.x >= kPer * lo && (int)threadIdx.x < kPer * hi;
        if (mover) {
            ms[threadIdx.x] = mscale[threadIdx.x];
            vs[threadIdx.x] = vscale[threadIdx.x];
        }
        __syncthreads();
#pragma unroll 1
        for (int i = warp; i < hi; i += 8) {
            if (i < lo) continue;
            const uint32_t j = i * kTile + 8 * lane, at = j / B;
            float m[8], v[8];
            if (shifted) {
                float p[8], g[8];
                const int64_t tile = (int64_t)(base + i * kTile);
                decode8(ld_rw_u2(mc + j), ms[at], m);
                decode8(ld_rw_u2(vc + j), vs[at], v);
                load_shifted((const T *)a.grad[t], tile, lane, g);
                load_shifted((const float *)a.param[t], tile, lane, p);
#pragma unroll
                for (int k = 0; k < 8; ++k) adamw_update(a, __fmul_rn(g[k], scale), p[k], m[k], v[k]);
                store_shifted(a.param[t], tile, lane, p);
                if constexpr (COPY) store_shifted((T *)a.copy[t], tile, lane, p);
            } else {
                const TileLoads<T, B> r = {{ld_rw_u2(mc + j), ld_rw_u2(vc + j)}, ld_rw_v8(a.param[t] + base + j), ld_grad8((const T *)a.grad[t] + base + j)};
                decode8(r.m, ms[at], m);
                decode8(r.v, vs[at], v);
                adamw_vectors<T, B, COPY>(a, a.param[t] + base + j, COPY ? (T *)a.copy[t] + base + j : nullptr, scale, r, m, v);
            }
            float new_ms, new_vs;
            uint2 new_m, new_v;
            encode_states<B>(group_random(a.key[t], (base + j) >> 3), lane, m, v, new_m, new_v, new_ms, new_vs);
            st_u2(mc + j, new_m);
            st_u2(vc + j, new_v);
            if ((lane & (B / 8 - 1)) == 0) {  // the old ones have been read: the warp has met in encode_states
                ms[at] = new_ms;
                vs[at] = new_vs;
            }
        }
        for (int i = warp; i < tiles; i += 8)
            if (i < lo || i >= hi) adamw_tile_elements<T, B, COPY>(a, t, (int64_t)(base + i * kTile), scale);
        __syncthreads();
        if (mover) {
            mscale[threadIdx.x] = ms[threadIdx.x];
            vscale[threadIdx.x] = vs[threadIdx.x];
        }
        // a thread's own slots are the next span's: no other barrier is needed
    }
}

template <typename T, int B, bool COPY, int N>
static cudaError_t adamw8(const AdamwArgs<N> &a, dim3 grid, cudaStream_t s) {
    for (int t = 0; t < a.n_tensors; ++t)
        if (a.layout[t] == kScattered) return launch_pdl(k_adamw8<T, B, COPY, true, N>, grid, 256, 0, a, s);
    return launch_pdl(k_adamw8<T, B, COPY, false, N>, grid, 256, 0, a, s);
}

template <typename T, bool COPY, int N>
static cudaError_t adamw_states(const AdamwArgs<N> &a, int state_block, cudaStream_t s) {
    const uint32_t want = state_block ? a.spans : (a.spans + 7) / 8, cap = (uint32_t)sm_count() * 256;
    const dim3 grid(want < cap ? want : cap);
    switch (state_block) {
    case 0: return launch_pdl(k_adamw<T, COPY, N>, grid, 256, 0, a, s);
    case 128: return adamw8<T, 128, COPY>(a, grid, s);
    default: return adamw8<T, 256, COPY>(a, grid, s);
    }
}

template <typename T, int N>
static cudaError_t adamw_copies(const AdamwArgs<N> &a, int state_block, bool copies, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (copies) return adamw_states<T, true>(a, state_block, s);
    return adamw_states<T, false>(a, state_block, s);
}

template <int N>
cudaError_t launch_adamw(const AdamwArgs<N> &a, int dtype, int state_block, bool copies, cudaStream_t s) {
    switch (dtype) {
    case GB_F32: return adamw_copies<float>(a, state_block, copies, s);
    case GB_BF16: return adamw_copies<__nv_bfloat16>(a, state_block, copies, s);
    default: return adamw_copies<__half>(a, state_block, copies, s);
    }
}
template cudaError_t launch_adamw<kFewTensors>(const AdamwArgs<kFewTensors> &, int, int, bool, cudaStream_t);
template cudaError_t launch_adamw<kAdamwTensors>(const AdamwArgs<kAdamwTensors> &, int, int, bool, cudaStream_t);

}  // namespace gb
