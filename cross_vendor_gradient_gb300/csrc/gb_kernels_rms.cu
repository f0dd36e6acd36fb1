// RMS norm with the residual's addition, and its gradient (sm_103a).
//
// Forward, per row of `cols` elements:
//   h = round(x + residual);  rstd = 1 / sqrt(sum h^2 / cols + eps)
//   y = (h w) rstd, rounded to the rows' type, or encoded to OCP fp8 with one
//   power-of-two scale per block of 128 / 256 elements of the row (the block
//   rule of the bridge codec; the blocks start at the row's first element).
//   In 16-bit types h w is exact in float32, so y is rounded once before that.
// Backward, from dy, the h of the forward pass and rstd:
//   xhat = h rstd;  a = dy w;  c = sum(a xhat) / cols
//   dx = rstd (a - xhat c) + dsum;  dweight = sum over the rows of dy xhat
// All of it in float32.  Both are streaming work, one pass over the data: a
// row stays in the registers of a team of threads between its sum and its
// output.
#include <atomic>

#include "gb_rows.cuh"
#include "gb_train.cuh"

namespace gb {

// ------------------------------------------------------------------- rows
// The own part of vector v.
template <int V> __device__ __forceinline__ int own_lo(const Mine<V> &m, int v) { return m.head >> v & 1 ? m.lo : 0; }
template <int V> __device__ __forceinline__ int own_hi(const Mine<V> &m, int v) { return m.tail >> v & 1 ? m.hi : 8; }

// Predicated vector accesses: a row's threads take them without branching.
__device__ __forceinline__ uint4 ld_if_u4(const void *p, bool yes) {
    uint4 r;
    asm volatile("{.reg .pred q; setp.ne.b32 q, %5, 0; mov.b32 %0, 0; mov.b32 %1, 0; mov.b32 %2, 0; mov.b32 %3, 0;"
                 " @q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];}"
                 : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w) : "l"(p), "r"((int)yes) : "memory");
    return r;
}
__device__ __forceinline__ U8x32 ld_if_v8(const void *p, bool yes) {
    U8x32 r;
    asm volatile("{.reg .pred q; setp.ne.b32 q, %9, 0; mov.b32 %0, 0; mov.b32 %1, 0; mov.b32 %2, 0; mov.b32 %3, 0;"
                 " mov.b32 %4, 0; mov.b32 %5, 0; mov.b32 %6, 0; mov.b32 %7, 0;"
                 " @q ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];}"
                 : "=&r"(r.w[0]), "=&r"(r.w[1]), "=&r"(r.w[2]), "=&r"(r.w[3]), "=&r"(r.w[4]), "=&r"(r.w[5]),
                   "=&r"(r.w[6]), "=&r"(r.w[7])
                 : "l"(p), "r"((int)yes) : "memory");
    return r;
}
__device__ __forceinline__ void st_if_u4(void *p, uint4 v, bool yes) {
    asm volatile("{.reg .pred q; setp.ne.b32 q, %5, 0; @q st.global.v4.u32 [%0], {%1, %2, %3, %4};}" ::"l"(p), "r"(v.x),
                 "r"(v.y), "r"(v.z), "r"(v.w), "r"((int)yes) : "memory");
}
// WIDE: float32 rows in 32-byte accesses (every buffer starts on 32 bytes),
// else two of 16.
template <typename T, bool WIDE>
__device__ __forceinline__ Raw8<T> load_vector(const T *p, bool yes) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 2) {
        r.w = ld_if_u4(p, yes);
    } else if constexpr (WIDE) {
        r.w = ld_if_v8(p, yes);
    } else {
        const uint4 a = ld_if_u4(p, yes), b = ld_if_u4(p + 4, yes);
        r.w = U8x32{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
    return r;
}
template <typename T, bool WIDE>
__device__ __forceinline__ void store_vector(T *p, const Raw8<T> &r, bool yes) {
    if constexpr (sizeof(T) == 2) {
        st_if_u4(p, r.w, yes);
    } else if constexpr (WIDE) {
        if (yes) st_v8(p, r.w.w);
    } else {
        st_if_u4(p, make_uint4(r.w.w[0], r.w.w[1], r.w.w[2], r.w.w[3]), yes);
        st_if_u4(p + 4, make_uint4(r.w.w[4], r.w.w[5], r.w.w[6], r.w.w[7]), yes);
    }
}
template <typename T>
__device__ __forceinline__ Raw8<T> pack8(const float v[8]) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k) r.w.w[k] = __float_as_uint(v[k]);
    } else {
        r.w = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
    }
    return r;
}
// Elements outside [lo, hi) become zero.
template <typename T>
__device__ __forceinline__ void keep_own(Raw8<T> &r, int lo, int hi) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k) r.w.w[k] = k >= lo && k < hi ? r.w.w[k] : 0u;
    } else {
        uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (!(2 * k >= lo && 2 * k < hi)) w[k] &= 0xFFFF0000u;
            if (!(2 * k + 1 >= lo && 2 * k + 1 < hi)) w[k] &= 0x0000FFFFu;
        }
        r.w = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
// A thread's vectors of a row, the row's boundary at element `at`.  With a
// skew the end vectors are read whole, with elements of the rows beside this
// one (which another team may be overwriting in place; they are not used);
// in a row that is `cut` the last vector reaches beyond the tensor's end, and
// goes element by element.
template <typename T, int V, bool WIDE, bool SKEW>
__device__ __forceinline__ void load_row(Raw8<T> x[V], const T *tensor, uint64_t at, const Mine<V> &m, int i, int team, bool row,
                                         bool cut) {
    const T *const p = tensor + at + 8 * i;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const uint32_t whole = whole_vectors<V>(m, SKEW && cut);
        x[v] = load_vector<T, WIDE>(p + 8 * v * team, row && (whole >> v & 1));
    }
    if constexpr (SKEW) {
        if (!cut || !m.tail) return;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (m.tail >> v & 1) {
                float f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = k < m.hi ? to_f32(p[8 * v * team + k]) : 0.0f;
                x[v] = pack8<T>(f);
            }
    }
}
// What load_row read from the rows beside this one becomes zero.
template <typename T, int V>
__device__ __forceinline__ void cut_row(Raw8<T> x[V], const Mine<V> &m) {
    if (!(m.head | m.tail)) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if ((m.head | m.tail) >> v & 1) keep_own<T>(x[v], own_lo(m, v), own_hi(m, v));
}
template <typename T, int V, bool WIDE, bool SKEW>
__device__ __forceinline__ void store_row(T *tensor, uint64_t at, const Mine<V> &m, int i, int team, bool row, const Raw8<T> x[V]) {
    T *const p = tensor + at + 8 * i;
    const uint32_t cut = m.head | m.tail;
#pragma unroll
    for (int v = 0; v < V; ++v) store_vector<T, WIDE>(p + 8 * v * team, x[v], row && ((m.has & ~cut) >> v & 1));
    if constexpr (SKEW) {
        if (!cut || !row) return;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!(cut >> v & 1)) continue;
            const int lo = own_lo(m, v), hi = own_hi(m, v);
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k >= lo && k < hi) p[8 * v * team + k] = __uint_as_float(x[v].w.w[k]);
            } else {
                const uint32_t w[4] = {x[v].w.x, x[v].w.y, x[v].w.z, x[v].w.w};
                unsigned short *q = (unsigned short *)p + 8 * v * team;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k >= lo && k < hi) q[k] = (unsigned short)(k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xFFFFu);
            }
        }
    }
}
// The thread's weights: column p - skew + k.  They may lie at any element (a
// parameter in a packed bucket): once a kernel, so no matter.
template <typename T, int V, bool WIDE, bool SKEW>
__device__ __forceinline__ void load_weights(Raw8<T> w[V], const T *weight, const Mine<V> &m, int i, int team, uint32_t cols) {
    if (!SKEW && ((uintptr_t)weight & (WIDE ? 31u : 15u)) == 0) {
        load_row<T, V, WIDE, false>(w, weight, 0, m, i, team, true, false);
        return;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = 8 * (i + v * team) + k - m.skew;
            f[k] = c >= 0 && c < (int)cols ? to_f32(weight[c]) : 0.0f;
        }
        w[v] = pack8<T>(f);
    }
}

// Eight elements, two to an instruction (rounded as single ones).
__device__ __forceinline__ void fma2(float &x, float &y, float ax, float ay, float bx, float by) {
    asm("{.reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%0, %1}; fma.rn.f32x2 c, a, b, c;"
        " mov.b64 {%0, %1}, c;}" : "+f"(x), "+f"(y) : "f"(ax), "f"(ay), "f"(bx), "f"(by));
}
__device__ __forceinline__ void mul2(float &x, float &y, float ax, float ay) {
    asm("{.reg .b64 a, c; mov.b64 a, {%2, %3}; mov.b64 c, {%0, %1}; mul.rn.f32x2 c, a, c; mov.b64 {%0, %1}, c;}"
        : "+f"(x), "+f"(y) : "f"(ax), "f"(ay));
}
__device__ __forceinline__ void add2(float &x, float &y, float ax, float ay) {
    asm("{.reg .b64 a, c; mov.b64 a, {%2, %3}; mov.b64 c, {%0, %1}; add.rn.f32x2 c, a, c; mov.b64 {%0, %1}, c;}"
        : "+f"(x), "+f"(y) : "f"(ax), "f"(ay));
}
__device__ __forceinline__ void fma8(float x[8], const float a[8], const float b[8]) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) fma2(x[k], x[k + 1], a[k], a[k + 1], b[k], b[k + 1]);
}
__device__ __forceinline__ void mul8(float x[8], const float a[8]) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) mul2(x[k], x[k + 1], a[k], a[k + 1]);
}
__device__ __forceinline__ void scale8(float x[8], float a) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) mul2(x[k], x[k + 1], a, a);
}
__device__ __forceinline__ void add8(float x[8], const float a[8]) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) add2(x[k], x[k + 1], a[k], a[k + 1]);
}
__device__ __forceinline__ float tree8(const float s[8]) {
    return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}
// The sum over the team, in each of its threads.  part: 32 floats a team; two
// sets of them used in turn make one barrier a row enough.  A team of several
// warps has a barrier of its own (number 1 + its place in the block).
__device__ __forceinline__ float team_sum(float v, int team, float part[32], int place) {
    for (int o = min(team, 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (team <= 32) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[(threadIdx.x - place * team) >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + place), "r"(team) : "memory");
    v = lane < team >> 5 ? part[lane] : 0.0f;
#pragma unroll
    for (int o = kMaxTeam / 64; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return __shfl_sync(0xFFFFFFFFu, v, 0);
}
static_assert(kMaxTeam == 512, "team_sum joins 16 warps");

template <int CODEC>
__device__ __forceinline__ uint2 encode8(const float y[8]) {
    return make_uint2(cvt_fp8x2<CODEC>(y[0], y[1]) | cvt_fp8x2<CODEC>(y[2], y[3]) << 16,
                      cvt_fp8x2<CODEC>(y[4], y[5]) | cvt_fp8x2<CODEC>(y[6], y[7]) << 16);
}

// CODEC: GB_CODEC_NONE, or the 8-bit output's format in blocks of B elements
// of the row.  SKEW: cols is no multiple of 8.  The weights stay in
// registers, and the next row is loaded before this one is summed (where
// there are registers for it).
//
// 8-bit blocks.  A group of B / 8 vectors starts at every B-th position; it
// holds the block but for the block's last `skew` elements, which are the
// first ones of the next group's first vector.  Rounding keeps order, so a
// block's largest |y| is rstd times its largest |h w|, known before rstd:
// groups leave the largest of their own part and of the part before in shared
// memory, and the row's one barrier serves both.
template <typename T, int CODEC, int B, int V, bool WIDE, bool SKEW>
__global__ void __launch_bounds__(kMaxTeam) k_rms_norm(const __grid_constant__ RmsArgs a) {
    constexpr bool kEight = CODEC != GB_CODEC_NONE;
    constexpr bool kAhead = V * sizeof(T) <= 8;  // a row ahead where the registers hold it
    constexpr int kGroup = B / 8;
    constexpr int kGroups = kEight && SKEW ? V * kMaxTeam / kGroup + 1 : 1;
    __shared__ float part[2][32];
    __shared__ float own_max[2][kGroups], before_max[2][kGroups];
    const int team = a.team, i = team > 32 ? threadIdx.x : threadIdx.x & (team - 1);
    const uint64_t per = blockDim.x / team, stride = gridDim.x * per;
    uint64_t row = blockIdx.x * per + threadIdx.x / team + wait_prior_grid();
    const Mine<V> m = mine_of<V>(row, a.cols, i, team);
    uint64_t at = row * a.cols - m.skew;
    if constexpr (kEight && SKEW) {
        if (team >= 32) {
            for (int g = threadIdx.x; g < 2 * kGroups; g += blockDim.x) (&before_max[0][0])[g] = (&own_max[0][0])[g] = 0.0f;
            __syncthreads();
        }
    }
    Raw8<T> w[V], x[V], res[V];
    load_weights<T, V, WIDE, SKEW>(w, (const T *)a.weight, m, i, team, a.cols);
    auto load = [&]() {
        const bool valid = row < a.rows, cut = row - a.whole_rows < a.rows - a.whole_rows;  // whole_rows <= row < rows
        load_row<T, V, WIDE, SKEW>(x, (const T *)a.x, at, m, i, team, valid, cut);
        if (a.residual) load_row<T, V, WIDE, SKEW>(res, (const T *)a.residual, at, m, i, team, valid, cut);
    };
    if (kAhead) load();
    int parity = 0;
    // a warp's teams go on together
    for (uint64_t base = row - (team < 32 ? (threadIdx.x & 31) / team : 0); base < a.rows; base += stride, parity ^= 1) {
        if (!kAhead) load();
        const uint64_t this_row = row, this_at = at;
        const bool valid = row < a.rows;
        Raw8<T> h[V];
        float ss[8] = {}, lane_max = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = x[v];
            if (a.residual) {
                float f[8], y[8];
                unpack8(h[v], f);
                unpack8(res[v], y);
                add8(f, y);
                h[v] = pack8<T>(f);
            }
        }
        if (a.sum) store_row<T, V, WIDE, SKEW>((T *)a.sum, this_at, m, i, team, valid, h);
        if constexpr (SKEW) cut_row<T, V>(h, m);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f[8];
            unpack8(h[v], f);
            fma8(ss, f, f);
            if constexpr (kEight && SKEW) {
                float g[8];
                unpack8(w[v], g);
                mul8(f, g);
                const int vec = i + v * team;
                const bool leads = vec % kGroup == 0;
                float front = 0.0f, rest = 0.0f;  // the skew is the team's: a uniform choice
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (k < m.skew) front = fmaxf(front, fabsf(f[k]));
                    else rest = fmaxf(rest, fabsf(f[k]));
                }
                float own = leads ? rest : fmaxf(front, rest);
                const float before = leads ? front : 0.0f;
                for (int o = min(team, kGroup) / 2; o > 0; o >>= 1) own = fmaxf(own, __shfl_xor_sync(0xFFFFFFFFu, own, o));
                if (team >= 32) {
                    if (leads) {
                        own_max[parity][vec / kGroup] = own;
                        before_max[parity][vec / kGroup] = before;
                    }
                } else {  // such a row lies in one group
                    lane_max = own;
                }
            }
        }
        row += stride;
        at += stride * a.cols;
        if (kAhead) load();
        const float sum = team_sum(tree8(ss), team, part[parity], 0);
        if constexpr (kEight && SKEW)
            if (team == 32) __syncwarp();
        const float rstd = 1.0f / sqrtf(fmaf(sum, a.inv_cols, a.eps));
        if (i == 0 && a.rstd && valid) a.rstd[this_row] = rstd;
        const uint32_t blocks = (a.cols + B - 1) / B;
        float *const scales = (float *)((unsigned char *)a.out + a.scales_off) + this_row * blocks;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int vec = i + v * team;
            float y[8], g[8];
            unpack8(h[v], y);
            unpack8(w[v], g);
            mul8(y, g);
            scale8(y, rstd);
            if constexpr (!kEight) {
                h[v] = pack8<T>(y);
            } else {
                unsigned char *const codes = (unsigned char *)a.out + this_at + 8 * vec;
                const bool mine = valid && (m.has >> v & 1);
                if constexpr (!SKEW) {
                    float top = 0.0f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(y[k]));
                    for (int o = min(team, kGroup) / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    const int kexp = block_scale_exp<CODEC>(top);
                    scale8(y, pow2f(-kexp));
                    const uint2 c = encode8<CODEC>(y);
                    if (mine) {
                        st_u2(codes, c);
                        if (vec % kGroup == 0) scales[vec / kGroup] = pow2f(kexp);
                    }
                } else {
                    const int group = vec / kGroup;
                    float top = lane_max, last = 0.0f;
                    if (team >= 32) {
                        top = fmaxf(own_max[parity][group], before_max[parity][group + 1]);
                        last = group ? fmaxf(own_max[parity][group - 1], before_max[parity][group]) : 0.0f;
                    }
                    // a NaN, of 0 times infinity or of the row's, counts as no magnitude, as in the maxima
                    const int kexp = block_scale_exp<CODEC>(fmaxf(top * rstd, 0.0f));
                    const int klast = block_scale_exp<CODEC>(fmaxf(last * rstd, 0.0f));
                    const float inv = pow2f(-kexp), inv_front = vec % kGroup == 0 ? pow2f(-klast) : inv;
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] *= k < m.skew ? inv_front : inv;
                    const uint2 c = encode8<CODEC>(y);
                    if (mine) {
                        const int lo = own_lo(m, v), hi = own_hi(m, v);
                        if (lo == 0 && hi == 8) {
                            st_u2(codes, c);
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (k >= lo && k < hi) codes[k] = (unsigned char)((k < 4 ? c.x : c.y) >> 8 * (k & 3));
                        }
                        if (vec % kGroup == 0 && group < (int)blocks) scales[group] = pow2f(kexp);
                    }
                }
            }
        }
        if constexpr (!kEight) store_row<T, V, WIDE, SKEW>((T *)a.out, this_at, m, i, team, valid, h);
    }
}

// Rows that no team's registers hold: a block per row, element by element,
// the row read twice.  Every element is read and written by one
// thread, which reads it first: outputs may be the inputs themselves.
constexpr int kRowThreads = 256;
__device__ __forceinline__ float block_sum(float v, float *part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();  // the last use of part
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowThreads / 32; ++w) v += part[w];
    return v;
}

template <typename T, int CODEC, int B>
__global__ void __launch_bounds__(kRowThreads) k_rms_norm_elements(const __grid_constant__ RmsArgs a) {
    __shared__ float part[kRowThreads / 32];
    const T *w = (const T *)a.weight;
    const int lane = threadIdx.x & 31;
    for (uint64_t row = blockIdx.x + wait_prior_grid(); row < a.rows; row += gridDim.x) {
        const T *x = (const T *)a.x + row * a.cols;
        const T *res = a.residual ? (const T *)a.residual + row * a.cols : nullptr;
        auto h = [&](uint32_t c) {
            const float v = to_f32(x[c]);
            return res ? to_f32(from_f32<T>(v + to_f32(res[c]))) : v;
        };
        float s[8] = {};
        for (uint32_t c = threadIdx.x; c < a.cols; c += 8 * kRowThreads)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float v = c + k * kRowThreads < a.cols ? h(c + k * kRowThreads) : 0.0f;
                s[k] = fmaf(v, v, s[k]);
            }
        const float sum = block_sum(tree8(s), part);
        const float rstd = 1.0f / sqrtf(fmaf(sum, a.inv_cols, a.eps));
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
        constexpr uint32_t kB = CODEC == GB_CODEC_NONE ? 256 : B;
        const uint32_t nb = (a.cols + kB - 1) / kB;
        for (uint32_t b = threadIdx.x >> 5; b < nb; b += kRowThreads / 32) {
            float y[kB / 32];
            float m = 0.0f;
#pragma unroll
            for (int k = 0; k < (int)kB / 32; ++k) {
                const uint32_t c = b * kB + 32 * k + lane;
                y[k] = 0.0f;
                if (c >= a.cols) continue;
                const float v = h(c);
                y[k] = v * to_f32(w[c]) * rstd;
                if (a.sum) ((T *)a.sum)[row * a.cols + c] = from_f32<T>(v);
                if constexpr (CODEC == GB_CODEC_NONE) ((T *)a.out)[row * a.cols + c] = from_f32<T>(y[k]);
                m = fmaxf(m, fabsf(y[k]));
            }
            if constexpr (CODEC != GB_CODEC_NONE) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                const int kexp = block_scale_exp<CODEC>(m);
                const float inv = pow2f(-kexp);
#pragma unroll
                for (int k = 0; k < (int)kB / 32; ++k) {
                    const uint32_t c = b * kB + 32 * k + lane;
                    if (c < a.cols)
                        ((unsigned char *)a.out)[row * a.cols + c] =
                            (unsigned char)(cvt_fp8x2<CODEC>(y[k] * inv, 0.0f) & 0xFFu);
                }
                if (lane == 0) ((float *)((unsigned char *)a.out + a.scales_off))[row * nb + b] = pow2f(kexp);
            }
        }
    }
}

// --------------------------------------------------------------- gradient
// dx and, for the rows of each block, the sums of dy xhat of every column, in
// the registers of the thread that has the column: the rows of one team all
// have one skew.  A block's teams are joined in shared memory, the blocks by
// k_rms_dweight, both in a fixed order.
template <typename T, int V, bool WIDE, bool SKEW>
__global__ void __launch_bounds__(kMaxTeam) k_rms_grad(const __grid_constant__ RmsGradArgs a) {
    // A row ahead only where the registers hold it; of dsum not with a skew
    // either (2047 columns of bf16: 125 us, 157 with spills).
    constexpr bool kAhead = V * sizeof(T) <= 4, kAheadSum = kAhead && !SKEW;
    __shared__ float part[2][8][32];   // teams of several warps: 8 at most
    extern __shared__ float joined[];  // [teams, cols]
    const int team = a.team, place = threadIdx.x / team, i = threadIdx.x - place * team;
    const uint64_t per = blockDim.x / team, stride = gridDim.x * per;
    uint64_t row = blockIdx.x * per + place + wait_prior_grid();
    const Mine<V> m = mine_of<V>(row, a.cols, i, team);
    uint64_t at = row * a.cols - m.skew;
    Raw8<T> w[V], dy[V], h[V], ds[V];
    float acc[V][8] = {}, rstd = 0.0f;
    load_weights<T, V, WIDE, SKEW>(w, (const T *)a.weight, m, i, team, a.cols);
    auto load = [&]() {
        const bool valid = row < a.rows, cut = valid && row >= a.whole_rows;
        load_row<T, V, WIDE, SKEW>(dy, (const T *)a.dy, at, m, i, team, valid, cut);
        load_row<T, V, WIDE, SKEW>(h, (const T *)a.h, at, m, i, team, valid, cut);
        if (kAheadSum && a.dsum) load_row<T, V, WIDE, SKEW>(ds, (const T *)a.dsum, at, m, i, team, valid, cut);
        rstd = valid ? a.rstd[row] : 0.0f;
    };
    if (kAhead) load();
    int parity = 0;
    for (uint64_t base = row - (team < 32 ? (threadIdx.x & 31) / team : 0); base < a.rows; base += stride, parity ^= 1) {
        if (!kAhead) load();
        const uint64_t this_at = at;
        const bool valid = row < a.rows;
        const float scale = rstd;
        float s[8] = {};
        Raw8<T> this_dy[V], this_h[V], d[V];  // dy and h stay packed across the barrier
        if (!kAheadSum && a.dsum) load_row<T, V, WIDE, SKEW>(d, (const T *)a.dsum, at, m, i, team, valid, valid && row >= a.whole_rows);
        if constexpr (SKEW) {
            cut_row<T, V>(dy, m);
            cut_row<T, V>(h, m);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float e[8], xhat[8], f[8];
            this_dy[v] = dy[v];
            this_h[v] = h[v];
            if (kAheadSum && a.dsum) d[v] = ds[v];
            unpack8(dy[v], e);
            unpack8(h[v], xhat);
            unpack8(w[v], f);
            scale8(xhat, scale);
            fma8(acc[v], e, xhat);
            mul8(e, f);
            fma8(s, e, xhat);
        }
        row += stride;
        at += stride * a.cols;
        if (kAhead) load();
        const float c = -team_sum(tree8(s), team, part[parity][place & 7], place) * a.inv_cols;
        const float minus[8] = {c, c, c, c, c, c, c, c};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float e[8], xhat[8], f[8];
            unpack8(this_dy[v], e);
            unpack8(this_h[v], xhat);
            unpack8(w[v], f);
            mul8(e, f);
            scale8(xhat, scale);
            fma8(e, xhat, minus);
            scale8(e, scale);
            if (a.dsum) {
                unpack8(d[v], f);
                add8(e, f);
            }
            d[v] = pack8<T>(e);
        }
        store_row<T, V, WIDE, SKEW>((T *)a.dx, this_at, m, i, team, valid, d);
    }
    float *const out = a.partials + (uint64_t)blockIdx.x * a.cols;
    float *const to = per == 1 ? out : joined + place * a.cols;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = 8 * (i + v * team) + k - m.skew;
            if (c >= 0 && c < (int)a.cols) to[c] = acc[v][k];
        }
    if (per == 1) return;
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float s = 0.0f;
        for (uint32_t t = 0; t < per; ++t) s += joined[t * a.cols + c];
        out[c] = s;
    }
}

// dweight of 32 columns a block: 32 warps add every 32nd partial each, then
// one warp their sums.
template <typename T>
__global__ void __launch_bounds__(1024) k_rms_dweight(const __grid_constant__ RmsGradArgs a) {
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t c = blockIdx.x * 32 + lane + wait_prior_grid();
    float s = 0.0f;
    if (c < a.cols)
        for (int p = warp; p < a.n_partials; p += 32) s += __ldcg(a.partials + (uint64_t)p * a.cols + c);
    sums[lane][warp] = s;
    __syncthreads();
    s = sums[warp][lane];  // column `warp`
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const uint32_t mine = blockIdx.x * 32 + warp;
    if (lane == 0 && mine < a.cols) ((T *)a.dweight)[mine] = from_f32<T>(s);
}

// Rows that no team of registers holds: the columns' partial sums first (dx
// may overwrite dy), then dx, the row read twice.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) k_rms_partials_elements(const __grid_constant__ RmsGradArgs a) {
    const uint32_t c = blockIdx.x * kRowThreads + threadIdx.x + wait_prior_grid();
    if (c >= a.cols) return;
    float s = 0.0f;
    for (uint64_t row = blockIdx.y; row < a.rows; row += gridDim.y)
        s = fmaf(to_f32(((const T *)a.dy)[row * a.cols + c]), to_f32(((const T *)a.h)[row * a.cols + c]) * a.rstd[row], s);
    a.partials[(uint64_t)blockIdx.y * a.cols + c] = s;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) k_rms_dx_elements(const __grid_constant__ RmsGradArgs a) {
    __shared__ float part[kRowThreads / 32];
    const T *w = (const T *)a.weight;
    for (uint64_t row = blockIdx.x + wait_prior_grid(); row < a.rows; row += gridDim.x) {
        const T *dy = (const T *)a.dy + row * a.cols, *h = (const T *)a.h + row * a.cols;
        const T *dsum = a.dsum ? (const T *)a.dsum + row * a.cols : nullptr;
        T *dx = (T *)a.dx + row * a.cols;
        const float rstd = a.rstd[row];
        float s = 0.0f;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kRowThreads)
            s = fmaf(to_f32(dy[c]) * to_f32(w[c]), to_f32(h[c]) * rstd, s);
        const float mean = block_sum(s, part) * a.inv_cols;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kRowThreads) {
            float d = rstd * fmaf(-to_f32(h[c]) * rstd, mean, to_f32(dy[c]) * to_f32(w[c]));
            if (dsum) d += to_f32(dsum[c]);
            dx[c] = from_f32<T>(d);
        }
    }
}

// ----------------------------------------------------------------- launch
// Blocks of `threads` threads and `shared` dynamic bytes of a kernel that one
// SM holds; the runtime is asked when they are not those of the last call.
template <auto Kern>
static unsigned resident(unsigned threads, size_t shared) {
    static std::atomic<uint64_t> last{0};  // shared << 32 | threads << 16 | blocks
    const uint64_t key = (uint64_t)shared << 32 | (uint64_t)threads << 16, known = last.load(std::memory_order_relaxed);
    if (known && (known & ~0xFFFFull) == key) return (unsigned)(known & 0xFFFF);
    int v = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, Kern, (int)threads, shared) != cudaSuccess) cudaGetLastError();
    const unsigned n = v > 0 ? (unsigned)v : 1;
    last.store(key | n, std::memory_order_relaxed);
    return n;
}
// `waves` resident waves of blocks, fewer where there are fewer rows: each
// team walks over many rows, and its loads run one row ahead.  A multiple of
// 8 blocks, as the teams' rows are to keep their skew.
template <auto Kern>
static unsigned grid_of(uint64_t rows, int team, unsigned threads, size_t shared, unsigned waves) {
    const uint64_t per = threads / team, want = (rows + per - 1) / per;
    uint64_t cap = (uint64_t)sm_count() * resident<Kern>(threads, shared) * waves;
    cap = cap < 8 ? 8 : cap / 8 * 8;
    return (unsigned)(want < cap ? want : cap);
}

static bool wide(const void *const *p, int count) {
    for (int i = 0; i < count; ++i)
        if ((uintptr_t)p[i] & 31u) return false;
    return true;
}

template <typename T, int CODEC, int B, int V, bool WIDE, bool SKEW>
static cudaError_t rms_launch(RmsArgs &a, cudaStream_t s) {
    constexpr auto kern = k_rms_norm<T, CODEC, B, V, WIDE, SKEW>;
    a.team = team_of(a.cols, V);
    const unsigned threads = a.team >= 32 ? (unsigned)a.team : 256u;
    // Waves.  Float32: two (16384 x 2048 83 us, 65536 x 768 126; one wave 86
    // and 128; but 4099 x 769 takes 8.9 us, in one wave 7.9).  16 bits: one
    // (8192 x 5632 to E4M3 54 us, 4099 x 769 7.8; two waves 55 and 8.9; but
    // 32768 x 2048 in 16 bits takes 88 us, in two waves 84).
    return launch_pdl(kern, dim3(grid_of<kern>(a.rows, a.team, threads, 0, sizeof(T) == 4 ? 2 : 1)), threads, 0, a, s);
}

template <typename T, int CODEC, int B, int V>
static cudaError_t rms_rows(RmsArgs &a, cudaStream_t s) {
    const void *const buffers[] = {a.x, a.residual, a.sum, CODEC == GB_CODEC_NONE ? a.out : nullptr};
    const bool skew = a.cols % 8 != 0;
    if constexpr (sizeof(T) == 4)
        if (wide(buffers, 4))
            return skew ? rms_launch<T, CODEC, B, V, true, true>(a, s) : rms_launch<T, CODEC, B, V, true, false>(a, s);
    if constexpr (sizeof(T) == 2 && V == 2) return rms_launch<T, CODEC, B, V, false, true>(a, s);  // taken for a skew only
    else if constexpr (V == 3) return rms_launch<T, CODEC, B, V, false, false>(a, s);              // and without one
    else return skew ? rms_launch<T, CODEC, B, V, false, true>(a, s) : rms_launch<T, CODEC, B, V, false, false>(a, s);
}

template <typename T, int CODEC, int B>
static cudaError_t rms_forward(RmsArgs &a, cudaStream_t s) {
    // How many vectors a thread has.  One for rows within a warp, and for the
    // latency of few rows.  Four in 16-bit types (32768 x 2048 bf16 rows with
    // residual to E4M3: 75 us, 6.2 TB/s; two 78, one 106), or three where that
    // leaves no more lanes idle (65536 x 768 to E4M3: 56 us, four 66; 8192 x
    // 5632 to E5M2: 55 us, four 60); two where float32 or a skew needs the
    // registers (16384 x 2048 float32: 83 us, 6.5 TB/s; 2047 columns of bf16:
    // two 105 us, four 130).
    const bool skew = a.cols % 8 != 0;
    if (a.cols <= 249 || a.cols == 256 || (a.rows <= (uint64_t)sm_count() && team_of(a.cols, 1))) return rms_rows<T, CODEC, B, 1>(a, s);
    if ((sizeof(T) == 4 || skew) && team_of(a.cols, 2)) return rms_rows<T, CODEC, B, 2>(a, s);
    if constexpr (sizeof(T) == 2)
        if (!skew && team_of(a.cols, 3) && 3 * team_of(a.cols, 3) <= 4 * team_of(a.cols, 4)) return rms_rows<T, CODEC, B, 3>(a, s);
    if (team_of(a.cols, 4)) return rms_rows<T, CODEC, B, 4>(a, s);
    const uint64_t cap = (uint64_t)sm_count() * 64;
    return launch_pdl(k_rms_norm_elements<T, CODEC, B>, dim3((unsigned)(a.rows < cap ? a.rows : cap)), kRowThreads, 0, a, s);
}

template <typename T>
static cudaError_t rms_codec(RmsArgs &a, int codec, int block, cudaStream_t s) {
    switch (codec) {
    case GB_CODEC_NONE: return rms_forward<T, GB_CODEC_NONE, 256>(a, s);
    case GB_CODEC_E4M3: return block == 128 ? rms_forward<T, GB_CODEC_E4M3, 128>(a, s) : rms_forward<T, GB_CODEC_E4M3, 256>(a, s);
    default: return block == 128 ? rms_forward<T, GB_CODEC_E5M2, 128>(a, s) : rms_forward<T, GB_CODEC_E5M2, 256>(a, s);
    }
}

cudaError_t launch_rms_norm(RmsArgs &a, int dtype, int codec, int block, cudaStream_t s) {
    switch (dtype) {
    case GB_F32: return rms_codec<float>(a, codec, block, s);
    case GB_BF16: return rms_codec<__nv_bfloat16>(a, codec, block, s);
    default: return rms_codec<__half>(a, codec, block, s);
    }
}

// False: the blocks' partials do not fit the workspace, nothing is launched.
template <typename T, int V, bool WIDE, bool SKEW>
static bool grad_launch(RmsGradArgs &a, uint64_t fit, cudaStream_t s, cudaError_t &e) {
    constexpr auto kern = k_rms_grad<T, V, WIDE, SKEW>;
    a.team = team_of(a.cols, V);
    // as many teams as a block holds, for few partials
    const unsigned threads = a.team <= 32 ? 256u : (unsigned)(kMaxTeam / a.team * a.team);
    const size_t shared = threads > (unsigned)a.team ? threads / a.team * a.cols * sizeof(float) : 0;
    const unsigned blocks = grid_of<kern>(a.rows, a.team, threads, shared, 1);
    if (blocks > fit) return false;
    a.n_partials = (int)blocks;
    e = launch_pdl(kern, dim3(blocks), threads, shared, a, s);
    return true;
}
template <typename T, int V>
static bool grad_rows(RmsGradArgs &a, uint64_t fit, cudaStream_t s, cudaError_t &e) {
    const void *const buffers[] = {a.dy, a.h, a.dsum, a.dx};
    const bool skew = a.cols % 8 != 0;
    if constexpr (sizeof(T) == 4)
        if (wide(buffers, 4))
            return skew ? grad_launch<T, V, true, true>(a, fit, s, e) : grad_launch<T, V, true, false>(a, fit, s, e);
    return skew ? grad_launch<T, V, false, true>(a, fit, s, e) : grad_launch<T, V, false, false>(a, fit, s, e);
}

template <typename T>
static cudaError_t rms_backward(RmsGradArgs &a, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const uint64_t fit = kWorkFloats / a.cols;  // partials in the workspace, 1 or more
    a.n_partials = 0;
    // Two vectors a thread in 16-bit types (32768 x 2048 bf16 with dsum: 87 us,
    // 6.2 TB/s; one 110), one in float32 (16384 x 2048: 85 us, 6.3 TB/s; two 105).
    const bool one = a.cols <= 249 || a.cols == 256 || sizeof(T) == 4 || a.rows <= (uint64_t)sm_count();
    const bool rows = a.rows && ((one && team_of(a.cols, 1))   ? grad_rows<T, 1>(a, fit, s, e)
                                 : team_of(a.cols, 2) ? grad_rows<T, 2>(a, fit, s, e)
                                 : team_of(a.cols, 4) ? grad_rows<T, 4>(a, fit, s, e)
                                                      : false);
    if (a.rows && !rows) {
        const uint64_t most = fit < 608 ? fit : 608;
        a.n_partials = (int)(a.rows < most ? a.rows : most);
        e = launch_pdl(k_rms_partials_elements<T>, dim3((a.cols + kRowThreads - 1) / kRowThreads, a.n_partials), kRowThreads, 0, a, s);
    }
    if (e == cudaSuccess) e = launch_pdl(k_rms_dweight<T>, dim3((a.cols + 31) / 32), 1024, 0, a, s);
    if (e == cudaSuccess && a.rows && !rows) {
        const uint64_t cap = (uint64_t)sm_count() * 64;
        e = launch_pdl(k_rms_dx_elements<T>, dim3((unsigned)(a.rows < cap ? a.rows : cap)), kRowThreads, 0, a, s);
    }
    return e;
}

cudaError_t launch_rms_norm_backward(RmsGradArgs &a, int dtype, cudaStream_t s) {
    switch (dtype) {
    case GB_F32: return rms_backward<float>(a, s);
    case GB_BF16: return rms_backward<__nv_bfloat16>(a, s);
    default: return rms_backward<__half>(a, s);
    }
}

}  // namespace gb
