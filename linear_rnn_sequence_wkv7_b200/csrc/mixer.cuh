// Shared pieces of the state-space mixer's kernels (conv.cu, ssm_scan.cu,
// ssm_bwd.cu, rmsnorm.cu, act8.cu): typed loads and stores, the activation
// functions, and the 8-bit activation format.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "wkv7_ssm.h"

namespace wkv7 {
namespace mixer {

typedef __nv_bfloat16 bf16;
struct e4m3 { uint8_t code; };       // an 8-bit activation's code (its scale is kept apart)

constexpr int kBlk = WKV7_ACT8_BLOCK;
constexpr float kLog2e = 1.4426950408889634f;

// ---- V consecutive elements ---------------------------------------------------

template <bool CONST, typename W> __device__ __forceinline__ W word(const W *p) {
    if constexpr (CONST) return __ldg(p);
    else return *p;
}
// Raw words first, values later: a batch of loads is issued before the first
// conversion waits for one.
template <typename T, int V> struct Vec {
    static constexpr int BYTES = V * (int)sizeof(T);
    uint32_t w[(BYTES + 3) / 4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (BYTES + 3) / 4; ++i) w[i] = 0;
    }
    // CONST: nothing writes this memory during the kernel (a tensor that is updated in place is no such memory)
    template <bool CONST = true> __device__ __forceinline__ void load(const T *p) {
        if constexpr (BYTES == 1) w[0] = word<CONST>(reinterpret_cast<const uint8_t *>(p));
        else if constexpr (BYTES == 2) w[0] = word<CONST>(reinterpret_cast<const uint16_t *>(p));
        else if constexpr (BYTES == 4) w[0] = word<CONST>(reinterpret_cast<const uint32_t *>(p));
        else if constexpr (BYTES == 8) {
            const uint2 u = word<CONST>(reinterpret_cast<const uint2 *>(p));
            w[0] = u.x, w[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i) {
                const uint4 u = word<CONST>(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ void get(float (&f)[V]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = __uint_as_float(w[i]);
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                f[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
        } else if constexpr (V == 1) {
            f[0] = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)w[0], __NV_E4M3)));
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                    (__nv_fp8x2_storage_t)((w[i / 4] >> (8 * (i % 4))) & 0xffffu), __NV_E4M3);
                const float2 p = __half22float2(__half2(h));
                f[i] = p.x, f[i + 1] = p.y;
            }
        }
    }
};

template <int V> __device__ __forceinline__ void storev(float *p, const float (&f)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    } else if constexpr (V == 2) {
        *reinterpret_cast<float2 *>(p) = make_float2(f[0], f[1]);
    } else {
        p[0] = f[0];
    }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&t);
}
template <int V> __device__ __forceinline__ void storev(bf16 *p, const float (&f)[V]) {
    if constexpr (V == 8) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
    } else if constexpr (V == 2) {
        *reinterpret_cast<uint32_t *>(p) = pack2(f[0], f[1]);
    } else {
        p[0] = __float2bfloat16_rn(f[0]);
    }
}

// BYTES (4, 8 or 16) to shared memory without passing through registers; zeros when !in
template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES),
                 "r"(in ? BYTES : 0)
                 : "memory");
}

// ---- functions ------------------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + e^-x).  The exponent's rounding, |x| log2(e) 2^-24, is below a bf16
// result's half step for every |x| < 88; PRECISE (fp32 results; in the scan fp32
// inputs as well) uses expf.  (The fp32 parameter gradients of a call with bf16
// gradients carry it: |z| log2(e) 2^-24 of a term, less than their sums collect.)
template <bool PRECISE> __device__ __forceinline__ float sigmoid(float x) {
    return rcp(1.f + (PRECISE ? expf(-x) : ex2(-x * kLog2e)));
}
template <bool PRECISE> __device__ __forceinline__ float2 sigmoid2(float2 x) {
    if constexpr (PRECISE) return make_float2(sigmoid<true>(x.x), sigmoid<true>(x.y));
    const float2 t = __fmul2_rn(x, make_float2(-kLog2e, -kLog2e));
    const float2 d = __fadd2_rn(make_float2(ex2(t.x), ex2(t.y)), make_float2(1.f, 1.f));
    return make_float2(rcp(d.x), rcp(d.y));
}
// log(1 + e^x) = max(x, 0) + log1p(e), e = e^-|x| in (0, 1]; log1p(e) / e by its
// Chebyshev interpolant of degree 9 on [0, 1] (off by 6e-9 of the value, 1e-7
// evaluated in fp32), which keeps small values exact where log(1 + e) would not.
// Not PRECISE (bf16 inputs, which are off by 2^-9 themselves): e by one ex2, off by
// |x| log2(e) 2^-24, no more than e moves by the rounding of x = delta + dt_bias to
// fp32.  Two values at a time: one packed instruction a step.
template <bool PRECISE> __device__ __forceinline__ float2 softplus2(float2 x) {
    float2 e;
    if constexpr (PRECISE) {
        e = make_float2(expf(-fabsf(x.x)), expf(-fabsf(x.y)));
    } else {
        const float2 t = __fmul2_rn(make_float2(fabsf(x.x), fabsf(x.y)), make_float2(-kLog2e, -kLog2e));
        e = make_float2(ex2(t.x), ex2(t.y));
    }
    constexpr float c[10] = {-3.1760570e-3f, 1.9542528e-2f, -5.6373615e-2f, 1.0543624e-1f, -1.5269667e-1f,
                             1.9663274e-1f,  -2.4951616e-1f, 3.3329710e-1f, -4.9999893e-1f, 1.f};
    float2 p = make_float2(c[0], c[0]);
#pragma unroll
    for (int i = 1; i < 10; ++i) p = __ffma2_rn(p, e, make_float2(c[i], c[i]));
    return __ffma2_rn(e, p, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}
template <bool PRECISE> __device__ __forceinline__ float softplus(float x) {
    return softplus2<PRECISE>(make_float2(x, x)).x;
}
// softplus of V values in place
template <bool PRECISE, int V> __device__ __forceinline__ void softplus_all(float (&x)[V]) {
    if constexpr (V == 1) x[0] = softplus<PRECISE>(x[0]);
    else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 r = softplus2<PRECISE>(make_float2(x[i], x[i + 1]));
            x[i] = r.x, x[i + 1] = r.y;
        }
    }
}

template <typename F> __device__ __forceinline__ F warp_add(F x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ---- roundings ---------------------------------------------------------------------

// The float next to the exact value s + err whose last bit is set (round to
// odd), or s when err is 0: rounding that to fewer bits gives what rounding the
// exact value once would.  |err| is at most half a step of s.
__device__ __forceinline__ float to_odd(float s, float err) {
    const int b = __float_as_int(s);
    const bool moves = (err < 0.f || err > 0.f) && !(b & 1);
    return moves ? __int_as_float(b + (((err > 0.f) == (b >= 0)) ? 1 : -1)) : s;
}
// (a + b) - fl(a + b), exactly, of two pairs: the two-sum of Knuth (The Art of
// Computer Programming, vol. 2, section 4.2.2); s = fl(a + b)
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.f, -1.f), a); }
__device__ __forceinline__ float2 sum_error(float2 a, float2 b, float2 s) {
    const float2 t = sub2(s, a);
    return __fadd2_rn(sub2(a, sub2(s, t)), sub2(b, t));
}

// ---- the 8-bit format --------------------------------------------------------------

// Exponent field of the least power of two >= amax / 448, at least 2^-117:
// amax = 1.m 2^e and 448 = 1.75 2^8, so 2^(e - 8), or the next above when 1.m > 1.75.
__device__ __forceinline__ uint32_t act8_exponent(uint32_t b) {     // b: amax's bits
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u);
    return (uint32_t)max(e, 10);
}

// The warp's block of 128 values, 4 in each lane.  Bits of absolute values order
// like the values, so amax is one warp-wide integer maximum.  NaN drops out of it
// (and converts to the NaN code by itself); an infinity shows.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t act8_top(const float (&v)[4]) {
    const float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
    return __reduce_max_sync(0xffffffffu, m == m ? __float_as_uint(m) : 0u);
}
__device__ __forceinline__ uint32_t act8_pack(const float (&q)[4]) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
// Scale and codes.  Infinities and NaN become NaN codes and are left out of amax.
__device__ __forceinline__ float act8_encode(const float (&x)[4], uint32_t &codes) {
    float v[4] = {x[0], x[1], x[2], x[3]};
    uint32_t top = act8_top(v);
    if (top >= 0x7f800000u) {                   // uniform in the warp, rare
        top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (abs_bits(v[i]) < 0x7f800000u) top = max(top, abs_bits(v[i]));
            else v[i] = __uint_as_float(0x7fffffffu);
        }
        top = __reduce_max_sync(0xffffffffu, top);
    }
    const uint32_t e = act8_exponent(top);
    const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= inv;
    if (e == 247u) {            // code 256 would stand for 2^128: the largest numbers take 240, within 2^-4 of them
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (fabsf(v[i]) > 240.f) v[i] = copysignf(240.f, v[i]);
    }
    codes = act8_pack(v);
    return __uint_as_float(e << 23);
}
// K blocks one after another; the usual case without a branch between them, so that their maxima overlap
template <int K>
__device__ __forceinline__ void act8_encode_all(const float (&x)[K][4], uint32_t (&codes)[K], float (&scale)[K]) {
    uint32_t top[K], worst = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        top[k] = act8_top(x[k]);
        worst = max(worst, top[k]);
    }
    if (worst >= 0x7f600000u) {                 // infinities, NaN, or within a step of 2^128
#pragma unroll
        for (int k = 0; k < K; ++k) scale[k] = act8_encode(x[k], codes[k]);
        return;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t e = act8_exponent(top[k]);
        const float inv = __uint_as_float((254u - e) << 23);
        const float q[4] = {x[k][0] * inv, x[k][1] * inv, x[k][2] * inv, x[k][3] * inv};
        codes[k] = act8_pack(q);
        scale[k] = __uint_as_float(e << 23);
    }
}
// The same where every value is known to within 2^-22 of itself only: false if a
// code or the scale could depend on more, that is if the values a 2^-21 below and
// above have other codes, amax is next to a power's border, or numbers are too
// large or too small for the scale.  A block of zeros (among them the blocks that a
// warp holds behind a row's end) or of NaN is sure: its codes are 0 or NaN.
// Uniform in the warp.
__device__ __forceinline__ bool act8_encode_sure(const float (&x)[4], uint32_t &codes, float &scale) {
    const uint32_t top = act8_top(x), e = act8_exponent(top);
    const float inv = __uint_as_float((254u - e) << 23);
    const bool border = (top & 0x7fffffu) - 0x5ffff8u <= 16u || top > 0x7b000000u || top - 1u < 0x08000000u - 1u;
    float lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float2 q = make_float2(x[i], x[i + 1]);
        const float a = inv * (1.f - 0x1p-21f), b = inv * (1.f + 0x1p-21f);
        const float2 l = __fmul2_rn(q, make_float2(a, a)), h = __fmul2_rn(q, make_float2(b, b));
        lo[i] = l.x, lo[i + 1] = l.y, hi[i] = h.x, hi[i + 1] = h.y;
    }
    codes = act8_pack(lo);
    scale = __uint_as_float(e << 23);
    return !__any_sync(0xffffffffu, border || codes != act8_pack(hi));
}

// ---- rows cut into blocks of 128 channels, a warp to a block -------------------------

// Channel of a lane's i-th element of block `blk`: four in a row where the row
// allows vector accesses, else one in every 32.
template <bool VEC> __device__ __forceinline__ int lane_channel(int blk, int lane, int i) {
    return blk * kBlk + (VEC ? 4 * lane + i : lane + 32 * i);
}
// A lane's four elements of a block: raw words first, values later
template <typename T, bool VEC> struct Row4 {
    Vec<T, VEC ? 4 : 1> v[VEC ? 1 : 4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (auto &e : v) e.zero();
    }
    template <bool CONST = true> __device__ __forceinline__ void load(const T *row, int blk, int lane, int D) {
#pragma unroll
        for (int i = 0; i < (VEC ? 1 : 4); ++i) {
            v[i].zero();
            const int c = lane_channel<VEC>(blk, lane, i);
            if (c < D) v[i].template load<CONST>(row + c);
        }
    }
    __device__ __forceinline__ void get(float (&f)[4]) const {
        if constexpr (VEC) v[0].get(f);
        else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float g[1];
                v[i].get(g);
                f[i] = g[0];
            }
        }
    }
};
template <bool VEC, bool CONST = true, typename T>
__device__ __forceinline__ void row_load(const T *row, int blk, int lane, int D, float (&f)[4]) {
    Row4<T, VEC> r;
    r.template load<CONST>(row, blk, lane, D);
    r.get(f);
}
template <bool VEC, typename T>
__device__ __forceinline__ void row_store(T *row, int blk, int lane, int D, const float (&f)[4]) {
    if constexpr (VEC) {
        const int c = lane_channel<true>(blk, lane, 0);
        if (c < D) storev<4>(row + c, f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = lane_channel<false>(blk, lane, i);
            const float g[1] = {f[i]};
            if (c < D) storev<1>(row + c, g);
        }
    }
}
template <bool VEC>
__device__ __forceinline__ void row_store_codes(uint8_t *row, int blk, int lane, int D, uint32_t codes) {
    if constexpr (VEC) {
        const int c = lane_channel<true>(blk, lane, 0);
        if (c < D) *reinterpret_cast<uint32_t *>(row + c) = codes;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = lane_channel<false>(blk, lane, i);
            if (c < D) row[c] = (uint8_t)(codes >> (8 * i));
        }
    }
}

// ---- host checks ----------------------------------------------------------------------

inline bool real_dtype(wkv7_dtype d) { return d == WKV7_F32 || d == WKV7_BF16; }
inline size_t dtype_size(wkv7_dtype d) { return d == WKV7_F32 ? 4 : d == WKV7_BF16 ? 2 : 1; }
inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// a pointer to elements of d: present and aligned to its element
inline bool elem_ok(const void *p, wkv7_dtype d) { return p != nullptr && aligned_to(p, dtype_size(d)); }
inline bool f32_ok(const void *p) { return p != nullptr && aligned_to(p, 4); }
inline bool f32_opt(const void *p) { return aligned_to(p, 4); }
inline int blocks_of(int D) { return (D + kBlk - 1) / kBlk; }
inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }
inline wkv7_status launch_status() { return cudaGetLastError() == cudaSuccess ? WKV7_OK : WKV7_ERR_CUDA; }
inline int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}
constexpr long long kMaxGrid = 2147483647LL;
constexpr int kMaxTokens = 1 << 30;

}  // namespace mixer
}  // namespace wkv7
