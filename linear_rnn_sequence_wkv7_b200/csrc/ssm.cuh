// What the scan's forward and backward share: the thread layout, its arguments
// and the joins over lanes.
#pragma once

#include <type_traits>

#include "mixer.cuh"

namespace wkv7 {
namespace mixer {

constexpr int kTile = 16;           // tokens a tile, and between saved states

// N padded to 8, 16, 32 or 64; a thread holds 4 n of TC channels
inline int scan_pad(int N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }
__host__ __device__ constexpr int scan_channels(int NP) { return NP == 8 ? 32 : NP == 64 ? 8 : 16; }      // of a block
__host__ __device__ constexpr int scan_threads(int NP, int TC) { return scan_channels(NP) * NP / (4 * TC); }

// blocks of 2 scan_threads an SM that the registers must leave room for (the
// summaries spill at 20 warps)
__host__ __device__ constexpr int scan_blocks(int NP, int TC, bool y) { return (y ? 20 : 16) * 16 / scan_threads(NP, TC); }

template <typename F> void by_pad(int NP, F &&f) {
    if (NP == 8) f(std::integral_constant<int, 8>{});
    else if (NP == 16) f(std::integral_constant<int, 16>{});
    else if (NP == 32) f(std::integral_constant<int, 32>{});
    else f(std::integral_constant<int, 64>{});
}

// PRECISE of the gates (mixer.cuh) as a template argument, by the results' type and the inputs'.  A branch
// on the results' type in the kernels instead cost 2% of a forward and 8% of a backward, expf everywhere 2% and 6%.
template <typename T, typename F> void by_precision(bool f32_results, F &&f) {
    if (sizeof(T) == 4 || f32_results) f(std::true_type{});
    else f(std::bool_constant<sizeof(T) == 4>{});
}

struct ScanArgs {
    int B, T, D, N, G, Dg, tiles;   // Dg channels a group, in `tiles` blocks
    const void *u, *delta, *z, *Bm, *Cm;
    long long u_bs, u_ts, d_bs, d_ts, z_bs, z_ts, b_bs, b_ts, c_bs, c_ts;
    const float *A, *Dskip, *dt_bias;
    int softplus;
    const int *lens;
    void *y;
    int y_f32;
    float *stateT;
    float *states;                  // [B][nck][D][N]: h before every tile
    int nck;
    int nseg, seg_len;              // segments of seg_len tokens, a multiple of the tile
    const float *entry;             // [nseg][B][D][N], or null for zeros
    float *seg_end, *seg_dt;        // summaries: end state from zero, sum of dt
};

// volatile: the compiler keeps their order, and with it the distance to their use
__device__ __forceinline__ float ex2_ahead(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2_ahead(x.x), ex2_ahead(x.y)); }
// exp(dt A) of two rates in units of log 2.  ex2.approx is low by 0.1 to 0.45 of a
// result's last place on average below 0 (measured over [-2^-k, -2^-k-1], k = 0 ..
// 15), and a state that lives for a thousand tokens collects that a thousand times;
// an exponent 0.3 of a last place higher brings the mean within 0.15.  dt = 0 still
// gives 1.
__device__ __forceinline__ float2 decay(float2 dt, float2 a) {
    constexpr float kLift = 2.58e-8f;
    return ex2(__ffma2_rn(dt, a, make_float2(kLift, kLift)));
}

// Four n of a token's B or C; `left`: how many are there
template <typename T, bool VEC> struct Quad {
    Vec<T, VEC ? 4 : 1> v[VEC ? 1 : 4];
    __device__ __forceinline__ void load(const T *p, int left) {
#pragma unroll
        for (int i = 0; i < (VEC ? 1 : 4); ++i) {
            v[i].zero();
            if (i < left) v[i].load(p + i);
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
    // to shared memory, in the order 0 xor p, 1 xor p, ...
    __device__ __forceinline__ void put(float *to, int p = 0) const {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = VEC ? v[0].w[VEC ? i % (sizeof(v[0].w) / 4) : 0] : v[VEC ? 0 : i].w[0];
        *reinterpret_cast<uint4 *>(to) = make_uint4(w[0 ^ p], w[1 ^ p], w[2 ^ p], w[3 ^ p]);
    }
    __device__ __forceinline__ void put(bf16 *to, int p = 0) const {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = VEC ? v[0].w[VEC ? i : 0] : (v[VEC ? 0 : 2 * i].w[0] | (v[VEC ? 0 : 2 * i + 1].w[0] << 16));
        if (p & 1) w[0] = __byte_perm(w[0], 0, 0x1032), w[1] = __byte_perm(w[1], 0, 0x1032);
        *reinterpret_cast<uint2 *>(to) = (p & 2) ? make_uint2(w[1], w[0]) : make_uint2(w[0], w[1]);
    }
};

// A thread's numbers of a channel's state row, n = ns .. ns + 3; N need not be a multiple of 4
__device__ __forceinline__ void store_state(float *row, int N, int ns, const float2 (&h)[2]) {
    if ((N & 3) == 0) {
        if (ns < N) *reinterpret_cast<float4 *>(row + ns) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
    } else {
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (ns + n < N) row[ns + n] = (n & 1) ? h[n / 2].y : h[n / 2].x;
    }
}
__device__ __forceinline__ void load_state(const float *row, int N, int ns, float2 (&h)[2]) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if ((N & 3) == 0) {
        if (ns < N) {
            const float4 q = *reinterpret_cast<const float4 *>(row + ns);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        }
    } else {
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (ns + n < N) v[n] = row[ns + n];
    }
    h[0] = make_float2(v[0], v[1]), h[1] = make_float2(v[2], v[3]);
}
// The rates of a thread's n in units of log 2 (0 for the padding, which keeps a zero state at zero)
__device__ __forceinline__ void load_rates(const float *row, int N, int ns, bool live, float2 (&a)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int n = ns + 2 * j;
        a[j].x = (live && n < N) ? __ldg(row + n) * kLog2e : 0.f;
        a[j].y = (live && n + 1 < N) ? __ldg(row + n + 1) * kLog2e : 0.f;
    }
}
// B and C in shared memory keep their own type: a warp-wide load costs a cycle of
// the SM's shared memory for every 4 bytes a lane, broadcast or not, and at 16
// bytes each for B and C that would be the scan's bound.
// A thread's n of a token:
__device__ __forceinline__ void shared_n(const float *p, float2 (&v)[2]) {
    const float4 q = *reinterpret_cast<const float4 *>(p);
    v[0] = make_float2(q.x, q.y), v[1] = make_float2(q.z, q.w);
}
__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void shared_n(const bf16 *p, float2 (&v)[2]) {
    const uint2 q = *reinterpret_cast<const uint2 *>(p);
    v[0] = bf16_pair(q.x), v[1] = bf16_pair(q.y);
}

// (a_i, b_i) of V channels in a row
template <int V> __device__ __forceinline__ void put_pairs(float2 *to, const float (&a)[V], const float (&b)[V]) {
    if constexpr (V == 1) to[0] = make_float2(a[0], b[0]);
    else {
#pragma unroll
        for (int i = 0; i < V; i += 2)
            *reinterpret_cast<float4 *>(to + i) = make_float4(a[i], b[i], a[i + 1], b[i + 1]);
    }
}

// Sums over the LN lanes of a channel, through shared memory: [kTile][LN][CC]
// partial values, the planes and rows shifted so that neither the lanes' stores
// nor the loads of four channels in a row meet in a bank.
template <int CC, int LN> struct Planes {
    static constexpr int PS = CC + 32 / LN, RS = LN * PS + (CC == 16 ? 16 : 0), FLOATS = kTile * RS;
    template <int TC> static __device__ __forceinline__ void put(float *s, int k, int ch, int nl, const float (&v)[TC]) {
        storev<TC>(s + k * RS + nl * PS + ch, v);
    }
    template <int V> static __device__ __forceinline__ void sum(const float *s, int k, int ch, float (&out)[V]) {
        const float *p = s + k * RS + ch;
        if constexpr (V % 4 == 0) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                float4 t = *reinterpret_cast<const float4 *>(p + i);
                float2 x = make_float2(t.x, t.y), y = make_float2(t.z, t.w);
#pragma unroll
                for (int l = 1; l < LN; ++l) {
                    t = *reinterpret_cast<const float4 *>(p + l * PS + i);
                    x = __fadd2_rn(x, make_float2(t.x, t.y)), y = __fadd2_rn(y, make_float2(t.z, t.w));
                }
                out[i] = x.x, out[i + 1] = x.y, out[i + 2] = y.x, out[i + 3] = y.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float t = p[i];
#pragma unroll
                for (int l = 1; l < LN; ++l) t += p[l * PS + i];
                out[i] = t;
            }
        }
    }
};

}  // namespace mixer
}  // namespace wkv7
