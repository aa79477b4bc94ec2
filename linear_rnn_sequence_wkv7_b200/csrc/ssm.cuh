// What the scan's forward and backward share: the thread layout, its arguments
// and the joins over lanes.
#pragma once

#include <type_traits>

#include "mixer.cuh"

namespace wkv7 {
namespace mixer {

constexpr int kTile = 16;           // tokens a tile, and between saved states
constexpr int kScanThreads = 128;

// lanes that share a channel pair: 4 n each
inline int scan_lanes(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
__host__ __device__ constexpr int scan_channels(int LN) { return 2 * kScanThreads / LN; }

template <typename F> void by_lanes(int LN, F &&f) {
    if (LN == 2) f(std::integral_constant<int, 2>{});
    else if (LN == 4) f(std::integral_constant<int, 4>{});
    else if (LN == 8) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 16>{});
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

__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }

// four numbers of a channel's state row; N need not be a multiple of 4
__device__ __forceinline__ void store_state(float *to, int N, int ns, const float2 (&h)[2]) {
    if ((N & 3) == 0) {
        if (ns < N) *reinterpret_cast<float4 *>(to) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
    } else {
        const float v[4] = {h[0].x, h[0].y, h[1].x, h[1].y};
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (ns + n < N) to[n] = v[n];
    }
}

// Sums of M values over L lanes side by side (l = lane in the group), scattered:
// while values are left to share out, a lane keeps the half that its lowest
// unused bit names and hands the other half over; then plain sums.  Afterwards a
// lane holds max(M / L, 1) sums, v[i] = that of value i min(L, M) + l mod min(L, M).
// STRIDE: lanes between neighbours of the group.
template <int L, int M, int STRIDE = 1> __device__ __forceinline__ void reduce_scatter(float (&v)[M], int l) {
    int left = M;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        if (left > 1) {
            left >>= 1;
            const bool up = l & o;
#pragma unroll
            for (int i = 0; i < M / 2; ++i) {
                if (i >= left) break;
                const float keep = up ? v[2 * i + 1] : v[2 * i], give = up ? v[2 * i] : v[2 * i + 1];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o * STRIDE);
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o * STRIDE);
        }
    }
}

}  // namespace mixer
}  // namespace wkv7
