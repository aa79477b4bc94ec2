// Short causal convolution (width 2 to 4), its single-token step and its
// backward.
//
//     p_t = bias + sum_j w_j x_{t-W+1+j},  y_t = p_t sigmoid(p_t)  (or p_t)
//     dp_t = dy_t act'(p_t),  dx_t = sum_j w_j dp_{t+W-1-j},  dw_j = sum_t dp_t x_{t-W+1+j}
//
// All three are bound by memory (2 + 2 bytes a bf16 element forward).  A warp
// holds a block of 128 channels, four a lane, and walks a run of tokens with
// the last W - 1 inputs in registers, so an input is read once and W - 1 halo
// tokens more a run; the 8-bit activation's scale belongs to exactly that block.
// What it took was bytes on their way: twelve tokens a warp through shared memory
// (cp.async) where eight in registers left too few warps.
//
// 8 x 4096 tokens x 2048 channels, W = 4, bf16: forward 52 us (269 MB, 80% of the
// measured copy rate), with its 8-bit copy 76 us (338 MB), from the codes 56 us
// (203 MB), backward from the codes 118 us (338 MB; 168 registers leave 12 warps an
// SM, which issue half of the cycles).
#include <type_traits>

#include "mixer.cuh"

namespace wkv7 {
namespace mixer {

void sum_parts(long long parts, long long cols, const float *partial, float *out, cudaStream_t st);

namespace {

constexpr int kConvWarps = 4;       // forward: warps a block, each a run of its own
constexpr int kConvMinRun = 16;
constexpr int kConvGroup = 4;       // tokens worked on together, unrolled
constexpr int kConvRing = 4;        // groups on their way or in use

// Four channels of one token, and the scale when they are codes
template <typename T, bool VEC> struct Token {
    Row4<T, VEC> r;
    float scale;
    __device__ __forceinline__ void zero() {
        r.zero();
        scale = 0.f;
    }
    __device__ __forceinline__ void load(const T *row, const float *scales, int blk, int lane, int D) {
        r.load(row, blk, lane, D);
        if constexpr (sizeof(T) == 1) scale = __ldg(scales);
    }
    __device__ __forceinline__ void get(float (&f)[4]) const {
        r.get(f);
        if constexpr (sizeof(T) == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] *= scale;
        }
    }
};

// Tokens on their way to a warp: kConvRing groups of kConvGroup, each lane's four
// channels in a slot of its own, copied (cp.async) by the lane that reads them.
// Where an element is too narrow for that (not VEC and not fp32), one group ahead
// in registers.
template <typename T, bool VEC> struct Stream {
    static constexpr bool ASYNC = VEC || sizeof(T) == 4;
    static constexpr int SLOT = 4 * (int)sizeof(T);
    static constexpr int WARP_BYTES = ASYNC ? kConvRing * kConvGroup * (32 * SLOT + (sizeof(T) == 1 ? 4 : 0)) : 0;   // a warp
    unsigned char *base;
    Token<T, VEC> next[ASYNC ? 1 : kConvGroup];
    __device__ __forceinline__ unsigned char *slot(int i, int lane) const { return base + (i * 32 + lane) * SLOT; }
    __device__ __forceinline__ float *scale(int i) const {
        return reinterpret_cast<float *>(base + kConvRing * kConvGroup * 32 * SLOT) + i;
    }
    // group g of tokens from `row` on, `left` of them there (the others count as zero)
    __device__ __forceinline__ void fetch(int g, const T *row, long long ts, const float *scales, int nblk, int left,
                                          int blk, int lane, int D) {
        if constexpr (!ASYNC) {
#pragma unroll
            for (int k = 0; k < kConvGroup; ++k) {
                next[k].zero();
                if (k < left) next[k].load(row + k * ts, scales + (long long)k * nblk, blk, lane, D);
            }
        } else {
            unsigned char *to = slot((g % kConvRing) * kConvGroup, lane);
            constexpr int PARTS = VEC ? 1 : 4, BYTES = SLOT / PARTS;
            const T *p[PARTS];
            bool there[PARTS];
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                const int c = lane_channel<VEC>(blk, lane, i);
                there[i] = c < D;
                p[i] = there[i] ? row + c : row;
            }
            if (VEC && left >= kConvGroup) {
#pragma unroll
                for (int k = 0; k < kConvGroup; ++k, p[0] += ts) copy_async<BYTES>(to + k * 32 * SLOT, p[0], there[0]);
            } else {
#pragma unroll
                for (int k = 0; k < kConvGroup; ++k) {
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) {
                        const bool in = there[i] && k < left;
                        copy_async<BYTES>(to + k * 32 * SLOT + i * BYTES, k < left ? p[i] : row, in);
                        p[i] += ts;
                    }
                }
            }
        }
        if constexpr (ASYNC && sizeof(T) == 1) {
            if (lane < kConvGroup) {
                const bool in = lane < left;
                copy_async<4>(scale((g % kConvRing) * kConvGroup + lane), in ? scales + (long long)lane * nblk : scales, in);
            }
        }
    }
    __device__ __forceinline__ void get(int g, int lane, float (&v)[kConvGroup][4]) const {
#pragma unroll
        for (int k = 0; k < kConvGroup; ++k) {
            if constexpr (ASYNC) {
                const int i = (g % kConvRing) * kConvGroup + k;
                Vec<T, 4> r;
                const uint32_t *w = reinterpret_cast<const uint32_t *>(slot(i, lane));
                if constexpr (SLOT == 16) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(w);
                    r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
                } else if constexpr (SLOT == 8) {
                    const uint2 q = *reinterpret_cast<const uint2 *>(w);
                    r.w[0] = q.x, r.w[1] = q.y;
                } else {
                    r.w[0] = w[0];
                }
                r.get(v[k]);
                if constexpr (sizeof(T) == 1) {
                    const float2 f = make_float2(*scale(i), *scale(i));
#pragma unroll
                    for (int c = 0; c < 4; c += 2) {
                        const float2 q = __fmul2_rn(make_float2(v[k][c], v[k][c + 1]), f);
                        v[k][c] = q.x, v[k][c + 1] = q.y;
                    }
                }
            } else {
                next[k].get(v[k]);
            }
        }
    }
};

template <bool VEC, typename T>
__device__ __forceinline__ void load4c(const T *row, int blk, int lane, int D, float (&f)[4]) {
    row_load<VEC>(row, blk, lane, D, f);
}
// Four channels as two pairs: one packed instruction works on a pair
__device__ __forceinline__ void pairs(const float (&f)[4], float2 (&p)[2]) {
    p[0] = make_float2(f[0], f[1]), p[1] = make_float2(f[2], f[3]);
}

// A lane's weights and biases; with vector accesses its 4 W weights are one stretch of memory
template <int W, bool VEC>
__device__ __forceinline__ void load_params(const float *weight, const float *bias, int blk, int lane, int D,
                                            float2 (&w)[W][2], float2 (&b)[2]) {
    float f[4], v[4 * W];
    if constexpr (VEC) {
        const int c = lane_channel<true>(blk, lane, 0);
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float4 q = c < D ? __ldg(reinterpret_cast<const float4 *>(weight + (size_t)c * W) + j) : zero;
            v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
        }
        const float4 q = (bias && c < D) ? __ldg(reinterpret_cast<const float4 *>(bias + c)) : zero;
        f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = lane_channel<false>(blk, lane, i);
            f[i] = (bias && c < D) ? __ldg(bias + c) : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) v[i * W + j] = c < D ? __ldg(weight + (size_t)c * W + j) : 0.f;
        }
    }
    pairs(f, b);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        w[j][0] = make_float2(v[j], v[W + j]);
        w[j][1] = make_float2(v[2 * W + j], v[3 * W + j]);
    }
}

struct ConvFwd {
    int B, T, D;
    const void *x;
    long long x_bs, x_ts;
    const float *x_scales;
    const float *weight, *bias;
    const void *state;
    const int *lens;
    int silu;
    void *y, *state_out;
    uint8_t *codes;
    float *scales;
    int runs, run;                  // runs of `run` tokens
};

// ST: the state's type (x's, or y's when x is codes).  SAVE: x's codes go out too.
template <typename T, typename ST, typename YT, int W, bool VEC, bool SAVE>
__global__ void __launch_bounds__(32 * kConvWarps, VEC && !SAVE ? 6 : 4)
conv_fwd_kernel(const ConvFwd P) {
    constexpr bool PRECISE = sizeof(YT) == 4;
    const int lane = threadIdx.x & 31, D = P.D, nblk = (D + kBlk - 1) / kBlk;
    const long long unit = (long long)blockIdx.x * kConvWarps + (threadIdx.x >> 5);
    const int blk = (int)(unit % nblk);
    const long long rest = unit / nblk;
    const int run = (int)(rest % P.runs);
    const long long b = rest / P.runs;
    if (b >= P.B) return;
    int len = P.T;
    if (P.lens) len = min(max(__ldg(P.lens + b), 0), P.T);
    const int t0 = min(run * P.run, len), t1 = min(t0 + P.run, len);
    const T *x = static_cast<const T *>(P.x) + b * P.x_bs;
    const ST *state = static_cast<const ST *>(P.state);
    const float *xs = sizeof(T) == 1 ? P.x_scales + b * P.T * nblk + blk : nullptr;
    auto past = [&](int t, float (&f)[4]) {         // x at t >= -(W - 1), t < len
        if (t >= 0) {
            Token<T, VEC> k;
            k.load(x + t * P.x_ts, xs + (long long)t * nblk, blk, lane, D);
            k.get(f);
        } else if (state) {
            load4c<VEC>(state + (b * (W - 1) + (t + W - 1)) * D, blk, lane, D, f);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = 0.f;
        }
    };
    if constexpr (sizeof(T) > 1) {
        if (P.state_out && run == 0) {              // the last W - 1 inputs of the sequence, as they are
            T *so = static_cast<T *>(P.state_out);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                float f[4];
                past(len - (W - 1) + j, f);
                row_store<VEC>(so + (b * (W - 1) + j) * D, blk, lane, D, f);
            }
        }
    }
    if (t0 >= t1) return;
    const long long row0 = b * P.T + t0;
    const T *px = x + t0 * P.x_ts;
    const float *ps = xs + (long long)t0 * nblk;
    YT *py = static_cast<YT *>(P.y) + row0 * D;
    uint8_t *pc = SAVE ? P.codes + row0 * D : nullptr;
    float *pq = SAVE ? P.scales + row0 * nblk + blk : nullptr;
    extern __shared__ __align__(16) unsigned char conv_smem[];
    Stream<T, VEC> in{conv_smem + (threadIdx.x >> 5) * Stream<T, VEC>::WARP_BYTES};
    constexpr bool ASYNC = Stream<T, VEC>::ASYNC;
    auto fetch = [&](int g) {           // in order: the pointers go on from group to group
        const int t = t0 + g * kConvGroup;
        if (t < t1) in.fetch(g, px, P.x_ts, ps, nblk, t1 - t, blk, lane, D);
        px += kConvGroup * P.x_ts;
        if (sizeof(T) == 1) ps += (long long)kConvGroup * nblk;
        if constexpr (ASYNC) cp_async_commit();
    };
    fetch(0);
    if constexpr (ASYNC) {
#pragma unroll
        for (int g = 1; g < kConvRing - 1; ++g) fetch(g);
    }
    float2 w[W][2], bias[2], h[W - 1][2];           // h: the last W - 1 inputs, oldest first
    load_params<W, VEC>(P.weight, P.bias, blk, lane, D, w, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        float f[4];
        past(t0 - (W - 1) + j, f);
        pairs(f, h[j]);
    }
    for (int g = 0, t = t0; t < t1; ++g, t += kConvGroup) {
        const int left = t1 - t;
        float v[kConvGroup][4];
        if constexpr (ASYNC) {
            if (sizeof(T) == 1) __syncwarp();       // the scales of the group that goes were read by all lanes
            fetch(g + kConvRing - 1);
            cp_async_wait<kConvRing - 1>();
            if (sizeof(T) == 1) __syncwarp();       // and those of this one copied by some
            in.get(g, lane, v);
        } else {
            in.get(g, lane, v);
            fetch(g + 1);
        }
        if constexpr (SAVE) {
            uint32_t q[kConvGroup];
            float scale[kConvGroup];
            act8_encode_all(v, q, scale);
#pragma unroll
            for (int k = 0; k < kConvGroup; ++k) {
                if (k >= left) break;
                row_store_codes<VEC>(pc + (long long)k * D, blk, lane, D, q[k]);
                if (lane == 0) pq[(long long)k * nblk] = scale[k];
            }
            pc += (long long)kConvGroup * D;
            pq += (long long)kConvGroup * nblk;
        }
#pragma unroll
        for (int k = 0; k < kConvGroup; ++k) {
            float2 now[2];
            float o[4];
            pairs(v[k], now);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float2 p = __ffma2_rn(w[W - 1][i], now[i], bias[i]);
#pragma unroll
                for (int j = W - 2; j >= 0; --j) p = __ffma2_rn(w[j][i], h[j][i], p);
                if (P.silu) p = __fmul2_rn(p, sigmoid2<PRECISE>(p));
                o[2 * i] = p.x, o[2 * i + 1] = p.y;
#pragma unroll
                for (int j = 0; j < W - 2; ++j) h[j][i] = h[j + 1][i];
                h[W - 2][i] = now[i];
            }
            if (k < left) row_store<VEC>(py + (long long)k * D, blk, lane, D, o);
        }
        py += (long long)kConvGroup * D;
    }
}

// One token: a thread per channel, its W - 1 state values moved on in place.
template <typename T, typename YT, int W>
__global__ void __launch_bounds__(256)
conv_step_kernel(long long total, int D, const T *__restrict__ x, long long x_bs, const float *__restrict__ weight,
                 const float *__restrict__ bias, T *state, int silu, YT *__restrict__ y) {
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= total) return;
    const long long b = id / D;
    const int c = (int)(id % D);
    T *s = state + b * (W - 1) * D + c;
    T h[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) h[j] = s[(size_t)j * D];
    const T in = x[b * x_bs + c];
    float p = fmaf(__ldg(weight + (size_t)c * W + W - 1), to_f32(in), bias ? __ldg(bias + c) : 0.f);
#pragma unroll
    for (int j = W - 2; j >= 0; --j) p = fmaf(__ldg(weight + (size_t)c * W + j), to_f32(h[j]), p);
#pragma unroll
    for (int j = 0; j < W - 2; ++j) s[(size_t)j * D] = h[j + 1];
    s[(size_t)(W - 2) * D] = in;
    y[id] = from_f32<YT>(silu ? p * sigmoid<sizeof(YT) == 4>(p) : p);
}

constexpr int kConvBwdWarps = 4;    // backward: runs a block, joined in shared memory
constexpr int kConvBwdRun = 64;    // tokens a run

struct ConvBwd {
    int B, T, D;
    const void *x;
    long long x_bs, x_ts;
    const float *x_scales;
    const float *weight, *bias;
    const void *state, *dy;
    const float *dstate_out;
    int silu;
    void *dx;
    float *dstate;
    float *partial;                 // [B * groups][W + 1][D]
    int groups;                     // blocks of runs a sequence
};

// A warp's run of tokens [t0, t1): at token t it has p_t and dp_t, hence
// dx_{t-W+1} = sum_j w_j dp_{t-j}; W - 1 tokens behind the run give the rest.
template <typename T, typename ST, typename DT, typename GT, int W, bool VEC>
__global__ void __launch_bounds__(32 * kConvBwdWarps, VEC ? 3 : 2)
conv_bwd_kernel(const ConvBwd P) {
    constexpr bool PRECISE = sizeof(GT) == 4;
    __shared__ float part[kConvBwdWarps][W + 1][kBlk];
    extern __shared__ __align__(16) unsigned char conv_smem[];
    Stream<T, VEC> xin{conv_smem + (threadIdx.x >> 5) * Stream<T, VEC>::WARP_BYTES};
    Stream<DT, VEC> gin{conv_smem + kConvBwdWarps * Stream<T, VEC>::WARP_BYTES + (threadIdx.x >> 5) * Stream<DT, VEC>::WARP_BYTES};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = P.D, nblk = (D + kBlk - 1) / kBlk;
    const int blk = (int)(blockIdx.x % nblk);
    const long long rest = blockIdx.x / nblk;
    const int group = (int)(rest % P.groups);
    const long long b = rest / P.groups;
    const int t0 = min((group * kConvBwdWarps + warp) * kConvBwdRun, P.T), t1 = min(t0 + kConvBwdRun, P.T);
    const bool first = t0 == 0 && warp == 0 && group == 0;
    const T *x = static_cast<const T *>(P.x) + b * P.x_bs;
    const ST *state = static_cast<const ST *>(P.state);
    const DT *dy = static_cast<const DT *>(P.dy) + b * P.T * (long long)D;
    GT *dx = static_cast<GT *>(P.dx) + b * P.T * (long long)D;
    const float *xs = sizeof(T) == 1 ? P.x_scales + b * P.T * nblk + blk : nullptr;
    float2 w[W][2], bias[2], dw[W][2], db[2];
    load_params<W, VEC>(P.weight, P.bias, blk, lane, D, w, bias);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        db[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = make_float2(0.f, 0.f);
    }
    if (t0 < t1) {
        float2 h[W][2], dp[W][2];                   // x and dp at t - W + 1 .. t
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int t = t0 - W + j;               // shifted once before the first token
            float f[4] = {0.f, 0.f, 0.f, 0.f};
            if (j > 0 && t >= 0) {
                Token<T, VEC> k;
                k.load(x + t * P.x_ts, xs + (long long)t * nblk, blk, lane, D);
                k.get(f);
            } else if (j > 0 && state) {
                load4c<VEC>(state + (b * (W - 1) + (t + W - 1)) * D, blk, lane, D, f);
            }
            pairs(f, h[j]);
            dp[j][0] = dp[j][1] = make_float2(0.f, 0.f);
        }
        const int end = t1 + W - 1, last = min(end, P.T);       // tokens behind the sequence count as zero
        constexpr bool ASYNC = Stream<T, VEC>::ASYNC && Stream<DT, VEC>::ASYNC;
        constexpr bool MIXED = !ASYNC && (Stream<T, VEC>::ASYNC || Stream<DT, VEC>::ASYNC);
        static_assert(!MIXED || !VEC, "vector accesses stream both");
        const T *px = x + t0 * P.x_ts;
        const float *ps = xs + (long long)t0 * nblk;
        const DT *pg = dy + (long long)t0 * D;
        auto fetch = [&](int g) {
            const int t = t0 + g * kConvGroup;
            if (t < end) {
                xin.fetch(g, px, P.x_ts, ps, nblk, last - t, blk, lane, D);
                gin.fetch(g, pg, D, nullptr, 0, last - t, blk, lane, D);
            }
            px += kConvGroup * P.x_ts;
            pg += (long long)kConvGroup * D;
            if (sizeof(T) == 1) ps += (long long)kConvGroup * nblk;
            if constexpr (ASYNC || MIXED) cp_async_commit();
        };
        fetch(0);
        if constexpr (ASYNC) {
#pragma unroll
            for (int g = 1; g < kConvRing - 1; ++g) fetch(g);
        }
        // one token: its dp, the parameters' sums (SUM), and the gradient W - 1 tokens back
        auto token = [&](const float (&v)[4], const float (&g)[4], bool sum, float (&o)[4]) {
            float2 in[2], e[2];
            pairs(v, in);
            pairs(g, e);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) h[j][i] = h[j + 1][i], dp[j][i] = dp[j + 1][i];
                h[W - 1][i] = in[i];
                if (P.silu) {
                    float2 p = bias[i];
#pragma unroll
                    for (int j = W - 1; j >= 0; --j) p = __ffma2_rn(w[j][i], h[j][i], p);
                    const float2 one = make_float2(1.f, 1.f), sg = sigmoid2<PRECISE>(p);
                    const float2 rest = __ffma2_rn(sg, make_float2(-1.f, -1.f), one);
                    e[i] = __fmul2_rn(__fmul2_rn(e[i], sg), __ffma2_rn(p, rest, one));
                }
                dp[W - 1][i] = e[i];
                if (sum) {
                    db[i] = __fadd2_rn(db[i], e[i]);
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[j][i] = __ffma2_rn(e[i], h[j][i], dw[j][i]);
                }
                float2 d = __fmul2_rn(w[0][i], dp[W - 1][i]);
#pragma unroll
                for (int j = 1; j < W; ++j) d = __ffma2_rn(w[j][i], dp[W - 1 - j][i], d);
                o[2 * i] = d.x, o[2 * i + 1] = d.y;
            }
        };
        for (int g = 0, tt = t0; tt < end; ++g, tt += kConvGroup) {
            float xv[kConvGroup][4], gv[kConvGroup][4];
            if constexpr (ASYNC) {
                if (sizeof(T) == 1) __syncwarp();
                fetch(g + kConvRing - 1);
                cp_async_wait<kConvRing - 1>();
                if (sizeof(T) == 1) __syncwarp();
            } else if constexpr (MIXED) {
                cp_async_wait<0>();
            }
            xin.get(g, lane, xv);
            gin.get(g, lane, gv);
            if constexpr (!ASYNC) fetch(g + 1);
            const bool states = (first && P.dstate && g == 0) || (P.dstate_out && tt + kConvGroup > P.T - (W - 1));
            if (!states) {
                GT *to = dx + ((long long)tt - (W - 1)) * D;
                if (g > 0 && tt + kConvGroup <= t1) {
#pragma unroll
                    for (int k = 0; k < kConvGroup; ++k) {
                        float o[4];
                        token(xv[k], gv[k], true, o);
                        row_store<VEC>(to + (long long)k * D, blk, lane, D, o);
                    }
                } else {                                    // a run's first and last tokens
#pragma unroll
                    for (int k = 0; k < kConvGroup; ++k) {
                        float o[4];
                        token(xv[k], gv[k], tt + k < t1, o);
                        if (tt + k - (W - 1) >= t0 && tt + k < end) row_store<VEC>(to + (long long)k * D, blk, lane, D, o);
                    }
                }
                continue;
            }
#pragma unroll 1
            for (int k = 0; k < kConvGroup; ++k) {          // where the states' gradients come in
                const int t = tt + k;
                if (t >= end) break;
                float o[4], xk[4], gk[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    xk[i] = xv[0][i], gk[i] = gv[0][i];
#pragma unroll
                    for (int m = 1; m < kConvGroup; ++m)
                        if (k == m) xk[i] = xv[m][i], gk[i] = gv[m][i];
                }
                token(xk, gk, t < t1, o);
                const int at = t - (W - 1);         // the token whose gradient is complete
                const int row = at - (P.T - (W - 1));
                if (P.dstate_out && row >= 0) {     // it is in state_out as well
                    float f[4];
                    load4c<VEC>(P.dstate_out + (b * (W - 1) + row) * D, blk, lane, D, f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] += f[i];
                }
                if (at >= t0) row_store<VEC>(dx + (long long)at * D, blk, lane, D, o);
                else if (first && P.dstate) row_store<VEC>(P.dstate + (b * (W - 1) + at + W - 1) * D, blk, lane, D, o);
            }
        }
    }
    // the block's runs, in order
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = lane_channel<VEC>(0, lane, i);
#pragma unroll
        for (int j = 0; j < W; ++j) part[warp][j][c] = (i & 1) ? dw[j][i / 2].y : dw[j][i / 2].x;
        part[warp][W][c] = (i & 1) ? db[i / 2].y : db[i / 2].x;
    }
    __syncthreads();
    float *out = P.partial + (b * P.groups + group) * (W + 1) * (long long)D;
    for (int e = threadIdx.x; e < (W + 1) * kBlk; e += blockDim.x) {
        const int j = e / kBlk, c = e % kBlk;
        if (blk * kBlk + c >= D) continue;
        float a = part[0][j][c];
#pragma unroll
        for (int k = 1; k < kConvBwdWarps; ++k) a += part[k][j][c];
        out[(long long)j * D + blk * kBlk + c] = a;
    }
}

// [W + 1][D] sums -> dweight [D][W] and dbias [D]
__global__ void conv_params_kernel(int D, int W, const float *__restrict__ sums, float *__restrict__ dweight,
                                   float *__restrict__ dbias) {
    const int e = blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= D * (W + 1)) return;
    const int j = e / D, c = e % D;
    if (j < W) dweight[(size_t)c * W + j] = sums[e];
    else if (dbias) dbias[c] = sums[e];
}

wkv7_status conv_dims(int B, int T, int D, int W) {
    if (B < 0 || T < 0 || D < 0 || W <= 0) return WKV7_ERR_INVALID_ARG;
    if (W < 2 || W > 4 || D > WKV7_SSM_MAX_D || T > kMaxTokens) return WKV7_ERR_UNSUPPORTED;
    const long long runs = ((long long)T + kConvMinRun - 1) / kConvMinRun + 1;
    // blocks of a launch, and of the step's
    if ((double)B * runs * blocks_of(D) > (double)kMaxGrid) return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}

// Tokens a run: the fewer, the more a run's start (W - 1 tokens again, the weights)
// costs, so 64 where that makes 12 warps an SM (8 x 4096 x 2048: 52 us; 68 us at
// 32), else 32 or 16.
int conv_run(int B, int T, int D) {
    const long long want = 12ll * sm_count();
    int run = 64;
    while (run > kConvMinRun && (long long)B * ((T + run - 1) / run) * blocks_of(D) < want) run /= 2;
    return run;
}

int conv_groups(int T) {
    const int per = kConvBwdWarps * kConvBwdRun;
    return (int)(((long long)T + per - 1) / per);
}

// width as a template argument, then the rest of the launch
template <typename F> void by_width(int W, F &&f) {
    if (W == 2) f(std::integral_constant<int, 2>{});
    else if (W == 3) f(std::integral_constant<int, 3>{});
    else f(std::integral_constant<int, 4>{});
}

// a kernel's dynamic shared memory, with leave to use it where it is large
template <typename K, typename P>
void conv_launch(K kernel, const P &p, unsigned grid, int threads, size_t smem, cudaStream_t st) {
    if (smem > 32 * 1024) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    kernel<<<grid, threads, smem, st>>>(p);
}

template <typename T, typename ST, typename YT, bool SAVE>
void launch_conv_fwd(const ConvFwd &P, int W, bool vec, cudaStream_t st) {
    const long long units = (long long)P.B * P.runs * blocks_of(P.D);
    const unsigned grid = (unsigned)((units + kConvWarps - 1) / kConvWarps);
    by_width(W, [&](auto w) {
        constexpr int WW = decltype(w)::value, th = 32 * kConvWarps;
        if (vec) conv_launch(conv_fwd_kernel<T, ST, YT, WW, true, SAVE>, P, grid, th, kConvWarps * Stream<T, true>::WARP_BYTES, st);
        else conv_launch(conv_fwd_kernel<T, ST, YT, WW, false, SAVE>, P, grid, th, kConvWarps * Stream<T, false>::WARP_BYTES, st);
    });
}

template <typename T, typename ST, typename DT, typename GT>
void launch_conv_bwd(const ConvBwd &P, int W, bool vec, cudaStream_t st) {
    const unsigned grid = (unsigned)((long long)P.B * P.groups * blocks_of(P.D));
    by_width(W, [&](auto w) {
        constexpr int WW = decltype(w)::value, th = 32 * kConvBwdWarps;
        if (vec)
            conv_launch(conv_bwd_kernel<T, ST, DT, GT, WW, true>, P, grid, th,
                        kConvBwdWarps * (Stream<T, true>::WARP_BYTES + Stream<DT, true>::WARP_BYTES), st);
        else
            conv_launch(conv_bwd_kernel<T, ST, DT, GT, WW, false>, P, grid, th,
                        kConvBwdWarps * (Stream<T, false>::WARP_BYTES + Stream<DT, false>::WARP_BYTES), st);
    });
}

}  // namespace
}  // namespace mixer
}  // namespace wkv7

extern "C" {

wkv7_status wkv7_conv_forward(int B, int T, int D, int W, wkv7_dtype x_dt, wkv7_dtype y_dt, const void *x,
                              long long x_bs, long long x_ts, const float *x_scales, const float *weight,
                              const float *bias, const void *state, const int *lens, int silu, void *y,
                              void *state_out, void *codes, float *scales, cudaStream_t stream) {
    using namespace wkv7::mixer;
    const wkv7_status st = conv_dims(B, T, D, W);
    if (st != WKV7_OK) return st;
    const bool q8 = x_dt == WKV7_E4M3;
    if (!(real_dtype(x_dt) || q8) || !real_dtype(y_dt) || x_bs < 0 || x_ts < 0) return WKV7_ERR_INVALID_ARG;
    if ((codes != nullptr) != (scales != nullptr)) return WKV7_ERR_INVALID_ARG;
    if ((q8 || lens) && codes) return WKV7_ERR_INVALID_ARG;
    if (q8 && state_out) return WKV7_ERR_INVALID_ARG;
    if (state_out && state_out == state) return WKV7_ERR_INVALID_ARG;
    if (B == 0 || D == 0) return WKV7_OK;
    const wkv7_dtype s_dt = q8 ? y_dt : x_dt;
    if (T > 0 && (!elem_ok(x, x_dt) || !elem_ok(y, y_dt))) return WKV7_ERR_INVALID_ARG;
    if (q8 != (x_scales != nullptr) || !f32_opt(x_scales)) return WKV7_ERR_INVALID_ARG;
    if (!f32_ok(weight) || !f32_opt(bias) || !f32_opt(scales) || !aligned_to(lens, 4) ||
        !aligned_to(state, dtype_size(s_dt)) || !aligned_to(state_out, dtype_size(s_dt)))
        return WKV7_ERR_INVALID_ARG;
    if (T == 0 && !state_out) return WKV7_OK;
    if (T > 0 && y == x) return WKV7_ERR_INVALID_ARG;       // a run reads W - 1 tokens of the run before
    if (q8) x_bs = (long long)T * D, x_ts = D;
    const int run = conv_run(B, T, D), runs = T > 0 ? (T + run - 1) / run : 1;      // T = 0: the state alone
    const ConvFwd P{B, T, D, x, x_bs, x_ts, x_scales, weight, bias, state, lens, silu, y, state_out,
                    (uint8_t *)codes, scales, runs, run};
    const bool vec = D % 4 == 0 && x_bs % 4 == 0 && x_ts % 4 == 0 && aligned_to(x, 4 * dtype_size(x_dt)) &&
                     aligned_to(y, 4 * dtype_size(y_dt)) && aligned_to(state, 4 * dtype_size(s_dt)) &&
                     aligned_to(state_out, 4 * dtype_size(s_dt)) && aligned_to(codes, 4) && aligned_to(weight, 16) &&
                     aligned_to(bias, 16);
    const bool yf = y_dt == WKV7_F32;
    if (q8) {
        if (yf) launch_conv_fwd<e4m3, float, float, false>(P, W, vec, stream);
        else launch_conv_fwd<e4m3, bf16, bf16, false>(P, W, vec, stream);
    } else if (x_dt == WKV7_F32) {
        if (codes) {
            if (yf) launch_conv_fwd<float, float, float, true>(P, W, vec, stream);
            else launch_conv_fwd<float, float, bf16, true>(P, W, vec, stream);
        } else {
            if (yf) launch_conv_fwd<float, float, float, false>(P, W, vec, stream);
            else launch_conv_fwd<float, float, bf16, false>(P, W, vec, stream);
        }
    } else {
        if (codes) {
            if (yf) launch_conv_fwd<bf16, bf16, float, true>(P, W, vec, stream);
            else launch_conv_fwd<bf16, bf16, bf16, true>(P, W, vec, stream);
        } else {
            if (yf) launch_conv_fwd<bf16, bf16, float, false>(P, W, vec, stream);
            else launch_conv_fwd<bf16, bf16, bf16, false>(P, W, vec, stream);
        }
    }
    return launch_status();
}

wkv7_status wkv7_conv_step(int B, int D, int W, wkv7_dtype x_dt, wkv7_dtype y_dt, const void *x, long long x_bs,
                           const float *weight, const float *bias, void *state, int silu, void *y,
                           cudaStream_t stream) {
    using namespace wkv7::mixer;
    const wkv7_status st = conv_dims(B, 1, D, W);
    if (st != WKV7_OK) return st;
    if (!real_dtype(x_dt) || !real_dtype(y_dt) || x_bs < 0) return WKV7_ERR_INVALID_ARG;
    if (B == 0 || D == 0) return WKV7_OK;
    if (!elem_ok(x, x_dt) || !elem_ok(y, y_dt) || !elem_ok(state, x_dt) || !f32_ok(weight) || !f32_opt(bias))
        return WKV7_ERR_INVALID_ARG;
    const long long total = (long long)B * D;
    const unsigned grid = (unsigned)((total + 255) / 256);
    by_width(W, [&](auto w) {
        constexpr int WW = decltype(w)::value;
#define WKV7_STEP(I, O)                                                                                        \
    conv_step_kernel<I, O, WW><<<grid, 256, 0, stream>>>(total, D, (const I *)x, x_bs, weight, bias, (I *)state, \
                                                         silu, (O *)y)
        if (x_dt == WKV7_F32 && y_dt == WKV7_F32) WKV7_STEP(float, float);
        else if (x_dt == WKV7_F32) WKV7_STEP(float, bf16);
        else if (y_dt == WKV7_F32) WKV7_STEP(bf16, float);
        else WKV7_STEP(bf16, bf16);
#undef WKV7_STEP
    });
    return launch_status();
}

size_t wkv7_conv_backward_workspace_size(int B, int T, int D, int W) {
    using namespace wkv7::mixer;
    if (B <= 0 || T <= 0 || D <= 0 || conv_dims(B, T, D, W) != WKV7_OK) return 0;
    const size_t cols = (size_t)D * (W + 1);
    return round256((size_t)B * conv_groups(T) * cols * sizeof(float)) + round256(cols * sizeof(float));
}

wkv7_status wkv7_conv_backward(int B, int T, int D, int W, wkv7_dtype x_dt, wkv7_dtype dy_dt, wkv7_dtype g_dt,
                               const void *x, long long x_bs, long long x_ts, const float *x_scales,
                               const float *weight, const float *bias, const void *state, const void *dy,
                               const float *dstate_out, int silu, void *dx, float *dweight, float *dbias,
                               float *dstate, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace wkv7::mixer;
    const wkv7_status st = conv_dims(B, T, D, W);
    if (st != WKV7_OK) return st;
    const bool q8 = x_dt == WKV7_E4M3;
    if (!(real_dtype(x_dt) || q8) || !real_dtype(dy_dt) || !real_dtype(g_dt) || x_bs < 0 || x_ts < 0)
        return WKV7_ERR_INVALID_ARG;
    if (D == 0) return WKV7_OK;
    if (!f32_ok(dweight) || !f32_opt(dbias) || !f32_opt(dstate) || !f32_opt(dstate_out)) return WKV7_ERR_INVALID_ARG;
    if (B == 0 || T == 0) {
        if (cudaMemsetAsync(dweight, 0, (size_t)D * W * 4, stream) != cudaSuccess) return WKV7_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)D * 4, stream) != cudaSuccess) return WKV7_ERR_CUDA;
        const size_t n = (size_t)B * (W - 1) * D * 4;       // without a token state_out is state
        if (dstate && n && dstate != dstate_out) {
            const cudaError_t e = dstate_out ? cudaMemcpyAsync(dstate, dstate_out, n, cudaMemcpyDeviceToDevice, stream)
                                             : cudaMemsetAsync(dstate, 0, n, stream);
            if (e != cudaSuccess) return WKV7_ERR_CUDA;
        }
        return WKV7_OK;
    }
    const wkv7_dtype s_dt = q8 ? g_dt : x_dt;
    if (!elem_ok(x, x_dt) || !elem_ok(dy, dy_dt) || !elem_ok(dx, g_dt) || !f32_ok(weight) || !f32_opt(bias) ||
        q8 != (x_scales != nullptr) || !f32_opt(x_scales) || !aligned_to(state, dtype_size(s_dt)))
        return WKV7_ERR_INVALID_ARG;
    if (dstate && dstate == dstate_out) return WKV7_ERR_INVALID_ARG;
    if (dx == dy || dx == x) return WKV7_ERR_INVALID_ARG;   // runs read W - 1 tokens of their neighbours
    if (workspace == nullptr || !aligned_to(workspace, 16) ||
        workspace_bytes < wkv7_conv_backward_workspace_size(B, T, D, W))
        return WKV7_ERR_INVALID_ARG;
    if (q8) x_bs = (long long)T * D, x_ts = D;
    const int groups = conv_groups(T);
    const size_t cols = (size_t)D * (W + 1);
    float *partial = (float *)workspace;
    float *sums = (float *)((char *)workspace + round256((size_t)B * groups * cols * sizeof(float)));
    const ConvBwd P{B, T, D, x, x_bs, x_ts, x_scales, weight, bias, state, dy, dstate_out, silu, dx, dstate, partial,
                    groups};
    const bool vec = D % 4 == 0 && x_bs % 4 == 0 && x_ts % 4 == 0 && aligned_to(x, 4 * dtype_size(x_dt)) &&
                     aligned_to(dy, 4 * dtype_size(dy_dt)) && aligned_to(dx, 4 * dtype_size(g_dt)) &&
                     aligned_to(state, 4 * dtype_size(s_dt)) && aligned_to(dstate, 16) && aligned_to(dstate_out, 16) &&
                     aligned_to(weight, 16) && aligned_to(bias, 16);
    const bool df = dy_dt == WKV7_F32, gf = g_dt == WKV7_F32;
#define WKV7_BWD(T, ST, DT, GT) launch_conv_bwd<T, ST, DT, GT>(P, W, vec, stream)
    if (q8) {
        if (df && gf) WKV7_BWD(e4m3, float, float, float);
        else if (df) WKV7_BWD(e4m3, bf16, float, bf16);
        else if (gf) WKV7_BWD(e4m3, float, bf16, float);
        else WKV7_BWD(e4m3, bf16, bf16, bf16);
    } else if (x_dt == WKV7_F32) {
        if (df && gf) WKV7_BWD(float, float, float, float);
        else if (df) WKV7_BWD(float, float, float, bf16);
        else if (gf) WKV7_BWD(float, float, bf16, float);
        else WKV7_BWD(float, float, bf16, bf16);
    } else {
        if (df && gf) WKV7_BWD(bf16, bf16, float, float);
        else if (df) WKV7_BWD(bf16, bf16, float, bf16);
        else if (gf) WKV7_BWD(bf16, bf16, bf16, float);
        else WKV7_BWD(bf16, bf16, bf16, bf16);
    }
#undef WKV7_BWD
    sum_parts((long long)B * groups, (long long)cols, partial, sums, stream);
    conv_params_kernel<<<(unsigned)((cols + 255) / 256), 256, 0, stream>>>(D, W, sums, dweight, dbias);
    return launch_status();
}

}  // extern "C"
