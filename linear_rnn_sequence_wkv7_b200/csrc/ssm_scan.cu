// Selective state-space scan, forward: whole sequences (wkv7_ssm_forward) and
// single tokens (wkv7_ssm_step).
//
//     dt = softplus(delta + bias),  h <- exp(dt A) h + dt u B,  y = (C . h + D u) z sigmoid(z)
//
// Bound: one exponential per (token, channel, n).  At N = 16 a channel-token
// moves 8 bytes but takes 16 exponentials, and an SM makes 16 a cycle; the
// state's update and readout (64 multiply-adds) stay below that.
//
// Mapping: a thread holds 2 channels x 4 n of the state in registers; LN = 2,
// 4, 8 or 16 lanes side by side share a channel pair (N up to 8, 16, 32, 64,
// the rest padded with zero rates and inputs, which keep a zero state at zero).
// A tile of 16 tokens is prepared by the whole block (softplus and dt u once per
// channel, not once per n) into shared memory, walked token by token, and its
// outputs, joined over the LN lanes by shuffles, are gated by the threads that
// loaded u and z.  Loads of the next tile are in flight meanwhile.
//
// Few channels over many tokens: the state map of a stretch of tokens is
// h -> exp(A sum dt) h + E, so the sequence is cut into segments: one pass takes
// every segment's E (from a zero state, no output) and sum dt, a chain gives the
// entry states, and the outputs come from a second pass over all segments.
#include <type_traits>

#include "mixer.cuh"
#include "ssm.cuh"

namespace wkv7 {
namespace mixer {
namespace {

template <typename T, int LN, int V, bool Y>
__global__ void __launch_bounds__(kScanThreads)
ssm_fwd_kernel(const ScanArgs P) {
    constexpr int CC = scan_channels(LN), NP = 4 * LN;          // channels a block, padded N
    constexpr int EPT = kTile * CC / kScanThreads, Q = EPT / V; // a thread's share of a tile, in Q vectors
    constexpr int NB = kTile * NP / kScanThreads;               // and of B (and C)
    constexpr bool PRECISE = sizeof(T) == 4;
    __shared__ __align__(16) float s_dt[kTile][CC], s_du[kTile][CC], s_y[Y ? kTile : 1][CC];
    __shared__ float4 s_B[kTile][LN], s_C[Y ? kTile : 1][LN];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long id = blockIdx.x;
    const int tile_c = (int)(id % P.tiles);
    id /= P.tiles;
    const int g = (int)(id % P.G);
    id /= P.G;
    const long long b = id % P.B;
    const int seg = (int)(id / P.B);
    const int c0 = g * P.Dg + tile_c * CC, c1 = (g + 1) * P.Dg;     // the block's channels [c0, min(c0 + CC, c1))
    int len = P.T;
    if (P.lens) len = min(max(__ldg(P.lens + b), 0), P.T);
    const int t0 = (int)min((long long)seg * P.seg_len, (long long)len);
    const int t1 = (int)min((long long)t0 + P.seg_len, (long long)len);

    // this thread's channels when it loads: V in a row, the same in each of its Q vectors
    const int lc = c0 + (tid % (CC / V)) * V, lt = tid / (CC / V);
    const bool live = lc < c1;
    float bias[V], skip[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = (live && P.dt_bias) ? __ldg(P.dt_bias + lc + i) : 0.f;
        skip[i] = (Y && live && P.Dskip) ? __ldg(P.Dskip + lc + i) : 0.f;
    }
    const T *u = static_cast<const T *>(P.u) + b * P.u_bs + lc, *de = static_cast<const T *>(P.delta) + b * P.d_bs + lc;
    const T *z = (Y && P.z) ? static_cast<const T *>(P.z) + b * P.z_bs + lc : nullptr;
    const T *Bm = static_cast<const T *>(P.Bm) + b * P.b_bs + g * P.N;
    const T *Cm = static_cast<const T *>(P.Cm) + b * P.c_bs + g * P.N;

    // and when it scans: channels cs, cs + 1 and n = ns .. ns + 3
    const int nl = lane % LN, cl = (warp * (32 / LN) + lane / LN) * 2, cs = c0 + cl, ns = 4 * nl;
    float2 a2[2][2], h[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float av[4], hv[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const bool in = cs + c < c1 && ns + n < P.N;
            av[n] = in ? __ldg(P.A + (size_t)(cs + c) * P.N + ns + n) * kLog2e : 0.f;
            hv[n] = (in && P.entry) ? P.entry[(((size_t)seg * P.B + b) * P.D + cs + c) * P.N + ns + n] : 0.f;
        }
        a2[c][0] = make_float2(av[0], av[1]), a2[c][1] = make_float2(av[2], av[3]);
        h[c][0] = make_float2(hv[0], hv[1]), h[c][1] = make_float2(hv[2], hv[3]);
    }
    double sum0 = 0, sum1 = 0;                      // of dt, when summarising

    Vec<T, V> nu[Q], nd[Q], nz[Q], cu[Q], cz[Q];
    Vec<T, 1> nb[NB], nc[NB];
    auto fetch = [&](int t) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int tt = t + lt + q * (kTile / Q);
            nu[q].zero(), nd[q].zero(), nz[q].zero();
            if (live && tt < t1) {
                nu[q].load(u + tt * P.u_ts);
                nd[q].load(de + tt * P.d_ts);
                if (z) nz[q].load(z + tt * P.z_ts);
            }
        }
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int e = tid + q * kScanThreads, tt = t + e / NP, n = e % NP;
            nb[q].zero(), nc[q].zero();
            if (tt < t1 && n < P.N) {
                nb[q].load(Bm + tt * P.b_ts + n);
                if (Y) nc[q].load(Cm + tt * P.c_ts + n);
            }
        }
    };
    auto prepare = [&](int t) {         // tokens behind t1: dt = dt u = B = 0 keep the state
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int k = lt + q * (kTile / Q), ch = lc - c0;
            float fu[V], fd[V];
            nu[q].get(fu), nd[q].get(fd);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float x = fd[i] + bias[i], dt = (live && t + k < t1) ? (P.softplus ? softplus(x) : x) : 0.f;
                fu[i] = dt != 0.f ? dt * fu[i] : 0.f;
                fd[i] = dt;
            }
            storev<V>(&s_dt[k][ch], fd);
            storev<V>(&s_du[k][ch], fu);
            cu[q] = nu[q], cz[q] = nz[q];
        }
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int e = tid + q * kScanThreads;
            float f[1];
            nb[q].get(f);
            reinterpret_cast<float *>(s_B)[e] = f[0];
            if (Y) {
                nc[q].get(f);
                reinterpret_cast<float *>(s_C)[e] = f[0];
            }
        }
    };

    fetch(t0);
    prepare(t0);
    __syncthreads();
    for (int t = t0; t < t1; t += kTile) {
        if (t + kTile < t1) fetch(t + kTile);
        if (P.states) {
            float *to = P.states + ((size_t)(b * P.nck + t / kTile) * P.D + cs) * P.N + ns;
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (cs + c < c1) store_state(to + (size_t)c * P.N, P.N, ns, h[c]);
        }
        const int count = min(kTile, t1 - t);
        float part0 = 0.f, part1 = 0.f;
#pragma unroll 1
        for (int k = 0; k < count; k += 2) {
            float yv[4];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const float2 dt = *reinterpret_cast<const float2 *>(&s_dt[k + kk][cl]);
                const float2 du = *reinterpret_cast<const float2 *>(&s_du[k + kk][cl]);
                const float4 B = s_B[k + kk][nl];
                const float2 B0 = make_float2(B.x, B.y), B1 = make_float2(B.z, B.w);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float d = c ? dt.y : dt.x, w = c ? du.y : du.x;
                    const float2 d2 = make_float2(d, d), w2 = make_float2(w, w);
                    h[c][0] = __ffma2_rn(ex2(__fmul2_rn(d2, a2[c][0])), h[c][0], __fmul2_rn(w2, B0));
                    h[c][1] = __ffma2_rn(ex2(__fmul2_rn(d2, a2[c][1])), h[c][1], __fmul2_rn(w2, B1));
                }
                if constexpr (Y) {
                    const float4 C = s_C[k + kk][nl];
                    const float2 C0 = make_float2(C.x, C.y), C1 = make_float2(C.z, C.w);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float2 p = __ffma2_rn(h[c][0], C0, __fmul2_rn(h[c][1], C1));
                        yv[2 * kk + c] = p.x + p.y;
                    }
                } else {
                    part0 += dt.x, part1 += dt.y;
                }
            }
            if constexpr (Y) {          // 2 tokens x 2 channels over LN lanes
                reduce_scatter<LN, 4>(yv, nl);
                if constexpr (LN == 2) {
                    s_y[k][cl + nl] = yv[0];
                    s_y[k + 1][cl + nl] = yv[1];
                } else if (nl < 4) {
                    s_y[k + (nl >> 1)][cl + (nl & 1)] = yv[0];
                }
            }
        }
        if constexpr (!Y) sum0 += part0, sum1 += part1;
        __syncthreads();
        if constexpr (Y) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int k = lt + q * (kTile / Q);
                if (!live || t + k >= t1) continue;
                float f[V], fu[V], fz[V];
                cu[q].get(fu), cz[q].get(fz);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    f[i] = fmaf(skip[i], fu[i], s_y[k][lc - c0 + i]);
                    if (z) f[i] *= fz[i] * sigmoid<PRECISE>(fz[i]);
                }
                const size_t at = ((size_t)b * P.T + t + k) * P.D + lc;
                if (P.y_f32) storev<V>(static_cast<float *>(P.y) + at, f);
                else storev<V>(static_cast<bf16 *>(P.y) + at, f);
            }
        }
        if (t + kTile < t1) prepare(t + kTile);
        __syncthreads();
    }
    if (seg == P.nseg - 1 && P.stateT)
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (cs + c < c1) store_state(P.stateT + ((size_t)b * P.D + cs + c) * P.N + ns, P.N, ns, h[c]);
    if (!Y && P.seg_end) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (cs + c >= c1) continue;
            const size_t at = ((size_t)seg * P.B + b) * P.D + cs + c;
            store_state(P.seg_end + at * P.N + ns, P.N, ns, h[c]);
            if (nl == 0) P.seg_dt[at] = (float)(c ? sum1 : sum0);
        }
    }
}

// Entry states of the segments, in place of their end states: a thread per (b, d, n).
__global__ void __launch_bounds__(256)
ssm_chain_kernel(long long total, int N, int nseg, const float *__restrict__ A, long long D,
                 const float *__restrict__ state0, const float *__restrict__ seg_dt, float *__restrict__ seg_end) {
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= total) return;
    const long long ch = id / N;
    const float a = __ldg(A + (ch % D) * N + id % N) * kLog2e;
    float h = state0 ? state0[id] : 0.f;
    const long long chans = total / N;
    for (int s = 0; s < nseg; ++s) {
        const float e = seg_end[s * total + id];
        seg_end[s * total + id] = h;
        h = fmaf(ex2(a * __ldg(seg_dt + s * chans + ch)), h, e);
    }
}

// One token: LN lanes a channel, 4 n a lane.  Bound by the state's read and
// write, 8 bytes an n.
struct StepArgs {
    long long total;                // B * D
    int D, N, G, Dg;
    const void *u, *delta, *Bm, *Cm, *z;
    long long u_bs, d_bs, b_bs, c_bs, z_bs;
    const float *A, *Dskip, *dt_bias;
    float *state;
    int softplus;
    void *y;
};

template <typename T, typename YT, int LN, bool VEC>
__global__ void __launch_bounds__(256)
ssm_step_kernel(const StepArgs P) {
    constexpr bool PRECISE = sizeof(YT) == 4;
    const long long ch = ((long long)blockIdx.x * 256 + threadIdx.x) / LN;
    const int nl = threadIdx.x % LN, ns = 4 * nl;
    if (ch >= P.total) return;                  // LN lanes leave together
    const long long b = ch / P.D;
    const int d = (int)(ch % P.D), g = d / P.Dg;
    float *S = P.state + (size_t)ch * P.N + ns;
    const float *A = P.A + (size_t)d * P.N + ns;
    float h[4], a[4], Bv[4], Cv[4];
    const T *Bm = static_cast<const T *>(P.Bm) + b * P.b_bs + g * P.N + ns;
    const T *Cm = static_cast<const T *>(P.Cm) + b * P.c_bs + g * P.N + ns;
    if constexpr (VEC) {                        // N = 4 LN
        const float4 s4 = __ldcs(reinterpret_cast<const float4 *>(S)), a4 = __ldg(reinterpret_cast<const float4 *>(A));
        h[0] = s4.x, h[1] = s4.y, h[2] = s4.z, h[3] = s4.w;
        a[0] = a4.x, a[1] = a4.y, a[2] = a4.z, a[3] = a4.w;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const bool in = VEC || ns + n < P.N;
        if constexpr (!VEC) h[n] = in ? S[n] : 0.f, a[n] = in ? __ldg(A + n) : 0.f;
        Bv[n] = in ? to_f32(Bm[n]) : 0.f;
        Cv[n] = in ? to_f32(Cm[n]) : 0.f;
    }
    const float u = to_f32(static_cast<const T *>(P.u)[b * P.u_bs + d]);
    const float x = to_f32(static_cast<const T *>(P.delta)[b * P.d_bs + d]) + (P.dt_bias ? __ldg(P.dt_bias + d) : 0.f);
    const float dt = P.softplus ? softplus(x) : x, du = dt * u;
    float y = 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        h[n] = fmaf(ex2(dt * (a[n] * kLog2e)), h[n], du * Bv[n]);
        y = fmaf(h[n], Cv[n], y);
    }
    if constexpr (VEC) __stcs(reinterpret_cast<float4 *>(S), make_float4(h[0], h[1], h[2], h[3]));
    else {
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (ns + n < P.N) S[n] = h[n];
    }
    const unsigned group = ((LN == 32 ? 0u : (1u << LN)) - 1u) << (threadIdx.x & 31 & ~(LN - 1));
#pragma unroll
    for (int o = 1; o < LN; o <<= 1) y += __shfl_xor_sync(group, y, o);
    if (nl == 0) {
        if (P.Dskip) y = fmaf(__ldg(P.Dskip + d), u, y);
        if (P.z) {
            const float z = to_f32(static_cast<const T *>(P.z)[b * P.z_bs + d]);
            y *= z * sigmoid<PRECISE>(z);
        }
        static_cast<YT *>(P.y)[ch] = from_f32<YT>(y);
    }
}

template <typename T, int LN, bool Y>
void launch_fwd(const ScanArgs &P, bool vec, cudaStream_t st) {
    constexpr int CC = scan_channels(LN), EPT = kTile * CC / kScanThreads, V = EPT < 8 ? EPT : 8;
    const unsigned grid = (unsigned)((long long)P.nseg * P.B * P.G * P.tiles);
    if (vec) ssm_fwd_kernel<T, LN, V, Y><<<grid, kScanThreads, 0, st>>>(P);
    else ssm_fwd_kernel<T, LN, 1, Y><<<grid, kScanThreads, 0, st>>>(P);
}

}  // namespace

// Segments of a forward over B sequences: enough that its blocks fill the SMs,
// if that makes at least three of them (each token is then scanned twice), each
// of at least 128 tokens.
int ssm_segments(int B, int T, int D, int N, int G, int sms) {
    const int CC = scan_channels(scan_lanes(N)), tiles = G > 0 ? (D / G + CC - 1) / CC : 0;
    const long long blocks = (long long)B * G * tiles;
    if (blocks <= 0 || sms <= 0) return 1;
    const long long want = (long long)sms * 4 / blocks;
    const long long most = T / 128;
    const long long s = want < most ? want : most;
    return s >= 3 ? (int)s : 1;
}

void ssm_fwd(const ScanArgs &P, wkv7_dtype dt, bool vec, bool y, cudaStream_t st) {
    by_lanes(scan_lanes(P.N), [&](auto ln) {
        constexpr int LN = decltype(ln)::value;
        if (dt == WKV7_F32) {
            if (y) launch_fwd<float, LN, true>(P, vec, st);
            else launch_fwd<float, LN, false>(P, vec, st);
        } else {
            if (y) launch_fwd<bf16, LN, true>(P, vec, st);
            else launch_fwd<bf16, LN, false>(P, vec, st);
        }
    });
}

// The forward in P's segments: with one, from state0 directly; with more, the
// segments' summaries and entry states first (in `ws`).
void ssm_fwd_all(ScanArgs P, const float *state0, int nseg, char *ws, wkv7_dtype dt, bool vec, bool y,
                 cudaStream_t st) {
    P.nseg = nseg;
    P.seg_len = (int)((((long long)P.T + nseg - 1) / nseg + kTile - 1) / kTile * kTile);
    P.entry = state0;
    if (nseg > 1) {
        const long long total = (long long)P.B * P.D * P.N;
        ScanArgs S = P;
        S.entry = nullptr, S.states = nullptr, S.stateT = nullptr;
        S.seg_end = (float *)ws;
        S.seg_dt = (float *)(ws + round256((size_t)nseg * total * sizeof(float)));
        ssm_fwd(S, dt, vec, false, st);
        ssm_chain_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(total, P.N, nseg, P.A, P.D, state0, S.seg_dt,
                                                                         S.seg_end);
        P.entry = S.seg_end;
    }
    ssm_fwd(P, dt, vec, y, st);
}

size_t ssm_segment_bytes(int B, int D, int N, int nseg) {
    if (nseg <= 1) return 0;
    const size_t ch = (size_t)nseg * B * D;
    return round256(ch * N * sizeof(float)) + round256(ch * sizeof(float));
}

wkv7_status ssm_dims(int B, int T, int D, int N, int G) {
    if (B < 0 || T < 0 || D < 0 || N <= 0 || G <= 0) return WKV7_ERR_INVALID_ARG;
    if (D % G != 0) return WKV7_ERR_INVALID_ARG;
    if (N > 64 || D > WKV7_SSM_MAX_D || T > kMaxTokens) return WKV7_ERR_UNSUPPORTED;
    // blocks of the largest launch: a channel a block at most 16 channels wide, times the segments
    const double chans = (double)B * (D + 16.0 * G);
    if (chans * 64 / 256 > (double)kMaxGrid || chans > (double)kMaxGrid) return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}

// 16-byte vectors of 8 channels everywhere they are read or written
bool ssm_vec(const ScanArgs &P, wkv7_dtype dt, const void *more, size_t more_size) {
    const size_t al = 8 * dtype_size(dt) > 16 ? 16 : 8 * dtype_size(dt);
    const long long st = P.u_bs | P.u_ts | P.d_bs | P.d_ts | (P.z ? P.z_bs | P.z_ts : 0);
    return P.Dg % 8 == 0 && st % 8 == 0 && aligned_to(P.u, al) && aligned_to(P.delta, al) && aligned_to(P.z, al) &&
           aligned_to(P.y, 16) && aligned_to(more, more_size ? more_size : 1);
}

}  // namespace mixer
}  // namespace wkv7

extern "C" {

size_t wkv7_ssm_forward_workspace_size(int B, int T, int D, int N, int G) {
    using namespace wkv7::mixer;
    if (B <= 0 || T <= 0 || D <= 0 || ssm_dims(B, T, D, N, G) != WKV7_OK) return 0;
    return ssm_segment_bytes(B, D, N, ssm_segments(B, T, D, N, G, sm_count()));
}

size_t wkv7_ssm_saved_states_size(int B, int T, int D, int N) {
    using namespace wkv7::mixer;
    if (B <= 0 || T <= 0 || D <= 0 || ssm_dims(B, T, D, N, 1) != WKV7_OK) return 0;
    return (size_t)B * ((T + kTile - 1) / kTile) * D * N * sizeof(float);
}

wkv7_status wkv7_ssm_forward(int B, int T, int D, int N, int G, wkv7_dtype in_dt, wkv7_dtype y_dt, const void *u,
                             long long u_bs, long long u_ts, const void *delta, long long d_bs, long long d_ts,
                             const float *A, const void *Bm, long long b_bs, long long b_ts, const void *Cm,
                             long long c_bs, long long c_ts, const float *Dskip, const void *z, long long z_bs,
                             long long z_ts, const float *dt_bias, const float *state0, int softplus,
                             const int *lens, void *y, float *stateT, float *states, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
    using namespace wkv7::mixer;
    const wkv7_status s = ssm_dims(B, T, D, N, G);
    if (s != WKV7_OK) return s;
    if (!real_dtype(in_dt) || !real_dtype(y_dt)) return WKV7_ERR_INVALID_ARG;
    for (long long v : {u_bs, u_ts, d_bs, d_ts, b_bs, b_ts, c_bs, c_ts, z_bs, z_ts})
        if (v < 0) return WKV7_ERR_INVALID_ARG;
    if (lens && states) return WKV7_ERR_INVALID_ARG;
    if (!aligned_to(state0, 16) || !aligned_to(stateT, 16) || !aligned_to(states, 16) || !aligned_to(lens, 4) ||
        !aligned_to(workspace, 16))
        return WKV7_ERR_INVALID_ARG;
    if (B == 0 || D == 0) return WKV7_OK;
    if (T == 0) {
        const size_t n = (size_t)B * D * N * sizeof(float);
        if (!stateT || stateT == state0) return WKV7_OK;
        const cudaError_t e = state0 ? cudaMemcpyAsync(stateT, state0, n, cudaMemcpyDeviceToDevice, stream)
                                     : cudaMemsetAsync(stateT, 0, n, stream);
        return e == cudaSuccess ? WKV7_OK : WKV7_ERR_CUDA;
    }
    if (!elem_ok(u, in_dt) || !elem_ok(delta, in_dt) || !elem_ok(Bm, in_dt) || !elem_ok(Cm, in_dt) ||
        !aligned_to(z, dtype_size(in_dt)) || !f32_ok(A) || !f32_opt(Dskip) || !f32_opt(dt_bias) || !elem_ok(y, y_dt))
        return WKV7_ERR_INVALID_ARG;
    ScanArgs P{};
    P.B = B, P.T = T, P.D = D, P.N = N, P.G = G, P.Dg = D / G;
    P.tiles = (P.Dg + scan_channels(scan_lanes(N)) - 1) / scan_channels(scan_lanes(N));
    P.u = u, P.u_bs = u_bs, P.u_ts = u_ts, P.delta = delta, P.d_bs = d_bs, P.d_ts = d_ts;
    P.z = z, P.z_bs = z_bs, P.z_ts = z_ts;
    P.Bm = Bm, P.b_bs = b_bs, P.b_ts = b_ts, P.Cm = Cm, P.c_bs = c_bs, P.c_ts = c_ts;
    P.A = A, P.Dskip = Dskip, P.dt_bias = dt_bias, P.softplus = softplus, P.lens = lens;
    P.y = y, P.y_f32 = y_dt == WKV7_F32, P.stateT = stateT, P.states = states, P.nck = (T + kTile - 1) / kTile;
    int nseg = ssm_segments(B, T, D, N, G, sm_count());
    if (nseg > 1 && (workspace == nullptr || workspace_bytes < ssm_segment_bytes(B, D, N, nseg))) nseg = 1;
    ssm_fwd_all(P, state0, nseg, (char *)workspace, in_dt, ssm_vec(P, in_dt, nullptr, 0), true, stream);
    return launch_status();
}

wkv7_status wkv7_ssm_step(int B, int D, int N, int G, wkv7_dtype in_dt, wkv7_dtype y_dt, const void *u,
                          long long u_bs, const void *delta, long long d_bs, const float *A, const void *Bm,
                          long long b_bs, const void *Cm, long long c_bs, const float *Dskip, const void *z,
                          long long z_bs, const float *dt_bias, float *state, int softplus, void *y,
                          cudaStream_t stream) {
    using namespace wkv7::mixer;
    const wkv7_status s = ssm_dims(B, 1, D, N, G);
    if (s != WKV7_OK) return s;
    if (!real_dtype(in_dt) || !real_dtype(y_dt)) return WKV7_ERR_INVALID_ARG;
    for (long long v : {u_bs, d_bs, b_bs, c_bs, z_bs})
        if (v < 0) return WKV7_ERR_INVALID_ARG;
    if (B == 0 || D == 0) return WKV7_OK;
    if (!elem_ok(u, in_dt) || !elem_ok(delta, in_dt) || !elem_ok(Bm, in_dt) || !elem_ok(Cm, in_dt) ||
        !aligned_to(z, dtype_size(in_dt)) || !f32_ok(A) || !f32_opt(Dskip) || !f32_opt(dt_bias) ||
        !elem_ok(y, y_dt) || state == nullptr || !aligned_to(state, 16))
        return WKV7_ERR_INVALID_ARG;
    const StepArgs P{(long long)B * D, D, N, G, D / G, u, delta, Bm, Cm, z, u_bs, d_bs, b_bs, c_bs, z_bs, A, Dskip,
                     dt_bias, state, softplus, y};
    by_lanes(scan_lanes(N), [&](auto ln) {
        constexpr int LN = decltype(ln)::value;
        const unsigned grid = (unsigned)((P.total * LN + 255) / 256);
        const bool vec = N == 4 * LN && aligned_to(A, 16);
#define WKV7_STEP(I, O)                                                                 \
    (vec ? (void)(ssm_step_kernel<I, O, LN, true><<<grid, 256, 0, stream>>>(P))         \
         : (void)(ssm_step_kernel<I, O, LN, false><<<grid, 256, 0, stream>>>(P)))
        if (in_dt == WKV7_F32 && y_dt == WKV7_F32) WKV7_STEP(float, float);
        else if (in_dt == WKV7_F32) WKV7_STEP(float, bf16);
        else if (y_dt == WKV7_F32) WKV7_STEP(bf16, float);
        else WKV7_STEP(bf16, bf16);
#undef WKV7_STEP
    });
    return launch_status();
}

}  // extern "C"
