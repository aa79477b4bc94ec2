// Selective state-space scan, forward: whole sequences (wkv7_ssm_forward) and
// single tokens (wkv7_ssm_step).
//
//     dt = softplus(delta + bias),  h <- exp(dt A) h + dt u B,  y = (C . h + D u) z sigmoid(z)
//
// Bound: one exponential per (token, channel, n).  At N = 16 a channel-token
// moves 8 bytes but takes 16 exponentials, and an SM makes 16 a cycle; the
// state's update and readout (64 multiply-adds) stay below that.
//
// Mapping: a thread holds 4 (or 2) of a channel's n in registers, the lanes of a
// channel side by side (N padded to 8, 16, 32 or 64 with zero rates and inputs,
// which keep a zero state at zero).  A tile of 16 tokens is prepared by the whole
// block (softplus and dt u once per channel, not once per n) into shared memory
// and walked token by token, unrolled, so that the exponentials of later tokens
// do not wait for the state.  Partial readouts go to shared memory lane by lane;
// the threads that loaded u and z add them up, gate and store.  Loads of the next
// tile are in flight meanwhile.
//
// Parallelism: one warp has 8 channels at N = 16 and needs about 50 instructions
// for each of their tokens, four cycles apart when it is alone on its scheduler,
// so blocks are small (16 channels).  Where even these leave schedulers with
// fewer than three warps, a thread takes 2 n instead of 4 (twice the warps for
// about a third more instructions).
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

template <typename T, int NP, int NPT, bool VEC, bool Y>
__global__ void __launch_bounds__(scan_threads(NP, NPT))
ssm_fwd_kernel(const ScanArgs P) {
    constexpr int CC = scan_channels(NP), LN = NP / NPT, THREADS = CC * LN;
    constexpr int EPT = kTile * CC / THREADS, V = VEC ? EPT : 1, Q = EPT / V;   // a thread's share of a tile
    constexpr int IB = 2 * kTile * NP / 4, NB = (IB + THREADS - 1) / THREADS;   // quads of B, then of C
    constexpr bool PRECISE = sizeof(T) == 4;
    __shared__ __align__(16) float2 s_dd[kTile][CC];                            // dt, dt u
    __shared__ __align__(16) T s_BC[Y ? 2 : 1][kTile][NP];
    using Sum = Planes<CC, LN>;
    __shared__ __align__(16) float s_y[Y ? Sum::FLOATS : 1];

    const int tid = threadIdx.x;
    unsigned id = blockIdx.x;
    const int tile_c = (int)(id % (unsigned)P.tiles);
    id /= (unsigned)P.tiles;
    const int g = (int)(id % (unsigned)P.G);
    id /= (unsigned)P.G;
    const long long b = id % (unsigned)P.B;
    const int seg = (int)(id / (unsigned)P.B);
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

    // and when it scans: channel cs and n = ns .. ns + NPT - 1
    const int nl = tid % LN, cl = tid / LN, cs = c0 + cl, ns = NPT * nl;
    const bool mine = cs < c1;
    float2 a2[NPT / 2], h[NPT / 2];
    load_rates<NPT>(P.A + (size_t)cs * P.N, P.N, ns, mine, a2);
#pragma unroll
    for (int j = 0; j < NPT / 2; ++j) h[j] = make_float2(0.f, 0.f);
    if (mine && P.entry) load_state<NPT>(P.entry + (((size_t)seg * P.B + b) * P.D + cs) * P.N, P.N, ns, h);
    double sum = 0;                                 // of dt, when summarising

    Vec<T, V> nu[Q], nd[Q], nz[Q], cu[Q], cz[Q];
    Quad<T, VEC> nb[NB];
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
            const int e = tid + q * THREADS, tt = t + (e / (NP / 4)) % kTile, n = e % (NP / 4) * 4;
            const bool c = e >= IB / 2, in = e < (Y ? IB : IB / 2) && tt < t1;
            nb[q].load((c ? Cm + tt * P.c_ts : Bm + tt * P.b_ts) + n, in ? P.N - n : 0);
        }
    };
    auto prepare = [&](int t) {         // tokens behind t1: dt = dt u = B = 0 keep the state
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int k = lt + q * (kTile / Q), ch = lc - c0;
            const bool in = live && t + k < t1;
            float fu[V], fd[V];
            nu[q].get(fu), nd[q].get(fd);
#pragma unroll
            for (int i = 0; i < V; ++i) fd[i] += bias[i];
            if (P.softplus) softplus_all<PRECISE>(fd);
#pragma unroll
            for (int i = 0; i < V; ++i) fd[i] = in ? fd[i] : 0.f, fu[i] = in ? fd[i] * fu[i] : 0.f;
            put_pairs<V>(&s_dd[k][ch], fd, fu);
            cu[q] = nu[q], cz[q] = nz[q];
        }
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int e = tid + q * THREADS;
            if (e < (Y ? IB : IB / 2)) nb[q].put(&s_BC[0][0][0] + 4 * e);
        }
    };

    if (t0 < t1) {
        fetch(t0);
        prepare(t0);
        __syncthreads();
    }
    for (int t = t0; t < t1; t += kTile) {
        if (t + kTile < t1) fetch(t + kTile);
        if (P.states && mine)
            store_state<NPT>(P.states + ((size_t)(b * P.nck + t / kTile) * P.D + cs) * P.N, P.N, ns, h);
        float part = 0.f;
#pragma unroll
        for (int k = 0; k < kTile; ++k) {
            const float2 dd = s_dd[k][cl];
            const float2 d2 = make_float2(dd.x, dd.x), w2 = make_float2(dd.y, dd.y);
            float2 B[NPT / 2];
            shared_n<NPT>(&s_BC[0][k][ns], B);
#pragma unroll
            for (int j = 0; j < NPT / 2; ++j)
                h[j] = __ffma2_rn(ex2(__fmul2_rn(d2, a2[j])), h[j], __fmul2_rn(w2, B[j]));
            if constexpr (Y) {
                float2 C[NPT / 2];
                shared_n<NPT>(&s_BC[Y ? 1 : 0][k][ns], C);
                float2 p = __fmul2_rn(h[0], C[0]);
                if constexpr (NPT == 4) p = __ffma2_rn(h[NPT / 2 - 1], C[NPT / 2 - 1], p);
                Sum::put(s_y, k, cl, nl, p.x + p.y);
            } else {
                part += dd.x;
            }
        }
        if constexpr (!Y) sum += part;
        __syncthreads();
        if constexpr (Y) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int k = lt + q * (kTile / Q);
                if (!live || t + k >= t1) continue;
                float f[V], fu[V], fz[V];
                cu[q].get(fu), cz[q].get(fz);
                Sum::template sum<V>(s_y, k, lc - c0, f);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    f[i] = fmaf(skip[i], fu[i], f[i]);
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
    if (!mine) return;
    if (seg == P.nseg - 1 && P.stateT) store_state<NPT>(P.stateT + ((size_t)b * P.D + cs) * P.N, P.N, ns, h);
    if (!Y && P.seg_end) {
        const size_t at = ((size_t)seg * P.B + b) * P.D + cs;
        store_state<NPT>(P.seg_end + at * P.N, P.N, ns, h);
        if (nl == 0) P.seg_dt[at] = (float)sum;
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
    const float dt = P.softplus ? softplus<sizeof(T) == 4>(x) : x, du = dt * u;
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

template <typename T, int NP, int NPT, bool Y> void launch_fwd(const ScanArgs &P, bool vec, cudaStream_t st) {
    const unsigned grid = (unsigned)((long long)P.nseg * P.B * P.G * P.tiles);
    if (vec) ssm_fwd_kernel<T, NP, NPT, true, Y><<<grid, scan_threads(NP, NPT), 0, st>>>(P);
    else ssm_fwd_kernel<T, NP, NPT, false, Y><<<grid, scan_threads(NP, NPT), 0, st>>>(P);
}
// Blocks, each of one schedule of warps: 2 n a thread where 4 would leave a
// scheduler (four an SM) with fewer than three warps.  Padded to 64 a channel has
// 16 lanes already.
template <typename T, int NP, bool Y> void launch_fwd_npt(const ScanArgs &P, int sms, bool vec, cudaStream_t st) {
    const long long warps = (long long)P.nseg * P.B * P.G * P.tiles * scan_threads(NP, 4) / 32;
    if constexpr (NP < 64) {
        if (warps < 12ll * sms) return launch_fwd<T, NP, 2, Y>(P, vec, st);
    }
    launch_fwd<T, NP, 4, Y>(P, vec, st);
}

}  // namespace

// Segments of a forward over B sequences: enough that its blocks fill the SMs,
// if that makes at least three of them (each token is then scanned twice), each
// of at least 128 tokens.
int ssm_segments(int B, int T, int D, int N, int G, int sms) {
    const int NP = scan_pad(N), CC = scan_channels(NP), tiles = G > 0 ? (D / G + CC - 1) / CC : 0;
    const long long warps = (long long)B * G * tiles * scan_threads(NP, 4) / 32;
    if (warps <= 0 || sms <= 0) return 1;
    const long long want = 16ll * sms / warps, most = T / 128;
    const long long s = want < most ? want : most;
    return s >= 3 ? (int)s : 1;
}

void ssm_fwd(const ScanArgs &P, wkv7_dtype dt, bool vec, bool y, cudaStream_t st) {
    const int sms = sm_count();
    by_pad(scan_pad(P.N), [&](auto np) {
        constexpr int NP = decltype(np)::value;
        if (dt == WKV7_F32) {
            if (y) launch_fwd_npt<float, NP, true>(P, sms, vec, st);
            else launch_fwd_npt<float, NP, false>(P, sms, vec, st);
        } else {
            if (y) launch_fwd_npt<bf16, NP, true>(P, sms, vec, st);
            else launch_fwd_npt<bf16, NP, false>(P, sms, vec, st);
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
    // a launch has at most 16 channels a block and 16 * 148 segments when that leaves SMs idle
    if ((double)B * (D + 16.0 * G) > (double)kMaxGrid) return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}

// Vectors of up to 8 channels and of 4 n everywhere they are read or written
bool ssm_vec(const ScanArgs &P, wkv7_dtype dt) {
    const size_t quad = 4 * dtype_size(dt);
    const long long st = P.u_bs | P.u_ts | P.d_bs | P.d_ts | (P.z ? P.z_bs | P.z_ts : 0);
    const long long sn = P.b_bs | P.b_ts | P.c_bs | P.c_ts;
    return P.Dg % 8 == 0 && st % 8 == 0 && P.N % 4 == 0 && sn % 4 == 0 && aligned_to(P.u, 16) &&
           aligned_to(P.delta, 16) && aligned_to(P.z, 16) && aligned_to(P.y, 16) && aligned_to(P.Bm, quad) &&
           aligned_to(P.Cm, quad);
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
    P.tiles = (P.Dg + scan_channels(scan_pad(N)) - 1) / scan_channels(scan_pad(N));
    P.u = u, P.u_bs = u_bs, P.u_ts = u_ts, P.delta = delta, P.d_bs = d_bs, P.d_ts = d_ts;
    P.z = z, P.z_bs = z_bs, P.z_ts = z_ts;
    P.Bm = Bm, P.b_bs = b_bs, P.b_ts = b_ts, P.Cm = Cm, P.c_bs = c_bs, P.c_ts = c_ts;
    P.A = A, P.Dskip = Dskip, P.dt_bias = dt_bias, P.softplus = softplus, P.lens = lens;
    P.y = y, P.y_f32 = y_dt == WKV7_F32, P.stateT = stateT, P.states = states, P.nck = (T + kTile - 1) / kTile;
    int nseg = ssm_segments(B, T, D, N, G, sm_count());
    if (nseg > 1 && (workspace == nullptr || workspace_bytes < ssm_segment_bytes(B, D, N, nseg))) nseg = 1;
    ssm_fwd_all(P, state0, nseg, (char *)workspace, in_dt, ssm_vec(P, in_dt), true, stream);
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
    by_pad(scan_pad(N), [&](auto np) {
        constexpr int LN = decltype(np)::value / 4;
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
