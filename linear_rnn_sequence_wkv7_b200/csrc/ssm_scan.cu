// Selective state-space scan, forward: whole sequences (wkv7_ssm_forward) and
// single tokens (wkv7_ssm_step).
//
//     dt = softplus(delta + bias),  h <- exp(dt A) h + dt u B,  y = (C . h + D u) z sigmoid(z)
//
// Bound: one exponential per (token, channel, n).  At N = 16 a channel-token
// moves 8 bytes but takes 16 exponentials, and an SM makes 16 a cycle; the
// state's update and readout (64 multiply-adds) stay below that.
//
// Mapping: a thread of the scanning half of a block holds 4 n of one or two
// channels in registers, the lanes of a channel side by side (N padded to 8, 16,
// 32 or 64 with zero rates and inputs, which keep a zero state at zero).  It walks
// tiles of 16 tokens, unrolled, with the exponentials of four tokens under way
// while the four before them run through the state, and leaves its part of C . h
// in shared memory, lane by lane.  The other half of the block copies tiles in
// (cp.async, three ahead), prepares the next tile (softplus and dt u once per
// channel, not once per n) and adds up, gates and stores the one before, so that
// neither kind of work waits for the other's latencies.
//
// 8 x 4096 tokens x 2048 channels, N = 16, bf16 in and out: 480 us, twice the
// exponentials alone; the schedulers issue 57% of cycles, the exponentials' pipe
// is busy for 65%.  One warp for both kinds of work took 511 us, B and C in fp32
// in shared memory or 8 tokens ahead no less.
//
// Few channels over many tokens: the state map of a stretch of tokens is
// h -> exp(A sum dt) h + E, so the sequence is cut into segments: one pass takes
// every segment's E (from a zero state, no output) and sum dt, a chain gives the
// entry states, and the outputs come from a second pass over all segments (1 x
// 65536 tokens x 2048 channels: 1.55 ms in 18 segments; one piece has 256
// scanning warps for 148 SMs).
#include <type_traits>

#include "mixer.cuh"
#include "ssm.cuh"

namespace wkv7 {
namespace mixer {
namespace {

constexpr int kRing = 4;            // tiles of raw inputs on their way or in use

// Shared memory of a block
template <typename T, int NP, bool Y> struct ScanShared {
    static constexpr int CC = scan_channels(NP), NIN = Y ? 3 : 2;
    float2 dd[2][kTile][CC];                        // dt, dt u
    T in[kRing][NIN][kTile][CC];                    // u, delta, z
    T BC[kRing][Y ? 2 : 1][kTile][NP];
    float y[Y ? 2 : 1][Y ? Planes<CC, NP / 4>::FLOATS : 4];     // C . h, lane by lane
};

template <typename T> __device__ __forceinline__ void put_raw(T *to, const Vec<T, 1> &v) {
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint16_t *>(to) = (uint16_t)v.w[0];
    else *reinterpret_cast<uint32_t *>(to) = v.w[0];
}
template <int V, typename T> __device__ __forceinline__ void shared_get(const T *p, float (&f)[V]) {
    Vec<T, V> v;
#pragma unroll
    for (int i = 0; i < (int)sizeof(v.w) / 4; ++i)
        v.w[i] = sizeof(T) * V < 4 ? *reinterpret_cast<const uint16_t *>(p) : 0;
    if constexpr (sizeof(v.w) == 16 && sizeof(T) * V == 16) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        v.w[0] = q.x, v.w[1] = q.y, v.w[2] = q.z, v.w[3] = q.w;
    } else if constexpr (sizeof(T) * V == 8) {
        const uint2 q = *reinterpret_cast<const uint2 *>(p);
        v.w[0] = q.x, v.w[1] = q.y;
    } else if constexpr (sizeof(T) * V == 4) {
        v.w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
    v.get(f);
}

template <int THREADS> __device__ __forceinline__ int scan_flip() {
    if constexpr (THREADS >= 256) return 0;
    __shared__ int flip;
    if (threadIdx.x == 0) {
        uint32_t slot;
        asm volatile("mov.u32 %0, %%warpid;" : "=r"(slot));
        flip = (slot >> 2) & 1;
    }
    __syncthreads();
    return flip;
}

// Y: outputs too, not a summary alone;  GATE: the gate's PRECISE
template <typename T, int NP, int TC, bool VEC, bool Y, bool GATE>
__global__ void __launch_bounds__(2 * scan_threads(NP, TC), scan_blocks(NP, TC, Y))
ssm_fwd_kernel(const ScanArgs P) {
    constexpr int CC = scan_channels(NP), LN = NP / 4, THREADS = scan_threads(NP, TC);     // of each kind
    constexpr int EPT = kTile * CC / THREADS, V = VEC ? (EPT < 4 ? EPT : 4) : 1, Q = EPT / V;   // a thread's share of a tile
    constexpr int IB = 2 * kTile * NP / 4, NB = (IB + THREADS - 1) / THREADS;   // quads of B, then of C
    constexpr bool PRECISE = sizeof(T) == 4;
    using Sum = Planes<CC, LN>;
    using S = ScanShared<T, NP, Y>;
    constexpr int NIN = S::NIN;
    extern __shared__ __align__(16) unsigned char scan_smem[];
    S &sh = *reinterpret_cast<S *>(scan_smem);
    auto &s_dd = sh.dd;
    auto &s_in = sh.in;
    auto &s_BC = sh.BC;
    auto &s_y = sh.y;

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
    const int nt = (t1 - t0 + kTile - 1) / kTile;

    // Which half of the block scans: a warp's place among the SM's four schedulers goes with its slot, so
    // blocks of fewer than four warps a half take turns, by the slot that the block got.  (Only the
    // balance hangs on it.)
    const int flip = scan_flip<2 * THREADS>();
    const int tid = threadIdx.x < THREADS ? threadIdx.x : threadIdx.x - THREADS;
    if ((threadIdx.x >= THREADS) != (flip != 0)) {
        // ---- the other half: tiles in, outputs out.  V channels in a row, the same in each of Q vectors.
        const int ch = (tid % (CC / V)) * V, lt = tid / (CC / V);
        const bool live = c0 + ch < c1;
        const int lc = live ? c0 + ch : c0;         // channels behind the group load others' values and store nothing
        float bias[V], skip[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bias[i] = P.dt_bias ? __ldg(P.dt_bias + lc + i) : 0.f;
            skip[i] = (Y && P.Dskip) ? __ldg(P.Dskip + lc + i) : 0.f;
        }
        const bool gate = Y && P.z != nullptr;
        constexpr int QT = kTile / Q;               // tokens between a thread's vectors
        const T *pu = static_cast<const T *>(P.u) + b * P.u_bs + (t0 + lt) * P.u_ts + lc;
        const T *pd = static_cast<const T *>(P.delta) + b * P.d_bs + (t0 + lt) * P.d_ts + lc;
        const T *pz = gate ? static_cast<const T *>(P.z) + b * P.z_bs + (t0 + lt) * P.z_ts + lc : nullptr;
        const T *Bm = static_cast<const T *>(P.Bm) + b * P.b_bs + t0 * P.b_ts + g * P.N;
        const T *Cm = static_cast<const T *>(P.Cm) + b * P.c_bs + t0 * P.c_ts + g * P.N;
        const size_t y0 = ((size_t)b * P.T + t0 + lt) * P.D + lc;
        float *yf = static_cast<float *>(P.y) + (Y ? y0 : 0);
        bf16 *yh = static_cast<bf16 *>(P.y) + (Y ? y0 : 0);
        // Tile j's inputs, as they are, into ring slot j mod kRing: u, delta, z for this thread, B and C for the scan
        auto fetch = [&](int j) {
            if (j < nt) {
                const int t = t0 + j * kTile, slot = j % kRing;
                const bool full = t + kTile <= t1;      // uniform
                if constexpr (V * sizeof(T) >= 4) {
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const int k = lt + q * QT;
                        if (!full && t + k >= t1) continue;
                        constexpr int BYTES = V * (int)sizeof(T);
                        copy_async<BYTES>(&s_in[slot][0][k][ch], pu + q * QT * P.u_ts, true);
                        copy_async<BYTES>(&s_in[slot][1][k][ch], pd + q * QT * P.d_ts, true);
                        if (gate) copy_async<BYTES>(&s_in[slot][NIN - 1][k][ch], pz + q * QT * P.z_ts, true);
                    }
                } else {                                // too narrow for that: through registers, loads first
                    static_assert(V == 1, "");
                    Vec<T, 1> r[Q][3];
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        if (!full && t + lt + q * QT >= t1) continue;
                        r[q][0].load(pu + q * QT * P.u_ts);
                        r[q][1].load(pd + q * QT * P.d_ts);
                        if (gate) r[q][2].load(pz + q * QT * P.z_ts);
                    }
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const int k = lt + q * QT;
                        if (!full && t + k >= t1) continue;
                        put_raw(&s_in[slot][0][k][ch], r[q][0]);
                        put_raw(&s_in[slot][1][k][ch], r[q][1]);
                        if (gate) put_raw(&s_in[slot][NIN - 1][k][ch], r[q][2]);
                    }
                }
                Quad<T, false> v[VEC ? 1 : NB];
#pragma unroll
                for (int q = 0; q < NB; ++q) {
                    const int e = tid + q * THREADS, k = (e / (NP / 4)) % kTile, n = e % (NP / 4) * 4;
                    if (e >= (Y ? IB : IB / 2)) break;
                    const bool in = full || t + k < t1;
                    const T *from = (Y && e >= IB / 2 ? Cm + k * P.c_ts : Bm + k * P.b_ts) + n;
                    if constexpr (VEC) copy_async<4 * (int)sizeof(T)>(&s_BC[slot][0][0][0] + 4 * e, from, in && n < P.N);
                    else v[q].load(from, in ? P.N - n : 0);
                }
                if constexpr (!VEC) {
#pragma unroll
                    for (int q = 0; q < NB; ++q) {
                        const int e = tid + q * THREADS;
                        if (e < (Y ? IB : IB / 2)) v[q].put(&s_BC[slot][0][0][0] + 4 * e);
                    }
                }
                pu += kTile * P.u_ts, pd += kTile * P.d_ts, Bm += kTile * P.b_ts, Cm += kTile * P.c_ts;
                if (gate) pz += kTile * P.z_ts;
            }
            cp_async_commit();
        };
        auto prepare = [&](int j) {     // tokens behind t1: dt = dt u = B = 0 keep the state
            const int t = t0 + j * kTile, slot = j % kRing;
            const bool full = t + kTile <= t1;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int k = lt + q * QT;
                float fu[V], fd[V];
                shared_get<V>(&s_in[slot][0][k][ch], fu);
                shared_get<V>(&s_in[slot][1][k][ch], fd);
#pragma unroll
                for (int i = 0; i < V; ++i) fd[i] += bias[i];
                if (P.softplus) softplus_all<PRECISE>(fd);
#pragma unroll
                for (int i = 0; i < V; ++i) fu[i] *= fd[i];
                if (!full && t + k >= t1) {
#pragma unroll
                    for (int i = 0; i < V; ++i) fd[i] = fu[i] = 0.f;
                }
                put_pairs<V>(&s_dd[j & 1][k][ch], fd, fu);
            }
        };
        auto finish = [&](int j) {
            if constexpr (Y) {
                const int t = t0 + j * kTile, slot = j % kRing;
                const bool full = t + kTile <= t1;
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const int k = lt + q * QT;
                    float f[V], fu[V], fz[V];
                    shared_get<V>(&s_in[slot][0][k][ch], fu);
                    if (gate) shared_get<V>(&s_in[slot][NIN - 1][k][ch], fz);
                    Sum::template sum<V>(s_y[j & 1], k, ch, f);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        f[i] = fmaf(skip[i], fu[i], f[i]);
                        if (gate) f[i] *= fz[i] * sigmoid<GATE>(fz[i]);
                    }
                    if (live && (full || t + k < t1)) {
                        if (P.y_f32) storev<V>(yf + (size_t)q * QT * P.D, f);
                        else storev<V>(yh + (size_t)q * QT * P.D, f);
                    }
                }
                yf += (size_t)kTile * P.D, yh += (size_t)kTile * P.D;
            }
        };
        // While tile j is in the scan: tile j - 1 goes out, which frees its slot for tile j + 3, and tile j + 1
        // is prepared.  A slot's u, delta and z are read by the thread that copied them; the barrier shows B and
        // C to the scan.
        fetch(0), fetch(1), fetch(2);
        cp_async_wait<2>();
        if (nt > 0) prepare(0);
        __syncthreads();
        for (int j = 0; j < nt; ++j) {
            if (j > 0) finish(j - 1);
            fetch(j + 3);
            cp_async_wait<2>();
            if (j + 1 < nt) prepare(j + 1);
            __syncthreads();
        }
        if (nt > 0) finish(nt - 1);
        return;
    }

    // ---- the scan: channels cs .. cs + TC - 1 and n = ns .. ns + 3
    const int nl = tid % LN, cl = tid / LN * TC, cs = c0 + cl, ns = 4 * nl;
    float2 a2[TC][2], h[TC][2];
#pragma unroll
    for (int c = 0; c < TC; ++c) {
        const bool mine = cs + c < c1;
        load_rates(P.A + (size_t)(cs + c) * P.N, P.N, ns, mine, a2[c]);
        h[c][0] = h[c][1] = make_float2(0.f, 0.f);
        if (mine && P.entry) load_state(P.entry + (((size_t)seg * P.B + b) * P.D + cs + c) * P.N, P.N, ns, h[c]);
    }
    double sum[TC] = {};                            // of dt, when summarising
    __syncthreads();
    for (int j = 0; j < nt; ++j) {
        const int buf = j & 1, slot = j % kRing;
        if (P.states) {
#pragma unroll
            for (int c = 0; c < TC; ++c)
                if (cs + c < c1)
                    store_state(P.states + ((size_t)(b * P.nck + t0 / kTile + j) * P.D + cs + c) * P.N, P.N, ns, h[c]);
        }
        float part[TC] = {};
        // A group's decays and inputs are on their way while the group before it runs through the state
        constexpr int GT = 4;
        float2 a[2][GT][TC][2], in[2][GT][TC][2];
        auto ready = [&](int k0, float2 (&av)[GT][TC][2], float2 (&bv)[GT][TC][2]) {
#pragma unroll
            for (int i = 0; i < GT; ++i) {
                float dt[TC], du[TC];
                if constexpr (TC == 2) {
                    const float4 q = *reinterpret_cast<const float4 *>(&s_dd[buf][k0 + i][cl]);
                    dt[0] = q.x, du[0] = q.y, dt[TC - 1] = q.z, du[TC - 1] = q.w;
                } else {
                    const float2 q = s_dd[buf][k0 + i][cl];
                    dt[0] = q.x, du[0] = q.y;
                }
                float2 B[2];
                shared_n(&s_BC[slot][0][k0 + i][ns], B);
#pragma unroll
                for (int c = 0; c < TC; ++c) {
                    const float2 d2 = make_float2(dt[c], dt[c]), w2 = make_float2(du[c], du[c]);
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        av[i][c][m] = decay(d2, a2[c][m]), bv[i][c][m] = __fmul2_rn(w2, B[m]);
                    if constexpr (!Y) part[c] += dt[c];
                }
            }
        };
        ready(0, a[0], in[0]);
#pragma unroll
        for (int k = 0; k < kTile; k += GT) {
            if (k + GT < kTile) ready(k + GT, a[(k / GT + 1) & 1], in[(k / GT + 1) & 1]);
#pragma unroll
            for (int i = 0; i < GT; ++i) {
                float2 C[2];
                if constexpr (Y) shared_n(&s_BC[slot][Y ? 1 : 0][k + i][ns], C);
                float y[TC];
#pragma unroll
                for (int c = 0; c < TC; ++c) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        h[c][m] = __ffma2_rn(a[(k / GT) & 1][i][c][m], h[c][m], in[(k / GT) & 1][i][c][m]);
                    if constexpr (Y) {
                        const float2 p = __ffma2_rn(h[c][1], C[1], __fmul2_rn(h[c][0], C[0]));
                        y[c] = p.x + p.y;
                    }
                }
                if constexpr (Y) Sum::template put<TC>(s_y[buf], k + i, cl, nl, y);
            }
        }
        if constexpr (!Y) {
#pragma unroll
            for (int c = 0; c < TC; ++c) sum[c] += part[c];
        }
        __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < TC; ++c) {
        if (cs + c >= c1) continue;
        if (seg == P.nseg - 1 && P.stateT) store_state(P.stateT + ((size_t)b * P.D + cs + c) * P.N, P.N, ns, h[c]);
        if (!Y && P.seg_end) {
            const size_t at = ((size_t)seg * P.B + b) * P.D + cs + c;
            store_state(P.seg_end + at * P.N, P.N, ns, h[c]);
            if (nl == 0) P.seg_dt[at] = (float)sum[c];
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
// write, 8 bytes an n.  R = 4: a thread takes the same channel of four sequences,
// so that four states are on their way and the rates are read once for them.
struct StepArgs {
    int B, D, N, Dg;
    long long total;                // ceil(B / R) * D
    const void *u, *delta, *Bm, *Cm, *z;
    long long u_bs, d_bs, b_bs, c_bs, z_bs;
    const float *A, *Dskip, *dt_bias;
    float *state;
    int softplus;
    void *y;
};

template <typename T, typename YT, int LN, int R, bool VEC>
__global__ void __launch_bounds__(256, 4)
ssm_step_kernel(const StepArgs P) {
    constexpr bool PRECISE = sizeof(T) == 4 || sizeof(YT) == 4;
    const long long unit = ((long long)blockIdx.x * 256 + threadIdx.x) / LN;
    const int nl = threadIdx.x % LN, ns = 4 * nl;
    if (unit >= P.total) return;                // LN lanes leave together
    const long long b0 = unit / P.D * R;
    const int d = (int)(unit % P.D), g = d / P.Dg, rows = (int)min((long long)R, P.B - b0);
    // the softplus and the gate of row r are lane r's (of rows nl, nl + LN, ... where lanes are fewer)
    constexpr int OWN = R > LN ? R / LN : 1;
    float4 h[R];
    Vec<T, 1> u[OWN], de[OWN], z[OWN];
    Quad<T, VEC> Bq[R], Cq[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const long long b = r < rows ? b0 + r : b0;
        const float *S = P.state + ((size_t)b * P.D + d) * P.N + ns;
        if constexpr (VEC) h[r] = __ldcs(reinterpret_cast<const float4 *>(S));     // N = 4 LN
        else {
            h[r].x = ns < P.N ? S[0] : 0.f, h[r].y = ns + 1 < P.N ? S[1] : 0.f;
            h[r].z = ns + 2 < P.N ? S[2] : 0.f, h[r].w = ns + 3 < P.N ? S[3] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int r = (nl + i * LN) % R;
        const long long b = r < rows ? b0 + r : b0;
        u[i].load(static_cast<const T *>(P.u) + b * P.u_bs + d);
        de[i].load(static_cast<const T *>(P.delta) + b * P.d_bs + d);
        z[i].zero();
        if (P.z) z[i].load(static_cast<const T *>(P.z) + b * P.z_bs + d);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const long long b = r < rows ? b0 + r : b0;
        Bq[r].load(static_cast<const T *>(P.Bm) + b * P.b_bs + g * P.N + ns, P.N - ns);
        Cq[r].load(static_cast<const T *>(P.Cm) + b * P.c_bs + g * P.N + ns, P.N - ns);
    }
    float2 a2[2];
    load_rates(P.A + (size_t)d * P.N, P.N, ns, true, a2);
    const float bias = P.dt_bias ? __ldg(P.dt_bias + d) : 0.f, skip = P.Dskip ? __ldg(P.Dskip + d) : 0.f;
    const unsigned lane = threadIdx.x & 31, first = lane & ~(LN - 1), group = ((1u << LN) - 1u) << first;
    float dts[OWN], us[OWN], ws[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        float fu[1], fd[1];
        u[i].get(fu), de[i].get(fd);
        const float x = fd[0] + bias;
        dts[i] = P.softplus ? softplus<sizeof(T) == 4>(x) : x;
        us[i] = fu[0], ws[i] = dts[i] * fu[0];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float B[4], C[4];
        Bq[r].get(B), Cq[r].get(C);
        float dt = dts[r / LN], w = ws[r / LN];
        if constexpr (R > 1) {
            dt = __shfl_sync(group, dt, first + r % LN);
            w = __shfl_sync(group, w, first + r % LN);
        }
        const float2 d2 = make_float2(dt, dt), w2 = make_float2(w, w);
        const float2 lo = __ffma2_rn(decay(d2, a2[0]), make_float2(h[r].x, h[r].y),
                                     __fmul2_rn(w2, make_float2(B[0], B[1])));
        const float2 hi = __ffma2_rn(decay(d2, a2[1]), make_float2(h[r].z, h[r].w),
                                     __fmul2_rn(w2, make_float2(B[2], B[3])));
        const float2 p = __ffma2_rn(hi, make_float2(C[2], C[3]), __fmul2_rn(lo, make_float2(C[0], C[1])));
        float y = p.x + p.y;
#pragma unroll
        for (int o = 1; o < LN; o <<= 1) y += __shfl_xor_sync(group, y, o);
        if (r >= rows) continue;
        const size_t at = (size_t)(b0 + r) * P.D + d;
        float *S = P.state + at * P.N + ns;
        if constexpr (VEC) __stcs(reinterpret_cast<float4 *>(S), make_float4(lo.x, lo.y, hi.x, hi.y));
        else {
            const float v[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (ns + n < P.N) S[n] = v[n];
        }
        if (nl == r % LN) {
            float fz[1];
            y = fmaf(skip, us[r / LN], y);
            if (P.z) {
                z[r / LN].get(fz);
                y *= fz[0] * sigmoid<PRECISE>(fz[0]);
            }
            static_cast<YT *>(P.y)[at] = from_f32<YT>(y);
        }
    }
}

template <typename T, int NP, int TC, bool Y> void launch_fwd(const ScanArgs &P, bool vec, cudaStream_t st) {
    const unsigned grid = (unsigned)((long long)P.nseg * P.B * P.G * P.tiles);
    constexpr int threads = 2 * scan_threads(NP, TC);
    constexpr size_t smem = sizeof(ScanShared<T, NP, Y>);
    auto launch = [&](auto gate) {
        constexpr bool GATE = decltype(gate)::value;
        auto kernel = vec ? ssm_fwd_kernel<T, NP, TC, true, Y, GATE> : ssm_fwd_kernel<T, NP, TC, false, Y, GATE>;
        if (smem > 40 * 1024) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        kernel<<<grid, threads, smem, st>>>(P);
    };
    if constexpr (Y) by_precision<T>(P.y_f32, launch);
    else launch(std::false_type{});
}
// Two channels a thread halve the loads of B and C and the instructions around
// them; one channel a thread makes twice the warps.  At N = 16 and 8 x 4096 tokens
// x 2048 channels (7 scanning warps an SM at two): 482 us at two, 503 us at one;
// below 6 warps an SM at two the schedulers run dry.
template <typename T, int NP, bool Y> void launch_fwd_tc(const ScanArgs &P, int sms, bool vec, cudaStream_t st) {
    const long long warps = (long long)P.nseg * P.B * P.G * P.tiles * scan_threads(NP, 2) / 32;
    if (warps < 6ll * sms) return launch_fwd<T, NP, 1, Y>(P, vec, st);
    launch_fwd<T, NP, 2, Y>(P, vec, st);
}

}  // namespace

// Segments of a forward over B sequences.  One piece takes 0.04 us a token while
// the SMs have up to two scanning warps each (0.05 at 3.5, 0.07 at 7); segments
// scan each token twice, on as many warps as the SMs take.  So segments for 32
// warps an SM where that makes twelve of them, and at least five of 128 tokens.
// Bf16, N = 16, segments against one piece: 1 x 4096 x 2048 125 / 158 us, 2 x
// 4096 x 2048 221 / 204, 1 x 1024 x 2048 46 / 45, 1 x 1024 x 256 23 / 42, 1 x 512
// x 2048 43 / 30.
int ssm_segments(int B, int T, int D, int N, int G, int sms) {
    const int NP = scan_pad(N), CC = scan_channels(NP), tiles = G > 0 ? (D / G + CC - 1) / CC : 0;
    const long long warps = (long long)B * G * tiles * scan_threads(NP, 1) / 32;
    if (warps <= 0 || sms <= 0) return 1;
    const long long want = 32ll * sms / warps, most = T / 128;
    if (want < 12 || most < 5) return 1;
    return (int)(want < most ? want : most);
}

void ssm_fwd(const ScanArgs &P, wkv7_dtype dt, bool vec, bool y, cudaStream_t st) {
    const int sms = sm_count();
    by_pad(scan_pad(P.N), [&](auto np) {
        constexpr int NP = decltype(np)::value;
        if (dt == WKV7_F32) {
            if (y) launch_fwd_tc<float, NP, true>(P, sms, vec, st);
            else launch_fwd_tc<float, NP, false>(P, sms, vec, st);
        } else {
            if (y) launch_fwd_tc<bf16, NP, true>(P, sms, vec, st);
            else launch_fwd_tc<bf16, NP, false>(P, sms, vec, st);
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
    // blocks of a launch: one for 8 channels (N > 32; 16 or more otherwise, 16 to 128 in the backward), rounded
    // up in each group; segments multiply them only where they are a few an SM
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
    // four sequences a thread where that still makes two blocks an SM
    const int lanes = scan_pad(N) / 4;
    const bool four = (long long)((B + 3) / 4) * D * lanes >= 512ll * sm_count();
    const StepArgs P{B, D, N, D / G, (four ? (long long)((B + 3) / 4) : B) * D, u, delta, Bm, Cm, z, u_bs, d_bs,
                     b_bs, c_bs, z_bs, A, Dskip, dt_bias, state, softplus, y};
    const size_t quad = 4 * dtype_size(in_dt);
    const bool quads = (b_bs | c_bs) % 4 == 0 && aligned_to(Bm, quad) && aligned_to(Cm, quad);
    by_pad(scan_pad(N), [&](auto np) {
        constexpr int LN = decltype(np)::value / 4;
        const unsigned grid = (unsigned)((P.total * LN + 255) / 256);
        const bool vec = N == 4 * LN && quads;
#define WKV7_STEP(I, O)                                                                 \
    (four ? (vec ? (void)(ssm_step_kernel<I, O, LN, 4, true><<<grid, 256, 0, stream>>>(P))    \
                 : (void)(ssm_step_kernel<I, O, LN, 4, false><<<grid, 256, 0, stream>>>(P)))  \
          : (vec ? (void)(ssm_step_kernel<I, O, LN, 1, true><<<grid, 256, 0, stream>>>(P))    \
                 : (void)(ssm_step_kernel<I, O, LN, 1, false><<<grid, 256, 0, stream>>>(P))))
        if (in_dt == WKV7_F32 && y_dt == WKV7_F32) WKV7_STEP(float, float);
        else if (in_dt == WKV7_F32) WKV7_STEP(float, bf16);
        else if (y_dt == WKV7_F32) WKV7_STEP(bf16, float);
        else WKV7_STEP(bf16, bf16);
#undef WKV7_STEP
    });
    return launch_status();
}

}  // extern "C"
