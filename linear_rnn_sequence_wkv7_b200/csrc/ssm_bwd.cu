// Backward of the selective scan (wkv7_ssm_backward).
//
//     ds_t = dy_t z sigmoid(z),     g_t = C_t ds_t + exp(dt_{t+1} A) g_{t+1}
//     p_t = exp(dt_t A) h_{t-1}
//     dC_t = sum_d ds_t h_t         dB_t = sum_d g_t dt_t u_t
//     du_t = dt_t sum_n g_t B_t + D ds_t
//     d(dt)_t = u_t sum_n g_t B_t + sum_n A p_t g_t,   ddelta = d(dt) softplus'
//     dA = sum_t dt_t p_t g_t       dD = sum ds u       dz = dy s (z sigmoid(z))'
//
// A thread holds 4 n of two channels, the lanes of a channel side by side, 128
// threads a block (64 channels at N = 16).  A block walks its tiles of 16 tokens
// from the last to the first, each in two halves: from the state saved before the
// tile it replays the half's 8 tokens with every h in registers, then runs the
// adjoint back over them.  2.5 exponentials per (token, channel, n), 1.5 in the
// replays and one on the way back.
//
// 4 x 4096 tokens x 2048 channels, N = 16, bf16: 0.94 ms in two segments, plus
// 0.22 ms for their summaries.  Bound by latency: two warps a scheduler is what
// 255 registers leave, each issues once in four cycles (all 16 tokens at once
// spilled; one channel a thread with twice the warps 0.99 ms; three blocks an SM
// at 168 registers spilled too, 1.04 ms).
//
// Sums over n (C . h, g . B, A . p g) go to shared memory lane by lane and are
// added up by the threads that write the outputs.  Sums over channels (dB, dC) run
// over the lanes of a warp by exchanges: a lane's four n are kept in an order of
// its own, slot j holding n = j xor (channel group mod 4), so that the half to
// hand over at a step is the same registers in every lane and needs no selects.
// The warps join in shared memory, the blocks through partial sums added up in
// order by a second kernel.  Few channels over many tokens: segments, as in the
// forward (summaries from a zero adjoint, a chain from the last to the first).
#include "ssm.cuh"

namespace wkv7 {
namespace mixer {

void sum_parts(long long parts, long long cols, const float *partial, float *out, cudaStream_t st);
wkv7_status ssm_dims(int B, int T, int D, int N, int G);
int ssm_segments(int B, int T, int D, int N, int G, int sms);
size_t ssm_segment_bytes(int B, int D, int N, int nseg);
void ssm_fwd_all(ScanArgs P, const float *state0, int nseg, char *ws, wkv7_dtype dt, bool vec, bool y,
                 cudaStream_t st);
bool ssm_vec(const ScanArgs &P, wkv7_dtype dt);

namespace {

struct BwdArgs {
    ScanArgs f;
    const void *dy;
    const float *exit;              // [nseg][B][D][N] adjoint behind each segment, or null for zeros
    int g_f32;
    void *du, *ddelta, *dz;
    float *dstate0;
    float *dbc;                     // [tiles][2][B][T][G][N] partial dB, dC
    float *dA;                      // [nseg * B][D][N] partial
    float *dpar;                    // [2][nseg * B][D] partial dD, ddt_bias
    float *seg_g, *seg_dt;          // summaries
};

// A segment's own adjoint (from zero behind it) and sum of dt
// GATE: PRECISE of the gates and of the softplus's slope
template <typename T, int NP, bool VEC, bool GATE>
__global__ void __launch_bounds__(scan_threads(NP, 1))
ssm_bwd_summary_kernel(const BwdArgs K) {
    const ScanArgs &P = K.f;
    constexpr int CC = scan_channels(NP), LN = NP / 4, THREADS = CC * LN;
    constexpr int EPT = kTile * CC / THREADS, V = VEC ? EPT : 1, Q = EPT / V;
    constexpr int IB = kTile * NP / 4, NB = (IB + THREADS - 1) / THREADS;
    constexpr bool PRECISE = sizeof(T) == 4;
    __shared__ __align__(16) float2 s_dd[kTile][CC];        // dt, ds
    __shared__ __align__(16) T s_C[kTile][NP];
    const int tid = threadIdx.x;
    unsigned id = blockIdx.x;
    const int per_g = (P.Dg + CC - 1) / CC, tile_c = (int)(id % (unsigned)per_g);
    id /= (unsigned)per_g;
    const int g = (int)(id % (unsigned)P.G);
    id /= (unsigned)P.G;
    const long long b = id % (unsigned)P.B;
    const int seg = (int)(id / (unsigned)P.B);
    const int c0 = g * P.Dg + tile_c * CC, c1 = (g + 1) * P.Dg;
    const int t0 = (int)min((long long)seg * P.seg_len, (long long)P.T);
    const int t1 = (int)min((long long)t0 + P.seg_len, (long long)P.T);
    const int lc = c0 + (tid % (CC / V)) * V, lt = tid / (CC / V);
    const bool live = lc < c1;
    const T *de = static_cast<const T *>(P.delta) + b * P.d_bs + lc;
    const T *z = P.z ? static_cast<const T *>(P.z) + b * P.z_bs + lc : nullptr;
    const T *dy = static_cast<const T *>(K.dy) + (size_t)b * P.T * P.D + lc;
    const T *Cm = static_cast<const T *>(P.Cm) + b * P.c_bs + g * P.N;
    const int nl = tid % LN, cl = tid / LN, cs = c0 + cl, ns = 4 * nl;
    float2 a2[2], w[2];
    load_rates(P.A + (size_t)cs * P.N, P.N, ns, cs < c1, a2);
    w[0] = w[1] = make_float2(0.f, 0.f);
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = (live && P.dt_bias) ? __ldg(P.dt_bias + lc + i) : 0.f;
    double sum = 0;
    Vec<T, V> nd[Q], ng[Q], nz[Q];
    Quad<T, VEC> nc[NB];
    auto fetch = [&](int t) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int tt = t + lt + q * (kTile / Q);
            nd[q].zero(), ng[q].zero(), nz[q].zero();
            if (live && tt < t1) {
                nd[q].load(de + tt * P.d_ts);
                ng[q].load(dy + (size_t)tt * P.D);
                if (z) nz[q].load(z + tt * P.z_ts);
            }
        }
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int e = tid + q * THREADS, tt = t + e / (NP / 4), n = e % (NP / 4) * 4;
            nc[q].load(Cm + tt * P.c_ts + n, e < IB && tt < t1 ? P.N - n : 0);
        }
    };
    const int last = t0 + (t1 - 1 - t0) / kTile * kTile;
    if (t0 < t1) fetch(last);
    for (int t = last; t >= t0 && t1 > t0; t -= kTile) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int k = lt + q * (kTile / Q);
            const bool in = live && t + k < t1;
            float fd[V], fg[V], fz[V];
            nd[q].get(fd), ng[q].get(fg), nz[q].get(fz);
#pragma unroll
            for (int i = 0; i < V; ++i) fd[i] += bias[i];
            if (P.softplus) softplus_all<PRECISE>(fd);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (z) fg[i] *= fz[i] * sigmoid<GATE>(fz[i]);
                fd[i] = in ? fd[i] : 0.f, fg[i] = in ? fg[i] : 0.f;
            }
            put_pairs<V>(&s_dd[k][lc - c0], fd, fg);
        }
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int e = tid + q * THREADS;
            if (e < IB) nc[q].put(&s_C[0][0] + 4 * e);
        }
        __syncthreads();
        if (t - kTile >= t0) fetch(t - kTile);
        float part = 0.f;
#pragma unroll
        for (int k = kTile - 1; k >= 0; --k) {
            const float2 dd = s_dd[k][cl], d2 = make_float2(dd.x, dd.x), e2 = make_float2(dd.y, dd.y);
            float2 C[2];
            shared_n(&s_C[k][ns], C);
#pragma unroll
            for (int j = 0; j < 2; ++j) w[j] = __fmul2_rn(decay(d2, a2[j]), __ffma2_rn(e2, C[j], w[j]));
            part += dd.x;
        }
        sum += part;
        __syncthreads();
    }
    if (cs >= c1) return;
    const size_t at = ((size_t)seg * P.B + b) * P.D + cs;
    store_state(K.seg_g + at * P.N, P.N, ns, w);
    if (nl == 0) K.seg_dt[at] = (float)sum;
}

// Adjoints behind the segments, in place of their own parts, last to first.
__global__ void __launch_bounds__(256)
ssm_bwd_chain_kernel(long long total, int N, int nseg, const float *__restrict__ A, long long D,
                     const float *__restrict__ dstateT, const float *__restrict__ seg_dt, float *__restrict__ seg_g) {
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= total) return;
    const long long ch = id / N;
    const float a = __ldg(A + (ch % D) * N + id % N) * kLog2e;
    float w = dstateT ? dstateT[id] : 0.f;
    const long long chans = total / N;
    for (int s = nseg - 1; s >= 0; --s) {
        const float e = seg_g[s * total + id];
        seg_g[s * total + id] = w;
        w = fmaf(ex2(a * __ldg(seg_dt + s * chans + ch)), w, e);
    }
}

constexpr int kBwdThreads = 128, kBwdTC = 2;        // channels a thread
__host__ __device__ constexpr int bwd_channels(int NP) { return kBwdTC * kBwdThreads * 4 / NP; }     // of a block

// slots <-> n: slot j holds n = j xor p, p = 0 .. 3; its own inverse
__device__ __forceinline__ void permute(float2 (&v)[2], int p) {
    const float2 a = v[0], b = v[1];
    const float2 x = (p & 2) ? b : a, y = (p & 2) ? a : b;
    v[0] = (p & 1) ? make_float2(x.y, x.x) : x;
    v[1] = (p & 1) ? make_float2(y.y, y.x) : y;
}

// Shared memory of a block, in floats
template <typename T, int NP> struct BwdShared {
    static constexpr int CC = bwd_channels(NP), LN = NP / 4, WARPS = kBwdThreads / 32;
    using Sum = Planes<CC, LN>;
    static constexpr int DD = 0;                                // [kTile][CC] dt, dt u
    static constexpr int DS = DD + 2 * kTile * CC;              // [kTile][CC]
    static constexpr int BC = DS + kTile * CC;                  // T [2][kTile][4][NP]: each token's n in four orders
    static constexpr int Y = BC + 2 * kTile * 4 * NP * (int)sizeof(T) / 4;      // C . h, lane by lane
    static constexpr int GB = Y + Sum::FLOATS;                  // g . B
    static constexpr int AP = GB + Sum::FLOATS;                 // A . p g
    static constexpr int PART = AP + Sum::FLOATS;               // [WARPS][kTile][2][NP] dB, dC
    static constexpr int DA = PART + WARPS * kTile * 2 * NP;    // [8 TC][threads]: sums and their errors
    static constexpr int ACC = DA + 8 * kBwdTC * kBwdThreads;   // [2 V][threads]: dD, ddt_bias
    static constexpr int FLOATS = ACC + 2 * 4 * kBwdThreads;
};

template <typename T, int NP, bool VEC, bool GATE>
__global__ void __launch_bounds__(kBwdThreads, 2)         // 255 registers; N > 32: shared memory for one
ssm_bwd_kernel(const BwdArgs K) {
    const ScanArgs &P = K.f;
    using S = BwdShared<T, NP>;
    using Sum = typename S::Sum;
    constexpr int CC = S::CC, LN = S::LN, CG = 32 / LN, THREADS = kBwdThreads;      // CG channels a warp
    constexpr int TC = kBwdTC, EPT = kTile * CC / THREADS, V = VEC ? (EPT < 4 ? EPT : 4) : 1, Q = EPT / V;
    constexpr int IB = 2 * kTile * NP / 4, NB = (IB + THREADS - 1) / THREADS;
    constexpr bool PRECISE = sizeof(T) == 4;
    extern __shared__ __align__(16) float smem[];
    float2(*s_dd)[CC] = reinterpret_cast<float2(*)[CC]>(smem + S::DD);
    float(*s_ds)[CC] = reinterpret_cast<float(*)[CC]>(smem + S::DS);
    T(*s_BC)[kTile][4][NP] = reinterpret_cast<T(*)[kTile][4][NP]>(smem + S::BC);
    float *s_y = smem + S::Y, *s_gb = smem + S::GB, *s_ap = smem + S::AP;
    float(*s_part)[kTile][2][NP] = reinterpret_cast<float(*)[kTile][2][NP]>(smem + S::PART);
    float *s_dA = smem + S::DA, *s_acc = smem + S::ACC;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned id = blockIdx.x;
    const int tile_c = (int)(id % (unsigned)P.tiles);
    id /= (unsigned)P.tiles;
    const int g = (int)(id % (unsigned)P.G);
    id /= (unsigned)P.G;
    const long long b = id % (unsigned)P.B;
    const int seg = (int)(id / (unsigned)P.B);
    const int c0 = g * P.Dg + tile_c * CC, c1 = (g + 1) * P.Dg;
    const int t0 = (int)min((long long)seg * P.seg_len, (long long)P.T);
    const int t1 = (int)min((long long)t0 + P.seg_len, (long long)P.T);

    const int lc = c0 + (tid % (CC / V)) * V, lt = tid / (CC / V);
    const bool live = lc < c1;
    const T *u = static_cast<const T *>(P.u) + b * P.u_bs + lc, *de = static_cast<const T *>(P.delta) + b * P.d_bs + lc;
    const T *z = P.z ? static_cast<const T *>(P.z) + b * P.z_bs + lc : nullptr;
    const T *dy = static_cast<const T *>(K.dy) + (size_t)b * P.T * P.D + lc;
    const T *Bm = static_cast<const T *>(P.Bm) + b * P.b_bs + g * P.N;
    const T *Cm = static_cast<const T *>(P.Cm) + b * P.c_bs + g * P.N;
    float bias[V], skip[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = (live && P.dt_bias) ? __ldg(P.dt_bias + lc + i) : 0.f;
        skip[i] = (live && P.Dskip) ? __ldg(P.Dskip + lc + i) : 0.f;
    }

    const int nl = tid % LN, cl = tid / LN * TC, cs = c0 + cl, ns = 4 * nl, cg = lane / LN, order = cg & 3;
    float2 a2[TC][2], w[TC][2];     // rates (log2), adjoint carried to the token before; by slots
#pragma unroll
    for (int c = 0; c < TC; ++c) {
        const bool mine = cs + c < c1;
        load_rates(P.A + (size_t)(cs + c) * P.N, P.N, ns, mine, a2[c]);
        permute(a2[c], order);
        w[c][0] = w[c][1] = make_float2(0.f, 0.f);
        if (mine && K.exit) load_state(K.exit + (((size_t)seg * P.B + b) * P.D + cs + c) * P.N, P.N, ns, w[c]);
        permute(w[c], order);
    }
    for (int i = 0; i < 2 * V; ++i) s_acc[i * THREADS + tid] = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * TC; ++i) s_dA[i * THREADS + tid] = 0.f;

    Vec<T, V> nu[Q], nd[Q], nz[Q], ng[Q], cu[Q], cd[Q], cz[Q], cy[Q];
    Quad<T, VEC> nb[NB];
    float2 h0[TC][2];
    auto fetch = [&](int t) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int tt = t + lt + q * (kTile / Q);
            nu[q].zero(), nd[q].zero(), nz[q].zero(), ng[q].zero();
            if (live && tt < t1) {
                nu[q].load(u + tt * P.u_ts);
                nd[q].load(de + tt * P.d_ts);
                ng[q].load(dy + (size_t)tt * P.D);
                if (z) nz[q].load(z + tt * P.z_ts);
            }
        }
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int e = tid + q * THREADS, tt = t + (e / (NP / 4)) % kTile, n = e % (NP / 4) * 4;
            nb[q].load((e >= IB / 2 ? Cm + tt * P.c_ts : Bm + tt * P.b_ts) + n, e < IB && tt < t1 ? P.N - n : 0);
        }
    };
    auto prepare = [&](int t) {     // tokens behind t1: dt = dt u = ds = B = C = 0 change nothing
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int k = lt + q * (kTile / Q), ch = lc - c0;
            const bool in = live && t + k < t1;
            float fu[V], fd[V], fz[V], fg[V];
            nu[q].get(fu), nd[q].get(fd), nz[q].get(fz), ng[q].get(fg);
#pragma unroll
            for (int i = 0; i < V; ++i) fd[i] += bias[i];
            if (P.softplus) softplus_all<PRECISE>(fd);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (z) fg[i] *= fz[i] * sigmoid<GATE>(fz[i]);
                fd[i] = in ? fd[i] : 0.f, fu[i] = in ? fd[i] * fu[i] : 0.f, fg[i] = in ? fg[i] : 0.f;
            }
            put_pairs<V>(&s_dd[k][ch], fd, fu);
            storev<V>(&s_ds[k][ch], fg);
            cu[q] = nu[q], cd[q] = nd[q], cz[q] = nz[q], cy[q] = ng[q];
        }
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int e = tid + q * THREADS;
            if (e >= IB) continue;
            T *to = &s_BC[e / (IB / 2)][(e / (NP / 4)) % kTile][0][e % (NP / 4) * 4];
#pragma unroll
            for (int p = 0; p < 4; ++p) nb[q].put(to + p * NP, p);
        }
#pragma unroll
        for (int c = 0; c < TC; ++c) {
            h0[c][0] = h0[c][1] = make_float2(0.f, 0.f);
            if (cs + c < c1)
                load_state(P.states + ((size_t)(b * P.nck + t / kTile) * P.D + cs + c) * P.N, P.N, ns, h0[c]);
            permute(h0[c], order);
        }
    };

    const int last = t0 + (t1 - 1 - t0) / kTile * kTile;
    if (t0 < t1) {
        fetch(last);
        prepare(last);
        __syncthreads();
    }
    for (int t = last; t >= t0 && t1 > t0; t -= kTile) {
        if (t - kTile >= t0) fetch(t - kTile);

        float2 dA[TC][2];
#pragma unroll
        for (int c = 0; c < TC; ++c) dA[c][0] = dA[c][1] = make_float2(0.f, 0.f);
        auto steps = [&](int k, float2 (&d2)[TC], float2 (&v2)[TC]) {      // dt and dt u of this thread's channels
            const float4 q = *reinterpret_cast<const float4 *>(&s_dd[k][cl]);
            d2[0] = make_float2(q.x, q.x), v2[0] = make_float2(q.y, q.y);
            d2[1] = make_float2(q.z, q.z), v2[1] = make_float2(q.w, q.w);
        };
#pragma unroll 1
        for (int half = kTile / 2; half >= 0; half -= kTile / 2) {
        // ---- replay: the state up to the half, then every h of it
        float2 h[kTile / 2][TC][2], hs[TC][2];
#pragma unroll
        for (int c = 0; c < TC; ++c) hs[c][0] = h0[c][0], hs[c][1] = h0[c][1];
        auto advance = [&](int k, const float2 (&from)[TC][2], float2 (&to)[TC][2]) {
            float2 d2[TC], v2[TC], B[2];
            steps(k, d2, v2);
            shared_n(&s_BC[0][k][order][ns], B);
#pragma unroll
            for (int c = 0; c < TC; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    to[c][j] = __ffma2_rn(decay(d2[c], a2[c][j]), from[c][j], __fmul2_rn(v2[c], B[j]));
        };
        if (half) {
#pragma unroll
            for (int k = 0; k < kTile / 2; ++k) advance(k, hs, hs);
        }
#pragma unroll
        for (int k = 0; k < kTile / 2; ++k) advance(half + k, k ? h[k - 1] : hs, h[k]);

        // ---- the way back
#pragma unroll
        for (int i = kTile / 2 - 1; i >= 0; --i) {
            const int k = half + i;
            float2 d2[TC], v2[TC], B[2], C[2], dB[2], dC[2];
            steps(k, d2, v2);
            const float2 e = *reinterpret_cast<const float2 *>(&s_ds[k][cl]);
            const float2 e2[TC] = {make_float2(e.x, e.x), make_float2(e.y, e.y)};
            shared_n(&s_BC[0][k][order][ns], B);
            shared_n(&s_BC[1][k][order][ns], C);
            if (z) {
                float yc[TC];
#pragma unroll
                for (int c = 0; c < TC; ++c) {
                    const float2 y = __ffma2_rn(h[i][c][1], C[1], __fmul2_rn(h[i][c][0], C[0]));
                    yc[c] = y.x + y.y;
                }
                Sum::template put<TC>(s_y, k, cl, nl, yc);
            }
            float gbs[TC], aps[TC];
#pragma unroll
            for (int c = 0; c < TC; ++c) {
                float2 gg[2], q[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 a = decay(d2[c], a2[c][j]);
                    gg[j] = __ffma2_rn(e2[c], C[j], w[c][j]);
                    w[c][j] = __fmul2_rn(a, gg[j]);
                    q[j] = __fmul2_rn(w[c][j], i ? h[i ? i - 1 : 0][c][j] : hs[c][j]);      // p g
                    dA[c][j] = __ffma2_rn(q[j], d2[c], dA[c][j]);
                    dB[j] = c ? __ffma2_rn(v2[c], gg[j], dB[j]) : __fmul2_rn(v2[c], gg[j]);
                    dC[j] = c ? __ffma2_rn(e2[c], h[i][c][j], dC[j]) : __fmul2_rn(e2[c], h[i][c][j]);
                }
                const float2 gb = __ffma2_rn(gg[1], B[1], __fmul2_rn(gg[0], B[0]));
                const float2 ap = __ffma2_rn(q[1], a2[c][1], __fmul2_rn(q[0], a2[c][0]));
                gbs[c] = gb.x + gb.y, aps[c] = ap.x + ap.y;
            }
            Sum::template put<TC>(s_gb, k, cl, nl, gbs);
            Sum::template put<TC>(s_ap, k, cl, nl, aps);
            // over the warp's channels: lanes LN apart whose orders differ in one bit
            float bc[2][4] = {{dB[0].x, dB[0].y, dB[1].x, dB[1].y}, {dC[0].x, dC[0].y, dC[1].x, dC[1].y}};
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                bc[m][0] += __shfl_xor_sync(0xffffffffu, bc[m][1], LN);
                bc[m][2] += __shfl_xor_sync(0xffffffffu, bc[m][3], LN);
                if constexpr (CG >= 4) bc[m][0] += __shfl_xor_sync(0xffffffffu, bc[m][2], 2 * LN);
            }
            float *to = &s_part[warp][k][0][ns + order];
            if constexpr (CG >= 8) {            // one of dB and dC a lane
                const bool up = cg & 4;
                const float give = up ? bc[0][0] : bc[1][0];
                float r = (up ? bc[1][0] : bc[0][0]) + __shfl_xor_sync(0xffffffffu, give, 4 * LN);
                if constexpr (CG == 16) r += __shfl_xor_sync(0xffffffffu, r, 8 * LN);
                if (CG == 8 || cg < 8) to[up ? NP : 0] = r;
            } else if constexpr (CG == 4) {
                to[0] = bc[0][0];
                to[NP] = bc[1][0];
            } else {                            // two lanes a group: n = order and order xor 2
                to[0] = bc[0][0];
                to[NP] = bc[1][0];
                float *other = &s_part[warp][k][0][ns + (order ^ 2)];
                other[0] = bc[0][2];
                other[NP] = bc[1][2];
            }
        }
        }
        // the tile's part of dA, into a sum with its rounding error kept (two-sum)
#pragma unroll
        for (int c = 0; c < TC; ++c) {
            const float tile_dA[4] = {dA[c][0].x, dA[c][0].y, dA[c][1].x, dA[c][1].y};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float *at = s_dA + (8 * c + 2 * i) * THREADS + tid;
                const float s = at[0], x = tile_dA[i], n = s + x, v = n - s;
                at[0] = n;
                at[THREADS] += (s - (n - v)) + (x - v);
            }
        }
        __syncthreads();

        // ---- outputs of the tile
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int k = lt + q * (kTile / Q), ch = lc - c0;
            if (!live || t + k >= t1) continue;
            float fu[V], fd[V], fz[V], fg[V], odu[V], odd[V], odz[V];
            cu[q].get(fu), cd[q].get(fd), cz[q].get(fz), cy[q].get(fg);
            float gb[V], ap[V], yc[V];
            Sum::template sum<V>(s_gb, k, ch, gb);
            Sum::template sum<V>(s_ap, k, ch, ap);
            if (z) Sum::template sum<V>(s_y, k, ch, yc);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float ds = s_ds[k][ch + i], dt = s_dd[k][ch + i].x;
                odu[i] = fmaf(dt, gb[i], skip[i] * ds);
                float dd = fmaf(fu[i], gb[i], ap[i] * 0.6931471805599453f);     // a2 is in units of log 2
                if (P.softplus) dd *= sigmoid<GATE>(fd[i] + bias[i]);
                odd[i] = dd;
                s_acc[i * THREADS + tid] += ds * fu[i];
                s_acc[(V + i) * THREADS + tid] += dd;
                if (z) {
                    const float sg = sigmoid<GATE>(fz[i]);
                    odz[i] = fg[i] * fmaf(skip[i], fu[i], yc[i]) *
                             (sg * fmaf(fz[i], 1.f - sg, 1.f));
                }
            }
            const size_t at = ((size_t)b * P.T + t + k) * P.D + lc;
            if (K.g_f32) {
                storev<V>(static_cast<float *>(K.du) + at, odu);
                storev<V>(static_cast<float *>(K.ddelta) + at, odd);
                if (z) storev<V>(static_cast<float *>(K.dz) + at, odz);
            } else {
                storev<V>(static_cast<bf16 *>(K.du) + at, odu);
                storev<V>(static_cast<bf16 *>(K.ddelta) + at, odd);
                if (z) storev<V>(static_cast<bf16 *>(K.dz) + at, odz);
            }
        }
        const size_t bt = (size_t)P.B * P.T * P.G * P.N;
        for (int e = tid; e < kTile * 2 * NP; e += THREADS) {
            const int which = e / (kTile * NP), k = (e / NP) % kTile, n = e % NP;
            if (t + k >= t1 || n >= P.N) continue;
            float s = s_part[0][k][which][n];
#pragma unroll
            for (int i = 1; i < S::WARPS; ++i) s += s_part[i][k][which][n];
            K.dbc[((size_t)tile_c * 2 + which) * bt + (((size_t)b * P.T + t + k) * P.G + g) * P.N + n] = s;
        }
        if (t - kTile >= t0) prepare(t - kTile);
        __syncthreads();
    }

    const size_t part = (size_t)seg * P.B + b;
#pragma unroll
    for (int c = 0; c < TC; ++c) {
        if (cs + c >= c1) continue;
        permute(w[c], order);
        if (seg == 0 && K.dstate0) store_state(K.dstate0 + ((size_t)b * P.D + cs + c) * P.N, P.N, ns, w[c]);
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = s_dA[(8 * c + 2 * i) * THREADS + tid] + s_dA[(8 * c + 2 * i + 1) * THREADS + tid];
        float2 v2[2] = {make_float2(v[0], v[1]), make_float2(v[2], v[3])};
        permute(v2, order);
        store_state(K.dA + (part * P.D + cs + c) * P.N, P.N, ns, v2);
    }
    // dD and ddt_bias: the threads that loaded the same channels, in order
    __syncthreads();
    constexpr int PER = CC / V;
    for (int e = tid; e < 2 * CC; e += THREADS) {
        const int which = e / CC, ch = e % CC;
        if (c0 + ch >= c1) continue;
        float s = 0.f;
        for (int i = 0; i < THREADS / PER; ++i) s += s_acc[(which * V + ch % V) * THREADS + i * PER + ch / V];
        K.dpar[((size_t)which * P.nseg * P.B + part) * P.D + c0 + ch] = s;
    }
}

// dB and dC from the channel blocks' partial sums
template <typename GT>
__global__ void __launch_bounds__(256)
ssm_dbc_kernel(long long n, int tiles, const float *__restrict__ partial, GT *__restrict__ dB, GT *__restrict__ dC) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= 2 * n) return;
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < tiles; ++k) s += __ldg(partial + 2 * n * k + i);
    if (i < n) dB[i] = from_f32<GT>(s);
    else dC[i - n] = from_f32<GT>(s);
}

template <typename T, int NP, bool VEC, bool GATE>
cudaError_t launch_bwd(const BwdArgs &K, const float *dstateT, cudaStream_t st) {
    const ScanArgs &P = K.f;
    BwdArgs M = K;
    M.exit = dstateT;
    if (P.nseg > 1) {
        const long long blocks = (long long)P.nseg * P.B * P.G * ((P.Dg + scan_channels(NP) - 1) / scan_channels(NP));
        ssm_bwd_summary_kernel<T, NP, VEC, GATE><<<(unsigned)blocks, scan_threads(NP, 1), 0, st>>>(K);
        const long long total = (long long)P.B * P.D * P.N;
        ssm_bwd_chain_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(total, P.N, P.nseg, P.A, P.D, dstateT,
                                                                             K.seg_dt, K.seg_g);
        M.exit = K.seg_g;
    }
    constexpr size_t smem = BwdShared<T, NP>::FLOATS * sizeof(float);
    auto kernel = ssm_bwd_kernel<T, NP, VEC, GATE>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)((long long)P.nseg * P.B * P.G * P.tiles), kBwdThreads, smem, st>>>(M);
    return cudaGetLastError();
}

int bwd_tiles(int D, int N, int G) {
    const int CC = bwd_channels(scan_pad(N));
    return (D / G + CC - 1) / CC;
}
// Segments of a backward: two blocks an SM, if that makes at least two segments
// (whose summaries cost about a fifth of a pass), each of at least 64 tokens.
// N = 16, segments against one piece: 4 x 4096 x 2048 1.21 / 1.52 ms, 1 x 4096 x
// 2048 0.30 / 1.45 ms, 1 x 256 x 2048 78 / 112 us.  (Two blocks fit up to N = 32; above
// that a block's shared memory, 120 KB and more, leaves room for one, and the
// segments run in two waves.)
int bwd_segments(int B, int T, int D, int N, int G, int sms) {
    const long long blocks = (long long)B * G * bwd_tiles(D, N, G);
    if (blocks <= 0 || sms <= 0) return 1;
    const long long want = (long long)sms * 2 / blocks, most = T / 64;
    const long long s = want < most ? want : most;
    return s >= 2 ? (int)s : 1;
}

struct BwdSpace {
    size_t states, fwd, dbc, dA, dpar, seg, total;
    int nseg, fseg;
};
BwdSpace bwd_space(int B, int T, int D, int N, int G, bool with_states) {
    BwdSpace w{};
    const int sms = sm_count(), tiles = bwd_tiles(D, N, G);
    w.nseg = bwd_segments(B, T, D, N, G, sms);
    w.fseg = ssm_segments(B, T, D, N, G, sms);
    w.states = with_states ? 0 : round256((size_t)B * ((T + kTile - 1) / kTile) * D * N * 4);
    w.fwd = with_states ? 0 : ssm_segment_bytes(B, D, N, w.fseg);
    w.dbc = round256((size_t)tiles * 2 * B * T * G * N * 4);
    w.dA = round256((size_t)w.nseg * B * D * N * 4);
    w.dpar = round256((size_t)2 * w.nseg * B * D * 4);
    w.seg = ssm_segment_bytes(B, D, N, w.nseg);
    w.total = w.states + w.fwd + w.dbc + w.dA + w.dpar + w.seg;
    return w;
}

}  // namespace
}  // namespace mixer
}  // namespace wkv7

extern "C" {

size_t wkv7_ssm_backward_workspace_size(int B, int T, int D, int N, int G, int with_states) {
    using namespace wkv7::mixer;
    if (B <= 0 || T <= 0 || D <= 0 || ssm_dims(B, T, D, N, G) != WKV7_OK) return 0;
    return bwd_space(B, T, D, N, G, with_states != 0).total;
}

wkv7_status wkv7_ssm_backward(int B, int T, int D, int N, int G, wkv7_dtype in_dt, wkv7_dtype g_dt, const void *u,
                              long long u_bs, long long u_ts, const void *delta, long long d_bs, long long d_ts,
                              const float *A, const void *Bm, long long b_bs, long long b_ts, const void *Cm,
                              long long c_bs, long long c_ts, const float *Dskip, const void *z, long long z_bs,
                              long long z_ts, const float *dt_bias, const float *state0, int softplus,
                              const float *states, const void *dy, const float *dstateT, void *du, void *ddelta,
                              float *dA, void *dB, void *dC, float *dD, void *dz, float *ddt_bias, float *dstate0,
                              void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace wkv7::mixer;
    const wkv7_status s = ssm_dims(B, T, D, N, G);
    if (s != WKV7_OK) return s;
    if (!real_dtype(in_dt) || !real_dtype(g_dt)) return WKV7_ERR_INVALID_ARG;
    for (long long v : {u_bs, u_ts, d_bs, d_ts, b_bs, b_ts, c_bs, c_ts, z_bs, z_ts})
        if (v < 0) return WKV7_ERR_INVALID_ARG;
    if (!aligned_to(state0, 16) || !aligned_to(dstateT, 16) || !aligned_to(states, 16) || !aligned_to(dstate0, 16) ||
        !f32_opt(dD) || !f32_opt(ddt_bias))
        return WKV7_ERR_INVALID_ARG;
    if (D == 0) return WKV7_OK;
    if (!f32_ok(dA)) return WKV7_ERR_INVALID_ARG;
    if (B == 0 || T == 0) {
        cudaError_t e = cudaMemsetAsync(dA, 0, (size_t)D * N * 4, stream);
        if (e == cudaSuccess && dD) e = cudaMemsetAsync(dD, 0, (size_t)D * 4, stream);
        if (e == cudaSuccess && ddt_bias) e = cudaMemsetAsync(ddt_bias, 0, (size_t)D * 4, stream);
        const size_t n = (size_t)B * D * N * 4;
        if (e == cudaSuccess && dstate0 && n && dstate0 != dstateT)
            e = dstateT ? cudaMemcpyAsync(dstate0, dstateT, n, cudaMemcpyDeviceToDevice, stream)
                        : cudaMemsetAsync(dstate0, 0, n, stream);
        return e == cudaSuccess ? WKV7_OK : WKV7_ERR_CUDA;
    }
    if (!elem_ok(u, in_dt) || !elem_ok(delta, in_dt) || !elem_ok(Bm, in_dt) || !elem_ok(Cm, in_dt) ||
        !aligned_to(z, dtype_size(in_dt)) || !f32_ok(A) || !f32_opt(Dskip) || !f32_opt(dt_bias) ||
        !elem_ok(dy, in_dt) || !elem_ok(du, g_dt) || !elem_ok(ddelta, g_dt) || !elem_ok(dB, g_dt) ||
        !elem_ok(dC, g_dt) || (z != nullptr) != (dz != nullptr) || !aligned_to(dz, dtype_size(g_dt)))
        return WKV7_ERR_INVALID_ARG;
    const BwdSpace w = bwd_space(B, T, D, N, G, states != nullptr);
    if (workspace == nullptr || !aligned_to(workspace, 16) || workspace_bytes < w.total) return WKV7_ERR_INVALID_ARG;
    char *ws = (char *)workspace;
    auto take = [&](size_t n) {
        char *p = ws;
        ws += n;
        return p;
    };
    BwdArgs K{};
    ScanArgs &P = K.f;
    P.B = B, P.T = T, P.D = D, P.N = N, P.G = G, P.Dg = D / G;
    P.u = u, P.u_bs = u_bs, P.u_ts = u_ts, P.delta = delta, P.d_bs = d_bs, P.d_ts = d_ts;
    P.z = z, P.z_bs = z_bs, P.z_ts = z_ts;
    P.Bm = Bm, P.b_bs = b_bs, P.b_ts = b_ts, P.Cm = Cm, P.c_bs = c_bs, P.c_ts = c_ts;
    P.A = A, P.Dskip = Dskip, P.dt_bias = dt_bias, P.softplus = softplus;
    P.nck = (T + kTile - 1) / kTile;
    const bool vec = ssm_vec(P, in_dt) && aligned_to(dy, 16) && aligned_to(du, 16) && aligned_to(ddelta, 16) && aligned_to(dz, 16);
    if (states == nullptr) {
        P.states = (float *)take(w.states);
        P.tiles = (P.Dg + scan_channels(scan_pad(N)) - 1) / scan_channels(scan_pad(N));
        ssm_fwd_all(P, state0, w.fseg, take(w.fwd), in_dt, vec, false, stream);
    } else {
        P.states = const_cast<float *>(states);         // read only from here on
    }
    K.dbc = (float *)take(w.dbc), K.dA = (float *)take(w.dA), K.dpar = (float *)take(w.dpar);
    if (w.nseg > 1) {
        K.seg_g = (float *)take(round256((size_t)w.nseg * B * D * N * 4));
        K.seg_dt = (float *)take(round256((size_t)w.nseg * B * D * 4));
    }
    P.nseg = w.nseg, P.tiles = bwd_tiles(D, N, G);
    P.seg_len = (int)((((long long)T + w.nseg - 1) / w.nseg + kTile - 1) / kTile * kTile);
    K.dy = dy, K.g_f32 = g_dt == WKV7_F32, K.du = du, K.ddelta = ddelta, K.dz = dz, K.dstate0 = dstate0;
    cudaError_t e = cudaSuccess;
    by_pad(scan_pad(N), [&](auto np) {
        constexpr int NP = decltype(np)::value;
        auto launch = [&](auto t) {
            using T = decltype(t);
            by_precision<T>(K.g_f32, [&](auto gate) {
                constexpr bool GATE = decltype(gate)::value;
                e = vec ? launch_bwd<T, NP, true, GATE>(K, dstateT, stream) : launch_bwd<T, NP, false, GATE>(K, dstateT, stream);
            });
        };
        if (in_dt == WKV7_F32) launch(float());
        else launch(bf16());
    });
    if (e != cudaSuccess) return WKV7_ERR_CUDA;
    const long long n = (long long)B * T * G * N;
    const unsigned grid = (unsigned)((2 * n + 255) / 256);
    if (g_dt == WKV7_F32) ssm_dbc_kernel<float><<<grid, 256, 0, stream>>>(n, P.tiles, K.dbc, (float *)dB, (float *)dC);
    else ssm_dbc_kernel<bf16><<<grid, 256, 0, stream>>>(n, P.tiles, K.dbc, (bf16 *)dB, (bf16 *)dC);
    const long long parts = (long long)w.nseg * B;
    sum_parts(parts, (long long)D * N, K.dA, dA, stream);
    if (dD) sum_parts(parts, D, K.dpar, dD, stream);
    if (ddt_bias) sum_parts(parts, D, K.dpar + parts * D, ddt_bias, stream);
    return launch_status();
}

}  // extern "C"
