// Backward of the selective scan (wkv7_ssm_backward).
//
//     ds_t = dy_t z sigmoid(z),     g_t = C_t ds_t + exp(dt_{t+1} A) g_{t+1}
//     p_t = exp(dt_t A) h_{t-1}
//     dC_t = sum_d ds_t h_t         dB_t = sum_d g_t dt_t u_t
//     du_t = dt_t sum_n g_t B_t + D ds_t
//     d(dt)_t = u_t sum_n g_t B_t + sum_n A p_t g_t,   ddelta = d(dt) softplus'
//     dA = sum_t dt_t p_t g_t       dD = sum ds u       dz = dy s (z sigmoid(z))'
//
// Layout as in the forward (2 channels x 4 n a thread, tiles of 16 tokens).  A
// block walks its tiles from the last to the first.  For each it starts from the
// state saved before the tile, replays the 16 tokens with every h in registers
// (128 of them, both loops unrolled), then runs the adjoint back over them.
// Bound: two exponentials per (token, channel, n), one a replay and one a way
// back, and about 200 multiply-adds a channel-token at N = 16.
//
// dB and dC join channels: 8 values over the lanes of a warp that share n,
// scattered while they are summed (7 exchanges for 8 lanes); the block's warps
// join in shared memory, the blocks through partial sums added up in order by a
// second kernel.  Few channels over many tokens: segments, as in the forward
// (summaries from a zero adjoint, a chain from the last segment to the first).
#include "ssm.cuh"

namespace wkv7 {
namespace mixer {

void sum_parts(long long parts, long long cols, const float *partial, float *out, cudaStream_t st);
wkv7_status ssm_dims(int B, int T, int D, int N, int G);
int ssm_segments(int B, int T, int D, int N, int G, int sms);
size_t ssm_segment_bytes(int B, int D, int N, int nseg);
void ssm_fwd_all(ScanArgs P, const float *state0, int nseg, char *ws, wkv7_dtype dt, bool vec, bool y,
                 cudaStream_t st);
bool ssm_vec(const ScanArgs &P, wkv7_dtype dt, const void *more, size_t more_size);

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

template <typename T, int LN, int V>
__global__ void __launch_bounds__(kScanThreads)
ssm_bwd_summary_kernel(const BwdArgs K) {
    const ScanArgs &P = K.f;
    constexpr int CC = scan_channels(LN), NP = 4 * LN;
    constexpr int EPT = kTile * CC / kScanThreads, Q = EPT / V, NB = kTile * NP / kScanThreads;
    constexpr bool PRECISE = sizeof(T) == 4;
    __shared__ __align__(16) float s_dt[kTile][CC], s_ds[kTile][CC];
    __shared__ float4 s_C[kTile][LN];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long id = blockIdx.x;
    const int tile_c = (int)(id % P.tiles);
    id /= P.tiles;
    const int g = (int)(id % P.G);
    id /= P.G;
    const long long b = id % P.B;
    const int seg = (int)(id / P.B);
    const int c0 = g * P.Dg + tile_c * CC, c1 = (g + 1) * P.Dg;
    const int t0 = (int)min((long long)seg * P.seg_len, (long long)P.T);
    const int t1 = (int)min((long long)t0 + P.seg_len, (long long)P.T);
    const int lc = c0 + (tid % (CC / V)) * V, lt = tid / (CC / V);
    const bool live = lc < c1;
    const T *de = static_cast<const T *>(P.delta) + b * P.d_bs + lc;
    const T *z = P.z ? static_cast<const T *>(P.z) + b * P.z_bs + lc : nullptr;
    const T *dy = static_cast<const T *>(K.dy) + (size_t)b * P.T * P.D + lc;
    const T *Cm = static_cast<const T *>(P.Cm) + b * P.c_bs + g * P.N;
    const int nl = lane % LN, cl = (warp * (32 / LN) + lane / LN) * 2, cs = c0 + cl, ns = 4 * nl;
    float2 a2[2][2], w[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float av[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
            av[n] = (cs + c < c1 && ns + n < P.N) ? __ldg(P.A + (size_t)(cs + c) * P.N + ns + n) * kLog2e : 0.f;
        a2[c][0] = make_float2(av[0], av[1]), a2[c][1] = make_float2(av[2], av[3]);
        w[c][0] = w[c][1] = make_float2(0.f, 0.f);
    }
    double sum0 = 0, sum1 = 0;
    for (int t = t0 + (t1 - 1 - t0) / kTile * kTile; t >= t0 && t1 > t0; t -= kTile) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int k = lt + q * (kTile / Q), tt = t + k;
            float fd[V], fg[V];
#pragma unroll
            for (int i = 0; i < V; ++i) fd[i] = fg[i] = 0.f;
            if (live && tt < t1) {
                Vec<T, V> d, e, v;
                d.load(de + tt * P.d_ts);
                e.load(dy + (size_t)tt * P.D);
                v.zero();
                if (z) v.load(z + tt * P.z_ts);
                float fz[V];
                d.get(fd), e.get(fg), v.get(fz);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float x = fd[i] + (P.dt_bias ? __ldg(P.dt_bias + lc + i) : 0.f);
                    fd[i] = P.softplus ? softplus(x) : x;
                    if (z) fg[i] *= fz[i] * sigmoid<PRECISE>(fz[i]);
                }
            }
            storev<V>(&s_dt[k][lc - c0], fd);
            storev<V>(&s_ds[k][lc - c0], fg);
        }
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int e = tid + q * kScanThreads, tt = t + e / NP, n = e % NP;
            reinterpret_cast<float *>(s_C)[e] = (tt < t1 && n < P.N) ? to_f32(Cm[tt * P.c_ts + n]) : 0.f;
        }
        __syncthreads();
        float part0 = 0.f, part1 = 0.f;
#pragma unroll 2
        for (int k = kTile - 1; k >= 0; --k) {
            const float2 dt = *reinterpret_cast<const float2 *>(&s_dt[k][cl]);
            const float2 ds = *reinterpret_cast<const float2 *>(&s_ds[k][cl]);
            const float4 C = s_C[k][nl];
            const float2 C2[2] = {make_float2(C.x, C.y), make_float2(C.z, C.w)};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float d = c ? dt.y : dt.x, e = c ? ds.y : ds.x;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    w[c][j] = __fmul2_rn(ex2(__fmul2_rn(make_float2(d, d), a2[c][j])),
                                         __ffma2_rn(make_float2(e, e), C2[j], w[c][j]));
            }
            part0 += dt.x, part1 += dt.y;
        }
        sum0 += part0, sum1 += part1;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (cs + c >= c1) continue;
        const size_t at = ((size_t)seg * P.B + b) * P.D + cs + c;
        store_state(K.seg_g + at * P.N + ns, P.N, ns, w[c]);
        if (nl == 0) K.seg_dt[at] = (float)(c ? sum1 : sum0);
    }
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

template <typename T, int LN, int V>
__global__ void __launch_bounds__(kScanThreads, 2)
ssm_bwd_kernel(const BwdArgs K) {
    const ScanArgs &P = K.f;
    constexpr int CC = scan_channels(LN), NP = 4 * LN, CG = 32 / LN;    // CG channel pairs a warp
    constexpr int EPT = kTile * CC / kScanThreads, Q = EPT / V, NB = kTile * NP / kScanThreads;
    constexpr int WARPS = kScanThreads / 32;
    constexpr bool PRECISE = sizeof(T) == 4;
    extern __shared__ __align__(16) float smem[];
    float(*s_dt)[CC] = reinterpret_cast<float(*)[CC]>(smem);            // each [kTile][CC]
    float(*s_du)[CC] = s_dt + kTile;                                    // dt u
    float(*s_ds)[CC] = s_du + kTile;
    float(*s_gb)[CC] = s_ds + kTile;                                    // sum_n g B
    float(*s_ap)[CC] = s_gb + kTile;                                    // sum_n A p g
    float(*s_y)[CC] = s_ap + kTile;                                     // C . h
    float4(*s_B)[LN] = reinterpret_cast<float4(*)[LN]>(s_y + kTile);    // [kTile][LN]
    float4(*s_C)[LN] = s_B + kTile;
    float(*s_part)[kTile][2][NP] = reinterpret_cast<float(*)[kTile][2][NP]>(s_C + kTile);   // [WARPS]
    float *s_acc = reinterpret_cast<float *>(s_part + WARPS);           // [2 V][threads]: dD, ddt_bias
    float *s_dA = s_acc + 2 * V * kScanThreads;                         // [16][threads]: sums and their errors

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long id = blockIdx.x;
    const int tile_c = (int)(id % P.tiles);
    id /= P.tiles;
    const int g = (int)(id % P.G);
    id /= P.G;
    const long long b = id % P.B;
    const int seg = (int)(id / P.B);
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

    const int nl = lane % LN, cg = lane / LN, cl = (warp * CG + cg) * 2, cs = c0 + cl, ns = 4 * nl;
    float2 a2[2][2], w[2][2];       // rates (log2), adjoint carried to the token before
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float av[4], wv[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const bool in = cs + c < c1 && ns + n < P.N;
            av[n] = in ? __ldg(P.A + (size_t)(cs + c) * P.N + ns + n) * kLog2e : 0.f;
            wv[n] = (in && K.exit) ? K.exit[(((size_t)seg * P.B + b) * P.D + cs + c) * P.N + ns + n] : 0.f;
        }
        a2[c][0] = make_float2(av[0], av[1]), a2[c][1] = make_float2(av[2], av[3]);
        w[c][0] = make_float2(wv[0], wv[1]), w[c][1] = make_float2(wv[2], wv[3]);
    }
    for (int i = 0; i < 2 * V; ++i) s_acc[i * kScanThreads + tid] = 0.f;
    for (int i = 0; i < 16; ++i) s_dA[i * kScanThreads + tid] = 0.f;

    for (int t = t0 + (t1 - 1 - t0) / kTile * kTile; t >= t0 && t1 > t0; t -= kTile) {
        // ---- the tile's inputs
        Vec<T, V> ru[Q], rd[Q], rz[Q], rg[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int tt = t + lt + q * (kTile / Q);
            ru[q].zero(), rd[q].zero(), rz[q].zero(), rg[q].zero();
            if (live && tt < t1) {
                ru[q].load(u + tt * P.u_ts);
                rd[q].load(de + tt * P.d_ts);
                rg[q].load(dy + (size_t)tt * P.D);
                if (z) rz[q].load(z + tt * P.z_ts);
            }
        }
        float2 h0[2][2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float hv[4] = {0.f, 0.f, 0.f, 0.f};
            const float *from = P.states + ((size_t)(b * P.nck + t / kTile) * P.D + cs + c) * P.N + ns;
            if (cs + c < c1) {
                if ((P.N & 3) == 0) {
                    if (ns < P.N) {
                        const float4 v = __ldg(reinterpret_cast<const float4 *>(from));
                        hv[0] = v.x, hv[1] = v.y, hv[2] = v.z, hv[3] = v.w;
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        if (ns + n < P.N) hv[n] = __ldg(from + n);
                }
            }
            h0[c][0] = make_float2(hv[0], hv[1]), h0[c][1] = make_float2(hv[2], hv[3]);
        }
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int e = tid + q * kScanThreads, tt = t + e / NP, n = e % NP;
            const bool in = tt < t1 && n < P.N;
            reinterpret_cast<float *>(s_B)[e] = in ? to_f32(Bm[tt * P.b_ts + n]) : 0.f;
            reinterpret_cast<float *>(s_C)[e] = in ? to_f32(Cm[tt * P.c_ts + n]) : 0.f;
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int k = lt + q * (kTile / Q), ch = lc - c0;
            const bool in = live && t + k < t1;
            float fu[V], fd[V], fz[V], fg[V];
            ru[q].get(fu), rd[q].get(fd), rz[q].get(fz), rg[q].get(fg);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float x = fd[i] + ((in && P.dt_bias) ? __ldg(P.dt_bias + lc + i) : 0.f);
                fd[i] = in ? (P.softplus ? softplus(x) : x) : 0.f;
                fu[i] = fd[i] != 0.f ? fd[i] * fu[i] : 0.f;
                if (z) fg[i] *= fz[i] * sigmoid<PRECISE>(fz[i]);
            }
            storev<V>(&s_dt[k][ch], fd);
            storev<V>(&s_du[k][ch], fu);
            storev<V>(&s_ds[k][ch], fg);
        }
        __syncthreads();

        // ---- replay: every h of the tile
        float2 h[kTile][2][2];
#pragma unroll
        for (int k = 0; k < kTile; ++k) {
            const float2 dt = *reinterpret_cast<const float2 *>(&s_dt[k][cl]);
            const float2 du = *reinterpret_cast<const float2 *>(&s_du[k][cl]);
            const float4 B = s_B[k][nl];
            const float2 B2[2] = {make_float2(B.x, B.y), make_float2(B.z, B.w)};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float d = c ? dt.y : dt.x, v = c ? du.y : du.x;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    h[k][c][j] = __ffma2_rn(ex2(__fmul2_rn(make_float2(d, d), a2[c][j])), k ? h[k - 1][c][j] : h0[c][j],
                                            __fmul2_rn(make_float2(v, v), B2[j]));
            }
        }
        if (z) {
#pragma unroll
            for (int k = 0; k < kTile; k += 2) {
                float yv[4];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const float4 C = s_C[k + kk][nl];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float2 p = __ffma2_rn(h[k + kk][c][0], make_float2(C.x, C.y),
                                                    __fmul2_rn(h[k + kk][c][1], make_float2(C.z, C.w)));
                        yv[2 * kk + c] = p.x + p.y;
                    }
                }
                reduce_scatter<LN, 4>(yv, nl);
                if constexpr (LN == 2) {
                    s_y[k][cl + nl] = yv[0];
                    s_y[k + 1][cl + nl] = yv[1];
                } else if (nl < 4) {
                    s_y[k + (nl >> 1)][cl + (nl & 1)] = yv[0];
                }
            }
        }

        // ---- the way back
        float2 dA[2][2];
#pragma unroll
        for (int c = 0; c < 2; ++c) dA[c][0] = dA[c][1] = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = kTile - 1; k >= 0; --k) {
            const float2 dt = *reinterpret_cast<const float2 *>(&s_dt[k][cl]);
            const float2 du = *reinterpret_cast<const float2 *>(&s_du[k][cl]);
            const float2 ds = *reinterpret_cast<const float2 *>(&s_ds[k][cl]);
            const float4 B = s_B[k][nl], C = s_C[k][nl];
            const float2 B2[2] = {make_float2(B.x, B.y), make_float2(B.z, B.w)};
            const float2 C2[2] = {make_float2(C.x, C.y), make_float2(C.z, C.w)};
            float2 dB2[2], dC2[2];
            float r[4];                             // sum_n g B and sum_n A p g of both channels
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float d = c ? dt.y : dt.x, v = c ? du.y : du.x, e = c ? ds.y : ds.x;
                const float2 d2 = make_float2(d, d), v2 = make_float2(v, v), e2 = make_float2(e, e);
                float2 gb, ap;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 hp = k ? h[k - 1][c][j] : h0[c][j];
                    const float2 a = ex2(__fmul2_rn(d2, a2[c][j]));
                    const float2 gg = __ffma2_rn(e2, C2[j], w[c][j]);
                    const float2 q = __fmul2_rn(__fmul2_rn(a, hp), gg);
                    dC2[j] = c ? __ffma2_rn(e2, h[k][c][j], dC2[j]) : __fmul2_rn(e2, h[k][c][j]);
                    dB2[j] = c ? __ffma2_rn(v2, gg, dB2[j]) : __fmul2_rn(v2, gg);
                    gb = j ? __ffma2_rn(gg, B2[j], gb) : __fmul2_rn(gg, B2[j]);
                    ap = j ? __ffma2_rn(q, a2[c][j], ap) : __fmul2_rn(q, a2[c][j]);
                    dA[c][j] = __ffma2_rn(q, d2, dA[c][j]);
                    w[c][j] = __fmul2_rn(a, gg);
                }
                r[c] = gb.x + gb.y;
                r[2 + c] = ap.x + ap.y;
            }
            reduce_scatter<LN, 4>(r, nl);
            if constexpr (LN == 2) {
                s_gb[k][cl + nl] = r[0];
                s_ap[k][cl + nl] = r[1];
            } else if (nl < 4) {
                ((nl >> 1) ? s_ap : s_gb)[k][cl + (nl & 1)] = r[0];
            }
            float bc[8] = {dB2[0].x, dB2[0].y, dB2[1].x, dB2[1].y, dC2[0].x, dC2[0].y, dC2[1].x, dC2[1].y};
            reduce_scatter<CG, 8, LN>(bc, cg);
            constexpr int KEEP = CG < 8 ? 8 / CG : 1, LOW = CG < 8 ? CG : 8;
            if (cg < LOW) {
#pragma unroll
                for (int i = 0; i < KEEP; ++i) {
                    const int v = i * LOW + cg;     // 4 of dB, then 4 of dC
                    s_part[warp][k][v >> 2][ns + (v & 3)] = bc[i];
                }
            }
        }
        // the tile's part of dA, into a sum with its rounding error kept (two-sum)
        {
            const float tile_dA[8] = {dA[0][0].x, dA[0][0].y, dA[0][1].x, dA[0][1].y,
                                      dA[1][0].x, dA[1][0].y, dA[1][1].x, dA[1][1].y};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = s_dA[2 * i * kScanThreads + tid], x = tile_dA[i], n = s + x, v = n - s;
                s_dA[2 * i * kScanThreads + tid] = n;
                s_dA[(2 * i + 1) * kScanThreads + tid] += (s - (n - v)) + (x - v);
            }
        }
        __syncthreads();

        // ---- outputs of the tile
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int k = lt + q * (kTile / Q), ch = lc - c0;
            if (!live || t + k >= t1) continue;
            float fu[V], fd[V], fz[V], fg[V], odu[V], odd[V], odz[V];
            ru[q].get(fu), rd[q].get(fd), rz[q].get(fz), rg[q].get(fg);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float gb = s_gb[k][ch + i], ap = s_ap[k][ch + i], ds = s_ds[k][ch + i], dt = s_dt[k][ch + i];
                const float skip = P.Dskip ? __ldg(P.Dskip + lc + i) : 0.f;
                odu[i] = fmaf(dt, gb, skip * ds);
                float dd = fmaf(fu[i], gb, ap * 0.6931471805599453f);       // a2 is in units of log 2
                if (P.softplus) dd *= sigmoid<true>(fd[i] + (P.dt_bias ? __ldg(P.dt_bias + lc + i) : 0.f));
                odd[i] = dd;
                s_acc[i * kScanThreads + tid] += ds * fu[i];
                s_acc[(V + i) * kScanThreads + tid] += dd;
                if (z) {
                    const float sg = sigmoid<PRECISE>(fz[i]);
                    odz[i] = fg[i] * fmaf(skip, fu[i], s_y[k][ch + i]) * (sg * fmaf(fz[i], 1.f - sg, 1.f));
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
        for (int e = tid; e < kTile * 2 * NP; e += kScanThreads) {
            const int which = e / (kTile * NP), k = (e / NP) % kTile, n = e % NP;
            if (t + k >= t1 || n >= P.N) continue;
            float s = s_part[0][k][which][n];
#pragma unroll
            for (int i = 1; i < WARPS; ++i) s += s_part[i][k][which][n];
            K.dbc[((size_t)tile_c * 2 + which) * bt + (((size_t)b * P.T + t + k) * P.G + g) * P.N + n] = s;
        }
        __syncthreads();
    }

    const size_t part = (size_t)seg * P.B + b;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (cs + c >= c1) continue;
        if (seg == 0 && K.dstate0) store_state(K.dstate0 + ((size_t)b * P.D + cs + c) * P.N + ns, P.N, ns, w[c]);
        float v[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
            v[n] = s_dA[2 * (4 * c + n) * kScanThreads + tid] + s_dA[(2 * (4 * c + n) + 1) * kScanThreads + tid];
        const float2 v2[2] = {make_float2(v[0], v[1]), make_float2(v[2], v[3])};
        store_state(K.dA + (part * P.D + cs + c) * P.N + ns, P.N, ns, v2);
    }
    // dD and ddt_bias: the threads that loaded the same channels, in order
    __syncthreads();
    constexpr int PER = CC / V;
    for (int e = tid; e < 2 * CC; e += kScanThreads) {
        const int which = e / CC, ch = e % CC;
        if (c0 + ch >= c1) continue;
        float s = 0.f;
        for (int i = 0; i < kScanThreads / PER; ++i)
            s += s_acc[(which * V + ch % V) * kScanThreads + i * PER + ch / V];
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

template <int LN, int V> constexpr size_t bwd_smem() {
    return sizeof(float) * ((size_t)6 * kTile * scan_channels(LN) + 2 * kTile * 4 * LN +
                            (size_t)(kScanThreads / 32) * kTile * 2 * 4 * LN + 2 * V * kScanThreads + 16 * kScanThreads);
}

template <typename T, int LN, int V>
cudaError_t launch_bwd(const BwdArgs &K, const float *dstateT, cudaStream_t st) {
    const ScanArgs &P = K.f;
    const unsigned grid = (unsigned)((long long)P.nseg * P.B * P.G * P.tiles);
    BwdArgs M = K;
    M.exit = dstateT;
    if (P.nseg > 1) {
        ssm_bwd_summary_kernel<T, LN, V><<<grid, kScanThreads, 0, st>>>(K);
        const long long total = (long long)P.B * P.D * P.N;
        ssm_bwd_chain_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(total, P.N, P.nseg, P.A, P.D, dstateT,
                                                                             K.seg_dt, K.seg_g);
        M.exit = K.seg_g;
    }
    constexpr size_t smem = bwd_smem<LN, V>();
    const cudaError_t e =
        cudaFuncSetAttribute(ssm_bwd_kernel<T, LN, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ssm_bwd_kernel<T, LN, V><<<grid, kScanThreads, smem, st>>>(M);
    return cudaGetLastError();
}

int bwd_segments(int B, int T, int D, int N, int G, int sms) {
    const int CC = scan_channels(scan_lanes(N)), tiles = (D / G + CC - 1) / CC;
    const long long blocks = (long long)B * G * tiles;
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
    const int sms = sm_count(), CC = scan_channels(scan_lanes(N)), tiles = (D / G + CC - 1) / CC;
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
    P.tiles = (P.Dg + scan_channels(scan_lanes(N)) - 1) / scan_channels(scan_lanes(N));
    P.u = u, P.u_bs = u_bs, P.u_ts = u_ts, P.delta = delta, P.d_bs = d_bs, P.d_ts = d_ts;
    P.z = z, P.z_bs = z_bs, P.z_ts = z_ts;
    P.Bm = Bm, P.b_bs = b_bs, P.b_ts = b_ts, P.Cm = Cm, P.c_bs = c_bs, P.c_ts = c_ts;
    P.A = A, P.Dskip = Dskip, P.dt_bias = dt_bias, P.softplus = softplus;
    P.nck = (T + kTile - 1) / kTile;
    const bool vec = ssm_vec(P, in_dt, dy, 16) && aligned_to(du, 16) && aligned_to(ddelta, 16) && aligned_to(dz, 16);
    if (states == nullptr) {
        P.states = (float *)take(w.states);
        ssm_fwd_all(P, state0, w.fseg, take(w.fwd), in_dt, vec, false, stream);
    } else {
        P.states = const_cast<float *>(states);         // read only from here on
    }
    K.dbc = (float *)take(w.dbc), K.dA = (float *)take(w.dA), K.dpar = (float *)take(w.dpar);
    if (w.nseg > 1) {
        K.seg_g = (float *)take(round256((size_t)w.nseg * B * D * N * 4));
        K.seg_dt = (float *)take(round256((size_t)w.nseg * B * D * 4));
    }
    P.nseg = w.nseg;
    P.seg_len = (int)((((long long)T + w.nseg - 1) / w.nseg + kTile - 1) / kTile * kTile);
    K.dy = dy, K.g_f32 = g_dt == WKV7_F32, K.du = du, K.ddelta = ddelta, K.dz = dz, K.dstate0 = dstate0;
    cudaError_t e = cudaSuccess;
    by_lanes(scan_lanes(N), [&](auto ln) {
        constexpr int LN = decltype(ln)::value, EPT = kTile * scan_channels(LN) / kScanThreads, V = EPT < 8 ? EPT : 8;
        if (in_dt == WKV7_F32) e = vec ? launch_bwd<float, LN, V>(K, dstateT, stream) : launch_bwd<float, LN, 1>(K, dstateT, stream);
        else e = vec ? launch_bwd<bf16, LN, V>(K, dstateT, stream) : launch_bwd<bf16, LN, 1>(K, dstateT, stream);
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
