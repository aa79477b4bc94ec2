// RMS norm with the residual's addition, an optional 8-bit output, an optional
// 8-bit copy of the normalised sum, and the backward that reads either.
//
//     s = x + residual,  rstd = 1 / sqrt(mean(s^2) + eps),  y = w s rstd
//     xh = s rstd,  c = mean(w dy xh),  dx = dres + rstd (w dy - c xh),  dw = sum dy xh
//
// Both directions are bound by memory (forward with an 8-bit output: 7 bytes a
// bf16 element).  A row is a block of warps; a warp owns blocks of 128 channels
// (the 8-bit format's), MB of them held in registers between the sum and the
// output, so the row is read once; the next two rows come through shared memory
// meanwhile.
//
// 32768 x 2048 bf16 with residual: 117 us to 8 bits (472 MB, 62% of the measured
// copy rate; the exact sums and the sure codes cost 41 instructions an element,
// and the schedulers issue 66% of cycles), 113 us to bf16 with the 8-bit copy of
// the sum (606 MB, 83%), 94 us to bf16 alone (537 MB, 88%), backward from the copy
// 89 us (473 MB, 82%).
//
// The 8-bit output rounds to 4 significant bits, and a value next to a border
// between two codes would fall on either side by fp32's rounding; the row's sum
// is therefore carried in fp64 from every four elements on, and where a block has
// a y next to a border (one block in a thousand) y is taken in two floats (value
// and error) and rounded once.
#include <type_traits>

#include "mixer.cuh"

namespace wkv7 {
namespace mixer {
namespace {

constexpr int kNormMaxWarps = 16;

// E: whether 8-bit codes can be among the types; WIDE: whether fp32 can
template <bool WIDE, bool E, typename F> __device__ __forceinline__ void by_dtype(wkv7_dtype dt, F &&f) {
    if (E && dt == WKV7_E4M3) f(e4m3());
    else if (!WIDE || dt == WKV7_BF16) f(bf16());
    else if constexpr (WIDE) f(float());
}
// MB blocks of a row, one branch around the batch.  Not CONST: residual and dresidual, which
// may be outputs as well.
template <bool VEC, int MB, bool WIDE, bool E, bool CONST = true>
__device__ __forceinline__ void batch_load(const void *p, wkv7_dtype dt, int blk0, int step, int lane, int D,
                                           float (&f)[MB][4]) {
    by_dtype<WIDE, E>(dt, [&](auto t) {
        const decltype(t) *row = static_cast<const decltype(t) *>(p);
#pragma unroll
        for (int m = 0; m < MB; ++m) row_load<VEC, CONST>(row, blk0 + m * step, lane, D, f[m]);
    });
}

// Rows on their way or in use: kAhead rows of each tensor, copied to shared memory
// (cp.async) by the thread that reads them, so no barrier is needed.  A slot is
// four values, 8 bytes or (WIDE) 16; slots behind the row's end stay zero.
constexpr int kAhead = 3;
template <int MB, bool WIDE, int TENSORS> struct Ring {
    static constexpr int SLOT = WIDE ? 16 : 8;
    unsigned char *base;
    __device__ __forceinline__ unsigned char *slot(int stage, int tensor, int m) const {
        return base + ((size_t)((stage * TENSORS + tensor) * MB + m) * blockDim.x + threadIdx.x) * SLOT;
    }
    __device__ __forceinline__ void clear() const {
        for (int i = 0; i < kAhead * TENSORS * MB; ++i)
            for (int k = 0; k < SLOT; k += 8) *reinterpret_cast<uint2 *>(slot(0, 0, i) + k) = make_uint2(0, 0);
    }
    template <bool E>
    __device__ __forceinline__ void fetch(int stage, int tensor, const void *p, wkv7_dtype dt, int blk0, int step, int lane,
                                          int D) const {
        by_dtype<WIDE, E>(dt, [&](auto t) {
            const decltype(t) *row = static_cast<const decltype(t) *>(p);
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                const int c = lane_channel<true>(blk0 + m * step, lane, 0);
                if (c < D) copy_async<4 * (int)sizeof(t)>(slot(stage, tensor, m), row + c, true);
            }
        });
    }
    template <bool E>
    __device__ __forceinline__ void get(int stage, int tensor, int m, wkv7_dtype dt, float (&f)[4]) const {
        by_dtype<WIDE, E>(dt, [&](auto t) {
            Vec<decltype(t), 4> v;
            const uint32_t *w = reinterpret_cast<const uint32_t *>(slot(stage, tensor, m));
            if constexpr (sizeof(v.w) == 16) {
                const uint4 q = *reinterpret_cast<const uint4 *>(w);
                v.w[0] = q.x, v.w[1] = q.y, v.w[2] = q.z, v.w[3] = q.w;
            } else if constexpr (sizeof(v.w) == 8) {
                const uint2 q = *reinterpret_cast<const uint2 *>(w);
                v.w[0] = q.x, v.w[1] = q.y;
            } else {
                v.w[0] = w[0];
            }
            v.get(f);
        });
    }
    template <bool E>
    __device__ __forceinline__ void get(int stage, int tensor, wkv7_dtype dt, float (&f)[MB][4]) const {
#pragma unroll
        for (int m = 0; m < MB; ++m) get<E>(stage, tensor, m, dt, f[m]);
    }
};
template <int MB, bool WIDE> constexpr size_t ring_bytes(int tensors, int threads) {
    return (size_t)kAhead * tensors * MB * threads * (WIDE ? 16 : 8);
}

template <bool VEC, int MB, bool WIDE>
__device__ __forceinline__ void batch_store(void *p, wkv7_dtype dt, int blk0, int step, int lane, int D,
                                            const float (&f)[MB][4]) {
    if (!WIDE || dt == WKV7_BF16) {
#pragma unroll
        for (int m = 0; m < MB; ++m) row_store<VEC>(static_cast<bf16 *>(p), blk0 + m * step, lane, D, f[m]);
    } else {
#pragma unroll
        for (int m = 0; m < MB; ++m) row_store<VEC>(static_cast<float *>(p), blk0 + m * step, lane, D, f[m]);
    }
}
__device__ __forceinline__ long long elem_size(wkv7_dtype dt) { return dt == WKV7_F32 ? 4 : dt == WKV7_BF16 ? 2 : 1; }
// A tensor's rows as a block walks them
struct Rows {
    char *p;
    long long step;
    __device__ __forceinline__ Rows(const void *base, wkv7_dtype dt, long long ld)
        : p(base ? (char *)base + blockIdx.x * ld * elem_size(dt) : nullptr), step(gridDim.x * ld * elem_size(dt)) {}
    __device__ __forceinline__ void next() { p += step; }
};

// sum over the block's warps of one value a warp; every thread gets it
template <typename F> __device__ __forceinline__ F block_add(F x, F *shared, int warp, int warps) {
    x = warp_add(x);
    if (warps == 1) return x;
    if ((threadIdx.x & 31) == 0) shared[warp] = x;
    __syncthreads();
    F t = shared[0];
    for (int i = 1; i < warps; ++i) t += shared[i];
    return t;
}

// unit / sqrt(x) in two floats, value and rest: the root in fp32 and one Newton step in fp64
__device__ __forceinline__ float2 rsqrt2(double x, double unit) {
    const double r = (double)rsqrtf((float)x), inv = fma(0.5 * r, fma(-x * r, r, 1.0), r) * unit;
    const float hi = (float)inv;
    return make_float2(hi, (float)(inv - (double)hi));
}
// A row whose squares left fp32's range (above 2^63, or below 2^-50 with an eps below that
// too; mean is infinite, tiny or NaN then): 1 / sqrt(mean square) from `sum`, a thread's
// squares of the row times far_unit.  Out of line: rare, and inline it took registers
// from every row.
__device__ __forceinline__ bool far_mean(double mean) {         // not in [2^-100, 2^126]
    return __float_as_uint((float)mean) - 0x0d800000u > 0x7e800000u - 0x0d800000u;
}
__device__ __forceinline__ float far_unit(double mean) { return mean > 1.0 ? 0x1p-68f : 0x1p100f; }
__device__ __noinline__ float2 far_row(double sum, double mean, double inv_D, double eps, double *shared) {
    const double unit = far_unit(mean);
    sum = block_add(sum, shared, threadIdx.x >> 5, blockDim.x >> 5);
    mean = fma(sum, inv_D, eps * unit * unit);
    if (mean == 0.0 || isinf(mean)) return make_float2(rsqrtf((float)mean), 0.f);
    const float2 r = rsqrt2(mean, unit);
    return make_float2(r.x, isinf(r.x) ? 0.f : r.y);
}

// blocks of 128 a warp holds, and the threads of a row's block at most
__host__ __device__ constexpr int norm_max_threads(int MB) { return MB <= 2 ? 32 : 512; }
// and the threads on an SM that the registers leave room for
__host__ __device__ constexpr int norm_sm_threads(int MB) { return MB <= 2 ? 1024 : 512; }

struct NormFwd {
    long long rows;
    int D;
    wkv7_dtype x_dt, r_dt, y_dt;
    const void *x;
    long long x_ld;
    const void *residual;
    const float *weight;
    double eps, inv_D;
    void *residual_out, *y;
    float *y_scales;
    uint8_t *s_codes;
    float *s_scales, *rstd;
};

// A block takes rows blockIdx.x, + gridDim.x, ...  RING: the next rows are on their
// way.  WIDE: fp32 can be among the types.
template <bool VEC, int MB, bool WIDE, bool RING>
__global__ void __launch_bounds__(norm_max_threads(MB), norm_sm_threads(MB) / norm_max_threads(MB))
rmsnorm_fwd_kernel(const NormFwd P) {
    constexpr bool KEEP = MB <= 4;      // the weight stays in registers
    __shared__ double shared[2][kNormMaxWarps];
    extern __shared__ __align__(16) unsigned char ring_mem[];
    const Ring<MB, WIDE, 2> ring{ring_mem};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nblk = (P.D + kBlk - 1) / kBlk, D = P.D;
    float w[MB][4];
    Rows x(P.x, P.x_dt, P.x_ld), res(P.residual, P.r_dt, D), res_out(P.residual_out, P.r_dt, D), y(P.y, P.y_dt, D);
    Rows codes(P.s_codes, WKV7_E4M3, D), scales(P.s_scales, WKV7_F32, nblk), y_scales(P.y_scales, WKV7_F32, nblk);
    long long ahead = blockIdx.x;       // the row that is fetched next
    auto fetch = [&](int stage) {
        if (ahead < P.rows) {
            ring.template fetch<false>(stage, 0, x.p, P.x_dt, warp, warps, lane, D);
            x.next();
            if (P.residual) {
                ring.template fetch<false>(stage, 1, res.p, P.r_dt, warp, warps, lane, D);
                res.next();
            }
            ahead += gridDim.x;
        }
        cp_async_commit();
    };
    if constexpr (RING) {
        ring.clear();
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i) fetch(i);
    }
    if (KEEP) {
#pragma unroll
        for (int m = 0; m < MB; ++m) row_load<VEC>(P.weight, warp + m * warps, lane, D, w[m]);
    }
    int turn = 0, stage = 0;
    for (long long row = blockIdx.x; row < P.rows; row += gridDim.x) {
        // No branch inside the loops over m: the blocks' work overlaps
        float s[MB][4];
        const int now = stage;
        if constexpr (RING) {
            fetch(stage == 0 ? kAhead - 1 : stage - 1);
            cp_async_wait<kAhead - 1>();
            stage = stage == kAhead - 1 ? 0 : stage + 1;
        }
        auto get_x = [&](float (&f)[MB][4]) {
            if constexpr (RING) ring.template get<false>(now, 0, P.x_dt, f);
            else batch_load<VEC, MB, WIDE, false>(x.p, P.x_dt, warp, warps, lane, D, f);
        };
        auto get_res = [&](float (&f)[MB][4]) {
            if constexpr (RING) ring.template get<false>(now, 1, P.r_dt, f);
            else batch_load<VEC, MB, WIDE, false, false>(res.p, P.r_dt, warp, warps, lane, D, f);
        };
        auto error = [&](const float (&a)[4], const float (&b)[4], const float (&t)[4], float (&e)[4]) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float2 v = sum_error(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]),
                                           make_float2(t[i], t[i + 1]));
                e[i] = v.x, e[i + 1] = v.y;
            }
        };
        bool inexact = false;       // a sum of two bf16 numbers only where they are 2^16 apart
        get_x(s);
        if (P.residual) {
            float r[MB][4];
            uint32_t bits = 0;
            get_res(r);
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                float t[4], e[4];
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const float2 v = __fadd2_rn(make_float2(s[m][i], s[m][i + 1]), make_float2(r[m][i], r[m][i + 1]));
                    t[i] = v.x, t[i + 1] = v.y;
                }
                error(s[m], r[m], t, e);
                bits |= abs_bits(e[0]) | abs_bits(e[1]) | abs_bits(e[2]) | abs_bits(e[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[m][i] = t[i];
            }
            inexact = __any_sync(0xffffffffu, bits != 0);
        }
        double sum = 0;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const float2 lo = make_float2(s[m][0], s[m][1]), hi = make_float2(s[m][2], s[m][3]);
            const float2 sq = __ffma2_rn(hi, hi, __fmul2_rn(lo, lo));
            sum += (double)(sq.x + sq.y);
        }
        auto keep = [&](const float (&o)[MB][4]) {      // what keeps fewer bits of the sum
            if (P.residual_out) {
                if (!WIDE || P.r_dt == WKV7_BF16) batch_store<VEC, MB, false>(res_out.p, WKV7_BF16, warp, warps, lane, D, o);
                else batch_store<VEC, MB, true>(res_out.p, WKV7_F32, warp, warps, lane, D, s);
            }
            if (P.s_codes) {
                uint32_t q[MB];
                float scale[MB];
                act8_encode_all(o, q, scale);
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const int blk = warp + m * warps;
                    row_store_codes<VEC>(reinterpret_cast<uint8_t *>(codes.p), blk, lane, D, q[m]);
                    if (lane == 0 && blk < nblk) reinterpret_cast<float *>(scales.p)[blk] = scale[m];
                }
            }
        };
        if (!inexact) keep(s);
        else {                      // rounded to odd, it rounds to fewer bits as the exact sum does
            float o[MB][4], r[MB][4];
            get_x(o);
            get_res(r);
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                float e[4];
                error(o[m], r[m], s[m], e);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][i] = to_odd(s[m][i], e[i]);
            }
            keep(o);
        }
        if constexpr (!RING) {
            x.next();
            res.next();
        }
        res_out.next();
        codes.next(), scales.next();
        // two buffers in turn: a warp that is a row ahead does not overwrite sums still being read
        sum = block_add(sum, shared[turn], warp, warps);
        turn ^= 1;
        const double mean = fma(sum, P.inv_D, P.eps);
        float2 inv;
        if (!__any_sync(0xffffffffu, far_mean(mean))) {         // uniform in the block; the vote tells the compiler so
            inv = rsqrt2(mean, 1.0);
        } else {
            const float unit = far_unit(mean);
            double far = 0;
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) far += (double)(s[m][i] * unit) * (double)(s[m][i] * unit);
            inv = far_row(far, mean, P.inv_D, P.eps, shared[turn]);
            turn ^= 1;
        }
        const float ih = inv.x, il = inv.y;
        if (P.rstd && threadIdx.x == 0) P.rstd[row] = ih;
        if (!KEEP) {
#pragma unroll
            for (int m = 0; m < MB; ++m) row_load<VEC>(P.weight, warp + m * warps, lane, D, w[m]);
        }
        if (P.y_dt != WKV7_E4M3) {
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[m][i] = s[m][i] * ih * w[m][i];
            batch_store<VEC, MB, true>(y.p, P.y_dt, warp, warps, lane, D, s);
            y.next();
            continue;
        }
        uint32_t q[MB];
        float scale[MB];
        bool sure[MB], all = true;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; i += 2) {        // off by 3 half steps at most
                const float2 t = __fmul2_rn(make_float2(s[m][i], s[m][i + 1]), make_float2(ih, ih));
                const float2 u = __fmul2_rn(t, make_float2(w[m][i], w[m][i + 1]));
                v[i] = u.x, v[i + 1] = u.y;
            }
            sure[m] = act8_encode_sure(v, q[m], scale[m]);
            all &= sure[m];
        }
        if (!all) {
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                if (sure[m]) continue;
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = s[m][i] * ih, pl = fmaf(s[m][i], il, fmaf(s[m][i], ih, -p));
                    const float t = p * w[m][i], tl = fmaf(pl, w[m][i], fmaf(p, w[m][i], -t));
                    const float top = t + tl;
                    v[i] = to_odd(top, tl - (top - t));
                }
                scale[m] = act8_encode(v, q[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int blk = warp + m * warps;
            row_store_codes<VEC>(reinterpret_cast<uint8_t *>(y.p), blk, lane, D, q[m]);
            if (lane == 0 && blk < nblk) reinterpret_cast<float *>(y_scales.p)[blk] = scale[m];
        }
        y.next(), y_scales.next();
    }
}

struct NormBwd {
    long long rows;
    int D;
    wkv7_dtype s_dt, dy_dt, g_dt;
    const void *s;
    const float *s_scales, *rstd, *weight;
    const void *dy, *dres;
    void *dx;
    float *partial;          // [grid][D]
    float inv_D;
};

// The same walk over rows; a block's share of dw goes to partial[blockIdx.x].
// KEEP: w and dw stay in registers (dw in shared memory otherwise).
template <bool VEC, int MB, bool WIDE, bool RING>
__global__ void __launch_bounds__(norm_max_threads(MB), norm_sm_threads(MB) / norm_max_threads(MB))
rmsnorm_bwd_kernel(const NormBwd P) {
    constexpr bool KEEP = MB <= 4;
    static_assert(KEEP || !RING, "dw and the rows share the dynamic shared memory");
    __shared__ float shared[2][kNormMaxWarps];
    extern __shared__ __align__(16) unsigned char ring_mem[];
    const Ring<MB, WIDE, 3> ring{ring_mem};
    float *s_dw = reinterpret_cast<float *>(ring_mem);      // [4 MB][threads] when not KEEP
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nblk = (P.D + kBlk - 1) / kBlk, D = P.D;
    float w[MB][4], dw[MB][4];
    float next_r = 0.f, next_scale[MB];
    Rows sr(P.s, P.s_dt, D), gr(P.dy, P.dy_dt, D), dr(P.dres, P.g_dt, D), xr(P.dx, P.g_dt, D);
    Rows qr(P.s_scales, WKV7_F32, nblk), rr(P.rstd, WKV7_F32, 1);
    long long ahead = blockIdx.x, small = blockIdx.x;       // the rows that are fetched next
    auto fetch = [&](int stage) {
        if (ahead < P.rows) {
            ring.template fetch<true>(stage, 0, sr.p, P.s_dt, warp, warps, lane, D);
            ring.template fetch<false>(stage, 1, gr.p, P.dy_dt, warp, warps, lane, D);
            sr.next(), gr.next();
            if (P.dres) {
                ring.template fetch<false>(stage, 2, dr.p, P.g_dt, warp, warps, lane, D);
                dr.next();
            }
            ahead += gridDim.x;
        }
        cp_async_commit();
    };
    auto fetch_small = [&]() {
        if (small >= P.rows) return;
        small += gridDim.x;
        next_r = __ldg(reinterpret_cast<const float *>(rr.p));
        rr.next();
        if (P.s_dt == WKV7_E4M3) {
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                const int blk = warp + m * warps;
                next_scale[m] = blk < nblk ? __ldg(reinterpret_cast<const float *>(qr.p) + blk) : 0.f;
            }
            qr.next();
        }
    };
    if constexpr (RING) {
        ring.clear();
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i) fetch(i);
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) next_scale[m] = 1.f;
    fetch_small();
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        if (KEEP) row_load<VEC>(P.weight, warp + m * warps, lane, D, w[m]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (KEEP) dw[m][i] = 0.f;
            else s_dw[(4 * m + i) * blockDim.x + threadIdx.x] = 0.f;
        }
    }
    int turn = 0, stage = 0;
    for (long long row = blockIdx.x; row < P.rows; row += gridDim.x) {
        float s[MB][4], g[MB][4];
        const int now = stage;
        if constexpr (RING) {
            fetch(stage == 0 ? kAhead - 1 : stage - 1);
            cp_async_wait<kAhead - 1>();
            ring.template get<true>(now, 0, P.s_dt, s);
            ring.template get<false>(now, 1, P.dy_dt, g);
            stage = stage == kAhead - 1 ? 0 : stage + 1;
        } else {
            batch_load<VEC, MB, WIDE, true>(sr.p, P.s_dt, warp, warps, lane, D, s);
            batch_load<VEC, MB, WIDE, false>(gr.p, P.dy_dt, warp, warps, lane, D, g);
            sr.next(), gr.next();
        }
        const float r = next_r;
        float2 c2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const float q = next_scale[m] * r;
            if (!KEEP) row_load<VEC>(P.weight, warp + m * warps, lane, D, w[m]);
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float2 xh = __fmul2_rn(make_float2(s[m][i], s[m][i + 1]), make_float2(q, q));
                const float2 gg = make_float2(g[m][i], g[m][i + 1]);
                if (KEEP) {
                    const float2 a = __ffma2_rn(gg, xh, make_float2(dw[m][i], dw[m][i + 1]));
                    dw[m][i] = a.x, dw[m][i + 1] = a.y;
                } else {
                    s_dw[(4 * m + i) * blockDim.x + threadIdx.x] += gg.x * xh.x;
                    s_dw[(4 * m + i + 1) * blockDim.x + threadIdx.x] += gg.y * xh.y;
                }
                const float2 wg = __fmul2_rn(gg, make_float2(w[m][i], w[m][i + 1]));
                c2 = __ffma2_rn(wg, xh, c2);
                s[m][i] = xh.x, s[m][i + 1] = xh.y;
                g[m][i] = wg.x, g[m][i + 1] = wg.y;
            }
        }
        fetch_small();
        // two buffers in turn, as in the forward
        const float c = block_add(c2.x + c2.y, shared[turn], warp, warps) * P.inv_D;
        turn ^= 1;
        const float2 nc = make_float2(-c, -c), r2 = make_float2(r, r);
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float2 v = __fmul2_rn(r2, __ffma2_rn(nc, make_float2(s[m][i], s[m][i + 1]),
                                                           make_float2(g[m][i], g[m][i + 1])));
                s[m][i] = v.x, s[m][i + 1] = v.y;
            }
        if (P.dres) {
            if constexpr (RING) ring.template get<false>(now, 2, P.g_dt, g);
            else {
                batch_load<VEC, MB, WIDE, false, false>(dr.p, P.g_dt, warp, warps, lane, D, g);
                dr.next();
            }
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[m][i] += g[m][i];
        }
        batch_store<VEC, MB, true>(xr.p, P.g_dt, warp, warps, lane, D, s);
        xr.next();
    }
    if (!KEEP) {
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) dw[m][i] = s_dw[(4 * m + i) * blockDim.x + threadIdx.x];
    }
    batch_store<VEC, MB, true>(P.partial + (size_t)blockIdx.x * D, WKV7_F32, warp, warps, lane, D, dw);
}

// A row's fixed work (the sum over warps, the root) costs a warp some 150
// instructions, so a warp takes four blocks where the row has them (32768 x 2048 to
// 8 bits: 115 us, 175 at two, when this was chosen).
int norm_batch(int nblk) { return nblk <= 2 ? nblk : nblk <= 64 ? 4 : 8; }

int norm_threads(int nblk) { return 32 * ((nblk + norm_batch(nblk) - 1) / norm_batch(nblk)); }

// Blocks that walk the rows: as many as the SMs hold
long long norm_grid(long long rows, int D) {
    const int sms = sm_count(), threads = norm_threads(blocks_of(D)), per_sm = norm_sm_threads(norm_batch(blocks_of(D)));
    if (sms <= 0) return 0;
    const long long most = (long long)sms * (per_sm / threads > 0 ? per_sm / threads : 1);
    return rows < most ? rows : most;
}

// What a kernel's dynamic shared memory may be at most.  The leave for it is a property of
// the kernel, not of the launch: it is this one number in every call, since a call
// that set its own size would take it from a call of a wider row on another host thread.
constexpr size_t kNormSmem = 200 * 1024;

template <typename K, typename P>
wkv7_status norm_launch(K kernel, const P &p, long long grid, int threads, size_t smem, cudaStream_t st) {
    if (smem > 40 * 1024 &&         // 48 KiB with the kernel's own arrays need no leave
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNormSmem) != cudaSuccess)
        return WKV7_ERR_CUDA;
    kernel<<<(unsigned)grid, threads, smem, st>>>(p);
    return launch_status();
}
// blocks of 128 a warp as a template argument; rows ahead where vector accesses
// are allowed and an SM's shared memory holds them
template <bool VEC, bool WIDE, int TENSORS, typename F> wkv7_status by_batch(int nblk, F &&f) {
    auto ring = [&](auto mb) {
        if constexpr (VEC) {
            if (ring_bytes<decltype(mb)::value, WIDE>(TENSORS, norm_threads(nblk)) <= kNormSmem)
                return f(mb, std::true_type{});
        }
        return f(mb, std::false_type{});
    };
    switch (norm_batch(nblk)) {
        case 1: return ring(std::integral_constant<int, 1>{});
        case 2: return ring(std::integral_constant<int, 2>{});
        case 4: return ring(std::integral_constant<int, 4>{});
    }
    // (the backward keeps dw in the shared memory that the rows would take)
    if constexpr (TENSORS == 2) return ring(std::integral_constant<int, 8>{});
    else return f(std::integral_constant<int, 8>{}, std::false_type{});
}

wkv7_status norm_dims(long long rows, int D) {
    if (rows < 0 || D < 0) return WKV7_ERR_INVALID_ARG;
    if (D > WKV7_NORM_MAX_D || rows > kMaxGrid) return WKV7_ERR_UNSUPPORTED;
    return WKV7_OK;
}

}  // namespace

// out[c] = sum over p of partial[p][c], in order: a block's 32 columns by 8 rows
// of threads that take every 8th part, joined in shared memory.
__global__ void __launch_bounds__(256)
sum_parts_kernel(long long parts, long long cols, const float *__restrict__ partial, float *__restrict__ out) {
    __shared__ float shared[8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + tx;
    float a = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (long long p = ty; p < parts; p += 8) a += __ldg(partial + p * cols + c);
    }
    shared[ty][tx] = a;
    __syncthreads();
    if (ty == 0 && c < cols) {
        float t = shared[0][tx];
#pragma unroll
        for (int i = 1; i < 8; ++i) t += shared[i][tx];
        out[c] = t;
    }
}

void sum_parts(long long parts, long long cols, const float *partial, float *out, cudaStream_t st) {
    if (cols > 0) sum_parts_kernel<<<(unsigned)((cols + 31) / 32), 256, 0, st>>>(parts, cols, partial, out);
}

}  // namespace mixer
}  // namespace wkv7

extern "C" {

wkv7_status wkv7_rmsnorm_forward(long long rows, int D, wkv7_dtype x_dt, wkv7_dtype r_dt, wkv7_dtype y_dt,
                                 const void *x, long long x_ld, const void *residual, const float *weight, float eps,
                                 void *residual_out, void *y, float *y_scales, void *s_codes, float *s_scales,
                                 float *rstd, cudaStream_t stream) {
    using namespace wkv7::mixer;
    const wkv7_status st = norm_dims(rows, D);
    if (st != WKV7_OK) return st;
    if (!real_dtype(x_dt) || !real_dtype(r_dt) || !(real_dtype(y_dt) || y_dt == WKV7_E4M3) || x_ld < 0 ||
        !(eps >= 0.f) || eps > 3.0e38f)
        return WKV7_ERR_INVALID_ARG;
    if (rows == 0 || D == 0) return WKV7_OK;
    if (!elem_ok(x, x_dt) || !f32_ok(weight) || !elem_ok(y, y_dt) || !f32_opt(rstd)) return WKV7_ERR_INVALID_ARG;
    if ((residual && !elem_ok(residual, r_dt)) || (residual_out && !elem_ok(residual_out, r_dt)))
        return WKV7_ERR_INVALID_ARG;
    if ((y_dt == WKV7_E4M3) != (y_scales != nullptr) || !f32_opt(y_scales)) return WKV7_ERR_INVALID_ARG;
    if ((s_codes != nullptr) != (s_scales != nullptr) || !f32_opt(s_scales)) return WKV7_ERR_INVALID_ARG;
    const NormFwd P{rows, D, x_dt, r_dt, y_dt, x, x_ld, residual, weight, (double)eps, 1.0 / D, residual_out, y,
                    y_scales, (uint8_t *)s_codes, s_scales, rstd};
    const long long grid = norm_grid(rows, D);
    if (grid <= 0) return WKV7_ERR_CUDA;
    const bool vec = D % 4 == 0 && x_ld % 4 == 0 && aligned_to(x, 4 * dtype_size(x_dt)) &&
                     aligned_to(residual, 4 * dtype_size(r_dt)) && aligned_to(residual_out, 4 * dtype_size(r_dt)) &&
                     aligned_to(y, 4 * dtype_size(y_dt)) && aligned_to(weight, 16) && aligned_to(s_codes, 4);
    const int nblk = blocks_of(D), threads = norm_threads(nblk);
    const bool narrow = x_dt == WKV7_BF16 && ((!residual && !residual_out) || r_dt == WKV7_BF16);
#define WKV7_NORM(V, R)                                                                                     \
    by_batch<V, R, 2>(nblk, [&](auto mb, auto ring) {                                                       \
        constexpr int M = decltype(mb)::value;                                                              \
        constexpr bool G = decltype(ring)::value;                                                           \
        return norm_launch(rmsnorm_fwd_kernel<V, M, R, G>, P, grid, threads,                                \
                           G ? ring_bytes<M, R>(2, threads) : 0, stream);                                   \
    })
    return vec && narrow ? WKV7_NORM(true, false) : vec ? WKV7_NORM(true, true) : WKV7_NORM(false, true);
#undef WKV7_NORM
}

size_t wkv7_rmsnorm_backward_workspace_size(long long rows, int D) {
    using namespace wkv7::mixer;
    if (rows <= 0 || D <= 0 || norm_dims(rows, D) != WKV7_OK) return 0;
    return (size_t)norm_grid(rows, D) * D * sizeof(float);
}

wkv7_status wkv7_rmsnorm_backward(long long rows, int D, wkv7_dtype s_dt, wkv7_dtype dy_dt, wkv7_dtype g_dt,
                                  const void *s, const float *s_scales, const float *rstd, const float *weight,
                                  const void *dy, const void *dresidual, void *dx, float *dweight, void *workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
    using namespace wkv7::mixer;
    const wkv7_status st = norm_dims(rows, D);
    if (st != WKV7_OK) return st;
    if (!(real_dtype(s_dt) || s_dt == WKV7_E4M3) || !real_dtype(dy_dt) || !real_dtype(g_dt))
        return WKV7_ERR_INVALID_ARG;
    if (D == 0) return WKV7_OK;
    if (!f32_ok(dweight)) return WKV7_ERR_INVALID_ARG;
    if (rows == 0)
        return cudaMemsetAsync(dweight, 0, (size_t)D * 4, stream) == cudaSuccess ? WKV7_OK : WKV7_ERR_CUDA;
    if (!elem_ok(s, s_dt) || !elem_ok(dy, dy_dt) || !elem_ok(dx, g_dt) || !f32_ok(rstd) || !f32_ok(weight) ||
        (dresidual && !elem_ok(dresidual, g_dt)))
        return WKV7_ERR_INVALID_ARG;
    if ((s_dt == WKV7_E4M3) != (s_scales != nullptr) || !f32_opt(s_scales)) return WKV7_ERR_INVALID_ARG;
    const long long grid = norm_grid(rows, D);
    if (grid <= 0) return WKV7_ERR_CUDA;
    if (workspace == nullptr || !aligned_to(workspace, 16) || workspace_bytes < (size_t)grid * D * sizeof(float))
        return WKV7_ERR_INVALID_ARG;
    const NormBwd P{rows, D, s_dt, dy_dt, g_dt, s, s_scales, rstd, weight, dy, dresidual, dx, (float *)workspace,
                    (float)(1.0 / D)};
    const bool vec = D % 4 == 0 && aligned_to(s, 4 * dtype_size(s_dt)) && aligned_to(dy, 4 * dtype_size(dy_dt)) &&
                     aligned_to(dresidual, 4 * dtype_size(g_dt)) && aligned_to(dx, 4 * dtype_size(g_dt)) &&
                     aligned_to(weight, 16);
    const int nblk = blocks_of(D), threads = norm_threads(nblk);
    const bool narrow = s_dt != WKV7_F32 && dy_dt == WKV7_BF16 && (!dresidual || g_dt == WKV7_BF16);
#define WKV7_NORM(V, R)                                                                                     \
    by_batch<V, R, 3>(nblk, [&](auto mb, auto ring) {                                                       \
        constexpr int M = decltype(mb)::value;                                                              \
        constexpr bool G = decltype(ring)::value;                                                           \
        return norm_launch(rmsnorm_bwd_kernel<V, M, R, G>, P, grid, threads,                                \
                           G ? ring_bytes<M, R>(3, threads) : M > 4 ? (size_t)4 * M * threads * sizeof(float) : 0, \
                           stream);                                                                         \
    })
    const wkv7_status done = vec && narrow ? WKV7_NORM(true, false) : vec ? WKV7_NORM(true, true) : WKV7_NORM(false, true);
#undef WKV7_NORM
    if (done != WKV7_OK) return done;
    sum_parts(grid, D, (const float *)workspace, dweight, stream);
    return launch_status();
}

}  // extern "C"
