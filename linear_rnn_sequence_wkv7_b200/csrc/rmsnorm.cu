// RMS norm with the residual's addition, an optional 8-bit output, an optional
// 8-bit copy of the normalised sum, and the backward that reads either.
//
//     s = x + residual,  rstd = 1 / sqrt(mean(s^2) + eps),  y = w s rstd
//     xh = s rstd,  c = mean(w dy xh),  dx = dres + rstd (w dy - c xh),  dw = sum dy xh
//
// Both directions are bound by memory (forward with an 8-bit output: 7 bytes a
// bf16 element).  A row is a block of warps; a warp owns blocks of 128 channels
// (the 8-bit format's), MB of them held in registers between the sum and the
// output, so the row is read once.
//
// The 8-bit output rounds to 4 significant bits, and a value next to a border
// between two codes would fall on either side by fp32's rounding; the row's sum
// is therefore carried in fp64 from every four elements on, and y in two floats
// (value and error), rounded once.
#include "mixer.cuh"

namespace wkv7 {
namespace mixer {
namespace {

constexpr int kNormMaxWarps = 16;

// MB blocks of a row by run-time type: one branch around the whole batch of loads
template <bool VEC, int MB>
__device__ __forceinline__ void batch_load(const void *p, wkv7_dtype dt, long long off, int blk0, int step, int nblk,
                                           int lane, int D, float (&f)[MB][4]) {
    if (dt == WKV7_BF16) {
        const bf16 *row = static_cast<const bf16 *>(p) + off;
#pragma unroll
        for (int m = 0; m < MB; ++m) row_load<VEC>(row, blk0 + m * step, lane, D, f[m]);
    } else if (dt == WKV7_F32) {
        const float *row = static_cast<const float *>(p) + off;
#pragma unroll
        for (int m = 0; m < MB; ++m) row_load<VEC>(row, blk0 + m * step, lane, D, f[m]);
    } else {
        const e4m3 *row = static_cast<const e4m3 *>(p) + off;
#pragma unroll
        for (int m = 0; m < MB; ++m) row_load<VEC>(row, blk0 + m * step, lane, D, f[m]);
    }
}
template <bool VEC, int MB>
__device__ __forceinline__ void batch_store(void *p, wkv7_dtype dt, long long off, int blk0, int step, int lane,
                                            int D, const float (&f)[MB][4]) {
    if (dt == WKV7_BF16) {
        bf16 *row = static_cast<bf16 *>(p) + off;
#pragma unroll
        for (int m = 0; m < MB; ++m) row_store<VEC>(row, blk0 + m * step, lane, D, f[m]);
    } else {
        float *row = static_cast<float *>(p) + off;
#pragma unroll
        for (int m = 0; m < MB; ++m) row_store<VEC>(row, blk0 + m * step, lane, D, f[m]);
    }
}

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

struct NormFwd {
    int D;
    wkv7_dtype x_dt, r_dt, y_dt;
    const void *x;
    long long x_ld;
    const void *residual;
    const float *weight;
    float eps;
    void *residual_out, *y;
    float *y_scales;
    uint8_t *s_codes;
    float *s_scales, *rstd;
};

template <bool VEC, int MB>
__global__ void __launch_bounds__(32 * kNormMaxWarps)
rmsnorm_fwd_kernel(const NormFwd P) {
    __shared__ double shared[kNormMaxWarps];
    const long long row = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nblk = (P.D + kBlk - 1) / kBlk, D = P.D;
    float s[MB][4], o[MB][4];       // the sum to nearest, and rounded to odd for what keeps fewer bits
    batch_load<VEC, MB>(P.x, P.x_dt, row * P.x_ld, warp, warps, nblk, lane, D, s);
    if (P.residual) batch_load<VEC, MB>(P.residual, P.r_dt, row * D, warp, warps, nblk, lane, D, o);
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = s[m][i], b = P.residual ? o[m][i] : 0.f;
            o[m][i] = add_odd(a, b);
            s[m][i] = a + b;
        }
    double sum = 0;
#pragma unroll
    for (int m = 0; m < MB; ++m)
        sum += (double)fmaf(s[m][0], s[m][0], fmaf(s[m][1], s[m][1], fmaf(s[m][2], s[m][2], s[m][3] * s[m][3])));
    if (P.residual_out) {
        if (P.r_dt == WKV7_BF16) batch_store<VEC, MB>(P.residual_out, WKV7_BF16, row * D, warp, warps, lane, D, o);
        else batch_store<VEC, MB>(P.residual_out, WKV7_F32, row * D, warp, warps, lane, D, s);
    }
    if (P.s_codes) {
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int blk = warp + m * warps;
            if (blk >= nblk) break;
            uint32_t q;
            const float scale = act8_encode(o[m], q);
            row_store_codes<VEC>(P.s_codes + row * D, blk, lane, D, q);
            if (lane == 0) P.s_scales[row * nblk + blk] = scale;
        }
    }
    sum = block_add(sum, shared, warp, warps);
    const double inv = 1.0 / sqrt(sum / D + (double)P.eps);
    const float ih = (float)inv, il = (float)(inv - (double)ih);
    if (P.rstd && threadIdx.x == 0) P.rstd[row] = ih;
    float w[MB][4];
    batch_load<VEC, MB>(P.weight, WKV7_F32, 0, warp, warps, nblk, lane, D, w);
    if (P.y_dt != WKV7_E4M3) {
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[m][i] = s[m][i] * ih * w[m][i];
        batch_store<VEC, MB>(P.y, P.y_dt, row * D, warp, warps, lane, D, s);
        return;
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const int blk = warp + m * warps;
        if (blk >= nblk) break;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float p = s[m][i] * w[m][i], pl = fmaf(s[m][i], w[m][i], -p);
            const float y = p * ih, yl = fmaf(p, ih, -y) + fmaf(pl, ih, p * il);
            const float top = y + yl;
            v[i] = to_odd(top, yl - (top - y));
        }
        uint32_t q;
        const float scale = act8_encode(v, q);
        row_store_codes<VEC>(static_cast<uint8_t *>(P.y) + row * D, blk, lane, D, q);
        if (lane == 0) P.y_scales[row * nblk + blk] = scale;
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
};

// A block takes rows blockIdx.x, + gridDim.x, ...; its share of dw stays in
// registers and goes to partial[blockIdx.x].
template <bool VEC, int MB>
__global__ void __launch_bounds__(32 * kNormMaxWarps)
rmsnorm_bwd_kernel(const NormBwd P) {
    __shared__ float shared[2][kNormMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nblk = (P.D + kBlk - 1) / kBlk, D = P.D;
    float w[MB][4], dw[MB][4];
    batch_load<VEC, MB>(P.weight, WKV7_F32, 0, warp, warps, nblk, lane, D, w);
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[m][i] = 0.f;
    int turn = 0;
    for (long long row = blockIdx.x; row < P.rows; row += gridDim.x, turn ^= 1) {
        float s[MB][4], g[MB][4], d[MB][4], scale[MB];
        batch_load<VEC, MB>(P.s, P.s_dt, row * D, warp, warps, nblk, lane, D, s);
        batch_load<VEC, MB>(P.dy, P.dy_dt, row * D, warp, warps, nblk, lane, D, g);
        if (P.dres) batch_load<VEC, MB>(P.dres, P.g_dt, row * D, warp, warps, nblk, lane, D, d);
        const float rs = __ldg(P.rstd + row);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int blk = warp + m * warps;
            scale[m] = (P.s_dt == WKV7_E4M3 && blk < nblk) ? __ldg(P.s_scales + row * nblk + blk) : 1.f;
        }
        float c = 0.f;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float xh = s[m][i] * scale[m] * rs;
                dw[m][i] = fmaf(g[m][i], xh, dw[m][i]);
                s[m][i] = xh;
                g[m][i] *= w[m][i];
                c = fmaf(g[m][i], xh, c);
            }
        // two buffers in turn: a warp that is a row ahead does not overwrite sums still being read
        c = block_add(c, shared[turn], warp, warps) / (float)D;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = rs * fmaf(-c, s[m][i], g[m][i]);
                s[m][i] = P.dres ? d[m][i] + v : v;
            }
        batch_store<VEC, MB>(P.dx, P.g_dt, row * D, warp, warps, lane, D, s);
    }
    batch_store<VEC, MB>(P.partial, WKV7_F32, (long long)blockIdx.x * D, warp, warps, lane, D, dw);
}

int norm_batch(int nblk) { return nblk <= 8 ? 1 : nblk <= 16 ? 2 : nblk <= 32 ? 4 : 8; }

long long norm_bwd_grid(long long rows, int D) {
    const int sms = sm_count(), nblk = blocks_of(D), mb = norm_batch(nblk);
    if (sms <= 0) return 0;
    const int threads = 32 * ((nblk + mb - 1) / mb);
    // as many rows in flight as the SMs hold at about 100 registers a thread
    const long long most = (long long)sms * (640 / threads > 0 ? 640 / threads : 1);
    return rows < most ? rows : most;
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
    const NormFwd P{D, x_dt, r_dt, y_dt, x, x_ld, residual, weight, eps, residual_out, y, y_scales,
                    (uint8_t *)s_codes, s_scales, rstd};
    const bool vec = D % 4 == 0 && x_ld % 4 == 0 && aligned_to(x, 4 * dtype_size(x_dt)) &&
                     aligned_to(residual, 4 * dtype_size(r_dt)) && aligned_to(residual_out, 4 * dtype_size(r_dt)) &&
                     aligned_to(y, 4 * dtype_size(y_dt)) && aligned_to(weight, 16) && aligned_to(s_codes, 4);
    const int nblk = blocks_of(D), mb = norm_batch(nblk), threads = 32 * ((nblk + mb - 1) / mb);
#define WKV7_NORM(V, M) rmsnorm_fwd_kernel<V, M><<<(unsigned)rows, threads, 0, stream>>>(P)
#define WKV7_NORM_MB(V)                                                                                   \
    (mb == 1 ? (void)(WKV7_NORM(V, 1)) : mb == 2 ? (void)(WKV7_NORM(V, 2)) : mb == 4 ? (void)(WKV7_NORM(V, 4)) \
                                                                            : (void)(WKV7_NORM(V, 8)))
    if (vec) WKV7_NORM_MB(true);
    else WKV7_NORM_MB(false);
#undef WKV7_NORM_MB
#undef WKV7_NORM
    return launch_status();
}

size_t wkv7_rmsnorm_backward_workspace_size(long long rows, int D) {
    using namespace wkv7::mixer;
    if (rows <= 0 || D <= 0 || norm_dims(rows, D) != WKV7_OK) return 0;
    return (size_t)norm_bwd_grid(rows, D) * D * sizeof(float);
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
    const long long grid = norm_bwd_grid(rows, D);
    if (grid <= 0) return WKV7_ERR_CUDA;
    if (workspace == nullptr || !aligned_to(workspace, 16) || workspace_bytes < (size_t)grid * D * sizeof(float))
        return WKV7_ERR_INVALID_ARG;
    const NormBwd P{rows, D, s_dt, dy_dt, g_dt, s, s_scales, rstd, weight, dy, dresidual, dx, (float *)workspace};
    const bool vec = D % 4 == 0 && aligned_to(s, 4 * dtype_size(s_dt)) && aligned_to(dy, 4 * dtype_size(dy_dt)) &&
                     aligned_to(dresidual, 4 * dtype_size(g_dt)) && aligned_to(dx, 4 * dtype_size(g_dt)) &&
                     aligned_to(weight, 16);
    const int nblk = blocks_of(D), mb = norm_batch(nblk), threads = 32 * ((nblk + mb - 1) / mb);
#define WKV7_NORM(V, M) rmsnorm_bwd_kernel<V, M><<<(unsigned)grid, threads, 0, stream>>>(P)
#define WKV7_NORM_MB(V)                                                                                   \
    (mb == 1 ? (void)(WKV7_NORM(V, 1)) : mb == 2 ? (void)(WKV7_NORM(V, 2)) : mb == 4 ? (void)(WKV7_NORM(V, 4)) \
                                                                            : (void)(WKV7_NORM(V, 8)))
    if (vec) WKV7_NORM_MB(true);
    else WKV7_NORM_MB(false);
#undef WKV7_NORM_MB
#undef WKV7_NORM
    sum_parts(grid, D, (const float *)workspace, dweight, stream);
    return launch_status();
}

}  // extern "C"
