// 8-bit activations by themselves: wkv7_act8_save and wkv7_act8_load.  A warp
// holds a block of 128 channels, four values a lane, so amax is five shuffles;
// each warp takes four blocks and issues their loads together.  Bound by memory:
// 3 bytes a bf16 element.
#include "mixer.cuh"

namespace wkv7 {
namespace mixer {
namespace {

constexpr int kActWarps = 8, kActBatch = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kActWarps)
act8_save_kernel(long long units, int nblk, int D, const T *__restrict__ x, long long x_ld,
                 uint8_t *__restrict__ codes, float *__restrict__ scales) {
    const int lane = threadIdx.x & 31;
    const long long first = ((long long)blockIdx.x * kActWarps + (threadIdx.x >> 5)) * kActBatch;
    float v[kActBatch][4];
#pragma unroll
    for (int m = 0; m < kActBatch; ++m) {
        const long long u = first + m;
        if (u < units) row_load<VEC>(x + (u / nblk) * x_ld, (int)(u % nblk), lane, D, v[m]);
    }
#pragma unroll
    for (int m = 0; m < kActBatch; ++m) {
        const long long u = first + m;
        if (u >= units) break;
        uint32_t q;
        const float scale = act8_encode(v[m], q);
        row_store_codes<VEC>(codes + (u / nblk) * D, (int)(u % nblk), lane, D, q);
        if (lane == 0) scales[u] = scale;
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kActWarps)
act8_load_kernel(long long units, int nblk, int D, const e4m3 *__restrict__ codes,
                 const float *__restrict__ scales, T *__restrict__ out) {
    const int lane = threadIdx.x & 31;
    const long long first = ((long long)blockIdx.x * kActWarps + (threadIdx.x >> 5)) * kActBatch;
    float v[kActBatch][4], s[kActBatch];
#pragma unroll
    for (int m = 0; m < kActBatch; ++m) {
        const long long u = first + m;
        if (u < units) {
            row_load<VEC>(codes + (u / nblk) * D, (int)(u % nblk), lane, D, v[m]);
            s[m] = __ldg(scales + u);
        }
    }
#pragma unroll
    for (int m = 0; m < kActBatch; ++m) {
        const long long u = first + m;
        if (u >= units) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[m][i] *= s[m];
        row_store<VEC>(out + (u / nblk) * D, (int)(u % nblk), lane, D, v[m]);
    }
}

wkv7_status act8_dims(long long rows, int D, long long &blocks) {
    if (rows < 0 || D < 0) return WKV7_ERR_INVALID_ARG;
    if (D > WKV7_SSM_MAX_D) return WKV7_ERR_UNSUPPORTED;
    const long long per = kActWarps * kActBatch;
    if (rows > kMaxGrid) return WKV7_ERR_UNSUPPORTED;
    blocks = (rows * blocks_of(D) + per - 1) / per;
    return blocks > kMaxGrid ? WKV7_ERR_UNSUPPORTED : WKV7_OK;
}

}  // namespace
}  // namespace mixer
}  // namespace wkv7

extern "C" {

wkv7_status wkv7_act8_save(long long rows, int D, wkv7_dtype x_dt, const void *x, long long x_ld, void *codes,
                           float *scales, cudaStream_t stream) {
    using namespace wkv7::mixer;
    long long blocks = 0;
    const wkv7_status s = act8_dims(rows, D, blocks);
    if (s != WKV7_OK) return s;
    if (!real_dtype(x_dt) || x_ld < 0) return WKV7_ERR_INVALID_ARG;
    if (rows == 0 || D == 0) return WKV7_OK;
    if (!elem_ok(x, x_dt) || codes == nullptr || !f32_ok(scales)) return WKV7_ERR_INVALID_ARG;
    const bool vec = D % 4 == 0 && x_ld % 4 == 0 && aligned_to(x, 4 * dtype_size(x_dt)) && aligned_to(codes, 4);
    const int nblk = blocks_of(D);
    const long long units = rows * nblk;
#define WKV7_SAVE(T, V)                                                                                          \
    act8_save_kernel<T, V><<<(unsigned)blocks, 32 * kActWarps, 0, stream>>>(units, nblk, D, (const T *)x, x_ld, \
                                                                             (uint8_t *)codes, scales)
    if (x_dt == WKV7_F32) {
        if (vec) WKV7_SAVE(float, true);
        else WKV7_SAVE(float, false);
    } else {
        if (vec) WKV7_SAVE(bf16, true);
        else WKV7_SAVE(bf16, false);
    }
#undef WKV7_SAVE
    return launch_status();
}

wkv7_status wkv7_act8_load(long long rows, int D, const void *codes, const float *scales, wkv7_dtype out_dt,
                           void *out, cudaStream_t stream) {
    using namespace wkv7::mixer;
    long long blocks = 0;
    const wkv7_status s = act8_dims(rows, D, blocks);
    if (s != WKV7_OK) return s;
    if (!real_dtype(out_dt)) return WKV7_ERR_INVALID_ARG;
    if (rows == 0 || D == 0) return WKV7_OK;
    if (!elem_ok(out, out_dt) || codes == nullptr || !f32_ok(scales)) return WKV7_ERR_INVALID_ARG;
    const bool vec = D % 4 == 0 && aligned_to(out, 4 * dtype_size(out_dt)) && aligned_to(codes, 4);
    const int nblk = blocks_of(D);
    const long long units = rows * nblk;
#define WKV7_LOAD(T, V)                                                                       \
    act8_load_kernel<T, V><<<(unsigned)blocks, 32 * kActWarps, 0, stream>>>(                  \
        units, nblk, D, (const e4m3 *)codes, scales, (T *)out)
    if (out_dt == WKV7_F32) {
        if (vec) WKV7_LOAD(float, true);
        else WKV7_LOAD(float, false);
    } else {
        if (vec) WKV7_LOAD(bf16, true);
        else WKV7_LOAD(bf16, false);
    }
#undef WKV7_LOAD
    return launch_status();
}

}  // extern "C"
