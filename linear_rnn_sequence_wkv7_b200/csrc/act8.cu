// 8-bit activations by themselves: wkv7_act8_save and wkv7_act8_load.  A warp
// holds a block of 128 channels, four values a lane, and takes eight blocks in a
// row with their loads issued together.  Bound by memory: 3 bytes a bf16 element.
#include "mixer.cuh"

namespace wkv7 {
namespace mixer {
namespace {

// (row, block) of consecutive units: one division a warp
struct Unit {
    long long row;
    int blk;
    __device__ __forceinline__ Unit(long long u, int nblk) : row(u / nblk), blk((int)(u % nblk)) {}
    __device__ __forceinline__ void next(int nblk) {
        if (++blk == nblk) blk = 0, ++row;
    }
};

constexpr int kActWarps = 8, kActBatch = 8;

template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kActWarps)
act8_save_kernel(long long units, int nblk, int D, const T *__restrict__ x, long long x_ld,
                 uint8_t *__restrict__ codes, float *__restrict__ scales) {
    const int lane = threadIdx.x & 31;
    const long long first = ((long long)blockIdx.x * kActWarps + (threadIdx.x >> 5)) * kActBatch;
    const Unit start(first, nblk);
    Row4<T, VEC> v[kActBatch];
    Unit at = start;
#pragma unroll
    for (int m = 0; m < kActBatch; ++m, at.next(nblk)) v[m].load(x + at.row * x_ld, at.blk, lane, first + m < units ? D : 0);
    at = start;
#pragma unroll
    for (int m = 0; m < kActBatch; ++m, at.next(nblk)) {
        if (first + m >= units) break;
        uint32_t q;
        float f[4];
        v[m].get(f);
        const float scale = act8_encode(f, q);
        row_store_codes<VEC>(codes + at.row * D, at.blk, lane, D, q);
        if (lane == 0) scales[first + m] = scale;
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kActWarps)
act8_load_kernel(long long units, int nblk, int D, const e4m3 *__restrict__ codes,
                 const float *__restrict__ scales, T *__restrict__ out) {
    const int lane = threadIdx.x & 31;
    const long long first = ((long long)blockIdx.x * kActWarps + (threadIdx.x >> 5)) * kActBatch;
    const Unit start(first, nblk);
    Row4<e4m3, VEC> v[kActBatch];
    float s[kActBatch];
    Unit at = start;
#pragma unroll
    for (int m = 0; m < kActBatch; ++m, at.next(nblk)) {
        v[m].load(codes + at.row * D, at.blk, lane, first + m < units ? D : 0);
        s[m] = first + m < units ? __ldg(scales + first + m) : 0.f;
    }
    at = start;
#pragma unroll
    for (int m = 0; m < kActBatch; ++m, at.next(nblk)) {
        if (first + m >= units) break;
        float f[4];
        v[m].get(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] *= s[m];
        row_store<VEC>(out + at.row * D, at.blk, lane, D, f);
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
