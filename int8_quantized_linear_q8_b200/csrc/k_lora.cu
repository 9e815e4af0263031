// k_lora.cu -- the small products of the low-rank adapters beside the W8A16 linear:
//
//   h[m,r]     = sum_k x[m,k] A[i][r,k]                      i = ids[m]
//   g[m,r]     = c[i] sum_n dy[m,n] B[i][n,r]
//   dA[i][r,k] = sum_{m: ids[m] = i} g[m,r] x[m,k]
//   dB[i][n,r] = sum_{m: ids[m] = i} dy[m,n] (c[i] h[m,r])
#include "q8_kernels.cuh"

namespace q8 {

__device__ __forceinline__ float bf16_at(const uint16_t* p) {
    return __uint_as_float((uint32_t)__ldg(p) << 16);
}
// the value an exponent byte stands for: 2^(b - 127), 1 <= b <= 248
__device__ __forceinline__ float pow2_of(uint32_t b) { return __uint_as_float(b << 23); }

// h[m, r] (a warp per value): the row of its adapter's A against x, or, backward, the
// column of its B against dy, times the adapter's scale.
template <bool BWD>
__global__ __launch_bounds__(256) void k_lora_shrink_plain(const uint16_t* x, const uint16_t* w,
                                                           const float* scale, const int32_t* ids,
                                                           float* h, int64_t M, int C, int R,
                                                           int L) {
    const int64_t m = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const int id = __ldg(ids + m);
    for (int r = threadIdx.x >> 5; r < R; r += 8) {
        float v = 0.0f;
        if (id >= 0 && id < L)
            for (int c = lane; c < C; c += 32)
                v = fmaf(bf16_at(x + m * C + c),
                         bf16_at(w + (BWD ? ((int64_t)id * C + c) * R + r
                                          : ((int64_t)id * R + r) * C + c)),
                         v);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) h[m * R + r] = BWD && id >= 0 && id < L ? v * __ldg(scale + id) : v;
    }
}

// dA[i][r][p] (BYROW) or dB[i][p][r]: a thread per p, one adapter and r a block.
template <bool DB>
__global__ __launch_bounds__(128) void k_lora_wgrad_plain(const void* x, const uint8_t* exps, int G,
                                                          const float* low, const float* scale,
                                                          const int32_t* ids, float* out,
                                                          int accumulate, int64_t M, int P, int R) {
    const int p = blockIdx.x * 128 + threadIdx.x, r = blockIdx.y, i = blockIdx.z;
    if (p >= P) return;
    float v = 0.0f;
    for (int64_t m = 0; m < M; ++m) {
        if (__ldg(ids + m) != i) continue;
        float xv;
        if (G == 0)
            xv = bf16_at(reinterpret_cast<const uint16_t*>(x) + m * P + p);
        else
            xv = (float)reinterpret_cast<const int8_t*>(x)[m * P + p] *
                 pow2_of(exps[m * (P / G) + p / G]);
        v = fmaf(DB ? low[m * R + r] * __ldg(scale + i) : low[m * R + r], xv, v);
    }
    float* o = out + (DB ? ((int64_t)i * P + p) * R + r : ((int64_t)i * R + r) * P + p);
    *o = accumulate ? *o + v : v;
}

cudaError_t launch_lora_shrink(bool bwd, const uint16_t* x, const uint16_t* w, const float* scale,
                               const int32_t* ids, float* h, int64_t M, int C, int R, int L,
                               cudaStream_t st) {
    if (bwd)
        k_lora_shrink_plain<true><<<(unsigned)M, 256, 0, st>>>(x, w, scale, ids, h, M, C, R, L);
    else
        k_lora_shrink_plain<false><<<(unsigned)M, 256, 0, st>>>(x, w, scale, ids, h, M, C, R, L);
    return cudaGetLastError();
}

cudaError_t launch_lora_wgrad(bool db, const void* x, const uint8_t* exps, int G, const float* low,
                              const float* scale, const int32_t* ids, float* out, int accumulate,
                              int64_t M, int P, int R, int L, cudaStream_t st) {
    const dim3 grid((P + 127) / 128, R, L);
    if (db)
        k_lora_wgrad_plain<true><<<grid, 128, 0, st>>>(x, exps, G, low, scale, ids, out,
                                                       accumulate, M, P, R);
    else
        k_lora_wgrad_plain<false><<<grid, 128, 0, st>>>(x, exps, G, low, scale, ids, out,
                                                        accumulate, M, P, R);
    return cudaGetLastError();
}

}  // namespace q8
