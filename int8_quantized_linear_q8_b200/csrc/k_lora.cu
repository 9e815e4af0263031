// k_lora.cu -- low-rank adapters beside the W8A16 linear, forward and backward, and the
// weight gradient from an 8-bit checkpoint: plain shared-memory tiles on the fp32 pipes.
//
//   y[m,n]  = s_w[n] sum_k x[m,k] q[n,k] + bias[n] + c[i] sum_r h[m,r] B[i][n,r],  i = ids[m]
//   h[m,r]  = sum_k x[m,k] A[i][r,k]
//   g[m,r]  = c[i] sum_n dy[m,n] B[i][n,r]
//   dx[m,k] = sum_n dy[m,n] s_w[n] q[n,k] + sum_r g[m,r] A[i][r,k]
//   dA[i][r,k] = sum_{m: ids[m] = i} g[m,r] x[m,k]
//   dB[i][n,r] = c[i] sum_{m: ids[m] = i} dy[m,n] h[m,r]
//   dW[n,k] = sum_m dy[m,n] xhat[m,k]
//
// The three large products share one kernel: out[t, p] = sum_c P(p, c) T(t, c).
#include "q8_kernels.cuh"

namespace q8 {

constexpr int LS_TILE = 64, LS_BK = 16;

__device__ __forceinline__ float bf16_at(const uint16_t* p) {
    return __uint_as_float((uint32_t)__ldg(p) << 16);
}
// the value an exponent byte stands for: 2^(b - 127), 1 <= b <= 248
__device__ __forceinline__ float pow2_of(uint32_t b) { return __uint_as_float(b << 23); }

template <int MODE>
__global__ __launch_bounds__(256) void k_lora_gemm_plain(LoraGemm a) {
    __shared__ float sp[LS_BK][LS_TILE + 1], st[LS_BK][LS_TILE + 1];
    const int p0 = blockIdx.x * LS_TILE;
    const int64_t t0 = (int64_t)blockIdx.y * LS_TILE;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int c0 = 0; c0 < a.C; c0 += LS_BK) {
        for (int u = threadIdx.x; u < LS_BK * LS_TILE; u += 256) {
            float vp = 0.0f, vt = 0.0f;
            if (MODE == LORA_FWD) {
                const int cc = u % LS_BK, r = u / LS_BK, c = c0 + cc;
                if (c < a.C && p0 + r < a.P) vp = (float)a.q[(int64_t)(p0 + r) * a.C + c];
                if (c < a.C && t0 + r < a.T) vt = bf16_at(a.t + (t0 + r) * a.C + c);
                sp[cc][r] = vp;
                st[cc][r] = vt;
            } else {
                const int cc = u / LS_TILE, r = u % LS_TILE, c = c0 + cc;
                if (c < a.C && p0 + r < a.P) {
                    vp = (float)a.q[(int64_t)c * a.P + p0 + r];
                    vp *= MODE == LORA_DGRAD
                              ? __ldg(a.s_w + c)
                              : pow2_of(a.exps[(int64_t)c * (a.P / a.G) + (p0 + r) / a.G]);
                }
                sp[cc][r] = vp;
                if (MODE == LORA_WGRAD) {
                    if (c < a.C && t0 + r < a.T) vt = bf16_at(a.t + (int64_t)c * a.T + t0 + r);
                    st[cc][r] = vt;
                } else {
                    const int c2 = u % LS_BK, r2 = u / LS_BK;
                    if (c0 + c2 < a.C && t0 + r2 < a.T)
                        vt = bf16_at(a.t + (t0 + r2) * a.C + c0 + c2);
                    st[c2][r2] = vt;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int cc = 0; cc < LS_BK; ++cc)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(st[cc][ty * 4 + i], sp[cc][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + ty * 4 + i;
        if (t >= a.T) continue;
        const int id = a.ids ? __ldg(a.ids + t) : -1;
        for (int j = 0; j < 4; ++j) {
            const int p = p0 + tx + 16 * j;
            if (p >= a.P) continue;
            float v = acc[i][j];
            if (MODE == LORA_FWD) v = fmaf(v, __ldg(a.s_w + p), a.bias ? __ldg(a.bias + p) : 0.0f);
            if (MODE != LORA_WGRAD && id >= 0 && id < a.L) {
                float low = 0.0f;
                for (int r = 0; r < a.R; ++r)
                    low = fmaf(a.h[t * a.R + r],
                               MODE == LORA_FWD
                                   ? bf16_at(a.low + ((int64_t)id * a.P + p) * a.R + r)
                                   : bf16_at(a.low + ((int64_t)id * a.R + r) * a.P + p),
                               low);
                v += MODE == LORA_FWD ? __ldg(a.scale + id) * low : low;
            }
            const int64_t at = t * a.P + p;
            if (a.out_bf16)
                reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
            else {
                float* o = reinterpret_cast<float*>(a.out) + at;
                *o = a.accumulate ? *o + v : v;
            }
        }
    }
}

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

cudaError_t launch_lora_gemm(int mode, const LoraGemm& a, cudaStream_t st) {
    const dim3 grid((a.P + LS_TILE - 1) / LS_TILE, (unsigned)((a.T + LS_TILE - 1) / LS_TILE));
    if (mode == LORA_FWD)
        k_lora_gemm_plain<LORA_FWD><<<grid, 256, 0, st>>>(a);
    else if (mode == LORA_DGRAD)
        k_lora_gemm_plain<LORA_DGRAD><<<grid, 256, 0, st>>>(a);
    else
        k_lora_gemm_plain<LORA_WGRAD><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
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
