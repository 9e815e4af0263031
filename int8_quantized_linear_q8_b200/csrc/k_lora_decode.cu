// k_lora_decode.cu -- the low-rank term of up to 16 rows (decode), each with its own adapter:
//
//   h[m,r] = sum_k x[m,k] A[i][r,k]                              i = ids[m]
//   t[m,n] = bias[n] + c[i] sum_r h[m,r] B[i][n,r]
//
// t is what k_w8a16_tma's epilogue adds to s_w[n] * sum_k x q.  Rows share nothing here but the
// projection, so there is no product of matrices to form: each row reads its adapter once,
// M * rank * (K + N) * 2 bytes in all, against N * K of the int8 weight.  The three kernels are
// chained by programmatic dependent launch so that the weight stream starts at once: the
// first waits for the stream's earlier work before it lets the others start, the second lets
// the stream start before it waits for h, and the stream waits for t only when its first rows
// are summed.
#include "q8_kernels.cuh"

namespace q8 {

// A warp per h value: 16-byte pieces of the adapter row and of x, 256 k a turn.
__global__ __launch_bounds__(128) void k_lora_decode_h(const uint16_t* __restrict__ x,
                                                       const uint16_t* __restrict__ A,
                                                       const int32_t* __restrict__ ids,
                                                       float* __restrict__ h, int K, int R, int L) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int m = blockIdx.x, r = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r >= R) return;
    const int id = __ldg(ids + m);
    float v = 0.0f;
    if (id >= 0 && id < L) {
        const uint16_t* xp = x + (int64_t)m * K;
        const uint16_t* ap = A + ((int64_t)id * R + r) * K;
#pragma unroll 8
        for (int k = lane * 8; k < K; k += 256) {
            const uint4 a = ldg_keep(ap + k), b = ldg_keep(xp + k);
            v = fmaf(bf16lo(a.x), bf16lo(b.x), v);
            v = fmaf(bf16hi(a.x), bf16hi(b.x), v);
            v = fmaf(bf16lo(a.y), bf16lo(b.y), v);
            v = fmaf(bf16hi(a.y), bf16hi(b.y), v);
            v = fmaf(bf16lo(a.z), bf16lo(b.z), v);
            v = fmaf(bf16hi(a.z), bf16hi(b.z), v);
            v = fmaf(bf16lo(a.w), bf16lo(b.w), v);
            v = fmaf(bf16hi(a.w), bf16hi(b.w), v);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    if (lane == 0) h[(int64_t)m * R + r] = v;
}

// A thread per t value: its row of B, 16 bytes at a time, against h.
__global__ __launch_bounds__(128) void k_lora_decode_t(const float* __restrict__ h,
                                                       const uint16_t* __restrict__ B,
                                                       const float* __restrict__ scale,
                                                       const float* __restrict__ bias,
                                                       const int32_t* __restrict__ ids,
                                                       float* __restrict__ t, int64_t N, int R,
                                                       int L) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int m = blockIdx.y;
    const int64_t n = (int64_t)blockIdx.x * 128 + threadIdx.x;
    // ids, B and the bias are not written by the kernel before this one
    const int id = __ldg(ids + m);
    const bool has = id >= 0 && id < L;
    const uint16_t* bp = B + ((int64_t)(has ? id : 0) * N + (n < N ? n : 0)) * R;
    uint4 first = make_uint4(0, 0, 0, 0);
    if (has && n < N) first = ldg_keep(bp);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n >= N) return;
    float v = 0.0f;
    if (has) {
        const float* hp = h + (int64_t)m * R;
        for (int r = 0; r < R; r += 8) {
            const uint4 b = r == 0 ? first : ldg_keep(bp + r);
            const float4 h0 = ld_after4(hp + r), h1 = ld_after4(hp + r + 4);
            v = fmaf(bf16lo(b.x), h0.x, v);
            v = fmaf(bf16hi(b.x), h0.y, v);
            v = fmaf(bf16lo(b.y), h0.z, v);
            v = fmaf(bf16hi(b.y), h0.w, v);
            v = fmaf(bf16lo(b.z), h1.x, v);
            v = fmaf(bf16hi(b.z), h1.y, v);
            v = fmaf(bf16lo(b.w), h1.z, v);
            v = fmaf(bf16hi(b.w), h1.w, v);
        }
        v *= __ldg(scale + id);
    }
    t[(int64_t)m * N + n] = bias ? v + __ldg(bias + n) : v;
}

cudaError_t launch_lora_decode(const uint16_t* x, const uint16_t* A, const uint16_t* B,
                               const float* scale, const float* bias, const int32_t* ids, float* h,
                               float* t, int M, int64_t N, int K, int R, int L, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(M, (R + 3) / 4);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_lora_decode_h, x, A, ids, h, K, R, L);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)((N + 127) / 128), M);
    return cudaLaunchKernelEx(&cfg, k_lora_decode_t, (const float*)h, B, scale, bias, ids, t, N, R,
                              L);
}

}  // namespace q8
