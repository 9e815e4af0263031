// k_lora_decode.cu -- the low-rank term of up to 16 rows (decode), each with its own adapter:
//
//   h[m,r] = sum_k x[m,k] A[i][r,k]                              i = ids[m]
//   t[m,n] = bias[n] + c[i] sum_r h[m,r] B[i][n,r]
//
// t is what k_w8a16_tma's epilogue adds to s_w[n] * sum_k x q.  Rows share nothing here but the
// projection, so there is no product of matrices to form: each row reads its adapter once,
// M * rank * (K + N) * 2 bytes in all, against N * K of the int8 weight.
//
// A cluster of eight CTAs per row: its 64 warps share out the rank's rows of A (and parts of K
// when the rank is below 64), every warp leaves its sums in all eight CTAs' shared memory (behind
// a cluster barrier, since the others have to have started), and after a second barrier each CTA
// makes an eighth of the row of t.  The kernel lets the weight stream start as soon as the stream's
// earlier work is done (programmatic dependent launch); the stream waits for t only when its first
// rows are summed.
//
// 16 rows, 4096 x 11008, rank 16, 32 adapters: this kernel 6 us (h 2.7, t 3.2), the whole call 19.9 us
// back to back, the plain linear 14; 1 row, 960 x 2560, rank 8: 4.9 and 3.9 us.  What is left is the
// chain itself: the stream's CTAs of the larger shapes need the registers of the SMs that this
// kernel's CTAs still hold, so 50 to 130 of its 148 start when those end.  Not kept: a stream
// held to 128 registers, whose CTAs start at once (21.7 to 25 us: they slow this kernel down and
// wait for it all the same); this kernel on 128 threads (23.2); two kernels, h and t (5 us more).
#include "q8_kernels.cuh"

namespace q8 {

constexpr int LD_CTAS = 8, LD_WARPS = 8, LD_THREADS = 32 * LD_WARPS;
constexpr int LD_SUMS = 256;                // rank (at most 256) times parts of K (at most 64 / rank)

__global__ __cluster_dims__(LD_CTAS, 1, 1) __launch_bounds__(LD_THREADS) void k_lora_decode(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ A,
    const uint16_t* __restrict__ B, const float* __restrict__ scale,
    const float* __restrict__ bias, const int32_t* __restrict__ ids, float* __restrict__ h,
    float* __restrict__ t, int64_t N, int K, int R, int L) {
    __shared__ float sums[LD_SUMS];
    __shared__ __align__(16) float hs[256];
    // A CTA's shared memory may be written by another once it runs: each says so here and waits for
    // the others before its first sum leaves, by when the id has been read and they have.
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int m = blockIdx.y, part = blockIdx.x;            // a row's cluster: its CTAs in order
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int id = ld_after(ids + m);
    const bool has = id >= 0 && id < L;
    const int64_t n0 = N * part / LD_CTAS, n1 = N * (part + 1) / LD_CTAS;
    if (has) {
        // this CTA's rows of B on their way to L2 while h is made
        const char* b0 = reinterpret_cast<const char*>(B + ((int64_t)id * N + n0) * R);
        const int64_t bytes = (n1 - n0) * R * 2;
        for (int64_t o = (int64_t)tid * 128; o < bytes; o += LD_THREADS * 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(b0 + o) : "memory");
    }
    // h: sum j = r * parts + q is row r of A over the q-th part of K
    const int parts = R >= 64 ? 1 : 64 / R;
    const int chunks = (K + 255) / 256;                     // of 256 k: 8 a lane
    const uint32_t out = (uint32_t)__cvta_generic_to_shared(sums);
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int j = part * LD_WARPS + warp; j < R * parts; j += LD_CTAS * LD_WARPS) {
        float v = 0.0f;
        if (has) {
            const int r = j / parts, q = j - r * parts;
            const uint16_t* xp = x + (int64_t)m * K;
            const uint16_t* ap = A + ((int64_t)id * R + r) * K;
            const int c1 = chunks * (q + 1) / parts;
#pragma unroll 8
            for (int c = chunks * q / parts; c < c1; ++c) {
                const int k = c * 256 + lane * 8;
                if (k >= K) break;
                const uint4 a = ld_after16(ap + k), b = ld_after16(xp + k);
                v = fmaf(bf16lo(a.x), bf16lo(b.x), v);
                v = fmaf(bf16hi(a.x), bf16hi(b.x), v);
                v = fmaf(bf16lo(a.y), bf16lo(b.y), v);
                v = fmaf(bf16hi(a.y), bf16hi(b.y), v);
                v = fmaf(bf16lo(a.z), bf16lo(b.z), v);
                v = fmaf(bf16hi(a.z), bf16hi(b.z), v);
                v = fmaf(bf16lo(a.w), bf16lo(b.w), v);
                v = fmaf(bf16hi(a.w), bf16hi(b.w), v);
            }
            __syncwarp();
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        }
        if (lane < LD_CTAS)                                 // a copy for every CTA
            asm volatile(
                "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
                "st.shared::cluster.f32 [a], %2;\n\t}" ::"r"(out + j * 4),
                "r"(lane), "f"(v)
                : "memory");
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int r = tid; r < R; r += LD_THREADS) {
        float v = 0.0f;
        for (int q = 0; q < parts; ++q) v += sums[r * parts + q];
        hs[r] = v;
        if (part == 0) h[(int64_t)m * R + r] = v;
    }
    __syncthreads();
    // t: three n a thread at a time, their rows of B in 16-byte pieces
    const float c = has ? ld_after(scale + id) : 0.0f;
    constexpr int U = 3;
    for (int64_t n = n0 + tid; n < n1; n += U * LD_THREADS) {
        float v[U] = {};
        if (has) {
            const uint16_t* bp = B + ((int64_t)id * N + n) * R;
#pragma unroll 2
            for (int r = 0; r < R; r += 8) {
                uint4 b[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    b[u] = n + u * LD_THREADS < n1
                               ? ld_after16(bp + (int64_t)u * LD_THREADS * R + r)
                               : make_uint4(0, 0, 0, 0);
                const float4 h0 = *reinterpret_cast<const float4*>(hs + r);
                const float4 h1 = *reinterpret_cast<const float4*>(hs + r + 4);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    v[u] = fmaf(bf16lo(b[u].x), h0.x, v[u]);
                    v[u] = fmaf(bf16hi(b[u].x), h0.y, v[u]);
                    v[u] = fmaf(bf16lo(b[u].y), h0.z, v[u]);
                    v[u] = fmaf(bf16hi(b[u].y), h0.w, v[u]);
                    v[u] = fmaf(bf16lo(b[u].z), h1.x, v[u]);
                    v[u] = fmaf(bf16hi(b[u].z), h1.y, v[u]);
                    v[u] = fmaf(bf16lo(b[u].w), h1.z, v[u]);
                    v[u] = fmaf(bf16hi(b[u].w), h1.w, v[u]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t nn = n + u * LD_THREADS;
            if (nn < n1) t[(int64_t)m * N + nn] = bias ? fmaf(v[u], c, ld_after(bias + nn)) : v[u] * c;
        }
    }
}

cudaError_t launch_lora_decode(const uint16_t* x, const uint16_t* A, const uint16_t* B,
                               const float* scale, const float* bias, const int32_t* ids, float* h,
                               float* t, int M, int64_t N, int K, int R, int L, cudaStream_t st) {
    prefer_shared_memory<k_lora_decode>();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(LD_CTAS, M);
    cfg.blockDim = dim3(LD_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_lora_decode, x, A, B, scale, bias, ids, h, t, N, K, R, L);
}

}  // namespace q8
