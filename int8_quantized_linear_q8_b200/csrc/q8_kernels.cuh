// q8_kernels.cuh -- launcher declarations and device code shared between kernel files.
#pragma once

#include "q8_common.cuh"

namespace q8 {

// Sixteen static activation codes (first pass, and the two-pass residual's codes):
//   c1 = clamp(round(v * (1/s1)) + z1, -128, 127)
//   r  = v - (c1 - z1) * s1          (fp32 product, then fp32 difference; no FMA)
//   c2 = clamp(round(r * (1/s2)) + z2, -128, 127)
// packed four codes per word, lowest k in the lowest byte.
__device__ __forceinline__ void static_codes16(const float (&v)[16], float s1, float inv1,
                                               float z1f, int has2, float inv2, float z2f,
                                               uint32_t (&o1)[4], uint32_t (&o2)[4]) {
    int c1[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) c1[j] = act_code(v[j], inv1, z1f);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o1[j] = pack4_s8(c1[4 * j], c1[4 * j + 1], c1[4 * j + 2], c1[4 * j + 3]);
    if (has2) {
        int c2[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            float d1 = __fmul_rn(__fsub_rn((float)c1[j], z1f), s1);
            float r = __fsub_rn(v[j], d1);
            c2[j] = act_code(r, inv2, z2f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o2[j] = pack4_s8(c2[4 * j], c2[4 * j + 1], c2[4 * j + 2], c2[4 * j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) o2[j] = 0u;
    }
}

// Four int8 codes -> bf16 (b0, b1), (b2, b3), exact: as s8x4_to_bf16x2_eo, in order.
__device__ __forceinline__ void s8x4_to_bf16x2_seq(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t l = __byte_perm(w, 0, 0x4140), h = __byte_perm(w, 0, 0x4342);
    lo = bf16x2_sub(lop_and_or(l, 0x007F007Fu, 0x43004300u),
                    lop_and_or(l, 0x00800080u, 0x43004300u));
    hi = bf16x2_sub(lop_and_or(h, 0x007F007Fu, 0x43004300u),
                    lop_and_or(h, 0x00800080u, 0x43004300u));
}
__device__ __forceinline__ uint32_t bf16x2_mulrn(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t bf16_bits_rn(float v) {
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Loads of what an earlier kernel may have written, in kernels that start before it ends
// (programmatic dependent launch): volatile, so that none is moved ahead of the
// griddepcontrol.wait before it, as the compiler may a __ldg, and without the promise of ld.global.nc
// (ldg_stream and its like) that the memory does not change while the kernel lives.
__device__ __forceinline__ int ld_after(const int* p) {
    int v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float ld_after(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_after(const uint8_t* p) {
    uint32_t v;
    asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// 16 bytes at once: kept in L1 (small operands re-read by many warps), or streamed past it
__device__ __forceinline__ uint4 ld_after16(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint4 ld_after16_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// q8_abi.cu: host checks shared with the allocation-free entry point
q8_status w8a8_check_args(const float* x, const q8_qparams& first, const q8_qparams* second,
                          const int8_t* q, const int32_t* wsum, const float* s_w,
                          const float* bias, const float* y, int64_t M, int64_t N, int64_t K);
q8_status check_current_device();

// k_w4a16.cu (NVFP4 weight-only twin)
cudaError_t launch_quantize_weight_nvfp4(const float* W, int64_t N, int K, uint8_t* q4,
                                         uint8_t* sf, float* gsc, cudaStream_t st, int num_sms);
cudaError_t launch_w4a16_nvfp4(const uint16_t* x, const uint8_t* q4, const uint8_t* sf,
                               const float* gsc, void* y, int y_bf16, int64_t M, int64_t N, int K,
                               cudaStream_t st);

// k_quant.cu
// full: 0 = amax/127 on +-127, 1 = max(amax/127.5, FLT_EPSILON) on [-128, 127]
cudaError_t launch_quantize_weight(const float* W, int64_t N, int K, int full, int8_t* q,
                                   float* s_w, int32_t* wsum, cudaStream_t st);
cudaError_t launch_choose_qparams(const uint16_t* x, int64_t M, int K, float* s, int32_t* z,
                                  int8_t* xq, cudaStream_t st);
cudaError_t launch_choose_qparams_shifted(const uint16_t* x, int64_t M, int K, float* s,
                                          int32_t* z, uint16_t* xz, cudaStream_t st);
cudaError_t launch_quantize_static(const float* x, int64_t M, int K, float s1, int z1, int has2,
                                   float s2, int z2, int8_t* xq1, int8_t* xq2, cudaStream_t st,
                                   int num_sms);
// residual != 0: observe x - fake_quant(x, s1, z1) instead of x
cudaError_t launch_observe_minmax(const float* x, int64_t n, float* mm, int reset, int residual,
                                  float s1, int z1, cudaStream_t st, int num_sms);
cudaError_t launch_quantize_weight_q4gs(const float* W, int64_t N, int K, int G, uint8_t* q4,
                                        float* gs, cudaStream_t st);
cudaError_t launch_q4gs_zero_fold(const uint8_t* q4, const float* gs, int G, int64_t N, int K,
                                  float* c, cudaStream_t st);

// k_gemv_tma.cu
bool make_tmap_u8_2d(CUtensorMap* map, const void* base, int64_t rows, int64_t cols,
                     int box_cols, int box_rows, CUtensorMapSwizzle swz);
bool w8a16_tma_fits(int64_t M, int64_t K, bool bias = false);
// bias (nullable, fp32 [N]) is added after the scale in every linear launcher below
cudaError_t launch_w8a16_tma(const uint16_t* x, const int8_t* q, const float* s_w,
                             const float* bias, void* y, int y_bf16, int64_t M, int64_t N, int K,
                             cudaStream_t st, int num_sms, int* status, bool low = false);
// low: `bias` is an fp32 [M, N] term that the stream's last kernel writes
// (launch_lora_decode, and only that: see k_w8a16_tma)

// k_lora_decode.cu: h [M, R] and the term t [M, N] of up to 16 rows
cudaError_t launch_lora_decode(const uint16_t* x, const uint16_t* A, const uint16_t* B,
                               const float* scale, const float* bias, const int32_t* ids, float* h,
                               float* t, int M, int64_t N, int K, int R, int L, cudaStream_t st);

// k_gemm_tc.cu
cudaError_t launch_gemm_s8s8_s32_tc(const int8_t* a, const int8_t* b, int32_t* acc, int64_t M,
                                    int64_t N, int K, cudaStream_t st, int num_sms, int* status);
cudaError_t launch_w8a8_tc(const int8_t* xq1, const int8_t* xq2, float s1, int z1, int has2,
                           float s2, int z2, const int8_t* q, const int32_t* wsum,
                           const float* s_w, const float* bias, float* y, int64_t M, int64_t N,
                           int K, cudaStream_t st, int num_sms, int* status);

// k_q4.cu
cudaError_t launch_q4_gemv(const int8_t* xq, const float* s, const int32_t* z, const uint8_t* q4,
                           const float* gs, int G, float* y, int64_t M, int64_t N, int K,
                           cudaStream_t st);

// k_q4_tma.cu
bool q4_tma_fits(int64_t M, int64_t K, int G);
bool q4_tma_quantizes(int64_t M);
// qp: x bf16 [M, K] is quantized in the kernel and xq / s / z receive the codes and
// qparams; otherwise xq / s / z are the qparams kernel's output and x is unused.
cudaError_t launch_q4_tma(const uint16_t* x, int8_t* xq, float* s, int32_t* z, bool qp,
                          const uint8_t* q4, const float* gs, int G, float* y, int64_t M,
                          int64_t N, int K, cudaStream_t st, int num_sms, int* status);

// k_q4_i8.cu
cudaError_t launch_q4_group_sums16(const uint8_t* q4, int64_t N, int K, int G, float* sums16,
                                   cudaStream_t st, int num_sms);
cudaError_t launch_q4_gemm_i8(const int8_t* xq, const int32_t* z, const float* s,
                              const uint8_t* q4, const float* gs, const float* sums16, float* y,
                              int G, int64_t M, int64_t N, int K, cudaStream_t st, int num_sms,
                              int* status);
// k_q4_tc.cu
cudaError_t launch_q4_expand_bf16(const uint8_t* q4, int64_t N, int K, uint16_t* wb,
                                  cudaStream_t st, int num_sms);
// M <= 64: the GEMM expands the packed int4 weight itself (q4 [N, K/2], no bf16 copy)
bool q4_tc_fused(int64_t M);
// Workspace of the fused GEMM's K-split (the parts' partial sums; 0 without a split).
size_t q4_fused_workspace_bytes(int64_t M, int64_t N, int K, int G, int num_sms);
cudaError_t launch_q4_gemm_fused(const uint8_t* q4, const uint16_t* xz, const float* gs,
                                 const float* s, float* y, int G, int64_t M, int64_t N, int K,
                                 void* ws, cudaStream_t st, int num_sms, int* status);
cudaError_t launch_q4_gemm_tc(const uint16_t* wb, const uint16_t* xz, const float* gs,
                              const float* s, float* y, int G, int64_t M, int64_t N, int K,
                              cudaStream_t st, int num_sms, int* status);

// k_checkpoint.cu
cudaError_t launch_checkpoint_save(const void* x, int x_bf16, int64_t M, int K, int G,
                                   int8_t* codes, uint8_t* exps, cudaStream_t st);
cudaError_t launch_checkpoint_load(const int8_t* codes, const uint8_t* exps, int64_t M, int K,
                                   int G, void* y, int y_bf16, cudaStream_t st);

// k_lora.cu
// The three products of the adapter linear and of the checkpoint's weight gradient,
//   out[t, p] = sum_c P(p, c) T(t, c) + ...:
//   LORA_FWD    p = n, t = m, c = k:  q[p, c] x[t, c], times s_w[p], + bias[p] + adapter term
//   LORA_DGRAD  p = k, t = m, c = n:  s_w[c] q[c, p] dy[t, c], + adapter term
//   LORA_WGRAD  p = k, t = n, c = m:  codes[c, p] 2^e dy[c, t]
enum { LORA_FWD = 0, LORA_DGRAD = 1, LORA_WGRAD = 2 };
struct LoraGemm {
    const int8_t* q;            // int8 operand
    const uint16_t* pre;        // its bf16 expansion (launch_lora_expand), or nullptr
    const uint16_t* t;          // bf16 operand
    const float* s_w;
    const float* bias;          // nullable
    const uint8_t* exps;        // LORA_WGRAD: exponent bytes of groups of 1 << gshift
    int gshift;
    void* out;
    int out_bf16, accumulate;
    float* partial;             // long sums in fp32: lora_partial_bytes, or nullptr
    int P, C;
    int64_t T;
    // adapter term (LORA_WGRAD: none): low = b (LORA_FWD) or a (LORA_DGRAD)
    const int32_t* ids;
    const uint16_t* low;
    const uint16_t* hp;         // [T, parts * R]: scale * h (LORA_DGRAD: g) in lora_parts parts
    const int* lists;           // lora_plan_lists
    int R;
};
// bf16 parts that a row of scale * h or g enters its large product as.  Two leave off at most
// 2^-17, next to nothing where the result is rounded to bf16 (2^-8 of it); three hold the whole
// fp32 number, as results in fp32 need (two made their error that of 16 bits).
constexpr int lora_parts(bool out_bf16) { return out_bf16 ? 2 : 3; }
size_t lora_plan_bytes(int64_t M);               // workspace of the plan
const int* lora_plan_lists(const void* ws);
cudaError_t launch_lora_plan(const int32_t* ids, int64_t M, int L, void* ws, cudaStream_t st);
// h (or, backward, g) of every row, and its bf16 parts hp [M, parts * R]; ws: the plan of its ids
cudaError_t launch_lora_shrink(bool bwd, const uint16_t* x, const uint16_t* w, const float* scale,
                               const void* ws, float* h, uint16_t* hp, int parts, int64_t M, int C,
                               int R, int L, cudaStream_t st, int num_sms);
// dB from dy and h, dA from the layer's input (bf16, or codes with exps) and g, each if wanted
cudaError_t launch_lora_wgrad(const void* dy, const float* h, float* db, const void* x,
                              const uint8_t* exps, int gshift, const float* g, float* da,
                              const float* scale, const void* ws, int accumulate, int64_t M, int N,
                              int K, int R, int L, cudaStream_t st, int num_sms);

// k_lora_tc.cu
// adapter list of a token tile: [0] their number, then their ids in ascending order
constexpr int LT_LIST = 260;
int lora_tc_tile(int64_t T);                    // tokens per tile
// bytes of the expansion, and of the partial sums; 0: none
size_t lora_pre_bytes(int mode, int64_t P, int64_t C, int64_t T);
size_t lora_partial_bytes(int mode, int64_t P, int64_t C, int64_t T);
// beside: right behind launch_lora_shrink on the stream, and at the same time
cudaError_t launch_lora_expand(int mode, const LoraGemm& a, uint16_t* out, bool beside,
                               cudaStream_t st);
size_t lora_list_bytes(int64_t T);
cudaError_t launch_lora_tc(int mode, const LoraGemm& a, cudaStream_t st, int num_sms,
                           int* status);

// k_gptq.cu
struct GptqPlan {
    size_t buf0, buf1, buf2, w, err, dead, bytes;     // byte offsets in the workspace
};
GptqPlan plan_gptq(int64_t N, int64_t K);
bool gptq_block_ok(int64_t block);
cudaError_t launch_hessian_accumulate(const float* x, int64_t R, int K, double* H, int reset,
                                      cudaStream_t st);
cudaError_t launch_gptq_int8(const float* W, const double* H, int64_t N, int K, double damp,
                             int block, int8_t* q, float* s_w, int32_t* wsum, void* ws,
                             cudaStream_t st, int num_sms, int* status);

// k_gemv.cu
cudaError_t launch_w8a16_gemv(const uint16_t* x, const int8_t* q, const float* s_w,
                              const float* bias, void* y, int y_bf16, int64_t M, int64_t N, int K,
                              cudaStream_t st, int num_sms);
cudaError_t launch_w8a8_gemv(const float* x, float s1, int z1, int has2, float s2, int z2,
                             const int8_t* q, const int32_t* wsum, const float* s_w,
                             const float* bias, float* y, int64_t M, int64_t N, int K,
                             cudaStream_t st);

}  // namespace q8
