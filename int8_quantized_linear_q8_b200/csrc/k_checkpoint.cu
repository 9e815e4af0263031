// k_checkpoint.cu -- 8-bit activation checkpoints.
//
// A group of G consecutive values of a row is kept as G int8 codes and one exponent byte b:
//     e = the smallest whole number with absmax <= 127 * 2^e, clamped to [-126, 121]
//     code = clamp(round(x * 2^-e), -127, 127)      (ties to even; b = e + 127)
// The step is a power of two so that code * 2^e is a bf16 number: restoring rounds nothing,
// and the weight gradient can feed restored values to the bf16 tensor cores exactly.  The
// price is a step of up to twice absmax / 127.
//
// With absmax = 1.f * 2^p (fraction bits f), 127 * 2^e >= absmax first holds at e = p - 6
// when 1.f <= 127 / 64, else at p - 5; in exponent bytes b = byte(absmax) - 6 (+ 1 when the
// fraction is above 0x7E0000).  -126 keeps 2^e a normal number, 121 keeps 127 * 2^e finite.
//
// A NaN or an infinity must not come back as a number, or the gradients made from it would hide
// it.  Its group gets b = 255, whose 2^e is infinite in bf16 and fp32 alike: codes of +-127 restore
// infinities, code 0 a NaN (0 * inf), which the group's other values become as well.
//
// Bound by HBM: 3 bytes a bf16 value (and 1 / G) each way.  One thread per 16 values; 4096 x 11008,
// G = 128: save 26.9 us (5.1 TB/s), load 22.8 us (6.0 TB/s; a copy reaches 6.55).  More pieces a
// thread were slower (two: 28.0 and 24.6 us, four: 32.4 and 26.5), streaming stores the same.
#include "q8_kernels.cuh"

namespace q8 {

constexpr uint32_t CKPT_INF = 0x7F800000u, CKPT_NONE = 255u;
__device__ __forceinline__ uint32_t ckpt_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax) & 0x7FFFFFFFu;
    if (u >= CKPT_INF) return CKPT_NONE;
    const int b = (int)(u >> 23) - 6 + ((u & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
    return (uint32_t)min(max(b, 1), 248);
}

// The larger one, or NaN if either is (fmaxf would drop it).
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// One thread per 16 values; the G / 16 threads of a group are neighbours in a warp.
template <bool BF16>
__global__ __launch_bounds__(256) void k_checkpoint_save(const void* __restrict__ x, int64_t n16,
                                                         int G, int8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ exps) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int per = G >> 4;
    const bool live = i < n16;
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = 0.0f;
    if (live) {
        if (BF16) {
            const uint4* p = reinterpret_cast<const uint4*>(x) + 2 * i;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 w = ld_after16_stream(p + h);
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[8 * h + 2 * j] = bf16lo(ws[j]);
                    v[8 * h + 2 * j + 1] = bf16hi(ws[j]);
                }
            }
        } else {
            const uint4* p = reinterpret_cast<const uint4*>(x) + 4 * i;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const uint4 w = ld_after16_stream(p + h);
                v[4 * h] = __uint_as_float(w.x);
                v[4 * h + 1] = __uint_as_float(w.y);
                v[4 * h + 2] = __uint_as_float(w.z);
                v[4 * h + 3] = __uint_as_float(w.w);
            }
        }
    }
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = max_or_nan(amax, fabsf(v[j]));
    for (int o = per >> 1; o > 0; o >>= 1)
        amax = max_or_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!live) return;
    const uint32_t b = ckpt_exponent(amax);
    const float inv = __uint_as_float((254u - b) << 23);       // 2^-e
    uint32_t o[4];
    if (b != CKPT_NONE) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                c[k] = __float2int_rn(fminf(fmaxf(rintf(v[4 * j + k] * inv), -127.0f), 127.0f));
            o[j] = pack4_s8(c[0], c[1], c[2], c[3]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t u = __float_as_uint(v[4 * j + k]);
                c[k] = u == CKPT_INF ? 127 : u == (CKPT_INF | 0x80000000u) ? -127 : 0;
            }
            o[j] = pack4_s8(c[0], c[1], c[2], c[3]);
        }
    }
    reinterpret_cast<uint4*>(codes)[i] = make_uint4(o[0], o[1], o[2], o[3]);
    if ((i & (per - 1)) == 0) exps[i / per] = (uint8_t)b;
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_checkpoint_load(const int8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ exps,
                                                         int64_t n16, int G, void* __restrict__ y) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n16) return;
    const int shift = G == 32 ? 1 : G == 64 ? 2 : G == 128 ? 3 : 4;    // pieces of a group, log2
    const uint4 w = ld_after16_stream(codes + 16 * i);
    const uint32_t e = ld_after(exps + (i >> shift));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    if (BF16) {
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {     // exact: small whole numbers times a power of two
            s8x4_to_bf16x2_seq(ws[j], o[2 * j], o[2 * j + 1]);
            o[2 * j] = bf16x2_mulrn(o[2 * j], e << 7 | e << 23);
            o[2 * j + 1] = bf16x2_mulrn(o[2 * j + 1], e << 7 | e << 23);
        }
        uint4* out = reinterpret_cast<uint4*>(y) + 2 * i;
        out[0] = make_uint4(o[0], o[1], o[2], o[3]);
        out[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
        float4* out = reinterpret_cast<float4*>(y) + 4 * i;
        const float s = __uint_as_float(e << 23);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = (float)(int8_t)(ws[h] >> (8 * j)) * s;
            out[h] = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
}

template <typename... KArgs, typename... Args>
static cudaError_t launch_checkpoint(void (*k)(KArgs...), int64_t n16, cudaStream_t st,
                                     Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((n16 + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

cudaError_t launch_checkpoint_save(const void* x, int x_bf16, int64_t M, int K, int G,
                                   int8_t* codes, uint8_t* exps, cudaStream_t st) {
    const int64_t n16 = M * (K / 16);
    return x_bf16 ? launch_checkpoint(k_checkpoint_save<true>, n16, st, x, n16, G, codes, exps)
                  : launch_checkpoint(k_checkpoint_save<false>, n16, st, x, n16, G, codes, exps);
}

cudaError_t launch_checkpoint_load(const int8_t* codes, const uint8_t* exps, int64_t M, int K,
                                   int G, void* y, int y_bf16, cudaStream_t st) {
    const int64_t n16 = M * (K / 16);
    return y_bf16 ? launch_checkpoint(k_checkpoint_load<true>, n16, st, codes, exps, n16, G, y)
                  : launch_checkpoint(k_checkpoint_load<false>, n16, st, codes, exps, n16, G, y);
}

}  // namespace q8
