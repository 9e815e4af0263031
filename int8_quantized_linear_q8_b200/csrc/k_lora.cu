// k_lora.cu -- the small products of the low-rank adapters beside the W8A16 linear:
//
//   h[m,r]     = sum_k x[m,k] A[i][r,k]                      i = ids[m]
//   g[m,r]     = c[i] sum_n dy[m,n] B[i][n,r]
//   dA[i][r,k] = sum_{m: ids[m] = i} g[m,r] x[m,k]
//   dB[i][n,r] = sum_{m: ids[m] = i} dy[m,n] (c[i] h[m,r])
//
// All are bound by reading the long operand (x, dy) once; the rank is small.  The rows are
// first sorted by adapter (stable, so that every sum has one order), after which each product
// works on blocks of rows of one adapter, gathered row by row through the permutation; rows
// without an adapter form a last group, whose h is zero.  The products run on the warp-level
// bf16 MMA: with at most 64 columns of rank per block there is no tile for tcgen05, and the
// operand loads, not the MMAs, take the time.  fp32 rows (h, g) enter as two bf16 parts, high
// and rest, off by at most 2^-17.
#include "q8_kernels.cuh"

namespace q8 {

// ------------------------------------------------------------------------- the plan
// Rows sorted by adapter, blocks of up to LP_ROWS rows of one adapter, and, by further CTAs,
// the list of adapters of each row tile of the large GEMM.
constexpr int LP_ROWS = 64;
constexpr int LP_KEYS = 1025;                       // up to 1024 adapters, and "none"

struct LoraPlan {
    size_t lists, perm, off, tiles, bytes;          // byte offsets in the workspace
    int64_t max_tiles;
};
static inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }
static LoraPlan plan_of(int64_t M) {
    LoraPlan p;
    p.max_tiles = (M + LP_ROWS - 1) / LP_ROWS + (M < LP_KEYS ? M : LP_KEYS) + 1;
    p.lists = 0;
    p.perm = up256(lora_list_bytes(M));
    p.off = p.perm + up256((size_t)M * 4);
    p.tiles = p.off + up256((LP_KEYS + 2) * 4);
    p.bytes = p.tiles + up256((size_t)p.max_tiles * 12);
    return p;
}
size_t lora_plan_bytes(int64_t M) { return plan_of(M).bytes; }
const int* lora_plan_lists(const void* ws) { return reinterpret_cast<const int*>(ws); }

// Block 0 sorts; block 1 + j lists tile j (BN rows).  off[key] is the first position of a
// key's rows (off[L + 1] = M); tiles holds {key, first position, rows}, their number at
// off[LP_KEYS + 1].
__global__ __launch_bounds__(1024) void k_lora_plan(const int32_t* __restrict__ ids, int M, int L,
                                                    int BN, int* __restrict__ lists, int list_len,
                                                    int* __restrict__ perm, int* __restrict__ off,
                                                    int* __restrict__ tiles) {
    __shared__ int cnt[LP_KEYS + 1], pos[LP_KEYS + 1], tpos[LP_KEYS + 1];
    __shared__ int wsum[2][32];
    __shared__ uint8_t part[32][LP_KEYS + 3];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x > 0) {
        uint32_t* seen = reinterpret_cast<uint32_t*>(cnt);
        if (tid < 32) seen[tid] = 0;
        __syncthreads();
        const int64_t t = (int64_t)(blockIdx.x - 1) * BN + tid;
        if (tid < BN && t < M) {
            const int id = __ldg(ids + t);
            if (id >= 0 && id < L) atomicOr(&seen[id >> 5], 1u << (id & 31));
        }
        __syncthreads();
        if (tid < 32) {
            int* out = lists + (int64_t)(blockIdx.x - 1) * list_len;
            uint32_t w = seen[tid];
            const int n = __popc(w);
            int before = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, before, o);
                if (tid >= o) before += v;
            }
            if (tid == 31) out[0] = before;
            before -= n;
            while (w) {
                const int b = __ffs(w) - 1;
                w &= w - 1;
                out[1 + before++] = tid * 32 + b;
            }
        }
        return;
    }
    for (int i = tid; i <= L; i += 1024) cnt[i] = 0;
    for (int i = tid; i < 32 * (LP_KEYS + 3); i += 1024) (&part[0][0])[i] = 0;
    __syncthreads();
    // keys of eight rounds of 1024 rows at a time; they stay in registers for the second pass
    // when there are no more
    const int rounds = (int)(((int64_t)M + 1023) / 1024);
    int keys[8];
    auto load_keys = [&](int c0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t m = (int64_t)(c0 + j) * 1024 + tid;
            keys[j] = m < M ? __ldg(ids + m) : -1;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t m = (int64_t)(c0 + j) * 1024 + tid;
            keys[j] = m >= M ? -1 : keys[j] >= 0 && keys[j] < L ? keys[j] : L;
        }
    };
    for (int c0 = 0; c0 < rounds; c0 += 8) {
        load_keys(c0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (c0 + j >= rounds) break;
            const uint32_t same = __match_any_sync(0xffffffffu, keys[j]);
            if (keys[j] >= 0 && lane == __ffs(same) - 1) atomicAdd(&cnt[keys[j]], __popc(same));
        }
    }
    __syncthreads();
    // exclusive sums over the keys of rows and of blocks of rows; key 1024 follows the rest
    int n = tid <= L ? cnt[tid] : 0, b = (n + LP_ROWS - 1) / LP_ROWS;
    int sn = n, sb = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sn, o), u = __shfl_up_sync(0xffffffffu, sb, o);
        if (lane >= o) { sn += v; sb += u; }
    }
    if (lane == 31) { wsum[0][warp] = sn; wsum[1][warp] = sb; }
    __syncthreads();
    if (warp == 0) {
        int v = wsum[0][lane], u = wsum[1][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, v, o), y = __shfl_up_sync(0xffffffffu, u, o);
            if (lane >= o) { v += x; u += y; }
        }
        wsum[0][lane] = v;
        wsum[1][lane] = u;
    }
    __syncthreads();
    sn += warp ? wsum[0][warp - 1] : 0;
    sb += warp ? wsum[1][warp - 1] : 0;
    pos[tid] = sn - n;
    tpos[tid] = sb - b;
    if (tid == 1023) {                              // reached only when L = 1024
        pos[1024] = sn;
        tpos[1024] = sb;
    }
    __syncthreads();
    const int last = tpos[L] + (cnt[L] + LP_ROWS - 1) / LP_ROWS;       // blocks in all
    for (int i = tid; i <= L; i += 1024) off[i] = pos[i];
    if (tid == 0) {
        off[L + 1] = M;
        off[LP_KEYS + 1] = last;
    }
    for (int j = tid; j < last; j += 1024) {
        int lo = 0, hi = L;                         // the last key whose first block is <= j
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (tpos[mid] <= j) lo = mid; else hi = mid - 1;
        }
        const int in = (j - tpos[lo]) * LP_ROWS;
        tiles[3 * j] = lo < L ? lo : -1;
        tiles[3 * j + 1] = pos[lo] + in;
        tiles[3 * j + 2] = min(LP_ROWS, cnt[lo] - in);
    }
    __syncthreads();
    for (int c0 = 0; c0 < rounds; c0 += 8) {
        if (rounds > 8) load_keys(c0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (c0 + j >= rounds) break;
            const int key = keys[j];
            const uint32_t same = __match_any_sync(0xffffffffu, key);
            const bool lead = key >= 0 && lane == __ffs(same) - 1;
            if (lead) part[warp][key] = (uint8_t)__popc(same);
            __syncthreads();
            if (key >= 0) {
                int at = pos[key] + __popc(same & ((1u << lane) - 1u));
                for (int w = 0; w < warp; ++w) at += part[w][key];
                perm[at] = (c0 + j) * 1024 + tid;
            }
            __syncthreads();
            if (lead) {
                atomicAdd(&pos[key], __popc(same));
                part[warp][key] = 0;
            }
            __syncthreads();
        }
    }
}

cudaError_t launch_lora_plan(const int32_t* ids, int64_t M, int L, void* ws, cudaStream_t st) {
    const LoraPlan p = plan_of(M);
    uint8_t* w = (uint8_t*)ws;
    const int BN = lora_tc_tile(LORA_FWD, M);
    const unsigned grid = 1 + (unsigned)((M + BN - 1) / BN);
    k_lora_plan<<<grid, 1024, 0, st>>>(ids, (int)M, L, BN, (int*)(w + p.lists), LT_LIST,
                                       (int*)(w + p.perm), (int*)(w + p.off),
                                       (int*)(w + p.tiles));
    return cudaGetLastError();
}

// --------------------------------------------------------------------- shared pieces
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a float of another CTA of the cluster (its shared memory, same offset)
__device__ __forceinline__ float ld_peer(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
        "ld.shared::cluster.f32 %0, [a];\n\t}"
        : "=f"(v)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// ------------------------------------------------------------------------- h and g
// One block of rows of one adapter, up to 8 * NT columns of the rank, a part of the summed
// axis: the CTAs of a cluster split that axis and add their parts in rank order.
//   BWD == false: long operand x [M, C], adapter rows W[i] = A[i] [R, C] (c contiguous)
//   BWD == true : long operand dy [M, C], W[i] = B[i] [C, R] (r contiguous), times scale[i]
// Steps of 64 c through a ring of four shared-memory stages (cp.async, 16-byte pieces placed
// at piece ^ (row & 7): conflict-free for the copies and for ldmatrix).
constexpr int LSH_STAGES = 4;
constexpr int LSH_BYTES = LSH_STAGES * 2 * 64 * 128;

template <int NT, bool BWD>
__global__ __launch_bounds__(128) void k_lora_shrink(const uint16_t* __restrict__ x,
                                                     const uint16_t* __restrict__ W,
                                                     const float* __restrict__ scale,
                                                     const int* __restrict__ perm,
                                                     const int* __restrict__ off,
                                                     const int* __restrict__ tiles, int C, int R,
                                                     int S, float* __restrict__ h,
                                                     uint16_t* __restrict__ hp) {
    extern __shared__ __align__(1024) uint8_t sm[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tile = blockIdx.x / S;
    if (tile >= ld_after(off + LP_KEYS + 1)) return;               // uniform over the cluster
    const int part = S > 1 ? (int)cluster_rank() : 0;
    const int key = ld_after(tiles + 3 * tile), start = ld_after(tiles + 3 * tile + 1);
    const int rows = ld_after(tiles + 3 * tile + 2);
    const int r0 = blockIdx.y * (8 * NT), rn = min(8 * NT, R - r0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (key < 0) {                                              // rows without an adapter
        if (part == 0)
            for (int u = tid; u < rows * rn; u += 128)
                h[(int64_t)ld_after(perm + start + u / rn) * R + r0 + u % rn] = 0.0f;
        return;
    }
    const int steps = (C + 63) / 64;
    const int s0 = steps * part / S, s1 = steps * (part + 1) / S;
    const uint32_t base = smem_u32(sm);
    // copies: thread -> row tid >> 1, four 16-byte pieces from 4 * (tid & 1)
    const int crow = tid >> 1, cp0 = (tid & 1) * 4;
    const uint16_t* xrow =
        x + (int64_t)ld_after(perm + start + (crow < rows ? crow : 0)) * C;
    const uint16_t* wmat = W + (int64_t)key * R * C;
    auto load = [&](int st, int slot) {
        const uint32_t xs = base + slot * 16384, wsm = xs + 8192;
        const int c0 = st * 64;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int pc = cp0 + j, c = c0 + pc * 8;
            const bool live = crow < rows && c < C;
            cp_async16(xs + crow * 128 + ((pc ^ (crow & 7)) << 4), live ? xrow + c : x, live);
            if (!BWD) {
                if (crow < 8 * NT) {
                    const bool lw = crow < rn && c < C;
                    cp_async16(wsm + crow * 128 + ((pc ^ (crow & 7)) << 4),
                               lw ? wmat + (int64_t)(r0 + crow) * C + c : W, lw);
                }
            } else if (pc < NT) {
                const int cc = c0 + crow;
                const bool lw = cc < C && pc * 8 < rn;
                cp_async16(wsm + crow * 128 + ((pc ^ (crow & 7)) << 4),
                           lw ? wmat + (int64_t)cc * R + r0 + pc * 8 : W, lw);
            }
        }
    };
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < LSH_STAGES - 1; ++i) {
        if (s0 + i < s1) load(s0 + i, i);
        cp_commit();
    }
    int slot = 0;
    for (int st = s0; st < s1; ++st) {
        cp_wait<LSH_STAGES - 2>();
        __syncthreads();
        if (st + LSH_STAGES - 1 < s1) load(st + LSH_STAGES - 1, (slot + LSH_STAGES - 1) % LSH_STAGES);
        cp_commit();
        const uint32_t xs = base + slot * 16384, wsm = xs + 8192;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t a[4];
            const int ar = warp * 16 + (lane & 15);
            ldsm4(xs + ar * 128 + (((2 * k + (lane >> 4)) ^ (ar & 7)) << 4), a);
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t b[4];
                if (!BWD) {
                    // rows r of two n-tiles, k halves
                    const int br = (n + (NT > 1 ? lane >> 4 : 0)) * 8 + (lane & 7);
                    ldsm4(wsm + br * 128 + (((2 * k + ((lane >> 3) & 1)) ^ (br & 7)) << 4), b);
                } else {
                    const int br = k * 16 + (lane & 15);
                    const int pc = n + (NT > 1 ? lane >> 4 : 0);
                    ldsm4_t(wsm + br * 128 + ((pc ^ (br & 7)) << 4), b);
                }
                mma_bf16_16816(acc[n], a[0], a[1], a[2], a[3], b[0], b[1]);
                if (NT > 1) mma_bf16_16816(acc[n + (NT > 1)], a[0], a[1], a[2], a[3], b[2], b[3]);
            }
        }
        slot = (slot + 1) % LSH_STAGES;
    }
    // h (or g) in fp32, and times the scale in two bf16 parts, [M, 2 R]: high, rest
    const float f = __ldg(scale + key);
    auto put = [&](int row, int r, float v) {
        const int64_t m = ld_after(perm + start + row);
        const float sv = v * f;
        h[m * R + r0 + r] = BWD ? sv : v;
        const uint32_t hi = bf16_bits_rn(sv);
        hp[m * 2 * R + r0 + r] = (uint16_t)hi;
        hp[m * 2 * R + R + r0 + r] = (uint16_t)bf16_bits_rn(sv - __uint_as_float(hi << 16));
    };
    const int g = lane >> 2, t = lane & 3;
    if (S == 1) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = warp * 16 + g + 8 * (i >> 1), r = n * 8 + 2 * t + (i & 1);
                if (row < rows && r < rn) put(row, r, acc[n][i]);
            }
        return;
    }
    // parts in shared memory [64][8 NT + 1], added over the cluster in rank order
    cp_wait<0>();
    __syncthreads();
    constexpr int LD = 8 * NT + 1;
    float* mine = reinterpret_cast<float*>(sm);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mine[(warp * 16 + g + 8 * (i >> 1)) * LD + n * 8 + 2 * t + (i & 1)] = acc[n][i];
    cluster_sync_all();
    const int per = (rows + S - 1) / S, lo = part * per, hi = min(rows, lo + per);
    for (int u = tid; u < (hi - lo) * rn; u += 128) {
        const int row = lo + u / rn, r = u % rn;
        float v = 0.0f;
        for (int q = 0; q < S; ++q) v += ld_peer(base + (row * LD + r) * 4, q);
        put(row, r, v);
    }
    cluster_sync_all();                             // nobody leaves while its part is read
}

// ------------------------------------------------------------------------- dA and dB
// out[p, r] = sum over the rows m of adapter i of X[m, p] * low[m, r], for 128 p and up to
// 8 * NT columns of the rank; X is dy (dB) or the layer's input in bf16 or 8 bits (dA).  Steps
// of 32 rows: the next step's X pieces and low values wait in registers while this step's
// MMAs run, then go to the other shared-memory buffer (8-bit codes are expanded on the way,
// exactly).  X^T is read with transposing ldmatrix.  Clusters split the rows as above.
// One launch makes both: CTAs of dA (KIND 0: from bf16, 1: from codes) after those of dB (2).
constexpr int LW_ROWS = 32;
constexpr int LW_X = LW_ROWS * 256, LW_LOW = LW_ROWS * 128;    // one part (hi or rest)
constexpr int LW_STAGE = LW_X + 2 * LW_LOW;
template <int NT>
constexpr int lw_smem() {
    return 2 * LW_STAGE > 128 * (8 * NT + 1) * 4 ? 2 * LW_STAGE : 128 * (8 * NT + 1) * 4;
}
struct LoraGrad {
    const void* X;              // [M, P]
    const float* low;           // [M, R]
    float* out;
    int P;
    int blocks;                 // CTAs along x: P tiles times parts; 0: not wanted
};

template <int NT, int KIND>
__device__ __forceinline__ void lora_grad_tile(const LoraGrad& q, int bx,
                                               const uint8_t* __restrict__ exps, int gshift,
                                               const float* __restrict__ scale,
                                               const int* __restrict__ perm,
                                               const int* __restrict__ off, int accumulate, int R,
                                               int S) {
    const void* X = q.X;
    const float* low = q.low;
    float* out = q.out;
    const int P = q.P;
    extern __shared__ __align__(1024) uint8_t sm[];
    const int part = S > 1 ? (int)cluster_rank() : 0;
    const int p0 = bx / S * 128, r0 = blockIdx.y * (8 * NT), rn = min(8 * NT, R - r0);
    const int key = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = ld_after(off + key), total = ld_after(off + key + 1) - first;
    const int steps = (total + LW_ROWS - 1) / LW_ROWS;
    const int s0 = (int)((int64_t)steps * part / S), s1 = (int)((int64_t)steps * (part + 1) / S);
    const uint32_t base = smem_u32(sm);
    const float f = KIND == 2 && total > 0 ? __ldg(scale + key) : 1.0f;

    // X: thread -> row tid >> 2, 32 p from 32 * (tid & 3); low: row tid >> 2, 2 * NT columns
    const int xr = tid >> 2, xp = (tid & 3) * 32;
    uint4 xv[4];
    uint32_t xe = 0;
    float lv[2 * NT];
    int row_next = 0;                               // the row after the one fetched next
    auto look = [&](int st) {
        const int at = st * LW_ROWS + xr;
        row_next = at < total ? ld_after(perm + first + at) : -1;
    };
    auto fetch = [&](int st) {
        const bool live = row_next >= 0;
        const int64_t m = live ? row_next : 0;
        if (st + 1 < s1) look(st + 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) xv[j] = make_uint4(0, 0, 0, 0);
        if (KIND == 1) {
            const int8_t* src = reinterpret_cast<const int8_t*>(X) + m * P + p0 + xp;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (live && p0 + xp + 16 * j < P) xv[j] = ldg_stream(src + 16 * j);
            xe = live && p0 + xp < P
                     ? __ldg(exps + m * (P >> gshift) + ((p0 + xp) >> gshift)) : 0u;
        } else {
            const uint16_t* src = reinterpret_cast<const uint16_t*>(X) + m * P + p0 + xp;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (live && p0 + xp + 8 * j < P) xv[j] = ldg_stream(src + 8 * j);
        }
        // 2 NT columns, in pieces of at most 4 (rn is a multiple of 8)
#pragma unroll
        for (int j = 0; j < 2 * NT; ++j) lv[j] = 0.0f;
        const int r = (tid & 3) * 2 * NT;
        const float* lp = low + m * R + r0 + r;
        if (NT == 1) {
            if (live)
                asm volatile("ld.global.v2.f32 {%0,%1}, [%2];"
                             : "=f"(lv[0]), "=f"(lv[1])
                             : "l"(lp)
                             : "memory");
        } else {
#pragma unroll
            for (int j = 0; j + 3 < 2 * NT; j += 4)
                if (live && r + j < rn) {
                    const float4 v = ld_after4(lp + j);
                    lv[j] = v.x;
                    lv[j + 1] = v.y;
                    lv[j + 2] = v.z;
                    lv[j + 3] = v.w;
                }
        }
    };
    auto place = [&](int buf) {
        const uint32_t xs = base + buf * LW_STAGE;
        // row of 256 bytes, 16-byte pieces at piece ^ (row & 7)
        if (KIND == 1) {
            const uint32_t e2 = xe << 7 | xe << 23;             // 2^e twice, as bf16
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t w[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
                uint32_t o[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    s8x4_to_bf16x2_seq(w[q], o[2 * q], o[2 * q + 1]);
                    o[2 * q] = bf16x2_mulrn(o[2 * q], e2);
                    o[2 * q + 1] = bf16x2_mulrn(o[2 * q + 1], e2);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int pc = (tid & 3) * 4 + 2 * j + q;
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                                     xs + xr * 256 + ((pc ^ (xr & 7)) << 4)),
                                 "r"(o[4 * q]), "r"(o[4 * q + 1]), "r"(o[4 * q + 2]),
                                 "r"(o[4 * q + 3])
                                 : "memory");
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int pc = (tid & 3) * 4 + j;
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                                 xs + xr * 256 + ((pc ^ (xr & 7)) << 4)),
                             "r"(xv[j].x), "r"(xv[j].y), "r"(xv[j].z), "r"(xv[j].w)
                             : "memory");
            }
        }
#pragma unroll
        for (int j = 0; j < 2 * NT; j += 2) {
            const int r = (tid & 3) * 2 * NT + j;
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float v = lv[j + q] * f;
                const uint32_t b = bf16_bits_rn(v);
                hi |= b << (16 * q);
                lo |= bf16_bits_rn(v - __uint_as_float(b << 16)) << (16 * q);
            }
            const uint32_t at = xs + LW_X + xr * 128 + (((r >> 3) ^ (xr & 7)) << 4) + (r & 7) * 2;
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(hi) : "memory");
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + LW_LOW), "r"(lo) : "memory");
        }
    };
    float acc[2][NT][4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[a][i][j] = 0.0f;
    if (s0 < s1) {
        look(s0);
        fetch(s0);
        place(0);
    }
    __syncthreads();
    for (int st = s0; st < s1; ++st) {
        const int buf = (st - s0) & 1;
        if (st + 1 < s1) fetch(st + 1);
        const uint32_t xs = base + buf * LW_STAGE;
#pragma unroll
        for (int k = 0; k < LW_ROWS / 16; ++k) {
            uint32_t a[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                // stored rows m (k), 8 p a piece: matrices (m 0-7, p 0-7), (m 0-7, p 8-15),
                // (m 8-15, p 0-7), (m 8-15, p 8-15), each transposed
                const int m = k * 16 + (lane & 7) + ((lane >> 4) << 3);
                const int pc = warp * 4 + q * 2 + ((lane >> 3) & 1);
                ldsm4_t(xs + m * 256 + ((pc ^ (m & 7)) << 4), a[q]);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t b[4];
                    const int m = k * 16 + (lane & 15), pc = n + (NT > 1 ? lane >> 4 : 0);
                    ldsm4_t(xs + LW_X + half * LW_LOW + m * 128 + ((pc ^ (m & 7)) << 4), b);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        mma_bf16_16816(acc[q][n], a[q][0], a[q][1], a[q][2], a[q][3], b[0], b[1]);
                        if (NT > 1)
                            mma_bf16_16816(acc[q][n + (NT > 1)], a[q][0], a[q][1], a[q][2],
                                           a[q][3], b[2], b[3]);
                    }
                }
        }
        if (st + 1 < s1) place(buf ^ 1);
        __syncthreads();
    }
    // the tile in shared memory [128][8 NT + 1], added over the cluster in rank order
    constexpr int LD = 8 * NT + 1;
    float* mine = reinterpret_cast<float*>(sm);
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mine[(warp * 32 + q * 16 + g + 8 * (i >> 1)) * LD + n * 8 + 2 * t + (i & 1)] =
                    acc[q][n][i];
    if (S > 1) cluster_sync_all(); else __syncthreads();
    const int pn = min(128, P - p0), per = (pn + S - 1) / S;
    const int lo = part * per, hi = min(pn, lo + per), wide = max(hi - lo, 0);
    for (int u = tid; u < wide * rn; u += 128) {
        const int p = lo + (KIND == 2 ? u / rn : u % wide), r = KIND == 2 ? u % rn : u / wide;
        float v = 0.0f;
        if (S > 1)
            for (int o = 0; o < S; ++o) v += ld_peer(base + (p * LD + r) * 4, o);
        else
            v = mine[p * LD + r];
        float* to = out + (KIND == 2 ? ((int64_t)key * P + p0 + p) * R + r0 + r
                                    : ((int64_t)key * R + r0 + r) * P + p0 + p);
        *to = accumulate ? *to + v : v;
    }
    if (S > 1) cluster_sync_all();              // nobody leaves while its part is read
}

template <int NT, int KIND>
__global__ __launch_bounds__(128) void k_lora_wgrad(const LoraGrad db, const LoraGrad da,
                                                    const uint8_t* __restrict__ exps, int gshift,
                                                    const float* __restrict__ scale,
                                                    const int* __restrict__ perm,
                                                    const int* __restrict__ off, int accumulate,
                                                    int R, int S) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int bx = blockIdx.x;                      // a cluster lies in one of the two ranges
    if (bx < db.blocks)
        lora_grad_tile<NT, 2>(db, bx, exps, gshift, scale, perm, off, accumulate, R, S);
    else
        lora_grad_tile<NT, KIND>(da, bx - db.blocks, exps, gshift, scale, perm, off, accumulate,
                                 R, S);
}

// ----------------------------------------------------------------------- host side
template <typename... KArgs, typename... Args>
static cudaError_t launch_clustered(void (*k)(KArgs...), dim3 grid, int S, size_t smem,
                                    cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k, args...);
}
// columns of the rank per CTA, in n-tiles of 8
static int rank_tiles(int R) { return R <= 8 ? 1 : R <= 16 ? 2 : R <= 32 ? 4 : 8; }

cudaError_t launch_lora_shrink(bool bwd, const uint16_t* x, const uint16_t* w, const float* scale,
                               const void* ws, float* h, uint16_t* hp, int64_t M, int C, int R,
                               int L, cudaStream_t st, int num_sms) {
    const LoraPlan p = plan_of(M);
    const uint8_t* wsb = (const uint8_t*)ws;
    const int* perm = (const int*)(wsb + p.perm);
    const int* off = (const int*)(wsb + p.off);
    const int* tl = (const int*)(wsb + p.tiles);
    const int NT = rank_tiles(R), z = (R + 8 * NT - 1) / (8 * NT);
    const int64_t tiles = (M + LP_ROWS - 1) / LP_ROWS + (M < L + 1 ? M : L + 1);
    // parts of the summed axis: as many CTAs as run at once (three per SM), at least 256 of c each
    int S = 1;
    while (S < 8 && tiles * z * 2 * S <= 3 * num_sms && C / (2 * S) >= 256) S *= 2;
    const dim3 grid((unsigned)(tiles * S), z);
#define LORA_SHRINK(NT_, B_)                                                                  \
    do {                                                                                      \
        cudaError_t e = ensure_dyn_smem<k_lora_shrink<NT_, B_>>(LSH_BYTES);                   \
        if (e != cudaSuccess) return e;                                                       \
        return launch_clustered(k_lora_shrink<NT_, B_>, grid, S, LSH_BYTES, st, x, w, scale,  \
                                perm, off, tl, C, R, S, h, hp);                                   \
    } while (0)
#define LORA_SHRINK_NT(NT_)              \
    do {                                 \
        if (bwd) LORA_SHRINK(NT_, true); \
        LORA_SHRINK(NT_, false);         \
    } while (0)
    if (NT == 1) LORA_SHRINK_NT(1);
    if (NT == 2) LORA_SHRINK_NT(2);
    if (NT == 4) LORA_SHRINK_NT(4);
    LORA_SHRINK_NT(8);
#undef LORA_SHRINK
#undef LORA_SHRINK_NT
}

cudaError_t launch_lora_wgrad(const void* dy, const float* h, float* db, const void* x,
                              const uint8_t* exps, int gshift, const float* g, float* da,
                              const float* scale, const void* ws, int accumulate, int64_t M, int N,
                              int K, int R, int L, cudaStream_t st, int num_sms) {
    const LoraPlan p = plan_of(M);
    const uint8_t* wsb = (const uint8_t*)ws;
    const int* perm = (const int*)(wsb + p.perm);
    const int* off = (const int*)(wsb + p.off);
    const int NT = rank_tiles(R), z = (R + 8 * NT - 1) / (8 * NT);
    LoraGrad gb = {dy, h, db, N, db ? (N + 127) / 128 : 0};
    LoraGrad ga = {x, g, da, K, da ? (K + 127) / 128 : 0};
    // parts of an adapter's rows: until four CTAs per SM, at least 64 rows each if the
    // adapters share the batch evenly
    int S = 1;
    while (S < 8 && (int64_t)(gb.blocks + ga.blocks) * z * L * 2 * S <= 4 * num_sms &&
           M / L / (2 * S) >= 64)
        S *= 2;
    gb.blocks *= S;
    ga.blocks *= S;
    const dim3 grid(gb.blocks + ga.blocks, z, L);
#define LORA_WG(NT_, K_)                                                                      \
    do {                                                                                      \
        cudaError_t e = ensure_dyn_smem<k_lora_wgrad<NT_, K_>>(lw_smem<NT_>());               \
        if (e != cudaSuccess) return e;                                                       \
        return launch_clustered(k_lora_wgrad<NT_, K_>, grid, S, lw_smem<NT_>(), st, gb, ga,   \
                                exps, gshift, scale, perm, off, accumulate, R, S);            \
    } while (0)
#define LORA_WG_NT(NT_)                    \
    do {                                   \
        if (exps) LORA_WG(NT_, 1);         \
        LORA_WG(NT_, 0);                   \
    } while (0)
    if (NT == 1) LORA_WG_NT(1);
    if (NT == 2) LORA_WG_NT(2);
    if (NT == 4) LORA_WG_NT(4);
    LORA_WG_NT(8);
#undef LORA_WG
#undef LORA_WG_NT
}

}  // namespace q8
