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
// bf16 MMA: with at most 64 columns of rank per block there is no tile for tcgen05, and up to
// rank 32 the operand loads, not the MMAs, take the time (at rank 64 dA and dB are bound by
// that MMA's rate, 2048 multiply-adds in 8 cycles a quarter of an SM).
//
// Measured at M = 4096, rank 16, 4 adapters: plan 10 us beside the expansion; h from 33 MB of x
// 10 us; g from 90 MB of dy 25 us (3.6 TB/s); dA and dB from 107 MB 54 us, where the largest
// adapter, with 1.8 times its share of the rows, is the last to end.  Most was gained by letting eight neighbouring threads
// copy a row's whole line (g 40 -> 26 us), reading a k step's fragments before the MMAs of the
// one before, and vector loads of the low rows (84 -> 54 us).
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
//
// The sort counts: each warp takes a run of rows, counts its keys in a table of its own, and a
// key's rows of all warps follow one another in warp order.  Up to LP_CHUNK rows the keys stay
// in registers and are counted once; more go chunk by chunk.  Everything on the way to h waits for
// this kernel, so it has few barriers: with three for every 1024 rows it took 13 us instead of 10
// for 4096 rows (beside the expansion) and 4.3 instead of 3.8 for 77.
constexpr int LP_THREADS = 512, LP_WARPS = LP_THREADS / 32, LP_ITERS = 8;
constexpr int LP_CHUNK = LP_THREADS * LP_ITERS;
__global__ __launch_bounds__(LP_THREADS) void k_lora_plan(const int32_t* __restrict__ ids, int M,
                                                          int L, int BN, int* __restrict__ lists,
                                                          int list_len, int* __restrict__ perm,
                                                          int* __restrict__ off,
                                                          int* __restrict__ tiles) {
    __shared__ int cnt[LP_KEYS + 1], pos[LP_KEYS + 1], tpos[LP_KEYS + 1];
    __shared__ int wsum[2][LP_WARPS];
    __shared__ __align__(16) uint16_t part[LP_WARPS][LP_KEYS + 3];      // rows of a key in each warp
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // launched after all of the stream's earlier work (no early start): the kernels behind it
    // that start early rely on it
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x > 0) {
        uint32_t* seen = reinterpret_cast<uint32_t*>(cnt);
        if (tid < 32) seen[tid] = 0;
        __syncthreads();
        const int64_t t = (int64_t)(blockIdx.x - 1) * BN + tid;
        if (tid < BN && t < M) {
            const int id = ld_after(ids + t);
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
    // A chunk's keys: warp w has rows (w * iters + j) * 32 + lane, j < iters (-1: no row).
    int keys[LP_ITERS], iters = 0;
    auto load_keys = [&](int c0) {
        iters = (min(M - c0, LP_CHUNK) + LP_THREADS - 1) / LP_THREADS;
#pragma unroll
        for (int j = 0; j < LP_ITERS; ++j) {
            const int64_t m = (int64_t)c0 + (warp * iters + j) * 32 + lane;
            keys[j] = j < iters && m < M ? ld_after(ids + m) : 0;
        }
#pragma unroll
        for (int j = 0; j < LP_ITERS; ++j) {
            const int64_t m = (int64_t)c0 + (warp * iters + j) * 32 + lane;
            keys[j] = j >= iters || m >= M ? -1 : keys[j] >= 0 && keys[j] < L ? keys[j] : L;
        }
    };
    // the chunk's table: counts, then (a thread a key) a warp's first place among the key's rows;
    // the key's rows go to cnt
    auto count = [&]() {
#pragma unroll
        for (int j = 0; j < LP_ITERS; ++j) {
            if (j >= iters) break;
            const uint32_t same = __match_any_sync(0xffffffffu, keys[j]);
            if (keys[j] >= 0 && lane == __ffs(same) - 1)
                part[warp][keys[j]] += (uint16_t)__popc(same);
            __syncwarp();
        }
        __syncthreads();
        for (int k = tid; k <= L; k += LP_THREADS) {
            int c[LP_WARPS], run = 0;
#pragma unroll
            for (int w = 0; w < LP_WARPS; ++w) c[w] = part[w][k];
#pragma unroll
            for (int w = 0; w < LP_WARPS; ++w) {
                part[w][k] = (uint16_t)run;
                run += c[w];
            }
            cnt[k] = run;
        }
    };
    auto clear = [&]() {                            // this warp's row of the table
        for (int k = lane; k <= L; k += 32) part[warp][k] = 0;
        __syncwarp();
    };
    const bool single = M <= LP_CHUNK;
    load_keys(0);
    if (single) {
        clear();
        count();
    } else {
        for (int k = tid; k <= L; k += LP_THREADS) cnt[k] = 0;
        __syncthreads();
        for (int64_t c0 = 0; c0 < M; c0 += LP_CHUNK) {
            if (c0) load_keys((int)c0);
#pragma unroll
            for (int j = 0; j < LP_ITERS; ++j) {
                const uint32_t same = __match_any_sync(0xffffffffu, keys[j]);
                if (keys[j] >= 0 && lane == __ffs(same) - 1) atomicAdd(&cnt[keys[j]], __popc(same));
            }
        }
    }
    __syncthreads();
    // exclusive sums over the keys of rows and of blocks of rows, two keys a thread; key 1024
    // follows the rest
    const int k0 = 2 * tid;
    const int n0 = k0 <= L ? cnt[k0] : 0, n1 = k0 + 1 <= L ? cnt[k0 + 1] : 0;
    const int b0 = (n0 + LP_ROWS - 1) / LP_ROWS, b1 = (n1 + LP_ROWS - 1) / LP_ROWS;
    int sn = n0 + n1, sb = b0 + b1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sn, o), u = __shfl_up_sync(0xffffffffu, sb, o);
        if (lane >= o) { sn += v; sb += u; }
    }
    if (lane == 31) { wsum[0][warp] = sn; wsum[1][warp] = sb; }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < LP_WARPS; ++w)
        if (w < warp) { sn += wsum[0][w]; sb += wsum[1][w]; }
    pos[k0] = sn - n0 - n1;
    pos[k0 + 1] = sn - n1;
    tpos[k0] = sb - b0 - b1;
    tpos[k0 + 1] = sb - b1;
    if (tid == LP_THREADS - 1) {                    // reached only when L = 1024
        pos[1024] = sn;
        tpos[1024] = sb;
    }
    __syncthreads();
    const int last = tpos[L] + (cnt[L] + LP_ROWS - 1) / LP_ROWS;       // blocks in all
    for (int i = tid; i <= L; i += LP_THREADS) off[i] = pos[i];
    if (tid == 0) {
        off[L + 1] = M;
        off[LP_KEYS + 1] = last;
    }
    for (int j = tid; j < last; j += LP_THREADS) {
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
    for (int64_t c0 = 0; c0 < M; c0 += LP_CHUNK) {
        if (!single) {
            load_keys((int)c0);
            __syncthreads();                        // the last chunk's (or the tiles') cnt is read
            if (c0)
                for (int k = tid; k <= L; k += LP_THREADS) pos[k] += cnt[k];
            clear();
            count();
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < LP_ITERS; ++j) {
            if (j >= iters) break;
            const int key = keys[j];
            const uint32_t same = __match_any_sync(0xffffffffu, key);
            if (key >= 0)
                perm[pos[key] + part[warp][key] + __popc(same & ((1u << lane) - 1u))] =
                    (int)c0 + (warp * iters + j) * 32 + lane;
            __syncwarp();
            if (key >= 0 && lane == __ffs(same) - 1) part[warp][key] += (uint16_t)__popc(same);
            __syncwarp();
        }
    }
}

cudaError_t launch_lora_plan(const int32_t* ids, int64_t M, int L, void* ws, cudaStream_t st) {
    const LoraPlan p = plan_of(M);
    uint8_t* w = (uint8_t*)ws;
    const int BN = lora_tc_tile(M);
    const unsigned grid = 1 + (unsigned)((M + BN - 1) / BN);
    k_lora_plan<<<grid, LP_THREADS, 0, st>>>(ids, (int)M, L, BN, (int*)(w + p.lists), LT_LIST,
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
// Four floats at the same place of every CTA's shared memory, added in rank order.  All loads are
// on their way before the first addition: a load from another CTA takes most of a microsecond.
__device__ __forceinline__ float4 cluster_sum4(uint32_t addr, int S) {
    float4 q[8];
#pragma unroll
    for (int o = 0; o < 8; ++o)
        if (o < S)
            asm volatile(
                "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
                "ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [a];\n\t}"
                : "=f"(q[o].x), "=f"(q[o].y), "=f"(q[o].z), "=f"(q[o].w)
                : "r"(addr), "r"(o)
                : "memory");
    float4 v = q[0];
#pragma unroll
    for (int o = 1; o < 8; ++o)
        if (o < S) {
            v.x += q[o].x;
            v.y += q[o].y;
            v.z += q[o].z;
            v.w += q[o].w;
        }
    return v;
}

// ------------------------------------------------------------------------- h and g
// One block of rows of one adapter, up to 8 * NT columns of the rank, a part of the summed
// axis: the CTAs of a cluster split that axis and add their parts in rank order.
//   BWD == false: long operand x [M, C], adapter rows W[i] = A[i] [R, C] (c contiguous)
//   BWD == true : long operand dy [M, C], W[i] = B[i] [C, R] (r contiguous), times scale[i]
// Steps of 64 c through a ring of shared-memory stages (cp.async): 64 rows of x (128 bytes, 16-byte
// pieces at piece ^ (row & 7)) and the adapter's piece: 8 NT rows of 128 bytes placed likewise,
// or, backward, 64 rows of 16 NT bytes, their pieces rotated so that eight rows fill all banks.
constexpr int LSH = 4;                              // stages
__host__ __device__ constexpr int lsh_stage(int nt) { return 8192 + 1024 * nt; }
template <int NT>
__device__ __forceinline__ uint32_t lsh_piece(int row, int pc) {       // backward
    return (uint32_t)(row * 16 * NT + ((pc ^ ((row * NT >> 3) & (NT - 1))) << 4));
}

template <int NT, bool BWD>
__global__ __launch_bounds__(128) void k_lora_shrink(const uint16_t* __restrict__ x,
                                                     const uint16_t* __restrict__ W,
                                                     const float* __restrict__ scale,
                                                     const int* __restrict__ perm,
                                                     const int* __restrict__ off,
                                                     const int* __restrict__ tiles, int C, int R,
                                                     int S, float* __restrict__ h,
                                                     uint16_t* __restrict__ hp, int hparts) {
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
    // copies: eight neighbouring threads take a row's 128 bytes (a whole line a request: two
    // threads with four pieces each made half-used sectors of every request, and the kernel
    // half as fast); thread: piece tid & 7 of rows tid >> 3, + 16, + 32, + 48
    const int cr = tid >> 3, cpc = tid & 7;
    const uint16_t* xrow[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int row = cr + 16 * j;
        xrow[j] = x + (int64_t)ld_after(perm + start + (row < rows ? row : 0)) * C + cpc * 8;
    }
    const uint16_t* wmat = W + (int64_t)key * R * C;
    auto load = [&](int st, int slot) {
        const uint32_t xs = base + slot * lsh_stage(NT), wsm = xs + 8192;
        const int c0 = st * 64, c = c0 + cpc * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = cr + 16 * j;
            const bool live = row < rows && c < C;
            cp_async16(xs + row * 128 + ((cpc ^ (row & 7)) << 4), live ? xrow[j] + c0 : x, live);
        }
        if (!BWD) {
#pragma unroll
            for (int j = 0; j < (8 * NT + 15) / 16; ++j) {
                const int row = cr + 16 * j;
                if (row < 8 * NT) {
                    const bool lw = row < rn && c < C;
                    cp_async16(wsm + row * 128 + ((cpc ^ (row & 7)) << 4),
                               lw ? wmat + (int64_t)(r0 + row) * C + c : W, lw);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < (NT + 1) / 2; ++j) {
                const int u = tid + 128 * j, row = u / NT, pc = u % NT;
                if (row < 64) {
                    const int cc = c0 + row;
                    const bool lw = cc < C && pc * 8 < rn;
                    cp_async16(wsm + lsh_piece<NT>(row, pc),
                               lw ? wmat + (int64_t)cc * R + r0 + pc * 8 : W, lw);
                }
            }
        }
    };
    // The warp-level MMA cuts the running sum off where it adds, towards zero, which over
    // hundreds of MMAs adds up: the sum of a step (four MMAs) is added to the others here,
    // rounded to nearest.
    float acc[NT][4], sum[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = sum[i][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < LSH - 1; ++i) {
        if (s0 + i < s1) load(s0 + i, i);
        cp_commit();
    }
    int slot = 0;
    for (int st = s0; st < s1; ++st) {
        cp_wait<LSH - 2>();
        __syncthreads();
        if (st + LSH - 1 < s1) load(st + LSH - 1, (slot + LSH - 1) % LSH);
        cp_commit();
        const uint32_t xs = base + slot * lsh_stage(NT), wsm = xs + 8192;
        // fragments of a k step are read before the MMAs of the step before it: the few warps of
        // a block wait on nothing else
        uint32_t fa[2][4], fb[2][(NT + 1) / 2][4];
        auto frags = [&](int k) {
            const int ar = warp * 16 + (lane & 15);
            ldsm4(xs + ar * 128 + (((2 * k + (lane >> 4)) ^ (ar & 7)) << 4), fa[k & 1]);
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                if (!BWD) {
                    // rows r of two n-tiles, k halves
                    const int br = (n + (NT > 1 ? lane >> 4 : 0)) * 8 + (lane & 7);
                    ldsm4(wsm + br * 128 + (((2 * k + ((lane >> 3) & 1)) ^ (br & 7)) << 4),
                          fb[k & 1][n >> 1]);
                } else {
                    const int br = k * 16 + (lane & 15);
                    const int pc = n + (NT > 1 ? lane >> 4 : 0);
                    ldsm4_t(wsm + lsh_piece<NT>(br, pc), fb[k & 1][n >> 1]);
                }
            }
        };
        frags(0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k < 3) frags(k + 1);
            const uint32_t* a = fa[k & 1];
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                const uint32_t* b = fb[k & 1][n >> 1];
                mma_bf16_16816(acc[n], a[0], a[1], a[2], a[3], b[0], b[1]);
                if (NT > 1) mma_bf16_16816(acc[n + (NT > 1)], a[0], a[1], a[2], a[3], b[2], b[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[i][j] += acc[i][j];
                acc[i][j] = 0.0f;
            }
        slot = (slot + 1) % LSH;
    }
    // h (or g) in fp32, and times the scale in bf16 parts, [M, parts * R]: each is what the ones
    // before it leave over, rounded to nearest
    const float f = ld_after(scale + key);
    auto put = [&](int row, int r, float v) {
        const int64_t m = ld_after(perm + start + row);
        const float sv = v * f;
        h[m * R + r0 + r] = BWD ? sv : v;
        const int parts = BWD ? lora_parts(true) : hparts;
        uint16_t* to = hp + m * parts * R + r0 + r;
        const uint32_t hi = bf16_bits_rn(sv);
        const float rest = sv - __uint_as_float(hi << 16);
        const uint32_t mid = bf16_bits_rn(rest);
        to[0] = (uint16_t)hi;
        to[R] = (uint16_t)mid;
        if (parts > 2) to[2 * R] = (uint16_t)bf16_bits_rn(rest - __uint_as_float(mid << 16));
    };
    const int g = lane >> 2, t = lane & 3;
    if (S == 1) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = warp * 16 + g + 8 * (i >> 1), r = n * 8 + 2 * t + (i & 1);
                if (row < rows && r < rn) put(row, r, sum[n][i]);
            }
        return;
    }
    // parts in shared memory [64][8 NT + 4], added over the cluster in rank order
    cp_wait<0>();
    __syncthreads();
    constexpr int LD = 8 * NT + 4;
    float* mine = reinterpret_cast<float*>(sm);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mine[(warp * 16 + g + 8 * (i >> 1)) * LD + n * 8 + 2 * t + (i & 1)] = sum[n][i];
    cluster_sync_all();
    const int per = (rows + S - 1) / S, lo = part * per, hi = min(rows, lo + per);
    const int quads = rn >> 2;
    for (int u = tid; u < (hi - lo) * quads; u += 128) {
        const int row = lo + u / quads, r = u % quads * 4;
        const float4 v = cluster_sum4(base + (row * LD + r) * 4, S);
        put(row, r, v.x);
        put(row, r + 1, v.y);
        put(row, r + 2, v.z);
        put(row, r + 3, v.w);
    }
    cluster_sync_all();                             // nobody leaves while its part is read
}

// ------------------------------------------------------------------------- dA and dB
// out[p, r] = sum over the rows m of adapter i of X[m, p] * low[m, r], for 128 p and up to
// 8 * NT columns of the rank; X is dy (dB) or the layer's input in bf16 or 8 bits (dA).  Steps
// of 32 rows through a ring of three shared-memory stages (cp.async of the gathered rows: X as it
// is kept, low in fp32); a step's low values become three bf16 tiles (8 bits of the number each,
// so that their sum is the fp32 value) and its codes a bf16 tile (exactly) in shared memory, then
// X^T and low are read with transposing ldmatrix.  Clusters split the rows as above.
// One launch makes both: CTAs of dA (KIND 0: from bf16, 1: from codes) after those of dB (2).
constexpr int LW_ROWS = 32, LW_STAGES = 3, LW_THREADS = 256;
constexpr int LW_X = LW_ROWS * 256, LW_LOW = LW_ROWS * 128;    // bf16 tiles: X, a part of low
__host__ __device__ constexpr int lw_stage(int nt) { return LW_X + LW_ROWS * 32 * nt; }
__host__ __device__ constexpr int lw_work(int nt) { return LW_STAGES * lw_stage(nt); }
template <int NT>
constexpr int lw_smem() {
    constexpr int loop = lw_work(NT) + 3 * LW_LOW + LW_X, tile = 128 * (8 * NT + 4) * 4;
    return loop > tile ? loop : tile;
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
    const float f = KIND == 2 && total > 0 ? ld_after(scale + key) : 1.0f;

    // thread: row tid >> 3 of a step, 16 of its p, an eighth of its low
    const int xr = tid >> 3, xq = tid & 7;
    const uint32_t work = base + lw_work(NT), xwork = work + 3 * LW_LOW;
    int row_next = -1;                              // this thread's row in the step loaded next
    // KIND 1: the exponent bytes of the steps on their way, oldest first (a load is not waited
    // for before the step after the one that issued it)
    uint32_t e_in[LW_STAGES - 1];
    auto look = [&](int st) {
        const int at = st * LW_ROWS + xr;
        row_next = st < s1 && at < total ? ld_after(perm + first + at) : -1;
    };
    auto load = [&](int st, int slot) {             // returns the exponent byte
        uint32_t e = 0;
        const uint32_t xs = base + slot * lw_stage(NT), ls = xs + LW_X;
        const bool live = row_next >= 0;
        const int64_t m = live ? row_next : 0;
        look(st + 1);
        if (KIND == 1) {
            const int8_t* src = reinterpret_cast<const int8_t*>(X) + m * P + p0 + xq * 16;
            const bool in = live && p0 + xq * 16 < P;
            cp_async16(xs + xr * 128 + ((xq ^ (xr & 7)) << 4), in ? (const void*)src : X, in);
            e = in ? ld_after(exps + m * (P >> gshift) + ((p0 + xq * 16) >> gshift)) : 0u;
        } else {
            // eight neighbouring threads: 128 bytes of a row at a time
            const uint16_t* src = reinterpret_cast<const uint16_t*>(X) + m * P + p0 + xq * 8;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool in = live && p0 + xq * 8 + 64 * j < P;
                cp_async16(xs + xr * 256 + (((xq + 8 * j) ^ (xr & 7)) << 4),
                           in ? (const void*)(src + 64 * j) : X, in);
            }
        }
#pragma unroll
        for (int j = 0; j < (NT + 3) / 4; ++j) {
            const int pc = xq + 8 * j;                          // 4 columns a piece
            if (pc < 2 * NT) {
                const bool in = live && pc * 4 < rn;
                cp_async16(ls + xr * 32 * NT + pc * 16, in ? low + m * R + r0 + pc * 4 : low, in);
            }
        }
        return e;
    };
    // sums of a step (six MMAs) are added up outside the tensor core, as in k_lora_shrink (db of
    // 4096 rows: off by 8.1e-6 in the norm before, 2.7e-7 so)
    float acc[NT][4], sum[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = sum[i][j] = 0.0f;
    look(s0);
#pragma unroll
    for (int i = 0; i < LW_STAGES - 1; ++i) {
        e_in[i] = s0 + i < s1 ? load(s0 + i, i) : 0u;
        cp_commit();
    }
    int slot = 0;
    for (int st = s0; st < s1; ++st) {
        cp_wait<LW_STAGES - 2>();
        __syncthreads();                            // the step is there, the work tiles are free
        const uint32_t e = e_in[0];
#pragma unroll
        for (int i = 0; i + 1 < LW_STAGES - 1; ++i) e_in[i] = e_in[i + 1];
        e_in[LW_STAGES - 2] =
            st + LW_STAGES - 1 < s1
                ? load(st + LW_STAGES - 1, (slot + LW_STAGES - 1) % LW_STAGES) : 0u;
        cp_commit();
        const uint32_t xs = base + slot * lw_stage(NT), ls = xs + LW_X;
        if (KIND == 1) {
            const uint32_t e2 = e << 7 | e << 23;               // 2^e twice, as bf16
            const uint4 c = lds128(xs + xr * 128 + ((xq ^ (xr & 7)) << 4));
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
            uint32_t o[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                s8x4_to_bf16x2_seq(w[q], o[2 * q], o[2 * q + 1]);
                o[2 * q] = bf16x2_mulrn(o[2 * q], e2);
                o[2 * q + 1] = bf16x2_mulrn(o[2 * q + 1], e2);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                                 xwork + xr * 256 + (((xq * 2 + q) ^ (xr & 7)) << 4)),
                             "r"(o[4 * q]), "r"(o[4 * q + 1]), "r"(o[4 * q + 2]),
                             "r"(o[4 * q + 3])
                             : "memory");
        }
        // NT columns a thread (for a rank tile of 8: two, in half of the threads), each cut into
        // three bf16 numbers: 8 bits at a time, which is the whole of an fp32 number
        constexpr int CW = NT == 1 ? 2 : NT;
        if (xq * CW < 8 * NT) {
            const int r = xq * CW;
            float v[CW];
            const uint32_t from = ls + xr * 32 * NT + r * 4;
#pragma unroll
            for (int j = 0; j < CW; j += 2)
                asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];"
                             : "=f"(v[j]), "=f"(v[j + 1])
                             : "r"(from + j * 4)
                             : "memory");
#pragma unroll
            for (int j = 0; j < CW; ++j) v[j] *= f;
            const uint32_t to = work + xr * 128 + (((r >> 3) ^ (xr & 7)) << 4) + (r & 7) * 2;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                uint32_t o[CW / 2];
#pragma unroll
                for (int j = 0; j < CW; j += 2) {
                    const uint32_t a = __float_as_uint(v[j]), b = __float_as_uint(v[j + 1]);
                    o[j >> 1] = __byte_perm(a, b, 0x7632);
                    v[j] -= __uint_as_float(a & 0xFFFF0000u);
                    v[j + 1] -= __uint_as_float(b & 0xFFFF0000u);
                }
                if (CW == 8)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + i * LW_LOW),
                                 "r"(o[0]), "r"(o[CW > 2 ? 1 : 0]), "r"(o[CW > 4 ? 2 : 0]),
                                 "r"(o[CW > 6 ? 3 : 0])
                                 : "memory");
                else if (CW == 4)
                    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(to + i * LW_LOW),
                                 "r"(o[0]), "r"(o[CW > 2 ? 1 : 0])
                                 : "memory");
                else
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + i * LW_LOW), "r"(o[0])
                                 : "memory");
            }
        }
        __syncthreads();
        const uint32_t xt = KIND == 1 ? xwork : xs;
        // Stored rows m (k), 8 p a piece: matrices (m 0-7, p 0-7), (m 0-7, p 8-15), (m 8-15, p 0-7),
        // (m 8-15, p 8-15), each transposed; a warp has 16 p.  Fragments are read ahead of the
        // MMAs before them, as above.
        uint32_t fa[2][4], fb[2][(NT + 1) / 2][4];
        auto frag_a = [&](int k) {
            const int am = k * 16 + (lane & 7) + ((lane >> 4) << 3);
            const int apc = warp * 2 + ((lane >> 3) & 1);
            ldsm4_t(xt + am * 256 + ((apc ^ (am & 7)) << 4), fa[k]);
        };
        auto frags_b = [&](int i) {                             // k step i / 3, part i % 3
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                const int m = i / 3 * 16 + (lane & 15), pc = n + (NT > 1 ? lane >> 4 : 0);
                ldsm4_t(work + i % 3 * LW_LOW + m * 128 + ((pc ^ (m & 7)) << 4),
                        fb[i & 1][n >> 1]);
            }
        };
        frag_a(0);
        frags_b(0);
        frag_a(1);
#pragma unroll
        for (int i = 0; i < 3 * LW_ROWS / 16; ++i) {
            if (i + 1 < 3 * LW_ROWS / 16) frags_b(i + 1);
            const uint32_t* a = fa[i / 3];
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                const uint32_t* b = fb[i & 1][n >> 1];
                mma_bf16_16816(acc[n], a[0], a[1], a[2], a[3], b[0], b[1]);
                if (NT > 1) mma_bf16_16816(acc[n + (NT > 1)], a[0], a[1], a[2], a[3], b[2], b[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[i][j] += acc[i][j];
                acc[i][j] = 0.0f;
            }
        slot = (slot + 1) % LW_STAGES;
    }
    cp_wait<0>();
    __syncthreads();
    // the tile in shared memory [128][8 NT + 4], added over the cluster in rank order
    constexpr int LD = 8 * NT + 4;
    float* mine = reinterpret_cast<float*>(sm);
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mine[(warp * 16 + g + 8 * (i >> 1)) * LD + n * 8 + 2 * t + (i & 1)] = sum[n][i];
    if (S > 1) cluster_sync_all(); else __syncthreads();
    const int pn = min(128, P - p0), per = (pn + S - 1) / S;
    const int lo = part * per, hi = min(pn, lo + per), wide = max(hi - lo, 0), quads = rn >> 2;
    for (int u = tid; u < wide * quads; u += LW_THREADS) {
        // neighbouring threads: neighbouring columns (dB) or p (dA)
        const int p = lo + (KIND == 2 ? u / quads : u % wide);
        const int r = (KIND == 2 ? u % quads : u / wide) * 4;
        float4 v;
        if (S > 1)
            v = cluster_sum4(base + (p * LD + r) * 4, S);
        else
            v = *reinterpret_cast<const float4*>(mine + p * LD + r);
        if (KIND == 2) {
            float4* to = reinterpret_cast<float4*>(out + ((int64_t)key * P + p0 + p) * R + r0 + r);
            if (accumulate) {
                const float4 w = *to;
                v = make_float4(w.x + v.x, w.y + v.y, w.z + v.z, w.w + v.w);
            }
            *to = v;
        } else {
            float* to = out + ((int64_t)key * R + r0 + r) * P + p0 + p;
            const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                to[(int64_t)j * P] = accumulate ? to[(int64_t)j * P] + w[j] : w[j];
        }
    }
    if (S > 1) cluster_sync_all();              // nobody leaves while its part is read
}

template <int NT, int KIND>
__global__ __launch_bounds__(LW_THREADS) void k_lora_wgrad(const LoraGrad db, const LoraGrad da,
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
static cudaError_t launch_clustered(void (*k)(KArgs...), dim3 grid, int threads, int S,
                                    size_t smem, bool early,
                                    cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = early;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k, args...);
}
template <int NT>
constexpr int lsh_smem() { return LSH * lsh_stage(NT); }
static_assert(lsh_smem<1>() >= 64 * 12 * 4 && lsh_smem<8>() >= 64 * 68 * 4, "room for the parts");
// columns of the rank per CTA, in n-tiles of 8
static int rank_tiles(int R) { return R <= 8 ? 1 : R <= 16 ? 2 : R <= 32 ? 4 : 8; }

cudaError_t launch_lora_shrink(bool bwd, const uint16_t* x, const uint16_t* w, const float* scale,
                               const void* ws, float* h, uint16_t* hp, int parts, int64_t M, int C,
                               int R, int L, cudaStream_t st, int num_sms) {
    const LoraPlan p = plan_of(M);
    const uint8_t* wsb = (const uint8_t*)ws;
    const int* perm = (const int*)(wsb + p.perm);
    const int* off = (const int*)(wsb + p.off);
    const int* tl = (const int*)(wsb + p.tiles);
    const int NT = rank_tiles(R), z = (R + 8 * NT - 1) / (8 * NT);
    const int64_t tiles = (M + LP_ROWS - 1) / LP_ROWS + (M < L + 1 ? M : L + 1);
    // parts of the summed axis: as many CTAs as run at once, at least 256 of c each
    const int64_t at_once = (int64_t)(227 * 1024 / (LSH * lsh_stage(NT) + 1024)) * num_sms;
    int S = 1;
    while (S < 8 && tiles * z * 2 * S <= at_once && C / (2 * S) >= 256) S *= 2;
    const dim3 grid((unsigned)(tiles * S), z);
#define LORA_SHRINK(NT_, B_)                                                                  \
    do {                                                                                      \
        cudaError_t e = ensure_dyn_smem<k_lora_shrink<NT_, B_>>(lsh_smem<NT_>());                   \
        if (e != cudaSuccess) return e;                                                       \
        return launch_clustered(k_lora_shrink<NT_, B_>, grid, 128, S, lsh_smem<NT_>(), true, st,   \
                                x, w, scale,                                                  \
                                perm, off, tl, C, R, S, h, hp, parts);                        \
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

// CTAs of the gradients' kernel that an SM takes, asked for once per device
template <int NT, int KIND>
static int lora_wgrad_occupancy() {
    static std::atomic<int> known[128];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) {
        cudaGetLastError();
        return 1;
    }
    n = known[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (ensure_dyn_smem<k_lora_wgrad<NT, KIND>>(lw_smem<NT>()) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_lora_wgrad<NT, KIND>, LW_THREADS,
                                                      lw_smem<NT>()) != cudaSuccess) {
        cudaGetLastError();
        return 1;
    }
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}
static int lora_wgrad_per_sm(int NT, bool codes) {
    if (NT == 1) return codes ? lora_wgrad_occupancy<1, 1>() : lora_wgrad_occupancy<1, 0>();
    if (NT == 2) return codes ? lora_wgrad_occupancy<2, 1>() : lora_wgrad_occupancy<2, 0>();
    if (NT == 4) return codes ? lora_wgrad_occupancy<4, 1>() : lora_wgrad_occupancy<4, 0>();
    return codes ? lora_wgrad_occupancy<8, 1>() : lora_wgrad_occupancy<8, 0>();
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
    // parts of an adapter's rows: as many CTAs as run at once, at least 64 rows each if the
    // adapters share the batch evenly (1000 rows of one adapter, 2048 x 8192, rank 64, in 3 parts,
    // 2 CTAs an SM: 26 us; in 4, which do not all run at once: 33)
    const int64_t ctas = (int64_t)(gb.blocks + ga.blocks) * z * L;
    const int64_t at_once = (int64_t)lora_wgrad_per_sm(NT, exps != nullptr) * num_sms;
    int S = 1;
    while (S < 8 && ctas * (S + 1) <= at_once && M / L / (S + 1) >= 64) ++S;
    gb.blocks *= S;
    ga.blocks *= S;
    const dim3 grid(gb.blocks + ga.blocks, z, L);
    // Not launched early: the CTAs would gather on the first SMs that the GEMM leaves and wait
    // there (measured: 216 us after the GEMM's end instead of 84).
#define LORA_WG(NT_, K_)                                                                      \
    do {                                                                                      \
        cudaError_t e = ensure_dyn_smem<k_lora_wgrad<NT_, K_>>(lw_smem<NT_>());               \
        if (e != cudaSuccess) return e;                                                       \
        return launch_clustered(k_lora_wgrad<NT_, K_>, grid, LW_THREADS, S, lw_smem<NT_>(),   \
                                false, st,                                                    \
                                gb, ga, exps, gshift, scale, perm, off, accumulate, R, S);            \
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
