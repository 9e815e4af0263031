// k_lora_tc.cu -- the three large products of the adapter linear and of the 8-bit checkpoint
// on the tcgen05 tensor cores, one bf16 operand and one int8 operand:
//
//   out[t, p] = sum_c P(p, c) T(t, c) + ...
//   LORA_FWD    p = n, t = m, c = k   P = q[p, c],            T = x[t, c]
//               y = s_w[p] * sum + bias[p] + sum_r b[i][p, r] (scale[i] h[t, r]),  i = ids[t]
//   LORA_DGRAD  p = k, t = m, c = n   P = s_w[c] q[c, p],     T = dy[t, c]
//               dx = sum + sum_r a[i][r, p] g[t, r]
//   LORA_WGRAD  p = k, t = n, c = m   P = codes[c, p] 2^e,    T = dy[c, t]
//
// The int8 operand stays int8 in HBM and L2 and becomes bf16 in shared memory: exactly for the
// forward pass (codes; s_w comes after the sum) and the weight gradient (codes times a power
// of two), with one rounding of s_w * q for dgrad, where s_w varies along the sum.
//
// A pair of CTAs (a cluster of two) computes a tile of 256 p x BN t with cta_group::2 MMAs:
// each CTA holds 128 rows of P, half of the T rows, and the accumulators of its own 128 rows
// (BN columns of tensor memory).  Against one CTA with 128 x 256 tiles this halves the shared
// memory traffic of the T operand, which leaves room for the conversion's.  BN is the T extent
// split evenly into tiles of at most 256, rounded up to 32 (what a pair's MMA takes).
//
// The adapter term is more of the same contraction: for the adapters that the tile's tokens
// use (a list made per tile beforehand), the rank's columns of b (or a) on the P side and of
// scale * h (or g) on the T side, zero for tokens of other adapters.  h comes as two bf16 parts
// (off by at most 2^-17) where the result is bf16, as three (all of the fp32 number) where it is
// fp32, so an adapter takes 2 or 3 * rank columns.  Forward it goes
// to the other accumulator buffer, since s_w applies to the base sum alone.
//
// Two variants.  PRE: the int8 operand was expanded to bf16 in the workspace beforehand
// (k_lora_expand) and both operands come by TMA.  Otherwise it stays int8 in HBM and L2 and the
// kernel converts it, which costs nothing extra to read but adds 24 KB of shared-memory traffic
// to the 64 KB that a stage and CTA move anyway, more than the port carries in the MMAs' time.
// With few rows the converters' own path is what a stage takes (77 rows: 0.57 us a stage when
// one loop did base and adapter stages, 0.4 with a loop of its own for the base).
//
// What bounds it, measured on the expanded form (cycles a stage of 64 c; its MMAs take 512): dgrad
// 538, tensor pipe active 93% of the time a pair has work; forward 608 (the adapter term's
// second accumulator, drained between tiles).  dgrad of 4096 x 11008 x 4096: 250 us, 1.48 PFLOP/s,
// of which the fourth round of tiles, which 34 of 74 pairs have, costs 13%.  Two things cost most
// on the way: cluster-scope acquire and release on the hand-offs (538 -> 328 us), and everything
// on the issuing warp's path between two stages.  Not kept: a second launch that splits the last
// round's tiles over clusters of two pairs (only 32 such clusters run at once; the exchange costs
// what it saves), L2 evict-last hints on the operands (no change), t blocks of 16 and 64 tiles
// (1% and 8% slower), both sums of 16 columns read under one wait (more spills).
//
// Few tiles (fewer than half the CTA pairs): S = 2 or 4 pairs of one cluster split a tile's
// stages; each owns 1 / S of the tile's columns and adds the other pairs' parts, which they
// store in its shared memory (free by then), in pair order.
//
// Roles: 0 and 2 TMA producers of the int8 and the bf16 operands; 1 tensor-memory
// allocator and, in the pair's first CTA, MMA issuer; then converters, two groups of four that
// take every other stage (PRE: one group, for the adapter columns; weight gradient: none), and
// four epilogue warps (PRE: eight).  A stage is 64 of c.  Its int8 box (8 KB) has a ring of its own,
// eight deep: that path is the longest (copy, conversion, MMA) and runs ahead.  Its P tile and its
// T tile (16 KB each) share a slot of a ring of five (PRE: seven), so that the issuing warp, whose
// own steps bound the main loop, has one barrier to wait for and one commit to make per stage; it
// tests the next stage's barrier before it issues this stage's MMAs, which hides the test.  Every
// wait is bounded, and what a warp does when one runs out goes by a vote: its lanes may differ.
#include "q8_kernels.cuh"

namespace q8 {

constexpr int LT_BK = 64;
constexpr int LT_A = 128 * 128, LT_B = 128 * 128, LT_RAW = 128 * 64;
constexpr int LT_N_MAX = 7, LT_NR = 8;                  // ring depths
__host__ __device__ constexpr int lt_slots(bool pre) { return pre ? 7 : 5; }
constexpr int LT_SLOT = LT_A + LT_B, LT_RT = 5 * LT_SLOT;
constexpr int LT_CTRL = LT_RT + LT_NR * LT_RAW;
static_assert(LT_CTRL >= LT_N_MAX * LT_SLOT, "PRE uses the whole region for its slots");
// warps: 15, which leaves each thread 128 registers (19 would leave 96); 11 for the expanded
// weight gradient, which has nothing to convert and keeps its sums in registers (184)
__host__ __device__ constexpr int lt_conv(int mode, bool pre) {
    return !pre ? 8 : mode == LORA_WGRAD ? 0 : 4;
}
__host__ __device__ constexpr int lt_epi(bool pre) { return pre ? 8 : 4; }
constexpr int LT_CONV0 = 3;
__host__ __device__ constexpr int lt_threads(int mode, bool pre) {
    return 32 * (LT_CONV0 + lt_conv(mode, pre) + lt_epi(pre));
}
// The tensor core cuts a running sum off towards zero at every step, which over thousands of
// terms adds up (weight gradient of 4096 rows: 2.2e-6 off in the norm; plain fp32 3.0e-7).  Results
// that are not rounded to bf16, which is 1000 times as coarse, are sums of LT_SUM stages added up
// outside it (4.1e-7, for 2% of the time): the weight gradient and a forward pass with fp32
// output.  The expanded weight gradient adds them up in registers, the others in memory.
constexpr int LT_SUM = 16;
constexpr int LT_SMEM = LT_CTRL + 1024 + 512;
static_assert(LT_SMEM <= 227 * 1024, "shared memory");

// position in a ring: slot and the parity of its current phase
template <int N>
struct LtRing {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) { s = 0; ph ^= 1u; }
    }
    __device__ __forceinline__ void next2() {
        if ((s += 2) >= N) { s -= N; ph ^= 1u; }
    }
    __device__ __forceinline__ void skip(int n) {
        n += s;
        s = n % N;
        ph ^= (uint32_t)(n / N) & 1u;
    }
};

// ------------------------------------------------------------------ cluster and tcgen05
__device__ __forceinline__ uint32_t lt_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t lt_map(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void lt_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// arrive on a barrier of either CTA of the pair (a shared::cluster address).  What it announces
// is read by the tensor core (after fence.proxy.async) or was read from tensor memory (after
// tcgen05.wait), so no cluster-scope fence is asked for.
__device__ __forceinline__ void lt_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}
// TMA load into this CTA's shared memory, completion on a barrier of the pair's first CTA
__device__ __forceinline__ void lt_tma_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
// 128-byte-swizzled operand tiles.  K-major: rows of 64 c, groups of 8 rows 1024 bytes apart.
// MN-major: blocks of 64 rows (8192 bytes: 64 c of 128 bytes), groups of 8 c 1024 bytes apart.
__device__ __forceinline__ uint64_t lt_desc(uint32_t saddr, bool mn_major) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(mn_major ? 8192 >> 4 : 1) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16: bf16 operands, fp32 accumulator, M = 256 over the pair
__device__ __forceinline__ uint32_t lt_idesc(int bn, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(bn >> 3) << 17) | (16u << 24);
}
// one lane of a converged warp
__device__ __forceinline__ bool lt_elect() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}
// the next two are called by the elected lane
__device__ __forceinline__ void lt_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// arrives on the barrier at the same offset in the pair's CTAs once the MMAs issued so far are done
__device__ __forceinline__ void lt_commit(uint64_t* bar, uint16_t ctas) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(ctas)
        : "memory");
}
__device__ __forceinline__ void lt_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void lt_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void lt_ld_wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// ------------------------------------------------------------------------- conversion
// What a converter thread multiplies its codes by: nothing (forward), s_w as the bf16 pair
// hi + lo (hi * q + lo * q is rounded once, to bf16), or a power of two.  Loaded a turn ahead as
// raw bits, so that nothing waits on the load before its turn.
template <int MODE>
__device__ __forceinline__ uint32_t lt_scale_bits(const LoraGemm& a, int c, int p) {
    if (MODE == LORA_DGRAD && c < a.C) return __float_as_uint(ld_after(a.s_w + c));
    if (MODE == LORA_WGRAD && c < a.C && p < a.P)
        return ld_after(a.exps + (int64_t)c * (a.P >> a.gshift) + (p >> a.gshift));
    return 0u;
}
struct LtScale {
    uint32_t hi, lo;
};
template <int MODE>
__device__ __forceinline__ LtScale lt_scale(uint32_t bits) {
    LtScale s = {0u, 0u};
    if (MODE == LORA_DGRAD) {
        const float v = __uint_as_float(bits);
        const uint32_t h = bf16_bits_rn(v);
        const uint32_t l = bf16_bits_rn(v - __uint_as_float(h << 16));
        s.hi = h | h << 16;
        s.lo = l | l << 16;
    }
    if (MODE == LORA_WGRAD) s.hi = bits << 7 | bits << 23;
    return s;
}
template <int MODE>
__device__ __forceinline__ uint32_t lt_apply(uint32_t v, const LtScale& s) {
    if (MODE == LORA_DGRAD) return bf16x2_fma(v, s.hi, bf16x2_mulrn(v, s.lo));
    if (MODE == LORA_WGRAD) return bf16x2_mulrn(v, s.hi);
    return v;
}

// ------------------------------------------------------------------------- the kernel
// Writes W columns (t0 + j, those below t1) of this lane's p: v + bias, to out; fp32:
// first added to `from` (at the same places), then, `add`, to what is there.  All lanes of the warp
// call it.  Whole chunks go without a test or a product per store: with them a weight
// gradient's tile took 5.7 us to write, without 2.9 (40 x 11008 x 4096: 62 -> 32.5 us a call).
template <int MODE, int W, bool FULL>
__device__ __forceinline__ void lt_store_rows(const LoraGemm& a, int t0, int rows, int p,
                                              float (&v)[W], void* to, const float* from,
                                              bool add) {
    const int lane = threadIdx.x & 31;
    const int64_t step = a.P;
    if (MODE != LORA_WGRAD && a.out_bf16 && (a.P & 1) == 0) {
        // neighbouring lanes exchange, so that each stores two p of one t
        const int od = lane & 1;
        uint32_t* out = reinterpret_cast<uint32_t*>(to) + (((t0 + od) * step + (p & ~1)) >> 1);
#pragma unroll
        for (int j = 0; j < W; j += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, od ? v[j] : v[j + 1], 1);
            const uint32_t lo = bf16_bits_rn(od ? got : v[j]);
            const uint32_t hi = bf16_bits_rn(od ? v[j + 1] : got);
            if ((FULL || j + od < rows) && p < a.P) *out = lo | hi << 16;
            out += step;
        }
    } else if (MODE != LORA_WGRAD && a.out_bf16) {
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(to) + t0 * step + p;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if ((FULL || j < rows) && p < a.P) *out = __float2bfloat16_rn(v[j]);
            out += step;
        }
    } else if (p < a.P) {
        float* out = reinterpret_cast<float*>(to) + t0 * step + p;
        if (MODE != LORA_DGRAD && from) {
            const float* in = from + t0 * step + p;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (FULL || j < rows) v[j] += *in;
                in += step;
            }
        }
        if (MODE == LORA_WGRAD && add) {
            const float* in = out;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (FULL || j < rows) v[j] += *in;
                in += step;
            }
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (FULL || j < rows) {
                // a weight gradient is larger than L2 can hold beside the operands: streamed past
                // them (wgrad 4096 x 11008 x 4096: 292 -> 275 us)
                if (MODE == LORA_WGRAD)
                    st_stream_f32(out, v[j]);
                else
                    *out = v[j];
            }
            out += step;
        }
    }
}
template <int MODE, int W>
__device__ __forceinline__ void lt_store(const LoraGemm& a, int t0, int64_t t1, int p, float bs,
                                         float (&v)[W], void* to, const float* from,
                                         bool add) {
    if (MODE == LORA_FWD)
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] += bs;
    if (t0 + W <= t1)
        lt_store_rows<MODE, W, true>(a, t0, W, p, v, to, from, add);
    else
        lt_store_rows<MODE, W, false>(a, t0, (int)(t1 - t0), p, v, to, from, add);
}

// PARTS: bf16 parts of scale * h or g, lora_parts of the result's type.  (A constant, which leaves
// the bf16 forms as fast as when there was no third part.  fp32, 77 rows, 2048 x 8192, 8 adapters:
// rank 64, which takes 24 adapter stages a tile instead of 16, 26.4 -> 28.7 us; rank 16 27.6 -> 28.3.)
template <int MODE, bool PRE, int PARTS>
__global__ __launch_bounds__(lt_threads(MODE, PRE), 1) void k_lora_tc(
    const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap tmap,
    const LoraGemm a, int BN, int num_p, int num_t, int S, int* status) {
    constexpr bool A_MN = MODE != LORA_FWD;             // int8 operand with p contiguous
    constexpr bool B_MN = MODE == LORA_WGRAD;           // bf16 operand with t contiguous
    constexpr int LT_N = lt_slots(PRE), LT_CONV = lt_conv(MODE, PRE), LT_EPI = lt_epi(PRE);
    constexpr int GROUPS = LT_CONV == 8 ? 2 : 1, LT_EPI0 = LT_CONV0 + LT_CONV;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t* rfull = reinterpret_cast<uint64_t*>(smem + LT_CTRL);
    uint64_t* rempty = rfull + LT_NR;
    uint64_t* full = rempty + LT_NR;        // first CTA: both CTAs' P and T tiles are there
    uint64_t* empty = full + LT_N;
    uint64_t* tfull = empty + LT_N;
    uint64_t* tempty = tfull + 2;                       // first CTA
    uint64_t* lready = tempty + 2;          // PRE, first CTA: adapter columns written
    uint64_t* lgo = lready + LT_N;          // PRE: slot free for adapter columns
    uint64_t* mma_done = lgo + LT_N;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // pair of the cluster, CTA of the pair, and the cluster rank of the pair's first CTA
    const uint32_t crank = lt_rank(), rank = crank & 1u, lead = crank & ~1u;
    const int pair = (int)(crank >> 1);
    const uint16_t both = (uint16_t)(3u << lead);
    const int units = num_p * num_t;
    const int u0 = blockIdx.x / (2 * S), ustep = gridDim.x / (2 * S);
    const int nk = (a.C + LT_BK - 1) / LT_BK;
    const int half = BN >> 1;
    // stages of a sum, and this pair's sums of a tile
    const bool sums = MODE == LORA_WGRAD || (MODE == LORA_FWD && !a.out_bf16);
    const int most = (nk + S - 1) / S, own_nk = nk * (pair + 1) / S - nk * pair / S;
    const int sum_n = sums ? (most + LT_SUM - 1) / LT_SUM : 1, sum_len = (most + sum_n - 1) / sum_n;
    const int nsum = sums ? (own_nk + sum_len - 1) / sum_len : 1;
    // where all sums but the last are added up (the pairs of a tile: each in a place of its own)
    float* const partial = a.partial ? a.partial + (int64_t)pair * a.T * a.P
                                     : reinterpret_cast<float*>(a.out);
    // Tiles run over t first, in even blocks of at most 8 t tiles: the pairs that run at once share
    // both operands through L2 and the int8 operand is read from HBM once per block.
    const int tblk = (num_t + (num_t + 7) / 8 - 1) / ((num_t + 7) / 8);
    auto tile_of = [&](int u, int& p0, int& t0) {
        const int full = num_p * tblk, blk = u / full, rem = u - blk * full;
        const int tb = min(tblk, num_t - blk * tblk);
        p0 = rem / tb * 256 + (int)rank * 128;
        t0 = (blk * tblk + rem % tb) * BN;
    };
    // A tile's stages: first this pair's share of the nk of the base sum, then its share of
    // those of the adapter columns, numbered from nk.  The latter need what the kernels before
    // this one made (lists, hp).  The base sum does not, unless it reads the expansion: q, x and
    // dy are older than the plan, whose launch waited for all of the stream's earlier work,
    // so the forward and dgrad products start while h or g is still being made.
    constexpr bool EARLY = !PRE && MODE != LORA_WGRAD;
    struct Walk {
        int kb, end;
        bool low;               // in the adapter columns (or there are none)
    };
    auto walk = [&]() {
        return Walk{nk * pair / S, nk * (pair + 1) / S, MODE == LORA_WGRAD};
    };
    auto more = [&](Walk& w, int t0) {
        if (w.kb < w.end) return true;
        if (w.low) return false;
        if (EARLY) asm volatile("griddepcontrol.wait;" ::: "memory");
        const int cnt = ld_after(a.lists + (int64_t)(t0 / BN) * LT_LIST);
        const int total = (cnt * PARTS * a.R + LT_BK - 1) / LT_BK;
        w.low = true;
        w.kb = nk + total * pair / S;
        w.end = nk + total * (pair + 1) / S;
        return w.kb < w.end;
    };

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&pmap);
        tma_prefetch_desc(&tmap);
        for (int i = 0; i < LT_NR; ++i) {
            mbar_init(&rfull[i], 1);
            mbar_init(&rempty[i], 4);
        }
        for (int i = 0; i < LT_N; ++i) {
            // the copies' producer and, unless PRE, a converter group of either CTA
            mbar_init(&full[i], PRE ? 1 : 1 + 8);
            mbar_init(&lready[i], 8);
            mbar_init(&lgo[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * LT_EPI);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    lt_cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!EARLY) asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 0) {
        // ---------------------------------------------------------------- int8 producer
        LtRing<LT_NR> r;
        int it = 0;
        bool ok = true;
        for (int u = u0; u < units && ok && !PRE; u += ustep) {
            int p0, t0;
            tile_of(u, p0, t0);
            for (int kb = walk().kb; kb < walk().end; ++kb) {
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&rempty[r.s], r.ph ^ 1u, status, abort_flag));
                if (!ok) break;
                if (lane == 0) {
                    const int c0 = kb * LT_BK;
                    uint8_t* dst = smem + LT_RT + r.s * LT_RAW;
                    mbar_expect_tx(&rfull[r.s], LT_RAW);
                    if (A_MN)
                        tma_load_2d(dst, &pmap, p0, c0, &rfull[r.s]);
                    else
                        tma_load_2d(dst, &pmap, c0, p0, &rfull[r.s]);
                }
                ++it;
                r.next();
            }
        }
        // copies issued here have landed before the CTA leaves
        for (int i = max(0, it - LT_NR); i < it; ++i)
            mbar_drain(&rfull[i % LT_NR], (uint32_t)(i / LT_NR) & 1u, status);
    } else if (warp == 2) {
        // ---------------------------------------------------------------- bf16 producer
        const uint32_t full0 = lt_map(smem_u32(full), lead);
        // bytes of both CTAs' T boxes: rows of 64 c, or boxes of 64 t
        const uint32_t tbytes = B_MN ? (uint32_t)((half + 63) / 64) * 2u * 8192u : (uint32_t)BN * 128u;
        LtRing<LT_N> r;
        int it = 0;
        bool ok = true;
        for (int u = u0; u < units && ok; u += ustep) {
            int p0, t0;
            tile_of(u, p0, t0);
            const int tr = t0 + (int)rank * half;
            for (Walk w = walk(); more(w, t0); ++w.kb) {
                const int kb = w.kb;
                ok = __all_sync(0xffffffffu,
                                mbar_wait(&empty[r.s], r.ph ^ 1u, status, abort_flag));
                if (!ok) break;
                if (lane == 0) {
                    if (kb < nk) {
                        const int c0 = kb * LT_BK;
                        const uint32_t at = smem_u32(smem + r.s * LT_SLOT), bt = at + LT_A;
                        if (rank == 0)
                            mbar_expect_tx(&full[r.s], tbytes + (PRE ? 2 * LT_A : 0));
                        if (PRE && A_MN) {
                            lt_tma_pair(at, &pmap, p0 * 2, c0, full0 + r.s * 8);
                            lt_tma_pair(at + 8192, &pmap, (p0 + 64) * 2, c0, full0 + r.s * 8);
                        } else if (PRE) {
                            lt_tma_pair(at, &pmap, c0 * 2, p0, full0 + r.s * 8);
                        }
                        if (B_MN)
                            for (int b = 0; b < (half + 63) / 64; ++b)
                                lt_tma_pair(bt + b * 8192, &tmap, (tr + b * 64) * 2, c0,
                                            full0 + r.s * 8);
                        else
                            lt_tma_pair(bt, &tmap, c0 * 2, tr, full0 + r.s * 8);
                    } else {                            // written by the converters
                        if (rank == 0) mbar_arrive(&full[r.s]);
                        if (PRE) mbar_arrive(&lgo[r.s]);
                    }
                }
                ++it;
                r.next();
            }
        }
        if (rank == 0)
            for (int i = max(0, it - LT_N); i < it; ++i)
                mbar_drain(&full[i % LT_N], (uint32_t)(i / LT_N) & 1u, status);
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (rank == 0) {
            const uint32_t idesc = lt_idesc(BN, A_MN, B_MN);
            LtRing<LT_N> r;
            LtRing<2> rt;
            uint32_t lph = 0;                           // PRE: parity of each slot's lready
            bool ok = true, here = false;
            for (int u = u0; u < units && ok; u += ustep) {
                int p0, t0;
                tile_of(u, p0, t0);
                bool first = true, in_low = MODE != LORA_FWD;
                int left = sum_len;
                for (Walk w = walk(); ok && more(w, t0); ++w.kb) {
                    // a sum begins: of the base, or, forward, the adapter term
                    const bool begin_low = w.kb >= nk && !in_low;
                    const bool fresh = first || begin_low || (nsum > 1 && w.kb < nk && left == 0);
                    if (fresh) {
                        if (!first) {                   // the sum before it is complete
                            if (lt_elect()) lt_commit(&tfull[rt.s], both);
                            __syncwarp();
                            rt.next();
                        }
                        if (begin_low) in_low = true;
                        left = sum_len;
                        first = false;
                        ok = __all_sync(0xffffffffu,
                                        mbar_wait(&tempty[rt.s], rt.ph ^ 1u, status, abort_flag));
                        if (!ok) break;
                    }
                    --left;
                    if (!here) {
                        ok = __all_sync(0xffffffffu,
                                        mbar_wait(&full[r.s], r.ph, status, abort_flag));
                        if (!ok) break;
                    }
                    if (PRE && w.kb >= nk) {
                        ok = __all_sync(0xffffffffu, mbar_wait(&lready[r.s], lph >> r.s & 1u,
                                                               status, abort_flag));
                        if (!ok) break;
                        lph ^= 1u << r.s;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const int cur = r.s;
                    r.next();
                    here = mbar_test_wait(&full[r.s], r.ph);
                    if (lt_elect()) {
                        const uint32_t at = smem_u32(smem + cur * LT_SLOT);
                        const uint64_t ad = lt_desc(at, A_MN), bd = lt_desc(at + LT_A, B_MN);
                        const uint32_t d = tmem + (uint32_t)(rt.s * 256);
#pragma unroll
                        for (int k = 0; k < LT_BK / 16; ++k)
                            lt_mma(d, ad + (A_MN ? 128 : 2) * k, bd + (B_MN ? 128 : 2) * k, idesc,
                                   !(fresh && k == 0));
                        lt_commit(&empty[cur], both);
                    }
                    here = __all_sync(0xffffffffu, here);
                }
                if (!ok) break;
                if (lt_elect()) lt_commit(&tfull[rt.s], both);
                __syncwarp();
                rt.next();
            }
            if (lt_elect()) lt_commit(mma_done, both);  // before tensor memory is released
            __syncwarp();
            mbar_drain(mma_done, 0, status);
        }
        __syncwarp();
    } else if (warp < LT_EPI0) {
        // ---------------------------------------------------------------- converters
        const int grp = (warp - LT_CONV0) >> 2;
        const int tid = threadIdx.x - 32 * LT_CONV0 - grp * 128;
        const uint32_t full0 = lt_map(smem_u32(full), lead);
        const uint32_t lready0 = lt_map(smem_u32(lready), lead);
        LtRing<LT_NR> rr;
        LtRing<LT_N> r;
        uint32_t lph = 0;                   // PRE: parity of each slot's lgo
        int it = 0, pending = -1;           // slot whose adapter columns are still being copied
        bool live = true;
        auto hand_over = [&](int slot) {
            // make the generic-proxy writes visible to the tensor core, then hand over
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) lt_arrive((PRE ? lready0 : full0) + slot * 8);
        };
        for (int u = u0; u < units; u += ustep) {
            int p0, t0;
            tile_of(u, p0, t0);
            Walk w = walk();
            if (PRE) {                                  // the base stages are not theirs
                for (; w.kb < w.end; ++w.kb) r.next();
            } else {
                // Base stages: this group's are every other one.  A loop of its own, without
                // the adapter columns' bookkeeping: with few rows, what a group does between two
                // stages is what a stage takes (77 rows, 2048 x 8192: 0.57 us a stage before).
                const int sc = tid >> 3, sp = p0 + (tid & 7) * 16;  // this thread's first c, its p
                const int n = w.end - w.kb, skip = (it ^ grp) & 1;  // GROUPS == 2 here
                int kb = w.kb + skip;
                LtRing<LT_N> rc = r;
                LtRing<LT_NR> rq = rr;
                if (skip) {
                    rc.next();
                    rq.next();
                }
                uint32_t nxt[4];                        // the next turn's scales
                if (A_MN)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        nxt[i] = lt_scale_bits<MODE>(a, kb * LT_BK + i * 16 + sc, sp);
#pragma unroll 1
                for (; kb < w.end; kb += 2) {
                    const uint32_t raw = smem_u32(smem + LT_RT + rq.s * LT_RAW);
                    live = __all_sync(0xffffffffu, mbar_wait(&rfull[rq.s], rq.ph, status, abort_flag) &&
                                                       live);
                    uint4 cw[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        cw[i] = A_MN ? lds128(raw + (i * 16 + sc) * 128 + (tid & 7) * 16)
                                    : lds128(raw + tid * 64 + ((i ^ ((tid >> 1) & 3)) << 4));
                    uint32_t cur[4];
                    if (A_MN) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) cur[i] = nxt[i];
                        if (kb + 2 < w.end)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                nxt[i] = lt_scale_bits<MODE>(a, (kb + 2) * LT_BK + i * 16 + sc, sp);
                    }
                    // converted in registers first: what lies between a free tile and
                    // its hand-over is on the ring's critical path
                    uint32_t o[4][8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s8x4_to_bf16x2_seq(cw[i].x, o[i][0], o[i][1]);
                        s8x4_to_bf16x2_seq(cw[i].y, o[i][2], o[i][3]);
                        s8x4_to_bf16x2_seq(cw[i].z, o[i][4], o[i][5]);
                        s8x4_to_bf16x2_seq(cw[i].w, o[i][6], o[i][7]);
                        if (A_MN) {
                            const LtScale f = lt_scale<MODE>(cur[i]);
#pragma unroll
                            for (int j = 0; j < 8; ++j) o[i][j] = lt_apply<MODE>(o[i][j], f);
                        }
                    }
                    // The box is free once its codes are in registers, all lanes' and for the
                    // copy engine as well: handed back right behind the loads, it was
                    // overwritten under them now and then (20000 rows, 264 x 16384).
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&rempty[rq.s]);
                    rq.next2();
                    const uint32_t at = smem_u32(smem + rc.s * LT_SLOT);
                    live = __all_sync(0xffffffffu, mbar_wait(&empty[rc.s], rc.ph ^ 1u, status,
                                                             abort_flag) && live);
                    if (live) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (!A_MN) {
                                // thread: row tid, 64 codes
                                const uint32_t row = at + tid * 128;
                                sts128(row + (((2 * i) ^ (tid & 7)) << 4), o[i][0], o[i][1],
                                       o[i][2], o[i][3]);
                                sts128(row + (((2 * i + 1) ^ (tid & 7)) << 4), o[i][4], o[i][5],
                                       o[i][6], o[i][7]);
                            } else {
                                // thread: 16 codes of p in each of 4 rows of c, two 16-byte
                                // pieces; lanes of the second 64-p block write theirs in the
                                // other order, which keeps a row's lanes on different banks
                                const int ch = tid & 7, odd = ch >> 2, c = i * 16 + sc;
                                const uint32_t row = at + odd * 8192 + c * 128;
                                const int j0 = (ch & 3) * 2;
                                sts128(row + (((j0 + odd) ^ (c & 7)) << 4),
                                       odd ? o[i][4] : o[i][0], odd ? o[i][5] : o[i][1],
                                       odd ? o[i][6] : o[i][2], odd ? o[i][7] : o[i][3]);
                                sts128(row + (((j0 + 1 - odd) ^ (c & 7)) << 4),
                                       odd ? o[i][0] : o[i][4], odd ? o[i][1] : o[i][5],
                                       odd ? o[i][2] : o[i][6], odd ? o[i][3] : o[i][7]);
                            }
                        }
                    }
                    hand_over(rc.s);
                    rc.next2();
                }
                r.skip(n);
                rr.skip(n);
                it += n;
                w.kb = w.end;
            }
            // Adapter columns: both tiles are written here.  (PRE: the producer says when the
            // slot is free; who has not followed every phase of `empty` cannot tell one from the
            // one before the last.)
            if (!more(w, t0)) continue;
            const int* list = a.lists + (int64_t)(t0 / BN) * LT_LIST;
            const int cnt = ld_after(list), per = PARTS * (a.R >> 3);
            auto column = [&](int in) {                     // of the rank
                const int r8 = a.R >> 3;
                if (PARTS > 2 && in >= 2 * r8) in -= r8;
                return (in >= r8 ? in - r8 : in) * 8;
            };
            // Copies: eight neighbouring threads take a row's 128 bytes (a thread a row, every
            // request touched 32 lines, and a stage took 1.4 us).  Thread: piece pc of rows
            // pr, pr + 16, ...; b's rows for the P tile, h's (or g's) for the T tile.
            const int pr = tid >> 3, pc = tid & 7;
            const uint32_t swz = (uint32_t)(pr * 128 + ((pc ^ (pr & 7)) << 4));
            const int tr = t0 + (int)rank * half + pr;
            int ids[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ids[i] = 16 * i < half && tr + 16 * i < a.T ? ld_after(a.ids + tr + 16 * i) : -1;
            // the list's entries win .. win + 31, one a lane
            int win = (w.kb - nk) * 8 / per;
            int entry = ld_after(list + 1 + min(win + lane, 255));
            for (; w.kb < w.end; ++w.kb) {
                if (it % GROUPS == grp) {
                    const uint32_t at = smem_u32(smem + r.s * LT_SLOT), bt = at + LT_A;
                    live = __all_sync(0xffffffffu,
                                      mbar_wait(PRE ? &lgo[r.s] : &empty[r.s],
                                                PRE ? lph >> r.s & 1u : r.ph ^ 1u, status,
                                                abort_flag) && live);
                    lph ^= 1u << r.s;
                    // Columns (kb - nk) * 64 .. +64 of the adapter term, in pieces of 8: per adapter
                    // of the list R / 8 pieces against the high parts, then as many against
                    // each of the others; `in` is a piece's place among an adapter's.
                    const int first = (w.kb - nk) * 8, e0 = first / per;
                    if (e0 + 4 > win + 31) {                    // a stage spans at most 5 adapters
                        win = e0;
                        entry = ld_after(list + 1 + min(win + lane, 255));
                    }
                    const int e = (first + pc) / per, in = first + pc - e * per;
                    const int ad = __shfl_sync(0xffffffffu, entry, e - win);
                    if (live) {
                        if (A_MN) {                             // rows of a: r, 256 bytes of p each
                            const int ar = tid >> 4, ac = tid & 15, p = p0 + ac * 8;
                            const uint32_t to = at + (ac >> 3) * 8192 + ar * 128 +
                                                (((ac & 7) ^ ar) << 4);
                            int ec = e0, ic = first - e0 * per;
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const int adc = __shfl_sync(0xffffffffu, ad, c);
                                const int col = column(ic);
                                const bool pl = ec < cnt && p < a.P;
                                cp_async16(to + 1024 * c,
                                           pl ? a.low + ((int64_t)adc * a.R + col + ar) * a.P + p
                                              : a.low, pl);
                                if (++ic == per) {
                                    ic = 0;
                                    ++ec;
                                }
                            }
                        } else {
                            const int col = column(in);
                            const uint16_t* src =
                                a.low + ((int64_t)ad * a.P + p0 + pr) * a.R + col;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const bool pl = e < cnt && p0 + pr + 16 * i < a.P;
                                cp_async16(at + swz + 2048 * i,
                                           pl ? src + (int64_t)(16 * i) * a.R : a.low, pl);
                            }
                        }
                        const uint16_t* src = a.hp + (int64_t)tr * PARTS * a.R + in * 8;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (16 * i < half) {
                                const bool tl = e < cnt && ids[i] == ad;
                                cp_async16(bt + swz + 2048 * i,
                                           tl ? src + (int64_t)(16 * PARTS * i) * a.R : a.hp, tl);
                            }
                    }
                    // handed over a turn later, when the next copies are on their way
                    cp_commit();
                    if (pending >= 0) {
                        cp_wait<1>();
                        hand_over(pending);
                    }
                    pending = r.s;
                }
                ++it;
                r.next();
            }
            if (pending >= 0) {
                cp_wait<0>();
                hand_over(pending);
                pending = -1;
            }
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        // warp w: lane quarter w % 4 of the CTA's 128 p, every CS-th chunk of 32 t
        constexpr int CS = LT_EPI / 4;
        const int q = warp & 3, par = (warp - LT_EPI0) >> 2;
        const uint32_t tempty0 = lt_map(smem_u32(tempty), lead);
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        LtRing<2> rt;
        bool live = true;
        for (int u = u0; u < units; u += ustep) {
            int p0, t0;
            tile_of(u, p0, t0);
            const int p = p0 + q * 32 + lane;
            const int64_t t1 = min((int64_t)t0 + BN, a.T);
            const int chunks = (BN + 31) / 32;
            // a sum is there, or its place is free again
            auto wait_sum = [&](const LtRing<2>& x) {
                live = __all_sync(0xffffffffu, mbar_wait(&tfull[x.s], x.ph, status, abort_flag) &&
                                                   live);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            };
            auto free_sum = [&](const LtRing<2>& x) {
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) lt_arrive(tempty0 + x.s * 8);
            };
            if (PRE && MODE == LORA_WGRAD && S == 1) {
                // the sums are added up in registers, 128 a thread
                float total[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) total[i][j] = 0.0f;
#pragma unroll 1
                for (int n = 0; n < nsum; ++n) {
                    wait_sum(rt);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (live && par + 2 * i < chunks)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                uint32_t r[16];
                                lt_ld16(lanes + (uint32_t)(rt.s * 256 + (par + 2 * i) * 32 + k * 16),
                                        r);
                                lt_ld_wait();
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    total[i][k * 16 + j] += __uint_as_float(r[j]);
                            }
                    free_sum(rt);
                    rt.next();
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (live && par + 2 * i < chunks)
                        lt_store<MODE, 32>(a, t0 + (par + 2 * i) * 32, t1, p, 0.0f, total[i], a.out,
                                           nullptr, a.accumulate);
                continue;
            }
            float sw = 1.0f, bs = 0.0f;
            if (MODE == LORA_FWD && p < a.P) {
                sw = ld_after(a.s_w + p);
                if (a.bias && S == 1) bs = ld_after(a.bias + p);
            }
            const float* from = nullptr;
            if (MODE != LORA_DGRAD)
#pragma unroll 1
                for (int n = 1; n < nsum; ++n) {
                    wait_sum(rt);
#pragma unroll 1
                    for (int c = par; live && c < chunks; c += CS) {
                        uint32_t r[32];
                        lt_ld32(lanes + (uint32_t)(rt.s * 256 + c * 32), r);
                        lt_ld_wait();
                        float v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = MODE == LORA_FWD ? __uint_as_float(r[j]) * sw
                                                    : __uint_as_float(r[j]);
                        lt_store<MODE, 32>(a, t0 + c * 32, t1, p, bs, v, partial, from, false);
                    }
                    free_sum(rt);
                    rt.next();
                    from = partial;
                    bs = 0.0f;
                }
            if (S > 1) break;                           // finished below, by all warps
            // forward: whether this pair has an adapter term besides its base sum
            Walk w = walk();
            w.kb = w.end;
            const bool low = MODE == LORA_FWD && more(w, t0);
            const LtRing<2> r1 = rt;
            rt.next();
            const LtRing<2> r2 = rt;
            if (low) rt.next();
            wait_sum(r1);
            if (low) wait_sum(r2);
            auto free_sums = [&]() {
                free_sum(r1);
                if (low) free_sum(r2);
            };
            // this pair's part of 32 columns
            auto part = [&](int c, float (&v)[32]) {
                uint32_t r[32];
                lt_ld32(lanes + (uint32_t)(r1.s * 256 + c * 32), r);
                lt_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = MODE == LORA_FWD ? __uint_as_float(r[j]) * sw : __uint_as_float(r[j]);
                if (low) {
                    lt_ld32(lanes + (uint32_t)(r2.s * 256 + c * 32), r);
                    lt_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] += __uint_as_float(r[j]);
                }
            };
            bool held = true;
            if (PRE && MODE != LORA_WGRAD && a.out_bf16 && (a.P & 1) == 0) {
                // all of the warp's columns into registers, rounded and packed in pairs of t,
                // so that the accumulators are free before the stores
                uint32_t w[4][16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = par + 2 * i;
                    if (live && c < chunks) {
                        float v[32];
                        part(c, v);
#pragma unroll
                        for (int j = 0; j < 32; j += 2)
                            w[i][j >> 1] = bf16_bits_rn(v[j] + bs) | bf16_bits_rn(v[j + 1] + bs) << 16;
                    }
                }
                free_sums();
                held = false;
                const int od = lane & 1;
                const int64_t step = a.P;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = par + 2 * i;
                    if (!live || c >= chunks) continue;
                    const int rows = (int)min((int64_t)32, t1 - t0 - c * 32) - od;
                    uint32_t* out = reinterpret_cast<uint32_t*>(a.out) +
                                    (((t0 + c * 32 + od) * step + (p & ~1)) >> 1);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        // neighbouring lanes exchange, so that each stores two p of one t
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, w[i][j], 1);
                        const uint32_t two = od ? __byte_perm(got, w[i][j], 0x7632)
                                                : __byte_perm(w[i][j], got, 0x5410);
                        if (2 * j < rows && p < a.P) *out = two;
                        out += step;
                    }
                }
            } else {
#pragma unroll 1
                for (int c = par; live && c < chunks; c += CS) {
                    float v[32];
                    part(c, v);
                    lt_store<MODE, 32>(a, t0 + c * 32, t1, p, bs, v, a.out, from, a.accumulate);
                }
            }
            if (held) free_sums();
        }
    }
    if (S > 1) {
        // A tile of several pairs: all warps but the first three finish it.  Chunk c of 16 columns
        // belongs to pair c % S; a sender's parts of an owner's chunks lie at [sender][c / S]
        // [column / 4][128 p][4 columns] of the owner's ring region.  (Chunks of 16 and rolled
        // loops: this code runs once, and fetching its instructions is what it waits for.)
        __syncwarp();
        const int q = warp & 3, par = (warp - LT_CONV0) >> 2, step = (LT_CONV + LT_EPI) / 4;
        const int chunks = BN / 16, own = (chunks + S - 1) / S;
        const uint32_t ring = smem_u32(smem) + (uint32_t)((q * 32 + lane) * 16);
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        int p0, t0;
        tile_of(u0, p0, t0);
        const int p = p0 + q * 32 + lane;
        const int64_t t1 = min((int64_t)t0 + BN, a.T);
        float sw = 1.0f, bs = 0.0f;
        bool low = false, live = warp >= LT_CONV0;
        const int b1 = (nsum - 1) & 1, b2 = nsum & 1;           // buffers: last sum, adapter term
        if (live) {
            Walk w = walk();
            w.kb = w.end;
            low = MODE == LORA_FWD && more(w, t0);
            if (MODE == LORA_FWD && p < a.P) {
                sw = ld_after(a.s_w + p);
                if (a.bias) bs = ld_after(a.bias + p);
            }
        }
        auto part = [&](int c, float (&v)[16]) {
            uint32_t r[16];
            lt_ld16(lanes + (uint32_t)(b1 * 256 + c * 16), r);
            lt_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[j] = MODE == LORA_FWD ? __uint_as_float(r[j]) * sw : __uint_as_float(r[j]);
            if (low) {
                lt_ld16(lanes + (uint32_t)(b2 * 256 + c * 16), r);
                lt_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(r[j]);
            }
            if (nsum > 1) {
                const float* from = partial + (int64_t)(t0 + c * 16) * a.P + p;
                const int rows = p < a.P ? (int)min((int64_t)16, t1 - t0 - c * 16) : 0;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < rows) v[j] += ld_after(from + (int64_t)j * a.P);
            }
        };
        // Every pair's MMAs (their issuer has waited for the last) and copies are done behind this:
        // the sums are there and the rings are free.
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        lt_cluster_sync();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        live = __all_sync(0xffffffffu, *abort_flag == 0) && live;
#pragma unroll 1
        for (int c = par; live && c < chunks; c += step) {
            const int o = c % S;
            if (o == pair) continue;
            float v[16];
            part(c, v);
            const uint32_t to =
                lt_map(ring + (uint32_t)((pair * own + c / S) * 8192), (uint32_t)o * 2 + rank);
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(to + j * 512),
                             "f"(v[j]), "f"(v[j + 1]), "f"(v[j + 2]), "f"(v[j + 3])
                             : "memory");
        }
        __syncwarp();
        lt_cluster_sync();              // all parts are there
#pragma unroll 1
        for (int k = par; live && k * S + pair < chunks; k += step) {
            const int c = k * S + pair;
            float v[16], mine[16];
            part(c, mine);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.0f;
#pragma unroll 1
            for (int o = 0; o < S; ++o) {                               // in pair order
                const uint32_t from = ring + (uint32_t)((o * own + k) * 8192);
                float got[16];
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(got[j]), "=f"(got[j + 1]), "=f"(got[j + 2]),
                                   "=f"(got[j + 3])
                                 : "r"(from + j * 512)
                                 : "memory");
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += o == pair ? mine[j] : got[j];
            }
            lt_store<MODE, 16>(a, t0 + c * 16, t1, p, bs, v, a.out, nullptr, a.accumulate);
        }
        __syncwarp();
    }

    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    lt_cluster_sync();      // the other CTA's copies and its threads' arrivals here are complete
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 1) {
        // Arrivals of commits are the tensor core's, not a thread's, and the barrier above says
        // nothing of those in the pair's second CTA.  They come in the order of the commits, so the
        // last one's is the end of them.
        mbar_drain(mma_done, 0, status);
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
    }
}

// ----------------------------------------------------------------------- host side
int lora_tc_tile(int64_t T) {
    const int64_t tiles = (T + 255) / 256;
    return (int)(((T + tiles - 1) / tiles + 31) / 32 * 32);
}
// Most pairs that split a tile's stages (148 SMs: 74 pairs).
static int lora_max_split(int64_t P, int64_t T) {
    const int64_t BN = lora_tc_tile(T), tiles = (P + 255) / 256 * ((T + BN - 1) / BN);
    return tiles <= 18 ? 4 : tiles <= 37 ? 2 : 1;
}
size_t lora_list_bytes(int64_t T) {
    const int64_t BN = lora_tc_tile(T);
    return (size_t)((T + BN - 1) / BN) * LT_LIST * sizeof(int);
}

// Clusters of 2 * S CTAs that run at once (a cluster lies in one GPC, so larger ones leave SMs
// over), asked for once per device.
template <int MODE, bool PRE, int PARTS>
static int lora_tc_clusters(int S) {
    static std::atomic<int> known[128][3];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 0;
    std::atomic<int>& k = known[dev][S >> 1];
    int n = k.load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * S);
    cfg.blockDim = dim3(lt_threads(MODE, PRE));
    cfg.dynamicSmemBytes = LT_SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, k_lora_tc<MODE, PRE, PARTS>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    k.store(n, std::memory_order_relaxed);
    return n;
}

template <int MODE, bool PRE, int PARTS>
static cudaError_t launch_tc(const LoraGemm& a, cudaStream_t st, int num_sms, int* status) {
    const int BN = lora_tc_tile(a.T);
    CUtensorMap pm, tm;
    bool okp;
    if (PRE)
        okp = MODE == LORA_FWD ? make_tmap_u8_2d(&pm, a.pre, a.P, (int64_t)a.C * 2, 128, 128,
                                                 CU_TENSOR_MAP_SWIZZLE_128B)
                               : make_tmap_u8_2d(&pm, a.pre, a.C, (int64_t)a.P * 2, 128, LT_BK,
                                                 CU_TENSOR_MAP_SWIZZLE_128B);
    else
        okp = MODE == LORA_FWD
                  ? make_tmap_u8_2d(&pm, a.q, a.P, a.C, LT_BK, 128, CU_TENSOR_MAP_SWIZZLE_64B)
                  : make_tmap_u8_2d(&pm, a.q, a.C, a.P, 128, LT_BK, CU_TENSOR_MAP_SWIZZLE_NONE);
    const bool okt = MODE == LORA_WGRAD
                         ? make_tmap_u8_2d(&tm, a.t, a.C, a.T * 2, 128, LT_BK,
                                           CU_TENSOR_MAP_SWIZZLE_128B)
                         : make_tmap_u8_2d(&tm, a.t, a.T, (int64_t)a.C * 2, 128, BN / 2,
                                           CU_TENSOR_MAP_SWIZZLE_128B);
    if (!okp || !okt) return cudaErrorInvalidValue;
    cudaError_t e = ensure_dyn_smem<k_lora_tc<MODE, PRE, PARTS>>(LT_SMEM);
    if (e != cudaSuccess) return e;
    const int64_t num_p = (a.P + 255) / 256, num_t = (a.T + BN - 1) / BN, tiles = num_p * num_t;
    if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
    // Pairs that split a tile's stages: while all clusters run at once and each part keeps at
    // least 4 stages.
    int S = 1;
    while (2 * S <= lora_max_split(a.P, a.T) && tiles * 2 <= num_sms / 2 / S &&
           a.C / LT_BK >= 4 * 2 * S && tiles <= lora_tc_clusters<MODE, PRE, PARTS>(2 * S))
        S *= 2;
    const int64_t clusters = tiles < num_sms / 2 ? tiles : num_sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * S * clusters));
    cfg.blockDim = dim3(lt_threads(MODE, PRE));
    cfg.dynamicSmemBytes = LT_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2 * S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_lora_tc<MODE, PRE, PARTS>, pm, tm, a, BN, (int)num_p, (int)num_t,
                              S, status);
}

cudaError_t launch_lora_tc(int mode, const LoraGemm& a, cudaStream_t st, int num_sms,
                           int* status) {
#define LT_MODE(M_, PARTS_)                                       \
    (a.pre ? launch_tc<M_, true, PARTS_>(a, st, num_sms, status)  \
           : launch_tc<M_, false, PARTS_>(a, st, num_sms, status))
    if (mode == LORA_FWD)
        return a.out_bf16 ? LT_MODE(LORA_FWD, lora_parts(true)) : LT_MODE(LORA_FWD, lora_parts(false));
    if (mode == LORA_DGRAD) return LT_MODE(LORA_DGRAD, lora_parts(true));
    return LT_MODE(LORA_WGRAD, lora_parts(true));
#undef LT_MODE
}

// ------------------------------------------------------------------------- expansion
// The int8 operand in bf16 for PRE, twice 16 values a thread: q (forward), s_w[c] * q rounded once
// (dgrad), or code * 2^e.
template <int MODE>
__global__ __launch_bounds__(256) void k_lora_expand(const LoraGemm a, int64_t n16, int row16,
                                                     uint16_t* __restrict__ out, bool beside) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t i0 = (int64_t)blockIdx.x * 512 + threadIdx.x;
    uint4 w[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
        if (i0 + u * 256 < n16) w[u] = ldg_stream(reinterpret_cast<const uint4*>(a.q) + i0 + u * 256);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int64_t i = i0 + u * 256;
        if (i >= n16) break;
        uint32_t o[8];
        s8x4_to_bf16x2_seq(w[u].x, o[0], o[1]);
        s8x4_to_bf16x2_seq(w[u].y, o[2], o[3]);
        s8x4_to_bf16x2_seq(w[u].z, o[4], o[5]);
        s8x4_to_bf16x2_seq(w[u].w, o[6], o[7]);
        if (MODE != LORA_FWD) {
            const int64_t c = i / row16;
            const LtScale f =
                lt_scale<MODE>(lt_scale_bits<MODE>(a, (int)c, (int)(i - c * row16) * 16));
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = lt_apply<MODE>(o[j], f);
        }
        uint4* to = reinterpret_cast<uint4*>(out) + 2 * i;
        to[0] = make_uint4(o[0], o[1], o[2], o[3]);
        to[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    // beside the kernels that make h or g: it neither reads nor writes what they do, and what it
    // reads is older than the plan, whose launch waited for all of the stream's earlier work.
    // Who waits for this kernel waits for those too: its last block does.
    if (beside && blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The expansion moves 3 bytes a value and is a launch more; the conversion inside the GEMM costs up
// to a seventh of its time, which grows with the product.  Measured, us, expanded / converted
// inside, rank 16: forward, 4096 x 11008, T = 1024: 107 / 90, 2048: 159 / 151, 4096: 290 / 294;
// 2048 x 8192, 2048: 75 / 76, 4096: 121 / 128; 960 x 2560, 4096 (2e10 operations): 42 / 43.  dgrad,
// whose conversion rounds: 4096 x 11008, 768: 92 / 90, 1536: 149 / 162, 4096: 311 / 354; 4096 x 4096,
// 1024: 45 / 45, 2048: 67 / 74; 960 x 2560, 1536 (8e9): 28 / 29.  Weight gradient of M rows:
// 4096 x 11008, M = 512: 51 / 52, 4096: 310 / 327; 2048 x 8192, 768 (3e10): 30 / 29, 2048: 59 / 62.
// A weight gradient of more rows than one sum takes is expanded from T = 896 on whatever its size
// (960 x 2560, 2048 rows: 19 us either way): only that form adds its sums up in registers.
struct LtPreRule {
    int64_t t;
    double ops;
};
size_t lora_pre_bytes(int mode, int64_t P, int64_t C, int64_t T) {
    const LtPreRule r = mode == LORA_FWD     ? LtPreRule{2560, 3e10}
                        : mode == LORA_DGRAD ? LtPreRule{1280, 5e9}
                                             : LtPreRule{896, 3e10};
    const bool long_sum = mode == LORA_WGRAD && C > LT_SUM * LT_BK;
    return T >= r.t && (long_sum || 2.0 * (double)P * (double)C * (double)T >= r.ops)
               ? (size_t)P * (size_t)C * 2 : 0;
}
// Partial sums: of every pair that may split a tile, or of the whole where neither registers nor
// the result itself (accumulate) can hold them.
size_t lora_partial_bytes(int mode, int64_t P, int64_t C, int64_t T) {
    if (C <= LT_SUM * LT_BK || mode == LORA_DGRAD) return 0;
    int64_t copies = lora_max_split(P, T);
    if (copies == 1 && (mode == LORA_FWD || lora_pre_bytes(mode, P, C, T) > 0)) copies = 0;
    return (size_t)copies * (size_t)P * (size_t)T * 4;
}
cudaError_t launch_lora_expand(int mode, const LoraGemm& a, uint16_t* out, bool beside,
                               cudaStream_t st) {
    const int64_t n16 = (int64_t)a.P * a.C / 16;
    const int row16 = (mode == LORA_FWD ? a.C : a.P) / 16;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((n16 + 511) / 512));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = beside ? 1 : 0;
    if (mode == LORA_FWD)
        return cudaLaunchKernelEx(&cfg, k_lora_expand<LORA_FWD>, a, n16, row16, out, beside);
    if (mode == LORA_DGRAD)
        return cudaLaunchKernelEx(&cfg, k_lora_expand<LORA_DGRAD>, a, n16, row16, out, beside);
    return cudaLaunchKernelEx(&cfg, k_lora_expand<LORA_WGRAD>, a, n16, row16, out, beside);
}

}  // namespace q8
