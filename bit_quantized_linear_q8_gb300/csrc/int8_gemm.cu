// int8_gemm.cu -- W8A8 product: out[m, n] = BF16(sa[m] sw[n] sum_k a[m, k] w[n, k]), int8 codes with
// one fp32 scale per token and one per output channel.
//
// Design (GB300, sm_103a).  sm_103a's tcgen05 has no int8 kind, so the codes enter the FP16
// kind (kind::f16): an int8 code is exact in FP16, a product of two is exact in fp32, and the
// tensor core's fp32 sums are exact integers while they stay below 2^24 (beyond that they
// round like any fp32 sum).  The scales are applied once to the finished sum.
//  * The weight is the A operand and goes to the tensor core through tensor memory: a tile is up
//    to 128 weight rows (output channels = tensor-memory lanes) x N tokens (columns).  Expanding
//    the codes into tensor memory instead of shared memory keeps the expanded weight out of
//    the shared-memory port, which the activations' reads already fill.  An M128 N K16 MMA takes
//    about 34 + N / 2 cycles in these steps, 32 more with A in shared memory (alone and back to back N / 2).
//  * Weight codes stream through a ring of TMA boxes, R rows of 128 bytes (16 KB, 128-byte
//    swizzle).  Warps 4-11 (two groups of four, one lane quadrant a warp, one weight row a
//    thread; the groups take alternate steps) expand them: a byte permute puts code + 128 into
//    the mantissa of 1024, one packed subtraction of 1152 leaves the code (1.25 instructions a
//    value), and tcgen05.st writes the operand.
//  * Warp 0 issues the MMAs from warp-uniform operands by one elected lane, without branches:
//    operands that the compiler cannot prove uniform cost 155 cycles an MMA, a bounded wait
//    written as a loop in C 220-500 cycles where the one of mbar_wait_lean costs about 30
//    (16384 x 5120 at m = 2048: 282 us with neither, 262 with the first, 200 with both).
//  * Small-m form, m <= IG_SMALL_M: warps 2 and 3 (and with more than 32 tokens 12 and 13) take
//    alternate steps, copy the activations' codes by cp.async (a TMA request for a few hundred
//    bytes costs an SM as much as a weight box) and expand them into the B operand in shared
//    memory.  Warps 4-11 read the accumulator, scale and store.
//  * Large-m form: a kernel expands the codes once into the caller's scratch (2 m k bytes) and
//    warp 2 streams FP16 boxes by TMA.  Pairs of CTAs of a cluster run neighbouring weight tiles of
//    the same tokens as one M 256 MMA (cta_group::2): the weight rows in each CTA's own tensor memory, half of
//    every token box in each CTA's shared memory.  The first CTA issues for both; the second's expanding and
//    storing warps arrive on its barriers, relaxed (tensor memory is ordered by the tcgen05 fences; with a
//    release, which waits for the thread's other accesses, 2048 x 16384 x 5120 took 233 us, 188 without).
//    Warps 12-19 store, so that the expanding warps go on with the next tile.
//  * Few tiles: the K steps of a tile are split over a cluster of up to 8 CTAs, whose fp32
//    partial sums meet through distributed shared memory in a fixed order (ig_plan).
//  * Launched programmatically: the setup runs while the kernel before drains (every launch 2 us
//    sooner: 16384 x 5120 at m = 1 21.8 -> 19.5 us).
//  * Every wait is bounded.  A role whose wait gives up ends its loop after the step (nothing that it
//    reads or writes depends on the data), so the others' waits give up too, and the status word is
//    raised.
// Bound: small m by the weight's bytes, n k at the memory's rate, beside a fixed 6 us of launch,
// ring filling and reduction (16384 x 5120: 19.5 us at m = 1; 16384 x 20480: 62 us, 6.4 TB/s
// beyond the fixed part); large m by the tensor cores, with the expansion beside it (m = 2048,
// 16384 x 5120: 188 us, 1.83 PFLOP/s, in a run of a few milliseconds, 200 us under the power cap of a long one,
// the expansion of the activations included).
#include "common.cuh"

namespace bq8 {

static __device__ unsigned int g_int8_gemm_status;

unsigned int int8_gemm_status_take() {
    unsigned int v = 0, zero = 0;
    cudaDeviceSynchronize();
    cudaMemcpyFromSymbol(&v, g_int8_gemm_status, sizeof v);
    cudaMemcpyToSymbol(g_int8_gemm_status, &zero, sizeof zero);
    return v;
}

constexpr int IG_BM = 128;                      // weight rows per tile
constexpr uint32_t IG_ASTAGE = IG_BM * 128;     // 16 KB: 128 codes of each row
constexpr uint32_t IG_SMALL_M = 128;            // largest m whose codes the kernel expands itself
constexpr int IG_MAXN = 256;
constexpr int IG_THREADS = 14 * 32;             // small-m form: the expanding warps also store
constexpr int IG_THREADS_PRE = 20 * 32;         // large-m form: eight warps of their own store
constexpr int IG_MAXST = 16;                    // most stages of any ring

// The launch's shape, chosen on the host (ig_plan).
struct IgPlan {
    int N;        // tokens per tile, a multiple of 16
    int R;        // weight rows per tile, at most IG_BM (the lanes past R hold anything)
    int ntm;      // token tiles
    int ntiles;   // token tiles x weight tiles
    int split;    // CTAs of a cluster that share one tile's K steps
    int pair;     // 2: CTAs of a cluster run two weight tiles of the same tokens (large-m form), else 1
    int nA, nB;   // ring stages: weight codes (128 wide; even, so that a stage is always the same warp
                  // group's and its phases are waited for in turn), B operand (64 wide)
    int halves;   // 2: two warps a step expand the activations, half of the rows each (small-m form), else 1
    int xd;       // steps of activation codes in flight for each of two warps, 2 or 4 (small-m form)
    int nT;       // tensor-memory stages of the A operand (64 columns each)
    uint32_t smem;
    uint32_t grid;
};

// 1 in one lane of a converged warp.
__device__ __forceinline__ uint32_t ig_elect() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r;
}

// Arrival on `bar` once the MMAs issued before are done; in a pair on the barriers at the same place in both
// of its CTAs.
template <bool PAIR>
__device__ __forceinline__ void ig_commit(uint64_t* bar, uint32_t both, uint32_t one) {
    if (PAIR)
        asm volatile(
            "{\n.reg .pred e;\nsetp.ne.u32 e, %2, 0;\n"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)both), "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred e;\nsetp.ne.u32 e, %1, 0;\n"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
            "r"(one)
            : "memory");
}

// Arrival of a warp, by one lane and without a branch.
__device__ __forceinline__ void ig_arrive(uint64_t* bar, uint32_t one) {
    asm volatile(
        "{\n.reg .pred e;\nsetp.ne.u32 e, %1, 0;\n@e mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(smem_u32(bar)),
        "r"(one)
        : "memory");
}

// The same on a barrier of another CTA of the cluster (an address of ig_cluster_addr), after tcgen05 operations that
// were waited for and fenced: tensor memory needs no release of the thread's other accesses, which waits
// for all of them.
__device__ __forceinline__ void ig_arrive_cluster(uint32_t addr, uint32_t one) {
    asm volatile(
        "{\n.reg .pred e;\nsetp.ne.u32 e, %1, 0;\n@e mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n}\n" ::"r"(addr),
        "r"(one)
        : "memory");
}

// A tile load into this CTA whose bytes are counted on a barrier of the pair's first CTA.
__device__ __forceinline__ void ig_tma_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void ig_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void ig_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory descriptor of a K-major tile with the 128-byte swizzle (rows of 128 bytes,
// 8-row groups 1024 bytes apart).
__device__ __forceinline__ uint64_t ig_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// D[tmem] (+)= A[tmem] * B[smem]^T, FP16 in, fp32 accumulate, K 16, by the lane with `one`; for a pair M 256,
// the lanes of either CTA's tensor memory against the rows of B in both CTAs' shared memory.
template <bool PAIR>
__device__ __forceinline__ void ig_mma(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate,
                                       uint32_t one) {
    if (PAIR)
        asm volatile(
            "{\n.reg .pred p, e;\nsetp.ne.u32 p, %3, 0;\nsetp.ne.u32 e, %5, 0;\n"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %4, p;\n}\n" ::"r"(d),
            "r"(a), "l"(bdesc), "r"(accumulate), "r"(idesc), "r"(one));
    else
        asm volatile(
            "{\n.reg .pred p, e;\nsetp.ne.u32 p, %3, 0;\nsetp.ne.u32 e, %5, 0;\n"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n}\n" ::"r"(d),
            "r"(a), "l"(bdesc), "r"(accumulate), "r"(idesc), "r"(one));
}

__device__ __forceinline__ void ig_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void ig_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}

// Four int8 codes -> two FP16 pairs: code + 128 in the mantissa of 1024 (ulp 1), minus 1152.
__device__ __forceinline__ void ig_expand4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t off = 0x64806480u;
    const __half2 c = *reinterpret_cast<const __half2*>(&off);
    uint32_t p0 = __byte_perm(u, 0x64646464u, 0x4140u), p1 = __byte_perm(u, 0x64646464u, 0x4342u);
    __half2 h0 = __hsub2(*reinterpret_cast<__half2*>(&p0), c), h1 = __hsub2(*reinterpret_cast<__half2*>(&p1), c);
    lo = *reinterpret_cast<uint32_t*>(&h0);
    hi = *reinterpret_cast<uint32_t*>(&h1);
}

__device__ __forceinline__ void ig_expand16(const uint4& w, uint32_t* r) {
    ig_expand4(w.x, r[0], r[1]);
    ig_expand4(w.y, r[2], r[3]);
    ig_expand4(w.z, r[4], r[5]);
    ig_expand4(w.w, r[6], r[7]);
}

// A ring position: stage and the parity of its current use.
struct IgPos {
    int s = 0;
    uint32_t p = 0;
    __device__ __forceinline__ void next(int n) {
        if (++s == n) {
            s = 0;
            p ^= 1u;
        }
    }
};

__device__ __forceinline__ uint32_t ig_cluster_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void ig_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void ig_store(uint16_t* __restrict__ out, size_t at, float acc, float sa, float sw) {
    const __nv_bfloat16 b = __float2bfloat16_rn(acc * sa * sw);
    out[at] = *reinterpret_cast<const uint16_t*>(&b);
}

// PRE: the activations come expanded (FP16 [m][k]); otherwise as codes.  PAIR (of PRE): two CTAs run two
// neighbouring weight tiles of the same tokens as one M 256 MMA.
template <bool PRE, bool PAIR>
__global__ void __launch_bounds__(PRE ? IG_THREADS_PRE : IG_THREADS, PRE ? 1 : 2)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX,
                     const int8_t* __restrict__ xc, const float* __restrict__ sa, const float* __restrict__ sw,
                     uint16_t* __restrict__ out, int m, int n, int k, const IgPlan pl) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* aring = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // (stays a shared address for the compiler)
    constexpr int COLS = PRE ? 512 : 256;           // tensor-memory columns
    const uint32_t xbytes = (uint32_t)pl.N * (PAIR ? 64u : 128u);  // a 128-byte row per token (of half of a pair's)
    uint8_t* xring = aring + pl.nA * IG_ASTAGE;     // activation codes (not PRE)
    uint8_t* bring = xring + (PRE ? 0 : 2 * pl.xd * xbytes);
    uint64_t* afull = reinterpret_cast<uint64_t*>(bring + pl.nB * xbytes);
    uint64_t* aempty = afull + IG_MAXST;
    uint64_t* bfull = aempty + IG_MAXST;
    uint64_t* bempty = bfull + IG_MAXST;
    uint64_t* tfull = bempty + IG_MAXST;
    uint64_t* tempty = tfull + IG_MAXST;
    uint64_t* accf = tempty + IG_MAXST;
    uint64_t* acce = accf + 1;
    uint64_t* done = acce + 1;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
    int* failed = reinterpret_cast<int*>(tslot + 1);

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);  // uniform
    const int split = pl.split;
    constexpr int pair = PAIR ? 2 : 1;
    // a cluster: `split` shares of K, in each of which `pair` CTAs run neighbouring weight tiles
    const int place = (int)(blockIdx.x % (uint32_t)(split * pair)), rank = place / pair, prank = place % pair;
    const uint32_t both = 3u << (place - prank);  // this CTA and its partner
    // the pair's first CTA issues the MMAs; what they wait for arrives on its barriers
    auto first_cta = [&](uint64_t* bar) { return ig_cluster_addr(smem_u32(bar), (uint32_t)(place - prank)); };
    const int SA = (k + 127) >> 7;  // K steps of 128 codes
    const int s0 = (int)((int64_t)SA * rank / split), s1 = (int)((int64_t)SA * (rank + 1) / split);
    const int first = blockIdx.x / (split * pair), stride = gridDim.x / (split * pair);
    auto row0 = [&](int id) { return (id / pl.ntm * pair + prank) * pl.R; };  // first weight row of this CTA's tile

    // The thread that streams the weight makes the barriers and fills the ring before the CTA meets (the
    // first copies run under the allocation of tensor memory).
    int early = 0;
    if (threadIdx.x == 32) {
        for (int s = 0; s < pl.nA; s++) mbar_init(&afull[s], 1);
        fence_barrier_init();
        pdl_wait();
        if (first < pl.ntiles) {
            early = min(pl.nA, s1 - s0);
            for (int s = 0; s < early; s++) {
                mbar_arrive_expect_tx(&afull[s], (uint32_t)pl.R * 128u);
                tma_load_2d(aring + s * IG_ASTAGE, &mapW, (s0 + s) * 128, row0(first), &afull[s]);
            }
        }
        for (int s = 0; s < pl.nA; s++) mbar_init(&aempty[s], 4);  // one arrival per expanding warp
        for (int s = 0; s < pl.nB; s++) {
            mbar_init(&bfull[s], PRE ? 1u : (uint32_t)pl.halves);
            mbar_init(&bempty[s], 1);
        }
        for (int s = 0; s < pl.nT; s++) {
            mbar_init(&tfull[s], 4 * pair);
            mbar_init(&tempty[s], 1);
        }
        mbar_init(accf, 1);
        mbar_init(acce, 8 * pair);
        mbar_init(done, 1);
        *failed = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        if (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "n"(COLS));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "n"(COLS));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
        // The next kernel's CTAs may take free SM space from here on: not before the kernels before have
        // ended (some read their weights before they wait), nor before this CTA has its tensor
        // memory, which they could hold while they wait for this grid's end.
        pdl_wait();
        pdl_launch_dependents();
    }
    pdl_wait();  // the kernels before have ended: from here on memory is read and written
    ig_fence_before();
    __syncthreads();
    if (PAIR) ig_cluster_sync();  // both CTAs' barriers exist before any remote arrival
    ig_fence_after();
    const uint32_t tbase = __shfl_sync(0xffffffffu, *tslot, 0);
    const uint32_t tA = tbase + (uint32_t)(COLS - 64 * pl.nT);  // the A operand's stages

    if (warp == 1) {
        // ---------------------------------------------------------------- TMA: codes
        if (lane == 0) {
            IgPos a;
            int64_t cnt = 0;
            bool ok = true;
            for (int id = first; id < pl.ntiles && ok; id += stride) {
                const int n0 = row0(id);
                for (int s = s0; s < s1; s++, cnt++, a.next(pl.nA)) {
                    if (cnt < early) continue;
                    if (cnt >= pl.nA && !mbar_wait_lean(&aempty[a.s], a.p ^ 1u)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&afull[a.s], (uint32_t)pl.R * 128u);
                    tma_load_2d(aring + a.s * IG_ASTAGE, &mapW, s * 128, n0, &afull[a.s]);
                }
            }
            if (!ok) *failed = 1;
            // wind down: every copy requested has landed before the CTA ends
            for (int64_t j = cnt > pl.nA ? cnt - pl.nA : 0; j < cnt; j++)
                if (!mbar_wait_suspend(&afull[j % pl.nA], (uint32_t)(j / pl.nA) & 1u)) atomicOr(&g_int8_gemm_status, 2u);
        }
        __syncwarp();
    } else if (warp == 0 && prank > 0) {
        // (the pair's first CTA issues for both)
    } else if (warp == 0) {
        // ---------------------------------------------------------------- MMA issuer
        // The whole warp runs the loop, so that every operand is warp-uniform, and one elected lane
        // issues (operands that the compiler cannot prove uniform cost 155 cycles an MMA).
        // D fp32 (bit 4), A and B FP16, both K-major, N >> 3 at bits 17-22, M >> 4 at bits 24-28
        const uint32_t idesc = (1u << 4) | ((uint32_t)(pl.N >> 3) << 17) | ((uint32_t)(IG_BM * pair >> 4) << 24);
        const uint32_t bbase = __shfl_sync(0xffffffffu, smem_u32(bring), 0);
        const uint32_t one = ig_elect();
        IgPos t, b;
        bool ok = true;
        int ti = 0;
        for (int id = first; id < pl.ntiles && ok; id += stride, ti++) {
            if (ti > 0) ok = mbar_wait_lean<PAIR>(acce, (uint32_t)(ti - 1) & 1u);
            for (int s = s0; s < s1 && ok; s++) {
                ok = mbar_wait_lean<PAIR>(&tfull[t.s], t.p);
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    ok &= mbar_wait_lean(&bfull[b.s], b.p);
                    ig_fence_after();
                    const uint64_t bd = ig_desc(bbase + (uint32_t)b.s * xbytes);
                    const uint32_t aa = tA + 64u * t.s + 32u * h;
#pragma unroll
                    for (int kk = 0; kk < 4; kk++)
                        ig_mma<PAIR>(tbase, aa + 8u * kk, bd + 2u * kk, idesc, h | kk ? 1u : (uint32_t)(s - s0), one);
                    ig_commit<PAIR>(&bempty[b.s], both, one);
                    b.next(pl.nB);
                }
                ig_commit<PAIR>(&tempty[t.s], both, one);
                t.next(pl.nT);
            }
            ig_commit<PAIR>(accf, both, one);
        }
        ig_commit<PAIR>(done, both, one);  // completes once every MMA issued above has finished
        if (!mbar_wait_suspend(done, 0)) ok = false;
        if (!ok) *failed = 1;
    } else if (warp < 4 || (!PRE && warp >= 12)) {
        if (PRE) {
            // ------------------------------------------------------------ TMA: expanded activations
            if (warp == 2 && lane == 0) {
                IgPos b;
                int64_t cnt = 0;
                bool ok = true;
                for (int id = first; id < pl.ntiles && ok; id += stride) {
                    const int m0 = (id % pl.ntm) * pl.N;
                    for (int s = 2 * s0; s < 2 * s1; s++, cnt++, b.next(pl.nB)) {
                        if (cnt >= pl.nB && !mbar_wait_lean(&bempty[b.s], b.p ^ 1u)) {
                            ok = false;
                            break;
                        }
                        if (prank == 0) mbar_arrive_expect_tx(&bfull[b.s], xbytes * pair);
                        if (PAIR)  // half of the tokens in either CTA
                            ig_tma_pair(bring + b.s * xbytes, &mapX, s * 128, m0 + prank * (pl.N / 2), first_cta(&bfull[b.s]));
                        else
                            tma_load_2d(bring + b.s * xbytes, &mapX, s * 128, m0, &bfull[b.s]);
                    }
                }
                if (!ok) *failed = 1;
                // (a pair's first CTA waits for both; neither leaves before that)
                for (int64_t j = cnt > pl.nB ? cnt - pl.nB : 0; j < cnt && prank == 0; j++)
                    if (!mbar_wait_suspend(&bfull[j % pl.nB], (uint32_t)(j / pl.nB) & 1u))
                        atomicOr(&g_int8_gemm_status, 2u);
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ B operand from codes
            // Warps 2 (and 12) and 3 (and 13) take alternate steps, a half of the rows each.  Each lane copies
            // the 16-code runs that it will expand itself, xd of its steps ahead (asynchronous copies, not
            // TMA: a TMA request costs an SM as much as a whole weight box).  Lane: run lane % 8 of rows
            // lane / 8, + 4, ... of its half
            const int bw = warp & 1, nr = pl.N / (4 * pl.halves), run = lane & 7, r0 = (lane >> 3) + (warp >= 12 ? 4 * nr : 0);
            const uint32_t one = lane == 0, xsrc = (uint32_t)lane * 16u;
            uint8_t* xown = xring + bw * pl.xd * xbytes;
            const uint32_t xhalf = warp >= 12 ? (uint32_t)nr * 512u : 0u, xown_u = smem_u32(xown) + xhalf + xsrc;
            // the two 16-byte pieces of the operand's row that run `run` fills, before the swizzle
            const uint32_t bdst = (uint32_t)r0 * 128u, p0 = (uint32_t)(2 * (run & 3));
            const int64_t step_rows = (int64_t)4 * k;
            IgPos b;
            int cnt = 0;
            bool ok = true;
            for (int id = first; id < pl.ntiles && ok; id += stride) {
                const int m0 = (id % pl.ntm) * pl.N;
                const int8_t* xrow = xc + (int64_t)(m0 + r0) * k + run * 16;
                const int rows = m - m0 - r0;  // row r0 + 4 j is there while 4 j < rows
                // steps of this warp: s0 + bw', s0 + bw' + 2, ... (bw' so that the pair's steps alternate over tiles)
                const int sb = s0 + ((cnt & 1) ^ bw);
                auto fetch = [&](int s, int slot) {
                    if (s < s1) {
                        const bool in = s * 128 + run * 16 < k;
                        const int8_t* src = xrow + s * 128;
                        uint32_t dst = xown_u + (uint32_t)slot * xbytes;
#pragma unroll 4
                        for (int j = 0; j < nr; j++, src += step_rows, dst += 512u) {
                            const bool have = in && 4 * j < rows;  // zeros past the ends
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                                         "l"(reinterpret_cast<uint64_t>(have ? src : xc)), "r"(have ? 16 : 0)
                                         : "memory");
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                for (int d = 0; d < pl.xd - 1; d++) fetch(sb + 2 * d, d);
                int slot = 0;
                for (int s = s0; s < s1 && ok; s++, cnt++) {
                    IgPos b2 = b;
                    b2.next(pl.nB);
                    if ((cnt & 1) == bw) {
                        fetch(s + 2 * (pl.xd - 1), (slot + pl.xd - 1) & (pl.xd - 1));
                        if (pl.xd == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
                        else asm volatile("cp.async.wait_group 1;" ::: "memory");
                        if (2 * cnt >= pl.nB) {
                            ok = mbar_wait_lean(&bempty[b.s], b.p ^ 1u);
                            ok &= mbar_wait_lean(&bempty[b2.s], b2.p ^ 1u);
                        }
                        const uint8_t* src = xown + slot * xbytes + xhalf + xsrc;
                        uint8_t* dst = bring + ((run & 4) ? b2.s : b.s) * xbytes + bdst;
#pragma unroll 2
                        for (int j = 0; j < nr; j += 2, src += 1024, dst += 1024) {  // nr: a multiple of 2
                            uint4 w[2];
#pragma unroll
                            for (int i = 0; i < 2; i++) w[i] = *reinterpret_cast<const uint4*>(src + 512 * i);
#pragma unroll
                            for (int i = 0; i < 2; i++) {
                                const uint32_t x = (uint32_t)(r0 + 4 * (j + i)) & 7u;
                                uint32_t r[8];
                                ig_expand16(w[i], r);
                                *reinterpret_cast<uint4*>(dst + 512 * i + ((p0 ^ x) << 4)) = make_uint4(r[0], r[1], r[2], r[3]);
                                *reinterpret_cast<uint4*>(dst + 512 * i + (((p0 + 1u) ^ x) << 4)) =
                                    make_uint4(r[4], r[5], r[6], r[7]);
                            }
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        ig_arrive(&bfull[b.s], one);
                        ig_arrive(&bfull[b2.s], one);
                        slot = (slot + 1) & (pl.xd - 1);
                    }
                    b = b2;
                    b.next(pl.nB);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
            }
            if (!ok) *failed = 1;
        }
    } else if (!PRE || warp < 12) {
        // ---------------------------------------------------------------- A operand (and epilogue)
        const int qd = warp & 3, g = (warp - 4) >> 2;
        const int row = 32 * qd + lane;
        const uint32_t tq = (uint32_t)(32 * qd) << 16, one = lane == 0, tfull0 = PAIR ? first_cta(tfull) : 0u;
        IgPos a, t;
        int cnt = 0, ti = 0;
        bool ok = true;
        for (int id = first; id < pl.ntiles && ok; id += stride, ti++) {
            if (!PRE) {  // the scales on their way into L2
                const int nr = row0(id) + row, tok = (id % pl.ntm) * pl.N + row;
                if (g == 0 && nr < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(sw + nr));
                if (g == 1 && tok < m) asm volatile("prefetch.global.L2 [%0];" ::"l"(sa + tok));
            }
            for (int s = s0; s < s1; s++, cnt++, a.next(pl.nA), t.next(pl.nT)) {
                if ((cnt & 1) != g) continue;
                ok = mbar_wait_lean(&afull[a.s], a.p);
                if (cnt >= pl.nT) ok &= mbar_wait_lean(&tempty[t.s], t.p ^ 1u);
                if (!ok) break;
                ig_fence_after();
                const uint8_t* src = aring + a.s * IG_ASTAGE + row * 128;
                const uint32_t dst = tA + tq + 64u * t.s;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const uint4 w0 = *reinterpret_cast<const uint4*>(src + (((2 * c) ^ (row & 7)) << 4));
                    const uint4 w1 = *reinterpret_cast<const uint4*>(src + (((2 * c + 1) ^ (row & 7)) << 4));
                    uint32_t r[16];
                    ig_expand16(w0, r);
                    ig_expand16(w1, r + 8);
                    ig_st16(dst + 16u * c, r);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                ig_fence_before();
                __syncwarp();
                if (PAIR) ig_arrive_cluster(tfull0 + 8u * t.s, one);
                else ig_arrive(&tfull[t.s], one);
                ig_arrive(&aempty[a.s], one);
            }
            if (!PRE && ok) {
                ok = mbar_wait_lean(accf, (uint32_t)ti & 1u);
                if (!ok) break;
                ig_fence_after();
                const int m0 = (id % pl.ntm) * pl.N, nr = row0(id) + row;
                const bool mine = row < pl.R && nr < n;
                const float swr = (split == 1 && mine) ? sw[nr] : 0.0f;
                for (int c = 16 * g; c < pl.N; c += 32) {
                    if (m0 + c >= m) break;
                    float v[16];
                    ig_ld16(tbase + tq + (uint32_t)c, v);
                    if (split > 1) {
                        // this CTA's partial sums [token][row], over the ring (all of it consumed)
                        float* part = reinterpret_cast<float*>(aring) + c * IG_BM + row;
#pragma unroll
                        for (int j = 0; j < 16; j++) part[j * IG_BM] = v[j];
                    } else if (mine) {
#pragma unroll
                        for (int j = 0; j < 16; j++) {
                            const int tok = m0 + c + j;
                            if (tok < m) ig_store(out, (size_t)tok * n + nr, v[j], __ldg(sa + tok), swr);
                        }
                    }
                }
                ig_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce);
            }
        }
        if (!ok) *failed = 1;
    } else {
        // ---------------------------------------------------------------- epilogue (large m)
        // The whole accumulator goes to registers first (as BF16, half of the tokens a warp), so that the
        // next tile's MMAs wait for that only and not for the stores.
        const int qd = warp & 3, g = (warp - 12) >> 2;
        const int row = 32 * qd + lane;
        const uint32_t tq = (uint32_t)(32 * qd) << 16;
        const int half = pl.N / 2, odd = lane & 1;  // N is a multiple of 32 here
        const uint32_t acce0 = PAIR ? first_cta(acce) : 0u;
        int ti = 0;
        for (int id = first; id < pl.ntiles; id += stride, ti++) {
            if (!mbar_wait_lean(accf, (uint32_t)ti & 1u)) {
                *failed = 1;
                break;
            }
            ig_fence_after();
            const int m0 = (id % pl.ntm) * pl.N + half * g, nr = row0(id) + row;
            const bool mine = row < pl.R && nr < n;
            if (split > 1) {
                float* part = reinterpret_cast<float*>(aring) + half * g * IG_BM + row;
                for (int c = 0; c < half && m0 + c < m; c += 16) {
                    float v[16];
                    ig_ld16(tbase + tq + (uint32_t)(half * g + c), v);
#pragma unroll
                    for (int j = 0; j < 16; j++) part[(c + j) * IG_BM] = v[j];
                }
            } else {
                const float swr = mine ? sw[nr] : 0.0f;
                uint32_t o[IG_MAXN / 4];
#pragma unroll
                for (int c = 0; c < IG_MAXN / 2; c += 16) {
                    if (c < half) {
                        float v[16];
                        ig_ld16(tbase + tq + (uint32_t)(half * g + c), v);
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            const int tok = min(m0 + c + 2 * j, m - 1);
                            const float s0v = __ldg(sa + tok), s1v = __ldg(sa + min(tok + 1, m - 1));
                            o[c / 2 + j] = bf162_bits(__floats2bfloat162_rn(v[2 * j] * s0v * swr, v[2 * j + 1] * s1v * swr));
                        }
                    }
                }
                ig_fence_before();
                __syncwarp();
                if (PAIR) ig_arrive_cluster(acce0, lane == 0);
                else ig_arrive(acce, lane == 0);
                // Even n and R: neighbouring lanes exchange, the even one stores the pair's rows of the even
                // tokens and the odd one those of the odd tokens.
                const bool pairs = ((n | pl.R) & 1) == 0;
                const size_t at = (size_t)(m0 + (pairs ? odd : 0)) * n + (pairs ? nr & ~1 : nr);
                const int live = m - m0 - (pairs ? odd : 0);
#pragma unroll
                for (int c = 0; c < IG_MAXN / 2; c += 2) {
                    if (c < half) {
                        const uint32_t w = o[c / 2];
                        if (pairs) {
                            const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 1);
                            const uint32_t pr = odd ? __byte_perm(other, w, 0x7632u) : __byte_perm(w, other, 0x5410u);
                            if (mine && c < live) *reinterpret_cast<uint32_t*>(out + at + (size_t)c * n) = pr;
                        } else if (mine) {
                            if (c < live) out[at + (size_t)c * n] = (uint16_t)w;
                            if (c + 1 < live) out[at + (size_t)(c + 1) * n] = (uint16_t)(w >> 16);
                        }
                    }
                }
                continue;
            }
            ig_fence_before();
            __syncwarp();
            if (PAIR) ig_arrive_cluster(acce0, lane == 0);
            else ig_arrive(acce, lane == 0);
        }
    }

    ig_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *failed) atomicOr(&g_int8_gemm_status, 1u);
    if (PAIR) {
        // no MMA, copy or arrival of the pair is under way past this point
        if (threadIdx.x == 0 && prank > 0 && !mbar_wait_suspend(done, 0)) atomicOr(&g_int8_gemm_status, 2u);
        __syncwarp();
        ig_cluster_sync();
    }
    if (warp == 0) {
        ig_fence_after();
        if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "n"(COLS));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "n"(COLS));
    }
    if (split > 1) {
        // every CTA of the cluster sums the partials of its share of the tokens, rank by rank
        ig_cluster_sync();
        if (!*failed && first < pl.ntiles) {
            const int m0 = (first % pl.ntm) * pl.N, n0 = row0(first);
            const uint32_t base = smem_u32(aring);
            const int tokens = min(pl.N, m - m0);
            // four rows a thread; the loads of all ranks in flight at once (one after the other they cost 0.3 us each)
            for (int i = threadIdx.x; i < IG_BM / 4 * ((tokens + split - 1) / split); i += (int)blockDim.x) {
                const int row = 4 * (i & (IG_BM / 4 - 1)), c = i / (IG_BM / 4) * split + rank;
                if (c >= tokens || row >= pl.R || n0 + row >= n) continue;
                float4 v[8];
#pragma unroll
                for (int r = 0; r < 8; r++)
                    if (r < split)
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                                     : "r"(ig_cluster_addr(base + (uint32_t)(c * IG_BM + row) * 4u, (uint32_t)(r * pair + prank))));
                float acc[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
                for (int r = 1; r < 8; r++)
                    if (r < split) acc[0] += v[r].x, acc[1] += v[r].y, acc[2] += v[r].z, acc[3] += v[r].w;
                const float sav = __ldg(sa + m0 + c);
                const size_t at = (size_t)(m0 + c) * n + n0 + row;
                if ((n & 3) == 0) {
                    const float4 w = __ldg(reinterpret_cast<const float4*>(sw + n0 + row));
                    *reinterpret_cast<uint2*>(out + at) =
                        make_uint2(bf162_bits(__floats2bfloat162_rn(acc[0] * sav * w.x, acc[1] * sav * w.y)),
                                   bf162_bits(__floats2bfloat162_rn(acc[2] * sav * w.z, acc[3] * sav * w.w)));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        if (n0 + row + j < n) ig_store(out, at + j, acc[j], sav, __ldg(sw + n0 + row + j));
                }
            }
        }
        ig_cluster_sync();  // no CTA leaves while another still reads its partials
    }
}

// int8 codes -> FP16, 16 codes a thread and step (the activations of the large-m form).
__global__ void __launch_bounds__(256) int8_expand_kernel(const uint4* __restrict__ codes, uint4* __restrict__ out,
                                                          int64_t total) {
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        uint32_t r[8];
        ig_expand16(ldg_nc128(codes + i), r);
        out[2 * i] = make_uint4(r[0], r[1], r[2], r[3]);
        out[2 * i + 1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

constexpr uint32_t IG_SMEM1 = 227 * 1024, IG_SMEM2 = 112 * 1024;  // shared memory of one CTA an SM, of two

// CTAs of the small-m form that run at once in clusters of `size`, one or two an SM: clusters do not
// fill every group of SMs (152 SMs hold 46 clusters of 3 or 15 of 7, one CTA an SM).  Shared memory is
// what limits them, so a kernel without tensor memory is asked for: for one with it the runtime answers
// with one CTA an SM whatever it allocates, where two of 256 columns do run.
static int ig_capacity(int size, int per_sm) {
    static thread_local int cache[2][9] = {};
    int c = cache[per_sm - 1][size];
    if (c) return c;
    const uint32_t smem = per_sm == 1 ? IG_SMEM1 : IG_SMEM2;
    cudaFuncSetAttribute(int8_expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)IG_SMEM1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(size * 64));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)size;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, int8_expand_kernel, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = sm_count() / (size <= 2 ? size : 2 * size);
    }
    c = n * size;
    cache[per_sm - 1][size] = c;
    return c;
}

// The launch's shape, by a model of the time in cycles.  A step of 128 codes costs the larger of its
// MMAs, 8 (34 + N / 2), and its bytes: a weight box at about 3.4 cycles a 128-byte row, or what an
// SM takes from L2 (64 bytes a cycle); the CTAs of an SM add up.  A launch is as long as its fullest
// SM's, plus what a tile costs beside its steps (filling the rings, the epilogue, the cluster's
// reduction).  Tried: equal cuts of the tokens (up to 8 more than needed: 1000 x 5120 x 5120 in seven cuts
// 51.7 us, 62 in four; 4096 x 5120 x 6144 152 us), weight rows a tile from
// 128 down (tiles that divide more evenly among the SMs), clusters of up to 8 over K, and in the
// large-m form over K and pairs of weight tiles (150 x 5120 x 17408: 34.7 us, 63 over K alone).
static IgPlan ig_plan(uint32_t m, uint32_t n, uint32_t k) {
    const bool pre = m > IG_SMALL_M;
    const int SA = (int)((k + 127) / 128), sms = sm_count();
    const uint32_t bars = (6 * IG_MAXST + 3) * 8 + 16;
    IgPlan best = {};
    double best_t = 1e30;
    const uint32_t cuts0 = (m + IG_MAXN - 1) / IG_MAXN, cuts1 = pre ? cuts0 + (cuts0 < 4 ? 3 : cuts0 < 8 ? cuts0 : 8) : cuts0;
    for (uint32_t cuts = cuts0; cuts <= cuts1; cuts++) {
        IgPlan p = {};
        const uint32_t q = pre ? 32 : 16;
        p.N = (int)((((m + cuts - 1) / cuts) + q - 1) / q * q);
        p.ntm = (int)((m + p.N - 1) / p.N);
        for (int R = IG_BM; R >= 64; R -= 8) {
            const int64_t wt = (n + R - 1) / R;
            if ((int64_t)p.ntm * (wt + 1) * 8 >= (1ll << 31)) continue;
            for (int cluster = 1; cluster <= 16; cluster++) {
                // shares of K alone, then with pairs of weight tiles (which halve what an SM takes of the
                // activations); the large-m form with more than one weight tile always has pairs where one share is taken
                const int pair = cluster > 8 ? 2 : 1, split = cluster > 8 ? cluster - 8 : cluster;
                if (split * pair > 8 || (split > 1 && SA < 2 * split)) continue;
                if (pre && wt > 1 ? split == 1 && pair == 1 : pair == 2) continue;
                const int64_t tiles = (int64_t)p.ntm * ((wt + pair - 1) / pair), ctas = tiles * pair * split;
                // a split tile is a cluster's only one; two CTAs an SM only where their rings fit
                int64_t per = (ctas + sms - 1) / sms;  // of the fullest SM
                if (split > 1 && ctas > ig_capacity(split * pair, 1)) {
                    if (pre || p.N > 64 || ctas > ig_capacity(split, 2)) continue;
                    per = 2;
                }
                const double steps = (double)((SA + split - 1) / split);
                const double mma = 8.0 * (34.0 + p.N / 2.0);
                const double bytes = pre ? (128.0 * R + 256.0 * p.N / pair) / 60.0 : 3.4 * R;
                double step = per * (mma > bytes ? mma : bytes);
                if (!pre && step < 900.0) step = 900.0;  // the latency of one CTA's chain
                const double t = steps * step + (pre && split == 1 ? per * 1500.0 : 0.0) + 3000.0 + (split > 1 ? 2500.0 + 8.0 * p.N : 0.0);
                if (t < best_t * 0.999) {
                    best_t = t;
                    best = p;
                    best.R = R;
                    best.split = split;
                    best.pair = pair;
                    best.ntiles = (int)tiles;
                    best.grid = (uint32_t)ctas;
                }
            }
        }
    }
    if (best.grid == 0) return best;
    IgPlan& p = best;
    const uint32_t xbytes = (uint32_t)p.N * 128u / p.pair;
    // two CTAs an SM (half of the shared memory and of tensor memory each) only where one an SM is
    // too few: the bytes in flight count, not the CTAs
    const int per_sm =
        pre || p.N > 64 || p.grid <= (uint32_t)(p.split > 1 ? ig_capacity(p.split, 1) : sms) ? 1 : 2;
    const uint32_t room = (per_sm == 1 ? IG_SMEM1 : IG_SMEM2) - 1024 - bars;
    if (pre) {
        p.nA = 4;
        p.nB = (int)((room - p.nA * IG_ASTAGE) / xbytes);
        if (p.nB > 8) p.nB = 8;
        p.nT = 4;
        p.smem = 1024 + p.nA * IG_ASTAGE + p.nB * xbytes + bars;
    } else {
        // Two warps a step where one would take longer than the step: 64 x 5120 x 5120 13.8 us (one: 14.8),
        // but 24 x 5120 x 17408 26.3 us (one: 26.0) and 1 x 16384 x 5120 20.0 us (one: 19.6).
        p.halves = p.N > 32 ? 2 : 1;
        p.xd = p.N <= 32 ? 4 : 2;
        p.nB = p.N <= 32 && per_sm == 1 ? 8 : 4;  // a multiple of 4: a step's stages are always the same warp's
        p.nT = p.N <= 64 ? 3 : 2;
        p.nA = (int)((room - (2 * p.xd + p.nB) * xbytes) / IG_ASTAGE) & ~1;
        if (p.nA > 12) p.nA = 12;
        p.smem = 1024 + p.nA * IG_ASTAGE + (2 * p.xd + p.nB) * xbytes + bars;
    }
    const uint32_t slots = (uint32_t)(sms * per_sm) / p.pair * p.pair;
    if (p.split == 1 && p.grid > slots) p.grid = slots;
    return best;
}

template <bool PRE, bool PAIR>
static int ig_launch(const CUtensorMap& mw, const CUtensorMap& mx, const int8_t* xc, const float* sa, const float* sw, uint16_t* out,
                     uint32_t m, uint32_t n, uint32_t k, const IgPlan& pl, cudaStream_t stream, const char* who) {
    // the most that any plan takes, so that threads with different plans all write the same limit
    static int configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 63;
    if (!configured[dev]) {
        if (cudaFuncSetAttribute(int8_gemm_kernel<PRE, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)IG_SMEM1) !=
            cudaSuccess)
            return fail(BQ_ERR_LAUNCH, "%s: cannot reserve %u bytes of shared memory", who, IG_SMEM1);
        configured[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pl.grid);
    cfg.blockDim = dim3(PRE ? IG_THREADS_PRE : IG_THREADS - (pl.halves == 1 ? 64 : 0));
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)(pl.split * pl.pair);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = pl.split * pl.pair > 1 ? 2 : 1;
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, int8_gemm_kernel<PRE, PAIR>, mw, mx, xc, sa, sw, out, (int)m, (int)n, (int)k, pl);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(e == cudaErrorNoKernelImageForDevice ? BQ_ERR_UNSUPPORTED : BQ_ERR_LAUNCH, "%s: launch failed: %s", who,
                    cudaGetErrorString(e));
    }
    return check_launch(who);
}

}  // namespace bq8

using namespace bq8;

extern "C" size_t bq_int8_gemm_scratch_bytes(uint32_t m, uint32_t n, uint32_t k) {
    return (m > IG_SMALL_M && n > 0) ? (size_t)m * k * 2 : 0;
}

extern "C" int int8_gemm(const int8_t* a, const float* sa, const int8_t* w, const float* sw, uint16_t* out,
                         void* scratch, uint32_t m, uint32_t n, uint32_t k, bq_stream_t stream) {
    const char* who = "int8_gemm";
    if (k % 16 != 0) return fail(BQ_ERR_INVALID, "%s: k = %u must be a multiple of 16", who, k);
    if (m == 0 || n == 0) return ok();
    if (!out || !aligned16(out)) return fail(BQ_ERR_INVALID, "%s: out NULL or not 16-byte aligned", who);
    if (m > (1u << 24) || n > (1u << 24) || k > (1u << 24)) return fail(BQ_ERR_INVALID, "%s: shape too large", who);
    if (k == 0) {
        if (cudaMemsetAsync(out, 0, (size_t)m * n * 2, (cudaStream_t)stream) != cudaSuccess)
            return fail(BQ_ERR_LAUNCH, "%s: memset failed", who);
        return ok();
    }
    if (!a || !w || !sa || !sw || !aligned16(a) || !aligned16(w) || !aligned16(sa) || !aligned16(sw))
        return fail(BQ_ERR_INVALID, "%s: a, sa, w and sw must be non-NULL and 16-byte aligned", who);
    const size_t need = bq_int8_gemm_scratch_bytes(m, n, k);
    if (need && (!scratch || !aligned16(scratch)))
        return fail(BQ_ERR_INVALID, "%s: m = %u needs %zu bytes of 16-byte aligned scratch", who, m, need);
    // the plans of this thread's shapes are kept, one a place (forming one takes a microsecond for few
    // tokens, ten for many; a layer alternates between a few shapes)
    struct Kept {
        uint32_t m, n, k, sms;
        IgPlan pl;
    };
    static thread_local Kept kept[64] = {};
    const uint32_t sms = (uint32_t)sm_count();
    Kept& place = kept[((m * 0x9E3779B1u) ^ (n * 0x85EBCA77u) ^ (k * 0xC2B2AE3Du)) >> 26];
    if (place.m != m || place.n != n || place.k != k || place.sms != sms) place = {m, n, k, sms, ig_plan(m, n, k)};
    const IgPlan& pl = place.pl;
    if (pl.grid == 0) return fail(BQ_ERR_INVALID, "%s: too many output tiles", who);
    CUtensorMap mw, mx;
    int st = cached_tmap_2d_u8(&mw, w, k, n, k, 128, (uint32_t)pl.R, true, who);
    if (st) return st;
    if (!need) return ig_launch<false, false>(mw, mw, a, sa, sw, out, m, n, k, pl, (cudaStream_t)stream, who);
    if ((st = cached_tmap_2d_u8(&mx, scratch, (uint64_t)k * 2, m, (uint64_t)k * 2, 128, (uint32_t)(pl.N / pl.pair), true,
                                who)))
        return st;
    const int64_t total = (int64_t)m * k / 16;
    const int64_t want = (total + 255) / 256, most = (int64_t)sm_count() * 8;
    if ((st = launch_programmatic(who, int8_expand_kernel, (uint32_t)(want < most ? want : most), 256, 0, (cudaStream_t)stream,
                                  reinterpret_cast<const uint4*>(a), reinterpret_cast<uint4*>(scratch), total)))
        return st;
    return pl.pair > 1 ? ig_launch<true, true>(mw, mx, nullptr, sa, sw, out, m, n, k, pl, (cudaStream_t)stream, who)
                       : ig_launch<true, false>(mw, mx, nullptr, sa, sw, out, m, n, k, pl, (cudaStream_t)stream, who);
}
