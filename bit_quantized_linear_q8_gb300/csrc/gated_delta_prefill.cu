// gated_delta_prefill.cu -- the gated delta rule over whole prompts, in chunks of 64 tokens on the
// tcgen05 tensor cores.
//
// Per value head (gated_delta.cu has the recurrence), for a chunk of C = 64 tokens with k_i, q_i,
// v_i, beta_i and the running log decay b_i = g_1 + ... + g_i inside the chunk, S the state before:
//     A[i][j] = beta_i e^(b_i - b_j) (k_i . k_j)  for j < i;   T = (I + A)^-1
//     R_i = beta_i (v_i - e^(b_i) S^T k_i);                    V' = T R
//     P[i][j] = e^(b_i - b_j) (q_i . k_j)         for j <= i
//     o_i = scale (e^(b_i) S^T q_i + sum_j P[i][j] v'_j)
//     S  <- e^(b_C) S + sum_i e^(b_C - b_i) k_i v'_i^T
// (V' are the corrections u of the recurrence: unrolling u_i = beta_i (v_i - S_i^T k_i) over the chunk
// gives the unit lower triangular system (I + A) V' = R.)  All exponents are differences of b
// with j <= i, so nothing overflows however strong the decay.
//
// Two stages.  What does not depend on the state is prepared for every chunk on its own: the FP16 form
// of K and Q (once per key head), T, P and the per-token factors (per value head), into the caller's
// scratch in the layout that the tensor cores read.  The recurrence then runs one CTA per (sequence,
// value head) over its chunks.
//  * Many chains (pairs of a sequence and a value head): two kernels, the preparation on all SMs, five
//    blocks of one chunk each an SM, then the recurrence.
//  * Up to half as many chains as SMs: one launch, in which the SMs without a chain prepare the
//    chunks in the order of the chains' need and raise a flag for each (8192 tokens x 48 heads: 342 us,
//    428 with two kernels; 2048 x 48: 106 and 124 us; but 2 sequences, 700 + 300 tokens, x 48: 75 and 57
//    us, the remaining 56 SMs being too few).  A cooperative launch, one CTA an SM: the CTAs that are
//    waited for run.
// (Four warps in the recurrence's own CTA that prepared its next chunk took 811 us for 8192 x 48: a chunk
// of preparation is longer than one of recurrence.)
// Bound: the recurrence by its chain, about 4600 cycles a chunk: three dependent products (S K^T, T R, V''
// K; 2500 cycles of MMAs) and the conversions between them (over a launch a third of the SMs' issue slots
// and a fifth of the tensor pipe are used); the preparation by its barriers and the shared memory's latency (98 us for
// 8192 x 48 on all SMs).
//
// Precision.  All products run in the FP16 kind.  A row of K or Q is scaled by a power of two to
// below 2^8 and its BF16 values (8 bits) are then FP16 values exactly (down to 2^-25 of the row's
// norm).  What is fp32 (S, R, V' and T) is scaled per row by a power of two to below 2^15 and
// split into two FP16 terms, hi + lo = the value to 2^-22 of it, or 2^-39 of its row's largest:
// S K^T and V'' K take 2 products, T R takes 3 (lo x lo, below 2^-22, is dropped).  The two
// products that only reach the BF16 output, S Q^T and P V', take one term of S, P and V', rounded to
// nearest: 2^-11 of each, without a lean, against the output's own 2^-8.  (Three BF16 terms, 24 bits without any scaling, took 6 + 3 + 3 + 2 + 3 products
// for these 3 + 2 + 2 + 1 + 1.)  The state itself is held in fp32 registers and updated there, so the
// tensor cores' sums never run longer than one chunk.  b is a pair of floats, so that b_i - b_j is
// good to fp32 even when b itself is large.
//
// Layout of the recurrence.  Everything is transposed: tensor-memory lane = value column, so every
// thread owns one value column and no data of the recurrence ever crosses threads: S^T, R^T and
// V'^T go from the accumulators through registers back into tensor memory as the A operand of the
// next product, and the B operands (K, Q, T, P) come from shared memory.
//  * Warps 0-7 run the recurrence, two per lane quadrant: each holds half of the key dimensions of
//    the state (64 fp32 registers a thread) and takes half of the tokens of R and V'.  S is scaled
//    from its largest value before the chunk and a bound on dS, R by a bound that is known before
//    S^T k is, V' and V'' by R's scale and the row sums of |T|: the steps between two products are one
//    or two FMAs and the split, and the maxima that the scales need are taken while the tensor
//    cores work.  Operands are handed over in pieces of 16, so that the products of one piece
//    run under the arithmetic of the next.
//  * Warps 8-11 combine and store the outputs, warp 12 issues the MMAs, warp 13 streams the chunks'
//    operands by bulk copies, two chunks deep, warps 14 and 15 transpose the V tiles (a thread of
//    the recurrence reads its column of V as four 16-byte vectors instead of 32 halfwords).
//  * Registers: 128 a thread at launch, moved between the four warpgroups (192, 192, 80, 48).
//  * Tensor memory: S hi 64, S lo 64 (then V'' terms), S K^T 64 (then V'^T), S Q^T 64, (P V')^T 64,
//    dS^T 128 (before it the R terms), V' 32.
//  * Every wait is bounded.  A role whose wait gives up ends its loop after the chunk (no address
//    depends on the data), so the others' waits give up too; the state is not written and the status
//    word is raised.
#include "common.cuh"

namespace bq8 {

static __device__ unsigned int g_gated_delta_status;

unsigned int gated_delta_status_take() {
    unsigned int v = 0, zero = 0;
    cudaDeviceSynchronize();
    cudaMemcpyFromSymbol(&v, g_gated_delta_status, sizeof v);
    cudaMemcpyToSymbol(g_gated_delta_status, &zero, sizeof zero);
    return v;
}

constexpr int GC_C = 64;   // tokens a chunk
constexpr int GC_D = 128;  // head dimension
constexpr float GC_EPS = 1e-6f;
constexpr int GC_MAX_SORT = 384;              // sequences that are ordered by length
// Rows of the new state and of R are scaled as if their largest value were at least this times what stands for
// 1 in the state before: a row that is all zeros beside a large state would otherwise get a scale whose product
// with the state's own leaves fp32, and 0 times that is NaN.  Only rows 2^-115 below the state's bound see it.
constexpr float GC_FLOOR = 0x1p-100f;

// A chunk in the scratch.  Per key head the FP16 rows [K 64; Q 64] in two halves of the head
// dimension (128-byte rows, 128-byte swizzle); per value head T hi, T lo and P (64 x 64 FP16, the same
// swizzle) and the per-token factors.
constexpr uint32_t GC_HALF = 16384;  // K rows 8 KB, Q rows 8 KB
constexpr uint32_t GC_KQ = 2 * GC_HALF;
constexpr uint32_t GC_TILE = 8192;
struct GcScal {
    float beta[GC_C];  // beta_i
    float cr[GC_C];    // beta_i e^(b_i) rk_i
    float ft[GC_C];    // from the accumulated T R to the V' term: tinv_i / pt
    float fv[GC_C];    // to the V'' terms: tinv_i e^(b_C - b_i) rk_i / pd
    float co[GC_C];    // scale rq_i e^(b_i)
    float pinv[GC_C];  // 1 / (power of two of P's row)
    float dec;         // e^(b_C)
    float crmax;       // largest |cr_i|
    float pt, pd;      // powers of two above the row sums of |T|, and above those times e^(b_C - b_i) rk_i
};  // rk_i, rq_i: 1 / norm (or 1) over the power of two of the FP16 row; tinv_i: of T's row
constexpr uint32_t GC_TP_BYTES = 3 * GC_TILE + sizeof(GcScal);
constexpr uint32_t GC_TP = 3 * GC_TILE + 2048;  // stride
static_assert(GC_TP_BYTES <= GC_TP && GC_TP_BYTES % 16 == 0, "scratch block");

// Chunk c of sequence s has the slot cu[s] / 64 + s + c: ceil(len / 64) <= cu[s + 1] / 64 - cu[s] / 64 + 1,
// so no two chunks share one and total / 64 + seqs slots are enough, without a prefix sum.  (Of sequences
// that start below no earlier bound: the others are taken as empty, so that rows and slots have one owner.)
__host__ __device__ __forceinline__ int64_t gc_slots(int64_t seqs, int64_t total) { return total / GC_C + seqs; }

struct GcArgs {
    bq_heads g, beta;
    float* state;
    const int32_t* cu;
    const int32_t* idx;
    uint16_t* out;
    uint8_t* kq;  // [slot][key head][GC_KQ]
    uint8_t* tp;  // [slot][value head][GC_TP]
    int seqs, total, hk, hv, slots;
    float scale;
    int l2norm;
    int parts;  // preparation blocks a (chunk, key head)
    int* ready;  // [slot][value head]; with the preparation before the recurrence the first says whether bounds are out of order
};

// Row bounds of a sequence; invalid ones make it empty.  That it starts below an earlier bound is for the callers
// to find (gc_below).
__device__ __forceinline__ int gc_bounds(const GcArgs& p, int seq, int& start) {
    if (!p.cu) {
        start = 0;
        return p.total;
    }
    start = p.cu[seq];
    const int end = p.cu[seq + 1];
    return (start < 0 || end > p.total || end < start) ? 0 : end - start;
}

// Whether a bound before sequence `seq` lies above its start: every `threads`-th bound from `i` on.  Asked only
// where some bound is below the one before it.
__device__ __forceinline__ bool gc_below(const int* cu, int seq, int start, int i, int threads) {
    bool below = false;
    for (; i < seq; i += threads) below |= cu[i] > start;
    return below;
}

__device__ __forceinline__ int64_t gc_state_slot(const GcArgs& p, int seq) {
    const int64_t s = p.idx ? p.idx[seq] : seq;
    return s < p.slots ? s : -1;  // negative: no state
}

// The first 1024-byte boundary, by an offset from the array: through an integer the compiler would
// lose that these are shared addresses, and every access would be a generic one (the recurrence
// took 1.5 times as long).
__device__ __forceinline__ uint8_t* gc_align(uint8_t* p) { return p + ((0u - smem_u32(p)) & 1023u); }

// A whole warp waits, with one answer for all its lanes.
__device__ __forceinline__ bool gc_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_lean(bar, parity)) != 0;
}

// What one lane of a warp does goes without a branch: the predicate is an operand (a branch costs a
// converged warp about 25 cycles, and the products of a chunk wait for some fifty of these).
__device__ __forceinline__ void gc_arrive_warp(uint64_t* bar) {
    __syncwarp();
    asm volatile(
        "{\n.reg .pred e;\nsetp.eq.u32 e, %1, 0;\n@e mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(smem_u32(bar)),
        "r"(threadIdx.x & 31)
        : "memory");
}

// Arrival on `bar` once the MMAs issued before are done.
__device__ __forceinline__ void gc_commit(uint64_t* bar, uint32_t one) {
    asm volatile(
        "{\n.reg .pred e;\nsetp.ne.u32 e, %1, 0;\n"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
        "r"(one)
        : "memory");
}
__device__ __forceinline__ void gc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void gc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void gc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory descriptor, 128-byte swizzle, 8-row groups of 128-byte rows 1024 bytes apart.
// K-major: rows are N.  MN-major (the K tile as [tokens][head dimension]): rows are K, and `lbo` is the
// distance of the next 64 columns.
__device__ __forceinline__ uint64_t gc_desc(uint32_t addr, uint32_t lbo = 16) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// 1 in one lane of a converged warp.
__device__ __forceinline__ uint32_t gc_elect() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r;
}

// Instruction descriptor: D fp32, A and B FP16, M 128; `tb`: B is MN-major.
__host__ __device__ constexpr uint32_t gc_idesc(int n, int tb) {
    return (1u << 4) | ((uint32_t)tb << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B[smem], K 16, by the lane with `one`.
__device__ __forceinline__ void gc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t one) {
    asm volatile(
        "{\n.reg .pred p, e;\nsetp.ne.u32 p, %3, 0;\nsetp.ne.u32 e, %5, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(acc), "r"(idesc), "r"(one));
}
// D[tmem] (+)= A[smem] * B[smem], K 16, by the lane with `one`.
__device__ __forceinline__ void gc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t one) {
    asm volatile(
        "{\n.reg .pred p, e;\nsetp.ne.u32 p, %3, 0;\nsetp.ne.u32 e, %5, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(acc), "r"(idesc), "r"(one));
}

// 16 accumulator columns of this lane.  The load is asynchronous: the values are there after
// gc_wait16, which waits for every load before it.
__device__ __forceinline__ void gc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void gc_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ float2 gc_pair(const uint32_t (&r)[16], int j) {
    return make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
}

__device__ __forceinline__ void gc_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// The stores before this are done, and the MMAs may read them once `bar` has this warp's arrival.
__device__ __forceinline__ void gc_stored(uint64_t* bar) {
    gc_wait_st();
    gc_fence_before();
    gc_arrive_warp(bar);
}

// A pair's FP16 terms: the values with their low 13 mantissa bits cut off (exact in FP16 while
// normal) and the exact remainder, rounded.  ROUND: the values rounded to nearest and the remainder, for S:
// S Q^T takes the first term alone, and where a query meets its key all its terms have one sign, so a cut
// would shrink the outputs by about 2^-11 (8192 x 48: 340.1 us; 339.2 with the cut, 341.9 with every split
// rounded).
__device__ __forceinline__ uint32_t gc_half2(float2 v) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool ROUND = false>
__device__ __forceinline__ void gc_split(float2 v, uint32_t& hi, uint32_t& lo) {
    float2 h = make_float2(__uint_as_float(__float_as_uint(v.x) & 0xFFFFE000u),
                           __uint_as_float(__float_as_uint(v.y) & 0xFFFFE000u));
    hi = gc_half2(ROUND ? v : h);
    if (ROUND) h = __half22float2(*reinterpret_cast<__half2*>(&hi));
    lo = gc_half2(__ffma2_rn(h, make_float2(-1.0f, -1.0f), v));  // (an FMA: a packed sum has no sign)
}

// The power of two that brings a row with largest magnitude m below 2^15 (from 2^14 on), and its
// inverse; rows below 2^-112 keep the largest scale, 2^126.
__device__ __forceinline__ float gc_pow2(float m, float& inv) {
    const uint32_t e = max(__float_as_uint(m) >> 23, 15u);
    inv = __uint_as_float((e - 14u) << 23);
    return __uint_as_float((268u - e) << 23);
}

// 2^x (relative error below 2^-22).
__device__ __forceinline__ float gc_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (h, l) += (h2, l2), float pairs.
__device__ __forceinline__ void gc_pair_add(float& h, float& l, float h2, float l2) {
    const float s = h + h2, t = s - h;
    const float e = (h - (s - t)) + (h2 - t) + (l + l2);
    h = s + e;
    l = e - (h - s);
}

// 16 bytes of a row of a 64-column FP16 tile with the 128-byte swizzle: columns 8 c .. 8 c + 7.
__device__ __forceinline__ void gc_store_chunk(uint8_t* tile, int row, int c, uint32_t a, uint32_t b, uint32_t d, uint32_t e) {
    *reinterpret_cast<uint4*>(tile + row * 128 + ((c ^ (row & 7)) << 4)) = make_uint4(a, b, d, e);
}

// acc += a[0..3] * (rows b, b + ld, ...)[4 columns]
__device__ __forceinline__ void gp_mul4(float2 (&acc)[2], float4 a, const float* b, int ld) {
    const float u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float4 t = *reinterpret_cast<const float4*>(b + j * ld);
        acc[0] = __ffma2_rn(make_float2(u[j], u[j]), make_float2(t.x, t.y), acc[0]);
        acc[1] = __ffma2_rn(make_float2(u[j], u[j]), make_float2(t.z, t.w), acc[1]);
    }
}
__device__ __forceinline__ void gp_put4(float* at, const float2 (&acc)[2], float sign) {
    *reinterpret_cast<float4*>(at) = make_float4(sign * acc[0].x, sign * acc[0].y, sign * acc[1].x, sign * acc[1].y);
}

// The power of two above m > 0 (m below it), and its inverse.
__device__ __forceinline__ float gp_pow2_above(float m, float& inv) {
    const uint32_t e = min(max(__float_as_uint(m) >> 23, 1u), 252u) + 1u;
    inv = __uint_as_float((254u - e) << 23);
    return __uint_as_float(e << 23);
}

// Bulk copy shared -> global, and the waits of the thread that issued it: until the source may be
// overwritten, until the bytes are in memory.
__device__ __forceinline__ void gp_bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\ncp.async.bulk.commit_group;" ::"l"(
                     reinterpret_cast<uint64_t>(dst)),
                 "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void gp_bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void gp_bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ======================================================================================= prepare
constexpr int GP_LD = 68;   // row strides (floats) of the fp32 matrices
constexpr int GP_LX = 36;
constexpr int GP_HEADS = 4;  // value heads whose decays are formed at once, one a warp
struct GpMat {  // over the [K; Q] tile, once its product is done
    float T[GC_C][GP_LD];  // A, then block by block its inverse
    float X[32][GP_LX];
};
struct GpHead {
    float bh[GC_C], bl[GC_C];  // b in log2 units, high and low part
    float beta[GC_C];
    float grow[GC_C];          // largest b_i - b_j, j <= i, rounded up (0 unless some g is positive)
};
struct GpShared {
    GpHead head[GP_HEADS];
    float rk[GC_C], fk[GC_C], cr[GC_C], cv[GC_C], tinv[GC_C], tsum[GC_C];
    uint64_t full, kqdone;
    uint32_t tslot;
    int seq;
};
static_assert(sizeof(GpMat) <= GC_KQ, "the matrices lie over the tile");
constexpr size_t GP_SMEM = 1024 + GC_KQ + sizeof(GpShared);
constexpr uint32_t GP_COLS = 64;  // tensor-memory columns: [K; Q] K^T

// The 128 threads of a preparation meet, on a barrier of their own.
__device__ __forceinline__ void gp_sync(int bar) { asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory"); }
__device__ __forceinline__ bool gp_vote(int bar, bool ok) {  // true if it is for all of them
    uint32_t all;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.and.pred q, %2, 128, p;\nselp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(all)
        : "r"((uint32_t)ok), "r"(bar)
        : "memory");
    return all != 0;
}

// 128 threads prepare a (chunk, key head) for `heads` of its value heads from head0 on: norms, the FP16
// rows (sent to `kq` unless it is null), [K; Q] K^T, then for each of the value heads the decays, A
// and P, the inverse T by blocks of 16 (CUDA cores, fp32) and the terms.  Threads 0-63 own the rows of
// K (and A), 64-127 those of Q (and P).  False if a wait gave up.
__device__ __forceinline__ bool gp_chunk(const CUtensorMap* mapQ, const CUtensorMap* mapK, const GcArgs& p, uint8_t* tile,
                                         GpShared& sh, uint32_t tb, int bar, uint32_t parity, int64_t slot, int64_t t0,
                                         int live_rows, int kh, int head0, int heads, uint8_t* kq) {
    GpMat& mat = *reinterpret_cast<GpMat*>(tile);
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5) & 3, 0);
    const int pt = threadIdx.x & 127, row = pt & 63;
    if (pt == 0) {
        mbar_arrive_expect_tx(&sh.full, GC_KQ);
        for (int h = 0; h < 2; h++) {
            tma_load_3d(tile + h * GC_HALF, mapK, 64 * h, kh, (int)t0, &sh.full);
            tma_load_3d(tile + h * GC_HALF + 8192, mapQ, 64 * h, kh, (int)t0, &sh.full);
        }
    }
    // decay and write strength of two tokens, of the value head e + warp
    float gate[2], be2[2];
    auto load_gates = [&](int e) {
        const float* gp = (const float*)p.g.data + (head0 + e + warp) * p.g.head_stride;
        const float* bp = (const float*)p.beta.data + (head0 + e + warp) * p.beta.head_stride;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const bool in = 2 * lane + i < live_rows && e + warp < heads;
            gate[i] = in ? gp[(t0 + 2 * lane + i) * p.g.token_stride] : 0.0f;
            be2[i] = in ? bp[(t0 + 2 * lane + i) * p.beta.token_stride] : 0.0f;
        }
    };
    load_gates(0);  // (on their way while the rows come)
    bool ok = gc_wait(&sh.full, parity);

    // ---- this row of K or Q: norm, then FP16 in place, scaled by a power of two to below 2^8.  Rows
    // past the sequence's end belong to the next one (or to nothing): zeros.
    float rn = 1.0f;
    {
        uint8_t* at = tile + pt * 128;
        const bool in = row < live_rows;
        const int x7 = row & 7;
        float m = 0.0f;  // a bound on the row: its norm, or its largest magnitude
        bool by_max = !p.l2norm;
        if (p.l2norm) {
            float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll 4
            for (int x = 0; x < 16; x++) {
                const uint4 w = *reinterpret_cast<const uint4*>(at + (x >> 3) * GC_HALF + (((x & 7) ^ x7) << 4));
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 f = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
                    acc[i & 1] = __ffma2_rn(f, f, acc[i & 1]);
                }
            }
            const float2 a = __fadd2_rn(acc[0], acc[1]);
            const float ss = in ? a.x + a.y : 0.0f;
            rn = __fdiv_rn(1.0f, __fsqrt_rn(ss + GC_EPS));
            m = __fsqrt_rn(ss);
            by_max = in && ss < 0x1p-100f;  // squares that underflow say nothing about the values
        }
        if (by_max) {
            uint32_t a = 0, b = 0;  // largest magnitudes of the even and odd values, as bit patterns
#pragma unroll 4
            for (int x = 0; x < 16; x++) {
                const uint4 w = *reinterpret_cast<const uint4*>(at + (x >> 3) * GC_HALF + (((x & 7) ^ x7) << 4));
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    a = max(a, u[i] & 0x7FFF0000u);
                    b = max(b, (u[i] << 16) & 0x7FFF0000u);
                }
            }
            // (a norm of 128 values is below 12 times the largest)
            m = in ? __uint_as_float(max(a, b)) * (p.l2norm ? 12.0f : 1.0f) : 0.0f;
        }
        const uint32_t e = max(__float_as_uint(m) >> 23, 8u);
        const float sc = __uint_as_float((261u - e) << 23);
        rn *= __uint_as_float((e - 7u) << 23);
#pragma unroll 4
        for (int x = 0; x < 16; x++) {
            uint4* const w = reinterpret_cast<uint4*>(at + (x >> 3) * GC_HALF + (((x & 7) ^ x7) << 4));
            uint32_t u[4] = {w->x, w->y, w->z, w->w};
#pragma unroll
            for (int i = 0; i < 4; i++)
                u[i] = in ? gc_half2(__fmul2_rn(make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u)),
                                                make_float2(sc, sc)))
                          : 0u;
            *w = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
    if (pt < GC_C) sh.rk[row] = rn;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    ok = gp_vote(bar, ok);
    if (warp == 0 && ok) {
        gc_fence_after();
        const uint32_t s = __shfl_sync(0xffffffffu, smem_u32(tile), 0), one = gc_elect();
#pragma unroll
        for (int x = 0; x < 8; x++) {
            const uint64_t d = gc_desc(s + (x >> 2) * GC_HALF + 32 * (x & 3));
            gc_mma_ss(tb, d, d, gc_idesc(64, 0), x != 0, one);
        }
        gc_commit(&sh.kqdone, one);
        if (one && kq) {
            gp_bulk_store(kq, tile, GC_KQ);
            gp_bulk_wait_read();  // the tile may be overwritten
        }
        __syncwarp();
        ok = gc_wait(&sh.kqdone, parity);
    }
    ok = gp_vote(bar, ok);
    gc_fence_after();

    // |q . k| of the FP16 rows: norms below 2^8 each, or values below 2^8
    const float qkbound = p.l2norm ? 65536.0f : 8388608.0f;
    for (int e = 0; e < heads && ok; e++) {
        const int head = head0 + e;
        uint8_t* tT = p.tp + (slot * p.hv + head) * GC_TP;
        uint8_t* tP = tT + 2 * GC_TILE;
        GcScal& sc = *reinterpret_cast<GcScal*>(tT + 3 * GC_TILE);
        GpHead& hd = sh.head[e % GP_HEADS];
        // ---- decays of the next four heads, one a warp
        if (e % GP_HEADS == 0 && e + warp < heads) {
            float h[2], l[2];
            if (e > 0) load_gates(e);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const float g = gate[i];
                // log2 units; below -200 the factor is 0 in fp32 either way (this also bounds -infinity)
                const float x = g < -200.0f ? -200.0f : g;
                const float m = x * 1.44269502f;
                l[i] = fmaf(x, 1.92596303e-8f, fmaf(x, 1.44269502f, -m));
                h[i] = m;
            }
            gc_pair_add(h[1], l[1], h[0], l[0]);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float hn = __shfl_up_sync(0xffffffffu, h[1], o), ln = __shfl_up_sync(0xffffffffu, l[1], o);
                if (lane >= o) gc_pair_add(h[1], l[1], hn, ln);
            }
            const float hp = __shfl_up_sync(0xffffffffu, h[1], 1), lp = __shfl_up_sync(0xffffffffu, l[1], 1);
            if (lane > 0) gc_pair_add(h[0], l[0], hp, lp);
            float low = fminf(h[0], h[1]), before = __int_as_float(0x7f800000);  // smallest b so far
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, low, o);
                if (lane >= o) low = fminf(low, x);
            }
            before = __shfl_up_sync(0xffffffffu, low, 1);
            if (lane == 0) before = h[0];
            GpHead& o = sh.head[warp];
            *reinterpret_cast<float2*>(&o.bh[2 * lane]) = make_float2(h[0], h[1]);
            *reinterpret_cast<float2*>(&o.bl[2 * lane]) = make_float2(l[0], l[1]);
            *reinterpret_cast<float2*>(&o.beta[2 * lane]) = make_float2(be2[0], be2[1]);
            *reinterpret_cast<float2*>(&o.grow[2 * lane]) =
                make_float2(ceilf(h[0] - fminf(before, h[0])), ceilf(h[1] - fminf(low, h[1])));
        }
        if (e % GP_HEADS == 0) gp_sync(bar);
        const float bh = hd.bh[row], bl = hd.bl[row], beta = hd.beta[row];
        {
            const float eb = gc_exp2(bh + bl), ec = gc_exp2((hd.bh[63] - bh) + (hd.bl[63] - bl));
            if (pt < GC_C) {
                sc.beta[row] = beta;
                sc.cr[row] = sh.cr[row] = beta * eb * rn;
                sh.cv[row] = ec * rn;
                sh.fk[row] = gc_exp2((hd.bh[row | 15] - bh) + (hd.bl[row | 15] - bl)) * rn;
                if (row == 63) sc.dec = eb;
            } else {
                sc.co[row] = eb * rn * p.scale;
            }
        }
        gp_sync(bar);
        // ---- A (rows of K) and P (rows of Q) from [K; Q] K^T.  A block of 16 columns left of the row's
        // own: e^(b_i - b_j) = e^(b_i - m) e^(m - b_j), m the block's last b, neither above 1 (where no g
        // is positive).  P's row is scaled by a bound on it.
        {
            float mine = pt < GC_C ? beta * rn : rn * p.scale;
            if (pt >= GC_C) {
                float kmax = fmaxf(sh.rk[lane], sh.rk[lane + 32]), inv;
                kmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(kmax)));
                const float s = gc_pow2(fabsf(mine) * (kmax * qkbound) * gc_exp2(hd.grow[row]), inv);
                sc.pinv[row] = inv;
                mine *= s;
            }
            const int own = warp & 1;  // rows 32 own .. : columns 32 own .. + 31 hold the diagonal
            const int last = row - (pt < GC_C ? 1 : 0);  // largest column that is kept
            const uint32_t tr = tb + ((uint32_t)(32 * warp) << 16);
#pragma unroll 1
            for (int b = 0; b < 4; b++) {
                float2 v[8];
                if (b < 2 * own + 2) {
                    uint32_t r[16];
                    gc_ld16(tr + 16 * b, r);
                    gc_wait16(r);
                    if (b < 2 * own) {
                        const float eb = gc_exp2((bh - hd.bh[16 * b + 15]) + (bl - hd.bl[16 * b + 15])) * mine;
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            v[j] = __fmul2_rn(gc_pair(r, j), __fmul2_rn(*reinterpret_cast<const float2*>(&sh.fk[16 * b + 2 * j]), make_float2(eb, eb)));
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            const int col = 16 * b + 2 * j;
                            const float2 fh = *reinterpret_cast<const float2*>(&hd.bh[col]);
                            const float2 fl = *reinterpret_cast<const float2*>(&hd.bl[col]);
                            const float2 fr = *reinterpret_cast<const float2*>(&sh.rk[col]);
                            const float2 one = make_float2(-1.0f, -1.0f);
                            const float2 d = __fadd2_rn(__ffma2_rn(fh, one, make_float2(bh, bh)), __ffma2_rn(fl, one, make_float2(bl, bl)));
                            v[j] = __fmul2_rn(gc_pair(r, j), __fmul2_rn(__fmul2_rn(fr, make_float2(mine, mine)), make_float2(gc_exp2(d.x), gc_exp2(d.y))));
                            if (col > last) v[j].x = 0.0f;
                            if (col + 1 > last) v[j].y = 0.0f;
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j++) v[j] = make_float2(0.0f, 0.0f);
                }
                if (pt >= GC_C) {
                    // neighbouring lanes exchange, so that the two of them fill a 32-byte sector: first of the
                    // even lane's row, then of the odd one's
                    const bool odd = lane & 1;
                    uint32_t f[4], g[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const uint32_t c0 = gc_half2(v[j]), c1 = gc_half2(v[4 + j]);
                        const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? c0 : c1, 1);
                        f[j] = odd ? other : c0;
                        g[j] = odd ? c1 : other;
                    }
                    gc_store_chunk(tP, row & ~1, 2 * b + odd, f[0], f[1], f[2], f[3]);
                    gc_store_chunk(tP, row | 1, 2 * b + odd, g[0], g[1], g[2], g[3]);
                } else if (b < 2 * own + 2) {
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        *reinterpret_cast<float4*>(&mat.T[row][16 * b + 4 * j]) =
                            make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
                }
            }
        }
        if (pt < GC_C) {
            __syncwarp();
            // ---- T = (I + A)^-1, in place.  Diagonal blocks of 16 by substitution, one column a thread
            // (both blocks of a warp's rows are its own)
            const int base = row & ~15, col = row & 15;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; i++) {
                float s[4] = {i == col ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int l = 0; l < i; l += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(&mat.T[base + i][base + l]);
                    s[0] = fmaf(-a.x, x[l], s[0]);
                    if (l + 1 < i) s[1] = fmaf(-a.y, x[l + 1], s[1]);
                    if (l + 2 < i) s[2] = fmaf(-a.z, x[l + 2], s[2]);
                    if (l + 3 < i) s[3] = fmaf(-a.w, x[l + 3], s[3]);
                }
                x[i] = (s[0] + s[1]) + (s[2] + s[3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; i++) mat.T[base + i][base + col] = x[i];
        }
        gp_sync(bar);
        // the 16 x 16 blocks below the diagonal inside each half: T21 = -T22 (A21 T11); a warp's products
        // of X rows 16 h .. and columns are its own pair of warps'
        {
            const int o = 32 * (pt >> 6), r = (pt & 63) >> 2, cc = 4 * (pt & 3);
            float2 acc[2] = {make_float2(0, 0), make_float2(0, 0)};
#pragma unroll
            for (int k = 0; k < 16; k += 4) gp_mul4(acc, *reinterpret_cast<const float4*>(&mat.T[o + 16 + r][o + k]), &mat.T[o + k][o + cc], GP_LD);
            gp_put4(&mat.X[(o >> 1) + r][cc], acc, 1.0f);
            gp_sync(bar);
            acc[0] = acc[1] = make_float2(0, 0);
#pragma unroll
            for (int k = 0; k < 16; k += 4)
                gp_mul4(acc, *reinterpret_cast<const float4*>(&mat.T[o + 16 + r][o + 16 + k]), &mat.X[(o >> 1) + k][cc], GP_LX);
            gp_put4(&mat.T[o + 16 + r][o + cc], acc, -1.0f);
        }
        gp_sync(bar);
        // the 32 x 32 block: the same with halves (the zero quarter of each triangle is skipped)
        {
            const int r = 2 * (pt >> 3), cc = 4 * (pt & 7);
            float2 a0[2] = {make_float2(0, 0), make_float2(0, 0)}, a1[2] = {make_float2(0, 0), make_float2(0, 0)};
#pragma unroll 2
            for (int k = cc & 16; k < 32; k += 4) {  // T11's columns 16-31 start at row 16
                gp_mul4(a0, *reinterpret_cast<const float4*>(&mat.T[32 + r][k]), &mat.T[k][cc], GP_LD);
                gp_mul4(a1, *reinterpret_cast<const float4*>(&mat.T[33 + r][k]), &mat.T[k][cc], GP_LD);
            }
            gp_put4(&mat.X[r][cc], a0, 1.0f);
            gp_put4(&mat.X[r + 1][cc], a1, 1.0f);
            gp_sync(bar);
            a0[0] = a0[1] = a1[0] = a1[1] = make_float2(0, 0);
            const int kend = r < 16 ? 16 : 32;  // T22's rows 0-15 end at column 15
#pragma unroll 2
            for (int k = 0; k < kend; k += 4) {
                gp_mul4(a0, *reinterpret_cast<const float4*>(&mat.T[32 + r][32 + k]), &mat.X[k][cc], GP_LX);
                gp_mul4(a1, *reinterpret_cast<const float4*>(&mat.T[33 + r][32 + k]), &mat.X[k][cc], GP_LX);
            }
            gp_put4(&mat.T[32 + r][cc], a0, -1.0f);
            gp_put4(&mat.T[33 + r][cc], a1, -1.0f);
        }
        gp_sync(bar);
        // the terms of T, every other 16 bytes of a row a thread, so that two lanes fill a 32-byte sector
        // (blocks above the diagonal still hold anything)
        {
            const int r = pt >> 1, h = pt & 1;
            float sum = 0.0f, inv;  // the row sum of |T| bounds its largest as well
#pragma unroll
            for (int b = 0; b < 8; b++) {
                const int col = 16 * (b >> 1) + 8 * h + 4 * (b & 1);
                if (col <= (r | 15)) {
                    const float4 t = *reinterpret_cast<const float4*>(&mat.T[r][col]);
                    sum += (fabsf(t.x) + fabsf(t.y)) + (fabsf(t.z) + fabsf(t.w));
                }
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            const float s = gc_pow2(sum, inv);
            if (h == 0) {
                sh.tinv[r] = inv;
                sh.tsum[r] = sum;
            }
#pragma unroll
            for (int b = 0; b < 4; b++) {
                uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
                if (16 * b <= (r | 15)) {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        gc_split(__fmul2_rn(*reinterpret_cast<const float2*>(&mat.T[r][16 * b + 8 * h + 2 * i]), make_float2(s, s)), hi[i], lo[i]);
                }
                gc_store_chunk(tT, r, 2 * b + h, hi[0], hi[1], hi[2], hi[3]);
                gc_store_chunk(tT + GC_TILE, r, 2 * b + h, lo[0], lo[1], lo[2], lo[3]);
            }
        }
        gp_sync(bar);
        // the factors that need all rows (the others go on to the next head: what this reads is
        // written again only past barriers that this warp takes part in)
        if (warp == 3) {
            float pt2 = 0.0f, pd = 0.0f, cr = 0.0f;
#pragma unroll
            for (int i = lane; i < GC_C; i += 32) {
                pt2 = fmaxf(pt2, sh.tsum[i]);
                pd = fmaxf(pd, sh.tsum[i] * sh.cv[i]);
                cr = fmaxf(cr, fabsf(sh.cr[i]));
            }
            float ipt, ipd;
            pt2 = gp_pow2_above(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(pt2))), ipt);
            pd = gp_pow2_above(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(pd))), ipd);
            cr = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(cr)));
#pragma unroll
            for (int i = lane; i < GC_C; i += 32) {
                sc.ft[i] = sh.tinv[i] * ipt;
                sc.fv[i] = sh.tinv[i] * (sh.cv[i] * ipd);
            }
            if (lane == 0) {
                sc.crmax = cr;
                sc.pt = pt2;
                sc.pd = pd;
            }
        }
        gp_sync(bar);
    }
    if (warp == 0) gp_bulk_wait();  // the rows have reached the scratch (if they were sent)
    gc_fence_before();
    return ok;
}

// Preparation of its own: `parts` blocks a (chunk, key head), each for its share of the value heads.
// Five blocks an SM hide each other's latencies.
__global__ void __launch_bounds__(128, 5)
    gated_delta_prepare_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                               const GcArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* tile = gc_align(smem_raw);
    GpShared& sh = *reinterpret_cast<GpShared*>(tile + GC_KQ);
    const int part = blockIdx.x % p.parts, kh = blockIdx.x / p.parts % p.hk;
    const int64_t slot = blockIdx.x / (p.parts * p.hk);
    const int group = p.hv / p.hk, each = (group + p.parts - 1) / p.parts;  // value heads of a key head, of a block

    // whose chunk this is
    pdl_wait();
    if (threadIdx.x == 0) {
        sh.seq = p.seqs;
        mbar_init(&sh.full, 1);
        mbar_init(&sh.kqdone, 1);
        fence_barrier_init();
    }
    __syncthreads();
    bool disordered = false;
    for (int s = threadIdx.x; s < p.seqs; s += 128) {
        int start;
        const int len = gc_bounds(p, s, start);
        if (p.cu) disordered |= p.cu[s + 1] < start;
        const int64_t base = start / GC_C + s;
        if (slot >= base && slot < base + (len + GC_C - 1) / GC_C && gc_state_slot(p, s) >= 0)
            atomicMin(&sh.seq, s);  // (a later one with this slot starts below this one's end)
    }
    disordered = __syncthreads_or(disordered);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.ready[0] = disordered;
    const int seq = sh.seq;
    if (seq == p.seqs) return;
    int start;
    const int len = gc_bounds(p, seq, start);
    if (disordered && __syncthreads_or(gc_below(p.cu, seq, start, threadIdx.x, 128))) return;
    const int c = (int)(slot - (start / GC_C + seq));
    if (threadIdx.x < 32) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tslot)),
                     "n"(GP_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        pdl_launch_dependents();  // the recurrence's CTAs take all of the tensor memory: not before this has its own
    }
    gc_fence_before();
    __syncthreads();
    gc_fence_after();
    const uint32_t tb = __shfl_sync(0xffffffffu, sh.tslot, 0);
    if (!gp_chunk(&mapQ, &mapK, p, tile, sh, tb, 0, 0, slot, (int64_t)start + GC_C * c, min(GC_C, len - GC_C * c), kh,
                  kh * group + part * each, min(each, group - part * each),
                  part == 0 ? p.kq + (slot * p.hk + kh) * GC_KQ : nullptr) &&
        threadIdx.x == 0)
        atomicOr(&g_gated_delta_status, 1u);
    __syncthreads();
    if (threadIdx.x < 32) {
        gc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tb), "n"(GP_COLS));
    }
}

// ===================================================================================== recurrence
constexpr int GC_WOUT = 8, GC_WMMA = 12, GC_WTMA = 13;  // first warps of the roles
constexpr int GC_THREADS = 512;
constexpr int GC_REGS = 128;  // registers a thread at launch; the four shares below add up to 4 x this
constexpr int GC_REGS_S = 192, GC_REGS_OUT = 80, GC_REGS_MMA = 48;
static_assert(2 * GC_REGS_S + GC_REGS_OUT + GC_REGS_MMA == 4 * GC_REGS, "register shares");

// Tensor-memory columns.
constexpr uint32_t TC_SHI = 0;    // S^T hi
constexpr uint32_t TC_SLO = 64;   // S^T lo, then the V''^T terms (hi 64, lo 96)
constexpr uint32_t TC_KS = 128;   // S K^T, then V'^T
constexpr uint32_t TC_QS = 192;   // S Q^T
constexpr uint32_t TC_PV = 256;   // (P V')^T
constexpr uint32_t TC_DS = 320;   // dS^T (before it the R^T terms: hi 320, lo 352)
constexpr uint32_t TC_V = 448;    // V'^T, one term

// Shared memory: two stages of the MMAs' operands, [K; Q], T and P; two of V as it comes (64 tokens x two
// halves of 64 columns, 128-byte swizzle) and two of V^T (a 128-byte row of 64 tokens a value
// column, the same swizzle); the factors, four deep (the outputs read them up to a chunk later).
constexpr uint32_t GC_T = GC_KQ;
constexpr uint32_t GC_P = GC_T + 2 * GC_TILE;
constexpr uint32_t GC_STAGE = GC_P + GC_TILE;
constexpr uint32_t GC_VTILE = 16384;
static_assert(GC_STAGE % 1024 == 0, "swizzled tiles start on 1024 bytes");
struct GcShared {
    GcScal scal[4];
    float sinv[4][GC_D];      // 1 / (power of two of S's row); by chunk, as the outputs read it up to two later
    float vinv[4][GC_D];      // the same of V'
    float smax[2][2][GC_D];   // by chunk parity and warp half: largest |S| of the row's half,
    float dmax[2][2][GC_D];   // bound on the row of dS from the half's tokens,
    float vmax[2][2][GC_D];   // largest |beta v| of the half's tokens
    uint64_t ldfull[2], ldempty[2], vld[4], vtfull[2], vtempty[2], sfull[4], ksfull, rfull[2], d2full, vfull[2], bounds, dsfull, ofull, ofree, done;
    uint32_t tslot;
    int failed;
    int seq;
    int len[GC_MAX_SORT];  // where chunks are prepared 0 for a sequence that starts below an earlier bound
};
constexpr size_t GC_SMEM = 1024 + 2 * GC_STAGE + 4 * GC_VTILE + sizeof(GcShared);
static_assert(GC_SMEM <= 227 * 1024, "shared memory budget");

// Preparation beside the recurrence: four teams of 128 threads in a CTA of its own, a tile each.
constexpr uint32_t GP_TEAM = GC_KQ + (sizeof(GpShared) + 1023) / 1024 * 1024;
static_assert(4 * GP_TEAM <= 2 * GC_STAGE + 4 * GC_VTILE, "four teams lie below the barriers");

// The flag of a (chunk slot, value head): set once its terms are in the scratch.
__device__ __forceinline__ int* gc_ready(const GcArgs& p, int64_t slot, int head) { return p.ready + slot * p.hv + head; }

// Waits for a flag (bounded); what was written before it may then be copied by the asynchronous proxy.
__device__ __forceinline__ bool gc_wait_ready(const int* flag) {
#pragma unroll 1
    for (uint32_t it = 0; it < (1u << 22); it++) {
        int v;
        asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v) {
            asm volatile("fence.proxy.async;" ::: "memory");
            return true;
        }
    }
    return false;
}

// The chunks of all sequences, first chunks first, a value head at a time; `tb` and `smem` the CTA's.
__device__ __forceinline__ bool gp_teams(const CUtensorMap* mapQ, const CUtensorMap* mapK, const GcArgs& p, uint8_t* smem,
                                         uint32_t tb, int first, int workers, const int* lens) {
    const int team = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 7), 0), bar = 1 + team;
    uint8_t* tile = smem + team * GP_TEAM;
    GpShared& sh = *reinterpret_cast<GpShared*>(tile + GC_KQ);
    if ((threadIdx.x & 127) == 0) {
        mbar_init(&sh.full, 1);
        mbar_init(&sh.kqdone, 1);
        fence_barrier_init();
    }
    gp_sync(bar);
    const int group = p.hv / p.hk;
    // (the lengths of several sequences with those that start below an earlier bound as 0)
    auto bounds = [&](int s, int& start) {
        const int len = gc_bounds(p, s, start);
        return p.seqs > 1 ? min(len, lens[s]) : len;
    };
    int most = 0;
    for (int s = 0; s < p.seqs; s++) {
        int start;
        most = max(most, (bounds(s, start) + GC_C - 1) / GC_C);
    }
    const int64_t items = (int64_t)most * p.seqs * p.hv;
    uint32_t parity = 0;
    for (int64_t i = first + (int64_t)team * workers; i < items; i += 4 * (int64_t)workers) {
        const int head = (int)(i % p.hv), seq = (int)(i / p.hv % p.seqs), c = (int)(i / p.hv / p.seqs);
        int start;
        const int len = bounds(seq, start);
        if (GC_C * c >= len || gc_state_slot(p, seq) < 0) continue;
        const int64_t slot = start / GC_C + seq + c;
        const int kh = head / group;
        if (!gp_chunk(mapQ, mapK, p, tile, sh, tb + GP_COLS * team, bar, parity, slot, (int64_t)start + GC_C * c,
                      min(GC_C, len - GC_C * c), kh, head, 1, head % group == 0 ? p.kq + (slot * p.hk + kh) * GC_KQ : nullptr))
            return false;
        parity ^= 1u;
        // every thread's terms, then the flag; the tile may be filled again
        asm volatile("fence.proxy.async;" ::: "memory");
        gp_sync(bar);
        if ((threadIdx.x & 127) == 0) {
            __threadfence();
            asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(gc_ready(p, slot, head)), "r"(1) : "memory");
        }
    }
    return true;
}

// AHEAD: the preparation is done beside the recurrence, by the CTAs from seqs x value heads on (all
// CTAs run at once: one an SM), chunk by chunk ahead of it.
template <bool AHEAD>
__global__ void __launch_bounds__(GC_THREADS, 1)
    gated_delta_recur_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                             const __grid_constant__ CUtensorMap mapV, const GcArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = gc_align(smem_raw);
    uint8_t* vtiles = stages + 2 * GC_STAGE;  // V of even and odd chunks, then V^T
    GcShared& sh = *reinterpret_cast<GcShared*>(vtiles + 4 * GC_VTILE);
    const GcScal* scals = sh.scal;

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);  // uniform
    const int head = blockIdx.x % p.hv, kh = head / (p.hv / p.hk);
    const int order = blockIdx.x / p.hv;
    const bool prepares = AHEAD && order >= p.seqs;

    if (threadIdx.x == 0) {
        sh.seq = order;
        sh.failed = 0;
        for (int s = 0; s < 2; s++) {
            mbar_init(&sh.ldfull[s], 1);
            mbar_init(&sh.ldempty[s], 1);
            mbar_init(&sh.rfull[s], 8);
            mbar_init(&sh.vfull[s], 8);
            mbar_init(&sh.vtfull[s], 2);
            mbar_init(&sh.vtempty[s], 8);
        }
        for (int s = 0; s < 4; s++) mbar_init(&sh.sfull[s], 8);
        for (int s = 0; s < 4; s++) mbar_init(&sh.vld[s], 1);
        mbar_init(&sh.bounds, 8);
        mbar_init(&sh.ksfull, 1);
        mbar_init(&sh.d2full, 1);
        mbar_init(&sh.dsfull, 1);
        mbar_init(&sh.ofull, 1);
        mbar_init(&sh.ofree, 4);
        mbar_init(&sh.done, 1);
        fence_barrier_init();
    }
    if (warp == GC_WMMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tslot)), "n"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();  // (returns at once where the launch is not programmatic)
    gc_fence_before();
    __syncthreads();
    gc_fence_after();
    // The longest sequences start first: a CTA takes the sequence of rank `order` by length.
    bool disordered = !AHEAD && p.ready[0];  // (some bound is below the one before it)
    if (p.seqs > 1 && p.seqs <= GC_MAX_SORT) {
        const int i = threadIdx.x;
        bool below = false;
        if (i < p.seqs) {
            const int len = p.cu[i + 1] - p.cu[i];
            sh.len[i] = len;
            below = len < 0;
        }
        if (AHEAD) disordered = __syncthreads_or(below);  // (at most half as many sequences as SMs)
        else __syncthreads();
        if (prepares) {
            if (disordered && i < p.seqs && gc_below(p.cu, i, p.cu[i], 0, 1)) sh.len[i] = 0;
        } else if (i < p.seqs) {
            const int len = sh.len[i];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < p.seqs; j++) {
                const int lj = sh.len[j];
                rank += lj > len || (lj == len && j < i);
            }
            if (rank == order) sh.seq = i;
        }
        __syncthreads();
    }
    const int seq = prepares ? 0 : sh.seq;
    const uint32_t tb = __shfl_sync(0xffffffffu, sh.tslot, 0), su = __shfl_sync(0xffffffffu, smem_u32(stages), 0);
    int start;
    const int len = gc_bounds(p, seq, start);
    const int64_t slot = gc_state_slot(p, seq);
    const int n = slot >= 0 ? (len + GC_C - 1) / GC_C : 0;  // chunks
    const bool empty = disordered && __syncthreads_or(!prepares && gc_below(p.cu, seq, start, threadIdx.x, GC_THREADS));
    if (slot < 0 && len > 0 && !prepares && !empty) {       // no state: the outputs are zero
        uint4* row = reinterpret_cast<uint4*>(p.out + ((int64_t)start * p.hv + head) * GC_D) + threadIdx.x % (GC_D / 8);
        for (int i = threadIdx.x / (GC_D / 8); i < len; i += GC_THREADS / (GC_D / 8))  // (16 threads a row)
            row[(int64_t)i * p.hv * (GC_D / 8)] = make_uint4(0, 0, 0, 0);
    }

    if (prepares) {
        if (!gp_teams(&mapQ, &mapK, p, stages, tb, (int)blockIdx.x - p.seqs * p.hv, (int)gridDim.x - p.seqs * p.hv, sh.len)) sh.failed = 1;
    } else if (n == 0 || empty) {
        // nothing to do: the state stays as it is
    } else if (warp < GC_WOUT) {
        // ================================================================ the recurrence
        // Warp half hf holds key dimensions 64 hf .. + 63 of the state and takes tokens 32 hf .. + 31 of
        // R and V'.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(GC_REGS_S));
        const int hf = warp >> 2, dv = 32 * (warp & 3) + lane;
        const uint32_t tq = tb + ((uint32_t)(32 * (warp & 3)) << 16);
        // |S k| over the powers of two: |S| < 2^15 and 128 values; |k| < 2^8, as a whole row where
        // the norm scales it, as a value where the largest does
        const float kbound = p.l2norm ? 134217728.0f : 1073741824.0f;
        float* st = p.state + ((slot * p.hv + head) * GC_D + 64 * hf) * GC_D + dv;
        float2 S[32];   // the state times a power of two of this row, 1 / inv
        float2 bv[16];  // beta v of the chunk to come, then the same times R's power of two
        float inv = 1.0f, most = 0.0f, dinv = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; j++) S[j] = make_float2(__ldcs(st + 2 * j * GC_D), __ldcs(st + (2 * j + 1) * GC_D));
        {
            float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; j++) {
                m0 = fmaxf(m0, fabsf(S[j].x));
                m1 = fmaxf(m1, fabsf(S[j].y));
            }
            sh.smax[1][hf][dv] = fmaxf(m0, m1);  // as chunk -1 would
        }
        bool ok = true;
        for (int c = -1; c <= n && ok; c++) {
            const uint32_t par = (uint32_t)c & 1u, prev = par ^ 1u;
            const GcScal& sc = scals[c & 3];
            if (c >= 0) {
                // ---- S <- e^(b_C) S + dS of the chunk before, scaled by a bound on the new row
                ok &= gc_wait(&sh.bounds, par);
                const float old = inv;
                most = fmaxf(sh.smax[prev][0][dv], sh.smax[prev][1][dv]);
                float a = 1.0f, b = 0.0f;
                if (c > 0) {
                    const float dec = scals[(c - 1) & 3].dec;
                    most = fmaxf(fmaf(most, dec, sh.dmax[prev][0][dv] + sh.dmax[prev][1][dv]), old * GC_FLOOR);
                    a = dec * old;  // (before the new scale: dec may be zero and s * old above fp32)
                }
                float s = gc_pow2(most, inv);
                a *= s;
                b = dinv * s;
                const float2 a2 = make_float2(a, a), b2 = make_float2(b, b);
                if (hf == 0) sh.sinv[c & 3][dv] = inv;
                if (c > 0) {
                    ok &= gc_wait(&sh.dsfull, prev);
                    gc_fence_after();
                }
                // pieces of 16 columns: the next piece's load and this one's stores run under the arithmetic
                uint32_t d[2][16];
                if (c > 0) gc_ld16(tq + TC_DS + 64 * hf, d[0]);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    if (c > 0) {
                        gc_wait16(d[e & 1]);
                        if (e < 3) gc_ld16(tq + TC_DS + 64 * hf + 16 * (e + 1), d[(e + 1) & 1]);
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            S[8 * e + j] = __ffma2_rn(S[8 * e + j], a2, __fmul2_rn(gc_pair(d[e & 1], j), b2));
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; j++) S[8 * e + j] = __fmul2_rn(S[8 * e + j], a2);
                    }
                    if (c < n) {
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int j = 0; j < 8; j++) gc_split<true>(S[8 * e + j], hi[j], lo[j]);
                        if (e > 0) gc_stored(&sh.sfull[e - 1]);
                        gc_st8(tq + TC_SHI + 32 * hf + 8 * e, hi);
                        gc_st8(tq + TC_SLO + 32 * hf + 8 * e, lo);
                    }
                }
                if (c == n) break;
                gc_stored(&sh.sfull[3]);
                // while S^T k is formed: the state's largest value
                float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
                for (int j = 0; j < 32; j++) {
                    m0 = fmaxf(m0, fabsf(S[j].x));
                    m1 = fmaxf(m1, fabsf(S[j].y));
                }
                sh.smax[par][hf][dv] = fmaxf(m0, m1) * inv;
                // ---- R = beta v - (beta e^b rk) S^T k, scaled by a power of two from a bound on the row, so
                // that all but one FMA and the split is done before S^T k is there
                float rinv;
                s = gc_pow2(fmaxf(fmaf(sc.crmax * inv, kbound, fmaxf(sh.vmax[prev][0][dv], sh.vmax[prev][1][dv])), inv * GC_FLOOR), rinv);
                const float2 s2 = make_float2(s, s), cs2 = make_float2(-inv * s, -inv * s);
#pragma unroll
                for (int j = 0; j < 16; j++) bv[j] = __fmul2_rn(bv[j], s2);
                dinv = rinv * sc.pd;
                if (hf == 0) sh.vinv[c & 3][dv] = rinv * sc.pt;
                ok &= gc_wait(&sh.ksfull, par);
                gc_fence_after();
                gc_ld16(tq + TC_KS + 32 * hf, d[0]);
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    gc_wait16(d[e]);
                    if (e == 0) gc_ld16(tq + TC_KS + 32 * hf + 16, d[1]);
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        gc_split(__ffma2_rn(gc_pair(d[e], j),
                                            __fmul2_rn(*reinterpret_cast<const float2*>(&sc.cr[32 * hf + 16 * e + 2 * j]), cs2), bv[8 * e + j]),
                                 hi[j], lo[j]);
                    if (e == 1) gc_stored(&sh.rfull[0]);
                    gc_st8(tq + TC_DS + 16 * hf + 8 * e, hi);
                    gc_st8(tq + TC_DS + 32 + 16 * hf + 8 * e, lo);
                }
                gc_stored(&sh.rfull[1]);
            }
            // ---- while T R runs: the next chunk's V
            if (c + 1 < n) {
                const GcScal& sn = scals[(c + 1) & 3];
                const uint8_t* vt = vtiles + (2 + (par ^ 1u)) * GC_VTILE + dv * 128;
                const int live_rows = len - GC_C * (c + 1) - 32 * hf;  // of this half's
                ok &= gc_wait(&sh.vtfull[par ^ 1u], (uint32_t)((c + 1) >> 1) & 1u);
                float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint4 w = *reinterpret_cast<const uint4*>(vt + (((4 * hf + i) ^ (dv & 7)) << 4));
                    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float2 be = *reinterpret_cast<const float2*>(&sn.beta[32 * hf + 8 * i + 2 * j]);
                        bv[4 * i + j] = __fmul2_rn(be, make_float2(__uint_as_float(v[j] << 16), __uint_as_float(v[j] & 0xFFFF0000u)));
                    }
                }
                gc_arrive_warp(&sh.vtempty[par ^ 1u]);
                if (live_rows < 32) {  // the rows past the end hold anything
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        if (2 * j >= live_rows) bv[j].x = 0.0f;
                        if (2 * j + 1 >= live_rows) bv[j].y = 0.0f;
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    m0 = fmaxf(m0, fabsf(bv[j].x));
                    m1 = fmaxf(m1, fabsf(bv[j].y));
                }
                sh.vmax[par][hf][dv] = fmaxf(m0, m1);
            }
            if (c >= 0) {
                // ---- V' and V'' = e^(b_C - b) rk V', scaled by the row's power of two and the chunk's
                ok &= gc_wait(&sh.d2full, par);
                gc_fence_after();
                __half2 big = __floats2half2_rn(0.0f, 0.0f);
                uint32_t u[2][16];
                gc_ld16(tq + TC_KS + 32 * hf, u[0]);
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    gc_wait16(u[e]);
                    if (e == 0) gc_ld16(tq + TC_KS + 32 * hf + 16, u[1]);
                    uint32_t hi[8], lo[8], v1[8];
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const int i = 32 * hf + 16 * e + 2 * j;
                        const float2 x = gc_pair(u[e], j);
                        gc_split(__fmul2_rn(x, *reinterpret_cast<const float2*>(&sc.fv[i])), hi[j], lo[j]);
                        v1[j] = gc_half2(__fmul2_rn(x, *reinterpret_cast<const float2*>(&sc.ft[i])));
                    }
                    if (e == 1) gc_stored(&sh.vfull[0]);
                    gc_st8(tq + TC_SLO + 16 * hf + 8 * e, hi);
                    gc_st8(tq + TC_SLO + 32 + 16 * hf + 8 * e, lo);
                    gc_st8(tq + TC_V + 16 * hf + 8 * e, v1);
#pragma unroll
                    for (int j = 0; j < 8; j++) big = __hmax2(big, __habs2(*reinterpret_cast<__half2*>(&hi[j])));
                }
                gc_stored(&sh.vfull[1]);
                // |dS| <= 32 tokens x (largest V'' term + its last place) x 2^8
                const float2 bf = __half22float2(big);
                sh.dmax[par][hf][dv] = fmaf(fmaxf(bf.x, bf.y), 1.002f, 0x1p-13f) * (8192.0f * dinv);
            }
            gc_arrive_warp(&sh.bounds);
        }
        if (!ok) sh.failed = 1;
        if (ok) {
#pragma unroll
            for (int j = 0; j < 32; j++) {
                __stcs(st + 2 * j * GC_D, S[j].x * inv);
                __stcs(st + (2 * j + 1) * GC_D, S[j].y * inv);
            }
        }
    } else if (warp < GC_WMMA) {
        // ================================================================ outputs
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(GC_REGS_OUT));
        const int dv = 32 * (warp & 3) + lane;
        const uint32_t tq = tb + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t step = (uint32_t)p.hv * (GC_D * 2);  // bytes a token
        // neighbouring lanes exchange, so that each stores two value columns: the even one the even tokens
        const int odd = lane & 1;
        uint8_t* dst = reinterpret_cast<uint8_t*>(p.out + ((int64_t)start * p.hv + head) * GC_D);
        const uint32_t mine = (uint32_t)odd * step + 2u * (uint32_t)(dv & ~1);
        for (int c = 0; c < n; c++) {
            const uint32_t par = (uint32_t)c & 1u;
            const GcScal& sc = scals[c & 3];
            const int live_rows = min(GC_C, len - GC_C * c);
            bool ok = gc_wait(&sh.vld[c & 3], (uint32_t)(c >> 2) & 1u);
            ok &= gc_wait(&sh.ofull, par);
            if (!ok) {
                sh.failed = 1;
                break;
            }
            gc_fence_after();
            const float si = sh.sinv[c & 3][dv], vi = sh.vinv[c & 3][dv];
            const float2 si2 = make_float2(si, si), vi2 = make_float2(vi, vi);
            const int lim = live_rows - odd;
            uint32_t off = mine;
#pragma unroll
            for (int b = 0; b < 4; b++) {
                uint32_t qs[16], pv[16];
                gc_ld16(tq + TC_QS + 16 * b, qs);
                gc_ld16(tq + TC_PV + 16 * b, pv);
                gc_wait16(qs);
                gc_wait16(pv);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int i = 16 * b + 2 * j;
                    const float2 co = *reinterpret_cast<const float2*>(&sc.co[i]);
                    const float2 pi = *reinterpret_cast<const float2*>(&sc.pinv[i]);
                    const float2 y = __ffma2_rn(gc_pair(qs, j), __fmul2_rn(co, si2), __fmul2_rn(gc_pair(pv, j), __fmul2_rn(pi, vi2)));
                    const uint32_t o = bf162_bits(__floats2bfloat162_rn(y.x, y.y));
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, o, 1);
                    // even lane: token i of columns dv, dv + 1; odd lane: token i + 1 of dv - 1, dv
                    const uint32_t pair = odd ? __byte_perm(other, o, 0x7632u) : __byte_perm(o, other, 0x5410u);
                    if (i < lim) *reinterpret_cast<uint32_t*>(dst + off) = pair;
                    off += 2 * step;
                }
            }
            gc_fence_before();
            gc_arrive_warp(&sh.ofree);  // the accumulators and the factors are read
            dst += (int64_t)GC_C * step;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(GC_REGS_MMA));
        if (warp == GC_WMMA) {
            // ============================================================ MMA issuer
            // The whole warp runs the loop (so that every operand is warp-uniform); one elected lane issues.
            const uint32_t I64 = gc_idesc(64, 0), I48 = gc_idesc(48, 0), I32 = gc_idesc(32, 0), I16 = gc_idesc(16, 0), I128T = gc_idesc(128, 1);
            const uint32_t one = gc_elect();
            bool ok = true;
            for (int c = 0; c < n && ok; c++) {
                const uint32_t par = (uint32_t)c & 1u;
                const uint32_t s = su + par * GC_STAGE;
                ok = gc_wait(&sh.ldfull[par], (uint32_t)(c >> 1) & 1u);
                // S K^T, in the order in which both warp halves store their terms
#pragma unroll 1
                for (uint32_t e = 0; e < 4; e++) {
                    ok &= gc_wait(&sh.sfull[e], par);
                    gc_fence_after();
#pragma unroll
                    for (int k = 1; k >= 0; k--)
#pragma unroll
                        for (int h = 0; h < 2; h++)
                            gc_mma(tb + TC_KS, tb + (k ? TC_SLO : TC_SHI) + 32 * h + 8 * e, gc_desc(s + h * GC_HALF + 32 * e), I64,
                                   k == 1 && h == 0 ? e : 1u, one);
                }
                gc_commit(&sh.ksfull, one);
                // V'^T = R^T T^T: lo T_hi + hi T_lo + hi T_hi, by 16 tokens of either half.  T is lower
                // triangular: columns 16 x .. have rows 16 x .. only.
                ok &= gc_wait(&sh.rfull[0], par);
                gc_fence_after();
#pragma unroll
                for (int e = 0; e < 3; e++) {
                    gc_mma(tb + TC_KS, tb + TC_DS + (e == 0 ? 32 : 0), gc_desc(s + GC_T + (e == 1 ? GC_TILE : 0)), I64, e, one);
                    gc_mma(tb + TC_KS + 32, tb + TC_DS + (e == 0 ? 32 : 0) + 16,
                           gc_desc(s + GC_T + 32 * 128 + (e == 1 ? GC_TILE : 0) + 64), I32, 1u, one);
                }
                ok &= gc_wait(&sh.rfull[1], par);
                gc_fence_after();
#pragma unroll
                for (int e = 0; e < 3; e++) {
                    gc_mma(tb + TC_KS + 16, tb + TC_DS + (e == 0 ? 32 : 0) + 8,
                           gc_desc(s + GC_T + 16 * 128 + (e == 1 ? GC_TILE : 0) + 32), I48, 1u, one);
                    gc_mma(tb + TC_KS + 48, tb + TC_DS + (e == 0 ? 32 : 0) + 24,
                           gc_desc(s + GC_T + 48 * 128 + (e == 1 ? GC_TILE : 0) + 96), I16, 1u, one);
                }
                gc_commit(&sh.d2full, one);
                // S Q^T (its accumulator is free once the outputs of the chunk before are read)
                if (c > 0) ok &= gc_wait(&sh.ofree, par ^ 1u);
                gc_fence_after();
#pragma unroll
                for (int x = 0; x < 8; x++)
                    gc_mma(tb + TC_QS, tb + TC_SHI + 8 * x, gc_desc(s + (x >> 2) * GC_HALF + 8192 + 32 * (x & 3)), I64, x != 0, one);
                // dS^T = V''^T K (the K tile as [tokens][head dimension]), by 16 tokens of either half
#pragma unroll 1
                for (uint32_t e = 0; e < 2; e++) {
                    ok &= gc_wait(&sh.vfull[e], par);
                    gc_fence_after();
#pragma unroll
                    for (int k = 1; k >= 0; k--)
#pragma unroll
                        for (int h = 0; h < 2; h++)
                            gc_mma(tb + TC_DS, tb + TC_SLO + 32 * k + 16 * h + 8 * e, gc_desc(s + 4096 * h + 2048 * e, GC_HALF),
                                   I128T, k == 1 && h == 0 ? e : 1u, one);
                }
                gc_commit(&sh.dsfull, one);
                // (P V')^T
#pragma unroll
                for (int kk = 0; kk < 4; kk++)
                    gc_mma(tb + TC_PV, tb + TC_V + 8 * kk, gc_desc(s + GC_P + 32 * kk), I64, kk, one);
                gc_commit(&sh.ofull, one);
                gc_commit(&sh.ldempty[par], one);
            }
            if (!ok) sh.failed = 1;
            gc_commit(&sh.done, one);  // completes once every MMA issued above has finished
            if (!mbar_wait_suspend(&sh.done, 0)) sh.failed = 1;
            __syncwarp();
        } else if (warp == GC_WTMA) {
            // ============================================================ the chunks' operands
            if (lane == 0) {
                // V and the factors run one chunk ahead of the MMAs' operands: V once the tile of two chunks
                // before is transposed; the factors overwrite those of four chunks before, whose outputs
                // were read before the operands' stage came free.
                const int64_t base = start / GC_C + seq;
                auto load_v = [&](int c) {
                    uint8_t* dst = vtiles + (c & 1) * GC_VTILE;
                    mbar_arrive_expect_tx(&sh.vld[c & 3], GC_VTILE + (uint32_t)sizeof(GcScal));
                    bulk_load(&sh.scal[c & 3], p.tp + ((base + c) * p.hv + head) * GC_TP + 3 * GC_TILE, sizeof(GcScal), &sh.vld[c & 3]);
                    tma_load_3d(dst, &mapV, 0, head, start + GC_C * c, &sh.vld[c & 3]);
                    tma_load_3d(dst + GC_VTILE / 2, &mapV, 64, head, start + GC_C * c, &sh.vld[c & 3]);
                };
                auto ready = [&](int c) {
                    if (!AHEAD) return true;
                    const int group = p.hv / p.hk;  // the key head's rows come with its first value head
                    const bool there = gc_wait_ready(gc_ready(p, base + c, kh * group)) && gc_wait_ready(gc_ready(p, base + c, head));
                    if (!there) sh.failed = 1;
                    return there;
                };
                int c = 0, v = 0;
                if (ready(0)) load_v(v++);
                for (; c < v; c++) {
                    const int s = c & 1;
                    if (c >= 2 && !mbar_wait_lean(&sh.ldempty[s], (uint32_t)((c >> 1) - 1) & 1u)) {
                        sh.failed = 1;
                        break;
                    }
                    uint8_t* dst = stages + s * GC_STAGE;
                    mbar_arrive_expect_tx(&sh.ldfull[s], GC_STAGE);
                    bulk_load(dst, p.kq + ((base + c) * p.hk + kh) * GC_KQ, GC_KQ, &sh.ldfull[s]);
                    bulk_load(dst + GC_T, p.tp + ((base + c) * p.hv + head) * GC_TP, 3 * GC_TILE, &sh.ldfull[s]);
                    if (c + 1 < n) {
                        if (c >= 1 && !mbar_wait_lean(&sh.vtfull[(c - 1) & 1], (uint32_t)((c - 1) >> 1) & 1u)) {
                            sh.failed = 1;
                            c++;
                            break;
                        }
                        if (ready(v)) load_v(v++);
                    }
                }
                // the copies requested last have landed
                for (int j = c > 2 ? c - 2 : 0; j < c; j++)
                    if (!mbar_wait_suspend(&sh.ldfull[j & 1], (uint32_t)(j >> 1) & 1u)) atomicOr(&g_gated_delta_status, 2u);
                for (int j = v > 4 ? v - 4 : 0; j < v; j++)
                    if (!mbar_wait_suspend(&sh.vld[j & 3], (uint32_t)(j >> 2) & 1u)) atomicOr(&g_gated_delta_status, 2u);
            }
            __syncwarp();
        } else {
            // ============================================================ V^T, 32 tokens a warp
            // 8 x 8 blocks: a transposed matrix load of four blocks along the tokens, a matrix store
            const int th = warp - GC_WTMA - 1, r8 = lane & 7, m = lane >> 3;
            const uint32_t src = smem_u32(vtiles) + (uint32_t)(32 * th + lane) * 128u;  // row of block m: token 8 m + r8
            const uint32_t dst = smem_u32(vtiles) + 2 * GC_VTILE + (uint32_t)r8 * 128u + (uint32_t)(((4 * th + m) ^ r8) << 4);
            for (int c = 0; c < n; c++) {
                bool ok = gc_wait(&sh.vld[c & 3], (uint32_t)(c >> 2) & 1u);
                if (c >= 2) ok &= gc_wait(&sh.vtempty[c & 1], (uint32_t)((c >> 1) - 1) & 1u);
                if (!ok) {
                    sh.failed = 1;
                    break;
                }
                const uint32_t o = (uint32_t)(c & 1) * GC_VTILE;
#pragma unroll 4
                for (int g = 0; g < 16; g++) {  // value columns 8 g .. 8 g + 7
                    uint32_t r[4];
                    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                                 : "r"(src + o + (uint32_t)(g >> 3) * (GC_VTILE / 2) + (uint32_t)(((g & 7) ^ r8) << 4))
                                 : "memory");
                    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(dst + o + (uint32_t)g * 1024u),
                                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                                 : "memory");
                }
                gc_arrive_warp(&sh.vtfull[c & 1]);
            }
        }
    }

    gc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sh.failed) atomicOr(&g_gated_delta_status, 1u);
    if (warp == GC_WMMA) {
        gc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tb), "n"(512));
    }
}

// [tokens][heads][128] BF16 as a 3-D map (128, heads, tokens), boxes of 64 tokens x 64 columns of one
// head with the 128-byte swizzle.
static int gc_map(CUtensorMap* map, const bq_heads* h, uint32_t tokens, uint32_t heads, const char* who) {
    const uint64_t ts = tokens > 1 ? (uint64_t)h->token_stride : (uint64_t)GC_D * heads;
    const uint64_t hs = heads > 1 ? (uint64_t)h->head_stride : GC_D;
    return make_tmap_heads(map, h->data, GC_D, heads, tokens, hs * 2, ts * 2, 64, GC_C, true, who);
}

}  // namespace bq8

using namespace bq8;

extern "C" size_t bq_gated_delta_prefill_scratch_bytes(uint32_t seqs, uint32_t total, uint32_t heads_k, uint32_t heads_v) {
    if (seqs == 0 || total == 0) return 0;
    const size_t slots = (size_t)gc_slots(seqs, total);
    return slots * ((size_t)heads_k * GC_KQ + (size_t)heads_v * GC_TP) + (slots * heads_v * 4 + 15) / 16 * 16;
}

extern "C" int gated_delta_prefill(const bq_heads* q, const bq_heads* k, const bq_heads* v, const bq_heads* g,
                                   const bq_heads* beta, float* state, const int32_t* cu_seqlens,
                                   const int32_t* state_idx, uint16_t* out, void* scratch, uint32_t seqs, uint32_t total,
                                   uint32_t heads_k, uint32_t heads_v, uint32_t head_dim, uint32_t slots, float scale,
                                   int l2norm, bq_stream_t stream) {
    const char* who = "gated_delta_prefill";
    if (seqs == 0 || total == 0) return ok();
    int st = gd_check(q, k, v, g, beta, state, out, heads_k, heads_v, head_dim, slots, who);
    if (st) return st;
    if (!aligned4(cu_seqlens) || !aligned4(state_idx))
        return fail(BQ_ERR_INVALID, "%s: cu_seqlens and state_idx must be 4-byte aligned", who);
    if (!cu_seqlens && seqs != 1) return fail(BQ_ERR_INVALID, "%s: cu_seqlens is NULL for %u sequences", who, seqs);
    if (!state_idx && slots < seqs) return fail(BQ_ERR_INVALID, "%s: %u slots for %u sequences", who, slots, seqs);
    const uint64_t blocks = (uint64_t)gc_slots(seqs, total) * heads_k;
    if (total >= (1u << 30) || (uint64_t)seqs * heads_v >= (1ull << 31) || blocks >= (1ull << 31))
        return fail(BQ_ERR_INVALID, "%s: shape too large", who);
    if (!scratch || !aligned16(scratch))
        return fail(BQ_ERR_INVALID, "%s: needs %zu bytes of 16-byte aligned scratch", who,
                    bq_gated_delta_prefill_scratch_bytes(seqs, total, heads_k, heads_v));
    const bq_heads* h[3] = {q, k, v};
    const uint32_t nh[3] = {heads_k, heads_k, heads_v};
    CUtensorMap map[3];
    for (int i = 0; i < 3; i++) {
        if ((total > 1 && h[i]->token_stride == 0) || (nh[i] > 1 && h[i]->head_stride == 0))
            return fail(BQ_ERR_INVALID, "%s: %c is broadcast (a stride of 0)", who, "qkv"[i]);
        if ((st = gc_map(&map[i], h[i], total, nh[i], who))) return st;
    }
    static int configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 63;
    if (!configured[dev]) {
        // the warpgroups' register shares wait for what the launch holds: it must be exactly this
        cudaFuncAttributes fa[2];
        if (cudaFuncGetAttributes(&fa[0], gated_delta_recur_kernel<false>) != cudaSuccess ||
            cudaFuncGetAttributes(&fa[1], gated_delta_recur_kernel<true>) != cudaSuccess || fa[0].numRegs != GC_REGS ||
            fa[1].numRegs != GC_REGS)
            return fail(BQ_ERR_UNSUPPORTED, "%s: built with %d and %d registers a thread, needs %d", who, fa[0].numRegs,
                        fa[1].numRegs, GC_REGS);
        const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
        if (cudaFuncSetAttribute(gated_delta_recur_kernel<false>, at, (int)GC_SMEM) != cudaSuccess ||
            cudaFuncSetAttribute(gated_delta_recur_kernel<true>, at, (int)GC_SMEM) != cudaSuccess ||
            cudaFuncSetAttribute(gated_delta_prepare_kernel, at, (int)GP_SMEM) != cudaSuccess)
            return fail(BQ_ERR_LAUNCH, "%s: cannot reserve %zu bytes of shared memory", who, GC_SMEM);
        configured[dev] = 1;
    }
    uint8_t* kq = (uint8_t*)scratch;
    uint8_t* tp = kq + (size_t)blocks * GC_KQ;
    const size_t flags = (size_t)gc_slots(seqs, total) * heads_v;
    GcArgs a = {*g,  *beta,     state,      cu_seqlens,   state_idx,    out,        kq, tp,
                (int)seqs, (int)total, (int)heads_k, (int)heads_v, (int)slots, scale, l2norm != 0, 1,
                reinterpret_cast<int*>(tp + flags * GC_TP)};
    const uint32_t chains = seqs * heads_v, sms = (uint32_t)sm_count();
    if (2 * (uint64_t)chains <= sms) {  // (both sides' times at the top of this file)
        if (cudaMemsetAsync(a.ready, 0, flags * sizeof(int), (cudaStream_t)stream) != cudaSuccess)
            return fail(BQ_ERR_LAUNCH, "%s: %s", who, cudaGetErrorString(cudaGetLastError()));
        const uint64_t most = chains + (uint64_t)gc_slots(seqs, total) * heads_v;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(most < sms ? most : sms));
        cfg.blockDim = dim3(GC_THREADS);
        cfg.dynamicSmemBytes = GC_SMEM;
        cfg.stream = (cudaStream_t)stream;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeCooperative;  // the CTAs wait for one another's flags
        at[0].val.cooperative = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, gated_delta_recur_kernel<true>, map[0], map[1], map[2], a);
        if (e == cudaSuccess) return check_launch(who);
        cudaGetLastError();
        // (a process that holds a part of the device cannot have a CTA on every SM at once: the two kernels below)
        if (e != cudaErrorCooperativeLaunchTooLarge) return fail(BQ_ERR_LAUNCH, "%s: %s", who, cudaGetErrorString(e));
    }
    // A block for every value head while all of them run at once (64 tokens x 48 heads: 20.7 us, 26.9 with
    // one a key head), else one a key head, which forms [K; Q] K^T once for its value heads (8192 x 48:
    // 428 and 454 us).
    const uint32_t group = heads_v / heads_k;
    if (blocks * group <= 5ull * sms) a.parts = (int)group;
    if ((st = launch_programmatic(who, gated_delta_prepare_kernel, (uint32_t)(blocks * a.parts), 128, GP_SMEM,
                                  (cudaStream_t)stream, map[0], map[1], a)))
        return st;
    return launch_programmatic(who, gated_delta_recur_kernel<false>, chains, GC_THREADS, GC_SMEM, (cudaStream_t)stream,
                               map[0], map[1], map[2], a);
}
