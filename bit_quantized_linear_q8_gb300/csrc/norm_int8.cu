// norm_int8.cu -- root-mean-square norm with the residual's addition and an 8-bit output, the
// row quantiser without the norm, and the expansion of int8 codes to BF16.
//
//   h = x + residual (fp32);  y = h / sqrt(mean(h^2) + eps) * weight (fp32)
//   int8: s = max|y| / 127 per row, code = round-half-away(y / s);   q8_1: the same per 32 values
//   with s = d sum(code) beside d (the layout of quantize_act_q8_1).
//
// The codes are taken from the fp32 y, not from a BF16 copy of it, so the only roundings are the
// code itself and the scale.  All sums and maxima are fp32.
//
// The row stays in registers between its two reductions (sum of squares, maximum), so each
// value is read once and written once: 7 bytes a value with a residual (x, residual, sum and
// code), 3 without.  Bound: HBM for large m with a residual (4096 x 5120: 24.9 us, 5.9 TB/s), latency
// without one (2048 x 6144: 11.9 us, the row quantiser 8.4, their bytes 5.6: one row a block, its load, two
// block reductions and its store one after the other; 43 % of the issue slots are used), the launch and the
// reductions' latency for few rows (4 x 5120: 2.6 us).  The q8_1 output: 27.3 us for 4096 x 5120 with a
// residual, 13.8 for 2048 x 6144 without.  (All of these from a graph.)  Packed arithmetic and a division
// decided once a row took 4096 x 5120 from 38.3 to 28.8 us; all kernels here are launched
// programmatically, which takes 1.4-3.6 us off each.
// (Streaming loads or stores change nothing or lose 1 us.)
#include "common.cuh"

namespace bq8 {

constexpr int NQ_INT8 = 0, NQ_Q8_1 = 1;

struct NqArgs {
    const uint16_t* x;
    const uint16_t* residual;  // or NULL
    const uint16_t* weight;    // NULL: no norm (the row quantiser)
    uint16_t* sum;             // BF16(h), or NULL
    uint16_t* y;               // BF16(y), or NULL
    uint8_t* codes;
    float* scales;             // int8: [m]; q8_1: (d, s) pairs [m][kp / 32]
    float eps;
    uint32_t m, k, kp;         // kp: code row stride (q8_1: k rounded up to 256)
};

// Reduction over a row's threads: the whole warp first, then the warps through shared memory
// (nw warps; nw = 1 needs no barrier).  MAX: unsigned maximum of the bit patterns of |v|, whose
// order is that of the values with infinity and NaN on top, so a NaN in the row is kept.
template <bool MAX>
__device__ __forceinline__ float nq_reduce(float v, float* sm, int nw) {
    if (MAX) {
        v = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    if (nw == 1) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) sm[warp] = v;
    __syncthreads();
    v = lane < nw ? sm[lane] : 0.0f;
    if (MAX) {
        v = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

__device__ __forceinline__ float nq_abs_bits(float v) { return __uint_as_float(__float_as_uint(v) & 0x7FFFFFFFu); }

// max(m, |v|), a NaN kept.
__device__ __forceinline__ float nq_max_abs(float m, float v) {
    float r;
    asm("{\n.reg .f32 a;\nabs.f32 a, %2;\nmax.NaN.f32 %0, %1, a;\n}\n" : "=f"(r) : "f"(m), "f"(v));
    return r;
}

// 1 / sqrt(mean(h^2) + eps) from the sum of squares.  A sum that leaves fp32 (finite values above 2^63 or so) would
// give 0 and a row of zeros without a sign of it: NaN, so that the row reads as NaN.
__device__ __forceinline__ float nq_inv_rms(float ss, const NqArgs& p) {
    const float rs = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)p.k) + p.eps));
    return ss <= 3.4028235e38f ? rs : __int_as_float(0x7fffffff);
}

// The arithmetic runs on pairs (packed fp32: two values an instruction, each rounded as alone).
__device__ __forceinline__ void nq_unpack8(const uint4& w, float2 (&v)[4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 nq_pack8(const float2 (&v)[4]) {
    return make_uint4(bf162_bits(__floats2bfloat162_rn(v[0].x, v[0].y)), bf162_bits(__floats2bfloat162_rn(v[1].x, v[1].y)),
                      bf162_bits(__floats2bfloat162_rn(v[2].x, v[2].y)), bf162_bits(__floats2bfloat162_rn(v[3].x, v[3].y)));
}

// Round half away from zero: adding the largest float below 1/2 and truncating is exact for
// every |t| < 2^22 (with 1/2 itself, 0.49999997 would round up to 1).
__device__ __forceinline__ int nq_round(float t) { return __float2int_rz(t + copysignf(0.49999997f, t)); }

// Codes of one row from its scale.  y / s is y times RN(1/s), within 2 units in the last place of
// the quotient, so a code can differ from the exact quotient's only where that lies as close to
// a half-way point.  Scales whose reciprocal is not a normal number take the division, and as a subnormal
// scale is rounded to whole units of 2^-149 (128 to 190 units of |y| to one), their codes stop at 127.  A row
// with a NaN or an infinity has the scale NaN or infinity (its decoded values are NaN) and codes 0.
struct NqScale {
    float s, inv;
    bool divide, none;
    __device__ __forceinline__ explicit NqScale(float amax) {
        s = __fdiv_rn(amax, 127.0f);
        none = !(s > 0.0f) || !(amax <= 3.4028235e38f);
        divide = amax < 1e-30f;
        inv = none || divide ? 0.0f : __frcp_rn(s);
    }
    __device__ __forceinline__ int divided(float y) const { return min(max(nq_round(__fdiv_rn(y, s)), -127), 127); }
    __device__ __forceinline__ int code(float y) const {
        if (none) return 0;
        return divide ? divided(y) : nq_round(y * inv);
    }
    // Eight codes; whether to divide is decided once (a division beside every product took the
    // kernel twice as long).  Without codes inv is 0, and 0 times anything rounds to the code 0.
    __device__ __forceinline__ void codes(const float2 (&y)[4], int (&q)[8]) const {
        if (divide && !none) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                q[2 * j] = divided(y[j].x);
                q[2 * j + 1] = divided(y[j].y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float2 t = __fmul2_rn(y[j], make_float2(inv, inv));
                const float2 r = __fadd2_rn(t, make_float2(copysignf(0.49999997f, t.x), copysignf(0.49999997f, t.y)));
                q[2 * j] = __float2int_rz(r.x);
                q[2 * j + 1] = __float2int_rz(r.y);
            }
        }
    }
};

__device__ __forceinline__ uint32_t nq_pack4(int a, int b, int c, int d) {
    return __byte_perm(__byte_perm((uint32_t)a, (uint32_t)b, 0x0040u), __byte_perm((uint32_t)c, (uint32_t)d, 0x0040u), 0x5410u);
}

// k % 8 == 0: eight values a thread and vector, V vectors a thread at stride T, the row in
// registers.  ROWS rows a block of ROWS warps when a warp holds a row (T = 32), else one.
template <int FMT, int V, bool NORM>
__global__ void __launch_bounds__(1024) norm_int8_kernel(const NqArgs p, int T) {
    __shared__ float red[2][32];
    pdl_wait();
    pdl_launch_dependents();
    const int rows = blockDim.x / T;
    const int t = threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * rows + threadIdx.x / T;
    if (row >= p.m) return;  // whole warps: T is a multiple of 32, and one row a block when T > 32
    const int nw = T >> 5, nv = (int)(p.k >> 3);
    const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.k);
    const uint4* r = p.residual ? reinterpret_cast<const uint4*>(p.residual + row * p.k) : nullptr;
    const uint4* w = reinterpret_cast<const uint4*>(p.weight);
    uint4 xv[V], rv[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int c = t + i * T;
        xv[i] = rv[i] = make_uint4(0, 0, 0, 0);
        if (c < nv) {
            xv[i] = x[c];
            if (NORM && r) rv[i] = r[c];
        }
    }
    float2 h[V][4];
    float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < V; i++) {
        nq_unpack8(xv[i], h[i]);
        if (NORM) {
            if (r) {
                float2 q[4];
                nq_unpack8(rv[i], q);
#pragma unroll
                for (int j = 0; j < 4; j++) h[i][j] = __fadd2_rn(h[i][j], q[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) s2 = __ffma2_rn(h[i][j], h[i][j], s2);
            const int c = t + i * T;
            if (p.sum && c < nv) reinterpret_cast<uint4*>(p.sum + row * p.k)[c] = nq_pack8(h[i]);
        }
    }
    float amax = 0.0f;
    if (NORM) {
        const float ss = nq_reduce<false>(s2.x + s2.y, red[0], nw);
        const float rs = nq_inv_rms(ss, p);
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int c = t + i * T;
            float2 g[4];
            nq_unpack8(c < nv ? w[c] : make_uint4(0, 0, 0, 0), g);
#pragma unroll
            for (int j = 0; j < 4; j++) h[i][j] = __fmul2_rn(__fmul2_rn(h[i][j], make_float2(rs, rs)), g[j]);
            if (p.y && c < nv) reinterpret_cast<uint4*>(p.y + row * p.k)[c] = nq_pack8(h[i]);
        }
    }
    if (FMT == NQ_INT8) {
#pragma unroll
        for (int i = 0; i < V; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) amax = nq_max_abs(nq_max_abs(amax, h[i][j].x), h[i][j].y);
        amax = nq_reduce<true>(amax, red[1], nw);
        const NqScale sc(amax);
        if (t == 0) p.scales[row] = sc.s;
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int c = t + i * T;
            int q[8];
            sc.codes(h[i], q);
            if (c < nv)
                *reinterpret_cast<uint2*>(p.codes + row * p.k + 8 * (int64_t)c) =
                    make_uint2(nq_pack4(q[0], q[1], q[2], q[3]), nq_pack4(q[4], q[5], q[6], q[7]));
        }
    } else {
        // a block of 32 values is four neighbouring threads' vectors; vectors past k are the
        // zeros of the padding to kp
        const int nvp = (int)(p.kp >> 3);
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int c = t + i * T;
            float bm = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; j++) bm = nq_max_abs(nq_max_abs(bm, h[i][j].x), h[i][j].y);
            bm = __uint_as_float(max(__float_as_uint(bm), __shfl_xor_sync(0xffffffffu, __float_as_uint(bm), 1)));
            bm = __uint_as_float(max(__float_as_uint(bm), __shfl_xor_sync(0xffffffffu, __float_as_uint(bm), 2)));
            const NqScale sc(bm);
            int q[8], sum = 0;
            sc.codes(h[i], q);
#pragma unroll
            for (int j = 0; j < 8; j++) sum += q[j];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (c < nvp) {
                *reinterpret_cast<uint2*>(p.codes + row * p.kp + 8 * (int64_t)c) =
                    make_uint2(nq_pack4(q[0], q[1], q[2], q[3]), nq_pack4(q[4], q[5], q[6], q[7]));
                if ((c & 3) == 0)
                    *reinterpret_cast<float2*>(p.scales + 2 * (row * (p.kp >> 5) + (c >> 2))) =
                        make_float2(sc.s, sc.s * (float)sum);
            }
        }
    }
}

// Any k (rows need not be 16-byte aligned, or are too long for the registers): one block a row,
// one value a thread and step, the row read again (from L2) for the codes.  The values are
// formed by the same operations as above.
template <int FMT, bool NORM>
__global__ void __launch_bounds__(1024) norm_int8_any_kernel(const NqArgs p) {
    __shared__ float red[2][32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const int T = blockDim.x, t = threadIdx.x, nw = T >> 5;
    const uint16_t* x = p.x + row * p.k;
    const uint16_t* r = NORM && p.residual ? p.residual + row * p.k : nullptr;
    auto h_at = [&](uint32_t c) {
        const float v = bf16_bits_to_f32(x[c]);
        return r ? v + bf16_bits_to_f32(r[c]) : v;
    };
    float rs = 1.0f;
    if (NORM) {
        float ss = 0.0f;
        for (uint32_t c = t; c < p.k; c += T) {
            const float h = h_at(c);
            ss = fmaf(h, h, ss);
        }
        ss = nq_reduce<false>(ss, red[0], nw);
        rs = nq_inv_rms(ss, p);
    }
    auto y_at = [&](uint32_t c) { return NORM ? h_at(c) * rs * bf16_bits_to_f32(p.weight[c]) : h_at(c); };
    float amax = 0.0f;
    if (FMT == NQ_INT8) {
        for (uint32_t c = t; c < p.k; c += T)
            amax = __uint_as_float(max(__float_as_uint(amax), __float_as_uint(nq_abs_bits(y_at(c)))));
        amax = nq_reduce<true>(amax, red[1], nw);
    }
    NqScale sc(amax);
    if (FMT == NQ_INT8 && t == 0) p.scales[row] = sc.s;
    const uint32_t lim = FMT == NQ_INT8 ? p.k : p.kp;  // kp: a multiple of 256, whole warps
    for (uint32_t c = t; c < lim; c += T) {
        const float h = c < p.k ? h_at(c) : 0.0f;
        const float y = c < p.k ? y_at(c) : 0.0f;
        if (FMT == NQ_Q8_1) {
            const float bm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(nq_abs_bits(y))));
            sc = NqScale(bm);
        }
        const int q = sc.code(y);
        if (FMT == NQ_Q8_1) {
            const int sum = __reduce_add_sync(0xffffffffu, q);
            if ((c & 31) == 0)
                *reinterpret_cast<float2*>(p.scales + 2 * (row * (p.kp >> 5) + (c >> 5))) =
                    make_float2(sc.s, sc.s * (float)sum);
        }
        p.codes[row * (FMT == NQ_INT8 ? p.k : p.kp) + c] = (uint8_t)(int8_t)q;
        if (NORM && c < p.k) {
            const __nv_bfloat16 hb = __float2bfloat16_rn(h), yb = __float2bfloat16_rn(y);
            if (p.y) p.y[row * p.k + c] = *reinterpret_cast<const uint16_t*>(&yb);
            // each value's own thread has read the residual's value above for the last time
            if (p.sum) p.sum[row * p.k + c] = *reinterpret_cast<const uint16_t*>(&hb);
        }
    }
}

template <int FMT, bool NORM>
static int nq_launch(const NqArgs& p, cudaStream_t stream, const char* who) {
    const uint32_t span = FMT == NQ_INT8 ? p.k : p.kp;
    const uint32_t nv = (span + 7) / 8;
    if (p.k % 8 == 0 && nv <= 1024 * 4) {
        // Many rows: four vectors a thread, so that a block's barriers cover more bytes (4096 x 5120:
        // 28.8 us, 29.3 with two, 37.8 with one; 4096 x 1024: 8.4 and 10.3 us with four and one).  Few:
        // the path through one row counts, two vectors a thread (333 x 6144: 6.2 us, 8.3 with one; 4 x
        // 5120: 4.2 us, 6.2 with four; all with plain launches).
        const bool many = p.m >= (uint32_t)sm_count() * 4;
        uint32_t V = many && nv >= 128 ? 4 : nv >= 256 ? 2 : 1;
        while (nv > 1024 * V) V *= 2;
        const uint32_t T = ((nv + V - 1) / V + 31) / 32 * 32;
        const uint32_t rows = T == 32 ? 4 : 1;
        const unsigned grid = (unsigned)((p.m + rows - 1) / rows), block = T * rows;
        auto* kernel = V == 1 ? norm_int8_kernel<FMT, 1, NORM> : V == 2 ? norm_int8_kernel<FMT, 2, NORM> : norm_int8_kernel<FMT, 4, NORM>;
        return launch_programmatic(who, kernel, grid, block, 0, stream, p, (int)T);
    } else {
        uint32_t T = (span + 31) / 32 * 32;
        if (T > 1024) T = 1024;
        return launch_programmatic(who, norm_int8_any_kernel<FMT, NORM>, p.m, T, 0, stream, p);
    }
}

// int8 codes -> BF16(code * scale of the row): 16 consecutive codes of the flat [rows][k] run a
// thread and step; a run that crosses a row's end takes each code's own scale.
__global__ void __launch_bounds__(256) int8_dequant_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                                                           uint16_t* __restrict__ out, int64_t total, uint32_t k) {
    const int64_t nv = (total + 15) / 16;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < nv; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t at = 16 * i;
        int64_t row = at < (1ll << 32) ? (int64_t)((uint32_t)at / k) : at / k;
        uint32_t c = (uint32_t)(at - row * k);
        if (at + 16 <= total && k - c >= 16) {  // (c + 16 could wrap)
            const uint4 w = ldg_nc128(codes + at);
            const float s = __ldg(scales + row);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float f0 = (float)(int8_t)(u[j]), f1 = (float)(int8_t)(u[j] >> 8), f2 = (float)(int8_t)(u[j] >> 16),
                            f3 = (float)(int8_t)(u[j] >> 24);
                o[2 * j] = bf162_bits(__floats2bfloat162_rn(f0 * s, f1 * s));
                o[2 * j + 1] = bf162_bits(__floats2bfloat162_rn(f2 * s, f3 * s));
            }
            uint4* dst = reinterpret_cast<uint4*>(out + at);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        } else {
            for (int64_t j = at; j < total && j < at + 16; j++) {
                const __nv_bfloat16 b = __float2bfloat16_rn((float)(int8_t)codes[j] * scales[row]);
                out[j] = *reinterpret_cast<const uint16_t*>(&b);
                if (++c == k) {
                    c = 0;
                    row++;
                }
            }
        }
    }
}

struct NqRange {
    const void* at;
    size_t bytes;
};
static bool nq_overlap(const NqRange& a, const NqRange& b) {
    const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
    return x && y && x < y + b.bytes && y < x + a.bytes;
}

// Checks shared by the norm and the row quantiser; kp and the scale plane are set for q8_1.
template <int FMT>
static int nq_run(NqArgs& p, bool norm, cudaStream_t stream, const char* who) {
    if (p.m == 0 || p.k == 0) return ok();
    if (p.m > (1u << 30) || p.k > (1u << 24)) return fail(BQ_ERR_INVALID, "%s: shape too large", who);
    if (!p.x || !aligned16(p.x) || !p.codes || !aligned16(p.codes) || !p.scales || !aligned16(p.scales))
        return fail(BQ_ERR_INVALID, "%s: x, the codes and the scales must be non-NULL and 16-byte aligned", who);
    if (norm) {
        if (!p.weight || !aligned16(p.weight))
            return fail(BQ_ERR_INVALID, "%s: weight must be non-NULL and 16-byte aligned", who);
        if (!aligned16(p.residual) || !aligned16(p.sum) || !aligned16(p.y))
            return fail(BQ_ERR_INVALID, "%s: residual, residual_out and y must be 16-byte aligned", who);
        if (p.sum && !p.residual) return fail(BQ_ERR_INVALID, "%s: residual_out needs a residual", who);
    }
    // residual_out may be the residual or x themselves (every value's thread reads it first); a row's codes
    // would lie over other rows' values
    const size_t nb = (size_t)p.m * p.k * 2;
    const NqRange in[3] = {{p.x, nb}, {p.residual, nb}, {p.weight, (size_t)p.k * 2}};
    const NqRange out[4] = {{p.sum, nb}, {p.y, nb}, {p.codes, (size_t)p.m * p.kp},
                            {p.scales, FMT == NQ_INT8 ? (size_t)p.m * 4 : (size_t)p.m * (p.kp / 32) * 8}};
    bool clash = false;
    for (int i = 0; i < 4; i++) {
        for (int j = 0; j < 3; j++) clash |= !(i == 0 && j < 2 && out[i].at == in[j].at) && nq_overlap(out[i], in[j]);
        for (int j = 0; j < i; j++) clash |= nq_overlap(out[i], out[j]);
    }
    if (clash)
        return fail(BQ_ERR_INVALID, "%s: outputs overlap each other or an input (residual_out may only be residual or x itself)", who);
    if (!(p.eps >= 0.0f)) return fail(BQ_ERR_INVALID, "%s: eps must not be negative", who);
    return norm ? nq_launch<FMT, true>(p, stream, who) : nq_launch<FMT, false>(p, stream, who);
}

}  // namespace bq8

using namespace bq8;

extern "C" int rms_norm_int8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                             uint16_t* residual_out, uint16_t* y, int8_t* codes, float* scales, uint32_t m, uint32_t k,
                             bq_stream_t stream) {
    NqArgs p = {x, residual, weight, residual_out, y, (uint8_t*)codes, scales, eps, m, k, k};
    return nq_run<NQ_INT8>(p, true, (cudaStream_t)stream, "rms_norm_int8");
}

extern "C" int rms_norm_q8_1(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                             uint16_t* residual_out, uint16_t* y, void* act_q8, uint32_t m, uint32_t k,
                             bq_stream_t stream) {
    const uint64_t kp = ((uint64_t)k + 255) / 256 * 256;
    NqArgs p = {x,   residual, weight, residual_out, y, (uint8_t*)act_q8, (float*)((uint8_t*)act_q8 + (uint64_t)m * kp),
                eps, m,        k,      (uint32_t)kp};
    return nq_run<NQ_Q8_1>(p, true, (cudaStream_t)stream, "rms_norm_q8_1");
}

extern "C" int quantize_int8(const uint16_t* x, int8_t* codes, float* scales, uint32_t m, uint32_t k,
                             bq_stream_t stream) {
    NqArgs p = {x, nullptr, nullptr, nullptr, nullptr, (uint8_t*)codes, scales, 0.0f, m, k, k};
    return nq_run<NQ_INT8>(p, false, (cudaStream_t)stream, "quantize_int8");
}

extern "C" int dequant_int8_to_bf16(const int8_t* codes, const float* scales, uint16_t* out, uint32_t rows, uint32_t k,
                                    bq_stream_t stream) {
    const char* who = "dequant_int8_to_bf16";
    if (rows == 0 || k == 0) return ok();
    if (!codes || !scales || !out || !aligned16(codes) || !aligned16(scales) || !aligned16(out))
        return fail(BQ_ERR_INVALID, "%s: codes, scales and out must be non-NULL and 16-byte aligned", who);
    const int64_t total = (int64_t)rows * k;
    const NqRange to = {out, (size_t)total * 2};
    if (nq_overlap(to, {codes, (size_t)total}) || nq_overlap(to, {scales, (size_t)rows * 4}))
        return fail(BQ_ERR_INVALID, "%s: out overlaps an input", who);
    const int64_t want = ((total + 15) / 16 + 255) / 256, most = (int64_t)sm_count() * 64;
    return launch_programmatic(who, int8_dequant_kernel, (uint32_t)(want < most ? want : most), 256, 0, (cudaStream_t)stream,
                               (const uint8_t*)codes, scales, out, total, k);
}
