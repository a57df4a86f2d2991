// gated_delta.cu -- the gated delta rule for single tokens, or a few, of every running sequence.
//
// Per value head, with state S [128 (key)][128 (value)] fp32, key k, query q, value v, log decay g
// and write strength beta:
//     S <- e^g S;   u = beta (v - S^T k);   S <- S + k u^T;   o = scale S^T q
// Written from the old state S0, with a = e^g:
//     u = beta (v - a S0^T k);   o = scale (a S0^T q + (q . k) u);   S = a S0 + k u^T
// so one pass over the state yields both products S0^T k and S0^T q, and the state is read once
// and written once: 128 KB a head and step.  That is the bound (HBM; 64 sequences x 48 heads: 59.6 us,
// 6.8 TB/s, the rate of a plain copy; one sequence: 2.9 us, the launch); arithmetic is 6 operations a
// state value.
//
// A block of four warps owns 32 value columns of one head of one sequence (four blocks a head, so
// that one sequence of 48 heads still gives every SM a block): warp w holds key rows
// 32 w .. 32 w + 31, a lane four columns of eight rows, 32 state values in registers.  The products
// reduce over lanes by shuffles and over the warps through shared memory; the state stays in
// registers for all of the sequence's tokens.  All arithmetic is fp32.
#include "common.cuh"

namespace bq8 {

constexpr int GD_D = 128;        // head dimension of keys and values
constexpr int GD_COLS = 32;      // value columns a block
constexpr float GD_EPS = 1e-6f;  // added to the sum of squares when keys and queries are normalised

struct GdArgs {
    bq_heads q, k, v, g, beta;
    float* state;
    const int32_t* idx;
    uint16_t* out;
    int tokens, hk, hv, slots;
    float scale;
    int l2norm;
};

__device__ __forceinline__ float gd_sum_warp(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void gd_unpack4(uint2 w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

__global__ void __launch_bounds__(128) gated_delta_decode_kernel(const GdArgs p) {
    __shared__ float4 part[2][2][4][8];  // [token parity][k, q product][warp][column quad]
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slab = blockIdx.x % (GD_D / GD_COLS);
    const int head = (int)(blockIdx.x / (GD_D / GD_COLS)) % p.hv;
    const int64_t seq = blockIdx.x / (GD_D / GD_COLS) / p.hv;
    const int kh = head / (p.hv / p.hk);
    const int quad = lane & 7, col = slab * GD_COLS + 4 * quad;
    const int r0 = 32 * warp + (lane >> 3);  // rows r0, r0 + 4, ..., r0 + 28
    const int64_t slot = p.idx ? p.idx[seq] : seq;
    const int64_t tok0 = seq * p.tokens;
    if (slot < 0 || slot >= p.slots) {  // no state: the outputs are zero
        for (int t = warp; t < p.tokens; t += 4)
            if (lane < 8)
                *reinterpret_cast<uint2*>(p.out + ((tok0 + t) * p.hv + head) * GD_D + col) = make_uint2(0u, 0u);
        return;
    }
    const uint16_t* q = (const uint16_t*)p.q.data + kh * p.q.head_stride;
    const uint16_t* k = (const uint16_t*)p.k.data + kh * p.k.head_stride;
    const uint16_t* v = (const uint16_t*)p.v.data + head * p.v.head_stride + col;
    const float* g = (const float*)p.g.data + head * p.g.head_stride;
    const float* beta = (const float*)p.beta.data + head * p.beta.head_stride;

    float* S = p.state + ((slot * p.hv + head) * GD_D + r0) * GD_D + col;
    float4 s[8];
#pragma unroll
    for (int j = 0; j < 8; j++) s[j] = __ldcs(reinterpret_cast<const float4*>(S + 4 * j * GD_D));

    for (int t = 0; t < p.tokens; t++) {
        const int64_t tok = tok0 + t;
        // four key and query values a lane for the whole-row sums, one of this warp's rows each
        const uint2 k4 = *reinterpret_cast<const uint2*>(k + tok * p.k.token_stride + 4 * lane);
        const uint2 q4 = *reinterpret_cast<const uint2*>(q + tok * p.q.token_stride + 4 * lane);
        const float kr = bf16_bits_to_f32(k[tok * p.k.token_stride + 32 * warp + lane]);
        const float qr = bf16_bits_to_f32(q[tok * p.q.token_stride + 32 * warp + lane]);
        const uint2 v4 = *reinterpret_cast<const uint2*>(v + tok * p.v.token_stride);
        const float a = expf(g[tok * p.g.token_stride]), b = beta[tok * p.beta.token_stride];
        float kv[4], qv[4], vv[4];
        gd_unpack4(k4, kv);
        gd_unpack4(q4, qv);
        gd_unpack4(v4, vv);
        float qk = gd_sum_warp(fmaf(qv[0], kv[0], fmaf(qv[1], kv[1], fmaf(qv[2], kv[2], qv[3] * kv[3]))));
        float rk = 1.0f, rq = p.scale;
        if (p.l2norm) {
            const float kk = gd_sum_warp(fmaf(kv[0], kv[0], fmaf(kv[1], kv[1], fmaf(kv[2], kv[2], kv[3] * kv[3]))));
            const float qq = gd_sum_warp(fmaf(qv[0], qv[0], fmaf(qv[1], qv[1], fmaf(qv[2], qv[2], qv[3] * qv[3]))));
            rk = __fdiv_rn(1.0f, __fsqrt_rn(kk + GD_EPS));
            rq = __fdiv_rn(p.scale, __fsqrt_rn(qq + GD_EPS));
        }
        float4 pk = make_float4(0, 0, 0, 0), pq = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float kj = __shfl_sync(0xffffffffu, kr, (lane >> 3) + 4 * j);
            const float qj = __shfl_sync(0xffffffffu, qr, (lane >> 3) + 4 * j);
            pk.x = fmaf(kj, s[j].x, pk.x);
            pk.y = fmaf(kj, s[j].y, pk.y);
            pk.z = fmaf(kj, s[j].z, pk.z);
            pk.w = fmaf(kj, s[j].w, pk.w);
            pq.x = fmaf(qj, s[j].x, pq.x);
            pq.y = fmaf(qj, s[j].y, pq.y);
            pq.z = fmaf(qj, s[j].z, pq.z);
            pq.w = fmaf(qj, s[j].w, pq.w);
        }
#pragma unroll
        for (int o = 8; o <= 16; o <<= 1) {
            pk.x += __shfl_xor_sync(0xffffffffu, pk.x, o);
            pk.y += __shfl_xor_sync(0xffffffffu, pk.y, o);
            pk.z += __shfl_xor_sync(0xffffffffu, pk.z, o);
            pk.w += __shfl_xor_sync(0xffffffffu, pk.w, o);
            pq.x += __shfl_xor_sync(0xffffffffu, pq.x, o);
            pq.y += __shfl_xor_sync(0xffffffffu, pq.y, o);
            pq.z += __shfl_xor_sync(0xffffffffu, pq.z, o);
            pq.w += __shfl_xor_sync(0xffffffffu, pq.w, o);
        }
        if (lane < 8) {
            part[t & 1][0][warp][quad] = pk;
            part[t & 1][1][warp][quad] = pq;
        }
        __syncthreads();  // the other parity's buffer is not written before the next barrier
        float4 sk = part[t & 1][0][0][quad];
#pragma unroll
        for (int w = 1; w < 4; w++) {
            const float4 x = part[t & 1][0][w][quad];
            sk.x += x.x;
            sk.y += x.y;
            sk.z += x.z;
            sk.w += x.w;
        }
        // (a state that is forgotten counts as zeros: its products may have left fp32, and 0 times infinity is not 0)
        if (a == 0.0f) sk = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float ark = a * rk;
        const float4 u = make_float4(b * (vv[0] - ark * sk.x), b * (vv[1] - ark * sk.y), b * (vv[2] - ark * sk.z),
                                     b * (vv[3] - ark * sk.w));
        if (warp == (t & 3) && lane < 8) {
            float4 sq = part[t & 1][1][0][quad];
#pragma unroll
            for (int w = 1; w < 4; w++) {
                const float4 x = part[t & 1][1][w][quad];
                sq.x += x.x;
                sq.y += x.y;
                sq.z += x.z;
                sq.w += x.w;
            }
            if (a == 0.0f) sq = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const float c = qk * rk;
            *reinterpret_cast<uint2*>(p.out + (tok * p.hv + head) * GD_D + col) =
                make_uint2(bf162_bits(__floats2bfloat162_rn(rq * fmaf(a, sq.x, c * u.x), rq * fmaf(a, sq.y, c * u.y))),
                           bf162_bits(__floats2bfloat162_rn(rq * fmaf(a, sq.z, c * u.z), rq * fmaf(a, sq.w, c * u.w))));
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float kj = __shfl_sync(0xffffffffu, kr, (lane >> 3) + 4 * j) * rk;
            s[j].x = fmaf(kj, u.x, a * s[j].x);
            s[j].y = fmaf(kj, u.y, a * s[j].y);
            s[j].z = fmaf(kj, u.z, a * s[j].z);
            s[j].w = fmaf(kj, u.w, a * s[j].w);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; j++) __stcs(reinterpret_cast<float4*>(S + 4 * j * GD_D), s[j]);
}

// Argument checks shared with the prefill form.
int gd_check(const bq_heads* q, const bq_heads* k, const bq_heads* v, const bq_heads* g, const bq_heads* beta,
             const float* state, const uint16_t* out, uint32_t heads_k, uint32_t heads_v, uint32_t head_dim,
             uint32_t slots, const char* who) {
    if (head_dim != GD_D) return fail(BQ_ERR_INVALID, "%s: head_dim %u, must be %d", who, head_dim, GD_D);
    if (heads_k == 0 || heads_v == 0 || heads_v % heads_k != 0 || heads_v > 65536)
        return fail(BQ_ERR_INVALID, "%s: heads_v %u must be a positive multiple of heads_k %u", who, heads_v, heads_k);
    if (!q || !k || !v || !g || !beta) return fail(BQ_ERR_INVALID, "%s: a tensor descriptor is NULL", who);
    const bq_heads* h[3] = {q, k, v};
    for (int i = 0; i < 3; i++) {
        if (!h[i]->data || !aligned16(h[i]->data))
            return fail(BQ_ERR_INVALID, "%s: %c must be non-NULL and 16-byte aligned", who, "qkv"[i]);
        if (h[i]->token_stride % 8 != 0 || h[i]->head_stride % 8 != 0 || h[i]->token_stride < 0 || h[i]->head_stride < 0)
            return fail(BQ_ERR_INVALID, "%s: strides of %c must be multiples of 8 and not negative", who, "qkv"[i]);
    }
    const bq_heads* f[2] = {g, beta};
    for (int i = 0; i < 2; i++) {
        const char* name = i ? "beta" : "g";
        if (!f[i]->data || !aligned4(f[i]->data))
            return fail(BQ_ERR_INVALID, "%s: %s must be non-NULL and 4-byte aligned", who, name);
        if (f[i]->token_stride < 0 || f[i]->head_stride < 0)
            return fail(BQ_ERR_INVALID, "%s: strides of %s must not be negative", who, name);
    }
    if (!state || !aligned16(state) || !out || !aligned16(out))
        return fail(BQ_ERR_INVALID, "%s: state and out must be non-NULL and 16-byte aligned", who);
    if (slots > (1u << 30)) return fail(BQ_ERR_INVALID, "%s: too many slots", who);
    return BQ_OK;
}

}  // namespace bq8

using namespace bq8;

extern "C" int gated_delta_decode(const bq_heads* q, const bq_heads* k, const bq_heads* v, const bq_heads* g,
                                  const bq_heads* beta, float* state, const int32_t* state_idx, uint16_t* out,
                                  uint32_t batch, uint32_t tokens, uint32_t heads_k, uint32_t heads_v, uint32_t head_dim,
                                  uint32_t slots, float scale, int l2norm, bq_stream_t stream) {
    const char* who = "gated_delta_decode";
    if (batch == 0 || tokens == 0) return ok();
    const int st = gd_check(q, k, v, g, beta, state, out, heads_k, heads_v, head_dim, slots, who);
    if (st) return st;
    if (!aligned4(state_idx)) return fail(BQ_ERR_INVALID, "%s: state_idx must be 4-byte aligned", who);
    if (!state_idx && slots < batch) return fail(BQ_ERR_INVALID, "%s: %u slots for a batch of %u", who, slots, batch);
    const uint64_t blocks = (uint64_t)batch * heads_v * (GD_D / GD_COLS);
    if (blocks >= (1ull << 31) || (uint64_t)batch * tokens >= (1ull << 31))
        return fail(BQ_ERR_INVALID, "%s: shape too large", who);
    GdArgs p = {*q,        *k,  *v, *g, *beta, state, state_idx, out, (int)tokens, (int)heads_k, (int)heads_v, (int)slots,
                scale, l2norm != 0};
    return launch_programmatic(who, gated_delta_decode_kernel, (uint32_t)blocks, 128, 0, (cudaStream_t)stream, p);
}
