// Append of a step's latent rows to a block-table paged cache, bf16 or E4M3:
//   y = x * rsqrt(mean_512(x^2) + eps) * w   (the 512 latent channels; y = x without w)
//   r = the 64 channels behind them rotated by the token's position (rope_dim 64)
//   cache row block_table[b][pos / page] * page + pos % page = round(y | r)
// and, in the same launch, the same rotation of the step's query heads into the
// rotated columns of the queries that the MLA takes.
//
// A rotated pair (x0, x1) becomes (x0 cos - x1 sin, x1 cos + x0 sin), cos and sin
// from the caller's fp32 table of positions: a table taken in 64 bits is right to
// the last bit at any position, where pos * frequency in 32 bits is off by
// pos * 2^-24 rad. All arithmetic is fp32 and rounded once, to the cache's type
// (a row is read as an operand of that type, so nothing finer would be used).
//
// Bound by bytes for a prompt's chunk and by the latency of one dependent chain
// for a decode step (position -> block table -> cos and sin -> store; the row's own
// loads depend on none of it and go out first). So: one warp a row, all of the row
// and its weights in flight before the first use, and one warp for every 16 query
// heads of a token, four 16-byte vectors a lane in flight. 48 registers keep five blocks on an SM
// (40 warps: a chunk's loads are what hides its latency; six warps a block row and 64
// registers took 8.2 us where this takes 6.7). One row with 16 heads and 64 rows with 128
// 2.1 and 2.6 us (the chain), 2048 tokens into E4M3 and 16336 rows of bf16 6.7 us (5.6 and 5.0
// TB/s).
#pragma once

#include "common.cuh"

namespace dsa {

constexpr int kAppendWarps = 8;
constexpr int kAppendBlocks = 5;                      // resident on an SM at least
constexpr int kAppendHeads = 16;                      // query heads a warp rotates
constexpr int kRopeDim = 64;                          // rotated channels, where there are any
constexpr int kRopeHalf = kRopeDim / 2;

struct AppendArgs {
    const __nv_bfloat16 *x;                           // [n] rows, x_stride elements apart
    int64_t x_stride;
    const __nv_bfloat16 *norm_w;                      // [512] or nullptr
    float eps;
    const float *cos_sin;                             // [max_pos][cos 32 | sin 32]
    int max_pos, interleaved;
    const int32_t *tok_req, *tok_pos;
    int n, rope;
    const int32_t *block_table;
    int B, max_blocks, page;
    void *cache;
    float inv_scale;                                  // E4M3: 1 / kv_scale
    int64_t kv_rows;
    const __nv_bfloat16 *q_in;                        // query heads, or nullptr
    int64_t q_tok_stride, q_head_stride;
    int Hm;
    __nv_bfloat16 *q_out;                             // [n][Hm][512 + rope]
};

// Two floats as an E4M3 pair, `lo` in the low byte; values beyond 448 saturate.
DSA_DEVINL uint16_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool kFp8>
__global__ void __launch_bounds__(kAppendWarps * 32, kAppendBlocks)
latent_append_kernel(const AppendArgs a) {
    // a warp a token; blockIdx.y 0: its row, p: its query heads 16 (p-1) .. + 15
    const int lane = threadIdx.x & 31, part = blockIdx.y;
    const long long i = (long long)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (i >= a.n) return;
    const int b = a.tok_req[i], pos = a.tok_pos[i];
    const int width = DSA_KV_LORA + a.rope;
    if (part == 0) {
        // ---- the latent row: lane l holds channels 8l .. 8l+7 and 256 + 8l .. + 7
        const __nv_bfloat16 *src = a.x + (size_t)i * a.x_stride;
        const uint4 u0 = *reinterpret_cast<const uint4 *>(src + 8 * lane);
        const uint4 u1 = *reinterpret_cast<const uint4 *>(src + 256 + 8 * lane);
        uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
        if (a.norm_w) {
            w0 = ldg_nc_v4(a.norm_w + 8 * lane);
            w1 = ldg_nc_v4(a.norm_w + 256 + 8 * lane);
        }
        float r0 = 0.f, r1 = 0.f;                    // the rotated pair of this lane
        if (a.rope) {
            const __nv_bfloat16 *pr = src + DSA_KV_LORA;
            r0 = __bfloat162float(pr[a.interleaved ? 2 * lane : lane]);
            r1 = __bfloat162float(pr[a.interleaved ? 2 * lane + 1 : kRopeHalf + lane]);
        }
        if (b < 0 || b >= a.B || pos < 0 || pos / a.page >= a.max_blocks) return;
        if (a.rope && pos >= a.max_pos) return;
        const int blk = a.block_table[(size_t)b * a.max_blocks + pos / a.page];
        if (blk < 0) return;
        const long long row = (long long)blk * a.page + pos % a.page;
        if (row >= a.kv_rows) return;
        float y[16];
        unpack8(u0, reinterpret_cast<float(&)[8]>(y[0]));
        unpack8(u1, reinterpret_cast<float(&)[8]>(y[8]));
        if (a.norm_w) {
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) ss = fmaf(y[k], y[k], ss);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float rstd = rsqrtf(ss * (1.0f / DSA_KV_LORA) + a.eps);
            const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                y[2 * k] = y[2 * k] * rstd * bf16lo(w[k]);
                y[2 * k + 1] = y[2 * k + 1] * rstd * bf16hi(w[k]);
            }
        }
        if (a.rope) {
            const float c = __ldg(a.cos_sin + (size_t)pos * kRopeDim + lane);
            const float s = __ldg(a.cos_sin + (size_t)pos * kRopeDim + kRopeHalf + lane);
            const float t0 = r0 * c - r1 * s, t1 = r1 * c + r0 * s;
            r0 = t0;
            r1 = t1;
        }
        if constexpr (!kFp8) {
            __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(a.cache) + (size_t)row * width;
            *reinterpret_cast<uint4 *>(dst + 8 * lane) =
                make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                           pack_bf16x2(y[6], y[7]));
            *reinterpret_cast<uint4 *>(dst + 256 + 8 * lane) =
                make_uint4(pack_bf16x2(y[8], y[9]), pack_bf16x2(y[10], y[11]),
                           pack_bf16x2(y[12], y[13]), pack_bf16x2(y[14], y[15]));
            if (a.rope) {
                __nv_bfloat16 *dr = dst + DSA_KV_LORA;
                if (a.interleaved) {
                    *reinterpret_cast<uint32_t *>(dr + 2 * lane) = pack_bf16x2(r0, r1);
                } else {
                    dr[lane] = __float2bfloat16_rn(r0);
                    dr[kRopeHalf + lane] = __float2bfloat16_rn(r1);
                }
            }
        } else {
            uint8_t *dst = reinterpret_cast<uint8_t *>(a.cache) + (size_t)row * width;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float *v = y + 8 * h + 4 * k;
                    w[k] = (uint32_t)pack_e4m3x2(v[0] * a.inv_scale, v[1] * a.inv_scale) |
                           ((uint32_t)pack_e4m3x2(v[2] * a.inv_scale, v[3] * a.inv_scale) << 16);
                }
                *reinterpret_cast<uint2 *>(dst + 256 * h + 8 * lane) = make_uint2(w[0], w[1]);
            }
            if (a.rope) {
                uint8_t *dr = dst + DSA_KV_LORA;
                const uint16_t p = pack_e4m3x2(r0 * a.inv_scale, r1 * a.inv_scale);
                if (a.interleaved) {
                    *reinterpret_cast<uint16_t *>(dr + 2 * lane) = p;
                } else {
                    dr[lane] = (uint8_t)(p & 0xFFu);
                    dr[kRopeHalf + lane] = (uint8_t)(p >> 8);
                }
            }
        }
        return;
    }
    // ---- query heads 16 (part-1) .. + 15 of token i: eight lanes a head, 8 channels a lane
    const int j = lane & 7;
    const int h0 = (part - 1) * kAppendHeads + (lane >> 3);
    uint4 u[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int h = h0 + 4 * t;
        u[t] = h < a.Hm ? *reinterpret_cast<const uint4 *>(a.q_in + (size_t)i * a.q_tok_stride +
                                                           (size_t)h * a.q_head_stride + 8 * j)
                        : make_uint4(0u, 0u, 0u, 0u);
    }
    if (b < 0 || b >= a.B || pos < 0 || pos >= a.max_pos) return;
    const float *cs = a.cos_sin + (size_t)pos * kRopeDim;
    float out[8];
    if (a.interleaved) {
        const float4 c = __ldg(reinterpret_cast<const float4 *>(cs + 4 * j));
        const float4 s = __ldg(reinterpret_cast<const float4 *>(cs + kRopeHalf + 4 * j));
        const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            float v[8];
            unpack8(u[t], v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                out[2 * k] = v[2 * k] * cc[k] - v[2 * k + 1] * sn[k];
                out[2 * k + 1] = v[2 * k + 1] * cc[k] + v[2 * k] * sn[k];
            }
            u[t] = make_uint4(pack_bf16x2(out[0], out[1]), pack_bf16x2(out[2], out[3]),
                              pack_bf16x2(out[4], out[5]), pack_bf16x2(out[6], out[7]));
        }
    } else {
        // lane j < 4 of a head holds first halves, its partner j + 4 the second halves
        float cc[8], sn[8];
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            const float4 c = __ldg(reinterpret_cast<const float4 *>(cs + 8 * (j & 3) + k));
            const float4 s = __ldg(reinterpret_cast<const float4 *>(cs + kRopeHalf + 8 * (j & 3) + k));
            cc[k] = c.x; cc[k + 1] = c.y; cc[k + 2] = c.z; cc[k + 3] = c.w;
            sn[k] = s.x; sn[k + 1] = s.y; sn[k + 2] = s.z; sn[k + 3] = s.w;
        }
        const float sign = j < 4 ? -1.f : 1.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            float v[8];
            unpack8(u[t], v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float o = __shfl_xor_sync(0xffffffffu, v[k], 4);
                out[k] = v[k] * cc[k] + sign * (o * sn[k]);
            }
            u[t] = make_uint4(pack_bf16x2(out[0], out[1]), pack_bf16x2(out[2], out[3]),
                              pack_bf16x2(out[4], out[5]), pack_bf16x2(out[6], out[7]));
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int h = h0 + 4 * t;
        if (h < a.Hm)
            *reinterpret_cast<uint4 *>(a.q_out + ((size_t)i * a.Hm + h) * width + DSA_KV_LORA + 8 * j) = u[t];
    }
}

template <bool kFp8>
inline int latent_append_launch(AppendArgs a, float kv_scale, int kv_lora, cudaStream_t stream) {
    if (a.n < 0 || kv_lora <= 0 || a.rope < 0 || a.B < 0 || a.max_blocks < 0 || a.page <= 0 ||
        a.kv_rows < 0 || a.max_pos < 0 || a.Hm < 0 || !(a.eps >= 0.f && a.eps < INFINITY))
        return DSA_ERR_INVALID_ARG;
    if (kFp8 && !(kv_scale > 0.f && kv_scale < INFINITY)) return DSA_ERR_INVALID_ARG;
    a.inv_scale = kFp8 ? 1.0f / kv_scale : 1.0f;
    if (!(a.inv_scale < INFINITY)) return DSA_ERR_INVALID_ARG;
    if (kv_lora != DSA_KV_LORA || (a.rope != 0 && a.rope != kRopeDim)) return DSA_ERR_UNSUPPORTED;
    const int width = DSA_KV_LORA + a.rope;
    const bool heads = a.q_in != nullptr || a.q_out != nullptr;
    if (a.x_stride < width || (a.rope && a.interleaved != 0 && a.interleaved != 1))
        return DSA_ERR_INVALID_ARG;
    if (heads && (!a.q_in || !a.q_out || !a.rope || a.Hm == 0 || a.q_head_stride < a.rope ||
                  a.q_tok_stride < (int64_t)(a.Hm - 1) * a.q_head_stride + a.rope))
        return DSA_ERR_INVALID_ARG;
    if (heads && a.Hm > DSA_MAX_MLA_HEADS) return DSA_ERR_UNSUPPORTED;
    if (a.n == 0 || a.B == 0) return DSA_OK;
    if (!a.x || !a.tok_req || !a.tok_pos || (a.max_blocks > 0 && !a.block_table) ||
        (a.kv_rows > 0 && !a.cache) || (a.rope && a.max_pos > 0 && !a.cos_sin))
        return DSA_ERR_INVALID_ARG;
    if (!aligned(a.x, 16) || a.x_stride % 8 || !aligned(a.norm_w, 16) || !aligned(a.cos_sin, 16) ||
        !aligned(a.tok_req, 4) || !aligned(a.tok_pos, 4) || !aligned(a.block_table, 4) ||
        !aligned(a.cache, 16) || !aligned(a.q_in, 16) || !aligned(a.q_out, 16) ||
        (heads && (a.q_tok_stride % 8 || a.q_head_stride % 8)))
        return DSA_ERR_ALIGNMENT;
    const int parts = 1 + (heads ? ceil_div(a.Hm, kAppendHeads) : 0);
    if (launch_pdl(latent_append_kernel<kFp8>, dim3(ceil_div(a.n, kAppendWarps), parts),
                   dim3(kAppendWarps * 32), 0, stream, a) != cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_status();
}

}  // namespace dsa
