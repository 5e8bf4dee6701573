// Dense MLA over a block-table paged latent cache for a batch whose requests
// share a prefix ("spark_model/layers/glm5next_dsa/mod.rs": the serve path's
// block-table paged MLA decode, walking 0..seq_len instead of a selected-index
// row). Plain form: one warp per (query, head), online softmax over the tokens.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "latent_append.cuh"

namespace dsa {

struct PrefixGeom {
    const int32_t *prefix_table;      // pages of the shared prefix
    const int32_t *prefix_len;        // [1] tokens of it
    const int32_t *block_table;       // [B, max_blocks] pages of each request
    const int32_t *seq_len, *q_req, *q_pos;
    int prefix_blocks, max_blocks, page, Q, B;
    int kv_rows;

    // Tokens of the prefix that its pages can hold.
    DSA_DEVINL int shared_len() const {
        if (prefix_blocks == 0) return 0;
        const long long cap = (long long)prefix_blocks * page;
        return (int)max(0ll, min((long long)prefix_len[0], min(cap, (long long)INT32_MAX)));
    }
    // Tokens 0 .. n-1 that query q sees; no more than its pages can hold.
    DSA_DEVINL int visible(int q, int P) const {
        const int b = q_req[q];
        if (b < 0 || b >= B) return 0;
        const long long n = min((long long)q_pos[q] + 1, (long long)seq_len[b]);
        const long long cap = max((long long)P, min((long long)max_blocks * page, (long long)INT32_MAX));
        return (int)max(0ll, min(n, cap));
    }
    // Cache row of token t of request b, -1 where there is none.
    DSA_DEVINL int row(int b, int t, int P) const {
        const int bi = t / page;
        int blk;
        if (t < P) {
            blk = __ldg(prefix_table + bi);
        } else {
            if (bi >= max_blocks) return -1;
            blk = __ldg(block_table + (size_t)b * max_blocks + bi);
        }
        if (blk < 0) return -1;
        const long long r = (long long)blk * page + (t - bi * page);
        return r < (long long)kv_rows ? (int)r : -1;
    }
};

template <bool kFp8>
__global__ void __launch_bounds__(128)
prefix_mla_plain_kernel(const __nv_bfloat16 *__restrict__ q, const void *__restrict__ kv,
                        const PrefixGeom g, int Hm, int rope, float scale_log2, float out_scale,
                        __nv_bfloat16 *__restrict__ out, float *__restrict__ lse) {
    const int lane = threadIdx.x & 31;
    const long long task = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (task >= (long long)g.Q * Hm) return;
    const int qi = (int)(task / Hm);
    const int width = DSA_KV_LORA + rope;
    const int P = g.shared_len(), n = g.visible(qi, P), b = g.q_req[qi];
    float qv[18], o[16];
    const __nv_bfloat16 *qr = q + (size_t)task * width;
    for (int k = 0; k < 16; ++k) { qv[k] = __bfloat162float(qr[32 * k + lane]); o[k] = 0.f; }
    for (int k = 0; k < 2; ++k) qv[16 + k] = rope ? __bfloat162float(qr[512 + 32 * k + lane]) : 0.f;
    float m = -INFINITY, l = 0.f;
    for (int t = 0; t < n; ++t) {
        const int row = g.row(b, t, P);
        if (row < 0) continue;
        float v[18], z = 0.f;
        for (int k = 0; k < 18; ++k) {
            if (k >= 16 && !rope) { v[k] = 0.f; continue; }
            const size_t at = (size_t)row * width + 32 * k + lane;
            if constexpr (kFp8) {
                uint32_t h2;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)reinterpret_cast<const uint8_t *>(kv)[at]));
                v[k] = __half2float(__ushort_as_half((uint16_t)(h2 & 0xFFFFu)));
            } else {
                v[k] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(kv)[at]);
            }
            z = fmaf(qv[k], v[k], z);
        }
        for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
        z *= scale_log2;
        const float mn = fmaxf(m, z);
        const float al = m == -INFINITY ? 0.f : ex2(m - mn), p = z == -INFINITY ? 0.f : ex2(z - mn);
        l = l * al + p;
        for (int k = 0; k < 16; ++k) o[k] = o[k] * al + p * v[k];
        m = mn;
    }
    const float inv = l != 0.f ? out_scale / l : 0.f;
    for (int k = 0; k < 16; ++k)
        out[(size_t)task * 512 + 32 * k + lane] = __float2bfloat16_rn(l != 0.f ? o[k] * inv : 0.f);
    if (lse && lane == 0) lse[task] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

inline size_t prefix_mla_workspace_bytes(int Q, int Hm) { return Q > 0 && Hm > 0 ? 16 : 0; }

template <bool kFp8>
inline int prefix_mla_launch(const void *q, const void *kv, float kv_scale, int64_t kv_rows,
                             PrefixGeom g, int Hm, int kv_lora, int rope, float sm_scale, void *out,
                             float *lse, void *ws, size_t ws_bytes, cudaStream_t stream) {
    if (g.Q < 0 || g.B < 0 || Hm <= 0 || kv_lora <= 0 || rope < 0 || kv_rows < 0 || g.page <= 0 ||
        g.max_blocks < 0 || g.prefix_blocks < 0)
        return DSA_ERR_INVALID_ARG;
    if (!(sm_scale == sm_scale) || sm_scale == INFINITY || sm_scale == -INFINITY)
        return DSA_ERR_INVALID_ARG;
    if (kFp8 && !(kv_scale > 0.f && kv_scale < INFINITY)) return DSA_ERR_INVALID_ARG;
    if (kv_lora != DSA_KV_LORA || (rope != 0 && rope != kRopeDim) || Hm % 16 != 0 ||
        Hm > DSA_MAX_MLA_HEADS)
        return DSA_ERR_UNSUPPORTED;
    if (kv_rows > (int64_t)INT32_MAX || g.Q > 65535) return DSA_ERR_UNSUPPORTED;
    if (g.Q == 0) return DSA_OK;
    if (!q || !g.q_req || !g.q_pos || !out || (kv_rows > 0 && !kv) || (g.B > 0 && !g.seq_len) ||
        (g.B > 0 && g.max_blocks > 0 && !g.block_table) ||
        (g.prefix_blocks > 0 && (!g.prefix_table || !g.prefix_len)))
        return DSA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(g.prefix_table, 4) ||
        !aligned(g.prefix_len, 4) || !aligned(g.block_table, 4) || !aligned(g.seq_len, 4) ||
        !aligned(g.q_req, 4) || !aligned(g.q_pos, 4) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(ws, 16))
        return DSA_ERR_ALIGNMENT;
    if (!ws || ws_bytes < prefix_mla_workspace_bytes(g.Q, Hm)) return DSA_ERR_WORKSPACE;
    g.kv_rows = (int)kv_rows;
    const float scale_log2 = (kFp8 ? sm_scale * kv_scale : sm_scale) * 1.4426950408889634f;
    const long long blocks = ((long long)g.Q * Hm + 3) / 4;
    if (launch_pdl(prefix_mla_plain_kernel<kFp8>, dim3((unsigned)blocks), dim3(128), 0, stream,
                   reinterpret_cast<const __nv_bfloat16 *>(q), kv, g, Hm, rope, scale_log2,
                   kFp8 ? kv_scale : 1.0f, reinterpret_cast<__nv_bfloat16 *>(out), lse) != cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_status();
}

}  // namespace dsa
