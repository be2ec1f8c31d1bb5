// Causal GQA attention of ragged chunks of new rows over a caller's paged KV cache.
//
// Sequence b has rows cu[b] .. cu[b + 1] - 1 of q and kv_len[b] cache rows, its own new
// rows last: row i of its n rows sits at position p = kv_len[b] - n + i and sees keys
// max(0, p - W + 1) .. p (W = window, all of 0 .. p without one) whose page lies in the pool:
//   out[r][h] = sum_j softmax_j(c(q[r][h] . K[j] scale)) V[j],  c(s) = cap tanh(s / cap).
// A row that sees no key gives zeros.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <exception>
#include <string>

#include "../../include/dec_api.h"
#include "common.cuh"
#include "kernels.h"

namespace dec {
namespace {

constexpr int kPage = 16;

dec_status bad(dec_status s, const std::string& why) {
    set_last_error(why);
    return s;
}

struct ChunkArgs {
    const uint16_t* q;
    long long ldq;
    const uint16_t* k_pool;
    const uint16_t* v_pool;
    int n_pages;
    const int32_t* table;
    int max_pages;
    const int32_t* cu;
    const int32_t* kv_len;
    int B, T, nq, nkv;
    float scale;
    int window;
    float cap;
    uint16_t* out;
};

// One CTA a (row, kv head): four warps take every fourth key, each for all G query heads.
template <int D>
__global__ void __launch_bounds__(128) chunk_attn_kernel(ChunkArgs a) {
    constexpr int N = D / 32;
    const int t = blockIdx.x, g = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.nq / a.nkv;
    if (t < a.cu[0] || t >= a.cu[a.B]) return;
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int b = lo;
    const int len = min(max(a.kv_len[b], 0), a.max_pages * kPage);
    const int p = len - (a.cu[b + 1] - t);
    const int first = a.window > 0 ? max(0, p + 1 - a.window) : 0;
    float m[16], l[16], o[16][N], q[16][N];
#pragma unroll
    for (int h = 0; h < 16; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int c = 0; c < N; ++c) {
            o[h][c] = 0.f;
            q[h][c] = h < G ? bf2f(a.q[(size_t)t * a.ldq + (size_t)(g * G + h) * D + lane + 32 * c]) : 0.f;
        }
    }
    for (int j = first + warp; j <= p; j += 4) {
        const int page = a.table[(size_t)b * a.max_pages + j / kPage];
        if (page < 0 || page >= a.n_pages) continue;
        const size_t at = (((size_t)page * a.nkv + g) * kPage + j % kPage) * D + lane;
        float k[N], v[N];
#pragma unroll
        for (int c = 0; c < N; ++c) {
            k[c] = bf2f(a.k_pool[at + 32 * c]);
            v[c] = bf2f(a.v_pool[at + 32 * c]);
        }
#pragma unroll
        for (int h = 0; h < 16; ++h) {
            if (h >= G) break;
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < N; ++c) s += q[h][c] * k[c];
            s = warp_sum(s) * a.scale;
            if (a.cap > 0.f) s = a.cap * tanhf(s / a.cap);
            if (s > m[h]) {
                const float f = expf(m[h] - s);
                l[h] *= f;
#pragma unroll
                for (int c = 0; c < N; ++c) o[h][c] *= f;
                m[h] = s;
            }
            const float e = m[h] == -INFINITY ? 0.f : expf(s - m[h]);
            l[h] += e;
#pragma unroll
            for (int c = 0; c < N; ++c) o[h][c] += e * v[c];
        }
    }
    __shared__ float sm[4][16], sl[4][16], so[4][16][D];
#pragma unroll
    for (int h = 0; h < 16; ++h) {
        if (lane == 0) {
            sm[warp][h] = m[h];
            sl[warp][h] = l[h];
        }
#pragma unroll
        for (int c = 0; c < N; ++c) so[warp][h][lane + 32 * c] = o[h][c];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += 128) {
        const int h = i / D, c = i % D;
        const float M = fmaxf(fmaxf(sm[0][h], sm[1][h]), fmaxf(sm[2][h], sm[3][h]));
        float L = 0.f, O = 0.f;
        for (int w = 0; w < 4; ++w) {
            const float f = M == -INFINITY || sm[w][h] == -INFINITY ? 0.f : expf(sm[w][h] - M);
            L += f * sl[w][h];
            O += f * so[w][h][c];
        }
        a.out[((size_t)t * a.nq + g * G + h) * D + c] = f2bf(L > 0.f || L != L ? O / L : 0.f);
    }
}

}  // namespace
}  // namespace dec

using namespace dec;

extern "C" {

int64_t gqa_chunk_attn_workspace(int32_t d) { return d == 64 || d == 128 ? 16 : 0; }

dec_status gqa_chunk_attn(const void* q, int64_t ldq, const void* k_pool, const void* v_pool, int32_t n_pages,
                          const int32_t* block_table, int32_t max_pages, const int32_t* cu_rows,
                          const int32_t* kv_len, int32_t B, int32_t T, int32_t nq, int32_t nkv, int32_t d,
                          int32_t page_size, float scale, int32_t window, float softcap, void* out, void* workspace,
                          int64_t workspace_bytes, dec_stream_t stream) try {
    set_last_error("");
    if (!k_pool || !v_pool || !block_table || !cu_rows || !kv_len || !workspace)
        return bad(DEC_ERR_INVALID_ARG, "NULL pointer");
    if (T > 0 && (!q || !out)) return bad(DEC_ERR_INVALID_ARG, "NULL pointer");
    if (B <= 0 || T < 0 || nq <= 0 || nkv <= 0 || nq % nkv != 0 || max_pages <= 0 || n_pages <= 0)
        return bad(DEC_ERR_INVALID_ARG, "bad B / T / heads / pages");
    if (!(scale > 0.f) || !(scale < INFINITY)) return bad(DEC_ERR_INVALID_ARG, "scale must be positive and finite");
    if (window < 0 || !(softcap >= 0.f) || !(softcap < INFINITY))
        return bad(DEC_ERR_INVALID_ARG, "window and softcap must not be negative");
    if (nq / nkv > 16) return bad(DEC_ERR_UNSUPPORTED, "more than 16 q heads per kv head");
    if (d != 64 && d != 128) return bad(DEC_ERR_UNSUPPORTED, "d must be 64 or 128");
    if (page_size != kPage) return bad(DEC_ERR_UNSUPPORTED, "page_size must be 16");
    if (B > 4096) return bad(DEC_ERR_UNSUPPORTED, "more than 4096 sequences");
    if (max_pages > (1 << 30) / kPage || T > (1 << 30))
        return bad(DEC_ERR_UNSUPPORTED, "positions and rows must stay below 2^30");
    if ((int64_t)n_pages * nkv > INT32_MAX / kPage) return bad(DEC_ERR_UNSUPPORTED, "pool rows must fit 32 bits");
    if (ldq < (int64_t)nq * d) return bad(DEC_ERR_INVALID_ARG, "ldq is smaller than a row");
    if (ldq % 8 != 0) return bad(DEC_ERR_UNSUPPORTED, "ldq must be a multiple of 8");
    if (((uintptr_t)q | (uintptr_t)k_pool | (uintptr_t)v_pool | (uintptr_t)out | (uintptr_t)workspace) % 16 != 0)
        return bad(DEC_ERR_UNSUPPORTED, "q, the pools, out and the workspace must be 16-byte aligned");
    if (workspace_bytes < gqa_chunk_attn_workspace(d)) return bad(DEC_ERR_INVALID_ARG, "workspace too small");
    if (T == 0) return DEC_OK;
    ChunkArgs a{static_cast<const uint16_t*>(q), ldq, static_cast<const uint16_t*>(k_pool),
                static_cast<const uint16_t*>(v_pool), n_pages, block_table, max_pages, cu_rows, kv_len, B, T, nq, nkv,
                scale, window, softcap, static_cast<uint16_t*>(out)};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d == 128)
        chunk_attn_kernel<128><<<dim3(T, nkv), 128, 0, st>>>(a);
    else
        chunk_attn_kernel<64><<<dim3(T, nkv), 128, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return bad(DEC_ERR_CUDA, std::string("gqa_chunk_attn: ") + cudaGetErrorString(e));
    return DEC_OK;
} catch (const std::exception&) {
    return DEC_ERR_OOM;
}

}  // extern "C"
