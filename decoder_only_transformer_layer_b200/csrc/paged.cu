// The bookkeeping of a paged KV cache whose pool and block table belong to the caller:
// paged_resize (block table, free list and slot map from sequence lengths) and
// paged_rope_append (QK-norm, RoPE and the store of a step's k and v rows in their slots).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
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

// ================================================================== paged_resize
//
// With held_b = ceil(old_b / 16) and want_b = ceil(new_b / 16), sequence b takes
// max(want_b - held_b, 0) pages and gives back max(held_b - want_b, 0). Three exclusive
// prefix sums over the sequences (new rows, pages taken, pages given back) place every
// row and every page, so all of them are then written independently:
//   i-th page taken      = free[F - 1 - i]             (F pages free before the call)
//   k-th page given back -> free[F - A + R - 1 - k]    (A taken, R given back)
//   row t of sequence b  : position p = old_b + (t - cu_b), slot 16 page(p) + p % 16
// both counted in the order (sequence, page). The given-back pages are stacked in
// reverse, so resizing back restores the free list and the table exactly.
// One cluster does the pages: every CTA scans the lengths for itself (no exchange), the
// pages are spread over the cluster's threads, and cluster barriers separate checking
// from writing, and reading the free list from stacking on it. A few thousand rows are
// spread over it too; more rows have a kernel of their own on all SMs, which reads the
// finished table (a 100,000-row step took 23 us with the rows in the cluster of 8 CTAs).
// Latency is the bound: a few dependent memory round trips and the barriers. 64 sequences
// decoding take 5 us, 500 sequences with 97,000 new rows 12.

constexpr int kRzThreads = 1024;
constexpr int kRzMaxB = 4096;  // prefix sums: 3 x 4097 int32 of shared memory
constexpr int kRzPer = kRzMaxB / kRzThreads;
constexpr int kRzRows = 4096;    // most rows that the cluster places itself

struct ResizeArgs {
    const int32_t* old_len;
    const int32_t* new_len;
    int B;
    int32_t* table;
    int max_pages;
    int32_t* free_pages;
    int n_pages;
    int32_t* n_free;
    int32_t* cu_rows;
    int32_t* slot;
    int32_t* row_pos;
    int T;
    int32_t* status;
    bool rows_here;  // the rows are placed here, not by paged_slots_kernel
};

DEC_DEVINL int page_count(int len) { return len / kPage + (len % kPage != 0); }

// The largest b with pre[b] <= i, for pre ascending from 0 over B + 1 entries, i < pre[B].
DEC_DEVINL int find_seq(const int32_t* pre, int B, int i) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kRzThreads) paged_resize_kernel(ResizeArgs a) {
    extern __shared__ int32_t rz_smem[];
    int32_t* cu = rz_smem;             // [B + 1] new rows before sequence b
    int32_t* tk = cu + a.B + 1;        // [B + 1] pages taken before it
    int32_t* gv = tk + a.B + 1;        // [B + 1] pages given back before it
    __shared__ long long part[3][33];  // warp totals, then their exclusive sums and the total
    __shared__ int flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank(), C = gridDim.x;  // the grid is one cluster
    const int gtid = rank * kRzThreads + tid, gn = C * kRzThreads;
    if (!a.rows_here) pdl_trigger();
    if (tid == 0) flag = 0;
    // the matching wait comes before the first store to another CTA's flag
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    // ---- scan: thread t owns sequences t * per .. t * per + per - 1
    const int per = (a.B + kRzThreads - 1) / kRzThreads;
    const int F = *a.n_free;
    const long long cap = (long long)a.max_pages * kPage;
    long long v[3] = {0, 0, 0};
    int rows[kRzPer], take[kRzPer], give[kRzPer];
    int st = F < 0 || F > a.n_pages ? 1 : 0;
    int over = 0;
#pragma unroll
    for (int k = 0; k < kRzPer; ++k) {
        rows[k] = take[k] = give[k] = 0;
        const int b = tid * per + k;
        if (k < per && b < a.B) {
            const int o = a.old_len[b], n = a.new_len[b];
            if (o < 0 || n < 0) {
                st = 1;
            } else {
                if (o > cap || n > cap) over = 1;
                const int d = page_count(n) - page_count(o);
                rows[k] = n > o ? n - o : 0;
                take[k] = d > 0 ? d : 0;
                give[k] = d < 0 ? -d : 0;
            }
        }
        v[0] += rows[k];
        v[1] += take[k];
        v[2] += give[k];
    }
    st = __syncthreads_or(st);
    over = __syncthreads_or(over);
    long long x[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        x[j] = v[j];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x[j], o);
            if (lane >= o) x[j] += y;
        }
        if (lane == 31) part[j][warp] = x[j];
    }
    __syncthreads();
    if (warp < 3) {
        const long long w = part[warp][lane];
        long long s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        part[warp][lane] = s - w;
        if (lane == 31) part[warp][32] = s;
    }
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const long long n_rows = part[0][32], A = part[1][32], R = part[2][32];
    if (n_rows > a.T || F - A + R > a.n_pages) st = 1;
    int code = st ? DEC_ERR_INVALID_ARG
                  : over ? DEC_ERR_CONTEXT_OVERFLOW : A > F ? DEC_ERR_PAGES_EXHAUSTED : DEC_OK;

    if (code == DEC_OK) {
        long long p0 = part[0][warp] + x[0] - v[0], p1 = part[1][warp] + x[1] - v[1], p2 = part[2][warp] + x[2] - v[2];
#pragma unroll
        for (int k = 0; k < kRzPer; ++k) {
            const int b = tid * per + k;
            if (k < per && b < a.B) {
                cu[b] = (int)p0;
                tk[b] = (int)p1;
                gv[b] = (int)p2;
            }
            p0 += rows[k];
            p1 += take[k];
            p2 += give[k];
        }
        if (tid == 0) {
            cu[a.B] = (int)n_rows;
            tk[a.B] = (int)A;
            gv[a.B] = (int)R;
        }
        __syncthreads();
        // ---- every page that changes hands lies in the pool, or nothing is changed
        int wrong = 0;
        for (int i = gtid; i < (int)A; i += gn) {
            const int pg = a.free_pages[F - 1 - i];
            wrong |= pg < 0 || pg >= a.n_pages;
        }
        for (int k = gtid; k < (int)R; k += gn) {
            const int b = find_seq(gv, a.B, k);
            const int pg = a.table[(size_t)b * a.max_pages + page_count(a.new_len[b]) + (k - gv[b])];
            wrong |= pg < 0 || pg >= a.n_pages;
        }
        if (__syncthreads_or(wrong) && tid < C)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_map(smem_u32(&flag), tid)), "r"(1) : "memory");
    }
    cluster_sync();  // every CTA reaches it: the code so far is the same in all of them
    if (flag) code = DEC_ERR_INVALID_ARG;

    if (code != DEC_OK) {
        for (int i = gtid; a.rows_here && i < a.T; i += gn) a.slot[i] = a.row_pos[i] = -1;
        for (int b = gtid; b <= a.B; b += gn) a.cu_rows[b] = 0;
        if (gtid == 0) *a.status = code;
        return;
    }
    for (int b = gtid; b <= a.B; b += gn) a.cu_rows[b] = cu[b];
    for (int i = gtid; a.rows_here && i < a.T; i += gn) {
        int slot = -1, p = -1;
        if (i < (int)n_rows) {
            const int b = find_seq(cu, a.B, i);
            p = a.old_len[b] + (i - cu[b]);
            const int held = page_count(a.old_len[b]), pi = p / kPage;
            const int pg = pi < held ? a.table[(size_t)b * a.max_pages + pi] : a.free_pages[F - 1 - (tk[b] + pi - held)];
            if (pg >= 0 && pg < a.n_pages) slot = pg * kPage + p % kPage;
        }
        a.slot[i] = slot;
        a.row_pos[i] = p;
    }
    for (int i = gtid; i < (int)A; i += gn) {
        const int b = find_seq(tk, a.B, i);
        a.table[(size_t)b * a.max_pages + page_count(a.old_len[b]) + (i - tk[b])] = a.free_pages[F - 1 - i];
    }
    cluster_sync();  // the free list has been read (and no CTA reads another's shared memory from here)
    for (int k = gtid; k < (int)R; k += gn) {
        const int b = find_seq(gv, a.B, k);
        int32_t* e = a.table + (size_t)b * a.max_pages + page_count(a.new_len[b]) + (k - gv[b]);
        a.free_pages[F - (int)A + (int)R - 1 - k] = *e;
        *e = -1;
    }
    if (gtid == 0) {
        *a.n_free = F - (int)A + (int)R;
        *a.status = DEC_OK;
    }
}

// Slots and positions of the rows, from the table that paged_resize_kernel left (row starts of 0
// after a failure: no rows).
__global__ void __launch_bounds__(256) paged_slots_kernel(ResizeArgs a) {
    pdl_wait();
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= a.T) return;
    int slot = -1, p = -1;
    if (i < a.cu_rows[a.B]) {
        const int b = find_seq(a.cu_rows, a.B, i);
        p = a.old_len[b] + (i - a.cu_rows[b]);
        const int pg = a.table[(size_t)b * a.max_pages + p / kPage];
        if (pg >= 0 && pg < a.n_pages) slot = pg * kPage + p % kPage;
    }
    a.slot[i] = slot;
    a.row_pos[i] = p;
}

// ================================================================== paged_rope_append
//
// Row t of the fp32 QKV projection holds nq q heads, nkv k heads, nkv v heads of d values.
// q and k heads are (optionally) RMS-normalised with a gain, then rotated: with
// c = cos(p theta_i), s = sin(p theta_i), theta_i = base^(-2 i / d),
//   y_i = x_i c - x_{i + d/2} s,   y_{i + d/2} = x_{i + d/2} c + x_i s,
// in fp32, and rounded once to bf16. v is rounded as it is. HBM is the bound: 4 bytes
// read and 2 written for each value; 8192 rows of 32/8 heads of 128 (302 MB) take 49 us alone, 57
// in a row of calls (5.3 TB/s), 32 rows 2.4 us.

struct AppendArgs {
    const float* qkv;
    long long ld;
    const float* q_norm;
    const float* k_norm;
    float eps;
    float base;
    const int32_t* slot;
    const int32_t* row_pos;
    int T, nq, nkv;
    uint16_t* q_out;
    uint16_t* k_pool;
    uint16_t* v_pool;
    int n_slots;
    bool aligned;  // qkv's rows begin on 16 bytes
};

//
// A block takes row after row (a grid of what the SMs hold at once); D / 8 lanes a head, each with
// two runs of four values d / 2 apart, so every load is 16 bytes and every pair is in one lane. The
// angles are fp64 in turns (p theta / 2 pi, reduced to [-1/2, 1/2]; theta by one pow a block), one
// sine and cosine a pair and row, shared by all heads through shared memory.

constexpr int kApThreads = 256;

template <int D>
__global__ void __launch_bounds__(kApThreads, 4) paged_rope_append_kernel(AppendArgs a) {
    constexpr int H = D / 2, LH = D / 8;     // lanes of a head
    constexpr int kAtOnce = kApThreads / LH;  // heads a block has in hand
    __shared__ float2 cs[2][H];               // (cos, sin) of the row, double-buffered
    const int tid = threadIdx.x, sub = tid % LH, head0 = tid / LH;
    double turns = 0.0;  // theta_i / 2 pi
    if (tid < H) turns = pow((double)a.base, -2.0 * tid / D) * 0.15915494309189533577;
    pdl_wait();     // the power above ran beside the last kernel in the stream
    pdl_trigger();
    const int heads = a.nq + 2 * a.nkv;
    float4 gq0, gq1, gk0, gk1;
    if (a.q_norm) gq0 = *reinterpret_cast<const float4*>(a.q_norm + 4 * sub), gq1 = *reinterpret_cast<const float4*>(a.q_norm + H + 4 * sub);
    if (a.k_norm) gk0 = *reinterpret_cast<const float4*>(a.k_norm + 4 * sub), gk1 = *reinterpret_cast<const float4*>(a.k_norm + H + 4 * sub);
    int buf = 0;
    // the values of the head in hand next: of this row, or after its last head of the next row
    float4 x, y;
    bool loaded = false;
    auto load = [&](int t, int h) {
        if (h >= heads) return;
        const float* src = a.qkv + (size_t)t * a.ld + (size_t)h * D + 4 * sub;
        if (a.aligned) {
            x = __ldcs(reinterpret_cast<const float4*>(src));
            y = __ldcs(reinterpret_cast<const float4*>(src + H));
        } else {
            x = make_float4(src[0], src[1], src[2], src[3]);
            y = make_float4(src[H], src[H + 1], src[H + 2], src[H + 3]);
        }
    };
    int next_slot = a.slot[blockIdx.x], next_p = a.row_pos[blockIdx.x];  // the grid has at most T blocks
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int slot = next_slot, p = next_p;
        if (t + (int)gridDim.x < a.T) {  // asked for a row ahead
            next_slot = a.slot[t + gridDim.x];
            next_p = a.row_pos[t + gridDim.x];
        }
        if (slot < 0 || slot >= a.n_slots) continue;  // the whole block
        if (!loaded) load(t, head0);
        loaded = false;
        if (tid < H) {
            const double r = (double)p * turns, f = r - rint(r);
            float c, s;
            sincospif((float)(2.0 * f), &s, &c);
            cs[buf][tid] = make_float2(c, s);
        }
        __syncthreads();
        const float4 cs01 = *reinterpret_cast<const float4*>(&cs[buf][4 * sub]);
        const float4 cs23 = *reinterpret_cast<const float4*>(&cs[buf][4 * sub + 2]);
        buf ^= 1;
        const size_t page = slot / kPage, off = slot % kPage;
        for (int h = head0; h < heads; h += kAtOnce) {
            float4 u = x, v = y;
            if (h + kAtOnce < heads) {
                load(t, h + kAtOnce);
            } else if (t + (int)gridDim.x < a.T && next_slot >= 0 && next_slot < a.n_slots) {
                load(t + gridDim.x, head0);
                loaded = true;
            }
            const bool isq = h < a.nq, isv = h >= a.nq + a.nkv;
            const int j = isq ? h : isv ? h - a.nq - a.nkv : h - a.nq;
            uint16_t* dst = isq ? a.q_out + ((size_t)t * a.nq + j) * D
                                : (isv ? a.v_pool : a.k_pool) + ((page * a.nkv + j) * kPage + off) * D;
            if (!isv) {
                if (isq ? a.q_norm != nullptr : a.k_norm != nullptr) {
                    float ss = u.x * u.x + u.y * u.y + u.z * u.z + u.w * u.w + v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
                    const unsigned group = ((1u << LH) - 1) << (tid & 31 & ~(LH - 1));  // LH is 8 or 16
#pragma unroll
                    for (int o = LH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
                    const float r = 1.0f / sqrtf(ss / D + a.eps);
                    const float4 g0 = isq ? gq0 : gk0, g1 = isq ? gq1 : gk1;
                    u.x = u.x * r * g0.x, u.y = u.y * r * g0.y, u.z = u.z * r * g0.z, u.w = u.w * r * g0.w;
                    v.x = v.x * r * g1.x, v.y = v.y * r * g1.y, v.z = v.z * r * g1.z, v.w = v.w * r * g1.w;
                }
                const float4 s = u, w = v;
                u.x = s.x * cs01.x - w.x * cs01.y, v.x = w.x * cs01.x + s.x * cs01.y;
                u.y = s.y * cs01.z - w.y * cs01.w, v.y = w.y * cs01.z + s.y * cs01.w;
                u.z = s.z * cs23.x - w.z * cs23.y, v.z = w.z * cs23.x + s.z * cs23.y;
                u.w = s.w * cs23.z - w.w * cs23.w, v.w = w.w * cs23.z + s.w * cs23.w;
            }
            *reinterpret_cast<uint2*>(dst + 4 * sub) = make_uint2(pack_bf2(u.x, u.y), pack_bf2(u.z, u.w));
            *reinterpret_cast<uint2*>(dst + H + 4 * sub) = make_uint2(pack_bf2(v.x, v.y), pack_bf2(v.z, v.w));
        }
    }
}

}  // namespace
}  // namespace dec

using namespace dec;

extern "C" {

dec_status paged_resize(const int32_t* old_len, const int32_t* new_len, int32_t B, int32_t* block_table,
                        int32_t max_pages, int32_t page_size, int32_t* free_pages, int32_t n_pages, int32_t* n_free,
                        int32_t* cu_rows, int32_t* slot, int32_t* row_pos, int32_t T, int32_t* status,
                        dec_stream_t stream) try {
    set_last_error("");
    if (!old_len || !new_len || !block_table || !free_pages || !n_free || !cu_rows || !status)
        return bad(DEC_ERR_INVALID_ARG, "NULL pointer");
    if (T > 0 && (!slot || !row_pos)) return bad(DEC_ERR_INVALID_ARG, "NULL pointer");
    if (B <= 0 || max_pages <= 0 || n_pages <= 0 || T < 0) return bad(DEC_ERR_INVALID_ARG, "bad B / max_pages / n_pages / T");
    if (page_size != kPage) return bad(DEC_ERR_UNSUPPORTED, "page_size must be 16");
    if (B > kRzMaxB) return bad(DEC_ERR_UNSUPPORTED, "more than 4096 sequences");
    if (n_pages > INT32_MAX / kPage || max_pages > INT32_MAX / kPage || T > (1 << 30))
        return bad(DEC_ERR_UNSUPPORTED, "slots and positions must fit 32 bits, rows 2^30");
    ResizeArgs a{old_len, new_len, B, block_table, max_pages, free_pages, n_pages, n_free, cu_rows, slot, row_pos, T,
                 status, T <= kRzRows};
    // one CTA, or eight when it would place more than three rows (or pages of rows) a thread. 1 / 8 CTAs:
    // 64 sequences, 64 rows 4.7 / 6.0 us; 1000, 1000 6.1 / 7.4; 64, 4096 6.7 / 6.5; 1000, 4000 8.2 / 7.7
    const int C = (a.rows_here ? T : T / kPage) + B > 3 * kRzThreads ? 8 : 1;
    const int smem = 3 * (B + 1) * (int)sizeof(int32_t);
    cudaError_t e = ensure_smem(reinterpret_cast<const void*>(paged_resize_kernel), smem);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kRzThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = C > 1 ? 1 : 0;  // one CTA is a cluster of its own without the attribute, and launches sooner
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, paged_resize_kernel, a);
    cfg.numAttrs = 1;
    if (e == cudaSuccess && !a.rows_here) {
        cfg.gridDim = dim3((T + 255) / 256);
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = 0;
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        e = cudaLaunchKernelEx(&cfg, paged_slots_kernel, a);
    }
    if (e != cudaSuccess) return bad(DEC_ERR_CUDA, std::string("paged_resize: ") + cudaGetErrorString(e));
    return DEC_OK;
} catch (const std::exception&) {
    return DEC_ERR_OOM;
}

dec_status paged_rope_append(const float* qkv, int64_t ld, const float* q_norm, const float* k_norm, float eps,
                             float rope_base, const int32_t* slot, const int32_t* row_pos, int32_t T, int32_t nq,
                             int32_t nkv, int32_t d, int32_t page_size, void* q_out, void* k_pool, void* v_pool,
                             int32_t n_pages, dec_stream_t stream) try {
    set_last_error("");
    if (T < 0 || nq <= 0 || nkv <= 0 || n_pages <= 0) return bad(DEC_ERR_INVALID_ARG, "bad T / heads / n_pages");
    if (T > 0 && (!qkv || !slot || !row_pos || !q_out)) return bad(DEC_ERR_INVALID_ARG, "NULL pointer");
    if (!k_pool || !v_pool) return bad(DEC_ERR_INVALID_ARG, "NULL pointer");
    if (!(rope_base > 0.f)) return bad(DEC_ERR_INVALID_ARG, "rope_base must be positive");
    if ((q_norm || k_norm) && !(eps >= 0.f)) return bad(DEC_ERR_INVALID_ARG, "eps must not be negative");
    if (d != 64 && d != 128) return bad(DEC_ERR_UNSUPPORTED, "d must be 64 or 128");
    if (page_size != kPage) return bad(DEC_ERR_UNSUPPORTED, "page_size must be 16");
    const int64_t width = ((int64_t)nq + 2 * (int64_t)nkv) * d;
    if (ld < width) return bad(DEC_ERR_INVALID_ARG, "ld is smaller than a row");
    if (n_pages > INT32_MAX / kPage || T > (1 << 30) || nq > (1 << 20) || nkv > (1 << 20))
        return bad(DEC_ERR_UNSUPPORTED, "slots must fit 32 bits, rows 2^30, heads 2^20");
    if (((uintptr_t)q_out | (uintptr_t)k_pool | (uintptr_t)v_pool | (uintptr_t)q_norm | (uintptr_t)k_norm) % 16 != 0)
        return bad(DEC_ERR_UNSUPPORTED, "q_out, the pools and the norm gains must be 16-byte aligned");
    if (T == 0) return DEC_OK;
    AppendArgs a{qkv, ld, q_norm, k_norm, eps, rope_base, slot, row_pos, T, nq, nkv, static_cast<uint16_t*>(q_out),
                 static_cast<uint16_t*>(k_pool), static_cast<uint16_t*>(v_pool), n_pages * kPage,
                 ((uintptr_t)qkv | (uintptr_t)(ld * 4)) % 16 == 0};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int grid = std::min(T, 148 * 4);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kApThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, d == 128 ? paged_rope_append_kernel<128> : paged_rope_append_kernel<64>, a);
    if (e != cudaSuccess) return bad(DEC_ERR_CUDA, std::string("paged_rope_append: ") + cudaGetErrorString(e));
    return DEC_OK;
} catch (const std::exception&) {
    return DEC_ERR_OOM;
}

}  // extern "C"
