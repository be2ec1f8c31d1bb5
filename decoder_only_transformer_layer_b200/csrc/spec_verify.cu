// Verification of drafted tokens against the target model's distribution, from given
// uniform random numbers (the rejection rule of speculative sampling).
//
// Sequence b has n_b drafted tokens x_0 .. x_{n_b - 1}; p_i is the softmax of target row i
// over the temperature, q_i that of draft row i (or the point mass at x_i). Drafts are
// accepted while u_i q_i(x_i) < p_i(x_i); at the first one that is not, the next token is
// drawn from max(p_i - q_i, 0) normalised, after the last one from p_{n_b}. The draw is
// the least token whose cumulative weight exceeds us * (total weight). At temperature 0 a
// draft is accepted when it is the argmax of its target row (the lowest index on ties).
//
// Two kernels. The first reads every row once: maximum, argmax and sum of exponentials of
// a piece of a row, in fp32. It is bound by HBM. The second, a cluster a sequence, joins
// the pieces, finds the first rejection, and draws the token from that one row, which it
// reads again (from L2). A drawn token lies between two neighbouring values of a
// cumulative sum over the whole vocabulary, a spacing of 1e-5 or less, so that row's
// exponentials, sums and cumulative sums are in fp64. An acceptance whose two sides are
// too close for the fp32 sums is decided again with fp64 sums.
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

dec_status bad(dec_status s, const std::string& why) {
    set_last_error(why);
    return s;
}

struct Stat {  // a piece of a row: max, sum of e^((l - max) / T), argmax
    float m, s;
    int arg, pad;
};

struct VerifyArgs {
    const float* target;
    long long t_row, t_seq;  // strides in floats
    const float* draft;      // null: point masses
    long long d_row, d_seq;
    const int32_t* tok;      // [B][n]
    const int32_t* count;    // [B] or null
    const float* temp;       // [B] or null: 1
    const float* u;          // [B][n]
    const float* us;         // [B]
    int B, n, V, splits, piece;
    Stat* stats;             // [B][2n + 1][splits]: target rows, then draft rows
    int32_t* accepted;
    int32_t* tokens;         // [B][n + 1]
};

DEC_DEVINL int drafts_of(const VerifyArgs& a, int b) {
    return a.count ? min(max(a.count[b], 0), a.n) : a.n;
}

constexpr int kStatThreads = 256;

// One piece of one row.
__global__ void __launch_bounds__(kStatThreads) verify_stats_kernel(VerifyArgs a) {
    const int b = blockIdx.y / (2 * a.n + 1), i = blockIdx.y % (2 * a.n + 1);
    const int nb = drafts_of(a, b);
    const float T = a.temp ? a.temp[b] : 1.f;
    const bool dr = i > a.n;
    if (dr ? (!a.draft || T <= 0.f || i - a.n - 1 >= nb) : i > nb) return;
    const float* row = dr ? a.draft + b * a.d_seq + (i - a.n - 1) * a.d_row : a.target + b * a.t_seq + i * a.t_row;
    const int lo = blockIdx.x * a.piece, hi = min(a.V, lo + a.piece);
    const float k = T > 0.f ? 1.4426950408889634f / T : 0.f;
    float m = -INFINITY, s = 0.f;
    int arg = 0x7fffffff;
    for (int j = lo + threadIdx.x; j < hi; j += kStatThreads) {
        const float l = row[j];
        if (l > m) {
            s *= exp2f((m - l) * k);
            m = l;
            arg = j;
        }
        if (m > -INFINITY) s += exp2f((l - m) * k);
    }
    __shared__ Stat sh[kStatThreads];
    sh[threadIdx.x] = Stat{m, s, arg, 0};
    __syncthreads();
    for (int o = kStatThreads / 2; o > 0; o >>= 1) {
        if (threadIdx.x < o) {
            const Stat x = sh[threadIdx.x], y = sh[threadIdx.x + o];
            Stat z;
            z.m = fmaxf(x.m, y.m);
            z.s = z.m == -INFINITY ? 0.f : x.s * exp2f((x.m - z.m) * k) + y.s * exp2f((y.m - z.m) * k);
            z.arg = x.m > y.m || (x.m == y.m && x.arg < y.arg) ? x.arg : y.arg;
            z.pad = 0;
            sh[threadIdx.x] = z;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) a.stats[(size_t)blockIdx.y * a.splits + blockIdx.x] = sh[0];
}

constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPickMaxCluster = 8;

struct PickShared {
    Stat row[1];
    double warp[2][kPickWarps];
    double cta[2][kPickMaxCluster];  // written by every CTA of the cluster
};

DEC_DEVINL double warp_sum_d(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sums over the cluster of x and y (one value a thread), in a fixed order; also this
// CTA's own totals in sh.cta. Every thread of the cluster calls it.
DEC_DEVINL double2 cluster_sum(PickShared& sh, double x, double y, int rank, int C) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    x = warp_sum_d(x);
    y = warp_sum_d(y);
    cluster_sync();  // the last call's values have been read
    if (lane == 0) {
        sh.warp[0][warp] = x;
        sh.warp[1][warp] = y;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double t = 0.0;
        for (int w = 0; w < kPickWarps; ++w) t += sh.warp[threadIdx.x][w];
        for (int r = 0; r < C; ++r)
            asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(dsmem_map(smem_u32(&sh.cta[threadIdx.x][rank]), r)),
                         "d"(t)
                         : "memory");
    }
    cluster_sync();
    double2 t = make_double2(0.0, 0.0);
    for (int r = 0; r < C; ++r) {
        t.x += sh.cta[0][r];
        t.y += sh.cta[1][r];
    }
    return t;
}

__global__ void __launch_bounds__(kPickThreads) verify_pick_kernel(VerifyArgs a) {
    __shared__ PickShared sh;
    const int C = gridDim.x, rank = blockIdx.x, b = blockIdx.y;  // one cluster a sequence
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nb = drafts_of(a, b);
    const float T = a.temp ? a.temp[b] : 1.f;
    const bool warm = T > 0.f;
    const double invT = warm ? 1.0 / (double)T : 0.0;
    const float k = warm ? 1.4426950408889634f / T : 0.f;

    // the whole row's max, sum and argmax from its pieces (each thread for itself)
    auto row_stat = [&](int i) {
        const Stat* p = a.stats + ((size_t)b * (2 * a.n + 1) + i) * a.splits;
        Stat z = p[0];
        for (int s = 1; s < a.splits; ++s) {
            const Stat y = p[s];
            const float m = fmaxf(z.m, y.m);
            z.s = m == -INFINITY ? 0.f : z.s * exp2f((z.m - m) * k) + y.s * exp2f((y.m - m) * k);
            z.arg = z.m >= y.m ? z.arg : y.arg;
            z.m = m;
        }
        return z;
    };
    const int per = (a.V + C * kPickWarps - 1) / (C * kPickWarps);  // a warp's run of the vocabulary
    const int j0 = min(a.V, (rank * kPickWarps + warp) * per), j1 = min(a.V, j0 + per);
    // fp64 sums of e^((l - m) / T) of the target row and of the draft row (null: 0)
    auto sums = [&](const float* pr, float pm, const float* qr, float qm) {
        double x = 0.0, y = 0.0;
        for (int j = j0 + lane; j < j1; j += 32) {
            if (pm > -INFINITY) x += exp(((double)pr[j] - (double)pm) * invT);
            if (qr && qm > -INFINITY) y += exp(((double)qr[j] - (double)qm) * invT);
        }
        return cluster_sum(sh, x, y, rank, C);
    };

    // ---- the first draft that is not accepted
    int acc = 0, arg = 0;
    for (; acc < nb; ++acc) {
        const int x = a.tok[(size_t)b * a.n + acc];
        const Stat p = row_stat(acc);
        if (!warm) {
            if (x != p.arg) break;
            continue;
        }
        if (x < 0 || x >= a.V) break;
        const float* pr = a.target + b * a.t_seq + acc * a.t_row;
        const float* qr = a.draft ? a.draft + b * a.d_seq + acc * a.d_row : nullptr;
        const double u = a.u[(size_t)b * a.n + acc];
        const double ep = p.m > -INFINITY ? exp(((double)pr[x] - (double)p.m) * invT) : 0.0;
        double left, right;
        if (!qr) {
            left = u * (double)p.s;
            right = ep;
        } else {
            const Stat q = row_stat(a.n + 1 + acc);
            const double eq = q.m > -INFINITY ? exp(((double)qr[x] - (double)q.m) * invT) : 0.0;
            left = u * eq * (double)p.s;
            right = ep * (double)q.s;
        }
        // the fp32 sums are within 1e-5 of the exact ones (each term within 2^-22 (l - m) / T,
        // which is below 2^-22 * 40 where it counts)
        if (fabs(left - right) <= 4e-5 * fmax(left, right)) {
            const Stat q = qr ? row_stat(a.n + 1 + acc) : Stat{0.f, 1.f, 0, 0};
            const double2 z = sums(pr, p.m, qr, q.m);
            const double eq = !qr ? 1.0 : q.m > -INFINITY ? exp(((double)qr[x] - (double)q.m) * invT) : 0.0;
            left = u * eq * z.x;
            right = ep * (qr ? z.y : 1.0);
        }
        if (!(left < right)) break;
    }
    const Stat p = row_stat(acc);
    arg = p.arg;
    int pick = -1;
    if (!warm) {
        pick = arg < a.V ? arg : -1;
    } else if (p.m > -INFINITY) {
        // ---- draw from max(p - q, 0) of row acc, or from p after the last draft
        const float* pr = a.target + b * a.t_seq + acc * a.t_row;
        const bool rej = acc < nb;
        const float* qr = rej && a.draft ? a.draft + b * a.d_seq + acc * a.d_row : nullptr;
        const int x = rej && !a.draft ? a.tok[(size_t)b * a.n + acc] : -1;
        const float qm = qr ? row_stat(a.n + 1 + acc).m : -INFINITY;
        const double2 z = sums(pr, p.m, qr, qm);
        const double ip = 1.0 / z.x, iq = qr && z.y > 0.0 ? 1.0 / z.y : 0.0;
        bool plain = false;  // no weight left in p - q: p itself
        auto weight = [&](int j) {
            const double pj = exp(((double)pr[j] - (double)p.m) * invT) * ip;
            if (plain) return pj;
            double qj = j == x ? 1.0 : 0.0;
            if (iq > 0.0) qj = exp(((double)qr[j] - (double)qm) * invT) * iq;
            return fmax(pj - qj, 0.0);
        };
        double own = 0.0;
        double2 tot;
        for (;;) {
            own = 0.0;
            for (int j = j0 + lane; j < j1; j += 32) own += weight(j);
            tot = cluster_sum(sh, own, 0.0, rank, C);
            if (tot.x > 0.0 || plain) break;
            plain = true;
        }
        // the run of the vocabulary in which the cumulative weight passes us * total: the
        // first one whose end is above it (the last one with any weight when rounding leaves none)
        const double goal = (double)a.us[b] * tot.x;
        double before = 0.0, upto = 0.0;
        int cta = -1, w = -1;
        double base = 0.0;
        for (int r = 0; r < C; ++r) {
            upto = before + sh.cta[0][r];
            if (sh.cta[0][r] > 0.0) {
                cta = r;
                base = before;
                if (upto > goal) break;
            }
            before = upto;
        }
        if (cta == rank) {
            before = base;
            for (int v = 0; v < kPickWarps; ++v) {
                upto = before + sh.warp[0][v];
                if (sh.warp[0][v] > 0.0) {
                    w = v;
                    base = before;
                    if (upto > goal) break;
                }
                before = upto;
            }
            if (w == warp) {
                int last = -1;
                double run = base;
                for (int j = j0; j < j1 && pick < 0; j += 32) {
                    const double wj = j + lane < j1 ? weight(j + lane) : 0.0;
                    double c = wj;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const double y = __shfl_up_sync(0xffffffffu, c, o);
                        if (lane >= o) c += y;
                    }
                    const unsigned some = __ballot_sync(0xffffffffu, wj > 0.0);
                    const unsigned hit = __ballot_sync(0xffffffffu, wj > 0.0 && run + c > goal);
                    if (hit) pick = j + __ffs(hit) - 1;
                    if (some) last = j + 31 - __clz(some);
                    run += __shfl_sync(0xffffffffu, c, 31);
                }
                if (pick < 0) pick = last;
                if (lane == 0) a.tokens[(size_t)b * (a.n + 1) + acc] = pick;
            }
        }
    }
    if (rank == 0) {
        for (int i = threadIdx.x; i <= a.n; i += kPickThreads) {
            if (i < acc) a.tokens[(size_t)b * (a.n + 1) + i] = a.tok[(size_t)b * a.n + i];
            if (i > acc) a.tokens[(size_t)b * (a.n + 1) + i] = -1;
            if (i == acc && (!warm || !(p.m > -INFINITY))) a.tokens[(size_t)b * (a.n + 1) + i] = pick;
        }
        if (threadIdx.x == 0) a.accepted[b] = acc;
    }
    cluster_sync();  // no CTA leaves while another may still store to its shared memory
}

int verify_splits(int B, int n, int V) {
    // pieces of at least 4096 values, and enough of them to fill the GPU several times over
    const long long rows = (long long)B * (2 * n + 1);
    int s = (V + 4095) / 4096;
    while (s > 1 && rows * s > 148 * 32) s = (s + 1) / 2;
    return s;
}

}  // namespace
}  // namespace dec

using namespace dec;

extern "C" {

int64_t spec_verify_workspace(int32_t B, int32_t n, int32_t V) {
    if (B <= 0 || n < 0 || V <= 0) return 0;
    return (int64_t)B * (2 * (int64_t)n + 1) * verify_splits(B, n, V) * (int64_t)sizeof(Stat);
}

dec_status spec_verify(const float* target, int64_t target_row, int64_t target_seq, const float* draft,
                       int64_t draft_row, int64_t draft_seq, const int32_t* draft_tok, const int32_t* n_draft,
                       const float* temperature, const float* u_accept, const float* u_sample, int32_t B, int32_t n,
                       int32_t V, int32_t* n_accepted, int32_t* tokens, void* workspace, int64_t workspace_bytes,
                       dec_stream_t stream) try {
    set_last_error("");
    if (!target || !u_sample || !n_accepted || !tokens || !workspace) return bad(DEC_ERR_INVALID_ARG, "NULL pointer");
    if (B <= 0 || n < 0 || V <= 0) return bad(DEC_ERR_INVALID_ARG, "bad B / n / V");
    if (n > 0 && (!draft_tok || !u_accept)) return bad(DEC_ERR_INVALID_ARG, "NULL pointer");
    if (n > 64) return bad(DEC_ERR_UNSUPPORTED, "more than 64 drafted tokens");
    if ((int64_t)B * (2 * n + 1) > 65535) return bad(DEC_ERR_UNSUPPORTED, "B * (2 n + 1) above 65535");
    if (V > (1 << 30)) return bad(DEC_ERR_UNSUPPORTED, "V above 2^30");
    if (target_row < V || target_seq < 0) return bad(DEC_ERR_INVALID_ARG, "bad target strides");
    if (draft && n > 0 && (draft_row < V || draft_seq < 0)) return bad(DEC_ERR_INVALID_ARG, "bad draft strides");
    if ((uintptr_t)workspace % 16) return bad(DEC_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    if (workspace_bytes < spec_verify_workspace(B, n, V)) return bad(DEC_ERR_INVALID_ARG, "workspace too small");
    VerifyArgs a{};
    a.target = target;
    a.t_row = target_row;
    a.t_seq = target_seq;
    a.draft = n > 0 ? draft : nullptr;
    a.d_row = draft_row;
    a.d_seq = draft_seq;
    a.tok = draft_tok;
    a.count = n_draft;
    a.temp = temperature;
    a.u = u_accept;
    a.us = u_sample;
    a.B = B;
    a.n = n;
    a.V = V;
    a.splits = verify_splits(B, n, V);
    a.piece = (V + a.splits - 1) / a.splits;
    a.stats = static_cast<Stat*>(workspace);
    a.accepted = n_accepted;
    a.tokens = tokens;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    verify_stats_kernel<<<dim3(a.splits, B * (2 * n + 1)), kStatThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPickMaxCluster, B);
    cfg.blockDim = dim3(kPickThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kPickMaxCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, verify_pick_kernel, a);
    if (e != cudaSuccess) return bad(DEC_ERR_CUDA, std::string("spec_verify: ") + cudaGetErrorString(e));
    return DEC_OK;
} catch (const std::exception&) {
    return DEC_ERR_OOM;
}

}  // extern "C"
