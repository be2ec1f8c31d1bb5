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
// too close for the fp32 sums (verify_margin) is decided again with fp64 sums.
//
// Measured (B200): 32 sequences of up to 7 drafts over 128256 tokens, 158 MB of rows that count, take 61 us
// on the device: 27 for the first kernel (5.8 TB/s) and 34 for the draw. For a rejected row that is two passes
// of 8 us over both rows on 8 SMs, bound by instructions (25 for an exponential, half of them fp64, at 16 warps
// an SM), and 6 us of cluster barriers and dependent reads. Loads two steps ahead and a table of 16 entries
// without bank conflicts changed nothing. One sequence of 4 drafts takes 13.4 us. Weights kept in registers between the
// two passes over a rejected row changed nothing (13.6 us either way).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <exception>
#include <mutex>
#include <set>
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

struct Stat {  // a piece of a row: max, sum of e^((l - max) / T) (0 in a greedy sequence), argmax (greedy only)
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
    double margin;           // sides of an acceptance closer than this (relative) are compared again in fp64
    Stat* stats;             // [B][2n + 1][splits]: target rows, then draft rows
    int32_t* accepted;
    int32_t* tokens;         // [B][n + 1]
};

constexpr int kMaxDrafts = 64;

DEC_DEVINL int drafts_of(const VerifyArgs& a, int b) {
    return a.count ? min(max(a.count[b], 0), a.n) : a.n;
}

// log2(e) / T for T > 0, as fp32 and as fp64. A temperature below 2^-126, the smallest normal number, counts as that (so
// this stays finite). At T = +inf every token has the same weight but those of -inf: the factor is the
// smallest number above 0, since -inf times 0 would be NaN.
constexpr float kMinT = 0x1p-126f;
DEC_DEVINL float log2e_over(float T) { return fmaxf(1.4426950408889634f / fmaxf(T, kMinT), 0x1p-149f); }
DEC_DEVINL double log2e_over_d(float T) { return fmax(1.4426950408889634074 / (double)fmaxf(T, kMinT), 1e-300); }

DEC_DEVINL float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr int kStatThreads = 256;
constexpr int kBatch = 4;  // 16-byte loads a thread has in flight

// x joined to y, of pieces in this order: the first largest value keeps its index.
DEC_DEVINL Stat join(const Stat& x, const Stat& y, float k) {
    Stat z;
    z.m = fmaxf(x.m, y.m);
    z.s = z.m == -INFINITY ? 0.f : x.s * ex2f((x.m - z.m) * k) + y.s * ex2f((y.m - z.m) * k);
    z.arg = x.m > y.m || (x.m == y.m && x.arg < y.arg) ? x.arg : y.arg;
    z.pad = 0;
    return z;
}

// One piece of one row. A thread takes 16-byte vectors (the row's first and last values one by
// one, where it does not begin or end on a vector), four at a time, with one move of its maximum
// for the four.
__global__ void __launch_bounds__(kStatThreads) verify_stats_kernel(VerifyArgs a) {
    pdl_wait();
    pdl_trigger();
    const int rows = 2 * a.n + 1;
    const int b = blockIdx.y / rows, i = blockIdx.y - b * rows;
    const int nb = drafts_of(a, b);
    const float T = a.temp ? a.temp[b] : 1.f;
    const bool dr = i > a.n, warm = T > 0.f;
    if (dr ? (!a.draft || !warm || i - a.n - 1 >= nb) : i > nb) return;
    const float* row = dr ? a.draft + b * a.d_seq + (i - a.n - 1) * a.d_row : a.target + b * a.t_seq + i * a.t_row;
    const int lo = blockIdx.x * a.piece, hi = min(a.V, lo + a.piece);
    const float k = log2e_over(T);
    Stat st{-INFINITY, 0.f, 0x7fffffff, 0};
    auto one = [&](float l, int j) {
        const float mn = fmaxf(st.m, l);
        if (warm)
            st.s = mn == -INFINITY ? 0.f : st.s * ex2f((st.m - mn) * k) + ex2f((l - mn) * k);
        else if (l > st.m)
            st.arg = j;
        st.m = mn;
    };
    // vectors v0 .. v1 - 1 from `base`, the first 16-byte boundary at or after lo
    const int skip = min((int)((16 - ((uintptr_t)(row + lo) & 15)) & 15) / 4, hi - lo);
    const int base = lo + skip, nv = (hi - base) / 4;
    if (threadIdx.x < skip) one(row[lo + threadIdx.x], lo + threadIdx.x);
    const float4* vec = reinterpret_cast<const float4*>(row + base);
    for (int v0 = threadIdx.x; v0 < nv; v0 += kStatThreads * kBatch) {
        float4 x[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int v = v0 + q * kStatThreads;
            x[q] = v < nv ? __ldcs(vec + v) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        }
        float mn = st.m;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) mn = fmaxf(mn, fmaxf(fmaxf(x[q].x, x[q].y), fmaxf(x[q].z, x[q].w)));
        if (warm) {
            if (mn == -INFINITY) continue;
            float s0 = st.s * ex2f((st.m - mn) * k), s1 = 0.f;
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                s0 += ex2f((x[q].x - mn) * k) + ex2f((x[q].y - mn) * k);
                s1 += ex2f((x[q].z - mn) * k) + ex2f((x[q].w - mn) * k);
            }
            st.s = s0 + s1;
        } else if (mn > st.m) {
#pragma unroll
            for (int q = kBatch - 1; q >= 0; --q) {  // ends at the first place of the largest value
                const int j = base + 4 * (v0 + q * kStatThreads);
                if (x[q].w == mn) st.arg = j + 3;
                if (x[q].z == mn) st.arg = j + 2;
                if (x[q].y == mn) st.arg = j + 1;
                if (x[q].x == mn) st.arg = j;
            }
        }
        st.m = mn;
    }
    for (int j = base + 4 * nv + threadIdx.x; j < hi; j += kStatThreads) one(row[j], j);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Stat y;
        y.m = __shfl_down_sync(0xffffffffu, st.m, o);
        y.s = __shfl_down_sync(0xffffffffu, st.s, o);
        y.arg = __shfl_down_sync(0xffffffffu, st.arg, o);
        st = join(st, y, k);
    }
    __shared__ Stat sh[kStatThreads / 32];
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = st;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kStatThreads / 32; ++w) st = join(st, sh[w], k);
        a.stats[(size_t)blockIdx.y * a.splits + blockIdx.x] = st;
    }
}

constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPickCluster = 16;  // most CTAs of a sequence

// 2^x in fp64 for x <= 0, to some 2^-50: x = n + i / 64 + f with |f| <= 1/128, 2^(i / 64) from a
// table, the exponential series of f ln 2 up to the 5th power (the next term is below 2^-54), n into
// the exponent. Below 2^-1000 it is 0, which no sum of at most 2^30 terms with a term of 1 among
// them can tell. 10 fp64 operations; the series alone took 18, and fp64 is what bounds the draw.
// N values side by side, so that each step's latency is shared.
template <int N>
DEC_DEVINL void exp2_d(double (&x)[N], const double* table) {
    constexpr double kLn2 = 0.69314718055994530942, kMagic = 105553116266496.0;  // 1.5 x 2^46: steps of 1/64
    constexpr double c5 = kLn2 * kLn2 * kLn2 * kLn2 * kLn2 / 120.0, c4 = kLn2 * kLn2 * kLn2 * kLn2 / 24.0,
                     c3 = kLn2 * kLn2 * kLn2 / 6.0, c2 = kLn2 * kLn2 / 2.0;
    double f[N], p[N], w[N];
    int n[N];
    bool in[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        // -1000 and above, by the upper word (0xC08F4000 is -1000's; a NaN may give anything)
        in[i] = (unsigned)__double2hiint(x[i]) < 0xC08F4000u;
        const double t = x[i] + kMagic;
        n[i] = __double2loint(t);
        f[i] = x[i] - (t - kMagic);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = table[n[i] & 63];
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = fma(c5, f[i], c4);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = fma(p[i], f[i], c3);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = fma(p[i], f[i], c2);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = fma(p[i], f[i], kLn2);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = fma(p[i], f[i], 1.0) * w[i];
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = in[i] ? __hiloint2double(__double2hiint(p[i]) + ((n[i] >> 6) << 20), __double2loint(p[i])) : 0.0;
}

// Values of the vocabulary a lane has, with C CTAs a sequence.
__host__ __device__ inline int run_per_lane(int V, int C) {
    const long long lanes = (long long)C * kPickThreads;
    return (int)(((V + lanes - 1) / lanes + 3) / 4 * 4);
}

struct PickShared {
    Stat row[2 * kMaxDrafts + 1];
    int verdict[kMaxDrafts];         // of each draft: 1 accepted, 0 not, 2 too close for fp32 sums
    // of the last two sums, in turn (a CTA that stores to the next sum's place has seen all CTAs leave the
    // one before the last, whose place it is)
    double warp[2][2][kPickWarps];
    double cta[2][2][kPickCluster];  // written by every CTA of the cluster
    double table[64];                // 2^(i / 64)
};

DEC_DEVINL double warp_sum_d(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sums over the cluster of x and y (one value a thread), in a fixed order; also this
// CTA's own warps' totals in sh.warp[at] and every CTA's in sh.cta[at], `at` another one at each call.
// Every thread of the cluster calls it. A cluster barrier costs 1400 cycles here.
DEC_DEVINL double2 cluster_sum(PickShared& sh, int at, double x, double y, int rank, int C) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    x = warp_sum_d(x);
    y = warp_sum_d(y);
    if (lane == 0) {
        sh.warp[at][0][warp] = x;
        sh.warp[at][1][warp] = y;
    }
    __syncthreads();
    if (warp < 2) {  // warp w sums kind w and hands it to CTA `lane`
        double t = 0.0;
        for (int w = 0; w < kPickWarps; ++w) t += sh.warp[at][warp][w];
        if (lane < C)
            asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(dsmem_map(smem_u32(&sh.cta[at][warp][rank]), lane)),
                         "d"(t)
                         : "memory");
    }
    cluster_sync();
    double2 t = make_double2(0.0, 0.0);
    for (int r = 0; r < C; ++r) {
        t.x += sh.cta[at][0][r];
        t.y += sh.cta[at][1][r];
    }
    return t;
}

__global__ void __launch_bounds__(kPickThreads, 2) verify_pick_kernel(VerifyArgs a) {
    __shared__ PickShared sh;
    const int rank = blockIdx.x, C = gridDim.x, b = blockIdx.y;  // one cluster a sequence
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < 64) sh.table[threadIdx.x] = exp2(threadIdx.x / 64.0);
    // the matching wait comes before the first store to another CTA's shared memory
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    // Nothing that another kernel writes is read before this wait, the counts and temperatures among it: that the
    // first kernel has waited for whoever wrote them makes them visible to that kernel, not to this one.
    pdl_wait();
    pdl_trigger();
    const int nb = drafts_of(a, b);
    const float T = a.temp ? a.temp[b] : 1.f;
    const bool warm = T > 0.f;
    const double c = log2e_over_d(T);  // e^(l / T) = 2^(c l)
    const float k = log2e_over(T);

    // ---- the rows' statistics from their pieces, a warp a row
    for (int i = warp; i < 2 * a.n + 1; i += kPickWarps) {
        const bool there = i > a.n ? a.draft && warm && i - a.n - 1 < nb : i <= nb;
        if (!there) continue;
        const Stat* p = a.stats + ((size_t)b * (2 * a.n + 1) + i) * a.splits;
        Stat z{-INFINITY, 0.f, 0x7fffffff, 0};
        for (int s = lane; s < a.splits; s += 32) z = join(z, p[s], k);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Stat y;
            y.m = __shfl_down_sync(0xffffffffu, z.m, o);
            y.s = __shfl_down_sync(0xffffffffu, z.s, o);
            y.arg = __shfl_down_sync(0xffffffffu, z.arg, o);
            z = join(z, y, k);
        }
        if (lane == 0) sh.row[i] = z;
    }
    __syncthreads();
    auto target_row = [&](int i) { return a.target + b * a.t_seq + i * a.t_row; };
    auto draft_row = [&](int i) { return a.draft ? a.draft + b * a.d_seq + i * a.d_row : nullptr; };
    // e^((l - m) / T) in fp64; a row of -inf counts from 0, and every weight is 0
    auto origin = [](float m) { return m > -INFINITY ? (double)m : 0.0; };
    auto weight_of = [&](float l, double m) {
        double x[1] = {((double)l - m) * c};
        exp2_d(x, sh.table);
        return x[0];
    };
    auto weights_of = [&](const float (&l)[4], double m, double (&x)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = ((double)l[i] - m) * c;
        exp2_d(x, sh.table);
    };

    // ---- every draft's verdict by the fp32 sums, a thread a draft
    if (threadIdx.x < nb) {
        const int i = threadIdx.x, x = a.tok[(size_t)b * a.n + i];
        const Stat p = sh.row[i];
        int v = 0;
        if (!warm) {
            v = x == p.arg && x < a.V;  // the argmax of a row of -inf is none
        } else if (x >= 0 && x < a.V) {
            // u q < p, multiplied out
            const double u = a.u[(size_t)b * a.n + i];
            double left = u * (double)p.s, right = weight_of(target_row(i)[x], origin(p.m));
            if (a.draft) {
                const Stat q = sh.row[a.n + 1 + i];
                left *= weight_of(draft_row(i)[x], origin(q.m));
                right *= (double)q.s;
            }
            v = left < right;
            if (fabs(left - right) <= a.margin * fmax(left, right)) v = 2;
        }
        sh.verdict[i] = v;
    }
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    int at = 0;  // of the last cluster_sum

    // The vocabulary in runs of 32 E values, one a warp (E a multiple of 4): in step t of E / 4 lane l takes
    // values 128 t + 4 l .. + 3 of the run, so that a warp reads whole lines.
    const int E = run_per_lane(a.V, C);
    const long long run0 = (long long)(rank * kPickWarps + warp) * 32 * E;
    // values j .. j + 3 of a row (-inf past the vocabulary's end)
    auto load4 = [&](const float* row, long long j, float (&x)[4]) {
        if (j + 4 <= a.V && ((uintptr_t)(row + j) & 15) == 0) {
            const float4 v = *reinterpret_cast<const float4*>(row + j);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = j + q < a.V ? row[j + q] : -INFINITY;
        }
    };
    // fp64 sums of a target row and of a draft row (null: 0)
    auto sums = [&](const float* pr, double pm, const float* qr, double qm) {
        double x[2] = {0.0, 0.0}, y[2] = {0.0, 0.0};
#pragma unroll 2
        for (int t = 0; t < E / 4; ++t) {
            float p[4], q[4];
            load4(pr, run0 + 128 * t + 4 * lane, p);
            if (qr) load4(qr, run0 + 128 * t + 4 * lane, q);
            double e[4];
            weights_of(p, pm, e);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i & 1] += e[i];
            if (qr) {
                weights_of(q, qm, e);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i & 1] += e[i];
            }
        }
        return cluster_sum(sh, at ^= 1, x[0] + x[1], y[0] + y[1], rank, C);
    };

    // ---- the first draft that is not accepted
    int acc = 0;
    double2 z = make_double2(0.0, 0.0);  // row acc's sums, where they are known
    bool known = false;
    for (; acc < nb; ++acc) {
        int v = sh.verdict[acc];
        if (v == 2) {
            const int x = a.tok[(size_t)b * a.n + acc];
            const double pm = origin(sh.row[acc].m), qm = a.draft ? origin(sh.row[a.n + 1 + acc].m) : 0.0;
            z = sums(target_row(acc), pm, draft_row(acc), qm);
            const double q = a.draft ? weight_of(draft_row(acc)[x], qm) : 1.0;
            v = (double)a.u[(size_t)b * a.n + acc] * q * z.x < weight_of(target_row(acc)[x], pm) * (a.draft ? z.y : 1.0);
            known = !v;
        }
        if (!v) break;
    }
    const Stat p = sh.row[acc];
    int32_t* out = a.tokens + (size_t)b * (a.n + 1);
    if (rank == 0) {
        for (int i = threadIdx.x; i <= a.n; i += kPickThreads) {
            if (i < acc) out[i] = a.tok[(size_t)b * a.n + i];
            // a drawn token replaces the -1 at acc, after the cluster barriers below
            if (i >= acc) out[i] = i == acc && !warm && p.arg < a.V ? p.arg : -1;
        }
        if (threadIdx.x == 0) a.accepted[b] = acc;
    }
    if (warm && p.m > -INFINITY) {
        // ---- draw from max(p - q, 0) of row acc, or from p after the last draft
        const float* pr = target_row(acc);
        const bool rej = acc < nb;
        const float* qr = rej ? draft_row(acc) : nullptr;
        // a point mass at a token outside the vocabulary takes nothing away
        const int tok = rej && !a.draft ? a.tok[(size_t)b * a.n + acc] : -1, x = tok < a.V ? tok : -1;
        const double pm = origin(p.m), qm = qr ? origin(sh.row[a.n + 1 + acc].m) : 0.0;
        if (!known) z = sums(pr, pm, qr, qm);
        // drawing from p alone, the sums just taken are the weights' (times 1 / z.x): no second pass
        const bool bare = !qr && x < 0;
        const double ip = bare ? 1.0 : 1.0 / z.x, iq = qr && z.y > 0.0 ? 1.0 / z.y : 0.0;
        bool plain = false;  // no weight left in p - q: p itself
        auto weight = [&](double ep, double eq, long long j) {
            double w = ep * ip;
            if (plain) return w;
            if (qr) w -= eq * iq;
            if (j == x) w -= 1.0;
            return fmax(w, 0.0);
        };
        double total = z.x;
        while (!bare) {
            double own[2] = {0.0, 0.0};
#pragma unroll 2
            for (int t = 0; t < E / 4; ++t) {
                const long long j = run0 + 128 * t + 4 * lane;
                float lp[4], lq[4];
                load4(pr, j, lp);
                if (qr) load4(qr, j, lq);
                double ep[4], eq[4] = {0.0, 0.0, 0.0, 0.0};
                weights_of(lp, pm, ep);
                if (qr) weights_of(lq, qm, eq);
#pragma unroll
                for (int i = 0; i < 4; ++i) own[i & 1] += weight(ep[i], eq[i], j + i);
            }
            total = cluster_sum(sh, at ^= 1, own[0] + own[1], 0.0, rank, C).x;
            if (total > 0.0 || plain) break;
            plain = true;
        }
        // The place where the cumulative weight passes us * total: the CTA, its warp's run, then (all warps of the CTA
        // sharing that run, 2 E values a warp) the warp, the lane and the value, each time the first with weight
        // whose end is above the goal (the last with weight, should rounding leave none).
        const double goal = (double)a.us[b] * total;
        auto find = [&](const double* s, int n, double* base) {
            double before = *base;
            int at = -1;
            for (int r = 0; r < n; ++r) {
                const double upto = before + s[r];
                if (s[r] > 0.0) {
                    at = r;
                    *base = before;
                    if (upto > goal) break;
                }
                before = upto;
            }
            return at;
        };
        double base = 0.0;
        if (find(sh.cta[at][0], C, &base) == rank) {
            const int w = find(sh.warp[at][0], kPickWarps, &base);
            const int per = E / 16 > 0 ? (E + 15) / 16 : 1;  // values a lane has of the run: 512 lanes, 32 E values
            const long long begin = (long long)(rank * kPickWarps + w) * 32 * E, end = min((long long)a.V, begin + 32 * E);
            const long long j = begin + (long long)threadIdx.x * per;
            double own = 0.0;
            for (int i = 0; i < per; ++i)
                if (j + i < end) own += weight(weight_of(pr[j + i], pm), qr ? weight_of(qr[j + i], qm) : 0.0, j + i);
            double cum = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, cum, o);
                if (lane >= o) cum += y;
            }
            __syncthreads();  // sh.warp has been read
            if (lane == 31) sh.warp[at][0][warp] = cum;
            __syncthreads();
            if (find(sh.warp[at][0], kPickWarps, &base) == warp) {
                const unsigned some = __ballot_sync(0xffffffffu, own > 0.0);
                const unsigned hit = __ballot_sync(0xffffffffu, own > 0.0 && base + cum > goal);
                if (lane == (hit ? __ffs(hit) - 1 : 31 - __clz(some))) {
                    double run = base + (cum - own);
                    int pick = -1;
                    for (int i = 0; i < per && j + i < end; ++i) {
                        const double s = weight(weight_of(pr[j + i], pm), qr ? weight_of(qr[j + i], qm) : 0.0, j + i);
                        if (s > 0.0) {
                            pick = (int)(j + i);
                            run += s;
                            if (run > goal) break;
                        }
                    }
                    out[acc] = pick;
                }
            }
        }
    }
    cluster_sync();  // no CTA leaves while another may still store to its shared memory
}

// Clusters of 16 CTAs need the kernel's consent, once a device.
cudaError_t allow_wide_cluster() {
    static std::mutex mu;
    static std::set<int> done;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (done.count(dev)) return cudaSuccess;
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(verify_pick_kernel),
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.insert(dev);
    return e;
}

// Pieces of a row: of at most 4096 values, or longer where pieces that short would be more than fill the GPU
// several times over.
constexpr int kPiece = 4096, kPieces = 148 * 32;

int verify_splits(int B, int n, int V) {
    const long long rows = (long long)B * (2 * n + 1);
    int s = (V + kPiece - 1) / kPiece;
    while (s > 1 && rows * s > kPieces) s = (s + 1) / 2;
    return s;
}

// How far apart (relative) the two sides of an acceptance have to be for the fp32 sums to decide it. In units of
// 2^-24, a term of a sum is off by 4 for each ex2 and 1 for each product or addition on its way: its own ex2; 12
// for each step over 16 values a thread takes (one move of the maximum, six additions) and for the row's ends; 6
// for each join (5 and 7 in a CTA, one for every 32 pieces and 5 over the pieces). All exponents on that way add up to the
// term's own, off by 4 x 2^-24 of itself; it is below 60 where the term counts (2^30 terms of 2^-60 are
// 2^-30), so 4 x 60 x ln 2 = 166 more. Two sums, and a quarter more for what the errors' products add. For a
// vocabulary of 128256 that is 4.7e-5 (pieces of 4008) to 1e-4 (one piece): one acceptance in 10^4 costs fp64 sums.
double verify_margin(int piece, int splits) {
    const double steps = piece / (4.0 * kBatch * kStatThreads) + 2.0, joins = 17.0 + (splits + 31) / 32;
    return 2.5 * (170.0 + 12.0 * steps + 6.0 * joins) * 0x1p-24;
}

}  // namespace
}  // namespace dec

using namespace dec;

extern "C" {

int64_t spec_verify_workspace(int32_t B, int32_t n, int32_t V) {
    if (B <= 0 || n < 0 || V <= 0) return 0;
    // no fewer than verify_splits gives, and never fewer for more sequences, drafts or values
    const int64_t rows = (int64_t)B * (2 * (int64_t)n + 1), most = std::max<int64_t>(kPieces, rows);
    return std::min(rows * ((V - 1) / kPiece + 1), most) * (int64_t)sizeof(Stat);
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
    if (n > kMaxDrafts) return bad(DEC_ERR_UNSUPPORTED, "more than 64 drafted tokens");
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
    a.margin = verify_margin(a.piece, a.splits);
    a.stats = static_cast<Stat*>(workspace);
    a.accepted = n_accepted;
    a.tokens = tokens;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.splits, B * (2 * n + 1));
    cfg.blockDim = dim3(kStatThreads);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, verify_stats_kernel, a);
    if (e == cudaSuccess) e = allow_wide_cluster();
    // CTAs a sequence: the draw is shorter the more SMs it has, while all its clusters run at once or nearly so. The SMs
    // have 296 places, but a cluster's lie in one GPC: 14 clusters of 16 run at once, 33 of 8, 71 of 4, 148 of 2.
    // So 16 up to 18 sequences, 8 up to 52, 4 up to 105, else 2. Device time of a call in us, n drafts, thousands of tokens:
    //   16 / 8: n 4, 128k   8 sequences 27.5 / 32.5, 16 42.3 / 42.1, 18 44.1 / 46.1, 20 47.5 / 50.1, 24 52.9 / 50.3,
    //           32 69.2 / 58.3;  49k, 20: n 1 23.6 / 20.1, n 4 34.3 / 27.3
    //   8 / 4:  n 4, 128k   37 69.3 / 82.8, 48 86.8 / 91.4, 52 91.9 / 91.0;  49k, 48: n 1 31.4 / 32.7, n 4 45.2 / 42.6
    //   4 / 2:  n 4, 128k   90 136.9 / 166.4, 110 167.2 / 179.6;  49k, 100: n 1 47.0 / 54.3, n 4 65.2 / 70.8, 120: 53.4 / 59.2,
    //           76.8 / 75.1, 148: 59.1 / 57.7, 91.6 / 82.1
    //   2 / 1:  49k   149: n 1 60.1 / 79.3, n 4 82.2 / 118.1, 300: 103.5 / 113.1, 158.9 / 163.4, 1000: 263.9 / 259.8, 454.3 / 449.6
    const int C = B <= 18 ? 16 : B <= 52 ? 8 : B <= 105 ? 4 : 2;
    cfg.gridDim = dim3(C, B);
    cfg.blockDim = dim3(kPickThreads);
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = C;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, verify_pick_kernel, a);
    if (e != cudaSuccess) return bad(DEC_ERR_CUDA, std::string("spec_verify: ") + cudaGetErrorString(e));
    return DEC_OK;
} catch (const std::exception&) {
    return DEC_ERR_OOM;
}

}  // extern "C"
