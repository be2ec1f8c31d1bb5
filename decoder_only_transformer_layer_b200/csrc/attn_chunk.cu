// Causal GQA attention of ragged chunks of new rows over a caller's paged KV cache, on the
// tensor cores (tcgen05, TMEM).
//
// Sequence b has rows cu[b] .. cu[b + 1] - 1 of q and kv_len[b] cache rows, its own new
// rows last: row i of its n rows sits at position p = kv_len[b] - n + i and sees keys
// max(0, p - W + 1) .. p (W = window, all of 0 .. p without one) whose page lies in the pool:
//   out[r][h] = sum_j softmax_j(c(q[r][h] . K[j] scale)) V[j],  c(s) = cap tanh(s / cap).
// A row that sees no key gives zeros.
//
// Tiles. The G query heads that share a kv head are packed with the tokens: a sub-tile is
// 128 / G tokens x G heads = up to 128 MMA rows, a tile two sub-tiles (0 and 1), each with
// four softmax warps, a thread a row. Two ways to use the pair:
//   two   the tile has rows for both: both read the same key blocks, so a K or V block is
//         loaded once for 256 rows, and while one sub-tile's scores are being exponentiated
//         the tensor cores work for the other;
//   one   the rows fit one sub-tile (a decode, a few drafts): both hold the same rows, 0
//         takes the even key blocks and 1 the odd ones, and the two partial results are
//         joined in TMEM at the end. Such a tile is bound by the stream of K and V.
// Per 128-key block and sub-tile: S = Q K^T (M = N = 128, fp32 in TMEM), P = 2^(S' - m) as
// bf16 over S in TMEM, O += P V (A = P from TMEM). The maximum m is moved, and O rescaled,
// only when a row's maximum grows by more than 2^8: P <= 2^8 never overflows and O / l does
// not depend on m. P is rounded to bf16 once: each weight is off by at most 2^-9 of itself,
// as much as the rounding of the result; l sums the unrounded fp32 values.
//
// Work split. Lengths are known on the device only, so every CTA cuts the work for itself:
// the (tile, key block) pairs of all sequences, kv heads and tiles form one list, cut into
// equal runs, one for each of 148 CTAs (the number of blocks of the first t tiles of a sequence
// has a closed form, so finding a run's start takes a scan over the sequences and a binary
// search). A long prompt, a batch of decodes, or both at once keep every SM equally busy. A
// tile cut between CTAs leaves unnormalised fp32 pieces (O, m, l) in the workspace, which a
// second kernel joins in the order of the runs, so results do not depend on timing.
//
// Masked places. Scores outside a row's keys are replaced, so K may hold anything there.
// V reaches a row through P = 0, and 0 x NaN is NaN: in every block in which some row of the
// tile does not see some key, two warps set V rows outside the tile's keys to zero in shared
// memory, and where tokens of the tile see different keys, also take out values that are not
// finite, note their keys, and the epilogue adds those values back to the rows that do see them.
//
// Warps: 0-3 and 4-7 softmax and epilogue of sub-tiles 0 and 1, 8 TMA producer, 9 MMA
// issuer, 10-11 V cleaning. Shared memory: Q [2 sub-tiles][d / 64][128][64] and a ring of
// K and V blocks [d / 64][128][64] in the order of their use (all 128-byte swizzled).
// TMEM columns: S/P of sub-tiles 0, 1 at 0, 128; O at 256, 256 + d.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <exception>
#include <string>

#include "../../include/dec_api.h"
#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace dec {
namespace {

constexpr int kPage = 16;
constexpr int kKeys = 128;     // keys of a block
constexpr int kRows = 128;     // MMA rows of a sub-tile
constexpr int kCtas = 148;     // runs the work is cut into: the SMs of a B200
constexpr int kThreads = 384;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;  // log2 units
constexpr int kDirty = 8;      // more than the V blocks a ring holds
constexpr int kPoison = 8;     // masked blocks a tile can have: at most 3 on its diagonal and 3 at its window's edge

__device__ int g_chunk_err;    // a bounded wait ran out

dec_status bad(dec_status s, const std::string& why) {
    set_last_error(why);
    return s;
}

template <int D>
struct Shape {
    static constexpr uint32_t kBlock = kKeys * D * 2;  // bytes of a K or V block, and of a sub-tile of Q
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr uint32_t kOffRing = 2 * kBlock;
    static constexpr uint32_t kOffCtl = kOffRing + kStages * kBlock;
    // pieces in the workspace: each CTA's run may begin inside a tile (slot 0) and end inside one (slot 1)
    static constexpr int kSubFloats = kRows * D + 2 * kRows;  // O [d / 4][row][4], m [row], l [row]
    static constexpr int kSlotFloats = 2 * kSubFloats;
};

struct ChunkArgs {
    const int32_t* table;
    const int32_t* cu;
    const int32_t* kv_len;
    int n_pages, max_pages;
    int B, T, nq, nkv, G;
    int tps;         // tokens of a sub-tile
    float scale;
    int window;
    float cap;
    const uint16_t* v_pool;
    uint16_t* out;
    float* ws;
};

// A tile's last run says how to join it (one entry a CTA, at the start of the workspace).
struct Join {
    int first;   // CTA of the tile's first run; -1: nothing to join here
    int row0;    // first q row
    int ntok;    // tokens
    int g;       // kv head
};
constexpr size_t kJoinBytes = 4096;
static_assert(sizeof(Join) * kCtas <= kJoinBytes, "join table");

#define DEC_HD __host__ __device__ __forceinline__

// ------------------------------------------------------------------ work split

struct Seq {
    int row0, n, p0;  // first q row, rows, position of the first row
};

DEC_HD Seq seq_of(const ChunkArgs& a, int b) {
    Seq s;
    const int c0 = min(max(a.cu[b], 0), a.T), c1 = min(max(a.cu[b + 1], c0), a.T);
    s.row0 = c0;
    s.n = c1 - c0;
    s.p0 = min(max(a.kv_len[b], 0), a.max_pages * kPage) - s.n;
    return s;
}

// sum over i < n of floor((a i + b) / m), a, b >= 0, by Euclid's algorithm on (a, m).
__host__ __device__ __noinline__ long long floor_sum(long long n, unsigned m, unsigned a, unsigned b) {
    long long s = 0;
    while (n > 0) {
        s += (n - 1) * n / 2 * (a / m) + n * (b / m);
        a %= m;
        b %= m;
        const unsigned long long y = (unsigned long long)a * (unsigned long long)n + b;
        if (y < m) break;
        n = (long long)(y / m);
        b = (unsigned)(y % m);
        const unsigned t = m;
        m = a;
        a = t;
    }
    return s;
}

// sum over i < t of floor(max(c + i step, 0) / 128)
DEC_HD long long block_sum(int t, int c, int step) {
    const int skip = c < 0 ? (int)((-(long long)c + step - 1) / step) : 0;
    return t > skip ? floor_sum(t - skip, kKeys, step, c + skip * step) : 0;
}

// Last and first key that rows t0 .. t1 of a sequence see, for the block range: a range that
// lies below position 0 still gets block 0, so that its rows are visited (and set to zero).
DEC_HD int hi_key(const Seq& s, int t1) { return max(s.p0 + t1, 0); }
DEC_HD int lo_key(const ChunkArgs& a, const Seq& s, int t0) {
    return a.window > 0 ? (int)max((long long)s.p0 + t0 + 1 - a.window, 0ll) : 0;
}

// Blocks of the first t tiles, all of them full.
DEC_HD long long blocks_before(const ChunkArgs& a, const Seq& s, int t) {
    if (t == 0) return 0;
    const int tpt = 2 * a.tps;
    long long f = t + block_sum(t, s.p0 + tpt - 1, tpt);
    // before position 0 the window starts at 0 as well: p0 + 1 - W is at least -2^30 - 2^31 and may
    // leave 32 bits, where every term of such a tile count is 0
    const long long c = (long long)s.p0 + 1 - a.window;
    if (a.window > 0 && c + (long long)t * tpt > 0) f -= block_sum(t, (int)c, tpt);
    return f;
}

DEC_HD int tile_count(const ChunkArgs& a, const Seq& s) { return (s.n + 2 * a.tps - 1) / (2 * a.tps); }

DEC_HD int tile_blocks(const ChunkArgs& a, const Seq& s, int t) {
    const int t0 = t * 2 * a.tps, t1 = min(s.n, t0 + 2 * a.tps) - 1;
    return hi_key(s, t1) / kKeys - lo_key(a, s, t0) / kKeys + 1;
}

// Blocks of one kv head of a sequence.
DEC_HD long long seq_blocks(const ChunkArgs& a, const Seq& s) {
    if (s.n == 0) return 0;
    const int nt = tile_count(a, s);
    return blocks_before(a, s, nt - 1) + tile_blocks(a, s, nt - 1);
}

// The run of one CTA: where it starts, and how many blocks it has.
struct Run {
    int b, g, tile, off;  // sequence, kv head, tile, block within the tile
    int len;
    int first;            // CTA of the run in which the first tile starts
};

// The run of units u0 .. u1 - 1, which starts in sequence b or after it (`before`: units of the
// sequences below b).
DEC_HD Run run_from(const ChunkArgs& a, int b, long long before, long long u0, long long u1, long long runs,
                    long long total) {
    long long r = u0 - before;
    Seq s = seq_of(a, b);
    long long per_head = seq_blocks(a, s);
    while (r >= per_head * a.nkv) {
        r -= per_head * a.nkv;
        s = seq_of(a, ++b);
        per_head = seq_blocks(a, s);
    }
    Run f;
    f.b = b;
    f.g = (int)(r / per_head);
    r %= per_head;
    int lo = 0, hi = tile_count(a, s);
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (blocks_before(a, s, mid) <= r)
            lo = mid;
        else
            hi = mid;
    }
    f.tile = lo;
    f.off = (int)(r - blocks_before(a, s, lo));
    f.len = (int)(u1 - u0);
    // runs are never empty, so the CTA whose run holds unit u is the last one that starts at or before it
    f.first = (int)(((u0 - f.off + 1) * runs - 1) / total);
    return f;
}

// Called by all threads of a CTA; scratch: 40 long longs of shared memory.
DEC_DEVINL Run find_run(const ChunkArgs& a, int cta, long long* scratch) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
    long long own = 0;
    for (int b = b0; b < b1; ++b) own += seq_blocks(a, seq_of(a, b)) * a.nkv;
    long long x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    Run* found = reinterpret_cast<Run*>(scratch + 34);
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    const long long runs = min((long long)kCtas, total);
    if (cta < runs) {
        const long long u0 = cta * total / runs, u1 = (cta + 1) * total / runs;
        before += x - own;
        if (u0 >= before && u0 < before + own) {
            *found = run_from(a, b0, before, u0, u1, runs, total);
        }
    }
    __syncthreads();
    Run f;
    if (cta < runs) {
        f = *found;
    } else {
        f.b = f.g = f.tile = f.off = f.len = f.first = 0;
    }
    __syncthreads();
    return f;
}

// A piece of the run: consecutive blocks of one tile.
struct Piece {
    int b, g, t0, ntok, row0, p0;
    int kb0, nb;      // blocks kb0 .. kb0 + nb - 1
    int hi, lo;       // the tile's last and first key
    bool two, starts, ends;

    // Block range [from, to) of sub-tile s, relative to kb0 (two = true).
    DEC_HD void range(const ChunkArgs& a, int s, int* from, int* to) const {
        const int f = s * a.tps, l = min(ntok, f + a.tps) - 1;  // tokens of the tile
        const int h = p0 + t0 + l;
        const long long w = a.window > 0 ? (long long)p0 + t0 + f + 1 - a.window : 0;
        const int lw = w > 0 ? (int)w : 0;
        *from = min(max(lw / kKeys - kb0, 0), nb);
        *to = h < 0 ? *from : min(max(h / kKeys + 1 - kb0, *from), nb);
    }
    // Whether rows of the tile differ in the keys they see, or see none: then no value of V
    // that is not finite may stay in a masked block.
    DEC_HD bool notes() const { return ntok > 1 || p0 + t0 < 0; }
    // Whether some row of the tile does not see some key of block kb for its position alone.
    DEC_HD bool masked(const ChunkArgs& a, int kb) const {
        if (kb * kKeys + kKeys - 1 > p0 + t0) return true;
        return a.window > 0 && (long long)kb * kKeys < (long long)p0 + t0 + ntok - a.window;
    }
};

// Walks a run piece by piece; every warp does so for itself.
struct Walk {
    Run r;
    Seq s;
    DEC_HD Walk(const ChunkArgs& a, const Run& run) : r(run) {
        if (r.len > 0) s = seq_of(a, r.b);
    }
    DEC_HD bool next(const ChunkArgs& a, Piece* p) {
        if (r.len <= 0) return false;
        p->b = r.b;
        p->g = r.g;
        p->t0 = r.tile * 2 * a.tps;
        p->ntok = min(s.n - p->t0, 2 * a.tps);
        p->row0 = s.row0 + p->t0;
        p->p0 = s.p0;
        p->hi = hi_key(s, p->t0 + p->ntok - 1);
        p->lo = lo_key(a, s, p->t0);
        p->two = p->ntok > a.tps;
        const int blocks = p->hi / kKeys - p->lo / kKeys + 1;
        p->kb0 = p->lo / kKeys + r.off;
        p->nb = min(blocks - r.off, r.len);
        p->starts = r.off == 0;
        p->ends = r.off + p->nb == blocks;
        r.len -= p->nb;
        r.off = 0;
        if (r.len > 0) {  // the tile is done
            if (++r.tile == tile_count(a, s)) {
                r.tile = 0;
                if (++r.g == a.nkv) {
                    r.g = 0;
                    do s = seq_of(a, ++r.b);
                    while (s.n == 0);
                }
            }
        }
        return true;
    }
};

// ------------------------------------------------------------------ kernel

struct Poison {
    int n;                 // entries
    int kb[kPoison];
    uint32_t keys[kPoison][4];
};

struct Control {
    uint64_t q_full, q_empty;
    uint64_t full[10], empty[10];
    uint64_t dirty[kDirty]; // loads of V blocks to be cleaned, in their order; the cleaning completes full[stage]
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t o_free;       // the epilogue has read O: 8 warps
    uint64_t clean_done;   // a piece's notes are complete: 2 warps
    uint32_t tmem;
    Poison poison;
    union {
        long long scratch[40];
        float2 xch[2][kRows];  // (m, l) of the two halves of a `one` tile
    };
};

// A barrier over `n` threads that tells all of them whether every one passed true.
DEC_DEVINL bool named_bar_and(uint32_t id, uint32_t n, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}

DEC_DEVINL void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
    tmem_ld16_issue(taddr, r);
    tmem_ld16_issue(taddr + 16, r + 16);
}

// The softcapped score c tanh(x / c) in log2 units, by tanh(y) = 1 - 2 / (e^2y + 1): off by
// some 2^-21 c, which for c <= 64 moves a weight by less than 2^-14. Larger caps take tanhf.
DEC_DEVINL float capped(float raw, float k2, float c, float c_log2e) {
    float e = ex2f(raw * k2), r;  // k2 = 2 log2(e) scale / c
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.0f));
    return fmaf(-2.0f * c_log2e, r, c_log2e);
}
__device__ __noinline__ float capped_large(float raw, float scale, float c) {
    return c * tanhf(raw * scale / c) * kLog2e;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const ChunkArgs a) {
    using S = Shape<D>;
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    Control& ctl = *reinterpret_cast<Control*>(smem + S::kOffCtl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* err = &g_chunk_err;

    if (threadIdx.x == 0) {
        mbar_init(&ctl.q_full, 1);
        mbar_init(&ctl.q_empty, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.empty[i], 1);
        }
        for (int i = 0; i < kDirty; ++i) mbar_init(&ctl.dirty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.s_full[i], 1);
            mbar_init(&ctl.p_full[i], 4);
            mbar_init(&ctl.pv_done[i], 1);
        }
        mbar_init(&ctl.o_free, 8);
        mbar_init(&ctl.clean_done, 2);
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    const uint32_t tO = tmem + 2 * kKeys;  // S/P of sub-tile s at tmem + 128 s, its O at tO + D s
    pdl_trigger();
    const Run run = find_run(a, blockIdx.x, ctl.scratch);
    Walk walk(a, run);
    Piece pc;

    if (warp == 8) {
        // ---------------------------------------------------------- TMA producer
        // lane l loads half l / 8 (64 columns) of page l % 8 of a block
        const int pool_rows = a.n_pages * a.nkv * kPage;
        int item = 0, n = 0, nd = 0;  // ring items, pieces, blocks to be cleaned
        bool ok = true;
        while (ok && walk.next(a, &pc)) {
            const int page_lo = pc.lo / kPage, page_hi = pc.hi / kPage;
            const int32_t* tab = a.table + (size_t)pc.b * a.max_pages;
            // pool row of the lane's page of block k of the piece; a page outside the pool gets a row
            // past its end, which the TMA unit fills with zeros; -1: no key of the tile is on the page
            auto row_of = [&](int k) {
                const int pi = (pc.kb0 + k) * (kKeys / kPage) + (lane & 7);
                if (k >= pc.nb || pi < page_lo || pi > page_hi) return -1;
                const int pg = tab[pi];
                return pg >= 0 && pg < a.n_pages ? (pg * a.nkv + pc.g) * kPage : pool_rows;
            };
            const int LA = pc.two ? 1 : 2;
            int r0 = row_of(0), r1 = row_of(1), r2 = row_of(2), r3;
            if (n > 0 && !mbar_wait_bounded(&ctl.q_empty, (n - 1) & 1, err)) break;
            if (lane == 0) {
                const int subs = pc.two ? 2 : 1;
                mbar_arrive_expect_tx(&ctl.q_full, (uint32_t)(subs * a.tps * a.G * D * 2));
                for (int s = 0; s < subs; ++s)
                    for (int h = 0; h < D / 64; ++h)
                        tma_load_3d(smem + s * S::kBlock + h * 16384, &tmQ, h * 64, pc.g * a.G, pc.row0 + s * a.tps,
                                    &ctl.q_full);
            }
            __syncwarp();
            auto load = [&](const CUtensorMap* tm, int row, bool clean) {
                const int st = item % kStages;
                if (item >= kStages && !mbar_wait_bounded(&ctl.empty[st], (item / kStages - 1) & 1, err)) {
                    ok = false;
                    return;
                }
                ++item;
                uint64_t* bar = clean ? &ctl.dirty[nd++ % kDirty] : &ctl.full[st];
                const int pages = __popc(__ballot_sync(0xffffffffu, lane < 8 && row >= 0));
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(pages * kPage * D * 2));
                __syncwarp();
                if (row >= 0 && lane < D / 8)
                    tma_load_2d(smem + S::kOffRing + st * S::kBlock + (lane >> 3) * 16384 + (lane & 7) * 2048, tm,
                                (lane >> 3) * 64, row, bar);
                __syncwarp();
            };
            load(&tmK, r0, false);
            if (ok && LA == 2 && pc.nb > 1) load(&tmK, r1, false);
            for (int k = 0; k < pc.nb && ok; ++k) {
                r3 = row_of(k + 3);
                load(&tmV, r0, pc.masked(a, pc.kb0 + k));
                if (ok && k + LA < pc.nb) load(&tmK, LA == 1 ? r1 : r2, false);
                r0 = r1;
                r1 = r2;
                r2 = r3;
            }
            ++n;
        }
    } else if (warp == 9) {
        // ---------------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_tc<128, 128, false>();
            constexpr uint32_t id_o = idesc_tc<128, D, true>();
            const uint32_t sb = smem_u32(smem);
            int item = 0, n = 0;
            uint32_t p_par = 0;               // parity of p_full[s] in bit s
            bool ok = true;
            auto take = [&](int* st) {        // the next ring item, loaded
                *st = item % kStages;
                ok = ok && mbar_wait_bounded(&ctl.full[*st], (item / kStages) & 1, err);
                ++item;
            };
            auto issue_s = [&](int s, int st, bool two) {
                const uint32_t qb = sb + (two ? s : 0) * S::kBlock, kb = sb + S::kOffRing + st * S::kBlock;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_mma(tmem + s * kKeys, sdesc_sw128(qb + (kk >> 2) * 16384 + (kk & 3) * 32),
                           sdesc_sw128(kb + (kk >> 2) * 16384 + (kk & 3) * 32), id_s, kk > 0 ? 1u : 0u);
                tc_commit(&ctl.s_full[s]);
            };
            auto wait_p = [&](int s) {
                ok = ok && mbar_wait_bounded(&ctl.p_full[s], (p_par >> s) & 1, err);
                p_par ^= 1u << s;
            };
            auto issue_o = [&](int s, int st, bool first) {
                const uint32_t vb = sb + S::kOffRing + st * S::kBlock;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    tc_mma_tmem_a(tO + s * D, tmem + s * kKeys + kk * 8, sdesc_sw128_mn(vb + kk * 2048), id_o,
                                  !first || kk > 0 ? 1u : 0u);
                tc_commit(&ctl.pv_done[s]);
            };
            while (ok && walk.next(a, &pc)) {
                ok = mbar_wait_bounded(&ctl.q_full, n & 1, err);
                int st = 0, sk = 0;
                bool freed = n == 0;  // the last piece's O has been read
                auto wait_o = [&]() {
                    if (!freed) ok = ok && mbar_wait_bounded(&ctl.o_free, (n - 1) & 1, err);
                    freed = true;
                };
                if (pc.two) {
                    int from[2], to[2];
                    pc.range(a, 0, &from[0], &to[0]);
                    pc.range(a, 1, &from[1], &to[1]);
                    if (ok) take(&sk);
                    for (int s = 0; s < 2 && ok; ++s)
                        if (from[s] == 0 && to[s] > 0) issue_s(s, sk, true);
                    if (ok) tc_commit(&ctl.empty[sk]);
                    if (ok && pc.nb == 1) tc_commit(&ctl.q_empty);
                    for (int j = 0; j < pc.nb && ok; ++j) {
                        take(&st);
                        for (int s = 0; s < 2 && ok; ++s) {
                            if (j >= from[s] && j < to[s]) {
                                wait_p(s);
                                wait_o();
                                if (!ok) break;
                                issue_o(s, st, j == from[s]);
                            }
                            if (s == 1) tc_commit(&ctl.empty[st]);
                            if (j + 1 < pc.nb) {
                                if (s == 0) take(&sk);
                                if (!ok) break;
                                if (j + 1 >= from[s] && j + 1 < to[s]) issue_s(s, sk, true);
                                if (s == 1) tc_commit(&ctl.empty[sk]);
                                if (s == 1 && j + 2 == pc.nb) tc_commit(&ctl.q_empty);
                            }
                        }
                    }
                } else {
                    for (int k = 0; k < 2 && k < pc.nb && ok; ++k) {
                        take(&sk);
                        if (!ok) break;
                        issue_s(k, sk, false);
                        tc_commit(&ctl.empty[sk]);
                        if (k + 1 == pc.nb || (k == 1 && pc.nb == 2)) tc_commit(&ctl.q_empty);
                    }
                    for (int k = 0; k < pc.nb && ok; ++k) {
                        const int s = k & 1;
                        take(&st);
                        wait_p(s);
                        wait_o();
                        if (!ok) break;
                        issue_o(s, st, k < 2);
                        tc_commit(&ctl.empty[st]);
                        if (k + 2 < pc.nb) {
                            take(&sk);
                            if (!ok) break;
                            issue_s(s, sk, false);
                            tc_commit(&ctl.empty[sk]);
                            if (k + 3 == pc.nb) tc_commit(&ctl.q_empty);
                        }
                    }
                }
                ++n;
            }
        }
        __syncwarp();
    } else if (warp >= 10) {
        // ---------------------------------------------------------- V cleaning (two warps, half the keys each)
        const int half = warp - 10;
        int item = 0, n = 0, nd = 0;
        bool ok = true;
        while (ok && walk.next(a, &pc)) {
            const bool notes = pc.notes();
            // the last piece's notes have been read; waited for at every piece, because a parity tells
            // only neighbouring phases apart
            if (n > 0) ok = mbar_wait_bounded(&ctl.o_free, (n - 1) & 1, err);
            if (notes && half == 0 && lane == 0) ctl.poison.n = 0;
            ok = named_bar_and(2, 64, ok);
            int entry = 0;
            const int LA = pc.two ? 1 : 2;
            item += min(LA, pc.nb);  // the first K blocks
            for (int k = 0; k < pc.nb && ok; ++k) {
                const int st = item % kStages;
                item += k + LA < pc.nb ? 2 : 1;
                const int kb = pc.kb0 + k;
                if (!pc.masked(a, kb)) continue;
                // every masked block is waited for, in order, and the MMA of a block waits for its cleaning
                ok = named_bar_and(2, 64, mbar_wait_bounded(&ctl.dirty[nd % kDirty], (nd / kDirty) & 1, err));
                if (!ok) break;
                ++nd;
                uint8_t* blk = smem + S::kOffRing + st * S::kBlock;
                uint32_t found[2] = {0u, 0u};  // keys of this half with values that are not finite
                // 8 lanes a 128-byte row (its 16-byte chunks are permuted by the swizzle, which does not matter here)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll 4
                    for (int i = 0; i < 8 * (D / 64); ++i) {
                        const int r = 4 * (i & 7) + (lane >> 3);
                        const int key = half * 64 + q * 32 + r, pos = kb * kKeys + key;
                        uint4* at = reinterpret_cast<uint4*>(blk + (i >> 3) * 16384 + key * 128 + (lane & 7) * 16);
                        if (pos < pc.lo || pos > pc.hi) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                        } else if (notes) {
                            uint4 v = *at;
                            // a bf16 that is not finite has all exponent bits: adding 1 there carries into the sign's place
                            const uint32_t m = 0x7f807f80u, one = 0x00800080u, top = 0x80008000u;
                            const uint32_t any = ((((v.x & m) + one) | ((v.y & m) + one)) |
                                                  (((v.z & m) + one) | ((v.w & m) + one))) & top;
                            if (any) {
                                uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint32_t t = ((w[i] & m) + one) & top;
                                    if (t & 0x8000u) w[i] &= 0xffff0000u;
                                    if (t & 0x80000000u) w[i] &= 0x0000ffffu;
                                }
                                *at = v;
                                found[q] |= 1u << r;
                            }
                        }
                    }
                if (notes) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        found[i] = __reduce_or_sync(0xffffffffu, found[i]);
                        if (lane == 0 && entry < kPoison) ctl.poison.keys[entry][2 * half + i] = found[i];
                    }
                    if (half == 0 && lane == 0 && entry < kPoison) ctl.poison.kb[entry] = kb;
                    ++entry;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMA reads what was stored here
                named_bar_sync(2, 64);
                if (half == 0 && lane == 0) mbar_arrive(&ctl.full[st]);
            }
            if (half == 0 && lane == 0 && notes) ctl.poison.n = min(entry, kPoison);
            __syncwarp();
            if (lane == 0 && notes) mbar_arrive(&ctl.clean_done);
            ++n;
        }
    } else {
        // ---------------------------------------------------------- softmax and epilogue
        const int s = warp >> 2;               // sub-tile
        const int r = (warp & 3) * 32 + lane;  // row of the sub-tile = TMEM lane
        const int tl = r / a.G, hh = r - tl * a.G;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t sa = tmem + s * kKeys + lane_off;
        const float sl2 = a.scale * kLog2e;
        const bool cap = a.cap > 0.f;
        const float k2 = cap ? 2.0f * kLog2e * a.scale / a.cap : 0.f, c_log2e = a.cap * kLog2e;
        int noted = 0;        // pieces with notes so far
        int cnt[2] = {0, 0};  // blocks of either sub-tile so far (phases of s_full and pv_done)
        bool ok = true;
        while (walk.next(a, &pc)) {
            const int tok = pc.two ? s * a.tps + tl : tl;  // token of the tile
            const bool valid = tl < a.tps && tok < pc.ntok;
            const int pos = pc.p0 + pc.t0 + tok;
            const int lo = a.window > 0 ? (int)max((long long)pos + 1 - a.window, 0ll) : 0;
            int from[2], to[2];  // blocks of either sub-tile: from, from + step, .. < to
            const int step = pc.two ? 1 : 2;
            if (pc.two) {
                pc.range(a, 0, &from[0], &to[0]);
                pc.range(a, 1, &from[1], &to[1]);
            } else {
                from[0] = 0;
                from[1] = 1;
                to[0] = to[1] = pc.nb;
            }
            const int32_t* tab = a.table + (size_t)pc.b * a.max_pages;
            auto page_ok = [&](int k) {  // whether the lane's page of block k lies in the pool
                const int pi = (pc.kb0 + k) * (kKeys / kPage) + (lane & 7);
                if (k >= to[s] || pi >= a.max_pages) return false;
                const int pg = tab[pi];
                return pg >= 0 && pg < a.n_pages;
            };
            bool pg = page_ok(from[s]);
            float m = -INFINITY, l = 0.f;
            for (int j = from[s]; j < to[s]; j += step) {
                const uint32_t good = __ballot_sync(0xffffffffu, pg) & 0xffu;
                pg = page_ok(j + step);
                const int key0 = (pc.kb0 + j) * kKeys;
                const bool none = !valid || key0 > pos || key0 + kKeys - 1 < lo;
                const bool whole = !none && key0 + kKeys - 1 <= pos && key0 >= lo && good == 0xffu;
                if (ok && !mbar_wait_bounded(&ctl.s_full[s], cnt[s] & 1, err)) ok = false;
                tc_fence_after();
                uint32_t v[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_issue(sa + 32 * c, v[c]);
                tmem_ld_wait32(v[3]);
                reg_fence32(v[0]);
                reg_fence32(v[1]);
                reg_fence32(v[2]);
                if (cap) {
                    if (a.cap <= 64.f) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int q = 0; q < 32; ++q)
                                v[c][q] = __float_as_uint(capped(__uint_as_float(v[c][q]), k2, a.cap, c_log2e));
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int q = 0; q < 32; ++q)
                                v[c][q] = __float_as_uint(capped_large(__uint_as_float(v[c][q]), a.scale, a.cap));
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int q = 0; q < 32; ++q) {
                            const int key = key0 + 32 * c + q;
                            if (none || key > pos || key < lo || !((good >> (2 * c + q / 16)) & 1))
                                v[c][q] = __float_as_uint(-INFINITY);
                        }
                }
                float bm4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int q = 0; q < 32; ++q) bm4[q & 3] = fmaxf(bm4[q & 3], __uint_as_float(v[c][q]));
                const float bm = fmaxf(fmaxf(bm4[0], bm4[1]), fmaxf(bm4[2], bm4[3])) * (cap ? 1.f : sl2);
                const float mn = fmaxf(m, bm);
                const bool grow = m != -INFINITY && mn > m + kRescale;
                const float corr = grow ? ex2f(m - mn) : 1.f;
                if (grow || m == -INFINITY) m = mn;
                l *= corr;
                // P = 2^(S' - m), rounded to bf16, over the scores (keys 2i, 2i + 1 in column i)
                const float2 mul2 = cap ? make_float2(1.f, 1.f) : make_float2(sl2, sl2);
                const float nm = m == -INFINITY ? 0.f : -m;  // nothing seen yet: every score is -inf, 2^-inf = 0
                const float2 nm2 = make_float2(nm, nm);
                float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t ph[16];
#pragma unroll
                    for (int q = 0; q < 32; q += 2) {
                        const float2 x =
                            ffma2(make_float2(__uint_as_float(v[c][q]), __uint_as_float(v[c][q + 1])), mul2, nm2);
                        const float2 p = make_float2(ex2f(x.x), ex2f(x.y));
                        sum2[(q >> 1) & 1] = fadd2(sum2[(q >> 1) & 1], p);
                        ph[q / 2] = pack_bf2(p.x, p.y);
                    }
                    tmem_st16(sa + 16 * c, ph);
                }
                l += (sum2[0].x + sum2[1].x) + (sum2[0].y + sum2[1].y);
                if (__any_sync(0xffffffffu, grow) && j > from[s]) {
                    // O of the rows that grew, once the last block's product is in
                    if (ok && !mbar_wait_bounded(&ctl.pv_done[s], (cnt[s] - 1) & 1, err)) ok = false;
                    tc_fence_after();
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld32_issue(tO + s * D + lane_off + c0, o);
                        tmem_ld_wait32(o);
#pragma unroll
                        for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * corr);
                        tmem_st16(tO + s * D + lane_off + c0, o);
                        tmem_st16(tO + s * D + lane_off + c0 + 16, o + 16);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_full[s]);
                ++cnt[s];
            }
            {  // the other sub-tile's count
                const int o = s ^ 1;
                cnt[o] += from[o] < to[o] ? (to[o] - from[o] + step - 1) / step : 0;
            }

            // ---- epilogue
            const bool have[2] = {from[0] < to[0], from[1] < to[1]};
            if (have[s] && ok && !mbar_wait_bounded(&ctl.pv_done[s], (cnt[s] - 1) & 1, err)) ok = false;
            float w[2] = {1.f, 1.f};  // weights of the two O's
            if (!pc.two) {
                if (have[s ^ 1] && ok && !mbar_wait_bounded(&ctl.pv_done[s ^ 1], (cnt[s ^ 1] - 1) & 1, err)) ok = false;
                ctl.xch[s][r] = make_float2(m, l);
                named_bar_sync(1, 256);
                const float2 x = ctl.xch[0][r], y = ctl.xch[1][r];
                m = fmaxf(x.x, y.x);
                w[0] = x.x == -INFINITY ? 0.f : ex2f(x.x - m);
                w[1] = y.x == -INFINITY ? 0.f : ex2f(y.x - m);
                l = x.y * w[0] + y.y * w[1];
                named_bar_sync(1, 256);
            }
            int poisoned = 0;
            if (pc.notes()) {
                if (ok && !mbar_wait_bounded(&ctl.clean_done, noted & 1, err)) ok = false;
                ++noted;
                poisoned = ctl.poison.n;
            }
            tc_fence_after();
            // columns of this thread: all of its sub-tile's, or half of the joined result's
            const int c_lo = pc.two ? 0 : s * (D / 2), c_hi = pc.two ? D : c_lo + D / 2;
            const bool whole_tile = pc.starts && pc.ends;
            const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
            uint16_t* dst = a.out + ((size_t)(pc.row0 + tok) * a.nq + (size_t)pc.g * a.G + hh) * D;
            float* slot = a.ws + (size_t)(2 * blockIdx.x + (pc.starts ? 1 : 0)) * S::kSlotFloats +
                          (pc.two ? s * S::kSubFloats : 0);
            for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
                uint32_t o[32];
                if (pc.two) {
                    if (have[s]) {
                        tmem_ld32_issue(tO + s * D + lane_off + c0, o);
                        tmem_ld_wait32(o);
                    } else {
#pragma unroll
                        for (int q = 0; q < 32; ++q) o[q] = 0u;
                    }
                } else {
                    tmem_ld32_issue(tO + lane_off + c0, o);  // sub-tile 0 has the first block of every piece
                    tmem_ld_wait32(o);
#pragma unroll
                    for (int q = 0; q < 32; ++q)
                        o[q] = w[0] == 0.f ? 0u : __float_as_uint(__uint_as_float(o[q]) * w[0]);
                    if (have[1]) {
                        uint32_t o1[32];
                        tmem_ld32_issue(tO + D + lane_off + c0, o1);
                        tmem_ld_wait32(o1);
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            if (w[1] != 0.f)
                                o[q] = __float_as_uint(fmaf(__uint_as_float(o1[q]), w[1], __uint_as_float(o[q])));
                    }
                }
                if (poisoned && valid) {
                    for (int e = 0; e < poisoned; ++e)
                        for (int i = 0; i < 4; ++i)
                            for (uint32_t bits = ctl.poison.keys[e][i]; bits; bits &= bits - 1) {
                                const int key = ctl.poison.kb[e] * kKeys + 32 * i + __ffs(bits) - 1;
                                if (key > pos || key < lo) continue;
                                const int page = tab[key / kPage];
                                if (page < 0 || page >= a.n_pages) continue;
                                const uint16_t* vr =
                                    a.v_pool + (((size_t)page * a.nkv + pc.g) * kPage + key % kPage) * D + c0;
#pragma unroll
                                for (int q = 0; q < 32; ++q) {
                                    const float x = bf2f(vr[q]);
                                    if (!(fabsf(x) < INFINITY)) o[q] = __float_as_uint(__uint_as_float(o[q]) + x);
                                }
                            }
                }
                if (valid && ok) {
                    if (whole_tile) {
#pragma unroll
                        for (int q = 0; q < 32; q += 8) {
                            uint4 y;
                            y.x = pack_bf2(__uint_as_float(o[q]) * inv, __uint_as_float(o[q + 1]) * inv);
                            y.y = pack_bf2(__uint_as_float(o[q + 2]) * inv, __uint_as_float(o[q + 3]) * inv);
                            y.z = pack_bf2(__uint_as_float(o[q + 4]) * inv, __uint_as_float(o[q + 5]) * inv);
                            y.w = pack_bf2(__uint_as_float(o[q + 6]) * inv, __uint_as_float(o[q + 7]) * inv);
                            *reinterpret_cast<uint4*>(dst + c0 + q) = y;
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 32; q += 4)
                            *reinterpret_cast<uint4*>(slot + ((size_t)((c0 + q) / 4) * kRows + r) * 4) =
                                make_uint4(o[q], o[q + 1], o[q + 2], o[q + 3]);
                    }
                }
            }
            if (valid && ok && !whole_tile && c_lo == 0) {
                slot[kRows * D + r] = m;
                slot[kRows * D + kRows + r] = l;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.o_free);
        }
    }
    // what the join needs to know of a tile that this run ends without having started it: the
    // run's first piece
    if (threadIdx.x == 0) {
        Join jn{-1, 0, 0, 0};
        Walk w2(a, run);
        if (w2.next(a, &pc) && !pc.starts && pc.ends) jn = Join{run.first, pc.row0, pc.ntok, pc.g};
        reinterpret_cast<Join*>(reinterpret_cast<char*>(a.ws) - kJoinBytes)[blockIdx.x] = jn;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Joins the pieces of the tile whose last piece is CTA blockIdx.x's first: with M the largest m,
// O = sum 2^(m_i - M) O_i, l = sum 2^(m_i - M) l_i, in the order of the runs. A block takes 32 rows.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const ChunkArgs a) {
    using S = Shape<D>;
    pdl_wait();
    const int last = blockIdx.x, part = blockIdx.y;
    const Join jn = reinterpret_cast<const Join*>(reinterpret_cast<const char*>(a.ws) - kJoinBytes)[last];
    if (jn.first < 0) return;
    const int sub = part >> 2, rows = 32 * (part & 3) + (threadIdx.x & 31);
    const int tok = sub * a.tps + rows / a.G, hh = rows % a.G;
    if (rows / a.G >= a.tps || tok >= jn.ntok) return;
    auto piece = [&](int c) {  // a run's piece of the tile: the tail of the first, the head of the others
        return a.ws + (size_t)(2 * c + (c == jn.first ? 1 : 0)) * S::kSlotFloats + sub * S::kSubFloats;
    };
    float M = -INFINITY;
    for (int c = jn.first; c <= last; ++c) M = fmaxf(M, piece(c)[kRows * D + rows]);
    float L = 0.f;
    for (int c = jn.first; c <= last; ++c) {
        const float* p = piece(c);
        const float m = p[kRows * D + rows];
        // a piece that saw nothing adds its l, 0 (NaN when every score was)
        L += (m == -INFINITY ? 1.f : ex2f(m - M)) * p[kRows * D + kRows + rows];
    }
    const float inv = L > 0.f || L != L ? 1.0f / L : 0.f;
    uint16_t* dst = a.out + ((size_t)(jn.row0 + tok) * a.nq + (size_t)jn.g * a.G + hh) * D;
    for (int c4 = threadIdx.x >> 5; c4 < D / 4; c4 += 8) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = jn.first; c <= last; ++c) {
            const float* p = piece(c);
            const float m = p[kRows * D + rows];
            if (m == -INFINITY) continue;
            const float w = ex2f(m - M);
            const float4 x = *reinterpret_cast<const float4*>(p + ((size_t)c4 * kRows + rows) * 4);
            o.x = fmaf(w, x.x, o.x);
            o.y = fmaf(w, x.y, o.y);
            o.z = fmaf(w, x.z, o.z);
            o.w = fmaf(w, x.w, o.w);
        }
        uint2 y;
        y.x = pack_bf2(o.x * inv, o.y * inv);
        y.y = pack_bf2(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2*>(dst + 4 * c4) = y;
    }
}

template <int D>
int64_t workspace_bytes_for() {
    return (int64_t)kJoinBytes + (int64_t)kCtas * 2 * Shape<D>::kSlotFloats * (int64_t)sizeof(float);
}

template <int D>
cudaError_t launch(const ChunkArgs& a, const void* q, int64_t ldq, const void* k_pool, cudaStream_t st) {
    using S = Shape<D>;
    constexpr int smem = (int)(S::kOffCtl + sizeof(Control));
    static_assert(smem <= 232448, "fits the 227 KB a CTA may use");
    CUtensorMap tmQ, tmK, tmV;
    {
        const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.nq, (uint64_t)a.T};
        const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)ldq * 2};
        const uint32_t box[3] = {64, (uint32_t)a.G, (uint32_t)a.tps};
        cudaError_t e = tmap_bf16_sw128(&tmQ, q, 3, dims, strides, box);
        if (e != cudaSuccess) return e;
    }
    {
        const uint64_t dims[2] = {(uint64_t)D, (uint64_t)a.n_pages * a.nkv * kPage};
        const uint64_t strides[1] = {(uint64_t)D * 2};
        const uint32_t box[2] = {64, kPage};
        cudaError_t e = tmap_bf16_sw128(&tmK, k_pool, 2, dims, strides, box);
        if (e == cudaSuccess) e = tmap_bf16_sw128(&tmV, a.v_pool, 2, dims, strides, box);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = ensure_smem(reinterpret_cast<const void*>(chunk_attn_kernel<D>), smem);
    if (e != cudaSuccess) return e;
    chunk_attn_kernel<D><<<kCtas, kThreads, smem, st>>>(tmQ, tmK, tmV, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtas, 8);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, chunk_join_kernel<D>, a);
}

}  // namespace

// The work split on the host: every (tile, block) of every kv head in exactly one piece, in order,
// every cut tile joined once, from the run that starts it. Returns the number of violations.
int chunk_split_check(const int32_t* cu, const int32_t* kv_len, int B, int T, int max_pages, int G, int nkv,
                      int window) {
    ChunkArgs a{};
    a.cu = cu;
    a.kv_len = kv_len;
    a.B = B;
    a.T = T;
    a.max_pages = max_pages;
    a.nkv = nkv;
    a.G = G;
    a.tps = kRows / G;
    a.window = window;
    int wrong = 0;
    long long total = 0;
    for (int b = 0; b < B; ++b) {
        const Seq s = seq_of(a, b);
        long long n = 0;
        for (int t = 0; t < tile_count(a, s); ++t) {
            if (blocks_before(a, s, t) != n) ++wrong;
            if (tile_blocks(a, s, t) < 1) ++wrong;
            n += tile_blocks(a, s, t);
        }
        if (seq_blocks(a, s) != n) ++wrong;
        total += n * nkv;
    }
    // the tiles in order, walked beside the pieces
    int b = -1, g = nkv - 1, t = 0, tiles = 0, off = 0, start_cta = -1;
    auto next_tile = [&]() {
        if (++t >= tiles) {
            t = 0;
            if (++g >= nkv) {
                g = 0;
                do
                    if (++b >= B) return false;
                while ((tiles = tile_count(a, seq_of(a, b))) == 0);
            }
        }
        off = 0;
        return true;
    };
    bool left = next_tile();
    const long long runs = min((long long)kCtas, total);
    for (int c = 0; c < runs; ++c) {
        const Run run = run_from(a, 0, 0, c * total / runs, (c + 1) * total / runs, runs, total);
        Walk w(a, run);
        Piece p;
        int pieces = 0;
        long long len = 0;
        while (w.next(a, &p)) {
            if (!left) return wrong + 1;
            const Seq s = seq_of(a, b);
            const int blocks = tile_blocks(a, s, t);
            if (p.b != b || p.g != g || p.t0 != t * 2 * a.tps || p.nb < 1 || off + p.nb > blocks) ++wrong;
            if (p.kb0 != lo_key(a, s, p.t0) / kKeys + off) ++wrong;
            if (p.starts != (off == 0) || p.ends != (off + p.nb == blocks)) ++wrong;
            if (off == 0) start_cta = c;
            if (!p.starts && (pieces > 0 || run.first != start_cta)) ++wrong;  // only a run's first piece continues a tile
            int from[2], to[2];
            for (int s2 = 0; s2 < 2; ++s2) p.range(a, s2, &from[s2], &to[s2]);
            if (p.two)  // every block is some sub-tile's, and none is outside the piece
                for (int j = 0; j < p.nb; ++j)
                    if (p.p0 + p.t0 >= 0 && !(j >= from[0] && j < to[0]) && !(j >= from[1] && j < to[1])) ++wrong;
            off += p.nb;
            len += p.nb;
            ++pieces;
            if (off == blocks) left = next_tile();
        }
        if (len != run.len) ++wrong;
    }
    return left ? wrong + 1 : wrong;
}

cudaError_t chunk_take_error(int* set) {
    cudaError_t e = cudaMemcpyFromSymbol(set, g_chunk_err, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *set) e = cudaMemcpyToSymbol(g_chunk_err, &zero, sizeof(int));
    return e;
}

}  // namespace dec

using namespace dec;

extern "C" {

int64_t gqa_chunk_attn_workspace(int32_t d) {
    return d == 128 ? workspace_bytes_for<128>() : d == 64 ? workspace_bytes_for<64>() : 0;
}

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
    ChunkArgs a{};
    a.table = block_table;
    a.cu = cu_rows;
    a.kv_len = kv_len;
    a.n_pages = n_pages;
    a.max_pages = max_pages;
    a.B = B;
    a.T = T;
    a.nq = nq;
    a.nkv = nkv;
    a.G = nq / nkv;
    a.tps = kRows / a.G;
    a.scale = scale;
    a.window = window;
    a.cap = softcap;
    a.v_pool = static_cast<const uint16_t*>(v_pool);
    a.out = static_cast<uint16_t*>(out);
    a.ws = reinterpret_cast<float*>(static_cast<char*>(workspace) + kJoinBytes);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = d == 128 ? launch<128>(a, q, ldq, k_pool, st) : launch<64>(a, q, ldq, k_pool, st);
    if (e != cudaSuccess) return bad(DEC_ERR_CUDA, std::string("gqa_chunk_attn: ") + cudaGetErrorString(e));
    return DEC_OK;
} catch (const std::exception&) {
    return DEC_ERR_OOM;
}

}  // extern "C"
