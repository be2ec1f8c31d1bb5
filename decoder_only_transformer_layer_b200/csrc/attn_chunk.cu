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
// not depend on m. P is rounded to bf16 once: each weight is off by at most 2^-8 of itself,
// as much as the rounding of the result; l sums the unrounded fp32 values.
//
// Work split. Lengths are known on the device only, so every CTA cuts the work for itself:
// the (tile, key block) pairs of all sequences, kv heads and tiles form one list, cut into runs
// of equal cost, one for each of 148 CTAs (the number of blocks of the first t tiles of a sequence
// has a closed form, so finding a run's start takes a scan over the sequences and a binary
// search). A long prompt, a batch of decodes, or both at once keep every SM equally busy. A
// tile cut between CTAs leaves unnormalised fp32 pieces (O, m, l) in the workspace, which a
// second kernel joins in the order of the runs, so results do not depend on timing.
//
// Measured (B200, 6.56 TB/s copy, 1610 TFLOP/s cuBLAS). A prompt of 8192 rows, 32/8 heads of 128: 510 us in the
// first calls after a pause (1,078 TFLOP/s), 575-583 in seconds of calls, when the power cap holds the SMs at 1.7
// GHz (cuBLAS does 1370 TFLOP/s then); in both 0.98 M cycles, bound by each sub-tile's chain of scores, softmax
// and products, two of which overlap (tensor cores and exponentials are busy 56% of the time). 32 sequences of
// 5-8 rows at 1000-8000 keys: 117 us (5.3 TB/s), 133-136 in seconds of calls (1.6 GHz, same cause); bound by the
// stream of K and V, and by starting and joining (6 and 8 us). 5 rows at 4096: 17.8 us of latencies. Score blocks of 64 keys, two buffers a sub-tile, would overlap a sub-tile's scores with its own
// products, but a product with N = 64 costs as much as one with N = 128 and every step's issue comes twice: 610 us.
//
// Masked places. Scores outside a row's keys are replaced, so K may hold anything there.
// V reaches a row through P = 0, and 0 x NaN is NaN: in every block in which some row of the
// tile does not see some key, two warps set V rows outside the tile's keys to zero in shared
// memory, and where tokens of the tile see different keys, also take out values that are not
// finite, note their keys, and the epilogue adds those values back to the rows that do see them.
//
// Warps: 0-3 and 4-7 softmax and epilogue of sub-tiles 0 and 1, 8 TMA producer, 9 MMA issuer,
// 10-11 V cleaning. Shared memory: Q [2 sub-tiles][d / 64][128][64] and a ring of
// K and V blocks [d / 64][128][64] in the order of their use (all 128-byte swizzled).
// TMEM columns: S/P of sub-tiles 0, 1 at 0, 128; O at 256, 256 + d.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
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
constexpr int kSubWarps = 4;    // softmax warps of a sub-tile, a thread a row
constexpr int kSoftWarps = 2 * kSubWarps;
constexpr int kThreads = 32 * (kSoftWarps + 4);  // softmax, TMA, MMA, two for cleaning V
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;  // log2 units
// tanh(y) / y as a polynomial in y^2 <= 9/16 (relative minimax fit, off by 2^-20.8 at most)
constexpr float kT0 = 0.999999463558197f, kT1 = -0.3332825005054474f, kT2 = 0.13258983194828033f,
                kT3 = -0.05005630478262901f, kT4 = 0.01292963232845068f;
template <int N>
struct Int {
    static constexpr int value = N;
};
constexpr int kDirty = 8;      // more than the V blocks a ring holds
constexpr long long kLimit = 1ll << 31;  // cycles after which a wait gives up
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
    int stall;  // test hook: this kind of barrier (Stall) never completes
};
enum Stall { kNoStall, kQFull, kQEmpty, kFull, kEmpty, kDirtyBar, kSFull, kPFull, kPvDone, kOFree, kCleanDone, kStalls };

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

// a / b for 0 <= a, 0 < b, in 32 bits where they fit (nearly always): a 64-bit division is a long
// chain of instructions.
DEC_HD long long div_small(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

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
        n = div_small((long long)y, m);
        b = (unsigned)((long long)y - n * m);
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

// What a tile costs beside its blocks (filling the pipeline, the epilogue), in blocks: the runs are
// equal in tiles' costs. A tile's units are kTileCost for nothing, then one for each block. With 3, 4, 5, 6 and 8:
// 24 sequences of which 21 decode 33.2, 33.1, 33.9, 35.6, 36.7 us; 1500 rows in a window of 1024 65.2, 63.9, 67.2, 67.5,
// 65.7; a prompt of 8192 580, 583, 585, 589, 596; 32 sequences of 5-8 rows 135, 136, 136, 136, 138.
constexpr int kTileCost = 4;
// The block at which unit u of a tile lies; a run that ends within the first units has none of it.
DEC_HD int block_at(int u) { return u > kTileCost ? u - kTileCost : 0; }

// Units of the first t tiles, all of them full.
DEC_HD long long units_before(const ChunkArgs& a, const Seq& s, int t) {
    if (t == 0) return 0;
    const int tpt = 2 * a.tps;
    long long f = (long long)t * (1 + kTileCost) + block_sum(t, s.p0 + tpt - 1, tpt);
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

// So many tiles are summed one by one, the closed form is for more. (Without that: 24 sequences with few rows each
// 34.8 instead of 33.1 us, 1500 rows in a window 65.1 instead of 64.0, but one sequence of 5 rows 17.1 instead of 17.8.)
constexpr int kFewTiles = 32;

// Units of one kv head of a sequence.
DEC_HD long long seq_units(const ChunkArgs& a, const Seq& s) {
    if (s.n == 0) return 0;
    const int nt = tile_count(a, s);
    if (nt <= kFewTiles) {
        int u = 0;
        for (int t = 0; t < nt; ++t) u += kTileCost + tile_blocks(a, s, t);
        return u;
    }
    return units_before(a, s, nt - 1) + kTileCost + tile_blocks(a, s, nt - 1);
}

// The run of one CTA: where it starts, and how many units it has.
struct Run {
    int b, g, tile, off;  // sequence, kv head, tile, unit within the tile
    int len;
    int first;            // CTA of the run in which the first tile starts
};

// All units (tile blocks of every kv head) cut into kCtas runs of q or q + 1, the longer ones first.
struct Cut {
    long long q, rem;
    DEC_HD explicit Cut(long long total) : q(total / kCtas), rem(total % kCtas) {}
    DEC_HD long long start(int c) const { return c * q + (c < rem ? c : rem); }
    DEC_HD long long len(int c) const { return q + (c < rem ? 1 : 0); }
    // the CTA whose run holds unit u
    DEC_HD int cta_of(long long u) const {
        const long long longer = rem * (q + 1);
        return (int)(u < longer ? div_small(u, q + 1) : rem + div_small(u - longer, q));
    }
};

// The run of CTA cta, which starts in sequence b or after it (`before`: units of the sequences
// below b).
DEC_HD Run run_from(const ChunkArgs& a, int b, long long before, const Cut& cut, int cta) {
    long long r = cut.start(cta) - before;
    Seq s = seq_of(a, b);
    long long per_head = seq_units(a, s);
    while (r >= per_head * a.nkv) {
        r -= per_head * a.nkv;
        s = seq_of(a, ++b);
        per_head = seq_units(a, s);
    }
    Run f;
    f.b = b;
    f.g = (int)div_small(r, per_head);
    r -= f.g * per_head;
    int lo = 0, hi = tile_count(a, s);
    if (hi <= kFewTiles) {
        for (int u; r >= (u = kTileCost + tile_blocks(a, s, lo)); ++lo) r -= u;
    } else {
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (units_before(a, s, mid) <= r)
                lo = mid;
            else
                hi = mid;
        }
        r -= units_before(a, s, lo);
    }
    f.tile = lo;
    f.off = (int)r;
    f.len = (int)cut.len(cta);
    f.first = cut.cta_of(cut.start(cta) - f.off + kTileCost);
    return f;
}

// Called by all threads of a CTA; scratch: 40 long longs of shared memory.
DEC_DEVINL Run find_run(const ChunkArgs& a, int cta, long long* scratch) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
    long long own = 0;
    for (int b = b0; b < b1; ++b) own += seq_units(a, seq_of(a, b)) * a.nkv;
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
    const Cut cut(total);
    const long long u0 = cut.start(cta);
    before += x - own;
    if (cut.len(cta) > 0 && u0 >= before && u0 < before + own) *found = run_from(a, b0, before, cut, cta);
    __syncthreads();
    Run f{0, 0, 0, 0, 0, 0};
    if (cut.len(cta) > 0) f = *found;
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
    int tiles;
    DEC_HD Walk(const ChunkArgs& a, const Run& run) : r(run) {
        if (r.len > 0) {
            s = seq_of(a, r.b);
            tiles = tile_count(a, s);
        }
    }
    DEC_HD bool next(const ChunkArgs& a, Piece* p) {
        while (r.len > 0)
            if (step(a, p)) return true;
        return false;
    }
    DEC_HD bool step(const ChunkArgs& a, Piece* p) {
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
        const int units = min(kTileCost + blocks - r.off, r.len);
        const int b0 = block_at(r.off);
        p->kb0 = p->lo / kKeys + b0;
        p->nb = block_at(r.off + units) - b0;
        p->starts = b0 == 0;
        p->ends = b0 + p->nb == blocks;
        r.len -= units;
        r.off = 0;
        if (r.len > 0) {  // the tile is done
            if (++r.tile == tiles) {
                r.tile = 0;
                if (++r.g == a.nkv) {
                    r.g = 0;
                    do s = seq_of(a, ++r.b);
                    while (s.n == 0);
                    tiles = tile_count(a, s);
                }
            }
        }
        return p->nb > 0;
    }
};

// ------------------------------------------------------------------ kernel

struct Poison {
    int n;                 // masked blocks noted so far
    uint32_t some[2];      // whether either half has any key noted
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
    uint64_t drain;        // after a failure: every product issued is done
    uint32_t tmem;
    int failed;            // a wait of this CTA gave up
    int qs;                // pieces whose Q is loaded or on its way
    uint32_t sent[10];     // of each place in the ring the last load's barrier (shared address) and phase parity; 0: none
    Poison poison;
    union {
        long long scratch[64];
        float2 ml[2][kRows];  // m and l of the two halves of a `one` tile
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

// A bounded wait (2^31 cycles, about a second), letting the hardware suspend the thread for up to 20 us at a time: a
// warp that polls takes issue slots from the others. Every lane has its own answer, so no control flow that leads to a
// warp-wide instruction depends on it: after a failure a warp walks on to the end of its run without waiting again, and
// only what its lanes issue and store is left out. The loop is kept as small as it can be: looking at the clock
// only every 32nd time takes a prompt of 8192 rows from 573 to 597 us (more polls), a vote over the warp to 619.
DEC_DEVINL bool wait(uint64_t* bar, uint32_t parity, volatile int* failed) {
    auto test = [&]() {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
            : "memory");
        return done != 0;
    };
    if (test()) return true;
    const long long t0 = clock64();
    while (!test()) {
        if (clock64() - t0 > kLimit) {
            *failed = 1;
            return false;
        }
    }
    return true;
}

// tcgen05.ld of 32 columns without waiting.
DEC_DEVINL void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// As reg_fence32, for 16.
DEC_DEVINL void reg_fence16(uint32_t (&r)[16]) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]));
}

constexpr uint32_t kDescHi = (1024 >> 4) | (1 << 14) | (2 << 29);
// Shared-memory descriptors (128-byte swizzle, 8-row groups 1 KB apart) in two words: the upper one
// is constant, the lower one (address and leading offset, in 16 bytes) moves by an addition. The
// MMA thread shares its scheduler with busy softmax warps, so every instruction between two
// MMAs costs: with descriptors built afresh for each, issuing took longer than the products.
//
// MMA and TMA instructions take their operands from uniform registers. From code that only one
// lane runs, each operand goes there by moves of its own, and this warp gets one issue slot in
// several while softmax warps run. So all lanes compute the operands, a reduction over the warp puts
// what they share into a uniform register, and only the instructions are in an elected lane's
// branch: 8 MMAs of 64 cycles then take 512 cycles beside idle warps and 700 beside 16 warps of
// FMAs (lane 0 alone: 512 and 950; predicated one by one: 570 and 1140).
DEC_DEVINL uint32_t uniform(uint32_t v) { return __reduce_or_sync(0xffffffffu, v); }

// One lane of a converged warp, as a predicate the compiler knows to be one.
DEC_DEVINL bool elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// D (+)= A B, both from shared memory.
DEC_DEVINL void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accum), "n"(kDescHi)
        : "memory");
}
// The same with A from TMEM (lanes = rows, two 16-bit elements a column).
DEC_DEVINL void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(idesc), "r"(accum), "n"(kDescHi)
        : "memory");
}
// Arrives on `bar` once all products issued before it are done, if the issuing lane is `ok`. A commit covers what its
// own thread issued, and the products are issued by the lane that elect.sync gives (the same one for the same mask,
// but which one it is nobody promises), so that lane commits. Called by the whole warp.
DEC_DEVINL void commit_elected(uint64_t* bar, bool ok) {
    asm volatile(
        "{\n\t.reg .pred e, o;\n\tsetp.ne.u32 o, %1, 0;\n\telect.sync _|e, 0xffffffff;\n\tand.pred e, e, o;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"((uint32_t)ok)
        : "memory");
}
DEC_DEVINL uint32_t desc_lo(uint32_t saddr, uint32_t leading) { return (saddr >> 4) | (leading << 16); }
// The largest of three, NaN if any is.
DEC_DEVINL float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
DEC_DEVINL float2 fmul2(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}
DEC_DEVINL float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// tanh(y) = 1 - 2 / (e^2y + 1), off by some 2^-22 (2^-20 of the value at 1/4), above |y| = 1/4, its Taylor series
// (next term 62 y^9 / 2835, 2^-21.5 of the value there) below, so that the error of c tanh(s / c) stays
// below a 2^-18 part of the score whatever the cap.
DEC_DEVINL float tanh_exact(float y) {
    const float y2 = y * y;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2f(y * (2.0f * kLog2e)) + 1.0f));
    const float big = fmaf(-2.0f, r, 1.0f);
    const float small = y * fmaf(y2, fmaf(y2, fmaf(y2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.0f);
    return y2 < 0.0625f ? small : big;
}

// After a failure: shared memory and TMEM go to the next CTA only when nothing is in flight into them. Called by the MMA
// warp, which waits for the products it issued, the last loads into the ring (at most one a stage) and the last Q.
// Out of line: inside the kernel it costs the shortest calls 0.1 us.
__device__ __noinline__ void drain(Control& ctl, int stages) {
    volatile int* failed = &ctl.failed;
    if ((threadIdx.x & 31) == 0) atomicExch(&g_chunk_err, 1);
    commit_elected(&ctl.drain, true);
    bool in = wait(&ctl.drain, 0, failed);
    for (int i = 0; in && i < stages; ++i)
        if (const uint32_t at = ctl.sent[i])
            in = wait(reinterpret_cast<uint64_t*>(__cvta_shared_to_generic(at & ~1u)), at & 1, failed);
    if (in && ctl.qs > 0) wait(&ctl.q_full, (ctl.qs - 1) & 1, failed);
    __syncwarp();
}

template <int D, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const ChunkArgs a) {
    using S = Shape<D>;
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    Control& ctl = *reinterpret_cast<Control*>(smem + S::kOffCtl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* failed = &ctl.failed;

    if (threadIdx.x == 0) {
        auto init = [&](uint64_t* bar, int arrivals, Stall kind) {
            mbar_init(bar, arrivals + (a.stall == kind ? 1 << 16 : 0));
        };
        init(&ctl.q_full, 1, kQFull);
        init(&ctl.q_empty, 1, kQEmpty);
        for (int i = 0; i < kStages; ++i) {
            init(&ctl.full[i], 1, kFull);
            init(&ctl.empty[i], 1, kEmpty);
        }
        for (int i = 0; i < kDirty; ++i) init(&ctl.dirty[i], 1, kDirtyBar);
        for (int i = 0; i < 2; ++i) {
            init(&ctl.s_full[i], 1, kSFull);
            init(&ctl.p_full[i], kSubWarps, kPFull);
            init(&ctl.pv_done[i], 1, kPvDone);
        }
        init(&ctl.o_free, kSoftWarps, kOFree);
        init(&ctl.clean_done, 2, kCleanDone);
        mbar_init(&ctl.drain, 1);
        fence_mbar_init();
        ctl.failed = ctl.qs = 0;
        for (int i = 0; i < kStages; ++i) ctl.sent[i] = 0;
    }
    if (warp == kSoftWarps && lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    // All of the above ran beside the last kernel in the stream. TMEM is taken after the wait: that kernel
    // may still be about to take its own on this SM, and would wait for this one.
    pdl_wait();
    if (warp == kSoftWarps + 1) {
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
    // 384 threads start with 168 registers each, 64512 in all: 8 softmax warps x 208 + 4 x 88 is as many
    if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kSoftWarps) {
        // ---------------------------------------------------------- TMA producer
        const int pool_rows = a.n_pages * a.nkv * kPage;
        int item = 0, n = 0, nd = 0;  // ring items, pieces, blocks to be cleaned
        bool ok = true;
        while (walk.next(a, &pc)) {
            const int page_lo = pc.lo / kPage, page_hi = pc.hi / kPage;
            const int32_t* tab = a.table + (size_t)pc.b * a.max_pages;
            // The lanes hold the table entries of four blocks (lane 8 i + p: page p of block 4 q + i), the next
            // four's are on their way; a block's eight rows go to uniform registers.
            auto entries = [&](int q) {
                const int pi = (pc.kb0 + 4 * q) * (kKeys / kPage) + lane;
                return pi >= page_lo && pi <= page_hi ? tab[pi] : 0;
            };
            int have = 0, cur = entries(0), nxt = entries(1);
            const int LA = pc.two ? 1 : 2;
            if (n > 0) ok = ok && wait(&ctl.q_empty, (n - 1) & 1, failed);
            if (elected() && ok) {
                const int subs = pc.two ? 2 : 1;
                ctl.qs = n + 1;
                mbar_arrive_expect_tx(&ctl.q_full, (uint32_t)(subs * a.tps * a.G * D * 2));
                for (int s = 0; s < subs; ++s)
                    for (int h = 0; h < D / 64; ++h)
                        tma_load_3d(smem + s * S::kBlock + h * 16384, &tmQ, h * 64, pc.g * a.G, pc.row0 + s * a.tps,
                                    &ctl.q_full);
            }
            __syncwarp();
            auto load = [&](const CUtensorMap* tm, int k, bool clean) {
                const int st = item % kStages;
                if (item >= kStages) ok = ok && wait(&ctl.empty[st], (item / kStages - 1) & 1, failed);
                uint64_t* bar = clean ? &ctl.dirty[nd % kDirty] : &ctl.full[st];
                const uint32_t phase = clean ? nd / kDirty : item / kStages;
                ++item;
                nd += clean;
                const int first = (pc.kb0 + k) * (kKeys / kPage);  // the block's pages that hold keys of the tile
                const int p0 = max(page_lo - first, 0), p1 = min(page_hi - first, kKeys / kPage - 1);
                const int pg = (k >> 2) == have ? cur : nxt;
                // a page outside the pool gets a row past its end, which the TMA unit fills with zeros
                const uint32_t row = pg >= 0 && pg < a.n_pages ? (pg * a.nkv + pc.g) * kPage : pool_rows;
                uint32_t y[kKeys / kPage];
#pragma unroll
                for (int i = 0; i < kKeys / kPage; ++i) y[i] = uniform(lane == (k & 3) * 8 + i ? row : 0u);
                uint8_t* dst = smem + S::kOffRing + st * S::kBlock;
                if (elected() && ok) {
                    ctl.sent[st] = smem_u32(bar) | (phase & 1);
                    mbar_arrive_expect_tx(bar, (uint32_t)((p1 - p0 + 1) * kPage * D * 2));
#pragma unroll
                    for (int i = 0; i < kKeys / kPage; ++i)
                        if (i >= p0 && i <= p1)
#pragma unroll
                            for (int h = 0; h < D / 64; ++h)
                                tma_load_2d(dst + h * 16384 + i * 2048, tm, h * 64, (int)y[i], bar);
                }
                __syncwarp();
            };
            load(&tmK, 0, false);
            if (LA == 2 && pc.nb > 1) load(&tmK, 1, false);
            for (int k = 0; k < pc.nb; ++k) {
                if ((k >> 2) != have) {
                    cur = nxt;
                    nxt = entries(++have + 1);
                }
                load(&tmV, k, pc.masked(a, pc.kb0 + k));
                if (k + LA < pc.nb) load(&tmK, k + LA, false);
            }
            ++n;
        }
    } else if (warp == kSoftWarps + 1) {
        // ---------------------------------------------------------- MMA issuer
        // all lanes walk along, one issues: see mma_ss
        constexpr uint32_t id_s = idesc_tc<128, 128, false>();
        constexpr uint32_t id_o = idesc_tc<128, D, true>();
        const uint32_t sb = smem_u32(smem), tm = uniform(tmem);
        int item = 0, n = 0;
        uint32_t p_par = 0;               // parity of p_full[s] in bit s
        bool ok = true;
        auto take = [&](int* st) {        // the next ring item, loaded
            *st = item % kStages;
            ok = ok && wait(&ctl.full[*st], (item / kStages) & 1, failed);
            ++item;
        };
        auto issue_s = [&](int s, int st, bool two) {
            const uint32_t q = uniform(desc_lo(sb + (two ? s : 0) * S::kBlock, 1));
            const uint32_t k = uniform(desc_lo(sb + S::kOffRing + st * S::kBlock, 1));
            tc_fence_after();
            if (elected() && ok) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t at = (kk >> 2) * (16384 >> 4) + (kk & 3) * (32 >> 4);
                    mma_ss(tm + s * kKeys, q + at, k + at, id_s, kk > 0 ? 1u : 0u);
                }
                tc_commit(&ctl.s_full[s]);
            }
            __syncwarp();
        };
        auto wait_p = [&](int s) {
            ok = ok && wait(&ctl.p_full[s], (p_par >> s) & 1, failed);
            p_par ^= 1u << s;
        };
        auto issue_o = [&](int s, int st, bool first) {
            const uint32_t v = uniform(desc_lo(sb + S::kOffRing + st * S::kBlock, 16384 >> 4));
            const uint32_t d = tm + 2 * kKeys + s * D, p = tm + s * kKeys, more = uniform(first ? 0u : 1u);
            tc_fence_after();
            if (elected() && ok) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_ts(d, p + kk * 8, v + kk * (2048 >> 4), id_o, kk > 0 ? 1u : more);
                tc_commit(&ctl.pv_done[s]);
            }
            __syncwarp();
        };
        // the next piece is worked out while this one's first scores are on their way
        Piece nx;
        bool more = walk.next(a, &nx);
        while (more) {
            pc = nx;
            ok = ok && wait(&ctl.q_full, n & 1, failed);
            int st = 0, sk = 0;
            bool freed = n == 0;  // the last piece's O has been read
            auto wait_o = [&]() {
                if (!freed) ok = ok && wait(&ctl.o_free, (n - 1) & 1, failed);
                freed = true;
            };
            if (pc.two) {
                int from[2], to[2];
                pc.range(a, 0, &from[0], &to[0]);
                pc.range(a, 1, &from[1], &to[1]);
                take(&sk);
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (from[s] == 0 && to[s] > 0) issue_s(s, sk, true);
                commit_elected(&ctl.empty[sk], ok);
                if (pc.nb == 1) commit_elected(&ctl.q_empty, ok);
                more = walk.next(a, &nx);
                for (int j = 0; j < pc.nb; ++j) {
                    take(&st);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (j >= from[s] && j < to[s]) {
                            wait_p(s);
                            wait_o();
                            issue_o(s, st, j == from[s]);
                        }
                        if (s == 1) commit_elected(&ctl.empty[st], ok);
                        if (j + 1 < pc.nb) {
                            if (s == 0) take(&sk);
                            if (j + 1 >= from[s] && j + 1 < to[s]) issue_s(s, sk, true);
                            if (s == 1) commit_elected(&ctl.empty[sk], ok);
                            if (s == 1 && j + 2 == pc.nb) commit_elected(&ctl.q_empty, ok);
                        }
                    }
                }
            } else {
                for (int k = 0; k < 2 && k < pc.nb; ++k) {
                    take(&sk);
                    issue_s(k, sk, false);
                    commit_elected(&ctl.empty[sk], ok);
                    if (k + 1 == pc.nb) commit_elected(&ctl.q_empty, ok);
                }
                more = walk.next(a, &nx);
                for (int k = 0; k < pc.nb; ++k) {
                    const int s = k & 1;
                    take(&st);
                    wait_p(s);
                    wait_o();
                    issue_o(s, st, k < 2);
                    commit_elected(&ctl.empty[st], ok);
                    if (k + 2 < pc.nb) {
                        take(&sk);
                        issue_s(s, sk, false);
                        commit_elected(&ctl.empty[sk], ok);
                        if (k + 3 == pc.nb) commit_elected(&ctl.q_empty, ok);
                    }
                }
            }
            ++n;
        }
    } else {
        // ---------------------------------------------------------- V cleaning (two warps, half the keys each)
        const int half = warp - (kSoftWarps + 2);
        int item = 0, n = 0, nd = 0;
        bool ok = true;
        if (warp == kSoftWarps + 3 && lane == 0) {
            // what the join needs to know of a tile that this run's first piece ends without starting it
            Join jn{-1, 0, 0, 0};
            Walk w2(a, run);
            if (w2.next(a, &pc) && !pc.starts && pc.ends) jn = Join{run.first, pc.row0, pc.ntok, pc.g};
            reinterpret_cast<Join*>(reinterpret_cast<char*>(a.ws) - kJoinBytes)[blockIdx.x] = jn;
        }
        __syncwarp();
        while (ok && walk.next(a, &pc)) {
            const bool notes = pc.notes();
            // the last piece's notes have been read; waited for at every piece, because a parity tells
            // only neighbouring phases apart
            if (n > 0) ok = wait(&ctl.o_free, (n - 1) & 1, failed);
            ok = named_bar_and(2, 64, ok);
            int entry = 0;
            uint32_t some = 0;
            const int LA = pc.two ? 1 : 2;
            item += min(LA, pc.nb);  // the first K blocks
            for (int k = 0; k < pc.nb && ok; ++k) {
                const int st = item % kStages;
                item += k + LA < pc.nb ? 2 : 1;
                const int kb = pc.kb0 + k;
                if (!pc.masked(a, kb)) continue;
                // every masked block is waited for, in order, and the MMA of a block waits for its cleaning
                ok = named_bar_and(2, 64, wait(&ctl.dirty[nd % kDirty], (nd / kDirty) & 1, failed));
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
                        some |= found[i];
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
            if (lane == 0 && notes) ctl.poison.some[half] = some;
            __syncwarp();
            if (lane == 0 && notes) mbar_arrive(&ctl.clean_done);
            ++n;
        }
    }
    } else {
        // ---------------------------------------------------------- softmax and epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        constexpr int NC = kKeys / 32;
        const int s = warp / kSubWarps;                   // sub-tile
        const int quad = warp & 3;                        // TMEM lanes 32 quad ..
        const int r = quad * 32 + lane;                   // row of the sub-tile = TMEM lane
        const int tl = r / a.G, hh = r - tl * a.G;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t sa = tmem + s * kKeys + lane_off;
        const float sl2 = a.scale * kLog2e;
        const float cap_k = CAP ? a.scale / a.cap : 0.f, cap_raw = CAP ? a.cap / a.scale : 0.f;
        int noted = 0;        // pieces with notes so far
        int cnt = 0, cnt_o = 0;  // blocks so far of this sub-tile, of the other (phases of s_full and pv_done)
        bool ok = true;
        Piece nx;
        bool more = walk.next(a, &nx);
        while (more) {
            pc = nx;
            const int tok = pc.two ? s * a.tps + tl : tl;  // token of the tile
            const bool valid = tl < a.tps && tok < pc.ntok;
            const int pos = pc.p0 + pc.t0 + tok;
            const int lo = a.window > 0 ? (int)max((long long)pos + 1 - a.window, 0ll) : 0;
            // blocks of this sub-tile: from, from + step, .. < to, and of the other (scalars: an array
            // indexed by the sub-tile would live in local memory)
            int from = s, to = pc.nb, from_o = s ^ 1, to_o = pc.nb;
            const int step = pc.two ? 1 : 2;
            if (pc.two) {
                pc.range(a, s, &from, &to);
                pc.range(a, s ^ 1, &from_o, &to_o);
            }
            const bool have = from < to, have_o = from_o < to_o;
            if (have_o) cnt_o += (to_o - from_o + step - 1) / step;
            const int32_t* tab = a.table + (size_t)pc.b * a.max_pages;
            auto page_ok = [&](int k) {  // whether the lane's page of block k lies in the pool
                const int pi = (pc.kb0 + k) * (kKeys / kPage) + lane % (kKeys / kPage);
                if (k >= to || pi >= a.max_pages) return false;
                const int pg = tab[pi];
                return pg >= 0 && pg < a.n_pages;
            };
            bool pg = page_ok(from);
            const bool busy = __any_sync(0xffffffffu, valid);
            float m = -INFINITY, l = 0.f;
            for (int j = from; j < to; j += step) {
                constexpr uint32_t kAll = (1u << (kKeys / kPage)) - 1;
                const uint32_t good = __ballot_sync(0xffffffffu, pg) & kAll;
                pg = page_ok(j + step);
                const int key0 = (pc.kb0 + j) * kKeys;
                // a row of nobody goes along unmasked: what it computes reaches no other row
                const bool whole = !valid || (key0 + kKeys - 1 <= pos && key0 >= lo && good == kAll);
                if (ok && !wait(&ctl.s_full[s], cnt & 1, failed)) ok = false;
                tc_fence_after();
                if (!busy) {  // no row of this warp is anybody's: its P may stay what it is
                    if (lane == 0) mbar_arrive(&ctl.p_full[s]);
                    ++cnt;
                    continue;
                }
                uint32_t v[NC][32];
#pragma unroll
                for (int c = 0; c < NC; ++c) tmem_ld32(sa + 32 * c, v[c]);
                tmem_ld_wait32(v[0]);
#pragma unroll
                for (int c = 1; c < NC; ++c) reg_fence32(v[c]);
                if (CAP) {
                    // in units of the raw score: raw tanh(y) / y, y = raw scale / cap, by a polynomial in y^2 where no
                    // |y| is above 3/4 (in practice nowhere), packed two by two; else one by one from scores read again
                    const float2 k2 = make_float2(cap_k * cap_k, cap_k * cap_k);
                    float tm4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int q = 0; q < 32; q += 2) {
                            const float2 x = make_float2(__uint_as_float(v[c][q]), __uint_as_float(v[c][q + 1]));
                            const float2 t = fmul2(fmul2(x, k2), x);
                            tm4[(q >> 1) & 3] = max3_nan(tm4[(q >> 1) & 3], t.x, t.y);
                            float2 u = ffma2(t, make_float2(kT4, kT4), make_float2(kT3, kT3));
                            u = ffma2(u, t, make_float2(kT2, kT2));
                            u = ffma2(u, t, make_float2(kT1, kT1));
                            u = fmul2(ffma2(u, t, make_float2(kT0, kT0)), x);
                            v[c][q] = __float_as_uint(u.x);
                            v[c][q + 1] = __float_as_uint(u.y);
                        }
                    const float tmx = max_nan(max_nan(tm4[0], tm4[1]), max_nan(tm4[2], tm4[3]));
                    if (__any_sync(0xffffffffu, !(tmx <= 0.5625f))) {
#pragma unroll 1
                        for (int c0 = 0; c0 < kKeys; c0 += 32) {
                            uint32_t x[32];
                            tmem_ld32(sa + c0, x);
                            tmem_ld_wait32(x);
#pragma unroll
                            for (int q = 0; q < 32; ++q) x[q] = __float_as_uint(cap_raw * tanh_exact(__uint_as_float(x[q]) * cap_k));
                            tmem_st16(sa + c0, x);
                            tmem_st16(sa + c0 + 16, x + 16);
                        }
                        tmem_st_wait();
#pragma unroll
                        for (int c = 0; c < NC; ++c) tmem_ld32(sa + 32 * c, v[c]);
                        tmem_ld_wait32(v[0]);
#pragma unroll
                        for (int c = 1; c < NC; ++c) reg_fence32(v[c]);
                    }
                }
                const bool masked = __any_sync(0xffffffffu, !whole);
                if (masked) {
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        // bit q: the row sees key 32 c + q of these (its keys are lo .. pos; pages may be missing)
                        const int b0 = lo - key0 - 32 * c, b1 = pos - key0 - 32 * c;
                        uint32_t see = b1 < 0 ? 0u : 0xffffffffu >> (31 - min(b1, 31));
                        see &= b0 > 31 ? 0u : 0xffffffffu << max(b0, 0);
                        see &= ((good >> (2 * c)) & 1 ? 0x0000ffffu : 0u) | ((good >> (2 * c)) & 2 ? 0xffff0000u : 0u);
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            if (!((see >> q) & 1)) v[c][q] = __float_as_uint(-INFINITY);
                    }
                }
                float bm4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int q = 0; q < 32; q += 2)
                        bm4[(q >> 1) & 3] =
                            max3_nan(bm4[(q >> 1) & 3], __uint_as_float(v[c][q]), __uint_as_float(v[c][q + 1]));
                float mn = max_nan(max_nan(bm4[0], bm4[1]), max_nan(bm4[2], bm4[3])) * sl2;
                // almost always no row has grown past its m by 2^8, and m stays
                const bool over = valid && !(mn <= m + kRescale);
                if (__any_sync(0xffffffffu, over)) {
                    mn = max_nan(m, mn);
                    if (!(mn < INFINITY)) mn = NAN;  // a score that is NaN or +inf makes the row NaN, from here on
                    const bool grown = valid && m != -INFINITY && mn > m + kRescale;
                    const float corr = grown ? ex2f(m - mn) : 1.f;
                    if (grown || m == -INFINITY || mn != mn) m = mn;
                    l *= corr;
                    if (__any_sync(0xffffffffu, grown) && j > from) {
                        // O of the rows that grew, once the last block's product is in
                        if (ok && !wait(&ctl.pv_done[s], (cnt - 1) & 1, failed)) ok = false;
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 16) {
                            uint32_t o[16];
                            tmem_ld16_issue(tO + s * D + lane_off + c0, o);
                            tmem_ld_wait16(o);
#pragma unroll
                            for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * corr);
                            tmem_st16(tO + s * D + lane_off + c0, o);
                        }
                    }
                }
                // P = 2^(S' - m), rounded to bf16, over the scores (keys 2i, 2i + 1 in column i).
                const float2 mul2 = make_float2(sl2, sl2);
                const float nm = m == -INFINITY ? 0.f : -m;  // nothing seen yet: every score is -inf, 2^-inf = 0
                const float2 nm2 = make_float2(nm, nm);
                float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
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
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_full[s]);
                ++cnt;
            }

            more = walk.next(a, &nx);  // while the last products are on their way

            // ---- epilogue: m and l of a `one` tile, over both sub-tiles
            float w0 = 1.f, w1 = 0.f;  // weights of this sub-tile's O, of the other's
            if (!pc.two) {
                ctl.ml[s][r] = make_float2(m, l);
                named_bar_sync(1, 32 * kSoftWarps);
                const float mo = ctl.ml[s ^ 1][r].x, lo2 = ctl.ml[s ^ 1][r].y, ms = m;
                named_bar_sync(1, 32 * kSoftWarps);
                m = fmaxf(ms, mo);
                w0 = ms == -INFINITY ? 0.f : ex2f(ms - m);
                w1 = mo == -INFINITY ? 0.f : ex2f(mo - m);
                // rounded alike in both sub-tiles' threads
                l = __fadd_rn(__fmul_rn(l, w0), __fmul_rn(lo2, w1));
            }
            if (have && ok && !wait(&ctl.pv_done[s], (cnt - 1) & 1, failed)) ok = false;
            if (!pc.two && have_o && ok && !wait(&ctl.pv_done[s ^ 1], (cnt_o - 1) & 1, failed)) ok = false;
            // an O that no block went into holds anything
            const bool use = have && w0 != 0.f, use_o = !pc.two && have_o && w1 != 0.f;
            int poisoned = 0;
            if (pc.notes()) {
                if (ok && !wait(&ctl.clean_done, noted & 1, failed)) ok = false;
                ++noted;
                if (ok && (ctl.poison.some[0] | ctl.poison.some[1])) poisoned = ctl.poison.n;
            }
            tc_fence_after();
            // columns of this thread: its sub-tile's, or half of the joined result's
            const int c_lo = pc.two ? 0 : s * (D / 2), c_hi = pc.two ? D : c_lo + D / 2;
            const bool whole_tile = pc.starts && pc.ends;
            const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
            float* slot = a.ws + (size_t)(2 * blockIdx.x + (pc.starts ? 1 : 0)) * S::kSlotFloats +
                          (pc.two ? s * S::kSubFloats : 0);
            uint16_t* dst = a.out + ((size_t)(pc.row0 + tok) * a.nq + (size_t)pc.g * a.G + hh) * D;
#pragma unroll 1
            for (int c0 = busy ? c_lo : c_hi; c0 < c_hi; c0 += 16) {
                uint32_t o[16], o1[16];
                tmem_ld16_issue(tO + s * D + lane_off + c0, o);
                if (!pc.two) tmem_ld16_issue(tO + (s ^ 1) * D + lane_off + c0, o1);
                tmem_ld_wait16(o);
                reg_fence16(o1);
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    float x = use ? __uint_as_float(o[q]) * w0 : 0.f;
                    if (use_o) x = fmaf(__uint_as_float(o1[q]), w1, x);
                    o[q] = __float_as_uint(x);
                }
                if (poisoned && valid) {
#pragma unroll 1
                    for (int e = 0; e < poisoned; ++e)
#pragma unroll 1
                        for (int i = 0; i < 4; ++i)
                            for (uint32_t bits = ctl.poison.keys[e][i]; bits; bits &= bits - 1) {
                                const int key = ctl.poison.kb[e] * kKeys + 32 * i + __ffs(bits) - 1;
                                if (key > pos || key < lo) continue;
                                const int page = tab[key / kPage];
                                if (page < 0 || page >= a.n_pages) continue;
                                const uint16_t* vr =
                                    a.v_pool + (((size_t)page * a.nkv + pc.g) * kPage + key % kPage) * D + c0;
#pragma unroll
                                for (int q = 0; q < 16; ++q) {
                                    const float x = bf2f(vr[q]);
                                    if (!(fabsf(x) < INFINITY)) o[q] = __float_as_uint(__uint_as_float(o[q]) + x);
                                }
                            }
                }
                if (valid && ok) {
                    if (whole_tile) {
                        // a whole 32-byte sector of the thread's row
#pragma unroll
                        for (int q = 0; q < 16; q += 8) {
                            uint4 y;
                            y.x = pack_bf2(__uint_as_float(o[q]) * inv, __uint_as_float(o[q + 1]) * inv);
                            y.y = pack_bf2(__uint_as_float(o[q + 2]) * inv, __uint_as_float(o[q + 3]) * inv);
                            y.z = pack_bf2(__uint_as_float(o[q + 4]) * inv, __uint_as_float(o[q + 5]) * inv);
                            y.w = pack_bf2(__uint_as_float(o[q + 6]) * inv, __uint_as_float(o[q + 7]) * inv);
                            *reinterpret_cast<uint4*>(dst + c0 + q) = y;
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 16; q += 4)
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
    tc_fence_before();
    __syncthreads();
    if (warp == kSoftWarps + 1) {
        tc_fence_after();
        if (ctl.failed) drain(ctl, kStages);
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Joins the pieces of the tile whose last piece is CTA blockIdx.x's first: with M the largest m,
// O = sum 2^(m_i - M) O_i, l = sum 2^(m_i - M) l_i, in the order of the runs. Up to eight blocks share
// a tile: by groups of 32 rows, then, where it has at most four, by columns (a decode's tile has one group
// and many pieces, a prompt's eight and two). The pieces' m and l are read all at once, into
// weights in shared memory. Latency is the bound: three dependent reads of what other SMs have just
// written.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinBlocks = 8, kJoinSharing = 4;

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 4) chunk_join_kernel(const ChunkArgs a) {
    using S = Shape<D>;
    // of each piece and row: m, then the weight 2^(m - M); and l (two arrays of 18.5 KB)
    __shared__ float wt[kCtas][32], wl[kCtas][32];
    __shared__ float red[2][kJoinWarps][32];
    const int last = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const Join jn = reinterpret_cast<const Join*>(reinterpret_cast<const char*>(a.ws) - kJoinBytes)[last];
    if (jn.first < 0) return;
    const int np = last - jn.first + 1;
    const int groups0 = (min(jn.ntok, a.tps) * a.G + 31) / 32, groups1 = (max(jn.ntok - a.tps, 0) * a.G + 31) / 32;
    // blocks of a group of rows (8 of them: 148 cut tiles with one group each would need two waves of blocks, 116.1
    // us instead of 115.0 for 32 sequences of 5-8 rows; 2: 18.5 instead of 17.3 us for 5 rows at 4096)
    int sharing = kJoinSharing;
    while (sharing > 1 && sharing * (groups0 + groups1) > kJoinBlocks) sharing >>= 1;
    const int group = blockIdx.y / sharing, share = blockIdx.y % sharing;
    if (group >= groups0 + groups1) return;
    const int sub = group >= groups0, row = 32 * (group - (sub ? groups0 : 0)) + lane;
    const int tl = row / a.G, hh = row - tl * a.G, tok = sub * a.tps + tl;
    const bool valid = tl < a.tps && tok < jn.ntok;
    auto piece = [&](int i) {  // the tail of the first run, the head of the others
        return a.ws + (size_t)(2 * (jn.first + i) + (i == 0 ? 1 : 0)) * S::kSlotFloats + sub * S::kSubFloats;
    };
    float M = -INFINITY;
    for (int i = warp; i < np; i += kJoinWarps) {
        const float* p = piece(i) + kRows * D + row;
        const float m = valid ? p[0] : -INFINITY;
        wl[i][lane] = valid ? p[kRows] : 0.f;
        wt[i][lane] = m;
        M = fmaxf(M, m);
    }
    red[0][warp][lane] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, red[0][w][lane]);
    // a piece that saw nothing adds its l, 0 (NaN when every score was), and no O
    float L = 0.f;
    for (int i = warp; i < np; i += kJoinWarps) {
        const float m = wt[i][lane], w = m == -INFINITY ? 0.f : ex2f(m - M);
        wt[i][lane] = w;
        L += m == -INFINITY ? wl[i][lane] : w * wl[i][lane];
    }
    red[1][warp][lane] = L;
    __syncthreads();
    L = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) L += red[1][w][lane];
    if (!valid) return;
    const float inv = L > 0.f || L != L ? 1.0f / L : 0.f;
    uint16_t* dst = a.out + ((size_t)(jn.row0 + tok) * a.nq + (size_t)jn.g * a.G + hh) * D;
    const int cols = D / 4 / sharing;  // float4 columns of this block
    // KC columns (warp, warp + 8, ..) of KP pieces at once, none of the loads behind a test of its weight: one
    // after the other they took 34 us for 18 pieces. A piece of weight 0 holds finite values (or its
    // row is not finite anyway); past the last piece the last one is read again, and not used.
    auto columns = [&](auto kc, auto kp, int c0) {
        constexpr int KC = decltype(kc)::value, KP = decltype(kp)::value;
        const size_t at = ((size_t)c0 * kRows + row) * 4;
        float4 o[KC];
#pragma unroll
        for (int k = 0; k < KC; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < np; i0 += KP) {
            float4 x[KP][KC];
#pragma unroll
            for (int u = 0; u < KP; ++u) {
                const float* p = piece(min(i0 + u, np - 1)) + at;
#pragma unroll
                for (int k = 0; k < KC; ++k)
                    x[u][k] = __ldcg(reinterpret_cast<const float4*>(p + (size_t)k * kJoinWarps * kRows * 4));
            }
#pragma unroll
            for (int u = 0; u < KP; ++u)
                if (i0 + u < np) {
                    const float w = wt[i0 + u][lane];
#pragma unroll
                    for (int k = 0; k < KC; ++k) {
                        o[k].x = fmaf(w, x[u][k].x, o[k].x);
                        o[k].y = fmaf(w, x[u][k].y, o[k].y);
                        o[k].z = fmaf(w, x[u][k].z, o[k].z);
                        o[k].w = fmaf(w, x[u][k].w, o[k].w);
                    }
                }
        }
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            uint2 y;
            y.x = pack_bf2(o[k].x * inv, o[k].y * inv);
            y.y = pack_bf2(o[k].z * inv, o[k].w * inv);
            *reinterpret_cast<uint2*>(dst + 4 * (c0 + kJoinWarps * k)) = y;
        }
    };
    const int c0 = share * cols + warp;
    if (cols == 4 * kJoinWarps)
        columns(Int<4>(), Int<2>(), c0);
    else if (cols == 2 * kJoinWarps)
        columns(Int<2>(), Int<4>(), c0);
    else if (warp < cols)
        columns(Int<1>(), Int<8>(), c0);
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
    const auto kernel = a.cap > 0.f ? chunk_attn_kernel<D, true> : chunk_attn_kernel<D, false>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, tmQ, tmK, tmV, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(kCtas, kJoinBlocks);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
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
            if (units_before(a, s, t) != n) ++wrong;
            if (tile_blocks(a, s, t) < 1) ++wrong;
            n += kTileCost + tile_blocks(a, s, t);
        }
        if (seq_units(a, s) != n) ++wrong;
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
    const Cut cut(total);
    for (int c = 0; c < kCtas && cut.len(c) > 0; ++c) {
        const Run run = run_from(a, 0, 0, cut, c);
        Walk w(a, run);
        Piece p;
        int pieces = 0;
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
            ++pieces;
            if (off == blocks) left = next_tile();
        }
    }
    return left ? wrong + 1 : wrong;
}

namespace {
std::atomic<int> g_test_stall{0};
}  // namespace

bool chunk_set_test_wait(int kind) {
    if (kind < 0 || kind >= kStalls) return false;
    g_test_stall = kind;
    return true;
}

namespace {
// Devices on which gqa_chunk_attn has been called (index 63: that one and all above).
std::atomic<bool> g_used[64];

std::atomic<bool>& used_here() {
    int dev = 0;
    cudaGetDevice(&dev);
    return g_used[dev < 63 ? dev : 63];
}
}  // namespace

cudaError_t chunk_take_error(int* set, cudaStream_t st) {
    *set = 0;
    if (!used_here()) return cudaSuccess;
    cudaError_t e = cudaMemcpyFromSymbolAsync(set, g_chunk_err, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess || !*set) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_chunk_err, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st);
    return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
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
    if (scale < 0x1p-40f || scale > 0x1p40f || (softcap > 0.f && softcap < 0x1p-20f))
        return bad(DEC_ERR_UNSUPPORTED, "scale must lie within 2^-40 .. 2^40, a softcap not below 2^-20");
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
    a.stall = g_test_stall;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    used_here() = true;
    cudaError_t e = d == 128 ? launch<128>(a, q, ldq, k_pool, st) : launch<64>(a, q, ldq, k_pool, st);
    if (e != cudaSuccess) return bad(DEC_ERR_CUDA, std::string("gqa_chunk_attn: ") + cudaGetErrorString(e));
    return DEC_OK;
} catch (const std::exception&) {
    return DEC_ERR_OOM;
}

}  // extern "C"
