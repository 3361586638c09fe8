// The attention weight that every cached key gets from more than 16 query rows per key head (prompts,
// chunks, the last tokens of a prompt): bf16, d = 64 or 128, pages of at least 8 keys, clip_k <= 127.
//
// S^T = K Q^T on tcgen05 with the keys as the 128 rows of the accumulator: a thread has one key and adds
// up its weights over the columns, the query rows, so nothing crosses threads and nothing but the sums
// leaves the SM. A unit is two tiles of keys of one head, which stay in shared memory while the
// request's query tiles pass by; each of them meets both. Units are taken by ticket, the heads of a
// request together and its first keys first: every row of a prompt sees those, so the long units come first.
// A row's constant nl (the table term of far keys less the log-sum-exp) is formed in front and
// lies in shared memory beside its query tile, so a weight is one FMA and one exponential. Where some key of
// a unit is less than clip_k back, R = Q aK^T is one product more of the query tile, its accumulator
// drained into shared memory by one group's threads (a row each).
//
// Roles (512 threads, one CTA per SM): warp 3 takes tickets and announces units, warp 0 loads keys, tables and
// query tiles, warp 2 the rows' constants, warp 1 issues the MMAs; three groups of four warps, 4-7, 8-11 and 12-15, add up
// the products in turn, each out of its own accumulator, 32 columns while the next come. What the groups have of a key meets
// in shared memory, in the order of the unit's turns, so equal calls give equal bits. (Two groups, a tile of the pair each, with
// all of a row's scores in registers: a query tile with a pair 1.10 us in place of 0.90, since two warps to a scheduler do not
// hide each other's waits and loads; a single query tile 7 % faster, whose keys are the bound. Sixteen warps with half of the
// columns each 1.30. A second R beside the first: 247 us in place of 242 on the prompts below, for a stage of queries less.)
// TMEM: three accumulators of 128 columns, and the unit's keys, copied there where more than one query
// tile passes by: a 128 x 128 product with both operands in shared memory reads as much as that can give.
//
// What bounds it. Many rows: the sums, 1800 cycles for a query tile with both key tiles where the tensor cores work 1024
// and the exponentials (32 a cycle) take as long. A chunk of 4096 tokens over 64K keys, 8 heads of 128: 380 us, 1400
// TFLOP/s, 0.73 of the tensor rate. Four prompts of 4096 tokens, 16 heads of 128: 152 us, with the key term 220: the rows'
// constants 17, R and its gathers 50. One query tile to a request (32 tokens, 16 / 4 heads of 128, 4K - 32K keys): 43
// us, of which 25 stream the keys at 4.9 TB/s; the rest are the set-up's launch, the first ticket and loads, and the last units.
#include <cstdint>
#include <cstring>

#include "relattn_paged_tma.cuh"
#include "relattn_paged_weights.cuh"

namespace relattn {
namespace paged {
namespace {

using tc::BM;
using tc::dup;
using tc::pair;
using tc::put;
using tc::Shared;
using tc::wait_bar;
using tc::wait_bar_ctrl;

constexpr int kAccs = 3;             // accumulators, a group of four summing warps to each
constexpr int kSumWarps = 4 * kAccs;
constexpr int kThreads = 128 + 32 * kSumWarps;
constexpr int KB = 32;               // columns read from an accumulator at a time
constexpr int kUnits = 4;            // announced ahead
constexpr int kMaxK = 4, kMaxQ = 4;  // stages
constexpr int kParts = 1;            // pairs of tiles whose sums are joined at once
constexpr uint32_t kPartBytes = kAccs * 2 * kTile * 4;
constexpr int kSides = 8;            // tiles whose page numbers are held
constexpr int kBatch = 4;            // query tiles whose constants come together ...
constexpr int kBatches = 2;          // ... and how often
constexpr uint32_t kSideBytes = 64;  // of a tile, 16 at most

enum : int {
    B_K_FULL = 0, B_K_EMPTY = B_K_FULL + kMaxK, B_Q_FULL = B_K_EMPTY + kMaxK, B_Q_EMPTY = B_Q_FULL + kMaxQ,
    B_AK_FULL = B_Q_EMPTY + kMaxQ, B_AK_EMPTY, B_UNIT_FULL, B_UNIT_EMPTY = B_UNIT_FULL + kUnits,
    B_ACC_FULL = B_UNIT_EMPTY + kUnits, B_ACC_EMPTY = B_ACC_FULL + kAccs, B_SIDE_FULL = B_ACC_EMPTY + kAccs,
    B_SIDE_EMPTY = B_SIDE_FULL + kSides, B_NL_FULL = B_SIDE_EMPTY + kSides, B_NL_EMPTY = B_NL_FULL + kBatches,
    B_R_FULL = B_NL_EMPTY + kBatches, B_R_EMPTY, B_PART_FULL, B_PART_EMPTY = B_PART_FULL + kParts,
    B_KEYS_FREE = B_PART_EMPTY + kParts, B_DRAIN, kNumBars
};

struct Unit {
    int row0, n, pos0;   // first query token of the request, its new tokens, position of the first
    int row, kvh;        // of the block table; key head
    int t0, t1;          // tiles, in pairs
    int ns, lo;          // Item: where they lie
    int qa, qb;          // query tiles (one, where there are several pairs)
    int band;            // some row may be less than clip_k past some key
    int more, pad[3];
    __device__ __forceinline__ int key(int t) const { return t < t1 ? (t < ns ? t : lo + t - ns) * kTile : -1; }
};
static_assert(sizeof(Unit) == 64, "unit");

struct TcParams {
    WeightParams w;
    int TS;              // tokens of a query tile
    int npad, SR;        // table rows rounded up to 16; row stride (floats) of R in shared memory
    int box;             // keys per TMA box
    int nk, nq;          // stages of keys and of query tiles
    uint32_t tile_bytes, off_q, off_ak, off_r, off_nl, off_side, off_part, off_unit, off_bar;
};

// what a query tile is to a unit, the same for every role
struct QueryTile {
    int tok0, ntok, pos_lo, pos_hi;
    bool band;           // with the tiles at j0 and j1
};
__device__ __forceinline__ QueryTile query_tile(const TcParams &tp, const Unit &u, int q, int j0, int j1) {
    QueryTile t;
    t.tok0 = q * tp.TS;
    t.ntok = min(tp.TS, u.n - t.tok0);
    t.pos_lo = u.pos0 + t.tok0;
    t.pos_hi = t.pos_lo + t.ntok - 1;
    auto near = [&](int j) { return j >= 0 && j + kTile - 1 > t.pos_lo - tp.w.p.clip_k && j <= t.pos_hi; };
    t.band = u.band && (near(j0) || near(j1));
    return t;
}

struct Units {
    uint32_t bars;
    const Unit *ring;
    uint32_t it;
    __device__ __forceinline__ Units(const TcParams &tp, const Shared &sh)
        : bars(sh.base + tp.off_bar), ring(reinterpret_cast<const Unit *>(sh.ptr + tp.off_unit)), it(0) {}
    __device__ __forceinline__ uint32_t full() const { return bars + 8u * (B_UNIT_FULL + (it & (kUnits - 1))); }
    __device__ __forceinline__ uint32_t empty() const { return bars + 8u * (B_UNIT_EMPTY + (it & (kUnits - 1))); }
    __device__ __forceinline__ uint32_t parity() const { return (it / kUnits) & 1u; }
    // (through a broadcast: the compiler then knows the fields to be warp-uniform)
    __device__ __forceinline__ Unit get() const {
        const Unit &s = ring[it & (kUnits - 1)];
        auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
        return Unit{uni(s.row0), uni(s.n),  uni(s.pos0), uni(s.row), uni(s.kvh),  uni(s.t0),  uni(s.t1),
                    uni(s.ns),   uni(s.lo), uni(s.qa),   uni(s.qb),  uni(s.band), uni(s.more), {}};
    }
};

struct Ring {
    int st, n;
    uint32_t ph;
    __device__ __forceinline__ explicit Ring(int stages) : st(0), n(stages), ph(0) {}
    __device__ __forceinline__ void next() {
        if (++st == n) {
            st = 0;
            ph ^= 1u;
        }
    }
};

// ======================================================================= tickets
template <bool AK>
__device__ void ticket_role(const TcParams &tp, const Shared &sh) {
    const Params &p = tp.w.p;
    const int lane = threadIdx.x & 31;
    Units units(tp, sh);
    Unit *ring = reinterpret_cast<Unit *>(sh.ptr + tp.off_unit);
    const int count = *tp.w.count;
    const long long total = tp.w.start[count];
    for (bool begin = true;; begin = false) {
        unsigned long long t = blockIdx.x;   // the first ticket is the CTA's own
        if (!begin && lane == 0) t = gridDim.x + atomicAdd(tp.w.ticket, 1ull);
        t = __shfl_sync(0xffffffffu, t, 0);
        Unit u{};
        if ((long long)t < total) {
            long long rest;
            u.row = tp.w.busy[find_unit(tp.w, count, (long long)t, rest)];
            const Seq s = load_seq(p, u.row);
            const Item it = make_item(p, s, 0);
            const int step = 2 * tp.w.pairs(s.n), i = (int)(rest / p.Hkv);
            u.kvh = (int)(rest - (long long)i * p.Hkv);
            u.row0 = s.q0;
            u.n = s.n;
            u.pos0 = s.pos0;
            u.t0 = i * step;
            u.t1 = min(u.t0 + step, it.nt);
            u.ns = it.ns;
            u.lo = it.lo;
            int lo = s.n, hi = 0;
            for (int q = u.t0; q < u.t1; ++q) {
                lo = min(lo, first_token(u.key(q), s.pos0));
                hi = max(hi, end_token(p, u.key(q), kTile, s.pos0, s.n));
            }
            u.qa = lo / tp.TS;
            u.qb = (hi + tp.TS - 1) / tp.TS;
            u.band = AK && p.clip_k > 0 && u.key(u.t1 - 1) + kTile - 1 > s.pos0 + u.qa * tp.TS - p.clip_k;
            u.more = 1;
        }
        bool ok = wait_bar_ctrl(units.empty(), units.parity() ^ 1u, sh, p.err);
        ok = __all_sync(0xffffffffu, ok ? 1 : 0) != 0;
        if (!ok) return;
        if (lane == 0) ring[units.it & (kUnits - 1)] = u;
        __syncwarp();
        ptx::mbar_arrive_w(units.full());
        ++units.it;
        if (!u.more) return;
    }
}

// ======================================================================= loads
template <int D, bool AK>
__device__ void load_role(const TcParams &tp, const Shared &sh, const CUtensorMap *tm_q, const CUtensorMap *tm_k,
                          const CUtensorMap *tm_ak) {
    const Params &p = tp.w.p;
    constexpr int DB = D / 64;
    const int lane = threadIdx.x & 31;
    const uint32_t bars = sh.base + tp.off_bar;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        const bool r = wait_bar_ctrl(b, parity, sh, p.err);
        return __all_sync(0xffffffffu, r ? 1 : 0) != 0;
    };
    const int nbox = kTile / tp.box, my_box = lane % nbox, my_blk = lane / nbox;
    Units units(tp, sh);
    Ring kr(tp.nk), qr(tp.nq), sr(kSides);
    uint32_t ak_it = 0, k_count = 0, q_count = 0;
    bool ok = true;
    for (; ok; ++units.it) {
        if (!(ok = wait(units.full(), units.parity()))) break;
        const Unit u = units.get();
        if (!u.more) break;
        const int *bt = p.bt + (long long)u.row * p.bt_stride;
        const int pos_hi = u.pos0 + u.n - 1;
        const int first = p.window > 0 ? max(0, max(u.pos0, 0) - p.window + 1) : 0;
        // the tile's pages, one a lane, looked up a tile ahead; their numbers come along
        auto lookup = [&](int t, bool &seen) -> int {
            const int j = u.key(t) + my_box * tp.box;
            seen = t < u.t1 && j <= pos_hi && (j + tp.box > first || j < p.sinks);
            return seen ? __ldg(bt + (j >> p.pshift)) : -1;
        };
        bool seen_next;
        int pg_next = lookup(u.t0, seen_next);
        auto load_keys = [&](int t) -> bool {
            const bool seen = seen_next;
            int pg = pg_next;
            pg_next = lookup(t + 1, seen_next);
            if (!wait(bar(B_SIDE_EMPTY + sr.st), sr.ph ^ 1u) || !wait(bar(B_K_EMPTY + kr.st), kr.ph ^ 1u)) return false;
            const int j = u.key(t) + my_box * tp.box, row = j & ((1 << p.pshift) - 1);
            const bool bad = seen && (unsigned)pg >= (unsigned)p.num_pages;
            if (bad) report_page(p);
            if (my_blk == 0) reinterpret_cast<int *>(sh.ptr + tp.off_side + sr.st * kSideBytes)[my_box] = bad ? -1 : pg;
            __syncwarp();
            const unsigned m = __ballot_sync(0xffffffffu, seen && my_blk == 0);
            ptx::mbar_arrive_w(bar(B_SIDE_FULL + sr.st));
            ptx::mbar_expect_tx_w(bar(B_K_FULL + kr.st), (uint32_t)(__popc(m) * tp.box * D * 2));
            __syncwarp();
            if (seen && my_blk < DB)   // a page outside the cache: a box outside the tensor, which reads as zeros
                tma_load_4d(sh.base + (uint32_t)kr.st * tp.tile_bytes + my_blk * kTile * 128 + my_box * tp.box * 128, tm_k,
                            bar(B_K_FULL + kr.st), my_blk * 64, row, u.kvh, bad ? p.num_pages : pg);
            __syncwarp();
            kr.next();
            sr.next();
            ++k_count;
            return true;
        };
        for (int t = u.t0; t < u.t1 && t < u.t0 + 2 && ok; ++t) ok = load_keys(t);
        if (!ok) break;
        if (AK && u.band) {
            if (!(ok = wait(bar(B_AK_EMPTY), (ak_it & 1u) ^ 1u))) break;
            ptx::mbar_expect_tx_w(bar(B_AK_FULL), (uint32_t)tp.npad * D * 2);
#pragma unroll
            for (int blk = 0; blk < DB; ++blk)
                ptx::tma_load_3d_w(sh.base + tp.off_ak + blk * tp.npad * 128, tm_ak, bar(B_AK_FULL), blk * 64, 0,
                                   p.ths ? u.kvh : 0);
            ++ak_it;
        }
        for (int q = u.qa; q < u.qb; ++q) {
            if (!(ok = wait(bar(B_Q_EMPTY + qr.st), qr.ph ^ 1u))) break;
            ptx::mbar_expect_tx_w(bar(B_Q_FULL + qr.st), (uint32_t)tp.TS * p.g * D * 2);
#pragma unroll
            for (int blk = 0; blk < DB && !(p.withhold && q_count == 0); ++blk)
                ptx::tma_load_3d_w(sh.base + tp.off_q + (uint32_t)qr.st * tp.tile_bytes + blk * BM * 128, tm_q,
                                   bar(B_Q_FULL + qr.st), blk * 64, u.kvh * p.g, u.row0 + q * tp.TS);
            qr.next();
            ++q_count;
        }
        for (int t = u.t0 + 2; t < u.t1 && ok; ++t) ok = load_keys(t);
        if (ok) ptx::mbar_arrive_w(units.empty());
    }
    // no copy is in flight when the CTA exits
    for (uint32_t i = k_count > (uint32_t)tp.nk ? k_count - tp.nk : 0; i < k_count; ++i)
        tc::drain_bar(bar(B_K_FULL + (int)(i % tp.nk)), (i / tp.nk) & 1u, sh.limit);
    // (nothing is in flight on these; without the waits the compiler lays the kernel out so that four prompts of 4096
    // take 225.5 us in place of 220.4)
    for (uint32_t i = k_count > (uint32_t)kSides ? k_count - kSides : 0; i < k_count; ++i)
        tc::drain_bar(bar(B_SIDE_FULL + (int)(i % kSides)), (i / kSides) & 1u, sh.limit);
    for (uint32_t i = q_count > (uint32_t)tp.nq ? q_count - tp.nq : 0; i < q_count; ++i)
        tc::drain_bar(bar(B_Q_FULL + (int)(i % tp.nq)), (i / tp.nq) & 1u, sh.limit);
    if (AK && ak_it) tc::drain_bar(bar(B_AK_FULL), (ak_it - 1) & 1u, sh.limit);
}

// The rows' constants beside their query tile, four columns a lane; -infinity where there is no row.
__device__ void const_role(const TcParams &tp, const Shared &sh) {
    const Params &p = tp.w.p;
    const int lane = threadIdx.x & 31;
    const uint32_t bars = sh.base + tp.off_bar;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        const bool r = wait_bar_ctrl(b, parity, sh, p.err);
        return __all_sync(0xffffffffu, r ? 1 : 0) != 0;
    };
    int tok[4], head[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = 4 * lane + e;
        tok[e] = i < tp.TS * p.g ? i / p.g : 1 << 29;
        head[e] = i - i / p.g * p.g;
    }
    Units units(tp, sh);
    Ring nr(kBatches);
    for (bool ok = true; ok; ++units.it) {
        if (!(ok = wait(units.full(), units.parity()))) break;
        const Unit u = units.get();
        if (!u.more) break;
        for (int q0 = u.qa; q0 < u.qb; q0 += kBatch) {
            float v[kBatch][4];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[i][e] = q0 + i < u.qb && tok[e] < u.n - (q0 + i) * tp.TS
                                  ? __ldg(tp.w.nl + (long long)(u.row0 + (q0 + i) * tp.TS + tok[e]) * p.H + u.kvh * p.g + head[e])
                                  : -INFINITY;
            if (!(ok = wait(bar(B_NL_EMPTY + nr.st), nr.ph ^ 1u))) break;
            float4 *dst = reinterpret_cast<float4 *>(sh.ptr + tp.off_nl + nr.st * kBatch * BM * 4);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) dst[i * 32 + lane] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
            __syncwarp();
            ptx::mbar_arrive_w(bar(B_NL_FULL + nr.st));
            nr.next();
        }
        if (ok) ptx::mbar_arrive_w(units.empty());
    }
}

// ======================================================================= MMAs
constexpr uint32_t kAccCol = 128;    // first accumulator; the keys of tile s lie at D / 2 * s

// D = A B over D / 16 k-steps, one elect for the chain: A in TMEM, 8 columns a step, B K-major with 128-byte
// swizzle and 128 rows
#define RELATTN_STEP(A, B) \
    "add.u32 a1, %1, " #A ";\n\tadd.s64 b1, %2, " #B ";\n\t" \
    "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
template <int D>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
    if (D == 64)
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 t, %5, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
            RELATTN_STEP(8, 2) RELATTN_STEP(16, 4) RELATTN_STEP(24, 6) "}\n" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(0u), "r"(1u)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 t, %5, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
            RELATTN_STEP(8, 2) RELATTN_STEP(16, 4) RELATTN_STEP(24, 6) RELATTN_STEP(32, 1024) RELATTN_STEP(40, 1026)
            RELATTN_STEP(48, 1028) RELATTN_STEP(56, 1030) "}\n" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(0u), "r"(1u)
            : "memory");
}
#undef RELATTN_STEP
// 128 rows x 16 elements of a K-major tile with 128-byte swizzle to 8 columns, a row per lane: an A operand
__device__ __forceinline__ void copy_keys(uint32_t cols, uint64_t desc) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.cp.cta_group::1.128x256b [%0], %1;\n\t}\n" ::"r"(cols), "l"(desc)
        : "memory");
}

template <int D, bool AK>
__device__ void mma_role(const TcParams &tp, const Shared &sh, uint32_t tmem) {
    const Params &p = tp.w.p;
    const uint32_t bars = sh.base + tp.off_bar;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        const bool r = wait_bar_ctrl(b, parity, sh, p.err);
        return __all_sync(0xffffffffu, r ? 1 : 0) != 0;
    };
    const uint64_t dk0 = ptx::sdesc_sw128(sh.base, 16, 1024);
    const uint64_t dq0 = ptx::sdesc_sw128(sh.base + tp.off_q, 16, 1024);
    const uint64_t da = ptx::sdesc_sw128(sh.base + tp.off_ak, 16, 1024);
    const uint64_t tile16 = tp.tile_bytes >> 4;
    constexpr uint32_t idS = ptx::idesc_bf16(BM, kTile, 0);
    const uint32_t idR = ptx::idesc_bf16(BM, (uint32_t)tp.npad, 0);
    Units units(tp, sh);
    Ring kr(tp.nk), qr(tp.nq);
    uint32_t ak_it = 0, keys_it = 0;
    int acc_i = 0;
    uint32_t acc_ph = 0;
    bool ok = true;
    // the accumulators in turn
    auto claim = [&]() -> bool {
        if (!wait(bar(B_ACC_EMPTY + acc_i), acc_ph ^ 1u)) return false;
        ptx::tc_fence_after();
        return true;
    };
    auto acc_at = [&]() { return tmem + kAccCol + (uint32_t)acc_i * kTile; };
    auto acc_done = [&]() {
        ptx::tc_commit_w(bar(B_ACC_FULL + acc_i));
        if (++acc_i == kAccs) {
            acc_i = 0;
            acc_ph ^= 1u;
        }
    };
    for (; ok; ++units.it) {
        if (!(ok = wait(units.full(), units.parity()))) break;
        const Unit u = units.get();
        if (!u.more) break;
        if (AK && u.band) ok = wait(bar(B_AK_FULL), ak_it++ & 1u);
        for (int t = u.t0; t < u.t1 && ok; t += 2) {
            const int tiles = min(2, u.t1 - t);
            int kst[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s >= tiles || !ok) break;
                kst[s] = kr.st;
                ok = wait(bar(B_K_FULL + kr.st), kr.ph);
                kr.next();
            }
            const bool ts = u.qb - u.qa > 1;   // the keys meet more than one query tile: into TMEM, once their
            if (ok && ts) {                    // predecessors there have been multiplied for the last time
                if (keys_it && !(ok = wait(bar(B_KEYS_FREE), (keys_it - 1) & 1u))) break;
                ptx::tc_fence_after();
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (s >= tiles) break;
#pragma unroll 1
                    for (int kk = 0; kk < D / 16; ++kk)
                        copy_keys(tmem + (uint32_t)(s * (D / 2) + 8 * kk),
                                  dk0 + (uint64_t)kst[s] * tile16 + (uint64_t)(((kk >> 2) * BM * 128 + (kk & 3) * 32) >> 4));
                    ptx::tc_commit_w(bar(B_K_EMPTY + kst[s]));
                }
            }
            for (int q = u.qa; q < u.qb && ok; ++q) {
                if (t == u.t0 && !(ok = wait(bar(B_Q_FULL + qr.st), qr.ph))) break;
                ptx::tc_fence_after();
                const uint64_t dq = dq0 + (uint64_t)qr.st * tile16;
                if (AK && query_tile(tp, u, q, u.key(t), u.key(t + 1)).band) {
                    if (!(ok = claim())) break;
#pragma unroll 1
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t at_q = (uint64_t)(((kk >> 2) * BM * 128 + (kk & 3) * 32) >> 4);
                        const uint64_t at_a = (uint64_t)(((kk >> 2) * tp.npad * 128 + (kk & 3) * 32) >> 4);
                        ptx::tc_mma_w(acc_at(), dq + at_q, da + at_a, idR, kk > 0 ? 1u : 0u);
                    }
                    acc_done();
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (s >= tiles) break;
                    if (!(ok = claim())) break;
                    const uint64_t dk = dk0 + (uint64_t)kst[s] * tile16;
                    if (ts) mma_ts<D>(acc_at(), tmem + (uint32_t)(s * (D / 2)), dq, idS);
                    else if (D == 128) ptx::tc_mma_ss_k128(acc_at(), dk, dq, idS, 0u);
                    else ptx::tc_mma_ss_k64(acc_at(), dk, dq, idS, 0u);
                    acc_done();
                }
                if (!ok) break;
                if (t + 2 >= u.t1) {   // (the query tile of a unit of several pairs stays)
                    ptx::tc_commit_w(bar(B_Q_EMPTY + qr.st));
                    qr.next();
                }
            }
            if (!ok) break;
            if (ts) {
                ptx::tc_commit_w(bar(B_KEYS_FREE));
                ++keys_it;
            } else {
                for (int s = 0; s < tiles; ++s) ptx::tc_commit_w(bar(B_K_EMPTY + kst[s]));
            }
        }
        if (!ok) break;
        if (AK && u.band) ptx::tc_commit_w(bar(B_AK_EMPTY));
        ptx::mbar_arrive_w(units.empty());
    }
    // every MMA issued by this warp completes before TMEM is released
    ptx::tc_commit_w(bar(B_DRAIN));
    tc::drain_bar(bar(B_DRAIN), 0, sh.limit);
}

// ======================================================================= sums
// the bits below n of 32
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

template <int D, bool AK>
__device__ void sum_role(const TcParams &tp, const Shared &sh, uint32_t tmem, int group_in) {
    const Params &p = tp.w.p;
    const int group = __shfl_sync(0xffffffffu, group_in, 0);
    const int lane = threadIdx.x & 31;
    const int quad = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5) & 3, 0);
    const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + kAccCol + (uint32_t)group * kTile;
    const uint32_t bars = sh.base + tp.off_bar;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    const float sl2 = p.scale_log2;
    const int k = p.clip_k;
    float *Rs = reinterpret_cast<float *>(sh.ptr + tp.off_r);
    uint32_t r_it = 0, acc_ph = 0;
    int turn = 0;                        // the group that the next product is for
    bool bad = false;
    // a wait that runs out marks the lane, whose warp leaves at the next unit (the flag that it has set ends
    // the others' waits; there is no barrier that they would miss it at)
    auto wait_own = [&](uint32_t b, uint32_t parity) {
        bad = !wait_bar(b, parity, sh, p.err) || bad;
        __syncwarp();
    };
    auto arrive = [&](uint32_t b) {
        __syncwarp();
        ptx::mbar_arrive_w(b);
    };
    auto my_turn = [&]() {
        const bool mine = turn == group;
        turn = turn == kAccs - 1 ? 0 : turn + 1;
        return mine;
    };
    auto wait_acc = [&]() {
        wait_own(bar(B_ACC_FULL + group), acc_ph);
        ptx::tc_fence_after();
        acc_ph ^= 1u;
    };
    auto release_acc = [&]() {
        ptx::tc_fence_before();
        arrive(bar(B_ACC_EMPTY + group));
    };
    Units units(tp, sh);
    Ring nr(kBatches), sr(kSides), pr(kParts);
    for (;; ++units.it) {
        wait_own(units.full(), units.parity());
        if (__any_sync(0xffffffffu, bad)) break;
        const Unit u = units.get();
        arrive(units.empty());
        if (!u.more) break;
        // the group's place in the turns of this unit, in whose order the sums are joined
        const int place = group >= turn ? group - turn : group - turn + kAccs;
        const int last = u.pos0 + u.n - 1, first = p.window > 0 ? max(0, max(u.pos0, 0) - p.window + 1) : 0;
        for (int t0 = u.t0; t0 < u.t1; t0 += 2) {
            const bool two = t0 + 1 < u.t1;
            const int ja = u.key(t0), jb = u.key(t0 + 1);
            // Query tiles from plain0 on lie past the band of either tile, those from there to plain1 - 1 are also whole and
            // see all of the warp's keys: no masks, no tables. They come after the first one or two, but for windows.
            const int plain0 = (max(max(ja, jb) + kTile - 1 + (AK ? k : 0), u.pos0) - u.pos0 + tp.TS - 1) / tp.TS;
            auto plain_end = [&](int j_lo) {
                int end = u.pos0 < 0 ? 0 : min(u.n / tp.TS, u.qb);
                if (p.window > 0 && j_lo + 31 >= p.sinks)
                    end = (int)max(0LL, min((long long)end, ((long long)j_lo + p.window - u.pos0) / tp.TS));
                return end;
            };
            const int end_a = plain_end(ja + quad * 32), end_b = plain_end(jb + quad * 32);
            float2 a01 = dup(0.f), a23 = dup(0.f), b01 = dup(0.f), b23 = dup(0.f);   // of the two tiles
            int tile = -1;               // what this group has of the query tile
            for (int q = u.qa; q < u.qb; ++q) {
                const int in = (q - u.qa) & (kBatch - 1);
                if (in == 0 && t0 == u.t0) wait_own(bar(B_NL_FULL + nr.st), nr.ph);
                const float *nl = reinterpret_cast<const float *>(sh.ptr + tp.off_nl + (nr.st * kBatch + in) * BM * 4);
                const bool band = AK && q < plain0 && query_tile(tp, u, q, ja, jb).band;
                if (AK && band) {
                    if (my_turn()) {   // R, a row each
                        wait_acc();
                        wait_own(bar(B_R_EMPTY), (r_it & 1u) ^ 1u);   // the last one has been read
                        float *row = Rs + (quad * 32 + lane) * tp.SR;
                        float r0 = 0.f;
                        for (int c0 = 0; c0 < tp.npad; c0 += 16) {
                            uint32_t r[16];
                            ptx::tmem_ld16(acc + (uint32_t)c0, r);
                            ptx::tmem_ld_wait();
                            if (c0 == 0) r0 = __uint_as_float(r[0]);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (c0 + e <= k) row[c0 + e] = (__uint_as_float(r[e]) - r0) * sl2;
                        }
                        release_acc();
                        ptx::mbar_arrive_w(bar(B_R_FULL));
                    }
                    wait_own(bar(B_R_FULL), r_it & 1u);
                    ++r_it;
                }
                tile = my_turn() ? 0 : -1;
                if (two && my_turn()) tile = 1;
                if (tile >= 0) {
                    float2 s01 = tile ? b01 : a01, s23 = tile ? b23 : a23;
                    auto weights = [&](float *x, int c) {   // of 32 columns, with their constants
#pragma unroll
                        for (int e = 0; e < KB; e += 4) {
                            const float4 n = *reinterpret_cast<const float4 *>(nl + c + e);
                            const float2 v = __ffma2_rn(pair(x, e), dup(sl2), make_float2(n.x, n.y));
                            const float2 w = __ffma2_rn(pair(x, e + 2), dup(sl2), make_float2(n.z, n.w));
                            x[e] = ptx::ex2(v.x);
                            x[e + 1] = ptx::ex2(v.y);
                            x[e + 2] = ptx::ex2(w.x);
                            x[e + 3] = ptx::ex2(w.y);
                        }
                    };
                    auto add = [&](const float *x) {
#pragma unroll
                        for (int e = 0; e < KB; e += 4) {
                            s01 = __fadd2_rn(s01, make_float2(x[e], x[e + 1]));
                            s23 = __fadd2_rn(s23, make_float2(x[e + 2], x[e + 3]));
                        }
                    };
                    wait_acc();
                    if (q >= plain0 && q < (tile ? end_b : end_a)) {
                        float x[2][KB];                     // 32 columns come while the last ones are added up
                        ptx::tmem_ld32f(acc, x[0]);
#pragma unroll
                        for (int i = 0; i < kTile / KB; ++i) {
                            ptx::tmem_ld_wait();
                            if (i + 1 < kTile / KB) ptx::tmem_ld32f(acc + (uint32_t)((i + 1) * KB), x[(i + 1) & 1]);
                            else release_acc();
                            weights(x[i & 1], i * KB);
                            add(x[i & 1]);
                        }
                    } else {
                        const int j = (tile ? jb : ja) + quad * 32 + lane, j_lo = j - lane, j_hi = j_lo + 31;
                        const QueryTile t = query_tile(tp, u, q, ja, jb);
                        const bool far = !AK || k == 0 || j_hi <= t.pos_lo - k;   // else R is there
                        const bool full = t.ntok == tp.TS && j_hi <= t.pos_lo &&
                                          (p.window == 0 || j_lo > t.pos_hi - p.window || j_hi < p.sinks);
                        const bool dead = j_lo > t.pos_hi || (p.window > 0 && j_hi <= t.pos_lo - p.window && j_lo >= p.sinks);
                        if (!dead) {
                            // the columns that see this key: tokens from its own on, as far as the window reaches
                            int c_lo = 0, c_hi = kTile;
                            if (!full) {
                                c_lo = max(0, j - t.pos_lo) * p.g;
                                c_hi = t.ntok * p.g;
                                if (p.window > 0 && j >= p.sinks)
                                    c_hi = (int)max(0LL, min((long long)c_hi, ((long long)j + p.window - t.pos_lo) * p.g));
                            }
                            int hh = 0, lab = j - t.pos_lo + k;
                            const float *row = Rs;
#pragma unroll 1
                            for (int c = 0; c < t.ntok * p.g; c += KB) {
                                // 32 columns, whose tokens stand at p0 .. p1
                                const int p0 = t.pos_lo + c / p.g, p1 = t.pos_lo + (c + KB - 1) / p.g;
                                const bool past = far || p0 - k >= j_hi;   // of the band for all of the warp's keys
                                if (p1 < j_lo) {                            // none of them in sight yet
                                    row += KB * tp.SR;
                                    hh = (hh + KB) % p.g;
                                    lab = j - t.pos_lo + k - (c + KB) / p.g;
                                    continue;
                                }
                                float x[KB];
                                ptx::tmem_ld32f(acc + (uint32_t)c, x);
                                ptx::tmem_ld_wait();
                                if (past) {
                                    weights(x, c);
                                    row += KB * tp.SR;
                                    hh = (hh + KB) % p.g;
                                    lab = j - t.pos_lo + k - (c + KB) / p.g;
                                } else if (p.g == 1) {   // R of token i: its entry for key j, one further back with every token
#pragma unroll
                                    for (int e = 0; e < KB; e += 4) {
                                        const float4 n = *reinterpret_cast<const float4 *>(nl + c + e);
                                        const float ns[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
                                        for (int i = 0; i < 4; ++i) {
                                            x[e + i] = ptx::ex2(fmaf(x[e + i], sl2, ns[i] + row[__viaddmin_s32_relu(lab, -(e + i), k)]));
                                            row += tp.SR;
                                        }
                                    }
                                    lab -= KB;
                                } else {
#pragma unroll
                                    for (int e = 0; e < KB; ++e) {
                                        x[e] = ptx::ex2(fmaf(x[e], sl2, nl[c + e] + row[min(max(lab, 0), k)]));
                                        row += tp.SR;
                                        if (++hh == p.g) {
                                            hh = 0;
                                            --lab;
                                        }
                                    }
                                }
                                // (masked where a row does not see a key of the warp's, or is none)
                                if (!full && (p.window > 0 || p0 < j_hi || c + KB > t.ntok * p.g)) {
                                    const uint32_t on = below(c_hi - c) & ~below(c_lo - c);
#pragma unroll
                                    for (int e = 0; e < KB; ++e) x[e] = on >> e & 1 ? x[e] : 0.f;
                                }
                                add(x);
                                __syncwarp();
                            }
                        }
                        release_acc();
                    }
                    if (tile) {
                        b01 = s01;
                        b23 = s23;
                    } else {
                        a01 = s01;
                        a23 = s23;
                    }
                }
                if (AK && band) arrive(bar(B_R_EMPTY));
                if ((in == kBatch - 1 || q + 1 == u.qb) && t0 + 2 >= u.t1) {
                    arrive(bar(B_NL_EMPTY + nr.st));
                    nr.next();
                }
            }
            // ---- the sums: of several query tiles joined by one group for either tile
            int mine = tile;             // the tile that this group finishes
            const float sum_a = (a01.x + a01.y) + (a23.x + a23.y), sum_b = (b01.x + b01.y) + (b23.x + b23.y);
            float sum = tile > 0 ? sum_b : sum_a;
            if (u.qb - u.qa != 1) {
                float *part = reinterpret_cast<float *>(sh.ptr + tp.off_part + pr.st * kPartBytes) + quad * 32 + lane;
                wait_own(bar(B_PART_EMPTY + pr.st), pr.ph ^ 1u);
                part[place * 2 * kTile] = sum_a;
                part[(place * 2 + 1) * kTile] = sum_b;
                arrive(bar(B_PART_FULL + pr.st));
                mine = group == 0 || (group == 1 && two) ? group : -1;
                if (group < 2) {
                    wait_own(bar(B_PART_FULL + pr.st), pr.ph);
                    sum = 0.f;
#pragma unroll
                    for (int i = 0; i < kAccs; ++i) sum += part[(i * 2 + group) * kTile];
                    arrive(bar(B_PART_EMPTY + pr.st));
                }
                pr.next();
            }
            for (int i = 0; i < (two ? 2 : 1); ++i, sr.next()) {
                if (mine != i) continue;
                const int j0 = i ? jb : ja, j = j0 + quad * 32 + lane;
                wait_own(bar(B_SIDE_FULL + sr.st), sr.ph);
                const uint8_t *side = sh.ptr + tp.off_side + sr.st * kSideBytes;
                const int pg = reinterpret_cast<const int *>(side)[(j - j0) / tp.box];
                const bool seen = pg >= 0 && j <= last && (j >= first || j < p.sinks);
                float *at = tp.w.mass + (long long)pg * tp.w.mass_stride +
                            (((long long)u.kvh << p.pshift) + (j & ((1 << p.pshift) - 1)));
                arrive(bar(B_SIDE_EMPTY + sr.st));
                if (seen && !bad) leave_mass(tp.w, at, sum, j, u.pos0);
            }
        }
    }
}

// ======================================================================= kernel
template <int D, bool AK>
__global__ void __launch_bounds__(kThreads, 1)
    weights_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_ak, const __grid_constant__ TcParams tp) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Shared sh;
    sh.base = ptx::smem_u32(smem_raw);
    sh.ptr = smem_raw;
    uint64_t *bar_ptr = reinterpret_cast<uint64_t *>(sh.ptr + tp.off_bar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_ptr + kNumBars);
    sh.abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    sh.limit = tp.w.p.wait_limit;
    const int warp = threadIdx.x >> 5;
    const uint32_t bars = sh.base + tp.off_bar;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t n = 1;
            if (i >= B_UNIT_EMPTY && i < B_ACC_FULL) n = 3 + kSumWarps;
            if (i >= B_ACC_EMPTY && i < B_SIDE_FULL) n = 4;                    // a group
            if (i >= B_SIDE_EMPTY && i < B_NL_FULL) n = 4;                     // a group
            if (i >= B_NL_EMPTY && i < B_R_FULL) n = kSumWarps;
            if (i == B_R_FULL) n = 4;
            if (i == B_R_EMPTY) n = kSumWarps;
            if (i >= B_PART_FULL && i < B_PART_EMPTY) n = kSumWarps;
            if (i >= B_PART_EMPTY && i < B_KEYS_FREE) n = 8;                   // two groups
            ptx::mbar_init(bars + 8u * (uint32_t)i, n);
        }
        *sh.abort_flag = 0;
        ptx::mbar_init_fence();
        ptx::tma_prefetch_desc(&tm_q);
        ptx::tma_prefetch_desc(&tm_k);
    }
    // rows of a query tile that no copy writes (128 is no multiple of the group)
    for (int i = threadIdx.x; i < tp.nq * (int)tp.tile_bytes / 16; i += kThreads)
        reinterpret_cast<uint4 *>(sh.ptr + tp.off_q)[i] = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async_smem();
    if (warp == 1) ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    grid_wait();
    grid_release();
    if (warp < 4) {
        if (warp == 0) load_role<D, AK>(tp, sh, &tm_q, &tm_k, &tm_ak);
        else if (warp == 1) mma_role<D, AK>(tp, sh, tmem);
        else if (warp == 2) const_role(tp, sh);
        else ticket_role<AK>(tp, sh);
    } else {
        sum_role<D, AK>(tp, sh, tmem, (warp - 4) >> 2);
    }
    __syncwarp();
    ptx::tc_fence_before();
    ptx::cta_barrier();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <int D, bool AK>
cudaError_t launch_variant(const CUtensorMap (&tm)[3], const TcParams &tp, uint32_t smem, int grid, cudaStream_t s) {
    auto kern = weights_tc_kernel<D, AK>;
    const cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kern), device_info());
    if (e != cudaSuccess) return e;
    return launch_early(kern, dim3(grid), kThreads, smem, s, tm[0], tm[1], tm[2], tp);
}

template <int D>
cudaError_t launch_d(const PagedWeightsArgs &wa, const WeightParams &w, cudaStream_t s) {
    const PagedArgs &a = wa.a;
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return cudaErrorInvalidDevice;
    TcParams tp;
    std::memset(&tp, 0, sizeof(tp));
    tp.w = w;
    const Params &p = w.p;
    const bool ak = a.aK != nullptr;
    tp.TS = BM / p.g;
    tp.w.tile_tokens = tp.TS;
    tp.npad = (p.clip_k + 1 + 15) / 16 * 16;
    tp.SR = (p.clip_k + 1) | 1;   // a column walk of R hits 32 banks
    tp.box = a.page_size < kTile ? a.page_size : kTile;
    tp.tile_bytes = (uint32_t)kTile * D * 2;
    const uint32_t ak_bytes = ak && p.clip_k ? (uint32_t)tp.npad * D * 2 : 0, r_bytes = ak && p.clip_k ? BM * tp.SR * 4 : 0;
    const uint32_t rest = r_bytes + kBatches * kBatch * BM * 4 + kSides * kSideBytes + kParts * kPartBytes + kUnits * sizeof(Unit) + kNumBars * 8 + 16;
    int stages = (int)(((uint32_t)di.smem_optin - rest - ak_bytes) / tp.tile_bytes);
    if (stages > kMaxK + kMaxQ) stages = kMaxK + kMaxQ;
    if (stages < 3) return cudaErrorNotSupported;
    // Two tiles of keys are enough where they move on to TMEM. One query tile to a request: the keys stream
    // by and the query tile stays, so more keys are on their way
    const long long rows = (long long)(a.max_new > 0 ? a.max_new : a.tokens / a.B) * p.g;
    tp.nk = rows <= BM && stages > 4 ? (stages - 2 < kMaxK ? stages - 2 : kMaxK) : 2;
    tp.nq = stages - tp.nk < kMaxQ ? stages - tp.nk : kMaxQ;
    tp.off_q = tp.nk * tp.tile_bytes;
    tp.off_ak = tp.off_q + tp.nq * tp.tile_bytes;
    tp.off_nl = tp.off_ak + ak_bytes;
    tp.off_side = tp.off_nl + kBatches * kBatch * BM * 4;
    tp.off_part = tp.off_side + kSides * kSideBytes;
    tp.off_unit = tp.off_part + kParts * kPartBytes;
    tp.off_bar = tp.off_unit + kUnits * sizeof(Unit);
    tp.off_r = tp.off_bar + kNumBars * 8 + 16;
    uint32_t smem = tp.off_r + r_bytes;
    // TMEM is taken whole, so one CTA to an SM, whatever its tables leave
    if (smem < 120 * 1024) smem = 120 * 1024;
    CUtensorMap tm[3];
    if (!make_query_map(&tm[0], a, p.g, tp.TS) || !make_page_map(&tm[1], a.k_pages, a, tp.box)) return cudaErrorInvalidValue;
    tm[2] = tm[0];
    const uint64_t Ht = a.ths ? (uint64_t)a.Hkv : 1, hs = a.ths ? (uint64_t)a.ths * 2 : (uint64_t)(2 * a.clip_k + 1) * D * 2;
    if (ak && !tc::make_map(&tm[2], a.aK, D, p.clip_k + 1, Ht, D * 2, hs, (uint32_t)tp.npad)) return cudaErrorInvalidValue;
    cudaError_t e = launch_weights_prep(tp.w, true, s);
    if (e != cudaSuccess) return e;
    return ak ? launch_variant<D, true>(tm, tp, smem, di.sms, s) : launch_variant<D, false>(tm, tp, smem, di.sms, s);
}

}  // namespace

bool weights_tc_covers(const PagedWeightsArgs &a) { return a.a.clip_k <= 127 && pages_by_tma(a.a); }

cudaError_t launch_weights_tc(const PagedWeightsArgs &a, WeightParams w, cudaStream_t s) {
    w.per_tile = 0;
    return a.a.d == 64 ? launch_d<64>(a, w, s) : launch_d<128>(a, w, s);
}

}  // namespace paged
}  // namespace relattn
