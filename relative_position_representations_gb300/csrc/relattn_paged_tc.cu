// Paged attention on the tensor cores: chunks of prompts, whole prompts and generated tokens in
// one launch. bf16, d = 64 or 128, pages of at least 8 keys, clip_k <= 127.
//
// The formulas are those of relattn_tc_kernel.cuh (section 3.4, eq. 3 and eq. 4 in split form,
// causal): S = Q K^T, R = Q aK^T over the k + 1 table rows, O = P V + beta aV. What differs is where
// the rows and keys come from and how the work is cut.
//
// Rows. The g query heads that share a key head are packed: TS = 128 / g tokens make one 128-row
// tile, loaded by one TMA box of TS tokens x g heads. An item has up to two such tiles
// ("slots") of one request and key head. Two full tiles share every K/V tile (the L2 traffic per
// product halves). An item of one tile only runs its key tiles alternately in the two slots,
// with a softmax state each, joined at its end: otherwise a generated token would leave half of
// the CTA idle.
// Keys. The producer looks up the pages of a tile (one lane per page, K and V share the entry) and
// every lane issues the TMA box of its own page; pages that no row of the item sees are
// skipped. Rows of V that no row sees may hold anything, NaN among it, and 0 * NaN is NaN: the
// MMA warps overwrite them with zeros first (at most two tiles of a piece have such rows). K needs
// no such care, scores of unseen keys are replaced, not added to.
// Work is split over the CTAs by keys (relattn_paged.cuh).
//
// What bounds it. d = 128: the chain of a slot, S, softmax (1750 cycles), P V and the next S over P's
// columns (1700 with the hand-offs), 3450 cycles per tile of both slots where the tensor cores work
// 2048; TMEM is full, so no second S can wait. d = 64 (P beside S): the issue of the softmax, two
// warps to a scheduler, 2550 cycles a tile. A piece costs 8 to 10 thousand cycles beside its tiles
// (R, masks and band, write-out). A generated token fills g of the 128 rows of its tiles. Four prompts
// of 4096 tokens, 16 heads of 128, key term: 285 us, 982 TFLOP/s; a mixed step (20 generated tokens, 4
// chunks of about 500, up to 8K keys): 110 us, 685, where the generated tokens are 20 of 1989 tokens,
// 2156 of 7092 tiles and by the measured costs 26 % of the work;
// chunks of 2048 under a window of 4096, d = 64, both terms: 115 us, 605. Dropped: scores in halves
// of 64 keys with two buffers (mixed step 132 -> 137 us, prompts 318 -> 439: N = 64 products read A
// twice as often, and every half pays the hand-offs), part of the exponentials as a polynomial (318
// -> 343 us: the issue slots are scarcer than the unit, which does a warp's in 4 cycles).
//
// Roles (384 threads, one CTA per SM): warp 3 walks the CTA's range, announces the pieces and loads
// their query tiles, warp 0 feeds the ring (aK, K and V tiles, aV, in the order of use), warps 1 and
// 2 issue the MMAs of slot 0 and 1, warps 4-7 and 8-11 run the rows of slot 0 and 1, one thread per row. TMEM as in relattn_tc_kernel.cuh: S of
// slot s at 128 s, O at 256 + d s, P (bf16) at 384 + 64 s (d = 64) or over the lower half of S
// (d = 128), beta over the upper half of S.
// The band of the last k keys needs no accumulation: each of its table rows meets one key per
// query row, so the score (log2 domain) replaces the R entry it has just used, and beta is
// formed from the scores at the end.
#include <cstdint>
#include <cstring>
#include <mutex>

#include "relattn_paged_tma.cuh"

namespace relattn {
namespace paged {
namespace {

using tc::BM;
using tc::dup;
using tc::max32;
using tc::pair;
using tc::put;
using tc::Shared;
using tc::slot_sync;
using tc::wait_bar;
using tc::wait_bar_ctrl;

constexpr int kThreads = tc::kThreads;
constexpr int kTcGrid = 160;                 // CTAs at most: one per SM
static_assert(kTcGrid * 2 * BM <= kMaxGrid * kRecordRows, "records of the workspace");
constexpr int KB = 32;                       // keys per softmax chunk
constexpr int NCH = kTile / KB;
constexpr int kMaxStages = 8;
constexpr uint32_t kStatBytes = 2 * BM * 8;
constexpr uint32_t kOutBytes = 32 * 64;   // staging of a warp's output rows
constexpr float kRescaleLog2 = tc::kRescaleLog2;

template <int D>
struct Tm {
    static constexpr bool P_ALIAS = D == 128;
    static __device__ __forceinline__ uint32_t S(int s) { return 128u * (uint32_t)s; }
    static __device__ __forceinline__ uint32_t O(int s) { return 256u + (uint32_t)(D * s); }
    static __device__ __forceinline__ uint32_t P(int s) { return P_ALIAS ? 128u * (uint32_t)s : 384u + 64u * (uint32_t)s; }
    static __device__ __forceinline__ uint32_t Bn(int s) { return S(s) + 64u; }
};

enum : int { SB_S_FULL = 0, SB_S_EMPTY, SB_P_FULL, SB_P_HALF, SB_PV_DONE, SB_O_FULL, SB_DRAIN, SB_BN_FULL, SB_BN_DONE, kSlotBars };
enum : int {
    B_Q_FULL = 0, B_Q_EMPTY = 2, B_X = 4, B_PIECE_FULL, B_PIECE_EMPTY = B_PIECE_FULL + kPieces,
    B_SLOT0 = B_PIECE_EMPTY + kPieces, B_KV0 = B_SLOT0 + 2 * kSlotBars
};
constexpr int kNumBars = B_KV0 + 2 * kMaxStages;

struct TcParams {
    Params p;
    int TS;              // tokens per slot
    int W, npad;         // table rows (clip_k + 1), rounded up to 16
    int SR;              // row stride (floats) of the R rows in shared memory
    int box;             // keys per TMA box: min(page_size, 128)
    int stages;
    uint32_t stage_bytes;
    uint32_t off_q[2], off_kv, off_r[2], off_stat, off_piece, off_bar;
};

// the pieces in order; `wait` is the role's own bounded wait
struct Pieces {
    uint32_t bars;
    const Piece *ring;
    uint32_t it;
    __device__ __forceinline__ Pieces(const TcParams &tp, const Shared &sh)
        : bars(sh.base + tp.off_bar), ring(reinterpret_cast<const Piece *>(sh.ptr + tp.off_piece)), it(0) {}
    // false: the wait ran out, or there is no more
    template <typename Wait>
    __device__ __forceinline__ bool next(Wait wait, Piece &g, bool &ok) {
        if (!(ok = wait(bars + 8u * (B_PIECE_FULL + (it & (kPieces - 1))), (it / kPieces) & 1u))) return false;
        // through a broadcast of lane 0: the compiler then knows every field, and each branch on it, to
        // be warp-uniform (tcgen05 and TMA operands stay in uniform registers)
        const Piece &s = ring[it & (kPieces - 1)];
        auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
        g = Piece{uni(s.row0), uni(s.cnt), uni(s.pos_lo), uni(s.pos_hi), uni(s.ns), uni(s.lo),
                  uni(s.nt),   uni(s.t0),  uni(s.t1),     uni(s.kvh),    uni(s.b),  uni(s.act)};
        return g.cnt > 0;
    }
    __device__ __forceinline__ uint32_t empty() const { return bars + 8u * (B_PIECE_EMPTY + (it & (kPieces - 1))); }
};

// D += A B over 64 keys (4 k-steps), one elect for the chain: A (P, bf16 pairs) in TMEM, 8 columns per
// step, B (V) MN-major with 128-byte swizzle, 16 rows x 128 bytes per step
__device__ __forceinline__ void mma_ts_k64(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 t, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.s64 b1, %2, 128;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "add.u32 a1, %1, 16;\n\tadd.s64 b1, %2, 256;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "add.u32 a1, %1, 24;\n\tadd.s64 b1, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "}\n" ::"r"(d),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate), "r"(1u)
        : "memory");
}

// one slot's share of a piece
struct SlotWork {
    bool split;          // the two slots take the tiles of the same rows in turn
    int tok0, ntok;      // tokens of the slot within the item
    int pos_lo, pos_hi;  // their positions
    int first;           // first key in the window of the slot's first token
    int t_last;          // the last tile of the piece that the slot uses (t0 - 1: none)
    __device__ __forceinline__ bool uses(const Params &p, const Piece &g, int slot, int t) const {
        if (split) return ((t - g.t0) & 1) == slot;
        const int j0 = g.tile(t) * kTile;
        return j0 <= pos_hi && (j0 + kTile > first || j0 < p.sinks);
    }
};

__device__ __forceinline__ SlotWork slot_work(const TcParams &tp, const Piece &g, int slot) {
    const Params &p = tp.p;
    SlotWork w;
    w.split = g.cnt <= tp.TS;
    w.tok0 = w.split ? 0 : slot * tp.TS;
    w.ntok = min(tp.TS, g.cnt - w.tok0);
    w.pos_lo = g.pos_lo + w.tok0;
    w.pos_hi = w.pos_lo + w.ntok - 1;
    w.first = p.window > 0 ? max(0, max(w.pos_lo, 0) - p.window + 1) : 0;
    w.t_last = g.t1 - 1;
    while (w.t_last >= g.t0 && !w.uses(p, g, slot, w.t_last)) --w.t_last;
    return w;
}

// position in the ring
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

// Order of the ring entries of a piece: aK; then for i = 0, 1, ...: K_i, V_{i - lag}; aV. With P in
// its own columns (d = 64) a slot's next scores are computed while its softmax still works, so its
// next K comes before its V: one tile ahead, two where the slots take turns.
template <int D>
__device__ __forceinline__ int v_lag(bool split) {
    return Tm<D>::P_ALIAS ? 0 : (split ? 2 : 1);
}

// ======================================================================= producers
template <int D, bool AK, bool AV>
__device__ void kv_role(const TcParams &tp, const Shared &sh, const CUtensorMap *tm_k,
                        const CUtensorMap *tm_v, const CUtensorMap *tm_ak, const CUtensorMap *tm_av) {
    const Params &p = tp.p;
    constexpr int DB = D / 64;
    const int lane = threadIdx.x & 31;
    const uint32_t bars = sh.base + tp.off_bar, sKV = sh.base + tp.off_kv;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        const bool r = wait_bar_ctrl(b, parity, sh, p.err);
        return __all_sync(0xffffffffu, r ? 1 : 0) != 0;
    };
    const int nbox = kTile / tp.box;                 // boxes of a tile, at most 16
    const int my_box = lane % nbox, my_blk = lane / nbox;
    Ring ring(tp.stages);
    uint32_t count = 0;
    bool ok = true;
    auto claim = [&]() -> bool { return wait(bar(B_KV0 + kMaxStages + ring.st), ring.ph ^ 1u); };
    auto step = [&]() {
        ring.next();
        ++count;
    };
    auto table = [&](const CUtensorMap *tm, int kvh) -> bool {
        if (!claim()) return false;
        ptx::mbar_expect_tx_w(bar(B_KV0 + ring.st), (uint32_t)tp.npad * D * 2);
#pragma unroll
        for (int blk = 0; blk < DB; ++blk)
            ptx::tma_load_3d_w(sKV + (uint32_t)ring.st * tp.stage_bytes + blk * tp.npad * 128, tm,
                               bar(B_KV0 + ring.st), blk * 64, 0, p.ths ? kvh : 0);
        step();
        return true;
    };
    Pieces pieces(tp, sh);
    Piece g;
    for (; ok && pieces.next(wait, g, ok); ptx::mbar_arrive_w(pieces.empty()), ++pieces.it) {
        const int nt = g.t1 - g.t0;
        if (nt == 0) continue;
        const bool split = g.cnt <= tp.TS;
        const int lag = v_lag<D>(split);
        const int first = g.first(p);
        const int *bt = p.bt + (long long)g.b * p.bt_stride;
        if (AK && !(ok = table(tm_ak, g.kvh))) break;
        // this lane's box of tile t: page number (or -1), and whether any row sees a key of it
        auto lookup = [&](int t, bool &seen) -> int {
            const int j = g.tile(t) * kTile + my_box * tp.box;
            seen = t < g.t1 && j <= g.pos_hi && (j + tp.box > first || j < p.sinks);
            return seen ? __ldg(bt + (j >> p.pshift)) : -1;
        };
        // pages of tiles i, i - 1 and i - 2 (V comes up to two tiles behind K), tile i + 1 ahead
        bool sn, s0 = false, s1 = false, s2 = false;
        int pn = lookup(g.t0, sn), p0 = -1, p1 = -1, p2 = -1;
        auto load = [&](const CUtensorMap *tm, int t, int pg, bool seen) -> bool {
            if (!claim()) return false;
            const uint32_t full = bar(B_KV0 + ring.st);
            const unsigned m = __ballot_sync(0xffffffffu, seen && my_blk == 0);
            ptx::mbar_expect_tx_w(full, (uint32_t)__popc(m) * tp.box * D * 2);
            __syncwarp();
            const int j = g.tile(t) * kTile + my_box * tp.box;
            const int row = j & ((1 << p.pshift) - 1);
            if (seen && my_blk < DB) {
                const bool bad = (unsigned)pg >= (unsigned)p.num_pages;
                if (bad) report_page(p);
                // a page outside the cache: a box outside the tensor, which reads as zeros
                tma_load_4d(sKV + (uint32_t)ring.st * tp.stage_bytes + my_blk * kTile * 128 + my_box * tp.box * 128, tm,
                            full, my_blk * 64, row, g.kvh, bad ? p.num_pages : pg);
            }
            __syncwarp();
            step();
            return true;
        };
        for (int i = 0; i < nt + lag && ok; ++i) {
            p2 = p1; s2 = s1;
            p1 = p0; s1 = s0;
            p0 = pn; s0 = sn;
            if (i < nt) {
                pn = lookup(g.t0 + i + 1, sn);
                if (!(ok = load(tm_k, g.t0 + i, p0, s0))) break;
            }
            if (i >= lag) {
                const int pv = lag == 0 ? p0 : lag == 1 ? p1 : p2;
                const bool sv = lag == 0 ? s0 : lag == 1 ? s1 : s2;
                ok = load(tm_v, g.t0 + i - lag, pv, sv);
            }
        }
        if (ok && AV) ok = table(tm_av, g.kvh);
    }
    // the copies issued into shared memory have landed before the CTA exits
    for (uint32_t i = count > (uint32_t)tp.stages ? count - tp.stages : 0; i < count; ++i)
        tc::drain_bar(bar(B_KV0 + (int)(i % tp.stages)), (i / tp.stages) & 1u, sh.limit);
}

// Walks the CTA's range, announces its pieces and loads their query tiles.
template <int D>
__device__ void walk_role(const TcParams &tp, const Range rg, const Shared &sh, const CUtensorMap *tm_q) {
    const Params &p = tp.p;
    constexpr int DB = D / 64;
    const int lane = threadIdx.x & 31;
    const uint32_t bars = sh.base + tp.off_bar;
    const uint32_t full = bars + 8u * B_Q_FULL, empty = bars + 8u * B_Q_EMPTY;
    Piece *ring = reinterpret_cast<Piece *>(sh.ptr + tp.off_piece);
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        const bool r = wait_bar_ctrl(b, parity, sh, p.err);
        return __all_sync(0xffffffffu, r ? 1 : 0) != 0;
    };
    Walk walk(p, rg);
    Segment g{};
    uint32_t it = 0, q_it[2] = {0, 0};
    bool more = true, any = false;
    while (more) {
        more = walk.next(p, g);
        any = any || more;
        const int i = it & (kPieces - 1);
        if (!wait(bars + 8u * (B_PIECE_EMPTY + i), ((it / kPieces) & 1u) ^ 1u)) break;
        Piece pc = make_piece(g, more);
        if (more && g.t1 > g.t0)   // (here, where nothing waits for it)
            for (int s = 0; s < 2; ++s)
                if (slot_work(tp, pc, s).t_last >= pc.t0) pc.act |= 1 << s;
        if (lane == 0) ring[i] = pc;
        __syncwarp();
        ptx::mbar_arrive_w(bars + 8u * (B_PIECE_FULL + i));
        ++it;
        if (!more || g.t1 == g.t0) continue;
        const int ns = g.it.cnt <= tp.TS ? 1 : 2;
        bool ok = true;
        for (int s = 0; s < ns && ok; ++s) {
            if (!(ok = wait(empty + 8 * s, (q_it[s] & 1u) ^ 1u))) break;
            ptx::mbar_expect_tx_w(full + 8 * s, (uint32_t)tp.TS * p.g * D * 2);
#pragma unroll
            for (int blk = 0; blk < DB && !(p.withhold && it == 1); ++blk)
                ptx::tma_load_3d_w(sh.base + tp.off_q[s] + blk * BM * 128, tm_q, full + 8 * s, blk * 64, g.kvh * p.g,
                                   g.s.q0 + g.it.i0 + s * tp.TS);
            ++q_it[s];
        }
        if (!ok) break;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
        if (q_it[s]) tc::drain_bar(full + 8 * s, (q_it[s] - 1) & 1u, sh.limit);
    // (after an abort the pieces' records hold anything, as does the output)
    if (lane == 0) write_desc(p, any ? &g : nullptr, rg.total);
}

// ======================================================================= MMA issuers
// One warp per slot; both walk every ring entry and each releases it, so the release barriers
// count two arrivals; an entry, or Q, is released only after it was waited for.
template <int D, bool AK, bool AV>
__device__ void mma_role(const TcParams &tp, const Shared &sh, uint32_t tmem, int slot_in) {
    using T = Tm<D>;
    const Params &p = tp.p;
    const int slot = __shfl_sync(0xffffffffu, slot_in, 0);
    const int lane = threadIdx.x & 31;
    const uint32_t bars = sh.base + tp.off_bar;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto sbar = [&](int which) { return bar(B_SLOT0 + kSlotBars * slot + which); };
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        const bool r = wait_bar_ctrl(b, parity, sh, p.err);
        return __all_sync(0xffffffffu, r ? 1 : 0) != 0;
    };
    const uint64_t dk0 = ptx::sdesc_sw128(sh.base + tp.off_kv, 16, 1024);
    const uint64_t dv0 = ptx::sdesc_sw128(sh.base + tp.off_kv, kTile * 128, 1024);
    const uint64_t stage16 = tp.stage_bytes >> 4;
    const uint32_t tS = tmem + T::S(slot), tO = tmem + T::O(slot), tP = tmem + T::P(slot), tB = tmem + T::Bn(slot);
    constexpr uint32_t idS = ptx::idesc_bf16(BM, kTile, 0), idPV = ptx::idesc_bf16(BM, D, 1);
    auto kstep = [](int kk, int rows) -> uint64_t {
        return (uint64_t)(((kk >> 2) * rows * 128 + (kk & 3) * 32) >> 4);
    };
    Ring ring(tp.stages);
    uint32_t q_it[2] = {0, 0}, s_it = 0, p_it = 0, pv_it = 0, bn_it = 0, bd_it = 0;
    bool pv_pending = false, bn_pending = false, ok = true;

    // before an MMA writes the slot's S columns: the rows have read the previous scores, and the
    // MMAs that read P (over S) or beta from those columns are done
    auto claim_s = [&]() -> bool {
        if (bn_pending) {
            if (!wait(sbar(SB_BN_DONE), (bd_it - 1u) & 1u)) return false;
            bn_pending = false;
        }
        if (T::P_ALIAS && pv_pending) {
            if (!wait(sbar(SB_PV_DONE), (pv_it - 1u) & 1u)) return false;
            pv_pending = false;
        }
        if (!wait(sbar(SB_S_EMPTY), (s_it & 1u) ^ 1u)) return false;
        ++s_it;
        ptx::tc_fence_after();
        return true;
    };
    Pieces pieces(tp, sh);
    Piece g;
    for (; ok && pieces.next(wait, g, ok); ptx::mbar_arrive_w(pieces.empty()), ++pieces.it) {
        const int nt = g.t1 - g.t0;
        if (nt == 0) continue;
        const SlotWork w = slot_work(tp, g, slot);
        const bool act = w.t_last >= g.t0;
        const bool tables = act && (!w.split || slot == 0);   // R and beta belong to this slot
        const int lag = v_lag<D>(w.split);
        const uint64_t dq = ptx::sdesc_sw128(sh.base + tp.off_q[w.split ? 0 : slot], 16, 1024);
        const int first = g.first(p);
        // the query tile that this slot reads; the other one is released as soon as it is there
        const int mine = w.split ? 0 : slot;
        for (int b = 0; b < (w.split ? 1 : 2) && ok; ++b) {
            if (!(ok = wait(bar(B_Q_FULL + b), q_it[b] & 1u))) break;
            ++q_it[b];
            if (b != mine || !act) ptx::mbar_arrive_w(bar(B_Q_EMPTY + b));
            if (b == mine) break;
        }
        if (!ok) break;
        ptx::tc_fence_after();
        if (AK) {   // R = Q aK^T into the slot's S columns
            if (!(ok = wait(bar(B_KV0 + ring.st), ring.ph))) break;
            const uint32_t empty = bar(B_KV0 + kMaxStages + ring.st);
            if (tables) {
                if (!(ok = claim_s())) break;
                const uint32_t idR = ptx::idesc_bf16(BM, (uint32_t)tp.npad, 0);
                const uint64_t da = dk0 + (uint64_t)ring.st * stage16;
#pragma unroll 1
                for (int kk = 0; kk < D / 16; ++kk)
                    ptx::tc_mma_w(tS, dq + kstep(kk, BM), da + kstep(kk, tp.npad), idR, kk > 0 ? 1u : 0u);
                ptx::tc_commit_w(sbar(SB_S_FULL));
                ptx::tc_commit_w(empty);
            } else {
                ptx::mbar_arrive_w(empty);
            }
            ring.next();
        }
        bool started = false;
        for (int i = 0; i < nt + lag && ok; ++i) {
            if (i < nt) {   // S_i = Q K_i^T
                const int t = g.t0 + i;
                if (!(ok = wait(bar(B_KV0 + ring.st), ring.ph))) break;
                const uint32_t empty = bar(B_KV0 + kMaxStages + ring.st);
                if (w.uses(p, g, slot, t)) {
                    ptx::tc_fence_after();
                    if (!(ok = claim_s())) break;
                    const uint64_t dk = dk0 + (uint64_t)ring.st * stage16;
                    if (D == 128) ptx::tc_mma_ss_k128(tS, dq, dk, idS, 0u);
                    else ptx::tc_mma_ss_k64(tS, dq, dk, idS, 0u);
                    ptx::tc_commit_w(sbar(SB_S_FULL));
                    ptx::tc_commit_w(empty);
                    if (t == w.t_last) ptx::tc_commit_w(bar(B_Q_EMPTY + mine));   // last read of Q
                } else {
                    ptx::mbar_arrive_w(empty);
                }
                ring.next();
            }
            if (i >= lag) {   // O += P V
                const int t = g.t0 + i - lag;
                if (!(ok = wait(bar(B_KV0 + ring.st), ring.ph))) break;
                const uint32_t empty = bar(B_KV0 + kMaxStages + ring.st);
                if (w.uses(p, g, slot, t)) {
                    // rows of V that no row of the item sees
                    const int j0 = g.tile(t) * kTile;
                    const int n_seen = g.pos_hi + 1 - j0;                   // rows below are within the cache
                    const int u0 = max(0, p.sinks - j0), u1 = first - j0;      // rows u0 .. u1 - 1 lie behind the window
                    if (n_seen < kTile || u1 > u0) {
                        const uint32_t base = sh.base + tp.off_kv + (uint32_t)ring.st * tp.stage_bytes;
                        for (int r = lane; r < kTile; r += 32)
                            if (r >= n_seen || (r >= u0 && r < u1)) {
#pragma unroll
                                for (int blk = 0; blk < D / 64; ++blk)
#pragma unroll
                                    for (int c = 0; c < 8; ++c)
                                        ptx::st_shared_v4(base + blk * kTile * 128 + r * 128 + c * 16, 0, 0, 0, 0);
                            }
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                    }
                    // the first 64 keys' product runs while the rows work on the others' weights
                    const uint64_t dv = dv0 + (uint64_t)ring.st * stage16;
                    if (!(ok = wait(sbar(SB_P_HALF), p_it & 1u))) break;
                    ptx::tc_fence_after();
                    mma_ts_k64(tO, tP, dv, idPV, started ? 1u : 0u);
                    if (!(ok = wait(sbar(SB_P_FULL), p_it & 1u))) break;
                    ++p_it;
                    ptx::tc_fence_after();
                    mma_ts_k64(tO, tP + 32u, dv + 512u, idPV, 1u);
                    started = true;
                    ptx::tc_commit_w(sbar(SB_PV_DONE));
                    ++pv_it;
                    pv_pending = true;
                    ptx::tc_commit_w(empty);
                    // (the other slot may have tiles left, which this warp only passes on)
                    if (t == w.t_last && !(AV && tables)) ptx::tc_commit_w(sbar(SB_O_FULL));
                } else {
                    ptx::mbar_arrive_w(empty);
                }
                ring.next();
            }
        }
        if (!ok) break;
        if (AV) {   // O += beta aV
            if (!(ok = wait(bar(B_KV0 + ring.st), ring.ph))) break;
            const uint32_t empty = bar(B_KV0 + kMaxStages + ring.st);
            if (tables) {
                if (!(ok = wait(sbar(SB_BN_FULL), bn_it & 1u))) break;
                ++bn_it;
                ptx::tc_fence_after();
                const uint64_t da = ptx::sdesc_sw128(sh.base + tp.off_kv + (uint32_t)ring.st * tp.stage_bytes,
                                                     (uint32_t)tp.npad * 128, 1024);
#pragma unroll 1
                for (int kk = 0; kk < tp.npad / 16; ++kk)
                    ptx::tc_mma_ts_w(tO, tB + (uint32_t)(kk * 8), da + (uint64_t)(kk * 16 * 128 >> 4), idPV, 1u);
                ptx::tc_commit_w(sbar(SB_BN_DONE));
                ++bd_it;
                bn_pending = true;
                ptx::tc_commit_w(empty);
                ptx::tc_commit_w(sbar(SB_O_FULL));
            } else {
                ptx::mbar_arrive_w(empty);
            }
            ring.next();
        }
        if (!w.split && slot == 0) {   // slot 1's query tile
            if (!(ok = wait(bar(B_Q_FULL + 1), q_it[1] & 1u))) break;
            ++q_it[1];
            ptx::mbar_arrive_w(bar(B_Q_EMPTY + 1));
        }
    }
    // every MMA issued by this warp completes before TMEM is released
    ptx::tc_commit_w(sbar(SB_DRAIN));
    tc::drain_bar(sbar(SB_DRAIN), 0, sh.limit);
}

// ======================================================================= softmax / epilogue
// the bits below n of 32
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

template <int D, bool AK, bool AV>
__device__ void row_role(const TcParams &tp, const Shared &sh, uint32_t tmem, int slot_in) {
    using T = Tm<D>;
    const Params &p = tp.p;
    const int slot = __shfl_sync(0xffffffffu, slot_in, 0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const int quad = uni(warp & 3);
    const int row = quad * 32 + lane;
    const int tok = row / p.g, hh = row - tok * p.g;   // token within the slot, head within the group
    const int tok_lo = (quad * 32) / p.g, tok_hi = (quad * 32 + 31) / p.g;   // of this warp's rows
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t bars = sh.base + tp.off_bar;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto sbar_of = [&](int s, int which) { return bar(B_SLOT0 + kSlotBars * s + which); };
    auto sbar = [&](int which) { return sbar_of(slot, which); };
    float2 *stat = reinterpret_cast<float2 *>(sh.ptr + tp.off_stat);   // [slot][row] {m, l}
    const float sl2 = p.scale_log2;
    const bool pos_scale = sl2 >= 0.f;
    const int k = p.clip_k, W = tp.W;
    uint32_t s_it = 0, pv_it = 0, x_it = 0, o_it[2] = {0, 0};
    bool ok = true, bad = false;
    // one warp of the slot polls, the others meet it at the slot's named barrier (bad: a wait of
    // this warp's own ran out)
    auto wait_w = [&](uint32_t b, uint32_t parity) -> bool {
        bool r = !bad;
        if (quad == 0) {
            r = r && wait_bar(b, parity, sh, p.err);
            r = __all_sync(0xffffffffu, r ? 1 : 0) != 0;
        }
        return slot_sync(slot, r);
    };
    auto wait_s = [&]() -> bool {
        if (!wait_w(sbar(SB_S_FULL), s_it & 1u)) return false;
        ++s_it;
        ptx::tc_fence_after();
        __syncwarp();
        return true;
    };
    // Inside the tile loop each warp waits for itself (a meeting of the four takes 250 cycles more). A
    // wait that runs out marks the warp; it goes on, and the four leave together at their next meeting.
    auto wait_own = [&](uint32_t b, uint32_t parity) {
        if (!bad) {
            const bool r = wait_bar(b, parity, sh, p.err);
            bad = __all_sync(0xffffffffu, r ? 1 : 0) == 0;
        }
        ptx::tc_fence_after();
        __syncwarp();
    };
    // the warp's arrival, after all its lanes
    auto arrive = [&](uint32_t b) {
        ptx::tc_fence_before();
        __syncwarp();
        ptx::mbar_arrive_w(b);
    };
    auto release_s = [&]() { arrive(sbar(SB_S_EMPTY)); };
    auto wait_pv = [&](uint32_t c) -> bool {
        if (!wait_w(sbar(SB_PV_DONE), c & 1u)) return false;
        ptx::tc_fence_after();
        __syncwarp();
        return true;
    };
    // both slots' rows (a bounded wait like every other, so an abort reaches both)
    auto sync_slots = [&]() -> bool {
        arrive(bar(B_X));
        if (!wait_w(bar(B_X), x_it & 1u)) return false;
        ++x_it;
        ptx::tc_fence_after();
        __syncwarp();
        return true;
    };
    auto wait_o = [&](int s) -> bool {
        if (!wait_w(sbar_of(s, SB_O_FULL), o_it[s] & 1u)) return false;
        ptx::tc_fence_after();
        __syncwarp();
        return true;
    };
    // O *= f (rows of this warp)
    auto scale_o = [&](float f) {
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t r[32];
            ptx::tmem_ld32(lane_base + T::O(slot) + (uint32_t)c0, r);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const float2 v = __fmul2_rn(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), dup(f));
                r[e] = __float_as_uint(v.x);
                r[e + 1] = __float_as_uint(v.y);
            }
            ptx::tmem_st32(lane_base + T::O(slot) + (uint32_t)c0, r);
        }
        ptx::tmem_st_wait();
    };
    Pieces pieces(tp, sh);
    Piece g;
    for (; ok && pieces.next(wait_w, g, ok); arrive(pieces.empty()), ++pieces.it) {
        const SlotWork w = slot_work(tp, g, slot);
        const bool split = w.split;
        const bool act = g.act >> slot & 1;
        const bool two = split && g.t1 - g.t0 > 1;      // the other slot works on the same rows
        const int rows = w.ntok * p.g;                  // may be negative: no rows in this slot
        const bool mine = quad * 32 < rows;             // this warp has rows
        const bool valid = row < rows;
        const int pos = valid ? w.pos_lo + tok : -1;
        const int pmin = uni(w.pos_lo + tok_lo), pmax = uni(min(w.pos_lo + tok_hi, w.pos_hi));
        float *Rrow = reinterpret_cast<float *>(sh.ptr + tp.off_r[split ? 0 : slot]) + row * tp.SR;
        const bool whole = g.whole();
        const int rrow = (split ? 0 : slot * tp.TS * p.g) + row;
        float *rec = whole ? nullptr : record(p, blockIdx.x, g.record());
        __nv_bfloat16 *orow = static_cast<__nv_bfloat16 *>(p.out) +
                              ((long long)(g.row0 + w.tok0 + tok) * p.H + g.kvh * p.g + hh) * D;
        if (g.t1 == g.t0 || (!split && !act)) {   // no key in this piece for any row of the slot
            if (valid && !(split && slot == 1)) {
                if (whole) {
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4 *>(orow)[c] = make_uint4(0, 0, 0, 0);
                } else {
                    rec[rrow] = -INFINITY;
                    rec[p.rec_rows + rrow] = 0.f;
                    for (int c = 0; c < D; c += 2)
                        *reinterpret_cast<float2 *>(rec + 2 * p.rec_rows + (long long)rrow * D + c) = make_float2(0.f, 0.f);
                }
            }
            if (split || g.t1 == g.t0) continue;
            // (pair mode) the other slot may have tiles of its own; nothing is shared with it
            if (slot == 1) o_it[0] += g.act & 1;
            else o_it[1] += g.act >> 1;
            continue;
        }
        if (AK && (!split || slot == 0)) {   // R row -> shared memory (log2 domain)
            if (!(ok = wait_s())) break;
            if (mine)
                for (int c0 = 0; c0 < tp.npad; c0 += 16) {
                    uint32_t r[16];
                    ptx::tmem_ld16(lane_base + T::S(slot) + (uint32_t)c0, r);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (c0 + e < W) Rrow[c0 + e] = __uint_as_float(r[e]) * sl2;
                }
            release_s();
        }
        if (split && !(ok = sync_slots())) break;
        const float c_left = AK && mine ? Rrow[0] : 0.f;
        float m_ref = -INFINITY, l = 0.f;
        uint32_t n = 0;   // tiles of the slot so far

        for (int t = g.t0; t <= w.t_last; ++t) {
            if (!w.uses(p, g, slot, t)) continue;
            const int j0 = g.tile(t) * kTile;
            wait_own(sbar(SB_S_FULL), s_it & 1u);
            ++s_it;
            const bool last = t == w.t_last;
            const bool keep_s = AV && last && (!split || slot == 0);   // beta will lie there
            // chunk of 32 keys from e0: seen by no row of the warp / without masks / beyond the band
            auto dead = [&](int e0) -> bool {
                return e0 > pmax || (p.window > 0 && e0 + KB - 1 <= pmin - p.window && e0 >= p.sinks);
            };
            auto full = [&](int e0, int len) -> bool {
                return e0 + len - 1 <= pmin && (p.window == 0 || e0 > pmax - p.window || e0 + len <= p.sinks);
            };
            auto far = [&](int e0, int len) -> bool { return e0 + len - 1 <= pmin - k; };
            // Most tiles need no mask and lie beyond the band: their scores stay raw in registers (scale
            // and constant go into the exponent) and the code is straight-line. The others take two
            // rolled passes over the score columns, 32 keys at a time, with the logits written back.
            const bool plain = mine && pos_scale && full(j0, kTile) && (!(AK || AV) || far(j0, kTile));
            float x[kTile];
            float rmax = -INFINITY;
            if (plain) {
#pragma unroll
                for (int c = 0; c < NCH; ++c) ptx::tmem_ld32f(lane_base + T::S(slot) + (uint32_t)(c * KB), x + c * KB);
                ptx::tmem_ld_wait();
                if (!keep_s) release_s();
                rmax = fmaxf(fmaxf(max32(x), max32(x + 32)), fmaxf(max32(x + 64), max32(x + 96)));
                rmax = fmaf(rmax, sl2, c_left);
            } else if (mine) {
#pragma unroll 1
                for (int c = 0; c < NCH; ++c) {
                    const int e0 = j0 + c * KB;
                    if (dead(e0)) continue;
                    const uint32_t at = lane_base + T::S(slot) + (uint32_t)(c * KB);
                    float xc[KB];
                    ptx::tmem_ld32f(at, xc);
                    ptx::tmem_ld_wait();
                    const int rb = e0 - pos + k;   // table row of element 0, before clamping
                    const bool band = (AK || AV) && !far(e0, KB);
                    if (AK && band) {
#pragma unroll
                        for (int e = 0; e < KB; e += 2) {
                            const float2 r = make_float2(Rrow[__viaddmin_s32_relu(rb, e, k)], Rrow[__viaddmin_s32_relu(rb, e + 1, k)]);
                            put(xc, e, __ffma2_rn(pair(xc, e), dup(sl2), r));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < KB; e += 2) put(xc, e, __ffma2_rn(pair(xc, e), dup(sl2), dup(c_left)));
                    }
                    if (!full(e0, KB)) {
                        // the keys seen as bits: up to the row's position, and inside the window or first
                        uint32_t seen = below(pos - e0 + 1);
                        if (p.window > 0) seen &= ~below(pos - p.window - e0 + 1) | below(p.sinks - e0);
#pragma unroll
                        for (int e = 0; e < KB; ++e) xc[e] = seen & (1u << e) ? xc[e] : -INFINITY;
                    }
                    if (AV && band) {   // the score takes the place of the table row it used
#pragma unroll
                        for (int e = 0; e < KB; ++e)
                            if ((unsigned)(rb + e - 1) < (unsigned)k) Rrow[rb + e] = xc[e];
                    }
                    rmax = fmaxf(rmax, max32(xc));
                    __syncwarp();
                    ptx::tmem_st32f(at, xc);
                }
                ptx::tmem_st_wait();
            }
            float alpha = 1.f;
            if (rmax > m_ref + kRescaleLog2) {
                alpha = ptx::ex2(m_ref - rmax);
                m_ref = rmax;
            }
            // P and O are free once the previous P V is done (P over S: S_j was issued after it)
            if (!T::P_ALIAS && n > 0) wait_own(sbar(SB_PV_DONE), (pv_it + n - 1u) & 1u);
            if (mine) {
                if (n > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    l *= alpha;
                    __syncwarp();
                    scale_o(alpha);
                }
                const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                // P of 32 keys from logits a xc + b, its sum into l, bf16 pairs (the tensor cores'
                // operand; l keeps the fp32 values) into TMEM
                auto weights = [&](float *xc, float2 a2, float2 b2, int c) {
                    float2 s01 = dup(0.f), s23 = dup(0.f);
#pragma unroll
                    for (int e = 0; e < KB; e += 4) {
                        const float2 t0 = __ffma2_rn(pair(xc, e), a2, b2);
                        const float2 t1 = __ffma2_rn(pair(xc, e + 2), a2, b2);
                        xc[e] = ptx::ex2(t0.x);
                        xc[e + 1] = ptx::ex2(t0.y);
                        xc[e + 2] = ptx::ex2(t1.x);
                        xc[e + 3] = ptx::ex2(t1.y);
                        s01 = __fadd2_rn(s01, pair(xc, e));
                        s23 = __fadd2_rn(s23, pair(xc, e + 2));
                    }
                    l += (s01.x + s01.y) + (s23.x + s23.y);
#pragma unroll
                    for (int e = 0; e < KB / 2; ++e)
                        xc[e] = __uint_as_float(ptx::pack_bf16x2(xc[2 * e], xc[2 * e + 1]));
                    ptx::tmem_st16f(lane_base + T::P(slot) + (uint32_t)(c * (KB / 2)), xc);
                };
                auto half_done = [&]() {
                    ptx::tmem_st_wait();
                    arrive(sbar(SB_P_HALF));
                };
                if (plain) {
                    const float2 a2 = dup(sl2), b2 = dup(c_left - m_use);
#pragma unroll
                    for (int c = 0; c < NCH; ++c) {
                        weights(x + c * KB, a2, b2, c);
                        if (c == NCH / 2 - 1) half_done();
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < NCH; ++c) {
                        float xc[KB];
                        if (dead(j0 + c * KB)) {
#pragma unroll
                            for (int e = 0; e < KB; ++e) xc[e] = -INFINITY;
                        } else {
                            ptx::tmem_ld32f(lane_base + T::S(slot) + (uint32_t)(c * KB), xc);
                            ptx::tmem_ld_wait();
                        }
                        __syncwarp();
                        weights(xc, dup(1.f), dup(-m_use), c);
                        if (c == NCH / 2 - 1) half_done();
                    }
                }
                ptx::tmem_st_wait();
            } else {
                arrive(sbar(SB_P_HALF));
            }
            if (!keep_s && !plain) release_s();
            arrive(sbar(SB_P_FULL));
            ++n;
        }
        pv_it += n;
        // ---- the row's maximum and sum; where the slots shared the rows, of both
        float M = m_ref, f0 = 1.f, f1 = 0.f;
        if (two) {
            stat[slot * BM + row] = make_float2(m_ref, l);
            if (!(ok = sync_slots())) break;
            const float2 other = stat[(1 - slot) * BM + row];
            M = fmaxf(m_ref, other.x);
            const float Mu = M == -INFINITY ? 0.f : M;
            const float fm = ptx::ex2(m_ref - Mu), fo = ptx::ex2(other.x - Mu);
            l = slot == 0 ? fmaf(l, fm, other.y * fo) : fmaf(other.y, fo, l * fm);
            f0 = slot == 0 ? fm : fo;
            f1 = slot == 0 ? fo : fm;
        }
        if (AV) {
            if (!split || slot == 0) {
                if (two) {   // beta joins O of slot 0, which takes the common maximum first
                    if (!(ok = wait_pv(pv_it - 1u))) break;
                    if (mine) scale_o(f0);
                }
                if (mine) {
                    // weights of the band's rows from their scores; row 0 gets the rest of the sum
                    const float Mu = M == -INFINITY ? 0.f : M;
                    const int jb = pos - k;   // key of table row r: jb + r
                    // keys of this piece: s0 .. s1 - 1 of the first tokens, w0 .. w1 - 1 of the window
                    const int s0 = g.t0 * kTile, s1 = min(g.t1, g.ns) * kTile;
                    const int w0 = (max(g.t0, g.ns) - g.ns + g.lo) * kTile, w1 = (g.t1 - g.ns + g.lo) * kTile;
                    const int from = !valid ? 1 << 30 : p.window > 0 ? max(0, pos - p.window + 1) : 0;
                    float band = 0.f;
#pragma unroll 4
                    for (int r = 1; r <= k; ++r) {
                        const int j = jb + r;
                        const bool here = ((j >= w0 && j < w1) || (j >= s0 && j < s1)) &&
                                          (j >= from || (valid && j >= 0 && j < p.sinks));
                        const float b = here ? ptx::ex2(Rrow[r] - Mu) : 0.f;
                        Rrow[r] = b;
                        band += b;
                    }
                    Rrow[0] = fmaxf(0.f, l - band);
                    for (int c0 = 0; c0 < tp.npad; c0 += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int r0 = c0 + 2 * e;
                            pk[e] = ptx::pack_bf16x2(r0 <= k ? Rrow[r0] : 0.f, r0 < k ? Rrow[r0 + 1] : 0.f);
                        }
                        __syncwarp();
                        ptx::tmem_st16(lane_base + T::Bn(slot) + (uint32_t)(c0 / 2), pk);
                    }
                    ptx::tmem_st_wait();
                }
                arrive(sbar(SB_BN_FULL));
                release_s();
            }
            if (two) f0 = 1.f;
        }
        // ---- epilogue
        if (two || slot == 0 || !split) {
            if (!(ok = wait_o(split ? 0 : slot))) break;
            if (two && !(ok = wait_o(1))) break;
            if (mine) {
                const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
                if (valid && !whole && slot == (split ? 0 : slot)) {
                    rec[rrow] = M;
                    rec[p.rec_rows + rrow] = l;
                }
                const uint32_t oA = lane_base + T::O(split ? 0 : slot), oB = lane_base + T::O(1);
                // Rows leave through the slot's R rows (all of its warps are past them): a thread holds a row, but a store of 16
                // bytes per lane should cover 64 bytes of each of 8 rows (one of 16 bytes of 32 rows
                // takes twice the sectors, each half written: 5.5k cycles a tile instead of 2k).
                const uint32_t stage = sh.base + tp.off_r[slot] + (uint32_t)quad * kOutBytes;
                const uint32_t st_at = stage + lane * 64, sw = (lane >> 1) & 3;
                const uint32_t my16 = whole ? (uint32_t)(((long long)tok * p.H + hh) * (D / 8)) : (uint32_t)(rrow * (D / 4));
                char *out0 = whole ? reinterpret_cast<char *>(static_cast<__nv_bfloat16 *>(p.out) +
                                                              ((long long)(g.row0 + w.tok0) * p.H + g.kvh * p.g) * D)
                                   : reinterpret_cast<char *>(rec + 2 * p.rec_rows);
                // 64 bytes of each row, at byte `off` of the row
                auto put64 = [&](const uint32_t *v, int off) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        ptx::st_shared_v4(st_at + ((q ^ sw) << 4), v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int r = 8 * q + (lane >> 2);
                        uint4 o;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                                     : "r"(stage + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4)));
                        const uint32_t at = __shfl_sync(0xffffffffu, my16, r);
                        if (quad * 32 + r < rows)
                            *reinterpret_cast<uint4 *>(out0 + (size_t)at * 16 + off + (lane & 3) * 16) = o;
                    }
                    __syncwarp();
                };
                // each slot writes half of the columns where both hold the rows
                const int cb = two && slot == 1 ? D / 2 : 0, ce = two && slot == 0 ? D / 2 : D;
#pragma unroll 1
                for (int c0 = cb; c0 < ce; c0 += 32) {
                    float r[32];
                    ptx::tmem_ld32f(oA + (uint32_t)c0, r);
                    ptx::tmem_ld_wait();
                    if (two) {
                        float r1[32];
                        ptx::tmem_ld32f(oB + (uint32_t)c0, r1);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            put(r, e, __ffma2_rn(pair(r1, e), dup(f1), __fmul2_rn(pair(r, e), dup(f0))));
                    }
                    uint32_t v[32];
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 o = __fmul2_rn(pair(r, 2 * e), dup(inv));
                            v[e] = ptx::pack_bf16x2(o.x, o.y);
                        }
                        put64(v, 2 * c0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(r[e]);
                        put64(v, 4 * c0);
                        put64(v + 16, 4 * c0 + 64);
                    }
                }
            }
            ptx::tc_fence_before();
        }
        // completions of both slots' O barriers in this piece
        if (split) {
            ++o_it[0];
            if (two) ++o_it[1];
            if (!(ok = sync_slots())) break;   // O, R and the statistics go to the next piece
        } else {
            ++o_it[slot];
            o_it[1 - slot] += g.act >> (1 - slot) & 1;
        }
    }
}

// ======================================================================= kernel
template <int D, bool AK, bool AV>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_ak,
                    const __grid_constant__ CUtensorMap tm_av, const __grid_constant__ TcParams tp) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const Params &p = tp.p;
    Shared sh;
    sh.base = ptx::smem_u32(smem_raw);
    sh.ptr = smem_raw;
    uint64_t *bar_ptr = reinterpret_cast<uint64_t *>(sh.ptr + tp.off_bar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_ptr + kNumBars);
    sh.abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    sh.limit = p.wait_limit;
    const int warp = threadIdx.x >> 5;
    const uint32_t bars = sh.base + tp.off_bar;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t cnt = 1;
            if (i >= B_SLOT0 && i < B_KV0) {
                const int which = (i - B_SLOT0) % kSlotBars;
                if (which == SB_S_EMPTY || which == SB_P_FULL || which == SB_P_HALF || which == SB_BN_FULL) cnt = 4;   // the slot's warps
            }
            if ((i >= B_Q_EMPTY && i < B_X) || i >= B_KV0 + kMaxStages) cnt = 2;     // both MMA warps
            if (i == B_X) cnt = 8;                                                   // both slots' warps
            if (i >= B_PIECE_EMPTY && i < B_PIECE_EMPTY + kPieces) cnt = 3 + 8;      // all but warp 3
            ptx::mbar_init(bars + 8u * (uint32_t)i, cnt);
        }
        *sh.abort_flag = 0;
        ptx::mbar_init_fence();
        ptx::tma_prefetch_desc(&tm_q);
        ptx::tma_prefetch_desc(&tm_k);
        ptx::tma_prefetch_desc(&tm_v);
    }
    // Before the warpgroups trade registers (the scan needs more than a control warp keeps), and by
    // every warp alike: the compiler fails to allocate a branch of one warp here.
    Range *range = reinterpret_cast<Range *>(sh.ptr + tp.off_stat);
    grid_wait();
    grid_release();
    {
        // (64 requests at a time: at 128 the cold code costs a short step 0.4 us, at 32 the loop costs a
        // step of 1024 requests 4 us)
        const Range r = find_range_t<int, 2>(p, (int)blockIdx.x, (int)gridDim.x);
        if (threadIdx.x == 96) *range = r;
    }
    if (warp == 1) ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_raw = *tmem_slot;
    const Range rg = *range;
    __syncthreads();   // the rows' statistics go there
    if (warp < tc::kSoftWarp0) {
        ptx::reg_dealloc<tc::kCtrlRegs>();
        if (warp == 0) {
            (void)__shfl_sync(0xffffffffu, tmem_raw, 0);
            kv_role<D, AK, AV>(tp, sh, &tm_k, &tm_v, &tm_ak, &tm_av);
        } else if (warp == 3) {
            (void)__shfl_sync(0xffffffffu, tmem_raw, 0);
            walk_role<D>(tp, rg, sh, &tm_q);
        } else {
            const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_raw, 0);
            mma_role<D, AK, AV>(tp, sh, tmem, warp - 1);
        }
        __syncwarp();
    } else {
        ptx::reg_alloc<tc::kSoftRegs>();
        const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_raw, 0);
        row_role<D, AK, AV>(tp, sh, tmem, (warp - tc::kSoftWarp0) >> 2);
    }
    ptx::tc_fence_before();
    ptx::cta_barrier();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_raw, 512);
    }
}

// ======================================================================= host
// Shared memory for items of two tiles (wide) or one; false when fewer than `min_stages` stages
// of the ring fit.
template <int D>
bool layout(TcParams *tp, bool wide, int smem_optin, int min_stages) {
    uint32_t off = 0;
    for (int s = 0; s < 2; ++s) {
        tp->off_q[s] = off;
        if (s == 0 || wide) off += (uint32_t)BM * D * 2;
    }
    tp->off_kv = off;
    // R rows of each slot, through which its output rows leave too; slots that share their rows use
    // slot 0's R, so the statistics that they exchange lie in the last of slot 1's where there is room
    // behind the output's staging
    const uint32_t r_bytes = (uint32_t)BM * tp->SR * 4;
    const uint32_t r1_bytes = wide ? r_bytes : 4 * kOutBytes;
    const bool stat_in_r = wide && r_bytes >= 4 * kOutBytes + kStatBytes;
    const uint32_t stat_bytes = stat_in_r ? 0 : kStatBytes;
    const uint32_t fixed = off + r_bytes + r1_bytes + stat_bytes + kPieces * sizeof(Piece) + kNumBars * 8 + 16;
    tp->stage_bytes = (uint32_t)kTile * D * 2;
    if ((int)fixed > smem_optin) return false;
    int st = (int)((smem_optin - fixed) / tp->stage_bytes);
    if (st > kMaxStages) st = kMaxStages;
    if (st < min_stages) return false;
    tp->stages = st;
    uint32_t rest = off + (uint32_t)st * tp->stage_bytes;
    tp->off_r[0] = rest;
    rest += r_bytes;
    tp->off_r[1] = rest;
    rest += r1_bytes;
    tp->off_stat = stat_in_r ? rest - kStatBytes : rest;
    rest += stat_bytes;
    tp->off_piece = rest;
    rest += kPieces * sizeof(Piece);
    tp->off_bar = rest;
    return true;
}

template <int D, bool AK, bool AV>
cudaError_t launch_variant(const CUtensorMap (&tm)[5], const TcParams &tp, cudaStream_t s) {
    auto kern = paged_tc_kernel<D, AK, AV>;
    const DeviceInfo di = device_info();
    cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kern), di);
    if (e != cudaSuccess) return e;
    {   // the warpgroups' register shares add up only at this count (checked once per device)
        static bool checked[64] = {};
        static std::mutex mu;
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lk(mu);
        if (!checked[dev & 63]) {
            cudaFuncAttributes fa;
            e = cudaFuncGetAttributes(&fa, kern);
            if (e != cudaSuccess) return e;
            if (fa.numRegs != tc::kLaunchRegs) return cudaErrorNotSupported;
            checked[dev & 63] = true;
        }
    }
    const int grid = di.sms < kTcGrid ? di.sms : kTcGrid;
    const uint32_t smem = tp.off_bar + kNumBars * 8 + 16;
    e = launch_early(kern, dim3(grid), kThreads, smem, s, tm[0], tm[1], tm[2], tm[3], tm[4], tp);
    if (e != cudaSuccess) return e;
    return launch_merge(tp.p, grid, true, s);
}

template <int D>
cudaError_t launch_d(const PagedArgs &a, cudaStream_t s) {
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return cudaErrorInvalidDevice;
    TcParams tp;
    std::memset(&tp, 0, sizeof(tp));
    Params &p = tp.p;
    fill_params(a, &p);
    tp.TS = BM / p.g;
    tp.W = a.clip_k + 1;
    tp.npad = (tp.W + 15) / 16 * 16;
    tp.SR = tp.W > 16 ? tp.W : 16;    // room for the output's staging (8 KB); even, so that a warp's gathers along the band (stride SR - 1) hit
    while (tp.SR % 4 != 2) ++tp.SR;   // 32 banks; 2 mod 4, so that its column walks hit 16
    tp.box = a.page_size < kTile ? a.page_size : kTile;
    // two tiles per item where that leaves a ring of two stages, else one
    const bool wide = layout<D>(&tp, true, di.smem_optin, 2);
    if (!wide && !layout<D>(&tp, false, di.smem_optin, 2)) return cudaErrorNotSupported;
    p.T = wide ? 2 * tp.TS : tp.TS;
    p.T1 = tp.TS;
    // Measured (prompts, mixed steps, windows): a tile of both slots counts 4, one of a slot's rows
    // alone 3, an item 10. With 5 : 6 : 16 a mixed step takes 117 us in place of 114, with 1 : 1 : 3 122;
    // with 3 : 4 : 8 four prompts 298 us in place of 295.
    p.c0 = 10;
    p.wt = 3;
    p.wt2 = 4;
    p.rec_rows = 2 * BM;
    if (line_is_long(p)) return cudaErrorNotSupported;
    p.likely_rows = likely_rows(a, p.T, p.g);
    CUtensorMap tm[5];
    if (!make_query_map(&tm[0], a, p.g, tp.TS) || !make_page_map(&tm[1], a.k_pages, a, tp.box) ||
        !make_page_map(&tm[2], a.v_pages, a, tp.box))
        return cudaErrorInvalidValue;
    tm[3] = tm[4] = tm[0];
    const uint64_t Ht = a.ths ? (uint64_t)a.Hkv : 1, hs = a.ths ? (uint64_t)a.ths * 2 : (uint64_t)(2 * a.clip_k + 1) * D * 2;
    if (a.aK && !tc::make_map(&tm[3], a.aK, D, tp.W, Ht, D * 2, hs, (uint32_t)tp.npad)) return cudaErrorInvalidValue;
    if (a.aV && !tc::make_map(&tm[4], a.aV, D, tp.W, Ht, D * 2, hs, (uint32_t)tp.npad)) return cudaErrorInvalidValue;
    if (a.aK && a.aV) return launch_variant<D, true, true>(tm, tp, s);
    if (a.aK) return launch_variant<D, true, false>(tm, tp, s);
    if (a.aV) return launch_variant<D, false, true>(tm, tp, s);
    return launch_variant<D, false, false>(tm, tp, s);
}

}  // namespace
}  // namespace paged

bool paged_tc_covers(const PagedArgs &a) {
    // (a row's place among an item's outputs is counted in 16-byte units, in 32 bits)
    return a.clip_k <= 127 && a.H <= 1 << 20 && paged::pages_by_tma(a);
}

cudaError_t launch_paged_tc(const PagedArgs &a, cudaStream_t s) {
    return a.d == 64 ? paged::launch_d<64>(a, s) : paged::launch_d<128>(a, s);
}

}  // namespace relattn
