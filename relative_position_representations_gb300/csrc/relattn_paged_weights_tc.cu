// The attention weight that every cached key gets from more than 16 query rows per key head (prompts,
// chunks, the last tokens of a prompt): bf16, d = 64 or 128, pages of at least 8 keys, clip_k <= 127.
//
// S^T = K Q^T on tcgen05 with the keys as the 128 rows of the accumulator: a thread has one key and adds
// up its weights over the columns, the query rows, so nothing crosses threads and nothing but the sums
// leaves the SM. A unit is two tiles of keys of one head, which stay in shared memory while the
// request's query tiles pass by; each of them meets both. Units are taken by ticket, longest first
// within a head (the first keys of a prompt are seen by every row).
// A row's constant nl (the table term of far keys less the log-sum-exp) is formed in front and
// lies in shared memory beside its query tile, so a weight is one FMA and one exponential. Where some key of
// a unit is less than clip_k back, R = Q aK^T is one product more of the query tile, its accumulator
// drained into shared memory by the first tile's threads (a row each).
//
// Roles (384 threads, one CTA per SM): warp 3 takes tickets and announces units, warp 0 loads keys, tables and
// query tiles, warp 2 the rows' constants, warp 1 issues the MMAs, warps 4-7 and 8-11 sum the unit's
// first and second tile. TMEM: two accumulators of 128 columns for each tile.
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

constexpr int kThreads = 384;
constexpr int kRowThreads = 256;
constexpr int KB = 32;               // columns read from an accumulator at a time
constexpr int kUnits = 4;            // announced ahead
constexpr int kMaxK = 4, kMaxQ = 4;  // stages

enum : int {
    B_K_FULL = 0, B_K_EMPTY = B_K_FULL + kMaxK, B_Q_FULL = B_K_EMPTY + kMaxK, B_Q_EMPTY = B_Q_FULL + kMaxQ,
    B_AK_FULL = B_Q_EMPTY + kMaxQ, B_AK_EMPTY, B_UNIT_FULL, B_UNIT_EMPTY = B_UNIT_FULL + kUnits,
    B_ACC_FULL = B_UNIT_EMPTY + kUnits, B_ACC_EMPTY = B_ACC_FULL + 4, B_DRAIN = B_ACC_EMPTY + 4, kNumBars
};

struct Unit {
    int row0, n, pos0;   // first query token of the request, its new tokens, position of the first
    int b, kvh;
    int j0, j1;          // first keys of the tiles (j1 < 0: one tile only)
    int qa, qb;          // query tiles
    int band;            // some row may be less than clip_k past some key
    int more, pad;
};
static_assert(sizeof(Unit) == 48, "unit");

struct TcParams {
    WeightParams w;
    int TS;              // tokens of a query tile
    int npad, SR;        // table rows rounded up to 16; row stride (floats) of R in shared memory
    int box;             // keys per TMA box
    int nk, nq;          // stages of keys and of query tiles
    uint32_t tile_bytes, off_q, off_ak, off_r, off_nl, off_unit, off_bar;
};

// what a query tile is to a unit, the same for every role
struct QueryTile {
    int tok0, ntok, pos_lo, pos_hi;
    bool band;
};
__device__ __forceinline__ QueryTile query_tile(const TcParams &tp, const Unit &u, int q) {
    QueryTile t;
    t.tok0 = q * tp.TS;
    t.ntok = min(tp.TS, u.n - t.tok0);
    t.pos_lo = u.pos0 + t.tok0;
    t.pos_hi = t.pos_lo + t.ntok - 1;
    auto near = [&](int j) { return j >= 0 && j + kTile - 1 > t.pos_lo - tp.w.p.clip_k && j <= t.pos_hi; };
    t.band = u.band && (near(u.j0) || near(u.j1));
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
        return Unit{uni(s.row0), uni(s.n),  uni(s.pos0), uni(s.b),    uni(s.kvh),  uni(s.j0),
                    uni(s.j1),   uni(s.qa), uni(s.qb),   uni(s.band), uni(s.more), 0};
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
    for (;;) {
        unsigned long long t = 0;
        if (lane == 0) t = atomicAdd(tp.w.ticket, 1ull);
        t = __shfl_sync(0xffffffffu, t, 0);
        Unit u{};
        if ((long long)t < total) {
            long long rest;
            u.b = tp.w.busy[find_unit(tp.w, count, (long long)t, rest)];
            const Seq s = load_seq(p, u.b);
            const Item it = make_item(p, s, 0);
            const int per = (it.nt + 1) / 2;
            u.kvh = min((int)(rest / per), p.Hkv - 1);
            const int a = 2 * (int)(rest - (long long)u.kvh * per);
            u.row0 = s.q0;
            u.n = s.n;
            u.pos0 = s.pos0;
            u.j0 = it.tile(a) * kTile;
            u.j1 = a + 1 < it.nt ? it.tile(a + 1) * kTile : -1;
            int lo = first_token(u.j0, s.pos0), hi = end_token(p, u.j0, kTile, s.pos0, s.n);
            if (u.j1 >= 0) {
                lo = min(lo, first_token(u.j1, s.pos0));
                hi = max(hi, end_token(p, u.j1, kTile, s.pos0, s.n));
            }
            u.qa = lo / tp.TS;
            u.qb = (hi + tp.TS - 1) / tp.TS;
            u.band = AK && p.clip_k > 0 && max(u.j0, u.j1) + kTile - 1 > s.pos0 + u.qa * tp.TS - p.clip_k;
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
    Ring kr(tp.nk), qr(tp.nq);
    uint32_t ak_it = 0, k_count = 0, q_count = 0;
    bool ok = true;
    for (; ok; ++units.it) {
        if (!(ok = wait(units.full(), units.parity()))) break;
        const Unit u = units.get();
        if (!u.more) break;
        const int *bt = p.bt + (long long)u.b * p.bt_stride;
        const int pos_hi = u.pos0 + u.n - 1;
        const int first = p.window > 0 ? max(0, max(u.pos0, 0) - p.window + 1) : 0;
        for (int s = 0; s < 2 && ok; ++s) {
            const int j0 = s ? u.j1 : u.j0;
            if (j0 < 0) break;
            const int j = j0 + my_box * tp.box;
            const bool seen = j <= pos_hi && (j + tp.box > first || j < p.sinks);
            int pg = seen ? __ldg(bt + (j >> p.pshift)) : -1;
            if (!(ok = wait(bar(B_K_EMPTY + kr.st), kr.ph ^ 1u))) break;
            const unsigned m = __ballot_sync(0xffffffffu, seen && my_blk == 0);
            ptx::mbar_expect_tx_w(bar(B_K_FULL + kr.st), (uint32_t)__popc(m) * tp.box * D * 2);
            __syncwarp();
            if (seen && my_blk < DB) {
                if ((unsigned)pg >= (unsigned)p.num_pages) {
                    report_page(p);
                    pg = p.num_pages;   // a box outside the tensor: zeros
                }
                tma_load_4d(sh.base + (uint32_t)kr.st * tp.tile_bytes + my_blk * kTile * 128 + my_box * tp.box * 128, tm_k,
                            bar(B_K_FULL + kr.st), my_blk * 64, j & ((1 << p.pshift) - 1), u.kvh, pg);
            }
            __syncwarp();
            kr.next();
            ++k_count;
        }
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
        if (ok) ptx::mbar_arrive_w(units.empty());
    }
    // no copy is in flight when the CTA exits
    for (uint32_t i = k_count > (uint32_t)tp.nk ? k_count - tp.nk : 0; i < k_count; ++i)
        tc::drain_bar(bar(B_K_FULL + (int)(i % tp.nk)), (i / tp.nk) & 1u, sh.limit);
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
    Ring qr(tp.nq);
    for (bool ok = true; ok; ++units.it) {
        if (!(ok = wait(units.full(), units.parity()))) break;
        const Unit u = units.get();
        if (!u.more) break;
        for (int q = u.qa; q < u.qb; ++q) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = tok[e] < u.n - q * tp.TS
                           ? __ldg(tp.w.nl + (long long)(u.row0 + q * tp.TS + tok[e]) * p.H + u.kvh * p.g + head[e])
                           : -INFINITY;
            if (!(ok = wait(bar(B_Q_EMPTY + qr.st), qr.ph ^ 1u))) break;
            float4 *dst = reinterpret_cast<float4 *>(sh.ptr + tp.off_nl + qr.st * BM * 4);
            dst[lane] = make_float4(v[0], v[1], v[2], v[3]);
            __syncwarp();
            ptx::mbar_arrive_w(bar(B_Q_FULL + qr.st));
            qr.next();
        }
        if (ok) ptx::mbar_arrive_w(units.empty());
    }
}

// ======================================================================= MMAs
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
    uint32_t cnt[2] = {0, 0}, ak_it = 0;
    bool ok = true;
    // the next accumulator of tile s
    auto claim = [&](int s) -> bool {
        const uint32_t c = cnt[s];
        if (!wait(bar(B_ACC_EMPTY + 2 * s + (int)(c & 1u)), ((c >> 1) & 1u) ^ 1u)) return false;
        ptx::tc_fence_after();
        return true;
    };
    for (; ok; ++units.it) {
        if (!(ok = wait(units.full(), units.parity()))) break;
        const Unit u = units.get();
        if (!u.more) break;
        const int tiles = u.j1 >= 0 ? 2 : 1;
        int kst[2];
        for (int s = 0; s < tiles && ok; ++s) {
            kst[s] = kr.st;
            ok = wait(bar(B_K_FULL + kr.st), kr.ph);
            kr.next();
        }
        if (ok && AK && u.band) ok = wait(bar(B_AK_FULL), ak_it++ & 1u);
        for (int q = u.qa; q < u.qb && ok; ++q) {
            if (!(ok = wait(bar(B_Q_FULL + qr.st), qr.ph))) break;
            ptx::tc_fence_after();
            const uint64_t dq = dq0 + (uint64_t)qr.st * tile16;
            if (AK && query_tile(tp, u, q).band) {
                if (!(ok = claim(0))) break;
                const uint32_t acc = tmem + (cnt[0] & 1u) * kTile;
#pragma unroll 1
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t at_q = (uint64_t)(((kk >> 2) * BM * 128 + (kk & 3) * 32) >> 4);
                    const uint64_t at_a = (uint64_t)(((kk >> 2) * tp.npad * 128 + (kk & 3) * 32) >> 4);
                    ptx::tc_mma_w(acc, dq + at_q, da + at_a, idR, kk > 0 ? 1u : 0u);
                }
                ptx::tc_commit_w(bar(B_ACC_FULL + (int)(cnt[0] & 1u)));
                ++cnt[0];
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s >= tiles) break;
                if (!(ok = claim(s))) break;
                const uint32_t acc = tmem + (2 * s + (cnt[s] & 1u)) * kTile;
                const uint64_t dk = dk0 + (uint64_t)kst[s] * tile16;
                if (D == 128) ptx::tc_mma_ss_k128(acc, dk, dq, idS, 0u);
                else ptx::tc_mma_ss_k64(acc, dk, dq, idS, 0u);
                ptx::tc_commit_w(bar(B_ACC_FULL + 2 * s + (int)(cnt[s] & 1u)));
                ++cnt[s];
            }
            if (!ok) break;
            ptx::tc_commit_w(bar(B_Q_EMPTY + qr.st));
            qr.next();
        }
        if (!ok) break;
        for (int s = 0; s < tiles; ++s) ptx::tc_commit_w(bar(B_K_EMPTY + kst[s]));
        if (AK && u.band) ptx::tc_commit_w(bar(B_AK_EMPTY));
        ptx::mbar_arrive_w(units.empty());
    }
    // every MMA issued by this warp completes before TMEM is released
    ptx::tc_commit_w(bar(B_DRAIN));
    tc::drain_bar(bar(B_DRAIN), 0, sh.limit);
}

// ======================================================================= sums
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

template <int D, bool AK>
__device__ void sum_role(const TcParams &tp, const Shared &sh, uint32_t tmem, int slot_in) {
    const Params &p = tp.w.p;
    const int slot = __shfl_sync(0xffffffffu, slot_in, 0);
    const int lane = threadIdx.x & 31;
    const int quad = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5) & 3, 0);
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t bars = sh.base + tp.off_bar;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    const float sl2 = p.scale_log2;
    const int k = p.clip_k;
    float *Rs = reinterpret_cast<float *>(sh.ptr + tp.off_r);
    uint32_t cnt = 0;
    bool bad = false;
    // a wait that runs out marks the warp; it goes on, and all leave together at the next unit
    auto wait_own = [&](uint32_t b, uint32_t parity) {
        if (!bad) {
            const bool r = wait_bar(b, parity, sh, p.err);
            bad = __all_sync(0xffffffffu, r ? 1 : 0) == 0;
        }
        __syncwarp();
    };
    auto wait_acc = [&]() {
        wait_own(bar(B_ACC_FULL + 2 * slot + (int)(cnt & 1u)), (cnt >> 1) & 1u);
        ptx::tc_fence_after();
    };
    auto release_acc = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        ptx::mbar_arrive_w(bar(B_ACC_EMPTY + 2 * slot + (int)(cnt & 1u)));
        ++cnt;
    };
    Units units(tp, sh);
    Ring qr(tp.nq);
    for (;; ++units.it) {
        wait_own(units.full(), units.parity());
        if (!ptx::bar_red_and(1, kRowThreads, !bad)) break;
        const Unit u = units.get();
        __syncwarp();
        ptx::mbar_arrive_w(units.empty());
        if (!u.more) break;
        const int j0 = slot ? u.j1 : u.j0;
        const bool have = j0 >= 0;
        const int j = j0 + quad * 32 + lane, j_lo = j0 + quad * 32, j_hi = j_lo + 31;
        // where the key's mass is, and what it holds
        float *at = nullptr;
        float old = 0.f;
        {
            const int pos_hi = u.pos0 + u.n - 1, first = p.window > 0 ? max(0, max(u.pos0, 0) - p.window + 1) : 0;
            if (have && j <= pos_hi && (j >= first || j < p.sinks)) {
                const int pg = __ldg(p.bt + (long long)u.b * p.bt_stride + (j >> p.pshift));
                if ((unsigned)pg < (unsigned)p.num_pages) {
                    at = tp.w.mass + (long long)pg * tp.w.mass_stride +
                         (((long long)u.kvh << p.pshift) + (j & ((1 << p.pshift) - 1)));
                    if (tp.w.accumulate && j < u.pos0) old = *at;
                }
            }
        }
        float2 s01 = dup(0.f), s23 = dup(0.f);
        for (int q = u.qa; q < u.qb; ++q) {
            const QueryTile t = query_tile(tp, u, q);
            wait_own(bar(B_Q_FULL + qr.st), qr.ph);   // the constants
            const float *nl = reinterpret_cast<const float *>(sh.ptr + tp.off_nl + qr.st * BM * 4);
            if (AK && t.band) {
                ptx::named_bar_sync(2, kRowThreads);   // the last R has been read
                if (slot == 0) {
                    wait_acc();
                    float *row = Rs + (quad * 32 + lane) * tp.SR;
                    float r0 = 0.f;
                    for (int c0 = 0; c0 < tp.npad; c0 += 16) {
                        uint32_t r[16];
                        ptx::tmem_ld16(lanes + (cnt & 1u) * kTile + (uint32_t)c0, r);
                        ptx::tmem_ld_wait();
                        if (c0 == 0) r0 = __uint_as_float(r[0]);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (c0 + e <= k) row[c0 + e] = (__uint_as_float(r[e]) - r0) * sl2;
                    }
                    release_acc();
                }
                ptx::named_bar_sync(2, kRowThreads);
            }
            if (have) {
                wait_acc();
                const uint32_t acc = lanes + (uint32_t)(2 * slot + (cnt & 1u)) * kTile;
                const bool far = !AK || k == 0 || j_hi <= t.pos_lo - k;   // else the tile is a band tile: R is there
                const bool full = t.ntok == tp.TS && j_hi <= t.pos_lo &&
                                  (p.window == 0 || j_lo > t.pos_hi - p.window || j_hi < p.sinks);
                const bool dead = j_lo > t.pos_hi || (p.window > 0 && j_hi <= t.pos_lo - p.window && j_lo >= p.sinks);
                // weights of 32 columns, their logits a x + nl
                auto weights = [&](float *x, int c) {
                    const float4 *n4 = reinterpret_cast<const float4 *>(nl + c);
#pragma unroll
                    for (int e = 0; e < KB; e += 4) {
                        const float4 n = n4[e / 4];
                        const float2 a = __ffma2_rn(pair(x, e), dup(sl2), make_float2(n.x, n.y));
                        const float2 b = __ffma2_rn(pair(x, e + 2), dup(sl2), make_float2(n.z, n.w));
                        x[e] = ptx::ex2(a.x);
                        x[e + 1] = ptx::ex2(a.y);
                        x[e + 2] = ptx::ex2(b.x);
                        x[e + 3] = ptx::ex2(b.y);
                    }
                };
                auto add = [&](const float *x) {
#pragma unroll
                    for (int e = 0; e < KB; e += 4) {
                        s01 = __fadd2_rn(s01, make_float2(x[e], x[e + 1]));
                        s23 = __fadd2_rn(s23, make_float2(x[e + 2], x[e + 3]));
                    }
                };
                if (full && far) {
                    float x[2][KB];
                    ptx::tmem_ld32f(acc, x[0]);
#pragma unroll
                    for (int c = 0; c < kTile / KB; ++c) {
                        ptx::tmem_ld_wait();
                        if (c + 1 < kTile / KB) ptx::tmem_ld32f(acc + (uint32_t)((c + 1) * KB), x[(c + 1) & 1]);
                        else release_acc();
                        weights(x[c & 1], c * KB);
                        add(x[c & 1]);
                    }
                } else if (!dead) {
                    // the columns that see this key: tokens from its own on, as far as the window reaches
                    const int rows = t.ntok * p.g, c_lo = max(0, j - t.pos_lo) * p.g;
                    int c_hi = rows;
                    if (p.window > 0 && j >= p.sinks)
                        c_hi = (int)max(0LL, min((long long)rows, ((long long)j + p.window - t.pos_lo) * p.g));
#pragma unroll 1
                    for (int c = 0; c < kTile; c += KB) {
                        float x[KB];
                        ptx::tmem_ld32f(acc + (uint32_t)c, x);
                        ptx::tmem_ld_wait();
                        if (!far) {
                            int tok = c / p.g, hh = c - tok * p.g;
#pragma unroll
                            for (int e = 0; e < KB; ++e) {
                                const int lab = min(max(j - t.pos_lo - tok + k, 0), k);
                                x[e] = fmaf(x[e], sl2, nl[c + e] + Rs[(c + e) * tp.SR + lab]);
                                if (++hh == p.g) {
                                    hh = 0;
                                    ++tok;
                                }
                            }
#pragma unroll
                            for (int e = 0; e < KB; ++e) x[e] = ptx::ex2(x[e]);
                        } else {
                            weights(x, c);
                        }
                        const uint32_t on = below(c_hi - c) & ~below(c_lo - c);
#pragma unroll
                        for (int e = 0; e < KB; ++e) x[e] = on & (1u << e) ? x[e] : 0.f;
                        add(x);
                        __syncwarp();
                    }
                    release_acc();
                } else {
                    release_acc();
                }
            }
            __syncwarp();
            ptx::mbar_arrive_w(bar(B_Q_EMPTY + qr.st));
            qr.next();
        }
        if (at) *at = old + ((s01.x + s01.y) + (s23.x + s23.y));
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
            if (i >= B_Q_FULL && i < B_Q_EMPTY) n = 2;                         // the copy and the constants
            if (i >= B_Q_EMPTY && i < B_AK_FULL) n = 1 + kRowThreads / 32;     // the MMAs and the sums
            if (i >= B_UNIT_EMPTY && i < B_ACC_FULL) n = 3 + kRowThreads / 32;
            if (i >= B_ACC_EMPTY && i < B_DRAIN) n = 4;
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
    if (warp == 0) load_role<D, AK>(tp, sh, &tm_q, &tm_k, &tm_ak);
    else if (warp == 1) mma_role<D, AK>(tp, sh, tmem);
    else if (warp == 2) const_role(tp, sh);
    else if (warp == 3) ticket_role<AK>(tp, sh);
    else sum_role<D, AK>(tp, sh, tmem, (warp - 4) >> 2);
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
    tp.npad = (p.clip_k + 1 + 15) / 16 * 16;
    tp.SR = (p.clip_k + 1) | 1;   // a column walk of R hits 32 banks
    tp.box = a.page_size < kTile ? a.page_size : kTile;
    tp.tile_bytes = (uint32_t)kTile * D * 2;
    const uint32_t ak_bytes = ak && p.clip_k ? (uint32_t)tp.npad * D * 2 : 0, r_bytes = ak && p.clip_k ? BM * tp.SR * 4 : 0;
    const uint32_t rest = (r_bytes + 15) / 16 * 16 + kMaxQ * BM * 4 + kUnits * sizeof(Unit) + kNumBars * 8 + 16;
    // two tiles of keys at least, more query tiles than key tiles
    int stages = (int)(((uint32_t)di.smem_optin - rest - ak_bytes) / tp.tile_bytes);
    if (stages > kMaxK + kMaxQ) stages = kMaxK + kMaxQ;
    if (stages < 4) return cudaErrorNotSupported;
    tp.nk = stages / 2;
    tp.nq = stages - tp.nk;
    tp.off_q = tp.nk * tp.tile_bytes;
    tp.off_ak = tp.off_q + tp.nq * tp.tile_bytes;
    tp.off_nl = tp.off_ak + ak_bytes;
    tp.off_unit = tp.off_nl + kMaxQ * BM * 4;
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
    cudaError_t e = launch_weights_prep(w, true, s);
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
