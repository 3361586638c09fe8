// What the paged attention kernels share: the parameters, the split of the work over the CTAs,
// and the records that the merge kernel joins.
//
// Work. An item is a run of T consecutive new tokens of one request with one key/value head: its
// query rows are the tokens' g = H / Hkv query heads, row r = (token r / g, head r % g), so that
// the heads that share keys share their loads. Its keys come in tiles of kTile: the tiles that
// hold first tokens (sinks) and the tiles from the window's start to the last token's position.
// The requests differ in length by orders of magnitude and nothing about them is known on the
// host, so the items' costs (c0 + wt tiles) are laid end to end in (request, key/value head,
// token) order and cut into one equal range per CTA; each CTA finds its range's start by a scan
// over the requests and walks on from there. An item that lies in several ranges is computed in
// pieces: each piece writes its rows' maximum, sum and unnormalised output to the workspace and
// a second kernel joins them in the order of their keys, so results do not depend on timing.
// A CTA has at most two such pieces: the end of an item that began before its range (record 0)
// and the beginning of one that goes on behind it (record 1).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "relattn_internal.h"

namespace relattn {
namespace paged {

constexpr int kTile = 128;               // keys per tile
constexpr int kMaxGrid = 320;            // CTAs of one launch at most
constexpr int kRecordRows = 128;         // kMaxGrid * kRecordRows rows bound the records of a launch
constexpr int kInvalidArg = 1;           // RELATTN_ERR_INVALID_ARG in the status word
constexpr float kLog2e = 1.4426950408889634f;

// What CTA c left unfinished at its range's end, for the merge (64 bytes)
struct Desc {
    int valid;         // 0: nothing
    int row0, cnt;     // first query token and tokens of the item
    int kvh, nt;       // key/value head, tiles of the item
    int c0, wt;        // the item's cost: c0 + wt * nt
    int pad;
    long long x;       // position of the item's start in the cost line
    long long total;   // length of the cost line
    long long pad2[2];
};
static_assert(sizeof(Desc) == 64, "descriptor");

struct Params {
    const void *q, *k, *v, *aK, *aV;
    long long q_stride, page_stride, bt_stride, ths;
    const int *bt, *q_start, *kv_len;
    int num_pages, pshift, max_pages, cap;   // cap: keys a block table row can hold
    int clip_k, window, sinks;
    float scale_log2;                        // scale * log2(e)
    int B, tokens, H, Hkv, g, d;
    int T;                                   // tokens per item
    int c0, wt;                              // cost of an item: c0 + wt * tiles
    int wt2, T1;                             // wt2 in place of wt for items of more than T1 tokens
    int rec_rows;                            // rows of a record
    void *out;
    Desc *desc;                              // [gridDim.x]
    float *part;                             // [gridDim.x][2] records {m[rows], l[rows], O[rows][d]}
    int *err;
    long long wait_limit;
};

inline size_t desc_bytes() { return (size_t)kMaxGrid * sizeof(Desc); }

// ------------------------------------------------------------------ requests and items
struct Seq {
    int q0, n;      // first query row and new tokens
    int pos0;       // position of the first new token (negative: fewer keys than new tokens)
};

__device__ __forceinline__ Seq load_seq(const Params &p, int b) {
    Seq s;
    s.q0 = min(max(p.q_start[b], 0), p.tokens);
    const int q1 = min(max(p.q_start[b + 1], s.q0), p.tokens);
    s.n = q1 - s.q0;
    s.pos0 = min(max(p.kv_len[b], 0), p.cap) - s.n;
    return s;
}

struct Item {
    int i0, cnt;          // first token (within the request) and tokens
    int pos_lo, pos_hi;   // positions of the first and the last token
    int ns, lo, nt;       // tiles: 0 .. ns - 1, then lo .. lo + nt - ns - 1
    int cost, wt;
    __device__ __forceinline__ int tile(int t) const { return t < ns ? t : lo + t - ns; }
    // tiles of the item that lie before cost position y of it
    __device__ __forceinline__ int tile_at(const Params &p, long long y) const {
        if (y >= cost) return nt;
        if (y <= p.c0) return 0;
        return (int)((y - p.c0 + wt - 1) / wt);
    }
};

__device__ __forceinline__ Item make_item(const Params &p, const Seq &s, int qt) {
    Item it;
    it.i0 = qt * p.T;
    it.cnt = min(p.T, s.n - it.i0);
    it.pos_lo = s.pos0 + it.i0;
    it.pos_hi = it.pos_lo + it.cnt - 1;
    it.ns = it.lo = it.nt = 0;
    if (it.pos_hi >= 0) {
        const int first = p.window > 0 ? max(0, max(it.pos_lo, 0) - p.window + 1) : 0;  // first key in the window
        it.lo = first / kTile;
        it.ns = min((min(p.sinks, first) + kTile - 1) / kTile, it.lo);
        it.nt = it.ns + it.pos_hi / kTile + 1 - it.lo;
    }
    it.wt = it.cnt > p.T1 ? p.wt2 : p.wt;
    it.cost = p.c0 + it.wt * it.nt;
    return it;
}

__device__ __forceinline__ long long range_begin(long long total, int c, int G) {
    return total / G * c + total % G * c / G;   // floor(total * c / G) without overflow
}

// ------------------------------------------------------------------ a CTA's range
struct Range {
    long long total, x0, x1;   // the cost line and this CTA's part of it
    int b, kvh, qt;            // the item that holds x0
    long long x;               // where that item starts
};

// All threads of the CTA call it; `sm` is scratch of at least 80 8-byte words (freed on return
// after the caller's next __syncthreads). Every thread returns the same range.
template <int THREADS>
__device__ Range find_range(const Params &p, long long *sm) {
    constexpr int W = THREADS / 32;
    static_assert(W <= 32, "warps");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // cost of one key/value head of request b, summed by the warp for the long requests
    auto cost_of = [&](int b) -> long long {
        Seq s{0, 0, 0};
        if (b < p.B) s = load_seq(p, b);
        const int nq = (s.n + p.T - 1) / p.T;
        long long c = 0;
        const bool big = nq > 4;
        if (!big)
            for (int i = 0; i < nq; ++i) c += make_item(p, s, i).cost;
        unsigned todo = __ballot_sync(0xffffffffu, big);
        while (todo) {
            const int src = __ffs(todo) - 1;
            todo &= todo - 1;
            Seq t;
            t.q0 = 0;
            t.n = __shfl_sync(0xffffffffu, s.n, src);
            t.pos0 = __shfl_sync(0xffffffffu, s.pos0, src);
            const int m = (t.n + p.T - 1) / p.T;
            long long part = 0;
            for (int i = lane; i < m; i += 32) part += make_item(p, t, i).cost;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
            if (lane == src) c = part;
        }
        return c;
    };
    auto scan = [&](long long v) -> long long {  // inclusive over the block; the total in sm[32 + W]
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        __syncthreads();
        if (lane == 31) sm[warp] = v;
        __syncthreads();
        if (tid == 0) {
            long long a = 0;
            for (int w = 0; w < W; ++w) {
                sm[32 + w] = a;
                a += sm[w];
            }
            sm[32 + W] = a;
        }
        __syncthreads();
        return v + sm[32 + warp];
    };
    Range r;
    const int G = (int)gridDim.x, c = (int)blockIdx.x;
    long long total = 0;
    const bool once = p.B <= THREADS;
    long long mine = 0, incl = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        mine = cost_of(b0 + tid) * p.Hkv;
        incl = scan(mine);
        total += sm[32 + W];
    }
    r.total = total;
    r.x0 = range_begin(total, c, G);
    r.x1 = range_begin(total, c + 1, G);
    if (tid == 0) sm[70] = p.B;   // an empty range at the end finds no request
    __syncthreads();
    long long carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        if (!once) {
            mine = cost_of(b0 + tid) * p.Hkv;
            incl = scan(mine);
        }
        const long long lo = carry + incl - mine;
        if (mine > 0 && lo <= r.x0 && r.x0 < lo + mine) {
            sm[70] = b0 + tid;
            sm[71] = lo;
            sm[72] = mine / p.Hkv;
        }
        if (!once) carry += sm[32 + W];
    }
    __syncthreads();
    r.b = (int)sm[70];
    r.kvh = r.qt = 0;
    r.x = r.x1;
    if (r.b < p.B) {
        const long long per = sm[72];
        const long long y = r.x0 - sm[71];
        r.kvh = (int)(y / per);
        const long long base = sm[71] + per * r.kvh, z = r.x0 - base;
        if (warp == 0) {  // the item within the head
            const Seq s = load_seq(p, r.b);
            const int nq = (s.n + p.T - 1) / p.T;
            long long at = 0;
            for (int i0 = 0; i0 < nq; i0 += 32) {
                const int i = i0 + lane;
                const long long cst = i < nq ? make_item(p, s, i).cost : 0;
                long long inc = cst;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long u = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += u;
                }
                const long long lo = at + inc - cst;
                const bool hit = cst > 0 && lo <= z && z < lo + cst;
                if (hit) {
                    sm[73] = i;
                    sm[74] = base + lo;
                }
                if (__ballot_sync(0xffffffffu, hit)) break;
                at += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        __syncthreads();
        r.qt = (int)sm[73];
        r.x = sm[74];
    }
    return r;
}

// ------------------------------------------------------------------ the walk over a range
struct Segment {
    int b, kvh;
    Seq s;
    Item it;
    int t0, t1;          // tiles of the item in this piece
    long long x;         // the item's start in the cost line
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == it.nt; }
    __device__ __forceinline__ int record() const { return t0 > 0 ? 0 : 1; }
};

struct Walk {
    int b, kvh, qt, nq;
    long long x, x0, x1;
    Seq s;
    __device__ __forceinline__ Walk(const Params &p, const Range &r)
        : b(r.b), kvh(r.kvh), qt(r.qt), nq(0), x(r.x), x0(r.x0), x1(r.x1), s{0, 0, 0} {
        if (b < p.B) {
            s = load_seq(p, b);
            nq = (s.n + p.T - 1) / p.T;
        }
    }
    // the next piece of work of the range; an item without any key comes as one piece with no
    // tiles, in the range where it starts
    __device__ __forceinline__ bool next(const Params &p, Segment &g) {
        while (x < x1 && b < p.B) {
            if (qt >= nq) {
                qt = 0;
                if (nq == 0 || ++kvh >= p.Hkv) {
                    kvh = 0;
                    if (++b >= p.B) return false;
                    s = load_seq(p, b);
                    nq = (s.n + p.T - 1) / p.T;
                }
                continue;
            }
            g.it = make_item(p, s, qt);
            g.b = b;
            g.kvh = kvh;
            g.s = s;
            g.x = x;
            g.t0 = g.it.tile_at(p, max(0LL, x0 - x));
            g.t1 = g.it.tile_at(p, x1 - x);
            const bool empty = g.it.nt == 0 && x >= x0;
            x += g.it.cost;
            ++qt;
            if (empty || g.t1 > g.t0) return true;
        }
        return false;
    }
    // the same out of line, for a kernel that walks in several places: its loops' code should
    // stay in the instruction cache
    __device__ __noinline__ bool next_call(const Params &p, Segment &g) { return next(p, g); }
};

// Leaves the descriptor of the item that goes on behind the range (one thread per CTA calls it,
// once, with the last segment of the range).
__device__ __forceinline__ void write_desc(const Params &p, const Segment *g, long long total) {
    Desc d;
    d.valid = 0;
    d.row0 = d.cnt = d.kvh = d.nt = d.c0 = d.wt = d.pad = 0;
    d.x = d.total = d.pad2[0] = d.pad2[1] = 0;
    if (g && g->t0 == 0 && g->t1 > 0 && g->t1 < g->it.nt) {
        d.valid = 1;
        d.row0 = g->s.q0 + g->it.i0;
        d.cnt = g->it.cnt;
        d.kvh = g->kvh;
        d.nt = g->it.nt;
        d.c0 = p.c0;
        d.wt = g->it.wt;
        d.x = g->x;
        d.total = total;
    }
    p.desc[blockIdx.x] = d;
}

__device__ __forceinline__ float *record(const Params &p, int c, int which) {
    return p.part + ((long long)c * 2 + which) * p.rec_rows * (p.d + 2);
}

// one status for a page entry outside the cache: its keys and values count as zeros
__device__ __forceinline__ void report_page(const Params &p) { atomicCAS(p.err, 0, kInvalidArg); }

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16(x); }

struct DeviceInfo {
    int sms = 0;
    int smem_optin = 0;   // most dynamic shared memory of one block
};
// of the current device, asked once per device
DeviceInfo device_info();
// lets `kern` use all of it, once per kernel and device
cudaError_t opt_in_smem(const void *kern, const DeviceInfo &di);
// every row of q, the pages, the tables and out starts on a 16-byte boundary
bool wide_rows(const PagedArgs &a);
// Fills the parts of Params that do not depend on the kernel.
void fill_params(const PagedArgs &a, Params *p);
// joins the pieces of split items; launched behind the attention kernel as its dependent
cudaError_t launch_merge(const Params &p, int grid, bool bf16, cudaStream_t s);

}  // namespace paged
}  // namespace relattn
