// What the paged attention kernels share: the parameters, the split of the work over the CTAs,
// and the records that the merge kernel joins.
//
// Work. An item is a run of T consecutive new tokens of one request with one key/value head: its
// query rows are the tokens' g = H / Hkv query heads, row r = (token r / g, head r % g), so that
// the heads that share keys share their loads. Its keys come in tiles of kTile: the tiles that
// hold first tokens (sinks) and the tiles from the window's start to the last token's position.
// The requests differ in length by orders of magnitude and nothing about them is known on the
// host, so the items' costs (c0 + wt per tile) are laid end to end in (request, key/value head,
// token) order and cut into one equal range per CTA; each CTA finds its range's start by a scan
// over the requests and walks on from there. An item that lies in several ranges is computed in
// pieces: each piece writes its rows' maximum, sum and unnormalised output to the workspace and
// a second kernel joins them in the order of their keys, so results do not depend on timing.
// A CTA has at most two such pieces: the end of an item that began before its range (record 0)
// and the beginning of one that goes on behind it (record 1).
#pragma once

#include <cstdint>
#include <type_traits>
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
    int n;             // pieces, in the CTAs c .. c + n - 1; 0: some of the CTAs from c on may have none
    long long x;       // position of the item's start in the cost line
    long long total;   // length of the cost line
    long long pad2[2];
};
static_assert(sizeof(Desc) == 64, "descriptor");

// Params are those of a plain call, PartParams those of a part of a call whose requests share prefixes
// (relattn_paged_shared.cu). The kernels are compiled for either: what only parts have costs plain calls registers and
// cold code otherwise (four prompts of 4096, key term 284 -> 295 us, 128 windows of 1024 33.1 -> 34.8).
struct Params {
    const void *q, *k, *v, *aK, *aV;
    long long q_stride, page_stride, bt_stride, ths;
    const int *bt, *q_start, *kv_len;
    int num_pages, pshift, cap;   // cap: keys a block table row can hold
    int clip_k, window, sinks;
    float scale_log2;                        // scale * log2(e)
    int B, tokens, H, Hkv, g, d;
    int T;                                   // tokens per item
    int c0, wt;                              // cost of an item: c0 + wt * tiles
    int wt2, T1;                             // wt2 in place of wt for items of more than T1 tokens
    int long_line;                           // the cost line may pass 31 bits
    int likely_rows;                         // rows of an item at most, going by max_new
    int rec_rows;                            // rows of a record
    void *out;
    float *lse;                              // [tokens][H] or null
    Desc *desc;                              // [gridDim.x]
    float *part;                             // [gridDim.x][2] records {m[rows], l[rows], O[rows][d]}
    int *err;
    long long wait_limit;
    int withhold;                            // test hook: a CTA's first queries are announced, not loaded
    // what PartParams has, for code that knows either
    static constexpr int step = 1, f32_out = 0, overlap = 0;
    static constexpr const int *first_key = nullptr, *row_of = nullptr, *ctas = nullptr;
    static constexpr int *owner = nullptr;
};
struct PartParams : Params {
    int step;                                // 1; 0: all tokens of a request stand at its last position
    int f32_out;                             // out is fp32 whatever the inputs are
    int overlap;                             // runs beside the kernel in front of it, and ends after it
    const int *first_key;                    // [tokens] or null: first key of the token's request (whole tiles)
    const int *row_of;                       // [B] or null: the request's row of the block table
    const int *ctas;                         // CTAs that share the work (the others have none); null: all
    int *owner;                              // [tokens][Hkv] or null: the CTA that begins a token's item, where
                                             // the item goes on behind its range; else -1 (out has its rows)
    PagedLeft *left;                         // host
};

inline size_t desc_bytes() { return (size_t)kMaxGrid * sizeof(Desc); }

// ------------------------------------------------------------------ requests and items
struct Seq {
    int q0, n;      // first query row and new tokens
    int pos0;       // position of the first new token (negative: fewer keys than new tokens)
    int lo;         // first tile of its keys
};

template <typename PP>
__device__ __forceinline__ Seq load_seq(const PP &p, int b) {
    Seq s;
    s.q0 = min(max(p.q_start[b], 0), p.tokens);
    const int q1 = min(max(p.q_start[b + 1], s.q0), p.tokens);
    s.n = q1 - s.q0;
    s.pos0 = min(max(p.kv_len[b], 0), p.cap) - s.n;
    s.lo = p.first_key && s.n > 0 ? p.first_key[s.q0] / kTile : 0;
    return s;
}

// items of one key/value head
__device__ __forceinline__ int items_of(const Params &p, const Seq &s) {
    return s.n <= p.T ? (s.n > 0 ? 1 : 0) : (s.n + p.T - 1) / p.T;
}

// tiles of an item of cost c0 + wt nt that begin before cost position y of it
__device__ __forceinline__ int tiles_before(long long y, int c0, int wt, int nt) {
    if (y >= c0 + (long long)wt * nt) return nt;
    if (y <= c0) return 0;
    return ((int)y - c0 + wt - 1) / wt;
}

struct Item {
    int i0, cnt;          // first token (within the request) and tokens
    int pos_lo, pos_hi;   // positions of the first and the last token
    int ns, lo, nt;       // tiles: 0 .. ns - 1, then lo .. lo + nt - ns - 1
    int cost, wt;
    __device__ __forceinline__ int tile(int t) const { return t < ns ? t : lo + t - ns; }
    // tiles of the item that lie before cost position y of it
    __device__ __forceinline__ int tile_at(const Params &p, long long y) const {
        return tiles_before(y, p.c0, wt, nt);
    }
};

template <typename PP>
__device__ __forceinline__ Item make_item(const PP &p, const Seq &s, int qt) {
    Item it;
    it.i0 = qt * p.T;
    it.cnt = min(p.T, s.n - it.i0);
    it.pos_lo = p.step ? s.pos0 + it.i0 : s.pos0 + s.n - 1;
    it.pos_hi = p.step ? it.pos_lo + it.cnt - 1 : it.pos_lo;
    it.ns = it.lo = it.nt = 0;
    if (it.pos_hi >= 0) {
        const int first = p.window > 0 ? max(0, max(it.pos_lo, 0) - p.window + 1) : 0;  // first key in the window
        it.lo = max(first / kTile, s.lo);
        it.ns = min((min(p.sinks, first) + kTile - 1) / kTile, it.lo);
        it.nt = max(it.ns + it.pos_hi / kTile + 1 - it.lo, 0);
    }
    it.wt = it.cnt > p.T1 ? p.wt2 : p.wt;
    it.cost = p.c0 + it.wt * it.nt;
    return it;
}

// floor(total * c / G) without overflow
__device__ __forceinline__ int range_begin(int total, int c, int G) {
    const unsigned t = (unsigned)total, g = (unsigned)G, q = t / g, r = t - q * g;
    return (int)(q * c + r * (unsigned)c / g);
}
__device__ __forceinline__ long long range_begin(long long total, int c, int G) {
    if (total < (1LL << 31)) return range_begin((int)total, c, G);
    return total / G * c + total % G * c / G;
}
// CTAs of the launch that take part
template <typename PP>
__device__ __forceinline__ int grid_of(const PP &p, int launched) {
    return p.ctas ? min(max(*p.ctas, 1), launched) : launched;
}

// ------------------------------------------------------------------ a CTA's range
struct Range {
    long long total, x0, x1;   // the cost line and this CTA's part of it
    int b, kvh, qt;            // the item that holds x0
    long long x;               // where that item starts
};

// One warp calls it; every lane returns the range of CTA c of G and the item that holds its first
// position. The lanes take the requests in turn, kBatch of each lane's loaded at once (their latency
// is most of what a small step costs), and add up the items of a request with many of them
// together. I: a type that holds the whole line (32 bits where the host has seen that they do: this
// code runs once, cold, in front of everything else, so every instruction of it counts). Every CTA
// looks at all requests, twice where a batch does not hold them: 13 to 17 us for each 1000 of them.
template <typename I, int kBatch = 4, typename PP>
__device__ __forceinline__ Range find_range_t(const PP &p, int c, int G) {
    constexpr unsigned kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    auto scan = [&](I v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const I u = __shfl_up_sync(kAll, v, o);
            if (lane >= o) v += u;
        }
        return v;
    };
    auto sum = [&](I v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
        return v;
    };
    // cost of one key/value head of requests b0 + 32 i + lane
    auto costs = [&](int b0, I (&cost)[kBatch]) {
        Seq s[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int b = b0 + 32 * i + lane;
            cost[i] = 0;
            s[i] = Seq{0, 0, 0, 0};
            if (b < p.B) s[i] = load_seq(p, b);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (b0 + 32 * i >= p.B) break;
            if (s[i].n > 0 && s[i].n <= p.T) cost[i] = make_item(p, s[i], 0).cost;
            unsigned todo = __ballot_sync(kAll, s[i].n > p.T);
            while (todo) {
                const int src = __ffs(todo) - 1;
                todo &= todo - 1;
                Seq t;
                t.q0 = 0;
                t.n = __shfl_sync(kAll, s[i].n, src);
                t.pos0 = __shfl_sync(kAll, s[i].pos0, src);
                t.lo = __shfl_sync(kAll, s[i].lo, src);
                const int m = items_of(p, t);
                I part = 0;
                for (int q = lane; q < m; q += 32) part += make_item(p, t, q).cost;
                part = sum(part);
                if (lane == src) cost[i] = part;
            }
        }
    };
    I cost[kBatch], total = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32 * kBatch) {
        costs(b0, cost);
        I all = cost[0];
#pragma unroll
        for (int i = 1; i < kBatch; ++i) all += cost[i];
        total += sum(all) * p.Hkv;
    }
    Range r;
    r.total = total;
    r.x0 = range_begin(total, c, G);
    r.x1 = range_begin(total, c + 1, G);
    r.b = p.B;   // an empty range at the end finds no request
    r.kvh = r.qt = 0;
    r.x = r.x1;
    const I x0 = (I)r.x0;
    I at = 0, per = 0, x = 0;
    for (int b0 = 0; b0 < p.B && r.b == p.B && r.x0 < r.x1; b0 += 32 * kBatch) {
        if (p.B > 32 * kBatch) costs(b0, cost);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (b0 + 32 * i >= p.B || r.b != p.B) break;
            const I mine = cost[i] * p.Hkv, incl = at + scan(mine), lo = incl - mine;
            const unsigned hit = __ballot_sync(kAll, lo <= x0 && x0 < incl);
            if (hit) {
                const int src = __ffs(hit) - 1;
                r.b = b0 + 32 * i + src;
                per = __shfl_sync(kAll, cost[i], src);
                x = __shfl_sync(kAll, lo, src);
            }
            at = __shfl_sync(kAll, incl, 31);
        }
    }
    if (r.b == p.B) return r;
    // the head, then the item within it
    // (clamped: offsets that do not ascend give rows to several requests, and the line may then pass
    // what the host has allowed for; what follows stays within the arrays for any numbers)
    r.kvh = min(max((int)((x0 - x) / per), 0), p.Hkv - 1);
    x += per * r.kvh;
    const Seq s = load_seq(p, r.b);
    if (s.n > p.T) {
        const int nq = items_of(p, s);
        for (int i0 = 0; i0 < nq; i0 += 32) {
            const int i = i0 + lane;
            const I cst = i < nq ? make_item(p, s, i).cost : 0;
            const I incl = x + scan(cst);
            const unsigned hit = __ballot_sync(kAll, incl - cst <= x0 && x0 < incl);
            if (hit) {
                const int src = __ffs(hit) - 1;
                r.qt = i0 + src;
                x = __shfl_sync(kAll, incl - cst, src);
                break;
            }
            x = __shfl_sync(kAll, incl, 31);
        }
    }
    r.x = x;
    return r;
}

template <typename PP>
__device__ __forceinline__ Range find_range(const PP &p) {
    const int c = (int)blockIdx.x, G = grid_of(p, (int)gridDim.x);
    return p.long_line ? find_range_t<long long>(p, c, G) : find_range_t<int>(p, c, G);
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

// The first request from b on with new tokens (p.B: none). The lanes of the warp look at 128 requests
// at a time: a batch of fixed slots may have thousands of idle ones in a row, whose loads one after
// the other would be the step's time (three busy slots of 4096 with 20000 keys each, d = 64: 312 us in
// place of 66; of 16384: 1416 and 230, of which 214 are the scan in front).
template <typename PP>
__device__ __forceinline__ int next_busy(const PP &p, int b) {
    const int lane = threadIdx.x & 31;
    for (; b < p.B; b += 128) {
        int n[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = b + 32 * i + lane;
            n[i] = at < p.B ? load_seq(p, at).n : 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned m = __ballot_sync(0xffffffffu, n[i] > 0);
            if (m) return b + 32 * i + __ffs(m) - 1;
        }
    }
    return p.B;
}

// Every lane of a warp holds the same walk and steps it.
struct Walk {
    int b, kvh, qt, nq;
    long long x, x0, x1;
    Seq s;
    template <typename PP>
    __device__ __forceinline__ Walk(const PP &p, const Range &r)
        : b(r.b), kvh(r.kvh), qt(r.qt), nq(0), x(r.x), x0(r.x0), x1(r.x1), s{0, 0, 0, 0} {
        if (b < p.B) {
            s = load_seq(p, b);
            nq = items_of(p, s);
        }
    }
    // the next piece of work of the range; an item without any key comes as one piece with no
    // tiles, in the range where it starts
    template <typename PP>
    __device__ __forceinline__ bool next(const PP &p, Segment &g) {
        while (x < x1 && b < p.B) {
            if (qt >= nq) {
                qt = 0;
                if (++kvh >= p.Hkv) {
                    kvh = 0;
                    if (++b >= p.B) return false;
                    s = load_seq(p, b);
                    if (s.n == 0) {
                        if ((b = next_busy(p, b + 1)) >= p.B) return false;
                        s = load_seq(p, b);
                    }
                    nq = items_of(p, s);
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
};

// A piece as the warp that walks the CTA's range announces it to the others in shared memory (cnt 0:
// there is no more)
struct Piece {
    int row0, cnt;         // first query token, tokens of the item
    int pos_lo, pos_hi;    // their positions
    int ns, lo, nt;        // Item: its tiles
    int t0, t1;            // those of this piece
    int kvh, b;
    int act;               // tcgen05 kernel: bit s: slot s uses a tile of the piece
    __device__ __forceinline__ int tile(int t) const { return t < ns ? t : lo + t - ns; }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == nt; }
    __device__ __forceinline__ int record() const { return t0 > 0 ? 0 : 1; }
    // first key of the window of the item's first token
    __device__ __forceinline__ int first(const Params &p) const {
        return p.window > 0 ? max(0, max(pos_lo, 0) - p.window + 1) : 0;
    }
};
static_assert(sizeof(Piece) == 48, "piece");
constexpr int kPieces = 4;   // announced ahead

template <typename PP>
__device__ __forceinline__ int table_row(const PP &p, int b) { return p.row_of && b < p.B ? p.row_of[b] : b; }

template <typename PP>
__device__ __forceinline__ Piece make_piece(const PP &p, const Segment &g, bool more) {
    return Piece{g.s.q0 + g.it.i0, more ? g.it.cnt : 0, g.it.pos_lo, g.it.pos_hi, g.it.ns, g.it.lo,
                 g.it.nt, g.t0, g.t1, g.kvh, table_row(p, g.b), 0};
}

// Says where the rows of the segment's item are, if it is the item's first (a warp calls it).
template <typename PP>
__device__ __forceinline__ void write_owner(const PP &p, const Segment &g) {
    if (p.owner && g.t0 == 0)
        for (int i = threadIdx.x & 31; i < g.it.cnt; i += 32)
            p.owner[(long long)(g.s.q0 + g.it.i0 + i) * p.Hkv + g.kvh] = g.whole() ? -1 : (int)blockIdx.x;
}

// Leaves the descriptor of the item that goes on behind the range (one thread per CTA calls it,
// once, with the last segment of the range).
template <typename PP>
__device__ __forceinline__ void write_desc(const PP &p, const Segment *g, long long total) {
    Desc d;
    d.valid = 0;
    d.row0 = d.cnt = d.kvh = d.nt = d.c0 = d.wt = d.n = 0;
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
        // A tile belongs to the range that holds its first position. Ranges as long as a tile hold
        // one each, up to the range of the last tile; position y lies in range ((y + 1) G - 1) / total.
        const int G = grid_of(p, (int)gridDim.x);
        if (total / G >= g->it.wt) {
            const long long y = g->x + p.c0 + (long long)g->it.wt * (g->it.nt - 1);
            d.n = (int)min(((y + 1) * G - 1) / total, (long long)G - 1) - (int)blockIdx.x + 1;   // in the grid
        }
    }
    p.desc[blockIdx.x] = d;
}

// a CTA of the launch without a part in the work
template <typename PP>
__device__ __forceinline__ bool idle_cta(const PP &p) {
    if (!p.ctas || (int)blockIdx.x < grid_of(p, (int)gridDim.x)) return false;
    if (threadIdx.x == 0) p.desc[blockIdx.x].valid = 0;
    return true;
}

__device__ __forceinline__ float *record(const Params &p, int c, int which) {
    return p.part + ((long long)c * 2 + which) * p.rec_rows * (p.d + 2);
}

// log-sum-exp of a row from its maximum (log2 domain) and sum
__device__ __forceinline__ float row_lse(float m, float l) {
    return l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
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
// whether the cost line of this launch may pass 31 bits (T, c0, wt, wt2 set)
inline int line_is_long(const Params &p) {
    const double items = ((double)p.tokens / p.T + p.B) * p.Hkv;
    return items * (p.c0 + (double)p.wt2 * (p.cap / kTile + 1)) > 2.0e9;
}
inline int likely_rows(const PagedArgs &a, int T, int g) {
    const int n = a.max_new > 0 && a.max_new < a.tokens ? a.max_new : a.tokens;
    return (n < T ? n : T) * g;
}
// A launch that may begin before the kernel in front of it in the stream has ended: every kernel of
// a paged call runs grid_wait() before it touches what others write or read.
template <typename... Args>
cudaError_t launch_early(void (*kern)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                         std::common_type_t<Args>... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// A kernel's start. With p.overlap it begins when the one in front of it has passed grid_wait() itself, so that what
// stands in front of that one is over, and waits for it at its own end. What those earlier kernels have written
// is seen through the release and the acquire of p.ctas, which the last of them writes at its end.
template <typename PP>
__device__ __forceinline__ void grid_start(const PP &p) {
    if (!p.overlap) {
        grid_wait();
        return;
    }
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p.ctas) : "memory");
    asm volatile("fence.proxy.async.global;" ::: "memory");   // (pages and queries are read by TMA too)
}
// Lets the dependent kernel's CTAs come up beside this one's. After grid_wait(): what stands in front
// of this kernel is then over for the dependent too.
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Fills the parts of Params that do not depend on the kernel.
void fill_params(const PagedArgs &a, Params *p);
void fill_params(const PagedArgs &a, PartParams *p);
// joins the pieces of split items; launched behind the attention kernel as its dependent
cudaError_t launch_merge(const Params &p, int grid, bool bf16, cudaStream_t s);
// leaves a part's pieces to the caller, and says where they are
cudaError_t launch_merge(const PartParams &p, int grid, bool bf16, cudaStream_t s);

}  // namespace paged

}  // namespace relattn
