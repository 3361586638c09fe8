// Paged attention for few query rows per key/value head (generated tokens: T tokens x g heads
// <= 16 rows), bf16, d = 64 or 128, pages of at least 8 keys.
//
// Every cached key and value is read once and meets at most 16 rows, so HBM bounds the kernel:
// 4 d bytes per key against 64 d multiply-adds. The rows are the narrow side (N = 8 or 16) of
// m16n8k16 products whose wide side are the keys (S^T = K Q^T) and the columns (O^T = V^T P^T); a
// 128-row tcgen05 tile would be padding for the most part and would need the keys staged for the
// async proxy, and at these sizes the products take a tenth of the time that the bytes take.
//
// A tile of 128 keys is 16 keys for each of a CTA's 8 row warps; each keeps its own running
// maximum, sum and output over its keys, and the warps are joined once per piece. A ninth warp
// walks the CTA's range, announces the pieces and loads their queries and tiles by TMA (one lane
// per page), so the row warps' loop has no barrier and almost no addresses, and the ring runs ahead
// over the ends of the pieces: joining the warps costs no bandwidth while it is shorter than the
// ring. (Row warps that copied their own keys, by cp.async or by TMA boxes of their own, and walked
// the range themselves took 470 instructions a tile and 7.5 us a piece.)
// The fragments come out of the swizzled rows without bank conflicts and without transposing V:
//   S^T: the order of the contracted columns is free, so lane (key slot l / 4, c = l % 4) takes
//     columns 32 s + 8 c .. + 7 of its keys as the k-slots of two MMA steps, and Q alike;
//   O^T: the lane takes 8 columns of the keys in slots 2 c, 2 c + 1 (+ 8) and pairs two keys by
//     byte permutes; P^T comes out of S^T's accumulators by two 8 x 8 transpositions.
//   Slot i of 8 keys is row perm(i) = 0 4 1 5 2 6 3 7, and dim slot i is the 16-byte chunk perm(i) of
//     64 columns: eight lanes' 16-byte reads then fall in the eight chunks of a 128-byte line.
// Rows of a page that no token sees may hold NaN: their V is replaced by zeros in registers.
// The weights (and the bins of the value term) go into their product in two bf16 parts, so that a
// generated token's are within 2^-16, not within 2^-8 (relattn_decode_fwd's are fp32). The tensor pipe
// is 8 % busy with one product each; the second costs up to 8 rows 0.1 to 0.8 us of 33 to 97 (under
// 1 %), with 16 rows, where the warps' own latency counts, 4 to 6 % (64 requests of 2K - 16K keys, one
// key head of 128: 59.3 -> 62.8 us; with both terms, two key heads of 64: 75.0 -> 79.3).
//
// 64 requests with 2K - 16K keys (8 query heads per key head, d = 128): 96 us, 6.2 TB/s; 32 requests
// with 1K - 2K keys, both terms (16 heads of 64): 41.7 us, 4.7 TB/s; a step with a handful of keys
// takes 6.0 us (scan of the lengths, first loads, two launches), which is what the latter lacks.
//
// Relative terms: R = Q aK^T (k + 1 rows) once per piece by the same MMA; keys at most k - 1
// back add their own R entry and leave their score in a bin; the other keys share entry 0 and
// their weights are summed. At the end of the piece each warp adds 16 rows' beta_r aV_r at a time.
#include <cstdint>

#include <cstring>

#include "relattn_paged_tma.cuh"

namespace relattn {
namespace paged {
namespace {

constexpr int kWarps = 8;                // row warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kRowThreads = 32 * kWarps;
constexpr int kGroup = 16;               // keys of a warp per tile
constexpr int kMaxStages = 4;
static_assert(kWarps * kGroup == kTile, "a tile is one group per warp");

// D = 64 has half the bytes per key: two CTAs share an SM (their joins overlap)
template <int D>
constexpr int kCtasPerSm = D == 64 ? 2 : 1;
template <int D>
constexpr int kStageBytes = 2 * kTile * D * 2;    // one tile: blocks of 64 columns of K, then of V

enum : int { B_FULL = 0, B_EMPTY = kMaxStages, B_PIECE_FULL = 2 * kMaxStages, B_PIECE_EMPTY = B_PIECE_FULL + kPieces,
             kNumBars = B_PIECE_EMPTY + kPieces };

struct Layout {
    uint32_t q, piece, bar, o, ml, R, Bn, bytes;   // byte offsets; the ring comes first
    int lw;
    template <int D, int NT>
    static __host__ __device__ Layout make(int clip_k, bool tables, int stages) {
        Layout L;
        constexpr int rows = 8 * NT;
        L.lw = tables ? (clip_k + 1) | 1 : 0;
        uint32_t off = (uint32_t)stages * kStageBytes<D>;
        L.q = off;     off += kPieces * rows * D * 2;
        L.piece = off; off += kPieces * sizeof(Piece);
        L.bar = off;   off += kNumBars * 8 + 16;
        L.o = off;     off += kWarps * rows * D * 4;
        L.ml = off;    off += kWarps * rows * 4 * 4;
        L.R = off;     off += rows * L.lw * 4;
        L.Bn = off;    off += rows * L.lw * 4;
        L.bytes = off;
        return L;
    }
};
static_assert((kPieces * sizeof(Piece) + kNumBars * 8 + 16) % 16 == 0, "alignment of what follows");

// The joined outputs: 16-byte chunk `ch` of row `row`, swizzled so that the fragments' stores of
// neighbouring rows fall in different banks
template <int D, int NT>
__device__ __forceinline__ int out_at(int warp, int row, int ch) {
    return (warp * 8 * NT + row) * D + ((ch ^ (row & 6)) << 2);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
// D += A B, m16n8k16, bf16 with fp32 accumulation
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// transposes an 8 x 8 matrix of 16-bit elements, lane l holding row l / 4, columns 2 (l % 4), + 1
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// x, y as two pairs of bf16: the rounded values and what the rounding left out
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = ptx::pack_bf16x2(x, y);
    lo = ptx::pack_bf16x2(x - ptx::bf16lo_to_f32(hi), y - __uint_as_float(hi & 0xffff0000u));
}

// row of key slot i of 8 (and chunk of dim slot i)
__device__ __forceinline__ int perm(int i) { return (i >> 1) | ((i & 1) << 2); }

// A wait that runs out sets the status word and the CTA's abort flag; later waits then give up at
// once.
struct Waits {
    volatile int *abort_flag;
    int *err;
    long long limit;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
        if (ptx::mbar_try(bar, parity)) return true;
        return tc::wait_bar_slow_call(bar, parity, abort_flag, err, limit);
    }
};

// ======================================================================= the walking warp
template <int D, int NT, typename PP>
__device__ void feed_role(const PP &p, const Layout &L, uint8_t *smem, const Waits &waits, const CUtensorMap *tm_q,
                          const CUtensorMap *tm_k, const CUtensorMap *tm_v, int stages, int box) {
    constexpr int DB = D / 64;
    const int lane = threadIdx.x & 31;
    const uint32_t base = ptx::smem_u32(smem), bars = base + L.bar;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto wait = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, waits(b, parity) ? 1 : 0) != 0; };
    Piece *ring = reinterpret_cast<Piece *>(smem + L.piece);
    // the boxes of a tile: 128 / box pages (at most 16) x DB blocks of columns, one per lane
    const int nbox = kTile / box, my_box = lane % nbox, my_blk = lane / nbox;
    const uint32_t my_dst = base + my_blk * (kTile * 128) + my_box * box * 128;
    const Range rg = find_range_t<int>(p, (int)blockIdx.x, grid_of(p, (int)gridDim.x));
    Walk walk(p, rg);
    Segment g{};
    uint32_t it = 0, tiles = 0;
    int st = 0;
    uint32_t ph = 0;
    bool more = true, any = false, ok = true;
    while (more && ok) {
        more = walk.next(p, g);
        any = any || more;
        const int i = it & (kPieces - 1);
        if (!(ok = wait(bar(B_PIECE_EMPTY + i), ((it / kPieces) & 1u) ^ 1u))) break;
        if (more) write_owner(p, g);
        if (lane == 0) {
            ring[i] = make_piece(p, g, more);
            if (more) {
                ptx::mbar_expect_tx(bar(B_PIECE_FULL + i), (uint32_t)(p.T * p.g) * D * 2);
#pragma unroll
                for (int blk = 0; blk < DB && !(p.withhold && it == 0); ++blk)
                    ptx::tma_load_3d(base + L.q + (i * DB + blk) * (8 * NT * 128), tm_q, bar(B_PIECE_FULL + i), blk * 64,
                                     g.kvh * p.g, g.s.q0 + g.it.i0);
            } else {
                ptx::mbar_arrive(bar(B_PIECE_FULL + i));
            }
        }
        __syncwarp();
        ++it;
        if (!more) break;
        const int first = p.window > 0 ? max(0, max(g.it.pos_lo, 0) - p.window + 1) : 0;
        const int *bt = p.bt + (long long)table_row(p, g.b) * p.bt_stride;
        // this lane's page of tile t, looked up one tile ahead
        auto lookup = [&](int t, bool &seen) -> int {
            const int j = g.it.tile(t) * kTile + my_box * box;
            seen = t < g.t1 && j <= g.it.pos_hi && (j + box > first || j < p.sinks);
            return seen ? __ldg(bt + (j >> p.pshift)) : -1;
        };
        bool seen_next;
        int pg_next = lookup(g.t0, seen_next);
        for (int t = g.t0; t < g.t1; ++t) {
            const bool seen = seen_next;
            int pg = pg_next;
            pg_next = lookup(t + 1, seen_next);
            if (!(ok = wait(bar(B_EMPTY + st), ph ^ 1u))) break;
            const unsigned m = __ballot_sync(0xffffffffu, seen && my_blk == 0);
            if (lane == 0) ptx::mbar_expect_tx(bar(B_FULL + st), (uint32_t)__popc(m) * box * D * 2 * 2);
            __syncwarp();
            if (seen && my_blk < DB) {
                if ((unsigned)pg >= (unsigned)p.num_pages) {
                    report_page(p);
                    pg = p.num_pages;   // outside the tensor: zeros
                }
                const int row = (g.it.tile(t) * kTile + my_box * box) & ((1 << p.pshift) - 1);
                const uint32_t dst = my_dst + st * kStageBytes<D>;
                tma_load_4d(dst, tm_k, bar(B_FULL + st), my_blk * 64, row, g.kvh, pg);
                tma_load_4d(dst + kStageBytes<D> / 2, tm_v, bar(B_FULL + st), my_blk * 64, row, g.kvh, pg);
            }
            __syncwarp();
            ++tiles;
            if (++st == stages) {
                st = 0;
                ph ^= 1u;
            }
        }
    }
    // no copy is in flight when the CTA exits (they have all been consumed, except after an abort)
    for (uint32_t i = tiles > (uint32_t)stages ? tiles - stages : 0; i < tiles; ++i)
        tc::drain_bar(bar(B_FULL + (int)(i % stages)), (i / stages) & 1u, p.wait_limit);
    for (uint32_t i = it > (uint32_t)kPieces ? it - kPieces : 0; i < it; ++i)
        tc::drain_bar(bar(B_PIECE_FULL + (int)(i & (kPieces - 1))), (i / kPieces) & 1u, p.wait_limit);
    if (lane == 0) write_desc(p, any ? &g : nullptr, rg.total);
}

// ======================================================================= the row warps
template <int D, int NT, bool AK, bool AV, typename PP>
__device__ void row_role(const PP &p, const Layout &L, uint8_t *smem, const Waits &wait, int stages) {
    constexpr int kRows = 8 * NT;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int c = lane & 3, rq = lane >> 2;
    const uint32_t base = ptx::smem_u32(smem), bars = base + L.bar;
    float *so = reinterpret_cast<float *>(smem + L.o);
    float4 *sml = reinterpret_cast<float4 *>(smem + L.ml);   // {m, l, far, -} of [warp][row]
    float *Rs = reinterpret_cast<float *>(smem + L.R), *Bs = reinterpret_cast<float *>(smem + L.Bn);
    const Piece *pieces = reinterpret_cast<const Piece *>(smem + L.piece);
    const int k = p.clip_k, W = k + 1;
    uint32_t stage = 0, phase = 0;
    // this lane's chunks within a block of 64 columns: key rows perm(rq) (+ 8) for S, rows c, c + 4
    // (+ 8) for O; the chunk's place is its number xor (row mod 8)
    const int kr = perm(rq);
    const uint32_t ring = base + warp * (kGroup * 128);
    const uint32_t k_at[2] = {(uint32_t)(kr * 128 + ((c ^ kr) << 4)), (uint32_t)(kr * 128 + (((c + 4) ^ kr) << 4))};
    const uint32_t v_at[2] = {(uint32_t)(c * 128 + ((kr ^ c) << 4)), (uint32_t)((c + 4) * 128 + ((kr ^ (c + 4)) << 4))};
    auto sync = [&]() { ptx::named_bar_sync(1, kRowThreads); };

    for (uint32_t it = 0;; ++it) {
        const int slot = it & (kPieces - 1);
        // all row warps go on together, or leave together; the last piece's shared arrays are free
        const bool ok = wait(bars + 8u * (B_PIECE_FULL + slot), (it / kPieces) & 1u);
        if (!ptx::bar_red_and(1, kRowThreads, ok)) break;
        const Piece g = pieces[slot];
        if (g.cnt == 0) break;
        const int rows = g.cnt * p.g;
        const int pos_lo = g.pos_lo, pos_hi = g.pos_hi, first = g.first(p);
        // ---- Q fragments: lane (row rq, columns 32 s + 8 c .. + 7); positions of rows 2 c, 2 c + 1
        uint4 qf[NT][D / 32];
        int pos[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int s = 0; s < D / 32; ++s)
                qf[n][s] = lds128(base + L.q + (slot * (D / 64) + (s >> 1)) * (kRows * 128) + (8 * n + rq) * 128 +
                                  (((c + 4 * (s & 1)) ^ rq) << 4));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = 8 * n + 2 * c + e;
                pos[n][e] = pos_lo + (rr < rows ? rr / p.g * p.step : 0);
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + 8u * (B_PIECE_EMPTY + slot));
        // products of 16 rows (chunks lo of rows 0-7, hi of rows 8-15) with all query rows
        auto scores = [&](float (&x)[NT][4], const uint4 &lo, const uint4 &hi, int s) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma(x[n], lo.x, hi.x, lo.y, hi.y, qf[n][s].x, qf[n][s].y);
                mma(x[n], lo.z, hi.z, lo.w, hi.w, qf[n][s].z, qf[n][s].w);
            }
        };
        if (AK) {   // R = Q aK^T, 16 table rows at a time
            const __nv_bfloat16 *aK = static_cast<const __nv_bfloat16 *>(p.aK) + (long long)g.kvh * p.ths + 8 * c;
            for (int w0 = 16 * warp; w0 < W; w0 += 16 * kWarps) {
                float x[NT][4] = {};
                uint4 a[2][D / 32];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int s = 0; s < D / 32; ++s)
                        a[h][s] = w0 + rq + 8 * h < W
                                      ? __ldg(reinterpret_cast<const uint4 *>(aK + (long long)(w0 + rq + 8 * h) * D + 32 * s))
                                      : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int s = 0; s < D / 32; ++s) scores(x, a[0][s], a[1][s], s);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int w = w0 + rq + 8 * (e >> 1);
                        if (w < W) Rs[(8 * n + 2 * c + (e & 1)) * L.lw + w] = x[n][e] * p.scale_log2;
                    }
            }
        }
        if (AV)
            for (int i = tid; i < kRows * L.lw; i += kRowThreads) Bs[i] = -INFINITY;
        if (AK || AV) sync();
        float r0[NT][2], m[NT][2], l[NT][2], far[NT][2];
        float o[NT][D / 16][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                r0[n][e] = AK ? Rs[(8 * n + 2 * c + e) * L.lw] : 0.f;
                m[n][e] = -INFINITY;
                l[n][e] = far[n][e] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
        }
        // O^T += A^T (B + Bl) over 16 keys (or table rows): chunks v of rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9
        auto outputs = [&](const uint4 (&v)[4], int u, const uint32_t (&b)[NT][2], const uint32_t (&bl)[NT][2]) {
            const uint32_t *v0 = reinterpret_cast<const uint32_t *>(&v[0]), *v1 = reinterpret_cast<const uint32_t *>(&v[1]);
            const uint32_t *v2 = reinterpret_cast<const uint32_t *>(&v[2]), *v3 = reinterpret_cast<const uint32_t *>(&v[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a0 = __byte_perm(v0[i], v1[i], 0x5410), a1 = __byte_perm(v0[i], v1[i], 0x7632);
                const uint32_t a2 = __byte_perm(v2[i], v3[i], 0x5410), a3 = __byte_perm(v2[i], v3[i], 0x7632);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma(o[n][4 * u + i], a0, a1, a2, a3, b[n][0], b[n][1]);
                    mma(o[n][4 * u + i], a0, a1, a2, a3, bl[n][0], bl[n][1]);
                }
            }
        };

#pragma unroll 1
        for (int t = g.t0; t < g.t1; ++t) {
            const int j0 = g.tile(t) * kTile + warp * kGroup;
            const uint32_t st = ring + stage * kStageBytes<D>;
            const uint32_t empty = bars + 8u * (B_EMPTY + stage);
            wait(bars + 8u * (B_FULL + stage), phase);
            if (++stage == (uint32_t)stages) {
                stage = 0;
                phase ^= 1u;
            }
            __syncwarp();
            float x[NT][4] = {};
#pragma unroll
            for (int s = 0; s < D / 32; ++s) {
                const uint32_t a = st + (s >> 1) * (kTile * 128) + k_at[s & 1];
                scores(x, lds128(a), lds128(a + 1024), s);
            }
            // ---- logits in the log2 domain
            const bool near = j0 + kGroup - 1 > pos_lo - k;   // some key has a table row of its own
            const bool full = j0 + kGroup - 1 <= pos_lo &&
                              (p.window == 0 || j0 > pos_hi - p.window || j0 + kGroup <= p.sinks);
            if (AK && near) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int lab = min(max(j0 + kr + 8 * (e >> 1) - pos[n][e & 1], -k) + k, k);
                        x[n][e] = fmaf(x[n][e], p.scale_log2, Rs[(8 * n + 2 * c + (e & 1)) * L.lw + lab]);
                    }
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] = fmaf(x[n][e], p.scale_log2, r0[n][e & 1]);
            }
            if (!full) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + kr + 8 * (e >> 1), q = pos[n][e & 1];
                        const bool on = j <= q && (p.window == 0 || j > q - p.window || j < p.sinks);
                        x[n][e] = on ? x[n][e] : -INFINITY;
                    }
            }
            // ---- the running maximum of each row: moved only where some lane's scores exceed it
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) grow = grow || fmaxf(x[n][e], x[n][2 + e]) > m[n][e];
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float al[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(x[n][e], x[n][2 + e]);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float mn = fmaxf(m[n][e], mx);
                        al[e] = mn == -INFINITY ? 1.f : ptx::ex2(m[n][e] - mn);
                        m[n][e] = mn;
                        l[n][e] *= al[e];
                        far[n][e] *= al[e];
                    }
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][i][e] *= al[e & 1];
                }
            }
            uint32_t b[NT][2], bl[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float pr[4];
                const float mu[2] = {m[n][0] == -INFINITY ? 0.f : m[n][0], m[n][1] == -INFINITY ? 0.f : m[n][1]};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pr[e] = ptx::ex2(x[n][e] - mu[e & 1]);
                    l[n][e & 1] += pr[e];
                }
                if (AV && near) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int lab = j0 + kr + 8 * (e >> 1) - pos[n][e & 1] + k;
                        if (lab > 0) {
                            if (lab <= k) Bs[(8 * n + 2 * c + (e & 1)) * L.lw + lab] = x[n][e];
                        } else {
                            far[n][e & 1] += pr[e];
                        }
                    }
                } else if (AV) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) far[n][e & 1] += pr[e];
                }
                // P for the tensor cores in two bf16 parts, 16 bits in all; the sums above keep fp32
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    split2(pr[2 * h], pr[2 * h + 1], b[n][h], bl[n][h]);
                    b[n][h] = transpose8(b[n][h]);
                    bl[n][h] = transpose8(bl[n][h]);
                }
            }
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                uint4 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = lds128(st + (D / 64 + u) * (kTile * 128) + (e >> 1) * 1024 + v_at[e & 1]);
                if (!full) {   // rows that no token sees
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + c + 4 * (e & 1) + 8 * (e >> 1);
                        if (!(j <= pos_hi && (j >= first || j < p.sinks))) v[e] = make_uint4(0, 0, 0, 0);
                    }
                }
                outputs(v, u, b, bl);
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty);
        }
        // ---- join the warps: maxima and sums first
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int sh = 4; sh < 32; sh *= 2) {
                    l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], sh);
                    if (AV) far[n][e] += __shfl_xor_sync(0xffffffffu, far[n][e], sh);
                }
                if (rq == 0) sml[warp * kRows + 8 * n + 2 * c + e] = make_float4(m[n][e], l[n][e], far[n][e], 0.f);
            }
        sync();
        auto row_max = [&](int row) {
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w * kRows + row].x);
            return M == -INFINITY ? 0.f : M;
        };
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = ptx::ex2(m[n][e] - row_max(8 * n + 2 * c + e));
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    o[n][i][e] *= f;
                    o[n][i][2 + e] *= f;
                }
            }
        if (AV) {   // 16 rows of the table per warp at a time: beta from the scores in the bins
            const __nv_bfloat16 *aV = static_cast<const __nv_bfloat16 *>(p.aV) + (long long)g.kvh * p.ths + 8 * kr;
            for (int w0 = 16 * warp; w0 < W; w0 += 16 * kWarps) {
                uint4 v[D / 64][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int w = w0 + 2 * c + (e & 1) + 8 * (e >> 1);
#pragma unroll
                    for (int u = 0; u < D / 64; ++u)
                        v[u][e] = w < W ? __ldg(reinterpret_cast<const uint4 *>(aV + (long long)w * D + 64 * u))
                                        : make_uint4(0, 0, 0, 0);
                }
                uint32_t b[NT][2], bl[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int row = 8 * n + rq;
                    const float M = row_max(row);
                    float be[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int w = w0 + 2 * c + (e & 1) + 8 * (e >> 1);
                        be[e] = w < W && w > 0 ? ptx::ex2(Bs[row * L.lw + w] - M) : 0.f;
                        if (w == 0) {
#pragma unroll
                            for (int q = 0; q < kWarps; ++q) {
                                const float4 s = sml[q * kRows + row];
                                be[e] = fmaf(s.z, ptx::ex2(s.x - M), be[e]);
                            }
                        }
                    }
                    split2(be[0], be[1], b[n][0], bl[n][0]);
                    split2(be[2], be[3], b[n][1], bl[n][1]);
                }
#pragma unroll
                for (int u = 0; u < D / 64; ++u) outputs(v[u], u, b, bl);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * n + 2 * c + e;
                if (row < rows) {
#pragma unroll
                    for (int u = 0; u < D / 64; ++u)
#pragma unroll
                        for (int i = 0; i < 4; i += 2)
                            *reinterpret_cast<float4 *>(so + out_at<D, NT>(warp, row, 16 * u + 2 * kr + i / 2)) =
                                make_float4(o[n][4 * u + i][e], o[n][4 * u + i][2 + e], o[n][4 * u + i + 1][e],
                                            o[n][4 * u + i + 1][2 + e]);
                }
            }
        sync();
        const bool whole = g.whole();
        float *rec = whole ? nullptr : record(p, blockIdx.x, g.record());
        // four columns a thread
        for (int i = tid; i < rows * (D / 4); i += kRowThreads) {
            const int row = i / (D / 4), ch = i - row * (D / 4);
            float M = -INFINITY, ls = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w * kRows + row].x);
            const float Mu = M == -INFINITY ? 0.f : M;
            float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 s = sml[w * kRows + row];
                const float4 ow = *reinterpret_cast<const float4 *>(so + out_at<D, NT>(w, row, ch));
                ls = fmaf(ptx::ex2(s.x - Mu), s.y, ls);
                z.x += ow.x;
                z.y += ow.y;
                z.z += ow.z;
                z.w += ow.w;
            }
            if (whole) {
                const float inv = ls > 0.f ? 1.f / ls : 0.f;
                const int tok = row / p.g, hh = row - tok * p.g;
                const long long at = (long long)(g.row0 + tok) * p.H + g.kvh * p.g + hh;
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + at * D + 4 * ch;
                if (p.lse && ch == 0) p.lse[at] = row_lse(M, ls);
                if (p.f32_out)
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at * D + 4 * ch) =
                        make_float4(z.x * inv, z.y * inv, z.z * inv, z.w * inv);
                else
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(ptx::pack_bf16x2(z.x * inv, z.y * inv),
                                                                 ptx::pack_bf16x2(z.z * inv, z.w * inv));
            } else {
                if (ch == 0) {
                    rec[row] = M;
                    rec[p.rec_rows + row] = ls;
                }
                *reinterpret_cast<float4 *>(rec + 2 * p.rec_rows + row * D + 4 * ch) = z;
            }
        }
    }
}

template <int D, int NT, bool AK, bool AV, typename PP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<D>)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PP p, int stages, int box) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const Layout L = Layout::make<D, NT>(p.clip_k, AK || AV, stages);
    const uint32_t bars = ptx::smem_u32(smem) + L.bar;
    Waits waits{reinterpret_cast<volatile int *>(smem + L.bar + kNumBars * 8), p.err, p.wait_limit};
    if (threadIdx.x == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            const bool by_rows = (i >= B_EMPTY && i < B_EMPTY + kMaxStages) || i >= B_PIECE_EMPTY;
            ptx::mbar_init(bars + 8u * (uint32_t)i, by_rows ? kWarps : 1);
        }
        *waits.abort_flag = 0;
        ptx::mbar_init_fence();
        ptx::tma_prefetch_desc(&tm_q);
        ptx::tma_prefetch_desc(&tm_k);
        ptx::tma_prefetch_desc(&tm_v);
    }
    __syncthreads();
    grid_start(p);
    grid_release();
    if (!idle_cta(p)) {
        if (threadIdx.x >= kRowThreads)
            feed_role<D, NT>(p, L, smem, waits, &tm_q, &tm_k, &tm_v, stages, box);
        else
            row_role<D, NT, AK, AV>(p, L, smem, waits, stages);
    }
    if (p.overlap) grid_wait();
}

template <int D, int NT, bool AK, bool AV, typename PP>
cudaError_t launch_variant(const CUtensorMap (&tm)[3], const PP &p, int box, cudaStream_t s) {
    auto kern = paged_decode_kernel<D, NT, AK, AV, PP>;
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return cudaErrorInvalidDevice;
    // as many stages as the CTA's share of the SM's shared memory holds (1 KB per CTA is the
    // system's); two, at the cost of the second CTA, where long tables leave fewer; one at d = 128
    // with 16 rows and clip_k > 131, whose tables leave no room for two at all
    const int share = (di.smem_optin + 1024) / kCtasPerSm<D> - 1024;
    auto bytes = [&](int n) { return (int)Layout::make<D, NT>(p.clip_k, AK || AV, n).bytes; };
    int stages = kMaxStages;
    while (stages > 1 && bytes(stages) > (stages > 2 ? share : di.smem_optin)) --stages;
    const uint32_t smem = Layout::make<D, NT>(p.clip_k, AK || AV, stages).bytes;
    const cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kern), di);
    if (e != cudaSuccess) return e;
    const int want = di.sms * kCtasPerSm<D>;
    const int grid = want < kMaxGrid ? want : kMaxGrid;
    const cudaError_t le = launch_early(kern, dim3(grid), kThreads, smem, s, tm[0], tm[1], tm[2], p, stages, box);
    if (le != cudaSuccess) return le;
    return launch_merge(p, grid, true, s);
}

template <int D, int NT, typename PP>
cudaError_t launch_rows(const PagedArgs &a, cudaStream_t s) {
    PP p;
    fill_params(a, &p);
    p.T = 8 * NT / p.g;
    p.T1 = p.T;
    p.c0 = 1;   // joining the warps costs about a tile's time
    p.wt = p.wt2 = 1;
    p.rec_rows = 8 * NT;
    if (line_is_long(p)) return cudaErrorNotSupported;
    p.likely_rows = likely_rows(a, p.T, p.g);
    CUtensorMap tm[3];
    const int box = a.page_size < kTile ? a.page_size : kTile;
    if (!make_query_map(&tm[0], a, p.g, p.T) || !make_page_map(&tm[1], a.k_pages, a, box) ||
        !make_page_map(&tm[2], a.v_pages, a, box))
        return cudaErrorInvalidValue;
    if (a.aK && a.aV) return launch_variant<D, NT, true, true>(tm, p, box, s);
    if (a.aK) return launch_variant<D, NT, true, false>(tm, p, box, s);
    if (a.aV) return launch_variant<D, NT, false, true>(tm, p, box, s);
    return launch_variant<D, NT, false, false>(tm, p, box, s);
}

template <typename PP>
cudaError_t launch_for(const PagedArgs &a, cudaStream_t s) {
    const bool eight = (long long)a.max_new * (a.H / a.Hkv) <= 8;
    if (a.d == 64) return eight ? launch_rows<64, 1, PP>(a, s) : launch_rows<64, 2, PP>(a, s);
    return eight ? launch_rows<128, 1, PP>(a, s) : launch_rows<128, 2, PP>(a, s);
}

constexpr int kMostRows = 16;

}  // namespace
}  // namespace paged

bool paged_decode_covers(const PagedArgs &a) {
    const int g = a.H / a.Hkv;
    return a.max_new >= 1 && (long long)a.max_new * g <= paged::kMostRows && paged::pages_by_tma(a);
}

cudaError_t launch_paged_decode(const PagedArgs &a, cudaStream_t s) {
    return a.owner ? paged::launch_for<paged::PartParams>(a, s) : paged::launch_for<paged::Params>(a, s);
}

}  // namespace relattn
