// The attention weight that every cached key gets from the new tokens: the kernel for generated
// tokens, the SIMT kernel for every type and shape, and the set-up for tickets.
#include <cstdint>
#include <cstring>

#include "relattn_paged_tma.cuh"
#include "relattn_paged_weights.cuh"

namespace relattn {
namespace paged {
namespace {

// ======================================================================= set-up
// nl, 16 lanes to a row, four rows at a time; the last block lists the units of the requests with new
// tokens. Reads q once where there are tables.
constexpr int kPrepThreads = 256;
constexpr int kPrepRows = kPrepThreads / 16 * 4;

template <typename T, int E>
__device__ __forceinline__ float dot(const T *a, const T *b) {
    if (E == 1) return to_f(a[0]) * to_f(b[0]);
    const uint4 x = *reinterpret_cast<const uint4 *>(a), y = *reinterpret_cast<const uint4 *>(b);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (sizeof(T) == 4) {
            s = fmaf(__uint_as_float(xs[i]), __uint_as_float(ys[i]), s);
        } else {
            s = fmaf(ptx::bf16lo_to_f32(xs[i]), ptx::bf16lo_to_f32(ys[i]), s);
            s = fmaf(ptx::bf16hi_to_f32(xs[i]), ptx::bf16hi_to_f32(ys[i]), s);
        }
    }
    return s;
}

// E: elements of a 16-byte load, or 1
template <typename T, int E>
__global__ void __launch_bounds__(kPrepThreads) weights_prep_kernel(const __grid_constant__ WeightParams w) {
    const Params &p = w.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_wait();
    grid_release();
    if (blockIdx.x == gridDim.x - 1) {
        __shared__ long long units_s[kPrepThreads / 32];
        __shared__ int count_s[kPrepThreads / 32];
        long long at = 0;
        int busy = 0;
        for (int b0 = 0; b0 < p.B; b0 += kPrepThreads) {
            const int b = b0 + tid;
            long long u = 0;
            int c = 0;
            if (b < p.B) {
                const Seq s = load_seq(p, b);
                if (s.n > 0) {
                    u = (long long)p.Hkv * units_of(w, make_item(p, s, 0).nt, s.n);
                    c = u > 0;
                }
            }
            const long long mine = u;
            const int one = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, u, o);
                const int y = __shfl_up_sync(0xffffffffu, c, o);
                if (lane >= o) {
                    u += x;
                    c += y;
                }
            }
            __syncthreads();
            if (lane == 31) {
                units_s[warp] = u;
                count_s[warp] = c;
            }
            __syncthreads();
            long long all = 0;
            int some = 0;
            for (int i = 0; i < kPrepThreads / 32; ++i) {
                if (i < warp) {
                    u += units_s[i];
                    c += count_s[i];
                }
                all += units_s[i];
                some += count_s[i];
            }
            // (offsets that do not ascend may give more requests rows than there are tokens: the first ones count)
            const int entry = busy + c - 1;
            if (one && entry <= p.tokens) {
                w.start[entry] = at + u - mine;
                if (entry < p.tokens) w.busy[entry] = b;
            }
            at += all;
            busy += some;
        }
        __syncthreads();
        if (tid == 0) {
            *w.ticket = 0;
            if (busy <= p.tokens) w.start[busy] = at;
            *w.count = min(busy, p.tokens);
        }
        return;
    }
    const int l16 = tid & 15, g16 = tid >> 4;
    const uint32_t rows = (uint32_t)p.tokens * (uint32_t)p.H, r0 = blockIdx.x * kPrepRows + g16;   // below 2^31
    const T *q = static_cast<const T *>(p.q), *aK = static_cast<const T *>(p.aK);
    float s[4] = {};
    const uint32_t mine = r0 + 16 * (l16 & 3);
    const float e = l16 < 4 && mine < rows ? w.lse[mine] : 0.f;
    if (aK) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t r = r0 + 16 * u;
            if (r >= rows) continue;
            const uint32_t t = r / (uint32_t)p.H, h = r - t * (uint32_t)p.H;
            const T *x = q + (long long)t * p.q_stride + h * (uint32_t)p.d, *y = aK + (long long)(h / (uint32_t)p.g) * p.ths;
            for (int c = l16 * E; c < p.d; c += 16 * E) s[u] += dot<T, E>(x + c, y + c);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
    }
    if (l16 < 4 && mine < rows) {
        const float x = l16 == 0 ? s[0] : l16 == 1 ? s[1] : l16 == 2 ? s[2] : s[3];
        w.nl[mine] = e == -INFINITY ? -INFINITY : fmaf(x, p.scale_log2, -e * kLog2e);
    }
}

// ======================================================================= SIMT
// A unit is 32 keys of one head, staged in shared memory as fp32; the rows that see any of them come 32 at a
// time, four to a warp, lane = key. A lane adds up its key's weights over the rows; the warps are joined
// at the end, in order (three chunks of 61 - 127 tokens over 100 - 700 keys, 8 heads of 64, fp32, key term: 29 us, 4 of them
// the set-up). The next rows are on their way into registers meanwhile. Bound by latency (a CTA takes
// 2 us for 32 rows) and shared memory, as the attention's SIMT kernel.
constexpr int kSimtThreads = 256;
constexpr int kRun = 32;
constexpr int kRunsPerTile = kTile / kRun;

struct SimtLayout {
    int d4, ld, lw;
    int q, k, a, R, nl, part, words;
    __host__ __device__ SimtLayout(int d, int clip_k, bool ak) {
        d4 = (d + 3) & ~3;
        ld = d4 + 4;
        lw = (clip_k + 1 + kRun - 1) / kRun * kRun + 1;
        int o = 0;
        q = o;    o += kRun * d4;
        k = o;    o += kRun * ld;
        a = o;    o += ak ? kRun * ld : 0;
        nl = o;   o += kRun;
        part = o; o += kSimtThreads;
        R = o;    o += ak ? kRun * lw : 0;
        words = o;
    }
};

template <typename T>
__device__ __forceinline__ float4 load4(const T *row, int c, int d, bool vec) {
    if (vec) {
        if (sizeof(T) == 4) return *reinterpret_cast<const float4 *>(row + c);
        const uint2 w = *reinterpret_cast<const uint2 *>(row + c);
        return make_float4(ptx::bf16lo_to_f32(w.x), ptx::bf16hi_to_f32(w.x), ptx::bf16lo_to_f32(w.y), ptx::bf16hi_to_f32(w.y));
    }
    return make_float4(to_f(row[c]), c + 1 < d ? to_f(row[c + 1]) : 0.f, c + 2 < d ? to_f(row[c + 2]) : 0.f,
                       c + 3 < d ? to_f(row[c + 3]) : 0.f);
}

// N4: 16-byte chunks of a row that a thread's share of 32 rows needs, ceil(d / 4 / 8)
template <typename T, int N4>
__global__ void __launch_bounds__(kSimtThreads, 2) weights_simt_kernel(const __grid_constant__ WeightParams w, int vec) {
    extern __shared__ __align__(16) float smf[];
    __shared__ int entry_s;
    __shared__ long long unit_s, rest_s;
    const Params &p = w.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int d = p.d, k = p.clip_k, P = 1 << p.pshift;
    const bool ak = p.aK != nullptr, wide = vec != 0;
    const SimtLayout L(d, k, ak);
    float *qs = smf + L.q, *Ks = smf + L.k, *As = smf + L.a, *Rs = smf + L.R, *nls = smf + L.nl, *part = smf + L.part;
    grid_wait();
    grid_release();
    const int count = *w.count;
    const long long total = w.start[count];
    const int my_row = tid >> 3, my_c = tid & 7;
    // products of this lane's staged row with the warp's four query rows
    auto scores = [&](const float *rows, float (&s)[4]) {
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] = 0.f;
#pragma unroll 2
        for (int c = 0; c < L.d4; c += 4) {
            const float4 kx = *reinterpret_cast<const float4 *>(rows + lane * L.ld + c);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 qx = *reinterpret_cast<const float4 *>(qs + (warp * 4 + u) * L.d4 + c);
                s[u] = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, fmaf(qx.z, kx.z, fmaf(qx.w, kx.w, s[u]))));
            }
        }
    };
    // eight threads to a row: chunks my_c, my_c + 8, ...; null: zeros
    auto fetch = [&](float4 (&x)[N4], const T *row) {
#pragma unroll
        for (int i = 0; i < N4; ++i) {
            const int c = 4 * (my_c + 8 * i);
            x[i] = row && c < L.d4 ? load4(row, c, d, wide) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    auto put = [&](float *dst, int ld, const float4 (&x)[N4]) {
#pragma unroll
        for (int i = 0; i < N4; ++i) {
            const int c = 4 * (my_c + 8 * i);
            if (c < L.d4) *reinterpret_cast<float4 *>(dst + my_row * ld + c) = x[i];
        }
    };
    for (bool begin = true;; begin = false) {
        __syncthreads();
        if (warp == 0) {
            unsigned long long u = blockIdx.x;   // the first ticket is the CTA's own
            if (!begin && lane == 0) u = gridDim.x + atomicAdd(w.ticket, 1ull);
            u = __shfl_sync(0xffffffffu, u, 0);
            long long rest = 0;
            int e = 0;
            if ((long long)u < total) e = find_unit(w, count, (long long)u, rest);
            if (lane == 0) {
                unit_s = (long long)u;
                entry_s = e;
                rest_s = rest;
            }
        }
        __syncthreads();
        if (unit_s >= total) break;
        const int b = w.busy[entry_s];
        const Seq s = load_seq(p, b);
        const Item it = make_item(p, s, 0);
        const int run = min((int)(rest_s / p.Hkv), it.nt * kRunsPerTile - 1);
        const int kvh = (int)(rest_s % p.Hkv);
        const int j0 = it.tile(run / kRunsPerTile) * kTile + (run % kRunsPerTile) * kRun;
        const int first = p.window > 0 ? max(0, max(it.pos_lo, 0) - p.window + 1) : 0;
        auto seen = [&](int j) { return j <= it.pos_hi && (j >= first || j < p.sinks); };
        const int *bt = p.bt + (long long)b * p.bt_stride;
        auto slot = [&](int j, long long &at) {   // whether the key's page exists, and its row
            const int pg = bt[j >> p.pshift];
            at = (long long)kvh * P + (j & (P - 1));
            if ((unsigned)pg >= (unsigned)p.num_pages) return -1;
            return pg;
        };
        {
            const int j = j0 + my_row;
            const T *row = nullptr;
            if (seen(j)) {
                long long at;
                const int pg = slot(j, at);
                if (pg >= 0) row = static_cast<const T *>(p.k) + (long long)pg * p.page_stride + at * d;
                else if (my_c == 0) report_page(p);
            }
            float4 x[N4];
            fetch(x, row);
            put(Ks, L.ld, x);
        }
        const int t_lo = first_token(j0, s.pos0), t_hi = end_token(p, j0, kRun, s.pos0, s.n);
        const long long r_end = (long long)t_hi * p.g;
        float sum = 0.f;
        float4 qx[N4];
        float nx;
        auto fetch_rows = [&](long long r0) {
            const long long r = r0 + my_row;
            const int tok = (int)(r / p.g), hh = (int)(r - (long long)tok * p.g);
            const bool on = r < r_end;
            fetch(qx, on ? static_cast<const T *>(p.q) + (long long)(s.q0 + tok) * p.q_stride + (long long)(kvh * p.g + hh) * d
                         : nullptr);
            nx = on ? w.nl[(long long)(s.q0 + tok) * p.H + kvh * p.g + hh] : -INFINITY;
        };
        fetch_rows((long long)t_lo * p.g);
        for (long long r0 = (long long)t_lo * p.g; r0 < r_end; r0 += kRun) {
            const int nr = (int)min((long long)kRun, r_end - r0);
            __syncthreads();                 // the previous rows are done
            put(qs, L.d4, qx);
            if (my_c == 0) nls[my_row] = nx;
            fetch_rows(r0 + kRun);
            const bool band = ak && j0 + kRun - 1 > s.pos0 + (int)(r0 / p.g) - k;
            if (band)
                for (int w0 = 0; w0 <= k; w0 += kRun) {
                    __syncthreads();
                    float4 x4[N4];
                    fetch(x4, w0 + my_row <= k ? static_cast<const T *>(p.aK) + (long long)kvh * p.ths + (long long)(w0 + my_row) * d
                                               : nullptr);
                    put(As, L.ld, x4);
                    __syncthreads();
                    float x[4];
                    scores(As, x);
#pragma unroll
                    for (int u = 0; u < 4; ++u) Rs[(warp * 4 + u) * L.lw + w0 + lane] = x[u] * p.scale_log2;
                }
            __syncthreads();
            float x[4];
            scores(Ks, x);
            const int j = j0 + lane;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = warp * 4 + u, pos = s.pos0 + (int)((r0 + r) / p.g);
                const bool on = r < nr && j <= pos && (p.window == 0 || j > pos - p.window || j < p.sinks);
                float e = fmaf(x[u], p.scale_log2, nls[r]);
                if (band && on) e += Rs[r * L.lw + max(j - pos + k, 0)] - Rs[r * L.lw];
                sum += on ? exp2f(e) : 0.f;
            }
        }
        part[tid] = sum;
        __syncthreads();
        const int j = j0 + lane;
        if (warp == 0 && seen(j)) {
            long long at;
            const int pg = slot(j, at);
            float all = 0.f;
#pragma unroll
            for (int i = 0; i < kSimtThreads / 32; ++i) all += part[32 * i + lane];
            if (pg >= 0) {
                leave_mass(w, w.mass + (long long)pg * w.mass_stride + at, all, j, s.pos0);
            }
        }
    }
}

template <typename T, int N4>
cudaError_t launch_simt_n(WeightParams w, cudaStream_t s) {
    w.per_tile = kRunsPerTile;
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return cudaErrorInvalidDevice;
    cudaError_t e = launch_weights_prep(w, sizeof(T) == 2, s);
    if (e != cudaSuccess) return e;
    const Params &p = w.p;
    const SimtLayout L(p.d, p.clip_k, p.aK != nullptr);
    // 16-byte (fp32) or 8-byte (bf16) loads where every row starts on such a boundary
    const long long es = sizeof(T);
    const uint64_t al = (uint64_t)(p.d * es) | (uint64_t)(p.q_stride * es) | (uint64_t)(p.page_stride * es) |
                        (uint64_t)(p.ths * es) | reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                        reinterpret_cast<uintptr_t>(p.aK);
    e = opt_in_smem(reinterpret_cast<const void *>(weights_simt_kernel<T, N4>), di);
    if (e != cudaSuccess) return e;
    return launch_early(weights_simt_kernel<T, N4>, dim3(2 * di.sms), kSimtThreads, L.words * sizeof(float), s, w,
                        al % (4 * es) == 0 ? 1 : 0);
}

template <typename T>
cudaError_t launch_simt(const WeightParams &w, cudaStream_t s) {
    return w.p.d <= 32 ? launch_simt_n<T, 1>(w, s) : w.p.d <= 64 ? launch_simt_n<T, 2>(w, s) : launch_simt_n<T, 4>(w, s);
}

// ======================================================================= generated tokens
// At most 16 query rows per key head (bf16, d = 64 or 128, pages of at least 8 keys): keys are the wide
// side of m16n8k16 products, as in the attention of generated tokens, whose staging this has: a ninth
// warp walks the CTA's share of the tiles and feeds a ring by TMA, eight row warps take 16 keys of a tile
// each. A key's weights of all rows come together in one warp, so nothing is joined; the page numbers come with the
// keys. HBM bounds it: a key is 2 d bytes and 8 of mass.
constexpr int kWarps = 8;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kRowThreads = 32 * kWarps;
constexpr int kGroup = 16;               // keys of a warp per tile
constexpr int kMaxStages = 4;
constexpr uint32_t kSideBytes = 64;      // a tile's page numbers, 16 at most

template <int D>
constexpr int kStageBytes = kTile * D * 2;
// A row warp's chain on a tile (products, exponentials, two shuffles) is latency, so several CTAs share an SM (with two and
// one: 32 requests of 1K-2K keys, 16 heads of 64: 28.2 us in place of 26.5; 64 of 2K-16K, two key heads of 128: 55.2, 53.6;
// 25.2 and 51.1 as the kernel is now)
template <int D>
constexpr int kCtasPerSm = D == 64 ? 3 : 2;

enum : int { B_FULL = 0, B_EMPTY = kMaxStages, B_PIECE_FULL = 2 * kMaxStages, B_PIECE_EMPTY = B_PIECE_FULL + kPieces,
             kNumBars = B_PIECE_EMPTY + kPieces };

struct Layout {
    uint32_t piece, bar, side, R, bytes;
    int lw;
    template <int D, int NT>
    static __host__ __device__ Layout make(int clip_k, bool ak, int stages) {
        Layout L;
        L.lw = ak ? (clip_k + 1) | 1 : 0;
        uint32_t off = (uint32_t)stages * kStageBytes<D>;
        L.piece = off; off += kPieces * sizeof(Piece);
        L.bar = off;   off += kNumBars * 8 + 16;
        L.side = off;  off += (uint32_t)stages * kSideBytes;
        L.R = off;     off += 8 * NT * L.lw * 4;
        L.bytes = off;
        return L;
    }
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// row of key slot i of 8: neighbouring lanes' 16-byte reads then fall in the eight chunks of a line
__device__ __forceinline__ int perm(int i) { return (i >> 1) | ((i & 1) << 2); }

struct Waits {
    volatile int *abort_flag;
    int *err;
    long long limit;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
        if (ptx::mbar_try(bar, parity)) return true;
        return tc::wait_bar_slow_call(bar, parity, abort_flag, err, limit);
    }
};

template <int D>
__device__ void feed_role(const WeightParams &w, const Layout &L, uint8_t *smem, const Waits &waits,
                          const CUtensorMap *tm_k, int stages, int box) {
    const Params &p = w.p;
    constexpr int DB = D / 64;
    const int lane = threadIdx.x & 31;
    const uint32_t base = ptx::smem_u32(smem), bars = base + L.bar;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto wait = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, waits(b, parity) ? 1 : 0) != 0; };
    Piece *ring = reinterpret_cast<Piece *>(smem + L.piece);
    const int nbox = kTile / box, my_box = lane % nbox, my_blk = lane / nbox;
    const uint32_t my_dst = base + my_blk * (kTile * 128) + my_box * box * 128;
    Walk walk(p, find_range(p));
    Segment g{};
    uint32_t it = 0, tiles = 0;
    int st = 0;
    uint32_t ph = 0;
    bool more = true, ok = true;
    while (more && ok) {
        more = walk.next(p, g);
        if (more && g.t1 == g.t0) continue;   // no keys: nothing to do
        const int i = it & (kPieces - 1);
        if (!(ok = wait(bar(B_PIECE_EMPTY + i), ((it / kPieces) & 1u) ^ 1u))) break;
        if (lane == 0) {
            ring[i] = make_piece(p, g, more);
            ptx::mbar_arrive(bar(B_PIECE_FULL + i));
        }
        __syncwarp();
        ++it;
        if (!more) break;
        const int first = p.window > 0 ? max(0, max(g.it.pos_lo, 0) - p.window + 1) : 0;
        const int *bt = p.bt + (long long)g.b * p.bt_stride;
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
            const int j = g.it.tile(t) * kTile + my_box * box, row = j & ((1 << p.pshift) - 1);
            const bool bad = seen && (unsigned)pg >= (unsigned)p.num_pages;
            if (bad) report_page(p);
            if (my_blk == 0) reinterpret_cast<int *>(smem + L.side + st * kSideBytes)[my_box] = bad ? -1 : pg;
            __syncwarp();
            const unsigned m = __ballot_sync(0xffffffffu, seen && my_blk == 0);
            if (lane == 0) ptx::mbar_expect_tx(bar(B_FULL + st), (uint32_t)(__popc(m) * box * D * 2));
            __syncwarp();
            if (seen && my_blk < DB && !(p.withhold && tiles == 0))   // a page outside the cache: zeros
                tma_load_4d(my_dst + st * kStageBytes<D>, tm_k, bar(B_FULL + st), my_blk * 64, row, g.kvh,
                            bad ? p.num_pages : pg);
            __syncwarp();
            ++tiles;
            if (++st == stages) {
                st = 0;
                ph ^= 1u;
            }
        }
    }
    // no copy is in flight when the CTA exits
    for (uint32_t i = tiles > (uint32_t)stages ? tiles - stages : 0; i < tiles; ++i)
        tc::drain_bar(bar(B_FULL + (int)(i % stages)), (i / stages) & 1u, p.wait_limit);
}

template <int D, int NT, bool AK>
__device__ void row_role(const WeightParams &w, const Layout &L, uint8_t *smem, const Waits &wait, int stages, int box) {
    constexpr int kRows = 8 * NT;
    const Params &p = w.p;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int c = lane & 3, rq = lane >> 2;
    const uint32_t base = ptx::smem_u32(smem), bars = base + L.bar;
    float *Rs = reinterpret_cast<float *>(smem + L.R);
    const Piece *pieces = reinterpret_cast<const Piece *>(smem + L.piece);
    const int k = p.clip_k, W = k + 1;
    uint32_t stage = 0, phase = 0;
    const int kr = perm(rq);
    const uint32_t ring = base + warp * (kGroup * 128);
    const uint32_t k_at[2] = {(uint32_t)(kr * 128 + ((c ^ kr) << 4)), (uint32_t)(kr * 128 + (((c + 4) ^ kr) << 4))};
    for (uint32_t it = 0;; ++it) {
        const int slot = it & (kPieces - 1);
        // all row warps go on together, or leave together
        const bool ok = wait(bars + 8u * (B_PIECE_FULL + slot), (it / kPieces) & 1u);
        if (!ptx::bar_red_and(1, kRowThreads, ok)) break;
        const Piece g = pieces[slot];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + 8u * (B_PIECE_EMPTY + slot));
        if (g.cnt == 0) break;
        const int rows = g.cnt * p.g, first = g.first(p);
        const bool many = rows > kRows;      // (a max_new that was too small) the rows in groups, each tile anew
        uint4 qf[NT][D / 32];
        int pos[NT][2];
        float nl[NT][2], r0[NT][2];
        auto scores = [&](float (&x)[NT][4], const uint4 &lo, const uint4 &hi, int s) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma(x[n], lo.x, hi.x, lo.y, hi.y, qf[n][s].x, qf[n][s].y);
                mma(x[n], lo.z, hi.z, lo.w, hi.w, qf[n][s].z, qf[n][s].w);
            }
        };
        // rows g0 .. g0 + kRows - 1: fragments (lane: row rq, columns 32 s + 8 c .. + 7), positions and
        // constants of rows 2 c, 2 c + 1, and R = Q aK^T
        auto set_rows = [&](int g0) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = g0 + 8 * n + rq, tok = r / p.g, hh = r - tok * p.g;
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + (long long)(g.row0 + tok) * p.q_stride +
                                         (long long)(g.kvh * p.g + hh) * D + 8 * c;
#pragma unroll
                for (int s = 0; s < D / 32; ++s)
                    qf[n][s] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(q + 32 * s)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r2 = g0 + 8 * n + 2 * c + e, t2 = r2 / p.g, h2 = r2 - t2 * p.g;
                    pos[n][e] = g.pos_lo + (r2 < rows ? t2 : 0);
                    nl[n][e] = -INFINITY;   // (of a row without keys, as its log-sum-exp says, too)
                    if (r2 < rows) {
                        const float lse = __ldg(w.lse + (long long)(g.row0 + t2) * p.H + g.kvh * p.g + h2);
                        if (lse != -INFINITY) nl[n][e] = -kLog2e * lse;
                    }
                }
            }
            if (AK) {
                ptx::named_bar_sync(1, kRowThreads);   // the last rows' entries have been read
                const __nv_bfloat16 *aK = static_cast<const __nv_bfloat16 *>(p.aK) + (long long)g.kvh * p.ths + 8 * c;
                for (int w0 = 16 * warp; w0 < W; w0 += 16 * kWarps) {
                    float x[NT][4] = {};
#pragma unroll
                    for (int s = 0; s < D / 32; ++s) {
                        uint4 a[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            a[h] = w0 + rq + 8 * h < W
                                       ? __ldg(reinterpret_cast<const uint4 *>(aK + (long long)(w0 + rq + 8 * h) * D + 32 * s))
                                       : make_uint4(0, 0, 0, 0);
                        scores(x, a[0], a[1], s);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int row = w0 + rq + 8 * (e >> 1);
                            if (row < W) Rs[(8 * n + 2 * c + (e & 1)) * L.lw + row] = x[n][e] * p.scale_log2;
                        }
                }
                ptx::named_bar_sync(1, kRowThreads);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) r0[n][e] = nl[n][e] + (AK ? Rs[(8 * n + 2 * c + e) * L.lw] : 0.f);
        };
        const int mine = warp * kGroup + kr + 8 * c;   // this lane's key of a tile, where c < 2
        if (!many) set_rows(0);
#pragma unroll 1
        for (int t = g.t0; t < g.t1; ++t) {
            const int j0 = g.tile(t) * kTile + warp * kGroup;
            const uint32_t st = ring + stage * kStageBytes<D>;
            const uint32_t empty = bars + 8u * (B_EMPTY + stage);
            const uint8_t *side = smem + L.side + stage * kSideBytes;
            wait(bars + 8u * (B_FULL + stage), phase);
            if (++stage == (uint32_t)stages) {
                stage = 0;
                phase ^= 1u;
            }
            __syncwarp();
            float sum[2] = {0.f, 0.f};
            for (int g0 = 0; g0 < rows; g0 += kRows) {
                if (many) set_rows(g0);
                float x[NT][4] = {};
#pragma unroll
                for (int s = 0; s < D / 32; ++s) {
                    const uint32_t a = st + (s >> 1) * (kTile * 128) + k_at[s & 1];
                    scores(x, lds128(a), lds128(a + 1024), s);
                }
                const int p_lo = g.pos_lo + g0 / p.g;
                const bool near = j0 + kGroup - 1 > p_lo - k;
                const bool full = j0 + kGroup - 1 <= p_lo &&
                                  (p.window == 0 || j0 > g.pos_hi - p.window || j0 + kGroup <= p.sinks);
                if (AK && near) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int lab = min(max(j0 + kr + 8 * (e >> 1) - pos[n][e & 1], -k) + k, k);
                            x[n][e] = fmaf(x[n][e], p.scale_log2, Rs[(8 * n + 2 * c + (e & 1)) * L.lw + lab] + nl[n][e & 1]);
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
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[e >> 1] += ptx::ex2(x[n][e]);
            }
            const int j = g.tile(t) * kTile + mine;
            int pg = -1;
            if (c < 2 && j <= g.pos_hi && (j >= first || j < p.sinks)) pg = reinterpret_cast<const int *>(side)[mine / box];
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
                sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
            }
            if (pg >= 0)
                leave_mass(w, w.mass + (long long)pg * w.mass_stride + (((long long)g.kvh << p.pshift) + (j & ((1 << p.pshift) - 1))),
                           c == 0 ? sum[0] : sum[1], j, g.pos_lo);
        }
    }
}

template <int D, int NT, bool AK>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<D>)
    weights_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ WeightParams w, int stages,
                          int box) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const Params &p = w.p;
    const Layout L = Layout::make<D, NT>(p.clip_k, AK, stages);
    const uint32_t bars = ptx::smem_u32(smem) + L.bar;
    Waits waits{reinterpret_cast<volatile int *>(smem + L.bar + kNumBars * 8), p.err, p.wait_limit};
    if (threadIdx.x == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            const bool by_rows = (i >= B_EMPTY && i < B_EMPTY + kMaxStages) || i >= B_PIECE_EMPTY;
            ptx::mbar_init(bars + 8u * (uint32_t)i, by_rows ? kWarps : 1);
        }
        *waits.abort_flag = 0;
        ptx::mbar_init_fence();
        ptx::tma_prefetch_desc(&tm_k);
    }
    __syncthreads();
    grid_wait();
    grid_release();
    if (threadIdx.x >= kRowThreads)
        feed_role<D>(w, L, smem, waits, &tm_k, stages, box);
    else
        row_role<D, NT, AK>(w, L, smem, waits, stages, box);
}

template <int D, int NT, bool AK>
cudaError_t launch_decode(const PagedWeightsArgs &a, const WeightParams &w, cudaStream_t s) {
    auto kern = weights_decode_kernel<D, NT, AK>;
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return cudaErrorInvalidDevice;
    CUtensorMap tm;
    const int box = a.a.page_size < kTile ? a.a.page_size : kTile;
    if (!make_page_map(&tm, a.a.k_pages, a.a, box)) return cudaErrorInvalidValue;
    const int share = (di.smem_optin + 1024) / kCtasPerSm<D> - 1024;
    int stages = kMaxStages;
    while (stages > 1 && (int)Layout::make<D, NT>(w.p.clip_k, AK, stages).bytes > share) --stages;
    const cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kern), di);
    if (e != cudaSuccess) return e;
    return launch_early(kern, dim3(di.sms * kCtasPerSm<D>), kThreads, Layout::make<D, NT>(w.p.clip_k, AK, stages).bytes, s,
                        tm, w, stages, box);
}

template <int D, int NT>
cudaError_t launch_decode_terms(const PagedWeightsArgs &a, const WeightParams &w, cudaStream_t s) {
    return a.a.aK ? launch_decode<D, NT, true>(a, w, s) : launch_decode<D, NT, false>(a, w, s);
}

size_t round16(size_t x) { return (x + 15) & ~(size_t)15; }

}  // namespace

cudaError_t launch_weights_prep(const WeightParams &w, bool bf16, cudaStream_t s) {
    const Params &p = w.p;
    const long long blocks = ((long long)p.tokens * p.H + kPrepRows - 1) / kPrepRows + 1;
    const long long es = bf16 ? 2 : 4;
    const uint64_t m = (uint64_t)(p.d * es) | (uint64_t)(p.q_stride * es) | (uint64_t)(p.ths * es) |
                       reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.aK);
    const dim3 g((unsigned)blocks);
    if (bf16)
        return m % 16 == 0 ? launch_early(weights_prep_kernel<__nv_bfloat16, 8>, g, kPrepThreads, 0, s, w)
                           : launch_early(weights_prep_kernel<__nv_bfloat16, 1>, g, kPrepThreads, 0, s, w);
    return m % 16 == 0 ? launch_early(weights_prep_kernel<float, 4>, g, kPrepThreads, 0, s, w)
                       : launch_early(weights_prep_kernel<float, 1>, g, kPrepThreads, 0, s, w);
}

}  // namespace paged

// workspace: {ticket, count}, unit starts, request numbers, row constants
unsigned long long paged_weights_workspace_bytes(int tokens, int H) {
    return 16 + paged::round16(((size_t)tokens + 1) * 8) + paged::round16((size_t)tokens * 4) +
           paged::round16((size_t)tokens * H * 4);
}

cudaError_t launch_paged_weights(const PagedWeightsArgs &a, cudaStream_t s) {
    using namespace paged;
    WeightParams w;
    std::memset(&w, 0, sizeof(w));
    fill_params(a.a, &w.p);
    Params &p = w.p;
    p.T = p.T1 = 0x3fffffff;     // all tokens of a request: one item
    p.c0 = p.wt = p.wt2 = 1;
    w.lse = a.lse;
    w.mass = a.mass;
    w.mass_stride = a.mass_stride;
    w.accumulate = a.accumulate;
    char *ws = static_cast<char *>(a.workspace);
    w.ticket = reinterpret_cast<unsigned long long *>(ws);
    w.count = reinterpret_cast<int *>(ws + 8);
    w.start = reinterpret_cast<long long *>(ws + 16);
    ws += 16 + round16(((size_t)p.tokens + 1) * 8);
    w.busy = reinterpret_cast<int *>(ws);
    w.nl = reinterpret_cast<float *>(ws + round16((size_t)p.tokens * 4));
    const long long rows = (long long)a.a.max_new * p.g;
    if (a.a.max_new >= 1 && rows <= 16 && pages_by_tma(a.a)) {
        p.long_line = line_is_long(p);
        if (a.a.d == 64) return rows <= 8 ? launch_decode_terms<64, 1>(a, w, s) : launch_decode_terms<64, 2>(a, w, s);
        return rows <= 8 ? launch_decode_terms<128, 1>(a, w, s) : launch_decode_terms<128, 2>(a, w, s);
    }
    if (weights_tc_covers(a)) {
        const cudaError_t e = launch_weights_tc(a, w, s);
        if (e != cudaErrorNotSupported) return e;
    }
    return a.a.bf16 ? launch_simt<__nv_bfloat16>(w, s) : launch_simt<float>(w, s);
}

}  // namespace relattn
