// Paged attention for few query rows per key/value head (generated tokens: T tokens x g heads
// <= 16 rows), bf16, d = 64 or 128, pages of at least 8 keys.
//
// Every cached key and value is read once and meets at most 16 rows, so HBM bounds the kernel:
// 4 d bytes per key against 64 d multiply-adds. The rows fill one m16n8k16 tensor-core tile (a
// 128-row tcgen05 tile would be seven eighths padding and would need the keys staged for the
// async proxy; at 16 rows the products are a tenth of the time the bytes take).
//
// One CTA of 8 warps per SM. A tile of 128 keys is 16 keys per warp; each warp keeps its own
// running maximum, sum and output over the keys it gets, and the warps are joined once per piece.
// Loads run through a ring of kStages groups of 16 keys per warp by 16-byte cp.async. The ring
// is private to each lane: the lane copies exactly the 16-byte chunks that its own fragments
// need and reads them back itself, so the loop has no barrier, no swizzle and no transposition:
//   S = Q K^T: the order of the contracted columns is free, so lane (key l / 4, c = l % 4) takes
//     columns 32 s + 8 c .. + 7 of its key as the k-slots of two MMA steps, and Q alike;
//   O = P V: the lane takes columns 64 u + 8 (l / 4) .. + 7 of keys 2 c, 2 c + 1 (+ 8) and pairs
//     two keys' columns by byte permutes: the n-slot l / 4 of step (u, i) is column
//     64 u + 8 (l / 4) + i. A lane's outputs are then 16 consecutive columns of a row.
// The ring runs ahead over the ends of the pieces (a second walk over the CTA's range issues the
// loads), so joining the warps costs no bandwidth while it is shorter than the ring.
//
// Relative terms: R = Q aK^T (k + 1 rows) once per piece by the same MMA; keys at most k - 1
// back add their own R entry and leave their score in a bin; the other keys share entry 0 and
// their weights are summed. At the end of the piece sum_r beta_r aV_r joins the output.
#include <cstdint>

#include "relattn_paged.cuh"
#include "sm103_ptx.cuh"

namespace relattn {
namespace paged {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;                // query rows of an item
constexpr int kGroup = 16;               // keys of a warp per tile
static_assert(kWarps * kGroup == kTile, "a tile is one group per warp");

template <int D>
struct Cfg {
    static constexpr int kStageBytes = 2 * kGroup * D * 2;    // one warp's group: K and V
    static constexpr int kStages = D == 64 ? 4 : 2;
};

// The joined outputs: 16-byte chunk `ch` of row `row`, swizzled so that the fragments' stores of
// neighbouring rows fall in different banks
template <int D>
__device__ __forceinline__ int out_at(int warp, int row, int ch) {
    return (warp * kRows + row) * D + ((ch ^ (row & 7)) << 2);
}

struct Layout {
    uint32_t o, ml, R, Bn, bytes;        // byte offsets behind the ring
    int lw;
    template <int D>
    static __host__ __device__ Layout make(int clip_k) {
        Layout L;
        L.lw = (clip_k + 1) | 1;
        uint32_t off = (uint32_t)kWarps * Cfg<D>::kStages * Cfg<D>::kStageBytes;
        L.o = off;  off += kWarps * kRows * D * 4;
        L.ml = off; off += kWarps * kRows * 4 * 4;
        L.R = off;  off += kRows * L.lw * 4;
        L.Bn = off; off += kRows * L.lw * 4;
        L.bytes = off;
        return L;
    }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// The groups that a warp gets over the CTA's range, one per call: tile after tile of piece after
// piece. `page` holds the page numbers of the next group's two halves (8 keys each), loaded one
// call ahead so that the copies do not wait for the table.
template <int D>
struct Feed {
    Walk walk;
    Segment g;
    int t;               // next tile of the piece
    bool more;
    int pg[2], j0;       // of the next group
    __device__ __forceinline__ Feed(const Params &p, const Range &r) : walk(p, r), t(0), more(true), pg{0, 0}, j0(0) {}
    __device__ __forceinline__ void advance(const Params &p, int warp, bool begin) {
        if (!begin) ++t;
        while (begin || t >= g.t1) {
            if (!walk.next(p, g)) {
                more = false;
                return;
            }
            t = g.t0;
            begin = false;
        }
        j0 = g.it.tile(t) * kTile + warp * kGroup;
        const int first = p.window > 0 ? max(0, max(g.it.pos_lo, 0) - p.window + 1) : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = j0 + 8 * h;
            const bool seen = j <= g.it.pos_hi && (j + 8 > first || j < p.sinks);
            // -2: nothing to load; -1 (or a number past the cache): no such page
            pg[h] = seen ? max(-1, __ldg(p.bt + (long long)g.b * p.bt_stride + (j >> p.pshift))) : -2;
        }
    }
    // issues the copies of the next group into ring stage `dst` (this lane's address)
    __device__ __forceinline__ void issue(const Params &p, uint32_t dst, int lane) {
        const int P = 1 << p.pshift;
        const int first = p.window > 0 ? max(0, max(g.it.pos_lo, 0) - p.window + 1) : 0;
        const int c = lane & 3, rq = lane >> 2;
        const __nv_bfloat16 *kb = static_cast<const __nv_bfloat16 *>(p.k), *vb = static_cast<const __nv_bfloat16 *>(p.v);
        long long base[2];
        bool ok[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ok[h] = (unsigned)pg[h] < (unsigned)p.num_pages;
            if (!ok[h] && pg[h] != -2 && lane == 0) report_page(p);
            base[h] = ok[h] ? (long long)pg[h] * p.page_stride +
                                  ((long long)g.kvh * P + ((j0 + 8 * h) & (P - 1))) * D
                            : 0;
        }
        auto seen = [&](int j) { return j <= g.it.pos_hi && (j >= first || j < p.sinks); };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool on = ok[h] && seen(j0 + 8 * h + rq);
            const __nv_bfloat16 *src = kb + base[h] + (long long)rq * D + 8 * c;
#pragma unroll
            for (int s = 0; s < D / 32; ++s) cp16(dst + (h * (D / 32) + s) * 512, src + 32 * s, on);
        }
        dst += (D / 16) * 512;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool on = ok[h] && seen(j0 + 8 * h + 2 * c + e);
                const __nv_bfloat16 *src = vb + base[h] + (long long)(2 * c + e) * D + 8 * rq;
#pragma unroll
                for (int u = 0; u < D / 64; ++u) cp16(dst + ((2 * h + e) * (D / 64) + u) * 512, src + 64 * u, on);
            }
    }
};

template <int D, bool AK, bool AV>
__global__ void __launch_bounds__(kThreads, 1) paged_decode_kernel(const __grid_constant__ Params p) {
    using C = Cfg<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scr[80];
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int c = lane & 3, rq = lane >> 2;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Range rg = find_range<kThreads>(p, scr);
    const Layout L = Layout::make<D>(p.clip_k);
    const uint32_t ring = ptx::smem_u32(smem) + (uint32_t)warp * C::kStages * C::kStageBytes + lane * 16;
    float *so = reinterpret_cast<float *>(smem + L.o);
    float4 *sml = reinterpret_cast<float4 *>(smem + L.ml);   // {m, l, far, -} of [warp][row]
    float *Rs = reinterpret_cast<float *>(smem + L.R), *Bs = reinterpret_cast<float *>(smem + L.Bn);
    const int k = p.clip_k, W = k + 1;

    // ---- fill the ring
    Feed<D> feed(p, rg);
    feed.advance(p, warp, true);
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) {
        if (feed.more) {
            feed.issue(p, ring + s * C::kStageBytes, lane);
            feed.advance(p, warp, false);
        }
        cp_commit();
    }
    uint32_t stage = 0;

    Walk walk(p, rg);
    Segment g{};
    bool any = false;
    while (walk.next(p, g)) {
        any = true;
        const int rows = g.it.cnt * p.g;
        // ---- Q fragments of rows rq and rq + 8
        uint4 qa[D / 32], qb[D / 32];
        int pos[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = rq + 8 * h;
            const int tok = r / p.g, hh = r - tok * p.g;
            pos[h] = g.it.pos_lo + (r < rows ? tok : 0);
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) +
                                     (long long)(g.s.q0 + g.it.i0 + tok) * p.q_stride +
                                     (long long)(g.kvh * p.g + hh) * D + 8 * c;
#pragma unroll
            for (int s = 0; s < D / 32; ++s) {
                const uint4 x = r < rows ? __ldg(reinterpret_cast<const uint4 *>(q + 32 * s)) : make_uint4(0, 0, 0, 0);
                if (h == 0) qa[s] = x; else qb[s] = x;
            }
        }
        // S of 8 keys from their chunks
        auto scores = [&](float (&acc)[4], const uint4 &kx, int s) {
            mma(acc, qa[s].x, qb[s].x, qa[s].y, qb[s].y, kx.x, kx.y);
            mma(acc, qa[s].z, qb[s].z, qa[s].w, qb[s].w, kx.z, kx.w);
        };
        if (AK) {   // R = Q aK^T, 8 table rows per MMA column tile
            const __nv_bfloat16 *aK = static_cast<const __nv_bfloat16 *>(p.aK) + (long long)g.kvh * p.ths;
            for (int w0 = 8 * warp; w0 < W; w0 += 8 * kWarps) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < D / 32; ++s) {
                    const uint4 x = w0 + rq < W ? __ldg(reinterpret_cast<const uint4 *>(aK + (long long)(w0 + rq) * D + 8 * c + 32 * s))
                                                : make_uint4(0, 0, 0, 0);
                    scores(acc, x, s);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int w = w0 + 2 * c + (e & 1);
                    if (w < W) Rs[(rq + 8 * (e >> 1)) * L.lw + w] = acc[e] * p.scale_log2;
                }
            }
        }
        if (AV)
            for (int i = tid; i < kRows * L.lw; i += kThreads) Bs[i] = -INFINITY;
        if (AK || AV) __syncthreads();
        const float r0a = AK ? Rs[rq * L.lw] : 0.f, r0b = AK ? Rs[(rq + 8) * L.lw] : 0.f;

        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, far[2] = {0.f, 0.f};
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

        for (int t = g.t0; t < g.t1; ++t) {
            const int j0 = g.it.tile(t) * kTile + warp * kGroup;
            const uint32_t st = ring + stage * C::kStageBytes;
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
            cp_wait<C::kStages - 1>();
            float x[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[h][e] = 0.f;
#pragma unroll
                for (int s = 0; s < D / 32; ++s) scores(x[h], lds128(st + (h * (D / 32) + s) * 512), s);
            }
            // ---- logits in the log2 domain
            const bool near = j0 + kGroup - 1 > g.it.pos_lo - k;   // some key has an entry of its own
            const bool full = j0 + kGroup - 1 <= g.it.pos_lo &&
                              (p.window == 0 || j0 > g.it.pos_hi - p.window || j0 + kGroup <= p.sinks);
            if (!(AK || AV) || !near) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[h][e] = fmaf(x[h][e], p.scale_log2, e < 2 ? r0a : r0b);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int lab = min(max(j0 + 8 * h + 2 * c + (e & 1) - pos[e >> 1], -k) + k, k);
                        const float r = AK ? Rs[(rq + 8 * (e >> 1)) * L.lw + lab] : 0.f;
                        x[h][e] = fmaf(x[h][e], p.scale_log2, r);
                    }
            }
            if (!full) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + 8 * h + 2 * c + (e & 1), q = pos[e >> 1];
                        const bool seen = j <= q && (p.window == 0 || j > q - p.window || j < p.sinks);
                        x[h][e] = seen ? x[h][e] : -INFINITY;
                    }
            }
            // ---- the running maximum of each row, over the four lanes that share it
            float mx[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mx[r] = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            }
            if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
                float al[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float mn = fmaxf(m[r], mx[r]);
                    al[r] = mn == -INFINITY ? 1.f : ptx::ex2(m[r] - mn);
                    m[r] = mn;
                    l[r] *= al[r];
                    far[r] *= al[r];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][e] *= al[e >> 1];
            }
            const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
            float pr[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pr[h][e] = ptx::ex2(x[h][e] - mu[e >> 1]);
                    l[e >> 1] += pr[h][e];
                }
            if (AV) {
                if (near) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int lab = j0 + 8 * h + 2 * c + (e & 1) - pos[e >> 1] + k;
                            if (lab > 0 && lab <= k) Bs[(rq + 8 * (e >> 1)) * L.lw + lab] = x[h][e];
                            else far[e >> 1] += pr[h][e];
                        }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) far[e >> 1] += pr[h][e];
                }
            }
            // ---- O += P V (P rounded to bf16 for the tensor cores; the sums above keep fp32)
            const uint32_t a0 = ptx::pack_bf16x2(pr[0][0], pr[0][1]), a1 = ptx::pack_bf16x2(pr[0][2], pr[0][3]);
            const uint32_t a2 = ptx::pack_bf16x2(pr[1][0], pr[1][1]), a3 = ptx::pack_bf16x2(pr[1][2], pr[1][3]);
            const uint32_t sv = st + (D / 16) * 512;
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                uint4 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = lds128(sv + (e * (D / 64) + u) * 512);
                const uint32_t *v0 = reinterpret_cast<const uint32_t *>(&v[0]), *v1 = reinterpret_cast<const uint32_t *>(&v[1]);
                const uint32_t *v2 = reinterpret_cast<const uint32_t *>(&v[2]), *v3 = reinterpret_cast<const uint32_t *>(&v[3]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t sel = i & 1 ? 0x7632 : 0x5410;
                    mma(o[8 * u + i], a0, a1, a2, a3, __byte_perm(v0[i / 2], v1[i / 2], sel),
                        __byte_perm(v2[i / 2], v3[i / 2], sel));
                }
            }
            // ---- the stage is free: the group kStages ahead
            if (feed.more) {
                feed.issue(p, st, lane);
                feed.advance(p, warp, false);
            }
            cp_commit();
        }
        // ---- join the warps
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (AV) {
                far[r] += __shfl_xor_sync(0xffffffffu, far[r], 1);
                far[r] += __shfl_xor_sync(0xffffffffu, far[r], 2);
            }
            const int row = rq + 8 * r;
            if (row < rows) {
                if (c == 0) sml[warp * kRows + row] = make_float4(m[r], l[r], far[r], 0.f);
#pragma unroll
                for (int u = 0; u < D / 64; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < 8; i += 4)
                            *reinterpret_cast<float4 *>(so + out_at<D>(warp, row, 16 * u + 4 * c + 2 * e + i / 4)) =
                                make_float4(o[8 * u + i][2 * r + e], o[8 * u + i + 1][2 * r + e],
                                            o[8 * u + i + 2][2 * r + e], o[8 * u + i + 3][2 * r + e]);
            }
        }
        __syncthreads();
        auto row_max = [&](int row) {
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w * kRows + row].x);
            return M;
        };
        if (AV) {   // the bins' weights in place of their scores
            for (int i = tid; i < rows * W; i += kThreads) {
                const int row = i / W, w = i - row * W;
                const float M = row_max(row), Mu = M == -INFINITY ? 0.f : M;
                float b;
                if (w == 0) {
                    b = 0.f;
#pragma unroll
                    for (int q = 0; q < kWarps; ++q) b += sml[q * kRows + row].z * ptx::ex2(sml[q * kRows + row].x - Mu);
                } else {
                    b = ptx::ex2(Bs[row * L.lw + w] - Mu);
                }
                Bs[row * L.lw + w] = b;
            }
            __syncthreads();
        }
        const bool whole = g.whole();
        float *rec = whole ? nullptr : record(p, blockIdx.x, g.record());
        // four columns a thread
        for (int i = tid; i < rows * (D / 4); i += kThreads) {
            const int row = i / (D / 4), col = (i - row * (D / 4)) * 4;
            const float M = row_max(row), Mu = M == -INFINITY ? 0.f : M;
            float ls = 0.f;
            float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 s = sml[w * kRows + row];
                const float f = ptx::ex2(s.x - Mu);
                const float4 ow = *reinterpret_cast<const float4 *>(so + out_at<D>(w, row, col / 4));
                ls = fmaf(f, s.y, ls);
                z.x = fmaf(f, ow.x, z.x);
                z.y = fmaf(f, ow.y, z.y);
                z.z = fmaf(f, ow.z, z.z);
                z.w = fmaf(f, ow.w, z.w);
            }
            if (AV) {
                const __nv_bfloat16 *aV = static_cast<const __nv_bfloat16 *>(p.aV) + (long long)g.kvh * p.ths + col;
#pragma unroll 8
                for (int w = 0; w < W; ++w) {
                    const float b = Bs[row * L.lw + w];
                    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(aV + (long long)w * D));
                    z.x = fmaf(b, ptx::bf16lo_to_f32(v.x), z.x);
                    z.y = fmaf(b, ptx::bf16hi_to_f32(v.x), z.y);
                    z.z = fmaf(b, ptx::bf16lo_to_f32(v.y), z.z);
                    z.w = fmaf(b, ptx::bf16hi_to_f32(v.y), z.w);
                }
            }
            if (whole) {
                const float inv = ls > 0.f ? 1.f / ls : 0.f;
                const int tok = row / p.g, hh = row - tok * p.g;
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                                     ((long long)(g.s.q0 + g.it.i0 + tok) * p.H + g.kvh * p.g + hh) * D + col;
                *reinterpret_cast<uint2 *>(dst) = make_uint2(ptx::pack_bf16x2(z.x * inv, z.y * inv),
                                                             ptx::pack_bf16x2(z.z * inv, z.w * inv));
            } else {
                if (col == 0) {
                    rec[row] = M;
                    rec[p.rec_rows + row] = ls;
                }
                *reinterpret_cast<float2 *>(rec + 2 * p.rec_rows + row * D + col) = make_float2(z.x, z.y);
                *reinterpret_cast<float2 *>(rec + 2 * p.rec_rows + row * D + col + 2) = make_float2(z.z, z.w);
            }
        }
        __syncthreads();   // the next piece writes the shared arrays
    }
    cp_wait<0>();
    if (tid == 0) write_desc(p, any ? &g : nullptr, rg.total);
}

template <int D, bool AK, bool AV>
cudaError_t launch_variant(const Params &p, cudaStream_t s) {
    auto kern = paged_decode_kernel<D, AK, AV>;
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return cudaErrorInvalidDevice;
    const uint32_t smem = Layout::make<D>(p.clip_k).bytes;
    const cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kern), di);
    if (e != cudaSuccess) return e;
    const int grid = di.sms < kMaxGrid ? di.sms : kMaxGrid;
    kern<<<grid, kThreads, smem, s>>>(p);
    const cudaError_t le = cudaGetLastError();
    if (le != cudaSuccess) return le;
    return launch_merge(p, grid, true, s);
}

template <int D>
cudaError_t launch_d(const PagedArgs &a, cudaStream_t s) {
    Params p;
    fill_params(a, &p);
    p.T = kRows / p.g;
    p.T1 = p.T;
    p.c0 = D == 64 ? 2 : 1;   // joining the warps costs about a tile's time at d = 128
    p.wt = p.wt2 = 1;
    p.rec_rows = kRows;
    if (a.aK && a.aV) return launch_variant<D, true, true>(p, s);
    if (a.aK) return launch_variant<D, true, false>(p, s);
    if (a.aV) return launch_variant<D, false, true>(p, s);
    return launch_variant<D, false, false>(p, s);
}

}  // namespace
}  // namespace paged

bool paged_decode_covers(const PagedArgs &a) {
    if (!a.bf16 || (a.d != 64 && a.d != 128) || a.page_size < 8) return false;
    const int g = a.H / a.Hkv;
    if (a.max_new < 1 || (long long)a.max_new * g > paged::kRows) return false;
    return paged::wide_rows(a);
}

cudaError_t launch_paged_decode(const PagedArgs &a, cudaStream_t s) {
    return a.d == 64 ? paged::launch_d<64>(a, s) : paged::launch_d<128>(a, s);
}

}  // namespace relattn
