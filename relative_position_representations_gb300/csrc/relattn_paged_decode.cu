// Paged attention for few query rows per key/value head (generated tokens: T tokens x g heads
// <= 16 rows), bf16, d = 64 or 128, pages of at least 8 keys.
//
// Every cached key and value is read once and meets at most 16 rows, so HBM bounds the kernel:
// 4 d bytes per key against 64 d multiply-adds. The rows are the narrow side (N = 8 or 16) of
// m16n8k16 products whose wide side are the keys (S^T = K Q^T) and the columns (O^T = V^T P^T); a
// 128-row tcgen05 tile would be padding for the most part and would need the keys staged for the
// async proxy, and at these sizes the products take a tenth of the time that the bytes take.
//
// A tile of 128 keys is 16 keys for each of a CTA's 8 warps; each warp keeps its own running
// maximum, sum and output over its keys, and the warps are joined once per piece. Loads run
// through a ring of kStages groups of 16 keys per warp by 16-byte cp.async. The ring is private
// to each lane: the lane copies exactly the 16-byte chunks that its own fragments need and reads
// them back itself, so the loop has no barrier, no swizzle and no transposition:
//   S^T: the order of the contracted columns is free, so lane (key l / 4, c = l % 4) takes columns
//     32 s + 8 c .. + 7 of its keys as the k-slots of two MMA steps, and Q alike;
//   O^T: the lane takes columns 64 u + 8 (l / 4) .. + 7 of keys 2 c, 2 c + 1 (+ 8) and pairs two
//     keys by byte permutes; P^T comes out of S^T's accumulators by two 8 x 8 transpositions.
//     A lane's outputs are then 8 consecutive columns of rows 2 c, 2 c + 1.
// The ring runs ahead over the ends of the pieces (a second walk over the CTA's range issues the
// loads), so joining the warps costs no bandwidth while it is shorter than the ring.
//
// Relative terms: R = Q aK^T (k + 1 rows) once per piece by the same MMA; keys at most k - 1
// back add their own R entry and leave their score in a bin; the other keys share entry 0 and
// their weights are summed. At the end of the piece each warp adds 16 rows' beta_r aV_r at a time.
#include <cstdint>

#include "relattn_paged.cuh"
#include "sm103_ptx.cuh"

namespace relattn {
namespace paged {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 16;               // keys of a warp per tile
constexpr int kStages = 2;
static_assert(kWarps * kGroup == kTile, "a tile is one group per warp");

// D = 64 holds half the bytes per key in a group: two CTAs share an SM (their joins overlap)
template <int D>
constexpr int kCtasPerSm = D == 64 ? 2 : 1;
template <int D>
constexpr int kStageBytes = 2 * kGroup * D * 2;   // one warp's group: K and V

struct Layout {
    uint32_t o, ml, R, Bn, bytes;        // byte offsets behind the ring
    int lw;
    template <int D, int NT>
    static __host__ __device__ Layout make(int clip_k, bool tables) {
        Layout L;
        constexpr int rows = 8 * NT;
        L.lw = tables ? (clip_k + 1) | 1 : 0;
        uint32_t off = (uint32_t)kWarps * kStages * kStageBytes<D>;
        L.o = off;  off += kWarps * rows * D * 4;
        L.ml = off; off += kWarps * rows * 4 * 4;
        L.R = off;  off += rows * L.lw * 4;
        L.Bn = off; off += rows * L.lw * 4;
        L.bytes = off;
        return L;
    }
};

// The joined outputs: 16-byte chunk `ch` of row `row`, swizzled so that the fragments' stores of
// neighbouring rows fall in different banks
template <int D, int NT>
__device__ __forceinline__ int out_at(int warp, int row, int ch) {
    return (warp * 8 * NT + row) * D + ((ch ^ (row & 6)) << 2);
}

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
// transposes an 8 x 8 matrix of 16-bit elements, lane l holding row l / 4, columns 2 (l % 4), + 1
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// The groups that a warp gets over the CTA's range, one per call: tile after tile of piece after
// piece. `pg` holds the page numbers of the next group's two halves (8 keys each), loaded one
// call ahead so that the copies do not wait for the table.
template <int D>
struct Feed {
    Walk walk;
    bool more;
    int t, t1, ns, lo;           // next tile of the piece, its end; Item::tile
    int pos_hi, first;           // keys that some row sees: <= pos_hi and (>= first or < sinks)
    const int *bt;
    long long head;              // element offset of the head within a page
    int pg[2], j0;               // of the next group
    __device__ __forceinline__ Feed(const Params &p, const Range &r) : walk(p, r), more(true), t(0), t1(0) {}
    __device__ __forceinline__ bool seen(const Params &p, int j) const {
        return j <= pos_hi && (j >= first || j < p.sinks);
    }
    __device__ __forceinline__ void advance(const Params &p, int warp) {
        if (++t >= t1) {
            Segment g;
            do {
                if (!walk.next_call(p, g)) {
                    more = false;
                    return;
                }
            } while (g.t0 >= g.t1);
            t = g.t0;
            t1 = g.t1;
            ns = g.it.ns;
            lo = g.it.lo - g.it.ns;
            pos_hi = g.it.pos_hi;
            first = p.window > 0 ? max(0, max(g.it.pos_lo, 0) - p.window + 1) : 0;
            bt = p.bt + (long long)g.b * p.bt_stride;
            head = ((long long)g.kvh << p.pshift) * D;
        }
        j0 = (t < ns ? t : lo + t) * kTile + warp * kGroup;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = j0 + 8 * h;
            // -2: nothing to load; -1 (or a number past the cache): no such page
            pg[h] = j <= pos_hi && (j + 8 > first || j < p.sinks) ? max(-1, __ldg(bt + (j >> p.pshift))) : -2;
        }
    }
    // issues the copies of the next group into ring stage `dst` (this lane's address)
    __device__ __forceinline__ void issue(const Params &p, uint32_t dst, int lane) {
        const int pm = (1 << p.pshift) - 1;
        const int c = lane & 3, rq = lane >> 2;
        const char *base[2];
        bool ok[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ok[h] = (unsigned)pg[h] < (unsigned)p.num_pages;
            if (!ok[h] && pg[h] != -2 && lane == 0) report_page(p);
            const long long off = ok[h] ? pg[h] * p.page_stride + head + ((j0 + 8 * h) & pm) * D : 0;
            base[h] = static_cast<const char *>(p.k) + 2 * off;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool on = ok[h] && seen(p, j0 + 8 * h + rq);
            const char *src = base[h] + (rq * D + 8 * c) * 2;
#pragma unroll
            for (int s = 0; s < D / 32; ++s) cp16(dst + (h * (D / 32) + s) * 512, src + 64 * s, on);
        }
        dst += (D / 16) * 512;
        const long long dv = static_cast<const char *>(p.v) - static_cast<const char *>(p.k);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const char *src = base[h] + dv + (2 * c * D + 8 * rq) * 2;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool on = ok[h] && seen(p, j0 + 8 * h + 2 * c + e);
#pragma unroll
                for (int u = 0; u < D / 64; ++u)
                    cp16(dst + ((2 * h + e) * (D / 64) + u) * 512, src + e * D * 2 + 128 * u, on);
            }
        }
    }
};

template <int D, int NT, bool AK, bool AV>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<D>) paged_decode_kernel(const __grid_constant__ Params p) {
    constexpr int kRows = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scr[80];
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int c = lane & 3, rq = lane >> 2;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Range rg = find_range<kThreads>(p, scr);
    const Layout L = Layout::make<D, NT>(p.clip_k, AK || AV);
    const uint32_t ring = ptx::smem_u32(smem) + (uint32_t)warp * kStages * kStageBytes<D> + lane * 16;
    float *so = reinterpret_cast<float *>(smem + L.o);
    float4 *sml = reinterpret_cast<float4 *>(smem + L.ml);   // {m, l, far, -} of [warp][row]
    float *Rs = reinterpret_cast<float *>(smem + L.R), *Bs = reinterpret_cast<float *>(smem + L.Bn);
    const int k = p.clip_k, W = k + 1;

    // ---- fill the ring
    Feed<D> feed(p, rg);
    feed.advance(p, warp);
#pragma unroll 1
    for (int s = 0; s < kStages; ++s) {
        if (feed.more) {
            feed.issue(p, ring + s * kStageBytes<D>, lane);
            feed.advance(p, warp);
        }
        cp_commit();
    }
    uint32_t stage = 0;

    Walk walk(p, rg);
    Segment g{};
    bool any = false;
    while (walk.next_call(p, g)) {
        any = true;
        const int rows = g.it.cnt * p.g;
        const int pos_lo = g.it.pos_lo, pos_hi = g.it.pos_hi;
        // ---- Q fragments: lane (row rq, columns 32 s + 8 c .. + 7); positions of rows 2 c, 2 c + 1
        uint4 qf[NT][D / 32];
        int pos[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + rq;
            const int tok = r / p.g, hh = r - tok * p.g;
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) +
                                     (long long)(g.s.q0 + g.it.i0 + tok) * p.q_stride +
                                     (long long)(g.kvh * p.g + hh) * D + 8 * c;
#pragma unroll
            for (int s = 0; s < D / 32; ++s)
                qf[n][s] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(q + 32 * s)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = 8 * n + 2 * c + e;
                pos[n][e] = pos_lo + (rr < rows ? rr / p.g : 0);
            }
        }
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
            for (int i = tid; i < kRows * L.lw; i += kThreads) Bs[i] = -INFINITY;
        if (AK || AV) __syncthreads();
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
        // O^T += A^T B over 16 keys (or table rows): chunks v of rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9
        auto outputs = [&](const uint4 (&v)[4], int u, const uint32_t (&b)[NT][2]) {
            const uint32_t *v0 = reinterpret_cast<const uint32_t *>(&v[0]), *v1 = reinterpret_cast<const uint32_t *>(&v[1]);
            const uint32_t *v2 = reinterpret_cast<const uint32_t *>(&v[2]), *v3 = reinterpret_cast<const uint32_t *>(&v[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a0 = __byte_perm(v0[i], v1[i], 0x5410), a1 = __byte_perm(v0[i], v1[i], 0x7632);
                const uint32_t a2 = __byte_perm(v2[i], v3[i], 0x5410), a3 = __byte_perm(v2[i], v3[i], 0x7632);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma(o[n][4 * u + i], a0, a1, a2, a3, b[n][0], b[n][1]);
            }
        };

#pragma unroll 1
        for (int t = g.t0; t < g.t1; ++t) {
            const int j0 = g.it.tile(t) * kTile + warp * kGroup;
            const uint32_t st = ring + stage * kStageBytes<D>;
            stage ^= 1u;
            static_assert(kStages == 2, "the ring's position is one bit");
            cp_wait<kStages - 1>();
            float x[NT][4] = {};
#pragma unroll
            for (int s = 0; s < D / 32; ++s) scores(x, lds128(st + s * 512), lds128(st + (D / 32 + s) * 512), s);
            // ---- logits in the log2 domain
            const bool near = j0 + kGroup - 1 > pos_lo - k;   // some key has a table row of its own
            const bool full = j0 + kGroup - 1 <= pos_lo &&
                              (p.window == 0 || j0 > pos_hi - p.window || j0 + kGroup <= p.sinks);
            if (AK && near) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int lab = min(max(j0 + rq + 8 * (e >> 1) - pos[n][e & 1], -k) + k, k);
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
                        const int j = j0 + rq + 8 * (e >> 1), q = pos[n][e & 1];
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
            uint32_t b[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float pr[4];
                const float mu[2] = {m[n][0] == -INFINITY ? 0.f : m[n][0], m[n][1] == -INFINITY ? 0.f : m[n][1]};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pr[e] = ptx::ex2(x[n][e] - mu[e & 1]);
                    l[n][e & 1] += pr[e];
                }
                if (AV) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int lab = j0 + rq + 8 * (e >> 1) - pos[n][e & 1] + k;
                        if (near && lab > 0) {
                            if (lab <= k) Bs[(8 * n + 2 * c + (e & 1)) * L.lw + lab] = x[n][e];
                        } else {
                            far[n][e & 1] += pr[e];
                        }
                    }
                }
                // P rounded to bf16 for the tensor cores; the sums above keep fp32
                b[n][0] = transpose8(ptx::pack_bf16x2(pr[0], pr[1]));
                b[n][1] = transpose8(ptx::pack_bf16x2(pr[2], pr[3]));
            }
            const uint32_t sv = st + (D / 16) * 512;
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                uint4 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = lds128(sv + (e * (D / 64) + u) * 512);
                outputs(v, u, b);
            }
            // ---- the stage is free: the group kStages ahead
            if (feed.more) {
                feed.issue(p, st, lane);
                feed.advance(p, warp);
            }
            cp_commit();
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
        __syncthreads();
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
            const __nv_bfloat16 *aV = static_cast<const __nv_bfloat16 *>(p.aV) + (long long)g.kvh * p.ths + 8 * rq;
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
                uint32_t b[NT][2];
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
                    b[n][0] = ptx::pack_bf16x2(be[0], be[1]);
                    b[n][1] = ptx::pack_bf16x2(be[2], be[3]);
                }
#pragma unroll
                for (int u = 0; u < D / 64; ++u) outputs(v[u], u, b);
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
                            *reinterpret_cast<float4 *>(so + out_at<D, NT>(warp, row, 16 * u + 2 * rq + i / 2)) =
                                make_float4(o[n][4 * u + i][e], o[n][4 * u + i][2 + e], o[n][4 * u + i + 1][e],
                                            o[n][4 * u + i + 1][2 + e]);
                }
            }
        __syncthreads();
        const bool whole = g.whole();
        float *rec = whole ? nullptr : record(p, blockIdx.x, g.record());
        // four columns a thread
        for (int i = tid; i < rows * (D / 4); i += kThreads) {
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
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                                     ((long long)(g.s.q0 + g.it.i0 + tok) * p.H + g.kvh * p.g + hh) * D + 4 * ch;
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
        __syncthreads();   // the next piece writes the shared arrays
    }
    cp_wait<0>();
    if (tid == 0) write_desc(p, any ? &g : nullptr, rg.total);
}

template <int D, int NT, bool AK, bool AV>
cudaError_t launch_variant(const Params &p, cudaStream_t s) {
    auto kern = paged_decode_kernel<D, NT, AK, AV>;
    const DeviceInfo di = device_info();
    if (di.sms <= 0) return cudaErrorInvalidDevice;
    const uint32_t smem = Layout::make<D, NT>(p.clip_k, AK || AV).bytes;
    const cudaError_t e = opt_in_smem(reinterpret_cast<const void *>(kern), di);
    if (e != cudaSuccess) return e;
    const int want = di.sms * kCtasPerSm<D>;
    const int grid = want < kMaxGrid ? want : kMaxGrid;
    kern<<<grid, kThreads, smem, s>>>(p);
    const cudaError_t le = cudaGetLastError();
    if (le != cudaSuccess) return le;
    return launch_merge(p, grid, true, s);
}

template <int D, int NT>
cudaError_t launch_rows(const PagedArgs &a, cudaStream_t s) {
    Params p;
    fill_params(a, &p);
    p.T = 8 * NT / p.g;
    p.T1 = p.T;
    p.c0 = 1;   // joining the warps costs about a tile's time
    p.wt = p.wt2 = 1;
    p.rec_rows = 8 * NT;
    if (a.aK && a.aV) return launch_variant<D, NT, true, true>(p, s);
    if (a.aK) return launch_variant<D, NT, true, false>(p, s);
    if (a.aV) return launch_variant<D, NT, false, true>(p, s);
    return launch_variant<D, NT, false, false>(p, s);
}

constexpr int kMostRows = 16;

}  // namespace
}  // namespace paged

bool paged_decode_covers(const PagedArgs &a) {
    if (!a.bf16 || (a.d != 64 && a.d != 128) || a.page_size < 8) return false;
    const int g = a.H / a.Hkv;
    if (a.max_new < 1 || (long long)a.max_new * g > paged::kMostRows) return false;
    return paged::wide_rows(a);
}

cudaError_t launch_paged_decode(const PagedArgs &a, cudaStream_t s) {
    const bool eight = (long long)a.max_new * (a.H / a.Hkv) <= 8;
    if (a.d == 64) return eight ? paged::launch_rows<64, 1>(a, s) : paged::launch_rows<64, 2>(a, s);
    return eight ? paged::launch_rows<128, 1>(a, s) : paged::launch_rows<128, 2>(a, s);
}

}  // namespace relattn
