// paged_estimate.cu -- page selection for every new token from the key bounds of
// the stored pages.
//
// With min_jc <= k_c <= max_jc for every key k of page j, no key of the page has a
// larger q . k than sum_c max(q_c min_jc, q_c max_jc).  Summed over a kv-head's
// query heads g that is linear in the bounds,
//     score(j) = sum_c Q+_c max_jc + Q-_c min_jc,
//     Q+_c = sum_g max(q_gc, 0),  Q-_c = sum_g min(q_gc, 0),
// one 256-long dot product per (token, kv-head, page) whatever the group.  A token
// keeps its own page and the topk - 1 best earlier ones, ties to the lower page.
//
// Two kernels:
//   scores  bound by reading the bounds (512 B per page and kv-head) for single
//           tokens, by the matrix instructions for chunks.  16 pages are the rows
//           of an m16n8k16 product; each warp brings its own pages in through a ring
//           of bulk copies, one per page, at a stride of 528 B that ldmatrix reads
//           without bank conflicts.  The columns are four tokens' Q, each as the sum
//           of two 16-bit parts, which carries Q to 2^-16.  The scores are
//           approximate, with a bound E on their error.
//   select  one warp (many rows) or one CTA (few) per row: the k-th largest
//           approximate score t by counting over a shrinking range of its key bits
//           until few keys are left, which are ranked; then every page within 2 E of
//           t is scored again in 64 bits; all others are decided by the
//           approximation.  So the selection is that of exact scores.
// E = (2^-15 + G 2^-23) |Q|_1 max|bound|: the two-part split of bf16 loses 2^-16
// (fp16's less), sixteen accumulation steps at 2^-22 of the magnitudes each lose
// 2^-18, the sums Q lose G 2^-24; 1.6 times their sum, since the instruction's
// rounding is not documented.
#include <algorithm>

#include "internal.h"
#include "paged.cuh"

namespace minf {

namespace {

constexpr int kStepPages = 16;
constexpr uint32_t kPageBytes = 512;   // bounds of a page for one kv-head
constexpr uint32_t kPageStride = 528;  // in shared memory
constexpr uint32_t kStepBytes = kStepPages * kPageStride;

// Power of two that brings |x| <= top to 2^14 at most (fp16 parts; 1 for bf16).
template <class Ty>
__device__ __forceinline__ float part_scale(float top);
template <>
__device__ __forceinline__ float part_scale<Bf16>(float) {
    return 1.f;
}
template <>
__device__ __forceinline__ float part_scale<Fp16>(float top) {
    if (!(top > 0.f)) return 1.f;
    int e;
    frexpf(top, &e);  // top < 2^e
    return ldexpf(1.f, min(14 - e, 100));
}

// Q+ and Q- of channels 8 c .. 8 c + 7 of a token, fp32 (all terms of one sign).
template <class Ty>
__device__ __forceinline__ void q_sums(const EstimateParams &P, int tok, int h, int c, float (&up)[8], float (&down)[8]) {
    const typename Ty::T *q = static_cast<const typename Ty::T *>(P.q) + (long long)tok * P.q_ts +
                              (long long)h * P.group * P.q_hs + c * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) up[i] = down[i] = 0.f;
#pragma unroll 4
    for (int g = 0; g < P.group; ++g) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(q + (long long)g * P.q_hs));
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Ty::unpack(x[i]);
            up[2 * i] += fmaxf(f.x, 0.f);
            up[2 * i + 1] += fmaxf(f.y, 0.f);
            down[2 * i] += fminf(f.x, 0.f);
            down[2 * i + 1] += fminf(f.y, 0.f);
        }
    }
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// ------------------------------------------------------------------ scores
// grid: x = sequence * tiles + token tile, y = kv-head, z = page range.
template <int NT>
struct ScoreShape {
    static constexpr int kWarps = NT == 1 ? 6 : 4, kThreads = 32 * kWarps, kStages = 2;
    static constexpr uint32_t kRing = kWarps * kStages * kStepBytes;
    static constexpr uint32_t kFrag = NT * 8 * 32 * 16;
    static constexpr uint32_t kBytes = kRing + kFrag + 192;
};

template <class Ty, int NT>
__global__ void __launch_bounds__(ScoreShape<NT>::kThreads, 2)
    paged_scores_kernel(const __grid_constant__ EstimateParams P) {
    using T = typename Ty::T;
    using Shape = ScoreShape<NT>;
    constexpr int kTok = 4 * NT, kStages = Shape::kStages, kWarps = Shape::kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    uint4 *qf = reinterpret_cast<uint4 *>(smem + Shape::kRing);  // column fragments [NT][8][32]
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Shape::kRing + Shape::kFrag);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + kWarps * kStages);
    float *warp_top = reinterpret_cast<float *>(bars + kWarps * kStages + 1);
    const PagedSeqs &S = P.seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int s = blockIdx.x / P.tiles, h = blockIdx.y;
    const SeqView v = seq_view(S, s, P.hdr);
    const int ta = max(v.q0, P.t0) + (int)(blockIdx.x % P.tiles) * kTok;
    const int tb = min(min(v.q0 + v.n, P.t1), ta + kTok);
    if (ta >= tb) return;
    // pages before the last token's own
    const int last_pos = v.len - v.n + (tb - 1 - v.q0);
    const int n_pages = last_pos < 0 ? 0 : last_pos >> S.page_log2;
    const int pa = blockIdx.z * P.pages_per_cta, pb = min(pa + P.pages_per_cta, n_pages);
    if (pa >= pb) return;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * kStages; ++i) mbar_init(smem_u32(bars + i), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    const WaitCtl wc{abort_flag, &P.hdr->status, P.wait_limit_ns};

    // this warp's ring: 16 pages a stage, one copy per lane
    constexpr int kStride = kWarps * kStepPages;
    const uint32_t ring = smem_u32(smem) + warp * kStages * kStepBytes, bar0 = smem_u32(bars + warp * kStages);
    const T *kb = static_cast<const T *>(P.bounds) + (long long)h * 2 * kD;
    const long long page_stride = (long long)P.hkv * 2 * kD;
    auto id_at = [&](int j0) -> int { return lane < kStepPages && j0 + lane < pb ? page_of(S, s, j0 + lane, P.hdr) : -1; };
    auto fill = [&](int st, int id) {
        const int n = __popc(__ballot_sync(0xffffffffu, id >= 0));
        if (lane == 0) mbar_arrive_expect_tx(bar0 + st * 8, (uint32_t)n * kPageBytes);
        __syncwarp();
        if (id >= 0) bulk_copy(ring + st * kStepBytes + lane * kPageStride, kb + id * page_stride, kPageBytes, bar0 + st * 8);
    };
    const int first = pa + warp * kStepPages;
    int id[kStages + 1];
#pragma unroll
    for (int st = 0; st <= kStages; ++st) id[st] = id_at(first + st * kStride);
    int id_next = id[kStages];
#pragma unroll
    for (int st = 0; st < kStages; ++st)
        if (first + st * kStride < pb) fill(st, id[st]);

    // column fragments: column n of tile nt is part n & 1 of token 4 nt + n / 2; sixteen
    // threads a token, 8 channels each, element = side * 128 + channel
    {
        constexpr int kPass = Shape::kThreads / 16;
        const int ch = threadIdx.x & 15;
#pragma unroll
        for (int x0 = 0; x0 < (kTok + kPass - 1) / kPass; ++x0) {
            const int x = x0 * kPass + (threadIdx.x >> 4);
            if (x >= kTok) break;  // whole warps: kTok is a multiple of 4
            float up[8] = {}, down[8] = {};
            if (ta + x < tb) q_sums<Ty>(P, ta + x, h, ch, up, down);
            float sc = 1.f;
            if (Ty::kIdescType == 0) {  // fp16: scaled by the row's largest
                float mx = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fmaxf(up[i], -down[i]));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                sc = part_scale<Ty>(mx);
            }
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                // element e = side * 128 + 8 ch + 2 p: k-step e / 16, register (e / 8) % 2, lane column p
                const int kk = side * 8 + (ch >> 1), reg = (kk & 1) * 2 + (ch & 1);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float a = (side ? up : down)[2 * p] * sc, b = (side ? up : down)[2 * p + 1] * sc;
                    const uint32_t hi = Ty::pack(a, b);
                    const float2 f = Ty::unpack(hi);
                    const uint32_t mid = Ty::pack(a - f.x, b - f.y);
                    uint32_t *w = reinterpret_cast<uint32_t *>(qf + ((x >> 2) * 8 + (kk >> 1)) * 32);
                    w[((2 * (x & 3)) * 4 + p) * 4 + reg] = hi;
                    w[((2 * (x & 3) + 1) * 4 + p) * 4 + reg] = mid;
                }
            }
        }
    }
    __syncthreads();

    int st = 0;
    uint32_t phase = 0;
    // No key exceeds its page's max nor falls below its min, so the largest |bound| is
    // the largest max or the largest -min.
    uint32_t hi2 = Ty::kNegInf2, lo2 = Ty::kPosInf2;
    const uint32_t row_addr = ring + (lane & 15) * kPageStride + (lane >> 4) * 16;
    for (int j0 = first; j0 < pb; j0 += kStride) {
        const bool got = wait_bounded(bar0 + st * 8, (phase >> st) & 1, wc, wait_site(8, st, j0));
        if (__any_sync(0xffffffffu, !got)) {  // let the copies in flight land before the CTA exits
            volatile int no_abort = 0;
            const WaitCtl drain{&no_abort, nullptr, 50000000ull};
            for (int x = 0; x < kStages; ++x)
                if (j0 + x * kStride < pb) wait_bounded(bar0 + ((st + x) % kStages) * 8, (phase >> ((st + x) % kStages)) & 1, drain);
            break;
        }
        phase ^= 1u << st;
        uint32_t a[16][4];
#pragma unroll
        for (int kk = 0; kk < 16; ++kk) ldmatrix4(a[kk], row_addr + st * kStepBytes + kk * 32);
        __syncwarp();  // every lane has read the stage
        if (j0 + kStages * kStride < pb) {
            fill(st, id_next);
            id_next = id_at(j0 + (kStages + 1) * kStride);
        }
        st = st == kStages - 1 ? 0 : st + 1;
        const bool r0 = j0 + r < pb, r1 = j0 + r + 8 < pb;  // rows behind the range hold anything
        uint32_t h0 = Ty::kNegInf2, h1 = Ty::kNegInf2, l0 = Ty::kPosInf2, l1 = Ty::kPosInf2;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            l0 = Ty::vmin(l0, Ty::vmin(a[kk][0], a[kk][2]));
            l1 = Ty::vmin(l1, Ty::vmin(a[kk][1], a[kk][3]));
            h0 = Ty::vmax(h0, Ty::vmax(a[8 + kk][0], a[8 + kk][2]));
            h1 = Ty::vmax(h1, Ty::vmax(a[8 + kk][1], a[8 + kk][3]));
        }
        if (r0) {
            lo2 = Ty::vmin(lo2, l0);
            hi2 = Ty::vmax(hi2, h0);
        }
        if (r1) {
            lo2 = Ty::vmin(lo2, l1);
            hi2 = Ty::vmax(hi2, h1);
        }
        // two token tiles at a time: four chains of products
        constexpr int kPair = NT == 1 ? 1 : 2;
#pragma unroll
        for (int t = 0; t < NT; t += kPair) {
            if (4 * t < tb - ta) {
                float d[kPair][2][4] = {};
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int y = 0; y < kPair; ++y) {
                        const uint4 b = qf[((t + y) * 8 + i) * 32 + lane];
                        Ty::mma(d[y][0], a[2 * i][0], a[2 * i][1], a[2 * i][2], a[2 * i][3], b.x, b.y);
                        Ty::mma(d[y][1], a[2 * i + 1][0], a[2 * i + 1][1], a[2 * i + 1][2], a[2 * i + 1][3], b.z, b.w);
                    }
#pragma unroll
                for (int y = 0; y < kPair; ++y) {
                    const int tok = ta + 4 * (t + y) + c;
                    if (tok < tb) {
                        float *dst = P.scores + ((long long)(tok - P.t0) * P.hkv + h) * P.score_stride + j0 + r;
                        if (r0) dst[0] = (d[y][0][0] + d[y][1][0]) + (d[y][0][1] + d[y][1][1]);
                        if (r1) dst[8] = (d[y][0][2] + d[y][1][2]) + (d[y][0][3] + d[y][1][3]);
                    }
                }
            }
        }
    }
    // largest |bound| of this tile's page range
    {
        const float2 fh = Ty::unpack(hi2), fl = Ty::unpack(lo2);
        float top = fmaxf(fmaxf(fh.x, fh.y), fmaxf(-fl.x, -fl.y));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) warp_top[warp] = top;
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, warp_top[w]);
            P.top[((long long)blockIdx.x * P.hkv + h) * gridDim.z + blockIdx.z] = fmaxf(top, 0.f);
        }
    }
    launch_dependents();
}

// ------------------------------------------------------------------ select
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);  // -0 counts as +0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long order_key64(double x) {
    const unsigned long long b = (unsigned long long)__double_as_longlong(x + 0.0);
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// Exact scores of four pages (j < 0: none) by one warp, one in each group of eight
// lanes: 64 bytes of the bounds a lane, every page in the same order.
template <class Ty>
__device__ __forceinline__ double exact_score(const EstimateParams &P, int s, int h, int j, const double *q, int lane) {
    using T = typename Ty::T;
    const int pg = j >= 0 ? page_of(P.seqs, s, j, P.hdr) : -1, l = lane & 7;
    double acc = 0.0;
    if (pg >= 0) {
        const uint4 *b = reinterpret_cast<const uint4 *>(static_cast<const T *>(P.bounds) +
                                                         ((long long)pg * P.hkv + h) * 2 * kD);
        uint4 w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) w[x] = __ldg(b + x * 8 + l);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t v[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = Ty::unpack(v[i]);
                const double2 qq = *reinterpret_cast<const double2 *>(q + (x * 8 + l) * 8 + 2 * i);
                acc = fma((double)f.x, qq.x, acc);
                acc = fma((double)f.y, qq.y, acc);
            }
        }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    return acc;
}

constexpr int kSelectWarps = 8, kSelectThreads = 32 * kSelectWarps;
constexpr int kBins = 512;
constexpr int kBorder = 1024;  // pages a CTA's row ranks in shared memory by their exact scores
constexpr int kWarpBorder = 128;

// One (token, kv-head) row: where its candidates, scores and lists lie.
struct Row {
    int s, tok, h, n, take;  // n candidate pages, take of them wanted; page n is the token's own
    int tile_range0;         // first entry of its tile's page ranges in EstimateParams::top
    const float *sc;
    int *out;
};

// Fills `w` for row `row_in` of the launch and writes what needs no scores; false
// if nothing is left to select.  `tid` of `nt` threads share the work.
__device__ __forceinline__ bool row_setup(const EstimateParams &P, int row_in, int s, int tid, int nt, Row &w) {
    const PagedSeqs &S = P.seqs;
    w.tok = P.t0 + row_in / P.hkv;
    w.h = row_in % P.hkv;
    w.s = s;
    if (s < 0) return false;  // a row behind the last sequence
    const SeqView v = seq_view(S, s, P.hdr);
    if (v.n == 0) return false;
    const int pos = v.len - v.n + (w.tok - v.q0);
    const long long row = (long long)w.tok * P.hkv + w.h;
    w.out = P.blk_idx + row * P.topk;
    if (pos < 0) {  // no key is visible
        for (int i = tid; i < P.topk; i += nt) w.out[i] = -1;
        if (tid == 0) P.blk_cnt[row] = 0;
        return false;
    }
    w.n = pos >> S.page_log2;
    w.take = min(P.topk - 1, w.n);
    for (int i = w.take + 1 + tid; i < P.topk; i += nt) w.out[i] = -1;
    if (tid == 0) {
        w.out[w.take] = w.n;
        P.blk_cnt[row] = w.take + 1;
    }
    if (w.take == w.n) {
        for (int i = tid; i < w.n; i += nt) w.out[i] = i;
        return false;
    }
    if (w.take == 0) return false;
    const int tile = s * P.tiles + (w.tok - max(v.q0, P.t0)) / P.tile_tokens;
    w.tile_range0 = (tile * P.hkv + w.h) * P.ranges;
    w.sc = P.scores + (row - (long long)P.t0 * P.hkv) * P.score_stride;
    return true;
}

__device__ __forceinline__ int seq_of(const PagedSeqs &S, int tok, int s) {
    return s < S.n_seqs && __ldg(S.cu_q + s) <= tok && tok < __ldg(S.cu_q + s + 1) ? s : -1;
}

// Sixteen lanes: Q in 64 bits (8 channels a lane) to q (Q- then Q+), its 1-norm and
// largest element in l1 and mx of each lane (the lane's own share).
template <class Ty>
__device__ __forceinline__ void exact_q(const EstimateParams &P, const Row &w, int lane, double *q, float &l1, float &mx) {
    double up[8] = {}, down[8] = {};
    const typename Ty::T *src = static_cast<const typename Ty::T *>(P.q) + (long long)w.tok * P.q_ts +
                                (long long)w.h * P.group * P.q_hs + lane * 8;
    for (int g = 0; g < P.group; ++g) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + (long long)g * P.q_hs));
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Ty::unpack(x[i]);
            up[2 * i] += (double)fmaxf(f.x, 0.f);
            up[2 * i + 1] += (double)fmaxf(f.y, 0.f);
            down[2 * i] += (double)fminf(f.x, 0.f);
            down[2 * i + 1] += (double)fminf(f.y, 0.f);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[lane * 8 + i] = down[i];
        q[kD + lane * 8 + i] = up[i];
        l1 += (float)(up[i] - down[i]);
        mx = fmaxf(mx, (float)fmax(up[i], -down[i]));
    }
}

// The bound E on a row's score error; the largest element is scaled a hair down, so
// that a sum rounded to the other side of a power of two here cannot make the
// scale, and with it the bound, too small.
template <class Ty>
__device__ __forceinline__ float error_bound(const EstimateParams &P, float l1, float mxq, float top) {
    return (3.0517578125e-5f + 1.1920929e-7f * (float)P.group) * l1 * part_scale<Ty>(mxq * 0.999999f) * top;
}

// Keys around the threshold t whose order the approximation leaves open: 2 E to
// either side (0.1 % wider: the roundings here).
__device__ __forceinline__ void doubt_range(uint32_t t_key, float err, uint32_t &k_lo, uint32_t &k_hi) {
    const float t = from_key(t_key), width = 2.002f * err + 1e-6f * fabsf(t);
    k_lo = order_key(t - width);
    k_hi = order_key(t + width);
}

// Many pages in doubt (repeated pages): counts over the bits of their exact scores,
// computed anew for each byte, with `hist` of 256 bins.  `key(i)` is candidate
// i's key; `mark(i, yes)` takes the decision.  One warp.
template <class Ty, class Key, class Mark>
__device__ __noinline__ void select_many(const EstimateParams &P, const Row &w, const double *q, unsigned *hist,
                                         uint32_t k_lo, uint32_t k_hi, unsigned want, Key key, Mark mark) {
    const int lane = threadIdx.x & 31;
    unsigned long long prefix = 0;
    unsigned left = want;
    for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = lane; i < 256; i += 32) hist[i] = 0;
        __syncwarp();
        for (int i0 = 0; i0 < w.n; i0 += 4) {
            const int i = i0 + (lane >> 3);
            const uint32_t k = i < w.n ? key(i) : 0;
            const bool in = i < w.n && k >= k_lo && k <= k_hi;
            if (!__any_sync(0xffffffffu, in)) continue;
            const unsigned long long x = order_key64(exact_score<Ty>(P, w.s, w.h, in ? i : -1, q, lane));
            if (in && (lane & 7) == 0 && (shift == 56 || (x >> (shift + 8)) == prefix))
                atomicAdd(&hist[(x >> shift) & 255u], 1u);
        }
        __syncwarp();
        unsigned bin = 255, above = 0;
        while (bin > 0 && above + hist[bin] < left) above += hist[bin--];
        left -= above;
        prefix = (prefix << 8) | bin;
        __syncwarp();
    }
    // larger ones are taken, and the first `left` equal ones
    unsigned ties = 0;
    for (int i0 = 0; i0 < w.n; i0 += 4) {
        const int i = i0 + (lane >> 3);
        const uint32_t k = i < w.n ? key(i) : 0;
        const bool in = i < w.n && k >= k_lo && k <= k_hi;
        if (!__any_sync(0xffffffffu, in)) continue;
        const unsigned long long x = order_key64(exact_score<Ty>(P, w.s, w.h, in ? i : -1, q, lane));
        const unsigned same = __ballot_sync(0xffffffffu, in && x == prefix) & 0x01010101u;
        const unsigned before = ties + __popc(same & ((1u << (lane & 24)) - 1u));
        if (in && (lane & 7) == 0) mark(i, x > prefix || (x == prefix && before < left));
        ties += __popc(same);
        __syncwarp();
    }
}

// ---- one warp per row, its keys in registers (candidate 32 e + lane in key[e])
struct alignas(16) WarpShared {
    double q[2 * kD];  // Q- then Q+, read 16 bytes at a time
    union {
        double exact[kWarpBorder];
        unsigned hist[kBins];
    };
    int border[kWarpBorder];
    unsigned chosen[64];  // bit set of the pages in doubt that are taken
    unsigned n_border;
};

template <class Ty, int kPer>
__global__ void __launch_bounds__(kSelectThreads, kPer == 32 ? 3 : 2)
    paged_select_warp_kernel(const __grid_constant__ EstimateParams P) {
    __shared__ WarpShared all[kSelectWarps];
    const int lane = threadIdx.x & 31;
    WarpShared &sh = all[threadIdx.x >> 5];
    const int row_in = blockIdx.x * kSelectWarps + (threadIdx.x >> 5);
    if (row_in >= (P.t1 - P.t0) * P.hkv) return;
    int s = -1;
    for (int s0 = 0; s0 < P.seqs.n_seqs && s < 0; s0 += 32)
        s = __reduce_max_sync(0xffffffffu, seq_of(P.seqs, P.t0 + row_in / P.hkv, s0 + lane));
    Row w;
    if (!row_setup(P, row_in, s, lane, 32, w)) return;
    float l1 = 0.f, mxq = 0.f, top = 0.f;
    if (lane < 16) exact_q<Ty>(P, w, lane, sh.q, l1, mxq);
#pragma unroll
    for (int e = 0; e < 64 / 32; ++e) sh.chosen[e * 32 + lane] = 0;
    wait_for_primary();  // the scores
    const int ranges = (w.n + P.pages_per_cta - 1) / P.pages_per_cta;
    for (int i = lane; i < ranges; i += 32) top = fmaxf(top, P.top[w.tile_range0 + i]);
    uint32_t key[kPer];
    uint32_t kmin = 0xffffffffu, kmax = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) key[e] = e * 32 + lane < w.n ? __float_as_uint(w.sc[e * 32 + lane]) : 0u;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const bool in = e * 32 + lane < w.n;
        key[e] = in ? order_key(__uint_as_float(key[e])) : 0u;  // no number's key is 0
        kmin = in ? min(kmin, key[e]) : kmin;
        kmax = max(kmax, key[e]);
    }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
        mxq = fmaxf(mxq, __shfl_xor_sync(0xffffffffu, mxq, o));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    uint32_t lo = kmin, hi = kmax;
    unsigned need = w.take;
    while (lo < hi) {
        const int shift = max(0, 32 - __clz(hi - lo) - 9);
        const uint32_t range = hi - lo;
#pragma unroll
        for (int i = 0; i < kBins / 32; ++i) sh.hist[i * 32 + lane] = 0;
        if (lane == 0) sh.n_border = 0;
        __syncwarp();
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            if (key[e] - lo <= range) atomicAdd(&sh.hist[(key[e] - lo) >> shift], 1u);
        __syncwarp();
        // lane's bins: 16 from the top down
        unsigned mine[kBins / 32], sum = 0;
#pragma unroll
        for (int i = 0; i < kBins / 32; ++i) {
            mine[i] = sh.hist[kBins - 1 - (i + lane * (kBins / 32))];
            sum += mine[i];
        }
        unsigned inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        unsigned before = inc - sum, bin = 0, above = 0, size = 0;
#pragma unroll
        for (int i = 0; i < kBins / 32; ++i) {
            if (before < need && need <= before + mine[i]) {
                bin = kBins - 1 - (i + lane * (kBins / 32));
                above = before;
                size = mine[i];
            }
            before += mine[i];
        }
        const int at = __ffs(__ballot_sync(0xffffffffu, size > 0)) - 1;
        bin = __shfl_sync(0xffffffffu, bin, at);
        need -= __shfl_sync(0xffffffffu, above, at);
        size = __shfl_sync(0xffffffffu, size, at);
        lo += bin << shift;
        hi = min(hi, lo + ((1u << shift) - 1));
        if (lo < hi && size <= 32) {  // rank the few that are left, one to a lane
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (key[e] - lo <= hi - lo) sh.border[atomicAdd(&sh.n_border, 1u)] = (int)key[e];
            __syncwarp();
            const uint32_t k = lane < (int)size ? (uint32_t)sh.border[lane] : 0u;
            unsigned more = 0, same = 0;
            for (unsigned j = 0; j < size; ++j) {
                const uint32_t y = __shfl_sync(0xffffffffu, k, j);
                more += y > k;
                same += y == k;
            }
            const bool me = lane < (int)size && more < need && need <= more + same;
            lo = hi = __shfl_sync(0xffffffffu, k, __ffs(__ballot_sync(0xffffffffu, me)) - 1);
        }
        __syncwarp();
    }
    uint32_t k_lo, k_hi;
    doubt_range(lo, error_bound<Ty>(P, l1, mxq, top), k_lo, k_hi);
    k_lo = max(k_lo, 1u);
    unsigned n_hi = 0, n_in = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        n_hi += key[e] > k_hi;
        n_in += key[e] >= k_lo;
    }
    n_hi = __reduce_add_sync(0xffffffffu, n_hi);
    n_in = __reduce_add_sync(0xffffffffu, n_in) - n_hi;
    const unsigned want = w.take - n_hi;  // of the pages in doubt
    const bool open = n_in != want;
    if (open) {
        if (lane == 0) sh.n_border = 0;
        __syncwarp();
        if (n_in <= kWarpBorder) {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (key[e] - k_lo <= k_hi - k_lo) sh.border[atomicAdd(&sh.n_border, 1u)] = e * 32 + lane;  // any order
            __syncwarp();
            for (unsigned i0 = 0; i0 < n_in; i0 += 4) {
                const unsigned i = i0 + (lane >> 3);
                const double x = exact_score<Ty>(P, w.s, w.h, i < n_in ? sh.border[i] : -1, sh.q, lane);
                if ((lane & 7) == 0 && i < n_in) sh.exact[i] = x;
            }
            __syncwarp();
            for (unsigned i = lane; i < n_in; i += 32) {
                const unsigned long long x = order_key64(sh.exact[i]);
                const int xi = sh.border[i];
                unsigned rank = 0;
                for (unsigned j = 0; j < n_in; ++j) {
                    const unsigned long long y = order_key64(sh.exact[j]);
                    rank += y > x || (y == x && sh.border[j] < xi);
                }
                if (rank < want) atomicOr(&sh.chosen[xi >> 5], 1u << (xi & 31));
            }
        } else {
            select_many<Ty>(
                P, w, sh.q, sh.hist, k_lo, k_hi, want, [&](int i) { return order_key(w.sc[i]); },
                [&](int i, bool yes) {
                    if (yes) atomicOr(&sh.chosen[i >> 5], 1u << (i & 31));
                });
        }
        __syncwarp();
    }
    unsigned to = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const bool doubt = key[e] >= k_lo && key[e] <= k_hi;
        const bool yes = key[e] > k_hi || (doubt && (!open || (sh.chosen[e] >> lane) & 1u));
        const unsigned bal = __ballot_sync(0xffffffffu, yes);
        const unsigned at = to + __popc(bal & ((1u << lane) - 1u));
        if (yes && at < (unsigned)w.take) w.out[at] = e * 32 + lane;
        to += __popc(bal);
    }
}

// ---- one CTA per row, its keys in shared memory
struct alignas(16) SelectShared {
    double q[2 * kD];  // Q- then Q+, read 16 bytes at a time
    union {  // the counting is over where the others are used
        double exact[kBorder];
        unsigned hist[kBins];
    };
    int border[kBorder];
    unsigned part[kSelectWarps][4];
    unsigned bin, above, n_border;
    float l1, mxq;
    int seq;
};

// Sum over the block of one unsigned per thread; the exclusive prefix is returned.
__device__ __forceinline__ unsigned block_prefix(unsigned x, unsigned &total, SelectShared &sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) sh.part[warp][0] = inc;
    __syncthreads();
    unsigned before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kSelectWarps; ++w) {
        if (w < warp) before += sh.part[w][0];
        total += sh.part[w][0];
    }
    return before + inc - x;
}

template <class Ty>
__global__ void __launch_bounds__(kSelectThreads) paged_select_kernel(const __grid_constant__ EstimateParams P) {
    extern __shared__ uint32_t keys[];  // [candidates]
    __shared__ SelectShared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    if (tid == 0) sh.seq = -1;
    __syncthreads();
    for (int s = tid; s < P.seqs.n_seqs; s += kSelectThreads)
        if (seq_of(P.seqs, P.t0 + (int)blockIdx.x / P.hkv, s) >= 0) atomicMax(&sh.seq, s);
    __syncthreads();
    Row w;
    if (!row_setup(P, blockIdx.x, sh.seq, tid, kSelectThreads, w)) return;
    if (warp == 0) {
        float l1 = 0.f, mxq = 0.f;
        if (lane < 16) exact_q<Ty>(P, w, lane, sh.q, l1, mxq);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            l1 += __shfl_xor_sync(0xffffffffu, l1, o);
            mxq = fmaxf(mxq, __shfl_xor_sync(0xffffffffu, mxq, o));
        }
        if (lane == 0) {
            sh.l1 = l1;
            sh.mxq = mxq;
        }
    }
    wait_for_primary();  // the scores
    float top = 0.f;
    const int ranges = (w.n + P.pages_per_cta - 1) / P.pages_per_cta;
    for (int i = tid; i < ranges; i += kSelectThreads) top = fmaxf(top, P.top[w.tile_range0 + i]);
    unsigned kmin = 0xffffffffu, kmax = 0;
#pragma unroll 8
    for (int i = tid; i < w.n; i += kSelectThreads) {
        const uint32_t k = order_key(w.sc[i]);
        keys[i] = k;
        kmin = min(kmin, k);
        kmax = max(kmax, k);
    }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    unsigned topb = __reduce_max_sync(0xffffffffu, __float_as_uint(top));  // not negative: ordered as bits
    if (lane == 0) {
        sh.part[warp][1] = kmin;
        sh.part[warp][2] = kmax;
        sh.part[warp][3] = topb;
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kSelectWarps; ++x) {
        kmin = min(kmin, sh.part[x][1]);
        kmax = max(kmax, sh.part[x][2]);
        topb = max(topb, sh.part[x][3]);
    }

    // the take-th largest key: kBins bins over [lo, hi], then over the bin that
    // holds it, until its keys are few enough to rank (or all alike)
    uint32_t lo = kmin, hi = kmax;
    unsigned need = w.take;
    while (lo < hi) {
        const int shift = max(0, 32 - __clz(hi - lo) - 9);
        for (int i = tid; i < kBins; i += kSelectThreads) sh.hist[i] = 0;
        if (tid == 0) sh.n_border = 0;
        __syncthreads();
        for (int i = tid; i < w.n; i += kSelectThreads) {
            const uint32_t k = keys[i];
            if (k - lo <= hi - lo) atomicAdd(&sh.hist[(k - lo) >> shift], 1u);
        }
        __syncthreads();
        {  // two bins a thread, from the top down
            const unsigned m0 = sh.hist[kBins - 1 - 2 * tid], m1 = sh.hist[kBins - 2 - 2 * tid];
            unsigned total;
            const unsigned before = block_prefix(m0 + m1, total, sh);
            if (before < need && need <= before + m0) {
                sh.bin = kBins - 1 - 2 * tid;
                sh.above = before;
            } else if (before + m0 < need && need <= before + m0 + m1) {
                sh.bin = kBins - 2 - 2 * tid;
                sh.above = before + m0;
            }
        }
        __syncthreads();
        const unsigned in_bin = sh.hist[sh.bin];
        need -= sh.above;
        lo += sh.bin << shift;
        hi = min(hi, lo + ((1u << shift) - 1));
        if (lo < hi && in_bin <= 64) {
            for (int i = tid; i < w.n; i += kSelectThreads) {
                const uint32_t k = keys[i];
                if (k - lo <= hi - lo) sh.border[atomicAdd(&sh.n_border, 1u)] = (int)k;
            }
            __syncthreads();
            if (tid < (int)in_bin) {
                const uint32_t k = (uint32_t)sh.border[tid];
                unsigned more = 0, same = 0;
                for (unsigned j = 0; j < in_bin; ++j) {
                    more += (uint32_t)sh.border[j] > k;
                    same += (uint32_t)sh.border[j] == k;
                }
                if (more < need && need <= more + same) sh.bin = k;  // equal keys write the same
            }
            __syncthreads();
            lo = hi = sh.bin;
        }
        __syncthreads();
    }
    uint32_t k_lo, k_hi;
    doubt_range(lo, error_bound<Ty>(P, sh.l1, sh.mxq, __uint_as_float(topb)), k_lo, k_hi);
    // pages in doubt, in page order: each warp counts a contiguous share
    const int share = ((w.n + kSelectThreads - 1) / kSelectThreads) * 32;
    const int wa = min(w.n, warp * share), wb = min(w.n, wa + share);
    unsigned n_hi = 0, n_in = 0;
    for (int i = wa + lane; i < wb; i += 32) {
        const uint32_t k = keys[i];
        n_hi += k > k_hi;
        n_in += k >= k_lo && k <= k_hi;
    }
    unsigned all_hi, all_in;
    block_prefix(n_hi, all_hi, sh);
    block_prefix(n_in, all_in, sh);
    const unsigned want = w.take - all_hi;  // of the pages in doubt
    if (all_in != want) {
        __syncthreads();
        if (tid == 0) sh.n_border = 0;
        __syncthreads();
        if (all_in <= kBorder) {
            for (int i = tid; i < w.n; i += kSelectThreads) {
                const uint32_t k = keys[i];
                if (k >= k_lo && k <= k_hi) sh.border[atomicAdd(&sh.n_border, 1u)] = i;  // any order
            }
            __syncthreads();
            for (unsigned i0 = 4 * warp; i0 < all_in; i0 += 4 * kSelectWarps) {
                const unsigned i = i0 + (lane >> 3);
                const double x = exact_score<Ty>(P, w.s, w.h, i < all_in ? sh.border[i] : -1, sh.q, lane);
                if ((lane & 7) == 0 && i < all_in) sh.exact[i] = x;
            }
            __syncthreads();
            for (unsigned i = tid; i < all_in; i += kSelectThreads) {
                const unsigned long long x = order_key64(sh.exact[i]);
                const int xi = sh.border[i];
                unsigned rank = 0;
                for (unsigned j = 0; j < all_in; ++j) {
                    const unsigned long long y = order_key64(sh.exact[j]);
                    rank += y > x || (y == x && sh.border[j] < xi);
                }
                keys[xi] = rank < want ? 0xffffffffu : 0u;
            }
        } else if (warp == 0) {
            select_many<Ty>(
                P, w, sh.q, sh.hist, k_lo, k_hi, want, [&](int i) { return keys[i]; },
                [&](int i, bool yes) { keys[i] = yes ? 0xffffffffu : 0u; });
        }
        __syncthreads();
    }
    // pages in ascending order; all in doubt are wanted, or those marked above
    const uint32_t cut = all_in == want ? k_lo : k_hi + 1;
    unsigned cnt = 0;
    for (int i = wa + lane; i < wb; i += 32) cnt += keys[i] >= cut;
    unsigned total;
    const unsigned before = block_prefix(cnt, total, sh);
    unsigned at = __shfl_sync(0xffffffffu, before, 0);
    for (int i0 = wa; i0 < wb; i0 += 32) {
        const bool yes = i0 + lane < wb && keys[i0 + lane] >= cut;
        const unsigned bal = __ballot_sync(0xffffffffu, yes);
        const unsigned to = at + __popc(bal & ((1u << lane) - 1u));
        if (yes && to < (unsigned)w.take) w.out[to] = i0 + lane;
        at += __popc(bal);
    }
}

constexpr int kTokSmall = 4, kTokLarge = 32;

constexpr int kMaxRanges = 64;  // page ranges of a score launch

template <class Ty, int NT>
cudaError_t launch_scores(EstimateParams &P, cudaStream_t st) {
    const PagedSeqs &S = P.seqs;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(paged_scores_kernel<Ty, NT>), (int)ScoreShape<NT>::kBytes,
                               done);
    if (e != cudaSuccess) return e;
    // page ranges: about two CTAs to an SM over all (sequence, tile, kv-head)s
    const long long rows = (long long)S.n_seqs * P.tiles * P.hkv;
    const int step = ScoreShape<NT>::kWarps * kStepPages;
    const int most = (S.width + step - 1) / step;
    const int z = (int)std::max<long long>(1, std::min<long long>({most, 296 / rows, kMaxRanges}));
    P.pages_per_cta = ((S.width + z - 1) / z + step - 1) / step * step;
    P.ranges = (S.width + P.pages_per_cta - 1) / P.pages_per_cta;
    const dim3 grid((unsigned)(S.n_seqs * P.tiles), P.hkv, P.ranges);
    paged_scores_kernel<Ty, NT><<<grid, ScoreShape<NT>::kThreads, ScoreShape<NT>::kBytes, st>>>(P);
    return cudaGetLastError();
}

template <class Ty>
cudaError_t launch_select(const EstimateParams &P, cudaStream_t st) {
    const int rows = (P.t1 - P.t0) * P.hkv;
    // A warp per row once the rows fill the SMs that way: 4,096 rows of 1,016 pages take
    // 30 us so and 40 us with a CTA each.  128 rows of 2,048 pages take 13 us with a CTA each.
    const int most = P.seqs.width - 1;  // candidates: the token's own page is none
    if (rows >= 1024 && most <= 2048) {
        const dim3 grid((rows + kSelectWarps - 1) / kSelectWarps);
        if (most <= 1024)
            return launch_after(paged_select_warp_kernel<Ty, 32>, grid, dim3(kSelectThreads), 0, st, P);
        return launch_after(paged_select_warp_kernel<Ty, 64>, grid, dim3(kSelectThreads), 0, st, P);
    }
    const size_t bytes = (size_t)P.score_stride * sizeof(uint32_t);
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(paged_select_kernel<Ty>), kMaxBlocks * (int)sizeof(uint32_t),
                               done);
    if (e != cudaSuccess) return e;
    return launch_after(paged_select_kernel<Ty>, dim3(rows), dim3(kSelectThreads), bytes, st, P);
}

template <class Ty>
cudaError_t launch(EstimateParams P, cudaStream_t st) {
    const PagedSeqs &S = P.seqs;
    ProfScope prof("paged_estimate", st);
    const int batch = P.batch;
    for (int t0 = 0; t0 < S.total; t0 += batch) {
        P.t0 = t0;
        P.t1 = min(S.total, t0 + batch);
        const int most = min(S.max_q, P.t1 - P.t0);
        const bool small = most <= kTokSmall;
        const int tok = small ? kTokSmall : kTokLarge;
        P.tiles = (most + tok - 1) / tok;
        P.tile_tokens = tok;
        cudaError_t e = small ? launch_scores<Ty, kTokSmall / 4>(P, st) : launch_scores<Ty, kTokLarge / 4>(P, st);
        if (e != cudaSuccess) return e;
        e = launch_select<Ty>(P, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

EstimatePlan paged_estimate_plan(int total, int n_seqs, int max_q, int hkv, int width) {
    EstimatePlan p{};
    p.score_stride = (width + 3) & ~3;
    // 64 MiB of scores at a time: written and read back inside L2
    const long long row = (long long)p.score_stride * 4 * hkv;
    p.batch = (int)std::max<long long>(1, std::min<long long>(total, (64ll << 20) / row));
    p.n_scores = (size_t)p.batch * hkv * p.score_stride;
    // tiles of a launch: at most these (the last batch is no longer than the others, but
    // may fall into the small tiles), times their ranges
    const long long most = std::min(max_q, p.batch);
    const long long tiles = std::max<long long>((most + kTokLarge - 1) / kTokLarge,
                                                std::min<long long>(most, kTokSmall) > 0 ? 1 : 0);
    const long long rows = (long long)n_seqs * tiles * hkv;
    p.n_top = (size_t)std::max<long long>(rows, std::min<long long>(rows * kMaxRanges, 296));
    return p;
}

cudaError_t run_paged_estimate(const EstimateParams &P, bool fp16, cudaStream_t st) {
    if (P.seqs.n_seqs == 0 || P.seqs.total == 0) return cudaSuccess;
    return fp16 ? launch<Fp16>(P, st) : launch<Bf16>(P, st);
}

}  // namespace minf
