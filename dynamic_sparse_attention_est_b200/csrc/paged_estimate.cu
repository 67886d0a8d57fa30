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
//   scores  a product of pages by tokens, Q as the sum of two 16-bit parts, which
//           carries it to 2^-16: approximate, with a bound E on the error.  Up to
//           four new tokens: bound by reading the bounds (512 B per page and
//           kv-head); 16 pages are the rows of an m16n8k16 product, whose columns
//           are the four tokens' parts; each warp brings its own pages in through a
//           ring of bulk copies, one per page, at a stride of 528 B that ldmatrix
//           reads without bank conflicts.  Chunks: 128 pages by 64 tokens' parts on
//           the tensor cores (tcgen05, K = 256), pages gathered by cp.async into the
//           swizzled layout.  (mma.sync there took 29.5 us for 512 tokens over 1,016
//           pages and eight kv-heads, at about a tenth of the tensor cores' rate.)
//   select  one warp (many rows) or one CTA (few) per row: the k-th largest
//           approximate score t by counting over a shrinking range of its key bits
//           until few keys are left, which are ranked; then every page within 2 E of
//           t is scored again in 64 bits; all others are decided by the
//           approximation.  So the selection is that of 64-bit scores (which decide
//           ties to their own rounding: pages of equal bounds score alike to the bit).
// E = (2^-15 + G 2^-23) |Q|_1 max|bound|: the two-part split of bf16 loses 2^-16
// (fp16's less), the sums Q lose G 2^-24, and sixteen accumulation steps are taken to
// lose 2^-18, 2^-22 of the magnitudes each; 1.6 times their sum.  The last of the three
// is an assumption, since the instruction's rounding is not documented; scores made to
// cancel, to round one way or to drop their last bits come to 0.08 E at most, with
// either score kernel and either type.
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

template <class Ty>
__device__ __forceinline__ void add_signed(const uint4 &w, float (&up)[8], float (&down)[8]) {
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

// Q+ and Q- of channels 8 c .. 8 c + 7 of a token, fp32 (all terms of one sign).
template <class Ty>
__device__ __forceinline__ void q_sums(const EstimateParams &P, int tok, int h, int c, float (&up)[8], float (&down)[8]) {
    const typename Ty::T *q = static_cast<const typename Ty::T *>(P.q) + (long long)tok * P.q_ts +
                              (long long)h * P.group * P.q_hs + c * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) up[i] = down[i] = 0.f;
#pragma unroll 4
    for (int g = 0; g < P.group; ++g)
        add_signed<Ty>(__ldg(reinterpret_cast<const uint4 *>(q + (long long)g * P.q_hs)), up, down);
}

// The scale of a token's parts (sixteen lanes hold its sums): 1, or for fp16 the
// power of two that suits its largest.
template <class Ty>
__device__ __forceinline__ float row_scale(const float (&up)[8], const float (&down)[8]) {
    if (Ty::kIdescType != 0) return 1.f;  // bf16
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fmaxf(up[i], -down[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    return part_scale<Ty>(mx);
}

// x sc as the sum of two 16-bit parts.
template <class Ty>
__device__ __forceinline__ void two_parts(const float (&x)[8], float sc, uint32_t (&hi)[4], uint32_t (&mid)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i] * sc, b = x[2 * i + 1] * sc;
        hi[i] = Ty::pack(a, b);
        const float2 f = Ty::unpack(hi[i]);
        mid[i] = Ty::pack(a - f.x, b - f.y);
    }
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// ------------------------------------------------------------------ scores
// grid: x = sequence * tiles + token tile, y = kv-head, z = page range.
constexpr int kTokSmall = 4, kTokLarge = 64;  // tokens of a tile

struct ScoreShape {
    static constexpr int kWarps = 6, kThreads = 32 * kWarps, kStages = 2;
    static constexpr uint32_t kRing = kWarps * kStages * kStepBytes;
    static constexpr uint32_t kFrag = 8 * 32 * 16;
    static constexpr uint32_t kBytes = kRing + kFrag + 192;
};

template <class Ty>
__global__ void __launch_bounds__(ScoreShape::kThreads, 2) paged_scores_kernel(const __grid_constant__ EstimateParams P) {
    using T = typename Ty::T;
    using Shape = ScoreShape;
    constexpr int kTok = kTokSmall, kStages = Shape::kStages, kWarps = Shape::kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    uint4 *qf = reinterpret_cast<uint4 *>(smem + Shape::kRing);  // column fragments [8][32]
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

    // column fragments: column n is part n & 1 of token n / 2; sixteen threads a token,
    // 8 channels each, element = side * 128 + channel
    if (threadIdx.x < 16 * kTok) {
        const int ch = threadIdx.x & 15, x = threadIdx.x >> 4;
        float up[8] = {}, down[8] = {};
        if (ta + x < tb) q_sums<Ty>(P, ta + x, h, ch, up, down);
        const float sc = row_scale<Ty>(up, down);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            // element side * 128 + 8 ch + 2 p: k-step / 16, register (/ 8) % 2, lane column p
            const int kk = side * 8 + (ch >> 1), reg = (kk & 1) * 2 + (ch & 1);
            uint32_t hi[4], mid[4];
            two_parts<Ty>(side ? up : down, sc, hi, mid);
            uint32_t *w = reinterpret_cast<uint32_t *>(qf + (kk >> 1) * 32);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                w[((2 * x) * 4 + p) * 4 + reg] = hi[p];
                w[((2 * x + 1) * 4 + p) * 4 + reg] = mid[p];
            }
        }
    }
    __syncthreads();
    launch_dependents();  // the selection's own preparations run beside the rest of this

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
        float d[2][4] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4 b = qf[i * 32 + lane];
            Ty::mma(d[0], a[2 * i][0], a[2 * i][1], a[2 * i][2], a[2 * i][3], b.x, b.y);
            Ty::mma(d[1], a[2 * i + 1][0], a[2 * i + 1][1], a[2 * i + 1][2], a[2 * i + 1][3], b.z, b.w);
        }
        if (ta + c < tb) {
            float *dst = P.scores + ((long long)(ta + c - P.t0) * P.hkv + h) * P.score_stride + j0 + r;
            if (r0) dst[0] = (d[0][0] + d[1][0]) + (d[0][1] + d[1][1]);
            if (r1) dst[8] = (d[0][2] + d[1][2]) + (d[0][3] + d[1][3]);
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
            P.top[((long long)(ta - P.t0) * P.hkv + h) * P.ranges + blockIdx.z] = fmaxf(top, 0.f);
        }
    }
}

// Chunks: 128 pages (rows, K-major in 128-byte swizzle: four 64-channel pieces of 16
// KB) by 64 tokens' two parts (128 rows alike), K = 256.  Two page tiles in shared
// memory: while the tensor cores multiply one, the next is on its way.
constexpr int kTcThreads = 256, kPageTile = 128;
constexpr uint32_t kPieceBytes = 16384, kTileBytes = 4 * kPieceBytes;
constexpr uint32_t kTcBar = 3 * kTileBytes;  // two page tiles, the token tile
constexpr uint32_t kTcBytes = kTcBar + 128 + 1024;

template <class Ty>
__global__ void __launch_bounds__(kTcThreads, 1) paged_scores_tc_kernel(const __grid_constant__ EstimateParams P) {
    using T = typename Ty::T;
    extern __shared__ uint8_t tc_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(tc_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sA = smem_u32(smem), sB = sA + 2 * kTileBytes;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kTcBar);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bar + 1);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + 2);
    float *warp_top = reinterpret_cast<float *>(bar + 3);  // [8]
    const PagedSeqs &S = P.seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y;
    int s = blockIdx.x / P.tiles, tile = blockIdx.x % P.tiles;
    if (P.packed) {
        auto tiles = [&](int x) -> int {
            const SeqView w = seq_view(S, x, P.hdr);
            return (max(0, min(w.q0 + w.n, P.t1) - max(w.q0, P.t0)) + kTokLarge - 1) / kTokLarge;
        };
        if (!find_item<kTcThreads>(S.n_seqs, blockIdx.x, tiles, s, tile)) return;
    }
    const SeqView v = seq_view(S, s, P.hdr);
    const int ta = max(v.q0, P.t0) + tile * kTokLarge;
    const int tb = min(min(v.q0 + v.n, P.t1), ta + kTokLarge);
    if (ta >= tb) return;
    const int last_pos = v.len - v.n + (tb - 1 - v.q0);
    const int n_pages = last_pos < 0 ? 0 : last_pos >> S.page_log2;  // pages before the last token's own
    const int pa = blockIdx.z * P.pages_per_cta, pb = min(pa + P.pages_per_cta, n_pages);
    if (pa >= pb) return;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(bar), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), 128);
        tmem_relinquish();
    }
    const WaitCtl wc{abort_flag, &P.hdr->status, P.wait_limit_ns};

    // a warp brings in 16 pages, a lane 16 bytes of each: lanes 0 - 15 min, 16 - 31 max
    const int side = lane >> 4;
    const T *kb = static_cast<const T *>(P.bounds) + (long long)h * 2 * kD + lane * 8;
    const long long page_stride = (long long)P.hkv * 2 * kD;
    auto id_at = [&](int j0) -> int {  // lane i: page id of the warp's row i
        const int j = j0 + warp * 16 + lane;
        return lane < 16 && j < pb ? page_of(S, s, j, P.hdr) : -1;
    };
    auto piece = [&](int i) -> uint32_t {  // shared offset of the lane's 16 bytes of the warp's row i
        const int row = warp * 16 + i;
        return (lane >> 3) * kPieceBytes + row * 128 + (((lane & 7) ^ (row & 7)) << 4);
    };
    auto fill = [&](int st, int ids) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int id = __shfl_sync(0xffffffffu, ids, i);
            if (id >= 0) cp_async16(sA + st * kTileBytes + piece(i), kb + id * page_stride);
        }
    };
    int id = id_at(pa), id_next = id_at(pa + kPageTile);
    fill(0, id);
    // The tokens' parts: row 2 x + part; sixteen threads a token, 8 channels each, the
    // loads of all its four tokens in flight together.
    {
        constexpr int kPass = kTokLarge * 16 / kTcThreads;
        const int ch = threadIdx.x & 15, x0 = threadIdx.x >> 4;
        float up[kPass][8] = {}, down[kPass][8] = {};
        const T *q = static_cast<const T *>(P.q) + (long long)(ta + x0) * P.q_ts + (long long)h * P.group * P.q_hs + ch * 8;
        for (int g0 = 0; g0 < P.group; g0 += 4) {
            uint4 w[kPass][4];
#pragma unroll
            for (int x = 0; x < kPass; ++x)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    w[x][g] = ta + x0 + 16 * x < tb && g0 + g < P.group
                                  ? __ldg(reinterpret_cast<const uint4 *>(q + (long long)(16 * x) * P.q_ts +
                                                                          (long long)(g0 + g) * P.q_hs))
                                  : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int x = 0; x < kPass; ++x)
#pragma unroll
                for (int g = 0; g < 4; ++g) add_signed<Ty>(w[x][g], up[x], down[x]);
        }
#pragma unroll
        for (int y = 0; y < kPass; ++y) {
            const int x = x0 + 16 * y;
            const float sc = row_scale<Ty>(up[y], down[y]);
#pragma unroll
            for (int sd = 0; sd < 2; ++sd) {
                uint32_t hi[4], mid[4];
                two_parts<Ty>(sd ? up[y] : down[y], sc, hi, mid);
                uint8_t *dst = smem + 2 * kTileBytes + (2 * sd + (ch >> 3)) * kPieceBytes;
                const int r0 = 2 * x, r1 = 2 * x + 1, c16 = ch & 7;
                *reinterpret_cast<uint4 *>(dst + r0 * 128 + ((c16 ^ (r0 & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(dst + r1 * 128 + ((c16 ^ (r1 & 7)) << 4)) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
            }
        }
    }
    launch_dependents();  // the selection's own preparations run beside the rest of this
    constexpr uint32_t kIdesc = (1u << 4) | Ty::kIdescType | ((128u >> 3) << 17) | ((128u >> 4) << 24);
    const uint64_t da = sdesc_sw128(sA, 16, 1024), db = sdesc_sw128(sB, 16, 1024);
    uint32_t ext2 = side ? Ty::kNegInf2 : Ty::kPosInf2;  // largest max, or smallest min
    int st = 0, par = 0;
    bool ok = true;
    for (int j0 = pa; j0 < pb; j0 += kPageTile) {
        cp_async_wait_all();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();  // the tile is complete, and the products and reads of the one before are over
        tc_fence_after();
        const uint32_t tmem = *tmem_slot;
        if (warp == 0) {
            // K = 256 as two calls of eight K = 16 steps over two pieces each
            const uint64_t a0 = da + (uint64_t)(st * (kTileBytes >> 4));
            umma_ss_tile_warp(tmem, a0, db, kIdesc, 0u);
            umma_ss_tile_warp(tmem, a0 + 2 * (kPieceBytes >> 4), db + 2 * (kPieceBytes >> 4), kIdesc, 1u);
            umma_commit_warp(smem_u32(bar));
        }
        const int id_here = id;
        id = id_next;
        if (j0 + kPageTile < pb) {
            fill(st ^ 1, id);
            id_next = id_at(j0 + 2 * kPageTile);
        }
        // No key exceeds its page's max nor falls below its min, so the largest |bound| is
        // the largest max or the largest -min.
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (__shfl_sync(0xffffffffu, id_here, i) >= 0) {
                const uint4 w = *reinterpret_cast<const uint4 *>(smem + st * kTileBytes + piece(i));
                const uint32_t a = side ? Ty::vmax(Ty::vmax(w.x, w.y), Ty::vmax(w.z, w.w))
                                        : Ty::vmin(Ty::vmin(w.x, w.y), Ty::vmin(w.z, w.w));
                ext2 = side ? Ty::vmax(ext2, a) : Ty::vmin(ext2, a);
            }
        const bool got = wait_bounded(smem_u32(bar), par, wc, wait_site(9, 0, j0));
        ok = !__syncthreads_or(!got);
        if (!ok) break;
        par ^= 1;
        tc_fence_after();
        // lane = page; a warp takes half of its quarter's columns: 32 tokens' pairs of parts
        const int page = j0 + (warp & 3) * 32 + lane, t0 = ta + (warp >> 2) * 32;
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (warp >> 2) * 64;
        uint32_t d[2][32];
        tmem_ld32(at, d[0]);
        tmem_ld32(at + 32, d[1]);
        tmem_ld_wait(d[0]);
        tmem_ld_wait(d[1]);
        const int n_tok = page < pb ? tb - t0 : 0;
        const long long step = (long long)P.hkv * P.score_stride;
        float *dst = P.scores + ((long long)(t0 - P.t0) * P.hkv + h) * P.score_stride + page;
#pragma unroll
        for (int y = 0; y < 32; ++y) {
            if (y < n_tok) *dst = __uint_as_float(d[y >> 4][2 * (y & 15)]) + __uint_as_float(d[y >> 4][2 * (y & 15) + 1]);
            dst += step;
        }
        st ^= 1;
    }
    cp_async_wait_all();  // none is in flight when the CTA exits
    {
        const float2 f = Ty::unpack(ext2);
        float top = side ? fmaxf(f.x, f.y) : fmaxf(-f.x, -f.y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) warp_top[warp] = top;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int w = 0; w < kTcThreads / 32; ++w) top = fmaxf(top, warp_top[w]);
            P.top[((long long)(ta - P.t0) * P.hkv + h) * P.ranges + blockIdx.z] = fmaxf(top, 0.f);
        }
        if (warp == 0) tmem_dealloc(*tmem_slot, 128);
    }
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
    long long tile_range0;   // first entry of its tile's page ranges in EstimateParams::top
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
    const int t_first = max(v.q0, P.t0), tile = t_first + (w.tok - t_first) / P.tile_tokens * P.tile_tokens;
    w.tile_range0 = ((long long)(tile - P.t0) * P.hkv + w.h) * P.ranges;
    w.sc = P.scores + (row - (long long)P.t0 * P.hkv) * P.score_stride;
    return true;
}

__device__ __forceinline__ int seq_of(const PagedSeqs &S, int tok, int s) {
    return s < S.n_seqs && __ldg(S.cu_q + s) <= tok && tok < __ldg(S.cu_q + s + 1) ? s : -1;
}

// One warp: Q in 64 bits (4 channels a lane) to q (Q- then Q+), its 1-norm and
// largest element in l1 and mx of each lane (the lane's own share).
template <class Ty>
__device__ __forceinline__ void exact_q(const EstimateParams &P, const Row &w, int lane, double *q, float &l1, float &mx) {
    double up[4] = {}, down[4] = {};
    const typename Ty::T *src = static_cast<const typename Ty::T *>(P.q) + (long long)w.tok * P.q_ts +
                                (long long)w.h * P.group * P.q_hs + lane * 4;
#pragma unroll 4
    for (int g = 0; g < P.group; ++g) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src + (long long)g * P.q_hs));
        const float2 f0 = Ty::unpack(v.x), f1 = Ty::unpack(v.y);
        const float f[4] = {f0.x, f0.y, f1.x, f1.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double d = (double)f[i];
            up[i] += f[i] > 0.f ? d : 0.0;
            down[i] += f[i] < 0.f ? d : 0.0;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[lane * 4 + i] = down[i];
        q[kD + lane * 4 + i] = up[i];
        l1 += (float)(up[i] - down[i]);
        mx = fmaxf(mx, fmaxf((float)up[i], (float)-down[i]));
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
    k_lo = max(order_key(t - width), 1u);
    k_hi = min(order_key(t + width), 0xfffffffeu);
    if (k_lo > t_key || k_hi < t_key) {  // infinities or NaN among the bounds: everything is in doubt
        k_lo = 1u;
        k_hi = 0xfffffffeu;
    }
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
__device__ __forceinline__ void select_row_warp(const EstimateParams &P) {
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
    exact_q<Ty>(P, w, lane, sh.q, l1, mxq);
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
    // From here on bit sets: lane e (and 32 + e, kPer = 64) has the candidates 32 e ..
    // 32 e + 31 that are taken for sure, and those in doubt.
    constexpr int kSets = kPer / 32;
    unsigned sure[kSets] = {}, doubt[kSets] = {};
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const unsigned a = __ballot_sync(0xffffffffu, key[e] > k_hi), b = __ballot_sync(0xffffffffu, key[e] >= k_lo);
        if (lane == (e & 31)) {
            sure[e >> 5] = a;
            doubt[e >> 5] = b & ~a;
        }
    }
    unsigned n_hi = 0, n_in = 0;
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
        n_hi += __popc(sure[i]);
        n_in += __popc(doubt[i]);
    }
    n_hi = __reduce_add_sync(0xffffffffu, n_hi);
    n_in = __reduce_add_sync(0xffffffffu, n_in);
    const unsigned want = w.take - n_hi;  // of the pages in doubt
    if (n_in != want) {
        if (lane == 0) sh.n_border = 0;
        __syncwarp();
        if (n_in <= kWarpBorder) {
#pragma unroll
            for (int i = 0; i < kSets; ++i)
                for (unsigned m = doubt[i]; m; m &= m - 1)
                    sh.border[atomicAdd(&sh.n_border, 1u)] = (i * 32 + lane) * 32 + __ffs(m) - 1;  // any order
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
#pragma unroll
        for (int i = 0; i < kSets; ++i) doubt[i] = sh.chosen[i * 32 + lane];
    }
    unsigned base = 0;
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
        unsigned m = sure[i] | doubt[i];
        const unsigned n_mine = __popc(m);
        unsigned inc = n_mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        for (unsigned at = base + inc - n_mine; m; m &= m - 1, ++at)
            if (at < (unsigned)w.take) w.out[at] = (i * 32 + lane) * 32 + __ffs(m) - 1;
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
}

template <class Ty, int kPer>
__global__ void __launch_bounds__(kSelectThreads, kPer == 32 ? 3 : 2)
    paged_select_warp_kernel(const __grid_constant__ EstimateParams P) {
    select_row_warp<Ty, kPer>(P);
    end_after_primary();
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
__device__ __forceinline__ void select_row(const EstimateParams &P) {
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
        exact_q<Ty>(P, w, lane, sh.q, l1, mxq);
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

template <class Ty>
__global__ void __launch_bounds__(kSelectThreads) paged_select_kernel(const __grid_constant__ EstimateParams P) {
    select_row<Ty>(P);
    end_after_primary();
}

constexpr int kMaxRanges = 64;  // page ranges of a score launch

template <class Ty>
cudaError_t launch_scores(EstimateParams &P, bool small, cudaStream_t st) {
    const PagedSeqs &S = P.seqs;
    static std::atomic<unsigned long long> done_small{0}, done_tc{0};
    cudaError_t e =
        small ? allow_smem(reinterpret_cast<const void *>(paged_scores_kernel<Ty>), (int)ScoreShape::kBytes, done_small)
              : allow_smem(reinterpret_cast<const void *>(paged_scores_tc_kernel<Ty>), (int)kTcBytes, done_tc);
    if (e != cudaSuccess) return e;
    // Tiles of the longest sequence for every one, or, where that is far above what all
    // tokens can fill (a chunk beside many single tokens), that bound, each CTA finding
    // its tile.
    const long long by_seq = (long long)S.n_seqs * P.tiles, all = (P.t1 - P.t0) / kTokLarge + S.n_seqs;
    P.packed = !small && by_seq > 2 * all;
    const long long x = P.packed ? all : by_seq;
    // page ranges: one wave of CTAs over all of them
    const int step = small ? ScoreShape::kWarps * kStepPages : kPageTile;
    const int pages = std::max(1, S.width - 1);  // candidates: the token's own page is none
    const int most = (pages + step - 1) / step;
    const int z = (int)std::max<long long>(1, std::min<long long>({most, (small ? 296 : 148) / (x * P.hkv), kMaxRanges}));
    P.pages_per_cta = (most + z - 1) / z * step;
    P.ranges = (pages + P.pages_per_cta - 1) / P.pages_per_cta;
    const dim3 grid((unsigned)x, P.hkv, P.ranges);
    if (small) paged_scores_kernel<Ty><<<grid, ScoreShape::kThreads, ScoreShape::kBytes, st>>>(P);
    else paged_scores_tc_kernel<Ty><<<grid, kTcThreads, kTcBytes, st>>>(P);
    return cudaGetLastError();
}

template <class Ty>
cudaError_t launch_select(const EstimateParams &P, cudaStream_t st) {
    const int rows = (P.t1 - P.t0) * P.hkv;
    // A warp per row once the rows fill the SMs that way: 4,096 rows of 1,016 pages take
    // 22 us so and 40 us with a CTA each; 128 rows of 2,048 pages 13 us with a CTA each.
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
        cudaError_t e = launch_scores<Ty>(P, small, st);
        if (e != cudaSuccess) return e;
        e = launch_select<Ty>(P, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

static int score_stride(int width) { return (width + 3) & ~3; }

// 64 MiB of scores at a time: written and read back inside L2
constexpr long long kBatchScores = (64ll << 20) / 4;
static int score_batch(int total, int hkv, int width) {
    const long long row = (long long)score_stride(width) * hkv;
    return (int)std::max<long long>(1, std::min<long long>(total, kBatchScores / row));
}

// Page ranges of a launch, of which launch_scores takes no more.
constexpr int kRangePages = ScoreShape::kWarps * kStepPages;
static long long score_ranges(int n_seqs, int hkv, int width) {
    const long long most = (std::max(1, width - 1) + kRangePages - 1) / kRangePages;
    return std::max<long long>(1, std::min<long long>({most, 296 / ((long long)n_seqs * hkv), kMaxRanges}));
}

EstimatePlan paged_estimate_plan(int total, int n_seqs, int hkv, int width) {
    EstimatePlan p{};
    p.score_stride = score_stride(width);
    p.batch = score_batch(total, hkv, width);
    p.n_scores = (size_t)p.batch * hkv * p.score_stride;
    p.n_top = (size_t)p.batch * hkv * score_ranges(n_seqs, hkv, width);
    return p;
}

EstimatePlan paged_estimate_reserve(int total, int hkv, int width) {
    EstimatePlan p = paged_estimate_plan(total, 1, hkv, width);
    // a narrower table's batch of more tokens may come closer to the 64 MiB
    const long long row = (long long)p.score_stride * hkv;
    p.n_scores = (size_t)std::min(total * row, std::max(kBatchScores, row));
    // fewer sequences have more ranges; of the tables with r ranges, the narrowest has the
    // largest batch
    for (long long r = score_ranges(1, hkv, width); r >= 1; --r)
        p.n_top = std::max(p.n_top, (size_t)(r * hkv * score_batch(total, hkv, (int)(r - 1) * kRangePages + (r > 1 ? 2 : 1))));
    return p;
}

cudaError_t run_paged_estimate(const EstimateParams &P, bool fp16, cudaStream_t st) {
    if (P.seqs.n_seqs == 0 || P.seqs.total == 0) return cudaSuccess;
    return fp16 ? launch<Fp16>(P, st) : launch<Bf16>(P, st);
}

}  // namespace minf
