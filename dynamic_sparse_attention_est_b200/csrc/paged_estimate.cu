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
//           of an m16n8k16 product, straight from global memory to its registers
//           (the contraction may take the channels in any order); its columns are
//           four tokens' Q, each as the sum of two 16-bit parts, which carries Q
//           to 2^-16.  The scores are approximate, with a bound E on their error.
//   select  one CTA per row: the k-th largest approximate score t by counting over
//           a shrinking range of its key bits, then every page within 2 E of t is
//           scored again in 64 bits; all others are decided by the approximation.
//           So the selection is that of exact scores.
// E = (2^-15 + G 2^-23) |Q|_1 max|bound|: the two-part split of bf16 loses 2^-16
// (fp16's less), sixteen accumulation steps at 2^-22 of the magnitudes each lose
// 2^-18, the sums Q lose G 2^-24; 1.6 times their sum, since the instruction's
// rounding is not documented.
#include <algorithm>

#include "internal.h"
#include "paged.cuh"

namespace minf {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kStepPages = 16;
constexpr int kBorder = 1024;  // pages a row ranks in shared memory by their exact scores

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
__device__ __forceinline__ float to_f32(typename Ty::T x);
template <>
__device__ __forceinline__ float to_f32<Bf16>(__nv_bfloat16 x) {
    return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float to_f32<Fp16>(__half x) {
    return __half2float(x);
}

// Q+ and Q- of channel c of a token, fp32 (all terms of one sign).
template <class Ty>
__device__ __forceinline__ void q_sums(const EstimateParams &P, int tok, int h, int c, float &up, float &down) {
    const typename Ty::T *q = static_cast<const typename Ty::T *>(P.q) + (long long)tok * P.q_ts +
                              (long long)h * P.group * P.q_hs + c;
    up = down = 0.f;
#pragma unroll 4
    for (int g = 0; g < P.group; ++g) {
        const float x = to_f32<Ty>(__ldg(q + (long long)g * P.q_hs));
        up += fmaxf(x, 0.f);
        down += fminf(x, 0.f);
    }
}

// ------------------------------------------------------------------ scores
// grid: x = sequence * tiles + token tile, y = kv-head, z = page range.
template <class Ty, int NT>
__global__ void __launch_bounds__(kThreads) paged_scores_kernel(const __grid_constant__ EstimateParams P) {
    using T = typename Ty::T;
    constexpr int kTok = 4 * NT;
    __shared__ uint4 qf[NT][8][32];     // column fragments
    __shared__ float top[kWarps];
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

    // column fragments: column n of tile nt is part n & 1 of token 4 nt + n / 2;
    // thread = channel, element (min part: Q-, max part: Q+)
    {
        const int ch = threadIdx.x;
        for (int x = 0; x < kTok; ++x) {
            float up = 0.f, down = 0.f;
            if (ta + x < tb) q_sums<Ty>(P, ta + x, h, ch, up, down);
            float sc = 1.f;
            if (sizeof(T) == 2 && Ty::kIdescType == 0) {  // fp16: scale by the row's largest
                float mx = fmaxf(up, -down);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                if (lane == 0) top[warp] = mx;
                __syncthreads();
                mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                __syncthreads();
                sc = part_scale<Ty>(mx);
            }
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const float val = (side ? up : down) * sc;
                const uint32_t hi = Ty::pack(val, 0.f) & 0xffffu;
                const uint32_t mid = Ty::pack(val - Ty::unpack(hi).x, 0.f) & 0xffffu;
                const int el = side * kD + ch;         // element of the 256
                const int i = el >> 5, cc = (el >> 3) & 3, b = el & 7;
                uint16_t *w0 = reinterpret_cast<uint16_t *>(&qf[x >> 2][i][(2 * (x & 3)) * 4 + cc]) + b;
                uint16_t *w1 = reinterpret_cast<uint16_t *>(&qf[x >> 2][i][(2 * (x & 3) + 1) * 4 + cc]) + b;
                *w0 = (uint16_t)hi;
                *w1 = (uint16_t)mid;
            }
        }
    }
    __syncthreads();

    const T *kb = static_cast<const T *>(P.bounds) + (long long)h * 2 * kD + c * 8;
    const long long page_stride = (long long)P.hkv * 2 * kD;
    auto pages_at = [&](int j0, int (&pg)[2]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int j = j0 + r + 8 * e;
            pg[e] = j < pb ? page_of(S, s, j, P.hdr) : -1;
        }
    };
    auto load = [&](uint4(&a)[16], const int (&pg)[2]) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                a[e * 8 + i] = pg[e] >= 0 ? __ldg(reinterpret_cast<const uint4 *>(kb + pg[e] * page_stride + i * 32))
                                          : make_uint4(0, 0, 0, 0);
    };
    constexpr int kStride = kWarps * kStepPages;
    int pg[2], pn[2];
    uint4 a[16];
    int j0 = pa + warp * kStepPages;
    if (j0 >= pb) return;
    pages_at(j0, pg);
    load(a, pg);
    for (; j0 < pb; j0 += kStride) {
        uint4 nx[16];
        if (j0 + kStride < pb) {
            pages_at(j0 + kStride, pn);
            load(nx, pn);
        }
        // largest |bound| of the 16 pages
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            mx = Ty::vmax(mx, a[i].x & 0x7fff7fffu);
            mx = Ty::vmax(mx, a[i].y & 0x7fff7fffu);
            mx = Ty::vmax(mx, a[i].z & 0x7fff7fffu);
            mx = Ty::vmax(mx, a[i].w & 0x7fff7fffu);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = Ty::vmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0) {
            const float2 f = Ty::unpack(mx);
            P.top[((long long)s * P.hkv + h) * P.top_stride + j0 / kStepPages] = fmaxf(f.x, f.y);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (4 * t < tb - ta) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 b = qf[t][i][lane];
                    Ty::mma(d, a[i].x, a[8 + i].x, a[i].y, a[8 + i].y, b.x, b.y);
                    Ty::mma(d, a[i].z, a[8 + i].z, a[i].w, a[8 + i].w, b.z, b.w);
                }
                const int tok = ta + 4 * t + c;
                if (tok < tb) {
                    float *dst = P.scores + ((long long)(tok - P.t0) * P.hkv + h) * P.score_stride + j0 + r;
                    if (j0 + r < pb) dst[0] = d[0] + d[1];
                    if (j0 + r + 8 < pb) dst[8] = d[2] + d[3];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = nx[i];
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

// Exact score of a page, by one warp: 16 bytes of the bounds a lane, every page in
// the same order.
template <class Ty>
__device__ __forceinline__ double exact_score(const EstimateParams &P, int s, int h, int j, const double *q, int lane) {
    using T = typename Ty::T;
    const int pg = page_of(P.seqs, s, j, P.hdr);
    double acc = 0.0;
    if (pg >= 0) {
        const T *b = static_cast<const T *>(P.bounds) + ((long long)pg * P.hkv + h) * 2 * kD + lane * 8;
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(b));
        const uint32_t *x = reinterpret_cast<const uint32_t *>(&w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Ty::unpack(x[i]);
            acc = fma((double)f.x, q[lane * 8 + 2 * i], acc);
            acc = fma((double)f.y, q[lane * 8 + 2 * i + 1], acc);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    return acc;
}

struct SelectShared {
    double q[2 * kD];  // Q- then Q+
    double exact[kBorder];
    int border[kBorder];
    unsigned hist[512];
    unsigned wsum[kWarps];
    float fsum[kWarps], fmx[kWarps];
    unsigned kmin[kWarps], kmax[kWarps];
    unsigned bin, above, n_border;
    int seq;
};

// Sum over the block of one unsigned per thread, exclusive prefix returned.
__device__ __forceinline__ unsigned block_prefix(unsigned x, unsigned &total, SelectShared &sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) sh.wsum[warp] = inc;
    __syncthreads();
    unsigned before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sh.wsum[w];
        total += sh.wsum[w];
    }
    return before + inc - x;
}

// From the histogram (512 bins, four per thread, bin 511 the largest keys): the
// bin that holds the need-th largest entry, and how many lie above it.
__device__ __forceinline__ void find_bin(unsigned need, SelectShared &sh) {
    unsigned mine[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mine[i] = sh.hist[511 - (4 * threadIdx.x + i)];
        sum += mine[i];
    }
    unsigned total;
    unsigned before = block_prefix(sum, total, sh);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (before < need && need <= before + mine[i]) {
            sh.bin = 511 - (4 * threadIdx.x + i);
            sh.above = before;
        }
        before += mine[i];
    }
    __syncthreads();
}

template <class Ty>
__global__ void __launch_bounds__(kThreads) paged_select_kernel(const __grid_constant__ EstimateParams P) {
    extern __shared__ uint32_t keys[];  // [pages before the token's own]
    __shared__ SelectShared sh;
    const PagedSeqs &S = P.seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tok = P.t0 + (int)(blockIdx.x / P.hkv), h = blockIdx.x % P.hkv;
    if (threadIdx.x == 0) sh.seq = -1;
    __syncthreads();
    for (int s = threadIdx.x; s < S.n_seqs; s += kThreads)
        if (__ldg(S.cu_q + s) <= tok && tok < __ldg(S.cu_q + s + 1)) sh.seq = s;
    __syncthreads();
    const int s = sh.seq;
    if (s < 0) return;  // a row behind the last sequence
    const SeqView v = seq_view(S, s, P.hdr);
    if (v.n == 0) return;
    const int pos = v.len - v.n + (tok - v.q0);
    const long long row = (long long)tok * P.hkv + h;
    int *out = P.blk_idx + row * P.topk;
    if (pos < 0) {  // no key is visible
        for (int i = threadIdx.x; i < P.topk; i += kThreads) out[i] = -1;
        if (threadIdx.x == 0) P.blk_cnt[row] = 0;
        return;
    }
    const int n = pos >> S.page_log2;  // candidates; page n is the token's own
    const int take = min(P.topk - 1, n);
    for (int i = take + 1 + threadIdx.x; i < P.topk; i += kThreads) out[i] = -1;
    if (threadIdx.x == 0) {
        out[take] = n;
        P.blk_cnt[row] = take + 1;
    }
    if (take == n) {
        for (int i = threadIdx.x; i < n; i += kThreads) out[i] = i;
        return;
    }
    if (take == 0) return;

    // Q in 64 bits (thread = channel), its 1-norm in the scores' scale, the largest bound
    float l1, top;
    {
        double up = 0.0, down = 0.0;
        const typename Ty::T *q = static_cast<const typename Ty::T *>(P.q) + (long long)tok * P.q_ts +
                                  (long long)h * P.group * P.q_hs + threadIdx.x;
        for (int g = 0; g < P.group; ++g) {
            const float x = to_f32<Ty>(__ldg(q + (long long)g * P.q_hs));
            up += (double)fmaxf(x, 0.f);
            down += (double)fminf(x, 0.f);
        }
        sh.q[threadIdx.x] = down;
        sh.q[kD + threadIdx.x] = up;
        float fu, fd;
        q_sums<Ty>(P, tok, h, threadIdx.x, fu, fd);
        float sum = fu - fd, mxq = fmaxf(fu, -fd), mxb = 0.f;
        const float *tp = P.top + ((long long)s * P.hkv + h) * P.top_stride;
        for (int i = threadIdx.x; i < (n + kStepPages - 1) / kStepPages; i += kThreads) mxb = fmaxf(mxb, tp[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            mxq = fmaxf(mxq, __shfl_xor_sync(0xffffffffu, mxq, o));
            mxb = fmaxf(mxb, __shfl_xor_sync(0xffffffffu, mxb, o));
        }
        if (lane == 0) {
            sh.fsum[warp] = sum;
            sh.fmx[warp] = mxq;
            sh.wsum[warp] = __float_as_uint(mxb);
        }
    }
    // keys, their smallest and largest
    const float *sc = P.scores + (row - (long long)P.t0 * P.hkv) * P.score_stride;
    unsigned kmin = 0xffffffffu, kmax = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t k = order_key(sc[i]);
        keys[i] = k;
        kmin = min(kmin, k);
        kmax = max(kmax, k);
    }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (lane == 0) {
        sh.kmin[warp] = kmin;
        sh.kmax[warp] = kmax;
    }
    __syncthreads();
    {
        float mxq = 0.f;
        l1 = top = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            l1 += sh.fsum[w];
            mxq = fmaxf(mxq, sh.fmx[w]);
            top = fmaxf(top, __uint_as_float(sh.wsum[w]));
            kmin = min(kmin, sh.kmin[w]);
            kmax = max(kmax, sh.kmax[w]);
        }
        l1 *= part_scale<Ty>(mxq);
    }

    // the take-th largest key: 512 bins over [lo, hi], then over the bin that holds it
    uint32_t lo = kmin, hi = kmax;
    unsigned need = take;
    while (lo < hi) {
        const int bits = 32 - __clz(hi - lo);
        const int shift = max(0, bits - 9);
        for (int i = threadIdx.x; i < 512; i += kThreads) sh.hist[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint32_t k = keys[i];
            if (k >= lo && k <= hi) atomicAdd(&sh.hist[(k - lo) >> shift], 1u);
        }
        __syncthreads();
        find_bin(need, sh);
        need -= sh.above;
        lo += sh.bin << shift;
        hi = min(hi, lo + ((1u << shift) - 1));
        __syncthreads();
    }
    const float t = from_key(lo);
    const float err = (3.0517578125e-5f + 1.1920929e-7f * (float)P.group) * l1 * top;
    // every page outside [t - 2 err, t + 2 err] is decided (0.1 % wider: the roundings here)
    const float width = 2.002f * err + 1e-6f * fabsf(t);
    const uint32_t k_lo = order_key(t - width), k_hi = order_key(t + width);
    // pages in doubt, in page order: each warp counts and lists its quarter
    const int q4 = ((n + 127) >> 7) << 5;  // a multiple of 32
    const int wa = min(n, warp * q4), wb = min(n, wa + q4);
    unsigned n_hi = 0, n_in = 0;
    for (int i = wa + lane; i < wb; i += 32) {
        const uint32_t k = keys[i];
        n_hi += k > k_hi;
        n_in += k >= k_lo && k <= k_hi;
    }
    unsigned all_hi, all_in;
    block_prefix(n_hi, all_hi, sh);
    __syncthreads();
    block_prefix(n_in, all_in, sh);
    const unsigned want = take - all_hi;  // of the pages in doubt
    if (all_in != want) {
        if (all_in <= kBorder) {
            if (threadIdx.x == 0) sh.n_border = 0;
            __syncthreads();
            for (int i = threadIdx.x; i < n; i += kThreads) {
                const uint32_t k = keys[i];
                if (k >= k_lo && k <= k_hi) sh.border[atomicAdd(&sh.n_border, 1u)] = i;  // any order
            }
            __syncthreads();
            for (unsigned i = warp; i < all_in; i += kWarps) {
                const double x = exact_score<Ty>(P, s, h, sh.border[i], sh.q, lane);
                if (lane == 0) sh.exact[i] = x;
            }
            __syncthreads();
            for (unsigned i = threadIdx.x; i < all_in; i += kThreads) {
                const unsigned long long x = order_key64(sh.exact[i]);
                const int xi = sh.border[i];
                unsigned rank = 0;
                for (unsigned j = 0; j < all_in; ++j) {
                    const unsigned long long y = order_key64(sh.exact[j]);
                    rank += y > x || (y == x && sh.border[j] < xi);
                }
                keys[xi] = rank < want ? 0xffffffffu : 0u;
            }
        } else {
            // many pages in doubt (repeated pages): count over the bits of the exact
            // scores, computed anew for each byte
            unsigned long long prefix = 0;
            unsigned left = want;
            for (int shift = 56; shift >= 0; shift -= 8) {
                for (int i = threadIdx.x; i < 512; i += kThreads) sh.hist[i] = 0;
                __syncthreads();
                for (int i = warp; i < n; i += kWarps) {
                    const uint32_t k = keys[i];
                    if (k < k_lo || k > k_hi) continue;
                    const unsigned long long x = order_key64(exact_score<Ty>(P, s, h, i, sh.q, lane));
                    if (lane == 0 && (shift == 56 || (x >> (shift + 8)) == prefix))
                        atomicAdd(&sh.hist[(x >> shift) & 255u], 1u);
                }
                __syncthreads();
                find_bin(left, sh);
                left -= sh.above;
                prefix = (prefix << 8) | sh.bin;
                __syncthreads();
            }
            // larger ones are taken, and the first `left` equal ones
            if (warp == 0) {
                unsigned ties = 0;
                for (int i = 0; i < n; ++i) {
                    const uint32_t k = keys[i];
                    if (k < k_lo || k > k_hi) continue;
                    const unsigned long long x = order_key64(exact_score<Ty>(P, s, h, i, sh.q, lane));
                    const bool yes = x > prefix || (x == prefix && ties < left);
                    ties += x == prefix;
                    __syncwarp();
                    if (lane == 0) keys[i] = yes ? 0xffffffffu : 0u;
                    __syncwarp();
                }
            }
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
        if (yes && to < (unsigned)take) out[to] = i0 + lane;
        at += __popc(bal);
    }
}

constexpr int kTokSmall = 4, kTokLarge = 32;

template <class Ty>
cudaError_t launch(EstimateParams P, cudaStream_t st) {
    const PagedSeqs &S = P.seqs;
    cudaError_t e = cudaFuncSetAttribute(paged_select_kernel<Ty>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMaxBlocks * (int)sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    ProfScope prof("paged_estimate", st);
    const int batch = P.batch;
    for (int t0 = 0; t0 < S.total; t0 += batch) {
        P.t0 = t0;
        P.t1 = min(S.total, t0 + batch);
        const int most = min(S.max_q, P.t1 - P.t0);
        const bool small = most <= kTokSmall;
        const int tok = small ? kTokSmall : kTokLarge;
        P.tiles = (most + tok - 1) / tok;
        P.pages_per_cta = 4 * kWarps * kStepPages;
        const dim3 grid((unsigned)(S.n_seqs * P.tiles), P.hkv, (S.width + P.pages_per_cta - 1) / P.pages_per_cta);
        if (small) paged_scores_kernel<Ty, kTokSmall / 4><<<grid, kThreads, 0, st>>>(P);
        else paged_scores_kernel<Ty, kTokLarge / 4><<<grid, kThreads, 0, st>>>(P);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        paged_select_kernel<Ty><<<(unsigned)(P.t1 - P.t0) * P.hkv, kThreads, S.width * sizeof(uint32_t), st>>>(P);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

EstimatePlan paged_estimate_plan(int total, int n_seqs, int hkv, int width) {
    EstimatePlan p{};
    p.score_stride = (width + 3) & ~3;
    p.top_stride = (width + kStepPages - 1) / kStepPages;
    // 64 MiB of scores at a time: written and read back inside L2
    const long long row = (long long)p.score_stride * 4 * hkv;
    p.batch = (int)std::max<long long>(1, std::min<long long>(total, (64ll << 20) / row));
    p.n_scores = (size_t)p.batch * hkv * p.score_stride;
    p.n_top = (size_t)n_seqs * hkv * p.top_stride;
    return p;
}

cudaError_t run_paged_estimate(const EstimateParams &P, bool fp16, cudaStream_t st) {
    if (P.seqs.n_seqs == 0 || P.seqs.total == 0) return cudaSuccess;
    return fp16 ? launch<Fp16>(P, st) : launch<Bf16>(P, st);
}

}  // namespace minf
