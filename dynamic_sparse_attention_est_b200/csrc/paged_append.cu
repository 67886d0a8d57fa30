// paged_append.cu -- rotation of new queries and keys, and their keys and values
// stored into the paged cache.
//
// For a token at position p and channel pair (a, b) of the rotated part,
//     y_a = x_a cos_p - x_b sin_p,   y_b = x_b cos_p + x_a sin_p,
// in fp32 from the stored 16-bit values and the fp32 table row p, rounded once to
// the cache's type.  Each (page, kv-head) also keeps the smallest and the largest
// stored key per channel: the bounds the page selection scores with.
//
// HBM-bound: every row is read and written once.  One CTA takes the new tokens of
// one page for one kv-head (their K rows, V rows and the group's q rows), so the
// bounds of the page need no atomics and do not depend on any order.  Eight
// threads take a row, 16 channels each as two 16-byte pieces that hold both
// members of their pairs; they work on a token's K and V, or on two of its q
// rows, at a time, which share one read of the table.  72 registers keep seven
// CTAs on an SM (eight with 64 registers spill: 38.4 us below).
// 8,192 tokens, 32 q-heads and 8 kv-heads (206 MB): 37.0 us, 5.6 TB/s.
#include "internal.h"
#include "paged.cuh"

namespace minf {

namespace {

constexpr int kThreads = 128;
constexpr int kRowGroups = kThreads / 8;
constexpr int kQRows = 2;  // q rows of a token that a thread takes together

// Rotates the pairs of a thread's two pieces by (cs, sn).  Half split: piece a holds
// channels 8j .. 8j + 7, piece b their partners rot / 2 further on.  Interleaved: each
// piece holds four whole pairs.
template <class Ty, bool kInterleaved>
__device__ __forceinline__ void rotate(uint4 &a, uint4 &b, const float (&cs)[8], const float (&sn)[8]) {
    uint32_t pa[4] = {a.x, a.y, a.z, a.w}, pb[4] = {b.x, b.y, b.z, b.w};
    if constexpr (kInterleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = Ty::unpack(pa[i]), y = Ty::unpack(pb[i]);
            pa[i] = Ty::pack(x.x * cs[i] - x.y * sn[i], x.y * cs[i] + x.x * sn[i]);
            pb[i] = Ty::pack(y.x * cs[4 + i] - y.y * sn[4 + i], y.y * cs[4 + i] + y.x * sn[4 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = Ty::unpack(pa[i]), y = Ty::unpack(pb[i]);
            pa[i] = Ty::pack(x.x * cs[2 * i] - y.x * sn[2 * i], x.y * cs[2 * i + 1] - y.y * sn[2 * i + 1]);
            pb[i] = Ty::pack(y.x * cs[2 * i] + x.x * sn[2 * i], y.y * cs[2 * i + 1] + x.y * sn[2 * i + 1]);
        }
    }
    a = make_uint4(pa[0], pa[1], pa[2], pa[3]);
    b = make_uint4(pb[0], pb[1], pb[2], pb[3]);
}

template <class Ty>
__device__ __forceinline__ void widen(uint4 &mn, uint4 &mx, const uint4 &x) {
    mn = make_uint4(Ty::vmin(mn.x, x.x), Ty::vmin(mn.y, x.y), Ty::vmin(mn.z, x.z), Ty::vmin(mn.w, x.w));
    mx = make_uint4(Ty::vmax(mx.x, x.x), Ty::vmax(mx.y, x.y), Ty::vmax(mx.z, x.z), Ty::vmax(mx.w, x.w));
}

template <class Ty, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 7) paged_append_kernel(const __grid_constant__ AppendParams P) {
    using T = typename Ty::T;
    __shared__ uint4 red[2][kThreads / 32][16];
    const PagedSeqs &S = P.seqs;
    const int h = blockIdx.y;
    int s = blockIdx.z, page = blockIdx.x;  // the page-th page that sequence s appends to
    if (P.packed) {
        auto pages = [&](int x) -> int {
            const SeqView w = seq_view(S, x, P.hdr);
            if (w.n > w.len) flag_invalid(P.hdr, BAD_POSITION);
            return w.n == 0 || w.n > w.len ? 0 : ((w.len - 1) >> S.page_log2) - ((w.len - w.n) >> S.page_log2) + 1;
        };
        if (!find_item<kThreads>(S.n_seqs, blockIdx.x, pages, s, page)) return;
    }
    const SeqView v = seq_view(S, s, P.hdr);
    if (v.n == 0) return;
    const int p0 = v.len - v.n;  // position of the first new token
    if (p0 < 0 || (P.rope && v.len > P.rope_rows)) {
        flag_invalid(P.hdr, BAD_POSITION);
        return;
    }
    const int blk = (p0 >> S.page_log2) + page;
    if (blk > ((v.len - 1) >> S.page_log2)) return;
    const int pg = page_of(S, s, blk, P.hdr);
    if (pg < 0) return;
    const int first = max(p0, blk << S.page_log2);
    const int nt = min(v.len, (blk + 1) << S.page_log2) - first;
    const int slot0 = first & (S.page - 1);
    const long long tok0 = v.q0 + (first - p0);
    const int group = P.hq / P.hkv;

    // this thread's two 8-channel pieces; both or none lie in the rotated part
    const int j = threadIdx.x & 7, rg = threadIdx.x >> 3, pairs = P.rot >> 4;
    const bool rotated = j < pairs;
    const int ca = kInterleaved || !rotated ? 2 * j : j, cb = kInterleaved || !rotated ? 2 * j + 1 : j + pairs;

    uint4 mn[2], mx[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        mn[i] = make_uint4(Ty::kPosInf2, Ty::kPosInf2, Ty::kPosInf2, Ty::kPosInf2);
        mx[i] = make_uint4(Ty::kNegInf2, Ty::kNegInf2, Ty::kNegInf2, Ty::kNegInf2);
    }
    // work of the item: every token's K and V, then every token's first two q rows, ...
    const int chunks = 1 + (P.q ? (group + kQRows - 1) / kQRows : 0);
    int t = rg, c = 0;
    while (t >= nt && c < chunks) {
        t -= nt;
        ++c;
    }
    while (c < chunks) {
        const T *src[kQRows];
        T *dst[kQRows];
        if (c == 0) {
            src[0] = static_cast<const T *>(P.k) + (tok0 + t) * P.k_ts + (long long)h * P.k_hs;
            src[1] = static_cast<const T *>(P.v) + (tok0 + t) * P.v_ts + (long long)h * P.v_hs;
            const long long at = ((long long)h * S.page + slot0 + t) * kD;
            dst[0] = static_cast<T *>(P.k_cache) + (long long)pg * P.kc_ps + at;
            dst[1] = static_cast<T *>(P.v_cache) + (long long)pg * P.vc_ps + at;
        } else {
            const int h0 = h * group + (c - 1) * kQRows;
#pragma unroll
            for (int i = 0; i < kQRows; ++i) {
                src[i] = static_cast<const T *>(P.q) + (tok0 + t) * P.q_ts + (long long)(h0 + i) * P.q_hs;
                dst[i] = static_cast<T *>(P.q_out) + (tok0 + t) * P.qo_ts + (long long)(h0 + i) * P.qo_hs;
            }
        }
        const int n = c == 0 ? 2 : min(kQRows, group - (c - 1) * kQRows);
        uint4 a[kQRows], b[kQRows];
#pragma unroll
        for (int i = 0; i < kQRows; ++i)
            if (i < n) {
                a[i] = reinterpret_cast<const uint4 *>(src[i])[ca];
                b[i] = reinterpret_cast<const uint4 *>(src[i])[cb];
            }
        if (rotated) {
            float cs[8], sn[8];
            const float4 *row = reinterpret_cast<const float4 *>(P.rope + (long long)(first + t) * P.rot + 8 * j);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 x = __ldg(row + i), y = __ldg(row + (P.rot >> 3) + i);
                cs[4 * i] = x.x, cs[4 * i + 1] = x.y, cs[4 * i + 2] = x.z, cs[4 * i + 3] = x.w;
                sn[4 * i] = y.x, sn[4 * i + 1] = y.y, sn[4 * i + 2] = y.z, sn[4 * i + 3] = y.w;
            }
            rotate<Ty, kInterleaved>(a[0], b[0], cs, sn);
            if (c > 0 && n > 1) rotate<Ty, kInterleaved>(a[1], b[1], cs, sn);
        }
        if (c == 0) {
            widen<Ty>(mn[0], mx[0], a[0]);
            widen<Ty>(mn[1], mx[1], b[0]);
        }
#pragma unroll
        for (int i = 0; i < kQRows; ++i)
            if (i < n) {
                reinterpret_cast<uint4 *>(dst[i])[ca] = a[i];
                reinterpret_cast<uint4 *>(dst[i])[cb] = b[i];
            }
        t += kRowGroups;
        while (t >= nt) {
            t -= nt;
            ++c;
        }
    }
    if (!P.k_bounds) return;
    // join the row groups: four in a warp, then the warps
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        uint32_t *n = reinterpret_cast<uint32_t *>(&mn[t]), *m = reinterpret_cast<uint32_t *>(&mx[t]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int o = 8; o < 32; o <<= 1) {
                n[i] = Ty::vmin(n[i], __shfl_xor_sync(0xffffffffu, n[i], o));
                m[i] = Ty::vmax(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
            }
    }
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) < 8) {
        red[0][warp][ca] = mn[0];
        red[0][warp][cb] = mn[1];
        red[1][warp][ca] = mx[0];
        red[1][warp][cb] = mx[1];
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int which = threadIdx.x >> 4, c = threadIdx.x & 15;
        uint4 *slot = reinterpret_cast<uint4 *>(static_cast<T *>(P.k_bounds) +
                                                (((long long)pg * P.hkv + h) * 2 + which) * kD) + c;
        uint4 acc = red[which][0][c];
        uint32_t *x = reinterpret_cast<uint32_t *>(&acc);
        auto join = [&](const uint4 &o) {
            const uint32_t *y = reinterpret_cast<const uint32_t *>(&o);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = which ? Ty::vmax(x[i], y[i]) : Ty::vmin(x[i], y[i]);
        };
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) join(red[which][w][c]);
        if (slot0 > 0) join(*slot);  // the page held keys before: its bounds cover them
        *slot = acc;
    }
}

}  // namespace

cudaError_t run_paged_append(const AppendParams &P, bool fp16, bool interleaved, cudaStream_t st) {
    const PagedSeqs &S = P.seqs;
    if (S.n_seqs == 0 || S.total == 0) return cudaSuccess;
    // Pages that max_q new tokens can touch, wherever in a page the first one lands, for
    // every sequence; or, where that is far above what all tokens can touch (a chunk
    // beside many single tokens), that bound, each CTA finding its page: 256 single tokens
    // and a chunk of 8,192 (pages of 16) take 51 us packed, 582 us by sequence.
    const long long pages = (S.max_q + S.page - 2) / S.page + 1, all = S.total / S.page + 2ll * S.n_seqs;
    AppendParams A = P;
    A.packed = pages * S.n_seqs > 2 * all;
    const dim3 grid((unsigned)(A.packed ? all : pages), P.hkv, A.packed ? 1 : S.n_seqs);
    ProfScope prof("paged_append", st);
    if (fp16) {
        if (interleaved) paged_append_kernel<Fp16, true><<<grid, kThreads, 0, st>>>(A);
        else paged_append_kernel<Fp16, false><<<grid, kThreads, 0, st>>>(A);
    } else {
        if (interleaved) paged_append_kernel<Bf16, true><<<grid, kThreads, 0, st>>>(A);
        else paged_append_kernel<Bf16, false><<<grid, kThreads, 0, st>>>(A);
    }
    return cudaGetLastError();
}

}  // namespace minf
