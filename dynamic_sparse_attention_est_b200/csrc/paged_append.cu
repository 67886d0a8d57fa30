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
// bounds of the page need no atomics and do not depend on any order; eight
// threads take a row, 16 channels each as two 16-byte pieces that hold both
// members of their pairs.
#include "internal.h"
#include "paged.cuh"

namespace minf {

namespace {

constexpr int kThreads = 128;
constexpr int kRowsPerPass = kThreads / 8;
constexpr int kUnroll = 2;

// Rotates the 16 channels of a thread's two pieces.  Half split: piece a holds
// channels 8j.., piece b their partners rot/2 further on.  Interleaved: each
// piece holds four whole pairs.
template <class Ty, bool kInterleaved>
__device__ __forceinline__ void rotate(uint4 &a, uint4 &b, const float *row, int half, int ca, bool rot_a, bool rot_b) {
    uint32_t *pa = reinterpret_cast<uint32_t *>(&a), *pb = reinterpret_cast<uint32_t *>(&b);
    if constexpr (kInterleaved) {
        // pairs (2i, 2i + 1): table entry i
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (!(t ? rot_b : rot_a)) continue;
            uint32_t *p = t ? pb : pa;
            const float4 c = __ldg(reinterpret_cast<const float4 *>(row + (ca + t) * 4));
            const float4 s = __ldg(reinterpret_cast<const float4 *>(row + half + (ca + t) * 4));
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = Ty::unpack(p[i]);
                p[i] = Ty::pack(x.x * cc[i] - x.y * ss[i], x.y * cc[i] + x.x * ss[i]);
            }
        }
    } else {
        if (!rot_a) return;
        const float4 *cp = reinterpret_cast<const float4 *>(row + ca * 8);
        const float4 *sp = reinterpret_cast<const float4 *>(row + half + ca * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 c = __ldg(cp + i), s = __ldg(sp + i);
            const float2 xa = Ty::unpack(pa[2 * i]), xb = Ty::unpack(pb[2 * i]);
            const float2 ya = Ty::unpack(pa[2 * i + 1]), yb = Ty::unpack(pb[2 * i + 1]);
            pa[2 * i] = Ty::pack(xa.x * c.x - xb.x * s.x, xa.y * c.y - xb.y * s.y);
            pb[2 * i] = Ty::pack(xb.x * c.x + xa.x * s.x, xb.y * c.y + xa.y * s.y);
            pa[2 * i + 1] = Ty::pack(ya.x * c.z - yb.x * s.z, ya.y * c.w - yb.y * s.w);
            pb[2 * i + 1] = Ty::pack(yb.x * c.z + ya.x * s.z, yb.y * c.w + ya.y * s.w);
        }
    }
}

template <class Ty, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ AppendParams P) {
    using T = typename Ty::T;
    __shared__ uint4 red[2][kThreads / 32][16];
    const PagedSeqs &S = P.seqs;
    const int s = blockIdx.z, h = blockIdx.y;
    const SeqView sv = seq_view(S, s, P.hdr);
    if (sv.n == 0) return;
    const int p0 = sv.len - sv.n;  // position of the first new token
    if (p0 < 0) {
        flag_invalid(P.hdr, BAD_POSITION);
        return;
    }
    const int blk = (p0 >> S.page_log2) + (int)blockIdx.x;
    if (blk > ((sv.len - 1) >> S.page_log2)) return;
    if (P.rope && sv.len > P.rope_rows) {
        flag_invalid(P.hdr, BAD_POSITION);
        return;
    }
    const int pg = page_of(S, s, blk, P.hdr);
    if (pg < 0) return;
    const int first = max(p0, blk << S.page_log2);
    const int nt = min(sv.len, (blk + 1) << S.page_log2) - first;
    const int slot0 = first & (S.page - 1);
    const int tok0 = sv.q0 + (first - p0);
    const int group = P.hq / P.hkv;

    const int j = threadIdx.x & 7, rg = threadIdx.x >> 3;
    const int half = P.rot >> 1;
    // this thread's two 8-channel pieces, and whether they are rotated
    int ca, cb;
    bool rot_a, rot_b;
    if (kInterleaved) {
        ca = 2 * j;
        cb = 2 * j + 1;
        rot_a = ca * 8 < P.rot;
        rot_b = cb * 8 < P.rot;
    } else {
        const int pairs = P.rot >> 4;  // piece pairs inside the rotated part
        rot_a = rot_b = j < pairs;
        ca = rot_a ? j : 2 * j;
        cb = rot_a ? j + pairs : 2 * j + 1;
    }

    const T *kp = static_cast<const T *>(P.k) + (long long)tok0 * P.k_ts + (long long)h * P.k_hs;
    const T *vp = static_cast<const T *>(P.v) + (long long)tok0 * P.v_ts + (long long)h * P.v_hs;
    T *kd = static_cast<T *>(P.k_cache) + (long long)pg * P.kc_ps + ((long long)h * S.page + slot0) * kD;
    T *vd = static_cast<T *>(P.v_cache) + (long long)pg * P.vc_ps + ((long long)h * S.page + slot0) * kD;

    uint4 mn[2], mx[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        mn[i] = make_uint4(Ty::kPosInf2, Ty::kPosInf2, Ty::kPosInf2, Ty::kPosInf2);
        mx[i] = make_uint4(Ty::kNegInf2, Ty::kNegInf2, Ty::kNegInf2, Ty::kNegInf2);
    }
    // rows of the item: nt keys, nt values, then the group's query rows token by token
    const int rows = nt * (2 + (P.q ? group : 0));
    for (int r0 = rg; r0 < rows; r0 += kRowsPerPass * kUnroll) {
        uint4 a[kUnroll], b[kUnroll];
        int kind[kUnroll], tok[kUnroll];
        uint4 *dst[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = r0 + u * kRowsPerPass;
            kind[u] = r >= rows ? 3 : (r < nt ? 0 : (r < 2 * nt ? 1 : 2));
            const T *src = nullptr;
            if (kind[u] == 0) {
                tok[u] = r;
                src = kp + (long long)r * P.k_ts;
                dst[u] = reinterpret_cast<uint4 *>(kd + (long long)r * kD);
            } else if (kind[u] == 1) {
                tok[u] = r - nt;
                src = vp + (long long)tok[u] * P.v_ts;
                dst[u] = reinterpret_cast<uint4 *>(vd + (long long)tok[u] * kD);
            } else if (kind[u] == 2) {
                const int x = r - 2 * nt;
                tok[u] = x / group;
                const int hh = h * group + x % group;
                src = static_cast<const T *>(P.q) + (long long)(tok0 + tok[u]) * P.q_ts + (long long)hh * P.q_hs;
                dst[u] = reinterpret_cast<uint4 *>(static_cast<T *>(P.q_out) + (long long)(tok0 + tok[u]) * P.qo_ts +
                                                   (long long)hh * P.qo_hs);
            }
            if (kind[u] != 3) {
                a[u] = reinterpret_cast<const uint4 *>(src)[ca];
                b[u] = reinterpret_cast<const uint4 *>(src)[cb];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (kind[u] == 3) continue;
            if (kind[u] != 1 && P.rope)
                rotate<Ty, kInterleaved>(a[u], b[u], P.rope + (long long)(first + tok[u]) * P.rot, half, ca, rot_a,
                                         rot_b);
            dst[u][ca] = a[u];
            dst[u][cb] = b[u];
            if (kind[u] == 0) {
                const uint32_t *xa = reinterpret_cast<const uint32_t *>(&a[u]),
                               *xb = reinterpret_cast<const uint32_t *>(&b[u]);
                uint32_t *n0 = reinterpret_cast<uint32_t *>(&mn[0]), *n1 = reinterpret_cast<uint32_t *>(&mn[1]);
                uint32_t *m0 = reinterpret_cast<uint32_t *>(&mx[0]), *m1 = reinterpret_cast<uint32_t *>(&mx[1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    n0[i] = Ty::vmin(n0[i], xa[i]);
                    n1[i] = Ty::vmin(n1[i], xb[i]);
                    m0[i] = Ty::vmax(m0[i], xa[i]);
                    m1[i] = Ty::vmax(m1[i], xb[i]);
                }
            }
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
    // pages that max_q new tokens can touch, wherever in a page the first one lands
    const int pages = (S.max_q + S.page - 2) / S.page + 1;
    const dim3 grid(pages, P.hkv, S.n_seqs);
    ProfScope prof("paged_append", st);
    if (fp16) {
        if (interleaved) paged_append_kernel<Fp16, true><<<grid, kThreads, 0, st>>>(P);
        else paged_append_kernel<Fp16, false><<<grid, kThreads, 0, st>>>(P);
    } else {
        if (interleaved) paged_append_kernel<Bf16, true><<<grid, kThreads, 0, st>>>(P);
        else paged_append_kernel<Bf16, false><<<grid, kThreads, 0, st>>>(P);
    }
    return cudaGetLastError();
}

}  // namespace minf
