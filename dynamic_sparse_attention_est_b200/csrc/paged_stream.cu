// paged_stream.cu -- attention of few query rows over many stored keys: decoding
// steps over everything stored, and every token over its own selected pages.
//
// A work item is one kv-head of one sequence (dense) or token (selected pages)
// with up to 8 NT of its query rows (tokens x the group's q-heads).  Its K and V
// are read once and used for a handful of rows, so the time is that of reading
// them: HBM when each key belongs to one item, L2 when the tokens of a chunk
// share their pages.  The kernel is built around the loads.
//
//   * Warps take 16-key groups and keep a softmax state of their own; nothing
//     synchronises until the end of an item.  Each warp feeds itself: a ring of two
//     or three groups (8 KB of K and V each) that its first lane fills by TMA, 192 KB
//     in flight on an SM.  The boxes are 128-byte swizzled, so ldmatrix reads them
//     without bank conflicts.
//   * With keys on the 16-row side and query rows on the 8-column side
//     (m16n8k16: S^T = K Q^T, then O^T += V^T P^T), four or eight q-heads of a
//     group fill the tile, where a 128-row tensor-memory tile would compute 16 to
//     32 rows for each one used.
//   * Running maximum and sum per row in fp32, log2 domain; the maximum moves
//     only past a margin, which one vote per group decides.
//   * The work of a call is cut into equal shares, one for each CTA of a single wave,
//     wherever in an item a share ends: the 16-key groups of all sequences (each CTA
//     takes the prefix sums of the lengths itself, so that a captured launch follows
//     them), or the entries of all page lists.  An item's parts are joined by a second
//     small kernel in a fixed order.  Lists are cut as if they were topk long: where they
//     are far shorter, the CTAs whose shares lie behind the counts have nothing to do.
#include <algorithm>
#include <cstring>

#include "internal.h"
#include "paged.cuh"

namespace minf {

namespace {

constexpr int kGroup = 16;         // keys per warp step
constexpr int kStreamGrid = 296;   // two CTAs (their rings: 192 KB) on each of 148 SMs
constexpr int kOPad = 132;         // floats per row of the CTA's join buffer
constexpr uint32_t kBoxBytes = 2048;             // 16 keys x 64 channels
constexpr uint32_t kStageBytes = 4 * kBoxBytes;  // K low, K high, V low, V high channels
constexpr uint32_t kRingBytes = 12 * kStageBytes;
constexpr uint32_t kSmemBar = kRingBytes;         // mbarriers, abort flag
// [n_seqs + 1] units before a sequence (dense): beside the rings there is room for two CTAs
// on an SM up to 2,015 sequences; from there on the shares run in two waves
constexpr uint32_t kSmemPre = kSmemBar + 256;

// Warps of a CTA and groups in flight to each, by the registers that NT row tiles
// take: six warps of two with one tile (313 tokens with 64 pages of 32: 64.6 us; four of
// three: 75.4 us), four of three with two tiles.
template <int NT>
struct Shape {
    static constexpr int kWarps = NT == 1 ? 6 : 4, kStages = 12 / kWarps, kThreads = 32 * kWarps;
};
constexpr int kJoinWarps = 4;

struct StreamParams {
    CUtensorMap tmap_k;  // {128, P, hkv, pages}, box {64, 16, 1, 1}
    CUtensorMap tmap_v;
    PagedAttnParams a;
};

// 8x8 transpose of 16-bit elements over a warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// The pages a warp walks: 32 (logical block, page) entries at a time, one per
// lane, the next 32 loaded ahead (once the first loads of keys are out: each entry
// takes two or three dependent reads).
template <bool kSparse>
struct PageWalk {
    const PagedSeqs *S;
    WsHeader *hdr;
    const int *list;  // selected blocks (sparse)
    int seq, n_slots, last_blk, base;
    int blk, pg, blk_next, pg_next;

    __device__ __forceinline__ void fetch(int slot, int &b, int &p) const {
        b = p = -1;
        if (slot >= n_slots) return;
        if (kSparse) {
            const int before = __ldg(list + max(slot - 1, 0));
            b = __ldg(list + slot);
            // an entry that is negative, past the query's own page or not above the one before it is left out
            if (b < 0 || b > last_blk || (slot > 0 && b <= before)) {
                b = -1;
                return;
            }
        } else {
            b = slot;
        }
        p = page_of(*S, seq, b, hdr);
    }
    __device__ __forceinline__ void start(int slot, int lane) {
        base = slot;
        fetch(base + lane, blk, pg);
        blk_next = pg_next = -1;
    }
    __device__ __forceinline__ void ahead(int lane) { fetch(base + 32 + lane, blk_next, pg_next); }
    // Entry `slot`, not before the one asked for last; the whole warp calls it.
    __device__ __forceinline__ void get(int slot, int lane, int &b, int &p) {
        while (slot >= base + 32) {
            base += 32;
            blk = blk_next;
            pg = pg_next;
            ahead(lane);
        }
        b = __shfl_sync(0xffffffffu, blk, slot - base);
        p = __shfl_sync(0xffffffffu, pg, slot - base);
    }
};

struct Item {
    int seq, h, row0, rows;  // rows row0 .. row0 + rows - 1 of the (token, q-head of the group) list
    int tok0;                // q row of the sequence's first token (sparse: of the token)
    int pos0;                // position of that token
    int len;                 // stored tokens
};

template <class Ty, int NT>
struct State {
    float m[NT][2], l[NT][2];
    float o[NT][8][4];
};

// One 16-key group at shared address `stage`: scores, softmax, P V.
template <class Ty, int NT>
__device__ __forceinline__ void step(State<Ty, NT> &st, uint32_t stage, const uint32_t (&qf)[NT][8][2], int key0,
                                     const int (&lim)[NT][2], int min_lim, int len, float sl2, int lane) {
    const int r = lane >> 2, c = lane & 3;
    float s[2][NT][4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[x][t][i] = 0.f;
    // K: rows (keys) lane % 16, 16-byte chunk 2 kk + lane / 16 of the 16 in a row
    {
        const int row = lane & 15;
        const uint32_t base = stage + row * 128;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            uint32_t a[4];
            const int chunk = (2 * kk & 7) + (lane >> 4);
            ldmatrix4(a, base + (kk >> 2) * kBoxBytes + ((chunk ^ (row & 7)) << 4));
#pragma unroll
            for (int t = 0; t < NT; ++t) Ty::mma(s[kk & 1][t], a[0], a[1], a[2], a[3], qf[t][kk][0], qf[t][kk][1]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[0][t][i] += s[1][t][i];
    }
    if (key0 + kGroup > min_lim) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (key0 + r >= lim[t][i]) s[0][t][i] = -INFINITY;
                if (key0 + r + 8 >= lim[t][i]) s[0][t][2 + i] = -INFINITY;
            }
    }
    bool grow = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) grow |= fmaxf(s[0][t][i], s[0][t][2 + i]) * sl2 > st.m[t][i] + Ty::kLag;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = fmaxf(s[0][t][i], s[0][t][2 + i]);
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16)) * sl2;
                if (x > st.m[t][i] + Ty::kLag) {  // the same decision in the eight lanes of a row
                    const float a = ex2_approx(st.m[t][i] - x);  // 0 from -inf
                    st.m[t][i] = x;
                    st.l[t][i] *= a;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        st.o[t][e][i] *= a;
                        st.o[t][e][2 + i] *= a;
                    }
                }
            }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float sub = st.m[t][i] == -INFINITY ? 0.f : st.m[t][i] - Ty::kShift;
            p[i] = ex2_approx(fmaf(s[0][t][i], sl2, -sub));
            p[2 + i] = ex2_approx(fmaf(s[0][t][2 + i], sl2, -sub));
            st.l[t][i] += p[i] + p[2 + i];
        }
        // P is rounded to the cache's type for the product (half a step, 2^-8 of a
        // bf16 weight: the size of the output's own rounding); the sum keeps fp32.  P in
        // two parts leaves the output's rounding alone (error against 64 bits 0.0017 of
        // the norm instead of 0.0023 in bf16, 0.00021 instead of 0.00029 in fp16) and
        // takes 1 % longer on 64 sequences of up to 32K tokens, 7 % on one sequence's 100
        // pages, 5 to 8 % on chunks over their pages: not worth it beside the prompt's
        // kernels, which round alike.
        pb[t][0] = transpose8x8(Ty::pack(p[0], p[1]));
        pb[t][1] = transpose8x8(Ty::pack(p[2], p[3]));
    }
    // V^T: 16 channels of the 16 keys, transposed on the way
    const int key = (lane & 7) + ((lane >> 4) << 3), hc = (lane >> 3) & 1;
    const uint32_t vb = stage + 2 * kBoxBytes + key * 128;
    const bool tail = key0 + kGroup > len;
    uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
    if (tail) {  // slots behind the stored tokens may hold anything
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int k = key0 + 8 * x + 2 * c;
            keep[x] = (k < len ? 0xffffu : 0u) | (k + 1 < len ? 0xffff0000u : 0u);
        }
    }
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        uint32_t a[4];
        const int chunk = (2 * m & 7) + hc;
        ldmatrix4_trans(a, vb + (m >> 2) * kBoxBytes + ((chunk ^ (key & 7)) << 4));
        if (tail) {
            a[0] &= keep[0];
            a[1] &= keep[0];
            a[2] &= keep[1];
            a[3] &= keep[1];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) Ty::mma(st.o[t][m], a[0], a[1], a[2], a[3], pb[t][0], pb[t][1]);
    }
}

struct Ring {
    uint32_t stage0, bar0;  // this warp's stages and mbarriers
    uint32_t phase;         // bit per stage: parity of its next fill
};

// Groups g0 .. g1 - 1 of an item, joined over the CTA's warps; the result goes to
// the output, or to partial slot `slot` (>= 0).
template <class Ty, int NT, bool kSparse>
__device__ __forceinline__ void run_piece(const StreamParams &SP, const Item &it, const int *list, int n_list, int g0,
                                          int g1, int slot, Ring &ring, const WaitCtl &wc, float *sm_o,
                                          float2 *sm_ml) {
    using T = typename Ty::T;
    constexpr int kWarps = Shape<NT>::kWarps, kStages = Shape<NT>::kStages;
    const PagedAttnParams &P = SP.a;
    const PagedSeqs &S = P.seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int gp_log2 = S.page_log2 - 4;  // 16-key groups per page
    const int gp_mask = (1 << gp_log2) - 1;

    PageWalk<kSparse> walk;
    walk.S = &S;
    walk.hdr = P.hdr;
    walk.list = list;
    walk.seq = it.seq;
    walk.last_blk = kSparse ? it.pos0 >> S.page_log2 : 0;
    walk.n_slots = min(kSparse ? n_list : (it.len + S.page - 1) >> S.page_log2, ((g1 - 1) >> gp_log2) + 1);
    walk.start((g0 + warp) >> gp_log2, lane);

    int stage_key = -1;  // lane s: first key of the group in stage s, -1 if none
    auto fill = [&](int st, int g) {
        int key0 = -1, pg = -1;
        if (g < g1) {
            int blk;
            walk.get(g >> gp_log2, lane, blk, pg);
            key0 = pg >= 0 ? (blk << S.page_log2) + (g & gp_mask) * kGroup : -1;
            if (key0 >= it.len) key0 = -1;
        }
        if (lane == st) stage_key = key0;
        if (key0 >= 0 && lane == 0) {
            const uint32_t bar = ring.bar0 + st * 8, dst = ring.stage0 + st * kStageBytes;
            const int row = (g & gp_mask) * kGroup;
            mbar_arrive_expect_tx(bar, kStageBytes);
            tma_load_4d(dst, &SP.tmap_k, bar, 0, row, it.h, pg);
            tma_load_4d(dst + kBoxBytes, &SP.tmap_k, bar, 64, row, it.h, pg);
            tma_load_4d(dst + 2 * kBoxBytes, &SP.tmap_v, bar, 0, row, it.h, pg);
            tma_load_4d(dst + 3 * kBoxBytes, &SP.tmap_v, bar, 64, row, it.h, pg);
        }
    };
    bool ok = !*wc.abort_flag;
    ok = __all_sync(0xffffffffu, ok);
    if (ok)
#pragma unroll
        for (int st = 0; st < kStages; ++st) fill(st, g0 + warp + st * kWarps);
    walk.ahead(lane);

    // query fragments: row r of each 8-row tile, channels 16 kk + 2 c, + 1, + 8, + 9
    uint32_t qf[NT][8][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int x = it.row0 + t * 8 + r;
        const bool in = t * 8 + r < it.rows;
        const T *src = static_cast<const T *>(P.q) + (long long)(it.tok0 + x / P.group) * P.q_ts +
                       (long long)(it.h * P.group + x % P.group) * P.q_hs + c * 2;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                qf[t][kk][i] = in ? __ldg(reinterpret_cast<const unsigned *>(src + kk * 16 + i * 8)) : 0u;
    }
    // keys each of this lane's score columns sees
    int lim[NT][2];
    const int min_lim = it.pos0 + it.row0 / P.group + 1;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int x = min(it.row0 + t * 8 + 2 * c + i, it.row0 + it.rows - 1);
            lim[t][i] = it.pos0 + x / P.group + 1;
        }
    State<Ty, NT> st;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        st.m[t][0] = st.m[t][1] = -INFINITY;
        st.l[t][0] = st.l[t][1] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[t][e][i] = 0.f;
    }

    if (ok) {
        int s = 0;
        for (int g = g0 + warp; g < g1; g += kWarps) {
            const int key0 = __shfl_sync(0xffffffffu, stage_key, s);
            if (key0 >= 0) {
                const bool got = wait_bounded(ring.bar0 + s * 8, (ring.phase >> s) & 1, wc, wait_site(7, s, g));
                if (__any_sync(0xffffffffu, !got)) {
                    ok = false;
                    break;
                }
                ring.phase ^= 1u << s;
                step<Ty, NT>(st, ring.stage0 + s * kStageBytes, qf, key0, lim, min_lim, it.len, P.scale_log2, lane);
                __syncwarp();  // every lane has read the stage
            }
            fill(s, g + kStages * kWarps);
            s = s == kStages - 1 ? 0 : s + 1;
        }
        if (!ok) {  // let the loads in flight land before the CTA exits
            volatile int no_abort = 0;
            const WaitCtl drain{&no_abort, nullptr, 50000000ull};
            for (int x = 0; x < kStages; ++x)
                if (__shfl_sync(0xffffffffu, stage_key, x) >= 0)
                    wait_bounded(ring.bar0 + x * 8, (ring.phase >> x) & 1, drain);
        }
    }

    // ---- join the warps (the rings are idle: the buffer lies over them)
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float l = st.l[t][i];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (r == 0) sm_ml[warp * 8 * NT + t * 8 + 2 * c + i] = make_float2(st.m[t][i], l);
            float *dst = sm_o + (size_t)(warp * 8 * NT + t * 8 + 2 * c + i) * kOPad + r;
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                dst[16 * m] = st.o[t][m][i];
                dst[16 * m + 8] = st.o[t][m][2 + i];
            }
        }
    __syncthreads();
    for (int row = warp; row < it.rows; row += kWarps) {
        float2 ml[kWarps];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            ml[w] = sm_ml[w * 8 * NT + row];
            m = fmaxf(m, ml[w].x);
        }
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float a = ml[w].x == -INFINITY ? 0.f : ex2_approx(ml[w].x - m);
            const float4 x = *reinterpret_cast<const float4 *>(sm_o + (size_t)(w * 8 * NT + row) * kOPad + lane * 4);
            l = fmaf(ml[w].y, a, l);
            o.x = fmaf(x.x, a, o.x);
            o.y = fmaf(x.y, a, o.y);
            o.z = fmaf(x.z, a, o.z);
            o.w = fmaf(x.w, a, o.w);
        }
        if (slot >= 0) {
            reinterpret_cast<float4 *>(P.part_o)[((size_t)slot * 8 * NT + row) * 32 + lane] = o;
            if (lane == 0) P.part_ml[(size_t)slot * 8 * NT + row] = make_float2(m, l);
        } else {
            const int x = it.row0 + row, tok = it.tok0 + x / P.group, hh = it.h * P.group + x % P.group;
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // a NaN sum stays one
            uint2 *dst = reinterpret_cast<uint2 *>(static_cast<T *>(P.out) + (long long)tok * P.o_ts +
                                                   (long long)hh * P.o_hs) + lane;
            *dst = make_uint2(Ty::pack(o.x * inv, o.y * inv), Ty::pack(o.z * inv, o.w * inv));
            if (lane == 0 && P.lse)
                P.lse[(size_t)tok * P.hq + hh] =
                    l == 0.f ? -INFINITY : (m - Ty::kShift + __log2f(l)) * 0.69314718055994531f;
        }
    }
    fence_proxy_async_smem();  // the buffer's accesses come before the next piece's loads
    __syncthreads();
}

// Barriers and ring of the calling warp; the whole CTA calls it.
template <int NT>
__device__ __forceinline__ Ring ring_init(uint8_t *smem, WaitCtl &wc, const StreamParams &SP) {
    constexpr int kWarps = Shape<NT>::kWarps, kStages = Shape<NT>::kStages;
    const PagedAttnParams &P = SP.a;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kSmemBar);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + kWarps * kStages);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * kStages; ++i) mbar_init(smem_u32(bars + i), 1);
        *abort_flag = 0;
        fence_mbar_init();
    } else if (threadIdx.x == 32) {
        tma_prefetch_desc(&SP.tmap_k);
        tma_prefetch_desc(&SP.tmap_v);
    }
    __syncthreads();
    wc.abort_flag = abort_flag;
    wc.status = &P.hdr->status;
    wc.limit_ns = P.wait_limit_ns;
    return {smem_u32(smem) + warp * kStages * kStageBytes, smem_u32(bars + warp * kStages), 0u};
}

__device__ __forceinline__ uint8_t *align_1k(uint8_t *p) {
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

static_assert(6 * 8 * (kOPad * 4 + 8) <= kRingBytes && 4 * 16 * (kOPad * 4 + 8) <= kRingBytes, "the join buffer fits over the rings");

// CTAs that share `total` 16-key groups: four groups at least to each, so that none
// of them is without work and an item's parts sit in consecutive CTAs.
__device__ __forceinline__ int dense_ctas(long long total) {
    return (int)min((long long)kStreamGrid, max(1ll, total >> 2));
}
// a / b for a >= 0, b > 0: the 64-bit division takes a fifth of a microsecond, and
// nearly all calls fit 32 bits.
__device__ __forceinline__ long long quot(long long a, long long b) {
    return ((unsigned long long)(a | b) >> 32) ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// ------------------------------------------------------------------ dense
// 16-key groups of a sequence, over its kv-heads and row tiles.
template <int NT>
__device__ __forceinline__ long long seq_units(const SeqView &v, const PagedAttnParams &P) {
    const int tiles = (v.n * P.group + 8 * NT - 1) / (8 * NT);
    return (long long)tiles * P.hkv * ((v.len + kGroup - 1) / kGroup);
}

// Work units: 16-key groups, sequence after sequence; within one, (kv-head, row
// tile) after one another.  CTA c of C takes units [U c / C, U (c + 1) / C).
template <class Ty, int NT>
__global__ void __launch_bounds__(Shape<NT>::kThreads, 2)
    paged_dense_kernel(const __grid_constant__ StreamParams SP) {
    constexpr int kWarps = Shape<NT>::kWarps, kThreads = Shape<NT>::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1k(smem_raw);
    float *sm_o = reinterpret_cast<float *>(smem);
    float2 *sm_ml = reinterpret_cast<float2 *>(smem + kWarps * 8 * NT * kOPad * 4);
    long long *pre = reinterpret_cast<long long *>(smem + kSmemPre);
    __shared__ long long warp_sum[kWarps];
    const PagedAttnParams &P = SP.a;
    const PagedSeqs &S = P.seqs;
    WaitCtl wc;
    Ring ring = ring_init<NT>(smem, wc, SP);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int per = (S.n_seqs + kThreads - 1) / kThreads;
    const int sa = min(threadIdx.x * per, S.n_seqs), sb = min(sa + per, S.n_seqs);
    auto units = [&](int s) { return seq_units<NT>(seq_view(S, s, P.hdr), P); };
    long long mine = 0;
    for (int s = sa; s < sb; ++s) mine += units(s);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    long long at = inc - mine;
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    for (int s = sa; s < sb; ++s) {
        pre[s] = at;
        at += units(s);
    }
    if (threadIdx.x == 0) {
        long long t = 0;
        for (int w = 0; w < kWarps; ++w) t += warp_sum[w];
        pre[S.n_seqs] = t;
    }
    __syncthreads();
    const long long total = pre[S.n_seqs];
    if (blockIdx.x == 0)  // the joining kernel's copy
        for (int x = threadIdx.x; x <= S.n_seqs; x += kThreads) P.plan[x] = pre[x];
    launch_dependents();

    // sequences with new tokens and nothing stored: their rows see no key
    for (int s = blockIdx.x; s < S.n_seqs; s += gridDim.x) {
        const SeqView v = seq_view(S, s, P.hdr);
        if (v.n == 0 || v.len > 0) continue;
        for (int i = threadIdx.x; i < v.n * P.hq * 16; i += kThreads) {
            const int row = i >> 4, tok = v.q0 + row / P.hq, hh = row % P.hq;
            reinterpret_cast<uint4 *>(static_cast<typename Ty::T *>(P.out) + (long long)tok * P.o_ts +
                                      (long long)hh * P.o_hs)[i & 15] = make_uint4(0, 0, 0, 0);
            if ((i & 15) == 0 && P.lse) P.lse[(size_t)tok * P.hq + hh] = -INFINITY;
        }
    }

    const int n_cta = dense_ctas(total);
    const long long me = min((int)blockIdx.x, n_cta);
    const long long u0 = quot(total * me, n_cta), u1 = quot(total * min(me + 1, (long long)n_cta), n_cta);
    long long u = u0;
    int s = 0;
    {
        int lo = 0, hi = S.n_seqs;  // last sequence starting at or before u
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= u) lo = mid;
            else hi = mid;
        }
        s = lo;
    }
    while (u < u1) {
        while (pre[s + 1] <= u) ++s;  // also steps over sequences without units
        const SeqView v = seq_view(S, s, P.hdr);
        const int groups = (v.len + kGroup - 1) / kGroup;
        const int tiles = (v.n * P.group + 8 * NT - 1) / (8 * NT);
        const long long rem = u - pre[s];
        const int in_seq = (int)quot(rem, groups), ga = (int)(rem - (long long)in_seq * groups);
        const int gb = (int)min((long long)groups, ga + (u1 - u));
        Item it;
        it.seq = s;
        it.h = in_seq / tiles;
        it.row0 = (in_seq % tiles) * 8 * NT;
        it.rows = min(8 * NT, v.n * P.group - it.row0);
        it.tok0 = v.q0;
        it.pos0 = v.len - v.n;
        it.len = v.len;
        const bool whole = ga == 0 && gb == groups;
        // a cut piece is a CTA's first or its last
        const int slot = whole ? -1 : 2 * (int)blockIdx.x + (u == u0 ? 0 : 1);
        run_piece<Ty, NT, false>(SP, it, nullptr, 0, ga, gb, slot, ring, wc, sm_o, sm_ml);
        u += gb - ga;
    }
}

// ------------------------------------------------------------------ selected pages
// Work units: entries of the page lists (topk to an item, those behind its count
// empty), item after item; an item is a (token, kv-head, row tile).  CTA c of C takes
// units [U c / C, U (c + 1) / C); with a CTA to each item, that is its list.
template <class Ty, int NT>
__global__ void __launch_bounds__(Shape<NT>::kThreads, 2)
    paged_sparse_kernel(const __grid_constant__ StreamParams SP) {
    constexpr int kWarps = Shape<NT>::kWarps, kThreads = Shape<NT>::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1k(smem_raw);
    float *sm_o = reinterpret_cast<float *>(smem);
    float2 *sm_ml = reinterpret_cast<float2 *>(smem + kWarps * 8 * NT * kOPad * 4);
    __shared__ int found;
    const PagedAttnParams &P = SP.a;
    const PagedSeqs &S = P.seqs;
    WaitCtl wc;
    Ring ring = ring_init<NT>(smem, wc, SP);
    launch_dependents();
    if (blockIdx.x == 0)  // no row leads to a sequence that ends before it begins: report it here
        for (int s = threadIdx.x; s < S.n_seqs; s += kThreads) seq_view(S, s, P.hdr);
    const int tiles = (P.group + 8 * NT - 1) / (8 * NT);
    const long long total = (long long)S.total * P.hkv * tiles * P.topk;
    const long long u0 = quot(total * blockIdx.x, gridDim.x), u1 = quot(total * (blockIdx.x + 1), gridDim.x);
    const int gp = S.page >> 4;
    for (long long u = u0; u < u1;) {
        const int item = (int)quot(u, P.topk), a = (int)(u - (long long)item * P.topk);
        const int b = (int)min((long long)P.topk, a + (u1 - u));
        const int slot = a == 0 && b == P.topk ? -1 : 2 * (int)blockIdx.x + (u == u0 ? 0 : 1);
        u += b - a;
        const int rt = item % tiles, h = (item / tiles) % P.hkv, t = item / tiles / P.hkv;
        if (threadIdx.x == 0) found = -1;
        __syncthreads();
        for (int s = threadIdx.x; s < S.n_seqs; s += kThreads)
            if (__ldg(S.cu_q + s) <= t && t < __ldg(S.cu_q + s + 1)) atomicMax(&found, s);
        __syncthreads();
        const int s = found;
        __syncthreads();        // read by all before it is set again
        if (s < 0) continue;  // a row behind the last sequence
        const SeqView v = seq_view(S, s, P.hdr);
        if (v.n == 0) continue;
        Item it;
        it.seq = s;
        it.h = h;
        it.row0 = rt * 8 * NT;
        it.rows = min(8 * NT, P.group - it.row0);
        it.tok0 = t;
        it.pos0 = v.len - v.n + (t - v.q0);
        it.len = v.len;
        const int li = t * P.hkv + h;
        int cnt = __ldg(P.blk_cnt + li);
        if (cnt < 0 || cnt > P.topk) {
            flag_invalid(P.hdr, BAD_BLOCK);
            cnt = max(0, min(cnt, P.topk));
        }
        if (it.pos0 < 0) cnt = 0;
        run_piece<Ty, NT, true>(SP, it, P.blk_idx + (long long)li * P.topk, cnt, min(a, cnt) * gp, min(b, cnt) * gp, slot,
                                ring, wc, sm_o, sm_ml);
    }
}

// ------------------------------------------------------------------ join
// One CTA per (item, row): the parts in order, a quarter of them to each warp, four in
// flight.  Which parts an item has follows from its units and the shares, as the
// kernel before cut them; all that needs no result of that kernel is done while it
// still runs.
template <class Ty, int NT, bool kSparse>
__device__ __forceinline__ void join_row(const PagedAttnParams &P) {
    constexpr int kWarps = kJoinWarps, kThreads = 32 * kJoinWarps;
    __shared__ float4 so[kWarps][32];
    __shared__ float2 sml[kWarps];
    __shared__ long long sums[kWarps][2];
    const PagedSeqs &S = P.seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int id = blockIdx.x, row = blockIdx.y;
    int h, x, tok0, n_cta;
    long long first, units, total;  // the item's units, of all
    if (kSparse) {
        const int tiles = (P.group + 8 * NT - 1) / (8 * NT);
        h = (id / tiles) % P.hkv;
        x = (id % tiles) * 8 * NT + row;
        tok0 = id / tiles / P.hkv;
        if (x >= P.group) return;
        // rows behind the last sequence, and rows of one left out, are not written
        int hit = -1;
        for (int s = threadIdx.x; s < S.n_seqs; s += kThreads)
            if (__ldg(S.cu_q + s) <= tok0 && tok0 < __ldg(S.cu_q + s + 1) && seq_view(S, s, P.hdr).n > 0) hit = s;
        if (!__syncthreads_or(hit >= 0)) return;
        units = P.topk;
        first = (long long)id * units;
        total = (long long)S.total * P.hkv * tiles * units;
        n_cta = P.n_slots / 2;
    } else {
        const int rt_max = (S.max_q * P.group + 8 * NT - 1) / (8 * NT);
        const int s = id / rt_max / P.hkv, rt = id % rt_max;
        h = (id / rt_max) % P.hkv;
        x = rt * 8 * NT + row;
        const SeqView v = seq_view(S, s, P.hdr);
        tok0 = v.q0;
        if (x >= v.n * P.group || v.len == 0) return;
        units = (v.len + kGroup - 1) / kGroup;
        const long long before = (h * (long long)((v.n * P.group + 8 * NT - 1) / (8 * NT)) + rt) * units;
        if (S.n_seqs <= kThreads) {
            long long mine = 0;
            if (threadIdx.x < S.n_seqs) mine = seq_units<NT>(seq_view(S, threadIdx.x, P.hdr), P);
            long long head = threadIdx.x < s ? mine : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                mine += __shfl_xor_sync(0xffffffffu, mine, o);
                head += __shfl_xor_sync(0xffffffffu, head, o);
            }
            if (lane == 0) {
                sums[warp][0] = mine;
                sums[warp][1] = head;
            }
            __syncthreads();
            total = first = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                total += sums[w][0];
                first += sums[w][1];
            }
        } else {
            wait_for_primary();
            total = P.plan[S.n_seqs];
            first = P.plan[s];
        }
        first += before;
        n_cta = dense_ctas(total);
    }
    // CTA c holds units total c / n_cta .. total (c + 1) / n_cta - 1
    const int c0 = (int)quot((first + 1) * n_cta - 1, total), c1 = (int)quot((first + units) * n_cta - 1, total);
    if (c0 == c1) return;  // whole, already written
    const int n_part = c1 - c0 + 1;
    const int slot0 = 2 * c0 + (first == quot(total * c0, n_cta) ? 0 : 1);
    wait_for_primary();
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float a, float pl, const float4 &o) {
        l = fmaf(pl, a, l);
        acc.x = fmaf(o.x, a, acc.x);
        acc.y = fmaf(o.y, a, acc.y);
        acc.z = fmaf(o.z, a, acc.z);
        acc.w = fmaf(o.w, a, acc.w);
    };
    auto raise = [&](float top) {  // m to a larger maximum
        const float a = m == -INFINITY ? 0.f : ex2_approx(m - top);
        m = top;
        l *= a;
        acc = make_float4(acc.x * a, acc.y * a, acc.z * a, acc.w * a);
    };
    for (int i0 = warp; i0 < n_part; i0 += 4 * kWarps) {
        float2 ml[4];
        float4 o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * kWarps;
            const size_t si = (size_t)(i == 0 ? slot0 : 2 * (c0 + i)) * 8 * NT + row;
            ml[j] = i < n_part ? P.part_ml[si] : make_float2(-INFINITY, 0.f);
            o[j] = i < n_part ? reinterpret_cast<const float4 *>(P.part_o)[si * 32 + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float top = fmaxf(fmaxf(m, ml[0].x), fmaxf(ml[1].x, fmaxf(ml[2].x, ml[3].x)));
        if (top > m) raise(top);
#pragma unroll
        for (int j = 0; j < 4; ++j) add(ml[j].x == -INFINITY ? 0.f : ex2_approx(ml[j].x - m), ml[j].y, o[j]);
    }
    so[warp][lane] = acc;
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
        const float2 ml = sml[w];
        if (ml.x > m) raise(ml.x);
        add(ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m), ml.y, so[w][lane]);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const int tok = tok0 + x / P.group, hh = h * P.group + x % P.group;
    uint2 *dst = reinterpret_cast<uint2 *>(static_cast<typename Ty::T *>(P.out) + (long long)tok * P.o_ts +
                                           (long long)hh * P.o_hs) + lane;
    *dst = make_uint2(Ty::pack(acc.x * inv, acc.y * inv), Ty::pack(acc.z * inv, acc.w * inv));
    if (lane == 0 && P.lse)
        P.lse[(size_t)tok * P.hq + hh] = l == 0.f ? -INFINITY : (m - Ty::kShift + __log2f(l)) * 0.69314718055994531f;
}

template <class Ty, int NT, bool kSparse>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_kernel(const __grid_constant__ PagedAttnParams P) {
    join_row<Ty, NT, kSparse>(P);
    end_after_primary();
}

template <class Ty, int NT>
cudaError_t launch_dense(const StreamParams &SP, cudaStream_t st) {
    const PagedAttnParams &P = SP.a;
    const PagedSeqs &S = P.seqs;
    const int bytes = (int)kSmemPre + (S.n_seqs + 1) * (int)sizeof(long long) + 1024;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(paged_dense_kernel<Ty, NT>),
                               (int)kSmemPre + (kMaxSeqs + 1) * (int)sizeof(long long) + 1024, done);
    if (e != cudaSuccess) return e;
    const int rt = (S.max_q * P.group + 8 * NT - 1) / (8 * NT);
    ProfScope prof("paged_dense", st);
    paged_dense_kernel<Ty, NT><<<kStreamGrid, Shape<NT>::kThreads, bytes, st>>>(SP);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after(paged_join_kernel<Ty, NT, false>,
                        dim3(S.n_seqs * P.hkv * rt, min(8 * NT, S.max_q * P.group)), dim3(32 * kJoinWarps), 0, st, P);
}

template <class Ty, int NT>
cudaError_t launch_sparse(const StreamParams &SP, cudaStream_t st) {
    const PagedAttnParams &P = SP.a;
    const long long items = (long long)P.seqs.total * P.hkv * ((P.group + 8 * NT - 1) / (8 * NT));
    if (items > 0x7fffffffll) return cudaErrorInvalidValue;
    const unsigned ctas = P.n_slots > 0 ? P.n_slots / 2 : (unsigned)items;
    const int bytes = (int)kSmemPre + 1024;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(paged_sparse_kernel<Ty, NT>), bytes, done);
    if (e != cudaSuccess) return e;
    ProfScope prof("paged_sparse", st);
    paged_sparse_kernel<Ty, NT><<<ctas, Shape<NT>::kThreads, bytes, st>>>(SP);
    e = cudaGetLastError();
    if (e != cudaSuccess || P.n_slots == 0) return e;
    return launch_after(paged_join_kernel<Ty, NT, true>, dim3((unsigned)items, min(8 * NT, P.group)), dim3(32 * kJoinWarps), 0, st, P);
}

cudaError_t stream_maps(StreamParams &SP, const PagedAttnParams &P, bool fp16) {
    memset(&SP, 0, sizeof(SP));
    SP.a = P;
    const PagedSeqs &S = P.seqs;
    cudaError_t e = make_tmap_pages(&SP.tmap_k, P.k, fp16, S.page, P.hkv, S.num_pages, P.kc_ps, kGroup);
    if (e == cudaSuccess) e = make_tmap_pages(&SP.tmap_v, P.v, fp16, S.page, P.hkv, S.num_pages, P.vc_ps, kGroup);
    return e;
}

}  // namespace

StreamPlan paged_stream_plan(int group, int max_q) { return {max_q * group <= 8 ? 8 : 16, 2 * kStreamGrid}; }

// CTAs that share the page lists of so many items.
static long long sparse_shares(long long items, int topk, int page) {
    return std::max(1ll, std::min<long long>({kStreamGrid, items * topk, items * topk * page / (4 * kGroup)}));
}

StreamPlan paged_sparse_plan(int total, int hkv, int group, int topk, int page) {
    const int rows = group <= 8 ? 8 : 16;
    const long long items = (long long)total * hkv * ((group + rows - 1) / rows);
    // From four waves of items on, a CTA to each (their pages meet in L2 while neighbouring
    // tokens run side by side); below, equal shares of one wave, of four 16-key groups
    // at least.
    if (items >= 4 * kStreamGrid) return {rows, 0};
    return {rows, 2 * (int)sparse_shares(items, topk, page)};
}

// Shares grow with the items, the lists and the pages, up to where a call has none; a call
// of that size reserves what a smaller one of the same heads takes.
StreamPlan paged_sparse_reserve(int total, int hkv, int group, int topk) {
    const int rows = group <= 8 ? 8 : 16;
    const long long items = (long long)total * hkv * ((group + rows - 1) / rows);
    return {rows, 2 * (int)sparse_shares(items, topk, 128)};
}

cudaError_t run_paged_stream(const PagedAttnParams &P, bool fp16, int rows, cudaStream_t st) {
    if (P.seqs.n_seqs == 0 || P.seqs.total == 0) return cudaSuccess;
    StreamParams SP;
    const cudaError_t e = stream_maps(SP, P, fp16);
    if (e != cudaSuccess) return e;
    if (fp16) return rows == 8 ? launch_dense<Fp16, 1>(SP, st) : launch_dense<Fp16, 2>(SP, st);
    return rows == 8 ? launch_dense<Bf16, 1>(SP, st) : launch_dense<Bf16, 2>(SP, st);
}

cudaError_t run_paged_sparse(const PagedAttnParams &P, bool fp16, int rows, cudaStream_t st) {
    if (P.seqs.n_seqs == 0 || P.seqs.total == 0) return cudaSuccess;
    StreamParams SP;
    const cudaError_t e = stream_maps(SP, P, fp16);
    if (e != cudaSuccess) return e;
    if (fp16) return rows == 8 ? launch_sparse<Fp16, 1>(SP, st) : launch_sparse<Fp16, 2>(SP, st);
    return rows == 8 ? launch_sparse<Bf16, 1>(SP, st) : launch_sparse<Bf16, 2>(SP, st);
}

}  // namespace minf
