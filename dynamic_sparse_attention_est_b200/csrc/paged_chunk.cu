// paged_chunk.cu -- causal attention of chunks of new tokens over the paged cache
// (tcgen05 + TMEM + TMA), for more query rows than the streaming kernel takes.
//
// Rows are (token, q-head of the group) pairs, token by token: a 128-row tile
// holds 128 / G tokens of one kv-head, so every K and V tile it loads serves the
// whole group and the causal diagonal crosses few tiles.  A work unit is two such
// tiles against a range of 128-key tiles: each K and V tile is loaded once for
// 256 rows, and while the tensor cores multiply for one tile the softmax of the
// other runs.
//
// Per 128x128 tile the tensor pipe needs 1,024 clocks (S = Q K^T and O += P V),
// the 16,384 exponentials 1,024 clocks of MUFU, and shared memory about 1,000
// clocks (operands 96 KB, the TMA's writes 32 KB per tile since two tiles share
// them, at 128 B a clock).
//
// Warp roles (384 threads, one persistent CTA per SM):
//   warp 0       TMA producer: Q of a unit, then K and V tiles in turn through one
//                ring; looks the pages up, one lane per box
//   warp 1       TMEM allocator, tcgen05.mma issue
//   warps 4..7   softmax and output of row tile 0
//   warps 8..11  softmax and output of row tile 1
// TMEM columns: S0 [0,128) S1 [128,256) O0 [256,384) O1 [384,512); P overwrites the
// first half of its S.
//
// Units: the key tiles of a row-tile pair are cut into parts of one length, chosen
// by every CTA alike from the lengths on the device so that the units fill the SMs
// in whole rounds; units that run side by side share their kv-head and key range,
// which keeps K and V in L2.  Parts of a cut pair are joined by a second kernel.
#include <cstring>

#include "internal.h"
#include "paged.cuh"

namespace minf {

namespace {

constexpr int kThreads = 384;
constexpr int kGrid = 148;
constexpr int kStages = 4;
constexpr int kKeyTile = 128;
constexpr uint32_t kTileBytes = 32768;  // 128 rows x 128 16-bit values
constexpr uint32_t kSmemQ = 0;          // two row tiles
constexpr uint32_t kSmemRing = 2 * kTileBytes;
constexpr uint32_t kSmemBar = kSmemRing + kStages * kTileBytes;
constexpr uint32_t kSmemPlan = kSmemBar + 256;  // int2 [n_seqs + 1]
constexpr uint32_t kSmemMax = 232448;
static_assert(kSmemPlan + 8 * (kMaxSeqs + 1) + 1024 <= kSmemMax, "the plan of kMaxSeqs sequences fits");
// Register split after setmaxnreg: 128 x 72 + 256 x 216 = 384 x 168.
constexpr int kRegsLaunch = 168, kRegsLoad = 72, kRegsSoftmax = 216;
static_assert(128 * kRegsLoad + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "register split");

enum : int { B_Q_FULL = 0, B_Q_EMPTY = 1, B_FULL = 2, B_EMPTY = 6, B_S_FULL = 10, B_P_FULL = 12, B_O_FULL = 14,
             B_COUNT = 16 };

constexpr uint32_t idesc(uint32_t type, bool b_mn_major) {
    return (1u << 4) | type | ((b_mn_major ? 1u : 0u) << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
}

struct ChunkParams {
    CUtensorMap tmap_q;  // {128, G, total, hkv}, box {64, G, tokens per tile, 1}
    CUtensorMap tmap_k;  // {128, P, hkv, pages}, box {64, min(P, 64), 1, 1}
    CUtensorMap tmap_v;
    PagedAttnParams a;
    int tpt;         // tokens per 128-row tile
    int part_rows;   // rows per partial slot: 128 or 256
    int max_slots;
};

// ------------------------------------------------------------------ plan
__device__ __forceinline__ int seq_pairs(const SeqView &v, int tpt) { return (v.n + 2 * tpt - 1) / (2 * tpt); }
__device__ __forceinline__ int seq_ktiles(const SeqView &v) { return (v.len + kKeyTile - 1) / kKeyTile; }
__device__ __forceinline__ int seq_parts(int ktiles, int part_len) {
    return max(1, (ktiles + part_len - 1) / part_len);
}

// Chooses the part length: candidate i cuts the longest sequence into i + 1 parts.
// The estimated time of a candidate is that of its rounds of units (kGrid at a
// time) of average length, a tail of one longest unit, and two tiles' time per
// unit for its prologue and epilogue; candidates whose cut units exceed the
// partial slots are out.  Every CTA computes the same result.
__device__ int choose_part_len(const ChunkParams &P, int *len_sh) {
    const PagedSeqs &S = P.a.seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        int kt_max = 1;
        for (int s = lane; s < S.n_seqs; s += 32) {
            const SeqView v = seq_view(S, s, P.a.hdr);
            if (v.n > 0) kt_max = max(kt_max, seq_ktiles(v));
        }
        kt_max = __reduce_max_sync(0xffffffffu, kt_max);
        const int len = (kt_max + lane) / (lane + 1);
        long long units = 0, cut = 0;
        float work = 0.f;
        for (int s = 0; s < S.n_seqs; ++s) {
            const SeqView v = seq_view(S, s, P.a.hdr);
            if (v.n == 0) continue;
            const int kt = seq_ktiles(v), parts = seq_parts(kt, len);
            const long long items = (long long)P.a.hkv * seq_pairs(v, P.tpt);
            units += items * parts;
            if (parts > 1) cut += items * parts;
            work += (float)items * (float)kt;
        }
        float cost = INFINITY;
        if (cut <= P.max_slots && units > 0) {
            const float avg = work / (float)units;
            const float rounds = (float)((units + kGrid - 1) / kGrid);
            cost = rounds * (avg + 2.f) + fmaxf(0.f, (float)len - avg);
        }
        float best = cost;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, o));
        const unsigned at = __ballot_sync(0xffffffffu, cost <= best);
        if (lane == __ffs(at) - 1) *len_sh = max(1, len);
    }
    __syncthreads();
    return *len_sh;
}

struct Unit {
    int s, h, pair, part, parts;
    int ka, kb;        // key tiles
    int tok0, n_tok;   // first token (in its sequence) and tokens of the pair
    int q0, pos0, len; // sequence: first q row, position of its first new token, stored tokens
    int slot;          // partial slot, or -1
    bool two;          // the second row tile holds tokens
};

__device__ __forceinline__ Unit unit_at(const ChunkParams &P, const int2 *pre, int part_len, int u) {
    const PagedSeqs &S = P.a.seqs;
    int lo = 0, hi = S.n_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid].x <= u) lo = mid;
        else hi = mid;
    }
    // sequences without units share their start with the next one: the last of them is found
    Unit n;
    n.s = lo;
    const SeqView v = seq_view(S, lo, P.a.hdr);
    const int pairs = seq_pairs(v, P.tpt);
    n.parts = seq_parts(seq_ktiles(v), part_len);
    const int rem = u - pre[lo].x;
    n.pair = pairs - 1 - rem % pairs;  // the longest first
    n.part = (rem / pairs) % n.parts;
    n.h = rem / pairs / n.parts;
    n.tok0 = n.pair * 2 * P.tpt;
    n.n_tok = min(2 * P.tpt, v.n - n.tok0);
    n.two = n.n_tok > P.tpt;
    n.q0 = v.q0;
    n.pos0 = v.len - v.n;
    n.len = v.len;
    const int last = n.pos0 + n.tok0 + n.n_tok - 1;  // position of the pair's last token
    const int kt = last < 0 ? 0 : last / kKeyTile + 1;
    n.ka = (int)((long long)kt * n.part / n.parts);
    n.kb = (int)((long long)kt * (n.part + 1) / n.parts);
    n.slot = n.parts > 1 ? pre[lo].y + rem : -1;
    return n;
}

template <class Ty>
__global__ void __launch_bounds__(kThreads, 1) paged_chunk_kernel(const __grid_constant__ ChunkParams P) {
    using T = typename Ty::T;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t sQ = sbase + kSmemQ, sR = sbase + kSmemRing;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kSmemBar);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + B_COUNT);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + B_COUNT + 1);
    int *len_sh = reinterpret_cast<int *>(bars + B_COUNT + 2);
    int2 *warp_sum = reinterpret_cast<int2 *>(bars + B_COUNT + 3);  // [12]
    int2 *pre = reinterpret_cast<int2 *>(smem + kSmemPlan);
    auto bar = [&](int i) { return smem_u32(bars + i); };
    const PagedSeqs &S = P.a.seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(bar(B_Q_FULL), 1);
        mbar_init(bar(B_Q_EMPTY), 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(B_FULL + s), 1);
            mbar_init(bar(B_EMPTY + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(B_S_FULL + b), 1);
            mbar_init(bar(B_P_FULL + b), 128);
            mbar_init(bar(B_O_FULL + b), 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&P.tmap_q);
        tma_prefetch_desc(&P.tmap_k);
        tma_prefetch_desc(&P.tmap_v);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    // ---- plan: part length, then per sequence the units and partial slots before it
    const int part_len = choose_part_len(P, len_sh);
    {
        const int per = (S.n_seqs + kThreads - 1) / kThreads;
        const int sa = min((int)threadIdx.x * per, S.n_seqs), sb = min(sa + per, S.n_seqs);
        auto count = [&](int s) -> int2 {
            const SeqView v = seq_view(S, s, P.a.hdr);
            if (v.n == 0) return make_int2(0, 0);
            const int parts = seq_parts(seq_ktiles(v), part_len);
            const int u = P.a.hkv * seq_pairs(v, P.tpt) * parts;
            return make_int2(u, parts > 1 ? u : 0);
        };
        int2 mine = make_int2(0, 0);
        for (int s = sa; s < sb; ++s) {
            const int2 c = count(s);
            mine.x += c.x;
            mine.y += c.y;
        }
        int2 inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, inc.x, o), y = __shfl_up_sync(0xffffffffu, inc.y, o);
            if (lane >= o) {
                inc.x += x;
                inc.y += y;
            }
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        int2 at = make_int2(inc.x - mine.x, inc.y - mine.y);
        for (int w = 0; w < warp; ++w) {
            at.x += warp_sum[w].x;
            at.y += warp_sum[w].y;
        }
        for (int s = sa; s < sb; ++s) {
            pre[s] = at;
            const int2 c = count(s);
            at.x += c.x;
            at.y += c.y;
        }
        if (threadIdx.x == kThreads - 1) pre[S.n_seqs] = at;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int n_units = pre[S.n_seqs].x;
    if (blockIdx.x == 0) {  // the joining kernel's copy of the plan
        for (int s = threadIdx.x; s <= S.n_seqs; s += kThreads) P.a.part_item[1 + s] = pre[s].y;
        if (threadIdx.x == 0) P.a.part_item[0] = part_len;
    }
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{abort_flag, &P.a.hdr->status, P.a.wait_limit_ns};

    if (warp < 4) {
        setmaxnreg_dec<kRegsLoad>();
        if (warp == 0) {
            // ------------------------------------------------------ TMA producer
            const int box = min(S.page, 64), n_box = kKeyTile / box;
            const int rb = lane >> 1, half = lane & 1;  // this lane's box of a tile
            const uint32_t q_bytes = 2u * 64u * 2u * (uint32_t)(P.tpt * P.a.group);
            int fill = 0, n_q = 0;
            bool ok = true;
            auto page_for = [&](const Unit &n, int j) -> int {
                const int key = j * kKeyTile + rb * box;
                if (rb >= n_box || j >= n.kb || key >= n.len) return -1;
                return max(0, page_of(S, n.s, key >> S.page_log2, P.a.hdr));  // a bad one is flagged, its keys are page 0's
            };
            for (int u = blockIdx.x; ok && u < n_units; u += gridDim.x) {
                const Unit n = unit_at(P, pre, part_len, u);
                if (n.ka >= n.kb) continue;
                int pg = page_for(n, n.ka);
                ok = __all_sync(0xffffffffu, wait_bounded(bar(B_Q_EMPTY), (n_q & 1) ^ 1, wc, wait_site(1, B_Q_EMPTY, u)));
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(B_Q_FULL), n.two ? 2 * q_bytes : q_bytes);
                    for (int t = 0; t < (n.two ? 2 : 1); ++t)
                        for (int x = 0; x < 2; ++x)
                            tma_load_4d(sQ + t * kTileBytes + x * 16384, &P.tmap_q, bar(B_Q_FULL), x * 64, 0,
                                        n.q0 + n.tok0 + t * P.tpt, n.h);
                }
                ++n_q;
                for (int j = n.ka; ok && j < n.kb; ++j) {
                    const int pg_next = page_for(n, j + 1);
                    const int n_load = __popc(__ballot_sync(0xffffffffu, pg >= 0));
                    for (int kv = 0; kv < 2; ++kv) {
                        const int st = fill % kStages;
                        ok = __all_sync(0xffffffffu, wait_bounded(bar(B_EMPTY + st), ((fill / kStages) & 1) ^ 1, wc,
                                                                  wait_site(1, B_EMPTY + st, j)));
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(bar(B_FULL + st), (uint32_t)(n_load * box * 128));
                        __syncwarp();
                        if (pg >= 0)
                            tma_load_4d(sR + st * kTileBytes + half * 16384 + rb * box * 128,
                                        kv ? &P.tmap_v : &P.tmap_k, bar(B_FULL + st), half * 64,
                                        (rb * box) & (S.page - 1), n.h, pg);
                        __syncwarp();
                        ++fill;
                    }
                    pg = pg_next;
                }
            }
            if (*abort_flag && lane == 0) {
                // let the loads already issued land before the CTA exits
                volatile int no_abort = 0;
                const WaitCtl drain{&no_abort, nullptr, 50000000ull};
                for (int f = max(0, fill - kStages); f < fill; ++f)
                    wait_bounded(bar(B_FULL + f % kStages), (f / kStages) & 1, drain);
                if (n_q > 0) wait_bounded(bar(B_Q_FULL), (n_q - 1) & 1, drain);
            }
        } else if (warp == 1) {
            // ------------------------------------------------------ MMA issue (whole warp; one lane issues)
            constexpr uint32_t kQK = idesc(Ty::kIdescType, false), kPV = idesc(Ty::kIdescType, true);
            const uint64_t dq = sdesc_sw128(sQ, 16, 1024), dk = sdesc_sw128(sR, 16, 1024);
            const uint64_t dv = sdesc_sw128(sR, 16384, 1024);
            int used = 0, n_q = 0;           // ring stages taken (K then V per key tile), Q loads seen
            int np[2] = {0, 0};              // P tiles seen per row tile
            bool ok = true;
            auto wait_full = [&](int f, int site) -> bool {
                return __all_sync(0xffffffffu, wait_bounded(bar(B_FULL + f % kStages), (f / kStages) & 1, wc, site));
            };
            auto issue_s = [&](int t, int f) {
                umma_ss_tile_warp(tmem + t * 128, dq + (uint64_t)((t * kTileBytes) >> 4),
                                  dk + (uint64_t)(((f % kStages) * kTileBytes) >> 4), kQK, 0u);
                umma_commit_warp(bar(B_S_FULL + t));
            };
            for (int u = blockIdx.x; ok && u < n_units; u += gridDim.x) {
                const Unit n = unit_at(P, pre, part_len, u);
                const int T = n.kb - n.ka, nt = n.two ? 2 : 1;
                if (T <= 0) continue;
                ok = __all_sync(0xffffffffu, wait_bounded(bar(B_Q_FULL), n_q & 1, wc, wait_site(3, B_Q_FULL, u)));
                if (!ok || !(ok = wait_full(used, wait_site(3, B_FULL, 0)))) break;
                ++n_q;
                tc_fence_after();
                for (int t = 0; t < nt; ++t) issue_s(t, used);
                umma_commit_warp(bar(B_EMPTY + used % kStages));
                if (T == 1) umma_commit_warp(bar(B_Q_EMPTY));
                for (int j = 0; ok && j < T; ++j) {
                    const int fv = used + 1, fk = used + 2;  // this tile's V, the next tile's K
                    for (int t = 0; ok && t < nt; ++t) {
                        ok = __all_sync(0xffffffffu, wait_bounded(bar(B_P_FULL + t), np[t] & 1, wc,
                                                                  wait_site(3, B_P_FULL + t, j)));
                        if (!ok) break;
                        ++np[t];
                        if (t == 0) {
                            if (!(ok = wait_full(fv, wait_site(3, B_FULL + 1, j)))) break;
                            const int valid = n.len - (n.ka + j) * kKeyTile;
                            if (valid < kKeyTile) {
                                // rows behind the stored tokens: whatever they hold, 0 * it must be 0
                                const uint32_t st = sR + (fv % kStages) * kTileBytes;
                                for (int i = valid * 8 + lane; i < kKeyTile * 8; i += 32)
#pragma unroll
                                    for (int x = 0; x < 2; ++x)
                                        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(st + x * 16384 + i * 16),
                                                     "r"(0u)
                                                     : "memory");
                                fence_proxy_async_smem();
                                __syncwarp();
                            }
                        }
                        tc_fence_after();
                        umma_ts_tile_warp(tmem + 256 + t * 128, tmem + t * 128,
                                          dv + (uint64_t)(((fv % kStages) * kTileBytes) >> 4), kPV, j > 0 ? 1u : 0u);
                        if (t == nt - 1) umma_commit_warp(bar(B_EMPTY + fv % kStages));
                        if (j + 1 < T) {
                            if (t == 0 && !(ok = wait_full(fk, wait_site(3, B_FULL + 2, j)))) break;
                            tc_fence_after();
                            issue_s(t, fk);
                            if (t == nt - 1) {
                                umma_commit_warp(bar(B_EMPTY + fk % kStages));
                                if (j + 2 == T) umma_commit_warp(bar(B_Q_EMPTY));  // the unit's last use of Q
                            }
                        } else {
                            umma_commit_warp(bar(B_O_FULL + t));
                        }
                    }
                    used += 2;
                }
            }
        }
    } else {
        // ---------------------------------------------------------- softmax warpgroups
        setmaxnreg_inc<kRegsSoftmax>();
        const int t = (warp - 4) >> 2;            // row tile
        const int r = (threadIdx.x - 128) & 127;  // row = TMEM lane
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + t * 128;
        const uint32_t tO = tmem + lane_off + 256 + t * 128;
        const float sl2 = P.a.scale_log2;
        const int G = P.a.group;
        int ns = 0, no = 0;  // S tiles and outputs seen
        bool ok = true;
        for (int u = blockIdx.x; ok && u < n_units; u += gridDim.x) {
            const Unit n = unit_at(P, pre, part_len, u);
            if (t == 1 && !n.two) continue;
            const int tok = n.tok0 + t * P.tpt + r / G;  // in the sequence
            const int n_here = min(P.tpt, n.n_tok - t * P.tpt);
            const bool live = r < n_here * G;
            const int pos = n.pos0 + n.tok0 + t * P.tpt + min(r / G, n_here - 1);
            const int pos_min = n.pos0 + n.tok0 + t * P.tpt;
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = n.ka; j < n.kb; ++j) {
                const bool got = wait_bounded(bar(B_S_FULL + t), ns & 1, wc, wait_site(4 + t, B_S_FULL + t, j));
                if (__any_sync(0xffffffffu, !got)) {  // tcgen05.ld below is warp-wide
                    ok = false;
                    break;
                }
                ++ns;
                tc_fence_after();
                uint32_t sr[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, sr[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld_wait(sr[c]);
                if (pos_min + 1 < (j + 1) * kKeyTile) {  // the diagonal or the end crosses this tile
                    const int vis = pos + 1 - j * kKeyTile;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c * 32 + e >= vis) sr[c][e] = 0xff800000u;  // -inf
                    }
                }
                float mc[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mc[c] = fmaxf(__uint_as_float(sr[c][0]), __uint_as_float(sr[c][1]));
#pragma unroll
                    for (int e = 2; e < 32; e += 2)
                        mc[c] = fmax3(mc[c], __uint_as_float(sr[c][e]), __uint_as_float(sr[c][e + 1]));
                }
                const float m_new = fmaxf(m_run, fmax3(mc[0], mc[1], fmaxf(mc[2], mc[3])) * sl2);
                const bool want = m_new > m_run + Ty::kLag;  // includes m_run = -inf with a finite m_new
                const float alpha = want ? ex2_approx(m_run - m_new) : 1.f;
                // the P V of the tiles before is complete (S of this tile was issued after it)
                if (j > n.ka && __any_sync(0xffffffffu, want && m_run != -INFINITY)) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + c * 32, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(tO + c * 32, o);
                    }
                }
                if (want) {
                    l_run *= alpha;
                    m_run = m_new;
                }
                const float m_use = m_run == -INFINITY ? 0.f : m_run - Ty::kShift;
                const uint64_t sl2x2 = f32x2_splat(sl2), negm = f32x2_splat(-m_use);
                uint64_t acc0 = 0, acc1 = 0;
                uint32_t pp[2][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const uint64_t x = f32x2_fma(
                            f32x2_pack(__uint_as_float(sr[c][2 * e]), __uint_as_float(sr[c][2 * e + 1])), sl2x2, negm);
                        float p0, p1;
                        f32x2_unpack(x, p0, p1);
                        p0 = ex2_approx(p0);
                        p1 = ex2_approx(p1);
                        if (e & 1) acc1 = f32x2_add(acc1, f32x2_pack(p0, p1));
                        else acc0 = f32x2_add(acc0, f32x2_pack(p0, p1));
                        // P is rounded to the cache's type for the product (the size of the
                        // output's own rounding); the sum keeps fp32
                        pp[c >> 1][(c & 1) * 16 + e] = Ty::pack(p0, p1);
                    }
                    if (c == 1) tmem_st32(tS, pp[0]);
                }
                float a0, a1, b0, b1;
                f32x2_unpack(acc0, a0, a1);
                f32x2_unpack(acc1, b0, b1);
                l_run += (a0 + a1) + (b0 + b1);
                tmem_st32(tS + 32, pp[1]);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar(B_P_FULL + t));
            }
            if (!ok) break;
            // -------------------------------------------------------- output
            const bool any = n.kb > n.ka;
            if (any) {
                const bool got = wait_bounded(bar(B_O_FULL + t), no & 1, wc, wait_site(4 + t, B_O_FULL + t, u));
                if (__any_sync(0xffffffffu, !got)) break;
                ++no;
                tc_fence_after();
            }
            const int hh = n.h * G + r % G;
            const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);  // a NaN sum stays one
            T *dst = static_cast<T *>(P.a.out) + (long long)(n.q0 + tok) * P.a.o_ts + (long long)hh * P.a.o_hs;
            const size_t prow = (size_t)max(n.slot, 0) * P.part_rows + t * 128 + r;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                if (any) {  // uniform over the CTA
                    tmem_ld32(tO + c * 32, o);
                    tmem_ld_wait(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                if (!live) continue;
                if (n.slot >= 0) {
                    uint4 *d4 = reinterpret_cast<uint4 *>(P.a.part_o + prow * kD + c * 32);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d4[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                } else {
                    uint4 *d4 = reinterpret_cast<uint4 *>(dst + c * 32);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = Ty::pack(__uint_as_float(o[8 * e + 2 * i]) * inv,
                                            __uint_as_float(o[8 * e + 2 * i + 1]) * inv);
                        d4[e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            if (live) {
                if (n.slot >= 0)
                    P.a.part_ml[prow] = make_float2(m_run, l_run);
                else if (P.a.lse)
                    P.a.lse[(size_t)(n.q0 + tok) * P.a.hq + hh] =
                        l_run == 0.f ? -INFINITY : (m_run - Ty::kShift + __log2f(l_run)) * 0.69314718055994531f;
            }
            tc_fence_before();  // the loads of O come before the next unit's P hand-over
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join
// One warp per row of a cut pair: its parts in order.
template <class Ty>
__global__ void __launch_bounds__(256) paged_chunk_join_kernel(const __grid_constant__ PagedAttnParams P, int tpt,
                                                               int part_rows) {
    const PagedSeqs &S = P.seqs;
    const int lane = threadIdx.x & 31;
    const int part_len = P.part_item[0];
    const int *pre = P.part_item + 1;  // partial slots before each sequence
    const int n_slots = pre[S.n_seqs];
    const int step = gridDim.x * (blockDim.x >> 5);
    const long long rows = (long long)n_slots * part_rows;
    for (long long w = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < rows; w += step) {
        const int slot = (int)(w / part_rows), r = (int)(w % part_rows);
        int lo = 0, hi = S.n_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= slot) lo = mid;
            else hi = mid;
        }
        const SeqView v = seq_view(S, lo, P.hdr);
        const int pairs = seq_pairs(v, tpt), parts = seq_parts(seq_ktiles(v), part_len);
        const int rem = slot - pre[lo];
        if ((rem / pairs) % parts != 0) continue;  // the first part's warp joins them all
        const int pair = pairs - 1 - rem % pairs, h = rem / pairs / parts;
        const int t = r >> 7, x = (r & 127) / P.group;
        const int tok = pair * 2 * tpt + t * tpt + x;
        if (x >= tpt || tok >= v.n) continue;
        float m = -INFINITY;
        for (int i = lane; i < parts; i += 32)
            m = fmaxf(m, P.part_ml[(size_t)(slot + i * pairs) * part_rows + r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
            const size_t row = (size_t)(slot + i * pairs) * part_rows + r;
            const float2 ml = P.part_ml[row];
            const float a = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (ml.y != 0.f) o = reinterpret_cast<const float4 *>(P.part_o)[row * 32 + lane];
            l = fmaf(ml.y, a, l);
            acc.x = fmaf(o.x, a, acc.x);
            acc.y = fmaf(o.y, a, acc.y);
            acc.z = fmaf(o.z, a, acc.z);
            acc.w = fmaf(o.w, a, acc.w);
        }
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        const int hh = h * P.group + (r & 127) % P.group;
        uint2 *dst = reinterpret_cast<uint2 *>(static_cast<typename Ty::T *>(P.out) +
                                               (long long)(v.q0 + tok) * P.o_ts + (long long)hh * P.o_hs) + lane;
        *dst = make_uint2(Ty::pack(acc.x * inv, acc.y * inv), Ty::pack(acc.z * inv, acc.w * inv));
        if (lane == 0 && P.lse)
            P.lse[(size_t)(v.q0 + tok) * P.hq + hh] =
                l == 0.f ? -INFINITY : (m - Ty::kShift + __log2f(l)) * 0.69314718055994531f;
    }
}

template <class Ty>
cudaError_t launch_chunk(const ChunkParams &C, cudaStream_t st) {
    const PagedSeqs &S = C.a.seqs;
    cudaError_t e = cudaFuncSetAttribute(paged_chunk_kernel<Ty>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemMax);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc waits for registers the launch reserved: refuse to launch a
    // build whose register count at entry would make the split wait forever
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, paged_chunk_kernel<Ty>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
    ProfScope prof("paged_chunk", st);
    const int bytes = (int)kSmemPlan + 8 * (S.n_seqs + 1) + 1024;
    paged_chunk_kernel<Ty><<<kGrid, kThreads, bytes, st>>>(C);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    paged_chunk_join_kernel<Ty><<<2 * kGrid, 256, 0, st>>>(C.a, C.tpt, C.part_rows);
    return cudaGetLastError();
}

}  // namespace

ChunkPlan paged_chunk_plan(int n_seqs, int group, int max_q) {
    ChunkPlan p{};
    p.part_rows = max_q <= 128 / group ? 128 : 256;
    p.n_slots = 8 * kGrid;
    p.n_items = 2 + n_seqs;
    return p;
}

cudaError_t run_paged_chunk(const PagedAttnParams &P, bool fp16, int part_rows, cudaStream_t st) {
    const PagedSeqs &S = P.seqs;
    if (S.n_seqs == 0 || S.total == 0) return cudaSuccess;
    ChunkParams C;
    memset(&C, 0, sizeof(C));
    C.a = P;
    C.tpt = 128 / P.group;
    C.part_rows = part_rows;
    C.max_slots = P.n_slots;
    const cuuint64_t G = P.group;
    // the stride of a dimension of one element is never used
    const cuuint64_t hs = P.hq > 1 ? P.q_hs : kD, ts = S.total > 1 ? P.q_ts : kD;
    cudaError_t e = make_tmap_4d(&C.tmap_q, P.q, fp16, {kD, G, (cuuint64_t)S.total, (cuuint64_t)P.hkv},
                              {hs * 2, ts * 2, G * hs * 2},
                              {64, (cuuint32_t)P.group, (cuuint32_t)C.tpt, 1});
    const int box = S.page < 64 ? S.page : 64;
    if (e == cudaSuccess) e = make_tmap_pages(&C.tmap_k, P.k, fp16, S.page, P.hkv, S.num_pages, P.kc_ps, box);
    if (e == cudaSuccess) e = make_tmap_pages(&C.tmap_v, P.v, fp16, S.page, P.hkv, S.num_pages, P.vc_ps, box);
    if (e != cudaSuccess) return e;
    return fp16 ? launch_chunk<Fp16>(C, st) : launch_chunk<Bf16>(C, st);
}

}  // namespace minf
