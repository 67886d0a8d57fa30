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
// A row tile's S has two 64-key halves that are handed over separately: while the
// softmax works on one half, the tensor cores multiply P of the other half by V
// and write the S of 64 keys further on over it, so neither side waits for the
// other's latency.  With whole 128-key tiles S -> softmax -> P V -> S is one chain
// per row tile: 2,048 tokens over 55,296 + 2,048 kept the SMs busy for 1,575 us, with
// halves for 1,524 us (3,750 and 3,590 clocks for 128 keys against 256 rows; both
// with one issuing warp a row tile).
//
// Warp roles (384 threads, one persistent CTA per SM):
//   warp 0       TMA producer: Q of a unit, then K and V tiles in turn through one
//                ring; looks the pages up, one lane per box
//   warps 1, 2   tcgen05.mma issue of row tile 0 and 1 (warp 1 allocates TMEM)
//   warps 4..7   softmax and output of row tile 0
//   warps 8..11  softmax and output of row tile 1
// TMEM columns: S0 [0,128) S1 [128,256) O0 [256,384) O1 [384,512); the P of a 64-key
// half overwrites the first 32 columns of its S.
//
// Units: the key tiles of a row-tile pair are cut into parts of one length, chosen
// by every CTA alike from the lengths on the device so that the units fill the SMs
// in whole rounds; units that run side by side share their kv-head and key range,
// which keeps K and V in L2.  Parts of a cut pair are joined by a second kernel.
//
// O grows in TMEM by the tensor cores' fp32 additions, which truncate: over one page
// repeated, uncut, it comes out low by 1.1e-4 of the value after 128K keys and by
// 9.0e-4 after 1M, in either type.
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
constexpr uint32_t kSmemPlan = kSmemBar + 320;  // int2 [n_seqs + 1]
constexpr uint32_t kSmemMax = 232448;
static_assert(kSmemPlan + 8 * (kMaxSeqs + 1) + 1024 <= kSmemMax, "the plan of kMaxSeqs sequences fits");
// Register split after setmaxnreg: 128 x 72 + 256 x 216 = 384 x 168.
constexpr int kRegsLaunch = 168, kRegsLoad = 72, kRegsSoftmax = 216;
static_assert(128 * kRegsLoad + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "register split");

// S_FULL and P_FULL: one per row tile and 64-key half (2 t + h); O_PREV and O_FULL,
// once a unit: O holds all steps but the last, and all of them
enum : int { B_Q_FULL = 0, B_Q_EMPTY = 1, B_FULL = 2, B_EMPTY = 6, B_S_FULL = 10, B_P_FULL = 14, B_O_PREV = 18,
             B_O_FULL = 20, B_COUNT = 22 };
constexpr uint32_t kSmemWarpSum = kSmemBar + 208;  // int2 [12]

constexpr uint32_t idesc(uint32_t type, int n, bool b_mn_major) {
    return (1u << 4) | type | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// O += P V for 64 keys: A = P from TMEM (8 columns per 16 keys), B = 64 rows of V
// (2 KB per 16 keys).  The whole warp calls it, one lane issues; the first step
// accumulates into D iff acc_first.
__device__ __forceinline__ void umma_ts_half_warp(uint32_t d, uint32_t a_tmem, uint64_t b0, uint32_t idesc,
                                                  uint32_t acc_first) {
    asm volatile(
        "{\n\t.reg .pred p, t, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 t, %3, %3;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%5], %6, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%7], %8, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%9], %10, %3, t;\n\t}\n" ::"r"(d),
        "r"(a_tmem), "l"(b0), "r"(idesc), "r"(acc_first), "r"(a_tmem + 8), "l"(b0 + 128), "r"(a_tmem + 16),
        "l"(b0 + 256), "r"(a_tmem + 24), "l"(b0 + 384)
        : "memory");
}

// The MMA warps' wait: P is a few hundred clocks away most of the time, and two
// spinning warps leave the SM's issue slots alone (2 % of the kernel's time; spinning
// softmax warps, eight of them, cost 16 %).  Bounded like the others in the end.
__device__ __forceinline__ bool wait_spin(uint32_t bar, uint32_t parity, const WaitCtl &w, int site) {
#pragma unroll 1
    for (int i = 0; i < 100000; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return wait_bounded(bar, parity, w, site);
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
// A plan: the part length, and whether whole rounds of pairs stay uncut (part_len < 0
// in the encoded form), which a call with one sequence to work on may choose.
struct PartPlan {
    int len;
    bool tail;
};
__device__ __forceinline__ PartPlan part_plan(int code) { return {abs(code), code < 0}; }
// How a sequence's pairs (over its kv-heads) are cut: the first `whole` are units of
// their own, the others are cut into `parts` each.
struct SeqCut {
    int items, whole, parts;
    __device__ int units() const { return whole + (items - whole) * parts; }
    __device__ int slots() const { return parts > 1 ? (items - whole) * parts : 0; }
};
__device__ __forceinline__ SeqCut seq_cut(const SeqView &v, int hkv, int tpt, const PartPlan &p) {
    SeqCut c;
    c.items = hkv * seq_pairs(v, tpt);
    c.parts = seq_parts(seq_ktiles(v), p.len);
    c.whole = c.parts > 1 && p.tail ? c.items / kGrid * kGrid : 0;
    return c;
}

// Chooses the part length: candidate i cuts the longest sequence into i + 1 parts.
// The estimated time of a candidate is that of its rounds of units (kGrid at a
// time) of average length, a tail of one longest unit, and per unit two tiles'
// time for its prologue and epilogue, four more for the traffic of its partial
// result (256 KB written and read); candidates whose cut units exceed the
// partial slots are out.  If a single sequence has new tokens (a chunk of a long
// prompt), its whole rounds of pairs may stay uncut and the rest alone be cut: 256
// pairs of 448 tiles take 1,637 us cut into 4 each, 1,578 us with the last 108 cut.  Every
// CTA computes the same result.  Starts that contradict each other can name the same rows
// over and over; if they make more pairs than `total` rows can, none is worked on.
constexpr int kNoPlan = 1 << 30;  // as a part length (no sequence is cut): no units
struct PlanSum {
    long long units, cut;
    float work;
    int kt, seqs;
};
__device__ int choose_part_len(const ChunkParams &P, PlanSum (*sum)[32], int *len_sh) {
    const PagedSeqs &S = P.a.seqs;
    constexpr int kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int kt_max = 1, seqs = 0;
    for (int s = threadIdx.x; s < S.n_seqs; s += kThreads) {
        const SeqView v = seq_view(S, s, P.a.hdr);
        if (v.n > 0) {
            kt_max = max(kt_max, seq_ktiles(v));
            ++seqs;
        }
    }
    kt_max = __reduce_max_sync(0xffffffffu, kt_max);
    seqs = __reduce_add_sync(0xffffffffu, seqs);
    if (lane == 0) {
        sum[warp][0].kt = kt_max;
        sum[warp][0].seqs = seqs;
    }
    __syncthreads();
    seqs = 0;
    for (int w = 0; w < kWarps; ++w) {
        kt_max = max(kt_max, sum[w][0].kt);
        seqs += sum[w][0].seqs;
    }
    __syncthreads();
    // lane = candidate, each warp its share of the sequences
    const int len = (kt_max + lane) / (lane + 1);
    PlanSum mine{0, 0, 0.f, 0, 0};
    for (int s = warp; s < S.n_seqs; s += kWarps) {
        const SeqView v = seq_view(S, s, P.a.hdr);
        if (v.n == 0) continue;
        const SeqCut c = seq_cut(v, P.a.hkv, P.tpt, {len, false});
        mine.units += c.units();
        mine.cut += c.slots();
        mine.work += (float)c.items * (float)seq_ktiles(v);
    }
    sum[warp][lane] = mine;
    __syncthreads();
    if (warp == 0) {
        for (int w = 1; w < kWarps; ++w) {
            mine.units += sum[w][lane].units;
            mine.cut += sum[w][lane].cut;
            mine.work += sum[w][lane].work;
        }
        constexpr float kOwn = 2.f, kCut = 6.f;  // tiles' time that a unit, a cut unit costs besides its tiles
        float cost = INFINITY;
        int code = len;
        if (mine.cut <= P.max_slots && mine.units > 0) {
            const float avg = mine.work / (float)mine.units;
            const float rounds = (float)((mine.units + kGrid - 1) / kGrid);
            cost = rounds * (avg + (mine.cut > 0 ? kCut : kOwn)) + fmaxf(0.f, (float)len - avg);
        }
        if (seqs == 1 && lane > 0 && mine.units > 0) {
            const int parts = seq_parts(kt_max, len);
            const long long items = mine.units / parts, rest = items % kGrid;
            if (rest > 0 && rest * parts <= P.max_slots) {
                const float c = (float)(items / kGrid) * ((float)kt_max + kOwn) +
                                (float)((rest * parts + kGrid - 1) / kGrid) * ((float)kt_max / (float)parts + kCut);
                if (c < cost) {
                    cost = c;
                    code = -len;
                }
            }
        }
        float best = cost;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, o));
        const unsigned at = __ballot_sync(0xffffffffu, cost <= best);
        if (lane == __ffs(at) - 1) *len_sh = code;
        __syncwarp();
        // lane 0 cuts nothing, its units are the pairs
        if (lane == 0 && mine.units > P.a.hkv * (S.total / (2ll * P.tpt) + S.n_seqs)) {
            flag_invalid(P.a.hdr, BAD_SEQ);
            *len_sh = kNoPlan;
        }
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

__device__ __forceinline__ Unit unit_at(const ChunkParams &P, const int2 *pre, const PartPlan &plan, int u) {
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
    const int pairs = seq_pairs(v, P.tpt), rem = u - pre[lo].x;
    const SeqCut c = seq_cut(v, P.a.hkv, P.tpt, plan);
    int item = rem;
    n.part = 0;
    n.parts = 1;
    n.slot = -1;
    if (rem >= c.whole && c.parts > 1) {
        const int cut = c.items - c.whole;
        n.parts = c.parts;
        n.part = (rem - c.whole) / cut;  // a part of every pair before the next
        item = c.whole + (rem - c.whole) % cut;
        n.slot = pre[lo].y + rem - c.whole;
    }
    n.h = item / pairs;
    n.pair = pairs - 1 - item % pairs;  // the longest first
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
    int2 *warp_sum = reinterpret_cast<int2 *>(smem + kSmemWarpSum);
    int2 *pre = reinterpret_cast<int2 *>(smem + kSmemPlan);
    auto bar = [&](int i) { return smem_u32(bars + i); };
    const PagedSeqs &S = P.a.seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(bar(B_Q_FULL), 1);
        mbar_init(bar(B_Q_EMPTY), 2);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(B_FULL + s), 1);
            mbar_init(bar(B_EMPTY + s), 2);
        }
        for (int b = 0; b < 4; ++b) {
            mbar_init(bar(B_S_FULL + b), 1);
            mbar_init(bar(B_P_FULL + b), 128);
            mbar_init(bar(B_O_PREV + b), 1);  // B_O_FULL follows it
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
    const int code =
        choose_part_len(P, reinterpret_cast<PlanSum(*)[32]>(smem + kSmemRing), len_sh);  // the ring is not in use yet
    const PartPlan plan = part_plan(code);
    {
        const int per = (S.n_seqs + kThreads - 1) / kThreads;
        const int sa = min((int)threadIdx.x * per, S.n_seqs), sb = min(sa + per, S.n_seqs);
        auto count = [&](int s) -> int2 {
            const SeqView v = seq_view(S, s, P.a.hdr);
            if (v.n == 0) return make_int2(0, 0);
            const SeqCut c = seq_cut(v, P.a.hkv, P.tpt, plan);
            return make_int2(c.units(), c.slots());
        };
        int2 mine = make_int2(0, 0);
        for (int s = sa; s < sb; ++s) {  // all of them fit 31 bits, or no unit is worked on
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
    fence_proxy_async_smem();  // the plan's sums lay where the first loads go
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int n_units = code == kNoPlan ? 0 : pre[S.n_seqs].x;
    if (blockIdx.x == 0 && warp == 3) {  // the joining kernel's copy: (slots, pairs) cut before each sequence
        int2 *dst = reinterpret_cast<int2 *>(P.a.plan + 1);
        int cut = 0;
        for (int s0 = 0; s0 <= S.n_seqs; s0 += 32) {
            const int s = s0 + lane;
            int mine = 0;
            if (s < S.n_seqs && pre[s + 1].y > pre[s].y) {
                const SeqView v = seq_view(S, s, P.a.hdr);
                const SeqCut c = seq_cut(v, P.a.hkv, P.tpt, plan);
                mine = c.items - c.whole;
            }
            int inc = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (s <= S.n_seqs) dst[s] = make_int2(pre[s].y, cut + inc - mine);
            cut += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) P.a.plan[0] = code;
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
                const Unit n = unit_at(P, pre, plan, u);
                if (n.ka >= n.kb) continue;
                int pg = page_for(n, n.ka);
                ok = __all_sync(0xffffffffu, wait_bounded_sleep(bar(B_Q_EMPTY), (n_q & 1) ^ 1, wc, wait_site(1, B_Q_EMPTY, u)));
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
                        ok = __all_sync(0xffffffffu, wait_bounded_sleep(bar(B_EMPTY + st), ((fill / kStages) & 1) ^ 1, wc,
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
                    wait_bounded_sleep(bar(B_FULL + f % kStages), (f / kStages) & 1, drain);
                if (n_q > 0) wait_bounded_sleep(bar(B_Q_FULL), (n_q - 1) & 1, drain);
            }
        } else if (warp < 3) {
            // ------------------------------------------------------ MMA issue (whole warp; one lane issues)
            // One warp per row tile: an instruction takes its issuer about as long as the
            // tensor pipe, so a single warp would be the bound.
            // Step i is 64 keys (half h = i & 1 of key tile i / 2).  S_t(i + 2) goes out
            // after P_t(i) V(i), which the tensor pipe finishes first, so P is consumed
            // before S overwrites it; the barrier of S_t(i + 2) also says that O holds the
            // steps up to i.
            constexpr uint32_t kQK = idesc(Ty::kIdescType, 64, false), kPV = idesc(Ty::kIdescType, 128, true);
            const uint64_t dq = sdesc_sw128(sQ, 16, 1024), dk = sdesc_sw128(sR, 16, 1024);
            const uint64_t dv = sdesc_sw128(sR, 16384, 1024);
            const int t = warp - 1;  // row tile
            int used = 0, n_q = 0;   // ring stages taken (K then V per key tile), Q loads seen
            uint32_t pp = 0;         // parity of the next P of each half
            bool ok = true;
            auto wait_full = [&](int f, int site) -> bool {
                return __all_sync(0xffffffffu, wait_spin(bar(B_FULL + f % kStages), (f / kStages) & 1, wc, site));
            };
            auto issue_s = [&](int h, int f) {
                umma_ss_tile_warp(tmem + t * 128 + h * 64, dq + (uint64_t)((t * kTileBytes) >> 4),
                                  dk + (uint64_t)(((f % kStages) * kTileBytes + h * 8192) >> 4), kQK, 0u);
            };
            for (int u = blockIdx.x; ok && u < n_units; u += gridDim.x) {
                const Unit n = unit_at(P, pre, plan, u);
                const int T = n.kb - n.ka;
                if (T <= 0) continue;
                if (t == 1 && !n.two) {
                    // Nothing to multiply, but every stage is taken and given back: a warp that
                    // ran ahead of the ring would take an older phase's parity for its own.
                    ok = __all_sync(0xffffffffu, wait_spin(bar(B_Q_FULL), n_q & 1, wc, wait_site(3, B_Q_FULL, u)));
                    if (!ok) break;
                    ++n_q;
                    if (lane == 0) mbar_arrive(bar(B_Q_EMPTY));
                    for (int x = 0; ok && x < 2 * T; ++x, ++used) {
                        ok = wait_full(used, wait_site(3, B_FULL + 3, x));
                        if (ok && lane == 0) mbar_arrive(bar(B_EMPTY + used % kStages));
                    }
                    continue;
                }
                ok = __all_sync(0xffffffffu, wait_spin(bar(B_Q_FULL), n_q & 1, wc, wait_site(3, B_Q_FULL, u)));
                if (!ok || !(ok = wait_full(used, wait_site(3, B_FULL, 0)))) break;
                ++n_q;
                tc_fence_after();
                for (int h = 0; h < 2; ++h) {
                    issue_s(h, used);
                    umma_commit_warp(bar(B_S_FULL + 2 * t + h));
                }
                umma_commit_warp(bar(B_EMPTY + used % kStages));
                if (T == 1) umma_commit_warp(bar(B_Q_EMPTY));
                for (int j = 0; ok && j < T; ++j) {
                    const int fv = used + 1, fk = used + 2;  // this tile's V, the next tile's K
                    const bool more = j + 1 < T;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int b = 2 * t + h;
                        ok = __all_sync(0xffffffffu, wait_spin(bar(B_P_FULL + b), (pp >> h) & 1, wc,
                                                                  wait_site(3, B_P_FULL + b, j)));
                        if (!ok) break;
                        pp ^= 1u << h;
                        if (h == 0) {
                            if (!(ok = wait_full(fv, wait_site(3, B_FULL + 1, j)))) break;
                            const int valid = n.len - (n.ka + j) * kKeyTile;
                            if (valid < kKeyTile) {
                                // rows behind the stored tokens: whatever they hold, 0 * it must be 0
                                // (both warps write the same zeros)
                                const uint32_t st = sR + (fv % kStages) * kTileBytes;
                                for (int i = valid * 8 + lane; i < kKeyTile * 8; i += 32)
#pragma unroll
                                    for (int y = 0; y < 2; ++y)
                                        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(st + y * 16384 + i * 16),
                                                     "r"(0u)
                                                     : "memory");
                                fence_proxy_async_smem();
                                __syncwarp();
                            }
                        }
                        tc_fence_after();
                        umma_ts_half_warp(tmem + 256 + t * 128, tmem + t * 128 + h * 64,
                                          dv + (uint64_t)(((fv % kStages) * kTileBytes + h * 8192) >> 4), kPV,
                                          j > 0 || h > 0 ? 1u : 0u);
                        if (more) {
                            if (h == 0) {
                                if (!(ok = wait_full(fk, wait_site(3, B_FULL + 2, j)))) break;
                                tc_fence_after();
                            }
                            issue_s(h, fk);
                        }
                        umma_commit_warp(bar(more ? B_S_FULL + b : (h == 0 ? B_O_PREV : B_O_FULL) + t));
                    }
                    if (!ok) break;
                    umma_commit_warp(bar(B_EMPTY + fv % kStages));  // free when both row tiles are done
                    if (more) {
                        umma_commit_warp(bar(B_EMPTY + fk % kStages));
                        if (j + 2 == T) umma_commit_warp(bar(B_Q_EMPTY));  // the unit's last use of Q
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
        uint32_t sp = 0, op = 0;  // parity of the next S of each half, and of the unit's O
        bool ok = true;
        for (int u = blockIdx.x; ok && u < n_units; u += gridDim.x) {
            const Unit n = unit_at(P, pre, plan, u);
            if (t == 1 && !n.two) continue;
            const int tok = n.tok0 + t * P.tpt + r / G;  // in the sequence
            const int n_here = min(P.tpt, n.n_tok - t * P.tpt);
            const bool live = r < n_here * G;
            const int pos = n.pos0 + n.tok0 + t * P.tpt + min(r / G, n_here - 1);
            const int pos_min = n.pos0 + n.tok0 + t * P.tpt;
            float m_run = -INFINITY, l_run = 0.f;
            const int i0 = 2 * n.ka, i1 = 2 * n.kb;
            for (int i = i0; i < i1; ++i) {
                const int h = i & 1;
                const uint32_t tSh = tS + h * 64;
                const bool got = wait_bounded_sleep(bar(B_S_FULL + 2 * t + h), (sp >> h) & 1, wc,
                                              wait_site(4 + t, B_S_FULL + 2 * t + h, i));
                if (__any_sync(0xffffffffu, !got)) {  // tcgen05.ld below is warp-wide
                    ok = false;
                    break;
                }
                sp ^= 1u << h;
                tc_fence_after();
                uint32_t sr[2][32];
#pragma unroll
                for (int c = 0; c < 2; ++c) tmem_ld32(tSh + c * 32, sr[c]);
#pragma unroll
                for (int c = 0; c < 2; ++c) tmem_ld_wait(sr[c]);
                if (pos_min + 1 < (i + 1) * 64) {  // the diagonal or the end crosses these keys
                    const int vis = pos + 1 - i * 64;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c * 32 + e >= vis) sr[c][e] = 0xff800000u;  // -inf
                    }
                }
                float mc[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t *x = &sr[c >> 1][(c & 1) * 16];
                    mc[c] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
                    for (int e = 2; e < 16; e += 2)
                        mc[c] = fmax3(mc[c], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                }
                const float m_new = fmaxf(m_run, fmax3(mc[0], mc[1], fmaxf(mc[2], mc[3])) * sl2);
                const bool want = m_new > m_run + Ty::kLag;  // includes m_run = -inf with a finite m_new
                const float alpha = want ? ex2_approx(m_run - m_new) : 1.f;
                if (i > i0 && __any_sync(0xffffffffu, want && m_run != -INFINITY)) {
                    // O must hold the steps before this one: the next step's S was issued after them
                    const int next = i + 1 < i1 ? B_S_FULL + 2 * t + (h ^ 1) : B_O_PREV + t;
                    const bool done = wait_bounded_sleep(bar(next), i + 1 < i1 ? (sp >> (h ^ 1)) & 1 : op, wc,
                                                         wait_site(6, next, i));
                    if (__any_sync(0xffffffffu, !done)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
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
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
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
                        pk[c * 16 + e] = Ty::pack(p0, p1);
                    }
                }
                tmem_st32(tSh, pk);
                float a0, a1, b0, b1;
                f32x2_unpack(acc0, a0, a1);
                f32x2_unpack(acc1, b0, b1);
                l_run += (a0 + a1) + (b0 + b1);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar(B_P_FULL + 2 * t + h));
            }
            if (!ok) break;
            // -------------------------------------------------------- output
            const bool any = n.kb > n.ka;
            if (any) {
                const bool got = wait_bounded_sleep(bar(B_O_FULL + t), op, wc, wait_site(4 + t, B_O_FULL + t, u));
                if (__any_sync(0xffffffffu, !got)) break;
                op ^= 1u;
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
    launch_dependents();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join
// One CTA per 32 rows of a cut pair at a time, one warp per row: its parts in order.
constexpr int kJoinRows = 32;
template <class Ty>
__global__ void __launch_bounds__(256, 4) paged_chunk_join_kernel(const __grid_constant__ PagedAttnParams P, int tpt,
                                                               int part_rows) {
    const PagedSeqs &S = P.seqs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_for_primary();
    const PartPlan plan = part_plan((int)P.plan[0]);
    const int2 *pre = reinterpret_cast<const int2 *>(P.plan + 1);  // (slots, pairs) cut before each sequence
    const int n_pairs = pre[S.n_seqs].y;
    const int per = part_rows / kJoinRows;
    for (int w = blockIdx.x; w < n_pairs * per; w += gridDim.x) {
        const int item = w / per;
        int lo = 0, hi = S.n_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid].y <= item) lo = mid;
            else hi = mid;
        }
        const SeqView v = seq_view(S, lo, P.hdr);
        const int pairs = seq_pairs(v, tpt), rem = item - pre[lo].y;
        const SeqCut c = seq_cut(v, P.hkv, tpt, plan);
        const int parts = c.parts, cut = c.items - c.whole;  // part i of a pair: i * cut slots further on
        const int h = (c.whole + rem) / pairs, at = (c.whole + rem) % pairs;
        const size_t slot0 = (size_t)pre[lo].x + (size_t)rem;
#pragma unroll 2
        for (int x = warp; x < kJoinRows; x += 8) {
            const int r = (w % per) * kJoinRows + x, in = (r & 127) / P.group;
            const int tok = ((pairs - 1 - at) * 2 + (r >> 7)) * tpt + in;
            if (in >= tpt || tok >= v.n) continue;
            float m = -INFINITY, l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = 0; i0 < parts; i0 += 4) {  // four parts in flight
                float2 ml[4];
                float4 o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const size_t row = (slot0 + (size_t)(i0 + j) * cut) * part_rows + r;
                    ml[j] = i0 + j < parts ? P.part_ml[row] : make_float2(-INFINITY, 0.f);
                    o[j] = i0 + j < parts ? reinterpret_cast<const float4 *>(P.part_o)[row * 32 + lane]
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                const float top = fmaxf(fmaxf(m, ml[0].x), fmaxf(ml[1].x, fmaxf(ml[2].x, ml[3].x)));
                const float a0 = m == -INFINITY ? 0.f : ex2_approx(m - top);
                m = top;
                l *= a0;
                acc = make_float4(acc.x * a0, acc.y * a0, acc.z * a0, acc.w * a0);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = ml[j].x == -INFINITY ? 0.f : ex2_approx(ml[j].x - m);
                    l = fmaf(ml[j].y, a, l);
                    acc.x = fmaf(o[j].x, a, acc.x);
                    acc.y = fmaf(o[j].y, a, acc.y);
                    acc.z = fmaf(o[j].z, a, acc.z);
                    acc.w = fmaf(o[j].w, a, acc.w);
                }
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
}

template <class Ty>
cudaError_t launch_chunk(const ChunkParams &C, cudaStream_t st) {
    const PagedSeqs &S = C.a.seqs;
    static std::atomic<unsigned long long> done{0};
    static std::atomic<int> regs{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(paged_chunk_kernel<Ty>), (int)kSmemMax, done);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc waits for registers the launch reserved: refuse to launch a
    // build whose register count at entry would make the split wait forever
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, paged_chunk_kernel<Ty>);
        if (e != cudaSuccess) return e;
        regs.store(fa.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < kRegsLaunch) return cudaErrorInvalidConfiguration;
    ProfScope prof("paged_chunk", st);
    const int bytes = (int)kSmemPlan + 8 * (S.n_seqs + 1) + 1024;
    paged_chunk_kernel<Ty><<<kGrid, kThreads, bytes, st>>>(C);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after(paged_chunk_join_kernel<Ty>, dim3(8 * kGrid), dim3(256), 0, st, C.a, C.tpt, C.part_rows);
}

}  // namespace

ChunkPlan paged_chunk_plan(int group, int max_q) { return {max_q <= 128 / group ? 128 : 256, 8 * kGrid}; }

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
