// paged.cuh -- definitions shared by the kernels of the paged key/value cache.
//
// A cache holds pages of P tokens, [num_pages][hkv][P][128]; a sequence's token
// at position p lives in page block_tables[s][p / P], row p % P.  The new
// tokens of sequence s are rows cu_q[s] .. cu_q[s + 1] - 1 of q, k and v, at
// positions kv_lens[s] - n .. kv_lens[s] - 1.  Lengths, tables and lists live on
// the device, so a captured graph can be replayed as the sequences grow; what
// the host cannot check, the kernels check before they use it.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "sm100.cuh"

namespace minf {

constexpr int kMaxSeqs = 4096;  // sequences per call (their prefix sums sit in shared memory)

// Data errors a kernel found (status MINF_ERR_INVALID, read back by minf_status);
// the sequence or page concerned is left out.
enum : int { BAD_SEQ = 1, BAD_PAGE = 2, BAD_POSITION = 3, BAD_BLOCK = 4 };

__device__ __forceinline__ void flag_invalid(WsHeader *hdr, int what) {
    // every CTA may find the same fault thousands of times: only the first ones write
    if (*reinterpret_cast<volatile int *>(&hdr->status) != 0 && *reinterpret_cast<volatile int *>(&hdr->site) != 0) return;
    atomicCAS(&hdr->status, 0, MINF_ERR_INVALID);
    atomicCAS(&hdr->site, 0, what | 0x20000000);
}

struct PagedSeqs {
    const int *cu_q;          // [n_seqs + 1]
    const int *kv_lens;       // [n_seqs]
    const int *tables;        // [n_seqs][tstride]
    long long tstride;
    int n_seqs, total, width, max_q, page, page_log2, num_pages;
};

struct SeqView {
    int q0, n, len;  // first row, new tokens, tokens stored (new ones included)
};

// Sequence s, or an empty one (n = 0) where its numbers contradict the call's.
// The comparisons hold for every 32-bit value the device arrays may carry.
__device__ __forceinline__ SeqView seq_view(const PagedSeqs &S, int s, WsHeader *hdr) {
    const int q0 = __ldg(S.cu_q + s), q1 = __ldg(S.cu_q + s + 1), len = __ldg(S.kv_lens + s);
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= S.total && q1 - q0 <= S.max_q && len >= 0 &&
                    (long long)len <= (long long)S.width * S.page;
    if (!ok) {
        flag_invalid(hdr, BAD_SEQ);
        return {0, 0, 0};
    }
    return {q0, q1 - q0, len};
}

// Page of logical block b (< width) of sequence s, or -1.
__device__ __forceinline__ int page_of(const PagedSeqs &S, int s, int b, WsHeader *hdr) {
    const int p = __ldg(S.tables + (long long)s * S.tstride + b);
    if ((unsigned)p >= (unsigned)S.num_pages) {
        flag_invalid(hdr, BAD_PAGE);
        return -1;
    }
    return p;
}

// Item `idx` of a call in which sequence s has count(s) items: its sequence and which
// of that one's items it is.  The whole CTA calls it; false if there are fewer items.  Sums are
// 64-bit: starts that contradict each other can name the same rows over and over.
template <int kThreads, class Count>
__device__ __forceinline__ bool find_item(int n_seqs, int idx, Count count, int &seq, int &item) {
    __shared__ long long sums[kThreads / 32];
    __shared__ int hit[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (n_seqs + kThreads - 1) / kThreads;
    const int sa = min((int)threadIdx.x * per, n_seqs), sb = min(sa + per, n_seqs);
    long long mine = 0;
    for (int s = sa; s < sb; ++s) mine += count(s);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) sums[warp] = inc;
    if (threadIdx.x == 0) hit[0] = -1;
    __syncthreads();
    long long at = inc - mine;
    for (int w = 0; w < warp; ++w) at += sums[w];
    if (at <= idx && idx < at + mine) {
        for (int s = sa;; ++s) {
            const int n = count(s);
            if (idx < at + n) {
                hit[0] = s;
                hit[1] = (int)(idx - at);
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    seq = hit[0];
    item = hit[1];
    return seq >= 0;
}

// 16-bit float pairs of the two cache types.
struct Bf16 {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
    static __device__ __forceinline__ uint32_t vmin(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t vmax(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static constexpr uint32_t kPosInf2 = 0x7f807f80u, kNegInf2 = 0xff80ff80u;
    // D (16x8 fp32) += A (16x16) B (16x8)
    static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
    static constexpr uint32_t kIdescType = (1u << 7) | (1u << 10);  // A and B format: bf16
    // P = 2^(x - m + shift): bf16 has fp32's range and needs no shift
    static constexpr float kShift = 0.f, kLag = 8.f;
};

struct Fp16 {
    using T = __half;
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ uint32_t vmin(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t vmax(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static constexpr uint32_t kPosInf2 = 0x7c007c00u, kNegInf2 = 0xfc00fc00u;
    static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
    static constexpr uint32_t kIdescType = 0;
    // fp16 ends at 2^-24 below and 65504 above: P is formed 2^10 larger, and the
    // running max may lag by 2^4, so P stays below 2^14 and a weight keeps its
    // 11 bits down to 2^-24 of the row's largest.
    static constexpr float kShift = 10.f, kLag = 4.f;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, uint32_t bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(tmap), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// One launch after another may start while the first still runs (its wait below);
// the first allows it with launch_dependents.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The end of a kernel launched that way.  Its CTAs may leave without needing the first
// kernel's results, but the grid must not end before that kernel: what follows it in the
// stream waits for this grid alone.  One CTA that waits holds the grid.
__device__ __forceinline__ void end_after_primary() {
    if ((blockIdx.x | blockIdx.y | blockIdx.z) == 0) wait_for_primary();
}

// Lets `kernel` take `bytes` of dynamic shared memory on the current device; a
// kernel's `done` remembers the devices on which that is set (a launch per layer
// of a decoding step would pay for it each time).
inline cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<unsigned long long> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Launches a kernel so that its start overlaps the end of the one before it in
// the stream; it waits for that one's results itself (wait_for_primary).
template <class... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------------------------ launches
// TMA descriptors with 128-byte swizzle: any 4-D 16-bit tensor (strides in bytes),
// and the pages of a cache, {128, P, hkv, pages} with `rows` keys x 64 channels a box.
cudaError_t make_tmap_4d(CUtensorMap *map, const void *base, bool fp16, const cuuint64_t (&dims)[4],
                         const cuuint64_t (&strides)[3], const cuuint32_t (&box)[4]);
cudaError_t make_tmap_pages(CUtensorMap *map, const void *base, bool fp16, int page, int hkv, int num_pages,
                            long long page_stride, int rows);

struct AppendParams {
    PagedSeqs seqs;
    const void *k, *v, *q;
    void *q_out, *k_cache, *v_cache, *k_bounds;
    const float *rope;
    long long k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, qo_ts, qo_hs;  // token and head strides, in elements
    long long kc_ps, vc_ps;                                      // page strides of the caches
    int hq, hkv, rot, rope_rows;
    bool packed;  // grid x counts the pages of all sequences, not those of one
    WsHeader *hdr;
};
cudaError_t run_paged_append(const AppendParams &P, bool fp16, bool interleaved, cudaStream_t st);

struct PagedAttnParams {
    PagedSeqs seqs;
    const void *q, *k, *v;
    void *out;
    float *lse;                         // [total][hq], nullable
    long long q_ts, q_hs, o_ts, o_hs;   // token and head strides, in elements
    long long kc_ps, vc_ps;             // page strides of the caches
    int hq, hkv, group;
    float scale_log2;
    const int *blk_idx, *blk_cnt;       // per-token page lists (null: every stored page)
    int topk;
    // partial states of split work: unnormalised O [slot][rows][128], (max, sum)
    // [slot][rows]; and the kernel's plan, for the one that joins them
    float *part_o;
    float2 *part_ml;
    long long *plan;
    int n_slots;
    WsHeader *hdr;
    unsigned long long wait_limit_ns;
};
// The streaming kernel's query rows per tile, and partial slots: two to a CTA that
// takes a share of the work (page lists: 0 with a CTA to each item).
struct StreamPlan {
    int rows, n_slots;
};
StreamPlan paged_stream_plan(int group, int max_q);
StreamPlan paged_sparse_plan(int total, int hkv, int group, int topk, int page);
// The largest plan of a call of at most so many tokens and list entries, for any page size.
StreamPlan paged_sparse_reserve(int total, int hkv, int group, int topk);
cudaError_t run_paged_stream(const PagedAttnParams &P, bool fp16, int rows, cudaStream_t st);
cudaError_t run_paged_sparse(const PagedAttnParams &P, bool fp16, int rows, cudaStream_t st);

// The chunk kernel's partial slots, and their rows.
struct ChunkPlan {
    int part_rows, n_slots;
};
ChunkPlan paged_chunk_plan(int group, int max_q);
cudaError_t run_paged_chunk(const PagedAttnParams &P, bool fp16, int part_rows, cudaStream_t st);

constexpr int kMaxBlocks = 32768;  // pages of a sequence the selection handles
struct EstimateParams {
    PagedSeqs seqs;
    const void *q, *bounds;
    long long q_ts, q_hs;
    int hq, hkv, group, topk;
    int *blk_idx, *blk_cnt;  // [total][hkv][topk], [total][hkv]
    float *scores;           // [batch][hkv][score_stride]
    float *top;              // [batch][hkv][ranges] at a tile's first token: largest |bound| of its page range
    bool packed;             // grid x counts the tiles of all sequences, not those of one
    int score_stride, batch;
    int t0, t1, tiles, tile_tokens, pages_per_cta, ranges;  // per launch
    WsHeader *hdr;
    unsigned long long wait_limit_ns;
};
struct EstimatePlan {
    int score_stride, batch;  // batch: tokens scored at a time
    size_t n_scores, n_top;
};
EstimatePlan paged_estimate_plan(int total, int n_seqs, int hkv, int width);
// Scores and tops that suffice for every call of at most so many tokens and table columns.
EstimatePlan paged_estimate_reserve(int total, int hkv, int width);
cudaError_t run_paged_estimate(const EstimateParams &P, bool fp16, cudaStream_t st);

}  // namespace minf
