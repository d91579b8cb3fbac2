// sha_suffix_kernel.cuh -- the rows' own keys in sha_decode_prefix, the part of its
// blocks that do not work on the prefix (sha_prefix_kernel.cuh): for each
// selected (batch row, slot) unit the attention of its G query rows over keys
// [P, len) of the row's pages, left as partial states (O, m, l) for the merge.
//
// What bounds it.  HBM traffic where rows have grown long; but behind a shared
// prefix a row's own keys are often few (a turn of a dialogue, the tokens sampled
// so far), and then it is the latency of each unit: its head id, its queries, its
// first tile, its result.  A block that walks units one after the other with all
// its warps (the grouped decode kernel) spent 3 us on a unit of 128 keys, twice
// the time its bytes take.  Here every warp is a worker of its own: it has its own
// ring of key stages in shared memory, issues its own TMA loads, keeps its own
// softmax state in registers and writes it out itself, with no barrier between
// warps.  The workers of an SM (6 at d = 128, 10 at d = 64) hide one another's
// latencies, and their rings (2 stages of 32 keys) together keep 190 KiB in flight.
//
// How, for a stage of 32 keys.  The products are turned over, keys and head
// elements on the MMA's 16-wide side and the G query rows on its 8-wide side (two
// of them for G > 8), so that groups of up to 8 waste nothing: S^T = K Q^T by
// mma.sync m16n8k16, K fragments by ldmatrix from the 128-byte-swizzled boxes, Q
// as the B operand in registers; online softmax down the columns; O^T += V^T P^T
// with V^T by ldmatrix.trans and P, rounded to the tensor type, transposed in
// registers (movmatrix).  The sums l and O stay fp32.  With the query rows on the
// 16-wide side the same stage took twice the MMAs and exponentials.
//
// How the work is cut.  A unit weighs its stages plus kUnitCost for its latency;
// the weights of all units, in unit order, are cut into equal contiguous ranges,
// one per worker.  Run (unit u, worker w) leaves its state in slot u + w: the next
// run exceeds it, u or w or both having advanced.
#pragma once

#include <cuda.h>

#include "sha_device.cuh"
#include "sha_gqa_kernel.cuh"
#include "sha_mma.cuh"

namespace sha {

struct SuffixParams {
    const void *q;
    const int32_t *idx, *seqlens, *block_table;
    int B, H_q, H_kv, top_k;
    int min_len, max_len;        // valid row lengths: [P, max_pages * page_size]
    bool empty_rows;             // a length of 0 marks a row without a token, not bad input
    int key0;                    // first key loaded: P rounded down to a TMA box
    int page_shift, max_pages, num_pages;    // pages of 2^page_shift keys
    float scale_log2;            // scale * log2(e)
    int2 *runs;                  // unit u's runs: slots runs[u].x .. , runs[u].y of them
    float *slots;                // O (G x d, unnormalised), m (G, log2 units), l (G)
    int slot_floats;
};

// How keys lie in shared memory here and in the prefix's tiles: groups of 8 keys, each
// 64 elements of the 8 (128-byte rows, 1 KiB, 128-byte-swizzled), then the next 64.
// One copy of a 5-D map [64 elements][8 keys][d/64][groups][pages and heads] brings
// a whole run of keys of a page that way.  (Two boxes of [keys][64 elements] per run
// take twice the copies, and a lone warp issues one in about 115 clocks: pages of 16
// keys then bound the prefix at 3700 clocks a tile.)
template <int D>
struct KeyGroups {
    static constexpr int kBytes = 1024 * (D / 64);
};
__device__ __forceinline__ void tma_load_groups(void *dst, const CUtensorMap *map, int group,
                                                int plane, uint64_t *bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %2, %2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(plane), "r"(smem_addr(bar)),
        "l"(policy)
        : "memory");
}

template <int D>
struct SuffixConfig {
    static constexpr int kWorkers = D == 128 ? 6 : 10;   // warps of the block at work
    static constexpr int kStage = 32;                    // keys
    static constexpr int kStages = 2;
    static constexpr int kBoxes = D / 64;
    static constexpr int kGroupBytes = KeyGroups<D>::kBytes;
    static constexpr int kTileBytes = kStage / 8 * kGroupBytes;  // K or V of a stage
    static constexpr int kRingBytes = kStages * 2 * kTileBytes;
    // a unit's latency in stages: with 6 workers an SM streams a 32-key stage in
    // 0.37 us, and a unit costs a worker about 4 us, 0.7 us of the SM
    static constexpr int kUnitCost = 2;
    static constexpr int kMinWeight = 4;                 // of a worker's range
    static constexpr int kMaxRuns = 64;                  // of a unit, about
};

// Stages of a row's own keys (at least one: a row that ends with the prefix still
// has a state to leave), 0 for a length outside the valid range.
__device__ __forceinline__ int suffix_stages(const SuffixParams &p, int len, int stage)
{
    if (len < p.min_len || len > p.max_len) return 0;
    const int n = len - p.key0;
    return n > stage ? (n + stage - 1) / stage : 1;
}

// a / b, b >= 1, exactly.  The integer divisions of a plan stand one behind the other
// in a lone warp, 150 clocks each in 32 bits and 700 in 64.  For a < 2^20 a float
// quotient is exact: (a + 1/2) / b lies at least 1/(2b) from an integer, and the
// approximate division (2 ulp) is off by at most 2^-22 of a quotient below 2^20 / b.
__host__ __device__ __forceinline__ unsigned div_fast(unsigned a, unsigned b)
{
#ifdef __CUDA_ARCH__
    if (a < (1u << 20)) return (unsigned)__fdividef((float)a + 0.5f, (float)min(b, 1u << 24));
#endif
    return a / b;
}
__device__ __forceinline__ long long div_fast(long long a, long long b)
{
    if (((a | b) >> 32) == 0) return div_fast((unsigned)a, (unsigned)b);
    return a / b;
}

struct SuffixRun {
    int unit, b;
    int first, n;        // stages of the unit
    int keys;            // of the unit, from key0 on
    long long end;       // weight at which the unit ends
};

// A worker's range of the units' weights, walked unit by unit.
struct SuffixWalk {
    long long base, t, t_end;          // workers have base weights, the first `extra` one more
    long long unit_start;
    int extra;
    int b, k, T, len;                  // current unit: row, slot, stages, row length

    __device__ __forceinline__ long long begin(int w) const
    {
        return w * base + (w < extra ? w : extra);
    }
    // the last worker of the unit that this worker's run `r` begins
    __device__ __forceinline__ int last_worker(const SuffixRun &r, int worker) const
    {
        if (r.end <= t_end) return worker;
        const long long last = r.end - 1, split = (long long)extra * (base + 1);
        return last < split ? (int)div_fast(last, base + 1)
                            : extra + (int)div_fast(last - split, base);
    }
    template <int D>
    __device__ __forceinline__ bool next(const SuffixParams &p, SuffixRun &r)
    {
        using C = SuffixConfig<D>;
        while (t < t_end) {
            const long long unit_end = unit_start + T + C::kUnitCost;
            const long long end = unit_end < t_end ? unit_end : t_end;
            const int x0 = (int)(t - unit_start) - C::kUnitCost;
            const int x1 = (int)(end - unit_start) - C::kUnitCost;
            r.unit = b * p.top_k + k;
            r.b = b;
            r.first = x0 > 0 ? x0 : 0;
            r.n = x1 - r.first;
            r.keys = len - p.key0;
            r.end = unit_end;
            t = end;
            if (end == unit_end && t < t_end) {            // on to the next unit that has stages
                unit_start = unit_end;
                if (++k == p.top_k) {
                    k = 0;
                    do {
                        ++b;
                        len = p.seqlens[b];
                        T = suffix_stages(p, len, C::kStage);
                    } while (T == 0);
                }
            }
            if (r.n > 0) return true;
        }
        return false;
    }
};

// The weights of all units and the longest row's stages.  All NT threads of the
// block; scratch: shared, 2 * NT / 32 longs.  The caller synchronises before and
// after; `sum` and `longest` come from the scratch by suffix_read_totals.
template <int D, int NT>
__device__ __forceinline__ void suffix_totals(const SuffixParams &p, long long *scratch)
{
    using C = SuffixConfig<D>;
    const unsigned FULL = 0xffffffffu;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long sum = 0;
    int tmax = 0;
    for (int r = tid; r < p.B; r += NT) {
        const int len = p.seqlens[r], T = suffix_stages(p, len, C::kStage);
        if (T == 0) {
            if (blockIdx.x == 0 && !(p.empty_rows && len == 0))
                atomicOr(&g_sha_status, kStatusBadIndex);
        } else {
            sum += (long long)p.top_k * (T + C::kUnitCost);
            tmax = max(tmax, T);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        sum += __shfl_xor_sync(FULL, sum, off);
        tmax = max(tmax, __shfl_xor_sync(FULL, tmax, off));
    }
    if (lane == 0) {
        scratch[2 * warp] = sum;
        scratch[2 * warp + 1] = tmax;
    }
}
template <int NT>
__device__ __forceinline__ void suffix_read_totals(const long long *scratch, long long &sum,
                                                   int &longest)
{
    sum = 0;
    longest = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        sum += scratch[2 * i];
        longest = max(longest, (int)scratch[2 * i + 1]);
    }
}

// The walk of worker `worker` of all `all` (a whole warp calls it together): false if
// it has nothing to do.
template <int D>
__device__ __forceinline__ bool suffix_plan(const SuffixParams &p, long long total, int longest,
                                            int all, int worker, SuffixWalk &w)
{
    using C = SuffixConfig<D>;
    const unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    if (total == 0) return false;
    // workers in use: each with kMinWeight at least, and no unit in many more than
    // kMaxRuns pieces
    long long least = (longest + C::kMaxRuns - 1) / C::kMaxRuns;
    if (least < C::kMinWeight) least = C::kMinWeight;
    const int n = total >= all * least ? all : total < least ? 1 : (int)div_fast(total, least);
    if (worker >= n) return false;
    w.base = div_fast(total, (long long)n);
    w.extra = (int)(total - w.base * n);
    w.t = w.begin(worker);
    w.t_end = w.begin(worker + 1);

    // the row that holds weight t: prefix sums over rows, 32 at a time
    long long base = 0;
    for (int r0 = 0;; r0 += 32) {
        const int r = r0 + lane;
        const int len = r < p.B ? p.seqlens[r] : -1;
        const int T = r < p.B ? suffix_stages(p, len, C::kStage) : 0;
        const long long val = T ? (long long)p.top_k * (T + C::kUnitCost) : 0;
        long long incl = val;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long x = __shfl_up_sync(FULL, incl, off);
            if (lane >= off) incl += x;
        }
        const long long row_start = base + incl - val;
        const unsigned here =
            __ballot_sync(FULL, val > 0 && row_start <= w.t && w.t < row_start + val);
        if (here) {
            const int src = __ffs(here) - 1;
            w.b = r0 + src;
            w.T = __shfl_sync(FULL, T, src);
            w.len = __shfl_sync(FULL, len, src);
            const long long start = __shfl_sync(FULL, row_start, src);
            w.k = (int)div_fast(w.t - start, (long long)(w.T + C::kUnitCost));
            w.unit_start = start + (long long)w.k * (w.T + C::kUnitCost);
            return true;
        }
        base += __shfl_sync(FULL, incl, 31);
    }
}

// The softmax's reference lies this far below the running maximum (log2 units): fp16
// weights, up to 2^15, use the type's upper exponents, too, and are rounded by at most
// 2^-40 of the largest instead of 2^-25.  bf16 has the exponents of fp32.
template <typename T>
constexpr float kSuffixLift = std::is_same<T, __half>::value ? 15.f : 0.f;

// An 8 x 8 tile of 16-bit elements, one packed pair per lane, transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// One worker (a warp) of a block.  kNT: 8-row tiles of query rows (1 for G <= 8, else
// 2).  ring: this worker's, 1 KiB aligned; full: its kStages barriers, initialised.
template <typename T, int D, int kNT>
__device__ __forceinline__ void suffix_worker(const SuffixParams &p, const CUtensorMap &tm_k,
                                              const CUtensorMap &tm_v, SuffixWalk walk, int worker,
                                              unsigned char *ring, uint64_t *full,
                                              volatile int *abort_flag)
{
    using C = SuffixConfig<D>;
    constexpr int kKT = C::kStage / 16;                 // 16-key tiles of a stage
    const int lane = threadIdx.x & 31;
    const unsigned FULL = 0xffffffffu;
    const int G = p.H_q / p.H_kv;

    // ---- the loads: stage by stage through this worker's runs, ahead of the use
    const uint64_t policy = l2_policy_evict_first();
    const int box_shift = min(p.page_shift, 5);
    static_assert(C::kStage == 32, "boxes of up to 2^5 keys");
    const int box_kv = lane & 1, box_c = lane >> 1;
    const CUtensorMap *box_map = box_kv ? &tm_v : &tm_k;
    const uint32_t box_bytes = (uint32_t)(2 * C::kBoxes * 128) << box_shift;   // a chunk, K and V
    unsigned char *box_dst =
        ring + box_kv * C::kTileBytes + (box_c << box_shift) / 8 * C::kGroupBytes;
    SuffixWalk lw = walk;
    SuffixRun lr = {}, ln = {};          // the run being loaded, the next one
    int lh, lnh = 0, li = 0;             // their head ids; the next stage of lr
    bool more, next_more;
    int page = 0, chunks = 0, key = 0;   // that stage: this lane's page, boxes, this lane's key
    int issued = 0;
    auto look_up = [&]() {               // used a stage later
        const int n0 = (lr.first + li) * C::kStage;
        chunks = (min(C::kStage, lr.keys - n0) + (1 << box_shift) - 1) >> box_shift;  // 0: no key
        key = p.key0 + n0 + (box_c << box_shift);
        if (box_c < chunks) page = p.block_table[(size_t)lr.b * p.max_pages + (key >> p.page_shift)];
    };
    auto next_run = [&]() {
        do {
            more = next_more;
            lr = ln;
            lh = lnh;
            if (!more) return;
            next_more = lw.next<D>(p, ln);
            if (next_more) lnh = p.idx[ln.unit];
        } while ((unsigned)lh >= (unsigned)p.H_kv);
        li = 0;
        look_up();
    };
    auto issue = [&]() {
        if (!more) return;
        const int stage = issued % C::kStages;
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], chunks * box_bytes);
        __syncwarp();
        if (box_c < chunks) {
            if ((unsigned)page >= (unsigned)p.num_pages) {
                atomicOr(&g_sha_status, kStatusBadIndex);
                page = 0;                               // stay inside the pool
            }
            tma_load_groups(box_dst + stage * 2 * C::kTileBytes, box_map,
                            (key & ((1 << p.page_shift) - 1)) >> 3, page * p.H_kv + lh,
                            &full[stage], policy);
        }
        ++issued;
        if (++li == lr.n) next_run();
        else look_up();
    };
    next_more = lw.next<D>(p, ln);
    if (next_more) lnh = p.idx[ln.unit];
    next_run();
    for (int s = 0; s < C::kStages; ++s) issue();

    // ---- the products
    const int g = lane >> 2, qd = lane & 3, mi = lane >> 3, mr = lane & 7;
    // ldmatrix rows of this lane: K tiles are (keys, d), V^T tiles (d, keys)
    const uint32_t k_row = smem_addr(ring) + (mi & 1) * C::kGroupBytes + mr * 128;
    const uint32_t v_row =
        smem_addr(ring) + C::kTileBytes + (mi >> 1) * C::kGroupBytes + mr * 128;
    const uint32_t k_half = (uint32_t)(mi >> 1), v_half = (uint32_t)(mi & 1);
    // the 16-byte chunk of a box row, swizzled by the row (which is mr modulo 8)
    auto chunk_at = [&](uint32_t chunk) { return ((chunk & 7) ^ (uint32_t)mr) << 4; };
    int used = 0;
    bool ok = true;
    SuffixRun run, run_next;
    int h = 0, h_next = 0;
    bool has = walk.next<D>(p, run_next);
    if (has) h_next = p.idx[run_next.unit];
    while (has) {
        run = run_next;
        h = h_next;
        has = walk.next<D>(p, run_next);
        if (has) h_next = p.idx[run_next.unit];
        if ((unsigned)h >= (unsigned)p.H_kv) {
            if (lane == 0) atomicOr(&g_sha_status, kStatusBadIndex);
            continue;
        }
        // Q^T of the group as the MMA's B operand: row 8 nt + g (zero past G)
        uint32_t qb[kNT][D / 16][2];
        {
            const T *qg = static_cast<const T *>(p.q) + ((size_t)run.b * p.H_q + (size_t)h * G) * D;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                const int row = nt * 8 + g;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        qb[nt][ks][e] = row < G ? *reinterpret_cast<const uint32_t *>(
                                                      qg + row * D + ks * 16 + qd * 2 + 8 * e)
                                                : 0u;
            }
        }
        if (run.first == 0 && lane == 0)
            p.runs[run.unit] =
                make_int2(run.unit + worker, walk.last_worker(run, worker) - worker + 1);
        // state of query rows 8 nt + 2 qd + {0, 1}; l over this lane's keys only
        float m_run[kNT][2], l_run[kNT][2];
        float o[kNT][D / 16][4];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            m_run[nt][0] = m_run[nt][1] = -INFINITY;
            l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
            for (int n = 0; n < D / 16; ++n) o[nt][n][0] = o[nt][n][1] = o[nt][n][2] = o[nt][n][3] = 0.f;
        }

        for (int i = 0; i < run.n; ++i) {
            const int stage = used % C::kStages;
            if (ok) {
                ok = __all_sync(FULL, *abort_flag == 0 &&
                                          mbar_wait(&full[stage], (used / C::kStages) & 1));
                if (!ok && lane == 0) {
                    if (*abort_flag == 0) atomicOr(&g_sha_status, kStatusTimeout);
                    *abort_flag = 1;
                }
            }
            if (!ok) continue;
            const int rows = min(C::kStage, run.keys - (run.first + i) * C::kStage);
            // a unit's first stage begins with the prefix's last keys
            const int lo = run.first + i == 0 ? p.min_len - p.key0 : 0;
            const bool ragged = rows < C::kStage || lo > 0;
            if (ragged) {
                // keys outside the row's own may be anything: zero V there (0 * NaN)
                unsigned char *v = ring + (stage * 2 + 1) * C::kTileBytes;
                for (int e = lane; e < C::kStage * C::kBoxes * 8; e += 32) {
                    const int chunk = e & 7, bx = (e >> 3) % C::kBoxes, kk = (e >> 3) / C::kBoxes;
                    if (kk >= rows || kk < lo)
                        *reinterpret_cast<uint4 *>(v + (kk >> 3) * C::kGroupBytes + bx * 1024 +
                                                   (kk & 7) * 128 + chunk * 16) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_shared();   // before the stage is refilled by TMA
                __syncwarp();
            }
            const uint32_t kt = k_row + stage * 2 * C::kTileBytes;
            const uint32_t vt = v_row + stage * 2 * C::kTileBytes;
            // S^T: 16-key tiles; entries (key g, row 2 qd + {0, 1}), (key g + 8, the same)
            float s[kNT][kKT][4];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int kk = 0; kk < kKT; ++kk)
                    s[nt][kk][0] = s[nt][kk][1] = s[nt][kk][2] = s[nt][kk][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int kk = 0; kk < kKT; ++kk) {
                    uint32_t ka[4];
                    ldmatrix_x4(kt + (ks >> 2) * 1024 + kk * 2 * C::kGroupBytes +
                                    chunk_at(ks * 2 + k_half),
                                ka);
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
                        mma_16816<T>(s[nt][kk], ka, qb[nt][ks][0], qb[nt][ks][1]);
                }
            uint32_t pb[kNT][kKT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int kk = 0; kk < kKT; ++kk)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[nt][kk][e] *= p.scale_log2;
                        if (ragged) {
                            const int k = kk * 16 + (e >> 1) * 8 + g;
                            if (k >= rows || k < lo) s[nt][kk][e] = -INFINITY;
                        }
                        mt[e & 1] = fmaxf(mt[e & 1], s[nt][kk][e]);
                    }
                float ref[2], alpha[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    mt[r] = fmaxf(mt[r], __shfl_xor_sync(FULL, mt[r], 4));
                    mt[r] = fmaxf(mt[r], __shfl_xor_sync(FULL, mt[r], 8));
                    mt[r] = fmaxf(mt[r], __shfl_xor_sync(FULL, mt[r], 16));
                    const float m_new = fmaxf(m_run[nt][r], mt[r] - kSuffixLift<T>);
                    ref[r] = m_new == -INFINITY ? 0.f : m_new;
                    alpha[r] = exp2_approx(m_run[nt][r] - ref[r]);
                    m_run[nt][r] = m_new;
                    l_run[nt][r] *= alpha[r];
                }
#pragma unroll
                for (int kk = 0; kk < kKT; ++kk) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[nt][kk][e] = exp2_approx(s[nt][kk][e] - ref[e & 1]);
                        l_run[nt][e & 1] += s[nt][kk][e];
                    }
                    pb[nt][kk][0] = movmatrix_trans(pack2<T>(s[nt][kk][0], s[nt][kk][1]));
                    pb[nt][kk][1] = movmatrix_trans(pack2<T>(s[nt][kk][2], s[nt][kk][3]));
                }
                // a maximum that did not move leaves O as it is
                if (__any_sync(FULL, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                    for (int n = 0; n < D / 16; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[nt][n][e] *= alpha[e & 1];
                }
            }
            // O^T += V^T P^T
#pragma unroll
            for (int kk = 0; kk < kKT; ++kk)
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t va[4];
                    ldmatrix_x4_trans(vt + (n >> 2) * 1024 + kk * 2 * C::kGroupBytes +
                                          chunk_at(n * 2 + v_half),
                                      va);
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
                        mma_16816<T>(o[nt][n], va, pb[nt][kk][0], pb[nt][kk][1]);
                }
            ++used;
            __syncwarp();                     // the stage has been read
            issue();
        }

        // this run's state
        float *slot = p.slots + (size_t)(run.unit + worker) * p.slot_floats;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float l = l_run[nt][r];
                l += __shfl_xor_sync(FULL, l, 4);
                l += __shfl_xor_sync(FULL, l, 8);
                l += __shfl_xor_sync(FULL, l, 16);
                const int row = nt * 8 + qd * 2 + r;
                if (row < G) {
#pragma unroll
                    for (int n = 0; n < D / 16; ++n) {
                        slot[row * D + n * 16 + g] = o[nt][n][r];
                        slot[row * D + n * 16 + 8 + g] = o[nt][n][2 + r];
                    }
                    if (g == 0) {
                        slot[G * D + row] = m_run[nt][r];
                        slot[G * D + G + row] = l;
                    }
                }
            }
    }
    // after a wait that gave up: the loads in flight still write into this block
    for (; used < issued; ++used)
        if (lane == 0) mbar_wait_drain(&full[used % C::kStages], (used / C::kStages) & 1);
    __syncwarp();
}

}  // namespace sha
