// sha_prefix_kernel.cuh -- the shared-prefix pass of sha_decode_prefix.
//
// When every row of a batch begins with the same P keys, the attention over
// them is, for each KV head h, one dense product: the query rows of all the
// (batch row, slot) units that select h -- R_h of them, G each -- against the
// same K_h, V_h [P, d].  Reading the prefix once per head instead of once per
// unit divides its traffic by R_h (about B * top_k / H_kv).  The softmax over a
// row's whole key range is put together from its two parts by the log-sum-exp
// rule: this kernel leaves (O, m, l) of each query row over [0, P), the suffix
// pass (sha_suffix_kernel.cuh) those over the row's own keys, and a
// third kernel, wide enough to keep many loads in flight, puts them together.  (Put
// together by the suffix pass at the end of each unit they cost it 3 us a unit, its
// ring standing full meanwhile: 113 us against 78 for the OPT-66B-shaped batch.)
//
// How the work is cut.  The selection is on the device, so each block plans for
// itself: a histogram of batch_head_index gives every head's units, 256 / G units
// make one row tile of up to 256 query rows, and the row tiles x key tiles (128
// keys) are numbered row-tile-major and cut into equal contiguous ranges, one per
// block, like the key tiles of the other kernels.  A run of key tiles within one
// row tile is one partial state, and the runs, in order, take the slots 0, 1, 2,
// ... : run (row tile r, block c) has slot r + c, since every next run advances
// one of the two or both.
//
// How a tile is computed.  Two streams of 128 query rows share the tensor cores:
//   * a producer warp brings the K and V tiles into a ring with TMA, in the order
//     in which they are used;
//   * one thread issues the products: S = Q K^T (both operands in shared memory)
//     into 128 columns of tensor memory per stream, O += P V (P from tensor memory,
//     V as it lies, MN-major) into d more;
//   * each stream's four softmax warps own one query row per thread: they read S,
//     write P = 2^(S c - m) over it, 16 bits wide (the type of the operands; the
//     sums l stay fp32 and add the unrounded P), and sum l.  A row's reference m
//     moves only when a tile's maximum exceeds it by more than 2^8: the weights
//     then stay below 256, any m is exact, and the accumulator in tensor memory is
//     rescaled in a few tiles instead of in all.
// While one stream's warps work on their scores the other stream's products run.
// A row tile of more than 128 rows gives each stream 128 of them and the same key
// tiles (compute-bound: the exponentials, 16 a clock, and the products, 2 x 512
// clocks a tile and stream, are about level); one of up to 128 rows gives both
// streams the same rows and every other key tile each (memory-bound: two key tiles
// in flight hide the chain S -> softmax -> P V of each).
#pragma once

#include <cuda.h>

#include "sha_device.cuh"
#include "sha_gqa_kernel.cuh"
#include "sha_tcgen05.cuh"

namespace sha {

constexpr int kPrefixMaxHeads = 1024;

// Where the prefix pass leaves its results.  Unit u's part over the prefix lies in
// ref[u].y consecutive slots from slot ref[u].x on, one per run of the prefix's key
// tiles, its G rows at rows ref[u].z .. of each -- and, with ref[u].w = 1, at those
// rows of the slot's second half, over other keys of the run.  A slot holds O (rows
// x d, unnormalised), then (m, l) per row, m in log2 units (-inf: no keys, and O is
// not to be read).
struct PrefixParts {
    int4 *ref;
    float *slots;
    int slot_floats, slot_rows;
};

struct PrefixParams {
    const void *q;
    const int32_t *idx;
    const int32_t *table;        // pages of the shared keys
    int B, H_q, H_kv, top_k;
    int keys;                    // P
    int page_size, num_pages;
    float scale_log2;            // scale * log2(e)
    PrefixParts parts;
};

// The last kernel of a call: units' states over the prefix and over their own keys
// put together.
struct PrefixMergeParams {
    const int32_t *idx, *seqlens;
    void *out;
    int B, H_q, H_kv, top_k;
    int min_len, max_len;
    PrefixParts parts;
    const int2 *runs;            // the suffix pass's runs of each unit, and their slots:
    const float *slots;          // O (G x d), then m (G), then l (G)
    int slot_floats;
};

template <int D>
struct PrefixConfig {
    using Tile = GqaConfig<D>;                       // key tiles and their swizzle
    static constexpr int kThreads = 384;             // producer, MMA, 2 spare warps; 2 x 4 softmax warps
    static constexpr int kSoftmax = 256;
    static constexpr int kSoftmaxWarp = 4;           // the first one
    static constexpr int kStreamRows = 128;
    static constexpr int kRows = 2 * kStreamRows;    // query rows of a row tile
    static constexpr int kTile = Tile::kTile;
    static constexpr int kTileBytes = Tile::kTileBytes;
    static constexpr int kBufs = D == 128 ? 4 : 8;   // ring of K and V tiles
    static constexpr int kQOffset = kBufs * kTileBytes;
    static constexpr int kQBytes = kTileBytes;       // 128 query rows, laid out like a key tile
    static constexpr int kBarOffset = kQOffset + 2 * kQBytes;
    static constexpr int kBars = 2 * kBufs + 1 + 2 + 2 + 2 + 2 + 1;
    static constexpr int kCtlOffset = kBarOffset + 8 * kBars + 8;   // abort, mode, TMEM base
    static constexpr int kWarpOffset = kCtlOffset + 16;             // warp counts of the list
    static constexpr int kUnitOffset = kWarpOffset + 4 * 8;         // a row tile's units
    static constexpr int kStartOffset = kUnitOffset + 4 * kRows;    // first row tile of each head
    static constexpr int kSmemBytes = 1024 + kStartOffset + 4 * (kPrefixMaxHeads + 1);
    // tensor memory: S (and P) of the two streams, then O
    static constexpr int kTmemCols = 512;
    static constexpr int kTmemO = 256;
    static_assert(kTile == 128, "128 keys: the N of S, the K of P V");
    static_assert(kBarOffset % 8 == 0 && kCtlOffset % 4 == 0, "alignment");
    static_assert(kTmemO + 2 * D <= kTmemCols, "S and O of both streams fit");
};

// A row's reference m moves when a tile's maximum exceeds it by more than this
// (log2 units): P stays below 2^8, far inside fp16.
constexpr float kPrefixSlack = 8.f;

// First row tile of every head (start[H_kv] = all of them), from the histogram
// of the selection.  All threads of the block; ends with a barrier.
template <int NT>
__device__ __forceinline__ void prefix_row_tiles(const PrefixParams &p, int units_per_tile,
                                                 int *start)
{
    const int tid = threadIdx.x;
    for (int h = tid; h <= p.H_kv; h += NT) start[h] = 0;
    __syncthreads();
    const int units = p.B * p.top_k;
    for (int u0 = tid; u0 < units; u0 += 4 * NT) {
        int h[4];                                    // four loads on the way at a time
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = u0 + i * NT < units ? p.idx[u0 + i * NT] : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((unsigned)h[i] < (unsigned)p.H_kv) atomicAdd(&start[h[i]], 1);
    }
    __syncthreads();
    if (tid < 32) {                                  // counts -> exclusive sums of row tiles
        int base = 0;
        for (int h0 = 0; h0 <= p.H_kv; h0 += 32) {
            const int h = h0 + tid;
            const int n = h < p.H_kv ? (start[h] + units_per_tile - 1) / units_per_tile : 0;
            int incl = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, off);
                if (tid >= off) incl += x;
            }
            if (h <= p.H_kv) start[h] = base + incl - n;
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __syncthreads();
}

// How the row tiles x key tiles are cut over the blocks: contiguous ranges of the
// tiles, numbered row-tile-major.  Beginning a run (its list, its queries, its
// state written out) takes a block about as long as kRunTiles key tiles, so whole
// row tiles, or equal pieces of them, go to the blocks where the busiest then has
// no more to do than under the even cut, which gives most blocks two runs.
// (OPT-66B-shaped, 72 row tiles of 15 key tiles: 2 pieces of 7 or 8 each, 144
// runs, against 219.)  All in 32 bits -- the host keeps the tiles of a call below
// 2^31 -- since a 64-bit division costs a lone thread 0.4 us.
constexpr unsigned kRunTiles = 3;

// A run: tiles [first, first + n) of row tile `row_tile`.
struct PrefixRun {
    int row_tile, first, n;
};

struct PrefixCut {
    unsigned key_tiles, blocks;
    unsigned pieces;             // > 0: a row tile is cut into this many, one per block
    unsigned base, extra;        // else block c has base tiles, the first `extra` one more
    unsigned t, t_end;           // this block's range

    __device__ __forceinline__ unsigned begin(unsigned c) const
    {
        return c * base + min(c, extra);
    }
    __device__ __forceinline__ void plan(unsigned row_tiles, unsigned tiles, unsigned grid,
                                         unsigned block)
    {
        key_tiles = tiles;
        const unsigned total = row_tiles * tiles;
        blocks = min(total, grid);
        pieces = 0;
        base = extra = t = t_end = 0;
        if (total == 0) return;
        const unsigned even = (total + blocks - 1) / blocks + 2 * kRunTiles;
        if (row_tiles <= blocks) {
            const unsigned p = min(blocks / row_tiles, tiles);
            if ((tiles + p - 1) / p + kRunTiles <= even) {
                pieces = p;
                blocks = row_tiles * p;
            }
        }
        if (pieces) {
            if (block < blocks) {
                const unsigned r = block / pieces, k = block - r * pieces;
                const unsigned b = tiles / pieces, x = tiles - b * pieces;
                t = r * tiles + k * b + min(k, x);
                t_end = t + b + (k < x);
            }
            return;
        }
        const unsigned whole = (row_tiles + blocks - 1) / blocks;
        if (row_tiles > blocks && whole * (tiles + kRunTiles) <= even) {
            t = min(block * whole, row_tiles) * tiles;
            t_end = min((block + 1) * whole, row_tiles) * tiles;
            base = whole * tiles;                    // begin() of a block in use
            return;
        }
        base = total / blocks;
        extra = total - base * blocks;
        if (block < blocks) {
            t = begin(block);
            t_end = begin(block + 1);
        }
    }
    __device__ __forceinline__ bool next(PrefixRun &r)
    {
        if (t >= t_end) return false;
        r.row_tile = (int)(t / key_tiles);
        const unsigned end = ((unsigned)r.row_tile + 1) * key_tiles;
        r.first = (int)(t - (unsigned)r.row_tile * key_tiles);
        r.n = (int)(min(end, t_end) - t);
        t += (unsigned)r.n;
        return true;
    }
    // Blocks that share the row tile which this block's run begins.
    __device__ __forceinline__ int sharers(const PrefixRun &r, unsigned block) const
    {
        if (r.first + r.n == (int)key_tiles) return 1;
        if (pieces) return (int)pieces;
        const unsigned last = ((unsigned)r.row_tile + 1) * key_tiles - 1;
        const unsigned split = extra * (base + 1);
        const unsigned c = last < split ? last / (base + 1) : extra + (last - split) / base;
        return (int)(c - block) + 1;
    }
};

// The head of row tile r: the last h with start[h] <= r among those that have tiles.
__device__ __forceinline__ int prefix_head_of(const int *start, int H_kv, int r)
{
    int lo = 0, hi = H_kv;                           // start[lo] <= r < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Ring position of a run's K and V tiles: K_0, then K_i, V_(i-1) for i = 1 .. n-1,
// then V_(n-1) -- the order in which the products use them.
__device__ __forceinline__ int prefix_k_pos(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int prefix_v_pos(int i, int n) { return i < n - 1 ? 2 * i + 2 : 2 * n - 1; }

template <typename T, int D>
__global__ void __launch_bounds__(PrefixConfig<D>::kThreads, 1)
    sha_prefix_kernel(const PrefixParams p, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v)
{
    using C = PrefixConfig<D>;
    using Tile = typename C::Tile;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t kIdescS = umma_idesc_f16(kBf16, 128, C::kTile);
    constexpr uint32_t kIdescO = umma_idesc_f16(kBf16, 128, D, false, true);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOffset);
    uint64_t *empty = full + C::kBufs;
    uint64_t *q_full = empty + C::kBufs;       // a run's queries are in shared memory
    uint64_t *s_full = q_full + 1;             // [stream] S is in tensor memory
    uint64_t *p_full = s_full + 2;             // [stream] P is
    uint64_t *pv_done = p_full + 2;            // [stream] P V has read P
    uint64_t *o_done = pv_done + 2;            // [stream] the run's last P V is done
    uint64_t *drain = o_done + 2;
    volatile int *ctl = reinterpret_cast<volatile int *>(smem + C::kCtlOffset);
    volatile int *abort_flag = ctl, *paired = ctl + 1;
    int *warp_counts = reinterpret_cast<int *>(smem + C::kWarpOffset);
    int *unit_list = reinterpret_cast<int *>(smem + C::kUnitOffset);
    int *start = reinterpret_cast<int *>(smem + C::kStartOffset);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int G = p.H_q / p.H_kv;
    const int units_per_tile = C::kRows / G;
    const int units = p.B * p.top_k;

    if (tid == 0) {
        for (int s = 0; s < C::kBufs; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(q_full, C::kSoftmax / 32);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
            mbar_init(&pv_done[s], 1);
            mbar_init(&o_done[s], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == 1) {
        tmem_alloc(reinterpret_cast<uint32_t *>(smem + C::kCtlOffset) + 2, C::kTmemCols);
        tmem_relinquish();
        tc_fence_before_sync();
    }
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = (uint32_t)ctl[2];
    pdl_wait();
    pdl_launch_dependents();

    prefix_row_tiles<C::kThreads>(p, units_per_tile, start);
    PrefixCut wk;
    wk.plan((unsigned)start[p.H_kv], (unsigned)((p.keys + C::kTile - 1) / C::kTile), gridDim.x,
            blockIdx.x);
    PrefixRun run;

    // waits give up together: the first that runs out raises the abort flag
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (*abort_flag) return false;
        if (mbar_wait(bar, parity)) return true;
        atomicOr(&g_sha_status, kStatusTimeout);
        *abort_flag = 1;
        return false;
    };

    if (warp == 0) {
        // -------------------------------------------------------- producer
        // every call reads the prefix again: the L2's default policy may keep it
        uint64_t policy;
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
        uint32_t used = 0, last_parity = 0;
        long long base = 0;
        bool ok = true;
        const int box_rows = min(p.page_size, C::kTile);
        while (ok && wk.next(run)) {
            const int h = prefix_head_of(start, p.H_kv, run.row_tile);
            const int n = run.n;
            for (int i = 0; ok && i < 2 * n; ++i) {
                // position i is K_0, K_((i+1)/2) (odd i < 2n-1) or V
                const bool is_k = i == 0 || ((i & 1) && i < 2 * n - 1);
                const int jj = is_k ? (i + 1) / 2 : (i == 2 * n - 1 ? n - 1 : i / 2 - 1);
                const int buf = (int)((base + i) % C::kBufs);
                const uint32_t parity = (uint32_t)((base + i) / C::kBufs) & 1u;
                if (lane == 0) ok = wait(&empty[buf], parity ^ 1);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const int n0 = (run.first + jj) * C::kTile;
                const int rows = min(C::kTile, p.keys - n0);
                const int chunks = (rows + box_rows - 1) / box_rows;
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[buf],
                                          (uint32_t)(chunks * Tile::kBoxes * box_rows * 128));
                __syncwarp();
                unsigned char *dst = smem + buf * C::kTileBytes;
                for (int c = lane; c < chunks; c += 32) {
                    const int key = n0 + c * box_rows;
                    const int pi = key / p.page_size, off = key - pi * p.page_size;
                    int page = p.table[pi];
                    if ((unsigned)page >= (unsigned)p.num_pages) {
                        atomicOr(&g_sha_status, kStatusBadIndex);
                        page = 0;                       // stay inside the pool
                    }
                    for (int bx = 0; bx < Tile::kBoxes; ++bx)
                        tma_load_3d(dst + bx * Tile::kBoxBytes + c * box_rows * 128,
                                    is_k ? &tm_k : &tm_v, bx * 64, off, page * p.H_kv + h,
                                    &full[buf], policy);
                }
                last_parity = (last_parity & ~(1u << buf)) | (parity << buf);
                used |= 1u << buf;
            }
            base += 2 * n;
        }
        if (lane == 0)
            for (int s = 0; s < C::kBufs; ++s)
                if (used & (1u << s)) mbar_wait_drain(&full[s], (last_parity >> s) & 1u);
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------- products
        if (lane == 0) {
            long long base = 0;
            uint32_t q_parity = 0, p_parity = 0, pv_parity = 0;    // bit per stream
            bool ok = true;
            while (ok && wk.next(run)) {
                const int n = run.n;
                ok = wait(q_full, q_parity);
                q_parity ^= 1;
                if (!ok) break;
                tc_fence_after_sync();
                const bool pair = *paired != 0;
                // S of tile i for a stream; `last`: no other stream reads this K tile after it
                auto scores = [&](int st, int i, bool last) {
                    const long long pos = base + prefix_k_pos(i);
                    const int buf = (int)(pos % C::kBufs);
                    if (!wait(&full[buf], (uint32_t)(pos / C::kBufs) & 1u)) return false;
                    const uint32_t qa = smem_addr(smem + C::kQOffset + (pair ? st : 0) * C::kQBytes);
                    const uint32_t kb = smem_addr(smem + buf * C::kTileBytes);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t at = (ks >> 2) * Tile::kBoxBytes + (ks & 3) * 32;
                        umma_f16(tmem + st * 128, umma_desc_k_sw128(qa + at),
                                 umma_desc_k_sw128(kb + at), kIdescS, ks > 0);
                    }
                    umma_commit(&s_full[st]);
                    if (last) umma_commit(&empty[buf]);
                    return true;
                };
                // O += P V of tile i; then S of tile `next` may take P's place
                auto outputs = [&](int st, int i, bool first, bool last, bool end) {
                    if (!wait(&p_full[st], (p_parity >> st) & 1u)) return false;
                    p_parity ^= 1u << st;
                    const long long pos = base + prefix_v_pos(i, n);
                    const int buf = (int)(pos % C::kBufs);
                    if (!wait(&full[buf], (uint32_t)(pos / C::kBufs) & 1u)) return false;
                    tc_fence_after_sync();
                    const uint32_t vb = smem_addr(smem + buf * C::kTileBytes);
#pragma unroll
                    for (int ks = 0; ks < C::kTile / 16; ++ks)
                        umma_f16_tmem_a(tmem + C::kTmemO + st * D, tmem + st * 128 + ks * 8,
                                        umma_desc_mn_sw128(vb + ks * 2048, Tile::kBoxBytes, 1024),
                                        kIdescO, !(first && ks == 0));
                    umma_commit(&pv_done[st]);
                    if (last) umma_commit(&empty[buf]);
                    if (end) umma_commit(&o_done[st]);
                    return true;
                };
                auto read_p = [&](int st) {              // P V has read P: S may overwrite it
                    const bool done = wait(&pv_done[st], (pv_parity >> st) & 1u);
                    pv_parity ^= 1u << st;
                    return done;
                };
                if (pair) {
                    ok = scores(0, 0, false) && scores(1, 0, true);
                    for (int i = 0; ok && i < n; ++i)
                        for (int st = 0; ok && st < 2; ++st) {
                            ok = outputs(st, i, i == 0, st == 1, i == n - 1) && read_p(st);
                            if (ok && i + 1 < n) ok = scores(st, i + 1, st == 1);
                        }
                } else {
                    ok = scores(0, 0, true);
                    if (ok && n > 1) ok = scores(1, 1, true);
                    for (int i = 0; ok && i < n; ++i) {
                        const int st = i & 1;
                        ok = outputs(st, i, i < 2, true, i + 2 >= n) && read_p(st);
                        if (ok && i + 2 < n) ok = scores(st, i + 2, true);
                    }
                }
                base += 2 * n;
            }
            umma_commit(drain);                          // before tensor memory is freed
            mbar_wait_drain(drain, 0);
        }
        __syncwarp();
    } else if (warp >= C::kSoftmaxWarp) {
        // -------------------------------------------------------- softmax
        const unsigned FULL = 0xffffffffu;
        const int stid = tid - 32 * C::kSoftmaxWarp;     // 0 .. 255
        const int swarp = warp - C::kSoftmaxWarp;
        const int st = swarp >> 2;
        const int row = (swarp & 3) * 32 + lane;         // of the stream: this thread's TMEM lane
        const uint32_t lanes = (uint32_t)((swarp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + st * 128;
        const uint32_t o_at = tmem + lanes + C::kTmemO + st * D;
        const float scale = fabsf(p.scale_log2);
        const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;   // -q instead of -scale
        uint32_t s_parity = 0, o_parity = 0;
        long long base = 0;
        bool ok = true;
        while (wk.next(run)) {
            const int rt = run.row_tile;
            const int h = prefix_head_of(start, p.H_kv, rt);
            // this row tile's units: those of the head's units, in order, that the
            // tiles before it have not taken
            const int rank0 = (rt - start[h]) * units_per_tile;
            named_barrier(1, C::kSoftmax);                // the last run's list has been read
            // (a contiguous share of the units per thread: count, scan, then place)
            const int per = (units + C::kSoftmax - 1) / C::kSoftmax;
            const int share0 = min(stid * per, units), share1 = min(share0 + per, units);
            int mine = 0;
            for (int u = share0; u < share1; u += 8) {        // eight loads on the way
#pragma unroll
                for (int i = 0; i < 8; ++i) mine += u + i < share1 && p.idx[u + i] == h;
            }
            int incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(FULL, incl, off);
                if (lane >= off) incl += x;
            }
            if (lane == 31) warp_counts[swarp] = incl;
            named_barrier(1, C::kSoftmax);
            int rank = incl - mine - rank0, seen = 0;
#pragma unroll
            for (int w = 0; w < C::kSoftmax / 32; ++w) {
                if (w < swarp) rank += warp_counts[w];
                seen += warp_counts[w];
            }
            if (mine > 0 && rank < units_per_tile && rank + mine > 0)
                for (int u = share0; u < share1; ++u)
                    if (p.idx[u] == h) {
                        if (rank >= 0 && rank < units_per_tile) unit_list[rank] = u;
                        ++rank;
                    }
            named_barrier(1, C::kSoftmax);
            const int n_units = min(seen - rank0, units_per_tile);
            const int n_rows = n_units * G;
            const bool pair = n_rows > C::kStreamRows;
            const int slot_id = rt + (int)blockIdx.x;
            if (run.first == 0) {
                const int sharers = wk.sharers(run, blockIdx.x);
                for (int i = stid; i < n_units; i += C::kSoftmax)
                    p.parts.ref[unit_list[i]] =
                        make_int4(slot_id, sharers, i * G, pair ? 0 : 1);
            }

            // the queries, swizzled like a key tile; the last 32 rows are filled up
            // with zeros, and what lies behind them is nobody's
            constexpr int kChunks = D / 8, kPass = C::kSoftmax / kChunks;
            const int c = stid % kChunks;
#pragma unroll 4
            for (int r = stid / kChunks; r < ((n_rows + 31) & ~31); r += kPass) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (r < n_rows) {
                    const int e = r / G, u = unit_list[e];
                    x = *reinterpret_cast<const uint4 *>(
                        static_cast<const T *>(p.q) +
                        ((size_t)(u / p.top_k) * p.H_q + (size_t)h * G + (r - e * G)) * D + c * 8);
                    x.x ^= flip;
                    x.y ^= flip;
                    x.z ^= flip;
                    x.w ^= flip;
                }
                const int rr = r & (C::kStreamRows - 1);
                *reinterpret_cast<uint4 *>(smem + C::kQOffset + (r >> 7) * C::kQBytes +
                                           (c >> 3) * Tile::kBoxBytes + rr * 128 +
                                           (((c & 7) ^ (rr & 7)) << 4)) = x;
            }
            if (stid == 0) *paired = pair;
            fence_proxy_async_shared();
            tc_fence_before_sync();                       // the last run's O has been read
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);

            const int n = run.n;
            const int tile_row = (pair ? st * C::kStreamRows : 0) + (swarp & 3) * 32;
            const bool busy = tile_row < n_rows;          // this warp has rows
            float m_ref = -INFINITY, l0 = 0.f, l1 = 0.f;
            int done = 0;
            for (int i = pair ? 0 : st; i < n; i += pair ? 1 : 2) {
                if (ok) ok = __all_sync(FULL, wait(&s_full[st], s_parity));
                s_parity ^= 1;
                const int rows = min(C::kTile, p.keys - (run.first + i) * C::kTile);
                if (rows < C::kTile) {
                    // rows past the prefix hold other keys or nothing: zero V there
                    // (0 * NaN) before any product with this tile's P.  Both streams
                    // of a pair read the tile: they zero half each, and meet.
                    const long long pos = base + prefix_v_pos(i, n);
                    const int buf = (int)(pos % C::kBufs);
                    if (ok) ok = __all_sync(FULL, wait(&full[buf], (uint32_t)(pos / C::kBufs) & 1u));
                    if (ok) {
                        unsigned char *vt = smem + buf * C::kTileBytes;
                        const int left = (C::kTile - rows) * Tile::kBoxes * 8;
                        for (int e = pair ? stid : stid & 127; e < left; e += pair ? 256 : 128) {
                            const int chunk = e & 7, bx = (e >> 3) % Tile::kBoxes;
                            const int key = rows + (e >> 3) / Tile::kBoxes;
                            *reinterpret_cast<uint4 *>(vt + bx * Tile::kBoxBytes + key * 128 +
                                                       chunk * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_shared();
                    }
                    if (pair) named_barrier(1, C::kSoftmax);
                }
                if (ok && busy) {
                    tc_fence_after_sync();
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float s[32];
                        tmem_ld32(s_at + c * 32, s);
                        tmem_ld_wait();
                        if (rows < C::kTile) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (c * 32 + e >= rows) s[e] = -INFINITY;
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e) top = fmaxf(top, s[e]);
                    }
                    top *= scale;
                    // the first tile sets the reference, later ones move it rarely
                    const bool move = done == 0 || top > m_ref + kPrefixSlack;
                    if (__any_sync(FULL, move)) {
                        const float m_new = move ? top : m_ref;
                        if (done > 0) {
                            const float a = move ? exp2_approx(m_ref - m_new) : 1.f;
                            l0 *= a;
                            l1 *= a;
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                float o[32];
                                tmem_ld32(o_at + c * 32, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= a;
                                tmem_st32(o_at + c * 32, o);
                            }
                        }
                        m_ref = m_new;
                    }
                    const float m0 = m_ref == -INFINITY ? 0.f : m_ref;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float s[32];
                        tmem_ld32(s_at + c * 32, s);
                        tmem_ld_wait();
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            s[e] = exp2_approx(fmaf(s[e], scale, -m0));
                            if (rows < C::kTile && c * 32 + e >= rows) s[e] = 0.f;
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            l0 += s[2 * e];
                            l1 += s[2 * e + 1];
                            w[e] = pack2<T>(s[2 * e], s[2 * e + 1]);
                        }
                        tmem_st16(s_at + c * 16, w);
                    }
                    tmem_st_wait();
                }
                ++done;
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[st]);
            }

            // this run's partial state: rows of slot rt + block, the second stream's
            // behind the first's (its own rows, or the other half of the keys)
            if (done > 0) {
                if (ok) ok = __all_sync(FULL, wait(&o_done[st], o_parity));
                o_parity ^= 1;
            }
            if (tile_row + lane < n_rows) {
                float *slot = p.parts.slots + (size_t)slot_id * p.parts.slot_floats;
                const int r = st * C::kStreamRows + row;
                *reinterpret_cast<float2 *>(slot + (size_t)C::kRows * D + 2 * r) =
                    make_float2(ok && done > 0 ? m_ref : -INFINITY, l0 + l1);
            }
            if (ok && done > 0 && busy) {
                tc_fence_after_sync();
                float *out = p.parts.slots + (size_t)slot_id * p.parts.slot_floats +
                             (size_t)(st * C::kStreamRows + row) * D;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(o_at + c * 32, o);
                    tmem_ld_wait();
                    if (tile_row + lane < n_rows) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(out + c * 32 + e) =
                                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
            }
            base += 2 * n;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// One output row per D/4 lanes, four elements a lane.  The parts' (m, l) are read
// one per lane, so that all of them, their weights 2^(m - M) and the sum L cost one
// trip to memory; then the lanes add up the weighted O rows, eight loads in flight.
// More parts than lanes go in rounds, the sums rescaled in between.  The order is
// fixed: suffix runs, then prefix runs.
template <typename T, int D>
__global__ void __launch_bounds__(256) sha_prefix_merge_kernel(const PrefixMergeParams p)
{
    constexpr int kLanes = D / 4;
    const unsigned FULL = 0xffffffffu;
    const int G = p.H_q / p.H_kv;
    const int sub = threadIdx.x % kLanes;
    const long long rows = (long long)p.B * p.top_k * G;
    const long long at = ((long long)blockIdx.x * 256 + threadIdx.x) / kLanes;
    // (the call's inputs were complete before the passes began)
    const bool inside = at < rows;
    const int u = inside ? (int)(at / G) : 0, j = inside ? (int)(at - (long long)u * G) : 0;
    const int b = u / p.top_k, h = p.idx[u], len = p.seqlens[b];
    // units that no pass has touched
    const bool live = inside && (unsigned)h < (unsigned)p.H_kv && len >= p.min_len && len <= p.max_len;
    pdl_wait();
    pdl_launch_dependents();
    int2 run = make_int2(0, 0);
    int4 ref = make_int4(0, 0, 0, 0);
    if (live) {
        run = __ldcg(p.runs + u);
        ref = __ldcg(p.parts.ref + u);
    }
    const int halves = 1 + ref.w;
    const int n = run.y + ref.y * halves;
    int rounds = (n + kLanes - 1) / kLanes;
    if (kLanes < 32) rounds = max(rounds, __shfl_xor_sync(FULL, rounds, 16));

    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, L = 0.f;
    for (int r = 0; r < rounds; ++r) {
        // this lane's part: where its row of O is, its (m, l)
        const int i = r * kLanes + sub;
        const float *o = nullptr;
        float m = -INFINITY, l = 0.f;
        if (i < run.y) {
            const float *slot = p.slots + (size_t)(run.x + i) * p.slot_floats;
            o = slot + j * D;
            m = __ldcg(slot + G * D + j);
            l = __ldcg(slot + G * D + G + j);
        } else if (i < n) {
            const int k = i - run.y;
            const float *slot = p.parts.slots + (size_t)(ref.x + k / halves) * p.parts.slot_floats;
            const int row = ref.z + j + (k & ref.w) * (p.parts.slot_rows / 2);
            o = slot + (size_t)row * D;
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(
                slot + (size_t)p.parts.slot_rows * D + 2 * row));
            m = ml.x;
            l = ml.y;
        }
        float top = m;
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(FULL, top, off));
        const float m_new = fmaxf(M, top);
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float a = exp2f(M - base);
        const float w = exp2f(m - base);
        float sum = w * l;
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(FULL, sum, off);
        L = fmaf(a, L, sum);
        M = m_new;
        O.x *= a;
        O.y *= a;
        O.z *= a;
        O.w *= a;
        int parts = min(n - r * kLanes, kLanes);
        if (kLanes < 32) parts = max(parts, __shfl_xor_sync(FULL, parts, 16));
#pragma unroll 8
        for (int k = 0; k < parts; ++k) {
            const float wk = __shfl_sync(FULL, w, k, kLanes);
            const float *ok = reinterpret_cast<const float *>(__shfl_sync(
                FULL, reinterpret_cast<unsigned long long>(o), k, kLanes));
            if (wk != 0.f) {                     // (no keys, or nothing left of them)
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(ok + 4 * sub));
                O.x = fmaf(wk, x.x, O.x);
                O.y = fmaf(wk, x.y, O.y);
                O.z = fmaf(wk, x.z, O.z);
                O.w = fmaf(wk, x.w, O.w);
            }
        }
    }
    if (!live) return;
    T *dst = static_cast<T *>(p.out) + ((size_t)b * p.H_q + (size_t)h * G + j) * D + 4 * sub;
    *reinterpret_cast<uint2 *>(dst) =
        make_uint2(pack2<T>(O.x / L, O.y / L), pack2<T>(O.z / L, O.w / L));
}

}  // namespace sha
