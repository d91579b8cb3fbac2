// sha_prefix_kernel.cuh -- the kernels of sha_decode_prefix.
//
// When every row of a batch begins with the same P keys, the attention over
// them is, for each KV head h, one dense product: the query rows of all the
// (batch row, slot) units that select h -- R_h of them, G each -- against the
// same K_h, V_h [P, d].  Reading the prefix once per head instead of once per
// unit divides its traffic by R_h (about B * top_k / H_kv).  The softmax over a
// row's whole key range is put together from its two parts by the log-sum-exp
// rule: some blocks of the first kernel leave (O, m, l) of each query row over
// [0, P), the others (sha_suffix_kernel.cuh) those over the rows' own keys, and a
// second kernel, wide enough to keep many loads in flight, puts them together.
// (Put together at the end of each unit they cost its block 3 us a unit, its ring
// standing full meanwhile.)
//
// The two parts run side by side, not one after the other: each alone leaves the
// memory idle while it plans, fetches its first tiles and writes its states.  How
// many blocks take the prefix is decided on the device, by a small cost model of
// both parts (prefix_share).
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
// How a tile is computed.  Two streams of 128 query rows share the tensor cores, in
// steps of 64 keys:
//   * one warp brings the K tiles, one the V tiles into a ring with TMA, in the order
//     in which they are used;
//   * one warp per stream issues its products: S = Q K^T (both operands in shared
//     memory) into 64 columns of tensor memory, O += P V (P from 32 columns of
//     tensor memory, V as it lies, MN-major) into d more.  (A lone warp takes about
//     500 clocks to wait for and issue a product: one for both streams was the
//     bound, 7500 clocks a tile of 256 rows by 128 keys.)
//   * each stream's four softmax warps own one query row per thread: they read S
//     into registers, which frees it for the next step's product at once, and write
//     P = 2^(S c - m), 16 bits wide (the type of the operands; the sums l stay fp32
//     and add the unrounded P).  A row's reference m moves only when a step's
//     maximum exceeds the last one by kPrefixSlack: any m is exact, and the
//     accumulator in tensor memory is rescaled in a few steps instead of in all.
// So a step's exponentials run beside the next step's S and the last one's P V.
// (Steps of 128 keys leave P no columns of its own but S's: each product then waits
// for the one before it and the exponentials for both, 4840 clocks for a tile of 256
// rows by 128 keys against 4350.)
// A row tile of more than 128 rows gives each stream 128 of them and every key of a
// tile (bound by the exponentials, 16 a clock, and the products, about level); one
// of up to 128 rows gives both streams the same rows and one half of each key tile
// (bound by memory).
#pragma once

#include <cuda.h>

#include "sha_device.cuh"
#include "sha_gqa_kernel.cuh"
#include "sha_suffix_kernel.cuh"
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
    using Tile = GqaConfig<D>;                       // key tiles
    static constexpr int kGroupBytes = KeyGroups<D>::kBytes;
    static constexpr int kThreads = 384;             // K, 2 MMA, V; 2 x 4 softmax warps
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
    static constexpr int kStep = 64;                 // keys of a step
    static constexpr int kBars = 2 * kBufs + 2 + 2 + 2 + 2 + 2 + 2;
    static constexpr int kCtlOffset = kBarOffset + 8 * kBars + 8;   // abort, mode, TMEM base
    static constexpr int kWarpOffset = kCtlOffset + 16;             // warp counts of the list
    static constexpr int kLastOffset = kWarpOffset + 4 * 8;         // ring position last in each buffer
    static constexpr int kUnitOffset = kLastOffset + 4 * kBufs;     // a row tile's units
    static constexpr int kQRowOffset = kUnitOffset + 4 * kRows;     // and the rows of q they are
    static constexpr int kStartOffset = kQRowOffset + 4 * kRows;    // first row tile of each head
    static constexpr int kPairOffset = kStartOffset + 4 * (kPrefixMaxHeads + 1);
    static constexpr int kPlanOffset = (kPairOffset + 4 * (kPrefixMaxHeads + 1) + 7) / 8 * 8;
    static constexpr int kSuffixBarOffset = kPlanOffset + 16 * (kThreads / 32);
    static constexpr int kSmemBytes =
        1024 + kSuffixBarOffset + 8 * SuffixConfig<D>::kWorkers * SuffixConfig<D>::kStages;
    // tensor memory: S of the two streams, P, then O
    static constexpr int kTmemCols = 512;
    static constexpr int kTmemP = 2 * kStep;
    static constexpr int kTmemO = 256;
    static_assert(kTile == 2 * kStep, "two steps of a tile, one per stream or two of both");
    static_assert(kBarOffset % 8 == 0 && kCtlOffset % 4 == 0, "alignment");
    static_assert(SuffixConfig<D>::kWorkers * SuffixConfig<D>::kRingBytes <= kBarOffset,
                  "the workers' rings lie where the tiles and queries would");
    static_assert(SuffixConfig<D>::kWorkers <= kThreads / 32, "a warp per worker");
    static_assert(kTmemP + kStep <= kTmemO && kTmemO + 2 * D <= kTmemCols, "S, P and O fit");
};

// A row's reference m moves when a step's maximum exceeds the one it was taken from by
// more than the slack (log2 units), and lies the lift below that one.  fp16 weights so
// use the type's upper exponents, too (up to 2^15), and are rounded by at most 2^-36 of
// the largest; with m the maximum itself that is 2^-25, below which they were lost, and
// many such keys together are not small beside one key's output.  bf16 has the exponents
// of fp32.
template <typename T>
constexpr float kPrefixSlack = std::is_same<T, __half>::value ? 4.f : 8.f;
template <typename T>
constexpr float kPrefixLift = std::is_same<T, __half>::value ? 11.f : 0.f;

// First row tile of every head (start[H_kv] = all of them), and how many row tiles
// of more than 128 rows come before it (pairs[H_kv] = all of those), from the
// histogram of the selection.  All threads of the block; ends with a barrier.
template <int NT>
__device__ __forceinline__ void prefix_row_tiles(const PrefixParams &p, int G, int units_per_tile,
                                                 int *start, int *pairs)
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
    if (tid < 32) {                                  // counts -> exclusive sums
        int base = 0, pair_base = 0;
        for (int h0 = 0; h0 <= p.H_kv; h0 += 32) {
            const int h = h0 + tid;
            const int count = h < p.H_kv ? start[h] : 0;
            const int n = (count + units_per_tile - 1) / units_per_tile;
            // all but a head's last row tile are full
            const int m = n > 0 ? n - 1 + ((count - (n - 1) * units_per_tile) * G > 128) : 0;
            int incl = n, pair_incl = m;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, off);
                const int y = __shfl_up_sync(0xffffffffu, pair_incl, off);
                if (tid >= off) {
                    incl += x;
                    pair_incl += y;
                }
            }
            if (h <= p.H_kv) {
                start[h] = base + incl - n;
                pairs[h] = pair_base + pair_incl - m;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
            pair_base += __shfl_sync(0xffffffffu, pair_incl, 31);
        }
    }
    __syncthreads();
}

// How the row tiles x key tiles are cut over the blocks: contiguous ranges of the
// tiles, numbered row-tile-major.  Beginning a run (its list, its queries, its
// state written out) takes a block about as long as kRunTiles key tiles, so equal
// pieces of row tiles go to the blocks, one each, where there are enough blocks:
// twice as many pieces of a row tile of more than 128 rows, whose key tiles take
// twice the products (16K document, heads with 256 + 64 rows: 26 us against 37 with
// pieces alike), and no more pieces than the longest one needs, since each leaves a
// state to be merged.  (OPT-66B-shaped, 72 row tiles of 15 key tiles: 2 pieces of 7
// or 8 each, 144 runs, against 219 under the even cut.)  With more row tiles than
// blocks, whole row tiles or an even cut of the tiles.  All in 32 bits -- the host
// keeps the tiles of a call below 2^31 -- since a 64-bit division costs a lone
// thread 0.4 us.
constexpr unsigned kRunTiles = 3;

// A run: tiles [first, first + n) of row tile `row_tile`, of head `head`.
struct PrefixRun {
    int row_tile, head, first, n;
};

struct PrefixCut {
    const int *start, *pairs;    // of the heads (prefix_row_tiles)
    int heads;
    unsigned key_tiles;
    unsigned pieces, pieces2;    // > 0: pieces of a row tile of up to, of more than 128 rows
    unsigned used;               // blocks with tiles
    unsigned base, extra;        // else block c has base tiles, the first `extra` one more
    unsigned t, t_end;           // this block's range
    int own_pieces;              // (pieces) those of this block's row tile

    __host__ __device__ __forceinline__ unsigned begin(unsigned c) const
    {
        return c * base + min(c, extra);
    }
    // First block of head h, under pieces.
    __host__ __device__ __forceinline__ unsigned block_of(int h) const
    {
        return (unsigned)start[h] * pieces + (unsigned)pairs[h] * (pieces2 - pieces);
    }
    // The last head whose first f(head) is at most x: among equal ones the last is
    // the one that has row tiles.
    template <class F>
    __host__ __device__ __forceinline__ int search(unsigned x, F f) const
    {
        int lo = 0, hi = heads;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (f(mid) <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    }
    __host__ __device__ __forceinline__ void plan(const int *start_, const int *pairs_, int heads_,
                                         unsigned tiles, unsigned grid, unsigned block)
    {
        start = start_;
        pairs = pairs_;
        heads = heads_;
        key_tiles = tiles;
        pieces = pieces2 = base = extra = t = t_end = used = 0;
        const unsigned row_tiles = (unsigned)start[heads], wide = (unsigned)pairs[heads];
        const unsigned total = row_tiles * tiles;
        if (total == 0) return;
        const unsigned weight = row_tiles + wide;
        if (weight <= grid) {
            // the longest piece of each kind, then as few pieces as keep to it
            const unsigned p1 = min(div_fast(grid, weight), tiles);
            const unsigned p2 = min(div_fast(2 * grid, weight), tiles);
            const unsigned q1 = div_fast(tiles + p1 - 1, p1), q2 = div_fast(tiles + p2 - 1, p2);
            pieces = div_fast(tiles + q1 - 1, q1);
            pieces2 = div_fast(tiles + q2 - 1, q2);
            used = block_of(heads);
            if (block >= used) return;
            const int h = search(block, [&](int x) { return block_of(x); });
            unsigned k = block - block_of(h);
            const unsigned wide_tiles = (unsigned)(pairs[h + 1] - pairs[h]);
            unsigned r = div_fast(k, pieces2), own = pieces2;
            if (r >= wide_tiles) {               // the last row tile, of up to 128 rows
                r = wide_tiles;
                own = pieces;
            }
            k -= r * pieces2;
            const unsigned b = div_fast(tiles, own), x = tiles - b * own;
            t = ((unsigned)start[h] + r) * tiles + k * b + min(k, x);
            t_end = t + b + (k < x);
            own_pieces = (int)own;
            return;
        }
        const unsigned blocks = min(total, grid);
        const unsigned even = (total + blocks - 1) / blocks + 2 * kRunTiles;
        const unsigned whole = (row_tiles + blocks - 1) / blocks;
        if (whole * (tiles + kRunTiles) <= even) {
            used = (row_tiles + whole - 1) / whole;
            t = min(block * whole, row_tiles) * tiles;
            t_end = min((block + 1) * whole, row_tiles) * tiles;
            return;
        }
        used = blocks;
        base = total / blocks;
        extra = total - base * blocks;
        if (block < blocks) {
            t = begin(block);
            t_end = begin(block + 1);
        }
    }
    __host__ __device__ __forceinline__ bool next(PrefixRun &r)
    {
        if (t >= t_end) return false;
        r.row_tile = (int)div_fast(t, key_tiles);
        r.head = search((unsigned)r.row_tile, [&](int x) { return (unsigned)start[x]; });
        const unsigned end = ((unsigned)r.row_tile + 1) * key_tiles;
        r.first = (int)(t - (unsigned)r.row_tile * key_tiles);
        r.n = (int)(min(end, t_end) - t);
        t += (unsigned)r.n;
        return true;
    }
    // Blocks that share the row tile which this block's run begins.
    __host__ __device__ __forceinline__ int sharers(const PrefixRun &r, unsigned block) const
    {
        if (r.first + r.n == (int)key_tiles) return 1;
        if (pieces) return own_pieces;
        const unsigned last = ((unsigned)r.row_tile + 1) * key_tiles - 1;
        const unsigned split = extra * (base + 1);
        const unsigned c = last < split ? last / (base + 1) : extra + (last - split) / base;
        return (int)(c - block) + 1;
    }
};

// How many of the call's `blocks` blocks the prefix may take: the number at which
// the slower of the two parts is done first, out of 32 evenly spaced ones, one per
// lane of the calling warp.  Times in ns, measured: a run's beginning and end; a key
// tile of 128 keys by up to 128 rows, and by more; a worker's beginning; an SM's
// share of a weight of the suffix (32 keys' bytes, per 64 elements of d).
constexpr float kPrefixRunNs = 10000.f, kPrefixTileNs = 1600.f, kPrefixWideNs = 2450.f;
constexpr float kSuffixRunNs = 5000.f, kSuffixWeightNs = 100.f;

// A quotient for the estimates below, the division approximate on the device.
__host__ __device__ __forceinline__ float div_approx(float a, float b)
{
#ifdef __CUDA_ARCH__
    return __fdividef(a, b);
#else
    return a / b;
#endif
}
// The i-th share tried, and the time that the call takes with it.
__host__ __device__ __forceinline__ int prefix_share_at(int i, int blocks)
{
    return max(1, min(blocks - 1, (i + 1) * blocks / 33));
}
__host__ __device__ __forceinline__ float prefix_share_ns(int share, int row_tiles, int wide,
                                                          int tiles, long long weights, int d64,
                                                          int blocks)
{
    const int weight = row_tiles + wide;
    float t;
    const float f = (float)tiles;
    if (weight <= share) {
        const float per = div_approx((float)share + 0.5f, (float)weight);
        const float p1 = fminf(floorf(per), f), p2 = fminf(floorf(2.f * per), f);
        t = fmaxf(row_tiles > wide ? ceilf(div_approx(f, p1) - 1e-3f) * kPrefixTileNs : 0.f,
                  wide > 0 ? ceilf(div_approx(f, p2) - 1e-3f) * kPrefixWideNs : 0.f) +
            kPrefixRunNs;
    } else {
        const float each = div_approx(1.f, (float)share);
        t = ((float)(row_tiles - wide) * kPrefixTileNs + (float)wide * kPrefixWideNs) * f * each +
            ceilf((float)row_tiles * each) * kPrefixRunNs;
    }
    return fmaxf(t, kSuffixRunNs + div_approx((float)weights * (kSuffixWeightNs * (float)d64),
                                              (float)(blocks - share)));
}
__device__ __forceinline__ int prefix_share(int row_tiles, int wide, int tiles, long long weights,
                                            int d64, int blocks)
{
    int best = prefix_share_at(threadIdx.x & 31, blocks);
    float t = prefix_share_ns(best, row_tiles, wide, tiles, weights, d64, blocks);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, t, off);
        const int y = __shfl_xor_sync(0xffffffffu, best, off);
        if (x < t || (x == t && y < best)) {
            t = x;
            best = y;
        }
    }
    return best;
}

// Ring position of a run's K and V tiles: K_0, then K_i, V_(i-1) for i = 1 .. n-1,
// then V_(n-1) -- the order in which the products use them.
__host__ __device__ __forceinline__ int prefix_k_pos(int i) { return i == 0 ? 0 : 2 * i - 1; }
__host__ __device__ __forceinline__ int prefix_v_pos(int i, int n) { return i < n - 1 ? 2 * i + 2 : 2 * n - 1; }

// The steps of 64 keys that the two streams take through a run of `tiles` key
// tiles, the last with `rows` keys: paired streams take both halves of every tile,
// others one each.  Stream 1 never takes more than stream 0.
struct PrefixSteps {
    bool pair;
    int tiles, last_halves;          // halves of the last tile that hold keys: 1 or 2

    __host__ __device__ __forceinline__ PrefixSteps(bool pair_, int tiles_, int rows)
        : pair(pair_), tiles(tiles_), last_halves(rows > 64 ? 2 : 1)
    {
    }
    __host__ __device__ __forceinline__ int count(int st) const
    {
        return pair ? 2 * tiles - 2 + last_halves : st < last_halves ? tiles : tiles - 1;
    }
    __host__ __device__ __forceinline__ int tile(int step) const { return pair ? step >> 1 : step; }
    __host__ __device__ __forceinline__ int half(int st, int step) const { return pair ? step & 1 : st; }
    // whether no later step of the stream needs this step's tile
    __host__ __device__ __forceinline__ bool last_of_tile(int st, int step) const
    {
        return !pair || (step & 1) || step == count(st) - 1;
    }
    // whether the stream has a step in the last tile
    __host__ __device__ __forceinline__ bool takes_last(int st) const { return pair || st < last_halves; }
};

// kNT: see suffix_worker.  Maps in groups of 8 keys (KeyGroups): tm_k, tm_v with boxes
// of up to 128 keys, ts_k, ts_v of up to 32.
template <typename T, int D, int kNT>
__global__ void __launch_bounds__(PrefixConfig<D>::kThreads, 1)
    sha_prefix_kernel(const PrefixParams p, const SuffixParams suffix,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap ts_k,
                      const __grid_constant__ CUtensorMap ts_v)
{
    using C = PrefixConfig<D>;
    using Tile = typename C::Tile;
    using Suffix = SuffixConfig<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t kIdescS = umma_idesc_f16(kBf16, 128, C::kStep);
    constexpr uint32_t kIdescO = umma_idesc_f16(kBf16, 128, D, false, true);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOffset);
    uint64_t *empty = full + C::kBufs;
    uint64_t *q_full = empty + C::kBufs;       // a run's queries are in shared memory
    uint64_t *q_seen = q_full + 1;             // both streams' MMA warps have begun the run
    uint64_t *s_full = q_seen + 1;             // [stream] S is in tensor memory
    uint64_t *s_free = s_full + 2;             // [stream] S has been read
    uint64_t *p_full = s_free + 2;             // [stream] P is in tensor memory
    uint64_t *pv_done = p_full + 2;            // [stream] P V is done: P read, O up to date
    uint64_t *drain = pv_done + 2;             // [stream] before tensor memory is freed
    volatile int *ctl = reinterpret_cast<volatile int *>(smem + C::kCtlOffset);
    volatile int *abort_flag = ctl, *paired = ctl + 1;
    int *warp_counts = reinterpret_cast<int *>(smem + C::kWarpOffset);
    int *unit_list = reinterpret_cast<int *>(smem + C::kUnitOffset);
    volatile int *last_load = reinterpret_cast<volatile int *>(smem + C::kLastOffset);
    int *q_rows = reinterpret_cast<int *>(smem + C::kQRowOffset);
    int *start = reinterpret_cast<int *>(smem + C::kStartOffset);
    int *pairs = reinterpret_cast<int *>(smem + C::kPairOffset);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int G = p.H_q / p.H_kv;
    const int units_per_tile = C::kRows / G;
    const int units = p.B * p.top_k;

    if (tid == 0) {
        for (int s = 0; s < C::kBufs; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);                 // both streams have used the tile
            last_load[s] = -1;
        }
        mbar_init(q_full, C::kSoftmax / 32);
        mbar_init(q_seen, 2);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_free[s], 4);
            mbar_init(&p_full[s], 4);
            mbar_init(&pv_done[s], 1);
            mbar_init(&drain[s], 1);
        }
        *abort_flag = 0;
        uint64_t *own = reinterpret_cast<uint64_t *>(smem + C::kSuffixBarOffset);
        for (int s = 0; s < Suffix::kWorkers * Suffix::kStages; ++s) mbar_init(&own[s], 1);
        mbar_init_fence();
    }
    pdl_wait();
    pdl_launch_dependents();

    // the two parts' work, and who does what
    long long *plan = reinterpret_cast<long long *>(smem + C::kPlanOffset);
    suffix_totals<D, C::kThreads>(suffix, plan);
    prefix_row_tiles<C::kThreads>(p, G, units_per_tile, start, pairs);
    const int key_tiles = (p.keys + C::kTile - 1) / C::kTile;
    long long weights;
    int longest;
    suffix_read_totals<C::kThreads>(plan, weights, longest);
    const int share = prefix_share(start[p.H_kv], pairs[p.H_kv], key_tiles, weights, D / 64,
                                   (int)gridDim.x);
    PrefixCut wk;
    wk.plan(start, pairs, p.H_kv, (unsigned)key_tiles, (unsigned)share, blockIdx.x);
    if (blockIdx.x >= wk.used) {
        // ------------------------------------------------------------ rows' own keys
        if (warp >= Suffix::kWorkers) return;
        const int blocks = (int)(gridDim.x - wk.used);
        // neighbouring workers on different SMs, so that a small call uses them all
        const int worker = warp * blocks + (int)(blockIdx.x - wk.used);
        SuffixWalk walk;
        if (suffix_plan<D>(suffix, weights, longest, blocks * Suffix::kWorkers, worker, walk))
            suffix_worker<T, D, kNT>(
                suffix, ts_k, ts_v, walk, worker, smem + warp * Suffix::kRingBytes,
                reinterpret_cast<uint64_t *>(smem + C::kSuffixBarOffset) + warp * Suffix::kStages,
                abort_flag);
        return;
    }
    // ---------------------------------------------------------------- the shared keys
    if (warp == 1) {
        tmem_alloc(reinterpret_cast<uint32_t *>(smem + C::kCtlOffset) + 2, C::kTmemCols);
        tmem_relinquish();
        tc_fence_before_sync();
    }
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = (uint32_t)ctl[2];
    PrefixRun run;

    // waits give up together: the first that runs out raises the abort flag
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (mbar_wait(bar, parity)) return true;
        atomicOr(&g_sha_status, kStatusTimeout);
        *abort_flag = 1;
        return false;
    };
    auto wait_warp = [&](uint64_t *bar, uint32_t parity) {      // by a whole warp, agreed
        return (bool)__all_sync(0xffffffffu, wait(bar, parity));
    };
    if (warp == 0 || warp == 3) {
        // -------------------------------------------------------- loads
        // every call reads the prefix again: the L2's default policy may keep it
        uint64_t policy;
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
        const bool is_k = warp == 0;
        const CUtensorMap *map = is_k ? &tm_k : &tm_v;
        uint32_t base = 0;
        const int box_rows = min(p.page_size, C::kTile);
        // a tile's pages, one per lane (at most 16), looked up a tile ahead
        auto page_of = [&](int tile) {
            const int key = tile * C::kTile + lane * box_rows;
            return lane * box_rows < C::kTile && key < p.keys ? p.table[key / p.page_size] : 0;
        };
        bool ok = true;
        while (ok && wk.next(run)) {
            int next = page_of(run.first);
            for (int i = 0; i < run.n; ++i) {
                const int tile = run.first + i;
                int page = next;
                if (i + 1 < run.n) next = page_of(tile + 1);
                const uint32_t pos = base + (is_k ? prefix_k_pos(i) : prefix_v_pos(i, run.n));
                const int buf = (int)(pos % C::kBufs);
                const uint32_t parity = (pos / C::kBufs) & 1u;
                if (lane == 0) ok = wait(&empty[buf], parity ^ 1);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const int rows = min(C::kTile, p.keys - tile * C::kTile);
                const int chunks = (rows + box_rows - 1) / box_rows;
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[buf],
                                          (uint32_t)(chunks * box_rows / 8 * C::kGroupBytes));
                __syncwarp();
                if (lane < chunks) {
                    if ((unsigned)page >= (unsigned)p.num_pages) {
                        atomicOr(&g_sha_status, kStatusBadIndex);
                        page = 0;                       // stay inside the pool
                    }
                    const int off = (tile * C::kTile + lane * box_rows) % p.page_size;
                    tma_load_groups(
                        smem + buf * C::kTileBytes + lane * box_rows / 8 * C::kGroupBytes, map,
                        off >> 3, page * p.H_kv + run.head, &full[buf], policy);
                }
                if (lane == 0) last_load[buf] = (int)pos;
            }
            base += 2 * run.n;
        }
        // the copies still in flight after a wait that gave up: the last one of every
        // buffer, whichever warp issued it (a buffer's phases alternate: one that has
        // gone through two since cannot be told from one that has gone through none)
        named_barrier(4, 64);
        if (is_k && lane == 0)
            for (int s = 0; s < C::kBufs; ++s)
                if (last_load[s] >= 0)
                    mbar_wait_drain(&full[s], ((uint32_t)last_load[s] / C::kBufs) & 1u);
        __syncwarp();
    } else if (warp <= 2) {
        // -------------------------------------------------------- products
        // (the whole warp runs this, and one lane of it issues: see elect_one)
        const int st = warp - 1;
        const uint32_t leader = elect_one();
        uint32_t base = 0, q_parity = 0, s_parity = 0, p_parity = 0;
        // a descriptor's address field counts 16-byte units: tiles and k-steps add to
        // the whole
        const uint64_t q_desc = umma_desc_k_sw128(smem_addr(smem + C::kQOffset));
        const uint64_t k_desc = umma_desc_k_sw128(smem_addr(smem), C::kGroupBytes);
        const uint64_t v_desc = umma_desc_mn_sw128(smem_addr(smem), 1024, C::kGroupBytes);
        constexpr uint32_t kHalf = C::kStep / 8 * C::kGroupBytes >> 4;     // 64 keys
        const uint32_t s_at = tmem + st * C::kStep, o_at = tmem + C::kTmemO + st * D;
        const uint32_t p_at = tmem + C::kTmemP + st * (C::kStep / 2);
        bool ok = true;
        while (ok && wk.next(run)) {
            const int n = run.n;
            ok = wait_warp(q_full, q_parity);
            q_parity ^= 1;
            if (!ok) break;
            tc_fence_after_sync();
            const bool pair = __any_sync(0xffffffffu, *paired != 0);
            if (lane == 0) mbar_arrive(q_seen);
            const PrefixSteps steps(pair, n, p.keys - (run.first + n - 1) * C::kTile);
            const int count = steps.count(st);
            const uint64_t qd = q_desc + (pair ? st : 0) * (C::kQBytes >> 4);
            // S of a step; this stream's last one of a tile gives up its K
            auto scores = [&](int step) {
                const uint32_t pos = base + prefix_k_pos(steps.tile(step));
                const uint32_t buf = pos % C::kBufs;
                if (!wait_warp(&full[buf], (pos / C::kBufs) & 1u)) return false;
                const uint64_t kd = k_desc + buf * (C::kTileBytes >> 4) +
                                    (uint32_t)steps.half(st, step) * kHalf;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    umma_f16_elected(leader, s_at,
                                     qd + (ks >> 2) * (Tile::kBoxBytes >> 4) + (ks & 3) * 2,
                                     kd + (ks >> 2) * (1024 >> 4) + (ks & 3) * 2, kIdescS, ks > 0);
                }
                umma_commit_elected(leader, &s_full[st]);
                if (steps.last_of_tile(st, step)) umma_commit_elected(leader, &empty[buf]);
                return true;
            };
            if (count > 0) ok = scores(0);
            for (int step = 0; ok && step < count; ++step) {
                // S has been read: the next step's may take its place
                if (step + 1 < count) {
                    ok = wait_warp(&s_free[st], s_parity);
                    tc_fence_after_sync();
                    ok = ok && scores(step + 1);
                }
                s_parity ^= 1;
                // O += P V; this stream's last one of a tile gives up its V
                const uint32_t pos = base + prefix_v_pos(steps.tile(step), n);
                const uint32_t buf = pos % C::kBufs;
                ok = ok && wait_warp(&full[buf], (pos / C::kBufs) & 1u);
                ok = ok && wait_warp(&p_full[st], p_parity);
                p_parity ^= 1;
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t vd = v_desc + buf * (C::kTileBytes >> 4) +
                                    (uint32_t)steps.half(st, step) * kHalf;
#pragma unroll
                for (int ks = 0; ks < C::kStep / 16; ++ks)
                    umma_f16_tmem_a_elected(leader, o_at, p_at + ks * 8,
                                            vd + ks * (2 * C::kGroupBytes >> 4),
                                            kIdescO, ks > 0 ? 1u : step > 0);
                umma_commit_elected(leader, &pv_done[st]);
                if (steps.last_of_tile(st, step)) umma_commit_elected(leader, &empty[buf]);
            }
            // A tile without this stream: it gives up K and V of it, too, but only once they
            // have arrived, and behind its own products.  (Given up before, this would count
            // for the tile that the buffer still holds, in place of the other stream's; given
            // up by a plain arrival, it could overtake this stream's last P V, and a load two
            // rounds of the ring ahead would take that one's buffer for free.)
            if (!steps.takes_last(st)) {
                const uint32_t k_at = base + prefix_k_pos(n - 1);
                const uint32_t v_at = base + prefix_v_pos(n - 1, n);
                ok = ok && wait_warp(&full[k_at % C::kBufs], (k_at / C::kBufs) & 1u);
                if (ok) umma_commit_elected(leader, &empty[k_at % C::kBufs]);
                ok = ok && wait_warp(&full[v_at % C::kBufs], (v_at / C::kBufs) & 1u);
                if (ok) umma_commit_elected(leader, &empty[v_at % C::kBufs]);
            }
            base += 2 * n;
        }
        umma_commit_elected(leader, &drain[st]);           // before tensor memory is freed
        __syncwarp();
        mbar_wait_drain(&drain[st], 0);
        __syncwarp();
    } else if (warp >= C::kSoftmaxWarp) {
        // -------------------------------------------------------- softmax
        const unsigned FULL = 0xffffffffu;
        const int stid = tid - 32 * C::kSoftmaxWarp;     // 0 .. 255
        const int swarp = warp - C::kSoftmaxWarp;
        const int st = swarp >> 2;
        const int row = (swarp & 3) * 32 + lane;         // of the stream: this thread's TMEM lane
        const uint32_t lanes = (uint32_t)((swarp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + st * C::kStep;
        const uint32_t p_at = tmem + lanes + C::kTmemP + st * (C::kStep / 2);
        const uint32_t o_at = tmem + lanes + C::kTmemO + st * D;
        const float scale = fabsf(p.scale_log2);
        const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;   // -q instead of -scale
        uint32_t s_parity = 0, pv_parity = 0;
        int runs = 0;
        if (st == 1) named_barrier_arrive(2, C::kSoftmax);      // stream 0 has the first turn
        uint32_t base = 0;
        bool ok = true;
        while (wk.next(run)) {
            const int rt = run.row_tile;
            const int h = run.head;
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

            // (a stream without a step in the last run may only now begin it)
            if (runs > 0 && ok) ok = __all_sync(FULL, wait(q_seen, (uint32_t)(runs - 1) & 1u));
            ++runs;
            // the queries, swizzled like a key tile; the last 32 rows are filled up
            // with zeros, and what lies behind them is nobody's
            if (stid < n_rows) {
                const int e = stid / G, u = unit_list[e];
                q_rows[stid] = (u / p.top_k) * p.H_q + h * G + (stid - e * G);
            }
            named_barrier(1, C::kSoftmax);
            constexpr int kChunks = D / 8, kPass = C::kSoftmax / kChunks, kBatch = 8;
            const int c = stid % kChunks;
            for (int r0 = stid / kChunks; r0 < ((n_rows + 31) & ~31); r0 += kBatch * kPass) {
                uint4 x[kBatch];                          // all on the way before the first is stored
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int r = r0 + i * kPass;
                    x[i] = make_uint4(0, 0, 0, 0);
                    if (r < n_rows)
                        x[i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) +
                                                                (size_t)q_rows[r] * D + c * 8);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int r = r0 + i * kPass, rr = r & (C::kStreamRows - 1);
                    if (r < ((n_rows + 31) & ~31)) {
                        x[i].x ^= flip;
                        x[i].y ^= flip;
                        x[i].z ^= flip;
                        x[i].w ^= flip;
                        *reinterpret_cast<uint4 *>(smem + C::kQOffset + (r >> 7) * C::kQBytes +
                                                   (c >> 3) * Tile::kBoxBytes + rr * 128 +
                                                   (((c & 7) ^ (rr & 7)) << 4)) = x[i];
                    }
                }
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
            const PrefixSteps steps(pair, n, p.keys - (run.first + n - 1) * C::kTile);
            const int count = steps.count(st);
            for (int step = 0; step < count; ++step) {
                if (ok) ok = __all_sync(FULL, wait(&s_full[st], s_parity));
                s_parity ^= 1;
                const int i = steps.tile(step);
                const int rows = min(C::kStep, p.keys - (run.first + i) * C::kTile -
                                                   steps.half(st, step) * C::kStep);
                float s[C::kStep];
                if (ok && busy) {
                    tc_fence_after_sync();
                    tmem_ld32(s_at, reinterpret_cast<float(&)[32]>(s[0]));
                    tmem_ld32(s_at + 32, reinterpret_cast<float(&)[32]>(s[32]));
                    tmem_ld_wait();
                    tc_fence_before_sync();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free[st]);
                if (rows < C::kStep) {
                    // rows past the prefix hold other keys or nothing: zero V there
                    // (0 * NaN) before any product with this step's P.  Both streams
                    // of a pair take the step: they zero half each, and meet.
                    const uint32_t pos = base + prefix_v_pos(i, n);
                    const int buf = (int)(pos % C::kBufs);
                    if (ok) ok = __all_sync(FULL, wait(&full[buf], (pos / C::kBufs) & 1u));
                    if (ok) {
                        unsigned char *vt = smem + buf * C::kTileBytes +
                                            steps.half(st, step) * (C::kStep / 8) * C::kGroupBytes;
                        const int left = (C::kStep - rows) * Tile::kBoxes * 8;
                        for (int e = pair ? stid : stid & 127; e < left; e += pair ? 256 : 128) {
                            const int chunk = e & 7, bx = (e >> 3) % Tile::kBoxes;
                            const int key = rows + (e >> 3) / Tile::kBoxes;
                            *reinterpret_cast<uint4 *>(vt + (key >> 3) * C::kGroupBytes +
                                                       bx * 1024 + (key & 7) * 128 + chunk * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_shared();
                    }
                    if (pair) named_barrier(1, C::kSoftmax);
                }
                float top = 0.f;
                if (ok && busy) {
                    if (rows < C::kStep) {
#pragma unroll
                        for (int e = 0; e < C::kStep; ++e)
                            if (e >= rows) s[e] = -INFINITY;
                    }
                    float tops[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int e = 4; e + 4 < C::kStep; e += 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i)      // (three-operand maxima)
                            tops[i] = fmaxf(fmaxf(tops[i], s[e + i]), s[e + 4 + i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) tops[i] = fmaxf(tops[i], s[C::kStep - 4 + i]);
                    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * scale;
                }
                // the last step's product has read P, and O is up to date (warps without
                // rows wait, too: their arrival for this step must not count for the last)
                if (step > 0) {
                    if (ok) ok = __all_sync(FULL, wait(&pv_done[st], pv_parity));
                    pv_parity ^= 1;
                    tc_fence_after_sync();        // P and O are written next
                }
                if (ok && busy) {
                    // the first step sets the reference, later ones move it rarely
                    const bool move = step == 0 || top > m_ref + (kPrefixSlack<T> + kPrefixLift<T>);
                    if (__any_sync(FULL, move)) {
                        const float m_new = move ? top - kPrefixLift<T> : m_ref;
                        if (step > 0) {
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
                }
                // the streams of a pair take turns at the exponentials: each then has the
                // unit, which they saturate, to itself while the other one reads its next
                // scores (2175 clocks a step against 2360 in step with each other)
                if (pair) named_barrier(2 + st, C::kSoftmax);
                if (ok && busy) {
                    const float m0 = m_ref == -INFINITY ? 0.f : m_ref;
#pragma unroll
                    for (int c = 0; c < C::kStep / 32; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float *x = s + c * 32 + 2 * e;
                            x[0] = exp2_approx(fmaf(x[0], scale, -m0));
                            x[1] = exp2_approx(fmaf(x[1], scale, -m0));
                            if (rows < C::kStep) {       // (scale 0 makes NaN of -inf)
                                if (c * 32 + 2 * e >= rows) x[0] = 0.f;
                                if (c * 32 + 2 * e + 1 >= rows) x[1] = 0.f;
                            }
                            l0 += x[0];
                            l1 += x[1];
                            w[e] = pack2<T>(x[0], x[1]);
                        }
                        tmem_st16(p_at + c * 16, w);
                    }
                }
                if (pair) named_barrier_arrive(3 - st, C::kSoftmax);
                if (ok && busy) tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[st]);
            }

            // this run's partial state: rows of slot rt + block, the second stream's
            // behind the first's (its own rows, or the other half of the keys)
            if (count > 0) {
                if (ok) ok = __all_sync(FULL, wait(&pv_done[st], pv_parity));
                pv_parity ^= 1;
            }
            if (tile_row + lane < n_rows) {
                float *slot = p.parts.slots + (size_t)slot_id * p.parts.slot_floats;
                const int r = st * C::kStreamRows + row;
                *reinterpret_cast<float2 *>(slot + (size_t)C::kRows * D + 2 * r) =
                    make_float2(ok && count > 0 ? m_ref : -INFINITY, l0 + l1);
            }
            if (ok && count > 0 && busy) {
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
                        for (int e = 0; e < 32; e += 8) store8(out + c * 32 + e, o + e);
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

// One output row per D/4 lanes and kWays warps, four elements a lane.  The parts of
// a row go round its warps; each reads its parts' (m, l) one per lane, so that all
// of them, their weights 2^(m - M) and the sum L cost one trip to memory, then the
// lanes add up the weighted O rows, eight loads in flight.  More parts than lanes go
// in rounds, the sums rescaled in between; the warps meet in shared memory.  The
// order is fixed: suffix runs, then prefix runs.  A call of few rows takes kWays =
// 4, for the loads in flight: four of a row's trips to memory become one.
constexpr int kMergeThreads = 256;

template <typename T, int D, int kWays>
__global__ void __launch_bounds__(kMergeThreads) sha_prefix_merge_kernel(const PrefixMergeParams p)
{
    constexpr int kLanes = D / 4;
    constexpr int kRowsPerWarp = 32 / kLanes;
    constexpr int kRowsPerBlock = kMergeThreads / 32 / kWays * kRowsPerWarp;
    __shared__ float4 s_o[kWays > 1 ? kMergeThreads : 1];
    __shared__ float2 s_ml[kWays > 1 ? kMergeThreads / kLanes : 1];
    const unsigned FULL = 0xffffffffu;
    const int G = p.H_q / p.H_kv;
    const int sub = threadIdx.x % kLanes, warp = threadIdx.x >> 5;
    const int way = warp % kWays;
    const int local = warp / kWays * kRowsPerWarp + (threadIdx.x & 31) / kLanes;
    const long long rows = (long long)p.B * p.top_k * G;
    const long long at = (long long)blockIdx.x * kRowsPerBlock + local;
    // (the call's inputs were complete before the first kernel's blocks began)
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
    const int mine = (n - way + kWays - 1) / kWays;      // parts way, way + kWays, ...
    int rounds = (mine + kLanes - 1) / kLanes;
    if (kLanes < 32) rounds = max(rounds, __shfl_xor_sync(FULL, rounds, 16));

    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, L = 0.f;
    for (int r = 0; r < rounds; ++r) {
        // this lane's part: where its row of O is, its (m, l)
        const int i = (r * kLanes + sub) * kWays + way;
        const float *o = nullptr;
        float m = -INFINITY, l = 0.f;
        if (i < run.y) {
            const float *slot = p.slots + (size_t)(run.x + i) * p.slot_floats;
            o = slot + j * D;
            m = __ldcg(slot + G * D + j);
            l = __ldcg(slot + G * D + G + j);
        } else if (i < n) {
            const int k = i - run.y;
            const float *slot =
                p.parts.slots + (size_t)(ref.x + (k >> ref.w)) * p.parts.slot_floats;
            const int row = ref.z + j + (k & ref.w) * (p.parts.slot_rows / 2);
            o = slot + (size_t)row * D;
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(
                slot + (size_t)p.parts.slot_rows * D + 2 * row));
            m = ml.x;
            l = ml.y;
        }
        // the first parts' O on the way beside all (m, l), before their weights are known
        constexpr int kAhead = 4;
        float4 ahead[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const float *ok = reinterpret_cast<const float *>(__shfl_sync(
                FULL, reinterpret_cast<unsigned long long>(o), k, kLanes));
            ahead[k] = ok ? __ldcg(reinterpret_cast<const float4 *>(ok + 4 * sub))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
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
        int parts = min(mine - r * kLanes, kLanes);
        if (kLanes < 32) parts = max(parts, __shfl_xor_sync(FULL, parts, 16));
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const float wk = __shfl_sync(FULL, w, k, kLanes);
            if (wk != 0.f) {                     // (no keys, or nothing left of them)
                O.x = fmaf(wk, ahead[k].x, O.x);
                O.y = fmaf(wk, ahead[k].y, O.y);
                O.z = fmaf(wk, ahead[k].z, O.z);
                O.w = fmaf(wk, ahead[k].w, O.w);
            }
        }
#pragma unroll 8
        for (int k = kAhead; k < parts; ++k) {
            const float wk = __shfl_sync(FULL, w, k, kLanes);
            const float *ok = reinterpret_cast<const float *>(__shfl_sync(
                FULL, reinterpret_cast<unsigned long long>(o), k, kLanes));
            if (wk != 0.f) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(ok + 4 * sub));
                O.x = fmaf(wk, x.x, O.x);
                O.y = fmaf(wk, x.y, O.y);
                O.z = fmaf(wk, x.z, O.z);
                O.w = fmaf(wk, x.w, O.w);
            }
        }
    }
    if constexpr (kWays > 1) {
        s_o[threadIdx.x] = O;
        if (sub == 0) s_ml[threadIdx.x / kLanes] = make_float2(M, L);
        __syncthreads();
        if (way > 0) return;
        float top = M;
#pragma unroll
        for (int v = 1; v < kWays; ++v) top = fmaxf(top, s_ml[threadIdx.x / kLanes + v * kRowsPerWarp].x);
        const float base = top == -INFINITY ? 0.f : top;
        float a = exp2f(M - base);
        O = make_float4(a * O.x, a * O.y, a * O.z, a * O.w);
        L *= a;
#pragma unroll
        for (int v = 1; v < kWays; ++v) {
            const float2 ml = s_ml[threadIdx.x / kLanes + v * kRowsPerWarp];
            const float4 x = s_o[threadIdx.x + 32 * v];
            a = exp2f(ml.x - base);
            O.x = fmaf(a, x.x, O.x);
            O.y = fmaf(a, x.y, O.y);
            O.z = fmaf(a, x.z, O.z);
            O.w = fmaf(a, x.w, O.w);
            L = fmaf(a, ml.y, L);
        }
    }
    if (!live) return;
    T *dst = static_cast<T *>(p.out) + ((size_t)b * p.H_q + (size_t)h * G + j) * D + 4 * sub;
    *reinterpret_cast<uint2 *>(dst) =
        make_uint2(pack2<T>(O.x / L, O.y / L), pack2<T>(O.z / L, O.w / L));
}

}  // namespace sha
