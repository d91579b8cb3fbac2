// sha_prefix_kernel.cuh -- the shared-prefix pass of sha_decode_prefix.
//
// When every row of a batch begins with the same P keys, the attention over
// them is, for each KV head h, one dense product: the query rows of all the
// (batch row, slot) units that select h -- R_h of them, G each -- against the
// same K_h, V_h [P, d].  Reading the prefix once per head instead of once per
// unit divides its traffic by R_h (about B * top_k / H_kv).  The softmax over a
// row's whole key range is put together from its two parts by the log-sum-exp
// rule: this kernel leaves (O, m, l) of each query row over [0, P), and the
// suffix pass (sha_gqa_kernel.cuh, kLayoutSuffix) folds them into its own state
// over [P, len) when it finishes the unit.
//
// How the work is cut.  The selection is on the device, so each block plans for
// itself: a histogram of batch_head_index gives every head's units, kUnits =
// kRows / G units make one row tile of kRows query rows, and the row tiles x key
// tiles (of kTile keys) are numbered row-tile-major and cut into equal contiguous
// ranges, one per block, like the key tiles of the other kernels.  A run of key
// tiles within one row tile is one partial state, and the runs, in order, take
// the slots 0, 1, 2, ... : run (row tile r, block c) has slot r + c, since every
// next run advances one of the two or both.
#pragma once

#include <cuda.h>

#include "sha_device.cuh"
#include "sha_gqa_kernel.cuh"
#include "sha_mma.cuh"

namespace sha {

constexpr int kPrefixMaxHeads = 1024;

struct PrefixParams {
    const void *q;
    const int32_t *idx;
    const int32_t *table;        // pages of the shared keys
    int B, H_q, H_kv, top_k;
    int keys;                    // P
    int page_size, num_pages;
    float scale_log2;            // scale * log2(e)
    PrefixParts parts;
    int *counters;               // arrival counters of the suffix pass, cleared here
    int num_counters;
};

template <int D>
struct PrefixConfig {
    using Tile = GqaConfig<D>;                       // key tiles and their swizzle
    static constexpr int kConsumerWarps = 8;
    static constexpr int kConsumers = 32 * kConsumerWarps;
    static constexpr int kThreads = kConsumers + 32;
    static constexpr int kRows = 16 * kConsumerWarps;    // query rows of a row tile
    static constexpr int kTile = Tile::kTile;
    static constexpr int kStages = 3;
    static constexpr int kTileBytes = Tile::kTileBytes;
    static constexpr int kBarOffset = 2 * kStages * kTileBytes;
    static constexpr int kFlagOffset = kBarOffset + 2 * kStages * 8;
    static constexpr int kWarpOffset = kFlagOffset + 16;            // warp counts of the list
    static constexpr int kUnitOffset = kWarpOffset + 4 * 32;        // a row tile's units
    static constexpr int kStartOffset = kUnitOffset + 4 * kRows;    // first row tile of each head
    static constexpr int kSmemBytes = 1024 + kStartOffset + 4 * (kPrefixMaxHeads + 1);
};

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
    for (int u = tid; u < units; u += NT) {
        const int h = p.idx[u];
        if ((unsigned)h < (unsigned)p.H_kv) atomicAdd(&start[h], 1);
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

template <typename T, int D>
__global__ void __launch_bounds__(PrefixConfig<D>::kThreads, 1)
    sha_prefix_kernel(const PrefixParams p, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v)
{
    using C = PrefixConfig<D>;
    using G4 = GqaConfig<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *k_ring = smem;
    unsigned char *v_ring = smem + C::kStages * C::kTileBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOffset);
    uint64_t *empty = full + C::kStages;
    volatile int *flags = reinterpret_cast<volatile int *>(smem + C::kFlagOffset);
    int *warp_counts = reinterpret_cast<int *>(smem + C::kWarpOffset);
    int *unit_list = reinterpret_cast<int *>(smem + C::kUnitOffset);
    int *start = reinterpret_cast<int *>(smem + C::kStartOffset);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int G = p.H_q / p.H_kv;
    const int units_per_tile = C::kRows / G;
    const int units = p.B * p.top_k;

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], C::kConsumerWarps);
        }
        flags[0] = 0;
        mbar_init_fence();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0)
        for (int i = tid; i < p.num_counters; i += C::kThreads) p.counters[i] = 0;

    prefix_row_tiles<C::kThreads>(p, units_per_tile, start);
    const int key_tiles = (p.keys + C::kTile - 1) / C::kTile;
    Schedule S;
    S.tiles_per_unit = key_tiles;                    // a "unit" here is a row tile
    S.total_tiles = (long long)start[p.H_kv] * key_tiles;
    S.pieces = 0;
    if (S.total_tiles == 0) return;
    S.num_ctas = S.total_tiles < gridDim.x ? (int)S.total_tiles : (int)gridDim.x;
    if ((int)blockIdx.x >= S.num_ctas) return;
    UniformWalk wk;
    wk.S = S;
    wk.t = S.begin(blockIdx.x);
    wk.t_end = S.begin(blockIdx.x + 1);
    wk.n_keys = p.keys;
    Seg seg;

    // ------------------------------------------------------------ producer
    if (warp == C::kConsumerWarps) {
        // the prefix is read by few row tiles each, but every call reads it again:
        // the L2's default policy may keep it
        uint64_t policy;
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
        int stage = 0;
        uint32_t phase = 0, last_parity = 0, used = 0;
        bool ok = true;
        const int box_rows = min(p.page_size, C::kTile);
        while (ok && wk.next(seg)) {
            const int h = prefix_head_of(start, p.H_kv, (int)seg.unit);
            for (int j = seg.first_tile; j < seg.first_tile + seg.num_tiles; ++j) {
                bool go = true;
                if (lane == 0) {
                    if (flags[0]) {
                        go = false;
                    } else if (!mbar_wait(&empty[stage], phase ^ 1)) {
                        atomicOr(&g_sha_status, kStatusTimeout);
                        flags[0] = 1;
                        go = false;
                    } else if (flags[0]) {
                        go = false;
                    }
                }
                go = __shfl_sync(0xffffffffu, go, 0);
                if (!go) { ok = false; break; }
                const int n0 = j * C::kTile;
                const int rows = min(C::kTile, p.keys - n0);
                const int chunks = (rows + box_rows - 1) / box_rows;
                if (lane == 0)
                    mbar_arrive_expect_tx(
                        &full[stage], (uint32_t)(2 * chunks * G4::kBoxes * box_rows * 128));
                __syncwarp();
                for (int c = lane; c < chunks; c += 32) {
                    const int key = n0 + c * box_rows;
                    const int pi = key / p.page_size, off = key - pi * p.page_size;
                    int page = p.table[pi];
                    if ((unsigned)page >= (unsigned)p.num_pages) {
                        atomicOr(&g_sha_status, kStatusBadIndex);
                        page = 0;                       // stay inside the pool
                    }
                    const int plane = page * p.H_kv + h;
                    for (int bx = 0; bx < G4::kBoxes; ++bx) {
                        const int at = stage * C::kTileBytes + bx * G4::kBoxBytes + c * box_rows * 128;
                        tma_load_3d(k_ring + at, &tm_k, bx * 64, off, plane, &full[stage], policy);
                        tma_load_3d(v_ring + at, &tm_v, bx * 64, off, plane, &full[stage], policy);
                    }
                }
                last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
                used |= 1u << stage;
                if (++stage == C::kStages) { stage = 0; phase ^= 1; }
            }
        }
        if (lane == 0)
            for (int s = 0; s < C::kStages; ++s)
                if (used & (1u << s)) mbar_wait_drain(&full[s], (last_parity >> s) & 1u);
        __syncwarp();
        return;
    }

    // ------------------------------------------------------------ consumers
    const int g = lane >> 2, qd = lane & 3;
    const unsigned FULL = 0xffffffffu;
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t k_base = smem_addr(k_ring), v_base = smem_addr(v_ring);
    int stage = 0;
    uint32_t phase = 0;
    while (wk.next(seg)) {
        const int rt = (int)seg.unit;
        const int h = prefix_head_of(start, p.H_kv, rt);
        // this row tile's units: those of the head's units, in order, that the
        // tiles before it have not taken
        const int rank0 = (rt - start[h]) * units_per_tile;
        int seen = 0, n_units = 0;
        named_barrier(1, C::kConsumers);              // the last tile's list has been read
        for (int u0 = 0; u0 < units && seen < rank0 + units_per_tile; u0 += C::kConsumers) {
            const int u = u0 + tid;
            const bool hit = u < units && p.idx[u] == h;
            const unsigned votes = __ballot_sync(FULL, hit);
            if (lane == 0) warp_counts[warp] = __popc(votes);
            named_barrier(1, C::kConsumers);
            int before = seen, total = 0;
            for (int w = 0; w < C::kConsumerWarps; ++w) {
                if (w < warp) before += warp_counts[w];
                total += warp_counts[w];
            }
            const int rank = before + __popc(votes & ((1u << lane) - 1)) - rank0;
            if (hit && rank >= 0 && rank < units_per_tile) unit_list[rank] = u;
            seen += total;
            named_barrier(1, C::kConsumers);
        }
        n_units = min(seen - rank0, units_per_tile);
        const int n_rows = n_units * G;
        const int slot_id = rt + (int)blockIdx.x;
        if (seg.first_tile == 0) {
            const int last = S.cta_of(seg.unit_start + key_tiles - 1);
            for (int i = tid; i < n_units; i += C::kConsumers)
                p.parts.ref[unit_list[i]] =
                    make_int4(slot_id, last - (int)blockIdx.x + 1, i * G, 0);
        }

        // Q of this warp's 16 rows as the MMA's A operand (zero past the tile's rows)
        const int row0 = warp * 16;
        const bool busy = row0 < n_rows;
        uint32_t qa[G4::kKSteps][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = row0 + g + 8 * r;
            const T *src = nullptr;
            if (row < n_rows) {
                const int e = row / G, u = unit_list[e];
                src = static_cast<const T *>(p.q) +
                      ((size_t)(u / p.top_k) * p.H_q + (size_t)h * G + (row - e * G)) * D;
            }
#pragma unroll
            for (int ks = 0; ks < G4::kKSteps; ++ks) {
                const int c0 = ks * 16 + qd * 2;
                qa[ks][r] = src ? *reinterpret_cast<const uint32_t *>(src + c0) : 0u;
                qa[ks][2 + r] = src ? *reinterpret_cast<const uint32_t *>(src + c0 + 8) : 0u;
            }
        }
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
        float o[G4::kONTiles][4];
#pragma unroll
        for (int n = 0; n < G4::kONTiles; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

        for (int j = seg.first_tile; j < seg.first_tile + seg.num_tiles; ++j) {
            bool live = !__any_sync(FULL, flags[0] != 0);
            if (live) {
                live = __all_sync(FULL, mbar_wait(&full[stage], phase));
                if (!live && lane == 0) {
                    atomicOr(&g_sha_status, kStatusTimeout);
                    flags[0] = 1;
                }
            }
            const int rows = min(C::kTile, p.keys - j * C::kTile);
            if (live && rows < C::kTile) {
                // rows past the prefix hold other keys or nothing: zero V there (0 * NaN)
                unsigned char *vt = v_ring + stage * C::kTileBytes;
                for (int i = tid; i < (C::kTile - rows) * G4::kBoxes * 8; i += C::kConsumers) {
                    const int chunk = i & 7, bx = (i >> 3) % G4::kBoxes;
                    const int key = rows + (i >> 3) / G4::kBoxes;
                    *reinterpret_cast<uint4 *>(vt + bx * G4::kBoxBytes + key * 128 + chunk * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_shared();           // before the stage is refilled by TMA
            }
            if (rows < C::kTile) named_barrier(1, C::kConsumers);
            if (live && busy) {
                const uint32_t kt = k_base + stage * C::kTileBytes;
                const uint32_t vt = v_base + stage * C::kTileBytes;
                for (int s0 = 0; s0 < C::kTile; s0 += 64) {
                    if (s0 >= rows) break;
                    float s[8][4];
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
                    for (int ks = 0; ks < G4::kKSteps; ++ks)
#pragma unroll
                        for (int np = 0; np < 4; ++np) {
                            uint32_t kb[4];
                            ldmatrix_x4(swizzled<D>(kt, s0 + np * 16 + (mi >> 1) * 8 + mr,
                                                    ks * 2 + (mi & 1)),
                                        kb);
                            mma_16816<T>(s[2 * np], qa[ks], kb[0], kb[1]);
                            mma_16816<T>(s[2 * np + 1], qa[ks], kb[2], kb[3]);
                        }
                    float alpha[2], ref[2], mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = s0 + nt * 8 + qd * 2 + (e & 1);
                            s[nt][e] = key < rows ? s[nt][e] * p.scale_log2 : -INFINITY;
                            mt[e >> 1] = fmaxf(mt[e >> 1], s[nt][e]);
                        }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        mt[r] = fmaxf(mt[r], __shfl_xor_sync(FULL, mt[r], 1));
                        mt[r] = fmaxf(mt[r], __shfl_xor_sync(FULL, mt[r], 2));
                        const float m_new = fmaxf(m_run[r], mt[r]);
                        ref[r] = m_new == -INFINITY ? 0.f : m_new;
                        alpha[r] = exp2f(m_run[r] - ref[r]);
                        m_run[r] = m_new;
                        l_run[r] *= alpha[r];
                    }
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[nt][e] = exp2f(s[nt][e] - ref[e >> 1]);
                            l_run[e >> 1] += s[nt][e];
                        }
#pragma unroll
                    for (int n = 0; n < G4::kONTiles; ++n) {
                        o[n][0] *= alpha[0];
                        o[n][1] *= alpha[0];
                        o[n][2] *= alpha[1];
                        o[n][3] *= alpha[1];
                    }
                    // P rounds to the tensor type, the MMA's operand type; the sums
                    // l and O stay fp32
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        uint32_t pa[4];
                        pa[0] = pack2<T>(s[2 * kk][0], s[2 * kk][1]);
                        pa[1] = pack2<T>(s[2 * kk][2], s[2 * kk][3]);
                        pa[2] = pack2<T>(s[2 * kk + 1][0], s[2 * kk + 1][1]);
                        pa[3] = pack2<T>(s[2 * kk + 1][2], s[2 * kk + 1][3]);
#pragma unroll
                        for (int dn = 0; dn < D / 16; ++dn) {
                            uint32_t vb[4];
                            ldmatrix_x4_trans(swizzled<D>(vt, s0 + kk * 16 + (mi & 1) * 8 + mr,
                                                          dn * 2 + (mi >> 1)),
                                              vb);
                            mma_16816<T>(o[2 * dn], pa, vb[0], vb[1]);
                            mma_16816<T>(o[2 * dn + 1], pa, vb[2], vb[3]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
            if (++stage == C::kStages) { stage = 0; phase ^= 1; }
        }

        // this run's partial state: slot rt + block
        float *slot = p.parts.slots + (size_t)slot_id * p.parts.slot_floats;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l_run[r] += __shfl_xor_sync(FULL, l_run[r], 1);
            l_run[r] += __shfl_xor_sync(FULL, l_run[r], 2);
            const int row = row0 + g + 8 * r;
            if (row < n_rows) {
#pragma unroll
                for (int n = 0; n < G4::kONTiles; ++n)
                    *reinterpret_cast<float2 *>(slot + (size_t)row * D + n * 8 + qd * 2) =
                        make_float2(o[n][2 * r], o[n][2 * r + 1]);
                if (qd == 0)
                    *reinterpret_cast<float2 *>(slot + (size_t)p.parts.slot_rows * D + 2 * row) =
                        make_float2(m_run[r], l_run[r]);
            }
        }
    }
}

}  // namespace sha
