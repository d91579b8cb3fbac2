// sha_rope_kernel.cuh -- rotary positions, and the rotation of new queries and
// keys on their way into a paged cache.
//
// The rotation.  A head's first `rotary` elements form rotary/2 pairs -- element
// i with i + rotary/2 (half layout), or 2i with 2i + 1 (interleaved) -- and pair
// i of the token at position p turns by the angle a = p * inv_freq[i]:
//     y1 = m (x1 cos a - x2 sin a),   y2 = m (x2 cos a + x1 sin a),
// m the long-context factor on cos and sin (1 without one).  The elements past
// `rotary` are copied.  The products and sums are fp32, rounded once to the
// tensor's type.  The angle is not: at position 2^17 an fp32 product p * inv_freq
// is already 2^-8 rad off, as much as a bf16 output's rounding.  So it is formed
// in fp64 in turns, reduced to [-1/2, 1/2] turn there, and only the remainder
// (2^-25 turn off) is rounded for sincospif.
//
// What bounds it.  Two passes' worth of memory traffic (each element read once,
// written once) and, in small calls, launch latency.  A block takes tok_per_block
// tokens and a run of their heads: its first threads compute the tokens' cos and
// sin once into shared memory (one fp64 multiply pair and one sincospif per token
// and pair, shared by all heads), then every thread turns pairs in vectors of P
// (16-byte loads and stores for P = 8), P the largest of 8, 4, 2, 1 that divides
// rotary/2, so a partial or odd rotation keeps the widest aligned access.
//
// Appending.  Token t's K row of head h goes to page
// block_table[row, pos / page_size] of the pool, row pos % page_size; the same
// launch rotates q into its own tensor and copies V, so a decode step touches
// each of the new rows once and pays one launch.
#pragma once

#include "sha_device.cuh"

namespace sha {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 512;          // items of a head row fit the block's threads
constexpr int kRopeMaxAngles = 1024;      // (token, pair) angles of a block, in shared memory
constexpr int kRopeMaxTokens = 64;        // tokens of a block

struct RopeParams {
    // rotated heads: H_a of them from a to a_out, then (append) H_kv from k to k_pages
    const void *a;
    void *a_out;
    long long a_tok, a_head, o_tok, o_head;         // strides, elements
    int H_a;
    const void *k, *v;
    void *k_pages, *v_pages;
    long long k_tok, k_head, v_tok, v_head;
    int H_kv;
    const int32_t *positions, *rows, *block_table;
    const double *inv_freq;
    int T, B, num_pages, page_size, max_pages;
    int d, rotary;
    float mscale;
    int *clear;                  // append: words set to zero for the stream's next kernel,
    int clear_words;             // the arrival counters of a step's decode; or null
    int tok_per_block, heads_per_block, v_per_block;
};

// N 16-bit elements moved as one access (N = 1, 2, 4, 8).
template <int N> struct Vec;
template <> struct Vec<1> { using type = uint16_t; };
template <> struct Vec<2> { using type = uint32_t; };
template <> struct Vec<4> { using type = uint2; };
template <> struct Vec<8> { using type = uint4; };

template <typename T, int N> struct Pack {
    union {
        typename Vec<N>::type raw;
        T e[N];
    };
    __device__ __forceinline__ Pack() {}
    __device__ __forceinline__ void load(const T *p)
    {
        raw = *reinterpret_cast<const typename Vec<N>::type *>(p);
    }
    __device__ __forceinline__ void store(T *p) const
    {
        *reinterpret_cast<typename Vec<N>::type *>(p) = raw;
    }
};

template <typename T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x)
{
    return __bfloat162float(x);
}

// Item `c` of a head row: P pairs turned (c < pairs/P), or a run copied.
template <typename T, int P, bool kInterleaved>
__device__ __forceinline__ void rope_item(const T *src, T *dst, int c, const float2 *cs, int d,
                                          int rotary)
{
    constexpr int kCopy = 2 * P < 8 ? 2 * P : 8;
    const int pairs = rotary >> 1, items = pairs / P;
    if (c >= items) {                              // past the rotated part
        const int e = rotary + (c - items) * kCopy;
        if (src + e == dst + e) return;            // in place
        Pack<T, kCopy> x;
        x.load(src + e);
        x.store(dst + e);
        return;
    }
    const int i = c * P;
    const int e1 = kInterleaved ? 2 * i : i, e2 = kInterleaved ? 2 * i + P : i + pairs;
    Pack<T, P> x, y;                               // both halves, or 2P neighbours
    x.load(src + e1);
    y.load(src + e2);
    float in[2 * P], out[2 * P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        in[j] = to_f32(x.e[j]);
        in[P + j] = to_f32(y.e[j]);
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const float2 w = cs[i + j];
        const int a = kInterleaved ? 2 * j : j, b = kInterleaved ? 2 * j + 1 : P + j;
        out[a] = in[a] * w.x - in[b] * w.y;
        out[b] = in[b] * w.x + in[a] * w.y;
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
        x.e[j] = Elem<T>::from_float(out[j]);
        y.e[j] = Elem<T>::from_float(out[P + j]);
    }
    x.store(dst + e1);
    y.store(dst + e2);
}

// grid: (token groups, head runs).  kAppend: K rows follow the H_a heads in the
// run, V rows are copied, and the tokens' slots in the pool are looked up.
template <typename T, int P, bool kInterleaved, bool kAppend>
__global__ void __launch_bounds__(kRopeThreads) sha_rope_kernel(const RopeParams p)
{
    __shared__ float2 cs[kRopeMaxAngles];
    __shared__ long long slot[kRopeMaxTokens];     // append: row of (page, head 0) in the pool, or -1
    const int tid = threadIdx.x;
    const int pairs = p.rotary >> 1;
    const long long t0 = (long long)blockIdx.x * p.tok_per_block;
    const int toks = (int)(p.T - t0 < p.tok_per_block ? p.T - t0 : p.tok_per_block);

    // positions, tables and the tensors may come from the previous kernel
    pdl_wait();
    pdl_launch_dependents();

    for (int i = tid; i < toks * pairs; i += kRopeThreads) {
        const int t = i / pairs, f = i - t * pairs;
        const double turns = (double)p.positions[t0 + t] * p.inv_freq[f] * 0.15915494309189535;
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        cs[i] = make_float2(c * p.mscale, s * p.mscale);
    }
    if constexpr (kAppend) {
        if (p.clear && blockIdx.x == 0 && blockIdx.y == 0)
            for (int i = tid; i < p.clear_words; i += kRopeThreads) p.clear[i] = 0;
        if (tid < toks) {
            const long long t = t0 + tid;
            const int pos = p.positions[t];
            const long long row = p.rows ? p.rows[t] : t;
            long long at = -1;
            if (pos != -1) {                       // -1: no token here (a padded batch)
                const long long pi = pos / p.page_size;
                bool bad = pos < 0 || row < 0 || row >= p.B || pi >= p.max_pages;
                if (!bad) {
                    const int page = p.block_table[row * p.max_pages + pi];
                    bad = page < 0 || page >= p.num_pages;
                    if (!bad)
                        at = (long long)page * p.H_kv * p.page_size + (pos - pi * p.page_size);
                }
                if (bad) atomicOr(&g_sha_status, kStatusBadIndex);
            }
            slot[tid] = at;
        }
    }
    __syncthreads();

    // rotated rows of this block: heads [h0, h0 + heads) of each token
    constexpr int kCopy = 2 * P < 8 ? 2 * P : 8;
    const int per_row = pairs / P + (p.d - p.rotary) / kCopy;
    const int rot_heads = p.H_a + (kAppend ? p.H_kv : 0);
    const int h0 = blockIdx.y * p.heads_per_block;
    const int heads = min(p.heads_per_block, rot_heads - h0);
    const int lanes = kRopeThreads / per_row;      // rows turned at a time
    const int lane_row = tid / per_row, c = tid - lane_row * per_row;
    if (heads > 0 && lane_row < lanes) {
        for (int r = lane_row; r < toks * heads; r += lanes) {
            const int tt = r / heads, h = h0 + r - tt * heads;
            const long long t = t0 + tt;
            const T *src;
            T *dst;
            if (!kAppend || h < p.H_a) {
                src = static_cast<const T *>(p.a) + t * p.a_tok + h * p.a_head;
                dst = static_cast<T *>(p.a_out) + t * p.o_tok + h * p.o_head;
            } else {
                const int hk = h - p.H_a;
                src = static_cast<const T *>(p.k) + t * p.k_tok + hk * p.k_head;
                dst = static_cast<T *>(p.k_pages) +
                      (slot[tt] + (long long)hk * p.page_size) * p.d;
            }
            if (kAppend && slot[tt] < 0) continue;
            rope_item<T, P, kInterleaved>(src, dst, c, cs + tt * pairs, p.d, p.rotary);
        }
    }
    if constexpr (kAppend) {
        const int v0 = blockIdx.y * p.v_per_block;
        const int vh = min(p.v_per_block, p.H_kv - v0), chunks = p.d / 8;
        for (int i = tid; i < toks * vh * chunks; i += kRopeThreads) {
            const int r = i / chunks, e = (i - r * chunks) * 8;
            const int tt = r / vh, h = v0 + r - tt * vh;
            if (slot[tt] < 0) continue;
            Pack<T, 8> x;
            x.load(static_cast<const T *>(p.v) + (t0 + tt) * p.v_tok + h * p.v_head + e);
            x.store(static_cast<T *>(p.v_pages) + (slot[tt] + (long long)h * p.page_size) * p.d + e);
        }
    }
}

}  // namespace sha
