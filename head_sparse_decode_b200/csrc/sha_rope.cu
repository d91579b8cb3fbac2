// sha_rope.cu -- C ABI of the rotary positions and of appending to a paged
// cache: argument checks, the block shape and the launches.  The operations
// and every argument are specified in include/sha_decode.h.
#include <cmath>

#include "sha_decode.h"
#include "sha_rope_kernel.cuh"

sha_status_t sha_launch_failed(cudaError_t e);   // sha_decode.cu: keeps the error's name

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Elements of the pair vectors (sha_rope_kernel.cuh): the widest that divides
// the pairs, so that both halves of a pair vector stay aligned.
int pairs_per_item(int rotary)
{
    const int pairs = rotary / 2;
    return pairs % 8 == 0 ? 8 : pairs % 4 == 0 ? 4 : pairs % 2 == 0 ? 2 : 1;
}

// Tokens and heads of a block.  A block of a rotation wants about four items a
// thread, so that its angles are shared by many heads (8192 x 64 x 128 bf16: 46.0
// us, with 2 or 9 a thread 48.0 or 47.1).  Appending wants sixteen: its tokens'
// slots take three dependent loads, which more tokens a block go through together
// (6001 tokens of 64 + 8 + 8 heads: 44.5 us, with four a thread 55.1).  A call that
// then has fewer blocks than the device has SMs takes smaller blocks, each repeating
// its tokens' angles, since it is latency that bounds it.
constexpr long long kWantBlocks = 148;
constexpr int kRopeItems = 4, kAppendItems = 16;

void block_shape(sha::RopeParams &p, bool append, int &grid_x, int &grid_y)
{
    const int P = pairs_per_item(p.rotary);
    const int copy = 2 * P < 8 ? 2 * P : 8;
    const int per_row = p.rotary / 2 / P + (p.d - p.rotary) / copy;
    const int heads = p.H_a + (append ? p.H_kv : 0);
    const int lanes = sha::kRopeThreads / per_row;            // rows a pass
    int rows = lanes * (append ? kAppendItems : kRopeItems);
    while (rows > lanes && ((long long)p.T * heads + rows - 1) / rows < kWantBlocks) rows -= lanes;
    int hpb = heads < rows ? heads : rows;
    int runs = (heads + hpb - 1) / hpb;
    hpb = (heads + runs - 1) / runs;
    int toks = rows / hpb;
    if (p.rotary > 0 && toks > sha::kRopeMaxAngles / (p.rotary / 2))
        toks = sha::kRopeMaxAngles / (p.rotary / 2);
    if (toks > sha::kRopeMaxTokens) toks = sha::kRopeMaxTokens;
    if (toks > p.T) toks = p.T;
    if (toks < 1) toks = 1;
    p.tok_per_block = toks;
    p.heads_per_block = hpb;
    p.v_per_block = append ? (p.H_kv + runs - 1) / runs : 0;
    grid_x = (int)(((long long)p.T + toks - 1) / toks);
    grid_y = runs;
}

template <typename T, int P, bool kInterleaved, bool kAppend>
cudaError_t launch(const sha::RopeParams &p, int gx, int gy, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(gx, gy);
    cfg.blockDim = dim3(sha::kRopeThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sha::sha_rope_kernel<T, P, kInterleaved, kAppend>, p);
}

template <typename T, int P>
cudaError_t launch_p(const sha::RopeParams &p, bool interleaved, bool append, int gx, int gy,
                     cudaStream_t s)
{
    if (append)
        return interleaved ? launch<T, P, true, true>(p, gx, gy, s)
                           : launch<T, P, false, true>(p, gx, gy, s);
    return interleaved ? launch<T, P, true, false>(p, gx, gy, s)
                       : launch<T, P, false, false>(p, gx, gy, s);
}

template <typename T>
sha_status_t run(sha::RopeParams &p, bool interleaved, bool append, cudaStream_t s)
{
    int gx, gy;
    block_shape(p, append, gx, gy);
    if (gy > 65535) return SHA_ERR_UNSUPPORTED;
    cudaError_t e;
    switch (pairs_per_item(p.rotary)) {
    case 8: e = launch_p<T, 8>(p, interleaved, append, gx, gy, s); break;
    case 4: e = launch_p<T, 4>(p, interleaved, append, gx, gy, s); break;
    case 2: e = launch_p<T, 2>(p, interleaved, append, gx, gy, s); break;
    default: e = launch_p<T, 1>(p, interleaved, append, gx, gy, s); break;
    }
    return e == cudaSuccess ? SHA_OK : sha_launch_failed(e);
}

// Checks shared by both entry points: the rotation and the head dim.
sha_status_t check_rotation(int T, int d, int rotary, int interleaved, float mscale,
                            sha_dtype_t dtype)
{
    if (dtype != SHA_FP16 && dtype != SHA_BF16) return SHA_ERR_UNSUPPORTED;
    if (T < 0 || d < 1 || (interleaved != 0 && interleaved != 1)) return SHA_ERR_INVALID_ARG;
    if (rotary < 0 || rotary > d || rotary % 2 != 0) return SHA_ERR_INVALID_ARG;
    if (!std::isfinite(mscale)) return SHA_ERR_INVALID_ARG;
    if (d % 8 != 0 || d > sha::kRopeMaxDim) return SHA_ERR_UNSUPPORTED;
    return SHA_OK;
}

// Whether rows of d elements at a * s0 + b * s1 (a < n0, b < n1; s0, s1 >= d) are all
// apart: at once where one dimension's extent fits the other's stride, else by the
// nearest two rows for every difference along the shorter dimension.
bool rows_lie_apart(int64_t s0, int64_t n0, int64_t s1, int64_t n1, int64_t d)
{
    const auto fits = [&](int64_t big, int64_t small, int64_t n) {
        return small <= (big - d) / (n - 1);                  // small * (n - 1) + d <= big
    };
    if (fits(s0, s1, n1) || fits(s1, s0, n0)) return true;
    if (n0 > n1) {
        const int64_t s = s0, n = n0;
        s0 = s1;
        n0 = n1;
        s1 = s;
        n1 = n;
    }
    for (int64_t a = 1; a < n0; ++a) {
        if (s0 > INT64_MAX / a) break;                        // past any address
        const int64_t b = a * s0 / s1, left = a * s0 - b * s1;
        if (b < n1 && left < d) return false;
        if (b + 1 < n1 && s1 - left < d) return false;
    }
    return true;
}

// A [T, H, d] view: strides of dimensions longer than one are checked, and that the
// rows of one that is written lie apart.
sha_status_t check_view(const int64_t strides[2], int T, int H, int d, bool written)
{
    for (int i = 0; i < 2; ++i) {
        if ((i == 0 ? T : H) <= 1) continue;
        if (strides[i] < 0) return SHA_ERR_INVALID_ARG;
        if (strides[i] % 8 != 0) return SHA_ERR_MISALIGNED;
        if (written && strides[i] < d) return SHA_ERR_INVALID_ARG;
    }
    if (written && T > 1 && H > 1 && !rows_lie_apart(strides[0], T, strides[1], H, d))
        return SHA_ERR_INVALID_ARG;
    return SHA_OK;
}

}  // namespace

unsigned sha_rope_take_status()
{
    unsigned flags = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&flags, sha::g_sha_status, sizeof flags) == cudaSuccess && flags)
        cudaMemcpyToSymbol(sha::g_sha_status, &zero, sizeof zero);
    return flags;
}

extern "C" sha_status_t sha_rope(const void *x, const int32_t *positions, const double *inv_freq,
                                 int T, int H, int d, int rotary, int interleaved, float mscale,
                                 const int64_t x_strides[2], void *out,
                                 const int64_t out_strides[2], sha_dtype_t dtype, void *stream)
{
    sha_status_t st = check_rotation(T, d, rotary, interleaved, mscale, dtype);
    if (st != SHA_OK) return st;
    if (H < 0 || rotary < 2) return SHA_ERR_INVALID_ARG;
    if (T == 0 || H == 0) return SHA_OK;
    if (!x || !out || !positions || !inv_freq || !x_strides || !out_strides)
        return SHA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(positions, 4) || !aligned(inv_freq, 8))
        return SHA_ERR_MISALIGNED;
    st = check_view(x_strides, T, H, d, false);
    if (st == SHA_OK) st = check_view(out_strides, T, H, d, true);
    if (st != SHA_OK) return st;
    sha::RopeParams p = {};
    p.a = x;
    p.a_out = out;
    p.a_tok = x_strides[0];
    p.a_head = x_strides[1];
    p.o_tok = out_strides[0];
    p.o_head = out_strides[1];
    p.H_a = H;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.T = T;
    p.d = d;
    p.rotary = rotary;
    p.mscale = mscale;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SHA_FP16 ? run<__half>(p, interleaved, false, s)
                             : run<__nv_bfloat16>(p, interleaved, false, s);
}

// sha_append_paged, or (launch false) its checks alone: a step that appends and then
// decodes launches nothing unless both calls' arguments hold.  clear: words that the
// launch sets to zero, too (RopeParams::clear).
sha_status_t sha_append_call(
    const void *k, const void *v, const int64_t k_strides[2], const int64_t v_strides[2], int T,
    int H_kv, int d, void *k_pages, void *v_pages, const int32_t *block_table,
    const int32_t *rows, const int32_t *positions, int B, int num_pages, int page_size,
    int max_pages, const double *inv_freq, int rotary, int interleaved, float mscale,
    const void *q, const int64_t q_strides[2], int H_q, void *q_out, const int64_t q_out_strides[2],
    sha_dtype_t dtype, void *stream, bool launch, int *clear, int clear_words)
{
    sha_status_t st = check_rotation(T, d, rotary, interleaved, mscale, dtype);
    if (st != SHA_OK) return st;
    if (H_kv < 1 || H_q < 0 || B < 0 || num_pages < 1 || page_size < 1 || max_pages < 1)
        return SHA_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size > (1 << 30)) return SHA_ERR_INVALID_ARG;
    if (!rows && T > B) return SHA_ERR_INVALID_ARG;         // token t is row t's
    if (rotary == 0 && H_q > 0) return SHA_ERR_INVALID_ARG; // nothing to do to q
    if (T == 0) return SHA_OK;
    if (!k || !v || !k_strides || !v_strides || !k_pages || !v_pages || !block_table || !positions ||
        (rotary > 0 && !inv_freq) || (H_q > 0 && (!q || !q_out || !q_strides || !q_out_strides)))
        return SHA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
        !aligned(block_table, 4) || !aligned(positions, 4) || (rows && !aligned(rows, 4)) ||
        (rotary > 0 && !aligned(inv_freq, 8)) ||
        (H_q > 0 && (!aligned(q, 16) || !aligned(q_out, 16))))
        return SHA_ERR_MISALIGNED;
    st = check_view(k_strides, T, H_kv, d, false);
    if (st == SHA_OK) st = check_view(v_strides, T, H_kv, d, false);
    if (st == SHA_OK && H_q > 0) st = check_view(q_strides, T, H_q, d, false);
    if (st == SHA_OK && H_q > 0) st = check_view(q_out_strides, T, H_q, d, true);
    if (st != SHA_OK || !launch) return st;
    sha::RopeParams p = {};
    if (H_q > 0) {
        p.a = q;
        p.a_out = q_out;
        p.a_tok = q_strides[0];
        p.a_head = q_strides[1];
        p.o_tok = q_out_strides[0];
        p.o_head = q_out_strides[1];
    }
    p.H_a = H_q;
    p.k = k;
    p.v = v;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_tok = k_strides[0];
    p.k_head = k_strides[1];
    p.v_tok = v_strides[0];
    p.v_head = v_strides[1];
    p.H_kv = H_kv;
    p.positions = positions;
    p.rows = rows;
    p.block_table = block_table;
    p.inv_freq = inv_freq;
    p.T = T;
    p.B = B;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.d = d;
    p.rotary = rotary;
    p.mscale = mscale;
    p.clear = clear;
    p.clear_words = clear_words;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SHA_FP16 ? run<__half>(p, interleaved, true, s)
                             : run<__nv_bfloat16>(p, interleaved, true, s);
}

extern "C" sha_status_t sha_append_paged(
    const void *k, const void *v, const int64_t k_strides[2], const int64_t v_strides[2], int T,
    int H_kv, int d, void *k_pages, void *v_pages, const int32_t *block_table,
    const int32_t *rows, const int32_t *positions, int B, int num_pages, int page_size,
    int max_pages, const double *inv_freq, int rotary, int interleaved, float mscale,
    const void *q, const int64_t q_strides[2], int H_q, void *q_out, const int64_t q_out_strides[2],
    sha_dtype_t dtype, void *stream)
{
    return sha_append_call(k, v, k_strides, v_strides, T, H_kv, d, k_pages, v_pages, block_table,
                           rows, positions, B, num_pages, page_size, max_pages, inv_freq, rotary,
                           interleaved, mscale, q, q_strides, H_q, q_out, q_out_strides, dtype,
                           stream, true, nullptr, 0);
}

#ifdef SHA_TEST_HOOKS
// Test builds only (not part of the ABI).
extern "C" int sha_test_rows_lie_apart(int64_t s0, int64_t n0, int64_t s1, int64_t n1, int64_t d)
{
    return rows_lie_apart(s0, n0, s1, n1, d);
}
#endif
