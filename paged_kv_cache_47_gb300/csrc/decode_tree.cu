// Tree attention (include/pkv_tree.h): list, checks, and the kernel of 32-bit
// caches on the CUDA cores.
//
// A CTA takes its share of tiles of 32 tokens (tree_list.cuh). K and V of a
// tile and the unit's 32 rows of q lie in shared memory as fp32; eight threads
// share a row: four scores each, the row's maximum and sum by shuffles, and
// D / 8 of the row's outputs in registers. It is bound by its instructions and
// shared-memory reads: 64 requests of 512 to 4096 tokens, 16 drafted, 32 q and 8 kv
// heads 2330 us (18 TFLOP/s); one request of 1000 tokens 45 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "device_utils.cuh"
#include "launch_utils.h"
#include "pkv_internal.h"
#include "tree_list.cuh"

namespace {

using pkv::launch_chained;
using pkv::TreeParams;
using pkv::TreePlace;
using pkv::TreeSeq;
using pkv::TreeShare;

constexpr int kTile = 32, kRows = 32, kThreads = 256;
constexpr int kCtasPerSm = 3;

template <int D>
struct Shared {
    static constexpr int kPitch = D + 4;             // rows 16 bytes apart in the banks
    float q[kRows][kPitch], k[kTile][kPitch], v[kTile][kPitch];
    float p[kRows][kTile + 1];
    int prefix[pkv::kTreeMaxSeqs + 1];
    int scan[kThreads / 32];
    pkv::TreeCut cuts[2];
};

__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) tree_simt_kernel(const __grid_constant__ TreeParams p) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared<D> &sh = *reinterpret_cast<Shared<D> *>(raw);
    constexpr int V4 = D / 4, J = D / 32;            // vectors of a row; of a thread's outputs
    const int tid = threadIdx.x, r = tid / 8, e = tid % 8;
    pkv::grid_dependents_launch();
    pkv::grid_dependency_wait();
    TreePlace at;
    const int total = pkv::tree_tiles<kTile, kThreads>(p, sh.prefix, sh.scan);
    const TreeShare share = pkv::tree_share<kTile>(p, sh.prefix, total, blockIdx.x, gridDim.x, at);
    if (tid < 2) sh.cuts[tid].parts = 0;
    const float *kp = static_cast<const float *>(p.k), *vp = static_cast<const float *>(p.v), *qp = static_cast<const float *>(p.q);
    const int B = 1 << p.b.lb;
    for (int left = share.Z - share.A, done = 0; left > 0;) {
        const int count = min(at.tiles - at.i, left), i0 = at.i, P = at.q.L - at.q.n;
        const int chunks = at.units / p.Hk, g = at.u / chunks, r0 = (at.u - g * chunks) * p.RC;
        const int nr = min(p.RC, at.q.n * p.G - r0);
        __syncthreads();                             // (prefix, and the last segment's q)
        for (int x = tid; x < kRows * V4; x += kThreads) {
            const int row = x / V4, c = x - row * V4;
            const float4 z = row < nr ? load4(qp + pkv::tree_row(p, at.q.o, g, r0 + row) * D + 4 * c)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4 *>(&sh.q[row][4 * c]) = z;
        }
        const int token = (r0 + min(r, nr - 1)) / p.G;          // this row's drafted token
        float m = -INFINITY, l = 0.f;
        float4 o[J];
#pragma unroll
        for (int j = 0; j < J; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int t = 0; t < count; ++t) {
            const int t0 = (i0 + t) * kTile;
            __syncthreads();
            for (int x = tid; x < kTile * V4; x += kThreads) {
                const int row = x / V4, c = x - row * V4, pos = t0 + row;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
                if (pos < at.q.L) {
                    const int id = __ldg(p.tables + (int64_t)at.s * p.b.M + (pos >> p.b.lb));
                    if ((unsigned)id < (unsigned)p.NB) {
                        const size_t src = ((((size_t)id * p.Hk + g) << p.b.lb) + (pos & (B - 1))) * D + 4 * c;
                        a = load4(kp + src);
                        b = load4(vp + src);
                    } else {
                        atomicOr(p.b.err, PKV_DEVERR_BLOCK_ID);
                    }
                }
                *reinterpret_cast<float4 *>(&sh.k[row][4 * c]) = a;
                *reinterpret_cast<float4 *>(&sh.v[row][4 * c]) = b;
            }
            __syncthreads();
            // ---- scores of row r, tokens e + 8 i
            float z[4] = {};
            for (int c = 0; c < V4; ++c) {
                const float4 a = *reinterpret_cast<const float4 *>(&sh.q[r][4 * c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 b = *reinterpret_cast<const float4 *>(&sh.k[e + 8 * i][4 * c]);
                    z[i] = fmaf(a.x, b.x, z[i]);
                    z[i] = fmaf(a.y, b.y, z[i]);
                    z[i] = fmaf(a.z, b.z, z[i]);
                    z[i] = fmaf(a.w, b.w, z[i]);
                }
            }
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = t0 + e + 8 * i - P;    // place among the drafted tokens
                bool sees = d < 0;
                if (!sees && d < at.q.n)
                    sees = p.masks ? __ldg(p.masks + (size_t)(at.q.o + token) * p.W + d / 64) >> (d % 64) & 1 : d <= token;
                z[i] = sees ? z[i] * p.scale_log2 : -INFINITY;
                top = fmaxf(top, z[i]);
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            const float nm = fmaxf(m, top), ref = nm == -INFINITY ? 0.f : nm;
            const float f = m == -INFINITY ? 0.f : exp2f(m - ref);
            m = nm;
            l *= f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = exp2f(z[i] - ref);
                l += w;
                sh.p[r][e + 8 * i] = w;
            }
            __syncwarp();
            // ---- outputs 4 e + 32 j of row r; what has no weight is not looked at
#pragma unroll
            for (int j = 0; j < J; ++j) o[j].x *= f, o[j].y *= f, o[j].z *= f, o[j].w *= f;
            for (int c = 0; c < kTile; ++c) {
                const float w = sh.p[r][c];
                if (w == 0.f) continue;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const float4 b = *reinterpret_cast<const float4 *>(&sh.v[c][4 * e + 32 * j]);
                    o[j].x = fmaf(w, b.x, o[j].x);
                    o[j].y = fmaf(w, b.y, o[j].y);
                    o[j].z = fmaf(w, b.z, o[j].z);
                    o[j].w = fmaf(w, b.w, o[j].w);
                }
            }
        }
        // ---- the unit's rows, or a piece of them
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) l += __shfl_xor_sync(~0u, l, d);
        const bool whole = count == at.tiles;
        const float inv = l == 0.f ? 0.f : 1.f / l, lse = l == 0.f ? -INFINITY : m + log2f(l);
        if (r < nr) {
            const size_t row = whole ? pkv::tree_row(p, at.q.o, g, r0 + r)
                                     : (size_t)(2 * blockIdx.x + (i0 ? 0 : 1)) * p.RC + r;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float x[4] = {o[j].x * inv, o[j].y * inv, o[j].z * inv, o[j].w * inv};
                if (whole) pkv::tree_store<4>(p.out, p.out_dtype, row * D + 4 * e + 32 * j, x);
                else *reinterpret_cast<float4 *>(p.ws_o + row * D + 4 * e + 32 * j) = make_float4(x[0], x[1], x[2], x[3]);
            }
            if (e == 0) {
                if (!whole) p.ws_lse[row] = lse;
                else if (p.lse_out) p.lse_out[row] = lse;
            }
        }
        if (!whole && tid == 0) {
            sh.cuts[i0 ? 0 : 1] = pkv::tree_cut(share, share.A + done - i0, at.tiles, at.q.o, g, r0, nr);
            sh.cuts[i0 ? 0 : 1].due = 1;
        }
        left -= count;
        done += count;
        if (left > 0) at.next_unit<kTile>(p);
    }
    pkv::tree_join_cuts<D, kThreads / 32, 2, 2>(p, sh.cuts);
}

template <int D>
cudaError_t launch_simt(const TreeParams &p, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(tree_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared<D>));
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch_chained(tree_simt_kernel<D>, dim3((unsigned)p.C), kThreads, sizeof(Shared<D>), stream, p);
}

template <int D>
cudaError_t launch(int dtype, const TreeParams &p, cudaStream_t stream) {
    return dtype == PKV_F32   ? launch_simt<D>(p, stream)
           : dtype == PKV_F16 ? pkv::launch_tree_f16(D, p, stream)
                              : pkv::launch_tree_bf16(D, p, stream);
}

// Rows of a unit and workers of a launch.
struct Shape {
    int rows, workers;
};
// Tables of fewer tokens: units of one row tile at most. Two row tiles share each
// tile of K and V, which units of one read again; but their joins are twice as long
// and a CTA has one worker instead of two that fill each other's gaps. 256 and 128
// rows: one request of 1000 tokens with 64 drafted 66 and 46 us, 32 of 512 to 4096
// tokens with 33 to 64 drafted 156 and 137, 8 of 4000 (32 drafted, 8 q heads a kv
// head) 74 and 77, of 8000 107 and 115, of 32000 300 and 345; 32 of 8000 311 and 359.
constexpr int kTwoRowTiles = 4096 + PKV_TREE_MAX_TOKENS;
Shape shape_of(const pkv_cache_desc *c, int Hq, int max_tree, int64_t capacity, int ctas) {
    if (c->dtype == PKV_F32) return {kRows, ctas};
    const int64_t rows = (int64_t)max_tree * (Hq / c->num_kv_heads), one = pkv::kTreeMmaRows;
    const int64_t most = capacity > kTwoRowTiles ? 2 * one : one;
    // (one row tile: two workers a CTA, at most 2 PKV_MAX_DECODE_CTAS counters)
    return {(int)(rows < most ? rows : most), rows > one && most > one ? ctas : 2 * ctas};
}
pkv_status ctas_of(const pkv_cache_desc *c, int *ctas) {
    if (*ctas) return PKV_OK;
    const pkv_status st = pkv::device_sm_count(ctas);
    if (st != PKV_OK) return st;
    if (c->dtype == PKV_F32) *ctas *= kCtasPerSm;
    if (*ctas > PKV_MAX_DECODE_CTAS) *ctas = PKV_MAX_DECODE_CTAS;
    return PKV_OK;
}

// workspace: counters (a fixed region, whatever the launch), then [workers][2]
// pieces of rows and their denominators; as much for one worker of two row tiles as
// for two of one, as it does not depend on the table's width
constexpr size_t kCounterBytes = 2 * PKV_MAX_DECODE_CTAS * sizeof(unsigned);
size_t workspace_for(const pkv_cache_desc *c, int Hq, int max_tree, int ctas) {
    const Shape s = shape_of(c, Hq, max_tree, 0, ctas);
    return kCounterBytes + (size_t)s.workers * 2 * s.rows * (c->head_dim + 1) * sizeof(float);
}

pkv_status check_shape(const pkv_cache_desc *cache, int Hq, int max_tree, int ctas) {
    pkv_status st = pkv::check_cache_desc(cache);
    if (st != PKV_OK) return st;
    if (Hq < 1 || Hq % cache->num_kv_heads)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_q_heads %d is not a positive multiple of num_kv_heads %d", Hq,
                                   cache->num_kv_heads);
    if (Hq / cache->num_kv_heads > 4096)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "%d q heads for a kv head (at most 4096)", Hq / cache->num_kv_heads);
    if (max_tree < 1 || max_tree > PKV_TREE_MAX_TOKENS)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "max_tree %d (1..%d)", max_tree, PKV_TREE_MAX_TOKENS);
    if (ctas < 0 || ctas > PKV_MAX_DECODE_CTAS)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_ctas %d outside [0, %d]", ctas, PKV_MAX_DECODE_CTAS);
    return PKV_OK;
}

bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

}  // namespace

extern "C" {

size_t pkv_decode_tree_workspace_bytes(const pkv_cache_desc *cache, int32_t num_q_heads,
                                       int32_t max_tree, int32_t num_ctas) {
    if (check_shape(cache, num_q_heads, max_tree, num_ctas) != PKV_OK) return 0;
    int ctas = num_ctas;
    if (ctas_of(cache, &ctas) != PKV_OK) return 0;
    return workspace_for(cache, num_q_heads, max_tree, ctas);
}

pkv_status pkv_decode_attention_tree(const pkv_cache_desc *cache, const void *q,
                                     int32_t num_tokens, int32_t num_q_heads, const void *k_pool,
                                     const void *v_pool, const int32_t *block_tables,
                                     int32_t num_seqs, int32_t max_blocks_per_seq,
                                     const int32_t *context_lens, const int32_t *token_offsets,
                                     const uint64_t *masks, int32_t mask_words, int32_t max_tree,
                                     float scale, void *out, int32_t out_dtype, void *workspace,
                                     size_t workspace_bytes, void *stream,
                                     const pkv_tree_options *options) {
    const int asked = options ? options->num_ctas : 0, M = max_blocks_per_seq;
    pkv_status st = check_shape(cache, num_q_heads, max_tree, asked);
    if (st != PKV_OK) return st;
    if (num_seqs < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_seqs %d", num_seqs);
    if (num_tokens < 0) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "num_tokens %d", num_tokens);
    if (out_dtype != PKV_F32 && out_dtype != PKV_F16 && out_dtype != PKV_BF16)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "out_dtype %d", out_dtype);
    if (M < 1) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "max_blocks_per_seq %d", M);
    if (!isfinite(scale)) return pkv::set_last_error(PKV_ERR_INVALID_ARG, "scale is not finite");
    if (masks && (mask_words < 1 || mask_words > PKV_TREE_MAX_TOKENS / 64))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "mask_words %d (1..%d)", mask_words, PKV_TREE_MAX_TOKENS / 64);
    if (masks && max_tree > 64 * mask_words)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "max_tree %d above the masks' %d", max_tree, 64 * mask_words);
    if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
    if (!q || !k_pool || !v_pool || !block_tables || !context_lens || !token_offsets || !out)
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "a pointer argument is NULL");
    const int D = cache->head_dim, Hk = cache->num_kv_heads;
    if (misaligned(q, 16) || misaligned(k_pool, 16) || misaligned(v_pool, 16) || misaligned(out, 32) ||
        misaligned(block_tables, 4) || misaligned(context_lens, 4) || misaligned(token_offsets, 4) ||
        misaligned(masks, 8) || (options && misaligned(options->lse_out, 4)))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG,
                                   "q and the pools must be 16-byte aligned, out 32-byte aligned, the others to their elements");
    const int64_t capacity = (int64_t)M * cache->block_size;
    const int G = num_q_heads / Hk, RC = shape_of(cache, num_q_heads, max_tree, capacity, 1).rows;
    const int tile = cache->dtype == PKV_F32 ? kTile : pkv::kTreeMmaTile;
    // the list's places fit 32 bits
    const int64_t seqs = num_seqs < pkv::kTreeMaxSeqs ? num_seqs : pkv::kTreeMaxSeqs;
    const int64_t units = (int64_t)Hk * (((int64_t)max_tree * G + RC - 1) / RC);
    if (capacity > INT32_MAX / 2 || seqs * units * ((capacity + tile - 1) / tile) >= (int64_t)INT32_MAX)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "batch x context too large for one launch");
    if ((int64_t)cache->num_blocks * Hk > INT32_MAX)
        return pkv::set_last_error(PKV_ERR_UNSUPPORTED, "num_blocks * num_kv_heads is 2^31 or more");
    int ctas = asked;
    if ((st = ctas_of(cache, &ctas)) != PKV_OK) return st;
    const size_t need = workspace_for(cache, num_q_heads, max_tree, ctas);
    if (!workspace || workspace_bytes < need)
        return pkv::set_last_error(PKV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                                   workspace ? workspace_bytes : (size_t)0);
    if (misaligned(workspace, 32))
        return pkv::set_last_error(PKV_ERR_INVALID_ARG, "workspace must be 32-byte aligned");
    TreeParams p = {};
    if ((st = pkv::device_error_word(&p.b.err)) != PKV_OK) return st;
    if (cache->dtype != PKV_F32) pkv::next_wait_fault(&p.wait_ns, &p.drop_arrival);
    p.b.T = num_tokens;
    p.b.N = max_tree;
    p.b.M = M;
    p.b.lb = cache->block_size == 8 ? 3 : cache->block_size == 16 ? 4 : 5;
    p.b.cap = (int)capacity;
    p.masks = masks;
    p.W = masks ? mask_words : 0;
    p.q = q;
    p.k = k_pool;
    p.v = v_pool;
    p.out = out;
    p.lse_out = options ? options->lse_out : nullptr;
    p.out_dtype = out_dtype;
    p.NB = cache->num_blocks;
    p.Hk = Hk;
    p.Hq = num_q_heads;
    p.G = G;
    p.RC = RC;
    p.C = shape_of(cache, num_q_heads, max_tree, capacity, ctas).workers;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.count = static_cast<unsigned *>(workspace);
    p.ws_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kCounterBytes);
    p.ws_lse = p.ws_o + (size_t)p.C * 2 * RC * D;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (int s0 = 0; s0 < num_seqs; s0 += pkv::kTreeMaxSeqs) {
        p.S = num_seqs - s0 < pkv::kTreeMaxSeqs ? num_seqs - s0 : pkv::kTreeMaxSeqs;
        p.b.offs = token_offsets + s0;
        p.b.lens = context_lens + s0;
        p.tables = block_tables + (size_t)s0 * M;
        const cudaError_t e = D == 128 ? launch<128>(cache->dtype, p, s) : launch<64>(cache->dtype, p, s);
        if (e != cudaSuccess)
            return pkv::set_last_error(PKV_ERR_CUDA, "decode_tree launch: %s", cudaGetErrorString(e));
    }
    return PKV_OK;
}

}  // extern "C"
