// dfw_embed.cuh -- rows of an embedding table by token id, with scaling, from
// an entropy-coded scope or a bf16 table, and the table's gradient (included
// by dfw_decode.cu only).
//
//   out[t, :] = bf16(scale E[id[t], :]),   zeros where id[t] < 0
//   dE[v, :]  = scale sum over {t : id[t] = v} of dY[t, :]
//
// The coded form is random access into the known-start plan (the LazyWeights
// write-up's lanes with known starts; the DFloat11 abstract's block-level
// decompression, here of a row): group_start gives a group's first bit, a
// prefix sum of chunk_bits each chunk's, so a row's chunks are decoded alone.
#pragma once

#include <cuda_bf16.h>

#include "dfw_lanes.cuh"
#include "dfw_q4.cuh"

namespace dfw {
namespace {

struct IdSource {
    const void *ids;
    uint32_t wide;  // 64-bit ids
    uint32_t tokens;
    uint64_t rows;
};

// Row of token t; false for padding (negative) and for ids past the table,
// which are also reported.
__device__ __forceinline__ bool token_row(const IdSource &s, uint32_t t, uint64_t &row, bool report) {
    const int64_t id = s.wide ? __ldg(static_cast<const long long *>(s.ids) + t)
                              : (int64_t)__ldg(static_cast<const int *>(s.ids) + t);
    if (id < 0) return false;
    if ((uint64_t)id >= s.rows) {
        if (report) atomicOr(&g_status, ST_INDEX);
        return false;
    }
    row = (uint64_t)id;
    return true;
}

// bf16(scale w), rounded to nearest even; scale 1 keeps the bits (NaN
// payloads included), as the decoder does.
__device__ __forceinline__ uint16_t scaled(uint16_t w, float scale, bool one) {
    if (one) return w;
    return __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float((uint32_t)w << 16) * scale));
}

// ------------------------------------------------------- rows of a bf16 table

struct RowsOfTable {
    IdSource ids;
    const uint16_t *table;
    uint16_t *out;
    uint64_t ldt, ldo;
    uint32_t dim;
    float scale;
};

__global__ void __launch_bounds__(256) embed_table_rows(const RowsOfTable p) {
    const bool one = p.scale == 1.f;
    const uint32_t lane = threadIdx.x & 31u;
    for (uint32_t t = blockIdx.x * 8u + (threadIdx.x >> 5); t < p.ids.tokens; t += gridDim.x * 8u) {
        uint64_t row = 0;
        const bool have = token_row(p.ids, t, row, lane == 0u);
        for (uint32_t c = lane; c < p.dim; c += 32u)
            p.out[t * p.ldo + c] = have ? scaled(__ldg(p.table + row * p.ldt + c), p.scale, one) : (uint16_t)0;
    }
}

// ------------------------------------------------------ rows of a coded scope

struct RowsOfLanes {
    IdSource ids;
    LanesParams lanes;     // the scope (out unused)
    uint64_t first;        // the table's first weight in the scope
    uint64_t total_bits;
    uint16_t *out;
    uint64_t ldo;
    uint32_t dim, row_groups;  // groups a row can touch
    uint32_t single;       // total_bits == 0: every exponent is this one
    float scale;
};

// One warp per (token, group the row touches); each lane decodes its chunk of
// the group if the row needs it, one codeword per lookup of the byte-keyed
// table 0 (1 KB of shared memory).
__global__ void __launch_bounds__(128) embed_lanes_rows(const RowsOfLanes p) {
    __shared__ uint32_t s_root[256];
    __shared__ uint32_t s_exp[4][16 * 32];  // word k of lane l's chunk at 32 k + l
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t *hier = p.lanes.lut + (2u << p.lanes.fast_bits);
    if (p.total_bits)
        for (uint32_t i = threadIdx.x; i < 256u; i += 128u) s_root[i] = __ldg(hier + i);
    __syncthreads();
    const bool one = p.scale == 1.f;
    const uint64_t items = (uint64_t)p.ids.tokens * p.row_groups;
    for (uint64_t item = blockIdx.x * 4ull + warp; item < items; item += gridDim.x * 4ull) {
        const uint32_t t = (uint32_t)(item / p.row_groups);
        uint64_t row = 0;
        const bool have = token_row(p.ids, t, row, lane == 0u);
        uint16_t *out = p.out + t * p.ldo;
        if (!have) {
            if (item % p.row_groups == 0u)
                for (uint32_t c = lane; c < p.dim; c += 32u) out[c] = 0;
            continue;
        }
        const uint64_t w0 = p.first + row * p.dim, w1 = w0 + p.dim;
        const uint64_t g = w0 / GROUP_SYMS + item % p.row_groups;
        if (g * GROUP_SYMS >= w1) continue;
        const uint64_t c = g * GROUP_CHUNKS + lane;  // this lane's chunk
        const bool need = c * LANE_SYMS < w1 && (c + 1u) * LANE_SYMS > w0;
        bool ok = true;
        uint32_t err = 0;
        __syncwarp();  // the previous item's slots have been read
        if (p.total_bits == 0u) {
            for (uint32_t k = 0; k < 16u; ++k) s_exp[warp][32u * k + lane] = rot_sym(p.single) * 0x01010101u;
        } else {
            const uint64_t gs0 = __ldg(p.lanes.group_start + g), gs1 = __ldg(p.lanes.group_start + g + 1);
            const uint32_t cbits = __ldg(p.lanes.chunk_bits + c);
            uint32_t incl = cbits;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                if (lane >= (uint32_t)d) incl += y;
            }
            const uint32_t gbits = __shfl_sync(0xFFFFFFFFu, incl, 31);
            ok = __all_sync(0xFFFFFFFFu, cbits <= 32u * LANE_SYMS) && gs1 - gs0 == gbits && gs1 <= p.total_bits;
            if (ok && need) {
                const uint32_t n = chunk_weights(p.lanes, (uint32_t)c);
                const uint64_t start = gs0 + incl - cbits;
                const uint32_t *words = reinterpret_cast<const uint32_t *>(p.lanes.stream);
                const uint64_t last = p.lanes.stream_bytes / 4u - 1u;
                uint64_t at = start >> 5;
                uint32_t a = bswap32(__ldg(words + min(at, last))), b = bswap32(__ldg(words + min(at + 1u, last)));
                uint32_t nxt = __ldg(words + min(at + 2u, last));
                uint32_t pos = (uint32_t)start & 31u, used = 0, acc = 0;
                for (uint32_t i = 0; i < n; ++i) {
                    const uint32_t x = __funnelshift_l(b, a, pos);
                    uint32_t e = s_root[x >> 24];
                    if (e & LUT_PTR) e = resolve_escape(x, hier, p.lanes.n_tables);
                    if (e & ESC_BAD) err |= ST_LUT;
                    const uint32_t len = (e >> LUT_LEN_SHIFT) & 63u;
                    used += len;
                    pos += len;
                    if (pos >= 32u) {
                        pos -= 32u;
                        a = b;
                        b = bswap32(nxt);
                        ++at;
                        nxt = __ldg(words + min(at + 2u, last));
                    }
                    acc |= rot_sym(e) << (8u * (i & 3u));
                    if ((i & 3u) == 3u || i + 1u == n) {
                        s_exp[warp][32u * (i >> 2) + lane] = acc;
                        acc = 0;
                    }
                }
                if (used != cbits) err |= ST_COUNT;
            }
        }
        if (!__all_sync(0xFFFFFFFFu, ok && err == 0u)) {
            if (!ok) err = ST_RANGE;
            if (err) atomicOr(&g_status, err);
            continue;  // a damaged group writes nothing
        }
        __syncwarp();  // the join reads other lanes' slots
        const uint64_t lo = max(w0, g * GROUP_SYMS), hi = min(w1, (g + 1u) * GROUP_SYMS);
        for (uint64_t w = lo + lane; w < hi; w += 32u) {
            const uint32_t i = (uint32_t)(w % LANE_SYMS), ch = (uint32_t)(w / LANE_SYMS % GROUP_CHUNKS);
            const uint32_t e = (s_exp[warp][32u * (i >> 2) + ch] >> (8u * (i & 3u))) & 0xFFu;
            out[w - w0] = scaled(join1(e, __ldg(p.lanes.mant + w)), p.scale, one);
        }
    }
}

// ------------------------------------------------------ the table's gradient

struct GradParams {
    IdSource ids;
    const void *dy;
    void *grad;
    uint64_t ld_dy;
    uint32_t dim, dy_fp32, grad_fp32, accumulate;
    float scale;
};

// One CTA per table row: it scans the ids in order and adds the matching
// tokens' rows, so the sum's order is fixed.
__global__ void __launch_bounds__(256) embed_grad_scan(const GradParams p) {
    __shared__ uint32_t s_hits[256 / 32];
    for (uint64_t v = blockIdx.x; v < p.ids.rows; v += gridDim.x) {
        for (uint32_t c0 = 0; c0 < p.dim; c0 += 256u) {
            const uint32_t c = c0 + threadIdx.x;
            float sum = 0.f;
            bool any = false;
            for (uint32_t t0 = 0; t0 < p.ids.tokens; t0 += 256u) {
                const uint32_t t = t0 + threadIdx.x;
                uint64_t row = 0;
                const bool hit = t < p.ids.tokens && token_row(p.ids, t, row, v == 0u && c0 == 0u) && row == v;
                const uint32_t m = __ballot_sync(0xFFFFFFFFu, hit);
                if ((threadIdx.x & 31u) == 0u) s_hits[threadIdx.x >> 5] = m;
                __syncthreads();
                for (uint32_t q = 0; q < 8u; ++q)
                    for (uint32_t b = s_hits[q]; b; b &= b - 1u) {
                        const uint64_t at = (uint64_t)(t0 + 32u * q + __ffs(b) - 1u) * p.ld_dy + c;
                        any = true;
                        if (c < p.dim)
                            sum += p.dy_fp32 ? static_cast<const float *>(p.dy)[at]
                                             : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.dy)[at]);
                    }
                __syncthreads();
            }
            if (c >= p.dim || (p.accumulate && !any)) continue;
            float g = p.scale * sum;
            const uint64_t at = v * p.dim + c;
            if (p.grad_fp32) {
                float *out = static_cast<float *>(p.grad) + at;
                *out = p.accumulate ? *out + g : (any ? g : 0.f);
            } else {
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.grad) + at;
                *out = __float2bfloat16_rn(p.accumulate ? __bfloat162float(*out) + g : (any ? g : 0.f));
            }
        }
    }
}

dfw_status ids_checked(const void *d_ids, int ids64, uint64_t tokens, uint64_t rows, IdSource &s) {
    if ((ids64 != 0 && ids64 != 1) || tokens > DFW_EMBED_MAX_TOKENS || rows < 1u || rows > DFW_EMBED_MAX_ROWS ||
        (tokens && !d_ids))
        return DFW_EINVAL;
    if (reinterpret_cast<uintptr_t>(d_ids) & (ids64 ? 7u : 3u)) return DFW_EALIGN;
    s.ids = d_ids;
    s.wide = (uint32_t)ids64;
    s.tokens = (uint32_t)tokens;
    s.rows = rows;
    return DFW_OK;
}

}  // namespace

dfw_status launch_embed_rows(const uint16_t *d_table, uint64_t rows, uint32_t dim, uint64_t ld_table, const void *d_ids,
                             int ids64, uint64_t tokens, float scale, uint16_t *d_out, uint64_t ld_out,
                             cudaStream_t s) {
    RowsOfTable p;
    dfw_status st = ids_checked(d_ids, ids64, tokens, rows, p.ids);
    if (st != DFW_OK) return st;
    if (dim < 1u || dim > DFW_EMBED_MAX_DIM || !d_table || (rows > 1u && ld_table < dim) || (tokens > 1u && ld_out < dim) || (tokens && !d_out))
        return DFW_EINVAL;
    if ((reinterpret_cast<uintptr_t>(d_table) | reinterpret_cast<uintptr_t>(d_out)) & 1u) return DFW_EALIGN;
    if (tokens == 0u) return DFW_OK;
    int sms = 0;
    if ((st = device_sms(sms)) != DFW_OK) return st;
    p.table = d_table;
    p.out = d_out;
    p.ldt = ld_table;
    p.ldo = ld_out;
    p.dim = dim;
    p.scale = scale;
    const uint64_t want = (tokens + 7u) / 8u, cap = (uint64_t)sms * 8u;
    embed_table_rows<<<(unsigned)(want < cap ? want : cap), 256, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? DFW_OK : DFW_ECUDA;
}

dfw_status launch_embed_lanes(const dfw_lanes_scope *scope, uint64_t first, uint64_t rows, uint32_t dim,
                              const void *d_ids, int ids64, uint64_t tokens, float scale, uint16_t *d_out,
                              uint64_t ld_out, cudaStream_t s) {
    if (!scope || !scope->table || !scope->info) return DFW_EINVAL;
    const dfw_table *table = scope->table;
    dfw_status st = validate_table(table);
    if (st != DFW_OK) return st;
    RowsOfLanes p;
    std::memset(&p, 0, sizeof(p));
    if ((st = ids_checked(d_ids, ids64, tokens, rows, p.ids)) != DFW_OK) return st;
    if (dim < 1u || dim > DFW_EMBED_MAX_DIM || first > table->n || rows > (table->n - first) / dim ||
        (tokens > 1u && ld_out < dim) || !scope->d_mant || (tokens && !d_out))
        return DFW_EINVAL;
    if (reinterpret_cast<uintptr_t>(scope->d_mant) & 15u || reinterpret_cast<uintptr_t>(d_out) & 1u) return DFW_EALIGN;
    if (table->total_bits) {
        st = lanes_params(scope->d_stream, scope->d_mant, scope->d_lut, scope->d_chunk_bits, scope->d_group_start,
                          table, scope->info, p.lanes);
        if (st != DFW_OK) return st;
    } else {
        p.lanes.mant = scope->d_mant;
    }
    if (tokens == 0u) return DFW_OK;
    int sms = 0;
    if ((st = device_sms(sms)) != DFW_OK) return st;
    p.lanes.mant = scope->d_mant;
    p.first = first;
    p.total_bits = table->total_bits;
    p.out = d_out;
    p.ldo = ld_out;
    p.dim = dim;
    p.single = table->single_symbol;
    p.scale = scale;
    // whole groups per row when every row starts on a group boundary or rows
    // divide a group; else a row may touch one group more
    const uint32_t whole = (dim + GROUP_SYMS - 1u) / GROUP_SYMS;
    const bool even = first % GROUP_SYMS == 0u && (dim % GROUP_SYMS == 0u || GROUP_SYMS % dim == 0u);
    p.row_groups = even ? whole : (dim + GROUP_SYMS - 2u) / GROUP_SYMS + 1u;
    const uint64_t want = (tokens * p.row_groups + 3u) / 4u, cap = (uint64_t)sms * 16u;
    embed_lanes_rows<<<(unsigned)(want < cap ? want : cap), 128, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? DFW_OK : DFW_ECUDA;
}

uint64_t embed_grad_scratch(uint64_t tokens, uint32_t) { return tokens ? 16u : 0u; }

dfw_status launch_embed_grad(const void *d_ids, int ids64, uint64_t tokens, const void *d_dy, int dy_fp32,
                             uint64_t ld_dy, uint64_t rows, uint32_t dim, float scale, void *d_grad, int grad_fp32,
                             int accumulate, void *d_scratch, uint64_t scratch_bytes, cudaStream_t s) {
    GradParams p;
    dfw_status st = ids_checked(d_ids, ids64, tokens, rows, p.ids);
    if (st != DFW_OK) return st;
    if (dim < 1u || dim > DFW_EMBED_MAX_DIM || !d_grad || (tokens && (!d_dy || !d_scratch)) || (tokens > 1u && ld_dy < dim) ||
        (dy_fp32 | grad_fp32 | accumulate) & ~1)
        return DFW_EINVAL;
    if ((reinterpret_cast<uintptr_t>(d_dy) & (dy_fp32 ? 3u : 1u)) || (reinterpret_cast<uintptr_t>(d_grad) & (grad_fp32 ? 3u : 1u)) ||
        (reinterpret_cast<uintptr_t>(d_scratch) & 15u))
        return DFW_EALIGN;
    if (scratch_bytes < embed_grad_scratch(tokens, dim)) return DFW_ENOMEM;
    if (tokens == 0u && accumulate) return DFW_OK;
    int sms = 0;
    if ((st = device_sms(sms)) != DFW_OK) return st;
    p.dy = d_dy;
    p.grad = d_grad;
    p.ld_dy = ld_dy;
    p.dim = dim;
    p.dy_fp32 = (uint32_t)dy_fp32;
    p.grad_fp32 = (uint32_t)grad_fp32;
    p.accumulate = (uint32_t)accumulate;
    p.scale = scale;
    const uint64_t cap = (uint64_t)sms * 8u;
    embed_grad_scan<<<(unsigned)(rows < cap ? rows : cap), 256, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? DFW_OK : DFW_ECUDA;
}

}  // namespace dfw
