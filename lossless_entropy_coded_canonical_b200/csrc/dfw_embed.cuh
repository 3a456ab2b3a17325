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

#include <algorithm>

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

// Sorting.  A CTA sorts a block of up to 1024 IPT tokens by row, stably, in
// shared memory: 8 bits a pass from the lowest, each warp ranking its own run
// of tokens (equal digits of 32 tokens found by one match instruction, so no
// atomics and a fixed order), then one scan over (digit, warp).  Tokens
// without a row get key `rows` and end up behind all others.
constexpr uint32_t SORT_THREADS = 1024, SORT_WARPS = 32, SORT_STRIDE = 257;

struct SortParams {
    IdSource ids;
    uint32_t *keys, *pos;  // per block: sorted keys and the tokens they belong to
    uint32_t blocks, passes;
    uint8_t *fill;         // zeroed meanwhile by the CTAs past the sorting ones (null: nothing)
    uint64_t fill_bytes;
};

template <int IPT>
constexpr uint32_t sort_smem() {
    return SORT_WARPS * SORT_STRIDE * 4u + 32u * 4u + SORT_THREADS * IPT * 6u;
}

// Zeroes bytes [0, n) of p from the CTAs [first, gridDim.x).
__device__ __forceinline__ void zero_fill(uint8_t *p, uint64_t n, uint32_t first) {
    const uint64_t me = (uint64_t)(blockIdx.x - first) * blockDim.x + threadIdx.x;
    const uint64_t all = (uint64_t)(gridDim.x - first) * blockDim.x;
    const uint64_t head = min(n, (uint64_t)(-reinterpret_cast<uintptr_t>(p) & 31u));
    const uint64_t body = (n - head) >> 5, tail = n - head - (body << 5);
    if (me < head) p[me] = 0;
    if (me < tail) p[n - 1u - me] = 0;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    for (uint64_t i = me; i < body; i += all) stg256_cs(p + head + (i << 5), z, z);
}

template <int IPT>
__global__ void __launch_bounds__(SORT_THREADS, 1) grad_sort(const SortParams p) {
    if (blockIdx.x >= p.blocks) {
        zero_fill(p.fill, p.fill_bytes, p.blocks);
        return;
    }
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t *cnt = reinterpret_cast<uint32_t *>(smem);  // [warp][digit], rows of SORT_STRIDE: a scan's reads hit 32 banks
    uint32_t *sums = cnt + SORT_WARPS * SORT_STRIDE;
    uint32_t *s_key = sums + 32;
    uint16_t *s_pos = reinterpret_cast<uint16_t *>(s_key + SORT_THREADS * IPT);
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const uint32_t base = blockIdx.x * SORT_THREADS * IPT, run = warp * 32u * IPT + lane;
    uint32_t key[IPT];
    uint16_t pos[IPT];
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
        const uint32_t t = base + run + 32u * j;
        uint64_t row = p.ids.rows;
        pos[j] = (uint16_t)(run + 32u * j);
        key[j] = 0xFFFFFFFFu;
        if (t < p.ids.tokens) key[j] = token_row(p.ids, t, row, true) ? (uint32_t)row : (uint32_t)p.ids.rows;
    }
    for (uint32_t pass = 0; pass < p.passes; ++pass) {
        const uint32_t shift = 8u * pass;
        for (uint32_t i = lane; i < 256u; i += 32u) cnt[warp * SORT_STRIDE + i] = 0u;
        __syncwarp();
        uint16_t rank[IPT];
#pragma unroll
        for (int j = 0; j < IPT; ++j) {
            const uint32_t d = (key[j] >> shift) & 255u;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, d), leader = __ffs(same) - 1u;
            uint32_t *c = cnt + warp * SORT_STRIDE + d;
            uint32_t old = 0;
            if (lane == leader) {
                old = *c;
                *c = old + __popc(same);
            }
            rank[j] = (uint16_t)(__shfl_sync(0xFFFFFFFFu, old, leader) + __popc(same & ((1u << lane) - 1u)));
            __syncwarp();
        }
        __syncthreads();
        // exclusive offsets in (digit, warp) order: thread i takes digit i / 4, warps 8 (i mod 4) .. + 7
        uint32_t *mine = cnt + 8u * (tid & 3u) * SORT_STRIDE + (tid >> 2), sum = 0;
#pragma unroll
        for (uint32_t k = 0; k < 8u; ++k) {
            const uint32_t v = mine[k * SORT_STRIDE];
            mine[k * SORT_STRIDE] = sum;
            sum += v;
        }
        uint32_t incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= (uint32_t)d) incl += y;
        }
        if (lane == 31u) sums[warp] = incl;
        __syncthreads();
        uint32_t before = sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, before, d);
            if (lane >= (uint32_t)d) before += y;
        }
        before = __shfl_sync(0xFFFFFFFFu, before, (warp + 31u) & 31u);
        const uint32_t off = (warp ? before : 0u) + incl - sum;
#pragma unroll
        for (uint32_t k = 0; k < 8u; ++k) mine[k * SORT_STRIDE] += off;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < IPT; ++j) {
            const uint32_t to = cnt[warp * SORT_STRIDE + ((key[j] >> shift) & 255u)] + rank[j];
            s_key[to] = key[j];
            s_pos[to] = pos[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < IPT; ++j) {
            key[j] = s_key[run + 32u * j];
            pos[j] = s_pos[run + 32u * j];
        }
    }
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
        const uint32_t t = base + run + 32u * j;
        if (t < p.ids.tokens) {
            p.keys[t] = key[j];
            p.pos[t] = base + pos[j];
        }
    }
}

// Joins sorted blocks into one order: a token's place is its place in its own
// block plus, for every other block, how many of its keys come before (equal
// keys of earlier blocks do, those of later ones do not).  LANES lanes share
// a token's blocks, each a binary search.
struct MergeParams {
    const uint32_t *keys, *pos;
    uint32_t *out_keys, *out_pos;
    uint32_t tokens, blocks, block;
};

template <int LANES>
__global__ void __launch_bounds__(256) grad_merge(const MergeParams p) {
    const uint64_t i = (blockIdx.x * 256ull + threadIdx.x) / LANES;
    const uint32_t sub = threadIdx.x % LANES;
    const uint32_t t = (uint32_t)min(i, (uint64_t)p.tokens - 1u);
    const uint32_t key = __ldg(p.keys + t), own = t / p.block;
    uint32_t place = 0;
    for (uint32_t b = sub; b < p.blocks; b += LANES) {
        const uint32_t lo0 = b * p.block;
        if (b == own) {
            place += t - lo0;
            continue;
        }
        uint32_t lo = lo0, hi = min(lo0 + p.block, p.tokens);
        const uint32_t below = b < own ? key + 1u : key;  // keys are below 2^31
        while (lo < hi) {
            const uint32_t mid = (lo + hi) >> 1;
            if (__ldg(p.keys + mid) < below) lo = mid + 1u;
            else hi = mid;
        }
        place += lo - lo0;
    }
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) place += __shfl_xor_sync(0xFFFFFFFFu, place, d);
    if (sub == 0u && i < p.tokens) {
        p.out_keys[place] = key;
        p.out_pos[place] = __ldg(p.pos + t);
    }
}

// Summing.  The sorted tokens are cut into windows of `window`; a thread
// walks a window with VEC columns, eight rows of dy in flight, and writes a
// row's sum when the next row's tokens begin.  A row whose tokens reach past
// the window leaves a partial sum instead (slot 0 if it came from the window
// before, else slot 1); grad_join adds those up in window order.
struct ReduceParams {
    const uint32_t *keys, *pos;
    const void *dy;
    void *grad;
    float *partial;  // [windows][2][dim]
    uint64_t ld_dy;
    uint32_t tokens, windows, window, dim, rows;
    uint32_t tpr;          // threads per window (a power of two)
    uint32_t col_blocks;
    uint32_t accumulate;
    float scale;
};

template <typename T>
__device__ __forceinline__ float as_float(T v);
template <>
__device__ __forceinline__ float as_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int N>
struct __align__(sizeof(T) * N) Pack {
    T v[N];
};

// Writes (or adds) scale x sum to VEC columns of a row, rounded once.
template <typename OUT, int VEC>
__device__ __forceinline__ void put_row(void *grad, uint64_t at, const float (&acc)[VEC], float scale, bool add) {
    constexpr int N = VEC * sizeof(OUT) > 16 ? 16 / sizeof(OUT) : VEC;  // at most 16 bytes at once
#pragma unroll
    for (int i = 0; i < VEC; i += N) {
        Pack<OUT, N> *dst = reinterpret_cast<Pack<OUT, N> *>(static_cast<OUT *>(grad) + at + i);
        Pack<OUT, N> o;
        if (add) o = *dst;
#pragma unroll
        for (int j = 0; j < N; ++j) o.v[j] = from_float<OUT>(add ? fmaf(scale, acc[i + j], as_float<OUT>(o.v[j])) : scale * acc[i + j]);
        *dst = o;
    }
}

template <typename DY, typename OUT, int VEC>
__global__ void __launch_bounds__(128) grad_reduce(const ReduceParams p) {
    constexpr int U = 8;  // rows in flight
    const uint32_t per = 128u / p.tpr;  // windows a CTA walks at once
    const uint32_t w = blockIdx.x / p.col_blocks * per + threadIdx.x / p.tpr;
    const uint32_t col = (blockIdx.x % p.col_blocks * p.tpr + threadIdx.x % p.tpr) * VEC;
    if (w >= p.windows || col >= p.dim) return;
    const uint32_t i0 = w * p.window, n = min(p.window, p.tokens - i0);
    const uint32_t prev = i0 ? __ldg(p.keys + i0 - 1u) : 0xFFFFFFFFu;
    const uint32_t next = i0 + n < p.tokens ? __ldg(p.keys + i0 + n) : 0xFFFFFFFFu;
    float acc[VEC];
    uint32_t cur = 0xFFFFFFFFu;  // the row being summed
    bool first = true;           // its tokens began before the window, or at its first token
    auto flush = [&](bool last) {
        if (cur >= p.rows) return;
        const bool left = first && cur == prev, right = last && cur == next;
        if (left || right) {
            float *dst = p.partial + ((uint64_t)w * 2u + (left ? 0u : 1u)) * p.dim + col;
            constexpr int N = VEC > 4 ? 4 : VEC;
#pragma unroll
            for (int k = 0; k < VEC; k += N) {
                Pack<float, N> o;
#pragma unroll
                for (int j = 0; j < N; ++j) o.v[j] = acc[k + j];
                *reinterpret_cast<Pack<float, N> *>(dst + k) = o;
            }
        } else {
            put_row<OUT, VEC>(p.grad, (uint64_t)cur * p.dim + col, acc, p.scale, p.accumulate != 0u);
        }
    };
    for (uint32_t i = 0; i < n; i += U) {
        uint32_t key[U];
        Pack<DY, VEC> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            key[u] = i + u < n ? __ldg(p.keys + i0 + i + u) : 0xFFFFFFFFu;
            if (key[u] < p.rows)
                v[u] = *reinterpret_cast<const Pack<DY, VEC> *>(static_cast<const DY *>(p.dy) +
                                                               (uint64_t)__ldg(p.pos + i0 + i + u) * p.ld_dy + col);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u >= n) break;
            if (key[u] != cur) {
                if (i + u) {
                    flush(false);
                    first = false;
                }
                cur = key[u];
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
            }
            if (cur < p.rows) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] += as_float<DY>(v[u].v[k]);
            }
        }
    }
    flush(true);
}

// One CTA per (window, 32 columns) whose last row begins in that window and
// goes on in the next: it adds that row's partial sums, eight threads to a
// column, each every eighth window, then their eight sums in order.
template <typename OUT>
__global__ void __launch_bounds__(256) grad_join(const ReduceParams p) {
    __shared__ float s_sum[8][33];
    const uint32_t w = blockIdx.x / p.col_blocks, col = blockIdx.x % p.col_blocks * 32u + (threadIdx.x & 31u);
    const uint32_t i0 = w * p.window, end = i0 + p.window, sub = threadIdx.x >> 5;
    if (end >= p.tokens) return;
    const uint32_t key = __ldg(p.keys + end);
    if (key >= p.rows || __ldg(p.keys + end - 1u) != key) return;
    if (__ldg(p.keys + i0) == key && i0 && __ldg(p.keys + i0 - 1u) == key) return;  // it began earlier
    uint32_t lo = end, hi = p.tokens;  // the first token behind the row's
    while (lo < hi) {
        const uint32_t mid = (lo + hi) >> 1;
        if (__ldg(p.keys + mid) <= key) lo = mid + 1u;
        else hi = mid;
    }
    const uint32_t last = (lo - 1u) / p.window;
    float sum = 0.f;
    if (col < p.dim)
        for (uint32_t k = w + sub; k <= last; k += 8u)
            sum += p.partial[((uint64_t)k * 2u + (k == w ? 1u : 0u)) * p.dim + col];
    s_sum[sub][threadIdx.x & 31u] = sum;
    __syncthreads();
    if (sub || col >= p.dim) return;
    for (uint32_t k = 1; k < 8u; ++k) sum += s_sum[k][threadIdx.x];
    const float acc[1] = {sum};
    put_row<OUT, 1>(p.grad, (uint64_t)key * p.dim + col, acc, p.scale, p.accumulate != 0u);
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

// How the gradient of `tokens` tokens is cut: blocks of `block` tokens for
// sorting (one if a CTA can hold them all), windows for summing.
struct GradCut {
    uint32_t ipt, block, blocks, window, windows;
    uint64_t list;  // bytes of one array of keys or positions
};

GradCut grad_cut(uint64_t tokens) {
    GradCut c;
    c.ipt = tokens <= 1024u ? 1u : tokens <= 4096u ? 4u : 16u;
    c.block = SORT_THREADS * c.ipt;
    c.blocks = (uint32_t)((tokens + c.block - 1u) / c.block);
    c.window = tokens <= (1u << 14) ? 32u : tokens <= (1u << 17) ? 64u : 128u;
    c.windows = (uint32_t)((tokens + c.window - 1u) / c.window);
    c.list = (tokens * 4u + 15u) & ~15ull;
    return c;
}

uint64_t embed_grad_scratch(uint64_t tokens, uint32_t dim) {
    const GradCut c = grad_cut(tokens);
    return c.list * (c.blocks > 1u ? 4u : 2u) + (c.windows > 1u ? (uint64_t)c.windows * 2u * dim * 4u : 0u);
}

template <int IPT>
dfw_status launch_grad_sort(const SortParams &p, unsigned grid, cudaStream_t s) {
    static int opted[16];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 16) return DFW_ECUDA;
    if (!opted[dev]) {
        if (cudaFuncSetAttribute(grad_sort<IPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, sort_smem<IPT>()) != cudaSuccess)
            return DFW_ECUDA;
        opted[dev] = 1;
    }
    grad_sort<IPT><<<grid, SORT_THREADS, sort_smem<IPT>(), s>>>(p);
    return cudaGetLastError() == cudaSuccess ? DFW_OK : DFW_ECUDA;
}

template <typename DY, typename OUT>
dfw_status launch_grad_reduce(ReduceParams p, bool vec, cudaStream_t s) {
    constexpr uint32_t V = 16 / sizeof(DY);
    const uint32_t threads = vec ? p.dim / V : p.dim;
    p.tpr = 1u;
    while (p.tpr < 128u && p.tpr < threads) p.tpr *= 2u;
    p.col_blocks = (threads + p.tpr - 1u) / p.tpr;
    const uint64_t per = 128u / p.tpr, grid = (p.windows + per - 1u) / per * p.col_blocks;
    if (grid > 0x7FFFFFFFull) return DFW_EINVAL;
    if (vec) grad_reduce<DY, OUT, (int)V><<<(unsigned)grid, 128, 0, s>>>(p);
    else grad_reduce<DY, OUT, 1><<<(unsigned)grid, 128, 0, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return DFW_ECUDA;
    if (p.windows < 2u) return DFW_OK;
    p.col_blocks = (p.dim + 31u) / 32u;
    const uint64_t joins = (uint64_t)(p.windows - 1u) * p.col_blocks;
    if (joins > 0x7FFFFFFFull) return DFW_EINVAL;
    grad_join<OUT><<<(unsigned)joins, 256, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? DFW_OK : DFW_ECUDA;
}

dfw_status launch_embed_grad(const void *d_ids, int ids64, uint64_t tokens, const void *d_dy, int dy_fp32,
                             uint64_t ld_dy, uint64_t rows, uint32_t dim, float scale, void *d_grad, int grad_fp32,
                             int accumulate, void *d_scratch, uint64_t scratch_bytes, cudaStream_t s) {
    SortParams sp;
    dfw_status st = ids_checked(d_ids, ids64, tokens, rows, sp.ids);
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
    const GradCut cut = grad_cut(tokens);
    uint8_t *const scratch = static_cast<uint8_t *>(d_scratch);
    uint32_t *lists[4];
    for (int i = 0; i < 4; ++i) lists[i] = reinterpret_cast<uint32_t *>(scratch + i * cut.list);
    // sort the blocks; the other SMs zero the gradient meanwhile
    sp.keys = lists[0];
    sp.pos = lists[1];
    sp.blocks = cut.blocks;
    sp.passes = 1u;
    while (rows >> (8u * sp.passes)) ++sp.passes;  // keys go up to `rows`
    sp.fill = accumulate ? nullptr : static_cast<uint8_t *>(d_grad);
    sp.fill_bytes = accumulate ? 0u : rows * dim * (grad_fp32 ? 4u : 2u);
    const uint64_t fillers = sp.fill_bytes ? std::min<uint64_t>((sp.fill_bytes + (1u << 15) - 1u) >> 15, (uint64_t)sms) : 0u;
    const unsigned grid = (unsigned)(cut.blocks + fillers);
    st = cut.ipt == 1u ? launch_grad_sort<1>(sp, grid, s) : cut.ipt == 4u ? launch_grad_sort<4>(sp, grid, s) : launch_grad_sort<16>(sp, grid, s);
    if (st != DFW_OK || tokens == 0u) return st;
    ReduceParams p;
    p.keys = lists[0];
    p.pos = lists[1];
    if (cut.blocks > 1u) {
        MergeParams m = {lists[0], lists[1], lists[2], lists[3], (uint32_t)tokens, cut.blocks, cut.block};
        const auto blocks = [&](uint64_t lanes) { return (unsigned)((tokens * lanes + 255u) / 256u); };
        if (cut.blocks <= 4u) grad_merge<4><<<blocks(4), 256, 0, s>>>(m);
        else grad_merge<16><<<blocks(16), 256, 0, s>>>(m);
        if (cudaGetLastError() != cudaSuccess) return DFW_ECUDA;
        p.keys = lists[2];
        p.pos = lists[3];
    }
    p.dy = d_dy;
    p.grad = d_grad;
    p.partial = reinterpret_cast<float *>(scratch + (cut.blocks > 1u ? 4u : 2u) * cut.list);
    p.ld_dy = ld_dy;
    p.tokens = (uint32_t)tokens;
    p.windows = cut.windows;
    p.window = cut.window;
    p.dim = dim;
    p.rows = (uint32_t)rows;
    p.accumulate = (uint32_t)accumulate;
    p.scale = scale;
    // 16-byte loads where every row of dy, and every piece of a gradient row, is aligned for them
    const bool vec = dim % 8u == 0u && ((reinterpret_cast<uintptr_t>(d_dy) | reinterpret_cast<uintptr_t>(d_grad)) & 15u) == 0u &&
                     (tokens == 1u || ld_dy * (dy_fp32 ? 4u : 2u) % 16u == 0u);
    if (dy_fp32) return grad_fp32 ? launch_grad_reduce<float, float>(p, vec, s) : launch_grad_reduce<float, __nv_bfloat16>(p, vec, s);
    return grad_fp32 ? launch_grad_reduce<__nv_bfloat16, float>(p, vec, s) : launch_grad_reduce<__nv_bfloat16, __nv_bfloat16>(p, vec, s);
}

}  // namespace dfw
