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
#include <cstring>
#include <type_traits>

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
    const int64_t id = s.wide ? (int64_t)ld_after(static_cast<const uint64_t *>(s.ids) + t)
                              : (int64_t)(int32_t)ld_after(static_cast<const uint32_t *>(s.ids) + t);
    if (id < 0) return false;
    if ((uint64_t)id >= s.rows) {
        if (report) atomicOr(&g_status, ST_INDEX);
        return false;
    }
    row = (uint64_t)id;
    return true;
}

// a b and a b + c for a bf16 result: the exact value if fp32 has it, else of its
// two neighbours in fp32 the one whose last bit is set.  Such a value is on a
// tie of a bf16 only if the exact one is, so the conversion to bf16 is the only
// rounding.  (From the nearest fp32, a value beside a tie could land on it: for
// some scales 1 in 130 weights went the wrong way.)  The neighbours' bits are
// consecutive numbers, so one of them is odd.  It costs little: a bf16 gradient
// of 8192 rows of 4096 takes 71.0 us against 70.0, 45.6 against 42.1 if it is
// added to the old values, as many coded rows with such a scale 32 to 33
// against 31.  (Working out again only what is a tie in fp32: 75 to 79 us, as
// the second copy of the arithmetic takes registers from the rows in flight.)
__device__ __forceinline__ float mul_odd(float a, float b) {
    return __uint_as_float(__float_as_uint(__fmul_rz(a, b)) | (__float_as_uint(__fmul_ru(fabsf(a), fabsf(b))) & 1u));
}
__device__ __forceinline__ float fma_odd(float a, float b, float c) {
    const uint32_t both = __float_as_uint(__fmaf_rd(a, b, c)) | __float_as_uint(__fmaf_ru(a, b, c));
    return __uint_as_float(__float_as_uint(__fmaf_rz(a, b, c)) | (both & 1u));
}

// bf16(scale w), rounded once to nearest even, of two weights at a time.
// Scale 1 keeps the bits (NaN payloads included), as the decoder does.  A scale
// that is a bf16 itself takes one packed multiplication; others go by mul_odd.
enum ScaleKind { SCALE_ONE, SCALE_BF16, SCALE_FP32 };
struct RowScale {
    float f;
    uint32_t pair;  // the scale's upper half, twice
    ScaleKind kind;
};
RowScale row_scale(float scale) {
    uint32_t u;
    std::memcpy(&u, &scale, 4);
    return {scale, (u >> 16) * 0x10001u, scale == 1.f ? SCALE_ONE : (u & 0xFFFFu) == 0u ? SCALE_BF16 : SCALE_FP32};
}
template <ScaleKind KIND>
__device__ __forceinline__ uint32_t scaled2(uint32_t w, const RowScale &s) {
    if constexpr (KIND == SCALE_ONE) return w;
    uint32_t r;
    if constexpr (KIND == SCALE_BF16) {
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(s.pair));
    } else {
        const float lo = mul_odd(__uint_as_float(w << 16), s.f), hi = mul_odd(__uint_as_float(w & 0xFFFF0000u), s.f);
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    }
    return r;
}
template <ScaleKind KIND>
__device__ __forceinline__ uint4 scaled8(uint4 w, const RowScale &s) {
    return make_uint4(scaled2<KIND>(w.x, s), scaled2<KIND>(w.y, s), scaled2<KIND>(w.z, s), scaled2<KIND>(w.w, s));
}
template <ScaleKind KIND>
__device__ __forceinline__ uint16_t scaled1(uint32_t w, const RowScale &s) {
    return (uint16_t)scaled2<KIND>(w, s);
}

// ------------------------------------------------------- rows of a bf16 table

struct RowsOfTable {
    IdSource ids;
    const uint16_t *table;
    uint16_t *out;
    uint64_t ldt, ldo;
    uint32_t dim, parts;  // parts: pieces of EMBED_PART a row is cut into
    RowScale scale;
};

// A warp copies one piece of a row: VEC weights per lane and access, four
// accesses in flight.  Bound by memory: 16384 rows of 2048 take 12.5 us (134 MB
// read and written; rows that repeat come from L2).
constexpr uint32_t EMBED_PART = 1024;

template <ScaleKind KIND, int VEC>
__device__ __forceinline__ void copy_piece(const RowScale &s, const uint16_t *src, uint16_t *dst, uint32_t c0, uint32_t end,
                                           bool have, uint32_t lane) {
    if constexpr (VEC == 8) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = c0 + 256u * i + 8u * lane;
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (have && c < end) v[i] = ld_after(reinterpret_cast<const uint4 *>(src + c));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = c0 + 256u * i + 8u * lane;
            if (c < end) __stcs(reinterpret_cast<uint4 *>(dst + c), have ? scaled8<KIND>(v[i], s) : v[i]);
        }
    } else {
        auto batch = [&](uint32_t at, auto count, bool whole) {  // all loads, then all stores
            constexpr int U = decltype(count)::value;
            uint16_t v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                v[i] = 0;
                if (have && (whole || at + 32u * i < end)) v[i] = ld_after(src + at + 32u * i);
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (whole || at + 32u * i < end) dst[at + 32u * i] = have ? scaled1<KIND>(v[i], s) : (uint16_t)0;
        };
        uint32_t at = c0 + lane;
        for (; at + 32u * 7u < end; at += 256u) batch(at, std::integral_constant<int, 8>(), true);
        for (; at < end; at += 128u) batch(at, std::integral_constant<int, 4>(), false);
    }
}

template <int VEC>
__global__ void __launch_bounds__(256) embed_table_rows(const RowsOfTable p) {
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t lane = threadIdx.x & 31u;
    const uint64_t piece = blockIdx.x * 8ull + (threadIdx.x >> 5);
    const uint32_t t = (uint32_t)(piece / p.parts), c0 = (uint32_t)(piece % p.parts) * EMBED_PART;
    if (t >= p.ids.tokens) return;
    uint64_t row = 0;
    const bool have = token_row(p.ids, t, row, lane == 0u);
    const uint16_t *src = p.table + row * p.ldt;
    uint16_t *dst = p.out + t * p.ldo;
    const uint32_t end = min(p.dim, c0 + EMBED_PART);
    switch (p.scale.kind) {
        case SCALE_ONE: copy_piece<SCALE_ONE, VEC>(p.scale, src, dst, c0, end, have, lane); break;
        case SCALE_BF16: copy_piece<SCALE_BF16, VEC>(p.scale, src, dst, c0, end, have, lane); break;
        default: copy_piece<SCALE_FP32, VEC>(p.scale, src, dst, c0, end, have, lane);
    }
}

// ------------------------------------------------------ rows of a coded scope

struct RowsOfLanes {
    IdSource ids;
    LanesParams lanes;     // the scope (out unused)
    uint64_t first;        // the table's first weight in the scope
    uint16_t *out;
    uint64_t ldo;
    uint32_t dim;
    uint32_t units;        // the most groups a row meets
    uint32_t single;       // embed_single_rows: every exponent is this one
    RowScale scale;
};

// Writes zeros to weights [c0, c1) of a token's row.
__device__ __forceinline__ void zero_row(uint16_t *out, uint32_t c0, uint32_t c1, uint32_t lane) {
    for (uint32_t c = c0 + lane; c < c1; c += 32u) out[c] = 0;
}

// Joins, scales and writes weights [lo, hi) of a decoded group (raw bytes at
// mbuf, exponents at exps0) to out + lo, out + lo + 1, ...
template <ScaleKind KIND, int V>
__device__ __forceinline__ void join_row(const RowScale &s, uint16_t *out, uint32_t lo, uint32_t hi, uint32_t mbuf,
                                         uint32_t exps0, uint32_t lane) {
    if constexpr (V == 16) {
        const uint32_t mrow = mbuf + 16u * lane, erow = exps0 + 4u * (lane >> 2) + 4u * EXP_STRIDE * (lane & 3u);
#pragma unroll
        for (uint32_t j = 0; j < 4u; ++j) {
            const uint32_t i = 512u * j + 16u * lane;
            if (i < lo || i >= hi || !check(i + V <= hi, CK_EMBED_STORE)) continue;
            uint4 a, b;
            join16(mrow + 512u * j, erow + 32u * j, a, b);
            stg256_cs(out + i, scaled8<KIND>(a, s), scaled8<KIND>(b, s));
        }
    } else if constexpr (V == 8) {
#pragma unroll 4
        for (uint32_t j = 0; j < 8u; ++j) {  // piece lane + 32 j: words 2 (piece mod 8) and + 1 of chunk piece / 8
            const uint32_t piece = lane + 32u * j, i = 8u * piece;
            if (i < lo || i >= hi || !check(i + V <= hi, CK_EMBED_STORE)) continue;
            const uint32_t e = exps0 + 4u * (piece >> 3) + 2u * EXP_STRIDE * (piece & 7u), m = mbuf + 8u * piece;
            uint4 v;
            join4(lds32(e), lds32(m), v.x, v.y);
            join4(lds32(e + EXP_STRIDE), lds32(m + 4u), v.z, v.w);
            __stcs(reinterpret_cast<uint4 *>(out + i), scaled8<KIND>(v, s));
        }
    } else {
#pragma unroll 4
        for (uint32_t i = lo + lane; i < hi; i += 32u) {
            const uint32_t e = lds32(exps0 + 4u * (i >> 6) + EXP_STRIDE * ((i & 63u) >> 2)) >> (8u * (i & 3u));
            const uint32_t m = lds32(mbuf + (i & ~3u)) >> (8u * (i & 3u));
            out[i] = scaled1<KIND>(join1(e & 0xFFu, m & 0xFFu), s);
        }
    }
}

// The decode kernel's work on chosen groups: a unit is one group of a token's
// row (the first ones of all tokens, then the second ones; rows that begin
// anywhere meet fewer groups than others, and those units are passed over),
// staged as decode_lanes stages its own (the same copies, positions, lookups
// and checks: a group is read whole), except that lanes whose chunk the row
// does not touch decode nothing, and the join scales and writes the row's part
// of the group.  (Rows that are not whole groups as one unit each: 3 rows of
// 20000 32 us, so 7; 67 of 5365 17.7 and 8.3; 2000 of 5365 27 and 23; 8000 of
// 1000 21.6 and 21.3; 4000 of 1001 15.4 and 16.8.)
// The starts of the group after the current one are loaded ahead; the table's
// copy and check overlap the first group's three dependent loads (id, group
// start, stream).
// 8192 rows of 4096 take 29.3 us, 0.18 per group and SM past 10 of start (32 us
// with a unit's id loaded by itself): 1245 warp instructions per group (the
// decode's 1011), 64% of the issue slots, 55% of the integer pipe.  One row 6.1,
// a chain of dependent loads.  Rows narrower than a group cost a group each:
// 16384 rows of 192 24.9 us, of 72 23.6.
// V: the join's weights per access; every row begins at a multiple of V in
// the scope and at 2 V bytes in the output (V = 1: no alignment).
template <int NT, int V>
__global__ void __launch_bounds__(NT) embed_lanes_rows(const RowsOfLanes p) {
    constexpr uint32_t NWARP = NT / 32;
    extern __shared__ __align__(16) uint8_t smem[];
    griddep_wait();
    griddep_launch_dependents();
    const LanesParams &prm = p.lanes;
    const uint32_t n_fast = 1u << prm.fast_bits;
    uint2 *s_fast = reinterpret_cast<uint2 *>(smem);
    const uint32_t wbytes = warp_smem_bytes(prm.sbuf_bytes);
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    uint8_t *wbase = smem + (8u << prm.fast_bits) + warp * wbytes;
    const uint32_t bar_s0 = smem_u32(wbase), bar_m = bar_s0 + 16u, bar_t = smem_u32(smem + (8u << prm.fast_bits)) + 24u;
    uint8_t *wslots = wbase + 32;
    const uint32_t slot_bytes = 64u + prm.sbuf_bytes;
    uint8_t *mbuf = wslots + 2u * slot_bytes;
    const uint32_t exps0 = smem_u32(mbuf + GROUP_SYMS), exps = exps0 + 4u * lane;
    const uint32_t *g_hier = prm.lut + 2u * n_fast;
    const uint32_t kshift = 32u - prm.fast_bits;
    if (lane == 0u) {
        mbar_init(bar_s0, 1);
        mbar_init(bar_s0 + 8u, 1);
        mbar_init(bar_m, 1);
        if (tid == 0u) mbar_init(bar_t, 1);
        fence_mbar_init();
        if (tid == 0u) {
            mbar_expect_tx(bar_t, 8u << prm.fast_bits);
            bulk_load(smem_u32(s_fast), prm.lut, 8u << prm.fast_bits, bar_t);
        }
    }

    // a group of a token's row
    struct Item {
        uint64_t s0, s1;  // the group's bits
        uint32_t t, g;    // token, group
        int32_t from;     // the row's first weight, from the group's
    };
    // this warp's units are unit0, unit0 + stride, ...; the lanes look at the
    // next 32 at once: unit u is group u / tokens of token u mod tokens's row
    const uint32_t stride = gridDim.x * NWARP, all = p.ids.tokens * p.units;
    uint32_t next = warp * gridDim.x + blockIdx.x, my_row = 0, my_unit = 0, rows = 0, pads = 0;  // my_unit: token | group << 20
    auto advance = [&](Item &it) {
        while (!rows) {
            for (; pads; pads &= pads - 1u) {
                const uint32_t unit = __shfl_sync(0xFFFFFFFFu, my_unit, __ffs(pads) - 1), c0 = (unit >> 20) * GROUP_SYMS;
                zero_row(p.out + (unit & 0xFFFFFu) * p.ldo, c0, min(c0 + GROUP_SYMS, p.dim), lane);
            }
            if (next >= all) return false;
            const uint32_t u = next + lane * stride, part = u / p.ids.tokens, t = u - part * p.ids.tokens;
            next += 32u * stride;
            uint64_t row = 0;
            const bool have = u < all && token_row(p.ids, t, row, part == 0u);
            const uint64_t w0 = p.first + row * p.dim;
            my_row = (uint32_t)row;
            my_unit = t | part << 20;
            rows = __ballot_sync(0xFFFFFFFFu, have && (w0 / GROUP_SYMS + part) * GROUP_SYMS < w0 + p.dim);
            pads = __ballot_sync(0xFFFFFFFFu, u < all && !have);
        }
        const int from = __ffs(rows) - 1;
        rows &= rows - 1u;
        const uint32_t unit = __shfl_sync(0xFFFFFFFFu, my_unit, from);
        const uint64_t w0 = p.first + (uint64_t)__shfl_sync(0xFFFFFFFFu, my_row, from) * p.dim;
        it.t = unit & 0xFFFFFu;
        it.g = (uint32_t)(w0 / GROUP_SYMS) + (unit >> 20);
        it.from = (int32_t)(w0 % GROUP_SYMS) - (int32_t)(GROUP_SYMS * (unit >> 20));
        it.s0 = ld_after(prm.group_start + it.g);
        it.s1 = ld_after(prm.group_start + it.g + 1u);
        return true;
    };
    // lane 0: chunk bits and stream span into slot s / the raw bytes
    auto issue_stream = [&](const Item &it, uint32_t s) {
        uint8_t *slot = wslots + s * slot_bytes;
        const uint32_t bar = bar_s0 + 8u * s;
        const uint64_t sb0 = (it.s0 >> 3) & ~15ull, d = it.s1 - it.s0;
        uint32_t sbytes = 0;
        if (sb0 < prm.stream_bytes) {  // (a corrupt plan copies a full slot and is rejected before it is decoded)
            sbytes = min(span_bytes((uint32_t)it.s0 & 127u, d < (1u << 17) ? (uint32_t)d : (1u << 17)), prm.sbuf_bytes);
            sbytes = (uint32_t)min((uint64_t)sbytes, prm.stream_bytes - sb0);
        }
        const bool cb_ok = check(it.g < prm.n_groups, CK_EMBED_COPY);
        const bool st_ok = check(sbytes <= prm.sbuf_bytes && (sbytes == 0u || sb0 + sbytes <= prm.stream_bytes), CK_EMBED_COPY);
        fence_proxy_async();
        mbar_expect_tx(bar, (cb_ok ? 64u : 0u) + (st_ok ? sbytes : 0u));
        if (cb_ok) bulk_load(smem_u32(slot), prm.chunk_bits + (size_t)it.g * GROUP_CHUNKS, 64u, bar);
        if (st_ok && sbytes) bulk_load(smem_u32(slot + 64), prm.stream + sb0, sbytes, bar);
    };
    auto issue_mant = [&](const Item &it) {
        const uint64_t m0 = (uint64_t)it.g * GROUP_SYMS;
        const uint32_t bytes = (uint32_t)min((uint64_t)GROUP_SYMS, prm.mant_bytes - m0);
        const bool ok = check(m0 < prm.mant_bytes && m0 + bytes <= prm.mant_bytes, CK_EMBED_COPY);
        fence_proxy_async();
        mbar_expect_tx(bar_m, ok ? bytes : 0u);
        if (ok) bulk_load(smem_u32(mbuf), prm.mant + m0, bytes, bar_m);
    };
    Item cur = {}, nxt;
    bool live = advance(cur);
    if (live && lane == 0u) {
        issue_stream(cur, 0);
        issue_mant(cur);
    }
    nxt = cur;
    bool more = live && advance(nxt);

    __syncthreads();  // the table's barrier is initialised
    const bool tok = mbar_wait(bar_t, 0u);
    const bool bad = tok && check_fast_table<NT>(s_fast, n_fast, prm.fast_bits, (int)tid);
    const bool all_in = __syncthreads_and(tok);
    if (__syncthreads_or(bad || !all_in)) {  // a malformed table, or its copy never came: nothing is decoded
        if (tid == 0u) {
            atomicOr(&g_status, all_in ? ST_LUT : ST_TIMEOUT);
            if (!all_in) mbar_wait_bounded(bar_t, 0u);
        }
        if (live && lane == 0u) {  // the copies in flight land first
            mbar_wait(bar_s0, 0u);
            mbar_wait(bar_m, 0u);
        }
        return;
    }

    for (uint32_t k = 0; live; ++k) {
        const uint32_t s = k & 1u;
        const uint8_t *slot = wslots + s * slot_bytes;
        __syncwarp();  // every lane is done with the other slot
        if (more && lane == 0u) issue_stream(nxt, s ^ 1u);

        bool ok = mbar_wait(bar_s0 + 8u * s, (k >> 1) & 1u);
        const uint32_t cbits = reinterpret_cast<const uint16_t *>(slot)[lane];
        uint32_t incl = cbits;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= (uint32_t)d) incl += y;
        }
        const uint32_t excl = incl - cbits, gbits = __shfl_sync(0xFFFFFFFFu, incl, 31);
        const uint32_t c = cur.g * GROUP_CHUNKS + lane, n = chunk_weights(prm, c);
        const uint32_t r0 = (uint32_t)cur.s0 & 127u, span = span_bytes(r0, gbits);
        const bool valid = __all_sync(0xFFFFFFFFu, cur.s1 - cur.s0 == gbits && cbits <= 32u * LANE_SYMS && span <= prm.sbuf_bytes &&
                                                       ((cur.s0 >> 3) & ~15ull) + span <= prm.stream_bytes &&
                                                       (n != 0u || cbits == 0u));
        // the row's weights of the group: [lo, hi) of its 2048
        const uint32_t lo = (uint32_t)max(cur.from, 0), hi = (uint32_t)min(cur.from + (int32_t)p.dim, (int32_t)GROUP_SYMS);
        uint32_t err = 0;
        if (ok && valid && LANE_SYMS * lane < hi && LANE_SYMS * lane + n > lo) {  // the row touches this chunk
            const uint32_t r = r0 + excl;
            uint32_t rd_end, wr_end;
            const uint32_t to = decode_chunk(smem_u32(slot + 64), r, (int)(8u * n), smem_u32(s_fast), kshift, g_hier,
                                             prm.n_tables, exps, err, rd_end, wr_end);
            if (to != r + cbits) err |= ST_COUNT;
            check(rd_end <= smem_u32(wbase) + wbytes, CK_EMBED_READ);
            check(wr_end < exps + EXP_STRIDE * EXP_WORDS, CK_EMBED_READ);
        }
        Item ahead = nxt;
        const bool ahead_live = more && advance(ahead);
        ok = mbar_wait(bar_m, k & 1u) && ok;
        if (!__all_sync(0xFFFFFFFFu, ok)) {  // a bulk copy never completed: give up
            if (lane == 0u) {  // report, then give each copy in flight one more bounded wait
                atomicOr(&g_status, ST_TIMEOUT);
                mbar_wait_bounded(bar_s0 + 8u * s, (k >> 1) & 1u);
                mbar_wait_bounded(bar_m, k & 1u);
                if (more) mbar_wait_bounded(bar_s0 + 8u * (s ^ 1u), ((k + 1u) >> 1) & 1u);
            }
            return;
        }
        const bool good = valid && !__any_sync(0xFFFFFFFFu, err != 0u);
        if (!valid) {
            if (lane == 0u) atomicOr(&g_status, ST_RANGE);
        } else if (!good) {
            if (err) atomicOr(&g_status, err);
        } else {
            __syncwarp();  // the join reads other lanes' exponent slots
            uint16_t *out = p.out + (int64_t)(cur.t * p.ldo) - cur.from;
            const uint32_t mb = smem_u32(mbuf);
            switch (p.scale.kind) {
                case SCALE_ONE: join_row<SCALE_ONE, V>(p.scale, out, lo, hi, mb, exps0, lane); break;
                case SCALE_BF16: join_row<SCALE_BF16, V>(p.scale, out, lo, hi, mb, exps0, lane); break;
                default: join_row<SCALE_FP32, V>(p.scale, out, lo, hi, mb, exps0, lane);
            }
        }
        if (!more) break;
        __syncwarp();  // every lane has read the raw bytes
        if (lane == 0u) issue_mant(nxt);
        cur = nxt;
        nxt = ahead;
        more = ahead_live;
    }
}

// Rows of a scope with one exponent (no stream): raw bytes joined with it.
// Bound by memory: 8192 rows of 4096 take 14.3 us (7.0 TB/s, repeated rows from
// L2), one row 2.1.  (Whole batches without bounds only where they are
// 16 bytes wide: 4000 rows of 1001 4.7 us with bounds, 5.6 without, one row of
// 4096 2.4 and 2.1.  Eight accesses in flight: 15.7 us.)
template <ScaleKind KIND, int V>
__device__ __forceinline__ void single_row(const RowScale &s, const uint8_t *m, uint32_t E, uint16_t *out, uint32_t dim, uint32_t lane) {
    using Bytes = std::conditional_t<V == 8, uint2, uint8_t>;
    constexpr uint32_t U = 4, STEP = 32u * V;  // accesses in flight
    auto batch = [&](uint32_t c0, bool whole) {  // all loads, then all stores
        Bytes b[U];
#pragma unroll
        for (uint32_t i = 0; i < U; ++i)
            if (whole || c0 + i * STEP < dim) b[i] = ld_after(reinterpret_cast<const Bytes *>(m + c0 + i * STEP));
#pragma unroll
        for (uint32_t i = 0; i < U; ++i) {
            const uint32_t c = c0 + i * STEP;
            if (!whole && c >= dim) break;
            if constexpr (V == 8) {
                uint4 v;
                join4(E, b[i].x, v.x, v.y);
                join4(E, b[i].y, v.z, v.w);
                __stcs(reinterpret_cast<uint4 *>(out + c), scaled8<KIND>(v, s));
            } else {
                out[c] = scaled1<KIND>(join1(E & 0xFFu, b[i]), s);
            }
        }
    };
    uint32_t c = V * lane;
    for (; V == 8 && c + (U - 1u) * STEP < dim; c += U * STEP) batch(c, true);
    for (; c < dim; c += U * STEP) batch(c, false);
}

template <int V>
__global__ void __launch_bounds__(256) embed_single_rows(const RowsOfLanes p) {
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t E = rot_sym(p.single) * 0x01010101u, lane = threadIdx.x & 31u;
    for (uint32_t t = blockIdx.x * 8u + (threadIdx.x >> 5); t < p.ids.tokens; t += gridDim.x * 8u) {
        uint64_t row = 0;
        uint16_t *out = p.out + t * p.ldo;
        if (!token_row(p.ids, t, row, lane == 0u)) {
            zero_row(out, 0u, p.dim, lane);
            continue;
        }
        const uint8_t *m = p.lanes.mant + p.first + row * p.dim;
        switch (p.scale.kind) {
            case SCALE_ONE: single_row<SCALE_ONE, V>(p.scale, m, E, out, p.dim, lane); break;
            case SCALE_BF16: single_row<SCALE_BF16, V>(p.scale, m, E, out, p.dim, lane); break;
            default: single_row<SCALE_FP32, V>(p.scale, m, E, out, p.dim, lane);
        }
    }
}

// ------------------------------------------------------ the table's gradient

// Thread `me` of `all` zeroes its share of n bytes.
__device__ __forceinline__ void zero_span(uint8_t *p, uint64_t n, uint64_t me, uint64_t all) {
    const uint64_t head = min(n, (uint64_t)(-reinterpret_cast<uintptr_t>(p) & 31u));
    const uint64_t body = (n - head) >> 5, tail = n - head - (body << 5);
    if (me < head) p[me] = 0;
    if (me < tail) p[n - 1u - me] = 0;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    for (uint64_t i = me; i < body; i += all) stg256_cs(p + head + (i << 5), z, z);
}

// Sorting.  A cluster of C CTAs sorts a block of up to 1024 C IPT tokens by
// row, stably: up to 8 bits a pass from the lowest.  Each warp ranks its own run of
// tokens (equal digits of 32 tokens found by a ballot per bit: no atomics, a
// fixed order); each CTA puts its tokens in digit order in its own shared
// memory, and from there, with the other CTAs' digit counts read through
// distributed shared memory, in their places in the cluster's order: the
// remote writes of neighbouring lanes are then neighbours too (writing every
// token straight to its place: 65 us against 27 for 65536 tokens at that step).
// Tokens without a row get key `rows` and end up behind all others.
// PACK: key and place within the block fit 16 bits each and travel as one word.
// Bound by the issue of the one cluster's SMs and its barriers: 8192 tokens of
// 32000 rows 10.4 us, 65536 of 259 22.8 (8 SMs each).
constexpr uint32_t SORT_THREADS = 1024, SORT_WARPS = 32, SORT_STRIDE = 257;

struct SortParams {
    IdSource ids;
    uint32_t *keys, *pos;  // per block: sorted keys and the tokens they belong to
    uint32_t *joins;       // the two counters of JoinLists, cleared here
    uint32_t passes, bits;  // digits of a key and their width, at most 8
    uint32_t ctas;         // CTAs that sort; those past them zero the gradient
    uint8_t *fill;
    uint64_t fill_bytes;
};

template <int C, int IPT, bool PACK>
constexpr uint32_t sort_smem() {
    return SORT_WARPS * SORT_STRIDE * 4u + (256u + 256u + 32u) * 4u + SORT_THREADS * IPT * (PACK ? 4u : 8u) * (C > 1 ? 2u : 1u);
}

template <int C, int IPT, bool PACK>
__global__ void __launch_bounds__(SORT_THREADS, 1) grad_sort(const SortParams p) {
    constexpr uint32_t CAP = SORT_THREADS * IPT;
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t *cnt = reinterpret_cast<uint32_t *>(smem);  // [warp][digit], rows of SORT_STRIDE: a scan's reads hit 32 banks
    uint32_t *total = cnt + SORT_WARPS * SORT_STRIDE;    // this CTA's count of each digit
    uint32_t *shift_by = total + 256;                    // from a digit's place in this CTA's order to the cluster's
    uint32_t *sums = shift_by + 256;
    constexpr uint32_t WORDS = PACK ? CAP : 2u * CAP;
    uint32_t *s_key = sums + 32, *s_pos = s_key + CAP;                             // this CTA's part of the order
    uint32_t *l_key = C > 1 ? s_key + WORDS : s_key, *l_pos = l_key + CAP;  // this CTA's tokens in digit order
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const uint32_t rank = blockIdx.x % C, base = blockIdx.x * CAP, run = warp * 32u * IPT + lane;
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x >= p.ctas) {  // (whole clusters)
        zero_span(p.fill, p.fill_bytes, (uint64_t)(blockIdx.x - p.ctas) * SORT_THREADS + tid,
                  (uint64_t)(gridDim.x - p.ctas) * SORT_THREADS);
        return;
    }
    if (blockIdx.x == 0u && tid < 2u) p.joins[tid] = 0u;
    const uint32_t block = base - rank * CAP;  // the cluster's first token
    uint32_t key[IPT], pos[PACK ? 1 : IPT];  // PACK: key[j] holds both
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
        uint64_t row = p.ids.rows;
        const uint32_t t = base + run + 32u * j;
        key[j] = 0xFFFFFFFFu;  // behind every token
        if (t < p.ids.tokens) {
            key[j] = token_row(p.ids, t, row, true) ? (uint32_t)row : (uint32_t)p.ids.rows;
            if constexpr (PACK) key[j] = key[j] << 16 | (t - block);
        }
        if constexpr (!PACK) pos[j] = t;
    }
    for (uint32_t pass = 0; pass < p.passes; ++pass) {
        const uint32_t shift = p.bits * pass + (PACK ? 16u : 0u), mask = (1u << p.bits) - 1u;
        for (uint32_t i = lane; i < 256u; i += 32u) cnt[warp * SORT_STRIDE + i] = 0u;
        __syncwarp();
        uint32_t at[IPT];
#pragma unroll
        for (int j = 0; j < IPT; ++j) {
            const uint32_t d = (key[j] >> shift) & mask;
            uint32_t same = 0xFFFFFFFFu;
#pragma unroll
            for (uint32_t b = 0; b < 8u; ++b) {
                if (b >= p.bits) break;
                const uint32_t v = __ballot_sync(0xFFFFFFFFu, (d >> b) & 1u);
                same &= (d >> b) & 1u ? v : ~v;
            }
            uint32_t *c = cnt + warp * SORT_STRIDE + d;
            at[j] = *c + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (lane == __ffs(same) - 1u) *c += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        // offsets in (digit, warp) order: thread i takes digit i / 4, warps 8 (i mod 4) .. + 7
        uint32_t *mine = cnt + 8u * (tid & 3u) * SORT_STRIDE + (tid >> 2), sum = 0;
#pragma unroll
        for (uint32_t k = 0; k < 8u; ++k) {
            const uint32_t v = mine[k * SORT_STRIDE];
            mine[k * SORT_STRIDE] = sum;
            sum += v;
        }
        uint32_t four = sum;  // prefix over the digit's four threads
#pragma unroll
        for (uint32_t d = 1; d < 4u; d <<= 1) {
            const uint32_t z = __shfl_up_sync(0xFFFFFFFFu, four, d);
            if ((tid & 3u) >= d) four += z;
        }
        const uint32_t all4 = __shfl_sync(0xFFFFFFFFu, four, lane | 3u), warps_before = four - sum;
        // exclusive prefix over the digits of v, which every fourth thread holds for its digit
        auto before_digit = [&](uint32_t v) {
            uint32_t incl = v;
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                const uint32_t z = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                if (lane >= (uint32_t)d) incl += z;
            }
            __syncthreads();  // sums may still be read from the last call
            if (lane == 31u) sums[warp] = incl;
            __syncthreads();
            uint32_t w = sums[lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t z = __shfl_up_sync(0xFFFFFFFFu, w, d);
                if (lane >= (uint32_t)d) w += z;
            }
            w = __shfl_sync(0xFFFFFFFFu, w, (warp + 31u) & 31u);
            return (warp ? w : 0u) + incl - v;
        };
        const uint32_t here = before_digit(all4);
#pragma unroll
        for (uint32_t k = 0; k < 8u; ++k) mine[k * SORT_STRIDE] += here + warps_before;
        if (C > 1 && !(tid & 3u)) total[tid >> 2] = all4;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < IPT; ++j) {
            const uint32_t to = cnt[warp * SORT_STRIDE + ((key[j] >> shift) & mask)] + at[j];
            if (!check(to < CAP, CK_GRAD_SORT)) continue;
            l_key[to] = key[j];
            if constexpr (!PACK) l_pos[to] = pos[j];
        }
        if constexpr (C > 1) {
            cluster_sync();  // every CTA's counts are out, and its part of the last order has been read
            uint32_t v[C], everywhere = 0, earlier = 0;
            const uint32_t a = smem_u32(total + (tid >> 2));
#pragma unroll
            for (uint32_t r = 0; r < C; ++r) v[r] = ld_cluster(map_rank(a, r));
#pragma unroll
            for (uint32_t r = 0; r < C; ++r) {
                everywhere += v[r];
                if (r < rank) earlier += v[r];
            }
            const uint32_t there = before_digit(everywhere) + earlier;
            if (!(tid & 3u)) shift_by[tid >> 2] = there - here;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < IPT; ++j) {
                const uint32_t from = run + 32u * j, k = l_key[from];
                const uint32_t to = from + shift_by[(k >> shift) & mask], r = to / CAP, i = to % CAP;
                if (!check(r < C, CK_GRAD_SORT)) continue;
                st_cluster(map_rank(smem_u32(s_key + i), r), k);
                if constexpr (!PACK) st_cluster(map_rank(smem_u32(s_pos + i), r), l_pos[from]);
            }
            cluster_sync();
        } else {
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < IPT; ++j) {
            key[j] = s_key[run + 32u * j];
            if constexpr (!PACK) pos[j] = s_pos[run + 32u * j];
        }
        if constexpr (C == 1) __syncthreads();  // before the next pass writes
    }
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
        const uint32_t t = base + run + 32u * j;
        if (t < p.ids.tokens) {
            p.keys[t] = PACK ? key[j] >> 16 : key[j];
            p.pos[t] = PACK ? block + (key[j] & 0xFFFFu) : pos[PACK ? 0 : j];
        }
    }
}

// Zeroes a large gradient while the tokens are sorted: a programmatic
// dependent of the sort that starts beside it, and ends after it (so that what
// follows on the stream follows both).  A small one (FILL_BESIDE) is zeroed by
// CTAs of the sort's own launch; more of those would wait for each other, as a
// cluster's CTAs find fewer SMs (262 MB beside 8192 tokens: 55 us, 42 here,
// 6.2 TB/s).
constexpr uint64_t FILL_BESIDE = 4u << 20;

__global__ void __launch_bounds__(512) grad_zero(uint8_t *p, uint64_t n) {
    griddep_launch_dependents();
    zero_span(p, n, (uint64_t)blockIdx.x * blockDim.x + threadIdx.x, (uint64_t)gridDim.x * blockDim.x);
    griddep_wait();
}

// Joins sorted blocks into one order: a token's place is its place in its own
// block plus, for every other block, how many of its keys come before (equal
// keys of earlier blocks do, those of later ones do not).  LANES lanes share
// a token's blocks, each a binary search: a chain of loads from L2.
struct MergeParams {
    const uint32_t *keys, *pos;
    uint32_t *out_keys, *out_pos;
    uint32_t tokens, blocks, block;
};

template <int LANES>
__global__ void __launch_bounds__(256) grad_merge(const MergeParams p) {
    griddep_launch_dependents();
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
    if (sub == 0u && i < p.tokens && check(place < p.tokens, CK_GRAD_SORT)) {
        p.out_keys[place] = key;
        p.out_pos[place] = __ldg(p.pos + t);
    }
}

// Rows that begin in a window and go on in the next, for grad_join: joins[0]
// and joins[1] count two lists of such windows, those whose row ends within
// JOIN_FEW more windows (window | further windows << 24, at joins + 4) and the
// rest (at joins + 4 + windows).  Their order does not matter: each is joined
// by itself.
constexpr uint32_t JOIN_FEW = 8;

// Summing.  The sorted tokens are cut into windows of `window`; a thread
// walks a window with VEC columns, eight rows of dy in flight, and writes a
// row's sum when the next row's tokens begin.  A row whose tokens reach past
// the window leaves a partial sum instead (slot 0 if it came from the window
// before, else slot 1); grad_join adds those up in window order.  Bound by the
// loads' latency (20 warps an SM, each waiting for its eight rows): 8192 rows
// of 4096 bf16 19.7 us, 65536 of 1024 27 (5.0 TB/s).
struct ReduceParams {
    const uint32_t *keys, *pos;
    const void *dy;
    void *grad;
    float *partial;  // [windows][2][dim]
    uint32_t *joins;
    uint64_t ld_dy;
    uint32_t tokens, windows, window, dim, rows;
    uint32_t tpr;          // threads per window (a power of two)
    uint32_t col_blocks;
    uint32_t accumulate;
    float scale;
};

template <typename T, int N>
struct __align__(sizeof(T) * N) Pack {
    T v[N];
};

// VEC values of a row of dy as they are in memory: whole words, so that the
// rows in flight take no more registers than bytes.
template <typename T, int VEC>
struct Raw;
template <int VEC>
struct Raw<float, VEC> {
    Pack<float, VEC> p;
    __device__ __forceinline__ float get(int k) const { return p.v[k]; }
};
template <>
struct Raw<__nv_bfloat16, 1> {
    uint16_t p;
    __device__ __forceinline__ float get(int) const { return __uint_as_float((uint32_t)p << 16); }
};
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 p;
    __device__ __forceinline__ float get(int k) const {
        const uint32_t w = k < 2 ? p.x : k < 4 ? p.y : k < 6 ? p.z : p.w;
        return __uint_as_float(k & 1 ? w & 0xFFFF0000u : w << 16);
    }
};

// scale sum and scale sum + old, each rounded once.
template <typename OUT>
__device__ __forceinline__ OUT scaled(float scale, float sum) {
    if constexpr (sizeof(OUT) == 4) return scale * sum;
    else return __float2bfloat16_rn(mul_odd(scale, sum));
}
__device__ __forceinline__ float scaled_sum(float scale, float sum, float old) { return fmaf(scale, sum, old); }
__device__ __forceinline__ __nv_bfloat16 scaled_sum(float scale, float sum, __nv_bfloat16 old) {
    return __float2bfloat16_rn(fma_odd(scale, sum, __bfloat162float(old)));
}

// Writes (or adds) scale x sum to VEC columns of a row, rounded once; `size` is
// the gradient's, for the checks build.
template <typename OUT, int VEC>
__device__ __forceinline__ void put_row(void *grad, uint64_t at, const float (&acc)[VEC], float scale, bool add, uint64_t size) {
    if (!check(at + VEC <= size, CK_GRAD_STORE)) return;
    constexpr int N = VEC * sizeof(OUT) > 16 ? 16 / sizeof(OUT) : VEC;  // at most 16 bytes at once
#pragma unroll
    for (int i = 0; i < VEC; i += N) {
        Pack<OUT, N> *dst = reinterpret_cast<Pack<OUT, N> *>(static_cast<OUT *>(grad) + at + i);
        Pack<OUT, N> o;
        if (add) {
            o = *dst;
#pragma unroll
            for (int j = 0; j < N; ++j) o.v[j] = scaled_sum(scale, acc[i + j], o.v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) o.v[j] = scaled<OUT>(scale, acc[i + j]);
        }
        *dst = o;
    }
}

template <typename DY, typename OUT, int VEC>
__global__ void __launch_bounds__(128, 6) grad_reduce(const ReduceParams p) {
    constexpr int U = 8;  // rows in flight
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ uint32_t s_list[];  // keys, then positions, of the CTA's windows
    const uint32_t per = 128u / p.tpr;    // windows a CTA walks at once
    const uint32_t w0 = blockIdx.x / p.col_blocks * per, list = per * p.window;
    for (uint32_t i = threadIdx.x; i < list; i += 128u) {
        const uint64_t t = (uint64_t)w0 * p.window + i;
        const bool in = t < p.tokens;
        s_list[i] = in ? ld_after(p.keys + t) : 0xFFFFFFFFu;
        s_list[list + i] = in ? ld_after(p.pos + t) : 0u;
    }
    const uint32_t w = w0 + threadIdx.x / p.tpr;
    const uint32_t col = (blockIdx.x % p.col_blocks * p.tpr + threadIdx.x % p.tpr) * VEC;
    const bool live = w < p.windows && col < p.dim;
    const uint32_t i0 = w * p.window, n = live ? min(p.window, p.tokens - i0) : 0u;
    const uint32_t prev = live && i0 ? ld_after(p.keys + i0 - 1u) : 0xFFFFFFFFu;
    const uint32_t next = live && i0 + n < p.tokens ? ld_after(p.keys + i0 + n) : 0xFFFFFFFFu;
    __syncthreads();
    if (!live) return;
    const uint32_t *keys = s_list + threadIdx.x / p.tpr * p.window, *pos = keys + list;
    if (col == 0u && n == p.window) {
        const uint32_t tail = keys[n - 1u];
        if (tail < p.rows && tail == next && !(keys[0] == tail && prev == tail)) {
            uint32_t more = 1u;  // windows after this one that begin with the row
            bool on = true;
#pragma unroll
            for (uint32_t k = 2; k <= JOIN_FEW; ++k) {
                const uint64_t t = (uint64_t)(w + k) * p.window;
                on = on && t < p.tokens && ld_after(p.keys + min(t, (uint64_t)p.tokens - 1u)) == tail;
                more += on;
            }
            const uint32_t at = atomicAdd(p.joins + (more < JOIN_FEW ? 0 : 1), 1u);
            if (check(at < p.windows, CK_GRAD_PARTIAL)) p.joins[4u + (more < JOIN_FEW ? 0u : p.windows) + at] = more < JOIN_FEW ? w | more << 24 : w;
        }
    }
    const DY *dy = static_cast<const DY *>(p.dy) + col;
    float acc[VEC];
    uint32_t cur = 0xFFFFFFFFu;  // the row being summed
    bool first = true;           // it is the window's first
    auto flush = [&](bool last) {
        if (cur >= p.rows) return;
        const bool left = first && cur == prev, right = last && cur == next;
        if (left || right) {
            if (!check(w < p.windows && col + VEC <= p.dim, CK_GRAD_PARTIAL)) return;
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
            put_row<OUT, VEC>(p.grad, (uint64_t)cur * p.dim + col, acc, p.scale, p.accumulate != 0u, (uint64_t)p.rows * p.dim);
        }
    };
    for (uint32_t i = 0; i < n; i += U) {  // window is a multiple of U: keys past the last token read as no row
        Raw<DY, VEC> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (keys[i + u] < p.rows && check(pos[i + u] < p.tokens, CK_GRAD_READ)) v[u] = *reinterpret_cast<const Raw<DY, VEC> *>(dy + (uint64_t)pos[i + u] * p.ld_dy);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t key = keys[i + u];
            if (key != cur) {
                if (i + u) {
                    flush(false);
                    first = false;
                }
                cur = key;
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
            }
            if (cur < p.rows) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] += v[u].get(k);
            }
        }
    }
    flush(true);
}

// Adds the partial sums of the listed rows.  Few windows: a thread adds all
// of them for its VEC columns.  Many (a row that a good part of the tokens
// share): for 32 VEC columns at a time each warp adds every eighth window,
// then the eight sums are added in order.  Bound by the latency of three loads
// in a chain (list, key, sums): 9.2 us after 8192 rows of 4096, 14.3 after
// 65536 of 1024 into 259 rows.
template <typename OUT, int VEC>
__global__ void __launch_bounds__(256) grad_join(const ReduceParams p) {
    __shared__ float s_sum[8][32 * VEC];
    griddep_wait();
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t few = *reinterpret_cast<volatile uint32_t *>(p.joins), many = *reinterpret_cast<volatile uint32_t *>(p.joins + 1);
    const uint32_t narrow = (p.dim + 32u * VEC - 1u) / (32u * VEC), wide = (p.dim + 256u * VEC - 1u) / (256u * VEC);
    auto add = [&](float (&sum)[VEC], uint32_t k, uint32_t slot, uint32_t col) {
        const Pack<float, VEC> v = *reinterpret_cast<const Pack<float, VEC> *>(p.partial + ((uint64_t)k * 2u + slot) * p.dim + col);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[j] += v.v[j];
    };
    for (uint64_t item = blockIdx.x; item < (uint64_t)many * narrow; item += gridDim.x) {
        const uint32_t w = p.joins[4u + p.windows + (uint32_t)(item / narrow)];
        const uint32_t col = (uint32_t)(item % narrow) * 32u * VEC + lane * VEC, key = ld_after(p.keys + (uint64_t)(w + 1u) * p.window);
        // the last window that begins with the row: the windows that do come
        // first, so 32 probes at a time narrow it down
        uint32_t last = w + JOIN_FEW, over = p.windows;
        while (over - last > 1u) {
            const uint32_t step = (over - last + 31u) / 32u;
            const uint64_t probe = (uint64_t)last + (uint64_t)step * (lane + 1u);
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, probe < over && ld_after(p.keys + (probe < over ? probe : w) * p.window) == key);
            last += step * __popc(m);
            over = min(over, last + step);
        }
        float sum[VEC] = {};
        if (col < p.dim) {
#pragma unroll 8
            for (uint32_t k = w + warp; k <= last; k += 8u) add(sum, k, k == w ? 1u : 0u, col);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VEC; ++j) s_sum[warp][lane * VEC + j] = sum[j];
        __syncthreads();
        if (warp || col >= p.dim) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            for (uint32_t k = 1; k < 8u; ++k) sum[j] += s_sum[k][lane * VEC + j];
        put_row<OUT, VEC>(p.grad, (uint64_t)key * p.dim + col, sum, p.scale, p.accumulate != 0u, (uint64_t)p.rows * p.dim);
    }
    // (CTAs without an item of the first list begin here)
    const uint32_t busy = (uint32_t)((uint64_t)many * narrow % gridDim.x);
    for (uint64_t item = blockIdx.x >= busy ? blockIdx.x - busy : blockIdx.x + gridDim.x - busy; item < (uint64_t)few * wide;
         item += gridDim.x) {
        const uint32_t entry = p.joins[4u + (uint32_t)(item / wide)], w = entry & 0xFFFFFFu, more = entry >> 24;
        const uint32_t col = ((uint32_t)(item % wide) * 256u + threadIdx.x) * VEC;
        if (col >= p.dim) continue;
        const uint32_t key = ld_after(p.keys + (uint64_t)(w + 1u) * p.window);
        float sum[VEC] = {};
        add(sum, w, 1u, col);
        Pack<float, VEC> v[JOIN_FEW - 1];  // (all loads first; those past the row's windows read its last one again)
#pragma unroll
        for (uint32_t k = 1; k < JOIN_FEW; ++k)
            v[k - 1u] = *reinterpret_cast<const Pack<float, VEC> *>(p.partial + (uint64_t)(w + min(k, more)) * 2u * p.dim + col);
#pragma unroll
        for (uint32_t k = 1; k < JOIN_FEW; ++k) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum[j] += k <= more ? v[k - 1u].v[j] : 0.f;
        }
        put_row<OUT, VEC>(p.grad, (uint64_t)key * p.dim + col, sum, p.scale, p.accumulate != 0u, (uint64_t)p.rows * p.dim);
    }
}

// Few tokens (up to GRAD_FEW): one launch.  A CTA takes some rows of the
// gradient and 256 VEC columns, zeroes them, lists the tokens whose row it
// has, orders the list by (row, token), and sums each row's tokens in order.
// Against the sorting kernels: 33 tokens of 129 into 1000 rows 2.2 us (7.4),
// 128 of 4096 into 32000 rows 43.2 (50.9), 128 tokens that share one row 13.1
// (9.9): past 128 the shared row would cost more than the launches saved.
constexpr uint32_t GRAD_FEW = 128;

struct FewParams {
    IdSource ids;
    const void *dy;
    void *grad;
    uint64_t ld_dy;
    uint32_t dim, rows_per, col_blocks, accumulate;
    float scale;
};

template <typename DY, typename OUT, int VEC>
__global__ void __launch_bounds__(256) grad_few(const FewParams p) {
    constexpr int U = 8;  // rows in flight
    __shared__ uint32_t s_row[GRAD_FEW], s_tok[GRAD_FEW], s_row2[GRAD_FEW], s_tok2[GRAD_FEW], s_count[GRAD_FEW / 32];
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const uint64_t r0 = (uint64_t)(blockIdx.x / p.col_blocks) * p.rows_per, r1 = min(r0 + p.rows_per, p.ids.rows);
    const uint32_t c0 = blockIdx.x % p.col_blocks * 256u * VEC, col = c0 + tid * VEC;
    // the tokens of these rows, in order
    uint64_t row = 0;
    bool mine = false;
    if (tid < p.ids.tokens) mine = token_row(p.ids, tid, row, blockIdx.x == 0u) && row >= r0 && row < r1;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, mine);
    if (warp < GRAD_FEW / 32u && lane == 0u) s_count[warp] = __popc(m);
    if (!p.accumulate && p.col_blocks == 1u) {
        zero_span(reinterpret_cast<uint8_t *>(static_cast<OUT *>(p.grad) + r0 * p.dim), (r1 - r0) * p.dim * sizeof(OUT), tid, 256u);
    } else if (!p.accumulate && col < p.dim) {
        constexpr int N = VEC * sizeof(OUT) > 16 ? 16 / sizeof(OUT) : VEC;
        Pack<OUT, N> z;
#pragma unroll
        for (int j = 0; j < N; ++j) z.v[j] = OUT(0.f);
        OUT *dst = static_cast<OUT *>(p.grad) + r0 * p.dim + col;
        for (uint64_t r = r0; r < r1; ++r, dst += p.dim) {
#pragma unroll
            for (int j = 0; j < VEC; j += N) *reinterpret_cast<Pack<OUT, N> *>(dst + j) = z;
        }
    }
    __syncthreads();
    uint32_t n = 0, before = 0;
#pragma unroll
    for (uint32_t w = 0; w < GRAD_FEW / 32u; ++w) {
        if (w < warp) before += s_count[w];
        n += s_count[w];
    }
    if (mine) {
        const uint32_t at = before + __popc(m & ((1u << lane) - 1u));
        s_row[at] = (uint32_t)row;
        s_tok[at] = tid;
    }
    __syncthreads();
    if (n == 0u) return;
    if (tid < n) {  // place: entries with a lower row, or the same row and earlier
        const uint32_t r = s_row[tid];
        uint32_t place = 0;
        for (uint32_t j = 0; j < n; ++j) place += s_row[j] < r || (s_row[j] == r && j < tid) ? 1u : 0u;
        s_row2[place] = r;
        s_tok2[place] = s_tok[tid];
    }
    __syncthreads();
    if (col >= p.dim) return;
    const DY *dy = static_cast<const DY *>(p.dy) + col;
    float acc[VEC] = {};
    for (uint32_t i = 0; i < n; i += U) {
        Raw<DY, VEC> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < n) v[u] = *reinterpret_cast<const Raw<DY, VEC> *>(dy + (uint64_t)s_tok2[i + u] * p.ld_dy);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u >= n) break;
#pragma unroll
            for (int k = 0; k < VEC; ++k) acc[k] += v[u].get(k);
            const uint32_t r = s_row2[i + u];
            if (i + u + 1u < n && s_row2[i + u + 1u] == r) continue;
            put_row<OUT, VEC>(p.grad, (uint64_t)r * p.dim + col, acc, p.scale, p.accumulate != 0u, p.ids.rows * p.dim);
#pragma unroll
            for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
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
    p.scale = row_scale(scale);
    const bool vec = dim % 8u == 0u && ((reinterpret_cast<uintptr_t>(d_table) | reinterpret_cast<uintptr_t>(d_out)) & 15u) == 0u &&
                     (rows == 1u || ld_table % 8u == 0u) && (tokens == 1u || ld_out % 8u == 0u);
    p.parts = (dim + EMBED_PART - 1u) / EMBED_PART;
    return launch_with(vec ? embed_table_rows<8> : embed_table_rows<1>, (tokens * p.parts + 7u) / 8u, 256, 0, true, 1, s, p);
}

// One CTA shape and join width of embed_lanes_rows.
template <int NT, int V>
dfw_status launch_embed_groups(const RowsOfLanes &p, uint32_t smem, int sms, cudaStream_t s) {
    static int opted[16];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 16) return DFW_ECUDA;
    const auto fn = embed_lanes_rows<NT, V>;
    if (!opted[dev]) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MOST) != cudaSuccess) return DFW_ECUDA;
        opted[dev] = 1;
    }
    // one CTA per SM (more of the smallest shape, which serves long codewords): units go to all SMs first, then to more warps
    const uint64_t ctas = (uint64_t)sms * (NT == 32 ? SMEM_MOST / smem : 1u), units = (uint64_t)p.ids.tokens * p.units;
    return launch_with(fn, std::min(ctas, units), NT, smem, true, 1, s, p);
}

template <int V>
dfw_status launch_embed_width(const RowsOfLanes &p, int sms, cudaStream_t s) {
    const uint32_t table = 8u << p.lanes.fast_bits, warp = warp_smem_bytes(p.lanes.sbuf_bytes);
    // 32 warps per SM; fewer where their slots do not fit (long codewords; the
    // scope's longest group decides: 2048 weights of 23 bits among 131e6 of 2.6
    // make 8192 rows of 4096 97 us instead of 29.6, one row 20.8 instead of 6.1,
    // as every one-warp CTA copies and checks a table of its own)
    if (table + 32u * warp <= SMEM_MOST) return launch_embed_groups<1024, V>(p, table + 32u * warp, sms, s);
    if (table + 16u * warp <= SMEM_MOST) return launch_embed_groups<512, V>(p, table + 16u * warp, sms, s);
    return launch_embed_groups<32, V>(p, table + warp, sms, s);
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
    p.out = d_out;
    p.ldo = ld_out;
    p.dim = dim;
    p.single = table->single_symbol;
    p.scale = row_scale(scale);
    const bool out16 = (reinterpret_cast<uintptr_t>(d_out) & 15u) == 0u && (tokens == 1u || ld_out % 8u == 0u);
    const bool out32 = (reinterpret_cast<uintptr_t>(d_out) & 31u) == 0u && (tokens == 1u || ld_out % 16u == 0u);
    if (table->total_bits == 0u) {
        const uint64_t want = (tokens + 7u) / 8u;
        const bool vec = out16 && first % 8u == 0u && dim % 8u == 0u;
        return launch_with(vec ? embed_single_rows<8> : embed_single_rows<1>, std::min<uint64_t>(want, (uint64_t)sms * 8u), 256, 0,
                           true, 1, s, p);
    }
    const bool whole = first % GROUP_SYMS == 0u && (dim % GROUP_SYMS == 0u || GROUP_SYMS % dim == 0u);
    p.units = (dim + GROUP_SYMS - (whole ? 1u : 2u)) / GROUP_SYMS + (whole ? 0u : 1u);
    if (out32 && first % 16u == 0u && dim % 16u == 0u) return launch_embed_width<16>(p, sms, s);
    if (out16 && first % 8u == 0u && dim % 8u == 0u) return launch_embed_width<8>(p, sms, s);
    return launch_embed_width<1>(p, sms, s);
}

// How the gradient of more than GRAD_FEW tokens is cut: blocks of `block`
// tokens that a cluster sorts, windows of at most GRAD_WINDOW for summing.  The
// cut is the same on every device (it fixes the order of the sums and the
// size of the scratch), made for 148 SMs.
constexpr uint32_t GRAD_WINDOW = 128;
struct GradCut {
    uint32_t ctas, ipt, block, blocks, window, windows;
    uint32_t joins;  // bytes of the joins lists
    uint64_t list;   // bytes of one array of keys or positions
};

GradCut grad_cut(uint64_t tokens, uint32_t dim) {
    GradCut c;
    c.ctas = tokens <= 1024u ? 1u : 8u;
    c.ipt = tokens <= 8192u ? 1u : tokens <= 32768u ? 4u : 8u;
    c.block = SORT_THREADS * c.ctas * c.ipt;
    c.blocks = (uint32_t)((tokens + c.block - 1u) / c.block);
    // Windows such that the summing CTAs (128 threads of 8 columns, 6 to an SM
    // of 148) all run at once where windows of 16 (64 for many tokens) to 128
    // allow it: a second, almost empty round of CTAs would double the time.
    // (65536 x 1024: 65.1 us with windows of 80, 72.8 with 64; 60000 x 64: 44.4
    // with 64, 49.1 with 16, whose partial sums outweigh the shorter walks.)
    uint64_t threads = 8u;
    while (threads < 128u && threads * 8u < dim) threads *= 2u;
    threads *= (dim + 8u * threads - 1u) / (8u * threads);
    const uint64_t window = (tokens * threads + 128u * 888u - 1u) / (128u * 888u);
    static_assert(GRAD_WINDOW <= GRAD_FEW, "at least two windows: there is always something that may have to be joined");
    c.window = (uint32_t)std::min<uint64_t>(GRAD_WINDOW, std::max<uint64_t>(tokens <= 1024u ? 8u : tokens <= 16384u ? 16u : 64u, (window + 7u) & ~7ull));
    c.windows = (uint32_t)((tokens + c.window - 1u) / c.window);
    c.list = (tokens * 4u + 15u) & ~15ull;
    c.joins = ((4u + 2u * c.windows) * 4u + 15u) & ~15u;
    return c;
}

uint64_t embed_grad_scratch(uint64_t tokens, uint32_t dim) {
    if (tokens <= GRAD_FEW) return 0u;
    const GradCut c = grad_cut(tokens, dim);
    return c.joins + c.list * (c.blocks > 1u ? 4u : 2u) + (uint64_t)c.windows * 2u * dim * 4u;
}

template <int C, int IPT, bool PACK>
dfw_status launch_grad_sort(SortParams p, uint32_t blocks, cudaStream_t s) {
    static int opted[16];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 16) return DFW_ECUDA;
    constexpr uint32_t smem = sort_smem<C, IPT, PACK>();
    if (!opted[dev]) {
        if (cudaFuncSetAttribute(grad_sort<C, IPT, PACK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return DFW_ECUDA;
        opted[dev] = 1;
    }
    p.ctas = blocks * C;
    const uint64_t fillers = (p.fill_bytes + (1u << 16) - 1u) >> 16;  // 64 KB each, in whole clusters
    return launch_with(grad_sort<C, IPT, PACK>, p.ctas + (fillers + C - 1u) / C * C, SORT_THREADS, smem, true, C, s, p);
}
template <bool PACK>
dfw_status launch_grad_sort(const SortParams &p, const GradCut &cut, cudaStream_t s) {
    if (cut.ctas == 1u) return launch_grad_sort<1, 1, PACK>(p, cut.blocks, s);
    if (cut.ipt == 1u) return launch_grad_sort<8, 1, PACK>(p, cut.blocks, s);
    if (cut.ipt == 4u) return launch_grad_sort<8, 4, PACK>(p, cut.blocks, s);
    return launch_grad_sort<8, 8, PACK>(p, cut.blocks, s);
}

template <typename DY, typename OUT, int V>
dfw_status launch_grad_reduce(ReduceParams p, int sms, cudaStream_t s) {
    const uint32_t threads = (p.dim + V - 1u) / V;
    p.tpr = 8u;
    while (p.tpr < 128u && p.tpr < threads) p.tpr *= 2u;
    p.col_blocks = (threads + p.tpr - 1u) / p.tpr;
    const uint64_t per = 128u / p.tpr;
    dfw_status st = launch_with(grad_reduce<DY, OUT, V>, (p.windows + per - 1u) / per * p.col_blocks, 128, per * p.window * 8u,
                                true, 1, s, p);
    if (st != DFW_OK) return st;
    constexpr uint32_t J = V > 4 ? 4 : V;
    const uint64_t most = (uint64_t)(p.windows - 1u) * ((p.dim + 32u * J - 1u) / (32u * J));
    return launch_with(grad_join<OUT, (int)J>, std::min<uint64_t>(most, (uint64_t)sms * 8u), 256, 0, true, 1, s, p);
}

template <typename DY, typename OUT, int V>
dfw_status launch_grad_few(FewParams p, int sms, cudaStream_t s) {
    p.col_blocks = (p.dim + 256u * V - 1u) / (256u * V);
    // about eight CTAs per SM, of 8 KB at least
    const uint64_t most = std::max<uint64_t>(1u, (uint64_t)sms * 8u / p.col_blocks), row_bytes = (uint64_t)std::min(p.dim, 256u * V) * sizeof(OUT);
    p.rows_per = (uint32_t)std::max((p.ids.rows + most - 1u) / most, ((uint64_t)8192u + row_bytes - 1u) / row_bytes);
    return launch_with(grad_few<DY, OUT, V>, (p.ids.rows + p.rows_per - 1u) / p.rows_per * p.col_blocks, 256, 0, true, 1, s, p);
}

// Calls f<DY, OUT, VEC>(p, sms, s) for the call's types and alignment.
#define DFW_GRAD_DISPATCH(f)                                                                                                      \
    (vec ? (dy_fp32 ? (grad_fp32 ? f<float, float, 4>(p, sms, s) : f<float, __nv_bfloat16, 4>(p, sms, s))                         \
                    : (grad_fp32 ? f<__nv_bfloat16, float, 8>(p, sms, s) : f<__nv_bfloat16, __nv_bfloat16, 8>(p, sms, s)))        \
         : (dy_fp32 ? (grad_fp32 ? f<float, float, 1>(p, sms, s) : f<float, __nv_bfloat16, 1>(p, sms, s))                         \
                    : (grad_fp32 ? f<__nv_bfloat16, float, 1>(p, sms, s) : f<__nv_bfloat16, __nv_bfloat16, 1>(p, sms, s))))

dfw_status launch_embed_grad(const void *d_ids, int ids64, uint64_t tokens, const void *d_dy, int dy_fp32,
                             uint64_t ld_dy, uint64_t rows, uint32_t dim, float scale, void *d_grad, int grad_fp32,
                             int accumulate, void *d_scratch, uint64_t scratch_bytes, cudaStream_t s) {
    SortParams sp;
    dfw_status st = ids_checked(d_ids, ids64, tokens, rows, sp.ids);
    if (st != DFW_OK) return st;
    if (dim < 1u || dim > DFW_EMBED_MAX_DIM || !d_grad || (tokens && !d_dy) || (tokens > GRAD_FEW && !d_scratch) ||
        (tokens > 1u && ld_dy < dim) ||
        (dy_fp32 | grad_fp32 | accumulate) & ~1)
        return DFW_EINVAL;
    if ((reinterpret_cast<uintptr_t>(d_dy) & (dy_fp32 ? 3u : 1u)) || (reinterpret_cast<uintptr_t>(d_grad) & (grad_fp32 ? 3u : 1u)) ||
        (reinterpret_cast<uintptr_t>(d_scratch) & 15u))
        return DFW_EALIGN;
    if (scratch_bytes < embed_grad_scratch(tokens, dim)) return DFW_ENOMEM;
    if (tokens == 0u && accumulate) return DFW_OK;
    int sms = 0;
    if ((st = device_sms(sms)) != DFW_OK) return st;
    // 16-byte loads where every row of dy, and every piece of a gradient row, is aligned for them
    const bool vec = dim % 8u == 0u && ((reinterpret_cast<uintptr_t>(d_dy) | reinterpret_cast<uintptr_t>(d_grad)) & 15u) == 0u &&
                     (tokens <= 1u || ld_dy * (dy_fp32 ? 4u : 2u) % 16u == 0u);
    if (tokens && tokens <= GRAD_FEW) {
        FewParams p = {sp.ids, d_dy, d_grad, ld_dy, dim, 0u, 0u, (uint32_t)accumulate, scale};
        return DFW_GRAD_DISPATCH(launch_grad_few);
    }
    uint8_t *const fill = static_cast<uint8_t *>(d_grad);
    const uint64_t fill_bytes = accumulate ? 0u : rows * dim * (grad_fp32 ? 4u : 2u);
    const uint64_t fillers = std::min<uint64_t>((fill_bytes + (1u << 14) - 1u) >> 14, (uint64_t)sms * 4u);
    if (tokens == 0u) return launch_with(grad_zero, fillers, 512, 0, false, 1, s, fill, fill_bytes);
    const GradCut cut = grad_cut(tokens, dim);
    uint8_t *const scratch = static_cast<uint8_t *>(d_scratch);
    uint32_t *lists[4];
    for (int i = 0; i < 4; ++i) lists[i] = reinterpret_cast<uint32_t *>(scratch + cut.joins + i * cut.list);
    sp.keys = lists[0];
    sp.pos = lists[1];
    sp.joins = reinterpret_cast<uint32_t *>(scratch);
    uint32_t key_bits = 1u;
    while (rows >> key_bits) ++key_bits;  // keys go up to `rows`
    sp.passes = (key_bits + 7u) / 8u;
    sp.bits = (key_bits + sp.passes - 1u) / sp.passes;
    sp.fill = fill;
    sp.fill_bytes = fill_bytes <= FILL_BESIDE ? fill_bytes : 0u;
    st = key_bits <= 16u ? launch_grad_sort<true>(sp, cut, s) : launch_grad_sort<false>(sp, cut, s);
    if (st != DFW_OK) return st;
    if (fill_bytes > FILL_BESIDE && (st = launch_with(grad_zero, fillers, 512, 0, true, 1, s, fill, fill_bytes)) != DFW_OK) return st;
    ReduceParams p;
    p.keys = lists[0];
    p.pos = lists[1];
    if (cut.blocks > 1u) {
        MergeParams m = {lists[0], lists[1], lists[2], lists[3], (uint32_t)tokens, cut.blocks, cut.block};
        if ((st = launch_with(grad_merge<16>, (tokens * 16u + 255u) / 256u, 256, 0, false, 1, s, m)) != DFW_OK) return st;
        p.keys = lists[2];
        p.pos = lists[3];
    }
    p.dy = d_dy;
    p.grad = d_grad;
    p.partial = reinterpret_cast<float *>(scratch + cut.joins + (cut.blocks > 1u ? 4u : 2u) * cut.list);
    p.joins = sp.joins;
    p.ld_dy = ld_dy;
    p.tokens = (uint32_t)tokens;
    p.windows = cut.windows;
    p.window = cut.window;
    p.dim = dim;
    p.rows = (uint32_t)rows;
    p.accumulate = (uint32_t)accumulate;
    p.scale = scale;
    return DFW_GRAD_DISPATCH(launch_grad_reduce);
}
#undef DFW_GRAD_DISPATCH

}  // namespace dfw
