// dfw_q4.cuh -- 4-bit weights with group scales and their products with a few
// vectors (included by dfw_decode.cu only).  The lossy neighbour of the fused
// decode + matrix-vector product: the LazyWeights write-up's weights are
// group-quantised integers, these are the same numbers without the Huffman
// code, 4.1 to 4.8 bits per weight instead of 10.6.
//
// w[n, k] = s[n, k / G] (q[n, k] - z[n, k / G]), q and z whole numbers 0..15,
// s bf16; z = 8 everywhere when the matrix has no zero points.
//
// Layout.  A tile is 16 rows x 128 columns, stored as one contiguous piece:
//   1024 bytes of codes: row half h (rows 8 h + g), lane l = 4 g + t, word w
//        (0..3) at 512 h + 16 l + 4 w holds row 8 h + g, columns 32 w + 8 t +
//        0..7: the even ones in its low half, the odd ones in its high half,
//        so that one mask takes two neighbours into a register's two halves.
//        A lane of the multiplying warp thus gets one 16-byte load per row
//        half, a warp's load is 512 contiguous bytes, and word w of every lane
//        lies in columns 32 w .. 32 w + 31, so each matrix instruction stays
//        inside one group even at G = 32;
//   32 GT bytes of scales (GT = 128 / G groups): row r's GT bf16 at 2 GT r;
//   16 GT bytes of zero points, if any: row r's GT bytes at GT r.
// Tiles follow each other along the columns, then down the rows.  Rows and
// columns past the matrix's end hold code 8 (0 with zero points), scale and
// zero point 0, so they contribute exactly 0.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>

#include "dfw_lanes.cuh"

namespace dfw {
namespace {

// ------------------------------------------------------- clusters and launches

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared word `a` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// A launch that may be a programmatic dependent of the one before, whichever
// that is, or run in clusters.  A dependent is set up while the one before
// still runs and waits for its end (griddep_wait) before it touches memory; it
// lets its own dependents be set up only after that wait, so that none of them
// runs beside anything earlier.  A stream of calls gains 2 us on each (4096 x
// 14336 products 18.7 -> 16.7 us, 8192 coded rows 33.8 -> 31.6).
template <typename F, typename... A>
dfw_status launch_with(F fn, uint64_t grid, unsigned block, uint32_t smem, bool dependent, unsigned cluster, cudaStream_t s,
                       A... args) {
    if (grid > 0x7FFFFFFFull) return DFW_EINVAL;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    cfg.numAttrs = 0;
    if (dependent) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1u) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = cluster;
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    return cudaLaunchKernelEx(&cfg, fn, args...) == cudaSuccess ? DFW_OK : DFW_ECUDA;
}

constexpr uint32_t SMEM_MOST = 227u * 1024u;  // a CTA's largest shared memory

// ----------------------------------------------------------------- 4-bit tiles

constexpr uint32_t Q4_ROWS = 16, Q4_COLS = 128, Q4_CODES = 1024;

struct Q4Params {
    uint32_t rows, cols, col_tiles, gt, zeros, tile_bytes;
    uint64_t row_tiles;
};

__host__ __device__ __forceinline__ uint32_t q4_tile_bytes(uint32_t gt, uint32_t zeros) {
    return Q4_CODES + 32u * gt + (zeros ? 16u * gt : 0u);
}

// The 32-bit word of codes for (row, 8 columns from col) inside a tile.
__device__ __forceinline__ uint32_t q4_word_at(uint32_t r, uint32_t c) {
    return 512u * (r >> 3) + 16u * (4u * (r & 7u) + ((c >> 3) & 3u)) + 4u * (c >> 5);
}

__device__ __forceinline__ uint4 ldg_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Eight codes in column order (column i in bits 4 i .. 4 i + 3) -> even ones
// in the low half, odd ones in the high half.
__device__ __forceinline__ uint32_t q4_split(uint32_t w) {
    uint32_t e = w & 0x0F0F0F0Fu, o = (w >> 4) & 0x0F0F0F0Fu;
    e = (e | e >> 4) & 0x00FF00FFu;
    o = (o | o >> 4) & 0x00FF00FFu;
    return ((e | e >> 8) & 0xFFFFu) | (o | o >> 8) << 16;
}

// Row-major codes (two to a byte, even column in the low half), scales and
// zero points -> tiles.  One thread per word of codes; the first threads of a
// tile also place its scales and zero points.  (Here and in the next two a
// CTA walks tiles of one row tile: dividing a running tile number cost 0.3 to
// 0.7 ms on 128256 x 4096.)  Bound by instructions, which fill 70% of the
// issue slots and 64% of the integer pipe: 128256 x 4096 takes 141 us, 3.8 TB/s
// read and written.
__global__ void __launch_bounds__(256) q4_pack_tiles(const uint8_t *__restrict__ codes,
                                                     const uint16_t *__restrict__ scales,
                                                     const uint8_t *__restrict__ zeros, const Q4Params p,
                                                     uint8_t *__restrict__ out) {
    const uint32_t groups = p.cols * p.gt / Q4_COLS, r = threadIdx.x >> 4, c = 8u * (threadIdx.x & 15u);
    const uint64_t r0 = (uint64_t)blockIdx.x * Q4_ROWS;
    auto load = [&](uint32_t ct) {
        const uint32_t col = ct * Q4_COLS + c;
        if (ct >= p.col_tiles || r0 + r >= p.rows || col >= p.cols) return p.zeros ? 0u : 0x88888888u;
        return __ldg(reinterpret_cast<const uint32_t *>(codes + ((r0 + r) * p.cols + col) / 2u));
    };
    uint32_t next = load(blockIdx.y), after = load(blockIdx.y + gridDim.y);
    for (uint32_t ct = blockIdx.y; ct < p.col_tiles; ct += gridDim.y) {
        const uint32_t c0 = ct * Q4_COLS, word = next;
        next = after;
        after = load(ct + 2u * gridDim.y);
        uint8_t *dst = out + (blockIdx.x * (uint64_t)p.col_tiles + ct) * p.tile_bytes;
        *reinterpret_cast<uint32_t *>(dst + q4_word_at(r, c)) = q4_split(word);
        if (threadIdx.x < Q4_ROWS * p.gt) {
            const uint32_t rr = threadIdx.x / p.gt, gi = threadIdx.x % p.gt;
            const uint32_t gr = c0 * p.gt / Q4_COLS + gi;
            const bool in = r0 + rr < p.rows && gr < groups;
            reinterpret_cast<uint16_t *>(dst + Q4_CODES)[threadIdx.x] = in ? scales[(r0 + rr) * groups + gr] : (uint16_t)0;
            if (p.zeros)
                dst[Q4_CODES + 32u * p.gt + threadIdx.x] = in ? (uint8_t)(zeros[(r0 + rr) * groups + gr] & 15u) : (uint8_t)0;
        }
    }
}

// w / s rounded to the nearest whole number, ties to even, from r ~ 1 / s.
// Both are bf16: the quotient is a tie exactly or at least 1/1020 from one, so
// rounding the product to a multiple of 2^-11 first (by adding 6144) makes
// ties of ties and moves nothing across one; adding 1.5 2^23 then rounds to a
// whole number in the sum's low bits.  Where 1 / s overflows, divide.
template <bool DIVIDE>
__device__ __forceinline__ int q4_round(float w, float s, float r) {
    const float t = DIVIDE ? w / s : __fsub_rn(__fmaf_rn(w, r, 6144.f), 6144.f);
    return __float_as_int(__fadd_rn(t, 12582912.f)) - 0x4B400000;
}
template <bool DIVIDE>
__device__ __forceinline__ uint32_t q4_codes(const uint32_t (&u)[4], float s, float r, int zp) {
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // the word's halves hold the even and the odd columns
        const int a = min(max(q4_round<DIVIDE>(__uint_as_float(u[i] << 16), s, r) + zp, 0), 15);
        const int b = min(max(q4_round<DIVIDE>(__uint_as_float(u[i] & 0xFFFF0000u), s, r) + zp, 0), 15);
        word |= (uint32_t)a << (4 * i) | (uint32_t)b << (4 * i + 16);
    }
    return word;
}

// The larger of two bf16 in both halves, NaN if either is.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// bf16 weights -> tiles.  A thread takes a word's eight columns, sixteen
// threads a row of a tile, 16 / GT of them a group, whose extremes they find
// by shuffles.  The codes are those of the formula in include/dfw.h.  Bound by
// instructions, which fill 87% of the issue slots: 128256 x 4096 takes 505 us,
// 2.6 TB/s read and written, against
// 709 with the extremes of a thread's weights found in fp32 and the choice
// between product and division made per weight, 1384 with a division per weight.
__global__ void __launch_bounds__(256) q4_quantise_tiles(const uint16_t *__restrict__ w, uint64_t ldw, uint32_t vec,
                                                         const Q4Params p, uint8_t *__restrict__ out) {
    const uint32_t r = threadIdx.x >> 4, c = 8u * (threadIdx.x & 15u), span = 16u / p.gt;  // threads per group
    const uint64_t row = (uint64_t)blockIdx.x * Q4_ROWS + r;
    auto load = [&](uint32_t ct) {
        const uint32_t col = ct * Q4_COLS + c;
        if (ct >= p.col_tiles || row >= p.rows || col >= p.cols) return make_uint4(0u, 0u, 0u, 0u);
        const uint16_t *src = w + row * ldw + col;
        if (vec) return ldg_stream(src);
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = __ldg(src + i);
        return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    };
    uint4 next = load(blockIdx.y);
    for (uint32_t ct = blockIdx.y; ct < p.col_tiles; ct += gridDim.y) {
        const uint4 cur = next;
        next = load(ct + gridDim.y);
        const bool in = row < p.rows && ct * Q4_COLS + c < p.cols;
        const uint32_t u[4] = {cur.x, cur.y, cur.z, cur.w};
        uint32_t up = 0u, down = 0u;  // the largest w and the largest -w, at least 0, of the even and odd columns
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            up = max_bf16x2(up, u[i]);
            down = max_bf16x2(down, u[i] ^ 0x80008000u);
        }
        uint32_t most = max_bf16x2(__byte_perm(up, down, 0x5410), __byte_perm(up, down, 0x7632));  // w low, -w high
        for (uint32_t d = 1; d < span; d <<= 1) most = max_bf16x2(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
        const float hi = __uint_as_float(most << 16), lo = -__uint_as_float(most & 0xFFFF0000u);
        const bool bad = !(hi <= 3.4e38f && lo >= -3.4e38f);  // an infinity or NaN
        const float range = p.zeros ? __fsub_rn(hi / 15.f, lo / 15.f) : fmaxf(hi, -lo) / 7.f;
        const __nv_bfloat16 sb = __float2bfloat16_rn(bad ? __uint_as_float(0x7FC00000u) : range);
        const float s = __bfloat162float(sb), inv = 1.f / s;
        // a group whose scale is 0 (all zero, or too small for bf16) has codes
        // equal to its zero point; one with a NaN or infinity has scale NaN
        const bool live = s > 0.f, tiny = s < 0x1p-120f;
        int zp = p.zeros ? 0 : 8;
        if (p.zeros && live) zp = min(max(tiny ? q4_round<true>(-lo, s, inv) : q4_round<false>(-lo, s, inv), 0), 15);
        uint32_t word = (uint32_t)zp * 0x11111111u;
        if (live) word = tiny ? q4_codes<true>(u, s, inv, zp) : q4_codes<false>(u, s, inv, zp);
        uint8_t *dst = out + (blockIdx.x * (uint64_t)p.col_tiles + ct) * p.tile_bytes;
        *reinterpret_cast<uint32_t *>(dst + q4_word_at(r, c)) = in ? word : p.zeros ? 0u : 0x88888888u;
        if ((threadIdx.x & 15u) % span == 0u) {
            const uint32_t gi = (threadIdx.x & 15u) / span;
            reinterpret_cast<uint16_t *>(dst + Q4_CODES)[r * p.gt + gi] = in ? __bfloat16_as_ushort(sb) : (uint16_t)0;
            if (p.zeros) dst[Q4_CODES + 32u * p.gt + r * p.gt + gi] = in ? (uint8_t)zp : (uint8_t)0;
        }
    }
}

// Tiles -> bf16 weights s (q - z), rounded once (the product has 12 bits).
// Bound by HBM: 128256 x 4096 takes 264 us, 5.0 TB/s read and written.
__global__ void __launch_bounds__(256) q4_dequantise_tiles(const uint8_t *__restrict__ packed, const Q4Params p,
                                                           uint16_t *__restrict__ out) {
    const uint32_t r = threadIdx.x >> 4, c = 8u * (threadIdx.x & 15u);
    const uint64_t row = (uint64_t)blockIdx.x * Q4_ROWS + r;
    if (row >= p.rows) return;
#pragma unroll 2
    for (uint32_t ct = blockIdx.y; ct < p.col_tiles; ct += gridDim.y) {
        const uint32_t col = ct * Q4_COLS + c;
        if (col >= p.cols) break;
        const uint8_t *src = packed + (blockIdx.x * (uint64_t)p.col_tiles + ct) * p.tile_bytes;
        const uint32_t word = __ldg(reinterpret_cast<const uint32_t *>(src + q4_word_at(r, c)));
        const uint32_t gi = c * p.gt / Q4_COLS;
        const float s = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(src + Q4_CODES)[r * p.gt + gi] << 16);
        const int z = p.zeros ? src[Q4_CODES + 32u * p.gt + r * p.gt + gi] : 8;
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = s * (float)((int)((word >> (4 * i)) & 15u) - z);
            const float b = s * (float)((int)((word >> (4 * i + 16)) & 15u) - z);
            v[i] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(a)) |
                   ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(b)) << 16);
        }
        *reinterpret_cast<uint4 *>(out + row * p.cols + col) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// y = W x.  The products run on the matrix instruction m16n8k16: a tile's 16
// rows are its rows, up to 8 vectors its columns (unused columns repeat the
// last vector and are dropped), so 1 to 8 vectors cost the same and the codes
// are expanded once for all.  Expanding is what the kernel is short of
// instructions for, so it takes two per pair of codes and half a shift: a
// masked code in bits 0..3 or 4..7 of a bf16 is the number q 2^-133 or
// 16 q 2^-133 (below 2^-125 a bf16's bits are a plain integer), so one
// multiply-add with 2^127 or 2^123 and -z / 64 gives (q - z) / 64, exact.  A
// group's products are summed by the instruction in fp32 before its scale
// multiplies the sum (a bf16 weight s (q - z) would round); the 64 multiplies
// the finished sum.
//
// A CTA takes consecutive row tiles, `pass` of them at a time, and its warps
// take equal runs of their tiles, whichever rows they fall in (giving each
// warp, or each few warps, whole row tiles left them unequal: 28672 rows are
// 12.1 row tiles per SM).  The next two tiles are on their way into the warp's
// ring in shared memory (asynchronous copies: tiles in flight in registers
// left room for half the warps).  A warp leaves its sums of each row tile it
// touched in shared memory; at the end of the pass they are added in the
// warps' order.  When the vectors are too long for one SM's shared memory, a
// cluster of 2 to 8 CTAs shares the columns and joins its sums the same way
// (no CTA of it is without column tiles: vectors that long have 34 of them for
// 2 CTAs, 59 for 4, 117 for 8).
// Up to 8 vectors take 32 warps of 64 registers, or 16 where their shared
// memory does not allow 32 or the CTA has few tiles; 9 to 16 have twice the
// sums and take 16.
//
// What bounds it: 128256 x 4096 with 4 vectors takes 48.1 us, 5.7 TB/s of the
// 6.5 a copy reaches; the same loop takes 46.1 us with neither expansion nor
// products, so the copies bound it (the shift in the expansion as a
// multiplication's high half, meant to spare the integer pipe, made that
// 54.5).  That holds below the power limit: such calls without a pause reach
// it, the clock falls to 1.64 to 1.73 GHz, and one takes 55 to 58 us.  Small
// matrices are bound by the chain of a launch, the first copies and the join:
// 1024 x 4096, one vector, 3.3 us, of which a launch of one tile takes 2.7;
// 6144 x 4096 7.0 us, 6.2 without the arithmetic.  In between, 16 warps an SM
// do not hide what each waits for: 4096 x 14336 with 16 vectors fills 45% of
// the issue slots (14.9 us), 4091 x 11008, G = 32, with 5 49% (12.1 us; some
// SMs have twice the row tiles of others).
constexpr uint32_t Q4_STEP = 2;                   // tiles a warp takes at a time
constexpr uint32_t Q4_JOIN_BYTES = 16u * 1024u;   // a CTA's buffer for its cluster's sums
// Steps in a warp's ring: three where 16 warps leave room for them.
__host__ __device__ constexpr uint32_t q4_ring(int nt, uint32_t warps) { return nt == 1 && warps == 16u ? 3u : 2u; }

struct Q4GemvParams {
    Q4Params q;
    const uint8_t *packed;
    const uint16_t *x;
    void *y;
    uint64_t ldx, ldy;
    uint32_t m, y_fp32;
    uint32_t split;    // CTAs along the columns (the cluster)
    uint32_t tiles;    // column tiles per CTA
    uint32_t pitch;    // bytes from one vector to the next in shared memory
    uint32_t pass;     // row tiles between two joins of the warps' sums
    uint32_t share, extra;  // row tiles per cluster, and how many clusters take one more
    uint32_t outs_inv; // ceil(2^32 / (16 m)): i / (16 m) is the high word of i times it (i below 2^24)
    uint32_t threads_log;  // log2 of the threads that copy a vector
    uint32_t xvec;     // the vectors can be read 16 bytes at a time
};

__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until all but this thread's N newest groups of copies have landed.
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// d = c + the products of a 16 x 16 and a 16 x 8 tile of bf16; `first`: c is 0.
__device__ __forceinline__ void mma_bf16(float (&d)[4], bool first, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    const float z = 0.f;
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(first ? z : d[0]), "f"(first ? z : d[1]),
          "f"(first ? z : d[2]), "f"(first ? z : d[3]));
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// A word's eight codes, less the zero point, over 64: columns 2 i and 2 i + 1
// in the halves of e[i].  off: -z / 64 in both halves.
__device__ __forceinline__ void q4_expand(uint32_t word, uint32_t off, uint32_t (&e)[4]) {
    constexpr uint32_t LOW = 0x7F007F00u, HIGH = 0x7D007D00u;  // 2^127, 2^123
    const uint32_t up = word >> 8;
    e[0] = fma_bf16x2(word & 0x000F000Fu, LOW, off);
    e[1] = fma_bf16x2(word & 0x00F000F0u, HIGH, off);
    e[2] = fma_bf16x2(up & 0x000F000Fu, LOW, off);
    e[3] = fma_bf16x2(up & 0x00F000F0u, HIGH, off);
}

// A tile as one lane takes it from the ring: its words of both row halves
// (from shared address cp, the tile + 16 lane), and the scales and zero points
// of rows g and g + 8 (from sp, the tile + 2 GT g).
template <int GT, bool Z>
struct Q4Tile {
    uint4 lo, hi;
    uint32_t s[GT == 4 ? 4 : 2];  // GT = 4: two words per row, else one
    uint32_t z[Z ? 2 : 1];
    __device__ __forceinline__ Q4Tile(uint32_t cp, uint32_t sp, uint32_t g) {
        const uint32_t zp = sp + Q4_CODES + 32u * GT - GT * g;
        lo = lds128(cp);
        hi = lds128(cp + 512u);
        sp += Q4_CODES;
        if constexpr (GT == 4) {
            s[0] = lds32(sp), s[1] = lds32(sp + 4u), s[2] = lds32(sp + 64u), s[3] = lds32(sp + 68u);
        } else if constexpr (GT == 2) {
            s[0] = lds32(sp), s[1] = lds32(sp + 32u);
        } else {
            s[0] = lds16(sp), s[1] = lds16(sp + 16u);
        }
        if constexpr (Z && GT == 4) z[0] = lds32(zp), z[1] = lds32(zp + 32u);
        if constexpr (Z && GT == 2) z[0] = lds16(zp), z[1] = lds16(zp + 16u);
        if constexpr (Z && GT == 1) z[0] = lds8(zp), z[1] = lds8(zp + 8u);
    }
    __device__ __forceinline__ float scale(int half, int gi) const {
        const uint32_t w = GT == 4 ? s[2 * half + (gi >> 1)] : s[half];
        return __uint_as_float(gi & 1 ? w & 0xFFFF0000u : w << 16);
    }
    __device__ __forceinline__ uint32_t offset(int half, int gi) const {  // -z / 64
        if constexpr (!Z) return 0xBE00BE00u;  // -8 / 64
        else return fma_bf16x2(((z[half] >> (8 * gi)) & 0xFu) * 0x10001u, 0xFF00FF00u, 0x80008000u);  // z 2^-133 x -2^127
    }
};

// acc += the tile's products with NT x 8 vectors, whose words for its columns
// start at shared address xs (+ 64 per word of codes, + nt_step per 8 vectors).
template <int GT, bool Z, int NT>
__device__ __forceinline__ void q4_tile_products(const Q4Tile<GT, Z> &b, uint32_t xs, uint32_t nt_step, float (&acc)[NT][4]) {
    const uint32_t lo[4] = {b.lo.x, b.lo.y, b.lo.z, b.lo.w}, hi[4] = {b.hi.x, b.hi.y, b.hi.z, b.hi.w};
#pragma unroll
    for (int gi = 0; gi < GT; ++gi) {
        float sum[NT][4];
        const uint32_t off0 = b.offset(0, gi), off1 = b.offset(1, gi);
#pragma unroll
        for (int w = gi * 4 / GT; w < (gi + 1) * 4 / GT; ++w) {
            uint32_t l[4], h[4];
            q4_expand(lo[w], off0, l);
            q4_expand(hi[w], off1, h);
            const bool first = w == gi * 4 / GT;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint4 x = lds128(xs + 64u * w + nt * nt_step);
                mma_bf16(sum[nt], first, l[0], h[0], l[1], h[1], x.x, x.y);
                mma_bf16(sum[nt], false, l[2], h[2], l[3], h[3], x.z, x.w);
            }
        }
        const float s0 = b.scale(0, gi), s1 = b.scale(1, gi);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            acc[nt][0] = fmaf(s0, sum[nt][0], acc[nt][0]);
            acc[nt][1] = fmaf(s0, sum[nt][1], acc[nt][1]);
            acc[nt][2] = fmaf(s1, sum[nt][2], acc[nt][2]);
            acc[nt][3] = fmaf(s1, sum[nt][3], acc[nt][3]);
        }
    }
}

__device__ __forceinline__ void q4_store(const Q4GemvParams &a, uint64_t row, uint32_t col, float v) {
    if (row >= a.q.rows || !check(col < a.m, CK_Q4_STORE)) return;
    v *= 64.f;
    if (a.y_fp32) static_cast<float *>(a.y)[col * a.ldy + row] = v;
    else static_cast<__nv_bfloat16 *>(a.y)[col * a.ldy + row] = __float2bfloat16_rn(v);
}

// Shared memory: the warps' rings | the sums of (warp, row tile), at index
// warp + row tile of the pass: in the order of the tiles each next pair has a
// larger one | the vectors | [clusters] the sums of the cluster's CTAs.
template <int GT, bool Z, int NT, uint32_t W, bool SPLIT>
__global__ void __launch_bounds__(32 * W, 1) q4_gemv_tiles(const Q4GemvParams a) {
    extern __shared__ __align__(16) uint8_t smem[];
    griddep_wait();
    griddep_launch_dependents();
    constexpr uint32_t TILE = Q4_CODES + 32u * GT + (Z ? 16u * GT : 0u), SLOT = Q4_STEP * TILE, RING = q4_ring(NT, W);
    const uint32_t outs = 16u * a.m;  // sums of a row tile, column by column
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3u;
    const uint32_t split = SPLIT ? a.split : 1u, rank = blockIdx.x % split, me = blockIdx.x / split;
    const uint32_t ct0 = rank * a.tiles, cts = min(a.tiles, a.q.col_tiles - ct0);
    const uint32_t rt0 = me * a.share + min(me, a.extra), rows = a.share + (me < a.extra ? 1u : 0u);  // row tiles
    const uint32_t ring = smem_u32(smem) + warp * RING * SLOT + 16u * lane;  // a lane's own place in it
    float *sums = reinterpret_cast<float *>(smem + W * RING * SLOT);
    uint8_t *vecs = reinterpret_cast<uint8_t *>(sums + (W + a.pass - 1u) * outs);
    float *join = reinterpret_cast<float *>(vecs + a.m * a.pitch);
    // this warp's tiles of a pass over `n` row tiles: [first(warp), first(warp + 1))
    auto first = [&](uint32_t w, uint32_t n) { return w * (n * cts) / W; };

    // tiles are copied in the order they are multiplied, a group of copies per
    // step (empty ones after the last, so that the newest RING - 1 groups are
    // always those ahead)
    uint32_t in_row = 0, in_left = 0, in_ct = 0, slot_in = ring;
    const uint8_t *src = nullptr;
    auto next_slot = [&](uint32_t slot) {
        return RING == 2u ? slot ^ ring ^ (ring + SLOT) : slot + SLOT == ring + RING * SLOT ? ring : slot + SLOT;
    };
    auto in_bounds = [&](uint32_t dst, const uint8_t *from) {  // of one 16-byte copy (checks build)
        return check(from >= a.packed && from + 16u <= a.packed + a.q.row_tiles * a.q.col_tiles * TILE &&
                         dst >= smem_u32(smem) + warp * RING * SLOT && dst + 16u <= smem_u32(smem) + (warp + 1u) * RING * SLOT,
                     CK_Q4_COPY);
    };
    auto fetch = [&]() {
        while (in_left == 0u && in_row < rows) {  // the next pass
            const uint32_t n = min(a.pass, rows - in_row), lo = first(warp, n);
            in_left = first(warp + 1u, n) - lo;
            in_ct = lo % cts;
            src = a.packed + ((uint64_t)(rt0 + in_row + lo / cts) * a.q.col_tiles + ct0 + in_ct) * TILE + 16u * lane;
            in_row += n;
        }
        if (in_left >= Q4_STEP && (!SPLIT || in_ct + Q4_STEP <= cts)) {  // a whole step, contiguous
#pragma unroll
            for (uint32_t at = 0; at < SLOT; at += 512u)
                if ((at + 512u <= SLOT || lane < (SLOT - at) / 16u) && in_bounds(slot_in + at, src + at))
                    cp_async16(slot_in + at, src + at);
            src += SLOT;
            in_left -= Q4_STEP;
            in_ct += Q4_STEP;
            if (SPLIT && in_ct == cts) {
                in_ct = 0;
                src += (uint64_t)(a.q.col_tiles - cts) * TILE;
            }
        } else {
            for (uint32_t u = 0; u < Q4_STEP && in_left; ++u) {
                const uint32_t dst = slot_in + u * TILE;
                if (in_bounds(dst, src)) cp_async16(dst, src);
                if (in_bounds(dst + 512u, src + 512)) cp_async16(dst + 512u, src + 512);
                if (lane < (TILE - Q4_CODES) / 16u && in_bounds(dst + Q4_CODES, src + Q4_CODES))
                    cp_async16(dst + Q4_CODES, src + Q4_CODES);
                src += TILE;
                if (SPLIT && ++in_ct == cts) {
                    in_ct = 0;
                    src += (uint64_t)(a.q.col_tiles - cts) * TILE;
                }
                --in_left;
            }
        }
        slot_in = next_slot(slot_in);
        cp_async_commit();
    };
#pragma unroll
    for (uint32_t u = 0; u + 1u < RING; ++u) fetch();

    // the vectors' columns [128 ct0, 128 (ct0 + cts)), zeros past the matrix; 2^log threads to a vector
    const uint32_t log = a.threads_log, v = threadIdx.x >> log;
    if (v < a.m) {
        const uint16_t *x = a.x + v * a.ldx + Q4_COLS * ct0;
        uint8_t *dst = vecs + v * a.pitch;
        const uint32_t here = (min(a.q.cols, Q4_COLS * (ct0 + cts)) - Q4_COLS * ct0) / 8u;
        for (uint32_t c = threadIdx.x & ((1u << log) - 1u); c < 16u * cts; c += 1u << log) {
            if (c >= here) {
                *reinterpret_cast<uint4 *>(dst + 16u * c) = make_uint4(0u, 0u, 0u, 0u);
            } else if (a.xvec) {
                cp_async16(smem_u32(dst + 16u * c), x + 8u * c);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) reinterpret_cast<uint16_t *>(dst + 16u * c)[j] = ld_after(x + 8u * c + j);
            }
        }
    }
    cp_async_commit();
    cp_async_wait<0>();
    if constexpr (SPLIT) cluster_sync();  // (and the other CTAs run: their shared memory can be written)
    else __syncthreads();

    const uint32_t x0 = smem_u32(vecs) + min(g, a.m - 1u) * a.pitch + 16u * t;
    const uint32_t nt_step = NT > 1 ? (min(g + 8u, a.m - 1u) - min(g, a.m - 1u)) * a.pitch : 0u;
    float acc[NT][4] = {};
    uint32_t slot = ring;
    auto put_away = [&](uint32_t row) {
        if (!check(warp + row < W + a.pass - 1u, CK_Q4_SUMS)) return;
        float *p = sums + (warp + row) * outs;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t col = 8u * nt + 2u * t + j;
                if (col < a.m) {
                    p[16u * col + g] = acc[nt][j];
                    p[16u * col + g + 8u] = acc[nt][2 + j];
                }
                acc[nt][j] = acc[nt][2 + j] = 0.f;
            }
        }
    };

    for (uint32_t done = 0; done < rows; done += a.pass) {
        const uint32_t n = min(a.pass, rows - done), lo = first(warp, n), hi = first(warp + 1u, n);
        uint32_t row = lo / cts, ct = lo - row * cts;
        for (uint32_t i = lo; i < hi; i += Q4_STEP) {
            cp_async_wait<(int)RING - 2>();
            __syncwarp();  // every lane's copies, and every lane is done with the slot that fetch() fills
            fetch();
#pragma unroll
            for (uint32_t u = 0; u < Q4_STEP; ++u) {
                if (i + u >= hi) break;
                const uint32_t cp = slot + u * TILE, sp = cp - 16u * lane + 2u * GT * g;
                q4_tile_products<GT, Z, NT>(Q4Tile<GT, Z>(cp, sp, g), x0 + 256u * ct, nt_step, acc);
                if (++ct == cts) {
                    put_away(row++);
                    ct = 0;
                }
            }
            slot = next_slot(slot);
        }
        if (ct || lo == hi) put_away(row);  // (a warp without tiles puts zeros between its neighbours' sums)
        __syncthreads();
        // row tile r's sums: those of the warps whose runs meet tiles [r cts,
        // (r + 1) cts), from the first that ends behind r cts
        const uint32_t tiles = n * cts, inv = 0xFFFFFFFFu / tiles;
        auto quotient = [&](uint32_t x) {  // x / tiles (x below 2^25: the estimate is at most one short)
            const uint32_t q = __umulhi(x, inv);
            return (q + 1u) * tiles <= x ? q + 1u : q;
        };
        for (uint32_t i = threadIdx.x; i < n * outs; i += 32u * W) {
            const uint32_t r = __umulhi(i, a.outs_inv), o = i - r * outs;
            const uint32_t w0 = quotient((r * cts + 1u) * W + tiles - 1u) - 1u, w1 = quotient((r + 1u) * cts * W + tiles - 1u);
            float v = 0.f;
#pragma unroll 8
            for (uint32_t w = w0; w < w1; ++w) v += sums[(w + r) * outs + o];
            if constexpr (!SPLIT) {
                q4_store(a, (uint64_t)Q4_ROWS * (rt0 + done + r) + (o & 15u), o >> 4, v);
            } else {
                const uint32_t at = (r / split * split + rank) * outs + o;
                if (check(at * 4u < Q4_JOIN_BYTES, CK_Q4_SUMS)) st_cluster_f32(map_rank(smem_u32(join + at), r % split), v);
            }
        }
        if constexpr (SPLIT) {  // row tile r of the pass is added up by CTA r mod split
            cluster_sync();
            for (uint32_t i = threadIdx.x;; i += 32u * W) {
                const uint32_t mine = __umulhi(i, a.outs_inv), r = rank + mine * split, o = i - mine * outs;
                if (r >= n) break;
                const float *p = join + (r / split) * split * outs + o;
                float v = p[0];
                for (uint32_t w = 1; w < split; ++w) v += p[w * outs];
                q4_store(a, (uint64_t)Q4_ROWS * (rt0 + done + r) + (o & 15u), o >> 4, v);
            }
            cluster_sync();
        } else {
            __syncthreads();
        }
    }
}

// The tile shape of a matrix; false if the shape is not supported.
bool q4_shape(const dfw_q4_info *info, Q4Params &p) {
    if (info->rows < 1u || info->rows > (1u << 30) || info->cols < 1u || info->cols > DFW_Q4_MAX_COLS || info->zeros > 1u ||
        (info->group != 32u && info->group != 64u && info->group != 128u) || info->cols % info->group)
        return false;
    p.rows = info->rows;
    p.cols = info->cols;
    p.col_tiles = (info->cols + Q4_COLS - 1u) / Q4_COLS;
    p.row_tiles = (info->rows + Q4_ROWS - 1u) / Q4_ROWS;
    p.gt = Q4_COLS / info->group;
    p.zeros = info->zeros;
    p.tile_bytes = q4_tile_bytes(p.gt, p.zeros);
    return true;
}

dfw_status q4_checked(const dfw_q4_info *info, const void *d_packed, Q4Params &p) {
    if (!info || !d_packed || !q4_shape(info, p) || info->bytes != p.row_tiles * p.col_tiles * p.tile_bytes)
        return DFW_EINVAL;
    return reinterpret_cast<uintptr_t>(d_packed) & 15u ? DFW_EALIGN : DFW_OK;
}

// The current device's multiprocessors (asked once per device).
dfw_status device_sms(int &sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 16) return DFW_ECUDA;
    if (!g_sms[dev] && cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return DFW_ECUDA;
    sms = g_sms[dev];
    return DFW_OK;
}

// A CTA per row tile, several where there are few row tiles.
dim3 q4_grid(const Q4Params &p, int sms) {
    const uint64_t want = ((uint64_t)sms * 16u + p.row_tiles - 1u) / p.row_tiles;
    return dim3((unsigned)p.row_tiles, (unsigned)std::min<uint64_t>(want, p.col_tiles));
}

}  // namespace

dfw_status launch_q4_pack(const uint8_t *d_codes, const uint16_t *d_scales, const uint8_t *d_zeros,
                          const dfw_q4_info *info, uint8_t *d_packed, cudaStream_t s) {
    Q4Params p;
    int sms = 0;
    dfw_status st = q4_checked(info, d_packed, p);
    if (st != DFW_OK) return st;
    if (!d_codes || !d_scales || (d_zeros != nullptr) != (p.zeros != 0u)) return DFW_EINVAL;
    if ((reinterpret_cast<uintptr_t>(d_codes) & 3u) || (reinterpret_cast<uintptr_t>(d_scales) & 1u)) return DFW_EALIGN;
    if ((st = device_sms(sms)) != DFW_OK) return st;
    q4_pack_tiles<<<q4_grid(p, sms), 256, 0, s>>>(d_codes, d_scales, d_zeros, p, d_packed);
    return cudaGetLastError() == cudaSuccess ? DFW_OK : DFW_ECUDA;
}

dfw_status launch_q4_quantise(const uint16_t *d_w, uint64_t ldw, const dfw_q4_info *info, uint8_t *d_packed,
                              cudaStream_t s) {
    Q4Params p;
    int sms = 0;
    dfw_status st = q4_checked(info, d_packed, p);
    if (st != DFW_OK) return st;
    if (!d_w || ldw < p.cols) return DFW_EINVAL;
    if (reinterpret_cast<uintptr_t>(d_w) & 1u) return DFW_EALIGN;
    const uint32_t vec = (reinterpret_cast<uintptr_t>(d_w) & 15u) == 0u && (p.rows == 1u || ldw % 8u == 0u);
    if ((st = device_sms(sms)) != DFW_OK) return st;
    q4_quantise_tiles<<<q4_grid(p, sms), 256, 0, s>>>(d_w, ldw, vec, p, d_packed);
    return cudaGetLastError() == cudaSuccess ? DFW_OK : DFW_ECUDA;
}

dfw_status launch_q4_dequantise(const uint8_t *d_packed, const dfw_q4_info *info, uint16_t *d_out, cudaStream_t s) {
    Q4Params p;
    int sms = 0;
    dfw_status st = q4_checked(info, d_packed, p);
    if (st != DFW_OK) return st;
    if (!d_out) return DFW_EINVAL;
    if (reinterpret_cast<uintptr_t>(d_out) & 15u) return DFW_EALIGN;
    if ((st = device_sms(sms)) != DFW_OK) return st;
    q4_dequantise_tiles<<<q4_grid(p, sms), 256, 0, s>>>(d_packed, p, d_out);
    return cudaGetLastError() == cudaSuccess ? DFW_OK : DFW_ECUDA;
}

namespace {

typedef void (*q4_fn)(const Q4GemvParams);
template <int GT, bool Z>
q4_fn q4_variant(int nt, uint32_t warps, bool split) {
    if (nt == 2) return split ? q4_gemv_tiles<GT, Z, 2, 16, true> : q4_gemv_tiles<GT, Z, 2, 16, false>;
    if (warps == 16u) return split ? q4_gemv_tiles<GT, Z, 1, 16, true> : q4_gemv_tiles<GT, Z, 1, 16, false>;
    return split ? q4_gemv_tiles<GT, Z, 1, 32, true> : q4_gemv_tiles<GT, Z, 1, 32, false>;
}
q4_fn q4_variant(const Q4Params &q, int nt, uint32_t warps, bool split) {
    switch (q.gt) {
        case 1: return q.zeros ? q4_variant<1, true>(nt, warps, split) : q4_variant<1, false>(nt, warps, split);
        case 2: return q.zeros ? q4_variant<2, true>(nt, warps, split) : q4_variant<2, false>(nt, warps, split);
        default: return q.zeros ? q4_variant<4, true>(nt, warps, split) : q4_variant<4, false>(nt, warps, split);
    }
}

dfw_status launch_q4_pass(Q4GemvParams a, int dev, int sms, cudaStream_t s) {
    const int nt = a.m > 8u ? 2 : 1;
    // as few CTAs to a row tile as their shared memory allows, then as many
    // warps, but 16 where a CTA has fewer than 256 tiles (4096 x 4096, 64 tiles:
    // 5.96 us with 16, 6.25 with 32; 65536 x 4096, 886 tiles: 30.9 and 29.4)
    const uint64_t row_share = (a.q.row_tiles + (uint64_t)sms - 1u) / (uint64_t)sms;
    uint32_t split = 1, warps = 0, smem = 0;
    for (; split <= 8u && !warps; split *= 2u) {
        const uint32_t tiles = (a.q.col_tiles + split - 1u) / split;
        a.pitch = tiles * 2u * Q4_COLS + 64u;  // neighbouring vectors 16 banks apart
        for (uint32_t w = nt == 1 && row_share * tiles >= 256u ? 32u : 16u; w >= 16u && !warps; w -= 16u) {
            smem = w * (q4_ring(nt, w) * Q4_STEP * a.q.tile_bytes + 64u * a.m) + a.m * a.pitch + (split > 1u ? Q4_JOIN_BYTES : 0u);
            if (smem <= SMEM_MOST) warps = w;
        }
    }
    split /= 2u;
    if (!warps) return DFW_EINVAL;  // (not reached: the caller bounds m by cols)
    const q4_fn fn = q4_variant(a.q, nt, warps, split > 1u);
    static bool opted[16][36];
    const uint32_t vi = (a.q.gt == 1u ? 0u : a.q.gt == 2u ? 1u : 2u) * 12u + a.q.zeros * 6u + (nt == 2 ? 2u : warps == 16u ? 1u : 0u) * 2u + (split > 1u ? 1u : 0u);
    if (!opted[dev][vi]) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MOST) != cudaSuccess) return DFW_ECUDA;
        opted[dev][vi] = true;
    }
    uint32_t ctas = (uint32_t)sms;
    if (split > 1u) {  // clusters that find room at once: not every SM can be in one
        static int room[16][2][9];  // by device, warps, cluster size (every variant fills an SM)
        int &fit = room[dev][warps / 16u - 1u][split];
        if (!fit) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(split);
            cfg.blockDim = dim3(32u * warps);
            cfg.dynamicSmemBytes = SMEM_MOST;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = split;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) return DFW_ECUDA;
            fit = n;
        }
        ctas = (uint32_t)fit * split;
    }
    a.split = split;
    a.tiles = (a.q.col_tiles + split - 1u) / split;
    const uint64_t clusters = std::min<uint64_t>(ctas / split, a.q.row_tiles);
    // as many row tiles to a pass as there is room for their sums
    const uint64_t rows = (a.q.row_tiles + clusters - 1u) / clusters;
    uint64_t room = 1u + (SMEM_MOST - smem) / (64u * a.m);
    if (split > 1u) room = std::min<uint64_t>(room, Q4_JOIN_BYTES / (64u * a.m) / split * split);
    a.pass = (uint32_t)std::min(rows, room);
    a.outs_inv = (uint32_t)(((1ull << 32) + 16u * a.m - 1u) / (16u * a.m));
    a.threads_log = warps == 32u ? 10u : 9u;
    for (uint32_t k = 1; k < a.m; k *= 2u) --a.threads_log;
    a.share = (uint32_t)(a.q.row_tiles / clusters);
    a.extra = (uint32_t)(a.q.row_tiles % clusters);
    smem += (a.pass - 1u) * 64u * a.m;
    return launch_with(fn, clusters * split, 32u * warps, smem, true, split, s, a);
}

}  // namespace

dfw_status launch_q4_gemv(const uint8_t *d_packed, const dfw_q4_info *info, uint32_t m, const uint16_t *d_x,
                          uint64_t ldx, void *d_y, int y_fp32, uint64_t ldy, cudaStream_t s) {
    Q4GemvParams a;
    int sms = 0, dev = 0;
    dfw_status st = q4_checked(info, d_packed, a.q);
    if (st != DFW_OK) return st;
    if (m > DFW_Q4_MAX_VECTORS || (m && (!d_x || !d_y)) || (m > 1u && (ldx < a.q.cols || ldy < a.q.rows)) ||
        (y_fp32 != 0 && y_fp32 != 1))
        return DFW_EINVAL;
    if ((reinterpret_cast<uintptr_t>(d_x) & 1u) || (reinterpret_cast<uintptr_t>(d_y) & (y_fp32 ? 3u : 1u))) return DFW_EALIGN;
    if (m == 0u) return DFW_OK;
    if ((st = device_sms(sms)) != DFW_OK) return st;
    if (cudaGetDevice(&dev) != cudaSuccess) return DFW_ECUDA;
    a.packed = d_packed;
    a.ldx = ldx;
    a.ldy = ldy;
    a.y_fp32 = (uint32_t)y_fp32;
    a.xvec = (reinterpret_cast<uintptr_t>(d_x) & 15u) == 0u && (m == 1u || ldx % 8u == 0u);
    // 16 vectors a pass, or 8 where 16 would not fit the eight CTAs of the largest cluster
    const uint32_t most = a.q.col_tiles <= 192u ? 16u : a.q.col_tiles <= 256u ? 8u : 4u;
    for (uint32_t j = 0; j < m; j += most) {
        a.m = std::min(most, m - j);
        a.x = d_x + j * ldx;
        a.y = static_cast<uint8_t *>(d_y) + j * ldy * (y_fp32 ? 4u : 2u);
        if ((st = launch_q4_pass(a, dev, sms, s)) != DFW_OK) return st;
    }
    return DFW_OK;
}

}  // namespace dfw
