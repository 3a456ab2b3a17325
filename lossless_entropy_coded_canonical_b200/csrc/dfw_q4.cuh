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
//        i in bits 4 i .. 4 i + 3.  A lane of the multiplying warp thus gets
//        one 16-byte load per row half, a warp's load is 512 contiguous
//        bytes, and word w of every lane lies in columns 32 w .. 32 w + 31, so
//        each matrix instruction stays inside one group even at G = 32;
//   32 GT bytes of scales (GT = 128 / G groups): row r's GT bf16 at 2 GT r;
//   16 GT bytes of zero points, if any: row r's GT bytes at GT r.
// Tiles follow each other along the columns, then down the rows.  Rows and
// columns past the matrix's end hold code 8 (0 with zero points), scale and
// zero point 0, so they contribute exactly 0.
#pragma once

#include <cuda_bf16.h>

#include "dfw_device.cuh"

namespace dfw {
namespace {

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

// Row-major codes (two to a byte, even column in the low half), scales and
// zero points -> tiles.  One thread per word of codes; the first threads of a
// tile also place its scales and zero points.
__global__ void __launch_bounds__(256) q4_pack_tiles(const uint8_t *__restrict__ codes,
                                                     const uint16_t *__restrict__ scales,
                                                     const uint8_t *__restrict__ zeros, const Q4Params p,
                                                     uint8_t *__restrict__ out) {
    const uint32_t groups = p.cols * p.gt / Q4_COLS;
    for (uint64_t tile = blockIdx.x; tile < p.row_tiles * p.col_tiles; tile += gridDim.x) {
        const uint64_t r0 = tile / p.col_tiles * Q4_ROWS;
        const uint32_t c0 = (uint32_t)(tile % p.col_tiles) * Q4_COLS;
        uint8_t *dst = out + tile * p.tile_bytes;
        const uint32_t r = threadIdx.x >> 4, c = 8u * (threadIdx.x & 15u);
        uint32_t word = p.zeros ? 0u : 0x88888888u;
        if (r0 + r < p.rows && c0 + c < p.cols)
            word = __ldg(reinterpret_cast<const uint32_t *>(codes + ((r0 + r) * p.cols + c0 + c) / 2u));
        *reinterpret_cast<uint32_t *>(dst + q4_word_at(r, c)) = word;
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

// bf16 weights -> tiles.  A warp takes a row's 128 columns, lane l columns
// 4 l .. 4 l + 3; a group's 32 / GT lanes find its extremes by shuffles.  The
// quotients are correctly rounded fp32 divisions, so the codes are those of
// the formula in include/dfw.h whatever the order of work.
__global__ void __launch_bounds__(512) q4_quantise_tiles(const uint16_t *__restrict__ w, uint64_t ldw, uint32_t vec,
                                                         const Q4Params p, uint8_t *__restrict__ out) {
    const uint32_t lane = threadIdx.x & 31u, r = threadIdx.x >> 5;
    const uint32_t span = 32u / p.gt;  // lanes per group
    for (uint64_t tile = blockIdx.x; tile < p.row_tiles * p.col_tiles; tile += gridDim.x) {
        const uint64_t row = tile / p.col_tiles * Q4_ROWS + r;
        const uint32_t col = (uint32_t)(tile % p.col_tiles) * Q4_COLS + 4u * lane;
        const bool in = row < p.rows && col < p.cols;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (in) {
            const uint16_t *src = w + row * ldw + col;
            uint32_t u[4];
            if (vec) {
                const uint2 q = __ldg(reinterpret_cast<const uint2 *>(src));
                u[0] = q.x << 16, u[1] = q.x & 0xFFFF0000u, u[2] = q.y << 16, u[3] = q.y & 0xFFFF0000u;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = (uint32_t)__ldg(src + i) << 16;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(u[i]);
        }
        float lo = 0.f, hi = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo = fminf(lo, v[i]);
            hi = fmaxf(hi, v[i]);
            bad |= !(fabsf(v[i]) <= 3.4e38f);  // infinities and NaN
        }
        for (uint32_t d = 1; d < span; d <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, d));
            hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, d));
            bad |= __shfl_xor_sync(0xFFFFFFFFu, (int)bad, d) != 0;
        }
        const float range = p.zeros ? __fsub_rn(hi / 15.f, lo / 15.f) : fmaxf(hi, -lo) / 7.f;
        const __nv_bfloat16 sb = __float2bfloat16_rn(bad ? __uint_as_float(0x7FC00000u) : range);
        const float s = __bfloat162float(sb);
        // a group whose scale is 0 (all zero, or too small for bf16) has codes
        // equal to its zero point; one with a NaN or infinity has scale NaN
        const bool live = s > 0.f;
        const float zp = p.zeros ? (live ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f) : 8.f;
        uint32_t half = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float q = live ? rintf(v[i] / s) + zp : zp;
            half |= (uint32_t)fminf(fmaxf(q, 0.f), 15.f) << (4 * i);
        }
        if (!in) half = p.zeros ? 0u : 0x8888u;
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, half, 1);
        uint8_t *dst = out + tile * p.tile_bytes;
        if (!(lane & 1u)) *reinterpret_cast<uint32_t *>(dst + q4_word_at(r, 4u * lane)) = half | (other << 16);
        if (lane % span == 0u) {
            const uint32_t gi = lane / span;
            reinterpret_cast<uint16_t *>(dst + Q4_CODES)[r * p.gt + gi] = in ? __bfloat16_as_ushort(sb) : (uint16_t)0;
            if (p.zeros) dst[Q4_CODES + 32u * p.gt + r * p.gt + gi] = in ? (uint8_t)zp : (uint8_t)0;
        }
    }
}

// Tiles -> bf16 weights s (q - z), rounded once (the product has 12 bits).
__global__ void __launch_bounds__(256) q4_dequantise_tiles(const uint8_t *__restrict__ packed, const Q4Params p,
                                                           uint16_t *__restrict__ out) {
    for (uint64_t tile = blockIdx.x; tile < p.row_tiles * p.col_tiles; tile += gridDim.x) {
        const uint32_t r = threadIdx.x >> 4, c = 8u * (threadIdx.x & 15u);
        const uint64_t row = tile / p.col_tiles * Q4_ROWS + r;
        const uint32_t col = (uint32_t)(tile % p.col_tiles) * Q4_COLS + c;
        if (row >= p.rows || col >= p.cols) continue;
        const uint8_t *src = packed + tile * p.tile_bytes;
        const uint32_t word = __ldg(reinterpret_cast<const uint32_t *>(src + q4_word_at(r, c)));
        const uint32_t gi = c * p.gt / Q4_COLS;
        const float s = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(src + Q4_CODES)[r * p.gt + gi] << 16);
        const int z = p.zeros ? src[Q4_CODES + 32u * p.gt + r * p.gt + gi] : 8;
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = s * (float)((int)((word >> (8 * i)) & 15u) - z);
            const float b = s * (float)((int)((word >> (8 * i + 4)) & 15u) - z);
            v[i] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(a)) |
                   ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(b)) << 16);
        }
        *reinterpret_cast<uint4 *>(out + row * p.cols + col) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

struct Q4GemvParams {
    Q4Params q;
    const uint8_t *packed;
    const uint16_t *x;
    void *y;
    uint64_t ldx, ldy;
    uint32_t m, y_fp32;
};

// y[m, n] = sum over groups of s (sum of (q - z) x), one thread per element.
__global__ void __launch_bounds__(256) q4_gemv_plain(const Q4GemvParams a) {
    const Q4Params &p = a.q;
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < (uint64_t)p.rows * a.m; i += gridDim.x * 256ull) {
        const uint32_t n = (uint32_t)(i % p.rows), m = (uint32_t)(i / p.rows), r = n % Q4_ROWS;
        const uint16_t *x = a.x + m * a.ldx;
        float y = 0.f;
        for (uint32_t ct = 0; ct < p.col_tiles; ++ct) {
            const uint8_t *tile = a.packed + ((uint64_t)(n / Q4_ROWS) * p.col_tiles + ct) * p.tile_bytes;
            const uint32_t span = Q4_COLS / p.gt;
            for (uint32_t gi = 0; gi < p.gt && ct * Q4_COLS + gi * span < p.cols; ++gi) {
                const float s = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(tile + Q4_CODES)[r * p.gt + gi] << 16);
                const int z = p.zeros ? tile[Q4_CODES + 32u * p.gt + r * p.gt + gi] : 8;
                float sum = 0.f;
                for (uint32_t c = gi * span; c < (gi + 1u) * span; c += 8u) {
                    const uint32_t word = *reinterpret_cast<const uint32_t *>(tile + q4_word_at(r, c));
                    for (uint32_t j = 0; j < 8u; ++j)
                        sum += (float)((int)((word >> (4u * j)) & 15u) - z) *
                               __uint_as_float((uint32_t)x[ct * Q4_COLS + c + j] << 16);
                }
                y += s * sum;
            }
        }
        if (a.y_fp32) static_cast<float *>(a.y)[m * a.ldy + n] = y;
        else static_cast<__nv_bfloat16 *>(a.y)[m * a.ldy + n] = __float2bfloat16_rn(y);
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

unsigned q4_grid(const Q4Params &p, int sms, unsigned per_sm) {
    const uint64_t tiles = p.row_tiles * p.col_tiles, cap = (uint64_t)sms * per_sm;
    return (unsigned)(tiles < cap ? tiles : cap);
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
    q4_pack_tiles<<<q4_grid(p, sms, 8), 256, 0, s>>>(d_codes, d_scales, d_zeros, p, d_packed);
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
    const uint32_t vec = (reinterpret_cast<uintptr_t>(d_w) & 7u) == 0u && ldw % 4u == 0u;
    if ((st = device_sms(sms)) != DFW_OK) return st;
    q4_quantise_tiles<<<q4_grid(p, sms, 4), 512, 0, s>>>(d_w, ldw, vec, p, d_packed);
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
    q4_dequantise_tiles<<<q4_grid(p, sms, 8), 256, 0, s>>>(d_packed, p, d_out);
    return cudaGetLastError() == cudaSuccess ? DFW_OK : DFW_ECUDA;
}

dfw_status launch_q4_gemv(const uint8_t *d_packed, const dfw_q4_info *info, uint32_t m, const uint16_t *d_x,
                          uint64_t ldx, void *d_y, int y_fp32, uint64_t ldy, cudaStream_t s) {
    Q4GemvParams a;
    int sms = 0;
    dfw_status st = q4_checked(info, d_packed, a.q);
    if (st != DFW_OK) return st;
    if (m > DFW_Q4_MAX_VECTORS || (m && (!d_x || !d_y)) || (m > 1u && (ldx < a.q.cols || ldy < a.q.rows)) ||
        (y_fp32 != 0 && y_fp32 != 1))
        return DFW_EINVAL;
    if ((reinterpret_cast<uintptr_t>(d_x) & 1u) || (reinterpret_cast<uintptr_t>(d_y) & (y_fp32 ? 3u : 1u))) return DFW_EALIGN;
    if (m == 0u) return DFW_OK;
    if ((st = device_sms(sms)) != DFW_OK) return st;
    a.packed = d_packed;
    a.x = d_x;
    a.y = d_y;
    a.ldx = ldx;
    a.ldy = ldy;
    a.m = m;
    a.y_fp32 = (uint32_t)y_fp32;
    const uint64_t want = ((uint64_t)a.q.rows * m + 255u) / 256u, cap = (uint64_t)sms * 16u;
    q4_gemv_plain<<<(unsigned)(want < cap ? want : cap), 256, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? DFW_OK : DFW_ECUDA;
}

}  // namespace dfw
