// mx4.hpp -- microscaled 4-bit floating point (OCP MX: e2m1 values in blocks of 32 along
// a row, one power-of-two e8m0 scale for each block): quantisation, its inverse, the
// scales' layout and the matrix product.
//
// A matrix of R rows and K columns is held as
//   codes   R x 16*ceil(K/32) bytes, element 2i in the low half of byte i; a row's last
//           block is filled with zeros
//   scales  tiles of 32 rows x 8 blocks (256 columns), 256 bytes each, a row of tiles
//           after the other; in a tile the byte of row r and block b is at
//           128*(b/4) + 4*r + b%4
// In v_mfma_scale_f32_32x32x64 lane l holds 32 consecutive k of row l%32 and one scale
// byte out of four in a register.  k is only summed, so a wave may give its lane halves
// any blocks as long as A and B agree: half h takes blocks 4h .. 4h+3 of a tile in four
// MFMAs, and the four scale bytes of a lane are then one dword of the tile, the 64 lanes'
// dwords 256 consecutive bytes.
#pragma once

#include "grouped.hpp"
#include "sg_device.hpp"

namespace sg {

constexpr int kMxBlock = 32;          // elements that share a scale
constexpr int kMxTileRows = 32;       // rows and blocks of a tile of scales
constexpr int kMxTileBlocks = 8;
constexpr int kMxTileBytes = kMxTileRows * kMxTileBlocks;
constexpr int kMxNaN = 255;           // the scale that makes its block NaN

__host__ __device__ constexpr int64_t mx_blocks(int64_t K) { return (K + 31) / 32; }
__host__ __device__ constexpr int64_t mx_row_bytes(int64_t K) { return 16 * mx_blocks(K); }
__host__ __device__ constexpr int64_t mx_tiles_k(int64_t K) { return (K + 255) / 256; }
__host__ __device__ constexpr int64_t mx_scale_bytes(int64_t R, int64_t K) {
    return (R + 31) / 32 * mx_tiles_k(K) * kMxTileBytes;
}

// the byte of row r (of its matrix) and block b, `tiles_k` tiles in a row of tiles
__device__ __forceinline__ int64_t mx_scale_at(int r, int b, int tiles_k) {
    return ((int64_t)(r >> 5) * tiles_k + (b >> 3)) * kMxTileBytes + ((b >> 2) & 1) * 128 +
           (r & 31) * 4 + (b & 3);
}

struct MxQuantParams {
    const void* X;        // M x K rows, ldx elements apart; `batch` matrices sX bytes apart
    uint8_t* codes;       // each matrix M x mx_row_bytes(K)
    uint8_t* scales;      // each matrix mx_scale_bytes(M, K)
    void* values;         // nullptr, or M x K of X's type, rows ldv elements apart
    int64_t ldx, ldv, sX, sV;
    int M, K;
    int vec_x, vec_v;     // rows of X / values allow 16-byte accesses
};

// ---------------------------------------------------------------------------
// Quantisation.  t = max |x| of a block, s = 2^(floor(log2 t) - 2) so that t/s lies in
// [4, 8); the codes are x/s to the nearest e2m1 value (0, .5, 1, 1.5, 2, 3, 4, 6; ties to
// the even code), above 6 saturating.  s is held in [2^-127, 2^125], which every finite t
// keeps it in but for t < 2^-125, where s = 2^-127.  A block with an infinity or a NaN
// gets the NaN scale and zero codes.  Both scalings are by powers of two: exact.
//
// Bound by memory (2 bytes read and 17/32 written an element from bf16).  A work-group
// takes one tile of scales, 32 rows x 256 columns: four lanes a block, eight elements
// each, so that a row is read in 512 consecutive bytes; the four rows of a thread are in
// flight together, and the tile's 256 scale bytes leave as one line.  From bf16, 16384 x
// 2048: 19.6 us, 4.3 TB/s; 8192 x 4096 to rounded values instead: 24.3 us, 5.5 TB/s.
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ void mx_load8(const void* X, int64_t at, int left, bool vec,
                                         float (&v)[8]) {
    if (vec && left >= 8) {
        if constexpr (DT == DT_F32) {
            const f32x4* s = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(X) + at);
            const f32x4 a = s[0], b = s[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
        } else {
            const u32x4 w =
                *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(X) + at);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = to_f32<DT>((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = 0.0f;
        if (e < left) {
            if constexpr (DT == DT_F32) v[e] = reinterpret_cast<const float*>(X)[at + e];
            else v[e] = to_f32<DT>(reinterpret_cast<const uint16_t*>(X)[at + e]);
        }
    }
}

template <int DT>
__device__ __forceinline__ void mx_store8(void* X, int64_t at, int left, bool vec,
                                          const float (&v)[8]) {
    if (vec && left >= 8) {
        if constexpr (DT == DT_F32) {
            f32x4* d = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(X) + at);
            d[0] = f32x4{v[0], v[1], v[2], v[3]};
            d[1] = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(X) + at) =
                u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]),
                      pack2<DT>(v[6], v[7])};
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < left) {
            if constexpr (DT == DT_F32) reinterpret_cast<float*>(X)[at + e] = v[e];
            else reinterpret_cast<uint16_t*>(X)[at + e] = from_f32<DT>(v[e]);
        }
}

// eight e2m1 codes of v (already divided by the scale), the first in the low bits:
// v_cvt_scalef32_pk_fp4_f32 at scale 1 rounds to nearest, ties to even, and saturates
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8]) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.0f, 3);
    return w;
}

// the values of eight codes times the scale 2^(s - 127); s == 255: NaN
__device__ __forceinline__ void mx_values8(uint32_t w, int s, float (&v)[8]) {
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    const float x[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = s == kMxNaN ? __builtin_nanf("") : __builtin_ldexpf(x[e], s - 127);
}

template <int DT>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const MxQuantParams p) {
    __shared__ uint32_t tile[kMxTileBytes / 4];
    const int tiles_k = (int)mx_tiles_k(p.K), nb = (int)mx_blocks(p.K);
    const int kt = blockIdx.x % tiles_k, rt = blockIdx.x / tiles_k;
    const int64_t z = blockIdx.z;
    const char* X = reinterpret_cast<const char*>(p.X) + z * p.sX;
    char* V = reinterpret_cast<char*>(p.values) + z * p.sV;
    const int64_t row_bytes = mx_row_bytes(p.K);
    uint8_t* codes = p.codes + z * p.M * row_bytes;
    const int col = threadIdx.x & 31, sub = threadIdx.x >> 5;   // 8 columns, rows sub + 8 i
    const int k = kt * 256 + col * 8, b = k >> 5;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = rt * 32 + sub + 8 * i;
        mx_load8<DT>(X, (int64_t)r * p.ldx + k, r < p.M ? p.K - k : 0, p.vec_x != 0, v[i]);
    }
    uint8_t* ts = reinterpret_cast<uint8_t*>(tile);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int lr = sub + 8 * i, r = rt * 32 + lr;
        uint32_t t = 0;                                         // max |x| by its bits
#pragma unroll
        for (int e = 0; e < 8; ++e)
            t = max(t, __builtin_bit_cast(uint32_t, v[i][e]) & 0x7fffffffu);
        // over the block's four lanes: quad_perm [1,0,3,2], then [2,3,0,1]
        t = max(t, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)t, 0xB1, 0xf, 0xf, false));
        t = max(t, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)t, 0x4E, 0xf, 0xf, false));
        const bool bad = t >= 0x7f800000u;
        const int s = bad ? kMxNaN : max((int)(t >> 23) - 2, 0);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = bad ? 0.0f : __builtin_ldexpf(v[i][e], 127 - s);
        const uint32_t w = mx_codes8(y);
        if ((col & 3) == 0) ts[((col >> 2) >> 2) * 128 + lr * 4 + ((col >> 2) & 3)] = (uint8_t)s;
        if (r < p.M && b < nb) {
            if (p.codes)
                *reinterpret_cast<uint32_t*>(codes + r * row_bytes + kt * 128 + col * 4) = w;
            if (p.values && k < p.K) {
                float o[8];
                mx_values8(w, s, o);
                mx_store8<DT>(V, (int64_t)r * p.ldv + k, p.K - k, p.vec_v != 0, o);
            }
        }
    }
    __syncthreads();
    if (p.scales && threadIdx.x < 64) {
        uint8_t* out = p.scales + z * mx_scale_bytes(p.M, p.K) +
                       ((int64_t)rt * tiles_k + kt) * kMxTileBytes;
        reinterpret_cast<uint32_t*>(out)[threadIdx.x] = tile[threadIdx.x];
    }
}

// The inverse: X = codes * scales, rounded once to X's type.  Eight columns a thread.
template <int DT>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const MxQuantParams p) {
    const int tiles_k = (int)mx_tiles_k(p.K);
    const int kt = blockIdx.x % tiles_k, rt = blockIdx.x / tiles_k;
    const int64_t z = blockIdx.z, row_bytes = mx_row_bytes(p.K);
    const uint8_t* codes = p.codes + z * p.M * row_bytes;
    const uint8_t* scales = p.scales + z * mx_scale_bytes(p.M, p.K);
    char* V = reinterpret_cast<char*>(p.values) + z * p.sV;
    const int col = threadIdx.x & 31, k = kt * 256 + col * 8;
    if (k >= p.K) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = rt * 32 + (threadIdx.x >> 5) + 8 * i;
        if (r >= p.M) break;
        float o[8];
        mx_values8(*reinterpret_cast<const uint32_t*>(codes + r * row_bytes + kt * 128 + col * 4),
                   scales[mx_scale_at(r, k >> 5, tiles_k)], o);
        mx_store8<DT>(V, (int64_t)r * p.ldv + k, p.K - k, p.vec_v != 0, o);
    }
}

// Scales from rows of bytes (M x blocks, `ld` apart) to tiles; the tiles' padding is 0.
// One dword (a row's four blocks of a tile) a thread.
__global__ static void __launch_bounds__(256)
    mx_tile_scales_kernel(const uint8_t* src, int64_t ld, int64_t stride, uint8_t* dst, int M,
                          int nb) {
    const int tiles_k = (nb + 7) / 8;
    const int64_t dwords = (int64_t)((M + 31) / 32) * tiles_k * (kMxTileBytes / 4);
    src += blockIdx.z * stride;
    uint32_t* out = reinterpret_cast<uint32_t*>(dst) + blockIdx.z * dwords;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < dwords;
         i += (int64_t)gridDim.x * 256) {
        const int64_t t = i >> 6;
        const int r = (int)(t / tiles_k) * 32 + (int)(i & 31);
        const int b = (int)(t % tiles_k) * 8 + (int)((i >> 5) & 1) * 4;
        uint32_t w = 0;
        if (r < M)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (b + j < nb) w |= (uint32_t)src[(int64_t)r * ld + b + j] << (8 * j);
        out[i] = w;
    }
}

// ---------------------------------------------------------------------------
// The product C = alpha * A * B^T of two such matrices, A's rows grouped by expert where
// there are offsets.  GroupedParams: A, B codes; lda, ldb row bytes; g.K blocks.
// ---------------------------------------------------------------------------
struct MxParams {
    GroupedParams q;
    const uint8_t* As;       // scales of A (all rows), of B (each expert's sBs bytes apart)
    const uint8_t* Bs;
    int64_t sBs;
    int tiles_k;
};

// dt: the output type; cfg: the tile.  blocks: the host's upper bound of the items.
hipError_t launch_mx4(int epi, int dt, int cfg, const MxParams& x, unsigned blocks,
                      hipStream_t st);

}  // namespace sg
