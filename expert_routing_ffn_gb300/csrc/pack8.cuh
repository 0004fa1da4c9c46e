// Rows in 8 bits: blocks of 32 columns that share a power of two (the format
// stands in moe_train.h), read and written by eight columns a thread.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {
namespace pack8 {

// E of a block from the bits of its largest magnitude (0x7f800000 and above: not
// finite).  With the magnitude m 2^e, 1 <= m < 2, the step is 2^(e - 6), which
// brings it to 64 m < 128, or twice that where 64 m would round to 128; not in the
// last binade, where a step more would read as infinite: 127 steps it is there.
constexpr uint32_t kTop = 248u;
__device__ __forceinline__ uint32_t exponent(uint32_t magnitude) {
    if (magnitude >= 0x7f800000u) return 255u;
    const int e = (int)(magnitude >> 23) - 6 + ((magnitude & 0x7fffffu) >= 0x7f0000u ? 1 : 0);
    return (uint32_t)min(max(e, 0), (int)kTop);
}
// a value of a block of the last binade, held to 127 steps
__device__ __forceinline__ float within(float x, uint32_t E) {
    return E == kTop ? fminf(fmaxf(x, -127.f * 0x1p121f), 127.f * 0x1p121f) : x;
}
// 2^(127 - E), what values are multiplied by (exact); 0 for a block that is not finite
__device__ __forceinline__ float to_steps(uint32_t E) { return E == 255u ? 0.f : __uint_as_float((254u - E) << 23); }
// 2^(E - 127); infinite for E = 255, so that 0 times it is NaN
__device__ __forceinline__ float step(uint32_t E) { return __uint_as_float(E ? E << 23 : 0x400000u); }

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// x in steps, rounded to nearest (ties to even), in the low byte: 1.5 2^23 + x
// has a unit of 1 in its last place, and the sum rounds once.  Where the block
// is not finite `inv` is 0 and the byte says nothing (quantise gives zeros).
__device__ __forceinline__ uint32_t quantise(float x, float inv) { return __float_as_uint(fmaf(x, inv, 12582912.f)); }

// byte i of a word of packed values as a float: 2^23 + 128 + q has q + 128 in its low byte
__device__ __forceinline__ uint32_t biased(uint32_t word) { return word ^ 0x80808080u; }
__device__ __forceinline__ float value(uint32_t biased_word, int i) {
    return __uint_as_float(__byte_perm(biased_word, 0x4b000000u, 0x7440 | i)) - 8388736.f;
}
template <int I>
__device__ __forceinline__ float value(uint32_t biased_word) { return value(biased_word, I); }
// the same before kRaw is taken off
constexpr float kRaw = 8388736.f;
template <int I>
__device__ __forceinline__ float raw(uint32_t biased_word) { return __uint_as_float(__byte_perm(biased_word, 0x4b000000u, 0x7440 | I)); }

__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Four lanes (aligned) exchange 16-bit pieces: lane t's pieces for lanes 0 .. 3 are
// the halves of r0 and r1; it gets x = those of lanes 0 and 2 for it, y = of 1 and 3.
__device__ __forceinline__ void exchange(uint32_t r0, uint32_t r1, uint32_t& x, uint32_t& y) {
    const bool up = threadIdx.x & 2, odd = threadIdx.x & 1;
    const uint32_t far = __shfl_xor_sync(0xffffffffu, up ? r0 : r1, 2);
    const uint32_t a = up ? far : r0, b = up ? r1 : far;  // pieces 2 (t / 2), + 1 of lanes t % 2 and t % 2 + 2
    const uint32_t lo = __byte_perm(a, b, 0x5410), hi = __byte_perm(a, b, 0x7632);
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1), mine = odd ? hi : lo;
    x = odd ? got : mine;
    y = odd ? mine : got;
}
// Columns 8 j .. 8 j + 7 of a block on lane j of four, as bytes (p0: the first four)
// <-> words 2 j and 2 j + 1 of the packed block.
__device__ __forceinline__ uint2 to_packed(uint32_t p0, uint32_t p1) {
    uint32_t x, y;
    exchange(p0, p1, x, y);
    return make_uint2(__byte_perm(x, y, 0x6240), __byte_perm(x, y, 0x7351));
}
__device__ __forceinline__ uint2 to_columns(uint2 w) {
    const uint32_t x = __byte_perm(w.x, w.y, 0x6240), y = __byte_perm(w.x, w.y, 0x7351);
    uint32_t a, b;
    exchange(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632), a, b);
    return make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
}

// eight columns from c on of a row, zeros past its end; VEC: the row starts on 16 bytes and has whole vectors
template <typename W, bool VEC>
__device__ __forceinline__ void load8(const W* row, int c, int cols, float (&f)[8]) {
    if constexpr (VEC && sizeof(W) == 2) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c < cols) v = *reinterpret_cast<const uint4*>(row + c);
        unpack16(v, f, (__nv_bfloat16*)nullptr);
    } else if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + 4 * h < cols) v = *reinterpret_cast<const float4*>(row + c + 4 * h);
            f[4 * h] = v.x; f[4 * h + 1] = v.y; f[4 * h + 2] = v.z; f[4 * h + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < cols ? to_f32(row[c + i]) : 0.f;
    }
}
template <typename W, bool VEC>
__device__ __forceinline__ void store8(W* row, int c, int cols, const float (&f)[8]) {
    if constexpr (VEC && sizeof(W) == 2) {
        if (c < cols) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (c + 4 * h < cols)
                *reinterpret_cast<float4*>(row + c + 4 * h) = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) {
                if constexpr (sizeof(W) == 2) row[c + i] = __float2bfloat16_rn(f[i]);
                else row[c + i] = f[i];
            }
    }
}

// The eight values of a row whose packed bytes lie in a lane's two words: with j the
// lane of four and c its first column in load8's order, columns 2 j + 8 m and
// 2 j + 1 + 8 m of the block, m = 0 .. 3, at f[2 m] and f[2 m + 1].
template <typename W, bool VEC>
__device__ __forceinline__ void load_interleaved(const W* row, int c, int cols, float (&f)[8]) {
    const int first = (c & ~31) + (c >> 3 & 3) * 2;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int at = first + 8 * m;
        f[2 * m] = f[2 * m + 1] = 0.f;
        if constexpr (VEC) {  // whole vectors: both values or none
            if (at < cols) {
                if constexpr (sizeof(W) == 2) {
                    const uint32_t v = *reinterpret_cast<const uint32_t*>(row + at);
                    f[2 * m] = bf16_lo(v); f[2 * m + 1] = bf16_hi(v);
                } else {
                    const float2 v = *reinterpret_cast<const float2*>(row + at);
                    f[2 * m] = v.x; f[2 * m + 1] = v.y;
                }
            }
        } else {
            if (at < cols) f[2 * m] = to_f32(row[at]);
            if (at + 1 < cols) f[2 * m + 1] = to_f32(row[at + 1]);
        }
    }
}

// one value of packed rows of nb blocks: a byte and a scale fetched for each (down gradient on the CUDA cores, 128
// float32 rows an expert, d 256, I 512: 33 us against 27 from g and u in float32; 256 rows, d 1024: 141 against 131)
__device__ __forceinline__ float value_at(const int8_t* q, const uint8_t* scale, int64_t row, int col, int nb) {
    const int64_t block = row * nb + col / 32;
    const int c = col & 31;
    return (float)q[block * 32 + 4 * (c & 7) + (c >> 3)] * step(scale[block]);
}

}  // namespace pack8
}  // namespace moe
