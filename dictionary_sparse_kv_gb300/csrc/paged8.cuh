// Shared by the kernels of the 8-bit paged cache: arguments and the two
// formats' codes.
#pragma once

#include "paged.cuh"

namespace fadkv {

struct Append8Args {
    fadkv_append8_params p;
    int shift, bshift;        // page_size = 1 << shift, block = 1 << bshift
    const void* k;
    const void* v;
    const int32_t* slots;
    uint8_t* k_pages;
    uint8_t* v_pages;
    float* k_scales;
    float* v_scales;
};
cudaError_t launch_paged8_append(const Append8Args& a, cudaStream_t st);

struct Read8Args {
    fadkv_read8_params p;
    int shift, bshift;
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    const float* k_scales;
    const float* v_scales;
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* first;       // or null
    const int32_t* out_table;   // or null
    void* k_out;
    void* v_out;
};
cudaError_t launch_paged8_read(const Read8Args& a, cudaStream_t st);

struct Paged8Args {
    fadkv_paged8_params p;
    int shift, bshift, grp;   // grp: query heads per KV head
    float scale_log2;         // scale * log2(e)
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scales;
    const float* v_scales;
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* positions;   // or null
    const void* q;
    void* out;
    float* lse;
    void* ws;
};
size_t paged8_attend_workspace(const fadkv_paged8_params& p);
cudaError_t launch_paged8_attend(const Paged8Args& a, cudaStream_t st);

namespace paged8 {

using paged::Num;

// Index of a block's scale.
__device__ __forceinline__ size_t scale_at(int page, int head, int token, int heads, int shift, int bshift)
{
    return (((size_t)page * heads + head) << (shift - bshift)) + (token >> bshift);
}

// Lengths and block tables on their way to L2 while the kernel before this one
// ends: a hint that returns nothing, so that it may come before the wait for
// that kernel.
__device__ __forceinline__ void prefetch_tables(const int32_t* lengths, const int32_t* table, int B, int max_pages)
{
    const unsigned line = blockIdx.x * blockDim.x + threadIdx.x;
    if (line * 32u < (unsigned)B) asm volatile("prefetch.global.L2 [%0];" ::"l"(lengths + line * 32u));
    if (line * 32ull < (unsigned long long)B * max_pages) asm volatile("prefetch.global.L2 [%0];" ::"l"(table + (size_t)line * 32));
}

// Codes as binary16 values (both formats' are exact there) and in 32 bits.
template <int FORMAT> struct Code;

template <> struct Code<FADKV_E4M3> {
    // bytes 0, 1 and bytes 2, 3
    static __device__ __forceinline__ void halves(uint32_t x, uint32_t& a, uint32_t& b)
    {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(a), "=r"(b)
            : "r"(x));
    }
    // bytes 0, 2 and bytes 1, 3
    static __device__ __forceinline__ void crossed(uint32_t x, uint32_t& a, uint32_t& b)
    {
        halves(__byte_perm(x, 0u, 0x3120), a, b);
    }
    // as halves, but for a factor and an offset, which are put right in a sum of products q code: sum = kUnit sum' - kOffset sum(q)
    static constexpr float kUnit = 1.f, kOffset = 0.f;
    static __device__ __forceinline__ void shifted(uint32_t x, uint32_t& a, uint32_t& b) { halves(x, a, b); }
    // the nearest codes of four y inv that are finite and in the type's range; in pack_any what is not finite becomes NaN
    static __device__ __forceinline__ uint32_t pack(const float* y, float inv)
    {
        uint32_t r;
        asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
            "mov.b32 %0, {l, h};\n\t}"
            : "=r"(r)
            : "f"(y[0] * inv), "f"(y[1] * inv), "f"(y[2] * inv), "f"(y[3] * inv));
        return r;
    }
    static __device__ __forceinline__ uint32_t pack_any(const float* y, float inv)
    {
        const float z[4] = {fmaf(y[0], 0.f, y[0]), fmaf(y[1], 0.f, y[1]), fmaf(y[2], 0.f, y[2]), fmaf(y[3], 0.f, y[3])};
        return pack(z, inv);
    }
    // biased exponent of the least power of two t with a <= 448 t (448 = 1.75 2^8), a by its bits
    static __device__ __forceinline__ int exponent(uint32_t a) { return (int)(a >> 23) - 8 + ((a & 0x7fffffu) > 0x600000u); }
};

template <> struct Code<FADKV_I8> {
    static __device__ __forceinline__ uint32_t centred(uint32_t x)      // 1024 + 128 + code, less 1152
    {
        const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ void halves(uint32_t x, uint32_t& a, uint32_t& b)
    {
        x ^= 0x80808080u;
        a = centred(__byte_perm(x, 0x64646464u, 0x4140));
        b = centred(__byte_perm(x, 0x64646464u, 0x4342));
    }
    static __device__ __forceinline__ void crossed(uint32_t x, uint32_t& a, uint32_t& b)
    {
        x ^= 0x80808080u;
        a = centred(__byte_perm(x, 0x64646464u, 0x4240));
        b = centred(__byte_perm(x, 0x64646464u, 0x4341));
    }
    // (code + 128) 2^-24: a byte is a number below binary16's normal range as it stands
    static constexpr float kUnit = 16777216.f, kOffset = 128.f;
    static __device__ __forceinline__ void shifted(uint32_t x, uint32_t& a, uint32_t& b)
    {
        x ^= 0x80808080u;
        a = __byte_perm(x, 0u, 0x4140);
        b = __byte_perm(x, 0u, 0x4342);
    }
    // the nearest whole numbers of four y inv, by the low byte of 1.5 2^23 + y inv; in pack_any NaN becomes 0 and an infinity
    // the largest
    static __device__ __forceinline__ uint32_t pack(const float* y, float inv)
    {
        uint32_t z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = __float_as_uint(__fadd_rn(__fmul_rn(y[i], inv), 12582912.f));
        return __byte_perm(__byte_perm(z[0], z[1], 0x0040), __byte_perm(z[2], z[3], 0x0040), 0x5410);
    }
    static __device__ __forceinline__ uint32_t pack_any(const float* y, float inv)
    {
        float z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = y[i] == y[i] ? fminf(fmaxf(y[i] * inv, -127.f), 127.f) : 0.f;
        return pack(z, 1.f);
    }
    // 127 = 1.984375 2^6
    static __device__ __forceinline__ int exponent(uint32_t a) { return (int)(a >> 23) - 6 + ((a & 0x7fffffu) > 0x7e0000u); }
};

// Four codes in 32 bits.
template <int FORMAT>
__device__ __forceinline__ void values(uint32_t x, float* y)
{
    uint32_t a, b;
    Code<FORMAT>::halves(x, a, b);
    const float2 f = Num<__half>::unpack(a), g = Num<__half>::unpack(b);
    y[0] = f.x, y[1] = f.y, y[2] = g.x, y[3] = g.y;
}

}  // namespace paged8
}  // namespace fadkv
