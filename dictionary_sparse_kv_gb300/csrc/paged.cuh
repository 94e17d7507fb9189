// Shared by the paged-cache kernels: arguments, 16-bit matrix instructions for
// both storage types, asynchronous copies and the mapping of work to blocks.
#pragma once

#include <cuda_bf16.h>

#include "fadkv_internal.cuh"

namespace fadkv {

struct PlanArgs {
    int B, shift, num_pages, max_pages, max_tokens;   // page_size = 1 << shift
    const int32_t* add;
    const int32_t* lengths;
    int32_t* table;
    int32_t* free_pages;
    const int32_t* free_count;
    int32_t* lengths_out;
    int32_t* free_count_out;
    int32_t* starts;
    int32_t* positions;
    int32_t* slots;
    int32_t* refused;
};
cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t st);

struct QkArgs {
    fadkv_qk_params p;
    fadkv_rope rope;
    int shift;
    const void* q;
    const void* k;
    const void* v;
    const void* wq;
    const void* wk;
    const int32_t* positions;
    const int32_t* slots;
    void* q_out;
    void* k_out;
    void* k_pages;
    void* v_pages;
};
cudaError_t launch_qk_norm_rope(const QkArgs& a, cudaStream_t st);

struct PagedArgs {
    fadkv_paged_params p;
    int shift, grp;           // page_size = 1 << shift; query heads per KV head
    int split;                // prefill: whether items may be cut along their keys (the launcher sets it)
    unsigned long long wait_ns;   // prefill: limit of the waits (0: the launcher sets the default)
    unsigned int tile_ns;         // prefill: what waits for an item's end are given for each of its key tiles
    float scale_log2;         // scale * log2(e): scores in units of powers of two
    const void* k;
    const void* v;
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* starts;
    const int32_t* positions;   // or null
    const void* q;
    void* out;
    float* lse;
    void* ws;
};
size_t paged_attend_workspace(const fadkv_paged_params& p);
cudaError_t launch_paged_attend(const PagedArgs& a, cudaStream_t st);
size_t paged_prefill_workspace(const fadkv_paged_params& p);
cudaError_t launch_paged_prefill(const PagedArgs& a, cudaStream_t st);

namespace paged {

// The workspaces' heads, which have to be zero between calls, lie apart, so
// that one workspace can serve both calls in turn: the prefill's first, then
// (from kDecodeHead on) the counters of the single-token call, then what
// either keeps only while it runs.
constexpr size_t kDecodeHead = 4096, kHeadBytes = 16384;

constexpr float kLn2 = 0.693147180559945f;

// Type traits of the two 16-bit storage types.
template <typename T> struct Num;
template <> struct Num<__half> {
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u)
    {
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Num<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u)
    {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// The 8x8 matrix of 16-bit values held one pair a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// 16 bytes global -> shared, asynchronous; zeros (and no read) unless valid.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two 32-bit values in one register pair: one instruction for both.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Byte offset of 16-byte chunk c of row r in a tile of ROW-byte rows whose
// chunks are swapped by row, so that eight rows at one chunk lie in eight
// different bank groups.
template <int ROW>
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * ROW + ((c ^ (r & 7)) << 4)); }

// The keys that the query at position len - 1 sees, as one list: the first
// `first` tokens, then those from `from` on; `count` in all.
struct Seen {
    int first, from, count;
};
__device__ __forceinline__ int clamp_len(int len, const PagedArgs& a)
{
    const int most = a.p.max_pages << a.shift;
    return len < 0 ? 0 : (len > most ? most : len);
}
// The tokens of request b, whose first row is `row` (below T): none for a
// request that the plan refused, as its rows are not the last ones of those.
__device__ __forceinline__ int length_of(int b, int row, const PagedArgs& a)
{
    const int pos = a.positions ? __ldg(a.positions + row) : 0, len = __ldg(a.lengths + b);
    return pos < 0 ? 0 : clamp_len(len, a);
}
__device__ __forceinline__ Seen seen_of(int len, const PagedArgs& a)
{
    Seen s;
    s.from = (a.p.window > 0 && len > a.p.window) ? len - a.p.window : 0;
    s.first = min(a.p.sinks, s.from);
    s.count = s.first + len - s.from;
    return s;
}

// Exclusive prefix sum over the block's threads; `total` gets the sum.
template <int THREADS>
__device__ __forceinline__ long long block_scan(long long v, long long* total)
{
    __shared__ long long part[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    long long before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += part[w];
        sum += part[w];
    }
    __syncthreads();
    *total = sum;
    return before + x - v;
}

}  // namespace paged
}  // namespace fadkv
