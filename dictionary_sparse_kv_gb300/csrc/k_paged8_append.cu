// Quantises a step's keys and values into the 8-bit pages.
//
// For a block of tokens and a head, with a the largest |x| of its new rows:
//   t = 2^e, e least with a <= M 2^e;  s = t or max(old scale, t);
//   code = rn(x / s);  codes of earlier tokens, if s grew: rn(code old / s).
// Powers of two make every division exact, so a code is x with one rounding,
// and keep what is rounded again within a step (a grown scale has doubled at
// least).
//
// The new rows have to be read once and the codes written once: HBM for
// prompts, latency for single tokens.  A warp takes one (block, head, keys or
// values): its rows (up to 16 of 128 elements) stay in registers between the
// maximum and the rounding, longer runs are read a second time, from L2.  The
// runs of rows that share a block are found by the warps themselves, from the
// slots: the warp whose rows a run begins in takes it.
#include <algorithm>

#include "paged8.cuh"

namespace fadkv {
namespace {

using namespace paged8;

constexpr int kThreads = 128;
// Steps of rows kept in shared memory between the two passes, 8 KB a warp.
constexpr int kHeldBytes = 8192;
template <typename T> constexpr int kHeld = kHeldBytes / (256 * (int)sizeof(T));

// Eight consecutive elements as loaded; their largest |x| as the type's bits.
template <typename T> struct Raw8 {
    uint4 a;
    // a lane's 16 bytes of step u in its warp's buffer
    static __device__ __forceinline__ void copy(uint32_t buf, int u, const T* p) { paged::cp16(buf + u * 512, p, true); }
    __device__ __forceinline__ void held(const unsigned char* buf, int u) { a = *reinterpret_cast<const uint4*>(buf + u * 512); }
    static constexpr uint32_t kInfinite = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    __device__ __forceinline__ void load(const T* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float* x) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Num<T>::unpack(w[i]);
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    __device__ __forceinline__ uint32_t most() const
    {
        const uint32_t m = 0x7fff7fffu;
        const uint32_t v = __vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m));
        return max(v & 0xffffu, v >> 16);
    }
    static __device__ __forceinline__ uint32_t wide(uint32_t bits) { return __float_as_uint(Num<T>::unpack(bits).x); }
};
template <> struct Raw8<float> {
    float4 a, b;
    static __device__ __forceinline__ void copy(uint32_t buf, int u, const float* p)
    {
        paged::cp16(buf + u * 1024, p, true);
        paged::cp16(buf + u * 1024 + 512, p + 4, true);
    }
    __device__ __forceinline__ void held(const unsigned char* buf, int u)
    {
        a = *reinterpret_cast<const float4*>(buf + u * 1024);
        b = *reinterpret_cast<const float4*>(buf + u * 1024 + 512);
    }
    static constexpr uint32_t kInfinite = 0x7f800000u;
    __device__ __forceinline__ void load(const float* p)
    {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void get(float* x) const
    {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ uint32_t most() const
    {
        const float m = fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                              fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
        const float n = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));   // NaN, where one is
        return n == n ? __float_as_uint(m) : 0x7fc00000u;
    }
    static __device__ __forceinline__ uint32_t wide(uint32_t bits) { return bits; }
};

// A run of rows that share a block: its first row and number of rows, the
// first of their places in the block, and whether the places follow one another.
struct Run {
    int row0, n, first;
    bool even;
};
// What it is written to: the block's first token (this head) and its scale.
struct Place {
    uint8_t* block;
    float* scale;
};

template <typename T, int D, int FORMAT>
__device__ __forceinline__ void quantise(const Append8Args& a, const T* x, long long stride, const Place& to, const Run& run, int lane,
                                         unsigned char* buf)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR;                        // lanes a row, rows a step
    const int sub = lane / LPR, l = lane % LPR, n = run.n, first = run.first;
    const bool held = n <= kHeld<T> * RPW;
    float old = first > 0 && lane == 0 ? *to.scale : 0.f;
    x += (run.row0 + sub) * stride + l * 8;
    const long long step = RPW * stride;
    uint32_t top = 0;
    // a lane reads back what it has copied itself, so nothing but its own copies is waited for
    if (held) {
        const T* p = x;
#pragma unroll 4
        for (int i = sub, u = 0; i < n; i += RPW, ++u, p += step) Raw8<T>::copy(paged::saddr(buf), u, p);
        paged::cp_commit();
        paged::cp_wait<0>();
#pragma unroll 4
        for (int i = sub, u = 0; i < n; i += RPW, ++u) {
            Raw8<T> r;
            r.held(buf, u);
            top = max(top, r.most());
        }
    } else {
        const T* p = x;
#pragma unroll 4
        for (int i = sub; i < n; i += RPW, p += step) {
            Raw8<T> r;
            r.load(p);
            top = max(top, r.most());
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const bool finite = top < Raw8<T>::kInfinite;
    if (!finite) {                                     // the largest finite one
        top = 0;
        const T* p = x;
#pragma unroll 1
        for (int i = sub; i < n; i += RPW, p += step) {
            Raw8<T> r;
            float f[8];
            r.load(p);
            r.get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = __float_as_uint(fabsf(f[j]));
                top = max(top, b < 0x7f800000u ? b : 0u);
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
    } else {
        top = Raw8<T>::wide(top);
    }
    const float t = __uint_as_float((uint32_t)max(Code<FORMAT>::exponent(top), 1) << 23);
    old = __shfl_sync(0xffffffffu, old, 0);
    const float s = first > 0 ? fmaxf(old, t) : t;
    // 1 / s of a power of two by its exponent
    const uint32_t bits = __float_as_uint(s);
    const float inv = (bits & 0x7fffffu) == 0u && bits < (254u << 23) ? __uint_as_float((254u << 23) - bits) : 1.f / s;
    if (lane == 0) *to.scale = s;
    if (first > 0 && s > old) {
        const float ratio = old * inv;                 // s is t here
        uint8_t* q = to.block + sub * a.p.token_stride + l * 8;
#pragma unroll 2
        for (int i = sub; i < first; i += RPW, q += RPW * a.p.token_stride) {
            const uint2 c = *reinterpret_cast<const uint2*>(q);
            float y[8];
            values<FORMAT>(c.x, y);
            values<FORMAT>(c.y, y + 4);
            *reinterpret_cast<uint2*>(q) = make_uint2(Code<FORMAT>::pack(y, ratio), Code<FORMAT>::pack(y + 4, ratio));
        }
    }
    auto put = [&](const Raw8<T>& r, int i) {
        float y[8];
        r.get(y);
        const int token = run.even ? first + i : __ldg(a.slots + run.row0 + i) & ((1 << a.bshift) - 1);
        *reinterpret_cast<uint2*>(to.block + token * a.p.token_stride + l * 8) =
            finite ? make_uint2(Code<FORMAT>::pack(y, inv), Code<FORMAT>::pack(y + 4, inv))
                   : make_uint2(Code<FORMAT>::pack_any(y, inv), Code<FORMAT>::pack_any(y + 4, inv));
    };
    if (held && finite && run.even) {
        uint8_t* q = to.block + (first + sub) * a.p.token_stride + l * 8;
#pragma unroll 2
        for (int i = sub, u = 0; i < n; i += RPW, ++u, q += RPW * a.p.token_stride) {
            Raw8<T> r;
            float y[8];
            r.held(buf, u);
            r.get(y);
            *reinterpret_cast<uint2*>(q) = make_uint2(Code<FORMAT>::pack(y, inv), Code<FORMAT>::pack(y + 4, inv));
        }
        return;
    }
    const T* p = x;
#pragma unroll 2
    for (int i = sub; i < n; i += RPW, p += step) {
        Raw8<T> r;
        r.load(p);
        put(r, i);
    }
}

// A warp takes `each` rows (at most 31) of one head's keys or values: the runs
// that begin there.
template <int D, int FORMAT>
__global__ void __launch_bounds__(kThreads, 6)
paged8_append_kernel(const __grid_constant__ Append8Args a, int each)
{
    __shared__ __align__(16) unsigned char smem[kThreads / 32 * kHeldBytes];
    pdl_begin();
    const unsigned int w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), columns = 2u * (unsigned int)a.p.Hkv;
    const int lane = threadIdx.x & 31, column = (int)(w % columns);
    const long long r0 = (long long)(w / columns) * each;
    if (r0 >= a.p.T) return;
    unsigned char* buf = smem + (threadIdx.x >> 5) * kHeldBytes + lane * 16;
    const bool is_v = column >= a.p.Hkv;
    const int head = is_v ? column - a.p.Hkv : column;

    const int type = is_v ? a.p.v_dtype : a.p.k_dtype;
    const void* x = is_v ? a.v : a.k;
    const long long stride = is_v ? a.p.v_stride : a.p.k_stride;
    const int limit = a.p.num_pages << (a.shift - a.bshift);          // blocks of a pool
    auto slot_of = [&](long long row) {                               // -1: skipped
        const int slot = row >= 0 && row < a.p.T ? __ldg(a.slots + row) : -1;
        return slot >= 0 && (slot >> a.bshift) < limit ? slot : -1;
    };
    // lane l: row r0 - 1 + l, and the 32 after those
    const int slot = slot_of(r0 - 1 + lane), later = slot_of(r0 + 31 + lane), blk = slot >> a.bshift;
    const int before = __shfl_up_sync(0xffffffffu, blk, 1);
    uint32_t leads = __ballot_sync(0xffffffffu, lane >= 1 && lane <= each && blk >= 0 && blk != before);
    for (; leads; leads &= leads - 1) {
        const int at = __ffs(leads) - 1, b = __shfl_sync(0xffffffffu, blk, at), s0 = __shfl_sync(0xffffffffu, slot, at);
        Run run;
        run.row0 = (int)r0 - 1 + at;
        uint32_t other = __ballot_sync(0xffffffffu, lane >= at && blk != b);
        run.n = (other ? __ffs(other) - 1 : 32) - at;
        const bool mine = lane >= at && lane < at + run.n;
        int first = mine ? slot : 0x7fffffff;
        run.even = __all_sync(0xffffffffu, !mine || slot - s0 == lane - at);
        if (!other)
            for (int i = run.row0 + run.n, s = later;; i += 32, s = slot_of((long long)i + lane)) {
                other = __ballot_sync(0xffffffffu, (s >> a.bshift) != b);
                const int more = other ? __ffs(other) - 1 : 32;
                if (lane < more) first = min(first, s);
                run.even = run.even && __all_sync(0xffffffffu, lane >= more || s - s0 == run.n + lane);
                run.n += more;
                if (other) break;
            }
        run.first = __reduce_min_sync(0xffffffffu, first) & ((1 << a.bshift) - 1);
        const int token = (b << a.bshift) & ((1 << a.shift) - 1), page = (b << a.bshift) >> a.shift;
        Place to;
        to.block = (is_v ? a.v_pages : a.k_pages) + page * a.p.page_stride + head * a.p.head_stride + token * a.p.token_stride;
        to.scale = (is_v ? a.v_scales : a.k_scales) + scale_at(page, head, token, a.p.Hkv, a.shift, a.bshift);
        if (type == FADKV_F32) quantise<float, D, FORMAT>(a, (const float*)x + head * D, stride, to, run, lane, buf);
        else if (type == FADKV_F16) quantise<__half, D, FORMAT>(a, (const __half*)x + head * D, stride, to, run, lane, buf);
        else quantise<__nv_bfloat16, D, FORMAT>(a, (const __nv_bfloat16*)x + head * D, stride, to, run, lane, buf);
    }
}

template <int D, int FORMAT>
cudaError_t launch_t(const Append8Args& a, cudaStream_t st)
{
    const long long columns = 2ll * a.p.Hkv;
    const long long want = a.p.T * columns / (152 * 24);
    const int each = (int)std::max(1ll, std::min(want, a.p.block > 16 ? 31ll : 16ll));
    const long long warps = (a.p.T + each - 1) / each * columns;
    if (warps > 0x7fffffffll) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    return launch_pdl(paged8_append_kernel<D, FORMAT>, dim3(grid), dim3(kThreads), 0, st, a, each);
}

}  // namespace

cudaError_t launch_paged8_append(const Append8Args& a, cudaStream_t st)
{
    if (a.p.T <= 0 || a.p.num_pages <= 0) return cudaSuccess;
    if (a.p.format == FADKV_E4M3) return a.p.d == 128 ? launch_t<128, FADKV_E4M3>(a, st) : launch_t<64, FADKV_E4M3>(a, st);
    return a.p.d == 128 ? launch_t<128, FADKV_I8>(a, st) : launch_t<64, FADKV_I8>(a, st);
}

}  // namespace fadkv
