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
// values), and its rows wait in shared memory between the maximum and the
// rounding (8 KB a warp, 24 warps a multiprocessor: enough in flight, and
// few registers; kept in registers 28 us, read a second time from L2 35, for
// the first case below); blocks too large for that are four warps' work.
// The runs of rows that share a block are found by the warps themselves, from
// the slots: the warp whose rows a run begins in takes it.  What is not finite is
// looked at only where the maximum says so.  Three prompts of up to 8000 tokens
// of 8 heads of 128, bfloat16 to I8: 22.0 us, 5.8 TB/s; 16 single tokens 2.1 us,
// of which a launch is most.
#include <algorithm>

#include "paged8.cuh"

namespace fadkv {
namespace {

using namespace paged8;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kWindow = 31;      // rows whose runs a warp looks for at a time (their slots and the one before: a lane each)
// Steps of rows kept in shared memory between the two passes, 8 KB a warp.
constexpr int kHeldBytes = 8192;
template <typename T> constexpr int kHeld = kHeldBytes / (256 * (int)sizeof(T));

// Eight elements of a row as loaded, those from first(l) on for lane l: eight that
// follow one another, or in 32 bits four and four half a row on, so that a row's
// lanes read whole sectors together; their largest |x| as the type's bits.
template <typename T, int D> struct Raw8 {
    uint4 a;
    static constexpr int kGap = 4;
    static __device__ __forceinline__ int first(int l) { return l * 8; }
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
template <int D> struct Raw8<float, D> {
    float4 a, b;
    static constexpr int kGap = D / 2;
    static __device__ __forceinline__ int first(int l) { return l * 4; }
    static __device__ __forceinline__ void copy(uint32_t buf, int u, const float* p)
    {
        paged::cp16(buf + u * 1024, p, true);
        paged::cp16(buf + u * 1024 + 512, p + kGap, true);
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
        b = __ldg(reinterpret_cast<const float4*>(p + kGap));
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

// One run's keys (values) of a head, by a warp, or by warp `warp` of the block's
// (team), which then take a part of the rows each and share their maxima.
template <typename T, int D, int FORMAT>
__device__ __forceinline__ void quantise(const Append8Args& a, const T* x, long long stride, const Place& to, const Run& run, bool team,
                                         int warp, unsigned char* buf, uint32_t* maxima)
{
    using Raw = Raw8<T, D>;
    constexpr int LPR = D / 8, RPW = 32 / LPR;                        // lanes a row, rows a step
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR, first = run.first;
    const int i0 = team ? run.n * warp / kWarps : 0, i1 = team ? run.n * (warp + 1) / kWarps : run.n;
    const bool held = i1 - i0 <= kHeld<T> * RPW;
    float old = first > 0 && lane == 0 ? *to.scale : 0.f;
    x += ((long long)run.row0 + i0 + sub) * stride + Raw::first(l);
    const long long step = RPW * stride;
    uint32_t top = 0;
    // a lane reads back what it has copied itself, so nothing but its own copies is waited for
    if (held) {
        const T* p = x;
#pragma unroll 4
        for (int i = i0 + sub, u = 0; i < i1; i += RPW, ++u, p += step) Raw::copy(paged::saddr(buf), u, p);
        paged::cp_commit();
        paged::cp_wait<0>();
#pragma unroll 4
        for (int i = i0 + sub, u = 0; i < i1; i += RPW, ++u) {
            Raw r;
            r.held(buf, u);
            top = max(top, r.most());
        }
    } else {
        const T* p = x;
#pragma unroll 4
        for (int i = i0 + sub; i < i1; i += RPW, p += step) {
            Raw r;
            r.load(p);
            top = max(top, r.most());
        }
    }
    int turn = 0;
    auto largest = [&] {
        top = __reduce_max_sync(0xffffffffu, top);
        if (team) {
            if (lane == 0) maxima[turn * kWarps + warp] = top;
            __syncthreads();
#pragma unroll
            for (int x = 0; x < kWarps; ++x) top = max(top, maxima[turn * kWarps + x]);
            ++turn;
        }
    };
    largest();
    const bool finite = top < Raw::kInfinite;
    if (!finite) {                                     // the largest finite one
        top = 0;
        const T* p = x;
#pragma unroll 1
        for (int i = i0 + sub; i < i1; i += RPW, p += step) {
            Raw r;
            float f[8];
            r.load(p);
            r.get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = __float_as_uint(fabsf(f[j]));
                top = max(top, b < 0x7f800000u ? b : 0u);
            }
        }
        largest();
    } else {
        top = Raw::wide(top);
    }
    const float t = __uint_as_float((uint32_t)max(Code<FORMAT>::exponent(top), 1) << 23);
    old = __shfl_sync(0xffffffffu, old, 0);
    const float s = first > 0 ? fmaxf(old, t) : t;
    // 1 / s of a power of two by its exponent
    const uint32_t bits = __float_as_uint(s);
    const float inv = (bits & 0x7fffffu) == 0u && bits < (254u << 23) ? __uint_as_float((254u << 23) - bits) : 1.f / s;
    if (lane == 0 && (!team || warp == 0)) *to.scale = s;              // (every warp has read the old one)
    if (first > 0 && s > old) {
        const float ratio = old * inv;                 // s is t here
        const int each = RPW * (team ? kWarps : 1), begin = sub + (team ? warp * RPW : 0);
        uint8_t* q = to.block + begin * a.p.token_stride + l * 8;
#pragma unroll 2
        for (int i = begin; i < first; i += each, q += each * a.p.token_stride) {
            const uint2 c = *reinterpret_cast<const uint2*>(q);
            float y[8];
            values<FORMAT>(c.x, y);
            values<FORMAT>(c.y, y + 4);
            *reinterpret_cast<uint2*>(q) = make_uint2(Code<FORMAT>::pack(y, ratio), Code<FORMAT>::pack(y + 4, ratio));
        }
    }
    auto put = [&](uint8_t* q, uint32_t c0, uint32_t c1) {
        if (Raw::kGap == 4) {
            *reinterpret_cast<uint2*>(q) = make_uint2(c0, c1);
        } else {
            *reinterpret_cast<uint32_t*>(q) = c0;
            *reinterpret_cast<uint32_t*>(q + Raw::kGap) = c1;
        }
    };
    uint8_t* q = to.block + Raw::first(l);
    if (held && finite && run.even) {
        q += (long long)(first + i0 + sub) * a.p.token_stride;
#pragma unroll 2
        for (int i = i0 + sub, u = 0; i < i1; i += RPW, ++u, q += RPW * a.p.token_stride) {
            Raw r;
            float y[8];
            r.held(buf, u);
            r.get(y);
            put(q, Code<FORMAT>::pack(y, inv), Code<FORMAT>::pack(y + 4, inv));
        }
        return;
    }
    const T* p = x;
#pragma unroll 2
    for (int i = i0 + sub; i < i1; i += RPW, p += step) {
        Raw r;
        float y[8];
        r.load(p);
        r.get(y);
        const int token = run.even ? first + i : __ldg(a.slots + run.row0 + i) & ((1 << a.bshift) - 1);
        put(q + token * a.p.token_stride, finite ? Code<FORMAT>::pack(y, inv) : Code<FORMAT>::pack_any(y, inv),
            finite ? Code<FORMAT>::pack(y + 4, inv) : Code<FORMAT>::pack_any(y + 4, inv));
    }
}

// A warp (a block of threads, team) takes `each` rows of one head's keys or
// values: the runs that begin there.
template <int D, int FORMAT>
__global__ void __launch_bounds__(kThreads, 6)
paged8_append_kernel(const __grid_constant__ Append8Args a, int each, int team)
{
    __shared__ __align__(16) unsigned char smem[kWarps * kHeldBytes];
    __shared__ uint32_t s_maxima[2][2 * kWarps];                      // of two runs in turn
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned int w = team ? blockIdx.x : blockIdx.x * kWarps + warp, columns = 2u * (unsigned int)a.p.Hkv;
    const int column = (int)(w % columns);
    const long long begin = (long long)(w / columns) * each, end = min((long long)a.p.T, begin + each);
    unsigned char* buf = smem + warp * kHeldBytes + lane * 16;
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
    int runs = 0;
    for (long long r0 = begin; r0 < end; r0 += kWindow) {
        // lane l: row r0 - 1 + l, and the 32 after those
        const int slot = slot_of(r0 - 1 + lane), later = slot_of(r0 + 31 + lane), blk = slot >> a.bshift;
        const int before = __shfl_up_sync(0xffffffffu, blk, 1);
        uint32_t leads = __ballot_sync(0xffffffffu, lane >= 1 && r0 - 1 + lane < end && blk >= 0 && blk != before);
        for (; leads; leads &= leads - 1) {
            const int at = __ffs(leads) - 1, b = __shfl_sync(0xffffffffu, blk, at), s0 = __shfl_sync(0xffffffffu, slot, at);
            Run run;
            run.row0 = (int)r0 - 1 + at;
            uint32_t other = __ballot_sync(0xffffffffu, lane >= at && blk != b);
            run.n = (other ? __ffs(other) - 1 : 32) - at;
            const bool mine = lane >= at && lane < at + run.n;
            int first = mine ? slot : 0x7fffffff;
            run.even = __all_sync(0xffffffffu, !mine || slot - s0 == lane - at);
            if (!other) {
                int s = later;
                for (long long i = r0 + 31;; i += 32, s = slot_of(i + lane)) {
                    other = __ballot_sync(0xffffffffu, (s >> a.bshift) != b);
                    const int more = other ? __ffs(other) - 1 : 32;
                    if (lane < more) first = min(first, s);
                    run.even = run.even && __all_sync(0xffffffffu, lane >= more || s - s0 == run.n + lane);
                    run.n += more;
                    if (other) break;
                }
            }
            run.first = __reduce_min_sync(0xffffffffu, first) & ((1 << a.bshift) - 1);
            const int token = (b << a.bshift) & ((1 << a.shift) - 1), page = (b << a.bshift) >> a.shift;
            Place to;
            to.block = (is_v ? a.v_pages : a.k_pages) + page * a.p.page_stride + head * a.p.head_stride + token * a.p.token_stride;
            to.scale = (is_v ? a.v_scales : a.k_scales) + scale_at(page, head, token, a.p.Hkv, a.shift, a.bshift);
            uint32_t* maxima = s_maxima[runs++ & 1];
            if (type == FADKV_F32) quantise<float, D, FORMAT>(a, (const float*)x + head * D, stride, to, run, team, warp, buf, maxima);
            else if (type == FADKV_F16) quantise<__half, D, FORMAT>(a, (const __half*)x + head * D, stride, to, run, team, warp, buf, maxima);
            else quantise<__nv_bfloat16, D, FORMAT>(a, (const __nv_bfloat16*)x + head * D, stride, to, run, team, warp, buf, maxima);
        }
    }
}

template <int D, int FORMAT>
cudaError_t launch_t(const Append8Args& a, cudaStream_t st)
{
    const long long columns = 2ll * a.p.Hkv;
    // A block of tokens that does not fit a warp's buffer is four warps' work (24000 tokens of 8 heads of 128 in blocks of 128, in
    // 16 bits: 29 us, 68 a warp a block), where there are rows for whole ones.
    const int size = a.p.k_dtype == FADKV_F32 || a.p.v_dtype == FADKV_F32 ? 4 : 2;
    const int team = a.p.block * D * size > kHeldBytes && a.p.T > kWindow;
    // Rows a warp (a team) looks for runs in: about a block, less where there are fewer rows than warps to be busy.
    const long long want = a.p.T * columns / (152 * (team ? 6 : 24)), most = a.p.block <= 16 ? 16 : (a.p.block + 31) / 32 * kWindow;
    const int each = (int)std::max(1ll, std::min(want, most));
    const long long warps = (a.p.T + each - 1) / each * columns * (team ? kWarps : 1);
    if (warps > 0x7fffffffll) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    return launch_pdl(paged8_append_kernel<D, FORMAT>, dim3(grid), dim3(kThreads), 0, st, a, each, team);
}

}  // namespace

cudaError_t launch_paged8_append(const Append8Args& a, cudaStream_t st)
{
    if (a.p.T <= 0 || a.p.num_pages <= 0) return cudaSuccess;
    if (a.p.format == FADKV_E4M3) return a.p.d == 128 ? launch_t<128, FADKV_E4M3>(a, st) : launch_t<64, FADKV_E4M3>(a, st);
    return a.p.d == 128 ? launch_t<128, FADKV_I8>(a, st) : launch_t<64, FADKV_I8>(a, st);
}

}  // namespace fadkv
