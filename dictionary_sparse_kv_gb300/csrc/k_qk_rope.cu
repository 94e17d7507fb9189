// Norms of queries and keys for each head, rotation of positions, and the
// append to the paged cache, in one pass over a step's projections.
//
// y = rotate(x / sqrt(mean(x^2) + eps) * w).  Pair i at position p turns by
// the angle 2 pi p F_i with F_i a fraction of a turn a position.  F_i is kept
// as a 64-bit fraction, so p F_i mod 1 is an integer product that wraps
// around: exact for every position, where a 32-bit product loses the angle of
// far positions (at position 10^6 it is off by 0.06 radians).  The top 32
// bits of the product are the angle in half turns for sincospi.
//
// The work is T (Hq + 2 Hkv) rows of d elements, read once and written once
// (keys twice with k_out): HBM for long prompts, latency for single tokens.
// A row is d / 8 lanes and a warp takes 32 / (d / 8) rows of one token at a
// time.  A lane holds eight elements as two groups of four: with pairs
// (i, i + rotary_dim / 2) the two groups are partners, with neighbouring pairs
// they are side by side, so a pair is always in one lane, nothing is
// exchanged, and four angles a lane, worked out once a warp for all the rows
// of its token, do for both layouts.  1 / sqrt goes into the cosines and
// sines, and products run two values an instruction.  16384 tokens of 32 + 8
// heads of 128 in bfloat16: 72 us, 6.1 TB/s.
#include "paged.cuh"

namespace fadkv {
namespace {

constexpr int kQkThreads = 128;
constexpr int kUnroll = 2;       // steps a warp works on, while so many more are on their way
constexpr int kValues = 4;       // values' steps in flight

// Four consecutive elements as loaded.
template <typename T> struct Raw4 {
    uint2 a;
    __device__ __forceinline__ void load(const T* p) { a = __ldg(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void get(float* x) const
    {
        const float2 f = paged::Num<T>::unpack(a.x), g = paged::Num<T>::unpack(a.y);
        x[0] = f.x, x[1] = f.y, x[2] = g.x, x[3] = g.y;
    }
};
template <> struct Raw4<float> {
    float4 a;
    __device__ __forceinline__ void load(const float* p) { a = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void get(float* x) const { x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w; }
};

__device__ __forceinline__ void store4(void* base, int dtype, long long at, const float* y)
{
    if (dtype == FADKV_F32) {
        *reinterpret_cast<float4*>((float*)base + at) = make_float4(y[0], y[1], y[2], y[3]);
    } else if (dtype == FADKV_F16) {
        using N = paged::Num<__half>;
        *reinterpret_cast<uint2*>((__half*)base + at) = make_uint2(N::pack(y[0], y[1]), N::pack(y[2], y[3]));
    } else {
        using N = paged::Num<__nv_bfloat16>;
        *reinterpret_cast<uint2*>((__nv_bfloat16*)base + at) = make_uint2(N::pack(y[0], y[1]), N::pack(y[2], y[3]));
    }
}

template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(kQkThreads)
qk_norm_rope_kernel(const __grid_constant__ QkArgs a, int each, int parts)
{
    using paged::add2;
    using paged::fma2;
    using paged::mul2;
    using paged::pair;
    using paged::unpair;
    constexpr int LPR = D / 8;            // lanes per row
    constexpr int RPW = 32 / LPR;         // rows per warp step
    __shared__ unsigned long long turns[FADKV_ROPE_MAX_PAIRS];
    const int rd = a.rope.rotary_dim, half = rd / 2;
    if (threadIdx.x < half) turns[threadIdx.x] = a.rope.turns[threadIdx.x];
    __syncthreads();
    pdl_begin();

    const unsigned int w = blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(w / (unsigned int)parts), part = (int)(w % (unsigned int)parts);
    if (t >= a.p.T) return;
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    const int pos = a.positions[t];
    const int slot = a.slots ? a.slots[t] : -1;
    const bool append = pos >= 0 && slot >= 0 && (slot >> a.shift) < a.p.num_pages;
    const long long at = (long long)(slot >> a.shift) * a.p.page_stride +
                         (long long)(slot & ((1 << a.shift) - 1)) * a.p.token_stride;

    // this lane's two groups: the first rd / 8 lanes of a row take the rotated part
    const bool turned = l < rd / 8;
    const int e0 = PAIRS || !turned ? l * 8 : l * 4, e1 = PAIRS || !turned ? e0 + 4 : e0 + half;
    // Eight values as four pairs of registers: the first members of the pairs that turn, x[0] and x[1], and the second,
    // x[2] and x[3].
    auto pack8 = [](const Raw4<T> (&r)[2], uint64_t (&x)[4]) {
        float f[8];
        r[0].get(f);
        r[1].get(f + 4);
        if (PAIRS) {
            x[0] = pair(f[0], f[2]), x[1] = pair(f[4], f[6]);
            x[2] = pair(f[1], f[3]), x[3] = pair(f[5], f[7]);
        } else {
            x[0] = pair(f[0], f[1]), x[1] = pair(f[2], f[3]);
            x[2] = pair(f[4], f[5]), x[3] = pair(f[6], f[7]);
        }
    };
    auto put = [&](void* base, int dtype, long long row, const uint64_t (&x)[4]) {
        float f[8];
        if (PAIRS) {
            unpair(x[0], f[0], f[2]), unpair(x[1], f[4], f[6]);
            unpair(x[2], f[1], f[3]), unpair(x[3], f[5], f[7]);
        } else {
            unpair(x[0], f[0], f[1]), unpair(x[1], f[2], f[3]);
            unpair(x[2], f[4], f[5]), unpair(x[3], f[6], f[7]);
        }
        store4(base, dtype, row + e0, f);
        store4(base, dtype, row + e1, f + 4);
    };
    // cosines and sines of the four pairs; 1 and 0 where nothing turns (there amplitude does not enter either)
    uint64_t cs[2], sn[2], ns[2];
    {
        float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
        if (turned) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const unsigned long long phase = (unsigned long long)(long long)pos * turns[l * 4 + k];
                sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s[k], &c[k]);
                c[k] *= a.rope.amplitude;
                s[k] *= a.rope.amplitude;
            }
        }
        cs[0] = pair(c[0], c[1]), cs[1] = pair(c[2], c[3]);
        sn[0] = pair(s[0], s[1]), sn[1] = pair(s[2], s[3]);
        ns[0] = pair(-s[0], -s[1]), ns[1] = pair(-s[2], -s[3]);
    }

    // steps of RPW rows: queries, then keys, then values; this warp's from `begin` on, `count` of them
    const int q_steps = (a.p.Hq + RPW - 1) / RPW, kv_steps = (a.p.Hkv + RPW - 1) / RPW;
    const int begin = part * each, end = min(q_steps + 2 * kv_steps, begin + each);

    auto rotated = [&](const T* src, const T* weight, int rows, int s0, int s1, auto&& store) {
        uint64_t wt[4];
        if (weight) {
            Raw4<T> r[2];
            r[0].load(weight + e0), r[1].load(weight + e1);
            pack8(r, wt);
        }
        Raw4<T> raw[kUnroll][2], ahead[kUnroll][2];
        auto load = [&](Raw4<T> (&to)[kUnroll][2], int s) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const T* p = src + (size_t)min((s + u) * RPW + sub, rows - 1) * D;
                to[u][0].load(p + e0);
                to[u][1].load(p + e1);
            }
        };
        load(ahead, s0);
        for (int s = s0; s < s1; s += kUnroll) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) raw[u][0] = ahead[u][0], raw[u][1] = ahead[u][1];
            if (s + kUnroll < s1) load(ahead, s + kUnroll);    // on their way while these are worked on
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (s + u >= s1) break;
                const int h = (s + u) * RPW + sub;
                uint64_t x[4], c[2] = {cs[0], cs[1]}, sp[2] = {sn[0], sn[1]}, sm[2] = {ns[0], ns[1]};
                pack8(raw[u], x);
                if (weight) {
                    float s0f, s1f;
                    unpair(add2(fma2(x[0], x[0], mul2(x[1], x[1])), fma2(x[2], x[2], mul2(x[3], x[3]))), s0f, s1f);
                    float ss = s0f + s1f;
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float inv = rsqrtf(ss * (1.f / D) + a.p.eps);
                    const uint64_t inv2 = pair(inv, inv);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], wt[i]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) c[i] = mul2(c[i], inv2), sp[i] = mul2(sp[i], inv2), sm[i] = mul2(sm[i], inv2);
                }
                uint64_t y[4];
                if (turned) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        y[i] = fma2(x[i], c[i], mul2(x[i + 2], sm[i]));
                        y[i + 2] = fma2(x[i], sp[i], mul2(x[i + 2], c[i]));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = mul2(x[i], c[i & 1]);
                }
                if (pos < 0) y[0] = y[1] = y[2] = y[3] = 0ull;
                if (h < rows) store(h, y);
            }
        }
    };
    if (begin < q_steps)
        rotated((const T*)a.q + t * a.p.q_stride, (const T*)a.wq, a.p.Hq, begin, min(end, q_steps),
                [&](int h, const uint64_t (&y)[4]) { put(a.q_out, a.p.q_dtype, ((long long)t * a.p.Hq + h) * D, y); });
    const int k0 = max(begin - q_steps, 0), k1 = min(end - q_steps, kv_steps);
    if (k0 < k1)
        rotated((const T*)a.k + t * a.p.k_stride, (const T*)a.wk, a.p.Hkv, k0, k1, [&](int h, const uint64_t (&y)[4]) {
            if (a.k_out) put(a.k_out, a.p.kv_dtype, ((long long)t * a.p.Hkv + h) * D, y);
            if (append) put(a.k_pages, a.p.kv_dtype, at + h * a.p.head_stride, y);
        });
    if (!append) return;
    const int v0 = max(begin - q_steps - kv_steps, 0), v1 = end - q_steps - kv_steps;
    for (int s = v0; s < v1; s += kValues) {
        Raw4<T> raw[kValues][2];
        const T* v = (const T*)a.v + t * a.p.v_stride;
#pragma unroll
        for (int u = 0; u < kValues; ++u) {
            const T* p = v + (size_t)min((s + u) * RPW + sub, a.p.Hkv - 1) * D;
            raw[u][0].load(p + e0);
            raw[u][1].load(p + e1);
        }
#pragma unroll
        for (int u = 0; u < kValues; ++u) {
            const int h = (s + u) * RPW + sub;
            if (s + u >= v1 || h >= a.p.Hkv) break;
            uint64_t x[4];
            pack8(raw[u], x);
            put(a.v_pages, a.p.kv_dtype, at + h * a.p.head_stride, x);
        }
    }
}

template <typename T, int D>
cudaError_t launch_t(const QkArgs& a, cudaStream_t st)
{
    constexpr int RPW = 32 / (D / 8);
    const long long steps = (a.p.Hq + RPW - 1) / RPW + 2 * ((a.p.Hkv + RPW - 1) / RPW);
    // A token's steps are cut into as many even parts as give every
    // multiprocessor (152) some 16 warps, and not more: the angles are worked
    // out once a warp.  (1024 tokens of 32 + 8 heads: 7.1 us in 4 parts, 9.5
    // in 8; 4096: 19.2 us in one part, 24.8 in two.)
    const long long want = (152ll * 16 + a.p.T - 1) / a.p.T;
    const long long each = (steps + (want < steps ? want : steps) - 1) / (want < steps ? want : steps);
    const int parts = (int)((steps + each - 1) / each);
    const long long warps = (long long)a.p.T * parts;
    if (warps > 0x7fffffffll) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)((warps + kQkThreads / 32 - 1) / (kQkThreads / 32));
    return launch_pdl(a.rope.interleaved ? qk_norm_rope_kernel<T, D, true> : qk_norm_rope_kernel<T, D, false>, dim3(grid),
                      dim3(kQkThreads), 0, st, a, (int)each, parts);
}

template <typename T>
cudaError_t launch_d(const QkArgs& a, cudaStream_t st)
{
    return a.p.d == 128 ? launch_t<T, 128>(a, st) : launch_t<T, 64>(a, st);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkArgs& a, cudaStream_t st)
{
    if (a.p.T <= 0) return cudaSuccess;
    if (a.p.dtype == FADKV_F32) return launch_d<float>(a, st);
    if (a.p.dtype == FADKV_F16) return launch_d<__half>(a, st);
    return launch_d<__nv_bfloat16>(a, st);
}

}  // namespace fadkv
