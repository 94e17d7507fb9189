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
// of its token, do for both layouts.
#include "paged.cuh"

namespace fadkv {
namespace {

constexpr int kQkThreads = 256;
constexpr int kUnroll = 4;       // rows in flight a lane

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
    constexpr int LPR = D / 8;            // lanes per row
    constexpr int RPW = 32 / LPR;         // rows per warp step
    __shared__ unsigned long long turns[FADKV_ROPE_MAX_PAIRS];
    const int rd = a.rope.rotary_dim, half = rd / 2;
    if (threadIdx.x < half) turns[threadIdx.x] = a.rope.turns[threadIdx.x];
    __syncthreads();

    const unsigned int w = blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(w / (unsigned int)parts), part = (int)(w % (unsigned int)parts);
    if (t >= a.p.T) return;
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    const int Hq = a.p.Hq, Hk = Hq + a.p.Hkv, rows = Hk + a.p.Hkv;   // rows: queries, keys, values
    const int pos = a.positions[t];
    const int slot = a.slots ? a.slots[t] : -1;
    const bool append = pos >= 0 && slot >= 0 && (slot >> a.shift) < a.p.num_pages;
    const long long at = (long long)(slot >> a.shift) * a.p.page_stride +
                         (long long)(slot & ((1 << a.shift) - 1)) * a.p.token_stride;

    // this lane's two groups: the first rd / 8 lanes of a row take the rotated part
    const bool turned = l < rd / 8;
    const int e0 = PAIRS || !turned ? l * 8 : l * 4, e1 = PAIRS || !turned ? e0 + 4 : e0 + half;
    float cs[4], sn[4];
    if (turned) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned long long phase = (unsigned long long)(long long)pos * turns[l * 4 + k];
            sincospif((float)(int)(phase >> 32) * 0x1p-31f, &sn[k], &cs[k]);
            cs[k] *= a.rope.amplitude;
            sn[k] *= a.rope.amplitude;
        }
    }
    const bool norm = a.wq || a.wk;
    float wq[8], wk[8];
    if (a.wq) {
        Raw4<T> r[2];
        r[0].load((const T*)a.wq + e0), r[1].load((const T*)a.wq + e1);
        r[0].get(wq), r[1].get(wq + 4);
    }
    if (a.wk) {
        Raw4<T> r[2];
        r[0].load((const T*)a.wk + e0), r[1].load((const T*)a.wk + e1);
        r[0].get(wk), r[1].get(wk + 4);
    }

    const T* q = (const T*)a.q + t * a.p.q_stride;
    const T* k = (const T*)a.k + t * a.p.k_stride;
    const T* v = (const T*)a.v + t * a.p.v_stride;
    const int last = min(rows, (part + 1) * each * RPW);
    for (int r0 = part * each * RPW; r0 < last; r0 += RPW * kUnroll) {
        Raw4<T> raw[kUnroll][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = min(r0 + u * RPW + sub, rows - 1);
            const T* p = r < Hq ? q + r * D : r < Hk ? k + (r - Hq) * D : v + (r - Hk) * D;
            raw[u][0].load(p + e0);
            raw[u][1].load(p + e1);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (r0 + u * RPW >= last) break;
            const int r = r0 + u * RPW + sub;
            float x[8];
            raw[u][0].get(x);
            raw[u][1].get(x + 4);
            const bool is_q = r < Hq;
            if (r0 + u * RPW < Hk) {                       // not values alone
                const bool is_v = r >= Hk;
                if (norm) {
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s0 = fmaf(x[i], x[i], s0);
                        s1 = fmaf(x[i + 4], x[i + 4], s1);
                    }
                    float ss = s0 + s1;
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float inv = rsqrtf(ss * (1.f / D) + a.p.eps);
                    if (is_q ? a.wq != nullptr : (!is_v && a.wk != nullptr)) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] *= inv * (is_q ? wq[i] : wk[i]);
                    }
                }
                if (turned && !is_v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& p0 = PAIRS ? x[2 * i] : x[i];
                        float& p1 = PAIRS ? x[2 * i + 1] : x[i + 4];
                        const float c = p0 * cs[i] - p1 * sn[i];
                        p1 = p0 * sn[i] + p1 * cs[i];
                        p0 = c;
                    }
                }
                if (!is_v && pos < 0)
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = 0.f;
            }
            if (r >= last) continue;
            auto put = [&](void* base, int dtype, long long row) {
                store4(base, dtype, row + e0, x);
                store4(base, dtype, row + e1, x + 4);
            };
            if (is_q) {
                put(a.q_out, a.p.q_dtype, ((long long)t * Hq + r) * D);
            } else if (r < Hk) {
                const int h = r - Hq;
                if (a.k_out) put(a.k_out, a.p.kv_dtype, ((long long)t * a.p.Hkv + h) * D);
                if (append) put(a.k_pages, a.p.kv_dtype, at + h * a.p.head_stride);
            } else if (append) {
                put(a.v_pages, a.p.kv_dtype, at + (r - Hk) * a.p.head_stride);
            }
        }
    }
}

template <typename T, int D>
cudaError_t launch_t(const QkArgs& a, cudaStream_t st)
{
    constexpr int RPW = 32 / (D / 8);
    const long long steps = (a.p.Hq + 2 * a.p.Hkv + RPW - 1) / RPW;
    // warp steps a warp takes: one while the warps do not fill the GPU (152
    // multiprocessors of 64 warps), then up to a whole token, so that the
    // angles are worked out as few times as that allows
    long long each = (long long)a.p.T * steps / (152 * 64);
    each = each < 1 ? 1 : each > steps ? steps : each;
    if (each > kUnroll) each = (each + kUnroll - 1) / kUnroll * kUnroll;
    const int parts = (int)((steps + each - 1) / each);
    const long long warps = (long long)a.p.T * parts;
    if (warps > 0x7fffffffll) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)((warps + kQkThreads / 32 - 1) / (kQkThreads / 32));
    if (a.rope.interleaved)
        qk_norm_rope_kernel<T, D, true><<<grid, kQkThreads, 0, st>>>(a, (int)each, parts);
    else
        qk_norm_rope_kernel<T, D, false><<<grid, kQkThreads, 0, st>>>(a, (int)each, parts);
    return cudaGetLastError();
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
