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
// Eight elements a lane (one or two 16-byte loads), so a row is d / 8 lanes
// and a warp takes 32 / (d / 8) rows of one token at a time; the angles of a
// token are worked out once a warp and used for all the rows it takes.
#include "paged.cuh"

namespace fadkv {
namespace {

constexpr int kQkThreads = 256;
constexpr int kUnroll = 4;       // rows in flight a lane

template <typename T> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
template <typename T> struct Raw8 {
    uint4 a;
    __device__ __forceinline__ void load(const T* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = paged::Num<T>::unpack(u[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};

__device__ __forceinline__ void store8(void* base, int dtype, long long at, const float (&y)[8])
{
    if (dtype == FADKV_F32) {
        float4* p = reinterpret_cast<float4*>((float*)base + at);
        p[0] = make_float4(y[0], y[1], y[2], y[3]);
        p[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else if (dtype == FADKV_F16) {
        using N = paged::Num<__half>;
        *reinterpret_cast<uint4*>((__half*)base + at) =
            make_uint4(N::pack(y[0], y[1]), N::pack(y[2], y[3]), N::pack(y[4], y[5]), N::pack(y[6], y[7]));
    } else {
        using N = paged::Num<__nv_bfloat16>;
        *reinterpret_cast<uint4*>((__nv_bfloat16*)base + at) =
            make_uint4(N::pack(y[0], y[1]), N::pack(y[2], y[3]), N::pack(y[4], y[5]), N::pack(y[6], y[7]));
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

    const long long w = (long long)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(w / parts), part = (int)(w % parts);
    if (t >= a.p.T) return;
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR, e0 = l * 8;
    const int Hq = a.p.Hq, Hkv = a.p.Hkv, rows = Hq + 2 * Hkv;
    const int pos = a.positions[t];
    const int slot = a.slots ? a.slots[t] : -1;
    const bool append = pos >= 0 && slot >= 0 && (slot >> a.shift) < a.p.num_pages;
    const long long at = (long long)(slot >> a.shift) * a.p.page_stride +
                         (long long)(slot & ((1 << a.shift) - 1)) * a.p.token_stride;

    // cosines and sines of this lane's elements (pairs: one a pair of them)
    const bool turned = e0 < rd;
    float cs[8], sn[8];
    int partner = lane;
    if (turned) {
        const int i0 = PAIRS ? e0 / 2 : (e0 < half ? e0 : e0 - half);
#pragma unroll
        for (int k = 0; k < (PAIRS ? 4 : 8); ++k) {
            const unsigned long long phase = (unsigned long long)(long long)pos * turns[i0 + k];
            sincospif((float)(int)(phase >> 32) * 0x1p-31f, &sn[k], &cs[k]);
            cs[k] *= a.rope.amplitude;
            sn[k] *= a.rope.amplitude;
            if (!PAIRS && e0 < half) sn[k] = -sn[k];
        }
        if (!PAIRS) partner = sub * LPR + (e0 < half ? l + half / 8 : l - half / 8);
    }
    float wq[8], wk[8];
    if (a.wq) {
        Raw8<T> r;
        r.load((const T*)a.wq + e0);
        r.get(wq);
    }
    if (a.wk) {
        Raw8<T> r;
        r.load((const T*)a.wk + e0);
        r.get(wk);
    }

    const T* q = (const T*)a.q + t * a.p.q_stride + e0;
    const T* k = (const T*)a.k + t * a.p.k_stride + e0;
    const T* v = (const T*)a.v + t * a.p.v_stride + e0;
    const int last = min(rows, (part + 1) * each * RPW);
    for (int r0 = part * each * RPW; r0 < last; r0 += RPW * kUnroll) {
        Raw8<T> raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = min(r0 + u * RPW + sub, rows - 1);
            raw[u].load(r < Hq ? q + r * D : r < Hq + Hkv ? k + (r - Hq) * D : v + (r - Hq - Hkv) * D);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = r0 + u * RPW + sub;
            float x[8];
            raw[u].get(x);
            const bool is_q = r < Hq, is_v = r >= Hq + Hkv;
            if (a.wq || a.wk) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = rsqrtf(ss * (1.f / D) + a.p.eps);
                if (is_q ? a.wq != nullptr : (!is_v && a.wk != nullptr)) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * (is_q ? wq[i] : wk[i]);
                }
            }
            if (rd > 0) {
                float y[8];
                if (PAIRS) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
                        y[2 * i + 1] = x[2 * i] * sn[i] + x[2 * i + 1] * cs[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = x[i] * cs[i] + __shfl_sync(0xffffffffu, x[i], partner) * sn[i];
                }
                if (turned && !is_v)
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = y[i];
            }
            if (r >= last) continue;
            if (!is_v && pos < 0)
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.f;
            if (is_q) {
                store8(a.q_out, a.p.q_dtype, ((long long)t * Hq + r) * D + e0, x);
            } else if (!is_v) {
                const int h = r - Hq;
                if (a.k_out) store8(a.k_out, a.p.kv_dtype, ((long long)t * Hkv + h) * D + e0, x);
                if (append) store8(a.k_pages, a.p.kv_dtype, at + h * a.p.head_stride + e0, x);
            } else if (append) {
                store8(a.v_pages, a.p.kv_dtype, at + (r - Hq - Hkv) * a.p.head_stride + e0, x);
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
