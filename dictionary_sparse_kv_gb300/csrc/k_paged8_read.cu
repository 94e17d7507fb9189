// Reads tokens of the 8-bit pages back as full vectors: code * scale in 32
// bits, rounded once.
//
// Codes are read and vectors written once: HBM.  The work is one list of
// 16-token tiles, request by request, tile by tile and head by head; every CTA
// takes an even contiguous share, its warps every fourth tile of it, keys and
// values together.  A warp has the next tile's codes on their way while it
// stores one, and has looked up the place of the one behind it.  8 requests of
// up to 4096 tokens of 8 heads of 128 to binary16: 25 us, 5.3 TB/s (3 us of them
// until the first codes arrive); 113 times the last 1024 tokens of two heads of
// 64: 17.4 us (one tile in flight a warp: 18.8).
#include "paged8.cuh"

namespace fadkv {
namespace {

using namespace paged8;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;
// CTAs a multiprocessor: what the registers of two tiles in flight allow.
template <int D> constexpr int kPerSm = D == 128 ? 4 : 6;

// SECTORS: the output pools lie on multiples of 32 bytes (the launcher looks), and so does every row of them, whose strides are
// multiples of 32 bytes.  (16 requests of up to 4096 tokens of 8 heads of 128 to 32 bits: 58 us; two 16-byte stores, a sector's
// halves apart, 74.)
template <bool SECTORS>
__device__ __forceinline__ void store8(float* p, const float* y)
{
    if (SECTORS) {
        // (32 bytes a lane in one instruction: a sector is written whole)
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]),
                     "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7])
                     : "memory");
    } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
}
template <bool SECTORS, typename T>
__device__ __forceinline__ void store8(T* p, const float* y)
{
    *reinterpret_cast<uint4*>(p) = make_uint4(Num<T>::pack(y[0], y[1]), Num<T>::pack(y[2], y[3]), Num<T>::pack(y[4], y[5]),
                                              Num<T>::pack(y[6], y[7]));
}

template <typename T, int D, int FORMAT, bool SECTORS>
__global__ void __launch_bounds__(kThreads, kPerSm<D>)
paged8_read_kernel(const __grid_constant__ Read8Args a)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, STEPS = kTile / RPW;    // lanes a row, rows a step, steps a tile
    __shared__ int s_b;
    __shared__ long long s_base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.p.B, heads = a.p.Hkv;
    const int most = a.p.max_pages << a.shift;
    prefetch_tables(a.lengths, a.table, B, a.p.max_pages);
    pdl_begin();

    // tokens lo .. hi-1 of request b, in tiles from t0 on
    struct Range { int lo, hi, t0, tiles; };
    auto range = [&](int b) {
        Range r;
        r.hi = min(max(__ldg(a.lengths + b), 0), most);
        r.lo = a.first ? max(__ldg(a.first + b), 0) : 0;
        r.t0 = r.lo / kTile;
        r.tiles = r.hi > r.lo ? (r.hi + kTile - 1) / kTile - r.t0 : 0;
        return r;
    };
    long long U, u, u1, base;
    int cur;
    {
        const int each = (B + kThreads - 1) / kThreads, b0 = min(B, tid * each), b1 = min(B, b0 + each);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += (long long)range(b).tiles * heads;
        long long at = paged::block_scan<kThreads>(mine, &U);
        if (U == 0) return;
        const long long C = min((long long)gridDim.x, U);
        if ((long long)blockIdx.x >= C) return;
        u = U * blockIdx.x / C;
        u1 = U * (blockIdx.x + 1) / C;
        if (u >= at && u < at + mine) {
            int b = b0;
            for (long long n; u >= at + (n = (long long)range(b).tiles * heads); ++b) at += n;
            s_b = b;
            s_base = at;
        }
        __syncthreads();
        cur = s_b;
        base = s_base;
    }
    // where a unit's tile lies: page (-1: nothing to do) and output page, scales, tokens lo .. hi-1 of it
    struct Tile { int page, head, at, lo, hi; long long to; float ks, vs; };
    auto locate = [&](long long u) {
        Tile t;
        t.page = -1;
        t.head = t.at = t.lo = t.hi = 0;
        if (u >= u1) return t;
        Range r = range(cur);
        while (u >= base + (long long)r.tiles * heads) {
            base += (long long)r.tiles * heads;
            r = range(++cur);
        }
        const long long rel = u - base;
        const int tile = rel < 0x7fffffffll ? (int)rel / heads : (int)(rel / heads);
        const int token = (r.t0 + tile) * kTile, column = token >> a.shift;
        const long long entry = (long long)cur * a.p.max_pages + column;
        t.head = (int)(rel - (long long)tile * heads);
        t.at = token & ((1 << a.shift) - 1);
        t.lo = r.lo - token;
        t.hi = r.hi - token;
        t.page = __ldg(a.table + entry);
        t.to = a.out_table ? __ldg(a.out_table + entry) : entry;
        if (t.page >= a.p.num_pages || t.to < 0 || t.to >= a.p.out_pages) t.page = -1;
        if (t.page >= 0) {
            const size_t sc = scale_at(t.page, t.head, t.at, heads, a.shift, a.bshift);
            t.ks = __ldg(a.k_scales + sc);
            t.vs = __ldg(a.v_scales + sc);
        }
        return t;
    };
    const int sub = lane / LPR, l = lane % LPR;
    struct Codes { uint2 c[2][STEPS]; };
    const long long from_step = RPW * a.p.token_stride, to_step = RPW * a.p.out_token_stride;
    auto load = [&](const Tile& t, Codes& x) {
        if (t.page < 0) return;
        const long long from = t.page * a.p.page_stride + t.head * a.p.head_stride + (t.at + sub) * a.p.token_stride + l * 8;
        const uint8_t *k = a.k_pages + from, *v = a.v_pages + from;
        if (t.lo <= 0 && t.hi >= kTile) {
#pragma unroll
            for (int j = 0; j < STEPS; ++j, k += from_step, v += from_step) {
                x.c[0][j] = __ldg(reinterpret_cast<const uint2*>(k));
                x.c[1][j] = __ldg(reinterpret_cast<const uint2*>(v));
            }
        } else {
#pragma unroll
            for (int j = 0; j < STEPS; ++j, k += from_step, v += from_step) {
                const int i = j * RPW + sub;
                const bool live = i >= t.lo && i < t.hi;
                x.c[0][j] = live ? __ldg(reinterpret_cast<const uint2*>(k)) : make_uint2(0u, 0u);
                x.c[1][j] = live ? __ldg(reinterpret_cast<const uint2*>(v)) : make_uint2(0u, 0u);
            }
        }
    };
    auto store = [&](const Tile& t, const Codes& x) {
        if (t.page < 0) return;
        const long long dst = t.to * a.p.out_page_stride + t.head * a.p.out_head_stride + (t.at + sub) * a.p.out_token_stride + l * 8;
        const bool full = t.lo <= 0 && t.hi >= kTile;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            T* out = (T*)(kv ? a.v_out : a.k_out) + dst;
            const float s = kv ? t.vs : t.ks;
#pragma unroll
            for (int j = 0; j < STEPS; ++j, out += to_step) {
                const uint2 c = x.c[kv][j];
                if (!full && (j * RPW + sub < t.lo || j * RPW + sub >= t.hi)) continue;
                float y[8];
                values<FORMAT>(c.x, y);
                values<FORMAT>(c.y, y + 4);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= s;
                store8<SECTORS>(out, y);
            }
        }
    };
    // a tile's codes are on their way while the one before it is stored, and the place of the one behind it is looked up
    Codes now, ahead;
    u += warp;
    Tile t = locate(u);
    load(t, now);
    Tile next = locate(u + kWarps);
    for (; u < u1; u += kWarps) {
        load(next, ahead);
        const Tile after = locate(u + 2 * kWarps);
        store(t, now);
        now = ahead;
        t = next;
        next = after;
    }
}

template <typename T, int D, bool SECTORS>
cudaError_t launch_t(const Read8Args& a, cudaStream_t st)
{
    // an upper bound of the tiles: lengths are known on the device only
    const long long tiles = (((long long)a.p.max_pages << a.shift) / kTile) * a.p.B * a.p.Hkv;
    const long long ctas = 152 * kPerSm<D>;
    const unsigned grid = (unsigned)(tiles < ctas ? tiles : ctas);
    return launch_pdl(a.p.format == FADKV_E4M3 ? paged8_read_kernel<T, D, FADKV_E4M3, SECTORS> : paged8_read_kernel<T, D, FADKV_I8, SECTORS>,
                      dim3(grid), dim3(kThreads), 0, st, a);
}

template <typename T, bool SECTORS = false>
cudaError_t launch_d(const Read8Args& a, cudaStream_t st)
{
    return a.p.d == 128 ? launch_t<T, 128, SECTORS>(a, st) : launch_t<T, 64, SECTORS>(a, st);
}

}  // namespace

cudaError_t launch_paged8_read(const Read8Args& a, cudaStream_t st)
{
    if (a.p.B <= 0 || a.p.num_pages <= 0 || a.p.out_pages <= 0) return cudaSuccess;
    if (a.p.out_dtype == FADKV_F32) {
        // 32-bit pools may lie 16 bytes off a sector
        const bool sectors = (((uintptr_t)a.k_out | (uintptr_t)a.v_out) & 31u) == 0;
        return sectors ? launch_d<float, true>(a, st) : launch_d<float>(a, st);
    }
    if (a.p.out_dtype == FADKV_F16) return launch_d<__half>(a, st);
    return launch_d<__nv_bfloat16>(a, st);
}

}  // namespace fadkv
