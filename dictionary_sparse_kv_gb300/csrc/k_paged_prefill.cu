// Attention of chunks of new tokens over the paged cache.
//
// One pass over the keys with the running maximum m and sum l of the softmax:
//   x = scale log2(e) q k^T,  p = 2^(x - m),  o = o 2^(m_old - m) + p v,
// out = o / l.  Rows of a tile are (token, head) pairs of the query heads that
// share a KV head, token by token, so that a key tile that is loaded serves
// the whole group and chunks of a few tokens still fill the rows.
#include "paged.cuh"

namespace fadkv {
namespace {

using namespace paged;

constexpr int kPreThreads = 128;
constexpr int kRows = 64;                          // (token, head) rows per CTA
constexpr int kKeys = 64;                          // keys per tile

template <int D> constexpr int pre_smem() { return 2 * 2 * kKeys * D * 2; }

template <typename T, int D>
__global__ void __launch_bounds__(kPreThreads)
paged_prefill_kernel(const __grid_constant__ PagedArgs a)
{
    constexpr int ROW = D * 2, CPR = D / 8, KS = D / 16, TILE = kKeys * ROW;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ int s_b;
    __shared__ long long s_base;
    __shared__ unsigned char s_ok[2][kKeys];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = a.grp, B = a.p.B;
    const int gch = min(grp, kRows), chunks = (grp + gch - 1) / gch, tq = kRows / gch;   // tokens per tile
    const int hk = blockIdx.y / chunks, h0 = (blockIdx.y % chunks) * gch, hn = min(gch, grp - h0);

    auto rows_of = [&](int b) {
        const int s = a.starts[b];
        return s < 0 ? 0 : max(0, min(a.starts[b + 1], a.p.T) - s);
    };
    {
        const int each = (B + kPreThreads - 1) / kPreThreads, b0 = min(B, tid * each), b1 = min(B, b0 + each);
        long long mine = 0, all;
        for (int b = b0; b < b1; ++b) mine += (rows_of(b) + tq - 1) / tq;
        long long at = block_scan<kPreThreads>(mine, &all);
        const long long u = all - 1 - blockIdx.x;      // the last tiles see the most keys: first
        if (u < 0) return;
        if (u >= at && u < at + mine) {
            int b = b0;
            for (long long n; u >= at + (n = (rows_of(b) + tq - 1) / tq); ++b) at += n;
            s_b = b;
            s_base = u - at;
        }
        __syncthreads();
    }
    const int b = s_b, t0 = (int)s_base * tq, start = a.starts[b];
    const int n = rows_of(b), nt = min(tq, n - t0);
    const int len = clamp_len(a.lengths[b], a);
    // positions by the rows that the request has, those cut off at T included
    const int first = len - (a.starts[b + 1] - start) + t0, last = first + nt - 1;
    const int32_t* table = a.table + (size_t)b * a.p.max_pages;
    const T* kp = (const T*)a.k + hk * a.p.head_stride;
    const T* vp = (const T*)a.v + hk * a.p.head_stride;

    // this thread's two rows of the tile (warp's 16 rows: lane/4 and lane/4 + 8)
    int pos[2], tok[2], hd[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = warp * 16 + (lane >> 2) + 8 * i, t = r / gch;
        const bool live = t < nt && r % gch < hn;
        tok[i] = live ? start + t0 + t : -1;
        hd[i] = hk * grp + h0 + r % gch;
        pos[i] = live ? first + t : -1;
    }
    uint32_t qf[KS][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>((const T*)a.q + (size_t)max(tok[i], 0) * a.p.q_stride +
                                                              (size_t)hd[i] * D) + (lane & 3);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            qf[k][i] = tok[i] >= 0 ? __ldg(q + k * 8) : 0u;
            qf[k][i + 2] = tok[i] >= 0 ? __ldg(q + k * 8 + 4) : 0u;
        }
    }

    // key tiles: those of the first tokens, then those of the window (or all)
    const int W = min(a.p.window, 1 << 30), S = min(a.p.sinks, len);
    const int tiles_to = last >= 0 ? last / kKeys + 1 : 0;
    const int from = W > 0 ? (int)(max(0ll, (long long)first - W + 1) / kKeys) : 0;
    const int sink_tiles = W > 0 ? min(from, (S + kKeys - 1) / kKeys) : 0;
    const int tiles = tiles_to > from ? sink_tiles + tiles_to - from : 0;
    auto key0 = [&](int i) { return (i < sink_tiles ? i : i - sink_tiles + from) * kKeys; };
    auto load = [&](int i) {
        const int s = i & 1, k0 = key0(i);
        const uint32_t dst = saddr(smem) + s * 2 * TILE;
#pragma unroll 4
        for (int j = tid; j < kKeys * CPR; j += kPreThreads) {
            const int r = j / CPR, c = j % CPR, key = k0 + r;
            // keys that no row of the tile sees enter as zeros: what their slots hold may be anything
            const bool any = key <= last && (W == 0 || key > first - W || key < S);
            const int page = any ? __ldg(table + (key >> a.shift)) : -1;
            const bool ok = page >= 0 && page < a.p.num_pages;
            const long long o = ok ? page * a.p.page_stride + (key & ((1 << a.shift) - 1)) * a.p.token_stride + c * 8 : 0;
            if (c == 0) s_ok[s][r] = ok;
            cp16(dst + swz<ROW>(r, c), kp + o, ok);
            cp16(dst + TILE + swz<ROW>(r, c), vp + o, ok);
        }
        cp_commit();
    };

    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < D / 8; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
    if (tiles > 0) load(0);
    for (int i = 0; i < tiles; ++i) {
        if (i + 1 < tiles) {
            load(i + 1);
            cp_wait<1>();
        } else {
            cp_wait<0>();
        }
        __syncthreads();
        const int s = i & 1, k0 = key0(i);
        const uint32_t kt = saddr(smem) + s * 2 * TILE, vt = kt + TILE;
        float sc[kKeys / 8][4];
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int j = 0; j < kKeys / 16; ++j) {
                uint32_t f[4];
                ldsm_x4(f, kt + swz<ROW>(j * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
                Num<T>::mma(sc[2 * j], qf[k], f[0], f[1]);
                Num<T>::mma(sc[2 * j + 1], qf[k], f[2], f[3]);
            }
        float mt[2] = {m[0], m[1]};
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int c = j * 8 + 2 * (lane & 3) + (x & 1), key = k0 + c, p = pos[x >> 1];
                const bool ok = key <= p && (W == 0 || key > p - W || key < S) && s_ok[s][c];
                sc[j][x] = ok ? sc[j][x] * a.scale_log2 : -INFINITY;
                mt[x >> 1] = fmaxf(mt[x >> 1], sc[j][x]);
            }
        float f[2], m0[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            mt[x] = fmaxf(mt[x], __shfl_xor_sync(0xffffffffu, mt[x], 1));
            mt[x] = fmaxf(mt[x], __shfl_xor_sync(0xffffffffu, mt[x], 2));
            f[x] = mt[x] > m[x] ? exp2_fast(m[x] - mt[x]) : 1.f;
            m[x] = mt[x];
            m0[x] = m[x] == -INFINITY ? 0.f : m[x];
            l[x] *= f[x];
        }
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
            o[k][0] *= f[0];
            o[k][1] *= f[0];
            o[k][2] *= f[1];
            o[k][3] *= f[1];
        }
        uint32_t pf[kKeys / 16][4];
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) {
            const float p0 = exp2_fast(sc[j][0] - m0[0]), p1 = exp2_fast(sc[j][1] - m0[0]);
            const float p2 = exp2_fast(sc[j][2] - m0[1]), p3 = exp2_fast(sc[j][3] - m0[1]);
            l[0] += p0 + p1;
            l[1] += p2 + p3;
            pf[j / 2][(j & 1) * 2] = Num<T>::pack(p0, p1);
            pf[j / 2][(j & 1) * 2 + 1] = Num<T>::pack(p2, p3);
        }
#pragma unroll
        for (int j = 0; j < kKeys / 16; ++j)
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t v[4];
                ldsm_x4_trans(v, vt + swz<ROW>(j * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)));
                Num<T>::mma(o[2 * k], pf[j], v[0], v[1]);
                Num<T>::mma(o[2 * k + 1], pf[j], v[2], v[3]);
            }
        __syncthreads();
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        if (tok[x] < 0) continue;
        const float inv = l[x] > 0.f ? 1.f / l[x] : (l[x] == l[x] ? 0.f : l[x]);
        uint32_t* out = reinterpret_cast<uint32_t*>((T*)a.out + (size_t)tok[x] * a.p.out_stride + (size_t)hd[x] * D) +
                        (lane & 3);
#pragma unroll
        for (int k = 0; k < D / 8; ++k) out[k * 4] = Num<T>::pack(o[k][2 * x] * inv, o[k][2 * x + 1] * inv);
        if ((lane & 3) == 0 && a.lse)
            a.lse[(size_t)tok[x] * a.p.Hq + hd[x]] = l[x] == 0.f ? -INFINITY : (m[x] + log2f(l[x])) * kLn2;
    }
}

template <typename T, int D>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t st)
{
    auto k = paged_prefill_kernel<T, D>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, pre_smem<D>());
    if (e != cudaSuccess) return e;
    const int gch = a.grp < kRows ? a.grp : kRows, chunks = (a.grp + gch - 1) / gch, tq = kRows / gch;
    const long long tiles = a.p.T / tq + a.p.B;
    k<<<dim3((unsigned)tiles, (unsigned)(a.p.Hkv * chunks)), kPreThreads, pre_smem<D>(), st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t paged_prefill_workspace(const fadkv_paged_params&) { return 0; }

cudaError_t launch_paged_prefill(const PagedArgs& a, cudaStream_t st)
{
    if (a.p.B <= 0 || a.p.T <= 0) return cudaSuccess;
    if (a.p.dtype == FADKV_F16) return a.p.d == 128 ? launch_t<__half, 128>(a, st) : launch_t<__half, 64>(a, st);
    return a.p.d == 128 ? launch_t<__nv_bfloat16, 128>(a, st) : launch_t<__nv_bfloat16, 64>(a, st);
}

}  // namespace fadkv
