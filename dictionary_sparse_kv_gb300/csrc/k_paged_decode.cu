// Attention of one new token per request over the paged cache.
//
// out = sum_j p_j v_j / sum_j p_j with p_j = 2^(x_j - m), x_j = scale log2(e)
// <q, k_j>, m the running maximum: one pass over the keys and values, the sums
// rescaled when m grows.  Partial results (m, l = sum p, o = sum p v) of
// disjoint key sets join by
//   m = max m_i,  l = sum 2^(m_i - m) l_i,  o = sum 2^(m_i - m) o_i.
//
// The keys and values that are seen have to be read once: HBM.  The work is
// one list of 64-token blocks, request by request and KV head by KV head; every
// CTA takes an even contiguous share of it, so long and short requests mix
// without a tail, and a share may begin or end inside a (request, KV head).
// Such pieces go to the workspace, and the CTA that arrives last at a
// (request, KV head) joins its pieces in their order: one launch, and results
// that do not depend on which CTA that was.
//
// Inside a CTA each of four warps takes every fourth 16-token tile through a
// pipeline of its own (cp.async, one block-table lookup per token), with its
// own m, l and o; nothing synchronises the warps until the piece ends.  The
// products run on the warp's matrix instructions with the tokens as rows and
// the query heads that share the KV head as the eight columns:
//   S^T = K Q^T   [16 tokens][8 heads],   O^T += V^T P^T   [d][8 heads],
// so a group of up to eight heads fills one instruction and nothing is padded
// to 16 rows of queries.  P enters as two 16-bit terms (hi + lo): the tensor
// pipe is idle most of the time here, and the output is then as exact as one
// computed in 32 bits.
#include "paged.cuh"

namespace fadkv {
namespace {

using namespace paged;

constexpr int kDecThreads = 128;
constexpr int kDecWarps = kDecThreads / 32;
constexpr int kTile = 16;                          // tokens per warp step
constexpr int kBlock = kTile * kDecWarps;          // tokens per unit of work
constexpr int kDecCtas = 304;                      // two per multiprocessor (152)
constexpr int kMaxHeads = 16;                      // query heads per piece; larger groups are several pieces
constexpr size_t kCounterBytes = 4096;             // at the workspace's start whatever the parameters

template <int D> struct DecCfg {
    static constexpr int STAGES = D == 128 ? 3 : 6;
    static constexpr int TILE_BYTES = kTile * D * 2;
    static constexpr int WARP_BYTES = STAGES * 2 * TILE_BYTES;
    static constexpr int SMEM = kDecWarps * WARP_BYTES;
};

struct Piece {                                     // layout of the workspace behind the counters
    static __host__ __device__ constexpr size_t floats(int d) { return (size_t)kMaxHeads * (d + 2); }
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kDecThreads)
paged_decode_kernel(const __grid_constant__ PagedArgs a)
{
    using Cfg = DecCfg<D>;
    constexpr int STAGES = Cfg::STAGES, ROW = D * 2, CPR = D / 8;      // bytes and 16-byte chunks per row
    constexpr int KS = D / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ int s_b, s_last;
    __shared__ long long s_base;
    __shared__ float s_m[kDecWarps][8 * NT], s_l[kDecWarps][8 * NT];
    __shared__ uint32_t s_ok[kDecWarps][STAGES];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = a.p.Hkv, grp = a.grp, B = a.p.B;
    const int chunks = (grp + 8 * NT - 1) / (8 * NT);                 // pieces per KV head
    const int segs = Hkv * chunks;
    unsigned char* wsm = smem + warp * Cfg::WARP_BYTES;
    const uint32_t wbase = saddr(wsm);

    // blocks of a request: at least one, so that one which sees nothing is written too
    auto blocks = [&](int b) { return max(1, (seen_of(clamp_len(a.lengths[b], a), a).count + kBlock - 1) / kBlock); };
    long long u0, u1, U;
    int C;
    {
        const int each = (B + kDecThreads - 1) / kDecThreads, b0 = min(B, tid * each), b1 = min(B, b0 + each);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += (long long)blocks(b) * segs;
        long long at = block_scan<kDecThreads>(mine, &U);
        C = (int)min((long long)gridDim.x, U);
        if ((int)blockIdx.x >= C) return;
        u0 = U * blockIdx.x / C;
        u1 = U * (blockIdx.x + 1) / C;
        if (u0 >= at && u0 < at + mine) {
            int b = b0;
            for (long long n; u0 >= at + (n = (long long)blocks(b) * segs); ++b) at += n;
            s_b = b;
            s_base = at;
        }
        __syncthreads();
    }
    int b = s_b;
    long long base = s_base;

    for (long long u = u0; u < u1;) {
        const int len = clamp_len(a.lengths[b], a);
        const Seen seen = seen_of(len, a);
        const int nb = max(1, (seen.count + kBlock - 1) / kBlock);
        const int seg = (int)((u - base) / nb), blk0 = (int)((u - base) % nb);
        const int blk1 = (int)min((long long)nb, blk0 + (u1 - u));
        const int hk = seg / chunks, h0 = (seg % chunks) * 8 * NT, hn = min(8 * NT, grp - h0);
        const size_t head0 = (size_t)hk * grp + h0;
        const T* kp = (const T*)a.k + hk * a.p.head_stride;
        const T* vp = (const T*)a.v + hk * a.p.head_stride;
        const int32_t* table = a.table + (size_t)b * a.p.max_pages;
        const int end = min(blk1 * kBlock, seen.count);               // list indices of this piece: [blk0 kBlock, end)
        const int tile0 = blk0 * kDecWarps + warp;
        const int tiles = max(0, ((end + kTile - 1) / kTile - tile0 + kDecWarps - 1) / kDecWarps);

        // queries as the B operand: lane holds head lane/4, elements 2 (lane % 4) + {0, 1} of each half step
        uint32_t qf[NT][KS][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int h = n * 8 + (lane >> 2);
            const uint32_t* q = reinterpret_cast<const uint32_t*>((const T*)a.q + (size_t)b * a.p.q_stride +
                                                                  (head0 + (h < hn ? h : 0)) * D) + (lane & 3);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[n][k][0] = h < hn ? __ldg(q + k * 8) : 0u;
                qf[n][k][1] = h < hn ? __ldg(q + k * 8 + 4) : 0u;
            }
        }

        // lane (and lane + 16): token lane % 16 of a tile
        auto token_of = [&](int tile) {
            const int i = (tile0 + tile * kDecWarps) * kTile + (lane & 15);
            return i < end ? (i < seen.first ? i : i - seen.first + seen.from) : -1;
        };
        auto page_of = [&](int tok) { return tok >= 0 ? __ldg(table + (tok >> a.shift)) : -1; };
        auto load = [&](int tile, int tok, int page) {
            const int s = tile % STAGES;
            const bool ok = page >= 0 && page < a.p.num_pages;
            const long long off = ok ? page * a.p.page_stride + (tok & ((1 << a.shift) - 1)) * a.p.token_stride : 0;
            const uint32_t oks = __ballot_sync(0xffffffffu, ok);
            if (lane == 0) s_ok[warp][s] = oks;
            const uint32_t dst = wbase + s * 2 * Cfg::TILE_BYTES;
#pragma unroll
            for (int j = 0; j < kTile * CPR / 32; ++j) {
                const int r = (j * 32 + lane) / CPR, c = (j * 32 + lane) % CPR;
                const long long o = __shfl_sync(0xffffffffu, off, r) + c * 8;
                const bool v = (oks >> r) & 1u;
                cp16(dst + swz<ROW>(r, c), kp + o, v);
                cp16(dst + Cfg::TILE_BYTES + swz<ROW>(r, c), vp + o, v);
            }
        };

        float o[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }

        int tok = tiles > 0 ? token_of(0) : -1, page = page_of(tok);
        for (int t = 0; t < STAGES - 1; ++t) {
            if (t < tiles) {
                load(t, tok, page);
                tok = token_of(t + 1);
                page = page_of(tok);
            }
            cp_commit();
        }
        for (int t = 0; t < tiles; ++t) {
            cp_wait<STAGES - 2>();
            __syncwarp();
            if (t + STAGES - 1 < tiles) {
                load(t + STAGES - 1, tok, page);
                tok = token_of(t + STAGES);
                page = page_of(tok);
            }
            cp_commit();
            const int s = t % STAGES;
            const uint32_t kt = wbase + s * 2 * Cfg::TILE_BYTES, vt = kt + Cfg::TILE_BYTES;
            const uint32_t oks = s_ok[warp][s];

            float sc[NT][4], sc2[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[n][i] = sc2[n][i] = 0.f;
            {
                const int r = (lane & 7) + ((lane >> 3) & 1) * 8, c = lane >> 4;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t f[4];
                    ldsm_x4(f, kt + swz<ROW>(r, 2 * k + c));
#pragma unroll
                    for (int n = 0; n < NT; ++n) Num<T>::mma(k & 1 ? sc2[n] : sc[n], f, qf[n][k][0], qf[n][k][1]);
                }
            }
            const bool ok0 = (oks >> (lane >> 2)) & 1u, ok1 = (oks >> ((lane >> 2) + 8)) & 1u;
            float mt[NT][2];
            bool grew = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sc[n][i] = (i < 2 ? ok0 : ok1) ? (sc[n][i] + sc2[n][i]) * a.scale_log2 : -INFINITY;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v = fmaxf(sc[n][i], sc[n][i + 2]);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    mt[n][i] = fmaxf(v, m[n][i]);
                    grew |= mt[n][i] > m[n][i];
                }
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float f0 = mt[n][0] > m[n][0] ? exp2_fast(m[n][0] - mt[n][0]) : 1.f;
                    const float f1 = mt[n][1] > m[n][1] ? exp2_fast(m[n][1] - mt[n][1]) : 1.f;
                    m[n][0] = mt[n][0];
                    m[n][1] = mt[n][1];
                    l[n][0] *= f0;
                    l[n][1] *= f1;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        o[n][k][0] *= f0;
                        o[n][k][1] *= f1;
                        o[n][k][2] *= f0;
                        o[n][k][3] *= f1;
                    }
                }
            }
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                // a head that has seen nothing yet: every score is -inf and every p is 0
                const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
                const float p0 = exp2_fast(sc[n][0] - m0), p1 = exp2_fast(sc[n][1] - m1);
                const float p2 = exp2_fast(sc[n][2] - m0), p3 = exp2_fast(sc[n][3] - m1);
                l[n][0] += p0 + p2;
                l[n][1] += p1 + p3;
                const uint32_t a0 = Num<T>::pack(p0, p1), a1 = Num<T>::pack(p2, p3);
                const float2 r0 = Num<T>::unpack(a0), r1 = Num<T>::unpack(a1);
                ph[n][0] = transpose8(a0);
                ph[n][1] = transpose8(a1);
                pl[n][0] = transpose8(Num<T>::pack(p0 - r0.x, p1 - r0.y));
                pl[n][1] = transpose8(Num<T>::pack(p2 - r1.x, p3 - r1.y));
            }
            {
                const int r = (lane & 7) + (lane >> 4) * 8, c = (lane >> 3) & 1;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t f[4];
                    ldsm_x4_trans(f, vt + swz<ROW>(r, 2 * k + c));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        Num<T>::mma(o[n][k], f, ph[n][0], ph[n][1]);
                        Num<T>::mma(o[n][k], f, pl[n][0], pl[n][1]);
                    }
                }
            }
        }
        cp_wait<0>();
        __syncwarp();

        // the warps' results, through the (now idle) pipeline buffers: [head][D] per warp
        float* wo = reinterpret_cast<float*>(wsm);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v = l[n][i];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                const int h = n * 8 + 2 * (lane & 3) + i;
                if (lane < 4) {
                    s_m[warp][h] = m[n][i];
                    s_l[warp][h] = v;
                }
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    wo[h * D + k * 16 + (lane >> 2)] = o[n][k][i];
                    wo[h * D + k * 16 + (lane >> 2) + 8] = o[n][k][i + 2];
                }
            }
        __syncthreads();
        const bool whole = blk0 == 0 && blk1 == nb;
        float* piece = reinterpret_cast<float*>((unsigned char*)a.ws + kCounterBytes);
        const size_t psize = Piece::floats(D);
        float* mine = piece + (2 * (size_t)blockIdx.x + (blk0 == 0 ? 1 : 0)) * psize;
        auto finish = [&](int h, int c, float mh, float lh, float oh) {
            const size_t row = (size_t)b * a.p.Hq + head0 + h;
            T* out = (T*)a.out + (size_t)b * a.p.out_stride + (head0 + h) * D;
            const float y = lh > 0.f ? oh / lh : (lh == lh ? 0.f : lh);
            out[c] = (T)y;
            if (c == 0 && a.lse) a.lse[row] = lh == 0.f ? -INFINITY : (mh + log2f(lh)) * kLn2;
        };
        for (int i = tid; i < hn * D; i += kDecThreads) {
            const int h = i / D, c = i % D;
            float mh = -INFINITY, lh = 0.f, oh = 0.f;
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) mh = fmaxf(mh, s_m[w][h]);
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) {
                const float f = s_m[w][h] == -INFINITY ? 0.f : exp2_fast(s_m[w][h] - mh);
                lh = fmaf(f, s_l[w][h], lh);
                oh = fmaf(f, reinterpret_cast<const float*>(smem + w * Cfg::WARP_BYTES)[h * D + c], oh);
            }
            if (whole) {
                finish(h, c, mh, lh, oh);
            } else {
                mine[h * D + c] = oh;
                if (c == 0) {
                    mine[kMaxHeads * D + h] = mh;
                    mine[kMaxHeads * D + kMaxHeads + h] = lh;
                }
            }
        }
        if (!whole) {
            // CTAs whose shares hold a part of this (request, heads): unit x is in share ((x + 1) C - 1) / U
            const long long s0 = base + (long long)seg * nb;
            const int c0 = (int)(((s0 + 1) * C - 1) / U), c1 = (int)(((s0 + nb) * C - 1) / U);
            int* counter = reinterpret_cast<int*>(a.ws) + c0;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                s_last = atomicAdd(counter, 1) == c1 - c0;
                if (s_last) *counter = 0;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int i = tid; i < hn * D; i += kDecThreads) {
                    const int h = i / D, c = i % D;
                    float mh = -INFINITY, lh = 0.f, oh = 0.f;
                    for (int x = c0; x <= c1; ++x) {
                        const float* p = piece + (2 * (size_t)x + (x == c0 ? 1 : 0)) * psize;
                        mh = fmaxf(mh, __ldcg(p + kMaxHeads * D + h));
                    }
#pragma unroll 4
                    for (int x = c0; x <= c1; ++x) {
                        const float* p = piece + (2 * (size_t)x + (x == c0 ? 1 : 0)) * psize;
                        const float pm = __ldcg(p + kMaxHeads * D + h);
                        const float f = pm == -INFINITY ? 0.f : exp2_fast(pm - mh);
                        lh = fmaf(f, __ldcg(p + kMaxHeads * D + kMaxHeads + h), lh);
                        oh = fmaf(f, __ldcg(p + h * D + c), oh);
                    }
                    finish(h, c, mh, lh, oh);
                }
            }
        }
        __syncthreads();                                // the buffers and s_m, s_l are written again
        u += blk1 - blk0;
        if (blk1 == nb && seg == segs - 1) {
            base += (long long)nb * segs;
            ++b;
        }
    }
}

template <typename T, int D, int NT>
cudaError_t launch_nt(const PagedArgs& a, cudaStream_t st)
{
    auto k = paged_decode_kernel<T, D, NT>;
    const int smem = DecCfg<D>::SMEM;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // an upper bound of the units: lengths are known on the device only
    long long most = (long long)a.p.max_pages << a.shift;
    if (a.p.window > 0) most = most < (long long)a.p.window + a.p.sinks ? most : (long long)a.p.window + a.p.sinks;
    const long long chunks = (a.grp + 8 * NT - 1) / (8 * NT);
    const long long units = ((most + kBlock - 1) / kBlock + 1) * a.p.B * a.p.Hkv * chunks;
    k<<<(unsigned)(units < kDecCtas ? units : kDecCtas), kDecThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t st)
{
    return a.grp <= 8 ? launch_nt<T, D, 1>(a, st) : launch_nt<T, D, 2>(a, st);
}

}  // namespace

size_t paged_attend_workspace(const fadkv_paged_params& p)
{
    return kCounterBytes + (size_t)2 * kDecCtas * Piece::floats(p.d) * sizeof(float);
}

cudaError_t launch_paged_attend(const PagedArgs& a, cudaStream_t st)
{
    if (a.p.B <= 0) return cudaSuccess;
    if (a.p.dtype == FADKV_F16) return a.p.d == 128 ? launch_t<__half, 128>(a, st) : launch_t<__half, 64>(a, st);
    return a.p.d == 128 ? launch_t<__nv_bfloat16, 128>(a, st) : launch_t<__nv_bfloat16, 64>(a, st);
}

}  // namespace fadkv
