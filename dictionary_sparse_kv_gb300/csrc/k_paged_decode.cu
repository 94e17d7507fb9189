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
// that do not depend on which CTA that was (pieces and groups of pieces are
// the same every time).  Requests of about one length (a
// full window, say) are cut into equal parts instead, one a CTA, where that
// fills the grid: a share that begins in one (request, KV head) and ends in the
// next costs two beginnings and two joins.
//
// Inside a CTA each of four warps takes every fourth 16-token tile through a
// pipeline of its own (cp.async, one block-table lookup per token), with its
// own m, l and o; nothing synchronises the warps until the piece ends, and the
// first tiles of the next piece are asked for before the last one's results
// are joined.  The products run on the warp's matrix instructions with the
// tokens as rows and the query heads that share the KV head as the eight
// columns:
//   S^T = K Q^T   [16 tokens][8 heads],   O^T += V^T P^T   [d][8 heads],
// so a group of up to eight heads fills one instruction and nothing is padded
// to 16 rows of queries.  P enters as two 16-bit terms (hi + lo), 22 bits of
// it in binary16 and 16 in bfloat16: the tensor pipe is idle most of the time
// here, and the rounding of the output is then all that can be seen of it.
// Binary16 ends at 2^-24, and on a long cache many small p add up, so P (at
// most 1) is multiplied by 2^15 for the product and the sums by 2^-15 when the
// warps join: a p is lost below 2^-40, not 2^-25 (131072 keys 12.1 below one
// whose value is 0 came out 0.3% small, 32768 keys 17.5 below it as 0).
//
// 64 requests of 16384 tokens, 32 heads over 8 of 128 in bfloat16: 0.32 ms,
// 6.8 TB/s.  Few or short requests are bound by the chain lengths -> block
// table -> keys and the joins: 7 us for one of 777 tokens.
#include "paged.cuh"

namespace fadkv {
namespace {

using namespace paged;

constexpr int kDecThreads = 128;
constexpr int kDecWarps = kDecThreads / 32;
constexpr int kTile = 16;                          // tokens per warp step
constexpr int kBlock = kTile * kDecWarps;          // tokens per unit of work
// CTAs: two per multiprocessor (152), three at d = 64, whose buffers are half as large (us on the device, against two CTAs
// of six stages at d = 64: 113 requests of 1024 tokens, two KV heads, 12.2 and 12.9; 16 of up to 4096, eight KV heads, 15.8
// and 18.9; 64 of up to 16384 162 and 168; d = 128 with three CTAs of two stages: 16 of 4096 34.8 against 27.7)
__host__ __device__ constexpr int dec_ctas(int d) { return d == 128 ? 304 : 456; }
constexpr int kMaxHeads = 16;                      // query heads per piece; larger groups are several pieces

// What P is multiplied by for the product with V.
template <typename T> constexpr float kUp = std::is_same<T, __half>::value ? 32768.f : 1.f;

template <int D> struct DecCfg {
    static constexpr int STAGES = 3;
    static constexpr int CTAS = dec_ctas(D);
    static constexpr int TILE_BYTES = kTile * D * 2;
    static constexpr int WARP_BYTES = STAGES * 2 * TILE_BYTES;
    // warps' results of eight heads: three quarters each, as the owner of a quarter keeps its own
    static constexpr int JOIN_BYTES = kDecWarps * 3 * (D / 16 / kDecWarps) * 32 * 16;
    static constexpr int SMEM = kDecWarps * WARP_BYTES + JOIN_BYTES;
};

// Pieces that one CTA joins: more are joined in groups, each by the last CTA
// of its group, and the groups by the last group.  (32768 tokens of one KV head
// in 304 pieces: 28.6 us joined by one CTA, 11.6 in groups; 4 requests of up to
// 2000 tokens with 24 heads over 8, some 20 pieces each: 10.9 at once, 12.7 in
// groups.)
constexpr int kAtOnce = 32, kGroup = 16;
constexpr int kCounters = 512;                     // of first groups, of other groups and of the groups of a (request, heads)
static_assert(dec_ctas(64) <= kCounters && dec_ctas(128) <= kCounters, "counters");
static_assert(3 * kCounters * sizeof(int) <= kHeadBytes - kDecodeHead, "workspace head");

// A piece in the workspace: kMaxHeads rows of d sums, then their m and l.
__host__ __device__ constexpr size_t piece_floats(int d) { return (size_t)kMaxHeads * (d + 2); }

// One piece of work: blocks blk0 .. blk1-1 of nb of request b and a set of
// heads that share a KV head.
struct Work {
    int b, hk, head0, hn, nb, blk0, blk1;
    int end, tile0, tiles;     // list indices end at `end`; this warp's tiles
    long long first;           // unit number of block 0 (shares)
    Seen seen;
};

__device__ __forceinline__ int add_acq_rel(int* p, int v)
{
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kDecThreads, dec_ctas(D) / 152)
paged_decode_kernel(const __grid_constant__ PagedArgs a)
{
    using Cfg = DecCfg<D>;
    constexpr int STAGES = Cfg::STAGES, ROW = D * 2, CPR = D / 8;      // bytes and 16-byte chunks per row
    constexpr int KS = D / 16, KQ = KS / kDecWarps;                    // 16-element steps; those a warp writes out
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ int s_b, s_last, s_longest;
    __shared__ long long s_base;
    __shared__ float s_m[kDecWarps][8 * NT], s_l[kDecWarps][8 * NT];
    __shared__ uint32_t s_ok[kDecWarps][STAGES];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = a.grp, B = a.p.B;
    const int chunks = (grp + 8 * NT - 1) / (8 * NT);                 // pieces per KV head
    const int segs = a.p.Hkv * chunks;
    const uint32_t wbase = saddr(smem + warp * Cfg::WARP_BYTES);
    float4* joinbuf = reinterpret_cast<float4*>(smem + kDecWarps * Cfg::WARP_BYTES);
    pdl_begin();

    // blocks of a request: at least one, so that one which sees nothing is written too
    auto blocks_of = [&](const Seen& s) { return max(1, (s.count + kBlock - 1) / kBlock); };
    auto blocks = [&](int b) { return blocks_of(seen_of(length_of(b, b, a), a)); };
    long long u, u1, U, base;                                          // this CTA's units; all; the first of request cur_b
    int C, cur_b, longest, parts = 0;                                  // parts > 0: (request, heads) in so many equal parts
    // Equal parts: the lengths are within an eighth of the longest one on average, and the parts are at least three
    // fifths of the grid.  Measured over 1 to 152 requests of 500 to 20000 tokens, us on the device in equal parts and in
    // shares: of one length 113 requests of 1024 tokens with two KV heads of 64 12.0 and 14.0, 4 of 4096 with eight of 128
    // 12.5 and 14.3, 64 of 3000 with four of 128 59.5 and 64.2, 152 of 20000 with one of 128 227 and 227.  With a mean of
    // 7/8 of the longest 11.6 and 13.6, 12.3 and 14.0, 55.6 and 55.8, 197 and 197; of 3/4, where shares are taken, 11.5
    // and 13.0, 12.3 and 13.2, 49.5 and 48.5, 178 and 166.  Below three fifths of the grid (60 requests of 1100 with four KV
    // heads of 64, 240 parts on 456 places): 16.6 and 14.7.
    auto share = [&] {
        const int pieces = B * segs, grid = (int)gridDim.x;
        C = (int)min((long long)grid, U);
        if (pieces <= grid && 8 * U >= 7ll * pieces * longest) {
            parts = min(longest, grid / pieces);
            if (5 * pieces * parts >= 3 * C) C = pieces * parts;
            else parts = 0;
        }
        if (U < (1 << 22)) {                                          // C <= 456: the products fit 32 bits
            u = (int)U * (int)blockIdx.x / C;
            u1 = (int)U * (int)(blockIdx.x + 1) / C;
        } else {
            u = U * blockIdx.x / C;
            u1 = U * (blockIdx.x + 1) / C;
        }
    };
    if (B <= 32) {                                                    // a lane a request, each warp for itself
        const int nb = lane < B ? blocks(lane) : 0;
        const long long mine = (long long)nb * segs;
        long long upto = mine;
        longest = __reduce_max_sync(0xffffffffu, nb);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        U = __shfl_sync(0xffffffffu, upto, 31);
        share();
        if ((int)blockIdx.x >= C) return;
        if (parts == 0) {
            cur_b = __ffs(__ballot_sync(0xffffffffu, upto > u)) - 1;
            base = __shfl_sync(0xffffffffu, upto - mine, cur_b);
        }
    } else {
        const int each = (B + kDecThreads - 1) / kDecThreads, b0 = min(B, tid * each), b1 = min(B, b0 + each);
        long long mine = 0;
        int most = 0;
        if (tid == 0) s_longest = 0;
        for (int b = b0; b < b1; ++b) {
            const int nb = blocks(b);
            mine += (long long)nb * segs;
            most = max(most, nb);
        }
        long long at = block_scan<kDecThreads>(mine, &U);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) atomicMax(&s_longest, most);
        __syncthreads();
        longest = s_longest;
        share();
        if ((int)blockIdx.x >= C) return;
        if (parts == 0 && u >= at && u < at + mine) {
            int b = b0;
            for (long long n; u >= at + (n = (long long)blocks(b) * segs); ++b) at += n;
            s_b = b;
            s_base = at;
        }
        __syncthreads();
        cur_b = s_b;
        base = s_base;
    }

    // the piece that begins at unit u (u < u1); u, cur_b and base move past it
    auto next_work = [&] {
        Work w;
        w.b = cur_b;
        w.seen = seen_of(length_of(cur_b, cur_b, a), a);
        w.nb = blocks_of(w.seen);
        int seg;
        if (parts > 0) {
            seg = (int)blockIdx.x / parts % segs;
            const int n = min(parts, w.nb), part = (int)blockIdx.x % parts;   // a short request has fewer parts
            const int each = w.nb / n, rest = w.nb % n;                      // the first `rest` parts take one block more
            w.blk0 = part * each + min(part, rest);
            w.blk1 = part < n ? w.blk0 + each + (part < rest) : w.blk0;
            u = u1;
        } else {
            const long long rel = u - base;
            seg = rel < 0x7fffffffll ? (int)rel / w.nb : (int)(rel / w.nb);
            w.first = base + (long long)seg * w.nb;
            w.blk0 = (int)(u - w.first);
            w.blk1 = (int)min((long long)w.nb, w.blk0 + (u1 - u));
            u += w.blk1 - w.blk0;
            if (w.blk1 == w.nb && seg == segs - 1) {
                base += (long long)w.nb * segs;
                ++cur_b;
            }
        }
        w.hk = chunks == 1 ? seg : seg / chunks;
        const int h0 = chunks == 1 ? 0 : (seg % chunks) * 8 * NT;
        w.hn = min(8 * NT, grp - h0);
        w.head0 = w.hk * grp + h0;
        w.end = min(w.blk1 * kBlock, w.seen.count);
        w.tile0 = w.blk0 * kDecWarps + warp;
        w.tiles = max(0, ((w.end + kTile - 1) / kTile - w.tile0 + kDecWarps - 1) / kDecWarps);
        return w;
    };

    // lane (and lane + 16): token lane % 16 of the piece's tile t, its page one step ahead of its load
    int tok = -1, page = -1;
    auto look_up = [&](const Work& w, int t) {
        const int i = (w.tile0 + t * kDecWarps) * kTile + (lane & 15);
        tok = i < w.end ? (i < w.seen.first ? i : i - w.seen.first + w.seen.from) : -1;
        page = tok >= 0 ? __ldg(a.table + (size_t)w.b * a.p.max_pages + (tok >> a.shift)) : -1;
    };
    auto load = [&](const Work& w, int t) {
        const int s = t % STAGES;
        const T* kp = (const T*)a.k + w.hk * a.p.head_stride;
        const T* vp = (const T*)a.v + w.hk * a.p.head_stride;
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
    auto begin = [&](const Work& w) {                                   // the first tiles, STAGES - 1 copy groups
        if (w.tiles > 0) look_up(w, 0);
        for (int t = 0; t < STAGES - 1; ++t) {
            if (t < w.tiles) {
                load(w, t);
                look_up(w, t + 1);
            }
            cp_commit();
        }
    };
    // queries as the B operand: lane holds head lane/4, elements 2 (lane % 4) + {0, 1} of each half step
    uint32_t qf[NT][KS][2];
    auto load_q = [&](const Work& w) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int h = n * 8 + (lane >> 2);
            const uint32_t* q = reinterpret_cast<const uint32_t*>((const T*)a.q + (size_t)w.b * a.p.q_stride +
                                                                  (size_t)(w.head0 + (h < w.hn ? h : 0)) * D) + (lane & 3);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[n][k][0] = h < w.hn ? __ldg(q + k * 8) : 0u;
                qf[n][k][1] = h < w.hn ? __ldg(q + k * 8 + 4) : 0u;
            }
        }
    };

    if (parts > 0) cur_b = (int)blockIdx.x / parts / segs;
    Work w = next_work();
    if (w.blk0 == w.blk1) return;                                       // a part that a short request does not have
    begin(w);
    load_q(w);
    for (;;) {
        float o[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }
        for (int t = 0; t < w.tiles; ++t) {
            cp_wait<STAGES - 2>();
            __syncwarp();
            if (t + STAGES - 1 < w.tiles) {
                load(w, t + STAGES - 1);
                look_up(w, t + STAGES);
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
                const float e0 = p0 * kUp<T>, e1 = p1 * kUp<T>, e2 = p2 * kUp<T>, e3 = p3 * kUp<T>;
                const uint32_t a0 = Num<T>::pack(e0, e1), a1 = Num<T>::pack(e2, e3);
                const float2 r0 = Num<T>::unpack(a0), r1 = Num<T>::unpack(a1);
                ph[n][0] = transpose8(a0);
                ph[n][1] = transpose8(a1);
                pl[n][0] = transpose8(Num<T>::pack(e0 - r0.x, e1 - r0.y));
                pl[n][1] = transpose8(Num<T>::pack(e2 - r1.x, e3 - r1.y));
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
        __syncwarp();
        const Work done = w;
        const bool more = u < u1;
        if (more) {                                                     // every buffer of this warp is free
            w = next_work();
            begin(w);
            load_q(w);
        }

        // this piece's results: the warps' m and l, then quarter by quarter of d, each by one warp.  o[n][k] holds heads
        // n 8 + 2 (lane % 4) + {0, 1} of elements k 16 + lane / 4 + {0, 8}, the same in every warp.
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v = l[n][i];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (lane < 4) {
                    s_m[warp][n * 8 + 2 * lane + i] = m[n][i];
                    s_l[warp][n * 8 + 2 * lane + i] = v;
                }
            }
        const bool whole = done.blk0 == 0 && done.blk1 == done.nb;
        float* pieces = reinterpret_cast<float*>((unsigned char*)a.ws + kHeadBytes);
        constexpr size_t PF = piece_floats(D);
        float* mine = pieces + (2 * (size_t)blockIdx.x + (done.blk0 == 0 ? 1 : 0)) * PF;
        auto lse_of = [&](float mh, float lh) { return lh == 0.f ? -INFINITY : (mh + log2f(lh)) * kLn2; };
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            // slot of warp x's quarter y (y != x): [x][y or y - 1][step][lane]
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int y = k / KQ;
                if (y != warp)
                    joinbuf[((warp * 3 + (y < warp ? y : y - 1)) * KQ + k % KQ) * 32 + lane] =
                        make_float4(o[n][k][0], o[n][k][1], o[n][k][2], o[n][k][3]);
            }
            __syncthreads();
            float f[kDecWarps][2], mh[2], lh[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int h = n * 8 + 2 * (lane & 3) + i;
                mh[i] = -INFINITY;
                lh[i] = 0.f;
#pragma unroll
                for (int x = 0; x < kDecWarps; ++x) mh[i] = fmaxf(mh[i], s_m[x][h]);
#pragma unroll
                for (int x = 0; x < kDecWarps; ++x) {
                    f[x][i] = s_m[x][h] == -INFINITY ? 0.f : exp2_fast(s_m[x][h] - mh[i]);
                    lh[i] = fmaf(f[x][i], s_l[x][h], lh[i]);
                    f[x][i] *= 1.f / kUp<T>;               // of the sums of p v
                }
            }
#pragma unroll
            for (int k = 0; k < KQ; ++k) {
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int x = 0; x < kDecWarps; ++x) {
                    float4 v;
                    if (x == warp) {
                        // o[n][warp KQ + k], with constant indexes
                        v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int y = 0; y < kDecWarps; ++y)
                            if (y == warp) v = make_float4(o[n][y * KQ + k][0], o[n][y * KQ + k][1], o[n][y * KQ + k][2], o[n][y * KQ + k][3]);
                    } else {
                        v = joinbuf[((x * 3 + (warp < x ? warp : warp - 1)) * KQ + k) * 32 + lane];
                    }
                    acc.x = fmaf(f[x][0], v.x, acc.x);
                    acc.y = fmaf(f[x][1], v.y, acc.y);
                    acc.z = fmaf(f[x][0], v.z, acc.z);
                    acc.w = fmaf(f[x][1], v.w, acc.w);
                }
                const int c = (warp * KQ + k) * 16 + (lane >> 2);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int h = n * 8 + 2 * (lane & 3) + i;
                    const float y0 = i ? acc.y : acc.x, y1 = i ? acc.w : acc.z;
                    if (h >= done.hn) continue;
                    if (whole) {
                        T* out = (T*)a.out + (size_t)done.b * a.p.out_stride + (size_t)(done.head0 + h) * D + c;
                        const float inv = lh[i] > 0.f ? 1.f / lh[i] : (lh[i] == lh[i] ? 0.f : lh[i]);
                        out[0] = (T)(y0 * inv);
                        out[8] = (T)(y1 * inv);
                        if (k == 0 && warp == 0 && lane < 4 && a.lse)
                            a.lse[(size_t)done.b * a.p.Hq + done.head0 + h] = lse_of(mh[i], lh[i]);
                    } else {
                        mine[h * D + c] = y0;
                        mine[h * D + c + 8] = y1;
                        if (k == 0 && warp == 0 && lane < 4) {
                            mine[kMaxHeads * D + h] = mh[i];
                            mine[kMaxHeads * (D + 1) + h] = lh[i];
                        }
                    }
                }
            }
            __syncthreads();                            // the buffer, and s_m and s_l, are written again
        }
        if (!whole) {
            // the CTAs that have its parts; of shares, unit x is in share ((x + 1) C - 1) / U
            int c0, c1;
            if (parts > 0) {
                c0 = (int)blockIdx.x / parts * parts;
                c1 = c0 + min(parts, done.nb) - 1;
            } else if (U < (1 << 22)) {
                c0 = (int)(((unsigned int)done.first + 1) * (unsigned int)C - 1) / (int)U;
                c1 = (int)(((unsigned int)done.first + done.nb) * (unsigned int)C - 1) / (int)U;
            } else {
                c0 = (int)(((done.first + 1) * C - 1) / U);
                c1 = (int)(((done.first + done.nb) * C - 1) / U);
            }
            // whether this CTA is the last of n at a counter; the counter is back at zero then
            auto last_at = [&](int index, int n) {
                __syncthreads();
                if (tid == 0) {
                    int* counter = reinterpret_cast<int*>((unsigned char*)a.ws + kDecodeHead) + index;
                    s_last = add_acq_rel(counter, 1) == n - 1;   // the block's stores before it, the other blocks' after it
                    if (s_last) *counter = 0;
                }
                __syncthreads();
                return s_last != 0;
            };
            auto piece = [&](int x) { return pieces + (2 * (size_t)x + (x == c0 ? 1 : 0)) * PF; };
            // joins pieces x0, x0 + step, ... (n of them) in their order, so that it does not matter who does it: four columns
            // a thread, all rows at once; into the first one, or as the result
            auto join = [&](int x0, int n, int step, bool result) {
                constexpr int TPR = D / 4;              // threads per row, all of one warp
                for (int h = tid / TPR; h < done.hn; h += kDecThreads / TPR) {
                    const int c = tid % TPR * 4;
                    float mh = -INFINITY, lh = 0.f;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                    // eight pieces at a time, all their loads in flight; past the last one the last one again, with weight 0
#pragma unroll 1
                    for (int i0 = 0; i0 < n; i0 += 8) {
                        float pm[8], ll[8];
                        float4 v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float* q = piece(x0 + min(i0 + j, n - 1) * step);
                            pm[j] = __ldcg(q + kMaxHeads * D + h);
                            ll[j] = __ldcg(q + kMaxHeads * (D + 1) + h);
                            v[j] = __ldcg(reinterpret_cast<const float4*>(q + h * D + c));
                        }
                        float top = mh;
#pragma unroll
                        for (int j = 0; j < 8; ++j) top = fmaxf(top, pm[j]);
                        const float g = mh == -INFINITY ? 0.f : exp2_fast(mh - top);
                        mh = top;
                        lh *= g;
                        y.x *= g, y.y *= g, y.z *= g, y.w *= g;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float f = pm[j] == -INFINITY || i0 + j >= n ? 0.f : exp2_fast(pm[j] - mh);
                            lh = fmaf(f, ll[j], lh);
                            y.x = fmaf(f, v[j].x, y.x);
                            y.y = fmaf(f, v[j].y, y.y);
                            y.z = fmaf(f, v[j].z, y.z);
                            y.w = fmaf(f, v[j].w, y.w);
                        }
                    }
                    if (result) {
                        const float inv = lh > 0.f ? 1.f / lh : (lh == lh ? 0.f : lh);
                        T* out = (T*)a.out + (size_t)done.b * a.p.out_stride + (size_t)(done.head0 + h) * D + c;
                        *reinterpret_cast<uint2*>(out) = make_uint2(Num<T>::pack(y.x * inv, y.y * inv), Num<T>::pack(y.z * inv, y.w * inv));
                        if (c == 0 && a.lse) a.lse[(size_t)done.b * a.p.Hq + done.head0 + h] = lse_of(mh, lh);
                    } else {
                        float* q = piece(x0);
                        __syncwarp(__activemask());     // every thread of the row has read its m and l
                        *reinterpret_cast<float4*>(q + h * D + c) = y;
                        if (c == 0) {
                            q[kMaxHeads * D + h] = mh;
                            q[kMaxHeads * (D + 1) + h] = lh;
                        }
                    }
                }
            };
            // (a CTA that begins one (request, heads) may also be within another: their counters lie apart)
            const int n = c1 - c0 + 1, size = n <= kAtOnce ? kAtOnce : kGroup;
            const int groups = (n + size - 1) / size, group = ((int)blockIdx.x - c0) / size;
            int x0 = c0 + group * size, count = min(size, n - group * size), step = 1;
            int index = group == 0 ? c0 : kCounters + x0;
            bool result = groups == 1;
#pragma unroll 1
            while (last_at(index, count)) {
                join(x0, count, step, result);
                if (result) break;
                result = true;
                index = 2 * kCounters + c0;
                x0 = c0;
                count = groups;
                step = size;
            }
            __syncthreads();                            // s_last is written again
        }
        if (!more) break;
    }
}

template <typename T, int D, int NT>
cudaError_t launch_nt(const PagedArgs& a, cudaStream_t st)
{
    auto k = paged_decode_kernel<T, D, NT>;
    const int smem = DecCfg<D>::SMEM, ctas = DecCfg<D>::CTAS;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // an upper bound of the units: lengths are known on the device only
    long long most = (long long)a.p.max_pages << a.shift;
    if (a.p.window > 0) most = most < (long long)a.p.window + a.p.sinks ? most : (long long)a.p.window + a.p.sinks;
    const long long chunks = (a.grp + 8 * NT - 1) / (8 * NT);
    const long long units = ((most + kBlock - 1) / kBlock + 1) * a.p.B * a.p.Hkv * chunks;
    return launch_pdl(k, dim3((unsigned)(units < ctas ? units : ctas)), dim3(kDecThreads), smem, st, a);
}

template <typename T, int D>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t st)
{
    return a.grp <= 8 ? launch_nt<T, D, 1>(a, st) : launch_nt<T, D, 2>(a, st);
}

}  // namespace

size_t paged_attend_workspace(const fadkv_paged_params& p)
{
    return kHeadBytes + (size_t)2 * dec_ctas(p.d) * piece_floats(p.d) * sizeof(float);
}

cudaError_t launch_paged_attend(const PagedArgs& a, cudaStream_t st)
{
    if (a.p.B <= 0) return cudaSuccess;
    if (a.p.dtype == FADKV_F16) return a.p.d == 128 ? launch_t<__half, 128>(a, st) : launch_t<__half, 64>(a, st);
    return a.p.d == 128 ? launch_t<__nv_bfloat16, 128>(a, st) : launch_t<__nv_bfloat16, 64>(a, st);
}

}  // namespace fadkv
