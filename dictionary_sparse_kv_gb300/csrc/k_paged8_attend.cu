// Attention of one new token per request over the 8-bit pages.
//
//   x_j = scale log2(e) sk_j <q, ck_j>,  p_j = 2^(x_j - m),  l = sum p_j,
//   o = sum w_j cv_j,  w_j = 2^(x_j + log2 sv_j - M),  out = o 2^(M - m) / l,
// ck, cv the codes and sk, sv the scales of their blocks, in one pass over the
// codes.  m and M are running references of x and of x + log2 sv, each near its
// own maximum, so that a block of large values that is hardly seen does not
// push the others' weights out of binary16's range.  They move only when
// something has grown by more than 2^4 past them (o / l is the same), so most
// tiles need one vote and no maximum.  Results of disjoint key sets join as
//   m = max m_i,  l = sum 2^(m_i - m) l_i,  out = sum 2^(m_i - m) l_i out_i / l.
//
// The codes that are seen have to be read once: HBM, at half the bytes of the
// 16-bit pages, so the instructions per token count twice as much.  Both
// formats' codes are exact in binary16, which the products run in whatever the
// type of q: 8-bit bytes come out of shared memory by the 16-bit matrix loads,
// four codes a lane, in an order of elements that q's fragments follow (keys)
// or that the rows of the sums follow (values), so that two conversions and, for
// the values, one byte permutation give two registers of a fragment.  Scales
// enter behind the products, one of each kind for a 16-token tile, which lies in
// one block.
//
// The work is cut as in the 16-bit kernel: one list of 64-token blocks, request
// by request and KV head by KV head, an even share a CTA, or equal parts where
// the lengths are about even; pieces go to the workspace and the CTA that
// arrives last joins them in their order.  Blocks lie at multiples of 64 tokens
// (a window's first one is partly seen), so that a tile is one page, one block
// of scales and one run of bytes.
#include "paged8.cuh"

namespace fadkv {
namespace {

using namespace paged;
using namespace paged8;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;                          // tokens per warp step
constexpr int kBlock = kTile * kWarps;             // tokens per unit of work
constexpr int kMaxHeads = 16;                      // query heads per piece; larger groups are several pieces
constexpr float kGrow = 4.f;                       // growth (log2) that moves m and M
constexpr float kUp = 2048.f;                      // 2^(15 - kGrow): what w is multiplied by for the product
constexpr int kSms = 152;

template <int D> struct Cfg {
    static constexpr int PER_SM = D == 128 ? 3 : 4;
    static constexpr int STAGES = D == 128 ? 3 : 4;
    static constexpr int CTAS = PER_SM * kSms;
    static constexpr int TILE_BYTES = kTile * D;
    static constexpr int WARP_BYTES = STAGES * 2 * TILE_BYTES;
    static constexpr int JOIN_BYTES = kWarps * 3 * (D / 16 / kWarps) * 32 * 16;
    static constexpr int SMEM = kWarps * WARP_BYTES + JOIN_BYTES;
};

// Pieces that one CTA joins: more are joined in groups, as in the 16-bit kernel.
constexpr int kAtOnce = 32, kGroup = 16;
constexpr int kCounters = 1024;
static_assert(Cfg<64>::CTAS <= kCounters && Cfg<128>::CTAS <= kCounters, "counters");
static_assert(3 * kCounters * sizeof(int) <= kHeadBytes - kDecodeHead, "workspace head");

// A piece in the workspace: kMaxHeads rows of d results, then their m and l.
__host__ __device__ constexpr size_t piece_floats(int d) { return (size_t)kMaxHeads * (d + 2); }

// Byte offset of 16-byte chunk c of row r: eight rows at one chunk lie in
// eight different bank groups.
template <int D>
__device__ __forceinline__ uint32_t swz8(int r, int c)
{
    return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void cp4(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ int add_acq_rel(int* p, int v)
{
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// Bits 0 .. n-1 set (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// The tokens that the query at position len - 1 sees, the first `first` ones
// and those from `from` on, as a list of 64-token blocks: `sinks` ones from
// token 0 on, then those from block `from_block` on; `count` in all.
struct Blocks {
    int len, first, from, sinks, from_block, count;
    __device__ __forceinline__ int token(int i) const { return (i < sinks ? i : i - sinks + from_block) * kBlock; }
    __device__ __forceinline__ uint32_t seen(int token) const         // of the 16 from `token` on
    {
        return low_bits(min(len - token, kTile)) & (~low_bits(from - token) | low_bits(first - token));
    }
};

struct Work {
    int b, hk, head0, hn, nb, blk0, blk1;
    long long unit0;           // unit number of block 0 (shares)
    Blocks seen;
};

template <typename T, int D, int NT, int FORMAT>
__global__ void __launch_bounds__(kThreads, Cfg<D>::PER_SM)
paged8_attend_kernel(const __grid_constant__ Paged8Args a)
{
    using C_ = Cfg<D>;
    constexpr int STAGES = C_::STAGES, CPR = D / 16;                   // 16-byte chunks per row
    constexpr int KS = D / 16, KQ = KS / kWarps;                       // 16-element steps; those a warp writes out
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ int s_b, s_last, s_longest;
    __shared__ long long s_base;
    __shared__ float s_m[kWarps][8 * NT], s_l[kWarps][8 * NT];
    __shared__ uint32_t s_ok[kWarps][STAGES];
    __shared__ float s_scale[kWarps][STAGES][2];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = a.grp, B = a.p.B;
    const int chunks = (grp + 8 * NT - 1) / (8 * NT);                 // pieces per KV head
    const int segs = a.p.Hkv * chunks;
    const uint32_t wbase = saddr(smem + warp * C_::WARP_BYTES);
    float4* joinbuf = reinterpret_cast<float4*>(smem + kWarps * C_::WARP_BYTES);
    pdl_begin();

    auto blocks_of = [&](int b) {
        Blocks s;
        const int pos = a.positions ? __ldg(a.positions + b) : 0, len = __ldg(a.lengths + b);
        s.len = pos < 0 ? 0 : min(max(len, 0), a.p.max_pages << a.shift);
        s.from = a.p.window > 0 && s.len > a.p.window ? s.len - a.p.window : 0;
        s.first = min(a.p.sinks, s.from);
        s.from_block = s.from / kBlock;
        s.sinks = min((s.first + kBlock - 1) / kBlock, s.from_block);
        s.count = s.sinks + (s.len + kBlock - 1) / kBlock - s.from_block;
        return s;
    };
    // at least one, so that a request which sees nothing is written too
    auto units_of = [&](int b) { return max(1, blocks_of(b).count); };
    long long u, u1, U, base;                                          // this CTA's units; all; the first of request cur_b
    int C, cur_b = 0, longest, parts = 0;                              // parts > 0: (request, heads) in so many equal parts
    auto share = [&] {
        const int pieces = B * segs, grid = (int)gridDim.x;
        C = (int)min((long long)grid, U);
        if (pieces <= grid && 8 * U >= 7ll * pieces * longest) {
            parts = min(longest, grid / pieces);
            if (5 * pieces * parts >= 3 * C) C = pieces * parts;
            else parts = 0;
        }
        if (U < (1 << 21)) {                                          // C <= 1024: the products fit 32 bits
            u = (int)U * (int)blockIdx.x / C;
            u1 = (int)U * (int)(blockIdx.x + 1) / C;
        } else {
            u = U * blockIdx.x / C;
            u1 = U * (blockIdx.x + 1) / C;
        }
    };
    if (B <= 32) {                                                    // a lane a request, each warp for itself
        const int nb = lane < B ? units_of(lane) : 0;
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
        const int each = (B + kThreads - 1) / kThreads, b0 = min(B, tid * each), b1 = min(B, b0 + each);
        long long mine = 0;
        int most = 0;
        if (tid == 0) s_longest = 0;
        for (int b = b0; b < b1; ++b) {
            const int nb = units_of(b);
            mine += (long long)nb * segs;
            most = max(most, nb);
        }
        long long at = block_scan<kThreads>(mine, &U);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) atomicMax(&s_longest, most);
        __syncthreads();
        longest = s_longest;
        share();
        if ((int)blockIdx.x >= C) return;
        if (parts == 0 && u >= at && u < at + mine) {
            int b = b0;
            for (long long n; u >= at + (n = (long long)units_of(b) * segs); ++b) at += n;
            s_b = b;
            s_base = at;
        }
        __syncthreads();
        if (parts == 0) {
            cur_b = s_b;
            base = s_base;
        }
    }
    if (parts > 0) cur_b = (int)blockIdx.x / parts / segs;

    // the piece that begins at unit u (u < u1); u, cur_b and base move past it
    auto next_work = [&] {
        Work w;
        w.b = cur_b;
        w.seen = blocks_of(cur_b);
        w.nb = max(1, w.seen.count);
        w.unit0 = 0;
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
            w.unit0 = base + (long long)seg * w.nb;
            w.blk0 = (int)(u - w.unit0);
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
        return w;
    };

    // this warp's 16 tokens of the piece's tile t (block blk0 + t): their page one step ahead of their load
    int tok = 0, page = -1;
    auto look_up = [&](const Work& w, int t) {
        page = -1;
        if (w.blk0 + t >= w.blk1) return;
        tok = w.seen.token(w.blk0 + t) + warp * kTile;
        if (w.seen.seen(tok)) page = __ldg(a.table + (size_t)w.b * a.p.max_pages + (tok >> a.shift));
    };
    const int row0 = lane / CPR, chunk = lane % CPR;                   // this lane's pieces of a tile: rows row0 + j 32 / CPR
    const long long lane_off = row0 * a.p.token_stride + chunk * 16, step_off = (32 / CPR) * a.p.token_stride;
    auto load = [&](const Work& w, int t) {
        const int s = t % STAGES;
        const bool ok = page >= 0 && page < a.p.num_pages;
        const uint32_t bits = ok ? w.seen.seen(tok) : 0u;
        const int at = tok & ((1 << a.shift) - 1);
        const long long off = ok ? page * a.p.page_stride + w.hk * a.p.head_stride + at * a.p.token_stride + lane_off : 0;
        const uint32_t dst = wbase + s * 2 * C_::TILE_BYTES;
#pragma unroll
        for (int j = 0; j < kTile * CPR / 32; ++j) {
            const int r = row0 + j * (32 / CPR);
            const bool v = (bits >> r) & 1u;
            cp16(dst + swz8<D>(r, chunk), a.k + off + j * step_off, v);
            cp16(dst + C_::TILE_BYTES + swz8<D>(r, chunk), a.v + off + j * step_off, v);
        }
        if (lane < 2) {
            if (lane == 0) s_ok[warp][s] = bits;
            if (ok) cp4(saddr(&s_scale[warp][s][lane]), (lane ? a.v_scales : a.k_scales) + scale_at(page, w.hk, at, a.p.Hkv, a.shift, a.bshift));
            else s_scale[warp][s][lane] = 1.f;
        }
    };
    auto begin = [&](const Work& w) {                                   // the first tiles, STAGES - 1 copy groups
        look_up(w, 0);
        for (int t = 0; t < STAGES - 1; ++t) {
            if (w.blk0 + t < w.blk1) {
                load(w, t);
                look_up(w, t + 1);
            }
            cp_commit();
        }
    };
    // Queries as the B operand: lane holds head lane / 4; of step k its elements 16 k + 4 (lane % 4) + {0, 1, 2, 3}, the
    // order in which the lanes have a row's bytes.  qs: what the scores of heads 2 (lane % 4) + {0, 1} are multiplied by.
    uint32_t qf[NT][KS][2];
    float qs[NT][2];
    auto load_q = [&](const Work& w) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int h = n * 8 + (lane >> 2);
            const uint2* q = reinterpret_cast<const uint2*>((const T*)a.q + (size_t)w.b * a.p.q_stride + (size_t)(w.head0 + (h < w.hn ? h : 0)) * D) + (lane & 3);
            float mine = a.scale_log2;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint2 r = h < w.hn ? __ldg(q + k * 4) : make_uint2(0u, 0u);
                qf[n][k][0] = r.x;
                qf[n][k][1] = r.y;
            }
            if (std::is_same<T, __nv_bfloat16>::value) {
                // as binary16 values, the head's largest between 2^14 and 2^15
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < KS; ++k) top = __vmaxu2(top, __vmaxu2(qf[n][k][0] & 0x7fff7fffu, qf[n][k][1] & 0x7fff7fffu));
                top = max(top & 0xffffu, top >> 16);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const uint32_t e = min(max(top >> 7, 15u), 254u);
                const float f = __uint_as_float((268u - e) << 23);
                mine *= __uint_as_float((e - 14u) << 23);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 y = Num<__nv_bfloat16>::unpack(qf[n][k][i]);
                        qf[n][k][i] = Num<__half>::pack(y.x * f, y.y * f);
                    }
            }
            qs[n][0] = __shfl_sync(0xffffffffu, mine, (lane & 3) * 8);
            qs[n][1] = __shfl_sync(0xffffffffu, mine, (lane & 3) * 8 + 4);
        }
    };

    Work w = next_work();
    if (w.blk0 == w.blk1) return;                                       // a part that a short request does not have
    begin(w);
    load_q(w);
    for (;;) {
        float o[NT][KS][4], m[NT][2], M[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = M[n][0] = M[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }
        const int tiles = w.blk1 - w.blk0;
        for (int t = 0; t < tiles; ++t) {
            cp_wait<STAGES - 2>();
            __syncwarp();
            if (t + STAGES - 1 < tiles) {
                load(w, t + STAGES - 1);
                look_up(w, t + STAGES);
            }
            cp_commit();
            const int s = t % STAGES;
            const uint32_t kt = wbase + s * 2 * C_::TILE_BYTES, vt = kt + C_::TILE_BYTES;
            const uint32_t oks = s_ok[warp][s];
            if (oks == 0u) continue;
            const float ks = s_scale[warp][s][0], ls = __log2f(s_scale[warp][s][1]);

            float sc[NT][4], sc2[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[n][i] = sc2[n][i] = 0.f;
            {
                const int r = (lane & 7) + ((lane >> 3) & 1) * 8, c = lane >> 4;
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    uint32_t b[4];
                    ldsm_x4(b, kt + swz8<D>(r, k + c));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t f[4];
                        Code<FORMAT>::halves(b[2 * i], f[0], f[2]);
                        Code<FORMAT>::halves(b[2 * i + 1], f[1], f[3]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) Num<__half>::mma(i ? sc2[n] : sc[n], f, qf[n][k + i][0], qf[n][k + i][1]);
                    }
                }
            }
            bool grew = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[n][i] = (sc[n][i] + sc2[n][i]) * (ks * qs[n][i & 1]);
                if (oks != 0xffffu) {
                    const bool ok0 = (oks >> (lane >> 2)) & 1u, ok1 = (oks >> ((lane >> 2) + 8)) & 1u;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!(i < 2 ? ok0 : ok1)) sc[n][i] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float v = fmaxf(sc[n][i], sc[n][i + 2]);
                    grew |= v > m[n][i] + kGrow || v + ls > M[n][i] + kGrow;
                }
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float f[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float v = fmaxf(sc[n][i], sc[n][i + 2]);
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        if (v > m[n][i]) {
                            l[n][i] *= exp2_fast(m[n][i] - v);
                            m[n][i] = v;
                        }
                        f[i] = 1.f;
                        if (v + ls > M[n][i]) {
                            f[i] = exp2_fast(M[n][i] - (v + ls));
                            M[n][i] = v + ls;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        o[n][k][0] *= f[0];
                        o[n][k][1] *= f[1];
                        o[n][k][2] *= f[0];
                        o[n][k][3] *= f[1];
                    }
                }
            }
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // a head that has seen nothing yet: every score is -inf and every p is 0
                    const float mi = m[n][i & 1] == -INFINITY ? 0.f : m[n][i & 1], Mi = M[n][i & 1] == -INFINITY ? 0.f : M[n][i & 1];
                    l[n][i & 1] += exp2_fast(sc[n][i] - mi);
                    e[i] = exp2_fast(sc[n][i] + ls - Mi) * kUp;
                }
                const uint32_t a0 = Num<__half>::pack(e[0], e[1]), a1 = Num<__half>::pack(e[2], e[3]);
                const float2 r0 = Num<__half>::unpack(a0), r1 = Num<__half>::unpack(a1);
                ph[n][0] = transpose8(a0);
                ph[n][1] = transpose8(a1);
                pl[n][0] = transpose8(Num<__half>::pack(e[0] - r0.x, e[1] - r0.y));
                pl[n][1] = transpose8(Num<__half>::pack(e[2] - r1.x, e[3] - r1.y));
            }
            {
                const int r = (lane & 7) + ((lane >> 3) & 1) * 8, c = lane >> 4;
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    uint32_t b[4];
                    ldsm_x4_trans(b, vt + swz8<D>(r, k + c));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t f[4];
                        Code<FORMAT>::crossed(b[2 * i], f[0], f[1]);
                        Code<FORMAT>::crossed(b[2 * i + 1], f[2], f[3]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            Num<__half>::mma(o[n][k + i], f, ph[n][0], ph[n][1]);
                            Num<__half>::mma(o[n][k + i], f, pl[n][0], pl[n][1]);
                        }
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

        // this piece's results: each warp's divided by its l, and joined quarter by quarter of d, each by one warp.
        // o[n][k] holds heads n 8 + 2 (lane % 4) + {0, 1} of elements k 16 + 2 (lane / 4) (first two) and the one after it.
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[2];
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
                // (v is 0 where nothing was seen, and M - m not a number)
                f[i] = v == 0.f ? 0.f : (M[n][i] == -INFINITY ? 0.f : exp2_fast(M[n][i] - m[n][i])) / (v * kUp);
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                o[n][k][0] *= f[0];
                o[n][k][1] *= f[1];
                o[n][k][2] *= f[0];
                o[n][k][3] *= f[1];
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
            float f[kWarps][2], mh[2], lh[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int h = n * 8 + 2 * (lane & 3) + i;
                mh[i] = -INFINITY;
                lh[i] = 0.f;
#pragma unroll
                for (int x = 0; x < kWarps; ++x) mh[i] = fmaxf(mh[i], s_m[x][h]);
                const float top = mh[i] == -INFINITY ? 0.f : mh[i];
#pragma unroll
                for (int x = 0; x < kWarps; ++x) {
                    f[x][i] = exp2_fast(s_m[x][h] - top) * s_l[x][h];
                    lh[i] += f[x][i];
                }
                const float inv = lh[i] == 0.f ? 0.f : 1.f / lh[i];
#pragma unroll
                for (int x = 0; x < kWarps; ++x) f[x][i] *= inv;
            }
#pragma unroll
            for (int k = 0; k < KQ; ++k) {
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int x = 0; x < kWarps; ++x) {
                    float4 v;
                    if (x == warp) {
                        // o[n][warp KQ + k], with constant indexes
                        v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int y = 0; y < kWarps; ++y)
                            if (y == warp) v = make_float4(o[n][y * KQ + k][0], o[n][y * KQ + k][1], o[n][y * KQ + k][2], o[n][y * KQ + k][3]);
                    } else {
                        v = joinbuf[((x * 3 + (warp < x ? warp : warp - 1)) * KQ + k) * 32 + lane];
                    }
                    acc.x = fmaf(f[x][0], v.x, acc.x);
                    acc.y = fmaf(f[x][1], v.y, acc.y);
                    acc.z = fmaf(f[x][0], v.z, acc.z);
                    acc.w = fmaf(f[x][1], v.w, acc.w);
                }
                const int c = (warp * KQ + k) * 16 + (lane >> 2) * 2;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int h = n * 8 + 2 * (lane & 3) + i;
                    const float y0 = i ? acc.y : acc.x, y1 = i ? acc.w : acc.z;
                    if (h >= done.hn) continue;
                    if (whole) {
                        T* out = (T*)a.out + (size_t)done.b * a.p.out_stride + (size_t)(done.head0 + h) * D + c;
                        *reinterpret_cast<uint32_t*>(out) = Num<T>::pack(y0, y1);
                        if (k == 0 && warp == 0 && lane < 4 && a.lse)
                            a.lse[(size_t)done.b * a.p.Hq + done.head0 + h] = lse_of(mh[i], lh[i]);
                    } else {
                        *reinterpret_cast<float2*>(mine + h * D + c) = make_float2(y0, y1);
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
            } else if (U < (1 << 21)) {
                c0 = (int)(((unsigned int)done.unit0 + 1) * (unsigned int)C - 1) / (int)U;
                c1 = (int)(((unsigned int)done.unit0 + done.nb) * (unsigned int)C - 1) / (int)U;
            } else {
                c0 = (int)(((done.unit0 + 1) * C - 1) / U);
                c1 = (int)(((done.unit0 + done.nb) * C - 1) / U);
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
                for (int h = tid / TPR; h < done.hn; h += kThreads / TPR) {
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
                        const float ref = top == -INFINITY ? 0.f : top, g = exp2_fast(mh - ref);
                        mh = top;
                        lh *= g;
                        y.x *= g, y.y *= g, y.z *= g, y.w *= g;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (i0 + j >= n) break;
                            const float f = exp2_fast(pm[j] - ref) * ll[j];
                            lh += f;
                            y.x = fmaf(f, v[j].x, y.x);
                            y.y = fmaf(f, v[j].y, y.y);
                            y.z = fmaf(f, v[j].z, y.z);
                            y.w = fmaf(f, v[j].w, y.w);
                        }
                    }
                    const float inv = lh == 0.f ? 0.f : 1.f / lh;
                    y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
                    if (result) {
                        T* out = (T*)a.out + (size_t)done.b * a.p.out_stride + (size_t)(done.head0 + h) * D + c;
                        *reinterpret_cast<uint2*>(out) = make_uint2(Num<T>::pack(y.x, y.y), Num<T>::pack(y.z, y.w));
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

template <typename T, int D, int NT, int FORMAT>
cudaError_t launch_nt(const Paged8Args& a, cudaStream_t st)
{
    auto k = paged8_attend_kernel<T, D, NT, FORMAT>;
    const int smem = Cfg<D>::SMEM, ctas = Cfg<D>::CTAS;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // an upper bound of the units: lengths are known on the device only
    long long most = (long long)a.p.max_pages << a.shift;
    if (a.p.window > 0) most = most < (long long)a.p.window + a.p.sinks ? most : (long long)a.p.window + a.p.sinks;
    const long long chunks = (a.grp + 8 * NT - 1) / (8 * NT);
    const long long units = ((most + kBlock - 1) / kBlock + 2) * a.p.B * a.p.Hkv * chunks;
    return launch_pdl(k, dim3((unsigned)(units < ctas ? units : ctas)), dim3(kThreads), smem, st, a);
}

template <typename T, int D>
cudaError_t launch_t(const Paged8Args& a, cudaStream_t st)
{
    if (a.p.format == FADKV_E4M3) return a.grp <= 8 ? launch_nt<T, D, 1, FADKV_E4M3>(a, st) : launch_nt<T, D, 2, FADKV_E4M3>(a, st);
    return a.grp <= 8 ? launch_nt<T, D, 1, FADKV_I8>(a, st) : launch_nt<T, D, 2, FADKV_I8>(a, st);
}

}  // namespace

size_t paged8_attend_workspace(const fadkv_paged8_params& p)
{
    return kHeadBytes + (size_t)2 * (p.d == 128 ? Cfg<128>::CTAS : Cfg<64>::CTAS) * piece_floats(p.d) * sizeof(float);
}

cudaError_t launch_paged8_attend(const Paged8Args& a, cudaStream_t st)
{
    if (a.p.B <= 0) return cudaSuccess;
    if (a.p.dtype == FADKV_F16) return a.p.d == 128 ? launch_t<__half, 128>(a, st) : launch_t<__half, 64>(a, st);
    return a.p.d == 128 ? launch_t<__nv_bfloat16, 128>(a, st) : launch_t<__nv_bfloat16, 64>(a, st);
}

}  // namespace fadkv
