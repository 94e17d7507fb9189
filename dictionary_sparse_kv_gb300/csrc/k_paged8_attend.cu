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
// one block of tokens.  The weights enter as two binary16 terms; up to four heads
// leave half of a product's eight columns idle, which then take the second
// terms (16 products a tile in place of 24).  Pages, places and scales are looked
// up for 32 tiles at a time, a lane each.
//
// The work is one list of 64-token blocks, request by request and KV head by
// KV head.  Blocks lie at multiples of 64 tokens (a window's first one is partly
// seen), so that a warp's tile is one page, one block of scales and one run of
// bytes.  Mostly a CTA takes one piece of one (request, KV head), of equal parts
// no longer than they have to be, and joins where its tiles were; where there
// are more (request, heads) than CTAs, an even share of the list.  Pieces go to
// the workspace and the CTA that arrives last joins them in their order, so the
// result does not depend on which one that was.
//
// 64 requests of up to 16384 tokens, 32 heads over 8 of 128: 166 us, 6.6 TB/s
// (I8 the same; d = 64 5.9 TB/s, instructions; 16 heads a KV head 3.8 TB/s,
// instruction latency).  16 of up to 4096 18.8 us: 2 until the lengths are cut, 3
// until every warp has codes, 8 of codes at 6 TB/s, 3 of joins, and pieces that
// end apart.  One of 777 tokens 7.1 us: the chain lengths -> table -> codes 2.3,
// the joins 3.5.  Tiles by TMA, one box each of keys and values: 183 us where
// this took 184 (an instruction count of three quarters did not show), and half
// a microsecond more before the first tile.
#include <algorithm>

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
constexpr float kUp = 11.f;                        // 15 - kGrow: w is multiplied by 2^kUp for the product
constexpr int kExtra = 3;                          // units that a piece costs beside its blocks
constexpr int kSms = 152;

// ONE: a CTA takes one piece, and joins where its tiles were.  WIDE: sixteen
// heads a piece, whose sums want the registers of fewer CTAs.  (us, 16 requests of
// up to 4096 tokens of 8 heads of 128, 113 of 1024 of two of 64: 18.8 and 15.7,
// with a stage or two more 19.5 and 16.2; 64 of up to 16384 of eight of 64: 92, a
// stage more 95; 64 of up to 32000 with 16 heads over one of 128: 62, with three
// CTAs 71.)
template <int D, bool ONE, bool WIDE> struct Cfg {
    static constexpr int PER_SM = D == 128 ? (WIDE ? 2 : 3) : (WIDE ? 3 : 4);
    static constexpr int STAGES = ONE && D == 64 ? 4 : 3;
    static constexpr int TILE_BYTES = kTile * D;
    static constexpr int WARP_BYTES = STAGES * 2 * TILE_BYTES;
    static constexpr int ROW = D + 8;                                  // floats of a result: d values, m, l; padding
    static constexpr int JOIN_BYTES = ONE ? kWarps * WARP_BYTES : D == 128 ? 24576 : 16384;   // results that are joined
    static constexpr int SMEM = kWarps * WARP_BYTES + (ONE ? 0 : JOIN_BYTES);
};
template <int D, bool WIDE = false> constexpr int kCtas = Cfg<D, true, WIDE>::PER_SM * kSms;

// Pieces that one CTA joins: more are joined in groups, as in the 16-bit kernel.
constexpr int kAtOnce = 32, kGroup = 16;
constexpr int kCounters = 1024;
static_assert(kCtas<64> <= kCounters && kCtas<128> <= kCounters, "counters");
static_assert(3 * kCounters * sizeof(int) <= kHeadBytes - kDecodeHead, "workspace head");

template <int D> constexpr int kLeastJoin = (kAtOnce > 8 * kWarps ? kAtOnce : 8 * kWarps) * (D + 8) * 4;
static_assert(Cfg<64, true, false>::JOIN_BYTES >= kLeastJoin<64> && Cfg<64, false, false>::JOIN_BYTES >= kLeastJoin<64> &&
              Cfg<128, true, false>::JOIN_BYTES >= kLeastJoin<128> && Cfg<128, false, false>::JOIN_BYTES >= kLeastJoin<128>, "join");

// A piece in the workspace: a row for each of its heads.
__host__ __device__ constexpr size_t piece_floats(int d) { return (size_t)kMaxHeads * (d + 8); }

// Byte offset of 16-byte chunk c of row r: eight rows at one chunk lie in
// eight different bank groups.
template <int D>
__device__ __forceinline__ uint32_t swz8(int r, int c)
{
    return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void cp16_all(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

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

// TILES of eight heads; 0: four heads, twice, for the two terms of their
// weights, which one product then takes together.
template <typename T, int D, int TILES, int FORMAT, bool ONE>
__global__ void __launch_bounds__(kThreads, Cfg<D, ONE, TILES == 2>::PER_SM)
paged8_attend_kernel(const __grid_constant__ Paged8Args a)
{
    constexpr bool TWO = TILES == 0;
    constexpr int NT = TWO ? 1 : TILES;
    using C_ = Cfg<D, ONE, TILES == 2>;
    constexpr int STAGES = C_::STAGES, CPR = D / 16;                   // 16-byte chunks per row
    constexpr int KS = D / 16, ROW = C_::ROW;                          // 16-element steps; floats of a result
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ int s_b, s_last, s_sum[2][kWarps];
    __shared__ long long s_unit;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = a.grp, B = a.p.B, grid = (int)gridDim.x;
    const int chunks = (grp + 8 * NT - 1) / (8 * NT);                 // pieces per KV head
    const int segs = a.p.Hkv * chunks, sets = B * segs;
    unsigned char* wsmem = smem + warp * C_::WARP_BYTES;
    const uint32_t wbase = saddr(wsmem);
    float* rows = reinterpret_cast<float*>(smem + (ONE ? 0 : kWarps * C_::WARP_BYTES));
    prefetch_tables(a.lengths, a.table, B, a.p.max_pages);
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

    // How the work is cut.  Where the (request, heads) are no more than the CTAs, every CTA takes one piece: as many for
    // each as keep its pieces at `most` blocks or fewer, the least that the grid has room for.  Where they are more, the
    // list is cut into even shares, each (request, heads) kExtra units longer than its blocks, which is what a piece costs.
    int cur_b, parts = 1, part = 0, seg = 0;                           // one: this CTA's piece
    int C = 1;                                                         // shares: how many, no more than units, so that none is empty
    long long u = 0, u1 = 1, U = 0, base = 0;                          // shares: this CTA's units; all; the first of request cur_b
    // Each thread has the requests b0 .. b1-1: a lane each, the same in every warp, for up to 32; else over the block.
    const bool few = B <= 32;
    const int each = few ? 1 : (B + kThreads - 1) / kThreads, b0 = min(B, (few ? lane : tid) * each), b1 = min(B, b0 + each);
    auto total = [&](int v, int slot) {                                // over the requests; the slots in turn
        v = __reduce_add_sync(0xffffffffu, v);
        if (!few) {
            if (lane == 0) s_sum[slot][warp] = v;
            __syncthreads();
            v = 0;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) v += s_sum[slot][x];
        }
        return v;
    };
    if (ONE) {
        constexpr int kEach = (kCtas<D> + kThreads - 1) / kThreads;   // there are no more requests than CTAs
        int nb[kEach], sum = 0, longest = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            nb[i] = b0 + i < b1 ? units_of(b0 + i) : 0;
            sum += nb[i];
            longest = max(longest, nb[i]);
        }
        const unsigned all = (unsigned)total(sum, 0) * (unsigned)segs;
        auto pieces = [&](int x) {                                     // of at most x blocks
            int n = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (i < each) n += (int)(((unsigned)nb[i] + (unsigned)x - 1u) / (unsigned)x);
            return n;
        };
        // (all / x + sets of them are too many: this x is large enough)
        int lo = (int)((all + grid - 1) / grid), hi = 0x7fffffff;
        if (few) longest = __reduce_max_sync(0xffffffffu, longest);
        if (sets < grid) hi = (int)(all / (unsigned)(grid - sets)) + 1;
        else hi = few ? longest : (int)all;
        // Few requests: pieces that are worth their join, which grows with their number (one request of 24 heads over 8 of 128, us: 5
        // blocks 6.1 whole and 6.6 in 5 pieces; 24 blocks 9.1 in 24, 7.9 in 12, 8.3 in 6; 47 blocks 10.6 in 47, 10.1 in 16, 11.1 in
        // 6; 63 blocks of 8 heads over 1 13.2 in 63, 12.5 in 16 and in 8).
        if (few) lo = max(lo, longest <= 6 ? longest : (int)ceilf(sqrtf((float)longest * (1.f / 6.f))));
        hi = max(lo, hi);
        int slot = 1;
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (total(pieces(mid), slot) * segs <= grid) hi = mid;
            else lo = mid + 1;
            slot ^= 1;
        }
        const int mine = pieces(hi) * segs;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        int end = __shfl_sync(0xffffffffu, upto, 31);
        if (!few) {
            if (lane == 31) s_sum[slot][warp] = upto;
            __syncthreads();
            end = 0;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                if (x < warp) upto += s_sum[slot][x];
                end += s_sum[slot][x];
            }
        }
        if ((int)blockIdx.x >= end) return;
        int from = upto - mine;
        if (few) {
            cur_b = __ffs(__ballot_sync(0xffffffffu, upto > (int)blockIdx.x)) - 1;
            from = __shfl_sync(0xffffffffu, from, cur_b);
        } else {
            if ((int)blockIdx.x >= from && (int)blockIdx.x < upto) {
                int b = b0;
                for (int n; (int)blockIdx.x >= from + (n = (units_of(b) + hi - 1) / hi * segs); ++b) from += n;
                s_b = b;
                s_unit = from;
            }
            __syncthreads();
            cur_b = s_b;
            from = (int)s_unit;
        }
        parts = (units_of(cur_b) + hi - 1) / hi;
        const int rel = (int)blockIdx.x - from;
        seg = rel / parts;
        part = rel - seg * parts;
    } else {
        auto units = [&](int b) { return (long long)(units_of(b) + kExtra) * segs; };
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += units(b);
        long long from;
        if (few) {
            long long upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            U = __shfl_sync(0xffffffffu, upto, 31);
            from = upto - mine;
        } else {
            from = block_scan<kThreads>(mine, &U);
        }
        C = (int)min((long long)grid, U);
        if ((int)blockIdx.x >= C) return;
        u = U * blockIdx.x / C;
        u1 = U * (blockIdx.x + 1) / C;
        if (few) {
            cur_b = __ffs(__ballot_sync(0xffffffffu, from + mine > u)) - 1;
            base = __shfl_sync(0xffffffffu, from, cur_b);
        } else {
            if (u >= from && u < from + mine) {
                int b = b0;
                for (long long n; u >= from + (n = units(b)); ++b) from += n;
                s_b = b;
                s_unit = from;
            }
            __syncthreads();
            cur_b = s_b;
            base = s_unit;
        }
    }

    // the next piece from unit u on (none: blk0 == blk1); u, cur_b and base move past it
    auto next_work = [&] {
        Work w;
        for (;;) {
            w.b = cur_b;
            w.seen = blocks_of(cur_b);
            w.nb = max(1, w.seen.count);
            w.unit0 = 0;
            if (ONE) {
                const int each = w.nb / parts, rest = w.nb % parts;          // the first `rest` parts take one block more
                w.blk0 = part * each + min(part, rest);
                w.blk1 = w.blk0 + each + (part < rest);
                u = u1;
                break;
            }
            const int len = w.nb + kExtra;
            const long long rel = u - base;
            seg = rel < 0x7fffffffll ? (int)rel / len : (int)(rel / len);
            w.unit0 = base + (long long)seg * len;
            const int lo = (int)(u - w.unit0), hi = (int)min((long long)len, lo + (u1 - u));
            w.blk0 = min(lo, w.nb);
            w.blk1 = min(hi, w.nb);
            u += hi - lo;
            if (hi == len && seg == segs - 1) {
                base += (long long)len * segs;
                ++cur_b;
            }
            if (w.blk0 < w.blk1 || u >= u1) break;                           // (what is left of a share may be past the blocks)
        }
        w.hk = chunks == 1 ? seg : seg / chunks;
        const int h0 = chunks == 1 ? 0 : (seg % chunks) * 8 * NT;
        w.hn = min(8 * NT, grp - h0);
        w.head0 = w.hk * grp + h0;
        return w;
    };

    // The piece's tiles of this warp (16 tokens of each block), 32 at a time, a lane each: page, tokens that are seen (none on
    // a page that is none), where they lie in the pools, scale of the keys, log2 of the values'.
    struct Info { int page; uint32_t seen; long long off; float ks, ls; };
    Info cur, nxt;
    auto token_of = [&](const Work& w, int t) { return w.seen.token(w.blk0 + t) + warp * kTile; };
    auto pages = [&](const Work& w, int t, Info& f) {
        f.page = -1;
        f.seen = 0u;
        if (w.blk0 + t + lane < w.blk1) {
            const int tok = token_of(w, t + lane);
            f.seen = w.seen.seen(tok);
            if (f.seen) f.page = __ldg(a.table + (size_t)w.b * a.p.max_pages + (tok >> a.shift));
        }
    };
    auto places = [&](const Work& w, int t, Info& f) {
        if (f.page < 0 || f.page >= a.p.num_pages) f.seen = 0u;
        f.off = f.seen ? f.page * a.p.page_stride + (token_of(w, t + lane) & ((1 << a.shift) - 1)) * a.p.token_stride : 0;
    };
    auto scales = [&](const Work& w, int t, Info& f) {
        f.ks = f.ls = 0.f;
        if (f.seen) {
            const size_t at = scale_at(f.page, w.hk, token_of(w, t + lane) & ((1 << a.shift) - 1), a.p.Hkv, a.shift, a.bshift);
            f.ks = __ldg(a.k_scales + at);
            f.ks = fmaf(f.ks, 0.f, f.ks);                              // an infinity as NaN: its score would be -inf, which nothing shows
            f.ls = __log2f(__ldg(a.v_scales + at));
        }
    };
    const int row0 = lane / CPR, chunk = lane % CPR;                   // this lane's chunks of a tile: rows row0 + j 32 / CPR
    const long long lane_off = row0 * a.p.token_stride + chunk * 16, step_off = (32 / CPR) * a.p.token_stride;
    int st_in = 0, st_out = 0;                                         // the ring's next tile to load and to use
    // tile t, whose Info is in f
    auto load = [&](const Work& w, int t, const Info& f) {
        const uint32_t seen = __shfl_sync(0xffffffffu, f.seen, t & 31);
        const uint32_t dst = wbase + st_in * 2 * C_::TILE_BYTES;
        st_in = st_in + 1 == STAGES ? 0 : st_in + 1;
        const long long off = __shfl_sync(0xffffffffu, f.off, t & 31) + w.hk * a.p.head_stride + lane_off;
        const uint8_t *k = a.k + off, *v = a.v + off;
        if (seen == 0xffffu) {
#pragma unroll
            for (int j = 0; j < kTile * CPR / 32; ++j) {
                cp16_all(dst + swz8<D>(row0 + j * (32 / CPR), chunk), k + j * step_off);
                cp16_all(dst + C_::TILE_BYTES + swz8<D>(row0 + j * (32 / CPR), chunk), v + j * step_off);
            }
        } else if (seen) {
#pragma unroll
            for (int j = 0; j < kTile * CPR / 32; ++j) {
                const int r = row0 + j * (32 / CPR);
                cp16(dst + swz8<D>(r, chunk), k + j * step_off, (seen >> r) & 1u);
                cp16(dst + C_::TILE_BYTES + swz8<D>(r, chunk), v + j * step_off, (seen >> r) & 1u);
            }
        }
    };
    auto begin = [&](const Work& w) {                                   // the first tiles, STAGES - 1 copy groups
        st_in = st_out = 0;
        pages(w, 0, cur);
        places(w, 0, cur);
        for (int t = 0; t < STAGES - 1; ++t) {
            if (w.blk0 + t < w.blk1) load(w, t, cur);
            cp_commit();
        }
        scales(w, 0, cur);
        pages(w, 32, nxt);
    };
    // Queries as the B operand: lane holds head lane / 4; of step k its elements 16 k + 4 (lane % 4) + {0, 1, 2, 3}, the
    // order in which the lanes have a row's bytes.  qs: what the scores of heads 2 (lane % 4) + {0, 1} are multiplied by.
    uint32_t qf[NT][KS][2];
    float qs[NT][2], qo[NT][2];                                        // (qo: kOffset times the sum of their elements)
    auto load_q = [&](const Work& w) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int h = n * 8 + (TWO ? lane >> 2 & 3 : lane >> 2);
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
            if (Code<FORMAT>::kOffset != 0.f) {
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const float2 y = Num<__half>::unpack(qf[n][k][0]), z = Num<__half>::unpack(qf[n][k][1]);
                    sum += (y.x + y.y) + (z.x + z.y);
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                sum *= Code<FORMAT>::kOffset;
                qo[n][0] = __shfl_sync(0xffffffffu, sum, (lane & 3) * 8);
                qo[n][1] = __shfl_sync(0xffffffffu, sum, (lane & 3) * 8 + 4);
            }
        }
    };

    Work w = next_work();
    if (w.blk0 == w.blk1) return;                                       // a share without a block
    begin(w);
    load_q(w);
    for (;;) {
        // references mr and Mr of the exponents (0 before the first token) and what has to be passed to move them
        float o[NT][KS][4], mr[NT][2], Mr[NT][2], mg[NT][2], Mg[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mr[n][0] = mr[n][1] = Mr[n][0] = Mr[n][1] = 0.f;
            mg[n][0] = mg[n][1] = Mg[n][0] = Mg[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }
        const int tiles = w.blk1 - w.blk0;
        for (int t = 0; t < tiles; ++t) {
            if ((t & 31) == 0 && t > 0) {
                cur = nxt;
                pages(w, t + 32, nxt);
            }
            if ((t & 31) == 16) {
                places(w, (t & ~31) + 32, nxt);
                scales(w, (t & ~31) + 32, nxt);
            }
            cp_wait<STAGES - 2>();
            __syncwarp();
            const int ahead = t + STAGES - 1;
            if (ahead < tiles) load(w, ahead, (ahead ^ t) < 32 ? cur : nxt);
            cp_commit();
            const uint32_t kt = wbase + st_out * 2 * C_::TILE_BYTES, vt = kt + C_::TILE_BYTES;
            st_out = st_out + 1 == STAGES ? 0 : st_out + 1;
            const uint32_t oks = __shfl_sync(0xffffffffu, cur.seen, t & 31);
            if (oks == 0u) continue;
            const float ks = __shfl_sync(0xffffffffu, cur.ks, t & 31), ls = __shfl_sync(0xffffffffu, cur.ls, t & 31);
            float sc[NT][4], sc2[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[n][i] = sc2[n][i] = 0.f;
            const int r = (lane & 7) + ((lane >> 3) & 1) * 8, c = lane >> 4;
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
                uint32_t b[4];
                ldsm_x4(b, kt + swz8<D>(r, k + c));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t f[4];
                    Code<FORMAT>::shifted(b[2 * i], f[0], f[2]);
                    Code<FORMAT>::shifted(b[2 * i + 1], f[1], f[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) Num<__half>::mma(i ? sc2[n] : sc[n], f, qf[n][k + i][0], qf[n][k + i][1]);
                }
            }
            bool grew = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sc[n][i] += sc2[n][i];
                    if (Code<FORMAT>::kOffset != 0.f) sc[n][i] = fmaf(sc[n][i], Code<FORMAT>::kUnit, -qo[n][i & 1]);
                    sc[n][i] *= ks * qs[n][i & 1];
                }
                if (oks != 0xffffu) {
                    const bool ok0 = (oks >> (lane >> 2)) & 1u, ok1 = (oks >> ((lane >> 2) + 8)) & 1u;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!(i < 2 ? ok0 : ok1)) sc[n][i] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float v = fmaxf(sc[n][i], sc[n][i + 2]);
                    grew |= v > fminf(mg[n][i], Mg[n][i] - ls);
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
                        // (the first time there is nothing to rescale)
                        const bool first = mg[n][i] == -INFINITY, First = Mg[n][i] == -INFINITY;
                        if (first ? v > mg[n][i] : v > mr[n][i]) {
                            l[n][i] *= first ? 0.f : exp2_fast(mr[n][i] - v);
                            mr[n][i] = v;
                            mg[n][i] = v + kGrow;
                        }
                        f[i] = 1.f;
                        v += ls;
                        if (First ? v > Mg[n][i] : v > Mr[n][i]) {
                            f[i] = First ? 0.f : exp2_fast(Mr[n][i] - v);
                            Mr[n][i] = v;
                            Mg[n][i] = v + kGrow;
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
                const float up[2] = {ls - Mr[n][0] + kUp, ls - Mr[n][1] + kUp};
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    l[n][i & 1] += exp2_fast(sc[n][i] - mr[n][i & 1]);
                    e[i] = exp2_fast(sc[n][i] + up[i & 1]);
                }
                const uint32_t a0 = Num<__half>::pack(e[0], e[1]), a1 = Num<__half>::pack(e[2], e[3]);
                const float2 r0 = Num<__half>::unpack(a0), r1 = Num<__half>::unpack(a1);
                const uint32_t b0 = Num<__half>::pack(e[0] - r0.x, e[1] - r0.y), b1 = Num<__half>::pack(e[2] - r1.x, e[3] - r1.y);
                ph[n][0] = transpose8(TWO && (lane & 2) ? b0 : a0);
                ph[n][1] = transpose8(TWO && (lane & 2) ? b1 : a1);
                if (!TWO) {
                    pl[n][0] = transpose8(b0);
                    pl[n][1] = transpose8(b1);
                }
            }
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
                        if (!TWO) Num<__half>::mma(o[n][k + i], f, pl[n][0], pl[n][1]);
                    }
                }
            }
        }
        __syncwarp();
        if (ONE) {                                                      // the joins' rows lie over every warp's tiles
            cp_wait<0>();
            __syncthreads();
        }
        const Work done = w;
        bool more = !ONE && u < u1;
        if (more) {                                                     // every buffer of this warp is free
            w = next_work();
            more = w.blk0 < w.blk1;
            if (more) {
                begin(w);
                load_q(w);
            }
        }

        // Results are rows of d values, m and l, the values divided by l.  Joins n rows of each of the heads h0 .. h0 + heads - 1
        // of the piece, row (j, h) at rows + (j each + h) ROW, four columns a thread: as the result, or into a piece.
        auto combine = [&](int n, int each, int heads, int h0, bool result, float* piece) {
            constexpr int TPR = D / 4;                  // threads per row
            const int c = tid % TPR * 4, step = each * ROW;
#pragma unroll 1
            for (int h = tid / TPR; h < heads; h += kThreads / TPR) {
                const float* r = rows + h * ROW;
                float top = -INFINITY, lh = 0.f;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int j = 0; j < n; ++j) top = fmaxf(top, r[j * step + D]);
                const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 4
                for (int j = 0; j < n; ++j) {
                    const float f = exp2_fast(r[j * step + D] - ref) * r[j * step + D + 1];
                    const float4 v = *reinterpret_cast<const float4*>(r + j * step + c);
                    lh += f;
                    y.x = fmaf(f, v.x, y.x);
                    y.y = fmaf(f, v.y, y.y);
                    y.z = fmaf(f, v.z, y.z);
                    y.w = fmaf(f, v.w, y.w);
                }
                const float inv = lh == 0.f ? 0.f : __fdividef(1.f, lh);
                y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
                if (result) {
                    const size_t row = (size_t)done.b * a.p.Hq + done.head0 + h0 + h;
                    T* out = (T*)a.out + (size_t)done.b * a.p.out_stride + (size_t)(done.head0 + h0 + h) * D + c;
                    *reinterpret_cast<uint2*>(out) = make_uint2(Num<T>::pack(y.x, y.y), Num<T>::pack(y.z, y.w));
                    if (c == 0 && a.lse) a.lse[row] = lh == 0.f ? -INFINITY : (top + __log2f(lh)) * kLn2;
                } else {
                    float* q = piece + (size_t)(h0 + h) * ROW;
                    *reinterpret_cast<float4*>(q + c) = y;
                    if (c == 0) *reinterpret_cast<float2*>(q + D) = make_float2(top, lh);
                }
            }
        };
        const bool whole = done.blk0 == 0 && done.blk1 == done.nb;
        float* pieces = reinterpret_cast<float*>((unsigned char*)a.ws + kHeadBytes);
        constexpr size_t PF = piece_floats(D);
        float* mine = pieces + (2 * (size_t)blockIdx.x + (done.blk0 == 0 ? 1 : 0)) * PF;
        // the warps' results, eight heads at a time.  o[n][k] holds heads n 8 + 2 (lane % 4) + {0, 1} of elements
        // k 16 + 2 (lane / 4) (first two) and the one after it.
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v = l[n][i];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                // 2^(M - m) / l; for values so small that it is no number of the normal range, in two steps
                const float e = Mg[n][i] == -INFINITY ? 0.f : Mr[n][i] - mr[n][i] - kUp;
                const float f = v == 0.f ? 0.f : __fdividef(exp2_fast(e < -64.f ? e + 64.f : e), v);
                const float g = e < -64.f ? 0x1p-64f : 1.f;
                float* r = rows + (warp * 8 + 2 * (lane & 3) + i) * ROW;       // (f is 0 where nothing was seen)
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    float2 y = make_float2(o[n][k][i], o[n][k][i + 2]);
                    if (TWO) {                          // both terms' sums
                        y.x += __shfl_xor_sync(0xffffffffu, y.x, 2);
                        y.y += __shfl_xor_sync(0xffffffffu, y.y, 2);
                    }
                    *reinterpret_cast<float2*>(r + k * 16 + (lane >> 2) * 2) = make_float2(y.x * f * g, y.y * f * g);
                }
                if (lane < 4) *reinterpret_cast<float2*>(r + D) = make_float2(mg[n][i] == -INFINITY ? -INFINITY : mr[n][i], v);
            }
            __syncthreads();
            combine(kWarps, 8, min(8, done.hn - n * 8), n * 8, whole, mine);
            __syncthreads();                            // the rows are written again
        }
        if (!whole) {
            // the CTAs that have its pieces; of shares, unit x is in share ((x + 1) C - 1) / U
            int c0, c1;
            if (ONE) {
                c0 = (int)blockIdx.x - part;
                c1 = c0 + parts - 1;
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
            // pieces x0, x0 + step, ... (n of them) in their order, so that it does not matter who joins them; as many heads at a
            // time as there is room for; into the first one, or as the result
            auto join = [&](int x0, int n, int step, bool result) {
                constexpr int CPW = ROW / 4;            // 16-byte chunks per row
                const int group = min(done.hn, C_::JOIN_BYTES / (n * ROW * 4));
#pragma unroll 1
                for (int h0 = 0; h0 < done.hn; h0 += group) {
                    const int heads = min(group, done.hn - h0);
#pragma unroll 1
                    for (int x = tid; x < n * heads * CPW; x += kThreads) {
                        const int row = x / CPW, j = row / heads;
                        cp16(saddr(rows) + x * 16, piece(x0 + j * step) + (h0 + row - j * heads) * ROW + (x - row * CPW) * 4, true);
                    }
                    cp_commit();
                    cp_wait<0>();
                    __syncthreads();
                    combine(n, heads, heads, h0, result, piece(x0));
                    __syncthreads();
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
        }
        if (!more) break;
    }
}

template <typename T, int D, int TILES, int FORMAT, bool ONE>
cudaError_t launch_one(const Paged8Args& a, int grid, cudaStream_t st)
{
    auto k = paged8_attend_kernel<T, D, TILES, FORMAT, ONE>;
    const int smem = Cfg<D, ONE, TILES == 2>::SMEM;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(k, dim3((unsigned)grid), dim3(kThreads), smem, st, a);
}

template <typename T, int D, int TILES, int FORMAT>
cudaError_t launch_nt(const Paged8Args& a, cudaStream_t st)
{
    constexpr int NT = TILES == 0 ? 1 : TILES;
    // an upper bound of the units: lengths are known on the device only
    long long most = (long long)a.p.max_pages << a.shift;
    if (a.p.window > 0) most = most < (long long)a.p.window + a.p.sinks ? most : (long long)a.p.window + a.p.sinks;
    const long long sets = (long long)a.p.B * a.p.Hkv * ((a.grp + 8 * NT - 1) / (8 * NT));
    const long long units = ((most + kBlock - 1) / kBlock + 2) * sets;
    const int grid = (int)std::min(units, (long long)kCtas<D, TILES == 2>);
    // A piece a CTA, or even shares: where the (request, heads) are between half of the CTAs and all of them, few can be cut, and
    // long ones leave many CTAs waiting (us, requests of 24 heads over 8 of 128, in pieces and in shares: 40 of 300 tokens 10.0 and
    // 13.3, of 1500 27.1 and 27.2, of 6000 83 and 80; of up to 6000 51 and 45; 56 of up to 6000 77 and 61).  What the tables have
    // room for is all that is known of the lengths here, so short requests in wide tables take the shares: 40 of 300 tokens in tables
    // of 32768 13.4, in tables of 300 9.9; 56 of 300 15.6 and 12.4.  (In pieces sums of units are kept in 32 bits.)
    if (sets <= grid && (2 * sets <= grid || most <= 4096) && units < 0x7fffffffll) return launch_one<T, D, TILES, FORMAT, true>(a, grid, st);
    return launch_one<T, D, TILES, FORMAT, false>(a, grid, st);
}

template <typename T, int D, int FORMAT>
cudaError_t launch_f(const Paged8Args& a, cudaStream_t st)
{
    if (a.grp <= 4) return launch_nt<T, D, 0, FORMAT>(a, st);
    return a.grp <= 8 ? launch_nt<T, D, 1, FORMAT>(a, st) : launch_nt<T, D, 2, FORMAT>(a, st);
}

template <typename T, int D>
cudaError_t launch_t(const Paged8Args& a, cudaStream_t st)
{
    return a.p.format == FADKV_E4M3 ? launch_f<T, D, FADKV_E4M3>(a, st) : launch_f<T, D, FADKV_I8>(a, st);
}

}  // namespace

size_t paged8_attend_workspace(const fadkv_paged8_params& p)
{
    return kHeadBytes + (size_t)2 * (p.d == 128 ? kCtas<128> : kCtas<64>) * piece_floats(p.d) * sizeof(float);
}

cudaError_t launch_paged8_attend(const Paged8Args& a, cudaStream_t st)
{
    if (a.p.B <= 0) return cudaSuccess;
    if (a.p.dtype == FADKV_F16) return a.p.d == 128 ? launch_t<__half, 128>(a, st) : launch_t<__half, 64>(a, st);
    return a.p.d == 128 ? launch_t<__nv_bfloat16, 128>(a, st) : launch_t<__nv_bfloat16, 64>(a, st);
}

}  // namespace fadkv
