// Attention of chunks of new tokens over the paged cache, on the 5th-generation
// tensor cores.
//
// One pass over the keys with the running maximum m and sum l of the softmax:
//   x = scale log2(e) q k^T,  p = 2^(x - m),  o = o 2^(m_old - m) + p v,
// out = o / l.  Rows of a tile are (token, head) pairs of the query heads that
// share a KV head, token by token, so that a key tile that is loaded serves
// the whole group, chunks of a few tokens still fill the rows and a tile spans
// few positions (42 tokens with three heads a KV head), which leaves little of
// the last key tiles masked.
//
// A CTA takes two tiles of 128 rows against key tiles of 128 tokens: S = Q K^T
// and O += P V are tcgen05 products (M = 128, FP32 sums in TMEM: two S and two
// O accumulators), Q, K and V in shared memory, P in TMEM as 16-bit values
// over its own S.  While one tile's softmax runs on four warps (a thread a
// row), the tensor cores work on the other tile: per 128 x 128 scores at d =
// 128 the two products take 1024 cycles of a multiprocessor's tensor cores,
// the exponentials 512 of its special-function units.  The tensor cores bound
// it: 8192 tokens of 24 heads over 8 of 128 in bfloat16 take 255 us, 1.6 PFLOP/s
// (280 us, 1.5, in long runs under the power limit).  At d = 64 a step's
// products take half as long as its softmax: 12001 tokens of 8 heads over 2,
// window 1024, 57 us.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since
// the last time, which after the first tiles is rare (o / l is the same); the
// rescale goes through registers in the softmax warps.  m need not be the
// maximum itself: p = 2^(x - m) with m 7 below it in binary16, where p then
// reaches 2^15 at most and is lost below 2^-25, that is 2^-32 of the largest
// (with m the maximum 32768 keys 17.5 below one whose value is 0 came out as
// 0).  bfloat16 has the exponents of 32 bits, and m is the maximum there.
//
// p is rounded once to the type of v (half a step at most, 2^-8 of it in bfloat16,
// 2^-11 in binary16), as tensor cores that bound the kernel take it; l is the sum of the
// unrounded ones.  The roundings are independent, so that out's error, which the
// rounding of out itself sets (2-norm over 2-norm 1.65e-3 in bfloat16, 2.1e-4 in
// binary16), comes to 1.1 (300 keys) to 1.35 (6000) times that: 2.15e-3, 2.8e-4.  A
// second term would be half as many products again.
//
// K and V pages come by TMA, one box a page and 64-element half, through one
// ring of stages; pages outside the pool and pages that no row sees are asked
// for outside the map and arrive as zeros.  Keys that a row does not see are
// masked in registers, in the key tiles where that can happen.  What a seen
// page holds past the tokens that the tile sees may be anything, so its value
// rows are zeroed in shared memory before the product (0 x NaN would be NaN).
//
// CTAs are persistent, one a multiprocessor, and take items (two tiles of one
// request and KV head) from a counter, a request's last tiles, which see the
// most keys, first, and several requests' tiles in turns of about as many keys,
// the most first (lengths are known on the device alone, so every CTA walks
// the requests by itself, a lane each).  The next item's queries and first pages are on their way
// while the last tiles of the current one are worked on; only the reading of
// O by the softmax warps stands between two items' products.
//
// Where the items are fewer than the multiprocessors (a short chunk on a long
// cache) each is cut along its keys into as many pieces as fill them (twice,
// where two pieces an item would leave many idle); the pieces' sums go to the
// workspace, and a second kernel joins them as
//   m = max m_i,  l = sum 2^(m_i - m) l_i,  o = sum 2^(m_i - m) o_i.
//
// Packed prompts (ROWS) are the same with keys and values as rows of their own:
// a key tile is one box a half, rows behind the prompt's last one are masked
// and cleared as those of a page are.  4 prompts of up to 6000 tokens, 32 heads
// over 8 of 128 in bfloat16: 385 to 433 us by the power limit, 1.45 to 1.6
// PFLOP/s; a part of the exponentials as polynomials on the other pipes cost more
// than it saved at either d (5 of 16 pairs at d = 64: 69.5 -> 74 us for prompts with
// a window; 2 of 16 at 128: 385 -> 430): the special-function units do not bound it.
//
// Warps: 0 TMA, 1 MMA, 2 the items, 3 TMEM, 4..7 and 8..11 softmax of the two
// tiles.  Every wait is bounded; one that runs out sets
// FADKV_DEV_TIMEOUT in the workspace's first word, and the CTA drains and
// returns: the copies, the products and the stores to TMEM that its warps
// issued are waited for before TMEM is given back.
#include <algorithm>

#include "paged.cuh"
#include "tc_common.cuh"

namespace fadkv {
namespace {

using namespace paged;
using namespace tc;

constexpr int kPreThreads = 384;
constexpr int kRows = 128;                         // (token, head) rows per tile, two tiles per CTA
constexpr int kKeys = 128;                         // keys per tile
constexpr int kOkRing = 16;                        // key tiles whose page masks are kept
constexpr int kPart = 64;                          // keys whose P is handed over first; the rest follows
constexpr float kGrow = 8.f;                       // growth of the maximum (log2) that rescales
template <typename T> constexpr float kBelow = std::is_same<T, __half>::value ? 7.f : 0.f;   // m below the maximum (log2)

constexpr int kPreCtas = 152;                      // one per multiprocessor
constexpr int kItemReaders = 10;                   // warps that read an item

// Waits for the next item last as long as the current one: a key tile takes
// 0.7 to 1.3 us, so that the 200 ms of a wait are over after 20 to 35 million keys.
// Those waits get this much more for each tile of the item.
constexpr unsigned int kTileNs = 8000;

// Pieces of an item: at most so many, and none shorter than so many key tiles
// (a piece costs about two tiles' time to begin, write out and join).
constexpr int kMaxParts = 64;
constexpr int kLeastTiles = 4;
constexpr int kSplitSlots = 2 * kPreCtas;          // pieces of all items where items are cut

// Turns in which the tiles of 2 to kSorted requests come, where they are more
// than the multiprocessors (d = 128; in turns against request by request, us:
// 16 requests of up to 300 tokens on 4000, 24 heads over 8: 59 against 74; 32 of
// 64 on 8000: 103 against 119; 40 of 200 on 2000: 81 against 85; 8 of 500 on
// 4000: 67.3 and 67.4.  Four turns: 60, 102, 81, 68.6; sixteen: 59, 103, 86, 68.1).
// Every turn walks all requests, so many come one by one (in turns 70 of 64 on
// 8000 take 189 against 214, 100 of 64 on 4000 166 and 171, but 200 of 20 on
// 4000 262 against 256 and 500 of 16 on 1000 250 against 210).
constexpr int kLevels = 8;
constexpr int kSorted = 96;

// Head of the workspace.
struct PreHead {
    unsigned long long status;
    unsigned int taken, left;                      // pieces handed out, CTAs that are done: zero between calls
    int parts, items;                              // of this call, for the join
    struct { int row0, nt, head0, hn; } item[kPreCtas];
};
static_assert(sizeof(PreHead) <= kDecodeHead && offsetof(PreHead, status) == 0, "workspace head");
__host__ __device__ constexpr size_t slot_floats(int d) { return (size_t)kRows * (d + 2); }   // a tile's rows: o by column, m, l

template <int D> struct PreCfg {
    static constexpr int NST = D == 128 ? 5 : 8;   // stages of the K / V ring
    static constexpr int TILE = kRows * D * 2;     // bytes of a Q, K or V tile
    static constexpr int bar_off = (2 + NST) * TILE;
    static constexpr int n_bars = 2 * NST + 19;
    static constexpr int ok_off = bar_off + n_bars * 8;
    static constexpr int alloc = ok_off + kOkRing * 20 + 16 + 1024;
    static_assert(alloc <= 227 * 1024 - 256, "shared memory");
    // TMEM columns.  d = 128: P over the first half of its S, so the next
    // scores are written where the product issued just before them reads P.
    // PTX promises the order of one thread's products for one accumulator
    // only; that two accumulators' products run in the order of their issue
    // is measured, not promised: 180 inputs of 60 shapes, three to eight runs
    // each, gave the same bits as a build that waits for the first one (302
    // us instead of 277 for a prompt of 8192 tokens, 75 instead of 70.5 for 8
    // chunks of 500).  d = 64: room for its own, so the next scores go ahead
    // of the product that reads P.
    static constexpr bool kOwnP = D == 64;
    static constexpr int S(int q) { return q * 128; }
    static constexpr int O(int q) { return 256 + q * D; }
    static constexpr int P(int q) { return kOwnP ? 384 + q * 64 : q * 128; }
};

// An item as the scheduling warp hands it to the others.
struct Item {
    int live;                  // 0: no more items
    int row0, nt;              // first row of q, tokens
    int first, len;            // position of the first row; tokens of the request
    int b, head0, hk, hn;      // request, first query head, KV head, query heads
    int index, piece, parts;   // number of the item; which part of its key tiles
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// mbar_wait for an item: the current one's share of the limit is read where
// the time is looked at, as the items' warp works it out behind the item.
__device__ __forceinline__ bool wait_item(uint32_t bar, uint32_t parity, unsigned long long* status, unsigned long long limit_ns,
                                          const volatile unsigned long long* item_ns)
{
    if (mbar_try(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    for (uint32_t i = 0;; ++i) {
        if (mbar_try(bar, parity)) return true;
        if ((i & 255u) == 255u && globaltimer() - t0 > limit_ns + *item_ns) {
            atomicOr(status, (unsigned long long)FADKV_DEV_TIMEOUT);
            return false;
        }
    }
}

// Shared-memory matrix descriptor of V [keys][d] as the B operand with d
// along the rows of 128 bytes (N-major, 128-byte swizzle): 8-key groups 1024
// bytes apart, 64-element halves of d one panel apart.
__device__ __forceinline__ uint64_t sdesc_n(uint32_t addr)
{
    uint64_t d = (uint64_t)((addr >> 4) & 0x3FFFu);
    d |= (uint64_t)((kKeys * 128u) >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

template <typename T> __host__ __device__ constexpr uint32_t idesc_of(int M, int N, bool b_n_major)
{
    const uint32_t t = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return idesc_f16(M, N) | (t << 7) | (t << 10) | (b_n_major ? 1u << 16 : 0u);
}

constexpr uint32_t kNegateA = 1u << 13;            // of the instruction descriptor

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 104;"); }

__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The key tiles of an item: those of the window (or all), then those of the
// first tokens, whose few keys would set a maximum that the next tile exceeds.
struct Tiles {
    int first, last, W, S, from, sinks, all, lo, count;     // count tiles of all from number lo on
    __device__ __forceinline__ Tiles(const Item& it, const PagedArgs& a)
    {
        first = it.first;
        last = it.first + it.nt - 1;
        W = a.p.window;        // below 2^31 - 4096 (the launcher); an item with keys to see begins at position -256 or later
        S = min(a.p.sinks, it.len);
        const int to = last >= 0 ? last / kKeys + 1 : 0;
        from = W > 0 ? max(0, first - W + 1) / kKeys : 0;
        sinks = W > 0 ? min(from, (S + kKeys - 1) / kKeys) : 0;
        count = all = to > from ? sinks + to - from : 0;
        lo = 0;
        if (it.parts > 1) {
            lo = count * it.piece / it.parts;
            count = count * (it.piece + 1) / it.parts - lo;
        }
    }
    __device__ __forceinline__ int key0(int i) const
    {
        i += lo;
        return (i < all - sinks ? i + from : i - (all - sinks)) * kKeys;
    }
    // whether some row of the item sees a key; whether a tile holds keys that none sees
    __device__ __forceinline__ bool seen(int key) const { return key <= last && (W == 0 || key > first - W || key < S); }
    __device__ __forceinline__ bool ragged(int k0) const
    {
        return !(k0 + kKeys - 1 <= last && (W == 0 || k0 > first - W || k0 + kKeys <= S));
    }
};

// Stage and parity of the ring's next entry.
template <int NST> struct Ring {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next()
    {
        if (++st == NST) {
            st = 0;
            ph ^= 1u;
        }
    }
};

// ROWS: keys and values are rows of their own (packed prompts), row i of a
// request its token i; no pages and no cached tokens.
template <typename T, int D, bool ROWS>
__global__ void __launch_bounds__(kPreThreads, 1)
paged_prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ PagedArgs a)
{
    using C = PreCfg<D>;
    constexpr int NST = C::NST, HALVES = D / 64, TILE = C::TILE;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t s_taddr;
    __shared__ Item s_item;
    __shared__ unsigned long long s_item_ns;           // what waits for the end of this item are given
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sQ = smem_u32(smem), sR = sQ + 2 * TILE, bar0 = sQ + C::bar_off;
    uint32_t* ok_ring = reinterpret_cast<uint32_t*>(smem + C::ok_off);   // [kOkRing][5]: all ok, four words of key bits
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (NST + s); };
    auto bar = [&](int k) { return bar0 + 8u * (2 * NST + k); };
    auto sfull = [&](int q) { return bar(q); };                 // scores are in TMEM
    auto sfree = [&](int q) { return bar(2 + q); };             // scores are in registers (d = 64)
    auto pvdone = [&](int q) { return bar(4 + q); };            // products with V are done
    auto ofree = [&](int q) { return bar(6 + q); };             // O has been read
    auto qfull = [&](int q) { return bar(8 + q); };
    auto qempty = [&](int q) { return bar(10 + q); };
    auto pfull = [&](int q, int part) { return bar(12 + 2 * q + part); };
    const uint32_t ifull = bar(16), iempty = bar(17), drained = bar(18);
    PreHead* head = reinterpret_cast<PreHead*>(a.ws);
    unsigned long long* status = &head->status;

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int grp = a.grp;
    const int gch = min(grp, kRows), chunks = (grp + gch - 1) / gch, tq = kRows / gch;   // heads and tokens per tile
    const int per_item = 2 * tq;

    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int q = 0; q < 2; ++q) {
            mbar_init(sfull(q), 1);
            mbar_init(sfree(q), 4);
            mbar_init(pvdone(q), 1);
            mbar_init(ofree(q), 4);
            mbar_init(qfull(q), 1);
            mbar_init(qempty(q), 1);
            mbar_init(pfull(q, 0), 4);
            mbar_init(pfull(q, 1), 4);
        }
        mbar_init(ifull, 1);
        mbar_init(iempty, kItemReaders);
        mbar_init(drained, 1);
        s_item_ns = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // (waits only: blocks of the join that are let in early slow the last pieces down: 84 tokens on 32768 43.1 against 40.6 us,
    // on 8192 23.4 against 21.5)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (ROWS && a.split == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // no join follows
    // the items' warp reads its first requests meanwhile: a lane each, its first row, its rows, its rows before T is cut
    // off, its tokens, its pairs of tiles
    int start = 0, cnt = 0, all = 0, my_len = 0, tiles = 0;
    auto look = [&](int hi) {
        const int b = hi - lane;
        cnt = start = all = my_len = 0;
        if (b >= 0) {
            start = __ldg(a.starts + b);
            const int stop = __ldg(a.starts + b + 1);
            if (start >= 0 && stop > start && start < a.p.T) {
                cnt = min(stop, a.p.T) - start;
                if (ROWS) {
                    all = cnt;
                    my_len = a.positions && __ldg(a.positions + start) < 0 ? 0 : cnt;
                } else {
                    all = stop - start;
                    my_len = length_of(b, start, a);
                }
            }
        }
        tiles = (cnt + per_item - 1) / per_item;
    };
    if (warp == 2) look(a.p.B - 1);
    if (warp == 3) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_taddr)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tbase = __shfl_sync(0xffffffffu, s_taddr, 0);

    bool ok = true;                                    // no wait of this warp has run out
    auto wait = [&](uint32_t b, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(b, parity, status, a.wait_ns));
        return ok;
    };
    // the n-th item of this CTA, read by a whole warp; false when there is none.  The TMA warp hands the slot back
    // only after its last load for the item: the next one is then taken, late enough for an even share of a short
    // list and early enough to be hidden behind the tiles in flight.
    auto next_item = [&](int n, Item& it) {
        ok = ok && __all_sync(0xffffffffu, wait_item(ifull, (uint32_t)n & 1u, status, a.wait_ns, &s_item_ns));
        if (!ok) return false;
        it = s_item;
        __syncwarp();
        if (warp != 0 && lane == 0) mbar_arrive(iempty);
        return it.live != 0;
    };

    // Registers: 168 a thread at launch (384 threads, 64512 in all); the four
    // service warps keep 104, the eight softmax warps take 200.
    if (warp == 0) {
        regs_dec();
        // ---------------- queries, K and V pages ----------------
        const int rows = min(1 << a.shift, kKeys), pages = kKeys / rows;   // at most 16
        const int row = lane * rows;                           // lane l holds page l of a tile
        const bool leader = elect_one();
        Ring<NST> ring;
        int issued = 0, gtile = 0, uses[2] = {0, 0};
        Item it;
        for (int n = 0; next_item(n, it); ++n) {
            const Tiles ts(it, a);
            const int tiles = ts.count, nq = it.nt > tq ? 2 : 1;
            auto page_of = [&](int i) {
                int page = a.p.num_pages;                      // outside the map: zeros
                if (ROWS) return 0;                            // (the rows of a tile are there, or behind the last one: zeros)
                if (i < tiles && lane < pages) {
                    const int key = ts.key0(i) + row;
                    // a page is asked for if any of its keys is seen: its first one (of the first tokens) or its last
                    if (key <= ts.last && (ts.seen(key) || ts.seen(min(key + rows - 1, ts.last))))
                        page = __ldg(a.table + (size_t)it.b * a.p.max_pages + (key >> a.shift));
                    if (page < 0 || page > a.p.num_pages) page = a.p.num_pages;
                }
                return page;
            };
            int page = page_of(0);
            for (int i = 0; i < tiles && ok; ++i, ++gtile) {
                const int k0 = ts.key0(i), next = page_of(i + 1);
                const uint32_t good = ROWS ? 0xffffffffu : __ballot_sync(0xffffffffu, page < a.p.num_pages || lane >= pages);
                for (int kv = 0; kv < 2; ++kv) {
                    if (!wait(empty(ring.st), ring.ph ^ 1u)) break;
                    if (lane == 0) {
                        if (kv == 0) {
                            uint32_t* o = ok_ring + (gtile & (kOkRing - 1)) * 5;
                            o[0] = good == 0xffffffffu;
                            if (good != 0xffffffffu) {
                                for (int w = 0; w < 4; ++w) {
                                    uint32_t bits = 0;
                                    for (int r = 0; r < 32; r += 8)
                                        if ((good >> ((w * 32 + r) / rows)) & 1u) bits |= 0xffu << r;
                                    o[1 + w] = bits;
                                }
                            }
                        }
                        mbar_expect_tx(full(ring.st), TILE);
                    }
                    __syncwarp();
                    const CUtensorMap* map = kv ? &map_v : &map_k;
                    const uint32_t dst = sR + ring.st * TILE;
                    if (ROWS) {
                        if (leader)
#pragma unroll
                            for (int h = 0; h < HALVES; ++h)
                                tma_load_3d(dst + h * (kKeys * 128), map, h * 64, it.hk, it.row0 - it.first + k0, full(ring.st));
                    } else {
                        const int y = k0 & ((1 << a.shift) - 1) & ~(rows - 1);
#pragma unroll 4
                        for (int j = 0; j < pages; ++j) {
                            const int w = __shfl_sync(0xffffffffu, page, j);
                            if (leader)
#pragma unroll
                                for (int h = 0; h < HALVES; ++h)
                                    tma_load_4d(dst + j * rows * 128 + h * (kKeys * 128), map, h * 64, y, it.hk, w, full(ring.st));
                        }
                    }
                    ring.next();
                    ++issued;
                    if (i == 0 && kv == 0)
                        for (int q = 0; q < nq; ++q) {
                            if (!wait(qempty(q), (uint32_t)(uses[q] & 1) ^ 1u)) break;
                            ++uses[q];
                            if (lane == 0) {
                                mbar_expect_tx(qfull(q), HALVES * gch * tq * 128);
                                for (int h = 0; h < HALVES; ++h)
                                    tma_load_3d(sQ + q * TILE + h * (kRows * 128), &map_q, h * 64, it.head0,
                                                it.row0 + q * tq, qfull(q));
                            }
                            __syncwarp();
                        }
                    if (!ok) break;
                }
                page = next;
            }
            if (lane == 0) mbar_arrive(iempty);
        }
        // drain: every issued load lands before the CTA exits
        for (int i = max(0, issued - NST); i < issued; ++i) mbar_wait(full(i % NST), (uint32_t)(i / NST) & 1u, status);
        for (int q = 0; q < 2; ++q)
            if (uses[q] > 0) mbar_wait(qfull(q), (uint32_t)(uses[q] - 1) & 1u, status);
    } else if (warp == 1) {
        regs_dec();
        // ---------------- products ----------------
        // The whole warp walks the tiles, so that descriptors and addresses stay in
        // uniform registers; one thread issues.  (With the walk in one thread alone
        // each product costs about 90 cycles to issue, against 64 to run.)
        constexpr uint32_t kPV = idesc_of<T>(kRows, D, true);
        const uint32_t kQK = idesc_of<T>(kRows, kKeys, false) | (a.p.scale < 0.f ? kNegateA : 0u);
        const bool leader = elect_one();
        Ring<NST> ring;
        int uses[2] = {0, 0}, qks[2] = {0, 0}, pvs[2] = {0, 0};   // items, score products, value products of a tile
        const uint64_t dq0 = sdesc(sQ), dr0 = sdesc(sR), dn0 = sdesc_n(sR);
        // descriptors count in 16 bytes: 32 bytes a step of 16 elements, a half of 64 elements one panel on
        auto qk = [&](int q, int stage) {
            const uint64_t dq = dq0 + (uint64_t)(q * (TILE >> 4)), dk = dr0 + (uint64_t)(stage * (TILE >> 4));
            if (leader) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t off = (uint64_t)(((k >> 2) * 128 * 128 + (k & 3) * 32) >> 4);
                    mma_ss(tbase + C::S(q), dq + off, dk + off, kQK, k > 0 ? 1u : 0u);
                }
                mma_commit(sfull(q));
            }
            ++qks[q];
        };
        // 16-key steps j0 .. j1-1
        auto pv = [&](int q, int stage, int j0, int j1, bool add) {
            const uint64_t dv = dn0 + (uint64_t)(stage * (TILE >> 4));
            if (leader)
#pragma unroll
                for (int j = j0; j < j1; ++j)
                    mma_ts(tbase + C::O(q), tbase + C::P(q) + j * 8, dv + (uint64_t)(j * 2048 >> 4), kPV,
                           add || j > 0 ? 1u : 0u);
        };
        // value rows that no row of the item sees: zeros (while the softmax works on the scores)
        auto clear = [&](const Tiles& ts, int k0, int stage) {
            unsigned char* v = smem + (2 + stage) * TILE;
            auto rows = [&](int r0, int r1) {                  // whole rows, so wherever the swizzle puts their pieces
                for (int x = r0 * (D / 8) + lane; x < r1 * (D / 8); x += 32) {
                    const int row = x / (D / 8), c = x % (D / 8);
                    *reinterpret_cast<uint4*>(v + (c / 8) * (kKeys * 128) + row * 128 + (c % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
            };
            rows(max(0, ts.last + 1 - k0), kKeys);
            if (ts.W > 0) rows(max(0, ts.S - k0), min(kKeys, ts.first - ts.W + 1 - k0));
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
        };
        // scores of the previous tile are in registers (with P over S: the wait for P says so)
        auto wait_s = [&](int q) {
            if (C::kOwnP && qks[q] > 0) wait(sfree(q), (uint32_t)(qks[q] - 1) & 1u);
        };
        Item it;
        for (int n = 0; next_item(n, it); ++n) {
            const Tiles ts(it, a);
            const int tiles = __shfl_sync(0xffffffffu, ts.count, 0);
            const int nq = __shfl_sync(0xffffffffu, it.nt > tq ? 2 : 1, 0);
            if (tiles == 0) continue;
            wait(full(ring.st), ring.ph);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (q >= nq || !ok) continue;
                wait(qfull(q), (uint32_t)uses[q] & 1u);
                wait_s(q);
                if (!ok) break;
                fence_after();
                qk(q, ring.st);
                if (tiles == 1 && leader) mma_commit(qempty(q));
            }
            if (!ok) break;
            if (leader) mma_commit(empty(ring.st));
            ring.next();
            for (int i = 0; i < tiles && ok; ++i) {
                const Ring<NST> rv = ring;
                ring.next();                               // now the next tile's K
                const bool more = i + 1 < tiles;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (q >= nq || !ok) continue;
                    if (C::kOwnP && more) {
                        if (q == 0) wait(full(ring.st), ring.ph);
                        wait_s(q);
                        if (!ok) break;
                        fence_after();
                        qk(q, ring.st);
                        if (i + 2 == tiles && leader) mma_commit(qempty(q));
                        if (q == nq - 1 && leader) mma_commit(empty(ring.st));
                    }
                    if (q == 0) {
                        if (wait(full(rv.st), rv.ph) && ts.ragged(ts.key0(i))) clear(ts, ts.key0(i), rv.st);
                    }
                    if (i == 0 && uses[q] > 0) wait(ofree(q), (uint32_t)(uses[q] - 1) & 1u);
                    wait(pfull(q, 0), (uint32_t)pvs[q] & 1u);
                    if (!ok) break;
                    fence_after();
                    pv(q, rv.st, 0, kPart / 16, i > 0);
                    if (!C::kOwnP && q == 0 && more) wait(full(ring.st), ring.ph);
                    wait(pfull(q, 1), (uint32_t)pvs[q] & 1u);
                    if (!ok) break;
                    fence_after();
                    pv(q, rv.st, kPart / 16, kKeys / 16, true);
                    if (leader) mma_commit(pvdone(q));
                    ++pvs[q];
                    if (q == nq - 1 && leader) mma_commit(empty(rv.st));
                    if (!C::kOwnP && more) {
                        qk(q, ring.st);
                        if (i + 2 == tiles && leader) mma_commit(qempty(q));
                        if (q == nq - 1 && leader) mma_commit(empty(ring.st));
                    }
                }
                if (more) ring.next();
            }
            for (int q = 0; q < nq; ++q) ++uses[q];
        }
        // drain: every product that was issued (after a wait that ran out that may be half of a tile's, which no other
        // barrier tells of) is complete before TMEM is freed
        if (leader) mma_commit(drained);
        mbar_wait(drained, 0u, status);
        __syncwarp();
    } else if (warp == 2) {
        regs_dec();
        // ---------------- items ----------------
        // Item x is heads x % heads of tile x / heads, tiles counted from the last
        // request's last one.  Requests are looked at 32 at a time, a lane each.
        // Several requests' tiles come in kLevels turns, those that see the most
        // keys first, so that the multiprocessors end together.
        const int heads = a.p.Hkv * chunks;
        const float inverse = 1.f / (float)per_item;
        int hi = a.p.B - 1;                                // lane l looks at request hi - l
        long long base = 0;                                // tiles before the requests looked at
        int level = 0, most = 0;                           // this turn (the last one: 0), the most keys of a tile
        int t0 = 0, upto = 0;                              // of this lane's request: its first tile of the turn, tiles up to and with it
        // how many of this lane's tiles come at this level or a later one: about those that see no more than so many keys
        // (they grow with the positions, up to a window's)
        auto below = [&](int lv) {
            const int keys = (int)((long long)most * lv / kLevels), f = my_len - all;
            if (f + cnt <= keys || (a.p.window > 0 && keys >= a.p.window)) return tiles;
            return max(0, min(tiles - 1, (int)((float)(keys - f) * inverse)));
        };
        auto turn = [&] {
            int t1 = tiles;
            t0 = 0;
            if (most > 0) {
                if (level < kLevels - 1) t1 = below(level + 1);
                if (level > 0) t0 = below(level);
            }
            upto = t1 - t0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
        };
        Item it;
        unsigned int parts = 1;
        const bool sorted = a.p.B > 1 && a.p.B <= kSorted;
        if (a.split || sorted) {
            // every CTA comes to the same number of parts, and to the same order
            long long items = 0;
            int longest = 0;
            for (;;) {
                items += __reduce_add_sync(0xffffffffu, tiles);
                if (cnt > 0) most = max(most, a.p.window > 0 ? min(my_len, a.p.window) : my_len);
                if (a.split && cnt > 0) {                      // the request's last item sees the most keys
                    const int t = (cnt - 1) / per_item * per_item;
                    it.parts = 1;
                    it.len = my_len;
                    it.first = my_len - all + t;
                    it.nt = cnt - t;
                    longest = max(longest, Tiles(it, a).count);
                }
                if (hi < 32) break;
                hi -= 32;
                look(hi);
            }
            if (hi != a.p.B - 1) {
                hi = a.p.B - 1;
                look(hi);
            }
            items *= heads;
            most = sorted && items > kPreCtas ? __reduce_max_sync(0xffffffffu, most) : 0;
            if (most > 0) level = kLevels - 1;
            if (a.split) {
                longest = __reduce_max_sync(0xffffffffu, longest);
                if (items > 0 && items <= kPreCtas)
                    parts = (unsigned int)max(1, min(min(kMaxParts, longest / kLeastTiles),
                                                     (items <= kPreCtas / 2 ? kPreCtas : kSplitSlots) / (int)items));
                if (blockIdx.x == 0 && lane == 0) {
                    head->parts = (int)parts;
                    head->items = (int)min(items, (long long)kPreCtas);
                }
            }
        }
        turn();
        for (int n = 0; ok; ++n) {
            // the first one by the CTA's number, the others from the counter
            unsigned int x = blockIdx.x;
            if (n > 0) {
                if (lane == 0) x = gridDim.x + atomicAdd(&head->taken, 1u);
                x = __shfl_sync(0xffffffffu, x, 0);
            }
            it.parts = (int)parts;
            it.piece = (int)(x % parts);
            it.index = (int)(x / parts);
            const long long u = it.index / heads;
            const int kvh = it.index % heads;
            while (hi >= 0 && u >= base + __shfl_sync(0xffffffffu, upto, 31)) {
                base += __shfl_sync(0xffffffffu, upto, 31);
                hi -= 32;
                if (hi < 0 && level > 0) {
                    --level;
                    hi = a.p.B - 1;
                }
                if (hi >= 0 && a.p.B > 32) look(hi);
                turn();
            }
            it.live = hi >= 0;
            const int at = hi >= 0 ? __ffs(__ballot_sync(0xffffffffu, base + upto > u)) - 1 : 0;   // the lane whose request it is
            const int t = __shfl_sync(0xffffffffu, t0, at) + (int)(base + __shfl_sync(0xffffffffu, upto, at) - u) - 1;
            const int rows = __shfl_sync(0xffffffffu, cnt, at), rows_all = __shfl_sync(0xffffffffu, all, at);
            const int s0 = __shfl_sync(0xffffffffu, start, at);
            it.len = __shfl_sync(0xffffffffu, my_len, at);
            if (it.live) {
                const int row = t * per_item;
                it.b = hi - at;
                it.row0 = s0 + row;
                it.nt = min(per_item, rows - row);
                // positions by the rows that the request has, those cut off at T included
                it.first = it.len - rows_all + row;
                it.hk = kvh / chunks;
                const int h0 = (kvh % chunks) * gch;
                it.head0 = it.hk * grp + h0;
                it.hn = min(gch, grp - h0);
            }
            if (lane == 0) {
                if (it.live && it.parts > 1 && it.piece == 0) {
                    head->item[it.index].row0 = it.row0;
                    head->item[it.index].nt = it.nt;
                    head->item[it.index].head0 = it.head0;
                    head->item[it.index].hn = it.hn;
                }
                s_item = it;
                mbar_arrive(ifull);
            }
            __syncwarp();
            if (!it.live) break;
            const unsigned long long item_ns = (unsigned long long)Tiles(it, a).count * a.tile_ns;
            if (lane == 0) s_item_ns = item_ns;
            ok = __all_sync(0xffffffffu, mbar_wait(iempty, (uint32_t)n & 1u, status, a.wait_ns + item_ns));
        }
        // the last CTA to stop leaves the counters at zero for the next call
        if (lane == 0) {
            __threadfence();
            if (atomicAdd(&head->left, 1u) == gridDim.x - 1) {
                head->taken = 0u;
                head->left = 0u;
            }
        }
    } else if (warp == 3) {
        regs_dec();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---------------- softmax ----------------
        const int q = (warp - 4) >> 2, r = tid & 127;
        const uint32_t inv_gch = 65536u / (uint32_t)gch + 1u;          // r / gch = r * inv_gch >> 16 for r < 128
        const int tr = (int)((r * inv_gch) >> 16), h = r - tr * gch;   // token and head of this thread's row
        const uint32_t lanes = tbase + ((uint32_t)((warp & 3) * 32) << 16);
        // positive, so that the largest score gives the largest exponent (a negative scale's sign is in the product);
        // in place of 0 a scale that leaves every exponent 0, as 0 x -inf would not
        const float scale = fmaxf(fabsf(a.scale_log2), 1e-37f);
        int gtile = 0, its = 0;                                        // tiles of all items; those of this half's
        Item it;
        for (int n = 0; next_item(n, it); ++n) {
            const Tiles ts(it, a);
            const int tiles = ts.count, gt0 = gtile;
            gtile += tiles;
            if (q == 1 && it.nt <= tq) continue;
            const int t = q * tq + tr;
            const bool live = tr < tq && t < it.nt && h < it.hn;
            const int pos = live ? it.first + t : -1;
            // the lowest and highest position among the warp's rows (no rows: nothing to mask)
            const int pmin = __reduce_min_sync(0xffffffffu, live ? pos : 0x3fffffff);
            const int pmax = __reduce_max_sync(0xffffffffu, live ? pos : -1);
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < tiles && ok; ++i, ++its) {
                const int k0 = ts.key0(i);
                const uint32_t* okr = ok_ring + ((gt0 + i) & (kOkRing - 1)) * 5;
                // masks only where some row of the warp does not see some key (worked out while the scores are on their way)
                const bool masked = !(k0 + kKeys - 1 <= pmin && (ts.W == 0 || k0 > pmax - ts.W || k0 + kKeys <= ts.S));
                if (!wait(sfull(q), (uint32_t)its & 1u)) break;
                fence_after();
                const bool all_ok = okr[0] != 0;
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_async(lanes + C::S(q) + c * 32, s[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_wait32(s[c]);
                if (C::kOwnP) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sfree(q));
                }
                if (masked || !all_ok) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int k = k0 + c * 32;
                        uint32_t bits = low_bits(pos - k + 1);
                        // (unsigned: wraps around for rows that see nothing)
                        if (ts.W > 0) bits &= ~low_bits((int)((uint32_t)(pos - k + 1) - (uint32_t)ts.W)) | low_bits(ts.S - k);
                        if (!all_ok) bits &= okr[1 + c];
                        if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!((bits >> j) & 1u)) s[c][j] = 0xff800000u;
                    }
                }
                float mx;
                {
                    float x[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        x[c] = fmaxf(__uint_as_float(s[c >> 1][(c & 1) * 16]), __uint_as_float(s[c >> 1][(c & 1) * 16 + 1]));
#pragma unroll
                    for (int j = 2; j < 16; j += 2)
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            x[c] = max3(x[c], __uint_as_float(s[c >> 1][(c & 1) * 16 + j]),
                                        __uint_as_float(s[c >> 1][(c & 1) * 16 + j + 1]));
                    mx = max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), fmaxf(x[6], x[7])) * scale;
                }
                const bool grow = mx > m + (kGrow + kBelow<T>);
                if (__any_sync(0xffffffffu, grow)) {
                    float f = 1.f;
                    if (grow) {
                        mx -= kBelow<T>;
                        f = exp2_fast(m - mx);
                        m = mx;
                        l *= f;
                    }
                    if (i > 0) {
                        if (!wait(pvdone(q), (uint32_t)(its - 1) & 1u)) break;
                        fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(lanes + C::O(q) + c * 32, o);
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st32(lanes + C::O(q) + c * 32, o);
                        }
                    }
                }
                const float mm = m == -INFINITY ? 0.f : m;     // nothing seen yet: every p is 0
                const uint64_t sc2 = pair(scale, scale), mm2 = pair(-mm, -mm);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float p0, p1;
                        unpair(fma2(pair(__uint_as_float(s[c][2 * j]), __uint_as_float(s[c][2 * j + 1])), sc2, mm2), p0, p1);
                        p0 = exp2_fast(p0);
                        p1 = exp2_fast(p1);
                        sum[j & 1] = add2(sum[j & 1], pair(p0, p1));
                        p[j] = Num<T>::pack(p0, p1);
                    }
                    // P in its own columns: the product that read the last one must be done (it is, mostly)
                    if (C::kOwnP && c == 0 && i > 0 && !wait(pvdone(q), (uint32_t)(its - 1) & 1u)) break;
                    tmem_st16(lanes + C::P(q) + c * 16, p);
                    if (c == kPart / 32 - 1 || c == 3) {       // the product may begin on these keys
                        tmem_st_wait();
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(pfull(q, c == 3));
                    }
                }
                if (!ok) break;
                float x0, x1;
                unpair(add2(sum[0], sum[1]), x0, x1);
                l += x0 + x1;
            }
            if (tiles > 0 && ok) {
                wait(pvdone(q), (uint32_t)(its - 1) & 1u);
                fence_after();
            }
            if (!ok) break;
            if (it.parts > 1) {
                // a piece: its sums, column by column, a lane a row
                float* part = reinterpret_cast<float*>((unsigned char*)a.ws + kHeadBytes) +
                              ((size_t)(it.index * it.parts + it.piece) * a.split + q) * slot_floats(D) + r;
                part[(size_t)D * kRows] = tiles > 0 ? m : -INFINITY;
                part[(size_t)(D + 1) * kRows] = l;
                if (tiles > 0) {
                    const bool any = __any_sync(0xffffffffu, live);
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(lanes + C::O(q) + c * 32, o);
                        if (any)
#pragma unroll
                            for (int j = 0; j < 32; ++j) part[(size_t)(c * 32 + j) * kRows] = __uint_as_float(o[j]);
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ofree(q));
                }
                continue;
            }
            const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
            if (live && a.lse)
                a.lse[(size_t)(it.row0 + t) * a.p.Hq + it.head0 + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            // rows out: four lanes exchange their 16-byte pieces, so that each stores 64 bytes of a row together
            T* orow[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int rr = (r & ~3) + k, tk = (int)((rr * inv_gch) >> 16), hh = rr - tk * gch, tt = q * tq + tk;
                orow[k] = tk < tq && tt < it.nt && hh < it.hn
                              ? (T*)a.out + (size_t)(it.row0 + tt) * a.p.out_stride + (size_t)(it.head0 + hh) * D + (lane & 3) * 8
                              : nullptr;
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (tiles > 0) {
                    tmem_ld32(lanes + C::O(q) + c * 32, o);
                    if (c == D / 32 - 1) {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(ofree(q));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0u;
                }
                uint32_t v[4][4];                              // [piece of the row][word]
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j >> 2][j & 3] = Num<T>::pack(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                // 4 x 4 transpose over the lanes of a quad: piece k of row j <-> piece j of row k
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const bool odd = lane & 1, high = lane & 2;
                    uint32_t x = __shfl_xor_sync(0xffffffffu, odd ? v[0][w] : v[1][w], 1);
                    uint32_t y = __shfl_xor_sync(0xffffffffu, odd ? v[2][w] : v[3][w], 1);
                    if (odd) v[0][w] = x, v[2][w] = y;
                    else v[1][w] = x, v[3][w] = y;
                    x = __shfl_xor_sync(0xffffffffu, high ? v[0][w] : v[2][w], 2);
                    y = __shfl_xor_sync(0xffffffffu, high ? v[1][w] : v[3][w], 2);
                    if (high) v[0][w] = x, v[1][w] = y;
                    else v[2][w] = x, v[3][w] = y;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (orow[k]) *reinterpret_cast<uint4*>(orow[k] + c * 32) = make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
            }
        }
        if (!ok) tmem_st_wait();                       // drain: as above, but that nothing waited for these
    }

    fence_before();
    __syncthreads();
    if (warp == 3) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512));
    }
}

// Joins the pieces of cut items: a block takes 8 columns of a tile's 128 rows.
template <typename T, int D>
__global__ void __launch_bounds__(kRows)
paged_prefill_join_kernel(const __grid_constant__ PagedArgs a)
{
    // (waits only: a dependent let in early would take the registers that the other blocks of this grid need)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PreHead* head = reinterpret_cast<const PreHead*>(a.ws);
    const int parts = head->parts, item = blockIdx.x / a.split, q = blockIdx.x % a.split;
    if (parts <= 1 || item >= head->items) return;
    const int gch = min(a.grp, kRows), tq = kRows / gch, r = threadIdx.x, t = q * tq + r / gch, h = r % gch;
    const int row0 = head->item[item].row0, head0 = head->item[item].head0;
    if (r / gch >= tq || t >= head->item[item].nt || h >= head->item[item].hn) return;
    if (row0 < 0 || row0 + t >= a.p.T || head0 < 0 || head0 + h >= a.p.Hq) return;   // (after a wait that ran out)
    const size_t step = slot_floats(D) * a.split;
    const float* part = reinterpret_cast<const float*>((const unsigned char*)a.ws + kHeadBytes) +
                        ((size_t)item * parts * a.split + q) * slot_floats(D) + r;
    const int c0 = blockIdx.y * 8;
    float m = -INFINITY, l = 0.f, o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = 0.f;
    // eight pieces at a time, all their loads in flight; past the last one the last one again, with weight 0
    for (int p0 = 0; p0 < parts; p0 += 8) {
        float pm[8], pl[8], v[8][8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const float* at = part + min(p0 + p, parts - 1) * step;
            pm[p] = at[(size_t)D * kRows];
            pl[p] = at[(size_t)(D + 1) * kRows];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[p][j] = at[(size_t)(c0 + j) * kRows];
        }
        float top = m;
#pragma unroll
        for (int p = 0; p < 8; ++p) top = fmaxf(top, pm[p]);
        const float g = m == -INFINITY ? 0.f : exp2_fast(m - top);
        m = top;
        l *= g;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] *= g;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            // a piece that saw nothing of this row may have left its columns unwritten
            const float f = pm[p] == -INFINITY || p0 + p >= parts ? 0.f : exp2_fast(pm[p] - m);
            if (f > 0.f) {
                l = fmaf(f, pl[p], l);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = fmaf(f, v[p][j], o[j]);
            } else if (pl[p] != pl[p]) {
                l = pl[p];
            }
        }
    }
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    const size_t row = (size_t)row0 + t, hd = (size_t)head0 + h;
    *reinterpret_cast<uint4*>((T*)a.out + row * a.p.out_stride + hd * D + c0) =
        make_uint4(Num<T>::pack(o[0] * inv, o[1] * inv), Num<T>::pack(o[2] * inv, o[3] * inv),
                   Num<T>::pack(o[4] * inv, o[5] * inv), Num<T>::pack(o[6] * inv, o[7] * inv));
    if (c0 == 0 && a.lse) a.lse[row * a.p.Hq + hd] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// A pool as (element, token in page, head, page), boxes of 64 elements by up
// to 128 tokens of one page and head.
bool pool_map(CUtensorMap* map, const void* base, const PagedArgs& a)
{
    auto fn = tma_encode_fn();
    if (!fn) return false;
    const fadkv_paged_params& p = a.p;
    cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.page_size, (cuuint64_t)p.Hkv, (cuuint64_t)p.num_pages};
    cuuint64_t strides[3] = {(cuuint64_t)p.token_stride * 2, (cuuint64_t)p.head_stride * 2, (cuuint64_t)p.page_stride * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)(p.page_size < kKeys ? p.page_size : kKeys), 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, p.dtype == FADKV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows as (element, head, row).  Queries: boxes of 64 elements by the heads
// and tokens of a tile, row by row as the tile has them; keys and values of
// prompts: of one head and a tile's rows.
bool row_map(CUtensorMap* map, const PagedArgs& a, const void* base, int all, int64_t row, int heads, int tokens)
{
    auto fn = tma_encode_fn();
    if (!fn) return false;
    const fadkv_paged_params& p = a.p;
    cuuint64_t dims[3] = {(cuuint64_t)p.d, (cuuint64_t)all, (cuuint64_t)p.T};
    cuuint64_t strides[2] = {(cuuint64_t)p.d * 2, (cuuint64_t)row * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, p.dtype == FADKV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct PreShape {
    int gch, chunks, tq;       // heads of a tile, tiles a KV head's group takes, tokens of a tile
    long long items;           // at most
    int split;                 // 0: items are not cut; else the tiles of an item that can hold rows
};

// Whether a call of B requests whose rows fill `items` items at least may cut them.  Cutting can pay only if they are fewer than
// the multiprocessors, however the rows are spread over requests, and if there can be keys for two pieces.  How many pieces
// there are is decided on the device.  (What fewer requests and items, more rows and keys take from a yes is never a no.)
bool may_cut(const fadkv_paged_params& p, bool rows, int B, long long items)
{
    long long most = (long long)p.max_pages * p.page_size;
    if (p.window > 0) most = most < (long long)p.window + p.sinks + 2 * kKeys ? most : (long long)p.window + p.sinks + 2 * kKeys;
    if (B > 256 || items > kPreCtas || most < 2 * kLeastTiles * kKeys) return false;
    if (!rows) return true;
    // Prompts: T bounds the keys, mostly from far above, so the longest prompt is taken for twice the mean.  Cutting saves
    // its key tiles' time (1.2 us each) but for items / 152 of it, and the pieces and their join cost some 10 us (8 heads over
    // 1 of 128, 1500 tokens in 47 items: 21.2 us cut and 21.7 whole; 8 over 2, 1100 in 36: 23.5 and 20.2; 24 over 8, 1100
    // in 112: 33 and 19; one head, 4000 in 16: 18 and 50).
    const long long keys = std::min(std::min(most, (long long)p.T), 2ll * p.T / std::max(B, 1));
    return 3 * items <= kPreCtas && keys / kKeys * (kPreCtas - items) >= 1300;
}

PreShape pre_shape(const fadkv_paged_params& p, bool rows)
{
    PreShape s;
    const int grp = p.Hq / p.Hkv;
    s.gch = grp < kRows ? grp : kRows;
    s.chunks = (grp + s.gch - 1) / s.gch;
    s.tq = kRows / s.gch;
    const long long heads = (long long)p.Hkv * s.chunks, tiles = p.T / (2 * s.tq);
    s.items = (tiles + (p.B < p.T ? p.B : p.T)) * heads;           // one more a request than its rows fill
    s.split = !may_cut(p, rows, p.B, (tiles + 1) * heads) ? 0 : (p.T <= s.tq ? 1 : 2);
    return s;
}

template <typename T, int D, bool ROWS>
cudaError_t launch_rows(const PagedArgs& args, cudaStream_t st)
{
    auto k = paged_prefill_kernel<T, D, ROWS>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, PreCfg<D>::alloc);
    if (e != cudaSuccess) return e;
    PagedArgs a = args;
    const PreShape s = pre_shape(a.p, ROWS);
    a.split = s.split;
    if (a.p.window >= a.p.max_pages << a.shift) a.p.window = 0;   // hides nothing
    a.tile_ns = a.wait_ns ? 0 : kTileNs;               // (a test's limit is the whole limit)
    a.wait_ns = a.wait_ns ? a.wait_ns : kWaitNs;
    CUtensorMap mq, mk, mv;
    if (!row_map(&mq, a, a.q, a.p.Hq, a.p.q_stride, s.gch, s.tq)) return cudaErrorInvalidValue;
    if (ROWS ? !row_map(&mk, a, a.k, a.p.Hkv, a.k_row, 1, kKeys) || !row_map(&mv, a, a.v, a.p.Hkv, a.v_row, 1, kKeys)
             : !pool_map(&mk, a.k, a) || !pool_map(&mv, a.v, a))
        return cudaErrorInvalidValue;
    if (s.items > 0x7fffffffll) return cudaErrorInvalidValue;
    const int ctas = s.split || s.items > kPreCtas ? kPreCtas : (int)s.items;
    e = launch_pdl(k, dim3(ctas), dim3(kPreThreads), PreCfg<D>::alloc, st, mq, mk, mv, a);
    if (e != cudaSuccess || !s.split) return e;
    const int items = (int)(s.items < kPreCtas ? s.items : kPreCtas);
    return launch_pdl(paged_prefill_join_kernel<T, D>, dim3(items * s.split, D / 8), dim3(kRows), 0, st, a);
}

template <typename T, int D>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t st, bool rows)
{
    return rows ? launch_rows<T, D, true>(a, st) : launch_rows<T, D, false>(a, st);
}

}  // namespace

size_t paged_prefill_workspace(const fadkv_paged_params& p, bool rows)
{
    return kHeadBytes + (size_t)kSplitSlots * pre_shape(p, rows).split * slot_floats(p.d) * sizeof(float);
}

size_t paged_prefill_workspace_most(const fadkv_paged_params& p, bool rows)
{
    const PreShape s = pre_shape(p, rows);
    const bool cut = p.B > 0 && may_cut(p, rows, 1, (long long)p.Hkv * s.chunks);
    return kHeadBytes + (size_t)kSplitSlots * (!cut ? 0 : p.T <= s.tq ? 1 : 2) * slot_floats(p.d) * sizeof(float);
}

cudaError_t launch_paged_prefill(const PagedArgs& a, cudaStream_t st, bool rows)
{
    if (a.p.B <= 0 || a.p.T <= 0) return cudaSuccess;
    if (a.p.dtype == FADKV_F16) return a.p.d == 128 ? launch_t<__half, 128>(a, st, rows) : launch_t<__half, 64>(a, st, rows);
    return a.p.d == 128 ? launch_t<__nv_bfloat16, 128>(a, st, rows) : launch_t<__nv_bfloat16, 64>(a, st, rows);
}

}  // namespace fadkv
